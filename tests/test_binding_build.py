"""How the compiled module of the tree calls is built and found, without a GPU."""
import os
import subprocess
import threading
import time
import types

import block_sparse_attention_prefill_gb300 as msa
from block_sparse_attention_prefill_gb300 import build


def test_threads_that_ask_at_once_compile_once(monkeypatch, tmp_path):
    path, running, runs = str(tmp_path / "module.so"), [], []

    def compile(cmd, **kw):
        out = cmd[cmd.index("-o") + 1]
        assert not running, "two compilers at once"
        running.append(out)
        with open(out, "w") as f:
            f.write("half")
            f.flush()
            time.sleep(0.2)
            f.write(" and half")
        running.pop()
        runs.append(out)
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(build, "binding_path", lambda: path)
    monkeypatch.setattr(subprocess, "run", compile)
    got, errors = [], []

    def ask():
        try:
            got.append(build.build_binding())
            with open(path) as f:
                assert f.read() == "half and half"
        except BaseException as e:
            errors.append(e)

    threads = [threading.Thread(target=ask) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    assert got == [path] * 4 and len(runs) == 1 and os.listdir(tmp_path) == ["module.so"]


def test_threads_get_one_module():
    got = []
    threads = [threading.Thread(target=lambda: got.append(msa.load_binding())) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(got) == 4 and all(m is got[0] for m in got)
