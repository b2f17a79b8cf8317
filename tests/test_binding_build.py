"""How the compiled module of the tree calls is built and found, without a GPU."""
import os
import subprocess
import threading
import time
import types

import pytest
import torch

import block_sparse_attention_prefill_gb300 as msa
from block_sparse_attention_prefill_gb300 import build, tree


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


@pytest.fixture
def no_compiler(monkeypatch):
    def fails(*args, **kw):
        raise FileNotFoundError("g++")

    monkeypatch.setattr(tree, "_binding", None)
    monkeypatch.setattr(tree, "_way", None)
    monkeypatch.setattr(build, "build_binding", fails)


def test_calls_do_without_the_module(no_compiler):
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    with pytest.warns(RuntimeWarning, match="could not be built"):
        with pytest.raises(msa.MsaError, match="CUDA tensors"):
            msa.msa_tree_mask(i32(6), i32(3), i32(3), 6)
    with pytest.raises(msa.MsaError, match="CUDA tensors"):  # (no second warning)
        msa.msa_logprobs(torch.zeros((4, 50)), i32(4))
    with pytest.raises(OSError):  # asked for by name it is missed
        msa.load_binding()


@pytest.mark.gpu
@pytest.mark.filterwarnings("ignore:the tree calls")
@pytest.mark.parametrize("name", ["rope", "rope4", "mask", "attend", "accept", "accept4", "logprobs"])
def test_calls_without_the_module_give_the_same(name, monkeypatch):
    from test_tree_calls_gpu import _all, _arguments, _call, _same

    args = _arguments(name)
    want = _all(_call(name, args), args)
    monkeypatch.setattr(tree, "_way", tree._Checked)
    args = _arguments(name)
    assert _same(_all(_call(name, args), args), want)
