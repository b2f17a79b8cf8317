"""The tree calls that write pools, on another stream than the current one, and
on two streams at once with pools of their own."""
import pytest
import torch

import block_sparse_attention_prefill_gb300 as msa
from test_tree_calls_gpu import _all, _arguments, _call, _same

pytestmark = pytest.mark.gpu

NAMES = ["rope", "rope4", "accept", "accept4"]


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("name", NAMES)
def test_pools_written_on_another_stream(name, raw):
    args = _arguments(name)
    want = _all(_call(name, args), args)
    if name.startswith("accept"):  # rows are moved
        before = _arguments(name)["kv"]
        assert not all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(args["kv"], before))
    side = torch.cuda.Stream()
    for current in (False, True):
        args = _arguments(name)
        torch.cuda.synchronize()
        if current:
            with torch.cuda.stream(side):
                out = _call(name, args)
        else:
            out = _call(name, args, stream=side.cuda_stream if raw else side)
        side.synchronize()
        assert _same(_all(out, args), want)


def test_two_streams_at_once():
    want = {}
    for name in NAMES:
        args = _arguments(name)
        want[name] = _all(_call(name, args), args)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        args = [{name: _arguments(name) for name in NAMES} for _ in streams]
        torch.cuda.synchronize()
        got = [{} for _ in streams]
        for name in NAMES:
            for i, s in enumerate(streams):
                with torch.cuda.stream(s):
                    got[i][name] = _call(name, args[i][name])
        torch.cuda.synchronize()
        for i in range(len(streams)):
            for name in NAMES:
                assert _same(_all(got[i][name], args[i][name]), want[name])
