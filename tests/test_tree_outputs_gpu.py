"""Outputs that the tree calls make are tensors of their own: one that is resized
leaves the others as they are."""
import pytest
import torch

from test_tree_calls_gpu import _arguments, _call, _slow

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("way", ["compiled", "checked"])
@pytest.mark.parametrize("name", ["rope", "mask", "attend", "accept", "logprobs"])
def test_a_resized_output_leaves_the_others(name, way):
    out = _call(name, _arguments(name), **({} if way == "compiled" else _slow(name)))
    outs = list(out) if isinstance(out, tuple) else [out]
    for t in outs:
        assert t.storage_offset() == 0 and t.untyped_storage().nbytes() == t.numel() * t.element_size()
    for i, t in enumerate(outs):
        want = [o.clone() for o in outs]
        t.resize_(t.numel() * 3 + 500)
        t.view(torch.uint8).fill_(0xA5)
        t.resize_(want[i].shape)
        assert all(torch.equal(o.view(torch.uint8), w.view(torch.uint8)) for j, (o, w) in enumerate(zip(outs, want)) if j != i)
