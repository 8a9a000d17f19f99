"""Calls of a tree-drafted step that its documentation allows or refuses, beside the operators' own tests."""
import pytest
import torch

from test_gpu_tree import Tree, kvc  # noqa: F401  (kvc is a fixture)

pytestmark = pytest.mark.gpu


def test_a_workspace_among_the_tensors_of_its_call_is_refused(kvc):
    w = Tree(30, [30000], [4], 4, 4, 2, 64)
    w.run(kvc)
    d = w.d
    need = kvc.paged_decode_tree_plan(1, 4, 2, 64, w.max_ctx, 4)
    assert need > 0
    room = torch.zeros(need + 4096, dtype=torch.uint8, device="cuda")
    q = room[need - 512:need - 512 + d["q"].numel() * 2].view(torch.float16).view_as(d["q"])
    out = room[:w.out.numel() * 2].view(torch.float16).view_as(w.out)
    args = lambda q, out: (q, d["k"], d["v"], d["table"], d["ctx"], d["masks"], w.scale, out, room[:need], w.max_ctx)  # noqa: E731
    for a in (args(q, w.out), args(d["q"], out)):
        with pytest.raises(kvc.KvcError, match="overlaps") as e:
            kvc.paged_decode_tree_attention(*a)
        assert e.value.name == "KVC_ERR_INVALID"
    got = room[need:need + w.out.numel() * 2].view(torch.float16).view_as(w.out)  # behind it
    kvc.paged_decode_tree_attention(*args(d["q"], got))
    assert torch.equal(got, w.out)
