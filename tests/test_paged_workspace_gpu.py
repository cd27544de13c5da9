"""The workspaces of the paged cache's operators: what they have to hold before a call, and which calls share one."""
import pytest
import torch

import test_paged_attn_gpu as paged
import test_prompt_attn_gpu as prompt

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def cut_pairs():
    """Requests whose pairs are split over several CTAs and joined."""
    return paged.make([3000, 129, 1500], 2, 8, 2, 128, 16, mask="tree")


def room(dtlib, s):
    B, n, Hq, d = s["q"].shape
    return dtlib.dt_paged_attention_workspace_bytes(B, n, Hq, s["kc"].shape[1], d)


def test_only_a_workspace_s_header_has_to_be_zero(dtlib):
    s = cut_pairs()
    want = paged.run(dtlib, s).clone()
    for fill in (0xFF, 0x01, 0x7F):
        ws = dtlib.new_workspace(room(dtlib, s))
        ws[256:] = fill
        for _ in range(2):
            out = torch.full_like(want, float("nan"))
            paged.run(dtlib, s, out=out, workspace=ws)
            assert torch.equal(out, want)
        assert dtlib.dt_get_error(ws) == dtlib.Status.OK
        assert (ws[:256] == 0).all()  # left as it has to be found


def test_a_workspace_that_the_tree_attention_used(dtlib):
    """The verify pass over a dense cache and over pages, turn by turn, on one workspace."""
    s = cut_pairs()
    g = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *shape: torch.randn(*shape, generator=g, device="cuda").to(BF)
    B, n, L, Hq, Hkv, d = 2, 8, 3000, 32, 8, 128
    q, k, v = rnd(B, n, Hq, d), rnd(B, Hkv, L + n, d), rnd(B, Hkv, L + n, d)
    mask = torch.eye(n, dtype=torch.uint8, device="cuda").repeat(B, 1, 1)
    p = prompt.make([300, 700], 8, 2, 64)
    tree = lambda **kw: dtlib.dt_tree_attention(q, k, v, mask, 0.1, **kw)
    want = tree().clone(), paged.run(dtlib, s).clone(), prompt.run(dtlib, p).clone()
    ws = dtlib.new_workspace(max(dtlib.dt_tree_attention_workspace_bytes(B, n, L, Hq, Hkv, d), room(dtlib, s)))
    for _ in range(3):
        assert torch.equal(tree(workspace=ws), want[0])
        assert torch.equal(paged.run(dtlib, s, workspace=ws), want[1])
        assert torch.equal(prompt.run(dtlib, p, workspace=ws), want[2])
    assert dtlib.dt_get_error(ws) == dtlib.Status.OK
