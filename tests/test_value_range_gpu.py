"""Values of up to 10^30 give finite outputs, however long the sequence and however far the scores of its later keys
exceed those of its first: the weights' sums times the values stay below fp32's largest number."""
import math

import pytest
import torch

import test_paged_attn_gpu as paged
import test_prompt_attn_gpu as prompt

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("growth", [0.0, 12.0, 19.9, 21.5, 40.0])
@pytest.mark.parametrize("size", [1e30, 1e-28])
def test_values_of_a_prompt(dtlib, d, growth, size):
    """All values of one sign; every key behind the first block scores higher by 2^growth."""
    s = prompt.make([4500], 2, 1, d, fused=False, spread=0.1)
    s["q"][..., 0], s["k"][..., 0] = 4.0, 0.0
    s["k"][128:, :, 0] = growth * math.log(2) / 4 / s["scale"]
    s["v"].copy_((0.5 + 0.5 * torch.rand(s["v"].shape, device="cuda")) * size)
    prompt.parity(dtlib, s, rows=[0, 127, 128, 255, 256, 300, 1000, 2047, 4095, 4498, 4499])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("size", [1e30, 1e-28])
def test_values_over_the_longest_cache(dtlib, d, size):
    """2^24 tokens (one page many times over), all of one value but the first page's, whose keys score lower by 2^19.9.
    The output is that value: off by the weights' rounding and the output's (2^-8 each), by sums of a CTA's share of 863
    blocks (11 and then one addition a block of the weights; 8 products a block of the outputs, two steps each, of
    2^-23) and by 152 parts joined (three steps of 2^-22 each)."""
    page, T = 256, 1 << 24
    kc, vc = (torch.zeros(2, 1, page, d, dtype=BF, device="cuda") for _ in range(2))
    kc[1, ..., 0] = 19.9 * math.log(2) / 4
    vc[1], vc[0] = size, -size
    q = torch.zeros(1, 1, 2, d, dtype=BF, device="cuda")
    q[..., 0] = 4.0
    table = torch.ones(1, T // page, dtype=torch.int32, device="cuda")
    table[0, 0] = 0
    lens = torch.tensor([T], dtype=torch.int32, device="cuda")
    ws = dtlib.new_workspace(dtlib.dt_paged_attention_workspace_bytes(1, 1, 2, 1, d))
    out = dtlib.dt_paged_attention(q, kc, vc, table, lens, 1.0, workspace=ws)
    assert dtlib.dt_get_error(ws) == dtlib.Status.OK
    want = float(torch.tensor(size, dtype=BF))
    off = 2 * 2.0 ** -8 + (11 + 863) * 2.0 ** -23 + 16 * 863 * 2.0 ** -23 + 3 * 152 * 2.0 ** -22
    assert ((out.double() / want - 1).abs() <= off).all(), (out.double() / want - 1).abs().max()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("size", [1e30, 1e-28])
def test_values_of_tree_nodes(dtlib, d, size):
    s = paged.make([2000, 300, 16], 16, 8, 2, d, 16, mask="tree", spread=0.1)
    s["vc"] *= size / 8
    s["vc"].clamp_(-size, size)
    paged.parity(dtlib, s)
