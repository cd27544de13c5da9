"""A call that runs longer than the limit of any one wait inside it (4 s)."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def test_a_share_of_whole_blocks_longer_than_a_wait(dtlib):
    """1400 requests of 2^24 tokens on one shared page of 256 and, at the end of the last CTA's share, the first that ends
    inside a block: the warps that clean its values have had nothing to do for seconds.

    Every output is the softmax over the page, to within the roundings of weights and output (2^-8 each of the values'
    size) and of sums over a CTA's part of a request (131072 blocks: one addition and 16 product steps a block, 2^-23
    each; a cancelling half of the values is taken at its worst)."""
    B, Hkv, d, page, T = 1400, 8, 64, 256, 1 << 24
    g = torch.Generator(device="cuda").manual_seed(1)
    kc = torch.zeros(1, Hkv, page, d, dtype=BF, device="cuda")
    vc = torch.randint(1, 9, (1, Hkv, page, d), generator=g, device="cuda").to(BF)
    q = torch.ones(B, 1, Hkv, d, dtype=BF, device="cuda")
    table = torch.zeros(B, T // page, dtype=torch.int32, device="cuda")
    lens = torch.full((B,), T, dtype=torch.int32, device="cuda")
    lens[-1] = T - 1
    ws = dtlib.new_workspace(dtlib.dt_paged_attention_workspace_bytes(B, 1, Hkv, Hkv, d))
    out = torch.full_like(q, float("nan"))
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    dtlib.dt_paged_attention(q, kc, vc, table, lens, 0.125, out=out, workspace=ws)
    end.record()
    assert dtlib.dt_get_error(ws) == dtlib.Status.OK
    print(f"{start.elapsed_time(end):.0f} ms")
    want = vc[0].double().mean(1)
    assert ((out[:, 0].double() / want - 1).abs() <= 2 * 2.0 ** -8 + 17 * 131072 * 2.0 ** -23).all()
