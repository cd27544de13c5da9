"""The paged cache's operators together with others of their kind and at the ends of their envelope: calls at the same
time on two streams, two captured graphs on one workspace, nothing to do, the most requests and heads, tables without a
spare entry, rows past 2^31 elements. Against attention in 64 bits as in the operators' own tests."""
import math

import pytest
import torch

import test_paged_attn_gpu as paged
import test_prompt_attn_gpu as prompt
from attention_ref import attend, check

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def test_two_calls_at_the_same_time(dtlib):
    """Two streams, a workspace each: the results are those of the calls alone, time after time."""
    a = paged.make([3000, 17, 900, 4], 4, 16, 4, 128, 16, mask="tree")
    b = paged.make([500] * 40, 1, 16, 4, 64, 32, mask=None, seed=6)
    c, d = prompt.make([700, 33, 1500], 8, 2, 128), prompt.make([64] * 30, 4, 4, 64, seed=8)
    calls = [lambda kw: paged.run(dtlib, a, **kw), lambda kw: paged.run(dtlib, b, **kw),
             lambda kw: prompt.run(dtlib, c, **kw), lambda kw: prompt.run(dtlib, d, **kw)]
    room = max(dtlib.dt_paged_attention_workspace_bytes(4, 4, 16, 4, 128),
               dtlib.dt_paged_attention_workspace_bytes(40, 1, 16, 4, 64))
    want = [call({}).clone() for call in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    spaces = [dtlib.new_workspace(room) for _ in calls]
    outs = [torch.empty_like(w) for w in want]
    torch.cuda.synchronize()
    for _ in range(20):
        for out in outs:
            out.fill_(float("nan"))
        torch.cuda.synchronize()
        for _ in range(3):
            for call, s, ws, out in zip(calls, streams, spaces, outs):
                call(dict(out=out, workspace=ws, stream=s))
        torch.cuda.synchronize()
        for out, w in zip(outs, want):
            assert torch.equal(out, w)
    assert all(dtlib.dt_get_error(ws) == dtlib.Status.OK for ws in spaces)


def test_two_graphs_on_one_workspace(dtlib):
    """Captured apart, replayed in turn: each call leaves the workspace ready for the other's."""
    a = paged.make([300, 2000], 2, 8, 2, 128, 16, mask="tree")
    b = prompt.make([400, 900], 8, 2, 64)
    want = [paged.run(dtlib, a).clone(), prompt.run(dtlib, b).clone()]
    ws = dtlib.new_workspace(dtlib.dt_paged_attention_workspace_bytes(2, 2, 8, 2, 128))
    outs = [torch.empty_like(w) for w in want]
    calls = [lambda: paged.run(dtlib, a, out=outs[0], workspace=ws),
             lambda: prompt.run(dtlib, b, out=outs[1], workspace=ws)]
    graphs, side = [], torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for call in calls:
        with torch.cuda.stream(side):
            call()
        side.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            call()
            call()
        graphs.append(g)
    for _ in range(5):
        for out in outs:
            out.fill_(float("nan"))
        for g in graphs + graphs[::-1]:
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out, w) for out, w in zip(outs, want))


def test_nothing_to_do(dtlib):
    s = paged.make([30, 20], 2, 8, 2, 64, 16, mask="tree")
    empty = dtlib.dt_paged_attention(s["q"][:0], s["kc"], s["vc"], s["table"][:0], s["lens"][:0], 0.1,
                                     mask=s["mask"][:0])
    assert empty.shape == (0, 2, 8, 64)
    p = prompt.make([30], 4, 2, 64)
    assert dtlib.dt_prompt_attention(p["q"][:0], p["k"][:0], p["v"][:0], p["cu"][:1] * 0, 0.1).shape == (0, 4, 64)
    out = torch.full((30, 4, 64), 7.0, dtype=BF, device="cuda")
    dtlib.dt_prompt_attention(p["q"], p["k"], p["v"], p["cu"][:1], 0.1, out=out)  # rows, but no prompt
    torch.cuda.synchronize()
    assert (out == 7).all()


def test_a_table_without_a_spare_entry(dtlib):
    s = paged.make([64, 128, 127], 1, 8, 2, 128, 16, mask=None)
    s["table"] = s["table"][:, :8].contiguous()
    paged.parity(dtlib, s)
    s = paged.make([16, 7], 3, 8, 2, 64, 16, mask="tree")
    s["table"] = s["table"][:, :1].contiguous()
    paged.parity(dtlib, s)


def test_the_most_requests(dtlib):
    lens = [(13 * i) % 200 if i % 7 else 0 for i in range(2048)]
    paged.parity(dtlib, paged.make(lens, 1, 4, 2, 64, 16, mask=None), requests=[0, 1, 6, 7, 8, 1000, 2046, 2047])


@pytest.mark.parametrize("Hq,Hkv", [(256, 256), (256, 2), (128, 1)])
def test_the_most_heads(dtlib, Hq, Hkv):
    paged.parity(dtlib, paged.make([300, 5], 1, Hq, Hkv, 128, 16, mask=None), heads=[0, 1, Hq // 2, Hq - 1])
    prompt.parity(dtlib, prompt.make([140, 300], Hq, Hkv, 64), heads=[0, 1, Hq // 2, Hq - 1])


@pytest.mark.parametrize("d", [64, 128])
def test_large_values_under_growing_scores(dtlib, d):
    """Values of 10^30 under scores that grow along the sequence by less than what raises the running maximum at once:
    the weights above the first block's maximum times the values stay finite."""
    grow = lambda n: torch.linspace(0, 2, n, device="cuda")[:, None, None]
    s = prompt.make([900], 4, 2, d, fused=False, spread=0.02)
    s["q"][..., 0], s["k"][..., 0] = 4.0, (grow(900) * math.sqrt(d))[..., 0].to(BF)
    s["v"] *= 1e30
    prompt.parity(dtlib, s)
    p = paged.make([1500, 300], 2, 8, 2, d, 16, mask="tree", spread=0.02)
    p["q"][..., 0] = 4.0
    for b in range(2):
        n = int(p["lens"][b])
        for i in range(-(-n // 16)):
            p["kc"][p["table"][b, i].long(), :, :, 0] = float(grow(n)[16 * i] * math.sqrt(d))
            p["vc"][p["table"][b, i].long()] *= 1e30
    paged.parity(dtlib, p)


def test_prompt_rows_past_two_to_the_31_elements(dtlib):
    n, count, Hq, Hkv, d = 5000, 108, 32, 1, 128
    total = n * count
    assert total * Hq * d > 2 ** 31
    q, k, v = (torch.zeros(total, h, d, dtype=BF, device="cuda") for h in (Hq, Hkv, Hkv))
    g = torch.Generator(device="cuda").manual_seed(2)
    for x in (q, k, v):
        x[-n:] = torch.randn(n, x.shape[1], d, generator=g, device="cuda").to(BF)
    cu = torch.arange(0, total + 1, n, dtype=torch.int32, device="cuda")
    out = dtlib.dt_prompt_attention(q, k, v, cu, 1 / math.sqrt(d))
    rows = torch.tensor([0, 1, 2499, n - 1], device="cuda")
    seen = torch.arange(n, device="cuda") <= rows[:, None]
    for h in (0, 17, 31):
        check(out[-n:, h][rows], *attend(q[-n:, h][rows], k[-n:, 0], v[-n:, 0], seen, 1 / math.sqrt(d)))
    assert (out[:n] == 0).all()
