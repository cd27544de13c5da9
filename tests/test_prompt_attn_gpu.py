"""dt_prompt_attention on the GPU against plain attention in 64 bits, one head at a time (attention_ref: the bound is
derived there)."""
import math

import pytest
import torch

from attention_ref import attend, check

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def make(lens, Hq, Hkv, d, before=0, behind=0, fused=True, seed=7, spread=1.5):
    """Rows that belong to no prompt hold NaN."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    total = before + sum(lens) + behind
    x = torch.randn(total, Hq + 2 * Hkv, d, generator=g, device="cuda")
    x[:, :Hq] *= spread
    x[:before], x[total - behind:] = float("nan"), float("nan")
    x = x.to(BF)
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    cu = [before]
    for n in lens:
        cu.append(cu[-1] + n)
    return dict(q=q, k=k, v=v, cu=torch.tensor(cu, dtype=torch.int32, device="cuda"), scale=1 / math.sqrt(d))


def run(dtlib, s, **kw):
    return dtlib.dt_prompt_attention(s["q"], s["k"], s["v"], s["cu"], s["scale"], **kw)


def parity(dtlib, s, prompts=None, heads=None, rows=None):
    total, Hq, d = s["q"].shape
    G = Hq // s["k"].shape[1]
    ws = dtlib.new_workspace(dtlib.dt_prompt_attention_workspace_bytes(total, len(s["cu"]) - 1, Hq, Hq // G, d))
    out = torch.full((total, Hq, d), 7.0, dtype=BF, device="cuda")
    run(dtlib, s, out=out, workspace=ws)
    assert dtlib.dt_get_error(ws) == dtlib.Status.OK
    cu = s["cu"].tolist()
    for b in prompts if prompts is not None else range(len(cu) - 1):
        lo, hi = cu[b], cu[b + 1]
        if lo == hi:
            continue
        for h in heads if heads is not None else range(Hq):
            at = torch.tensor(rows, device="cuda") if rows else torch.arange(hi - lo, device="cuda")
            seen = torch.arange(hi - lo, device="cuda") <= at[:, None]
            check(out[lo:hi, h][at], *attend(s["q"][lo:hi, h][at], s["k"][lo:hi, h // G], s["v"][lo:hi, h // G], seen,
                                             s["scale"]))
    assert (out[:cu[0]] == 7).all() and (out[cu[-1]:] == 7).all()  # rows of no prompt are left as they were
    again = torch.full_like(out, 7.0)
    run(dtlib, s, out=again, workspace=ws)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))
    return out


@pytest.mark.parametrize("lens,Hq,Hkv,d,before,behind,fused", [
    ([1], 1, 1, 64, 0, 0, False),                           # one token
    ([1, 1, 1], 4, 2, 128, 0, 3, True),
    ([2, 127, 128, 129], 4, 2, 128, 0, 0, True),            # around a tile
    ([255, 256, 257], 4, 1, 64, 0, 1, True),                # around a CTA's rows
    ([511, 512, 513, 1], 2, 2, 128, 5, 200, True),
    ([0, 3, 0, 0, 300, 0], 8, 2, 64, 0, 0, False),          # empty prompts
    ([0, 0], 2, 1, 128, 0, 9, False),                       # nothing but empty prompts
    ([77], 32, 8, 128, 0, 0, False),
    ([640, 33, 1000], 12, 2, 64, 1, 1, True),
    ([385, 2000], 5, 5, 128, 0, 0, True),
    ([700], 8, 1, 128, 300, 300, True),
])
def test_prompts(dtlib, lens, Hq, Hkv, d, before, behind, fused):
    parity(dtlib, make(lens, Hq, Hkv, d, before, behind, fused))


def test_many_prompts(dtlib):
    """More prompts than one search round covers."""
    lens = [(31 * i) % 70 for i in range(1500)]
    s = make(lens, 2, 1, 64)
    parity(dtlib, s, prompts=[0, 1, 2, 31, 32, 33, 999, 1023, 1024, 1025, 1498, 1499])


@pytest.mark.parametrize("d", [64, 128])
def test_a_long_prompt(dtlib, d):
    n = 8200
    parity(dtlib, make([n, 40], 4, 2, d), prompts=[0], heads=[0, 3],
           rows=[0, 1, 127, 128, 255, 256, 1000, 4095, 4096, 8063, 8064, 8191, 8192, n - 1])


def test_scores_far_apart(dtlib):
    """Scores that grow by hundreds along the prompt: the running maximum is raised again and again."""
    s = make([900], 4, 2, 128, fused=False, spread=20.0)
    s["k"] *= (torch.arange(900, device="cuda") // 60 + 1)[:, None, None] / 8
    parity(dtlib, s)


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("token", [0, 60, 127, 128, 200, 255, 256, 299])
def test_what_is_not_finite_stays_with_the_rows_that_see_it(dtlib, bad, token):
    s = make([50, 300, 400], 4, 2, 128, fused=False)
    clean = run(dtlib, s).clone()
    at = 50 + token
    s["v"][at, 1, 77] = bad
    out = run(dtlib, s)
    hit = torch.zeros_like(out, dtype=torch.bool)
    hit[at:350, 2:, 77] = True
    assert torch.equal(out[~hit], clean[~hit])
    assert out[hit].isnan().all() if math.isnan(bad) else (out[hit] == bad).all()
    s["v"][at, 1, 77] = 1.0
    s["k"][at, 0, 3] = float("nan")
    out = run(dtlib, s)
    hit[:] = False
    hit[at:350, :2] = True
    assert out[hit].isnan().all() and out[~hit].isfinite().all()
    assert torch.equal(out[:at, :2], clean[:at, :2]) and torch.equal(out[350:], clean[350:])


def test_a_row_of_infinities_among_the_queries(dtlib):
    s = make([300], 2, 1, 64, fused=False)
    clean = run(dtlib, s).clone()
    s["q"][130, 1] = float("inf")
    out = run(dtlib, s)
    assert out[130, 1].isnan().all()
    out[130, 1] = clean[130, 1]
    assert torch.equal(out, clean)


def test_bad_lengths_are_reported(dtlib):
    s = make([100, 200, 300], 2, 1, 64)
    ws = dtlib.new_workspace(256)
    for cu in ([-1, 100, 300, 600], [0, 100, 300, 601], [0, 300, 100, 600], [0, 2 ** 31 - 1, 5, 600]):
        out = torch.full((600, 2, 64), 7.0, dtype=BF, device="cuda")
        run(dtlib, {**s, "cu": torch.tensor(cu, dtype=torch.int32, device="cuda")}, out=out, workspace=ws)
        assert dtlib.dt_get_error(ws) == dtlib.Status.INVALID_ARG, cu
    assert torch.equal(run(dtlib, s, workspace=ws), run(dtlib, s))
    assert dtlib.dt_get_error(ws) == dtlib.Status.OK


def test_a_captured_call_follows_the_lengths(dtlib):
    a, b = make([100, 200, 300], 4, 2, 128, fused=False), make([500, 0, 20], 4, 2, 128, behind=80, fused=False, seed=11)
    want = [run(dtlib, x, out=torch.zeros_like(x["q"])) for x in (a, b)]
    ws, out = dtlib.new_workspace(256), torch.zeros_like(a["q"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(dtlib, a, out=out, workspace=ws)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        run(dtlib, a, out=out, workspace=ws)
    for x, w in ((a, want[0]), (b, want[1])):
        for key in ("q", "k", "v", "cu"):
            a[key].copy_(x[key])
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, w)


def test_prompt_attention_refuses(dtlib):
    s = make([30, 20], 4, 2, 64, fused=False)
    for key, wrong, error in [("q", s["q"].float(), TypeError), ("q", s["q"][:, :3], dtlib.DTError),
                              ("k", s["k"][1:], ValueError), ("v", s["v"].half(), TypeError),
                              ("v", s["v"].transpose(0, 1).contiguous().transpose(0, 1), ValueError),
                              ("cu", s["cu"].long(), TypeError), ("cu", s["cu"].cpu(), TypeError),
                              ("k", s["k"].cpu(), TypeError), ("scale", 0.0, dtlib.DTError)]:
        with pytest.raises(error):
            run(dtlib, {**s, key: wrong})
