"""How the 8-bit cache's operators and the page plan may be called, and the ends of their envelope: on a stream that is given,
captured without a workspace or an output, workspaces shared with other operators, nothing to do, the most heads, requests
and rows, the longest cache, rows that leave the headroom, codes that are NaN at every token in turn. Against the same in 64
bits, with the bounds of the operators' own tests."""
import math
import random

import pytest
import torch

import test_paged_attn8_gpu as paged8
import test_paged_attn_gpu as paged
import test_prompt_attn_gpu as prompt
from test_kv_append8_gpu import pool, same
from test_kv_append_gpu import close, make, turned
from test_page_plan_gpu import Pool, ints
from test_paged_attn8_gpu import make8, parity, room, run

pytestmark = pytest.mark.gpu
BF, F8, I32 = torch.bfloat16, torch.float8_e4m3fn, torch.int32


def late(stream, *pairs):
    """On `stream`, behind some milliseconds of other work: each pair's second tensor into its first."""
    with torch.cuda.stream(stream):
        torch.cuda._sleep(10_000_000)
        for to, x in pairs:
            to.copy_(x)


def test_on_the_stream_that_is_given(dtlib):
    """The inputs come late on that stream: a call on another one would not see them."""
    side = torch.cuda.Stream()
    s = make8([3000, 40, 700], 4, 16, 2, 128, 16, 16)
    want, q0 = run(dtlib, s).clone(), s["q"].clone()
    for given in (side, side.cuda_stream):
        for ws in (room(dtlib, s), None):
            s["q"].zero_()
            out = torch.full_like(want, float("nan"))
            torch.cuda.synchronize()
            late(side, (s["q"], q0))
            got = run(dtlib, s, out=out, workspace=ws, stream=given)
            side.synchronize()
            assert got is out and torch.equal(out, want)
    s["q"].zero_()
    torch.cuda.synchronize()
    late(side, (s["q"], q0))
    got = run(dtlib, s, stream=side)
    side.synchronize()
    assert torch.equal(got, want)

    for N in (40, 700):
        _, k, v, kc, _, slots, _ = make(N, 4, 2, 64, 16, 0)
        (kc, ks), (vc, vs) = (pool(kc.shape[0], 2, 16, 64, 16, seed) for seed in (1, 2))
        want, slots0 = [x.clone() for x in (kc, vc, ks, vs)], slots.clone()
        dtlib.dt_kv_append8(k, v, *want, slots)
        slots.fill_(-1)
        torch.cuda.synchronize()
        late(side, (slots, slots0))
        dtlib.dt_kv_append8(k, v, kc, vc, ks, vs, slots, stream=side)
        side.synchronize()
        assert all(same(a, b) for a, b in zip((kc, vc, ks, vs), want))

    lens, grow = ints([7, 30, 0]), ints([0] * 3)
    ref = Pool(3, 40, 10, 8)
    state = ref.tensors()
    ref.step([0] * 3, [7, 30, 0], rows=37)
    dtlib.dt_page_plan(ints([0] * 3), lens, page_size=8, num_pages=40, **state)
    want, _ = ref.step([7, 30, 0], [3, 9, 20], rows=32)
    after = ints([3, 9, 20])
    torch.cuda.synchronize()
    late(side, (grow, after))
    out = dtlib.dt_page_plan(lens, grow, page_size=8, num_pages=40, rows=32, stream=side, **state)
    side.synchronize()
    assert [out[x].tolist() for x in ("lens", "cu_seqlens", "slots", "positions")] == list(want)
    none = ints([])
    out = dtlib.dt_page_plan(none, none, state["page_table"][:0], 8, 40, stream=side)
    side.synchronize()
    assert out["cu_seqlens"].tolist() == [0]


def test_captured_without_a_workspace_or_an_output(dtlib):
    """A step of a decoding loop as a graph whose calls allocate for themselves: plan, append, attention; replayed, each
    replay a token further, against the same steps one by one."""
    B, Hq, Hkv, d, page, pages = 5, 8, 2, 64, 16, 40
    g = torch.Generator(device="cuda").manual_seed(3)
    start = [1, 15, 16, 40, 0]
    rope = dtlib.rope_table(200, d)

    def program():
        cache = dtlib.new_paged_cache8(pages, Hkv, page, d)
        state = dict(page_table=torch.full((B, 8), -1, dtype=I32, device="cuda"), held=ints([0] * B),
                     free_pages=torch.arange(pages, dtype=I32, device="cuda"), free_count=ints([pages]))
        lens, one = ints(start), ints([1] * B)
        x = torch.zeros(B, Hq + 2 * Hkv, d, dtype=BF, device="cuda")
        first = dtlib.dt_page_plan(ints([0] * B), lens, page_size=page, num_pages=pages, rows=sum(start), **state)
        k = torch.randn(sum(start), Hkv, d, generator=torch.Generator(device="cuda").manual_seed(9), device="cuda").to(BF)
        dtlib.dt_kv_append8(k, k, *cache, first["slots"], positions=first["positions"], rope=rope)

        def step():
            plan = dtlib.dt_page_plan(lens, one, page_size=page, num_pages=pages, n=1, **state)
            q = dtlib.dt_kv_append8(x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], *cache, plan["slots"],
                                    positions=plan["positions"], rope=rope, q=x[:, :Hq])
            out = dtlib.dt_paged_attention8(q[:, None].contiguous(), *cache, state["page_table"], plan["lens"], 0.125)
            lens.copy_(plan["lens"])
            return out
        return x, step, cache, state
    x, step, cache, state = program()
    y, same_step, cache2, state2 = program()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for _ in range(20):
        new = torch.randn(x.shape, generator=g, device="cuda").to(BF)
        x.copy_(new), y.copy_(new)
        graph.replay()
        assert torch.equal(out, same_step())
    for b in range(B):
        for i in range(int(state["held"][b])):
            p, p2 = int(state["page_table"][b, i]), int(state2["page_table"][b, i])
            assert p == p2
    assert state["free_count"].tolist() == state2["free_count"].tolist()


def test_a_plan_of_many_blocks_captured_and_replayed(dtlib):
    """The last block to finish leaves the counts, and the workspace, ready for the next replay."""
    B = 300
    r = random.Random(2)
    grow = [r.randint(0, 60) for _ in range(B)]
    ref = Pool(B, B * 60, 60, 16, seed=1)
    state = ref.tensors()
    lens, more = ints([0] * B), ints(grow)
    out = dict(lens=lens, cu_seqlens=ints([0] * (B + 1)), slots=ints([0] * sum(grow)), positions=ints([0] * sum(grow)))
    ws = dtlib.new_workspace(dtlib.dt_page_plan_workspace_bytes(B))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dtlib.dt_page_plan(lens, more, page_size=16, num_pages=ref.pages, out=out, workspace=ws, **state)
    have = [0] * B
    for _ in range(8):
        want, _ = ref.step(have, grow, rows=sum(grow))
        g.replay()
        assert [out[x].tolist() for x in ("lens", "cu_seqlens", "slots", "positions")] == list(want)
        assert state["free_count"].tolist() == [ref.count] and state["page_table"].tolist() == ref.table
        have = want[0]
    assert dtlib.dt_get_error(ws) == dtlib.Status.OK and not ws[:256].any()


def test_only_a_workspace_s_header_has_to_be_zero(dtlib):
    """One workspace for all operators of a cache, in any order; only its first 256 bytes are found, and they are left so."""
    a, b = make8([3000, 129, 1500], 2, 8, 2, 128, 16, 16), make8([700] * 9, 16, 8, 2, 64, 16, 16)
    c, p = paged.make([3000, 129], 2, 8, 2, 128, 16, mask="tree"), prompt.make([300, 700], 8, 2, 64)
    N = 900
    _, k, v, kc, _, slots, _ = make(N, 4, 2, 64, 16, 0)
    fresh = [x for seed in (1, 2) for x in pool(kc.shape[0], 2, 16, 64, 16, seed)]
    cache = lambda: [fresh[i].clone() for i in (0, 2, 1, 3)]

    def append(**kw):
        out = cache()
        dtlib.dt_kv_append8(k, v, *out, slots, **kw)
        return torch.cat([x.view(torch.uint8).flatten() for x in out])

    def plan(**kw):
        ref = Pool(300, 9000, 60, 16)
        out = dtlib.dt_page_plan(ints([0] * 300), ints([40] * 300), page_size=16, num_pages=9000, rows=12000, **ref.tensors(),
                                 **kw)
        return torch.cat([out[x] for x in ("lens", "cu_seqlens", "slots", "positions")])
    calls = [lambda **kw: run(dtlib, a, **kw), append, lambda **kw: paged.run(dtlib, c, **kw), plan,
             lambda **kw: run(dtlib, b, **kw), lambda **kw: prompt.run(dtlib, p, **kw)]
    bits = lambda x: x.contiguous().view(torch.uint8)
    want = [bits(call()).clone() for call in calls]
    ws = dtlib.new_workspace(max(room(dtlib, a).numel(), room(dtlib, b).numel(),
                                 dtlib.dt_kv_append8_workspace_bytes(N, kc.shape[0], 16),
                                 dtlib.dt_paged_attention_workspace_bytes(2, 2, 8, 2, 128)))
    order = list(range(len(calls)))
    r = random.Random(1)
    for fill in (0xFF, 0x01, 0x7F, 0):
        ws[256:] = fill
        for _ in range(3):
            for i in order:
                assert torch.equal(bits(calls[i](workspace=ws)), want[i]), i
            r.shuffle(order)
        assert dtlib.dt_get_error(ws) == dtlib.Status.OK and not ws[:256].any()


def test_nothing_to_do(dtlib):
    s = make8([30, 20], 2, 8, 2, 64, 16, 16)
    out = dtlib.dt_paged_attention8(s["q"][:0], s["kc"], s["vc"], s["ks"], s["vs"], s["table"][:0], s["lens"][:0], 0.1,
                                    mask=s["mask"][:0])
    assert out.shape == (0, 2, 8, 64)
    q, k, v, kc, _, slots, positions = make(5, 4, 2, 64, 16, 64)
    (kc, ks), (vc, vs) = (pool(kc.shape[0], 2, 16, 64, 16, seed) for seed in (1, 2))
    was = [x.clone() for x in (kc, vc, ks, vs)]
    got = dtlib.dt_kv_append8(k[:0], v[:0], kc, vc, ks, vs, slots[:0], positions=positions[:0],
                              rope=dtlib.rope_table(100, 64), q=q[:0], out_k=k[:0].contiguous())
    torch.cuda.synchronize()
    assert got.shape == (0, 4, 64) and all(same(a, b) for a, b in zip((kc, vc, ks, vs), was))


def test_a_table_without_a_spare_entry(dtlib):
    for lens, n, page, width in (([64, 128, 127], 1, 16, 8), ([16, 7], 3, 16, 1), ([256, 129], 2, 256, 1), ([64, 9], 1, 8, 8)):
        s = make8(lens, n, 8, 2, 64 if n == 3 else 128, page, 8, mask="tree" if n > 1 else None)
        s["table"] = s["table"][:, :width].contiguous()
        parity(dtlib, s)


@pytest.mark.parametrize("Hq,Hkv", [(256, 256), (256, 2), (128, 1)])
def test_the_most_heads(dtlib, Hq, Hkv):
    for d in (64, 128):
        parity(dtlib, make8([300, 5], 1, Hq, Hkv, d, 16, 16, mask=None), heads=[0, 1, Hq // 2, Hq - 1])


@pytest.mark.parametrize("d", [64, 128])
def test_the_most_of_everything(dtlib, d):
    """The most requests, nodes and query rows at once (the plan and the queries leave the ring its least room)."""
    lens = [64 + (29 * i) % 150 if i % 9 else 0 for i in range(2048)]
    parity(dtlib, make8(lens, 64, 2, 1, d, 16, 16), requests=[0, 1, 2, 9, 700, 2046, 2047])


# growth of a row's scores in base 2: within the headroom (2^11 above where a row starts), about its end, far beyond
GROWTH = [5.0, 10.5, 11.5, 13.0, 27.0, 300.0]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,Hq", [(1, 8), (3, 8), (8, 8), (16, 8), (32, 8)])
@pytest.mark.parametrize("start", [1, 100, 128, 256, 500, 997])
def test_rows_that_leave_the_headroom(dtlib, d, n, Hq, start):
    """From key `start` on every second query head's scores are higher: in a block's middle and at its ends, in the first
    and the second block of a step, in the last block alone; for each number of rows."""
    for growth in GROWTH:
        s = paged.make([1000, 515, 128 + n], n, Hq, 2, d, 16, mask="tree" if n > 1 else None, spread=0.5)
        s["q"][..., 0] = 0.0
        s["q"][:, :, 1::2, 0] = 4.0
        s["kc"][..., 0] = torch.where(s["kc"][..., 0].isnan(), s["kc"][..., 0], 0.0)
        for b in range(3):
            for key in range(start, int(s["lens"][b])):
                if key % 16 == 0 or key == start:  # the rest of a page at once
                    rows = s["kc"][int(s["table"][b, key // 16]), :, key % 16:, 0]
                    rows.copy_(torch.where(rows.isnan(), rows, growth * math.log(2) / 4 / s["scale"]))
        g = torch.Generator(device="cuda").manual_seed(6)
        s["kc"], s["ks"] = paged8.coded(s["kc"], 16)
        s["vc"], s["vs"] = paged8.coded(s["vc"], 16, g)
        parity(dtlib, s, heads=[0, 1, Hq - 1])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,Hq", [(1, 4), (6, 8), (16, 8)])
def test_nan_codes_at_every_token(dtlib, d, n, Hq):
    """A NaN code among the keys or the values, at every token of a request in turn, reaches the rows that see it and no
    other, bit for bit."""
    s = make8([50, 150, 33], n, Hq, 2, d, 16, 16, mask="tree" if n > 1 else None)
    clean = run(dtlib, s).clone()
    G = Hq // 2
    for at in range(150):
        row = slice(None) if at < 150 - n else (s["mask"][1, :, at - (150 - n)] != 0 if n > 1 else slice(None))
        for name, head, column in (("vc", 1, d - 3), ("kc", 0, 5)):
            page = int(s["table"][1, at // 16])
            code = s[name].view(torch.uint8)[page, head, at % 16, column]
            was = code.clone()
            code.fill_(0xFF if at % 2 else 0x7F)
            out = run(dtlib, s)
            code.copy_(was)
            hit = torch.zeros_like(clean, dtype=torch.bool)
            part = hit[1, :, head * G:(head + 1) * G]
            part[row] = True
            if name == "vc":
                part[..., :column] = part[..., column + 1:] = False
            assert out[hit].isnan().all() and torch.equal(out[~hit], clean[~hit]), (at, name)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq", [2, 64])
def test_over_the_longest_cache(dtlib, d, Hq):
    """2^24 tokens (one page many times over), all of one value but the first page's, whose keys score lower by 2^9: within
    the headroom. The output is that value: the first page's 256 values weigh 2^-9 each, of 2^24; the weights' rounding to
    fp16 (2^-11), the output's (2^-8), sums of a CTA's share of 863 blocks (11 and one addition a block of the weights; 8
    products a block of the outputs, two steps each, of 2^-23) and 152 parts joined (three steps of 2^-22 each)."""
    page, T = 256, 1 << 24
    kc, vc, ks, vs = dtlib.new_paged_cache8(2, 1, page, d, scale_block=64)
    k = torch.zeros(2, 1, page, d, device="cuda")
    k[1, ..., 0] = 448
    kc.copy_(k.to(F8))
    ks.fill_(9 * math.log(2) / 4 / 448)
    vc[1].copy_(torch.full((1, page, d), 3.0, device="cuda").to(F8)), vc[0].copy_(torch.full((1, page, d), -3.0, device="cuda").to(F8))
    vs.fill_(0.75)
    q = torch.zeros(1, 1, Hq, d, dtype=BF, device="cuda")
    q[..., 0] = 4.0
    table = torch.ones(1, T // page, dtype=I32, device="cuda")
    table[0, 0] = 0
    lens = torch.tensor([T], dtype=I32, device="cuda")
    ws = dtlib.new_workspace(dtlib.dt_paged_attention8_workspace_bytes(1, 1, Hq, 1, d))
    out = dtlib.dt_paged_attention8(q, kc, vc, ks, vs, table, lens, 1.0, workspace=ws)
    assert dtlib.dt_get_error(ws) == dtlib.Status.OK
    off = 2.0 ** -11 + 2.0 ** -8 + (11 + 863) * 2.0 ** -23 + 16 * 863 * 2.0 ** -23 + 3 * 152 * 2.0 ** -22 + 2 * 256 * 2.0 ** -33
    assert ((out.double() / 2.25 - 1).abs() <= off).all(), (out.double() / 2.25 - 1).abs().max()


def test_queries_past_two_to_the_31_elements(dtlib):
    """Appended tokens whose queries and dense keys lie past 2^31 elements, in a pool past 2^31 codes."""
    N, Hq, Hkv, d, page = 530_011, 32, 32, 128, 256
    assert N * Hq * d > 2 ** 31
    pages = -(-N // page) + 1
    g = torch.Generator(device="cuda").manual_seed(5)
    q, k = (torch.zeros(N, h, d, dtype=BF, device="cuda") for h in (Hq, Hkv))
    at = torch.cat([torch.arange(3, device="cuda"), torch.randint(0, N, (40,), generator=g, device="cuda"),
                    torch.arange(N - 30, N, device="cuda")])
    for x in (q, k):
        x[at] = torch.randn(at.numel(), x.shape[1], d, generator=g, device="cuda").to(BF)
    cache = dtlib.new_paged_cache8(pages, Hkv, page, d, scale_block=16)
    slots = torch.arange(N, dtype=I32, device="cuda") + 17
    positions = torch.arange(N, dtype=I32, device="cuda") % 4000
    rope = dtlib.rope_table(4000, d)
    out_k = torch.full_like(k, 7.0)
    ws = dtlib.new_workspace(dtlib.dt_kv_append8_workspace_bytes(N, pages, page))
    out_q = dtlib.dt_kv_append8(k, k, *cache, slots, positions=positions, rope=rope, q=q, out_k=out_k, workspace=ws)
    assert dtlib.dt_get_error(ws) == dtlib.Status.OK
    for got, x in ((out_q, q), (out_k, k)):
        close(got[at], turned(x[at], rope, positions[at], d, False))
    to, row = slots[at].long() // page, slots[at].long() % page
    for name, x in (("k", turned(k[at], rope, positions[at], d, False)[0]), ("v", k[at].double())):
        codes, scale = (cache[0], cache[2]) if name == "k" else (cache[1], cache[3])
        s = scale[to, :, row // 16].double()[..., None]
        got = codes.view(torch.uint8)[to, :, row].view(F8).double() * s
        e = 2.0 ** -21 * k[at].abs().max().double() if name == "k" else 0.0  # the rotation's error, at most
        assert ((got - x).abs() <= torch.maximum(2.0 ** -4 * (x.abs() + e), 2.0 ** -10 * s) + e).all()
