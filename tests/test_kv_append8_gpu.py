"""dt_kv_append8 on the GPU against the same appends in 64 bits.

A stored element x, of a block whose scale is s: rounded once, to e4m3 under s, so off by 2^-4 |x| or, below e4m3's normal
range, by half its least step, 2^-10 s; a rotated key is off by 2^-22 (|a| + |b|) before that (test_kv_append_gpu), which
adds as much, and 2^-4 of it. A kept row that is coded again is exact but below the normal range: 2^-10 s of the new
scale. A scale is the least power of two that brings the largest element to 448: equal, where no element lies within the
rotation's error of a border. Values are copied, not rotated: their codes and scales are equal bit for bit."""
import math

import pytest
import torch

from test_kv_append_gpu import close, make, turned

pytestmark = pytest.mark.gpu
BF, F8 = torch.bfloat16, torch.float8_e4m3fn
LOW, HIGH = -48, 48


def pow2(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def scale_for(amax):
    """The least 2^e with amax <= 448 2^e, e within the limits."""
    e = torch.full(amax.shape, LOW, dtype=torch.int64, device=amax.device)
    for x in range(LOW, HIGH):
        e = torch.where(amax > 448 * 2.0 ** x, x + 1, e)
    return pow2(e)


def to_f8(x):
    """To nearest even in e4m3, what is beyond 448 or no number to NaN: in 64 bits, so rounded once."""
    mag = x.abs()
    step = pow2(torch.floor(torch.log2(mag.clamp(min=2.0 ** -6, max=1e9)) + 1e-12).long() - 3)
    y = torch.round(mag / step) * step  # torch.round: halves to even
    y = torch.where(mag <= 448, y, math.nan)
    return torch.copysign(y, x).float().to(F8)


def pool(pages, Hkv, page, d, block, seed=9, spread=1.0):
    """A cache that earlier tokens fill: codes and their scales."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(pages, Hkv, page // block, block * d, generator=g, device="cuda") * spread
    x = x * 2.0 ** torch.randint(-3, 4, (pages, Hkv, page // block, 1), generator=g, device="cuda")
    scale = scale_for(x.abs().amax(-1).double()).float()
    return to_f8((x / scale[..., None]).double()).view(pages, Hkv, page, d), scale


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def grouped(slots, positions, block, max_pos, end):
    """{block: {row: token}} of the tokens that are appended."""
    out = {}
    for t, slot in enumerate(slots.tolist()):
        if 0 <= slot < end and (positions is None or 0 <= int(positions[t]) < max_pos):
            out.setdefault(slot // block, {})[slot % block] = t
    return out


def check_append8(dtlib, q, k, v, cache, slots, positions, table, interleaved, block, keep_k=False, status=None, ws=None):
    kc, vc, ks, vs = cache
    was = [x.clone() for x in cache]
    pages, Hkv, page, d = kc.shape
    rot = table.shape[1] if table is not None else 0
    out_k = torch.full(k.shape, 7.0, dtype=BF, device="cuda") if keep_k else None
    out_q = torch.full(q.shape, 7.0, dtype=BF, device="cuda") if q is not None else None
    ws = dtlib.new_workspace(dtlib.dt_kv_append8_workspace_bytes(k.shape[0], pages, page)) if ws is None else ws
    dtlib.dt_kv_append8(k, v, kc, vc, ks, vs, slots, positions=positions, rope=table, interleaved=interleaved, q=q,
                        out_q=out_q, out_k=out_k, workspace=ws)
    assert dtlib.dt_get_error(ws) == (status if status is not None else dtlib.Status.OK)
    blocks = grouped(slots, positions if rot else None, block, table.shape[0] if rot else 0, pages * page)
    kept = sorted(t for rows in blocks.values() for t in rows.values())
    at = torch.tensor(kept, dtype=torch.long, device="cuda")

    def rotated(x):
        return turned(x[at], table, positions[at], rot, interleaved) if rot else (
            x[at].double(), torch.zeros_like(x[at].double()))
    left = torch.ones(k.shape[0], dtype=torch.bool, device="cuda")
    left[at] = False
    if q is not None:
        close(out_q[at], rotated(q))
        assert (out_q[left] == 7).all()
    if keep_k:
        close(out_k[at], rotated(k))
        assert (out_k[left] == 7).all()
    if not kept:
        assert all(same(a, b) for a, b in zip(cache, was))
        return
    index = {t: i for i, t in enumerate(kept)}
    ids = sorted(blocks)
    per = page // block
    where = torch.tensor(ids, device="cuda")
    source = torch.tensor([[index[blocks[i][r]] if r in blocks[i] else -1 for r in range(block)] for i in ids],
                          device="cuda")
    written = source >= 0
    low = torch.where(written, torch.arange(block, device="cuda"), block).amin(1)
    below = torch.arange(block, device="cuda") < low[:, None]  # [blocks, block]

    def of(x, *tail):  # [pages, Hkv, per, ...] -> the touched blocks' [blocks, Hkv, ...]
        return x.view(pages, Hkv, per, *tail).transpose(1, 2).flatten(0, 1)[where]
    for cache_now, scale_now, cache_was, scale_was, x, exact in ((kc, ks, was[0], was[2], rotated(k), rot == 0),
                                                                 (vc, vs, was[1], was[3], (v[at].double(), None), True)):
        new = x[0][source.clamp(min=0)].transpose(1, 2)  # [blocks, Hkv, block, d]
        fine = torch.where(written[:, None, :, None] & new.isfinite() & (new.abs() <= 448 * 2.0 ** HIGH), new.abs(), 0)
        amax = fine.amax((2, 3))
        old = of(scale_was).double()
        keep = (low > 0)[:, None] & (scale_for((old * 448).nan_to_num(0, 0, 0).clamp(0, 1e30)) == old)
        want = torch.where(keep, torch.maximum(scale_for(amax), old), scale_for(amax))
        got = of(scale_now).double()
        assert torch.equal(got, want), (got != want).nonzero()[:4]
        code_was = of(cache_was.view(torch.uint8), block, d).view(F8)
        code_now = of(cache_now.view(torch.uint8), block, d).view(F8)
        again = to_f8(code_was.double() * (old / want).nan_to_num(0)[..., None, None])
        again = torch.where((keep & (want > old))[..., None, None] & below[:, None, :, None], again.view(torch.uint8),
                            code_was.view(torch.uint8)).view(F8)
        mine = written[:, None, :, None].expand_as(code_now)
        assert torch.equal(code_now.double().nan_to_num(999)[~mine], again.double().nan_to_num(999)[~mine])
        if exact:
            assert torch.equal(code_now.double().nan_to_num(999)[mine],
                               to_f8(new / want[..., None, None]).double().nan_to_num(999)[mine])
        else:
            bound = torch.zeros_like(new)
            pre = turned_bound(k[at], table, positions[at], rot, interleaved)[source.clamp(min=0)].transpose(1, 2)
            bound = torch.maximum(2.0 ** -4 * (new.abs() + pre), 2.0 ** -10 * want[..., None, None]) + pre
            off = (code_now.double() * want[..., None, None] - new).abs()
            ok = (off <= bound) | ~new.isfinite()
            assert ok[mine].all()
            assert (code_now.double().isnan() == ~new.isfinite())[mine].all()
    rest = torch.ones(pages * per, dtype=torch.bool, device="cuda")
    rest[where] = False
    for now, before, tail in ((kc, was[0], (block, d)), (vc, was[1], (block, d)), (ks, was[2], ()), (vs, was[3], ())):
        cut = lambda x: (x.view(torch.uint8) if x.dtype == F8 else x.view(torch.int32)).view(
            pages, Hkv, per, *tail).transpose(1, 2).flatten(0, 1)[rest]
        assert torch.equal(cut(now), cut(before))  # every other block of the pool is as it was


def turned_bound(x, table, positions, rot, interleaved):
    """2^-22 (|a| + |b|) of each rotated element, zero of the others."""
    x = x.double()
    i = torch.arange(rot // 2, device=x.device)
    first, second = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    out = torch.zeros_like(x)
    out[..., first] = out[..., second] = 2.0 ** -22 * (x[..., first].abs() + x[..., second].abs())
    return out


SHAPES = [
    (1, 32, 8, 128, 64, 16, 128, False, True, False),      # one request's next token
    (1, 1, 1, 64, 8, 8, 64, False, False, True),           # the smallest of everything
    (37, 32, 8, 128, 16, 16, 128, False, True, True),
    (300, 8, 1, 128, 16, 8, 64, False, True, False),       # half of each head rotated
    (300, 12, 2, 64, 32, 32, 32, True, True, True),        # neighbouring pairs, half rotated
    (129, 16, 16, 64, 8, 8, 64, True, False, False),
    (65, 5, 5, 128, 256, 256, 16, False, False, True),     # odd heads, the least rotation, the largest blocks
    (65, 3, 3, 128, 128, 64, 112, True, True, False),      # an interleaved rotation that ends inside an item
    (65, 3, 3, 128, 128, 32, 48, False, True, False),
    (2500, 40, 8, 128, 64, 16, 128, False, True, False),   # tokens found through the index
    (2500, 12, 2, 64, 256, 128, 64, False, True, True),
    (2048, 4, 1, 64, 16, 16, 64, False, True, False), (2049, 4, 1, 64, 16, 16, 64, False, True, False),
    (512, 4, 1, 64, 16, 16, 64, False, True, False), (513, 4, 1, 64, 16, 16, 64, False, True, False),  # the border
]


@pytest.mark.parametrize("N,Hq,Hkv,d,page,block,rot,interleaved,fused,keep_k", SHAPES)
def test_tokens_in_any_order(dtlib, N, Hq, Hkv, d, page, block, rot, interleaved, fused, keep_k):
    """Random slots: blocks with holes, tokens of one block anywhere in the call."""
    q, k, v, kc, _, slots, positions = make(N, Hq, Hkv, d, page, rot, fused=fused)
    (kc, ks), (vc, vs) = (pool(kc.shape[0], Hkv, page, d, block, seed) for seed in (1, 2))
    table = dtlib.rope_table(5000, rot)
    check_append8(dtlib, q, k, v, (kc, vc, ks, vs), slots, positions, table, interleaved, block, keep_k)


@pytest.mark.parametrize("N,Hq,Hkv,d,page,block,rot,interleaved,fused,keep_k", SHAPES)
def test_tokens_in_a_row(dtlib, N, Hq, Hkv, d, page, block, rot, interleaved, fused, keep_k):
    """Runs of consecutive slots that start inside a block, in calls one after the other: rows are kept, and coded again
    where a larger token comes."""
    q, k, v, kc, _, _, positions = make(N, Hq, Hkv, d, page, rot, fused=fused)
    pages = 2 * kc.shape[0]
    (kc, ks), (vc, vs) = (pool(pages, Hkv, page, d, block, seed) for seed in (1, 2))
    table = dtlib.rope_table(5000, rot)
    start = block // 2 + 1
    for grow in (1.0, 4.0, 1.0):
        kk, vv = (k.float() * grow).to(BF), (v.float() * grow).to(BF)
        slots = torch.arange(start, start + N, dtype=torch.int32, device="cuda")
        check_append8(dtlib, q, kk, vv, (kc, vc, ks, vs), slots, positions, table, interleaved, block, keep_k)
        start = min(start + N // 2 + 1, pages * page - N)


@pytest.mark.parametrize("N,Hq,Hkv,d,page,block,rot,interleaved,fused,keep_k", [x for x in SHAPES if x[0] > 1])
def test_rotated_keys_get_the_nearest_codes(dtlib, N, Hq, Hkv, d, page, block, rot, interleaved, fused, keep_k):
    """A rotated key is off by `pre` at most before it is coded, and to_f8 does not decrease: where both ends of that range
    have one code, the stored code is it, bit for bit. Few elements lie so near a border that the ends differ: a code's
    steps are 2^-4 apart or more, relative to elements of 2^-20 and less of error; less than 2% even where the terms cancel."""
    q, k, v, kc, _, slots, positions = make(N, Hq, Hkv, d, page, rot, fused=fused)
    (kc, ks), (vc, vs) = (pool(kc.shape[0], Hkv, page, d, block, seed) for seed in (1, 2))
    table = dtlib.rope_table(5000, rot)
    dtlib.dt_kv_append8(k, v, kc, vc, ks, vs, slots, positions=positions, rope=table, interleaved=interleaved)
    new, pre = turned(k, table, positions, rot, interleaved)[0], turned_bound(k, table, positions, rot, interleaved)
    at, row = slots.long() // page, slots.long() % page
    scale = ks[at, :, row // block].double()[..., None]
    low, high = (to_f8(x / scale).view(torch.uint8) for x in (new - pre, new + pre))
    sure = low == high
    assert sure.double().mean() > 0.98
    got = kc.view(torch.uint8)[at, :, row]
    assert torch.equal(got[sure], low[sure])
    other = got[~sure]
    assert ((other == low[~sure]) | (other == high[~sure]) | (low[~sure] >> 7 != high[~sure] >> 7)).all()


@pytest.mark.parametrize("N", [200, 3000])
def test_padding_tokens_are_left_out(dtlib, N):
    q, k, v, kc, _, slots, positions = make(N, 8, 2, 128, 16, 128)
    (kc, ks), (vc, vs) = (pool(kc.shape[0], 2, 16, 128, 8, seed) for seed in (1, 2))
    slots[::3] = -1
    slots[5] = -2 ** 31
    positions[::3] = 10 ** 6  # not looked at
    positions[5] = -3
    check_append8(dtlib, q, k, v, (kc, vc, ks, vs), slots, positions, dtlib.rope_table(5000, 128), False, 8, keep_k=True)
    slots[:] = -1
    check_append8(dtlib, q, k, v, (kc, vc, ks, vs), slots, positions, dtlib.rope_table(5000, 128), False, 8, keep_k=True)


@pytest.mark.parametrize("N", [120, 2500])
def test_bad_slots_and_positions_are_reported_and_left_out(dtlib, N):
    q, k, v, kc, _, slots, positions = make(N, 4, 2, 64, 16, 64)
    (kc, ks), (vc, vs) = (pool(kc.shape[0], 2, 16, 64, 16, seed) for seed in (1, 2))
    table = dtlib.rope_table(5000, 64)
    for where, value in (("slot", kc.shape[0] * 16), ("slot", 2 ** 31 - 1), ("pos", 5000), ("pos", -1), ("pos", -2 ** 31)):
        s, pos = slots.clone(), positions.clone()
        (s if where == "slot" else pos)[N // 2] = value
        check_append8(dtlib, q, k, v, (kc, vc, ks, vs), s, pos, table, False, 16, status=dtlib.Status.INVALID_ARG)


def test_without_rotation_or_queries(dtlib):
    _, k, v, kc, _, slots, _ = make(70, 4, 2, 64, 16, 0)
    (kc, ks), (vc, vs) = (pool(kc.shape[0], 2, 16, 64, 16, seed) for seed in (1, 2))
    check_append8(dtlib, None, k, v, (kc, vc, ks, vs), slots, None, None, False, 16, keep_k=True)


def test_borders_of_the_scale_and_ties(dtlib):
    """Largest elements on both sides of 448 2^e for every e, ties of the rounding, the smallest and the largest bf16."""
    N, d = 400, 128
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(N, 1, d, generator=g, device="cuda")
    x = x * 2.0 ** torch.randint(-60, 60, (N, 1, 1), generator=g, device="cuda")
    for t in range(0, N, 2):
        e = t // 2 - 100
        x[t] = (torch.randint(0, 33, (1, d), generator=g, device="cuda") - 16) / 16 * 2.0 ** e  # ties among them
        x[t, 0, 5] = 1.75 * 2.0 ** e if t % 4 else 1.7578125 * 2.0 ** e  # the border, and the next bf16 above it
    x[7], x[9], x[11, 0, 3], x[13] = 0, 1e-40, 3.3e38, -0.0
    x = x.to(BF)
    page = block = 8
    kc, vc, ks, vs = dtlib.new_paged_cache8(N + 1, 1, page, d, scale_block=block)
    kc.view(torch.uint8).fill_(0x7F), vc.view(torch.uint8).fill_(0x7F)
    slots = torch.arange(N, dtype=torch.int32, device="cuda") * page  # a block each
    check_append8(dtlib, None, x, x.flip(0), (kc, vc, ks, vs), slots, None, None, False, block)
    check_append8(dtlib, None, x.flip(0), x, (kc, vc, ks, vs), slots + 1, None, None, False, block)  # behind kept rows


def test_what_is_not_finite_is_stored_as_nan_and_leaves_the_rest_alone(dtlib):
    q, k, v, kc, _, _, positions = make(40, 4, 2, 128, 16, 64)
    (kc, ks), (vc, vs) = (pool(8, 2, 16, 128, 16, seed) for seed in (1, 2))
    k[3, 1, 100], v[3, 0, 5], v[4, 1, 127], v[20, 1, 3] = float("nan"), float("inf"), float("nan"), float("-inf")
    k[6, 0, 2] = float("-inf")
    v[30] = float("nan")
    positions[6] = 17
    slots = torch.arange(9, 49, dtype=torch.int32, device="cuda")
    check_append8(dtlib, q, k, v, (kc, vc, ks, vs), slots, positions, dtlib.rope_table(5000, 64), False, 16)


@pytest.mark.parametrize("scale", [0.0, -1.0, 3.0, float("nan"), float("inf"), 2.0 ** 49, 2.0 ** -49, 1e-42])
def test_a_scale_that_is_none_keeps_no_rows(dtlib, scale):
    _, k, v, kc, _, _, _ = make(20, 4, 2, 64, 16, 0)
    (kc, ks), (vc, vs) = (pool(4, 2, 16, 64, 16, seed) for seed in (1, 2))
    ks[0], vs[0] = scale, scale
    slots = torch.arange(5, 25, dtype=torch.int32, device="cuda")
    check_append8(dtlib, None, k, v, (kc, vc, ks, vs), slots, None, None, False, 16)


def test_a_scale_grows_by_any_step_and_starts_anew_with_the_block(dtlib):
    (kc, ks), (vc, vs) = (pool(2, 1, 32, 64, 16, seed) for seed in (1, 2))
    table = None
    for step, row in ((-3, 3), (0, 4), (1, 5), (7, 6), (30, 7), (2, 8), (0, 0), (-40, 0), (100, 1), (0, 2)):
        k, v = (torch.randn(1, 1, 64, device="cuda").mul(2.0 ** step).to(BF) for _ in range(2))
        slots = torch.tensor([row], dtype=torch.int32, device="cuda")
        check_append8(dtlib, None, k, v, (kc, vc, ks, vs), slots, None, table, False, 16)


def test_a_slot_named_twice_holds_one_of_the_two(dtlib):
    for N in (64, 2600):
        _, k, v, kc, _, slots, _ = make(N, 4, 2, 64, 16, 0)
        (kc, ks), (vc, vs) = (pool(kc.shape[0], 2, 16, 64, 16, seed) for seed in (1, 2))
        slots[N - 5] = slots[9]
        dtlib.dt_kv_append8(k, v, kc, vc, ks, vs, slots)
        at, row = int(slots[9]) // 16, int(slots[9]) % 16
        for x, c, s in ((k, kc, ks), (v, vc, vs)):
            got = c.view(torch.uint8)[at, :, row].view(F8).double()
            both = [to_f8(x[t].double() / s[at, :, 0, None].double()).double() for t in (9, N - 5)]
            assert torch.equal(got, both[0]) or torch.equal(got, both[1])


@pytest.mark.parametrize("N", [64, 512, 513, 2600])
@pytest.mark.parametrize("d,block,rot,interleaved", [(64, 16, 64, False), (128, 64, 64, True), (128, 16, 0, False)])
def test_out_k_of_a_slot_named_twice_is_written_for_both(dtlib, N, d, block, rot, interleaved):
    """The cache keeps one of the tokens, the dense keys and queries hold each: far apart, side by side, three of a slot, the
    first and the last token; into arrays of their own and in place."""
    page, max_pos = 64, 5000
    q, k, v, kc, _, slots, positions = make(N, 4, 2, d, page, rot, fused=False)
    for seed in (0, 1):
        if seed:  # tokens in order, as a prompt's
            slots = torch.arange(7, N + 7, dtype=torch.int32, device="cuda")
        slots[N - 5] = slots[9]
        slots[21] = slots[20]
        slots[40], slots[N // 2] = slots[33], slots[33]
        slots[0] = slots[N - 1]
        table = dtlib.rope_table(max_pos, rot) if rot else None
        kw = dict(positions=positions, rope=table) if rot else {}
        want_k, want_q = ((turned(x, table, positions, rot, interleaved) if rot else
                           (x.double(), torch.zeros_like(x.double()))) for x in (k, q))
        caches = []
        for place in (False, True):
            (c, ks), (vc, vs) = (pool(kc.shape[0] + 2, 2, page, d, block, s) for s in (1, 2))
            kk, qq = k.clone(), q.clone()
            out_k, out_q = (kk, qq) if place else (torch.full_like(k, 7.0), torch.full_like(q, 7.0))
            ws = dtlib.new_workspace(dtlib.dt_kv_append8_workspace_bytes(N, c.shape[0], page))
            dtlib.dt_kv_append8(kk, v, c, vc, ks, vs, slots, interleaved=interleaved, q=qq, out_q=out_q, out_k=out_k,
                                workspace=ws, **kw)
            assert dtlib.dt_get_error(ws) == dtlib.Status.OK
            close(out_q, want_q)
            close(out_k, want_k)
            caches.append((c, vc, ks, vs))
        turn = 2.0 ** -21 * k.abs().max().double()  # the rotation's error, at most
        bound = lambda x, s: torch.maximum(2.0 ** -4 * (x.abs() + turn), 2.0 ** -10 * s) + turn
        for c, vc, ks, vs in caches:
            for named in ((9, N - 5), (20, 21), (33, 40, N // 2), (0, N - 1)):  # the key and the value are one token's
                at, row = int(slots[named[0]]) // page, int(slots[named[0]]) % page
                near = []
                for x, cache, scale in ((want_k[0], c, ks), (v.double(), vc, vs)):
                    s = scale[at, :, row // block, None].double()
                    got = cache.view(torch.uint8)[at, :, row].view(F8).double() * s
                    near.append([bool(((got - x[t]).abs() <= bound(x[t], s)).all()) for t in named])
                assert any(a and b for a, b in zip(*near)), (named, near)


def test_in_place_on_dense_queries_and_keys(dtlib):
    for N in (50, 2100):
        q, k, v, kc, _, slots, positions = make(N, 8, 2, 128, 16, 128, fused=False)
        (kc, ks), (vc, vs) = (pool(kc.shape[0], 2, 16, 128, 16, seed) for seed in (1, 2))
        table = dtlib.rope_table(5000, 128)
        q0, k0 = q.clone(), k.clone()
        other = [x.clone() for x in (kc, vc, ks, vs)]
        dtlib.dt_kv_append8(k0, v, *other, slots, positions=positions, rope=table)
        dtlib.dt_kv_append8(k, v, kc, vc, ks, vs, slots, positions=positions, rope=table, q=q, out_q=q, out_k=k)
        close(q, turned(q0, table, positions, 128, False))
        close(k, turned(k0, table, positions, 128, False))
        assert all(same(a, b) for a, b in zip((kc, vc, ks, vs), other))


def test_the_workspace_holds_nothing_between_calls(dtlib):
    """Another call's index, and what other operators leave, are not mistaken for this call's."""
    N, Hkv, page, d = 2600, 2, 16, 64
    ws = None
    for seed in (3, 4, 5):
        _, k, v, kc, _, slots, _ = make(N, 4, Hkv, d, page, 0, seed=seed)
        if ws is None:
            ws = dtlib.new_workspace(dtlib.dt_kv_append8_workspace_bytes(N, kc.shape[0], page))
        else:
            ws[256:] = torch.randint(0, 256, (ws.numel() - 256,), dtype=torch.uint8, device="cuda") * (seed == 5)
        (kc, ks), (vc, vs) = (pool(kc.shape[0], Hkv, page, d, 16, seed) for seed in (1, 2))
        slots[::seed] = -1
        check_append8(dtlib, None, k, v, (kc, vc, ks, vs), slots, None, None, False, 16, ws=ws)


def test_captured_and_replayed_on_other_tokens(dtlib):
    for N in (70, 2300):
        q, k, v, kc, _, slots, positions = make(N, 8, 2, 128, 16, 128, fused=False)
        (kc, ks), (vc, vs) = (pool(kc.shape[0], 2, 16, 128, 16, seed) for seed in (1, 2))
        table, fresh = dtlib.rope_table(5000, 128), [x.clone() for x in (kc, vc, ks, vs)]
        ws = dtlib.new_workspace(dtlib.dt_kv_append8_workspace_bytes(N, kc.shape[0], 16))
        out_q = torch.zeros_like(q)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            dtlib.dt_kv_append8(k, v, kc, vc, ks, vs, slots, positions=positions, rope=table, q=q, out_q=out_q,
                                workspace=ws)
        for _ in range(3):
            slots.copy_(slots[torch.randperm(N, device="cuda")])
            k.copy_(k.flip(0)), q.copy_(q.flip(1))
            for a, b in zip((kc, vc, ks, vs), fresh):
                a.view(torch.uint8).copy_(b.view(torch.uint8))
            want = [x.clone() for x in fresh]
            want_q = dtlib.dt_kv_append8(k, v, *want, slots, positions=positions, rope=table, q=q)
            g.replay()
            torch.cuda.synchronize()
            assert all(same(a, b) for a, b in zip((kc, vc, ks, vs), want)) and torch.equal(out_q, want_q)


def test_far_into_a_large_pool(dtlib):
    """Slots whose bytes lie past 2^32 of the pool."""
    page, Hkv, d = 256, 8, 128
    pages = 2 ** 32 // (page * Hkv * d) + 5
    kc, vc, ks, vs = dtlib.new_paged_cache8(pages, Hkv, page, d, scale_block=16)
    g = torch.Generator(device="cuda").manual_seed(1)
    for N in (4, 2200):
        k, v = (torch.randn(N, Hkv, d, generator=g, device="cuda").to(BF) for _ in range(2))
        slots = (pages * page - 1 - 3 * torch.arange(N, device="cuda")).to(torch.int32)
        slots[1], slots[2] = 0, 5
        dtlib.dt_kv_append8(k, v, kc, vc, ks, vs, slots)
        at, row = slots.long() // page, slots.long() % page
        for x, c, s in ((k, kc, ks), (v, vc, vs)):
            scale = s[at, :, row // 16].double()[..., None]
            got = c.view(torch.uint8)[at, :, row].view(F8).double()
            assert torch.equal(got, to_f8(x.double() / scale).double())


def test_two_calls_at_once(dtlib):
    """Two streams, two caches, a workspace each: tokens found by a look at all of them, and through the index."""
    calls = []
    for N, seed in ((200, 3), (5000, 4)):
        _, k, v, kc, _, slots, _ = make(N, 4, 2, 64, 16, 0, seed=seed)
        (kc, ks), (vc, vs) = (pool(kc.shape[0], 2, 16, 64, 16, seed + i) for i in (1, 2))
        ws = dtlib.new_workspace(dtlib.dt_kv_append8_workspace_bytes(N, kc.shape[0], 16))
        want = [x.clone() for x in (kc, vc, ks, vs)]
        for _ in range(5):
            dtlib.dt_kv_append8(k, v, *want, slots)
        calls.append((k, v, (kc, vc, ks, vs), slots, ws, want, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(5):
        for k, v, cache, slots, ws, _, stream in calls:
            dtlib.dt_kv_append8(k, v, *cache, slots, workspace=ws, stream=stream)
    torch.cuda.synchronize()
    for _, _, cache, _, ws, want, _ in calls:
        assert all(same(a, b) for a, b in zip(cache, want)) and dtlib.dt_get_error(ws) == dtlib.Status.OK


def test_nothing_to_append(dtlib):
    _, k, v, kc, _, slots, _ = make(6, 4, 2, 64, 16, 64)
    (kc, ks), (vc, vs) = (pool(kc.shape[0], 2, 16, 64, 16, seed) for seed in (1, 2))
    was = [x.clone() for x in (kc, vc, ks, vs)]
    dtlib.dt_kv_append8(k[:0], v[:0], kc, vc, ks, vs, slots[:0])
    torch.cuda.synchronize()
    assert all(same(a, b) for a, b in zip((kc, vc, ks, vs), was))


def test_refuses(dtlib):
    q, k, v, kc, _, slots, positions = make(6, 4, 2, 64, 16, 64)
    (kc, ks), (vc, vs) = (pool(kc.shape[0], 2, 16, 64, 8, seed) for seed in (1, 2))
    table = dtlib.rope_table(100, 64)
    call = lambda **kw: dtlib.dt_kv_append8(**{**dict(k=k, v=v, k_cache=kc, v_cache=vc, k_scale=ks, v_scale=vs, slots=slots),
                                               **kw})
    for bad in (dict(rope=table), dict(out_q=q), dict(v=v[:5]), dict(k_cache=kc[:, :1]), dict(k_scale=ks[:, :, :1]),
                dict(v_scale=vs[:1]), dict(k_scale=ks.repeat(1, 1, 3)), dict(v_cache=vc[..., :32].contiguous()),
                dict(k=k.transpose(0, 1).contiguous().transpose(0, 1))):
        with pytest.raises(ValueError):
            call(**bad)
    for bad in (dict(k=k.float()), dict(k_cache=kc.view(torch.uint8)), dict(v_scale=vs.double()), dict(slots=slots.long()),
                dict(slots=slots.cpu())):
        with pytest.raises(TypeError):
            call(**bad)
    four = ks.repeat(1, 1, 2)  # a scale for each four rows
    for bad in (dict(positions=positions, rope=table[:, :24].contiguous()), dict(k_scale=four, v_scale=four),
                dict(workspace=torch.zeros(128, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(dtlib.DTError):
            call(**bad)
    N = 2100
    _, k, v, _, _, slots, _ = make(N, 4, 2, 64, 16, 64)
    with pytest.raises(dtlib.DTError):  # many tokens need the index's room
        dtlib.dt_kv_append8(k, v, kc, vc, ks, vs, slots, workspace=dtlib.new_workspace(256))
