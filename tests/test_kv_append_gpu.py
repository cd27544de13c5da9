"""dt_kv_append on the GPU against the rotation in 64 bits.

Tolerance of a rotated element a c - b s: two fp32 products and a difference, each off by 2^-24 of its value, so at
most 2^-22 (|a| + |b|) in all, then one rounding to bf16 of the value so changed, 2^-8 of it. Everything that is copied
is equal bit for bit."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def make(N, Hq, Hkv, d, page, rot, pages=None, fused=True, seed=3, max_pos=5000):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF)
    if fused:
        qkv = rnd(N, Hq + 2 * Hkv, d)
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    else:
        q, k, v = rnd(N, Hq, d), rnd(N, Hkv, d), rnd(N, Hkv, d)
    pages = pages or -(-N // page) + 3
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:N].to(torch.int32)
    positions = torch.randint(0, max_pos, (N,), generator=g, device="cuda", dtype=torch.int32)
    return q, k, v, rnd(pages, Hkv, page, d), rnd(pages, Hkv, page, d), slots, positions


def turned(x, table, positions, rot, interleaved):
    """The rotation in 64 bits, and its bound."""
    x = x.double()
    t = table.double()[positions.long()][:, None]
    c, s = t[..., :rot // 2], t[..., rot // 2:]
    i = torch.arange(rot // 2, device=x.device)
    first, second = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    a, b = x[..., first], x[..., second]
    out, bound = x.clone(), torch.zeros_like(x)
    out[..., first], out[..., second] = a * c - b * s, b * c + a * s
    small = 2.0 ** -22 * (a.abs() + b.abs())
    for cols in (first, second):
        bound[..., cols] = 2.0 ** -8 * (out[..., cols].abs() + small) + small
    return out, bound


def close(got, want):
    out, bound = want
    off = (got.double() - out).abs()
    assert (off <= bound).all(), (off - bound).max().item()


def check_append(dtlib, q, k, v, kc, vc, slots, positions, table, interleaved, keep_k=False, **kw):
    kc0, vc0 = kc.clone(), vc.clone()
    rot = table.shape[1] if table is not None else 0
    out_k = torch.full(k.shape, 7.0, dtype=BF, device="cuda") if keep_k else None
    out_q = torch.full(q.shape, 7.0, dtype=BF, device="cuda") if q is not None else None
    ws = dtlib.new_workspace(256)
    dtlib.dt_kv_append(k, v, kc, vc, slots, positions=positions, rope=table, interleaved=interleaved, q=q, out_q=out_q,
                       out_k=out_k, workspace=ws, **kw)
    assert dtlib.dt_get_error(ws) == dtlib.Status.OK
    kept = (slots >= 0).nonzero()[:, 0]
    page, row = slots[kept].long() // kc.shape[2], slots[kept].long() % kc.shape[2]

    def rotated(x):
        if rot == 0:
            return x[kept].double(), torch.zeros_like(x[kept].double())
        return turned(x[kept], table, positions[kept], rot, interleaved)
    close(kc[page, :, row], rotated(k))
    assert torch.equal(vc[page, :, row], v[kept])
    if keep_k:
        assert torch.equal(out_k[kept], kc[page, :, row])
        assert (out_k[slots < 0] == 7).all()
    if q is not None:
        close(out_q[kept], rotated(q))
        assert (out_q[slots < 0] == 7).all()
    rest = torch.ones(kc.shape[0], kc.shape[2], dtype=torch.bool, device="cuda")
    rest[page, row] = False
    for now, was in ((kc, kc0), (vc, vc0)):  # every other row of the pool is as it was
        assert torch.equal(now.transpose(1, 2)[rest], was.transpose(1, 2)[rest])


@pytest.mark.parametrize("N,Hq,Hkv,d,page,rot,interleaved,fused,keep_k", [
    (1, 32, 8, 128, 64, 128, False, True, False),     # one request's next token
    (1, 1, 1, 64, 8, 64, False, False, True),         # the smallest of everything
    (37, 32, 8, 128, 16, 128, False, True, True),
    (300, 8, 1, 128, 16, 64, False, True, False),     # half of each head rotated
    (300, 12, 2, 64, 32, 32, True, True, True),       # neighbouring pairs, half rotated
    (129, 16, 16, 64, 8, 64, True, False, False),
    (65, 5, 5, 128, 256, 16, False, False, True),     # odd heads, the least rotation
    (65, 3, 3, 128, 128, 112, True, True, False),     # an interleaved rotation that ends inside an item
    (2500, 40, 8, 128, 64, 128, False, True, False),  # more tokens than resident CTAs
])
def test_append_parity(dtlib, N, Hq, Hkv, d, page, rot, interleaved, fused, keep_k):
    q, k, v, kc, vc, slots, positions = make(N, Hq, Hkv, d, page, rot, fused=fused)
    table = dtlib.rope_table(5000, rot)
    check_append(dtlib, q, k, v, kc, vc, slots, positions, table, interleaved, keep_k)


def test_append_leaves_padding_tokens_out(dtlib):
    q, k, v, kc, vc, slots, positions = make(200, 8, 2, 128, 16, 128)
    slots[::3] = -1
    slots[5] = -2 ** 31
    positions[::3] = 10 ** 6  # not looked at
    check_append(dtlib, q, k, v, kc, vc, slots, positions, dtlib.rope_table(5000, 128), False, keep_k=True)


def test_append_without_rotation_or_queries_copies(dtlib):
    _, k, v, kc, vc, slots, _ = make(70, 4, 2, 64, 16, 0)
    check_append(dtlib, None, k, v, kc, vc, slots, None, None, False, keep_k=True)


def test_append_keeps_what_is_not_finite_where_it_is(dtlib):
    """Infinities and NaN in a token reach that token's rows only, and copied elements keep their bits."""
    q, k, v, kc, vc, slots, positions = make(9, 4, 2, 128, 16, 64)
    k[3, 1, 100], v[3, 0, 5], v[4, 1, 127] = float("nan"), float("inf"), float("nan")
    k[6, 0, 2] = float("-inf")
    positions[6] = 17
    table = dtlib.rope_table(5000, 64)
    dtlib.dt_kv_append(k, v, kc, vc, slots, positions=positions, rope=table, q=q)
    rows = lambda c: c[slots.long() // 16, :, slots.long() % 16]
    assert torch.equal(rows(vc).view(torch.int16), v.contiguous().view(torch.int16))
    out, bound = turned(k, table, positions, 64, False)
    got = rows(kc).double()
    assert torch.equal(got.isnan(), out.isnan()) and torch.equal(got.isinf(), out.isinf())
    fine = out.isfinite()
    assert ((got - out).abs()[fine] <= bound[fine]).all()


def test_append_in_place_on_dense_queries_and_keys(dtlib):
    q, k, v, kc, vc, slots, positions = make(50, 8, 2, 128, 16, 128, fused=False)
    table = dtlib.rope_table(5000, 128)
    q0, k0 = q.clone(), k.clone()
    dtlib.dt_kv_append(k, v, kc, vc, slots, positions=positions, rope=table, q=q, out_q=q, out_k=k)
    close(q, turned(q0, table, positions, 128, False))
    close(k, turned(k0, table, positions, 128, False))


def test_append_reports_bad_slots_and_positions_and_leaves_them_out(dtlib):
    q, k, v, kc, vc, slots, positions = make(12, 4, 2, 64, 16, 64)
    table, ws = dtlib.rope_table(5000, 64), dtlib.new_workspace(256)
    for spoil in ("slot", "late", "negative"):
        s, pos = slots.clone(), positions.clone()
        if spoil == "slot":
            s[4] = kc.shape[0] * 16
        else:
            pos[4] = 5000 if spoil == "late" else -1
        a, b, oq = kc.clone(), vc.clone(), torch.full_like(q, 7.0)
        dtlib.dt_kv_append(k, v, a, b, s, positions=pos, rope=table, q=q, out_q=oq, workspace=ws)
        assert dtlib.dt_get_error(ws) == dtlib.Status.INVALID_ARG
        s[4] = -1
        a2, b2, oq2 = kc.clone(), vc.clone(), torch.full_like(q, 7.0)
        dtlib.dt_kv_append(k, v, a2, b2, s, positions=positions, rope=table, q=q, out_q=oq2, workspace=ws)
        assert dtlib.dt_get_error(ws) == dtlib.Status.OK
        assert torch.equal(a, a2) and torch.equal(b, b2) and torch.equal(oq, oq2)


def test_append_far_into_a_large_pool(dtlib):
    """Slots whose elements lie past 2^31 (and whose bytes past 2^32) of the pool."""
    page, Hkv, d = 256, 8, 128
    pages = 2 ** 31 // (page * Hkv * d) + 5
    kc, vc = dtlib.new_paged_cache(pages, Hkv, page, d)
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v = (torch.randn(4, Hkv, d, generator=g, device="cuda").to(BF) for _ in range(2))
    slots = torch.tensor([pages * page - 1, (pages - 2) * page, 0, 5], dtype=torch.int32, device="cuda")
    dtlib.dt_kv_append(k, v, kc, vc, slots)
    at, row = slots.long() // page, slots.long() % page
    assert torch.equal(kc[at, :, row], k) and torch.equal(vc[at, :, row], v)


def test_append_refuses(dtlib):
    q, k, v, kc, vc, slots, positions = make(6, 4, 2, 64, 16, 64)
    table = dtlib.rope_table(100, 64)
    with pytest.raises(ValueError):
        dtlib.dt_kv_append(k, v, kc, vc, slots, rope=table)                                    # no positions
    with pytest.raises(ValueError):
        dtlib.dt_kv_append(k, v, kc, vc, slots, out_q=q)                                       # out_q without q
    with pytest.raises(ValueError):
        dtlib.dt_kv_append(k, v[:5], kc, vc, slots)
    with pytest.raises(ValueError):
        dtlib.dt_kv_append(k.transpose(0, 1).contiguous().transpose(0, 1), v, kc, vc, slots)   # heads not dense
    with pytest.raises(ValueError):
        dtlib.dt_kv_append(k, v, kc.transpose(1, 2), vc, slots)
    with pytest.raises(TypeError):
        dtlib.dt_kv_append(k.float(), v, kc, vc, slots)
    with pytest.raises(TypeError):
        dtlib.dt_kv_append(k, v, kc, vc, slots.long())
    with pytest.raises(TypeError):
        dtlib.dt_kv_append(k, v, kc, vc, slots.cpu())
    with pytest.raises(dtlib.DTError):
        dtlib.dt_kv_append(k, v, kc, vc, slots, positions=positions, rope=table[:, :24].contiguous())


def test_append_of_nothing(dtlib):
    _, k, v, kc, vc, slots, _ = make(6, 4, 2, 64, 16, 64)
    a, b = kc.clone(), vc.clone()
    dtlib.dt_kv_append(k[:0], v[:0], kc, vc, slots[:0])
    torch.cuda.synchronize()
    assert torch.equal(a, kc) and torch.equal(b, vc)
