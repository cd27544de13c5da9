"""The page plan's and the 8-bit cache's entry points reject bad arguments on the host, before anything is launched (no
GPU needed)."""
import pytest
import torch

OK, INVALID, UNSUPPORTED = 0, 1, 2
A = 1 << 20  # a 16-byte-aligned fake device address: validation must reject before any dereference
BF16, F32 = 1, 0


def test_plan_rejects_bad_arguments(dtlib):
    f = dtlib.lib().dt_page_plan

    def call(B=4, n=0, N=30, page=16, pages=40, width=10, lens=A, grow=A, depth=None, path=None, table=A, held=A, free=A,
             count=A, out=A, cu=A, slots=A, pos=A, ws=A, wsb=1 << 20):
        return f(B, n, N, page, pages, width, lens, grow, depth, path, table, held, free, count, out, cu, slots, pos, ws,
                 wsb, None)
    for bad in [dict(B=-1), dict(n=-1), dict(N=-1), dict(page=0), dict(pages=0), dict(width=0), dict(depth=A),
                dict(path=A), dict(n=5, N=20, depth=A, path=A), dict(n=5), dict(n=5, N=19), dict(slots=None),
                dict(pos=None), dict(slots=None, pos=None), dict(held=None), dict(free=None), dict(count=None),
                dict(held=None, free=None), dict(lens=None), dict(grow=None), dict(table=None), dict(lens=A + 2),
                dict(grow=A + 1), dict(n=5, N=20, depth=A + 2), dict(n=5, N=20, path=A + 2), dict(table=A + 2),
                dict(held=A + 2), dict(free=A + 1), dict(count=A + 2), dict(out=A + 2), dict(cu=A + 1),
                dict(slots=A + 2), dict(pos=A + 2), dict(ws=None), dict(ws=A + 8), dict(wsb=128)]:
        assert call(**bad) == INVALID, bad
    for big in [dict(B=2049), dict(N=(1 << 31) - 1), dict(page=4), dict(page=512), dict(page=24),
                dict(pages=1 << 28), dict(width=1 << 21)]:
        assert call(**big) == UNSUPPORTED, big
    assert call(B=0, N=0, slots=None, pos=None) == OK
    assert call(B=0, N=0, lens=None, grow=None, table=None) == OK


def test_append_rejects_bad_arguments(dtlib):
    f = dtlib.lib().dt_kv_append8

    def call(N=4, Hq=8, Hkv=2, d=128, q=A, qs=1536, k=A, ks=1536, v=A, vs=1536, dtype=BF16, slots=A, pos=A, rope=A,
             max_pos=100, rot=128, inter=0, out_q=A, out_k=A, kc=A, vc=A, ksc=A, vsc=A, pages=4, page=16, block=16, ws=A,
             wsb=256):
        return f(N, Hq, Hkv, d, q, qs, k, ks, v, vs, dtype, slots, pos, rope, max_pos, rot, inter, out_q, out_k, kc,
                 vc, ksc, vsc, pages, page, block, ws, wsb, None)
    for bad in [dict(N=-1), dict(Hq=-1), dict(Hkv=0), dict(d=0), dict(pages=0), dict(page=0), dict(block=0), dict(rot=-2),
                dict(rot=130), dict(rot=7), dict(dtype=7), dict(inter=2), dict(q=None), dict(out_q=None),
                dict(Hq=0), dict(k=None), dict(v=None), dict(kc=None), dict(vc=None), dict(ksc=None), dict(vsc=None),
                dict(ksc=A + 2), dict(vsc=A + 1), dict(ws=None), dict(slots=None),
                dict(pos=None), dict(rope=None), dict(max_pos=0), dict(k=A + 8), dict(v=A + 2), dict(q=A + 4),
                dict(out_k=A + 8), dict(rope=A + 4), dict(slots=A + 2), dict(pos=A + 1), dict(wsb=128),
                dict(ks=248), dict(vs=260), dict(qs=1020), dict(ks=1 << 40), dict(N=100000, wsb=256),
                dict(N=100000, wsb=256 + 4 * 63)]:
        assert call(**bad) == INVALID, bad
    for big in [dict(dtype=F32), dict(d=96, rot=96), dict(rot=24), dict(page=24), dict(page=4, block=4), dict(page=512),
                dict(block=4), dict(block=12), dict(block=32), dict(pages=1 << 28, page=16),
                dict(Hkv=300, ks=38400, vs=38400), dict(N=(1 << 31) - 1), dict(pages=1 << 24, page=8, block=8, Hkv=256,
                                                                              ks=32768, vs=32768)]:
        assert call(**big) == UNSUPPORTED, big
    assert call(N=0) == OK                                                    # nothing to do, nothing launched
    assert call(N=0, Hq=0, q=None, out_q=None) == OK
    assert call(N=0, rot=0, rope=None, pos=None, max_pos=0) == OK


def test_attention_rejects_bad_arguments(dtlib):
    f = dtlib.lib().dt_paged_attention8

    def call(B=2, n=1, Hq=8, Hkv=2, d=128, q=A, kc=A, vc=A, ks=A, vs=A, dtype=BF16, pages=4, page=16, block=16, table=A,
             width=4, lens=A, mask=None, scale=0.1, out=A, ws=A, wsb=1 << 30):
        return f(B, n, Hq, Hkv, d, q, kc, vc, ks, vs, dtype, pages, page, block, table, width, lens, mask, scale, out, ws,
                 wsb, None)
    for bad in [dict(B=-1), dict(n=0), dict(Hq=0), dict(Hq=7), dict(Hkv=0), dict(d=0), dict(pages=0), dict(page=0),
                dict(block=0), dict(width=0), dict(dtype=9), dict(scale=0.0), dict(scale=-1.0), dict(scale=3e38),
                dict(scale=float("nan")), dict(scale=float("inf")), dict(q=None), dict(q=A + 8), dict(kc=None),
                dict(vc=A + 4), dict(ks=None), dict(vs=None), dict(ks=A + 2), dict(vs=A + 1), dict(out=None),
                dict(ws=A + 8), dict(table=None), dict(lens=None), dict(table=A + 2), dict(lens=A + 1)]:
        assert call(**bad) == INVALID, bad
    for big in [dict(dtype=F32), dict(d=96), dict(d=256), dict(n=65, Hq=2), dict(n=33), dict(B=2049), dict(page=24),
                dict(page=4, block=4), dict(page=512), dict(block=4), dict(block=32), dict(block=12),
                dict(pages=1 << 28, page=16), dict(width=1 << 21, page=16), dict(Hq=300, Hkv=300),
                dict(pages=1 << 27, page=8, block=8, Hq=64, Hkv=32)]:
        assert call(**big) == UNSUPPORTED, big
    assert call(B=0) == OK


def test_workspace_sizes_of_empty_or_unsupported_shapes(dtlib):
    L = dtlib.lib()
    assert L.dt_page_plan_workspace_bytes(0) == 0 and L.dt_page_plan_workspace_bytes(2049) == 0
    assert L.dt_page_plan_workspace_bytes(1) >= 256
    assert L.dt_kv_append8_workspace_bytes(-1, 4, 16) == 0 and L.dt_kv_append8_workspace_bytes(5, 0, 16) == 0
    assert L.dt_kv_append8_workspace_bytes(5, 4, 16) == 256
    assert L.dt_kv_append8_workspace_bytes(100000, 1 << 20, 64) >= 4 << 26
    for args in [(0, 1, 8, 2, 128), (1, 0, 8, 2, 128), (1, 1, 7, 2, 128), (1, 1, 8, 0, 128), (1, 1, 8, 2, 0),
                 (1, 40, 8, 2, 128)]:
        assert L.dt_paged_attention8_workspace_bytes(*args) == 0, args


def test_binding_refuses_host_tensors(dtlib):
    bf, i32, f8 = torch.bfloat16, torch.int32, torch.float8_e4m3fn
    q, k = torch.zeros(2, 4, 64, dtype=bf), torch.zeros(2, 1, 64, dtype=bf)
    cache, scale = torch.zeros(3, 1, 16, 64).to(f8), torch.zeros(3, 1, 1)
    ints = torch.zeros(3, dtype=i32)
    with pytest.raises(TypeError):
        dtlib.dt_page_plan(ints, ints, ints[None], 16, 3)
    with pytest.raises(TypeError):
        dtlib.dt_kv_append8(k, k, cache, cache, scale, scale, ints[:2])
    with pytest.raises(TypeError):
        dtlib.dt_paged_attention8(q[None], cache, cache, scale, scale, ints[None], ints[:1], 0.1)


def test_new_cache(dtlib):
    kc, vc, ks, vs = dtlib.new_paged_cache8(5, 2, 64, 128, scale_block=32, device="cpu")
    assert kc.shape == vc.shape == (5, 2, 64, 128) and kc.dtype == vc.dtype == torch.float8_e4m3fn
    assert ks.shape == vs.shape == (5, 2, 2) and ks.dtype == torch.float32 and not ks.any() and not vs.any()


def test_a_plan_without_requests_holds_nothing(dtlib):
    """No requests: an array of what each holds may have no address, with a pool as without one."""
    f = dtlib.lib().dt_page_plan

    def call(free=A, count=A):
        return f(0, 0, 0, 16, 40, 10, None, None, None, None, None, None, free, count, None, None, None, None, A, 1 << 20,
                 None)
    assert call() == OK
    assert call(free=None, count=None) == OK
    assert call(free=None) == INVALID and call(count=None) == INVALID


def test_new_cache_refuses_blocks_that_do_not_fill_a_page(dtlib):
    for page, block in ((64, 48), (16, 12), (16, 32), (16, 0), (16, -4)):
        with pytest.raises(ValueError):
            dtlib.new_paged_cache8(5, 2, page, 128, scale_block=block, device="cpu")
