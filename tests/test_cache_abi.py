"""The paged cache's entry points reject bad arguments on the host, before anything is launched (no GPU needed)."""
import pytest
import torch

OK, INVALID, UNSUPPORTED = 0, 1, 2
A = 1 << 20  # a 16-byte-aligned fake device address: validation must reject before any dereference
BF16, F32 = 1, 0


def test_append_rejects_bad_arguments(dtlib):
    f = dtlib.lib().dt_kv_append

    def call(N=4, Hq=8, Hkv=2, d=128, q=A, qs=1536, k=A, ks=1536, v=A, vs=1536, dtype=BF16, slots=A, pos=A, rope=A,
             max_pos=100, rot=128, inter=0, out_q=A, out_k=A, kc=A, vc=A, pages=4, page=16, ws=A, wsb=256):
        return f(N, Hq, Hkv, d, q, qs, k, ks, v, vs, dtype, slots, pos, rope, max_pos, rot, inter, out_q, out_k, kc,
                 vc, pages, page, ws, wsb, None)
    for bad in [dict(N=-1), dict(Hq=-1), dict(Hkv=0), dict(d=0), dict(pages=0), dict(page=0), dict(rot=-2),
                dict(rot=130), dict(rot=7), dict(dtype=7), dict(inter=2), dict(q=None), dict(out_q=None),
                dict(Hq=0), dict(k=None), dict(v=None), dict(kc=None), dict(vc=None), dict(ws=None), dict(slots=None),
                dict(pos=None), dict(rope=None), dict(max_pos=0), dict(k=A + 8), dict(v=A + 2), dict(q=A + 4),
                dict(out_k=A + 8), dict(rope=A + 4), dict(slots=A + 2), dict(pos=A + 1), dict(wsb=128),
                dict(ks=248), dict(vs=260), dict(qs=1020), dict(ks=1 << 40)]:
        assert call(**bad) == INVALID, bad
    for big in [dict(dtype=F32), dict(d=96, rot=96), dict(rot=24), dict(page=24), dict(page=4), dict(page=512),
                dict(pages=1 << 28, page=16), dict(Hkv=300, ks=38400, vs=38400), dict(N=(1 << 31) - 1)]:
        assert call(**big) == UNSUPPORTED, big
    assert call(N=0) == OK                                                    # nothing to do, nothing launched
    assert call(N=0, Hq=0, q=None, out_q=None) == OK
    assert call(N=0, rot=0, rope=None, pos=None, max_pos=0) == OK


def test_paged_attention_rejects_bad_arguments(dtlib):
    f = dtlib.lib().dt_paged_attention

    def call(B=2, n=1, Hq=8, Hkv=2, d=128, q=A, kc=A, vc=A, dtype=BF16, pages=4, page=16, table=A, width=4, lens=A,
             mask=None, scale=0.1, out=A, ws=A, wsb=1 << 30):
        return f(B, n, Hq, Hkv, d, q, kc, vc, dtype, pages, page, table, width, lens, mask, scale, out, ws, wsb, None)
    for bad in [dict(B=-1), dict(n=0), dict(Hq=0), dict(Hq=7), dict(Hkv=0), dict(d=0), dict(pages=0), dict(page=0),
                dict(width=0), dict(dtype=9), dict(scale=0.0), dict(scale=-1.0), dict(scale=3e38),
                dict(scale=float("nan")),
                dict(scale=float("inf")), dict(q=None), dict(q=A + 8), dict(kc=None), dict(vc=A + 4), dict(out=None),
                dict(ws=A + 8), dict(table=None), dict(lens=None), dict(table=A + 2), dict(lens=A + 1)]:
        assert call(**bad) == INVALID, bad
    for big in [dict(dtype=F32), dict(d=96), dict(d=256), dict(n=65, Hq=2), dict(n=33), dict(B=2049), dict(page=24),
                dict(page=4), dict(page=512), dict(pages=1 << 28, page=16), dict(width=1 << 21, page=16),
                dict(Hq=300, Hkv=300), dict(pages=1 << 27, page=8, Hq=64, Hkv=32)]:
        assert call(**big) == UNSUPPORTED, big
    assert call(B=0) == OK


def test_prompt_attention_rejects_bad_arguments(dtlib):
    f = dtlib.lib().dt_prompt_attention

    def call(total=300, B=2, Hq=8, Hkv=2, d=128, q=A, qs=1024, k=A, ks=256, v=A, vs=256, dtype=BF16, cu=A, scale=0.1,
             out=A, ws=A, wsb=256):
        return f(total, B, Hq, Hkv, d, q, qs, k, ks, v, vs, dtype, cu, scale, out, ws, wsb, None)
    for bad in [dict(total=-1), dict(B=-1), dict(Hq=0), dict(Hq=7), dict(Hkv=0), dict(d=0), dict(dtype=9),
                dict(scale=0.0), dict(scale=float("nan")), dict(q=None), dict(k=None), dict(v=A + 8), dict(out=None),
                dict(out=A + 2), dict(ws=None), dict(cu=None), dict(cu=A + 2), dict(wsb=64), dict(qs=1016),
                dict(ks=260), dict(vs=1 << 33)]:
        assert call(**bad) == INVALID, bad
    for big in [dict(dtype=F32), dict(d=96), dict(d=256, qs=2048, ks=512, vs=512),
                dict(Hq=300, Hkv=300, qs=38400, ks=38400, vs=38400), dict(total=(1 << 31) - 1),
                dict(B=1 << 23, Hq=256, qs=32768)]:
        assert call(**big) == UNSUPPORTED, big
    assert call(total=0) == OK
    assert call(B=0) == OK


def test_workspace_sizes_of_empty_or_unsupported_shapes(dtlib):
    L = dtlib.lib()
    for args in [(0, 1, 8, 2, 128), (1, 0, 8, 2, 128), (1, 1, 7, 2, 128), (1, 1, 8, 0, 128), (1, 1, 8, 2, 0),
                 (1, 40, 8, 2, 128)]:
        assert L.dt_paged_attention_workspace_bytes(*args) == 0, args
    for args in [(0, 1, 8, 2, 128), (9, 0, 8, 2, 128), (9, 1, 7, 2, 128), (9, 1, 8, 2, 0)]:
        assert L.dt_prompt_attention_workspace_bytes(*args) == 0, args
    assert L.dt_prompt_attention_workspace_bytes(9, 1, 8, 2, 128) >= 256


def test_binding_refuses_host_tensors(dtlib):
    bf, i32 = torch.bfloat16, torch.int32
    q, k, cache = torch.zeros(2, 4, 64, dtype=bf), torch.zeros(2, 1, 64, dtype=bf), torch.zeros(3, 1, 16, 64, dtype=bf)
    ints = torch.zeros(3, dtype=i32)
    with pytest.raises(TypeError):
        dtlib.dt_kv_append(k, k, cache, cache, ints[:2])
    with pytest.raises(TypeError):
        dtlib.dt_paged_attention(q[None], cache, cache, ints[None], ints[:1], 0.1)
    with pytest.raises(TypeError):
        dtlib.dt_prompt_attention(q, k, k, ints, 0.1)


def test_rope_table(dtlib):
    t = dtlib.rope_table(5, 8, 100.0, device="cpu")
    assert t.shape == (5, 8) and t.dtype == torch.float32
    assert torch.equal(t[0], torch.tensor([1.0] * 4 + [0.0] * 4))
    angle = torch.tensor(3.0, dtype=torch.float64) * 100.0 ** (-2 / 8)
    assert t[3, 1] == angle.cos().float() and t[3, 5] == angle.sin().float()
