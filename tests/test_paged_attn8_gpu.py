"""dt_paged_attention8 on the GPU against plain attention in 64 bits over the codes times their scales. The pools' rows
that no request uses hold NaN codes, their blocks NaN scales, unused table entries a page that does not exist.

The bound, element by element (attention_ref derives its like for bf16). A rounding is off by at most half a step: 2^-11
of the value in fp16, 2^-8 in bf16, 2^-23 for an fp32 step of the tensor cores, which may cut. With p_j the softmax
weights, w_j = p_j times the scale of value j, c_j its code, A = sum_j p_j |v_j|, T keys:
- a row of q is brought to more than 224 and at most 448 and split into two e4m3 terms. The first is off by at most eight
  steps of the element's eighth bit; that is four bits, so the second is exact unless it falls below e4m3's normal range:
  off by 2^-10 then, which is 2^-17 of the row's largest. A score is d products twice: off by e = scale ((2 d + 4) 2^-23
  sum |q||k| + 2^-17 max|q| sum |k|), a weight by the factor e + 2^-21 (the approximate exponential), and so is the sum
  that divides: 2 (e + 2^-21) A;
- w_j to fp16, products in fp32 before it: (2^-11 + 2^-22) A, and where it is a subnormal number, half a step of 2^-24, the
  largest w that is seen being 2^4 at least: 2^-29 max w sum |c_j|;
- the sums over T keys in fp32: 2 T 2^-23 A; the output's rounding to bf16: 2^-8 |out|."""
import math

import pytest
import torch

import test_paged_attn_gpu as paged
from attention_ref import check

pytestmark = pytest.mark.gpu
BF, F8 = torch.bfloat16, torch.float8_e4m3fn


def coded(x, block, gen=None):
    """x [pages,Hkv,page,d] with NaN where no row is -> codes, scales [pages,Hkv,page/block]. With `gen` the scales are
    no powers of two, and differ by more from block to block."""
    pages, Hkv, page, d = x.shape
    blocks = x.float().view(pages, Hkv, page // block, block, d)
    if gen is not None:
        blocks = blocks * 2 ** torch.randn(pages, Hkv, page // block, 1, 1, generator=gen, device="cuda").mul(2).clamp(-4, 4)
    amax = blocks.nan_to_num(0).abs().amax((3, 4))
    scale = 2.0 ** torch.ceil(torch.log2(amax / 448))
    if gen is not None:
        scale = amax / 448 * (1 + torch.rand(amax.shape, generator=gen, device="cuda"))
    scale = torch.where(amax > 0, scale, math.nan).float()
    return (blocks / scale[..., None, None]).view(pages, Hkv, page, d).to(F8), scale


def values(codes, scale, at, head):
    """The rows of pages `at`, in 64 bits."""
    x = codes.view(torch.uint8)[at, head].view(F8).double()
    s = scale[at, head].double()
    block = x.shape[1] // s.shape[1]
    return (x.view(*s.shape, block, -1) * s[..., None, None]).flatten(0, 2), s.repeat_interleave(block, 1).flatten()


def make8(lens, n, Hq, Hkv, d, page, block, mask="tree", odd=True, seed=5, **kw):
    s = paged.make(lens, n, Hq, Hkv, d, page, mask=mask, seed=seed, **kw)
    g = torch.Generator(device="cuda").manual_seed(seed + 1) if odd else None
    s["kc"], s["ks"] = coded(s["kc"], block, None)
    s["vc"], s["vs"] = coded(s["vc"], block, g)
    if odd:  # keys: scales that are no powers of two
        s["ks"] = s["ks"] * (0.5 + torch.rand(s["ks"].shape, generator=g, device="cuda"))
    return s


def attend8(q, k, v, vs, seen, scale):
    used = seen.any(0)
    q, k, v, vs, seen = q.double(), k[used], v[used], vs[used], seen[:, used]
    if k.shape[0] == 0:
        return torch.zeros_like(q), torch.zeros_like(q)
    z = (q @ k.t() * scale).masked_fill(~seen, -math.inf)
    top = z.amax(1, keepdim=True)
    p = torch.exp(z - torch.where(top == -math.inf, torch.zeros_like(top), top)) * seen
    total = p.sum(1, keepdim=True)
    p = torch.where(total > 0, p / total, torch.zeros_like(p))
    out, A = p @ v, p @ v.abs()
    d, T = q.shape[1], k.shape[0]
    e = scale * ((2 * d + 4) * 2.0 ** -23 * (q.abs() @ k.abs().t()) +
                 2.0 ** -17 * q.abs().amax(1, keepdim=True) * k.abs().sum(1)).mul(seen).amax(1, keepdim=True)
    floor = 2.0 ** -29 * (p * vs).amax(1, keepdim=True) * (seen.double() @ (v.abs() / vs[:, None]))
    return out, A * (2 * (e + 2.0 ** -21) + 2.0 ** -11 + 2.0 ** -22 + 2 * T * 2.0 ** -23) + floor + 2.0 ** -8 * out.abs()


def reference(s, b, head):
    n, Hq = s["q"].shape[1:3]
    Hkv, page, d = s["kc"].shape[1:]
    length = int(s["lens"][b])
    at = s["table"][b, :-(-length // page)].long()
    (k, _), (v, vs) = (values(s[c], s[x], at, head // (Hq // Hkv)) for c, x in (("kc", "ks"), ("vc", "vs")))
    tree = s["mask"][b] != 0 if s["mask"] is not None else torch.ones(n, n, dtype=torch.bool, device="cuda").tril()
    seen = torch.cat([torch.ones(n, length - n, dtype=torch.bool, device="cuda"), tree], 1)
    return attend8(s["q"][b, :, head], k[:length], v[:length], vs[:length], seen, s["scale"])


def run(dtlib, s, **kw):
    return dtlib.dt_paged_attention8(s["q"], s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["lens"], s["scale"],
                                     mask=s["mask"], **kw)


def room(dtlib, s):
    B, n, Hq, d = s["q"].shape
    return dtlib.new_workspace(dtlib.dt_paged_attention8_workspace_bytes(B, n, Hq, s["kc"].shape[1], d))


def parity(dtlib, s, requests=None, heads=None):
    B, n, Hq, d = s["q"].shape
    ws = room(dtlib, s)
    out = torch.full((B, n, Hq, d), float("nan"), dtype=BF, device="cuda")
    run(dtlib, s, out=out, workspace=ws)
    assert dtlib.dt_get_error(ws) == dtlib.Status.OK
    for b in requests if requests is not None else range(B):
        if s["lens"][b] <= 0:
            assert (out[b] == 0).all(), b
            continue
        for h in heads if heads is not None else range(Hq):
            check(out[b, :, h], *reference(s, b, h))
    again = torch.zeros_like(out)
    run(dtlib, s, out=again, workspace=ws)  # the workspace is ready for the next call, and the result is the same
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))
    return out


@pytest.mark.parametrize("lens,Hq,Hkv,d,page,block", [
    ([1], 1, 1, 64, 8, 8),                                   # one key
    ([1, 2, 63, 64, 65, 127, 128, 129], 8, 2, 128, 16, 8),   # around the blocks' borders
    ([200, 0, 7, -3, 1, 0], 8, 2, 64, 32, 16),               # unused rows of the batch
    ([0, 0, 0], 4, 4, 128, 16, 16),                          # nothing but unused rows
    ([2049], 32, 8, 128, 64, 64),
    ([30000], 8, 1, 128, 64, 16),                            # one head over every CTA
    ([20011, 3, 700], 16, 16, 64, 128, 128),
    ([777, 1500, 12], 40, 8, 128, 256, 256),
    ([777, 1500, 12], 40, 8, 128, 256, 8),
    ([513] * 3, 64, 1, 128, 8, 8),                           # 64 heads on one, the smallest pages
    ([300, 41], 128, 1, 64, 16, 16),                         # every query row
    ([300, 41], 100, 1, 128, 32, 8),
    ([500, 90], 12, 2, 64, 16, 8),
    ([1000, 64], 17, 17, 128, 32, 32),
    ([1000, 64, 333], 20, 1, 64, 64, 32),                    # 20 rows
    ([1000, 64, 333], 33, 1, 64, 64, 32),
])
def test_one_new_token(dtlib, lens, Hq, Hkv, d, page, block):
    parity(dtlib, make8(lens, 1, Hq, Hkv, d, page, block, mask=None))


@pytest.mark.parametrize("lens,n,Hq,Hkv,d,page,mask", [
    ([16, 17, 100], 16, 32, 8, 128, 16, "tree"),      # no prefix, a prefix of one, 64 rows
    ([64 + 16, 64 + 5, 128 + 10], 16, 32, 8, 128, 64, "tree"),   # trees across the blocks' borders
    ([2064], 16, 32, 8, 128, 64, "tree"),
    ([333, 70], 32, 32, 8, 128, 16, "tree"),          # 128 rows
    ([333, 64], 64, 4, 2, 64, 32, "tree"),            # 64 nodes, 128 rows
    ([333, 65, 64], 64, 2, 2, 128, 16, None),         # causal among 64
    ([40, 5], 5, 12, 2, 64, 8, None),
    ([16, 300, 90], 16, 8, 2, 128, 16, "random"),     # a node that sees nothing at all where there is no prefix
    ([3, 50], 3, 8, 2, 64, 16, "random"),
    ([2, 129, 64], 2, 2, 2, 128, 16, "random"),
    ([9, 0, 800], 7, 14, 2, 64, 128, "tree"),
    ([5000], 3, 40, 8, 128, 16, "tree"),
    ([1, 40], 1, 8, 2, 128, 16, "random"),            # one token whose mask hides itself
])
@pytest.mark.parametrize("odd", [False, True])
def test_tree_nodes(dtlib, lens, n, Hq, Hkv, d, page, mask, odd):
    parity(dtlib, make8(lens, n, Hq, Hkv, d, page, min(page, 16), mask=mask, odd=odd))


def test_a_node_without_visible_keys_is_zero(dtlib):
    s = make8([4, 4], 4, 8, 2, 128, 16, 16)
    s["mask"][1, 2] = 0
    out = parity(dtlib, s)
    assert (out[1, 2] == 0).all() and (out[1, 1] != 0).any()


def test_many_requests(dtlib):
    """More (request, head) pairs than CTAs, all lengths different, unused rows in between; sampled requests."""
    lens = [(37 * i) % 900 if i % 11 else 0 for i in range(500)]
    parity(dtlib, make8(lens, 1, 8, 2, 128, 16, 16, mask=None), requests=[0, 1, 2, 11, 100, 257, 498, 499])


@pytest.mark.parametrize("n", [1, 6])
def test_long_contexts(dtlib, n):
    parity(dtlib, make8([100003, 40, 65536], n, 16, 2, 128, 64, 16), heads=[0, 7, 8, 15])


def test_shared_pages(dtlib):
    """Two requests with the same first pages."""
    s = make8([200, 150], 1, 8, 2, 128, 32, 16, mask=None)
    s["table"][1, :4] = s["table"][0, :4]
    parity(dtlib, s)


def test_scales_at_the_ends_of_their_range(dtlib):
    """Blocks of keys and values whose scales lie at 2^-48, 2^48 and in between, in one request."""
    s = make8([600, 300], 2, 8, 2, 128, 16, 16, odd=False)
    g = torch.Generator(device="cuda").manual_seed(8)
    e = torch.randint(-48, 49, s["vs"].shape, generator=g, device="cuda")
    s["vs"] = torch.where(s["vs"].isnan(), s["vs"], 2.0 ** e)
    parity(dtlib, s)
    for e in (-48, 48):
        s["vs"] = torch.where(s["vs"].isnan(), s["vs"], 2.0 ** e)
        parity(dtlib, s)
    s["ks"] = torch.where(s["ks"].isnan(), s["ks"], 2.0 ** -48)  # every score is nearly zero: the plain mean
    parity(dtlib, s)


def test_rows_of_queries_of_very_different_sizes(dtlib):
    """One head's queries are 10^30 times another's, one all zero, one with elements 2^-40 below its largest."""
    s = make8([400, 90], 3, 8, 2, 128, 16, 16)
    q = s["q"].float()
    q[:, :, 1] *= 1e-30
    q[:, :, 2] = 0
    q[:, 1, 3, ::2] *= 2.0 ** -40
    q[:, :, 5] *= 1e-5
    s["q"] = q.to(BF)
    parity(dtlib, s)


def test_a_row_that_is_not_finite_leaves_the_others_alone(dtlib):
    s = make8([400, 90], 3, 8, 2, 128, 16, 16)
    want = run(dtlib, s).clone()
    s["q"][0, 1, 2, 5], s["q"][1, 0, 7, 100] = float("nan"), float("inf")
    got = run(dtlib, s)
    assert got[0, 1, 2].isnan().all() and got[1, 0, 7].isnan().all()
    got[0, 1, 2], got[1, 0, 7] = want[0, 1, 2], want[1, 0, 7]
    assert torch.equal(got, want)


def test_late_keys_above_all_before_them(dtlib):
    """Scores that rise along the cache, past the headroom block after block: the sums are scaled down again and again."""
    s = make8([1500, 700], 1, 8, 2, 128, 16, 16, mask=None)
    at = s["table"][0, :94].long()
    rise = torch.linspace(0.02, 3, 94, device="cuda")
    s["ks"][at] = s["ks"][at] * rise[:, None, None]
    s["q"] = (s["q"].float() * 4).to(BF)
    parity(dtlib, s)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [2, 3, 4, 8, 16, 32])
def test_late_keys_above_all_before_them_for_any_rows(dtlib, n, d):
    """The same under trees of 8 to 128 rows a head, and in some heads' rows alone."""
    s = make8([1500, 700], n, 8, 2, d, 16, 16)
    at = s["table"][0, :94].long()
    s["ks"][at] = s["ks"][at] * torch.linspace(0.02, 3, 94, device="cuda")[:, None, None]
    q = s["q"].float()
    q[:, :, ::3] *= 4
    s["q"] = q.to(BF)
    parity(dtlib, s, requests=[0, 1], heads=[0, 1, 3, 6])


@pytest.mark.parametrize("lens,n,Hq,Hkv,d,page", [
    ([20011, 70, 9000], 64, 4, 2, 128, 16),        # 128 rows, one pair over many CTAs
    ([20011, 16, 9000, 400], 16, 32, 8, 128, 64),  # 64 rows, several segments a CTA
    ([6001, 8, 250], 8, 8, 2, 64, 8),              # 32 rows, the smallest pages
    ([9001, 4, 129], 4, 16, 4, 64, 8),             # 16 rows
])
def test_long_contexts_under_trees(dtlib, lens, n, Hq, Hkv, d, page):
    parity(dtlib, make8(lens, n, Hq, Hkv, d, page, 8), heads=[0, Hq - 1])


def test_the_largest_batch(dtlib):
    """As many requests as there may be, most of them short, some unused: segments that are parts of a block's worth."""
    lens = [(i * 53) % 190 + 1 if i % 7 else 0 for i in range(2048)]
    lens[1000] = 4000
    parity(dtlib, make8(lens, 1, 8, 4, 64, 16, 16, mask=None), requests=[0, 1, 6, 999, 1000, 1001, 2046, 2047])


def test_two_calls_at_once(dtlib):
    """Two streams, a workspace each: a long call and many short ones beside it."""
    a, b = make8([60000, 31000], 3, 16, 2, 128, 64, 16), make8([700] * 9, 16, 8, 2, 64, 16, 16)
    rooms = [room(dtlib, s) for s in (a, b)]
    want = run(dtlib, a).clone(), run(dtlib, b).clone()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], [[], []]
    torch.cuda.synchronize()
    for _ in range(6):
        for i, s in enumerate((a, b)):
            with torch.cuda.stream(streams[i]):
                got[i].append(run(dtlib, s, workspace=rooms[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(x, want[i]) for x in got[i]) and dtlib.dt_get_error(rooms[i]) == dtlib.Status.OK


def nan_code(s, name, b, token, head, column):
    page = int(s["table"][b, token // s["kc"].shape[2]])
    s[name].view(torch.uint8)[page, head, token % s["kc"].shape[2], column] = 0x7F


@pytest.mark.parametrize("d", [64, 128])
def test_codes_that_are_nan_reach_those_that_see_them(dtlib, d):
    """A NaN among the nodes' keys or values, and in the prefix."""
    s = make8([300, 90, 513], 6, 8, 2, d, 16, 16)
    want = run(dtlib, s).clone()
    nan_code(s, "vc", 0, 296, 1, d - 3)   # node 2 of request 0
    nan_code(s, "kc", 1, 85, 0, 7)        # node 1 of request 1
    nan_code(s, "vc", 2, 100, 0, 5)       # request 2's prefix: every node sees it
    got = run(dtlib, s)
    sees = s["mask"] != 0
    for i in range(6):
        for h in range(8):
            g, w = got[0, i, h].clone(), want[0, i, h]
            if h >= 4 and sees[0, i, 2]:
                assert g[d - 3].isnan()
                g[d - 3] = w[d - 3]
            assert torch.equal(g, w)
            if h < 4 and sees[1, i, 1]:
                assert got[1, i, h].isnan().all()
            else:
                assert torch.equal(got[1, i, h], want[1, i, h])
            g, w = got[2, i, h].clone(), want[2, i, h]
            if h < 4:
                assert g[5].isnan()
                g[5] = w[5]
            assert torch.equal(g, w)


def test_a_block_of_zeros_and_scales_of_zero(dtlib):
    s = make8([100], 1, 4, 1, 64, 16, 16, mask=None, odd=False)
    page = int(s["table"][0, 2])
    s["vc"].view(torch.uint8)[page] = 0
    s["kc"].view(torch.uint8)[page] = 0x80  # minus zero
    s["vs"][page] = s["ks"][page] = 2.0 ** -48
    parity(dtlib, s)


def test_far_into_a_large_pool(dtlib):
    """Pages whose bytes lie past 2^32 of the pool, scales past 2^27."""
    page, Hkv, d = 256, 8, 128
    pages = 2 ** 32 // (page * Hkv * d) + 9
    kc, vc, ks, vs = dtlib.new_paged_cache8(pages, Hkv, page, d, scale_block=8)
    s = make8([700, 256], 1, 16, 8, d, page, 8, mask=None)
    to = torch.tensor([pages - 1 - 2 * i for i in range(s["kc"].shape[0])], device="cuda")
    for big, name in ((kc, "kc"), (vc, "vc")):
        big.view(torch.uint8)[to] = s[name].view(torch.uint8)
        s[name] = big
    for big, name in ((ks, "ks"), (vs, "vs")):
        big[to] = s[name]
        s[name] = big
    s["table"] = torch.where(s["table"] >= 0, to[s["table"].long().clamp(min=0)].to(torch.int32), -7)
    parity(dtlib, s, heads=[0, 1, 15])


def test_bad_lengths_and_pages_are_reported(dtlib):
    s = make8([100, 50, 30], 2, 4, 2, 64, 16, 16)
    ws = room(dtlib, s)
    want = run(dtlib, s).clone()
    for spoil in (1, s["table"].shape[1] * 16 + 1):  # fewer than the nodes, more than the table holds
        s["lens"][1] = spoil
        got = run(dtlib, s, workspace=ws)
        assert dtlib.dt_get_error(ws) == dtlib.Status.INVALID_ARG
        assert (got[1] == 0).all() and torch.equal(got[[0, 2]], want[[0, 2]])
    s["lens"][1] = 50
    for page in (-1, s["kc"].shape[0], 2 ** 31 - 1):
        keep = int(s["table"][0, 3])
        s["table"][0, 3] = page
        got = run(dtlib, s, workspace=ws)
        assert dtlib.dt_get_error(ws) == dtlib.Status.INVALID_ARG
        assert torch.equal(got[1:], want[1:])
        s["table"][0, 3] = keep
    assert torch.equal(run(dtlib, s, workspace=ws), want) and dtlib.dt_get_error(ws) == dtlib.Status.OK


def test_on_another_stream_and_captured(dtlib):
    s = make8([3000, 40, 700], 4, 16, 2, 128, 16, 16)
    want = run(dtlib, s).clone()
    side, q0 = torch.cuda.Stream(), s["q"].clone()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = run(dtlib, s)
    side.synchronize()
    assert torch.equal(got, want)
    assert torch.equal(run(dtlib, s, stream=side), want) or side.synchronize() is None
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        a = run(dtlib, s)
    for _ in range(3):
        s["q"].zero_(), a.fill_(float("nan"))
        s["q"].copy_(q0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(a, want)


def test_two_graphs_share_a_workspace_in_turn(dtlib):
    """Cut pairs leave the tickets at zero: another shape finds them so."""
    a, b = make8([9000, 5000], 1, 8, 1, 128, 64, 16, mask=None), make8([700] * 9, 3, 8, 2, 64, 16, 16)
    ws = dtlib.new_workspace(max(room(dtlib, a).numel(), room(dtlib, b).numel()))
    want = run(dtlib, a).clone(), run(dtlib, b).clone()
    graphs = []
    for s in (a, b):
        s["out"] = torch.empty_like(s["q"])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run(dtlib, s, out=s["out"], workspace=ws)
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert torch.equal(a["out"], want[0]) and torch.equal(b["out"], want[1])
    assert dtlib.dt_get_error(ws) == dtlib.Status.OK


def test_refuses(dtlib):
    s = make8([40, 20], 2, 8, 2, 128, 16, 8)
    call = lambda **kw: run(dtlib, {**s, **kw})
    with pytest.raises(TypeError):
        call(kc=s["kc"].view(torch.uint8))
    with pytest.raises(TypeError):
        call(vs=s["vs"].half())
    with pytest.raises(ValueError):
        call(ks=s["ks"][:, :, :1].contiguous())          # another block than the values'
    with pytest.raises(ValueError):
        call(ks=s["ks"][:, :1].contiguous())
    with pytest.raises(ValueError):
        call(ks=torch.cat([s["ks"], s["ks"][:, :, :1]], 2))
    with pytest.raises(ValueError):
        call(vc=s["vc"][..., :64].contiguous())
    with pytest.raises(TypeError):
        call(q=s["q"].float())
    with pytest.raises(TypeError):
        call(lens=s["lens"].long())
    with pytest.raises(dtlib.DTError):
        call(scale=0.0)
    four = lambda x: x.repeat_interleave(2, 2)  # a scale for each four rows
    with pytest.raises(dtlib.DTError):
        call(ks=four(s["ks"]), vs=four(s["vs"]))
