"""dt_paged_attention on the GPU against plain attention in 64 bits, one head at a time (attention_ref: the bound is
derived there). The pools' rows that no request uses hold NaN, unused table entries a page that does not exist."""
import math

import pytest
import torch

from attention_ref import attend, check

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def make(lens, n, Hq, Hkv, d, page, mask="tree", seed=5, pages=None, spread=1.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")
    B = len(lens)
    used = [-(-max(x, 0) // page) for x in lens]
    pages = pages or sum(used) + 2
    kc, vc = (torch.full((pages, Hkv, page, d), float("nan"), dtype=BF, device="cuda") for _ in range(2))
    order = (pages - 1 - torch.randperm(sum(used) + 2, generator=g, device="cuda")).tolist()
    table = torch.full((B, max(used + [1]) + 1), -7, dtype=torch.int32)
    for b, x in enumerate(lens):
        for i in range(used[b]):
            at, rows = order.pop(), min(page, x - i * page)
            table[b, i] = at
            kc[at, :, :rows] = rnd(Hkv, rows, d).to(BF)
            vc[at, :, :rows] = rnd(Hkv, rows, d).to(BF)
    q = (rnd(B, n, Hq, d) * spread).to(BF)
    m = None
    if mask == "tree":
        m = torch.zeros(B, n, n, dtype=torch.uint8)
        pick = torch.rand(B, n, generator=g, device="cuda").cpu()
        for b in range(B):
            for i in range(n):
                parent = int(pick[b, i] * (i + 1)) - 1
                m[b, i, i] = 1
                if parent >= 0:
                    m[b, i] |= m[b, parent]
    elif mask == "random":  # any bytes: rows without a visible node among them
        m = (torch.rand(B, n, n, generator=g, device="cuda").cpu() < 0.3).to(torch.uint8) * 3
        m[:, n // 2] = 0
    return dict(q=q, kc=kc, vc=vc, table=table.cuda(), lens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
                mask=m.cuda() if m is not None else None, scale=1 / math.sqrt(d))


def reference(s, b, head):
    n, Hq = s["q"].shape[1:3]
    Hkv, page, d = s["kc"].shape[1:]
    length = int(s["lens"][b])
    at = s["table"][b, :-(-length // page)].long()
    k, v = (c[at, head // (Hq // Hkv)].reshape(-1, d)[:length] for c in (s["kc"], s["vc"]))
    tree = s["mask"][b] != 0 if s["mask"] is not None else torch.ones(n, n, dtype=torch.bool, device="cuda").tril()
    seen = torch.cat([torch.ones(n, length - n, dtype=torch.bool, device="cuda"), tree], 1)
    return attend(s["q"][b, :, head], k, v, seen, s["scale"])


def run(dtlib, s, **kw):
    return dtlib.dt_paged_attention(s["q"], s["kc"], s["vc"], s["table"], s["lens"], s["scale"], mask=s["mask"], **kw)


def parity(dtlib, s, requests=None, heads=None):
    B, n, Hq, d = s["q"].shape
    ws = dtlib.new_workspace(dtlib.dt_paged_attention_workspace_bytes(B, n, Hq, s["kc"].shape[1], d))
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


TOKEN = [
    ([1], 1, 1, 64, 8),                                   # one key
    ([1, 2, 63, 64, 65, 127, 128, 129], 8, 2, 128, 16),   # around the blocks' borders
    ([200, 0, 7, -3, 1, 0], 8, 2, 64, 32),                # unused rows of the batch
    ([0, 0, 0], 4, 4, 128, 16),                           # nothing but unused rows
    ([2049], 32, 8, 128, 64),
    ([30000], 8, 1, 128, 64),                             # one head over every CTA
    ([20011, 3, 700], 16, 16, 64, 128),
    ([777, 1500, 12], 40, 8, 128, 256),
    ([513] * 3, 64, 1, 128, 8),                           # 64 heads on one, the smallest pages
    ([300, 41], 128, 1, 64, 16),                          # every query row
    ([500, 90], 12, 2, 64, 16),
    ([1000, 64], 17, 17, 128, 32),
]


@pytest.mark.parametrize("lens,Hq,Hkv,d,page", TOKEN)
def test_one_new_token(dtlib, lens, Hq, Hkv, d, page):
    parity(dtlib, make(lens, 1, Hq, Hkv, d, page, mask=None))


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
def test_tree_nodes(dtlib, lens, n, Hq, Hkv, d, page, mask):
    parity(dtlib, make(lens, n, Hq, Hkv, d, page, mask=mask))


def test_a_node_without_visible_keys_is_zero(dtlib):
    s = make([4, 4], 4, 8, 2, 128, 16, mask="tree")
    s["mask"][1, 2] = 0
    out = parity(dtlib, s)
    assert (out[1, 2] == 0).all() and (out[1, 1] != 0).any()


def test_many_requests(dtlib):
    """More (request, head) pairs than CTAs, all lengths different, unused rows in between; sampled requests."""
    lens = [(37 * i) % 900 if i % 11 else 0 for i in range(500)]
    parity(dtlib, make(lens, 1, 8, 2, 128, 16, mask=None), requests=[0, 1, 2, 11, 100, 257, 498, 499])


@pytest.mark.parametrize("n", [1, 6])
def test_long_contexts(dtlib, n):
    parity(dtlib, make([100003, 40, 65536], n, 16, 2, 128, 64, mask="tree"), heads=[0, 7, 8, 15])


def test_shared_pages(dtlib):
    """Two requests with the same first pages."""
    s = make([200, 150], 1, 8, 2, 128, 32, mask=None)
    s["table"][1, :3] = s["table"][0, :3]
    parity(dtlib, s)


def test_scores_far_apart(dtlib):
    """Scores that grow by hundreds along the cache: the running maximum is raised again and again."""
    s = make([1500, 300], 2, 8, 2, 128, 16, mask="tree", spread=20.0)
    for b in range(2):
        for i in range(int(s["lens"][b]) // 16):
            s["kc"][s["table"][b, i].long()] *= (i + 1) / 16
    parity(dtlib, s)


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("Hq", [2, 32])
def test_what_is_not_finite_stays_with_the_nodes_that_see_it(dtlib, bad, Hq):
    """A node's value or key that is not finite reaches the nodes that see it, and no other."""
    n = 8 if Hq == 2 else 4
    s = make([130, 64, n], n, Hq, 2, 128, 16, mask="tree")
    s["mask"][:] = torch.eye(n, dtype=torch.uint8, device="cuda")
    s["mask"][:, 3, 1] = 1
    clean = run(dtlib, s).clone()
    for b in range(3):
        key = int(s["lens"][b]) - n + 1  # node 1's: seen by nodes 1 and 3
        s["vc"][s["table"][b, key // 16].long(), 1, key % 16, 77] = bad
    out = run(dtlib, s)
    hit = torch.zeros_like(out, dtype=torch.bool)
    hit[:, [1, 3], Hq // 2:, 77] = True
    assert torch.equal(out[~hit], clean[~hit])
    assert out[hit].isnan().all() if math.isnan(bad) else (out[hit] == bad).all()
    for b in range(3):
        key = int(s["lens"][b]) - n + 1
        s["vc"][s["table"][b, key // 16].long(), 1, key % 16, 77] = 1.0
        s["kc"][s["table"][b, key // 16].long(), 1, key % 16, 5] = float("nan")
    out = run(dtlib, s)
    hit[:, [1, 3], Hq // 2:] = True
    assert torch.equal(out[~hit], clean[~hit]) and out[hit].isnan().all()


def test_what_is_not_finite_in_one_request_stays_there(dtlib):
    s = make([70, 70, 70], 1, 8, 2, 64, 16, mask=None)
    clean = run(dtlib, s).clone()
    s["vc"][s["table"][1, 0].long()] = float("nan")
    out = run(dtlib, s)
    assert torch.equal(out[[0, 2]], clean[[0, 2]]) and out[1].isnan().all()
    s["q"][2] = float("nan")
    out = run(dtlib, s)
    assert torch.equal(out[0], clean[0]) and out[2].isnan().all()


def test_far_into_a_large_pool(dtlib):
    """Pages whose elements lie past 2^31 of the pool."""
    page, Hkv, d = 256, 8, 128
    pages = 2 ** 31 // (page * Hkv * d) + 3
    s = make([700, 90], 1, 16, Hkv, d, page, mask=None, pages=pages)
    assert int(s["table"].max()) * page * Hkv * d >= 2 ** 31
    parity(dtlib, s, heads=[0, 5, 15])


def test_bad_lengths_and_pages_are_reported(dtlib):
    s = make([40, 50, 60], 4, 8, 2, 64, 16, mask="tree")
    clean = run(dtlib, s).clone()
    ws = dtlib.new_workspace(dtlib.dt_paged_attention_workspace_bytes(3, 4, 8, 2, 64))
    good = s["lens"].clone()
    for wrong in (3, s["table"].shape[1] * 16 + 1, 2 ** 31 - 1):
        s["lens"][1] = wrong
        out = run(dtlib, s, workspace=ws)
        assert dtlib.dt_get_error(ws) == dtlib.Status.INVALID_ARG
        assert (out[1] == 0).all() and torch.equal(out[[0, 2]], clean[[0, 2]])
    s["lens"] = good
    for wrong in (-1, s["kc"].shape[0], 2 ** 31 - 1, -2 ** 31):
        was = int(s["table"][1, 1])
        s["table"][1, 1] = wrong
        out = run(dtlib, s, workspace=ws)
        assert dtlib.dt_get_error(ws) == dtlib.Status.INVALID_ARG
        assert torch.equal(out[[0, 2]], clean[[0, 2]])
        s["table"][1, 1] = was
    assert torch.equal(run(dtlib, s, workspace=ws), clean)
    assert dtlib.dt_get_error(ws) == dtlib.Status.OK


def test_a_captured_call_follows_the_lengths(dtlib):
    """Replayed after the lengths, the table and the pools changed in place, on a stream of its own."""
    s, other = make([300, 1, 90], 1, 8, 2, 128, 16, mask=None), make([7, 310, 0], 1, 8, 2, 128, 16, mask=None, seed=9)
    width, pages = (max(x[key].shape[dim] for x in (s, other)) for key, dim in (("table", 1), ("kc", 0)))

    def grown(t, rows, dim):
        pad = torch.full_like(t, -1).narrow(dim, 0, 1).repeat_interleave(rows - t.shape[dim], dim)
        return torch.cat([t, pad], dim).contiguous()
    for x in (s, other):
        x["table"] = grown(x["table"], width, 1)
        x["kc"], x["vc"] = grown(x["kc"], pages, 0), grown(x["vc"], pages, 0)
    ws = dtlib.new_workspace(dtlib.dt_paged_attention_workspace_bytes(3, 1, 8, 2, 128))
    out = torch.empty(3, 1, 8, 128, dtype=BF, device="cuda")
    want = [run(dtlib, x).clone() for x in (s, other)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(dtlib, s, out=out, workspace=ws)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        run(dtlib, s, out=out, workspace=ws)
    for x, w in ((s, want[0]), (other, want[1])):
        for key in ("q", "kc", "vc", "table", "lens"):
            s[key].copy_(x[key])
        out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, w)


def test_on_another_stream(dtlib):
    s = make([300, 20], 1, 8, 2, 128, 16, mask=None)
    want = run(dtlib, s)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        out = run(dtlib, s, stream=stream)  # its output and workspace are the stream's own
        side.synchronize()
        assert torch.equal(out, want)


def test_paged_attention_refuses(dtlib):
    s = make([30, 20], 2, 8, 2, 64, 16, mask="tree")
    for key, wrong, error in [("q", s["q"].float(), TypeError), ("q", s["q"][:, :, ::2], ValueError),
                              ("kc", s["kc"].float(), TypeError), ("vc", s["vc"][1:], ValueError),
                              ("table", s["table"].long(), TypeError), ("table", s["table"][:1], ValueError),
                              ("lens", s["lens"].cpu(), TypeError), ("mask", s["mask"].bool(), TypeError),
                              ("mask", s["mask"][:, :1], ValueError)]:
        with pytest.raises(error):
            run(dtlib, {**s, key: wrong})
    with pytest.raises(dtlib.DTError):
        run(dtlib, s, workspace=dtlib.new_workspace(256))                    # too small
    with pytest.raises(dtlib.DTError):
        run(dtlib, {**s, "scale": -1.0})
