"""The 8-bit cache's operators together, as a serving program runs them around the drafting round, with no length, page or
slot on the host: prompts admitted, single tokens, draft trees verified, their accepted paths kept, requests that end and
others in their place. Each attention is checked against one in 64 bits over the tokens that the step stands for, read
from the pages by the host's own account of them."""
import math

import pytest
import torch

from attention_ref import attend, check
from test_paged_attn8_gpu import attend8, values

pytestmark = pytest.mark.gpu
BF, F8 = torch.bfloat16, torch.float8_e4m3fn


@pytest.mark.parametrize("d,page,block", [(128, 16, 16), (64, 32, 8)])
def test_prompts_tokens_trees_and_accepted_paths(dtlib, d, page, block):
    B, Hq, Hkv, n, pages, width = 3, 8, 2, 12, 60, 20
    G, scale = Hq // Hkv, 1 / math.sqrt(d)
    g = torch.Generator(device="cuda").manual_seed(4)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    kc, vc, ks, vs = dtlib.new_paged_cache8(pages, Hkv, page, d, scale_block=block)
    kc.view(torch.uint8).fill_(0x7F), vc.view(torch.uint8).fill_(0x7F)
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    pool = dict(held=ints([0] * B), free_pages=torch.randperm(pages, generator=g, device="cuda").to(torch.int32),
                free_count=ints([pages]))
    rope = dtlib.rope_table(1000, d)
    ws = dtlib.new_workspace(max(dtlib.dt_paged_attention8_workspace_bytes(B, n, Hq, Hkv, d),
                                 dtlib.dt_kv_append8_workspace_bytes(300, pages, page),
                                 dtlib.dt_page_plan_workspace_bytes(B)))
    project = lambda N: (torch.randn(N, Hq + 2 * Hkv, d, generator=g, device="cuda") * 1.2).to(BF)
    split = lambda x: (x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:])
    plan = lambda lens, grow, **kw: dtlib.dt_page_plan(lens, grow, table, page, pages, workspace=ws, **pool, **kw)

    def append(x, step, **kw):
        q, k, v = split(x)
        return dtlib.dt_kv_append8(k, v, kc, vc, ks, vs, step["slots"], positions=step["positions"], rope=rope, q=q,
                                   workspace=ws, **kw)

    def attention(q, lens, **kw):
        return dtlib.dt_paged_attention8(q, kc, vc, ks, vs, table, lens, scale, workspace=ws, **kw)

    def against(out, q, b, length, seen=None):
        """out, q [Hq,d] of a token that sees the first `length` tokens of request b, or those of `seen`."""
        at = table[b, :-(-length // page)].long()
        for h in range(Hq):
            (k, _), (v, s) = (values(c, x, at, h // G) for c, x in ((kc, ks), (vc, vs)))
            sees = torch.ones(1, length, dtype=torch.bool, device="cuda") if seen is None else seen
            check(out[h][None], *attend8(q[h][None], k[:length], v[:length], s[:length], sees, scale))

    def stored(x, step, b, lens):
        """The tokens' values are in the cache, within their rounding."""
        for t in range(x.shape[0]):
            slot = int(step["slots"][t])
            if slot < 0 or t % 7:
                continue
            for h in range(Hkv):
                got, s = (f(vc, vs) for f in (lambda c, y: c.view(torch.uint8)[slot // page, h, slot % page].view(F8).double(),
                                              lambda c, y: y[slot // page, h, slot % page // block].double()))
                want = split(x)[2][t, h].double()
                off = (got * s - want).abs()
                # rounded once, and again by as much at most each time that the block's scale grew
                assert (off <= torch.maximum(2.0 ** -4 * want.abs(), 2.0 ** -9 * s)).all()

    prompts = [70, 1, 129]
    step = plan(ints([0] * B), ints(prompts), rows=sum(prompts))
    x = project(sum(prompts))
    out_k = torch.zeros(sum(prompts), Hkv, d, dtype=BF, device="cuda")
    q = append(x, step, out_k=out_k)
    stored(x, step, None, None)
    assert step["lens"].tolist() == prompts and step["cu_seqlens"].tolist() == [0, 70, 71, 200]
    out = dtlib.dt_prompt_attention(q, out_k, split(x)[2], step["cu_seqlens"], scale, workspace=ws)
    for row, (first, b) in ((69, (0, 0)), (70, (70, 1)), (199, (71, 2))):
        k, v = out_k[first:row + 1], split(x)[2][first:row + 1]
        for h in (0, 7):
            sees = torch.ones(1, row + 1 - first, dtype=torch.bool, device="cuda")
            check(out[row, h][None], *attend(q[row, h][None], k[:, h // G], v[:, h // G], sees, scale))
    last = (step["cu_seqlens"][1:] - 1).long()
    lens = step["lens"]
    again = attention(q[last][:, None].contiguous(), lens)
    host = list(prompts)
    for b in range(B):
        against(again[b, 0], q[last[b]], b, host[b])

    for round_ in range(3):
        # a draft tree per request: pages for every node, the nodes behind the prefix
        ids, vals = dtlib.dt_topm(torch.randn(B, 6, 500, generator=g, device="cuda"), 4)
        tree = dtlib.dt_build_trees_marginal(ids, vals, 500, n, 6, 1.0)
        before = plan(lens, ints([n] * B), n=n, depth=tree["depth"])
        x = project(B * n)
        q = append(x, before)
        stored(x, before, None, None)
        out = attention(q.view(B, n, Hq, d), before["lens"], mask=tree["mask"])
        for b in range(B):
            for i in (0, 1, n - 1):
                seen = torch.cat([torch.ones(host[b], dtype=torch.bool, device="cuda"), tree["mask"][b, i] != 0])[None]
                against(out[b, i], q[b * n + i], b, host[b] + n, seen)
        tokens, parents = tree["tokens"].tolist(), tree["parents"].tolist()
        want = [[next((tokens[b][j] for j in range(n) if parents[b][j] == u), -5) for u in range(-1, n)]
                for b in range(B)]
        got = dtlib.dt_accept_paths(tree["tokens"], tree["parents"], ints(want))
        after = plan(lens, got["accept_len"], n=n, path=got["path"])  # the rejected nodes' pages go back
        append(x, after)  # the accepted nodes again, behind the prefix
        stored(x, after, None, None)
        host = [a + c for a, c in zip(host, got["accept_len"].tolist())]
        assert after["lens"].tolist() == host
        assert pool["held"].tolist() == [-(-h // page) for h in host]
        # the bonus token, one per request
        step = plan(after["lens"], ints([1] * B), n=1)
        x = project(B)
        q = append(x, step)
        host, lens = [h + 1 for h in host], step["lens"]
        out = attention(q[:, None].contiguous(), lens)
        for b in range(B):
            against(out[b, 0], q[b], b, host[b])
        if round_ == 1:  # request 1 ends, another takes its place: its blocks start anew
            plan(torch.where(ints([0, 1, 0]) > 0, -1, lens).to(torch.int32), ints([0] * B))
            assert pool["held"].tolist()[1] == 0
            step = plan(torch.where(ints([0, 1, 0]) > 0, 0, lens).to(torch.int32), ints([0, 50, 0]), rows=50)
            x = project(50)
            q = append(x, step)
            stored(x, step, None, None)
            host[1], lens = 50, step["lens"]
            assert lens.tolist() == host
            out = attention(torch.stack([q[0], q[49], q[1]])[:, None].contiguous(), lens)
            against(out[1, 0], q[49], 1, 50)
    assert dtlib.dt_get_error(ws) == dtlib.Status.OK
    assert int(pool["free_count"]) + sum(pool["held"].tolist()) == pages
