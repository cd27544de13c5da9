"""The paged cache's operators together, as a serving program runs them around the drafting round: prompts, single
tokens, a draft tree's verify pass, its accepted path kept, and the next token, each against attention in 64 bits over
the sequence that the step stands for."""
import math

import torch
import pytest

from attention_ref import attend, check

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def test_prompt_tokens_tree_and_accepted_path(dtlib):
    B, Hq, Hkv, d, page, n, width = 3, 8, 2, 128, 16, 12, 20
    lens, G, scale = [70, 1, 129], Hq // Hkv, 1 / math.sqrt(d)
    g = torch.Generator(device="cuda").manual_seed(4)
    table = torch.randperm(B * width, generator=g, device="cuda").to(torch.int32).view(B, width)
    kc, vc = dtlib.new_paged_cache(B * width, Hkv, page, d)
    kc.fill_(float("nan")), vc.fill_(float("nan"))
    rope = dtlib.rope_table(1000, d)
    ws = dtlib.new_workspace(dtlib.dt_paged_attention_workspace_bytes(B, n, Hq, Hkv, d))
    project = lambda N: (torch.randn(N, Hq + 2 * Hkv, d, generator=g, device="cuda") * 1.2).to(BF)
    split = lambda x: (x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:])
    slot = lambda b, i: table[b, i // page] * page + i % page
    history = [[] for _ in range(B)]  # each request's (rotated keys, values) [Hkv,d], in order

    def append(x, where, positions):
        slots = torch.stack([slot(b, i) if b >= 0 else torch.tensor(-1, dtype=torch.int32, device="cuda")
                             for b, i in where]).to(torch.int32)
        q, k, v = split(x)
        out_k = torch.zeros(len(where), Hkv, d, dtype=BF, device="cuda")
        q = dtlib.dt_kv_append(k, v, kc, vc, slots, positions=torch.tensor(positions, dtype=torch.int32, device="cuda"),
                               rope=rope, q=q, out_k=out_k, workspace=ws)
        return q, out_k, v

    def against(out, q, keys):
        """out, q [Hq,d] of one token that sees `keys`."""
        k, v = (torch.stack([x[i] for x in keys]) for i in (0, 1))
        for h in range(Hq):
            seen = torch.ones(1, len(keys), dtype=torch.bool, device="cuda")
            check(out[h][None], *attend(q[h][None], k[:, h // G], v[:, h // G], seen, scale))

    # the prompts: into the cache, and attention over their packed rows
    where = [(b, i) for b in range(B) for i in range(lens[b])]
    q, k, v = append(project(len(where)), where, [i for _, i in where])
    cu = torch.tensor([0, 70, 71, 200], dtype=torch.int32, device="cuda")
    out = dtlib.dt_prompt_attention(q, k, v, cu, scale, workspace=ws)
    for r, (b, i) in enumerate(where):
        history[b].append((k[r], v[r]))
        if i in (0, 1, 69, 128):
            against(out[r], q[r], history[b])
    # the last prompt token by the single-token call: the same attention, read from the pages
    last = torch.tensor([69, 70, 199], device="cuda")
    length = torch.tensor(lens, dtype=torch.int32, device="cuda")
    again = dtlib.dt_paged_attention(q[last][:, None].contiguous(), kc, vc, table, length, scale, workspace=ws)
    for b in range(B):
        against(again[b, 0], q[last[b]], history[b])

    for round_ in range(2):
        # a draft tree per request: the marginal builder's trees, their nodes' keys behind the prefix
        ids, vals = dtlib.dt_topm(torch.randn(B, 6, 500, generator=g, device="cuda"), 4)
        tree = dtlib.dt_build_trees_marginal(ids, vals, 500, n, 6, 1.0)
        start = [len(x) for x in history]
        depth = tree["depth"].tolist()
        x = project(B * n)
        q, k, v = append(x, [(b, start[b] + i) for b in range(B) for i in range(n)],
                         [start[b] + depth[b][i] - 1 for b in range(B) for i in range(n)])
        length = torch.tensor([s + n for s in start], dtype=torch.int32, device="cuda")
        out = dtlib.dt_paged_attention(q.view(B, n, Hq, d), kc, vc, table, length, scale, mask=tree["mask"],
                                       workspace=ws)
        mask = tree["mask"].tolist()
        for b in range(B):
            for i in range(n):
                path = [(k[b * n + j], v[b * n + j]) for j in range(n) if mask[b][i][j]]
                against(out[b, i], q[b * n + i], history[b] + path)
        # accept a path: the target wants, at every node, its first child's token
        tokens, parents = tree["tokens"].tolist(), tree["parents"].tolist()
        want = [[next((tokens[b][j] for j in range(n) if parents[b][j] == u), -5) for u in range(-1, n)]
                for b in range(B)]
        got = dtlib.dt_accept_paths(tree["tokens"], tree["parents"],
                                    torch.tensor(want, dtype=torch.int32, device="cuda"))
        path = got["path"].tolist()
        where, positions = [(-1, 0)] * (B * n), [0] * (B * n)
        for b in range(B):
            for j, u in enumerate(u for u in path[b] if u >= 0):
                where[b * n + u], positions[b * n + u] = (b, start[b] + j), start[b] + j
                assert depth[b][u] == j + 1
                history[b].append((k[b * n + u], v[b * n + u]))
        append(x, where, positions)  # the accepted nodes again, behind the prefix; the others are left out
        # the bonus token, one per request
        x = project(B)
        q, k, v = append(x, [(b, len(history[b])) for b in range(B)], [len(history[b]) for b in range(B)])
        for b in range(B):
            history[b].append((k[b], v[b]))
        length = torch.tensor([len(h) for h in history], dtype=torch.int32, device="cuda")
        out = dtlib.dt_paged_attention(q[:, None].contiguous(), kc, vc, table, length, scale, workspace=ws)
        for b in range(B):
            against(out[b, 0], q[b], history[b])
    assert dtlib.dt_get_error(ws) == dtlib.Status.OK
