"""The paged key/value cache and its attention: the cases they are timed at, their plain forms, and their exact values.

Three operators, as a serving program calls them around the drafting round:

- ``append``  keys and values of new tokens go into a paged cache, rotated by their positions; queries are rotated too
- ``paged``   attention of one new token, or of a draft tree's nodes, over each request's pages
- ``prompt``  causal attention over whole prompts, packed one after the other
"""
import math

import torch

own = False

# (query heads, key/value heads, head dimension)
LAYOUTS = [(32, 8, 128), (32, 8, 64), (16, 8, 128), (8, 1, 128), (16, 16, 64), (40, 8, 128), (12, 2, 64)]
PAGE_SIZES = [16, 32, 64, 128]


def listed():
    return [
        # one request's next token: the smallest call, all latency
        dict(name="append-token", op="append", tokens=1, Hq=32, Hkv=8, d=128, page=64, rot=128, interleaved=False,
             skipped=0.0, keep_k=False),
        # the nodes of 64 draft trees of 16, before the verify pass
        dict(name="append-trees", op="append", tokens=1024, Hq=32, Hkv=8, d=128, page=16, rot=128, interleaved=False,
             skipped=0.0, keep_k=False),
        # prompts whose rotated keys the prompt attention reads next
        dict(name="append-prompt", op="append", tokens=16384, Hq=32, Hkv=8, d=128, page=64, rot=128,
             interleaved=False, skipped=0.0, keep_k=True),
        # narrow heads, half of each rotated in neighbouring pairs, a padded batch with a fifth of its rows unused
        dict(name="append-padded-d64", op="append", tokens=5003, Hq=32, Hkv=8, d=64, page=32, rot=32,
             interleaved=True, skipped=0.2, keep_k=False),
        # one request's next token over a chat's length
        dict(name="token-b1", op="paged", B=1, n=1, Hq=32, Hkv=8, d=128, page=64, longest=2049, shortest=2049),
        # a serving batch's next tokens, every length its own
        dict(name="token-b64", op="paged", B=64, n=1, Hq=32, Hkv=8, d=128, page=16, longest=8191, shortest=1),
        # few requests with very long contexts
        dict(name="token-long", op="paged", B=3, n=1, Hq=32, Hkv=8, d=128, page=64, longest=131072, shortest=100001),
        # the verify pass: 64 draft trees of 16 nodes over their prefixes
        dict(name="tree-b64", op="paged", B=64, n=16, Hq=32, Hkv=8, d=128, page=64, longest=4099, shortest=130),
        # one short prompt: latency again
        dict(name="prompt-short", op="prompt", B=1, Hq=32, Hkv=8, d=128, longest=77, shortest=77),
        # a batch of prompts of mixed lengths
        dict(name="prompt-packed", op="prompt", B=12, Hq=32, Hkv=8, d=128, longest=2500, shortest=33),
        # one long document
        dict(name="prompt-long", op="prompt", B=1, Hq=32, Hkv=8, d=128, longest=16384, shortest=16384),
        # narrow heads
        dict(name="prompt-d64", op="prompt", B=5, Hq=32, Hkv=8, d=64, longest=4097, shortest=1000),
    ]


def _log_int(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    Hq, Hkv, d = rng.choice(LAYOUTS)
    op = rng.choice(["append", "paged", "prompt"])
    if op == "append":
        return dict(op=op, tokens=_log_int(rng, 1, 16384 * 32 // max(Hq, 32)), Hq=Hq, Hkv=Hkv, d=d,
                    page=rng.choice(PAGE_SIZES), rot=rng.choice([d, d, d // 2]), interleaved=rng.random() < 0.3,
                    skipped=rng.choice([0.0, 0.0, 0.1, 0.3]), keep_k=rng.random() < 0.3)
    if op == "paged":
        B = _log_int(rng, 1, 96)
        n = 1 if rng.random() < 0.6 else rng.randint(2, 16)
        longest = max(n, _log_int(rng, 1, min(131072, 400000 * 8 // (max(Hkv, 8) * B))))
        return dict(op=op, B=B, n=n, Hq=Hq, Hkv=Hkv, d=d, page=rng.choice(PAGE_SIZES), longest=longest,
                    shortest=max(n, int(longest * rng.random())))
    B = _log_int(rng, 1, 24)
    longest = _log_int(rng, 1, int(16384 * math.sqrt(32 / (max(Hq, 32) * B))))
    return dict(op=op, B=B, Hq=Hq, Hkv=Hkv, d=d, longest=longest, shortest=max(1, int(longest * rng.random())))


def _lengths(case):
    """The case's lengths: spread evenly from the shortest to the longest, in a fixed mixed order."""
    B, lo, hi = case["B"], case["shortest"], case["longest"]
    return [hi if B == 1 else lo + (hi - lo) * ((i * 101 + 7) % B) // (B - 1) for i in range(B)]


def _tree_mask(B, n, gen):
    """Ancestor masks of random trees: node i's parent is an earlier node or the root."""
    pick = torch.rand(B, n, generator=gen, device="cuda")
    parent = (pick * torch.arange(1, n + 1, device="cuda")).long() - 1  # -1 for the root, else below i
    mask = torch.eye(n, dtype=torch.uint8, device="cuda").repeat(B, 1, 1)
    rows = torch.arange(B, device="cuda")
    for i in range(n):
        has = (parent[:, i] >= 0).to(torch.uint8)[:, None]
        mask[:, i] |= mask[rows, parent[:, i].clamp(min=0)] * has
    return mask.contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]

    def normal(*shape, spread=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * spread).to(torch.bfloat16)

    s = dict(case=case)
    if case["op"] == "append":
        N, page, rot, max_pos = case["tokens"], case["page"], case["rot"], 32768
        pages = -(-N // page) * 5 // 4 + 2
        qkv = normal(N, Hq + 2 * Hkv, d)  # the fused projection's output, split by views
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        slots = torch.randperm(pages * page, generator=gen, device="cuda")[:N].to(torch.int32)
        skip = torch.rand(N, generator=gen, device="cuda") < case["skipped"]
        s["slots"] = torch.where(skip, -1, slots).to(torch.int32)
        s["positions"] = torch.randint(0, max_pos, (N,), generator=gen, device="cuda", dtype=torch.int32)
        angle = torch.arange(max_pos, device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (
            -torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
        s["rope"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        s["k_cache"], s["v_cache"] = normal(pages, Hkv, page, d), normal(pages, Hkv, page, d)
        s["out_q"] = torch.zeros(N, Hq, d, dtype=torch.bfloat16, device="cuda")
        s["out_k"] = torch.zeros(N, Hkv, d, dtype=torch.bfloat16, device="cuda") if case["keep_k"] else None
    elif case["op"] == "paged":
        B, n, page = case["B"], case["n"], case["page"]
        lens = _lengths(case)
        used = [-(-x // page) for x in lens]
        pages = sum(used) + 3
        order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
        width = torch.arange(max(used), device="cuda")
        first = torch.tensor([sum(used[:b]) for b in range(B)], device="cuda")
        count = torch.tensor(used, device="cuda")
        at = (first[:, None] + width).clamp(max=pages - 1)
        s["page_table"] = torch.where(width < count[:, None], order[at], -1).to(torch.int32).contiguous()
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["k_cache"], s["v_cache"] = normal(pages, Hkv, page, d), normal(pages, Hkv, page, d)
        s["q"] = normal(B, n, Hq, d, spread=1.5)  # some keys stand out, as they do in a trained model
        s["mask"] = _tree_mask(B, n, gen) if n > 1 else None
        s["out"] = torch.zeros(B, n, Hq, d, dtype=torch.bfloat16, device="cuda")
    else:
        lens = _lengths(case)
        ends = [sum(lens[:b]) for b in range(len(lens) + 1)]
        s["longest"] = case["longest"]  # a serving program knows its longest prompt
        s["cu_seqlens"] = torch.tensor(ends, dtype=torch.int32, device="cuda")
        s["q"], s["k"] = normal(ends[-1], Hq, d, spread=1.5), normal(ends[-1], Hkv, d)
        qkv = normal(ends[-1], Hq + 2 * Hkv, d)  # the values stay where the fused projection left them
        s["v"] = qkv[:, Hq + Hkv:]
        s["out"] = torch.zeros(ends[-1], Hq, d, dtype=torch.bfloat16, device="cuda")
    if own:  # the workspace that such a program keeps
        from speculative_decoding_tree_top_gb300 import dominotree as dt
        room = 256 if case["op"] == "append" else (
            dt.dt_paged_attention_workspace_bytes(case["B"], case["n"], Hq, Hkv, d) if case["op"] == "paged" else
            dt.dt_prompt_attention_workspace_bytes(s["q"].shape[0], case["B"], Hq, Hkv, d))
        s["dt"], s["ws"] = dt, dt.new_workspace(room)
    return s


# ---- the plain forms ------------------------------------------------------------------------------------------

def _rotated(x, cos, sin, rot, interleaved):
    x = x.float()
    part = x[..., :rot]
    a, b = (part[..., 0::2], part[..., 1::2]) if interleaved else (part[..., :rot // 2], part[..., rot // 2:])
    a, b = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([turned, x[..., rot:]], -1).to(torch.bfloat16)


def _plain_append(s):
    c = s["case"]
    rot, page = c["rot"], c["page"]
    kept = (s["slots"] >= 0).nonzero()[:, 0]
    turn = s["rope"][s["positions"].long()][:, None]
    cos, sin = turn[..., :rot // 2], turn[..., rot // 2:]
    k = _rotated(s["k"], cos, sin, rot, c["interleaved"])
    s["out_q"][kept] = _rotated(s["q"], cos, sin, rot, c["interleaved"])[kept]
    slots = s["slots"][kept].long()
    s["k_cache"][slots // page, :, slots % page] = k[kept]
    s["v_cache"][slots // page, :, slots % page] = s["v"][kept]
    if s["out_k"] is not None:
        s["out_k"][kept] = k[kept]


def _plain_paged(s):
    c = s["case"]
    B, n, Hq, Hkv, d = c["B"], c["n"], c["Hq"], c["Hkv"], c["d"]
    G, table = Hq // Hkv, s["page_table"].clamp(min=0).long()
    k = s["k_cache"][table].transpose(1, 2).reshape(B, Hkv, -1, d).float()
    v = s["v_cache"][table].transpose(1, 2).reshape(B, Hkv, -1, d).float()
    q = s["q"].float().view(B, n, Hkv, G, d).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * n, d)
    score = (q @ k.transpose(2, 3)).view(B, Hkv, G, n, -1) * (1 / math.sqrt(d))
    at = torch.arange(k.shape[2], device=k.device)
    node = at - (s["lens"][:, None] - n)  # [B, keys]: the key's node, below 0 in the prefix, n and more past the end
    seen = (node < 0)[:, None].expand(B, n, -1)
    if n > 1:
        tree = s["mask"].bool().gather(2, node.clamp(0, n - 1)[:, None].expand(B, n, -1))
        seen = seen | (tree & ((node >= 0) & (node < n))[:, None])
    else:
        seen = seen | (node == 0)[:, None]
    score.masked_fill_(~seen[:, None, None], -math.inf)
    p = (score - score.amax(-1, keepdim=True)).exp_()
    p = p / p.sum(-1, keepdim=True)
    out = p.view(B, Hkv, G * n, -1) @ v
    return out.view(B, Hkv, G, n, d).permute(0, 3, 1, 2, 4).reshape(B, n, Hq, d).to(torch.bfloat16)


def _plain_prompt(s):
    c = s["case"]
    B, Hq, Hkv, d, L = c["B"], c["Hq"], c["Hkv"], c["d"], s["longest"]
    G, cu, total = Hq // Hkv, s["cu_seqlens"].long(), s["q"].shape[0]
    at = torch.arange(L, device=cu.device)
    row = (cu[:-1, None] + at).clamp(max=total - 1)  # padded to the longest; what lies behind a prompt is masked
    q = s["q"][row].float().view(B, L, Hkv, G, d).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * L, d)
    k = s["k"][row].float().transpose(1, 2)
    v = s["v"][row].float().transpose(1, 2)
    score = (q @ k.transpose(2, 3)).mul_(1 / math.sqrt(d)).view(B, Hkv, G, L, L)
    score.masked_fill_(at > at[:, None], -math.inf)
    p = score.sub_(score.amax(-1, keepdim=True)).exp_()
    p = p.div_(p.sum(-1, keepdim=True)).view(B, Hkv, G * L, L)
    out = (p @ v).view(B, Hkv, G, L, d).permute(0, 3, 1, 2, 4).reshape(B, L, Hq, d).to(torch.bfloat16)
    token = torch.arange(total, device=cu.device)
    b = torch.searchsorted(cu[1:], token, right=True)
    return out[b, token - cu[b]]


# ---- one pass -------------------------------------------------------------------------------------------------

def run(s):
    c = s["case"]
    scale = 1 / math.sqrt(c["d"])
    if c["op"] == "append":
        if own:
            s["dt"].dt_kv_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["slots"], positions=s["positions"],
                                 rope=s["rope"], interleaved=c["interleaved"], q=s["q"], out_q=s["out_q"],
                                 out_k=s["out_k"], workspace=s["ws"])
        else:
            _plain_append(s)
        out = dict(q=s["out_q"], k_cache=s["k_cache"], v_cache=s["v_cache"])
        return dict(out, k=s["out_k"]) if c["keep_k"] else out
    if c["op"] == "paged":
        if own:
            return s["dt"].dt_paged_attention(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["lens"], scale,
                                              mask=s["mask"], out=s["out"], workspace=s["ws"])
        return _plain_paged(s)
    if own:
        return s["dt"].dt_prompt_attention(s["q"], s["k"], s["v"], s["cu_seqlens"], scale, out=s["out"],
                                           workspace=s["ws"])
    return _plain_prompt(s)


def work(case):
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    if case["op"] == "append":
        kept = case["tokens"] * (1 - case["skipped"])
        per_token = (2 * Hq + 4 * Hkv + (Hkv if case["keep_k"] else 0)) * d * 2 + case["rot"] * 4 + 4
        return dict(bytes=kept * per_token + case["tokens"] * 4, flops=kept * (Hq + Hkv) * case["rot"] * 3)
    lens = _lengths(case)
    if case["op"] == "paged":
        rows = case["B"] * case["n"]
        table = sum(-(-x // case["page"]) for x in lens) * 4
        return dict(bytes=sum(lens) * Hkv * d * 4 + rows * Hq * d * 4 + table + case["B"] * 4 +
                    (rows * case["n"] if case["n"] > 1 else 0), flops=4 * Hq * case["n"] * d * sum(lens))
    return dict(bytes=sum(lens) * (2 * Hq + 2 * Hkv) * d * 2 + 4 * len(lens),
                flops=4 * Hq * d * sum(x * (x + 1) // 2 for x in lens))


# ---- the exact values, from the definitions in 64 bits, one token or one head at a time ------------------------

def _exact_append(s):
    c = s["case"]
    rot, page, half = c["rot"], c["page"], c["rot"] // 2
    i = torch.arange(half, device="cuda")
    first, second = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + half)

    def turn(x, positions):  # complex numbers times e^(i angle)
        x = x.double()
        t = s["rope"].double()[positions.long()]
        z = torch.complex(x[..., first], x[..., second]) * torch.complex(t[:, :half], t[:, half:])[:, None]
        x = x.clone()
        x[..., first], x[..., second] = z.real, z.imag
        return x

    kept = [t for t, slot in enumerate(s["slots"].tolist()) if slot >= 0]
    kept = torch.tensor(kept, device="cuda", dtype=torch.long)
    position, slot = s["positions"][kept], s["slots"][kept].long()
    out = dict(q=s["out_q"].double(), k_cache=s["k_cache"].double(), v_cache=s["v_cache"].double())
    out["q"][kept] = turn(s["q"][kept], position)
    k = turn(s["k"][kept], position)
    pages = out["k_cache"].shape[0]
    line = torch.arange(pages * page, device="cuda").view(pages, page)
    where = torch.full((pages * page,), -1, device="cuda", dtype=torch.long)
    where[slot] = torch.arange(len(kept), device="cuda")
    source = where[line]  # [pages, page]: the kept token that goes there, or -1
    written = (source >= 0)[:, None, :, None]
    if len(kept):
        out["k_cache"] = torch.where(written, k[source.clamp(min=0)].transpose(1, 2), out["k_cache"])
        out["v_cache"] = torch.where(written, s["v"][kept].double()[source.clamp(min=0)].transpose(1, 2),
                                     out["v_cache"])
    if c["keep_k"]:
        out["k"] = s["out_k"].double()
        out["k"][kept] = k
    return out


def _exact_rows(q, k, v, seen):
    """softmax(q k^T / sqrt(d)) v of some rows [rows, d] against [keys, d], in 64 bits."""
    z = (q.double() @ k.double().t() / math.sqrt(q.shape[-1])).masked_fill(~seen, -math.inf)
    return torch.softmax(z, -1) @ v.double()


def _exact_paged(s):
    c = s["case"]
    n, G, page = c["n"], c["Hq"] // c["Hkv"], c["page"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for b, length in enumerate(s["lens"].tolist()):
        pages = s["page_table"][b, :-(-length // page)].long()
        tree = s["mask"][b].bool() if n > 1 else torch.ones(1, 1, dtype=torch.bool, device="cuda")
        seen = torch.cat([torch.ones(n, length - n, dtype=torch.bool, device="cuda"), tree], 1).repeat(G, 1)
        for g in range(c["Hkv"]):
            k, v = (x[pages, g].reshape(-1, c["d"])[:length] for x in (s["k_cache"], s["v_cache"]))
            q = s["q"][b, :, g * G:(g + 1) * G].transpose(0, 1).reshape(G * n, c["d"])
            out[b, :, g * G:(g + 1) * G] = _exact_rows(q, k, v, seen).view(G, n, c["d"]).transpose(0, 1)
    return out


def _exact_prompt(s):
    G = s["case"]["Hq"] // s["case"]["Hkv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    ends = s["cu_seqlens"].tolist()
    for lo, hi in zip(ends, ends[1:]):
        for a in range(lo, hi, 2048):  # rows a to z see the keys up to their own
            z = min(hi, a + 2048)
            seen = torch.ones(z - a, z - lo, dtype=torch.bool, device="cuda").tril(a - lo)
            for h in range(s["q"].shape[1]):
                out[a:z, h] = _exact_rows(s["q"][a:z, h], s["k"][lo:z, h // G], s["v"][lo:z, h // G], seen)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return dict(append=_exact_append, paged=_exact_paged, prompt=_exact_prompt)[case["op"]](s)
