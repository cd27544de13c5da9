"""The paged cache in 8 bits, and its pages: the cases they are timed at, their plain forms, and their exact values.

Three operators, as a serving program calls them around the drafting round:

- ``plan``    request lengths become pages taken from and given back to a pool, slots and positions of the new tokens
- ``append8`` keys and values of new tokens go into a paged cache in e4m3, one scale for each block of tokens and head
- ``paged8``  attention of one new token, or of a draft tree's nodes, over each request's pages of that cache
"""
import math

import torch

own = False

# (query heads, key/value heads, head dimension)
LAYOUTS = [(32, 8, 128), (32, 8, 64), (16, 8, 128), (8, 1, 128), (16, 16, 64), (40, 8, 128), (12, 2, 64)]
PAGE_SIZES = [16, 32, 64, 128]
LOWEST, HIGHEST = -48, 48  # the exponents that a scale may have


def listed():
    return [
        # one request's draft tree: its pages and slots before the verify pass and after it, all latency
        dict(name="plan-tree-b1", op="plan", B=1, n=8, page=64, longest=2049, shortest=2049),
        # 64 draft trees of 16 nodes, the pages that their rejected nodes held given back
        dict(name="plan-tree-b64", op="plan", B=64, n=16, page=16, longest=8191, shortest=1),
        # packed prompts admitted, and their requests ended
        dict(name="plan-prompts", op="plan", B=256, n=0, page=16, longest=2500, shortest=33),
        # one request's next token: the smallest append
        dict(name="append8-token", op="append8", requests=1, per=1, Hq=32, Hkv=8, d=128, page=64, block=16, rot=128,
             interleaved=False, skipped=0.0, keep_k=False),
        # the nodes of 64 draft trees of 16, before the verify pass: most meet a block that holds rows already
        dict(name="append8-trees", op="append8", requests=64, per=16, Hq=32, Hkv=8, d=128, page=16, block=16, rot=128,
             interleaved=False, skipped=0.0, keep_k=False),
        # prompts whose rotated keys the prompt attention reads next
        dict(name="append8-prompt", op="append8", requests=8, per=2048, Hq=32, Hkv=8, d=128, page=64, block=16,
             rot=128, interleaved=False, skipped=0.0, keep_k=True),
        # narrow heads, half of each rotated in neighbouring pairs, a padded batch with a fifth of its rows unused
        dict(name="append8-padded-d64", op="append8", requests=17, per=295, Hq=32, Hkv=8, d=64, page=32, block=32,
             rot=32, interleaved=True, skipped=0.2, keep_k=False),
        # one request's next token over a chat's length
        dict(name="token8-b1", op="paged8", B=1, n=1, Hq=32, Hkv=8, d=128, page=64, block=16, longest=2049,
             shortest=2049),
        # a serving batch's next tokens, every length its own
        dict(name="token8-b64", op="paged8", B=64, n=1, Hq=32, Hkv=8, d=128, page=16, block=16, longest=8191,
             shortest=1),
        # few requests with very long contexts
        dict(name="token8-long", op="paged8", B=3, n=1, Hq=32, Hkv=8, d=128, page=64, block=64, longest=131072,
             shortest=100001),
        # the verify pass: 64 draft trees of 16 nodes over their prefixes
        dict(name="tree8-b64", op="paged8", B=64, n=16, Hq=32, Hkv=8, d=128, page=64, block=16, longest=4099,
             shortest=130),
        # narrow heads
        dict(name="token8-d64", op="paged8", B=64, n=1, Hq=32, Hkv=8, d=64, page=64, block=32, longest=8191,
             shortest=1),
    ]


def _log_int(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    Hq, Hkv, d = rng.choice(LAYOUTS)
    page = rng.choice(PAGE_SIZES)
    block = rng.choice([x for x in (8, 16, 32, 64) if x <= page])
    op = rng.choice(["plan", "append8", "append8", "paged8", "paged8"])
    if op == "plan":
        B = _log_int(rng, 1, 256)
        n = 0 if rng.random() < 0.4 else rng.randint(2, 32)
        longest = max(n, _log_int(rng, 1, 300000 // B if n == 0 else 8191))
        return dict(op=op, B=B, n=n, page=page, longest=longest, shortest=max(1, int(longest * rng.random())))
    if op == "append8":
        tokens = _log_int(rng, 1, 16384 * 32 // max(Hq, 32))
        requests = _log_int(rng, 1, min(256, tokens))
        return dict(op=op, requests=requests, per=max(1, tokens // requests), Hq=Hq, Hkv=Hkv, d=d, page=page,
                    block=block, rot=rng.choice([d, d, d // 2]), interleaved=rng.random() < 0.3,
                    skipped=rng.choice([0.0, 0.0, 0.1, 0.3]), keep_k=rng.random() < 0.3)
    B = _log_int(rng, 1, 96)
    n = 1 if rng.random() < 0.6 else rng.randint(2, 16)
    longest = max(n, _log_int(rng, 1, min(131072, 400000 * 8 // (max(Hkv, 8) * B))))
    return dict(op=op, B=B, n=n, Hq=Hq, Hkv=Hkv, d=d, page=page, block=block, longest=longest,
                shortest=max(n, int(longest * rng.random())))


def _lengths(case):
    """The case's lengths: spread evenly from the shortest to the longest, in a fixed mixed order."""
    B, lo, hi = case["B"], case["shortest"], case["longest"]
    return [hi if B == 1 else lo + (hi - lo) * ((i * 101 + 7) % B) // (B - 1) for i in range(B)]


def _tree_mask(B, n, gen):
    """Ancestor masks and depths (from 1) of random trees: node i's parent is an earlier node or the root."""
    pick = torch.rand(B, n, generator=gen, device="cuda")
    parent = (pick * torch.arange(1, n + 1, device="cuda")).long() - 1  # -1 for the root, else below i
    mask = torch.eye(n, dtype=torch.uint8, device="cuda").repeat(B, 1, 1)
    rows = torch.arange(B, device="cuda")
    for i in range(n):
        has = (parent[:, i] >= 0).to(torch.uint8)[:, None]
        mask[:, i] |= mask[rows, parent[:, i].clamp(min=0)] * has
    return mask.contiguous(), mask.sum(2).to(torch.int32)


def _tables(used, pages, gen):
    """Page tables of requests that hold `used` pages each, in random order; behind them no page."""
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    count = torch.tensor(used, device="cuda")
    first = count.cumsum(0) - count
    at = torch.arange(max(max(used), 1), device="cuda")
    table = torch.where(at < count[:, None], order[(first[:, None] + at).clamp(max=pages - 1)], -1)
    return table.to(torch.int32).contiguous(), order[sum(used):]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case=case)

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    def normal(*shape, spread=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * spread).to(torch.bfloat16)

    if case["op"] == "plan":
        B, n, page, lens = case["B"], case["n"], case["page"], _lengths(case)
        most = [-(-(x + n) // page) for x in lens]
        pages = sum(most) + 5
        if n:
            kept = (torch.rand(B, generator=gen, device="cuda") * min(n, 7)).to(torch.int32)  # accepted nodes
            keep = kept.tolist()
            used = [-(-(x + a) // page) for x, a in zip(lens, keep)]
            nodes = torch.rand(B, n, generator=gen, device="cuda").argsort(1)
            there = torch.arange(n, device="cuda") < kept[:, None]
            nodes = torch.where(there, nodes, n).sort(1).values
            s["path"] = torch.where(there, nodes, -1).to(torch.int32).contiguous()
            s["depth"] = _tree_mask(B, n, gen)[1].contiguous()
            s["lens"], s["grow"], s["kept"] = ints(lens), ints([n] * B), kept
        else:
            used = [0] * B
            s["lens"], s["grow"], s["gone"] = ints([0] * B), ints(lens), ints([-1] * B)
        table, left = _tables(used, pages, gen)
        s["table"] = torch.full((B, max(most) + 1), -1, dtype=torch.int32, device="cuda")
        s["table"][:, :table.shape[1]] = table
        s["held"], s["count"] = ints(used), ints([left.numel()])
        s["free"] = torch.full((pages,), -1, dtype=torch.int32, device="cuda")
        s["free"][:left.numel()] = left
        rows = B * n if n else sum(lens)
        s["pages"], s["rows"] = pages, rows
        for i in (1, 2):
            s["out%d" % i] = dict(lens=ints([0] * B), cu_seqlens=ints([0] * (B + 1)))
            if n or i == 1:
                s["out%d" % i].update(slots=ints([0] * rows), positions=ints([0] * rows))
    elif case["op"] == "append8":
        R, per, page, block = case["requests"], case["per"], case["page"], case["block"]
        Hq, Hkv, d, rot, max_pos, N = case["Hq"], case["Hkv"], case["d"], case["rot"], 32768, R * per
        start = torch.randint(0, 2 * page, (R,), generator=gen, device="cuda")  # rows that are there already
        used = [-(-(2 * page - 1 + per) // page)] * R
        pages = sum(used) + 2
        table, _ = _tables(used, pages, gen)
        at = start[:, None] + torch.arange(per, device="cuda")
        slots = (table.gather(1, at // page).long() * page + at % page).flatten()
        skip = torch.rand(N, generator=gen, device="cuda") < case["skipped"]
        s["slots"] = torch.where(skip, -1, slots).to(torch.int32)
        s["positions"] = torch.randint(0, max_pos, (N,), generator=gen, device="cuda", dtype=torch.int32)
        loud = 1 + 3 * (torch.rand(N, 1, 1, generator=gen, device="cuda") < 0.02)  # tokens that stand out
        qkv = (torch.randn(N, Hq + 2 * Hkv, d, generator=gen, device="cuda") * loud).to(torch.bfloat16)
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        angle = torch.arange(max_pos, device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (
            -torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
        s["rope"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        for kv in "kv":
            s[kv + "_cache"], s[kv + "_scale"] = _coded(normal(pages, Hkv, page, d).float(), block)
        s["out_q"] = torch.zeros(N, Hq, d, dtype=torch.bfloat16, device="cuda")
        s["out_k"] = torch.zeros(N, Hkv, d, dtype=torch.bfloat16, device="cuda") if case["keep_k"] else None
    else:
        B, n, page, block, lens = case["B"], case["n"], case["page"], case["block"], _lengths(case)
        Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
        used = [-(-x // page) for x in lens]
        pages = sum(used) + 3
        s["page_table"], _ = _tables(used, pages, gen)
        s["lens"] = ints(lens)
        for kv in "kv":
            # blocks of different sizes of value, so that their scales differ
            spread = 2 ** torch.randn(pages, Hkv, page // block, 1, 1, generator=gen, device="cuda").clamp(-3, 3)
            x = torch.randn(pages, Hkv, page // block, block, d, generator=gen, device="cuda") * spread
            s[kv + "_cache"], s[kv + "_scale"] = _coded(x.view(pages, Hkv, page, d), block)
            del x
        s["q"] = normal(B, n, Hq, d)
        s["mask"] = _tree_mask(B, n, gen)[0] if n > 1 else None
        s["out"] = torch.zeros(B, n, Hq, d, dtype=torch.bfloat16, device="cuda")
    if own:  # the workspace that such a program keeps
        from speculative_decoding_tree_top_gb300 import dominotree as dt
        room = {"plan": lambda: dt.dt_page_plan_workspace_bytes(case["B"]),
                "append8": lambda: dt.dt_kv_append8_workspace_bytes(N, pages, page),
                "paged8": lambda: dt.dt_paged_attention8_workspace_bytes(B, n, Hq, Hkv, d)}[case["op"]]()
        s["dt"], s["ws"] = dt, dt.new_workspace(room)
    return s


# ---- the plain forms ------------------------------------------------------------------------------------------

def _scale_of(amax):
    """The smallest power of two, within its limits, that brings values of up to `amax` into e4m3's 448."""
    m, e = torch.frexp(amax)  # amax = m 2^e, m in [1/2, 1): 448 = 0.875 2^9
    e = torch.where(amax > 0, e - 9 + (m > 0.875).int(), LOWEST).clamp(LOWEST, HIGHEST)
    return ((e.int() + 127) << 23).view(torch.float32)


def _coded(x, block):
    """x [pages,Hkv,page,d] fp32 in e4m3 with a scale for each block of a page's rows and head."""
    pages, Hkv, page, d = x.shape
    scale = _scale_of(x.view(pages, Hkv, page // block, block * d).abs().amax(-1))
    return (x / scale.repeat_interleave(block, 2)[..., None]).to(torch.float8_e4m3fn), scale


def _rotated(x, cos, sin, rot, interleaved):
    x = x.float()
    part = x[..., :rot]
    a, b = (part[..., 0::2], part[..., 1::2]) if interleaved else (part[..., :rot // 2], part[..., rot // 2:])
    a, b = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _plain_store(x, slots, cache, scale, block):
    """x [T,Hkv,d] fp32 into the cache's rows `slots`. Of each block that they reach, the rows below the lowest of them
    are kept: coded again where the scale grows."""
    pages, Hkv, page, d = cache.shape
    per = page // block
    line, row = slots // block, slots % block
    reached = torch.zeros(pages * per, dtype=torch.bool, device=x.device)
    reached[line] = True
    ids = reached.nonzero()[:, 0]
    at = (reached.cumsum(0) - 1)[line]
    low = torch.full((ids.numel(),), block, device=x.device).scatter_reduce(0, at, row, "amin")
    amax = torch.zeros(ids.numel(), Hkv, device=x.device).scatter_reduce(
        0, at[:, None].expand(-1, Hkv), x.abs().amax(-1), "amax")
    codes = cache.view(torch.uint8).view(pages, Hkv, per, block, d)
    was = codes[ids // per, :, ids % per]
    old = scale[ids // per, :, ids % per]
    kept = (low > 0)[:, None] & (old > 0)
    new = torch.where(kept, torch.maximum(_scale_of(amax), old), _scale_of(amax))
    again = (was.view(torch.float8_e4m3fn).float() * (old / new)[..., None, None]).to(torch.float8_e4m3fn)
    below = (torch.arange(block, device=x.device) < low[:, None])[:, None] & kept[..., None]
    now = torch.where(below[..., None], again.view(torch.uint8), was)
    now[at, :, row] = (x / new[at][..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
    codes[ids // per, :, ids % per] = now
    scale[ids // per, :, ids % per] = new


def _plain_append(s):
    c = s["case"]
    rot, kept = c["rot"], (s["slots"] >= 0).nonzero()[:, 0]
    turn = s["rope"][s["positions"][kept].long()][:, None]
    cos, sin = turn[..., :rot // 2], turn[..., rot // 2:]
    s["out_q"][kept] = _rotated(s["q"][kept], cos, sin, rot, c["interleaved"]).to(torch.bfloat16)
    k, slots = _rotated(s["k"][kept], cos, sin, rot, c["interleaved"]), s["slots"][kept].long()
    if s["out_k"] is not None:
        s["out_k"][kept] = k.to(torch.bfloat16)
    _plain_store(k, slots, s["k_cache"], s["k_scale"], c["block"])
    _plain_store(s["v"][kept].float(), slots, s["v_cache"], s["v_scale"], c["block"])


def _plain_paged(s):
    c = s["case"]
    B, n, Hq, Hkv, d, block = c["B"], c["n"], c["Hq"], c["Hkv"], c["d"], c["block"]
    G, table = Hq // Hkv, s["page_table"].clamp(min=0).long()

    def rows(cache, scale):  # the requests' rows, in order
        x = cache.view(torch.uint8)[table].view(torch.float8_e4m3fn).float()  # [B, width, Hkv, page, d]
        x = x.view(*x.shape[:3], -1, block, d) * scale[table][..., None, None]
        return x.flatten(3, 4).transpose(1, 2).reshape(B, Hkv, -1, d)

    k, v = rows(s["k_cache"], s["k_scale"]), rows(s["v_cache"], s["v_scale"])
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


def _plain_plan(s, lens, grow, out, depth=None, path=None):
    """Pages taken from the top of the stack in the requests' order and given back in the opposite one."""
    n, page, table, held, free, count = s["case"]["n"], s["case"]["page"], s["table"], s["held"], s["free"], s["count"]
    there, lens = lens >= 0, lens.clamp(min=0).long()
    grow = grow.long() * there
    want = (lens + grow + page - 1) // page
    take, give = (want - held).clamp(min=0), (held - want).clamp(min=0)
    i = torch.arange(table.shape[1], device=lens.device)
    taken, given = (i >= held[:, None]) & (i < want[:, None]), (i >= want[:, None]) & (i < held[:, None])
    gives, end = give.sum(), free.numel()
    rank = give.cumsum(0)[:, None] - give[:, None] + i - want[:, None]
    stack = torch.cat([free, free[:1]])  # its last place takes what is not given
    stack.scatter_(0, torch.where(given, count + gives - 1 - rank, end).flatten(), table.flatten())
    rank = take.cumsum(0)[:, None] - take[:, None] + i - held[:, None]
    got = stack[torch.where(taken, count + gives - 1 - rank, end)]
    table.copy_(torch.where(taken, got, table))
    left = count + gives - take.sum()
    free.copy_(torch.where(torch.arange(end, device=lens.device) < left, stack[:-1], free))
    held.copy_(want)
    count.copy_(left)
    out["lens"].copy_(lens + grow)
    cu = torch.cat([grow.new_zeros(1), (grow if n == 0 else torch.full_like(grow, n)).cumsum(0)])
    out["cu_seqlens"].copy_(cu)
    if "slots" not in out:
        return
    row = torch.arange(out["slots"].numel(), device=lens.device)
    b = torch.searchsorted(cu[1:].contiguous(), row, right=True)
    token = row - cu[b]
    if path is not None:
        hit = path.long()[b] == token[:, None]
        live = hit.any(1)
        token = hit.int().argmax(1)
        live = live & (token < grow[b])
    else:
        live = token < grow[b]
    at = lens[b] + token
    slot = table[b, (at // page).clamp(max=table.shape[1] - 1)] * page + at % page
    position = lens[b] + depth.flatten().long() - 1 if depth is not None else at
    out["slots"].copy_(torch.where(live, slot, -1))
    out["positions"].copy_(torch.where(live, position, 0))


# ---- one pass -------------------------------------------------------------------------------------------------

def run(s):
    c = s["case"]
    if c["op"] == "plan":
        first, second = dict(n=c["n"], depth=s.get("depth")), dict(n=c["n"], path=s.get("path"))
        then = (s["lens"], s["kept"]) if c["n"] else (s["gone"], s["grow"])
        if own:
            pool = dict(held=s["held"], free_pages=s["free"], free_count=s["count"], workspace=s["ws"])
            args = s["table"], c["page"], s["pages"]
            s["dt"].dt_page_plan(s["lens"], s["grow"], *args, out=s["out1"], **pool, **first)
            s["dt"].dt_page_plan(*then, *args, out=s["out2"], **pool, **second)
        else:
            _plain_plan(s, s["lens"], s["grow"], s["out1"], depth=s.get("depth"))
            _plain_plan(s, *then, s["out2"], path=s.get("path"))
        return dict(before=s["out1"], after=s["out2"], table=s["table"], held=s["held"], free=s["free"],
                    count=s["count"])
    if c["op"] == "append8":
        if own:
            s["dt"].dt_kv_append8(s["k"], s["v"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["slots"],
                                  positions=s["positions"], rope=s["rope"], interleaved=c["interleaved"], q=s["q"],
                                  out_q=s["out_q"], out_k=s["out_k"], workspace=s["ws"])
        else:
            _plain_append(s)
        out = dict(q=s["out_q"], k_cache=s["k_cache"], v_cache=s["v_cache"], k_scale=s["k_scale"],
                   v_scale=s["v_scale"])
        return dict(out, k=s["out_k"]) if c["keep_k"] else out
    if own:
        return s["dt"].dt_paged_attention8(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"],
                                           s["page_table"], s["lens"], 1 / math.sqrt(c["d"]), mask=s["mask"],
                                           out=s["out"], workspace=s["ws"])
    return _plain_paged(s)


def work(case):
    if case["op"] == "plan":
        B, n, lens = case["B"], case["n"], _lengths(case)
        rows = B * n if n else sum(lens)
        moved = sum(-(-(x + n) // case["page"]) - (-(-x // case["page"]) if n else 0) for x in lens)
        # per call: lengths and growth read, lengths and starts written, the state read and written; slots and positions
        # of each row; each page that moves read and written twice
        return dict(bytes=2 * 24 * B + (2 * 12 * rows if n else 8 * rows) + 2 * 8 * moved, flops=4 * rows + 20 * B)
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    if case["op"] == "append8":
        tokens = case["requests"] * case["per"]
        kept = tokens * (1 - case["skipped"])
        # queries in and out, keys and values in as bf16 and out in 8 bits, the rotation, slot and position
        per_token = (4 * Hq + 4 * Hkv + 2 * Hkv + (2 * Hkv if case["keep_k"] else 0)) * d + case["rot"] * 4 + 4
        scales = kept / case["block"] * Hkv * 2 * 4
        return dict(bytes=kept * per_token + tokens * 4 + scales,
                    flops=kept * ((Hq + Hkv) * case["rot"] * 3 + 2 * Hkv * d * 3))
    lens = _lengths(case)
    rows = case["B"] * case["n"]
    table = sum(-(-x // case["page"]) for x in lens) * 4
    scales = sum(-(-x // case["block"]) for x in lens) * Hkv * 2 * 4
    return dict(bytes=sum(lens) * Hkv * d * 2 + scales + rows * Hq * d * 4 + table + case["B"] * 4 +
                (rows * case["n"] if case["n"] > 1 else 0), flops=4 * Hq * case["n"] * d * sum(lens))


# ---- the exact values, from the definitions in 64 bits ---------------------------------------------------------

def _exact_append(s):
    c = s["case"]
    rot, page, block, half = c["rot"], c["page"], c["block"], c["rot"] // 2
    i = torch.arange(half, device="cuda")
    first, second = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + half)

    def turn(x, positions):  # complex numbers times e^(i angle)
        x = x.double()
        t = s["rope"].double()[positions.long()]
        z = torch.complex(x[..., first], x[..., second]) * torch.complex(t[:, :half], t[:, half:])[:, None]
        x = x.clone()
        x[..., first], x[..., second] = z.real, z.imag
        return x

    def power(e):
        return ((e + 1023) << 52).view(torch.float64)

    slots = s["slots"].tolist()
    kept = torch.tensor([t for t, slot in enumerate(slots) if slot >= 0], device="cuda", dtype=torch.long)
    out = dict(q=s["out_q"].double())
    out["q"][kept] = turn(s["q"][kept], s["positions"][kept])
    new = dict(k=turn(s["k"][kept], s["positions"][kept]), v=s["v"][kept].double())
    if c["keep_k"]:
        out["k"] = s["out_k"].double()
        out["k"][kept] = new["k"]
    pages, Hkv, _, d = s["k_cache"].shape
    blocks = pages * page // block
    # which token goes to which row of which block, -1 for none
    source = torch.full((pages * page,), -1, device="cuda", dtype=torch.long)
    source[s["slots"][kept].long()] = torch.arange(kept.numel(), device="cuda")
    source = source.view(blocks, block)
    written = source >= 0
    low = torch.where(written, torch.arange(block, device="cuda"), block).amin(1)
    for kv in "kv":
        def flat(x, *tail):  # [pages, Hkv, per, ...] -> [blocks, Hkv, ...]
            return x.view(pages, Hkv, page // block, *tail).transpose(1, 2).reshape(blocks, Hkv, *tail)

        def back(x, *tail):
            return x.view(pages, page // block, Hkv, *tail).transpose(1, 2)

        codes = flat(s[kv + "_cache"].double(), block, d)
        old = flat(s[kv + "_scale"]).double()
        rows = new[kv][source.clamp(min=0)].transpose(1, 2) if kept.numel() else torch.zeros_like(codes)
        rows = rows * written[:, None, :, None]
        # the exponent: the least whole e with amax <= 448 2^e (a power by its bits: `**` is off in its last place)
        amax = rows.abs().amax((2, 3))
        e = torch.ceil(torch.log2(amax / 448)).clamp(LOWEST - 1, HIGHEST)
        e = e.long() - (amax <= 448 * power(e.long() - 1)).long() + (amax > 448 * power(e.long())).long()
        scale = power(e.clamp(LOWEST, HIGHEST))
        scale = torch.where((low > 0)[:, None] & (old > 0), torch.maximum(scale, old), scale)
        scale = torch.where(written.any(1)[:, None], scale, old)
        keep = (torch.arange(block, device="cuda") < low[:, None])[:, None, :, None] & (low < block)[:, None, None, None]
        codes = torch.where(keep, codes * (old / scale)[..., None, None], codes)
        codes = torch.where(written[:, None, :, None], rows / scale[..., None, None], codes)
        out[kv + "_cache"] = back(codes, block, d).reshape(pages, Hkv, page, d)
        out[kv + "_scale"] = back(scale).reshape(pages, Hkv, page // block)
    return out


def _exact_paged(s):
    c = s["case"]
    n, G, page, block, d = c["n"], c["Hq"] // c["Hkv"], c["page"], c["block"], c["d"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for b, length in enumerate(s["lens"].tolist()):
        at = s["page_table"][b, :-(-length // page)].long()
        tree = s["mask"][b].bool() if n > 1 else torch.ones(1, 1, dtype=torch.bool, device="cuda")
        seen = torch.cat([torch.ones(n, length - n, dtype=torch.bool, device="cuda"), tree], 1).repeat(G, 1)
        for g in range(c["Hkv"]):
            k, v = ((s[kv + "_cache"].view(torch.uint8)[at, g].view(torch.float8_e4m3fn).double().view(-1, block, d) *
                     s[kv + "_scale"][at, g].double().view(-1, 1, 1)).view(-1, d)[:length] for kv in "kv")
            q = s["q"][b, :, g * G:(g + 1) * G].transpose(0, 1).reshape(G * n, d).double()
            z = (q @ k.t() / math.sqrt(d)).masked_fill(~seen, -math.inf)
            o = torch.softmax(z, -1) @ v
            out[b, :, g * G:(g + 1) * G] = o.view(G, n, d).transpose(0, 1)
    return out


def _exact_plan(s):
    """The same bookkeeping with lists, one request after the other."""
    c = s["case"]
    n, page, B = c["n"], c["page"], c["B"]
    table, held, free = s["table"].tolist(), s["held"].tolist(), s["free"].tolist()
    count = s["count"].tolist()[0]

    def step(lens, grow, rows, depth=None, path=None):
        nonlocal count
        want = [-(-(x + g) // page) if x >= 0 else 0 for x, g in zip(lens, grow)]
        for b in reversed(range(B)):
            for i in reversed(range(want[b], held[b])):
                free[count], count = table[b][i], count + 1
        for b in range(B):
            for i in range(held[b], want[b]):
                count -= 1
                table[b][i] = free[count]
            held[b] = want[b]
        slots, positions, starts = [], [], [0]
        for b in range(B):
            tokens = grow[b] if lens[b] >= 0 else 0
            for i in range(n or tokens):
                j = i if path is None else path[b].index(i) if i in path[b] else tokens
                at = lens[b] + j
                slots.append(table[b][at // page] * page + at % page if j < tokens else -1)
                positions.append((at if depth is None else lens[b] + depth[b][i] - 1) if j < tokens else 0)
            starts.append(starts[-1] + (n or tokens))
        out = dict(lens=[max(x, 0) + g if x >= 0 else 0 for x, g in zip(lens, grow)], cu_seqlens=starts)
        return dict(out, slots=slots, positions=positions) if rows else out

    lens, grow = s["lens"].tolist(), s["grow"].tolist()
    before = step(lens, grow, True, depth=s["depth"].tolist() if n else None)
    after = step(lens, s["kept"].tolist(), True, path=s["path"].tolist()) if n else step([-1] * B, grow, False)

    def tensors(x):
        return {k: tensors(v) for k, v in x.items()} if isinstance(x, dict) else torch.tensor(
            x, dtype=torch.int32, device="cuda")
    return tensors(dict(before=before, after=after, table=table, held=held, free=free, count=[count]))


def exact(case, seed):
    s = prepare(case, seed)
    return dict(plan=_exact_plan, append8=_exact_append, paged8=_exact_paged)[case["op"]](s)
