"""Long caches and prompts on the GPU with the inputs of level_ref, where a block of keys that is lost, taken twice or
joined with a wrong weight shows (test_level_ref checks that it does)."""
import math

import pytest
import torch

import level_ref as lv

BF = torch.bfloat16
SMS = 152

# lens, nodes, key/value heads, head width, page size
PAGED = [
    ([100003], 1, 2, 128, 64),          # some 76 segments a pair
    ([65536, 40, 1000], 1, 2, 128, 64),
    ([30000], 1, 1, 128, 64),           # one pair over every CTA
    ([20011, 3, 700], 1, 4, 64, 128),
    ([131071], 1, 8, 64, 16),
    ([5000, 9000, 300], 3, 1, 64, 16),
    ([2049], 1, 8, 128, 64),
    ([4000, 3000, 130, 129], 16, 2, 128, 16),
    ([40000, 257], 16, 1, 64, 256),
]
PROMPTS = [(8200, 64), (8200, 128), (20000, 64), (385, 128), (1025, 64)]


def paged_chain(lens, Hkv):
    """Additions in a row of a thread's weights, and segments of a pair, at most: a CTA's share is an even part of the
    blocks and a unit per pair; of a block a thread adds 16 weights of a row by two chains of eight."""
    units = sum(-(-T // lv.BLOCK) + 1 for T in lens) * Hkv
    share = -(-units // SMS) + 1
    longest = -(-max(lens) // lv.BLOCK)
    return 10 * share + 4, min(SMS, longest // max(share - 2, 1) + 2)


def prompt_chain(T):
    return 10 * -(-T // lv.BLOCK) + 4, 0


def within(out, exact, limit):
    off = (out.double() - exact).abs()
    assert not off.isnan().any()
    assert (off <= limit).all(), f"off by {off.max().item():.3g}, over by {(off - limit).max().item():.3g}"


@pytest.mark.gpu
@pytest.mark.parametrize("case", PAGED, ids=str)
def test_every_block_of_a_long_cache_counts_once(dtlib, case):
    lens, n, Hkv, d, page = case
    S, B = len(lv.SLOPES), len(lens)
    used = [-(-T // page) for T in lens]
    order = torch.randperm(sum(used) + 2, generator=torch.Generator().manual_seed(1)).tolist()
    kc, vc = (torch.full((sum(used) + 2, Hkv, page, d), float("nan"), dtype=BF, device="cuda") for _ in range(2))
    table = torch.full((B, max(used)), -7, dtype=torch.int32)
    lev, val = {}, {}
    for b, T in enumerate(lens):
        pages = [order.pop() for _ in range(used[b])]
        table[b, :used[b]] = torch.tensor(pages)
        for g in range(Hkv):
            lev[b, g], v = lv.levels(T, 17 * b + g), lv.values(T, d, 17 * b + g)
            for pool, x in ((kc, lv.keys(lev[b, g], d, 17 * b + g)), (vc, v.to(BF))):
                rows = torch.full((used[b] * page, d), float("nan"), dtype=BF)
                rows[:T] = x
                pool[torch.tensor(pages, device="cuda"), g] = rows.view(used[b], page, d).cuda()
            lev[b, g], val[b, g] = lev[b, g].cuda(), v.cuda()
    q = lv.queries(d).cuda().repeat(Hkv, 1).expand(B, n, Hkv * S, d).contiguous()
    mask = torch.eye(n, dtype=torch.uint8, device="cuda").repeat(B, 1, 1) if n > 1 else None  # a node and the prefix
    ws = dtlib.new_workspace(dtlib.dt_paged_attention_workspace_bytes(B, n, Hkv * S, Hkv, d))
    out = dtlib.dt_paged_attention(q, kc, vc, table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                   lv.base2_scale(), mask=mask, workspace=ws)
    assert dtlib.dt_get_error(ws) == dtlib.Status.OK
    chain, segments = paged_chain(lens, Hkv)
    for b, T in enumerate(lens):
        for g in range(Hkv):
            w, v = lv.weights(lev[b, g]), val[b, g]
            pre = T - n
            O, A, l = w[:, :pre] @ v[:pre], w[:, :pre] @ v[:pre].abs(), w[:, :pre].sum(1, keepdim=True)
            for i in range(n):
                own = w[:, pre + i, None]
                exact, a = (O + own * v[pre + i]) / (l + own), (A + own * v[pre + i].abs()) / (l + own)
                within(out[b, i, g * S:(g + 1) * S], exact, lv.bound(exact, a, chain, segments))


@pytest.mark.gpu
@pytest.mark.parametrize("T,d", PROMPTS)
def test_every_block_of_a_long_prompt_counts_once(dtlib, T, d):
    S, Hkv, other = len(lv.SLOPES), 2, 70
    lev = [lv.levels(T, g) for g in range(Hkv)]
    val = [lv.values(T, d, g) for g in range(Hkv)]
    k, v = (torch.randn(T + other, Hkv, d, generator=torch.Generator().manual_seed(3)).to(BF) for _ in range(2))
    for g in range(Hkv):
        k[:T, g], v[:T, g] = lv.keys(lev[g], d, g), val[g].to(BF)
    q = lv.queries(d).repeat(Hkv, 1).expand(T + other, Hkv * S, d).contiguous().cuda()
    cu = torch.tensor([0, T, T + other], dtype=torch.int32, device="cuda")
    out = dtlib.dt_prompt_attention(q, k.cuda(), v.cuda(), cu, lv.base2_scale())
    chain, segments = prompt_chain(T)
    for g in range(Hkv):
        w, x = lv.weights(lev[g].cuda()), val[g].cuda()
        for r in range(S):
            l = w[r].cumsum(0)[:, None]
            exact, A = (w[r][:, None] * x).cumsum(0) / l, (w[r][:, None] * x.abs()).cumsum(0) / l
            within(out[:T, g * S + r], exact, lv.bound(exact, A, chain, segments))
