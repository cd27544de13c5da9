"""Rows whose scores leave the headroom of the running maximum, and values that are not finite, at both head widths and
in every place of a block: the branches that random inputs hardly take. Against attention in 64 bits (attention_ref); at
these lengths the bound's sums are small beside its roundings."""
import math

import pytest
import torch

import test_paged_attn_gpu as paged
import test_prompt_attn_gpu as prompt

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
# growth of a row's scores in base 2: inside the headroom (2^20), between it and what a sum of weights may reach (2^26),
# just beyond, far beyond
GROWTH = [19.5, 22.0, 25.5, 27.0, 60.0, 300.0]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("start", [20, 127, 128, 200, 259, 384, 511, 530])
@pytest.mark.parametrize("some", [1, 3, 16])
def test_prompt_rows_that_leave_the_headroom(dtlib, d, start, some):
    """From key `start` on every key (or one of `some`) scores higher, for one of `some` query rows: in a block's middle
    and at its ends, in the block on the diagonal of the first and of the second tile, in some rows of a warp only."""
    for growth in GROWTH:
        s = prompt.make([600, 300], 4, 2, d, fused=False, spread=0.5)
        s["q"][..., 0] = 0.0
        s["q"][some - 1::some, :, 0] = 4.0
        s["k"][..., 0] = 0.0
        s["k"][start::some, :, 0] = growth * math.log(2) / 4 / s["scale"]
        prompt.parity(dtlib, s)


@pytest.mark.parametrize("d", [64, 128])
def test_prompt_scores_that_rise_block_by_block(dtlib, d):
    """Every block of every row leaves the headroom that the blocks before it set."""
    s = prompt.make([900], 4, 2, d, fused=False, spread=0.5)
    s["q"][..., 0] = 4.0
    s["k"][..., 0] = (torch.arange(900, device="cuda") // 128 * 30.0 * math.log(2) / 4 / s["scale"])[:, None]
    prompt.parity(dtlib, s)


@pytest.mark.parametrize("d", [64, 128])
def test_prompt_scores_far_apart(dtlib, d):
    s = prompt.make([900], 4, 2, d, fused=False, spread=20.0)
    s["k"] *= (torch.arange(900, device="cuda") // 60 + 1)[:, None, None] / 8
    prompt.parity(dtlib, s)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,Hq", [(1, 8), (4, 8), (16, 16)])
@pytest.mark.parametrize("start", [1, 100, 128, 500, 997])
def test_paged_rows_that_leave_the_headroom(dtlib, d, n, Hq, start):
    """As for prompts; every second query head's scores grow."""
    for growth in GROWTH:
        s = paged.make([1000, 515, 128 + n], n, Hq, 2, d, 16, mask="tree" if n > 1 else None, spread=0.5)
        s["q"][..., 0] = 0.0
        s["q"][:, :, 1::2, 0] = 4.0
        s["kc"][..., 0] = 0.0
        for b in range(3):
            for key in range(start, int(s["lens"][b])):
                if key % 16 == 0 or key == start:  # the rest of a page at once
                    page = int(s["table"][b, key // 16])
                    s["kc"][page, :, key % 16:, 0] = growth * math.log(2) / 4 / s["scale"]
        paged.parity(dtlib, s)


@pytest.mark.parametrize("d", [64, 128])
def test_paged_scores_far_apart(dtlib, d):
    s = paged.make([1500, 300], 2, 8, 2, d, 16, mask="tree", spread=20.0)
    for b in range(2):
        for i in range(int(s["lens"][b]) // 16):
            s["kc"][s["table"][b, i].long()] *= (i + 1) / 16
    paged.parity(dtlib, s)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_what_is_not_finite_in_a_prompt_at_every_token(dtlib, d, bad):
    """A value that is not finite, at every token of a prompt in turn, reaches the rows that see it and no other, bit for
    bit; so does a key."""
    s = prompt.make([50, 300, 400], 4, 2, d, fused=False)
    clean = prompt.run(dtlib, s).clone()
    hit = torch.zeros_like(clean, dtype=torch.bool)
    for at in range(50, 350):
        v0, k0 = s["v"][at, 1, d - 3].clone(), s["k"][at, 0, 3].clone()
        s["v"][at, 1, d - 3] = bad
        out = prompt.run(dtlib, s)
        hit[:] = False
        hit[at:350, 2:, d - 3] = True
        assert torch.equal(out[~hit], clean[~hit]), at
        assert out[hit].isnan().all() if math.isnan(bad) else (out[hit] == bad).all(), at
        s["v"][at, 1, d - 3] = v0
        if math.isnan(bad):
            s["k"][at, 0, 3] = bad
            out = prompt.run(dtlib, s)
            hit[:] = False
            hit[at:350, :2] = True
            assert out[hit].isnan().all() and torch.equal(out[~hit], clean[~hit]), at
            s["k"][at, 0, 3] = k0


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("Hq", [2, 32])
def test_what_is_not_finite_in_a_tree_of_narrow_heads(dtlib, bad, Hq):
    n = 8 if Hq == 2 else 4
    s = paged.make([130, 64, n], n, Hq, 2, 64, 16, mask="tree")
    s["mask"][:] = torch.eye(n, dtype=torch.uint8, device="cuda")
    s["mask"][:, 3, 1] = 1
    clean = paged.run(dtlib, s).clone()
    for b in range(3):
        key = int(s["lens"][b]) - n + 1  # node 1's: seen by nodes 1 and 3
        s["vc"][s["table"][b, key // 16].long(), 1, key % 16, 33] = bad
    out = paged.run(dtlib, s)
    hit = torch.zeros_like(out, dtype=torch.bool)
    hit[:, [1, 3], Hq // 2:, 33] = True
    assert torch.equal(out[~hit], clean[~hit])
    assert out[hit].isnan().all() if math.isnan(bad) else (out[hit] == bad).all()


@pytest.mark.parametrize("d", [64, 128])
def test_the_most_of_everything(dtlib, d):
    """The most requests, nodes and query rows at once (the plan and the queries leave the ring its least room)."""
    lens = [64 + (29 * i) % 150 if i % 9 else 0 for i in range(2048)]
    paged.parity(dtlib, paged.make(lens, 64, 2, 1, d, 16, mask="tree"), requests=[0, 1, 2, 9, 700, 2046, 2047])
