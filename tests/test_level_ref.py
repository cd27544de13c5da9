"""The inputs of level_ref show a block of keys that is left out, taken twice, or weighted by a wrong power of two, at
every length that the GPU tests use them at (no GPU needed: the wrong results are computed here, in 64 bits)."""
import pytest
import torch

import level_ref as lv
from test_levels_gpu import PAGED, PROMPTS, paged_chain, prompt_chain


def block_sums(x):
    """[rows, T, d] or [rows, T] -> the sums over blocks of 128 keys."""
    pad = -x.shape[1] % lv.BLOCK
    x = torch.cat([x, x.new_zeros(x.shape[:1] + (pad,) + x.shape[2:])], 1)
    return x.view(x.shape[0], -1, lv.BLOCK, *x.shape[2:]).sum(2)


def shows_every_block(T, d, seed, chain, segments):
    lev, v = lv.levels(T, seed), lv.values(T, d, seed)
    w = lv.weights(lev)
    l_b = block_sums(w)                                                # [rows, blocks]
    o_b, a_b = (torch.stack([block_sums((row[:, None] * x)[None])[0] for row in w]) for x in (v, v.abs()))
    O, l, A = o_b.sum(1), l_b.sum(1)[:, None], a_b.sum(1)
    exact = O / l
    limit = lv.bound(exact, A / l, chain, segments)
    assert limit.median() < 0.02
    if l_b.shape[1] == 1:
        return
    for times in (-1.0, 1.0, -0.5):  # left out, taken twice, at half its weight
        wrong = (O[:, None] + times * o_b) / (l[:, None] + times * l_b[..., None])
        off = (wrong.to(torch.bfloat16).double() - exact[:, None]).abs() > limit[:, None]
        seen = off.flatten(2).any(2).any(0)                            # by block
        assert seen.all(), (T, d, times, (~seen).nonzero()[:, 0].tolist()[:5])


@pytest.mark.parametrize("case", PAGED, ids=str)
def test_paged_inputs(case):
    lens, n, Hkv, d, _ = case
    for b, T in enumerate(lens):
        for g in {0, Hkv - 1}:
            shows_every_block(T, d, 17 * b + g, *paged_chain(lens, Hkv))


@pytest.mark.parametrize("T,d", PROMPTS)
def test_prompt_inputs(T, d):
    for g in range(2):
        shows_every_block(T, d, g, *prompt_chain(T))


def test_the_scale_is_one_in_base_two():
    assert abs(lv.base2_scale() - 0.6931471805599453) < 1e-7
