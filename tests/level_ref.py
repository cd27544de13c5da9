"""Attention whose exact result shows every single block of 128 keys, however long the sequence.

With random real inputs an output shrinks like 1 / sqrt(keys) while the bound on sums of many terms grows, and a lost
block of a long cache hides below it. Here the inputs make a kernel's weights and weighted sums exact, so that the bound
stays small:
- a key's score is a * level, a small whole number (the query is (a, 0, 0, ...), the key (level, noise ...)), in base 2
  because scale * log2(e) is 1 in fp32; a weight is a power of two times 1 + 2^-22 at most, and rounded to bf16 it is
  that power;
- the values are whole numbers of at most 8 in size: sums of weighted values are multiples of the least weight, and as
  long as they stay below 2^24 of it (levels to 3, a to 2: 2^6 * 8 per key, up to 32000 keys in one sum) fp32 holds
  them exactly in any order.
What is left for a kernel that adds a row's weights in fp32 by chains of `chain` additions, joins `segments` parts by
powers of two (three roundings of 2^-22 each), divides and rounds to bf16: with A = sum_j w_j |v_j| / sum_j w_j
    |out - exact| <= 2^-8 |exact| + A (2^-20 + chain 2^-24 + 3 segments 2^-22)."""
import numpy as np
import torch

SLOPES = (0, 1, 2, -1)  # a query head's a: flat, rising, steep, falling
BLOCK = 128


def base2_scale():
    """The fp32 scale whose product with log2(e) is 1 in fp32."""
    log2e = np.float32(1.4426950408889634)
    near = np.float32(np.log(2.0))
    for s in (near, np.nextafter(near, np.float32(0)), np.nextafter(near, np.float32(1))):
        if np.float32(s * log2e) == np.float32(1):
            return float(s)
    raise AssertionError("no such scale")


def levels(T, seed):
    """Levels 0 to 3 of T keys: a block's, and one more for half of its keys."""
    g = torch.Generator().manual_seed(seed)
    block = torch.randint(0, 3, (-(-T // BLOCK),), generator=g).repeat_interleave(BLOCK)[:T]
    return block + torch.randint(0, 2, (T,), generator=g)


def values(T, d, seed):
    return torch.randint(-8, 9, (T, d), generator=torch.Generator().manual_seed(seed + 1000)).double()


def keys(lev, d, seed):
    g = torch.Generator().manual_seed(seed + 2000)
    k = torch.randn(len(lev), d, generator=g)
    k[:, 0] = lev.float()
    return k.to(torch.bfloat16)


def queries(d):
    """[4, d]: one row per slope."""
    q = torch.zeros(len(SLOPES), d)
    q[:, 0] = torch.tensor(SLOPES, dtype=torch.float32)
    return q.to(torch.bfloat16)


def weights(lev):
    """[slopes, T] fp64."""
    return 2.0 ** (torch.tensor(SLOPES, dtype=torch.float64, device=lev.device)[:, None] * lev.double())


def bound(exact, A, chain, segments):
    return 2.0 ** -8 * exact.abs() + A * (2.0 ** -20 + chain * 2.0 ** -24 + 3 * segments * 2.0 ** -22)
