"""Plain attention in 64 bits, row by row, with the error that bf16 kernels may make on it.

The bound, element by element, for a kernel that multiplies bf16 inputs exactly, accumulates in fp32, rounds the softmax
weights to bf16 and the output to bf16 (a rounding is off by at most half a step, 2^-8 of the value in bf16, 2^-24 in
fp32; the tensor cores may cut instead of rounding, so their fp32 steps count 2^-23). With A = sum_j w_j |v_j|:
- the weights' rounding: 2^-8 A; the output's: 2^-8 |out|;
- a score is d products: off by at most (d + 4) 2^-23 sum |q||k| scale =: e; a weight is exp of it, off by the factor
  e + 2^-21 (the approximate exponential), and so is the sum that divides: 2 (e + 2^-21) A;
- sums over T keys in fp32, of the weights and of the weighted values: 2 T 2^-23 A."""
import torch


def attend(q, k, v, seen, scale):
    """One head: q [rows,d], k, v [keys,d], seen [rows,keys] bool -> (out, bound) [rows,d] fp64. A row that sees nothing
    is zero; what a row does not see does not enter it."""
    q, k, v = q.double(), k.double(), v.double()
    used = seen.any(0)
    q, k, v, seen = q, k[used], v[used], seen[:, used]
    if k.shape[0] == 0:
        return torch.zeros_like(q), torch.zeros_like(q)
    z = (q @ k.t() * scale).masked_fill(~seen, -torch.inf)
    top = z.amax(1, keepdim=True)
    w = torch.exp(z - torch.where(top == -torch.inf, torch.zeros_like(top), top)) * seen
    total = w.sum(1, keepdim=True)
    w = torch.where(total > 0, w / total, torch.zeros_like(w))
    out, A = w @ v, w @ v.abs()
    d, T = q.shape[1], k.shape[0]
    e = (d + 4) * 2.0 ** -23 * scale * (q.abs() @ k.abs().t()).mul(seen).amax(1, keepdim=True)
    return out, 2.0 ** -8 * (A + out.abs()) + A * (2 * (e + 2.0 ** -21) + 2 * T * 2.0 ** -23)


def check(out, ref, bound):
    """Every element within its bound (and exactly zero where the bound is zero and the reference is)."""
    off = (out.double() - ref).abs()
    worst = (off - bound).max().item()
    assert not torch.isnan(off).any(), "NaN in the output"
    assert worst <= 0, f"off by {off.max().item():.3g}, over the bound by {worst:.3g}"
