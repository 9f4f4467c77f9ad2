"""Error bounds of paged attention that stay below the outputs at long contexts.

kv_ref.bounds allows for n fp32 roundings of a sum over n keys, and for 2^-25 per key below
f16's range. The kernels do better, and these bounds hold them to it:
  * sums: an fp32 number takes one rounding (of at most 2^-23, truncation included) per
    16 keys of one product or per few keys of a lane's own sum, and 64 more for the joining of lanes,
    warps and parts: (n / 16 + 64) 2^-23, with 2^-20 for the exponential;
  * f16 probabilities (all caches but BF16) stand at 2^7 or more for a row's largest, so what
    f16's smallest step rounds off is at most 2^-25 2^-7 of the largest each.
The other terms are kv_ref's.
"""
import torch


def tight(fmt, out, lse, mag, dots, n, vmax):
    """(bound of |out error| [T, Hq, D], bound of |lse error| [T, Hq]); arguments as kv_ref.bounds."""
    D = out.shape[-1]
    logit = (D + 4) * 2.0 ** -24 * dots + 2.0 ** -22 * (1.45 * dots + 1)
    if fmt == "q8_0":
        logit = logit + 2.0 ** -11 * dots
    sums = (n / 16 + 64) * 2.0 ** -23 + 2.0 ** -20
    u = 2.0 ** -8 if fmt == "bf16" else 2.0 ** -11
    if fmt == "q8_0":
        u += 2.0 ** -11
    rel = torch.expm1(2 * logit) + u + 2 * sums
    small = 0.0 if fmt == "bf16" else n * 2.0 ** -32 * vmax
    b = mag * rel[..., None] + small
    b = b + 2.0 ** -8 * (out.abs() + b) + 1e-38
    return b, logit + sums + 2.0 ** -22 * lse.abs().nan_to_num(0, 0, 0) + 1e-6


def drift(n, heads, dim, g, device="cpu"):
    """Value means [n, heads, dim] of size 3 that turn once along the sequence, each channel at a
    phase of its own: their sum over the whole sequence is near zero, over any contiguous
    part it is not in some channel, so an output that misses, doubles or misweights a part is
    off by about three times the part's softmax weight."""
    phase = 6.2831853 * torch.rand((1, heads, dim), generator=g, device=device)
    turn = 6.2831853 * torch.arange(n, device=device)[:, None, None] / n
    return 3 * torch.cos(turn + phase)
