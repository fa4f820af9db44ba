"""Plain 64-bit forms of the packed pages and of attention over them, for the tests (numpy on the host)."""
from fractions import Fraction

import numpy as np
import torch

PAGE = 16


def pack_group(x):
    """(scale, lowest, codes) of one group of bf16 values, in exact arithmetic; None for a group with a value
    that is not finite."""
    x = [float(v) for v in x]
    if not all(np.isfinite(x)):
        return None
    lo, hi = min(x), max(x)
    want = (Fraction(hi) - Fraction(lo)) / 15
    # the least bf16 >= want, by bisection over the bit patterns of the non-negative bf16 numbers
    a, b = 0, 0x7F7F
    while a < b:
        m = (a + b) // 2
        if Fraction(float(np.uint32(m << 16).view(np.float32))) >= want:
            b = m
        else:
            a = m + 1
    s = Fraction(float(np.uint32(a << 16).view(np.float32)))
    codes = [0 if s == 0 else round((Fraction(v) - Fraction(lo)) / s) for v in x]   # round() of a Fraction: ties to even
    return float(s), lo, codes


def chunk_parts(chunk, d):
    """Codes [2][16][d], scales and lowest values [2][16][d / 64] of one (page, head) chunk (uint8)."""
    nb = d // 64
    c = np.asarray(chunk, np.uint8)
    n = nb * PAGE * 32
    by = c[:2 * n].reshape(2, nb, PAGE, 32)
    codes = np.stack([by & 15, by >> 4], axis=-1).reshape(2, nb, PAGE, 64).transpose(0, 2, 1, 3).reshape(2, PAGE, d)
    par = c[2 * n:].copy().view(np.uint16).reshape(2, nb, PAGE, 2).transpose(0, 2, 1, 3)
    f = (par.astype(np.uint32) << 16).view(np.float32)
    return codes, f[..., 0], f[..., 1]


def chunk_values(chunk, d):
    """Keys and values [2][16][d] that a chunk stands for, in 64 bits, and the same of scale * code and |lowest|."""
    codes, s, lo = chunk_parts(chunk, d)
    s64 = np.repeat(s.astype(np.float64), 64, axis=2)
    l64 = np.repeat(lo.astype(np.float64), 64, axis=2)
    return l64 + s64 * codes, s64 * codes, np.abs(l64)


def random_chunks(n, hkv, d, g):
    """Packed chunks [n][hkv][bytes] with random codes and parameters of a cache's size."""
    nb = d // 64
    codes = torch.randint(0, 256, (n, hkv, 4 * nb * PAGE * 16), generator=g, dtype=torch.uint8)
    s = 0.3 * torch.exp(0.3 * torch.randn(n, hkv, 2, nb, PAGE, generator=g))
    lo = -s * (7.5 + torch.randn(n, hkv, 2, nb, PAGE, generator=g))
    par = torch.stack([s, lo], dim=-1).to(torch.bfloat16).reshape(n, hkv, -1).view(torch.uint8)
    return torch.cat([codes, par], dim=-1).contiguous()


def attend(q, tokens, d):
    """One query [d] over `tokens`: a list of (key, value, scale * code of the value or None, bound of |key|, bound of
    |value|) rows. Returns the output, the log-sum-exp and the pieces that the tolerances are made of:
    sum p |v|, sum p (scale * code), max over tokens of sum |q| |k| / sqrt(d)."""
    if not tokens:
        return np.zeros(d), -np.inf, np.zeros(d), np.zeros(d), 0.0
    k = np.stack([t[0] for t in tokens])
    v = np.stack([t[1] for t in tokens])
    vc = np.stack([t[2] for t in tokens])
    ka = np.stack([t[3] for t in tokens])
    va = np.stack([t[4] for t in tokens])
    x = k @ q / np.sqrt(d)
    m = x.max()
    p = np.exp(x - m)
    z = p.sum()
    p = p / z
    return p @ v, m + np.log(z), p @ va, p @ vc, float((ka @ np.abs(q)).max() / np.sqrt(d))


def tolerances(d, T, lse, pv, pvc, s):
    """(of the output, of the log-sum-exp), before the output's own rounding to bf16.

    A logit is a sum of d products of exact factors in fp32 (each step off by at most 2^-23 of the sum of magnitudes s
    where partial sums are cut, plus a handful of steps for scale, lowest value and the constant log2 e): (d + 16) 2^-23 s.
    Every probability is then off by that, by exp2's 2^-22 and the fp32 rounding of its argument (below 2^-18 for logits
    below 64 / log2 e apart in what counts); sums of T terms add T 2^-24. The value product takes p * scale as fp16: half
    a step is 2^-11 of scale * code; 16-bit pages take p as two bf16 terms: 2^-16 of |v|."""
    dx = (d + 16) * 2.0 ** -23 * s + 2.0 ** -18 + T * 2.0 ** -24
    return 2 * dx * pv + 2.0 ** -11 * pvc + 2.0 ** -16 * pv, dx + 2.0 ** -22 * abs(lse)
