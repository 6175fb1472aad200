"""Plain 64-bit forms of the serving operations with bounds that count the
roundings of the kernels' own order, for tests of what a looser bound would hide."""
from __future__ import annotations

import math

import numpy as np
import torch

from tests.serving_reference import HALF_STEP, SUBNORMAL, f64


# -- attention ---------------------------------------------------------------------

def split_len(n):
    """Keys of a piece of a request of n keys."""
    s = 256 if n <= 2048 else 512
    while n > 128 * s:
        s *= 2
    return s


def attention_rel(n, D, group, dtype, A):
    """Relative error of a result, of sum p |v|, from the order that the header states.

    A: the largest scale * sum |q_d k_d|.  A score takes D / 16 tensor-core steps, each
    off by at most 2^-22 of A, and two roundings: eps_t in base 2 and, after t - m (at most
    2 A log2 e apart, 2^-24), in the exponent.  2^x is good to 2^-21; a key's weight goes
    through one for itself, one for every later tile of its warp that raises the maximum, and
    one in each join (two of warps for each of the H, one of pieces, one of groups).
    The weights count in the sum of v and in the sum that it is divided by.
    Sums of p v: a tensor-core step for each 16 keys of a warp and piece of p, 2^-22 each;
    a product with a raised maximum's factor a tile, and two roundings a join, 2^-24 each:
    H of warps, 16 of pieces, 8 of groups.  Sums of p: 2 KT adds of a tile and lane and one
    to the running sum, 3 of lanes, and the joins.  Pieces of p: 2^-24 (three bf16) or
    2^-22 (two fp16).  The division, two roundings."""
    W = 8 if D == 256 or (D == 128 and group > 8) else 4
    KT = 1 if D == 256 else 2
    H = W // 2
    own = -(-min(split_len(n), n) // (W * 16 * KT)) * 16 * KT  # keys of a warp
    tiles = own // (16 * KT)
    pieces, u = (2, 2.0 ** -22) if dtype == torch.float16 else (3, 2.0 ** -24)
    eps_t = A * math.log2(math.e) * (D / 16 * 2.0 ** -22 + 2.0 ** -23 + 2.0 ** -23)
    weight = math.log(2) * eps_t + (1 + tiles + H + 2) * 2.0 ** -21
    joins = 2 * (H + 16 + 8) * 2.0 ** -24
    sums = own / 16 * pieces * 2.0 ** -22 + tiles * 2.0 ** -24 + joins
    total = (tiles * (2 * KT + 2) + 3) * 2.0 ** -24 + joins
    return u + 2 * weight + sums + total + 2.0 ** -22


def attention(q, k, v, scale, dtype, out_dtype):
    """(result, bound) of one request: q [Hq, D] over its keys and values [n, Hkv, D] in order."""
    q, k, v = (f64(x) if isinstance(x, torch.Tensor) else x for x in (q, k, v))
    (Hq, D), (n, Hkv, _) = q.shape, k.shape
    G = Hq // Hkv
    ref, bound = np.zeros((Hq, D)), np.zeros((Hq, D))
    for g in range(Hkv):
        kh, vh, qh = k[:, g], v[:, g], q[g * G:(g + 1) * G]
        s = scale * (qh @ kh.T)
        A = abs(scale) * (np.abs(qh) @ np.abs(kh).T).max()
        p = np.exp(s - s.max(-1, keepdims=True))
        p /= p.sum(-1, keepdims=True)
        o = p @ vh
        err = attention_rel(n, D, G, dtype, A) * (p @ np.abs(vh))
        if dtype == torch.float16:
            # p is scaled by 2^15 before it is cut into fp16 numbers, whose subnormals are
            # 2^-24 apart: 2^-40 of a warp's largest weight, which is at most the largest
            err = err + 2.0 ** -40 * p.max(-1, keepdims=True) * np.abs(vh).sum(0)
        ref[g * G:(g + 1) * G] = o
        bound[g * G:(g + 1) * G] = err + (np.abs(o) + err) * HALF_STEP[out_dtype] + SUBNORMAL[out_dtype]
    return ref, bound


# -- rotary positions -----------------------------------------------------------------

PI_BITS = 1400


def _pi():
    """pi * 2^PI_BITS, by 16 arctan(1/5) - 4 arctan(1/239)."""
    one = 1 << (PI_BITS + 32)

    def arctan_inverse(x):
        term = total = one // x
        k, sign = 3, -1
        while term:
            term //= x * x
            total += sign * (term // k)
            k, sign = k + 2, -sign
        return total
    return (16 * arctan_inverse(5) - 4 * arctan_inverse(239)) >> 32


PI = _pi()


def turns(f, n, bits):
    """n f / (2 pi) modulo one turn, in units of 2^-bits turns, rounded down (a double f, an integer n)."""
    num, den = float(f).as_integer_ratio()
    # num n / den / (2 pi) = num n 2^PI_BITS / (2 PI den)
    return ((num * int(n)) << (PI_BITS + bits)) // (2 * PI * den) % (1 << bits)


def angles(freq, pos):
    """The reduced angles in (-pi, pi], [positions, pairs], to the precision of a double."""
    out = np.zeros((len(pos), len(freq)))
    for i, n in enumerate(pos):
        for j, f in enumerate(freq):
            t = turns(f, n, 128)
            out[i, j] = (t - (1 << 128) if t > 1 << 127 else t) / 2.0 ** 127 * math.pi
    return out


# -- values that show every key's share ---------------------------------------------------

def marked_values(n, Hkv, D, every):
    """Values [n, Hkv, D] that are one number in one dimension and 0 in the others: blocks of
    `every` keys take the dimensions in turn, the number 1 in the first round, 1.5 in the
    second and so on, so a result is the mass of few blocks and none averages out."""
    block = np.arange(n) // every
    v = np.zeros((n, Hkv, D))
    v[np.arange(n), :, block % D] = (1 + 0.5 * (block // D))[:, None]
    return v


# -- token log probabilities -----------------------------------------------------------------

def logprobs_sum_error(N, dtype):
    """Relative error of a row's sum of exponentials, from the order that the header states:
    16 adds of a chunk and one of its halves (2^-24 each); a join of every slice of a group, of
    every group, of 5 rounds of lanes and 3 of warps, two roundings and one factor 2^x (2^-22)
    each; and 2^x of the element itself."""
    slices = -(-N // (4096 if dtype == torch.float32 else 8192))
    per_group = -(-slices // 8)
    joins = per_group + -(-slices // per_group) + 8
    return (17 + 2 * joins) * 2.0 ** -24 + (joins + 1) * 2.0 ** -22


def logprobs_bounds(x, lp, dtype):
    """Bounds of (log probabilities lp, entropies) of ordinary rows x [R, N] in 64 bits: the argument
    of 2^x is one rounding of x log2 e - m', log2 e itself good to 2^-26: 2^-22 |z| in the exponential."""
    z = x - x.max(-1, keepdims=True)
    e = np.exp(z)
    S = e.sum(-1)
    with np.errstate(invalid="ignore"):
        spread = np.where(e > 0, -e * z, 0.0).sum(-1) / S
        square = np.where(e > 0, e * z * z, 0.0).sum(-1) / S
    err = logprobs_sum_error(x.shape[1], dtype)
    log_sum = err + 2.0 ** -22 * spread + 2.0 ** -22 * np.abs(np.log(S))
    at = (...,) + (None,) * (lp.ndim - 1)
    # the differences' and the result's roundings
    lp_bound = log_sum[at] + 2.0 ** -23 * np.abs(np.where(np.isfinite(lp), lp, 0.0)) + 2.0 ** -23 * np.log(S)[at]
    # H is a sum of terms of one sign: its own sum's error and S's, t's rounding, the division
    entropy = log_sum + (2 * err + 2.0 ** -21) * spread + 2.0 ** -22 * square + 2.0 ** -23 * (spread + np.log(S))
    return lp_bound, entropy


def marked_rows(N, dtype):
    """Index sets on whose elements a row may have all its weight: the last and first ones, and
    those at and around the boundaries of units, warps, stages, slices and groups."""
    E = 4 if dtype == torch.float32 else 8
    slices = -(-N // (1024 * E))
    sets = [range(N - k, N) for k in range(1, 17)] + [range(k) for k in (1, 2, 3, 5, 7, 8, 9, 16)]
    for b in (E, 31 * E, 32 * E, 33 * E, 255 * E, 256 * E, 512 * E, 768 * E, 1024 * E, 1024 * E * -(-slices // 8),
              1024 * E * (slices - 1), N // E * E, N // (256 * E) * 256 * E):
        sets += [range(b - 1, b + 1), range(b, b + E), range(b - E, b), range(b - 3, b + 13)]
    sets = [[j for j in s if 0 <= j < N] for s in sets]
    return [s for s in sets if s]
