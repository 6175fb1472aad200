"""Plain 64-bit implementations of the serving operations, and the bounds the
kernels' results are held to (derived at each bound)."""
from __future__ import annotations

import math

import numpy as np
import torch

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
# half the spacing of the subnormals (bf16 and fp32 reach far below any value here)
SUBNORMAL = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25, torch.float32: 0.0}


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def assert_within(got, ref, bound, what=""):
    g = f64(got)
    assert g.shape == ref.shape, (g.shape, ref.shape)
    bad = ~(np.abs(g - ref) <= bound)  # a NaN fails
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} out of bounds, first at {i}: "
                             f"{g[i]} for {ref[i]}, allowed {np.broadcast_to(bound, g.shape)[i]}")


# -- page planning -----------------------------------------------------------------

def plan(ctx, new, table, pool, page, T):
    ctx, new = [max(0, int(c)) for c in ctx], [max(0, int(n)) for n in new]
    table = np.array(table)
    W, F = table.shape[1], len(pool)
    pos, slots = np.zeros(T, np.int32), np.full(T, -1, np.int64)
    at = taken = 0
    offsets = [0]
    for b, (c, n) in enumerate(zip(ctx, new)):
        for col in range(-(-c // page), -(-(c + n) // page)):
            if col < W:
                table[b, col] = pool[taken] if taken < F else -1
            taken += 1
        for i in range(n):
            p = c + i
            if at + i < T:
                pos[at + i] = p
                pg = table[b, p // page] if p // page < W else -1
                slots[at + i] = -1 if pg < 0 else int(pg) * page + p % page
        at += n
        offsets.append(at)
    return table, np.array(ctx) + np.array(new), np.array(offsets), pos, slots, np.array([taken, at])


# -- rotary positions ------------------------------------------------------------------

def frequencies(rotary, base=10000.0, kind=None, factor=1.0, original=0.0, low=0.0, high=0.0):
    if kind == "base":
        base = base * factor ** (rotary / (rotary - 2))
    f = [base ** (-2.0 * i / rotary) for i in range(rotary // 2)]
    if kind == "linear":
        f = [x / factor for x in f]
    elif kind == "ramp_turns":
        for i, x in enumerate(f):
            g = min(1.0, max(0.0, (original * x / (2 * math.pi) - low) / (high - low)))
            f[i] = x * (g + (1 - g) / factor)
    elif kind == "ramp_index":
        def idx(r):
            return rotary * math.log(original / (2 * math.pi * r)) / (2 * math.log(base))
        hi, lo = max(math.floor(idx(high)), 0), min(math.ceil(idx(low)), rotary - 1)
        for i, x in enumerate(f):
            g = 1 - min(1.0, max(0.0, (i - hi) / max(lo - hi, 1e-3)))
            f[i] = x * (g + (1 - g) / factor)
    return np.array(f)


def rope(x, pos, freq, interleaved, backward=False, magnitude=1.0):
    """(result, |x1| + |x2| of each element's pair, 0 for copied elements)"""
    x = f64(x) if isinstance(x, torch.Tensor) else np.array(x, np.float64)
    pos = [int(p) for p in pos]
    half = len(freq)
    # the angle's whole turns are taken off in extended integers: positions of any size
    turns = np.array([[math.fmod(p * f / (2 * math.pi), 1.0) if abs(p) < 2 ** 22 else
                       float((int(p) * int(f / (2 * math.pi) * 2 ** 80)) % 2 ** 80) / 2 ** 80 for f in freq]
                      for p in pos]).reshape(len(pos), half)
    c, s = np.cos(2 * np.pi * turns)[:, None], np.sin(2 * np.pi * turns)[:, None]
    if backward:
        s = -s
    i1 = np.arange(half) * 2 if interleaved else np.arange(half)
    i2 = i1 + (1 if interleaved else half)
    y, size = x.copy(), np.zeros_like(x)
    y[..., i1] = magnitude * (x[..., i1] * c - x[..., i2] * s)
    y[..., i2] = magnitude * (x[..., i1] * s + x[..., i2] * c)
    size[..., i1] = size[..., i2] = abs(magnitude) * (np.abs(x[..., i1]) + np.abs(x[..., i2]))
    return y, size


def rope_bound(ref, size, dtype):
    """The half-turn argument is off by 2^-25 + 2^-31 (its fp32 rounding and the dropped
    low word), 9.5e-8 in the angle; sincospif by 2 ulp at most, 2^-23; the multiply by
    the magnitude by 2^-24: 2.8e-7 of |x1| + |x2|.  The pair's product and fused
    multiply-add add 2^-24 each, 1.2e-7.  Together under 2^-21 = 4.8e-7, then the
    rounding to the output type."""
    e = 2.0 ** -21 * size
    return e + (np.abs(ref) + e) * HALF_STEP[dtype] + SUBNORMAL[dtype]


# -- attention -----------------------------------------------------------------------------

def attention(q, kc, vc, table, lens, scale, out_dtype):
    """(result, bound) of one token per request over the paged cache."""
    B, Hq, D = q.shape
    P, page, Hkv, _ = kc.shape
    G = Hq // Hkv
    table, lens = table.cpu().numpy(), lens.cpu().numpy()
    q64 = f64(q)
    ref, bound = np.zeros((B, Hq, D)), np.zeros((B, Hq, D))
    u = HALF_STEP[q.dtype] ** (3 if q.dtype == torch.bfloat16 and out_dtype == torch.float32 else 2)
    for b in range(B):
        n = max(0, min(int(lens[b]), table.shape[1] * page))
        j = np.arange(n)
        pages = table[b, j // page]
        ok = (pages >= 0) & (pages < P)
        j, pages = j[ok], pages[ok]
        n = len(j)
        if n == 0:
            continue
        flat = torch.as_tensor(pages.astype(np.int64) * page + j % page, device=kc.device)
        # rows gathered on the device (a cache may be larger than host memory)
        k, v = f64(kc[flat // page, flat % page]), f64(vc[flat // page, flat % page])
        for h in range(Hq):
            kh, vh = k[:, h // G], v[:, h // G]
            s = scale * (kh @ q64[b, h])
            A = abs(scale) * np.max(np.abs(kh) @ np.abs(q64[b, h]))
            e = np.exp(s - s.max())
            p = e / e.sum()
            ref[b, h] = p @ vh
            # A score takes D / 16 <= 16 tensor-core steps, each off by at most 2^-22 of
            # A (products exact, sums truncated), the scaled score two roundings: under
            # 2^-17 A; t - m and m's own rescaling add 2^-22 A: 2^-16 A in the exponent.
            # 2^x is good to 2^-21.  Both count in p and in the sum it is divided by.
            # p is carried in two pieces of the cache's type, three bf16 for an fp32 result: u.
            # The sums over n keys: n 2^-23.  The division, two roundings: 2^-22.
            rel = u + 2 * (2.0 ** -16 * A + 2.0 ** -21) + n * 2.0 ** -23 + 2.0 ** -22
            err = rel * (p @ np.abs(vh))
            # fp16 pieces below 2^-14 are subnormal: half a spacing a key, in units of
            # the largest p, which is at most p.max() after the division
            err = err + n * 2.0 ** -25 * p.max() * np.abs(vh).max() * (q.dtype == torch.float16)
            bound[b, h] = err + (np.abs(ref[b, h]) + err) * HALF_STEP[out_dtype] + SUBNORMAL[out_dtype]
    return ref, bound


# -- token log probabilities ---------------------------------------------------------------

def logprobs(x, tokens, top):
    """(lp, entropy, top lp, top ids) and the bounds of the first three."""
    x = f64(x)
    R, N = x.shape
    tokens = [int(t) for t in tokens]
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        m = x.max(-1, keepdims=True)
        z = x - m
        e = np.exp(z)
        S = e.sum(-1, keepdims=True)
        logp = z - np.log(S)
        ez = np.where(e > 0, e * z, 0.0 * e)
        ent = np.log(S[:, 0]) - ez.sum(-1) / S[:, 0]
        lp = np.array([logp[r, t] if 0 <= t < N else -np.inf for r, t in enumerate(tokens)])
        # NaN first, then by value, then by index
        ids = np.stack([np.lexsort((np.arange(N), -np.where(np.isnan(r), np.inf, r), ~np.isnan(r)))[:top] for r in x]) \
            if R else np.zeros((0, top), np.int64)
        tlp = np.take_along_axis(logp, ids, -1) if R else np.zeros((0, top))

        # 2^x is good to 2^-21.  Its argument is one rounding of x log2 e - m', so off by
        # 2^-24 |z| log2 e, and log2 e by 2^-26 of itself: 2^-22 |z| in the exponential.  A
        # sum goes through at most 16 adds of a chunk, 8 joins of groups and 9 of lanes and
        # warps, in rows of up to 8 slices a group (longer ones add one join a slice), three
        # roundings each: 2^-24 * 100 < 2^-17.  Rows out of the ordinary take expf and up to
        # 600 adds a thread: 2^-24 * 640 < 2^-14.6 at N = 300001.  2^-14 covers both.
        spread = np.where(e > 0, e * np.abs(z), 0.0).sum(-1) / S[:, 0]
        square = np.where(e > 0, e * z * z, 0.0).sum(-1) / S[:, 0]
        d_lse = 2.0 ** -14 + 2.0 ** -22 * spread + 2.0 ** -22 * np.abs(np.log(S[:, 0]))

        def lp_bound(v):  # z's, the subtraction's and the result's roundings
            return d_lse.reshape((-1,) + (1,) * (v.ndim - 1)) + 2.0 ** -23 * np.abs(np.where(np.isfinite(v), v, 0.0)) + \
                2.0 ** -23 * np.abs(np.log(S)).reshape((-1,) + (1,) * (v.ndim - 1))
        ent_bound = d_lse + 2.0 ** -13 * spread + 2.0 ** -21 * square + 2.0 ** -23 * np.abs(ent)
    return lp, ent, tlp, ids, lp_bound(lp), ent_bound, lp_bound(tlp)


def assert_same_nonfinite(got, ref, bound, what=""):
    g = f64(got)
    fin = np.isfinite(ref)
    assert np.array_equal(np.isnan(g), np.isnan(ref)), what
    assert np.array_equal(g[~fin & ~np.isnan(ref)], ref[~fin & ~np.isnan(ref)]), what
    with np.errstate(invalid="ignore"):
        assert np.all(np.abs(g - ref)[fin] <= np.broadcast_to(bound, ref.shape)[fin]), \
            (what, np.nanmax(np.abs(g - ref)[fin]))
