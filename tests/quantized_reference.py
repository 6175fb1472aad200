"""Plain 64-bit implementations of the 8-bit operations and of token sampling,
and the bounds the kernels' results are held to (derived at each bound)."""
from __future__ import annotations

import math

import numpy as np
import torch

from tests.serving_reference import HALF_STEP, SUBNORMAL, f64

E4M3 = torch.float8_e4m3fn


# -- e4m3 and scales ----------------------------------------------------------------

def round_e4m3(v):
    """The nearest e4m3 number, ties to the even one, at most 448 (NaN stays)."""
    with np.errstate(divide="ignore", invalid="ignore"):
        e = np.maximum(np.floor(np.log2(np.abs(np.where(v == 0, 1.0, v)))), -6.0)
        step = np.exp2(np.where(np.isfinite(e), e, 0.0) - 3)
        return np.clip(np.rint(v / step) * step, -448.0, 448.0)


def scale_of(size):
    """2^e of each size (float64 array of fp32 numbers), by the definition alone."""
    out = np.ones_like(size)
    for i, s in np.ndenumerate(size):
        if not np.isfinite(s):
            out[i] = np.nan
        elif s > 0:
            e = -126
            if 448.0 * 2.0 ** e < s:
                e = math.frexp(s)[1] - 12
                while 448.0 * 2.0 ** e < s:
                    e += 1
            out[i] = 2.0 ** max(e, -126)
    return out


def quantize_blocks(x, block_rows):
    x = f64(x)
    M, K = x.shape
    mb, kb = -(-M // block_rows), -(-K // 128)
    scales, q = np.ones((mb, kb)), np.zeros((M, K))
    for i in range(mb):
        for j in range(kb):
            part = np.s_[i * block_rows:(i + 1) * block_rows, j * 128:(j + 1) * 128]
            size = np.abs(x[part]).max(initial=0.0)
            if np.isnan(x[part]).any():
                size = np.nan
            scales[i, j] = scale_of(np.array([size]))[0]
            with np.errstate(invalid="ignore"):
                q[part] = round_e4m3(x[part] / scales[i, j])
    return q, scales


def from_e4m3(t):
    return t.detach().float().cpu().double().numpy()


# -- the block-scaled product --------------------------------------------------------

def mm(a, sa, b, sb, bias, out_dtype):
    """(result, bound).  Products and scales are exact.  A tensor-core step adds 32 products to
    the running sum, off by at most 2^-22 of the magnitudes summed so far in its segment of
    64 steps (terms aligned to the largest and truncated, and a rounding): min(64, K / 32)
    2^-22 of the whole at most.  Segments and the bias are added in fp32, 2^-24 each."""
    a, b, sa, sb = from_e4m3(a), from_e4m3(b), f64(sa), f64(sb)
    K = a.shape[1]
    a = a * np.repeat(sa, 128, 1)[:, :K]
    b = b * np.repeat(np.repeat(sb, 128, 0)[:K], 128, 1)[:, :b.shape[1]]
    ref, size = a @ b, np.abs(a) @ np.abs(b)
    if bias is not None:
        ref, size = ref + f64(bias), size + np.abs(f64(bias))
    err = (min(64, -(-K // 32)) * 2.0 ** -22 + (-(-K // 2048) + 3) * 2.0 ** -24) * size
    return ref, err + (np.abs(ref) + err) * HALF_STEP[out_dtype] + SUBNORMAL[out_dtype]


# -- attention over caches in 8 bits ----------------------------------------------------

def attention(q, kc, ks, vc, vs, table, lens, scale, out_dtype):
    """(result, bound) of one token per request."""
    B, Hq, D = q.shape
    P, page, Hkv, _ = kc.shape
    G = Hq // Hkv
    table, lens = table.cpu().numpy(), lens.cpu().numpy()
    q64 = f64(q)
    ref, bound = np.zeros((B, Hq, D)), np.zeros((B, Hq, D))
    kb, vb = kc.view(torch.uint8), vc.view(torch.uint8)
    for b in range(B):
        n = max(0, min(int(lens[b]), table.shape[1] * page))
        j = np.arange(n)
        pages = table[b, j // page]
        ok = (pages >= 0) & (pages < P)
        j, pages = j[ok], pages[ok]
        n = len(j)
        if n == 0:
            continue
        at = torch.as_tensor(pages.astype(np.int64), device=kc.device), torch.as_tensor(j % page, device=kc.device)
        k8, v8 = from_e4m3(kb[at].view(E4M3)), from_e4m3(vb[at].view(E4M3))
        k, sv = k8 * f64(ks[at])[..., None], f64(vs[at])
        v = v8 * sv[..., None]
        for h in range(Hq):
            kh, vh, svh = k[:, h // G], v[:, h // G], np.abs(sv[:, h // G])
            s = scale * (kh @ q64[b, h])
            A = abs(scale) * np.max(np.abs(kh) @ np.abs(q64[b, h]))
            p = np.exp(s - s.max())
            p = p / p.sum()
            ref[b, h] = p @ vh
            # A score takes D / 16 <= 16 tensor-core steps, each off by at most 2^-22 of A,
            # q's rounding to fp16 (2^-39 of its largest element, D of them: under 2^-30 of
            # max |q| sum |k|, which is at most D A) and four roundings: under 2^-17 A.  With
            # log2 of the value's scale (L at most) added, t + L has one more, and t - m
            # one: 2^-16 A + 2^-23 L.  2^x is good to 2^-21; a weight goes through one for
            # itself, one for each tile of its warp that raises a maximum, two at its unit's
            # end and in each of four joins: (tiles + 8) 2^-21.  Weights are carried in two
            # fp16 (2^-22); sums over n keys: n 2^-23; the division and the unit's factor: 2^-22.
            tiles = min(n, 512 * 2 ** max(0, math.ceil(math.log2(max(1.0, n / 65536))))) / 64 + 1
            L = np.abs(np.log2(svh[svh > 0])).max(initial=0.0) + 1
            rel = 2.0 ** -22 + 2 * (2.0 ** -16 * A + 2.0 ** -23 * L + (tiles + 8) * 2.0 ** -21) + n * 2.0 ** -23 + 2.0 ** -22
            err = rel * (p @ np.abs(vh))
            # the second fp16 of a weight ends at 2^-39 of the largest p |v_scale| of its warp (times 2)
            err = err + 2.0 ** -38 * (p * svh).max() * np.abs(v8[:, h // G]).sum(0)
            bound[b, h] = err + (np.abs(ref[b, h]) + err) * HALF_STEP[out_dtype] + SUBNORMAL[out_dtype]
    return ref, bound


# -- sampling ---------------------------------------------------------------------------

MARGIN = 2.0 ** -30  # relative distance from a border within which either side may be taken


def sample(x, u, t=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, whether a border is nearer than MARGIN) of one row: float64 logits, settings as the
    kernel gets them (fp32 numbers)."""
    n = len(x)
    if not (0 <= u < 1) or not (0 <= t <= 2.0 ** 20) or math.isnan(top_p) or math.isnan(min_p):
        return -1, False
    if np.isnan(x).any() or (x == np.inf).any() or not (x > -np.inf).any():
        return -1, False
    best = int(np.argmax(x))
    if t < 2.0 ** -20 or top_k == 1 or top_p <= 0:
        return best, False
    near = False
    with np.errstate(over="ignore"):
        w = np.exp((x - x[best]) / t)
    order = np.argsort(-x, kind="stable")
    if 0 < top_k < n:
        order = order[:top_k]
    if top_p < 1:
        mass = np.cumsum(w[order])
        want = top_p * mass[-1]
        exact = all(float(v).is_integer() for v in w[order][w[order] > 0])  # equal logits: sums without rounding
        near |= not exact and np.abs(mass - want).min() < MARGIN * mass[-1]
        order = order[:1 + int(np.searchsorted(mass, want, side="left"))]
    if min_p > 0:
        limit = min(min_p, 1.0)
        near |= bool((np.abs(w[order] - limit) < MARGIN * limit)[w[order] != limit].any())
        order = order[w[order] >= limit]
    order = np.sort(order)
    mass = np.cumsum(w[order])
    want = u * mass[-1]
    exact = all(float(v).is_integer() for v in w[order][w[order] > 0])
    near |= not exact and np.abs(mass - want).min() < MARGIN * mass[-1]
    return int(order[np.searchsorted(mass, want, side="right")]), near
