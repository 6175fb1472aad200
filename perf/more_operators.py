"""Workloads of the 8-bit serving operators and of token sampling: quantisation
in blocks and the block-scaled matrix product, the paged cache in 8 bits (cache
writes, reading back, single-token attention) and sampling from the logits.

Each case is computed in a plain form (elementary torch operations in 32 bits,
64 where sums and borders need it) or, with ``own`` set, by the library's entry
points.
"""
from __future__ import annotations

import math
import random

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
_E4M3 = torch.float8_e4m3fn


# -- cases ----------------------------------------------------------------------

def listed():
    return [
        # the input rows of one decode step's linear layer: pure latency
        dict(name="quantize_decode", op="quantize", rows=16, cols=4096, block_rows=1, dtype="bf16"),
        # a linear layer's weight as a checkpoint holds it, once a load
        dict(name="quantize_weight", op="quantize", rows=14336, cols=4096, block_rows=128, dtype="bf16"),
        # a decode step's linear layer: the weight is read once for a few rows
        dict(name="linear_decode", op="mm", m=16, k=4096, n=14336, out="bf16", bias=False),
        # a prompt's linear layer
        dict(name="linear_prompt", op="mm", m=8192, k=4096, n=14336, out="bf16", bias=True),
        # one decode step: rotate q and k, write k and v in 8 bits, far positions
        dict(name="store_decode", op="store", tokens=64, heads=32, kv_heads=8, dim=128, rotary=128,
             interleaved=False, farthest=131072, page=16, dtype="bf16"),
        # a prefill chunk of odd length
        dict(name="store_prefill", op="store", tokens=8191, heads=32, kv_heads=8, dim=128, rotary=128,
             interleaved=False, farthest=8192, page=64, dtype="bf16"),
        # one request's cached prefix, for a prompt that goes on from it
        dict(name="load_one", op="load", tokens=1021, kv_heads=8, dim=128, page=16, dtype="bf16"),
        # a long shared document
        dict(name="load_long", op="load", tokens=131071, kv_heads=8, dim=128, page=64, dtype="bf16"),
        # one request, a short cache: latency
        dict(name="attend_one", op="attend", batch=1, heads=32, kv_heads=8, dim=128, page=16, longest=1021,
             even=True, dtype="bf16", out="bf16"),
        # a ragged serving batch with an empty row, grouped heads
        dict(name="attend_batch", op="attend", batch=64, heads=32, kv_heads=8, dim=128, page=16, longest=8192,
             even=False, dtype="bf16", out="bf16"),
        # a small decode batch, the usual filters
        dict(name="sample_decode", op="sample", rows=8, vocab=128256, dtype="fp32", top_k=50, top_p=0.9, min_p=0.0),
        # a large decode batch, nucleus and floor without a count, some rows greedy
        dict(name="sample_batch", op="sample", rows=256, vocab=128256, dtype="bf16", top_k=0, top_p=0.95, min_p=0.01),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "mm", "mm", "store", "load", "attend", "attend", "sample", "sample"])
    page = rng.choice([8, 16, 24, 32, 64, 128])
    if op == "quantize":
        dtype = rng.choice(["bf16", "fp16", "fp32"])
        rows = _log_uniform(rng, 1, 16384)
        most = 14336 * 4096 * 2 // _SIZE[dtype] // rows
        return dict(op=op, rows=rows, cols=_log_uniform(rng, 64, min(16384, max(65, most))),
                    block_rows=rng.choice([1, 128]), dtype=dtype)
    if op == "mm":
        m = _log_uniform(rng, 1, 8192)
        k = _log_uniform(rng, 64, 14336)
        most = 8192 * 4096 * 14336 // (m * k)
        return dict(op=op, m=m, k=k, n=_log_uniform(rng, 64, min(16384, most)),
                    out=rng.choice(["bf16", "bf16", "fp16", "fp32"]), bias=rng.random() < 0.5)
    if op == "store":
        dim = rng.choice([64, 128, 256])
        c = dict(op=op, tokens=_log_uniform(rng, 1, 8191), heads=rng.choice([8, 16, 32]) * 128 // dim, dim=dim,
                 rotary=rng.choice([dim, dim // 2]), interleaved=rng.random() < 0.5,
                 farthest=_log_uniform(rng, 8192, 131072), page=page, dtype=rng.choice(["bf16", "fp16"]))
        c["kv_heads"] = max(1, c["heads"] // rng.choice([2, 4, 8]))
        return c
    if op == "load":
        dim, kv = rng.choice([64, 128, 256]), rng.choice([1, 2, 8])
        most = 131071 * 1024 // (kv * dim)
        return dict(op=op, tokens=_log_uniform(rng, 1, min(131071, most)), kv_heads=kv, dim=dim, page=page,
                    dtype=rng.choice(["bf16", "fp16"]))
    if op == "attend":
        dim = rng.choice([64, 128, 256])
        group = rng.choice([1, 2, 4, 5, 8, 16])
        kv = rng.choice([1, 2, 8])
        batch = _log_uniform(rng, 1, 64)
        room = 64 * 4096 * 8 * 128 // (dim * kv * batch)  # keys a request, within the largest listed case
        longest = _log_uniform(rng, 1, min(131071, max(16, room)))
        dtype = rng.choice(["bf16", "fp16"])
        return dict(op=op, batch=batch, heads=kv * group, kv_heads=kv, dim=dim, page=page, longest=longest,
                    even=rng.random() < 0.3, dtype=dtype, out=rng.choice([dtype, "fp32"]))
    rows = _log_uniform(rng, 1, 256)
    dtype = rng.choice(["bf16", "fp16", "fp32"])
    most = 256 * 128256 * 2 // (rows * _SIZE[dtype])
    return dict(op=op, rows=rows, vocab=_log_uniform(rng, 1000, min(160000, most)), dtype=dtype,
                top_k=rng.choice([0, 0, 1, 20, 50, 1000]), top_p=rng.choice([1.0, 1.0, 0.5, 0.9, 0.95]),
                min_p=rng.choice([0.0, 0.0, 0.01, 0.1]))


# -- inputs -----------------------------------------------------------------------

def _lengths(c):
    """The requests' lengths, a function of the case alone."""
    if c["even"]:
        return [c["longest"]] * c["batch"]
    rng = random.Random(c["batch"] * 7919 + c["longest"])
    lens = [rng.randint(1, c["longest"]) for _ in range(c["batch"])]
    lens[0] = c["longest"]
    if c["batch"] > 1:
        lens[-1] = 0  # a padded row of a captured batch
    return lens


def _frequencies(c):
    """Angular frequencies of the rotary pairs as python floats."""
    return [10000.0 ** (-2.0 * i / c["rotary"]) for i in range(c["rotary"] // 2)]


def _scale_of(amax):
    """2^e with the least e that amax <= 448 * 2^e holds for, e >= -126; 1 for a block of zeros."""
    m, x = torch.frexp(amax)
    e = torch.where(m <= 0.875, x - 9, x - 8).clamp(min=-126)
    return torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), e), torch.ones_like(amax))


def _to_e4m3(x, scale):
    return (x * (1.0 / scale)).clamp(-448.0, 448.0).to(_E4M3)


def _blocks(rows, block_rows, cols):
    return -(-rows // block_rows), -(-cols // 128)


def _plain_quantize(x, block_rows):
    """([M, K] in 8 bits, [ceil(M / block_rows), ceil(K / 128)] scales)."""
    M, K = x.shape
    mb, kb = _blocks(M, block_rows, K)
    x = torch.nn.functional.pad(x.float(), (0, kb * 128 - K, 0, mb * block_rows - M))
    x = x.view(mb, block_rows, kb, 128)
    scale = _scale_of(x.abs().amax((1, 3)))
    q = _to_e4m3(x, scale[:, None, :, None]).view(mb * block_rows, kb * 128)
    return q[:M, :K], scale


def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    s = {"case": c}

    def normal(shape, dtype, std=1.0):
        return (torch.randn(shape, generator=g, device=dev, dtype=torch.float32) * std).to(_DT[dtype])

    def uniform(shape):
        return torch.rand(shape, generator=g, device=dev, dtype=torch.float32)

    def permutation(n):
        return torch.randperm(n, generator=g, device=dev)

    def padded(x8):  # rows on 16 bytes, as the quantiser lays them out
        store = torch.zeros((x8.shape[0], -(-x8.shape[1] // 16) * 16), dtype=torch.uint8, device=dev)
        store[:, :x8.shape[1]] = x8.view(torch.uint8)
        return store.view(_E4M3)[:, :x8.shape[1]]

    if c["op"] == "quantize":
        # rows of unequal size, as activations and weights are
        s["x"] = (normal((c["rows"], c["cols"]), "fp32") * torch.exp2(4 * uniform((c["rows"], 1)) - 2)).to(_DT[c["dtype"]])
    elif c["op"] == "mm":
        a, sa = _plain_quantize(normal((c["m"], c["k"]), "bf16"), 1)
        b, sb = _plain_quantize(normal((c["n"], c["k"]), "bf16", 0.02), 128)
        s["a"], s["sa"], s["b"], s["sb"] = padded(a), sa, padded(b).t(), sb.t()
        s["bias"] = normal((c["n"],), "bf16", 0.01) if c["bias"] else None
    elif c["op"] == "store":
        T, hq, hkv, d, ps = c["tokens"], c["heads"], c["kv_heads"], c["dim"], c["page"]
        qkv = normal((T, hq + 2 * hkv, d), c["dtype"])  # one projection's output, q, k and v beside one another
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        s["pos"] = torch.randint(0, c["farthest"], (T,), generator=g, device=dev, dtype=torch.int32)
        pages = 2 * (-(-T // ps)) + 1
        s["slots"] = permutation(pages * ps)[:T].contiguous()
        if T > 2:
            s["slots"][T // 2] = -1  # a padded token
        s["kc"] = normal((pages, ps, hkv, d), "fp32").to(_E4M3)
        s["vc"] = normal((pages, ps, hkv, d), "fp32").to(_E4M3)
        s["ks"] = torch.exp2(torch.floor(4 * uniform((pages, ps, hkv))))
        s["vs"] = torch.exp2(torch.floor(4 * uniform((pages, ps, hkv))))
        if own:
            from invariant_gemm_bi_gb300 import binding
            s["config"] = binding.bi_rope_config(c["rotary"], base=10000.0, interleaved=c["interleaved"])
        else:
            s["freq"] = torch.tensor(_frequencies(c), dtype=torch.float64, device=dev)
    elif c["op"] in ("load", "attend"):
        ps = c["page"]
        lens = _lengths(c) if c["op"] == "attend" else [c["tokens"]]
        need = [-(-x // ps) for x in lens]
        pages = sum(need) + 3
        ids = permutation(pages).to(torch.int32).cpu()
        table = torch.zeros((len(lens), max(1, max(need))), dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = ids[at:at + n]
            at += n
        s["table"] = table.to(dev)
        shape = (pages, ps, c["kv_heads"], c["dim"])

        def cache():
            x = normal(shape, "fp32") * torch.exp2(2 * uniform(shape[:3]) - 1)[..., None]
            scale = _scale_of(x.abs().amax(-1))
            return _to_e4m3(x, scale[..., None]), scale
        s["kc"], s["ks"] = cache()
        s["vc"], s["vs"] = cache()
        if c["op"] == "load":
            j = torch.arange(c["tokens"], device=dev)
            s["slots"] = s["table"][0, j // ps].long() * ps + j % ps
        else:
            s["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
            s["q"] = normal((c["batch"], c["heads"], c["dim"]), c["dtype"])
            if own:
                from invariant_gemm_bi_gb300 import binding
                n = binding.bi_paged_attention_workspace_bytes(c["batch"], c["heads"], c["dim"], s["table"].shape[1] * ps)
                s["ws"] = torch.empty(max(n, 16), dtype=torch.uint8, device=dev)
    else:
        R = c["rows"]
        s["x"] = normal((R, c["vocab"]), c["dtype"], 3.0)
        s["u"] = uniform((R,))
        # requests of one batch have settings of their own
        s["temperature"] = torch.where(uniform((R,)) < 0.1, 0.0, 0.5 + uniform((R,)))
        s["top_k"] = torch.where(uniform((R,)) < 0.8, c["top_k"], 0).to(torch.int32)
        s["top_p"] = torch.where(uniform((R,)) < 0.8, c["top_p"], 1.0).float()
        s["min_p"] = torch.where(uniform((R,)) < 0.8, c["min_p"], 0.0).float()
    return s


# -- plain forms ------------------------------------------------------------------

def _plain_mm(s):
    c = s["case"]
    M, K, N = c["m"], c["k"], c["n"]
    a = s["a"].float() * s["sa"].repeat_interleave(128, 1)[:, :K]
    b = s["b"].float() * s["sb"].repeat_interleave(128, 0)[:K].repeat_interleave(128, 1)[:, :N]
    y = torch.matmul(a, b)
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return y.to(_DT[c["out"]])


def _plain_rope(x, pos, freq, interleaved):
    half = freq.shape[0]
    angle = pos.to(torch.float64)[:, None] * freq[None, :]
    cos, sin = torch.cos(angle).float()[:, None, :], torch.sin(angle).float()[:, None, :]
    x = x.float()
    y = x.clone()
    a, b = (x[..., 0:2 * half:2], x[..., 1:2 * half:2]) if interleaved else (x[..., :half], x[..., half:2 * half])
    ya, yb = a * cos - b * sin, a * sin + b * cos
    if interleaved:
        y[..., 0:2 * half:2], y[..., 1:2 * half:2] = ya, yb
    else:
        y[..., :half], y[..., half:2 * half] = ya, yb
    return y, (a.abs() + b.abs()).amax(-1)  # what no angle takes an element of a pair past


def _plain_store(s):
    c = s["case"]
    n = c["rotary"]
    q, _ = _plain_rope(s["q"], s["pos"], s["freq"], c["interleaved"])
    k, size = _plain_rope(s["k"], s["pos"], s["freq"], c["interleaved"])
    if n < c["dim"]:
        size = torch.maximum(size, s["k"][..., n:].float().abs().amax(-1))
    v = s["v"].float()
    ks, vs = _scale_of(size), _scale_of(v.abs().amax(-1))
    kept = s["slots"] >= 0
    slots = s["slots"][kept]
    hkv, d = c["kv_heads"], c["dim"]
    s["kc"].view(torch.uint8).view(-1, hkv, d)[slots] = _to_e4m3(k, ks[..., None]).view(torch.uint8)[kept]
    s["vc"].view(torch.uint8).view(-1, hkv, d)[slots] = _to_e4m3(v, vs[..., None]).view(torch.uint8)[kept]
    s["ks"].view(-1, hkv)[slots] = ks[kept]
    s["vs"].view(-1, hkv)[slots] = vs[kept]
    return q.to(_DT[c["dtype"]]), s["kc"], s["ks"], s["vc"], s["vs"]


def _rows_of(cache, scales, page, row):
    """Dequantised rows at the places (page, row)."""
    return cache.view(torch.uint8)[page, row].view(_E4M3).float() * scales[page, row][..., None]


def _plain_attend(s):
    c = s["case"]
    hkv, d, ps, B = c["kv_heads"], c["dim"], c["page"], c["batch"]
    j = torch.arange(s["table"].shape[1] * ps, device=s["q"].device)
    page, row = s["table"].long()[:, j // ps], (j % ps).expand(B, -1)
    k = _rows_of(s["kc"], s["ks"], page, row).permute(0, 2, 3, 1)
    v = _rows_of(s["vc"], s["vs"], page, row).permute(0, 2, 1, 3)
    q = s["q"].float().view(B, hkv, -1, d)
    t = torch.matmul(q, k) * d ** -0.5
    t = t.masked_fill(j[None, None, None, :] >= s["lens"][:, None, None, None], float("-inf"))
    e = torch.exp(t - t.amax(-1, keepdim=True).clamp(min=-3e38))
    out = torch.matmul(e, v) / e.sum(-1, keepdim=True)
    out = torch.where(s["lens"][:, None, None, None] > 0, out, torch.zeros_like(out))
    return out.reshape(B, c["heads"], d).to(_DT[c["out"]])


def _plain_sample(s):
    """In 64 bits: a boundary of the distribution is as near to the given number as chance will have it."""
    x = s["x"].double()
    n = x.shape[1]
    greedy = s["temperature"][:, None] <= 0
    t = torch.where(greedy, torch.ones_like(s["temperature"][:, None]), s["temperature"][:, None]).double()
    sx, order = torch.sort(x, dim=-1, descending=True, stable=True)
    e = torch.exp((sx - sx[:, :1]) / t)
    rank = torch.arange(n, device=x.device)[None, :]
    k = torch.where(s["top_k"] <= 0, n, s["top_k"].long())[:, None]
    top_p, min_p = s["top_p"].double()[:, None], s["min_p"].double()[:, None]
    e = torch.where(rank < k, e, torch.zeros_like(e))
    cum = torch.cumsum(e, -1)
    before = torch.nn.functional.pad(cum[:, :-1], (1, 0))
    keep = ((top_p >= 1) | (before < top_p * cum[:, -1:])) & (e >= min_p)
    keep[:, 0] = True
    w = torch.zeros_like(x).scatter_(1, order, torch.where(keep, e, torch.zeros_like(e)))
    cw = torch.cumsum(w, -1)
    token = (cw <= s["u"].double()[:, None] * cw[:, -1:]).sum(-1)
    return torch.where(greedy[:, 0], order[:, 0], token)


def run(state):
    s = state
    c = s["case"]
    op = c["op"]
    if own:
        return _run_own(s)
    if op == "quantize":
        return _plain_quantize(s["x"], c["block_rows"])
    if op == "mm":
        return _plain_mm(s)
    if op == "store":
        return _plain_store(s)
    if op == "load":
        page, row = s["slots"] // c["page"], s["slots"] % c["page"]
        return (_rows_of(s["kc"], s["ks"], page, row).to(_DT[c["dtype"]]),
                _rows_of(s["vc"], s["vs"], page, row).to(_DT[c["dtype"]]))
    if op == "attend":
        return _plain_attend(s)
    return _plain_sample(s)


def _run_own(s):
    from invariant_gemm_bi_gb300 import binding as bi
    c = s["case"]
    op = c["op"]
    if op == "quantize":
        return tuple(bi.bi_quantize_blocks(s["x"], c["block_rows"]))
    if op == "mm":
        return bi.bi_mm_blockscaled(s["a"], s["sa"], s["b"], s["sb"], bias=s["bias"], out_dtype=_DT[c["out"]])
    if op == "store":
        q = bi.bi_paged_store_quantized(s["k"], s["v"], s["slots"], s["kc"], s["ks"], s["vc"], s["vs"], q=s["q"],
                                        positions=s["pos"], config=s["config"])
        return q, s["kc"], s["ks"], s["vc"], s["vs"]
    if op == "load":
        return tuple(bi.bi_paged_load_quantized(s["slots"], s["kc"], s["ks"], s["vc"], s["vs"],
                                                out_dtype=_DT[c["dtype"]]))
    if op == "attend":
        return bi.bi_paged_attention_quantized(s["q"], s["kc"], s["ks"], s["vc"], s["vs"], s["table"], s["lens"],
                                               c["dim"] ** -0.5, out_dtype=_DT[c["out"]], workspace=s["ws"])
    return bi.bi_sample_tokens(s["x"], s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                               min_p=s["min_p"])


# -- cost -----------------------------------------------------------------------------

def work(case):
    c = case
    if c["op"] == "quantize":
        mb, kb = _blocks(c["rows"], c["block_rows"], c["cols"])
        n = c["rows"] * c["cols"]
        return {"bytes": n * (_SIZE[c["dtype"]] + 1) + 4 * mb * kb, "flops": 2 * n}
    if c["op"] == "mm":
        m, k, n = c["m"], c["k"], c["n"]
        kb = -(-k // 128)
        return {"bytes": (m + n) * k + 4 * kb * (m + -(-n // 128)) + m * n * _SIZE[c["out"]] + 2 * n * c["bias"],
                "flops": 2 * m * n * k}
    if c["op"] == "store":
        e, kv = _SIZE[c["dtype"]], 2 * c["tokens"] * c["kv_heads"]
        return {"bytes": 2 * c["tokens"] * c["heads"] * c["dim"] * e + kv * (c["dim"] * (e + 1) + 4) + 12 * c["tokens"],
                "flops": 3 * c["tokens"] * (c["heads"] + c["kv_heads"]) * c["rotary"] + 2 * kv * c["dim"]}
    if c["op"] == "load":
        n = 2 * c["tokens"] * c["kv_heads"]
        return {"bytes": n * (c["dim"] * (1 + _SIZE[c["dtype"]]) + 4) + 8 * c["tokens"], "flops": n * c["dim"]}
    if c["op"] == "attend":
        lens = _lengths(c)
        rows = c["batch"] * c["heads"] * c["dim"]
        return {"bytes": 2 * sum(lens) * c["kv_heads"] * (c["dim"] + 4)
                + rows * (_SIZE[c["dtype"]] + _SIZE[c["out"]])
                + 4 * sum(-(-n // c["page"]) for n in lens) + 4 * c["batch"],
                "flops": 4 * sum(lens) * c["heads"] * c["dim"]}
    return {"bytes": c["rows"] * (c["vocab"] * _SIZE[c["dtype"]] + 28), "flops": 4 * c["rows"] * c["vocab"]}


# -- 64-bit values ---------------------------------------------------------------------

def _grid(v):
    """The nearest numbers of 4 exponent and 3 mantissa bits (ties to the even one), at most 448."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(v / step) * step).clamp(-448, 448)


def _least_power(amax):
    """The least power of two that 448 times reaches amax: 2^ceil(log2(amax / 448)), put right at its borders."""
    p = torch.exp2(torch.ceil(torch.log2(amax.clamp(min=1e-300) / 448)))
    p = torch.where(448 * p < amax, 2 * p, p)
    p = torch.where(448 * p / 2 >= amax, p / 2, p)
    return torch.where(amax > 0, p.clamp(min=2.0 ** -126), torch.ones_like(p))


def exact(case, seed):
    c = case
    s = prepare(c, seed)
    if c["op"] == "quantize":
        x, br = s["x"].double(), c["block_rows"]
        q, sc = torch.zeros_like(x), torch.zeros(_blocks(c["rows"], br, c["cols"]), dtype=torch.float64, device=x.device)
        for j in range(sc.shape[1]):
            part = x[:, 128 * j:128 * j + 128]
            size = part.abs().amax(1)
            if br > 1:
                size = torch.stack([y.amax() for y in size.split(br)])
            p = _least_power(size)
            sc[:, j] = p
            q[:, 128 * j:128 * j + 128] = _grid(part / p.repeat_interleave(br)[:c["rows"], None])
        return q, sc
    if c["op"] == "mm":
        y = torch.zeros((c["m"], c["n"]), dtype=torch.float64, device=s["a"].device)
        for j in range(s["sa"].shape[1]):
            part = slice(128 * j, min(128 * j + 128, c["k"]))
            b = s["b"][part].double() * s["sb"][j].double().repeat_interleave(128)[:c["n"]]
            y += s["sa"][:, j:j + 1].double() * (s["a"][:, part].double() @ b)
        return y if s["bias"] is None else y + s["bias"].double()
    if c["op"] == "store":
        f = np.array(_frequencies(c))
        turn = np.exp(1j * (s["pos"].cpu().numpy().astype(np.float64)[:, None, None] * f))
        first = np.arange(f.size) * 2 if c["interleaved"] else np.arange(f.size)
        second = first + (1 if c["interleaved"] else f.size)

        def rotated(x):
            y = x.copy()
            z = (x[..., first] + 1j * x[..., second]) * turn
            y[..., first], y[..., second] = z.real, z.imag
            return torch.from_numpy(y)
        q, k, v = (s[n].double().cpu().numpy() for n in ("q", "k", "v"))
        bound = (np.abs(k[..., first]) + np.abs(k[..., second])).max(-1)
        if c["rotary"] < c["dim"]:
            bound = np.maximum(bound, np.abs(k[..., c["rotary"]:]).max(-1))
        out = []
        live = [(t, x // c["page"], x % c["page"]) for t, x in enumerate(s["slots"].tolist()) if x >= 0]
        t, page, row = (torch.tensor(i) for i in zip(*live))
        for rows, size, cache, scales in ((rotated(k), bound, "kc", "ks"), (torch.from_numpy(v), np.abs(v).max(-1), "vc", "vs")):
            # sums of two numbers of 16 bits can have more than fit 32: the scale goes by the rounded one
            p = _least_power(torch.from_numpy(size.astype(np.float32).astype(np.float64)))
            y, sc = s[cache].double().cpu(), s[scales].double().cpu()
            y[page, row], sc[page, row] = _grid(rows / p[..., None])[t], p[t]
            out += [y, sc]
        return rotated(q), *out
    if c["op"] == "load":
        out = []
        for cache, scales in (("kc", "ks"), ("vc", "vs")):
            flat = s[cache].view(torch.uint8).flatten(0, 1)[s["slots"]]
            out.append(flat.view(_E4M3).double() * s[scales].flatten(0, 1)[s["slots"]][..., None].double())
        return tuple(out)
    if c["op"] == "attend":
        ps, group = c["page"], c["heads"] // c["kv_heads"]
        out = torch.zeros((c["batch"], c["heads"], c["dim"]), dtype=torch.float64)
        for b, n in enumerate(_lengths(c)):
            j = torch.arange(n, device=s["q"].device)
            slot = s["table"][b, j // ps].long() * ps + j % ps
            for h in range(c["kv_heads"] if n else 0):
                k, v = (s[x].view(torch.uint8).flatten(0, 1)[slot, h].view(_E4M3).double()
                        * s[y].flatten(0, 1)[slot, h].double()[:, None] for x, y in (("kc", "ks"), ("vc", "vs")))
                q = s["q"][b, h * group:(h + 1) * group].double()
                p = torch.softmax(q @ k.T / math.sqrt(c["dim"]), -1)
                out[b, h * group:(h + 1) * group] = (p @ v).cpu()
        return out
    tokens = np.zeros(c["rows"], dtype=np.int64)
    for r in range(c["rows"]):
        x = s["x"][r].double().cpu().numpy()
        t, k, tp, mp, u = (float(s[n][r]) for n in ("temperature", "top_k", "top_p", "min_p", "u"))
        best = int(x.argmax())
        if t <= 0:
            tokens[r] = best
            continue
        w = np.exp((x - x[best]) / t)
        order = np.argsort(-x, kind="stable")[:int(k) if k > 0 else None]
        mass = np.cumsum(w[order])
        if tp < 1:
            order = order[:1 + int(np.searchsorted(mass, tp * mass[-1], side="left"))]
        order = np.sort(order[w[order] >= mp])
        mass = np.cumsum(w[order])
        tokens[r] = order[np.searchsorted(mass, u * mass[-1], side="right")]
    return tokens
