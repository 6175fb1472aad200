"""Workloads of the paged-cache serving operators: page planning, rotary
positions, cache writes, single-token attention over the paged cache and token
log probabilities.

Each case is computed in a plain form (elementary torch operations in 32 bits,
64 where angles need it) or, with ``own`` set, by the library's entry points.
"""
from __future__ import annotations

import math
import random

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}


# -- cases ----------------------------------------------------------------------

def listed():
    return [
        # one decode step's page bookkeeping of a small batch: pure latency
        dict(name="plan_decode", op="plan", batch=8, longest=8192, new=1, page=16, pad=0),
        # a chunked prefill of a large batch, ragged, in a token buffer padded at its end
        dict(name="plan_prefill", op="plan", batch=256, longest=32768, new=1024, page=16, pad=1000),
        # queries of one short action chunk, wide heads, fp32 projections
        dict(name="rope_small", op="rope", tokens=7, heads=8, dim=256, rotary=256, interleaved=False,
             scaling="none", farthest=816, dtype="fp32", out="bf16", backward=False),
        # a training micro-batch's query gradient, interleaved pairs, half of each head
        dict(name="rope_gradient", op="rope", tokens=16383, heads=32, dim=128, rotary=64, interleaved=True,
             scaling="linear", farthest=32768, dtype="bf16", out="bf16", backward=True),
        # one decode step: rotate q and k, write k and v, far positions, scaled frequencies
        dict(name="store_decode", op="store", tokens=64, heads=32, kv_heads=8, dim=128, rotary=128,
             interleaved=False, scaling="ramp", farthest=131072, page=16, dtype="bf16"),
        # a prefill chunk of odd length
        dict(name="store_prefill", op="store", tokens=8191, heads=32, kv_heads=8, dim=128, rotary=128,
             interleaved=False, scaling="none", farthest=8192, page=64, dtype="bf16"),
        # one request, a short cache: latency
        dict(name="attend_one", op="attend", batch=1, heads=32, kv_heads=8, dim=128, page=16, longest=1021,
             even=True, dtype="bf16", out="bf16"),
        # a ragged serving batch with an empty row, grouped heads
        dict(name="attend_batch", op="attend", batch=64, heads=32, kv_heads=8, dim=128, page=16, longest=8192,
             even=False, dtype="bf16", out="bf16"),
        # few requests with a very long cache, one key-value head of 256
        dict(name="attend_long", op="attend", batch=4, heads=8, kv_heads=1, dim=256, page=64, longest=131071,
             even=True, dtype="fp16", out="fp16"),
        # as many key-value heads as query heads, narrow heads, fp32 result
        dict(name="attend_ungrouped", op="attend", batch=32, heads=16, kv_heads=16, dim=64, page=32, longest=4096,
             even=True, dtype="bf16", out="fp32"),
        # one decode step's sampled tokens over a large vocabulary
        dict(name="logprobs_decode", op="logprobs", rows=8, vocab=128256, top=20, dtype="fp32", masked=False),
        # log probabilities of a prompt, bf16 logits, some tokens forbidden
        dict(name="logprobs_prompt", op="logprobs", rows=2048, vocab=128256, top=5, dtype="bf16", masked=True),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "rope", "store", "attend", "attend", "logprobs"])
    page = rng.choice([8, 16, 24, 32, 64, 128])
    if op == "plan":
        return dict(op=op, batch=_log_uniform(rng, 1, 256), longest=_log_uniform(rng, 1, 32768),
                    new=_log_uniform(rng, 1, 1024), page=page, pad=rng.randint(0, 1000))
    if op in ("rope", "store"):
        dim = rng.choice([64, 128, 256])
        rotary = rng.choice([dim, dim // 2])
        c = dict(op=op, tokens=_log_uniform(rng, 1, 8191 if op == "store" else 16383),
                 heads=rng.choice([8, 16, 32]) * 128 // dim, dim=dim, rotary=rotary,
                 interleaved=rng.random() < 0.5, scaling=rng.choice(["none", "linear", "ramp"]),
                 farthest=_log_uniform(rng, 8192, 131072))
        if op == "rope":
            c["dtype"] = c["out"] = rng.choice(["bf16", "fp16"])
            if rng.random() < 0.2 and c["tokens"] <= 4096:
                c["dtype"] = "fp32"
            c["backward"] = rng.random() < 0.5
        else:
            c["kv_heads"] = max(1, c["heads"] // rng.choice([1, 2, 4]))
            c["tokens"] = max(1, c["tokens"] // (2 if c["kv_heads"] == c["heads"] else 1))
            c["page"] = page
            c["dtype"] = rng.choice(["bf16", "fp16"])
        return c
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
    rows = _log_uniform(rng, 1, 2048)
    dtype = rng.choice(["bf16", "fp16", "fp32"])
    most = 2048 * 128256 * 2 // (rows * _SIZE[dtype])
    vocab = _log_uniform(rng, 1000, min(160000, max(1001, most)))
    return dict(op=op, rows=rows, vocab=vocab, top=rng.choice([0, 1, 5, 20, 64]), dtype=dtype,
                masked=rng.random() < 0.5)


# -- inputs -----------------------------------------------------------------------

def _lengths(c):
    """The requests' lengths, a function of the case alone."""
    rng = random.Random(c["batch"] * 7919 + c["longest"])
    if c["op"] == "plan":
        ctx = [rng.randint(0, c["longest"]) for _ in range(c["batch"])]
        new = [1 if c["new"] == 1 else rng.randint(0, c["new"]) for _ in range(c["batch"])]
        return ctx, new
    if c["even"]:
        return [c["longest"]] * c["batch"]
    lens = [rng.randint(1, c["longest"]) for _ in range(c["batch"])]
    lens[0] = c["longest"]
    if c["batch"] > 1:
        lens[-1] = 0  # a padded row of a captured batch
    return lens


def _frequencies(c):
    """Angular frequencies of the rotary pairs as python floats."""
    n, base, far = c["rotary"], 10000.0, float(c["farthest"])
    f = [base ** (-2.0 * i / n) for i in range(n // 2)]
    if c["scaling"] == "linear":
        return [x / 4.0 for x in f]
    if c["scaling"] == "ramp":  # slow pairs interpolated, fast ones kept, by turns over the original length
        out = []
        for x in f:
            turns = far / 8.0 * x / (2 * math.pi)
            g = min(1.0, max(0.0, (turns - 1.0) / (4.0 - 1.0)))
            out.append(x * (g + (1 - g) / 8.0))
        return out
    return f


def _rope_config(c):
    from invariant_gemm_bi_gb300 import binding
    scaling = None
    if c["scaling"] == "linear":
        scaling = binding.RopeScaling("linear", factor=4.0)
    elif c["scaling"] == "ramp":
        scaling = binding.RopeScaling("ramp_turns", factor=8.0, original_length=c["farthest"] / 8.0, low=1.0, high=4.0)
    return binding.bi_rope_config(c["rotary"], base=10000.0, interleaved=c["interleaved"], scaling=scaling)


def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    s = {"case": c}

    def normal(shape, dtype, std=1.0):
        return (torch.randn(shape, generator=g, device=dev, dtype=torch.float32) * std).to(_DT[dtype])

    def permutation(n):
        return torch.randperm(n, generator=g, device=dev)

    if c["op"] == "plan":
        ctx, new = _lengths(c)
        ps = c["page"]
        held = [-(-x // ps) for x in ctx]
        need = [-(-(x + n) // ps) for x, n in zip(ctx, new)]
        width = max(1, max(need))
        total, take = sum(held), sum(need) - sum(held)
        ids = permutation(total + take + 64).to(torch.int32)
        table = torch.full((c["batch"], width), -1, dtype=torch.int32)
        ids_host, at = ids.cpu(), 0
        for b, h in enumerate(held):
            table[b, :h] = ids_host[at:at + h]
            at += h
        s["table"] = table.to(dev)
        s["free"] = ids[total:].contiguous()
        s["ctx"] = torch.tensor(ctx, dtype=torch.int32, device=dev)
        s["new"] = torch.tensor(new, dtype=torch.int32, device=dev)
        s["tokens"] = sum(new) + c["pad"]
        if own:
            from invariant_gemm_bi_gb300 import binding
            s["plan"] = binding.bi_paged_plan_buffers(c["batch"], s["tokens"], dev)
    elif c["op"] == "rope":
        s["x"] = normal((c["tokens"], c["heads"], c["dim"]), c["dtype"])
        s["pos"] = torch.randint(0, c["farthest"], (c["tokens"],), generator=g, device=dev, dtype=torch.int32)
    elif c["op"] == "store":
        T, hq, hkv, d, ps = c["tokens"], c["heads"], c["kv_heads"], c["dim"], c["page"]
        qkv = normal((T, hq + 2 * hkv, d), c["dtype"])  # one projection's output, q, k and v beside one another
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        s["pos"] = torch.randint(0, c["farthest"], (T,), generator=g, device=dev, dtype=torch.int32)
        pages = 2 * (-(-T // ps)) + 1
        s["slots"] = permutation(pages * ps)[:T].contiguous()
        if T > 2:
            s["slots"][T // 2] = -1  # a padded token
        s["kc"] = normal((pages, ps, hkv, d), c["dtype"])
        s["vc"] = normal((pages, ps, hkv, d), c["dtype"])
    elif c["op"] == "attend":
        lens, ps = _lengths(c), c["page"]
        need = [-(-x // ps) for x in lens]
        pages = sum(need) + 3
        ids = permutation(pages).to(torch.int32).cpu()
        table = torch.zeros((c["batch"], max(1, max(need))), dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = ids[at:at + n]
            at += n
        s["table"] = table.to(dev)
        s["lens_host"] = lens
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
        s["q"] = normal((c["batch"], c["heads"], c["dim"]), c["dtype"])
        s["kc"] = normal((pages, ps, c["kv_heads"], c["dim"]), c["dtype"])
        s["vc"] = normal((pages, ps, c["kv_heads"], c["dim"]), c["dtype"])
        if own:
            from invariant_gemm_bi_gb300 import binding
            n = binding.bi_paged_attention_workspace_bytes(c["batch"], c["heads"], c["dim"], s["table"].shape[1] * ps)
            s["ws"] = torch.empty(max(n, 16), dtype=torch.uint8, device=dev)
    else:
        x = normal((c["rows"], c["vocab"]), c["dtype"], 3.0)
        if c["masked"]:
            ban = torch.rand((c["vocab"],), generator=g, device=dev) < 0.1
            ban[:80] = False
            x.masked_fill_(ban, float("-inf"))
        s["x"] = x
        s["tokens"] = torch.randint(0, c["vocab"], (c["rows"],), generator=g, device=dev, dtype=torch.int64)
    if c["op"] in ("rope", "store"):
        if own:
            s["config"] = _rope_config(c)
        else:
            s["freq"] = torch.tensor(_frequencies(c), dtype=torch.float64, device=dev)
    return s


# -- plain forms ------------------------------------------------------------------

def _plain_rope(x, pos, freq, interleaved, backward):
    half = freq.shape[0]
    angle = pos.to(torch.float64)[:, None] * freq[None, :]
    cos, sin = torch.cos(angle).float()[:, None, :], torch.sin(angle).float()[:, None, :]
    if backward:
        sin = -sin
    x = x.float()
    y = x.clone()
    a, b = (x[..., 0:2 * half:2], x[..., 1:2 * half:2]) if interleaved else (x[..., :half], x[..., half:2 * half])
    ya, yb = a * cos - b * sin, a * sin + b * cos
    if interleaved:
        y[..., 0:2 * half:2], y[..., 1:2 * half:2] = ya, yb
    else:
        y[..., :half], y[..., half:2 * half] = ya, yb
    return y


def _plain_plan(s):
    c = s["case"]
    ps, T = c["page"], s["tokens"]
    ctx, new, table, free = s["ctx"].long(), s["new"].long(), s["table"], s["free"]
    held = (ctx + ps - 1) // ps
    take = (ctx + new + ps - 1) // ps - held
    end, pend = torch.cumsum(new, 0), torch.cumsum(take, 0)
    start = pend - take
    col = torch.arange(table.shape[1], device=table.device)[None, :]
    fresh = (col >= held[:, None]) & (col < (held + take)[:, None])
    pick = (start[:, None] + col - held[:, None]).clamp(0, free.shape[0] - 1)
    table.copy_(torch.where(fresh, free[pick], table))
    t = torch.arange(T, device=table.device)
    live = t < end[-1]
    b = (t[:, None] >= end[None, :]).sum(1).clamp(max=c["batch"] - 1) if c["batch"] * T <= 1 << 26 else \
        torch.searchsorted(end, t, right=True).clamp(max=c["batch"] - 1)
    pos = ctx[b] + t - (end - new)[b]
    page = table[b, (pos // ps).clamp(0, table.shape[1] - 1)].long()
    slots = torch.where(live, page * ps + pos % ps, -1)
    pos = torch.where(live, pos, 0).int()
    offsets = torch.cat([end.new_zeros(1), end]).int()
    return table, (ctx + new).int(), offsets, pos, slots, torch.stack([pend[-1], end[-1]]).int()


def _plain_attend(s):
    c = s["case"]
    hkv, d, ps = c["kv_heads"], c["dim"], c["page"]
    group = c["heads"] // hkv
    out = torch.zeros((c["batch"], c["heads"], d), dtype=torch.float32, device=s["q"].device)
    for b, n in enumerate(s["lens_host"]):
        if n == 0:
            continue
        pages = s["table"][b, :-(-n // ps)].long()
        k = s["kc"][pages].reshape(-1, hkv, d)[:n].float().permute(1, 2, 0)
        v = s["vc"][pages].reshape(-1, hkv, d)[:n].float().permute(1, 0, 2)
        q = s["q"][b].float().reshape(hkv, group, d)
        t = torch.matmul(q, k) * d ** -0.5
        e = torch.exp(t - t.amax(-1, keepdim=True))
        out[b] = (torch.matmul(e, v) / e.sum(-1, keepdim=True)).reshape(c["heads"], d)
    return out.to(_DT[c["out"]])


def _plain_logprobs(s):
    c = s["case"]
    x = s["x"].float()
    mx = x.amax(-1, keepdim=True)
    z = x - mx
    e = torch.exp(z)
    total = e.sum(-1, keepdim=True)
    lse = torch.log(total)
    lp = torch.gather(z, 1, s["tokens"][:, None]) - lse
    entropy = lse[:, 0] - torch.where(e > 0, e * z, torch.zeros_like(e)).sum(-1) / total[:, 0]
    if c["top"] == 0:
        return lp[:, 0], entropy
    values, ids = torch.sort(x, dim=-1, descending=True, stable=True)
    return lp[:, 0], entropy, values[:, :c["top"]] - mx - lse, ids[:, :c["top"]].int()


def run(state):
    s = state
    c = s["case"]
    op = c["op"]
    if own:
        return _run_own(s)
    if op == "plan":
        return _plain_plan(s)
    if op == "rope":
        return _plain_rope(s["x"], s["pos"], s["freq"], c["interleaved"], c["backward"]).to(_DT[c["out"]])
    if op == "store":
        dt = _DT[c["dtype"]]
        q = _plain_rope(s["q"], s["pos"], s["freq"], c["interleaved"], False).to(dt)
        k = _plain_rope(s["k"], s["pos"], s["freq"], c["interleaved"], False).to(dt)
        kept = s["slots"] >= 0
        slots = s["slots"][kept]
        s["kc"].view(-1, c["kv_heads"], c["dim"])[slots] = k[kept]
        s["vc"].view(-1, c["kv_heads"], c["dim"])[slots] = s["v"][kept]
        return q, s["kc"], s["vc"]
    if op == "attend":
        return _plain_attend(s)
    return _plain_logprobs(s)


def _run_own(s):
    from invariant_gemm_bi_gb300 import binding as bi
    c = s["case"]
    op = c["op"]
    if op == "plan":
        p = bi.bi_paged_plan(s["ctx"], s["new"], s["table"], s["free"], c["page"], s["tokens"], out=s["plan"])
        return s["table"], p.seq_lens, p.token_offsets, p.positions, p.slots, p.totals
    if op == "rope":
        return bi.bi_rope(s["x"], s["pos"], s["config"], backward=c["backward"], out_dtype=_DT[c["out"]])
    if op == "store":
        q = bi.bi_paged_store(s["k"], s["v"], s["slots"], s["kc"], s["vc"], q=s["q"], positions=s["pos"],
                              config=s["config"])
        return q, s["kc"], s["vc"]
    if op == "attend":
        return bi.bi_paged_attention(s["q"], s["kc"], s["vc"], s["table"], s["lens"], c["dim"] ** -0.5,
                                     out_dtype=_DT[c["out"]], workspace=s["ws"])
    r = bi.bi_token_logprobs(s["x"], s["tokens"], top=c["top"])
    return (r.logprobs, r.entropy) if c["top"] == 0 else (r.logprobs, r.entropy, r.top_logprobs, r.top_ids)


# -- cost -----------------------------------------------------------------------------

def work(case):
    c = case
    if c["op"] == "plan":
        ctx, new = _lengths(c)
        ps = c["page"]
        tokens, fresh = sum(new), sum(-(-(x + n) // ps) + (-x // ps) for x, n in zip(ctx, new))
        touched = sum(-(-(x + n) // ps) - x // ps for x, n in zip(ctx, new) if n)  # pages that new tokens fall in
        return {"bytes": 16 * c["batch"] + 4 + 4 * (touched + fresh) + 12 * (tokens + c["pad"]) + 8,
                "flops": 4 * (tokens + c["pad"])}
    if c["op"] == "rope":
        n = c["tokens"] * c["heads"]
        return {"bytes": n * c["dim"] * (_SIZE[c["dtype"]] + _SIZE[c["out"]]) + 4 * c["tokens"],
                "flops": 3 * n * c["rotary"]}
    if c["op"] == "store":
        n = c["tokens"] * (c["heads"] + 2 * c["kv_heads"])
        return {"bytes": 2 * n * c["dim"] * _SIZE[c["dtype"]] + 12 * c["tokens"],
                "flops": 3 * c["tokens"] * (c["heads"] + c["kv_heads"]) * c["rotary"]}
    if c["op"] == "attend":
        lens = _lengths(c)
        e = _SIZE[c["dtype"]]
        rows = c["batch"] * c["heads"] * c["dim"]
        return {"bytes": 2 * sum(lens) * c["kv_heads"] * c["dim"] * e + rows * (e + _SIZE[c["out"]])
                + 4 * sum(-(-n // c["page"]) for n in lens) + 4 * c["batch"],
                "flops": 4 * sum(lens) * c["heads"] * c["dim"]}
    return {"bytes": c["rows"] * (c["vocab"] * _SIZE[c["dtype"]] + 16 + 8 * c["top"]),
            "flops": 6 * c["rows"] * c["vocab"]}


# -- 64-bit values ---------------------------------------------------------------------

def _exact_rotation(x, pos, case, backward):
    """Each pair as a complex number times exp(+-i pos f)."""
    f = np.array(_frequencies(case))
    x = x.double().cpu().numpy()
    half = f.size
    turn = np.exp((-1j if backward else 1j) * (pos.cpu().numpy().astype(np.float64)[:, None, None] * f))
    first = np.arange(half) * 2 if case["interleaved"] else np.arange(half)
    second = first + (1 if case["interleaved"] else half)
    z = (x[..., first] + 1j * x[..., second]) * turn
    y = x.copy()
    y[..., first], y[..., second] = z.real, z.imag
    return torch.from_numpy(y)


def exact(case, seed):
    c = case
    s = prepare(c, seed)
    if c["op"] == "plan":
        ps = c["page"]
        ctx, new = s["ctx"].tolist(), s["new"].tolist()
        table, free = s["table"].cpu().numpy().copy(), s["free"].tolist()
        slots = np.full(s["tokens"], -1, dtype=np.int64)
        pos = np.zeros(s["tokens"], dtype=np.int32)
        at, taken, offsets = 0, 0, [0]
        for b in range(c["batch"]):
            for page in range(-(-ctx[b] // ps), -(-(ctx[b] + new[b]) // ps)):
                table[b, page] = free[taken]
                taken += 1
            p = ctx[b] + np.arange(new[b])
            pos[at:at + new[b]] = p
            slots[at:at + new[b]] = table[b, p // ps].astype(np.int64) * ps + p % ps
            at += new[b]
            offsets.append(at)
        lens = np.array(ctx, dtype=np.int32) + np.array(new, dtype=np.int32)
        return (table, lens, np.array(offsets, dtype=np.int32), pos, slots, np.array([taken, at], dtype=np.int32))
    if c["op"] == "rope":
        return _exact_rotation(s["x"], s["pos"], c, c["backward"])
    if c["op"] == "store":
        q = _exact_rotation(s["q"], s["pos"], c, False)
        k = _exact_rotation(s["k"], s["pos"], c, False)
        kc, vc = s["kc"].double().cpu(), s["vc"].double().cpu()
        v, ps = s["v"].double().cpu(), c["page"]
        for t, slot in enumerate(s["slots"].tolist()):
            if slot >= 0:
                kc[slot // ps, slot % ps] = k[t]
                vc[slot // ps, slot % ps] = v[t]
        return q, kc, vc
    if c["op"] == "attend":
        lens, ps = s["lens_host"], c["page"]
        group = c["heads"] // c["kv_heads"]
        kc, vc = s["kc"].flatten(0, 1), s["vc"].flatten(0, 1)
        out = torch.zeros((c["batch"], c["heads"], c["dim"]), dtype=torch.float64)
        for b, n in enumerate(lens):
            j = torch.arange(n, device=kc.device)
            slot = s["table"][b, j // ps].long() * ps + j % ps
            for h in range(c["kv_heads"] if n else 0):
                k, v = kc[slot, h].double(), vc[slot, h].double()
                q = s["q"][b, h * group:(h + 1) * group].double()
                p = torch.softmax(q @ k.T / math.sqrt(c["dim"]), -1)
                out[b, h * group:(h + 1) * group] = (p @ v).cpu()
        return out
    outs = [[], [], [], []]
    for r in range(0, c["rows"], 64):
        logp = torch.log_softmax(s["x"][r:r + 64].double(), -1)
        outs[0].append(logp.gather(1, s["tokens"][r:r + 64, None])[:, 0].cpu())
        outs[1].append(-torch.special.xlogy(logp.exp(), logp.exp()).sum(-1).cpu())
        if c["top"]:
            order = torch.sort(s["x"][r:r + 64].double(), dim=-1, descending=True, stable=True).indices[:, :c["top"]]
            outs[2].append(logp.gather(1, order).cpu())
            outs[3].append(order.int().cpu())
    return tuple(torch.cat(o) for o in outs if o)
