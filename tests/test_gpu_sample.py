"""Token sampling on the GPU against a plain 64-bit implementation
(tests/quantized_reference.py): the same token, except where a row's given number
or limit is within 2^-30 of a border, which hardly any row's is; and the whole
decode step in 8 bits."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from invariant_gemm_bi_gb300 import binding as bi
from tests import quantized_reference as ref
from tests import serving_reference as sref
from tests.gpu_helpers import bits_equal

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
INF = float("inf")


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(shape, dtype, seed, std=1.0):
    return (torch.randn(shape, generator=_gen(seed), device="cuda", dtype=F32) * std).to(dtype)


def _f32(v):
    return torch.tensor(v, dtype=F32, device="cuda")


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.fixture(autouse=True)
def _clean_status():
    bi.load()
    assert bi.bi_device_status() == bi.BI_OK
    yield
    assert bi.bi_device_status() == bi.BI_OK


def _settings(R, seed, ks=(0, 1, 2, 7, 40), ps=(1.0, 0.5, 0.9, 0.05, 0.0, 1.5), ms=(0.0, 0.01, 0.3, 1.0, -1.0),
              ts=(1.0, 0.7, 0.2, 0.0, 3.0, 1e-7)):
    rng = np.random.default_rng(seed)
    return dict(temperature=_f32(rng.choice(ts, R)), top_k=_i32(rng.choice(ks, R)), top_p=_f32(rng.choice(ps, R)),
                min_p=_f32(rng.choice(ms, R)))


def _check(x, u, most_near=2, **settings):
    got = bi.bi_sample_tokens(x, u, **settings).tolist()
    x64, u64 = sref.f64(x), sref.f64(u)
    s = {k: v.double().cpu().numpy() for k, v in settings.items()}
    skipped = 0
    for r in range(x.shape[0]):
        want, near = ref.sample(x64[r], u64[r], s["temperature"][r] if "temperature" in s else 1.0,
                                int(s["top_k"][r]) if "top_k" in s else 0, s["top_p"][r] if "top_p" in s else 1.0,
                                s["min_p"][r] if "min_p" in s else 0.0)
        if near:
            skipped += 1
        else:
            assert got[r] == want, (r, got[r], want, {k: v[r] for k, v in s.items()}, u64[r])
    assert skipped <= most_near
    return got


@pytest.mark.parametrize("R,N,dt", [(300, 1, F32), (300, 2, BF16), (300, 7, F32), (200, 33, F16), (200, 1000, BF16),
                                    (100, 4097, F32), (60, 16384, F16), (60, 16385, F32), (40, 50001, BF16),
                                    (20, 128256, F32), (20, 128256, BF16), (6, 327680, F32), (6, 327679, F16)])
def test_sample_matches_reference(R, N, dt):
    x = _normal((R, N), dt, N, 3.0)
    u = torch.rand((R,), generator=_gen(R + N), device="cuda")
    _check(x, u)
    _check(x, u, **_settings(R, N))


@pytest.mark.parametrize("std", [0.01, 0.3, 20.0, 1000.0])
@pytest.mark.parametrize("dt", [F32, BF16])
def test_sample_flat_and_steep_rows(std, dt):
    x = _normal((60, 30000), dt, 3, std)
    u = torch.rand((60,), generator=_gen(4), device="cuda")
    _check(x, u)
    _check(x, u, **_settings(60, 5, ks=(0, 50, 1000, 20000, 29999, 30000, 10 ** 9)))


def test_sample_many_equal_logits():
    # few values, so that every limit falls among equals, which go by their index
    x = torch.randint(-3, 4, (300, 500), generator=_gen(1), device="cuda").float()
    u = torch.rand((300,), generator=_gen(2), device="cuda")
    _check(x, u, **_settings(300, 3, ks=(0, 1, 2, 50, 100, 499, 500), ps=(1.0, 0.3, 0.9, 0.99)))
    x = torch.zeros((400, 1000), dtype=BF16, device="cuda")
    u = (torch.arange(400, device="cuda") / 400.0)
    # 400 shares of a row, all sums without rounding (2 / 400 in fp32 is below 0.005: token 4)
    assert _check(x, u, 0)[:4] == [0, 2, 4, 7]
    assert max(_check(x, u, 0, top_k=_i32([10] * 400))) == 9
    assert max(_check(x, u, 0, top_p=_f32([0.5] * 400))) == 498  # 399 / 400 of 500
    assert max(_check(x, u, 0, top_p=_f32([0.5] * 400), top_k=_i32([100] * 400))) == 49
    assert set(_check(x, u, 0, temperature=_f32([0.0] * 400))) == {0}


def test_sample_ends_of_the_unit_interval():
    x = _normal((64, 3000), F32, 7, 2.0)
    top = np.nextafter(np.float32(1), np.float32(0))
    zero = bi.bi_sample_tokens(x, _f32([0.0] * 64)).tolist()
    assert zero == [0] * 64  # every token has a weight: the first
    last = bi.bi_sample_tokens(x, _f32([top] * 64)).tolist()
    for r in range(64):
        w = np.exp(sref.f64(x[r]) - float(x[r].max()))
        tail = np.cumsum(w[::-1])[::-1] / w.sum()
        assert tail[last[r]] >= 2.0 ** -24 * (1 - 1e-6)  # that share of the row's end reaches it
    _check(x, _f32([float(top)] * 64), 64)


def test_sample_masked_rows():
    N = 5000
    x = _normal((12, N), F32, 9, 2.0)
    keep = [17, 18, 300, 4999]
    low = torch.finfo(F32).min
    for r, fill in ((0, -INF), (1, low), (2, -1e30)):
        m = torch.full((N,), fill, device="cuda")
        m[keep] = x[r, keep]
        x[r] = m
    x[3] = low         # nothing but the type's lowest value: all alike
    x[4] = -INF        # nothing left
    x[5, 100] = float("nan")
    x[6, 100] = INF
    x[7] = -INF
    x[7, 4321] = -5.0  # one left
    x[8] = -INF
    x[8, 10], x[8, 11] = low, low
    x[9, ::2] = 3e38
    x[9, 1::2] = -3e38
    x[10] = 0.0
    x[10, 1::2] = -0.0
    x[11] = 1e-45
    u = torch.rand((12,), generator=_gen(1), device="cuda")
    for s in ({}, _settings(12, 1, ts=(1.0, 0.5)), dict(top_k=_i32([3] * 12)), dict(top_p=_f32([0.9] * 12)),
              dict(min_p=_f32([0.1] * 12)), dict(temperature=_f32([0.0] * 12))):
        got = _check(x, u, 1, **s)
        assert got[4:8] == [-1, -1, -1, 4321] and got[0] in keep and got[1] in keep and got[2] in keep
        assert got[8] in (10, 11)
        y = x[:5].clamp(min=-65504).to(F16)  # masks of fp16's lowest value
        y[4] = -65504.0
        _check(y, u[:5], 1, **{k: v[:5] for k, v in s.items()})


def test_sample_settings_that_are_none():
    x = _normal((9, 100), BF16, 2)
    u = _f32([0.5, 1.0, -0.1, float("nan"), 0.5, 0.5, 0.5, 0.5, 0.5])
    t = _f32([1, 1, 1, 1, -1.0, float("nan"), INF, 1, 1])
    p = _f32([1] * 7 + [float("nan"), 1])
    m = _f32([0] * 8 + [float("nan")])
    got = bi.bi_sample_tokens(x, u, temperature=t, top_p=p, min_p=m).tolist()
    assert got[0] >= 0 and got[1:] == [-1] * 8
    assert bi.bi_device_status() == bi.BI_ERR_INVALID_ARG and "setting" in bi.last_error_message()
    edge = _f32([2.0 ** 20, 2.0 ** -20, 2.0 ** -21, 1e-40])
    _check(x[:4], u[[0, 0, 0, 0]], temperature=edge)


def test_sample_rows_do_not_depend_on_the_batch_or_the_layout():
    R, N = 70, 40001
    x = _normal((R, N), BF16, 5, 3.0)
    u = torch.rand((R,), generator=_gen(6), device="cuda")
    s = _settings(R, 8)
    full = bi.bi_sample_tokens(x, u, **s)
    for r in (0, 1, 33, 69):
        one = {k: v[r:r + 1] for k, v in s.items()}
        assert torch.equal(bi.bi_sample_tokens(x[r:r + 1], u[r:r + 1], **one), full[r:r + 1])
    wide = torch.full((R, N + 13), 50.0, dtype=BF16, device="cuda")  # neighbours that would win
    for off in (0, 1, 5, 8, 13):
        wide.fill_(50.0)
        wide[:, off:off + N] = x
        assert torch.equal(bi.bi_sample_tokens(wide[:, off:off + N], u, **s), full), off
    out = torch.full((R + 2,), 7, dtype=torch.int32, device="cuda")
    bi.bi_sample_tokens(x, u, out=out[1:-1], **s)
    assert out[1:-1].tolist() == full.tolist() and out[0] == 7 and out[-1] == 7
    # bf16 logits as fp32: the same numbers, the same tokens
    assert torch.equal(bi.bi_sample_tokens(x.float(), u, **s), full)
    assert bi.bi_sample_tokens(x[:0], u[:0]).shape == (0,)


def test_sample_shares_follow_the_distribution():
    # a thousand numbers in equal steps give each token its share to within a step
    p = np.array([0.4, 0.05, 0.3, 0.0, 0.25])
    with np.errstate(divide="ignore"):
        x = torch.from_numpy(np.log(p)).float().cuda().expand(1000, 5).contiguous()
    got = np.bincount(bi.bi_sample_tokens(x, (torch.arange(1000, device="cuda") + 0.5) / 1000).cpu().numpy(), minlength=5)
    assert np.all(np.abs(got / 1000 - p) <= 1.001e-3) and got[3] == 0


# -- the decode step in 8 bits, as it is used --------------------------------------------------

def _step(st):
    """One decode step: x -> qkv -> store -> attend -> output and logits -> tokens."""
    B, hq, hkv, d = st["B"], st["hq"], st["hkv"], st["d"]
    plan = bi.bi_paged_plan(st["ctx"], st["new"], st["table"], st["pool"], st["page"], out=st["plan"])
    x = bi.bi_quantize_blocks(st["x"])
    qkv = bi.bi_mm_blockscaled(x.values, x.scales, st["wqkv"].values.t(), st["wqkv"].scales.t()).view(B, hq + 2 * hkv, d)
    q = bi.bi_paged_store_quantized(qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], plan.slots, st["kc"], st["ks"], st["vc"],
                                    st["vs"], q=qkv[:, :hq], positions=plan.positions, config=st["config"])
    o = bi.bi_paged_attention_quantized(q, st["kc"], st["ks"], st["vc"], st["vs"], st["table"], plan.seq_lens,
                                        d ** -0.5, out_dtype=BF16, workspace=st["ws"])
    y = bi.bi_quantize_blocks(o.view(B, hq * d))
    logits = bi.bi_mm_blockscaled(y.values, y.scales, st["head"].values.t(), st["head"].scales.t(), out_dtype=F32)
    tokens = bi.bi_sample_tokens(logits, st["u"], temperature=st["t"], top_k=st["k"], top_p=st["p"])
    lp = bi.bi_token_logprobs(logits, tokens)
    return q, o, logits, tokens, lp.logprobs


def _state(B=5, seed=0):
    hq, hkv, d, page, vocab, E = 8, 2, 64, 16, 1000, 300
    W = 6
    table = torch.full((B, W), -1, dtype=torch.int32)
    ctx = [0, 15, 16, 40, 77, 3, 90][:B]
    at = 0
    for b, n in enumerate(ctx):
        need = -(-n // page)
        table[b, :need] = torch.arange(at, at + need)
        at += need
    P = at + B + 2
    ws = bi.bi_paged_attention_workspace_bytes(B, hq, d, W * page)
    kx, vx = (_normal((P, page, hkv, d), F32, seed + i) for i in (1, 2))
    return dict(B=B, hq=hq, hkv=hkv, d=d, page=page, ctx=_i32(ctx), new=_i32([1] * B), table=table.cuda(),
                pool=torch.arange(at, P, dtype=torch.int32, device="cuda"), plan=bi.bi_paged_plan_buffers(B, B),
                x=_normal((B, E), BF16, seed + 3), wqkv=bi.bi_quantize_blocks(_normal(((hq + 2 * hkv) * d, E), BF16, seed + 4, 0.1), 128),
                head=bi.bi_quantize_blocks(_normal((vocab, hq * d), BF16, seed + 5, 0.3), 128),
                kc=(kx * 100).to(torch.float8_e4m3fn), ks=torch.full((P, page, hkv), 0.01, device="cuda"),
                vc=(vx * 100).to(torch.float8_e4m3fn), vs=torch.full((P, page, hkv), 0.01, device="cuda"),
                config=bi.bi_rope_config(d), u=torch.rand((B,), generator=_gen(seed), device="cuda"),
                t=_f32([0.8] * B), k=_i32([50] * B), p=_f32([0.9] * B), ws=torch.empty(max(ws, 16), dtype=torch.uint8, device="cuda"))


def test_decode_step_in_8_bits():
    st = _state()
    q, o, logits, tokens, lp = _step(st)
    # each stage against the plain form of the stage before it
    want, bound = ref.attention(q, st["kc"], st["ks"], st["vc"], st["vs"], st["table"], st["plan"].seq_lens, 0.125, BF16)
    sref.assert_within(o, want, bound, "attention")
    y, ys = ref.quantize_blocks(o.reshape(5, -1), 1)
    h = ref.from_e4m3(st["head"].values) * np.repeat(np.repeat(sref.f64(st["head"].scales), 128, 0)[:1000], 128, 1)
    plain = (y * np.repeat(ys, 128, 1)) @ h.T
    size = np.abs(y * np.repeat(ys, 128, 1)) @ np.abs(h).T
    sref.assert_within(logits, plain, (16 * 2.0 ** -22 + 4 * 2.0 ** -24) * size + 2.0 ** -24 * np.abs(plain), "logits")
    for b in range(5):
        t, near = ref.sample(sref.f64(logits[b]), float(st["u"][b]), float(np.float32(0.8)), 50, float(np.float32(0.9)))
        assert near or int(tokens[b]) == t
    lref = sref.logprobs(logits, tokens.tolist(), 1)
    sref.assert_within(lp, lref[0], lref[4], "log probabilities")
    # the keys just written read back are the step's own, and a request's step does not depend on the batch
    rows = bi.bi_paged_load_quantized(st["plan"].slots, st["kc"], st["ks"], st["vc"], st["vs"], out_dtype=F32)
    assert rows.k.shape == (5, 2, 64) and torch.isfinite(rows.k).all() and torch.isfinite(rows.v).all()
    one = _state()
    for name in ("ctx", "new", "u", "t", "k", "p"):
        one[name] = one[name][3:4].contiguous()
    one.update(B=1, x=one["x"][3:4], table=one["table"][3:4], plan=bi.bi_paged_plan_buffers(1, 1))
    alone = _step(one)
    for a, b in zip(alone, (q, o, logits, tokens, lp)):
        assert bits_equal(a.contiguous(), b[3:4].contiguous())


def test_decode_step_captured_replayed_and_on_another_stream():
    st = _state(seed=9)
    first = [t.clone() for t in _step(st)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        eager = [t.clone() for t in _step(st)]
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(eager, first):
        assert bits_equal(a, b)
    with torch.cuda.graph(graph):
        out = _step(st)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(out, first):
        assert bits_equal(a, b)
    # other inputs and longer requests in the captured extents
    st["x"].copy_(_normal(st["x"].shape, BF16, 77))
    st["ctx"].copy_(_i32([10, 20, 30, 5, 60]))
    st["u"].copy_(_f32([0.1, 0.9, 0.3, 0.7, 0.5]))
    for b in range(5):
        st["table"][b] = torch.arange(6 * b, 6 * b + 6, device="cuda") % st["kc"].shape[0]
    graph.replay()
    torch.cuda.synchronize()
    again = [t.clone() for t in out]
    for a, b in zip(_step(st), again):
        assert bits_equal(a, b)


def test_streams_run_side_by_side():
    # calls on two streams at once, workspaces of their own
    x = [_normal((9, 50000), F32, i, 3.0) for i in range(2)]
    u = [torch.rand((9,), generator=_gen(i), device="cuda") for i in range(2)]
    s = _settings(9, 3)
    want = [bi.bi_sample_tokens(x[i], u[i], **s) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(10):
        for i in range(2):
            got[i].append(bi.bi_sample_tokens(x[i], u[i], stream=streams[i], **s))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            assert torch.equal(g, want[i])
