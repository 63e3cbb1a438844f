"""The few-token mixture-of-experts layer against its definition in float64.

The reference is computed on the CPU in numpy float64 from the same inputs (weights as
the oracle dequantizes them): a stable sort for the choices, softmax or sigmoid weights,
and the three products expert by expert.

Tolerances (relative Frobenius error over all tokens). The kernels sum exact products of
bf16 values in fp32, h enters its product as the sum of two bf16 values (2^-17 of it at
most is dropped) and exp is good to a few 2^-23: float32 outputs are held to 2e-5. A bf16
output adds one rounding: up to 2^-8 of a value, 2^-9.2 in the root mean square over values
spread in their mantissas, here bounded by 2^-9. Weights: 1e-6, a few fp32 roundings.
"""

import numpy as np
import pytest
import torch

import mxfp8_block_scaled_amd as mx
from mxfp8_block_scaled_amd import synth

from gpu_util import dev_bf16, host, require_gpu, say

pytestmark = pytest.mark.gpu

F32_TOL = 2e-5
BF16_TOL = 2.0**-9 + F32_TOL
W_TOL = 1e-6


@pytest.fixture(scope="module", autouse=True)
def gpu():
    require_gpu()


def choose(logits, topk, score, renorm, scale):
    """(ids, weights) in float64, ties to the lowest index, NaN as -infinity."""
    lg = np.where(np.isnan(logits), -np.inf, logits).astype(np.float64)
    ids = np.argsort(-lg, axis=1, kind="stable")[:, :topk]
    lg = np.minimum(lg, np.finfo(np.float32).max)
    sel = np.take_along_axis(lg, ids, 1)
    if score == mx.MX_SCORE_SOFTMAX:
        top = np.where(np.isfinite(lg.max(1, keepdims=True)), lg.max(1, keepdims=True), 0)
        e = np.where(np.isfinite(sel), np.exp(sel - top), 0.0)
        den = np.where(np.isfinite(lg), np.exp(lg - top), 0.0).sum(1, keepdims=True)
    else:
        with np.errstate(over="ignore"):  # a score too small for float64 is 0
            e = np.where(np.isfinite(sel), 1 / (1 + np.exp(-sel)), 0.0)
        den = np.ones((len(lg), 1))
    if renorm:
        den = e.sum(1, keepdims=True)
    return ids, scale * np.divide(e, den, out=np.zeros_like(e), where=den > 0)


class Layer:
    """Seeded inputs of a layer and its float64 result."""

    def __init__(self, oracle, seed, tokens, hidden, ffn, local, kind="mx"):
        rng = np.random.default_rng(seed)
        self.tokens, self.hidden, self.ffn, self.local, self.kind = tokens, hidden, ffn, local, kind
        self.x = synth.normal_bf16(rng, (tokens, hidden), 1.0)
        w1 = synth.normal_bf16(rng, (local * 2 * ffn, hidden), hidden**-0.5)
        w2 = synth.normal_bf16(rng, (local * hidden, ffn), ffn**-0.5)
        self.res = synth.normal_bf16(rng, (tokens, hidden), 1.0)
        self.rng = rng
        if kind == "mx":
            (q1, s1), (q2, s2) = oracle.quantize_dim0(w1), oracle.quantize_dim0(w2)
            self.v1, self.v2 = oracle.dequantize(q1, s1), oracle.dequantize(q2, s2)
            up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to("cuda:0")  # noqa: E731
            self.dev_w = (up(q1), up(oracle.scales_to_physical(s1)), up(q2), up(oracle.scales_to_physical(s2)))
        else:
            self.v1, self.v2 = oracle.bf16_to_f64(w1), oracle.bf16_to_f64(w2)
            self.dev_w = (dev_bf16(w1), dev_bf16(w2))
        self.x64, self.res64 = oracle.bf16_to_f64(self.x), oracle.bf16_to_f64(self.res)

    def call(self, *args, **kw):
        f = mx.mx_moe_layer if self.kind == "mx" else mx.mx_moe_layer_bf16
        return f(*args[:2], *self.dev_w, self.ffn, *args[2:], **kw)

    def ref(self, ids, w, first, residual):
        v1 = self.v1.reshape(self.local, 2 * self.ffn, self.hidden)
        v2 = self.v2.reshape(self.local, self.hidden, self.ffn)
        y = self.res64.copy() if residual else np.zeros((self.tokens, self.hidden))
        for t in range(self.tokens):
            for e, we in zip(ids[t] - first, w[t]):
                if 0 <= e < self.local and we != 0:
                    z = v1[e] @ self.x64[t]
                    gate = z[: self.ffn]
                    y[t] += we * (v2[e] @ (gate / (1 + np.exp(-gate)) * z[self.ffn:]))
        return y


def close(got, ref, tol, name):
    err = np.linalg.norm(got - ref) / max(np.linalg.norm(ref), 1e-300) if ref.size else 0.0
    say(f"[moe] {name}: rel {err:.2e} (bound {tol:.2e})")
    assert np.isfinite(got).all() and err <= tol


CASES = [
    # tokens, hidden, ffn, experts, first, local, topk, score, renorm, scale, kind
    (1, 32, 32, 1, 0, 1, 1, 0, True, 1.0, "mx"),
    (1, 576, 256, 16, 0, 16, 2, 0, True, 1.0, "mx"),
    (2, 160, 96, 8, 4, 4, 8, 1, False, 2.5, "mx"),  # hidden and ffn not multiples of 128
    (5, 128, 64, 300, 100, 40, 6, 0, False, 1.0, "mx"),
    (16, 96, 160, 3, 0, 3, 3, 1, True, 1.0, "mx"),  # every token takes every expert
    (17, 288, 32, 4, 1, 2, 1, 0, True, 1.0, "mx"),
    (33, 64, 128, 65, 0, 65, 32, 0, True, 0.5, "mx"),
    (64, 256, 352, 8, 0, 8, 2, 1, True, 1.0, "mx"),
    (65, 64, 64, 2, 0, 2, 2, 0, True, 1.0, "mx"),  # 65 tokens for one expert: a second pass
    (200, 128, 96, 1024, 0, 1024, 4, 0, False, 1.0, "mx"),
    (256, 64, 32, 5, 0, 5, 5, 0, True, 1.0, "mx"),
    (1, 96, 64, 4, 0, 4, 2, 0, True, 1.0, "bf16"),
    (20, 160, 96, 6, 2, 3, 3, 1, True, 1.0, "bf16"),
]


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("out_dtype", [mx.MX_OUT_F32, mx.MX_OUT_BF16])
@pytest.mark.parametrize("case", CASES, ids=["-".join(str(v) for v in c) for c in CASES])
def test_matches_definition(oracle, case, out_dtype, residual):
    T, H, F, E, first, local, topk, score, renorm, scale, kind = case
    lay = Layer(oracle, T * 1000 + H + F, T, H, F, local, kind)
    logits = lay.rng.standard_normal((T, E)).astype(np.float32) * 2
    ids, w = choose(logits, topk, score, renorm, scale)
    say(f"[moe] case {case} out {out_dtype} residual {residual}")
    y, gi, gw = lay.call(dev_bf16(lay.x), torch.from_numpy(logits).to("cuda:0"), topk, expert_first=first, score=score,
                         renormalize=renorm, scale=scale, residual=dev_bf16(lay.res) if residual else None,
                         out_dtype=out_dtype)
    assert np.array_equal(host(gi), ids)
    close(host(gw), w, W_TOL, "weights")
    got = oracle.bf16_to_f64(host(y)) if out_dtype == mx.MX_OUT_BF16 else host(y).astype(np.float64)
    close(got, lay.ref(ids, w, first, residual), BF16_TOL if out_dtype == mx.MX_OUT_BF16 else F32_TOL, "y")


@pytest.mark.parametrize("score", [mx.MX_SCORE_SOFTMAX, mx.MX_SCORE_SIGMOID])
@pytest.mark.parametrize("renorm", [False, True])
def test_masks_ties_and_special_logits(oracle, score, renorm):
    T, H, F, E, topk = 9, 64, 64, 70, 4
    lay = Layer(oracle, 5, T, H, F, E)
    lg = lay.rng.standard_normal((T, E)).astype(np.float32)
    lg[0] = 0.25  # all equal: the lowest indexes
    lg[1] = -np.inf  # nothing to choose
    lg[2] = -np.inf
    lg[2, 41] = 1.0  # one choice
    lg[3] = np.nan
    lg[3, [5, 60, 69]] = [-1.0, 3.0, 2.0]  # NaN below every number
    lg[4] = np.finfo(np.float32).min  # the type's lowest value everywhere
    lg[5] = np.finfo(np.float32).min
    lg[5, [7, 66]] = 0.5
    lg[6, 3], lg[6, 50] = np.inf, np.inf
    lg[7] = 0.0
    lg[7, ::2] = -0.0  # zeros of either sign are equal
    ids, w = choose(lg, topk, score, renorm, 1.0)
    y, gi, gw = lay.call(dev_bf16(lay.x), torch.from_numpy(lg).to("cuda:0"), topk, score=score, renormalize=renorm,
                         out_dtype=mx.MX_OUT_F32)
    assert np.array_equal(host(gi), ids)
    close(host(gw), w, W_TOL, "weights")
    got, ref = host(y).astype(np.float64), lay.ref(ids, w, 0, False)
    close(got, ref, F32_TOL, "y")
    assert np.all(got[1] == 0)


def test_no_tokens():
    z = torch.zeros
    w1, w2 = z(64, 32, dtype=torch.uint8, device="cuda"), z(32, 32, dtype=torch.uint8, device="cuda")
    s = lambda r, c: z(mx.mx_scale_bytes(r, c), dtype=torch.uint8, device="cuda")  # noqa: E731
    y, ids, w = mx.mx_moe_layer(z(0, 32, dtype=torch.bfloat16, device="cuda"), z(0, 4, device="cuda"), w1, s(64, 32),
                                w2, s(32, 32), 32, 2)
    assert y.shape == (0, 32) and ids.shape == w.shape == (0, 2)


def test_strides_residual_in_place_and_repeat(oracle):
    """Rows of wider tensors, out on top of the residual, and the same bits every time."""
    T, H, F, E, topk = 21, 96, 64, 10, 3
    lay = Layer(oracle, 8, T, H, F, E)
    logits = lay.rng.standard_normal((T, E)).astype(np.float32)
    wide_x = torch.full((T, H + 40), float("nan"), dtype=torch.bfloat16, device="cuda:0")
    wide_x[:, 8:8 + H] = dev_bf16(lay.x)
    wide_l = torch.full((T, E + 7), float("inf"), device="cuda:0")
    wide_l[:, 3:3 + E] = torch.from_numpy(logits).to("cuda:0")
    plain = lay.call(dev_bf16(lay.x), torch.from_numpy(logits).to("cuda:0"), topk, residual=dev_bf16(lay.res))
    res = dev_bf16(lay.res)
    y, ids, w = lay.call(wide_x[:, 8:8 + H], wide_l[:, 3:3 + E], topk, residual=res, out=res)
    for a, b in zip(plain, (y, ids, w)):
        assert torch.equal(a, b)
    for _ in range(3):
        assert torch.equal(lay.call(dev_bf16(lay.x), torch.from_numpy(logits).to("cuda:0"), topk,
                                    residual=dev_bf16(lay.res))[0], plain[0])


def test_scales_over_the_whole_range(oracle):
    """Scale bytes far from 127, among them 0 and 1: exact powers of two all the way."""
    T, H, F = 3, 128, 64
    lay = Layer(oracle, 9, T, H, F, 1)
    s1 = np.full(mx.mx_scale_bytes(2 * F, H), 127, np.uint8)
    s2 = np.full(mx.mx_scale_bytes(H, F), 127, np.uint8)
    q1, q2 = host(lay.dev_w[0]), host(lay.dev_w[2])
    # gate rows tiny in half of their blocks (bytes 0 and 1 vanish beside the others), down rows scaled by 2^90
    log1 = lay.rng.choice([0, 1, 60, 120], size=(2 * F, H // 32)).astype(np.uint8)
    log2 = np.full((H, F // 32), 217, np.uint8)
    s1[:] = oracle.scales_to_physical(log1)
    s2[:] = oracle.scales_to_physical(log2)
    lay.v1, lay.v2 = oracle.dequantize(q1, log1), oracle.dequantize(q2, log2)
    lay.dev_w = (lay.dev_w[0], torch.from_numpy(s1).to("cuda:0"), lay.dev_w[2], torch.from_numpy(s2).to("cuda:0"))
    logits = np.zeros((T, 1), np.float32)
    y, ids, w = lay.call(dev_bf16(lay.x), torch.from_numpy(logits).to("cuda:0"), 1, out_dtype=mx.MX_OUT_F32)
    close(host(y).astype(np.float64), lay.ref(np.zeros((T, 1), int), np.ones((T, 1)), 0, False), F32_TOL, "scales")


def test_side_stream_and_graph(oracle):
    T, H, F, E, topk = 7, 128, 64, 6, 2
    lay = Layer(oracle, 11, T, H, F, E)
    x = dev_bf16(lay.x)
    lg = [torch.randn(T, E, device="cuda:0") for _ in range(3)]
    want = [lay.call(x, g, topk) for g in lg]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = lay.call(x, lg[0], topk)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want[0]))
    cur = lg[0].clone()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        out = lay.call(x, cur, topk)
    for k in (0, 1, 2, 1):
        cur.copy_(lg[k])
        lay.call(x, lg[(k + 1) % 3], topk)  # eager work between the replays
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want[k])), k


def test_refusals(oracle):
    lay = Layer(oracle, 12, 2, 64, 32, 4)
    x, lg = dev_bf16(lay.x), torch.zeros(2, 4, device="cuda:0")
    ok = lay.call(x, lg, 2)
    assert ok[0].shape == (2, 64)
    with pytest.raises(mx.MXError, match="topk"):
        lay.call(x, lg, 5)
    with pytest.raises(mx.MXError, match="experts"):
        lay.call(x, lg, 2, expert_first=1)
    with pytest.raises(mx.MXError, match="score"):
        lay.call(x, lg, 2, score=3)
    with pytest.raises(mx.MXError, match="scale"):
        lay.call(x, lg, 2, scale=float("nan"))
    with pytest.raises(mx.MXError, match="workspace"):
        lay.call(x, lg, 2, workspace=torch.empty(16, dtype=torch.uint8, device="cuda:0"))
    with pytest.raises(ValueError, match="logits"):
        lay.call(x, lg.double(), 2)
    with pytest.raises(ValueError, match="logits"):
        lay.call(x, lg[:1], 2)
    with pytest.raises(ValueError, match="w1"):
        mx.mx_moe_layer(x, lg, lay.dev_w[0][:-1], *lay.dev_w[1:], 32, 2)
    with pytest.raises(ValueError, match="w2"):
        mx.mx_moe_layer(x, lg, *lay.dev_w[:2], lay.dev_w[2][:-1], lay.dev_w[3], 32, 2)
    with pytest.raises(ValueError, match="residual"):
        lay.call(x, lg, 2, residual=dev_bf16(lay.res)[:1])
    with pytest.raises(ValueError):
        mx.mx_moe_layer_workspace_bytes(257, 32, 32, 2)


@pytest.mark.parametrize("kind", ["mx", "bf16"])
@pytest.mark.parametrize("tokens", [65, 130, 256])
def test_many_tokens_same_bits(oracle, kind, tokens):
    """Above 64 tokens an expert's tokens take several runs, whose sums meet in memory: the same
    bits on every call, and the definition's values."""
    H, F, E, topk = 288, 160, 7, 5
    lay = Layer(oracle, tokens, tokens, H, F, E, kind)
    logits = lay.rng.standard_normal((tokens, E)).astype(np.float32)
    x, lg, res = dev_bf16(lay.x), torch.from_numpy(logits).to("cuda:0"), dev_bf16(lay.res)
    want = lay.call(x, lg, topk, residual=res, out_dtype=mx.MX_OUT_F32)
    ids, w = choose(logits, topk, mx.MX_SCORE_SOFTMAX, True, 1.0)
    assert np.array_equal(host(want[1]), ids)
    close(host(want[0]).astype(np.float64), lay.ref(ids, w, 0, True), F32_TOL, "y")
    flush = torch.empty(1 << 29, dtype=torch.uint8, device="cuda:0")
    for i in range(6):
        if i % 2:
            flush.fill_(i)
        again = lay.call(x, lg, topk, residual=res, out_dtype=mx.MX_OUT_F32)
        assert all(torch.equal(a, b) for a, b in zip(again, want)), i


# Contractions that go round the prefetch of every kernel: 33 and 32 steps of 128 elements over
# eight waves in the gate/up products, and a down product whose steps cross experts in every wave
# (5 experts of 9 steps, the last one short). Per batch size the kernels with 4, 8 and 16 columns,
# the ones for more tokens in one pass and in several.
LONG = [(t, 4128, 96, 3, 0, 3, 3, 0, True, 1.0) for t in (1, 4, 6, 8, 12, 40, 64, 130)]
LONG += [(12, 4128, 352, 3, 0, 3, 2, 0, True, 1.0), (3, 4096, 64, 4, 1, 2, 4, 1, True, 1.0),
         (70, 4096, 64, 4, 1, 2, 4, 1, True, 1.0)]
LONG += [(t, 96, 1120, 5, 0, 5, 5, 1, True, 1.0) for t in (1, 4, 6, 12, 40, 64, 130, 256)]
LONG += [(t, 160, 2080, 6, 0, 6, 3, 0, True, 1.0) for t in (2, 7, 15, 33, 100)]


@pytest.mark.parametrize("kind", ["mx", "bf16"])
@pytest.mark.parametrize("case", LONG, ids=["-".join(str(v) for v in c[:7]) for c in LONG])
def test_long_contractions(oracle, case, kind):
    test_matches_definition(oracle, (*case, kind), mx.MX_OUT_F32, True)


@pytest.mark.parametrize("kind", ["mx", "bf16"])
@pytest.mark.parametrize("tokens", [3, 8, 14, 40, 100])
def test_a_token_of_nan_stays_alone(oracle, kind, tokens):
    """NaN and infinity in one token's x reach that token's output alone, whichever tokens share its expert."""
    H, F, E, topk = 416, 288, 4, 2
    lay = Layer(oracle, tokens, tokens, H, F, E, kind)
    logits = torch.from_numpy(lay.rng.standard_normal((tokens, E)).astype(np.float32)).to("cuda:0")
    x = dev_bf16(lay.x)
    want = lay.call(x, logits, topk, out_dtype=mx.MX_OUT_F32)[0]
    bad = x.clone()
    bad[1] = float("nan")
    bad[tokens - 1, 5] = float("inf")
    got = lay.call(bad, logits, topk, out_dtype=mx.MX_OUT_F32)[0]
    rest = [t for t in range(tokens) if t not in (1, tokens - 1)]
    assert torch.equal(got[rest], want[rest])
    assert torch.isnan(got[1]).all()
