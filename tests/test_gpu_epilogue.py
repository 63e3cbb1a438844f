"""The grouped products with bias, activation and residual in their epilogue, and the
backward of that epilogue, against float64 on the CPU.

Tolerances. z = A B^T + bias: with MXFP8 operands the block-scaled MFMA leaves a relative
error (Frobenius) of about 1.45e-5 in A B^T, bounded here by 2e-5; with bf16 operands fp32
sums leave 1e-6. The error of out follows to first order: every activation's slope is below
1.13, and silu(g) u takes 1.1 |u| of g's error and |g| of u's; errors of z do not depend on
the values they meet, so norms multiply as root mean squares (margin 1.5). exp and the
reciprocal add 1e-6. A bf16 result adds a rounding of half a unit in its last place (8 bits:
up to 2^-8 of a value, 2^-9.2 in the root mean square over values spread in their mantissas,
here bounded by 2^-9 in norms; element by element the half unit itself is used).
"""

import numpy as np
import pytest
import torch

import mxfp8_block_scaled_amd as mx
from mxfp8_block_scaled_amd import synth

from gpu_util import dev_bf16, dev_i32, host, require_gpu, say

pytestmark = pytest.mark.gpu

NONE, RELU, GELU, SILU, SWIGLU = (mx.MX_ACT_NONE, mx.MX_ACT_RELU, mx.MX_ACT_GELU, mx.MX_ACT_SILU, mx.MX_ACT_SWIGLU)
BF16, F32 = mx.MX_OUT_BF16, mx.MX_OUT_F32


@pytest.fixture(scope="module", autouse=True)
def gpu():
    require_gpu()


def sigmoid(z):
    with np.errstate(over="ignore"):
        return 1 / (1 + np.exp(-z))


def act64(z, act):
    if act == RELU:
        return np.maximum(z, 0)
    if act == GELU:
        return 0.5 * z * (1 + np.tanh(np.sqrt(2 / np.pi) * (z + 0.044715 * z**3)))
    if act == SILU:
        return z * sigmoid(z)
    if act == SWIGLU:
        g, u = np.split(z, 2, axis=1)
        return g * sigmoid(g) * u
    return z


def half_ulp_bf16(v):
    """Half a unit in the last place of bf16 (8 significant bits) at v."""
    return np.exp2(np.floor(np.log2(np.maximum(np.abs(v), 2.0**-126))) - 8)


def rms(a):
    return float(np.sqrt(np.mean(a * a))) if a.size else 0.0


def out_bound(z, y, act, e, bf16):
    """Bound of the Frobenius error of out, e the relative error of z."""
    ez = e * rms(z)
    if act == SWIGLU:
        g, u = np.split(z, 2, axis=1)
        per = 1.5 * ez * (1.1 * rms(u) + rms(g))
    else:
        per = 1.13 * ez
    return np.sqrt(y.size) * (per + 1e-6 * rms(y)) + (2.0**-9 * np.linalg.norm(y) if bf16 else 0.0)


def check(got, ref, bound, name):
    assert np.isfinite(got).all(), name
    err = float(np.linalg.norm(got - ref))
    say(f"[epilogue] {name}: error {err:.3e}, bound {bound:.3e}")
    assert err <= bound, name


def val(oracle, t):
    h = host(t)
    return oracle.bf16_to_f64(h) if h.dtype == np.uint16 else h.astype(np.float64)


CASES = [
    # kind, m, n, k, group sizes (None: dense), act, bias, residual, pre, out
    ("mx", 1, 1, 32, None, SILU, True, True, True, F32),
    ("mx", 40, 37, 64, None, GELU, True, True, True, BF16),  # n odd: element by element
    ("mx", 129, 72, 96, None, RELU, True, False, True, BF16),  # ragged right edge of whole chunks
    ("mx", 300, 260, 160, None, SILU, True, True, True, F32),
    ("mx", 256, 256, 256, None, SILU, True, False, False, BF16),
    ("mx", 160, 64, 64, [32, 0, 96], SWIGLU, True, True, True, BF16),  # rows past the last group; an empty one
    ("mx", 448, 192, 288, [64, 32, 0, 352], SWIGLU, True, True, True, F32),
    ("mx", 256, 320, 96, [0, 256], NONE, True, True, False, BF16),
    ("mx", 4096, 2112, 64, None, SWIGLU, True, True, True, BF16),  # 128x256 tiles, n not a multiple of 128
    ("mx", 4096, 2336, 64, [1024, 3072], GELU, False, True, True, BF16),
    ("mx", 4128, 4160, 1056, [2080, 0, 2048], SWIGLU, True, True, True, BF16),  # 256x256 tiles
    ("mx", 4100, 4104, 1056, None, GELU, True, True, True, F32),
    ("bf16", 1, 8, 8, None, GELU, True, True, True, BF16),
    ("bf16", 77, 45, 72, None, SILU, True, True, True, F32),
    ("bf16", 129, 128, 200, [1, 0, 100, 28], SWIGLU, True, True, True, BF16),  # group ends anywhere
    ("bf16", 130, 36, 64, [7, 120], NONE, True, True, True, F32),
    ("bf16", 4100, 2304, 64, [3000, 1100], SILU, True, True, True, BF16),
    ("bf16", 150, 131, 72, [50, 0, 99], GELU, True, True, True, BF16),  # odd rows of several groups
    ("bf16", 2200, 2154, 64, None, RELU, True, True, True, F32),
]


def operands(oracle, rng, kind, rows, k, std):
    bits = synth.normal_bf16(rng, (rows, k), std)
    if kind == "bf16":
        return oracle.bf16_to_f64(bits), (dev_bf16(bits),)
    q, s = oracle.quantize_dim0(bits)
    return oracle.dequantize(q, s), (torch.from_numpy(q).to("cuda:0"),
                                     torch.from_numpy(oracle.scales_to_physical(s)).to("cuda:0"))


@pytest.mark.parametrize("case", CASES, ids=["-".join(map(str, c[:4])) + f"-act{c[5]}" for c in CASES])
def test_forward(oracle, case):
    kind, m, n, k, sizes, act, bias, residual, pre, out_dtype = case
    rng = np.random.default_rng(m + n + k)
    G = 1 if sizes is None else len(sizes)
    a, da = operands(oracle, rng, kind, m, k, 1.0)
    b, db = operands(oracle, rng, kind, G * n, k, k**-0.5)
    offs = None if sizes is None else np.cumsum(sizes)
    live = m if offs is None else int(offs[-1])
    bias_np = rng.standard_normal((G, n)).astype(np.float32)
    n_out = n // 2 if act == SWIGLU else n
    res_bits = synth.normal_bf16(rng, (m, n_out), 1.0)
    res64 = oracle.bf16_to_f64(res_bits)
    ref = a[:, :] @ b[:n].T if G == 1 else np.concatenate(
        [a[s:e] @ b[g * n:(g + 1) * n].T for g, (s, e) in enumerate(zip([0, *offs[:-1]], offs))])
    ref = ref[:live]
    ab = rms(ref)
    if bias:
        ref = ref + np.repeat(bias_np.astype(np.float64), [m] if offs is None else sizes, axis=0)[:live]
    y = act64(ref, act) + (res64[:live] if residual else 0)
    dt = torch.bfloat16 if out_dtype == BF16 else torch.float32
    out = torch.full((m, n_out), 77.0, dtype=dt, device="cuda:0")
    pre_t = torch.full((m, n), 55.0, dtype=torch.bfloat16, device="cuda:0") if pre else None
    res_t = dev_bf16(res_bits) if residual else None
    if residual and out_dtype == F32:
        res_t = res_t.float()
    f = mx.mx_grouped_mm_fwd_epilogue if kind == "mx" else mx.mx_grouped_mm_bf16_fwd_epilogue
    say(f"[epilogue] {case}")
    got, z = f(*da, *db, None if offs is None else dev_i32(offs), m, n, k,
               bias=torch.from_numpy(bias_np).to("cuda:0") if bias else None, act=act, residual=res_t, out=out,
               pre=pre_t, out_dtype=out_dtype)
    e = (2e-5 if kind == "mx" else 1e-6) * ab / rms(ref)  # the product's error, relative to z
    got = val(oracle, got)
    check(got[:live], y, out_bound(ref, y, act, e + 1e-6, out_dtype == BF16), "out")
    assert np.all(got[live:] == 77.0)  # rows of no group stay as they were
    if pre:
        z = val(oracle, z)
        check(z[:live], ref, np.linalg.norm(ref) * (e + 1e-6 + 2.0**-9), "pre")
        assert np.all(z[live:] == 55.0)
    else:
        assert z is None


@pytest.mark.parametrize("act", [SWIGLU, SILU])
def test_forward_unpadded_outputs(oracle, act):
    """Token-group padded operand rows, unpadded out, residual and pre."""
    rng = np.random.default_rng(3)
    sizes, n, k = [5, 0, 70, 33], 128, 96
    m, G = sum(sizes), len(sizes)
    n_out = n // 2 if act == SWIGLU else n
    x = synth.normal_bf16(rng, (m, k), 1.0)
    w, dw = operands(oracle, rng, "mx", G * n, k, k**-0.5)
    offs = dev_i32(np.cumsum(sizes))
    q, s, _, _, offs_pad = mx.mx_pad_quantize_dim0_dim1(dev_bf16(x), offs)
    m_pad = q.shape[0]
    res = dev_bf16(synth.normal_bf16(rng, (m, n_out), 1.0))
    bias = torch.from_numpy(rng.standard_normal((G, n)).astype(np.float32)).to("cuda:0")
    out_dtype = BF16 if act == SWIGLU else F32
    out, pre = mx.mx_grouped_mm_fwd_epilogue(q, s, *dw, offs_pad, m_pad, n, k, bias=bias, act=act,
                                             residual=res if out_dtype == BF16 else res.float(), save_pre=True,
                                             offs_out=offs, m_out=m, out_dtype=out_dtype)
    xq, xs = oracle.quantize_dim0(x)
    a = oracle.dequantize(xq, xs)
    ends = np.cumsum([0] + sizes)
    z = np.concatenate([a[ends[g]:ends[g + 1]] @ w[g * n:(g + 1) * n].T + host(bias).astype(np.float64)[g]
                        for g in range(G)])
    y = act64(z, act) + val(oracle, res)
    check(val(oracle, out), y, out_bound(z, y, act, 2.1e-5, act == SWIGLU), "out")
    check(val(oracle, pre), z, np.linalg.norm(z) * (2.1e-5 + 2.0**-9), "pre")


def test_forward_equals_the_plain_product():
    """No activation, bias or residual: the same bits as the plain grouped product, fp32 and bf16."""
    rng = np.random.default_rng(4)
    m, n, k = 512, 384, 256
    q, s = mx.mx_quantize_dim0(dev_bf16(synth.normal_bf16(rng, (m, k), 1.0)))
    wq, ws = mx.mx_quantize_dim0(dev_bf16(synth.normal_bf16(rng, (2 * n, k), 0.05)))
    offs = dev_i32([96, 512])
    for dt in (F32, BF16):
        want = mx.mx_grouped_mm_fwd(q, s, wq, ws, offs, m, n, k, out_dtype=dt)
        got, _ = mx.mx_grouped_mm_fwd_epilogue(q, s, wq, ws, offs, m, n, k, out_dtype=dt)
        assert torch.equal(want, got)


def test_forward_special_values_and_aliasing(oracle):
    """Infinities and NaN in z stay where they are; out may be the residual."""
    m, n, k = 64, 64, 32
    rng = np.random.default_rng(5)
    a, b = synth.normal_bf16(rng, (m, k), 1.0), synth.normal_bf16(rng, (n, k), 0.2)
    bias = rng.standard_normal((1, n)).astype(np.float32)
    bias[0, 3], bias[0, 17], bias[0, 40] = np.inf, np.nan, -3e38
    res = dev_bf16(synth.normal_bf16(rng, (m, n), 1.0))
    for act in (NONE, RELU, SILU, GELU):
        want = res.float() + torch.from_numpy(act64_torch(a, b, bias, act, oracle)).to("cuda:0")
        got = res.clone()
        mx.mx_grouped_mm_bf16_fwd_epilogue(dev_bf16(a), dev_bf16(b), None, m, n, k, bias=torch.from_numpy(bias).to("cuda:0"),
                                           act=act, residual=got, out=got)
        fine = [c for c in range(n) if c not in (3, 17, 40)]
        w, g = host(want).astype(np.float64), val(oracle, got)
        check(g[:, fine], w[:, fine], 2.0**-8 * np.linalg.norm(w[:, fine]), f"act {act}")
        assert np.all(np.isposinf(g[:, 3]))
        assert np.all(np.isnan(g[:, 17]))
        if act in (RELU, SILU):
            check(g[:, [40]], host(res.float()).astype(np.float64)[:, [40]], 2.0**-8 * 8, "far below zero")


def act64_torch(a, b, bias, act, oracle):
    with np.errstate(all="ignore"):
        z = oracle.bf16_to_f64(a) @ oracle.bf16_to_f64(b).T + bias.astype(np.float64)
        z[:, [3, 17, 40]] = 0
        return act64(z, act).astype(np.float32)


# ---- backward --------------------------------------------------------------------------


def slope64(z, act):
    if act == RELU:
        return (z > 0).astype(np.float64)
    if act == GELU:
        c0, c1 = np.sqrt(2 / np.pi), 0.044715
        t = np.tanh(c0 * (z + c1 * z**3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c0 * (1 + 3 * c1 * z * z)
    if act == SILU:
        s = sigmoid(z)
        return s * (1 + z * (1 - s))
    return np.ones_like(z)


def backward64(dy, z, act):
    if act == SWIGLU:
        g, u = np.split(z, 2, axis=1)
        return np.concatenate([dy * u * slope64(g, SILU), dy * g * sigmoid(g)], axis=1)
    return dy * slope64(z, act)


BWD = [
    # m, n, group sizes, act
    (1, 1, None, GELU),
    (1, 2, None, SWIGLU),
    (3, 7, None, SILU),
    (70, 30, [30, 0, 33], SWIGLU),  # odd halves, an empty group, rows past the last
    (65, 8, [1, 64], RELU),
    (257, 72, [100, 100, 57], GELU),
    (1001, 576, None, GELU),
    (640, 1056, [0, 63, 65, 0, 512], SWIGLU),
    (512, 1040, None, NONE),
    (300, 64, [0, 0, 0], SILU),  # no rows in any group
    (2000, 16, [11] * 100, SILU),  # more groups than one wave scans
    (0, 64, [0, 0], SWIGLU),
]


@pytest.mark.parametrize("want_dbias", [True, False])
@pytest.mark.parametrize("m,n,sizes,act", BWD, ids=[f"{c[0]}-{c[1]}-act{c[3]}" for c in BWD])
def test_backward(oracle, m, n, sizes, act, want_dbias):
    rng = np.random.default_rng(m + n)
    n_out = n // 2 if act == SWIGLU else n
    dy_b, z_b = synth.normal_bf16(rng, (m, n_out), 1.0), synth.normal_bf16(rng, (m, n), 2.0)
    dy, z = oracle.bf16_to_f64(dy_b), oracle.bf16_to_f64(z_b)
    offs = None if sizes is None else np.cumsum(sizes)
    live = m if offs is None else int(offs[-1])
    ref = backward64(dy, z, act)
    ref[live:] = 0
    dpre = torch.full((m, n), 9.0, dtype=torch.bfloat16, device="cuda:0")
    say(f"[epilogue bwd] m={m} n={n} sizes={sizes and sizes[:8]} act={act}")
    got, dbias = mx.mx_epilogue_backward(dev_bf16(dy_b), dev_bf16(z_b), None if offs is None else dev_i32(offs), act,
                                         want_dbias=want_dbias, dpre=dpre)
    # fp32 slopes are good to about 1e-6 (1 + |z|), then one rounding to bf16
    weight = np.concatenate([dy, dy], axis=1) if act == SWIGLU else dy
    mag = np.abs(weight) * (1 + np.abs(z))
    if act == SWIGLU:
        mag = mag * (1 + np.abs(np.roll(z, n_out, axis=1)))
    g = val(oracle, got)
    assert np.all(np.abs(g - ref) <= 1.001 * half_ulp_bf16(ref) + 2e-6 * mag)
    assert np.all(g[live:] == 0)
    if not want_dbias:
        assert dbias is None
        return
    ends = [0, m] if offs is None else [0, *offs]
    for i in range(len(ends) - 1):
        s, e = ends[i], ends[i + 1]
        want, room = ref[s:e].sum(0), 4e-6 * mag[s:e].sum(0)
        d = host(dbias)[i].astype(np.float64)
        assert np.all(np.abs(d - want) <= room), i
        if s == e:
            assert np.all(d == 0)


@pytest.mark.parametrize("act", [GELU, SILU, SWIGLU])
def test_backward_against_differences(oracle, act):
    """dpre against central differences of the float64 forward (step 1e-5, error 1e-9)."""
    rng = np.random.default_rng(8)
    m, n = 9, 64
    n_out = n // 2 if act == SWIGLU else n
    dy_b, z_b = synth.normal_bf16(rng, (m, n_out), 1.0), synth.normal_bf16(rng, (m, n), 2.0)
    dy, z = oracle.bf16_to_f64(dy_b), oracle.bf16_to_f64(z_b)
    num = np.empty_like(z)
    for c in range(n):
        h = np.zeros(n)
        h[c] = 1e-5
        num[:, c] = ((act64(z + h, act) - act64(z - h, act)) * dy).sum(1) / 2e-5
    got, _ = mx.mx_epilogue_backward(dev_bf16(dy_b), dev_bf16(z_b), None, act)
    assert np.all(np.abs(val(oracle, got) - num) <= 1.001 * half_ulp_bf16(num) + 2e-5)


def test_backward_of_offs_out_of_contract():
    """Ends that fall or leave [0, m] are read clamped: no access outside, every row written."""
    m, n = 200, 64
    dy = torch.randn(m, n, device="cuda:0").bfloat16()
    z = torch.randn(m, n, device="cuda:0").bfloat16()
    offs = dev_i32([90, 40, 1000])
    got, dbias = mx.mx_epilogue_backward(dy, z, offs, SILU)
    want, wb = mx.mx_epilogue_backward(dy, z, dev_i32([90, 90, 200]), SILU)
    assert torch.equal(got, want) and torch.equal(dbias, wb)


def test_side_stream_and_graph():
    m, n, k = 96, 128, 64
    x, w = torch.randn(m, k, device="cuda:0").bfloat16(), torch.randn(n, k, device="cuda:0").bfloat16()
    dy = torch.randn(m, n // 2, device="cuda:0").bfloat16()

    def both():
        y, z = mx.mx_grouped_mm_bf16_fwd_epilogue(x, w, None, m, n, k, act=SWIGLU, save_pre=True)
        return (y, z, *mx.mx_epilogue_backward(dy, z, None, SWIGLU))

    want = both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = both()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        out = both()
    base = x.clone()
    for k2 in range(4):
        x.copy_(base * (1 + k2))
        now = both()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, now)), k2


def test_refusals():
    m, n, k = 64, 64, 64
    a = torch.zeros(m, k, dtype=torch.bfloat16, device="cuda:0")
    b = torch.zeros(n, k, dtype=torch.bfloat16, device="cuda:0")
    f = mx.mx_grouped_mm_bf16_fwd_epilogue
    with pytest.raises(mx.MXError, match="act"):
        f(a, b, None, m, n, k, act=9)
    with pytest.raises(mx.MXError, match="multiple of 64"):
        f(a, b, None, m, 32, k, act=SWIGLU)
    with pytest.raises(ValueError, match="bias"):
        f(a, b, None, m, n, k, bias=torch.zeros(n - 1, device="cuda:0"))
    with pytest.raises(TypeError, match="bias"):
        f(a, b, None, m, n, k, bias=torch.zeros(n, device="cuda:0", dtype=torch.bfloat16))
    with pytest.raises(TypeError, match="residual"):
        f(a, b, None, m, n, k, residual=torch.zeros(m, n, device="cuda:0"))
    with pytest.raises(ValueError, match="pre"):
        f(a, b, None, m, n, k, pre=torch.zeros(m, n - 1, device="cuda:0", dtype=torch.bfloat16))
    z = torch.zeros(m, n, dtype=torch.bfloat16, device="cuda:0")
    with pytest.raises(ValueError, match="columns"):
        mx.mx_epilogue_backward(z, z, None, SWIGLU)
    with pytest.raises(mx.MXError, match="act"):
        mx.mx_epilogue_backward(z, z, None, 7)
    with pytest.raises(mx.MXError, match="workspace"):
        mx.mx_epilogue_backward(z, z, None, SILU, workspace=None)
    with pytest.raises(ValueError, match="rows"):
        mx.mx_epilogue_backward(z[:3], z, None, SILU)


# ---- contractions that go round the chunk ring of the few-tile kernel --------------------
# Eight waves take 64-byte chunks in turn, so rows above 512 bytes give a wave a second chunk
# and above 1024 bytes reuse its first buffer. 32x64 tiles, 64x64 ones (129 to 256 tiles of 64x64)
# and 32x32 ones (rows above 4096 bytes); m and n that end 1 to 32 rows into a 64-wide tile,
# whose second band of scales is absent; contractions that end inside a chunk.
RING = [
    # kind, m, n, k, group sizes, act, bias, residual, pre, out
    ("mx", 40, 100, 4096, None, SILU, True, True, True, F32),
    ("mx", 84, 96, 1056, [32, 0, 32], NONE, True, True, False, BF16),
    ("mx", 33, 192, 4096, None, SWIGLU, True, True, True, BF16),
    ("mx", 96, 128, 2080, [32, 64], SWIGLU, False, False, True, F32),
    ("mx", 40, 72, 4128, None, GELU, True, True, True, BF16),
    ("mx", 65, 33, 4128, None, NONE, False, False, False, F32),
    ("mx", 96, 64, 4224, [64, 32], RELU, True, True, True, F32),
    ("mx", 84, 4116, 1056, None, NONE, True, True, True, F32),
    ("mx", 65, 4097, 544, None, GELU, True, True, True, BF16),
    ("mx", 20, 8288, 1120, None, SILU, False, False, False, F32),
    ("mx", 84, 4224, 1056, None, SWIGLU, True, True, True, BF16),
    ("mx", 96, 2080, 608, [32, 0, 64], SILU, True, False, True, F32),
    ("bf16", 40, 100, 2048, None, SILU, True, True, True, F32),
    ("bf16", 90, 192, 1032, [1, 0, 80], SWIGLU, True, True, True, BF16),
    ("bf16", 40, 72, 2056, None, GELU, True, True, True, F32),
    ("bf16", 50, 40, 2184, [17, 30], NONE, True, False, True, BF16),
    ("bf16", 84, 4116, 552, None, RELU, True, True, True, F32),
    ("bf16", 84, 4224, 600, None, SWIGLU, True, True, True, F32),
]


@pytest.mark.parametrize("case", RING, ids=["-".join(map(str, c[:4])) + f"-act{c[5]}" for c in RING])
def test_forward_long_contractions(oracle, case):
    test_forward(oracle, case)


@pytest.mark.parametrize("kind,m,n,k,act", [("mx", 84, 4116, 1056, NONE), ("mx", 40, 72, 4128, NONE),
                                            ("mx", 33, 192, 4096, SWIGLU), ("bf16", 84, 4116, 552, NONE)])
def test_forward_long_contractions_same_bits(kind, m, n, k, act):
    """Operands from memory and from the caches: the same bits however long the loads take."""
    a = torch.randn(m, k, device="cuda:0").bfloat16()
    b = (torch.randn(n, k, device="cuda:0") * k**-0.5).bfloat16()
    ops = (a, b) if kind == "bf16" else (*mx.mx_quantize_dim0(a), *mx.mx_quantize_dim0(b))
    f = mx.mx_grouped_mm_bf16_fwd_epilogue if kind == "bf16" else mx.mx_grouped_mm_fwd_epilogue
    want = f(*ops, None, m, n, k, act=act, out_dtype=F32)[0]
    flush = torch.empty(1 << 29, dtype=torch.uint8, device="cuda:0")  # larger than every cache
    for i in range(6):
        if i % 2:
            flush.fill_(i)
        assert torch.equal(f(*ops, None, m, n, k, act=act, out_dtype=F32)[0], want), i


def test_backward_relu_keeps_what_is_cut_off_out():
    """ReLU's gradient is a choice, dy or 0: an infinite or NaN dy where z <= 0 reaches neither
    dpre nor dbias, and where z > 0 it passes."""
    m, n = 70, 72
    z = torch.randn(m, n, device="cuda:0").bfloat16()
    dy = torch.randn(m, n, device="cuda:0").bfloat16()
    z[:, :4] = -z[:, :4].abs() - 0.5
    z[3, 2], z[4, 3] = 0.0, -0.0
    dy[1, 0], dy[2, 1], dy[3, 2], dy[4, 3] = float("inf"), float("nan"), float("-inf"), float("nan")
    z[5, 8], dy[5, 8] = 1.5, float("inf")
    got, dbias = mx.mx_epilogue_backward(dy, z, dev_i32([40, 70]), RELU)
    assert torch.equal(got, torch.where(z > 0, dy, torch.zeros_like(dy)))
    assert torch.all(dbias[:, :4] == 0)
    assert dbias[0, 8] == float("inf") and torch.isfinite(dbias[1]).all()
    assert torch.isfinite(dbias[:, 9:]).all()


@pytest.mark.parametrize("act", [GELU, SILU, SWIGLU])
def test_backward_of_large_values(oracle, act):
    """Finite z, dy and gradients far beyond where the activations saturate: slopes 0 and 1."""
    far = np.array([-3e38, -1e30, -2e19, -1e10, -3e4, -200, 200, 3e4, 1e10, 2e19, 1e30, 3e38, 0.0, 1.0, -1.0, 4.0])
    rows = np.array([1.0, -2.5, 1e-20, 1e30])
    z_t = torch.from_numpy(np.tile(far, (4, 1)).astype(np.float32)).bfloat16()
    dy_t = torch.from_numpy(np.tile(rows[:, None], (1, 16)).astype(np.float32)).bfloat16()
    if act == SWIGLU:  # up values that overflow with dy before the gate's slope makes them small
        up = np.where(far < -100, 1e25, 0.5)
        z_t = torch.cat([z_t, torch.from_numpy(np.tile(up, (4, 1)).astype(np.float32)).bfloat16()], 1)
    z, dy = z_t.double().numpy(), dy_t.double().numpy()
    with np.errstate(over="ignore"):
        ref = backward64(dy, z, act)
    got, dbias = mx.mx_epilogue_backward(dy_t.to("cuda:0"), z_t.to("cuda:0"), None, act)
    g = val(oracle, got)
    big = np.abs(ref) > 3.38e38  # beyond bf16: an infinity of the right sign
    assert np.all(np.isinf(g[big]) & (np.sign(g[big]) == np.sign(ref[big])))
    ok = ~big
    # slopes of these z are 0, 1 or moderate: fp32 errors of a few 1e-6, then the rounding; a sigmoid
    # below fp32's smallest normal number, 2^-126, counts as 0 (e^-200 beside dy u = 1e55)
    weight = np.abs(np.concatenate([dy, dy], 1) if act == SWIGLU else dy) * (1 + np.abs(z))
    if act == SWIGLU:
        weight[:, :16] *= np.abs(z[:, 16:])
    assert np.all(np.abs(g[ok] - ref[ok]) <=
                  1.001 * half_ulp_bf16(ref[ok]) + 1e-5 * np.abs(ref[ok]) + 2.0**-126 * weight[ok])
    assert torch.isfinite(dbias[0]).cpu().numpy()[~big.any(0)].all()


# ---- large products and gradients ----------------------------------------------------------
LARGE = [
    # two rounds of 256x256 tiles and a short one, whose tiles run as quarters
    ("mx", 8448, 4096, 1056, [4128, 0, 4320], SWIGLU, True, True, True, BF16),
    ("mx", 8448, 4096, 1056, [4128, 0, 4320], SILU, True, True, False, BF16),
    ("bf16", 8448, 4104, 1032, [1, 4200, 4247], GELU, True, True, True, BF16),
]


@pytest.mark.parametrize("case", LARGE, ids=["-".join(map(str, c[:4])) + f"-act{c[5]}" for c in LARGE])
def test_forward_short_last_round(oracle, case):
    test_forward(oracle, case)


@pytest.mark.parametrize("m,n,sizes,act", [(16384, 1040, [4096, 0, 33, 8000, 4000], SWIGLU),
                                           (16384, 1032, None, GELU), (4001, 1041, [1, 4000], SILU),
                                           (6000, 2002, None, SWIGLU)])
def test_backward_64_row_tiles(oracle, m, n, sizes, act):
    test_backward(oracle, m, n, sizes, act, True)


@pytest.mark.parametrize("kind,m,n,k,act", [("mx", 96, 128, 1056, SWIGLU), ("mx", 40, 72, 4128, SILU),
                                            ("bf16", 1024, 2304, 128, GELU), ("mx", 4096, 4160, 1056, SWIGLU)])
def test_a_row_of_nan_stays_alone(oracle, kind, m, n, k, act):
    """NaN in one row of A reaches that row of out and z alone, also across a tile's rows."""
    a = torch.randn(m, k, device="cuda:0").bfloat16()
    b = (torch.randn(n, k, device="cuda:0") * k**-0.5).bfloat16()
    ops = [a, b] if kind == "bf16" else [*mx.mx_quantize_dim0(a), *mx.mx_quantize_dim0(b)]
    f = mx.mx_grouped_mm_bf16_fwd_epilogue if kind == "bf16" else mx.mx_grouped_mm_fwd_epilogue
    want, z = f(*ops, None, m, n, k, act=act, save_pre=True)
    bad = ops[0].clone()
    bad.view(m, k)[m // 2] = float("nan") if kind == "bf16" else 0x7F  # 0x7F: the NaN code
    got, z2 = f(bad, *ops[1:], None, m, n, k, act=act, save_pre=True)
    rest = torch.arange(m, device="cuda:0") != m // 2
    assert torch.equal(got[rest], want[rest]) and torch.equal(z2[rest], z[rest])
    assert torch.isnan(got[m // 2]).all() and torch.isnan(z2[m // 2]).all()


# ---- many groups, no rows, ends out of contract ---------------------------------------------
MANY = [
    ("mx", 3264, 64, 64, [32, 0, 32, 64] * 25, SILU, True, True, True, BF16),  # 64x64 tiles
    ("mx", 9600, 128, 96, [0, 96, 0] * 100, SWIGLU, True, True, True, BF16),  # 128x128 tiles
    ("bf16", 700, 40, 72, [0, 1, 2, 11] * 50, GELU, True, True, True, F32),
]


@pytest.mark.parametrize("case", MANY, ids=["-".join(map(str, c[:4])) + f"-act{c[5]}" for c in MANY])
def test_forward_many_groups(oracle, case):
    test_forward(oracle, case)


@pytest.mark.parametrize("act", [NONE, SWIGLU])
def test_forward_without_rows(act):
    n, k, G = 128, 96, 3
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda:0")  # noqa: E731
    w = mx.mx_quantize_dim0(bf(G * n, k))
    none, s = (torch.zeros(v, dtype=torch.uint8, device="cuda:0") for v in ((0, k), 0))
    shape = (0, n // 2 if act == SWIGLU else n)
    for out, z in (mx.mx_grouped_mm_fwd_epilogue(none, s, *w, dev_i32([0] * G), 0, n, k, act=act, save_pre=True),
                   mx.mx_grouped_mm_bf16_fwd_epilogue(bf(0, k), bf(G * n, k), dev_i32([0] * G), 0, n, k, act=act, save_pre=True),
                   mx.mx_grouped_mm_bf16_fwd_epilogue(bf(0, k), bf(n, k), None, 0, n, k, act=act, save_pre=True)):
        assert out.shape == shape and z.shape == (0, n)
    torch.cuda.synchronize()


@pytest.mark.parametrize("kind", ["mx", "bf16"])
@pytest.mark.parametrize("m,n,k", [(192, 64, 1056), (4096, 2304, 96)])
def test_forward_of_offs_out_of_contract(kind, m, n, k):
    """Ends that fall or leave [0, m] are read clamped: the rows of a valid reading, no others."""
    a = torch.randn(m, k, device="cuda:0").bfloat16()
    b = (torch.randn(3 * n, k, device="cuda:0") * 0.1).bfloat16()
    ops = (a, b) if kind == "bf16" else (*mx.mx_quantize_dim0(a), *mx.mx_quantize_dim0(b))
    f = mx.mx_grouped_mm_bf16_fwd_epilogue if kind == "bf16" else mx.mx_grouped_mm_fwd_epilogue
    got, _ = f(*ops, dev_i32([96, 32, 1 << 30]), m, n, k, act=SILU)
    want, _ = f(*ops, dev_i32([96, 96, m]), m, n, k, act=SILU)
    assert torch.equal(got, want)
    out = torch.full((m, n), 7.0, dtype=torch.bfloat16, device="cuda:0")
    f(*ops, dev_i32([-5, 96, 64]), m, n, k, act=SILU, out=out)
    assert torch.all(out[96:] == 7.0) and torch.isfinite(out[:96]).all()
