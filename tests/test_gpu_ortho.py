"""Newton-Schulz orthogonalisation against the same iteration in float64 on the CPU.

Tolerance: the products round X, O and P to fp16 (2^-12 of a value at most), which reaches
the result without amplification by small singular values; the float32-and-fp16 arithmetic
written out on the CPU (512 x 2048 and smaller; Gaussian, low-rank, exponentially decaying,
rank-1 and single-spike inputs) was 0.2e-3 to 1.7e-3 off from 32 rows up, 3.1e-3 for rank 1
at 64 rows. The result is held to 4e-3 in the Frobenius norm, with its bf16 rounding (2^-9).
The momentum is elementwise: two float32 roundings.
"""

import numpy as np
import pytest
import torch

import mxfp8_block_scaled_amd as mx

from gpu_util import host, require_gpu, say

pytestmark = pytest.mark.gpu

TOL = 4e-3
MUON = (3.4445, -4.7750, 2.0315)


@pytest.fixture(scope="module", autouse=True)
def gpu():
    require_gpu()


def newton_schulz(u, steps=5, coefs=MUON, eps=1e-7):
    x = u / (np.linalg.norm(u) + eps)
    tall = u.shape[0] > u.shape[1]
    x = x.T if tall else x
    for i in range(steps):
        a, b, c = coefs if np.isscalar(coefs[0]) else coefs[i]
        p = x @ x.T
        x = a * x + (b * p + c * (p @ p)) @ x
    return x.T if tall else x


def matrix(rng, kind, rows, cols):
    r = min(rows, cols)
    if kind == "gauss":
        return rng.standard_normal((rows, cols))
    if kind == "lowrank":
        k = max(1, r // 16)
        return rng.standard_normal((rows, k)) @ rng.standard_normal((k, cols)) + 0.1 * rng.standard_normal((rows, cols))
    if kind == "decay":
        u = np.linalg.qr(rng.standard_normal((rows, r)))[0]
        v = np.linalg.qr(rng.standard_normal((cols, r)))[0]
        return (u * np.exp(-12 * np.arange(r) / r)) @ v.T
    if kind == "rank1":
        return rng.standard_normal((rows, 1)) @ rng.standard_normal((1, cols))
    return 1e-4 * rng.standard_normal((rows, cols)) + np.eye(rows, cols) * (np.arange(cols) == 0)  # spike


def val(t):
    h = t.float()
    return host(h).astype(np.float64)


def check(got, ref, name):
    err = np.linalg.norm(got - ref) / max(np.linalg.norm(ref), 1e-300)
    say(f"[ortho] {name}: rel {err:.2e}")
    assert np.isfinite(got).all() and err <= TOL, (name, err)


CASES = [
    # batch, rows, cols, kind, dtype
    (1, 1, 1, "gauss", torch.float32),
    (1, 1, 40, "gauss", torch.float32),
    (2, 40, 1, "gauss", torch.bfloat16),
    (1, 2, 3, "gauss", torch.float32),
    (3, 33, 65, "gauss", torch.float32),
    (1, 65, 33, "lowrank", torch.bfloat16),
    (1, 128, 128, "gauss", torch.float32),
    (2, 131, 250, "decay", torch.float32),
    (1, 256, 256, "rank1", torch.float32),
    (1, 576, 1000, "lowrank", torch.bfloat16),
    (1, 1000, 576, "gauss", torch.float32),
    (8, 264, 300, "gauss", torch.float32),
    (1, 300, 2052, "spike", torch.float32),
    (1, 17, 4100, "gauss", torch.float32),
    (12, 1040, 1028, "gauss", torch.bfloat16),  # 256x256 tiles in every product, ragged edges
    (13, 1028, 1040, "lowrank", torch.float32),
]


@pytest.mark.parametrize("case", CASES, ids=["-".join(map(str, c[:4])) for c in CASES])
def test_matches_float64(case):
    batch, rows, cols, kind, dtype = case
    rng = np.random.default_rng(rows * 7 + cols)
    g = torch.from_numpy(np.stack([matrix(rng, kind, rows, cols) for _ in range(batch)]).astype(np.float32) * 1e-3)
    g = g.to(dtype)
    say(f"[ortho] {case}")
    out, m = mx.mx_orthogonalize(g.to("cuda:0"))
    assert m is None and out.dtype == torch.bfloat16 and out.shape == g.shape
    got = val(out)
    for i in sorted({0, batch // 2, batch - 1}):
        check(got[i], newton_schulz(g[i].double().numpy()), f"{case} [{i}]")


@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("rows,cols,dtype", [(96, 160, torch.float32), (67, 35, torch.bfloat16)])
def test_momentum(rows, cols, dtype, nesterov):
    rng = np.random.default_rng(4)
    g = torch.from_numpy(rng.standard_normal((2, rows, cols)).astype(np.float32)).to(dtype)
    m = torch.from_numpy(rng.standard_normal((2, rows, cols)).astype(np.float32))
    mu = 0.9
    dm = m.to("cuda:0")
    out, new = mx.mx_orthogonalize(g.to("cuda:0"), momentum=dm, mu=mu, nesterov=nesterov)
    assert torch.equal(dm.cpu(), m)  # not in place unless asked
    want = np.float32(mu).astype(np.float64) * m.double().numpy() + g.double().numpy()
    assert np.all(np.abs(host(new) - want) <= 2.0**-22 * (np.abs(want) + np.abs(m.numpy())))
    u = g.double().numpy() + np.float32(mu).astype(np.float64) * want if nesterov else want
    for i in range(2):
        check(val(out)[i], newton_schulz(u[i]), f"momentum {i}")
    again, same = mx.mx_orthogonalize(g.to("cuda:0"), momentum=dm, mu=mu, nesterov=nesterov, momentum_out=dm)
    assert same is dm and torch.equal(dm, new) and torch.equal(again, out)


def test_coefficients_and_steps():
    """Steps with coefficients of their own, one step, and a schedule that converges to the polar factor."""
    rng = np.random.default_rng(6)
    g = torch.from_numpy(rng.standard_normal((48, 80)).astype(np.float32))
    d = g.to("cuda:0")
    check(val(mx.mx_orthogonalize(d, steps=1)[0]), newton_schulz(g.double().numpy(), steps=1), "one step")
    per = [(4.0, -6.0, 3.0), (3.0, -4.0, 2.0), (1.875, -1.25, 0.375)]
    check(val(mx.mx_orthogonalize(d, steps=3, coefs=per)[0]), newton_schulz(g.double().numpy(), 3, per), "own steps")
    u, _, vt = np.linalg.svd(g.double().numpy(), full_matrices=False)
    check(val(mx.mx_orthogonalize(d, steps=14, coefs=(1.875, -1.25, 0.375))[0]), u @ vt, "polar factor")


def test_scale_zero_and_special_values():
    rng = np.random.default_rng(7)
    g = torch.from_numpy(rng.standard_normal((6, 72, 40)).astype(np.float32))
    base = g[0].clone()
    g[1] = base * 1e-30  # far below eps: X stays small
    g[2] = base * 1e30  # squares beyond float32
    g[3] = 0
    g[4, 5, 7] = float("inf")
    g[5, 1, 1] = float("nan")
    out = val_any(mx.mx_orthogonalize(g.to("cuda:0"))[0])
    check(out[0], newton_schulz(base.double().numpy()), "plain")
    tiny = newton_schulz(g[1].double().numpy())
    assert np.linalg.norm(out[1] - tiny) <= 1e-2 * np.linalg.norm(tiny) + 1e-30
    check(out[2], newton_schulz(g[2].double().numpy()), "huge")
    assert np.all(out[3] == 0)
    assert np.all(np.isnan(out[4])) and np.all(np.isnan(out[5]))
    only_eps = mx.mx_orthogonalize((base * 1e-30).to("cuda:0"), eps=0.0)[0]
    check(val(only_eps), newton_schulz(base.double().numpy()), "no eps")


def val_any(t):
    return host(t.float()).astype(np.float64)


def test_same_bits_side_stream_and_graph():
    g = torch.randn(2, 192, 320, device="cuda:0")
    m = torch.randn(2, 192, 320, device="cuda:0")
    want = mx.mx_orthogonalize(g, momentum=m)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(mx.mx_orthogonalize(g, momentum=m), want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = mx.mx_orthogonalize(g, momentum=m)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    base = g.clone()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = mx.mx_orthogonalize(g, momentum=m)
    for k in range(4):
        g.copy_(base + k * m)
        now = mx.mx_orthogonalize(g, momentum=m)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, now)), k


def test_refusals():
    g = torch.zeros(32, 48, device="cuda:0")
    f = mx.mx_orthogonalize
    with pytest.raises(mx.MXError, match="steps"):
        f(g, steps=0, coefs=())
    with pytest.raises(mx.MXError, match="coefs"):
        f(g, coefs=(1.0, float("nan"), 0.0))
    with pytest.raises(ValueError, match="coefs"):
        f(g, coefs=[(1.0, 0.0, 0.0)] * 2)
    with pytest.raises(mx.MXError, match="eps"):
        f(g, eps=-1.0)
    with pytest.raises(mx.MXError, match="workspace"):
        f(g, workspace=torch.empty(64, dtype=torch.uint8, device="cuda:0"))
    with pytest.raises(TypeError, match="g has dtype"):
        f(g.half())
    with pytest.raises(ValueError, match="contiguous"):
        f(g.t())
    with pytest.raises(ValueError, match="momentum"):
        f(g, momentum=g[:16])
    with pytest.raises(ValueError, match="momentum_out"):
        f(g, momentum_out=g)
    with pytest.raises(ValueError):
        f(torch.zeros(0, 8, device="cuda:0"))
    with pytest.raises(ValueError, match="GPU memory"):
        f(torch.zeros(8, 8))
    assert mx.mx_orthogonalize_workspace_bytes(1, 65536, 8) > 0
    with pytest.raises(ValueError):
        mx.mx_orthogonalize_workspace_bytes(1, 65537, 8)


def test_norms_at_the_limits_of_float32():
    """eps = 0: a zero matrix gives zeros; norms below and above float32's range are norms like others."""
    rng = np.random.default_rng(9)
    base = torch.from_numpy(rng.standard_normal((72, 40)).astype(np.float32))
    g = torch.stack([torch.zeros(72, 40), base * 1e-41, base.clamp(-2, 2) * 1.7e38, base, base * 1e-36])
    assert torch.isfinite(g).all() and g[2].double().norm() > 3.4e38
    for eps in (0.0, 1e-42):
        out = val(mx.mx_orthogonalize(g.to("cuda:0"), eps=eps)[0])
        assert np.all(out[0] == 0)
        for i in range(1, 5):
            check(out[i], newton_schulz(g[i].double().numpy(), eps=eps), f"eps {eps} [{i}]")
    assert np.all(val(mx.mx_orthogonalize(torch.zeros(300, 200, device="cuda:0"), eps=0.0)[0]) == 0)
    # with momentum: the update's norm counts, not the gradient's
    m = torch.from_numpy(rng.standard_normal((5, 72, 40)).astype(np.float32))
    m[0] = 0
    out, new = mx.mx_orthogonalize(torch.zeros_like(g).to("cuda:0"), momentum=m.to("cuda:0"), mu=0.5, eps=0.0)
    assert np.all(val(out)[0] == 0) and torch.equal(new.cpu(), 0.5 * m)
    check(val(out)[1], newton_schulz(0.25 * m[1].double().numpy(), eps=0.0), "momentum alone")


# 128x128 tiles in the step product (the sizes between one round of 64x64 tiles and 192 of
# 256x256): a batch, a ragged one, a tall one
MIDDLE = [
    (8, 512, 512, "gauss", torch.float32),
    (1, 2048, 2040, "lowrank", torch.bfloat16),
    (3, 700, 1410, "decay", torch.float32),
    (2, 1801, 640, "gauss", torch.bfloat16),
]


@pytest.mark.parametrize("case", MIDDLE, ids=["-".join(map(str, c[:4])) for c in MIDDLE])
def test_128_tiles(case):
    test_matches_float64(case)


def test_a_matrix_of_nan_stays_alone_in_128_tiles():
    g = torch.randn(8, 520, 500, device="cuda:0")
    want = mx.mx_orthogonalize(g)[0]
    bad = g.clone()
    bad[3, 100, 100] = float("nan")
    bad[5, 0, 499] = float("inf")
    got = mx.mx_orthogonalize(bad)[0]
    rest = [0, 1, 2, 4, 6, 7]
    assert torch.equal(got[rest], want[rest])
    assert torch.isnan(got[3]).all() and torch.isnan(got[5]).all()
    again = mx.mx_orthogonalize(g)[0]
    assert torch.equal(again, want)
