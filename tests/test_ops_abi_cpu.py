"""Host-side validation of the expert-layer operators: refused arguments return their status
before any device access (valid ones reach the device check, or run where there is a GPU)."""

import ctypes

import pytest

from mxfp8_block_scaled_amd import _lib

MX_E_NULL, MX_E_SHAPE, MX_E_ALIGN, MX_E_LAYOUT, MX_E_DTYPE, MX_E_DEVICE = -1, -2, -3, -4, -5, -6
P, P2 = 0x10000, 0x20000  # aligned addresses, never dereferenced by a refused call


@pytest.fixture(scope="module")
def lib():
    import torch

    if torch.cuda.is_available():
        pytest.skip("made-up addresses: for a machine without a GPU")
    return _lib.load()


def test_epilogue_forward(lib):
    f = lib.mx_grouped_mm_fwd_epilogue

    def call(offs=P2, offs_out=None, groups=3, m=96, m_out=96, n=64, k=64, bias=P, act=3, res=P, pre=P, out=P, dt=1):
        return f(P, P, P, P, offs, offs_out, groups, m, m_out, n, k, bias, act, res, pre, out, dt, None)

    assert call() == MX_E_DEVICE
    assert call(act=4) == MX_E_DEVICE
    assert call(act=5) == MX_E_DTYPE and call(act=-1) == MX_E_DTYPE and call(dt=2) == MX_E_DTYPE
    assert call(act=4, n=32) == MX_E_SHAPE and call(n=40) == MX_E_SHAPE and call(k=40) == MX_E_SHAPE
    assert call(m_out=64) == MX_E_SHAPE and call(offs_out=P2, m_out=128) == MX_E_SHAPE
    assert call(offs_out=P2, m_out=64) == MX_E_DEVICE
    assert call(offs=None, offs_out=P2, groups=1) == MX_E_NULL and call(offs=None) == MX_E_SHAPE
    assert call(bias=P + 4) == MX_E_ALIGN and call(res=P + 8) == MX_E_ALIGN and call(pre=P + 2) == MX_E_ALIGN
    assert call(out=None) == MX_E_NULL and call(offs_out=P2 + 1, m_out=64) == MX_E_ALIGN
    assert call(n=(1 << 21) + 32, k=32) == MX_E_SHAPE  # residual limit
    assert call(n=(1 << 21) + 64, k=2048, act=4, res=None, pre=None) == MX_E_SHAPE  # one weight of 2^31 bytes and more


def test_epilogue_forward_bf16(lib):
    f = lib.mx_grouped_mm_bf16_fwd_epilogue

    def call(offs=P2, groups=3, m=100, n=36, k=64, bias=P, act=1, out=P):
        return f(P, P, offs, groups, m, n, k, bias, act, None, None, out, 0, None)

    assert call() == MX_E_DEVICE
    assert call(k=60) == MX_E_SHAPE and call(n=37) == MX_E_DEVICE
    assert call(act=4) == MX_E_SHAPE and call(k=(1 << 21) + 8) == MX_E_SHAPE and call(out=None) == MX_E_NULL


def test_epilogue_backward(lib):
    f = lib.mx_epilogue_backward
    need = lib.mx_epilogue_backward_workspace_bytes

    def call(dy=P, pre=P, offs=P2, groups=3, m=100, n=36, act=1, dpre=P, dbias=P, ws=P, nb=1 << 20):
        return f(dy, pre, offs, groups, m, n, act, dpre, dbias, ws, nb, None)

    assert call() == MX_E_DEVICE
    assert call(act=7) == MX_E_DTYPE and call(act=4, n=37) == MX_E_SHAPE
    assert call(groups=0) == MX_E_SHAPE and call(offs=None) == MX_E_SHAPE
    assert call(pre=None) == MX_E_NULL and call(dpre=None) == MX_E_NULL and call(dy=None) == MX_E_NULL
    assert call(act=0, pre=None, dpre=None) == MX_E_DEVICE
    assert call(nb=need(3, 1, 100, 36, 1)) == MX_E_DEVICE and call(nb=need(3, 1, 100, 36, 1) - 1) == MX_E_SHAPE
    assert call(ws=None, nb=0) == MX_E_SHAPE and call(ws=None, nb=0, dbias=None) == MX_E_DEVICE
    assert call(dbias=P + 4) == MX_E_ALIGN and call(dy=P + 2) == MX_E_ALIGN and call(offs=P2 + 2) == MX_E_ALIGN
    assert need(0, 1, 10, 8, 1) == -1 and need(2, 0, 10, 8, 1) == -1 and need(1, 0, 10, 9, 4) == -1
    assert need(1, 0, 0, 8, 1) == 0


def test_moe_layer(lib):
    f = lib.mx_moe_layer
    need = lib.mx_moe_layer_workspace_bytes

    def call(x=P, ld=64, logits=P, ldl=8, T=5, H=64, F=32, E=8, first=2, local=4, topk=2, score=0, scale=1.0, w1=P,
             w1_s=P, res=P, out=P, dt=1, ids=P, wts=P, ws=P, nb=None):
        return f(x, ld, logits, ldl, T, H, F, E, first, local, topk, score, 1, scale, w1, w1_s, P, P, res, out, dt, ids,
                 wts, ws, need(T, H, F, topk) if nb is None else nb, None)

    assert call() == MX_E_DEVICE and call(T=17) == MX_E_DEVICE and call(T=256) == MX_E_DEVICE
    assert call(T=257, nb=1 << 40) == MX_E_SHAPE and call(T=-1, nb=1 << 40) == MX_E_SHAPE
    assert call(H=48) == MX_E_SHAPE and call(F=40) == MX_E_SHAPE and call(E=1025, ldl=1025) == MX_E_SHAPE
    assert call(topk=9) == MX_E_SHAPE and call(topk=0, nb=1 << 20) == MX_E_SHAPE and call(first=5) == MX_E_SHAPE
    assert call(first=-1) == MX_E_SHAPE and call(local=0) == MX_E_SHAPE
    assert call(score=2) == MX_E_DTYPE and call(dt=3) == MX_E_DTYPE
    assert call(scale=0.0) == MX_E_SHAPE and call(scale=float("inf")) == MX_E_SHAPE
    assert call(ld=56) == MX_E_LAYOUT and call(ld=68) == MX_E_ALIGN and call(ldl=7) == MX_E_LAYOUT
    assert call(x=None) == MX_E_NULL and call(logits=None) == MX_E_NULL and call(ids=None) == MX_E_NULL
    assert call(w1_s=None) == MX_E_NULL and call(logits=P + 2) == MX_E_ALIGN and call(w1=P + 8) == MX_E_ALIGN
    assert call(nb=need(5, 64, 32, 2) - 1) == MX_E_SHAPE and call(ws=None) == MX_E_NULL
    assert call(x=None, logits=None, out=None, ids=None, wts=None, ws=None, T=0) == MX_E_DEVICE
    assert call(ld=1 << 28, T=8) == MX_E_SHAPE  # rows 2^31 elements apart
    assert call(H=1 << 16, F=1 << 15, ld=1 << 16) == MX_E_SHAPE  # one expert of 2^32 bytes
    assert need(1, 64, 33, 2) == -1 and need(1, 48, 32, 2) == -1 and need(0, 64, 32, 2) == 0


def test_orthogonalize(lib):
    f = lib.mx_orthogonalize
    need = lib.mx_orthogonalize_workspace_bytes

    def call(g=P, dt=0, m=P, mo=P, mu=0.9, batch=2, rows=40, cols=24, steps=2, coefs=(1.0, -1.0, 0.5) * 2, eps=1e-7,
             out=P, ws=P, nb=1 << 30):
        c = None if coefs is None else ctypes.cast((ctypes.c_float * 256)(*coefs), ctypes.c_void_p)
        return f(g, dt, m, mo, mu, 1, batch, rows, cols, steps, c, eps, out, ws, nb, None)

    assert call() == MX_E_DEVICE and call(m=None, mo=None, mu=float("nan")) == MX_E_DEVICE
    assert call(dt=2) == MX_E_DTYPE
    assert call(batch=0) == MX_E_SHAPE and call(rows=0) == MX_E_SHAPE and call(cols=65537) == MX_E_SHAPE
    assert call(steps=0) == MX_E_SHAPE and call(steps=65) == MX_E_SHAPE
    assert call(m=None) == MX_E_NULL and call(mo=None) == MX_E_NULL and call(coefs=None) == MX_E_NULL
    assert call(g=None) == MX_E_NULL and call(out=P + 8) == MX_E_ALIGN and call(m=P + 4) == MX_E_ALIGN
    assert call(mu=float("inf")) == MX_E_SHAPE and call(eps=-1.0) == MX_E_SHAPE and call(eps=float("nan")) == MX_E_SHAPE
    assert call(coefs=(1.0, 17.0, 0.0) * 2) == MX_E_SHAPE and call(coefs=(float("nan"), 0.0, 0.0) * 2) == MX_E_SHAPE
    assert call(nb=need(2, 40, 24)) == MX_E_DEVICE and call(nb=need(2, 40, 24) - 1) == MX_E_SHAPE
    assert call(ws=None) == MX_E_SHAPE and need(1, 0, 8) == -1 and need(65536, 8, 8) == -1


def test_moe_layer_forms_no_sum_by_atomics():
    """The header's promise: the layer's kernels have no atomic operation on floats (the integer
    ones build lists and bitmaps in LDS)."""
    import os
    import re

    path = os.path.join(os.path.dirname(_lib.LIB_PATH), "csrc", "moe.hip")
    with open(path) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    assert "unsafeAtomicAdd" not in code and "atomic_fadd" not in code
    assert set(re.findall(r"atomic\w*\((&?\w+)", code)) <= {"&bits", "&n_list", "&cnt"}
