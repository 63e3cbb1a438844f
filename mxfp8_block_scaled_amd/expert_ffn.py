"""The SwiGLU feed-forward of a mixture-of-experts layer, forward and backward, composed from
the library's calls: MXFP8 casts, grouped products with their epilogues, and the backward of
those epilogues. The same weights serve `mx_moe_layer` for a few tokens at a time.

  z = x W1_e^T + b1_e (gate, then up columns),  h = silu(z_gate) z_up,
  y = h W2_e^T + b2_e (+ residual)               for the rows of expert e

x [M, K] bf16 in groups of rows by `offs` (int32 ends, multiples of 32); W1 [E, 2F, K] and
W2 [E, K, F]. Rows past the last end belong to no expert: those of y and dx are left unwritten, and
they enter no other result. Every step runs in the library's kernels; this module only orders the calls.
"""

from . import (MX_ACT_NONE, MX_ACT_SWIGLU, MX_OUT_F32, mx_epilogue_backward, mx_grouped_mm_dgrad,
               mx_grouped_mm_fwd_epilogue, mx_grouped_mm_wgrad, mx_quantize_dim0_dim1)


class ExpertWeights:
    """The casts of bf16 weights w1 [E, 2F, K] and w2 [E, K, F]: rowwise codes and scales
    (`w1`, `w2`: forward and decoding) and transposed ones (`w1_t`, `w2_t`: dgrad)."""

    def __init__(self, w1, w2):
        self.experts, two_f, self.hidden = w1.shape
        self.ffn = two_f // 2
        if w2.shape != (self.experts, self.hidden, self.ffn):
            raise ValueError(f"w2 has shape {tuple(w2.shape)}; w1 asks for {(self.experts, self.hidden, self.ffn)}")
        q, s, q_t, s_t = mx_quantize_dim0_dim1(w1)
        self.w1, self.w1_t = (q, s), (q_t, s_t)
        q, s, q_t, s_t = mx_quantize_dim0_dim1(w2)
        self.w2, self.w2_t = (q, s), (q_t, s_t)


def forward(x, offs, w, b1=None, b2=None, residual=None):
    """(y [M, K] bf16, saved): b1 [E, 2F] and b2 [E, K] float32, residual [M, K] bf16."""
    m, k = x.shape
    xq, xs, xtq, xts = mx_quantize_dim0_dim1(x, stream_t=True)
    h, z = mx_grouped_mm_fwd_epilogue(xq, xs, *w.w1, offs, m, 2 * w.ffn, k, bias=b1, act=MX_ACT_SWIGLU, save_pre=True)
    hq, hs, htq, hts = mx_quantize_dim0_dim1(h, stream_t=True)
    y, _ = mx_grouped_mm_fwd_epilogue(hq, hs, *w.w2, offs, m, k, w.ffn, bias=b2, residual=residual)
    return y, (xtq, xts, z, htq, hts)


def backward(dy, offs, w, saved, dw_dtype=MX_OUT_F32, bias=False):
    """(dx [M, K], dw1 [E, 2F, K], dw2 [E, K, F], db1 [E, 2F], db2 [E, K]) for dy [M, K] bf16;
    the bias gradients are None unless `bias`. The residual's gradient is dy."""
    m, k = dy.shape
    xtq, xts, z, htq, hts = saved
    db2 = mx_epilogue_backward(dy, None, offs, MX_ACT_NONE)[1] if bias else None
    dyq, dys, dytq, dyts = mx_quantize_dim0_dim1(dy)
    dh = mx_grouped_mm_dgrad(dyq, dys, *w.w2_t, offs, m, k, w.ffn)
    dw2 = mx_grouped_mm_wgrad(dytq, dyts, htq, hts, offs, m, k, w.ffn, out_dtype=dw_dtype)
    dz, db1 = mx_epilogue_backward(dh, z, offs, MX_ACT_SWIGLU, want_dbias=bias)
    dzq, dzs, dztq, dzts = mx_quantize_dim0_dim1(dz)
    dx = mx_grouped_mm_dgrad(dzq, dzs, *w.w1_t, offs, m, 2 * w.ffn, k)
    dw1 = mx_grouped_mm_wgrad(dztq, dzts, xtq, xts, offs, m, 2 * w.ffn, k, out_dtype=dw_dtype)
    return dx, dw1, dw2, db1, db2
