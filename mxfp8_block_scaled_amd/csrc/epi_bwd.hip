// The backward of the product epilogues (bias, activation, residual): dpre = dy act'(z) and,
// per group, dbias = the column sums of dpre. Bound by HBM: 16384 rows of 2048 gate and 2048 up
// columns (336 MB) in 66 us, 5.1 TB/s, and 5 us for the bias sums' second launch.

#define MX_GEMM_CORE_ONLY
#include "gemm.hip"

namespace mx {

// dy act'(z) for the pointwise activations (sigmoidf as in the forward). ReLU's is a choice, not a
// product: what z <= 0 cuts off is 0 also for an infinite or NaN dy. From |z| = 1e4 on the sigmoid
// is 0 or 1 to the last bit and the terms with s (1 - s) vanish: z is clamped in them, as its
// powers would overflow and give 0 * inf.
template <int ACT>
__device__ inline float act_grad(float dy, float z) {
  if constexpr (ACT == ACT_RELU) return z > 0.f ? dy : 0.f;
  if constexpr (ACT == ACT_NONE) return dy;
  const float zc = fminf(fmaxf(z, -1e4f), 1e4f);
  if constexpr (ACT == ACT_GELU) {
    const float s = sigmoidf(kGelu0 * z * (1.f + kGelu1 * z * z));
    return dy * (s + zc * s * (1.f - s) * kGelu0 * (1.f + 3.f * kGelu1 * zc * zc));
  } else {
    const float s = sigmoidf(z);
    return dy * (s * (1.f + zc * (1.f - s)));
  }
}

__device__ inline float bf16_f32(uint16_t b) { return __builtin_bit_cast(float, (unsigned)b << 16); }

// V consecutive bf16 values of a row as floats, and back.
template <int V>
__device__ inline void load_bf16(const uint16_t* src, float* o) {
  if constexpr (V == 8) {
    const u32x4 d = __builtin_nontemporal_load((const u32x4*)src);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o[2 * i] = __builtin_bit_cast(float, d[i] << 16);
      o[2 * i + 1] = __builtin_bit_cast(float, d[i] & 0xffff0000u);
    }
  } else {
    o[0] = bf16_f32(src[0]);
  }
}
template <int V>
__device__ inline void store_bf16(uint16_t* dst, const float* v) {
  if constexpr (V == 8)
    *(u32x4*)dst = (u32x4){bf16x2_rne(v[0], v[1]), bf16x2_rne(v[2], v[3]), bf16x2_rne(v[4], v[5]), bf16x2_rne(v[6], v[7])};
  else
    dst[0] = (uint16_t)bf16x2_rne(v[0], 0.f);
}

struct EpiBwdArgs {
  const uint16_t* dy;   // [m x n_out]
  const uint16_t* pre;  // [m x n] (not read for ACT_NONE)
  GemmArgs groups;      // offs, groups, M: the row groups, for the shared group lookup
  int64_t n, n_out;
  int act;
  uint16_t* dpre;  // [m x n], or null (ACT_NONE: dy itself)
  float* part;     // [row tiles x n] column sums of each row tile, or null
  float* dbias;    // [groups x n]
};

constexpr int kBwdCols = 64;  // column chunks (of V) a block covers, one per lane

// One block: TR rows of one group (or of the rows past the last group, whose dpre is 0) by
// 64 chunks of V columns; wave w takes rows w, w + 4, ... Every dy and pre value is read
// and every dpre written once, 16 bytes per lane and 1 KB per wave and row; the column
// sums stay in registers, meet in LDS and leave as one partial row per row tile.
// The activation is a compile-time value: chosen at each unrolled value it cuts the rows' loop into
// pieces that each wait for their loads (kernel us, 1001 x 576 GELU 10 against 9, 16384 x 4096
// SiLU 77 against 67).
template <int TR, int V, int ACT>
__global__ __launch_bounds__(256) void k_epi_bwd(EpiBwdArgs p) {
  constexpr bool GLU = ACT == ACT_SWIGLU;
  __shared__ float sums[4][GLU ? 2 : 1][V][kBwdCols];
  const int l = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t mt = blockIdx.y;
  int64_t r0 = mt * TR, r1 = p.groups.M;
  bool real = true;
  if (p.groups.offs) {
    GroupChunk first{};
    const int64_t count = uniform(total_mtiles<TR>(p.groups, first));
    if (mt < count) {
      const GroupHit hit = find_group<TR>(p.groups, mt, first);
      r0 = uniform(hit.s + (mt - hit.cum) * TR);
      r1 = uniform(hit.e);
    } else {
      real = false;
      int32_t end = 0;  // the last group's end, clamped as the lookup reads it
      int32_t ce = 0, ceo = 0, cc = 0;
      for (int g0 = 0; g0 < p.groups.groups; g0 += 64) {
        const GroupChunk c = scan_chunk<TR>(p.groups, g0, ce, ceo, cc);
        end = ce = __builtin_amdgcn_readlane(c.e, 63);
        ceo = __builtin_amdgcn_readlane(c.eo, 63);
        cc = __builtin_amdgcn_readlane(c.cum, 63);
      }
      r0 = end + (mt - count) * TR;
    }
  }
  if (r0 >= r1) return;
  r1 = r0 + TR < r1 ? r0 + TR : r1;
  const int64_t col = ((int64_t)blockIdx.x * kBwdCols + l) * V;
  const bool in = col < p.n_out;
  float sg[V], su[V];
#pragma unroll
  for (int i = 0; i < V; ++i) sg[i] = su[i] = 0.f;
  if (in) {
#pragma unroll 4
    for (int64_t r = r0 + wave; r < r1; r += 4) {
      float dg[V], du[V];
#pragma unroll
      for (int i = 0; i < V; ++i) dg[i] = du[i] = 0.f;
      if (real) {
        float dy[V], z[V] = {}, u[V];
        load_bf16<V>(p.dy + r * p.n_out + col, dy);
        if (ACT != ACT_NONE) load_bf16<V>(p.pre + r * p.n + col, z);
        if (GLU) load_bf16<V>(p.pre + r * p.n + p.n_out + col, u);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          if (GLU) {
            // the factor that may be small first: dy u and dy z alone can overflow
            dg[i] = act_grad<ACT_SILU>(dy[i], z[i]) * u[i];
            du[i] = dy[i] * (z[i] * sigmoidf(z[i]));
          } else {
            dg[i] = act_grad<ACT>(dy[i], z[i]);
          }
          sg[i] += dg[i];
          if (GLU) su[i] += du[i];
        }
      }
      if (p.dpre) store_bf16<V>(p.dpre + r * p.n + col, dg);
      if (GLU) store_bf16<V>(p.dpre + r * p.n + p.n_out + col, du);
    }
  }
  if (!p.part || !real) return;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    sums[wave][0][i][l] = sg[i];
    if (GLU) sums[wave][1][i][l] = su[i];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < (GLU ? 2 : 1) * V * kBwdCols; i += 256) {
    const int half = i / (V * kBwdCols), c = i % (V * kBwdCols);  // column c of the block's
    const int64_t at = (int64_t)blockIdx.x * kBwdCols * V + c;
    if (at < p.n_out) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < 4; ++w) s += sums[w][half][c % V][c / V];
      p.part[mt * p.n + half * p.n_out + at] = s;
    }
  }
}

// dbias[g] = the sum of the partial rows of group g's row tiles: each of a block's four waves
// adds a quarter of the tiles, in order, for 64 columns, and the quarters add up in order.
template <int TR>
__global__ __launch_bounds__(256) void k_epi_dbias(EpiBwdArgs p) {
  __shared__ float quarter[4][64];
  const int l = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t col = (int64_t)blockIdx.x * 64 + l;
  const int g = blockIdx.y;
  int64_t t0 = 0, t1 = (p.groups.M + TR - 1) / TR;
  if (p.groups.offs) {
    int32_t ce = 0, ceo = 0, cc = 0;
    for (int g0 = 0; g0 < p.groups.groups; g0 += 64) {
      const GroupChunk c = scan_chunk<TR>(p.groups, g0, ce, ceo, cc);
      ce = __builtin_amdgcn_readlane(c.e, 63);
      ceo = __builtin_amdgcn_readlane(c.eo, 63);
      cc = __builtin_amdgcn_readlane(c.cum, 63);
      if (g < g0 + 64) {
        t1 = __builtin_amdgcn_readlane(c.cum, g - g0);
        t0 = t1 - __builtin_amdgcn_readlane(c.tiles, g - g0);
        break;
      }
    }
  }
  const int64_t n = t1 - t0, b = t0 + n * wave / 4, e = t0 + n * (wave + 1) / 4;
  float s = 0.f;
  if (col < p.n) {
#pragma unroll 16
    for (int64_t t = b; t < e; ++t) s += p.part[t * p.n + col];
  }
  quarter[wave][l] = s;
  __syncthreads();
  if (wave == 0 && col < p.n)
    p.dbias[(int64_t)g * p.n + col] = ((quarter[0][l] + quarter[1][l]) + quarter[2][l]) + quarter[3][l];
}

template <int TR, int V, int ACT>
hipError_t launch_bwd(const EpiBwdArgs& p, hipStream_t stream) {
  const int64_t tiles = (p.groups.M + TR - 1) / TR + (p.groups.offs ? p.groups.groups : 0);
  if (tiles > 0) {
    const dim3 grid((unsigned)((p.n_out + kBwdCols * V - 1) / (kBwdCols * V)), (unsigned)tiles);
    hipLaunchKernelGGL((k_epi_bwd<TR, V, ACT>), grid, dim3(256), 0, stream, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (p.dbias) {
    hipLaunchKernelGGL((k_epi_dbias<TR>), dim3((unsigned)((p.n + 63) / 64), (unsigned)p.groups.groups), dim3(256), 0,
                       stream, p);
    return hipGetLastError();
  }
  return hipSuccess;
}

// Rows per tile: 64, or 16 where 64-row tiles would be fewer than two blocks per compute unit (a
// wave's chain of rows is then what takes the time: 1001 x 576 GELU 33 us with 64 rows, 9 with 16).
int bwd_rows(int groups, int has_offs, int64_t m, int64_t n_out) {
  const int64_t tiles = (m + 63) / 64 + (has_offs ? groups : 0), v = n_out % 8 == 0 ? 8 : 1;
  return tiles * ((n_out + kBwdCols * v - 1) / (kBwdCols * v)) >= 512 ? 64 : 16;
}

template <int TR, int ACT>
hipError_t launch_bwd_act(const EpiBwdArgs& p, hipStream_t stream) {
  return p.n_out % 8 == 0 ? launch_bwd<TR, 8, ACT>(p, stream) : launch_bwd<TR, 1, ACT>(p, stream);
}

template <int TR>
hipError_t launch_bwd_rows(const EpiBwdArgs& p, hipStream_t stream) {
  switch (p.act) {
    case ACT_RELU: return launch_bwd_act<TR, ACT_RELU>(p, stream);
    case ACT_GELU: return launch_bwd_act<TR, ACT_GELU>(p, stream);
    case ACT_SILU: return launch_bwd_act<TR, ACT_SILU>(p, stream);
    case ACT_SWIGLU: return launch_bwd_act<TR, ACT_SWIGLU>(p, stream);
    default: return launch_bwd_act<TR, ACT_NONE>(p, stream);
  }
}

}  // namespace mx

// Row tiles of a call: the rows of the partial column sums, [tiles][n] floats of workspace.
int64_t mx_epilogue_backward_tiles(int groups, int has_offs, int64_t m, int64_t n, int act) {
  const int tr = mx::bwd_rows(groups, has_offs, m, act == mx::ACT_SWIGLU ? n / 2 : n);
  return (m + tr - 1) / tr + (has_offs ? groups : 0);
}

hipError_t mx_launch_epilogue_backward(const uint16_t* dy, const uint16_t* pre, const int32_t* offs, int groups,
                                       int64_t m, int64_t n, int act, uint16_t* dpre, float* dbias, float* part,
                                       hipStream_t stream) {
  mx::EpiBwdArgs p{};
  p.dy = dy; p.pre = pre; p.act = act; p.dpre = dpre; p.dbias = dbias; p.part = dbias ? part : nullptr;
  p.groups.offs = offs; p.groups.groups = groups; p.groups.M = m; p.groups.out_rows = m;
  p.n = n;
  p.n_out = act == mx::ACT_SWIGLU ? n / 2 : n;
  return mx::bwd_rows(groups, offs != nullptr, m, p.n_out) == 64 ? mx::launch_bwd_rows<64>(p, stream)
                                                                  : mx::launch_bwd_rows<16>(p, stream);
}
