// Launches of the grouped products with an epilogue (EP_POINT, EP_SWIGLU of gemm.hip).
// Included by one source per operand element kind, which keeps them separate compilations.
#pragma once

#define MX_GEMM_CORE_ONLY
#include "gemm.hip"

namespace mx {

// ---- few output tiles: the eight waves of a block split the contraction ----
// The kernel of gemm.hip runs a tile's contraction as one chain of k-steps, about 0.4 us each;
// with fewer tiles than compute units the chain is all there is (32 x 4096 outputs over 4096:
// 20 us on 32 units, where the operands take 3 us to read; 8 us here). Here a block takes a tile of TM x
// TN (64 or 32) and each wave every eighth 64-byte chunk of the contraction, which it brings
// into LDS of its own, one chunk ahead; the partial tiles meet in LDS, and every thread then
// finishes eight consecutive columns of one row. Nothing waits at a barrier inside the
// contraction. EP_SWIGLU: TN = 64, a band of 32 gate rows and one of 32 up rows.
// The chunk ahead stays in flight behind a counted wait, so every chunk issues the same LOADS
// instructions whatever lies inside the operands: codes and scales alike come in by LDS loads
// whose descriptors end with the operand, and what lies past that is zeros. (Scales loaded into
// registers under a branch on their band leave the count short where the band is absent.)
template <int TM, int TN, int EL>
struct SmallTile {
  static constexpr int PITCH = TN + 4;           // floats per row of a partial tile
  static constexpr int CODES = (TM + TN) * 64;   // one chunk of both operands
  static constexpr int BANDS = EL == EL_MXFP8 ? (TM + TN) / 32 : 0;  // 256 bytes of scales each
  static constexpr int CHUNK = CODES + BANDS * 256;
  static constexpr int LOADS = CODES / 1024 + BANDS;  // of a chunk, per wave
  static constexpr int PARTS = 8 * TM * PITCH * 4, RING = 8 * 2 * CHUNK;
  static constexpr int LDS = PARTS > RING ? PARTS : RING;
};

// ROWS operand rows, 64-byte chunk c of each, into LDS: piece q of row r at r * 64 + (q ^ ((r >>
// 2) & 3)) * 16, so that sixteen rows at one piece hit different banks. Rows past the
// descriptor's end and pieces past the contraction come in as zeros. The offset is opaque to the
// compiler, which otherwise makes two loads, one for each side of the choice.
template <int ROWS>
__device__ __forceinline__ void load_pieces(__amdgpu_buffer_rsrc_t rsrc, unsigned pitch, int c, uint8_t* dst, int l) {
#pragma unroll
  for (int i = 0; i < ROWS / 16; ++i) {
    const int r = 16 * i + (l >> 2);
    const unsigned k = (unsigned)c * 64 + ((l & 3) ^ ((r >> 2) & 3)) * 16;
    unsigned off = k < pitch ? (unsigned)r * pitch + k : 0x80000000u;
    asm("" : "+v"(off));
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_ptr_t)(dst + i * 1024), 16, off, 0, 0, 0);
  }
}

template <int TM, int TN, int EL, int OUT_BF16, int EP>
__global__ __launch_bounds__(512, 2) void k_epi_small(EpiArgs p) {
  constexpr bool GLU = EP == EP_SWIGLU, SCALED = EL == EL_MXFP8;
  using S = SmallTile<TM, TN, EL>;
  constexpr int IM = TM / 32, IN = TN / 32, PITCH = S::PITCH, CHUNK = S::CHUNK;
  static_assert(!GLU || TN == 64, "a gate band and an up band");
  extern __shared__ __attribute__((aligned(16))) float parts[];  // [8][TM][PITCH]
  const int tid = threadIdx.x, l = tid & 63, h = l >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  // the tile: m-tile fastest, so that neighbours share B's rows
  GroupChunk first{};
  GroupHit hit{0, p.M, 0, p.out_rows, 0, 0};
  const int64_t mt = blockIdx.x % p.mt_total, nt = blockIdx.x / p.mt_total;
  if (p.offs) {
    if (mt >= uniform(total_mtiles<TM>(p, first))) return;
    hit = find_group<TM>(p, mt, first);
    if (hit.g < 0) return;
  }
  const int64_t row0 = uniform(hit.s + (mt - hit.cum) * TM), row_end = uniform(hit.e);
  int64_t out_limit = row_end, out_shift = 0;
  if (p.offs_out) {
    const int64_t real_end = hit.s + (hit.eo - hit.so);
    out_shift = uniform(hit.so - hit.s);
    if (real_end < out_limit) out_limit = uniform(real_end);
  }
  const int g = __builtin_amdgcn_readfirstlane(hit.g);
  const int64_t a_rows = row_end - row0 < TM ? row_end - row0 : TM;
  // B's rows: TN from col0 on, or (EP_SWIGLU) 32 gate rows and the 32 up rows N/2 below
  const int64_t col0 = nt * TN, b_first = (int64_t)g * p.N + (GLU ? nt * 32 : col0);
  const int64_t b_rows = GLU ? 32 : (p.N - col0 < TN ? p.N - col0 : TN);
  const unsigned pitch = (unsigned)p.lda;
  const __amdgpu_buffer_rsrc_t ra =
      __builtin_amdgcn_make_buffer_rsrc((void*)(p.a + row0 * p.lda), (short)0, (int)(a_rows * p.lda), 0x00020000);
  const __amdgpu_buffer_rsrc_t rb =
      __builtin_amdgcn_make_buffer_rsrc((void*)(p.b + b_first * p.ldb), (short)0, (int)(b_rows * p.ldb), 0x00020000);
  const __amdgpu_buffer_rsrc_t ru = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(p.b + (b_first + (GLU ? p.N / 2 : 0)) * p.ldb), (short)0, (int)(b_rows * p.ldb), 0x00020000);
  // the scales of the tile's bands, A's, then B's (EP_SWIGLU: the gate band and, b_step further, the up band)
  const int64_t a_band = row0 / 32, b_band = b_first / 32, b_step = GLU ? p.N / 64 : 1;
  const int64_t a_left = (p.a_rows + 31) / 32 - a_band, b_left = (p.b_rows + 31) / 32 - b_band;
  const int64_t a_bands = a_left < IM ? a_left : IM, b_bands = GLU ? b_step + 1 : (b_left < IN ? b_left : IN);
  const __amdgpu_buffer_rsrc_t rsa = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(p.a_s + a_band * p.a_ktiles * 256), (short)0, (int)(SCALED ? a_bands * p.a_ktiles * 256 : 0), 0x00020000);
  const __amdgpu_buffer_rsrc_t rsb = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(p.b_s + b_band * p.b_ktiles * 256), (short)0, (int)(SCALED ? b_bands * p.b_ktiles * 256 : 0), 0x00020000);
  const int chunks = (int)((p.lda + 63) / 64);
  uint8_t* ring = (uint8_t*)parts + wave * 2 * CHUNK;
  // chunk c of both operands, with its 256-wide scale windows (lane l: row l % 32, block parity
  // l / 32; the chunk's byte is c % 4): S::LOADS instructions
  auto load = [&](int c, int buf) {
    uint8_t* dst = ring + buf * CHUNK;
    load_pieces<TM>(ra, pitch, c, dst, l);
    if constexpr (GLU) {
      load_pieces<32>(rb, pitch, c, dst + TM * 64, l);
      load_pieces<32>(ru, pitch, c, dst + TM * 64 + 32 * 64, l);
    } else {
      load_pieces<TN>(rb, pitch, c, dst + TM * 64, l);
    }
    if constexpr (SCALED) {
#pragma unroll
      for (int t = 0; t < IM + IN; ++t) {
        const unsigned band = t < IM ? (unsigned)t * (unsigned)p.a_ktiles : (unsigned)((t - IM) * b_step * p.b_ktiles);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(t < IM ? rsa : rsb, (lds_ptr_t)(dst + S::CODES + t * 256), 4,
                                                 (band + (c >> 2)) * 256 + 4 * l, 0, 0, 0);
      }
    }
  };
  v16f acc[IM][IN];
#pragma unroll
  for (int i = 0; i < IM; ++i)
#pragma unroll
    for (int j = 0; j < IN; ++j) acc[i][j] = (v16f){};
  if (wave < chunks) load(wave, 0);
  for (int c = wave, buf = 0; c < chunks; c += 8, buf ^= 1) {
    if (c + 8 < chunks) {
      load(c + 8, buf ^ 1);
      MX_WAIT_VMCNT(S::LOADS);  // all of chunk c
    } else {
      MX_WAIT_VMCNT(0);
    }
    lds_fence();
    u32x4 f[IM + IN][2];
#pragma unroll
    for (int t = 0; t < IM + IN; ++t)
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int r = 32 * t + (l & 31);
        f[t][q] = *(const u32x4*)(ring + buf * CHUNK + r * 64 + (((h + 2 * q) ^ ((r >> 2) & 3)) << 4));
      }
    int sc[IM + IN] = {};
    if constexpr (SCALED) {
#pragma unroll
      for (int t = 0; t < IM + IN; ++t)
        sc[t] = (int)(*(const unsigned*)(ring + buf * CHUNK + S::CODES + t * 256 + 4 * l) >> ((c & 3) * 8));
    }
#pragma unroll
    for (int i = 0; i < IM; ++i)
#pragma unroll
      for (int j = 0; j < IN; ++j) {
        const u32x4 a0 = f[i][0], a1 = f[i][1], b0 = f[IM + j][0], b1 = f[IM + j][1];
        if constexpr (SCALED) {
          const v8i a = (v8i){(int)a0[0], (int)a0[1], (int)a0[2], (int)a0[3], (int)a1[0], (int)a1[1], (int)a1[2], (int)a1[3]};
          const v8i b = (v8i){(int)b0[0], (int)b0[1], (int)b0[2], (int)b0[3], (int)b1[0], (int)b1[1], (int)b1[2], (int)b1[3]};
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b, a, acc[i][j], 0, 0, 0, sc[IM + j], 0, sc[i]);
        } else {
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, b0), __builtin_bit_cast(bf16x8, a0), acc[i][j], 0, 0, 0);
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, b1), __builtin_bit_cast(bf16x8, a1), acc[i][j], 0, 0, 0);
        }
      }
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): the next load overwrites what was read here
    lds_fence();
  }
  __syncthreads();  // every wave is done with its ring, which the partial tiles overlie
#pragma unroll
  for (int i = 0; i < IM; ++i)
#pragma unroll
    for (int j = 0; j < IN; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const v16f& c = acc[i][j];
        *(v4f*)&parts[(wave * TM + 32 * i + (l & 31)) * PITCH + 32 * j + 8 * q + 4 * h] =
            (v4f){c[4 * q], c[4 * q + 1], c[4 * q + 2], c[4 * q + 3]};
      }
  __syncthreads();
  constexpr int OC = GLU ? 32 : TN;  // output columns of the tile
  if (tid >= TM * OC / 8) return;
  const int r = tid / (OC / 8), c = tid % (OC / 8) * 8;
  const int64_t row = row0 + r, n_out = GLU ? p.N / 2 : p.N, col = (GLU ? nt * 32 : col0) + c;
  if (row >= out_limit || col >= n_out) return;
  const int64_t orow = row + out_shift;
  const int cols = n_out - col < 8 ? (int)(n_out - col) : 8;
  // z of the thread's columns from tile column c0 on: the waves' sums in order, then the bias
  auto sums = [&](int c0, int64_t bcol, float* z) {
#pragma unroll
    for (int e = 0; e < 8; e += 4) {
      v4f s = *(const v4f*)&parts[r * PITCH + c0 + e];
#pragma unroll
      for (int w = 1; w < 8; ++w) s += *(const v4f*)&parts[(w * TM + r) * PITCH + c0 + e];
#pragma unroll
      for (int q = 0; q < 4; ++q) z[e + q] = s[q] + (p.bias && e + q < cols ? p.bias[(int64_t)g * p.N + bcol + e + q] : 0.f);
    }
  };
  auto store_pre = [&](int64_t bcol, const float* z) {
    uint16_t* dst = p.pre + orow * p.N + bcol;
    if (p.N % 8 == 0)
      *(u32x4*)dst = (u32x4){bf16x2_rne(z[0], z[1]), bf16x2_rne(z[2], z[3]), bf16x2_rne(z[4], z[5]), bf16x2_rne(z[6], z[7])};
    else
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < cols) dst[e] = (uint16_t)bf16x2_rne(z[e], 0.f);
  };
  float z[8], u[8], y[8];
  sums(c, col, z);
  if (GLU) sums(c + 32, p.N / 2 + col, u);
  if (p.pre) {
    store_pre(col, z);
    if (GLU) store_pre(p.N / 2 + col, u);
  }
  const int64_t o = orow * p.ldo + col;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    y[e] = GLU ? z[e] * sigmoidf(z[e]) * u[e] : apply_act(z[e], p.act);
    if (p.residual && e < cols)
      y[e] += OUT_BF16 ? __builtin_bit_cast(float, (unsigned)((const uint16_t*)p.residual)[o + e] << 16)
                       : ((const float*)p.residual)[o + e];
  }
  if (p.ldo % 8 == 0) {  // then N is a multiple of 8 and every column is inside
    if (OUT_BF16) {
      *(u32x4*)((uint16_t*)p.out + o) = (u32x4){bf16x2_rne(y[0], y[1]), bf16x2_rne(y[2], y[3]), bf16x2_rne(y[4], y[5]), bf16x2_rne(y[6], y[7])};
    } else {
      *(v4f*)((float*)p.out + o) = (v4f){y[0], y[1], y[2], y[3]};
      *(v4f*)((float*)p.out + o + 4) = (v4f){y[4], y[5], y[6], y[7]};
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < cols) {
        if (OUT_BF16) ((uint16_t*)p.out)[o + e] = (uint16_t)bf16x2_rne(y[e], 0.f);
        else ((float*)p.out)[o + e] = y[e];
      }
  }
}

}  // namespace mx

namespace {

// The tiling. Up to a round of 64x64 tiles, k_epi_small: 64x64 tiles, 32x64 up to half a round,
// 32x32 where contraction rows above 4 KB then still leave units idle (kernel us, the kernel of
// gemm.hip / 64x64 / 32x64 / 32x32: 32 x 4096 over 4096 MXFP8 20 / 10 / 8 / 8, bf16 31 / 16 / 16
// / 11; 512 x 512 over 4096 MXFP8 19 / 10 / 8 / 8, bf16 30 / 20 / 15 / 12; 1024 x 1024 over 4096
// MXFP8 20 / 14 / 18 / 19; above: 512 x 4096 over 4096 21 / 29 / 35 / 36). Then few output tiles
// take quarter-size ones, short contractions and little more than half a round of the compute
// units 128x256 tiles, two blocks per unit, all else 256x256 ones with two waves per SIMD (one
// wave holding 256 sums is no faster beside a residual, 660 to 667 against 655 to 666 for 32768 x
// 7168 over 2048, and spills without one); two rounds and more of a bf16 output with groups run
// whole rounds and then the quarters of a short last one. Measured, us at 128x128 / 128x256 /
// 256x256: 2048 x 2048 x 2048 29 / 48 / 53 (bf16, 64 tiles of 256x256); 4096 x 2048 x 4096 46 /
// 41 / 45 (128 tiles); 4096 x 2560 x 2048 45 / 47 / 41 (160); 4096 x 2816 x 4096 bf16 115 / 125 /
// 96 (176); 8 groups, 16384 x 4096 x 4096 353 / 302 / 282, and 269 with the quarters.
template <int TM, int TN, int EL, int OUT, int EP>
hipError_t launch_epi_small(mx::EpiArgs p, hipStream_t stream) {
  constexpr int lds = mx::SmallTile<TM, TN, EL>::LDS;
  static const hipError_t attr = hipFuncSetAttribute((const void*)mx::k_epi_small<TM, TN, EL, OUT, EP>,
                                                     hipFuncAttributeMaxDynamicSharedMemorySize, lds);
  if (attr != hipSuccess) return attr;
  p.mt_total = (p.M + TM - 1) / TM + (p.offs ? p.groups : 0);
  p.nt = (p.N + TN - 1) / TN;
  if (p.mt_total * p.nt == 0) return hipSuccess;
  hipLaunchKernelGGL((mx::k_epi_small<TM, TN, EL, OUT, EP>), dim3((unsigned)(p.mt_total * p.nt)), dim3(512), lds, stream, p);
  return hipGetLastError();
}

template <int EL, int OUT, int EP>
hipError_t launch_epi(const mx::EpiArgs& p, hipStream_t stream) {
  constexpr int MODE = mx::MODE_MGROUP;
  constexpr int SMALL = EP == mx::EP_POINT_RES ? mx::EP_POINT : EP;  // k_epi_small asks at run time
  const int64_t tiles64 = ((p.M + 63) / 64 + (p.offs ? p.groups : 0)) * ((p.N + 63) / 64);
  if (tiles64 <= kComputeUnits / 2) {
    const int64_t tiles32 = ((p.M + 31) / 32 + (p.offs ? p.groups : 0)) * ((p.N + 31) / 32);
    if constexpr (EP != mx::EP_SWIGLU)
      if (p.lda > 4096 && tiles32 <= kComputeUnits) return launch_epi_small<32, 32, EL, OUT, SMALL>(p, stream);
    return launch_epi_small<32, 64, EL, OUT, SMALL>(p, stream);
  }
  if (tiles64 <= kComputeUnits) return launch_epi_small<64, 64, EL, OUT, SMALL>(p, stream);
  const int64_t big_tiles = ((p.M + 255) / 256) * ((p.N + 255) / 256);
  if (big_tiles < 128) return launch_cfg<128, 128, 2, 2, 4, 2, MODE, EL, OUT, EP>(p, stream);
  if (p.K <= 1024 || big_tiles < 160) return launch_cfg<128, 256, 2, 2, 3, 2, MODE, EL, OUT, EP>(p, stream);
  if (OUT && big_tiles >= 512 && p.offs) {
    mx::EpiArgs part = p;
    part.tail = mx::TAIL_MAIN;
    const hipError_t e = launch_cfg<256, 256, 2, 4, 4, 2, MODE, EL, OUT, EP>(part, stream);
    if (e != hipSuccess) return e;
    part.tail = mx::TAIL_SUB;
    return launch_cfg<128, 128, 2, 2, 4, 2, MODE, EL, OUT, EP>(part, stream, 2 * kComputeUnits);
  }
  return launch_cfg<256, 256, 2, 4, 4, 2, MODE, EL, OUT, EP>(p, stream);
}

template <int EL>
hipError_t launch_epi_any(const mx::EpiArgs& p, int out_bf16, hipStream_t stream) {
  if (p.act == mx::ACT_SWIGLU)
    return out_bf16 ? launch_epi<EL, 1, mx::EP_SWIGLU>(p, stream) : launch_epi<EL, 0, mx::EP_SWIGLU>(p, stream);
  if (p.residual)
    return out_bf16 ? launch_epi<EL, 1, mx::EP_POINT_RES>(p, stream) : launch_epi<EL, 0, mx::EP_POINT_RES>(p, stream);
  return out_bf16 ? launch_epi<EL, 1, mx::EP_POINT>(p, stream) : launch_epi<EL, 0, mx::EP_POINT>(p, stream);
}

}  // namespace

