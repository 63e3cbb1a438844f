// Orthogonalisation of a momentum update by Newton-Schulz products (the update of the Muon
// optimiser), for a batch of matrices (one per expert):
//
//   m' = mu m + g,  u = g + mu m' (Nesterov) or m';  X = u / (|u|_F + eps), transposed if tall
//   repeated:  A = X X^T,  X <- a X + (b A + c A^2) X
//
// X [R x L], R <= L. A step is three products, all on the GEMM kernel of gemm.hip with
// fp16 operands (the bf16 rate, three more bits):
//   EP_GRAM  X X^T and EP_POLY (.)^2, both symmetric: only the tiles on and above the
//            diagonal are computed, the others are written transposed from them
//   EP_STEP  B X, from B and the transpose of X (every operand is contraction-contiguous),
//            which adds the linear term and writes X and both its fp16 forms
//
// Rounding. The iteration multiplies small singular values by a (3.4) per step, and errors
// that look like small singular directions with them, so rounding X itself to 16 bits
// between the steps costs 1e-2 to 1 of the result where the input has few strong
// directions. Two things keep that out. The linear term a X is taken from X in fp32: what
// the products' rounded operands disturb then lies along strong directions, which the
// iteration does not amplify. And the symmetric matrices are stored less a multiple of the
// identity, which near orthogonality is most of them: with m = |X|^2 / R (the mean of A's
// diagonal), A = O + m I and
//   b A + c A^2 = s I + (b + 2 c m) O + c O^2,   s = b m + c m^2,
// so O and P = (b + 2 c m) O + c O^2 are rounded and s joins a in the fp32 term:
// X <- (a + s) X + P X. Any m gives the same result in exact arithmetic. Against 64 bits the
// outcome is 0.5e-3 to 1e-3 off (relative), below the rounding of a bf16 result; fp16 without
// the two is 1e-3 to 1.5e-1 off, bf16 1e-2 to 1. Powers of two scale the fp16 matrices
// away from fp16's limits: X by about sqrt(L), O by 2^12, P by 2^11.
//
// Bound by the matrix rate where the matrices are large (8 x 4096 x 4096, momentum and five steps:
// 13.2 ms, 0.84 PFLOP/s of the work with symmetric products halved; EP_STEP 1300 us its
// epilogue's 14 bytes per value included, EP_GRAM and EP_POLY 617 and 623 for 1088
// tiles, 4.25 rounds; norm and start 723), by the chain of 17 launches where they are small
// (256 x 256: 72 to 81 us, each kernel 4 to 5).

#include <cmath>

#define MX_GEMM_CORE_ONLY
#include "gemm.hip"

namespace mx {

constexpr float kScaleO = 4096.f, kScaleP = 2048.f;

__device__ inline float sum64(float v) {
#pragma unroll
  for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

__device__ inline unsigned f16_pair(float a, float b) {
  return __builtin_bit_cast(unsigned, (f16x2){(_Float16)a, (_Float16)b});
}
// two floats as two 16-bit values, fp16 or bf16 (round to nearest even)
template <bool BF16>
__device__ inline unsigned pair16(float a, float b) {
  return BF16 ? bf16x2_rne(a, b) : f16_pair(a, b);
}

// One wave's WM x WN block of 16-bit values, staged in LDS and written by whole row
// segments to dst [rows x cols] (pitch cols, a multiple of 8) at (row0, col0). acc holds the
// values times 1 / scale. TR: dst is the transpose, [cols-side rows]: dst[c][r].
template <class C, bool TR, bool BF16>
__device__ __forceinline__ void store16(const v16f (&acc)[C::TM][C::TN], float scale, uint16_t* dst, int64_t rows,
                                        int64_t cols, int64_t row0, int64_t col0, uint8_t* stg, int l) {
  constexpr int SR = TR ? C::WN : C::WM, SC = TR ? C::WM : C::WN;  // staged rows and columns
  constexpr int CPR = SC / 8;                                      // 16-byte chunks per staged row
  static_assert(SR * SC * 2 <= C::NST * C::STAGE_BYTES / C::WAVES && (CPR & (CPR - 1)) == 0, "staging");
  const int h = l >> 5;
  auto chunk = [&](int r, int ch) -> uint8_t* { return stg + (r * CPR + (ch ^ (r & (CPR - 1)))) * 16; };
#pragma unroll
  for (int i = 0; i < C::TM; ++i)
#pragma unroll
    for (int j = 0; j < C::TN; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int r = 32 * i + (l & 31), c = 32 * j + 8 * q + 4 * h;
        const v16f& a = acc[i][j];
        const unsigned lo = pair16<BF16>(a[4 * q] * scale, a[4 * q + 1] * scale);
        const unsigned hi = pair16<BF16>(a[4 * q + 2] * scale, a[4 * q + 3] * scale);
        if (!TR) {
          *(u32x2*)(chunk(r, c >> 3) + (c & 4) * 2) = (u32x2){lo, hi};
        } else {
          const uint16_t v[4] = {(uint16_t)lo, (uint16_t)(lo >> 16), (uint16_t)hi, (uint16_t)(hi >> 16)};
#pragma unroll
          for (int e = 0; e < 4; ++e) *(uint16_t*)(chunk(c + e, r >> 3) + (r & 7) * 2) = v[e];
        }
      }
  lds_fence();
  const int64_t d_row0 = TR ? col0 : row0, d_col0 = TR ? row0 : col0;
#pragma unroll 4
  for (int k = 0; k < SR * CPR / 64; ++k) {
    const int qi = 64 * k + l, r = qi / CPR, ch = qi % CPR;
    const u32x4 d = *(const u32x4*)chunk(r, ch);
    if (d_row0 + r < rows && d_col0 + ch * 8 < cols) *(u32x4*)(dst + (d_row0 + r) * cols + d_col0 + ch * 8) = d;
  }
  lds_fence();
}

template <class C, int EP>
__device__ __forceinline__ void ortho_epilogue(const OrthoArgs& p, const Tile& T, v16f (&acc)[C::TM][C::TN],
                                               uint8_t* stg, int wave, int l) {
  const int wm = wave / C::WAVE_COLS, wn = wave % C::WAVE_COLS, h = l >> 5;
  const int64_t row0 = T.a_row0 - T.g * p.M + wm * C::WM, col0 = T.col0 + wn * C::WN;
  float m = 0.f;
  for (int i = l; i < p.n_part; i += 64) m += p.part_in[(int64_t)T.g * p.n_part + i];
  m = sum64(m) / (float)(p.rows < p.cols ? p.rows : p.cols);  // rounded-up rows hold zeros and do not count
  if constexpr (EP == EP_GRAM) {
    const float inv = 1.f / (p.sx * p.sx);
#pragma unroll
    for (int i = 0; i < C::TM; ++i)
#pragma unroll
      for (int j = 0; j < C::TN; ++j)
#pragma unroll
        for (int v = 0; v < 16; ++v) {
          const int64_t r = row0 + 32 * i + (l & 31), c = col0 + 32 * j + 8 * (v / 4) + 4 * h + v % 4;
          acc[i][j][v] = acc[i][j][v] * inv - (r == c ? m : 0.f);
        }
    uint16_t* o = (uint16_t*)p.o16 + T.g * p.M * p.M;
    store16<C, false, false>(acc, kScaleO, o, p.M, p.M, row0, col0, stg, l);
    if (T.a_row0 - T.g * p.M != T.col0) store16<C, true, false>(acc, kScaleO, o, p.M, p.M, row0, col0, stg, l);
  } else if constexpr (EP == EP_POLY) {
    // O of the wave's block comes in by whole row segments and is read from LDS by the lane
    // that holds the matching sums
    constexpr int CPR = C::WN / 8;
    auto chunk = [&](int r, int ch) -> uint8_t* { return stg + (r * CPR + (ch ^ (r & (CPR - 1)))) * 16; };
    const uint16_t* o = (const uint16_t*)p.o16 + T.g * p.M * p.M;
    stage_rows<C::WM, CPR>(o, p.M * 2, p.M, p.M / 8, row0, col0 / 8, stg, l);
    const float k1 = (p.cb + 2.f * p.cc * m) / kScaleO, k2 = p.cc / (kScaleO * kScaleO);
#pragma unroll
    for (int i = 0; i < C::TM; ++i)
#pragma unroll
      for (int j = 0; j < C::TN; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int r = 32 * i + (l & 31), c = 32 * j + 8 * q + 4 * h;
          const u32x2 d = *(const u32x2*)(chunk(r, c >> 3) + (c & 4) * 2);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const unsigned two = d[e >> 1];
            const float ov = (float)__builtin_bit_cast(f16x2, two)[e & 1];
            acc[i][j][4 * q + e] = k1 * ov + k2 * acc[i][j][4 * q + e];
          }
        }
    lds_fence();
    uint16_t* b = (uint16_t*)p.b16 + T.g * p.M * p.M;
    store16<C, false, false>(acc, kScaleP, b, p.M, p.M, row0, col0, stg, l);
    if (T.a_row0 - T.g * p.M != T.col0) store16<C, true, false>(acc, kScaleP, b, p.M, p.M, row0, col0, stg, l);
  } else {
    // X <- (a + s) X + P X: X's fp32 rows come in and leave through LDS in whole segments
    const float lin = p.ca + p.cb * m + p.cc * m * m, inv = 1.f / (kScaleP * p.sx);
    constexpr int CPR = C::WN / 4;
    constexpr int RP = epi_rows(C::WM, C::NST * C::STAGE_BYTES / C::WAVES / (C::WN * 4));
    auto chunk = [&](int r, int ch) -> uint8_t* { return stg + (r * CPR + (ch ^ (r & (CPR - 1)))) * 16; };
    float* x = p.x32 + T.g * p.M * p.N;
    float sq = 0.f;
#pragma unroll
    for (int pass = 0; pass < C::WM / RP; ++pass) {
      const int64_t prow0 = row0 + pass * RP;
      stage_rows<RP, CPR>(x, p.N * 4, p.M, p.N / 4, prow0, col0 / 4, stg, l);
#pragma unroll
      for (int ii = 0; ii < RP / 32; ++ii)
#pragma unroll
        for (int j = 0; j < C::TN; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            v16f& a = acc[pass * (RP / 32) + ii][j];
            const int r = 32 * ii + (l & 31), c = 32 * j + 8 * q + 4 * h;
            v4f* at = (v4f*)chunk(r, c >> 2);
            const v4f old = *at;
            v4f y;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              y[e] = lin * old[e] + inv * a[4 * q + e];
              a[4 * q + e] = y[e];
              sq += y[e] * y[e];  // rows and columns outside X are zeros
            }
            if (!p.last) *at = y;
          }
      lds_fence();
      if (!p.last) {
#pragma unroll 4
        for (int k = 0; k < RP * CPR / 64; ++k) {
          const int qi = 64 * k + l, r = qi / CPR, ch = qi % CPR;
          const u32x4 d = *(const u32x4*)chunk(r, ch);
          if (prow0 + r < p.M && col0 + ch * 4 < p.N) *(u32x4*)(x + (prow0 + r) * p.N + col0 + ch * 4) = d;
        }
        lds_fence();
      }
    }
    if (!p.last) {
      sq = sum64(sq);
      const int64_t tile = (T.a_row0 - T.g * p.M) / (C::WM * (C::WAVES / C::WAVE_COLS)) * p.nt + T.col0 / (C::WN * C::WAVE_COLS);
      if (l == 0) p.part_out[(T.g * p.mt_total * p.nt + tile) * C::WAVES + wave] = sq;
      store16<C, false, false>(acc, p.sx, (uint16_t*)p.x16 + T.g * p.M * p.N, p.M, p.N, row0, col0, stg, l);
      store16<C, true, false>(acc, p.sx, (uint16_t*)p.xt16 + T.g * p.M * p.N, p.N, p.M, row0, col0, stg, l);
    } else {
      uint16_t* out = p.out + T.g * p.rows * p.cols;
      if (p.cols % 8 == 0) {
        if (p.tall) store16<C, true, true>(acc, 1.f, out, p.rows, p.cols, row0, col0, stg, l);
        else store16<C, false, true>(acc, 1.f, out, p.rows, p.cols, row0, col0, stg, l);
      } else {  // rows that are not 16-byte aligned
#pragma unroll
        for (int i = 0; i < C::TM; ++i)
#pragma unroll
          for (int j = 0; j < C::TN; ++j)
#pragma unroll
            for (int v = 0; v < 16; ++v) {
              const int64_t r = row0 + 32 * i + (l & 31), c = col0 + 32 * j + 8 * (v / 4) + 4 * h + v % 4;
              const int64_t orow = p.tall ? c : r, ocol = p.tall ? r : c;
              if (orow < p.rows && ocol < p.cols)
                out[orow * p.cols + ocol] = (uint16_t)bf16x2_rne(acc[i][j][v], 0.f);
            }
      }
    }
  }
}

// ---- few tiles: 64x64 tiles, the eight waves of a block split the contraction ----
// A matrix of a few hundred rows makes too few 128x128 tiles for the compute units, and each
// runs its whole contraction as one chain of steps. Here a block takes a 64x64 tile and each
// wave every eighth 32-element chunk of the contraction, which it brings into LDS of its own
// (whole 64-byte row pieces, one chunk ahead); the partial tiles meet in LDS, and every thread
// then holds eight consecutive columns of one row. Nothing waits at a barrier inside the
// contraction. (Operands straight from memory to the matrix layout's registers, 32 rows of 16
// bytes to a load, ran four times slower: the loads' cost goes by the rows they touch.)

// Tiles of TS x TS, 64 or 32.
template <int TS>
struct Small {
  static constexpr int PITCH = TS + 4;             // floats per row of a partial tile: 16-byte rows, spread over the banks
  static constexpr int KE = TS == 32 ? 64 : 32;    // elements of a row in a chunk
  static constexpr int CHUNK = 2 * TS * KE * 2;    // one chunk of both operands
  static constexpr int PARTS = 8 * TS * PITCH * 4, RING = 8 * 2 * CHUNK;
  static constexpr int LDS = PARTS > RING ? PARTS : RING;
};

// TS operand rows from row0 on, elements [KE c, KE c + KE), into LDS: 16-byte piece q of row r
// goes to r * KE * 2 + (q ^ (r * KE / 128 % (KE / 8))) * 16, so that sixteen rows at one piece hit
// different banks. Rows past the matrix are past the descriptor's end, pieces past K out of
// range: zeros.
template <int TS>
__device__ __forceinline__ int chunk_piece(int r, int q) {
  constexpr int KE = Small<TS>::KE;
  return q ^ (r / (128 / KE) % (KE / 8));
}
template <int TS>
__device__ __forceinline__ void load_chunk(__amdgpu_buffer_rsrc_t rsrc, int64_t row0, int c, int64_t K, uint8_t* dst,
                                           int l) {
  constexpr int KE = Small<TS>::KE, PIECES = KE / 8, ROWS = 64 / PIECES;  // rows of one load
#pragma unroll
  for (int i = 0; i < TS / ROWS; ++i) {
    const int r = ROWS * i + l / PIECES;
    const int64_t k = (int64_t)c * KE + chunk_piece<TS>(r, l % PIECES) * 8;
    const unsigned off = k < K ? (unsigned)((row0 + r) * K + k) * 2 : 0xfffffff0u;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_ptr_t)(dst + i * 1024), 16, off, 0, 0, 0);
  }
}

template <int EP, int TS>
__global__ __launch_bounds__(512, 2) void k_ortho_tile(OrthoArgs p) {
  constexpr bool SYM = EP == EP_GRAM || EP == EP_POLY;
  constexpr int T = TS / 32, PITCH = Small<TS>::PITCH, CHUNK = Small<TS>::CHUNK;
  extern __shared__ __attribute__((aligned(16))) float parts[];  // [8][TS][PITCH]
  const int tid = threadIdx.x, l = tid & 63, h = l >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t g = blockIdx.y, R = p.M, N = p.N, K = p.K;
  int64_t mt, nt;
  if (SYM) {  // row mt of the triangle has nt0 - mt tiles
    const int64_t nt0 = (N + TS - 1) / TS;
    int64_t t = blockIdx.x;
    for (mt = 0; t >= nt0 - mt; ++mt) t -= nt0 - mt;
    nt = mt + t;
  } else {
    const int64_t rows = (R + TS - 1) / TS;
    mt = blockIdx.x % rows;
    nt = blockIdx.x / rows;
  }
  const int64_t row0 = mt * TS, col0 = nt * TS;
  float m = 0.f;
  for (int i = l; i < p.n_part; i += 64) m += p.part_in[g * p.n_part + i];
  const __amdgpu_buffer_rsrc_t ra = __builtin_amdgcn_make_buffer_rsrc((void*)(p.a + g * R * K * 2), (short)0, (int)(R * K * 2), 0x00020000);
  const __amdgpu_buffer_rsrc_t rb = __builtin_amdgcn_make_buffer_rsrc((void*)(p.b + g * N * K * 2), (short)0, (int)(N * K * 2), 0x00020000);
  v16f acc[T][T];
#pragma unroll
  for (int i = 0; i < T; ++i)
#pragma unroll
    for (int j = 0; j < T; ++j) acc[i][j] = (v16f){};
  constexpr int KE = Small<TS>::KE;
  const int chunks = (int)((K + KE - 1) / KE);
  uint8_t* ring = (uint8_t*)parts + wave * 2 * CHUNK;
  auto load = [&](int c, int buf) {
    load_chunk<TS>(ra, row0, c, K, ring + buf * CHUNK, l);
    load_chunk<TS>(rb, col0, c, K, ring + buf * CHUNK + CHUNK / 2, l);
  };
  if (wave < chunks) load(wave, 0);
  for (int c = wave, buf = 0; c < chunks; c += 8, buf ^= 1) {
    if (c + 8 < chunks) {
      load(c + 8, buf ^ 1);
      MX_WAIT_VMCNT(CHUNK / 1024);
    } else {
      MX_WAIT_VMCNT(0);
    }
    lds_fence();
    // both operands take the chunk's elements in the same order: lane half h pieces h, h + 2, ...
    f16x8 f[2][T][KE / 16];  // operand, 32-row tile, piece
#pragma unroll
    for (int o = 0; o < 2; ++o)
#pragma unroll
      for (int t = 0; t < T; ++t)
#pragma unroll
        for (int q = 0; q < KE / 16; ++q) {
          const int r = 32 * t + (l & 31);
          f[o][t][q] = *(const f16x8*)(ring + buf * CHUNK + o * (CHUNK / 2) + r * KE * 2 +
                                       chunk_piece<TS>(r, h + 2 * q) * 16);
        }
#pragma unroll
    for (int q = 0; q < KE / 16; ++q)
#pragma unroll
      for (int i = 0; i < T; ++i)
#pragma unroll
        for (int j = 0; j < T; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(f[1][j][q], f[0][i][q], acc[i][j], 0, 0, 0);
    lds_fence();
  }
  __syncthreads();  // every wave is done with its ring, which the partial tiles overlie
  // row l % 32, columns 8 q + 4 h + {0..3} of each 32x32 tile
#pragma unroll
  for (int i = 0; i < T; ++i)
#pragma unroll
    for (int j = 0; j < T; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const v16f& c = acc[i][j];
        *(v4f*)&parts[(wave * TS + 32 * i + (l & 31)) * PITCH + 32 * j + 8 * q + 4 * h] =
            (v4f){c[4 * q], c[4 * q + 1], c[4 * q + 2], c[4 * q + 3]};
      }
  m = sum64(m) / (float)(p.rows < p.cols ? p.rows : p.cols);
  __syncthreads();
  const int r = tid / (TS / 8), c = tid % (TS / 8) * 8;
  const bool mine = tid < TS * TS / 8;  // whole waves
  const int64_t row = row0 + r, col = col0 + c;
  const bool in = mine && row < R && col < N;
  float y[8] = {};
  if (mine)
#pragma unroll
  for (int e = 0; e < 8; e += 4) {
    v4f s = *(const v4f*)&parts[r * PITCH + c + e];
#pragma unroll
    for (int w = 1; w < 8; ++w) s += *(const v4f*)&parts[(w * TS + r) * PITCH + c + e];
#pragma unroll
    for (int q = 0; q < 4; ++q) y[e + q] = s[q];
  }
  float scale = 1.f;
  _Float16 *same = nullptr, *turned = nullptr;  // [R][N] and [N][R]
  if constexpr (EP == EP_GRAM) {
    const float inv = 1.f / (p.sx * p.sx);
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = y[e] * inv - (row == col + e ? m : 0.f);
    scale = kScaleO;
    same = p.o16 + g * R * R;
    turned = mt != nt ? same : nullptr;
  } else if constexpr (EP == EP_POLY) {
    const float k1 = (p.cb + 2.f * p.cc * m) / kScaleO, k2 = p.cc / (kScaleO * kScaleO);
    const f16x8 o = in ? *(const f16x8*)(p.o16 + (g * R + row) * R + col) : (f16x8){};
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = k1 * (float)o[e] + k2 * y[e];
    scale = kScaleP;
    same = p.b16 + g * R * R;
    turned = mt != nt ? same : nullptr;
  } else {
    const float lin = p.ca + p.cb * m + p.cc * m * m, inv = 1.f / (kScaleP * p.sx);
    float* x = p.x32 + (g * R + row) * N + col;
    float sq = 0.f;
#pragma unroll
    for (int e = 0; e < 8; e += 4) {
      const v4f old = in ? *(const v4f*)(x + e) : (v4f){0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        y[e + q] = lin * old[q] + inv * y[e + q];
        sq += y[e + q] * y[e + q];
      }
      if (in && !p.last) *(v4f*)(x + e) = (v4f){y[e], y[e + 1], y[e + 2], y[e + 3]};
    }
    if (p.last) {
      uint16_t* out = p.out + g * p.rows * p.cols;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (!mine) break;
        const int64_t orow = p.tall ? col + e : row, ocol = p.tall ? row : col + e;
        if (orow < p.rows && ocol < p.cols) out[orow * p.cols + ocol] = (uint16_t)bf16x2_rne(y[e], 0.f);
      }
      return;
    }
    sq = sum64(sq);
    __syncthreads();  // every partial tile is read
    if (l == 0) parts[wave] = sq;
    __syncthreads();
    if (tid == 0) {
      float all = 0.f;
#pragma unroll
      for (int w = 0; w < 8; ++w) all += parts[w];
      p.part_out[g * gridDim.x + blockIdx.x] = all;
    }
    scale = p.sx;
    same = p.x16 + g * R * N;
    turned = p.xt16 + g * R * N;
  }
  if (in)
    *(u32x4*)(same + row * N + col) = (u32x4){f16_pair(y[0] * scale, y[1] * scale), f16_pair(y[2] * scale, y[3] * scale),
                                              f16_pair(y[4] * scale, y[5] * scale), f16_pair(y[6] * scale, y[7] * scale)};
  if (turned) {  // through LDS: eight consecutive rows of one column per thread
    __syncthreads();
    float* t = parts + 16;  // past what the sum above still reads
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (mine) t[r * (TS + 1) + c + e] = y[e];
    __syncthreads();
    if (mine && col0 + r < N && row0 + c < R) {
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = t[(c + e) * (TS + 1) + r] * scale;
      *(u32x4*)(turned + (col0 + r) * R + row0 + c) =
          (u32x4){f16_pair(y[0], y[1]), f16_pair(y[2], y[3]), f16_pair(y[4], y[5]), f16_pair(y[6], y[7])};
    }
  }
}

struct OrthoInput {
  const void* g;
  const float* mom;      // or null
  float* mom_out;
  float mu;
  int nesterov;
  int64_t rows, cols, rows_p, cols_p;  // and rounded up to multiples of 8
  double* norm;   // [groups][kNormBlocks] sums of squares
  float eps, sx;
  int tall;
  float* x32;
  _Float16 *same, *turned;  // [rows_p][cols_p] and [cols_p][rows_p]
  float* part0;   // [groups] |X|^2
};

constexpr int kNormBlocks = 256;

template <int BF16>
__device__ inline float input_at(const void* g, int64_t i) {
  return BF16 ? __builtin_bit_cast(float, (unsigned)((const uint16_t*)g)[i] << 16) : ((const float*)g)[i];
}

// m' and the squares of u: one pass over g and m, V values per thread at a time. Squares are
// summed in float64, so that neither the size of the values nor their number matters.
template <int BF16, int V>
__global__ __launch_bounds__(256) void k_ortho_norm(OrthoInput p) {
  __shared__ double part[4];
  const int64_t n = p.rows * p.cols, base = blockIdx.y * n;
  double s = 0.;
  for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * V; i < n; i += (int64_t)gridDim.x * 256 * V) {
    float g[V], m[V];
    if constexpr (V == 4) {
      if constexpr (BF16) {
        const u32x2 d = *(const u32x2*)((const uint16_t*)p.g + base + i);
#pragma unroll
        for (int e = 0; e < 4; ++e) g[e] = __builtin_bit_cast(float, e & 1 ? d[e >> 1] & 0xffff0000u : d[e >> 1] << 16);
      } else {
        *(v4f*)g = *(const v4f*)((const float*)p.g + base + i);
      }
      if (p.mom) *(v4f*)m = *(const v4f*)(p.mom + base + i);
    } else {
      g[0] = input_at<BF16>(p.g, base + i);
      if (p.mom) m[0] = p.mom[base + i];
    }
#pragma unroll
    for (int e = 0; e < V; ++e) {
      float u = g[e];
      if (p.mom) {
        m[e] = p.mu * m[e] + g[e];
        u = p.nesterov ? g[e] + p.mu * m[e] : m[e];
      }
      s += (double)u * (double)u;
    }
    if (p.mom) {
      if constexpr (V == 4) *(v4f*)(p.mom_out + base + i) = *(v4f*)m;
      else p.mom_out[base + i] = m[0];
    }
  }
#pragma unroll
  for (int d = 32; d; d >>= 1) s += __shfl_xor(s, d);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) p.norm[blockIdx.y * kNormBlocks + blockIdx.x] = part[0] + part[1] + part[2] + part[3];
}

// X in fp32 and both fp16 forms, one 64 x 64 tile of the input per block; zeros in the
// rounded-up margins.
template <int BF16>
__global__ __launch_bounds__(256) void k_ortho_init(OrthoInput p) {
  __shared__ float tile[64][65];
  const int tid = threadIdx.x, l = tid & 63;
  const int64_t b = blockIdx.z, r0 = (int64_t)blockIdx.y * 64, c0 = (int64_t)blockIdx.x * 64;
  const int64_t base = b * p.rows * p.cols;
  // All on their way before the norm is known. Places outside the matrix read its last row or
  // column instead and count as zero below: a branch around each load would wait for each.
  const int64_t c = c0 + l < p.cols ? c0 + l : p.cols - 1;
  float u[16], m[16];
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    const int64_t r = r0 + k * 4 + (tid >> 6), i = base + (r < p.rows ? r : p.rows - 1) * p.cols + c;
    u[k] = input_at<BF16>(p.g, i);
    m[k] = p.mom ? p.mom_out[i] : 0.f;
  }
  double s = 0.;
#pragma unroll
  for (int i = 0; i < kNormBlocks; i += 64) s += p.norm[b * kNormBlocks + i + l];
#pragma unroll
  for (int d = 32; d; d >>= 1) s += __shfl_xor(s, d);
  // A norm near or beyond float32's limits is brought back by a power of two, which v below takes
  // too; a zero matrix with eps = 0 stays zero.
  const double size = sqrt(s) + (double)p.eps;
  const float pre = size > 0x1p100 ? 0x1p-100f : size < 0x1p-100 ? 0x1p100f : 1.f;
  const float norm = (float)(sqrt(s) * pre), div = norm + p.eps * pre, inv = div == 0.f ? 0.f : 1.f / div;
  if (tid == 0 && blockIdx.x == 0 && blockIdx.y == 0) p.part0[b] = norm * inv * norm * inv;
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    const float v = !p.mom ? u[k] : p.nesterov ? u[k] + p.mu * m[k] : m[k];
    tile[k * 4 + (tid >> 6)][l] = r0 + k * 4 + (tid >> 6) < p.rows && c0 + l < p.cols ? v * pre * inv : 0.f;
  }
  __syncthreads();
  const int64_t pb = b * p.rows_p * p.cols_p;
#pragma unroll
  for (int turn = 0; turn < 2; ++turn) {
    const int64_t rr = turn ? p.cols_p : p.rows_p, cc = turn ? p.rows_p : p.cols_p;
    const int64_t dr0 = turn ? c0 : r0, dc0 = turn ? r0 : c0;
    _Float16* dst = (turn ? p.turned : p.same) + pb;
    float* dst32 = (p.tall != 0) == (turn != 0) ? p.x32 + pb : nullptr;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int i = k * 256 + tid, r = i >> 3, c = (i & 7) * 8;
      if (dr0 + r >= rr || dc0 + c >= cc) continue;
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = turn ? tile[c + e][r] : tile[r][c + e];
      const int64_t at = (dr0 + r) * cc + dc0 + c;
      *(u32x4*)(dst + at) = (u32x4){f16_pair(v[0] * p.sx, v[1] * p.sx), f16_pair(v[2] * p.sx, v[3] * p.sx),
                                    f16_pair(v[4] * p.sx, v[5] * p.sx), f16_pair(v[6] * p.sx, v[7] * p.sx)};
      if (dst32) {
        *(v4f*)(dst32 + at) = (v4f){v[0], v[1], v[2], v[3]};
        *(v4f*)(dst32 + at + 4) = (v4f){v[4], v[5], v[6], v[7]};
      }
    }
  }
}

}  // namespace mx

namespace {

// The tile rule, for EP_STEP and for the symmetric products, by the tiles there are: 256x256
// where they make most of a round of the 256 compute units; then 128x128; k_ortho_tile's 64x64
// where they are at most one round (its operands are read twice as often, so more tiles lose
// again), its 32x32 where even those would leave most units idle. Five steps, momentum left
// out, in us with all products at 128 / 64 / 32 / by the rule: 256 x 256 135 / 98 / 74 / 75;
// 576 x 4096 358 / 303 / 342 / 195; 1024 x 1024 244 / 159 / 238 / 159; 8 x 512 x 512 184 / 231 /
// 265 / 184; 2048 x 2048 432 / 727 / 1488 / 432. (8 x 4096 x 4096: EP_STEP in 128x256 tiles, two
// blocks to a compute unit, 1536 us against 1385 us at 256x256; the symmetric products' last
// 64 of 1088 tiles as 128x128 quarters, 635 us in two launches against 632 us.)
int tile_for(int64_t tiles256, int64_t tiles64, int64_t operand) {
  if (tiles256 >= 192) return 256;
  if (tiles64 > 256 || operand >= ((int64_t)1 << 29)) return 128;  // the small tiles' offsets are 32-bit
  return tiles64 > 96 ? 64 : 32;
}
int step_tile(int64_t batch, int64_t R, int64_t L) {
  return tile_for(batch * ((R + 255) / 256) * ((L + 255) / 256), batch * ((R + 63) / 64) * ((L + 63) / 64), R * L);
}
int square_tile(int64_t batch, int64_t R, int64_t L) {
  return tile_for(batch * mx::triangle_tiles((R + 255) / 256), batch * mx::triangle_tiles((R + 63) / 64), R * L);
}

template <int EP, int TS>
hipError_t launch_small(const mx::OrthoArgs& p, hipStream_t stream) {
  const int64_t mt = (p.M + TS - 1) / TS, nt = (p.N + TS - 1) / TS;
  const int64_t tiles = EP == mx::EP_STEP ? mt * nt : mx::triangle_tiles(nt);
  static const hipError_t attr = hipFuncSetAttribute((const void*)mx::k_ortho_tile<EP, TS>,
                                                     hipFuncAttributeMaxDynamicSharedMemorySize, mx::Small<TS>::LDS);
  if (attr != hipSuccess) return attr;
  hipLaunchKernelGGL((mx::k_ortho_tile<EP, TS>), dim3((unsigned)tiles, (unsigned)p.groups), dim3(512),
                     mx::Small<TS>::LDS, stream, p);
  return hipGetLastError();
}

void operands(mx::OrthoArgs& p, int64_t n, int64_t k, const _Float16* a, const _Float16* b) {
  p.a = (const uint8_t*)a;
  p.b = (const uint8_t*)b;
  p.N = n;
  p.K = k;
  p.lda = p.ldb = 2 * k;
  p.a_rows = (int64_t)p.groups * p.M;
  p.b_rows = (int64_t)p.groups * n;
  p.splits = 1;
}

template <int EP>
hipError_t square_product(mx::OrthoArgs p, int64_t k, const _Float16* a, hipStream_t stream) {
  operands(p, p.M, k, a, a);
  const int t = square_tile(p.groups, p.M, p.L);
  if (t == 32) return launch_small<EP, 32>(p, stream);
  if (t == 64) return launch_small<EP, 64>(p, stream);
  if (t == 256)
    return launch_cfg<256, 256, 2, 4, 4, 2, mx::MODE_BATCH, mx::EL_F16, 0, EP>(
        p, stream, p.groups * mx::triangle_tiles((p.M + 255) / 256));
  return launch_cfg<128, 128, 2, 2, 4, 2, mx::MODE_BATCH, mx::EL_F16, 0, EP>(
      p, stream, p.groups * mx::triangle_tiles((p.M + 127) / 128));
}

hipError_t step_product(mx::OrthoArgs p, int64_t L, const _Float16* xt, hipStream_t stream) {
  operands(p, L, p.M, p.b16, xt);
  const int t = step_tile(p.groups, p.M, L);
  if (t == 32) return launch_small<mx::EP_STEP, 32>(p, stream);
  if (t == 64) return launch_small<mx::EP_STEP, 64>(p, stream);
  if (t == 256)
    return launch_cfg<256, 256, 2, 4, 4, 2, mx::MODE_BATCH, mx::EL_F16, 0, mx::EP_STEP>(p, stream);
  return launch_cfg<128, 128, 2, 2, 4, 2, mx::MODE_BATCH, mx::EL_F16, 0, mx::EP_STEP>(p, stream);
}

struct Layout {  // workspace offsets (bytes)
  int64_t R, L, n_part, norm, part0, part[2], x32, x16, xt16[2], o16, b16, total;
};
Layout ortho_layout(int64_t batch, int64_t rows, int64_t cols) {
  Layout w{};
  const int64_t rp = (rows + 7) / 8 * 8, cp = (cols + 7) / 8 * 8;
  w.R = rows > cols ? cp : rp;
  w.L = rows > cols ? rp : cp;
  // one sum of squares per wave of a 256x256 or 128x128 tile, per 64x64 tile
  const int64_t t = step_tile(batch, w.R, w.L);
  w.n_part = ((w.R + t - 1) / t) * ((w.L + t - 1) / t) * (t == 256 ? 8 : t == 128 ? 4 : 1);
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t o = at;
    at += (bytes + 255) / 256 * 256;
    return o;
  };
  w.norm = take(batch * mx::kNormBlocks * 8);
  w.part0 = take(batch * 4);
  w.part[0] = take(batch * w.n_part * 4);
  w.part[1] = take(batch * w.n_part * 4);
  w.x32 = take(batch * w.R * w.L * 4);
  w.x16 = take(batch * w.R * w.L * 2);
  for (int64_t& x : w.xt16) x = take(batch * w.R * w.L * 2);
  w.o16 = take(batch * w.R * w.R * 2);
  w.b16 = take(batch * w.R * w.R * 2);
  w.total = at;
  return w;
}

}  // namespace

int64_t mx_ortho_workspace_bytes(int64_t batch, int64_t rows, int64_t cols) {
  return ortho_layout(batch, rows, cols).total;
}

hipError_t mx_launch_ortho(const void* g, int g_bf16, const float* mom, float* mom_out, float mu, int nesterov,
                           int64_t batch, int64_t rows, int64_t cols, int steps, const float* coefs, float eps,
                           uint16_t* out, void* ws, hipStream_t stream) {
  const Layout w = ortho_layout(batch, rows, cols);
  uint8_t* base = (uint8_t*)ws;
  mx::OrthoInput in{};
  in.g = g; in.mom = mom; in.mom_out = mom_out; in.mu = mu; in.nesterov = nesterov;
  in.rows = rows; in.cols = cols;
  in.rows_p = (rows + 7) / 8 * 8;
  in.cols_p = (cols + 7) / 8 * 8;
  in.norm = (double*)(base + w.norm);
  in.eps = eps;
  in.sx = 1.f;
  while ((double)in.sx * in.sx < (double)w.L) in.sx *= 2.f;
  in.tall = rows > cols;
  in.x32 = (float*)(base + w.x32);
  // two transposes: EP_STEP's blocks read all of the old one while they write the new one
  _Float16 *x16 = (_Float16*)(base + w.x16), *xt16[2] = {(_Float16*)(base + w.xt16[0]), (_Float16*)(base + w.xt16[1])};
  in.same = in.tall ? xt16[0] : x16;
  in.turned = in.tall ? x16 : xt16[0];
  in.part0 = (float*)(base + w.part0);
  const dim3 ngrid(mx::kNormBlocks, (unsigned)batch);
  const bool vec = rows * cols % 4 == 0;
  if (g_bf16) {
    if (vec) hipLaunchKernelGGL((mx::k_ortho_norm<1, 4>), ngrid, dim3(256), 0, stream, in);
    else hipLaunchKernelGGL((mx::k_ortho_norm<1, 1>), ngrid, dim3(256), 0, stream, in);
  } else {
    if (vec) hipLaunchKernelGGL((mx::k_ortho_norm<0, 4>), ngrid, dim3(256), 0, stream, in);
    else hipLaunchKernelGGL((mx::k_ortho_norm<0, 1>), ngrid, dim3(256), 0, stream, in);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const dim3 igrid((unsigned)((in.cols_p + 63) / 64), (unsigned)((in.rows_p + 63) / 64), (unsigned)batch);
  if (g_bf16) hipLaunchKernelGGL((mx::k_ortho_init<1>), igrid, dim3(256), 0, stream, in);
  else hipLaunchKernelGGL((mx::k_ortho_init<0>), igrid, dim3(256), 0, stream, in);
  if ((e = hipGetLastError()) != hipSuccess) return e;

  mx::OrthoArgs p{};
  p.groups = (int)batch;
  p.M = w.R;
  p.L = w.L;
  p.x32 = in.x32; p.x16 = x16;
  p.o16 = (_Float16*)(base + w.o16);
  p.b16 = (_Float16*)(base + w.b16);
  p.sx = in.sx;
  p.out = out; p.rows = rows; p.cols = cols; p.tall = in.tall;
  for (int i = 0; i < steps; ++i) {
    p.ca = coefs[3 * i]; p.cb = coefs[3 * i + 1]; p.cc = coefs[3 * i + 2];
    p.part_in = i == 0 ? in.part0 : (const float*)(base + w.part[i & 1]);
    p.n_part = i == 0 ? 1 : (int)w.n_part;
    p.part_out = (float*)(base + w.part[(i + 1) & 1]);
    p.last = i + 1 == steps;
    p.xt16 = xt16[(i + 1) & 1];
    if ((e = square_product<mx::EP_GRAM>(p, w.L, x16, stream)) != hipSuccess) return e;
    if ((e = square_product<mx::EP_POLY>(p, w.R, p.o16, stream)) != hipSuccess) return e;
    if ((e = step_product(p, w.L, xt16[i & 1], stream)) != hipSuccess) return e;
  }
  return hipSuccess;
}
