// A whole mixture-of-experts layer for a few tokens (decoding), on expert weights kept as
// MXFP8 codes with MFMA-blocked scales or as bf16:
//   z = W1_e x_t (gate rows, then up rows), h = silu(z_gate) z_up, y_t = sum_j w_tj W2_e h
// over the topk experts e = ids[t, j] of token t that are held here.
//
// With few tokens the work is reading the chosen experts' weights once, so every kernel
// streams weight rows and brings the (small) activations to them:
//   up to 8 (16) tokens   k_moe_up: a block per chosen expert and 16 gate + 16 up rows; its
//                         eight waves take 128-element steps of the contraction in turn and
//                         add up through LDS. k_moe_down: a block per 16 output columns over
//                         all chosen experts, so that no output is summed outside its block
//   more                  k_moe_up_many, k_moe_down_many: the tokens' values go through LDS
//                         and serve 128 weight rows; k_moe_sum adds the splits' partials
// Routing is a wave per token (topk rounds of a wave maximum): inside k_moe_up for up to 8
// tokens, else k_moe_route. Every sum has an order that depends on the routing alone.
//
// Bound by HBM up to 64 tokens. 32 experts, hidden 7168, ffn 2048, top 8: one token 75 us (k_moe_up
// 48, k_moe_down 29) for 363 MB, 4.8 TB/s; 64 tokens 294 us (183 + 115 + 5 + 5) for 1.45 GB, 4.9
// TB/s, where a 1 GiB device copy moves 5.05 TB/s; bf16 weights 150 us for 705 MB and 660 us for
// 2.8 GB. Above, by the latency of each step's loads (see k_moe_up_many): 200 tokens 496 us, 2.9
// TB/s, and 811 with bf16 weights; 109 tokens of 128 experts of 704 x 384 61 us, 1.7 TB/s.
// The products run on v_mfma_f32_16x16x32_bf16 with weight rows as the first operand and
// tokens as the second (up to 16 tokens per instruction): codes become bf16 in registers,
// exactly (E4M3 times a power of two; scale bytes 0 to 2 reach below bf16's smallest number, and
// codes lose bits there), x is bf16 as given, and h goes to the second product
// as the sum of two bf16 values (16 bits of significand), since one alone would cost as much
// accuracy as the rounding of the result.

#include <algorithm>
#include <cfloat>
#include <cmath>

#include "../../include/mxfp8.h"
#include "common.h"
#include "moe.h"

namespace mx {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

enum { W_MXFP8 = 0, W_BF16 = 1 };

// An order-preserving unsigned key of a logit: larger logit, larger key; -0 as +0, NaN as
// -infinity. Every key is above 0, which marks what is taken or absent.
__device__ inline unsigned logit_key(float v) {
  v = v != v ? -INFINITY : v + 0.0f;
  const unsigned b = __builtin_bit_cast(unsigned, v);
  return (b >> 31) ? ~b : (b | 0x80000000u);
}
__device__ inline float key_logit(unsigned k) {
  return __builtin_bit_cast(float, (k >> 31) ? (k ^ 0x80000000u) : ~k);
}

// The maximum over the wave, in DPP moves (the running maximum of rows of 16 lanes, then of
// the rows), read from lane 63: a shuffle through LDS per step takes ten times as long.
__device__ inline unsigned wave_max(unsigned v) {
#define MX_DPP_MAX(ctrl, rows) v = umax(v, (unsigned)__builtin_amdgcn_update_dpp(0, (int)v, ctrl, rows, 0xf, false))
  MX_DPP_MAX(0x111, 0xf);
  MX_DPP_MAX(0x112, 0xf);
  MX_DPP_MAX(0x114, 0xf);
  MX_DPP_MAX(0x118, 0xf);
  MX_DPP_MAX(0x142, 0xa);  // lane 15 of rows 0, 2 into rows 1, 3
  MX_DPP_MAX(0x143, 0xc);  // lane 31 into rows 2, 3
#undef MX_DPP_MAX
  return (unsigned)__builtin_amdgcn_readlane((int)v, 63);
}
__device__ inline float wave_sum(float v) {
#pragma unroll
  for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

// One wave: the topk experts of a token. Lane j < topk gets the j-th id and its weight.
// R = 64-expert registers per lane.
template <int R>
__device__ inline void route_token(const MoeArgs& p, int t, int& id, float& weight) {
  const int l = threadIdx.x & 63;
  unsigned key[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int e = 64 * i + l;
    key[i] = e < p.experts ? logit_key(p.logits[t * p.ld_logits + e]) : 0u;
  }
  unsigned top = 0;  // lane j: the key of the j-th choice
  id = -1;
  float all = 0.f;  // softmax: the sum over every expert
  float mx = 0.f;
  for (int j = 0; j < p.topk; ++j) {
    unsigned m = key[0];
#pragma unroll
    for (int i = 1; i < R; ++i) m = umax(m, key[i]);
    m = wave_max(m);
    if (j == 0) {
      // an infinite logit counts as the largest finite one, so that differences stay numbers
      mx = fminf(key_logit(m), FLT_MAX);
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < R; ++i)
        if (key[i]) s += __expf(fminf(key_logit(key[i]), FLT_MAX) - mx);
      all = wave_sum(s);
    }
    // the lowest index among equals
    bool found = false;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const uint64_t eq = __ballot(key[i] == m);
      if (!found && eq) {
        found = true;
        const int at = __ffsll((long long)eq) - 1;
        if (l == j) {
          id = 64 * i + at;
          top = m;
        }
        if (l == at) key[i] = 0;
      }
    }
  }
  const float lg = l < p.topk ? fminf(key_logit(top), FLT_MAX) : -INFINITY;
  float s;
  if (p.score == 0)
    s = lg == -INFINITY ? 0.f : __expf(lg - mx);
  else
    s = lg == -INFINITY ? 0.f : 1.f / (1.f + __expf(-lg));
  float den = p.score == 0 ? all : 1.f;
  if (p.renorm) den = wave_sum(s);
  weight = s > 0.f ? p.scale * (s / den) : 0.f;  // nothing to choose from: weight 0
}

template <int R>
__global__ __launch_bounds__(256) void k_moe_route(MoeArgs p) {
  const int t = blockIdx.x * 4 + (threadIdx.x >> 6), l = threadIdx.x & 63;
  if (t >= p.tokens) return;
  int id;
  float w;
  route_token<R>(p, t, id, w);
  if (l < p.topk) {
    p.ids[t * p.topk + l] = id;
    p.weights[t * p.topk + l] = w;
  }
}

constexpr int kWaves = 8;

// The chosen experts held here, as a bitmap in LDS: an expert counts as chosen when a choice
// of tokens [t0, t1) with a weight other than 0 names it.
__device__ inline void mark_chosen(const MoeArgs& p, int t0, int t1, unsigned* bits) {
  if (threadIdx.x < 32) bits[threadIdx.x] = 0;
  __syncthreads();
  for (int i = t0 * p.topk + threadIdx.x; i < t1 * p.topk; i += 64 * kWaves) {
    const int e = p.ids[i] - p.first;
    if (e >= 0 && e < p.local && p.weights[i] != 0.f) atomicOr(&bits[e >> 5], 1u << (e & 31));
  }
  __syncthreads();
}

// The a-th set bit of the bitmap (every wave on its own), -1 if there are no more; `count`:
// set bits in all.
__device__ inline int nth_chosen(const unsigned* bits, int a, int& count) {
  const int l = threadIdx.x & 63;
  const unsigned w = l < 32 ? bits[l] : 0u;
  int c = __popc(w);
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up(c, d);
    if (l >= d) c += o;
  }
  count = __builtin_amdgcn_readlane(c, 31);
  if (a >= count) return -1;
  const uint64_t past = __ballot(l < 32 && c > a);
  const int word = __ffsll((long long)past) - 1;
  unsigned v = (unsigned)__builtin_amdgcn_readlane((int)w, word);
  int skip = a - (__builtin_amdgcn_readlane(c, word) - __popc(v));
  while (skip--) v &= v - 1;
  return __builtin_amdgcn_readfirstlane(word * 32 + __ffs((int)v) - 1);
}

// One 128-element step of the contraction for 16 weight rows: lane l holds row l % 16 and
// the 32-element block l / 16 of the step, as raw memory (2 or 4 16-byte loads).
template <int W>
struct RawBlock {
  u32x4 d[W == W_MXFP8 ? 2 : 4];
  int byte;
};

// A lane's row of one expert's matrix: uniform bases, so that the step goes into scalar
// registers, and a lane's own 32-bit offsets (one expert's matrix is below 2^31 bytes).
template <int W>
struct Rows {
  const uint8_t *w, *s;
  unsigned w_off, s_off;
  int blocks;  // 32-element blocks of a row
};

// Row `row` (a lane's own) of expert e's matrix [rows x cols].
template <int W>
__device__ inline Rows<W> expert_rows(const uint8_t* w, const uint8_t* s, int e, int64_t rows, int64_t cols, int row) {
  constexpr int ES = W == W_MXFP8 ? 1 : 2;
  const int g = (threadIdx.x & 63) >> 4;
  const int64_t kt = scale_tiles_k(cols / 32);
  Rows<W> r;
  r.w = w + (int64_t)e * rows * cols * ES;
  r.w_off = (unsigned)row * (unsigned)(cols * ES) + (unsigned)(g * 32 * ES);
  r.blocks = (int)(cols / 32);
  r.s = s + scale_tile_base((int64_t)e * rows / 32, 0, kt);
  // block 4 s + g of the row: scale tile s / 2, byte as scale_in_tile places it
  r.s_off = (unsigned)(row >> 5) * (unsigned)(kt * 256) + (unsigned)scale_in_tile(row & 31, g);
  return r;
}

template <int W>
__device__ inline RawBlock<W> load_block(const Rows<W>& r, int s) {
  constexpr int N = W == W_MXFP8 ? 2 : 4, ES = W == W_MXFP8 ? 1 : 2;
  RawBlock<W> o;
  const bool in = 4 * s + (int)((threadIdx.x & 63) >> 4) < r.blocks;
  const uint8_t* w = r.w + (int64_t)s * (128 * ES);
#pragma unroll
  for (int i = 0; i < N; ++i) o.d[i] = in ? *(const u32x4*)(w + (r.w_off + 16 * i)) : (u32x4){0, 0, 0, 0};
  o.byte = 127;
  if (W == W_MXFP8 && in) o.byte = (r.s + ((s >> 1) * 256 + (s & 1) * 2))[r.s_off];
  return o;
}

// The block's 32 elements as four bf16 operands of eight.
template <int W>
__device__ inline void to_bf16(const RawBlock<W>& r, bf16x8 o[4]) {
  if constexpr (W == W_BF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = __builtin_bit_cast(bf16x8, r.d[i]);
  } else {
    const float sc = scale_operand(r.byte);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      unsigned v[4];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const unsigned c = r.d[i >> 1][(i & 1) * 2 + j];
        v[2 * j] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, sc, false));
        v[2 * j + 1] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, sc, true));
      }
      o[i] = __builtin_bit_cast(bf16x8, (u32x4){v[0], v[1], v[2], v[3]});
    }
  }
}

__device__ inline v4f mfma16(bf16x8 a, bf16x8 b, v4f c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

constexpr int kMaxTopk = MX_MOE_MAX_TOPK, kMaxExperts = MX_MOE_MAX_EXPERTS;

// h as its bf16 rounding and the rest (0 where the rounding is infinite).
__device__ inline void split_h(float h, float& hi, float& lo) {
  hi = __builtin_bit_cast(float, bf16x2_rne(h, 0.f) << 16);
  lo = fabsf(hi) == INFINITY ? 0.f : h - hi;
}
__device__ inline void store_h(const MoeArgs& p, int slot, int64_t f, float gate, float up) {
  float hi, lo;
  split_h(gate / (1.f + __expf(-gate)) * up, hi, lo);
  uint16_t* dst = p.h + (int64_t)slot * 2 * p.ffn + f;
  dst[0] = (uint16_t)bf16x2_rne(hi, 0.f);
  dst[p.ffn] = (uint16_t)bf16x2_rne(lo, 0.f);
}
// the same for four consecutive values
__device__ inline void store_h4(const MoeArgs& p, int slot, int64_t f, v4f gate, v4f up) {
  float hi[4], lo[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) split_h(gate[e] / (1.f + __expf(-gate[e])) * up[e], hi[e], lo[e]);
  uint16_t* dst = p.h + (int64_t)slot * 2 * p.ffn + f;
  *(u32x2*)dst = (u32x2){bf16x2_rne(hi[0], hi[1]), bf16x2_rne(hi[2], hi[3])};
  *(u32x2*)(dst + p.ffn) = (u32x2){bf16x2_rne(lo[0], lo[1]), bf16x2_rne(lo[2], lo[3])};
}

// one output value, with the residual
__device__ inline void store_y(const MoeArgs& p, int64_t o, float y) {
  if (p.residual) y += __builtin_bit_cast(float, (unsigned)p.residual[o] << 16);
  if (p.out_bf16)
    ((uint16_t*)p.out)[o] = (uint16_t)bf16x2_rne(y, 0.f);
  else
    ((float*)p.out)[o] = y;
}

// 16-byte chunk c of row r in a staged tile of 256-byte rows: sixteen rows at one chunk hit
// different banks
__device__ inline int staged(int r, int c) { return r * 16 + (c ^ (r & 15)); }

// ---- up to 16 tokens: the waves of a block share weight rows and split the contraction ----
// A wave issues the loads of a step DEPTH - 1 steps ahead, so that the weights in flight (16 waves
// of 2 KB a row tile and step on a compute unit) cover HBM's latency. The sets of registers are
// handed on by copies, which wait for the loads into them: as compiled a wave waits for all of
// its loads once a step, and it is the number of waves that keeps HBM busy. The tokens' values
// of a step are loaded as whole 256-byte rows, TQ 16-byte pieces a lane (4 rows each), and turned to the
// matrix operand's layout through a piece of LDS of the wave's own. Columns past the expert's
// tokens hold anything: a column of the product depends on its own token alone.

// Sets of registers: MXFP8 at 128 registers and two blocks on a compute unit; bf16 steps are
// twice as large and take 256 registers and one block. (k_moe_down at 16 columns spills, 10
// registers with MXFP8 weights and 3 with bf16.)
constexpr int few_waves(int w) { return w == W_MXFP8 ? 4 : 2; }
constexpr int up_depth(int w, int tq) { return w == W_BF16 || tq == 1 ? 3 : 2; }
constexpr int down_depth(int w, int tq) { return w == W_BF16 ? 4 : tq == 1 ? 4 : tq == 2 ? 3 : 2; }

// T <= 8: wave t of every block routes token t itself, which costs less than a launch; the
// choices and weights of all tokens into LDS, and from the first block also to memory.
__device__ inline void route_in_block(const MoeArgs& p, int* ids, float* weights) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = threadIdx.x & 63;
  if (wave < p.tokens) {
    int id;
    float w;
    if (p.experts <= 64) route_token<1>(p, wave, id, w);
    else if (p.experts <= 256) route_token<4>(p, wave, id, w);
    else route_token<16>(p, wave, id, w);
    if (l < p.topk) {
      ids[wave * p.topk + l] = id;
      weights[wave * p.topk + l] = w;
      if (blockIdx.x == 0 && blockIdx.y == 0) {
        p.ids[wave * p.topk + l] = id;
        p.weights[wave * p.topk + l] = w;
      }
    }
  }
}

// The choices to compute, as local experts (-1: not here, or weight 0), and the bitmap of the
// chosen ones.
__device__ inline void take_choices(const MoeArgs& p, const int32_t* ids, const float* weights, short* choice,
                                    unsigned* bits) {
  if (threadIdx.x < 32) bits[threadIdx.x] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < p.tokens * p.topk; i += 64 * kWaves) {
    const int e = ids[i] - p.first;
    const bool take = e >= 0 && e < p.local && weights[i] != 0.f;
    choice[i] = (short)(take ? e : -1);
    if (take) atomicOr(&bits[e >> 5], 1u << (e & 31));
  }
  __syncthreads();
}

// The entries of `choice` that name e, into this wave's list: their number.
__device__ inline int list_tokens(const short* choice, int entries, int e, int* list) {
  const int l = threadIdx.x & 63;
  int n = 0;
  for (int i0 = 0; i0 < entries; i0 += 64) {
    const bool hit = i0 + l < entries && choice[i0 + l] == e;
    const uint64_t b = __ballot(hit);
    if (hit) list[n + __popcll(b & ((1ull << l) - 1))] = i0 + l;
    n += __popcll(b);
  }
  // LDS takes a wave's accesses in order; the fence keeps the compiler from moving them
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  return n;
}

// One block per chosen expert and 16 gate + 16 up rows.
template <int W, int TQ>
__global__ __launch_bounds__(64 * kWaves, few_waves(W)) void k_moe_up(MoeArgs p) {
  constexpr int DEPTH = up_depth(W, TQ);
  __shared__ unsigned bits[32];
  __shared__ short choice[16 * kMaxTopk];
  __shared__ int own_ids[8 * kMaxTopk];
  __shared__ float own_weights[8 * kMaxTopk];
  __shared__ int lists[kWaves][16];
  __shared__ u32x4 stage[kWaves][TQ * 4 * 16];
  __shared__ v4f part[kWaves][2][64];
  const int tid = threadIdx.x, l = tid & 63, g = l >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  if (p.tokens <= 8) {
    route_in_block(p, own_ids, own_weights);
    __syncthreads();
    take_choices(p, own_ids, own_weights, choice, bits);
  } else {
    take_choices(p, p.ids, p.weights, choice, bits);
  }
  int count;
  const int e = nth_chosen(bits, blockIdx.y, count);
  if (e < 0) return;
  int* list = lists[wave];
  const int n = list_tokens(choice, p.tokens * p.topk, e, list);
  const int steps = (int)((p.hidden + 127) / 128);
  const int row = blockIdx.x * 16 + (l & 15);
  const Rows<W> rg = expert_rows<W>(p.w1, p.w1_s, e, 2 * p.ffn, p.hidden, row);
  const Rows<W> ru = expert_rows<W>(p.w1, p.w1_s, e, 2 * p.ffn, p.hidden, row + (int)p.ffn);
  unsigned xs[TQ];  // element offset of a token's row, ~0: no token
#pragma unroll
  for (int i = 0; i < TQ; ++i)
    xs[i] = 4 * i + g < n ? (unsigned)(list[4 * i + g] / p.topk) * (unsigned)p.ld_x + (l & 15) * 8 : ~0u;
  struct Flight {
    u32x4 x[TQ];
    RawBlock<W> wg, wu;
  };
  auto load = [&](Flight& o, int s) {
    const bool in = s * 128 + (l & 15) * 8 < p.hidden;
#pragma unroll
    for (int i = 0; i < TQ; ++i)
      o.x[i] = xs[i] != ~0u && in ? *(const u32x4*)(p.x + s * 128 + xs[i]) : (u32x4){0, 0, 0, 0};
    o.wg = load_block<W>(rg, s);
    o.wu = load_block<W>(ru, s);
  };
  v4f ag = (v4f){0.f, 0.f, 0.f, 0.f}, au = ag;
  Flight f[DEPTH];
#pragma unroll
  for (int d = 0; d < DEPTH - 1; ++d)
    if (wave + d * kWaves < steps) load(f[d], wave + d * kWaves);
#pragma unroll 1
  for (int s = wave; s < steps; s += kWaves) {
    if (s + (DEPTH - 1) * kWaves < steps) load(f[DEPTH - 1], s + (DEPTH - 1) * kWaves);
#pragma unroll
    for (int i = 0; i < TQ; ++i) stage[wave][staged(4 * i + g, l & 15)] = f[0].x[i];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    bf16x8 b[4], w[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) b[q] = __builtin_bit_cast(bf16x8, stage[wave][staged(l & (4 * TQ - 1), 4 * g + q)]);
    to_bf16<W>(f[0].wg, w);
#pragma unroll
    for (int q = 0; q < 4; ++q) ag = mfma16(w[q], b[q], ag);
    to_bf16<W>(f[0].wu, w);
#pragma unroll
    for (int q = 0; q < 4; ++q) au = mfma16(w[q], b[q], au);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
    for (int d = 0; d + 1 < DEPTH; ++d) f[d] = f[d + 1];
  }
  part[wave][0][l] = ag;
  part[wave][1][l] = au;
  __syncthreads();
  // lane l, register r of a tile: row 4 (l / 16) + r, column l % 16
  const int r = tid & 15, col = tid >> 4;
  if (tid < 256 && col < n) {
    const int at = (r >> 2) * 16 + col;
    float zg = 0.f, zu = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      zg += part[w][0][at][r & 3];
      zu += part[w][1][at][r & 3];
    }
    store_h(p, list[col], blockIdx.x * 16 + r, zg, zu);
  }
}

constexpr int kTotPitch = 20;  // floats per token in a wave's running sums: 16 rows and 4 that spread the banks

// One block per 16 output columns; the waves split the chosen experts' contractions, laid end to end.
template <int W, int TQ>
__global__ __launch_bounds__(64 * kWaves, few_waves(W)) void k_moe_down(MoeArgs p) {
  constexpr int DEPTH = down_depth(W, TQ);
  __shared__ unsigned bits[32];
  __shared__ short choice[16 * kMaxTopk];
  __shared__ int lists[kWaves][16];
  __shared__ u32x4 stage[kWaves][2][TQ * 4 * 16];  // high and low parts of h
  __shared__ __attribute__((aligned(16))) float tot[kWaves][TQ * 4][kTotPitch];
  const int tid = threadIdx.x, l = tid & 63, g = l >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int steps = (int)((p.ffn + 127) / 128);
  const int entries = p.tokens * p.topk;
  for (int i = l; i < TQ * 4 * kTotPitch; i += 64) (&tot[wave][0][0])[i] = 0.f;
  take_choices(p, p.ids, p.weights, choice, bits);
  int count;
  nth_chosen(bits, 0, count);
  const int64_t total = (int64_t)count * steps;
  const int beg = (int)(total * wave / kWaves), end = (int)(total * (wave + 1) / kWaves);
  // where the loads are: step s of the a-th chosen expert, its weight row, this lane's rows of h
  int a = beg / steps, s = beg - a * steps, slot = -1;
  Rows<W> rows = expert_rows<W>(p.w2, p.w2_s, 0, p.hidden, p.ffn, blockIdx.x * 16 + (l & 15));
  unsigned hs[TQ];  // element offset of a slot's high parts, ~0: none
  auto expert = [&]() {
    int cnt;
    const int e = nth_chosen(bits, a, cnt);
    rows = expert_rows<W>(p.w2, p.w2_s, e, p.hidden, p.ffn, blockIdx.x * 16 + (l & 15));
    int* list = lists[wave];
    const int n = list_tokens(choice, entries, e, list);
    slot = (l & 15) < n ? list[l & 15] : -1;
#pragma unroll
    for (int i = 0; i < TQ; ++i)
      hs[i] = 4 * i + g < n ? (unsigned)list[4 * i + g] * (unsigned)(2 * p.ffn) + (l & 15) * 8 : ~0u;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  };
  struct Flight {
    u32x4 h[TQ][2];
    RawBlock<W> w;
    int slot;
    bool last;  // of its expert, or of this wave's share
  };
  auto load = [&](Flight& o, int at) {
    const bool in = s * 128 + (l & 15) * 8 < p.ffn;
#pragma unroll
    for (int i = 0; i < TQ; ++i)
#pragma unroll
      for (int q = 0; q < 2; ++q)
        o.h[i][q] = hs[i] != ~0u && in ? *(const u32x4*)(p.h + q * p.ffn + s * 128 + hs[i]) : (u32x4){0, 0, 0, 0};
    o.w = load_block<W>(rows, s);
    o.slot = slot;
    o.last = s + 1 == steps || at + 1 == end;
    if (++s == steps && at + 1 < end) {
      s = 0;
      ++a;
      expert();
    }
  };
  v4f acc = (v4f){0.f, 0.f, 0.f, 0.f};
  Flight f[DEPTH];
  if (beg < end) expert();
#pragma unroll
  for (int d = 0; d < DEPTH - 1; ++d)
    if (beg + d < end) load(f[d], beg + d);
#pragma unroll 1
  for (int at = beg; at < end; ++at) {
    if (at + DEPTH - 1 < end) load(f[DEPTH - 1], at + DEPTH - 1);
#pragma unroll
    for (int i = 0; i < TQ; ++i)
#pragma unroll
      for (int q = 0; q < 2; ++q) stage[wave][q][staged(4 * i + g, l & 15)] = f[0].h[i][q];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    bf16x8 w[4];
    to_bf16<W>(f[0].w, w);
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int part = 0; part < 2; ++part)
        acc = mfma16(w[q], __builtin_bit_cast(bf16x8, stage[wave][part][staged(l & (4 * TQ - 1), 4 * g + q)]), acc);
    if (f[0].last) {  // this wave's part of the expert's product, into its tokens' sums
      const int now = f[0].slot;
      if (now >= 0) *(v4f*)&tot[wave][now / p.topk][g * 4] += p.weights[now] * acc;
      acc = (v4f){0.f, 0.f, 0.f, 0.f};
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
    for (int d = 0; d + 1 < DEPTH; ++d) f[d] = f[d + 1];
  }
  __syncthreads();
  if (tid < p.tokens * 16) {
    const int t = tid >> 4, r = tid & 15;
    float y = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) y += tot[w][t][r];
    store_y(p, (int64_t)t * p.hidden + blockIdx.x * 16 + r, y);
  }
}

// ---- more tokens: the waves of a block share the tokens, in LDS, and split the weight rows ----
// With 16 tokens to an expert a wave that streams 16 rows of codes needs as many bytes of x,
// and four times as many of h: read through LDS, each of them comes from L2 once per 128
// rows. Loads are issued two steps ahead of their use; handing the sets of registers on by copies
// waits for them at the end of each step, so a step costs the latency of its loads.

constexpr int kChunk = 64;    // tokens per pass of the kernels below
// k_moe_down_many: token tiles of one run (an expert with more tokens takes several). Four with
// MXFP8 weights spill 8 registers around the start of a run.
constexpr int down_tiles(bool in_lds) { return in_lds ? 2 : 4; }

// One block per chosen expert and 64 gate + 64 up rows: waves 0-3 take the gate rows, 4-7 the up rows.
template <int W>
__global__ __launch_bounds__(64 * kWaves, few_waves(W)) void k_moe_up_many(MoeArgs p) {
  constexpr int NT = kChunk / 16;
  __shared__ unsigned bits[32];
  __shared__ int n_list;
  __shared__ int list[256];
  __shared__ u32x4 stage[2][kChunk * 16];
  const int tid = threadIdx.x, l = tid & 63, g = l >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  mark_chosen(p, 0, p.tokens, bits);
  int count;
  const int e = nth_chosen(bits, blockIdx.y, count);
  if (e < 0) return;
  if (tid == 0) n_list = 0;
  __syncthreads();
  for (int i = tid; i < p.tokens * p.topk; i += 64 * kWaves)
    if (p.ids[i] - p.first == e && p.weights[i] != 0.f) list[atomicAdd(&n_list, 1)] = i;
  __syncthreads();
  const int n = n_list;
  const int steps = (int)((p.hidden + 127) / 128);
  const int64_t f0 = (int64_t)blockIdx.x * 64 + (wave & 3) * 16;
  const int64_t f_row = f0 + (l & 15) < p.ffn ? f0 + (l & 15) : p.ffn - 1;
  const Rows<W> rows = expert_rows<W>(p.w1, p.w1_s, e, 2 * p.ffn, p.hidden, (int)((wave >> 2) * p.ffn + f_row));
  for (int c0 = 0; c0 < n; c0 += kChunk) {
    const int nn = n - c0 < kChunk ? n - c0 : kChunk;
    struct Flight {
      RawBlock<W> w;
      u32x4 x[2];
    };
    const uint16_t* xs[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = 32 * i + (tid >> 4);
      xs[i] = r < nn ? p.x + (int64_t)(list[c0 + r] / p.topk) * p.ld_x : nullptr;
    }
    auto load = [&](Flight& o, int s) {
      const int64_t k = (int64_t)s * 128 + (tid & 15) * 8;
#pragma unroll
      for (int i = 0; i < 2; ++i)
        o.x[i] = xs[i] && k < p.hidden ? *(const u32x4*)(xs[i] + k) : (u32x4){0, 0, 0, 0};
      o.w = load_block<W>(rows, s);
    };
    auto put = [&](const Flight& o, int buf) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (32 * i < nn) stage[buf][staged(32 * i + (tid >> 4), tid & 15)] = o.x[i];
    };
    v4f acc[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) acc[i] = (v4f){0.f, 0.f, 0.f, 0.f};
    Flight cur, nxt, far;
    load(cur, 0);
    if (steps > 1) load(nxt, 1);
    put(cur, 0);
    __syncthreads();
    for (int s = 0; s < steps; ++s) {
      if (s + 2 < steps) load(far, s + 2);
      bf16x8 w[4];
      to_bf16<W>(cur.w, w);
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        if (16 * i >= nn) break;
#pragma unroll
        for (int q = 0; q < 4; ++q)
          acc[i] = mfma16(w[q], __builtin_bit_cast(bf16x8, stage[s & 1][staged(16 * i + (l & 15), 4 * g + q)]), acc[i]);
      }
      if (s + 1 < steps) put(nxt, (s + 1) & 1);
      __syncthreads();
      cur = nxt;
      nxt = far;
    }
    // the up halves go to the waves that hold the gates
    v4f* part = (v4f*)&stage[0][0];
    if (wave >= 4)
#pragma unroll
      for (int i = 0; i < NT; ++i) part[((wave - 4) * NT + i) * 64 + l] = acc[i];
    __syncthreads();
    const int64_t f = f0 + 4 * g;
    if (wave < 4 && f < p.ffn)
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const int c = 16 * i + (l & 15);
        if (c < nn) store_h4(p, list[c0 + c], f, acc[i], part[(wave * NT + i) * 64 + l]);
      }
    __syncthreads();
  }
}

// One block per 128 output columns and split of the work: the chosen experts' contractions,
// run after run (an expert with more than RUN tokens takes several runs), are cut evenly into
// p.splits pieces; each writes its sums as one partial, [splits][tokens][hidden]. A wave's
// sums of up to 64 tokens stay in LDS; more are added up in the partial itself: a value belongs
// to one wave, which reads, adds and writes it in the order of its runs.
template <int W, bool IN_LDS>
__global__ __launch_bounds__(64 * kWaves, few_waves(W)) void k_moe_down_many(MoeArgs p) {
  constexpr int HT = down_tiles(IN_LDS), RUN = 16 * HT;
  __shared__ int n_runs;
  __shared__ int lists[4][kWaves][RUN];  // of the run in use and of the three (of one step each) loaded ahead
  __shared__ u32x4 stage[2][2][RUN * 16];  // high and low parts of h
  __shared__ __attribute__((aligned(16))) float tot[IN_LDS ? kWaves : 1][IN_LDS ? kChunk : 1][16];
  extern __shared__ int more[];
  int* runs = more;  // [local + entries / RUN]: expert + 1024 * (which RUN of its tokens)
  const int entries = p.tokens * p.topk;
  short* choice = (short*)(more + p.local + entries / RUN);  // [entries]
  int* cnt = (int*)&stage[0][0][0];  // [kMaxExperts] while the runs are laid out
  const int tid = threadIdx.x, l = tid & 63, g = l >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int steps = (int)((p.ffn + 127) / 128);
  const int64_t wrow = (int64_t)blockIdx.x * 128 + wave * 16;  // the wave's first output column
  const int64_t row0 = wrow + (l & 15) < p.hidden ? wrow + (l & 15) : p.hidden - 1;
  float* part = p.part + (int64_t)blockIdx.y * p.tokens * p.hidden;
  if constexpr (IN_LDS) {
    for (int i = l; i < kChunk * 16; i += 64) (&tot[wave][0][0])[i] = 0.f;
  } else {
    for (int i = tid; i < p.tokens * 32; i += 64 * kWaves) {
      const int64_t col = (int64_t)blockIdx.x * 128 + (i & 31) * 4;
      if (col < p.hidden) *(v4f*)(part + (i >> 5) * p.hidden + col) = (v4f){0.f, 0.f, 0.f, 0.f};
    }
  }
  for (int i = tid; i < p.local; i += 64 * kWaves) cnt[i] = 0;
  __syncthreads();
  for (int i = tid; i < entries; i += 64 * kWaves) {
    const int e = p.ids[i] - p.first;
    const bool take = e >= 0 && e < p.local && p.weights[i] != 0.f;
    choice[i] = (short)(take ? e : -1);
    if (take) atomicAdd(&cnt[e], 1);
  }
  __syncthreads();
  if (wave == 0) {
    int at = 0;
    for (int e0 = 0; e0 < p.local; e0 += 64) {
      const int parts = e0 + l < p.local ? (cnt[e0 + l] + RUN - 1) / RUN : 0;
      int before = parts;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(before, d);
        if (l >= d) before += o;
      }
      for (int i = 0; i < parts; ++i) runs[at + before - parts + i] = e0 + l + 1024 * i;
      at += __builtin_amdgcn_readlane(before, 63);
    }
    if (l == 0) n_runs = at;
  }
  __syncthreads();
  const int64_t total = (int64_t)n_runs * steps;
  const int beg = (int)(total * blockIdx.y / p.splits), end = (int)(total * (blockIdx.y + 1) / p.splits);
  struct Flight {
    RawBlock<W> w;
    u32x4 h[HT];
    int n, list;  // tokens of the run, and which of the lists holds them
    bool last;    // of its run, or of this block's piece
  };
  // where the loads are: step s of run a, that run's weight row and tokens
  int a = beg / steps, s = beg - a * steps, n = 0, which = 0;
  Rows<W> rows = expert_rows<W>(p.w2, p.w2_s, 0, p.hidden, p.ffn, (int)row0);
  // this thread's part of the tile: high or low part, token (tid / 16) % 16 of each 16, chunk tid % 16
  const int part_of = tid >> 8, tok = (tid >> 4) & 15;
  unsigned hs[HT];  // element offset of a slot's part, ~0: none
  auto start = [&]() {
    which = (which + 1) & 3;
    int* list = lists[which][wave];
    const int run = __builtin_amdgcn_readfirstlane(runs[a]), e = run & 1023, skip = (run >> 10) * RUN;
    rows = expert_rows<W>(p.w2, p.w2_s, e, p.hidden, p.ffn, (int)row0);
    int seen = 0;
    for (int i0 = 0; i0 < entries; i0 += 64) {
      const bool hit = i0 + l < entries && choice[i0 + l] == e;
      const uint64_t b = __ballot(hit);
      const int at = seen + __popcll(b & ((1ull << l) - 1)) - skip;
      if (hit && at >= 0 && at < RUN) list[at] = i0 + l;
      seen += __popcll(b);
    }
    n = seen - skip < RUN ? seen - skip : RUN;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
    for (int i = 0; i < HT; ++i)
      hs[i] = 16 * i + tok < n ? ((unsigned)list[16 * i + tok] * 2 + part_of) * (unsigned)p.ffn + (tid & 15) * 8 : ~0u;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  };
  auto load = [&](Flight& o, int at) {
    const bool in = s * 128 + (tid & 15) * 8 < p.ffn;
#pragma unroll
    for (int i = 0; i < HT; ++i) o.h[i] = hs[i] != ~0u && in ? *(const u32x4*)(p.h + s * 128 + hs[i]) : (u32x4){0, 0, 0, 0};
    o.w = load_block<W>(rows, s);
    o.n = n;
    o.list = which;
    o.last = s + 1 == steps || at + 1 == end;
    if (++s == steps && at + 1 < end) {
      s = 0;
      ++a;
      start();
    }
  };
  auto put = [&](const Flight& o, int buf) {
#pragma unroll
    for (int i = 0; i < HT; ++i)
      if (16 * i < o.n) stage[buf][part_of][staged(16 * i + tok, tid & 15)] = o.h[i];
  };
  if (beg < end) {
    Flight cur, nxt, far;
    v4f acc[HT];
#pragma unroll
    for (int i = 0; i < HT; ++i) acc[i] = (v4f){0.f, 0.f, 0.f, 0.f};
    start();
    load(cur, beg);
    if (beg + 1 < end) load(nxt, beg + 1);
    put(cur, 0);
    __syncthreads();
    for (int at = beg; at < end; ++at) {
      const int buf = (at - beg) & 1;
      if (at + 2 < end) load(far, at + 2);
      bf16x8 w[4];
      to_bf16<W>(cur.w, w);
#pragma unroll
      for (int i = 0; i < HT; ++i) {
        if (16 * i >= cur.n) break;
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int half = 0; half < 2; ++half)
            acc[i] = mfma16(w[q], __builtin_bit_cast(bf16x8, stage[buf][half][staged(16 * i + (l & 15), 4 * g + q)]), acc[i]);
      }
      if (cur.last) {
        // The run's sums, into its tokens' sums (a run holds a token once). Places past the run
        // or past the columns read what the last ones do and write nothing: a branch around
        // each load would wait for each.
        const int64_t col = wrow + g * 4 < p.hidden ? wrow + g * 4 : p.hidden - 4;
        float share[HT];
        unsigned t[HT];
#pragma unroll
        for (int i = 0; i < HT; ++i) {
          const int at = 16 * i + (l & 15), slot = lists[cur.list][wave][at < cur.n ? at : cur.n - 1];
          share[i] = p.weights[slot];
          t[i] = slot / p.topk;
        }
        v4f sum[HT];
#pragma unroll
        for (int i = 0; i < HT; ++i) {
          if constexpr (IN_LDS) sum[i] = *(const v4f*)&tot[wave][t[i]][g * 4];
          else sum[i] = *(const v4f*)(part + col + t[i] * p.hidden);
        }
#pragma unroll
        for (int i = 0; i < HT; ++i) {
          sum[i] += share[i] * acc[i];
          if (16 * i + (l & 15) < cur.n) {
            if constexpr (IN_LDS) *(v4f*)&tot[wave][t[i]][g * 4] = sum[i];
            else if (wrow + g * 4 < p.hidden) *(v4f*)(part + col + t[i] * p.hidden) = sum[i];
          }
          acc[i] = (v4f){0.f, 0.f, 0.f, 0.f};
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      }
      if (at + 1 < end) put(nxt, buf ^ 1);
      __syncthreads();
      cur = nxt;
      nxt = far;
    }
  }
  if constexpr (IN_LDS) {
    __syncthreads();
    for (int i = tid; i < p.tokens * 128; i += 64 * kWaves) {
      const int t = i >> 7, c = i & 127;
      const int64_t col = (int64_t)blockIdx.x * 128 + c;
      if (col < p.hidden) part[(int64_t)t * p.hidden + col] = tot[c >> 4][t][c & 15];
    }
  }
}

// out = the partials' sum, in order, and the residual: four columns per thread.
__global__ __launch_bounds__(256) void k_moe_sum(MoeArgs p) {
  const int64_t n = (int64_t)p.tokens * p.hidden, i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= n) return;
  v4f y = *(const v4f*)(p.part + i);
#pragma unroll 4
  for (int s = 1; s < p.splits; ++s) y += *(const v4f*)(p.part + s * n + i);
#pragma unroll
  for (int e = 0; e < 4; ++e) store_y(p, i + e, y[e]);
}

// Which batches take the few-token kernels: up to 8 tokens, and up to 16 where an expert is
// below 4 MB and the launches weigh more than the streaming. Us, few / many: 8 tokens of 32
// experts of 7168 x 2048 243 / 261, 12 tokens 282 / 269, 16 tokens 296 / 276; 16 tokens of 16
// experts of 1024 x 512 24 / 26.
bool moe_few(int64_t tokens, int64_t hidden, int64_t ffn) {
  return tokens <= 8 || (tokens <= 16 && 3 * hidden * ffn < 4 << 20);
}

// Splits of k_moe_down_many: about two blocks per compute unit, but four 128-element steps to
// a split and 64 splits at most. (109 tokens, 128 experts of 704 x 384: 16 splits 83 us, 64 61
// us; 64 tokens, 16 experts of 1024 x 512, 64 steps in all: 16 splits 29 us, 64 33 us.)
int moe_splits(int64_t tokens, int64_t hidden, int64_t ffn, int64_t local, int64_t topk) {
  if (moe_few(tokens, hidden, ffn)) return 0;
  const int64_t tiles = (hidden + 127) / 128, steps = std::min(local, tokens * topk) * ((ffn + 127) / 128);
  return (int)std::max<int64_t>(1, std::min({512 / tiles, steps / 4, (int64_t)64}));
}

template <int W, int TQ>
hipError_t launch_moe_few(const MoeArgs& p, int chosen, hipStream_t stream) {
  hipLaunchKernelGGL((k_moe_up<W, TQ>), dim3((unsigned)(p.ffn / 16), (unsigned)chosen), dim3(64 * kWaves), 0, stream, p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((k_moe_down<W, TQ>), dim3((unsigned)(p.hidden / 16)), dim3(64 * kWaves), 0, stream, p);
  return hipGetLastError();
}

template <int W, bool IN_LDS>
hipError_t launch_moe_down_many(const MoeArgs& p, dim3 grid, hipStream_t stream) {
  auto bytes = [](int local, int entries) {  // runs, and the choices as 16-bit values
    return ((local + entries / (16 * down_tiles(IN_LDS))) * 4 + entries * 2 + 15) / 16 * 16;
  };
  static const hipError_t attr =
      hipFuncSetAttribute((const void*)k_moe_down_many<W, IN_LDS>, hipFuncAttributeMaxDynamicSharedMemorySize,
                          bytes(kMaxExperts, (IN_LDS ? kChunk : MX_MOE_MAX_TOKENS) * kMaxTopk));
  if (attr != hipSuccess) return attr;
  hipLaunchKernelGGL((k_moe_down_many<W, IN_LDS>), grid, dim3(64 * kWaves), bytes(p.local, p.tokens * p.topk), stream, p);
  return hipGetLastError();
}

template <int W>
hipError_t launch_moe_products(const MoeArgs& p, hipStream_t stream) {
  const int chosen = (int)(p.local < (int64_t)p.tokens * p.topk ? p.local : (int64_t)p.tokens * p.topk);
  if (!p.splits && p.tokens <= 4) return launch_moe_few<W, 1>(p, chosen, stream);
  if (!p.splits && p.tokens <= 8) return launch_moe_few<W, 2>(p, chosen, stream);
  if (!p.splits) return launch_moe_few<W, 4>(p, chosen, stream);
  hipLaunchKernelGGL((k_moe_up_many<W>), dim3((unsigned)((p.ffn + 63) / 64), (unsigned)chosen), dim3(64 * kWaves), 0,
                     stream, p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const dim3 grid((unsigned)((p.hidden + 127) / 128), (unsigned)p.splits);
  if ((e = p.tokens <= kChunk ? launch_moe_down_many<W, true>(p, grid, stream)
                              : launch_moe_down_many<W, false>(p, grid, stream)) != hipSuccess)
    return e;
  const int64_t n = (int64_t)p.tokens * p.hidden;
  hipLaunchKernelGGL(k_moe_sum, dim3((unsigned)((n / 4 + 255) / 256)), dim3(256), 0, stream, p);
  return hipGetLastError();
}

}  // namespace mx

// h, then the partials of the largest number of splits the sizes allow (any number of experts).
int64_t mx_moe_workspace_bytes(int64_t tokens, int64_t hidden, int64_t ffn, int topk) {
  return (tokens * topk * 2 * ffn * (int64_t)sizeof(uint16_t) + 255) / 256 * 256 +
         mx::moe_splits(tokens, hidden, ffn, MX_MOE_MAX_EXPERTS, topk) * tokens * hidden * (int64_t)sizeof(float);
}

hipError_t mx_launch_moe(mx::MoeArgs p, int bf16_weights, void* ws, hipStream_t stream) {
  if (p.tokens == 0) return hipSuccess;
  p.splits = mx::moe_splits(p.tokens, p.hidden, p.ffn, p.local, p.topk);
  p.h = (uint16_t*)ws;
  p.part = (float*)((uint8_t*)ws + ((int64_t)p.tokens * p.topk * 2 * p.ffn * (int64_t)sizeof(uint16_t) + 255) / 256 * 256);
  const dim3 grid((unsigned)((p.tokens + 3) / 4));
  if (!p.splits && p.tokens <= 8) {
  } else if (p.experts <= 64)  // up to 8 tokens are routed in k_moe_up
    hipLaunchKernelGGL(mx::k_moe_route<1>, grid, dim3(256), 0, stream, p);
  else if (p.experts <= 256)
    hipLaunchKernelGGL(mx::k_moe_route<4>, grid, dim3(256), 0, stream, p);
  else
    hipLaunchKernelGGL(mx::k_moe_route<16>, grid, dim3(256), 0, stream, p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  return bf16_weights ? mx::launch_moe_products<mx::W_BF16>(p, stream) : mx::launch_moe_products<mx::W_MXFP8>(p, stream);
}
