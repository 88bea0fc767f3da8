// The 4-bit K/V cache (gqe_kv4): storing rows, reading them back, and the
// decode attention over it.
//
// A row of d_head bf16 values is held as d_head codes of 4 bits (byte i:
// element 2i in the low half, 2i + 1 in the high half) and a (scale, zero)
// pair of bf16, value = zero + scale * code:
//   zero = min x,  scale = bf16((max x - min x) / 15),
//   code = clamp(round_half_even((x - zero) / scale), 0, 15).
// Every step of that is one IEEE fp32 operation, so the codes are the same
// wherever it is computed. A row with an infinity or NaN gets scale = zero =
// NaN: all of it reads as NaN.
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>

#include "gqe_internal.h"
#include "ptx.cuh"

namespace gqe {

namespace kv4_impl {

constexpr int kThreads = 256;

__device__ __forceinline__ float bf16_f(uint32_t v) { return __uint_as_float(v << 16); }

struct StoreArgs {
  const uint16_t* K;   // [B][G][T][dh]
  const uint16_t* V;
  uint16_t* Ko;        // read: the same layout
  uint16_t* Vo;
  gqe_kv4 c;
  const int32_t* start;
  int start0;          // without start
  const int32_t* count;
  int B, G, T;
};

// Cache row of (b, g, t), or -1: t is past the sequence's count, or the
// position is outside the cache (recorded, unless it is before position 0).
__device__ __forceinline__ long long cache_row(const StoreArgs& a, long long bg, int t) {
  const int b = static_cast<int>(bg / a.G);
  if (a.count != nullptr && t >= a.count[b]) return -1;
  const long long p = static_cast<long long>(a.start != nullptr ? a.start[b] : a.start0) + t;
  if (p < 0) return -1;
  if (p >= a.c.capacity) {
    set_status(GQE_ERR_DEVICE_CHECK);
    return -1;
  }
  return bg * a.c.capacity + p;
}

// This lane's 8 codes of a row, and the row's (scale, zero) word.
template <int LPR>
__device__ __forceinline__ uint32_t quantise(uint4 raw, uint32_t* meta) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  float x[8];
  float lo = INFINITY, hi = -INFINITY;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[i] = __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
    bad = bad || !(fabsf(x[i]) < INFINITY);
    lo = fminf(lo, x[i]);
    hi = fmaxf(hi, x[i]);
  }
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  const uint32_t group = ((1u << LPR) - 1u) << (threadIdx.x % 32 / LPR * LPR);
  if ((__ballot_sync(0xffffffffu, bad) & group) != 0u) {
    *meta = 0x7fff7fffu;
    return 0u;
  }
  // Halved throughout: max - min of two bf16 may pass the largest fp32, and
  // halving is exact.
  const uint16_t sb = __bfloat16_as_ushort(__float2bfloat16_rn(__fdiv_rn(0.5f * hi - 0.5f * lo, 7.5f)));
  const float s = bf16_f(sb), hs = 0.5f * s, hz = 0.5f * lo;
  *meta = sb | (__float_as_uint(lo) & 0xffff0000u);
  uint32_t codes = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float q = s > 0.0f ? fminf(fmaxf(rintf(__fdiv_rn(0.5f * x[i] - hz, hs)), 0.0f), 15.0f) : 0.0f;
    codes |= static_cast<uint32_t>(q) << (4 * i);
  }
  return codes;
}

// DH / 8 lanes per row: 16 bytes in, 4 bytes of codes out each.
template <int DH>
__global__ void __launch_bounds__(kThreads) append_kernel(StoreArgs a) {
  constexpr int LPR = DH / 8, ROWS = kThreads / LPR;
  pdl_wait();
  pdl_launch_dependents();
  const int l = threadIdx.x % LPR;
  const long long n = static_cast<long long>(a.B) * a.G * a.T;
  for (long long r0 = static_cast<long long>(blockIdx.x) * ROWS; r0 < n; r0 += static_cast<long long>(gridDim.x) * ROWS) {
    const long long r = r0 + threadIdx.x / LPR;
    const long long bg = r / a.T;
    const long long at = r < n ? cache_row(a, bg, static_cast<int>(r - bg * a.T)) : -1;
    uint4 k = make_uint4(0u, 0u, 0u, 0u), v = k;
    if (at >= 0) {
      k = __ldg(reinterpret_cast<const uint4*>(a.K + r * DH) + l);
      v = __ldg(reinterpret_cast<const uint4*>(a.V + r * DH) + l);
    }
    uint32_t mk, mv;
    const uint32_t ck = quantise<LPR>(k, &mk), cv = quantise<LPR>(v, &mv);
    if (at < 0) continue;
    reinterpret_cast<uint32_t*>(a.c.k_codes)[at * LPR + l] = ck;
    reinterpret_cast<uint32_t*>(a.c.v_codes)[at * LPR + l] = cv;
    if (l == 0) reinterpret_cast<uint2*>(a.c.meta)[at] = make_uint2(mk, mv);
  }
}

__device__ __forceinline__ uint4 decode8(uint32_t codes, uint32_t meta) {
  const float s = bf16_f(meta & 0xffffu), z = bf16_f(meta >> 16);
  float x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = fmaf(s, static_cast<float>((codes >> (4 * i)) & 15u), z);
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}

template <int DH>
__global__ void __launch_bounds__(kThreads) read_kernel(StoreArgs a) {
  constexpr int LPR = DH / 8, ROWS = kThreads / LPR;
  pdl_wait();
  pdl_launch_dependents();
  const int l = threadIdx.x % LPR;
  const long long n = static_cast<long long>(a.B) * a.G * a.T;
  for (long long r0 = static_cast<long long>(blockIdx.x) * ROWS; r0 < n; r0 += static_cast<long long>(gridDim.x) * ROWS) {
    const long long r = r0 + threadIdx.x / LPR;
    if (r >= n) break;
    const long long bg = r / a.T;
    const long long at = cache_row(a, bg, static_cast<int>(r - bg * a.T));
    if (at < 0) continue;
    const uint2 m = reinterpret_cast<const uint2*>(a.c.meta)[at];
    reinterpret_cast<uint4*>(a.Ko + r * DH)[l] = decode8(reinterpret_cast<const uint32_t*>(a.c.k_codes)[at * LPR + l], m.x);
    reinterpret_cast<uint4*>(a.Vo + r * DH)[l] = decode8(reinterpret_cast<const uint32_t*>(a.c.v_codes)[at * LPR + l], m.y);
  }
}

// ---------------------------------------------------------------------------
// Decode attention: o = softmax(q . K / sqrt(dh)) V over the sequence's keys.
//
// Bytes: d_head + 8 per key and KV group (codes of K and V, two (scale, zero)
// pairs), a quarter of the bf16 cache's 4 d_head. At that rate the CUDA cores
// would bound the kernel (two products and two conversions per element and
// head), so the products run on the tensor cores (mma.sync m16n8k16: with at
// most 16 query rows a 128-row tcgen05 tile would be nine tenths padding)
// and the codes become their operands by bit operations alone:
//  - Scores, keys x heads: a code n masked into the low mantissa bits of an
//    fp16 is the subnormal n 2^-24, exact; in the next four bits 16 n 2^-24,
//    undone in q. Of a row's 32-bit word that is one shift and four ANDs for
//    eight elements. q goes in as q 2^(14 - e), e the exponent of the head's
//    largest element: exact but for elements 2^-38 of that. Then
//    s = scale_k sum(q n) + zero_k sum(q) in fp32.
//  - Output, dims x heads, over the keys: 0x4300 | n is the bf16 128 + n. The
//    weight operand is p scale_v in bf16 (fp16 would not hold the range of the
//    scales), and sum p scale_v (128 + n) = sum p scale_v (n - 8) + 136 sum of
//    the same rounded weights (a product with ones); the rest, sum p (zero_v
//    + 8 scale_v), is kept in fp32. The rounding of p thus meets codes around
//    zero, |n - 8| <= 8.
//  - Heads sit in the even columns (up to 4 heads per group; else in all):
//    the scores' accumulator then holds one head per lane, and what the
//    softmax does per key is done once per lane and not twice.
//  - A transposed 8 x 8 move turns the weights from (key, head) to the second
//    product's (head, keys) order.
// Each warp streams its own tiles of 64 keys of the CTA's span by bulk copies
// through a ring of its own (no CTA-wide barrier in the loop) and keeps its
// own running maximum; the warps' states are joined at the end of the span
// and, with more than one span per sequence and group, by a second kernel.
constexpr int kAttnWarps = 8;
constexpr int kAttnThreads = 32 * kAttnWarps;
constexpr int kTile = 64;   // keys per warp tile
constexpr int kStages = 3;  // tiles in flight per warp
constexpr int kMinSpan = kTile * kAttnWarps;

struct AttnArgs {
  const uint16_t* Q;   // [B][G][k][dh]
  const uint16_t* Qs;  // [B][dh] or null
  gqe_kv4 c;
  const int32_t* lens;
  int len_add, B, G, T, k, H, spans, span;
  float* part_o;       // [B][G][spans][H][dh]
  float2* part_ml;     // [B][G][spans][H]
  uint16_t* out;
  int ldo;
  float scale_log2;
};

__device__ __forceinline__ int keys_of(const AttnArgs& a, int b) {
  const long long n = a.lens != nullptr ? static_cast<long long>(a.lens[b]) + a.len_add : a.T;
  return static_cast<int>(n < 0 ? 0 : n > a.T ? a.T : n);
}
__device__ __forceinline__ int heads_of_group(const AttnArgs& a, int g) { return a.k + (g == 0 && a.Qs != nullptr ? 1 : 0); }
__device__ __forceinline__ const uint16_t* query_row(const AttnArgs& a, int b, int g, int h, int dh) {
  return h < a.k ? a.Q + ((static_cast<long long>(b) * a.G + g) * a.k + h) * dh : a.Qs + static_cast<long long>(b) * dh;
}
__device__ __forceinline__ void store_out(const AttnArgs& a, int b, int g, int h, int d, int dh, float v) {
  const int col = h < a.k ? g * a.k + h : a.G * a.k;
  a.out[static_cast<long long>(b) * a.ldo + col * dh + d] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// Row r of a 16-key block holds key row_key(r): the order that keeps both the
// K reads (rows 0..3 and 4..7 together) and the V reads (even rows, odd rows
// together) on distinct banks (keys distinct mod 4).
__device__ __forceinline__ int row_key(int r) { return (0x57463120u >> (4 * (r & 7)) & 7) + (r & 8); }

template <int DH>
struct AttnShape {
  static constexpr int ROW = DH / 2;                       // bytes of a row's codes
  static constexpr int TILE_BYTES = kTile * (2 * ROW + 8);  // K, V, meta
  static constexpr int RING = kStages * TILE_BYTES;
  static constexpr int STATE = DH + 2;                     // floats of one head's state
  static constexpr size_t smem(int H) {
    const size_t ring = static_cast<size_t>(kAttnWarps) * RING, st = static_cast<size_t>(kAttnWarps) * H * STATE * 4;
    return (ring > st ? ring : st) + kAttnWarps * kStages * 8 + 16;
  }
};

// HPL: heads per lane (1: even columns, at most 4 heads; 2: all columns);
// NB: column blocks of 8 (2 only with HPL = 2).
template <int DH, int HPL, int NB>
__global__ void __launch_bounds__(kAttnThreads, 2) kv4_attn_kernel(AttnArgs a) {
  using S = AttnShape<DH>;
  constexpr int KS = DH / 16;  // k steps of the scores
  constexpr int MT = DH / 16;  // 16-row blocks of the output
  extern __shared__ __align__(128) uint8_t sm[];
  const int span = blockIdx.x, g = blockIdx.y % a.G, b = blockIdx.y / a.G;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, lr = lane >> 2, lc = lane & 3;
  const size_t state_bytes = static_cast<size_t>(kAttnWarps) * a.H * S::STATE * 4;
  const size_t data = static_cast<size_t>(kAttnWarps) * S::RING > state_bytes ? static_cast<size_t>(kAttnWarps) * S::RING : state_bytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + data);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + kAttnWarps * kStages);
  if (tid < kAttnWarps * kStages) mbar_init(bars + tid, 1u);
  if (tid == 0) *abort_flag = 0;
  fence_barrier_init();
  pdl_wait();  // q, lens and the newest rows come from earlier kernels
  pdl_launch_dependents();
  __syncthreads();
  const int n = keys_of(a, b), k0 = span * a.span;
  if (k0 >= n) {
    if (n == 0 && span == 0)
      for (int i = tid; i < heads_of_group(a, g) * DH; i += kAttnThreads) store_out(a, b, g, i / DH, i % DH, DH, 0.0f);
    return;
  }
  const int H = heads_of_group(a, g);
  const int k1 = min(n, k0 + a.span), tiles = (k1 - k0 + kTile - 1) / kTile;
  const long long row0 = (static_cast<long long>(b) * a.G + g) * a.c.capacity + k0;

  uint8_t* ring = sm + warp * S::RING;
  uint64_t* full = bars + warp * kStages;
  // Tile i of this warp: keys k0 + (warp + 8 i) 64 ..., at most to k1 (rounded
  // up to an even count: 16-byte pieces; the capacity is a multiple of 16).
  auto issue = [&](int i) {
    const int t = (warp + kAttnWarps * i) * kTile;
    const int nk = (min(kTile, k1 - k0 - t) + 1) & ~1;
    uint8_t* s = ring + (i % kStages) * S::TILE_BYTES;
    uint64_t* bar = full + i % kStages;
    mbar_arrive_expect_tx(bar, static_cast<uint32_t>(nk) * (2 * S::ROW + 8));
    bulk_load(s, a.c.k_codes + (row0 + t) * S::ROW, nk * S::ROW, bar);
    bulk_load(s + kTile * 2 * S::ROW, a.c.meta + (row0 + t) * 4, nk * 8, bar);
    bulk_load(s + kTile * S::ROW, a.c.v_codes + (row0 + t) * S::ROW, nk * S::ROW, bar);
  };
  const int mine = tiles > warp ? (tiles - warp + kAttnWarps - 1) / kAttnWarps : 0;
  if (lane == 0)
    for (int i = 0; i < min(mine, kStages); ++i) issue(i);

  // Queries: this lane's B fragments (column lr of each block), their sums.
  uint32_t qf[NB][KS][2];
  float fac[NB][HPL], qsum[NB][HPL];  // of this lane's score columns
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    const int h = HPL == 1 ? ((lr & 1) ? H : lr >> 1) : nb * 8 + lr;
    // Lane (lr, lc) holds words 2 lc, 2 lc + 1 of a 64-element row, word lc of a 32-element one.
    float v[DH / 4], mx = 0.0f, sum = 0.0f;
#pragma unroll
    for (int i = 0; i < DH / 4; ++i) {
      v[i] = h < H ? bf16_f(query_row(a, b, g, h, DH)[lc * (DH / 4) + i]) : 0.0f;
      mx = fmaxf(mx, fabsf(v[i]));
      sum += v[i];
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    const int e = mx > 0.0f && mx < INFINITY ? ilogbf(mx) : 0;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      // Step s: word s / 2, elements 2 (s % 2) + {0, 4} and, 16 times, {1, 5}.
      const int i = 8 * (s / 2) + 2 * (s % 2);
      const __half2 lo = __floats2half2_rn(scalbnf(v[i], 14 - e), scalbnf(v[i + 4], 14 - e));
      const __half2 hi = __floats2half2_rn(scalbnf(v[i + 1], 10 - e), scalbnf(v[i + 5], 10 - e));
      qf[nb][s][0] = *reinterpret_cast<const uint32_t*>(&lo);
      qf[nb][s][1] = *reinterpret_cast<const uint32_t*>(&hi);
    }
    // Score columns 2 lc (and 2 lc + 1): their factors from the lanes that formed them.
    const float f = scalbnf(a.scale_log2, 24 - 14 + e);
#pragma unroll
    for (int j = 0; j < HPL; ++j) {
      fac[nb][j] = __shfl_sync(0xffffffffu, f, (2 * lc + j) * 4);
      qsum[nb][j] = __shfl_sync(0xffffffffu, sum * a.scale_log2, (2 * lc + j) * 4);
    }
  }

  float m[NB][HPL], l[NB][HPL], zs[NB][HPL], acc[NB][MT][4], ones[NB][4];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
    for (int j = 0; j < HPL; ++j) {
      m[nb][j] = -INFINITY;
      l[nb][j] = zs[nb][j] = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      ones[nb][i] = 0.0f;
#pragma unroll
      for (int t = 0; t < MT; ++t) acc[nb][t][i] = 0.0f;
    }
  }
  const int kr = row_key(lr), v0 = row_key(2 * lc), v1 = row_key(2 * lc + 1);
  constexpr int SUB = kTile / 16;
  for (int i = 0; i < mine; ++i) {
    if (!__all_sync(0xffffffffu, mbar_wait(full + i % kStages, (i / kStages) & 1, abort_flag))) break;
    const uint8_t* tk = ring + (i % kStages) * S::TILE_BYTES;
    const uint8_t* tv = tk + kTile * S::ROW;
    const uint8_t* tm = tv + kTile * S::ROW;
    const int left = k1 - k0 - (warp + kAttnWarps * i) * kTile;  // keys of this tile and beyond
    float sc[NB][SUB][4];
#pragma unroll
    for (int u = 0; u < SUB; ++u) {
      uint32_t w[2][DH / 32];  // rows kr, kr + 8
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const uint8_t* p = tk + (16 * u + kr + 8 * r) * S::ROW + lc * (S::ROW / 4);
        if constexpr (DH == 64) {
          const uint2 x = *reinterpret_cast<const uint2*>(p);
          w[r][0] = x.x;
          w[r][DH / 32 - 1] = x.y;
        } else {
          w[r][0] = *reinterpret_cast<const uint32_t*>(p);
        }
      }
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int x = 0; x < 4; ++x) sc[nb][u][x] = 0.0f;
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const uint32_t x0 = s & 1 ? w[0][s / 2] >> 8 : w[0][s / 2], x1 = s & 1 ? w[1][s / 2] >> 8 : w[1][s / 2];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
          mma_f16(sc[nb][u], x0 & 0x000f000fu, x1 & 0x000f000fu, x0 & 0x00f000f0u, x1 & 0x00f000f0u, qf[nb][s][0],
                  qf[nb][s][1]);
      }
    }
    // Scores, then the tile's maximum per head.
    float mt[NB][HPL];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int j = 0; j < HPL; ++j) mt[nb][j] = -INFINITY;
    uint32_t mv[SUB][2];  // the values' (scale, zero)
#pragma unroll
    for (int u = 0; u < SUB; ++u)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int key = 16 * u + kr + 8 * r;
        const uint2 mm = *reinterpret_cast<const uint2*>(tm + key * 8);
        const bool on = key < left;
        const float ks = bf16_f(mm.x & 0xffffu), kz = __uint_as_float(mm.x & 0xffff0000u);
        mv[u][r] = on ? mm.y : 0u;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int j = 0; j < HPL; ++j) {
            float& s = sc[nb][u][2 * r + j];
            s = on ? fmaf(s * fac[nb][j], ks, kz * qsum[nb][j]) : -INFINITY;
            mt[nb][j] = fmaxf(mt[nb][j], s);
          }
      }
    bool grown = false;
    float al[NB][HPL];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int j = 0; j < HPL; ++j) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) mt[nb][j] = fmaxf(mt[nb][j], __shfl_xor_sync(0xffffffffu, mt[nb][j], o));
        const float mn = fmaxf(m[nb][j], mt[nb][j]);
        grown = grown || mn > m[nb][j];
        al[nb][j] = m[nb][j] == mn ? 1.0f : exp2f(m[nb][j] - mn);
        m[nb][j] = mn;
        mt[nb][j] = mn == -INFINITY ? 0.0f : mn;  // nothing but -inf so far: weights 0
      }
    if (__any_sync(0xffffffffu, grown)) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int j = 0; j < HPL; ++j) {
          const float f = al[nb][j];
          l[nb][j] *= f;
          zs[nb][j] *= f;
          ones[nb][j] *= f;
#pragma unroll
          for (int t = 0; t < MT; ++t) {
            acc[nb][t][j] *= f;
            acc[nb][t][j + 2] *= f;
          }
        }
    }
#pragma unroll
    for (int u = 0; u < SUB; ++u) {
      uint32_t pw[NB][2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float vs = bf16_f(mv[u][r] & 0xffffu), vc = fmaf(8.0f, vs, __uint_as_float(mv[u][r] & 0xffff0000u));
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          float w2[2] = {0.0f, 0.0f};
#pragma unroll
          for (int j = 0; j < HPL; ++j) {
            const float p = exp2f(sc[nb][u][2 * r + j] - mt[nb][j]);
            l[nb][j] += p;
            zs[nb][j] = fmaf(p, vc, zs[nb][j]);
            w2[j] = p * vs;
          }
          pw[nb][r] = transpose8(pack_bf16x2(w2[0], w2[1]));
        }
      }
      // V: keys of rows 2 lc, 2 lc + 1 (+ 8), word lr (half a word for 32 elements).
      uint32_t x[2][4];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int word = DH == 64 ? lr : lr >> 1;
        const uint32_t a0 = *reinterpret_cast<const uint32_t*>(tv + (16 * u + v0 + 8 * r) * S::ROW + word * 4);
        const uint32_t a1 = *reinterpret_cast<const uint32_t*>(tv + (16 * u + v1 + 8 * r) * S::ROW + word * 4);
        if constexpr (DH == 64) {
          x[r][0] = __byte_perm(a0, a1, 0x5410);
          x[r][1] = __byte_perm(a0, a1, 0x7632);
        } else {
          x[r][0] = __byte_perm(a0, a1, lr & 1 ? 0x7632 : 0x5410);
        }
      }
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        const int hw = t / 2, sh = 8 * (t & 1);
        uint32_t f[4];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          f[2 * r] = ((x[r][hw] >> sh) & 0x000f000fu) | 0x43004300u;
          f[2 * r + 1] = ((x[r][hw] >> (sh + 4)) & 0x000f000fu) | 0x43004300u;
        }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) mma_bf16(acc[nb][t], f[0], f[1], f[2], f[3], pw[nb][0], pw[nb][1]);
      }
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
        mma_bf16(ones[nb], 0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u, pw[nb][0], pw[nb][1]);
    }
    __syncwarp();
    if (lane == 0 && i + kStages < mine) issue(i + kStages);
  }

  // This warp's state per head: output (lane lr holds dims DH/8 lr ...), max, sum.
  __syncthreads();  // every warp is done with the ring
  float* st = reinterpret_cast<float*>(sm);
#pragma unroll
  for (int nb = 0; nb < NB; ++nb)
#pragma unroll
    for (int j = 0; j < HPL; ++j) {
      const int h = HPL == 1 ? lc : nb * 8 + 2 * lc + j;
      float ls = l[nb][j], z = zs[nb][j];
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        ls += __shfl_xor_sync(0xffffffffu, ls, o);
        z += __shfl_xor_sync(0xffffffffu, z, o);
      }
      if (h >= H) continue;
      float* d = st + (warp * a.H + h) * S::STATE;
      z = fmaf(-136.0f, ones[nb][j], z);
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        d[lr * (DH / 8) + 2 * t] = acc[nb][t][j] + z;
        d[lr * (DH / 8) + 2 * t + 1] = acc[nb][t][j + 2] + z;
      }
      if (lr == 0) {
        d[DH] = m[nb][j];
        d[DH + 1] = ls;
      }
    }
  __syncthreads();
  const bool whole = n <= a.span;
  for (int i = tid; i < H * DH; i += kAttnThreads) {
    const int h = i / DH, d = i % DH;
    float mx = -INFINITY;
#pragma unroll
    for (int w = 0; w < kAttnWarps; ++w) mx = fmaxf(mx, st[(w * a.H + h) * S::STATE + DH]);
    const float mu = mx == -INFINITY ? 0.0f : mx;
    float o = 0.0f, ls = 0.0f;
#pragma unroll
    for (int w = 0; w < kAttnWarps; ++w) {
      const float* s = st + (w * a.H + h) * S::STATE;
      const float f = exp2f(s[DH] - mu);
      o = fmaf(f, s[d], o);
      ls = fmaf(f, s[DH + 1], ls);
    }
    if (whole) {
      store_out(a, b, g, h, d, DH, o / ls);
    } else {
      const long long at = ((static_cast<long long>(b) * a.G + g) * a.spans + span) * a.H + h;
      a.part_o[at * DH + d] = o;
      if (d == 0) a.part_ml[at] = make_float2(mx, ls);
    }
  }
}

// Joins the spans of the sequences that have several: one CTA per (sequence,
// group), one thread per (head, element).
template <int DH>
__global__ void __launch_bounds__(1024) kv4_merge_kernel(AttnArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  const int g = blockIdx.x % a.G, b = blockIdx.x / a.G;
  const int h = threadIdx.x / DH, d = threadIdx.x % DH;
  const int n = keys_of(a, b);
  if (n <= a.span || h >= heads_of_group(a, g)) return;
  const int spans = (n + a.span - 1) / a.span;
  const long long at0 = (static_cast<long long>(b) * a.G + g) * a.spans;
  float m = -INFINITY;
#pragma unroll 8
  for (int c = 0; c < spans; ++c) m = fmaxf(m, a.part_ml[(at0 + c) * a.H + h].x);
  const float mu = m == -INFINITY ? 0.0f : m;
  float o = 0.0f, l = 0.0f;
#pragma unroll 8
  for (int c = 0; c < spans; ++c) {
    const float2 ml = a.part_ml[(at0 + c) * a.H + h];
    const float w = exp2f(ml.x - mu);
    l = fmaf(w, ml.y, l);
    o = fmaf(w, a.part_o[((at0 + c) * a.H + h) * DH + d], o);
  }
  store_out(a, b, g, h, d, DH, o / l);
}

// Spans per (sequence, group): enough CTAs for kAttnCtas, each with at least
// one tile per warp.
constexpr int kAttnCtas = 148 * 2 * 8;
int attn_spans(int B, int G, int T) {
  const long long units = static_cast<long long>(B) * G, most = (T + kMinSpan - 1) / kMinSpan;
  const long long want = (kAttnCtas + units - 1) / units;
  return static_cast<int>(want < most ? want : most);
}

template <int DH, int HPL, int NB>
int launch_attn(const AttnArgs& a, void* stream) {
  const size_t smem = AttnShape<DH>::smem(a.H);
  const int e = ensure_smem<kv4_attn_kernel<DH, HPL, NB>>(static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  return launch_pdl(kv4_attn_kernel<DH, HPL, NB>, dim3(a.spans, static_cast<unsigned>(a.B) * a.G), dim3(kAttnThreads),
                    smem, stream, a);
}

template <int DH>
int attention(const AttnArgs& a, void* stream) {
  const int e = a.H <= 4 ? launch_attn<DH, 1, 1>(a, stream)
                : a.H <= 8 ? launch_attn<DH, 2, 1>(a, stream)
                           : launch_attn<DH, 2, 2>(a, stream);
  if (e != cudaSuccess || a.spans == 1) return e;
  return launch_pdl(kv4_merge_kernel<DH>, dim3(static_cast<unsigned>(a.B) * a.G), dim3(a.H * DH), 0, stream, a);
}

unsigned store_ctas(int B, int G, int T, int dh) {
  const long long rows = kThreads / (dh / 8), n = (static_cast<long long>(B) * G * T + rows - 1) / rows;
  return static_cast<unsigned>(n < 148 * 8 ? n : 148 * 8);
}

}  // namespace kv4_impl
using namespace kv4_impl;

int kv4_append(int B, int G, int T, int dh, const uint16_t* K, const uint16_t* V, const int32_t* start, int start0,
               const int32_t* count, const gqe_kv4& cache, void* stream) {
  const StoreArgs a{K, V, nullptr, nullptr, cache, start, start0, count, B, G, T};
  const dim3 grid(store_ctas(B, G, T, dh));
  return dh == 64 ? launch_pdl(append_kernel<64>, grid, dim3(kv4_impl::kThreads), 0, stream, a)
                  : launch_pdl(append_kernel<32>, grid, dim3(kv4_impl::kThreads), 0, stream, a);
}

int kv4_read(int B, int G, int T, int dh, const gqe_kv4& cache, const int32_t* start, const int32_t* count,
             uint16_t* K, uint16_t* V, void* stream) {
  const StoreArgs a{nullptr, nullptr, K, V, cache, start, 0, count, B, G, T};
  const dim3 grid(store_ctas(B, G, T, dh));
  return dh == 64 ? launch_pdl(read_kernel<64>, grid, dim3(kv4_impl::kThreads), 0, stream, a)
                  : launch_pdl(read_kernel<32>, grid, dim3(kv4_impl::kThreads), 0, stream, a);
}

size_t kv4_attention_ws_bytes(int B, int G, int T, int H, int dh) {
  const size_t units = static_cast<size_t>(B) * G * attn_spans(B, G, T) * H;
  return (units * dh * 4 + 255) / 256 * 256 + units * 8;
}

int kv4_attention(int B, int G, int T, int k, int dh, const uint16_t* Q, const uint16_t* Qs, const gqe_kv4& cache,
                  const int32_t* lens, int len_add, uint16_t* out, int ldo, void* ws, void* stream) {
  AttnArgs a{};
  a.Q = Q;
  a.Qs = Qs;
  a.c = cache;
  a.lens = lens;
  a.len_add = len_add;
  a.B = B;
  a.G = G;
  a.T = T;
  a.k = k;
  a.H = k + (Qs != nullptr ? 1 : 0);
  const int spans = attn_spans(B, G, T);
  a.span = ((T + spans - 1) / spans + kTile - 1) / kTile * kTile;
  a.spans = (T + a.span - 1) / a.span;
  const size_t units = static_cast<size_t>(B) * G * a.spans * a.H;
  a.part_o = static_cast<float*>(ws);
  a.part_ml = reinterpret_cast<float2*>(static_cast<char*>(ws) + (units * dh * 4 + 255) / 256 * 256);
  a.out = out;
  a.ldo = ldo;
  a.scale_log2 = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(dh)));
  return dh == 64 ? attention<64>(a, stream) : attention<32>(a, stream);
}

}  // namespace gqe
