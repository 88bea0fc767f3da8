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
//
// Storing 4 x 8192 tokens of 8 groups (86 MB): 26 us, bound by latency as much as
// by arithmetic: at 78 registers 32 % of the warps are resident, ALU 49 % and DRAM
// 28 % busy, 2.5 instructions per cycle. Reading them back: 15 us (5.8 TB/s).
#include <cooperative_groups.h>
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
__device__ __forceinline__ __nv_bfloat162 bf162(uint32_t v) { return *reinterpret_cast<const __nv_bfloat162*>(&v); }

// Two fp32 values worked on by one instruction.
using F2 = uint64_t;
__device__ __forceinline__ F2 make_f2(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float f2_lo(F2 v) { return __uint_as_float(static_cast<uint32_t>(v)); }
__device__ __forceinline__ float f2_hi(F2 v) { return __uint_as_float(static_cast<uint32_t>(v >> 32)); }
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// n / d for n < 2^31 by a multiplication (a 32-bit division costs about 20
// instructions, two of them per row).
struct Divisor {
  uint32_t mul;
  int shift;
  explicit Divisor(uint32_t d) : shift(0) {
    while ((1ull << shift) < d) ++shift;
    mul = static_cast<uint32_t>(((1ull << 32) * ((1ull << shift) - d)) / d + 1);
  }
  Divisor() : mul(0), shift(0) {}
  __device__ __forceinline__ uint32_t of(uint32_t n) const { return (__umulhi(n, mul) + n) >> shift; }
};

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
  Divisor by_T, by_G;
};

// Cache row of row r = (b G + g) T + t (fewer than 2^31), or -1: t is past the
// sequence's count, or the position is outside the cache (recorded, unless it
// is before position 0).
__device__ __forceinline__ long long cache_row(const StoreArgs& a, uint32_t r) {
  const uint32_t bg = a.by_T.of(r), b = a.by_G.of(bg);
  const int t = static_cast<int>(r - bg * a.T);
  if (a.count != nullptr && t >= a.count[b]) return -1;
  const long long p = static_cast<long long>(a.start != nullptr ? a.start[b] : a.start0) + t;
  if (p < 0) return -1;
  if (p >= a.c.capacity) {
    set_status(GQE_ERR_DEVICE_CHECK);
    return -1;
  }
  return static_cast<long long>(bg) * a.c.capacity + p;
}

// Eight codes by the definition's division.
__device__ __noinline__ uint32_t divide_codes(uint4 p, float hz, float hs) {
  const uint32_t w[4] = {p.x, p.y, p.z, p.w};
  uint32_t codes = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float x = __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
    codes |= static_cast<uint32_t>(fminf(fmaxf(rintf(__fdiv_rn(0.5f * x - hz, hs)), 0.0f), 15.0f)) << (4 * i);
  }
  return codes;
}

// This lane's 16 elements of a row (two 16-byte pieces) to codes, 8 per word;
// the row's (scale, zero) word.
//
// The quotient (x - zero) / scale is needed to the nearest whole number only.
// A product with the approximate reciprocal is within 2^-17 of it; rounded to
// a multiple of 2^-15 first (adding 384 does that) it is exact where the
// quotient is a half, so that adding 1.5 * 2^23 then rounds halves to even as
// the definition's division does. Halves are frequent (0.2 % of the elements:
// values and scales have 8 bits), quotients within 2^-16 of one are not: they
// show in the remainder and take the definition's division, as do scales
// whose reciprocal leaves fp32.
template <int LPR>
__device__ __forceinline__ uint2 quantise(uint4 p0, uint4 p1, uint32_t* meta) {
  const uint32_t w[8] = {p0.x, p0.y, p0.z, p0.w, p1.x, p1.y, p1.z, p1.w};
  constexpr float kRound = 12582912.0f, kGrid = 384.0f;
  // Pairs are unpacked where they are used: registers are what limits the loads in flight.
  auto pair = [&](int i) { return make_f2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u)); };
  F2 zero_if_finite = make_f2(0.0f, 0.0f);
#pragma unroll
  for (int i = 0; i < 8; ++i) zero_if_finite = fma2(pair(i), make_f2(0.0f, 0.0f), zero_if_finite);
  __nv_bfloat162 lo2 = bf162(w[0]), hi2 = lo2;
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    lo2 = __hmin2(lo2, bf162(w[i]));
    hi2 = __hmax2(hi2, bf162(w[i]));
  }
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) {
    lo2 = __hmin2(lo2, __shfl_xor_sync(0xffffffffu, lo2, o));
    hi2 = __hmax2(hi2, __shfl_xor_sync(0xffffffffu, hi2, o));
  }
  const float lo = fminf(__low2float(lo2), __high2float(lo2)), hi = fmaxf(__low2float(hi2), __high2float(hi2));
  const uint32_t group = ((1u << LPR) - 1u) << (threadIdx.x % 32 / LPR * LPR);
  const float bad = f2_lo(zero_if_finite) + f2_hi(zero_if_finite);
  if ((__ballot_sync(0xffffffffu, bad != 0.0f) & group) != 0u) {  // NaN != 0
    *meta = 0x7fff7fffu;
    return make_uint2(0u, 0u);
  }
  // Halved throughout: max - min of two bf16 may pass the largest fp32, and
  // halving is exact. The scale's quotient as a product, too, unless that ends
  // within 4 units of a border between two bf16.
  const float range = 0.5f * hi - 0.5f * lo;
  float sq = range * (1.0f / 7.5f);
  if ((__float_as_uint(sq) & 0xffffu) - 0x7ffcu <= 8u || !(sq > 1e-30f)) sq = __fdiv_rn(range, 7.5f);
  const uint16_t sb = __bfloat16_as_ushort(__float2bfloat16_rn(sq));
  const float s = bf16_f(sb), hs = 0.5f * s, hz = 0.5f * lo;
  *meta = sb | (__float_as_uint(lo) & 0xffff0000u);
  if (!(s > 0.0f)) return make_uint2(0u, 0u);
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(hs));
  auto distance = [&](int i) { return fma2(pair(i), make_f2(0.5f, 0.5f), make_f2(-hz, -hz)); };  // (x - zero) / 2
  auto quotient = [&](F2 d) { return add2(add2(mul2(d, make_f2(inv, inv)), make_f2(kGrid, kGrid)), make_f2(-kGrid, -kGrid)); };
  auto whole = [&](F2 q) { return add2(add2(q, make_f2(kRound, kRound)), make_f2(-kRound, -kRound)); };
  float off = 0.0f;  // the largest distance from a whole number
  uint32_t half[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    F2 n[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const F2 q = quotient(distance(2 * j + i));
      n[i] = whole(q);
      const F2 f = fma2(n[i], make_f2(-1.0f, -1.0f), q);
      off = max_nan(off, fabsf(f2_lo(f)), fabsf(f2_hi(f)));
    }
    // Four codes as one whole number below 2^16, read off its bits: (n0 + 256 n2) + 16 (n1 + 256 n3).
    const F2 t = fma2(n[1], make_f2(256.0f, 256.0f), n[0]);
    half[j] = __float_as_uint(fmaf(f2_hi(t), 16.0f, f2_lo(t)) + 8388608.0f);
  }
  if (!(off < 0.5f)) {
    // A half whose remainder is not zero (or a NaN): the division.
    bool settled = off == 0.5f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const F2 d = distance(i), q = quotient(d), f = fma2(whole(q), make_f2(-1.0f, -1.0f), q), e = fma2(q, make_f2(-hs, -hs), d);
      settled = settled && (fabsf(f2_lo(f)) != 0.5f || f2_lo(e) == 0.0f) && (fabsf(f2_hi(f)) != 0.5f || f2_hi(e) == 0.0f);
    }
    if (!settled) return make_uint2(divide_codes(p0, hz, hs), divide_codes(p1, hz, hs));
  }
  return make_uint2(__byte_perm(half[0], half[1], 0x5410), __byte_perm(half[2], half[3], 0x5410));
}

// DH / 16 lanes per row, each with the 16-byte pieces l and l + lanes (what a
// row needs once is shared by 16 elements; 8 lanes per row: 34 us against 27
// at 4 x 8192 tokens).
template <int DH>
__global__ void __launch_bounds__(kThreads, 3) append_kernel(StoreArgs a) {
  constexpr int LPR = DH / 16, ROWS = kThreads / LPR;
  pdl_wait();
  pdl_launch_dependents();
  const int l = threadIdx.x % LPR;
  const uint32_t n = static_cast<uint32_t>(a.B) * a.G * a.T, step = gridDim.x * ROWS;
  for (uint32_t r0 = blockIdx.x * ROWS; r0 < n; r0 += step) {
    const uint32_t r = r0 + threadIdx.x / LPR;
    const long long at = r < n ? cache_row(a, r) : -1;
    uint4 k0 = make_uint4(0u, 0u, 0u, 0u), k1 = k0, v0 = k0, v1 = k0;
    if (at >= 0) {
      const uint4* kp = reinterpret_cast<const uint4*>(a.K + static_cast<size_t>(r) * DH) + l;
      const uint4* vp = reinterpret_cast<const uint4*>(a.V + static_cast<size_t>(r) * DH) + l;
      k0 = *kp;
      k1 = *(kp + LPR);
      v0 = *vp;
      v1 = *(vp + LPR);
    }
#pragma unroll 1
    for (int t = 0; t < 2; ++t) {  // K, then V (loaded above): one copy of the code, half the registers
      uint32_t m;
      const uint2 c = quantise<LPR>(k0, k1, &m);
      k0 = v0;
      k1 = v1;
      if (at < 0) continue;
      uint32_t* d = reinterpret_cast<uint32_t*>(t == 0 ? a.c.k_codes : a.c.v_codes) + at * (DH / 8) + l;
      d[0] = c.x;
      d[LPR] = c.y;
      if (l == 0) reinterpret_cast<uint32_t*>(a.c.meta)[2 * at + t] = m;
    }
  }
}

constexpr int kRowsAhead = 2;  // rows of a thread in flight
__device__ __forceinline__ uint4 decode8(uint32_t codes, uint32_t meta) {
  const float s = bf16_f(meta & 0xffffu), z = __uint_as_float(meta & 0xffff0000u);
  float x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)  // a code in the low bits of 2^23 is 2^23 + code
    x[i] = fmaf(s, __uint_as_float(((codes >> (4 * i)) & 15u) | 0x4b000000u) - 8388608.0f, z);
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}

template <int DH>
__global__ void __launch_bounds__(kThreads) read_kernel(StoreArgs a) {
  constexpr int LPR = DH / 8, ROWS = kThreads / LPR, U = kRowsAhead;
  pdl_wait();
  pdl_launch_dependents();
  const int l = threadIdx.x % LPR;
  const uint32_t n = static_cast<uint32_t>(a.B) * a.G * a.T, step = gridDim.x * ROWS;
  for (uint32_t r0 = blockIdx.x * ROWS; r0 < n; r0 += U * step) {
    uint32_t k[U], v[U];
    uint2 m[U];
    bool on[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t r = r0 + u * step + threadIdx.x / LPR;
      const long long at = r0 + u * step < n && r < n ? cache_row(a, r) : -1;
      on[u] = at >= 0;
      if (!on[u]) continue;
      m[u] = reinterpret_cast<const uint2*>(a.c.meta)[at];
      k[u] = reinterpret_cast<const uint32_t*>(a.c.k_codes)[at * LPR + l];
      v[u] = reinterpret_cast<const uint32_t*>(a.c.v_codes)[at * LPR + l];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (!on[u]) continue;
      const size_t r = r0 + u * step + threadIdx.x / LPR;
      reinterpret_cast<uint4*>(a.Ko + r * DH)[l] = decode8(k[u], m[u].x);
      reinterpret_cast<uint4*>(a.Vo + r * DH)[l] = decode8(v[u], m[u].y);
    }
  }
}

// ---------------------------------------------------------------------------
// Decode attention: o = softmax(q . K / sqrt(dh)) V over the sequence's keys.
//
// Bytes: d_head + 8 per key and KV group (codes of K and V, two (scale, zero)
// pairs), 28 % of the bf16 cache's 4 d_head (31 % at 32). At that rate the CUDA cores
// would bound the kernel (two products and two conversions per element and
// head), so the products run on the tensor cores (mma.sync m16n8k16: with at
// most 16 query rows a 128-row tcgen05 tile would be nine tenths padding)
// and the codes become their operands by bit operations alone:
//  - Scores, keys x heads: a code n masked into the low mantissa bits of an
//    fp16 is the subnormal n 2^-24, exact; in the next four bits 16 n 2^-24,
//    undone in q. Of a row's 32-bit word that is one shift and four ANDs for
//    eight elements. q goes in as q 2^(14 - e), e the exponent of the head's
//    largest element: exact but for elements 2^-38 of that. Then
//    s = scale_k sum(q n) + zero_k sum(q) in fp32, in units of 2^10 (kUnit).
//  - Output, dims x heads, over the keys: with n in the upper four mantissa
//    bits, 0x4180 | n << 3 is the bf16 16 + n. The weight operand is p scale_v
//    in two bf16 parts (fp16 would not hold the range of the scales; one part
//    alone, 8 bits, put the outputs 0.1 to 0.15 % off beside their own rounding's
//    0.17 %; the second costs 1 to 3 % up to 4 heads, about 15 % with 8 and 20 %
//    with 16): together 2^-16 of it, against codes taken around zero, since 24
//    times the sum of the same parts is taken off again, which leaves
//    sum p scale_v (n - 8); the rest, sum p (zero_v + 8 scale_v), is kept in
//    fp32. The tensor cores cut their sums off where they would round, always
//    downwards: each tile's sums start from zero and join the running ones in
//    fp32 (carried on in the accumulator, and with 128 + n, the 64 x 32k outputs
//    were 1.3 % off).
//  - Up to 4 heads per group: the heads sit in the even columns (the second
//    part of a weight in the odd one beside it: no product more), 4 / HP times
//    over (HP = 1, 2 or 4 >= the group's heads), so the scores' accumulator
//    holds one head per lane and every copy of the column can take other keys:
//    lane column lc forms the weights of head lc % HP for the 16-key blocks
//    u = lc / HP (mod 4 / HP) only, and leaves 0 in the others. The copies'
//    sums are added at the end of a unit. Without that one head's softmax
//    costs what four heads' does (64 x 32k, one head in 7 of 8 groups: 149
//    instructions per 16 keys against 164).
//  - A transposed 8 x 8 move turns the weights from (key, head) to the second
//    product's (head, keys) order.
// The work is cut over warps: the tiles of 64 keys of all (sequence, group)
// units, laid end to end, are dealt in equal contiguous shares, so that ragged
// lengths, few long sequences and many short ones all fill the SMs alike. A
// warp streams its tiles through a ring of its own, across the units' borders,
// with its own running maximum and no CTA-wide barrier in the loop (by
// cp.async: a bulk copy per array and tile took more instructions than its
// nine 512-byte pieces). A unit that lies in one warp's share is written out
// by it; the parts of the others are joined by a second kernel.
//
// Measured: 64 x 32768 keys, 8 groups, one or two heads each: 235 us (1.21 GB,
// 80 % of the copy rate, under the power cap; 201 us in a short run); 192 x 32768
// in a short run: 90 to 98 % of the copy rate; ALU pipe 59 % and tensor pipe 30 %
// busy. 1 x 2048 keys: 7.4 us, one launch (kv4_attn_unit_kernel). 9 to 16 heads
// (the registers of two column blocks pass 128, 0.7 KB of them spill): 32 x 32768
// keys of 4 groups with 16 heads each 149 to 160 us, floor 47.
constexpr int kAttnWarps = 8;
constexpr int kAttnThreads = 32 * kAttnWarps;
constexpr int kTile = 64;   // keys per tile
constexpr int kStages = 3;  // tiles in flight per warp
constexpr int kAttnCtasPerSm = 2;
constexpr int kMaxAttnWarps = 148 * kAttnCtasPerSm * kAttnWarps;
// Scores and their maxima are kept in units of 2^10: the factor of a query near
// bf16's largest, and the sum of its elements, then stay within fp32. The
// exponential's difference undoes it in the multiply-add that it is.
constexpr float kUnit = 1024.0f;

struct AttnArgs {
  const uint16_t* Q;   // [B][G][k][dh]
  const uint16_t* Qs;  // [B][dh] or null
  gqe_kv4 c;
  const int32_t* lens;
  int len_add, B, G, T, k, H;
  int ctas;  // of a cluster (unit kernel)
  // Part of warp w and unit u = b G + g: slot w + u (along the shares, w + u
  // grows with every part, and a unit's parts are consecutive).
  float* part_o;       // [slots][H][dh]
  float2* part_ml;     // [slots][H]: max (in kUnit), sum
  long long* starts;   // [B + 1]: tiles before sequence b; then the share
  uint16_t* out;
  int ldo;
  float scale_log2;
};

__device__ __forceinline__ int keys_of(const AttnArgs& a, int b) {
  const long long n = a.lens != nullptr ? static_cast<long long>(a.lens[b]) + a.len_add : a.T;
  return static_cast<int>(n < 0 ? 0 : n > a.T ? a.T : n);
}
__host__ __device__ __forceinline__ int tiles_of(int keys) {  // unsigned: keys may come near 2^31
  return static_cast<int>((static_cast<uint32_t>(keys) + kTile - 1) / kTile);
}
__device__ __forceinline__ int heads_of_group(const AttnArgs& a, int g) { return a.k + (g == 0 && a.Qs != nullptr ? 1 : 0); }
__device__ __forceinline__ const uint16_t* query_row(const AttnArgs& a, int b, int g, int h, int dh) {
  return h < a.k ? a.Q + ((static_cast<long long>(b) * a.G + g) * a.k + h) * dh : a.Qs + static_cast<long long>(b) * dh;
}
__device__ __forceinline__ uint16_t* out_row(const AttnArgs& a, int b, int g, int h, int dh) {
  return a.out + static_cast<long long>(b) * a.ldo + (h < a.k ? g * a.k + h : a.G * a.k) * dh;
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// D = A B.
__device__ __forceinline__ void mma_f16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ void mma_bf16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// (x & 0x00780078) | one in one instruction: with both masks as constants the
// compiler emits two, so `one` comes from a register that it cannot see into.
__device__ __forceinline__ uint32_t code_pair(uint32_t x, uint32_t one) {
  uint32_t r;
  asm("lop3.b32 %0, %1, 0x00780078, %2, 0xEA;" : "=r"(r) : "r"(x), "r"(one));
  return r;
}
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
// 2^x; results below 2^-126 are 0 (weights that far under the largest are lost
// in fp32 sums anyway).
__device__ __forceinline__ float exp2_ftz(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }  // -126 <= e <= 127
// 2^(a - b) of two maxima in kUnit; nothing but -inf so far (b as 0): 0.
__device__ __forceinline__ float exp2_less(float a, float b) { return exp2_ftz(fmaf(a, kUnit, -b * kUnit)); }

// Four 8 x 8 blocks of 16-bit elements, each read by rows (lane 8 i + j: row j
// of block i) and handed out by columns: lane (lr, lc) gets elements 2 lc and
// 2 lc + 1 of column lr of each.
__device__ __forceinline__ void load_transposed(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void load_transposed(uint32_t (&r)[2], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0,%1}, [%2];"
               : "=r"(r[0]), "=r"(r[1])
               : "r"(addr)
               : "memory");
}

template <int DH>
struct AttnShape {
  static constexpr int ROW = DH / 2;                       // bytes of a row's codes
  static constexpr int TILE_BYTES = kTile * (2 * ROW + 8);  // K, V, meta
  static constexpr int RING = kStages * TILE_BYTES;
  static constexpr size_t smem() { return static_cast<size_t>(kAttnWarps) * RING; }
};

// A place in the units' tiles: a unit and the keys from the place to its end.
struct Cursor {
  int b, g, left;
  __device__ __forceinline__ long long row(const AttnArgs& a) const {  // cache row of the place
    return (static_cast<long long>(b) * a.G + g) * a.c.capacity + (keys_of(a, b) - left);
  }
  // By all lanes of a warp: sequences without keys are passed over 32 at a time
  // (one by one, a length's latency each, 4095 idle ones took 320 us).
  __device__ __forceinline__ void next_unit(const AttnArgs& a, int lane) {
    if (++g == a.G) {
      g = 0;
      ++b;
      while (b < a.B) {
        const unsigned live = __ballot_sync(0xffffffffu, b + lane < a.B && keys_of(a, b + lane) > 0);
        b += live != 0u ? __ffs(live) - 1 : 32;
        if (live != 0u) break;
      }
    }
    left = b < a.B ? keys_of(a, b) : 0;
  }
};

// HPL: heads per lane (1: even columns, at most 4 heads; 2: all columns);
// NB: column blocks of 8 (2 only with HPL = 2). HP of the members: see above (4 with HPL = 2).
template <int DH, int HPL, int NB>
struct Warp {
  using S = AttnShape<DH>;
  static constexpr int KS = DH / 16;  // k steps of the scores
  static constexpr int MT = DH / 16;  // 16-row blocks of the output
  static constexpr int SUB = kTile / 16;
  uint32_t qf[NB][KS][2];               // B fragments of the queries (column lr)
  float fac[NB][HPL], qsum[NB][HPL];    // of this lane's score columns
  float m[NB][HPL], l[NB][HPL], zs[NB][HPL], acc[NB][MT][2 * HPL];  // acc: rows lr, then lr + 8
  int lr, lc;
  uint32_t k16;  // 0x41804180, bf16 16 twice

  __device__ __forceinline__ void start(const AttnArgs& a, int b, int g, int hp) {
    const int H = heads_of_group(a, g);
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int h = HPL == 1 ? ((lr & 1) ? H : (lr >> 1) & (hp - 1)) : nb * 8 + lr;
      // Lane (lr, lc) holds words 2 lc, 2 lc + 1 of a 64-element row, word lc of a 32-element one.
      float v[DH / 4], mx = 0.0f, sum = 0.0f;
#pragma unroll
      for (int i = 0; i < DH / 4; i += 8) {
        const uint4 w = h < H ? *reinterpret_cast<const uint4*>(query_row(a, b, g, h, DH) + lc * (DH / 4) + i)
                              : make_uint4(0u, 0u, 0u, 0u);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          v[i + 2 * q] = __uint_as_float(u[q] << 16);
          v[i + 2 * q + 1] = __uint_as_float(u[q] & 0xffff0000u);
        }
      }
#pragma unroll
      for (int i = 0; i < DH / 4; ++i) {
        mx = fmaxf(mx, fabsf(v[i]));
        sum = fmaf(v[i], 1.0f / kUnit, sum);  // exact terms: bf16's least times 2^-10 is an fp32
      }
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
      }
      // e: the exponent of the largest element (infinities and NaN pass as they are).
      const int e = mx < INFINITY ? max((__float_as_int(mx) >> 23) - 127, -100) : 0;
      const float up = pow2(14 - e), up16 = pow2(10 - e);
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        // Step s: word s / 2, elements 2 (s % 2) + {0, 4} and, 16 times, {1, 5}.
        const int i = 8 * (s / 2) + 2 * (s % 2);
        const __half2 lo = __floats2half2_rn(v[i] * up, v[i + 4] * up);
        const __half2 hi = __floats2half2_rn(v[i + 1] * up16, v[i + 5] * up16);
        qf[nb][s][0] = *reinterpret_cast<const uint32_t*>(&lo);
        qf[nb][s][1] = *reinterpret_cast<const uint32_t*>(&hi);
      }
      // Score columns 2 lc (and 2 lc + 1): their factors from the lanes that formed them.
      const float f = a.scale_log2 * pow2(e);  // 2^(24 - 14 + e), in kUnit
#pragma unroll
      for (int j = 0; j < HPL; ++j) {
        fac[nb][j] = __shfl_sync(0xffffffffu, f, (2 * lc + j) * 4);
        qsum[nb][j] = __shfl_sync(0xffffffffu, sum * a.scale_log2, (2 * lc + j) * 4);
        m[nb][j] = -INFINITY;
        l[nb][j] = zs[nb][j] = 0.0f;
      }
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int i = 0; i < 2 * HPL; ++i) acc[nb][t][i] = 0.0f;
    }
  }

  // One tile in shared memory; FULL: 64 keys, else the first `left`.
  template <int HP, bool FULL>
  __device__ __forceinline__ void tile(const uint8_t* tk, int left) {
    constexpr int R = 4 / HP;   // copies of a head's column
    constexpr int OWN = SUB / R;  // 16-key blocks whose weights a lane forms: part + R i
    const int part = lc / HP;
    const uint8_t* tm = tk + 2 * kTile * S::ROW;
    // This lane's row of the V blocks: 8-key half (lane / 8) % 2, 16-byte piece (lane / 16) of it.
    const int lane = 4 * lr + lc;
    const uint32_t tva = smem_u32(tk) + kTile * S::ROW + (lane & 15) * S::ROW + (DH == 64 ? lane & 16 : 0);
    float sc[NB][SUB][4];
#pragma unroll
    for (int u = 0; u < SUB; ++u) {
      uint32_t w[2][DH / 32];  // rows lr, lr + 8
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const uint8_t* p = tk + (16 * u + lr + 8 * r) * S::ROW + lc * (S::ROW / 4);
        if constexpr (DH == 64) {
          const uint2 x = *reinterpret_cast<const uint2*>(p);
          w[r][0] = x.x;
          w[r][DH / 32 - 1] = x.y;
        } else {
          w[r][0] = *reinterpret_cast<const uint32_t*>(p);
        }
      }
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const uint32_t x0 = s & 1 ? w[0][s / 2] >> 8 : w[0][s / 2], x1 = s & 1 ? w[1][s / 2] >> 8 : w[1][s / 2];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          const uint32_t f0 = x0 & 0x000f000fu, f1 = x1 & 0x000f000fu, f2 = x0 & 0x00f000f0u, f3 = x1 & 0x00f000f0u;
          if (s == 0) mma_f16_first(sc[nb][u], f0, f1, f2, f3, qf[nb][s][0], qf[nb][s][1]);
          else mma_f16(sc[nb][u], f0, f1, f2, f3, qf[nb][s][0], qf[nb][s][1]);
        }
      }
    }
    // Scores of this lane's blocks, then the tile's maximum per head.
    float mt[NB][HPL], ps[NB][HPL][OWN][2];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int j = 0; j < HPL; ++j) mt[nb][j] = -INFINITY;
    uint32_t mv[OWN][2];  // the values' (scale, zero)
#pragma unroll
    for (int i = 0; i < OWN; ++i)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int key = 16 * (part + R * i) + lr + 8 * r;
        const uint2 mm = *reinterpret_cast<const uint2*>(tm + key * 8);
        const bool on = FULL || key < left;
        const float ks = bf16_f(mm.x & 0xffffu), kz = __uint_as_float(mm.x & 0xffff0000u);
        mv[i][r] = on ? mm.y : 0u;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int j = 0; j < HPL; ++j) {
            float d = sc[nb][R * i][2 * r + j];
#pragma unroll
            for (int q = 1; q < R; ++q) d = part == q ? sc[nb][R * i + q][2 * r + j] : d;
            const float v = on ? fmaf(d * fac[nb][j], ks, kz * qsum[nb][j]) : -INFINITY;
            ps[nb][j][i][r] = v;
            mt[nb][j] = fmaxf(mt[nb][j], v);
          }
      }
    bool grown = false;
    float al[NB][HPL];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int j = 0; j < HPL; ++j) {
#pragma unroll
        for (int o = HP; o < 32; o <<= 1) mt[nb][j] = fmaxf(mt[nb][j], __shfl_xor_sync(0xffffffffu, mt[nb][j], o));
        const float mn = fmaxf(m[nb][j], mt[nb][j]);
        grown = grown || mn > m[nb][j];
        al[nb][j] = m[nb][j] == mn ? 1.0f : exp2_less(m[nb][j], mn);
        m[nb][j] = mn;
        mt[nb][j] = mn == -INFINITY ? 0.0f : mn * kUnit;  // nothing but -inf so far: weights 0
      }
    if (__any_sync(0xffffffffu, grown)) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int j = 0; j < HPL; ++j) {
          const float f = al[nb][j];
          l[nb][j] *= f;
          zs[nb][j] *= f;
#pragma unroll
          for (int t = 0; t < MT; ++t) {
            acc[nb][t][j] *= f;
            acc[nb][t][j + HPL] *= f;
          }
        }
    }
    // Weights p scale_v of this lane's blocks, in two bf16 parts: the upper half
    // of the fp32 value, and what that leaves. pk[0]: column 2 lc in the low half,
    // 2 lc + 1 in the high half. One head per lane: the first part in column
    // 2 lc, the second beside it in 2 lc + 1, the same products for both; two
    // heads: the second parts in pk[1], products of their own.
    constexpr int PARTS = HPL;
    uint32_t pk[PARTS][NB][OWN][2];
#pragma unroll
    for (int i = 0; i < OWN; ++i)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float vs = bf16_f(mv[i][r] & 0xffffu), vc = fmaf(8.0f, vs, __uint_as_float(mv[i][r] & 0xffff0000u));
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          float hi[HPL], rest[HPL];
#pragma unroll
          for (int j = 0; j < HPL; ++j) {
            const float p = exp2_ftz(fmaf(ps[nb][j][i][r], kUnit, -mt[nb][j]));
            l[nb][j] += p;
            zs[nb][j] = fmaf(p, vc, zs[nb][j]);
            const float w = p * vs;
            hi[j] = __uint_as_float(__float_as_uint(w) & 0xffff0000u);
            rest[j] = w - hi[j];
          }
          uint32_t second;
          if constexpr (HPL == 1) {
            second = pk[0][nb][i][r] = pack_bf16x2(hi[0], rest[0]);
          } else {
            pk[0][nb][i][r] = __byte_perm(__float_as_uint(hi[0]), __float_as_uint(hi[HPL - 1]), 0x7632);
            second = pk[PARTS - 1][nb][i][r] = pack_bf16x2(rest[0], rest[HPL - 1]);
          }
#pragma unroll
          for (int j = 0; j < HPL; ++j) {  // the weights as they go in, of the codes' 16 + 8
            const float lo = __uint_as_float(HPL == 1 || j == 1 ? second & 0xffff0000u : second << 16);
            zs[nb][j] = fmaf(-24.0f, hi[j], fmaf(-24.0f, lo, zs[nb][j]));
          }
        }
      }
    float sum[NB][MT][4];  // of this tile
#pragma unroll
    for (int u = 0; u < SUB; ++u) {
      uint32_t pw[PARTS][NB][2];
#pragma unroll
      for (int c = 0; c < PARTS; ++c)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int r = 0; r < 2; ++r) pw[c][nb][r] = transpose8(R == 1 || part == u % R ? pk[c][nb][u / R][r] : 0u);
      // V: 16-bit column lr (4 codes) of keys 2 lc, 2 lc + 1 (+ 8), for each
      // 32 elements of a row: element 32 x + 4 lr + nibble.
      uint32_t x[2 * (DH / 32)];  // [32 elements][keys + 8 r]
      load_transposed(x, tva + 16 * u * S::ROW);
#pragma unroll
      for (int t = 0; t < MT; ++t) {  // nibbles 2 (t % 2), 2 (t % 2) + 1
        uint32_t f[4];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const uint32_t v = x[2 * (t / 2) + r];
          f[2 * r] = code_pair(t & 1 ? v >> 5 : v << 3, k16);
          f[2 * r + 1] = code_pair(t & 1 ? v >> 9 : v >> 1, k16);
        }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          if (u == 0) mma_bf16_first(sum[nb][t], f[0], f[1], f[2], f[3], pw[0][nb][0], pw[0][nb][1]);
          else mma_bf16(sum[nb][t], f[0], f[1], f[2], f[3], pw[0][nb][0], pw[0][nb][1]);
          if (PARTS == 2) mma_bf16(sum[nb][t], f[0], f[1], f[2], f[3], pw[PARTS - 1][nb][0], pw[PARTS - 1][nb][1]);
        }
      }
    }
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int j = 0; j < HPL; ++j) {
          acc[nb][t][j] += HPL == 1 ? sum[nb][t][0] + sum[nb][t][1] : sum[nb][t][j];
          acc[nb][t][j + HPL] += HPL == 1 ? sum[nb][t][2] + sum[nb][t][3] : sum[nb][t][j + 2];
        }
  }

  __device__ __forceinline__ void any_tile(const uint8_t* s, int left, int hp) {
    if (HPL == 1 && hp == 1) {
      if (left >= kTile) tile<1, true>(s, left);
      else tile<1, false>(s, left);
    } else if (HPL == 1 && hp == 2) {
      if (left >= kTile) tile<2, true>(s, left);
      else tile<2, false>(s, left);
    } else {
      if (left >= kTile) tile<4, true>(s, left);
      else tile<4, false>(s, left);
    }
  }

  // The unit's outputs (whole), or this warp's part of them: sums [heads][DH] to po, (max, sum) [heads] to pml.
  __device__ __forceinline__ void finish(const AttnArgs& a, int b, int g, int hp, bool whole, float* po, float2* pml) {
    const int H = heads_of_group(a, g);
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int j = 0; j < HPL; ++j) {
        const int h = HPL == 1 ? lc : nb * 8 + 2 * lc + j;  // copies: h >= hp
        float ls = l[nb][j], z = zs[nb][j];
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {  // the copies of the head's column
          if (o < hp) continue;
          ls += __shfl_xor_sync(0xffffffffu, ls, o);
          z += __shfl_xor_sync(0xffffffffu, z, o);
#pragma unroll
          for (int t = 0; t < MT; ++t) {
            acc[nb][t][j] += __shfl_xor_sync(0xffffffffu, acc[nb][t][j], o);
            acc[nb][t][j + HPL] += __shfl_xor_sync(0xffffffffu, acc[nb][t][j + HPL], o);
          }
        }
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
          ls += __shfl_xor_sync(0xffffffffu, ls, o);
          z += __shfl_xor_sync(0xffffffffu, z, o);
        }
        if (h >= H || (HPL == 1 && h >= hp)) continue;
        const float f = whole ? 1.0f / ls : 1.0f;
        float o[DH / 8];  // elements 32 x + 4 lr + {0..3}, x < DH / 32
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          o[2 * t] = (acc[nb][t][j] + z) * f;
          o[2 * t + 1] = (acc[nb][t][j + HPL] + z) * f;
        }
        if (whole) {
          uint16_t* d = out_row(a, b, g, h, DH) + 4 * lr;
#pragma unroll
          for (int i = 0; i < DH / 32; ++i)
            *reinterpret_cast<uint2*>(d + 32 * i) = make_uint2(pack_bf16x2(o[4 * i], o[4 * i + 1]), pack_bf16x2(o[4 * i + 2], o[4 * i + 3]));
        } else {
          float* d = po + h * DH + 4 * lr;
#pragma unroll
          for (int i = 0; i < DH / 32; ++i)
            *reinterpret_cast<float4*>(d + 32 * i) = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
          if (lr == 0) pml[h] = make_float2(m[nb][j], ls);
        }
      }
  }
};

// Columns per head set (HPL = 1): 1, 2 or 4 >= the group's heads.
template <int HPL>
__device__ __forceinline__ int columns(int H) {
  return HPL == 2 || H > 2 ? 4 : H;
}

// Loads a lane's pieces of one tile, `left` keys from the rows at pk, pv, pm
// on, into the ring's place at d.
template <int DH>
__device__ __forceinline__ void load_tile(const AttnArgs& a, uint32_t d, const uint8_t* pk, const uint8_t* pv,
                                          const uint8_t* pm, int left, int lane) {
  using S = AttnShape<DH>;
  constexpr int CP = kTile * S::ROW / 512;  // 16-byte pieces of K (or V) per lane
  d += lane * 16;
  if (left >= kTile) {
#pragma unroll
    for (int j = 0; j < CP; ++j) cp_async_16(d + 512 * j, pk + 512 * j, 16);
    cp_async_16(d + 2 * kTile * S::ROW, pm, 16);
#pragma unroll
    for (int j = 0; j < CP; ++j) cp_async_16(d + kTile * S::ROW + 512 * j, pv + 512 * j, 16);
  } else {
    // The sequence's last tile: what lies behind it (and perhaps behind the
    // buffer) is not read, its place is filled with zeros.
#pragma unroll
    for (int j = 0; j < CP; ++j) {
      const bool on = 16 * (lane + 32 * j) < left * S::ROW;
      cp_async_16(d + 512 * j, on ? pk + 512 * j : a.c.k_codes, on ? 16 : 0);
      cp_async_16(d + kTile * S::ROW + 512 * j, on ? pv + 512 * j : a.c.v_codes, on ? 16 : 0);
    }
    const bool on = 2 * lane < left;  // two keys per piece (the capacity is even)
    cp_async_16(d + 2 * kTile * S::ROW, on ? pm : reinterpret_cast<const uint8_t*>(a.c.meta), on ? 16 : 0);
  }
}

template <int DH, int HPL, int NB>
__global__ void __launch_bounds__(kAttnThreads, kAttnCtasPerSm) kv4_attn_kernel(AttnArgs a) {
  using S = AttnShape<DH>;
  extern __shared__ __align__(128) uint8_t sm[];
  __shared__ long long before[kAttnThreads + 1];  // tiles before each thread's run of sequences
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();  // q, lens and the newest rows come from earlier kernels
  pdl_launch_dependents();
  // Tiles of all sequences before each run of `run` of them.
  const int run = (a.B + kAttnThreads - 1) / kAttnThreads;
  {
    long long s = 0;
    for (int b = tid * run; b < min(a.B, (tid + 1) * run); ++b) s += static_cast<long long>(tiles_of(keys_of(a, b))) * a.G;
    long long in = s;  // inclusive over the warp
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, in, o);
      if (lane >= o) in += v;
    }
    before[tid + 1] = in;
    if (tid == 0) before[0] = 0;
    __syncthreads();
    long long base = 0;
    for (int w = 0; w < warp; ++w) base += before[32 * (w + 1)];
    __syncthreads();
    before[tid + 1] = in + base;
    __syncthreads();
  }
  // Warps of all CTAs, first every CTA's warp 0: short work spreads over the SMs.
  const long long W = static_cast<long long>(gridDim.x) * kAttnWarps, gw = static_cast<long long>(warp) * gridDim.x + blockIdx.x;
  const long long total = before[kAttnThreads], share = max((total + W - 1) / W, 1ll);
  if (blockIdx.x == 0) {  // for the join
    long long s = before[tid];
    for (int b = tid * run; b < min(a.B, (tid + 1) * run); ++b) {
      a.starts[b] = s;
      s += static_cast<long long>(tiles_of(keys_of(a, b))) * a.G;
    }
    if (tid == 0) a.starts[a.B] = share;
  }
  // Sequences without keys: zeros.
  const long long units = static_cast<long long>(a.B) * a.G;
  for (long long u = gw * 32 + lane; u < units; u += W * 32) {
    const int b = static_cast<int>(u / a.G), g = static_cast<int>(u - static_cast<long long>(b) * a.G);
    if (keys_of(a, b) == 0)
      for (int h = 0; h < heads_of_group(a, g); ++h)
        for (int i = 0; i < DH / 8; ++i) reinterpret_cast<uint4*>(out_row(a, b, g, h, DH))[i] = make_uint4(0u, 0u, 0u, 0u);
  }
  const long long w0 = gw * share, w1 = min(total, w0 + share);
  if (w0 >= w1) return;
  // The share's first tile: the run of sequences, then the sequence.
  Cursor rd;
  bool first_whole;  // the share holds the unit's first tile
  {
    int lo = 0, hi = kAttnThreads;  // the last entry of `before` that is <= w0
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (before[mid] <= w0) lo = mid;
      else hi = mid;
    }
    long long s = before[lo];
    rd.b = lo * run;
    int n;
    for (;; ++rd.b) {
      n = keys_of(a, rd.b);
      const long long t = static_cast<long long>(tiles_of(n)) * a.G;
      if (w0 < s + t) break;
      s += t;
    }
    const int tb = tiles_of(n), at = static_cast<int>(w0 - s);
    rd.g = at / tb;
    rd.left = n - (at - rd.g * tb) * kTile;
    first_whole = rd.left == n;
  }
  const int count = static_cast<int>(w1 - w0);
  const uint32_t ring = smem_u32(sm) + warp * S::RING;
  // Loads: the next tile's place, and this lane's pointers at its cache row.
  Cursor wr = rd;
  const uint8_t *pk, *pv, *pm;
  auto seek = [&] {
    const long long row = wr.row(a);
    pk = a.c.k_codes + row * S::ROW + lane * 16;
    pv = a.c.v_codes + row * S::ROW + lane * 16;
    pm = reinterpret_cast<const uint8_t*>(a.c.meta) + row * 8 + lane * 16;
  };
  auto issue = [&](int i) {
    load_tile<DH>(a, ring + i * S::TILE_BYTES, pk, pv, pm, wr.left, lane);
    pk += kTile * S::ROW;
    pv += kTile * S::ROW;
    pm += kTile * 8;
    wr.left -= kTile;
    if (wr.left <= 0) {
      wr.next_unit(a, lane);
      if (wr.left > 0) seek();
    }
  };
  seek();
#pragma unroll
  for (int i = 0; i < kStages; ++i) {
    if (i < count) issue(i);
    cp_async_commit();
  }
  Warp<DH, HPL, NB> w;
  w.lr = lane >> 2;
  w.lc = lane & 3;
  asm volatile("mov.b32 %0, 0x41804180;" : "=r"(w.k16));
  int hp = columns<HPL>(heads_of_group(a, rd.g));
  w.start(a, rd.b, rd.g, hp);
  int stage = 0;
  for (int i = 0; i < count; ++i) {
    cp_async_wait<kStages - 1>();
    __syncwarp();
    const uint8_t* s = sm + warp * S::RING + stage * S::TILE_BYTES;
    const int left = rd.left;
    w.any_tile(s, left, hp);
    __syncwarp();
    if (i + kStages < count) issue(stage);
    cp_async_commit();
    stage = stage + 1 == kStages ? 0 : stage + 1;
    rd.left = left - kTile;
    if (rd.left <= 0 || i + 1 == count) {
      const long long slot = (gw + static_cast<long long>(rd.b) * a.G + rd.g) * a.H;
      w.finish(a, rd.b, rd.g, hp, first_whole && rd.left <= 0, a.part_o + slot * DH, a.part_ml + slot);
      if (i + 1 == count) break;
      rd.next_unit(a, lane);
      first_whole = true;
      hp = columns<HPL>(heads_of_group(a, rd.g));
      w.start(a, rd.b, rd.g, hp);
    }
  }
}

// The same for few units of moderate length, where launches and latencies
// count: the sequences' units take `ctas` CTAs each (a cluster), every one's
// tiles in equal shares over its warps, and the parts are joined out of shared
// memory: no second launch, no sums over the batch's lengths first.
// 1 x 2048 keys, 8 groups: 4.1 us on the device, 4 x 4096 6.2, 16 x 2048 9.8 (8.1
// from L2); equal shares of everything and a join took 8.6, 10.0 and 12.9.
constexpr int kUnitCtas = 8;   // of a cluster, at most
constexpr int kUnitTiles = 8;  // per warp, at most (see attention())
template <int DH, int HPL, int NB>
__global__ void __launch_bounds__(kAttnThreads, kAttnCtasPerSm) kv4_attn_unit_kernel(AttnArgs a) {
  using S = AttnShape<DH>;
  constexpr int MAXH = HPL * NB * 4 > 4 ? NB * 8 : 4;  // heads of a group
  static_assert(MAXH * (DH * 4 + 8) <= S::RING, "a warp's part lies in its ring");
  extern __shared__ __align__(128) uint8_t sm[];
  __shared__ float2 joined[MAXH];  // this CTA's (max in kUnit, sum)
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int C = a.ctas, u = blockIdx.x / C, rank = blockIdx.x - u * C, b = u / a.G, g = u - b * a.G;
  pdl_wait();
  pdl_launch_dependents();
  const int n = keys_of(a, b), tiles = tiles_of(n), H = heads_of_group(a, g);
  if (n == 0) {  // zeros
    if (rank == 0)
      for (int i = tid; i < H * (DH / 8); i += kAttnThreads)
        reinterpret_cast<uint4*>(out_row(a, b, g, i / (DH / 8), DH))[i % (DH / 8)] = make_uint4(0u, 0u, 0u, 0u);
    return;
  }
  const int share = (tiles + C * kAttnWarps - 1) / (C * kAttnWarps);
  const int first = (warp * C + rank) * share, count = min(share, tiles - first);
  uint8_t* mine = sm + warp * S::RING;
  if (count > 0) {
    const long long row = (static_cast<long long>(b) * a.G + g) * a.c.capacity + static_cast<long long>(first) * kTile;
    const uint8_t* pk = a.c.k_codes + row * S::ROW + lane * 16;
    const uint8_t* pv = a.c.v_codes + row * S::ROW + lane * 16;
    const uint8_t* pm = reinterpret_cast<const uint8_t*>(a.c.meta) + row * 8 + lane * 16;
    const int left = n - first * kTile;
    auto issue = [&](int i) {
      if (i < count)
        load_tile<DH>(a, smem_u32(mine) + i % kStages * S::TILE_BYTES, pk + static_cast<long long>(i) * kTile * S::ROW,
                      pv + static_cast<long long>(i) * kTile * S::ROW, pm + static_cast<long long>(i) * kTile * 8, left - i * kTile, lane);
      cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < kStages; ++i) issue(i);
    Warp<DH, HPL, NB> w;
    w.lr = lane >> 2;
    w.lc = lane & 3;
    asm volatile("mov.b32 %0, 0x41804180;" : "=r"(w.k16));
    const int hp = columns<HPL>(H);
    w.start(a, b, g, hp);
    for (int i = 0; i < count; ++i) {
      cp_async_wait<kStages - 1>();
      __syncwarp();
      w.any_tile(mine + i % kStages * S::TILE_BYTES, left - i * kTile, hp);
      __syncwarp();
      issue(i + kStages);
    }
    float* po = reinterpret_cast<float*>(mine);
    w.finish(a, b, g, hp, tiles == 1, po, reinterpret_cast<float2*>(po + MAXH * DH));
  }
  if (tiles == 1) return;  // the whole cluster
  // This CTA's warps (those with tiles come first), into warp 0's place.
  __syncthreads();
  const int have = min(kAttnWarps, ((tiles + share - 1) / share - rank + C - 1) / C);  // <= 0: none
  auto part_o = [&](int w) { return reinterpret_cast<float*>(sm + w * S::RING); };
  auto part_ml = [&](int w) { return reinterpret_cast<const float2*>(part_o(w) + MAXH * DH); };
  if (have > 0)
    for (int e = tid; e < H * DH; e += kAttnThreads) {
      const int h = e / DH;
      float m = -INFINITY, l = 0.0f, o = 0.0f;
      for (int w = 0; w < have; ++w) m = fmaxf(m, part_ml(w)[h].x);
      const float mu = m == -INFINITY ? 0.0f : m;
      for (int w = 0; w < have; ++w) {
        const float2 v = part_ml(w)[h];
        const float f = exp2_less(v.x, mu);
        l = fmaf(f, v.y, l);
        o = fmaf(f, part_o(w)[e], o);
      }
      part_o(0)[e] = o;
      if (e % DH == 0) joined[h] = make_float2(m, l);
    }
  const cooperative_groups::cluster_group cluster = cooperative_groups::this_cluster();
  cluster.sync();
  const int ctas = min(C, (tiles + share - 1) / share);  // those with tiles: the first ones
  for (int e = rank * kAttnThreads + tid; e < H * DH; e += C * kAttnThreads) {
    const int h = e / DH;
    float2 ml[kUnitCtas];
    float x[kUnitCtas], m = -INFINITY, l = 0.0f, o = 0.0f;
#pragma unroll
    for (int r = 0; r < kUnitCtas; ++r) {
      ml[r] = make_float2(-INFINITY, 0.0f);
      x[r] = 0.0f;
      if (r < ctas) {
        ml[r] = cluster.map_shared_rank(joined, r)[h];
        x[r] = cluster.map_shared_rank(part_o(0), r)[e];
        m = fmaxf(m, ml[r].x);
      }
    }
    const float mu = m == -INFINITY ? 0.0f : m;
#pragma unroll
    for (int r = 0; r < kUnitCtas; ++r) {
      const float f = exp2_less(ml[r].x, mu);
      l = fmaf(f, ml[r].y, l);
      o = fmaf(f, x[r], o);
    }
    out_row(a, b, g, h, DH)[e - h * DH] = __bfloat16_as_ushort(__float2bfloat16_rn(o / l));
  }
  cluster.sync();  // the others' memory stays until it is read
}

// Joins the parts of the units that lie in several shares: one CTA per unit
// and head, DH threads per part, blockDim / DH parts at a time (about as many
// as a unit has: 1 x 1M keys have 297 per unit).
constexpr int kJoinRows = 16;
template <int DH>
__global__ void __launch_bounds__(kJoinRows * DH) kv4_join_kernel(AttnArgs a) {
  __shared__ float jo[kJoinRows * DH], jm[kJoinRows], jl[kJoinRows];
  pdl_wait();
  pdl_launch_dependents();
  const int u = blockIdx.x / a.H, h = blockIdx.x - u * a.H;
  const int b = u / a.G, g = u - b * a.G;
  const int tb = tiles_of(keys_of(a, b));
  if (tb == 0 || h >= heads_of_group(a, g)) return;
  const long long share = a.starts[a.B], s0 = a.starts[b] + static_cast<long long>(g) * tb;
  const long long p0 = s0 / share, p1 = (s0 + tb - 1) / share;  // the warps of its tiles
  if (p0 == p1) return;
  const int row = threadIdx.x / DH, rows = blockDim.x / DH, d = threadIdx.x % DH;
  const int parts = static_cast<int>(p1 - p0 + 1);
  const float2* ml = a.part_ml + (p0 + u) * a.H + h;
  const float* po = a.part_o + ((p0 + u) * a.H + h) * DH + d;
  float m = -INFINITY, o = 0.0f, l = 0.0f;
#pragma unroll 4
  for (int c = row; c < parts; c += rows) m = fmaxf(m, ml[static_cast<long long>(c) * a.H].x);
  const float mu = m == -INFINITY ? 0.0f : m;
#pragma unroll 4
  for (int c = row; c < parts; c += rows) {
    const float2 v = ml[static_cast<long long>(c) * a.H];
    const float w = exp2_less(v.x, mu);
    l = fmaf(w, v.y, l);
    o = fmaf(w, po[static_cast<long long>(c) * a.H * DH], o);
  }
  jo[threadIdx.x] = o;
  if (d == 0) {
    jm[row] = m;
    jl[row] = l;
  }
  __syncthreads();
  if (row != 0) return;
  for (int r = 1; r < rows; ++r) m = fmaxf(m, jm[r]);
  const float all = m == -INFINITY ? 0.0f : m;
  o = l = 0.0f;
  for (int r = 0; r < rows; ++r) {
    const float w = exp2_less(jm[r], all);
    l = fmaf(w, jl[r], l);
    o = fmaf(w, jo[r * DH + d], o);
  }
  out_row(a, b, g, h, DH)[d] = __bfloat16_as_ushort(__float2bfloat16_rn(o / l));
}

int attn_ctas(int B, int G, int T) {
  int dev = 0, sms = 148;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  const long long most = static_cast<long long>(sms < 148 ? sms : 148) * kAttnCtasPerSm,
                  tiles = static_cast<long long>(B) * G * tiles_of(T);
  return static_cast<int>(tiles < most ? tiles : most);
}

template <int DH, int HPL, int NB>
int launch_attn(const AttnArgs& a, void* stream) {
  const int e = ensure_smem<kv4_attn_kernel<DH, HPL, NB>>(static_cast<int>(AttnShape<DH>::smem()));
  if (e != cudaSuccess) return e;
  return launch_pdl(kv4_attn_kernel<DH, HPL, NB>, dim3(attn_ctas(a.B, a.G, a.T)), dim3(kAttnThreads),
                    AttnShape<DH>::smem(), stream, a);
}

template <int DH, int HPL, int NB>
int launch_unit(AttnArgs a, int ctas, void* stream) {
  a.ctas = ctas;
  const int e = ensure_smem<kv4_attn_unit_kernel<DH, HPL, NB>>(static_cast<int>(AttnShape<DH>::smem()));
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {static_cast<unsigned>(ctas), 1, 1};
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(a.B) * a.G * ctas);
  cfg.blockDim = dim3(kAttnThreads);
  cfg.dynamicSmemBytes = AttnShape<DH>::smem();
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return static_cast<int>(cudaLaunchKernelEx(&cfg, kv4_attn_unit_kernel<DH, HPL, NB>, a));
}

template <int DH>
int attention(const AttnArgs& a, void* stream) {
  // A cluster per unit as long as all are resident (256: clusters do not fill
  // the SMs' last places; 72 units with 4 CTAs each took two rounds) and a
  // warp has at most 8 tiles. 16 x 8192 keys of 8 groups, in us: equal lengths
  // 28 against 34 for equal shares, lengths spread evenly 27 (28), one long
  // sequence among short ones 18 (18). 2 x 32768: 17.2 (16.8).
  const long long all = static_cast<long long>(a.B) * a.G;
  int ctas = kUnitCtas;
  while (ctas > 1 && all * ctas > 256) ctas /= 2;
  if (all <= 148 * kAttnCtasPerSm && a.T <= ctas * kAttnWarps * kTile * kUnitTiles)
    return a.H <= 4 ? launch_unit<DH, 1, 1>(a, ctas, stream)
           : a.H <= 8 ? launch_unit<DH, 2, 1>(a, ctas, stream)
                      : launch_unit<DH, 2, 2>(a, ctas, stream);
  const int e = a.H <= 4 ? launch_attn<DH, 1, 1>(a, stream)
                : a.H <= 8 ? launch_attn<DH, 2, 1>(a, stream)
                           : launch_attn<DH, 2, 2>(a, stream);
  if (e != cudaSuccess || a.T <= kTile) return e;  // one tile per unit: nothing to join
  // Rows: as many as a unit has parts, but one wave of threads (33 x 5003 keys
  // of 32 heads: 37 us with 16 rows, 29 with 4).
  const long long units = static_cast<long long>(a.B) * a.G, parts = kMaxAttnWarps / units + 2;
  int rows = 1;
  while (rows < kJoinRows && rows < parts && units * a.H * DH * rows * 2 <= 148 * 2048) rows *= 2;
  return launch_pdl(kv4_join_kernel<DH>, dim3(static_cast<unsigned>(units) * a.H), dim3(rows * DH), 0, stream, a);
}

// Workspace: the parts' slots, then the sequences' starts.
struct AttnWs {
  size_t ml, starts, total;
};
AttnWs attn_ws(int B, int G, int H, int dh) {
  const size_t slots = static_cast<size_t>(B) * G + kMaxAttnWarps;
  AttnWs w;
  w.ml = (slots * H * dh * 4 + 255) / 256 * 256;
  w.starts = (w.ml + slots * H * 8 + 255) / 256 * 256;
  w.total = w.starts + (static_cast<size_t>(B) + 1) * 8;
  return w;
}

// CTAs of the append and the read, `rows` rows of a CTA at a time: 16 per SM
// at most. 262144 rows: 25.7 us and 14.7 (8 per SM: 26.7 and 15.1; 28: 26.9
// and 14.4).
unsigned store_ctas(int B, int G, int T, int rows) {
  const long long n = (static_cast<long long>(B) * G * T + rows - 1) / rows;
  return static_cast<unsigned>(n < 148 * 16 ? n : 148 * 16);
}

}  // namespace kv4_impl
using namespace kv4_impl;

int kv4_append(int B, int G, int T, int dh, const uint16_t* K, const uint16_t* V, const int32_t* start, int start0,
               const int32_t* count, const gqe_kv4& cache, void* stream) {
  const StoreArgs a{K, V, nullptr, nullptr, cache, start, start0, count, B, G, T, Divisor(T), Divisor(G)};
  const dim3 grid(store_ctas(B, G, T, kv4_impl::kThreads / (dh / 16)));
  return dh == 64 ? launch_pdl(append_kernel<64>, grid, dim3(kv4_impl::kThreads), 0, stream, a)
                  : launch_pdl(append_kernel<32>, grid, dim3(kv4_impl::kThreads), 0, stream, a);
}

int kv4_read(int B, int G, int T, int dh, const gqe_kv4& cache, const int32_t* start, const int32_t* count,
             uint16_t* K, uint16_t* V, void* stream) {
  const StoreArgs a{nullptr, nullptr, K, V, cache, start, 0, count, B, G, T, Divisor(T), Divisor(G)};
  const dim3 grid(store_ctas(B, G, T, kv4_impl::kThreads / (dh / 8)));
  return dh == 64 ? launch_pdl(read_kernel<64>, grid, dim3(kv4_impl::kThreads), 0, stream, a)
                  : launch_pdl(read_kernel<32>, grid, dim3(kv4_impl::kThreads), 0, stream, a);
}

size_t kv4_attention_ws_bytes(int B, int G, int H, int dh) { return attn_ws(B, G, H, dh).total; }

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
  const AttnWs w = attn_ws(B, G, a.H, dh);
  a.part_o = static_cast<float*>(ws);
  a.part_ml = reinterpret_cast<float2*>(static_cast<char*>(ws) + w.ml);
  a.starts = reinterpret_cast<long long*>(static_cast<char*>(ws) + w.starts);
  a.out = out;
  a.ldo = ldo;
  a.scale_log2 = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(dh)));
  return dh == 64 ? attention<64>(a, stream) : attention<32>(a, stream);
}

}  // namespace gqe
