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
// Split over spans of 256 keys; per head a span writes its unnormalised
// output and (max, sum), merged by a second kernel.
constexpr int kSpan = 256;

struct AttnArgs {
  const uint16_t* Q;   // [B][G][k][dh]
  const uint16_t* Qs;  // [B][dh] or null
  gqe_kv4 c;
  const int32_t* lens;
  int len_add, B, G, T, k, H, spans;
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

template <int DH>
__global__ void __launch_bounds__(kSpan) kv4_partial_kernel(AttnArgs a) {
  __shared__ float q[DH], p[kSpan], red[kSpan / 32];
  pdl_wait();
  pdl_launch_dependents();
  const int span = blockIdx.x, g = blockIdx.y % a.G, b = blockIdx.y / a.G, tid = threadIdx.x;
  const int n = keys_of(a, b);
  if (span * kSpan >= n) return;
  const int heads = a.k + (g == 0 && a.Qs != nullptr ? 1 : 0);
  const long long row0 = (static_cast<long long>(b) * a.G + g) * a.c.capacity + span * kSpan;
  const int keys = min(kSpan, n - span * kSpan);
  const uint2 m = tid < keys ? reinterpret_cast<const uint2*>(a.c.meta)[row0 + tid] : make_uint2(0u, 0u);
  for (int h = 0; h < heads; ++h) {
    const uint16_t* qp = h < a.k ? a.Q + ((static_cast<long long>(b) * a.G + g) * a.k + h) * DH : a.Qs + static_cast<long long>(b) * DH;
    __syncthreads();
    if (tid < DH) q[tid] = bf16_f(qp[tid]) * a.scale_log2;
    __syncthreads();
    float s = -INFINITY;
    if (tid < keys) {
      const uint32_t* kc = reinterpret_cast<const uint32_t*>(a.c.k_codes) + (row0 + tid) * (DH / 8);
      const float ks = bf16_f(m.x & 0xffffu), kz = bf16_f(m.x >> 16);
      s = 0.0f;
      for (int w = 0; w < DH / 8; ++w)
        for (int i = 0; i < 8; ++i) s = fmaf(q[8 * w + i], fmaf(ks, static_cast<float>((kc[w] >> (4 * i)) & 15u), kz), s);
    }
    float mx = s;
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    if (tid % 32 == 0) red[tid / 32] = mx;
    __syncthreads();
    mx = red[0];
    for (int w = 1; w < kSpan / 32; ++w) mx = fmaxf(mx, red[w]);
    const float e = tid < keys ? exp2f(s - mx) : 0.0f;
    p[tid] = e;
    float l = e;
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    __syncthreads();
    if (tid % 32 == 0) red[tid / 32] = l;
    __syncthreads();
    const long long at = ((static_cast<long long>(b) * a.G + g) * a.spans + span) * a.H + h;
    if (tid == 0) {
      l = 0.0f;
      for (int w = 0; w < kSpan / 32; ++w) l += red[w];
      a.part_ml[at] = make_float2(mx, l);
    }
    if (tid < DH) {
      float o = 0.0f;
      for (int u = 0; u < keys; ++u) {
        const uint32_t mv = reinterpret_cast<const uint2*>(a.c.meta)[row0 + u].y;
        const uint8_t c = a.c.v_codes[(row0 + u) * (DH / 2) + tid / 2];
        o = fmaf(p[u], fmaf(bf16_f(mv & 0xffffu), static_cast<float>(tid & 1 ? c >> 4 : c & 15), bf16_f(mv >> 16)), o);
      }
      a.part_o[at * DH + tid] = o;
    }
  }
}

// One CTA per (sequence, group), one thread per (head, element).
template <int DH>
__global__ void __launch_bounds__(1024) kv4_merge_kernel(AttnArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  const int g = blockIdx.x % a.G, b = blockIdx.x / a.G;
  const int h = threadIdx.x / DH, d = threadIdx.x % DH;
  if (h >= a.k + (g == 0 && a.Qs != nullptr ? 1 : 0)) return;
  const int spans = (keys_of(a, b) + kSpan - 1) / kSpan;
  const long long at0 = (static_cast<long long>(b) * a.G + g) * a.spans;
  float m = -INFINITY;
  for (int c = 0; c < spans; ++c) m = fmaxf(m, a.part_ml[(at0 + c) * a.H + h].x);
  float o = 0.0f, l = 0.0f;
  for (int c = 0; c < spans; ++c) {
    const float2 ml = a.part_ml[(at0 + c) * a.H + h];
    const float w = exp2f(ml.x - m);
    l = fmaf(w, ml.y, l);
    o = fmaf(w, a.part_o[((at0 + c) * a.H + h) * DH + d], o);
  }
  const int col = h < a.k ? g * a.k + h : a.G * a.k;
  a.out[static_cast<long long>(b) * a.ldo + col * DH + d] = __bfloat16_as_ushort(__float2bfloat16_rn(spans > 0 ? o / l : 0.0f));
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
  const size_t units = static_cast<size_t>(B) * G * ((static_cast<size_t>(T) + kSpan - 1) / kSpan) * H;
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
  a.spans = (T + kSpan - 1) / kSpan;
  const size_t units = static_cast<size_t>(B) * G * a.spans * a.H;
  a.part_o = static_cast<float*>(ws);
  a.part_ml = reinterpret_cast<float2*>(static_cast<char*>(ws) + (units * dh * 4 + 255) / 256 * 256);
  a.out = out;
  a.ldo = ldo;
  a.scale_log2 = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(dh)));
  const dim3 grid(a.spans, static_cast<unsigned>(B) * G);
  int e = dh == 64 ? launch_pdl(kv4_partial_kernel<64>, grid, dim3(kSpan), 0, stream, a)
                   : launch_pdl(kv4_partial_kernel<32>, grid, dim3(kSpan), 0, stream, a);
  if (e != cudaSuccess) return e;
  return dh == 64 ? launch_pdl(kv4_merge_kernel<64>, dim3(static_cast<unsigned>(B) * G), dim3(a.H * 64), 0, stream, a)
                  : launch_pdl(kv4_merge_kernel<32>, dim3(static_cast<unsigned>(B) * G), dim3(a.H * 32), 0, stream, a);
}

}  // namespace gqe
