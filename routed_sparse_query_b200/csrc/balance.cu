// Balance loss of the router: per-expert counts, loss and logit gradient.
//
// With p = softmax of a group's M logits, n counted rows (mask != 0), c[g, j]
// the number of counted rows whose selection holds expert j of group g:
//   f = c / (k n), P = (1/n) sum p
//   L_balance = (M / G) sum_{g, j} f P          (1 where f and P are uniform)
//   L_z       = 1/(n G) sum_{rows, g} logsumexp(z)^2
//   dz[j] = c_balance M / (G n) p_j (f_j - sum_i p_i f_i) + c_z 2/(n G) lse p_j
// (the counts are a discrete choice and carry no gradient).
//
// Two passes over z, because every row's gradient needs the counts of all
// rows: stats (counts, sum of p, sum of lse^2; also what ranks of a
// data-parallel run add up before the gradient) and gradient. Both are bound
// by HBM (stats reads 4 bytes per logit and per selection, the gradient
// reads and writes 4 per logit). LANES lanes take one (row, group) pair, each
// with PER of its logits in registers; a thread keeps to one group, so that
// its partial sums stay in registers until the end. Sums run in fp32 per
// thread and CTA and in fp64 over the CTAs, always in the same order.
#include <cuda_runtime.h>

#include <cmath>

#include "gqe_internal.h"
#include "ptx.cuh"

namespace gqe {

namespace balance_impl {

constexpr int kThreads = 256;
constexpr int kMaxCtas = 148 * 4;

struct BalanceArgs {
  const float* z;       // [R, G M]
  const int32_t* idx;   // [R, G, k]
  const uint8_t* mask;  // [R] or null
  long long R;
  int G, M, k;
  float* part;          // [CTAs][2 N + 2]: counts (as int bits), sum p, sum lse^2, rows (int bits)
};

template <int LANES, int PER>
struct Pair {
  float z[PER], p[PER];
  float lse;
  // Softmax of the pair's logits; lane q holds experts q, q + LANES, ...
  // `live` lanes only; the others join the exchanges.
  __device__ __forceinline__ void load(const float* zp, int q, int M, bool live) {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int j = q + i * LANES;
      z[i] = live && j < M ? __ldg(zp + j) : -INFINITY;
      m = fmaxf(m, z[i]);
    }
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      p[i] = live && q + i * LANES < M ? expf(z[i] - m) : 0.0f;
      s += p[i];
    }
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
#pragma unroll
    for (int i = 0; i < PER; ++i) p[i] = live ? p[i] / s : 0.0f;
    lse = live ? m + logf(s) : 0.0f;
  }
};

// Threads of a CTA: `rows` rows x G groups x LANES lanes (the rest idle).
template <int LANES, int PER>
__global__ void __launch_bounds__(kThreads) stats_kernel(BalanceArgs a) {
  __shared__ float sp[kThreads * PER];
  __shared__ int sc[kThreads * PER];
  __shared__ float sl[kThreads];
  __shared__ int sn[kThreads];
  pdl_wait();
  pdl_launch_dependents();
  const int gl = a.G * LANES, rows = kThreads / gl;
  const int tid = threadIdx.x, rl = tid / gl, g = (tid % gl) / LANES, q = tid % LANES;
  const bool in = rl < rows;
  float psum[PER], lsum = 0.0f;
  int cnt[PER], n = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    psum[i] = 0.0f;
    cnt[i] = 0;
  }
  for (long long r0 = static_cast<long long>(blockIdx.x) * rows; r0 < a.R; r0 += static_cast<long long>(gridDim.x) * rows) {
    const long long r = r0 + rl;
    const bool live = in && r < a.R && (a.mask == nullptr || a.mask[r] != 0);
    Pair<LANES, PER> w;
    w.load(a.z + (r * a.G + g) * a.M, q, a.M, live);
    if (live) {
#pragma unroll
      for (int i = 0; i < PER; ++i) psum[i] += w.p[i];
      for (int s = 0; s < a.k; ++s) {
        const int j = __ldg(a.idx + (r * a.G + g) * a.k + s);
#pragma unroll
        for (int i = 0; i < PER; ++i) cnt[i] += j == q + i * LANES ? 1 : 0;
      }
      if (q == 0) lsum = fmaf(w.lse, w.lse, lsum);
      if (g == 0 && q == 0) ++n;
    }
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    sp[tid * PER + i] = psum[i];
    sc[tid * PER + i] = cnt[i];
  }
  sl[tid] = lsum;
  sn[tid] = n;
  __syncthreads();
  const int N = a.G * a.M;
  float* out = a.part + static_cast<size_t>(blockIdx.x) * (2 * N + 2);
  for (int e = tid; e < N; e += kThreads) {
    const int eg = e / a.M, j = e - eg * a.M;
    float s = 0.0f;
    int c = 0;
    for (int r = 0; r < rows; ++r) {
      const int at = ((r * a.G + eg) * LANES + j % LANES) * PER + j / LANES;
      s += sp[at];
      c += sc[at];
    }
    out[e] = __int_as_float(c);
    out[N + e] = s;
  }
  if (tid == kThreads - 1) {
    float s = 0.0f;
    int c = 0;
    for (int i = 0; i < kThreads; ++i) {
      s += sl[i];
      c += sn[i];
    }
    out[2 * N] = s;
    out[2 * N + 1] = __int_as_float(c);
  }
}

// One CTA: the sums over the stats CTAs. 8 lanes per column.
__global__ void __launch_bounds__(1024) finish_kernel(const float* part, int ctas, int N, int32_t* counts, float* sums) {
  pdl_wait();
  pdl_launch_dependents();
  const int cols = 2 * N + 2, q = threadIdx.x % 8;
  for (int c0 = 0; c0 < cols; c0 += 128) {
    const int col = c0 + threadIdx.x / 8;
    const bool whole = col < N || col == 2 * N + 1;
    double s = 0.0;
    if (col < cols)
      for (int i = q; i < ctas; i += 8) {
        const float v = part[static_cast<size_t>(i) * cols + col];
        s += whole ? static_cast<double>(__float_as_int(v)) : static_cast<double>(v);
      }
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (q == 0 && col < cols) {
      if (col < N) counts[col] = static_cast<int32_t>(s);
      else if (col <= 2 * N) sums[col - N] = static_cast<float>(s);
      else counts[N] = static_cast<int32_t>(s);
    }
  }
}

struct GradArgs {
  const float* z;
  const uint8_t* mask;
  const int32_t* counts;  // [N + 1]
  const float* sums;      // [N + 1]
  long long R;
  int G, M, k;
  float c_balance, c_z;
  float* loss;            // [3] or null
  float* dz;              // or null: the loss only
  int accumulate;
};

template <int LANES, int PER>
__global__ void __launch_bounds__(kThreads) grad_kernel(GradArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  const int N = a.G * a.M, tid = threadIdx.x;
  const double n = a.counts[N] > 0 ? static_cast<double>(a.counts[N]) : 1.0;
  if (blockIdx.x == 0 && a.loss != nullptr && tid < 32) {
    double s = 0.0;
    for (int e = tid; e < N; e += 32) s += static_cast<double>(a.counts[e]) * a.sums[e];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (tid == 0) {
      const double bal = static_cast<double>(a.M) / a.G * s / (a.k * n) / n, zl = a.sums[N] / (a.G * n);
      a.loss[0] = static_cast<float>(a.c_balance * bal + a.c_z * zl);
      a.loss[1] = static_cast<float>(bal);
      a.loss[2] = static_cast<float>(zl);
    }
  }
  if (a.dz == nullptr) return;
  const int gl = a.G * LANES, rows = kThreads / gl;
  const int rl = tid / gl, g = (tid % gl) / LANES, q = tid % LANES;
  const bool in = rl < rows;
  // Loads less their mean 1/M, from whole numbers: the softmax's Jacobian
  // does not see the mean, and near balance it would cost fp32 most bits of
  // what is left (f_j - sum p f is then far below f_j).
  float f[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int j = q + i * LANES;
    f[i] = in && j < a.M ? static_cast<float>((static_cast<double>(a.counts[g * a.M + j]) * a.M - a.k * n) / (a.M * a.k * n))
                         : 0.0f;
  }
  const float cb = static_cast<float>(static_cast<double>(a.c_balance) * a.M / (a.G * n));
  const float cz = static_cast<float>(2.0 * a.c_z / (a.G * n));
  for (long long r0 = static_cast<long long>(blockIdx.x) * rows; r0 < a.R; r0 += static_cast<long long>(gridDim.x) * rows) {
    const long long r = r0 + rl;
    const bool at = in && r < a.R;
    const bool live = at && (a.mask == nullptr || a.mask[r] != 0);
    Pair<LANES, PER> w;
    w.load(a.z + (r * a.G + g) * a.M, q, a.M, live);
    float mean = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i) mean = fmaf(w.p[i], f[i], mean);
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) mean += __shfl_xor_sync(0xffffffffu, mean, o);
    float* out = a.dz + (r * a.G + g) * a.M;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int j = q + i * LANES;
      if (!at || j >= a.M) continue;
      const float d = live ? w.p[i] * (cb * (f[i] - mean) + cz * w.lse) : 0.0f;
      if (!a.accumulate) out[j] = d;
      else if (live) out[j] += d;
    }
  }
}

// Instantiation for M: up to 8 logits in one lane, more on 8 lanes.
template <typename F>
int with_shape(int M, F f) {
  if (M <= 1) return f(std::integral_constant<int, 1>{}, std::integral_constant<int, 1>{});
  if (M <= 2) return f(std::integral_constant<int, 1>{}, std::integral_constant<int, 2>{});
  if (M <= 4) return f(std::integral_constant<int, 1>{}, std::integral_constant<int, 4>{});
  if (M <= 8) return f(std::integral_constant<int, 1>{}, std::integral_constant<int, 8>{});
  if (M <= 16) return f(std::integral_constant<int, 8>{}, std::integral_constant<int, 2>{});
  if (M <= 32) return f(std::integral_constant<int, 8>{}, std::integral_constant<int, 4>{});
  return f(std::integral_constant<int, 8>{}, std::integral_constant<int, 8>{});
}

int ctas_for(long long R, int G, int M) {
  const int rows = kThreads / (G * (M <= 8 ? 1 : 8));
  const long long n = (R + rows - 1) / rows;
  return static_cast<int>(n < kMaxCtas ? n : kMaxCtas);
}

}  // namespace balance_impl
using namespace balance_impl;

size_t balance_ws_bytes(int N) { return static_cast<size_t>(kMaxCtas) * (2 * N + 2) * 4; }

int balance_stats(const float* z, const int32_t* idx, const uint8_t* mask, long long R, int G, int M, int k,
                  int32_t* counts, float* sums, void* ws, void* stream) {
  const BalanceArgs a{z, idx, mask, R, G, M, k, static_cast<float*>(ws)};
  const int ctas = ctas_for(R, G, M);
  const int e = with_shape(M, [&](auto lanes, auto per) {
    return static_cast<int>(launch_pdl(stats_kernel<decltype(lanes)::value, decltype(per)::value>, dim3(ctas),
                                       dim3(balance_impl::kThreads), 0, stream, a));
  });
  if (e != cudaSuccess) return e;
  return launch_pdl(finish_kernel, dim3(1), dim3(1024), 0, stream, static_cast<const float*>(a.part), ctas, G * M,
                    counts, sums);
}

int balance_grad(const float* z, const uint8_t* mask, const int32_t* counts, const float* sums, long long R, int G,
                 int M, int k, float c_balance, float c_z, float* loss, float* dz, bool accumulate, void* stream) {
  const GradArgs a{z, mask, counts, sums, R, G, M, k, c_balance, c_z, loss, dz, accumulate ? 1 : 0};
  const int ctas = dz != nullptr ? ctas_for(R, G, M) : 1;
  return with_shape(M, [&](auto lanes, auto per) {
    return static_cast<int>(launch_pdl(grad_kernel<decltype(lanes)::value, decltype(per)::value>, dim3(ctas),
                                       dim3(balance_impl::kThreads), 0, stream, a));
  });
}

}  // namespace gqe
