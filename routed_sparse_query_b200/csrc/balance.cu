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
// thread, per CTA and over the up to 19 CTAs that a thread of the last kernel
// takes, and in fp64 over those threads (in one cluster: over its CTAs), always
// in the same order.
//
// Measured: 262144 rows of 8 x 4 logits, k = 2, masked: 27 us (84 MB; in a
// short run 13 for the two launches of stats, 9 for the gradient, whose logits
// come from L2): load latency of short passes, not bandwidth. As many CTAs as
// are resident, five rows per thread in flight: 23 us in the short run, 29 with
// a quarter more CTAs and four rows. 2048 rows of 8 x 2: 12 us, two launches.
// 262144 rows of one group of 64, k = 4: 61 us (floor 32), 24 and 32 of them the
// two large kernels: 72 to 80 registers leave 28 % of the warps, which wait for
// their loads first and for the six to nine exchanges among eight lanes of each
// pair next (2.0 to 2.2 instructions per cycle, DRAM 35 % busy).
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <cmath>

#include "gqe_internal.h"
#include "ptx.cuh"

namespace gqe {

namespace balance_impl {

constexpr int kThreads = 256;
constexpr int kMaxCtas = 148 * 4;  // resident CTAs
constexpr int kAheadFew = 5, kAheadMany = 3;  // rows of a thread in flight, up to 4 logits each and more
constexpr unsigned kCluster = 8;

struct BalanceArgs {
  const float* z;       // [R, G M]
  const int32_t* idx;   // [R, G, k]
  const uint8_t* mask;  // [R] or null
  long long R;
  int G, M, k;
  float* part;          // [CTAs][2 N + 2]: counts (as int bits), sum p, sum lse^2, rows (int bits)
  int32_t* counts;
  float* sums;
};

// Column of a partial row to its place in the outputs.
__device__ __forceinline__ void store_sum(int col, int N, double s, int32_t* counts, float* sums) {
  if (col < N) counts[col] = static_cast<int32_t>(s);
  else if (col <= 2 * N) sums[col - N] = static_cast<float>(s);
  else counts[N] = static_cast<int32_t>(s);
}

// Which logits of a (row, group) pair lane q holds: experts q, q + LANES, ...
// EXACT: in one lane, all (M = PER); in several, runs of four (M a multiple of
// 4; 262144 rows of one group of 64 experts: 75 us, 81 with single ones).
template <int LANES, int PER, bool EXACT>
__device__ __forceinline__ int expert_of(int q, int i) {
  return EXACT && LANES > 1 ? i / 4 * 4 * LANES + 4 * q + i % 4 : q + i * LANES;
}
// Its place among the pair's LANES PER values.
template <int LANES, int PER, bool EXACT>
__device__ __forceinline__ int place_of(int j) {
  return EXACT && LANES > 1 ? j / 4 % LANES * PER + j / (4 * LANES) * 4 + j % 4 : j % LANES * PER + j / LANES;
}

template <int LANES, int PER, bool EXACT>
__device__ __forceinline__ void load_logits(const float* zp, int q, int M, bool at, float (&z)[PER]) {
#pragma unroll
  for (int i = 0; i < PER; ++i) z[i] = -INFINITY;
  if (!at) return;
  if constexpr (EXACT && PER % 4 == 0) {
#pragma unroll
    for (int i = 0; i < PER; i += 4) {
      const int j = expert_of<LANES, PER, EXACT>(q, i);
      if (LANES > 1 && j >= M) continue;
      const float4 v = *reinterpret_cast<const float4*>(zp + j);
      z[i] = v.x; z[i + 1] = v.y; z[i + 2] = v.z; z[i + 3] = v.w;
    }
  } else if constexpr (EXACT && PER == 2) {
    const float2 v = *reinterpret_cast<const float2*>(zp);
    z[0] = v.x; z[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (q + i * LANES < M) z[i] = zp[q + i * LANES];
  }
}

// z to exp(z - max); 1 / their sum and log sum exp(z). exp and log are the
// hardware's (2^-21). The maximum is taken off before the scaling to base 2,
// which would overflow for a group of logits that are all the type's lowest
// value (every expert switched off: equal probabilities).
template <int LANES, int PER>
__device__ __forceinline__ void softmax(float (&z)[PER], float* inv, float* lse) {
  constexpr float kLog2e = 1.44269504088896340736f;
  float m = z[0];
#pragma unroll
  for (int i = 1; i < PER; ++i) m = fmaxf(m, z[i]);
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(z[i]) : "f"((z[i] - m) * kLog2e));
    s += z[i];
  }
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(*inv) : "f"(s));
  float l2;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(l2) : "f"(s));
  *lse = fmaf(l2, 0.69314718055994530942f, m);
}

// Threads of a CTA: `rows` rows x G groups x LANES lanes (the rest idle),
// several rows of each thread in flight. CLUSTER: the grid is one cluster, whose
// first CTA adds up the others' sums out of their shared memory (no second
// launch; see balance_stats).
template <int LANES, int PER, bool EXACT, bool CLUSTER>
__global__ void __launch_bounds__(kThreads, PER <= 4 ? 4 : 3) stats_kernel(BalanceArgs a) {
  constexpr int kAhead = PER <= 4 ? kAheadFew : kAheadMany;
  __shared__ float sp[kThreads * PER];
  // Counts per thread; or, with several lanes to a pair, per CTA: lane q takes
  // the row's selections q, q + LANES, ... and adds to their experts' (whole
  // numbers: in any order; every lane comparing all k selections with its
  // experts: 67 us against 57 at 262144 rows of 2 x 32, k = 4).
  constexpr bool HIST = LANES > 1;
  __shared__ int sc[HIST ? kMaxExperts : kThreads * PER];
  __shared__ float sl[kThreads];
  __shared__ int sn[kThreads];
  const int gl = a.G * LANES, rows = kThreads / gl;
  const int tid = threadIdx.x, rl = tid / gl, g = (tid % gl) / LANES, q = tid % LANES;
  if (HIST) {
    if (tid < kMaxExperts) sc[tid] = 0;
    __syncthreads();
  }
  pdl_wait();
  pdl_launch_dependents();
  const bool in = rl < rows;
  const long long step = static_cast<long long>(gridDim.x) * rows;
  float psum[PER], lsum = 0.0f;
  int cnt[PER], n = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    psum[i] = 0.0f;
    cnt[i] = 0;
  }
  auto count = [&](int j) {
    if constexpr (HIST) {
      if (j >= 0 && j < a.M) atomicAdd(&sc[g * a.M + j], 1);
    } else {
#pragma unroll
      for (int i = 0; i < PER; ++i) cnt[i] += j == expert_of<LANES, PER, EXACT>(q, i) ? 1 : 0;
    }
  };
  const long long zs = step * a.G * a.M, is = step * a.G * a.k;
  long long r = static_cast<long long>(blockIdx.x) * rows + rl;
  const float* zp = a.z + (r * a.G + g) * a.M;
  const int32_t* ip0 = a.idx + (r * a.G + g) * a.k;
  for (long long r0 = r - rl; r0 < a.R; r0 += kAhead * step, r += kAhead * step, zp += kAhead * zs, ip0 += kAhead * is) {
    float z[kAhead][PER];
    bool live[kAhead];
    int sel[kAhead][2];  // the selections of a row that counts, if k <= 2 (HIST: this lane's first)
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      live[u] = in && r + u * step < a.R;
      load_logits<LANES, PER, EXACT>(zp + u * zs, q, a.M, live[u], z[u]);
      sel[u][0] = sel[u][1] = -1;
    }
    // What is the same for all rows is asked once for all of them.
    if (HIST) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (live[u] && q < a.k) sel[u][0] = ip0[u * is + q];
    } else if (a.k == 2) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (live[u]) {
          const int2 v = *reinterpret_cast<const int2*>(ip0 + u * is);
          sel[u][0] = v.x;
          sel[u][1] = v.y;
        }
    } else if (a.k == 1) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (live[u]) sel[u][0] = ip0[u * is];
    }
    if (a.mask != nullptr) {
      uint8_t on[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) on[u] = live[u] ? a.mask[r + u * step] : 0;
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        live[u] = on[u] != 0;
        sel[u][0] = live[u] ? sel[u][0] : -1;
        sel[u][1] = live[u] ? sel[u][1] : -1;
      }
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      float inv, lse;
      softmax<LANES, PER>(z[u], &inv, &lse);
#pragma unroll
      for (int i = 0; i < PER; ++i) psum[i] = live[u] ? fmaf(z[u][i], inv, psum[i]) : psum[i];
      lsum = live[u] && q == 0 ? fmaf(lse, lse, lsum) : lsum;
      n += live[u] ? 1 : 0;
    }
    if (HIST) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        count(sel[u][0]);
        if (live[u])
          for (int s = q + LANES; s < a.k; s += LANES) count(ip0[u * is + s]);
      }
    } else if (a.k <= 2) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) count(sel[u][0]);
      if (a.k == 2) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) count(sel[u][1]);
      }
    } else {
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (live[u])
          for (int s = 0; s < a.k; ++s) count(ip0[u * is + s]);
    }
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    sp[tid * PER + i] = psum[i];
    if (!HIST) sc[tid * PER + i] = cnt[i];
  }
  sl[tid] = lsum;
  sn[tid] = g == 0 && q == 0 ? n : 0;
  __syncthreads();
  const int N = a.G * a.M;
  __shared__ float fin[CLUSTER ? 2 * kMaxExperts + 2 : 1];
  float* out = CLUSTER ? fin : a.part + static_cast<size_t>(blockIdx.x) * (2 * N + 2);
  for (int e = tid; e < N; e += kThreads) {
    const int eg = e / a.M, j = e - eg * a.M;
    float s = 0.0f;
    int c = 0;
    for (int r = 0; r < rows; ++r) {
      const int at = (r * a.G + eg) * LANES * PER + place_of<LANES, PER, EXACT>(j);
      s += sp[at];
      c += HIST ? 0 : sc[at];
    }
    if (HIST) c = sc[e];
    out[e] = __int_as_float(c);
    out[N + e] = s;
  }
  if (tid >= kThreads - 32) {  // the last warp: the two sums over all threads
    float s = 0.0f;
    int c = 0;
    for (int i = tid & 31; i < kThreads; i += 32) {
      s += sl[i];
      c += sn[i];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      s += __shfl_xor_sync(0xffffffffu, s, o);
      c += __shfl_xor_sync(0xffffffffu, c, o);
    }
    if (tid == kThreads - 1) {
      out[2 * N] = s;
      out[2 * N + 1] = __int_as_float(c);
    }
  }
  if constexpr (CLUSTER) {
    const cooperative_groups::cluster_group cluster = cooperative_groups::this_cluster();
    cluster.sync();
    if (blockIdx.x == 0 && tid < 2 * N + 2) {
      const bool whole = tid < N || tid == 2 * N + 1;
      double s = 0.0;
      for (unsigned i = 0; i < gridDim.x; ++i) {
        const float v = cluster.map_shared_rank(fin, i)[tid];
        s += whole ? static_cast<double>(__float_as_int(v)) : static_cast<double>(v);
      }
      store_sum(tid, N, s, a.counts, a.sums);
    }
    cluster.sync();  // the others' memory stays until it is read
  }
}

// The sums over the stats CTAs, 8 columns (32 bytes of a row) per CTA.
__global__ void __launch_bounds__(kThreads) finish_kernel(const float* part, int ctas, int N, int32_t* counts, float* sums) {
  __shared__ double acc[kThreads / 32][8];
  pdl_wait();
  pdl_launch_dependents();
  const int cols = 2 * N + 2, col = blockIdx.x * 8 + threadIdx.x % 8;
  const bool whole = col < N || col == 2 * N + 1;
  // A thread's few dozen parts in 32 bits, the threads' sums in 64 (a
  // conversion per part had cost more than the rest of the kernel).
  double s = 0.0;
  if (col < cols && whole) {
    int c = 0;
#pragma unroll 8
    for (int i = threadIdx.x / 8; i < ctas; i += kThreads / 8) c += __float_as_int(part[static_cast<size_t>(i) * cols + col]);
    s = c;
  } else if (col < cols) {
    float f = 0.0f;
#pragma unroll 8
    for (int i = threadIdx.x / 8; i < ctas; i += kThreads / 8) f += part[static_cast<size_t>(i) * cols + col];
    s = f;
  }
  s += __shfl_xor_sync(0xffffffffu, s, 8);
  s += __shfl_xor_sync(0xffffffffu, s, 16);
  if (threadIdx.x % 32 < 8) acc[threadIdx.x / 32][threadIdx.x % 8] = s;
  __syncthreads();
  if (threadIdx.x >= 8 || col >= cols) return;
  for (int i = 1; i < kThreads / 32; ++i) s += acc[i][threadIdx.x];
  store_sum(col, N, s, counts, sums);
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

template <int LANES, int PER, bool EXACT>
__global__ void __launch_bounds__(kThreads, PER <= 4 ? 4 : 3) grad_kernel(GradArgs a) {
  constexpr int kAhead = PER <= 4 ? kAheadFew : kAheadMany;
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
      // A factor of 0 leaves its term out, an infinite one too.
      a.loss[0] = static_cast<float>(a.c_balance * bal + (a.c_z != 0.0f ? a.c_z * zl : 0.0));
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
    const int j = expert_of<LANES, PER, EXACT>(q, i);
    f[i] = in && j < a.M ? static_cast<float>((static_cast<double>(a.counts[g * a.M + j]) * a.M - a.k * n) / (a.M * a.k * n))
                         : 0.0f;
  }
  const float cb = static_cast<float>(static_cast<double>(a.c_balance) * a.M / (a.G * n));
  const float cz = static_cast<float>(2.0 * a.c_z / (a.G * n));
  const long long step = static_cast<long long>(gridDim.x) * rows;
  const long long zs = step * a.G * a.M;
  long long r = static_cast<long long>(blockIdx.x) * rows + rl, at0 = (r * a.G + g) * a.M;
  for (long long r0 = r - rl; r0 < a.R; r0 += kAhead * step, r += kAhead * step, at0 += kAhead * zs) {
    float z[kAhead][PER];
    bool at[kAhead], live[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      at[u] = live[u] = in && r + u * step < a.R;
      load_logits<LANES, PER, EXACT>(a.z + at0 + u * zs, q, a.M, at[u], z[u]);
    }
    if (a.mask != nullptr) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) live[u] = at[u] && a.mask[r + u * step] != 0;
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      float inv, lse, mean = 0.0f;
      softmax<LANES, PER>(z[u], &inv, &lse);
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        z[u][i] *= inv;
        mean = fmaf(z[u][i], f[i], mean);
      }
#pragma unroll
      for (int o = LANES / 2; o > 0; o >>= 1) mean += __shfl_xor_sync(0xffffffffu, mean, o);
#pragma unroll
      for (int i = 0; i < PER; ++i) z[u][i] = live[u] ? z[u][i] * (cb * (f[i] - mean) + cz * lse) : 0.0f;
      if (!at[u]) continue;
      float* out = a.dz + at0 + u * zs;
      if constexpr (EXACT && PER % 4 == 0) {
#pragma unroll
        for (int i = 0; i < PER; i += 4) {
          const int j = expert_of<LANES, PER, EXACT>(q, i);
          if (LANES > 1 && j >= a.M) continue;
          float4* o = reinterpret_cast<float4*>(out + j);
          float4 v = make_float4(z[u][i], z[u][i + 1], z[u][i + 2], z[u][i + 3]);
          if (a.accumulate) {
            const float4 w = *o;
            v = make_float4(w.x + v.x, w.y + v.y, w.z + v.z, w.w + v.w);
          }
          *o = v;
        }
      } else if constexpr (EXACT && PER == 2) {
        float2* o = reinterpret_cast<float2*>(out);
        float2 v = make_float2(z[u][0], z[u][1]);
        if (a.accumulate) {
          const float2 w = *o;
          v = make_float2(w.x + v.x, w.y + v.y);
        }
        *o = v;
      } else {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          const int j = q + i * LANES;
          if (j < a.M) out[j] = a.accumulate ? out[j] + z[u][i] : z[u][i];
        }
      }
    }
  }
}

// Instantiation for M: up to 8 logits in one lane (1, 2, 4 and 8 in one
// piece), more on 8 lanes (multiples of 4 above 16 in pieces of four).
template <int L, int P, bool E>
struct Shape {
  static constexpr int LANES = L, PER = P;
  static constexpr bool EXACT = E;
};
template <typename F>
int with_shape(int M, F f) {
  if (M == 1) return f(Shape<1, 1, true>{});
  if (M == 2) return f(Shape<1, 2, true>{});
  if (M == 4) return f(Shape<1, 4, true>{});
  if (M == 8) return f(Shape<1, 8, true>{});
  if (M < 4) return f(Shape<1, 4, false>{});
  if (M < 8) return f(Shape<1, 8, false>{});
  if (M <= 16) return f(Shape<8, 2, false>{});
  if (M <= 32) return M % 4 == 0 ? f(Shape<8, 4, true>{}) : f(Shape<8, 4, false>{});
  return M % 4 == 0 ? f(Shape<8, 8, true>{}) : f(Shape<8, 8, false>{});
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
  const BalanceArgs a{z, idx, mask, R, G, M, k, static_cast<float*>(ws), counts, sums};
  const int ctas = ctas_for(R, G, M), rows = balance_impl::kThreads / (G * (M <= 8 ? 1 : 8));
  // Few rows, at most ten per thread: one cluster, no second
  // launch (2048 rows of 8 x 2 logits, both calls: 12.9 us against 14.3).
  if (R <= static_cast<long long>(kCluster) * rows * 10)
    return with_shape(M, [&](auto s) {
      using S = decltype(s);
      cudaLaunchAttribute attr[2];
      attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
      attr[0].val.programmaticStreamSerializationAllowed = 1;
      attr[1].id = cudaLaunchAttributeClusterDimension;
      attr[1].val.clusterDim = {kCluster, 1, 1};
      cudaLaunchConfig_t cfg{};
      cfg.gridDim = dim3(kCluster);
      cfg.blockDim = dim3(balance_impl::kThreads);
      cfg.stream = static_cast<cudaStream_t>(stream);
      cfg.attrs = attr;
      cfg.numAttrs = 2;
      return static_cast<int>(cudaLaunchKernelEx(&cfg, stats_kernel<S::LANES, S::PER, S::EXACT, true>, a));
    });
  const int e = with_shape(M, [&](auto s) {
    using S = decltype(s);
    return static_cast<int>(launch_pdl(stats_kernel<S::LANES, S::PER, S::EXACT, false>, dim3(ctas),
                                       dim3(balance_impl::kThreads), 0, stream, a));
  });
  if (e != cudaSuccess) return e;
  return launch_pdl(finish_kernel, dim3((2 * G * M + 2 + 7) / 8), dim3(balance_impl::kThreads), 0, stream,
                    static_cast<const float*>(a.part), ctas, G * M, counts, sums);
}

int balance_grad(const float* z, const uint8_t* mask, const int32_t* counts, const float* sums, long long R, int G,
                 int M, int k, float c_balance, float c_z, float* loss, float* dz, bool accumulate, void* stream) {
  const GradArgs a{z, mask, counts, sums, R, G, M, k, c_balance, c_z, loss, dz, accumulate ? 1 : 0};
  const int ctas = dz != nullptr ? ctas_for(R, G, M) : 1;
  return with_shape(M, [&](auto s) {
    using S = decltype(s);
    return static_cast<int>(launch_pdl(grad_kernel<S::LANES, S::PER, S::EXACT>, dim3(ctas),
                                       dim3(balance_impl::kThreads), 0, stream, a));
  });
}

}  // namespace gqe
