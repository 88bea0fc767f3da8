// Query/key norm and position rotation (gqe_qk_rope) and its backward.
//
// One row x (d_head values of one head at one token):
//   xh = x * rsqrt(mean(x^2) + eps), n = w * xh      (norm; without it n = x)
//   (a, b) -> scale * (a cos - b sin, a sin + b cos) for each rotated pair of n,
//   angle = position[axis of the pair][token] * inv_freq[pair].
// Backward, g = dL/dy: gn = the transposed rotation of g, gw = w gn,
//   dx = rstd * (gw - xh * mean(gw xh)), dw = sum over rows of gn xh.
//
// Bound by HBM (2 + 2 bytes per element forward, 2 + 4 + 4 backward), so the
// split serves the loads: d_head / 8 lanes take one token, each with two
// 4-element chunks chosen so that both members of a rotated pair sit in the
// same lane (no exchange but the norm's sum), and walk the token's heads, so
// that the angles -- the only expensive arithmetic, see turn() -- are formed
// once per token and not once per row. Neighbouring lane groups take
// neighbouring tokens: a warp reads whole 64-byte segments of a head.
#include <cuda_runtime.h>
#include <cuda_bf16.h>

#include "gqe_internal.h"
#include "ptx.cuh"

namespace gqe {

namespace rope_impl {

constexpr int kThreads = 256;

// cos and sin of 2 pi t. The angle of a far position times a frequency needs
// more than fp32's 24 bits (position 1e6 leaves 0.06 rad of error), so the
// caller forms t (in turns) in fp64; its fractional part is exact there and
// then fits fp32 with an error of 2^-25 turns.
__device__ __forceinline__ void turn(double t, float scale, float* c, float* s) {
  float sn, cs;
  sincospif(2.0f * static_cast<float>(t - rint(t)), &sn, &cs);
  *c = cs * scale;
  *s = sn * scale;
}

struct Lane {
  int c0, c1;  // this lane's two chunks of 4 elements
  bool rot;
};

// Lane l of a token: rotated lanes (l < d_rot / 8) hold chunk l and the chunk
// d_rot / 2 elements further; the others the next two chunks in order.
__device__ __forceinline__ Lane lane_of(int l, int d_rot) {
  const int nr = d_rot / 8;
  Lane r;
  r.rot = l < nr;
  r.c0 = r.rot ? l : 2 * l;
  r.c1 = r.rot ? l + nr : 2 * l + 1;
  return r;
}

// The four angles of a lane. HALF pairs: element j of c0 with element j of
// c1, pair 4 c0 + j. Adjacent pairs: (2i, 2i+1) inside each chunk.
__device__ __forceinline__ void angles(const RopeArgs& a, const Lane& ln, long long row, int b, int t, float (&cs)[4],
                                       float (&sn)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    cs[j] = 1.0f;
    sn[j] = 0.0f;
  }
  if (!ln.rot) return;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int pair = a.adjacent ? 2 * (j < 2 ? ln.c0 : ln.c1) + (j & 1) : 4 * ln.c0 + j;
    int ax = a.axis != nullptr ? a.axis[pair] : 0;
    if (ax < 0 || ax >= a.axes) {
      set_status(GQE_ERR_DEVICE_CHECK);
      ax = 0;
    }
    const int p = a.pos != nullptr ? a.pos[static_cast<long long>(ax) * a.R + row]
                                   : t + a.pos0 + (a.pos_len != nullptr ? max(a.pos_len[b], 0) : 0);
    turn(static_cast<double>(p) * a.inv_freq[pair] * 0.15915494309189533577, a.scale, &cs[j], &sn[j]);
  }
}

__device__ __forceinline__ void unpack(uint2 v, float* f) {
  f[0] = __uint_as_float(v.x << 16);
  f[1] = __uint_as_float(v.x & 0xffff0000u);
  f[2] = __uint_as_float(v.y << 16);
  f[3] = __uint_as_float(v.y & 0xffff0000u);
}

// v[0..3] chunk c0, v[4..7] chunk c1; sgn = 1 rotates, -1 rotates back.
__device__ __forceinline__ void rotate(bool adjacent, const float (&cs)[4], const float (&sn)[4], float sgn,
                                       float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int ia = adjacent ? 2 * j : j, ib = adjacent ? 2 * j + 1 : j + 4;
    const float x = v[ia], y = v[ib], s = sgn * sn[j];
    v[ia] = x * cs[j] - y * s;
    v[ib] = x * s + y * cs[j];
  }
}

template <int LPT>
__device__ __forceinline__ float lane_sum(float v) {
#pragma unroll
  for (int o = LPT / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The operand (0: routed queries, 1: shared head, 2: keys) and the head
// inside it of the flat head index h.
__device__ __forceinline__ int operand_of(const RopeArgs& a, int h, int* hh) {
  if (h < a.n[0]) {
    *hh = h;
    return 0;
  }
  if (h < a.n[0] + a.n[1]) {
    *hh = 0;
    return 1;
  }
  *hh = h - a.n[0] - a.n[1];
  return 2;
}

__device__ __forceinline__ long long offset_of(const RopeRows& r, int b, int t, int h) {
  return b * r.sb + h * r.sh + t * r.st;
}
// Token-list order (slot_pos from the dispatch): the row's list entry, or -1
// (recorded) where it does not name one.
__device__ __forceinline__ long long list_offset(const RopeArgs& a, long long row, int h, int dh) {
  const int32_t e = a.slot_pos[row * a.n[0] + h];
  if (e < 0 || e >= a.R * a.n[0]) {
    set_status(GQE_ERR_DEVICE_CHECK);
    return -1;
  }
  return static_cast<long long>(e) * dh;
}

template <int DH>
__global__ void __launch_bounds__(kThreads) rope_kernel(RopeArgs a) {
  constexpr int LPT = DH / 8, TOK = kThreads / LPT;
  pdl_wait();
  pdl_launch_dependents();
  const int l = threadIdx.x % LPT;
  const long long row = static_cast<long long>(blockIdx.x) * TOK + threadIdx.x / LPT;
  const bool on = row < a.R;
  const int b = on ? static_cast<int>(row / a.T) : 0, t = on ? static_cast<int>(row - static_cast<long long>(b) * a.T) : 0;
  const Lane ln = lane_of(l, a.d_rot);
  float cs[4], sn[4];
  if (on) angles(a, ln, row, b, t, cs, sn);
  const int H = a.n[0] + a.n[1] + a.n[2];
  const int h1 = min(H, (static_cast<int>(blockIdx.y) + 1) * a.hpc);
  for (int h = blockIdx.y * a.hpc; h < h1; ++h) {
    int hh;
    const int op = operand_of(a, h, &hh);
    const float* w = op == 2 ? a.w_k : a.w_q;
    float v[8];
    uint2 r0 = make_uint2(0u, 0u), r1 = r0;
    const bool list = op == 0 && a.slot_pos != nullptr;
    const long long lo = list && on ? list_offset(a, row, hh, DH) : 0;
    const bool live = on && lo >= 0;
    if (live) {
      const uint16_t* p = static_cast<const uint16_t*>(a.x[op].p) + (list ? lo : offset_of(a.x[op], b, t, hh));
      r0 = *reinterpret_cast<const uint2*>(p + 4 * ln.c0);
      r1 = *reinterpret_cast<const uint2*>(p + 4 * ln.c1);
    }
    unpack(r0, v);
    unpack(r1, v + 4);
    if (a.norm) {
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) s = fmaf(v[i], v[i], s);
      const float rstd = rsqrtf(lane_sum<LPT>(s) * (1.0f / DH) + a.eps);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float wi = w != nullptr ? __ldg(w + 4 * (i < 4 ? ln.c0 : ln.c1) + (i & 3)) : 1.0f;
        v[i] = v[i] * rstd * wi;
      }
    }
    if (!live) continue;
    if (ln.rot) rotate(a.adjacent, cs, sn, 1.0f, v);
    uint16_t* q = static_cast<uint16_t*>(a.y[op].p) + (list ? lo : offset_of(a.y[op], b, t, hh));
    *reinterpret_cast<uint2*>(q + 4 * ln.c0) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
    *reinterpret_cast<uint2*>(q + 4 * ln.c1) = make_uint2(pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  }
}

// Sum of a gradient row's parts (see RopeGrad), this lane's 8 elements.
__device__ __forceinline__ void load_grad(const RopeGrad& g, long long off, int hh, const Lane& ln, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = 0.0f;
  const float* base = static_cast<const float*>(g.rows.p) + off;
  auto add = [&](const float* p) {
    const float4 x = *reinterpret_cast<const float4*>(p + 4 * ln.c0), y = *reinterpret_cast<const float4*>(p + 4 * ln.c1);
    v[0] += x.x; v[1] += x.y; v[2] += x.z; v[3] += x.w;
    v[4] += y.x; v[5] += y.y; v[6] += y.z; v[7] += y.w;
  };
  for (int f = 0; f < g.parts; ++f) {
    for (int s = 0; s < g.streams; ++s) add(base + f * g.part_stride + s * g.stream_stride);
    if (g.extra != 0 && hh == 0) add(base + f * g.part_stride + g.extra);
  }
}

template <int DH>
__global__ void __launch_bounds__(kThreads) rope_bwd_kernel(RopeArgs a, RopeBwdArgs d) {
  constexpr int LPT = DH / 8, TOK = kThreads / LPT;
  __shared__ float red[kThreads / 32][2][DH];
  const int l = threadIdx.x % LPT;
  const Lane ln = lane_of(l, a.d_rot);
  const int H = a.n[0] + a.n[1] + a.n[2];
  const long long tiles = (a.R + TOK - 1) / TOK;
  const int chunks = (H + a.hpc - 1) / a.hpc;
  float dwq[8], dwk[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) dwq[i] = dwk[i] = 0.0f;
  for (long long it = blockIdx.x; it < tiles * chunks; it += gridDim.x) {
    const long long tile = it / chunks;
    const int ch = static_cast<int>(it - tile * chunks);
    const long long row = tile * TOK + threadIdx.x / LPT;
    const bool on = row < a.R;
    const int b = on ? static_cast<int>(row / a.T) : 0,
              t = on ? static_cast<int>(row - static_cast<long long>(b) * a.T) : 0;
    float cs[4], sn[4];
    if (on) angles(a, ln, row, b, t, cs, sn);
    const int h1 = min(H, (ch + 1) * a.hpc);
    for (int h = ch * a.hpc; h < h1; ++h) {
      int hh;
      const int op = operand_of(a, h, &hh);
      const bool list = op == 0 && a.slot_pos != nullptr;
      const long long lo = list && on ? list_offset(a, row, hh, DH) : 0;
      const bool live = on && lo >= 0;
      const float* w = op == 2 ? a.w_k : a.w_q;
      float g[8], x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) g[i] = x[i] = 0.0f;
      if (live) {
        load_grad(d.g[op], list ? lo : offset_of(d.g[op].rows, b, t, hh), hh, ln, g);
        if (ln.rot) rotate(a.adjacent, cs, sn, -1.0f, g);
        if (a.norm) {
          const uint16_t* p = static_cast<const uint16_t*>(a.x[op].p) + (list ? lo : offset_of(a.x[op], b, t, hh));
          unpack(*reinterpret_cast<const uint2*>(p + 4 * ln.c0), x);
          unpack(*reinterpret_cast<const uint2*>(p + 4 * ln.c1), x + 4);
        }
      }
      if (a.norm) {
        float s = 0.0f, gx = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) s = fmaf(x[i], x[i], s);
        const float rstd = rsqrtf(lane_sum<LPT>(s) * (1.0f / DH) + a.eps);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          x[i] *= rstd;
          const float dw = live ? g[i] * x[i] : 0.0f;
          if (op == 2) dwk[i] += dw;
          else dwq[i] += dw;
          if (w != nullptr) g[i] *= __ldg(w + 4 * (i < 4 ? ln.c0 : ln.c1) + (i & 3));
          gx = fmaf(g[i], x[i], gx);
        }
        gx = lane_sum<LPT>(gx) * (1.0f / DH);
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] = rstd * (g[i] - x[i] * gx);
      }
      if (!live) continue;
      float* q = static_cast<float*>(a.y[op].p) + (list ? lo : offset_of(a.y[op], b, t, hh));
      *reinterpret_cast<float4*>(q + 4 * ln.c0) = make_float4(g[0], g[1], g[2], g[3]);
      *reinterpret_cast<float4*>(q + 4 * ln.c1) = make_float4(g[4], g[5], g[6], g[7]);
    }
  }
  if (d.part == nullptr) return;
  // The weights' gradients: lanes of one column over the warp's tokens, then
  // the warps, in a fixed order; one partial row per CTA.
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int o = LPT; o < 32; o <<= 1) {
      dwq[i] += __shfl_xor_sync(0xffffffffu, dwq[i], o);
      dwk[i] += __shfl_xor_sync(0xffffffffu, dwk[i], o);
    }
  const int warp = threadIdx.x / 32;
  if (threadIdx.x % 32 < LPT)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int col = 4 * (i < 4 ? ln.c0 : ln.c1) + (i & 3);
      red[warp][0][col] = dwq[i];
      red[warp][1][col] = dwk[i];
    }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * DH; i += kThreads) {
    float s = 0.0f;
#pragma unroll
    for (int wp = 0; wp < kThreads / 32; ++wp) s += red[wp][i / DH][i % DH];
    d.part[static_cast<size_t>(blockIdx.x) * 2 * DH + i] = s;
  }
}

// dw[j] = sum over the CTAs' partials, one block per 4 columns, fixed order.
template <int DH>
__global__ void __launch_bounds__(kThreads) rope_dw_kernel(const float* part, int n, float* dw_q, float* dw_k) {
  __shared__ float4 red[kThreads];
  float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const float4 v = *reinterpret_cast<const float4*>(part + static_cast<size_t>(i) * 2 * DH + 4 * blockIdx.x);
    s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
  }
  red[threadIdx.x] = s;
  __syncthreads();
  for (int o = kThreads / 2; o > 0; o >>= 1) {
    if (threadIdx.x < o) {
      const float4 v = red[threadIdx.x + o];
      red[threadIdx.x].x += v.x; red[threadIdx.x].y += v.y; red[threadIdx.x].z += v.z; red[threadIdx.x].w += v.w;
    }
    __syncthreads();
  }
  if (threadIdx.x < 4) {
    const int col = 4 * blockIdx.x + threadIdx.x;
    float* dw = col < DH ? dw_q : dw_k;
    if (dw != nullptr) dw[col % DH] = reinterpret_cast<const float*>(red)[threadIdx.x];
  }
}

}  // namespace rope_impl
using namespace rope_impl;

// Heads one CTA walks: all of them where the token tiles alone fill the SMs
// (the angles are then formed once per token), fewer for short batches.
static int heads_per_cta(long long tiles, int H) {
  long long chunks = (kRopeCtas + tiles - 1) / tiles;
  chunks = chunks < 1 ? 1 : chunks > H ? H : chunks;
  return static_cast<int>((H + chunks - 1) / chunks);
}

int rope_fwd(RopeArgs a, int dh, void* stream) {
  const int tok = rope_impl::kThreads / (dh / 8), H = a.n[0] + a.n[1] + a.n[2];
  const long long tiles = (a.R + tok - 1) / tok;
  a.hpc = heads_per_cta(tiles, H);
  const dim3 grid(static_cast<unsigned>(tiles), static_cast<unsigned>((H + a.hpc - 1) / a.hpc));
  return dh == 64 ? launch_pdl(rope_kernel<64>, grid, dim3(rope_impl::kThreads), 0, stream, a)
                  : launch_pdl(rope_kernel<32>, grid, dim3(rope_impl::kThreads), 0, stream, a);
}

size_t rope_bwd_ws_bytes(int dh) { return static_cast<size_t>(kRopeCtas) * 2 * dh * sizeof(float); }

int rope_bwd(RopeArgs a, RopeBwdArgs d, int dh, float* dw_q, float* dw_k, void* ws, void* stream) {
  const int tok = rope_impl::kThreads / (dh / 8), H = a.n[0] + a.n[1] + a.n[2];
  const long long tiles = (a.R + tok - 1) / tok;
  a.hpc = heads_per_cta(tiles, H);
  const long long items = tiles * ((H + a.hpc - 1) / a.hpc);
  const int ctas = static_cast<int>(items < kRopeCtas ? items : kRopeCtas);
  const bool dw = a.norm && (dw_q != nullptr || dw_k != nullptr);
  d.part = dw ? static_cast<float*>(ws) : nullptr;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dh == 64) rope_bwd_kernel<64><<<ctas, rope_impl::kThreads, 0, st>>>(a, d);
  else rope_bwd_kernel<32><<<ctas, rope_impl::kThreads, 0, st>>>(a, d);
  if (dw && dh == 64) rope_dw_kernel<64><<<2 * 64 / 4, rope_impl::kThreads, 0, st>>>(d.part, ctas, dw_q, dw_k);
  if (dw && dh == 32) rope_dw_kernel<32><<<2 * 32 / 4, rope_impl::kThreads, 0, st>>>(d.part, ctas, dw_q, dw_k);
  return cudaGetLastError();
}

}  // namespace gqe
