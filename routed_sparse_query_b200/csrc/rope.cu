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
// same lane (no exchange but the norm's sums), and walk the token's heads, so
// that the angles -- the only expensive arithmetic, see turn() -- are formed
// once per token and not once per row. Neighbouring lane groups take
// neighbouring tokens: a warp reads whole 64-byte segments of a head. Bytes in
// flight come from four rows per thread in the forward, from many threads in
// the backward (64 registers; two or more rows per thread cost occupancy and
// were no faster, nor were rows ahead through shared memory). The norm's
// weights are multiplied into cos and sin once per token.
//
// Measured, 8 groups of d_head 64, share of the copy rate: forward of 4 x 8192
// tokens 29 us (142 MB, 76 %), of 262144 tokens 202 us (1.14 GB, 87 %; 181 us
// in a short run with one axis); backward of 4 x 8192 tokens and 25 heads
// 91 us (524 MB, 89 %). 64 tokens: 7 us, the launch. Backward of 2048 tokens
// (floor 3.4 us): 12 us, 10 of them on the device: a thread's rows one after the
// other, the first behind the angles, then the kernel of the weights' gradients.
// In the layer's backward (gradients in parts, the general form): 2048 tokens 19
// us cold; with the forward's rotation 21 of 362 us, at 4 x 8192 tokens of the
// pool 171 of 8470.
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
// then fits fp32 with an error of 2^-25 turns. What is left is within half a
// turn, where the hardware sine and cosine are within 2^-20.
__device__ __forceinline__ void turn(double t, float scale, float* c, float* s) {
  const float x = 6.28318530717958647692f * static_cast<float>(t - rint(t));
  *c = __cosf(x) * scale;
  *s = __sinf(x) * scale;
}

// Lane l of a token: rotated lanes (l < d_rot / 8) hold chunk l and the chunk
// d_rot / 2 elements further; the others the next two chunks in order. Its 8
// values are kept as pairs (A_j, B_j), j < 4: element j of the two chunks, or
// with adjacent pairs elements 2i and 2i + 1 of the chunks one after the other.
//
// USUAL: the norm, pairs half the head apart and every element rotated -- what
// most models do -- are known at compile time; else they are looked at for
// every row (256k tokens: 181 us against 230).
template <bool USUAL>
struct Lane {
  int c0, c1;
  bool rot, adjacent;
  __device__ __forceinline__ int pair(int j) const { return adjacent ? 2 * (j < 2 ? c0 : c1) + (j & 1) : 4 * c0 + j; }
  __device__ __forceinline__ int elem_a(int j) const { return adjacent ? 4 * (j < 2 ? c0 : c1) + 2 * (j & 1) : 4 * c0 + j; }
  __device__ __forceinline__ int elem_b(int j) const { return adjacent ? elem_a(j) + 1 : 4 * c1 + j; }
};

template <int DH, bool USUAL>
__device__ __forceinline__ Lane<USUAL> lane_of(int l, const RopeArgs& a) {
  const int nr = USUAL ? DH / 8 : a.d_rot / 8;
  Lane<USUAL> r;
  r.rot = USUAL || l < nr;
  r.adjacent = !USUAL && a.adjacent != 0;
  r.c0 = r.rot ? l : 2 * l;
  r.c1 = r.rot ? l + nr : 2 * l + 1;
  return r;
}

// The lane's angles; `on`: the token exists (else no rotation: its zeros stay zeros).
template <bool USUAL>
__device__ __forceinline__ void angles(const RopeArgs& a, const Lane<USUAL>& ln, bool on, long long row, int b, int t,
                                       float (&cs)[4], float (&sn)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    cs[j] = 1.0f;
    sn[j] = 0.0f;
  }
  if (!ln.rot || !on) return;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int pair = ln.pair(j);
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

// A row's raw words (A0 A1 | A2 A3 | B0 B1 | B2 B3 in chunk order) to pairs
// and back.
__device__ __forceinline__ void unpack(const uint2& r0, const uint2& r1, bool adjacent, float (&A)[4], float (&B)[4]) {
  uint32_t w[4] = {r0.x, r0.y, r1.x, r1.y};
  if (adjacent) {
    const uint32_t a0 = __byte_perm(w[0], w[1], 0x5410), a1 = __byte_perm(w[2], w[3], 0x5410),
                   b0 = __byte_perm(w[0], w[1], 0x7632), b1 = __byte_perm(w[2], w[3], 0x7632);
    w[0] = a0; w[1] = a1; w[2] = b0; w[3] = b1;
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    A[2 * i] = __uint_as_float(w[i] << 16);
    A[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    B[2 * i] = __uint_as_float(w[2 + i] << 16);
    B[2 * i + 1] = __uint_as_float(w[2 + i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void pack(const float (&A)[4], const float (&B)[4], bool adjacent, uint2* r0, uint2* r1) {
  uint32_t w[4] = {pack_bf16x2(A[0], A[1]), pack_bf16x2(A[2], A[3]), pack_bf16x2(B[0], B[1]), pack_bf16x2(B[2], B[3])};
  if (adjacent) {
    const uint32_t e0 = __byte_perm(w[0], w[2], 0x5410), e1 = __byte_perm(w[0], w[2], 0x7632),
                   e2 = __byte_perm(w[1], w[3], 0x5410), e3 = __byte_perm(w[1], w[3], 0x7632);
    w[0] = e0; w[1] = e1; w[2] = e2; w[3] = e3;
  }
  *r0 = make_uint2(w[0], w[1]);
  *r1 = make_uint2(w[2], w[3]);
}
// The same for fp32 chunks x, y.
__device__ __forceinline__ void to_pairs(const float4& x, const float4& y, bool adjacent, float (&A)[4], float (&B)[4]) {
  A[0] = x.x; B[3] = y.w;
  A[1] = adjacent ? x.z : x.y;
  A[2] = adjacent ? y.x : x.z;
  A[3] = adjacent ? y.z : x.w;
  B[0] = adjacent ? x.y : y.x;
  B[1] = adjacent ? x.w : y.y;
  B[2] = adjacent ? y.y : y.z;
}
__device__ __forceinline__ void from_pairs(const float (&A)[4], const float (&B)[4], bool adjacent, float4* x, float4* y) {
  *x = adjacent ? make_float4(A[0], B[0], A[1], B[1]) : make_float4(A[0], A[1], A[2], A[3]);
  *y = adjacent ? make_float4(A[2], B[2], A[3], B[3]) : make_float4(B[0], B[1], B[2], B[3]);
}

template <int LPT>
__device__ __forceinline__ float lane_sum(float v) {
#pragma unroll
  for (int o = LPT / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Token-list order (slot_pos from the dispatch): offset of the row of head h,
// or -1 for a list entry that does not exist (recorded).
__device__ __forceinline__ long long list_offset(const RopeArgs& a, long long row, int h, int dh) {
  const int32_t e = a.slot_pos[row * a.n[0] + h];
  if (e < 0 || e >= a.R * a.n[0]) {
    set_status(GQE_ERR_DEVICE_CHECK);
    return -1;
  }
  return static_cast<long long>(e) * dh;
}

// Coefficients of a lane's pairs for one operand: (x, y) -> (ca x - sb y, sa x + cb y).
struct Coef {
  float ca[4], sb[4], sa[4], cb[4];
};

// U rows of one lane group's token: inputs at p + u ps, outputs at q + u qs.
template <int DH, bool USUAL, int U>
__device__ __forceinline__ void rope_group(const RopeArgs& a, const Lane<USUAL>& ln, const Coef& c, bool live,
                                           const uint16_t* p, long long ps, uint16_t* q, long long qs) {
  constexpr int LPT = DH / 8;
  uint2 r0[U], r1[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    r0[u] = r1[u] = make_uint2(0u, 0u);
    if (live) {
      r0[u] = *reinterpret_cast<const uint2*>(p + u * ps + 4 * ln.c0);
      r1[u] = *reinterpret_cast<const uint2*>(p + u * ps + 4 * ln.c1);
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    float A[4], B[4];
    unpack(r0[u], r1[u], ln.adjacent, A, B);
    if (USUAL || a.norm) {
      float s = 0.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j) s = fmaf(A[j], A[j], fmaf(B[j], B[j], s));
      const float rstd = rsqrtf(fmaf(lane_sum<LPT>(s), 1.0f / DH, a.eps));
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        A[j] *= rstd;
        B[j] *= rstd;
      }
    }
    if (ln.rot) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float x = A[j], y = B[j];
        A[j] = fmaf(x, c.ca[j], -y * c.sb[j]);
        B[j] = fmaf(x, c.sa[j], y * c.cb[j]);
      }
    } else {  // elements that are not rotated do not meet their neighbour (0 * inf)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        A[j] *= c.ca[j];
        B[j] *= c.cb[j];
      }
    }
    if (!live) continue;
    pack(A, B, ln.adjacent, &r0[u], &r1[u]);
    *reinterpret_cast<uint2*>(q + u * qs + 4 * ln.c0) = r0[u];
    *reinterpret_cast<uint2*>(q + u * qs + 4 * ln.c1) = r1[u];
  }
}

template <int DH, bool USUAL>
__global__ void __launch_bounds__(kThreads, 4) rope_kernel(RopeArgs a) {
  constexpr int LPT = DH / 8, TOK = kThreads / LPT, U = 4;
  pdl_wait();
  pdl_launch_dependents();
  const long long row = static_cast<long long>(blockIdx.x) * TOK + threadIdx.x / LPT;
  const bool on = row < a.R;
  const int b = on ? static_cast<int>(row / a.T) : 0, t = on ? static_cast<int>(row - static_cast<long long>(b) * a.T) : 0;
  const Lane<USUAL> ln = lane_of<DH, USUAL>(threadIdx.x % LPT, a);
  float cs[4], sn[4];
  angles(a, ln, on, row, b, t, cs, sn);
  const int first = blockIdx.y * a.hpc, last = first + a.hpc;  // this CTA's heads of all operands
  int at = 0;
#pragma unroll 1
  for (int op = 0; op < 3; ++op) {
    const int h0 = max(first - at, 0), h1 = min(last - at, a.n[op]);
    at += a.n[op];
    if (h0 >= h1) continue;
    const float* w = USUAL || a.norm ? (op == 2 ? a.w_k : a.w_q) : nullptr;
    Coef c;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float wa = w != nullptr ? w[ln.elem_a(j)] : 1.0f, wb = w != nullptr ? w[ln.elem_b(j)] : 1.0f;
      c.ca[j] = cs[j] * wa;
      c.sb[j] = sn[j] * wb;
      c.sa[j] = sn[j] * wa;
      c.cb[j] = cs[j] * wb;
    }
    const uint16_t* p = static_cast<const uint16_t*>(a.x[op].p);
    uint16_t* q = static_cast<uint16_t*>(a.y[op].p);
    if (!USUAL && op == 0 && a.slot_pos != nullptr) {  // token-list order: inputs and outputs at the same rows
      for (int h = h0; h < h1; ++h) {
        const long long o = on ? list_offset(a, row, h, DH) : -1;
        rope_group<DH, USUAL, 1>(a, ln, c, o >= 0, p + o, 0, q + o, 0);
      }
      continue;
    }
    const long long ps = a.x[op].sh, qs = a.y[op].sh;
    p += b * a.x[op].sb + t * a.x[op].st + h0 * ps;
    q += b * a.y[op].sb + t * a.y[op].st + h0 * qs;
    int h = h0;
#pragma unroll 1
    for (; h + U <= h1; h += U, p += U * ps, q += U * qs) rope_group<DH, USUAL, U>(a, ln, c, on, p, ps, q, qs);
#pragma unroll 1
    for (; h < h1; ++h, p += ps, q += qs) rope_group<DH, USUAL, 1>(a, ln, c, on, p, 0, q, 0);
  }
}

// Sum of a gradient row's parts (see RopeGrad), this lane's 8 elements.
template <bool USUAL>
__device__ __forceinline__ void load_parts(const RopeGrad& g, const float* base, int hh, const Lane<USUAL>& ln, float4* x,
                                           float4* y) {
  *x = *y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  auto add = [&](const float* p) {
    const float4 u = *reinterpret_cast<const float4*>(p + 4 * ln.c0), v = *reinterpret_cast<const float4*>(p + 4 * ln.c1);
    x->x += u.x; x->y += u.y; x->z += u.z; x->w += u.w;
    y->x += v.x; y->y += v.y; y->z += v.z; y->w += v.w;
  };
  for (int f = 0; f < g.parts; ++f) {
    for (int s = 0; s < g.streams; ++s) add(base + f * g.part_stride + s * g.stream_stride);
    if (g.extra != 0 && hh == 0) add(base + f * g.part_stride + g.extra);
  }
}

// A lane's weights and its sums of their gradient.
struct Weights {
  float wa[4], wb[4], dwa[4], dwb[4];
};

// One row of a lane group's token backward: its gradient at g (PARTS: in
// parts, of head h), the forward's input at x, the output at y.
template <int DH, bool USUAL, bool PARTS>
__device__ __forceinline__ void rope_bwd_row(const RopeArgs& a, const RopeGrad& parts, const Lane<USUAL>& ln,
                                             const float (&cs)[4], const float (&sn)[4], Weights& w, bool live, int h,
                                             const float* g, const uint16_t* x, float* y) {
  constexpr int LPT = DH / 8;
  float4 g0 = make_float4(0.0f, 0.0f, 0.0f, 0.0f), g1 = g0;
  uint2 x0 = make_uint2(0u, 0u), x1 = x0;
  if (live) {
    if constexpr (PARTS) {
      load_parts(parts, g, h, ln, &g0, &g1);
    } else {
      g0 = *reinterpret_cast<const float4*>(g + 4 * ln.c0);
      g1 = *reinterpret_cast<const float4*>(g + 4 * ln.c1);
    }
    if (USUAL || a.norm) {
      x0 = *reinterpret_cast<const uint2*>(x + 4 * ln.c0);
      x1 = *reinterpret_cast<const uint2*>(x + 4 * ln.c1);
    }
  }
  float A[4], B[4];
  to_pairs(g0, g1, ln.adjacent, A, B);
  if (ln.rot) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float p = A[j], q = B[j];
      A[j] = fmaf(p, cs[j], q * sn[j]);
      B[j] = fmaf(q, cs[j], -p * sn[j]);
    }
  }
  if (USUAL || a.norm) {
    float X[4], Y[4], s = 0.0f, gx = 0.0f;
    unpack(x0, x1, ln.adjacent, X, Y);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      s = fmaf(X[j], X[j], fmaf(Y[j], Y[j], s));
      gx = fmaf(A[j] * w.wa[j], X[j], fmaf(B[j] * w.wb[j], Y[j], gx));
    }
    s = lane_sum<LPT>(s);
    gx = lane_sum<LPT>(gx);
    // An absent row (zeros) adds nothing to the sums, eps = 0 included.
    const float rstd = live ? rsqrtf(fmaf(s, 1.0f / DH, a.eps)) : 0.0f;
    const float mean = gx * rstd * (1.0f / DH);  // of gw xh
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      X[j] *= rstd;
      Y[j] *= rstd;
      w.dwa[j] = fmaf(A[j], X[j], w.dwa[j]);
      w.dwb[j] = fmaf(B[j], Y[j], w.dwb[j]);
      A[j] = rstd * fmaf(-X[j], mean, A[j] * w.wa[j]);
      B[j] = rstd * fmaf(-Y[j], mean, B[j] * w.wb[j]);
    }
  }
  if (!live) return;
  from_pairs(A, B, ln.adjacent, &g0, &g1);
  *reinterpret_cast<float4*>(y + 4 * ln.c0) = g0;
  *reinterpret_cast<float4*>(y + 4 * ln.c1) = g1;
}

// PARTS: the gradients come in parts (the layer's backward). CTAs below cq
// take the queries (routed and shared), the others the keys, so that a thread
// sums one weight gradient and keeps one set of weights.
template <int DH, bool USUAL, bool PARTS>
__global__ void __launch_bounds__(kThreads, kRopeBwdPerSm) rope_bwd_kernel(RopeArgs a, RopeBwdArgs d) {
  constexpr int LPT = DH / 8, TOK = kThreads / LPT;
  __shared__ float red[kThreads / 32][DH];
  const Lane<USUAL> ln = lane_of<DH, USUAL>(threadIdx.x % LPT, a);
  pdl_wait();
  pdl_launch_dependents();
  const bool keys = static_cast<int>(blockIdx.x) >= d.cq;
  const int ctas = keys ? gridDim.x - d.cq : d.cq, cta = keys ? blockIdx.x - d.cq : blockIdx.x;
  const int H = keys ? a.n[2] : a.n[0] + a.n[1], hpc = keys ? d.hpc_k : a.hpc, chunks = (H + hpc - 1) / hpc;
  const long long items = (a.R + TOK - 1) / TOK * chunks;
  const float* wp = USUAL || a.norm ? (keys ? a.w_k : a.w_q) : nullptr;
  Weights w;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    w.wa[j] = wp != nullptr ? wp[ln.elem_a(j)] : 1.0f;
    w.wb[j] = wp != nullptr ? wp[ln.elem_b(j)] : 1.0f;
    w.dwa[j] = w.dwb[j] = 0.0f;
  }
#pragma unroll 1
  for (long long it = cta; it < items; it += ctas) {
    const long long tile = it / chunks;
    const int first = static_cast<int>(it - tile * chunks) * hpc, last = min(first + hpc, H);
    const int row = static_cast<int>(tile * TOK) + threadIdx.x / LPT;
    const bool on = row < a.R;
    const int b = on ? row / a.T : 0, t = on ? row - b * a.T : 0;
    float cs[4], sn[4];
    angles(a, ln, on, row, b, t, cs, sn);
    // The queries' routed heads, then the shared one; or the keys.
#pragma unroll 1
    for (int op = keys ? 2 : 0; op < (keys ? 3 : 2); ++op) {
      const int at = op == 1 ? a.n[0] : 0, h0 = max(first - at, 0), h1 = min(last - at, a.n[op]);
      if (h0 >= h1) continue;
      const float* g = static_cast<const float*>(d.g[op].rows.p);
      const uint16_t* x = static_cast<const uint16_t*>(a.x[op].p);
      float* y = static_cast<float*>(a.y[op].p);
      if (!USUAL && op == 0 && a.slot_pos != nullptr) {  // token-list order: all three at the same rows
        for (int h = h0; h < h1; ++h) {
          const long long o = on ? list_offset(a, row, h, DH) : -1;
          rope_bwd_row<DH, USUAL, PARTS>(a, d.g[op], ln, cs, sn, w, o >= 0, h, g + o, x + o, y + o);
        }
        continue;
      }
      const long long gs = d.g[op].rows.sh, xs = a.x[op].sh, ys = a.y[op].sh;
      g += b * d.g[op].rows.sb + t * d.g[op].rows.st + h0 * gs;
      x += b * a.x[op].sb + t * a.x[op].st + h0 * xs;
      y += b * a.y[op].sb + t * a.y[op].st + h0 * ys;
#pragma unroll 1
      for (int h = h0; h < h1; ++h, g += gs, x += xs, y += ys)
        rope_bwd_row<DH, USUAL, PARTS>(a, d.g[op], ln, cs, sn, w, on, h, g, x, y);
    }
  }
  if (d.part == nullptr) return;
  // The weights' gradient: lanes of one column over the warp's tokens, then
  // the warps, in a fixed order; one partial row per CTA.
  const int warp = threadIdx.x / 32;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
#pragma unroll
    for (int o = LPT; o < 32; o <<= 1) {
      w.dwa[j] += __shfl_xor_sync(0xffffffffu, w.dwa[j], o);
      w.dwb[j] += __shfl_xor_sync(0xffffffffu, w.dwb[j], o);
    }
    if (threadIdx.x % 32 < LPT) {
      red[warp][ln.elem_a(j)] = w.dwa[j];
      red[warp][ln.elem_b(j)] = w.dwb[j];
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < DH; i += kThreads) {
    float s = 0.0f;
#pragma unroll
    for (int wi = 0; wi < kThreads / 32; ++wi) s += red[wi][i];
    d.part[static_cast<size_t>(blockIdx.x) * DH + i] = s;
  }
}

// dw[j] = sum over the CTAs' partials (rows below cq: the queries', then the
// keys'), one block per 4 columns, fixed order.
template <int DH>
__global__ void __launch_bounds__(kThreads) rope_dw_kernel(const float* part, int cq, int n, float* dw_q, float* dw_k) {
  __shared__ float4 red[kThreads];
  pdl_wait();
  pdl_launch_dependents();
  const bool keys = blockIdx.x >= DH / 4;
  const int col = 4 * (blockIdx.x % (DH / 4));
  float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int i = threadIdx.x + (keys ? cq : 0); i < (keys ? n : cq); i += kThreads) {
    const float4 v = *reinterpret_cast<const float4*>(part + static_cast<size_t>(i) * DH + col);
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
  float* dw = keys ? dw_k : dw_q;
  if (threadIdx.x < 4 && dw != nullptr) dw[col + threadIdx.x] = reinterpret_cast<const float*>(red)[threadIdx.x];
}

}  // namespace rope_impl
using namespace rope_impl;

// Heads one CTA walks: all of them where the token tiles alone make `ctas`
// CTAs (the angles are then formed once per token), fewer for short batches
// (forward with twice as many CTAs as are resident: 10.3 us against 9.7 at
// 10000 tokens, four times: 12.1).
static int heads_per_cta(long long tiles, int H, int ctas) {
  long long chunks = (ctas + tiles - 1) / tiles;
  chunks = chunks < 1 ? 1 : chunks > H ? H : chunks;
  return static_cast<int>((H + chunks - 1) / chunks);
}

static bool usual(const RopeArgs& a, int dh) { return a.norm && !a.adjacent && a.d_rot == dh && a.slot_pos == nullptr; }

int rope_fwd(RopeArgs a, int dh, void* stream) {
  const int tok = rope_impl::kThreads / (dh / 8), H = a.n[0] + a.n[1] + a.n[2];
  const long long tiles = (a.R + tok - 1) / tok;
  a.hpc = heads_per_cta(tiles, H, kRopeCtas);
  const dim3 grid(static_cast<unsigned>(tiles), static_cast<unsigned>((H + a.hpc - 1) / a.hpc));
  auto kernel = dh == 64 ? (usual(a, dh) ? rope_kernel<64, true> : rope_kernel<64, false>)
                         : (usual(a, dh) ? rope_kernel<32, true> : rope_kernel<32, false>);
  return launch_pdl(kernel, grid, dim3(rope_impl::kThreads), 0, stream, a);
}

size_t rope_bwd_ws_bytes(int dh) { return static_cast<size_t>(kRopeBwdCtas) * dh * sizeof(float); }

template <int DH>
static int launch_bwd(const RopeArgs& a, const RopeBwdArgs& d, int ctas, float* dw_q, float* dw_k, void* stream) {
  bool parts = false;
  for (int i = 0; i < 3; ++i) parts = parts || d.g[i].parts * d.g[i].streams != 1 || d.g[i].extra != 0;
  auto kernel = parts ? rope_bwd_kernel<DH, false, true>
                      : (usual(a, DH) ? rope_bwd_kernel<DH, true, false> : rope_bwd_kernel<DH, false, false>);
  int e = launch_pdl(kernel, dim3(ctas), dim3(rope_impl::kThreads), 0, stream, a, d);
  if (e == cudaSuccess && d.part != nullptr)
    e = launch_pdl(rope_dw_kernel<DH>, dim3(2 * DH / 4), dim3(rope_impl::kThreads), 0, stream,
                   static_cast<const float*>(d.part), d.cq, ctas, dw_q, dw_k);
  return e;
}

int rope_bwd(RopeArgs a, RopeBwdArgs d, int dh, float* dw_q, float* dw_k, void* ws, void* stream) {
  const int tok = rope_impl::kThreads / (dh / 8), Hq = a.n[0] + a.n[1], Hk = a.n[2];
  const long long tiles = (a.R + tok - 1) / tok;
  // Runs of heads of about one length in both classes; few tiles: one run per
  // resident CTA (2048 tokens of 17 heads: 10.3 us on the device against 11.3;
  // 10000 tokens: 25.5 against 23.6).
  const int hpc = heads_per_cta(tiles, Hq + Hk, 4 * tiles < kRopeBwdCtas ? kRopeBwdCtas : 2 * kRopeBwdCtas);
  const int nq = (Hq + hpc - 1) / hpc, nk = (Hk + hpc - 1) / hpc;
  a.hpc = nq > 0 ? (Hq + nq - 1) / nq : 1;
  d.hpc_k = nk > 0 ? (Hk + nk - 1) / nk : 1;
  const long long items = tiles * (nq + nk);
  const int ctas = static_cast<int>(items < kRopeBwdCtas ? items : kRopeBwdCtas);
  // Resident CTAs shared out by the classes' rows, at least one for each.
  int cq = (ctas * Hq + (Hq + Hk) / 2) / (Hq + Hk);
  if (Hq > 0 && cq == 0) cq = 1;
  if (Hk > 0 && cq == ctas) cq = ctas > 1 ? ctas - 1 : 0;
  d.cq = cq;
  d.part = a.norm && (dw_q != nullptr || dw_k != nullptr) ? static_cast<float*>(ws) : nullptr;
  return dh == 64 ? launch_bwd<64>(a, d, ctas, dw_q, dw_k, stream) : launch_bwd<32>(a, d, ctas, dw_q, dw_k, stream);
}

}  // namespace gqe
