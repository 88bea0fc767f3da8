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
// neighbouring tokens: a warp reads whole 64-byte segments of a head. Several
// heads' loads are in flight per thread. The norm's weights are multiplied
// into cos and sin once per token.
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
struct Lane {
  int c0, c1;
  bool rot, adjacent;
  __device__ __forceinline__ int pair(int j) const { return adjacent ? 2 * (j < 2 ? c0 : c1) + (j & 1) : 4 * c0 + j; }
  __device__ __forceinline__ int elem_a(int j) const { return adjacent ? 4 * (j < 2 ? c0 : c1) + 2 * (j & 1) : 4 * c0 + j; }
  __device__ __forceinline__ int elem_b(int j) const { return adjacent ? elem_a(j) + 1 : 4 * c1 + j; }
};

__device__ __forceinline__ Lane lane_of(int l, const RopeArgs& a) {
  const int nr = a.d_rot / 8;
  Lane r;
  r.rot = l < nr;
  r.adjacent = a.adjacent != 0;
  r.c0 = r.rot ? l : 2 * l;
  r.c1 = r.rot ? l + nr : 2 * l + 1;
  return r;
}

// The lane's angles; `on`: the token exists (else no rotation: its zeros stay zeros).
__device__ __forceinline__ void angles(const RopeArgs& a, const Lane& ln, bool on, long long row, int b, int t,
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

// Offset of a row of operand op (head h), or -1: in token-list order
// (slot_pos from the dispatch) a list entry that does not exist (recorded).
__device__ __forceinline__ long long row_offset(const RopeArgs& a, const RopeRows& r, int op, long long row, int b, int t,
                                                int h, int dh) {
  if (op != 0 || a.slot_pos == nullptr) return b * r.sb + h * r.sh + t * r.st;
  const int32_t e = a.slot_pos[row * a.n[0] + h];
  if (e < 0 || e >= a.R * a.n[0]) {
    set_status(GQE_ERR_DEVICE_CHECK);
    return -1;
  }
  return static_cast<long long>(e) * dh;
}

// One operand's heads [h0, h1) of this lane group's token, U rows in flight.
template <int DH, int U>
__device__ __forceinline__ void rope_rows_fwd(const RopeArgs& a, const Lane& ln, int op, int h0, int h1, bool on,
                                              long long row, int b, int t, const float (&ca)[4], const float (&sb)[4],
                                              const float (&sa)[4], const float (&cb)[4]) {
  constexpr int LPT = DH / 8;
  for (int h = h0; h < h1; h += U) {
    uint2 r0[U], r1[U];
    long long off[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      off[u] = on ? row_offset(a, a.x[op], op, row, b, t, h + u, DH) : -1;
      r0[u] = r1[u] = make_uint2(0u, 0u);
      if (off[u] >= 0) {
        const uint16_t* p = static_cast<const uint16_t*>(a.x[op].p) + off[u];
        r0[u] = *reinterpret_cast<const uint2*>(p + 4 * ln.c0);
        r1[u] = *reinterpret_cast<const uint2*>(p + 4 * ln.c1);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float A[4], B[4];
      unpack(r0[u], r1[u], ln.adjacent, A, B);
      if (a.norm) {
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
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float x = A[j], y = B[j];
        // Elements that are not rotated do not meet their neighbour (0 * inf).
        A[j] = ln.rot ? fmaf(x, ca[j], -y * sb[j]) : x * ca[j];
        B[j] = ln.rot ? fmaf(x, sa[j], y * cb[j]) : y * cb[j];
      }
      if (off[u] < 0) continue;
      pack(A, B, ln.adjacent, &r0[u], &r1[u]);
      // In token-list order inputs and outputs share their offsets.
      const long long o = op == 0 && a.slot_pos != nullptr ? off[u] : row_offset(a, a.y[op], 1, row, b, t, h + u, DH);
      uint16_t* q = static_cast<uint16_t*>(a.y[op].p) + o;
      *reinterpret_cast<uint2*>(q + 4 * ln.c0) = r0[u];
      *reinterpret_cast<uint2*>(q + 4 * ln.c1) = r1[u];
    }
  }
}

template <int DH>
__global__ void __launch_bounds__(kThreads) rope_kernel(RopeArgs a) {
  constexpr int LPT = DH / 8, TOK = kThreads / LPT, U = 4;
  pdl_wait();
  pdl_launch_dependents();
  const long long row = static_cast<long long>(blockIdx.x) * TOK + threadIdx.x / LPT;
  const bool on = row < a.R;
  const int b = on ? static_cast<int>(row / a.T) : 0, t = on ? static_cast<int>(row - static_cast<long long>(b) * a.T) : 0;
  const Lane ln = lane_of(threadIdx.x % LPT, a);
  float cs[4], sn[4];
  angles(a, ln, on, row, b, t, cs, sn);
  const int first = blockIdx.y * a.hpc, last = first + a.hpc;  // this CTA's heads of all operands
  int at = 0;
#pragma unroll 1
  for (int op = 0; op < 3; ++op) {
    const int h0 = max(first - at, 0), h1 = min(last - at, a.n[op]);
    at += a.n[op];
    if (h0 >= h1) continue;
    const float* w = a.norm ? (op == 2 ? a.w_k : a.w_q) : nullptr;
    float ca[4], sb[4], sa[4], cb[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float wa = w != nullptr ? __ldg(w + ln.elem_a(j)) : 1.0f, wb = w != nullptr ? __ldg(w + ln.elem_b(j)) : 1.0f;
      ca[j] = cs[j] * wa;
      sb[j] = sn[j] * wb;
      sa[j] = sn[j] * wa;
      cb[j] = cs[j] * wb;
    }
    const int mid = h0 + (h1 - h0) / U * U;
    rope_rows_fwd<DH, U>(a, ln, op, h0, mid, on, row, b, t, ca, sb, sa, cb);
    rope_rows_fwd<DH, 1>(a, ln, op, mid, h1, on, row, b, t, ca, sb, sa, cb);
  }
}

// The next row's operands of the backward, loaded while one is worked on.
struct BwdRow {
  float4 g0, g1;
  uint2 x0, x1;
  long long off;
};

// Sum of a gradient row's parts (see RopeGrad), this lane's 8 elements.
__device__ __forceinline__ void load_parts(const RopeGrad& g, const float* base, int hh, const Lane& ln, float4* x,
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

// PARTS: the gradients come in parts (the layer's backward).
template <int DH, bool PARTS>
__global__ void __launch_bounds__(kThreads) rope_bwd_kernel(RopeArgs a, RopeBwdArgs d) {
  constexpr int LPT = DH / 8, TOK = kThreads / LPT;
  __shared__ float red[kThreads / 32][2][DH];
  const Lane ln = lane_of(threadIdx.x % LPT, a);
  const int H = a.n[0] + a.n[1] + a.n[2];
  const long long tiles = (a.R + TOK - 1) / TOK;
  const int chunks = (H + a.hpc - 1) / a.hpc;
  float dwa[2][4], dwb[2][4];  // queries', keys' weight gradients
#pragma unroll
  for (int i = 0; i < 8; ++i) dwa[i / 4][i % 4] = dwb[i / 4][i % 4] = 0.0f;
  for (long long it = blockIdx.x; it < tiles * chunks; it += gridDim.x) {
    const long long tile = it / chunks;
    const int first = static_cast<int>(it - tile * chunks) * a.hpc, last = first + a.hpc;
    const long long row = tile * TOK + threadIdx.x / LPT;
    const bool on = row < a.R;
    const int b = on ? static_cast<int>(row / a.T) : 0,
              t = on ? static_cast<int>(row - static_cast<long long>(b) * a.T) : 0;
    float cs[4], sn[4];
    angles(a, ln, on, row, b, t, cs, sn);
    int at = 0;
#pragma unroll
    for (int op = 0; op < 3; ++op) {
      constexpr int kQueries = 0, kKeys = 1;
      const int wi = op == 2 ? kKeys : kQueries;
      const int h0 = max(first - at, 0), h1 = min(last - at, a.n[op]);
      at += a.n[op];
      if (h0 >= h1) continue;
      const float* w = a.norm ? (op == 2 ? a.w_k : a.w_q) : nullptr;
      float wa[4], wb[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        wa[j] = w != nullptr ? __ldg(w + ln.elem_a(j)) : 1.0f;
        wb[j] = w != nullptr ? __ldg(w + ln.elem_b(j)) : 1.0f;
      }
      auto load = [&](int h, BwdRow* r) {
        r->off = on ? row_offset(a, a.x[op], op, row, b, t, h, DH) : -1;
        r->g0 = r->g1 = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        r->x0 = r->x1 = make_uint2(0u, 0u);
        if (r->off < 0) return;
        const bool list = op == 0 && a.slot_pos != nullptr;
        const float* g = static_cast<const float*>(d.g[op].rows.p) + (list ? r->off : row_offset(a, d.g[op].rows, 1, row, b, t, h, DH));
        if constexpr (PARTS) {
          load_parts(d.g[op], g, h, ln, &r->g0, &r->g1);
        } else {
          r->g0 = *reinterpret_cast<const float4*>(g + 4 * ln.c0);
          r->g1 = *reinterpret_cast<const float4*>(g + 4 * ln.c1);
        }
        if (a.norm) {
          const uint16_t* p = static_cast<const uint16_t*>(a.x[op].p) + r->off;
          r->x0 = *reinterpret_cast<const uint2*>(p + 4 * ln.c0);
          r->x1 = *reinterpret_cast<const uint2*>(p + 4 * ln.c1);
        }
      };
      BwdRow next;
      load(h0, &next);
      for (int h = h0; h < h1; ++h) {
        const BwdRow r = next;
        if (h + 1 < h1) load(h + 1, &next);
        float A[4], B[4];
        to_pairs(r.g0, r.g1, ln.adjacent, A, B);
        if (ln.rot) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float x = A[j], y = B[j];
            A[j] = fmaf(x, cs[j], y * sn[j]);
            B[j] = fmaf(y, cs[j], -x * sn[j]);
          }
        }
        if (a.norm) {
          float X[4], Y[4], s = 0.0f, gx = 0.0f;
          unpack(r.x0, r.x1, ln.adjacent, X, Y);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            s = fmaf(X[j], X[j], fmaf(Y[j], Y[j], s));
            gx = fmaf(A[j] * wa[j], X[j], fmaf(B[j] * wb[j], Y[j], gx));
          }
          s = lane_sum<LPT>(s);
          gx = lane_sum<LPT>(gx);
          // An absent row (zeros) adds nothing to the sums, eps = 0 included.
          const float rstd = r.off < 0 ? 0.0f : rsqrtf(fmaf(s, 1.0f / DH, a.eps));
          const float mean = gx * rstd * (1.0f / DH);  // of gw xh
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            X[j] *= rstd;
            Y[j] *= rstd;
            dwa[wi][j] = fmaf(A[j], X[j], dwa[wi][j]);  // 0 where the row is absent
            dwb[wi][j] = fmaf(B[j], Y[j], dwb[wi][j]);
            A[j] = rstd * fmaf(-X[j], mean, A[j] * wa[j]);
            B[j] = rstd * fmaf(-Y[j], mean, B[j] * wb[j]);
          }
        }
        if (r.off < 0) continue;
        const bool list = op == 0 && a.slot_pos != nullptr;
        float* q = static_cast<float*>(a.y[op].p) + (list ? r.off : row_offset(a, a.y[op], 1, row, b, t, h, DH));
        float4 o0, o1;
        from_pairs(A, B, ln.adjacent, &o0, &o1);
        *reinterpret_cast<float4*>(q + 4 * ln.c0) = o0;
        *reinterpret_cast<float4*>(q + 4 * ln.c1) = o1;
      }
    }
  }
  if (d.part == nullptr) return;
  // The weights' gradients: lanes of one column over the warp's tokens, then
  // the warps, in a fixed order; one partial row per CTA.
  const int warp = threadIdx.x / 32;
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
      for (int o = LPT; o < 32; o <<= 1) {
        dwa[i][j] += __shfl_xor_sync(0xffffffffu, dwa[i][j], o);
        dwb[i][j] += __shfl_xor_sync(0xffffffffu, dwb[i][j], o);
      }
      if (threadIdx.x % 32 < LPT) {
        red[warp][i][ln.elem_a(j)] = dwa[i][j];
        red[warp][i][ln.elem_b(j)] = dwb[i][j];
      }
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
  bool parts = false;
  for (int i = 0; i < 3; ++i) parts = parts || d.g[i].parts * d.g[i].streams != 1 || d.g[i].extra != 0;
  auto kernel = dh == 64 ? (parts ? rope_bwd_kernel<64, true> : rope_bwd_kernel<64, false>)
                         : (parts ? rope_bwd_kernel<32, true> : rope_bwd_kernel<32, false>);
  kernel<<<ctas, rope_impl::kThreads, 0, st>>>(a, d);
  if (dw && dh == 64) rope_dw_kernel<64><<<2 * 64 / 4, rope_impl::kThreads, 0, st>>>(d.part, ctas, dw_q, dw_k);
  if (dw && dh == 32) rope_dw_kernel<32><<<2 * 32 / 4, rope_impl::kThreads, 0, st>>>(d.part, ctas, dw_q, dw_k);
  return cudaGetLastError();
}

}  // namespace gqe
