// Norms before and after a block, fused with the block's gate, the residual
// scale and (optionally) the weighted combine that closes a MoE layer.
//
// With N(v) = v / sqrt(mean_c v_c^2 + eps):
//   y   = the block's output, or sum_j w[t,j] Y[row_map[t,j]] (its k expert rows)
//   n   = N(y) w_post              (w_post NULL: n = y)
//   h1  = a h + rg[t] g[c] n       (row gate rg and channel gate g, each optional)
//   x   = N(h1) w_pre              (the next block's input)
// and the gradients, with D the whole gradient of h1:
//   z   = dx w_pre,  r = 1 / sqrt(mean h1^2 + eps)
//   D   = dh1 + r (z - h1 r^2 mean(z h1)),          dh = a D
//   q   = D rg g w_post,  ry = 1 / sqrt(mean y^2 + eps)
//   dy  = ry (q - y ry^2 mean(q y))
//   dw_pre[c] = sum_t dx h1 r,   S[c] = sum_t D rg y ry,
//   dw_post = g S,  dg = w_post S,  drg[t] = sum_c D g w_post y ry.
// Everything between the loads and the stores is float32 (h1 and y enter the
// norms unrounded); each output is rounded once.
//
// A row stays in registers from its load to its stores, so each tensor moves
// once; the backward needs no saved statistics, because the sums it takes
// anyway give them (sum h1^2, sum z h1 and sum y^2 come out of one reduction).
// The channel gradients are summed per thread over the rows a block walks
// (each thread owns fixed columns), written as one float32 row per block and
// added in block order by a second kernel: no atomics, the same bits each run.
//
// Both directions are bound by HBM (a large copy on the card: 4.9 TB/s), and the
// counters show each tensor moved once.  Measured at 16384 x 7168 bf16, both norms
// and a channel gate: forward 167 us = 5.6 TB/s, backward 296 us = 4.8 TB/s with
// the channel sums; with 4 expert rows combined, 8191 x 2880: 56 us = 5.9 TB/s; one
// row to a few: 5 us forward, 10 backward, a chain of loads and two reductions.
// What carried it: a row's loads issued while the row before is reduced (the
// forward's first form, a block a row, took 270 us), channel vectors in registers
// for all rows of a block, one chunk a lane where a row fits, the hardware's bf16
// conversion, and 8 to 16 waves per compute unit.
#include "common.hpp"
#include "spans.hpp"

#include <math.h>
#include <stddef.h>

#include <algorithm>
#include <type_traits>

namespace moe {

// A row belongs to LPR lanes of a wave (8, 16, 32 or all 64: rows of up to LPR NC
// chunks, several to a block), or (LPR 0) to a whole block of
// ceil(chunks / (64 NC)) waves.  A lane owns the 16-byte chunks lt, lt + tpr, ...
// of its row (NC of them; tpr lanes a row).
template <int LPR>
struct NormPlace {
  int tpr, lt, sub;      // lanes per row; lane within the row; row within the block
  __device__ __forceinline__ NormPlace()
      : tpr(LPR ? LPR : blockDim.x),
        lt(LPR ? threadIdx.x & (LPR - 1) : threadIdx.x),
        sub(LPR == 64  ? __builtin_amdgcn_readfirstlane(threadIdx.x >> 6)
            : LPR > 0 ? threadIdx.x / (LPR > 0 ? LPR : 1)
                      : 0) {}
};

// Sums of NV <= 4 values over a row's lanes, on every lane.  A wave's
// butterfly, then one over the row's waves through LDS.  `half` alternates
// between two halves: a thread writes one half again only after the barrier
// of the other, which every thread reaches after reading the first.
template <int NV, int LPR>
__device__ __forceinline__ void row_sums(float (&v)[NV], f32x4 (*lds)[16], int half) {
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int o = (LPR ? LPR : 64) / 2; o >= 1; o >>= 1) v[i] += __shfl_xor(v[i], o, 64);
  if constexpr (LPR == 0) {
    f32x4* b = lds[half];
    if ((threadIdx.x & 63) == 0) {
      f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < NV; ++i) o[i] = v[i];
      b[threadIdx.x >> 6] = o;
    }
    __syncthreads();
    // each group of 16 lanes adds the waves' sums in a butterfly
    const int w = threadIdx.x & 15;
    f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
    if (w < (int)(blockDim.x >> 6)) o = b[w];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      v[i] = o[i];
#pragma unroll
      for (int m = 8; m >= 1; m >>= 1) v[i] += __shfl_xor(v[i], m, 16);
    }
  }
}

// pack_chunk with the hardware's conversion (round to nearest even, two values
// an instruction): the bit arithmetic of f32_to_bf16_bits costs about seven,
// which these kernels, at 25 to 40 operations per element, would feel.
__device__ __forceinline__ u32x4 store_chunk(const float* v, BF16) {
  typedef float f32x8 __attribute__((ext_vector_type(8)));
  f32x8 f;
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = v[i];
  return __builtin_bit_cast(u32x4, __builtin_convertvector(f, bf16x8));
}
__device__ __forceinline__ u32x4 store_chunk(const float* v, F32) { return pack_chunk(v, F32()); }

// V consecutive floats of a per-channel vector (NULL: `fill`).
template <int V>
__device__ __forceinline__ void load_chan(const float* p, size_t c, float* v, float fill) {
#pragma unroll
  for (int i = 0; i < V; i += 4) {
    if (p) {
      const f32x4 w = *reinterpret_cast<const f32x4*>(p + c * V + i);
#pragma unroll
      for (int q = 0; q < 4; ++q) v[i + q] = w[q];
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q) v[i + q] = fill;
    }
  }
}

struct NormFwd {
  const u32x4 *h, *y;
  const float *w_post, *gate, *row_gate, *w_pre;
  const int32_t* row_map;
  const float* topk_w;
  u32x4 *h_out, *x_out, *y_out;
  int T, k, R, chunks;
  float res_scale, eps, inv_d;
  int stream;               // whether the outputs go past the L2
};

template <bool STREAM>
__device__ __forceinline__ void put_chunk(u32x4* p, const u32x4& v) {
  if constexpr (STREAM) __builtin_nontemporal_store(v, p);
  else *p = v;
}

// y[t]'s chunk c from its expert rows, up to four rows' loads in flight (their
// ids come in one scalar load: one by one they cost 1.5 times the whole kernel).
// The rows are read once: the nontemporal hint saves 10 %.
template <class EL>
__device__ __forceinline__ void combine_chunk(const NormFwd& p, int t, int c, float* y) {
  constexpr int V = EL::VEC;
  const int32_t* ids = p.row_map + (size_t)t * p.k;
  const float* ws = p.topk_w ? p.topk_w + (size_t)t * p.k : nullptr;
#pragma unroll
  for (int q = 0; q < V; ++q) y[q] = 0.0f;
  auto add = [&](auto N, int j0) {
    constexpr int n = decltype(N)::value;
    u32x4 raw[n];
#pragma unroll
    for (int j = 0; j < n; ++j) {
      int r = ids[j0 + j];
      r = (r < 0 || r >= p.R) ? 0 : r;
      raw[j] = __builtin_nontemporal_load(p.y + (size_t)r * p.chunks + c);
    }
#pragma unroll
    for (int j = 0; j < n; ++j) {
      const float w = ws ? ws[j0 + j] : 1.0f;
      float v[V];
      unpack_chunk(raw[j], v, EL());
#pragma unroll
      for (int q = 0; q < V; ++q) y[q] = fmaf(w, v[q], y[q]);
    }
  };
  int j = 0;
  for (; j + 4 <= p.k; j += 4) add(std::integral_constant<int, 4>(), j);
  const int left = p.k - j;
  if (left == 3) add(std::integral_constant<int, 3>(), j);
  else if (left == 2) add(std::integral_constant<int, 2>(), j);
  else if (left == 1) add(std::integral_constant<int, 1>(), j);
}

// Blocks walk the rows; a row's loads are issued while the one before it is
// reduced (not with 32 elements a thread, which would spill: 2048 x 32768 bf16 161 us,
// 247 ahead), and the channel vectors stay in registers throughout.  STREAM: h1 and
// x are stored nontemporally, where they are larger than the L2 anyway (16384 x
// 2880: 63 us against 71; the backward gains nothing from it).
template <class EL, int NC, int LPR, bool POST, bool PRE, bool COMB, bool STREAM>
__global__ void __launch_bounds__(LPR ? 256 : 1024) block_norm_fwd_kernel(const NormFwd p) {
  constexpr int V = EL::VEC;
  constexpr bool LOADY = POST && !COMB, AHEAD = NC * V <= 16;
  __shared__ f32x4 lds[2][16];
  const NormPlace<LPR> pl;
  const int lt = pl.lt, TPR = pl.tpr, rpb = LPR ? blockDim.x / (LPR ? LPR : 1) : 1;
  int t = blockIdx.x * rpb + pl.sub;
  const int step = gridDim.x * rpb;
  bool in[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) in[i] = lt + i * TPR < p.chunks;
  u32x4 hr[NC], yr[NC];
  const u32x4 zero = {0, 0, 0, 0};
  auto fetch = [&](int row) {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const size_t o = (size_t)row * p.chunks + lt + i * TPR;
      hr[i] = in[i] && row < p.T ? p.h[o] : zero;
      if constexpr (LOADY) yr[i] = in[i] && row < p.T ? p.y[o] : zero;
    }
  };
  if constexpr (AHEAD) fetch(t);
  float wg[NC][V], wp[NC][V];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
#pragma unroll
    for (int q = 0; q < V; ++q) wg[i][q] = wp[i][q] = 0.0f;
    if (in[i]) {
      const int c = lt + i * TPR;
      if constexpr (POST) {
        float g[V];
        load_chan<V>(p.w_post, c, wg[i], 1.0f);
        load_chan<V>(p.gate, c, g, 1.0f);
#pragma unroll
        for (int q = 0; q < V; ++q) wg[i][q] *= g[q];
      }
      if constexpr (PRE) load_chan<V>(p.w_pre, c, wp[i], 1.0f);
    }
  }
  for (; t < p.T; t += step) {
    const size_t row = (size_t)t * p.chunks + lt;
    float h[NC][V], y[NC][V];
    if constexpr (!AHEAD) fetch(t);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      unpack_chunk(hr[i], h[i], EL());
      if constexpr (LOADY) unpack_chunk(yr[i], y[i], EL());
    }
    if constexpr (AHEAD) fetch(t + step);
    if constexpr (POST) {
      float s[1] = {0.0f};
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        if constexpr (COMB) {
          if (in[i]) {
            combine_chunk<EL>(p, t, lt + i * TPR, y[i]);
            if (p.y_out) p.y_out[row + i * TPR] = store_chunk(y[i], EL());
          } else {
#pragma unroll
            for (int q = 0; q < V; ++q) y[i][q] = 0.0f;
          }
        }
#pragma unroll
        for (int q = 0; q < V; ++q) s[0] = fmaf(y[i][q], y[i][q], s[0]);
      }
      float f = p.row_gate ? p.row_gate[t] : 1.0f;
      if (p.w_post) {
        row_sums<1, LPR>(s, lds, 0);
        f *= 1.0f / sqrtf(s[0] * p.inv_d + p.eps);
      }
#pragma unroll
      for (int i = 0; i < NC; ++i) {
#pragma unroll
        for (int q = 0; q < V; ++q) h[i][q] = fmaf(p.res_scale, h[i][q], y[i][q] * (f * wg[i][q]));
        if (in[i]) put_chunk<STREAM>(p.h_out + row + i * TPR, store_chunk(h[i], EL()));
      }
    }
    if constexpr (PRE) {
      float s[1] = {0.0f};
#pragma unroll
      for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int q = 0; q < V; ++q) s[0] = fmaf(h[i][q], h[i][q], s[0]);
      row_sums<1, LPR>(s, lds, 1);
      const float r = 1.0f / sqrtf(s[0] * p.inv_d + p.eps);
#pragma unroll
      for (int i = 0; i < NC; ++i) {
#pragma unroll
        for (int q = 0; q < V; ++q) h[i][q] *= r * wp[i][q];
        if (in[i]) put_chunk<STREAM>(p.x_out + row + i * TPR, store_chunk(h[i], EL()));
      }
    }
    // a row with only one of the two reductions meets the same LDS half again
    // in the next step
    if (LPR == 0 && !(PRE && POST && p.w_post)) __syncthreads();
  }
}

// Threads of a block of the backward.
constexpr int norm_bwd_threads(int nc, int lpr, int waves) {
  return lpr == 0 ? 64 * waves : lpr == 64 ? (nc == 1 ? 1024 : 512) : 256;
}

// Keeps the compiler from holding a chunk's floats across a reduction, where its
// 16 bytes are enough and registers are short.
__device__ __forceinline__ void unpack_again(u32x4& c) { asm volatile("" : "+v"(c)); }

struct NormBwd {
  const u32x4 *h1, *y, *dh1, *dx;
  const float *w_post, *gate, *row_gate, *w_pre;
  u32x4 *dh, *dy;
  float* drow_gate;
  float *part_pre, *part_post;   // [gridDim.x][d] sums of the rows a block walked
  int T, chunks;
  float res_scale, eps, inv_d;
};

// A thread owns its columns' channel sums.  They are registers where a lane has one
// chunk or a wave has the row, else LDS, which wider rows would otherwise spill
// (4096 x 16384 bf16: 207 us, 567 with spilled sums); bf16 rows of more than 16384
// have room there for those of the norm in front only, those of y stay in the
// workspace.  Threads with 16 elements of a row or more do not load the next one
// ahead (207 us, 317 ahead): the registers that are left hold one row, and a row is
// long enough to cover most of the wait.
template <class EL, int NC, int LPR, bool POST, bool PRE>
__global__ void __launch_bounds__(norm_bwd_threads(NC, LPR, 16)) block_norm_bwd_kernel(
    const NormBwd p) {
  constexpr int V = EL::VEC;
  constexpr bool WIDE = LPR == 0 && NC > 1, AHEAD = !WIDE || NC * V <= 8;
  constexpr bool POST_OUT = NC * V > 16 && PRE && POST;      // sums of y in the workspace
  constexpr int SLOTS = NC * 1024, SETS = WIDE ? PRE + POST - POST_OUT : 0;
  __shared__ f32x4 lds[2][16];
  __shared__ f32x4 sums[SETS ? SETS * (V / 4) * SLOTS : 1];  // [set][V / 4][chunk]
  const NormPlace<LPR> pl;
  const int lt = pl.lt, TPR = pl.tpr, rpb = LPR ? blockDim.x / (LPR ? LPR : 1) : 1;
  const int step = gridDim.x * rpb;
  bool in[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) in[i] = lt + i * TPR < p.chunks;
  u32x4 hr[NC], zr[NC], yr[NC], gr[NC];
  const u32x4 zero = {0, 0, 0, 0};
  auto fetch = [&](int row) {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const size_t o = (size_t)row * p.chunks + lt + i * TPR;
      const bool ok = in[i] && row < p.T;
      gr[i] = ok && p.dh1 ? p.dh1[o] : zero;
      if constexpr (PRE) {
        hr[i] = ok ? p.h1[o] : zero;
        zr[i] = ok ? p.dx[o] : zero;
      }
      if constexpr (POST) yr[i] = ok ? p.y[o] : zero;
    }
  };
  int t = blockIdx.x * rpb + pl.sub;
  if constexpr (AHEAD) fetch(t);
  constexpr int AC = WIDE ? 1 : NC;
  float wg[NC][V], wp[NC][V], apre[AC][V], apost[AC][V];
  // where four sums (q = 0 or 4) of this thread's chunk i live
  const auto sum4 = [&](bool post, int i, int q) -> f32x4* {
    if (post && POST_OUT)
      return reinterpret_cast<f32x4*>(p.part_post + ((size_t)blockIdx.x * p.chunks + lt + i * TPR) * V + q);
    return sums + ((post && PRE) * (V / 4) + q / 4) * SLOTS + lt + i * TPR;
  };
  // adds a[q] b[q] to the sums of chunk i
  auto add = [&](auto post, float (&acc)[AC][V], int i, const float* a, const float* b) {
    constexpr bool P = decltype(post)::value;
    if constexpr (WIDE) {
      if (!in[i] || !(P ? p.part_post : p.part_pre)) return;
#pragma unroll
      for (int q = 0; q < V; q += 4) {
        f32x4* at = sum4(P, i, q);
        f32x4 v = *at;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = fmaf(a[q + e], b[q + e], v[e]);
        *at = v;
      }
    } else {
#pragma unroll
      for (int q = 0; q < V; ++q) acc[i][q] = fmaf(a[q], b[q], acc[i][q]);
    }
  };
#pragma unroll
  for (int i = 0; i < AC; ++i)
#pragma unroll
    for (int q = 0; q < V; ++q) apre[i][q] = apost[i][q] = 0.0f;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
#pragma unroll
    for (int q = 0; q < V; ++q) wg[i][q] = wp[i][q] = 0.0f;
    if (in[i]) {
      const int c = lt + i * TPR;
      if constexpr (WIDE) {
#pragma unroll
        for (int q = 0; q < V; q += 4) {
          const f32x4 none = {0.0f, 0.0f, 0.0f, 0.0f};
          if (PRE) *sum4(false, i, q) = none;
          if (POST && (!POST_OUT || p.part_post)) *sum4(true, i, q) = none;
        }
      }
      if constexpr (POST) {
        float g[V];
        load_chan<V>(p.w_post, c, wg[i], 1.0f);
        load_chan<V>(p.gate, c, g, 1.0f);
#pragma unroll
        for (int q = 0; q < V; ++q) wg[i][q] *= g[q];
      }
      if constexpr (PRE) load_chan<V>(p.w_pre, c, wp[i], 1.0f);
    }
  }
  for (; t < p.T; t += step) {
    const size_t row = (size_t)t * p.chunks + lt;
    u32x4 hc[NC], zc[NC], yc[NC], gc[NC];
    if constexpr (!AHEAD) fetch(t);
#pragma unroll
    for (int i = 0; i < NC; ++i) hc[i] = hr[i], zc[i] = zr[i], yc[i] = yr[i], gc[i] = gr[i];
    if constexpr (AHEAD) fetch(t + step);
    float s[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      float h[V], z[V], y[V];
      if constexpr (PRE) {
        unpack_chunk(hc[i], h, EL());
        unpack_chunk(zc[i], z, EL());
      }
      if constexpr (POST) unpack_chunk(yc[i], y, EL());
#pragma unroll
      for (int q = 0; q < V; ++q) {
        if constexpr (PRE) {
          s[0] = fmaf(h[q], h[q], s[0]);
          s[1] = fmaf(z[q] * wp[i][q], h[q], s[1]);
        }
        if constexpr (POST) s[2] = fmaf(y[q], y[q], s[2]);
      }
    }
    if (PRE || p.w_post) row_sums<3, LPR>(s, lds, 0);
    if constexpr (WIDE) {
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        if constexpr (PRE) {
          unpack_again(hc[i]);
          unpack_again(zc[i]);
        }
        if constexpr (POST) unpack_again(yc[i]);
      }
    }
    float D[NC][V];
    {
      const float r = 1.0f / sqrtf(s[0] * p.inv_d + p.eps);
      const float m = -r * r * (s[1] * p.inv_d);
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        unpack_chunk(gc[i], D[i], EL());
        if constexpr (PRE) {
          float h[V], z[V], hn[V];
          unpack_chunk(hc[i], h, EL());
          unpack_chunk(zc[i], z, EL());
#pragma unroll
          for (int q = 0; q < V; ++q) {
            const float zw = z[q] * wp[i][q];
            hn[q] = h[q] * r;
            D[i][q] = fmaf(r, fmaf(h[q], m, zw), D[i][q]);
          }
          add(std::false_type(), apre, i, z, hn);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      float o[V];
#pragma unroll
      for (int q = 0; q < V; ++q) o[q] = p.res_scale * D[i][q];
      if (in[i]) p.dh[row + i * TPR] = store_chunk(o, EL());
    }
    if constexpr (POST) {
      const float ry = p.w_post ? 1.0f / sqrtf(s[2] * p.inv_d + p.eps) : 1.0f;
      const float f = ry * (p.row_gate ? p.row_gate[t] : 1.0f);
      float s2[1] = {0.0f};
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        float y[V], yf[V];
        unpack_chunk(yc[i], y, EL());
#pragma unroll
        for (int q = 0; q < V; ++q) yf[q] = y[q] * f;
        add(std::true_type(), apost, i, D[i], yf);
#pragma unroll
        for (int q = 0; q < V; ++q) {
          D[i][q] *= wg[i][q];
          s2[0] = fmaf(D[i][q], y[q], s2[0]);
        }
      }
      if (p.w_post || p.drow_gate) row_sums<1, LPR>(s2, lds, 1);
      if (p.drow_gate && lt == 0) p.drow_gate[t] = ry * s2[0];
      const float m = p.w_post ? -f * (ry * ry * (s2[0] * p.inv_d)) : 0.0f;
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        if constexpr (WIDE) unpack_again(yc[i]);
        float o[V], y[V];
        unpack_chunk(yc[i], y, EL());
#pragma unroll
        for (int q = 0; q < V; ++q) o[q] = fmaf(y[q], m, f * D[i][q]);
        if (in[i]) p.dy[row + i * TPR] = store_chunk(o, EL());
      }
    }
    // a row with only one of the two reductions meets the same LDS half again
    if (LPR == 0 && !(POST && p.w_post)) __syncthreads();
  }
  // one row of sums per block: a wave's rows are added in a butterfly, the waves
  // of a block that holds several rows in order
  auto put = [&](auto post, float* part, float (&a)[AC][V]) {
    constexpr bool P = decltype(post)::value;
    if (!part || (P && WIDE && POST_OUT)) return;
    float* o = part + (size_t)blockIdx.x * p.chunks * V;
    if constexpr (LPR > 0) {
      __shared__ __align__(16) float acc[NC * LPR * V];
#pragma unroll
      for (int m = LPR; m < 64; m <<= 1)
#pragma unroll
        for (int i = 0; i < NC; ++i)
#pragma unroll
          for (int q = 0; q < V; ++q) a[i][q] += __shfl_xor(a[i][q], m, 64);
      for (int w = 0; w < (int)(blockDim.x >> 6); ++w) {
        __syncthreads();
        if (w != (int)(threadIdx.x >> 6) || (threadIdx.x & 63) >= LPR) continue;
#pragma unroll
        for (int i = 0; i < NC; ++i)
#pragma unroll
          for (int q = 0; q < V; q += 4) {
            float* s = acc + (lt + i * LPR) * V + q;
            f32x4 v = {a[i][q], a[i][q + 1], a[i][q + 2], a[i][q + 3]};
            if (w) v = *reinterpret_cast<f32x4*>(s) + v;
            *reinterpret_cast<f32x4*>(s) = v;
          }
      }
      __syncthreads();
      for (int i = threadIdx.x; i < p.chunks * V / 4; i += blockDim.x)
        reinterpret_cast<f32x4*>(o)[i] = reinterpret_cast<f32x4*>(acc)[i];
    } else {
#pragma unroll
      for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int q = 0; q < V; q += 4)
          if (in[i]) {
            float* at = o + (size_t)(lt + i * TPR) * V + q;
            if constexpr (WIDE) *reinterpret_cast<f32x4*>(at) = *sum4(P, i, q);
            else store4(at, &a[i][q]);
          }
    }
  };
  if constexpr (PRE) put(std::false_type(), p.part_pre, apre);
  if constexpr (POST) put(std::true_type(), p.part_post, apost);
}

// The channel gradients from the blocks' rows of sums, added in order: 32 groups
// of lanes share 32 columns (128 bytes), each adding every 32nd row, eight loads
// in flight.
struct NormFinish {
  const float *part_pre, *part_post, *w_post, *gate;
  float *dw_pre, *dw_post, *dgate;
  int rows, d, accumulate;
};

__global__ void __launch_bounds__(1024) block_norm_finish_kernel(const NormFinish p) {
  __shared__ float lds[32][33];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  const float* part = blockIdx.y ? p.part_post : p.part_pre;
  if (!part) return;
  float s = 0.0f;
  if (c < p.d) {
    int r = w;
    for (; r + 7 * 32 < p.rows; r += 8 * 32) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = part[(size_t)(r + 32 * i) * p.d + c];
#pragma unroll
      for (int i = 0; i < 8; ++i) s += v[i];
    }
    for (; r < p.rows; r += 32) s += part[(size_t)r * p.d + c];
  }
  lds[w][lane] = s;
  __syncthreads();
  if (w || c >= p.d) return;
  s = 0.0f;
#pragma unroll
  for (int i = 0; i < 32; ++i) s += lds[i][lane];
  auto put = [&](float* o, float v) {
    if (o) o[c] = p.accumulate ? o[c] + v : v;
  };
  if (blockIdx.y == 0) {
    put(p.dw_pre, s);
  } else {
    put(p.dw_post, s * (p.gate ? p.gate[c] : 1.0f));
    put(p.dgate, s * (p.w_post ? p.w_post[c] : 1.0f));
  }
}

// The geometry of a row: chunks per lane, lanes of a wave per row (0: the row has
// a block), waves per row of a block.
struct NormGeom {
  int nc, lpr, waves;
};
// Rows of up to 64 chunks share a wave where they can (16384 x 64: backward 9.9 us,
// a wave a row 18.6); the combine, whose expert rows are not loaded ahead, takes
// two chunks a lane to have more loads in flight (8191 x 2880, 4 rows: 59 us, one
// chunk 65).
static NormGeom norm_geom(int chunks, bool comb = false) {
  if (chunks <= 8) return {1, 8, 0};
  if (chunks <= 16) return {1, 16, 0};
  if (chunks <= 32) return {1, 32, 0};
  if (chunks <= 64) return {1, 64, 0};
  if (chunks <= 128) return {2, 64, 0};
  const int nc = chunks <= 1024 && !comb ? 1 : chunks <= 2048 ? 2 : 4;
  return {nc, 0, (chunks + 64 * nc - 1) / (64 * nc)};
}

// Calls f.template run<NC, LPR>(waves per row) for a row's geometry.
template <class F>
static moe_status_t norm_dispatch(const NormGeom& g, F&& f) {
  switch (g.lpr) {
    case 8: return f.template run<1, 8>(0);
    case 16: return f.template run<1, 16>(0);
    case 32: return f.template run<1, 32>(0);
    case 64: return g.nc == 1 ? f.template run<1, 64>(0) : f.template run<2, 64>(0);
  }
  return g.nc == 1   ? f.template run<1, 0>(g.waves)
         : g.nc == 2 ? f.template run<2, 0>(g.waves)
                     : f.template run<4, 0>(g.waves);
}

static constexpr int NORM_MAX_CHUNKS = 4096;
// a row past the last one is still a positive int
static constexpr int NORM_MAX_ROWS = INT32_MAX - (1 << 20);

// Blocks of the backward: enough to fill 256 compute units with 8 to 16 waves
// each, a fixed number (not the card's own count), so that the order of the
// channel sums is the same everywhere.
static int norm_bwd_blocks(int T, int chunks) {
  const NormGeom g = norm_geom(chunks);
  const int threads = norm_bwd_threads(g.nc, g.lpr, g.waves), rpb = g.lpr ? threads / g.lpr : 1;
  const int per_cu = g.lpr == 64 ? 1 : std::max(1, std::min(4, 1024 / threads));
  return std::min((T + rpb - 1) / rpb, 256 * per_cu);
}

template <class EL>
struct LaunchNormFwd {
  const NormFwd& p;
  hipStream_t s;
  template <int NC, int LPR, bool POST, bool PRE, bool COMB>
  moe_status_t go(int waves) const {
    const int threads = LPR ? 256 : 64 * waves, rpb = LPR ? threads / (LPR ? LPR : 1) : 1;
    const int blocks = std::min((p.T + rpb - 1) / rpb,
                                device_cu_count() * std::max(1, (COMB ? 960 : 1024) / threads));
    if (p.stream)
      hipLaunchKernelGGL((block_norm_fwd_kernel<EL, NC, LPR, POST, PRE, COMB, true>), dim3(blocks),
                         dim3(threads), 0, s, p);
    else
      hipLaunchKernelGGL((block_norm_fwd_kernel<EL, NC, LPR, POST, PRE, COMB, false>),
                         dim3(blocks), dim3(threads), 0, s, p);
    return launch_status();
  }
  template <int NC, int LPR>
  moe_status_t run(int waves) const {
    if (!p.y) return go<NC, LPR, false, true, false>(waves);
    if (p.row_map)
      return p.x_out ? go<NC, LPR, true, true, true>(waves) : go<NC, LPR, true, false, true>(waves);
    return p.x_out ? go<NC, LPR, true, true, false>(waves) : go<NC, LPR, true, false, false>(waves);
  }
};

template <class EL>
struct LaunchNormBwd {
  const NormBwd& p;
  hipStream_t s;
  int blocks;
  template <int NC, int LPR, bool POST, bool PRE>
  moe_status_t go(int waves) const {
    const int threads = norm_bwd_threads(NC, LPR, waves);
    hipLaunchKernelGGL((block_norm_bwd_kernel<EL, NC, LPR, POST, PRE>), dim3(blocks),
                       dim3(threads), 0, s, p);
    return launch_status();
  }
  template <int NC, int LPR>
  moe_status_t run(int waves) const {
    if (!p.y) return go<NC, LPR, false, true>(waves);
    return p.dx ? go<NC, LPR, true, true>(waves) : go<NC, LPR, true, false>(waves);
  }
};

}  // namespace moe

using namespace moe;

extern "C" {

moe_status_t moe_block_norm_fwd(const moe_block_norm_fwd_args_t* a, void* stream) {
  MOE_CHECK_ARG(a && a->struct_size >= sizeof(moe_block_norm_fwd_args_t));
  MOE_CHECK_ARG(a->T >= 0 && a->T <= NORM_MAX_ROWS && a->d > 0 && valid_dtype(a->dtype));
  MOE_CHECK_ARG(((size_t)a->d * dtype_size(a->dtype)) % 16 == 0);
  MOE_CHECK_ARG(a->eps > 0.0f && isfinite(a->eps) && isfinite(a->res_scale));
  if (a->T == 0) return MOE_OK;
  const bool post = a->y != nullptr;
  MOE_CHECK_ARG(post || a->w_pre);
  MOE_CHECK_ARG(post || (!a->w_post && !a->gate && !a->row_gate && !a->row_map && !a->topk_w &&
                         !a->h_out && !a->y_out));
  MOE_CHECK_ARG((a->w_pre == nullptr) == (a->x_out == nullptr));
  MOE_CHECK_ARG(a->row_map ? a->k >= 1 && a->k <= MOE_MAX_TOPK : !a->topk_w && !a->y_out);
  const int k = a->row_map ? a->k : 1;
  MOE_CHECK_ARG((size_t)a->T * k < (size_t)INT32_MAX);
  const size_t chunks = (size_t)a->d * dtype_size(a->dtype) / 16;
  if (chunks > NORM_MAX_CHUNKS) return MOE_ERR_UNSUPPORTED;
  MOE_CHECK_ARG(a->h && aligned16(a->h) && aligned16(a->y) && aligned16(a->w_post) &&
                aligned16(a->gate) && aligned16(a->w_pre) && aligned16(a->h_out) &&
                aligned16(a->x_out) && aligned16(a->y_out));
  MOE_CHECK_ARG(!post || a->h_out);
  const size_t n = (size_t)a->T * chunks * 16, nd = (size_t)a->d * 4, nk = (size_t)a->T * k * 4;
  MOE_CHECK_ARG(same_or_apart(a->h_out, a->h, n) && same_or_apart(a->x_out, a->h, n) &&
                (a->row_map || (same_or_apart(a->h_out, a->y, n) && same_or_apart(a->x_out, a->y, n))));
  // expert rows are read for other rows than the ones written
  MOE_CHECK_ARG(outputs_apart({{a->h_out, n}, {a->x_out, n}, {a->y_out, n}},
                              {{a->w_post, nd}, {a->gate, nd}, {a->w_pre, nd},
                               {a->row_gate, (size_t)a->T * 4}, {a->row_map, nk}, {a->topk_w, nk},
                               {a->row_map ? a->y : nullptr, n * k}}) &&
                !overlap({a->y_out, n}, {a->h, n}));
  const NormFwd p = {static_cast<const u32x4*>(a->h), static_cast<const u32x4*>(a->y),
                     a->w_post, a->gate, a->row_gate, a->w_pre, a->row_map, a->topk_w,
                     static_cast<u32x4*>(a->h_out), static_cast<u32x4*>(a->x_out),
                     static_cast<u32x4*>(a->y_out), a->T, k, a->T * k, (int)chunks, a->res_scale,
                     a->eps, 1.0f / (float)a->d, n >= (size_t)16 << 20};
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const NormGeom g = norm_geom((int)chunks, a->row_map != nullptr);
  return a->dtype == MOE_BF16 ? norm_dispatch(g, LaunchNormFwd<BF16>{p, s})
                              : norm_dispatch(g, LaunchNormFwd<F32>{p, s});
}

size_t moe_block_norm_bwd_workspace_size(int T, int d) {
  if (T <= 0 || d <= 0) return 0;
  // a row of sums per block for either norm; the larger of the two types' counts
  // (at most NORM_MAX_CHUNKS chunks: wider rows are refused)
  const int c16 = (int)std::min(((size_t)d + 7) / 8, (size_t)NORM_MAX_CHUNKS);
  const int c32 = (int)std::min(((size_t)d + 3) / 4, (size_t)NORM_MAX_CHUNKS);
  const size_t blocks = std::max(norm_bwd_blocks(T, c16), norm_bwd_blocks(T, c32));
  return blocks * d * 2 * sizeof(float);
}

moe_status_t moe_block_norm_bwd(const moe_block_norm_bwd_args_t* a, void* stream) {
  MOE_CHECK_ARG(a && a->struct_size >= sizeof(moe_block_norm_bwd_args_t));
  MOE_CHECK_ARG(a->T >= 0 && a->T <= NORM_MAX_ROWS && a->d > 0 && valid_dtype(a->dtype));
  MOE_CHECK_ARG(((size_t)a->d * dtype_size(a->dtype)) % 16 == 0);
  MOE_CHECK_ARG(a->eps > 0.0f && isfinite(a->eps) && isfinite(a->res_scale));
  const bool post = a->y != nullptr, pre = a->dx != nullptr;
  if (a->T > 0) {      // (tensors without rows have no address)
    MOE_CHECK_ARG((post || pre) && (pre || a->dh1));
    MOE_CHECK_ARG(pre ? a->w_pre && a->h1 : !a->w_pre && !a->dw_pre);
    MOE_CHECK_ARG(post ? a->dy != nullptr
                       : !a->w_post && !a->gate && !a->row_gate && !a->dw_post && !a->dgate &&
                             !a->drow_gate && !a->dy);
    MOE_CHECK_ARG(a->row_gate || !a->drow_gate);
  }
  MOE_CHECK_ARG((a->w_post || !a->dw_post) && (a->gate || !a->dgate) && (a->w_pre || !a->dw_pre));
  const size_t chunks = (size_t)a->d * dtype_size(a->dtype) / 16;
  if (chunks > NORM_MAX_CHUNKS) return MOE_ERR_UNSUPPORTED;
  MOE_CHECK_ARG(aligned16(a->h1) && aligned16(a->y) && aligned16(a->dh1) && aligned16(a->dx) &&
                aligned16(a->w_post) && aligned16(a->gate) && aligned16(a->w_pre) &&
                aligned16(a->dh) && aligned16(a->dy) && aligned16(a->ws));
  const bool chan_pre = a->dw_pre != nullptr, chan_post = a->dw_post || a->dgate;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  float* ws = static_cast<float*>(a->ws);
  const int rows = a->T > 0 ? norm_bwd_blocks(a->T, (int)chunks) : 0;
  if (a->T > 0) {
    MOE_CHECK_ARG(a->dh);
    const size_t n = (size_t)a->T * chunks * 16, nd = (size_t)a->d * 4, nt = (size_t)a->T * 4;
    const size_t need = moe_block_norm_bwd_workspace_size(a->T, a->d);
    if ((chan_pre || chan_post) &&
        (!ws || a->ws_bytes < need || need < (size_t)rows * a->d * 2 * sizeof(float)))
      return MOE_ERR_WORKSPACE;
    for (void* o : {a->dh, a->dy})
      for (const void* i : {a->h1, a->y, a->dh1, a->dx}) MOE_CHECK_ARG(same_or_apart(o, i, n));
    const Span part = {chan_pre || chan_post ? ws : nullptr, need};
    MOE_CHECK_ARG(outputs_apart({{a->dh, n}, {a->dy, n}, {a->dw_post, nd}, {a->dgate, nd},
                                 {a->dw_pre, nd}, {a->drow_gate, nt}, part},
                                {{a->w_post, nd}, {a->gate, nd}, {a->w_pre, nd},
                                 {a->row_gate, nt}}));
    MOE_CHECK_ARG(outputs_apart({part, {a->drow_gate, nt}},
                                {{a->h1, n}, {a->y, n}, {a->dh1, n}, {a->dx, n}}));
    for (const float* o : {a->dw_post, a->dgate, a->dw_pre})
      for (const void* i : {a->h1, a->y, a->dh1, a->dx}) MOE_CHECK_ARG(!overlap({o, nd}, {i, n}));
    float* part_pre = chan_pre ? ws : nullptr;
    float* part_post = chan_post ? ws + (size_t)rows * a->d : nullptr;
    const NormBwd p = {static_cast<const u32x4*>(a->h1), static_cast<const u32x4*>(a->y),
                       static_cast<const u32x4*>(a->dh1), static_cast<const u32x4*>(a->dx),
                       a->w_post, a->gate, a->row_gate, a->w_pre, static_cast<u32x4*>(a->dh),
                       static_cast<u32x4*>(a->dy), a->drow_gate, part_pre, part_post, a->T,
                       (int)chunks, post ? a->res_scale : 1.0f, a->eps, 1.0f / (float)a->d};
    const moe_status_t st =
        a->dtype == MOE_BF16 ? norm_dispatch(norm_geom((int)chunks), LaunchNormBwd<BF16>{p, s, rows})
                             : norm_dispatch(norm_geom((int)chunks), LaunchNormBwd<F32>{p, s, rows});
    if (st != MOE_OK) return st;
  }
  if (chan_pre || chan_post) {
    // no rows: exact zeros (or the existing values when accumulating)
    const float* base = rows ? ws : chan_pre ? a->w_pre : a->w_post ? a->w_post : a->gate;
    const NormFinish f = {chan_pre ? base : nullptr,
                          chan_post ? (rows ? ws + (size_t)rows * a->d : base) : nullptr,
                          a->w_post, a->gate, a->dw_pre, a->dw_post, a->dgate, rows, a->d,
                          a->accumulate};
    hipLaunchKernelGGL(block_norm_finish_kernel, dim3((a->d + 31) / 32, 2), dim3(1024), 0, s, f);
    return launch_status();
  }
  return MOE_OK;
}

}  // extern "C"
