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
#include "common.hpp"
#include "spans.hpp"

#include <math.h>
#include <stddef.h>

#include <algorithm>
#include <type_traits>

namespace moe {

// TPR threads share a row; a thread owns chunks tid, tid + TPR, ... (NC of them).
template <int TPR>
struct NormGeom {
  static constexpr int THREADS = TPR < 256 ? 256 : TPR;
  static constexpr int RPB = THREADS / TPR;      // rows per block and step
  static constexpr int WPR = TPR / 64;           // waves per row
};

// Sums of NV values over the TPR threads of a row, on every thread.  A wave's
// butterfly, then the row's waves in order through LDS.  `buf` alternates
// between two halves: a thread writes one half again only after the barrier
// of the other, which every thread reaches after reading the first.
template <int NV, int TPR>
__device__ __forceinline__ void row_sums(float (&v)[NV], float* lds, int half) {
#pragma unroll
  for (int i = 0; i < NV; ++i) v[i] = wave_sum(v[i]);
  if constexpr (TPR > 64) {
    constexpr int WPR = TPR / 64;
    float* b = lds + half * (WPR * 4);
    const int w = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int i = 0; i < NV; ++i) b[w * 4 + i] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] = 0.0f;
#pragma unroll
    for (int j = 0; j < WPR; ++j)
#pragma unroll
      for (int i = 0; i < NV; ++i) v[i] += b[j * 4 + i];
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
};

// y[t]'s chunk c from its expert rows, four rows' loads in flight.
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
      raw[j] = p.y[(size_t)r * p.chunks + c];
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
  for (; j < p.k; ++j) add(std::integral_constant<int, 1>(), j);
}

// Blocks walk the rows; a row's loads are issued while the one before it is
// reduced, and the channel vectors stay in registers throughout.
template <class EL, int TPR, int NC, bool POST, bool PRE, bool COMB>
__global__ void __launch_bounds__(NormGeom<TPR>::THREADS) block_norm_fwd_kernel(const NormFwd p) {
  typedef NormGeom<TPR> G;
  constexpr int V = EL::VEC;
  constexpr bool LOADY = POST && !COMB;
  __shared__ float lds[2 * G::WPR * 4];
  const int lt = threadIdx.x % TPR;
  // (uniform over a wave)
  int t = __builtin_amdgcn_readfirstlane(blockIdx.x * G::RPB + threadIdx.x / TPR);
  const int step = gridDim.x * G::RPB;
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
  fetch(t);
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
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      unpack_chunk(hr[i], h[i], EL());
      if constexpr (LOADY) unpack_chunk(yr[i], y[i], EL());
    }
    fetch(t + step);
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
        row_sums<1, TPR>(s, lds, 0);
        f *= 1.0f / sqrtf(s[0] * p.inv_d + p.eps);
      }
#pragma unroll
      for (int i = 0; i < NC; ++i) {
#pragma unroll
        for (int q = 0; q < V; ++q) h[i][q] = fmaf(p.res_scale, h[i][q], y[i][q] * (f * wg[i][q]));
        if (in[i]) p.h_out[row + i * TPR] = store_chunk(h[i], EL());
      }
    }
    if constexpr (PRE) {
      float s[1] = {0.0f};
#pragma unroll
      for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int q = 0; q < V; ++q) s[0] = fmaf(h[i][q], h[i][q], s[0]);
      row_sums<1, TPR>(s, lds, 1);
      const float r = 1.0f / sqrtf(s[0] * p.inv_d + p.eps);
#pragma unroll
      for (int i = 0; i < NC; ++i) {
#pragma unroll
        for (int q = 0; q < V; ++q) h[i][q] *= r * wp[i][q];
        if (in[i]) p.x_out[row + i * TPR] = store_chunk(h[i], EL());
      }
    }
    // a row with only one of the two reductions meets the same LDS half again
    // in the next step
    if (TPR > 64 && !(PRE && POST && p.w_post)) __syncthreads();
  }
}

struct NormBwd {
  const u32x4 *h1, *y, *dh1, *dx;
  const float *w_post, *gate, *row_gate, *w_pre;
  u32x4 *dh, *dy;
  float* drow_gate;
  float *part_pre, *part_post;   // [gridDim.x * RPB][d] sums of the rows a row group walked
  int T, chunks;
  float res_scale, eps, inv_d;
};

template <class EL, int TPR, int NC>
__global__ void __launch_bounds__(NormGeom<TPR>::THREADS) block_norm_bwd_kernel(const NormBwd p) {
  typedef NormGeom<TPR> G;
  constexpr int V = EL::VEC;
  __shared__ float lds[2 * G::WPR * 4];
  const int lt = threadIdx.x % TPR;
  float apre[NC][V], apost[NC][V];
#pragma unroll
  for (int i = 0; i < NC; ++i)
#pragma unroll
    for (int q = 0; q < V; ++q) apre[i][q] = apost[i][q] = 0.0f;
  for (int t = blockIdx.x * G::RPB + threadIdx.x / TPR; t < p.T; t += gridDim.x * G::RPB) {
    const size_t row = (size_t)t * p.chunks;
    float D[NC][V], h[NC][V], z[NC][V], y[NC][V];
    float s[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = lt + i * TPR;
#pragma unroll
      for (int q = 0; q < V; ++q) D[i][q] = h[i][q] = z[i][q] = y[i][q] = 0.0f;
      if (c < p.chunks) {
        if (p.dh1) unpack_chunk(p.dh1[row + c], D[i], EL());
        if (p.dx) {
          unpack_chunk(p.h1[row + c], h[i], EL());
          unpack_chunk(p.dx[row + c], z[i], EL());
        }
        if (p.y) unpack_chunk(p.y[row + c], y[i], EL());
      }
    }
    if (p.dx) {
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int c = lt + i * TPR;
        float w[V];
        if (c < p.chunks) load_chan<V>(p.w_pre, c, w, 1.0f);
#pragma unroll
        for (int q = 0; q < V; ++q) {
          s[0] = fmaf(h[i][q], h[i][q], s[0]);
          if (c < p.chunks) s[1] = fmaf(z[i][q] * w[q], h[i][q], s[1]);
        }
      }
    }
    if (p.y && p.w_post) {
#pragma unroll
      for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int q = 0; q < V; ++q) s[2] = fmaf(y[i][q], y[i][q], s[2]);
    }
    if (p.dx || (p.y && p.w_post)) row_sums<3, TPR>(s, lds, 0);
    if (p.dx) {
      const float r = 1.0f / sqrtf(s[0] * p.inv_d + p.eps);
      const float m = r * r * (s[1] * p.inv_d);
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int c = lt + i * TPR;
        if (c < p.chunks) {
          float w[V];
          load_chan<V>(p.w_pre, c, w, 1.0f);
#pragma unroll
          for (int q = 0; q < V; ++q) {
            apre[i][q] = fmaf(z[i][q], h[i][q] * r, apre[i][q]);
            D[i][q] = fmaf(r, fmaf(-h[i][q], m, z[i][q] * w[q]), D[i][q]);
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = lt + i * TPR;
      if (c < p.chunks) {
        float o[V];
#pragma unroll
        for (int q = 0; q < V; ++q) o[q] = p.res_scale * D[i][q];
        p.dh[row + c] = pack_chunk(o, EL());
      }
    }
    if (p.y) {
      const float ry = p.w_post ? 1.0f / sqrtf(s[2] * p.inv_d + p.eps) : 1.0f;
      const float rg = p.row_gate ? p.row_gate[t] : 1.0f;
      float s2[1] = {0.0f};
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int c = lt + i * TPR;
        if (c < p.chunks) {
          float w[V], g[V];
          load_chan<V>(p.w_post, c, w, 1.0f);
          load_chan<V>(p.gate, c, g, 1.0f);
#pragma unroll
          for (int q = 0; q < V; ++q) {
            apost[i][q] = fmaf(D[i][q], y[i][q] * (ry * rg), apost[i][q]);
            D[i][q] *= w[q] * g[q];
            s2[0] = fmaf(D[i][q], y[i][q], s2[0]);
          }
        }
      }
      if (p.w_post || p.drow_gate) row_sums<1, TPR>(s2, lds, 1);
      if (p.drow_gate && lt == 0) p.drow_gate[t] = ry * s2[0];
      const float m = p.w_post ? ry * ry * (s2[0] * p.inv_d) : 0.0f;
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int c = lt + i * TPR;
        if (c < p.chunks) {
          float o[V];
#pragma unroll
          for (int q = 0; q < V; ++q) o[q] = ry * rg * fmaf(-y[i][q], m, D[i][q]);
          p.dy[row + c] = pack_chunk(o, EL());
        }
      }
    }
    if (TPR > 64) __syncthreads();
  }
  const size_t prow = ((size_t)blockIdx.x * G::RPB + threadIdx.x / TPR) * p.chunks * V;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = lt + i * TPR;
    if (c < p.chunks) {
#pragma unroll
      for (int q = 0; q < V; q += 4) {
        if (p.part_pre) store4(p.part_pre + prow + (size_t)c * V + q, &apre[i][q]);
        if (p.part_post) store4(p.part_post + prow + (size_t)c * V + q, &apost[i][q]);
      }
    }
  }
}

// The channel gradients from the blocks' partial rows, added in order:
// 16 waves share 64 columns, each summing every 16th row.
struct NormFinish {
  const float *part_pre, *part_post, *w_post, *gate;
  float *dw_pre, *dw_post, *dgate;
  int rows, d, accumulate;
};

__global__ void __launch_bounds__(1024) block_norm_finish_kernel(const NormFinish p) {
  __shared__ float lds[16][64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int c = blockIdx.x * 64 + lane;
  const float* part = blockIdx.y ? p.part_post : p.part_pre;
  if (!part) return;
  float s = 0.0f;
  if (c < p.d)
    for (int r = w; r < p.rows; r += 16) s += part[(size_t)r * p.d + c];
  lds[w][lane] = s;
  __syncthreads();
  if (w || c >= p.d) return;
  s = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) s += lds[i][lane];
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

// Row groups of the backward's grid: a fixed number (not the card's CU count,
// so that the order of the channel sums is the same everywhere).
static constexpr int NORM_BWD_GROUPS = 512;

static int norm_groups(int T) { return T < NORM_BWD_GROUPS ? T : NORM_BWD_GROUPS; }

// Calls f.template run<TPR, NC>() for a row of `chunks` 16-byte chunks.
template <class F>
static moe_status_t norm_dispatch(int chunks, F&& f) {
  if (chunks <= 64) return f.template run<64, 1>();
  if (chunks <= 128) return f.template run<64, 2>();
  if (chunks <= 256) return f.template run<256, 1>();
  if (chunks <= 512) return f.template run<256, 2>();
  if (chunks <= 1024) return f.template run<512, 2>();
  if (chunks <= 2048) return f.template run<1024, 2>();
  return f.template run<1024, 4>();
}

static constexpr int NORM_MAX_CHUNKS = 4096;

template <class EL>
struct LaunchNormFwd {
  const NormFwd& p;
  hipStream_t s;
  template <int TPR, int NC, bool POST, bool PRE, bool COMB>
  moe_status_t go() const {
    typedef NormGeom<TPR> G;
    const int groups = (p.T + G::RPB - 1) / G::RPB;
    const int blocks = std::min(groups, device_cu_count() * (2048 / G::THREADS) / 2);
    hipLaunchKernelGGL((block_norm_fwd_kernel<EL, TPR, NC, POST, PRE, COMB>), dim3(blocks),
                       dim3(G::THREADS), 0, s, p);
    return launch_status();
  }
  template <int TPR, int NC>
  moe_status_t run() const {
    if (!p.y) return go<TPR, NC, false, true, false>();
    if (p.row_map)
      return p.x_out ? go<TPR, NC, true, true, true>() : go<TPR, NC, true, false, true>();
    return p.x_out ? go<TPR, NC, true, true, false>() : go<TPR, NC, true, false, false>();
  }
};

template <class EL>
struct LaunchNormBwd {
  const NormBwd& p;
  hipStream_t s;
  int* rows;      // partial rows written
  template <int TPR, int NC>
  moe_status_t run() const {
    typedef NormGeom<TPR> G;
    const int blocks = (norm_groups(p.T) + G::RPB - 1) / G::RPB;
    *rows = blocks * G::RPB;
    hipLaunchKernelGGL((block_norm_bwd_kernel<EL, TPR, NC>), dim3(blocks), dim3(G::THREADS), 0, s,
                       p);
    return launch_status();
  }
};

}  // namespace moe

using namespace moe;

extern "C" {

moe_status_t moe_block_norm_fwd(const moe_block_norm_fwd_args_t* a, void* stream) {
  MOE_CHECK_ARG(a && a->struct_size >= sizeof(moe_block_norm_fwd_args_t));
  MOE_CHECK_ARG(a->T >= 0 && a->d > 0 && valid_dtype(a->dtype));
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
                     a->eps, 1.0f / (float)a->d};
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  return a->dtype == MOE_BF16 ? norm_dispatch((int)chunks, LaunchNormFwd<BF16>{p, s})
                              : norm_dispatch((int)chunks, LaunchNormFwd<F32>{p, s});
}

size_t moe_block_norm_bwd_workspace_size(int T, int d) {
  if (T <= 0 || d <= 0) return 0;
  // two partial rows per row group; up to three groups more than rows where a
  // block holds four
  return (size_t)(norm_groups(T) + 3) * d * 2 * sizeof(float);
}

moe_status_t moe_block_norm_bwd(const moe_block_norm_bwd_args_t* a, void* stream) {
  MOE_CHECK_ARG(a && a->struct_size >= sizeof(moe_block_norm_bwd_args_t));
  MOE_CHECK_ARG(a->T >= 0 && a->d > 0 && valid_dtype(a->dtype));
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
  int rows = 0;
  if (a->T > 0) {
    MOE_CHECK_ARG(a->dh);
    const size_t n = (size_t)a->T * chunks * 16, nd = (size_t)a->d * 4, nt = (size_t)a->T * 4;
    const size_t need = moe_block_norm_bwd_workspace_size(a->T, a->d);
    if ((chan_pre || chan_post) && (!ws || a->ws_bytes < need)) return MOE_ERR_WORKSPACE;
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
    float* part_post = chan_post ? ws + (size_t)(norm_groups(a->T) + 3) * a->d : nullptr;
    const NormBwd p = {static_cast<const u32x4*>(a->h1), static_cast<const u32x4*>(a->y),
                       static_cast<const u32x4*>(a->dh1), static_cast<const u32x4*>(a->dx),
                       a->w_post, a->gate, a->row_gate, a->w_pre, static_cast<u32x4*>(a->dh),
                       static_cast<u32x4*>(a->dy), a->drow_gate, part_pre, part_post, a->T,
                       (int)chunks, post ? a->res_scale : 1.0f, a->eps, 1.0f / (float)a->d};
    const moe_status_t st =
        a->dtype == MOE_BF16 ? norm_dispatch((int)chunks, LaunchNormBwd<BF16>{p, s, &rows})
                             : norm_dispatch((int)chunks, LaunchNormBwd<F32>{p, s, &rows});
    if (st != MOE_OK) return st;
  }
  if (chan_pre || chan_post) {
    // no rows: exact zeros (or the existing values when accumulating)
    const float* base = rows ? ws : chan_pre ? a->w_pre : a->w_post ? a->w_post : a->gate;
    const NormFinish f = {chan_pre ? base : nullptr,
                          chan_post ? (rows ? ws + (size_t)(norm_groups(a->T) + 3) * a->d : base)
                                    : nullptr,
                          a->w_post, a->gate, a->dw_pre, a->dw_post, a->dgate, rows, a->d,
                          a->accumulate};
    hipLaunchKernelGGL(block_norm_finish_kernel, dim3((a->d + 63) / 64, 2), dim3(1024), 0, s, f);
    return launch_status();
  }
  return MOE_OK;
}

}  // extern "C"
