// Low-rank adapters of many requests beside a shared projection.
//
// The rows of a batch are grouped by adapter (offsets, and src_row for rows
// that are not stored in that order: moe_permute's outputs with one slot per
// token).  For the row at position p of adapter a's segment, token t:
//   forward   v[p] = A[a] x[t],            out[t] = y[t] + s[a] B[a] v[p]
//   backward  u[p] = s[a] B[a]^T dy[t],    dx_out[t] = dx[t] + A[a]^T u[p]
//             dA[a] = sum_p u[p] x[t]^T,   dB[a] = s[a] sum_p dy[t] v[p]^T
// with A [r, K], B [N, r], r much smaller than K and N: every product is bound
// by the memory it reads (x, y, dy once per pass, the adapters once per tile of
// rows), not by the matrix cores.
//
// Two kernels make a pass over activations: `shrink` reduces a tile of rows to
// its r values (the reduction split over waves, and over blocks where there are
// few rows; a block's partial sums go to the workspace and are added in order),
// `expand` adds their products with the other factor to the wide rows.  The r
// values stay float32 between the two: in front of the bf16 matrix cores each
// is split into a high and a low bf16 part (x = hi + lo up to 2^-17 |x|), laid
// side by side along the reduction, so a step over 32 covers 16 ranks at
// twice bf16's precision.  Weight gradients are float32 throughout.
#include "common.hpp"
#include "spans.hpp"

#include <math.h>
#include <stddef.h>

#include <algorithm>

namespace moe {

static constexpr int LORA_MAX_RANK = 128;
static constexpr int LORA_WAVES = 4;

// A tile of at most TM rows of one adapter's segment (adapter NA: the rows
// behind the last segment), or n == 0 past the last tile.
struct LoraTile {
  int a, p0, n;
};

// Tile i of the segments, each cut into tiles of TM rows.  Called by whole
// waves; the lanes take one segment each, 64 at a time.
template <int TM>
__device__ __forceinline__ LoraTile lora_tile(const int32_t* offsets, int NA, int T, int i) {
  const int lane = threadIdx.x & 63;
  int before = 0;
  for (int base = 0; base <= NA; base += 64) {
    const int a = base + lane;
    int s = T, e = T;
    if (a <= NA) {
      s = min(max(offsets[a], 0), T);
      e = a < NA ? min(max(offsets[a + 1], s), T) : T;
    }
    const int nt = (e - s + TM - 1) / TM;
    int incl = nt;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int v = __shfl_up(incl, o, 64);
      if (lane >= o) incl += v;
    }
    const uint64_t hit = __ballot(before + incl > i);
    if (hit) {
      const int l = __ffsll((unsigned long long)hit) - 1;
      const int first = before + __shfl(incl - nt, l, 64);
      const int p0 = __shfl(s, l, 64) + (i - first) * TM;
      return {base + l, p0, min(TM, __shfl(e, l, 64) - p0)};
    }
    before += __shfl(incl, 63, 64);
  }
  return {0, 0, 0};
}

__device__ __forceinline__ int lora_token(const int32_t* src_row, int p, int T) {
  const int t = src_row ? src_row[p] : p;
  return (unsigned)t < (unsigned)T ? t : -1;
}

__device__ __forceinline__ f32x4 mfma16(const u32x4& a, const u32x4& b, const f32x4& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                 __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// Eight elements of a column of w (row stride ld), rows i .. i + 7.
__device__ __forceinline__ u32x4 column8(const uint16_t* w, size_t ld) {
  u32x4 o;
#pragma unroll
  for (int q = 0; q < 4; ++q)
    o[q] = (uint32_t)w[(2 * q) * ld] | ((uint32_t)w[(2 * q + 1) * ld] << 16);
  return o;
}

struct LoraShrink {
  const uint16_t *x, *w;      // rows [T, C]; factor [NA, r, C], or [NA, C, r] (TRANS)
  const int32_t *offsets, *src_row;
  float* part;                // [splits][T][r], by position
  int T, C, r, NA, steps;     // steps of 32 along C
};

// part[split][p][j] = sum over the split's share of C of x[t(p)][c] w[a][j][c].
// The four waves share the block's steps; MFMA: first operand the factor's rows
// (register 4 (lane >> 4) + q = rank), second the activation rows (lane & 15).
template <int MT, int RT, bool TRANS>
__global__ void __launch_bounds__(64 * LORA_WAVES) lora_shrink_kernel(const LoraShrink p) {
  constexpr int TM = 16 * MT, R = 16 * RT;
  __shared__ float red[LORA_WAVES][16][R + 4];
  const LoraTile tl = lora_tile<TM>(p.offsets, p.NA, p.T, blockIdx.x);
  if (tl.n <= 0 || tl.a >= p.NA) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int l = lane & 15, g = lane >> 4;
  // rows past the tile, ranks past r: a valid row or rank is read again, its
  // results are dropped
  const uint16_t* xr[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int t = lora_token(p.src_row, tl.p0 + min(16 * m + l, tl.n - 1), p.T);
    xr[m] = p.x + (size_t)max(t, 0) * p.C + 8 * g;
  }
  const uint16_t* w = p.w + (size_t)tl.a * p.r * p.C;
  f32x4 acc[MT][RT] = {};
  const int parts = gridDim.y * LORA_WAVES, part = blockIdx.y * LORA_WAVES + wave;
  const int s0 = (int)((long long)p.steps * part / parts);
  const int s1 = (int)((long long)p.steps * (part + 1) / parts);
#pragma unroll 2
  for (int s = s0; s < s1; ++s) {
    u32x4 xa[MT], wa[RT];
#pragma unroll
    for (int m = 0; m < MT; ++m) xa[m] = *reinterpret_cast<const u32x4*>(xr[m] + 32 * s);
#pragma unroll
    for (int j = 0; j < RT; ++j) {
      const int rank = min(16 * j + l, p.r - 1);
      if constexpr (TRANS)
        wa[j] = column8(w + (size_t)(32 * s + 8 * g) * p.r + rank, p.r);
      else
        wa[j] = *reinterpret_cast<const u32x4*>(w + (size_t)rank * p.C + 32 * s + 8 * g);
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int j = 0; j < RT; ++j) acc[m][j] = mfma16(wa[j], xa[m], acc[m][j]);
  }
  // the waves' sums, in wave order, 16 rows at a time
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    if (m) __syncthreads();
#pragma unroll
    for (int j = 0; j < RT; ++j)
      *reinterpret_cast<f32x4*>(&red[wave][l][16 * j + 4 * g]) = acc[m][j];
    __syncthreads();
    for (int i = threadIdx.x; i < 16 * R / 4; i += 64 * LORA_WAVES) {
      const int row = i / (R / 4), c = i % (R / 4) * 4;
      if (16 * m + row < tl.n && c < p.r) {
        f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < LORA_WAVES; ++k) {
          const f32x4 o = *reinterpret_cast<const f32x4*>(&red[k][row][c]);
#pragma unroll
          for (int q = 0; q < 4; ++q) v[q] += o[q];
        }
        *reinterpret_cast<f32x4*>(p.part + ((size_t)blockIdx.y * p.T + tl.p0 + 16 * m + row) * p.r +
                                  c) = v;
      }
    }
  }
}

struct LoraExpand {
  const float* part;          // [splits][T][r]
  const uint16_t *w;          // factor [NA, C, r], or [NA, r, C] (TRANS)
  const float* scale;         // [NA] or NULL
  const int32_t *offsets, *src_row;
  const uint16_t* y;          // [T, C] or NULL (zeros)
  uint16_t* out;              // [T, C] or NULL (only v_out is wanted); may be y
  float* v_out;               // [T, r] or NULL: the added parts
  int T, C, r, NA, splits, scale_v;   // scale_v: v_out holds s[a] v
};

// out[t(p)][c] = y + sum_j s[a] v[p][j] w[a][c][j].  A wave takes 64 columns of
// the tile's rows: its four MFMA tiles hold columns 16 g + 4 i + q of lane
// group g (tile i, register q), so a lane ends up with 16 consecutive columns
// of its row: 32-byte loads of y and stores of out, whole 128-byte lines per row.
template <int MT, int RT, bool TRANS>
__global__ void __launch_bounds__(64 * LORA_WAVES) lora_expand_kernel(const LoraExpand p) {
  constexpr int TM = 16 * MT, R = 16 * RT;
  constexpr int KP = 2 * R;                 // hi and lo parts (r of each, then zeros)
  __shared__ __align__(16) uint16_t vs[TM][KP + 8];
  const LoraTile tl = lora_tile<TM>(p.offsets, p.NA, p.T, blockIdx.x);
  if (tl.n <= 0) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int l = lane & 15, g = lane >> 4;
  const int c0 = (blockIdx.y * LORA_WAVES + wave) * 64 + 16 * g;     // the lane's columns
  if (tl.a >= p.NA) {                       // no adapter: the row as it is
    if (p.out && p.out != p.y && c0 < p.C) {
      for (int i = l; i < tl.n; i += 16) {
        const int t = lora_token(p.src_row, tl.p0 + i, p.T);
        if (t < 0) continue;
        const u32x4 zero = {0, 0, 0, 0};
        const size_t o = (size_t)t * p.C + c0;
#pragma unroll
        for (int q = 0; q < 2; ++q)
          reinterpret_cast<u32x4*>(p.out + o)[q] =
              p.y ? reinterpret_cast<const u32x4*>(p.y + o)[q] : zero;
      }
    }
    return;
  }
  const float sc = p.scale ? p.scale[tl.a] : 1.0f;
  for (int i = threadIdx.x; i < TM * R; i += 64 * LORA_WAVES) {
    const int row = i / R, j = i % R;
    float v = 0.0f;
    if (row < tl.n && j < p.r) {
      const float* src = p.part + (size_t)(tl.p0 + row) * p.r + j;
      for (int k = 0; k < p.splits; ++k) v += src[(size_t)k * p.T * p.r];
      if (p.v_out && blockIdx.y == 0)
        p.v_out[(size_t)(tl.p0 + row) * p.r + j] = p.scale_v ? v * sc : v;
      v *= sc;
    }
    const uint32_t hi = f32_to_bf16_bits(v);
    const uint32_t lo = f32_to_bf16_bits(v - bf16_bits_to_f32(hi));
    // the two halves stand r apart; the ranks from r on fill the row's end with zeros
    if (j < p.r) {
      vs[row][j] = (uint16_t)hi;
      vs[row][p.r + j] = (uint16_t)lo;
    } else {
      vs[row][p.r + j] = 0;
      vs[row][R + j] = 0;
    }
  }
  __syncthreads();
  if (!p.out) return;
  const uint16_t* w = p.w + (size_t)tl.a * p.r * p.C;
  f32x4 acc[MT][4] = {};
  const int ksteps = (2 * p.r + 31) / 32;
  for (int s = 0; s < ksteps; ++s) {
    int j = 32 * s + 8 * g;
    j = j < p.r ? j : j < 2 * p.r ? j - p.r : 0;       // past both halves v is zero
    u32x4 wa[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = min((blockIdx.y * LORA_WAVES + wave) * 64 + 16 * (l >> 2) + 4 * i + (l & 3),
                        p.C - 1);
      if constexpr (TRANS) wa[i] = column8(w + (size_t)j * p.C + c, p.C);
      else wa[i] = *reinterpret_cast<const u32x4*>(w + (size_t)c * p.r + j);
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const u32x4 va = *reinterpret_cast<const u32x4*>(&vs[16 * m + l][32 * s + 8 * g]);
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[m][i] = mfma16(wa[i], va, acc[m][i]);
    }
  }
  if (c0 >= p.C) return;
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    if (16 * m + l >= tl.n) continue;
    const int t = lora_token(p.src_row, tl.p0 + 16 * m + l, p.T);
    if (t < 0) continue;
    const size_t o = (size_t)t * p.C + c0;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      float v[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
      if (p.y) unpack_chunk(reinterpret_cast<const u32x4*>(p.y + o)[q], v, BF16());
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] += acc[m][2 * q + e / 4][e % 4];
      reinterpret_cast<u32x4*>(p.out + o)[q] = pack_chunk(v, BF16());
    }
  }
}

struct LoraWgrad {
  const float* u;             // [T, r] by position
  const uint16_t* x;          // [T, C]
  const float* scale;         // [NA] or NULL: factor of the result
  const int32_t *offsets, *src_row;
  float* out;                 // [NA, r, C], or [NA, C, r] (TRANS)
  int T, C, r, NA, accumulate;
};

// out[a][j][c] (+)= s[a] sum over a's rows p of u[p][j] x[t(p)][c] on float32
// matrix cores (v_mfma_f32_16x16x4: lane l holds rank or column l & 15 of row
// l >> 4).  A block owns 64 columns of one adapter; its waves take every fourth
// group of four rows and are added in order.
template <int RT, bool TRANS>
__global__ void __launch_bounds__(64 * LORA_WAVES) lora_wgrad_kernel(const LoraWgrad p) {
  __shared__ float red[LORA_WAVES][16][64 + 4];
  const int a = blockIdx.y;
  const int s = min(max(p.offsets[a], 0), p.T), e = min(max(p.offsets[a + 1], s), p.T);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int l = lane & 15, g = lane >> 4;
  const int c0 = blockIdx.x * 64;
  f32x4 acc[RT][4] = {};
  for (int p0 = s + 4 * wave; p0 < e; p0 += 4 * LORA_WAVES) {
    const int row = p0 + g;
    const int t = row < e ? lora_token(p.src_row, row, p.T) : -1;
    float xv[4], uv[RT];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = c0 + 16 * i + l;
      xv[i] = t >= 0 && c < p.C ? bf16_bits_to_f32(p.x[(size_t)t * p.C + c]) : 0.0f;
    }
#pragma unroll
    for (int j = 0; j < RT; ++j)
      uv[j] = t >= 0 && 16 * j + l < p.r ? p.u[(size_t)row * p.r + 16 * j + l] : 0.0f;
#pragma unroll
    for (int j = 0; j < RT; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        acc[j][i] = __builtin_amdgcn_mfma_f32_16x16x4f32(uv[j], xv[i], acc[j][i], 0, 0, 0);
  }
  const float sc = p.scale ? p.scale[a] : 1.0f;
  float* out = p.out + (size_t)a * p.r * p.C;
#pragma unroll
  for (int j = 0; j < RT; ++j) {
    if (j) __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) red[wave][4 * g + q][16 * i + l] = acc[j][i][q];
    __syncthreads();
    for (int i = threadIdx.x; i < 16 * 64; i += 64 * LORA_WAVES) {
      const int rr = TRANS ? i % 16 : i / 64, cc = TRANS ? i / 16 : i % 64;
      const int rank = 16 * j + rr, c = c0 + cc;
      if (rank < p.r && c < p.C) {
        float v = 0.0f;
#pragma unroll
        for (int k = 0; k < LORA_WAVES; ++k) v += red[k][rr][cc];
        v *= sc;
        float* o = out + (TRANS ? (size_t)c * p.r + rank : (size_t)rank * p.C + c);
        *o = p.accumulate ? *o + v : v;
      }
    }
  }
}

// Rows per tile: 64 where the adapters average that many rows (a factor's tile
// is then read once for 64 rows), else 16.
static int lora_mt(int T, int NA) { return T >= 64 * NA ? 4 : 1; }
static int lora_tiles(int T, int NA, int mt) { return T / (16 * mt) + std::min(NA + 1, T) + 1; }

// Blocks along a reduction of `steps` steps: enough tiles x splits to fill the
// card twice, with at least two steps per wave.
static int lora_splits(int T, int NA, int mt, int steps) {
  const int tiles = std::max(1, T / (16 * mt) + (mt == 1 ? std::min(NA, T) / 2 : 0));
  return std::max(1, std::min({512 / tiles, steps / (2 * LORA_WAVES), 16}));
}

template <bool TRANS>
static moe_status_t launch_shrink(const LoraShrink& p, int mt, int splits, hipStream_t s) {
  const dim3 grid(lora_tiles(p.T, p.NA, mt), splits);
#define LORA_CASE(RR)                                                                            \
  case RR:                                                                                       \
    if (mt == 4) hipLaunchKernelGGL((lora_shrink_kernel<4, RR, TRANS>), grid, dim3(256), 0, s, p); \
    else hipLaunchKernelGGL((lora_shrink_kernel<1, RR, TRANS>), grid, dim3(256), 0, s, p);       \
    break;
  switch ((p.r + 15) / 16) {
    LORA_CASE(1) LORA_CASE(2) LORA_CASE(3) LORA_CASE(4)
    LORA_CASE(5) LORA_CASE(6) LORA_CASE(7) LORA_CASE(8)
  }
#undef LORA_CASE
  return launch_status();
}

template <bool TRANS>
static moe_status_t launch_expand(const LoraExpand& p, int mt, hipStream_t s) {
  const int cols = 64 * LORA_WAVES;
  const dim3 grid(lora_tiles(p.T, p.NA, mt), p.out ? (p.C + cols - 1) / cols : 1);
#define LORA_CASE(RR)                                                                            \
  case RR:                                                                                       \
    if (mt == 4) hipLaunchKernelGGL((lora_expand_kernel<4, RR, TRANS>), grid, dim3(256), 0, s, p); \
    else hipLaunchKernelGGL((lora_expand_kernel<1, RR, TRANS>), grid, dim3(256), 0, s, p);       \
    break;
  switch ((p.r + 15) / 16) {
    LORA_CASE(1) LORA_CASE(2) LORA_CASE(3) LORA_CASE(4)
    LORA_CASE(5) LORA_CASE(6) LORA_CASE(7) LORA_CASE(8)
  }
#undef LORA_CASE
  return launch_status();
}

template <bool TRANS>
static moe_status_t launch_wgrad(const LoraWgrad& p, hipStream_t s) {
  const dim3 grid((p.C + 63) / 64, p.NA);
#define LORA_CASE(RR)                                                                    \
  case RR:                                                                               \
    hipLaunchKernelGGL((lora_wgrad_kernel<RR, TRANS>), grid, dim3(256), 0, s, p);        \
    break;
  switch ((p.r + 15) / 16) {
    LORA_CASE(1) LORA_CASE(2) LORA_CASE(3) LORA_CASE(4)
    LORA_CASE(5) LORA_CASE(6) LORA_CASE(7) LORA_CASE(8)
  }
#undef LORA_CASE
  return launch_status();
}

static bool lora_sizes_ok(int T, int K, int N, int r, int NA) {
  return T >= 0 && K > 0 && N > 0 && K % 32 == 0 && N % 32 == 0 && r > 0 && r % 8 == 0 &&
         NA >= 1 && NA < MOE_MAX_EXPERTS;
}

}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_lora_workspace_size(int T, int K, int N, int r, int NA) {
  if (!lora_sizes_ok(T, K, N, r, NA) || T == 0) return 256;
  const int mt = lora_mt(T, NA);
  // the partial sums of the reduction with more splits, and the backward's u
  const int splits = std::max(lora_splits(T, NA, mt, K / 32), lora_splits(T, NA, mt, N / 32));
  return ((size_t)(splits + 1) * T * r * sizeof(float) + 255) / 256 * 256;
}

moe_status_t moe_lora_fwd(const moe_lora_fwd_args_t* a, void* stream) {
  MOE_CHECK_ARG(a && a->struct_size >= sizeof(moe_lora_fwd_args_t));
  MOE_CHECK_ARG(lora_sizes_ok(a->T, a->K, a->N, a->r, a->NA));
  if (a->dtype != MOE_BF16) return valid_dtype(a->dtype) ? MOE_ERR_UNSUPPORTED : MOE_ERR_INVALID_ARG;
  if (a->r > LORA_MAX_RANK) return MOE_ERR_UNSUPPORTED;
  if (a->T == 0) return MOE_OK;
  MOE_CHECK_ARG(a->x && a->A && a->B && a->y && a->out && a->offsets);
  MOE_CHECK_ARG(aligned16(a->x) && aligned16(a->A) && aligned16(a->B) && aligned16(a->y) &&
                aligned16(a->out) && aligned16(a->v_out) && aligned16(a->ws));
  if (!a->ws || a->ws_bytes < moe_lora_workspace_size(a->T, a->K, a->N, a->r, a->NA))
    return MOE_ERR_WORKSPACE;
  const size_t ny = (size_t)a->T * a->N * 2, nx = (size_t)a->T * a->K * 2, nt = (size_t)a->T * 4;
  const size_t nw = (size_t)a->NA * a->r * 2;
  MOE_CHECK_ARG(same_or_apart(a->out, a->y, ny));
  MOE_CHECK_ARG(outputs_apart({{a->out, ny}, {a->v_out, nt * a->r}, {a->ws, a->ws_bytes}},
                              {{a->x, nx}, {a->A, nw * a->K}, {a->B, nw * a->N},
                               {a->scale, (size_t)a->NA * 4}, {a->src_row, nt},
                               {a->offsets, (size_t)(a->NA + 1) * 4}}) &&
                outputs_apart({{a->v_out, nt * a->r}, {a->ws, a->ws_bytes}}, {{a->y, ny}}));
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const int mt = lora_mt(a->T, a->NA), splits = lora_splits(a->T, a->NA, mt, a->K / 32);
  float* part = static_cast<float*>(a->ws);
  const LoraShrink sh = {static_cast<const uint16_t*>(a->x), static_cast<const uint16_t*>(a->A),
                         a->offsets, a->src_row, part, a->T, a->K, a->r, a->NA, a->K / 32};
  moe_status_t st = launch_shrink<false>(sh, mt, splits, s);
  if (st != MOE_OK) return st;
  const LoraExpand ex = {part, static_cast<const uint16_t*>(a->B), a->scale, a->offsets, a->src_row,
                         static_cast<const uint16_t*>(a->y), static_cast<uint16_t*>(a->out),
                         a->v_out, a->T, a->N, a->r, a->NA, splits, 0};
  return launch_expand<false>(ex, mt, s);
}

moe_status_t moe_lora_bwd(const moe_lora_bwd_args_t* a, void* stream) {
  MOE_CHECK_ARG(a && a->struct_size >= sizeof(moe_lora_bwd_args_t));
  MOE_CHECK_ARG(lora_sizes_ok(a->T, a->K, a->N, a->r, a->NA));
  if (a->dtype != MOE_BF16) return valid_dtype(a->dtype) ? MOE_ERR_UNSUPPORTED : MOE_ERR_INVALID_ARG;
  if (a->r > LORA_MAX_RANK) return MOE_ERR_UNSUPPORTED;
  if (a->T == 0 && !a->dA && !a->dB) return MOE_OK;
  MOE_CHECK_ARG(a->dx_out || a->dA || a->dB);
  MOE_CHECK_ARG(a->offsets && (a->dx_out || !a->dx));
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const size_t nx = (size_t)a->T * a->K * 2;
  float *part = nullptr, *u = nullptr;
  const bool want_u = a->dx_out || a->dA;
  if (a->T > 0) {
    MOE_CHECK_ARG(a->dy && (!want_u || a->B) && (!a->dx_out || a->A) && (!a->dA || a->x) &&
                  (!a->dB || a->v));
    MOE_CHECK_ARG(aligned16(a->x) && aligned16(a->dy) && aligned16(a->A) && aligned16(a->B) &&
                  aligned16(a->v) && aligned16(a->dx) && aligned16(a->dx_out) &&
                  aligned16(a->dA) && aligned16(a->dB) && aligned16(a->ws));
    if (!a->ws || a->ws_bytes < moe_lora_workspace_size(a->T, a->K, a->N, a->r, a->NA))
      return MOE_ERR_WORKSPACE;
    const size_t ny = (size_t)a->T * a->N * 2, nt = (size_t)a->T * 4, nw = (size_t)a->NA * a->r * 2;
    MOE_CHECK_ARG(same_or_apart(a->dx_out, a->dx, nx));
    MOE_CHECK_ARG(outputs_apart({{a->dx_out, nx}, {a->dA, 2 * nw * a->K}, {a->dB, 2 * nw * a->N},
                                 {a->ws, a->ws_bytes}},
                                {{a->x, nx}, {a->dy, ny}, {a->A, nw * a->K}, {a->B, nw * a->N},
                                 {a->v, nt * a->r}, {a->scale, (size_t)a->NA * 4},
                                 {a->src_row, nt}, {a->offsets, (size_t)(a->NA + 1) * 4}}) &&
                  outputs_apart({{a->dA, 2 * nw * a->K}, {a->dB, 2 * nw * a->N},
                                 {a->ws, a->ws_bytes}}, {{a->dx, nx}}));
    if (want_u) {
      const int mt = lora_mt(a->T, a->NA), splits = lora_splits(a->T, a->NA, mt, a->N / 32);
      u = static_cast<float*>(a->ws);
      part = u + (size_t)a->T * a->r;
      const LoraShrink sh = {static_cast<const uint16_t*>(a->dy),
                             static_cast<const uint16_t*>(a->B), a->offsets, a->src_row, part,
                             a->T, a->N, a->r, a->NA, a->N / 32};
      moe_status_t st = launch_shrink<true>(sh, mt, splits, s);
      if (st != MOE_OK) return st;
      const LoraExpand ex = {part, static_cast<const uint16_t*>(a->A), a->scale, a->offsets,
                             a->src_row, static_cast<const uint16_t*>(a->dx),
                             static_cast<uint16_t*>(a->dx_out), a->dA ? u : nullptr, a->T, a->K,
                             a->r, a->NA, splits, 1};
      st = launch_expand<true>(ex, mt, s);
      if (st != MOE_OK) return st;
    }
  }
  if (a->dA) {
    const LoraWgrad w = {u, static_cast<const uint16_t*>(a->x), nullptr, a->offsets, a->src_row,
                         a->dA, a->T, a->K, a->r, a->NA, a->accumulate};
    const moe_status_t st = launch_wgrad<false>(w, s);
    if (st != MOE_OK) return st;
  }
  if (a->dB) {
    const LoraWgrad w = {a->v, static_cast<const uint16_t*>(a->dy), a->scale, a->offsets,
                         a->src_row, a->dB, a->T, a->N, a->r, a->NA, a->accumulate};
    return launch_wgrad<true>(w, s);
  }
  return MOE_OK;
}

}  // extern "C"
