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
#include <type_traits>

namespace moe {

static constexpr int LORA_MAX_RANK = 128;
static constexpr int LORA_WAVES = 4;

// A tile of at most `tm` rows of one adapter's segment (adapter NA: the rows
// behind the last segment), or n == -1 past the last tile.
struct LoraTile {
  int a, p0, n;
  int s0, rows;    // the whole segment
};

// Tile i of the segments, each cut into tiles of tm rows; EMPTY: an adapter
// without rows has one tile of none.  Called by whole waves; the lanes take one
// segment each, 64 at a time.
template <bool EMPTY>
__device__ __forceinline__ LoraTile lora_tile(const int32_t* offsets, int NA, int T, int tm, int i) {
  const int lane = threadIdx.x & 63;
  int before = 0;
  for (int base = 0; base <= NA; base += 64) {
    const int a = base + lane;
    int s = T, e = T;
    if (a <= NA) {
      s = min(max(offsets[a], 0), T);
      e = a < NA ? min(max(offsets[a + 1], s), T) : T;
    }
    int nt = (e - s + tm - 1) / tm;
    if (EMPTY && a < NA && nt == 0) nt = 1;
    int incl = nt;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int v = __shfl_up(incl, o, 64);
      if (lane >= o) incl += v;
    }
    const uint64_t hit = __ballot(before + incl > i);
    if (hit) {
      const int l = __ffsll((unsigned long long)hit) - 1;
      const int first = before + __builtin_amdgcn_readlane(incl - nt, l);
      const int s0 = __builtin_amdgcn_readlane(s, l), e0 = __builtin_amdgcn_readlane(e, l);
      const int p0 = s0 + (i - first) * tm;
      return {base + l, p0, min(tm, e0 - p0), s0, e0 - s0};
    }
    before += __builtin_amdgcn_readlane(incl, 63);
  }
  return {0, 0, -1, 0, 0};
}

__device__ __forceinline__ int lora_token(const int32_t* src_row, int p, int T) {
  const int t = src_row ? src_row[p] : p;
  return (unsigned)t < (unsigned)T ? t : -1;
}

__device__ __forceinline__ f32x4 mfma16(const u32x4& a, const u32x4& b, const f32x4& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                 __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// v as bf16 bits, to nearest even.
__device__ __forceinline__ uint32_t bf16_of(float v) {
  return __builtin_bit_cast(uint16_t, (__bf16)v);
}

// What bf16 bits b leave of v (nothing of an infinity).
__device__ __forceinline__ float rest_of(float v, uint32_t b) {
  const float h = bf16_bits_to_f32(b);
  return h == v ? 0.0f : v - h;
}

// The 4 x 16 block that a group of 16 lanes reads with ds_read_b64_tr_b16: lane
// 4 q + r addresses four elements of row q, lane i receives rows 0 .. 3 of
// element i & 3 of the segment that lanes r = i >> 2 address.
__device__ __forceinline__ u32x2 read_tr(const uint16_t* p) {
  typedef short i16x4 __attribute__((ext_vector_type(4)));
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                       (__attribute__((address_space(3))) i16x4*)(p)));
}
// LDS written by other lanes of the wave is read next (one wave's LDS accesses
// stay in order; this keeps the compiler from reordering them).
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
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
  constexpr int U = RT <= 2 ? 4 : 2;        // steps whose loads are in flight together
  __shared__ float red[LORA_WAVES][16][R + 4];
  const LoraTile tl = lora_tile<false>(p.offsets, p.NA, p.T, TM, blockIdx.x);
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
  auto load = [&](int s, u32x4 (&xa)[MT], u32x4 (&wa)[RT]) {
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
  };
  auto mma = [&](const u32x4 (&xa)[MT], const u32x4 (&wa)[RT]) {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int j = 0; j < RT; ++j) acc[m][j] = mfma16(wa[j], xa[m], acc[m][j]);
  };
  int s = s0;
  for (; s + U <= s1; s += U) {
    u32x4 xa[U][MT], wa[U][RT];
#pragma unroll
    for (int k = 0; k < U; ++k) load(s + k, xa[k], wa[k]);
#pragma unroll
    for (int k = 0; k < U; ++k) mma(xa[k], wa[k]);
  }
  for (; s < s1; ++s) {
    u32x4 xa[MT], wa[RT];
    load(s, xa, wa);
    mma(xa, wa);
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

// out[t(p)][c] = y + sum_j s[a] v[p][j] w[a][c][j].  A wave takes chunks of 64
// columns of the tile's rows, the next chunk's y loaded meanwhile: its four MFMA
// tiles hold columns 16 g + 4 i + q of lane group g (tile i, register q), so a
// lane ends up with 16 consecutive columns of its row: 32-byte loads of y and
// stores of out, whole 128-byte lines per row.  A factor stored the other way
// (TRANS) passes through LDS and is read transposed.
template <int MT, int RT, bool TRANS>
__global__ void __launch_bounds__(64 * LORA_WAVES) lora_expand_kernel(const LoraExpand p) {
  constexpr int TM = 16 * MT, R = 16 * RT;
  constexpr int KP = 2 * R;                 // hi and lo parts (r of each, then zeros)
  constexpr int WS = 64 + 8;                // row stride of a wave's factor tile
  __shared__ __align__(16) uint16_t vs[TM][KP + 8];
  __shared__ __align__(16) uint16_t wt[TRANS ? LORA_WAVES : 1][TRANS ? R : 1][WS];
  const LoraTile tl = lora_tile<false>(p.offsets, p.NA, p.T, TM, blockIdx.x);
  if (tl.n <= 0) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int l = lane & 15, g = lane >> 4;
  const int chunks = (p.C + 63) / 64, step = gridDim.y * LORA_WAVES;
  int ch = blockIdx.y * LORA_WAVES + wave;
  const u32x4 zero = {0, 0, 0, 0};
  if (tl.a >= p.NA) {                       // no adapter: the rows as they are
    if (!p.out || p.out == p.y) return;
    for (; ch < chunks; ch += step) {
      const int c = 64 * ch + 8 * (lane & 7);
      for (int i = lane >> 3; i < tl.n; i += 8) {
        const int t = lora_token(p.src_row, tl.p0 + i, p.T);
        if (t < 0 || c >= p.C) continue;
        const size_t o = (size_t)t * p.C + c;
        *reinterpret_cast<u32x4*>(p.out + o) =
            p.y ? *reinterpret_cast<const u32x4*>(p.y + o) : zero;
      }
    }
    return;
  }
  int t[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
    t[m] = 16 * m + l < tl.n ? lora_token(p.src_row, tl.p0 + 16 * m + l, p.T) : -1;
  u32x4 yr[MT][2];
  auto fetch = [&](int chunk) {
    const int c = 64 * chunk + 16 * g;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int q = 0; q < 2; ++q)
        yr[m][q] = p.y && p.out && t[m] >= 0 && c < p.C
                       ? reinterpret_cast<const u32x4*>(p.y + (size_t)t[m] * p.C + c)[q]
                       : zero;
  };
  fetch(ch);
  // the tile's ranks: the splits' parts added in order, four loads in flight
  const float sc = p.scale ? p.scale[tl.a] : 1.0f;
  const int quads = p.r / 4;
  for (int i = threadIdx.x; i < TM * quads; i += 64 * LORA_WAVES) {
    const int row = i / quads, j = (i - row * quads) * 4;
    f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
    if (row < tl.n) {
      const float* src = p.part + (size_t)(tl.p0 + row) * p.r + j;
      const size_t ld = (size_t)p.T * p.r;
      int k = 0;
      for (; k + 4 <= p.splits; k += 4) {
        f32x4 o[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) o[q] = *reinterpret_cast<const f32x4*>(src + (k + q) * ld);
#pragma unroll
        for (int q = 0; q < 4; ++q) v += o[q];
      }
      for (; k < p.splits; ++k) v += *reinterpret_cast<const f32x4*>(src + k * ld);
      const f32x4 sv = v * sc;
      if (p.v_out && blockIdx.y == 0)
        *reinterpret_cast<f32x4*>(p.v_out + (size_t)(tl.p0 + row) * p.r + j) = p.scale_v ? sv : v;
      v = sv;
    }
    u32x2 hi, lo;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const uint32_t h0 = bf16_of(v[2 * q]), h1 = bf16_of(v[2 * q + 1]);
      hi[q] = h0 | h1 << 16;
      lo[q] = bf16_of(rest_of(v[2 * q], h0)) | bf16_of(rest_of(v[2 * q + 1], h1)) << 16;
    }
    *reinterpret_cast<u32x2*>(&vs[row][j]) = hi;
    *reinterpret_cast<u32x2*>(&vs[row][p.r + j]) = lo;
  }
  // zeros behind the two parts
  const int tail = (KP - 2 * p.r) / 8;
  for (int i = threadIdx.x; i < TM * tail; i += 64 * LORA_WAVES)
    *reinterpret_cast<u32x4*>(&vs[i / tail][2 * p.r + 8 * (i % tail)]) = zero;
  __syncthreads();
  if (!p.out) return;
  const uint16_t* w = p.w + (size_t)tl.a * p.r * p.C;
  const int ksteps = (2 * p.r + 31) / 32;
  for (; ch < chunks; ch += step) {
    u32x4 yc[MT][2];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int q = 0; q < 2; ++q) yc[m][q] = yr[m][q];
    if (ch + step < chunks) fetch(ch + step);
    if constexpr (TRANS) {
      // eight rows of 128 bytes per instruction
      u32x4 raw[2 * RT];
      const int c = min(64 * ch + 8 * (lane & 7), p.C - 8);
#pragma unroll
      for (int i = 0; i < 2 * RT; ++i)
        raw[i] = *reinterpret_cast<const u32x4*>(
            w + (size_t)min(8 * i + (lane >> 3), p.r - 1) * p.C + c);
      wave_fence();
#pragma unroll
      for (int i = 0; i < 2 * RT; ++i)
        *reinterpret_cast<u32x4*>(&wt[wave][8 * i + (lane >> 3)][8 * (lane & 7)]) = raw[i];
      wave_fence();
    }
    f32x4 acc[MT][4] = {};
    for (int s = 0; s < ksteps; ++s) {
      int j = 32 * s + 8 * g;
      j = j < p.r ? j : j < 2 * p.r ? j - p.r : 0;       // past both halves v is zero
      u32x4 wa[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (TRANS) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const u32x2 v = read_tr(&wt[wave][j + 4 * h + (l >> 2)][16 * (l & 3) + 4 * i]);
            wa[i][2 * h] = v[0];
            wa[i][2 * h + 1] = v[1];
          }
        } else {
          const int c = min(64 * ch + 16 * (l >> 2) + 4 * i + (l & 3), p.C - 1);
          wa[i] = *reinterpret_cast<const u32x4*>(w + (size_t)c * p.r + j);
        }
      }
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const u32x4 va = *reinterpret_cast<const u32x4*>(&vs[16 * m + l][32 * s + 8 * g]);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[m][i] = mfma16(wa[i], va, acc[m][i]);
      }
    }
    const int c = 64 * ch + 16 * g;
    if (c >= p.C) continue;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      if (t[m] < 0) continue;
      const size_t o = (size_t)t[m] * p.C + c;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        typedef float f32x8 __attribute__((ext_vector_type(8)));
        float v[8];
        unpack_chunk(yc[m][q], v, BF16());
        f32x8 f;
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = v[e] + acc[m][2 * q + e / 4][e % 4];
        reinterpret_cast<u32x4*>(p.out + o)[q] =
            __builtin_bit_cast(u32x4, __builtin_convertvector(f, bf16x8));
      }
    }
  }
}

// One weight gradient: out[a][j][c] (dA), or out[a][c][j] (dB: trans), is s[a] times
// the sum over a's rows p of u[p][j] x[t(p)][c].
struct LoraGrad {
  const float* u;             // [T, r] by position
  const uint16_t* x;          // [T, C]
  const float* scale;         // [NA] or NULL
  float* out;                 // NULL: not wanted
  float* part;                // [slots][r][C]: sums of segments longer than a chunk
  int C, trans;
};
struct LoraWgrad {
  LoraGrad g[2];
  const int32_t *offsets, *src_row;
  int T, r, NA, chunk, accumulate;
};

// Where a chunk of a longer segment keeps its sum.  Chunks of `chunk` rows: two
// first chunks never start within the same `chunk` rows, nor two later ones.
__device__ __forceinline__ int lora_slot(int p0, int segment, int chunk) {
  return 2 * (p0 / chunk) + (p0 == segment);
}

// A block sums one chunk of a segment for 64 columns; its waves take 32 rows at a
// time.  The rows pass through LDS (a wave's own 32 x 64 tile, whole lines in,
// read transposed: the reduction runs over rows), u is split into three bf16
// parts, which hold its 24 bits, so the float32 sums are of float32 accuracy
// at three bf16 MFMAs a step: 830 TFLOP/s of the bf16 rate against 157 of
// v_mfma_f32.
template <int RT>
__global__ void __launch_bounds__(64 * LORA_WAVES) lora_wgrad_kernel(const LoraWgrad p) {
  constexpr int XS = 64 + 8;
  __shared__ __align__(16) uint16_t xs[LORA_WAVES][32][XS];
  __shared__ float red[LORA_WAVES][16][64 + 4];
  const LoraGrad& G = p.g[blockIdx.z];
  const int c0 = blockIdx.y * 64;
  if (!G.out || c0 >= G.C) return;
  const LoraTile tl = lora_tile<true>(p.offsets, p.NA, p.T, p.chunk, blockIdx.x);
  if (tl.n < 0 || tl.a >= p.NA) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int l = lane & 15, g = lane >> 4;
  const int xc = min(c0 + 8 * (lane & 7), G.C - 8);       // (C a multiple of 32)
  // the tokens of 32 rows, one a lane (both halves of the wave alike)
  auto tokens = [&](int s) {
    const int i = 32 * s + (lane & 31);
    return i < tl.n ? lora_token(p.src_row, tl.p0 + i, p.T) : -1;
  };
  const u32x4 zero = {0, 0, 0, 0};
  auto fetch = [&](int tok, u32x4 (&x)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = __shfl(tok, 8 * i + (lane >> 3), 64);
      x[i] = t >= 0 ? *reinterpret_cast<const u32x4*>(G.x + (size_t)t * G.C + xc) : zero;
    }
  };
  f32x4 acc[RT][4] = {};
  const int steps = (tl.n + 31) / 32;
  int tok = tokens(wave);
  u32x4 x[4];
  fetch(tok, x);
  int next = tokens(wave + LORA_WAVES);
  for (int s = wave; s < steps; s += LORA_WAVES) {
    const uint32_t valid = (uint32_t)__ballot(tok >= 0);
    wave_fence();
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<u32x4*>(&xs[wave][8 * i + (lane >> 3)][8 * (lane & 7)]) = x[i];
    wave_fence();
    tok = next;
    fetch(tok, x);
    next = tokens(s + 2 * LORA_WAVES);
    u32x4 xa[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const u32x2 v = read_tr(&xs[wave][8 * g + 4 * h + (l >> 2)][16 * i + 4 * (l & 3)]);
        xa[i][2 * h] = v[0];
        xa[i][2 * h + 1] = v[1];
      }
    const float* u = G.u + (size_t)(tl.p0 + 32 * s + 8 * g) * p.r;
#pragma unroll
    for (int j = 0; j < RT; ++j) {
      const int rank = 16 * j + l;
      u32x4 part[3];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint32_t b[3][2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int row = 2 * q + e;
          float v = rank < p.r && (valid >> (8 * g + row) & 1) ? u[(size_t)row * p.r + rank] : 0.0f;
#pragma unroll
          for (int k = 0; k < 3; ++k) {
            b[k][e] = bf16_of(v);
            v = rest_of(v, b[k][e]);
          }
        }
#pragma unroll
        for (int k = 0; k < 3; ++k) part[k][q] = b[k][0] | b[k][1] << 16;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int k = 0; k < 3; ++k) acc[j][i] = mfma16(part[k], xa[i], acc[j][i]);
    }
  }
  // the waves in order, 16 ranks at a time
  const bool whole = tl.rows <= p.chunk;
  const float sc = whole && G.scale ? G.scale[tl.a] : 1.0f;
  float* out = whole ? G.out + (size_t)tl.a * p.r * G.C
                     : G.part + (size_t)lora_slot(tl.p0, tl.s0, p.chunk) * p.r * G.C;
  const bool add = whole && p.accumulate;
#pragma unroll
  for (int j = 0; j < RT; ++j) {
    if (j) __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) red[wave][4 * g + q][16 * i + l] = acc[j][i][q];
    __syncthreads();
    for (int i = threadIdx.x; i < 16 * 64; i += 64 * LORA_WAVES) {
      const int rr = G.trans ? i % 16 : i / 64, cc = G.trans ? i / 16 : i % 64;
      const int rank = 16 * j + rr, c = c0 + cc;
      if (rank < p.r && c < G.C) {
        float v = 0.0f;
#pragma unroll
        for (int k = 0; k < LORA_WAVES; ++k) v += red[k][rr][cc];
        v *= sc;
        float* o = out + (G.trans ? (size_t)c * p.r + rank : (size_t)rank * G.C + c);
        *o = add ? *o + v : v;
      }
    }
  }
}

// Adds the chunks of the segments that have several, in order.
__global__ void __launch_bounds__(256) lora_wgrad_sum_kernel(const LoraWgrad p) {
  const LoraGrad& G = p.g[blockIdx.z];
  const int a = blockIdx.y;
  const int s = min(max(p.offsets[a], 0), p.T), e = min(max(p.offsets[a + 1], s), p.T);
  const size_t n = (size_t)p.r * G.C, i = ((size_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (!G.out || e - s <= p.chunk || i >= n) return;
  f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int p0 = s; p0 < e; p0 += p.chunk)
    v += *reinterpret_cast<const f32x4*>(G.part + lora_slot(p0, s, p.chunk) * n + i);
  if (G.scale) v *= G.scale[a];
  f32x4* o = reinterpret_cast<f32x4*>(G.out + a * n + i);
  *o = p.accumulate ? *o + v : v;
}

// Row tiles of 16, 32 or 64: the highest that the adapters fill on average and
// that still gives 96 tiles (a factor's tile is read once per tile of rows,
// while few tiles leave the card empty or cost splits of the reduction).
static int lora_mt(int T, int NA) {
  for (int mt = 4; mt > 1; mt /= 2)
    if (T >= 16 * mt * std::max(NA, 96)) return mt;
  return 1;
}
static int lora_tiles(int T, int NA, int mt) { return T / (16 * mt) + std::min(NA + 1, T) + 1; }

// Blocks along a reduction of `steps` steps: enough tiles x splits to fill the
// card twice, with at least two steps per wave.
static int lora_splits(int T, int NA, int mt, int steps) {
  const int tiles = std::max(1, T / (16 * mt) + (mt == 1 ? std::min(NA, T) / 2 : 0));
  return std::max(1, std::min({512 / tiles, steps / (2 * LORA_WAVES), 16}));
}

// Calls f(RT) for the rank tiles that cover r (1, 2, 3, 4, 6 or 8 of 16).
template <class F>
static moe_status_t lora_ranks(int r, F&& f) {
  switch ((r + 15) / 16) {
    case 1: f(std::integral_constant<int, 1>()); break;
    case 2: f(std::integral_constant<int, 2>()); break;
    case 3: f(std::integral_constant<int, 3>()); break;
    case 4: f(std::integral_constant<int, 4>()); break;
    case 5:
    case 6: f(std::integral_constant<int, 6>()); break;
    default: f(std::integral_constant<int, 8>()); break;
  }
  return launch_status();
}

template <bool TRANS>
static moe_status_t launch_shrink(const LoraShrink& p, int mt, int splits, hipStream_t s) {
  const dim3 grid(lora_tiles(p.T, p.NA, mt), splits), block(64 * LORA_WAVES);
  return lora_ranks(p.r, [&](auto N) {
    constexpr int RT = decltype(N)::value;
    if (mt == 4) hipLaunchKernelGGL((lora_shrink_kernel<4, RT, TRANS>), grid, block, 0, s, p);
    else if (mt == 2) hipLaunchKernelGGL((lora_shrink_kernel<2, RT, TRANS>), grid, block, 0, s, p);
    else hipLaunchKernelGGL((lora_shrink_kernel<1, RT, TRANS>), grid, block, 0, s, p);
  });
}

template <bool TRANS>
static moe_status_t launch_expand(const LoraExpand& p, int mt, hipStream_t s) {
  // blocks along the columns: one per 256 columns, fewer (each then walks several
  // chunks and reads the tile's ranks once) as long as 1024 blocks remain
  const int tiles = lora_tiles(p.T, p.NA, mt), cols = (p.C + 64 * LORA_WAVES - 1) / (64 * LORA_WAVES);
  const int by = p.out ? std::min(cols, std::max(1, (1024 + tiles - 1) / tiles)) : 1;
  const dim3 grid(tiles, by), block(64 * LORA_WAVES);
  return lora_ranks(p.r, [&](auto N) {
    constexpr int RT = decltype(N)::value;
    if (mt == 4) hipLaunchKernelGGL((lora_expand_kernel<4, RT, TRANS>), grid, block, 0, s, p);
    else if (mt == 2) hipLaunchKernelGGL((lora_expand_kernel<2, RT, TRANS>), grid, block, 0, s, p);
    else hipLaunchKernelGGL((lora_expand_kernel<1, RT, TRANS>), grid, block, 0, s, p);
  });
}

// Rows that a block of the weight gradients sums: an eighth of the batch, at
// least 1024, so that a batch of one adapter still fills the card.
static int lora_chunk(int T) { return std::max(1024, (T + 7) / 8); }
static size_t lora_slots(int T) {
  return T > lora_chunk(T) ? 2 * ((size_t)T / lora_chunk(T) + 1) : 0;
}

static moe_status_t launch_wgrad(const LoraWgrad& p, hipStream_t s) {
  const int wide = std::max(p.g[0].out ? p.g[0].C : 0, p.g[1].out ? p.g[1].C : 0);
  const dim3 grid(p.T / p.chunk + p.NA + 1, (wide + 63) / 64, 2), block(64 * LORA_WAVES);
  const moe_status_t st = lora_ranks(p.r, [&](auto N) {
    hipLaunchKernelGGL((lora_wgrad_kernel<decltype(N)::value>), grid, block, 0, s, p);
  });
  if (st != MOE_OK || p.T <= p.chunk) return st;
  const size_t quads = (size_t)p.r * wide / 4;
  hipLaunchKernelGGL(lora_wgrad_sum_kernel, dim3((unsigned)((quads + 255) / 256), p.NA, 2),
                     dim3(256), 0, s, p);
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
  // the backward's u, and the partial sums of the reduction with more splits or
  // (once those are used up) of the weight gradients' chunks
  const int splits = std::max(lora_splits(T, NA, mt, K / 32), lora_splits(T, NA, mt, N / 32));
  const size_t parts = std::max((size_t)splits * T * r, lora_slots(T) * r * ((size_t)K + N));
  return (((size_t)T * r + parts) * sizeof(float) + 255) / 256 * 256;
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
  float* u = static_cast<float*>(a->ws);
  float* part = u + (a->T > 0 ? (size_t)a->T * a->r : 0);
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
  if (!a->dA && !a->dB) return MOE_OK;
  const int chunk = lora_chunk(a->T);
  const LoraWgrad w = {
      {{u, static_cast<const uint16_t*>(a->x), nullptr, a->dA, part, a->K, 0},
       {a->v, static_cast<const uint16_t*>(a->dy), a->scale, a->dB,
        part + lora_slots(a->T) * a->r * a->K, a->N, 1}},
      a->offsets, a->src_row, a->T, a->r, a->NA, chunk, a->accumulate};
  return launch_wgrad(w, s);
}

}  // extern "C"
