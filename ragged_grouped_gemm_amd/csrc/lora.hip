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
// and `expand` (few rows) or `apply` (many) adds their products with the other
// factor to the wide rows.  The r values stay float32 between the two: in front
// of the bf16 matrix cores each is split into a high and a low bf16 part, which
// leave out at most 2^-16 of it (a float32 matrix instruction would run at a
// sixteenth of the rate).  Weight gradients are float32 throughout.
//
// Measured, as whole calls: 64 rows of 32 adapters, rank 16, 7168 x 7168: 11 us
// (two launches, each at the 5 us that its chain of dependent loads takes);
// 8192 rows of 16 adapters, rank 32, 7168 x 4096: 56 us, 4.5 TB/s of what must
// be moved; backward of 8192 rows of 8 adapters, rank 16, 4096 x 4096: 77 us,
// 3.4 TB/s.  A large copy on the same card reaches 4.9 TB/s.
#include "common.hpp"
#include "spans.hpp"

#include <math.h>
#include <stddef.h>

#include <algorithm>
#include <type_traits>

namespace moe {

static constexpr int LORA_MAX_RANK = 128;
static constexpr int LORA_WAVES = 4;
static constexpr int WGRAD_COLS = 64;     // columns of a block of the weight gradients

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

// v in three bf16 parts, which hold its 24 bits.
__device__ __forceinline__ void split3(float v, uint32_t& a, uint32_t& b, uint32_t& c) {
  a = bf16_of(v);
  v = rest_of(v, a);
  b = bf16_of(v);
  c = bf16_of(rest_of(v, b));
}

// Four values' high and low bf16 parts.
__device__ __forceinline__ void split_quad(const f32x4& v, u32x2& hi, u32x2& lo) {
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const uint32_t h0 = bf16_of(v[2 * q]), h1 = bf16_of(v[2 * q + 1]);
    hi[q] = h0 | h1 << 16;
    lo[q] = bf16_of(rest_of(v[2 * q], h0)) | bf16_of(rest_of(v[2 * q + 1], h1)) << 16;
  }
}

// Eight bf16 values plus eight float32 ones, rounded once.
__device__ __forceinline__ u32x4 add_chunk(const u32x4& y, const f32x4& a, const f32x4& b) {
  typedef float f32x8 __attribute__((ext_vector_type(8)));
  float v[8];
  unpack_chunk(y, v, BF16());
  f32x8 f;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    f[e] = v[e] + a[e];
    f[e + 4] = v[e + 4] + b[e];
  }
  return __builtin_bit_cast(u32x4, __builtin_convertvector(f, bf16x8));
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

struct LoraShrink {
  const uint16_t *x, *w;      // rows [T, C]; factor [NA, r, C], or [NA, C, r] (TRANS)
  const int32_t *offsets, *src_row;
  float* part;                // [splits][T][r], by position
  int T, C, r, NA, chunks, splits;    // chunks of KC along C
};

// part[split][p][j] = sum over the split's share of C of x[t(p)][c] w[a][j][c].
// The waves share the block's chunks of KC columns.  A wave stages its chunk of
// the rows and of the factor through LDS of its own: whole lines are loaded
// (KC / 8 lanes a row) while the chunk before is multiplied.  8192 x 7168 rows of
// rank 32: 27 us (3.9 TB/s; 36 us with MFMA fragments loaded straight from
// memory, 16 bytes from each of 16 rows at a time); what is left over the copy
// rate is the start of the blocks, three loads deep (offsets, source rows,
// rows), and their end.  MFMA: first operand the factor's
// rows (register 4 (lane >> 4) + q = rank), second the activation rows
// (lane & 15).  A factor whose reduction runs over its rows (TRANS) is read
// transposed.
template <int MT, int RT, bool TRANS>
__global__ void __launch_bounds__(64 * LORA_WAVES) lora_shrink_kernel(const LoraShrink p) {
  constexpr int TM = 16 * MT, R = 16 * RT;
  constexpr int KC = RT <= 4 ? 64 : 32;
  constexpr int LPR = KC / 8;                // lanes per row of a chunk
  constexpr int RPI = 64 / LPR;              // rows per load instruction
  constexpr int NX = TM / RPI, NW = R * KC / 512;   // load instructions per chunk
  constexpr int XS = KC + 8;                 // row strides in LDS, elements
  constexpr int WS = TRANS ? R + 8 : KC + 8, WROWS = TRANS ? KC : R;
  __shared__ __align__(16) uint16_t xs[LORA_WAVES][TM][XS];
  __shared__ __align__(16) uint16_t wt[LORA_WAVES][WROWS][WS];
  __shared__ __align__(16) float red[LORA_WAVES][16][16 + 4];
  const int split = blockIdx.x % p.splits;
  const LoraTile tl = lora_tile<false>(p.offsets, p.NA, p.T, TM, blockIdx.x / p.splits);
  if (tl.n <= 0 || tl.a >= p.NA) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int l = lane & 15, g = lane >> 4;
  const int lr = lane / LPR, lc = 8 * (lane % LPR);
  // rows past the tile read a valid row again, their results are dropped
  const uint16_t* xr[NX];
#pragma unroll
  for (int i = 0; i < NX; ++i) {
    const int t = lora_token(p.src_row, tl.p0 + min(RPI * i + lr, tl.n - 1), p.T);
    xr[i] = p.x + (size_t)max(t, 0) * p.C + lc;
  }
  const uint16_t* w = p.w + (size_t)tl.a * p.r * p.C;
  // TRANS: the factor's chunk is KC r consecutive elements, 16 bytes a lane and
  // instruction; where each lands
  int wo[NW], wd[NW];
#pragma unroll
  for (int i = 0; i < NW; ++i) {
    if constexpr (TRANS) {
      const int per = p.r / 8, k = 64 * i + lane, row = k / per;
      wo[i] = k < KC * per ? 8 * k : -1;
      wd[i] = row * WS + 8 * (k - row * per);
    } else {
      // ranks past r read the last one again, their results are dropped
      wo[i] = min(RPI * i + lr, p.r - 1) * p.C + lc;
      wd[i] = (RPI * i + lr) * WS + lc;
    }
  }
  // Every load is issued (past C: the last columns again), so that the compiler can
  // count the ones in flight; what lies past C becomes zero on its way to LDS.
  const u32x4 zero = {0, 0, 0, 0};
  // chunks in flight: at high ranks, where few waves fit, two (4096 x 7168 of rank 128
  // into 2048 columns, a forward: 55 us, one 62; at lower ranks no difference)
  constexpr int DEPTH = RT >= 6 ? 2 : 1;
  u32x4 xbuf[DEPTH][NX], wbuf[DEPTH][NW];
  auto fetch = [&](u32x4 (&xa)[NX], u32x4 (&wa)[NW], int s) {
    const int col = min(KC * s, p.C - 8 - lc);
#pragma unroll
    for (int i = 0; i < NX; ++i) xa[i] = *reinterpret_cast<const u32x4*>(xr[i] + col);
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      if constexpr (TRANS)
        wa[i] = *reinterpret_cast<const u32x4*>(w + min(KC * s * p.r + max(wo[i], 0), p.C * p.r - 8));
      else
        wa[i] = *reinterpret_cast<const u32x4*>(w + wo[i] + col);
    }
  };
  f32x4 acc[MT][RT] = {};
  // the waves of all splits of a tile (neighbours in the grid) take the chunks in
  // turn, so that together they walk the rows' lines in order
  const int stride = p.splits * LORA_WAVES, s0 = split * LORA_WAVES + wave;
#pragma unroll
  for (int d = 0; d < DEPTH; ++d) fetch(xbuf[d], wbuf[d], min(s0 + d * stride, p.chunks - 1));
  auto step = [&](u32x4 (&xa)[NX], u32x4 (&wa)[NW], int s) {
    wave_fence();
#pragma unroll
    for (int i = 0; i < NX; ++i)
      *reinterpret_cast<u32x4*>(&xs[wave][RPI * i + lr][lc]) = KC * s + lc < p.C ? xa[i] : zero;
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      const bool in = TRANS ? KC * s * p.r + wo[i] < p.C * p.r : KC * s + lc < p.C;
      if (!TRANS || wo[i] >= 0)
        *reinterpret_cast<u32x4*>(&wt[wave][0][0] + wd[i]) = in ? wa[i] : zero;
    }
    wave_fence();
    fetch(xa, wa, min(s + DEPTH * stride, p.chunks - 1));
#pragma unroll
    for (int k = 0; k < KC; k += 32) {
      u32x4 xf[MT], wf[RT];
#pragma unroll
      for (int m = 0; m < MT; ++m)
        xf[m] = *reinterpret_cast<const u32x4*>(&xs[wave][16 * m + l][k + 8 * g]);
#pragma unroll
      for (int j = 0; j < RT; ++j) {
        if constexpr (TRANS) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const u32x2 v =
                read_tr(&wt[wave][k + 8 * g + 4 * h + (l >> 2)][16 * j + 4 * (l & 3)]);
            wf[j][2 * h] = v[0];
            wf[j][2 * h + 1] = v[1];
          }
        } else {
          wf[j] = *reinterpret_cast<const u32x4*>(&wt[wave][16 * j + l][k + 8 * g]);
        }
      }
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int j = 0; j < RT; ++j) acc[m][j] = mfma16(wf[j], xf[m], acc[m][j]);
    }
  };
  for (int s = s0; s < p.chunks; s += DEPTH * stride)
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) {
      if (s + d * stride >= p.chunks) break;
      step(xbuf[d], wbuf[d], s + d * stride);
    }
  // the waves' sums, in wave order, 16 rows and ranks at a time
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int j = 0; j < RT; ++j) {
      if (m || j) __syncthreads();
      *reinterpret_cast<f32x4*>(&red[wave][l][4 * g]) = acc[m][j];
      __syncthreads();
      const int row = threadIdx.x >> 2, c = 4 * (threadIdx.x & 3);
      if (threadIdx.x < 64 && 16 * m + row < tl.n && 16 * j + c < p.r) {
        f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < LORA_WAVES; ++k) v += *reinterpret_cast<const f32x4*>(&red[k][row][c]);
        *reinterpret_cast<f32x4*>(p.part + ((size_t)split * p.T + tl.p0 + 16 * m + row) * p.r +
                                  16 * j + c) = v;
      }
    }
}

// The first of the four columns, within a wave's 64, that lane group g holds of
// MFMA tile i.
__device__ __forceinline__ int lora_column(int i, int g) { return 32 * (i >> 1) + 8 * g + 4 * (i & 1); }

struct LoraExpand {
  const float* part;          // [splits][T][r]
  const uint16_t *w;          // factor [NA, C, r], or [NA, r, C] (TRANS)
  const float* scale;         // [NA] or NULL
  const int32_t *offsets, *src_row;
  const uint16_t* y;          // [T, C] or NULL (zeros)
  uint16_t* out;              // [T, C] or NULL (only v_out is wanted); may be y
  float* v_out;               // [T, r] or NULL: the added parts
  int T, C, r, NA, splits, scale_v;   // scale_v: v_out holds s[a] v
  int col_blocks;
};

// A tile's rank values into LDS: the splits' parts added in order (eight loads in
// flight, the last one again past the end), scaled and split into two bf16 parts, the high one at the start of a
// row of `stride` elements and the low one at `lo`, zeros behind either up to
// `lo` and `len`; rows past the tile are zeros.  The block with `keep` writes v_out.
__device__ __forceinline__ void stage_ranks(const LoraExpand& p, const LoraTile& tl, int rows,
                                            bool keep, int lo, int len, uint16_t* vs, int stride) {
  const float sc = p.scale ? p.scale[tl.a] : 1.0f;
  const int quads = p.r / 4;
  for (int i = threadIdx.x; i < rows * quads; i += 64 * LORA_WAVES) {
    const int row = i / quads, j = (i - row * quads) * 4;
    f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
    if (row < tl.n) {
      const float* src = p.part + (size_t)(tl.p0 + row) * p.r + j;
      const size_t ld = (size_t)p.T * p.r;
      if (p.splits <= 2) {
        v = *reinterpret_cast<const f32x4*>(src);
        if (p.splits == 2) v += *reinterpret_cast<const f32x4*>(src + ld);
      } else {
        for (int k = 0; k < p.splits; k += 8) {
          f32x4 o[8];
#pragma unroll
          for (int q = 0; q < 8; ++q)
            o[q] = *reinterpret_cast<const f32x4*>(src + min(k + q, p.splits - 1) * ld);
#pragma unroll
          for (int q = 0; q < 8; ++q)
            if (k + q < p.splits) v += o[q];
        }
      }
      const f32x4 sv = v * sc;
      if (p.v_out && keep)
        *reinterpret_cast<f32x4*>(p.v_out + (size_t)(tl.p0 + row) * p.r + j) = p.scale_v ? sv : v;
      v = sv;
    }
    u32x2 hb, lb;
    split_quad(v, hb, lb);
    *reinterpret_cast<u32x2*>(vs + row * stride + j) = hb;
    *reinterpret_cast<u32x2*>(vs + row * stride + lo + j) = lb;
  }
  const int gap = (lo - p.r) / 8, pads = (len - 2 * p.r) / 8;
  const u32x4 zero = {0, 0, 0, 0};
  for (int i = threadIdx.x; i < rows * pads; i += 64 * LORA_WAVES) {
    const int row = i / pads, k = i - row * pads;
    *reinterpret_cast<u32x4*>(vs + row * stride + (k < gap ? p.r + 8 * k : lo + p.r + 8 * (k - gap))) =
        zero;
  }
}

// out[t(p)][c] = y + sum_j s[a] v[p][j] w[a][c][j].  A wave takes chunks of 64
// columns of the tile's rows, the next chunk's y loaded meanwhile: its four MFMA
// tiles hold columns 32 (i / 2) + 8 g + 4 (i % 2) + q of lane group g (tile i,
// register q), so a lane ends up with two runs of 8 columns of its row and each
// load of y and store of out covers 64 contiguous bytes of 16 rows.  A factor
// stored the other way (TRANS) passes through LDS and is read transposed.
template <int MT, int KH, bool TRANS>
__global__ void __launch_bounds__(64 * LORA_WAVES) lora_expand_kernel(const LoraExpand p) {
  constexpr int TM = 16 * MT, R = 32 * KH;
  constexpr int VS = 2 * R + 8;             // a row's two parts of R ranks
  constexpr int WS = 64 + 8;                // row stride of a wave's factor tile
  __shared__ __align__(16) uint16_t vs[TM][VS];
  __shared__ __align__(16) uint16_t wt[TRANS ? LORA_WAVES : 1][TRANS ? R : 1][WS];
  const int cb = blockIdx.x % p.col_blocks;
  const LoraTile tl = lora_tile<false>(p.offsets, p.NA, p.T, TM, blockIdx.x / p.col_blocks);
  if (tl.n <= 0) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int l = lane & 15, g = lane >> 4;
  const int chunks = (p.C + 63) / 64, step = p.col_blocks * LORA_WAVES;
  int ch = cb * LORA_WAVES + wave;
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
    const int c = 64 * chunk + 8 * g;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int q = 0; q < 2; ++q)
        yr[m][q] = p.y && p.out && t[m] >= 0 && c + 32 * q < p.C
                       ? *reinterpret_cast<const u32x4*>(p.y + (size_t)t[m] * p.C + c + 32 * q)
                       : zero;
  };
  fetch(ch);
  stage_ranks(p, tl, TM, cb == 0, R, 2 * R, &vs[0][0], VS);
  __syncthreads();
  if (!p.out) return;
  const uint16_t* w = p.w + (size_t)tl.a * p.r * p.C;
  for (; ch < chunks; ch += step) {
    u32x4 yc[MT][2];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int q = 0; q < 2; ++q) yc[m][q] = yr[m][q];
    // The chunk's factor in one round of loads (past r: any of its values, the rank
    // values are zero there).  Loads return in order, so the next chunk's y is asked
    // for behind them: waiting for the factor does not wait for it.
    u32x4 wa[KH][4];
    if constexpr (TRANS) {
      // eight rows of 128 bytes per instruction, turned in LDS
      u32x4 raw[4 * KH];
      const int c = min(64 * ch + 8 * (lane & 7), p.C - 8);
#pragma unroll
      for (int i = 0; i < 4 * KH; ++i)
        raw[i] = *reinterpret_cast<const u32x4*>(
            w + (size_t)min(8 * i + (lane >> 3), p.r - 1) * p.C + c);
      if (ch + step < chunks) fetch(ch + step);
      wave_fence();
#pragma unroll
      for (int i = 0; i < 4 * KH; ++i)
        *reinterpret_cast<u32x4*>(&wt[wave][8 * i + (lane >> 3)][8 * (lane & 7)]) = raw[i];
      wave_fence();
#pragma unroll
      for (int s = 0; s < KH; ++s)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const u32x2 v =
                read_tr(&wt[wave][32 * s + 8 * g + 4 * h + (l >> 2)][lora_column(i, l & 3)]);
            wa[s][i][2 * h] = v[0];
            wa[s][i][2 * h + 1] = v[1];
          }
    } else {
#pragma unroll
      for (int s = 0; s < KH; ++s)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c = min(64 * ch + lora_column(i, l >> 2) + (l & 3), p.C - 1);
          wa[s][i] = *reinterpret_cast<const u32x4*>(w + (size_t)c * p.r +
                                                     min(32 * s + 8 * g, p.r - 8));
        }
      if (ch + step < chunks) fetch(ch + step);
    }
    f32x4 acc[MT][4] = {};
#pragma unroll
    for (int s = 0; s < 2 * KH; ++s)
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const u32x4 va = *reinterpret_cast<const u32x4*>(&vs[16 * m + l][32 * s + 8 * g]);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[m][i] = mfma16(wa[s % KH][i], va, acc[m][i]);
      }
    const int c = 64 * ch + 8 * g;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      if (t[m] < 0) continue;
#pragma unroll
      for (int q = 0; q < 2; ++q)
        if (c + 32 * q < p.C)
          *reinterpret_cast<u32x4*>(p.out + (size_t)t[m] * p.C + c + 32 * q) =
              add_chunk(yc[m][q], acc[m][2 * q], acc[m][2 * q + 1]);
    }
  }
}

// Rows of one adapter that a block of lora_apply_kernel takes, at most.
constexpr int apply_rows(int kh) { return kh <= 2 ? 192 : 96; }

// expand for many rows: a wave keeps the factor of its 64 columns in registers
// and walks its block's rows 16 at a time, the loads of the next DEPTH steps in
// flight, so the factor is read once per block of rows and nothing but the
// rows moves in the loop.  Columns are placed as in lora_expand_kernel.
//
// What bounds it is how the memory is walked, measured with plain copies of
// 8192 x 8192 bytes cut the same way: 64 bytes of 16 rows an instruction
// 3.3 TB/s, 128 bytes of 8 rows 3.6, with the blocks of the same rows next to
// each other in the grid 5.0, with nontemporal stores 6.5.  So the column blocks
// come first in the grid, the outputs (far larger than the L2) are stored
// nontemporally, and two lanes that hold halves of two rows (l and l ^ 8)
// swap chunks, so that an instruction covers whole 128-byte lines of 8 rows.
// 8192 x 4096 at rank 32: 37 us, of which the rows' loop takes half; the blocks
// start together, and their first loads (factor, rank values, rows) queue up.
//
// The loop over whole steps has no branch and no mask (rows past the last one
// load the last one again): behind a load that may not have been issued the
// compiler can only wait for everything, stores included, which emptied the
// pipeline every round.  The last steps, their loads in flight already, are
// masked; rows without a source and columns past C take a plain loop.
template <int KH, bool TRANS>
__global__ void __launch_bounds__(64 * LORA_WAVES) lora_apply_kernel(const LoraExpand p,
                                                                     const int rows) {
  constexpr int DEPTH = KH <= 2 ? 4 : 2;
  constexpr int VS = 64 * KH + 8;           // a row's two parts of 32 KH ranks
  constexpr int WS = 64 + 8;                // row stride of a wave's factor tile
  static_assert(LORA_WAVES * 32 * WS <= apply_rows(KH) * VS, "the factor's tiles fit");
  __shared__ int toks[apply_rows(KH)];
  __shared__ __align__(16) uint16_t vs[apply_rows(KH) * VS];
  const LoraTile tl =
      lora_tile<false>(p.offsets, p.NA, p.T, rows, (int)(blockIdx.x / p.col_blocks));
  if (tl.n <= 0) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int l = lane & 15, g = lane >> 4;
  const int c0 = (int)(blockIdx.x % p.col_blocks * LORA_WAVES + wave) * 64, c = c0 + 8 * g;
  if (tl.a >= p.NA) {                       // no adapter: the rows as they are
    if (p.out == p.y) return;
    const u32x4 zero = {0, 0, 0, 0};
    const int cc = c0 + 8 * (lane & 7);
    for (int i = lane >> 3; i < tl.n; i += 8) {
      const int t = lora_token(p.src_row, tl.p0 + i, p.T);
      if (t < 0 || cc >= p.C) continue;
      const size_t o = (size_t)t * p.C + cc;
      *reinterpret_cast<u32x4*>(p.out + o) = p.y ? *reinterpret_cast<const u32x4*>(p.y + o) : zero;
    }
    return;
  }
  int bad = 0;
  for (int i = threadIdx.x; i < rows; i += 64 * LORA_WAVES) {
    const int t = i < tl.n ? lora_token(p.src_row, tl.p0 + i, p.T) : -1;
    bad |= i < tl.n && t < 0;
    toks[i] = t;
  }
  // (ranks past r: any of the factor's, the rank values are zero there)
  u32x4 wa[KH][4];
  const uint16_t* w = p.w + (size_t)tl.a * p.r * p.C;
  if constexpr (TRANS) {
    // whole lines, 8 ranks an instruction, turned in the memory that the rank values
    // take next, 32 ranks at a time (4096 x 7168 at rank 128: 43 us, 54 with two-byte
    // loads)
    uint16_t* wt = vs + wave * 32 * WS;
    const int cw = min(c0 + 8 * (lane & 7), p.C - 8);
    u32x4 raw[KH][4];
#pragma unroll
    for (int k = 0; k < 4 * KH; ++k)
      raw[k / 4][k % 4] = *reinterpret_cast<const u32x4*>(
          w + (size_t)min(8 * k + (lane >> 3), p.r - 1) * p.C + cw);
#pragma unroll
    for (int s = 0; s < KH; ++s) {
      wave_fence();
#pragma unroll
      for (int k = 0; k < 4; ++k)
        *reinterpret_cast<u32x4*>(wt + (8 * k + (lane >> 3)) * WS + 8 * (lane & 7)) = raw[s][k];
      wave_fence();
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const u32x2 v = read_tr(wt + (8 * g + 4 * h + (l >> 2)) * WS + lora_column(i, l & 3));
          wa[s][i][2 * h] = v[0];
          wa[s][i][2 * h + 1] = v[1];
        }
    }
    __syncthreads();
  } else {
#pragma unroll
    for (int s = 0; s < KH; ++s)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int cw = min(c0 + lora_column(i, l >> 2) + (l & 3), p.C - 1);
        wa[s][i] = *reinterpret_cast<const u32x4*>(w + (size_t)cw * p.r +
                                                   min(32 * s + 8 * g, p.r - 8));
      }
  }
  stage_ranks(p, tl, (tl.n + 15) & ~15, blockIdx.x % p.col_blocks == 0, 32 * KH, 64 * KH, vs, VS);
  const bool plain = __syncthreads_or(bad) || !p.y || c0 + 64 > p.C;
  if (c0 >= p.C) return;
  // o = y + the product, for rows 16 step + l
  auto add = [&](int step, const u32x4* y, u32x4* o) {
    const uint16_t* v = vs + (16 * step + l) * VS + 8 * g;
    f32x4 acc[4] = {};
#pragma unroll
    for (int k = 0; k < 2 * KH; ++k) {
      const u32x4 vf = *reinterpret_cast<const u32x4*>(v + 32 * k);
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] = mfma16(wa[k % KH][i], vf, acc[i]);
    }
#pragma unroll
    for (int q = 0; q < 2; ++q) o[q] = add_chunk(y[q], acc[2 * q], acc[2 * q + 1]);
  };
  int s = 0;
  if (!plain) {
    u32x4 yr[DEPTH][2];
    uint16_t* at[DEPTH][2];
    // instruction q: rows 8 q + (l & 7), chunk 4 (l >> 3) + g of the 128 bytes
    const int col = c0 + 32 * (l >> 3) + 8 * g;
    auto fetch = [&](int d, int step) {
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int row = min(16 * step + 8 * q + (l & 7), tl.n - 1);
        const size_t o = (size_t)toks[row] * p.C + col;
        at[d][q] = p.out + o;
        yr[d][q] = *reinterpret_cast<const u32x4*>(p.y + o);
      }
      __builtin_amdgcn_sched_barrier(0);
    };
    // lanes l < 8 give their second chunk for the first of lane l + 8 (its own inverse)
    auto swap = [&](u32x4* v) {
      const u32x4 give = l < 8 ? v[1] : v[0];
      u32x4 got;
#pragma unroll
      for (int i = 0; i < 4; ++i)          // row_ror:8: lane l ^ 8 of each 16
        got[i] = __builtin_amdgcn_update_dpp(0, (int)give[i], 0x128, 0xf, 0xf, false);
      if (l < 8) v[1] = got;
      else v[0] = got;
    };
    auto round = [&]() {
#pragma unroll
      for (int d = 0; d < DEPTH; ++d) {
        u32x4 o[2];
        swap(yr[d]);
        add(s + d, yr[d], o);
        swap(o);
        uint16_t* to[2] = {at[d][0], at[d][1]};
        fetch(d, s + DEPTH + d);
#pragma unroll
        for (int q = 0; q < 2; ++q)
          __builtin_nontemporal_store(o[q], reinterpret_cast<u32x4*>(to[q]));
        __builtin_amdgcn_sched_barrier(0);
      }
      s += DEPTH;
    };
    // The loads in order (the scheduling barriers), and the first round apart, so
    // that the loop is entered with the same accesses in flight as it repeats with.
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) fetch(d, d);
    const int whole = tl.n / 16 / DEPTH * DEPTH;
    if (whole > 0) {
      round();
      while (s < whole) round();
    }
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) {
      if (16 * (s + d) >= tl.n) break;
      u32x4 o[2];
      swap(yr[d]);
      add(s + d, yr[d], o);
      swap(o);
#pragma unroll
      for (int q = 0; q < 2; ++q)
        if (16 * (s + d) + 8 * q + (l & 7) < tl.n)
          __builtin_nontemporal_store(o[q], reinterpret_cast<u32x4*>(at[d][q]));
    }
    return;
  }
  for (; 16 * s < tl.n; ++s) {
    const int t = toks[16 * s + l];
    u32x4 y[2], o[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const u32x4 zero = {0, 0, 0, 0};
      y[q] = t >= 0 && p.y && c + 32 * q < p.C
                 ? *reinterpret_cast<const u32x4*>(p.y + (size_t)t * p.C + c + 32 * q)
                 : zero;
    }
    add(s, y, o);
#pragma unroll
    for (int q = 0; q < 2; ++q)
      if (t >= 0 && c + 32 * q < p.C)
        *reinterpret_cast<u32x4*>(p.out + (size_t)t * p.C + c + 32 * q) = o[q];
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

// A block sums one chunk of a segment; its waves take 32 rows and 64 columns at a time.
// The rows pass through LDS (a wave's own 32 x 64 tile, whole lines in, read
// transposed: the reduction runs over rows), u is split into three bf16 parts, which
// hold its 24 bits, so the float32 sums are of float32 accuracy at three bf16 MFMAs
// a step: 830 TFLOP/s of the bf16 rate against 157 of v_mfma_f32.  The waves share
// the rows of 64 columns and add their sums at the end; or (OWN) each has 64 columns
// and all rows, and the block splits u once for all of them, through LDS: a quarter
// of the loads of u and of the splitting, and no idle waves where a segment has few
// rows, but a quarter of the blocks, and two barriers a step.  Both gradients of 8192
// rows of 8 adapters, rank 16, 4096 x 4096: 30 us, 4.7 TB/s, bound by memory; rank 64,
// 2 adapters, 8192 x 8192: 85 us, 3.4 TB/s (shared rows 110).  128 columns a wave
// leave too few waves: 5 to 15 % slower at every size tried.
template <int RT, bool OWN>
__global__ void __launch_bounds__(64 * LORA_WAVES) lora_wgrad_kernel(const LoraWgrad p) {
  constexpr int CT = WGRAD_COLS / 16, COLS = WGRAD_COLS;
  constexpr int CPR = COLS / 8, NX = CPR / 2;      // chunks per row, loads per step
  constexpr int RPI = 64 / CPR;                    // rows per load instruction
  constexpr int US = 32 + 8;                       // row stride of u's parts, elements
  // a wave's rows, and when they are done with, its sums
  __shared__ __align__(16) union {
    uint16_t x[32][COLS + 8];
    float sum[16][COLS + 4];
  } lds[LORA_WAVES];
  __shared__ __align__(16) uint16_t us[OWN ? 3 : 1][OWN ? 16 * RT : 1][US];    // [part][rank][row]
  const LoraGrad& G = p.g[blockIdx.z & 1];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int b0 = blockIdx.x * COLS * (OWN ? LORA_WAVES : 1), c0 = b0 + (OWN ? wave * COLS : 0);
  const int r0 = (blockIdx.z >> 1) * 16 * RT;
  if (!G.out || b0 >= G.C) return;
  const LoraTile tl = lora_tile<true>(p.offsets, p.NA, p.T, p.chunk, blockIdx.y);
  if (tl.n < 0 || tl.a >= p.NA) return;
  constexpr int STEP = OWN ? 1 : LORA_WAVES;
  const int first = OWN ? 0 : wave;
  const int l = lane & 15, g = lane >> 4;
  const int xrow = lane / CPR, xcol = 8 * (lane % CPR);
  const int xc = min(c0 + xcol, G.C - 8);       // (C a multiple of 32)
  // the tokens of 32 rows, one a lane (both halves of the wave alike)
  auto tokens = [&](int s) {
    const int i = 32 * s + (lane & 31);
    const int t = lora_token(p.src_row, tl.p0 + min(i, tl.n - 1), p.T);
    return i < tl.n ? t : -1;
  };
  const u32x4 zero = {0, 0, 0, 0};
  // (every load is issued, rows without a token read row 0 and become zero on
  // their way to LDS: the compiler can then count the loads in flight)
  auto fetch = [&](int tok, u32x4 (&x)[NX]) {
#pragma unroll
    for (int i = 0; i < NX; ++i) {
      const int t = __shfl(tok, RPI * i + xrow, 64);
      x[i] = *reinterpret_cast<const u32x4*>(G.x + (size_t)max(t, 0) * G.C + xc);
    }
  };
  // OWN: u's four rows 4 (i / 16 RT) of rank i % 16 RT, all threads of the block
  constexpr int NU = (128 * RT + 64 * LORA_WAVES - 1) / (64 * LORA_WAVES);
  float ua[OWN ? NU : 1][4];
  auto fetch_u = [&](int s) {
    if constexpr (OWN) {
      const float* u = G.u + (size_t)(tl.p0 + 32 * s) * p.r;
      const int last = tl.n - 1 - 32 * s;
#pragma unroll
      for (int k = 0; k < NU; ++k) {
        const int i = threadIdx.x + 64 * LORA_WAVES * k, row = 4 * (i / (16 * RT));
        const int rank = min(r0 + i % (16 * RT), p.r - 1);
#pragma unroll
        for (int e = 0; e < 4; ++e) ua[k][e] = u[(size_t)min(row + e, last) * p.r + rank];
      }
    }
  };
  f32x4 acc[RT][CT] = {};
  const int steps = (tl.n + 31) / 32;
  u32x4 x[NX];
  int tok = -1, next = -1;
  if (first < steps) {          // (an adapter without rows reads nothing)
    tok = tokens(first);
    fetch_u(first);
    fetch(tok, x);
    next = tokens(first + STEP);
  }
  for (int s = first; s < steps; s += STEP) {
    const uint32_t valid = (uint32_t)__ballot(tok >= 0);
    if constexpr (OWN) {
      __syncthreads();
#pragma unroll
      for (int k = 0; k < NU; ++k) {
        const int i = threadIdx.x + 64 * LORA_WAVES * k, row = 4 * (i / (16 * RT)), rank = i % (16 * RT);
        if (i >= 128 * RT) break;
        u32x2 part[3];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t b[3][2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const bool in = r0 + rank < p.r && (valid >> (row + 2 * q + e) & 1);
            split3(in ? ua[k][2 * q + e] : 0.0f, b[0][e], b[1][e], b[2][e]);
          }
#pragma unroll
          for (int h = 0; h < 3; ++h) part[h][q] = b[h][0] | b[h][1] << 16;
        }
#pragma unroll
        for (int h = 0; h < 3; ++h) *reinterpret_cast<u32x2*>(&us[h][rank][row]) = part[h];
      }
    }
    wave_fence();
#pragma unroll
    for (int i = 0; i < NX; ++i)
      *reinterpret_cast<u32x4*>(&lds[wave].x[RPI * i + xrow][xcol]) =
          valid >> (RPI * i + xrow) & 1 ? x[i] : zero;
    if constexpr (OWN) __syncthreads();
    else wave_fence();
    // (u's loads in front of the next rows': loads return in order)
    float uv[OWN ? 1 : RT][8];
    if constexpr (!OWN) {
      const float* u = G.u + (size_t)(tl.p0 + 32 * s) * p.r;
      const int last = tl.n - 1 - 32 * s;
#pragma unroll
      for (int j = 0; j < RT; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i)
          uv[j][i] = u[(size_t)min(8 * g + i, last) * p.r + min(r0 + 16 * j + l, p.r - 1)];
    } else if (s + STEP < steps) {
      fetch_u(s + STEP);
    }
    tok = next;
    fetch(tok, x);
    next = tokens(s + 2 * STEP);
    u32x4 xa[CT];
#pragma unroll
    for (int i = 0; i < CT; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const u32x2 v = read_tr(&lds[wave].x[8 * g + 4 * h + (l >> 2)][16 * i + 4 * (l & 3)]);
        xa[i][2 * h] = v[0];
        xa[i][2 * h + 1] = v[1];
      }
    // rows without a token, and ranks past r, count as zero
    if constexpr (!OWN) {
      if (valid != 0xffffffffu || r0 + 16 * RT > p.r) {
#pragma unroll
        for (int j = 0; j < RT; ++j)
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (r0 + 16 * j + l >= p.r || !(valid >> (8 * g + i) & 1)) uv[j][i] = 0.0f;
      }
    }
#pragma unroll
    for (int j = 0; j < RT; ++j) {
      u32x4 part[3];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if constexpr (OWN) break;
        uint32_t b[3][2];
#pragma unroll
        for (int e = 0; e < 2; ++e)
          split3(uv[OWN ? 0 : j][2 * q + e], b[0][e], b[1][e], b[2][e]);
#pragma unroll
        for (int h = 0; h < 3; ++h) part[h][q] = b[h][0] | b[h][1] << 16;
      }
      if constexpr (OWN) {
#pragma unroll
        for (int h = 0; h < 3; ++h)
          part[h] = *reinterpret_cast<const u32x4*>(&us[h][16 * j + l][8 * g]);
      }
#pragma unroll
      for (int i = 0; i < CT; ++i)
#pragma unroll
        for (int h = 0; h < 3; ++h) acc[j][i] = mfma16(part[h], xa[i], acc[j][i]);
    }
  }
  // the waves in order, 16 ranks at a time
  const bool whole = tl.rows <= p.chunk;
  const float sc = whole && G.scale ? G.scale[tl.a] : 1.0f;
  float* out = whole ? G.out + (size_t)tl.a * p.r * G.C
                     : G.part + (size_t)lora_slot(tl.p0, tl.s0, p.chunk) * p.r * G.C;
  const bool add = whole && p.accumulate;
  auto sync = [&]() {
    if constexpr (OWN) wave_fence();
    else __syncthreads();
  };
#pragma unroll
  for (int j = 0; j < RT; ++j) {
    sync();
#pragma unroll
    for (int i = 0; i < CT; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) lds[wave].sum[4 * g + q][16 * i + l] = acc[j][i][q];
    sync();
    // four sums a lane, along the columns or (trans) the ranks
    for (int i = OWN ? lane : threadIdx.x; i < 4 * COLS; i += OWN ? 64 : 64 * LORA_WAVES) {
      const int rr = G.trans ? i % 4 * 4 : i / (COLS / 4), cc = G.trans ? i / 4 : i % (COLS / 4) * 4;
      const int rank = r0 + 16 * j + rr, c = c0 + cc;
      if (rank >= p.r || c >= G.C) continue;
      f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int k = 0; k < STEP; ++k) {
        const float(*from)[COLS + 4] = lds[OWN ? wave : k].sum;
        if (G.trans) {
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] += from[rr + e][cc];
        } else {
          v += *reinterpret_cast<const f32x4*>(&from[rr][cc]);
        }
      }
      v *= sc;
      f32x4* o = reinterpret_cast<f32x4*>(
          out + (G.trans ? (size_t)c * p.r + rank : (size_t)rank * G.C + c));
      *o = add ? *o + v : v;
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

// Row tiles of 16, 32 or 64 (at most `most` 16s): the highest that the adapters
// fill on average and that leaves `least` tiles.  A factor's tile is read once
// per tile of rows, so high tiles save reads of it, while few tiles leave the
// card empty or cost splits of the reduction.  Shrink, whose tiles are its
// blocks, asks for 192, above rank 64, where the factor weighs more than the
// rows, for 96 (8192 rows of rank 128: 41 us with 192, 38 us with 96; of rank
// 32: 27 and 30 us).  Expand, which has the columns to spread over, asks for
// 1024 tiles x 256 columns.
static int lora_mt(int T, int NA, int least, int most) {
  for (int mt = most; mt > 1; mt /= 2)
    if (T >= 16 * mt * std::max(NA, least)) return mt;
  return 1;
}
static int shrink_mt(int T, int NA, int r) { return lora_mt(T, NA, r > 64 ? 96 : 192, 4); }
static int expand_mt(int T, int NA, int C) { return lora_mt(T, NA, std::max(1, 1024 * 256 / C), 2); }
static int lora_tiles(int T, int NA, int mt) { return T / (16 * mt) + std::min(NA + 1, T) + 1; }

static int lora_rank_tiles(int r) { return r <= 64 ? (r + 15) / 16 : r <= 96 ? 6 : 8; }
// Chunks of the reduction over C (as lora_shrink_kernel cuts it).
static int lora_chunks(int C, int r) { return lora_rank_tiles(r) <= 4 ? (C + 63) / 64 : C / 32; }

// Blocks along a reduction: as many as fill the card, with at least two chunks
// per wave.
static int lora_splits(int T, int NA, int C, int r) {
  const int mt = shrink_mt(T, NA, r);
  const int tiles = std::max(1, T / (16 * mt) + (mt == 1 ? std::min(NA, T) / 2 : 0));
  return std::max(1, std::min({(r > 64 ? 320 : 512) / tiles, lora_chunks(C, r) / (2 * LORA_WAVES), 16}));
}

// Calls f(RT) for the rank tiles that cover r (1, 2, 3, 4, 6 or 8 of 16).
template <class F>
static moe_status_t lora_ranks(int r, F&& f) {
  switch (lora_rank_tiles(r)) {
    case 1: f(std::integral_constant<int, 1>()); break;
    case 2: f(std::integral_constant<int, 2>()); break;
    case 3: f(std::integral_constant<int, 3>()); break;
    case 4: f(std::integral_constant<int, 4>()); break;
    case 6: f(std::integral_constant<int, 6>()); break;
    default: f(std::integral_constant<int, 8>()); break;
  }
  return launch_status();
}

template <bool TRANS>
static moe_status_t launch_shrink(const LoraShrink& p, hipStream_t s) {
  const int mt = shrink_mt(p.T, p.NA, p.r);
  const size_t blocks = (size_t)lora_tiles(p.T, p.NA, mt) * p.splits;
  if (blocks > INT32_MAX) return MOE_ERR_UNSUPPORTED;
  const dim3 grid((unsigned)blocks), block(64 * LORA_WAVES);
  return lora_ranks(p.r, [&](auto N) {
    constexpr int RT = decltype(N)::value;
    if (mt == 4) hipLaunchKernelGGL((lora_shrink_kernel<4, RT, TRANS>), grid, block, 0, s, p);
    else if (mt == 2) hipLaunchKernelGGL((lora_shrink_kernel<2, RT, TRANS>), grid, block, 0, s, p);
    else hipLaunchKernelGGL((lora_shrink_kernel<1, RT, TRANS>), grid, block, 0, s, p);
  });
}

template <bool TRANS>
static moe_status_t launch_expand(LoraExpand p, hipStream_t s) {
  const int mt = expand_mt(p.T, p.NA, p.C);
  // blocks along the columns: one per 256 columns, fewer (each then walks several
  // chunks and reads the tile's ranks once) as long as 1024 blocks remain
  const int tiles = lora_tiles(p.T, p.NA, mt), cols = (p.C + 64 * LORA_WAVES - 1) / (64 * LORA_WAVES);
  p.col_blocks = p.out ? std::min(cols, std::max(1, 1024 / tiles)) : 1;
  const size_t blocks = (size_t)tiles * p.col_blocks;
  if (blocks > INT32_MAX) return MOE_ERR_UNSUPPORTED;
  const dim3 grid((unsigned)blocks), block(64 * LORA_WAVES);
  auto go = [&](auto N) {
    constexpr int KH = decltype(N)::value;
    if (mt == 2) hipLaunchKernelGGL((lora_expand_kernel<2, KH, TRANS>), grid, block, 0, s, p);
    else hipLaunchKernelGGL((lora_expand_kernel<1, KH, TRANS>), grid, block, 0, s, p);
  };
  switch ((p.r + 31) / 32) {
    case 1: go(std::integral_constant<int, 1>()); break;
    case 2: go(std::integral_constant<int, 2>()); break;
    case 3: go(std::integral_constant<int, 3>()); break;
    default: go(std::integral_constant<int, 4>()); break;
  }
  return launch_status();
}

template <bool TRANS>
static moe_status_t launch_apply(LoraExpand p, hipStream_t s) {
  const int kh = (p.r + 31) / 32;
  const int cols = (p.C + 64 * LORA_WAVES - 1) / (64 * LORA_WAVES);
  // rows a block: about 1300 blocks (measured: 300 to 700 long ones are slower, the
  // card's many short waits no longer overlap)
  const size_t share = (size_t)p.T * cols / 1300 / 16 * 16;
  const int rows = std::max(32, (int)std::min((size_t)apply_rows(kh), share));
  p.col_blocks = cols;
  const size_t blocks = (size_t)(p.T / rows + std::min(p.NA + 1, p.T) + 1) * cols;
  if (blocks > INT32_MAX) return MOE_ERR_UNSUPPORTED;
  const dim3 grid((unsigned)blocks), block(64 * LORA_WAVES);
  switch (kh) {
    case 1: hipLaunchKernelGGL((lora_apply_kernel<1, TRANS>), grid, block, 0, s, p, rows); break;
    case 2: hipLaunchKernelGGL((lora_apply_kernel<2, TRANS>), grid, block, 0, s, p, rows); break;
    case 3: hipLaunchKernelGGL((lora_apply_kernel<3, TRANS>), grid, block, 0, s, p, rows); break;
    default: hipLaunchKernelGGL((lora_apply_kernel<4, TRANS>), grid, block, 0, s, p, rows); break;
  }
  return launch_status();
}

// The second half of a pass over activations: expand for few rows; apply from 32
// rows per adapter on, if there are 8 MiB of output (whole forwards, expand and apply:
// 1027 x 5760 at rank 64 24.4 and 22.7 us, 1024 x 8192 of 32 adapters at rank 16 19.1
// and 17.1; 512 x 4096 of 2 at rank 32 11.4 and 11.8, 4096 x 256 8.8 and 9.9).
template <bool TRANS>
static moe_status_t launch_out(const LoraExpand& e, hipStream_t s) {
  const bool many = (size_t)e.T * e.C >= (1u << 22) && e.T >= 32 * e.NA;
  return e.out && many ? launch_apply<TRANS>(e, s) : launch_expand<TRANS>(e, s);
}

// Rows that a block of the weight gradients sums: an eighth of the batch, at
// least 1024, so that a batch of one adapter still fills the card.
static int lora_chunk(int T) { return std::max(1024, (T + 7) / 8); }
static size_t lora_slots(int T) {
  return T > lora_chunk(T) ? 2 * ((size_t)T / lora_chunk(T) + 1) : 0;
}

// Whether the waves take columns of their own (OWN; below, against rows shared).  For
// segments of few rows: 10 rows of 48 adapters at rank 16, 2048 x 8192, 17 us and 30;
// 16 rows of 16 at rank 64, 4096 x 4096, 12 and 30; 88 of 8, 10 and 9.  And with as many
// blocks as the card takes, fewer at high ranks, where u's share of the work is larger:
// 8192 x 8192, 8192 rows of 2 at rank 64 (512 blocks) 85 and 110; of 48 at rank 128 255
// and 426; 4096 x 4096, 8192 rows of 24 at rank 32 (768) 40 and 47, of 16 at rank 16
// (512) 43 and 32, of 8 at rank 16 (256) 47 and 30; whole backwards, 6000 rows of 18 at
// rank 40, 4096 x 5120 (648), 101 and 112.
static bool own_columns(const LoraWgrad& p, int parts) {
  const int wide = LORA_WAVES * WGRAD_COLS;
  size_t blocks = 0;
  for (const LoraGrad& g : p.g)
    if (g.out) blocks += (g.C + wide - 1) / wide;
  blocks *= (size_t)std::max(p.NA, (p.T + p.chunk - 1) / p.chunk) * parts;
  return p.T <= 80 * p.NA || blocks >= (p.r > 48 ? 512u : p.r > 16 ? 640u : 768u);
}

static moe_status_t launch_wgrad(const LoraWgrad& p, hipStream_t s) {
  const int wide = std::max(p.g[0].out ? p.g[0].C : 0, p.g[1].out ? p.g[1].C : 0);
  // up to four rank tiles a block: with eight, one wave per SIMD is left, and
  // nothing covers its waits (2000 rows of rank 128: 58 us against 38)
  const int tiles = (p.r + 15) / 16, rt = tiles <= 4 ? tiles : tiles <= 6 ? 3 : 4;
  const int parts = (tiles + rt - 1) / rt;
  const bool own = own_columns(p, parts);
  const int cols = own ? LORA_WAVES * WGRAD_COLS : WGRAD_COLS;
  const dim3 grid((wide + cols - 1) / cols, p.T / p.chunk + p.NA + 1, 2 * parts);
  const dim3 block(64 * LORA_WAVES);
  auto go = [&](auto N) {
    constexpr int RT = decltype(N)::value;
    if (own) hipLaunchKernelGGL((lora_wgrad_kernel<RT, true>), grid, block, 0, s, p);
    else hipLaunchKernelGGL((lora_wgrad_kernel<RT, false>), grid, block, 0, s, p);
  };
  switch (rt) {
    case 1: go(std::integral_constant<int, 1>()); break;
    case 2: go(std::integral_constant<int, 2>()); break;
    case 3: go(std::integral_constant<int, 3>()); break;
    default: go(std::integral_constant<int, 4>()); break;
  }
  const moe_status_t st = launch_status();
  if (st != MOE_OK || p.T <= p.chunk) return st;
  const size_t quads = (size_t)p.r * wide / 4;
  hipLaunchKernelGGL(lora_wgrad_sum_kernel, dim3((unsigned)((quads + 255) / 256), p.NA, 2),
                     dim3(256), 0, s, p);
  return launch_status();
}

static bool lora_sizes_ok(int T, int K, int N, int r, int NA) {
  // (offsets within one adapter's factor are 32-bit; so are positions and tiles)
  return T >= 0 && T <= (1 << 30) && K > 0 && N > 0 && K % 32 == 0 && N % 32 == 0 &&
         K <= (1 << 20) && N <= (1 << 20) && r > 0 && r % 8 == 0 && NA >= 1 &&
         NA < MOE_MAX_EXPERTS;
}

}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_lora_workspace_size(int T, int K, int N, int r, int NA) {
  if (!lora_sizes_ok(T, K, N, r, NA) || T == 0) return 256;
  // the backward's u, and the partial sums of the reduction with more splits or
  // (once those are used up) of the weight gradients' chunks
  const int splits = std::max(lora_splits(T, NA, K, r), lora_splits(T, NA, N, r));
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
  const int splits = lora_splits(a->T, a->NA, a->K, a->r);
  float* part = static_cast<float*>(a->ws);
  const LoraShrink sh = {static_cast<const uint16_t*>(a->x), static_cast<const uint16_t*>(a->A),
                         a->offsets, a->src_row, part, a->T, a->K, a->r, a->NA,
                         lora_chunks(a->K, a->r), splits};
  moe_status_t st = launch_shrink<false>(sh, s);
  if (st != MOE_OK) return st;
  const LoraExpand ex = {part, static_cast<const uint16_t*>(a->B), a->scale, a->offsets, a->src_row,
                         static_cast<const uint16_t*>(a->y), static_cast<uint16_t*>(a->out),
                         a->v_out, a->T, a->N, a->r, a->NA, splits, 0, 1};
  return launch_out<false>(ex, s);
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
  MOE_CHECK_ARG(aligned16(a->dA) && aligned16(a->dB));
  if (a->T > 0) {
    MOE_CHECK_ARG(a->dy && (!want_u || a->B) && (!a->dx_out || a->A) && (!a->dA || a->x) &&
                  (!a->dB || a->v));
    MOE_CHECK_ARG(aligned16(a->x) && aligned16(a->dy) && aligned16(a->A) && aligned16(a->B) &&
                  aligned16(a->v) && aligned16(a->dx) && aligned16(a->dx_out) &&
                  aligned16(a->ws));
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
      const int splits = lora_splits(a->T, a->NA, a->N, a->r);
      const LoraShrink sh = {static_cast<const uint16_t*>(a->dy),
                             static_cast<const uint16_t*>(a->B), a->offsets, a->src_row, part,
                             a->T, a->N, a->r, a->NA, lora_chunks(a->N, a->r), splits};
      moe_status_t st = launch_shrink<true>(sh, s);
      if (st != MOE_OK) return st;
      const LoraExpand ex = {part, static_cast<const uint16_t*>(a->A), a->scale, a->offsets,
                             a->src_row, static_cast<const uint16_t*>(a->dx),
                             static_cast<uint16_t*>(a->dx_out), a->dA ? u : nullptr, a->T, a->K,
                             a->r, a->NA, splits, 1, 1};
      st = launch_out<true>(ex, s);
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
