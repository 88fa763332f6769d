// Global gradient norm over many tensors, and clipping by it.
//
//   norm = sqrt(sum over tensors and elements of g^2)
//   c    = min(1, max_norm / (norm + eps)),   out = c g
//
// HBM-bound: the norm reads every element once, the clipping reads it again
// and writes it once (a second read of what fits the last-level cache costs
// less than one from HBM).  Squares are taken and added in float64: at two
// float64 operations per element read the vector units stay far under their
// rate, and no finite float32 gradient overflows or vanishes.
//
// Tensors are passed by value in the kernel arguments, CLIP_BATCH per launch
// (nothing is staged in memory, so a captured graph holds its own list), and
// cut into pieces of CLIP_PIECE elements that the blocks take in turn.  Block
// b keeps one float64 sum in slot b of the workspace: written by the first
// batch, added to by the next (launches of one stream follow each other), and
// summed in slot order by everyone who needs the norm: the same bits each run.
#include "common.hpp"

#include <math.h>

#include <algorithm>
#include <utility>
#include <vector>

namespace moe {

static constexpr int CLIP_BATCH = 96;
static constexpr int CLIP_SLOTS = 1024;
static constexpr int CLIP_PIECE = 16384;
static constexpr int CLIP_THREADS = 256;

struct ClipTensor {
  const void* in;
  void* out;
  int64_t numel;
  int piece0;        // first piece of the tensor within the batch
  uint8_t in_bf16, out_bf16, vec, skip_unit;   // skip_unit: in place, nothing to do for c == 1
};

struct ClipBatch {
  ClipTensor t[CLIP_BATCH];
  int n, pieces;
};

// The tensor that holds piece i of the batch (uniform over the block).
__device__ __forceinline__ int find_tensor(const ClipBatch& b, int i) {
  int lo = 0, hi = b.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (b.t[mid].piece0 <= i) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ double block_sum(double v, double* lds) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  v = 0.0;
#pragma unroll
  for (int i = 0; i < CLIP_THREADS / 64; ++i) v += lds[i];
  return v;
}

__device__ __forceinline__ float load1(const uint16_t* p) { return bf16_bits_to_f32(*p); }
__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ void store1(uint16_t* p, float v) { *p = (uint16_t)f32_to_bf16_bits(v); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }

template <class EL>
__device__ __forceinline__ double piece_squares(const void* base, int64_t i0, int n, bool vec) {
  typedef typename EL::storage S;
  constexpr int V = EL::VEC;
  const S* p = static_cast<const S*>(base) + i0;
  double s = 0.0;
  if (vec) {
    for (int i = threadIdx.x; i < n / V; i += CLIP_THREADS) {
      float v[V];
      unpack_chunk(reinterpret_cast<const u32x4*>(p)[i], v, EL());
#pragma unroll
      for (int q = 0; q < V; ++q) s = fma((double)v[q], (double)v[q], s);
    }
    const int r = n / V * V + threadIdx.x;
    if (r < n) {
      const double v = load1(p + r);
      s = fma(v, v, s);
    }
  } else {
    for (int i = threadIdx.x; i < n; i += CLIP_THREADS) {
      const double v = load1(p + i);
      s = fma(v, v, s);
    }
  }
  return s;
}

__global__ void __launch_bounds__(CLIP_THREADS) clip_squares_kernel(const ClipBatch b, int first,
                                                                    double* __restrict__ slots) {
  __shared__ double lds[CLIP_THREADS / 64];
  double s = 0.0;
  for (int i = blockIdx.x; i < b.pieces; i += gridDim.x) {
    const ClipTensor& t = b.t[find_tensor(b, i)];
    const int64_t i0 = (int64_t)(i - t.piece0) * CLIP_PIECE;
    const int n = (int)min((int64_t)CLIP_PIECE, t.numel - i0);
    s += t.in_bf16 ? piece_squares<BF16>(t.in, i0, n, t.vec)
                   : piece_squares<F32>(t.in, i0, n, t.vec);
  }
  s = block_sum(s, lds);
  if (threadIdx.x == 0) slots[blockIdx.x] = first ? s : slots[blockIdx.x] + s;
}

// The norm, from the slots: thread i adds slots i, i + CLIP_THREADS, ...
__device__ __forceinline__ double norm_of_slots(const double* slots, int nslots, double* lds) {
  double s = 0.0;
  for (int i = threadIdx.x; i < nslots; i += CLIP_THREADS) s += slots[i];
  return sqrt(block_sum(s, lds));
}

__global__ void __launch_bounds__(CLIP_THREADS) clip_norm_kernel(const double* __restrict__ slots,
                                                                 int nslots,
                                                                 float* __restrict__ norm) {
  __shared__ double lds[CLIP_THREADS / 64];
  const double v = norm_of_slots(slots, nslots, lds);
  if (threadIdx.x == 0) *norm = (float)v;
}

template <class IN, class OUT>
__device__ __forceinline__ void piece_scale(const void* in, void* out, int64_t i0, int n, bool vec,
                                            float c) {
  typedef typename IN::storage SI;
  typedef typename OUT::storage SO;
  // (no restrict: in and out are one tensor when clipping in place)
  const SI* p = static_cast<const SI*>(in) + i0;
  SO* o = static_cast<SO*>(out) + i0;
  int done = 0;
  if (vec) {
    done = n / 4 * 4;
    for (int i = threadIdx.x; i < n / 4; i += CLIP_THREADS) {
      float v[4];
      load4(p + 4 * i, v);
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] *= c;
      store4(o + 4 * i, v);
    }
  }
  for (int i = done + threadIdx.x; i < n; i += CLIP_THREADS) store1(o + i, load1(p + i) * c);
}

__global__ void __launch_bounds__(CLIP_THREADS) clip_scale_kernel(const ClipBatch b, double max_norm,
                                                                  double eps,
                                                                  const double* __restrict__ slots,
                                                                  int nslots, float* norm) {
  __shared__ double lds[CLIP_THREADS / 64];
  const double nv = norm_of_slots(slots, nslots, lds);
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)nv;
  const double cd = max_norm / (nv + eps);
  const float c = cd >= 1.0 ? 1.0f : (float)cd;       // a NaN norm gives NaN everywhere
  for (int i = blockIdx.x; i < b.pieces; i += gridDim.x) {
    const ClipTensor& t = b.t[find_tensor(b, i)];
    if (t.skip_unit && c == 1.0f) continue;
    const int64_t i0 = (int64_t)(i - t.piece0) * CLIP_PIECE;
    const int n = (int)min((int64_t)CLIP_PIECE, t.numel - i0);
    if (t.in_bf16) {
      if (t.out_bf16) piece_scale<BF16, BF16>(t.in, t.out, i0, n, t.vec, c);
      else piece_scale<BF16, F32>(t.in, t.out, i0, n, t.vec, c);
    } else {
      if (t.out_bf16) piece_scale<F32, BF16>(t.in, t.out, i0, n, t.vec, c);
      else piece_scale<F32, F32>(t.in, t.out, i0, n, t.vec, c);
    }
  }
}

static size_t tensor_bytes(int64_t numel, int dtype) { return (size_t)numel * dtype_size(dtype); }

// Checks the list; with `outs`, also that no output shares memory with another
// tensor, the norm or the workspace (its own input only where the two are the
// same tensor).
static moe_status_t clip_check(const moe_tensor_t* list, int n, bool outs, const float* norm,
                               const void* ws) try {
  MOE_CHECK_ARG(n >= 0 && (n == 0 || list) && norm && ws && aligned16(ws));
  struct Range {
    uintptr_t lo, hi;
    bool write;
  };
  std::vector<Range> spans;
  if (outs) {
    spans.reserve(2 * (size_t)n + 2);
    const uintptr_t nm = reinterpret_cast<uintptr_t>(norm), w = reinterpret_cast<uintptr_t>(ws);
    spans.push_back({nm, nm + sizeof(float), true});
    spans.push_back({w, w + CLIP_SLOTS * sizeof(double), true});
  }
  for (int i = 0; i < n; ++i) {
    const moe_tensor_t& t = list[i];
    MOE_CHECK_ARG(t.numel >= 0 && t.numel < ((int64_t)1 << 43) && valid_dtype(t.dtype));
    if (t.numel == 0) continue;
    const uintptr_t in = reinterpret_cast<uintptr_t>(t.data);
    MOE_CHECK_ARG(in && in % dtype_size(t.dtype) == 0);
    if (!outs) continue;
    const uintptr_t out = reinterpret_cast<uintptr_t>(t.out);
    MOE_CHECK_ARG(valid_dtype(t.out_dtype) && out && out % dtype_size(t.out_dtype) == 0);
    spans.push_back({out, out + tensor_bytes(t.numel, t.out_dtype), true});
    if (in != out || t.dtype != t.out_dtype)
      spans.push_back({in, in + tensor_bytes(t.numel, t.dtype), false});
  }
  std::sort(spans.begin(), spans.end(), [](const Range& a, const Range& b) { return a.lo < b.lo; });
  // furthest end of the spans so far: of the written ones, and of all of them
  uintptr_t wend = 0, end = 0;
  for (const Range& s : spans) {
    MOE_CHECK_ARG(s.lo >= wend && !(s.write && s.lo < end));
    end = std::max(end, s.hi);
    if (s.write) wend = std::max(wend, s.hi);
  }
  return MOE_OK;
} catch (...) {
  return MOE_ERR_HIP;      // host memory for the check ran out
}

// Calls launch(batch, first) for the list in batches; at least once.
template <class F>
static moe_status_t clip_batches(const moe_tensor_t* list, int n, bool outs, F&& launch) {
  ClipBatch b;
  b.n = b.pieces = 0;
  bool first = true;
  for (int i = 0; i < n; ++i) {
    const moe_tensor_t& t = list[i];
    const int64_t left = (t.numel + CLIP_PIECE - 1) / CLIP_PIECE;
    if (left == 0) continue;
    if (b.n == CLIP_BATCH || b.pieces + left > INT32_MAX / 2) {
      const moe_status_t st = launch(b, first);
      if (st != MOE_OK) return st;
      first = false;
      b.n = b.pieces = 0;
    }
    ClipTensor& c = b.t[b.n++];
    c.in = t.data;
    c.out = outs ? t.out : nullptr;
    c.numel = t.numel;
    c.piece0 = b.pieces;
    c.in_bf16 = t.dtype == MOE_BF16;
    c.out_bf16 = outs && t.out_dtype == MOE_BF16;
    c.vec = aligned16(t.data) && (!outs || aligned16(t.out));
    c.skip_unit = outs && t.data == t.out && t.dtype == t.out_dtype;
    b.pieces += (int)left;
  }
  if (b.n > 0 || first) return launch(b, first);
  return MOE_OK;
}

// Slots in use: as many as the largest batch has pieces, at most CLIP_SLOTS.
static int clip_slots(const moe_tensor_t* list, int n) {
  int64_t pieces = 0;
  for (int i = 0; i < n; ++i) pieces += (list[i].numel + CLIP_PIECE - 1) / CLIP_PIECE;
  return (int)std::max<int64_t>(1, std::min<int64_t>(pieces, CLIP_SLOTS));
}

static moe_status_t clip_squares(const moe_tensor_t* list, int n, int nslots, double* slots,
                                 hipStream_t s) {
  return clip_batches(list, n, false, [&](const ClipBatch& b, bool first) {
    // the first batch writes every slot; later ones add to those they have pieces for
    const int grid = first ? nslots : std::min(nslots, b.pieces);
    hipLaunchKernelGGL(clip_squares_kernel, dim3(grid), dim3(CLIP_THREADS), 0, s, b, (int)first,
                       slots);
    return launch_status();
  });
}

}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_grad_norm_workspace_size(int n) {
  (void)n;
  return CLIP_SLOTS * sizeof(double);
}

moe_status_t moe_grad_norm(const moe_tensor_t* tensors, int n, float* norm, void* ws,
                           size_t ws_bytes, void* stream) {
  moe_status_t st = clip_check(tensors, n, false, norm, ws);
  if (st != MOE_OK) return st;
  if (ws_bytes < moe_grad_norm_workspace_size(n)) return MOE_ERR_WORKSPACE;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  double* slots = static_cast<double*>(ws);
  const int nslots = clip_slots(tensors, n);
  st = clip_squares(tensors, n, nslots, slots, s);
  if (st != MOE_OK) return st;
  hipLaunchKernelGGL(clip_norm_kernel, dim3(1), dim3(CLIP_THREADS), 0, s, slots, nslots, norm);
  return launch_status();
}

moe_status_t moe_clip_grad_norm(const moe_tensor_t* tensors, int n, double max_norm, double eps,
                                float* norm, void* ws, size_t ws_bytes, void* stream) {
  MOE_CHECK_ARG(max_norm >= 0.0 && eps > 0.0 && isfinite(eps));
  moe_status_t st = clip_check(tensors, n, true, norm, ws);
  if (st != MOE_OK) return st;
  if (ws_bytes < moe_grad_norm_workspace_size(n)) return MOE_ERR_WORKSPACE;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  double* slots = static_cast<double*>(ws);
  const int nslots = clip_slots(tensors, n);
  st = clip_squares(tensors, n, nslots, slots, s);
  if (st != MOE_OK) return st;
  return clip_batches(tensors, n, true, [&](const ClipBatch& b, bool first) {
    const int grid = std::max(1, std::min(b.pieces, 2 * CLIP_SLOTS));
    hipLaunchKernelGGL(clip_scale_kernel, dim3(grid), dim3(CLIP_THREADS), 0, s, b, max_norm, eps,
                       slots, nslots, first ? norm : nullptr);
    return launch_status();
  });
}

}  // extern "C"
