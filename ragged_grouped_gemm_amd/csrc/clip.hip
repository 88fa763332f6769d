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
// cut into pieces that the blocks take in turn: of up to 32768 elements, fewer
// where the whole is small, so that about 1024 blocks share it.  Block b keeps
// one float64 sum in slot b of the workspace: written by the first batch, added
// to by the next (launches of one stream follow each other), and summed in slot
// order by everyone who needs the norm: the same bits each run.
//
// The clipping walks the pieces from the last to the first, so that it begins
// with what the norm's pass left in the last-level cache.
//
// Measured: 0.7 GB of bf16 in 49 tensors, norm alone 119 us (5.9 TB/s; a large copy
// reaches 4.9); 3.2 GB of float32 into 1.6 GB of bf16 1412 us (5.6 TB/s of the 8 GB
// that two passes move); 129 tensors of 22 MB together 18 us in two launches.
#include "common.hpp"

#include <math.h>

#include <algorithm>
#include <utility>
#include <vector>

namespace moe {

static constexpr int CLIP_BATCH = 140;      // (4096 bytes of kernel arguments)
static constexpr int CLIP_SLOTS = 1024;
static constexpr int CLIP_MIN_PIECE = 4096, CLIP_MAX_PIECE = 32768;
static constexpr int CLIP_THREADS = 256;
static constexpr int64_t CLIP_MAX_NUMEL = (int64_t)1 << 42;

struct ClipTensor {
  const void* in;
  void* out;
  // elements, and the flags from bit 48 on
  int64_t numel_flags;
  __host__ __device__ int64_t numel() const { return numel_flags & (((int64_t)1 << 48) - 1); }
  __host__ __device__ bool flag(int f) const { return numel_flags >> (48 + f) & 1; }
};
enum { CLIP_IN_BF16, CLIP_OUT_BF16, CLIP_VEC, CLIP_SKIP_UNIT };   // SKIP_UNIT: in place

struct ClipBatch {
  ClipTensor t[CLIP_BATCH];
  int piece0[CLIP_BATCH];   // first piece of each tensor within the batch
  int n, pieces, piece;     // elements per piece
};
static_assert(sizeof(ClipBatch) + 64 <= 4096, "kernel arguments");

// The tensor that holds piece i of the batch (uniform over the block): every wave
// counts the tensors that start at or before it.
__device__ __forceinline__ int find_tensor(const ClipBatch& b, int i) {
  const int lane = threadIdx.x & 63;
  int n = 0;
#pragma unroll
  for (int k = 0; k < CLIP_BATCH; k += 64)
    n += __popcll(__ballot(k + lane < b.n && b.piece0[min(k + lane, CLIP_BATCH - 1)] <= i));
  return n - 1;
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

// Sum of squares of n elements from p: 16-byte chunks, four loads in flight.
template <class EL>
__device__ __forceinline__ double piece_squares(const void* base, int64_t i0, int n, bool vec) {
  typedef typename EL::storage S;
  constexpr int V = EL::VEC;
  const S* p = static_cast<const S*>(base) + i0;
  double s[2] = {0.0, 0.0};
  int done = 0;
  if (vec) {
    const u32x4* c = reinterpret_cast<const u32x4*>(p);
    const int chunks = n / V;
    done = chunks * V;
    auto add = [&](const u32x4& raw) {
      float v[V];
      unpack_chunk(raw, v, EL());
#pragma unroll
      for (int q = 0; q < V; ++q) s[q & 1] = fma((double)v[q], (double)v[q], s[q & 1]);
    };
    int i = threadIdx.x;
    for (; i + 3 * CLIP_THREADS < chunks; i += 4 * CLIP_THREADS) {
      u32x4 raw[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) raw[k] = c[i + k * CLIP_THREADS];
#pragma unroll
      for (int k = 0; k < 4; ++k) add(raw[k]);
    }
    for (; i < chunks; i += CLIP_THREADS) add(c[i]);
  }
  for (int i = done + threadIdx.x; i < n; i += CLIP_THREADS) {
    const double v = load1(p + i);
    s[0] = fma(v, v, s[0]);
  }
  return s[0] + s[1];
}

__global__ void __launch_bounds__(CLIP_THREADS) clip_squares_kernel(const ClipBatch b, int first,
                                                                    double* __restrict__ slots) {
  __shared__ double lds[CLIP_THREADS / 64];
  double s = 0.0;
  for (int i = blockIdx.x; i < b.pieces; i += gridDim.x) {
    const int k = find_tensor(b, i);
    const ClipTensor& t = b.t[k];
    const int64_t i0 = (int64_t)(i - b.piece0[k]) * b.piece;
    const int n = (int)min((int64_t)b.piece, t.numel() - i0);
    const bool vec = t.flag(CLIP_VEC);
    s += t.flag(CLIP_IN_BF16) ? piece_squares<BF16>(t.in, i0, n, vec)
                              : piece_squares<F32>(t.in, i0, n, vec);
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

// Four values rounded to the storage type, past the caches: nothing reads them
// again soon, and what the norm's pass left there is still wanted.
__device__ __forceinline__ void stream4(uint16_t* p, const float* v) {
  typedef float f32x4v __attribute__((ext_vector_type(4)));
  typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
  const f32x4v f = {v[0], v[1], v[2], v[3]};
  __builtin_nontemporal_store(__builtin_bit_cast(u32x2, __builtin_convertvector(f, bf16x4)),
                              reinterpret_cast<u32x2*>(p));
}
__device__ __forceinline__ void stream4(float* p, const float* v) {
  const f32x4 f = {v[0], v[1], v[2], v[3]};
  __builtin_nontemporal_store(f, reinterpret_cast<f32x4*>(p));
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
    constexpr int U = 4;               // loads in flight
    const int quads = n / 4;
    done = quads * 4;
    int i = threadIdx.x;
    for (; i + (U - 1) * CLIP_THREADS < quads; i += U * CLIP_THREADS) {
      float v[U][4];
#pragma unroll
      for (int k = 0; k < U; ++k) load4(p + 4 * (i + k * CLIP_THREADS), v[k]);
#pragma unroll
      for (int k = 0; k < U; ++k) {
#pragma unroll
        for (int q = 0; q < 4; ++q) v[k][q] *= c;
        stream4(o + 4 * (i + k * CLIP_THREADS), v[k]);
      }
    }
    for (; i < quads; i += CLIP_THREADS) {
      float v[4];
      load4(p + 4 * i, v);
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] *= c;
      stream4(o + 4 * i, v);
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
  // (an infinite max_norm never clips, an infinite norm neither)
  const double cd = isinf(max_norm) && isinf(nv) ? 1.0 : max_norm / (nv + eps);
  const float c = cd >= 1.0 ? 1.0f : (float)cd;       // a NaN norm gives NaN everywhere
  for (int i = blockIdx.x; i < b.pieces; i += gridDim.x) {
    const int k = find_tensor(b, i);
    const ClipTensor& t = b.t[k];
    if (t.flag(CLIP_SKIP_UNIT) && c == 1.0f) continue;
    // the tensor's pieces from its last one on
    const int64_t i0 = ((t.numel() - 1) / b.piece - (i - b.piece0[k])) * b.piece;
    const int n = (int)min((int64_t)b.piece, t.numel() - i0);
    const bool vec = t.flag(CLIP_VEC), out_bf16 = t.flag(CLIP_OUT_BF16);
    if (t.flag(CLIP_IN_BF16)) {
      if (out_bf16) piece_scale<BF16, BF16>(t.in, t.out, i0, n, vec, c);
      else piece_scale<BF16, F32>(t.in, t.out, i0, n, vec, c);
    } else {
      if (out_bf16) piece_scale<F32, BF16>(t.in, t.out, i0, n, vec, c);
      else piece_scale<F32, F32>(t.in, t.out, i0, n, vec, c);
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
    MOE_CHECK_ARG(t.numel >= 0 && t.numel < CLIP_MAX_NUMEL && valid_dtype(t.dtype));
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

// Elements per piece, and the slots in use: one per piece up to CLIP_SLOTS.
struct ClipPlan {
  int piece, slots;
};
static ClipPlan clip_plan(const moe_tensor_t* list, int n) {
  double total = 0.0;      // (a sum of sizes may pass 64 bits)
  for (int i = 0; i < n; ++i) total += (double)list[i].numel;
  const double share = total / CLIP_SLOTS;
  ClipPlan p;
  p.piece = share >= CLIP_MAX_PIECE
                ? CLIP_MAX_PIECE
                : std::max(CLIP_MIN_PIECE, ((int)share + 1023) / 1024 * 1024);
  int64_t pieces = 0;
  for (int i = 0; i < n && pieces < CLIP_SLOTS; ++i)
    pieces += (list[i].numel + p.piece - 1) / p.piece;
  p.slots = (int)std::max<int64_t>(1, std::min<int64_t>(pieces, CLIP_SLOTS));
  return p;
}

// Calls launch(batch, first) for the list in batches, at least once: from the
// front for the norm, from the back for the clipping (outs).
template <class F>
static moe_status_t clip_batches(const moe_tensor_t* list, int n, int piece, bool outs, F&& launch) {
  ClipBatch b;
  b.piece = piece;
  b.n = b.pieces = 0;
  bool first = true;
  for (int i = 0; i < n; ++i) {
    const moe_tensor_t& t = outs ? list[n - 1 - i] : list[i];
    const int64_t left = (t.numel + piece - 1) / piece;
    if (left == 0) continue;
    if (b.n == CLIP_BATCH || b.pieces + left > INT32_MAX / 2) {
      const moe_status_t st = launch(b, first);
      if (st != MOE_OK) return st;
      first = false;
      b.n = b.pieces = 0;
    }
    const bool vec = aligned16(t.data) && (!outs || aligned16(t.out));
    const bool inplace = outs && t.data == t.out && t.dtype == t.out_dtype;
    const int64_t flags = (int64_t)(t.dtype == MOE_BF16) << CLIP_IN_BF16 |
                          (int64_t)(outs && t.out_dtype == MOE_BF16) << CLIP_OUT_BF16 |
                          (int64_t)vec << CLIP_VEC | (int64_t)inplace << CLIP_SKIP_UNIT;
    b.piece0[b.n] = b.pieces;
    b.t[b.n++] = {t.data, outs ? t.out : nullptr, t.numel | flags << 48};
    b.pieces += (int)left;
  }
  if (b.n > 0 || first) return launch(b, first);
  return MOE_OK;
}

static moe_status_t clip_squares(const moe_tensor_t* list, int n, const ClipPlan& plan,
                                 double* slots, hipStream_t s) {
  return clip_batches(list, n, plan.piece, false, [&](const ClipBatch& b, bool first) {
    // the first batch writes every slot; later ones add to those they have pieces for
    const int grid = first ? plan.slots : std::min(plan.slots, b.pieces);
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
  const ClipPlan plan = clip_plan(tensors, n);
  st = clip_squares(tensors, n, plan, slots, s);
  if (st != MOE_OK) return st;
  hipLaunchKernelGGL(clip_norm_kernel, dim3(1), dim3(CLIP_THREADS), 0, s, slots, plan.slots, norm);
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
  const ClipPlan plan = clip_plan(tensors, n);
  st = clip_squares(tensors, n, plan, slots, s);
  if (st != MOE_OK) return st;
  return clip_batches(tensors, n, plan.piece, true, [&](const ClipBatch& b, bool first) {
    const int grid = std::max(1, std::min(b.pieces, 2 * CLIP_SLOTS));
    hipLaunchKernelGGL(clip_scale_kernel, dim3(grid), dim3(CLIP_THREADS), 0, s, b, max_norm, eps,
                       slots, plan.slots, first ? norm : nullptr);
    return launch_status();
  });
}

}  // extern "C"
