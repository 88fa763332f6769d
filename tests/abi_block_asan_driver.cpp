// Host-side argument handling of the block norms, the gradient norm and the adapters
// (include/moe.h) under AddressSanitizer, with no GPU: every call here has an argument that
// must be refused before anything is enqueued, argument structs are passed at every size up
// to their own, allocated at exactly that size, and lists of tensors at exactly their length.
//
// Built and run by tests/test_abi_block_asan.py.
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <initializer_list>

#include "moe.h"

static int g_fail = 0;
#define EXPECT(cond)                                      \
  do {                                                    \
    if (!(cond)) {                                        \
      std::printf("FAIL line %d: %s\n", __LINE__, #cond); \
      ++g_fail;                                           \
    }                                                     \
  } while (0)

// 16-byte aligned addresses, 1 MiB apart, that are never dereferenced on the host
static void* P(int i) { return reinterpret_cast<void*>((uintptr_t)(i + 1) << 20); }
static float* F(int i) { return static_cast<float*>(P(i)); }

// Every size short of the whole struct is refused, without a read past it.
template <class A>
static void sweep(const char* what, moe_status_t (*fn)(const A*, void*), const A& full) {
  for (size_t n = sizeof(size_t); n < sizeof(A); n += 4) {
    char* p = static_cast<char*>(std::malloc(n));
    std::memcpy(p, &full, n);
    std::memcpy(p, &n, sizeof n);
    const moe_status_t st = fn(reinterpret_cast<const A*>(p), nullptr);
    std::free(p);
    if (st != MOE_ERR_INVALID_ARG) {
      std::printf("FAIL %s size %zu: status %d\n", what, n, (int)st);
      ++g_fail;
    }
  }
  EXPECT(fn(nullptr, nullptr) == MOE_ERR_INVALID_ARG);
}

static void norms() {
  moe_block_norm_fwd_args_t f{};
  f.struct_size = sizeof f;
  f.dtype = MOE_BF16; f.T = 4; f.d = 64; f.res_scale = 1.0f; f.eps = 1e-6f;
  f.h = P(0); f.y = P(1); f.w_pre = F(2); f.h_out = P(3); f.x_out = P(4);
  sweep("block_norm_fwd", moe_block_norm_fwd, f);
  auto g = f;
  g.x_out = P(3);
  EXPECT(moe_block_norm_fwd(&g, nullptr) == MOE_ERR_INVALID_ARG);
  g = f; g.T = INT32_MAX;
  EXPECT(moe_block_norm_fwd(&g, nullptr) == MOE_ERR_INVALID_ARG);
  g = f; g.T = INT32_MAX / 2; g.k = 4; g.row_map = reinterpret_cast<int32_t*>(P(5));
  EXPECT(moe_block_norm_fwd(&g, nullptr) == MOE_ERR_INVALID_ARG);
  g = f; g.d = INT32_MAX / 16 * 16;
  EXPECT(moe_block_norm_fwd(&g, nullptr) == MOE_ERR_UNSUPPORTED);
  moe_block_norm_bwd_args_t b{};
  b.struct_size = sizeof b;
  b.dtype = MOE_F32; b.T = 4; b.d = 64; b.res_scale = 1.0f; b.eps = 1e-6f;
  b.h1 = P(0); b.dx = P(1); b.w_pre = F(2); b.dh = P(3); b.dw_pre = F(4);
  sweep("block_norm_bwd", moe_block_norm_bwd, b);
  EXPECT(moe_block_norm_bwd(&b, nullptr) == MOE_ERR_WORKSPACE);
  b.ws = P(5);
  for (int d = 4; d <= 16384; d *= 2)
    for (int T = 1; T < 1 << 20; T = 3 * T + 1) {
      b.T = T; b.d = d; b.ws_bytes = moe_block_norm_bwd_workspace_size(T, d) - 1;
      EXPECT(moe_block_norm_bwd(&b, nullptr) == MOE_ERR_WORKSPACE);
    }
  EXPECT(moe_block_norm_bwd_workspace_size(-1, 64) == 0);
  EXPECT(moe_block_norm_bwd_workspace_size(4, INT32_MAX) > 0);
}

// Lists of n tensors, the last one bad, on the heap at exactly their length.
static void lists() {
  const size_t nb = moe_grad_norm_workspace_size(0);
  for (int n : {1, 2, 139, 140, 141, 1000}) {
    auto* t = static_cast<moe_tensor_t*>(std::malloc(n * sizeof(moe_tensor_t)));
    for (int i = 0; i < n; ++i) t[i] = {P(2 * i), P(2 * i + 1), 1000 + i, MOE_F32, MOE_BF16};
    auto both = [&](moe_status_t want_norm) {
      EXPECT(moe_clip_grad_norm(t, n, 1.0, 1e-6, F(4000), P(4001), nb, nullptr) ==
             MOE_ERR_INVALID_ARG);
      if (want_norm != MOE_OK)
        EXPECT(moe_grad_norm(t, n, F(4000), P(4001), nb, nullptr) == want_norm);
    };
    moe_tensor_t& last = t[n - 1];
    const moe_tensor_t good = last;
    last.numel = -1; both(MOE_ERR_INVALID_ARG); last = good;
    last.numel = INT64_MAX; both(MOE_ERR_INVALID_ARG); last = good;
    last.data = nullptr; both(MOE_ERR_INVALID_ARG); last = good;
    last.dtype = 77; both(MOE_ERR_INVALID_ARG); last = good;
    last.out = const_cast<void*>(last.data); both(MOE_OK); last = good;         // in place, of another type
    last.out = P(4001); both(MOE_OK); last = good;           // the workspace
    if (n > 1) { last.out = t[0].out; both(MOE_OK); last = good; }
    EXPECT(moe_clip_grad_norm(t, n, 1.0, 1e-6, F(4000), P(4001), nb - 1, nullptr) ==
           MOE_ERR_WORKSPACE);
    EXPECT(moe_grad_norm(t, n, F(4000), P(4001), nb - 1, nullptr) == MOE_ERR_WORKSPACE);
    std::free(t);
  }
  EXPECT(moe_grad_norm(nullptr, 1, F(0), P(1), nb, nullptr) == MOE_ERR_INVALID_ARG);
  EXPECT(moe_grad_norm(nullptr, -1, F(0), P(1), nb, nullptr) == MOE_ERR_INVALID_ARG);
}

static void adapters() {
  moe_lora_fwd_args_t f{};
  f.struct_size = sizeof f;
  f.dtype = MOE_BF16; f.T = 8; f.K = 64; f.N = 96; f.r = 16; f.NA = 3;
  f.x = P(0); f.A = P(1); f.B = P(2); f.offsets = reinterpret_cast<int32_t*>(P(3));
  f.y = P(4); f.out = P(5);
  sweep("lora_fwd", moe_lora_fwd, f);
  EXPECT(moe_lora_fwd(&f, nullptr) == MOE_ERR_WORKSPACE);
  moe_lora_bwd_args_t b{};
  b.struct_size = sizeof b;
  b.dtype = MOE_BF16; b.T = 8; b.K = 64; b.N = 96; b.r = 16; b.NA = 3;
  b.x = P(0); b.A = P(1); b.B = P(2); b.offsets = reinterpret_cast<int32_t*>(P(3));
  b.dy = P(4); b.v = F(5); b.dx_out = P(6); b.dA = F(7); b.dB = F(8);
  sweep("lora_bwd", moe_lora_bwd, b);
  EXPECT(moe_lora_bwd(&b, nullptr) == MOE_ERR_WORKSPACE);
  f.ws = b.ws = P(9);
  for (int T : {1, 63, 64, 1000, 1025, 9000, 1 << 30})
    for (int r : {8, 64, 72, 128})
      for (int NA : {1, 64, 1023}) {
        f.T = b.T = T; f.r = b.r = r; f.NA = b.NA = NA;
        f.ws_bytes = b.ws_bytes = moe_lora_workspace_size(T, 64, 96, r, NA) - 1;
        EXPECT(moe_lora_fwd(&f, nullptr) == MOE_ERR_WORKSPACE);
        EXPECT(moe_lora_bwd(&b, nullptr) == MOE_ERR_WORKSPACE);
      }
  for (int bad : {0, -8, 12, INT32_MAX}) EXPECT(moe_lora_workspace_size(8, 64, 96, bad, 3) == 256);
}

int main() {
  norms();
  lists();
  adapters();
  if (g_fail == 0) std::printf("abi host checks passed\n");
  return g_fail != 0;
}
