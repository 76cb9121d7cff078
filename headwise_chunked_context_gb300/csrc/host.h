// Host-side helpers shared by the entry-point files (upipe.cu for the
// attention layer, alst.cu for the sequence-tiled MLP and loss, qk_rope.cu,
// attn_window.cu, embed.cu and residual.cu for what stands around them): argument
// checks, device readiness, TMA tensor maps and launch accounting.  Defined
// in upipe.cu.
#pragma once

#include <atomic>
#include <cstring>
#include <vector>

#include "upipe.h"
#include "upipe_internal.h"

namespace upipe {

bool aligned16(const void* p);
// A bf16 tensor [L, D] given as rows (its head stride says nothing): 16-byte
// alignment of every row, and for a written tensor no element at two places.
inline bool matrix_ok(const upipe_rows* t, int64_t L, int64_t D, bool written) {
  constexpr int64_t kMost = int64_t(1) << 60;  // keeps offsets from overflowing
  if (!t || !t->p || !aligned16(t->p) || t->row < 0 || t->row % 8 != 0) return false;
  return L == 1 || (t->row <= kMost / L && (!written || t->row >= D));
}
// Bound of every device-side wait (UPIPE_SPIN_LIMIT_NS, default 2 s).
uint64_t spin_limit_ns();
// Checks that the current device is an sm_103 part and returns the address
// of its status word; UPIPE_OK or an error code.
int device_ready(int** status);
// bf16 [rows, cols] with leading dimension ld (elements); box 64 x box_rows,
// 128-byte swizzle.
bool map2d(CUtensorMap* m, const void* base, uint64_t cols, uint64_t rows, uint64_t ld, uint32_t box_rows);
// bf16 heads of 128: element (c, row, head) at base + row*row_stride + head*head_stride.
bool map3d(CUtensorMap* m, const void* base, uint64_t rows, uint64_t heads, uint64_t row_stride,
           uint64_t head_stride, uint32_t box_rows);
// bf16 rows of 16: element (c, row, head) at base + (head*rows + row)*16 + c;
// box 16 x box_rows, 32-byte swizzle.
bool map_rows16(CUtensorMap* m, const void* base, uint64_t rows, uint64_t heads, uint32_t box_rows);

// Launch accounting: a counter of every kernel launch, and optional CUDA
// event pairs recorded around each launch on the launching stream.
struct ProfRec {
  int kind;
  cudaEvent_t a, b;
};
extern std::atomic<int64_t> g_launches;
extern std::atomic<bool> g_profile;
extern thread_local bool t_no_profile;
extern std::vector<ProfRec> g_prof;
cudaEvent_t pool_event();

template <class F>
cudaError_t counted(int kind, cudaStream_t st, F&& launch) {
  g_launches.fetch_add(1, std::memory_order_relaxed);
  if (!g_profile.load(std::memory_order_relaxed) || t_no_profile) return launch();
  ProfRec r{kind, pool_event(), pool_event()};
  cudaEventRecord(r.a, st);
  const cudaError_t e = launch();
  cudaEventRecord(r.b, st);
  g_prof.push_back(r);
  return e;
}

// Allows `kernel` `bytes` of dynamic shared memory on the current device, once
// per device: `done`, a bit each, belongs to the kernel.
inline cudaError_t allow_smem(const void* kernel, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  if (cudaError_t e = cudaGetDevice(&dev)) return e;
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes)) return e;
  done.fetch_or(bit, std::memory_order_relaxed);
  return cudaSuccess;
}

// Launches a kernel that may be made ready while the one before it on the stream
// still runs.  Every thread of it begins with after_previous() (sm103_ptx.cuh),
// so that it touches nothing before that one has ended, and reads what kernels
// before it wrote past L1 (__ldcg), which may have been filled earlier; the one
// before allows it by let_next_start().
template <class P>
cudaError_t launch_next(void (*kernel)(P), dim3 grid, dim3 block, size_t smem, cudaStream_t st, const P& p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

// Runs two launches that read nothing of each other's at once: `side` on the
// device's second stream (greatest priority, forked from `st` and joined back
// by events), `own` on `st`; both on `st`, one after the other, while another
// capture holds the second stream.  Both are counted.  UPIPE_OK or an error code.
using LaunchFn = cudaError_t (*)(void* job, cudaStream_t on);
int launch_beside(int side_kind, LaunchFn side, int own_kind, LaunchFn own, void* job, cudaStream_t st);

inline GemmParams gemm_base(int* status, uint64_t limit) {
  GemmParams g;
  std::memset(&g, 0, sizeof(g));
  g.status = status;
  g.limit_ns = limit;
  return g;
}

}  // namespace upipe

#define UPIPE_CU(x)                                \
  do {                                             \
    if ((x) != cudaSuccess) return UPIPE_ERR_CUDA; \
  } while (0)
// Launch expression x on stream `st` (a local of the caller), counted.
#define UPIPE_LAUNCH(kind, x) UPIPE_CU(::upipe::counted(kind, st, [&] { return (x); }))
#define UPIPE_MAP(x)                 \
  do {                               \
    if (!(x)) return UPIPE_ERR_CUDA; \
  } while (0)
