// What carries the residual stream from one sublayer to the next: dropout
// from a counter-based generator, and layer norm (or RMS norm) over the model
// width with the residual sum and dropout in the same pass, forward and
// backward, and their C entry points.
//
// Mathematics, per row of D elements:
//   s = bf16(res + drop(x)),  m = mean(s) (0: RMS),  r = 1 / sqrt(mean((s - m)^2) + eps),
//   n = (s - m) r,  y = w n + b;
// backward, from dy and the gradient ds that reaches s by the residual path:
//   g = w dy,  dres = ds + r (g - mean(g) - n mean(g n)),  dx = drop(dres),
//   dw = sum over rows of dy n,  db = sum over rows of dy.
// The statistics are recomputed from s, which the backward reads in any case.
#include <cmath>
#include <cstring>

#include "host.h"
#include "philox.cuh"
#include "sm103_ptx.cuh"

namespace upipe {
namespace {

using bf16 = __nv_bfloat16;

constexpr int kThreads = 256;

// A [L, D] tensor of bf16 and its row stride in elements.
struct Mat {
  bf16* p;
  int64_t row;
};

struct NormParams {
  int64_t L;
  int D, rms;
  float eps;
  int dropped;
  Drop drop;
  Mat x, res, s, y;      // forward; backward: s is read
  Mat dy, ds, dres, dx;  // backward
  const float *w, *b;
  float* partial;  // backward: [gridDim.x][2][D] shares of dw and db
};

__device__ __forceinline__ void load8(const bf16* p, float (&v)[8]) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  v[0] = bf16_lo(u.x), v[1] = bf16_hi(u.x), v[2] = bf16_lo(u.y), v[3] = bf16_hi(u.y);
  v[4] = bf16_lo(u.z), v[5] = bf16_hi(u.z), v[6] = bf16_lo(u.w), v[7] = bf16_hi(u.w);
}
__device__ __forceinline__ void store8(bf16* p, const float (&v)[8]) {
  st_global_v4(p, pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}

// ---------------------------------------------------------------- dropout

struct DropParams {
  int64_t L;
  int D;
  Drop drop;
  Mat x, res, y;
};

__global__ void __launch_bounds__(kThreads) dropout_kernel(const __grid_constant__ DropParams p) {
  const int per = p.D / 8;
  const int64_t n = p.L * per, stride = static_cast<int64_t>(gridDim.x) * kThreads;
  const uint64_t call = drop_call(p.drop);
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < n; i += stride) {
    const int64_t row = i / per;
    const int col = static_cast<int>(i - row * per) * 8;
    float v[8];
    load8(p.x.p + row * p.x.row + col, v);
    drop8(p.drop, call, static_cast<uint64_t>(row) * p.D + col, v);
    if (p.res.p) {
      float r[8];
      load8(p.res.p + row * p.res.row + col, r);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = __fadd_rn(r[e], v[e]);
    }
    store8(p.y.p + row * p.y.row + col, v);
  }
}

// ------------------------------------------------------------------- norm

// Sums of three numbers over the CTA.
__device__ __forceinline__ float3 block_sum(float3 v, float3* shared) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
    v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
    v.z += __shfl_xor_sync(0xffffffffu, v.z, o);
  }
  __syncthreads();
  if (lane == 0) shared[warp] = v;
  __syncthreads();
  v = shared[0];
#pragma unroll
  for (int i = 1; i < kThreads / 32; ++i) {
    v.x += shared[i].x;
    v.y += shared[i].y;
    v.z += shared[i].z;
  }
  return v;
}

__global__ void __launch_bounds__(kThreads) layer_norm_fwd_kernel(const __grid_constant__ NormParams p) {
  __shared__ float3 shared[kThreads / 32];
  const uint64_t call = p.dropped ? drop_call(p.drop) : 0;
  for (int64_t row = blockIdx.x; row < p.L; row += gridDim.x) {
    const bool sum = p.s.p != nullptr;
    const bf16* s = sum ? p.s.p + row * p.s.row : p.x.p + row * p.x.row;
    float total = 0.f;
    for (int c = threadIdx.x * 8; c < p.D; c += kThreads * 8) {
      float v[8];
      load8(p.x.p + row * p.x.row + c, v);
      if (sum) {
        if (p.dropped) drop8(p.drop, call, static_cast<uint64_t>(row) * p.D + c, v);
        if (p.res.p) {
          float r[8];
          load8(p.res.p + row * p.res.row + c, r);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = __fadd_rn(r[e], v[e]);
        }
        store8(p.s.p + row * p.s.row + c, v);
        load8(s + c, v);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) total += v[e];
    }
    const float m = p.rms ? 0.f : block_sum(make_float3(total, 0.f, 0.f), shared).x / p.D;
    float sq = 0.f;
    for (int c = threadIdx.x * 8; c < p.D; c += kThreads * 8) {
      float v[8];
      load8(s + c, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) sq = fmaf(v[e] - m, v[e] - m, sq);
    }
    const float r = rsqrtf(block_sum(make_float3(sq, 0.f, 0.f), shared).x / p.D + p.eps);
    for (int c = threadIdx.x * 8; c < p.D; c += kThreads * 8) {
      float v[8];
      load8(s + c, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = fmaf((v[e] - m) * r, p.w[c + e], p.b ? p.b[c + e] : 0.f);
      store8(p.y.p + row * p.y.row + c, v);
    }
  }
}

__global__ void __launch_bounds__(kThreads) layer_norm_bwd_kernel(const __grid_constant__ NormParams p) {
  __shared__ float3 shared[kThreads / 32];
  const uint64_t call = p.dropped ? drop_call(p.drop) : 0;
  float* dw = p.partial + static_cast<int64_t>(blockIdx.x) * 2 * p.D;
  float* db = dw + p.D;
  for (int c = threadIdx.x * 8; c < p.D; c += kThreads * 8)
    for (int e = 0; e < 8; ++e) dw[c + e] = db[c + e] = 0.f;
  for (int64_t row = blockIdx.x; row < p.L; row += gridDim.x) {
    const bf16 *s = p.s.p + row * p.s.row, *dy = p.dy.p + row * p.dy.row;
    float total = 0.f;
    for (int c = threadIdx.x * 8; c < p.D; c += kThreads * 8) {
      float v[8];
      load8(s + c, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) total += v[e];
    }
    const float m = p.rms ? 0.f : block_sum(make_float3(total, 0.f, 0.f), shared).x / p.D;
    float3 sums = make_float3(0.f, 0.f, 0.f);  // (s - m)^2, g, g (s - m)
    for (int c = threadIdx.x * 8; c < p.D; c += kThreads * 8) {
      float v[8], g[8];
      load8(s + c, v);
      load8(dy + c, g);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float a = v[e] - m, gw = g[e] * p.w[c + e];
        sums.x = fmaf(a, a, sums.x);
        sums.y += gw;
        sums.z = fmaf(gw, a, sums.z);
      }
    }
    sums = block_sum(sums, shared);
    const float r = rsqrtf(sums.x / p.D + p.eps);
    const float mg = p.rms ? 0.f : sums.y / p.D, k = r * (sums.z / p.D);  // mean(g), mean(g n)
    for (int c = threadIdx.x * 8; c < p.D; c += kThreads * 8) {
      float v[8], g[8], d[8];
      load8(s + c, v);
      load8(dy + c, g);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float n = (v[e] - m) * r;
        dw[c + e] = fmaf(g[e], n, dw[c + e]);
        db[c + e] += g[e];
        d[e] = r * (g[e] * p.w[c + e] - mg - n * k);
      }
      if (p.ds.p) {
        load8(p.ds.p + row * p.ds.row + c, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) d[e] += v[e];
      }
      store8(p.dres.p + row * p.dres.row + c, d);
      if (p.dropped) {
        drop8(p.drop, call, static_cast<uint64_t>(row) * p.D + c, d);
        store8(p.dx.p + row * p.dx.row + c, d);
      }
    }
  }
}

// dw[i] and db[i], the sums over the n rows of partial [n][2][D], in a fixed
// order: thread row j adds rows j, j + 32, ..., then the 32 shares are added.
__global__ void __launch_bounds__(1024) weight_sum_kernel(const float* __restrict__ partial, int n, int D, float* dw,
                                                          float* db) {
  __shared__ float share[32][33];
  const int col = blockIdx.x * 32 + threadIdx.x;  // of 2 D, or D without db
  const int cols = db ? 2 * D : D;
  float g = 0.f;
  if (col < cols)
#pragma unroll 4
    for (int r = threadIdx.y; r < n; r += 32) g += partial[static_cast<int64_t>(r) * 2 * D + col];
  share[threadIdx.y][threadIdx.x] = g;
  __syncthreads();
  g = share[threadIdx.x][threadIdx.y];  // warp y adds column y
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) g += __shfl_xor_sync(0xffffffffu, g, o);
  const int out = blockIdx.x * 32 + threadIdx.y;
  if (threadIdx.x == 0 && out < cols) (out < D ? dw[out] : db[out - D]) = g;
}

// ------------------------------------------------------------------- host

constexpr int kMaxRows = 152 * 8;  // CTAs of the norm's forward
constexpr int kBwdCtas = 152 * 2;

bool norm_ok(const upipe_norm_cfg* c) {
  return c && c->L >= 1 && c->L <= 0x7fffffffLL && c->D >= 8 && c->D <= UPIPE_NORM_MAX_D && c->D % 8 == 0 &&
         (c->rms == 0 || c->rms == 1) && c->eps >= 0.f && std::isfinite(c->eps);
}

bool weight_ok(const float* w) { return w && reinterpret_cast<uintptr_t>(w) % sizeof(float) == 0; }

Mat mat_of(const upipe_rows* t) { return t ? Mat{reinterpret_cast<bf16*>(t->p), t->row} : Mat{nullptr, 0}; }

int bwd_ctas(const upipe_norm_cfg* c) { return static_cast<int>(c->L < kBwdCtas ? c->L : kBwdCtas); }

// The part of a norm's parameters that both directions share.
bool norm_params(const upipe_norm_cfg* c, const upipe_dropout* drop, NormParams* p) {
  std::memset(p, 0, sizeof(*p));
  p->L = c->L;
  p->D = c->D;
  p->rms = c->rms;
  p->eps = c->eps;
  if (!drop) return true;
  p->dropped = 1;
  return drop_of(drop, &p->drop);
}

}  // namespace
}  // namespace upipe

using namespace upipe;

extern "C" {

int upipe_dropout_apply(const upipe_dropout* drop, int64_t L, int32_t D, const upipe_rows* x, const upipe_rows* res,
                        const upipe_rows* y, void* stream) {
  if (!drop || L < 1 || L > 0x7fffffffLL || D < 8 || D % 8 != 0) return UPIPE_ERR_INVALID_ARG;
  if (!matrix_ok(x, L, D, false) || (res && !matrix_ok(res, L, D, false)) || !matrix_ok(y, L, D, true))
    return UPIPE_ERR_INVALID_ARG;
  DropParams p;
  if (!drop_of(drop, &p.drop)) return UPIPE_ERR_INVALID_ARG;
  p.L = L;
  p.D = D;
  p.x = mat_of(x);
  p.res = mat_of(res);
  p.y = mat_of(y);
  int* status = nullptr;
  if (int e = device_ready(&status)) return e;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int64_t need = (L * (D / 8) + kThreads - 1) / kThreads;
  const unsigned grid = static_cast<unsigned>(need < 152 * 8 ? need : 152 * 8);
  UPIPE_LAUNCH(UPIPE_KIND_DROPOUT, (dropout_kernel<<<grid, kThreads, 0, st>>>(p), cudaGetLastError()));
  return UPIPE_OK;
}

int upipe_layer_norm_fwd(const upipe_norm_cfg* c, const upipe_dropout* drop, const upipe_rows* x,
                         const upipe_rows* res, const float* w, const float* b, const upipe_rows* s,
                         const upipe_rows* y, void* stream) {
  if (!norm_ok(c) || !matrix_ok(x, c->L, c->D, false) || !matrix_ok(y, c->L, c->D, true) || !weight_ok(w))
    return UPIPE_ERR_INVALID_ARG;
  if ((res && !matrix_ok(res, c->L, c->D, false)) || (b && !weight_ok(b))) return UPIPE_ERR_INVALID_ARG;
  const bool sum = res || drop;
  if (sum ? !matrix_ok(s, c->L, c->D, true) : s != nullptr) return UPIPE_ERR_INVALID_ARG;
  NormParams p;
  if (!norm_params(c, drop, &p)) return UPIPE_ERR_INVALID_ARG;
  p.x = mat_of(x);
  p.res = mat_of(res);
  p.s = mat_of(s);
  p.y = mat_of(y);
  p.w = w;
  p.b = b;
  int* status = nullptr;
  if (int e = device_ready(&status)) return e;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const unsigned grid = static_cast<unsigned>(c->L < kMaxRows ? c->L : kMaxRows);
  UPIPE_LAUNCH(UPIPE_KIND_LAYER_NORM_FWD, (layer_norm_fwd_kernel<<<grid, kThreads, 0, st>>>(p), cudaGetLastError()));
  return UPIPE_OK;
}

size_t upipe_layer_norm_workspace_bytes(const upipe_norm_cfg* c) {
  return norm_ok(c) ? static_cast<size_t>(bwd_ctas(c)) * 2 * c->D * sizeof(float) : 0;
}

int upipe_layer_norm_bwd(const upipe_norm_cfg* c, const upipe_dropout* drop, const upipe_rows* s, const float* w,
                         const upipe_rows* dy, const upipe_rows* ds, const upipe_rows* dres, const upipe_rows* dx,
                         float* dw, float* db, void* ws, size_t ws_bytes, void* stream) {
  if (!norm_ok(c) || !matrix_ok(s, c->L, c->D, false) || !matrix_ok(dy, c->L, c->D, false) ||
      !matrix_ok(dres, c->L, c->D, true) || !weight_ok(w) || !weight_ok(dw))
    return UPIPE_ERR_INVALID_ARG;
  if ((ds && !matrix_ok(ds, c->L, c->D, false)) || (db && !weight_ok(db))) return UPIPE_ERR_INVALID_ARG;
  if (drop ? !matrix_ok(dx, c->L, c->D, true) : dx != nullptr) return UPIPE_ERR_INVALID_ARG;
  if (!ws || !aligned16(ws)) return UPIPE_ERR_INVALID_ARG;
  if (ws_bytes < upipe_layer_norm_workspace_bytes(c)) return UPIPE_ERR_WS_TOO_SMALL;
  NormParams p;
  if (!norm_params(c, drop, &p)) return UPIPE_ERR_INVALID_ARG;
  p.s = mat_of(s);
  p.dy = mat_of(dy);
  p.ds = mat_of(ds);
  p.dres = mat_of(dres);
  p.dx = mat_of(dx);
  p.w = w;
  p.partial = static_cast<float*>(ws);
  int* status = nullptr;
  if (int e = device_ready(&status)) return e;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int grid = bwd_ctas(c);
  UPIPE_LAUNCH(UPIPE_KIND_LAYER_NORM_BWD, (layer_norm_bwd_kernel<<<grid, kThreads, 0, st>>>(p), cudaGetLastError()));
  const unsigned cols = static_cast<unsigned>(db ? 2 * c->D : c->D);
  UPIPE_LAUNCH(UPIPE_KIND_NORM_SUM, (weight_sum_kernel<<<(cols + 31) / 32, dim3(32, 32), 0, st>>>(p.partial, grid,
                                                                                                 c->D, dw, db),
                                     cudaGetLastError()));
  return UPIPE_OK;
}

}  // extern "C"
