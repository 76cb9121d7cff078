// Token embedding and the gradient of its table, and their C entry points.
//
// Mathematics: y_i = bf16(scale W[t_i]); a negative token reads zeros and
// leaves no gradient, a token >= V reads NaN and leaves none.  The gradient is
// dW[v] = scale (sum over i with t_i = v of dy_i), in fp32.
//
// The gradient's sums have one order whatever runs when: the tokens are sorted
// by a stable radix sort (9 bits a pass), so that a row's positions stand
// behind one another in ascending order.
#include <cmath>
#include <cstring>

#include "host.h"
#include "sm103_ptx.cuh"

namespace upipe {
namespace {

using bf16 = __nv_bfloat16;

constexpr int kThreads = 256;
constexpr int kDigit = 9;
constexpr int kBins = 1 << kDigit;
constexpr int kSortThreads = kBins;  // a thread per bin
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kMaxTiles = 304;

struct EmbedParams {
  int64_t L;
  int V, D;
  int wide, master;  // 64-bit tokens, fp32 table
  float scale;
  const void* tokens;
  const void* table;
  const bf16* dy;
  int64_t row;  // row stride of y or dy
  bf16* y;
  float* dW;
  int add;
};

__device__ __forceinline__ int64_t token_at(const void* tokens, int wide, int64_t i) {
  return wide ? static_cast<const int64_t*>(tokens)[i] : static_cast<const int32_t*>(tokens)[i];
}

__global__ void __launch_bounds__(kThreads) embed_fwd_kernel(const __grid_constant__ EmbedParams p) {
  for (int64_t i = blockIdx.x; i < p.L; i += gridDim.x) {
    const int64_t t = token_at(p.tokens, p.wide, i);
    bf16* y = p.y + i * p.row;
    const float fill = t < 0 ? 0.f : __int_as_float(0x7fc00000);
    const bool real = t >= 0 && t < p.V;
    for (int c = threadIdx.x * 8; c < p.D; c += kThreads * 8) {
      float v[8];
      if (!real) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = fill;
      } else if (p.master) {
        const float4* w = reinterpret_cast<const float4*>(static_cast<const float*>(p.table) + t * p.D + c);
        const float4 a = w[0], b = w[1];
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
      } else {
        const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const bf16*>(p.table) + t * p.D + c);
        v[0] = bf16_lo(u.x), v[1] = bf16_hi(u.x), v[2] = bf16_lo(u.y), v[3] = bf16_hi(u.y);
        v[4] = bf16_lo(u.z), v[5] = bf16_hi(u.z), v[6] = bf16_lo(u.w), v[7] = bf16_hi(u.w);
      }
      if (real) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= p.scale;
      }
      st_global_v4(y + c, pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                   pack_bf16x2(v[6], v[7]));
    }
  }
}

// ------------------------------------------------------------------- sort

// One pass of the sort: keys by `bits` bits from `shift` on.  The first pass
// reads the tokens (those without a row get key V, behind all rows), later
// passes the (key, position) pairs of the pass before.
struct SortParams {
  int64_t L, tile;  // tokens per CTA, a multiple of 32 kSortWarps
  int tiles, V, wide, first, shift, bits;
  const void* tokens;
  const int2* in;
  int2* out;
  int32_t* counts;  // [tiles][kBins]
};

__device__ __forceinline__ int2 sort_item(const SortParams& p, int64_t i) {
  if (!p.first) return p.in[i];
  const int64_t t = token_at(p.tokens, p.wide, i);
  return make_int2(t >= 0 && t < p.V ? static_cast<int>(t) : p.V, static_cast<int>(i));
}

// Each warp counts the digits of its own part of the tile into its own row.
__device__ __forceinline__ void count_digits(const SortParams& p, int (*hist)[kBins]) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < kSortWarps * kBins; i += kSortThreads) (&hist[0][0])[i] = 0;
  __syncthreads();
  const int64_t part = p.tile / kSortWarps, from = blockIdx.x * p.tile + warp * part;
  for (int64_t i = from + lane; i < from + part; i += 32) {
    if (i < p.L) atomicAdd(&hist[warp][(sort_item(p, i).x >> p.shift) & ((1 << p.bits) - 1)], 1);
  }
  __syncthreads();
}

__global__ void __launch_bounds__(kSortThreads) embed_count_kernel(const __grid_constant__ SortParams p) {
  __shared__ int hist[kSortWarps][kBins];
  count_digits(p, hist);
  int n = 0;
#pragma unroll
  for (int w = 0; w < kSortWarps; ++w) n += hist[w][threadIdx.x];
  p.counts[static_cast<int64_t>(blockIdx.x) * kBins + threadIdx.x] = n;
}

// Where the tile's tokens go: behind all smaller digits, behind the same digit
// of earlier tiles, of earlier warps, of earlier lanes.
__global__ void __launch_bounds__(kSortThreads) embed_scatter_kernel(const __grid_constant__ SortParams p) {
  __shared__ int hist[kSortWarps][kBins];
  __shared__ int warp_total[kSortWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  count_digits(p, hist);
  int before = 0, all = 0;
  for (int t = 0; t < p.tiles; ++t) {
    const int n = p.counts[static_cast<int64_t>(t) * kBins + threadIdx.x];
    all += n;
    before += t < static_cast<int>(blockIdx.x) ? n : 0;
  }
  int scan = all;  // over the bins, inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, scan, o);
    if (lane >= o) scan += up;
  }
  if (lane == 31) warp_total[warp] = scan;
  __syncthreads();
  int at = before + scan - all;
  for (int w = 0; w < warp; ++w) at += warp_total[w];
#pragma unroll
  for (int w = 0; w < kSortWarps; ++w) {
    const int n = hist[w][threadIdx.x];
    hist[w][threadIdx.x] = at;
    at += n;
  }
  __syncthreads();
  const int64_t part = p.tile / kSortWarps, from = blockIdx.x * p.tile + warp * part;
  for (int64_t i = from + lane; i - lane < from + part; i += 32) {
    const bool on = i < p.L;
    const int2 item = on ? sort_item(p, i) : make_int2(0, 0);
    const int digit = on ? (item.x >> p.shift) & ((1 << p.bits) - 1) : kBins;
    const unsigned same = __match_any_sync(0xffffffffu, digit);
    const int rank = __popc(same & ((1u << lane) - 1));
    int to = 0;
    if (on) to = hist[warp][digit] + rank;
    __syncwarp();
    if (on && rank == 0) hist[warp][digit] += __popc(same);
    __syncwarp();
    if (on) p.out[to] = item;
  }
}

// --------------------------------------------------------------- gradient

// First of the n sorted items whose key is at least v.
__device__ __forceinline__ int64_t lower_bound(const int2* items, int64_t n, int v) {
  int64_t lo = 0, hi = n;
  while (lo < hi) {
    const int64_t mid = (lo + hi) >> 1;
    if (items[mid].x < v)
      lo = mid + 1;
    else
      hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kThreads) embed_bwd_kernel(const __grid_constant__ EmbedParams p,
                                                             const int2* __restrict__ items) {
  const int v = blockIdx.x;
  const int64_t from = lower_bound(items, p.L, v), to = lower_bound(items, p.L, v + 1);
  if (p.add && from == to) return;
  for (int c = threadIdx.x * 8; c < p.D; c += kThreads * 8) {
    float g[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int64_t i = from; i < to; ++i) {
      const uint4 u = *reinterpret_cast<const uint4*>(p.dy + items[i].y * p.row + c);
      g[0] += bf16_lo(u.x), g[1] += bf16_hi(u.x), g[2] += bf16_lo(u.y), g[3] += bf16_hi(u.y);
      g[4] += bf16_lo(u.z), g[5] += bf16_hi(u.z), g[6] += bf16_lo(u.w), g[7] += bf16_hi(u.w);
    }
    float* w = p.dW + static_cast<int64_t>(v) * p.D + c;
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = p.add ? fmaf(g[e], p.scale, w[e]) : from == to ? 0.f : g[e] * p.scale;
  }
}

// ------------------------------------------------------------------- host

bool embed_ok(const upipe_embed_cfg* c) {
  return c && c->L >= 1 && c->L <= 0x7fffffffLL && c->V >= 1 && c->D >= 8 && c->D <= UPIPE_EMBED_MAX_D &&
         c->D % 8 == 0 && (c->wide == 0 || c->wide == 1) && (c->master == 0 || c->master == 1) &&
         std::isfinite(c->scale);
}

bool tokens_ok(const upipe_embed_cfg* c, const void* tokens) {
  return tokens && reinterpret_cast<uintptr_t>(tokens) % (c->wide ? 8 : 4) == 0;
}

EmbedParams embed_params(const upipe_embed_cfg* c, const void* tokens) {
  EmbedParams p;
  std::memset(&p, 0, sizeof(p));
  p.L = c->L;
  p.V = c->V;
  p.D = c->D;
  p.wide = c->wide;
  p.master = c->master;
  p.scale = c->scale;
  p.tokens = tokens;
  return p;
}

// The sort's plan: tiles of whole rounds, as few as kMaxTiles hold, and the
// passes that the largest key, V, takes.
struct SortPlan {
  int64_t tile;
  int tiles, passes;
  size_t pairs, bytes;
};
SortPlan sort_plan(const upipe_embed_cfg* c) {
  SortPlan s;
  constexpr int64_t kRound = kSortThreads;
  s.tile = (c->L + kMaxTiles - 1) / kMaxTiles;
  s.tile = s.tile < 2048 ? 2048 : (s.tile + kRound - 1) / kRound * kRound;
  s.tiles = static_cast<int>((c->L + s.tile - 1) / s.tile);
  int bits = 1;
  while (bits < 31 && (c->V >> bits) != 0) ++bits;
  s.passes = (bits + kDigit - 1) / kDigit;
  s.pairs = (static_cast<size_t>(c->L) * sizeof(int2) + 15) / 16 * 16;
  s.bytes = 2 * s.pairs + static_cast<size_t>(s.tiles) * kBins * sizeof(int32_t);
  return s;
}

}  // namespace
}  // namespace upipe

using namespace upipe;

extern "C" {

int upipe_embed_fwd(const upipe_embed_cfg* c, const void* tokens, const void* W, const upipe_rows* y, void* stream) {
  if (!embed_ok(c) || !tokens_ok(c, tokens) || !W || !aligned16(W) || !matrix_ok(y, c->L, c->D, true))
    return UPIPE_ERR_INVALID_ARG;
  int* status = nullptr;
  if (int e = device_ready(&status)) return e;
  EmbedParams p = embed_params(c, tokens);
  p.table = W;
  p.y = reinterpret_cast<bf16*>(y->p);
  p.row = y->row;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const unsigned grid = static_cast<unsigned>(c->L < 152 * 8 ? c->L : 152 * 8);
  UPIPE_LAUNCH(UPIPE_KIND_EMBED_FWD, (embed_fwd_kernel<<<grid, kThreads, 0, st>>>(p), cudaGetLastError()));
  return UPIPE_OK;
}

size_t upipe_embed_workspace_bytes(const upipe_embed_cfg* c) { return embed_ok(c) ? sort_plan(c).bytes : 0; }

int upipe_embed_bwd(const upipe_embed_cfg* c, const void* tokens, const upipe_rows* dy, float* dW, int add, void* ws,
                    size_t ws_bytes, void* stream) {
  if (!embed_ok(c) || !tokens_ok(c, tokens) || !matrix_ok(dy, c->L, c->D, false) || !dW || !aligned16(dW))
    return UPIPE_ERR_INVALID_ARG;
  if ((add != 0 && add != 1) || !ws || !aligned16(ws)) return UPIPE_ERR_INVALID_ARG;
  const SortPlan plan = sort_plan(c);
  if (ws_bytes < plan.bytes) return UPIPE_ERR_WS_TOO_SMALL;
  int* status = nullptr;
  if (int e = device_ready(&status)) return e;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint8_t* at = static_cast<uint8_t*>(ws);
  SortParams s;
  std::memset(&s, 0, sizeof(s));
  s.L = c->L;
  s.tile = plan.tile;
  s.tiles = plan.tiles;
  s.V = c->V;
  s.wide = c->wide;
  s.tokens = tokens;
  s.bits = kDigit;
  s.counts = reinterpret_cast<int32_t*>(at + 2 * plan.pairs);
  for (int i = 0; i < plan.passes; ++i) {
    s.first = i == 0;
    s.shift = i * kDigit;
    s.in = reinterpret_cast<const int2*>(at + (i & 1 ? 0 : plan.pairs));
    s.out = reinterpret_cast<int2*>(at + (i & 1 ? plan.pairs : 0));
    UPIPE_LAUNCH(UPIPE_KIND_EMBED_SORT,
                 (embed_count_kernel<<<plan.tiles, kSortThreads, 0, st>>>(s), cudaGetLastError()));
    UPIPE_LAUNCH(UPIPE_KIND_EMBED_SORT,
                 (embed_scatter_kernel<<<plan.tiles, kSortThreads, 0, st>>>(s), cudaGetLastError()));
  }
  EmbedParams p = embed_params(c, tokens);
  p.dy = reinterpret_cast<const bf16*>(dy->p);
  p.row = dy->row;
  p.dW = dW;
  p.add = add;
  UPIPE_LAUNCH(UPIPE_KIND_EMBED_BWD, (embed_bwd_kernel<<<c->V, kThreads, 0, st>>>(p, s.out), cudaGetLastError()));
  return UPIPE_OK;
}

}  // extern "C"
