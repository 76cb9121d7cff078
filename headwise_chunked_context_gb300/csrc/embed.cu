// Token embedding and the gradient of its table, and their C entry points.
//
// Mathematics: y_i = bf16(scale W[t_i]); a negative token reads zeros and
// leaves no gradient, a token >= V reads NaN and leaves none.  The gradient is
// dW[v] = scale (sum over i with t_i = v of dy_i), in fp32.
//
// The gradient's sums have one order whatever runs when.  The tokens are sorted
// by a stable radix sort (9 bits a pass; up to kSmall tokens in one CTA's shared
// memory), so that a row's positions stand behind one another in ascending
// order, and cut into chunks of equal length.  A CTA adds up a chunk's runs of
// equal tokens: runs inside the chunk are a row of dW, the others leave shares,
// which are added in the chunks' order.  Rows without a token are zeros, written
// by CTAs of their own: beside the sums, looked up in the sorted tokens, those at
// the table's end beside the sort.
//
// What bounds it: HBM.  The gradient reads dy once and writes V rows, most of
// them zeros at a real vocabulary; the sort, of 4 to 12 bytes a token, is its
// launches.
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
constexpr int kSmall = 8192;         // tokens that one CTA sorts alone
constexpr int kSmallThreads = 1024;
constexpr int kSmallWarps = kSmallThreads / 32;
constexpr int kFwdCols = 512;        // columns that a warp looks up
constexpr int kSlice = 2048;         // columns of a CTA of the gradient: a vector of 8 per thread
constexpr int kMaxChunk = 64;        // positions of a chunk
constexpr int kZeroRows = 256;       // rows of a CTA that writes zeros, at most
constexpr int kZeroBytes = 1 << 16;  // bytes of them, or those of 32 rows (20000 tokens, 50257 x 768: 63 us, 89 with 768 KB)
// Of the table's end, set to zero beside a small sort, and beside each launch of a longer one.
constexpr int64_t kBesideSmall = int64_t(128) << 20, kBesideLaunch = int64_t(16) << 20;
constexpr int kShort = 16;           // chunks behind its first that a short run reaches at most
constexpr int kShortCols = 4 * kThreads;       // columns of a CTA that adds a short run's shares
constexpr int kLongCols = 32, kLongRows = 32;  // of one that adds a long run's: columns, shares at once

struct EmbedParams {
  int64_t L;
  int V, D;
  int wide;  // 64-bit tokens
  float scale;
  const void* tokens;
  const void* table;
  bf16* y;
  int64_t row;  // its row stride
};

__device__ __forceinline__ int64_t token_at(const void* tokens, int wide, int64_t i) {
  return wide ? static_cast<const int64_t*>(tokens)[i] : static_cast<const int32_t*>(tokens)[i];
}

// A warp copies kFwdCols columns of a row, all of its loads open at once; neighbouring
// CTAs take neighbouring tokens, so that frequent rows' parts stay in L2, past which
// y is written.  131072 tokens of 152064 x 5120: 323 us with 512 columns, 409 with
// 256, 344 with 1024, 436 with 2048, 388 with a token's parts side by side.
template <bool MASTER>
__global__ void __launch_bounds__(kThreads) embed_fwd_kernel(const __grid_constant__ EmbedParams p) {
  constexpr int kVec = MASTER ? 4 : 8;  // elements of a 16-byte load
  constexpr int kLoads = kFwdCols / (32 * kVec);
  const int lane = threadIdx.x & 31;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  if (i >= p.L) return;
  const int64_t t = token_at(p.tokens, p.wide, i);
  const int col = blockIdx.y * kFwdCols + lane * kVec;
  bf16* y = p.y + i * p.row + col;
  const bool real = t >= 0 && t < p.V;
  uint4 u[kLoads];
#pragma unroll
  for (int j = 0; j < kLoads; ++j)
    if (real && col + j * 32 * kVec < p.D)
      u[j] = MASTER ? ld_global_nc_v4(static_cast<const float*>(p.table) + t * p.D + col + j * 32 * kVec)
                    : ld_global_nc_v4(static_cast<const bf16*>(p.table) + t * p.D + col + j * 32 * kVec);
    else
      u[j] = make_uint4(0, 0, 0, 0);
  const uint32_t fill = t < 0 ? 0u : 0x7fc07fc0u;  // zeros or NaN
#pragma unroll
  for (int j = 0; j < kLoads; ++j) {
    if (col + j * 32 * kVec >= p.D) continue;
    if (MASTER) {
      const uint32_t a = pack_bf16x2(__uint_as_float(u[j].x) * p.scale, __uint_as_float(u[j].y) * p.scale);
      const uint32_t b = pack_bf16x2(__uint_as_float(u[j].z) * p.scale, __uint_as_float(u[j].w) * p.scale);
      __stcs(reinterpret_cast<uint2*>(y + j * 32 * kVec), real ? make_uint2(a, b) : make_uint2(fill, fill));
    } else {
      const uint32_t w[4] = {u[j].x, u[j].y, u[j].z, u[j].w};
      uint32_t v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        v[e] = real ? pack_bf16x2(bf16_lo(w[e]) * p.scale, bf16_hi(w[e]) * p.scale) : fill;
      __stcs(reinterpret_cast<uint4*>(y + j * 32 * kVec), make_uint4(v[0], v[1], v[2], v[3]));
    }
  }
}

// ------------------------------------------------------------------- sort

// Vectors of dW that CTAs beside the sort, which has no use for most SMs, set to
// zero: rows with tokens too, which the sums write over.  At the table's end, as
// frequent tokens mostly have small numbers, where there are more rows than tokens,
// and no more bytes than the sort takes time for, the rest being written beside the
// sums (8192 tokens, 128256 x 4096 316 us, 329 with none, 325 with 512 MB; 4099 tokens,
// 30011 x 1032 36 for 48 with none; 20000 tokens, 50257 x 768 63 for 70, with 64 MB a
// launch 68; 32768 tokens, 128256 x 4096 363 for 366, with 64 MB a launch 378).
struct Zeros {
  float4* dW;
  int64_t from, end;
};
__device__ __forceinline__ void write_zeros(const Zeros& z, int cta, int ctas) {
  const int64_t stride = static_cast<int64_t>(ctas) * blockDim.x;
#pragma unroll 8
  for (int64_t i = z.from + static_cast<int64_t>(cta) * blockDim.x + threadIdx.x; i < z.end; i += stride)
    z.dW[i] = make_float4(0.f, 0.f, 0.f, 0.f);
}

// One pass of the sort: keys by kDigit bits from `shift` on.  The first pass
// reads the tokens (those without a row get key V, behind all rows), later
// passes the (key, position) pairs of the pass before.
struct SortParams {
  int64_t L, tile;  // tokens per CTA, a multiple of 32 kSortWarps
  int tiles, V, wide, first, shift;
  const void* tokens;
  const int2* in;
  int2* out;
  int32_t* counts;  // [tiles][kBins]
  int* joins;       // [2], set to 0 on the way
  Zeros zeros;      // by the CTAs behind the tiles'
};

constexpr int kBatch = 4;  // items that a lane has open at once, 32 apart

// Items i, i + 32, ... of a lane; behind the last one: a digit of its own.
__device__ __forceinline__ void sort_items(const SortParams& p, int64_t i, int64_t end, int2 (&item)[kBatch],
                                           int (&digit)[kBatch]) {
#pragma unroll
  for (int k = 0; k < kBatch; ++k) {
    item[k] = make_int2(p.V, 0);
    if (i + 32 * k >= end) continue;
    if (p.first) {
      const int64_t t = token_at(p.tokens, p.wide, i + 32 * k);
      item[k] = make_int2(t >= 0 && t < p.V ? static_cast<int>(t) : p.V, static_cast<int>(i + 32 * k));
    } else {
      item[k] = __ldcg(p.in + i + 32 * k);
    }
  }
#pragma unroll
  for (int k = 0; k < kBatch; ++k)
    digit[k] = i + 32 * k < end ? (item[k].x >> p.shift) & (kBins - 1) : kBins;
}

// Ranks an item among its warp's of the same digit and counts on.
__device__ __forceinline__ int place_of(int digit, int lane, int* row) {
  const bool on = digit < kBins;
  const unsigned same = __match_any_sync(0xffffffffu, digit);
  const int rank = __popc(same & ((1u << lane) - 1));
  const int to = on ? row[digit] + rank : 0;
  __syncwarp();
  if (on && rank == 0) row[digit] += __popc(same);
  __syncwarp();
  return to;
}

// Each warp counts the digits of its own part of the tile into its own row.
__device__ __forceinline__ void count_digits(const SortParams& p, int (*hist)[kBins]) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < kSortWarps * kBins; i += kSortThreads) (&hist[0][0])[i] = 0;
  __syncthreads();
  const int64_t part = p.tile / kSortWarps, from = blockIdx.x * p.tile + warp * part;
  const int64_t end = from + part < p.L ? from + part : p.L;
  for (int64_t i = from; i < end; i += 32 * kBatch) {
    int2 item[kBatch];
    int digit[kBatch];
    sort_items(p, i + lane, end, item, digit);
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (digit[k] < kBins) atomicAdd(&hist[warp][digit[k]], 1);
  }
  __syncthreads();
}

__global__ void __launch_bounds__(kSortThreads) embed_count_kernel(const __grid_constant__ SortParams p) {
  after_previous();
  let_next_start();
  if (static_cast<int>(blockIdx.x) >= p.tiles) return write_zeros(p.zeros, blockIdx.x - p.tiles, gridDim.x - p.tiles);
  __shared__ int hist[kSortWarps][kBins];
  if (blockIdx.x == 0 && threadIdx.x < 2) p.joins[threadIdx.x] = 0;
  count_digits(p, hist);
  int n = 0;
#pragma unroll
  for (int w = 0; w < kSortWarps; ++w) n += hist[w][threadIdx.x];
  p.counts[static_cast<int64_t>(blockIdx.x) * kBins + threadIdx.x] = n;
}

// Where the tile's tokens go: behind all smaller digits, behind the same digit
// of earlier tiles, of earlier warps, of earlier lanes.
__global__ void __launch_bounds__(kSortThreads) embed_scatter_kernel(const __grid_constant__ SortParams p) {
  after_previous();
  let_next_start();
  if (static_cast<int>(blockIdx.x) >= p.tiles) return write_zeros(p.zeros, blockIdx.x - p.tiles, gridDim.x - p.tiles);
  __shared__ int hist[kSortWarps][kBins];
  __shared__ int warp_total[kSortWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  count_digits(p, hist);
  int before = 0, all = 0;
#pragma unroll 16
  for (int t = 0; t < p.tiles; ++t) {
    const int n = __ldcg(p.counts + static_cast<int64_t>(t) * kBins + threadIdx.x);
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
  const int64_t end = from + part < p.L ? from + part : p.L;
  for (int64_t i = from; i < end; i += 32 * kBatch) {
    int2 item[kBatch];
    int digit[kBatch];
    sort_items(p, i + lane, end, item, digit);
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int to = place_of(digit[k], lane, hist[warp]);
      if (digit[k] < kBins) p.out[to] = item[k];
    }
  }
}

// Up to kSmall tokens: one CTA sorts them, pairs in shared memory, a part of them
// to each warp, per pass as above.
struct SmallParams {
  int L, V, wide, passes;
  const void* tokens;
  int2* out;
  int* joins;
  Zeros zeros;
};
constexpr int kSmallBytes = 2 * kSmall * sizeof(int2) + kSmallWarps * kBins * sizeof(int);

__global__ void __launch_bounds__(kSmallThreads) embed_small_kernel(const __grid_constant__ SmallParams p) {
  let_next_start();
  extern __shared__ __align__(16) uint8_t mem[];
  __shared__ int warp_total[kSmallWarps];
  int2 *from = reinterpret_cast<int2*>(mem), *to = from + kSmall;
  int(*hist)[kBins] = reinterpret_cast<int(*)[kBins]>(mem + 2 * kSmall * sizeof(int2));
  if (blockIdx.x > 0) {
    write_zeros(p.zeros, blockIdx.x - 1, gridDim.x - 1);
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x < 2) p.joins[threadIdx.x] = 0;
  for (int i = threadIdx.x; i < p.L; i += kSmallThreads) {
    const int64_t t = token_at(p.tokens, p.wide, i);
    from[i] = make_int2(t >= 0 && t < p.V ? static_cast<int>(t) : p.V, i);
  }
  const int part = (p.L + kSmallThreads - 1) / kSmallThreads * 32, first = warp * part;
  for (int pass = 0; pass < p.passes; ++pass) {
    const int shift = pass * kDigit;
    for (int i = threadIdx.x; i < kSmallWarps * kBins; i += kSmallThreads) (&hist[0][0])[i] = 0;
    __syncthreads();
    for (int i = first + lane; i < first + part && i < p.L; i += 32)
      atomicAdd(&hist[warp][(from[i].x >> shift) & (kBins - 1)], 1);
    __syncthreads();
    int all = 0, scan = 0;
    if (threadIdx.x < kBins) {
#pragma unroll 8
      for (int w = 0; w < kSmallWarps; ++w) all += hist[w][threadIdx.x];
      scan = all;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, scan, o);
        if (lane >= o) scan += up;
      }
      if (lane == 31) warp_total[warp] = scan;
    }
    __syncthreads();
    if (threadIdx.x < kBins) {
      int at = scan - all;
      for (int w = 0; w < warp; ++w) at += warp_total[w];
#pragma unroll 8
      for (int w = 0; w < kSmallWarps; ++w) {
        const int n = hist[w][threadIdx.x];
        hist[w][threadIdx.x] = at;
        at += n;
      }
    }
    __syncthreads();
    for (int i = first + lane; i - lane < first + part && i - lane < p.L; i += 32) {
      const int2 item = i < p.L ? from[i] : make_int2(0, 0);
      const int digit = i < p.L ? (item.x >> shift) & (kBins - 1) : kBins;
      const int place = place_of(digit, lane, hist[warp]);
      if (digit < kBins) to[place] = item;
    }
    __syncthreads();
    int2* swap = from;
    from = to;
    to = swap;
  }
  for (int i = threadIdx.x; i < p.L; i += kSmallThreads) p.out[i] = from[i];
}

// --------------------------------------------------------------- gradient

struct GradParams {
  int64_t L;
  int V, D;
  int chunk, chunks;  // positions of a chunk, chunks
  int add;
  int zero_rows;      // rows of a CTA that writes zeros, at least 32
  int late;           // rows whose zeros the sort has not written
  float scale;
  const bf16* dy;
  int64_t row;
  float* dW;
  const int2* items;  // sorted (token, position)
  float* share;       // [chunks][2][D]: of the run that began before the chunk, of the one that goes on behind it
  int* joins;         // counters: short runs that span chunks, long ones
  int4* join;         // [2][chunks]: first chunk, last chunk, token of each
};

// The first of the n sorted items whose token is at least v, found by a whole warp
// with 32 probes at once.
__device__ __forceinline__ int64_t warp_lower_bound(const int2* items, int64_t n, int64_t v) {
  const int lane = threadIdx.x & 31;
  int64_t lo = 0, end = n;  // it is in [lo, end]
  while (lo < end) {
    const int64_t step = (end - lo + 31) / 32, at = lo + lane * step + step - 1;
    const bool less = at < end && __ldcg(&items[at].x) < v;
    lo += __popc(__ballot_sync(0xffffffffu, less)) * step;
    if (lo + step - 1 < end) end = lo + step - 1;
  }
  return lo;
}

__device__ __forceinline__ void write_row8(float* w, const float (&g)[8], float scale, int add) {
  float4 a = make_float4(g[0] * scale, g[1] * scale, g[2] * scale, g[3] * scale);
  float4 b = make_float4(g[4] * scale, g[5] * scale, g[6] * scale, g[7] * scale);
  float4* to = reinterpret_cast<float4*>(w);
  if (add) {
    const float4 x = to[0], y = to[1];
    a.x += x.x, a.y += x.y, a.z += x.z, a.w += x.w;
    b.x += y.x, b.y += y.y, b.z += y.z, b.w += y.w;
  }
  to[0] = a;
  to[1] = b;
}

// Chunks first, slice by slice, then rows to fill with zeros.  A thread has the
// loads of eight positions open; four CTAs per SM (131072 tokens, 152064 x 5120:
// 687 us, with three 704, with five 722).
__global__ void __launch_bounds__(kThreads, 4) embed_bwd_kernel(const __grid_constant__ GradParams p) {
  after_previous();
  let_next_start();
  const int slices = (p.D + kSlice - 1) / kSlice;
  const int64_t block = blockIdx.x;
  if (block >= static_cast<int64_t>(p.chunks) * slices) {
    // Which of the CTA's rows have no token: a warp finds the tokens of 32 rows, a
    // lane among them its own row's.
    __shared__ unsigned empty[kZeroRows / 32];
    const int64_t first = (block - static_cast<int64_t>(p.chunks) * slices) * p.zero_rows;
    const int64_t v = first + threadIdx.x;
    bool none = false;
    if (threadIdx.x < p.zero_rows) {  // whole warps
      int64_t lo = warp_lower_bound(p.items, p.L, v - (threadIdx.x & 31));
      int64_t hi = warp_lower_bound(p.items, p.L, v - (threadIdx.x & 31) + 32);
      const int64_t end = hi;
      while (lo < hi) {
        const int64_t mid = (lo + hi) >> 1;
        if (__ldcg(&p.items[mid].x) < v)
          lo = mid + 1;
        else
          hi = mid;
      }
      none = v < p.late && (lo == end || __ldcg(&p.items[lo].x) != v);
    }
    const unsigned mask = __ballot_sync(0xffffffffu, none);
    if ((threadIdx.x & 31) == 0) empty[threadIdx.x >> 5] = mask;
    __syncthreads();
    int across = 2;  // threads of a row
    while (across < kThreads && across * 4 < p.D) across *= 2;
    for (int k = threadIdx.x / across; k < p.zero_rows; k += kThreads / across) {
      if (!((empty[k / 32] >> (k % 32)) & 1)) continue;
      float4* to = reinterpret_cast<float4*>(p.dW + (first + k) * p.D);
      for (int c = threadIdx.x % across; c < p.D / 4; c += across) to[c] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    return;
  }
  __shared__ int2 items[kMaxChunk + 2];  // with the one before and the one behind
  const int chunk = static_cast<int>(block / slices);
  const int slice = static_cast<int>(block - static_cast<int64_t>(chunk) * slices);
  const int col = slice * kSlice + threadIdx.x * 8;
  const int64_t first = static_cast<int64_t>(chunk) * p.chunk;
  for (int i = threadIdx.x; i < p.chunk + 2; i += kThreads) {
    const int64_t at = first + i - 1;
    items[i] = at >= 0 && at < p.L ? __ldcg(p.items + at) : make_int2(-1, 0);
  }
  __syncthreads();
  const int before = items[0].x, behind = items[p.chunk + 1].x;
  // The chunk's tokens that are rows: those without one stand at the end of all.
  const int mine = threadIdx.x < p.chunk ? items[threadIdx.x + 1].x : -1;
  const int n = __syncthreads_count(mine >= 0 && mine < p.V);
  const bool goes_on = n == p.chunk && items[n].x == behind && !(items[1].x == behind && before == behind);
  if (goes_on && slice == 0 && threadIdx.x < 32) {
    // A run begins here and goes on to chunk `in`: in one of the next 31, which a
    // warp looks at, or further; the order of the lists says nothing.
    const int next = chunk + 1 + threadIdx.x;
    const bool same = next < p.chunks && __ldcg(&p.items[static_cast<int64_t>(next) * p.chunk].x) == behind;
    const unsigned others = ~__ballot_sync(0xffffffffu, same);
    int in = chunk + __ffs(others) - 1;
    if (others == 0)
      in = static_cast<int>((warp_lower_bound(p.items, p.L, static_cast<int64_t>(behind) + 1) - 1) / p.chunk);
    const int kind = in - chunk > kShort;
    if (threadIdx.x == 0) p.join[kind * p.chunks + atomicAdd(p.joins + kind, 1)] = make_int4(chunk, in, behind, 0);
  }
  if (col >= p.D) return;
  const bf16* dy = p.dy + col;
  float g[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  bool began = before != items[1].x;  // the current run began in this chunk
  constexpr int kAhead = 8;
  for (int i = 0; i < n; i += kAhead) {
    uint4 u[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (i + k < n) u[k] = ld_global_nc_v4(dy + items[i + k + 1].y * p.row);
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (i + k >= n) break;
      g[0] += bf16_lo(u[k].x), g[1] += bf16_hi(u[k].x), g[2] += bf16_lo(u[k].y), g[3] += bf16_hi(u[k].y);
      g[4] += bf16_lo(u[k].z), g[5] += bf16_hi(u[k].z), g[6] += bf16_lo(u[k].w), g[7] += bf16_hi(u[k].w);
      const int token = items[i + k + 1].x;
      if (token == items[i + k + 2].x) {
        if (i + k + 1 < n) continue;  // the run goes on in this chunk
      } else if (began) {             // the whole run is in this chunk
        write_row8(p.dW + static_cast<int64_t>(token) * p.D + col, g, p.scale, p.add);
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] = 0.f;
        continue;
      }
      write_row8(p.share + (2 * static_cast<int64_t>(chunk) + began) * p.D + col, g, 1.f, 0);
#pragma unroll
      for (int e = 0; e < 8; ++e) g[e] = 0.f;
      began = true;
    }
  }
}

// Rows whose runs span chunks: the share of the chunk that a run begins in, then
// those of the chunks behind it.  A short run's are added one after another, a
// long run's by kLongRows rows of threads, each taking every kLongRows-th.
__device__ __forceinline__ void add4(float4& g, const float4& f) { g.x += f.x, g.y += f.y, g.z += f.z, g.w += f.w; }

__device__ __forceinline__ void write_row4(const GradParams& p, int token, int col, float4 g) {
  float4* to = reinterpret_cast<float4*>(p.dW + static_cast<int64_t>(token) * p.D + col);
  g.x *= p.scale, g.y *= p.scale, g.z *= p.scale, g.w *= p.scale;
  if (p.add) add4(g, *to);
  *to = g;
}

__global__ void __launch_bounds__(kThreads) embed_join_kernel(const __grid_constant__ GradParams p) {
  after_previous();
  __shared__ float4 part[kLongRows][kLongCols / 4];
  const float4* share = reinterpret_cast<const float4*>(p.share);
  const int64_t pitch = p.D / 4;  // of a share
  const int counts[2] = {__ldcg(p.joins), __ldcg(p.joins + 1)};
  int slices = (p.D + kShortCols - 1) / kShortCols;
  int64_t work = static_cast<int64_t>(counts[0]) * slices;
  for (int64_t i = blockIdx.x; i < work; i += gridDim.x) {
    const int4 run = __ldcg(p.join + i / slices);
    const int quad = static_cast<int>(i % slices) * kThreads + threadIdx.x;
    if (quad >= pitch) continue;
    const float4* from = share + 2 * static_cast<int64_t>(run.x) * pitch + quad;
    float4 g = __ldcg(from + pitch);
#pragma unroll 4
    for (int k = run.x + 1; k <= run.y; ++k) add4(g, __ldcg(from += 2 * pitch));
    write_row4(p, run.z, quad * 4, g);
  }
  slices = (p.D + kLongCols - 1) / kLongCols;
  work = static_cast<int64_t>(counts[1]) * slices;
  const int row = threadIdx.x / (kLongCols / 4), lane = threadIdx.x % (kLongCols / 4);
  for (int64_t i = blockIdx.x; i < work; i += gridDim.x) {
    const int4 run = __ldcg(p.join + p.chunks + i / slices);
    const int quad = static_cast<int>(i % slices) * (kLongCols / 4) + lane;
    float4 g = make_float4(0.f, 0.f, 0.f, 0.f);
    if (quad < pitch) {
#pragma unroll 8
      for (int k = run.x + row; k <= run.y; k += kLongRows)
        add4(g, __ldcg(share + (2 * static_cast<int64_t>(k) + (k == run.x)) * pitch + quad));
    }
    __syncthreads();  // the sums before have been read
    part[row][lane] = g;
    __syncthreads();
    if (row == 0 && quad < pitch) {
#pragma unroll
      for (int j = 1; j < kLongRows; ++j) add4(g, part[j][lane]);
      write_row4(p, run.z, quad * 4, g);
    }
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
  p.scale = c->scale;
  p.tokens = tokens;
  return p;
}

// The plan of a gradient: the sort's tiles (whole rounds, as few as kMaxTiles
// hold) and passes (what the largest key, V, takes), the chunks, and the places
// of the workspace.
struct GradPlan {
  int64_t tile;
  int tiles, passes, chunk, chunks;
  size_t pairs[2], counts, share, join, bytes;
};
GradPlan grad_plan(const upipe_embed_cfg* c) {
  GradPlan s;
  constexpr int64_t kRound = kSortThreads;
  s.tile = (c->L + kMaxTiles - 1) / kMaxTiles;
  s.tile = s.tile < 2048 ? 2048 : (s.tile + kRound - 1) / kRound * kRound;
  s.tiles = static_cast<int>((c->L + s.tile - 1) / s.tile);
  int bits = 1;
  while (bits < 31 && (c->V >> bits) != 0) ++bits;
  s.passes = (bits + kDigit - 1) / kDigit;
  // Long chunks leave few shares, short ones give every SM some.
  s.chunk = kMaxChunk;
  while (s.chunk > 8 && c->L / s.chunk < 152 * 4) s.chunk /= 2;
  s.chunks = static_cast<int>((c->L + s.chunk - 1) / s.chunk);
  size_t at = 0;
  auto take = [&at](size_t bytes) {
    const size_t from = at;
    at += (bytes + 15) / 16 * 16;
    return from;
  };
  s.join = take((1 + 2 * static_cast<size_t>(s.chunks)) * sizeof(int4));  // the counters, then the lists
  s.pairs[0] = take(static_cast<size_t>(c->L) * sizeof(int2));
  const bool small = c->L <= kSmall;
  s.pairs[1] = small ? s.pairs[0] : take(static_cast<size_t>(c->L) * sizeof(int2));
  s.counts = small ? 0 : take(static_cast<size_t>(s.tiles) * kBins * sizeof(int32_t));
  s.share = take(2 * static_cast<size_t>(s.chunks) * c->D * sizeof(float));
  s.bytes = at;
  return s;
}

cudaError_t launch_small(const SmallParams& p, bool zeros, cudaStream_t st) {
  static std::atomic<uint64_t> allowed{0};
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(embed_small_kernel), kSmallBytes, allowed);
  if (e != cudaSuccess) return e;
  embed_small_kernel<<<zeros ? 152 : 1, kSmallThreads, kSmallBytes, st>>>(p);
  return cudaGetLastError();
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
  constexpr int kWarps = kThreads / 32;
  const dim3 grid(static_cast<unsigned>((c->L + kWarps - 1) / kWarps), static_cast<unsigned>((c->D + kFwdCols - 1) / kFwdCols));
  UPIPE_LAUNCH(UPIPE_KIND_EMBED_FWD, ((c->master ? embed_fwd_kernel<true> : embed_fwd_kernel<false>)<<<grid, kThreads, 0, st>>>(p),
                                      cudaGetLastError()));
  return UPIPE_OK;
}

size_t upipe_embed_workspace_bytes(const upipe_embed_cfg* c) { return embed_ok(c) ? grad_plan(c).bytes : 0; }

int upipe_embed_bwd(const upipe_embed_cfg* c, const void* tokens, const upipe_rows* dy, float* dW, int add, void* ws,
                    size_t ws_bytes, void* stream) {
  if (!embed_ok(c) || !tokens_ok(c, tokens) || !matrix_ok(dy, c->L, c->D, false) || !dW || !aligned16(dW))
    return UPIPE_ERR_INVALID_ARG;
  if ((add != 0 && add != 1) || !ws || !aligned16(ws)) return UPIPE_ERR_INVALID_ARG;
  const GradPlan plan = grad_plan(c);
  if (ws_bytes < plan.bytes) return UPIPE_ERR_WS_TOO_SMALL;
  int* status = nullptr;
  if (int e = device_ready(&status)) return e;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint8_t* at = static_cast<uint8_t*>(ws);
  GradParams g;
  std::memset(&g, 0, sizeof(g));
  g.joins = reinterpret_cast<int*>(at + plan.join);
  g.join = reinterpret_cast<int4*>(g.joins) + 1;
  // Rows from `late` on are set to zero beside the sort, launch by launch.
  const int launches = c->L <= kSmall ? 1 : 2 * plan.passes;
  int64_t early = add || c->L >= c->V ? 0 : (c->L <= kSmall ? kBesideSmall : kBesideLaunch * launches) / (4 * c->D);
  if (early > c->V) early = c->V;
  g.late = c->V - static_cast<int>(early);
  const int64_t from = static_cast<int64_t>(g.late) * (c->D / 4), vectors = early * (c->D / 4);
  auto zeros = [&](int k) {
    return Zeros{reinterpret_cast<float4*>(dW), from + vectors * k / launches, from + vectors * (k + 1) / launches};
  };
  const unsigned fill = early > 0 ? 152 : 0;
  if (c->L <= kSmall) {
    const SmallParams s{static_cast<int>(c->L), c->V, c->wide, plan.passes, tokens,
                        reinterpret_cast<int2*>(at + plan.pairs[0]), g.joins, zeros(0)};
    UPIPE_LAUNCH(UPIPE_KIND_EMBED_SORT, launch_small(s, early > 0, st));
    g.items = s.out;
  } else {
    SortParams s;
    std::memset(&s, 0, sizeof(s));
    s.L = c->L;
    s.tile = plan.tile;
    s.tiles = plan.tiles;
    s.V = c->V;
    s.wide = c->wide;
    s.tokens = tokens;
    s.joins = g.joins;
    s.counts = reinterpret_cast<int32_t*>(at + plan.counts);
    for (int i = 0; i < plan.passes; ++i) {
      s.first = i == 0;
      s.shift = i * kDigit;
      s.in = reinterpret_cast<const int2*>(at + plan.pairs[(i & 1) ^ 1]);
      s.out = reinterpret_cast<int2*>(at + plan.pairs[i & 1]);
      s.zeros = zeros(2 * i);
      UPIPE_LAUNCH(UPIPE_KIND_EMBED_SORT,
                   (i ? launch_next(embed_count_kernel, plan.tiles + fill, kSortThreads, 0, st, s)
                      : (embed_count_kernel<<<plan.tiles + fill, kSortThreads, 0, st>>>(s), cudaGetLastError())));
      s.zeros = zeros(2 * i + 1);
      UPIPE_LAUNCH(UPIPE_KIND_EMBED_SORT,
                   launch_next(embed_scatter_kernel, plan.tiles + fill, kSortThreads, 0, st, s));
    }
    g.items = s.out;
  }
  g.L = c->L;
  g.V = c->V;
  g.D = c->D;
  g.chunk = plan.chunk;
  g.chunks = plan.chunks;
  g.add = add;
  g.scale = c->scale;
  g.dy = reinterpret_cast<const bf16*>(dy->p);
  g.row = dy->row;
  g.dW = dW;
  g.share = reinterpret_cast<float*>(at + plan.share);
  const int64_t sums = static_cast<int64_t>(plan.chunks) * ((c->D + kSlice - 1) / kSlice);
  g.zero_rows = kZeroBytes / (4 * c->D) / 32 * 32;
  g.zero_rows = g.zero_rows < 32 ? 32 : g.zero_rows < kZeroRows ? g.zero_rows : kZeroRows;
  const int64_t empty = add ? 0 : (static_cast<int64_t>(g.late) + g.zero_rows - 1) / g.zero_rows;
  UPIPE_LAUNCH(UPIPE_KIND_EMBED_BWD,
               launch_next(embed_bwd_kernel, static_cast<unsigned>(sums + empty), kThreads, 0, st, g));
  UPIPE_LAUNCH(UPIPE_KIND_EMBED_BWD, launch_next(embed_join_kernel, 152 * 8, kThreads, 0, st, g));
  return UPIPE_OK;
}

}  // extern "C"
