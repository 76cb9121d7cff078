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
  int team;        // threads of a row in one CTA
  float* partial;  // backward: [row walks][2][D] shares of dw and db
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
//
// A team of threads holds a row, two 16-byte vectors a thread, and walks rows
// a grid apart; short rows share a CTA, long ones are split over the CTAs of a
// cluster, so that a CTA never has more than kMaxTeam threads and two of the
// largest fit an SM with the registers that the backward's column sums take.
// Copies run S - 1 rows ahead, asynchronously, into slots of shared memory that
// only the copying thread reads: there is nothing to wait for but its own
// copies.  What the team waits for are its sums: one barrier for the mean and
// one for the sums that need it.
constexpr int kMaxTeam = 320;
constexpr int kVecs = 2;  // per thread
constexpr int kMaxSlots = 40;  // warps of a team over its cluster: 4 x 10

struct Team {
  int size, teams;  // threads of a row in this CTA, rows at once
  int id, at;       // this thread's team, its place there
  int warps;        // of a row in this CTA
  int lane, warp;
};

__device__ __forceinline__ Team team_of(int size) {
  Team t;
  t.size = size;
  t.teams = blockDim.x / size;
  t.id = threadIdx.x / size;
  t.at = threadIdx.x - t.id * size;
  t.warps = size / 32;
  t.lane = threadIdx.x & 31;
  t.warp = t.at >> 5;
  return t;
}

__device__ __forceinline__ void st_cluster(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// Sums of N numbers over the row's team (and the other CTAs of its cluster),
// added in one order.  slots [N][kMaxSlots], zeros behind the warps' sums: a
// set of slots is used again two sums later at the earliest, when every thread
// has passed the barrier between.
template <int N, int CL>
__device__ __forceinline__ void team_sum(float (&v)[N], float (*slots)[kMaxSlots], const Team& t) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  if (CL == 1 && t.warps == 1) return;
  if (CL == 1) {
    if (t.lane == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) slots[i][t.warp] = v[i];
    asm volatile("bar.sync %0, %1;" ::"r"(t.id + 1), "r"(t.size) : "memory");
  } else {
    if (t.lane < CL) {
      const int at = static_cast<int>(cluster_rank()) * t.warps + t.warp;
#pragma unroll
      for (int i = 0; i < N; ++i) st_cluster(mapa_shared(smem_u32(&slots[i][at]), t.lane), v[i]);
    }
    __syncwarp();
    cluster_sync();
  }
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = 0.f;
  for (int k = 0; k < CL * t.warps; k += 4)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float4 f = *reinterpret_cast<const float4*>(&slots[i][k]);
      v[i] += (f.x + f.y) + (f.z + f.w);
    }
}

// T rows in flight, S deep; slots of this thread alone.
template <int T, int S>
struct Rows {
  static constexpr int kBytes = S * T * kVecs * 16;  // per thread
  uint32_t slot;
  uint32_t pitch;  // from one vector's slot to the next
  int at;
  __device__ __forceinline__ explicit Rows(const uint8_t* ring)
      : slot(smem_u32(ring) + threadIdx.x * 16), pitch(blockDim.x * 16), at(0) {}
  // Starts the copies of one row: vectors at columns col[j] of row[t]; off:
  // zeros, and nothing is read.
  __device__ __forceinline__ void start(const bf16* const (&row)[T], const int (&col)[kVecs],
                                        const bool (&on)[kVecs]) {
#pragma unroll
    for (int t = 0; t < T; ++t)
#pragma unroll
      for (int j = 0; j < kVecs; ++j) {
        const uint32_t to = slot + ((at * T + t) * kVecs + j) * pitch;
        const bf16* from = on[j] ? row[t] + col[j] : row[t];
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(on[j] ? 16 : 0)
                     : "memory");
      }
    asm volatile("cp.async.commit_group;" ::: "memory");
    at = at + 1 == S ? 0 : at + 1;
  }
  // The oldest row has arrived: it stands in the slot after the newest one's.
  __device__ __forceinline__ void wait() const { asm volatile("cp.async.wait_group %0;" ::"n"(S - 1) : "memory"); }
  __device__ __forceinline__ uint4 take(int t, int j) const {
    return ld_shared_v4(slot + ((at * T + t) * kVecs + j) * pitch);
  }
  static __device__ __forceinline__ void drain() { asm volatile("cp.async.wait_all;" ::: "memory"); }
};

__device__ __forceinline__ void unpack8(const uint4& u, float (&v)[8]) {
  v[0] = bf16_lo(u.x), v[1] = bf16_hi(u.x), v[2] = bf16_lo(u.y), v[3] = bf16_hi(u.y);
  v[4] = bf16_lo(u.z), v[5] = bf16_hi(u.z), v[6] = bf16_lo(u.w), v[7] = bf16_hi(u.w);
}
__device__ __forceinline__ void unpack4(const uint4& u, uint64_t (&v)[4]) {
  v[0] = f2_pack(bf16_lo(u.x), bf16_hi(u.x)), v[1] = f2_pack(bf16_lo(u.y), bf16_hi(u.y));
  v[2] = f2_pack(bf16_lo(u.z), bf16_hi(u.z)), v[3] = f2_pack(bf16_lo(u.w), bf16_hi(u.w));
}
__device__ __forceinline__ uint32_t round2(uint64_t v) {
  float a, b;
  f2_unpack(v, a, b);
  return pack_bf16x2(a, b);
}
__device__ __forceinline__ uint64_t f2_both(float v) { return f2_pack(v, v); }
__device__ __forceinline__ float f2_sum(uint64_t v) {
  float a, b;
  f2_unpack(v, a, b);
  return a + b;
}

// This thread's part of a row: columns of its vectors, and whether they exist.
template <int CL>
__device__ __forceinline__ void my_columns(const Team& t, int D, int (&col)[kVecs], bool (&live)[kVecs]) {
  const int rank = CL > 1 ? static_cast<int>(cluster_rank()) : 0;
#pragma unroll
  for (int j = 0; j < kVecs; ++j) {
    col[j] = (rank * kVecs * t.size + j * t.size + t.at) * 8;
    live[j] = col[j] < D;
  }
}

// A vector of a weight as four pairs; dead: zeros.
__device__ __forceinline__ void weight4(const float* w, int col, bool live, uint64_t (&v)[4]) {
#pragma unroll
  for (int e = 0; e < 4; ++e)
    v[e] = live && w ? f2_pack(__ldg(w + col + 2 * e), __ldg(w + col + 2 * e + 1)) : 0;
}

constexpr int kFwdDepth = 4;
__host__ __device__ constexpr int bwd_depth(bool ds) { return ds ? 3 : 4; }

template <bool RES, bool DROP, int CL>
__global__ void __launch_bounds__(kMaxTeam, 2) layer_norm_fwd_kernel(const __grid_constant__ NormParams p) {
  constexpr int T = RES ? 2 : 1;
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ __align__(16) float slots[4][4][1][kMaxSlots];  // of each team: two sums, each by turns of two
  const Team t = team_of(p.team);
  int col[kVecs];
  bool live[kVecs];
  my_columns<CL>(t, p.D, col, live);
  if (CL > 1 || t.warps > 1) {
    for (int i = threadIdx.x; i < 16 * kMaxSlots; i += blockDim.x) (&slots[0][0][0][0])[i] = 0.f;
    if (CL > 1)
      cluster_sync();
    else
      __syncthreads();
  }
  const int64_t step = static_cast<int64_t>(gridDim.x / CL) * t.teams;
  int64_t row = static_cast<int64_t>(blockIdx.x / CL) * t.teams + t.id, ahead = row;
  Rows<T, kFwdDepth> rows(ring);
  auto start = [&] {
    const bool in = ahead < p.L;
    const bf16* from[T];
    from[0] = in ? p.x.p + ahead * p.x.row : p.x.p;
    if (RES) from[T - 1] = in ? p.res.p + ahead * p.res.row : p.res.p;
    bool on[kVecs];
#pragma unroll
    for (int j = 0; j < kVecs; ++j) on[j] = in && live[j];
    rows.start(from, col, on);
    ahead += step;
  };
#pragma unroll
  for (int i = 0; i + 1 < kFwdDepth; ++i) start();
  uint64_t w[kVecs][4], b[kVecs][4];
#pragma unroll
  for (int j = 0; j < kVecs; ++j) {
    weight4(p.w, col[j], live[j], w[j]);
    weight4(p.b, col[j], live[j], b[j]);
  }
  const uint64_t call = DROP ? drop_call(p.drop) : 0;
  const float inv = 1.f / p.D;
  for (int turn = 0; row < p.L; row += step, turn ^= 1) {
    start();
    rows.wait();
    uint64_t s[kVecs][4];
    uint64_t sum = 0;
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      const uint4 x = rows.take(0, j);
      if (!RES && !DROP) {
        unpack4(x, s[j]);
      } else {
        float v[8];
        unpack8(x, v);
        if (DROP) drop8(p.drop, call, static_cast<uint64_t>(row) * p.D + col[j], v);
        if (RES) {
          float r[8];
          unpack8(rows.take(T - 1, j), r);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = __fadd_rn(r[e], v[e]);
        }
        const uint4 u = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                                   pack_bf16x2(v[6], v[7]));
        if (live[j]) st_global_v4(p.s.p + row * p.s.row + col[j], u.x, u.y, u.z, u.w);
        unpack4(u, s[j]);  // the norm is of s as it is stored
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) sum = f2_add(sum, s[j][e]);
    }
    if (!p.rms) {
      float m[1] = {f2_sum(sum)};
      team_sum<1, CL>(m, slots[t.id & 3][turn], t);
      const uint64_t mm = f2_both(m[0] * inv);
#pragma unroll
      for (int j = 0; j < kVecs; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[j][e] = f2_sub(s[j][e], mm);
    }
    uint64_t sq = 0;
#pragma unroll
    for (int j = 0; j < kVecs; ++j)
      if (live[j])
#pragma unroll
        for (int e = 0; e < 4; ++e) sq = f2_fma(s[j][e], s[j][e], sq);
    float q[1] = {f2_sum(sq)};
    team_sum<1, CL>(q, slots[t.id & 3][2 + turn], t);
    const uint64_t r = f2_both(rsqrtf(q[0] * inv + p.eps));
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      uint32_t y[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = round2(f2_fma(f2_mul(s[j][e], r), w[j][e], b[j][e]));
      if (live[j]) st_global_v4(p.y.p + row * p.y.row + col[j], y[0], y[1], y[2], y[3]);
    }
  }
  rows.drain();
  if (CL > 1) cluster_sync();  // nobody leaves while a peer may still write to it
}

// Each CTA keeps its columns' sums of dw and db in registers over all of its
// rows and writes one share of each (the teams' shares added in order), which
// weight_sum_kernel adds up.
template <bool DS, bool DROP, int CL>
__global__ void __launch_bounds__(kMaxTeam, 2) layer_norm_bwd_kernel(const __grid_constant__ NormParams p) {
  constexpr int T = DS ? 3 : 2;
  constexpr int S = bwd_depth(DS);
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ __align__(16) float slots_m[4][2][1][kMaxSlots], slots_g[4][2][3][kMaxSlots];
  const Team t = team_of(p.team);
  int col[kVecs];
  bool live[kVecs];
  my_columns<CL>(t, p.D, col, live);
  if (CL > 1 || t.warps > 1) {
    for (int i = threadIdx.x; i < 8 * kMaxSlots; i += blockDim.x) (&slots_m[0][0][0][0])[i] = 0.f;
    for (int i = threadIdx.x; i < 24 * kMaxSlots; i += blockDim.x) (&slots_g[0][0][0][0])[i] = 0.f;
    if (CL > 1)
      cluster_sync();
    else
      __syncthreads();
  }
  const int64_t step = static_cast<int64_t>(gridDim.x / CL) * t.teams;
  int64_t row = static_cast<int64_t>(blockIdx.x / CL) * t.teams + t.id, ahead = row;
  Rows<T, S> rows(ring);
  auto start = [&] {
    const bool in = ahead < p.L;
    const bf16* from[T];
    from[0] = in ? p.s.p + ahead * p.s.row : p.s.p;
    from[1] = in ? p.dy.p + ahead * p.dy.row : p.dy.p;
    if (DS) from[T - 1] = in ? p.ds.p + ahead * p.ds.row : p.ds.p;
    bool on[kVecs];
#pragma unroll
    for (int j = 0; j < kVecs; ++j) on[j] = in && live[j];
    rows.start(from, col, on);
    ahead += step;
  };
#pragma unroll
  for (int i = 0; i + 1 < S; ++i) start();
  uint64_t w[kVecs][4], dw[kVecs][4], db[kVecs][4];
#pragma unroll
  for (int j = 0; j < kVecs; ++j) {
    weight4(p.w, col[j], live[j], w[j]);
#pragma unroll
    for (int e = 0; e < 4; ++e) dw[j][e] = db[j][e] = 0;
  }
  const uint64_t call = DROP ? drop_call(p.drop) : 0;
  const float inv = 1.f / p.D;
  for (int turn = 0; row < p.L; row += step, turn ^= 1) {
    start();
    rows.wait();
    uint4 su[kVecs], gu[kVecs];
    uint64_t mm = 0;
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      su[j] = rows.take(0, j);
      gu[j] = rows.take(1, j);
    }
    if (!p.rms) {
      uint64_t sum = 0;
#pragma unroll
      for (int j = 0; j < kVecs; ++j) {
        uint64_t a[4];
        unpack4(su[j], a);
#pragma unroll
        for (int e = 0; e < 4; ++e) sum = f2_add(sum, a[e]);
      }
      float m[1] = {f2_sum(sum)};
      team_sum<1, CL>(m, slots_m[t.id & 3][turn], t);
      mm = f2_both(m[0] * inv);
    }
    uint64_t sq = 0, sg = 0, sd = 0;
#pragma unroll
    for (int j = 0; j < kVecs; ++j)
      if (live[j]) {
        uint64_t a[4], g[4];
        unpack4(su[j], a);
        unpack4(gu[j], g);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          a[e] = f2_sub(a[e], mm);
          g[e] = f2_mul(g[e], w[j][e]);
          sq = f2_fma(a[e], a[e], sq);
          sg = f2_add(sg, g[e]);
          sd = f2_fma(g[e], a[e], sd);
        }
      }
    float v[3] = {f2_sum(sq), f2_sum(sg), f2_sum(sd)};
    team_sum<3, CL>(v, slots_g[t.id & 3][turn], t);
    const float r = rsqrtf(v[0] * inv + p.eps);
    const uint64_t rr = f2_both(r);
    const uint64_t c0 = f2_both(p.rms ? 0.f : -r * (v[1] * inv));  // -r mean(g)
    const uint64_t c1 = f2_both(-r * (r * (v[2] * inv)));          // -r mean(g n)
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      if (!live[j]) continue;
      uint64_t a[4], g[4];
      unpack4(su[j], a);
      unpack4(gu[j], g);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint64_t n = f2_mul(f2_sub(a[e], mm), rr);
        dw[j][e] = f2_fma(g[e], n, dw[j][e]);
        db[j][e] = f2_add(db[j][e], g[e]);
        a[e] = f2_fma(n, c1, f2_fma(f2_mul(g[e], w[j][e]), rr, c0));
      }
      if (DS) {
        unpack4(rows.take(T - 1, j), g);
#pragma unroll
        for (int e = 0; e < 4; ++e) a[e] = f2_add(a[e], g[e]);
      }
      st_global_v4(p.dres.p + row * p.dres.row + col[j], round2(a[0]), round2(a[1]), round2(a[2]), round2(a[3]));
      if (DROP) {
        float d[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) f2_unpack(a[e], d[2 * e], d[2 * e + 1]);
        drop8(p.drop, call, static_cast<uint64_t>(row) * p.D + col[j], d);
        store8(p.dx.p + row * p.dx.row + col[j], d);
      }
    }
  }
  rows.drain();
  float* out = p.partial + static_cast<int64_t>(blockIdx.x / CL) * 2 * p.D;
  if (CL > 1 || t.teams == 1) {
#pragma unroll
    for (int j = 0; j < kVecs; ++j)
      if (live[j]) {
        uint64_t* to = reinterpret_cast<uint64_t*>(out + col[j]);
        uint64_t* to_b = reinterpret_cast<uint64_t*>(out + p.D + col[j]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          to[e] = dw[j][e];
          to_b[e] = db[j][e];
        }
      }
    if (CL > 1) cluster_sync();  // nobody leaves while a peer may still write to it
    return;
  }
  // The teams' shares, [team][2][D], in the ring's memory.
  float* share = reinterpret_cast<float*>(ring);
  __syncthreads();  // every team's copies have arrived and been read
#pragma unroll
  for (int j = 0; j < kVecs; ++j)
    if (live[j]) {
      uint64_t* to = reinterpret_cast<uint64_t*>(share + t.id * 2 * p.D + col[j]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        to[e] = dw[j][e];
        to[p.D / 2 + e] = db[j][e];
      }
    }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * p.D; i += blockDim.x) {
    float g = 0.f;
    for (int k = 0; k < t.teams; ++k) g += share[k * 2 * p.D + i];
    out[i] = g;
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

constexpr int kThreadsPerSm = 2 * kMaxTeam;

bool norm_ok(const upipe_norm_cfg* c) {
  return c && c->L >= 1 && c->L <= 0x7fffffffLL && c->D >= 8 && c->D <= UPIPE_NORM_MAX_D && c->D % 8 == 0 &&
         (c->rms == 0 || c->rms == 1) && c->eps >= 0.f && std::isfinite(c->eps);
}

bool weight_ok(const float* w) { return w && reinterpret_cast<uintptr_t>(w) % sizeof(float) == 0; }

Mat mat_of(const upipe_rows* t) { return t ? Mat{reinterpret_cast<bf16*>(t->p), t->row} : Mat{nullptr, 0}; }

// How rows of D elements lie: CTAs per row, threads of a row in one CTA, rows
// at once in one CTA, and how many CTAs (or clusters) walk the rows.
struct Layout {
  int cluster, team, teams, walks;
};
Layout layout_of(int64_t L, int D) {
  Layout y;
  const int most = kMaxTeam * kVecs * 8;  // elements of a CTA
  y.cluster = D <= most ? 1 : D <= 2 * most ? 2 : 4;
  const int lanes = (D / 8 + kVecs * y.cluster - 1) / (kVecs * y.cluster);
  y.team = (lanes + 31) / 32 * 32;
  y.teams = y.cluster > 1 || y.team > 128 ? 1 : 256 / y.team;
  const int64_t need = (L + y.teams - 1) / y.teams;
  const int room = 152 * (kThreadsPerSm / (y.team * y.teams)) / y.cluster;
  y.walks = static_cast<int>(need < room ? need : room);
  return y;
}

template <class K>
cudaError_t launch_rows(K kernel, const Layout& y, int bytes_per_thread, const NormParams& p, cudaStream_t st) {
  const int threads = y.team * y.teams;
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxTeam * bytes_per_thread);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(y.walks * y.cluster));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = static_cast<size_t>(threads) * bytes_per_thread;
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = static_cast<unsigned>(y.cluster);
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = y.cluster > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <bool RES, bool DROP>
cudaError_t launch_fwd(const Layout& y, const NormParams& p, cudaStream_t st) {
  constexpr int kBytes = Rows<RES ? 2 : 1, kFwdDepth>::kBytes;
  switch (y.cluster) {
    case 1: return launch_rows(layer_norm_fwd_kernel<RES, DROP, 1>, y, kBytes, p, st);
    case 2: return launch_rows(layer_norm_fwd_kernel<RES, DROP, 2>, y, kBytes, p, st);
  }
  return launch_rows(layer_norm_fwd_kernel<RES, DROP, 4>, y, kBytes, p, st);
}

template <bool DS, bool DROP>
cudaError_t launch_bwd(const Layout& y, const NormParams& p, cudaStream_t st) {
  constexpr int kBytes = Rows<DS ? 3 : 2, bwd_depth(DS)>::kBytes;
  switch (y.cluster) {
    case 1: return launch_rows(layer_norm_bwd_kernel<DS, DROP, 1>, y, kBytes, p, st);
    case 2: return launch_rows(layer_norm_bwd_kernel<DS, DROP, 2>, y, kBytes, p, st);
  }
  return launch_rows(layer_norm_bwd_kernel<DS, DROP, 4>, y, kBytes, p, st);
}

cudaError_t launch_weight_sum(const NormParams& p, int walks, float* dw, float* db, cudaStream_t st) {
  const unsigned cols = static_cast<unsigned>(db ? 2 * p.D : p.D);
  weight_sum_kernel<<<(cols + 31) / 32, dim3(32, 32), 0, st>>>(p.partial, walks, p.D, dw, db);
  return cudaGetLastError();
}

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
  const Layout lay = layout_of(c->L, c->D);
  p.team = lay.team;
  UPIPE_LAUNCH(UPIPE_KIND_LAYER_NORM_FWD, res ? (drop ? launch_fwd<true, true>(lay, p, st) : launch_fwd<true, false>(lay, p, st))
                                              : (drop ? launch_fwd<false, true>(lay, p, st) : launch_fwd<false, false>(lay, p, st)));
  return UPIPE_OK;
}

size_t upipe_layer_norm_workspace_bytes(const upipe_norm_cfg* c) {
  return norm_ok(c) ? static_cast<size_t>(layout_of(c->L, c->D).walks) * 2 * c->D * sizeof(float) : 0;
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
  const Layout lay = layout_of(c->L, c->D);
  p.team = lay.team;
  UPIPE_LAUNCH(UPIPE_KIND_LAYER_NORM_BWD,
               ds ? (drop ? launch_bwd<true, true>(lay, p, st) : launch_bwd<true, false>(lay, p, st))
                  : (drop ? launch_bwd<false, true>(lay, p, st) : launch_bwd<false, false>(lay, p, st)));
  UPIPE_LAUNCH(UPIPE_KIND_NORM_SUM, launch_weight_sum(p, lay.walks, dw, db, st));
  return UPIPE_OK;
}

}  // extern "C"
