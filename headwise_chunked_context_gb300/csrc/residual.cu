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
#include <type_traits>

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
  Drop drop;
  Mat x, res, s, y;      // forward; backward: s is read
  Mat dy, ds, dres, dx;  // backward
  const float *w, *b;
  int warps;       // of a row
  int ctas;
  float* partial;  // backward: [gridDim.x][2][D] shares of dw and db
};

__device__ __forceinline__ void unpack8(const uint4& u, float (&v)[8]) {
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
  int across;  // threads of a row (rows at a stride)
  Drop drop;
  Mat x, res, y;
};

// Vectors of 8 elements; every load of a thread is open before the first mask is
// drawn.  FLAT: dense tensors are one long row.
constexpr int kDropVecs = 4;

template <bool RES, bool FLAT>
__global__ void __launch_bounds__(kThreads) dropout_kernel(const __grid_constant__ DropParams p) {
  const int per = p.D / 8;
  int64_t row = 0, at, end;
  int step = kThreads;
  if (FLAT) {
    at = static_cast<int64_t>(blockIdx.x) * (kThreads * kDropVecs) + threadIdx.x;
    end = p.L * per;
  } else {
    const int y = threadIdx.x / p.across;
    row = static_cast<int64_t>(blockIdx.x) * (kThreads / p.across) + y;
    if (row >= p.L) return;
    step = p.across;
    at = threadIdx.x - y * p.across;
    end = per;
  }
  Mask mask(p.drop, drop_call(p.drop));
  const bf16 *x = p.x.p + row * p.x.row, *res = RES ? p.res.p + row * p.res.row : nullptr;
  bf16* y = p.y.p + row * p.y.row;
  do {
    uint4 u[kDropVecs], r[RES ? kDropVecs : 1];
    const bool all = at + (kDropVecs - 1) * step < end;
#pragma unroll
    for (int j = 0; j < kDropVecs; ++j)
      if (all || at + j * step < end) {
        u[j] = *reinterpret_cast<const uint4*>(x + at * 8 + j * step * 8);
        if (RES) r[j] = *reinterpret_cast<const uint4*>(res + at * 8 + j * step * 8);
      }
#pragma unroll
    for (int j = 0; j < kDropVecs; ++j)
      if (all || at + j * step < end) {
        float v[8];
        unpack8(u[j], v);
        const uint64_t e = static_cast<uint64_t>(row) * p.D + at * 8 + j * step * 8;
        if (RES) {
          float s[8];
          unpack8(r[j], s);
          mask.add(e, v, s);
          store8(y + at * 8 + j * step * 8, s);
        } else {
          mask.apply(e, v);
          store8(y + at * 8 + j * step * 8, v);
        }
      }
    at += kDropVecs * step;
  } while (!FLAT && at < end);
}

// ------------------------------------------------------------------- norm
//
// A lane holds NV 16-byte vectors of a row, 512 bytes apart, a warp so 256 NV
// columns; the warps of a row are a team.  One CTA per SM holds as many teams as
// its warps make, each on its own way over rows a grid apart.  Copies run ahead
// of the arithmetic, asynchronously, into slots of shared memory that only the
// copying lane reads: there is nothing to wait for but its own copies.  What a
// team waits for are its sums: one barrier for the mean and one for the sums
// that need it.
//
// LEAN: RMS norm without bias; otherwise either norm, with or without one.
__host__ __device__ constexpr int warps_of(int nv) { return nv == 4 ? 16 : nv == 2 ? 24 : 32; }  // per SM: by registers
constexpr int kMostWarps = 32;

struct NoMask {
  __device__ __forceinline__ NoMask(const Drop&, uint64_t) {}
  __device__ __forceinline__ void apply(uint64_t, float (&)[8]) const {}
  __device__ __forceinline__ void add(uint64_t, float (&)[8], float (&)[8]) const {}
};

// FULL: every vector exists.
template <int NV, bool FULL>
struct Team {
  int warps;       // of a row
  int id, teams;   // this thread's team, teams in the CTA
  int warp, lane;  // this thread's place in its team
  int col;         // first column of its first vector
  bool exists[FULL ? 1 : NV];
  __device__ __forceinline__ bool live(int j) const { return FULL || exists[FULL ? 0 : j]; }
  __device__ __forceinline__ explicit Team(const NormParams& p) {
    warps = p.warps;
    teams = blockDim.x / (32 * p.warps);
    id = (threadIdx.x >> 5) / p.warps;
    warp = (threadIdx.x >> 5) - id * p.warps;
    lane = threadIdx.x & 31;
    col = warp * NV * 256 + lane * 8;
    if (!FULL)
#pragma unroll
      for (int j = 0; j < NV; ++j) exists[j] = col + j * 256 < p.D;
  }
};

// Slots of the warps' sums, by turns of two: a set is used again two sums later
// at the earliest, when every thread has passed the barrier between.  A team's
// row of slots is as long as the team, rounded up to four, with zeros behind.
template <int N>
struct Slots {
  float f[2][N][kMostWarps];
};
template <int N>
__device__ __forceinline__ void clear(Slots<N>& s) {
  for (int i = threadIdx.x; i < static_cast<int>(sizeof(s) / 4); i += blockDim.x) (&s.f[0][0][0])[i] = 0.f;
}

// Sums of N numbers over the row's team, added in one order.
template <int N, int NV, bool FULL>
__device__ __forceinline__ void team_sum(float (&v)[N], Slots<N>& s, int turn, const Team<NV, FULL>& t) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  if (NV == 1 || t.warps == 1) return;  // NV = 1 holds rows of one warp only
  const int quads = (t.warps + 3) >> 2;
  float* slot = &s.f[turn][0][t.id * quads * 4];
  if (t.lane == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) slot[i * kMostWarps + t.warp] = v[i];
  __syncwarp();  // the barrier counts whole warps
  asm volatile("barrier.sync %0, %1;" ::"r"(t.id + 1), "r"(t.warps * 32) : "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = 0.f;
  for (int k = 0; k < quads; ++k)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float4 f = *reinterpret_cast<const float4*>(slot + i * kMostWarps + k * 4);
      v[i] += (f.x + f.y) + (f.z + f.w);
    }
}

// This lane's slots in the ring: blocks of a row's part, 512 NV bytes of a warp.
template <int NV, bool FULL>
__device__ __forceinline__ void copy_row(uint32_t block, const bf16* from, const Team<NV, FULL>& t) {
#pragma unroll
  for (int j = 0; j < NV; ++j)
    if (t.live(j))
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(block + j * 512), "l"(from + j * 256) : "memory");
}
__device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// Dead vectors are never copied: their slots are zeros from the start.
template <int BLOCKS, int NV, bool FULL>
__device__ __forceinline__ uint32_t ring_of(const uint8_t* ring, const Team<NV, FULL>& t) {
  const uint32_t at = smem_u32(ring) + (threadIdx.x >> 5) * (BLOCKS * NV * 512) + t.lane * 16;
#pragma unroll
  for (int j = 0; j < NV; ++j)
    if (!t.live(j))
      for (int i = 0; i < BLOCKS; ++i) st_shared_v4(at + (i * NV + j) * 512, 0, 0, 0, 0);
  return at;
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
template <int N>
__device__ __forceinline__ float f2_sum(const uint64_t (&v)[N]) {
  uint64_t s = v[0];
#pragma unroll
  for (int i = 1; i < N; ++i) s = f2_add(s, v[i]);
  float a, b;
  f2_unpack(s, a, b);
  return a + b;
}

// Vector j of a weight (at any float) as four pairs; none or dead: zeros.
template <int NV, bool FULL>
__device__ __forceinline__ void weight4(const float* w, const Team<NV, FULL>& t, int j, uint64_t (&v)[4]) {
  const float* at = w + t.col + j * 256;
  const bool on = t.live(j) && w != nullptr;
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = on ? f2_pack(__ldg(at + 2 * e), __ldg(at + 2 * e + 1)) : 0;
}

// Rows of x (and of res) in the ring: the one being worked on and the next.  With
// two on their way the reads crowd out the writes: RMS norm of 65536 x 5120 takes
// 227 us for 210.
constexpr int kFwdRows = 2;

template <int NV, bool RES, bool DROP, bool LEAN, bool FULL>
__global__ void __launch_bounds__(warps_of(NV) * 32, 1) layer_norm_fwd_kernel(const __grid_constant__ NormParams p) {
  constexpr int T = RES ? 2 : 1, S = kFwdRows, kBlock = NV * 512;
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ __align__(16) Slots<1> means, squares;
  const Team<NV, FULL> t(p);
  if (NV > 1) {
    clear(means);
    clear(squares);
    __syncthreads();
  }
  const uint32_t rows = static_cast<uint32_t>(p.L), step = gridDim.x * t.teams;  // rows below 2^31
  uint32_t row = blockIdx.x * t.teams + t.id, ahead = row;
  const uint32_t base = ring_of<T * S>(ring, t);
  uint32_t at = base;
  auto start = [&] {
    if (ahead < rows) {
      copy_row(at, p.x.p + ahead * p.x.row + t.col, t);
      if (RES) copy_row(at + kBlock, p.res.p + ahead * p.res.row + t.col, t);
    }
    commit();
    at = at == base + (S - 1) * T * kBlock ? base : at + T * kBlock;
    ahead += step;
  };
#pragma unroll
  for (int i = 0; i + 1 < S; ++i) start();
  uint64_t w[NV][4], b[LEAN ? 1 : NV][4];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    weight4(p.w, t, j, w[j]);
    if (!LEAN) weight4(p.b, t, j, b[j]);
  }
  std::conditional_t<DROP, Mask, NoMask> mask(p.drop, DROP ? drop_call(p.drop) : 0);
  const float inv = 1.f / p.D;
  for (int turn = 0; row < rows; row += step, turn ^= 1) {
    start();
    wait<S - 1>();  // the oldest row has arrived: it stands behind the newest one
    bf16* const s_to = RES || DROP ? p.s.p + row * p.s.row + t.col : nullptr;
    uint64_t s[NV][4], sum[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      uint4 u = ld_shared_v4(at + j * 512);
      if (RES || DROP) {
        float v[8];
        unpack8(u, v);
        const uint64_t at_e = static_cast<uint64_t>(row) * static_cast<uint32_t>(p.D) + t.col + j * 256;
        if (RES) {
          float r[8];
          unpack8(ld_shared_v4(at + kBlock + j * 512), r);
          if (!DROP)
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = __fadd_rn(r[e], v[e]);
          else if (t.live(j))
            mask.add(at_e, v, r);
          if (DROP)
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = r[e];
        } else if (t.live(j)) {
          mask.apply(at_e, v);
        }
        u = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                       pack_bf16x2(v[6], v[7]));
        if (t.live(j)) st_global_v4(s_to + j * 256, u.x, u.y, u.z, u.w);
      }
      unpack4(u, s[j]);  // the norm is of s as it is stored
      if (!LEAN) sum[j] = f2_add(f2_add(s[j][0], s[j][1]), f2_add(s[j][2], s[j][3]));
    }
    if (!LEAN) {
      float m[1] = {f2_sum(sum)};
      team_sum(m, means, turn, t);
      m[0] = p.rms ? 0.f : m[0] * inv;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const uint64_t mm = f2_both(t.live(j) ? m[0] : 0.f);
#pragma unroll
        for (int e = 0; e < 4; ++e) s[j][e] = f2_sub(s[j][e], mm);
      }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      sum[j] = f2_fma(s[j][0], s[j][0], f2_mul(s[j][1], s[j][1]));
      sum[j] = f2_fma(s[j][2], s[j][2], f2_fma(s[j][3], s[j][3], sum[j]));
    }
    float q[1] = {f2_sum(sum)};
    team_sum(q, squares, turn, t);
    const uint64_t r = f2_both(rsqrtf(q[0] * inv + p.eps));
    bf16* const y_to = p.y.p + row * p.y.row + t.col;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      uint32_t y[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[j][e] = f2_mul(s[j][e], r);
        y[e] = round2(LEAN ? f2_mul(s[j][e], w[j][e]) : f2_fma(s[j][e], w[j][e], b[j][e]));
      }
      if (t.live(j)) st_global_v4(y_to + j * 256, y[0], y[1], y[2], y[3]);
    }
  }
  wait<0>();
}

// Blocks of the ring per warp: two rows of s and dy, and one of ds, which is
// read last: its next row is on its way from then on.  The weight stands in
// shared memory in front of the ring, where all teams read it, once per row.
__host__ __device__ constexpr int bwd_blocks(bool ds) { return ds ? 5 : 4; }

// Each lane keeps its columns' sums of dw and db in registers over all of its
// rows; a CTA writes one share of each (its teams' shares added in order),
// which weight_sum_kernel adds up.
//
// Registers decide: what spills costs more than what is read again.  Held from
// one pass over the row to the next are s where nothing else needs the room, and
// g = w dy but where db's sums do (whole-warp rows with mask, without ds, hold it
// all the same: 65536 x 5120 537 us for 598; with ds 622 for 608).  With db and rows
// that leave lanes to spare, 12 warps hold g and do not spill where 16 do (65536 x
// 2560 199 us for 208, with ds 215 for 230, with mask too 341 for 372; but rows of
// five and seven warps leave too many of 12 out: 32768 x 5000 242 for 227, 16384 x
// 7000 202 for 177).
template <int NV, bool DS, bool DROP, bool LEAN, bool FULL, int WARPS>
__global__ void __launch_bounds__(WARPS * 32, 1) layer_norm_bwd_kernel(const __grid_constant__ NormParams p) {
  constexpr int kBlock = NV * 512;
  constexpr bool kHoldS = LEAN && !DS && !DROP, kHoldG = LEAN || NV == 1 || WARPS == 12 || (FULL && DROP && !DS);
  extern __shared__ __align__(16) uint8_t shared[];
  __shared__ __align__(16) Slots<1> means;
  __shared__ __align__(16) Slots<LEAN ? 2 : 3> sums;
  let_next_start();
  const Team<NV, FULL> t(p);
  const uint32_t rows = static_cast<uint32_t>(p.L), step = gridDim.x * t.teams;  // rows below 2^31
  uint32_t row = blockIdx.x * t.teams + t.id, ahead = row;
  uint8_t* ring = shared + t.warps * NV * 1024;
  const uint32_t base = ring_of<bwd_blocks(DS)>(ring, t);
  const uint32_t weight = smem_u32(shared) + t.warp * NV * 1024 + t.lane * 16;
  const uint32_t ds_at = base + 4 * kBlock;
  uint32_t at = 0;  // of the pair of blocks that is filled next: 0 or 2 kBlock
  auto start = [&] {
    if (ahead < rows) {
      copy_row(base + at, p.s.p + ahead * p.s.row + t.col, t);
      copy_row(base + at + kBlock, p.dy.p + ahead * p.dy.row + t.col, t);
    }
    commit();
    at ^= 2 * kBlock;
    ahead += step;
  };
  auto start_ds = [&](uint32_t of) {
    if (of < rows) copy_row(ds_at, p.ds.p + of * p.ds.row + t.col, t);
    commit();
  };
  start();
  if (DS) start_ds(row);
  clear(means);
  clear(sums);
  if (t.id == 0)  // the weight, in two planes of 16 bytes a lane
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      uint64_t v[4];
      weight4(p.w, t, j, v);
      float f[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) f2_unpack(v[e], f[2 * e], f[2 * e + 1]);
#pragma unroll
      for (int h = 0; h < 2; ++h)
        st_shared_v4(weight + (2 * j + h) * 512, __float_as_uint(f[4 * h]), __float_as_uint(f[4 * h + 1]),
                     __float_as_uint(f[4 * h + 2]), __float_as_uint(f[4 * h + 3]));
    }
  __syncthreads();
  auto read_w = [&](int j, uint64_t (&w)[4]) {
    const uint4 a = ld_shared_v4(weight + 2 * j * 512), b = ld_shared_v4(weight + (2 * j + 1) * 512);
    w[0] = f2_pack(__uint_as_float(a.x), __uint_as_float(a.y)), w[1] = f2_pack(__uint_as_float(a.z), __uint_as_float(a.w));
    w[2] = f2_pack(__uint_as_float(b.x), __uint_as_float(b.y)), w[3] = f2_pack(__uint_as_float(b.z), __uint_as_float(b.w));
  };
  uint64_t dw[NV][4], db[NV][4];
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) dw[j][e] = db[j][e] = 0;
  const uint64_t call = DROP ? drop_call(p.drop) : 0;
  const float inv = 1.f / p.D;
  for (int turn = 0; row < rows; row += step, turn ^= 1) {
    start();
    wait<DS ? 2 : 1>();  // this row's s and dy
    const uint32_t mine = base + at;
    uint4 su[kHoldS ? NV : 1];
    if (kHoldS)
#pragma unroll
      for (int j = 0; j < NV; ++j) su[j] = ld_shared_v4(mine + j * 512);
    float m = 0.f;
    if (!LEAN) {
      uint64_t sum[NV];
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        uint64_t a[4];
        unpack4(ld_shared_v4(mine + j * 512), a);
        sum[j] = f2_add(f2_add(a[0], a[1]), f2_add(a[2], a[3]));
      }
      float v[1] = {f2_sum(sum)};
      team_sum(v, means, turn, t);
      m = p.rms ? 0.f : v[0] * inv;
    }
    uint64_t gh[kHoldG ? NV : 1][4];
    uint64_t sq[2] = {0, 0}, sg[2] = {0, 0}, sd[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      uint64_t a[4], w[4];
      read_w(j, w);
      unpack4(kHoldS ? su[j] : ld_shared_v4(mine + j * 512), a);
      uint64_t (&g)[4] = gh[kHoldG ? j : 0];
      unpack4(ld_shared_v4(mine + kBlock + j * 512), g);
      if (!LEAN) {
        const uint64_t mm = f2_both(t.live(j) ? m : 0.f);
#pragma unroll
        for (int e = 0; e < 4; ++e) a[e] = f2_sub(a[e], mm);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        g[e] = f2_mul(g[e], w[e]);
        sq[e & 1] = f2_fma(a[e], a[e], sq[e & 1]);
        if (!LEAN) sg[e & 1] = f2_add(sg[e & 1], g[e]);
        sd[e & 1] = f2_fma(g[e], a[e], sd[e & 1]);
      }
    }
    float v[LEAN ? 2 : 3];
    v[0] = f2_sum(sq);
    v[1] = f2_sum(sd);
    if constexpr (!LEAN) v[2] = f2_sum(sg);
    team_sum(v, sums, turn, t);
    const float r = rsqrtf(v[0] * inv + p.eps);
    const uint64_t rr = f2_both(r), mr = f2_both(-m * r);
    uint64_t c0 = 0;  // -r mean(g)
    if constexpr (!LEAN) c0 = f2_both(p.rms ? 0.f : -r * (v[2] * inv));
    const uint64_t c1 = f2_both(-r * (r * (v[1] * inv)));  // -r mean(g n)
    bf16* const dres = p.dres.p + row * p.dres.row + t.col;
    bf16* const dx = DROP ? p.dx.p + row * p.dx.row + t.col : nullptr;
    if (DS) wait<1>();                                     // this row's ds
    std::conditional_t<DROP, Mask, NoMask> mask(p.drop, call);  // made anew: the row's sums need the registers
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      uint64_t a[4], d[4];
      unpack4(kHoldS ? su[j] : ld_shared_v4(mine + j * 512), a);
      unpack4(ld_shared_v4(mine + kBlock + j * 512), d);
      uint64_t (&g)[4] = gh[kHoldG ? j : 0];
      if (!kHoldG) {
        read_w(j, g);
#pragma unroll
        for (int e = 0; e < 4; ++e) g[e] = f2_mul(g[e], d[e]);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint64_t n = LEAN ? f2_mul(a[e], rr) : f2_fma(a[e], rr, mr);
        dw[j][e] = f2_fma(d[e], n, dw[j][e]);
        if (!LEAN) db[j][e] = f2_add(db[j][e], d[e]);
        a[e] = f2_fma(n, c1, LEAN ? f2_mul(g[e], rr) : f2_fma(g[e], rr, c0));
      }
      if (DS) {
        unpack4(ld_shared_v4(ds_at + j * 512), d);
#pragma unroll
        for (int e = 0; e < 4; ++e) a[e] = f2_add(a[e], d[e]);
      }
      if (t.live(j)) {
        st_global_v4(dres + j * 256, round2(a[0]), round2(a[1]), round2(a[2]), round2(a[3]));
        if (DROP) {
          float f[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) f2_unpack(a[e], f[2 * e], f[2 * e + 1]);
          mask.apply(static_cast<uint64_t>(row) * static_cast<uint32_t>(p.D) + t.col + j * 256, f);
          store8(dx + j * 256, f);
        }
      }
    }
    if (DS) start_ds(row + step);
  }
  wait<0>();
  // Shares [dw][db] of the CTA; of several teams by way of the ring's memory,
  // one half of them at a time.
  float* out = p.partial + static_cast<int64_t>(blockIdx.x) * 2 * p.D;
#pragma unroll
  for (int half = 0; half < (LEAN ? 1 : 2); ++half, out += p.D) {
    float* share = t.teams == 1 ? out : reinterpret_cast<float*>(ring) + t.id * p.D;
    __syncthreads();  // every team's copies, and the half before, have been read
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (t.live(j)) {
        uint64_t* to = reinterpret_cast<uint64_t*>(share + t.col + j * 256);
#pragma unroll
        for (int e = 0; e < 4; ++e) to[e] = half ? db[j][e] : dw[j][e];
      }
    if (t.teams == 1) continue;
    __syncthreads();
    for (int i = threadIdx.x; i < p.D; i += blockDim.x) {
      float f = 0.f;
      for (int k = 0; k < t.teams; ++k) f += reinterpret_cast<float*>(ring)[k * p.D + i];
      out[i] = f;
    }
  }
}

struct SumParams {
  const float* partial;
  int n, D;
  float *dw, *db;
};

// dw[i] and db[i], the sums over the n rows of partial [n][2][D], in a fixed
// order: 32 rows of threads take every 32nd row each, four columns a thread; the
// four rows of a warp are added, then the eight warps' sums.
constexpr int kSumCols = 32;

__global__ void __launch_bounds__(256) weight_sum_kernel(const __grid_constant__ SumParams p) {
  __shared__ float4 part[8][kSumCols / 4];
  after_previous();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int quad = lane & 7, row = warp * 4 + (lane >> 3);
  const int col = blockIdx.x * kSumCols + quad * 4;  // of 2 D, or D without db; D is a multiple of 8
  const int cols = p.db ? 2 * p.D : p.D;
  float4 g = make_float4(0.f, 0.f, 0.f, 0.f);
  if (col < cols)
#pragma unroll 5
    for (int r = row; r < p.n; r += 32) {
      const float4 f = __ldcg(reinterpret_cast<const float4*>(p.partial + static_cast<int64_t>(r) * 2 * p.D + col));
      g.x += f.x, g.y += f.y, g.z += f.z, g.w += f.w;
    }
#pragma unroll
  for (int o = 8; o < 32; o <<= 1) {
    g.x += __shfl_xor_sync(0xffffffffu, g.x, o);
    g.y += __shfl_xor_sync(0xffffffffu, g.y, o);
    g.z += __shfl_xor_sync(0xffffffffu, g.z, o);
    g.w += __shfl_xor_sync(0xffffffffu, g.w, o);
  }
  if (lane < 8) part[warp][quad] = g;
  __syncthreads();
  const int at = blockIdx.x * kSumCols + threadIdx.x;
  if (threadIdx.x >= kSumCols || at >= cols) return;
  float s = 0.f;
#pragma unroll
  for (int w = 0; w < 8; ++w) s += reinterpret_cast<const float*>(&part[w][0])[threadIdx.x];
  (at < p.D ? p.dw[at] : p.db[at - p.D]) = s;
}

// ------------------------------------------------------------------- host

bool norm_ok(const upipe_norm_cfg* c) {
  return c && c->L >= 1 && c->L <= 0x7fffffffLL && c->D >= 8 && c->D <= UPIPE_NORM_MAX_D && c->D % 8 == 0 &&
         (c->rms == 0 || c->rms == 1) && c->eps >= 0.f && std::isfinite(c->eps);
}

bool weight_ok(const float* w) { return w && reinterpret_cast<uintptr_t>(w) % sizeof(float) == 0; }

Mat mat_of(const upipe_rows* t) { return t ? Mat{reinterpret_cast<bf16*>(t->p), t->row} : Mat{nullptr, 0}; }

template <bool RES>
cudaError_t launch_dropout(DropParams& p, cudaStream_t st) {
  const bool flat = p.L == 1 || (p.x.row == p.D && p.y.row == p.D && (!RES || p.res.row == p.D));
  if (flat) {
    constexpr int64_t kPer = static_cast<int64_t>(kThreads) * kDropVecs;
    const int64_t grid = (p.L * (p.D / 8) + kPer - 1) / kPer;
    if (grid <= 0x7fffffff) {
      dropout_kernel<RES, true><<<static_cast<unsigned>(grid), kThreads, 0, st>>>(p);
      return cudaGetLastError();
    }
  }
  p.across = 8;  // rows of fewer vectors share a CTA
  while (p.across < kThreads && p.across * 8 < p.D) p.across *= 2;
  const int64_t rows = kThreads / p.across;
  dropout_kernel<RES, false><<<static_cast<unsigned>((p.L + rows - 1) / rows), kThreads, 0, st>>>(p);
  return cudaGetLastError();
}

// How rows of D elements lie: vectors of a lane, warps of a row, rows at once in
// one CTA (no more than it takes to give every SM one), and CTAs that walk the
// rows.  Four vectors a lane make the least of the sums over lanes and warps;
// fewer, with more warps, where four would stand half empty: forward of 131072
// rows of 256 24, 28 and 36 us with one, two and four; with mean and bias, 65536
// rows of 1536 71 and 72 with two and four, backward 121 and 136, 2048 91 and 93,
// backward 158 and 133.
struct Layout {
  int nv, warps, teams, ctas;
};
Layout layout_of(int64_t L, int D, int most_warps = kMostWarps) {
  Layout y;
  y.nv = D <= 256 ? 1 : D <= 512 || (D > 1024 && D <= 1536) ? 2 : 4;
  y.warps = (D + y.nv * 256 - 1) / (y.nv * 256);
  const int64_t want = (L + 151) / 152;
  const int held = most_warps < warps_of(y.nv) ? most_warps : warps_of(y.nv);
  const int most = held < y.warps ? 1 : held / y.warps;
  y.teams = static_cast<int>(want < most ? want : most);
  const int64_t need = (L + y.teams - 1) / y.teams;
  y.ctas = static_cast<int>(need < 152 ? need : 152);
  return y;
}
static_assert(UPIPE_NORM_MAX_D <= 1024 * warps_of(4), "the longest row fits a CTA");

// blocks: of the ring per warp; weights: whether the weight stands before it.
template <void (*kKernel)(NormParams)>
cudaError_t launch_rows(const Layout& y, int blocks, bool weights, NormParams& p, cudaStream_t st) {
  static std::atomic<uint64_t> allowed{0};
  const int block = y.nv * 512, warps = y.warps * y.teams;
  const int bytes = warps * blocks * block + (weights ? 2 * y.warps * block : 0);
  // for the longest rows: the same for every call of the kernel
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kKernel),
                                   warps_of(y.nv) * (blocks + (weights ? 2 : 0)) * block, allowed);
  if (e != cudaSuccess) return e;
  p.warps = y.warps;
  p.ctas = y.ctas;
  kKernel<<<static_cast<unsigned>(y.ctas), 32 * warps, bytes, st>>>(p);
  return cudaGetLastError();
}

// Rows of whole warps have kernels of their own where that pays, with means or
// biases: 65536 x 5120 backward 340 us for 403 (with mask and ds 608 for 726),
// forward with mask and residual 462 for 503.
template <int NV, bool RES, bool DROP>
cudaError_t launch_fwd_nv(const Layout& y, NormParams& p, cudaStream_t st) {
  constexpr int kBlocks = kFwdRows * (RES ? 2 : 1);
  if (p.rms && !p.b) return launch_rows<layer_norm_fwd_kernel<NV, RES, DROP, true, false>>(y, kBlocks, false, p, st);
  if constexpr (NV == 4)
    if (p.D % 1024 == 0)
      return launch_rows<layer_norm_fwd_kernel<NV, RES, DROP, false, true>>(y, kBlocks, false, p, st);
  return launch_rows<layer_norm_fwd_kernel<NV, RES, DROP, false, false>>(y, kBlocks, false, p, st);
}
template <int NV, bool DS, bool DROP>
cudaError_t launch_bwd_nv(const Layout& y, NormParams& p, bool lean, bool few, cudaStream_t st) {
  constexpr int kWarps = warps_of(NV), kBlocks = bwd_blocks(DS);
  if (lean) return launch_rows<layer_norm_bwd_kernel<NV, DS, DROP, true, false, kWarps>>(y, kBlocks, true, p, st);
  if constexpr (NV == 4 && (DS || !DROP))
    if (few) return launch_rows<layer_norm_bwd_kernel<NV, DS, DROP, false, false, 12>>(y, kBlocks, true, p, st);
  if constexpr (NV == 4)
    if (p.D % 1024 == 0)
      return launch_rows<layer_norm_bwd_kernel<NV, DS, DROP, false, true, kWarps>>(y, kBlocks, true, p, st);
  return launch_rows<layer_norm_bwd_kernel<NV, DS, DROP, false, false, kWarps>>(y, kBlocks, true, p, st);
}

template <bool RES, bool DROP>
cudaError_t launch_fwd(NormParams& p, cudaStream_t st) {
  // With a mask and a residual, rows of one or two warps of four vectors a lane do
  // better with 12 warps of 16: 131072 x 768 124 us for 144, 65536 x 2048 175 for
  // 191; longer ones mostly do not (65536 x 2560 221 for 210, 32768 x 3584 169 for
  // 152, but 32768 x 4096 174 for 187).
  const bool few = RES && DROP && p.D > 512 && p.D <= 2048 && (p.D <= 1024 || p.D > 1536);
  const Layout y = layout_of(p.L, p.D, few ? 12 : kMostWarps);
  switch (y.nv) {
    case 1: return launch_fwd_nv<1, RES, DROP>(y, p, st);
    case 2: return launch_fwd_nv<2, RES, DROP>(y, p, st);
  }
  return launch_fwd_nv<4, RES, DROP>(y, p, st);
}

template <bool DS, bool DROP>
cudaError_t launch_bwd(NormParams& p, bool bias, cudaStream_t st) {
  // 12 warps whose registers do not spill for 16 that do: rows of two to four warps
  // with lanes to spare.
  const bool lean = p.rms && !bias;
  const bool few = !lean && p.D % 1024 != 0 && (DS || !DROP) && p.D > 1536 && p.D <= 4096;
  const Layout y = layout_of(p.L, p.D, few ? 12 : kMostWarps);
  switch (y.nv) {
    case 1: return launch_bwd_nv<1, DS, DROP>(y, p, lean, false, st);
    case 2: return launch_bwd_nv<2, DS, DROP>(y, p, lean, false, st);
  }
  return launch_bwd_nv<4, DS, DROP>(y, p, lean, few, st);
}

cudaError_t launch_weight_sum(const NormParams& p, float* dw, float* db, cudaStream_t st) {
  const SumParams s{p.partial, p.ctas, p.D, dw, db};
  const unsigned cols = static_cast<unsigned>(db ? 2 * p.D : p.D);
  return launch_next(weight_sum_kernel, (cols + kSumCols - 1) / kSumCols, 256, 0, st, s);
}

// The part of a norm's parameters that both directions share.
bool norm_params(const upipe_norm_cfg* c, const upipe_dropout* drop, NormParams* p) {
  std::memset(p, 0, sizeof(*p));
  p->L = c->L;
  p->D = c->D;
  p->rms = c->rms;
  p->eps = c->eps;
  return !drop || drop_of(drop, &p->drop);
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
  UPIPE_LAUNCH(UPIPE_KIND_DROPOUT, res ? launch_dropout<true>(p, st) : launch_dropout<false>(p, st));
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
  UPIPE_LAUNCH(UPIPE_KIND_LAYER_NORM_FWD, res ? (drop ? launch_fwd<true, true>(p, st) : launch_fwd<true, false>(p, st))
                                              : (drop ? launch_fwd<false, true>(p, st) : launch_fwd<false, false>(p, st)));
  return UPIPE_OK;
}

size_t upipe_layer_norm_workspace_bytes(const upipe_norm_cfg* c) {
  return norm_ok(c) ? static_cast<size_t>(c->L < 152 ? c->L : 152) * 2 * c->D * sizeof(float) : 0;
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
  const bool bias = db != nullptr;
  UPIPE_LAUNCH(UPIPE_KIND_LAYER_NORM_BWD,
               ds ? (drop ? launch_bwd<true, true>(p, bias, st) : launch_bwd<true, false>(p, bias, st))
                  : (drop ? launch_bwd<false, true>(p, bias, st) : launch_bwd<false, false>(p, bias, st)));
  UPIPE_LAUNCH(UPIPE_KIND_NORM_SUM, launch_weight_sum(p, dw, db, st));
  return UPIPE_OK;
}

}  // extern "C"
