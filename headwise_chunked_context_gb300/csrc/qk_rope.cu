// Rotary positions of queries and keys, alone or in one pass with the RMS
// norm of each head, forward and backward, and their C entry points.
//
// Mathematics.  A head x of d elements, position p, frequencies f_i
// (i < rot / 2), magnitude c:
//   n = x / sqrt(mean(x^2) + eps),  z = w n                     (norm only)
//   y_a = c (z_a cos(p f_i) - z_b sin(p f_i))
//   y_b = c (z_a sin(p f_i) + z_b cos(p f_i))
// for the pair (a, b) = (i, i + rot/2) or (2i, 2i + 1); the elements from rot
// on pass through.  The backward turns dy by the transpose, dz, and
//   dw = sum dz n,  dn = w dz,  dx = (dn - n mean(dn n)) / sqrt(...),
// with the norm recomputed from x, which has to be read in any case.
//
// Angles.  p f_i reaches 2^31 radians, where fp32 has lost every digit.  A
// frequency enters as its turns per position, f / 2 pi modulo 1, in units of
// 2^-64; times the integer position in 64-bit wrapping arithmetic this IS the
// angle modulo one turn, with no range reduction and no fp64 (whose rate on
// this part would be the bound): off by p 2^-53 of f, as an fp64 product
// would be.  Its upper 32 bits go through sincospif, once per token and pair,
// shared by all heads of a token through shared memory.
//
// What bounds it: HBM.  Every element is read once and written once (the
// backward of the norm reads x and dy).  A warp owns one token (or a share of
// its heads when there are few tokens), a lane 16 elements of a head as two
// 16-byte vectors that hold both members of its 8 pairs, so the rotation
// stays in the lane and the norm is a reduction over d / 16 lanes.  Heads
// whose pairs do not fall on such vectors take the same kernel with 8-byte
// ones, or with single elements (path_of).
#include <cmath>
#include <cstring>

#include "host.h"
#include "sm103_ptx.cuh"

namespace upipe {
namespace {

using bf16 = __nv_bfloat16;

constexpr int kMaxPairs = UPIPE_ROPE_MAX_D / 2;
constexpr int kWarps = 8;  // per CTA

enum Mode { kTurn = 0, kNormTurn = 1 };  // of the forward kernel
// How a lane holds its pairs: vectors of 8 or 4 elements in either layout, or
// single elements (half layout; interleaved pairs always lie in vectors).
enum Path { kHalf8 = 0, kInter8 = 1, kHalf4 = 2, kInter4 = 3, kScalar = 4 };
__host__ __device__ constexpr bool is_half(int path) { return path == kHalf8 || path == kHalf4; }
__host__ __device__ constexpr int vec_of(int path) { return path == kHalf8 || path == kInter8 ? 8 : 4; }

// A [L, heads, d] tensor of bf16 with its strides in elements.
struct Rows {
  bf16* p;
  int64_t row, head;
};

struct QkParams {
  int64_t L, pos0;
  int nheads[2];  // query heads, key heads
  int d, rot;
  int lanes;      // lanes of a warp that share a head (a power of two)
  int parts;      // shares that a token's heads are split into
  float magnitude, eps, sign;  // sign: -1 turns by the transpose
  Rows x[2];   // the input (the norm's, or what is turned)
  Rows dy[2];  // backward: gradient of the output
  Rows y[2];   // the output, or dx
  const float* w[2];
  const int32_t* positions;
  float* partial;  // backward: [gridDim.x][2][d] shares of dw
  uint64_t step[kMaxPairs];
};

// Which elements of a head a lane holds: N pairs (a[e], b[e]), kept as N/2
// packed fp32 pairs of the first members and N/2 of the second (u[i] = (a[2i],
// a[2i+1]), v likewise), which halves the arithmetic's issue slots.
template <int PATH>
struct Lane {
  static constexpr int N = vec_of(PATH);  // elements per vector, pairs per lane
  static constexpr int M = N / 2;
  int sub;    // lane within its head
  int off_a;  // vector paths: first elements of the lane's two vectors
  int off_b;
  bool live;
  int d, rot;
  int turn_a, turn_b;  // interleaved: how many pairs of each vector's start turn

  __device__ __forceinline__ Lane(const QkParams& p, int lane) {
    d = p.d;
    rot = p.rot;
    sub = lane % p.lanes;
    live = PATH == kScalar || sub * 2 * N < d;
    // Neighbouring lanes hold neighbouring vectors, so that each access of a
    // warp covers whole sectors: of the rotated half the first vectors and,
    // rot/2 further, their partners; of what passes (and in the interleaved
    // layout, whose pairs lie inside a vector) the two halves likewise.
    const int turned = is_half(PATH) ? rot / (2 * N) : 0;  // lanes of the rotated part
    if (sub < turned) {
      off_a = N * sub;
      off_b = rot / 2 + N * sub;
    } else {
      const int from = 2 * N * turned;
      off_a = from + N * (sub - turned);
      off_b = off_a + (d - from) / 2;
    }
    turn_a = (rot - off_a) / 2;
    turn_b = (rot - off_b) / 2;
  }
  __device__ __forceinline__ int pair(int e) const {
    if (PATH == kScalar) return sub + 32 * e;
    if (is_half(PATH)) return N * sub + e;
    return e < M ? off_a / 2 + e : off_b / 2 + e - M;
  }
  __device__ __forceinline__ bool holds(int e) const { return PATH == kScalar ? 2 * pair(e) < d : live; }
  // Whether pair e turns, and word e of the lane's vectors (Raw::w) with it: a
  // word is a pair, or, in the half layout, part of two of a lane's pairs, which
  // all turn or all do not.  (The counts spare the interleaved layout a sum per
  // pair: 142 to 124 us for the norm's backward of 20011 tokens, 64 of 128.)
  __device__ __forceinline__ bool turns(int e) const {
    if (PATH == kScalar || is_half(PATH)) return 2 * pair(is_half(PATH) ? 0 : e) < rot;
    return e < M ? e < turn_a : e - M < turn_b;
  }
  __device__ __forceinline__ int first(int e) const {
    if (is_half(PATH)) return off_a + e;
    return PATH == kScalar && turns(e) ? pair(e) : 2 * pair(e);
  }
  __device__ __forceinline__ int second(int e) const {
    if (is_half(PATH)) return off_b + e;
    return PATH == kScalar && turns(e) ? pair(e) + rot / 2 : 2 * pair(e) + 1;
  }
};

// What a lane has in flight of one head: the words of its two vectors (the
// scalar path: one word per pair).
template <int PATH>
struct Raw {
  uint32_t w[Lane<PATH>::N];
  // Two-byte reads, volatile: an in-place call's own writes follow them.
  __device__ __forceinline__ void load(const bf16* head, bool on, const Lane<PATH>& ln) {
    const volatile uint16_t* h = reinterpret_cast<const volatile uint16_t*>(head);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      w[e] = 0u;
      if (on && ln.holds(e)) {
        const uint32_t lo = h[ln.first(e)], hi = h[ln.second(e)];
        w[e] = lo | (hi << 16);
      }
    }
  }
  __device__ __forceinline__ void unpack(uint64_t (&u)[Lane<PATH>::M], uint64_t (&v)[Lane<PATH>::M]) const {
    constexpr int M = Lane<PATH>::M;
#pragma unroll
    for (int i = 0; i < M; ++i) {
      if (is_half(PATH)) {
        u[i] = f2_pack(bf16_lo(w[i]), bf16_hi(w[i]));
        v[i] = f2_pack(bf16_lo(w[M + i]), bf16_hi(w[M + i]));
      } else {
        u[i] = f2_pack(bf16_lo(w[2 * i]), bf16_lo(w[2 * i + 1]));
        v[i] = f2_pack(bf16_hi(w[2 * i]), bf16_hi(w[2 * i + 1]));
      }
    }
  }
};

// T tensors' heads in flight ahead of the arithmetic.  The vector paths copy
// them asynchronously into the lane's own slots of a ring of S steps in
// shared memory: what is in flight then costs no registers, and one warp
// keeps S steps of loads open (in registers there was room for one, and a
// backward of 16 warps per SM ran at 4.4 TB/s).  A lane reads back only what
// it copied itself, so there is nothing to synchronise but the lane's own
// copies: two into one slot have no order unless the first has been waited for,
// so a pipe is drained before the next one takes its ring.  The scalar path
// holds one step in registers (a copy is four bytes at least).
template <int PATH, int T, int S>
struct Pipe {
  static constexpr int kBytes = PATH == kScalar ? 0 : S * T * 2 * 32 * 16;  // per warp
  uint32_t slot;
  int at;
  Raw<PATH> held[PATH == kScalar ? T : 1];

  __device__ __forceinline__ Pipe(uint32_t ring, int warp, int lane)
      : slot(ring + warp * kBytes + lane * 16), at(0) {}
  // One vector; off: zeros, and nothing is read.
  static __device__ __forceinline__ void copy(uint32_t to, const bf16* from, bool on) {
    if constexpr (vec_of(PATH) == 8)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(on ? 16 : 0) : "memory");
    else
      asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(to), "l"(from), "r"(on ? 8 : 0) : "memory");
  }
  // Starts the copies of one step.
  __device__ __forceinline__ void start(const bf16* const (&head)[T], bool on, const Lane<PATH>& ln) {
    if constexpr (PATH == kScalar) {
#pragma unroll
      for (int t = 0; t < T; ++t) held[t].load(head[t], on, ln);
    } else {
#pragma unroll
      for (int t = 0; t < T; ++t) {
        const uint32_t to = slot + (at * T + t) * 1024;
        copy(to, on ? head[t] + ln.off_a : head[t], on);
        copy(to + 512, on ? head[t] + ln.off_b : head[t], on);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
      at = at + 1 == S ? 0 : at + 1;
    }
  }
  // Waits for the copies in flight (at the end: zeros for the steps past it).
  static __device__ __forceinline__ void drain() {
    if constexpr (PATH != kScalar) asm volatile("cp.async.wait_all;" ::: "memory");
  }
  static constexpr int kAhead = PATH == kScalar ? 1 : S - 1;  // steps to start before the first turn
  // Starts one more step and takes the oldest.
  __device__ __forceinline__ void turn(const bf16* const (&head)[T], bool on, const Lane<PATH>& ln,
                                       Raw<PATH> (&out)[T]) {
    if constexpr (PATH == kScalar) {
#pragma unroll
      for (int t = 0; t < T; ++t) out[t] = held[t];
      start(head, on, ln);
    } else {
      start(head, on, ln);
      asm volatile("cp.async.wait_group %0;" ::"n"(S - 1) : "memory");
#pragma unroll
      for (int t = 0; t < T; ++t) {  // the slot after the newest one's
        const uint32_t from = slot + (at * T + t) * 1024;
        if constexpr (vec_of(PATH) == 8) {
          const uint4 a = ld_shared_v4(from), b = ld_shared_v4(from + 512);
          const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
          for (int i = 0; i < 8; ++i) out[t].w[i] = w[i];
        } else {
          asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(out[t].w[0]), "=r"(out[t].w[1]) : "r"(from));
          asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(out[t].w[2]), "=r"(out[t].w[3]) : "r"(from + 512));
        }
      }
    }
  }
};

// Pairs 2 i and 2 i + 1 of a lane turned by their angles.  KEEP: those past rot
// stay as they are; times 1 and 0 an infinity of one member would make the other
// NaN.
template <int PATH, bool KEEP>
__device__ __forceinline__ void turn_pairs(const Lane<PATH>& ln, int i, uint64_t c, uint64_t s, uint64_t& u,
                                           uint64_t& v) {
  const uint64_t a = f2_sub(f2_mul(u, c), f2_mul(v, s));
  const uint64_t b = f2_fma(u, s, f2_mul(v, c));
  if (!KEEP) {
    u = a;
    v = b;
    return;
  }
  const bool t0 = ln.turns(2 * i), t1 = ln.turns(2 * i + 1);
  float a0, a1, b0, b1, u0, u1, v0, v1;
  f2_unpack(a, a0, a1);
  f2_unpack(b, b0, b1);
  f2_unpack(u, u0, u1);
  f2_unpack(v, v0, v1);
  u = f2_pack(t0 ? a0 : u0, t1 ? a1 : u1);
  v = f2_pack(t0 ? b0 : v0, t1 ? b1 : v1);
}

// Rounds the lane's pairs to bf16, the only rounding of the pass, and stores
// them.  COPY: pairs that do not turn are stored bit for bit as they were read.
template <int PATH, bool COPY>
__device__ __forceinline__ void store(bf16* head, const Lane<PATH>& ln, const uint64_t (&u)[Lane<PATH>::M],
                                      const uint64_t (&v)[Lane<PATH>::M], const Raw<PATH>& as_read) {
  constexpr int M = Lane<PATH>::M;
  uint32_t w[2 * M];
#pragma unroll
  for (int i = 0; i < M; ++i) {
    float a0, a1, b0, b1;
    f2_unpack(u[i], a0, a1);
    f2_unpack(v[i], b0, b1);
    w[is_half(PATH) ? i : 2 * i] = is_half(PATH) ? pack_bf16x2(a0, a1) : pack_bf16x2(a0, b0);
    w[is_half(PATH) ? M + i : 2 * i + 1] = is_half(PATH) ? pack_bf16x2(b0, b1) : pack_bf16x2(a1, b1);
  }
  if (COPY) {
#pragma unroll
    for (int j = 0; j < 2 * M; ++j)
      if (!ln.turns(j)) w[j] = as_read.w[j];
  }
  if constexpr (PATH == kScalar) {
    uint16_t* h = reinterpret_cast<uint16_t*>(head);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (ln.holds(e)) {
        h[ln.first(e)] = static_cast<uint16_t>(w[e]);
        h[ln.second(e)] = static_cast<uint16_t>(w[e] >> 16);
      }
  } else if constexpr (M == 4) {
    st_global_v4(head + ln.off_a, w[0], w[1], w[2], w[3]);
    st_global_v4(head + ln.off_b, w[4], w[5], w[6], w[7]);
  } else {
    *reinterpret_cast<uint2*>(head + ln.off_a) = make_uint2(w[0], w[1]);
    *reinterpret_cast<uint2*>(head + ln.off_b) = make_uint2(w[2], w[3]);
  }
}

__device__ __forceinline__ float f2_sum(uint64_t v) {
  float a, b;
  f2_unpack(v, a, b);
  return a + b;
}

// Sum over the lanes that share a head.
__device__ __forceinline__ float head_sum(float x, int lanes) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (o < lanes) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// cos and sin of one token's pairs: the warp computes each once into its own
// shared-memory table, then every lane takes its pairs' values.
template <int PATH>
__device__ __forceinline__ void token_turns(const QkParams& p, int64_t token, int lane, float2* tab,
                                            const Lane<PATH>& ln, uint64_t (&c)[Lane<PATH>::M],
                                            uint64_t (&s)[Lane<PATH>::M]) {
  const int64_t pos = p.positions ? static_cast<int64_t>(p.positions[token]) : p.pos0 + token;
  __syncwarp();
  for (int i = lane; i < p.rot / 2; i += 32) {
    const uint64_t turn = p.step[i] * static_cast<uint64_t>(pos);
    float sn, cs;
    // signed: the nearest whole turn is taken off; 2^-31 half turns
    sincospif(static_cast<float>(static_cast<int32_t>(turn >> 32)) * 4.656612873077392578125e-10f, &sn, &cs);
    tab[i] = make_float2(cs * p.magnitude, sn * (p.magnitude * p.sign));
  }
  __syncwarp();
#pragma unroll
  for (int i = 0; i < Lane<PATH>::M; ++i) {
    const float2 t0 = ln.holds(2 * i) && ln.turns(2 * i) ? tab[ln.pair(2 * i)] : make_float2(1.f, 0.f);
    const float2 t1 = ln.holds(2 * i + 1) && ln.turns(2 * i + 1) ? tab[ln.pair(2 * i + 1)] : make_float2(1.f, 0.f);
    c[i] = f2_pack(t0.x, t1.x);
    s[i] = f2_pack(t0.y, t1.y);
  }
}

// A lane's pairs of a weight held in shared memory.
template <int PATH>
__device__ __forceinline__ void lane_weight(const float* w, const Lane<PATH>& ln, uint64_t (&wu)[Lane<PATH>::M],
                                            uint64_t (&wv)[Lane<PATH>::M]) {
  if constexpr (PATH == kScalar) {
    float f[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f[e] = ln.holds(e) ? w[ln.first(e)] : 0.f;
      f[4 + e] = ln.holds(e) ? w[ln.second(e)] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      wu[i] = f2_pack(f[2 * i], f[2 * i + 1]);
      wv[i] = f2_pack(f[4 + 2 * i], f[4 + 2 * i + 1]);
    }
  } else {
    constexpr int N = Lane<PATH>::N, M = Lane<PATH>::M;
    float f[2 * N];  // the lane's two vectors
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const float4 a = reinterpret_cast<const float4*>(w + (ln.live ? ln.off_a : 0))[i];
      const float4 b = reinterpret_cast<const float4*>(w + (ln.live ? ln.off_b : 0))[i];
      f[4 * i] = a.x, f[4 * i + 1] = a.y, f[4 * i + 2] = a.z, f[4 * i + 3] = a.w;
      f[N + 4 * i] = b.x, f[N + 4 * i + 1] = b.y, f[N + 4 * i + 2] = b.z, f[N + 4 * i + 3] = b.w;
    }
#pragma unroll
    for (int i = 0; i < M; ++i) {
      wu[i] = is_half(PATH) ? f2_pack(f[2 * i], f[2 * i + 1]) : f2_pack(f[4 * i], f[4 * i + 2]);
      wv[i] = is_half(PATH) ? f2_pack(f[N + 2 * i], f[N + 2 * i + 1]) : f2_pack(f[4 * i + 1], f[4 * i + 3]);
    }
  }
}

// One step of a warp: `per` heads of one token, the queries' steps first,
// then the keys'.
struct Steps {
  int per, q_steps, all;
  __device__ __forceinline__ explicit Steps(const QkParams& p)
      : per(32 / p.lanes), q_steps((p.nheads[0] + per - 1) / per), all(q_steps + (p.nheads[1] + per - 1) / per) {}
};

constexpr int kFwdSteps = 4, kBwdSteps = 4;  // steps in flight per warp

// CTAs per SM of the forward: the rotation by single elements, which has one
// step in flight, hides its loads behind other warps (262 us with four, 298 with
// three, of halves of 17 in 32768 tokens of 40 heads).
constexpr int fwd_ctas(int mode, int path) { return mode == kTurn && path == kScalar ? 4 : 3; }

template <int MODE, int PATH, bool WHOLE>
__global__ void __launch_bounds__(kWarps * 32, fwd_ctas(MODE, PATH))
    qk_rope_kernel(const __grid_constant__ QkParams p) {
  constexpr int M = Lane<PATH>::M;
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float2 tables[kWarps][kMaxPairs];
  __shared__ __align__(16) float weights[2][MODE == kNormTurn ? UPIPE_ROPE_MAX_D : 4];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if constexpr (MODE == kNormTurn) {
    for (int i = threadIdx.x; i < 2 * p.d; i += kWarps * 32) {
      const int t = i >= p.d;
      if (p.nheads[t]) weights[t][i - t * p.d] = __ldg(p.w[t] + i - t * p.d);
    }
    __syncthreads();
  }
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  const int64_t token = p.parts == 1 ? unit : unit / p.parts;
  if (token >= p.L) return;
  const int part = static_cast<int>(unit - token * p.parts);
  const Lane<PATH> ln(p, lane);
  const Steps st(p);
  const int mine = lane / p.lanes;
  const float inv_d = 1.f / p.d;
  const bf16 *const xq = p.x[0].p + token * p.x[0].row, *const xk = p.x[1].p + token * p.x[1].row;
  bf16 *const yq = p.y[0].p + token * p.y[0].row, *const yk = p.y[1].p + token * p.y[1].row;

  Pipe<PATH, 1, kFwdSteps> pipe(smem_u32(ring), warp, lane);
  auto head_at = [&](int step, bool& on) -> const bf16* {
    const int t = step >= st.q_steps;
    const int h = (step - (t ? st.q_steps : 0)) * st.per + mine;
    on = step < st.all && h < p.nheads[t] && ln.live;
    return on ? (t ? xk + h * p.x[1].head : xq + h * p.x[0].head) : p.x[0].p;
  };
  int ahead = part;
  bool on;
#pragma unroll
  for (int i = 0; i < Pipe<PATH, 1, kFwdSteps>::kAhead; ++i, ahead += p.parts) {
    const bf16* src[1] = {head_at(ahead, on)};
    pipe.start(src, on, ln);
  }
  uint64_t c[M], s[M];
  token_turns<PATH>(p, token, lane, tables[warp], ln, c, s);
  for (int step = part; step < st.all; step += p.parts, ahead += p.parts) {
    Raw<PATH> raw[1];
    const bf16* src[1] = {head_at(ahead, on)};
    pipe.turn(src, on, ln, raw);
    const int t = step >= st.q_steps;
    const int h = (step - (t ? st.q_steps : 0)) * st.per + mine;
    uint64_t u[M], v[M];
    raw[0].unpack(u, v);
    if constexpr (MODE == kNormTurn) {
      uint64_t q = 0;
#pragma unroll
      for (int e = 0; e < M; ++e) q = f2_fma(u[e], u[e], f2_fma(v[e], v[e], q));
      const float r = rsqrtf(head_sum(f2_sum(q), p.lanes) * inv_d + p.eps);
      const uint64_t rr = f2_pack(r, r);
      uint64_t wu[M], wv[M];
      lane_weight<PATH>(weights[t], ln, wu, wv);
#pragma unroll
      for (int e = 0; e < M; ++e) {
        u[e] = f2_mul(u[e], f2_mul(rr, wu[e]));
        v[e] = f2_mul(v[e], f2_mul(rr, wv[e]));
      }
    }
#pragma unroll
    for (int e = 0; e < M; ++e) turn_pairs<PATH, !WHOLE && MODE != kTurn>(ln, e, c[e], s[e], u[e], v[e]);
    if (h < p.nheads[t] && ln.live)
      store<PATH, !WHOLE && MODE == kTurn>(t ? yk + h * p.y[1].head : yq + h * p.y[0].head, ln, u, v, raw[0]);
  }
}

// Backward of the norm and rotation.  Each warp walks tokens (or shares of
// tokens) a grid apart, the queries of all of them first, then the keys, and
// keeps its lanes' shares of dw in registers; a CTA adds its warps' shares in
// a fixed order and writes one row per weight, which norm_sum_kernel adds up.
template <int PATH, bool WHOLE>
__global__ void __launch_bounds__(kWarps * 32, 2) qk_norm_rope_bwd_kernel(const __grid_constant__ QkParams p) {
  constexpr int M = Lane<PATH>::M;
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float2 tables[kWarps][kMaxPairs];
  __shared__ float shares[kWarps][UPIPE_ROPE_MAX_D];
  __shared__ __align__(16) float weights[UPIPE_ROPE_MAX_D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t units = p.L * p.parts;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kWarps;
  const Lane<PATH> ln(p, lane);
  const int per = 32 / p.lanes;
  const int mine = lane / p.lanes;
  const float inv_d = 1.f / p.d;
  for (int t = 0; t < 2; ++t) {
    const int nh = p.nheads[t];
    const int steps = (nh + per - 1) / per;
    __syncthreads();  // the last weight's shares have been added up
    for (int i = threadIdx.x; i < p.d && nh; i += kWarps * 32) weights[i] = __ldg(p.w[t] + i);
    __syncthreads();
    uint64_t wu[M], wv[M], gu[M], gv[M];
    lane_weight<PATH>(weights, ln, wu, wv);
#pragma unroll
    for (int e = 0; e < M; ++e) gu[e] = gv[e] = 0;

    struct At {
      int64_t unit, token;
      int step;
    };
    // the unit's first step, or the next unit that has one
    auto begin = [&](int64_t unit) {
      At a{unit, 0, 0};
      for (; a.unit < units; a.unit += stride) {
        a.token = p.parts == 1 ? a.unit : a.unit / p.parts;
        a.step = static_cast<int>(a.unit - a.token * p.parts);
        if (a.step < steps) break;
      }
      return a;
    };
    auto after = [&](At a) {
      a.step += p.parts;
      return a.step < steps ? a : begin(a.unit + stride);
    };
    using Loads = Pipe<PATH, 2, kBwdSteps>;
    Loads pipe(smem_u32(ring), warp, lane);
    auto heads_at = [&](const At& a, const bf16* (&src)[2]) {
      const int h = a.step * per + mine;
      const bool on = a.unit < units && h < nh && ln.live;
      src[0] = on ? p.x[t].p + a.token * p.x[t].row + h * p.x[t].head : p.x[t].p;
      src[1] = on ? p.dy[t].p + a.token * p.dy[t].row + h * p.dy[t].head : p.dy[t].p;
      return on;
    };
    At at = begin(nh ? static_cast<int64_t>(blockIdx.x) * kWarps + warp : units), ahead = at;
    if (at.unit < units) {
#pragma unroll
      for (int i = 0; i < Loads::kAhead; ++i) {
        const bf16* src[2];
        const bool on = heads_at(ahead, src);
        pipe.start(src, on, ln);
        if (ahead.unit < units) ahead = after(ahead);
      }
    }
    int64_t turned = -1;  // the token that c and s belong to
    uint64_t c[M], s[M];
    while (at.unit < units) {
      if (turned != at.token) {
        token_turns<PATH>(p, at.token, lane, tables[warp], ln, c, s);
        turned = at.token;
      }
      Raw<PATH> raw[2];
      const bf16* src[2];
      const bool on = heads_at(ahead, src);
      pipe.turn(src, on, ln, raw);
      if (ahead.unit < units) ahead = after(ahead);
      const int h = at.step * per + mine;
      uint64_t u[M], v[M], a[M], b[M];
      raw[0].unpack(u, v);
      raw[1].unpack(a, b);
      // sum x^2 and sum dn x in one reduction: neither needs the other
      uint64_t q = 0, dot = 0;
      uint64_t gx[M], gy[M];  // dz x, the terms of dw before the norm's factor
#pragma unroll
      for (int e = 0; e < M; ++e) {
        turn_pairs<PATH, !WHOLE>(ln, e, c[e], s[e], a[e], b[e]);  // dz: s holds -sin here
        q = f2_fma(u[e], u[e], f2_fma(v[e], v[e], q));
        gx[e] = f2_mul(a[e], u[e]);
        gy[e] = f2_mul(b[e], v[e]);
        dot = f2_fma(gx[e], wu[e], f2_fma(gy[e], wv[e], dot));
        a[e] = f2_mul(a[e], wu[e]);  // dn
        b[e] = f2_mul(b[e], wv[e]);
      }
      float qs = f2_sum(q), ds = f2_sum(dot);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
        if (o < p.lanes) {
          const float q2 = __shfl_xor_sync(0xffffffffu, qs, o), d2 = __shfl_xor_sync(0xffffffffu, ds, o);
          qs += q2;
          ds += d2;
        }
      // lanes without a head hold zeros, whose inverse root is infinite if eps is 0
      const float r = rsqrtf(qs * inv_d + (h < nh ? p.eps : 1.f));
      const float k = -(r * r) * (r * ds) * inv_d;  // dx = r dn - x r^3 mean(dn x)
      const uint64_t rr = f2_pack(r, r), kk = f2_pack(k, k);
#pragma unroll
      for (int e = 0; e < M; ++e) {
        gu[e] = f2_fma(gx[e], rr, gu[e]);
        gv[e] = f2_fma(gy[e], rr, gv[e]);
        a[e] = f2_fma(u[e], kk, f2_mul(a[e], rr));
        b[e] = f2_fma(v[e], kk, f2_mul(b[e], rr));
      }
      if (h < nh && ln.live) store<PATH, false>(p.y[t].p + at.token * p.y[t].row + h * p.y[t].head, ln, a, b, raw[0]);
      at = after(at);
    }
    pipe.drain();  // the next weight's pipe starts over in the same slots
    // The lanes that hold the same elements of different heads, then the warps.
#pragma unroll
    for (int i = 0; i < M; ++i) {
      for (int o = p.lanes; o < 32; o <<= 1) {
        gu[i] = f2_add(gu[i], __shfl_xor_sync(0xffffffffu, gu[i], o));
        gv[i] = f2_add(gv[i], __shfl_xor_sync(0xffffffffu, gv[i], o));
      }
      float a0, a1, b0, b1;
      f2_unpack(gu[i], a0, a1);
      f2_unpack(gv[i], b0, b1);
      if (mine == 0 && ln.holds(2 * i)) {
        shares[warp][ln.first(2 * i)] = a0;
        shares[warp][ln.second(2 * i)] = b0;
      }
      if (mine == 0 && ln.holds(2 * i + 1)) {
        shares[warp][ln.first(2 * i + 1)] = a1;
        shares[warp][ln.second(2 * i + 1)] = b1;
      }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < p.d; i += kWarps * 32) {
      float g = 0.f;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) g += shares[k][i];
      p.partial[(static_cast<int64_t>(blockIdx.x) * 2 + t) * p.d + i] = g;
    }
  }
}

// dw[t][i] = sum over the n rows of partial [n][2][d], in a fixed order:
// thread row j adds rows j, j + 32, ..., then the 32 shares are added.
__global__ void __launch_bounds__(1024) norm_sum_kernel(const float* __restrict__ partial, int n, int d, float* dwq,
                                                        float* dwk) {
  __shared__ float share[32][33];
  const int col = blockIdx.x * 32 + threadIdx.x;  // of 2 d
  float g = 0.f;
  if (col < 2 * d)
#pragma unroll 4
    for (int r = threadIdx.y; r < n; r += 32) g += partial[static_cast<int64_t>(r) * 2 * d + col];
  share[threadIdx.y][threadIdx.x] = g;
  __syncthreads();
  g = share[threadIdx.x][threadIdx.y];  // warp y adds column y
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) g += __shfl_xor_sync(0xffffffffu, g, o);
  const int out = blockIdx.x * 32 + threadIdx.y;
  if (threadIdx.x == 0 && out < 2 * d) {
    float* dw = out < d ? dwq : dwk;
    if (dw) dw[out < d ? out : out - d] = g;
  }
}

// ------------------------------------------------------------------- host

constexpr int kBwdCtas = 152 * 2;  // two resident per SM; the shares of dw are one row each

int lanes_of(int d, int path) {
  if (path == kScalar) return 32;
  int g = 1;
  while (g * 2 * vec_of(path) < d) g *= 2;
  return g;
}

bool rope_ok(const upipe_rope* r) {
  return r && r->d >= 8 && r->d <= UPIPE_ROPE_MAX_D && r->d % 8 == 0 && r->rot >= 0 && r->rot <= r->d &&
         r->rot % 2 == 0 && (r->layout == UPIPE_ROPE_HALF || r->layout == UPIPE_ROPE_INTERLEAVED) &&
         std::isfinite(r->magnitude);
}

// Shape, pointers and strides of one tensor [L, n, d]: 16-byte alignment of
// every head, and for a written tensor no element at two places.
bool rows_ok(const upipe_rows* t, int64_t L, int n, int d, bool written) {
  if (!t || !t->p || !aligned16(t->p)) return false;
  if (t->row < 0 || t->head < 0 || t->row % 8 != 0 || t->head % 8 != 0) return false;
  constexpr int64_t kMost = int64_t(1) << 60;  // keeps the products below from overflowing
  if ((L > 1 && t->row > kMost / L) || (n > 1 && t->head > kMost / n)) return false;
  if (!written) return true;
  const bool row_major = (n == 1 || t->head >= d) && (L == 1 || t->row >= (n - 1) * t->head + d);
  const bool head_major = (L == 1 || t->row >= d) && (n == 1 || t->head >= (L - 1) * t->row + d);
  return row_major || head_major;
}

// A weight or its gradient, which the kernels read and write by single floats.
bool weight_ok(const float* w) { return w && reinterpret_cast<uintptr_t>(w) % sizeof(float) == 0; }

bool call_ok(const upipe_rope* r, const upipe_qk_cfg* c) {
  return rope_ok(r) && c && c->L >= 1 && c->L <= 0x7fffffffLL && c->H >= 1 && c->H <= 65536 && c->Hkv >= 0 &&
         c->Hkv <= 65536 && c->pos0 > -(int64_t(1) << 62) && c->pos0 < (int64_t(1) << 62);
}

Rows to_rows(const upipe_rows* t) {
  return t ? Rows{reinterpret_cast<bf16*>(t->p), t->row, t->head} : Rows{nullptr, 0, 0};
}

QkParams base_params(const upipe_rope* r, const upipe_qk_cfg* c, const int32_t* positions, int path) {
  QkParams p;
  std::memset(&p, 0, sizeof(p));
  p.L = c->L;
  p.pos0 = c->pos0;
  p.nheads[0] = c->H;
  p.nheads[1] = c->Hkv;
  p.d = r->d;
  p.rot = r->rot;
  p.lanes = lanes_of(r->d, path);
  p.magnitude = static_cast<float>(r->magnitude);
  p.sign = 1.f;
  p.positions = positions;
  std::memcpy(p.step, r->step, sizeof(uint64_t) * (r->rot / 2));
  // A token's heads are split over more warps only while there are fewer
  // tokens than 16 warps on each of the 152 SMs, what hides the latency of
  // the loads; beyond, a share would only repeat the token's sines.
  const int per = 32 / p.lanes;
  const int steps = (c->H + per - 1) / per + (c->Hkv + per - 1) / per;
  const int64_t want = (152 * 16 + c->L - 1) / c->L;
  p.parts = static_cast<int>(want < steps ? want : steps);
  return p;
}

// The widest vectors that hold whole pairs (interleaved) or whose partners are
// vectors too (half), rotated and passing part alike.  The rotation of 32768
// tokens of 40 heads of 128: 102 us with 8 elements, 262 us of halves of 17,
// whose partners sit at odd elements; as many bytes in heads of 72 (58254
// tokens), 4 elements: 153 us.
int path_of(const upipe_rope* r) {
  const bool half = r->layout == UPIPE_ROPE_HALF;
  const int whole = half ? r->rot | r->d : r->d;
  if (whole % 16 == 0) return half ? kHalf8 : kInter8;
  if (whole % 8 == 0) return half ? kHalf4 : kInter4;
  return kScalar;
}

// Heads that turn whole have kernels of their own, which choose nothing per pair
// (single elements hold heads that turn in part only).  With the choice 32768
// tokens of 40 such heads take 105 us for 102 in the norm's forward and 184 for
// 180 in its backward, the rotation of 131072 tokens of 9 heads 128 for 113.
constexpr bool whole_kernel(int path) { return path != kScalar; }

template <int MODE, int PATH>
cudaError_t launch_fwd_path(const QkParams& p, cudaStream_t st) {
  const int64_t units = p.L * p.parts;
  const unsigned grid = static_cast<unsigned>((units + kWarps - 1) / kWarps);
  constexpr int kRing = kWarps * Pipe<PATH, 1, kFwdSteps>::kBytes;
  if (whole_kernel(PATH) && p.rot == p.d)
    qk_rope_kernel<MODE, PATH, whole_kernel(PATH)><<<grid, kWarps * 32, kRing, st>>>(p);
  else
    qk_rope_kernel<MODE, PATH, false><<<grid, kWarps * 32, kRing, st>>>(p);
  return cudaGetLastError();
}

template <int MODE>
cudaError_t launch_fwd(const QkParams& p, int path, cudaStream_t st) {
  switch (path) {
    case kHalf8: return launch_fwd_path<MODE, kHalf8>(p, st);
    case kInter8: return launch_fwd_path<MODE, kInter8>(p, st);
    case kHalf4: return launch_fwd_path<MODE, kHalf4>(p, st);
    case kInter4: return launch_fwd_path<MODE, kInter4>(p, st);
  }
  return launch_fwd_path<MODE, kScalar>(p, st);
}

int bwd_ctas(const QkParams& p) {
  const int64_t need = (p.L * p.parts + kWarps - 1) / kWarps;
  return static_cast<int>(need < kBwdCtas ? need : kBwdCtas);
}

template <int PATH>
cudaError_t launch_bwd_path(const QkParams& p, cudaStream_t st) {
  constexpr int kRing = kWarps * Pipe<PATH, 2, kBwdSteps>::kBytes;
  constexpr bool kWhole = whole_kernel(PATH);
  const auto kernel =
      kWhole && p.rot == p.d ? qk_norm_rope_bwd_kernel<PATH, kWhole> : qk_norm_rope_bwd_kernel<PATH, false>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRing);
  if (e != cudaSuccess) return e;
  kernel<<<bwd_ctas(p), kWarps * 32, kRing, st>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_bwd(const QkParams& p, int path, cudaStream_t st) {
  switch (path) {
    case kHalf8: return launch_bwd_path<kHalf8>(p, st);
    case kInter8: return launch_bwd_path<kInter8>(p, st);
    case kHalf4: return launch_bwd_path<kHalf4>(p, st);
    case kInter4: return launch_bwd_path<kInter4>(p, st);
  }
  return launch_bwd_path<kScalar>(p, st);
}

cudaError_t launch_norm_sum(const QkParams& p, float* dwq, float* dwk, cudaStream_t st) {
  norm_sum_kernel<<<(2 * p.d + 31) / 32, dim3(32, 32), 0, st>>>(p.partial, bwd_ctas(p), p.d, dwq, dwk);
  return cudaGetLastError();
}

}  // namespace
}  // namespace upipe

using namespace upipe;

extern "C" {

int upipe_rope_freqs(int rot, double theta, int scaling, double factor, double low, double high, int64_t orig_len,
                     double* freqs) {
  if (rot < 0 || rot > UPIPE_ROPE_MAX_D || rot % 2 != 0 || (rot && !freqs)) return UPIPE_ERR_INVALID_ARG;
  if (!(theta > 0.0) || !std::isfinite(theta)) return UPIPE_ERR_INVALID_ARG;
  if (scaling != UPIPE_ROPE_UNSCALED && scaling != UPIPE_ROPE_LINEAR && scaling != UPIPE_ROPE_BANDS)
    return UPIPE_ERR_INVALID_ARG;
  if (scaling != UPIPE_ROPE_UNSCALED && (!(factor > 0.0) || !std::isfinite(factor))) return UPIPE_ERR_INVALID_ARG;
  if (scaling == UPIPE_ROPE_BANDS &&
      (!std::isfinite(low) || !std::isfinite(high) || !(low < high) || orig_len < 1))
    return UPIPE_ERR_INVALID_ARG;
  for (int i = 0; i < rot / 2; ++i) {
    double f = std::pow(theta, -2.0 * i / rot);
    if (scaling == UPIPE_ROPE_LINEAR) f /= factor;
    if (scaling == UPIPE_ROPE_BANDS) {
      const double turns = static_cast<double>(orig_len) * f / 6.283185307179586477;
      double keep = (turns - low) / (high - low);
      keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
      f *= keep + (1.0 - keep) / factor;
    }
    freqs[i] = f;
  }
  return UPIPE_OK;
}

int upipe_rope_init(upipe_rope* r, int d, int rot, int layout, double magnitude, const double* freqs) {
  if (!r) return UPIPE_ERR_INVALID_ARG;
  upipe_rope v;
  std::memset(&v, 0, sizeof(v));
  v.d = d;
  v.rot = rot;
  v.layout = layout;
  v.magnitude = magnitude;
  if (!rope_ok(&v) || (rot && !freqs) || std::fabs(magnitude) > 1e30) return UPIPE_ERR_INVALID_ARG;
  for (int i = 0; i < rot / 2; ++i) {
    if (!std::isfinite(freqs[i])) return UPIPE_ERR_INVALID_ARG;
    const double turns = freqs[i] / 6.283185307179586477;
    // x - floor(x) of a tiny negative x rounds to 1.0, which is 0 turns
    const double frac = turns - std::floor(turns);
    v.step[i] = frac < 1.0 ? static_cast<uint64_t>(std::ldexp(frac, 64)) : 0;
  }
  *r = v;
  return UPIPE_OK;
}

int upipe_rope_apply(const upipe_rope* r, const upipe_qk_cfg* c, const upipe_rows* q, const upipe_rows* k,
                     const int32_t* positions, const upipe_rows* qo, const upipe_rows* ko, int transpose,
                     void* stream) {
  if (!call_ok(r, c)) return UPIPE_ERR_INVALID_ARG;
  if (!rows_ok(q, c->L, c->H, r->d, false) || !rows_ok(qo, c->L, c->H, r->d, true)) return UPIPE_ERR_INVALID_ARG;
  if (c->Hkv && (!rows_ok(k, c->L, c->Hkv, r->d, false) || !rows_ok(ko, c->L, c->Hkv, r->d, true)))
    return UPIPE_ERR_INVALID_ARG;
  if (transpose != 0 && transpose != 1) return UPIPE_ERR_INVALID_ARG;
  int* status = nullptr;
  if (int e = device_ready(&status)) return e;
  const int path = path_of(r);
  QkParams p = base_params(r, c, positions, path);
  p.x[0] = to_rows(q);
  p.y[0] = to_rows(qo);
  if (c->Hkv) {
    p.x[1] = to_rows(k);
    p.y[1] = to_rows(ko);
  }
  if (transpose) p.sign = -1.f;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  UPIPE_LAUNCH(UPIPE_KIND_QK_ROPE, launch_fwd<kTurn>(p, path, st));
  return UPIPE_OK;
}

int upipe_qk_norm_rope_fwd(const upipe_rope* r, const upipe_qk_cfg* c, const upipe_rows* q, const upipe_rows* k,
                           const float* wq, const float* wk, const int32_t* positions, const upipe_rows* qo,
                           const upipe_rows* ko, void* stream) {
  if (!call_ok(r, c) || !(c->eps >= 0.f) || !std::isfinite(c->eps)) return UPIPE_ERR_INVALID_ARG;
  if (!rows_ok(q, c->L, c->H, r->d, false) || !rows_ok(qo, c->L, c->H, r->d, true) || !weight_ok(wq))
    return UPIPE_ERR_INVALID_ARG;
  if (c->Hkv && (!rows_ok(k, c->L, c->Hkv, r->d, false) || !rows_ok(ko, c->L, c->Hkv, r->d, true) ||
                 !weight_ok(wk)))
    return UPIPE_ERR_INVALID_ARG;
  int* status = nullptr;
  if (int e = device_ready(&status)) return e;
  const int path = path_of(r);
  QkParams p = base_params(r, c, positions, path);
  p.eps = c->eps;
  p.x[0] = to_rows(q);
  p.y[0] = to_rows(qo);
  p.w[0] = wq;
  if (c->Hkv) {
    p.x[1] = to_rows(k);
    p.y[1] = to_rows(ko);
    p.w[1] = wk;
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  UPIPE_LAUNCH(UPIPE_KIND_QK_ROPE, launch_fwd<kNormTurn>(p, path, st));
  return UPIPE_OK;
}

size_t upipe_qk_norm_rope_workspace_bytes(const upipe_rope* r, const upipe_qk_cfg* c) {
  if (!call_ok(r, c)) return 0;
  const QkParams p = base_params(r, c, nullptr, path_of(r));
  return static_cast<size_t>(bwd_ctas(p)) * 2 * r->d * sizeof(float);
}

int upipe_qk_norm_rope_bwd(const upipe_rope* r, const upipe_qk_cfg* c, const upipe_rows* q, const upipe_rows* k,
                           const float* wq, const float* wk, const int32_t* positions, const upipe_rows* dqo,
                           const upipe_rows* dko, const upipe_rows* dq, const upipe_rows* dk, float* dwq, float* dwk,
                           void* ws, size_t ws_bytes, void* stream) {
  if (!call_ok(r, c) || !(c->eps >= 0.f) || !std::isfinite(c->eps)) return UPIPE_ERR_INVALID_ARG;
  if (!rows_ok(q, c->L, c->H, r->d, false) || !rows_ok(dqo, c->L, c->H, r->d, false) ||
      !rows_ok(dq, c->L, c->H, r->d, true) || !weight_ok(wq) || !weight_ok(dwq))
    return UPIPE_ERR_INVALID_ARG;
  if (c->Hkv && (!rows_ok(k, c->L, c->Hkv, r->d, false) || !rows_ok(dko, c->L, c->Hkv, r->d, false) ||
                 !rows_ok(dk, c->L, c->Hkv, r->d, true) || !weight_ok(wk) || !weight_ok(dwk)))
    return UPIPE_ERR_INVALID_ARG;
  if (!ws || !aligned16(ws)) return UPIPE_ERR_INVALID_ARG;
  if (ws_bytes < upipe_qk_norm_rope_workspace_bytes(r, c)) return UPIPE_ERR_WS_TOO_SMALL;
  int* status = nullptr;
  if (int e = device_ready(&status)) return e;
  const int path = path_of(r);
  QkParams p = base_params(r, c, positions, path);
  p.eps = c->eps;
  p.sign = -1.f;
  p.x[0] = to_rows(q);
  p.dy[0] = to_rows(dqo);
  p.y[0] = to_rows(dq);
  p.w[0] = wq;
  if (c->Hkv) {
    p.x[1] = to_rows(k);
    p.dy[1] = to_rows(dko);
    p.y[1] = to_rows(dk);
    p.w[1] = wk;
  }
  p.partial = static_cast<float*>(ws);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  UPIPE_LAUNCH(UPIPE_KIND_QK_ROPE, launch_bwd(p, path, st));
  UPIPE_LAUNCH(UPIPE_KIND_NORM_SUM, launch_norm_sum(p, dwq, c->Hkv ? dwk : nullptr, st));
  return UPIPE_OK;
}

}  // extern "C"
