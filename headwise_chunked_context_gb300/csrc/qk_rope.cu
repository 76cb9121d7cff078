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
// whose pairs do not fall on 16-byte vectors (d not a multiple of 16, or
// rot / 2 not a multiple of 8 in the half layout) take the same kernel with
// two-byte accesses, up to four pairs per lane and one head per warp.
#include <cmath>
#include <cstring>

#include "host.h"
#include "sm103_ptx.cuh"

namespace upipe {
namespace {

using bf16 = __nv_bfloat16;

constexpr int kMaxPairs = UPIPE_ROPE_MAX_D / 2;
constexpr int kWarps = 8;  // per CTA

enum Mode { kTurn = 0, kNormTurn = 1, kNormTurnBwd = 2 };
enum Path { kHalfVec = 0, kInterVec = 1, kScalar = 2 };

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
  int interleaved;  // pair layout (read by the scalar path; the vector paths have it as a parameter)
  float magnitude, eps, sign;  // sign: -1 turns by the transpose
  Rows x[2];   // the input (the norm's, or what is turned)
  Rows dy[2];  // backward: gradient of the output
  Rows y[2];   // the output, or dx
  const float* w[2];
  const int32_t* positions;
  float* partial;  // backward: [gridDim.x][2][d] shares of dw
  uint64_t step[kMaxPairs];
};

// Global reads that may alias this kernel's own later writes (in-place
// calls): plain loads, not the read-only path; every element is read and
// then written by one lane.
__device__ __forceinline__ uint4 ld_stream(const bf16* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// Which elements of a head a lane holds: N pairs (a[e], b[e]).
template <int PATH>
struct Lane {
  static constexpr int N = PATH == kScalar ? 4 : 8;
  int sub;    // lane within its head
  int off_a;  // vector paths: first element of the two 8-element vectors
  int off_b;
  bool live;
  int d, rot, interleaved;

  __device__ __forceinline__ Lane(const QkParams& p, int lane) {
    d = p.d;
    rot = p.rot;
    interleaved = p.interleaved;
    sub = lane % p.lanes;
    live = PATH == kScalar || sub * 16 < d;
    off_a = 16 * sub;
    off_b = off_a + 8;
    if (PATH == kHalfVec && sub * 16 < rot) {
      off_a = 8 * sub;
      off_b = rot / 2 + 8 * sub;
    }
  }
  __device__ __forceinline__ int pair(int e) const { return PATH == kScalar ? sub + 32 * e : 8 * sub + e; }
  __device__ __forceinline__ bool holds(int e) const { return PATH == kScalar ? 2 * pair(e) < d : live; }
  __device__ __forceinline__ bool turns(int e) const { return 2 * pair(e) < rot; }
  __device__ __forceinline__ int first(int e) const {
    if (PATH == kHalfVec) return off_a + e;
    if (PATH == kInterVec) return 2 * pair(e);
    return turns(e) && !interleaved ? pair(e) : 2 * pair(e);
  }
  __device__ __forceinline__ int second(int e) const {
    if (PATH == kHalfVec) return off_b + e;
    if (PATH == kInterVec) return 2 * pair(e) + 1;
    return turns(e) && !interleaved ? pair(e) + rot / 2 : 2 * pair(e) + 1;
  }
};

// What a lane has in flight of one head: its raw bits.
template <int PATH>
struct Raw {
  uint4 a, b;  // scalar path: the pairs' halves in the words of a
  __device__ __forceinline__ void load(const bf16* head, const Lane<PATH>& ln) {
    if constexpr (PATH == kScalar) {
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        w[e] = 0u;
        if (ln.holds(e)) {
          const uint16_t* h = reinterpret_cast<const uint16_t*>(head);
          const uint32_t lo = *reinterpret_cast<const volatile uint16_t*>(h + ln.first(e));
          const uint32_t hi = *reinterpret_cast<const volatile uint16_t*>(h + ln.second(e));
          w[e] = lo | (hi << 16);
        }
      }
      a = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      a = ld_stream(head + ln.off_a);
      b = ld_stream(head + ln.off_b);
    }
  }
  __device__ __forceinline__ void zero() { a = b = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void unpack(float (&u)[Lane<PATH>::N], float (&v)[Lane<PATH>::N]) const {
    const uint32_t wa[4] = {a.x, a.y, a.z, a.w};
    if constexpr (PATH == kScalar) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        u[e] = bf16_lo(wa[e]);
        v[e] = bf16_hi(wa[e]);
      }
    } else {
      const uint32_t wb[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (PATH == kHalfVec) {
          u[2 * e] = bf16_lo(wa[e]);
          u[2 * e + 1] = bf16_hi(wa[e]);
          v[2 * e] = bf16_lo(wb[e]);
          v[2 * e + 1] = bf16_hi(wb[e]);
        } else {
          u[e] = bf16_lo(wa[e]);
          v[e] = bf16_hi(wa[e]);
          u[4 + e] = bf16_lo(wb[e]);
          v[4 + e] = bf16_hi(wb[e]);
        }
      }
    }
  }
};

// Rounds the lane's pairs to bf16, the only rounding of the pass, and stores them.
template <int PATH>
__device__ __forceinline__ void store(bf16* head, const Lane<PATH>& ln, const float (&u)[Lane<PATH>::N],
                                      const float (&v)[Lane<PATH>::N]) {
  if constexpr (PATH == kScalar) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (ln.holds(e)) {
        head[ln.first(e)] = __float2bfloat16_rn(u[e]);
        head[ln.second(e)] = __float2bfloat16_rn(v[e]);
      }
  } else if constexpr (PATH == kHalfVec) {
    st_global_v4(head + ln.off_a, pack_bf16x2(u[0], u[1]), pack_bf16x2(u[2], u[3]), pack_bf16x2(u[4], u[5]),
                 pack_bf16x2(u[6], u[7]));
    st_global_v4(head + ln.off_b, pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                 pack_bf16x2(v[6], v[7]));
  } else {
    st_global_v4(head + ln.off_a, pack_bf16x2(u[0], v[0]), pack_bf16x2(u[1], v[1]), pack_bf16x2(u[2], v[2]),
                 pack_bf16x2(u[3], v[3]));
    st_global_v4(head + ln.off_b, pack_bf16x2(u[4], v[4]), pack_bf16x2(u[5], v[5]), pack_bf16x2(u[6], v[6]),
                 pack_bf16x2(u[7], v[7]));
  }
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
                                            const Lane<PATH>& ln, float (&c)[Lane<PATH>::N],
                                            float (&s)[Lane<PATH>::N]) {
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
  for (int e = 0; e < Lane<PATH>::N; ++e) {
    const float2 t = ln.holds(e) && ln.turns(e) ? tab[ln.pair(e)] : make_float2(1.f, 0.f);
    c[e] = t.x;
    s[e] = t.y;
  }
}

template <int PATH>
__device__ __forceinline__ void load_weight(const float* w, const Lane<PATH>& ln, float (&wu)[Lane<PATH>::N],
                                            float (&wv)[Lane<PATH>::N]) {
#pragma unroll
  for (int e = 0; e < Lane<PATH>::N; ++e) {
    wu[e] = ln.holds(e) ? __ldg(w + ln.first(e)) : 0.f;
    wv[e] = ln.holds(e) ? __ldg(w + ln.second(e)) : 0.f;
  }
}

template <int MODE, int PATH>
__global__ void __launch_bounds__(kWarps * 32) qk_rope_kernel(const __grid_constant__ QkParams p) {
  constexpr int N = Lane<PATH>::N;
  constexpr int U = 4;  // heads in flight per lane
  __shared__ float2 tables[kWarps][kMaxPairs];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  const int64_t token = unit / p.parts;
  if (token >= p.L) return;
  const int part = static_cast<int>(unit % p.parts);
  const Lane<PATH> ln(p, lane);
  const int per = 32 / p.lanes;  // heads per step of the warp
  const int mine = lane / p.lanes;
  const float inv_d = 1.f / p.d;
  float c[N], s[N];
  token_turns<PATH>(p, token, lane, tables[warp], ln, c, s);
  for (int t = 0; t < 2; ++t) {
    const int nh = p.nheads[t];
    const bf16* x = p.x[t].p + token * p.x[t].row;
    bf16* y = p.y[t].p + token * p.y[t].row;
    float wu[N], wv[N];
    if (MODE == kNormTurn && nh) load_weight<PATH>(p.w[t], ln, wu, wv);
    for (int h0 = part * per; h0 < nh; h0 += p.parts * per * U) {
      Raw<PATH> raw[U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int h = h0 + i * p.parts * per + mine;
        raw[i].zero();
        if (h < nh && ln.live) raw[i].load(x + h * p.x[t].head, ln);
      }
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int h = h0 + i * p.parts * per + mine;
        float u[N], v[N];
        raw[i].unpack(u, v);
        if constexpr (MODE == kNormTurn) {
          float q = 0.f;
#pragma unroll
          for (int e = 0; e < N; ++e) q = fmaf(u[e], u[e], fmaf(v[e], v[e], q));
          const float r = rsqrtf(head_sum(q, p.lanes) * inv_d + p.eps);
#pragma unroll
          for (int e = 0; e < N; ++e) {
            u[e] *= r * wu[e];
            v[e] *= r * wv[e];
          }
        }
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const float a = u[e] * c[e] - v[e] * s[e];
          v[e] = u[e] * s[e] + v[e] * c[e];
          u[e] = a;
        }
        if (h < nh && ln.live) store<PATH>(y + h * p.y[t].head, ln, u, v);
      }
    }
  }
}

// Backward of the norm and rotation.  Each warp walks tokens (or shares of
// tokens) a grid apart, the queries first, then the keys, and keeps its
// lanes' shares of dw in registers; a CTA adds its warps' shares in a fixed
// order and writes one row per weight, which norm_sum_kernel adds up.
template <int PATH>
__global__ void __launch_bounds__(kWarps * 32) qk_norm_rope_bwd_kernel(const __grid_constant__ QkParams p) {
  constexpr int N = Lane<PATH>::N;
  constexpr int U = 2;  // heads in flight per lane
  __shared__ float2 tables[kWarps][kMaxPairs];
  __shared__ float shares[kWarps][UPIPE_ROPE_MAX_D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t units = p.L * p.parts;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kWarps;
  const Lane<PATH> ln(p, lane);
  const int per = 32 / p.lanes;
  const int mine = lane / p.lanes;
  const float inv_d = 1.f / p.d;
  for (int t = 0; t < 2; ++t) {
    const int nh = p.nheads[t];
    float wu[N], wv[N], gu[N], gv[N];
    if (nh) load_weight<PATH>(p.w[t], ln, wu, wv);
#pragma unroll
    for (int e = 0; e < N; ++e) gu[e] = gv[e] = 0.f;
    for (int64_t unit = nh ? static_cast<int64_t>(blockIdx.x) * kWarps + warp : units; unit < units; unit += stride) {
      const int64_t token = unit / p.parts;
      const int part = static_cast<int>(unit % p.parts);
      float c[N], s[N];
      token_turns<PATH>(p, token, lane, tables[warp], ln, c, s);
      const bf16* x = p.x[t].p + token * p.x[t].row;
      const bf16* dy = p.dy[t].p + token * p.dy[t].row;
      bf16* dx = p.y[t].p + token * p.y[t].row;
      for (int h0 = part * per; h0 < nh; h0 += p.parts * per * U) {
        Raw<PATH> rx[U], ry[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const int h = h0 + i * p.parts * per + mine;
          rx[i].zero();
          ry[i].zero();
          if (h < nh && ln.live) {
            rx[i].load(x + h * p.x[t].head, ln);
            ry[i].load(dy + h * p.dy[t].head, ln);
          }
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const int h = h0 + i * p.parts * per + mine;
          float u[N], v[N], a[N], b[N];
          rx[i].unpack(u, v);
          ry[i].unpack(a, b);
          float q = 0.f;
#pragma unroll
          for (int e = 0; e < N; ++e) q = fmaf(u[e], u[e], fmaf(v[e], v[e], q));
          const float r = rsqrtf(head_sum(q, p.lanes) * inv_d + p.eps);
          float m = 0.f;
#pragma unroll
          for (int e = 0; e < N; ++e) {
            u[e] *= r;  // n
            v[e] *= r;
            const float za = a[e] * c[e] - b[e] * s[e];  // dz: s holds -sin here
            const float zb = a[e] * s[e] + b[e] * c[e];
            gu[e] = fmaf(za, u[e], gu[e]);
            gv[e] = fmaf(zb, v[e], gv[e]);
            a[e] = za * wu[e];  // dn
            b[e] = zb * wv[e];
            m = fmaf(a[e], u[e], fmaf(b[e], v[e], m));
          }
          m = head_sum(m, p.lanes) * inv_d;
#pragma unroll
          for (int e = 0; e < N; ++e) {
            a[e] = r * (a[e] - u[e] * m);
            b[e] = r * (b[e] - v[e] * m);
          }
          if (h < nh && ln.live) store<PATH>(dx + h * p.y[t].head, ln, a, b);
        }
      }
    }
    // The lanes that hold the same elements of different heads, then the warps.
#pragma unroll
    for (int e = 0; e < N; ++e) {
      for (int o = p.lanes; o < 32; o <<= 1) {
        gu[e] += __shfl_xor_sync(0xffffffffu, gu[e], o);
        gv[e] += __shfl_xor_sync(0xffffffffu, gv[e], o);
      }
      if (mine == 0 && ln.holds(e)) {
        shares[warp][ln.first(e)] = gu[e];
        shares[warp][ln.second(e)] = gv[e];
      }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < p.d; i += kWarps * 32) {
      float g = 0.f;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) g += shares[k][i];
      p.partial[(static_cast<int64_t>(blockIdx.x) * 2 + t) * p.d + i] = g;
    }
    __syncthreads();
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

constexpr int kBwdCtas = 152 * 3;  // three resident per SM; the shares of dw are one row each

int lanes_of(int d) {
  int g = 1;
  while (g * 16 < d) g *= 2;
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
  p.lanes = path == kScalar ? 32 : lanes_of(r->d);
  p.interleaved = r->layout == UPIPE_ROPE_INTERLEAVED;
  p.magnitude = static_cast<float>(r->magnitude);
  p.sign = 1.f;
  p.positions = positions;
  std::memcpy(p.step, r->step, sizeof(uint64_t) * (r->rot / 2));
  // A token's heads are split over more warps only while there are fewer
  // tokens than 16 warps on each of the 152 SMs, what hides the latency of
  // the loads; beyond, a share would only repeat the token's sines.
  const int per = 32 / p.lanes;
  const int steps = (c->H + per - 1) / per;
  const int64_t want = (152 * 16 + c->L - 1) / c->L;
  p.parts = static_cast<int>(want < steps ? want : steps);
  return p;
}

// The vector paths need 16-byte vectors that hold both members of each pair.
int path_of(const upipe_rope* r) {
  if (r->d % 16 != 0) return kScalar;
  if (r->layout == UPIPE_ROPE_INTERLEAVED) return kInterVec;
  return r->rot % 16 == 0 ? kHalfVec : kScalar;
}

template <int MODE>
cudaError_t launch_fwd(const QkParams& p, int path, cudaStream_t st) {
  const int64_t units = p.L * p.parts;
  const unsigned grid = static_cast<unsigned>((units + kWarps - 1) / kWarps);
  if (path == kHalfVec)
    qk_rope_kernel<MODE, kHalfVec><<<grid, kWarps * 32, 0, st>>>(p);
  else if (path == kInterVec)
    qk_rope_kernel<MODE, kInterVec><<<grid, kWarps * 32, 0, st>>>(p);
  else
    qk_rope_kernel<MODE, kScalar><<<grid, kWarps * 32, 0, st>>>(p);
  return cudaGetLastError();
}

int bwd_ctas(const QkParams& p) {
  const int64_t need = (p.L * p.parts + kWarps - 1) / kWarps;
  return static_cast<int>(need < kBwdCtas ? need : kBwdCtas);
}

cudaError_t launch_bwd(const QkParams& p, int path, cudaStream_t st) {
  const unsigned grid = static_cast<unsigned>(bwd_ctas(p));
  if (path == kHalfVec)
    qk_norm_rope_bwd_kernel<kHalfVec><<<grid, kWarps * 32, 0, st>>>(p);
  else if (path == kInterVec)
    qk_norm_rope_bwd_kernel<kInterVec><<<grid, kWarps * 32, 0, st>>>(p);
  else
    qk_norm_rope_bwd_kernel<kScalar><<<grid, kWarps * 32, 0, st>>>(p);
  return cudaGetLastError();
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
  if (!rows_ok(q, c->L, c->H, r->d, false) || !rows_ok(qo, c->L, c->H, r->d, true) || !wq || !aligned16(wq))
    return UPIPE_ERR_INVALID_ARG;
  if (c->Hkv && (!rows_ok(k, c->L, c->Hkv, r->d, false) || !rows_ok(ko, c->L, c->Hkv, r->d, true) || !wk ||
                 !aligned16(wk)))
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
      !rows_ok(dq, c->L, c->H, r->d, true) || !wq || !aligned16(wq) || !dwq || !aligned16(dwq))
    return UPIPE_ERR_INVALID_ARG;
  if (c->Hkv && (!rows_ok(k, c->L, c->Hkv, r->d, false) || !rows_ok(dko, c->L, c->Hkv, r->d, false) ||
                 !rows_ok(dk, c->L, c->Hkv, r->d, true) || !wk || !aligned16(wk) || !dwk || !aligned16(dwk)))
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
