// Random bits of dropout masks: Philox 4x32 with ten rounds (Salmon, Moraes,
// Dror, Shaw, "Parallel random numbers: as easy as 1, 2, 3", SC 2011), a
// function of a counter and a key.  Nothing is stored: element e of a tensor
// takes word e % 4 of the block whose counter is (e / 4, call) under the key
// `seed`, whichever kernel asks, and however it splits the tensor.
#pragma once

#include <cstdint>

#include "sm103_ptx.cuh"
#include "upipe.h"

namespace upipe {

// A mask as the kernels take it (upipe_dropout after its checks).
struct Drop {
  uint32_t key[20];  // of the ten rounds, which read them as operands out of constant memory
  uint64_t call, first;
  const uint64_t* step;  // device: added to call, or null
  uint32_t cut;          // kept iff the element's word >= cut: p = cut 2^-32
  float factor;          // 1 / (1 - p)
};

// False: p or first out of range.  cut is p in whole steps of 2^-32, and the
// factor is that of the steps, so that the mean is kept exactly.
inline bool drop_of(const upipe_dropout* u, Drop* d) {
  if (!(u->p >= 0.0) || !(u->p < 1.0) || u->first % 8 != 0 || u->first >> 63) return false;
  const double cut = static_cast<double>(static_cast<uint64_t>(u->p * 4294967296.0 + 0.5));
  if (cut > 4294967295.0) return false;
  if (reinterpret_cast<uintptr_t>(u->step) % sizeof(uint64_t) != 0) return false;
  for (uint32_t r = 0; r < 10; ++r) {
    d->key[2 * r] = static_cast<uint32_t>(u->seed) + r * 0x9E3779B9u;
    d->key[2 * r + 1] = static_cast<uint32_t>(u->seed >> 32) + r * 0xBB67AE85u;
  }
  d->call = u->call;
  d->first = u->first;
  d->step = u->step;
  d->cut = static_cast<uint32_t>(cut);
  d->factor = static_cast<float>(4294967296.0 / (4294967296.0 - cut));
  return true;
}

#ifdef __CUDACC__
// The call that a mask is drawn for.
__device__ __forceinline__ uint64_t drop_call(const Drop& d) { return d.call + (d.step ? *d.step : 0); }

// A mask being drawn.  With the call fixed, half of the first two rounds is the
// same for all blocks whose counters agree in their upper 32 bits (2^34
// elements): it is kept from one vector to the next.
class Mask {
 public:
  __device__ __forceinline__ Mask(const Drop& d, uint64_t call) : d_(d), first_(d.first >> 2) {
    c3_ = static_cast<uint32_t>(call >> 32);
    b_ = static_cast<uint64_t>(static_cast<uint32_t>(call)) * kB;
    enter(static_cast<uint32_t>(first_ >> 32));
  }
  // v[0..7], elements e .. e + 7 of the tensor (e a multiple of 8), behind the
  // mask.  A dropped element is 0 whatever it held.  One rounding per kept
  // element, and no contraction with a sum that follows: the sum of a mask with
  // p = 0 is the plain sum.
  __device__ __forceinline__ void apply(uint64_t e, float (&v)[8]) {
    float zero[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    each<false>(e, v, zero);
  }
  // r += v behind the mask: a kept element is added, a dropped one leaves r as it is.
  __device__ __forceinline__ void add(uint64_t e, float (&v)[8], float (&r)[8]) { each<true>(e, v, r); }

 private:
  template <bool ADD>
  __device__ __forceinline__ void each(uint64_t e, float (&v)[8], float (&r)[8]) {
    const uint64_t block = first_ + (e >> 2);  // even: the next one has the same upper half
    if (static_cast<uint32_t>(block >> 32) != upper_) enter(static_cast<uint32_t>(block >> 32));
    const uint64_t f = f2_pack(d_.factor, d_.factor);
#pragma unroll
    for (int i = 0; i < 4; ++i) f2_unpack(f2_mul(f2_pack(v[2 * i], v[2 * i + 1]), f), v[2 * i], v[2 * i + 1]);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t w[4];
      draw(static_cast<uint32_t>(block) + h, w);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float& a = v[4 * h + i];
        if (ADD) {
          if (w[i] >= d_.cut) r[4 * h + i] = __fadd_rn(r[4 * h + i], a);
        } else {
          a = w[i] >= d_.cut ? a : 0.f;
        }
      }
    }
  }

  static constexpr uint32_t kA = 0xD2511F53u, kB = 0xCD9E8D57u;
  const Drop& d_;
  uint64_t first_, a_, b_;  // a_: product of the second round, b_: of the first
  uint32_t c3_, upper_;

  __device__ __forceinline__ void enter(uint32_t upper) {
    upper_ = upper;
    a_ = static_cast<uint64_t>(static_cast<uint32_t>(b_ >> 32) ^ upper ^ d_.key[0]) * kA;
  }
  // Words of the counter (lower, upper_, call).
  __device__ __forceinline__ void draw(uint32_t lower, uint32_t (&w)[4]) const {
    uint64_t a = static_cast<uint64_t>(lower) * kA;  // round 1
    uint32_t c2 = static_cast<uint32_t>(a >> 32) ^ c3_ ^ d_.key[1], c3 = static_cast<uint32_t>(a);
    uint64_t b = static_cast<uint64_t>(c2) * kB;     // round 2
    uint32_t c0 = static_cast<uint32_t>(b >> 32) ^ static_cast<uint32_t>(b_) ^ d_.key[2];
    uint32_t c1 = static_cast<uint32_t>(b);
    c2 = static_cast<uint32_t>(a_ >> 32) ^ c3 ^ d_.key[3];
    c3 = static_cast<uint32_t>(a_);
#pragma unroll
    for (int r = 2; r < 10; ++r) {
      a = static_cast<uint64_t>(c0) * kA;
      b = static_cast<uint64_t>(c2) * kB;
      c0 = static_cast<uint32_t>(b >> 32) ^ c1 ^ d_.key[2 * r];
      c1 = static_cast<uint32_t>(b);
      c2 = static_cast<uint32_t>(a >> 32) ^ c3 ^ d_.key[2 * r + 1];
      c3 = static_cast<uint32_t>(a);
    }
    w[0] = c0, w[1] = c1, w[2] = c2, w[3] = c3;
  }
};
#endif

}  // namespace upipe
