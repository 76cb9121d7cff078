// Causal attention with a sliding window and sink tokens, forward and
// backward, tcgen05 + TMEM, and its C entry points.
//
// Query i sees key j iff j <= i and (i - j < W or j < S): the last W keys and
// the first S.  With these keys, per query head h and KV head h / g:
//   s_ij = q_i k_j / sqrt(d),  LSE_i = ln sum_j exp(s_ij),  P = exp(s - LSE),
//   O = P V;  dP = dO V^T,  Delta_i = sum_c dO_ic O_ic,  dS = P (dP - Delta),
//   dQ = dS K / sqrt(d),  dK = dS^T Q / sqrt(d),  dV = P^T dO.
// Every query sees itself, so no row is empty and the running maximum is
// finite from a tile's first block (the diagonal one) on.
//
// Tiles are 128 queries by 128 keys.  A query tile walks the blocks that hold
// the windows of its queries, the diagonal one first, then the sink blocks
// before them; a key tile walks the query tiles up to the last one whose
// window reaches it, all later ones if it holds a sink.  Blocks that every
// query of a tile sees whole take no mask.
//
// Scores, statistics and every sum are fp32.  P and dS are rounded to bf16
// where they enter a product (the tensor core's operand type); O, dQ, dK and
// dV are rounded to bf16 once, from TMEM.
#include <cmath>
#include <cstring>
#include <initializer_list>

#include "host.h"
#include "sm103_ptx.cuh"

namespace upipe {
namespace {

constexpr uint32_t kTmemCols = 512;

struct WinParams {
  int L, H, Hkv, g;   // q [L, H, 128], k and v [L, Hkv, 128]; g = H / Hkv
  int window, sinks;  // at most L each
  __nv_bfloat16* o;   // [L, H, 128]
  float* lse;         // [H, L]
  // Backward: what a query adds to its scores and to its dP, -LSE sqrt(d) and
  // -Delta, each as three bf16 whose sum is the fp32 value (a0 a1 a2 b0 b1 b2
  // and ten zeros): a K = 16 row that one more tcgen05.mma step multiplies by
  // ones.  [H, L, 16].
  const __nv_bfloat16* rec;
  const __nv_bfloat16* dout;  // [L, H, 128]
  __nv_bfloat16* dq;
  __nv_bfloat16* dk;
  __nv_bfloat16* dv;
  // Sink key tiles and the query tiles past their windows (see SinkPlan).
  int sink_tiles, near_tiles, far_chunk, far_slots, sink_rows, shared_keys;
  float* sink_part;
  // Tiles (dQ) and key items (dK/dV) handed out beyond each CTA's first.
  int* next_tile;
  int* next_item;
  int key_items;
  float scale;       // 1/sqrt(d)
  float scale_log2;  // log2(e)/sqrt(d)
  bool sectors;      // bf16 outputs start on 32-byte boundaries
  int* status;
  uint64_t limit_ns;
};

// Bits 0 .. n - 1 of a word (none below 1, all from 32 on).
__device__ __forceinline__ uint32_t bits_below(int n) {
  return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u;
}

// Which of the 32 keys from k0 on query i sees, bit c for key k0 + c.  A bit
// test per score costs the masked blocks half of what comparisons of each
// key's position would (0.55 us of a 1.4 us block).
__device__ __forceinline__ uint32_t seen_keys(int i, int k0, const WinParams& p) {
  return bits_below(i - k0 + 1) & ~(bits_below(i - p.window - k0 + 1) & ~bits_below(p.sinks - k0));
}

// Whether some query of tile qb does not see some key of block kb (of a pair
// that is walked at all).
__device__ __forceinline__ bool hides(int qb, int kb, const WinParams& p) {
  return qb == kb || (kb * 128 <= qb * 128 + 127 - p.window && kb * 128 + 127 >= p.sinks);
}

// The 128-key blocks that query tile qb walks.
struct QuerySpan {
  int qb, n_win, n_sink;
  __device__ __forceinline__ QuerySpan(int qb_, const WinParams& p) : qb(qb_) {
    const int lowest = qb * 128 - p.window + 1;  // first key in the first query's window
    const int first = lowest > 0 ? lowest >> 7 : 0;
    n_win = qb - first + 1;
    const int sink_blocks = (p.sinks >> 7) + ((p.sinks & 127) != 0);
    n_sink = sink_blocks < first ? sink_blocks : first;
  }
  __device__ __forceinline__ int count() const { return n_win + n_sink; }
  __device__ __forceinline__ int block(int j) const { return j < n_win ? qb - j : j - n_win; }
  __device__ __forceinline__ bool masked(int kb, const WinParams& p) const { return hides(qb, kb, p); }
};

// One CTA's share of dK and dV: key tile kb of a KV head and the query tiles
// [q0, q1) of the heads that read it.
struct KeyItem {
  int kv, kb, q0, q1;
  int slot;  // of sink_part; -1: the CTA alone sums its keys
  __device__ __forceinline__ KeyItem(int item, const WinParams& p) {
    const int tiles = ((p.L - 1) >> 7) + 1;
    kv = item % p.Hkv;
    item /= p.Hkv;
    const int far_items = p.sink_tiles * p.far_slots;
    if (item < far_items) {  // the longest first
      kb = item % p.sink_tiles;
      slot = 1 + item / p.sink_tiles;
      q0 = kb + p.near_tiles + (slot - 1) * p.far_chunk;
      q1 = q0 + p.far_chunk;
    } else {
      kb = item - far_items;
      slot = kb < p.sink_tiles ? 0 : -1;
      q0 = kb;
      // unless other CTAs have them, a sink tile's later queries are its own
      q1 = slot < 0 && kb * 128 < p.sinks ? tiles : kb + p.near_tiles;
    }
    q1 = q1 < tiles ? q1 : tiles;
  }
  __device__ __forceinline__ int tiles() const { return q1 - q0; }
  __device__ __forceinline__ bool empty() const { return q1 <= q0; }
  // fp32 share [2][sink_rows][128] of dK and dV
  __device__ __forceinline__ float* part(const WinParams& p) const {
    const int64_t at = (static_cast<int64_t>(kv) * p.sink_tiles + kb) * (p.far_slots + 1) + slot;
    return p.sink_part + at * 2 * p.sink_rows * kHeadDim;
  }
};

// An item's (query head, query tile) pairs in the order of its sums: the heads
// that read the KV head ascending, each one's tiles ascending.
struct KeyWalk {
  int h, qt, last_h, q0, q1;
  __device__ __forceinline__ KeyWalk(const KeyItem& item, const WinParams& p)
      : h(item.kv * p.g), qt(item.q0), last_h(h + p.g - 1), q0(item.q0), q1(item.q1) {}
  __device__ __forceinline__ bool next() {
    if (++qt < q1) return true;
    qt = q0;
    return ++h <= last_h;
  }
};

// Last query that sees key j.
__device__ __forceinline__ int last_query(int j, const WinParams& p) {
  const int64_t q = static_cast<int64_t>(j) + p.window - 1;
  return j < p.sinks || q > 0x7ffffffe ? 0x7ffffffe : static_cast<int>(q);
}

// Scores of one query row against keys k0 .. k0 + 127: -inf where hidden.
__device__ __forceinline__ void hide_row(float (&x)[128], int qpos, int k0, const WinParams& p) {
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const uint32_t seen = seen_keys(qpos, k0 + 32 * w, p);
#pragma unroll
    for (int c = 0; c < 32; ++c)
      if (!(seen >> c & 1u)) x[32 * w + c] = -INFINITY;
  }
}

__device__ __forceinline__ void st_global_v8(void* p, const uint32_t* v) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// 32 fp32 accumulators of one row, scaled and rounded to bf16.  A warp's rows
// lie apart, so that a store takes a sector of each: whole sectors (32-byte
// aligned outputs, as a rule) or halves.  131072 x 8 heads, window 1: 196 us
// with halves, 172 with whole ones; window 1024, backward: 1565 and 1526.
__device__ __forceinline__ void store32_bf16(__nv_bfloat16* out, const uint32_t (&a)[32], float scale, bool sectors) {
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    uint32_t h[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
      h[e] = pack_bf16x2(__uint_as_float(a[16 * q + 2 * e]) * scale, __uint_as_float(a[16 * q + 2 * e + 1]) * scale);
    if (sectors) {
      st_global_v8(out + q * 16, h);
    } else {
      st_global_v4(out + q * 16, h[0], h[1], h[2], h[3]);
      st_global_v4(out + q * 16 + 8, h[4], h[5], h[6], h[7]);
    }
  }
}

// Products issued by a whole converged warp, from which one lane is elected
// inside the instruction sequence: addresses and descriptors then stay in
// uniform registers.  Eight products of 128 x 128 x 16 from an idle pipe are
// seen complete after 705 cycles, 841 when a thread of its own issues them
// behind a branch (512 of them are the products).  The election is the same
// every time, so commits cover the same thread's products.
// Between products these warps wait suspended: probes in a loop take issue
// slots from the row warps of the same sub-partition, whose serial time per
// block is what every role waits for (with such loops the backward of 32768 x 32
// heads, window 4096, took 7 % longer, the forward 2 %).
__device__ __forceinline__ void umma_one(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void umma_ts_one(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void commit_one(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
      : "memory");
}

// ================================================================= forward
//
// One CTA per SM walks (head, query tile) pairs.  Warp 4 streams each tile's Q
// and the K/V blocks of 128 keys through 3-stage TMA rings; the softmax warps
// copy Q into TMEM, the next tile's as soon as this one's last scores have
// been formed.  Warp 5 issues S = Q K^T (Q from TMEM) into the TMEM score
// buffer, free again as soon as it has been read, warp 6 O += P V (P from one
// of two TMEM buffers).  Warps 0-3 own one query row per thread, so that row
// maximum and sum are thread-local; O is rescaled in TMEM only when a row's
// maximum grows by more than 2^8, which bounds every exponent.
//
// Measured: 32768 tokens, 32 heads, window 4096: 1.37 ms from rest, 1.49 call
// upon call, when the power limit holds the SMs at 1830 MHz.  From rest that is
// 820 ns per 128 x 128 block (1024 cycles of products at 2 GHz are 512), 765 with
// the full causal mask, the rest masked blocks and the tiles' seams; products
// and copies alone take 540 ns.  What bounds it is the chain scores
// -> softmax -> P of the one warp per scheduler; hence barriers are probed
// ahead, under arithmetic and stores (4 % of the time).  Two softmax groups
// that take the blocks in turn were 1 to 4 % faster with long windows and 3 to
// 20 % slower with short ones, because they share one running maximum and one
// P; eight warps with half a block's columns each were 7 % slower: the products'
// issue holds up the warps of its sub-partition, and the maxima are swapped.

namespace wf {
constexpr int kTile = 128 * 128 * 2;  // [128][128] bf16, stored as two 64-column halves
constexpr int kHalf = kTile / 2;
constexpr int kStages = 3;            // K and V ring depth
constexpr int OFF_Q = 0;
constexpr int OFF_K = OFF_Q + kTile;
constexpr int OFF_V = OFF_K + kStages * kTile;
constexpr int OFF_BAR = OFF_V + kStages * kTile;

enum {
  B_Q_FULL,
  B_Q_TMEM,  // Q copied into TMEM by the softmax warps
  B_K_FULL,
  B_K_EMPTY = B_K_FULL + kStages,
  B_V_FULL = B_K_EMPTY + kStages,
  B_V_EMPTY = B_V_FULL + kStages,
  B_S_FULL = B_V_EMPTY + kStages,
  B_S_READ,                  // the softmax warps have read the score buffer
  B_P_FULL,                  // P written, per P buffer
  B_P_EMPTY = B_P_FULL + 2,  // P V done: that P buffer free, O up to date
  B_DRAIN = B_P_EMPTY + 2,
  B_DRAIN_PV,
  B_COUNT
};
constexpr int OFF_TMEM_SLOT = OFF_BAR + B_COUNT * 8;
constexpr int OFF_ABORT = OFF_TMEM_SLOT + 8;
constexpr int kSmemBytes = OFF_ABORT + 8 + 1024;  // + alignment slack

constexpr int kThreads = 224;  // softmax warps 0-3, producer 4, S issuer 5, PV issuer 6
constexpr int TM_Q = 0;    // Q, packed bf16: columns [0, 64)
constexpr int TM_S = 64;   // scores: [64, 192)
constexpr int TM_O = 192;  // O accumulator: [192, 320)
constexpr int TM_P = 320;  // two P buffers, packed bf16: [320, 384), [384, 448)

}  // namespace wf

__global__ void __launch_bounds__(wf::kThreads, 1)
    window_fwd_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                    const __grid_constant__ CUtensorMap mv, const __grid_constant__ WinParams p) {
  using namespace wf;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(smem);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  // A CTA walks query tiles gridDim.x apart.  Heads vary fastest: the CTAs in
  // flight hold the same query blocks of every head, whose K/V blocks (shared
  // within a GQA group) stay in L2; the query blocks with the most KV blocks
  // come first.
  const int m_tiles = ((p.L - 1) >> 7) + 1;
  const int n_tiles = m_tiles * p.H;
  const int stride = static_cast<int>(gridDim.x);
  const int first = static_cast<int>(blockIdx.x);
  // Every second round runs the other way, so that a sequence's first tiles,
  // which have fewer blocks, spread over all CTAs.
  auto tile_of = [&](int n) { return n * stride + (n & 1 ? stride - 1 - first : first); };
  auto head_of = [&](int t) { return t % p.H; };
  auto block_of = [&](int t) { return m_tiles - 1 - t / p.H; };
  auto bar = [&](int i) -> uint32_t { return sb + OFF_BAR + 8 * i; };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + OFF_ABORT);
  const WaitCtl w{abort_flag, p.status, p.limit_ns};

  if (threadIdx.x == 0) {
    mbar_init(bar(B_Q_FULL), 1);
    mbar_init(bar(B_Q_TMEM), 4);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(bar(B_K_FULL + s), 1);
      mbar_init(bar(B_K_EMPTY + s), 1);
      mbar_init(bar(B_V_FULL + s), 1);
      mbar_init(bar(B_V_EMPTY + s), 1);
    }
    mbar_init(bar(B_S_FULL), 1);
    mbar_init(bar(B_S_READ), 4);
    for (int b = 0; b < 2; ++b) {
      mbar_init(bar(B_P_FULL + b), 4);
      mbar_init(bar(B_P_EMPTY + b), 1);
    }
    mbar_init(bar(B_DRAIN), 1);
    mbar_init(bar(B_DRAIN_PV), 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 5) {
    tmem_alloc(sb + OFF_TMEM_SLOT, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + OFF_TMEM_SLOT);

  if (warp == 4) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      tma_prefetch_map(&mq);
      tma_prefetch_map(&mk);
      tma_prefetch_map(&mv);
      auto load_q = [&](int t) {
        mbar_expect_tx(bar(B_Q_FULL), kTile);
        tma_load_3d(sb + OFF_Q, &mq, bar(B_Q_FULL), 0, block_of(t) * 128, head_of(t));
        tma_load_3d(sb + OFF_Q + kHalf, &mq, bar(B_Q_FULL), 64, block_of(t) * 128, head_of(t));
      };
      int last_k[kStages], last_v[kStages];
#pragma unroll
      for (int s = 0; s < kStages; ++s) last_k[s] = last_v[s] = -1;
      load_q(first);
      int last_q = 0;  // the Q load issued last
      int it = 0;      // KV blocks of all tiles so far
      bool ok = true;
      for (int n = 0, t = tile_of(0); ok && t < n_tiles; t = tile_of(++n)) {
        const QuerySpan sp(block_of(t), p);
        const int kz = head_of(t) / p.g;
        const int n_kv = sp.count();
        for (int j = 0; j < n_kv; ++j, ++it) {
          const int s = it % kStages;
          const uint32_t ph = (it / kStages) & 1;
          const int row = sp.block(j) * 128;
          if (!(ok = mbar_wait(bar(B_K_EMPTY + s), ph ^ 1, w))) break;
          mbar_expect_tx(bar(B_K_FULL + s), kTile);
          tma_load_3d(sb + OFF_K + s * kTile, &mk, bar(B_K_FULL + s), 0, row, kz);
          tma_load_3d(sb + OFF_K + s * kTile + kHalf, &mk, bar(B_K_FULL + s), 64, row, kz);
          last_k[s] = it;
          if (!(ok = mbar_wait(bar(B_V_EMPTY + s), ph ^ 1, w))) break;
          mbar_expect_tx(bar(B_V_FULL + s), kTile);
          tma_load_3d(sb + OFF_V + s * kTile, &mv, bar(B_V_FULL + s), 0, row, kz);
          tma_load_3d(sb + OFF_V + s * kTile + kHalf, &mv, bar(B_V_FULL + s), 64, row, kz);
          last_v[s] = it;
          // The next tile's Q as soon as this one's is in TMEM, a block or
          // more before it is wanted.
          if (j == (n_kv > 1 ? 1 : 0) && tile_of(n + 1) < n_tiles) {
            if (!(ok = mbar_wait(bar(B_Q_TMEM), n & 1, w))) break;
            load_q(tile_of(n + 1));
            last_q = n + 1;
          }
        }
      }
      if (*abort_flag) {  // let every issued copy land before the CTA exits
        mbar_wait_drain(bar(B_Q_FULL), last_q & 1, p.status);
        for (int s = 0; s < kStages; ++s) {
          if (last_k[s] >= 0) mbar_wait_drain(bar(B_K_FULL + s), (last_k[s] / kStages) & 1, p.status);
          if (last_v[s] >= 0) mbar_wait_drain(bar(B_V_FULL + s), (last_v[s] / kStages) & 1, p.status);
        }
      }
    }
  } else if (warp == 5) {
    // ------------------------------------------------------------ S issuer
    constexpr uint32_t id_s = idesc_bf16(128, 128, 0, 0);  // Q (TMEM) x K (smem, K-major)
    // S(j) once K(j) has landed and the softmax warps have read S(j - 1);
    // a tile's first one also wants its Q in TMEM.
    bool ok = true;
    int it = 0;
    for (int n = 0, t = tile_of(0); ok && t < n_tiles; t = tile_of(++n)) {
      const int n_kv = QuerySpan(block_of(t), p).count();
      if (!(ok = warp_wait<false, true>(bar(B_Q_TMEM), n & 1, w))) break;
      for (int j = 0; j < n_kv; ++j, ++it) {
        const int s = it % kStages;
        if (!(ok = warp_wait<false, true>(bar(B_K_FULL + s), (it / kStages) & 1, w))) break;
        if (!(ok = warp_wait<false, true>(bar(B_S_READ), (it & 1) ^ 1, w))) break;
        tc_fence_after();
        const uint32_t ka = sb + OFF_K + s * kTile;
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          umma_ts_one(tmem + TM_S, tmem + TM_Q + kk * 8,
                       sdesc_sw128(ka + (kk >> 2) * kHalf + (kk & 3) * 32, 16, 1024), id_s, kk > 0 ? 1u : 0u);
        }
        commit_one(bar(B_S_FULL));
        commit_one(bar(B_K_EMPTY + s));
      }
    }
    commit_one(bar(B_DRAIN));
    mbar_wait_drain(bar(B_DRAIN), 0, p.status);
  } else if (warp == 6) {
    // ----------------------------------------------------------- PV issuer
    constexpr uint32_t id_o = idesc_bf16(128, 128, 0, 1);  // P (TMEM) x V (smem, MN-major)
    bool ok = true;
    int it = 0;
    for (int n = 0, t = tile_of(0); ok && t < n_tiles; t = tile_of(++n)) {
      const int n_kv = QuerySpan(block_of(t), p).count();
      for (int j = 0; j < n_kv; ++j, ++it) {
        const int b = it & 1;
        const int s = it % kStages;
        // a tile's first P is written after the last tile's O has been read
        if (!(ok = warp_wait<false, true>(bar(B_P_FULL + b), (it >> 1) & 1, w))) break;
        if (!(ok = warp_wait<false, true>(bar(B_V_FULL + s), (it / kStages) & 1, w))) break;
        tc_fence_after();
        const uint32_t va = sb + OFF_V + s * kTile;
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          umma_ts_one(tmem + TM_O, tmem + TM_P + b * 64 + kk * 8, sdesc_sw128(va + kk * 2048, kHalf, 1024), id_o,
                       (j > 0 || kk > 0) ? 1u : 0u);
        }
        commit_one(bar(B_P_EMPTY + b));
        commit_one(bar(B_V_EMPTY + s));
      }
    }
    commit_one(bar(B_DRAIN_PV));
    mbar_wait_drain(bar(B_DRAIN_PV), 0, p.status);
  } else {
    // ------------------------------------------------------------- softmax
    const int r = warp * 32 + lane;  // query row in the tile = TMEM lane
    const uint32_t trow = tmem_lane_addr(tmem, warp, 0);
    const float sl2 = p.scale_log2;
    // Row r of the n-th tile's Q -> TMEM (packed bf16, element pairs per column).
    auto take_q = [&](int n) -> bool {
      if (!warp_wait(bar(B_Q_FULL), n & 1, w)) return false;
#pragma unroll
      for (int hq = 0; hq < 2; ++hq) {
        uint32_t q[32];
#pragma unroll
        for (int ch = 0; ch < 8; ++ch) {
          const uint4 v = ld_shared_v4(sb + OFF_Q + hq * kHalf + sw128_offset(r, ch));
          q[4 * ch] = v.x;
          q[4 * ch + 1] = v.y;
          q[4 * ch + 2] = v.z;
          q[4 * ch + 3] = v.w;
        }
        tmem_st32(trow + TM_Q + hq * 32, q);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B_Q_TMEM));
      return true;
    };
    bool ok = take_q(0);
    bool s_there = false;  // the next scores, by a probe made ahead
    int it = 0;
    for (int n = 0, t = tile_of(0); ok && t < n_tiles; t = tile_of(++n)) {
      const int h = head_of(t), qb = block_of(t);
      const QuerySpan sp(qb, p);
      const int n_kv = sp.count();
      const int qpos = qb * 128 + r;
      float m_use = -INFINITY;  // running max used as the exponent offset (log2 domain)
      float l = 0.f;
      for (int j = 0; j < n_kv; ++j, ++it) {
        const int b = it & 1;  // P buffer
        if (!__all_sync(0xffffffffu, s_there) && !(ok = warp_wait(bar(B_S_FULL), it & 1, w))) break;
        tc_fence_after();
        const uint32_t tsb = trow + TM_S;
        uint32_t v0[32], v1[32], v2[32], v3[32];
        tmem_ld32(tsb + 0, v0);
        tmem_ld32(tsb + 32, v1);
        tmem_ld32(tsb + 64, v2);
        tmem_ld32(tsb + 96, v3);
        tmem_ld_wait(v0);
        tmem_ld_wait(v1);
        tmem_ld_wait(v2);
        tmem_ld_wait(v3);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_S_READ));  // S(j + 1) may overwrite the scores

        float x[128];
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          x[c] = __uint_as_float(v0[c]);
          x[32 + c] = __uint_as_float(v1[c]);
          x[64 + c] = __uint_as_float(v2[c]);
          x[96 + c] = __uint_as_float(v3[c]);
        }
        const int kb = sp.block(j);
        if (sp.masked(kb, p)) hide_row(x, qpos, kb * 128, p);
        // Row max: four independent chains of 3-input max.
        float mc[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
        for (int c = 4; c < 124; c += 8) {
          mc[0] = fmax3(mc[0], x[c], x[c + 1]);
          mc[1] = fmax3(mc[1], x[c + 2], x[c + 3]);
          mc[2] = fmax3(mc[2], x[c + 4], x[c + 5]);
          mc[3] = fmax3(mc[3], x[c + 6], x[c + 7]);
        }
        mc[0] = fmax3(mc[0], x[124], x[125]);
        mc[1] = fmax3(mc[1], x[126], x[127]);
        const float mx = fmaxf(fmax3(mc[0], mc[1], mc[2]), mc[3]);
        const float m_new = fmaxf(m_use, mx * sl2);
        const bool need = m_new > m_use + 8.0f;
        if (j > 0 && __any_sync(0xffffffffu, need)) {
          // O holds PV(0..j-1) once PV(j - 1) completes: rescale the rows
          // that moved.
          if (!(ok = warp_wait(bar(B_P_EMPTY + ((it - 1) & 1)), ((it - 1) >> 1) & 1, w))) break;
          tc_fence_after();
          const float f = need ? ex2_approx(m_use - m_new) : 1.f;
#pragma unroll
          for (int c4 = 0; c4 < 4; ++c4) {
            uint32_t o[32];
            tmem_ld32(trow + TM_O + c4 * 32, o);
            tmem_ld_wait(o);
#pragma unroll
            for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * f);
            tmem_st32(trow + TM_O + c4 * 32, o);
          }
          l *= f;
        }
        if (need) m_use = m_new;

        // P buffer b held P(it - 2) until PV(it - 2) completed, long ago as a rule.
        const bool p_free = it < 2 || mbar_test(bar(B_P_EMPTY + b), ((it >> 1) & 1) ^ 1);
        uint32_t pk0[32], pk1[32];
        const uint64_t sl2x2 = f2_pack(sl2, sl2);
        const uint64_t nmx2 = f2_pack(-m_use, -m_use);
        uint64_t acc[4] = {0, 0, 0, 0};  // (+0, +0) pairs
#pragma unroll
        for (int c = 0; c < 64; c += 2) {
          float t0, t1, t2, t3;
          f2_unpack(f2_fma(f2_pack(x[c], x[c + 1]), sl2x2, nmx2), t0, t1);
          f2_unpack(f2_fma(f2_pack(x[64 + c], x[64 + c + 1]), sl2x2, nmx2), t2, t3);
          const float p0 = ex2_approx(t0), p1 = ex2_approx(t1);
          const float p2 = ex2_approx(t2), p3 = ex2_approx(t3);
          acc[(c >> 1) & 1] = f2_add(acc[(c >> 1) & 1], f2_pack(p0, p1));
          acc[2 + ((c >> 1) & 1)] = f2_add(acc[2 + ((c >> 1) & 1)], f2_pack(p2, p3));
          pk0[c >> 1] = pack_bf16x2(p0, p1);
          pk1[c >> 1] = pack_bf16x2(p2, p3);
        }
        if (!__all_sync(0xffffffffu, p_free) &&
            !(ok = warp_wait(bar(B_P_EMPTY + b), ((it >> 1) & 1) ^ 1, w)))
          break;
        tc_fence_after();
        tmem_st32(trow + TM_P + b * 64 + 0, pk0);
        tmem_st32(trow + TM_P + b * 64 + 32, pk1);
        // under the stores: the row's sum, and a look at the next scores
        float rs = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float a, b;
          f2_unpack(acc[i], a, b);
          rs += a + b;
        }
        l += rs;
        s_there = mbar_test(bar(B_S_FULL), (it & 1) ^ 1);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_P_FULL + b));
      }
      if (!ok) break;
      // All S of this tile are done: the next tile's Q goes over this one's, so
      // that its first S is formed under this tile's last PV and epilogue.
      if (tile_of(n + 1) < n_tiles && !(ok = take_q(n + 1))) break;
      // PV products complete in issue order: the last one completing means O is final.
      if (!(ok = warp_wait(bar(B_P_EMPTY + ((it - 1) & 1)), ((it - 1) >> 1) & 1, w))) break;
      tc_fence_after();
      const float inv = 1.f / l;
      const bool valid = qpos < p.L;
      __nv_bfloat16* orow = p.o + (static_cast<int64_t>(qpos) * p.H + h) * kHeadDim;
#pragma unroll
      for (int c4 = 0; c4 < 4; ++c4) {
        uint32_t o[32];
        tmem_ld32(trow + TM_O + c4 * 32, o);
        tmem_ld_wait(o);
        if (valid) store32_bf16(orow + c4 * 32, o, inv, p.sectors);
      }
      if (valid) p.lse[static_cast<int64_t>(h) * p.L + qpos] = (m_use + log2f(l)) * 0.69314718055994530942f;
    }
    tc_fence_before();
  }

  __syncthreads();
  if (warp == 5) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}


// dS row slice of the dq kernel: 32 keys of one query row, paired fp32
// math.  kMask: bit c of `seen` tells whether the query sees key c.
template <bool kMask>
__device__ __forceinline__ void ds_slice(const uint32_t (&sv)[32], const uint32_t (&dv)[32], float sl2, float nlse2,
                                         float dlt, uint32_t seen, uint32_t (&pk)[16]) {
  const uint64_t sl2x2 = f2_pack(sl2, sl2);
  const uint64_t nlx2 = f2_pack(nlse2, nlse2);
  const uint64_t dlx2 = f2_pack(dlt, dlt);
#pragma unroll
  for (int c = 0; c < 32; c += 2) {
    float t0, t1;
    f2_unpack(f2_fma(f2_pack(__uint_as_float(sv[c]), __uint_as_float(sv[c + 1])), sl2x2, nlx2), t0, t1);
    float p0 = ex2_approx(t0), p1 = ex2_approx(t1);
    if (kMask) {
      if (!(seen >> c & 1u)) p0 = 0.f;
      if (!(seen >> (c + 1) & 1u)) p1 = 0.f;
    }
    const uint64_t d = f2_sub(f2_pack(__uint_as_float(dv[c]), __uint_as_float(dv[c + 1])), dlx2);
    float d0, d1;
    f2_unpack(f2_mul(f2_pack(p0, p1), d), d0, d1);
    pk[c >> 1] = pack_bf16x2(d0, d1);
  }
}

// P^T row slice of the dkdv kernel: 16 queries of one key row, from scores
// that hold S - LSE sqrt(d).  kMask: bit c of `seen` tells whether query c
// sees the key.
template <bool kMask>
__device__ __forceinline__ void p_slice(const uint32_t (&sv)[16], float sl2, uint32_t seen, float* pf) {
  const uint64_t sl2x2 = f2_pack(sl2, sl2);
#pragma unroll
  for (int c = 0; c < 16; c += 2) {
    float t0, t1;
    f2_unpack(f2_mul(f2_pack(__uint_as_float(sv[c]), __uint_as_float(sv[c + 1])), sl2x2), t0, t1);
    pf[c] = ex2_approx(t0);
    pf[c + 1] = ex2_approx(t1);
    if (kMask) {
      if (!(seen >> c & 1u)) pf[c] = 0.f;
      if (!(seen >> (c + 1) & 1u)) pf[c + 1] = 0.f;
    }
  }
}

// dS^T row slice of the dkdv kernel: P (dP - Delta) for 16 queries, packed
// bf16, from sums that hold dP - Delta.
__device__ __forceinline__ void dst_slice(const uint32_t (&dv)[16], const float* pf, uint32_t (&dd)[8]) {
#pragma unroll
  for (int c = 0; c < 16; c += 2) {
    float s0, s1;
    f2_unpack(f2_mul(f2_pack(pf[c], pf[c + 1]), f2_pack(__uint_as_float(dv[c]), __uint_as_float(dv[c + 1]))), s0, s1);
    dd[c >> 1] = pack_bf16x2(s0, s1);
  }
}

// Shared-memory descriptor of a K-major operand of 16 columns (32-byte rows,
// 32-byte swizzle, groups of 8 rows 256 bytes apart).
__device__ __forceinline__ uint64_t sdesc_sw32(uint32_t saddr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(1) << 16;
  d |= static_cast<uint64_t>(256 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;  // tcgen05 descriptor version
  d |= static_cast<uint64_t>(6) << 61;  // 32-byte swizzle
  return d;
}

// ================================================================ backward
//
// Two kernels, in which every sum has one order: dQ by query tiles and dK/dV
// by key tiles, each recomputing S and dP (7 products for the gradient's 5: one
// kernel would need atomic or ordered sums of dQ and more TMEM than there is).
// Both keep one CTA per SM and take tiles from a counter, so that the one whose
// CTAs start as the other's end finishes evenly; which CTA computes a tile
// changes nothing in its sums.

// The queries' records, and the counters' zeros.  16 lanes per (query, head),
// 16 bytes of O and of dO each.  A CTA takes 32 queries of one head, so that
// their records and LSE are runs of memory (97 us for 32768 x 32 heads, 570
// MB; 111 us with neighbouring heads side by side, whose records lie L * 32
// bytes apart).
__global__ void __launch_bounds__(256) window_records_kernel(const __grid_constant__ WinParams p,
                                                             __nv_bfloat16* __restrict__ rec) {
  constexpr int U = 2;
  const int sub = threadIdx.x & 15;
  const int h = static_cast<int>(blockIdx.x) % p.H;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x / p.H) * 16 * U + (threadIdx.x >> 4);
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.next_tile = *p.next_item = 0;
  uint4 o[U], g[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t i = (row0 + u * 16) * p.H + h;
    o[u] = g[u] = make_uint4(0u, 0u, 0u, 0u);
    if (row0 + u * 16 < p.L) {
      o[u] = ld_global_nc_v4(p.o + i * kHeadDim + sub * 8);
      g[u] = ld_global_nc_v4(p.dout + i * kHeadDim + sub * 8);
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t ov[4] = {o[u].x, o[u].y, o[u].z, o[u].w}, gv[4] = {g[u].x, g[u].y, g[u].z, g[u].w};
    float acc = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      acc = fmaf(bf16_lo(ov[e]), bf16_lo(gv[e]), acc);
      acc = fmaf(bf16_hi(ov[e]), bf16_hi(gv[e]), acc);
    }
#pragma unroll
    for (int x = 8; x > 0; x >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, x);
    const int64_t row = row0 + u * 16;
    if (sub < 2 && row < p.L) {
      const int64_t at = static_cast<int64_t>(h) * p.L + row;
      uint32_t w[4] = {0u, 0u, 0u, 0u};
      if (sub == 0) {
        const float v[2] = {-p.lse[at] * 11.3137084989847603904f, -acc};  // sqrt(128)
        float part[6];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float left = v[k];
#pragma unroll
          for (int e = 0; e < 3; ++e) {
            part[3 * k + e] = __bfloat162float(__float2bfloat16_rn(left));
            left -= part[3 * k + e];
          }
        }
#pragma unroll
        for (int e = 0; e < 3; ++e) w[e] = pack_bf16x2(part[2 * e], part[2 * e + 1]);
      }
      st_global_v4(rec + at * 16 + sub * 8, w[0], w[1], w[2], w[3]);
    }
  }
}

// dQ: S = Q K^T into one of two TMEM buffers, dP = dO V^T into one that is free
// once read; the compute warps write dS, packed bf16, over the S columns they
// have read, and dQ += dS K takes it from there.  K is held until dQ (three
// stages), V until dP (two).  The next tile's Q and dO are loaded, and its
// first products formed, under this tile's last dQ product and epilogue.
// 32768 tokens, 32 heads, window 4096, alone and from rest: 1.7 ms, 1.03 us per block, of
// which the products by themselves take 0.97 (1536 cycles at 2 GHz are 0.77):
// S and dP read both operands from shared memory, which alone takes 107 cycles
// per 64-cycle product step, and TMEM has no room for Q and dO.
namespace wq {
constexpr int kComputeWarps = 8;
constexpr int kProducerWarp = 8;
constexpr int kMmaWarp = 9;    // issues S; allocates TMEM
constexpr int kGradWarp = 10;  // issues dQ, which consumes dS from TMEM
constexpr int kTile = 128 * 128 * 2;   // [128][128] bf16 as two 64-column halves
constexpr int kHalf = kTile / 2;
constexpr int kKStages = 3;
constexpr int kVStages = 2;
constexpr int kTileSlots = 8;
constexpr int OFF_Q = 0;
constexpr int OFF_DO = OFF_Q + kTile;
constexpr int OFF_K = OFF_DO + kTile;              // kKStages
constexpr int OFF_V = OFF_K + kKStages * kTile;    // kVStages
constexpr int OFF_BAR = OFF_V + kVStages * kTile;
enum {
  B_Q_FULL,
  B_Q_EMPTY,   // the tile's last S done
  B_DO_FULL,
  B_DO_EMPTY,  // the tile's last dP done
  B_TILE,      // a tile's number published, per slot
  B_K_FULL = B_TILE + kTileSlots,
  B_K_EMPTY = B_K_FULL + kKStages,
  B_V_FULL = B_K_EMPTY + kKStages,
  B_V_EMPTY = B_V_FULL + kVStages,
  B_S_FULL = B_V_EMPTY + kVStages,
  B_S_FREE = B_S_FULL + 2,   // dQ of that buffer done: its S/dS columns free
  B_DS_FULL = B_S_FREE + 2,
  B_DP_FULL = B_DS_FULL + 2,
  B_DP_EMPTY,                // the compute warps have read dP
  B_DQ_DONE,
  B_DRAIN,
  B_DRAIN_G,
  B_DRAIN_P,
  B_COUNT
};
constexpr int OFF_TMEM_SLOT = OFF_BAR + B_COUNT * 8;
constexpr int OFF_ABORT = OFF_TMEM_SLOT + 8;
constexpr int OFF_TILE = OFF_ABORT + 8;
constexpr int kSmemBytes = OFF_TILE + kTileSlots * 4 + 1024;
static_assert(kSmemBytes <= 227 * 1024, "dq kernel shared memory");
constexpr int TM_S = 0, TM_DP = 256, TM_DQ = 384;  // S: two 128-column buffers
// Warps 0-7 compute, 8 producer, 9 issues S, 10 issues dQ, 11 issues dP.
constexpr int kDpWarp = 11;
constexpr int kThreadsDq = 384;
}  // namespace wq

__global__ void __launch_bounds__(wq::kThreadsDq, 1)
    window_dq_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                       const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mdo,
                       const __grid_constant__ WinParams p) {
  using namespace wq;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(smem);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  // Tile t: heads vary fastest (GQA siblings share K/V blocks in L2), the query
  // blocks with the most KV blocks come first.
  const int m_tiles = ((p.L - 1) >> 7) + 1;
  const int n_tiles = m_tiles * p.H;
  auto head_of = [&](int t) { return t % p.H; };
  auto block_of = [&](int t) { return m_tiles - 1 - t / p.H; };
  volatile int* tiles = reinterpret_cast<volatile int*>(smem + OFF_TILE);
  auto bar = [&](int i) -> uint32_t { return sb + OFF_BAR + 8 * i; };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + OFF_ABORT);
  const WaitCtl w{abort_flag, p.status, p.limit_ns};

  if (threadIdx.x == 0) {
    for (int i : {B_Q_FULL, B_Q_EMPTY, B_DO_FULL, B_DO_EMPTY}) mbar_init(bar(i), 1);
    for (int i = 0; i < kTileSlots; ++i) mbar_init(bar(B_TILE + i), 1);
    for (int s = 0; s < kKStages; ++s) {
      mbar_init(bar(B_K_FULL + s), 1);
      mbar_init(bar(B_K_EMPTY + s), 1);
    }
    for (int s = 0; s < kVStages; ++s) {
      mbar_init(bar(B_V_FULL + s), 1);
      mbar_init(bar(B_V_EMPTY + s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(bar(B_S_FULL + b), 1);
      mbar_init(bar(B_S_FREE + b), 1);
      mbar_init(bar(B_DS_FULL + b), kComputeWarps);
    }
    mbar_init(bar(B_DP_FULL), 1);
    mbar_init(bar(B_DP_EMPTY), kComputeWarps);
    mbar_init(bar(B_DQ_DONE), 1);
    mbar_init(bar(B_DRAIN), 1);
    mbar_init(bar(B_DRAIN_G), 1);
    mbar_init(bar(B_DRAIN_P), 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(sb + OFF_TMEM_SLOT, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + OFF_TMEM_SLOT);

  if (warp == kProducerWarp) {
    if (lane == 0) {
      tma_prefetch_map(&mq);
      tma_prefetch_map(&mk);
      tma_prefetch_map(&mv);
      tma_prefetch_map(&mdo);
      // Four streams, each of which moves on as soon as it can: the tiles' Q
      // and dO, and the K and V blocks of all tiles behind one another.
      struct Walk {  // a stream's place among the blocks of all tiles
        int n, j, count, kz;
      };
      int published = 0;  // tiles given out so far
      int coming = 0;     // the next one's number, asked for a tile ahead
      auto publish = [&](int t) {
        tiles[published % kTileSlots] = t;
        mbar_arrive(bar(B_TILE + published % kTileSlots));
        ++published;
        if (t < n_tiles) coming = static_cast<int>(gridDim.x) + atomicAdd(p.next_tile, 1);
      };
      auto enter = [&](Walk& x) {  // the stream's next tile; false: no more
        const int t = tiles[x.n % kTileSlots];
        if (t >= n_tiles) return false;
        x.j = 0;
        x.count = QuerySpan(block_of(t), p).count();
        x.kz = head_of(t) / p.g;
        return true;
      };
      auto row_of = [&](const Walk& x) { return QuerySpan(block_of(tiles[x.n % kTileSlots]), p).block(x.j) * 128; };
      publish(static_cast<int>(blockIdx.x));
      Walk k{0, 0, 0, 0}, v{0, 0, 0, 0};
      enter(k);
      enter(v);
      int nq = 0, ndo = 0, nk = 0, nv = 0;  // loads issued
      bool k_on = true, v_on = true, q_on = true, do_on = true;
      Watchdog wd;
      wd.reset();
      bool ok = true;
      while (ok && (q_on || do_on || k_on || v_on)) {
        bool did = false;
        if (q_on && nq < published && mbar_test(bar(B_Q_EMPTY), (nq & 1) ^ 1)) {
          const int t = tiles[nq % kTileSlots];
          if ((q_on = t < n_tiles)) {
            mbar_expect_tx(bar(B_Q_FULL), kTile);
            tma_load_3d(sb + OFF_Q, &mq, bar(B_Q_FULL), 0, block_of(t) * 128, head_of(t));
            tma_load_3d(sb + OFF_Q + kHalf, &mq, bar(B_Q_FULL), 64, block_of(t) * 128, head_of(t));
            ++nq;
          }
          did = true;
        }
        if (k_on && mbar_test(bar(B_K_EMPTY + nk % kKStages), ((nk / kKStages) & 1) ^ 1)) {
          const int s = nk % kKStages;
          const int row = row_of(k);
          mbar_expect_tx(bar(B_K_FULL + s), kTile);
          tma_load_3d(sb + OFF_K + s * kTile, &mk, bar(B_K_FULL + s), 0, row, k.kz);
          tma_load_3d(sb + OFF_K + s * kTile + kHalf, &mk, bar(B_K_FULL + s), 64, row, k.kz);
          ++nk;
          if (++k.j == k.count) {  // the K stream is the one that asks for tiles
            publish(coming);
            ++k.n;
            k_on = enter(k);
          }
          did = true;
        }
        if (do_on && ndo < published && mbar_test(bar(B_DO_EMPTY), (ndo & 1) ^ 1)) {
          const int t = tiles[ndo % kTileSlots];
          if ((do_on = t < n_tiles)) {
            mbar_expect_tx(bar(B_DO_FULL), kTile);
            tma_load_3d(sb + OFF_DO, &mdo, bar(B_DO_FULL), 0, block_of(t) * 128, head_of(t));
            tma_load_3d(sb + OFF_DO + kHalf, &mdo, bar(B_DO_FULL), 64, block_of(t) * 128, head_of(t));
            ++ndo;
          }
          did = true;
        }
        if (v_on && v.j == v.count && v.n + 1 < published) {
          ++v.n;
          v_on = enter(v);
          did = true;
        }
        if (v_on && v.j < v.count && mbar_test(bar(B_V_EMPTY + nv % kVStages), ((nv / kVStages) & 1) ^ 1)) {
          const int s = nv % kVStages;
          const int row = row_of(v);
          mbar_expect_tx(bar(B_V_FULL + s), kTile);
          tma_load_3d(sb + OFF_V + s * kTile, &mv, bar(B_V_FULL + s), 0, row, v.kz);
          tma_load_3d(sb + OFF_V + s * kTile + kHalf, &mv, bar(B_V_FULL + s), 64, row, v.kz);
          ++nv;
          ++v.j;
          did = true;
        }
        if (did) wd.reset();
        else ok = wd.alive(w);
      }
      if (*abort_flag) {  // let every issued copy land before the CTA exits
        if (nq) mbar_wait_drain(bar(B_Q_FULL), (nq - 1) & 1, p.status);
        if (ndo) mbar_wait_drain(bar(B_DO_FULL), (ndo - 1) & 1, p.status);
        for (int i = nk > kKStages ? nk - kKStages : 0; i < nk; ++i)
          mbar_wait_drain(bar(B_K_FULL + i % kKStages), (i / kKStages) & 1, p.status);
        for (int i = nv > kVStages ? nv - kVStages : 0; i < nv; ++i)
          mbar_wait_drain(bar(B_V_FULL + i % kVStages), (i / kVStages) & 1, p.status);
      }
    }
  } else if (warp == kMmaWarp) {
    // S = Q K^T into buffer it & 1 once K has landed and the dQ product
    // two blocks ago has released the buffer.
    constexpr uint32_t id_kk = idesc_bf16(128, 128, 0, 0);
    bool ok = true;
    int it = 0;
    for (int n = 0; ok; ++n) {
      if (!(ok = warp_wait<false, true>(bar(B_TILE + n % kTileSlots), (n / kTileSlots) & 1, w))) break;
      const int t = tiles[n % kTileSlots];
      if (t >= n_tiles) break;
      const int n_kv = QuerySpan(block_of(t), p).count();
      if (!(ok = warp_wait<false, true>(bar(B_Q_FULL), n & 1, w))) break;
      for (int j = 0; j < n_kv; ++j, ++it) {
        const int s = it % kKStages;
        if (!(ok = warp_wait<false, true>(bar(B_K_FULL + s), (it / kKStages) & 1, w))) break;
        if (!(ok = warp_wait<false, true>(bar(B_S_FREE + (it & 1)), ((it >> 1) & 1) ^ 1, w))) break;
        tc_fence_after();
        const uint32_t ka = sb + OFF_K + s * kTile;
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          const uint32_t off = (kk >> 2) * kHalf + (kk & 3) * 32;
          umma_one(tmem + TM_S + (it & 1) * 128, sdesc_sw128(sb + OFF_Q + off, 16, 1024),
                    sdesc_sw128(ka + off, 16, 1024), id_kk, kk > 0 ? 1u : 0u);
        }
        commit_one(bar(B_S_FULL + (it & 1)));
      }
      if (ok) commit_one(bar(B_Q_EMPTY));
    }
    commit_one(bar(B_DRAIN));
    mbar_wait_drain(bar(B_DRAIN), 0, p.status);
  } else if (warp == kDpWarp) {
    // dP = dO V^T once V has landed and the last block's dP has been read.
    constexpr uint32_t id_kk = idesc_bf16(128, 128, 0, 0);
    bool ok = true;
    int it = 0;
    for (int n = 0; ok; ++n) {
      if (!(ok = warp_wait<false, true>(bar(B_TILE + n % kTileSlots), (n / kTileSlots) & 1, w))) break;
      const int t = tiles[n % kTileSlots];
      if (t >= n_tiles) break;
      const int n_kv = QuerySpan(block_of(t), p).count();
      if (!(ok = warp_wait<false, true>(bar(B_DO_FULL), n & 1, w))) break;
      for (int j = 0; j < n_kv; ++j, ++it) {
        const int s = it % kVStages;
        if (!(ok = warp_wait<false, true>(bar(B_V_FULL + s), (it / kVStages) & 1, w))) break;
        if (!(ok = warp_wait<false, true>(bar(B_DP_EMPTY), (it & 1) ^ 1, w))) break;
        tc_fence_after();
        const uint32_t va = sb + OFF_V + s * kTile;
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          const uint32_t off = (kk >> 2) * kHalf + (kk & 3) * 32;
          umma_one(tmem + TM_DP, sdesc_sw128(sb + OFF_DO + off, 16, 1024), sdesc_sw128(va + off, 16, 1024), id_kk,
                    kk > 0 ? 1u : 0u);
        }
        commit_one(bar(B_DP_FULL));
        commit_one(bar(B_V_EMPTY + s));
      }
      if (ok) commit_one(bar(B_DO_EMPTY));
    }
    commit_one(bar(B_DRAIN_P));
    mbar_wait_drain(bar(B_DRAIN_P), 0, p.status);
  } else if (warp == kGradWarp) {
    // dQ += dS K once dS is written; then its S buffer and K stage are free
    // (S had completed before dS existed).  A tile's first dS is written
    // after the compute warps have read the last tile's dQ.
    constexpr uint32_t id_q = idesc_bf16(128, 128, 0, 1);  // dS from TMEM, K MN-major
    bool ok = true;
    int it = 0;
    for (int n = 0; ok; ++n) {
      if (!(ok = warp_wait<false, true>(bar(B_TILE + n % kTileSlots), (n / kTileSlots) & 1, w))) break;
      const int t = tiles[n % kTileSlots];
      if (t >= n_tiles) break;
      const int n_kv = QuerySpan(block_of(t), p).count();
      for (int j = 0; j < n_kv; ++j, ++it) {
        const int b = it & 1;
        const int s = it % kKStages;
        if (!(ok = warp_wait<false, true>(bar(B_DS_FULL + b), (it >> 1) & 1, w))) break;
        tc_fence_after();
        const uint32_t ka = sb + OFF_K + s * kTile;
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          // keys 16 kk .. 16 kk + 15: compute half kk / 4 wrote them at its own
          // 64-column slice of the S buffer
          const uint32_t a = tmem + TM_S + b * 128 + (kk >> 2) * 64 + (kk & 3) * 8;
          umma_ts_one(tmem + TM_DQ, a, sdesc_sw128(ka + kk * 2048, kHalf, 1024), id_q,
                       (j > 0 || kk > 0) ? 1u : 0u);
        }
        commit_one(bar(B_S_FREE + b));
        commit_one(bar(B_K_EMPTY + s));
      }
      if (ok) commit_one(bar(B_DQ_DONE));
    }
    commit_one(bar(B_DRAIN_G));
    mbar_wait_drain(bar(B_DRAIN_G), 0, p.status);
  } else {
    // Compute warps: quadrant (warp & 3) of the TMEM lanes = query rows,
    // half (warp >> 2) of the 128 key columns of each block.
    const int quad = warp & 3;
    const int half = warp >> 2;
    const int r = quad * 32 + lane;
    const uint32_t trow = tmem_lane_addr(tmem, quad, 0);
    const float sl2 = p.scale_log2;
    // The n-th tile's number and this row's record of it.
    float nlse2 = 0.f, dlt = 0.f;  // -LSE * log2(e), Delta
    auto open = [&](int n, int& t) -> bool {
      if (!warp_wait<false, true>(bar(B_TILE + n % kTileSlots), (n / kTileSlots) & 1, w)) return false;
      t = tiles[n % kTileSlots];
      if (t < n_tiles) {
        const int qpos = block_of(t) * 128 + r;
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        if (qpos < p.L) x = ld_global_nc_v4(p.rec + (static_cast<int64_t>(head_of(t)) * p.L + qpos) * 16);
        nlse2 = ((bf16_lo(x.x) + bf16_hi(x.x)) + bf16_lo(x.y)) * sl2;
        dlt = -((bf16_hi(x.y) + bf16_lo(x.z)) + bf16_hi(x.z));
      }
      return true;
    };
    int t = 0, it = 0;
    bool ok = open(0, t);
    for (int n = 0; ok && t < n_tiles; ++n) {
      const int h = head_of(t);
      const QuerySpan sp(block_of(t), p);
      const int n_kv = sp.count();
      const int qpos = sp.qb * 128 + r;
      for (int j = 0; j < n_kv; ++j, ++it) {
        const int b = it & 1;
        if (!(ok = warp_wait<false, true>(bar(B_S_FULL + b), (it >> 1) & 1, w))) break;
        if (!(ok = warp_wait<false, true>(bar(B_DP_FULL), it & 1, w))) break;
        tc_fence_after();
        const uint32_t ts = trow + TM_S + b * 128 + half * 64;
        uint32_t s0[32], s1[32], d0[32], d1[32];
        tmem_ld32(ts, s0);
        tmem_ld32(ts + 32, s1);
        tmem_ld32(trow + TM_DP + half * 64, d0);
        tmem_ld32(trow + TM_DP + half * 64 + 32, d1);
        tmem_ld_wait(s0);
        tmem_ld_wait(s1);
        tmem_ld_wait(d0);
        tmem_ld_wait(d1);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_DP_EMPTY));
        const int kb = sp.block(j);
        const int k0 = kb * 128 + half * 64;  // key of this warp's first column
        uint32_t pk0[16], pk1[16];
        if (sp.masked(kb, p)) {  // warp-uniform
          ds_slice<true>(s0, d0, sl2, nlse2, dlt, seen_keys(qpos, k0, p), pk0);
          ds_slice<true>(s1, d1, sl2, nlse2, dlt, seen_keys(qpos, k0 + 32, p), pk1);
        } else {
          ds_slice<false>(s0, d0, sl2, nlse2, dlt, 0u, pk0);
          ds_slice<false>(s1, d1, sl2, nlse2, dlt, 0u, pk1);
        }
        // dS over the first 32 of the 64 S columns this warp just read.
        tmem_st16(ts, pk0);
        tmem_st16(ts + 16, pk1);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_DS_FULL + b));
      }
      if (!ok) break;
      // The next tile's record is on its way under the last dQ product.
      if (!(ok = open(n + 1, t))) break;
      if (!(ok = warp_wait<false, true>(bar(B_DQ_DONE), n & 1, w))) break;
      // Epilogue: this warp writes 64 columns of its rows.
      tc_fence_after();
      __nv_bfloat16* out = p.dq + (static_cast<int64_t>(qpos) * p.H + h) * kHeadDim + half * 64;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t a[32];
        tmem_ld32(trow + TM_DQ + half * 64 + c * 32, a);
        tmem_ld_wait(a);
        if (qpos < p.L) store32_bf16(out + c * 32, a, p.scale, p.sectors);
      }
    }
    tc_fence_before();
  }

  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}


// dK and dV: a key tile's K and V stay in shared memory while the query tiles
// of the heads that read it stream by.  TMEM holds dV, dK and two regions of
// 128 columns that swap roles every tile:
//   region i & 1:  S^T(i), then P^T(i) and dS^T(i), packed side by side
//   the other one: dP^T(i), then, once that has been read, S^T(i + 1)
// so that the next S^T is formed under this tile's dS^T, dV and dK, and only
// dS^T -> dK -> next dP^T is a chain.  The scores come with -LSE sqrt(d)
// already added and dP^T with -Delta: a K = 16 product step of ones with the
// queries' records, in which each fp32 value is the sum of three bf16 (exact
// to 2^-24 of it); the keys are the rows here, and each warp would otherwise
// have to broadcast every query's two values by shuffle.
// 32768 tokens, 32 heads, window 4096, alone and from rest: 2.7 ms, 1.62 us per tile, of
// which the products by themselves take 1.33 (2048 cycles at 2 GHz are 1.02;
// S^T and dP^T read both operands from shared memory).  With one region for
// each of S^T and dP^T and the values by shuffles it takes a tenth more.
namespace wkv {
constexpr int kTile = 128 * 128 * 2;  // K, V, Q or dO tile: [128 rows][128 d]
constexpr int kHalf = kTile / 2;
constexpr int kQStages = 2;           // Q and its records are held until dK, dO until dV
constexpr int kDoStages = 2;
constexpr int OFF_K = 0;
constexpr int OFF_V = OFF_K + kTile;
constexpr int OFF_Q = OFF_V + kTile;
constexpr int OFF_DO = OFF_Q + kQStages * kTile;
constexpr int kRec = 128 * 16 * 2;    // the records of a query tile
constexpr int OFF_REC = OFF_DO + kDoStages * kTile;
constexpr int OFF_ONES = OFF_REC + kQStages * kRec;  // ones that pick the records' LSE part, then their Delta part
constexpr int OFF_BAR = OFF_ONES + 2 * kRec;
constexpr int kItemSlots = 8;
enum {
  B_K_FULL,
  B_K_EMPTY,  // the item's last S^T done
  B_V_FULL,
  B_V_EMPTY,  // the item's last dP^T done
  B_ITEM,     // an item's number published, per slot
  B_Q_FULL = B_ITEM + kItemSlots,
  B_Q_EMPTY = B_Q_FULL + kQStages,
  B_DO_FULL = B_Q_EMPTY + kQStages,
  B_DO_EMPTY = B_DO_FULL + kDoStages,
  B_S_FULL = B_DO_EMPTY + kDoStages,
  B_P_FULL,                 // P^T written, per region and 64-query half (its 8 compute warps)
  B_DP_FULL = B_P_FULL + 4,
  B_DP_READ,                // the compute warps have read dP^T: its region free
  B_DS_FULL,                // dS^T written
  B_R_FREE,                 // dV and dK done: the region of P^T and dS^T free
  B_DKV_DONE,
  B_DKV_READ,               // the compute warps have read an item's dK and dV
  B_DRAIN,
  B_DRAIN_G,
  B_DRAIN_P,
  B_COUNT
};
constexpr int OFF_TMEM_SLOT = OFF_BAR + B_COUNT * 8;
constexpr int OFF_ABORT = OFF_TMEM_SLOT + 8;
constexpr int OFF_ITEM = OFF_ABORT + 8;
constexpr int kSmemBytes = OFF_ITEM + kItemSlots * 4 + 1024;
static_assert(kSmemBytes <= 227 * 1024, "dK/dV kernel shared memory");
constexpr int TM_R = 0;  // two score regions of 128 columns
constexpr int TM_P = 0, TM_DS = 16;  // of a 32-query slice: packed P^T, packed dS^T
constexpr int TM_DV = 256, TM_DK = 384;
// 16 compute warps: four per TMEM lane quadrant, each owning 32 of the 128
// query columns, so each SM sub-partition has four to hide TMEM and exp2
// latency; then the producer and three MMA-issuing warps (S^T; dV and dK;
// dP^T).
constexpr int kCompute = 16;
constexpr int kProducer = 16;
constexpr int kMma = 17;
constexpr int kGrad = 18;
constexpr int kDpMma = 19;
constexpr int kThreadsKv = 640;
}  // namespace wkv

__global__ void __launch_bounds__(wkv::kThreadsKv, 1)
    window_dkdv_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                         const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mdo,
                         const __grid_constant__ CUtensorMap mrec, const __grid_constant__ WinParams p) {
  using namespace wkv;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(smem);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int n_items = p.key_items;
  volatile int* items = reinterpret_cast<volatile int*>(smem + OFF_ITEM);
  auto bar = [&](int i) -> uint32_t { return sb + OFF_BAR + 8 * i; };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + OFF_ABORT);
  const WaitCtl w{abort_flag, p.status, p.limit_ns};

  if (threadIdx.x == 0) {
    for (int i : {B_K_FULL, B_K_EMPTY, B_V_FULL, B_V_EMPTY}) mbar_init(bar(i), 1);
    for (int i = 0; i < kItemSlots; ++i) mbar_init(bar(B_ITEM + i), 1);
    for (int s = 0; s < kQStages; ++s) {
      mbar_init(bar(B_Q_FULL + s), 1);
      mbar_init(bar(B_Q_EMPTY + s), 1);
    }
    for (int s = 0; s < kDoStages; ++s) {
      mbar_init(bar(B_DO_FULL + s), 1);
      mbar_init(bar(B_DO_EMPTY + s), 2);  // dP^T and dV read it
    }
    for (int i : {B_S_FULL, B_DP_FULL, B_R_FREE}) mbar_init(bar(i), 1);
    for (int i : {B_DP_READ, B_DS_FULL, B_DKV_READ}) mbar_init(bar(i), kCompute);
    for (int i = 0; i < 4; ++i) mbar_init(bar(B_P_FULL + i), kCompute / 2);
    mbar_init(bar(B_DKV_DONE), 1);
    mbar_init(bar(B_DRAIN), 1);
    mbar_init(bar(B_DRAIN_G), 1);
    mbar_init(bar(B_DRAIN_P), 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (threadIdx.x < 256) {  // row r of the two tiles of ones, swizzled as TMA does
    const int r = threadIdx.x & 127, k = threadIdx.x >> 7;
    const uint32_t row = sb + OFF_ONES + k * kRec + r * 32, flip = (r >> 2 & 1) << 4;
    if (k == 0)
      st_shared_v4(row + flip, 0x3F803F80u, 0x00003F80u, 0u, 0u);  // columns 0 1 2
    else
      st_shared_v4(row + flip, 0u, 0x3F800000u, 0x3F803F80u, 0u);  // columns 3 4 5
    st_shared_v4(row + (flip ^ 16), 0u, 0u, 0u, 0u);
    fence_async_smem();
  }
  if (warp == kMma) {
    tmem_alloc(sb + OFF_TMEM_SLOT, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + OFF_TMEM_SLOT);

  if (warp == kProducer) {
    // Four streams, each of which moves on as soon as it can: the items' K and
    // V, and the Q and dO tiles of all items behind one another.
    if (lane == 0) {
      tma_prefetch_map(&mq);
      tma_prefetch_map(&mk);
      tma_prefetch_map(&mv);
      tma_prefetch_map(&mdo);
      tma_prefetch_map(&mrec);
      int published = 0;  // items given out so far
      int coming = 0;     // the next one's number, asked for an item ahead
      auto ask = [&] { return static_cast<int>(gridDim.x) + atomicAdd(p.next_item, 1); };
      auto publish = [&](int i) {
        // a later sink tile's last shares hold nothing: no role sees them
        while (i < n_items && KeyItem(i, p).empty()) i = ask();
        items[published % kItemSlots] = i;
        mbar_arrive(bar(B_ITEM + published % kItemSlots));
        ++published;
        if (i < n_items) coming = ask();
      };
      publish(static_cast<int>(blockIdx.x));
      int nk = 0, nv = 0, nq = 0, ndo = 0;  // loads issued
      int q_item = 0, do_item = 0;          // the items that the Q and dO streams are in
      bool q_on = items[0] < n_items, do_on = q_on, k_on = true, v_on = true;
      KeyWalk xq(KeyItem(q_on ? items[0] : 0, p), p), xdo = xq;
      bool do_next = false;  // the dO stream is past its item's last tile
      Watchdog wd;
      wd.reset();
      bool ok = true;
      while (ok && (q_on || do_on || k_on || v_on)) {
        bool did = false;
        if (k_on && nk < published && mbar_test(bar(B_K_EMPTY), (nk & 1) ^ 1)) {
          const int i = items[nk % kItemSlots];
          if ((k_on = i < n_items)) {
            const KeyItem item(i, p);
            mbar_expect_tx(bar(B_K_FULL), kTile);
            tma_load_3d(sb + OFF_K, &mk, bar(B_K_FULL), 0, item.kb * 128, item.kv);
            tma_load_3d(sb + OFF_K + kHalf, &mk, bar(B_K_FULL), 64, item.kb * 128, item.kv);
            ++nk;
          }
          did = true;
        }
        if (q_on && mbar_test(bar(B_Q_EMPTY + nq % kQStages), ((nq / kQStages) & 1) ^ 1)) {
          const int s = nq % kQStages;
          mbar_expect_tx(bar(B_Q_FULL + s), kTile + kRec);
          tma_load_3d(sb + OFF_REC + s * kRec, &mrec, bar(B_Q_FULL + s), 0, xq.qt * 128, xq.h);
          tma_load_3d(sb + OFF_Q + s * kTile, &mq, bar(B_Q_FULL + s), 0, xq.qt * 128, xq.h);
          tma_load_3d(sb + OFF_Q + s * kTile + kHalf, &mq, bar(B_Q_FULL + s), 64, xq.qt * 128, xq.h);
          ++nq;
          if (!xq.next()) {  // this stream is the one that asks for items
            publish(coming);
            const int i = items[++q_item % kItemSlots];
            if ((q_on = i < n_items)) xq = KeyWalk(KeyItem(i, p), p);
          }
          did = true;
        }
        if (do_next && do_item + 1 < published) {
          const int i = items[++do_item % kItemSlots];
          do_next = false;
          if ((do_on = i < n_items)) xdo = KeyWalk(KeyItem(i, p), p);
          did = true;
        }
        if (do_on && !do_next && mbar_test(bar(B_DO_EMPTY + ndo % kDoStages), ((ndo / kDoStages) & 1) ^ 1)) {
          const int s = ndo % kDoStages;
          mbar_expect_tx(bar(B_DO_FULL + s), kTile);
          tma_load_3d(sb + OFF_DO + s * kTile, &mdo, bar(B_DO_FULL + s), 0, xdo.qt * 128, xdo.h);
          tma_load_3d(sb + OFF_DO + s * kTile + kHalf, &mdo, bar(B_DO_FULL + s), 64, xdo.qt * 128, xdo.h);
          ++ndo;
          do_next = !xdo.next();
          did = true;
        }
        if (v_on && nv < published && mbar_test(bar(B_V_EMPTY), (nv & 1) ^ 1)) {
          const int i = items[nv % kItemSlots];
          if ((v_on = i < n_items)) {
            const KeyItem item(i, p);
            mbar_expect_tx(bar(B_V_FULL), kTile);
            tma_load_3d(sb + OFF_V, &mv, bar(B_V_FULL), 0, item.kb * 128, item.kv);
            tma_load_3d(sb + OFF_V + kHalf, &mv, bar(B_V_FULL), 64, item.kb * 128, item.kv);
            ++nv;
          }
          did = true;
        }
        if (did) wd.reset();
        else ok = wd.alive(w);
      }
      if (*abort_flag) {  // let every issued copy land before the CTA exits
        if (nk) mbar_wait_drain(bar(B_K_FULL), (nk - 1) & 1, p.status);
        if (nv) mbar_wait_drain(bar(B_V_FULL), (nv - 1) & 1, p.status);
        for (int i = nq > kQStages ? nq - kQStages : 0; i < nq; ++i)
          mbar_wait_drain(bar(B_Q_FULL + i % kQStages), (i / kQStages) & 1, p.status);
        for (int i = ndo > kDoStages ? ndo - kDoStages : 0; i < ndo; ++i)
          mbar_wait_drain(bar(B_DO_FULL + i % kDoStages), (i / kDoStages) & 1, p.status);
      }
    }
  } else if (warp == kMma) {
    // S^T = K Q^T, and -LSE sqrt(d) of each query by the records' step, into
    // region it & 1 once Q has landed and the last tile's dP^T, which was
    // there, has been read.
    constexpr uint32_t id_s = idesc_bf16(128, 128, 0, 0);
    bool ok = true;
    int it = 0;
    for (int n = 0; ok; ++n) {
      if (!(ok = warp_wait<false, true>(bar(B_ITEM + n % kItemSlots), (n / kItemSlots) & 1, w))) break;
      const int i = items[n % kItemSlots];
      if (i >= n_items) break;
      const int n_it = KeyItem(i, p).tiles() * p.g;
      if (!(ok = warp_wait<false, true>(bar(B_K_FULL), n & 1, w))) break;
      for (const int end = it + n_it; it < end; ++it) {
        const int qs = it % kQStages;
        if (!(ok = warp_wait<false, true>(bar(B_Q_FULL + qs), (it / kQStages) & 1, w))) break;
        if (!(ok = warp_wait<false, true>(bar(B_DP_READ), (it & 1) ^ 1, w))) break;
        tc_fence_after();
        const uint32_t bq = sb + OFF_Q + qs * kTile;
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          const uint32_t off = (kk >> 2) * kHalf + (kk & 3) * 32;
          umma_one(tmem + TM_R + (it & 1) * 128, sdesc_sw128(sb + OFF_K + off, 16, 1024),
                    sdesc_sw128(bq + off, 16, 1024), id_s, kk > 0 ? 1u : 0u);
        }
        umma_one(tmem + TM_R + (it & 1) * 128, sdesc_sw32(sb + OFF_ONES), sdesc_sw32(sb + OFF_REC + qs * kRec), id_s,
                  1u);
        commit_one(bar(B_S_FULL));
      }
      if (ok) commit_one(bar(B_K_EMPTY));
    }
    commit_one(bar(B_DRAIN));
    mbar_wait_drain(bar(B_DRAIN), 0, p.status);
  } else if (warp == kDpMma) {
    // dP^T = V dO^T, and -Delta of each query by the records' step, into the
    // other region once dO (and Q, with the records) has landed and the last
    // tile's dV and dK, whose P^T and dS^T were there, are done.
    constexpr uint32_t id_s = idesc_bf16(128, 128, 0, 0);
    bool ok = true;
    int it = 0;
    for (int n = 0; ok; ++n) {
      if (!(ok = warp_wait<false, true>(bar(B_ITEM + n % kItemSlots), (n / kItemSlots) & 1, w))) break;
      const int i = items[n % kItemSlots];
      if (i >= n_items) break;
      const int n_it = KeyItem(i, p).tiles() * p.g;
      if (!(ok = warp_wait<false, true>(bar(B_V_FULL), n & 1, w))) break;
      for (const int end = it + n_it; it < end; ++it) {
        const int qs = it % kDoStages;
        if (!(ok = warp_wait<false, true>(bar(B_DO_FULL + qs), (it / kDoStages) & 1, w))) break;
        if (!(ok = warp_wait<false, true>(bar(B_Q_FULL + it % kQStages), (it / kQStages) & 1, w))) break;
        if (!(ok = warp_wait<false, true>(bar(B_R_FREE), (it & 1) ^ 1, w))) break;
        tc_fence_after();
        const uint32_t bq = sb + OFF_DO + qs * kTile;
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          const uint32_t off = (kk >> 2) * kHalf + (kk & 3) * 32;
          umma_one(tmem + TM_R + (~it & 1) * 128, sdesc_sw128(sb + OFF_V + off, 16, 1024),
                    sdesc_sw128(bq + off, 16, 1024), id_s, kk > 0 ? 1u : 0u);
        }
        umma_one(tmem + TM_R + (~it & 1) * 128, sdesc_sw32(sb + OFF_ONES + kRec),
                  sdesc_sw32(sb + OFF_REC + it % kQStages * kRec), id_s, 1u);
        commit_one(bar(B_DP_FULL));
        commit_one(bar(B_DO_EMPTY + qs));
      }
      if (ok) commit_one(bar(B_V_EMPTY));
    }
    commit_one(bar(B_DRAIN_P));
    mbar_wait_drain(bar(B_DRAIN_P), 0, p.status);
  } else if (warp == kGrad) {
    // dV += P^T dO half by half as each half's P^T is written, then dK +=
    // dS^T Q; both operands lie in region it & 1, free once both are done.
    // (P^T of the next tile may be written before this thread has seen this
    // one's, hence a barrier per region: the tile after next needs R_FREE.)
    constexpr uint32_t id_g = idesc_bf16(128, 128, 0, 1);  // A from TMEM, B MN-major
    auto issue_grad = [&](int it, bool more, int tm_a, uint32_t b, int tm_d, int kk0, int kk1) {
      for (int kk = kk0; kk < kk1; ++kk) {
        // queries 16 kk .. 16 kk + 15: compute group kk / 2 wrote them at
        // its own 32-column slice
        const uint32_t a = tmem + TM_R + (it & 1) * 128 + tm_a + (kk >> 1) * 32 + (kk & 1) * 8;
        umma_ts_one(tmem + tm_d, a, sdesc_sw128(b + kk * 2048, kHalf, 1024), id_g, (more || kk > 0) ? 1u : 0u);
      }
    };
    // An item's first product waits until all compute warps have read the
    // last item's sums (P^T of a half comes from half of them).
    bool ok = true;
    int it = 0;
    for (int n = 0; ok; ++n) {
      if (!(ok = warp_wait<false, true>(bar(B_ITEM + n % kItemSlots), (n / kItemSlots) & 1, w))) break;
      const int i = items[n % kItemSlots];
      if (i >= n_items) break;
      const int n_it = KeyItem(i, p).tiles() * p.g;
      const int begin = it;
      if (!(ok = warp_wait<false, true>(bar(B_DKV_READ), (n & 1) ^ 1, w))) break;
      for (const int end = it + n_it; ok && it < end; ++it) {
        // (P^T says nothing of dO, which dV reads from shared memory.)
        if (!(ok = warp_wait<false, true>(bar(B_DO_FULL + it % kDoStages), (it / kDoStages) & 1, w))) break;
        const uint32_t bdo = sb + OFF_DO + it % kDoStages * kTile;
        for (int hf = 0; hf < 2; ++hf) {
          if (!(ok = warp_wait<false, true>(bar(B_P_FULL + 2 * (it & 1) + hf), (it >> 1) & 1, w))) break;
          tc_fence_after();
          issue_grad(it, it > begin, TM_P, bdo, TM_DV, 4 * hf, 4 * hf + 4);
        }
        if (!ok) break;
        commit_one(bar(B_DO_EMPTY + it % kDoStages));
        if (!(ok = warp_wait<false, true>(bar(B_DS_FULL), it & 1, w))) break;
        tc_fence_after();
        issue_grad(it, it > begin, TM_DS, sb + OFF_Q + it % kQStages * kTile, TM_DK, 0, 8);
        commit_one(bar(B_R_FREE));
        commit_one(bar(B_Q_EMPTY + it % kQStages));
      }
      if (ok) commit_one(bar(B_DKV_DONE));
    }
    commit_one(bar(B_DRAIN_G));
    mbar_wait_drain(bar(B_DRAIN_G), 0, p.status);
  } else {
    // Compute warps: quadrant (warp & 3) of the key rows, group (warp >> 2)
    // of 32 query columns of each tile.
    const int quad = warp & 3;
    const int grp = warp >> 2;
    const int r = quad * 32 + lane;  // key row = TMEM lane
    const uint32_t trow = tmem_lane_addr(tmem, quad, 0);
    const float sl2 = p.scale_log2;
    // Epilogue: groups 0-1 own dK, 2-3 own dV, 64 columns each.
    const int which = grp >> 1;
    const int col0 = (grp & 1) * 64;
    const uint32_t my_tm = trow + (which == 0 ? TM_DK : TM_DV) + col0;
    bool ok = true;
    int it = 0;
    for (int n = 0; ok; ++n) {
      if (!(ok = warp_wait<false, true>(bar(B_ITEM + n % kItemSlots), (n / kItemSlots) & 1, w))) break;
      const int i = items[n % kItemSlots];
      if (i >= n_items) break;
      const KeyItem item(i, p);
      const int kpos = item.kb * 128 + r;
      const int last_q = last_query(kpos, p);
      KeyWalk x(item, p);
      do {
        const int qt = x.qt;
        const int q0 = qt * 128 + grp * 32;  // query of this warp's first column
        const bool masked = hides(qt, item.kb, p);  // warp-uniform
        // queries from the key's own to the last one whose window reaches it
        const uint32_t seen = masked ? bits_below(last_q - q0 + 1) & ~bits_below(kpos - q0) : ~0u;
        // ---- phase 1: P^T over the S^T columns, 16 at a time; the packed
        // P^T of columns 16 h .. 16 h + 15 goes to columns 8 h .. 8 h + 7, which
        // this warp has already read.
        const uint32_t ts = trow + TM_R + (it & 1) * 128 + grp * 32;
        const uint32_t td = trow + TM_R + (~it & 1) * 128 + grp * 32;
        if (!(ok = warp_wait<false, true>(bar(B_S_FULL), it & 1, w))) break;
        tc_fence_after();
        float pf[32];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t sv[16];
          tmem_ld16(ts + 16 * h, sv);
          tmem_ld_wait(sv);
          if (masked)
            p_slice<true>(sv, sl2, seen >> 16 * h, pf + 16 * h);
          else
            p_slice<false>(sv, sl2, 0u, pf + 16 * h);
          uint32_t pk[8];
#pragma unroll
          for (int c = 0; c < 8; ++c) pk[c] = pack_bf16x2(pf[16 * h + 2 * c], pf[16 * h + 2 * c + 1]);
          tmem_st8(ts + TM_P + 8 * h, pk);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_P_FULL + 2 * (it & 1) + (grp >> 1)));
        // ---- phase 2: dS^T = P^T * (dP^T - Delta) into the other half of the
        // S^T columns
        if (!(ok = warp_wait<false, true>(bar(B_DP_FULL), it & 1, w))) break;
        tc_fence_after();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t dv[16];
          tmem_ld16(td + 16 * h, dv);
          tmem_ld_wait(dv);
          if (h == 1) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(B_DP_READ));  // the next S^T may be formed there
          }
          uint32_t dd[8];
          dst_slice(dv, pf + 16 * h, dd);
          tmem_st8(ts + TM_DS + 8 * h, dd);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_DS_FULL));
        ++it;
      } while (x.next());
      if (!ok || !(ok = warp_wait<false, true>(bar(B_DKV_DONE), n & 1, w))) break;
      tc_fence_after();
      __nv_bfloat16* out = (which == 0 ? p.dk : p.dv) + (static_cast<int64_t>(kpos) * p.Hkv + item.kv) * kHeadDim + col0;
      const float scale = which == 0 ? p.scale : 1.f;
      // a sink's sum is shared by several CTAs, every other key's is complete in its tile's own
      float* part = item.slot >= 0 && kpos < p.sinks ? item.part(p) + (which * p.sink_rows + r) * kHeadDim + col0 : nullptr;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t v[32];
        tmem_ld32(my_tm + c * 32, v);
        tmem_ld_wait(v);
        if (part) {
#pragma unroll
          for (int q = 0; q < 8; ++q)
            st_global_v4(part + c * 32 + q * 4, v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
        } else if (kpos < p.L && item.slot <= 0) {
          store32_bf16(out + c * 32, v, scale, p.sectors);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B_DKV_READ));
    }
    tc_fence_before();
  }

  __syncthreads();
  if (warp == kMma) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// dK and dV of the sinks: the shares of one key are added in the order of
// their slots, the tile's own first.  One warp per (KV head, sink, dK or dV).
__global__ void __launch_bounds__(256) window_sink_kernel(const __grid_constant__ WinParams p) {
  const int64_t row = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (row >= static_cast<int64_t>(2) * p.shared_keys * p.Hkv) return;
  const int which = static_cast<int>(row & 1);
  const int key = static_cast<int>((row >> 1) % p.shared_keys);
  const int kv = static_cast<int>((row >> 1) / p.shared_keys);
  const int kb = key >> 7;
  const int far = ((p.L - 1) >> 7) + 1 - kb - p.near_tiles;  // query tiles past the tile's window
  const int slots = 1 + (far + p.far_chunk - 1) / p.far_chunk;
  const int64_t size = static_cast<int64_t>(2) * p.sink_rows * kHeadDim;
  const float* part = p.sink_part + (static_cast<int64_t>(kv) * p.sink_tiles + kb) * (p.far_slots + 1) * size +
                      (which * p.sink_rows + (key & 127)) * kHeadDim + lane * 4;
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (int i = 0; i < slots; ++i) {
    const float4 x = *reinterpret_cast<const float4*>(part + i * size);
    sum.x += x.x;
    sum.y += x.y;
    sum.z += x.z;
    sum.w += x.w;
  }
  const float scale = which == 0 ? p.scale : 1.f;
  __nv_bfloat16* out = (which == 0 ? p.dk : p.dv) + (static_cast<int64_t>(key) * p.Hkv + kv) * kHeadDim + lane * 4;
  *reinterpret_cast<uint2*>(out) =
      make_uint2(pack_bf16x2(sum.x * scale, sum.y * scale), pack_bf16x2(sum.z * scale, sum.w * scale));
}

// ------------------------------------------------------------------- host

constexpr int kSms = 152;  // persistent kernels: one CTA per SM

struct WinShape {
  int64_t L;
  int H, Hkv, m_tiles;
  int window, sinks;
};

bool check_window(const upipe_window_cfg* c, WinShape* s) {
  if (!c || c->L < 1 || c->L > 0x7fffffffLL || c->d != kHeadDim) return false;
  if (c->H < 1 || c->Hkv < 1 || c->H % c->Hkv != 0 || c->H + 2 * static_cast<int64_t>(c->Hkv) > kMaxSlots) return false;
  if (c->window < 1 || c->sinks < 0) return false;
  s->L = c->L;
  s->H = c->H;
  s->Hkv = c->Hkv;
  s->m_tiles = static_cast<int>((c->L + 127) / 128);
  s->window = static_cast<int>(c->window < c->L ? c->window : c->L);
  s->sinks = static_cast<int>(c->sinks < c->L ? c->sinks : c->L);
  return true;
}

// Key tiles that hold sinks are seen by every later query.  Their query tiles
// past the window are cut into chunks, one CTA each, whose fp32 sums of the
// sink rows window_sink_kernel adds up: one CTA for all of them would run on
// alone for most of a long sequence's backward (L = 131072, 8 heads of one KV
// head, window 1024: 14 of 17 ms).  A chunk is half of what an SM gets on
// average, so that the longest shares still balance.
struct SinkPlan {
  int tiles = 0, near = 0, chunk = 1, slots = 0, rows = 0;
  size_t bytes = 0;
};

SinkPlan sink_plan(const WinShape& s) {
  SinkPlan f;
  const int64_t reach = (static_cast<int64_t>(s.window) + 126) / 128 + 1;  // query tiles that a key tile's windows reach
  f.near = static_cast<int>(reach < s.m_tiles ? reach : s.m_tiles);
  f.tiles = (s.sinks + 127) / 128;
  f.rows = s.sinks < 128 ? s.sinks : 128;
  const int64_t far = s.m_tiles - f.near;  // of the first key tile; later ones have fewer
  if (f.tiles == 0 || far <= 0) {
    f.tiles = 0;
    return f;
  }
  if (f.tiles > far) f.tiles = static_cast<int>(far);  // key tiles that have queries past their window
  const int64_t all = static_cast<int64_t>(s.Hkv) * (static_cast<int64_t>(s.m_tiles) * f.near + far * f.tiles);
  const int64_t chunk = (all + 2 * 152 - 1) / (2 * 152);
  if (chunk >= far) {  // one CTA has them done in time
    f.tiles = 0;
    return f;
  }
  f.chunk = static_cast<int>(chunk);
  f.slots = static_cast<int>((far + f.chunk - 1) / f.chunk);
  f.bytes = static_cast<size_t>(s.Hkv) * f.tiles * (f.slots + 1) * 2 * f.rows * kHeadDim * sizeof(float);
  return f;
}

// Workspace: counters, the records of LSE and Delta, the shares of the sinks.
constexpr size_t kCounterBytes = 128;

size_t records_bytes(const WinShape& s) { return static_cast<size_t>(s.H) * static_cast<size_t>(s.L) * 32; }

size_t workspace_bytes(const WinShape& s) { return kCounterBytes + records_bytes(s) + sink_plan(s).bytes; }

bool on_sectors(const void* p) { return reinterpret_cast<uintptr_t>(p) % 32 == 0; }

WinParams base_params(const WinShape& s, int* status) {
  WinParams p;
  std::memset(&p, 0, sizeof(p));
  p.L = static_cast<int>(s.L);
  p.H = s.H;
  p.Hkv = s.Hkv;
  p.g = s.H / s.Hkv;
  p.window = s.window;
  p.sinks = s.sinks;
  p.scale = static_cast<float>(1.0 / std::sqrt(128.0));
  p.scale_log2 = static_cast<float>(1.4426950408889634 / std::sqrt(128.0));
  p.status = status;
  p.limit_ns = spin_limit_ns();
  return p;
}

cudaError_t launch_window_fwd(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const WinParams& p,
                              int m_tiles, cudaStream_t st) {
  cudaError_t e =
      cudaFuncSetAttribute(window_fwd_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, wf::kSmemBytes);
  if (e != cudaSuccess) return e;
  const int grid = m_tiles * p.H < kSms ? m_tiles * p.H : kSms;
  window_fwd_kernel<<<grid, wf::kThreads, wf::kSmemBytes, st>>>(q, k, v, p);
  return cudaGetLastError();
}

cudaError_t launch_window_dq(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const CUtensorMap& dO,
                             const WinParams& p, int m_tiles, cudaStream_t st) {
  cudaError_t e = cudaFuncSetAttribute(window_dq_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, wq::kSmemBytes);
  if (e != cudaSuccess) return e;
  const int grid = m_tiles * p.H < kSms ? m_tiles * p.H : kSms;
  window_dq_kernel<<<grid, wq::kThreadsDq, wq::kSmemBytes, st>>>(q, k, v, dO, p);
  return cudaGetLastError();
}

cudaError_t launch_window_dkdv(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                               const CUtensorMap& dO, const CUtensorMap& rec, const WinParams& p, cudaStream_t st) {
  cudaError_t e =
      cudaFuncSetAttribute(window_dkdv_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, wkv::kSmemBytes);
  if (e != cudaSuccess) return e;
  const int grid = p.key_items < kSms ? p.key_items : kSms;
  window_dkdv_kernel<<<grid, wkv::kThreadsKv, wkv::kSmemBytes, st>>>(q, k, v, dO, rec, p);
  return cudaGetLastError();
}

cudaError_t launch_window_records(const WinParams& p, __nv_bfloat16* rec, cudaStream_t st) {
  window_records_kernel<<<static_cast<unsigned>((static_cast<int64_t>(p.L) + 31) / 32 * p.H), 256, 0, st>>>(p, rec);
  return cudaGetLastError();
}

cudaError_t launch_window_sinks(const WinParams& p, cudaStream_t st) {
  const int64_t warps = static_cast<int64_t>(2) * p.shared_keys * p.Hkv;
  window_sink_kernel<<<static_cast<unsigned>((warps + 7) / 8), 256, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace
}  // namespace upipe

using namespace upipe;

extern "C" {

size_t upipe_window_workspace_bytes(const upipe_window_cfg* cfg) {
  WinShape s;
  return check_window(cfg, &s) ? workspace_bytes(s) : 0;
}

int upipe_window_fwd(const upipe_window_cfg* cfg, const uint16_t* q, const uint16_t* k, const uint16_t* v, uint16_t* o,
                     float* lse, void* stream) {
  WinShape s;
  if (!check_window(cfg, &s)) return UPIPE_ERR_INVALID_ARG;
  if (!q || !k || !v || !o || !lse) return UPIPE_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse))
    return UPIPE_ERR_INVALID_ARG;
  int* status = nullptr;
  if (int e = device_ready(&status)) return e;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  CUtensorMap mq, mk, mv;
  UPIPE_MAP(map3d(&mq, q, s.L, s.H, s.H * 128, 128, 128));
  UPIPE_MAP(map3d(&mk, k, s.L, s.Hkv, s.Hkv * 128, 128, 128));
  UPIPE_MAP(map3d(&mv, v, s.L, s.Hkv, s.Hkv * 128, 128, 128));
  WinParams p = base_params(s, status);
  p.o = reinterpret_cast<__nv_bfloat16*>(o);
  p.sectors = on_sectors(o);
  p.lse = lse;
  UPIPE_LAUNCH(UPIPE_KIND_WINDOW_FWD, launch_window_fwd(mq, mk, mv, p, s.m_tiles, st));
  return UPIPE_OK;
}

int upipe_window_bwd(const upipe_window_cfg* cfg, const uint16_t* q, const uint16_t* k, const uint16_t* v,
                     const uint16_t* o, const float* lse, const uint16_t* dout_o, uint16_t* dq, uint16_t* dk,
                     uint16_t* dv, void* ws, size_t ws_bytes, void* stream) {
  WinShape s;
  if (!check_window(cfg, &s)) return UPIPE_ERR_INVALID_ARG;
  if (!q || !k || !v || !o || !lse || !dout_o || !dq || !dk || !dv || !ws) return UPIPE_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse) || !aligned16(dout_o) ||
      !aligned16(dq) || !aligned16(dk) || !aligned16(dv) || !aligned16(ws))
    return UPIPE_ERR_INVALID_ARG;
  const SinkPlan f = sink_plan(s);
  if (ws_bytes < workspace_bytes(s)) return UPIPE_ERR_WS_TOO_SMALL;
  int* status = nullptr;
  if (int e = device_ready(&status)) return e;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  CUtensorMap mq, mk, mv, mdo;
  UPIPE_MAP(map3d(&mq, q, s.L, s.H, s.H * 128, 128, 128));
  UPIPE_MAP(map3d(&mk, k, s.L, s.Hkv, s.Hkv * 128, 128, 128));
  UPIPE_MAP(map3d(&mv, v, s.L, s.Hkv, s.Hkv * 128, 128, 128));
  UPIPE_MAP(map3d(&mdo, dout_o, s.L, s.H, s.H * 128, 128, 128));
  WinParams p = base_params(s, status);
  uint8_t* const at = static_cast<uint8_t*>(ws);
  __nv_bfloat16* rec = reinterpret_cast<__nv_bfloat16*>(at + kCounterBytes);
  CUtensorMap mrec;
  UPIPE_MAP(map_rows16(&mrec, rec, s.L, s.H, 128));
  p.rec = rec;
  p.o = reinterpret_cast<__nv_bfloat16*>(const_cast<uint16_t*>(o));  // read
  p.dout = reinterpret_cast<const __nv_bfloat16*>(dout_o);
  p.lse = const_cast<float*>(lse);  // read
  p.sink_tiles = f.tiles;
  p.near_tiles = f.near;
  p.far_chunk = f.chunk;
  p.far_slots = f.slots;
  p.sink_rows = f.rows;
  p.shared_keys = s.sinks < f.tiles * 128 ? s.sinks : f.tiles * 128;
  p.sink_part = reinterpret_cast<float*>(at + kCounterBytes + records_bytes(s));
  p.next_tile = reinterpret_cast<int*>(at);
  p.next_item = reinterpret_cast<int*>(at) + 16;
  p.key_items = (s.m_tiles + f.tiles * f.slots) * s.Hkv;
  p.dq = reinterpret_cast<__nv_bfloat16*>(dq);
  p.dk = reinterpret_cast<__nv_bfloat16*>(dk);
  p.dv = reinterpret_cast<__nv_bfloat16*>(dv);
  p.sectors = on_sectors(dq) && on_sectors(dk) && on_sectors(dv);
  UPIPE_LAUNCH(UPIPE_KIND_WINDOW_RECORDS, launch_window_records(p, rec, st));
  // Neither reads what the other writes.  dQ is launched first and on the stream
  // of greatest priority: a CTA of dK/dV starts where one of dQ has run out of
  // tiles, and its counter evens out the different starts.
  struct Job {
    const CUtensorMap &q, &k, &v, &dO, &rec;
    const WinParams& p;
    int m_tiles;
  } job{mq, mk, mv, mdo, mrec, p, s.m_tiles};
  if (int e = launch_beside(
          UPIPE_KIND_WINDOW_DQ,
          [](void* x, cudaStream_t on) {
            const Job& j = *static_cast<Job*>(x);
            return launch_window_dq(j.q, j.k, j.v, j.dO, j.p, j.m_tiles, on);
          },
          UPIPE_KIND_WINDOW_DKDV,
          [](void* x, cudaStream_t on) {
            const Job& j = *static_cast<Job*>(x);
            return launch_window_dkdv(j.q, j.k, j.v, j.dO, j.rec, j.p, on);
          },
          &job, st))
    return e;
  if (f.slots) UPIPE_LAUNCH(UPIPE_KIND_WINDOW_SINKS, launch_window_sinks(p, st));
  return UPIPE_OK;
}

}  // extern "C"
