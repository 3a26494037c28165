// Dense grouped-head (GQA) attention: whole packed prompts, and chunks of new
// tokens (one token: decode) over a paged cache.
//
// For row i of a sequence at position t, head h*G + g of kv head h:
//     l_j = scale q . k_j (j <= t),  out = sum_j exp(l_j - lse) v_j,
//     lse = ln sum_j exp(l_j)
// (the case m = 1, no overlap, every entry visible of the compressed
// attention).  One tcgen05 kernel serves every length; gqa_work.cuh splits the
// key tiles of all (sequence, kv head, row block) items evenly over the CTAs,
// and a second kernel joins the items that several CTAs worked on.
//
// Roles of a CTA (one per SM, 384 threads):
//   warps 0-3, 4-7  softmax warpgroups, one per stream: thread = row, 128
//                   scores read from TMEM, one pass with a running reference
//                   and sum, probabilities written back to TMEM as bf16
//   warp 8          TMA producer (128-byte swizzled K and V tiles, rings)
//   warps 9, 10     issue the MMAs of one stream each, so that neither waits
//                   for the other's softmax: S = Q K^T (both operands in shared
//                   memory), O += P V (P from TMEM, V as it lies in memory,
//                   channel-major for the MMA)
//   warp 11         none (it completes the warpgroup whose registers move)
// Two streams keep the tensor core busy while the other stream is in its
// softmax.  An item of two 128-row tiles gives one tile to each stream, and
// both read the same K/V tile; an item of at most one tile (decode) gives its
// even key tiles to one stream and its odd ones to the other, with their own
// references, sums and accumulators, joined in the epilogue.
// TMEM: S of stream 0 and 1 (128 fp32 columns each; the probabilities overlay
// their scores), O of stream 0 and 1.  A stream's chain is scores -> maximum ->
// exponentials -> product -> next scores; the probabilities are handed over in
// two halves of 64 keys, so that the first half's product runs under the second
// half's exponentials.
//
// The softmax reference of a row follows its running maximum lazily: O and the
// sum are rescaled only when a tile's maximum exceeds the reference by more
// than 2^8, so the accumulator is rarely touched; probabilities then reach at
// most 2^8, far inside bf16 and fp32, and the normalised result is the same.
// Sums are taken in fp32 over the unrounded probabilities; P is rounded to
// bf16 (half a step, 2^-8 relative at most) because the MMA takes 16-bit
// operands.
//
// Measured (B200, 8192-token prompt, 32 query and 8 kv heads of 128 channels,
// 550 GFLOP): 601 us in a sustained run at the power cap (0.56 of the measured
// bf16 peak); the tensor pipe is active half the time.  A 128-key tile takes a
// stream about 3900 clocks: 2400 of softmax (two warps share a scheduler's
// exponential and fp32 units), 770 of MMAs, the rest hand-overs: a barrier
// operation costs 100 to 250 clocks while the score MMAs read both operands from
// shared memory at its full 128 bytes a clock.  Decode (32 sequences of 1000 to
// 16384 tokens, 1.14 GB): 189 to 201 us from GPU to GPU, 0.87 to 0.92 of the
// measured copy bandwidth; there the K/V stream is the bound.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <cmath>
#include <cstring>

#include "common.cuh"
#include "gqa_device.cuh"
#include "gqa_host.h"
#include "gqa_work.cuh"
#include "host_util.h"
#include "tc.cuh"

namespace csa {
namespace {

using namespace gqa;

constexpr int kThreads = 384;
// Registers: 384 threads start with 168 each; the softmax warpgroups take more (a row of scores is 128 of them)
// and the third warpgroup gives up what it does not need: 2 * 208 + 88 = 3 * 168.
constexpr int kSoftmaxRegs = 208, kOtherRegs = 88;
constexpr int kWgThreads = 128;
constexpr int kStep = 64;  // keys of half a tile
constexpr float kRescaleLog2 = 8.f;
// A reference beyond this is subtracted from the scores themselves: the fused v * a - m * a is off by the rounding of
// m * a, 2^-24 of it, which from 2^31 on would leave the range of the exponential.
constexpr float kFarLog2 = 0x1p24f;

// SINGLE: every item of the call fits one 128-row tile (decode), so one Q tile
// is held and the space goes to more stages.
template <int DQK, int DV, bool SINGLE>
struct Shape {
  static constexpr int kQc = DQK / 64, kVc = DV / 64;  // 64-channel (128-byte) column blocks
  static constexpr int kQBytes = kTile * DQK * 2, kVBytes = kTile * DV * 2;
  static constexpr int kQTiles = SINGLE ? 1 : 2;
  static constexpr int kKStages = DQK == 64 ? 5 : (DQK == 128 ? 3 : 2);
  static constexpr int kVStages = DQK == 64 ? 5 : (DQK == 128 ? (SINGLE ? 3 : 2) : (SINGLE ? 2 : 1));
  static constexpr int kRows = kQTiles * kTile;
  static constexpr size_t kKOff = static_cast<size_t>(kQTiles) * kQBytes;
  static constexpr size_t kVOff = kKOff + static_cast<size_t>(kKStages) * kQBytes;
  static constexpr size_t kMiscOff = kVOff + static_cast<size_t>(kVStages) * kVBytes;
  static constexpr size_t kBars = 2 * kKStages + 2 * kVStages + 16;
  // barriers | partition scratch (40 int64) | TMEM slot | (reference, sum) of stream 1
  static constexpr size_t kStatOff = kMiscOff + 8 * kBars + 8 * 40 + 16;
  static constexpr size_t kSmem = ((kStatOff + 15) / 16) * 16 + kWgThreads * 8 + 1024;
  static_assert(kSmem <= 232448, "shared memory");
};

struct Params {
  Geometry g;
  const int32_t* block_table;  // [n_seqs, max_pages]
  int max_pages, page, n_pages;
  int64_t kv_rows;             // rows of the page pool: n_pages * Hkv * page
  int Hq;
  bool wide;                   // out and the workspace start on 32-byte boundaries
  float scale_log2;
  __nv_bfloat16* out;
  float* lse;
  float* part;  // [2 C, rows, DV] unnormalised partial outputs
  float2* ml;   // [2 C, rows] their references (log2 units) and sums
  int4* meta;   // [C] (flags, s, h, blk) of the CTA's first piece
};

constexpr int kMetaOwner = 1;   // the first piece ends its item and does not begin it: this CTA's merge
constexpr int kMetaBegins = 2;  // the last piece begins its item
constexpr int kMetaSingle = 4;  // the last piece is the first

// Pairs of every 8 whose exponentials are computed on the fp32 units.  The exponential unit gives a warp one result in
// 8 clocks, 2048 for two rows of 128 keys: longer than their MMAs where a key has 64 channels, and only there does it
// pay (sustained, two pairs against none: 8192-token prompt of 64 channels 464 against 482 us, documents 139 against
// 142, chunks 204 against 209; of 128 channels 597 and 596; of 192 channels 386 against 365; 4096 tokens, one query
// head per kv head, 103 against 98; three pairs lose everywhere).  A decode step waits for its K/V stream, and the
// polynomial is less exact (2.7e-6 against 2^-22): none.
constexpr int fp32_pairs(int dqk, bool single) { return dqk == 64 && !single ? 2 : 0; }

// Probabilities 2^(v * a + b) of a row's 64 scores: written as bf16 pairs to
// 32 TMEM columns; returns their sum (of the unrounded values).  FMAS of every
// 8 pairs are computed on the fp32 units instead of the exponential unit.
template <int FMAS>
__device__ __forceinline__ float probabilities(float* v, float a, float b, uint32_t tP) {
  // Sixteen at a time, and while the exponential unit works on these, the sums and roundings of the sixteen before: in
  // this order, which the volatile exponentials keep, one warp takes 9.3 clocks a number and two on a scheduler 7.8
  // (as the compiler orders it, 10.3 and 8.5).
  float l0 = 0.f, l1 = 0.f, l2 = 0.f, l3 = 0.f;
  uint32_t pk[16];
  auto finish = [&](int c, int i) {  // pair i of sixteen c
    float* d = v + 16 * c + 2 * i;
    if (i & 1)
      add2(l0, l1, d[0], d[1]);
    else
      add2(l2, l3, d[0], d[1]);
    pk[8 * (c & 1) + i] = pack_bf16x2(d[0], d[1]);
  };
#pragma unroll
  for (int c = 0; c < kStep / 16; ++c) {
    float* e = v + 16 * c;
#pragma unroll
    for (int i = 0; i < 8; ++i) fma2(e[2 * i], e[2 * i + 1], e[2 * i], e[2 * i + 1], a, b);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i >= 8 - FMAS) {
        exp2_fma2(e[2 * i], e[2 * i + 1]);
      } else {
        e[2 * i] = exp2_in_order(e[2 * i]);
        e[2 * i + 1] = exp2_in_order(e[2 * i + 1]);
      }
      if (c > 0) finish(c - 1, i);
    }
    if (c > 0 && c % 2 == 0) tmem_st16(tP + 8 * (c - 2), reinterpret_cast<const float*>(pk));
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) finish(kStep / 16 - 1, i);
  tmem_st16(tP + kStep / 2 - 16, reinterpret_cast<const float*>(pk));
  return (l0 + l1) + (l2 + l3);
}

// The tensor core's turn: an MMA warp says that it issues a stream's last product of a tile and its next scores, and the
// other lets them pass first, so that the core runs one stream's after the other's instead of alternating between them.
// (Alternating, both streams got their scores at the same, later time, and then kept the core idle together: 8192-token
// prompt 590 us, with turns 542.)  Nothing
// but the order depends on it: a warp that reads the word too early does no harm, and waiting ends by itself.
__device__ __forceinline__ void await_turn(const uint32_t* busy) {
  for (int it = 0; it < 64; ++it) {
    uint32_t other;
    asm volatile("ld.volatile.shared::cta.u32 %0, [%1];\n" : "=r"(other) : "r"(smem_u32(busy)) : "memory");
    if (!__any_sync(0xffffffffu, other)) return;
  }
}
__device__ __forceinline__ void set_turn(uint32_t* busy, uint32_t v) {
  asm volatile("st.volatile.shared::cta.u32 [%0], %1;\n" ::"r"(smem_u32(busy)), "r"(v) : "memory");
}

__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kOtherRegs));
}

// 64 scores of a row, -inf from column `vis` on where the tile is masked.
__device__ __forceinline__ void load_scores(float* v, uint32_t taddr, bool masked, int vis) {
  tmem_ld32_async(taddr, v);
  tmem_ld32_async(taddr + 32, v + 32);
  tc::tmem_wait_ld();
  fence_regs(v);
  fence_regs(v + 32);
  if (masked) {
#pragma unroll
    for (int i = 0; i < kStep; ++i) v[i] = i < vis ? v[i] : -INFINITY;
  }
}

// Halves (64 keys) of key tile j that stream s works on.  ks: the keys its last row sees.  An item of one tile of rows
// gives its even and odd key tiles to the two streams.
__device__ __forceinline__ int steps_of(bool one, int s, int j, int ks) {
  const int left = ks - j * kTile;
  if ((one && (j & 1) != s) || left <= 0) return 0;
  return left > kStep ? 2 : 1;
}
// Whether stream s has a tile of [t0, t1): its first one (it works on them up to its last row's keys).
__device__ __forceinline__ bool takes_part(bool one, int s, int t0, int t1, int ks) {
  const int j = one ? t0 + ((t0 & 1) ^ s) : t0;
  return j < t1 && ks > j * kTile;
}
// Keys the last row of stream s sees.
__device__ __forceinline__ int stream_keys(const Geometry& g, const Walk& w, int s) {
  const int tok = w.blk * g.tpb + (w.one ? 1 : s + 1) * g.tpt;
  return w.q.L - w.q.nq + (tok < w.q.nq ? tok : w.q.nq);
}
// Whether tile j holds keys past the sequence's end: each stream that works on it clears their rows of V before its own
// product (zeros over zeros for the second).
__device__ __forceinline__ bool clears_tail(int j, int L) { return L - j * kTile < kTile; }

template <int DQK, int DV, bool PAGED, bool SINGLE>
__global__ void __launch_bounds__(kThreads, 1)
    gqa_attn_kernel(const __grid_constant__ Params p, const __grid_constant__ CUtensorMap qmap,
                    const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
  using S = Shape<DQK, DV, SINGLE>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* Qs = smem;
  uint8_t* Ks = smem + S::kKOff;
  uint8_t* Vs = smem + S::kVOff;
  uint64_t* kfull = reinterpret_cast<uint64_t*>(smem + S::kMiscOff);
  uint64_t* kempty = kfull + S::kKStages;
  uint64_t* vfull = kempty + S::kKStages;
  uint64_t* vempty = vfull + S::kVStages;
  uint64_t* qfull = vempty + S::kVStages;  // [2]
  uint64_t* qempty = qfull + 2;            // [2]
  uint64_t* sfull = qempty + 2;            // [2] scores of a stream are in TMEM
  uint64_t* pfull = sfull + 2;             // [stream][half] probabilities are in TMEM
  uint64_t* odone = pfull + 4;             // [2] a stream's product of a tile is complete
  uint64_t* oempty = odone + 2;            // [2] a stream's O has been read out
  uint64_t* vland = oempty + 2;            // [2] V of a stream's tile with keys past the end has arrived
  int64_t* scratch = reinterpret_cast<int64_t*>(vland + 2);
  uint32_t* tslot = reinterpret_cast<uint32_t*>(scratch + 40);
  uint32_t* busy = tslot + 1;  // [2] a stream's MMAs are being issued
  float2* stat = reinterpret_cast<float2*>(smem + ((S::kStatOff + 15) / 16) * 16);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Geometry& g = p.g;

  // barriers, maps and TMEM need nothing of the kernel before; its results are first read by the partition
  if (tid == 0) {
    prefetch_map(&qmap);
    prefetch_map(&kmap);
    prefetch_map(&vmap);
    busy[0] = busy[1] = 0;
    for (int i = 0; i < S::kKStages; ++i) {
      tc::bar_init(&kfull[i], 1);
      tc::bar_init(&kempty[i], 2);
    }
    for (int i = 0; i < S::kVStages; ++i) {
      tc::bar_init(&vfull[i], 1);
      tc::bar_init(&vempty[i], 2);
    }
    for (int i = 0; i < 2; ++i) {
      tc::bar_init(&qfull[i], 1);
      tc::bar_init(&qempty[i], 2);
      tc::bar_init(&sfull[i], 1);
      tc::bar_init(&pfull[2 * i], 4);
      tc::bar_init(&pfull[2 * i + 1], 4);
      tc::bar_init(&odone[i], 1);
      tc::bar_init(&oempty[i], kWgThreads);
      tc::bar_init(&vland[i], 1);
    }
    tc::bar_init_fence();
  }
  if (warp == 9) tc::tmem_alloc(tslot, 512);
  // Rows of the Q tiles that no token fills stay zero, and with them their scores and (overlaid) probabilities: the
  // MMAs of a decode step, 8 rows of 128 in use, then burn less power, which is what the clocks hang on.
  const uint32_t rows_q = static_cast<uint32_t>(g.tpt * g.G);
  for (int i = tid; i < S::kQTiles * S::kQc * (kTile - static_cast<int>(rows_q)) * 8; i += kThreads) {
    const int per = (kTile - static_cast<int>(rows_q)) * 8, c = i / per;
    *reinterpret_cast<uint4*>(Qs + c * (kTile * 128) + rows_q * 128 + (i - c * per) * 16) = make_uint4(0, 0, 0, 0);
  }
  tc::fence_async_smem();
  pdl_wait();
  const gqa::Share share = gqa::find_share<gqa::Blocks>(g, blockIdx.x, gridDim.x, scratch);
  Walk w;
  bool more = w.begin(g, share);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tslot;

  if (warp == 8) {
    regs_down();
    // ===================== TMA producer =====================
    bool healthy = true;
    int items = 0, tk = 0, tv = 0, q_loads[2] = {0, 0};
    for (; more && healthy; more = w.next(g), ++items) {
      // a tile's 128 rows: one box (prompts), or one box per page and 64-channel block
      const int live = PAGED ? (w.q.L + p.page - 1) / p.page : 0;
      const int ppt = PAGED ? kTile / p.page : 1;
      auto page_row = [&](int j, int pg) -> int {  // first pool row of page pg of tile j
        const int at = j * ppt + pg;
        if (at >= live) return static_cast<int>(p.kv_rows);  // past the pool: filled with zeros
        const int id = __ldg(p.block_table + static_cast<int64_t>(w.s) * p.max_pages + at);
        if (id < 0 || id >= p.n_pages) return static_cast<int>(p.kv_rows);
        return (id * g.Hkv + w.h) * p.page;
      };
      auto load_tile = [&](bool is_v, int j, int row) {
        const int chunks = is_v ? S::kVc : S::kQc;
        const int st = is_v ? tv % S::kVStages : tk % S::kKStages;
        const int use = is_v ? tv / S::kVStages : tk / S::kKStages;
        uint64_t* full = is_v ? &vfull[st] : &kfull[st];
        uint64_t* empty = is_v ? &vempty[st] : &kempty[st];
        uint8_t* dst = is_v ? Vs + st * S::kVBytes : Ks + st * S::kQBytes;
        if (use > 0 && !wait_warp(empty, (use - 1) & 1)) return false;
        if (lane == 0) tc::bar_arrive_expect_tx(full, static_cast<uint32_t>(is_v ? S::kVBytes : S::kQBytes));
        __syncwarp();
        if constexpr (PAGED) {
          // at most 3 column blocks x 8 pages: a lane each
          const int pg = lane % ppt, c = lane / ppt;
          const int r = __shfl_sync(0xffffffffu, row, pg);
          if (c < chunks) tc::tma_load_2d(dst + c * (kTile * 128) + pg * p.page * 128, is_v ? &vmap : &kmap, c * 64, r, full);
          __syncwarp();
        } else if (lane == 0) {
          for (int c = 0; c < chunks; ++c)
            tc::tma_load_3d(dst + c * (kTile * 128), is_v ? &vmap : &kmap, c * 64, w.h,
                            w.q.row0 + j * kTile, full);
        }
        if (is_v) ++tv; else ++tk;
        return true;
      };
      // K runs one tile ahead of V, as the products use them; an item's first K tile does not wait for the
      // item before to be done with its queries
      int row_cur = PAGED && lane < ppt ? page_row(w.t0, lane) : 0;
      healthy = load_tile(false, w.t0, row_cur);
      if (!healthy) break;
      // queries: one or two tiles
      if (items > 0) {
        healthy = wait_warp(&qempty[0], (items - 1) & 1) && wait_warp(&qempty[1], (items - 1) & 1);
        if (!healthy) break;
      }
      ++q_loads[0];
      q_loads[1] += w.one ? 0 : 1;
      if (lane == 0) {
        const int nt = w.one ? 1 : 2;
        for (int s = 0; s < nt; ++s) {
          tc::bar_arrive_expect_tx(&qfull[s], rows_q * 128u * S::kQc);
          const int tok = w.q.row0 + w.blk * g.tpb + s * g.tpt;
          for (int c = 0; c < S::kQc; ++c)
            tc::tma_load_3d(Qs + s * S::kQBytes + c * (kTile * 128), &qmap, c * 64, w.h * g.G, tok, &qfull[s]);
        }
      }
      __syncwarp();
      for (int j = w.t0; j < w.t1 && healthy; ++j) {
        int row_next = row_cur;
        if (j + 1 < w.t1) {
          if (PAGED && lane < ppt) row_next = page_row(j + 1, lane);
          healthy = load_tile(false, j + 1, row_next);
        }
        if (healthy) healthy = load_tile(true, j, row_cur);
        row_cur = row_next;
      }
    }
    if (!healthy) {
      await_copies(kfull, S::kKStages, tk);
      await_copies(vfull, S::kVStages, tv);
      await_copies(&qfull[0], 1, q_loads[0]);
      await_copies(&qfull[1], 1, q_loads[1]);
    }
  } else if (warp == 9 || warp == 10) {
    regs_down();
    // ===================== MMA issue (a warp per stream walks, one lane issues) =====================
    // The operands of an MMA are uniform registers: the warp stays converged and descriptors advance by constants.
    constexpr uint32_t id_qk = tc::idesc_bf16(kTile, kTile, false, false);
    constexpr uint32_t id_pv = tc::idesc_bf16(kTile, DV, true, false);
    const int s = __shfl_sync(0xffffffffu, warp - 9, 0);
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    const uint32_t tS = tm + s * kTile, tO = tm + 2 * kTile + s * DV;
    const uint64_t q_desc = tc::desc_sw128(smem_u32(Qs), 16, 1024), k_desc = tc::desc_sw128(smem_u32(Ks), 16, 1024);
    const uint64_t v_desc = tc::desc_sw128(smem_u32(Vs), kTile * 128, 1024);
    bool healthy = true;
    int items = 0, pairs = 0;
    int base = 0;             // this CTA's tiles before the item
    int parts = 0;            // items the stream took part in
    uint32_t parity = 0;      // of pfull[s][half], a bit each
    for (; more && healthy; more = w.next(g), ++items) {
      const bool one = w.one;
      const int t0 = w.t0, t1 = w.t1;
      const int ks = stream_keys(g, w, s);
      // its queries: tile s, or the one tile there is
      healthy = wait_warp(&qfull[0], items & 1);
      if (s == 1 && !one) healthy = healthy && wait_warp(&qfull[1], pairs & 1);
      pairs += one ? 0 : 1;
      const uint64_t qd = q_desc + (one ? 0 : __shfl_sync(0xffffffffu, s * (S::kQBytes >> 4), 0));
      const int ahead = one ? 2 : 1;  // tiles to the stream's next
      bool fresh = true;  // no product yet
      // Every tile's stages are given back by both streams, each after the tile has arrived (and, where it uses it, when
      // its products are complete); with the last K tile, the queries too.
      // First the stream's first scores (its own of tile t0, or of t0 and t0 + 1), then tile by tile the products of
      // tile j, the last one followed at once by the scores of the stream's next tile jn.
      for (int j = t0 - ahead; j < t1 && healthy; ++j) {
        const int jn = j + ahead;
        const int t = base + j - t0, tn = t + ahead;
        const int sv = j >= t0 ? t % S::kVStages : 0, sk = tn % S::kKStages;
        const int c = j >= t0 ? steps_of(one, s, j, ks) : 0;
        const bool next = jn < t1, mine = next && steps_of(one, s, jn, ks) > 0;
        const uint64_t kd = k_desc + __shfl_sync(0xffffffffu, sk * (S::kQBytes >> 4), 0);
        const uint64_t vd = v_desc + __shfl_sync(0xffffffffu, sv * (S::kVBytes >> 4), 0);
        if (j >= t0) healthy = wait_warp(&vfull[sv], (t / S::kVStages) & 1);
        bar_arrive_if(&vland[s], lane == 0 && c > 0 && clears_tail(j, w.q.L));
        if (c > 0 && fresh && parts > 0) healthy = healthy && wait_warp(&oempty[s], (parts - 1) & 1);
        if (c == 2) {
          healthy = healthy && wait_warp(&pfull[2 * s], parity & 1u);
          parity ^= 1u;
          tc::fence_after_sync();
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < kStep / 16; ++k)
              mma_bf16_ts(tO, tS + k * 8, vd + k * (2048 >> 4), id_pv, k == 0 ? (fresh ? 0u : 1u) : 1u);
          }
          __syncwarp();
          fresh = false;
        }
        if (next) healthy = healthy && wait_warp(&kfull[sk], (tn / S::kKStages) & 1);
        if (c > 0) healthy = healthy && wait_warp(&pfull[2 * s + c - 1], (parity >> (c - 1)) & 1u);
        if (!healthy) break;
        if (c > 0) parity ^= 1u << (c - 1);
        const uint64_t vh = vd + (c == 2 ? kStep * 128 >> 4 : 0);
        const uint32_t tP = tS + (c == 2 ? kStep / 2 : 0), add = fresh ? 0u : 1u;
        if (c > 0) await_turn(&busy[s ^ 1]);
        tc::fence_after_sync();
        if (elect_one()) {
          set_turn(&busy[s], 1);
          if (c > 0) {
#pragma unroll
            for (int k = 0; k < kStep / 16; ++k) mma_bf16_ts(tO, tP + k * 8, vh + k * (2048 >> 4), id_pv, k == 0 ? add : 1u);
          }
          if (mine) {
#pragma unroll
            for (int k = 0; k < DQK / 16; ++k) {
              const uint32_t o = ((k >> 2) * (kTile * 128) + (k & 3) * 32) >> 4;  // descriptors count 16-byte units
              tc::mma_bf16_ss(tS, qd + o, kd + o, id_qk, k != 0 ? 1u : 0u);
            }
            tc::mma_commit(&sfull[s]);
          }
          set_turn(&busy[s], 0);
          if (c > 0) tc::mma_commit(&odone[s]);
          if (j >= t0) tc::mma_commit(&vempty[sv]);
          if (next) tc::mma_commit(&kempty[sk]);
          if (jn == t1 - 1) {
            tc::mma_commit(&qempty[0]);
            tc::mma_commit(&qempty[1]);
          }
        }
        __syncwarp();
        if (c > 0) fresh = false;
      }
      parts += takes_part(one, s, t0, t1, ks) ? 1 : 0;
      base += t1 - t0;
    }
  } else if (warp == 11) {
    regs_down();
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kSoftmaxRegs));
    // ===================== softmax, thread = row =====================
    const int s = warp >> 2;                 // stream
    const int r = (warp & 3) * 32 + lane;    // row of the tile = TMEM lane
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lane_base + s * kTile, tO = tmem + lane_base + 2 * kTile;
    const int rt = r / g.G, rg = r - rt * g.G;  // token of the tile, head of the group
    const bool row_used = rt < g.tpt;
    const float sl2 = p.scale_log2;
    const float step = kRescaleLog2 / sl2;
    uint32_t limit = tc::kWaitLimit;  // 1 once a wait has run out: the rest only keeps the barriers in step
    int items = 0, base = 0;
    int ns = 0;     // this stream's tiles so far
    int tails = 0;  // those whose V it cleared behind the sequence's end
    int flags = 0;
    for (; more; more = w.next(g), ++items) {
      const bool one = w.one;
      const int off = w.q.L - w.q.nq;
      const int ks = stream_keys(g, w, s);
      const int tok = w.blk * g.tpb + (one ? 0 : s * g.tpt) + rt;
      const bool valid = row_used && tok < w.q.nq;
      // keys this row sees; a row that is not one is left unmasked (nobody reads its result)
      const int lim = valid ? off + tok + 1 : 0x7fffffff;
      const bool warp_valid = __any_sync(0xffffffffu, valid);
      float m = -INFINITY, l = 0.f;
      bool any = false;  // a tile done
      bool far = false;  // a row's reference is far out
      for (int j = w.t0; j < w.t1; ++j) {
        const int halves = steps_of(one, s, j, ks);
        if (halves == 0) continue;
        if (!wait_warp(&sfull[s], ns & 1, limit)) limit = 1;
        tc::fence_after_sync();
        float ref = 0.f;
        const int vis = lim - j * kTile;
        const bool masked = __any_sync(0xffffffffu, vis < kTile);
        if (warp_valid) {
          float mt = -INFINITY;
#pragma unroll 1
          for (int hh = 0; hh < halves; ++hh) {
            float v[kStep];
            load_scores(v, tS + hh * kStep, masked, vis - hh * kStep);
            float x0 = max3(v[0], v[1], v[2]), x1 = max3(v[3], v[4], v[5]), x2 = max3(v[6], v[7], v[8]),
                  x3 = max3(v[9], v[10], v[11]);
#pragma unroll
            for (int i = 12; i + 8 <= kStep; i += 8) {
              x0 = max3(x0, v[i], v[i + 1]);
              x1 = max3(x1, v[i + 2], v[i + 3]);
              x2 = max3(x2, v[i + 4], v[i + 5]);
              x3 = max3(x3, v[i + 6], v[i + 7]);
            }
            x0 = max3(x0, v[kStep - 4], v[kStep - 3]);
            x1 = max3(x1, v[kStep - 2], v[kStep - 1]);
            mt = max3(mt, fmaxf(x0, x1), fmaxf(x2, x3));
          }
          const bool need = valid && mt > m + step;
          if (__any_sync(0xffffffffu, need)) {
            // O and l of the rows that need it move to the new reference (from none: by 0); the previous product is
            // complete, since these scores were issued after it
            const float f = need ? exp2_approx((m - mt) * sl2) : 1.f;
            if (need) m = mt;
            far = __any_sync(0xffffffffu, m != -INFINITY && fabsf(m) * sl2 > kFarLog2);
            l *= f;
            if (any) {
#pragma unroll 1
              for (int c = 0; c < DV / 16; ++c) {
                float o[16];
                tmem_ld16(tO + s * DV + 16 * c, o);
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] *= f;
                tmem_st16(tO + s * DV + 16 * c, o);
              }
            }
          }
          ref = m == -INFINITY ? 0.f : -m * sl2;
          if (far) {  // in TMEM, where they are read again: the way of ordinary rows stays as it is
            const float at = m == -INFINITY ? 0.f : m;
            ref = 0.f;
#pragma unroll 1
            for (int c = 0; c < halves * kStep; c += 16) {
              float x[16];
              tmem_ld16(tS + c, x);
#pragma unroll
              for (int i = 0; i < 16; ++i) x[i] -= at;
              tmem_st16(tS + c, x);
            }
            tc::tmem_wait_st();
          }
        }
        // keys past the sequence's end share its last tile: their values may be anything (another sequence,
        // a page never written), and 0 x NaN is NaN, so those rows of V become zeros.  The MMA warp, which
        // waits for every V tile in turn, says when this one is there.
        if (clears_tail(j, w.q.L)) {
          if (!wait_warp(&vland[s], tails & 1, limit)) limit = 1;
          ++tails;
          const int from = max(w.q.L - j * kTile, 0), n = (kTile - from) * 8;  // 16-byte pieces per column block
          uint8_t* vb = Vs + (base + j - w.t0) % S::kVStages * S::kVBytes + from * 128;
#pragma unroll
          for (int c = 0; c < S::kVc; ++c)
            for (int i = r; i < n; i += kWgThreads)
              *reinterpret_cast<uint4*>(vb + c * (kTile * 128) + i * 16) = make_uint4(0, 0, 0, 0);
          tc::fence_async_smem();
        }
#pragma unroll 1
        for (int hh = 0; hh < halves; ++hh) {
          if (warp_valid) {
            float v[kStep];
            load_scores(v, tS + hh * kStep, masked, vis - hh * kStep);
            constexpr int kPairs = fp32_pairs(DQK, SINGLE);
            // a masked tile's -inf needs an exact 0, which only the exponential unit gives
            if (kPairs == 0 || masked)
              l += probabilities<0>(v, sl2, ref, tS + hh * (kStep / 2));
            else
              l += probabilities<kPairs>(v, sl2, ref, tS + hh * (kStep / 2));
            tc::tmem_wait_st();
          }
          tc::fence_before_sync();
          __syncwarp();
          bar_arrive_if(&pfull[2 * s + hh], lane == 0);
        }
        ++ns;
        any = true;
      }
      // ---- epilogue ----
      if (items == 0) {
        if (tid == 0) *reinterpret_cast<int3*>(&p.meta[blockIdx.x].y) = make_int3(w.s, w.h, w.blk);
        if (w.t0 > 0 && w.t1 == w.n) flags |= kMetaOwner;
      }
      flags = (flags & kMetaOwner) | (w.t0 == 0 ? kMetaBegins : 0) | (items == 0 ? kMetaSingle : 0);
      if (any) {
        if (!wait_warp(&odone[s], (ns - 1) & 1, limit)) limit = 1;
        tc::fence_after_sync();
      }
      float mr = m == -INFINITY ? -INFINITY : m * sl2;  // log2 units
      float fa = mr != -INFINITY ? 1.f : 0.f, fb = 0.f;
      if (one) {
        if (s == 1) stat[r] = make_float2(mr, l);
        tc::fence_before_sync();
        named_sync(1, 2 * kWgThreads);
        tc::fence_after_sync();
        const float2 other = stat[r];
        named_sync(2, 2 * kWgThreads);  // stream 1 may write the next item's
        if (s == 0) {
          const float top = fmaxf(mr, other.x);
          const float ref = top == -INFINITY ? 0.f : top;
          fa = mr == -INFINITY ? 0.f : exp2f(mr - ref);
          fb = other.x == -INFINITY ? 0.f : exp2f(other.x - ref);
          l = l * fa + other.y * fb;
          mr = top;
        }
      }
      if (!(one && s == 1)) {
        const bool whole = w.whole();
        const float inv = whole ? (l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l)) : 1.f;  // NaN stays NaN
        const int64_t grow = static_cast<int64_t>(w.q.row0 + tok) * p.Hq + w.h * g.G + rg;
        const int64_t prow = (static_cast<int64_t>(2) * blockIdx.x + (items > 0 ? 1 : 0)) * S::kRows + s * kTile + r;
        const bool mine = valid && CSA_INBOUNDS(whole ? grow >= 0 && grow < g.total_q * p.Hq
                                                      : prow >= 0 && prow < static_cast<int64_t>(2) * gridDim.x * S::kRows);
        fa *= inv;
        fb *= inv;
        const bool any_a = __any_sync(0xffffffffu, valid && fa != 0.f), any_b = __any_sync(0xffffffffu, valid && fb != 0.f);
#pragma unroll 1
        for (int col = 0; col < DV; col += 16) {
          float o[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) o[i] = 0.f;
          if (any_a) {
            tmem_ld16(tO + s * DV + col, o);
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = fa != 0.f ? o[i] * fa : 0.f;
          }
          if (any_b) {
            float o2[16];
            tmem_ld16(tO + DV + col, o2);
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] += fb != 0.f ? o2[i] * fb : 0.f;
          }
          if (mine) {
            if (whole) {
              uint32_t u[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) u[i] = pack_bf16x2(o[2 * i], o[2 * i + 1]);
              st_global_32(p.out + grow * DV + col, u, p.wide);
            } else {
              float* dst = p.part + prow * DV + col;
              st_global_32(dst, reinterpret_cast<const uint32_t*>(o), p.wide);
              st_global_32(dst + 8, reinterpret_cast<const uint32_t*>(o + 8), p.wide);
            }
          }
        }
        if (mine) {
          if (whole) {
            if (p.lse != nullptr) p.lse[grow] = l == 0.f ? -INFINITY : (mr + log2f(l)) * kLn2;
          } else {
            p.ml[prow] = make_float2(mr, l);
          }
        }
        tc::fence_before_sync();
        // the next item in which a stream takes part may overwrite its O
        bar_arrive_if(&oempty[s], any);
        bar_arrive_if(&oempty[1], one && takes_part(true, 1, w.t0, w.t1, ks));
      }
      base += w.t1 - w.t0;
    }
    if (tid == 0) p.meta[blockIdx.x].x = flags;
    pdl_trigger();  // only the merge is left
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 9) tc::tmem_dealloc(tmem, 512);
}

// Joins the partial states of items that straddle CTAs.  Block (c, y): the
// item that CTA c's first piece ends, rows y*8 .. y*8+7, a warp per row.  The
// pieces are CTA c's first, every whole CTA before it, and the last piece of
// the CTA in which the item begins; they are added in that fixed order.
template <int DV, int ROWS>
__global__ void __launch_bounds__(256) gqa_merge_kernel(const __grid_constant__ Params p) {
  pdl_wait();
  const int c = blockIdx.x, lane = threadIdx.x & 31;
  // every load that needs no other is made first: lane i holds what CTA c - i left
  int4 info = p.meta[max(c - lane, 0)];
  const int flags = __shfl_sync(0xffffffffu, info.x, 0);
  if (!(flags & kMetaOwner)) return;
  const int s = __shfl_sync(0xffffffffu, info.y, 0), h = __shfl_sync(0xffffffffu, info.z, 0);
  const int blk = __shfl_sync(0xffffffffu, info.w, 0);
  const int row = blockIdx.y * 8 + (threadIdx.x >> 5);
  const int tile = row / kTile, r = row % kTile;
  const int rt = r / p.g.G, rg = r - rt * p.g.G;
  Seq q;
  q.load(p.g, s);
  const int tok = blk * p.g.tpb + tile * p.g.tpt + rt;
  if (rt >= p.g.tpt || tok >= q.nq) return;
  float top = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  // pieces c, c - 1, ... down to the nearest CTA below c whose last piece begins the item, 32 at a time
  for (int i0 = 0;; i0 += 32) {
    const int i = i0 + lane, from = c - i;
    if (i0 > 0) info = p.meta[max(from, 0)];
    const uint32_t begins = __ballot_sync(0xffffffffu, i > 0 && (from <= 0 || (info.x & kMetaBegins)));
    const int n = begins ? __ffs(begins) : 32;  // pieces here
    const int second = (i > 0 && !(info.x & kMetaSingle)) ? 1 : 0;
    int64_t slot = (static_cast<int64_t>(2) * max(from, 0) + second) * ROWS + row;
    const bool held = lane < n && CSA_INBOUNDS(from >= 0 && slot < static_cast<int64_t>(2) * gridDim.x * ROWS);
    if (!held) slot = 0;
    const float2 ml = held ? p.ml[slot] : make_float2(-INFINITY, 0.f);
    const float now = fmaxf(top, warp_max(ml.x)), ref = now == -INFINITY ? 0.f : now;
    const float old = top == -INFINITY ? 0.f : exp2f(top - ref);
    const float wgt = ml.x == -INFINITY ? 0.f : exp2f(ml.x - ref);
    top = now;
    l *= old;
    acc.x *= old;
    acc.y *= old;
    acc.z *= old;
    acc.w *= old;
    const float li = ml.y * wgt;
#pragma unroll 4
    for (int u = 0; u < n; ++u) {
      const int64_t at = __shfl_sync(0xffffffffu, slot, u);
      // (a piece without a key of this row holds zeros)
      const float4 o = lane < DV / 4 ? *reinterpret_cast<const float4*>(p.part + at * DV + 4 * lane)
                                     : make_float4(0.f, 0.f, 0.f, 0.f);
      const float wi = __shfl_sync(0xffffffffu, wgt, u);
      l += __shfl_sync(0xffffffffu, li, u);
      acc.x += o.x * wi;
      acc.y += o.y * wi;
      acc.z += o.z * wi;
      acc.w += o.w * wi;
    }
    if (begins) break;
  }
  const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
  const int64_t grow = static_cast<int64_t>(q.row0 + tok) * p.Hq + h * p.g.G + rg;
  if (!CSA_INBOUNDS(grow >= 0 && grow < p.g.total_q * p.Hq)) return;
  if (lane < DV / 4)
    *reinterpret_cast<uint2*>(p.out + grow * DV + 4 * lane) =
        make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
  if (lane == 0 && p.lse != nullptr) p.lse[grow] = l == 0.f ? -INFINITY : (top + log2f(l)) * kLn2;
}

struct Workspace {
  size_t part, ml, meta, bytes;
};
Workspace layout(int64_t max_rows, int dv) {
  const int rows = max_rows <= kTile ? kTile : 2 * kTile;
  const size_t slots = static_cast<size_t>(2) * num_sms() * rows;
  Workspace w;
  w.part = 0;
  w.ml = slots * dv * 4;
  w.meta = w.ml + slots * 8;
  w.bytes = w.meta + static_cast<size_t>(num_sms()) * 16;
  return w;
}

template <int DQK, int DV, bool PAGED, bool SINGLE>
csa_status launch(const char* what, const Params& p, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                  int64_t max_rows, cudaStream_t s) {
  using S = Shape<DQK, DV, SINGLE>;
  auto kern = gqa_attn_kernel<DQK, DV, PAGED, SINGLE>;
  if (!ensure_smem(reinterpret_cast<const void*>(kern), static_cast<int>(S::kSmem)))
    return fail(CSA_ERR_CUDA, "%s: cannot raise the shared memory limit", what);
  const int grid = num_sms();
  prof_begin(s);
  cudaError_t e = launch_pdl(kern, dim3(grid), dim3(kThreads), S::kSmem, s, 1, p, q, k, v);
  prof_end(s);
  if (csa_status st = check_launch(what, e); st != CSA_OK) return st;
  const int64_t rows = max_rows < S::kRows ? max_rows : S::kRows;
  // rows of a second tile start at 128 whatever the first tile's unused rows are
  const int used = rows <= kTile ? static_cast<int>(rows) : S::kRows;
  e = launch_pdl(gqa_merge_kernel<DV, S::kRows>, dim3(grid, (used + 7) / 8), dim3(256), 0, s, 1, p);
  return check_launch(what, e);
}

template <bool PAGED>
csa_status dispatch(const char* what, Params& p, const gqa::Heads& h, const CUtensorMap& q, const CUtensorMap& k,
                    const CUtensorMap& v, int64_t max_rows, cudaStream_t s) {
  const bool single = max_rows <= kTile;
  p.g.tpb = p.g.tpt * (single ? 1 : 2);
#define CSA_GQA_CASE(A, B)                                                                       \
  if (h.dqk == A && h.dv == B)                                                                   \
    return single ? launch<A, B, PAGED, true>(what, p, q, k, v, max_rows, s)                     \
                  : launch<A, B, PAGED, false>(what, p, q, k, v, max_rows, s);
  CSA_GQA_CASE(192, 128)
  CSA_GQA_CASE(128, 128)
  CSA_GQA_CASE(64, 64)
#undef CSA_GQA_CASE
  return fail(CSA_ERR_UNSUPPORTED, "%s: channel widths %d/%d", what, h.dqk, h.dv);
}

// Tokens of a row tile: what 128 rows hold, or a sequence brings.
int tokens_per_tile(int G, int64_t max_q) { return static_cast<int>(kTile / G < max_q ? kTile / G : max_q); }

// No item of any sequence has more rows than this.
int64_t rows_bound(int64_t max_q, int64_t G) { return max_q > 2 * kTile ? 2 * kTile : (max_q * G > 2 * kTile ? 2 * kTile : max_q * G); }

csa_status check_workspace(const char* what, int64_t max_q, const gqa::Heads& h, const void* workspace, size_t bytes) {
  const size_t need = layout(rows_bound(max_q, h.G), h.dv).bytes;
  if (workspace == nullptr || bytes < need)
    return fail(CSA_ERR_WORKSPACE, "%s: workspace of %zu bytes needed, %zu given", what, need,
                workspace == nullptr ? static_cast<size_t>(0) : bytes);
  CSA_REQUIRE(aligned16(workspace), "%s: workspace is not 16-byte aligned", what);
  return CSA_OK;
}

csa_status run(const char* what, bool paged, Params& p, const gqa::Heads& h, const CUtensorMap& q, const CUtensorMap& k,
               const CUtensorMap& v, int64_t max_q, float scale, void* out, float* lse, void* workspace,
               cudaStream_t s) {
  const int64_t max_rows = rows_bound(max_q, h.G);
  const Workspace w = layout(max_rows, h.dv);
  p.Hq = h.Hkv * h.G;
  p.scale_log2 = scale * kLog2e;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.wide = ((reinterpret_cast<uintptr_t>(out) | reinterpret_cast<uintptr_t>(workspace)) & 31u) == 0;
  p.lse = lse;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.part = reinterpret_cast<float*>(ws + w.part);
  p.ml = reinterpret_cast<float2*>(ws + w.ml);
  p.meta = reinterpret_cast<int4*>(ws + w.meta);
  return paged ? dispatch<true>(what, p, h, q, k, v, max_rows, s) : dispatch<false>(what, p, h, q, k, v, max_rows, s);
}

}  // namespace
}  // namespace csa

extern "C" {

size_t gqa_dense_workspace_size(int64_t max_q, int32_t H, int32_t H_kv, int32_t d_v) {
  if (max_q <= 0 || H_kv <= 0 || H < H_kv || d_v <= 0) return 0;
  return csa::layout(csa::rows_bound(max_q, H / H_kv), d_v).bytes;
}

csa_status gqa_dense_packed(const void* q, const void* k, const void* v, const csa_packed* packed, int32_t H,
                            int32_t H_kv, int32_t d_qk, int32_t d_v, float scale, void* out, float* lse,
                            void* workspace, size_t workspace_bytes, void* stream) {
  using namespace csa;
  const char* what = "gqa_dense_packed";
  clear_error();
  CSA_REQUIRE(packed != nullptr, "%s: packed is NULL", what);
  gqa::Heads h;
  if (csa_status st = gqa::check_heads(what, H, H_kv, d_qk, d_v, &h); st != CSA_OK) return st;
  if (csa_status st = gqa::check_scale(what, scale); st != CSA_OK) return st;
  CSA_REQUIRE(packed->n_seqs >= 0 && packed->max_tokens >= 0, "%s: negative sizes", what);
  CSA_REQUIRE(packed->total_tokens >= 0 && packed->total_tokens < (int64_t(1) << 31),
              "%s: total_tokens must be in [0, 2^31)", what);
  CSA_REQUIRE(packed->max_tokens <= packed->total_tokens, "%s: max_tokens is larger than total_tokens", what);
  if (packed->n_seqs == 0 || packed->total_tokens == 0) return CSA_OK;
  CSA_REQUIRE(packed->max_tokens >= 1, "%s: max_tokens is 0 but there are tokens", what);
  CSA_REQUIRE_PTR(q);
  CSA_REQUIRE_PTR(k);
  CSA_REQUIRE_PTR(v);
  CSA_REQUIRE_PTR(out);
  CSA_REQUIRE_PTR(packed->cu_tokens);
  CSA_REQUIRE(lse == nullptr || aligned16(lse), "%s: lse is not 16-byte aligned", what);
  if (csa_status st = check_workspace(what, packed->max_tokens, h, workspace, workspace_bytes); st != CSA_OK) return st;
  Params p;
  memset(&p, 0, sizeof(p));
  p.g.cu_q = packed->cu_tokens;
  p.g.cache_len = nullptr;
  p.g.n_seqs = packed->n_seqs;
  p.g.max_len = 0x7fffffff;
  p.g.total_q = packed->total_tokens;
  p.g.Hkv = h.Hkv;
  p.g.G = h.G;
  p.g.tpt = tokens_per_tile(h.G, packed->max_tokens);
  p.page = kTile;
  CUtensorMap qm, km, vm;
  const uint64_t rows = static_cast<uint64_t>(packed->total_tokens);
  csa_status st = gqa::map_tokens(what, &qm, q, h.dqk, H, rows, h.G, p.g.tpt);
  if (st == CSA_OK) st = gqa::map_tokens(what, &km, k, h.dqk, H_kv, rows, 1, kTile);
  if (st == CSA_OK) st = gqa::map_tokens(what, &vm, v, h.dv, H_kv, rows, 1, kTile);
  if (st != CSA_OK) return st;
  return run(what, false, p, h, qm, km, vm, packed->max_tokens, scale, out, lse, workspace,
             static_cast<cudaStream_t>(stream));
}

csa_status gqa_dense_paged(const void* q, const gqa_cache* cache, const gqa_batch* batch, int32_t H, float scale,
                           void* out, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  using namespace csa;
  const char* what = "gqa_dense_paged";
  clear_error();
  gqa::Heads h;
  if (csa_status st = gqa::check_paged(what, cache, batch, H, &h); st != CSA_OK) return st;
  if (csa_status st = gqa::check_scale(what, scale); st != CSA_OK) return st;
  if (batch->n_seqs == 0 || batch->total_q == 0) return CSA_OK;
  if (csa_status st = gqa::check_pool(what, cache, batch, true); st != CSA_OK) return st;
  CSA_REQUIRE_PTR(q);
  CSA_REQUIRE_PTR(out);
  CSA_REQUIRE(lse == nullptr || aligned16(lse), "%s: lse is not 16-byte aligned", what);
  if (csa_status st = check_workspace(what, batch->max_q, h, workspace, workspace_bytes); st != CSA_OK) return st;
  Params p;
  memset(&p, 0, sizeof(p));
  p.g.cu_q = batch->cu_q;
  p.g.cache_len = batch->cache_len;
  p.g.n_seqs = batch->n_seqs;
  p.g.max_len = gqa::max_len(cache, batch);
  p.g.total_q = batch->total_q;
  p.g.Hkv = h.Hkv;
  p.g.G = h.G;
  p.g.tpt = tokens_per_tile(h.G, batch->max_q);
  p.block_table = batch->block_table;
  p.max_pages = batch->max_pages;
  p.page = cache->page_size;
  p.n_pages = static_cast<int>(cache->n_pages);
  p.kv_rows = cache->n_pages * h.Hkv * cache->page_size;
  CUtensorMap qm, km, vm;
  csa_status st = gqa::map_tokens(what, &qm, q, h.dqk, H, static_cast<uint64_t>(batch->total_q), h.G, p.g.tpt);
  if (st == CSA_OK) st = gqa::map_rows(what, &km, cache->k, h.dqk, static_cast<uint64_t>(p.kv_rows), cache->page_size);
  if (st == CSA_OK) st = gqa::map_rows(what, &vm, cache->v, h.dv, static_cast<uint64_t>(p.kv_rows), cache->page_size);
  if (st != CSA_OK) return st;
  return run(what, true, p, h, qm, km, vm, batch->max_q, scale, out, lse, workspace,
             static_cast<cudaStream_t>(stream));
}

}  // extern "C"

namespace csa {
// Reads (and optionally clears) this unit's device error word.
CSA_DEFINE_DEVICE_ERROR_READER(gqa_device_error)
}  // namespace csa
