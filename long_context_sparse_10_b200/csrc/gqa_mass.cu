// Accumulated attention weight of cached tokens (grouped heads, paged cache):
//     mass[h, j] += sum over the rows i that see token j, and the G heads of
//                   kv head h, of exp(scale q[i, hG+g] . k[j, h] - lse[i, hG+g])
//
// The scores are computed transposed, S^T = K Q^T with 128 keys as the MMA's
// rows and up to 128 packed rows (token, head of the group) as its columns: a
// thread then owns a key and adds up its columns by itself, in a fixed order,
// without exchanging anything.  An item is a pair of key tiles of one
// (sequence, kv head); it walks over the row blocks that see it, each Q block
// serving both tiles.  gqa_work.cuh shares the items out by their cost.
//
// Bound: one new token per sequence reads K once (HBM; 16 sequences of 1500 to
// 16384 tokens, 302 MB: 54 us on the device, 0.85 of the measured copy
// bandwidth); many rows cost one exponential per (key, row), which the
// exponential unit gives at 16 a clock and SM (whole prompts of 4096 and 1500
// tokens, 32 heads: 212 us where the exponentials alone take 68).
//
// Roles of a CTA (one per SM, 320 threads): warps 0-3 and 4-7 take the two key
// tiles (two score buffers of 128 TMEM columns each), warp 8 loads by TMA, warp
// 9 issues the MMAs.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "gqa_device.cuh"
#include "gqa_host.h"
#include "gqa_work.cuh"

namespace csa {
namespace {

using namespace gqa;

constexpr int kThreads = 320;

struct MassParams {
  Pool c;
  Geometry g;  // tpb = tpt
  const float* lse;
  const int32_t* block_table;
  int max_pages;
  int64_t kv_rows;
  float scale_log2;
  int cols;              // columns of a Q block: tpt * G rounded up to 16
  int k_stages, q_stages;
};

template <int DQK>
struct MassShape {
  static constexpr int kChunks = DQK / 64;
  static constexpr int kKBytes = kTile * DQK * 2;
  static constexpr int kMaxStages = 8;
  // barriers | TMEM slot | row constants [tile][buffer][column] (first the partition's scratch); at the front, the
  // rings behind it on 1024-byte boundaries
  static constexpr int kBars = 4 * kMaxStages + 8;
  static constexpr int kConstOff = 8 * kBars + 16;
  static constexpr int kFront = ((kConstOff + 4 * kTile * 4 + 1023) / 1024) * 1024;
  static constexpr int kBudget = 232448 - 768 - kFront;  // bytes for the rings
};

// A ring of stages: the stage now, and the parity of its barriers' phase.
struct Ring {
  int st = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ void step(int n) {
    if (++st == n) {
      st = 0;
      ph ^= 1u;
    }
  }
};

template <int DQK>
__global__ void __launch_bounds__(kThreads, 1)
    gqa_mass_kernel(const __grid_constant__ MassParams p, const __grid_constant__ CUtensorMap qmap,
                    const __grid_constant__ CUtensorMap kmap) {
  using S = MassShape<DQK>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* kfull = reinterpret_cast<uint64_t*>(smem);
  uint64_t* kempty = kfull + S::kMaxStages;
  uint64_t* qfull = kempty + S::kMaxStages;
  uint64_t* qempty = qfull + S::kMaxStages;
  uint64_t* sfull = qempty + S::kMaxStages;  // [tile][buffer]
  uint64_t* sempty = sfull + 4;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(sempty + 4);
  float* consts = reinterpret_cast<float*>(smem + S::kConstOff);
  uint8_t* Ks = smem + S::kFront;
  uint8_t* Qs = Ks + p.k_stages * S::kKBytes;
  const int q_bytes = p.cols * DQK * 2;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Geometry& g = p.g;

  if (tid == 0) {
    prefetch_map(&qmap);
    prefetch_map(&kmap);
    for (int i = 0; i < S::kMaxStages; ++i) {
      tc::bar_init(&kfull[i], 1);
      tc::bar_init(&kempty[i], 1);
      tc::bar_init(&qfull[i], 1);
      tc::bar_init(&qempty[i], 1);
    }
    for (int i = 0; i < 4; ++i) {
      tc::bar_init(&sfull[i], 1);
      tc::bar_init(&sempty[i], 4);
    }
    tc::bar_init_fence();
  }
  if (warp == 9) tc::tmem_alloc(tslot, 512);
  pdl_wait();  // nothing above depends on the kernel before
  const Share share = find_share<KeyPairs>(g, blockIdx.x, gridDim.x, reinterpret_cast<int64_t*>(consts));
  MassWalk w;
  bool more = w.begin(g, share);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tslot;

  if (warp == 8) {
    // ===================== TMA producer =====================
    Ring kr, qr;
    int k_loads = 0, q_loads = 0;
    bool healthy = true;
    const int ppt = kTile / p.c.page;
    for (; more && healthy; more = w.next(g)) {
      const int live = (w.q.L + p.c.page - 1) / p.c.page;
      for (int t = 0; t < 2 && healthy; ++t) {
        const int j = 2 * w.pair + t;
        if (j * kTile >= w.q.L) break;
        // pages past the sequence's end or outside the pool: past the pool's rows, filled with zeros
        int row = static_cast<int>(p.kv_rows);
        const int pg = lane % ppt, c = lane / ppt, at = j * ppt + pg;
        if (at < live) {
          const int id = __ldg(p.block_table + static_cast<int64_t>(w.s) * p.max_pages + at);
          if (id >= 0 && id < p.c.n_pages) row = (id * g.Hkv + w.h) * p.c.page;
        }
        healthy = wait_warp(&kempty[kr.st], kr.ph ^ 1u);
        if (!healthy) break;
        if (lane == 0) tc::bar_arrive_expect_tx(&kfull[kr.st], S::kKBytes);
        __syncwarp();
        if (c < S::kChunks)
          tc::tma_load_2d(Ks + kr.st * S::kKBytes + c * (kTile * 128) + pg * p.c.page * 128, &kmap, c * 64, row,
                          &kfull[kr.st]);
        __syncwarp();
        kr.step(p.k_stages);
        ++k_loads;
      }
      for (int b = KeyPairs::first_block(g, w.q, w.pair); b < w.q.nblk && healthy; ++b) {
        healthy = wait_warp(&qempty[qr.st], qr.ph ^ 1u);
        if (!healthy) break;
        if (lane == 0) {
          tc::bar_arrive_expect_tx(&qfull[qr.st], static_cast<uint32_t>(g.tpt * g.G) * 128u * S::kChunks);
          for (int c = 0; c < S::kChunks; ++c)
            tc::tma_load_3d(Qs + qr.st * q_bytes + c * p.cols * 128, &qmap, c * 64, w.h * g.G, w.q.row0 + b * g.tpb,
                            &qfull[qr.st]);
        }
        __syncwarp();
        qr.step(p.q_stages);
        ++q_loads;
      }
    }
    if (!healthy) {
      await_copies(kfull, p.k_stages, k_loads);
      await_copies(qfull, p.q_stages, q_loads);
    }
  } else if (warp == 9) {
    // ===================== MMA issue =====================
    const uint32_t idesc = tc::idesc_bf16(kTile, p.cols, false, false);
    const uint64_t k_desc = tc::desc_sw128(smem_u32(Ks), 16, 1024), q_desc = tc::desc_sw128(smem_u32(Qs), 16, 1024);
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    const uint32_t q_chunk = __shfl_sync(0xffffffffu, p.cols * 128 >> 4, 0);
    Ring kr, qr;
    uint32_t blocks[2] = {0, 0};  // score tiles issued, by key tile of the pair
    bool healthy = true;
    for (; more && healthy; more = w.next(g)) {
      Ring k0 = kr, k1 = kr;
      k1.step(p.k_stages);
      const bool two = (2 * w.pair + 1) * kTile < w.q.L;
      healthy = wait_warp(&kfull[k0.st], k0.ph) && (!two || wait_warp(&kfull[k1.st], k1.ph));
      for (int b = KeyPairs::first_block(g, w.q, w.pair); b < w.q.nblk && healthy; ++b) {
        healthy = wait_warp(&qfull[qr.st], qr.ph);
        const uint64_t bd = q_desc + __shfl_sync(0xffffffffu, qr.st * (q_bytes >> 4), 0);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (!healthy || !w.active(g, t, b)) continue;
          const int buf = blocks[t] & 1;
          healthy = wait_warp(&sempty[2 * t + buf], ((blocks[t] >> 1) & 1u) ^ 1u);
          if (!healthy) continue;
          ++blocks[t];
          tc::fence_after_sync();
          const uint64_t a = k_desc + __shfl_sync(0xffffffffu, (t ? k1.st : k0.st) * (S::kKBytes >> 4), 0);
          const uint32_t d = tm + t * 2 * kTile + __shfl_sync(0xffffffffu, buf * kTile, 0);
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < DQK / 16; ++k)
              tc::mma_bf16_ss(d, a + (((k >> 2) * (kTile * 128) + (k & 3) * 32) >> 4),
                              bd + ((k >> 2) * q_chunk + ((k & 3) * 32 >> 4)), idesc, k != 0 ? 1u : 0u);
            tc::mma_commit(&sfull[2 * t + buf]);
          }
          __syncwarp();
        }
        if (elect_one()) tc::mma_commit(&qempty[qr.st]);
        __syncwarp();
        qr.step(p.q_stages);
      }
      if (elect_one()) {
        tc::mma_commit(&kempty[k0.st]);
        if (two) tc::mma_commit(&kempty[k1.st]);
      }
      __syncwarp();
      kr.step(p.k_stages);
      if (two) kr.step(p.k_stages);
    }
  } else {
    // ===================== sums, thread = key =====================
    const int t = warp >> 2;
    const int r = tid & (kTile - 1);
    const uint32_t tB = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + t * 2 * kTile;
    float* cst = consts + t * 2 * kTile;
    const int ct = r / g.G, cg = r - ct * g.G;  // token and head of column r
    const float sl2 = p.scale_log2;
    uint32_t limit = tc::kWaitLimit;
    uint32_t blocks = 0;
    for (; more; more = w.next(g)) {
      const int k0 = (2 * w.pair + t) * kTile;
      if (k0 >= w.q.L) continue;
      const int key = k0 + r, off = w.q.L - w.q.nq;
      const int64_t at =
          key < w.q.L ? slot_of(p.c, p.block_table + static_cast<int64_t>(w.s) * p.max_pages, p.max_pages, w.h, key) : -1;
      // -lse of column r in log2 units; rows that are none, or saw nothing, add nothing
      auto constant = [&](int b) {
        const int tok = b * g.tpb + ct;
        if (b >= w.q.nblk || ct >= g.tpt || tok >= w.q.nq || !CSA_INBOUNDS(tok >= 0 && w.q.row0 + tok < g.total_q))
          return -INFINITY;
        const float l = __ldg(p.lse + (static_cast<int64_t>(w.q.row0 + tok) * g.Hkv + w.h) * g.G + cg);
        return l == -INFINITY ? -INFINITY : -l * kLog2e;
      };
      int b = KeyPairs::first_block(g, w.q, w.pair);
      while (b < w.q.nblk && !w.active(g, t, b)) ++b;
      float cur = constant(b), sum = 0.f;
      for (; b < w.q.nblk; ++b) {
        const int buf = blocks & 1;
        cst[buf * kTile + r] = cur;
        const int nc = min(g.tpb, w.q.nq - b * g.tpb) * g.G;      // columns that are rows
        named_sync(1 + t, kTile);
        cur = constant(b + 1);
        if (!wait_warp(&sfull[2 * t + buf], (blocks >> 1) & 1u, limit)) limit = 1;
        tc::fence_after_sync();
        const int from = max(key - off - b * g.tpb, 0) * g.G;     // the first that sees the key
        float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll 1
        for (int c = 0; c < nc; c += 32) {
          float v[32];
          tmem_ld32_async(tB + buf * kTile + c, v);
          const float4* cc = reinterpret_cast<const float4*>(cst + buf * kTile + c);
          const bool part = __any_sync(0xffffffffu, from > c) || c + 32 > nc;
          tc::tmem_wait_ld();
          fence_regs(v);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float4 k = cc[i];
            float* e = v + 4 * i;
            fma2v(e[0], e[1], sl2, k.x, k.y);
            fma2v(e[2], e[3], sl2, k.z, k.w);
          }
          // all on the exponential unit: the weight is summed over a sequence's life, lse is the caller's (nothing bounds
          // the exponent), and two of eight pairs on the fp32 units gain nothing (64 rows of four sequences 20.6 us, both)
          if (part) {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = (c + i >= from && c + i < nc) ? exp2_approx(v[i]) : 0.f;
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = exp2_approx(v[i]);
          }
#pragma unroll
          for (int i = 0; i < 32; i += 4) {
            add2(s0, s1, v[i], v[i + 1]);
            add2(s2, s3, v[i + 2], v[i + 3]);
          }
        }
        sum += (s0 + s1) + (s2 + s3);
        tc::fence_before_sync();
        __syncwarp();
        bar_arrive_if(&sempty[2 * t + buf], lane == 0);
        ++blocks;
      }
      // the only addition of this call to the token, unless sequences share the page: theirs come in any order
      if (at >= 0) atomicAdd(p.c.mass + at, sum);
    }
    pdl_trigger();
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 9) tc::tmem_dealloc(tmem, 512);
}

template <int DQK>
csa_status launch(const char* what, MassParams& p, const CUtensorMap& q, const CUtensorMap& k, cudaStream_t s) {
  using S = MassShape<DQK>;
  // two to four Q blocks, the rest for K (its tiles are what one token per sequence streams)
  const int qb = p.cols * DQK * 2;
  p.q_stages = 4 * qb <= S::kBudget / 4 ? 4 : 2;
  p.k_stages = (S::kBudget - p.q_stages * qb) / S::kKBytes;
  if (p.k_stages > S::kMaxStages) p.k_stages = S::kMaxStages;
  const int smem = S::kFront + p.k_stages * S::kKBytes + p.q_stages * qb + 768;
  auto kern = gqa_mass_kernel<DQK>;
  if (!ensure_smem(reinterpret_cast<const void*>(kern), smem))
    return fail(CSA_ERR_CUDA, "%s: cannot raise the shared memory limit", what);
  prof_begin(s);
  const cudaError_t e = launch_pdl(kern, dim3(num_sms()), dim3(kThreads), static_cast<size_t>(smem), s, 1, p, q, k);
  prof_end(s);
  return check_launch(what, e);
}

}  // namespace
}  // namespace csa

extern "C" {

csa_status gqa_cache_mass(const void* q, const float* lse, const gqa_cache* cache, const gqa_batch* batch, int32_t H,
                          float scale, void* stream) {
  using namespace csa;
  const char* what = "gqa_cache_mass";
  clear_error();
  gqa::Heads h;
  if (csa_status st = gqa::check_paged(what, cache, batch, H, &h); st != CSA_OK) return st;
  if (csa_status st = gqa::check_scale(what, scale); st != CSA_OK) return st;
  CSA_REQUIRE(cache->mass != nullptr, "%s: the cache has no mass plane", what);
  if (batch->n_seqs == 0 || batch->total_q == 0) return CSA_OK;
  if (csa_status st = gqa::check_pool(what, cache, batch, true); st != CSA_OK) return st;
  CSA_REQUIRE_PTR(q);
  CSA_REQUIRE_PTR(lse);
  CSA_REQUIRE_PTR(cache->mass);
  MassParams p;
  memset(&p, 0, sizeof(p));
  p.c = gqa::pool_of(cache);
  p.g.cu_q = batch->cu_q;
  p.g.cache_len = batch->cache_len;
  p.g.n_seqs = batch->n_seqs;
  p.g.max_len = gqa::max_len(cache, batch);
  p.g.total_q = batch->total_q;
  p.g.Hkv = h.Hkv;
  p.g.G = h.G;
  // as many tokens a block as 128 columns hold, or as a sequence has
  p.g.tpt = gqa::kTile / h.G < batch->max_q ? gqa::kTile / h.G : batch->max_q;
  p.g.tpb = p.g.tpt;
  p.cols = (p.g.tpt * h.G + 15) / 16 * 16;
  p.lse = lse;
  p.block_table = batch->block_table;
  p.max_pages = batch->max_pages;
  p.kv_rows = cache->n_pages * h.Hkv * cache->page_size;
  p.scale_log2 = scale * kLog2e;
  CUtensorMap qm, km;
  csa_status st = gqa::map_tokens(what, &qm, q, h.dqk, H, static_cast<uint64_t>(batch->total_q), h.G, p.g.tpt);
  if (st == CSA_OK) st = gqa::map_rows(what, &km, cache->k, h.dqk, static_cast<uint64_t>(p.kv_rows), cache->page_size);
  if (st != CSA_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (h.dqk == 192) return launch<192>(what, p, qm, km, s);
  if (h.dqk == 128) return launch<128>(what, p, qm, km, s);
  return launch<64>(what, p, qm, km, s);
}

}  // extern "C"

namespace csa {
// Reads (and optionally clears) this unit's device error word.
CSA_DEFINE_DEVICE_ERROR_READER(gqa_mass_device_error)
}  // namespace csa
