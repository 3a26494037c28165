// The paged cache of the grouped-head (GQA) attention: appending a chunk, and
// eviction by accumulated weight.
#include <cooperative_groups.h>

#include "gqa_device.cuh"
#include "gqa_host.h"

namespace csa {
namespace {

using namespace gqa;

// ---------------------------------------------------------------------------
// Append: a warp per new token copies its rows of all kv heads, 16 bytes a
// lane.  Bound by the copy (read and write of each new row once; 13192 tokens of
// 8 heads, 108 MB: 16.5 us in a replayed graph, the measured copy bandwidth, and
// 20.5 call by call).
// ---------------------------------------------------------------------------
struct AppendParams {
  Pool c;
  const uint4* k;  // [total_q, Hkv, kp]
  const uint4* v;  // [total_q, Hkv, vp]
  const int32_t* block_table;
  const int32_t* cache_len;
  const int32_t* cu_q;
  int n_seqs, max_pages;
  int total_q;
};

__global__ void __launch_bounds__(256) gqa_append_kernel(const __grid_constant__ AppendParams p) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (row >= p.total_q || row >= __ldg(p.cu_q + p.n_seqs)) return;
  const int s = seq_of(p.cu_q, p.n_seqs, row);
  if (!CSA_INBOUNDS(s >= 0 && s < p.n_seqs)) return;
  const int end = __ldg(p.cu_q + s + 1);
  const int pos = __ldg(p.cache_len + s) - end + static_cast<int>(row);
  const int64_t at = slot_of(p.c, p.block_table + static_cast<int64_t>(s) * p.max_pages, p.max_pages, 0, pos);
  if (at < 0) return;
  const int64_t step = p.c.page;  // slots between two heads of a token
  for (int i = lane; i < p.c.Hkv * p.c.kp; i += 32) {
    const int h = i / p.c.kp, x = i - h * p.c.kp;
    p.c.k[(at + h * step) * p.c.kp + x] = __ldg(p.k + row * p.c.Hkv * p.c.kp + i);
  }
  for (int i = lane; i < p.c.Hkv * p.c.vp; i += 32) {
    const int h = i / p.c.vp, x = i - h * p.c.vp;
    p.c.v[(at + h * step) * p.c.vp + x] = __ldg(p.v + row * p.c.Hkv * p.c.vp + i);
  }
  if (p.c.mass != nullptr)
    for (int h = lane; h < p.c.Hkv; h += 32) p.c.mass[at + h * step] = 0.f;
}

// ---------------------------------------------------------------------------
// Eviction.  Select: a cluster of blocks per (sequence, kv head), each with its
// run of the positions.  The order-preserving 32-bit keys of the middle tokens'
// mass are read once, into shared memory where they fit; three radix rounds (11,
// 11 and 10 bits) over histograms added up across the cluster find the cut: its
// key, and how many of the tokens equal to it are kept (the first ones).  Each
// warp then counts and emits its own contiguous run of positions, so the list
// comes out ascending.  Gather: the kept tokens' planes to the new pages, 16
// bytes a thread and several loads in flight.  Measured at 32 lists of 40001 to
// 65536 positions cut to 4096: the two kernels 42 us (one block of 1024 threads
// per list and byte-wise rounds: 274); the selection's cluster barriers and
// latencies (seven rounds of about 3 us) are its bound, the gather runs at 0.6 of
// the copy bandwidth.
// ---------------------------------------------------------------------------
struct EvictParams {
  Pool c;
  const int32_t* block_table;
  const int32_t* cache_len;
  const int32_t* new_table;
  int n_seqs, max_pages, new_max_pages;
  int budget, sink, recent;
  int32_t* kept;
  int32_t* new_len;
  int held;  // keys a block holds in shared memory
};

constexpr int kSelThreads = 512, kSelWarps = kSelThreads / 32;
constexpr int kRun = 4 * kSelThreads;  // positions a block takes at a time, four a thread
constexpr int kBins = 2048;
constexpr int kMaxCluster = 8;
constexpr int kMaxHeld = 49152;  // keys a block can hold (192 KB)

__device__ __forceinline__ uint32_t mass_key(float m) { return m != m ? 0xffffffffu : f2key(m + 0.f); }

__global__ void __launch_bounds__(kSelThreads) gqa_evict_select_kernel(const __grid_constant__ EvictParams p) {
  pdl_wait();
  pdl_trigger();
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  __shared__ int hist[kBins], total[kBins];
  __shared__ int warp_gt[kSelWarps], warp_eq[kSelWarps], rank_gt, rank_eq;
  __shared__ uint32_t cut[2];
  extern __shared__ __align__(16) uint32_t keys[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ranks = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  const int h = blockIdx.y, s = blockIdx.z;
  int32_t* kept = p.kept + (static_cast<int64_t>(s) * p.c.Hkv + h) * p.budget;
  const int32_t* table = p.block_table + static_cast<int64_t>(s) * p.max_pages;
  int L = __ldg(p.cache_len + s);
  L = min(max(L, 0), p.max_pages * p.c.page);
  if (h == 0 && rank == 0 && tid == 0) p.new_len[s] = min(L, p.budget);
  if (L <= p.budget) {  // every block of the cluster
    for (int j = rank * kSelThreads + tid; j < p.budget; j += ranks * kSelThreads) kept[j] = j < L ? j : -1;
    return;
  }
  const int lo = p.sink, hi = L - p.recent, want = p.budget - p.sink - p.recent;
  // this block's positions [a, b), split evenly among the warps
  const int per = (L + ranks * kRun - 1) / (ranks * kRun) * kRun;
  const int a = min(rank * per, L), b = min(a + per, L);
  const bool held = per <= p.held;
  // keys of positions j .. j + 3 (j a multiple of 4: one page, on a 16-byte boundary)
  auto read4 = [&](int j) -> uint4 {
    const int64_t at = slot_of(p.c, table, p.max_pages, h, j);
    const float4 m = at < 0 ? make_float4(0.f, 0.f, 0.f, 0.f) : *reinterpret_cast<const float4*>(p.c.mass + at);
    return make_uint4(mass_key(m.x), mass_key(m.y), mass_key(m.z), mass_key(m.w));
  };
  auto keys4 = [&](int j) -> uint4 { return held ? *reinterpret_cast<const uint4*>(keys + (j - a)) : read4(j); };
  if (held) {
#pragma unroll 4
    for (int j = a + 4 * tid; j < b; j += kRun)
      if (CSA_INBOUNDS(j >= a && j - a + 4 <= p.held)) *reinterpret_cast<uint4*>(keys + (j - a)) = read4(j);
  }
  uint32_t prefix = 0;
  int need = want;  // of the keys that share the prefix
  if (want > 0) {
#pragma unroll 1
    for (int round = 0; round < 3; ++round) {
      const int shift = round == 0 ? 21 : (round == 1 ? 10 : 0), bits = round == 2 ? 10 : 11;
      const uint32_t mask = round == 0 ? 0u : ~0u << (round == 1 ? 21 : 10);
      for (int i = tid; i < kBins; i += kSelThreads) hist[i] = 0;
      __syncthreads();
      const int from = max(a, lo), to = min(b, hi);
#pragma unroll 4
      for (int j = a + 4 * tid; j < b; j += kRun) {
        const uint4 k4 = keys4(j);
        const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (j + u >= from && j + u < to && (k[u] & mask) == prefix)
            atomicAdd(&hist[(k[u] >> shift) & ((1u << bits) - 1u)], 1);
      }
      cluster.sync();
      if (ranks > 1) {
        // the cluster's sums: each block adds up a part of the bins and gives it to all
        const int part = kBins / ranks;
        for (int i = rank * part + tid; i < (rank + 1) * part; i += kSelThreads) {
          int c[kMaxCluster], sum = 0;
#pragma unroll
          for (int r = 0; r < kMaxCluster; ++r) c[r] = r < ranks ? *cluster.map_shared_rank(&hist[i], r) : 0;
#pragma unroll
          for (int r = 0; r < kMaxCluster; ++r) sum += c[r];
#pragma unroll
          for (int r = 0; r < kMaxCluster; ++r)
            if (r < ranks) *cluster.map_shared_rank(&total[i], r) = sum;
        }
        cluster.sync();
      }
      const int* sums = ranks > 1 ? total : hist;
      // thread t holds bins 2047 - 4 t down to 2044 - 4 t
      int c4[4], mine = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        c4[i] = sums[kBins - 1 - 4 * tid - i];
        mine += c4[i];
      }
      int inc = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
      }
      if (lane == 31) warp_gt[warp] = inc;
      __syncthreads();
      int before = inc - mine;
      for (int w = 0; w < warp; ++w) before += warp_gt[w];
      if (before < need && need <= before + mine) {
        int i = 0;
        while (before + c4[i] < need) before += c4[i++];
        cut[0] = static_cast<uint32_t>(kBins - 1 - 4 * tid - i);
        cut[1] = static_cast<uint32_t>(need - before);
      }
      __syncthreads();
      prefix |= cut[0] << shift;
      need = static_cast<int>(cut[1]);
    }
  }
  // kept: sink, recent, keys above the cut, and the first `need` keys equal to it
  const int seg = per / kSelWarps;  // positions per warp, a multiple of 128
  const int wa = min(a + warp * seg, b), wb = min(wa + seg, b);
  auto classify = [&](int j, uint32_t& gt, uint32_t& eq) {  // a bit for each of positions j .. j + 3
    gt = eq = 0;
    if (j >= wb) return;
    const uint4 k4 = keys4(j);
    const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (j + u >= wb) break;
      const bool ends = j + u < lo || j + u >= hi;
      gt |= (ends || (want > 0 && k[u] > prefix)) ? 1u << u : 0u;
      eq |= (!ends && want > 0 && k[u] == prefix) ? 1u << u : 0u;
    }
  };
  __syncthreads();
  int ngt = 0, neq = 0;
  for (int j = wa; j < wb; j += 128) {
    uint32_t gt, eq;
    classify(j + 4 * lane, gt, eq);
    ngt += __popc(gt);
    neq += __popc(eq);
  }
  ngt = warp_sum_i(ngt);
  neq = warp_sum_i(neq);
  if (lane == 0) {
    warp_gt[warp] = ngt;
    warp_eq[warp] = neq;
  }
  __syncthreads();
  if (warp == 0) {
    int g = lane < kSelWarps ? warp_gt[lane] : 0, e = lane < kSelWarps ? warp_eq[lane] : 0;
    g = warp_sum_i(g);
    e = warp_sum_i(e);
    if (lane == 0) {
      rank_gt = g;
      rank_eq = e;
    }
  }
  cluster.sync();
  int eq_at = 0, out_at = 0;
  for (int r = 0; r < rank; ++r) {
    out_at += *cluster.map_shared_rank(&rank_gt, r);
    eq_at += *cluster.map_shared_rank(&rank_eq, r);
  }
  for (int w = 0; w < warp; ++w) {
    out_at += warp_gt[w];
    eq_at += warp_eq[w];
  }
  out_at += min(eq_at, need);
  for (int j = wa; j < wb; j += 128) {
    uint32_t gt, eq;
    classify(j + 4 * lane, gt, eq);
    const int mine = __popc(gt) | (__popc(eq) << 16);
    int inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    const int all = __shfl_sync(0xffffffffu, inc, 31);
    const int open = max(need - eq_at, 0);  // equal keys still to be kept
    int eq_before = (inc - mine) >> 16;
    int at = out_at + ((inc - mine) & 0xffff) + min(open, eq_before);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const bool e = (eq >> u) & 1u, take = ((gt >> u) & 1u) || (e && eq_before < open);
      if (take && at < p.budget && CSA_INBOUNDS(at >= 0)) kept[at] = j + 4 * lane + u;
      at += take ? 1 : 0;
      eq_before += e ? 1 : 0;
    }
    out_at += (all & 0xffff) + min(open, all >> 16);
    eq_at += all >> 16;
  }
  cluster.sync();  // no block leaves while another may read its counts
}

constexpr int kGatherTokens = 64;

__global__ void __launch_bounds__(256) gqa_evict_gather_kernel(const __grid_constant__ EvictParams p) {
  pdl_wait();
  __shared__ int64_t src[kGatherTokens], dst[kGatherTokens];
  const int h = blockIdx.y, s = blockIdx.z, tid = threadIdx.x;
  const int j0 = blockIdx.x * kGatherTokens;
  if (tid < kGatherTokens) {
    const int j = j0 + tid;
    const int from = j < p.budget ? p.kept[(static_cast<int64_t>(s) * p.c.Hkv + h) * p.budget + j] : -1;
    int64_t a = -1, b = -1;
    if (from >= 0) {
      a = slot_of(p.c, p.block_table + static_cast<int64_t>(s) * p.max_pages, p.max_pages, h, from);
      b = slot_of(p.c, p.new_table + static_cast<int64_t>(s) * p.new_max_pages, p.new_max_pages, h, j);
    }
    src[tid] = a;  // -1: a page outside the pool, read as zeros
    dst[tid] = b;
    if (b >= 0) p.c.mass[b] = a < 0 ? 0.f : p.c.mass[a];
  }
  __syncthreads();
  const int per = p.c.kp + p.c.vp, n = kGatherTokens * per;
  for (int i0 = tid; i0 < n; i0 += 4 * 256) {
    uint4 v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int i = i0 + u * 256;
      if (i < n) {
        const int t = i / per, x = i - t * per;
        v[u] = make_uint4(0, 0, 0, 0);
        if (src[t] >= 0) v[u] = x < p.c.kp ? p.c.k[src[t] * p.c.kp + x] : p.c.v[src[t] * p.c.vp + x - p.c.kp];
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int i = i0 + u * 256;
      if (i < n) {
        const int t = i / per, x = i - t * per;
        if (dst[t] >= 0) {
          if (x < p.c.kp)
            p.c.k[dst[t] * p.c.kp + x] = v[u];
          else
            p.c.v[dst[t] * p.c.vp + x - p.c.kp] = v[u];
        }
      }
    }
  }
}

}  // namespace
}  // namespace csa

extern "C" {

csa_status gqa_cache_append(const void* k, const void* v, const gqa_cache* cache, const gqa_batch* batch,
                            void* stream) {
  using namespace csa;
  const char* what = "gqa_cache_append";
  clear_error();
  if (csa_status st = gqa::check_batch(what, cache, batch); st != CSA_OK) return st;
  if (batch->n_seqs == 0 || batch->total_q == 0) return CSA_OK;
  if (csa_status st = gqa::check_pool(what, cache, batch, true); st != CSA_OK) return st;
  CSA_REQUIRE_PTR(k);
  CSA_REQUIRE_PTR(v);
  CSA_REQUIRE(cache->mass == nullptr || aligned16(cache->mass), "%s: mass is not 16-byte aligned", what);
  AppendParams p;
  p.c = pool_of(cache);
  p.k = static_cast<const uint4*>(k);
  p.v = static_cast<const uint4*>(v);
  p.block_table = batch->block_table;
  p.cache_len = batch->cache_len;
  p.cu_q = batch->cu_q;
  p.n_seqs = batch->n_seqs;
  p.max_pages = batch->max_pages;
  p.total_q = static_cast<int>(batch->total_q);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const unsigned blocks = static_cast<unsigned>((batch->total_q + 7) / 8);
  prof_begin(s);
  const cudaError_t e = launch_pdl(gqa_append_kernel, dim3(blocks), dim3(256), 0, s, 1, p);
  prof_end(s);
  return check_launch(what, e);
}

csa_status gqa_cache_evict(const gqa_cache* cache, const gqa_batch* batch, int32_t budget, int32_t n_sink,
                           int32_t n_recent, const int32_t* new_table, int32_t new_max_pages, int32_t* kept,
                           int32_t* new_len, void* stream) {
  using namespace csa;
  const char* what = "gqa_cache_evict";
  clear_error();
  if (csa_status st = gqa::check_batch(what, cache, batch); st != CSA_OK) return st;
  CSA_REQUIRE(cache->mass != nullptr, "%s: the cache has no mass plane", what);
  CSA_REQUIRE(budget >= 1 && budget <= (1 << 30), "%s: budget must be in [1, 2^30] (got %d)", what, budget);
  CSA_REQUIRE(n_sink >= 0 && n_recent >= 0 && static_cast<int64_t>(n_sink) + n_recent <= budget,
              "%s: n_sink and n_recent must be >= 0 and together at most the budget", what);
  if (batch->n_seqs == 0) return CSA_OK;
  if (csa_status st = gqa::check_pool(what, cache, batch, false); st != CSA_OK) return st;
  CSA_REQUIRE(new_max_pages >= 1 && static_cast<int64_t>(new_max_pages) * cache->page_size >= budget,
              "%s: the new table's rows hold fewer tokens than the budget", what);
  CSA_REQUIRE_PTR(cache->mass);
  CSA_REQUIRE_PTR(new_table);
  CSA_REQUIRE_PTR(kept);
  CSA_REQUIRE_PTR(new_len);
  CSA_REQUIRE(new_table != batch->block_table, "%s: the new table is the old one: eviction needs pages of its own", what);
  CSA_REQUIRE(new_len != batch->cache_len, "%s: new_len is cache_len: it needs an array of its own", what);
  CSA_REQUIRE(batch->n_seqs <= 65535, "%s: at most 65535 sequences", what);
  EvictParams p;
  p.c = pool_of(cache);
  p.block_table = batch->block_table;
  p.cache_len = batch->cache_len;
  p.new_table = new_table;
  p.n_seqs = batch->n_seqs;
  p.max_pages = batch->max_pages;
  p.new_max_pages = new_max_pages;
  p.budget = budget;
  p.sink = n_sink;
  p.recent = n_recent;
  p.kept = kept;
  p.new_len = new_len;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  // A cluster per list: enough blocks that each has about 4096 positions of the longest (at 65536 positions and 32
  // lists: 274 us with one block of 1024 threads per list).
  const int longest = batch->max_pages * cache->page_size;
  int ranks = 1;
  while (ranks < kMaxCluster && longest > 4096 * ranks) ranks *= 2;
  p.held = static_cast<int>((static_cast<int64_t>(longest) + ranks * kRun - 1) / (ranks * kRun) * kRun);
  if (p.held > kMaxHeld) p.held = 0;  // read again each time
  const int smem = p.held * 4;
  if (!ensure_smem(reinterpret_cast<const void*>(gqa_evict_select_kernel), smem))
    return fail(CSA_ERR_CUDA, "%s: cannot raise the shared memory limit", what);
  prof_begin(s);
  cudaError_t e = launch_pdl(gqa_evict_select_kernel, dim3(ranks, cache->n_kv_heads, batch->n_seqs), dim3(kSelThreads),
                             static_cast<size_t>(smem), s, ranks, p);
  prof_end(s);
  if (csa_status st = check_launch(what, e); st != CSA_OK) return st;
  e = launch_pdl(gqa_evict_gather_kernel,
                 dim3((budget + kGatherTokens - 1) / kGatherTokens, cache->n_kv_heads, batch->n_seqs), dim3(256), 0, s,
                 1, p);
  return check_launch(what, e);
}

}  // extern "C"

namespace csa {
// Reads (and optionally clears) this unit's device error word.
CSA_DEFINE_DEVICE_ERROR_READER(gqa_cache_device_error)
}  // namespace csa
