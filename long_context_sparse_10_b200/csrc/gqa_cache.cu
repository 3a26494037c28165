// The paged cache of the grouped-head (GQA) attention: appending a chunk, and
// eviction by accumulated weight.
#include "gqa_device.cuh"
#include "gqa_host.h"

namespace csa {
namespace {

using namespace gqa;

// ---------------------------------------------------------------------------
// Append: a warp per new token copies its rows of all kv heads, 16 bytes a
// lane.  Bound by the copy (read and write of each new row once).
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
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (row >= p.total_q || row >= __ldg(p.cu_q + p.n_seqs)) return;
  const int s = seq_of(p.cu_q, p.n_seqs, row);
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
// Eviction.  Select: one block per (sequence, kv head); a radix select over
// the order-preserving 32-bit keys of the middle tokens' mass finds the cut
// (its key and how many of the tokens equal to it are kept, the first ones),
// then each warp counts and emits its own contiguous run of positions, so the
// list comes out ascending.  Gather: the kept tokens' planes to the new pages.
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
};

__device__ __forceinline__ uint32_t mass_key(float m) { return m != m ? 0xffffffffu : f2key(m + 0.f); }

__global__ void __launch_bounds__(1024) gqa_evict_select_kernel(const __grid_constant__ EvictParams p) {
  pdl_wait();
  __shared__ int hist[256];
  __shared__ int cnt_gt[32], cnt_eq[32];
  __shared__ uint32_t cut[2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int h = blockIdx.x, s = blockIdx.y;
  int32_t* kept = p.kept + (static_cast<int64_t>(s) * p.c.Hkv + h) * p.budget;
  const int32_t* table = p.block_table + static_cast<int64_t>(s) * p.max_pages;
  int L = __ldg(p.cache_len + s);
  L = min(max(L, 0), p.max_pages * p.c.page);
  if (h == 0 && tid == 0) p.new_len[s] = min(L, p.budget);
  if (L <= p.budget) {
    for (int j = tid; j < p.budget; j += 1024) kept[j] = j < L ? j : -1;
    return;
  }
  const int lo = p.sink, hi = L - p.recent, want = p.budget - p.sink - p.recent;
  auto key_of = [&](int j) -> uint32_t {
    const int64_t at = slot_of(p.c, table, p.max_pages, h, j);
    return mass_key(at < 0 ? 0.f : p.c.mass[at]);
  };
  uint32_t prefix = 0, mask = 0;
  int need = want;
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (tid < 256) hist[tid] = 0;
    __syncthreads();
    for (int j = lo + tid; j < hi; j += 1024) {
      const uint32_t k = key_of(j);
      if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & 255u], 1);
    }
    __syncthreads();
    if (warp == 0) {
      // lane l holds bins 255 - 8 l .. 248 - 8 l, from the top
      int c8 = 0;
      for (int i = 0; i < 8; ++i) c8 += hist[255 - 8 * lane - i];
      int inc = c8;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
      }
      int before = inc - c8;
      const bool mine = need > 0 ? (before < need && need <= inc) : lane == 0;
      if (mine) {
        int b = 255 - 8 * lane;
        if (need > 0) {
          while (before + hist[b] < need) before += hist[b--];
        }
        cut[0] = static_cast<uint32_t>(b);
        cut[1] = static_cast<uint32_t>(need > 0 ? need - before : 0);
      }
    }
    __syncthreads();
    prefix |= cut[0] << shift;
    mask |= 255u << shift;
    need = static_cast<int>(cut[1]);
    __syncthreads();
  }
  // want == 0: nothing of the middle, whatever its keys are
  const int seg = ((L + 31) / 32 + 31) / 32 * 32;  // positions per warp
  const int a = min(warp * seg, L), b = min(a + seg, L);
  auto classify = [&](int j, bool& gt, bool& eq) {
    gt = eq = false;
    if (j >= b) return;
    if (j < lo || j >= hi) {
      gt = true;
    } else if (want > 0) {
      const uint32_t k = key_of(j);
      gt = k > prefix;
      eq = k == prefix;
    }
  };
  int ngt = 0, neq = 0;
  for (int j = a; j < b; j += 32) {
    bool gt, eq;
    classify(j + lane, gt, eq);
    ngt += __popc(__ballot_sync(0xffffffffu, gt));
    neq += __popc(__ballot_sync(0xffffffffu, eq));
  }
  if (lane == 0) {
    cnt_gt[warp] = ngt;
    cnt_eq[warp] = neq;
  }
  __syncthreads();
  int eq_at = 0, out_at = 0;
  for (int w = 0; w < warp; ++w) {
    eq_at += cnt_eq[w];
    out_at += cnt_gt[w];
  }
  out_at += min(eq_at, need);
  for (int j = a; j < b; j += 32) {
    bool gt, eq;
    classify(j + lane, gt, eq);
    const uint32_t below = (1u << lane) - 1u;
    const uint32_t me = __ballot_sync(0xffffffffu, eq);
    const bool take = gt || (eq && eq_at + __popc(me & below) < need);
    const uint32_t mt = __ballot_sync(0xffffffffu, take);
    const int at = out_at + __popc(mt & below);
    if (take && at < p.budget) kept[at] = j + lane;
    eq_at += __popc(me);
    out_at += __popc(mt);
  }
}

__global__ void __launch_bounds__(256) gqa_evict_gather_kernel(const __grid_constant__ EvictParams p) {
  pdl_wait();
  const int h = blockIdx.y, s = blockIdx.z, lane = threadIdx.x & 31;
  const int32_t* kept = p.kept + (static_cast<int64_t>(s) * p.c.Hkv + h) * p.budget;
  for (int u = threadIdx.x >> 5; u < 64; u += 8) {
    const int j = blockIdx.x * 64 + u;
    if (j >= p.budget) return;
    const int from = kept[j];
    if (from < 0) return;
    const int64_t src = slot_of(p.c, p.block_table + static_cast<int64_t>(s) * p.max_pages, p.max_pages, h, from);
    const int64_t dst = slot_of(p.c, p.new_table + static_cast<int64_t>(s) * p.new_max_pages, p.new_max_pages, h, j);
    if (src < 0 || dst < 0) continue;
    for (int i = lane; i < p.c.kp + p.c.vp; i += 32) {
      if (i < p.c.kp)
        p.c.k[dst * p.c.kp + i] = p.c.k[src * p.c.kp + i];
      else
        p.c.v[dst * p.c.vp + i - p.c.kp] = p.c.v[src * p.c.vp + i - p.c.kp];
    }
    if (lane == 0) p.c.mass[dst] = p.c.mass[src];
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

size_t gqa_cache_evict_workspace_size(int32_t, int32_t, int32_t, int32_t) { return 0; }

csa_status gqa_cache_evict(const gqa_cache* cache, const gqa_batch* batch, int32_t budget, int32_t n_sink,
                           int32_t n_recent, const int32_t* new_table, int32_t new_max_pages, int32_t* kept,
                           int32_t* new_len, void* workspace, size_t workspace_bytes, void* stream) {
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
  (void)workspace;
  (void)workspace_bytes;
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
  prof_begin(s);
  cudaError_t e = launch_pdl(gqa_evict_select_kernel, dim3(cache->n_kv_heads, batch->n_seqs), dim3(1024), 0, s, 1, p);
  prof_end(s);
  if (csa_status st = check_launch(what, e); st != CSA_OK) return st;
  e = launch_pdl(gqa_evict_gather_kernel, dim3((budget + 63) / 64, cache->n_kv_heads, batch->n_seqs), dim3(256), 0, s,
                 1, p);
  return check_launch(what, e);
}

}  // extern "C"

namespace csa {
// Reads (and optionally clears) this unit's device error word.
CSA_DEFINE_DEVICE_ERROR_READER(gqa_cache_device_error)
}  // namespace csa
