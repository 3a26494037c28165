// Walks the grouped-head work partition (gqa_work.cuh) on the host: every CTA's share of a batch, item by item.
//   gqa_partition attention|weight H_kv G tokens_per_tile tokens_per_item CTAs  new held  [new held ...]
// Prints the units of the list, or what is wrong first (status 1).  Only the search of a share's first item is
// restated here (the kernels make it with a block's shuffles); all numbers are the header's.
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <vector>

#include "gqa_work.cuh"

using namespace csa::gqa;

struct Item {
  int s, h, blk;
};

template <typename Items>
static Share find(const Geometry& g, int cta, int n_ctas, int64_t* total_out) {
  std::vector<int64_t> head(g.n_seqs);  // units of one head of each sequence
  int64_t total = 0;
  Seq q;
  for (int s = 0; s < g.n_seqs; ++s) {
    q.load(g, s);
    head[s] = Items::units_before(g, q, Items::count(q));
    total += head[s] * g.Hkv;
  }
  *total_out = total;
  Share sh = {0, 0, 0, 0, 0};
  const int ctas = static_cast<int>(total < n_ctas ? total : n_ctas);
  if (cta >= ctas) return sh;
  int64_t at = share_range(total, ctas, cta, &sh.left);
  int s = 0;
  while (at >= head[s] * g.Hkv) at -= head[s++] * g.Hkv;
  sh.s = s;
  sh.h = head_of(at, head[s]);
  at -= sh.h * head[s];
  q.load(g, s);
  int lo = 0, hi = Items::count(q);  // the last item with units_before <= at
  while (hi - lo > 1) {
    const int mid = lo + (hi - lo) / 2;
    if (Items::units_before(g, q, mid) <= at) lo = mid; else hi = mid;
  }
  sh.blk = lo;
  sh.unit = static_cast<int>(at - Items::units_before(g, q, lo));
  if (at < 0 || sh.h >= g.Hkv) {
    printf("CTA %d of %d begins in head %d of %d, at unit %lld of it\n", cta, ctas, sh.h, g.Hkv,
           static_cast<long long>(at));
    exit(1);
  }
  return sh;
}

template <typename Items>
static bool next_item(const Geometry& g, Item& it) {  // false behind the last
  Seq q;
  for (++it.blk; it.s < g.n_seqs; ++it.s, it.h = 0, it.blk = 0)
    for (q.load(g, it.s); it.h < g.Hkv; ++it.h, it.blk = 0)
      if (it.blk < Items::count(q)) return true;
  return false;
}

static int wrong(int cta, const Item& it, const char* what) {
  printf("CTA %d, sequence %d, head %d, item %d: %s\n", cta, it.s, it.h, it.blk, what);
  return 1;
}

int main(int argc, char** argv) {
  if (argc < 9 || (argc - 7) % 2) return 2;
  const bool attention = !strcmp(argv[1], "attention");
  Geometry g;
  memset(&g, 0, sizeof(g));
  g.Hkv = atoi(argv[2]);
  g.G = atoi(argv[3]);
  g.tpt = atoi(argv[4]);
  g.tpb = atoi(argv[5]);
  const int ctas = atoi(argv[6]);
  std::vector<int32_t> cu(1, 0), len;
  for (int i = 7; i < argc; i += 2) {
    cu.push_back(cu.back() + atoi(argv[i]));
    len.push_back(atoi(argv[i + 1]));
  }
  g.cu_q = cu.data();
  g.cache_len = len.data();
  g.n_seqs = static_cast<int>(len.size());
  g.max_len = 0x7fffffff - 65536;
  g.total_q = cu.back();
  Item want = {0, 0, -1};
  bool open = attention ? next_item<Blocks>(g, want) : next_item<KeyPairs>(g, want);
  int tile = 0;  // of the item, the first that nobody had yet
  int64_t total = 0;
  for (int cta = 0; cta < ctas; ++cta) {
    if (attention) {
      const Share sh = find<Blocks>(g, cta, ctas, &total);
      Walk w;
      for (bool more = w.begin(g, sh); more; more = w.next(g)) {
        const Item it = {w.s, w.h, w.blk};
        if (!open || it.s != want.s || it.h != want.h || it.blk != want.blk) return wrong(cta, it, "not the next item");
        if (w.n != w.q.tiles(g, w.blk) || w.t0 != tile || w.t1 <= w.t0 || w.t1 > w.n) return wrong(cta, it, "not its next tiles");
        tile = w.t1;
        if (tile == w.n) {
          tile = 0;
          open = next_item<Blocks>(g, want);
        }
      }
    } else {
      const Share sh = find<KeyPairs>(g, cta, ctas, &total);
      MassWalk w;
      for (bool more = w.begin(g, sh); more; more = w.next(g)) {
        const Item it = {w.s, w.h, w.pair};
        if (!open || it.s != want.s || it.h != want.h || it.blk != want.blk) return wrong(cta, it, "not the next item");
        open = next_item<KeyPairs>(g, want);
      }
    }
  }
  if (open) return wrong(ctas, want, "nobody's item");
  printf("%lld\n", static_cast<long long>(total));
  return 0;
}
