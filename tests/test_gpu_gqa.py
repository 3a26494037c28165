"""GPU parity of the grouped-head dense attention and its paged cache against the float64 oracle.

Tolerances, per element:
  * out: each probability is rounded to bf16 (half a step, 2^-8 relative) and so is the result: at most
    2^-8 (sum p |v| + |out|), to which the products of both and fp32 arithmetic add less than 2 %;
  * scores: a dot product of d terms in fp32 is off by at most d 2^-23 sum |q c| (truncating accumulation), so lse and
    the logarithm of a weight by that plus 2^-18: exponentials off by at most 2.7e-6 = 2^-18.5 (the polynomial's bound;
    the unit's is 2^-22), log2 and the sums in fp32 with what is left.
"""
import math

import numpy as np
import pytest
import torch

import long_context_sparse_10_b200 as csa
from long_context_sparse_10_b200 import _lib
from oracle import gqa_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
DIMS = [(192, 128), (128, 128), (64, 64)]


def bf16(g, *shape, std=1.0):
    return torch.from_numpy((g.standard_normal(shape) * std).astype(np.float32)).to(torch.bfloat16)


def f64(t):
    return t.detach().cpu().double().numpy()


def score_tol(d, size):
    return (d + 8) * 2.0**-23 * size + 2.0**-18


def check_out(got, ref, size, what):
    tol = 1.02 * 2.0**-8 * (size + np.abs(ref)) + 1e-30
    assert got.shape == ref.shape and np.all(np.isfinite(got)), what
    worst = float((np.abs(got - ref) / tol).max()) if ref.size else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3f} of the tolerance"


def check_lse(got, ref, tol, what):
    assert np.array_equal(np.isneginf(got), np.isneginf(ref)), what
    fin = np.isfinite(ref)
    if fin.any():
        worst = float(np.abs(got[fin] - ref[fin]).max())
        assert worst <= tol, f"{what}: lse off by {worst:.3e}, {tol:.3e} allowed"


def no_device_error():
    lib = _lib.load()
    assert lib.csa_check_device_error(torch.cuda.current_stream().cuda_stream) == _lib.CSA_OK, lib.csa_last_error()


@pytest.mark.parametrize("lens,Hkv,G,dims", [
    ([1], 1, 1, (128, 128)),
    ([128], 2, 4, (128, 128)),
    ([129, 0, 1, 127], 2, 4, (192, 128)),
    ([0, 0, 3, 0], 3, 5, (64, 64)),
    ([300], 1, 16, (192, 128)),
    ([257, 64, 65], 2, 1, (128, 128)),
    ([200, 77], 1, 64, (192, 128)),
    ([70, 5], 1, 128, (64, 64)),
    ([513, 255], 2, 7, (128, 128)),
    ([31] * 9, 2, 12, (64, 64)),
    ([1100], 1, 3, (128, 128)),
])
def test_packed_prompts(lens, Hkv, G, dims):
    g = np.random.default_rng(sum(lens) + 7 * G)
    n = sum(lens)
    q, k, v = bf16(g, n, Hkv * G, dims[0]), bf16(g, n, Hkv, dims[0]), bf16(g, n, Hkv, dims[1])
    scale = 1 / math.sqrt(dims[0])
    out, lse = csa.gqa_dense_packed(q.to(DEV), k.to(DEV), v.to(DEV), csa.Packed(lens, 1), scale)
    torch.cuda.synchronize()
    no_device_error()
    a = 0
    for s in lens:
        qs, ks, vs = f64(q[a:a + s]), f64(k[a:a + s]), f64(v[a:a + s])
        ref, rl, size = R.attend(qs, ks, vs, scale, 0)
        check_out(f64(out[a:a + s]), ref, size, f"rows {a}")
        check_lse(f64(lse[a:a + s]), rl, score_tol(dims[0], R.score_size(qs, ks, scale)), f"rows {a}")
        a += s


@pytest.mark.parametrize("dims", DIMS)
def test_a_prompt_batch_gives_the_same_bits_every_time(dims):
    # last blocks of a few tokens (one tile of rows, two streams over its keys) beside full ones, on every SM
    lens = [2048, 513, 1, 777, 0, 4000, 1025, 128, 31, 1500, 2049]
    g = np.random.default_rng(6)
    n, Hkv, G = sum(lens), 4, 4
    q, k, v = bf16(g, n, Hkv * G, dims[0]), bf16(g, n, Hkv, dims[0]), bf16(g, n, Hkv, dims[1])
    args = (q.to(DEV), k.to(DEV), v.to(DEV), csa.Packed(lens, 1), 1 / math.sqrt(dims[0]))
    runs = [csa.gqa_dense_packed(*args) for _ in range(30)]
    torch.cuda.synchronize()
    no_device_error()
    for out, lse in runs[1:]:
        assert torch.equal(out, runs[0][0]) and torch.equal(lse, runs[0][1])
    a = 0
    for s in lens:  # the last rows of each sequence
        b = max(s - 3, 0)
        ref, _, size = R.attend(f64(q[a + b:a + s]), f64(k[a:a + s]), f64(v[a:a + s]), args[4], b)
        check_out(f64(runs[0][0][a + b:a + s]), ref, size, f"sequence at {a}")
        a += s


class Case:
    """A paged cache with its pages in random order; what no token lies in holds NaN."""

    def __init__(self, seed, lens, n, Hkv, G, dims, page, extra_rows=0, junk=float("nan"), std=1.0, width=None):
        g = np.random.default_rng(seed)
        self.g, self.lens, self.n, self.Hkv, self.G, self.dims, self.page = g, lens, n, Hkv, G, dims, page
        need = [-(-max(L, 0) // page) for L in lens]
        width = width or max(max(need), 1) + 1
        P = sum(need) + 2
        order = list(g.permutation(P))
        self.table = np.full((len(lens), width), -5, np.int32)
        for s, c in enumerate(need):
            self.table[s, :c] = [order.pop() for _ in range(c)]
        k, v = np.full((P, Hkv, page, dims[0]), junk, np.float32), np.full((P, Hkv, page, dims[1]), junk, np.float32)
        mass = np.zeros((P, Hkv, page), np.float32)
        for s, L in enumerate(lens):
            for j in range(max(L, 0)):
                pg, sl = self.table[s, j // page], j % page
                k[pg, :, sl] = g.standard_normal((Hkv, dims[0])) * std
                v[pg, :, sl] = g.standard_normal((Hkv, dims[1]))
                mass[pg, :, sl] = g.random(Hkv)
        self.cu = [0]
        for c in n:
            self.cu.append(self.cu[-1] + c)
        self.rows = self.cu[-1] + extra_rows
        self.k, self.v = torch.from_numpy(k).to(torch.bfloat16), torch.from_numpy(v).to(torch.bfloat16)
        self.mass = torch.from_numpy(mass)
        self.q = bf16(g, self.rows, Hkv * G, dims[0], std=std)
        self.scale = 1 / math.sqrt(dims[0])
        self.cache = csa.GqaCache(self.k.to(DEV), self.v.to(DEV), self.mass.to(DEV))
        self.batch = csa.GqaBatch(i32(self.table), i32(lens), i32(self.cu), max_q=max(max(n), 1), total_q=self.rows)

    def live(self, plane, s):
        return R.live(f64(plane), self.table[s], max(self.lens[s], 0))

    def check(self, out, lse, what=""):
        for s, L in enumerate(self.lens):
            a, b = self.cu[s], self.cu[s + 1]
            qs, ks, vs = f64(self.q[a:b]), self.live(self.k, s), self.live(self.v, s)
            ref, rl, size = R.attend(qs, ks, vs, self.scale, L - (b - a))
            check_out(f64(out[a:b]), ref, size, f"{what} sequence {s}")
            check_lse(f64(lse[a:b]), rl, score_tol(self.dims[0], R.score_size(qs, ks, self.scale)), f"{what} sequence {s}")


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


PAGED = [
    # lengths with the new tokens, new tokens, H_kv, G, dims, page
    ([1], [1], 1, 1, (128, 128), 16),
    ([777], [1], 2, 4, (128, 128), 16),
    ([127, 128, 129, 1], [1, 1, 1, 1], 2, 8, (64, 64), 32),
    ([300, 5, 1000], [1, 1, 1], 1, 64, (192, 128), 128),
    ([260, 40, 17, 128], [7, 40, 0, 1], 2, 4, (192, 128), 64),
    ([700, 33], [150, 33], 2, 3, (128, 128), 16),
    ([0, 9, 400], [0, 9, 300], 1, 5, (64, 64), 16),
    ([513], [513], 1, 2, (128, 128), 32),
    ([600, 64], [2, 3], 1, 128, (64, 64), 64),
    ([5000], [1], 1, 16, (192, 128), 64),
    ([900, 900], [64, 1], 3, 12, (128, 128), 128),
    ([190, 3], [5, 1], 1, 50, (128, 128), 16),
]


@pytest.mark.parametrize("lens,n,Hkv,G,dims,page", PAGED)
def test_paged_chunks(lens, n, Hkv, G, dims, page):
    c = Case(sum(lens) + G, lens, n, Hkv, G, dims, page)
    out, lse = csa.gqa_dense_paged(c.q.to(DEV), c.cache, c.batch, c.scale)
    torch.cuda.synchronize()
    no_device_error()
    c.check(out, lse)


def test_rows_without_a_key_and_rows_behind_the_last_sequence():
    # sequence 0 holds fewer tokens than its chunk (its first rows stand before token 0); sequence 2 holds none
    c = Case(3, [3, 200, 0], [5, 130, 4], 2, 4, (128, 128), 32, extra_rows=6)
    out = torch.full((c.rows, 8, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((c.rows, 8), 7.0, device=DEV)
    csa.gqa_dense_paged(c.q.to(DEV), c.cache, c.batch, c.scale, out=out, lse=lse)
    torch.cuda.synchronize()
    no_device_error()
    c.check(out, lse)
    assert torch.all(out[:2] == 0) and torch.all(torch.isneginf(lse[:2]))
    assert torch.all(out[c.cu[3]:] == 7.0) and torch.all(lse[c.cu[3]:] == 7.0)


@pytest.mark.parametrize("n", [1, 140])
def test_logits_that_grow_move_the_softmax_reference(n):
    # keys grow along the sequence, so the maximum rises in every tile; far beyond the range of exp in 32 bits
    c = Case(11, [1500], [n], 1, 4, (128, 128), 64)
    k = f64(c.k)
    for j in range(1500):
        k[c.table[0, j // 64], :, j % 64] *= 0.05 + 0.04 * (j / 16)
    c.k = torch.from_numpy(k).to(torch.bfloat16)
    c.cache.k.copy_(c.k)
    out, lse = csa.gqa_dense_paged(c.q.to(DEV), c.cache, c.batch, c.scale)
    torch.cuda.synchronize()
    no_device_error()
    c.check(out, lse)


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_a_key_that_is_not_finite_shows_in_the_rows_that_see_it_and_in_no_other(value):
    L, g = 420, np.random.default_rng(13)
    for j in list(range(64, 97)) + [0, 127, 128, 255, 300]:
        q, k, v = bf16(g, L, 2, 128), bf16(g, L, 1, 128), bf16(g, L, 1, 128)
        q[:, :, 0] = q[:, :, 0].abs() + 0.5  # +inf * q_0 = +inf
        k[j, 0, 0] = value
        scale = 0.09
        out, lse = csa.gqa_dense_packed(q.to(DEV), k.to(DEV), v.to(DEV), csa.Packed([L], 1), scale)
        out, lse = out.float().cpu(), lse.cpu()
        assert torch.all(torch.isfinite(out[:j])) and torch.all(torch.isfinite(lse[:j])), j
        assert torch.all(torch.isnan(out[j:])) and torch.all(torch.isnan(lse[j:])), j
        if j in (70, 300):
            ref, rl, size = R.attend(f64(q[:j]), f64(k[:j]), f64(v[:j]), scale, 0)
            check_out(out[:j].double().numpy(), ref, size, f"key {j}")
    no_device_error()


def test_one_long_sequence_is_shared_by_every_sm():
    c = Case(5, [20011], [1], 1, 8, (128, 128), 128)
    out, lse = csa.gqa_dense_paged(c.q.to(DEV), c.cache, c.batch, c.scale)
    again, lse2 = csa.gqa_dense_paged(c.q.to(DEV), c.cache, c.batch, c.scale)
    torch.cuda.synchronize()
    no_device_error()
    c.check(out, lse)
    assert torch.equal(out, again) and torch.equal(lse, lse2)  # partial states are joined in a fixed order


def test_junk_behind_the_end_reaches_neither_of_two_row_tiles():
    # every item has two tiles of rows over one key tile, whose end is junk (NaN): each stream's product waits for its
    # own clearing, whichever of them comes first
    lens = [33 + i % 60 for i in range(120)]
    c = Case(8, lens, [L - i % 2 for i, L in enumerate(lens)], 2, 4, (128, 128), 64)
    q = c.q.to(DEV)
    runs = [csa.gqa_dense_paged(q, c.cache, c.batch, c.scale) for _ in range(40)]
    torch.cuda.synchronize()
    no_device_error()
    c.check(*runs[0])
    for out, lse in runs[1:]:
        assert torch.equal(out, runs[0][0]) and torch.equal(lse, runs[0][1])


def test_items_in_which_a_stream_has_no_tile():
    # one-tile items give the second stream nothing, and so do rows whose keys end before a CTA's piece; no wait may
    # depend on which stream runs ahead
    for seed, (L, n) in enumerate(((100, 1), (128, 1), (129, 2), (40, 40), (300, 70))):
        lens = [max(n, L - i % 7) for i in range(300)]
        c = Case(50 + seed, lens, [n] * 300, 1, 4, (64, 64), 16)
        q = c.q.to(DEV)
        runs = [csa.gqa_dense_paged(q, c.cache, c.batch, c.scale) for _ in range(60)]
        torch.cuda.synchronize()
        no_device_error()
        for out, lse in runs[1:]:
            assert torch.equal(out, runs[0][0]) and torch.equal(lse, runs[0][1])


def test_many_sequences():
    g = np.random.default_rng(2)
    lens = [int(x) for x in g.integers(0, 90, 700)]
    n = [min(L, int(x)) for L, x in zip(lens, g.integers(0, 3, 700))]
    c = Case(9, lens, n, 1, 2, (64, 64), 16)
    out, lse = csa.gqa_dense_paged(c.q.to(DEV), c.cache, c.batch, c.scale)
    torch.cuda.synchronize()
    no_device_error()
    c.check(out, lse)


def test_a_prompt_through_the_cache_equals_the_prompt_itself():
    lens = [400, 130, 1]
    c = Case(21, lens, lens, 2, 4, (192, 128), 32)
    k = torch.cat([torch.from_numpy(c.live(c.k, s)) for s in range(3)]).to(torch.bfloat16).to(DEV)
    v = torch.cat([torch.from_numpy(c.live(c.v, s)) for s in range(3)]).to(torch.bfloat16).to(DEV)
    a = csa.gqa_dense_paged(c.q.to(DEV), c.cache, c.batch, c.scale)
    b = csa.gqa_dense_packed(c.q.to(DEV), k, v, csa.Packed(lens, 1), c.scale)
    torch.cuda.synchronize()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_pages_far_into_a_large_pool():
    # slots beyond 2^31 elements of the planes
    page, Hkv, d = 64, 8, 128
    P = (1 << 31) // (Hkv * page * d) + 40
    cache = csa.GqaCache(torch.empty(P, Hkv, page, d, dtype=torch.bfloat16, device=DEV),
                         torch.empty(P, Hkv, page, d, dtype=torch.bfloat16, device=DEV),
                         torch.empty(P, Hkv, page, device=DEV))
    g = np.random.default_rng(4)
    L = 200
    table = np.array([[P - 1, P - 3, P - 2, P - 9]], np.int32)
    k, v, q = bf16(g, L, Hkv, d), bf16(g, L, Hkv, d), bf16(g, L, Hkv * 2, d)
    batch = csa.GqaBatch(i32(table), i32([L]), i32([0, L]), max_q=L, total_q=L)
    csa.gqa_cache_append(k.to(DEV), v.to(DEV), cache, batch)
    out, lse = csa.gqa_dense_paged(q.to(DEV), cache, batch, 0.1)
    csa.gqa_cache_mass(q.to(DEV), lse, cache, batch, 0.1)
    new = np.array([[P - 5, P - 7]], np.int32)
    kept, new_len = csa.gqa_cache_evict(cache, batch, 100, i32(new), sink=3, recent=10)
    torch.cuda.synchronize()
    no_device_error()
    ref, rl, size = R.attend(f64(q), f64(k), f64(v), 0.1, 0)
    check_out(f64(out), ref, size, "large pool")
    assert int(new_len[0]) == 100
    for h in range(Hkv):
        ids = kept[0, h].cpu().long()
        held = torch.cat([cache.k[P - 5, h], cache.k[P - 7, h, :36]]).cpu()
        assert torch.equal(held, k[ids, h])


def test_replayed_with_other_lengths():
    c = Case(31, [300, 90], [1, 1], 2, 4, (128, 128), 32)
    q = c.q.to(DEV)
    out = torch.empty(2, 8, 128, dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(2, 8, device=DEV)
    ws = torch.empty(csa.gqa_dense_workspace_size(1, 8, 2, 128), dtype=torch.uint8, device=DEV)
    csa.gqa_dense_paged(q, c.cache, c.batch, c.scale, out=out, lse=lse, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        csa.gqa_dense_paged(q, c.cache, c.batch, c.scale, out=out, lse=lse, workspace=ws)
    for lens in ([300, 90], [17, 64], [256, 1]):
        c.lens = lens
        c.batch.cache_len.copy_(i32(lens))
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        c.check(out, lse, f"lengths {lens}")


def test_a_captured_chunk_replayed_with_other_chunks():
    # captured for chunks of up to 70 tokens; the same graph then takes one token a sequence, none, and long ones
    c = Case(35, [500, 300, 90], [70, 1, 30], 2, 4, (192, 128), 32)
    rows = 101
    q = c.q.to(DEV)
    out = torch.empty(rows, 8, 128, dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(rows, 8, device=DEV)
    ws = torch.empty(csa.gqa_dense_workspace_size(70, 8, 2, 128), dtype=torch.uint8, device=DEV)
    csa.gqa_dense_paged(q, c.cache, c.batch, c.scale, out=out, lse=lse, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        csa.gqa_dense_paged(q, c.cache, c.batch, c.scale, out=out, lse=lse, workspace=ws)
    for lens, n in (([500, 300, 90], [70, 1, 30]), ([129, 1, 64], [1, 1, 1]), ([400, 300, 70], [0, 31, 70])):
        c.lens, c.n = lens, n
        c.cu = [0, n[0], n[0] + n[1], sum(n)]
        c.batch.cache_len.copy_(i32(lens))
        c.batch.cu_q.copy_(i32(c.cu))
        out.fill_(5.0)
        graph.replay()
        torch.cuda.synchronize()
        no_device_error()
        c.check(out, lse, f"chunks {n}")
        assert torch.all(out[sum(n):] == 5.0)


def test_a_captured_decode_step_and_eviction():
    """append, attention, weight and eviction in one graph; what it computes is what the calls compute one by one."""
    c = Case(36, [300, 45], [1, 1], 2, 4, (128, 128), 16)
    pages = 3
    P = c.k.shape[0]
    new = i32(P + np.arange(2 * pages).reshape(2, pages))
    k, v = bf16(c.g, 2, 2, 128).to(DEV), bf16(c.g, 2, 2, 128).to(DEV)
    q = c.q.to(DEV)

    def pool():
        pad = [torch.zeros(2 * pages, *t.shape[1:], dtype=t.dtype) for t in (c.k, c.v, c.mass)]
        return csa.GqaCache(*[torch.cat([t, z]).to(DEV) for t, z in zip((c.k, c.v, c.mass), pad)])

    def step(cache):
        csa.gqa_cache_append(k, v, cache, c.batch)
        out, lse = csa.gqa_dense_paged(q, cache, c.batch, c.scale)
        csa.gqa_cache_mass(q, lse, cache, c.batch, c.scale)
        kept, new_len = csa.gqa_cache_evict(cache, c.batch, 40, new, sink=2, recent=5)
        return out, lse, kept, new_len

    eager, captured = pool(), pool()
    want = step(eager)
    backup = [t.clone() for t in (captured.k, captured.v, captured.mass)]
    graph = torch.cuda.CUDAGraph()
    step(captured)  # what a first call loads is loaded before the capture
    with torch.cuda.graph(graph):
        got = step(captured)
    for t, b in zip((captured.k, captured.v, captured.mass), backup):
        t.copy_(b)
    graph.replay()
    torch.cuda.synchronize()
    no_device_error()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    for a, b in ((captured.k, eager.k), (captured.v, eager.v), (captured.mass, eager.mass)):
        assert torch.equal(torch.nan_to_num(a, nan=9.0), torch.nan_to_num(b, nan=9.0))


def test_two_calls_at_once():
    cs = [Case(41 + i, [700, 60, 129], [40, 3, 1], 2, 4, (128, 128), 32) for i in range(2)]
    qs = [c.q.to(DEV) for c in cs]
    st = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(10):
        for i in range(2):
            outs[i].append(csa.gqa_dense_paged(qs[i], cs[i].cache, cs[i].batch, cs[i].scale, stream=st[i]))
    torch.cuda.synchronize()
    no_device_error()
    for i in range(2):
        cs[i].check(*outs[i][0])
        for out, lse in outs[i][1:]:
            assert torch.equal(out, outs[i][0][0]) and torch.equal(lse, outs[i][0][1])


@pytest.mark.parametrize("n", [1, 100])
def test_outputs_and_scratch_on_16_byte_boundaries_only(n):
    c = Case(43, [700], [n], 2, 4, (128, 128), 32)
    buf = torch.empty(n * 8 * 128 + 8, dtype=torch.bfloat16, device=DEV)
    out = buf[8:].view(n, 8, 128)
    ws = torch.empty(csa.gqa_dense_workspace_size(n, 8, 2, 128) + 16, dtype=torch.uint8, device=DEV)[16:]
    assert out.data_ptr() % 32 == 16 and ws.data_ptr() % 32 == 16
    c.check(*csa.gqa_dense_paged(c.q.to(DEV), c.cache, c.batch, c.scale, out=out, workspace=ws))
    no_device_error()


def test_pages_that_two_sequences_share():
    # a common prefix of two pages; each sequence continues on its own
    c = Case(44, [100, 100], [1, 1], 1, 4, (64, 64), 32)
    c.table[1, :2] = c.table[0, :2]
    c.batch.block_table.copy_(i32(c.table))
    q = c.q.to(DEV)
    out, lse = csa.gqa_dense_paged(q, c.cache, c.batch, c.scale)
    c.check(out, lse)
    before = f64(c.cache.mass)
    got = f64(csa.gqa_cache_mass(q, lse, c.cache, c.batch, c.scale)) - before
    add = [R.weights(f64(c.q[s:s + 1]), c.live(c.k, s), f64(lse[s:s + 1]), c.scale, 99)[0] for s in range(2)]
    for pg in range(2):
        want = add[0][32 * pg:32 * pg + 32] + add[1][32 * pg:32 * pg + 32]
        assert np.allclose(got[c.table[0, pg], 0], want, rtol=0, atol=2.0**-21)  # three additions near 1 in fp32
    no_device_error()


def test_evicting_a_page_outside_the_pool_reads_zeros():
    c = Case(45, [40], [0], 1, 1, (64, 64), 16)
    table = c.table.copy()
    table[0, 1] = 10**6
    P = c.k.shape[0]
    grow = [torch.cat([t, torch.full((2, *t.shape[1:]), 3.0, dtype=t.dtype)]).to(DEV) for t in (c.k, c.v, c.mass)]
    cache = csa.GqaCache(*grow)
    kept, _ = csa.gqa_cache_evict(cache, csa.GqaBatch(i32(table), i32([40]), None), 32, i32([[P, P + 1]]), recent=32)
    torch.cuda.synchronize()
    assert kept[0, 0].tolist() == list(range(8, 40))
    assert torch.equal(cache.k[P, 0, :8].cpu(), c.k[table[0, 0], 0, 8:])
    assert torch.all(cache.k[P, 0, 8:] == 0) and torch.all(cache.k[P + 1, 0, :8] == 0)
    assert torch.equal(cache.k[P + 1, 0, 8:16].cpu(), c.k[table[0, 2], 0, :8])


def test_wrong_tensors_are_refused():
    c = Case(46, [40], [2], 2, 2, (64, 64), 16)
    q = c.q.to(DEV)
    call = lambda **kw: csa.gqa_dense_paged(**{**dict(q=q, cache=c.cache, batch=c.batch, scale=0.1), **kw})  # noqa: E731
    with pytest.raises(ValueError, match="q must be"):
        call(q=q.float())
    with pytest.raises(ValueError, match="q must have shape"):
        call(q=q[:1])
    with pytest.raises(ValueError, match="contiguous"):
        call(q=q.transpose(0, 1).contiguous().transpose(0, 1))
    with pytest.raises(ValueError, match="cache.v"):
        call(cache=csa.GqaCache(c.cache.k, c.cache.v[:, :1].contiguous()))
    with pytest.raises(ValueError, match="block_table"):
        call(batch=csa.GqaBatch(c.batch.block_table.long(), c.batch.cache_len, c.batch.cu_q, 2, 2))
    with pytest.raises(ValueError, match="cache_len is on cpu"):
        call(batch=csa.GqaBatch(c.batch.block_table, c.batch.cache_len.cpu(), c.batch.cu_q, 2, 2))
    with pytest.raises(csa.CsaError, match="cu_q is NULL"):
        call(batch=csa.GqaBatch(c.batch.block_table, c.batch.cache_len, None, 2, 2))
    with pytest.raises(csa.CsaError, match="WORKSPACE"):
        call(workspace=torch.empty(64, dtype=torch.uint8, device=DEV))
    with pytest.raises(csa.CsaError, match="mass"):
        csa.gqa_cache_mass(q, torch.zeros(2, 4, device=DEV), csa.GqaCache(c.cache.k, c.cache.v), c.batch, 0.1)


def test_on_another_stream():
    c = Case(32, [1000, 20], [30, 20], 2, 4, (128, 128), 32)
    st = torch.cuda.Stream()
    q = c.q.to(DEV)
    torch.cuda.synchronize()
    outs = [csa.gqa_dense_paged(q, c.cache, c.batch, c.scale, stream=st) for _ in range(3)]
    st.synchronize()
    for out, lse in outs:
        c.check(out, lse)


@pytest.mark.parametrize("lens,n,Hkv,dims,page", [
    ([1], [1], 1, (64, 64), 16),
    ([40, 7, 130, 64], [1, 7, 100, 0], 3, (192, 128), 32),
    ([1000, 129], [999, 1], 40, (128, 128), 128),
])
def test_append(lens, n, Hkv, dims, page):
    c = Case(sum(lens), lens, n, Hkv, 1, dims, page, extra_rows=2)
    k, v = bf16(c.g, c.rows, Hkv, dims[0]), bf16(c.g, c.rows, Hkv, dims[1])
    want = [c.k.clone(), c.v.clone(), c.mass.clone()]
    for s, L in enumerate(lens):
        for i in range(n[s]):
            pos = L - n[s] + i
            pg, sl = c.table[s, pos // page], pos % page
            want[0][pg, :, sl], want[1][pg, :, sl], want[2][pg, :, sl] = k[c.cu[s] + i], v[c.cu[s] + i], 0.0
    csa.gqa_cache_append(k.to(DEV), v.to(DEV), c.cache, c.batch)
    torch.cuda.synchronize()
    no_device_error()
    for got, ref in zip((c.cache.k, c.cache.v, c.cache.mass), want):
        assert torch.equal(torch.nan_to_num(got.cpu(), nan=123.0), torch.nan_to_num(ref, nan=123.0))


def test_append_drops_rows_before_token_0_and_pages_outside_the_pool():
    c = Case(40, [2, 20], [4, 20], 2, 1, (64, 64), 16)
    c.batch.block_table[1, 1] = 10**6
    k, v = bf16(c.g, c.rows, 2, 64), bf16(c.g, c.rows, 2, 64)
    csa.gqa_cache_append(k.to(DEV), v.to(DEV), c.cache, c.batch)
    torch.cuda.synchronize()
    got = c.cache.k.cpu()
    assert torch.equal(got[c.table[0, 0], :, :2].transpose(0, 1), k[2:4])
    assert torch.equal(got[c.table[1, 0]].transpose(0, 1), k[4:20])
    assert torch.isnan(got[c.table[1, 1]][:, 4:].float()).all()  # and what followed is as it was


MASS = [
    ([1], [1], 1, 1, (128, 128), 16),
    ([777], [1], 2, 4, (128, 128), 16),
    ([127, 128, 129, 1], [1, 1, 1, 1], 2, 8, (64, 64), 32),
    ([300, 5, 600], [1, 1, 1], 1, 64, (192, 128), 128),
    ([260, 40, 17, 128], [7, 40, 0, 1], 2, 4, (192, 128), 64),
    ([700, 33], [150, 33], 2, 3, (128, 128), 16),
    ([0, 9, 400], [0, 9, 300], 1, 5, (64, 64), 16),
    ([600, 64], [2, 3], 1, 128, (64, 64), 64),
    ([3, 20], [5, 20], 1, 2, (128, 128), 16),
    ([900, 900], [64, 1], 3, 12, (128, 128), 128),
    ([190, 3], [5, 1], 1, 50, (128, 128), 16),
]


@pytest.mark.parametrize("lens,n,Hkv,G,dims,page", MASS)
def test_accumulated_weight(lens, n, Hkv, G, dims, page):
    c = Case(sum(lens) + G, lens, n, Hkv, G, dims, page, extra_rows=1)
    lse = np.full((c.rows, Hkv * G), np.nan, np.float32)
    for s, L in enumerate(lens):
        a, b = c.cu[s], c.cu[s + 1]
        lse[a:b] = R.attend(f64(c.q[a:b]), c.live(c.k, s), c.live(c.v, s), c.scale, L - (b - a))[1]
    got = f64(csa.gqa_cache_mass(c.q.to(DEV), torch.from_numpy(lse).to(DEV), c.cache, c.batch, c.scale))
    no_device_error()
    want, tol = f64(c.mass), np.zeros(c.mass.shape)
    for s, L in enumerate(lens):
        a, b = c.cu[s], c.cu[s + 1]
        qs, ks = f64(c.q[a:b]), c.live(c.k, s)
        add = R.weights(qs, ks, lse[a:b].astype(np.float64), c.scale, L - (b - a))
        # a weight's relative error, the sum of at most n G of them, and the addition to what was there
        rel = score_tol(dims[0], R.score_size(qs, ks, c.scale)) + (n[s] * G + 2) * 2.0**-24
        for j in range(max(L, 0)):
            pg, sl = c.table[s, j // page], j % page
            tol[pg, :, sl] = rel * add[:, j] + 2.0**-23 * (want[pg, :, sl] + add[:, j])
            want[pg, :, sl] += add[:, j]
    assert np.all(np.abs(got - want) <= tol), float((np.abs(got - want) - tol).max())


@pytest.mark.parametrize("lens,Hkv,dims,page,budget,sink,recent,width", [
    ([300, 64, 65, 0, 1], 2, (128, 128), 16, 64, 4, 16, None),
    ([500], 3, (192, 128), 128, 1, 0, 0, None),
    ([500, 77], 1, (64, 64), 32, 76, 0, 76, None),
    ([500, 77], 1, (64, 64), 32, 76, 76, 0, None),
    ([2100, 1030], 2, (64, 64), 64, 1029, 3, 100, None),
    ([40, 50], 2, (128, 128), 16, 200, 1, 1, None),
    ([9000, 30011, 4097], 1, (64, 64), 64, 3000, 4, 64, None),   # several blocks per list
    ([1500, 700, 3000], 2, (64, 64), 16, 640, 0, 1, 25000),      # a table too wide for keys to be held on chip
])
@pytest.mark.parametrize("kind", ["random", "equal", "few"])
def test_evict(lens, Hkv, dims, page, budget, sink, recent, width, kind):
    c = Case(sum(lens) + budget, lens, [0] * len(lens), Hkv, 1, dims, page, width=width)
    pages = -(-budget // page)
    P = c.k.shape[0]
    new = P + c.g.permutation(len(lens) * pages).reshape(len(lens), pages)
    more = len(lens) * pages
    k = torch.cat([c.k, torch.full((more, *c.k.shape[1:]), 5.0, dtype=torch.bfloat16)])
    v = torch.cat([c.v, torch.full((more, *c.v.shape[1:]), 5.0, dtype=torch.bfloat16)])
    mass = torch.cat([c.mass, torch.full((more, *c.mass.shape[1:]), 5.0)])
    if kind == "equal":
        mass[:P] = 0.25
    if kind == "few":  # few distinct values, signed zeros, infinities and NaN
        pick = torch.tensor([0.0, -0.0, 1.0, 1.0, 2.0, 3.5, float("inf"), float("nan"), 1e-42])
        mass[:P] = pick[torch.from_numpy(c.g.integers(0, len(pick), mass[:P].shape))]
    cache = csa.GqaCache(k.to(DEV), v.to(DEV), mass.to(DEV))
    batch = csa.GqaBatch(i32(c.table), i32(lens), None)
    kept, new_len = csa.gqa_cache_evict(cache, batch, budget, i32(new), sink=sink, recent=recent)
    torch.cuda.synchronize()
    no_device_error()
    for s, L in enumerate(lens):
        assert int(new_len[s]) == min(L, budget)
        for h in range(Hkv):
            ids = R.keep(R.live(mass.numpy(), c.table[s], L)[:, h], budget, sink, recent)
            assert kept[s, h].tolist() == ids + [-1] * (budget - len(ids)), (s, h)
            for plane in ("k", "v", "mass"):
                src = {"k": k, "v": v, "mass": mass}[plane]
                for i, j in enumerate(ids):
                    src[new[s, i // page], h, i % page] = src[c.table[s, j // page], h, j % page]
    for got, ref in zip((cache.k, cache.v, cache.mass), (k, v, mass)):
        assert torch.equal(torch.nan_to_num(got.cpu(), nan=77.0), torch.nan_to_num(ref, nan=77.0))


def test_a_prompt_its_chunks_and_an_eviction_in_sequence():
    """Prompt -> cache -> decode steps -> accumulated weight -> eviction -> decode over what is kept, against the
    oracle fed with the same stored numbers."""
    g = np.random.default_rng(77)
    Hkv, G, dims, page, budget = 2, 4, (128, 128), 16, 48
    H, scale = Hkv * G, 0.11
    prompt = [90, 33]
    P = 40
    cache = csa.GqaCache(torch.full((P, Hkv, page, 128), float("nan"), dtype=torch.bfloat16, device=DEV),
                         torch.full((P, Hkv, page, 128), float("nan"), dtype=torch.bfloat16, device=DEV),
                         torch.full((P, Hkv, page), float("nan"), device=DEV))
    order = g.permutation(P)
    table, new = order[:16].reshape(2, 8).astype(np.int32), order[16:24].reshape(2, 4).astype(np.int32)
    ks, vs, mass = [None, None], [None, None], [None, None]

    def step(n, tab, lens):
        cu = [0, n[0], n[0] + n[1]]
        q, k, v = bf16(g, cu[2], H, 128), bf16(g, cu[2], Hkv, 128), bf16(g, cu[2], Hkv, 128)
        batch = csa.GqaBatch(i32(tab), i32(lens), i32(cu), max_q=max(n), total_q=cu[2])
        csa.gqa_cache_append(k.to(DEV), v.to(DEV), cache, batch)
        out, lse = csa.gqa_dense_paged(q.to(DEV), cache, batch, scale)
        csa.gqa_cache_mass(q.to(DEV), lse, cache, batch, scale)
        torch.cuda.synchronize()
        no_device_error()
        for s in range(2):
            a, b = cu[s], cu[s + 1]
            new_k, new_v = f64(k[a:b]), f64(v[a:b])
            if mass[s] is None:
                ks[s], vs[s], mass[s] = new_k, new_v, np.zeros((Hkv, 0))
            else:
                ks[s], vs[s] = np.concatenate([ks[s], new_k]), np.concatenate([vs[s], new_v])
            mass[s] = np.concatenate([mass[s], np.zeros((Hkv, b - a))], 1)
            ref, rl, size = R.attend(f64(q[a:b]), ks[s], vs[s], scale, lens[s] - (b - a))
            check_out(f64(out[a:b]), ref, size, f"step {n}")
            mass[s] += R.weights(f64(q[a:b]), ks[s], f64(lse[a:b]), scale, lens[s] - (b - a))
        if n == prompt:
            direct = csa.gqa_dense_packed(q.to(DEV), k.to(DEV), v.to(DEV), csa.Packed(n, 1), scale)
            assert torch.equal(direct[0], out) and torch.equal(direct[1], lse)
        return batch

    lens = list(prompt)
    step(prompt, table, lens)
    for n in ([1, 1], [3, 1], [1, 2]):
        lens = [L + m for L, m in zip(lens, n)]
        batch = step(n, table, lens)
    kept, new_len = csa.gqa_cache_evict(cache, batch, budget, i32(new), sink=2, recent=8)
    torch.cuda.synchronize()
    for s in range(2):
        held = R.live(f64(cache.mass), new[s], int(new_len[s]))
        for h in range(Hkv):
            ids = [j for j in kept[s, h].tolist() if j >= 0]
            assert len(ids) == min(lens[s], budget) and ids == sorted(set(ids))
            assert np.allclose(held[:, h], mass[s][h, ids], rtol=1e-4, atol=1e-6)
        # the heads keep different tokens: the oracle's cache is cut per head
        ids = np.array([[j for j in kept[s, h].tolist() if j >= 0] for h in range(Hkv)])
        ks[s] = np.stack([ks[s][ids[h], h] for h in range(Hkv)], 1)
        vs[s] = np.stack([vs[s][ids[h], h] for h in range(Hkv)], 1)
        mass[s] = np.stack([mass[s][h, ids[h]] for h in range(Hkv)])
    lens = [int(x) for x in new_len]
    for n in ([1, 1], [2, 5]):
        lens = [L + m for L, m in zip(lens, n)]
        step(n, new, lens)
