"""Accumulated weight and grouped-head attention where their arithmetic can go wrong: large weights, single exponentials
to the exponential unit's accuracy.

ex2.approx is off by at most 2^-22 relative; a product or sum in fp32 by 2^-24, a constant rounded to fp32 likewise."""
import math

import numpy as np
import pytest
import torch

import long_context_sparse_10_b200 as csa
from oracle import gqa_ref as R
from test_gpu_gqa import DEV, DIMS, Case, bf16, check_lse, check_out, f64, i32, no_device_error, score_tol

pytestmark = pytest.mark.gpu


def one_channel(values, d):
    """Keys or queries [..., d] whose channel 0 holds the values: their products are exact."""
    t = torch.zeros(*values.shape, d)
    t[..., 0] = values
    return t.to(torch.bfloat16)


def close_or_infinite(got, want, tol):
    """The worst relative error of what fp32 holds; what it does not hold has to be +inf."""
    top = float(np.finfo(np.float32).max)
    assert bool(np.all(np.isposinf(got[want > top * (1 + tol)])))
    held = want < top * (1 - tol)
    worst = float(np.abs(got[held] / want[held] - 1).max()) if held.any() else 0.0
    assert worst <= tol, f"{worst:.3e}, {tol:.3e} allowed"


@pytest.mark.parametrize("dims", DIMS)
@pytest.mark.parametrize("lse", [-60.0, -86.0, -95.0, -200.0, -1e30])
def test_weights_of_an_lse_far_below_the_scores(dims, lse):
    # an lse that is not the rows' own: weights of e^(score - lse), which leave fp32 above e^88.7
    n, G, L, page = 32, 4, 300, 32
    c = Case(5, [L], [n], 1, G, dims, page)
    c.cache.k.zero_()
    c.cache.mass.zero_()
    q = torch.zeros(n, G, dims[0], dtype=torch.bfloat16, device=DEV)
    got = csa.gqa_cache_mass(q, torch.full((n, G), lse, device=DEV), c.cache, c.batch, 1.0)
    no_device_error()
    rows = np.array([min(n, L - j) for j in range(L)]) * G
    # the exponent -lse log2(e) is rounded (twice 2^-24 of up to 124.1, in units of ln 2), the unit 2^-22, 128 sums
    tol = (2 * 124.1 * math.log(2) + 4 + 128) * 2.0**-24
    close_or_infinite(R.live(f64(got), c.table[0], L)[:, 0], rows * np.exp(min(-lse, 700.0)), tol)


@pytest.mark.parametrize("lse", [-60.0, -86.0, -95.0, -178.0, -200.0, -1e30])
def test_one_weight_of_an_lse_far_below_the_scores(lse):
    # of 64 rows, one row of each 16 in turn; the others weigh e^-80
    n, L, page, d = 64, 200, 16, 64
    pages = -(-L // page)
    q = torch.zeros(n, 1, d, dtype=torch.bfloat16, device=DEV)
    k = torch.zeros(pages, 1, page, d, dtype=torch.bfloat16, device=DEV)
    batch = csa.GqaBatch(i32(np.arange(pages)[None]), i32([L]), i32([0, n]), max_q=n, total_q=n)
    tol = (2 * 124.1 * math.log(2) + 4 + 2) * 2.0**-24
    for row in range(16):
        mass = torch.zeros(pages, 1, page, device=DEV)
        at = torch.full((n, 1), 80.0, device=DEV)
        at[row] = lse
        csa.gqa_cache_mass(q, at, csa.GqaCache(k, k, mass), batch, 1.0)
        close_or_infinite(f64(mass).reshape(-1)[: L - n], np.full(L - n, np.exp(min(-lse, 700.0))), tol)
    no_device_error()


def test_a_weight_is_as_exact_as_the_exponential_unit():
    # 64 rows of one head; all but one weigh e^-80.  Every column of a 16-column run in turn, exponents in [-1, 1].
    n, L, page, d = 64, 200, 16, 128
    g = np.random.default_rng(3)
    x = torch.from_numpy(g.uniform(-1, 1, L).astype(np.float32)).to(torch.bfloat16).float()
    pages = -(-L // page)
    k = torch.zeros(pages, 1, page, d, dtype=torch.bfloat16)
    k.view(-1, d)[:L] = one_channel(x, d)
    v = torch.zeros_like(k)
    q = one_channel(torch.ones(n, 1), d).to(DEV)
    # exponent: scale log2(e) rounded (2 2^-24 relative, |x| <= 1), the fused product and sum 2^-24; the unit; the sum
    tol = (3 * math.log(2) + 4 + 2) * 2.0**-24
    for row in range(16):
        cache = csa.GqaCache(k.to(DEV), v.to(DEV), torch.zeros(pages, 1, page, device=DEV))
        batch = csa.GqaBatch(i32(np.arange(pages)[None]), i32([L]), i32([0, n]), max_q=n, total_q=n)
        lse = torch.full((n, 1), 80.0, device=DEV)
        lse[row] = 0.0
        got = f64(csa.gqa_cache_mass(q, lse, cache, batch, 1.0)).reshape(-1)[: L - n]
        want = np.exp(f64(x))[: L - n]
        worst = float(np.abs(got / want - 1).max())
        assert worst <= tol, f"row {row}: {worst:.3e}, {tol:.3e} allowed"
    no_device_error()


@pytest.mark.parametrize("dims", DIMS)
def test_lse_of_a_decode_step_is_as_exact_as_the_exponential_unit(dims):
    # Two keys count: one of score 0 in the first tile, one of score x ln 2, 1 <= x < 2, in the third (the same stream,
    # and not far enough above to move the reference); the others weigh nothing.  Many copies, so that most items are
    # one CTA's.
    L, page, copies, scale = 384, 128, 40, math.log(2)
    xs = [1 + i / 32 for i in range(32)]
    score = torch.full((len(xs), L), -5000.0)
    score[:, 0] = 0.0
    for i, x in enumerate(xs):
        score[i, 256 + 12 + i % 4 + 16 * (i % 8)] = x
    k = one_channel(score.view(len(xs) * 3, 1, page), dims[0])
    v = torch.zeros(len(xs) * 3, 1, page, dims[1], dtype=torch.bfloat16)
    n = len(xs) * copies
    table = np.arange(len(xs) * 3).reshape(-1, 3)[np.arange(n) % len(xs)]
    cache = csa.GqaCache(k.to(DEV), v.to(DEV))
    batch = csa.GqaBatch(i32(table), i32([L] * n), i32(range(n + 1)), max_q=1, total_q=n)
    q = one_channel(torch.ones(n, 1), dims[0]).to(DEV)
    _, lse = csa.gqa_dense_paged(q, cache, batch, scale)
    no_device_error()
    want = np.log1p(np.exp(np.array(xs) * float(np.float32(scale))))[np.arange(n) % len(xs)]
    # in log2 units and 2^-24: scale log2(e) 2 x; the exponent's rounding x; the unit 4 log2(e); the sum log2(e); log2f
    # (1 ulp below 4) 4; the result's sum and product with a rounded ln 2, below 2.33, 3 * 2.33: below 2^-19 all in all
    tol = math.log(2) * (2 * 2 + 2 + 5 * 1.4427 + 4 + 3 * 2.33) * 2.0**-24
    err = np.abs(f64(lse)[:, 0] - want)
    assert err.max() <= tol, f"{err.max():.3e}, {tol:.3e} allowed, at x = {xs[int(err.argmax()) % len(xs)]}"


@pytest.mark.parametrize("dims", DIMS)
def test_a_score_of_minus_infinity_weighs_nothing(dims):
    # keys whose product with every query is -inf, at both ends of tiles and of what a row sees; the rows that see no
    # other key have out 0 and lse -inf
    L, G, scale = 420, 2, 0.09
    bad = [0, 1, 63, 64, 127, 128, 129, 200, 255, 300, 419]
    g = np.random.default_rng(17)
    q, k, v = bf16(g, L, G, dims[0]), bf16(g, L, 1, dims[0]), bf16(g, L, 1, dims[1])
    q[:, :, 0] = q[:, :, 0].abs() + 0.5
    k[bad, 0, 0] = -math.inf
    out, lse = csa.gqa_dense_packed(q.to(DEV), k.to(DEV), v.to(DEV), csa.Packed([L], 1), scale)
    no_device_error()
    out, lse = f64(out), f64(lse)
    assert np.all(out[:2] == 0) and np.all(np.isneginf(lse[:2]))
    good = [j for j in range(L) if j not in bad]
    kg, vg = f64(k[good]), f64(v[good])
    for t in range(2, L):
        m = sum(j <= t for j in good)
        qs = f64(q[t:t + 1])
        ref, rl, size = R.attend(qs, kg, vg, scale, m - 1)
        check_out(out[t:t + 1], ref, size, f"row {t}")
        check_lse(lse[t:t + 1], rl, score_tol(dims[0], R.score_size(qs, kg[:m], scale)), f"row {t}")


@pytest.mark.parametrize("dims", DIMS)
@pytest.mark.parametrize("value", [float("nan"), math.inf, -math.inf])
def test_a_key_that_is_not_finite_in_a_long_cache(dims, value):
    # a decode step whose keys are shared out over many CTAs: the one key shows in the row, or weighs nothing
    L, G, page = 5000, 4, 64
    for at in (0, 130, 2500, 4999):
        c = Case(19, [L], [1], 1, G, dims, page)
        c.q[:, :, 0] = c.q[:, :, 0].abs() + 0.5
        c.cache.k[c.table[0, at // page], 0, at % page, 0] = value
        out, lse = csa.gqa_dense_paged(c.q.to(DEV), c.cache, c.batch, c.scale)
        before = c.cache.mass.clone()
        mass = csa.gqa_cache_mass(c.q.to(DEV), lse, c.cache, c.batch, c.scale)
        no_device_error()
        if value == -math.inf:
            ks, vs = np.delete(c.live(c.k, 0), at, 0), np.delete(c.live(c.v, 0), at, 0)
            ref, rl, size = R.attend(f64(c.q), ks, vs, c.scale, L - 2)
            check_out(f64(out), ref, size, f"key {at}")
            check_lse(f64(lse), rl, score_tol(dims[0], R.score_size(f64(c.q), ks, c.scale)), f"key {at}")
            pg, sl = c.table[0, at // page], at % page
            assert float(mass[pg, 0, sl]) == float(before[pg, 0, sl])
        else:
            assert bool(torch.isnan(out).all()) and bool(torch.isnan(lse).all()), at


def test_items_in_which_a_stream_has_no_tile_against_the_oracle():
    # decode rows of one key tile give the second stream nothing, and so do chunks whose keys end in their first tile:
    # the idle stream's accumulator, reference and sum, left by an item before, count for nothing
    for seed, (L, n) in enumerate(((100, 1), (128, 1), (129, 2), (257, 1), (40, 40), (300, 70))):
        lens = [max(n, L - i % 7) for i in range(200)]
        c = Case(60 + seed, lens, [n] * 200, 1, 4, (64, 64), 16)
        out, lse = csa.gqa_dense_paged(c.q.to(DEV), c.cache, c.batch, c.scale)
        torch.cuda.synchronize()
        no_device_error()
        out, lse = f64(out), f64(lse)
        for s in range(200):
            a, b = c.cu[s], c.cu[s + 1]
            rows = sorted({a, (a + b) // 2, b - 1})  # first, middle and last row of each sequence
            qs, ks, vs = f64(c.q[a:b]), c.live(c.k, s), c.live(c.v, s)
            for r in rows:
                ref, rl, size = R.attend(qs[r - a:r - a + 1], ks, vs, c.scale, lens[s] - (b - a) + r - a)
                check_out(out[r:r + 1], ref, size, f"{(L, n)} sequence {s}")
                check_lse(lse[r:r + 1], rl, score_tol(64, R.score_size(qs, ks, c.scale)), f"{(L, n)} sequence {s}")


def attend64(q, k, v, scale):
    """Causal attention of one prompt in 64 bits on the device: out, lse, the softmax mean of |v|, and for each row the
    largest scale * sum |q_c k_c|; a query head at a time."""
    n, H, _ = q.shape
    G = H // k.shape[1]
    hidden = torch.ones(n, n, dtype=torch.bool, device=q.device).triu(1)
    out, lse, mean, size = [], [], [], 0.0
    for h in range(H):
        qh, kh, vh = q[:, h].double(), k[:, h // G].double(), v[:, h // G].double()
        x = (scale * (qh @ kh.T)).masked_fill(hidden, -math.inf)
        m = torch.logsumexp(x, 1)
        p = torch.exp(x - m[:, None])
        out.append(p @ vh)
        mean.append(p @ vh.abs())
        lse.append(m)
        size = max(size, scale * float((qh.abs() @ kh.abs().T).max()))
    return torch.stack(out, 1), torch.stack(lse, 1), torch.stack(mean, 1), size


@pytest.mark.parametrize("lens,Hkv,G,dims", [
    ([4001], 2, 1, (128, 128)),
    ([4001], 1, 4, (192, 128)),
    ([2600, 1700, 3], 2, 2, (64, 64)),
    ([1300, 2050], 1, 12, (128, 128)),
    ([1600], 1, 8, (64, 64)),
])
def test_every_row_of_long_prompts_and_their_weight(lens, Hkv, G, dims):
    """Whole prompts against 64 bits, row by row, and the weight that all their rows give their tokens."""
    g = np.random.default_rng(sum(lens))
    page, scale, n = 64, 1 / math.sqrt(dims[0]), sum(lens)
    q, k, v = (t.to(DEV) for t in (bf16(g, n, Hkv * G, dims[0]), bf16(g, n, Hkv, dims[0]), bf16(g, n, Hkv, dims[1])))
    out, lse = csa.gqa_dense_packed(q, k, v, csa.Packed(lens, 1), scale)
    need = [-(-L // page) for L in lens]
    P = sum(need)
    order = iter(g.permutation(P))
    table = np.zeros((len(lens), max(need)), np.int32)
    for s, c in enumerate(need):
        table[s, :c] = [next(order) for _ in range(c)]
    cache = csa.GqaCache(*[torch.full((P, Hkv, page, d), float("nan"), dtype=torch.bfloat16, device=DEV) for d in dims],
                         torch.full((P, Hkv, page), float("nan"), device=DEV))
    cu = np.concatenate([[0], np.cumsum(lens)])
    batch = csa.GqaBatch(i32(table), i32(lens), i32(cu), max_q=max(lens), total_q=n)
    csa.gqa_cache_append(k, v, cache, batch)
    mass = csa.gqa_cache_mass(q, lse, cache, batch, scale)
    again = csa.GqaCache(cache.k, cache.v, torch.zeros_like(mass))
    csa.gqa_cache_mass(q, lse, again, batch, scale)
    torch.cuda.synchronize()
    no_device_error()
    for s, L in enumerate(lens):
        a, b = cu[s], cu[s + 1]
        ref, rl, mean, size = attend64(q[a:b], k[a:b], v[a:b], scale)
        check_out(f64(out[a:b]), f64(ref), f64(mean), f"sequence {s}")
        check_lse(f64(lse[a:b]), f64(rl), score_tol(dims[0], size), f"sequence {s}")
        add = torch.zeros(Hkv, L, dtype=torch.float64, device=DEV)
        hidden = torch.ones(L, L, dtype=torch.bool, device=DEV).triu(1)
        for h in range(Hkv * G):  # with the rows' own lse, as the call has it
            x = scale * (q[a:b, h].double() @ k[a:b, h // G].double().T) - lse[a:b, h].double()[:, None]
            add[h // G] += torch.exp(x.masked_fill(hidden, -math.inf)).sum(0)
        got = R.live(f64(mass), table[s], L).T
        # a weight's relative error and a sum of at most L G of them (four partial sums a block of rows, then the blocks)
        rel = score_tol(dims[0], size) + (128 // 4 + 4 + L * G // (128 // G * G) + 2) * 2.0**-24
        worst = float((np.abs(got - f64(add)) / f64(add)).max())
        assert worst <= rel, f"sequence {s}: {worst:.3e}, {rel:.3e} allowed"
        assert np.array_equal(R.live(f64(again.mass), table[s], L).T, got)  # the same bits every time


@pytest.mark.parametrize("lens,n,Hkv,G,dims", [
    ([1500, 700, 2049, 130], [4, 2, 8, 3], 2, 8, (128, 128)),   # one tile of rows
    ([1500, 700, 2049, 130], [8, 5, 8, 1], 1, 32, (64, 64)),    # two
    ([1200, 640], [5, 6], 2, 1, (192, 128)),
])
def test_a_few_new_rows_a_sequence(lens, n, Hkv, G, dims):
    c = Case(70 + G, lens, n, Hkv, G, dims, 64)
    out, lse = csa.gqa_dense_paged(c.q.to(DEV), c.cache, c.batch, c.scale)
    torch.cuda.synchronize()
    no_device_error()
    c.check(out, lse)


@pytest.mark.parametrize("dims", DIMS)
@pytest.mark.parametrize("top", [26, 31, 36, 64, 105])
def test_scores_far_beyond_the_exponent_range(dims, top):
    # scores of up to 2^top beside ordinary ones, row by row: a row is finite, one whose best key leads by more than fp32
    # can err on two scores (and e^-100 weighs nothing) is that key's value, and ordinary rows are as ordinary as ever
    L, G, scale = 700, 4, 0.09
    g = np.random.default_rng(top)
    power = g.integers(0, 2, (L, G)) * g.integers(0, top, (L, G)) * 1.0
    q = (bf16(g, L, G, dims[0]).float() * torch.from_numpy(2.0**power)[..., None]).to(torch.bfloat16).to(DEV)
    k, v = bf16(g, L, 1, dims[0]).to(DEV), bf16(g, L, 1, dims[1]).to(DEV)
    ref, rl, mean, _ = attend64(q, k, v, scale)
    size = scale * torch.einsum("thd,sd->ths", q.double().abs(), k[:, 0].double().abs()).amax(2)
    err = (dims[0] + 8) * 2.0**-23 * size
    x = scale * torch.einsum("thd,sd->ths", q.double(), k[:, 0].double())
    x = x.masked_fill(torch.ones(L, L, dtype=torch.bool, device=DEV).triu(1)[:, None], -math.inf)
    best = x.topk(2, 2).values
    sure = f64(((best[..., 0] - best[..., 1]) > 2 * err + 100)).astype(bool)
    near = power == 0  # scores as in every other test
    assert int(sure.sum()) > 100 and int(near.sum()) > 100
    table = np.arange(-(-L // 128))[None].astype(np.int32)
    pad = lambda t: torch.cat([t, t[: table.size * 128 - L]]).view(table.size, 128, 1, -1).transpose(1, 2).contiguous()  # noqa: E731
    cache = csa.GqaCache(pad(k), pad(v))
    calls = {"prompt": (0, csa.gqa_dense_packed(q, k, v, csa.Packed([L], 1), scale))}
    for n in (1, 3):  # the last rows as a decode step: their keys are shared out over several CTAs
        batch = csa.GqaBatch(i32(table), i32([L]), i32([0, n]), max_q=n, total_q=n)
        calls[f"last {n}"] = (L - n, csa.gqa_dense_paged(q[L - n:].contiguous(), cache, batch, scale))
    no_device_error()
    for what, (a, (out, lse)) in calls.items():
        out, lse = f64(out), f64(lse)
        assert bool(np.all(np.isfinite(out)) and np.all(np.isfinite(lse))), what
        pick = sure[a:] | near[a:]
        if pick.any():
            check_out(out[pick], f64(ref)[a:][pick], f64(mean)[a:][pick], what)
        worst = np.abs(lse - f64(rl)[a:]) / (f64(err)[a:] + 2.0**-18)
        assert float(worst.max()) <= 1.0, what
