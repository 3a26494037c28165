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
