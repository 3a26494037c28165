"""Refusals of the grouped-head calls (host side, nothing is enqueued) and the oracle's own reductions."""
import ctypes
import math

import numpy as np
import pytest

from long_context_sparse_10_b200 import _lib
from oracle import gqa_ref as R

INV, UNS, WS, OK = _lib.CSA_ERR_INVALID_ARG, _lib.CSA_ERR_UNSUPPORTED, _lib.CSA_ERR_WORKSPACE, _lib.CSA_OK


@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(_lib.LIB_PATH):
        from long_context_sparse_10_b200 import build
        build.build()
    return _lib.load()


def cache(**kw):
    f = dict(k=16, v=16, mass=16, n_pages=8, page_size=16, n_kv_heads=2, d_qk=128, d_v=128)
    f.update(kw)
    return _lib.GqaCacheDesc(**f)


def batch(**kw):
    f = dict(block_table=16, cache_len=16, cu_q=16, n_seqs=2, max_pages=4, max_q=1, reserved=0, total_q=2)
    f.update(kw)
    return _lib.GqaBatchDesc(**f)


def packed(**kw):
    f = dict(cu_tokens=16, cu_entries=None, n_seqs=1, max_tokens=4, total_tokens=4, total_entries=0)
    f.update(kw)
    return _lib.PackedDesc(**f)


def ref(x):
    return ctypes.byref(x)


def paged(lib, c=None, b=None, H=8, scale=0.1, q=16, out=16, lse=None, ws=None, nb=0):
    return lib.gqa_dense_paged(q, ref(c or cache()), ref(b or batch()), H, scale, out, lse, ws, nb, None)


def prompt(lib, p=None, H=8, Hk=2, d=(128, 128), scale=0.1, q=16, k=16, v=16, out=16, lse=None, ws=None, nb=0):
    return lib.gqa_dense_packed(q, k, v, ref(p or packed()), H, Hk, d[0], d[1], scale, out, lse, ws, nb, None)


def test_struct_layouts():
    assert ctypes.sizeof(_lib.GqaCacheDesc) == 3 * 8 + 8 + 4 * 4
    assert ctypes.sizeof(_lib.GqaBatchDesc) == 3 * 8 + 4 * 4 + 8


@pytest.mark.parametrize("kw,status,word", [
    (dict(H=7), INV, b"multiple of the kv heads"),
    (dict(H=0), INV, b"multiple of the kv heads"),
    (dict(H=258), UNS, b"at most 128"),
    (dict(scale=0.0), INV, b"scale"),
    (dict(scale=-1.0), INV, b"scale"),
    (dict(scale=math.nan), INV, b"scale"),
    (dict(scale=math.inf), INV, b"scale"),
    (dict(scale=1e-31), INV, b"scale"),
    (dict(scale=2e30), INV, b"scale"),
    (dict(c=cache(d_qk=96)), UNS, b"channel widths"),
    (dict(c=cache(d_qk=192, d_v=192)), UNS, b"channel widths"),
    (dict(c=cache(page_size=8)), INV, b"page_size"),
    (dict(c=cache(page_size=48)), INV, b"page_size"),
    (dict(c=cache(n_kv_heads=0)), INV, b"kv heads"),
    (dict(c=cache(n_pages=0)), INV, b"n_pages"),
    (dict(c=cache(n_pages=1 << 27)), INV, b"n_pages"),
    (dict(c=cache(k=None)), INV, b"k is NULL"),
    (dict(c=cache(v=8)), INV, b"not 16-byte aligned"),
    (dict(b=batch(reserved=1)), INV, b"reserved"),
    (dict(b=batch(n_seqs=-1)), INV, b"negative"),
    (dict(b=batch(max_pages=0)), INV, b"max_pages"),
    (dict(b=batch(max_pages=1 << 28)), INV, b"max_pages"),
    (dict(b=batch(max_q=0)), INV, b"max_q"),
    (dict(b=batch(total_q=1 << 31)), INV, b"total_q"),
    (dict(b=batch(block_table=None)), INV, b"block_table is NULL"),
    (dict(b=batch(cache_len=None)), INV, b"cache_len is NULL"),
    (dict(b=batch(cu_q=None)), INV, b"cu_q is NULL"),
    (dict(q=None), INV, b"q is NULL"),
    (dict(out=None), INV, b"out is NULL"),
    (dict(lse=4), INV, b"lse"),
])
def test_paged_refusals(lib, kw, status, word):
    assert paged(lib, **kw) == status
    assert word in lib.csa_last_error(), lib.csa_last_error()


@pytest.mark.parametrize("kw,status,word", [
    (dict(H=9), INV, b"multiple of the kv heads"),
    (dict(d=(128, 64)), UNS, b"channel widths"),
    (dict(scale=0.0), INV, b"scale"),
    (dict(p=packed(max_tokens=5)), INV, b"max_tokens"),
    (dict(p=packed(max_tokens=0)), INV, b"max_tokens"),
    (dict(p=packed(total_tokens=-1)), INV, b"total_tokens"),
    (dict(p=packed(cu_tokens=None)), INV, b"cu_tokens is NULL"),
    (dict(k=None), INV, b"k is NULL"),
    (dict(v=24), INV, b"not 16-byte aligned"),
])
def test_packed_refusals(lib, kw, status, word):
    assert prompt(lib, **kw) == status
    assert word in lib.csa_last_error(), lib.csa_last_error()


def test_null_structs(lib):
    assert lib.gqa_dense_paged(16, None, ref(batch()), 8, 0.1, 16, None, None, 0, None) == INV
    assert lib.gqa_dense_paged(16, ref(cache()), None, 8, 0.1, 16, None, None, 0, None) == INV
    assert lib.gqa_dense_packed(16, 16, 16, None, 8, 2, 128, 128, 0.1, 16, None, None, 0, None) == INV


def test_workspace(lib):
    need = lib.gqa_dense_workspace_size(1, 8, 2, 128)
    assert need > 0 and lib.gqa_dense_workspace_size(0, 8, 2, 128) == 0
    assert lib.gqa_dense_workspace_size(1 << 30, 8, 2, 128) > need
    assert paged(lib) == WS
    assert paged(lib, ws=16, nb=need - 1) == WS
    assert paged(lib, ws=8, nb=need) == INV
    assert prompt(lib) == WS
    assert b"workspace" in lib.csa_last_error()


def test_calls_without_rows_are_no_ops(lib):
    assert paged(lib, b=batch(total_q=0)) == OK
    assert paged(lib, b=batch(n_seqs=0)) == OK
    assert prompt(lib, p=packed(n_seqs=0)) == OK
    assert prompt(lib, p=packed(total_tokens=0, max_tokens=0)) == OK
    assert lib.gqa_cache_append(16, 16, ref(cache()), ref(batch(total_q=0)), None) == OK
    assert lib.gqa_cache_mass(16, 16, ref(cache()), ref(batch(n_seqs=0)), 8, 0.1, None) == OK
    assert lib.gqa_cache_evict(ref(cache()), ref(batch(n_seqs=0)), 16, 0, 0, 32, 1, 16, 32, None) == OK


def test_append_and_mass_refusals(lib):
    assert lib.gqa_cache_append(None, 16, ref(cache()), ref(batch()), None) == INV
    assert lib.gqa_cache_append(16, 8, ref(cache()), ref(batch()), None) == INV
    assert lib.gqa_cache_append(16, 16, ref(cache(mass=4)), ref(batch()), None) == INV
    assert lib.gqa_cache_mass(16, 16, ref(cache(mass=None)), ref(batch()), 8, 0.1, None) == INV
    assert b"mass" in lib.csa_last_error()
    assert lib.gqa_cache_mass(16, None, ref(cache()), ref(batch()), 8, 0.1, None) == INV
    assert lib.gqa_cache_mass(16, 16, ref(cache()), ref(batch()), 7, 0.1, None) == INV
    assert lib.gqa_cache_mass(16, 16, ref(cache()), ref(batch()), 8, -0.1, None) == INV


@pytest.mark.parametrize("kw,word", [
    (dict(budget=0), b"budget"),
    (dict(sink=-1), b"n_sink"),
    (dict(sink=10, recent=7), b"n_sink"),
    (dict(width=0), b"new table"),
    (dict(budget=17), b"new table"),
    (dict(table=16), b"the new table is the old one"),
    (dict(new_len=16), b"new_len is cache_len"),
    (dict(kept=None), b"kept is NULL"),
    (dict(c=cache(mass=None)), b"no mass"),
])
def test_evict_refusals(lib, kw, word):
    a = dict(c=cache(), b=batch(), budget=16, sink=0, recent=0, table=32, width=1, kept=16, new_len=32)
    a.update(kw)
    st = lib.gqa_cache_evict(ref(a["c"]), ref(a["b"]), a["budget"], a["sink"], a["recent"], a["table"], a["width"],
                             a["kept"], a["new_len"], None)
    assert st == INV and word in lib.csa_last_error(), lib.csa_last_error()


def test_cpu_tensors_are_refused():
    import torch

    import long_context_sparse_10_b200 as csa
    z = lambda *s, t=torch.bfloat16: torch.zeros(*s, dtype=t)  # noqa: E731
    cache = csa.GqaCache(z(2, 1, 16, 64), z(2, 1, 16, 64), z(2, 1, 16, t=torch.float32))
    bat = csa.GqaBatch(z(1, 1, t=torch.int32), z(1, t=torch.int32), z(2, t=torch.int32), 1, 1)
    for call in (lambda: csa.gqa_dense_paged(z(1, 1, 64), cache, bat, 0.1),
                 lambda: csa.gqa_cache_append(z(1, 1, 64), z(1, 1, 64), cache, bat),
                 lambda: csa.gqa_cache_mass(z(1, 1, 64), z(1, 1, t=torch.float32), cache, bat, 0.1),
                 lambda: csa.gqa_cache_evict(cache, bat, 16, z(1, 1, t=torch.int32))):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_the_oracle_row_by_row():
    g = np.random.default_rng(0)
    q, k, v = g.standard_normal((3, 4, 8)), g.standard_normal((5, 2, 8)), g.standard_normal((5, 2, 6))
    out, lse, _ = R.attend(q, k, v, 0.3, 2)
    x = np.array([0.3 * sum(q[1, 3, c] * k[j, 1, c] for c in range(8)) for j in range(4)])
    p = np.exp(x) / np.exp(x).sum()
    assert np.allclose(out[1, 3], sum(p[j] * v[j, 1] for j in range(4)))
    assert np.isclose(lse[1, 3], math.log(np.exp(x).sum()))
    # weights over all keys sum to the rows of the group
    assert np.allclose(R.weights(q, k, lse, 0.3, 2).sum(1), 3 * 2)
    # a row before token 0 sees nothing
    out, lse, _ = R.attend(q, k, v, 0.3, -1)
    assert np.all(out[0] == 0) and np.all(np.isneginf(lse[0])) and np.all(np.isfinite(lse[1]))


def test_the_oracle_keeps_ties_low():
    m = np.array([9.0, 1.0, 2.0, 2.0, 2.0, 0.0, np.nan, 5.0])
    assert R.keep(m, 4, 1, 1) == [0, 2, 6, 7]
    assert R.keep(m, 5, 0, 0) == [0, 2, 3, 6, 7]
    assert R.keep(m, 8, 0, 0) == list(range(8))
