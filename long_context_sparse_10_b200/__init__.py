"""B200-native Compressed Sparse Attention (CSA) and Heavily Compressed Attention (HCA).

Thin Python binding over the C ABI of ``libcsa.so`` (declared in include/csa.h).
Every function here only checks tensor metadata, allocates outputs and scratch
with torch (device memory is torch's job here) and calls the library entry point
of the same name; all arithmetic runs in the library's CUDA kernels.  There is
no CPU or PyTorch fallback: a missing library raises.

Shapes (B sequences, Tq query rows, N entries, H heads in {16, 64}):
  csa_compress / hca_compress: x bf16 [B, T, d] -> bf16 [B, N, d], or with
      ``fp8=True`` (d == 192) the split cache (nope e4m3 as uint8 [B, N, 128],
      rope bf16 [B, N, 64], scale fp32 [B, N]).
  csa_indexer_topk: qI bf16 [B, Tq, 4, 64], wI fp32 [B, Tq, 4], kIc bf16
      [B, N, 64] -> idx int32 [B, Tq, k] (ascending, -1 padded).
  csa_sparse_mqa / hca_dense_mqa: q bf16 [B, Tq, H, 192] -> (out bf16
      [B, Tq, H, 128], lse fp32 [B, Tq, H]).
  grouped_out_proj: out bf16 [..., H, 128], w bf16 [G, d_g, (H/G)*128] ->
      y bf16 [..., G, d_g].
  gqa_dense_packed: q bf16 [tokens, H, d_qk], k bf16 [tokens, H_kv, d_qk], v
      bf16 [tokens, H_kv, d_v] -> (out bf16 [tokens, H, d_v], lse fp32
      [tokens, H]); H a multiple of H_kv, (d_qk, d_v) = (192, 128), (128, 128)
      or (64, 64).
  gqa_dense_paged: q bf16 [new tokens, H, d_qk] over a GqaCache of pages
      [n_pages, H_kv, page_size, d]; gqa_cache_append, gqa_cache_mass and
      gqa_cache_evict fill it, weigh its tokens and cut it down.
"""
from __future__ import annotations

import ctypes
import dataclasses

import torch

from . import _lib

__all__ = ["CsaError", "KVCache", "Window", "csa_compress", "hca_compress", "csa_indexer_topk", "csa_indexer_topk_e4m3",
           "csa_indexer_topk_workspace_size", "csa_sparse_mqa", "csa_sparse_mqa_workspace_size", "hca_dense_mqa",
           "hca_dense_mqa_workspace_size", "grouped_out_proj", "launch_count", "version", "Packed", "csa_compress_append",
           "hca_compress_append", "csa_compress_packed", "hca_compress_packed", "csa_indexer_topk_packed",
           "csa_sparse_mqa_packed", "hca_dense_mqa_packed", "csa_indexer_topk_e2m1", "GqaCache", "GqaBatch",
           "gqa_dense_workspace_size", "gqa_dense_packed", "gqa_dense_paged", "gqa_cache_append", "gqa_cache_mass",
           "gqa_cache_evict"]


class CsaError(RuntimeError):
    def __init__(self, status: int, where: str):
        lib = _lib.load()
        msg = lib.csa_last_error().decode()
        super().__init__(f"{where}: {lib.csa_status_string(status).decode()} ({msg})")
        self.status = status


def _check(status: int, where: str):
    if status != _lib.CSA_OK:
        raise CsaError(status, where)


def _ptr(t: torch.Tensor | None):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensor must live on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def version() -> str:
    return _lib.load().csa_version().decode()


def launch_count() -> int:
    """Kernels the library has enqueued in this process (graph captures count once)."""
    return int(_lib.load().csa_launch_count())


@dataclasses.dataclass
class KVCache:
    """A compressed cache: bf16 (k, optional v) or split FP8 (nope, rope, scale)."""
    k: torch.Tensor | None = None
    v: torch.Tensor | None = None
    nope: torch.Tensor | None = None
    rope: torch.Tensor | None = None
    scale: torch.Tensor | None = None

    @property
    def split(self) -> bool:
        return self.nope is not None

    @property
    def n_entries(self) -> int:
        # entries per sequence ([B, N, ...]), or all entries of packed sequences ([total_entries, ...])
        return (self.nope if self.split else self.k).shape[-2]

    def desc(self) -> _lib.KVCacheDesc:
        d = _lib.KVCacheDesc()
        d.layout = _lib.CSA_KV_SPLIT_FP8 if self.split else _lib.CSA_KV_BF16
        d.reserved = 0
        d.n_entries = self.n_entries
        d.k, d.v = _ptr(self.k), _ptr(self.v)
        d.nope, d.rope, d.scale = _ptr(self.nope), _ptr(self.rope), _ptr(self.scale)
        return d


@dataclasses.dataclass
class Window:
    """Raw tokens for the sliding-window branch: rows hold positions pos0, pos0+1, ..."""
    k: torch.Tensor | None
    v: torch.Tensor | None = None
    pos0: int = 0
    length: int = 128

    def desc(self) -> _lib.WindowDesc:
        d = _lib.WindowDesc()
        d.k, d.v = _ptr(self.k), _ptr(self.v)
        d.pos0 = self.pos0
        # rows per sequence ([B, rows, 192]), or all packed tokens ([total_tokens, 192])
        d.rows = 0 if self.k is None else self.k.shape[-2]
        d.len = self.length
        d.reserved = 0
        return d


def _compress(fn_name, x, w, b_pos, stride, fp8, out, stream):
    lib = _lib.load()
    B, T, d = x.shape
    N = -(-T // stride)
    if fp8:
        nope, rope, scale = out if out is not None else (
            torch.empty(B, N, 128, dtype=torch.uint8, device=x.device),
            torch.empty(B, N, 64, dtype=torch.bfloat16, device=x.device),
            torch.empty(B, N, dtype=torch.float32, device=x.device))
        st = getattr(lib, fn_name)(_ptr(x), B, T, d, stride, _ptr(w), _ptr(b_pos), _lib.CSA_KV_SPLIT_FP8,
                                   _ptr(nope), _ptr(rope), _ptr(scale), _stream(stream))
        _check(st, fn_name)
        return nope, rope, scale
    y = out if out is not None else torch.empty(B, N, d, dtype=torch.bfloat16, device=x.device)
    st = getattr(lib, fn_name)(_ptr(x), B, T, d, stride, _ptr(w), _ptr(b_pos), _lib.CSA_KV_BF16, _ptr(y), None,
                               None, _stream(stream))
    _check(st, fn_name)
    return y


def csa_compress(x, w, b_pos, m, *, fp8=False, out=None, stream=None):
    """CSA compression: overlapping 2m-token windows with stride m."""
    return _compress("csa_compress", x, w, b_pos, m, fp8, out, stream)


def hca_compress(x, w, b_pos, m_prime, *, fp8=False, out=None, stream=None):
    """HCA compression: non-overlapping m'-token windows."""
    return _compress("hca_compress", x, w, b_pos, m_prime, fp8, out, stream)


def csa_indexer_topk_workspace_size(B, Tq, N, k) -> int:
    return int(_lib.load().csa_indexer_topk_workspace_size(B, Tq, N, k))


def csa_indexer_topk_coded_workspace_size(B, Tq, N, k) -> int:
    """Workspace of the E4M3 / E2M1 key calls and of csa_indexer_topk_with_scores."""
    return int(_lib.load().csa_indexer_topk_coded_workspace_size(B, Tq, N, k))


def csa_indexer_topk(qI, wI, kIc, m, k, *, q_pos0=0, idx=None, workspace=None, stream=None):
    """Lightning-indexer scores and top-k entry ids (int32 [B, Tq, k], ascending, -1 padded)."""
    lib = _lib.load()
    B, Tq = qI.shape[0], qI.shape[1]
    N = kIc.shape[1]
    if idx is None:
        idx = torch.empty(B, Tq, k, dtype=torch.int32, device=qI.device)
    need = csa_indexer_topk_workspace_size(B, Tq, N, k)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=qI.device)
    st = lib.csa_indexer_topk(_ptr(qI), _ptr(wI), _ptr(kIc), B, Tq, N, q_pos0, m, k, _ptr(idx), _ptr(workspace),
                              workspace.numel(), _stream(stream))
    _check(st, "csa_indexer_topk")
    return idx


def csa_indexer_topk_e4m3(qI, wI, kI_codes, kI_scale, m, k, *, q_pos0=0, idx=None, workspace=None, stream=None):
    """csa_indexer_topk over FP8 keys: kI_codes uint8 [B, N, 64] (E4M3), kI_scale fp32 [B, N]."""
    lib = _lib.load()
    B, Tq = qI.shape[0], qI.shape[1]
    N = kI_codes.shape[1]
    if idx is None:
        idx = torch.empty(B, Tq, k, dtype=torch.int32, device=qI.device)
    need = csa_indexer_topk_coded_workspace_size(B, Tq, N, k)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=qI.device)
    st = lib.csa_indexer_topk_e4m3(_ptr(qI), _ptr(wI), _ptr(kI_codes), _ptr(kI_scale), B, Tq, N, q_pos0, m, k,
                                   _ptr(idx), _ptr(workspace), workspace.numel(), _stream(stream))
    _check(st, "csa_indexer_topk_e4m3")
    return idx


def csa_indexer_topk_e2m1(qI, wI, kI_codes, kI_scale, m, k, *, q_pos0=0, idx=None, workspace=None, stream=None):
    """csa_indexer_topk over FP4 keys: kI_codes uint8 [B, N, 32] (E2M1, two per byte, low nibble = even
    dimension), kI_scale fp32 [B, N]."""
    lib = _lib.load()
    B, Tq = qI.shape[0], qI.shape[1]
    N = kI_codes.shape[1]
    if idx is None:
        idx = torch.empty(B, Tq, k, dtype=torch.int32, device=qI.device)
    need = csa_indexer_topk_coded_workspace_size(B, Tq, N, k)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=qI.device)
    st = lib.csa_indexer_topk_e2m1(_ptr(qI), _ptr(wI), _ptr(kI_codes), _ptr(kI_scale), B, Tq, N, q_pos0, m, k,
                                   _ptr(idx), _ptr(workspace), workspace.numel(), _stream(stream))
    _check(st, "csa_indexer_topk_e2m1")
    return idx


def csa_sparse_mqa_workspace_size(B, Tq, H, k, win_len) -> int:
    return int(_lib.load().csa_sparse_mqa_workspace_size(B, Tq, H, k, win_len))


def hca_dense_mqa_workspace_size(B, Tq, H, N, win_len) -> int:
    return int(_lib.load().hca_dense_mqa_workspace_size(B, Tq, H, N, win_len))


def _attn_out(q, out, lse):
    B, Tq, H, _ = q.shape
    if out is None:
        out = torch.empty(B, Tq, H, 128, dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty(B, Tq, H, dtype=torch.float32, device=q.device)
    return out, lse


def csa_sparse_mqa(q, cache: KVCache, m, idx, win: Window | None, scale, *, q_pos0=0, out=None, lse=None,
                   workspace=None, stream=None):
    """CSA core attention over the selected entries plus the sliding window (one softmax)."""
    lib = _lib.load()
    B, Tq, H, _ = q.shape
    k = idx.shape[-1]
    out, lse = _attn_out(q, out, lse)
    wlen = win.length if win is not None else 0
    need = csa_sparse_mqa_workspace_size(B, Tq, H, k, wlen)
    if workspace is None and need:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    cd = cache.desc()
    wd = win.desc() if win is not None else None
    st = lib.csa_sparse_mqa(_ptr(q), B, Tq, H, q_pos0, ctypes.byref(cd), m, _ptr(idx), k,
                            ctypes.byref(wd) if wd is not None else None, float(scale), _ptr(out), _ptr(lse),
                            _ptr(workspace), 0 if workspace is None else workspace.numel(), _stream(stream))
    _check(st, "csa_sparse_mqa")
    return out, lse


def hca_dense_mqa(q, cache: KVCache, m_prime, win: Window | None, scale, *, q_pos0=0, out=None, lse=None,
                  workspace=None, stream=None, max_sms=0):
    """HCA core attention over every visible entry plus the sliding window (one softmax).

    ``max_sms`` > 0 keeps the 64-head decode launch to that many SMs (``hca_dense_mqa_budget``), leaving the
    rest to work the caller runs beside it on another stream."""
    lib = _lib.load()
    B, Tq, H, _ = q.shape
    out, lse = _attn_out(q, out, lse)
    wlen = win.length if win is not None else 0
    need = hca_dense_mqa_workspace_size(B, Tq, H, cache.n_entries, wlen)
    if workspace is None and need:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    cd = cache.desc()
    wd = win.desc() if win is not None else None
    wsz = 0 if workspace is None else workspace.numel()
    if max_sms:
        st = lib.hca_dense_mqa_budget(_ptr(q), B, Tq, H, q_pos0, ctypes.byref(cd), m_prime,
                                      ctypes.byref(wd) if wd is not None else None, float(scale), _ptr(out), _ptr(lse),
                                      int(max_sms), _ptr(workspace), wsz, _stream(stream))
        _check(st, "hca_dense_mqa_budget")
    else:
        st = lib.hca_dense_mqa(_ptr(q), B, Tq, H, q_pos0, ctypes.byref(cd), m_prime,
                               ctypes.byref(wd) if wd is not None else None, float(scale), _ptr(out), _ptr(lse),
                               _ptr(workspace), wsz, _stream(stream))
        _check(st, "hca_dense_mqa")
    return out, lse


def grouped_out_proj(o, w, *, y=None, stream=None):
    """Grouped output projection: heads in G groups of H/G, group g's outputs times w[g]^T.

    o bf16 [..., H, 128] (attention output), w bf16 [G, d_g, (H/G)*128] -> y bf16 [..., G, d_g].
    """
    lib = _lib.load()
    H = o.shape[-2]
    G, dg = w.shape[0], w.shape[1]
    lead = tuple(o.shape[:-2])
    R = 1
    for n in lead:
        R *= n
    if y is None:
        y = torch.empty(*lead, G, dg, dtype=torch.bfloat16, device=o.device)
    st = lib.csa_grouped_out_proj(_ptr(o), R, H, G, dg, _ptr(w), _ptr(y), _stream(stream))
    _check(st, "csa_grouped_out_proj")
    return y


class Packed:
    """Packed sequences (e.g. the documents of a packed pre-training batch) for one stride.

    Built from the host-side sequence lengths: sequence s owns packed tokens [cu_tokens[s], cu_tokens[s+1])
    and entries [cu_entries[s], cu_entries[s+1]) (ceil(len / stride) of them).  The offsets are uploaded once.
    """

    def __init__(self, lengths, stride, device="cuda"):
        lens = [int(n) for n in lengths]
        if any(n < 0 for n in lens):
            raise ValueError("sequence lengths must be >= 0")
        ent = [-(-n // stride) for n in lens]
        cu_t, cu_e = [0], [0]
        for n, e in zip(lens, ent):
            cu_t.append(cu_t[-1] + n)
            cu_e.append(cu_e[-1] + e)
        self.lengths, self.stride = lens, stride
        self.cu_tokens_host, self.cu_entries_host = cu_t, cu_e
        self.cu_tokens = torch.tensor(cu_t, dtype=torch.int32, device=device)
        self.cu_entries = torch.tensor(cu_e, dtype=torch.int32, device=device)
        self.total_tokens, self.total_entries = cu_t[-1], cu_e[-1]
        self.max_tokens = max(lens) if lens else 0

    def desc(self) -> _lib.PackedDesc:
        d = _lib.PackedDesc()
        d.cu_tokens, d.cu_entries = _ptr(self.cu_tokens), _ptr(self.cu_entries)
        d.n_seqs = len(self.lengths)
        d.max_tokens = self.max_tokens
        d.total_tokens, d.total_entries = self.total_tokens, self.total_entries
        return d


def _compress_append(fn_name, x, x_pos0, t, w, b_pos, stride, cache, stream):
    lib = _lib.load()
    B, rows, d = x.shape
    if isinstance(cache, KVCache) and cache.split:
        st = getattr(lib, fn_name)(_ptr(x), B, rows, x_pos0, t, d, stride, _ptr(w), _ptr(b_pos),
                                   _lib.CSA_KV_SPLIT_FP8, _ptr(cache.nope), _ptr(cache.rope), _ptr(cache.scale),
                                   cache.nope.shape[1], _stream(stream))
    else:
        k = cache.k if isinstance(cache, KVCache) else cache
        st = getattr(lib, fn_name)(_ptr(x), B, rows, x_pos0, t, d, stride, _ptr(w), _ptr(b_pos), _lib.CSA_KV_BF16,
                                   _ptr(k), None, None, k.shape[1], _stream(stream))
    _check(st, fn_name)


def csa_compress_append(x, x_pos0, t, w, b_pos, m, cache, *, stream=None):
    """Decode-time append: if token t completes CSA entry i = (t+1)/m - 1, write it into cache slot i.

    x bf16 [B, rows, d] holds raw tokens at positions x_pos0 ..; cache is a bf16 tensor [B, n_cap, d] or a split
    FP8 KVCache (nope [B, n_cap, 128], rope, scale)."""
    _compress_append("csa_compress_append", x, x_pos0, t, w, b_pos, m, cache, stream)


def hca_compress_append(x, x_pos0, t, w, b_pos, m_prime, cache, *, stream=None):
    """Decode-time append of the HCA entry that token t completes (t + 1 a multiple of m')."""
    _compress_append("hca_compress_append", x, x_pos0, t, w, b_pos, m_prime, cache, stream)


def _compress_packed(fn_name, x, packed: Packed, w, b_pos, stride, fp8, stream):
    lib = _lib.load()
    d = x.shape[-1]
    E = packed.total_entries
    pd = packed.desc()
    if fp8:
        nope = torch.empty(E, 128, dtype=torch.uint8, device=x.device)
        rope = torch.empty(E, 64, dtype=torch.bfloat16, device=x.device)
        scale = torch.empty(E, dtype=torch.float32, device=x.device)
        st = getattr(lib, fn_name)(_ptr(x), ctypes.byref(pd), d, stride, _ptr(w), _ptr(b_pos), _lib.CSA_KV_SPLIT_FP8,
                                   _ptr(nope), _ptr(rope), _ptr(scale), _stream(stream))
        _check(st, fn_name)
        return nope, rope, scale
    y = torch.empty(E, d, dtype=torch.bfloat16, device=x.device)
    st = getattr(lib, fn_name)(_ptr(x), ctypes.byref(pd), d, stride, _ptr(w), _ptr(b_pos), _lib.CSA_KV_BF16, _ptr(y),
                               None, None, _stream(stream))
    _check(st, fn_name)
    return y


def csa_compress_packed(x, packed: Packed, w, b_pos, m, *, fp8=False, stream=None):
    """CSA compression of packed sequences x bf16 [total_tokens, d] -> entries [total_entries, d]."""
    if packed.stride != m:
        raise ValueError("packed descriptor was built for another stride")
    return _compress_packed("csa_compress_packed", x, packed, w, b_pos, m, fp8, stream)


def hca_compress_packed(x, packed: Packed, w, b_pos, m_prime, *, fp8=False, stream=None):
    """HCA compression of packed sequences x bf16 [total_tokens, d] -> entries [total_entries, d]."""
    if packed.stride != m_prime:
        raise ValueError("packed descriptor was built for another stride")
    return _compress_packed("hca_compress_packed", x, packed, w, b_pos, m_prime, fp8, stream)


def csa_indexer_topk_packed(qI, wI, kIc, packed: Packed, m, k, *, idx=None, workspace=None, stream=None):
    """Indexer top-k over packed sequences: qI [total_tokens, 4, 64] -> idx int32 [total_tokens, k] of entry
    indices within each row's own sequence (ascending, -1 padded)."""
    lib = _lib.load()
    if packed.stride != m:
        raise ValueError("packed descriptor was built for another stride")
    pd = packed.desc()
    if idx is None:
        idx = torch.empty(packed.total_tokens, k, dtype=torch.int32, device=qI.device)
    need = int(lib.csa_indexer_topk_packed_workspace_size(ctypes.byref(pd), m, k))
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=qI.device)
    st = lib.csa_indexer_topk_packed(_ptr(qI), _ptr(wI), _ptr(kIc), ctypes.byref(pd), m, k, _ptr(idx),
                                     _ptr(workspace), workspace.numel(), _stream(stream))
    _check(st, "csa_indexer_topk_packed")
    return idx


def _packed_window(k, v, packed, length):
    return Window(k=k, v=v, pos0=0, length=length)


def csa_sparse_mqa_packed(q, packed: Packed, cache: KVCache, m, idx, win_k, win_v, win_len, scale, *, out=None,
                          lse=None, workspace=None, stream=None):
    """CSA attention over packed sequences: q [total_tokens, H, 192]; the window is read from the packed raw
    tokens win_k [total_tokens, 192] (win_v [total_tokens, 128] or None)."""
    lib = _lib.load()
    TT, H = q.shape[0], q.shape[1]
    k = idx.shape[-1]
    out = out if out is not None else torch.empty(TT, H, 128, dtype=torch.bfloat16, device=q.device)
    lse = lse if lse is not None else torch.empty(TT, H, dtype=torch.float32, device=q.device)
    need = csa_sparse_mqa_workspace_size(1, TT, H, k, win_len)
    if workspace is None and need:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    pd, cd, wd = packed.desc(), cache.desc(), _packed_window(win_k, win_v, packed, win_len).desc()
    st = lib.csa_sparse_mqa_packed(_ptr(q), H, ctypes.byref(pd), ctypes.byref(cd), m, _ptr(idx), k, ctypes.byref(wd),
                                   float(scale), _ptr(out), _ptr(lse), _ptr(workspace),
                                   0 if workspace is None else workspace.numel(), _stream(stream))
    _check(st, "csa_sparse_mqa_packed")
    return out, lse


def hca_dense_mqa_packed(q, packed: Packed, cache: KVCache, m_prime, win_k, win_v, win_len, scale, *, out=None,
                         lse=None, workspace=None, stream=None):
    """HCA attention over packed sequences (every visible entry of the row's own sequence + its window)."""
    lib = _lib.load()
    TT, H = q.shape[0], q.shape[1]
    out = out if out is not None else torch.empty(TT, H, 128, dtype=torch.bfloat16, device=q.device)
    lse = lse if lse is not None else torch.empty(TT, H, dtype=torch.float32, device=q.device)
    need = hca_dense_mqa_workspace_size(1, TT, H, -(-packed.max_tokens // m_prime), win_len)
    if workspace is None and need:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    pd, cd, wd = packed.desc(), cache.desc(), _packed_window(win_k, win_v, packed, win_len).desc()
    st = lib.hca_dense_mqa_packed(_ptr(q), H, ctypes.byref(pd), ctypes.byref(cd), m_prime, ctypes.byref(wd),
                                  float(scale), _ptr(out), _ptr(lse), _ptr(workspace),
                                  0 if workspace is None else workspace.numel(), _stream(stream))
    _check(st, "hca_dense_mqa_packed")
    return out, lse


def _tensor(t, name, dtype, shape, device):
    """The address of a contiguous CUDA tensor of this type, shape and device."""
    if t.dtype is not dtype or t.shape != shape or t.device != device or not t.is_contiguous():
        if t.dtype is not dtype:
            raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
        if t.shape != shape:
            raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
        if t.device != device:
            raise ValueError(f"{name} is on {t.device}, not on {device}")
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _elsewhere(device, stream):
    """None where a call runs on the current device and stream, else a context that makes its own the current ones
    (outputs and scratch are then allocated for that stream)."""
    if device.type != "cuda":
        raise ValueError("tensor must live on a CUDA device")
    if stream is not None:
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(int(stream), device=device)
        if stream.device != device:
            raise ValueError(f"stream is on {stream.device}, not on {device}")
        return torch.cuda.stream(stream)
    return None if device.index == torch.cuda.current_device() else torch.cuda.device(device)


# torch's own short way to the current stream's handle, where it has it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _current_stream(device):
    return _raw_stream(device.index) if _raw_stream is not None else torch.cuda.current_stream(device).cuda_stream


def _dims(t, n, name):
    if t.dim() != n:
        raise ValueError(f"{name} must have {n} dimensions, got shape {tuple(t.shape)}")
    return t.shape


@dataclasses.dataclass
class GqaCache:
    """Pages of a grouped-head cache: k bf16 [n_pages, H_kv, page_size, d_qk], v bf16 [n_pages, H_kv, page_size,
    d_v], and optionally the accumulated weight of every token, mass fp32 [n_pages, H_kv, page_size]."""
    k: torch.Tensor
    v: torch.Tensor
    mass: torch.Tensor | None = None

    def desc(self, device) -> _lib.GqaCacheDesc:
        k, v, mass = self.k, self.v, self.mass
        P, H, S, d = _dims(k, 4, "cache.k")
        dv = _dims(v, 4, "cache.v")[3]
        return _lib.GqaCacheDesc(_tensor(k, "cache.k", torch.bfloat16, (P, H, S, d), device),
                                 _tensor(v, "cache.v", torch.bfloat16, (P, H, S, dv), device),
                                 None if mass is None else _tensor(mass, "cache.mass", torch.float32, (P, H, S), device),
                                 P, S, H, d, dv)


@dataclasses.dataclass
class GqaBatch:
    """The sequences of a call and their new tokens (device tensors, read when the call runs): block_table int32
    [n_seqs, max_pages], cache_len int32 [n_seqs] (tokens held, the new ones included), cu_q int32 [n_seqs + 1]
    (offsets of the new rows), and on the host max_q (at least the most new tokens of one sequence) and total_q
    (rows of the packed arrays)."""
    block_table: torch.Tensor
    cache_len: torch.Tensor
    cu_q: torch.Tensor | None
    max_q: int = 1
    total_q: int = 0

    def desc(self, device) -> _lib.GqaBatchDesc:
        n, m = _dims(self.block_table, 2, "block_table")
        return _lib.GqaBatchDesc(_tensor(self.block_table, "block_table", torch.int32, (n, m), device),
                                 _tensor(self.cache_len, "cache_len", torch.int32, (n,), device),
                                 None if self.cu_q is None else
                                 _tensor(self.cu_q, "cu_q", torch.int32, (n + 1,), device),
                                 n, m, self.max_q, 0, self.total_q)


def gqa_dense_workspace_size(max_q, H, H_kv, d_v) -> int:
    return int(_lib.load().gqa_dense_workspace_size(max_q, H, H_kv, d_v))


def _gqa_buffers(lib, q, shape, d_v, max_q, H_kv, out, lse, workspace):
    """Output, lse and workspace of a call (those not given are allocated) with their addresses, and the workspace's
    size."""
    R, H, _ = shape
    dev = q.device
    if out is None:
        out = q.new_empty((R, H, d_v))
        op = out.data_ptr()
    else:
        op = _tensor(out, "out", torch.bfloat16, (R, H, d_v), dev)
    if lse is None:
        lse = torch.empty((R, H), dtype=torch.float32, device=dev)
        lp = lse.data_ptr()
    else:
        lp = _tensor(lse, "lse", torch.float32, (R, H), dev)
    if workspace is None:
        size = lib.gqa_dense_workspace_size(max_q, H, H_kv, d_v)
        workspace = torch.empty(size, dtype=torch.uint8, device=dev)
        wp = workspace.data_ptr()
    else:
        size = workspace.numel()
        wp = _tensor(workspace, "workspace", torch.uint8, (size,), dev)
    return out, lse, workspace, op, lp, wp, size


def gqa_dense_packed(q, k, v, packed: Packed, scale, *, out=None, lse=None, workspace=None, stream=None):
    """Causal attention over whole packed prompts with grouped heads: row t of a sequence sees its tokens 0 .. t,
    query head h reads kv head h // (H / H_kv).  Returns (out, lse)."""
    dev = q.device
    if (ctx := _elsewhere(dev, stream)) is not None:
        with ctx:
            return gqa_dense_packed(q, k, v, packed, scale, out=out, lse=lse, workspace=workspace)
    lib = _lib.load()
    R, H, d_qk = _dims(q, 3, "q")
    _, H_kv, d_v = _dims(v, 3, "v")
    qp = _tensor(q, "q", torch.bfloat16, (packed.total_tokens, H, d_qk), dev)
    kp = _tensor(k, "k", torch.bfloat16, (R, H_kv, d_qk), dev)
    vp = _tensor(v, "v", torch.bfloat16, (R, H_kv, d_v), dev)
    n = len(packed.lengths)
    cu = _tensor(packed.cu_tokens, "the packed offsets", torch.int32, (n + 1,), dev)
    pd = _lib.PackedDesc(cu, None, n, packed.max_tokens, packed.total_tokens, 0)  # the entry offsets are not used
    out, lse, workspace, op, lp, wp, size = _gqa_buffers(lib, q, (R, H, d_qk), d_v, packed.max_tokens, H_kv, out, lse,
                                                         workspace)
    _check(lib.gqa_dense_packed(qp, kp, vp, ctypes.byref(pd), H, H_kv, d_qk, d_v, scale, op, lp, wp, size,
                                _current_stream(dev)), "gqa_dense_packed")
    return out, lse


def gqa_dense_paged(q, cache: GqaCache, batch: GqaBatch, scale, *, out=None, lse=None, workspace=None, stream=None):
    """Causal attention of a chunk of new tokens (one: decode) over the paged cache that holds them already.
    Returns (out, lse)."""
    dev = q.device
    if (ctx := _elsewhere(dev, stream)) is not None:
        with ctx:
            return gqa_dense_paged(q, cache, batch, scale, out=out, lse=lse, workspace=workspace)
    lib = _lib.load()
    cd, bd = cache.desc(dev), batch.desc(dev)
    shape = (batch.total_q, _dims(q, 3, "q")[1], cd.d_qk)
    qp = _tensor(q, "q", torch.bfloat16, shape, dev)
    out, lse, workspace, op, lp, wp, size = _gqa_buffers(lib, q, shape, cd.d_v, batch.max_q, cd.n_kv_heads, out, lse,
                                                         workspace)
    _check(lib.gqa_dense_paged(qp, ctypes.byref(cd), ctypes.byref(bd), shape[1], scale, op, lp, wp, size,
                               _current_stream(dev)), "gqa_dense_paged")
    return out, lse


def gqa_cache_append(k, v, cache: GqaCache, batch: GqaBatch, *, stream=None):
    """Writes the new tokens' k bf16 [total_q, H_kv, d_qk] and v bf16 [total_q, H_kv, d_v] into their slots, and 0
    into the slots' mass where the cache has one."""
    dev = cache.k.device
    if (ctx := _elsewhere(dev, stream)) is not None:
        with ctx:
            return gqa_cache_append(k, v, cache, batch)
    lib = _lib.load()
    cd, bd = cache.desc(dev), batch.desc(dev)
    kp = _tensor(k, "k", torch.bfloat16, (batch.total_q, cd.n_kv_heads, cd.d_qk), dev)
    vp = _tensor(v, "v", torch.bfloat16, (batch.total_q, cd.n_kv_heads, cd.d_v), dev)
    _check(lib.gqa_cache_append(kp, vp, ctypes.byref(cd), ctypes.byref(bd), _current_stream(dev)), "gqa_cache_append")


def gqa_cache_mass(q, lse, cache: GqaCache, batch: GqaBatch, scale, *, stream=None):
    """Adds to cache.mass the attention weight the chunk's rows give every cached token, summed over the rows and
    the heads of a group; lse is gqa_dense_paged's of the same rows.  Returns cache.mass."""
    dev = cache.k.device
    if (ctx := _elsewhere(dev, stream)) is not None:
        with ctx:
            return gqa_cache_mass(q, lse, cache, batch, scale)
    lib = _lib.load()
    cd, bd = cache.desc(dev), batch.desc(dev)
    H = _dims(q, 3, "q")[1]
    qp = _tensor(q, "q", torch.bfloat16, (batch.total_q, H, cd.d_qk), dev)
    lp = _tensor(lse, "lse", torch.float32, (batch.total_q, H), dev)
    _check(lib.gqa_cache_mass(qp, lp, ctypes.byref(cd), ctypes.byref(bd), H, scale, _current_stream(dev)),
           "gqa_cache_mass")
    return cache.mass


def gqa_cache_evict(cache: GqaCache, batch: GqaBatch, budget, new_table, *, sink=0, recent=0, kept=None, new_len=None,
                    stream=None):
    """Cuts caches of more than ``budget`` tokens down to it: every kv head keeps its first ``sink`` and last
    ``recent`` tokens and the heaviest (cache.mass) of those between, copied in order to the pages of new_table
    int32 [n_seqs, pages], which no sequence of the call reads.  Returns (kept int32 [n_seqs, H_kv, budget], -1
    padded, and new_len int32 [n_seqs])."""
    dev = cache.k.device
    if (ctx := _elsewhere(dev, stream)) is not None:
        with ctx:
            return gqa_cache_evict(cache, batch, budget, new_table, sink=sink, recent=recent, kept=kept,
                                   new_len=new_len)
    lib = _lib.load()
    cd, bd = cache.desc(dev), batch.desc(dev)
    n, H, pages = bd.n_seqs, cd.n_kv_heads, _dims(new_table, 2, "new_table")[1]
    tp = _tensor(new_table, "new_table", torch.int32, (n, pages), dev)
    if kept is None:
        kept = torch.empty((n, H, max(budget, 0)), dtype=torch.int32, device=dev)
    if new_len is None:
        new_len = torch.empty((n,), dtype=torch.int32, device=dev)
    kp = _tensor(kept, "kept", torch.int32, (n, H, budget), dev)
    np_ = _tensor(new_len, "new_len", torch.int32, (n,), dev)
    _check(lib.gqa_cache_evict(ctypes.byref(cd), ctypes.byref(bd), budget, sink, recent, tp, pages, kp, np_,
                               _current_stream(dev)), "gqa_cache_evict")
    return kept, new_len
