"""Float64 oracle of the grouped-head dense attention and its paged cache (numpy, shares no code with the GPU path)."""
from __future__ import annotations

import numpy as np


def attend(q, k, v, scale, first):
    """Rows q [n, H, d] at positions first .. first + n - 1 over keys k [L, H_kv, d], values v [L, H_kv, dv].

    Row i sees keys 0 .. first + i.  Returns out [n, H, dv], lse [n, H], and mean_abs [n, H, dv], the softmax mean of
    |v| (the size a rounding of the probabilities is relative to).  A row that sees nothing has out 0, lse -inf.
    """
    n, H, _ = q.shape
    L, Hk = k.shape[0], k.shape[1]
    G = H // Hk
    out = np.zeros((n, H, v.shape[2]))
    size = np.zeros((n, H, v.shape[2]))
    lse = np.full((n, H), -np.inf)
    for i in range(n):
        m = min(max(first + i + 1, 0), L)
        if m == 0:
            continue
        for h in range(H):
            x = scale * (k[:m, h // G] @ q[i, h])
            top = x.max()
            p = np.exp(x - top)
            lse[i, h] = top + np.log(p.sum())
            p = p / p.sum()
            out[i, h] = p @ v[:m, h // G]
            size[i, h] = p @ np.abs(v[:m, h // G])
    return out, lse, size


def weights(q, k, lse, scale, first):
    """Accumulated weight [H_kv, L] that the rows give each key, with the rows' lse [n, H] given."""
    n, H, _ = q.shape
    L, Hk = k.shape[0], k.shape[1]
    G = H // Hk
    add = np.zeros((Hk, L))
    for i in range(n):
        m = min(max(first + i + 1, 0), L)
        for h in range(H):
            if m and np.isfinite(lse[i, h]):
                add[h // G, :m] += np.exp(scale * (k[:m, h // G] @ q[i, h]) - lse[i, h])
    return add


def score_size(q, k, scale):
    """Largest scale * sum |q_c k_c| over all (row, head, key): what the rounding of a score is relative to."""
    H, Hk = q.shape[1], k.shape[1]
    if q.shape[0] == 0 or k.shape[0] == 0:
        return 0.0
    aq, ak = np.abs(q), np.abs(k)
    return scale * max(float((ak[:, h // (H // Hk)] @ aq[:, h].T).max()) for h in range(H))


def live(plane, table, length):
    """Tokens 0 .. length - 1 of one sequence: plane [pages, H_kv, page, ...] -> [length, H_kv, ...]."""
    page = plane.shape[2]
    return np.stack([plane[table[j // page], :, j % page] for j in range(length)]) if length else \
        np.zeros((0, plane.shape[1], *plane.shape[3:]), plane.dtype)


def keep(mass, budget, sink, recent):
    """Positions kept of one kv head's mass [L]."""
    L = len(mass)
    if L <= budget:
        return list(range(L))
    weight = np.where(np.isnan(mass), np.inf, mass)
    nan = np.isnan(mass)
    middle = sorted(range(sink, L - recent), key=lambda j: (not nan[j], -weight[j], j))[: budget - sink - recent]
    return list(range(sink)) + sorted(middle) + list(range(L - recent, L))
