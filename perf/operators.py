"""Grouped-head dense attention over packed prompts and paged caches: cases, plain forms and exact values.

Operators (``op`` of a case):
  prompt  gqa_dense_packed  causal attention over whole packed prompts
  paged   gqa_dense_paged   a chunk of new tokens (one token: decode) over a paged cache that holds them
  mass    gqa_cache_mass    the attention weight that a chunk gives to every cached token, accumulated
  append  gqa_cache_append  a chunk's keys and values into their pages
  evict   gqa_cache_evict   sink, recent and heaviest tokens of every kv head, compacted into new pages

Sequence s brings n[s] new tokens; its cache holds len[s] tokens with them, so row i stands at position
len[s] - n[s] + i and sees the tokens at or before it.  Pages are [page, kv head, slot, channel].
"""
import math
import random

import torch

own = False

DIMS = ((192, 128), (128, 128), (64, 64))


def listed():
    return [
        # a packed batch of documents of very different lengths, one of them empty, at the library's 192/128 width
        {"name": "prompt_documents", "op": "prompt", "n": "2048,513,1,777,0,4000,1025,128,31,1500,2049", "hkv": 4, "g": 4, "dqk": 192, "dv": 128},
        # one long prompt, grouped heads: the matrix-product-bound end
        {"name": "prompt_8192", "op": "prompt", "n": "8192", "hkv": 8, "g": 4, "dqk": 128, "dv": 128},
        # one user, one token, a short context: latency
        {"name": "decode_one", "op": "paged", "n": "1", "len": "777", "hkv": 8, "g": 4, "dqk": 128, "dv": 128, "page": 16},
        # a serving batch of unequal contexts, one token each
        {"name": "decode_batch", "op": "paged", "n": "1*32", "len": "1000:16384*32", "hkv": 8, "g": 8, "dqk": 128, "dv": 128, "page": 64},
        # 64 heads over one kv head at 128K tokens of context
        {"name": "decode_131072", "op": "paged", "n": "1*8", "len": "131072*8", "hkv": 1, "g": 64, "dqk": 192, "dv": 128, "page": 128},
        # chunked prefill beside a short decode-like row count
        {"name": "chunk_512", "op": "paged", "n": "512,512,300,77", "len": "16384,8192,5001,700", "hkv": 8, "g": 4, "dqk": 128, "dv": 128, "page": 32},
        # accumulated weight after a decode step
        {"name": "mass_decode", "op": "mass", "n": "1*16", "len": "1500:16384*16", "hkv": 8, "g": 4, "dqk": 128, "dv": 128, "page": 64},
        # accumulated weight of the last tokens of a prompt, before its cache is cut down
        {"name": "mass_last_64", "op": "mass", "n": "64*4", "len": "8192,8100,4095,1000", "hkv": 4, "g": 4, "dqk": 192, "dv": 128, "page": 32},
        # one decode step's tokens
        {"name": "append_step", "op": "append", "n": "1*64", "len": "100:4000*64", "hkv": 8, "dqk": 128, "dv": 128, "page": 16},
        # the tokens of two prompts
        {"name": "append_prompts", "op": "append", "n": "8192,5000", "len": "8192,9000", "hkv": 8, "dqk": 128, "dv": 128, "page": 64},
        # caches a little over their budget, one under it
        {"name": "evict_short", "op": "evict", "len": "1025,4000,700,2049,1500,3000,1024,2500", "budget": 1024, "sink": 4, "recent": 128, "hkv": 8, "dqk": 128, "dv": 128, "page": 16},
        # long caches cut down to a sixteenth
        {"name": "evict_long", "op": "evict", "len": "65536,65000,40001,65536", "budget": 4096, "sink": 16, "recent": 512, "hkv": 8, "dqk": 64, "dv": 64, "page": 64},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(("prompt", "paged", "paged", "mass", "append", "evict"))
    dqk, dv = rng.choice(DIMS)
    hkv = rng.choice((1, 2, 3, 4, 8))
    case = {"op": op, "hkv": hkv, "dqk": dqk, "dv": dv}
    if op != "prompt":
        case["page"] = rng.choice((16, 32, 64, 128))
    if op in ("prompt", "paged", "mass"):
        case["g"] = rng.choice((1, 2, 3, 4, 5, 7, 8, 12, 16)) if hkv > 1 else rng.choice((1, 4, 6, 8, 16, 64))
    if op == "prompt":
        # rows x heads x keys stay below those of one prompt of 8192 tokens with 32 heads
        top = min(8192, int(8192 * math.sqrt(32 / (hkv * case["g"]))))
        first = _log(rng, 1, top)
        case["n"] = ",".join(str(v) for v in [first] + [_log(rng, 1, max(1, top // 3)) for _ in range(rng.randrange(0, 7))])
        return case
    seqs = _log(rng, 1, 32)
    if op == "paged" or op == "mass":
        # live cache bytes stay below about 0.5 GB, and so do scores in 32 bits
        most = int(5e8 / (2 * seqs * hkv * (dqk + dv)))
        lens = [_log(rng, 64, max(64, min(65536, most))) for _ in range(seqs)]
        rows = rng.choice((1, 1, 1, rng.randrange(2, 9), _log(rng, 9, 600)))
        rows = max(1, min(rows, int(1.2e8 / (max(lens) * hkv * case["g"])))) if rows > 1 else 1
        n = [min(length, rows if rng.random() < 0.7 else rng.randrange(1, rows + 1)) for length in lens]
    elif op == "append":
        most = int(2e8 / (2 * seqs * hkv * (dqk + dv)))
        lens = [_log(rng, 1, max(1, min(16384, most))) for _ in range(seqs)]
        one = rng.random() < 0.5
        n = [1 if one else rng.randrange(0, length + 1) for length in lens]
        n[0] = max(1, n[0])
    else:
        seqs = _log(rng, 1, 16)
        most = int(5e8 / (2 * seqs * hkv * (dqk + dv)))
        lens = [_log(rng, 1, max(1, min(65536, most))) for _ in range(seqs)]
        budget = _log(rng, 1, max(1, max(lens)))
        sink = rng.randrange(0, min(16, budget) + 1)
        recent = rng.randrange(0, min(512, budget - sink) + 1)
        case.update({"len": ",".join(map(str, lens)), "budget": budget, "sink": sink, "recent": recent})
        return case
    case.update({"n": ",".join(map(str, n)), "len": ",".join(map(str, lens))})
    return case


def _lengths(text):
    """'5,7' = [5, 7]; '3*4' = [3] * 4; '10:40*4' = 4 lengths from 10 to 40, evenly, out of order."""
    out = []
    for part in text.split(","):
        value, _, times = part.partition("*")
        count = int(times or 1)
        lo, _, hi = value.partition(":")
        if not hi:
            out += [int(lo)] * count
        else:
            spread = [int(lo) + (int(hi) - int(lo)) * i // max(1, count - 1) for i in range(count)]
            out += [spread[(7 * i + 3) % count] for i in range(count)] if count % 7 else spread
    return out


def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32).to(torch.bfloat16)


def _offsets(n):
    cu = [0]
    for v in n:
        cu.append(cu[-1] + v)
    return cu


def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rng = random.Random(seed)
    hkv, dqk, dv, g = case["hkv"], case["dqk"], case["dv"], case.get("g", 1)
    state = {"case": dict(case), "scale": 1.0 / math.sqrt(dqk)}
    if case["op"] == "prompt":
        n = _lengths(case["n"])
        cu = _offsets(n)
        state.update({"n": n, "cu": cu, "q": _normal(gen, cu[-1], hkv * g, dqk), "k": _normal(gen, cu[-1], hkv, dqk), "v": _normal(gen, cu[-1], hkv, dv)})
        if own:
            import long_context_sparse_10_b200 as csa
            state["packed"] = csa.Packed(n, 1)
        return state
    lens, page = _lengths(case["len"]), case["page"]
    n = _lengths(case["n"]) if "n" in case else [0] * len(lens)
    cu = _offsets(n)
    # every sequence's pages, anywhere in the pool; eviction has its new pages there too
    need = [-(-length // page) for length in lens]
    fresh = [-(-min(length, case["budget"]) // page) for length in lens] if case["op"] == "evict" else [0] * len(lens)
    pool = list(range(sum(need) + sum(fresh) + 3))
    rng.shuffle(pool)
    width, wide = max(need), max(fresh)
    table = [[pool.pop() for _ in range(c)] + [0] * (width - c) for c in need]
    pages = sum(need) + sum(fresh) + 3
    state.update({"n": n, "cu": cu, "len": lens, "page": page, "table": _int32(table), "cache_len": _int32(lens), "cu_q": _int32(cu)})
    state["k"] = _normal(gen, pages, hkv, page, dqk)
    state["v"] = _normal(gen, pages, hkv, page, dv)
    state["mass"] = torch.zeros(pages, hkv, page, device="cuda")
    if case["op"] in ("paged", "mass"):
        state["q"] = _normal(gen, cu[-1], hkv * g, dqk)
    if case["op"] == "mass":
        state["mass"] += torch.rand(pages, hkv, page, generator=gen, device="cuda")
        state["lse"] = _plain_paged(state)[1]
    if case["op"] == "append":
        state["new_k"] = _normal(gen, cu[-1], hkv, dqk)
        state["new_v"] = _normal(gen, cu[-1], hkv, dv)
        state["mass"] += 1.0
    if case["op"] == "evict":
        # heavy-tailed weights, many of them equal (tokens that nothing has looked at yet)
        weight = torch.exp(2.0 * torch.randn(pages, hkv, page, generator=gen, device="cuda"))
        state["mass"] = torch.where(torch.rand(pages, hkv, page, generator=gen, device="cuda") < 0.1, torch.zeros_like(weight), weight)
        state["new_table"] = _int32([[pool.pop() for _ in range(c)] + [0] * (wide - c) for c in fresh])
    if own:
        import long_context_sparse_10_b200 as csa
        state["cache"] = csa.GqaCache(state["k"], state["v"], state["mass"])
        state["batch"] = csa.GqaBatch(state["table"], state["cache_len"], state["cu_q"], max_q=max(n), total_q=cu[-1])
    return state


def run(state):
    op, case = state["case"]["op"], state["case"]
    if own:
        import long_context_sparse_10_b200 as csa
        if op == "prompt":
            return csa.gqa_dense_packed(state["q"], state["k"], state["v"], state["packed"], state["scale"])
        if op == "paged":
            return csa.gqa_dense_paged(state["q"], state["cache"], state["batch"], state["scale"])
        if op == "mass":
            return csa.gqa_cache_mass(state["q"], state["lse"], state["cache"], state["batch"], state["scale"])
        if op == "append":
            csa.gqa_cache_append(state["new_k"], state["new_v"], state["cache"], state["batch"])
            return state["k"], state["v"], state["mass"]
        kept, new_len = csa.gqa_cache_evict(state["cache"], state["batch"], case["budget"], state["new_table"], sink=case["sink"], recent=case["recent"])
        return kept, new_len, state["k"], state["v"], state["mass"]
    if op == "prompt":
        return _plain_prompt(state)
    if op == "paged":
        return _plain_paged(state)
    if op == "mass":
        return _plain_mass(state)
    if op == "append":
        return _plain_append(state)
    return _plain_evict(state)


def _plain_attend(q, k, v, scale, first):
    """q [n, hkv, g, dqk], k [hkv, len, dqk], v [hkv, len, dv] in 32 bits -> out [n, hkv, g, dv], lse [n, hkv, g]."""
    n, hkv, g, d = q.shape
    rows = q.permute(1, 0, 2, 3).reshape(hkv, n * g, d)
    s = torch.bmm(rows, k.transpose(1, 2)).mul_(scale).view(hkv, n, g, -1)
    at = torch.arange(first, first + n, device=q.device)
    hidden = torch.arange(k.shape[1], device=q.device)[None, :] > at[:, None]
    s.masked_fill_(hidden[None, :, None, :], -math.inf)
    top = s.amax(-1, keepdim=True)
    p = s.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.bmm(p.view(hkv, n * g, -1), v).view(hkv, n, g, -1) / total
    lse = (top + total.log()).squeeze(-1)
    return o.permute(1, 0, 2, 3), lse.permute(1, 0, 2)


def _plain_prompt(state):
    q, k, v, cu = state["q"], state["k"], state["v"], state["cu"]
    hkv = k.shape[1]
    out = torch.empty(q.shape[0], q.shape[1], v.shape[2], dtype=torch.bfloat16, device=q.device)
    lse = torch.empty(q.shape[0], q.shape[1], device=q.device)
    for a, b in zip(cu[:-1], cu[1:]):
        if b > a:
            o, m = _plain_attend(q[a:b].float().view(b - a, hkv, -1, q.shape[2]), k[a:b].float().transpose(0, 1), v[a:b].float().transpose(0, 1), state["scale"], 0)
            out[a:b] = o.reshape(b - a, -1, v.shape[2])
            lse[a:b] = m.reshape(b - a, -1)
    return out, lse


def _plain_live(state, plane, s):
    """The first len[s] tokens of a plane of the cache: [hkv, len, channels]."""
    length = state["len"][s]
    held = state[plane][state["table"][s, : -(-length // state["page"])].long()]
    return held.transpose(0, 1).reshape(held.shape[1], -1, *held.shape[3:])[:, :length]


def _plain_paged(state):
    q, cu = state["q"], state["cu"]
    hkv, dv = state["v"].shape[1], state["v"].shape[3]
    out = torch.empty(q.shape[0], q.shape[1], dv, dtype=torch.bfloat16, device=q.device)
    lse = torch.empty(q.shape[0], q.shape[1], device=q.device)
    for s, (a, b) in enumerate(zip(cu[:-1], cu[1:])):
        if b > a:
            o, m = _plain_attend(q[a:b].float().view(b - a, hkv, -1, q.shape[2]), _plain_live(state, "k", s).float(), _plain_live(state, "v", s).float(), state["scale"], state["len"][s] - (b - a))
            out[a:b] = o.reshape(b - a, -1, dv)
            lse[a:b] = m.reshape(b - a, -1)
    return out, lse


def _plain_mass(state):
    q, cu, mass, page = state["q"], state["cu"], state["mass"], state["page"]
    hkv = state["k"].shape[1]
    for s, (a, b) in enumerate(zip(cu[:-1], cu[1:])):
        if b > a:
            length, n = state["len"][s], b - a
            k = _plain_live(state, "k", s).float()
            rows = q[a:b].float().view(n, hkv, -1, q.shape[2]).permute(1, 0, 2, 3).reshape(hkv, -1, q.shape[2])
            x = torch.bmm(rows, k.transpose(1, 2)).mul_(state["scale"]).view(hkv, n, -1, length)
            x.sub_(state["lse"][a:b].view(n, hkv, -1).permute(1, 0, 2)[..., None])
            at = torch.arange(length - n, length, device=q.device)
            x.masked_fill_((torch.arange(length, device=q.device)[None, :] > at[:, None])[None, :, None, :], -math.inf)
            add = x.exp_().sum((1, 2))
            at = torch.arange(length, device=q.device)
            where, slot = state["table"][s].long()[at // page], at % page
            mass[where, :, slot] = mass[where, :, slot] + add.t()
    return mass


def _plain_append(state):
    k, v, mass, cu, page = state["k"], state["v"], state["mass"], state["cu"], state["page"]
    for s, (a, b) in enumerate(zip(cu[:-1], cu[1:])):
        at = torch.arange(state["len"][s] - (b - a), state["len"][s], device=k.device)
        where, slot = state["table"][s].long()[at // page], at % page
        k[where, :, slot] = state["new_k"][a:b]
        v[where, :, slot] = state["new_v"][a:b]
        mass[where, :, slot] = 0.0
    return k, v, mass


def _plain_evict(state):
    case, page = state["case"], state["page"]
    k, v, mass = state["k"], state["v"], state["mass"]
    budget, sink, recent = case["budget"], case["sink"], case["recent"]
    hkv = k.shape[1]
    kept = torch.full((len(state["len"]), hkv, budget), -1, dtype=torch.int32, device=k.device)
    heads = torch.arange(hkv, device=k.device)[:, None]
    for s, length in enumerate(state["len"]):
        if length <= budget:
            ids = torch.arange(length, device=k.device).expand(hkv, length)
        else:
            middle = _plain_live(state, "mass", s)[:, sink : length - recent]
            order = torch.sort(middle, dim=1, descending=True, stable=True).indices[:, : budget - sink - recent]
            ids = torch.cat([torch.arange(sink, device=k.device).expand(hkv, sink), order.sort(1).values + sink, torch.arange(length - recent, length, device=k.device).expand(hkv, recent)], 1)
        kept[s, :, : ids.shape[1]] = ids.int()
        if length:
            source, target = state["table"][s].long()[ids // page], torch.arange(ids.shape[1], device=k.device)
            where, slot = state["new_table"][s].long()[target // page][None], (target % page)[None]
            for plane in (k, v, mass):
                plane[where, heads, slot] = plane[source, heads, ids % page]
    new_len = state["cache_len"].clamp(max=budget)
    return kept, new_len, k, v, mass


def _pairs(n, length):
    """Visible (row, key) pairs of n rows at the end of `length` tokens."""
    return n * length - n * (n - 1) // 2


def work(case):
    hkv, dqk, dv, g = case["hkv"], case["dqk"], case["dv"], case.get("g", 1)
    token = hkv * 2 * (dqk + dv)
    if case["op"] == "prompt":
        n = _lengths(case["n"])
        rows = sum(n)
        pairs = sum(_pairs(v, v) for v in n)
        return {"bytes": rows * (token + hkv * g * (2 * dqk + 2 * dv + 4)), "flops": 2 * (dqk + dv) * hkv * g * pairs}
    lens = _lengths(case["len"])
    n = _lengths(case["n"]) if "n" in case else [0] * len(lens)
    rows, held = sum(n), sum(lens)
    pairs = sum(_pairs(a, b) for a, b in zip(n, lens))
    if case["op"] == "paged":
        live = sum(b for a, b in zip(n, lens) if a)
        return {"bytes": live * token + rows * hkv * g * (2 * dqk + 2 * dv + 4), "flops": 2 * (dqk + dv) * hkv * g * pairs}
    if case["op"] == "mass":
        return {"bytes": held * hkv * (2 * dqk + 8) + rows * hkv * g * (2 * dqk + 4), "flops": 2 * dqk * hkv * g * pairs}
    if case["op"] == "append":
        return {"bytes": rows * (2 * token + 4 * hkv), "flops": 0}
    out = sum(min(length, case["budget"]) for length in lens)
    return {"bytes": held * hkv * 4 + out * (2 * token + 4 * hkv) + len(lens) * hkv * case["budget"] * 4, "flops": 0}


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "prompt":
        return _exact_prompt(state)
    if case["op"] == "paged":
        return _exact_paged(state)
    if case["op"] == "mass":
        return _exact_mass(state)
    if case["op"] == "append":
        return _exact_append(state)
    return _exact_evict(state)


def _slots(state, s, positions, table="table"):
    """Row of [pages * page] that holds each position of sequence s."""
    return state[table][s].long().index_select(0, torch.div(positions, state["page"], rounding_mode="floor")) * state["page"] + positions.remainder(state["page"])


def _exact_head(q, k, scale, first):
    """One query head in 64 bits: scores with what is hidden at -inf, and their log-sum-exp."""
    s = (q.double() @ k.double().T) * scale
    s = s.masked_fill(torch.ones_like(s, dtype=torch.bool).triu(first + 1), -math.inf)
    return s, torch.logsumexp(s, 1)


def _exact_prompt(state):
    q, k, v, cu = state["q"], state["k"], state["v"], state["cu"]
    g = q.shape[1] // k.shape[1]
    out = torch.zeros(q.shape[0], q.shape[1], v.shape[2], dtype=torch.float64, device=q.device)
    lse = torch.zeros(q.shape[0], q.shape[1], dtype=torch.float64, device=q.device)
    for a, b in zip(cu[:-1], cu[1:]):
        for h in range(q.shape[1] if b > a else 0):
            s, m = _exact_head(q[a:b, h], k[a:b, h // g], state["scale"], 0)
            out[a:b, h] = torch.exp(s - m[:, None]) @ v[a:b, h // g].double()
            lse[a:b, h] = m
    return out, lse


def _by_slot(plane):
    """[pages, hkv, page, ...] -> [hkv, pages * page, ...]."""
    return plane.transpose(0, 1).flatten(1, 2)


def _exact_paged(state):
    q, cu = state["q"], state["cu"]
    k, v = _by_slot(state["k"]), _by_slot(state["v"])
    g = q.shape[1] // k.shape[0]
    out = torch.zeros(q.shape[0], q.shape[1], v.shape[2], dtype=torch.float64, device=q.device)
    lse = torch.zeros(q.shape[0], q.shape[1], dtype=torch.float64, device=q.device)
    for s, (a, b) in enumerate(zip(cu[:-1], cu[1:])):
        at = _slots(state, s, torch.arange(state["len"][s], device=q.device))
        for h in range(q.shape[1] if b > a else 0):
            x, m = _exact_head(q[a:b, h], k[h // g, at], state["scale"], len(at) - (b - a))
            out[a:b, h] = torch.exp(x - m[:, None]) @ v[h // g, at].double()
            lse[a:b, h] = m
    return out, lse


def _exact_mass(state):
    q, cu = state["q"], state["cu"]
    k, mass = _by_slot(state["k"]), _by_slot(state["mass"]).double().clone()
    g = q.shape[1] // k.shape[0]
    for s, (a, b) in enumerate(zip(cu[:-1], cu[1:])):
        at = _slots(state, s, torch.arange(state["len"][s], device=q.device))
        for h in range(q.shape[1] if b > a else 0):
            x, _ = _exact_head(q[a:b, h], k[h // g, at], state["scale"], len(at) - (b - a))
            mass[h // g].index_add_(0, at, torch.exp(x - state["lse"][a:b, h].double()[:, None]).sum(0))
    return mass.view(k.shape[0], -1, state["page"]).transpose(0, 1)


def _exact_append(state):
    planes = []
    for old, new in (("k", state["new_k"]), ("v", state["new_v"]), ("mass", None)):
        flat = _by_slot(state[old]).double().clone()
        for s, (a, b) in enumerate(zip(state["cu"][:-1], state["cu"][1:])):
            at = _slots(state, s, torch.arange(state["len"][s] - (b - a), state["len"][s], device=flat.device))
            flat[:, at] = 0.0 if new is None else new[a:b].double().transpose(0, 1)
        planes.append(flat.view(flat.shape[0], -1, state["page"], *flat.shape[2:]).transpose(0, 1))
    return tuple(planes)


def _exact_evict(state):
    case = state["case"]
    budget, sink, recent = case["budget"], case["sink"], case["recent"]
    flat = [_by_slot(state[p]).double().clone() for p in ("k", "v", "mass")]
    weights = _by_slot(state["mass"]).cpu().double().numpy()
    kept = []
    for s, length in enumerate(state["len"]):
        at = _slots(state, s, torch.arange(length, device="cuda"))
        to = _slots(state, s, torch.arange(min(length, budget), device="cuda"), "new_table")
        kept.append([])
        for h in range(flat[0].shape[0]):
            ids = list(range(length))
            if length > budget:
                w = weights[h, at.cpu().numpy()]
                middle = sorted(range(sink, length - recent), key=lambda j: (-w[j], j))
                ids = ids[:sink] + sorted(middle[: budget - sink - recent]) + ids[length - recent :]
            kept[-1].append(ids + [-1] * (budget - len(ids)))
            for plane in flat:
                plane[h, to] = plane[h, at[torch.tensor(ids, dtype=torch.long, device="cuda")]]
    shaped = [f.view(f.shape[0], -1, state["page"], *f.shape[2:]).transpose(0, 1) for f in flat]
    return (torch.tensor(kept, dtype=torch.int32), torch.tensor([min(v, budget) for v in state["len"]], dtype=torch.int32), *shaped)
