"""The workloads that the shared-prefix attention and the cache eviction are measured on.

`run` computes each operator either in elementary torch operations (`own = False`) or through
the library (`own = True`):

attend   wh_prefix_attention: the queries of a batch attend over the keys of their group's
         shared prefix and over their own keys; with `weigh`, the attention weight that every
         key received is added to its accumulator.
evict    wh_cache_evict: every head of a cache keeps its most recent keys and, of the older
         ones, those with the most accumulated weight.
"""
import random

import torch

own = False

HD = 64           # values per head
MOST_BYTES = 1.2e9
MOST_FLOPS = 1.97e10


# ---------------------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------------------
def _attend(name, groups, batch, n_head, n_kv_head=None, n_query=1, prefix=0, prefix_low=None, mine=0, mine_low=None,
            ragged=False, weigh=False):
    """groups prefixes of prefix_low .. prefix keys shared by batch sequences (equally many each, or
    ragged), n_query queries a sequence, mine_low .. mine keys of a sequence's own."""
    return {"name": name, "op": "attend", "groups": groups, "batch": batch, "n_head": n_head,
            "n_kv_head": n_kv_head or n_head, "n_query": n_query, "prefix": prefix,
            "prefix_low": prefix if prefix_low is None else prefix_low, "mine": mine,
            "mine_low": mine if mine_low is None else mine_low, "ragged": ragged, "weigh": weigh}


def _evict(name, sets, n_head, cap, low, budget, recent, in_place=False):
    """sets caches of low .. cap keys, cut to budget keys, of which the last `recent` stay unasked."""
    return {"name": name, "op": "evict", "sets": sets, "n_head": n_head, "cap": cap, "low": low, "budget": budget,
            "recent": recent, "in_place": in_place}


def listed():
    return [
        # one window's five hypotheses in a tiny-width decoder layer, over the window's 1500 encoder positions:
        # a single utterance, where the latency of the call is all that counts
        _attend("beams_one_window", 1, 5, 6, prefix=1500),
        # the same at large-v3 width for 16 windows at once: the cross-attention of one beam-search step
        _attend("beams_16_windows", 16, 80, 20, prefix=1500),
        # best-of search with as many hypotheses as each window still has, windows of unequal encoder length, and
        # the weight of every encoder position kept (for word times, or to drop silent positions)
        _attend("beams_ragged_weights", 16, 83, 20, prefix=1500, prefix_low=211, ragged=True, weigh=True),
        # self-attention of 64 utterances decoded under one text prompt, each with its own tokens so far
        _attend("prompt_64", 1, 64, 20, prefix=223, mine=224, mine_low=1),
        # verifying a draft's four tokens for a few hypotheses of 16 windows, four query heads to a key head
        _attend("verify_grouped_heads", 16, 67, 20, 5, n_query=4, prefix=1500, prefix_low=977, mine=37, mine_low=0,
                ragged=True),
        # 32 sequences that ask the same 20 windows' memory (10 minutes of audio)
        _attend("long_memory", 1, 32, 20, prefix=30000),
        # 256 sequences under one long context, with some tokens of their own
        _attend("wide_batch", 1, 256, 20, prefix=15000, mine=61, mine_low=1),
        # no prefix: a decoder's self-attention that keeps the weight its keys received, for eviction
        _attend("own_weights", 0, 80, 20, mine=448, mine_low=1, weigh=True),
        # the caches of five hypotheses of one layer, cut to half
        _evict("evict_beams", 5, 6, 448, 448, 224, 32),
        # all 32 layers' self-attention caches of 16 sequences in one call
        _evict("evict_layers", 512, 20, 448, 301, 224, 64),
        # cross-attention keys of 16 windows of unequal length, cut to a third, in place
        _evict("evict_cross_in_place", 16, 20, 1500, 333, 500, 0, in_place=True),
        # one long memory
        _evict("evict_long", 1, 20, 30000, 30000, 4001, 100),
    ]


def _log(rng, low, high):
    return min(high, max(low, int(round(low * (high / low) ** rng.random()))))


def _draw_attend(rng):
    n_head = rng.choice([6, 8, 12, 20])
    rep = rng.choice([1, 1, 1, 2, n_head // 2 if n_head < 12 else 4])
    kind = rng.choice(["cross", "prompt", "verify", "long", "own"])
    weigh = rng.random() < 0.3
    if kind == "cross":
        groups = _log(rng, 1, 24)
        return _attend("", groups, groups * rng.randint(1, 8), n_head, n_head // rep, 1, _log(rng, 100, 1500),
                       prefix_low=1, ragged=rng.random() < 0.5, weigh=weigh)
    if kind == "prompt":
        return _attend("", _log(rng, 1, 8), _log(rng, 8, 256), n_head, n_head // rep, 1, _log(rng, 1, 447), mine=_log(rng, 1, 448),
                       mine_low=0, ragged=True, weigh=weigh)
    if kind == "verify":
        groups = _log(rng, 1, 24)
        return _attend("", groups, groups * rng.randint(1, 5), n_head, n_head // rep, rng.randint(2, 9),
                       _log(rng, 100, 1500), mine=_log(rng, 1, 448), mine_low=0, ragged=rng.random() < 0.5, weigh=weigh)
    if kind == "long":
        groups = rng.randint(1, 3)
        return _attend("", groups, groups * _log(rng, 1, 256), n_head, n_head // rep, 1, _log(rng, 2000, 60000),
                       mine=rng.choice([0, _log(rng, 1, 448)]), mine_low=0, weigh=weigh)
    return _attend("", 0, _log(rng, 1, 256), n_head, n_head // rep, rng.choice([1, 1, 3]), mine=_log(rng, 1, 2000),
                   mine_low=0, weigh=weigh)


def _draw_evict(rng):
    cap = _log(rng, 16, 30000)
    budget = max(1, int(cap * rng.uniform(0.1, 0.9)))
    return _evict("", _log(rng, 1, 512), rng.choice([6, 8, 12, 20]), cap, rng.choice([0, cap // 2, cap]), budget,
                  rng.choice([0, budget // 8, budget // 2, budget]), in_place=rng.random() < 0.3)


def draw(rng):
    while True:
        case = _draw_attend(rng) if rng.random() < 0.6 else _draw_evict(rng)
        w = work(case)
        held = case.get("sets", 0) * case.get("cap", 0) * case.get("n_head", 0) * 4 * HD
        if 0 < w["bytes"] <= MOST_BYTES and w["flops"] <= MOST_FLOPS and held <= MOST_BYTES:
            case.pop("name")
            return case


def _lengths(case):
    """What a case's lengths are: (group starts, prefix lengths, own lengths) or the key counts of
    the caches.  They belong to the case; the seed makes the values."""
    rng = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    if case["op"] == "evict":
        return [rng.randint(case["low"], case["cap"]) for _ in range(case["sets"])]
    groups, batch = case["groups"], case["batch"]
    if groups and case["ragged"]:
        starts = [0] + sorted(rng.randint(0, batch) for _ in range(groups - 1)) + [batch]
    else:
        starts = [g * (batch // groups) for g in range(groups + 1)] if groups else [0]
    return (starts, [rng.randint(case["prefix_low"], case["prefix"]) for _ in range(groups)],
            [rng.randint(case["mine_low"], case["mine"]) for _ in range(batch)])


def work(case):
    h = case.get("n_kv_head", case["n_head"])
    if case["op"] == "evict":
        counts = _lengths(case)
        moved = sum(min(n, case["budget"]) for n in counts)
        # the weights are read, and what stays is read and written: key, value, weight and index
        return {"bytes": h * (4.0 * sum(counts) + moved * (2.0 * 4 * HD + 4 + 4)), "flops": 0.0}
    starts, n_pre, n_own = _lengths(case)
    rows = case["batch"] * case["n_query"] * case["n_head"]
    size = [b - a for a, b in zip(starts, starts[1:])]
    used = [n for n, s in zip(n_pre, size) if s]            # a group without sequences is not read
    keys = sum(used) + sum(n_own)
    pairs = sum(s * n for s, n in zip(size, n_pre)) + sum(n_own)
    nbytes = keys * h * 4.0 * HD + rows * 4.0 * HD
    if case["weigh"]:
        nbytes += keys * h * 8.0
    return {"bytes": nbytes, "flops": pairs * case["n_query"] * case["n_head"] * 4.0 * HD}


# ---------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------
def _cache(gen, sets, cap, heads):
    """Keys and values as projections leave them: unit scale, some keys that most queries attend to
    (a first token, punctuation), values off centre."""
    k = torch.randn(sets, cap, heads * HD, generator=gen, device="cuda")
    k *= torch.where(torch.rand(sets, cap, 1, generator=gen, device="cuda") < 0.05, 2.0, 1.0)
    v = torch.randn(sets, cap, heads * HD, generator=gen, device="cuda") + 0.25
    return k.to(torch.bfloat16), v.to(torch.bfloat16)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    s = dict(case)
    if case["op"] == "evict":
        sets, h, cap = case["sets"], case["n_head"], case["cap"]
        s["k"], s["v"] = _cache(gen, sets, cap, h)
        # accumulated weights: a few keys took most of it, many took (next to) nothing and tie at zero
        w = torch.rand(sets, h, cap, generator=gen, device="cuda") ** 8 * 20
        s["weight"] = torch.where(w < 1e-4, torch.zeros_like(w), w)
        s["n_keys"] = _ints(_lengths(case))
        shape = (sets, cap if case["in_place"] else case["budget"])
        s["k_out"], s["v_out"] = torch.zeros(2, *shape, h * HD, dtype=torch.bfloat16, device="cuda").unbind(0)
        s["weight_out"] = torch.zeros(sets, h, shape[1], device="cuda")
        s["n_out"] = torch.zeros(sets, dtype=torch.int32, device="cuda")
        s["kept"] = torch.full((sets, h, case["budget"]), -1, dtype=torch.int32, device="cuda")
        return s
    starts, n_pre, n_own = _lengths(case)
    h, rows = case["n_kv_head"], case["batch"] * case["n_query"]
    s["q"] = (1.2 * torch.randn(rows, case["n_head"] * HD, generator=gen, device="cuda")).to(torch.bfloat16)
    for what, sets, cap, counts in (("pre", case["groups"], case["prefix"], n_pre), ("own", case["batch"], case["mine"], n_own)):
        if not sets or not cap:
            s[what] = None
            continue
        k, v = _cache(gen, sets, cap, h)
        s[what] = {"k": k, "v": v, "n_keys": _ints(counts)}
        if case["weigh"]:
            s[what]["weight"] = torch.rand(sets, h, cap, generator=gen, device="cuda")
    s["starts"] = _ints(starts)
    s["widest"] = max((b - a for a, b in zip(starts, starts[1:])), default=0)
    s["out"] = torch.empty(rows, case["n_head"] * HD, dtype=torch.bfloat16, device="cuda")
    return s


# ---------------------------------------------------------------------------------------
# The passes
# ---------------------------------------------------------------------------------------
def run(s):
    if s["op"] == "evict":
        return _evict_own(s) if own else _evict_plain(s)
    return _attend_own(s) if own else _attend_plain(s)


def _attend_own(s):
    from whisper_audio_encoder_gb300 import wh
    weights = {what: s[what]["weight"].clone() for what in ("pre", "own") if s["weigh"] and s[what]}
    keys = lambda what: wh.Keys(s[what]["k"], s[what]["v"], s[what]["n_keys"], weights.get(what)) if s[what] else None  # noqa: E731
    out = wh.wh_prefix_attention(s["q"], s["n_head"], prefix=keys("pre"), own=keys("own"), n_kv_head=s["n_kv_head"],
                                 n_query=s["n_query"], group_start=s["starts"] if s["ragged"] else None, out=s["out"])
    return {"out": out, **weights}


def _evict_own(s):
    from whisper_audio_encoder_gb300 import wh
    if s["in_place"]:
        k, v, weight, n = s["k_out"].copy_(s["k"]), s["v_out"].copy_(s["v"]), s["weight_out"].copy_(s["weight"]), s["n_out"].copy_(s["n_keys"])
        wh.wh_cache_evict(wh.Keys(k, v, n, weight), s["n_head"], s["budget"], s["recent"], kept=s["kept"])
    else:
        wh.wh_cache_evict(wh.Keys(s["k"], s["v"], s["n_keys"], s["weight"]), s["n_head"], s["budget"], s["recent"],
                          out=wh.Keys(s["k_out"], s["v_out"], s["n_out"], s["weight_out"]), kept=s["kept"])
    return {"k": s["k_out"], "v": s["v_out"], "weight": s["weight_out"], "n": s["n_out"], "kept": s["kept"]}


def _heads(x, h):
    """[sets][keys][h * 64] -> float32 [sets][h][keys][64]"""
    return x.float().view(x.shape[0], x.shape[1], h, HD).transpose(1, 2)


def _live(counts, cap, back=0):
    return torch.arange(cap, device="cuda") < (counts[:, None] - back)


def _attend_plain(s):
    b, h, nq, hq = s["batch"], s["n_kv_head"], s["n_query"], s["n_head"]
    rep, pre, mine = hq // h, s["pre"], s["own"]
    q = s["q"].float().view(b, nq, h, rep, HD) * HD ** -0.5
    scores = []
    if pre:
        # sequence i of group g is row (g, i) of a table as wide as the widest group
        starts = s["starts"].long()
        table = starts[:-1, None] + torch.arange(s["widest"], device="cuda")
        there = table < starts[1:, None]
        table = table.clamp(max=b - 1)
        seq = torch.arange(b, device="cuda")
        group = torch.searchsorted(starts[1:].contiguous(), seq, right=True)
        place = seq - starts[group]
        g, n = len(starts) - 1, pre["k"].shape[1]
        rows = q[table].permute(0, 3, 1, 2, 4, 5).reshape(g, h, -1, HD)
        x = (rows @ _heads(pre["k"], h).transpose(2, 3)).masked_fill(~_live(pre["n_keys"], n)[:, None, None], float("-inf"))
        scores.append(x.view(g, h, s["widest"], nq, rep, n)[group, :, place])
    if mine:
        m = mine["k"].shape[1]
        x = q.permute(0, 2, 1, 3, 4).reshape(b, h, nq * rep, HD) @ _heads(mine["k"], h).transpose(2, 3)
        # query i of nq is the sequence's (nq - i)-th last token: it sees no key behind its own
        seen = torch.stack([_live(mine["n_keys"], m, back) for back in reversed(range(nq))], 1)
        scores.append(x.view(b, h, nq, rep, m).masked_fill(~seen[:, None, :, None], float("-inf")))
    x = torch.cat(scores, -1)
    top = x.amax(-1, keepdim=True)
    x = torch.exp(x - torch.where(top.isinf(), torch.zeros_like(top), top))
    total = x.sum(-1, keepdim=True)
    x = x / torch.where(total == 0, torch.ones_like(total), total)
    o, got = 0, {}
    if pre:
        p = x[..., :n][table] * there[:, :, None, None, None, None]
        p = p.transpose(1, 2).reshape(g, h, -1, n)
        v = _heads(pre["v"], h).masked_fill(~_live(pre["n_keys"], n)[:, None, :, None], 0)
        o = o + (p @ v).view(g, h, s["widest"], nq, rep, HD)[group, :, place]
        if s["weigh"]:
            got["pre"] = pre["weight"] + p.sum(2)
    if mine:
        p = x[..., -m:].reshape(b, h, nq * rep, m)
        v = _heads(mine["v"], h).masked_fill(~_live(mine["n_keys"], m)[:, None, :, None], 0)
        o = o + (p @ v).view(b, h, nq, rep, HD)
        if s["weigh"]:
            got["own"] = mine["weight"] + p.sum(2)
    s["out"].copy_(o.transpose(1, 2).reshape(b * nq, hq * HD))
    return {"out": s["out"], **got}


def _evict_plain(s):
    k, v, w, n = s["k"], s["v"], s["weight"], s["n_keys"].long()
    sets, cap, h, m, r = s["sets"], s["cap"], s["n_head"], s["budget"], s["recent"]
    if s["in_place"]:
        s["k_out"].copy_(k), s["v_out"].copy_(v), s["weight_out"].copy_(w), s["n_out"].copy_(s["n_keys"])
    at = torch.arange(cap, device="cuda")
    rank = torch.where((at >= n[:, None] - r)[:, None], torch.inf, w).masked_fill((at >= n[:, None])[:, None], -torch.inf)
    # the m first in order of weight, equal ones in order of place; back in order of place
    best = rank.sort(dim=-1, descending=True, stable=True).indices[..., :m].sort(-1).values
    left = torch.minimum(n, torch.full_like(n, m))
    live = (torch.arange(m, device="cuda") < left[:, None])[:, None]
    s["kept"].copy_(torch.where(live, best.int(), s["kept"]))
    pick = best.transpose(1, 2)[..., None].expand(-1, -1, -1, HD)
    rows = live.transpose(1, 2)[..., None]
    for_keys = lambda x, to: torch.where(rows, x.view(sets, cap, h, HD).gather(1, pick), to[:, :m].view(sets, m, h, HD)).view(sets, m, h * HD)  # noqa: E731
    s["k_out"][:, :m] = for_keys(k, s["k_out"])
    s["v_out"][:, :m] = for_keys(v, s["v_out"])
    s["weight_out"][..., :m] = torch.where(live, w.gather(-1, best), s["weight_out"][..., :m])
    s["n_out"].copy_(left)
    return {"k": s["k_out"], "v": s["v_out"], "weight": s["weight_out"], "n": s["n_out"], "kept": s["kept"]}


# ---------------------------------------------------------------------------------------
# The definitions, in 64 bits, one sequence or head at a time
# ---------------------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return _evict_exact(s, case) if case["op"] == "evict" else _attend_exact(s, case)


def _attend_exact(s, case):
    starts, n_pre, n_own = _lengths(case)
    h, nq, hq = case["n_kv_head"], case["n_query"], case["n_head"]
    out = torch.zeros(case["batch"], nq, h, hq // h, HD, dtype=torch.float64, device="cuda")
    sums = {what: s[what]["weight"].double() for what in ("pre", "own") if case["weigh"] and s[what]}
    group_of = {b: g for g in range(case["groups"]) for b in range(starts[g], starts[g + 1])}
    for b in range(case["batch"]):
        q = s["q"][b * nq:(b + 1) * nq].double().view(nq, h, hq // h, HD)
        parts = []
        if b in group_of and s["pre"]:
            parts.append(("pre", group_of[b], n_pre[group_of[b]]))
        if s["own"]:
            parts.append(("own", b, n_own[b]))
        e, vs = [], []
        for what, at, n in parts:
            k = s[what]["k"][at, :n].double().view(n, h, HD)
            x = torch.einsum("ihrd,nhd->ihrn", q, k) / 8
            if what == "own":
                for i in range(nq):
                    x[i, :, :, max(0, n - (nq - 1 - i)):] = -torch.inf
            e.append(x)
            vs.append(s[what]["v"][at, :n].double().view(n, h, HD))
        p = torch.softmax(torch.cat(e, -1), -1).nan_to_num(0.0)   # a query that sees nothing: zeros
        out[b] = torch.einsum("ihrn,nhd->ihrd", p, torch.cat(vs))
        done = 0
        for what, at, n in parts:
            if what in sums:
                sums[what][at, :, :n] += p[..., done:done + n].sum((0, 2))
            done += n
    return {"out": out.view(-1, hq * HD), **sums}


def _evict_exact(s, case):
    import numpy as np
    m, r, h = case["budget"], case["recent"], case["n_head"]
    w, counts, kept = s["weight"].cpu().numpy(), _lengths(case), s["kept"].cpu().numpy()
    k, v, weight = (s[x].double() for x in (("k", "v", "weight") if case["in_place"] else ("k_out", "v_out", "weight_out")))
    for i, n in enumerate(counts):
        for j in range(h):
            stay = np.arange(n)
            if n > m:
                old = np.lexsort((np.arange(n - r), -w[i, j, :n - r]))[:m - r]
                stay = np.concatenate([np.sort(old), np.arange(n - r, n)])
            kept[i, j, :len(stay)] = stay
    for i, n in enumerate(counts):
        c = min(n, m)
        at = torch.from_numpy(kept[i, :, :c]).long().to("cuda")
        for src, to in (("k", k), ("v", v)):
            x = s[src][i].view(-1, h, HD).gather(0, at.T[..., None].expand(-1, -1, HD))
            to[i, :c] = x.reshape(c, h * HD).double()
        weight[i, :, :c] = s["weight"][i].gather(-1, at).double()
    return {"k": k, "v": v, "weight": weight, "n": np.minimum(counts, m).astype(np.int32), "kept": kept}
