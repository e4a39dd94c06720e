"""Measured calls of the operators that a speculative step with a drafted tree over a paged cache is made of.

* ``tree_masks``         - which nodes of its tree a drafted node sees, and its position, from parent indices;
* ``norm_rope_write_kv`` - norms of query and key heads, rotary positions and the paged write in one pass;
* ``attend_tree``        - attention of the nodes over their request's cached context and their own branch;
* ``accept_tree``        - the branch that the target model's choices confirm;
* ``compact_tree``       - that branch's keys and values moved together in every layer, blocks behind it given back.

``own`` chooses between the plain form (elementary torch operations in 32 bits) and the framework's calls.
Lengths and layouts are a function of the case; trees, values, and which block holds what, of the seed.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
DEVICE = "cuda"
EPS = 1e-6


# ---- cases ---------------------------------------------------------------------------------

def listed():
    qwen = {"hq": 28, "hkv": 4, "d": 128, "bs": 16}
    return [
        # trees of 16 nodes for each of 64 running requests: launch latency
        {"name": "masks_step", "op": "masks", "b": 64, "new_lo": 16, "new_hi": 16, "ctx_lo": 512, "ctx_hi": 4096, "lens": 1},
        # a large batch of ragged trees, some of several mask words, some requests without a tree
        {"name": "masks_ragged", "op": "masks", "b": 256, "new_lo": 0, "new_hi": 200, "ctx_lo": 0, "ctx_hi": 4096, "lens": 2},
        # odd token count, interleaved pairs over part of a small head, 32-bit cache, far positions, weights stored as w - 1
        {"name": "norm_rope_part_f32", "op": "norm", "t": 1001, "hq": 16, "hkv": 8, "d": 64, "bs": 16, "rot": 32,
         "dtype": "f32", "weights": "f32", "offset": 1.0, "layout": "interleaved", "max_pos": 1000000, "scaling": "linear"},
        # prompt chunk, or the trees of a very large batch: 8192 tokens, 16-bit cache
        {"name": "norm_rope_chunk", "op": "norm", "t": 8192, **qwen, "rot": 128, "dtype": "bf16", "weights": "bf16",
         "offset": 0.0, "layout": "half", "max_pos": 131072, "scaling": "ramp"},
        # trees of 16 nodes for each of 64 requests: bound by the cache's bytes
        {"name": "attend_tree_step", "op": "attend", "b": 64, "new_lo": 16, "new_hi": 16, "ctx_lo": 512, "ctx_hi": 4096,
         **qwen, "dtype": "bf16", "lens": 5},
        # few requests with wide trees: bound by the products
        {"name": "attend_tree_wide", "op": "attend", "b": 16, "new_lo": 48, "new_hi": 128, "ctx_lo": 2048, "ctx_hi": 8192,
         **qwen, "dtype": "bf16", "lens": 6},
        # single tokens and small trees on long contexts: the contexts have to be split
        {"name": "attend_tree_long", "op": "attend", "b": 8, "new_lo": 1, "new_hi": 8, "ctx_lo": 32768, "ctx_hi": 131072,
         "hq": 32, "hkv": 8, "d": 128, "bs": 16, "dtype": "bf16", "lens": 7},
        # ragged batch of short requests, head size 64, 32-token blocks, requests without a node among them
        {"name": "attend_tree_mixed_d64", "op": "attend", "b": 61, "new_lo": 0, "new_hi": 40, "ctx_lo": 0, "ctx_hi": 900,
         "hq": 16, "hkv": 4, "d": 64, "bs": 32, "dtype": "f16", "lens": 8},
        # trees of 16 nodes for each of 64 requests: launch latency
        {"name": "accept_step", "op": "accept", "b": 64, "new_lo": 16, "new_hi": 16, "depth": 8, "lens": 9},
        # a large batch of ragged trees
        {"name": "accept_ragged", "op": "accept", "b": 256, "new_lo": 0, "new_hi": 200, "depth": 16, "lens": 10},
        # 64 requests, a few nodes of 16 accepted, 28 layers
        {"name": "compact_step", "op": "compact", "b": 64, "new_lo": 16, "new_hi": 16, "ctx_lo": 16, "ctx_hi": 512,
         "depth": 5, "layers": 28, "hkv": 4, "d": 128, "bs": 16, "dtype": "bf16", "lens": 11},
        # 256 requests with ragged trees, up to 16 nodes accepted, 28 layers
        {"name": "compact_ragged", "op": "compact", "b": 256, "new_lo": 0, "new_hi": 64, "ctx_lo": 16, "ctx_hi": 256,
         "depth": 16, "layers": 28, "hkv": 4, "d": 128, "bs": 16, "dtype": "bf16", "lens": 12},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["masks", "norm", "attend", "accept", "compact"])
    case = {"op": op}
    if op == "norm":
        hkv, d = rng.choice([1, 2, 4, 8]), rng.choice([64, 80, 128, 256])
        dtype = rng.choice(["f32", "f16", "bf16"])
        return case | {"t": _log_int(rng, 1, 2048), "hkv": hkv, "hq": hkv * rng.choice([1, 2, 4, 7]), "d": d,
                       "bs": rng.choice([16, 32]), "rot": rng.choice([d // 4, d // 2, d]), "dtype": dtype,
                       "weights": rng.choice(["f32", dtype]), "offset": rng.choice([0.0, 1.0]),
                       "layout": rng.choice(["half", "interleaved"]), "max_pos": _log_int(rng, 64, 1000000),
                       "scaling": rng.choice(["none", "linear", "ramp"])}
    case["lens"] = rng.randrange(1 << 30)
    if op in ("masks", "accept"):
        lo, hi = sorted((_log_int(rng, 1, 200), _log_int(rng, 1, 200)))
        case |= {"b": _log_int(rng, 1, 256), "new_lo": lo - 1, "new_hi": hi}
        return case | ({"ctx_lo": 0, "ctx_hi": _log_int(rng, 16, 4096)} if op == "masks" else {"depth": _log_int(rng, 1, 32)})
    hkv, bs = rng.choice([1, 2, 4, 8]), rng.choice([16, 32])
    if op == "compact":
        lo, hi = sorted((_log_int(rng, 1, 64), _log_int(rng, 1, 64)))
        return case | {"b": _log_int(rng, 1, 64), "new_lo": lo - 1, "new_hi": hi, "ctx_lo": 0,
                       "ctx_hi": _log_int(rng, 16, 256), "depth": _log_int(rng, 1, 16), "layers": _log_int(rng, 1, 28),
                       "hkv": hkv, "d": rng.choice([64, 80, 128]), "bs": bs, "dtype": rng.choice(["f32", "f16", "bf16"])}
    # bounded so that no drawn case exceeds the case of wide trees
    lo, hi = sorted((_log_int(rng, 1, 64), _log_int(rng, 1, 64)))
    return case | {"b": _log_int(rng, 1, 8), "new_lo": lo - 1, "new_hi": hi, "ctx_lo": 0, "ctx_hi": _log_int(rng, 16, 8192),
                   "hkv": hkv, "hq": hkv * rng.choice([1, 2, 4] if hkv == 8 else [1, 2, 4, 7, 8]), "d": rng.choice([64, 128]),
                   "bs": bs, "dtype": rng.choice(["f16", "bf16"])}


def _lengths(case):
    """(cached tokens, nodes) of each request, int64."""
    rng = np.random.default_rng(case["lens"])
    b = case["b"]
    old = rng.integers(case.get("ctx_lo", 0), case.get("ctx_hi", 0) + 1, b)
    new = rng.integers(case["new_lo"], case["new_hi"] + 1, b)
    if new.max() <= 0:
        new[0] = 1
    return old, new


def _words(new):
    return (int(new.max()) + 63) // 64


def _blocks(n, bs):
    return (n + bs - 1) // bs


def _inv_freq(rot, scaling):
    """Angle per position of each pair, float64: plain, positions divided by a factor, or slow pairs alone divided."""
    inv = 10000.0 ** (-np.arange(0, rot, 2, dtype=np.float64) / rot)
    if scaling == "linear":
        inv = inv / 8.0
    elif scaling == "ramp":
        turns = 8192 * inv / (2.0 * np.pi)  # turns over the context the model was trained on
        keep = np.clip((turns - 1.0) / (32.0 - 1.0), 0.0, 1.0)
        inv = inv * keep + inv / 16.0 * (1.0 - keep)
    return inv


def _rope_factor(scaling):
    return 0.1 * math.log(16.0) + 1.0 if scaling == "ramp" else 1.0


# ---- inputs --------------------------------------------------------------------------------

def _up(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEVICE)


def _normal(gen, shape, dtype=torch.float32):
    return torch.randn(shape, generator=gen, device=DEVICE).to(dtype)


def _table(rng, counts, extra):
    """(blocks in the pool, a random block of the pool for each logical block, the blocks left)."""
    pool = int(counts.sum()) + extra
    perm = rng.permutation(pool).astype(np.int32)
    table = np.full((len(counts), max(1, int(counts.max()))), -1, np.int32)
    held = np.arange(table.shape[1]) < counts[:, None]
    table[held] = perm[:int(counts.sum())]
    return pool, table, perm[int(counts.sum()):]


def _trees(rng, new):
    """Parent of each node in its request (-1: the first): chains, narrow and wide trees, a request to a kind."""
    off = np.concatenate([[0], np.cumsum(new)])
    seq = np.repeat(np.arange(len(new)), new)
    i = np.arange(off[-1]) - off[seq]
    span = rng.choice([1, 3, 9, 1 << 30], len(new))[seq]  # how far back a parent may be
    parents = i - 1 - np.floor(rng.random(len(i)) * np.minimum(i, span)).astype(np.int64)
    return off.astype(np.int32), np.where(i == 0, -1, parents).astype(np.int32), i, seq


def _paths(rng, off, parents, new, depth):
    """A branch of each tree: `accepted` [requests, depth], first node first, -1 behind its last; and how many."""
    b = len(new)
    accepted, count = np.full((b, depth), -1, np.int32), np.zeros(b, np.int32)
    for r in np.flatnonzero(new > 0):
        node, path = int(rng.integers(0, new[r])), []
        while node >= 0:
            path.append(node)
            node = int(parents[off[r] + node])
        path = path[::-1][:depth]
        accepted[r, :len(path)], count[r] = path, len(path)
    return accepted, count


def prepare(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device=DEVICE).manual_seed(int(seed))
    s = {"case": case, "op": case["op"]}
    i32 = {"dtype": torch.int32, "device": DEVICE}
    if case["op"] == "norm":
        t, hq, hkv, d, bs, dt = case["t"], case["hq"], case["hkv"], case["d"], case["bs"], DTYPES[case["dtype"]]
        pool = _blocks(t, bs) + 8
        slots = rng.permutation(pool * bs)[:t].astype(np.int64)
        slots[rng.random(t) < 0.02] = -1  # padding rows
        # queries, keys and values as the projection leaves them: one row per token
        q, k, v = (_normal(gen, (t, (hq + 2 * hkv) * d)) * 2.0).to(dt).split([hq * d, hkv * d, hkv * d], 1)
        weights = [(1.0 + 0.2 * _normal(gen, (d,)) - case["offset"]).to(DTYPES[case["weights"]]) for _ in range(2)]
        return s | {"positions": _up(rng.integers(0, case["max_pos"], t).astype(np.int32)), "slots": _up(slots),
                    "key_cache": torch.zeros(pool, hkv, bs, d, dtype=dt, device=DEVICE),
                    "value_cache": torch.zeros(pool, hkv, bs, d, dtype=dt, device=DEVICE),
                    "query": q.unflatten(1, (hq, d)), "key": k.unflatten(1, (hkv, d)), "value": v.unflatten(1, (hkv, d)),
                    "query_out": torch.empty(t, hq, d, dtype=dt, device=DEVICE), "q_weight": weights[0],
                    "k_weight": weights[1], "inv_freq": _up(_inv_freq(case["rot"], case["scaling"])),
                    "factor": _rope_factor(case["scaling"])}
    old, new = _lengths(case)
    off, parents, local, seq = _trees(rng, new)
    t, b = int(off[-1]), len(new)
    s |= {"q_offsets": _up(off), "parents": _up(parents), "max_new": int(new.max())}
    if case["op"] == "masks":
        return s | {"context_lens": _up((old + new).astype(np.int32)), "words": _words(new),
                    "out": (torch.empty(t, **i32), torch.empty(t, _words(new), dtype=torch.int64, device=DEVICE))}
    if case["op"] == "accept":
        choices = rng.integers(0, 32000, t)
        tokens = rng.integers(0, 32000, t)
        right = (parents >= 0) & (rng.random(t) < 0.6)
        tokens[right] = choices[(off[seq] + parents)[right]]
        return s | {"tokens": _up(tokens), "choices": _up(choices), "depth": case["depth"],
                    "out": (torch.empty(b, case["depth"], **i32), torch.empty(b, **i32),
                            torch.empty(b, dtype=torch.int64, device=DEVICE))}
    hkv, d, bs, dt = case["hkv"], case["d"], case["bs"], DTYPES[case["dtype"]]
    lens = old + new
    pool, table, free = _table(rng, _blocks(lens, bs), 8)
    s |= {"block_tables": _up(table), "context_lens": _up(lens.astype(np.int32))}
    if case["op"] == "compact":
        accepted, count = _paths(rng, off, parents, new, case["depth"])
        pos = old[seq] + local
        stack = np.zeros(pool, np.int32)
        stack[:len(free)] = free
        shape = (case["layers"], pool, hkv, bs, d)
        return s | {"key_caches": _normal(gen, shape, dt), "value_caches": _normal(gen, shape, dt),
                    "slots": _up(table[seq, pos // bs].astype(np.int64) * bs + pos % bs), "accepted": _up(accepted),
                    "num_accepted": _up(count), "free_blocks": _up(stack),
                    "num_free": torch.tensor([len(free)], **i32), "out": (torch.empty(b, **i32), torch.empty(1, **i32))}
    s["mask"] = _plain_masks(s | {"words": _words(new)})["tree_mask"]
    s["key_cache"], s["value_cache"] = (_normal(gen, (pool, hkv, bs, d), dt) for _ in range(2))
    s["query"] = _normal(gen, (t, case["hq"], d), dt)
    return s | {"out": torch.empty(t, case["hq"], d, dtype=dt, device=DEVICE), "scale": 1.0 / math.sqrt(d)}


# ---- the plain form -------------------------------------------------------------------------

def _nodes(s):
    """(request, index in it, row of the parent or of the node itself where it has none) of each node."""
    off, parents = s["q_offsets"].long(), s["parents"].long()
    at = torch.arange(parents.shape[0], device=DEVICE)
    seq = torch.searchsorted(off, at, right=True) - 1
    return seq, at - off[seq], torch.where(parents >= 0, off[seq] + parents, at)


def _rounds(s):
    return range(max(1, (s["max_new"] - 1).bit_length()))


def _plain_masks(s):
    off = s["q_offsets"].long()
    seq, i, up = _nodes(s)
    w = s["words"]
    n = (off[1:] - off[:-1])[seq]
    bits = torch.zeros(len(i), 64 * w, dtype=torch.bool, device=DEVICE)
    bits[torch.arange(len(i), device=DEVICE), i] = True
    for _ in _rounds(s):  # twice as many ancestors each time
        bits, up = bits | bits[up], up[up]
    place = torch.ones(64, dtype=torch.int64, device=DEVICE) << torch.arange(64, device=DEVICE)
    mask = torch.where(bits.view(-1, w, 64), place, 0).sum(-1)
    pos = s["context_lens"].long()[seq] - n + bits.sum(1) - 1
    return {"positions": pos.int(), "tree_mask": mask}


def _plain_accept(s):
    off, depth = s["q_offsets"].long(), s["depth"]
    seq, i, up = _nodes(s)
    t, b = len(i), len(off) - 1
    at = torch.arange(t, device=DEVICE)
    right = (up != at) & (s["tokens"] == s["choices"][up])
    first = torch.full((t,), t, device=DEVICE).scatter_reduce_(0, up[right], at[right], "amin")
    good = (i == 0) | (right & (first[up] == at))
    for _ in _rounds(s):  # and so are its ancestors
        good, up = good & good[up], up[up]
    upto = torch.cat([good.new_zeros(1, dtype=torch.long), good.long().cumsum(0)])
    rank = upto[:-1] - upto[off[:-1]][seq]
    good &= rank < depth
    accepted = torch.full((b, depth), -1, dtype=torch.int32, device=DEVICE)
    accepted[seq[good], rank[good]] = i[good].int()
    count = (upto[off[1:]] - upto[off[:-1]]).clamp(max=depth)
    last = off[:-1] + accepted.gather(1, (count - 1).clamp(min=0)[:, None])[:, 0]
    token = torch.where(count > 0, s["choices"][last.clamp(0, t - 1)], -1)
    return {"accepted": accepted, "num_accepted": count.int(), "next_tokens": token}


def _plain_norm(s):
    case, bs = s["case"], s["case"]["bs"]
    q, k = (_rotate(_normed(s[n], s[w], case["offset"]), s["positions"], s).to(s[n].dtype)
            for n, w in (("query", "q_weight"), ("key", "k_weight")))
    ok = s["slots"] >= 0
    blk, off = s["slots"][ok] // bs, s["slots"][ok] % bs
    s["key_cache"][blk, :, off] = k[ok]
    s["value_cache"][blk, :, off] = s["value"][ok]
    return {"query": q, "key_cache": s["key_cache"], "value_cache": s["value_cache"]}


def _normed(x, weight, offset):
    x = x.float()
    return x / ((x * x).mean(-1, keepdim=True) + EPS).sqrt() * (weight.float() + offset)


def _rotate(x, pos, s):
    """Rotary positions of x [t, h, d] in 32 bits (angles in 64)."""
    inv, rot = s["inv_freq"], s["case"]["rot"]
    ang = pos.double()[:, None] * inv[None, :]
    c = (ang.cos() * s["factor"]).float()[:, None, :]
    n = (ang.sin() * s["factor"]).float()[:, None, :]
    r = x[..., :rot]
    if s["case"]["layout"] == "half":
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        r = torch.cat([a * c - b * n, a * n + b * c], -1)
    else:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * c - b * n, a * n + b * c], -1).flatten(-2)
    return torch.cat([r, x[..., rot:]], -1)


def _plain_attend(s):
    case = s["case"]
    hq, hkv, d, bs = case["hq"], case["hkv"], case["d"], case["bs"]
    g, n = hq // hkv, s["max_new"]
    table = s["block_tables"].long().clamp(min=0)
    b, m = table.shape
    k, v = (s[c][table].float().transpose(1, 2).reshape(b, hkv, m * bs, d) for c in ("key_cache", "value_cache"))
    off, lens = s["q_offsets"].long(), s["context_lens"].long()
    new = off[1:] - off[:-1]
    i = torch.arange(n, device=DEVICE)
    rows = (off[:-1, None] + i).clamp(max=s["query"].shape[0] - 1)
    q = s["query"][rows].float().reshape(b, n, hkv, g, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, g * n, d)
    x = (q @ k.transpose(2, 3)).view(b, hkv, g, n, m * bs).mul_(s["scale"])
    at = torch.arange(m * bs, device=DEVICE)[None, :] - (lens - new)[:, None]  # >= 0: a node of the tree
    words = s["mask"][rows]
    node = at[:, None, :].clamp(0, 64 * words.shape[2] - 1).expand(b, n, m * bs)
    seen = (words.gather(2, node >> 6) >> (node & 63)) & 1 == 1
    seen = (at < 0)[:, None, :] | (seen & (at < new[:, None])[:, None, :])
    x.masked_fill_(~seen[:, None, None], -math.inf)
    x.sub_(x.amax(-1, keepdim=True)).exp_()
    sums = x.sum(-1, keepdim=True)
    v = v.masked_fill((at >= new[:, None])[:, None, :, None], 0.0)
    o = (x.view(b, hkv, g * n, m * bs) @ v).view(b, hkv, g, n, d) / sums
    o = o.permute(0, 3, 1, 2, 4).reshape(b, n, hq, d)
    return o[i < new[:, None]].to(s["query"].dtype)


def _plain_compact(s):
    bs = s["case"]["bs"]
    off, lens, count, depth = s["q_offsets"].long(), s["context_lens"].long(), s["num_accepted"].long(), s["case"]["depth"]
    new = off[1:] - off[:-1]
    j = torch.arange(depth, device=DEVICE)
    seq, j = torch.nonzero(j < count[:, None], as_tuple=True)
    src, dst = s["slots"][off[seq] + s["accepted"][seq, j].long()], s["slots"][off[seq] + j]
    for c in (s["key_caches"], s["value_caches"]):
        c[:, dst // bs, :, dst % bs] = c[:, src // bs, :, src % bs]
    after = lens - new + count
    keep, had = (after + bs - 1) // bs, (lens + bs - 1) // bs
    back = had - keep
    col = torch.arange(s["block_tables"].shape[1], device=DEVICE)[None, :]
    give = (col >= keep[:, None]) & (col < had[:, None])
    at = (s["num_free"].long() + back.cumsum(0) - back)[:, None] + col - keep[:, None]
    s["free_blocks"][at[give]] = s["block_tables"][give]
    return _compact_outputs(s, after.int(), (s["num_free"] + back.sum()).int())


def _compact_outputs(s, lens, free):
    return {"key_caches": s["key_caches"], "value_caches": s["value_caches"], "context_lens": lens, "num_free": free,
            "free_blocks": s["free_blocks"]}


# ---- the framework's calls -------------------------------------------------------------------

def _own_run(s):
    import paged_kv_cache_129_gb300 as pa

    op = s["op"]
    if op == "masks":
        got = pa.tree_masks(s["parents"], s["context_lens"], s["q_offsets"], s["words"], out=s["out"])
        return {"positions": got.positions, "tree_mask": got.tree_mask}
    if op == "norm":
        case = s["case"]
        q = pa.norm_rope_write_kv(s["query"], s["key"], s["value"], s["key_cache"], s["value_cache"], s["q_weight"],
                                  s["k_weight"], s["inv_freq"], s["positions"], s["slots"], eps=EPS,
                                  weight_offset=case["offset"], layout=case["layout"], factor=s["factor"],
                                  query_out=s["query_out"])
        return {"query": q, "key_cache": s["key_cache"], "value_cache": s["value_cache"]}
    if op == "accept":
        got = pa.accept_tree(s["parents"], s["tokens"], s["choices"], s["q_offsets"], s["depth"], out=s["out"])
        return {"accepted": got.accepted, "num_accepted": got.num_accepted, "next_tokens": got.next_tokens}
    if op == "compact":
        got = pa.compact_tree(s["key_caches"], s["value_caches"], s["slots"], s["q_offsets"], s["accepted"],
                              s["num_accepted"], s["block_tables"], s["context_lens"], s["free_blocks"], s["num_free"],
                              out=s["out"])
        return _compact_outputs(s, got.context_lens, got.num_free)
    if "workspace" not in s:  # kept from call to call
        s["workspace"] = torch.empty(pa.attend_tree_workspace_size(
            s["query"].shape[0], s["block_tables"].shape[0], s["case"]["hq"], s["case"]["hkv"], s["case"]["d"],
            s["case"]["bs"], s["block_tables"].shape[1], s["query"].dtype), dtype=torch.uint8, device=DEVICE)
    return pa.attend_tree(s["query"], s["key_cache"], s["value_cache"], s["mask"], s["block_tables"], s["context_lens"],
                          s["q_offsets"], scale=s["scale"], out=s["out"], workspace=s["workspace"])


def run(state):
    if own:
        return _own_run(state)
    return {"masks": _plain_masks, "norm": _plain_norm, "attend": _plain_attend, "accept": _plain_accept,
            "compact": _plain_compact}[state["op"]](state)


# ---- what a pass cannot do without ---------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "norm":
        e, t = DTYPES[case["dtype"]].itemsize, case["t"]
        rows = case["hq"] + 2 * case["hkv"]
        normed = t * (case["hq"] + case["hkv"]) * case["d"]
        return {"bytes": 2 * t * rows * case["d"] * e + 12 * t + 4 * case["rot"] + 2 * case["d"] * DTYPES[case["weights"]].itemsize,
                "flops": 4 * normed + 3 * t * (case["hq"] + case["hkv"]) * case["rot"]}
    old, new = _lengths(case)
    t, b = int(new.sum()), len(new)
    if op == "masks":
        return {"bytes": t * (8 + 8 * _words(new)) + 8 * b, "flops": t * _words(new)}
    if op == "accept":
        return {"bytes": 20 * t + (16 + 4 * case["depth"]) * b, "flops": t}
    hkv, d, bs = case["hkv"], case["d"], case["bs"]
    e = DTYPES[case["dtype"]].itemsize
    if op == "compact":
        rng = np.random.default_rng(case["lens"] + 1)  # typical trees: those that a seed gives differ a little
        off, parents, _, _ = _trees(rng, new)
        accepted, _ = _paths(rng, off, parents, new, case["depth"])
        moved = int((accepted > np.arange(case["depth"])).sum())  # nodes that are not in their place already
        return {"bytes": moved * case["layers"] * 4 * hkv * d * e + 16 * moved + 20 * b, "flops": moved}
    used = np.where(new > 0, old + new, 0)
    off, parents, _, seq = _trees(np.random.default_rng(case["lens"] + 1), new)
    depth = np.ones(t, np.int64)
    for i in np.flatnonzero(parents >= 0):
        depth[i] += depth[off[seq[i]] + parents[i]]
    pairs = int((new * old).sum() + depth.sum())  # (query, key) pairs of a head that the mask leaves
    return {"bytes": int(used.sum()) * 2 * hkv * d * e + 4 * int(_blocks(used, bs).sum()) + 2 * t * case["hq"] * d * e
            + 8 * t * _words(new) + 8 * b, "flops": 4 * pairs * case["hq"] * d}


# ---- the definitions in 64 bits -------------------------------------------------------------------

def _cpu(t):
    return t.cpu().numpy()


def _branch(parents, node):
    """A node and its ancestors, the node first."""
    got = []
    while node >= 0:
        got.append(node)
        node = int(parents[node])
    return got


def _exact_masks(s):
    off, parents, lens = _cpu(s["q_offsets"]), _cpu(s["parents"]), _cpu(s["context_lens"])
    pos, mask = np.zeros(off[-1], np.int32), np.zeros((off[-1], s["words"]), np.uint64)
    for b in range(len(lens)):
        mine = parents[off[b]:off[b + 1]]
        for i in range(len(mine)):
            seen = _branch(mine, i)
            pos[off[b] + i] = lens[b] - len(mine) + len(seen) - 1
            for a in seen:
                mask[off[b] + i, a // 64] |= np.uint64(1 << (a % 64))
    return {"positions": pos, "tree_mask": mask.view(np.int64)}


def _exact_accept(s):
    off, parents, tokens, choices = (_cpu(s[n]) for n in ("q_offsets", "parents", "tokens", "choices"))
    b, depth = len(off) - 1, s["depth"]
    accepted, count, token = np.full((b, depth), -1, np.int32), np.zeros(b, np.int32), np.full(b, -1, np.int64)
    for r in range(b):
        node = 0 if off[r + 1] > off[r] else None
        while node is not None and count[r] < depth:
            accepted[r, count[r]] = node
            count[r] += 1
            token[r] = choices[off[r] + node]
            children = [c for c in range(node + 1, off[r + 1] - off[r])
                        if parents[off[r] + c] == node and tokens[off[r] + c] == token[r]]
            node = children[0] if children else None
    return {"accepted": accepted, "num_accepted": count, "next_tokens": token}


def _exact_norm(s):
    """Each head divided by its root mean square; then each pair (a, b) as the complex number a + ib, turned."""
    case = s["case"]
    bs, rot, half = case["bs"], case["rot"], case["rot"] // 2
    i = torch.arange(half, device=DEVICE)
    first = i if case["layout"] == "half" else 2 * i
    second = i + half if case["layout"] == "half" else 2 * i + 1
    freq = torch.from_numpy(_inv_freq(rot, case["scaling"])).to(DEVICE)
    turn = torch.polar(torch.tensor(s["factor"], dtype=torch.float64, device=DEVICE), s["positions"].double()[:, None] * freq)

    def one(x, weight):
        x = x.double()
        y = x * (x.square().sum(-1, keepdim=True) / case["d"] + EPS).rsqrt() * (weight.double() + case["offset"])
        z = torch.complex(y[..., first], y[..., second]) * turn[:, None, :]
        y[..., first], y[..., second] = z.real, z.imag
        return y

    q, k = one(s["query"], s["q_weight"]), one(s["key"], s["k_weight"])
    flat_k, flat_v = (s[c].double().transpose(1, 2).reshape(-1, case["hkv"], case["d"]) for c in ("key_cache", "value_cache"))
    use = torch.nonzero(s["slots"] >= 0)[:, 0]
    flat_k[s["slots"][use]] = k[use]
    flat_v[s["slots"][use]] = s["value"][use].double()
    kc, vc = (f.view(-1, bs, case["hkv"], case["d"]).transpose(1, 2).contiguous() for f in (flat_k, flat_v))
    return {"query": q, "key_cache": kc, "value_cache": vc}


def _exact_attend(s):
    case = s["case"]
    hkv, d, bs, g = case["hkv"], case["d"], case["bs"], case["hq"] // case["hkv"]
    old, new = _lengths(case)
    if float((new * (old + new)).sum()) * case["hq"] * d > 1e12:
        return None
    table, out, at, parents = s["block_tables"].long(), [], 0, _cpu(s["parents"])
    for b in range(len(old)):
        n, length = int(new[b]), int(old[b] + new[b])
        if n == 0:
            continue
        seen = torch.ones(n, length, dtype=torch.bool)
        seen[:, length - n:] = False
        for t in range(n):
            seen[t, [length - n + a for a in _branch(parents[at:at + n], t)]] = True
        seen = seen.to(DEVICE)
        ids = table[b, :_blocks(length, bs)]
        for h in range(hkv):
            k, v = (s[c][ids, h].double().reshape(-1, d)[:length] for c in ("key_cache", "value_cache"))
            q = s["query"][at:at + n, h * g:(h + 1) * g].double()
            x = torch.einsum("tgd,pd->tgp", q, k) * s["scale"]
            p = torch.softmax(x.masked_fill(~seen[:, None, :], -math.inf), -1)
            out.append((at, h, torch.einsum("tgp,pd->tgd", p, v)))
        at += n
    o = torch.empty(at, case["hq"], d, dtype=torch.float64, device=DEVICE)
    for a, h, x in out:
        o[a:a + x.shape[0], h * g:(h + 1) * g] = x
    return o


def _exact_compact(s):
    bs = s["case"]["bs"]
    off, lens, slots, accepted, count, table = (_cpu(s[n]) for n in ("q_offsets", "context_lens", "slots", "accepted",
                                                                   "num_accepted", "block_tables"))
    stack, free, lens = _cpu(s["free_blocks"]).copy(), int(s["num_free"]), lens.copy()
    out = {n: s[n].double() for n in ("key_caches", "value_caches")}
    src, dst = [], []
    for b in range(len(lens)):
        src += [slots[off[b] + a] for a in accepted[b, :count[b]]]
        dst += [slots[off[b] + j] for j in range(count[b])]
        had = _blocks(int(lens[b]), bs)
        lens[b] += count[b] - (off[b + 1] - off[b])
        gone = table[b, _blocks(int(lens[b]), bs):had]
        stack[free:free + len(gone)] = gone
        free += len(gone)
    src, dst = (torch.tensor(np.array(x, np.int64), device=DEVICE) for x in (src, dst))
    for c in out.values():
        for layer in c:
            rows = layer[src // bs, :, src % bs].clone()
            layer[dst // bs, :, dst % bs] = rows
    return out | {"context_lens": lens, "num_free": np.array([free], np.int32), "free_blocks": stack}


def exact(case, seed):
    s = prepare(case, seed)
    return {"masks": _exact_masks, "norm": _exact_norm, "attend": _exact_attend, "accept": _exact_accept,
            "compact": _exact_compact}[case["op"]](s)
