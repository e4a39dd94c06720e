"""Measured calls of the operators that a serving step over an 8-bit paged cache is made of.

* ``advance_tables``  - block tables, positions and slot maps of a step, from request lengths, on the GPU;
* ``rope_write_kv``   - rotary positions of queries and keys, with the paged write of keys and values;
* ``rope_append_fp8`` - the same for an FP8 (E4M3) cache, whose block scales follow the data;
* ``attend_fp8``      - causal attention of ragged runs of new tokens over that cache.

``own`` chooses between the plain form (elementary torch operations in 32 bits) and the framework's calls.
Lengths and layouts are a function of the case; the values, and which block holds what, of the seed.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
DEVICE = "cuda"


# ---- cases ---------------------------------------------------------------------------------

def listed():
    qwen = {"hq": 28, "hkv": 4, "d": 128, "bs": 16}
    return [
        # one token for each of 64 running requests: launch latency
        {"name": "tables_step", "op": "tables", "b": 64, "new_lo": 1, "new_hi": 1, "ctx_lo": 512, "ctx_hi": 4096,
         "released": 0, "bs": 16, "lens": 1},
        # a large mixed step: prompts of up to 512 tokens, a few requests finished and given back
        {"name": "tables_prompts", "op": "tables", "b": 256, "new_lo": 0, "new_hi": 512, "ctx_lo": 0, "ctx_hi": 4096,
         "released": 16, "bs": 16, "lens": 2},
        # decode step of 64 requests, 16-bit cache
        {"name": "rope_write_step", "op": "rope", "t": 64, **qwen, "rot": 128, "dtype": "bf16", "layout": "half",
         "max_pos": 4096, "scaling": "none", "lens": 3},
        # prompt chunk of 8192 tokens, 16-bit cache
        {"name": "rope_write_chunk", "op": "rope", "t": 8192, **qwen, "rot": 128, "dtype": "bf16", "layout": "half",
         "max_pos": 131072, "scaling": "ramp", "lens": 4},
        # odd token count, interleaved pairs over part of a small head, 32-bit cache, far positions
        {"name": "rope_write_part_f32", "op": "rope", "t": 1001, "hq": 4, "hkv": 2, "d": 64, "bs": 16, "rot": 32,
         "dtype": "f32", "layout": "interleaved", "max_pos": 1000000, "scaling": "linear", "lens": 5},
        # decode step of 64 requests, FP8 cache
        {"name": "append_step", "op": "append", "b": 64, "new_lo": 1, "new_hi": 1, "ctx_lo": 512, "ctx_hi": 4096, **qwen,
         "rot": 128, "dtype": "bf16", "layout": "half", "records": False, "lens": 6},
        # prompt chunks of eight requests, FP8 cache
        {"name": "append_chunk", "op": "append", "b": 8, "new_lo": 900, "new_hi": 1200, "ctx_lo": 0, "ctx_hi": 4096,
         **qwen, "rot": 128, "dtype": "bf16", "layout": "half", "records": False, "lens": 7},
        # ragged short prompts, as many key heads as query heads, 32-token blocks, K and V in one record
        {"name": "append_mha_records", "op": "append", "b": 37, "new_lo": 0, "new_hi": 130, "ctx_lo": 0, "ctx_hi": 700,
         "hq": 32, "hkv": 32, "d": 128, "bs": 32, "rot": 64, "dtype": "f16", "layout": "interleaved", "records": True,
         "lens": 8},
        # speculative verification: four tokens for each of 64 requests
        {"name": "attend_verify", "op": "attend", "b": 64, "new_lo": 4, "new_hi": 4, "ctx_lo": 512, "ctx_hi": 4096,
         **qwen, "dtype": "bf16", "records": False, "lens": 9},
        # prompt chunks on top of cached tokens: bound by the products
        {"name": "attend_chunk", "op": "attend", "b": 4, "new_lo": 1500, "new_hi": 2048, "ctx_lo": 2048, "ctx_hi": 6144,
         **qwen, "dtype": "bf16", "records": False, "lens": 10},
        # few rows on long contexts: the contexts have to be split
        {"name": "attend_long", "op": "attend", "b": 8, "new_lo": 1, "new_hi": 8, "ctx_lo": 32768, "ctx_hi": 131072,
         "hq": 32, "hkv": 8, "d": 128, "bs": 16, "dtype": "bf16", "records": False, "lens": 11},
        # ragged batch of short requests, head size 64, 32-token blocks, requests without a token among them
        {"name": "attend_mixed_d64", "op": "attend", "b": 61, "new_lo": 0, "new_hi": 200, "ctx_lo": 0, "ctx_hi": 900,
         "hq": 16, "hkv": 4, "d": 64, "bs": 32, "dtype": "f16", "records": True, "lens": 12},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["tables", "rope", "append", "attend"])
    bs = rng.choice([16, 32])
    case = {"op": op, "bs": bs, "lens": rng.randrange(1 << 30)}
    if op == "tables":
        lo, hi = sorted((_log_int(rng, 1, 512), _log_int(rng, 1, 512)))
        case |= {"b": _log_int(rng, 1, 256), "new_lo": lo - 1, "new_hi": hi, "ctx_lo": 0,
                 "ctx_hi": _log_int(rng, 16, 4096)}
        return case | {"released": rng.randrange(0, case["b"] // 8 + 1)}
    hkv = rng.choice([1, 2, 4, 8])
    case |= {"hkv": hkv, "hq": hkv * rng.choice([1, 2, 4, 7, 8]), "d": rng.choice([64, 128])}
    if op == "rope":
        return case | {"t": _log_int(rng, 1, 4096), "rot": rng.choice([case["d"] // 4, case["d"] // 2, case["d"]]),
                       "dtype": rng.choice(["f32", "f16", "bf16"]), "layout": rng.choice(["half", "interleaved"]),
                       "max_pos": _log_int(rng, 64, 1000000), "scaling": rng.choice(["none", "linear", "ramp"])}
    if op == "append":
        lo, hi = sorted((_log_int(rng, 1, 256), _log_int(rng, 1, 256)))
        return case | {"b": _log_int(rng, 1, 32), "new_lo": lo - 1, "new_hi": hi, "ctx_lo": 0,
                       "ctx_hi": _log_int(rng, 16, 2048), "rot": rng.choice([case["d"] // 2, case["d"]]),
                       "dtype": rng.choice(["f16", "bf16"]), "layout": rng.choice(["half", "interleaved"]),
                       "records": rng.random() < 0.5}
    # bounded so that no drawn case exceeds the prompt-chunk case
    lo, hi = sorted((_log_int(rng, 1, 512), _log_int(rng, 1, 512)))
    return case | {"b": _log_int(rng, 1, 8), "new_lo": lo - 1, "new_hi": hi, "ctx_lo": 0,
                   "ctx_hi": _log_int(rng, 16, 4096), "dtype": rng.choice(["f16", "bf16"]),
                   "records": rng.random() < 0.5}


def _lengths(case):
    """(cached tokens, new tokens) of each request, int64; a finished request has -1 new tokens."""
    rng = np.random.default_rng(case["lens"])
    b = case["b"]
    old = rng.integers(case["ctx_lo"], case["ctx_hi"] + 1, b)
    new = rng.integers(case["new_lo"], case["new_hi"] + 1, b)
    if new.max() <= 0:
        new[0] = 1
    if case.get("released"):
        new[rng.choice(b, case["released"], replace=False)] = -1
    return old, new


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

def _table(rng, counts, extra):
    """(blocks in the pool, a random block of the pool for each logical block)."""
    pool = int(counts.sum()) + extra
    perm = rng.permutation(pool).astype(np.int32)
    width = max(1, int(counts.max()))
    table = np.full((len(counts), width), -1, np.int32)
    at = 0
    for b, n in enumerate(counts):
        table[b, :n] = perm[at:at + n]
        at += n
    return pool, table, perm[at:]


def _up(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEVICE)


def _normal(gen, shape, dtype=torch.float32):
    return torch.randn(shape, generator=gen, device=DEVICE).to(dtype)


def _fp8_pool(gen, pool, case):
    """Codes and scales of a pool whose blocks hold normal values of different sizes, each block filling its range."""
    hkv, bs, d = case["hkv"], case["bs"], case["d"]
    codes, scales = [], []
    for _ in range(2):
        c = torch.empty(pool, hkv, bs, d, dtype=torch.float8_e4m3fn, device=DEVICE)
        s = torch.empty(pool, hkv, device=DEVICE)
        for at in range(0, pool, 8192):
            x = _normal(gen, (min(8192, pool - at), hkv, bs, d))
            x *= torch.rand(x.shape[:2], generator=gen, device=DEVICE)[:, :, None, None] + 0.5
            s[at:at + 8192] = x.abs().amax((2, 3)) / 448.0
            c[at:at + 8192] = (x / s[at:at + 8192, :, None, None]).to(torch.float8_e4m3fn)
        codes.append(c)
        scales.append(s)
    if case["records"]:
        both = torch.stack([x.view(torch.uint8) for x in codes], 2).contiguous().view(torch.float8_e4m3fn)
        return both, None, scales[0], scales[1]
    return codes[0], codes[1], scales[0], scales[1]


def prepare(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device=DEVICE).manual_seed(int(seed))
    s = {"case": case, "op": case["op"]}
    if case["op"] == "tables":
        old, new = _lengths(case)
        have, want = _blocks(old, case["bs"]), _blocks(old + np.maximum(new, 0), case["bs"])
        pool, table, free = _table(rng, have, int((want - have).sum()) + 64)
        width = max(1, int(want.max()))
        table = np.pad(table, ((0, 0), (0, max(0, width - table.shape[1]))), constant_values=-1)
        stack = np.zeros(pool, np.int32)
        stack[:len(free)] = free
        tokens = int(np.maximum(new, 0).sum())
        s |= {"block_tables": _up(table), "context_lens": _up(old.astype(np.int32)),
              "new_lens": _up(new.astype(np.int32)), "free_blocks": _up(stack),
              "num_free": torch.tensor([len(free)], dtype=torch.int32, device=DEVICE), "tokens": tokens}
        i32 = {"dtype": torch.int32, "device": DEVICE}  # the step's buffers, kept from step to step
        s["out"] = (torch.empty(len(old), **i32), torch.empty(1, **i32), torch.empty(len(old) + 1, **i32),
                    torch.empty(tokens, **i32), torch.empty(tokens, dtype=torch.int64, device=DEVICE))
        return s
    hq, hkv, d, bs, dt = case["hq"], case["hkv"], case["d"], case["bs"], DTYPES[case["dtype"]]
    if case["op"] == "rope":
        t = case["t"]
        pool = _blocks(t, bs) + 8
        slots = rng.permutation(pool * bs)[:t].astype(np.int64)
        slots[rng.random(t) < 0.02] = -1  # padding rows
        s |= {"positions": _up(rng.integers(0, case["max_pos"], t).astype(np.int32)), "slots": _up(slots),
              "key_cache": torch.zeros(pool, hkv, bs, d, dtype=dt, device=DEVICE),
              "value_cache": torch.zeros(pool, hkv, bs, d, dtype=dt, device=DEVICE)}
    else:
        old, new = _lengths(case)
        lens = old + new
        counts = _blocks(lens, bs)
        pool, table, _ = _table(rng, counts, 8)
        t = int(new.sum())
        s["key_cache"], s["value_cache"], s["k_scale"], s["v_scale"] = _fp8_pool(gen, pool, case)
        s |= {"block_tables": _up(table), "context_lens": _up(lens.astype(np.int32)),
              "q_offsets": _up(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)), "max_new": int(new.max())}
        if case["op"] == "attend":
            s["query"] = _normal(gen, (t, hq, d), dt)
            s["out"] = torch.empty(t, hq, d, dtype=dt, device=DEVICE)
            s["scale"] = 1.0 / math.sqrt(d)
            return s
    # queries, keys and values as the projection leaves them: one row per token
    qkv = _normal(gen, (t, (hq + 2 * hkv) * d), dt)
    q, k, v = qkv.split([hq * d, hkv * d, hkv * d], 1)
    scaling = case.get("scaling", "none")
    s |= {"query": q.unflatten(1, (hq, d)), "key": k.unflatten(1, (hkv, d)), "value": v.unflatten(1, (hkv, d)),
          "query_out": torch.empty(t, hq, d, dtype=dt, device=DEVICE),
          "inv_freq": _up(_inv_freq(case["rot"], scaling)), "factor": _rope_factor(scaling)}
    return s


# ---- the plain form -------------------------------------------------------------------------

def _token_rows(s, t):
    """(request, position) of each new token."""
    at = torch.arange(t, device=DEVICE)
    off = s["q_offsets"].long()
    seq = torch.searchsorted(off, at, right=True) - 1
    n = off[1:] - off[:-1]
    return seq, s["context_lens"].long()[seq] - n[seq] + at - off[seq]


def _rotate(x, pos, s):
    """Rotary positions of x [t, h, d], in 32 bits (angles in 64)."""
    inv, rot = s["inv_freq"], s["case"]["rot"]
    ang = pos.double()[:, None] * inv[None, :]
    c = (ang.cos() * s["factor"]).float()[:, None, :]
    n = (ang.sin() * s["factor"]).float()[:, None, :]
    x = x.float()
    r = x[..., :rot]
    if s["case"]["layout"] == "half":
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        r = torch.cat([a * c - b * n, a * n + b * c], -1)
    else:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * c - b * n, a * n + b * c], -1).flatten(-2)
    return torch.cat([r, x[..., rot:]], -1)


def _plain_tables(s):
    bs = s["case"]["bs"]
    old, new, table, stack = s["context_lens"].long(), s["new_lens"].long(), s["block_tables"], s["free_blocks"]
    b, m = table.shape
    out = new < 0
    have = (old + bs - 1) // bs
    back = torch.where(out, have, 0)
    j = torch.arange(m, device=DEVICE)[None, :]
    give = j < back[:, None]
    at = (s["num_free"].long() + back.cumsum(0) - back)[:, None] + j
    stack[at[give]] = table[give]
    top = s["num_free"].long() + back.sum()
    n = new.clamp(min=0)
    lens = torch.where(out, 0, old + n)
    need = torch.where(out, 0, (old + n + bs - 1) // bs - have)
    rank = (need.cumsum(0) - need)[:, None] + j - have[:, None]
    take = (j >= have[:, None]) & (j < (have + need)[:, None])
    table[take] = stack[(top - 1 - rank)[take]]
    off = torch.cat([n.new_zeros(1), n.cumsum(0)])
    t = torch.arange(s["tokens"], device=DEVICE)
    seq = torch.searchsorted(off, t, right=True) - 1
    pos = old[seq] + t - off[seq]
    slots = table[seq, pos // bs].long() * bs + pos % bs
    return {"block_tables": table, "context_lens": lens.int(), "num_free": (top - need.sum()).int(),
            "free_blocks": stack, "q_offsets": off.int(), "positions": pos.int(), "slots": slots}


def _plain_rope(s):
    bs = s["case"]["bs"]
    q, k = (_rotate(s[n], s["positions"], s).to(s[n].dtype) for n in ("query", "key"))
    ok = s["slots"] >= 0
    blk, off = s["slots"][ok] // bs, s["slots"][ok] % bs
    s["key_cache"][blk, :, off] = k[ok]
    s["value_cache"][blk, :, off] = s["value"][ok]
    return {"query": q, "key_cache": s["key_cache"], "value_cache": s["value_cache"]}


def _caches(s):
    """Views of the K and V codes, [blocks, heads, tokens, d] bytes."""
    k = s["key_cache"].view(torch.uint8)
    return (k[:, :, 0], k[:, :, 1]) if s["value_cache"] is None else (k, s["value_cache"].view(torch.uint8))


def _to_codes(x):
    return x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)


def _plain_append(s):
    bs = s["case"]["bs"]
    seq, pos = _token_rows(s, s["query"].shape[0])
    blk, off = s["block_tables"].long()[seq, pos // bs], pos % bs
    q = _rotate(s["query"], pos, s).to(s["query"].dtype)
    for x, cache, scale in zip((_rotate(s["key"], pos, s), s["value"].float()), _caches(s), (s["k_scale"], s["v_scale"])):
        n, hkv = scale.shape
        most = torch.zeros_like(scale).scatter_reduce_(0, blk[:, None].expand(-1, hkv), x.abs().amax(-1), "amax")
        first = torch.full((n,), bs, device=DEVICE).scatter_reduce_(0, blk, off, "amin")
        touched, fresh = (first < bs)[:, None], (first == 0)[:, None]
        held = torch.where(fresh, 0.0, scale)
        grown = torch.where(touched, torch.maximum(torch.maximum(held, most / 448.0), torch.tensor(2.0 ** -100)), scale)
        # the codes that a block holds already, in its new scale
        redo = (touched & ~fresh & (grown > scale))[:, :, None] & (torch.arange(bs, device=DEVICE) < first[:, None])[:, None]
        was = cache[redo].view(torch.float8_e4m3fn).float()
        cache[redo] = _to_codes(was * scale[:, :, None].expand(n, hkv, bs)[redo][:, None]
                                / grown[:, :, None].expand(n, hkv, bs)[redo][:, None])
        cache[blk, :, off] = _to_codes(x / grown[blk][:, :, None])
        scale.copy_(grown)
    return _append_outputs(s, q)


def _append_outputs(s, q):
    return {"query": q, "key_cache": s["key_cache"], "value_cache": s["value_cache"], "k_scale": s["k_scale"],
            "v_scale": s["v_scale"]}


def _plain_attend(s):
    case = s["case"]
    hq, hkv, d, bs = case["hq"], case["hkv"], case["d"], case["bs"]
    g, n = hq // hkv, s["max_new"]
    table = s["block_tables"].long().clamp(min=0)
    b, m = table.shape
    k, v = (c[table].view(torch.float8_e4m3fn).float() * sc[table][..., None, None]
            for c, sc in zip(_caches(s), (s["k_scale"], s["v_scale"])))
    k, v = (x.transpose(1, 2).reshape(b, hkv, m * bs, d) for x in (k, v))
    off, lens = s["q_offsets"].long(), s["context_lens"].long()
    new = off[1:] - off[:-1]
    i = torch.arange(n, device=DEVICE)
    rows = (off[:-1, None] + i).clamp(max=s["query"].shape[0] - 1)
    q = s["query"][rows].float().reshape(b, n, hkv, g, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, g * n, d)
    x = (q @ k.transpose(2, 3)).view(b, hkv, g, n, m * bs).mul_(s["scale"])
    last = (lens - new)[:, None] + i
    at = torch.arange(m * bs, device=DEVICE)
    x.masked_fill_((at > last[:, :, None])[:, None, None], -math.inf)
    x.sub_(x.amax(-1, keepdim=True)).exp_()
    sums = x.sum(-1, keepdim=True)
    v = v.masked_fill((at >= lens[:, None])[:, None, :, None], 0.0)
    o = (x.view(b, hkv, g * n, m * bs) @ v).view(b, hkv, g, n, d) / sums
    o = o.permute(0, 3, 1, 2, 4).reshape(b, n, hq, d)
    return o[i < new[:, None]].to(s["query"].dtype)


# ---- the framework's calls -------------------------------------------------------------------

def _own_run(s):
    import paged_kv_cache_129_gb300 as pa

    op = s["op"]
    if op == "tables":
        got = pa.advance_tables(s["block_tables"], s["context_lens"], s["new_lens"], s["free_blocks"], s["num_free"],
                                s["case"]["bs"], s["tokens"], out=s["out"])
        return {"block_tables": s["block_tables"], "context_lens": got.context_lens, "num_free": got.num_free,
                "free_blocks": s["free_blocks"], "q_offsets": got.q_offsets, "positions": got.positions,
                "slots": got.slot_mapping}
    if op == "rope":
        q = pa.rope_write_kv(s["query"], s["key"], s["value"], s["key_cache"], s["value_cache"], s["inv_freq"],
                             s["positions"], s["slots"], layout=s["case"]["layout"], factor=s["factor"],
                             query_out=s["query_out"])
        return {"query": q, "key_cache": s["key_cache"], "value_cache": s["value_cache"]}
    if op == "append":
        q = pa.rope_append_fp8(s["query"], s["key"], s["value"], s["key_cache"], s["value_cache"], s["k_scale"],
                               s["v_scale"], s["inv_freq"], s["block_tables"], s["context_lens"], s["q_offsets"],
                               layout=s["case"]["layout"], factor=s["factor"], query_out=s["query_out"])
        return _append_outputs(s, q)
    if "workspace" not in s:  # kept from call to call
        s["workspace"] = torch.empty(pa.attend_fp8_workspace_size(
            s["query"].shape[0], s["block_tables"].shape[0], s["case"]["hq"], s["case"]["hkv"], s["case"]["d"],
            s["case"]["bs"], s["block_tables"].shape[1], s["query"].dtype), dtype=torch.uint8, device=DEVICE)
    return pa.attend_fp8(s["query"], s["key_cache"], s["value_cache"], s["k_scale"], s["v_scale"], s["block_tables"],
                         s["context_lens"], s["q_offsets"], scale=s["scale"], out=s["out"], workspace=s["workspace"])


def run(state):
    if own:
        return _own_run(state)
    return {"tables": _plain_tables, "rope": _plain_rope, "append": _plain_append,
            "attend": _plain_attend}[state["op"]](state)


# ---- what a pass cannot do without ---------------------------------------------------------------

def work(case):
    bs, op = case["bs"], case["op"]
    if op == "rope":
        e, t = DTYPES[case["dtype"]].itemsize, case["t"]
        rows = case["hq"] + 2 * case["hkv"]
        return {"bytes": 2 * t * rows * case["d"] * e + 12 * t + 4 * case["rot"],
                "flops": 3 * t * (case["hq"] + case["hkv"]) * case["rot"]}
    old, new = _lengths(case)
    n = np.maximum(new, 0)
    t, b = int(n.sum()), len(old)
    if op == "tables":
        take = _blocks(old + n, bs) - _blocks(old, bs)
        give = np.where(new < 0, _blocks(old, bs), 0)
        return {"bytes": 8 * int(np.where(new < 0, 0, take).sum() + give.sum()) + 12 * t + 20 * b, "flops": 4 * t}
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if op == "append":
        pages = int(np.where(n > 0, _blocks(old + n, bs) - old // bs, 0).sum())
        return {"bytes": t * d * (2 * (2 * hq + 2 * hkv) + 2 * hkv) + 16 * pages * hkv + 4 * pages + 8 * b,
                "flops": t * d * (3 * hq + 7 * hkv)}
    used = np.where(n > 0, old + n, 0)
    pairs = int((n * old + n * (n + 1) // 2).sum())  # (query, key) pairs of a head that the mask leaves
    return {"bytes": int(used.sum()) * 2 * hkv * d + 12 * int(_blocks(used, bs).sum()) * hkv + 4 * t * hq * d + 8 * b,
            "flops": 4 * pairs * hq * d}


# ---- the definitions in 64 bits -------------------------------------------------------------------

def _cpu(t):
    return t.cpu().numpy()


def _exact_tables(s):
    bs = s["case"]["bs"]
    table, lens, new = _cpu(s["block_tables"]).copy(), _cpu(s["context_lens"]).copy(), _cpu(s["new_lens"])
    stack, free = _cpu(s["free_blocks"]).copy(), int(s["num_free"])
    for b in np.flatnonzero(new < 0):
        k = _blocks(int(lens[b]), bs)
        stack[free:free + k] = table[b, :k]
        free += k
        lens[b] = 0
    offsets, pos, slots = [0], [], []
    for b in range(len(lens)):
        for p in range(int(lens[b]), int(lens[b]) + max(0, int(new[b]))):
            if p % bs == 0:
                free -= 1
                table[b, p // bs] = stack[free]
            pos.append(p)
            slots.append(int(table[b, p // bs]) * bs + p % bs)
        lens[b] += max(0, new[b])
        offsets.append(len(pos))
    i32 = np.int32
    return {"block_tables": table, "context_lens": lens, "num_free": np.array([free], i32), "free_blocks": stack,
            "q_offsets": np.array(offsets, i32), "positions": np.array(pos, i32), "slots": np.array(slots, np.int64)}


def _exact_rotation(x, pos, case, factor):
    """Each pair (a, b) of a head as the complex number a + ib, turned by the angle of its position."""
    x = x.double()
    rot, half = case["rot"], case["rot"] // 2
    i = torch.arange(half, device=x.device)
    first = i if case["layout"] == "half" else 2 * i
    second = i + half if case["layout"] == "half" else 2 * i + 1
    freq = torch.from_numpy(_inv_freq(rot, case.get("scaling", "none"))).to(x.device)
    turn = torch.polar(torch.tensor(factor, dtype=torch.float64, device=x.device), pos.double()[:, None] * freq)
    z = torch.complex(x[..., first], x[..., second]) * turn[:, None, :]
    y = x.clone()
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_rope(s):
    case = s["case"]
    bs = case["bs"]
    q, k = (_exact_rotation(s[n], s["positions"], case, s["factor"]) for n in ("query", "key"))
    kc, vc = s["key_cache"].double(), s["value_cache"].double()
    flat_k, flat_v = kc.transpose(1, 2).reshape(-1, case["hkv"], case["d"]), vc.transpose(1, 2).reshape(-1, case["hkv"], case["d"])
    use = torch.nonzero(s["slots"] >= 0)[:, 0]
    flat_k[s["slots"][use]] = k[use]
    flat_v[s["slots"][use]] = s["value"][use].double()
    kc, vc = (f.view(-1, bs, case["hkv"], case["d"]).transpose(1, 2) for f in (flat_k, flat_v))
    return {"query": q, "key_cache": kc.contiguous(), "value_cache": vc.contiguous()}


def _nearest_code(x):
    """The E4M3 value next to x: 3 bits after the leading one down to 2^-6, steps of 2^-9 below; ties to even."""
    x = x.clamp(-448.0, 448.0)
    _, e = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), torch.clamp(e - 4, min=-9))
    return torch.round(x / step) * step


def _exact_append(s):
    case = s["case"]
    bs = case["bs"]
    old, new = _lengths(case)
    t = int(new.sum())
    pos = torch.from_numpy(np.concatenate([np.arange(a, a + n) for a, n in zip(old, new)])).to(DEVICE)
    out = {"query": _exact_rotation(s["query"], pos, case, s["factor"])}
    both = s["value_cache"] is None
    pool = s["key_cache"].to(torch.float64)
    pools = [pool[:, :, 0], pool[:, :, 1]] if both else [pool, s["value_cache"].to(torch.float64)]
    table = _cpu(s["block_tables"])
    for x, codes, name in zip((_exact_rotation(s["key"], pos, case, s["factor"]), s["value"].double()), pools,
                              ("k_scale", "v_scale")):
        scale = s[name].double()
        at = 0
        for b in range(len(old)):
            p, end = int(old[b]), int(old[b] + new[b])
            while p < end:
                n = min(end - p, bs - p % bs)
                blk, o = int(table[b, p // bs]), p % bs
                rows = x[at:at + n].transpose(0, 1)
                want = torch.clamp(rows.abs().amax((1, 2)) / 448.0, min=2.0 ** -100)
                if o:
                    want = torch.maximum(want, scale[blk])
                    held = codes[blk, :, :o]
                    grew = (want > scale[blk])[:, None, None]
                    codes[blk, :, :o] = torch.where(grew, _nearest_code(held * (scale[blk] / want)[:, None, None]), held)
                scale[blk] = want
                codes[blk, :, o:o + n] = _nearest_code(rows / want[:, None, None])
                p, at = p + n, at + n
        out[name] = scale
    assert at == t
    out["key_cache"] = torch.stack(pools, 2) if both else pools[0]
    out["value_cache"] = None if both else pools[1]
    return out


def _exact_attend(s):
    case = s["case"]
    hkv, d, bs, g = case["hkv"], case["d"], case["bs"], case["hq"] // case["hkv"]
    old, new = _lengths(case)
    if float((new * (old + new)).sum()) * case["hq"] * d > 1e12:
        return None
    both = s["value_cache"] is None
    table, out, at = s["block_tables"].long(), [], 0
    for b in range(len(old)):
        n, length = int(new[b]), int(old[b] + new[b])
        if n == 0:
            continue
        ids = table[b, :_blocks(length, bs)]
        for h in range(hkv):
            if both:
                rec = s["key_cache"].view(torch.uint8)[ids, h].view(torch.float8_e4m3fn).double()
                k, v = rec[:, 0], rec[:, 1]
            else:
                k, v = (s[c].view(torch.uint8)[ids, h].view(torch.float8_e4m3fn).double() for c in ("key_cache", "value_cache"))
            k = (k * s["k_scale"][ids, h].double()[:, None, None]).reshape(-1, d)[:length]
            v = (v * s["v_scale"][ids, h].double()[:, None, None]).reshape(-1, d)[:length]
            q = s["query"][at:at + n, h * g:(h + 1) * g].double()
            x = torch.einsum("tgd,pd->tgp", q, k) * s["scale"]
            seen = torch.arange(length, device=DEVICE)[None, :] <= (length - n + torch.arange(n, device=DEVICE))[:, None]
            p = torch.softmax(x.masked_fill(~seen[:, None, :], -math.inf), -1)
            out.append((at, h, torch.einsum("tgp,pd->tgd", p, v)))
        at += n
    o = torch.empty(at, case["hq"], d, dtype=torch.float64, device=DEVICE)
    for a, h, x in out:
        o[a:a + x.shape[0], h * g:(h + 1) * g] = x
    return o


def exact(case, seed):
    s = prepare(case, seed)
    return {"tables": _exact_tables, "rope": _exact_rope, "append": _exact_append, "attend": _exact_attend}[case["op"]](s)
