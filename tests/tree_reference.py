"""Plain float64 forms of the operators of a speculative step with a drafted tree, from their definitions (CPU, numpy)."""
import numpy as np
import torch

import step_reference as step


def trees(rng, sizes, kind="mixed"):
    """(offsets, parents) of trees of these sizes: chains, bushes (all children of node 0), forests, or random ones."""
    parents = []
    for r, n in enumerate(sizes):
        k = ["chain", "random", "bush", "forest", "narrow"][r % 5] if kind == "mixed" else kind
        i = np.arange(n)
        p = {"chain": i - 1, "bush": np.where(i == 0, -1, 0), "random": np.floor(rng.random(n) * i) if n else i,
             "narrow": i - 1 - np.floor(rng.random(n) * np.minimum(i, 4)),
             "forest": np.where(rng.random(n) < 0.3, -1, np.floor(rng.random(n) * i))}[k].astype(np.int32)
        if n:
            p[0] = -1
        parents.append(p)
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    return off, np.concatenate(parents + [np.zeros(0, np.int32)]).astype(np.int32)


def branch(parents, node):
    """A node and its ancestors, the node first."""
    got = []
    while node >= 0:
        got.append(int(node))
        node = parents[node]
    return got


def masks(off, parents, lens, words, rows):
    """(positions [rows], seen [rows, 64 * words] bool); rows behind the last node: 0, nothing."""
    pos, seen = np.zeros(rows, np.int32), np.zeros((rows, 64 * words), bool)
    for b in range(len(off) - 1):
        mine = parents[off[b]:off[b + 1]]
        for i in range(len(mine)):
            path = branch(mine, i)
            pos[off[b] + i] = lens[b] - len(mine) + len(path) - 1
            seen[off[b] + i, path] = True
    return pos, seen


def words_of(seen):
    """[rows, 64 * words] bool as int64 words."""
    bits = seen.reshape(seen.shape[0], -1, 64).astype(np.uint64)
    return (bits << np.arange(64, dtype=np.uint64)).sum(-1, dtype=np.uint64).view(np.int64)


def attend(q, kc, vc, tables, lens, off, seen, scale, dtype):
    """(out, bound) of the nodes' attention in float64; rows of no request are NaN.  kc, vc [N, H, bs, d] float64; positions
    with an id outside the pool are not seen.

    The bound, with A = sum p |v| of an element and S = the largest sum |q k| of the row's scores: half a step of the output
    (eps / 2 relative; below the smallest normal number steps are that number times eps); a weight rounded to dtype,
    half a step eps / 2 of A; scores from float32 sums of d <= 128 exact products, each off by 2^-23 of S in the worst
    order, which moves a weight by twice that; L / 16 + 16 sums of A in float32; in f16, weights below 2^-14 of an
    exponential that is no larger than the row's largest are off by half a step 2^-25 of it: 2^-25 sum |v|."""
    out, bound = np.full(q.shape, np.nan), np.full(q.shape, np.nan)
    hq, hkv, bs = q.shape[1], kc.shape[1], kc.shape[2]
    g, eps = hq // hkv, torch.finfo(dtype).eps
    tiny = torch.finfo(dtype).smallest_normal * eps / 2
    for b in range(len(lens)):
        lo, n, L = int(off[b]), int(off[b + 1] - off[b]), int(lens[b])
        if n == 0:
            continue
        pos = np.arange(L)
        blk = np.asarray(tables)[b][pos // bs]
        there = (blk >= 0) & (blk < kc.shape[0])
        for t in range(n):
            use = there.copy()
            node = pos - (L - n)
            inside = (node >= 0) & (node < seen.shape[1])
            use &= (node < 0) | inside
            use[inside] &= seen[lo + t, node[inside]]
            k, v = kc[blk[use], :, pos[use] % bs], vc[blk[use], :, pos[use] % bs]  # [seen, H, d]
            for h in range(hkv):
                at = (lo + t, slice(h * g, (h + 1) * g))
                if not use.any():
                    out[at], bound[at] = 0, 0
                    continue
                rows = q[at]
                s = scale * rows @ k[:, h].T
                p = np.exp(s - s.max(1, keepdims=True))
                p /= p.sum(1, keepdims=True)
                o, mass = p @ v[:, h], p @ np.abs(v[:, h])
                big = (abs(scale) * np.abs(rows) @ np.abs(k[:, h]).T).max(1, keepdims=True)
                out[at] = o
                bound[at] = eps / 2 * 1.01 * (np.abs(o) + mass) + mass * (2 * big * 128 * 2.0 ** -23 + (L / 16 + 16) * 2.0 ** -23) + tiny
                if dtype == torch.float16:
                    bound[at] += 2.0 ** -25 * np.abs(v[:, h]).sum(0)
    return out, bound


def norm_rotate(x, weight, eps, offset, pos, inv_freq, layout, factor):
    """Norm of each head of x [t, h, d] float64, then the rotation; and what float32 arithmetic may be off by.

    Squares and their sum in any order: (d + 1) 2^-24 of the sum, half of it in the root; division by d, eps, root and quotient 4 half steps,
    products with norm and weight 3 more: (d / 2 + 8) 2^-24 of each element, and of each pair's sum of magnitudes behind the turn."""
    x = np.asarray(x, np.float64)
    d = x.shape[-1]
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * (1.0 if weight is None else np.asarray(weight, np.float64) + offset)
    rel = (d / 2 + 8) * 2.0 ** -24
    if inv_freq is None or len(inv_freq) == 0:
        return y, np.abs(y) * rel
    want, slack = step.rotate(y, pos, inv_freq, layout, factor)
    turned = slack > 0
    return want, 2 * slack + np.where(turned, slack / 5e-7, np.abs(y)) * rel


def accept(off, parents, tokens, choices, depth):
    b = len(off) - 1
    accepted, count, token = np.full((b, depth), -1, np.int32), np.zeros(b, np.int32), np.full(b, -1, np.int64)
    for r in range(b):
        lo, n = off[r], off[r + 1] - off[r]
        node = 0 if n else None
        while node is not None and count[r] < depth:
            accepted[r, count[r]] = node
            count[r] += 1
            token[r] = choices[lo + node]
            node = next((c for c in range(node + 1, n) if parents[lo + c] == node and tokens[lo + c] == token[r]), None)
    return accepted, count, token


def compact(caches, slots, off, accepted, count, tables, lens, stack, free, bs):
    """caches: arrays [.., N, H, bs, d], changed in place.  Returns (lengths, stack, count)."""
    lens, stack = lens.copy(), stack.copy()
    for b in range(len(lens)):
        src = [slots[off[b] + a] for a in accepted[b, :count[b]]]
        for c in caches:
            rows = [c[..., s // bs, :, s % bs, :].copy() for s in src]
            for j, row in enumerate(rows):
                s = slots[off[b] + j]
                c[..., s // bs, :, s % bs, :] = row
        had = (lens[b] + bs - 1) // bs
        lens[b] += count[b] - (off[b + 1] - off[b])
        for j in range((lens[b] + bs - 1) // bs, had):
            stack[free] = tables[b, j]
            free += 1
    return lens, stack, free


def paged(rng, lens, hkv, d, bs, dtype, spare=3, extra=1, fill=float("nan")):
    """Caches [N, H, bs, d] (CPU tensors of dtype) of normal values for requests of these lengths, `fill` past every context
    and in spare blocks; tables [B, widest + extra]."""
    lens = np.asarray(lens, np.int32)
    count = (lens + bs - 1) // bs
    nb = int(count.sum()) + spare
    perm = rng.permutation(nb).astype(np.int32)
    tables = np.full((len(lens), max(1, int(count.max(initial=0)) + extra)), -1, np.int32)
    kc, vc = (torch.from_numpy(rng.standard_normal((nb, hkv, bs, d)).astype(np.float32)).to(dtype) for _ in range(2))
    at = 0
    for b, n in enumerate(count):
        tables[b, :n] = perm[at:at + n]
        at += n
        if lens[b] % bs:
            for c in (kc, vc):
                c[int(tables[b, n - 1]), :, int(lens[b]) % bs:] = fill
    for c in (kc, vc):
        c[torch.from_numpy(perm[at:].astype(np.int64))] = fill
    return kc, vc, tables, lens
