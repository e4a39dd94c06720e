"""Plain float64 forms of the serving-step operators, written from their definitions (CPU, numpy)."""
import numpy as np
import torch

E4M3 = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).double().numpy()


def rotate(x, pos, inv_freq, layout, factor):
    """x [T, h, d] float64 turned by pos [T]; also the bound of what float32 arithmetic may be off by.

    Per element (|x| + |y|) * factor times: 2^-25 half turns of angle = 9.4e-8, sincospi's 2 ulp = 1.2e-7,
    the factor's, the two products' and the sum's roundings = 4 * 6e-8: below 5e-7."""
    x = np.asarray(x, np.float64)
    half = len(inv_freq)
    i = np.arange(half)
    a, b = (i, i + half) if layout == "half" else (2 * i, 2 * i + 1)
    ang = np.asarray(pos, np.float64)[:, None] * np.asarray(inv_freq, np.float64)[None, :]
    c, s = np.cos(ang)[:, None, :] * factor, np.sin(ang)[:, None, :] * factor
    y, slack = x.copy(), np.zeros_like(x)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., a] * s + x[..., b] * c
    slack[..., a] = slack[..., b] = 5e-7 * abs(factor) * (np.abs(x[..., a]) + np.abs(x[..., b]))
    return y, slack


def gather(codes, scales, table, length, head):
    """Rows 0 .. length - 1 of one head as float64 (codes [N, H, bs, d] uint8)."""
    bs = codes.shape[2]
    pos = np.arange(length)
    blk = np.asarray(table)[pos // bs]
    return E4M3[codes[blk, head, pos % bs]] * scales.astype(np.float64)[blk, head][:, None]


def attend(q, k_codes, v_codes, ks, vs, tables, lens, offsets, scale, dtype):
    """(out, bound) of ragged causal attention, float64; rows behind the last request are NaN.

    The bound, with A = sum p |v| of an element and S = the largest sum |q k| of the row's scores: half a step of the
    output (eps / 2 relative; below the smallest normal number steps are that number times eps, f16: 2^-24); P in f16,
    half a step 2^-11 of A; scores from float32 sums of d exact products, each off by 2^-23 of S in the worst order,
    d <= 128, which moves p by twice that; and L / 16 + 16 sums of A in float32.  P of a small exponential, or of a block
    whose V scale is far below the largest, is subnormal in f16: off by half a step 2^-25 of the largest scale W seen by the
    request's rows, times |code|, with the exponentials' sum at least 1: 2^-25 W sum |code|."""
    out = np.full(q.shape, np.nan)
    bound = np.full(q.shape, np.nan)
    hq, hkv = q.shape[1], k_codes.shape[1]
    g = hq // hkv
    eps, tiny = torch.finfo(dtype).eps, torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2
    for b in range(len(lens)):
        lo, hi = int(offsets[b]), int(offsets[b + 1])
        n, L = hi - lo, int(lens[b])
        if n == 0:
            continue
        for h in range(hkv):
            k, v = gather(k_codes, ks, tables[b], L, h), gather(v_codes, vs, tables[b], L, h)
            ids = np.asarray(tables[b])[:(L + k_codes.shape[2] - 1) // k_codes.shape[2]]
            codes = np.abs(gather(v_codes, np.ones_like(vs), tables[b], L, h)).cumsum(0)
            small = 2.0 ** -25 * float(vs[ids, h].max(initial=0)) * codes
            for t in range(n):
                seen = L - n + t + 1
                rows = q[lo + t, h * g:(h + 1) * g]
                if seen <= 0:
                    out[lo + t, h * g:(h + 1) * g] = 0
                    bound[lo + t, h * g:(h + 1) * g] = 0
                    continue
                s = scale * rows @ k[:seen].T
                p = np.exp(s - s.max(1, keepdims=True))
                p /= p.sum(1, keepdims=True)
                o = p @ v[:seen]
                mass = p @ np.abs(v[:seen])
                big = (abs(scale) * np.abs(rows) @ np.abs(k[:seen]).T).max(1, keepdims=True)
                out[lo + t, h * g:(h + 1) * g] = o
                bound[lo + t, h * g:(h + 1) * g] = eps / 2 * np.abs(o) * 1.01 + mass * (
                    2.0 ** -11 + 2 * big * 128 * 2.0 ** -23 + (L / 16 + 16) * 2.0 ** -23) + small[seen - 1] + tiny
    return out, bound


def paged(rng, lens, hkv, d, bs, spare=3, sizes=(0.002, 0.02), nan_tail=True):
    """Random codes, scales and tables for requests of these lengths; NaN codes past every context and in spare blocks."""
    lens = np.asarray(lens, np.int32)
    count = (lens + bs - 1) // bs
    nb = int(count.sum()) + spare
    perm = rng.permutation(nb).astype(np.int32)
    tables = np.full((len(lens), max(1, int(count.max()) + 1)), -1, np.int32)
    kc, vc = (rng.integers(0, 256, (nb, hkv, bs, d), dtype=np.uint8) for _ in range(2))
    kc[(kc & 0x7F) == 0x7F] = 0x3A
    vc[(vc & 0x7F) == 0x7F] = 0x3B
    at = 0
    for b, n in enumerate(count):
        tables[b, :n] = perm[at:at + n]
        at += n
        if nan_tail and lens[b] % bs:
            kc[tables[b, n - 1], :, lens[b] % bs:] = 0x7F
            vc[tables[b, n - 1], :, lens[b] % bs:] = 0xFF
    ks, vs = (np.exp(rng.uniform(np.log(sizes[0]), np.log(sizes[1]), (nb, hkv))).astype(np.float32) for _ in range(2))
    if nan_tail:
        kc[perm[at:]], vc[perm[at:]] = 0x7F, 0x7F
        ks[perm[at:]] = vs[perm[at:]] = np.nan
    return kc, vc, ks, vs, tables, lens
