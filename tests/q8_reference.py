"""Plain 64-bit reference of the 8-bit paged cache's operators (CPU), and the
tolerances their kernels are held to. Shares no code with the library."""
from __future__ import annotations

import math

import torch

E4M3_MAX = 448.0
# every finite e4m3 magnitude, ascending: the code is the index
E4M3 = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()


def e4m3_round(x: torch.Tensor) -> torch.Tensor:
    """Nearest e4m3 value of a float64 tensor, ties to the even code, saturating;
    NaN stays NaN."""
    a = x.abs().clamp(max=E4M3_MAX)
    hi = torch.searchsorted(E4M3, a.nan_to_num().contiguous()).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    dl, dh = a - E4M3[lo], E4M3[hi] - a
    pick = torch.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return torch.where(x.isnan(), x, torch.copysign(E4M3[pick], x))


def needed_scale(amax: float) -> float:
    if amax == 0:
        return 2.0 ** -60
    e = max(-60, math.ceil(math.log2(amax / E4M3_MAX)) - 1)
    while E4M3_MAX * 2.0 ** e < amax:
        e += 1
    return 2.0 ** e


def append(k, v, ks, vs, table, bs, k_new, v_new, start, count=None):
    """New (k, v, ks, vs): pools as float64 code values, everything on the CPU."""
    B, T, H, hd = k_new.shape
    out = [x.double().clone() for x in (k, v, ks, vs)]
    for pool, scale, new in ((out[0], out[2], k_new.double()), (out[1], out[3], v_new.double())):
        for b in range(B):
            n = T if count is None else max(0, min(T, int(count[b])))
            p0 = int(start[b])
            for j in sorted({(p0 + t) // bs for t in range(n)}):
                if j >= table.shape[1]:
                    continue
                page = int(table[b, j])
                lo, hi = max(p0, j * bs), min(p0 + n, (j + 1) * bs)
                held = lo - j * bs
                for h in range(H):
                    x = new[b, lo - p0:hi - p0, h]
                    fin = x[x.isfinite()].abs()
                    s = needed_scale(float(fin.max()) if fin.numel() else 0.0)
                    if held:
                        s = max(s, float(scale[page, h]))
                        pool[page, h, :held] = e4m3_round(pool[page, h, :held] * (float(scale[page, h]) / s))
                    pool[page, h, held:held + hi - lo] = e4m3_round((x / s).clamp(-E4M3_MAX, E4M3_MAX))
                    scale[page, h] = s
    return out


def attend(q, k, v, ks, vs, table, bs, ids, ctx_len, q_start, scale=0.0, cap=0.0, slopes=None,
           first=None, last=None):
    """(out, lse, mass, sizes): fp64 results, and for the tolerances, per row and
    head, the largest sum of |scale * q_d * k_d| and the largest |v|."""
    B, S, Hq, hd = q.shape
    H, topk = k.shape[1], ids.shape[2]
    G = Hq // H
    scale = scale if scale > 0 else 1.0 / math.sqrt(hd)
    out = torch.zeros(B, S, Hq, hd, dtype=torch.float64)
    lse = torch.full((B, S, Hq), -math.inf, dtype=torch.float64)
    mass = torch.zeros(B, S, H, topk, dtype=torch.float64)
    reach = torch.zeros(B, S, Hq, dtype=torch.float64)
    vmax = torch.zeros(B, S, Hq, dtype=torch.float64)
    for b in range(B):
        for s in range(S):
            p = int(q_start[b]) + s
            hi = min(p if last is None else int(last[b, s]), int(ctx_len[b]) - 1)
            lo = max(0, 0 if first is None else int(first[b, s]))
            tok, slot = [], []
            for i, j in enumerate(ids[b, s].tolist()):
                if j >= 0:
                    t0 = max(j * bs, lo)
                    t = torch.arange(t0, max(t0, min((j + 1) * bs, hi + 1)))
                    tok.append(t)
                    slot.append(torch.full_like(t, i))
            tok = torch.cat(tok) if tok else torch.zeros(0, dtype=torch.long)
            if not tok.numel():
                continue
            slot = torch.cat(slot)
            page, off = table[b, tok // bs].long(), tok % bs
            for h in range(Hq):
                g = h // G
                K = k[page, g, off].double() * ks[page, g].double()[:, None]
                V = v[page, g, off].double() * vs[page, g].double()[:, None]
                qd = q[b, s, h].double()
                z = scale * (K @ qd)
                reach[b, s, h] = scale * (K.abs() @ qd.abs()).max()
                vmax[b, s, h] = V.abs().max()
                if cap > 0:
                    z = cap * torch.tanh(z / cap)
                if slopes is not None:
                    z = z - float(slopes[h]) * (tok - p).abs().double()
                L = torch.logsumexp(z, 0)
                w = torch.exp(z - L)
                out[b, s, h] = w @ V
                lse[b, s, h] = L / math.log(2.0)
                mass[b, s, g].index_add_(0, slot, w)
    return out, lse, mass, (reach, vmax)


def out_tolerance(ref, sizes, dtype, hd, p_bits=24):
    """A weight is off by twice the logit's error (a dot product of hd terms: at
    most (hd + 16) * 2^-24 of the sum of its magnitudes, the cap, bias and
    exponential within the 16) and by the rounding of p to p_bits bits; the
    output is off by that times the largest |v|, and by its own rounding."""
    reach, vmax = sizes
    logit = (hd + 16) * 2.0 ** -24 * (reach + 1.0)
    rel = 2 * logit + 2.0 ** -p_bits + 2.0 ** -20
    own = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    return (rel * vmax)[..., None] + own * ref.abs() + 1e-30


def weight_floor(q, k, v, ks, vs, table, bs, ids, ctx_len, q_start):
    """Per row, head and channel: the row's largest weight * v scale, times the sum
    of the attended codes' magnitudes. What weights that are off by no less than a
    fraction of the largest one can add up to, without that fraction."""
    B, S, Hq, hd = q.shape
    G = Hq // k.shape[1]
    out = torch.zeros(B, S, Hq, hd, dtype=torch.float64)
    for b in range(B):
        for s in range(S):
            hi = min(int(q_start[b]) + s, int(ctx_len[b]) - 1)
            tok = torch.cat([torch.arange(j * bs, max(j * bs, min((j + 1) * bs, hi + 1))) for j in ids[b, s].tolist() if j >= 0])
            page, off = table[b, tok // bs].long(), tok % bs
            for h in range(Hq):
                g = h // G
                z = (k[page, g, off].double() * ks[page, g].double()[:, None]) @ q[b, s, h].double() / math.sqrt(hd)
                out[b, s, h] = (torch.softmax(z, 0) * vs[page, g].double()).max() * v[page, g, off].double().abs().sum(0)
    return out


def share_tolerance(ref, share, floor, sizes, dtype, hd, p_bits):
    """Like out_tolerance, but relative: ``share`` is attend's output over |v|, the
    sum of weight * |v| of each channel, so that no token's error is measured by
    another token's larger value. A weight (times its v scale) keeps p_bits bits,
    half a step of 2^-p_bits of it, or is off by 2^-25 of the row's largest: what a
    channel sums is off by that much of the sum of its magnitudes, or of
    ``floor`` (weight_floor's)."""
    logit = (hd + 16) * 2.0 ** -24 * (sizes[0] + 1.0)
    rel = 2 * logit + 2.0 ** -p_bits + 2.0 ** -20
    own = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    return rel[..., None] * share + 2.0 ** -25 * floor + own * ref.abs() + 1e-30


def lse_tolerance(ref, sizes, hd):
    logit = (hd + 16) * 2.0 ** -24 * (sizes[0] + 1.0)
    return 1.5 * logit + 2.0 ** -20 + 2.0 ** -22 * ref.abs()


def mass_tolerance(ref, sizes, hd, G):
    B, S, Hq = sizes[0].shape
    logit = (hd + 16) * 2.0 ** -24 * (sizes[0].reshape(B, S, Hq // G, G).amax(-1) + 1.0)
    return (2 * logit + 2.0 ** -20)[..., None] * ref + G * 2.0 ** -22


def weight_update(weight, ids, mass, decay):
    out = weight.double() * decay
    B, S, topk = ids.shape
    for b in range(B):
        for s in range(S):
            for i, j in enumerate(ids[b, s].tolist()):
                if j >= 0:
                    out[b, j] += mass[b, s, :, i].double().sum()
    return out


def evict(table, ctx_len, weight, bs, budget, sink, recent):
    B, NB = table.shape
    t2, c2, w2 = table.clone(), ctx_len.clone(), torch.zeros_like(weight)
    kept = torch.full((B, budget), -1, dtype=torch.int32)
    freed = torch.zeros(B, dtype=torch.int32)
    for b in range(B):
        n = max(0, -(-int(ctx_len[b]) // bs))
        keep = list(range(n))
        if n > budget:
            sure = [j for j in keep if j < sink or j >= n - recent]
            mid = sorted((j for j in keep if sink <= j < n - recent),
                         key=lambda j: (0 if math.isnan(weight[b, j]) else 1, -float(weight[b, j]), j))
            keep = sorted(sure + mid[:budget - len(sure)])
        gone = [j for j in range(n) if j not in set(keep)]
        order = keep + gone + list(range(n, NB))
        t2[b] = table[b, order]
        w2[b, :len(keep)] = weight[b, keep]
        kept[b, :len(keep)] = torch.tensor(keep, dtype=torch.int32)
        freed[b] = len(gone)
        c2[b] = int(ctx_len[b]) - len(gone) * bs
    return t2, c2, w2, kept, freed
