"""Plain 64-bit forms of the prefix-cache compression operators, on the CPU,
written from their definitions; and the error bounds of the attention and of
the accumulated weight, derived from the roundings their kernels make.

Everything is float64 numpy/torch; the 8-bit rounding is done by arithmetic
(round to the nearest multiple of the step, ties to even), not by a cast.
"""
import math

import numpy as np
import torch

D = 256
F64 = torch.float64


def e4m3_round(x):
    """float64 array -> nearest e4m3 value (|x| <= 448; non-finite -> NaN)."""
    x = np.asarray(x, dtype=np.float64)
    out = np.full_like(x, np.nan)
    fin = np.isfinite(x)
    v = x[fin]
    _, e = np.frexp(np.abs(v))                 # |v| = f * 2^e, f in [0.5, 1)
    step = np.exp2(np.maximum(e - 1, -6) - 3.0)  # 3 fraction bits; smallest normal 2^-6
    out[fin] = np.rint(v / step) * step
    return out


def pow2_scale(amax):
    """The smallest power of two >= 2^-64 with amax <= 448 * it; 1 for 0."""
    if amax == 0:
        return 1.0
    t = -64
    while amax > 448.0 * 2.0 ** t:
        t += 1
    return 2.0 ** t


def lengths(valid, B, P):
    return [P] * B if valid is None else [min(max(int(x), 0), P) for x in valid]


def quantize(x, valid, block, first, codes, scales):
    """Writes rows [first, valid) of x (float64 [B,H,P,D]) into codes / scales."""
    B, H, P, _ = x.shape
    for b, n in enumerate(lengths(valid, B, P)):
        for h in range(H):
            for j in range(first, n, block):
                part = x[b, h, j:min(j + block, n)].numpy()
                fin = np.abs(part[np.isfinite(part)])
                s = pow2_scale(float(fin.max()) if fin.size else 0.0)
                scales[b, h, j // block] = s
                codes[b, h, j:j + part.shape[0]] = torch.from_numpy(e4m3_round(part / s))
    return codes, scales


def dequant(codes, scales, block):
    P = codes.shape[2]
    return codes * scales.repeat_interleave(block, dim=2)[:, :, :P, None]


def visible(valid, mask, B, P):
    vis = torch.zeros(B, P, dtype=torch.bool)
    for b, n in enumerate(lengths(valid, B, P)):
        vis[b, :n] = True
    return vis if mask is None else vis & (mask != 0)


def logit_error(q, keys):
    """Bound on |z - exact| of a scaled logit of query row q [.., D] against
    keys [n, D]: products of 256 terms summed in fp32 (256 * 2^-24 of the sum
    of magnitudes), and the query carried as two e4m3 terms of its row scaled
    so that its largest element lies in (224, 448]: the second term's
    smallest step is 2^-9, so the remainder is at most 2^-10 in those units,
    2^-10 / 224 < 2^-17 of the row's largest element."""
    a = torch.einsum("...d,kd->...k", q.abs(), keys.abs())
    top = q.abs().amax(-1, keepdim=True) * keys.abs().sum(-1)
    return ((2.0 ** -16 * a + 2.0 ** -17 * top) / math.sqrt(D)).amax(-1)


def attention(q, k, v, ks, vs, vis, v_step=None):
    """out, lse and their bounds.  q [B,Hq,S,D]; k, v [B,H,P,D]; all float64;
    v_step [B,H,P]: each prefix row's scale (the unit its weight is held in).

    Bound on out, per element: the output's bf16 rounding (2^-8 |o|); each
    weight held in two e4m3 terms of an fp16 value (2^-4 * 2^-4 + 2^-11) or,
    for suffix rows, in bf16 (2^-8); the two-term form's smallest step 2^-9,
    an error of at most 2^-10 in units in which the row's largest weight is at
    least 2^4, so 2^-14 of the largest (weight x scale) times each code; the
    logit error through p' = p dz, once in the sum and once in the normaliser; and fp32 sums."""
    B, Hq, S, _ = q.shape
    H = k.shape[1]
    G = Hq // H
    out = torch.zeros(B, Hq, S, D, dtype=F64)
    lse = torch.zeros(B, Hq, S, dtype=F64)
    tol = torch.zeros_like(out)
    tol_lse = torch.zeros_like(lse)
    for b in range(B):
        at = vis[b].nonzero()[:, 0]
        for h in range(H):
            keys = torch.cat([ks[b, h], k[b, h, at]])
            vals = torch.cat([vs[b, h], v[b, h, at]])
            step = torch.cat([torch.ones(S, dtype=F64), torch.ones(len(at), dtype=F64) if v_step is None else v_step[b, h, at]])
            sl = slice(h * G, (h + 1) * G)
            z = torch.einsum("gsd,kd->gsk", q[b, sl], keys) / math.sqrt(D)
            total = torch.logsumexp(z, -1)
            p = torch.exp(z - total[..., None])
            o = torch.einsum("gsk,kd->gsd", p, vals)
            dz = logit_error(q[b, sl], keys)
            n = keys.shape[0]
            sums = n * 2.0 ** -24 + 2.0 ** -21
            mags = torch.einsum("gsk,kd->gsd", p, vals.abs())
            small = (p * step).amax(-1)[..., None] * (vals / step[:, None]).abs().sum(0)
            out[b, sl], lse[b, sl] = o, total
            tol[b, sl] = (2.0 ** -8 * o.abs() + (2.0 ** -8 + 2.0 ** -11 + 2 * dz + 2 * sums)[..., None] * mags
                          + 2.0 ** -14 * small + 1e-30)
            tol_lse[b, sl] = dz + sums + 2.0 ** -21 * (1 + total.abs())
    return out, lse, tol, tol_lse


def mass(q, k, lse, vis, before):
    """mass and its bound: every weight carries its logit's error, the
    rounding of z * log2(e) - lse * log2(e) in fp32 (2^-22 of their sizes),
    the exponential's 2^-21, and the sum over the queries."""
    B, Hq, S, _ = q.shape
    H, P = k.shape[1], k.shape[2]
    G = Hq // H
    out = torch.zeros(B, H, P, dtype=F64) if before is None else before.to(F64).clone()
    tol = torch.zeros(B, H, P, dtype=F64)
    for b in range(B):
        at = vis[b].nonzero()[:, 0]
        if not len(at):
            continue
        for h in range(H):
            sl = slice(h * G, (h + 1) * G)
            keys = k[b, h, at]
            z = torch.einsum("gsd,kd->gsk", q[b, sl], keys) / math.sqrt(D)
            ls = lse[b, sl].to(F64)[..., None]
            w = torch.where(torch.isneginf(ls), 0.0, torch.exp(z - ls))
            size = z.abs() + torch.where(torch.isinf(ls), 0.0, ls.abs())
            rel = logit_error(q[b, sl], keys)[..., None] + 2.0 ** -21 * (size + 1) + G * S * 2.0 ** -24
            out[b, h, at] += w.sum((0, 1))
            tol[b, h, at] = (w * rel).sum((0, 1)) + 2.0 ** -23 * out[b, h, at].abs() + 1e-37
    return out, tol


def evict_order(m, vis, n, n_keep, n_first, n_last):
    """Kept positions (ascending) of one (sample, KV head); m: list of floats."""
    def key(j):
        guard = j < n_first or j >= n - n_last
        nan = not guard and m[j] != m[j]
        return (not guard, nan, 0.0 if guard or nan else -m[j], j)
    return sorted(sorted((j for j in range(len(m)) if vis[j]), key=key)[:n_keep])
