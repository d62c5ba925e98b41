"""What the suffix attention over an 8-bit cache may be off by, whatever the
size of its weights and of its values.

A prefix weight times its row's V scale is carried in units of a power of two
2^k of its own for each query row and step of 32 consecutive positions, in which the
step's largest lies in (2^7.8, 2^8.8]: rounded to fp16 (2^-11 of it, or 2^-25 below fp16's
smallest normal value), then as e4m3 (2^-4 of it, or 2^-10 below the smallest normal value,
and all of it below 2^-10) and what that leaves as e5m2 (2^-3 of that).  So
  |error| <= 2^-11 w + max(2^-7 w, min(2^-13, 2^-3 w)) + 2^-25 in those units,
           <= e(w) = (2^-7 + 2^-11) w + min(2^-20.8 top, 2^-3 w) + 2^-32.8 top
with the step's largest, `top` (over blocks that hold a value).  Suffix weights are
two bf16 terms (2^-16).  The codes of V are exact, hence
  |out - o| <= half a bf16 step of o + far,
  far = sum_prefix e(p_x s_x) |code_x| + 2^-16 sum_suffix p_x |v_x| + (2 dz + 2 sums) sum_x p_x |v_x|,
dz being the logits' error (prefix_cache_ref.logit_error: once in the sum, once
in the normaliser) and sums that of n fp32 additions.  No weight is off by more than 2^-3
of itself down to 2^-28 of the largest in its step, none by more than 2^-7 down
to 2^-14 of it, and no size of V matters.

Over many elements of zero-mean values two errors remain: the output's rounding, of a
relative rms of 2^-8 / sqrt(3) * sqrt(3 / (8 ln 2)) = 1.66e-3 (a mantissa spread evenly over
its logarithm, the error evenly over a step), and the weights', 2^-4 and 2^-3 in place
of 2^-8: 2.65e-2 * 5.31e-2 = 1.41e-3; together 2.18e-3."""
import math

import torch

import prefix_cache_ref as ref

F64 = torch.float64
STEP = 32
RMS = 1.25 * 2.0 ** -9  # of a whole call's outputs: the 2.18e-3 above, and 12 % for dz and the sample


def half_step(o):
    """Half a bf16 step at |o|."""
    _, e = torch.frexp(o.abs())
    return torch.where(o == 0, 0.0, torch.exp2((e - 1).clamp(min=-126).to(F64) - 8))


def bf16(x):
    """Rounded to bf16 from 64 bits."""
    return x.to(torch.float32).to(torch.bfloat16).to(F64)


def to_type(x, bits, low):
    """Rounded to `bits` fraction bits, with the steps of 2^low's binade below it."""
    _, e = torch.frexp(x.abs())
    step = torch.exp2(torch.clamp(e - 1, min=low).to(F64) - bits)
    return torch.round(x / step) * step


def attention(q, cache, ks, vs, vis):
    """out, lse [B,Hq,S(,D)] in 64 bits, far, and the bound of lse."""
    q, ks, vs = (t.to(F64) for t in (q, ks, vs))
    k, v = dense(cache)
    B, Hq, S, D = q.shape
    H, P, block = k.shape[1], k.shape[2], cache[4]
    G = Hq // H
    out, far = (torch.zeros(B, Hq, S, D, dtype=F64) for _ in range(2))
    lse, far_lse = (torch.zeros(B, Hq, S, dtype=F64) for _ in range(2))
    for b in range(B):
        at = vis[b].nonzero()[:, 0]
        for h in range(H):
            keys, vals = torch.cat([ks[b, h], k[b, h, at]]), torch.cat([vs[b, h], v[b, h, at]])
            sl = slice(h * G, (h + 1) * G)
            z = torch.einsum("gsd,kd->gsk", q[b, sl], keys) / math.sqrt(D)
            total = torch.logsumexp(z, -1)
            p = torch.exp(z - total[..., None])
            dz = ref.logit_error(q[b, sl], keys)
            sums = keys.shape[0] * 2.0 ** -24 + 2.0 ** -21
            out[b, sl] = torch.einsum("gsk,kd->gsd", p, vals)
            far[b, sl] = (2 * dz + 2 * sums)[..., None] * torch.einsum("gsk,kd->gsd", p, vals.abs())
            far[b, sl] += 2.0 ** -16 * torch.einsum("gsk,kd->gsd", p[..., :S], vals[:S].abs())
            lse[b, sl] = total
            far_lse[b, sl] = dz + sums + 2.0 ** -21 * (1 + total.abs())
            if len(at):
                codes = cache[1][b, h].to(F64)[at].abs()
                size = torch.zeros(-(-P // block), dtype=F64).scatter_reduce(0, at // block, codes.amax(-1), "amax")
                w = p[..., S:] * cache[3][b, h].to(F64)[at // block]
                step = (at // STEP).expand(G, S, -1)
                top = torch.zeros(G, S, -(-P // STEP), dtype=F64).scatter_reduce(
                    2, step, torch.where((size > 0)[at // block], w, 0.0), "amax").gather(2, step)
                e = (2.0 ** -7 + 2.0 ** -11) * w + torch.minimum(2.0 ** -20.8 * top, w / 8) + 2.0 ** -32.8 * top
                far[b, sl] += torch.einsum("gsk,kd->gsd", e, codes)
    return out, lse, far, far_lse


def off(out, o, far):
    """(largest part of the bound that |out - o| uses, relative rms error)."""
    err = (out.to(F64) - o).abs()
    # what is rounded is up to `far` from o, past the next power of two perhaps
    worst = torch.nan_to_num(err / (half_step(o.abs() + far) + far + 2.0 ** -133), nan=math.inf).max().item()
    return worst, ((out.to(F64) - o).norm() / o.norm()).item()


def dense(cache):
    return [ref.dequant(x.to(F64), s.to(F64), cache[4]) for x, s in ((cache[0], cache[2]), (cache[1], cache[3]))]


def with_weights(q, cache, ks, vs, vis, carry):
    """out in bf16 of an attention that carries its unnormalised weights (the
    row's largest is 1) as carry(weights of the suffix, of the prefix, scale of each prefix position)."""
    q, ks, vs = (t.to(F64) for t in (q, ks, vs))
    k, _ = dense(cache)
    B, Hq, S, D = q.shape
    H, P = k.shape[1], k.shape[2]
    G = Hq // H
    out = torch.zeros(B, Hq, S, D, dtype=F64)
    for b in range(B):
        for h in range(H):
            sl = slice(h * G, (h + 1) * G)
            z = torch.einsum("gsd,kd->gsk", q[b, sl], torch.cat([ks[b, h], k[b, h]])) / math.sqrt(D)
            z[..., S:] = torch.where(vis[b], z[..., S:], -math.inf)
            p = torch.exp(z - z.amax(-1, keepdim=True))
            scale = cache[3][b, h].to(F64).repeat_interleave(cache[4])[:P]
            suffix, prefix = carry(p[..., :S], p[..., S:], scale)
            o = suffix @ vs[b, h] + prefix @ torch.where(vis[b][:, None], cache[1][b, h].to(F64), 0.0)
            out[b, sl] = bf16(o / p.sum(-1, keepdim=True))
    return out


def bf16_weights(suffix, prefix, scale):
    """One bf16 rounding of each weight."""
    return bf16(suffix), bf16(prefix) * scale


def stepped_weights(suffix, prefix, scale):
    """The terms of the module's docstring."""
    w = prefix * scale
    P = w.shape[-1]
    w = torch.nn.functional.pad(w, (0, -P % STEP)).unflatten(-1, (-1, STEP))
    top = w.amax(-1, keepdim=True)
    k = torch.floor(torch.log2(torch.where(top > 0, top, 1.0)) + 0.2)
    x = to_type(w * torch.exp2(8 - k), 10, -14)
    hi = to_type(x, 3, -6)
    lo = to_type((x - hi) * 2.0 ** 11, 2, -14)
    w = (hi + lo * 2.0 ** -11) * torch.exp2(k - 8)
    return bf16(suffix) + bf16(suffix - bf16(suffix)), w.flatten(-2)[..., :P]


def sink_inputs(g, P, S, gap, sink_value, at, block, H=1, G=2):
    """One key `gap` nats above the others, whose values have a common mean;
    its own value row is sink_value.  Returns q, the cache, suffix K and V."""
    bf, f8 = torch.bfloat16, torch.float8_e4m3fn
    q = 0.25 * torch.randn(1, H * G, S, 256, generator=g)
    q[..., 0] = 16.0                                       # z = code 0 + noise of the rest
    k = torch.randn(1, H, P, 256, generator=g)
    k[..., 0] = 0.0
    k[:, :, at] = 0.0
    k[:, :, at, 0] = gap
    v = 1.0 + 0.1 * torch.randn(1, H, P, 256, generator=g)
    v[:, :, at] = sink_value
    n = -(-P // block)
    scale = torch.full((1, H, n), 2.0 ** -3)
    ks = torch.randn(1, H, S, 256, generator=g)
    ks[..., 0] = 0.0
    vs = 1.0 + 0.1 * torch.randn(1, H, S, 256, generator=g)
    return q.to(bf), (k.to(f8), (v * 8).to(f8), torch.ones(1, H, n), scale, block), ks.to(bf), vs.to(bf)
