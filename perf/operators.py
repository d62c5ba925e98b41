"""Cases of the prefix-cache compression operators, with their plain forms.

Four operators on a bucket-padded prefix KV cache [B, Hkv, P, 256]:

* ``quantize``: the 8-bit cache (e4m3 codes, one power-of-two scale for each
  block of tokens and KV head) from the bf16 prefix K/V;
* ``attn``: the suffix attention over that cache and the suffix's own bf16 K/V;
* ``mass``: the attention weight that each cache position received, summed
  over a KV head's queries, added to what it had received before;
* ``evict``: the rows of largest weight, gathered into a smaller bucket.
"""
import math

import torch

own = False

D = 256


# ------------------------------------------------------------------ cases

def listed():
    return [
        # filling the cache of one request of the smallest bucket (a LIBERO-shape prefix)
        dict(name="quantize b1 p576", op="quantize", B=1, Hq=8, Hkv=4, P=576, valid=512, block=64),
        # filling the cache of a full batch, every sample with a valid length of its own
        dict(name="quantize b32 p1024", op="quantize", B=32, Hq=8, Hkv=4, P=1024, valid=-576, block=64),
        # one query token against the smallest bucket: the single-token form
        dict(name="attn token b1 p576", op="attn", B=1, Hq=8, Hkv=4, P=576, valid=512, S=1, block=64, mask=False),
        # one denoising step of the base model's action chunk
        dict(name="attn chunk b1 p1024", op="attn", B=1, Hq=8, Hkv=4, P=1024, valid=900, S=50, block=64, mask=False),
        # the batched step with hidden prefix positions
        dict(name="attn chunk b32 p1024 mask", op="attn", B=32, Hq=8, Hkv=4, P=1024, valid=-576, S=50, block=64, mask=True),
        # a long history, odd bucket, small scale blocks, short chunk
        dict(name="attn long b2 p30016", op="attn", B=2, Hq=8, Hkv=4, P=30016, valid=29987, S=10, block=16, mask=False),
        # the weight of one step over a history prefix held in bf16
        dict(name="mass b1 p2048", op="mass", B=1, Hq=8, Hkv=4, P=2048, valid=1900, S=50, block=0, mask=False, add=False),
        # the weight of a batched step over the 8-bit cache, added to earlier steps' weight
        dict(name="mass b32 p1024 8-bit", op="mass", B=32, Hq=8, Hkv=4, P=1024, valid=-576, S=50, block=64, mask=True, add=True),
        # the same over a bf16 cache
        dict(name="mass b32 p1024", op="mass", B=32, Hq=8, Hkv=4, P=1024, valid=-576, S=50, block=0, mask=True, add=True),
        # a history bucket cut to the largest prefix bucket
        dict(name="evict b1 p2048", op="evict", B=1, Hq=8, Hkv=4, P=2048, valid=1900, block=0, mask=False, keep=1000,
             Pout=1024, first=16, last=64),
        # a batch of bf16 caches cut to the smallest bucket
        dict(name="evict b32 p1024", op="evict", B=32, Hq=8, Hkv=4, P=1024, valid=-576, block=0, mask=True, keep=512,
             Pout=576, first=0, last=0),
        # a batch of 8-bit caches cut to the smallest bucket
        dict(name="evict b32 p1024 8-bit", op="evict", B=32, Hq=8, Hkv=4, P=1024, valid=-576, block=64, mask=True,
             keep=512, Pout=576, first=4, last=32),
    ]


def draw(rng):
    op = rng.choice(("quantize", "attn", "attn", "mass", "evict"))
    Hkv = rng.choice((1, 2, 4, 8))
    G = rng.choice((1, 2, 4))
    B = int(round(math.exp(rng.uniform(0, math.log(33))))) or 1
    most = 131072 // (B * Hkv)  # rows of the listed batch
    P = max(1, min(int(math.exp(rng.uniform(math.log(16), math.log(32768)))), most))
    valid = rng.choice((P, -max(1, P // 2), -1, rng.randint(1, P)))
    c = dict(op=op, B=B, Hq=Hkv * G, Hkv=Hkv, P=P, valid=valid)
    block = rng.choice((16, 32, 64, 128))
    if op in ("attn", "mass"):
        c["S"] = rng.choice((1, rng.randint(1, 128 // G), rng.randint(1, 128 // G), 128 // G))
        c["mask"] = rng.random() < 0.5
    if op == "mass":
        c["add"] = rng.random() < 0.5
    if op == "evict":
        c["mask"] = rng.random() < 0.5
        c["keep"] = rng.randint(1, P)
        c["Pout"] = c["keep"] + rng.choice((0, 1, rng.randint(0, 200)))
        c["first"], c["last"] = rng.choice(((0, 0), (4, 0), (rng.randint(0, 32), rng.randint(0, 64))))
    c["block"] = block if op in ("quantize", "attn") or rng.random() < 0.5 else 0
    return c


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _lengths(case, g):
    """Valid lengths: the given one, or for a negative value -v uniform in [v, P]."""
    B, P, v = case["B"], case["P"], case["valid"]
    if v >= 0:
        return torch.full((B,), v, dtype=torch.int32, device="cuda")
    return torch.randint(-v, P + 1, (B,), generator=g, device="cuda", dtype=torch.int64).to(torch.int32)


def _visible(case, vl, mask):
    vis = torch.arange(case["P"], device=vl.device)[None] < vl[:, None]
    return vis if mask is None else vis & (mask != 0)


def _pack(x, block):
    """Plain codes and scales of x [B, Hkv, P, D], every row in range."""
    B, H, P, _ = x.shape
    n = (P + block - 1) // block
    pad = torch.zeros(B, H, n * block, D, dtype=torch.float32, device=x.device)
    pad[:, :, :P] = x.float()
    pad = pad.view(B, H, n, block * D)
    s = _pow2_scale(pad.abs().amax(-1))
    codes = (pad / s[..., None]).to(torch.float8_e4m3fn).view(B, H, n * block, D)[:, :, :P]
    return codes.contiguous(), s


def _pow2_scale(amax):
    """The smallest power of two s >= 2^-64 with amax <= 448 s; 1 for amax = 0."""
    m, e = torch.frexp(amax)
    t = torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-64)
    return torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), t), torch.ones_like(amax))


def prepare(case, seed):
    g = _gen(seed)
    B, Hq, Hkv, P, op = case["B"], case["Hq"], case["Hkv"], case["P"], case["op"]
    bf, dev = torch.bfloat16, "cuda"
    vl = _lengths(case, g)
    k = torch.randn(B, Hkv, P, D, generator=g, device=dev)
    # a few keys that draw much of the attention, and values whose size moves along the prefix
    peak = torch.rand(B, 1, P, 1, generator=g, device=dev) < 0.01
    k = torch.where(peak, 4.0 * k, k).to(bf)
    v = torch.randn(B, Hkv, P, D, generator=g, device=dev)
    v = (v * torch.exp2(2.0 * torch.rand(B, Hkv, P, 1, generator=g, device=dev))).to(bf)
    st = dict(case=case, valid=vl, mask=None)
    if case.get("mask"):
        st["mask"] = (torch.rand(B, P, generator=g, device=dev) >= 0.1).to(torch.uint8)
    block = case["block"]
    if op == "quantize":
        n = (P + block - 1) // block
        st.update(k=k, v=v)
        for name in ("k8", "v8"):
            st[name] = torch.zeros(B, Hkv, P, D, device=dev).to(torch.float8_e4m3fn)
        for name in ("ks", "vs"):
            st[name] = torch.ones(B, Hkv, n, device=dev)
        return st
    if block:
        st["k8"], st["ks"] = _pack(k, block)
        st["v8"], st["vs"] = _pack(v, block)
    else:
        st.update(k=k, v=v)
    if op in ("attn", "mass"):
        S = case["S"]
        st["q"] = torch.randn(B, Hq, S, D, generator=g, device=dev).to(bf)
        st["k_suffix"] = torch.randn(B, Hkv, S, D, generator=g, device=dev).to(bf)
        st["v_suffix"] = torch.randn(B, Hkv, S, D, generator=g, device=dev).to(bf)
        st["out"] = torch.empty(B, Hq, S, D, dtype=bf, device=dev)
        st["lse"] = torch.empty(B, Hq, S, device=dev)
    if op == "mass":
        _, st["lse"] = _attn(st)
        st["mass"] = torch.zeros(B, Hkv, P, device=dev)
        st["before"] = None
        if case["add"]:
            st["before"] = torch.empty(B, Hkv, P, device=dev).exponential_(0.2, generator=g)
        del st["k_suffix"], st["v_suffix"], st["out"]
        for name in ("v", "v8", "vs"):
            st.pop(name, None)
    if op == "evict":
        Pout = case["Pout"]
        # weight is spread unevenly, and positions nothing attended to tie at zero
        m = torch.empty(B, Hkv, P, device=dev).exponential_(1.0, generator=g) ** 3
        m = torch.where(torch.rand(B, Hkv, P, generator=g, device=dev) < 0.05, torch.zeros_like(m), m)
        st["mass"] = m
        new = lambda dt: torch.zeros(B, Hkv, Pout, D, device=dev).to(dt)  # noqa: E731
        st["k_new"], st["v_new"] = (new(torch.float8_e4m3fn), new(torch.float8_e4m3fn)) if block else (new(bf), new(bf))
        if block:
            n = (Pout + block - 1) // block
            st["ks_new"], st["vs_new"] = torch.ones(B, Hkv, n, device=dev), torch.ones(B, Hkv, n, device=dev)
        st["mass_new"] = torch.zeros(B, Hkv, Pout, device=dev)
        st["pos"] = torch.zeros(B, Hkv, Pout, dtype=torch.int32, device=dev)
        st["valid_new"] = torch.zeros(B, dtype=torch.int32, device=dev)
    return st


# ------------------------------------------------------------------ plain forms (fp32)

def _per_row(scale, block, P):
    return scale.repeat_interleave(block, dim=2)[:, :, :P, None]


def _dense(st, name):
    """The K or V prefix in fp32, from either form of the cache."""
    block = st["case"]["block"]
    if not block:
        return st[name].float()
    return st[name + "8"].float() * _per_row(st[name + "s"], block, st["case"]["P"])


def _quantize(st):
    c = st["case"]
    B, H, P, block = c["B"], c["Hkv"], c["P"], c["block"]
    n = (P + block - 1) // block
    inside = _visible(c, st["valid"], None)[:, None, :, None]
    any_row = (torch.arange(n, device=inside.device)[None] * block < st["valid"][:, None])[:, None]
    res = []
    for x, codes, scale in ((st["k"], st["k8"], st["ks"]), (st["v"], st["v8"], st["vs"])):
        x = torch.where(inside, x.float(), 0.0)
        pad = torch.zeros(B, H, n * block, D, device=x.device)
        pad[:, :, :P] = x
        s = _pow2_scale(pad.view(B, H, n, block * D).abs().amax(-1))
        new = (x / _per_row(s, block, P)).to(torch.float8_e4m3fn)
        res += [torch.where(inside, new.view(torch.uint8), codes.view(torch.uint8)).view(torch.float8_e4m3fn),
                torch.where(any_row, s, scale)]
    return dict(k=res[0], k_scale=res[1], v=res[2], v_scale=res[3])


def _attn(st):
    c = st["case"]
    B, Hq, H, P, S = c["B"], c["Hq"], c["Hkv"], c["P"], c["S"]
    vis = _visible(c, st["valid"], st["mask"])[:, None, :, None]
    q = st["q"].float().view(B, H, Hq // H * S, D)
    k = torch.cat([st["k_suffix"].float(), _dense(st, "k")], dim=2)
    v = torch.cat([st["v_suffix"].float(), torch.where(vis, _dense(st, "v"), 0.0)], dim=2)
    see = torch.cat([torch.ones(B, S, dtype=torch.bool, device=q.device), vis[:, 0, :, 0]], dim=1)[:, None, None]
    z = torch.matmul(q, k.transpose(2, 3)) * (1.0 / math.sqrt(D))
    z = torch.where(see, z, -math.inf)
    top = z.amax(-1, keepdim=True)
    p = torch.exp(z - top)
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v) / total
    lse = top + torch.log(total)
    return out.view(B, Hq, S, D).to(torch.bfloat16), lse.view(B, Hq, S)


def _mass(st):
    c = st["case"]
    B, Hq, H, S = c["B"], c["Hq"], c["Hkv"], c["S"]
    q = st["q"].float().view(B, H, Hq // H * S, D)
    z = torch.matmul(q, _dense(st, "k").transpose(2, 3)) * (1.0 / math.sqrt(D))
    w = torch.exp(z - st["lse"].view(B, H, Hq // H * S, 1))
    vis = _visible(c, st["valid"], st["mask"])[:, None]
    m = torch.where(vis, w.sum(2), 0.0)
    return m if st["before"] is None else st["before"] + m


def _order(mass, vis, valid, first, last):
    """Positions from the most to the least wanted: protected ones, then by
    weight, the lowest index first among equals; hidden ones last."""
    at = torch.arange(mass.shape[-1], device=mass.device)
    guard = (at[None] < first) | (at[None] >= valid[:, None] - last)
    score = torch.where(guard[:, None], math.inf, mass)
    score = torch.where(vis[:, None], score, -math.inf)
    return torch.sort(score, dim=-1, descending=True, stable=True).indices


def _evict(st):
    c = st["case"]
    B, H, Pout, block = c["B"], c["Hkv"], c["Pout"], c["block"]
    vis = _visible(c, st["valid"], st["mask"])
    count = vis.sum(-1).clamp(max=c["keep"])
    order = _order(st["mass"], vis, st["valid"], c["first"], c["last"])[..., :c["keep"]]
    inside = torch.arange(Pout, device=vis.device)[None] < count[:, None]
    far = torch.where(inside[:, None, :c["keep"]], order, c["P"])  # what is not kept sorts behind
    pos = torch.full((B, H, Pout), c["P"], dtype=torch.int64, device=vis.device)
    pos[..., :c["keep"]] = far.sort(-1).values
    src = pos.clamp(max=c["P"] - 1)
    inside = inside[:, None]
    res = dict(positions=torch.where(inside, pos, -1).to(torch.int32), valid_len=count.to(torch.int32),
               mass=torch.where(inside, st["mass"].gather(2, src), 0.0))
    rows = src[..., None].expand(B, H, Pout, D)
    for name in ("k", "v"):
        x = torch.where(inside[..., None], _dense(st, name).gather(2, rows), 0.0)
        if not block:
            res[name] = torch.where(inside[..., None], x.to(torch.bfloat16), st[name + "_new"])
            continue
        n = (Pout + block - 1) // block
        pad = torch.zeros(B, H, n * block, D, device=x.device)
        pad[:, :, :Pout] = x
        s = _pow2_scale(pad.view(B, H, n, block * D).abs().amax(-1))
        new = (x / _per_row(s, block, Pout)).to(torch.float8_e4m3fn)
        res[name] = torch.where(inside[..., None], new.view(torch.uint8),
                                st[name + "_new"].view(torch.uint8)).view(torch.float8_e4m3fn)
        any_row = (torch.arange(n, device=x.device)[None] * block < count[:, None])[:, None]
        res[name + "_scale"] = torch.where(any_row, s, st[name + "s_new"])
    return res


# ------------------------------------------------------------------ the framework's calls

def _run_own(st):
    from gqa_prefix_suffix_b200 import binding as bd
    c, op = st["case"], st["case"]["op"]
    if op == "quantize":
        cache = bd.Kv8Cache(st["k8"], st["v8"], st["ks"], st["vs"], c["block"])
        bd.kv8_quantize(st["k"], st["v"], valid_len=st["valid"], out=cache)
        return dict(k=cache.k, k_scale=cache.k_scale, v=cache.v, v_scale=cache.v_scale)
    if op == "attn":
        cache = bd.Kv8Cache(st["k8"], st["v8"], st["ks"], st["vs"], c["block"])
        out, lse = bd.suffix_attn_kv8(st["q"], cache, st["k_suffix"], st["v_suffix"], prefix_valid_len=st["valid"],
                                      prefix_mask=st["mask"], out=st["out"], lse=st["lse"])
        return dict(out=out, lse=lse)
    if op == "mass":
        if c["block"]:
            m = bd.prefix_attn_mass_kv8(st["q"], st["k8"], st["ks"], c["block"], st["lse"],
                                        prefix_valid_len=st["valid"], prefix_mask=st["mask"],
                                        mass_in=st["before"], mass=st["mass"])
        else:
            m = bd.prefix_attn_mass(st["q"], st["k"], st["lse"], prefix_valid_len=st["valid"],
                                    prefix_mask=st["mask"], mass_in=st["before"], mass=st["mass"])
        return dict(mass=m)
    kept = dict(n_keep=c["keep"], n_first=c["first"], n_last=c["last"], prefix_valid_len=st["valid"],
                prefix_mask=st["mask"])
    if c["block"]:
        new = bd.Kv8Cache(st["k_new"], st["v_new"], st["ks_new"], st["vs_new"], c["block"])
        e = bd.prefix_evict_kv8(bd.Kv8Cache(st["k8"], st["v8"], st["ks"], st["vs"], c["block"]), st["mass"],
                                out=new, mass_out=st["mass_new"], positions=st["pos"], valid_len=st["valid_new"],
                                **kept)
        return dict(k=new.k, k_scale=new.k_scale, v=new.v, v_scale=new.v_scale, mass=e.mass, positions=e.positions,
                    valid_len=e.valid_len)
    e = bd.prefix_evict(st["k"], st["v"], st["mass"], k_out=st["k_new"], v_out=st["v_new"], mass_out=st["mass_new"],
                        positions=st["pos"], valid_len=st["valid_new"], **kept)
    return dict(k=e.k, v=e.v, mass=e.mass, positions=e.positions, valid_len=e.valid_len)


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "quantize":
        return _quantize(state)
    if op == "attn":
        out, lse = _attn(state)
        return dict(out=out, lse=lse)
    if op == "mass":
        return dict(mass=_mass(state))
    return _evict(state)


def work(case):
    B, Hq, H, P, op = case["B"], case["Hq"], case["Hkv"], case["P"], case["op"]
    v = case["valid"]
    rows = B * H * (v if v >= 0 else (P - v) / 2)  # mean length of the drawn ones
    block = case["block"]
    n = B * H * ((P + block - 1) // block) if block else 0
    cell = (1 if block else 2) * D  # one row of K or of V
    seen = rows * (0.9 if case.get("mask") else 1.0)
    side = 4 * B + (B * P if case.get("mask") else 0)
    if op == "quantize":
        return dict(bytes=2 * rows * (2 * D + D) + 8 * n + side, flops=4 * rows * D)
    if op == "attn":
        S = case["S"]
        keys = seen + B * H * S
        byts = 2 * seen * cell + 8 * n + 2 * D * (2 * B * Hq * S + 2 * B * H * S) + 4 * B * Hq * S + side
        return dict(bytes=byts, flops=4 * D * (Hq // H) * S * keys)
    if op == "mass":
        S = case["S"]
        byts = seen * cell + 4 * n + 2 * D * B * Hq * S + 4 * B * Hq * S + side
        byts += 4 * B * H * P * (2 if case["add"] else 1)
        return dict(bytes=byts, flops=2 * D * (Hq // H) * S * seen)
    kept = min(B * H * case["keep"], seen)
    new = B * H * ((case["Pout"] + block - 1) // block) if block else 0
    return dict(bytes=4 * kept * cell + 4 * rows + 8 * B * H * case["Pout"] + 8 * (n + new) + side, flops=rows)


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    """The operators' definitions in 64 bits, one (sample, KV head) at a time."""
    st = prepare(case, seed)
    op, B, H, P, block = case["op"], case["B"], case["Hkv"], case["P"], case["block"]
    f64 = torch.float64
    lengths = st["valid"].tolist()

    def rows_of(b, h, name, at):
        if not block:
            return st[name][b, h, at].to(f64)
        return st[name + "8"][b, h, at].to(f64) * st[name + "s"][b, h, at // block].to(f64)[:, None]

    def shown(b):
        at = torch.arange(lengths[b], device="cuda")
        return at if st["mask"] is None else at[st["mask"][b, :lengths[b]] != 0]

    def fill(x, codes, scale):
        """Codes and scales of the rows x (64 bits) into codes [P, D] and scale [n]."""
        for j in range(0, x.shape[0], block):
            part = x[j:j + block]
            a = float(part.abs().max())
            s = 1.0
            if a > 0:
                t = max(-64, math.frexp(a)[1] - 10)
                while a > 448.0 * 2.0 ** t:
                    t += 1
                s = 2.0 ** t
            scale[j // block] = s
            codes[j:j + part.shape[0]] = (part / s).to(torch.float32)

    if op == "quantize":
        if B * H * P > 40000:
            return None
        res = dict(k=st["k8"].to(f64), k_scale=st["ks"].to(f64), v=st["v8"].to(f64), v_scale=st["vs"].to(f64))
        for b in range(B):
            for h in range(H):
                for name in ("k", "v"):
                    codes = torch.zeros(lengths[b], D, device="cuda")
                    fill(st[name][b, h, :lengths[b]].to(f64), codes, res[name + "_scale"][b, h])
                    res[name][b, h, :lengths[b]] = codes.to(torch.float8_e4m3fn).to(f64)
        return res
    if op == "attn":
        G, S = case["Hq"] // H, case["S"]
        out = torch.zeros(B, case["Hq"], S, D, dtype=f64, device="cuda")
        lse = torch.zeros(B, case["Hq"], S, dtype=f64, device="cuda")
        for b in range(B):
            at = shown(b)
            for h in range(H):
                keys = torch.cat([rows_of(b, h, "k", at), st["k_suffix"][b, h].to(f64)])
                vals = torch.cat([rows_of(b, h, "v", at), st["v_suffix"][b, h].to(f64)])
                z = torch.einsum("gsd,kd->gsk", st["q"][b, h * G:(h + 1) * G].to(f64), keys) / math.sqrt(D)
                total = torch.logsumexp(z, -1)
                lse[b, h * G:(h + 1) * G] = total
                out[b, h * G:(h + 1) * G] = torch.einsum("gsk,kd->gsd", torch.exp(z - total[..., None]), vals)
        return dict(out=out, lse=lse)
    if op == "mass":
        G = case["Hq"] // H
        res = torch.zeros(B, H, P, dtype=f64, device="cuda")
        for b in range(B):
            at = shown(b)
            for h in range(H):
                z = torch.einsum("gsd,kd->gsk", st["q"][b, h * G:(h + 1) * G].to(f64), rows_of(b, h, "k", at))
                w = torch.exp(z / math.sqrt(D) - st["lse"][b, h * G:(h + 1) * G, :, None].to(f64))
                res[b, h, at] = w.sum((0, 1))
        return dict(mass=res if st["before"] is None else res + st["before"].to(f64))
    # evict: the positions are whole numbers, found here once more from the definition
    Pout, keep, first, last = case["Pout"], case["keep"], case["first"], case["last"]
    if block and B * H * keep > 40000:
        return None
    k, v = st["k_new"].to(f64), st["v_new"].to(f64)
    res = dict(k=k, v=v, mass=torch.zeros(B, H, Pout, dtype=f64, device="cuda"),
               positions=torch.full((B, H, Pout), -1, dtype=torch.int32),
               valid_len=torch.zeros(B, dtype=torch.int32))
    if block:
        res["k_scale"], res["v_scale"] = st["ks_new"].to(f64), st["vs_new"].to(f64)
    for b in range(B):
        at = shown(b).tolist()
        for h in range(H):
            m = st["mass"][b, h].tolist()
            want = sorted(at, key=lambda j: (not (j < first or j >= lengths[b] - last), 0.0 if (
                j < first or j >= lengths[b] - last) else -m[j], j))[:keep]
            want = torch.tensor(sorted(want), dtype=torch.int64, device="cuda")
            n = want.numel()
            res["valid_len"][b] = n
            res["positions"][b, h, :n] = want.to(torch.int32).cpu()
            res["mass"][b, h, :n] = st["mass"][b, h, want].to(f64)
            for name in ("k", "v"):
                x = rows_of(b, h, name, want)
                if not block:
                    res[name][b, h, :n] = x
                    continue
                codes = torch.zeros(n, D, device="cuda")
                fill(x, codes, res[name + "_scale"][b, h])
                res[name][b, h, :n] = codes.to(torch.float8_e4m3fn).to(f64)
    return res
