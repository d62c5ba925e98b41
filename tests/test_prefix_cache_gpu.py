"""The prefix-cache compression operators on the GPU against their plain
64-bit forms (prefix_cache_ref), whose docstrings derive the bounds."""
import os
import subprocess
import sys
import threading

import pytest
import torch

import prefix_cache_ref as ref
from gqa_prefix_suffix_b200 import binding as bd

pytestmark = pytest.mark.gpu

BF, F8, F64 = torch.bfloat16, torch.float8_e4m3fn, torch.float64


@pytest.fixture(autouse=True)
def needs_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    rc, word = bd.dm05_get_error_word(None)
    assert rc == 0 and word == 0, f"error word {word:#x}"


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rand(g, *shape):
    return torch.randn(*shape, generator=g, dtype=torch.float32)


def i32(v):
    return None if v is None else torch.tensor(v, dtype=torch.int32)


def cu(t):
    return None if t is None else t.cuda()


def same(a, b):
    """Equal values, NaN where NaN."""
    a, b = a.to(F64).cpu(), b.to(F64).cpu()
    return bool(((a == b) | (torch.isnan(a) & torch.isnan(b))).all())


# ------------------------------------------------------------------ quantise

def check_quantize(k, v, valid, block, first=0):
    """Fresh buffers of recognisable content: what is not written must stay."""
    B, H, P, _ = k.shape
    n = -(-P // block)
    c0 = torch.full((B, H, P, 256), 0.5).to(F8)
    s0 = torch.full((B, H, n), 3.0)
    out = bd.Kv8Cache(c0.cuda(), c0.cuda(), s0.cuda(), s0.cuda(), block)
    bd.kv8_quantize(k.cuda(), v.cuda(), valid_len=cu(i32(valid)), first=first, out=out)
    for x, codes, scales in ((k, out.k, out.k_scale), (v, out.v, out.v_scale)):
        want, ws = ref.quantize(x.to(F64), valid, block, first, c0.to(F64), s0.to(F64))
        assert same(scales, ws)
        assert same(codes, want)


@pytest.mark.parametrize("block", [16, 32, 64, 128])
@pytest.mark.parametrize("P,valid", [(1, None), (1, [0, 1]), (15, [15, 7]), (16, None), (127, [127, 1]),
                                     (129, [128, 129]), (200, [0, 133]), (576, [512, 575]), (1000, None)])
def test_quantize(block, P, valid):
    g = gen(P * 7 + block)
    k = (rand(g, 2, 2, P, 256) * torch.exp2(6 * torch.rand(2, 2, P, 1, generator=g) - 3)).to(BF)
    v = (rand(g, 2, 2, P, 256) * 1e-3).to(BF)
    check_quantize(k, v, valid, block)


@pytest.mark.parametrize("first,valid", [(64, None), (128, [100, 300]), (256, [0, 255])])
def test_quantize_in_pieces(first, valid):
    g = gen(first)
    k, v = rand(g, 2, 3, 300, 256).to(BF), rand(g, 2, 3, 300, 256).to(BF)
    check_quantize(k, v, valid, 64, first)
    # the pieces together are the whole
    whole = bd.kv8_quantize(k.cuda(), v.cuda(), 64, cu(i32(valid)))
    parts = bd.kv8_quantize(k[:, :, :300].cuda(), v.cuda(), 64, cu(i32([min(x, first) for x in (valid or [300, 300])])))
    bd.kv8_quantize(k.cuda(), v.cuda(), valid_len=cu(i32(valid)), first=first, out=parts)
    for a, b in zip(whole[:4], parts[:4]):
        assert same(a, b)


def test_quantize_extreme_values():
    g = gen(3)
    k = rand(g, 1, 1, 96, 256)
    k[0, 0, :16] = 0.0                                   # a block of zeros
    k[0, 0, 16:32] *= 1e-38                              # below the smallest scale
    k[0, 0, 32:48] *= 1e37
    k[0, 0, 40, 3] = 3.38953139e38                       # the largest bf16 value
    k[0, 0, 48, 0], k[0, 0, 49, 1], k[0, 0, 50, 2] = float("inf"), float("-inf"), float("nan")
    k[0, 0, 64:80] = float("nan")                        # nothing finite in the block
    k[0, 0, 80] = 448.0
    k[0, 0, 81, :128] = -0.0
    v = torch.zeros(1, 1, 96, 256)
    v[0, 0, 0, 0] = 1.7578125                            # just over 1.75: the next scale
    v[0, 0, 16, 5] = 1.75
    v[0, 0, 32, 5] = 2.0 ** -133                         # the smallest bf16 subnormal
    check_quantize(k.to(BF), v.to(BF), None, 16)


def test_quantize_ignores_rows_out_of_range():
    g = gen(4)
    k, v = rand(g, 2, 2, 128, 256).to(BF), rand(g, 2, 2, 128, 256).to(BF)
    k[:, :, 70:] = float("nan")
    v[:, :, 70:] = 1e30
    check_quantize(k, v, [70, 64], 64)


# ------------------------------------------------------------------ attention

def make_cache(g, B, H, P, block, spread=2.0, pow2=True):
    """A random cache with scales that differ from block to block."""
    n = -(-P // block)
    codes = [rand(g, B, H, P, 256).mul(60).clamp(-448, 448).to(F8) for _ in range(2)]
    e = [torch.exp2(-6 + spread * (torch.rand(B, H, n, generator=g) - 0.5)) for _ in range(2)]
    if pow2:
        e = [torch.exp2(torch.round(torch.log2(x))) for x in e]
    return bd.Kv8Cache(codes[0], codes[1], e[0], e[1], block)


def on_gpu(c):
    return bd.Kv8Cache(c.k.cuda(), c.v.cuda(), c.k_scale.cuda(), c.v_scale.cuda(), c.block)


def check_attention(g, B, Hq, H, P, S, block, valid=None, mask=None, c=None, q=None, what="", **kw):
    c = make_cache(g, B, H, P, block) if c is None else c
    q = rand(g, B, Hq, S, 256).to(BF) if q is None else q
    ks, vs = rand(g, B, H, S, 256).to(BF), rand(g, B, H, S, 256).to(BF)
    out, lse = bd.suffix_attn_kv8(q.cuda(), on_gpu(c), ks.cuda(), vs.cuda(), cu(i32(valid)), cu(mask), **kw)
    vis = ref.visible(valid, mask, B, P)
    k, v = (ref.dequant(x.to(F64), s.to(F64), block) for x, s in ((c.k, c.k_scale), (c.v, c.v_scale)))
    step = c.v_scale.to(F64).repeat_interleave(block, dim=2)[:, :, :P]
    o, l, tol, tol_l = ref.attention(q.to(F64), k, v, ks.to(F64), vs.to(F64), vis, step)
    err, errl = (out.cpu().to(F64) - o).abs(), (lse.cpu().to(F64) - l).abs()
    rms = ((out.cpu().to(F64) - o).norm() / o.norm()).item()
    print(f"[{what or (B, Hq, H, P, S, block)}] out err/bound {(err / tol).max():.3f} rel {rms:.2e}; "
          f"lse err/bound {(errl / tol_l).max():.3f} max {errl.max():.2e}")
    assert (err <= tol).all(), (err / tol).max()
    assert (errl <= tol_l).all(), (errl / tol_l).max()
    return out, lse


@pytest.mark.parametrize("B,Hq,H,P,S,valid", [
    (1, 8, 4, 576, 1, [512]),          # one token
    (1, 8, 4, 0, 10, None),            # no prefix at all
    (1, 8, 4, 1, 1, None),
    (2, 8, 4, 63, 7, [0, 63]),         # a sample without prefix rows
    (2, 8, 4, 64, 50, [1, 64]),
    (2, 4, 4, 65, 65, [65, 64]),       # one head a group, two suffix tiles
    (1, 4, 4, 127, 128, None),
    (2, 8, 2, 128, 32, [128, 127]),    # four heads a group
    (2, 8, 1, 129, 16, [129, 100]),
    (3, 2, 1, 300, 64, [256, 257, 300]),
    (1, 8, 4, 1024, 50, [900]),        # the base model's chunk
    (1, 8, 4, 2048, 50, [1900]),
    (5, 8, 4, 1000, 33, [1000, 1, 500, 128, 999]),
])
@pytest.mark.parametrize("block", [16, 64])
def test_attention(B, Hq, H, P, S, valid, block):
    check_attention(gen(P + 3 * S + block), B, Hq, H, P, S, block, valid)


@pytest.mark.parametrize("block", [32, 128])
def test_attention_other_blocks(block):
    check_attention(gen(block), 2, 8, 4, 700, 20, block, [700, 333])


def test_attention_batch_with_mask():
    g = gen(77)
    mask = (torch.rand(12, 1024, generator=g) >= 0.1).to(torch.uint8)
    valid = torch.randint(576, 1025, (12,), generator=g).tolist()
    check_attention(g, 12, 8, 4, 1024, 50, 64, valid, mask)


@pytest.mark.parametrize("hide", ["all", "first tile", "all but one", "every other"])
def test_attention_masks(hide):
    g = gen(6)
    mask = torch.ones(2, 333, dtype=torch.uint8)
    if hide == "all":
        mask[:] = 0
    elif hide == "first tile":
        mask[:, :140] = 0
    elif hide == "all but one":
        mask[:] = 0
        mask[0, 331] = mask[1, 0] = 255                    # any nonzero byte shows
    else:
        mask[:, ::2] = 0
    check_attention(g, 2, 8, 4, 333, 9, 16, [333, 200], mask)


def test_attention_long_prefix():
    check_attention(gen(8), 1, 8, 4, 30016, 10, 16, [29987])


def test_attention_scales_that_are_no_powers_of_two():
    g = gen(9)
    check_attention(g, 2, 8, 4, 500, 25, 32, [500, 499], c=make_cache(g, 2, 4, 500, 32, 6.0, pow2=False))


def test_attention_values_of_very_different_size():
    # blocks of tiny values next to large ones, tiny ones holding the weight
    g = gen(10)
    c = make_cache(g, 1, 4, 256, 16)
    c.v_scale[:, :, ::2] = 2.0 ** -40
    c.v_scale[:, :, 1::4] = 2.0 ** 20
    check_attention(g, 1, 8, 4, 256, 20, 16, c=c)
    c.v_scale[:] = 2.0 ** -64                              # the whole cache far below the suffix's values
    check_attention(g, 1, 8, 4, 256, 20, 16, c=c)
    c.k_scale[:] = 2.0 ** -64
    check_attention(g, 1, 8, 4, 256, 20, 16, c=c)


def test_attention_peaked_and_growing_logits():
    # later keys win by ever larger margins: every tile rescales what came before
    g = gen(11)
    c = make_cache(g, 1, 4, 640, 16, spread=0.0)
    c.k_scale.mul_(torch.linspace(0.25, 24.0, 40)[None, None])
    check_attention(g, 1, 8, 4, 640, 50, 16, c=c, what="growing")
    c.k_scale.copy_(c.k_scale.flip(2).contiguous())
    check_attention(g, 1, 8, 4, 640, 50, 16, c=c, what="falling")


def test_attention_queries_of_very_different_size():
    g = gen(12)
    q = rand(g, 1, 8, 30, 256) * torch.exp2(torch.randint(-30, 3, (1, 8, 30, 1), generator=g).float())
    q[0, 0, 3] = 0.0
    q[0, 1, 4, 7] = 200.0                                  # one element far above the rest of its row
    check_attention(g, 1, 8, 4, 300, 30, 64, q=q.to(BF))


@pytest.mark.parametrize("splits", [1, 2, 3, 4, 7, 8, 16])
def test_attention_forced_plans(splits):
    try:
        assert bd.dm05_set_split_override(splits) == 0
        assert bd.dm05_suffix_attn_kv8_plan(2, 8, 4, 900, 50, 256)[1] == splits
        check_attention(gen(splits), 2, 8, 4, 900, 50, 64, [900, 130])
        check_attention(gen(splits), 1, 8, 4, 70, 11, 16, [3])   # more splits than tiles
    finally:
        bd.dm05_set_split_override(0)


def test_attention_never_uses_hidden_rows():
    """NaN codes in hidden and out-of-range rows, NaN scales in blocks without a visible row."""
    g = gen(13)
    mask = torch.ones(2, 400, dtype=torch.uint8)
    mask[:, 40:80] = 0
    mask[1, 128:256] = 0
    valid = [300, 333]
    a = dict(g=gen(14), B=2, Hq=8, H=4, P=400, S=12, block=32, valid=valid, mask=mask)
    c = make_cache(g, 2, 4, 400, 32)
    check_attention(c=c, **a)
    vis = ref.visible(valid, mask, 2, 400)
    bad = bd.Kv8Cache(c.k.clone(), c.v.clone(), c.k_scale.clone(), c.v_scale.clone(), 32)
    for x in (bad.k, bad.v):
        x.view(torch.uint8).masked_fill_(~vis[:, None, :, None], 0x7F)
    blocks = torch.nn.functional.pad(vis, (0, 16)).view(2, 13, 32).any(-1)
    for s in (bad.k_scale, bad.v_scale):
        s.masked_fill_(~blocks[:, None], float("nan"))
    q = rand(gen(15), 2, 8, 12, 256).to(BF).cuda()
    ks = rand(gen(16), 2, 4, 12, 256).to(BF).cuda()
    r1 = bd.suffix_attn_kv8(q, on_gpu(c), ks, ks, cu(i32(valid)), mask.cuda())
    r2 = bd.suffix_attn_kv8(q, on_gpu(bad), ks, ks, cu(i32(valid)), mask.cuda())
    assert torch.equal(r1[0], r2[0]) and torch.equal(r1[1], r2[1])


def test_attention_matches_the_bf16_call():
    """A cache whose values bf16 holds exactly: suffix_attn on the dequantised cache is the same sum."""
    g = gen(17)
    c = make_cache(g, 2, 4, 500, 64)
    k, v = (ref.dequant(x.to(F64), s.to(F64), 64).to(BF) for x, s in ((c.k, c.k_scale), (c.v, c.v_scale)))
    q, ks, vs = rand(g, 2, 8, 50, 256).to(BF), rand(g, 2, 4, 50, 256).to(BF), rand(g, 2, 4, 50, 256).to(BF)
    valid = i32([500, 411]).cuda()
    o8, l8 = bd.suffix_attn_kv8(q.cuda(), on_gpu(c), ks.cuda(), vs.cuda(), valid)
    o, l = bd.suffix_attn(q.cuda(), k.cuda(), v.cuda(), ks.cuda(), vs.cuda(), valid)
    # two bf16 roundings of nearly the same value and of the weights behind it
    assert (o8.double() - o.double()).abs().max() <= 4 * 2.0 ** -8 * v.double().abs().max()
    assert (l8 - l).abs().max() <= 1e-3


def test_attention_outputs_only_and_clamp_flag():
    g = gen(18)
    c = on_gpu(make_cache(g, 1, 4, 100, 16))
    q, ks = rand(g, 1, 8, 5, 256).to(BF).cuda(), rand(g, 1, 4, 5, 256).to(BF).cuda()
    big = torch.full((3, 8, 5, 256), 7.0, dtype=BF, device="cuda")
    lse = torch.full((3, 8, 5), 7.0, device="cuda")
    o, l = bd.suffix_attn_kv8(q, c, ks, ks, i32([500]).cuda(), out=big[1:2], lse=lse[1:2])
    assert (big[0] == 7).all() and (big[2] == 7).all() and (lse[0] == 7).all() and (lse[2] == 7).all()
    rc, word = bd.dm05_get_error_word(None)
    assert rc == 0 and word == bd.DM05_EW_VALID_LEN_CLAMPED
    full, _ = bd.suffix_attn_kv8(q, c, ks, ks, want_lse=False)
    assert _ is None and torch.equal(full, o)
    none, _ = bd.suffix_attn_kv8(q, c, ks, ks, i32([-3]).cuda())
    assert bd.dm05_get_error_word(None)[1] == bd.DM05_EW_VALID_LEN_CLAMPED
    empty, _ = bd.suffix_attn_kv8(q, c, ks, ks, i32([0]).cuda())
    assert torch.equal(none, empty)


@pytest.mark.parametrize("S,splits", [(1, 1), (4, 2), (10, 1), (16, 2), (17, 1), (32, 1), (32, 2), (33, 1), (50, 2), (60, 2)])
@pytest.mark.parametrize("masked", [False, True])
def test_attention_few_and_many_rows_on_long_runs(S, splits, masked):
    """Query rows laid once, twice and four times over the MMA's rows, and in blocks: every CTA walks several tiles."""
    g = gen(S * 8 + splits)
    mask = (torch.rand(2, 900, generator=g) >= 0.2).to(torch.uint8) if masked else None
    if masked:
        mask[0, 128:300] = 0                               # a whole tile hidden
        mask[1] = 0
    try:
        assert bd.dm05_set_split_override(splits) == 0
        check_attention(g, 2, 8, 4, 900, S, 32, [900, 130], mask)
        c = make_cache(g, 1, 2, 1030, 16, spread=0.0)      # growing logits, one head a group
        c.k_scale.mul_(torch.linspace(0.25, 24.0, 65)[None, None])
        check_attention(g, 1, 2, 2, 1030, S, 16, c=c)
        c.k_scale.copy_(c.k_scale.flip(2).contiguous())
        c.v_scale[:, :, ::3] = 2.0 ** -30
        check_attention(g, 1, 2, 2, 1030, S, 16, [1021], c=c)
    finally:
        bd.dm05_set_split_override(0)


@pytest.mark.parametrize("S", [9, 20, 50])
def test_attention_rows_do_not_touch_each_other(S):
    """A query row of NaN or infinity spoils its own output only."""
    g = gen(S)
    c = make_cache(g, 1, 4, 900, 16)
    q = rand(g, 1, 8, S, 256).to(BF)
    ks, vs = rand(g, 1, 4, S, 256).to(BF), rand(g, 1, 4, S, 256).to(BF)
    bad = q.clone()
    bad[0, 1, 3, 100], bad[0, 6, 7] = float("nan"), float("inf")
    keep = torch.ones(8, S, dtype=torch.bool)
    keep[1, 3] = keep[6, 7] = False
    out, lse = bd.suffix_attn_kv8(bad.cuda(), on_gpu(c), ks.cuda(), vs.cuda())
    k, v = (ref.dequant(x.to(F64), s.to(F64), 16) for x, s in ((c.k, c.k_scale), (c.v, c.v_scale)))
    step = c.v_scale.to(F64).repeat_interleave(16, dim=2)[:, :, :900]
    o, l, tol, tol_l = ref.attention(q.to(F64), k, v, ks.to(F64), vs.to(F64), torch.ones(1, 900, dtype=torch.bool), step)
    assert (out[0].cpu().to(F64) - o[0]).abs()[keep].le(tol[0][keep]).all()
    assert (lse[0].cpu().to(F64) - l[0]).abs()[keep].le(tol_l[0][keep]).all()
    assert torch.isnan(out[0].cpu()[~keep].float()).all()


def test_attention_workspace_of_the_caller():
    g = gen(19)
    c = on_gpu(make_cache(g, 1, 4, 3000, 64))
    q, ks = rand(g, 1, 8, 50, 256).to(BF).cuda(), rand(g, 1, 4, 50, 256).to(BF).cuda()
    rc, splits, rows, nbytes = bd.dm05_suffix_attn_kv8_plan(1, 8, 4, 3000, 50, 256)
    assert rc == 0 and splits > 1 and rows == 128 and nbytes > 0
    want = bd.suffix_attn_kv8(q, c, ks, ks)
    ws = torch.full((nbytes,), 0xFF, dtype=torch.uint8, device="cuda")
    got = bd.suffix_attn_kv8(q, c, ks, ks, workspace=ws)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    with pytest.raises(bd.Dm05Error):
        bd.suffix_attn_kv8(q, c, ks, ks, workspace=ws[:-16])


@pytest.mark.parametrize("B,P,S", [(1, 576, 1), (1, 200, 50), (2, 576, 50), (1, 1024, 50), (1, 1900, 64), (3, 300, 7),
                                   (2, 1024, 32), (4, 1024, 1), (1, 2500, 12)])
def test_attention_splits_joined_in_the_kernel_and_behind_it(B, P, S):
    """Clusters while they all run at once, a second kernel otherwise: with masks that leave splits without a key."""
    g = gen(B * P + S)
    check_attention(g, B, 8, 4, P, S, 16, [P] + [P // 3] * (B - 1))
    mask = torch.zeros(B, P, dtype=torch.uint8)
    mask[:, :3] = 1
    mask[0, P // 2] = 1
    check_attention(g, B, 8, 4, P, S, 16, [P] + [0] * (B - 1), mask)


def test_many_heads_of_one_row():
    """B * Hkv at its limit, and a batch whose heads fill several waves."""
    g = gen(20)
    B = 65535
    c = make_cache(g, B, 1, 1, 16)
    q, ks, vs = (rand(g, B, 1, 1, 256).to(BF) for _ in range(3))
    at = torch.tensor([0, 1, 147, 148, 32768, 65534])
    out, lse = bd.suffix_attn_kv8(q.cuda(), on_gpu(c), ks.cuda(), vs.cuda())
    m = bd.prefix_attn_mass_kv8(q.cuda(), c.k.cuda(), c.k_scale.cuda(), 16, lse)
    k, v = (ref.dequant(x[at].to(F64), s[at].to(F64), 16) for x, s in ((c.k, c.k_scale), (c.v, c.v_scale)))
    vis = torch.ones(len(at), 1, dtype=torch.bool)
    o, l, tol, tol_l = ref.attention(q[at].to(F64), k, v, ks[at].to(F64), vs[at].to(F64), vis, c.v_scale[at].to(F64))
    assert ((out.cpu()[at].to(F64) - o).abs() <= tol).all() and ((lse.cpu()[at].to(F64) - l).abs() <= tol_l).all()
    want, tol = ref.mass(q[at].to(F64), k, lse.cpu()[at], vis, None)
    assert ((m.cpu()[at].to(F64) - want).abs() <= tol).all()
    e = bd.prefix_evict_kv8(on_gpu(c), m, 1)
    assert torch.equal(e.mass, m) and (e.positions == 0).all() and (e.valid_len == 1).all()
    assert same(e.cache.k.float() * e.cache.k_scale[..., None], c.k.float() * c.k_scale[..., None])
    x = c.k.float().to(BF).cuda()
    assert same(bd.kv8_quantize(x, x, 16).k.float()[65534], ref.quantize(
        x[65534:].cpu().to(F64), None, 16, 0, torch.zeros(1, 1, 1, 256, dtype=F64), torch.ones(1, 1, 1, dtype=F64))[0][0])
    check_attention(g, 40, 8, 4, 140, 10, 16)              # 160 heads: more than one wave


def test_offsets_past_32_bits():
    """Caches whose last rows lie past 2^31 codes and 2^32 bytes."""
    g = gen(25)
    B, H, P, S, n = 2, 4, 1_200_000, 10, 320               # P is a multiple of the block, the last n rows are seen
    tail = rand(g, 2, 1, H, n, 256).to(BF)
    k, v = (torch.zeros(B, H, P, 256, dtype=BF, device="cuda") for _ in range(2))
    k[1, :, -n:], v[1, :, -n:] = tail[0, 0].cuda(), tail[1, 0].cuda()
    mask = torch.zeros(B, P, dtype=torch.uint8, device="cuda")
    mask[1, -n:] = 1
    mask[0, :5] = 1
    c = bd.kv8_quantize(k, v, 64)
    small = bd.kv8_quantize(tail[0].cuda(), tail[1].cuda(), 64)
    for a, b in zip(c[:4], small[:4]):
        assert torch.equal(a[1:, :, -b.shape[2]:].view(torch.uint8), b.view(torch.uint8))
    q, ks, vs = rand(g, B, 8, S, 256).to(BF), rand(g, B, H, S, 256).to(BF), rand(g, B, H, S, 256).to(BF)
    out, lse = bd.suffix_attn_kv8(q.cuda(), c, ks.cuda(), vs.cuda(), prefix_mask=mask)
    kd, vd = (ref.dequant(x.cpu().to(F64), s.cpu().to(F64), 64) for x, s in ((small.k, small.k_scale), (small.v, small.v_scale)))
    vis = torch.ones(1, n, dtype=torch.bool)
    d = lambda t: t[1:].cpu().to(F64)  # noqa: E731
    o, l, tol, tol_l = ref.attention(d(q), kd, vd, d(ks), d(vs), vis,
                                     small.v_scale.cpu().to(F64).repeat_interleave(64, dim=2))
    assert ((d(out) - o).abs() <= tol).all() and ((d(lse) - l).abs() <= tol_l).all()
    for m, keys in ((bd.prefix_attn_mass_kv8(q.cuda(), c.k, c.k_scale, 64, lse, prefix_mask=mask), kd),
                    (bd.prefix_attn_mass(q.cuda(), k, lse, prefix_mask=mask), tail[0].to(F64))):
        want, tol = ref.mass(d(q), keys, lse[1:].cpu(), vis, None)
        assert ((d(m)[:, :, -n:] - want).abs() <= tol).all()
        assert (m[1, :, :-n] == 0).all() and (m[0, :, 5:] == 0).all()
    e = bd.prefix_evict(k, v, m, 100, prefix_mask=mask)
    e8 = bd.prefix_evict_kv8(c, m, 100, prefix_mask=mask)
    assert e.valid_len.tolist() == [5, 100] and torch.equal(e8.positions, e.positions)
    for h in range(H):
        order = ref.evict_order(m[1, h, -n:].tolist(), [True] * n, n, 100, 0, 0)
        assert (e.positions[1, h].cpu() - (P - n)).tolist() == order
        assert torch.equal(e.k[1, h].cpu(), tail[0, 0, h, order]) and torch.equal(e.v[1, h].cpu(), tail[1, 0, h, order])
        assert same(e8.cache.v[1, h].float() * e8.cache.v_scale[1, h].repeat_interleave(64)[:100, None],
                    ref.dequant(*ref.quantize(vd[:, h:h + 1, order], None, 64, 0, torch.zeros(1, 1, 100, 256, dtype=F64),
                                              torch.ones(1, 1, 2, dtype=F64)), 64)[0, 0])


# ------------------------------------------------------------------ mass

def check_mass(g, B, Hq, H, P, S, block, valid=None, mask=None, before=None, lse=None, q=None, k=None):
    q = rand(g, B, Hq, S, 256).to(BF) if q is None else q
    if lse is None:
        lse = 4 + rand(g, B, Hq, S)
    if block:
        c = make_cache(g, B, H, P, block)
        kd = ref.dequant(c.k.to(F64), c.k_scale.to(F64), block)
        got = bd.prefix_attn_mass_kv8(q.cuda(), c.k.cuda(), c.k_scale.cuda(), block, lse.cuda(), cu(i32(valid)),
                                      cu(mask), cu(before))
    else:
        k = rand(g, B, H, P, 256).to(BF) if k is None else k
        kd = k.to(F64)
        got = bd.prefix_attn_mass(q.cuda(), k.cuda(), lse.cuda(), cu(i32(valid)), cu(mask), cu(before))
    want, tol = ref.mass(q.to(F64), kd, lse, ref.visible(valid, mask, B, P), before)
    err = (got.cpu().to(F64) - want).abs()
    print(f"mass err/bound {(err / tol.clamp(min=1e-300)).max():.3f} rel {(err.norm() / want.norm()).item():.2e}")
    assert (err <= tol).all(), (err - tol).max()
    return got


@pytest.mark.parametrize("block", [0, 16, 64, 128])
@pytest.mark.parametrize("B,Hq,H,P,S,valid", [
    (1, 8, 4, 576, 1, [512]), (1, 8, 4, 1, 1, None), (2, 8, 4, 63, 7, [0, 63]), (2, 4, 4, 129, 128, [129, 128]),
    (2, 8, 2, 128, 32, [127, 1]), (1, 8, 4, 2048, 50, [1900]), (3, 2, 1, 300, 64, [256, 257, 300])])
def test_mass(block, B, Hq, H, P, S, valid):
    check_mass(gen(P + S + block), B, Hq, H, P, S, block, valid)


@pytest.mark.parametrize("block", [0, 32])
def test_mass_added_masked_and_in_place(block):
    g = gen(21)
    mask = (torch.rand(6, 500, generator=g) >= 0.3).to(torch.uint8)
    mask[2] = 0
    before = torch.rand(6, 4, 500, generator=g) * 10
    valid = [500, 0, 500, 499, 33, 256]
    check_mass(gen(22), 6, 8, 4, 500, 50, block, valid, mask, before)
    q, lse = rand(g, 6, 8, 50, 256).to(BF).cuda(), (4 + rand(g, 6, 8, 50)).cuda()
    c = on_gpu(make_cache(g, 6, 4, 500, block or 32))
    k = rand(g, 6, 4, 500, 256).to(BF).cuda()

    def call(**kw):
        a = dict(prefix_valid_len=i32(valid).cuda(), prefix_mask=mask.cuda(), **kw)
        return bd.prefix_attn_mass_kv8(q, c.k, c.k_scale, block, lse, **a) if block else bd.prefix_attn_mass(q, k, lse, **a)
    want = call(mass_in=before.cuda())
    acc = before.cuda().clone()
    got = call(mass_in=acc, mass=acc)
    assert got is acc and torch.equal(acc, want)


@pytest.mark.parametrize("block", [0, 64])
def test_mass_rows_without_weight(block):
    g = gen(23)
    lse = 3 + rand(g, 1, 8, 20)
    lse[0, 2] = float("-inf")                              # rows that saw nothing
    lse[0, 3, 5] = float("inf")
    check_mass(g, 1, 8, 4, 200, 20, block, lse=lse)


def test_mass_never_uses_hidden_rows():
    g = gen(24)
    k = rand(g, 1, 4, 300, 256).to(BF)
    q, lse = rand(g, 1, 8, 9, 256).to(BF).cuda(), (4 + rand(g, 1, 8, 9)).cuda()
    mask = torch.ones(1, 300, dtype=torch.uint8)
    mask[0, 50:90] = 0
    a = bd.prefix_attn_mass(q, k.cuda(), lse, i32([250]).cuda(), mask.cuda())
    k[:, :, 50:90], k[:, :, 250:] = float("nan"), float("inf")
    b = bd.prefix_attn_mass(q, k.cuda(), lse, i32([250]).cuda(), mask.cuda())
    assert torch.equal(a, b) and (b[0, :, 50:90] == 0).all() and (b[0, :, 250:] == 0).all()


# ------------------------------------------------------------------ eviction

def check_evict(g, B, H, P, bucket, block, keep, first=0, last=0, valid=None, mask=None, m=None, c=None):
    m = torch.rand(B, H, P, generator=g) if m is None else m
    vis = ref.visible(valid, mask, B, P)
    ns = ref.lengths(valid, B, P)
    args = dict(n_keep=keep, n_first=first, n_last=last, prefix_valid_len=cu(i32(valid)), prefix_mask=cu(mask))
    pos0 = torch.full((B, H, bucket), 77, dtype=torch.int32, device="cuda")
    if block:
        c = make_cache(g, B, H, P, block) if c is None else c
        old = torch.full((B, H, bucket, 256), 0.75).to(F8)
        s0 = torch.full((B, H, -(-bucket // block)), 5.0)
        out = bd.Kv8Cache(old.cuda(), old.cuda(), s0.cuda(), s0.cuda(), block)
        e = bd.prefix_evict_kv8(on_gpu(c), m.cuda(), out=out, positions=pos0, **args)
        dense = [ref.dequant(x.to(F64), s.to(F64), block) for x, s in ((c.k, c.k_scale), (c.v, c.v_scale))]
        got = [(out.k, out.k_scale), (out.v, out.v_scale)]
    else:
        k, v = rand(g, B, H, P, 256).to(BF), rand(g, B, H, P, 256).to(BF)
        old = torch.full((B, H, bucket, 256), 0.75, dtype=BF)
        e = bd.prefix_evict(k.cuda(), v.cuda(), m.cuda(), k_out=old.cuda(), v_out=old.cuda(), positions=pos0, **args)
        dense, got = [k.to(F64), v.to(F64)], [(e.k, None), (e.v, None)]
    want = [old.to(F64), old.to(F64)]
    want_s = [s0.to(F64), s0.to(F64)] if block else None
    for b in range(B):
        for h in range(H):
            order = ref.evict_order(m[b, h].tolist(), vis[b].tolist(), ns[b], keep, first, last)
            n = len(order)
            assert int(e.valid_len[b]) == n
            assert e.positions[b, h].tolist() == order + [-1] * (bucket - n)
            assert same(e.mass[b, h], torch.cat([m[b, h, order], torch.zeros(bucket - n)]))
            for i in range(2):
                rows = dense[i][b:b + 1, h:h + 1, order]
                if block and n:
                    codes, scales = want[i][b:b + 1, h:h + 1, :n], want_s[i][b:b + 1, h:h + 1]
                    ref.quantize(rows, None, block, 0, codes, scales)
                elif n:
                    want[i][b, h, :n] = rows[0, 0]
    for i in range(2):
        assert same(got[i][0], want[i])
        if block:
            assert same(got[i][1], want_s[i])
    return e


@pytest.mark.parametrize("block", [0, 16, 64, 128])
@pytest.mark.parametrize("P,bucket,keep,first,last,valid", [
    (1, 1, 1, 0, 0, None), (1, 3, 0, 0, 0, None), (40, 40, 40, 0, 0, [40, 0]), (200, 64, 50, 4, 10, [200, 30]),
    (513, 200, 129, 0, 0, [513, 512]), (33, 100, 90, 40, 40, [33, 7]), (1000, 576, 512, 16, 64, [900, 700]), (777, 300, 17, 100, 0, [777, 5])])
def test_evict(block, P, bucket, keep, first, last, valid):
    check_evict(gen(P + keep + block), 1 if valid is None else 2, 2, P, bucket, block, keep, first, last, valid)


@pytest.mark.parametrize("block", [0, 32])
def test_evict_masked(block):
    g = gen(31)
    mask = (torch.rand(3, 600, generator=g) >= 0.4).to(torch.uint8)
    mask[1] = 0
    check_evict(g, 3, 2, 600, 256, block, 250, 3, 20, [600, 600, 300], mask)


@pytest.mark.parametrize("kind", ["all equal", "few values", "signs", "nan", "infinite", "close"])
def test_evict_ties_and_odd_weights(kind):
    g = gen(32)
    m = torch.rand(2, 2, 700, generator=g)
    if kind == "all equal":
        m[:] = 0.25
    elif kind == "few values":
        m = torch.randint(0, 4, (2, 2, 700), generator=g).float()
    elif kind == "signs":
        m = torch.where(torch.rand(2, 2, 700, generator=g) < 0.5, torch.zeros_like(m), -torch.zeros_like(m))
        m[0, 0, ::3] = -1.0
    elif kind == "nan":
        m[:, :, ::2] = float("nan")
        m[0, 0, 1::2] = -float("inf")
    elif kind == "infinite":
        m[:, :, 5::7] = float("inf")
        m[:, :, 3::7] = -float("inf")
    else:
        m = 1.0 + torch.randint(0, 50, (2, 2, 700), generator=g).float() * 2.0 ** -23
    check_evict(g, 2, 2, 700, 400, 0, 390, 0, 0, [700, 655], m=m)
    check_evict(g, 2, 2, 700, 400, 0, 100, 2, 3, [700, 655], m=m)


@pytest.mark.parametrize("P", [1023, 1024, 1025, 2048, 2049, 4096, 4097, 8192, 8193, 10000])
@pytest.mark.parametrize("block", [0, 16])
def test_evict_lengths(P, block):
    g = gen(P)
    m = torch.randint(0, 40, (2, 1, P), generator=g).float()   # many equal weights, some of them cut
    check_evict(g, 2, 1, P, 700, block, 650, 3, 5, [P, P - 7], m=m)
    mask = (torch.rand(2, P, generator=g) >= 0.5).to(torch.uint8)
    check_evict(g, 2, 1, P, P, block, P, 0, 0, [P, 900], mask, m=torch.rand(2, 1, P, generator=g))


@pytest.mark.parametrize("block", [0, 16, 128])
@pytest.mark.parametrize("B,H", [(5, 7), (37, 4), (149, 1), (75, 4)])
def test_evict_many_heads(B, H, block):
    g = gen(B)
    valid = torch.randint(0, 331, (B,), generator=g).tolist()
    check_evict(g, B, H, 330, 200, block, 190, 2, 9, valid)


def test_evict_long_prefix():
    g = gen(33)
    check_evict(g, 1, 1, 70001, 5000, 0, 4999, 8, 8, [69990])


def test_evict_keeps_nan_codes_and_scales_that_are_no_powers_of_two():
    g = gen(34)
    c = make_cache(g, 1, 2, 300, 16, 8.0, pow2=False)
    c.k.view(torch.uint8)[0, 0, 5, 7] = 0x7F
    c.v.view(torch.uint8)[0, 1, 9] = 0x7F
    # the products scale * code are rounded to fp32 before the new scale sees them
    k = (c.k.float() * c.k_scale.repeat_interleave(16, 2)[:, :, :300, None])
    v = (c.v.float() * c.v_scale.repeat_interleave(16, 2)[:, :, :300, None])
    m = torch.rand(1, 2, 300, generator=g)
    m[:, :, 5] = m[:, :, 9] = 9.0
    e = bd.prefix_evict_kv8(on_gpu(c), m.cuda(), 100, bucket=128)
    for h in range(2):
        at = e.positions[0, h, :100].cpu().long()
        for dense, codes, scale in ((k, e.cache.k, e.cache.k_scale), (v, e.cache.v, e.cache.v_scale)):
            want, ws = ref.quantize(dense[:, h:h + 1, at].to(F64), None, 16, 0, torch.zeros(1, 1, 100, 256, dtype=F64),
                                    torch.ones(1, 1, 7, dtype=F64))
            assert same(scale[:, h:h + 1, :7], ws) and same(codes[:, h:h + 1, :100], want)
    assert torch.isnan(e.cache.k.float()).any() and torch.isnan(e.cache.v.float()).any()


# ------------------------------------------------------------------ together

def chain(q, k, v, ks, vs, valid, steps=2, keep=200, bucket=256, stream=None):
    """A prefix quantised once, two denoising steps that collect weight, the
    cache cut to the positions that received most, one more step."""
    c = bd.kv8_quantize(k, v, 32, valid, stream=stream)
    m = None
    for i in range(steps):
        o, l = bd.suffix_attn_kv8(q[i], c, ks[i], vs[i], valid, stream=stream)
        m = bd.prefix_attn_mass_kv8(q[i], c.k, c.k_scale, 32, l, valid, mass_in=m, stream=stream)
    e = bd.prefix_evict_kv8(c, m, keep, 4, 16, valid, bucket=bucket, stream=stream)
    o, l = bd.suffix_attn_kv8(q[steps], e.cache, ks[steps], vs[steps], e.valid_len, stream=stream)
    return o, l, m, e


def chain_inputs(seed, B=2, P=700, S=30):
    g = gen(seed)
    q = [rand(g, B, 8, S, 256).to(BF).cuda() for _ in range(3)]
    ks = [rand(g, B, 4, S, 256).to(BF).cuda() for _ in range(3)]
    vs = [rand(g, B, 4, S, 256).to(BF).cuda() for _ in range(3)]
    k, v = rand(g, B, 4, P, 256).to(BF).cuda(), rand(g, B, 4, P, 256).to(BF).cuda()
    return q, k, v, ks, vs, i32([P, P - 111][:B]).cuda()


def test_chain_against_plain_forms():
    q, k, v, ks, vs, valid = chain_inputs(41)
    o, l, m, e = chain(q, k, v, ks, vs, valid)
    d = lambda t: t.cpu().to(F64)  # noqa: E731
    n = valid.tolist()
    B, P = 2, 700
    z = torch.zeros(B, 4, P, 256, dtype=F64)
    kc, kscale = ref.quantize(d(k), n, 32, 0, z.clone(), torch.ones(B, 4, 22, dtype=F64))
    vc, vscale = ref.quantize(d(v), n, 32, 0, z.clone(), torch.ones(B, 4, 22, dtype=F64))
    kd, vd = ref.dequant(kc, kscale, 32), ref.dequant(vc, vscale, 32)
    vis = ref.visible(n, None, B, P)
    mass, tol = None, 0
    for i in range(2):
        _, lse, _, tl = ref.attention(d(q[i]), kd, vd, d(ks[i]), d(vs[i]), vis)
        mass, t = ref.mass(d(q[i]), kd, lse, vis, mass)
        tol = tol + t + mass * 2 * tl.amax()               # the call's lse is off by its own bound
    assert ((m.cpu().to(F64) - mass).abs() <= tol).all()
    kept_k, kept_v = torch.zeros(B, 4, 200, 256, dtype=F64), torch.zeros(B, 4, 200, 256, dtype=F64)
    step = torch.zeros(B, 4, 200, dtype=F64)
    for b in range(B):
        for h in range(4):
            at = e.positions[b, h, :200].cpu().long()
            assert at.tolist() == ref.evict_order(m[b, h].tolist(), vis[b].tolist(), n[b], 200, 4, 16)
            for src, dst, st in ((kd, kept_k, None), (vd, kept_v, step)):
                c, s = ref.quantize(src[b:b + 1, h:h + 1, at], None, 32, 0, torch.zeros(1, 1, 200, 256, dtype=F64),
                                    torch.ones(1, 1, 7, dtype=F64))
                dst[b, h] = ref.dequant(c, s, 32)[0, 0]
                if st is not None:
                    st[b, h] = s.repeat_interleave(32, 2)[0, 0, :200]
    ro, rl, to, tl = ref.attention(d(q[2]), kept_k, kept_v, d(ks[2]), d(vs[2]), torch.ones(B, 200, dtype=torch.bool), step)
    assert ((o.cpu().to(F64) - ro).abs() <= to).all() and ((l.cpu().to(F64) - rl).abs() <= tl).all()


def test_evicted_bf16_cache_serves_the_bf16_call():
    q, k, v, ks, vs, valid = chain_inputs(42)
    _, l = bd.suffix_attn(q[0], k, v, ks[0], vs[0], valid)
    m = bd.prefix_attn_mass(q[0], k, l, valid)
    e = bd.prefix_evict(k, v, m, 150, prefix_valid_len=valid, bucket=192)
    o, l2 = bd.suffix_attn(q[1], e.k, e.v, ks[1], vs[1], e.valid_len)
    at = e.positions[:, :, :150].cpu().long()[..., None].expand(2, 4, 150, 256)
    d = lambda t: t.cpu().to(F64)  # noqa: E731
    ro, rl, to, tl = ref.attention(d(q[1]), d(k).gather(2, at), d(v).gather(2, at), d(ks[1]), d(vs[1]),
                                   torch.ones(2, 150, dtype=torch.bool))
    assert ((d(o) - ro).abs() <= to + 2.0 ** -8 * d(v).abs().max()).all()
    assert ((d(l2) - rl).abs() <= tl + 1e-4).all()


def flat(r):
    o, l, m, e = r
    return [o, l, m, e.cache.k.view(torch.uint8), e.cache.v.view(torch.uint8), e.cache.k_scale, e.cache.v_scale,
            e.mass, e.positions, e.valid_len]


def test_chain_repeats_bit_for_bit_and_on_other_streams():
    a = chain_inputs(43)
    want = flat(chain(*a))
    for _ in range(3):
        assert all(torch.equal(x, y) for x, y in zip(flat(chain(*a)), want))
    torch.cuda.synchronize()
    side = [torch.cuda.Stream() for _ in range(3)]
    got = [flat(chain(*a, stream=s)) for s in side for _ in range(2)]   # calls in flight at once
    handle = flat(chain(*a, stream=side[0].cuda_stream))
    torch.cuda.synchronize()
    for r in got + [handle]:
        assert all(torch.equal(x, y) for x, y in zip(r, want))


def test_two_captured_chains_replay_at_once():
    ins = [chain_inputs(44), chain_inputs(45)]
    want = [flat(chain(*a)) for a in ins]
    torch.cuda.synchronize()
    graphs, outs, streams = [], [], [torch.cuda.Stream() for _ in range(2)]
    for a in ins:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(flat(chain(*a)))
        graphs.append(g)
    for t in [x for r in outs for x in r]:
        t.zero_()
    torch.cuda.synchronize()
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for r, w in zip(outs, want):
        assert all(torch.equal(x, y) for x, y in zip(r, w))
    # new inputs in the captured buffers
    ins[0][1].copy_(ins[1][1])
    fresh = flat(chain(*ins[0]))
    graphs[0].replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(outs[0], fresh))


FIRST_IN_CAPTURE = """
import sys, torch
sys.path.insert(0, sys.argv[1])
import test_prefix_cache_gpu as t
a, big = t.chain_inputs(47), t.chain_inputs(48, B=2, P=3000, S=10)
t.bd.kv8_quantize(a[1], a[2], 32)                          # only the error word exists before the capture
torch.cuda.synchronize()
g, out = torch.cuda.CUDAGraph(), []
with torch.cuda.graph(g):
    for x in (a, big):
        out.append(t.flat(t.chain(*x)))
for _ in range(2):
    g.replay()
torch.cuda.synchronize()
for x, got in zip((a, big), out):
    assert all(torch.equal(p, q) for p, q in zip(got, t.flat(t.chain(*x))))
assert t.bd.dm05_get_error_word(None) == (0, 0)
print("same")
"""


def test_first_calls_inside_a_capture():
    here = os.path.dirname(os.path.abspath(__file__))
    r = subprocess.run([sys.executable, "-c", FIRST_IN_CAPTURE, here], cwd=os.path.dirname(here), capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "same", r.stderr[-2000:]


def test_calls_from_several_threads():
    """Threads with streams of their own, the first calls of all at the same time."""
    ins = [chain_inputs(50 + i, P=400 + 300 * i) for i in range(4)]
    torch.cuda.synchronize()
    got = [None] * 4

    def work(i):
        s = torch.cuda.Stream()
        for _ in range(5):
            got[i] = flat(chain(*ins[i], stream=s))
        s.synchronize()
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for a, r in zip(ins, got):
        assert all(torch.equal(x, y) for x, y in zip(r, flat(chain(*a))))


def test_front_end_refuses_bad_tensors():
    q, k, v, ks, vs, valid = chain_inputs(46)
    c = bd.kv8_quantize(k, v, 32, valid)
    ok = dict(prefix_valid_len=valid)
    for name, call in {
        "k must": lambda: bd.kv8_quantize(k.float(), v),
        "v must": lambda: bd.kv8_quantize(k, v[:, :, :10]),
        "block": lambda: bd.kv8_quantize(k, v, 100),
        "valid_len": lambda: bd.kv8_quantize(k, v, valid_len=valid.long()),
        "out.k_scale": lambda: bd.kv8_quantize(k, v, out=c._replace(k_scale=c.k_scale[:, :, :3])),
        "cache.k must": lambda: bd.suffix_attn_kv8(q[0], c._replace(k=c.k.view(torch.uint8)), ks[0], vs[0], **ok),
        "cache.v_scale": lambda: bd.suffix_attn_kv8(q[0], c._replace(v_scale=c.v_scale.double()), ks[0], vs[0], **ok),
        "k_suffix": lambda: bd.suffix_attn_kv8(q[0], c, ks[0][:, :, :5], vs[0], **ok),
        "q must": lambda: bd.suffix_attn_kv8(q[0].transpose(2, 3).contiguous().transpose(2, 3), c, ks[0], vs[0], **ok),
        "prefix_mask": lambda: bd.suffix_attn_kv8(q[0], c, ks[0], vs[0], prefix_mask=torch.ones(2, 699, device="cuda")),
        "workspace": lambda: bd.suffix_attn_kv8(q[0], c, ks[0], vs[0], workspace=torch.empty(4, device="cuda")),
        "lse": lambda: bd.prefix_attn_mass(q[0], k, torch.zeros(2, 8, 29, device="cuda")),
        "mass_in": lambda: bd.prefix_attn_mass(q[0], k, torch.zeros(2, 8, 30, device="cuda"), mass_in=torch.zeros(2, device="cuda")),
        "mass must": lambda: bd.prefix_evict(k, v, torch.zeros(2, 4, 10, device="cuda"), 5),
        "together": lambda: bd.prefix_evict(k, v, torch.zeros(2, 4, 700, device="cuda"), 5, k_out=k),
        "out must": lambda: bd.prefix_evict_kv8(c, torch.zeros(2, 4, 700, device="cuda"), 5, out=c, bucket=64),
    }.items():
        with pytest.raises(ValueError, match=name):
            call()
    with pytest.raises(bd.Dm05Error):
        bd.prefix_evict(k, v, torch.zeros(2, 4, 700, device="cuda"), 65, bucket=64)
    with pytest.raises(bd.Dm05Error):
        bd.kv8_quantize(k, v, 32, first=31)
    with pytest.raises(bd.Dm05Error):  # 65 queries of two heads: more than 128 rows
        bd.suffix_attn_kv8(torch.zeros(2, 8, 65, 256, dtype=BF, device="cuda"), c,
                           *[torch.zeros(2, 4, 65, 256, dtype=BF, device="cuda")] * 2)
