"""The 64-bit forms that the prefix-cache tests compare with, against library
routines and closed forms."""
import numpy as np
import torch

import prefix_cache_ref as ref


def test_rounding_matches_the_type():
    # every e4m3 value, every midpoint between neighbours, and values beside them
    codes = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    mids = (codes[1:] + codes[:-1]) / 2
    x = np.concatenate([codes, mids, mids * (1 + 2.0 ** -20), mids * (1 - 2.0 ** -20)])
    x = np.concatenate([x, -x])
    want = torch.from_numpy(x).float().to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ref.e4m3_round(x), want)
    assert np.isnan(ref.e4m3_round(np.array([np.inf, -np.inf, np.nan]))).all()


def test_scale_rule():
    for a, s in ((0.0, 1.0), (448.0, 1.0), (448.0 * (1 + 2.0 ** -8), 2.0), (1.0, 2.0 ** -8), (1.75, 2.0 ** -8),
                 (1.7578125, 2.0 ** -7), (2.0 ** -133, 2.0 ** -64), (3.38953139e38, 2.0 ** 120)):
        assert ref.pow2_scale(a) == s


def test_attention_form_matches_library_softmax():
    g = torch.Generator().manual_seed(5)
    q, k, v = (torch.randn(2, h, n, 256, generator=g, dtype=torch.float64) for h, n in ((4, 3), (2, 20), (2, 20)))
    ks, vs = (torch.randn(2, 2, 3, 256, generator=g, dtype=torch.float64) for _ in range(2))
    vis = torch.rand(2, 20, generator=g) < 0.5
    out, lse, tol, tol_lse = ref.attention(q, k, v, ks, vs, vis)
    see = torch.cat([torch.ones(2, 3, dtype=torch.bool), vis], 1)[:, None, None]
    keys, vals = (torch.cat([a, c], 2).repeat_interleave(2, 1) for a, c in ((ks, k), (vs, v)))
    want = torch.nn.functional.scaled_dot_product_attention(q, keys, vals, attn_mask=see)
    assert (out - want).abs().max() < 1e-12
    assert (tol > 0).all() and (tol_lse > 0).all()
    # the weight that all positions received is the queries' weight off the suffix
    m, _ = ref.mass(q, k, lse, vis, None)
    z = torch.einsum("bhsd,bhkd->bhsk", q, ks.repeat_interleave(2, 1)) / 16
    assert abs(m.sum() - (2 * 4 * 3 - torch.exp(z - lse[..., None]).sum())) < 1e-10


def test_eviction_order():
    m = [0.5, float("nan"), 0.5, 2.0, 0.0, 7.0]
    assert ref.evict_order(m, [1] * 6, 6, 3, 0, 0) == [0, 3, 5]
    assert ref.evict_order(m, [1] * 6, 6, 4, 0, 0) == [0, 2, 3, 5]
    assert ref.evict_order(m, [1, 1, 1, 1, 1, 0], 5, 2, 0, 1) == [3, 4]
    assert ref.evict_order(m, [1] * 6, 6, 1, 2, 0) == [0]
    assert ref.evict_order(m, [0] * 6, 6, 3, 0, 0) == []
    assert ref.evict_order(m, [1] * 6, 6, 6, 0, 0) == [0, 1, 2, 3, 4, 5]
