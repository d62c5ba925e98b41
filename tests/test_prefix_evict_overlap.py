"""An eviction whose outputs overlap its inputs, or one another, is refused:
CTAs of other heads still read what it would write."""
import pytest
import torch

from gqa_prefix_suffix_b200 import binding as bd

F, G = 0x7f0000001000, 1 << 36  # addresses, far apart, never dereferenced
NAMES = "k v k_scale v_scale mass valid_len mask k_out v_out k_scale_out v_scale_out mass_out positions valid_out".split()
AT = {n: F + i * G for i, n in enumerate(NAMES)}
SIZES = dict(B=2, Hkv=4, P=1024, P_out=576, D=256, n_keep=512, n_first=0, n_last=0, stream=None)
ORDER = ("k v mass valid_len mask k_out v_out mass_out positions valid_out B Hkv P P_out D n_keep n_first n_last "
         "stream").split()
ORDER8 = ("k v k_scale v_scale block mass valid_len mask k_out v_out k_scale_out v_scale_out mass_out positions "
          "valid_out B Hkv P P_out D n_keep n_first n_last stream").split()


@pytest.fixture(scope="module", autouse=True)
def lib():
    from gqa_prefix_suffix_b200 import build
    build.build()
    return bd.lib()


def call(order, **kw):
    a = dict(AT, block=64, **SIZES)
    a.update(kw)
    return (bd.dm05_prefix_evict_kv8 if order is ORDER8 else bd.dm05_prefix_evict)(*[a[n] for n in order])


LENGTH = dict(k=2 * 4 * 1024 * 256, mass=2 * 4 * 1024 * 4, valid_len=2 * 4, mask=2 * 1024, mass_out=2 * 4 * 576 * 4,
              k_out=2 * 4 * 576 * 256, positions=2 * 4 * 576 * 4, k_scale=2 * 4 * 16 * 4)
PAIRS = [("valid_out", "valid_len"), ("valid_out", "mask"), ("valid_out", "mass"), ("mass_out", "valid_len"),
         ("mass_out", "mask"), ("mass_out", "mass"), ("mass_out", "k"), ("positions", "mass"), ("positions", "valid_len"),
         ("positions", "mask"), ("k_out", "mass"), ("v_out", "valid_len"), ("k_out", "mask"), ("valid_out", "mass_out"),
         ("positions", "mass_out"), ("positions", "k_out"), ("valid_out", "k_out"), ("mass_out", "k_out"), ("v_out", "k_out"),
         ("v_out", "k")]


@pytest.mark.parametrize("out,other", PAIRS)
def test_overlaps_are_refused(out, other):
    for order in (ORDER, ORDER8):
        assert call(order, **{out: AT[other]}) == bd.DM05_ERR_UNSUPPORTED
        # the last bytes of the other array (its row is at least as long in either form)
        assert call(order, **{out: AT[other] + max(0, LENGTH[other] - 16)}) == bd.DM05_ERR_UNSUPPORTED


@pytest.mark.parametrize("out", ["k_out", "v_out", "mass_out"])
@pytest.mark.parametrize("scale", ["k_scale", "v_scale"])
def test_a_cache_on_the_scales_is_refused(out, scale):
    assert call(ORDER8, **{out: AT[scale]}) == bd.DM05_ERR_UNSUPPORTED


@pytest.mark.skipif(torch.cuda.is_available(), reason="for a machine without a GPU")
def test_neighbours_are_no_overlap():
    for order, row in ((ORDER, 512), (ORDER8, 256)):
        assert call(order) == bd.DM05_ERR_CUDA
        assert call(order, v=AT["k"]) == bd.DM05_ERR_CUDA  # inputs may
        assert call(order, valid_len=None, mask=None) == bd.DM05_ERR_CUDA
        for out, other, size in (("k_out", "k", 2 * 4 * 1024 * row), ("valid_out", "valid_len", 8),
                                 ("positions", "mass", 2 * 4 * 1024 * 4), ("mass_out", "mask", 2 * 1024)):
            assert call(order, **{out: AT[other] + size}) == bd.DM05_ERR_CUDA


def tensors(B=3, H=4, P=300, rows=128):
    bf, d = torch.bfloat16, "cuda"
    g = torch.Generator(device=d).manual_seed(3)
    k, v = (torch.randn(B, H, P, 256, generator=g, device=d).to(bf) for _ in range(2))
    m = torch.rand(B, H, P, generator=g, device=d)
    return k, v, m, torch.tensor([300, 150, 77], dtype=torch.int32, device=d)


@pytest.mark.gpu
def test_calls_in_place_are_refused_and_change_nothing():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    k, v, m, n = tensors()
    c = bd.kv8_quantize(k, v, 64, n)
    out = bd.Kv8Cache(torch.zeros_like(c.k[:, :, :128]), torch.zeros_like(c.v[:, :, :128]), torch.ones_like(c.k_scale[:, :, :2]),
                      torch.ones_like(c.v_scale[:, :, :2]), 64)
    before = [t.clone() for t in (m, n, c.k_scale, c.v_scale)]
    pos = torch.empty(3, 4, 128, dtype=torch.int32, device="cuda")
    codes = c.k.view(torch.uint8).view(-1)
    for kw in (dict(valid_len=n), dict(positions=m.view(torch.int32).view(-1)[:pos.numel()].view(3, 4, 128)),
               dict(mass_out=pos.view(torch.float32), positions=pos),
               dict(out=out._replace(k_scale=c.k_scale.view(-1)[:24].view(3, 4, 2))),
               dict(out=out._replace(v_scale=c.v_scale.view(-1)[8:32].view(3, 4, 2))),
               dict(out=out._replace(v_scale=c.k_scale.view(-1)[:24].view(3, 4, 2))),
               dict(out=out._replace(v_scale=out.k_scale)),
               dict(positions=codes[:4 * pos.numel()].view(torch.int32).view(3, 4, 128)),
               dict(valid_len=codes[:12].view(torch.int32)),
               dict(positions=pos, valid_len=pos.view(-1)[:3])):
        with pytest.raises(bd.Dm05Error):
            bd.prefix_evict_kv8(c, m, 100, prefix_valid_len=n, **dict(dict(out=out), **kw))
    for kw in (dict(valid_len=n), dict(positions=k.view(-1)[:2 * pos.numel()].view(torch.int32).view(3, 4, 128)),
               dict(positions=pos, valid_len=pos.view(-1)[5:8])):
        with pytest.raises(bd.Dm05Error):
            bd.prefix_evict(k, v, m, 100, prefix_valid_len=n, bucket=128, **kw)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(before, (m, n, c.k_scale, c.v_scale)))
    # the same with arrays of their own runs
    e = bd.prefix_evict_kv8(c, m, 100, prefix_valid_len=n, out=out, positions=pos)
    assert e.valid_len.tolist() == [100, 100, 77]
    assert bd.dm05_get_error_word(None) == (0, 0)
