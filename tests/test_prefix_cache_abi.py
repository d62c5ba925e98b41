"""The prefix-cache compression entry points without a GPU: bad arguments are
refused on the host, before anything touches CUDA."""
import pytest
import torch

from gqa_prefix_suffix_b200 import binding as bd

F = 0x7f0000001000  # 16-byte aligned, never dereferenced


@pytest.fixture(scope="module", autouse=True)
def lib():
    from gqa_prefix_suffix_b200 import build
    build.build()
    return bd.lib()


def _call(fn, order, defaults, kw):
    a = dict(defaults)
    a.update(kw)
    return fn(*[a[n] for n in order])


QUANT = "k v valid_len k8 v8 k_scale v_scale B Hkv P D block first stream".split()
QUANT_D = dict(k=F, v=F, valid_len=None, k8=F, v8=F, k_scale=F, v_scale=F, B=1, Hkv=4, P=1024, D=256, block=64,
               first=0, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), bd.DM05_ERR_NULL), (dict(v=None), bd.DM05_ERR_NULL), (dict(k8=None), bd.DM05_ERR_NULL),
    (dict(v8=None), bd.DM05_ERR_NULL), (dict(k_scale=None), bd.DM05_ERR_NULL),
    (dict(v_scale=None), bd.DM05_ERR_NULL), (dict(B=0), bd.DM05_ERR_SHAPE), (dict(Hkv=0), bd.DM05_ERR_SHAPE),
    (dict(P=0), bd.DM05_ERR_SHAPE), (dict(P=(1 << 24) + 1), bd.DM05_ERR_SHAPE),
    (dict(B=65536, Hkv=1), bd.DM05_ERR_SHAPE), (dict(D=128), bd.DM05_ERR_UNSUPPORTED),
    (dict(block=0), bd.DM05_ERR_UNSUPPORTED), (dict(block=48), bd.DM05_ERR_UNSUPPORTED),
    (dict(block=256), bd.DM05_ERR_UNSUPPORTED), (dict(first=-64), bd.DM05_ERR_SHAPE),
    (dict(first=32), bd.DM05_ERR_SHAPE), (dict(first=1024), bd.DM05_ERR_SHAPE),
    (dict(k=F + 8), bd.DM05_ERR_ALIGN), (dict(v8=F + 4), bd.DM05_ERR_ALIGN),
    (dict(k_scale=F + 2), bd.DM05_ERR_ALIGN), (dict(valid_len=F + 1), bd.DM05_ERR_ALIGN),
])
def test_quantize_refuses(kw, status):
    assert _call(bd.dm05_kv8_quantize, QUANT, QUANT_D, kw) == status


ATTN = ("q k8 v8 k_scale v_scale block valid_len mask k_suffix v_suffix out lse workspace workspace_bytes B Hq Hkv P "
        "S D stream").split()
ATTN_D = dict(q=F, k8=F, v8=F, k_scale=F, v_scale=F, block=64, valid_len=None, mask=None, k_suffix=F, v_suffix=F,
              out=F, lse=None, workspace=None, workspace_bytes=0, B=1, Hq=8, Hkv=4, P=1024, S=50, D=256, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), bd.DM05_ERR_NULL), (dict(k8=None), bd.DM05_ERR_NULL), (dict(v_scale=None), bd.DM05_ERR_NULL),
    (dict(v_suffix=None), bd.DM05_ERR_NULL), (dict(out=None), bd.DM05_ERR_NULL), (dict(B=0), bd.DM05_ERR_SHAPE),
    (dict(S=0), bd.DM05_ERR_SHAPE), (dict(P=-1), bd.DM05_ERR_SHAPE), (dict(Hq=6), bd.DM05_ERR_SHAPE),
    (dict(P=(1 << 24) + 1), bd.DM05_ERR_SHAPE), (dict(B=65536, Hq=1, Hkv=1), bd.DM05_ERR_SHAPE),
    (dict(S=65), bd.DM05_ERR_UNSUPPORTED), (dict(D=64), bd.DM05_ERR_UNSUPPORTED),
    (dict(block=8), bd.DM05_ERR_UNSUPPORTED), (dict(q=F + 8), bd.DM05_ERR_ALIGN), (dict(k8=F + 8), bd.DM05_ERR_ALIGN),
    (dict(out=F + 2), bd.DM05_ERR_ALIGN), (dict(lse=F + 2), bd.DM05_ERR_ALIGN), (dict(k_scale=F + 1), bd.DM05_ERR_ALIGN),
])
def test_attention_refuses(kw, status):
    assert _call(bd.dm05_suffix_attn_kv8, ATTN, ATTN_D, kw) == status


def test_attention_plan_refuses():
    assert bd.dm05_suffix_attn_kv8_plan(0, 8, 4, 1024, 50, 256)[0] == bd.DM05_ERR_SHAPE
    assert bd.dm05_suffix_attn_kv8_plan(1, 6, 4, 1024, 50, 256)[0] == bd.DM05_ERR_SHAPE


@pytest.mark.skipif(torch.cuda.is_available(), reason="for a machine without a GPU")
def test_valid_calls_without_a_gpu_return_an_error():
    assert bd.dm05_suffix_attn_kv8_plan(1, 8, 4, 1024, 50, 256)[0] == bd.DM05_ERR_CUDA
    assert _call(bd.dm05_kv8_quantize, QUANT, QUANT_D, {}) == bd.DM05_ERR_CUDA
    assert _call(bd.dm05_suffix_attn_kv8, ATTN, ATTN_D, {}) == bd.DM05_ERR_CUDA


MASS = "q k valid_len mask lse mass_in mass B Hq Hkv P S D stream".split()
MASS_D = dict(q=F, k=F, valid_len=None, mask=None, lse=F, mass_in=None, mass=F, B=1, Hq=8, Hkv=4, P=1024, S=50, D=256,
              stream=None)
MASS8 = "q k k_scale block valid_len mask lse mass_in mass B Hq Hkv P S D stream".split()


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), bd.DM05_ERR_NULL), (dict(k=None), bd.DM05_ERR_NULL), (dict(lse=None), bd.DM05_ERR_NULL),
    (dict(mass=None), bd.DM05_ERR_NULL), (dict(B=0), bd.DM05_ERR_SHAPE), (dict(P=0), bd.DM05_ERR_SHAPE),
    (dict(S=0), bd.DM05_ERR_SHAPE), (dict(Hq=9), bd.DM05_ERR_SHAPE), (dict(Hq=0), bd.DM05_ERR_SHAPE),
    (dict(S=65), bd.DM05_ERR_UNSUPPORTED), (dict(D=512), bd.DM05_ERR_UNSUPPORTED), (dict(k=F + 8), bd.DM05_ERR_ALIGN),
    (dict(mass=F + 2), bd.DM05_ERR_ALIGN), (dict(mass_in=F + 2), bd.DM05_ERR_ALIGN), (dict(lse=F + 2), bd.DM05_ERR_ALIGN),
])
def test_mass_refuses(kw, status):
    assert _call(bd.dm05_prefix_attn_mass, MASS, MASS_D, kw) == status
    assert _call(bd.dm05_prefix_attn_mass_kv8, MASS8, dict(MASS_D, k_scale=F, block=64), kw) == status


def test_mass_kv8_refuses():
    d = dict(MASS_D, k_scale=F, block=64)
    assert _call(bd.dm05_prefix_attn_mass_kv8, MASS8, d, dict(k_scale=None)) == bd.DM05_ERR_NULL
    assert _call(bd.dm05_prefix_attn_mass_kv8, MASS8, d, dict(block=20)) == bd.DM05_ERR_UNSUPPORTED
    assert _call(bd.dm05_prefix_attn_mass_kv8, MASS8, d, dict(k_scale=F + 2)) == bd.DM05_ERR_ALIGN


EVICT = ("k v mass valid_len mask k_out v_out mass_out positions valid_out B Hkv P P_out D n_keep n_first n_last "
         "stream").split()
EVICT_D = dict(k=F, v=F, mass=F, valid_len=None, mask=None, k_out=F, v_out=F, mass_out=F, positions=F, valid_out=F,
               B=1, Hkv=4, P=1024, P_out=576, D=256, n_keep=512, n_first=0, n_last=0, stream=None)
EVICT8 = ("k v k_scale v_scale block mass valid_len mask k_out v_out k_scale_out v_scale_out mass_out positions "
          "valid_out B Hkv P P_out D n_keep n_first n_last stream").split()
EVICT8_D = dict(EVICT_D, k_scale=F, v_scale=F, k_scale_out=F, v_scale_out=F, block=64)


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), bd.DM05_ERR_NULL), (dict(mass=None), bd.DM05_ERR_NULL), (dict(v_out=None), bd.DM05_ERR_NULL),
    (dict(mass_out=None), bd.DM05_ERR_NULL), (dict(positions=None), bd.DM05_ERR_NULL),
    (dict(valid_out=None), bd.DM05_ERR_NULL), (dict(B=0), bd.DM05_ERR_SHAPE), (dict(P=0), bd.DM05_ERR_SHAPE),
    (dict(P_out=0), bd.DM05_ERR_SHAPE), (dict(n_keep=577), bd.DM05_ERR_SHAPE), (dict(n_keep=-1), bd.DM05_ERR_SHAPE),
    (dict(n_first=-1), bd.DM05_ERR_SHAPE), (dict(n_last=-1), bd.DM05_ERR_SHAPE), (dict(D=255), bd.DM05_ERR_UNSUPPORTED),
    (dict(k_out=F + 8), bd.DM05_ERR_ALIGN), (dict(mass=F + 1), bd.DM05_ERR_ALIGN),
    (dict(positions=F + 2), bd.DM05_ERR_ALIGN),
])
def test_evict_refuses(kw, status):
    assert _call(bd.dm05_prefix_evict, EVICT, EVICT_D, kw) == status
    assert _call(bd.dm05_prefix_evict_kv8, EVICT8, EVICT8_D, kw) == status


def test_evict_refuses_to_work_in_place():
    G = 1 << 40
    apart = dict(v=F + G, k_out=F + 2 * G, v_out=F + 3 * G, mass=F + 4 * G, mass_out=F + 5 * G, B=2)
    for fn, order, d, row in ((bd.dm05_prefix_evict, EVICT, EVICT_D, 512), (bd.dm05_prefix_evict_kv8, EVICT8, EVICT8_D, 256)):
        d = dict(d, **apart)
        size = 2 * 4 * 1024 * row
        for kw in (dict(k_out=F), dict(v_out=F), dict(k_out=F + size - 16), dict(k_out=F + G - 16), dict(v_out=F + G + 512),
                   dict(v_out=F + 2 * G), dict(mass_out=F + 4 * G + 4)):
            assert _call(fn, order, d, kw) == bd.DM05_ERR_UNSUPPORTED
        if not torch.cuda.is_available():                  # one row behind the old cache is no overlap
            assert _call(fn, order, d, dict(k_out=F + size)) == bd.DM05_ERR_CUDA


def test_evict_kv8_refuses():
    for name in ("k_scale", "v_scale", "k_scale_out", "v_scale_out"):
        assert _call(bd.dm05_prefix_evict_kv8, EVICT8, EVICT8_D, {name: None}) == bd.DM05_ERR_NULL
        assert _call(bd.dm05_prefix_evict_kv8, EVICT8, EVICT8_D, {name: F + 2}) == bd.DM05_ERR_ALIGN
    assert _call(bd.dm05_prefix_evict_kv8, EVICT8, EVICT8_D, dict(block=24)) == bd.DM05_ERR_UNSUPPORTED


def test_front_end_refuses_host_tensors():
    bf = torch.bfloat16
    k = torch.zeros(1, 4, 64, 256, dtype=bf)
    q = torch.zeros(1, 8, 10, 256, dtype=bf)
    s = torch.zeros(1, 4, 10, 256, dtype=bf)
    c = bd.Kv8Cache(k.to(torch.float8_e4m3fn), k.to(torch.float8_e4m3fn), torch.ones(1, 4, 1), torch.ones(1, 4, 1), 64)
    with pytest.raises(ValueError, match="k must"):
        bd.kv8_quantize(k, k)
    with pytest.raises(ValueError, match="q must"):
        bd.suffix_attn_kv8(q, c, s, s)
    with pytest.raises(ValueError, match="q must"):
        bd.prefix_attn_mass(q, k, torch.zeros(1, 8, 10))
    with pytest.raises(ValueError, match="k must"):
        bd.prefix_evict(k, k, torch.zeros(1, 4, 64), 16)
    with pytest.raises(ValueError, match="cache.k must"):
        bd.prefix_evict_kv8(c, torch.zeros(1, 4, 64), 16)
    with pytest.raises(ValueError, match="block"):
        bd.prefix_evict_kv8(c._replace(block=65), torch.zeros(1, 4, 64), 16)
