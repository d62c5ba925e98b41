"""A long prefix is cut in several passes over its weights.  A caller that
changes them meanwhile (a missing wait between streams) gets positions that
mean nothing, but only positions of the prefix, and nothing outside the outputs
is read or written."""
import pytest
import torch

from gqa_prefix_suffix_b200 import binding as bd

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.mark.parametrize("block", [0, 64])
def test_weights_that_change_during_the_call(block):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    H, P, keep = 2, 40000, 3000
    g = torch.Generator(device="cuda").manual_seed(1)
    k = torch.randn(1, H, P, 256, generator=g, device="cuda").to(BF)
    c = bd.kv8_quantize(k, k, block) if block else None
    m = torch.rand(1, H, P, generator=g, device="cuda")
    other = torch.rand(1, H, P, generator=g, device="cuda")
    pos = torch.full((3, H, keep), 7, dtype=torch.int32, device="cuda")
    mass = torch.full((3, H, keep), 7.0, device="cuda")
    n = torch.full((3,), 7, dtype=torch.int32, device="cuda")
    rows = torch.full((3, H, keep, 256), 7.0, dtype=BF, device="cuda")
    codes = [rows.to(torch.float8_e4m3fn) for _ in range(2)]
    scales = [torch.full((3, H, -(-keep // 64)), 7.0, device="cuda") for _ in range(2)]
    mine, side = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(30):
        with torch.cuda.stream(side):
            for _ in range(20):
                m.copy_(other)
                m.neg_()
        with torch.cuda.stream(mine):
            out = dict(mass_out=mass[1:2], positions=pos[1:2], valid_len=n[1:2])
            if block:
                new = bd.Kv8Cache(codes[0][1:2], codes[1][1:2], scales[0][1:2], scales[1][1:2], block)
                bd.prefix_evict_kv8(c, m, keep, out=new, **out)
            else:
                bd.prefix_evict(k, k, m, keep, k_out=rows[1:2], v_out=torch.empty_like(rows[1:2]), **out)
    torch.cuda.synchronize()
    for t in (pos, mass, n, rows, *scales, *[x.view(torch.uint8) for x in codes]):
        assert (t[0] == t[0].flatten()[0]).all() and (t[2] == t[0].flatten()[0]).all()
    assert (pos[1] >= -1).all() and (pos[1] < P).all() and (n[1] <= keep).all()
    # and the same call with weights that stay is as it was
    m.copy_(other)
    e = bd.prefix_evict(k, k, m, keep)
    torch.cuda.synchronize()
    want = m.topk(keep, dim=-1).indices.sort(-1).values
    assert torch.equal(e.positions.long(), want) and (e.valid_len == keep).all()
    assert torch.equal(e.k, k.gather(2, want[..., None].expand(1, H, keep, 256)))
