"""Queries and keys that alternate inside one buffer, in place: the same bits as from copies of their own, and what lies
between them left as it was."""
import pytest
import torch

import group_wise_affine_qlinear_b200 as ql

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("CUDA GPU required for -m gpu tests")
    ql.lib()
    yield
    assert ql.device_status() == 0


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["mh3d", "h3md", "hm3d", "3hmd", "m3hd"])
@pytest.mark.parametrize("M,H,D,adjacent", [(1, 3, 64, False), (77, 5, 128, True), (2500, 3, 72, False)])
def test_in_place_inside_one_projection(M, H, D, adjacent, layout, dt):
    g = torch.Generator(device="cuda").manual_seed(M + D)
    sizes = {"m": M, "h": H, "3": 3, "d": D}
    buf = torch.randn([sizes[c] for c in layout], generator=g, device="cuda").to(dt)
    q, k, v = buf.permute([layout.index(c) for c in "3mhd"])
    turns, axes = ql.rotary_frequencies((16, 8, 8))
    pos = torch.randint(0, 50, (3, M), generator=g, device="cuda")
    weight = torch.randn(2, D, generator=g, device="cuda")
    kw = dict(q_weight=weight[0], k_weight=weight[1], adjacent=adjacent)
    kept = v.clone()
    want = ql.qk_norm_rotary(q.contiguous(), k.contiguous(), pos, (turns, axes), **kw)
    got = ql.qk_norm_rotary(q, k, pos, (turns, axes), q_out=q, k_out=k, **kw)
    assert got[0].data_ptr() == q.data_ptr() and torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(v, kept)
