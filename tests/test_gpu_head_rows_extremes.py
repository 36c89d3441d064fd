"""e4m3 rows whose values are huge, infinite or NaN, by the definition: scale = max(max |y|, 1e-12) / 448,
codes of y / scale.  Tolerances as in test_gpu_head_rows."""
import pytest
import torch

from sparse_attention_decode_ls_b200 import binding as B
from test_gpu_head_rows import check_rows, pools, reference

pytestmark = pytest.mark.gpu

DEV = "cuda"


def to_e4m3(x, layout):
    """Rows x [tokens, heads, dim] without a norm or rotation; "odd": not made of 16-byte chunks."""
    T, H, D = x.shape
    if layout == "odd":
        buf = torch.zeros(T, H * D + 3, dtype=x.dtype, device=DEV)
        buf[:, 1: 1 + H * D] = x.flatten(1)
        x = buf[:, 1: 1 + H * D].unflatten(1, (H, D))
    out = torch.full((T, H, D), 9, dtype=torch.uint8, device=DEV)
    scale = torch.full((T, H), 7.0, device=DEV)
    B.ls_qk_norm_rope(pos=torch.zeros(T, dtype=torch.int32, device=DEV), q=B.head_rows(x), q_out=out, q_scale=scale)
    assert B.ls_check_device_status() == 0
    return out, scale


@pytest.mark.parametrize("layout", ["packed", "odd"])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dim", [64, 128, 576, 1024])
def test_rows_up_to_the_largest_value(dt, layout, dim):
    """Maxima of 2^118 to the largest finite value of the type, and tiny ones down to below 1e-12."""
    g = torch.Generator(device=DEV).manual_seed(dim)
    x = 2 * torch.rand(20, 2, dim, generator=g, device=DEV, dtype=torch.float64) - 1
    x[:, 0, 3] = 1.0
    top = torch.tensor([2.0 ** e for e in (118, 124, 125, 126, 126.5, 127, 127.5)] + [torch.finfo(dt).max, 1.0, 1e-10, 1e-13, 1e-30],
                       dtype=torch.float64, device=DEV)
    x = (x * top.repeat(2)[:20, None, None]).to(dt)
    assert x.isfinite().all()
    out, scale = to_e4m3(x, layout)
    y, M = reference(x, None, norm=B.LS_NORM_NONE, norm_dim=dim, weight=None, bias=None, begin=None, pairs=False)
    check_rows(out, scale, y, M)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_append_of_a_huge_key(dt):
    g = torch.Generator(device=DEV).manual_seed(1)
    _, key, ks = pools(2, 128, dt, True, g)
    x = ((2 * torch.rand(2, 128, generator=g, device=DEV) - 1) * 2.0 ** 127).to(dt)
    B.ls_cache_append(page_table=torch.tensor([[1], [0]], dtype=torch.int32, device=DEV), start=torch.tensor([5, 6], dtype=torch.int32, device=DEV),
                      key=B.head_rows(x), key_pool=key, key_scale=ks)
    y, M = reference(x, None, norm=B.LS_NORM_NONE, norm_dim=128, weight=None, bias=None, begin=None, pairs=False)
    check_rows(torch.stack([key[1, 5], key[0, 6]]), torch.stack([ks[1, 5], ks[0, 6]]), y, M)
