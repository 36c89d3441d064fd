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


@pytest.mark.parametrize("layout", ["packed", "odd"])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dim", [64, 128, 576, 1024])
def test_infinite_and_nan_rows(dt, layout, dim):
    """An infinity: scale inf, its own code NaN (inf / inf), the finite values' zero.  A NaN anywhere: the
    maximum is NaN, so the scale and all codes are.  Other rows are not touched by either."""
    g = torch.Generator(device=DEV).manual_seed(dim)
    x = torch.randn(9, 3, dim, generator=g, device=DEV).to(dt)
    clean = x.clone()
    for t, d in enumerate((0, 1, dim // 2, dim - 1)):
        x[t, 1, d] = float("inf") if t % 2 else -float("inf")
        x[t + 4, 1, d] = float("nan")
    out, scale = to_e4m3(x, layout)
    v = out.view(torch.float8_e4m3fn).float()
    assert (scale[:4, 1] == float("inf")).all()
    inf = x[:4, 1].isinf()
    assert v[:4, 1][inf].isnan().all() and (v[:4, 1][~inf] == 0).all()
    assert scale[4:8, 1].isnan().all() and v[4:8, 1].isnan().all()
    want, want_scale = to_e4m3(clean, layout)
    others = torch.ones(9, 3, dtype=torch.bool, device=DEV)
    others[:8, 1] = False
    assert torch.equal(out[others], want[others]) and torch.equal(scale[others], want_scale[others])


@pytest.mark.parametrize("norm", [B.LS_NORM_RMS, B.LS_NORM_LAYER])
@pytest.mark.parametrize("layout", ["packed", "odd"])
def test_nan_through_a_norm(norm, layout):
    """The norm carries a NaN to every value of its row: NaN scale and codes, or NaN values."""
    g = torch.Generator(device=DEV).manual_seed(3)
    buf = torch.randn(4, 2 * 128 + (3 if layout == "odd" else 0), generator=g, device=DEV).to(torch.bfloat16)
    x = buf[:, (1 if layout == "odd" else 0):][:, :256].unflatten(1, (2, 128))
    x[2, 1, 77] = float("nan")
    pos = torch.zeros(4, dtype=torch.int32, device=DEV)
    out, scale, same = torch.zeros(4, 2, 128, dtype=torch.uint8, device=DEV), torch.zeros(4, 2, device=DEV), torch.zeros(4, 2, 128, dtype=torch.bfloat16, device=DEV)
    r = B.head_rows(x, norm=norm)
    B.ls_qk_norm_rope(pos=pos, q=r, q_out=out, q_scale=scale, k=r, k_out=same)
    nan = torch.zeros(4, 2, dtype=torch.bool, device=DEV)
    nan[2, 1] = True
    assert torch.equal(scale.isnan(), nan)
    v = out.view(torch.float8_e4m3fn).float()
    assert torch.equal(v.isnan(), nan[..., None].expand_as(v)) and torch.equal(same.isnan(), nan[..., None].expand_as(same))
