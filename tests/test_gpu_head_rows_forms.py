"""Forms of ls_qk_norm_rope and ls_cache_append beside the common ones: codes without a norm, a bias
without a weight, parameters in the other type than the rows', one cache alone, one operand of 16-byte
chunks beside one that is not."""
import pytest
import torch

from sparse_attention_decode_ls_b200 import binding as B
from test_gpu_head_rows import EPS, build, check_rows, pools, reference, table

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("layout", ["packed", "odd"])
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("dim,begin,rope,pairs", [(128, None, 2, False), (128, 0, 64, False), (128, 64, 64, True), (80, 0, 40, False), (576, 512, 64, True)])
def test_codes_without_a_norm(dim, begin, rope, pairs, dt, layout):
    case = (9, 5, dim, dt, B.LS_NORM_NONE, dim, begin, rope, pairs, True)
    x, _, _, pos, cs = build(case, 31, wide=3 * (layout == "odd"), shift=int(layout == "odd"))
    out, scale = torch.zeros(9, 5, dim, dtype=torch.uint8, device=DEV), torch.zeros(9, 5, device=DEV)
    B.ls_qk_norm_rope(pos=pos, cos_sin=cs, q=B.head_rows(x, rope_begin=begin, rope_layout=B.LS_ROPE_PAIRS if pairs else B.LS_ROPE_HALVES),
                      q_out=out, q_scale=scale)
    check_rows(out, scale, *reference(x, cs[pos.long()][:, None], norm=B.LS_NORM_NONE, norm_dim=dim, weight=None, bias=None, begin=begin, pairs=pairs))
    assert B.ls_check_device_status() == 0


@pytest.mark.parametrize("layout", ["packed", "odd"])
@pytest.mark.parametrize("weight,bias", [(False, True), (True, False), (False, False), (True, True)])
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("w_dtype", [BF, F32])
def test_layer_norm_with_any_of_its_parameters(weight, bias, dt, w_dtype, layout):
    case = (6, 3, 128, dt, B.LS_NORM_LAYER, 128, 0, 64, False, False)
    x, w, b, pos, cs = build(case, 32, w_dtype=w_dtype, wide=3 * (layout == "odd"), shift=int(layout == "odd"))
    w, b = w if weight else None, b if bias else None
    out = torch.zeros(6, 3, 128, dtype=dt, device=DEV)
    B.ls_qk_norm_rope(pos=pos, cos_sin=cs, q=B.head_rows(x, norm=B.LS_NORM_LAYER, weight=w, bias=b, eps=EPS, rope_begin=0), q_out=out)
    check_rows(out, None, *reference(x, cs[pos.long()][:, None], norm=B.LS_NORM_LAYER, norm_dim=128, weight=w, bias=b, begin=0, pairs=False))
    assert B.ls_check_device_status() == 0


@pytest.mark.parametrize("dt,key_dt", [(BF, torch.uint8), (BF, BF), (F32, F32)])
def test_append_of_one_cache_alone(dt, key_dt):
    g = torch.Generator(device=DEV).manual_seed(5)
    e4m3 = key_dt is torch.uint8
    kv, key, ks = pools(6, 128, dt, e4m3, g)
    kv0, key0, ks0 = kv.clone(), key.clone(), None if ks is None else ks.clone()
    x = torch.randn(70, 128, generator=g, device=DEV).to(dt)
    b = (0.2 * torch.randn(128, generator=g, device=DEV)).to(F32)
    cs = table(200, 64)
    tbl = torch.tensor([[3, 0], [1, 5]], dtype=torch.int32, device=DEV)
    start, cu = torch.tensor([30, 64], dtype=torch.int32, device=DEV), torch.tensor([0, 66, 70], dtype=torch.int32, device=DEV)
    B.ls_cache_append(page_table=tbl, start=start, cu_tokens=cu, cos_sin=cs, key_pool=key, key_scale=ks,
                      key=B.head_rows(x, norm=B.LS_NORM_LAYER, bias=b, eps=EPS, rope_begin=0))
    pos = torch.cat([torch.arange(30, 96), torch.arange(64, 68)]).to(DEV)
    req = torch.tensor([0] * 66 + [1] * 4, device=DEV)
    slot = tbl[req, pos // 64].long() * 64 + pos % 64
    y, M = reference(x, cs[pos], norm=B.LS_NORM_LAYER, norm_dim=128, weight=None, bias=b, begin=0, pairs=False)
    check_rows(key.flatten(0, 1)[slot], None if ks is None else ks.flatten()[slot], y, M)
    key.flatten(0, 1)[slot] = key0.flatten(0, 1)[slot]
    assert torch.equal(key, key0)
    if ks is not None:
        ks.view(-1)[slot] = ks0.view(-1)[slot]
        assert torch.equal(ks, ks0)
    # and the rows alone
    x = torch.randn(70, 576, generator=g, device=DEV).to(dt)
    B.ls_cache_append(page_table=tbl, start=start, cu_tokens=cu, kv=B.head_rows(x), kv_pool=kv)
    kv0.flatten(0, 1)[slot] = x
    assert torch.equal(kv, kv0) and B.ls_check_device_status() == 0


def test_one_operand_of_whole_chunks_beside_one_that_is_not():
    case = (40, 6, 128, BF, B.LS_NORM_RMS, 128, 0, 64, False, False)
    x, w, _, pos, cs = build(case, 33)
    xk, wk, _, _, _ = build((40, 1, 128, BF, B.LS_NORM_RMS, 128, 0, 64, False, True), 34, wide=3, shift=1)
    out, ko, ks = torch.zeros(40, 6, 128, dtype=BF, device=DEV), torch.zeros(40, 1, 128, dtype=torch.uint8, device=DEV), torch.zeros(40, 1, device=DEV)
    B.ls_qk_norm_rope(pos=pos, cos_sin=cs, q=B.head_rows(x, norm=B.LS_NORM_RMS, weight=w, eps=EPS, rope_begin=0), q_out=out,
                      k=B.head_rows(xk, norm=B.LS_NORM_RMS, weight=wk, eps=EPS, rope_begin=0), k_out=ko, k_scale=ks)
    angles = cs[pos.long()][:, None]
    check_rows(out, None, *reference(x, angles, norm=B.LS_NORM_RMS, norm_dim=128, weight=w, bias=None, begin=0, pairs=False))
    check_rows(ko, ks, *reference(xk, angles, norm=B.LS_NORM_RMS, norm_dim=128, weight=wk, bias=None, begin=0, pairs=False))
    assert B.ls_check_device_status() == 0
