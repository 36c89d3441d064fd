"""Calls large enough that a group of lanes takes several consecutive rows (a prefill chunk): the next
row loaded before the one at hand is finished, in place too, scratch that is used again, shares that do not
divide evenly, and requests, padding and ends of pages inside one group's rows.

A group takes min(8, blocks / (4 * 592 or 888)) rows, blocks of 8 to 32 rows: at least two from
151,552 bf16 rows of 128, 56,832 float32 ones, 37,888 bf16 rows of 576, or 30,310 appended tokens."""
import pytest
import torch

from sparse_attention_decode_ls_b200 import binding as B
from test_gpu_head_rows import EPS, append_case, build, check_rows, reference

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32
NONE, RMS, LAYER = B.LS_NORM_NONE, B.LS_NORM_RMS, B.LS_NORM_LAYER

LONG = [
    # tokens, heads, dim, dtype, norm, norm_dim, rope_begin, rope, pairs, e4m3
    (2501, 64, 128, BF, RMS, 128, 0, 64, False, True),       # halves in the same lane
    (7919, 64, 128, BF, RMS, 128, 0, 128, False, False),     # halves through shared memory, 6 to 7 rows
    (2501, 64, 128, BF, LAYER, 128, 32, 64, True, True),
    (2753, 61, 96, BF, NONE, 96, None, 2, False, True),      # e4m3 without a norm or rotation
    (2501, 64, 64, BF, NONE, 64, 0, 64, False, True),        # rotated, quantised, no norm
    (4097, 17, 128, F32, RMS, 128, 0, 128, False, False),
    (4097, 17, 128, F32, LAYER, 128, 0, 64, True, True),
    (613, 128, 576, BF, NONE, 576, 512, 64, True, False),    # moved, its last dims rotated
    (613, 128, 576, BF, RMS, 512, 512, 64, False, False),
    (613, 128, 200, BF, RMS, 200, 40, 80, False, True),
    (40001, 1, 1024, BF, LAYER, 1024, 0, 1024, False, False),
]


@pytest.mark.parametrize("case", LONG)
def test_many_rows_against_64_bits(case):
    T, H, D, dt, norm, nd, begin, rope, pairs, e4m3 = case
    x, w, b, pos, cs = build(case, 7)
    pos[::97] = -1            # padding tokens inside a group's rows
    pos[5::1013] = 1000       # beyond the table: flagged if rotated
    live = pos >= 0 if begin is None else (pos >= 0) & (pos < 1000)
    out = torch.full((T, H, D), 3, dtype=torch.uint8 if e4m3 else dt, device=DEV)
    scale = torch.full((T, H), 5.0, device=DEV) if e4m3 else None
    r = B.head_rows(x, norm=norm, norm_dim=nd, weight=w, bias=b, eps=EPS, rope_begin=begin,
                    rope_layout=B.LS_ROPE_PAIRS if pairs else B.LS_ROPE_HALVES)
    B.ls_qk_norm_rope(pos=pos, cos_sin=cs, q=r, q_out=out, q_scale=scale)
    assert B.ls_check_device_status() == (0 if begin is None else B.LS_DEV_BOUNDS)
    for part in live.nonzero()[:, 0].chunk(8):
        y, M = reference(x[part], cs[pos[part].long().clamp(max=999)][:, None], norm=norm, norm_dim=nd, weight=w, bias=b, begin=begin,
                         pairs=pairs)
        check_rows(out[part], None if scale is None else scale[part], y, M)
    assert (out[~live] == 3).all() and (scale is None or (scale[~live] == 5.0).all())
    if not e4m3:  # and in place: the next row has been read when this one is stored
        x0 = x.clone()
        B.ls_qk_norm_rope(pos=pos, cos_sin=cs, q=r, q_out=x)
        assert B.ls_check_device_status() == (0 if begin is None else B.LS_DEV_BOUNDS)
        assert torch.equal(x[live], out[live]) and torch.equal(x[~live], x0[~live])


def test_two_operands_of_many_rows():
    """Query heads and one key head (layer norm with a bias) to e4m3: the two take shares of their own."""
    T = 5003
    x, w, _, pos, cs = build((T, 64, 128, BF, RMS, 128, 0, 64, False, True), 8)
    xk, wk, bk, _, _ = build((T, 1, 128, BF, LAYER, 128, 0, 64, False, True), 9)
    qo, ko = torch.zeros(T, 64, 128, dtype=torch.uint8, device=DEV), torch.zeros(T, 1, 128, dtype=torch.uint8, device=DEV)
    qs, ks = torch.zeros(T, 64, device=DEV), torch.zeros(T, 1, device=DEV)
    B.ls_qk_norm_rope(pos=pos, cos_sin=cs, q=B.head_rows(x, norm=RMS, weight=w, eps=EPS, rope_begin=0), q_out=qo, q_scale=qs,
                      k=B.head_rows(xk, norm=LAYER, weight=wk, bias=bk, eps=EPS, rope_begin=0), k_out=ko, k_scale=ks)
    angles = cs[pos.long()][:, None]
    check_rows(qo, qs, *reference(x, angles, norm=RMS, norm_dim=128, weight=w, bias=None, begin=0, pairs=False))
    check_rows(ko, ks, *reference(xk, angles, norm=LAYER, norm_dim=128, weight=wk, bias=bk, begin=0, pairs=False))
    assert B.ls_check_device_status() == 0


@pytest.mark.parametrize("start,counts,dt,e4m3", [
    # many short requests, empty ones and padding requests among them: a group's rows pass over them
    ([-1 if i % 11 == 5 else (i * 37) % 130 for i in range(2600)], [(i * 29) % 31 for i in range(2600)], BF, True),
    ([(i * 997) % 3000 for i in range(14)], [(i * 7919) % 8191 for i in range(14)], BF, True),  # some 57,000 tokens: three rows each
    ([-1 if i % 7 == 3 else (i * 37) % 130 for i in range(900)], [(i * 29) % 41 for i in range(900)], F32, False),
    ([100, 0, 64], [9001, 0, 9013], F32, True),
])
def test_many_appended_tokens_against_64_bits(start, counts, dt, e4m3):
    assert append_case(start, counts, dt, e4m3, seed=len(start), pad_rows=77) == 0


def test_rows_before_the_first_request_are_padding():
    g = torch.Generator(device=DEV).manual_seed(2)
    x = torch.randn(40, 128, generator=g, device=DEV).to(BF)
    key = torch.zeros(4, 64, 128, dtype=BF, device=DEV)
    B.ls_cache_append(page_table=torch.tensor([[2, 0], [1, 3]], dtype=torch.int32, device=DEV),
                      start=torch.tensor([60, 0], dtype=torch.int32, device=DEV),
                      cu_tokens=torch.tensor([7, 17, 20], dtype=torch.int32, device=DEV), key=B.head_rows(x), key_pool=key)
    want = torch.zeros_like(key)
    want[2, 60:], want[0, :6], want[1, :3] = x[7:11], x[11:17], x[17:20]
    assert torch.equal(key, want) and B.ls_check_device_status() == 0
