"""NaN and infinities in ls_prefix_attn_decode: a NaN or +inf among a row's scores gives NaN in its o and
lse, whatever the split of its positions and the output's type; a score of -inf has no weight; other
requests, and requests that see nothing, are not touched."""
import math

import pytest
import torch

from sparse_attention_decode_ls_b200 import binding as B
from test_gpu_prefix_attn import SCALE, check, make, run

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float32]


def row_of(d, b, pos):
    return int(d["table"][b, pos // 64]), pos % 64


def same(a, b):
    return torch.equal(a.nan_to_num(nan=3e30), b.nan_to_num(nan=3e30)) and torch.equal(a.isnan(), b.isnan())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lens,heads,prefix,pos", [
    ([200], 128, 0, 70),                # one unit: it writes o and lse itself
    ([300, 200], 16, 0, 199),
    ([3000, 2500, 2700], 24, 0, 1500),  # own parts in several units
    ([3000, 2500, 2700], 128, 2048, 2100),
    ([128, 128], 128, 128, 5),          # shared pages only
])
@pytest.mark.parametrize("dim", [3, 575])
def test_one_nan_row(lens, heads, prefix, pos, dim, dtype):
    d = make(lens, heads, prefix, seed=21)
    clean = run(d, dtype=dtype)
    b = len(lens) - 1
    page, line = row_of(d, b, pos)
    d["pool"][page, line, dim] = float("nan")
    o, lse = run(d, dtype=dtype)
    seen = range(len(lens)) if pos < prefix // 64 * 64 else [b]
    for i in range(len(lens)):
        if i in seen:
            assert o[i].isnan().all() and lse[i].isnan().all(), i
        else:
            assert torch.equal(o[i], clean[0][i]) and torch.equal(lse[i], clean[1][i]), i
    assert B.ls_check_device_status() == 0


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lens,heads,prefix,pos", [([200], 128, 0, 70), ([3000, 2500], 24, 0, 1500), ([1000, 1100], 128, 960, 1001)])
def test_one_infinite_score(lens, heads, prefix, pos, dtype):
    """An infinity in a row's rotated part (V stays finite): +inf for the heads whose query is positive
    there, -inf, no weight, for the others."""
    d = make(lens, heads, prefix, seed=22)
    b = len(lens) - 1
    page, line = row_of(d, b, pos)
    d["pool"][page, line, 550] = float("inf")
    q = d["q"][b, :, 550]
    assert (q > 0).any() and (q < 0).any() and (q != 0).all()
    o, lse = run(d, dtype=dtype)
    assert o[b][q > 0].isnan().all() and lse[b][q > 0].isnan().all()
    # the other heads: as if the position were not there
    n = lens[b]
    rows = d["pool"][d["table"][b, : -(-n // 64)].long()].flatten(0, 1)[:n]
    e = dict(q=d["q"][b: b + 1, q < 0].contiguous(), pool=torch.cat([rows[:pos], rows[pos + 1:]]).unsqueeze(0),
             table=torch.zeros(1, 1, dtype=torch.int32, device=rows.device))
    e["pool"] = torch.nn.functional.pad(e["pool"], (0, 0, 0, 64 * -(-n // 64) - (n - 1))).unflatten(1, (-1, 64))[0]
    e["table"] = torch.arange(-(-n // 64), dtype=torch.int32, device=rows.device)[None]
    check(e, o[b: b + 1, q < 0], lse[b: b + 1, q < 0], lens=[n - 1])
    assert B.ls_check_device_status() == 0


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lens,prefix", [([128, 0], 128), ([3000, 0, 2900], 2048)])
def test_a_request_that_sees_nothing_beside_nan_on_the_shared_pages(lens, prefix, dtype):
    d = make(lens, 20, prefix, seed=23)
    d["pool"][int(d["table"][0, 1])] = float("nan")
    o, lse = run(d, dtype=dtype)
    for b, n in enumerate(lens):
        if n == 0:
            assert (o[b] == 0).all() and (lse[b] == -math.inf).all()
        else:
            assert o[b].isnan().all() and lse[b].isnan().all()
    assert B.ls_check_device_status() == 0


@pytest.mark.parametrize("dtype", DTYPES)
def test_queries_with_nan(dtype):
    d = make([700, 5000, 64], 40, 64, seed=24)
    clean = run(d, dtype=dtype)
    d["q"][1, 7, 100] = float("nan")
    o, lse = run(d, dtype=dtype)
    assert o[1, 7].isnan().all() and lse[1, 7].isnan()
    o[1, 7], lse[1, 7] = clean[0][1, 7], clean[1][1, 7]
    assert same(o, clean[0]) and same(lse, clean[1])
    assert B.ls_check_device_status() == 0
