"""What the Python builders of ls_qk_norm_rope, ls_cache_append and ls_prefix_attn_decode make of their
tensors, and which they refuse: the library sees addresses only, so types, shapes and strides are
checked here.  CPU only."""
import pytest
import torch

from sparse_attention_decode_ls_b200 import binding as B

BF, F32 = torch.bfloat16, torch.float32


# ------------------------------------------------------------------------------- weights and biases
@pytest.mark.parametrize("weight,bias,want", [
    (None, None, None), (BF, None, B.LS_BF16), (F32, None, B.LS_F32), (None, BF, B.LS_BF16), (None, F32, B.LS_F32),
    (BF, BF, B.LS_BF16), (F32, F32, B.LS_F32),
])
def test_type_of_weight_and_bias(weight, bias, want):
    x = torch.zeros(4, 3, 128, dtype=BF)
    w = None if weight is None else torch.ones(128, dtype=weight)
    b = None if bias is None else torch.ones(128, dtype=bias)
    r = B.head_rows(x, norm=B.LS_NORM_LAYER, weight=w, bias=b)
    if want is not None:
        assert r.w_dtype == want
    assert r.weight == (None if w is None else w.data_ptr()) and r.bias == (None if b is None else b.data_ptr())


@pytest.mark.parametrize("weight,bias", [
    (torch.ones(128), torch.ones(128, dtype=BF)), (torch.ones(128, dtype=BF), torch.ones(128)),
    (torch.ones(127), None), (None, torch.ones(127)), (torch.ones(256)[::2], None), (None, torch.ones(256)[::2]),
])
def test_weights_and_biases_that_are_refused(weight, bias):
    with pytest.raises(B.LsError):
        B.head_rows(torch.zeros(4, 3, 128, dtype=BF), norm=B.LS_NORM_LAYER, weight=weight, bias=bias)


def test_weights_as_long_as_the_normalised_part():
    x = torch.zeros(4, 576, dtype=BF)
    r = B.head_rows(x, norm=B.LS_NORM_RMS, norm_dim=512, weight=torch.ones(512))
    assert (r.norm_dim, r.w_dtype) == (512, B.LS_F32)
    with pytest.raises(B.LsError):
        B.head_rows(x, norm=B.LS_NORM_RMS, weight=torch.ones(512))


@pytest.mark.parametrize("shape", [(128,), (2, 4, 3, 128)])
def test_rows_of_another_rank_are_refused(shape):
    with pytest.raises(B.LsError):
        B.head_rows(torch.zeros(*shape, dtype=BF))


# ------------------------------------------------------------------------------- two operands
def heads_call(**kw):
    d = dict(pos=torch.zeros(4, dtype=torch.int32), cos_sin=torch.zeros(100, 64), q=B.head_rows(torch.zeros(4, 3, 128, dtype=BF)),
             q_out=torch.zeros(4, 3, 128, dtype=BF), k=B.head_rows(torch.zeros(4, 1, 576, dtype=BF)),
             k_out=torch.zeros(4, 1, 576, dtype=BF))
    d.update(kw)
    return B.qk_norm_rope_args(**d)


def append_call(**kw):
    d = dict(page_table=torch.zeros(2, 4, dtype=torch.int32), start=torch.zeros(2, dtype=torch.int32),
             cu_tokens=torch.tensor([0, 3, 5], dtype=torch.int32), cos_sin=torch.zeros(256, 64),
             kv=B.head_rows(torch.zeros(5, 576, dtype=BF)), kv_pool=torch.zeros(8, 64, 576, dtype=BF),
             key=B.head_rows(torch.zeros(5, 128, dtype=BF)), key_pool=torch.zeros(8, 64, 128, dtype=torch.uint8),
             key_scale=torch.zeros(8, 64))
    d.update(kw)
    return B.cache_append_args(**d)


def test_operands_of_two_dtypes_are_refused():
    with pytest.raises(B.LsError):
        heads_call(k=B.head_rows(torch.zeros(4, 1, 576)))
    with pytest.raises(B.LsError):
        append_call(key=B.head_rows(torch.zeros(5, 128)))


def test_operands_with_fewer_rows_than_tokens_are_refused():
    assert heads_call().tokens == 4
    assert heads_call(pos=torch.zeros(3, dtype=torch.int32)).tokens == 3  # longer buffers are fine
    for short in (dict(q=B.head_rows(torch.zeros(3, 3, 128, dtype=BF))), dict(k=B.head_rows(torch.zeros(3, 1, 576, dtype=BF)))):
        with pytest.raises(B.LsError):
            heads_call(**short)
    assert append_call().tokens == 5
    with pytest.raises(B.LsError):
        append_call(key=B.head_rows(torch.zeros(4, 128, dtype=BF)))


def test_a_call_without_operands_is_refused():
    with pytest.raises(B.LsError):
        heads_call(q=None, k=None)
    with pytest.raises(B.LsError):
        append_call(kv=None, key=None)


# ------------------------------------------------------------------------------- pools
def prefix_call(**kw):
    d = dict(q=torch.zeros(2, 8, 576, dtype=BF), kv_pool=torch.zeros(8, 64, 576, dtype=BF), page_table=torch.zeros(2, 4, dtype=torch.int32),
             lens=torch.zeros(2, dtype=torch.int32), o=torch.zeros(2, 8, 512, dtype=BF), lse=torch.zeros(2, 8), scale=1 / 24)
    d.update(kw)
    return B.prefix_attn_args(**d)


POOL_VIEWS = {
    "whole": (torch.zeros(8, 64, 576, dtype=BF), 576),
    "slice of wider rows": (torch.zeros(8, 64, 640, dtype=BF)[:, :, :576], 640),
    "wider rows": (torch.zeros(8, 64, 640, dtype=BF), 640),
    "layer of a stack": (torch.zeros(3, 8, 64, 576, dtype=BF)[1], 576),
    "layer between the rows": (torch.zeros(8, 64, 2, 576, dtype=BF)[:, :, 1], 1152),
    "one page": (torch.zeros(2, 2, 64, 576, dtype=BF)[:1, 0], 576),
}


@pytest.mark.parametrize("view", POOL_VIEWS)
def test_append_and_attention_see_the_same_rows_of_a_pool(view):
    pool, stride = POOL_VIEWS[view]
    a, p = append_call(kv_pool=pool), prefix_call(kv_pool=pool)
    assert a.kv_row_stride == p.row_stride == stride
    assert a.kv_pool == p.kv_pool == pool.data_ptr()


@pytest.mark.parametrize("pool", [
    torch.zeros(8, 2, 64, 576, dtype=BF)[:, 0],              # pages of several layers
    torch.zeros(8, 32, 576, dtype=BF), torch.zeros(512, 576, dtype=BF), torch.zeros(8, 64, 512, dtype=BF),
    torch.zeros(8, 64, 1152, dtype=BF)[:, :, ::2], torch.zeros(64, 8, 576, dtype=BF).transpose(0, 1), torch.zeros(8, 64, 576),
])
def test_pools_that_are_refused(pool):
    for call in (append_call, prefix_call):
        with pytest.raises(B.LsError):
            call(kv_pool=pool)


def test_key_pools():
    a = append_call(key_pool=torch.zeros(5, 64, 128, dtype=torch.uint8), key_scale=torch.zeros(5, 64))
    assert a.num_pages == 5 and a.key_row_stride == 128  # a page id has to exist in both pools
    for bad in (dict(key_pool=torch.zeros(8, 2, 64, 128, dtype=torch.uint8)[:, 0]), dict(key_pool=torch.zeros(8, 64, 64, dtype=torch.uint8)),
                dict(key_pool=None), dict(kv_pool=None), dict(key_scale=torch.zeros(8, 128)[:, ::2]),
                dict(key_scale=torch.zeros(7, 64)), dict(key_scale=torch.zeros(8, 64, dtype=BF))):
        with pytest.raises(B.LsError):
            append_call(**bad)
    assert append_call(kv=None, kv_pool=None).kv.heads == 0 and append_call(key=None, key_pool=None, key_scale=None).key.heads == 0


# ------------------------------------------------------------------------------- positions, lengths, tables
I64 = torch.int64


@pytest.mark.parametrize("pos", [torch.zeros(4, dtype=I64), torch.zeros(4), torch.zeros(8, dtype=torch.int32)[::2]])
def test_positions_are_int32_and_contiguous(pos):
    with pytest.raises(B.LsError):
        heads_call(pos=pos)


@pytest.mark.parametrize("cos_sin", [torch.zeros(100, 64, dtype=torch.float64), torch.zeros(100, 64, dtype=BF), torch.zeros(100, 128)[:, :64],
                                     torch.zeros(100, 32, 2)])
def test_angle_tables_that_are_refused(cos_sin):
    for call in (heads_call, append_call):
        with pytest.raises(B.LsError):
            call(cos_sin=cos_sin)


def test_angle_table_as_given():
    t = torch.zeros(100, 64)
    for a in (heads_call(cos_sin=t), append_call(cos_sin=t)):
        assert (a.max_pos, a.rope_dim, a.cos_sin) == (100, 64, t.data_ptr())


@pytest.mark.parametrize("kw", [
    dict(start=torch.zeros(2, dtype=I64)), dict(start=torch.zeros(1, dtype=torch.int32)), dict(start=torch.zeros(4, dtype=torch.int32)[::2]),
    dict(cu_tokens=torch.tensor([0, 3, 5])), dict(cu_tokens=torch.tensor([0, 3], dtype=torch.int32)),
    dict(page_table=torch.zeros(2, 4, dtype=I64)), dict(page_table=torch.zeros(2, 8, dtype=torch.int32)[:, :4]),
])
def test_append_indices_that_are_refused(kw):
    with pytest.raises(B.LsError):
        append_call(**kw)


@pytest.mark.parametrize("kw", [
    dict(lens=torch.zeros(2, dtype=I64)), dict(lens=torch.zeros(1, dtype=torch.int32)), dict(page_table=torch.zeros(2, 4, dtype=I64)),
    dict(page_table=torch.zeros(2, 8, dtype=torch.int32)[:, :4]), dict(page_table=torch.zeros(1, 4, dtype=torch.int32)),
])
def test_attention_indices_that_are_refused(kw):
    with pytest.raises(B.LsError):
        prefix_call(**kw)


# ------------------------------------------------------------------------------- outputs
U8 = torch.uint8


@pytest.mark.parametrize("kw", [
    dict(q_out=None), dict(q_out=torch.zeros(3, 3, 128, dtype=BF)), dict(q_out=torch.zeros(4, 2, 128, dtype=BF)),
    dict(q_out=torch.zeros(4, 3, 64, dtype=BF)), dict(q_out=torch.zeros(4, 128, dtype=BF)), dict(q_out=torch.zeros(4, 3, 256, dtype=BF)[:, :, ::2]),
    dict(k_out=torch.zeros(3, 1, 576, dtype=BF)), dict(k_out=torch.zeros(4, 2, 576, dtype=BF)),
    dict(q_out=torch.zeros(4, 3, 128, dtype=U8), q_scale=torch.zeros(4, 6)[:, ::2]),
    dict(q_out=torch.zeros(4, 3, 128, dtype=U8), q_scale=torch.zeros(4, 2)),
    dict(q_out=torch.zeros(4, 3, 128, dtype=U8), q_scale=torch.zeros(4, 3, dtype=BF)),
])
def test_outputs_of_head_rows_that_are_refused(kw):
    with pytest.raises(B.LsError):
        heads_call(**kw)


def test_outputs_of_head_rows_as_given():
    t = torch.zeros(3, 9, 128, dtype=U8)
    sc = torch.zeros(9, 3)
    a = heads_call(q_out=t.transpose(0, 1), q_scale=sc)
    assert (a.q_out.token_stride, a.q_out.head_stride, a.q_out.dtype) == (128, 9 * 128, B.LS_E4M3)
    assert (a.q_out.out, a.q_out.scale) == (t.data_ptr(), sc.data_ptr())
    a = heads_call(k=B.head_rows(torch.zeros(4, 576, dtype=BF)), k_out=torch.zeros(4, 640, dtype=BF)[:, :576])
    assert a.k_out.token_stride == 640 and a.k.heads == 1
    a = heads_call(k=None, k_out=None)
    assert a.k.heads == 0 and a.k_out.out is None


@pytest.mark.parametrize("kw", [
    dict(q=torch.zeros(2, 8, 640, dtype=BF)[:, :, :576]), dict(o=torch.zeros(1, 8, 512, dtype=BF)), dict(o=torch.zeros(2, 4, 512, dtype=BF)),
    dict(o=torch.zeros(2, 8, 1024, dtype=BF)[:, :, :512]), dict(lse=torch.zeros(2, 7)), dict(lse=torch.zeros(2, 16)[:, ::2]),
    dict(lse=torch.zeros(2, 8, dtype=BF)),
])
def test_queries_and_outputs_of_the_attention_that_are_refused(kw):
    with pytest.raises(B.LsError):
        prefix_call(**kw)


# ------------------------------------------------------------------------------- devices
@pytest.mark.parametrize("call", [heads_call, append_call, prefix_call])
def test_tensors_that_the_kernel_cannot_reach_are_refused(call):
    with pytest.raises(B.LsError):
        B._check_device(call(), 0)  # pageable host memory


class Elsewhere:
    """Stands for a tensor of device `dev`, or of host memory."""

    def __init__(self, dev, pinned=False):
        self.get_device, self.is_pinned = (lambda: dev), (lambda: pinned)


def test_devices_are_looked_at_once_for_each_device():
    a = prefix_call()
    a._refs = (Elsewhere(1), None, Elsewhere(-1, True))
    with pytest.raises(B.LsError):
        B._check_device(a, 0)
    B._check_device(a, 1)
    assert a._device == 1
    a._refs = (Elsewhere(0),)
    with pytest.raises(B.LsError):
        B._check_device(a, 2)
    B._check_device(B.PrefixAttnArgs(), 0)  # a struct filled in by hand: addresses only


# ------------------------------------------------------------------------------- operands that share memory
@pytest.fixture(scope="module")
def lib():
    from sparse_attention_decode_ls_b200 import build as build_mod
    build_mod.build()
    return B.lib()


def test_outputs_over_the_other_operand_are_refused(lib):
    q, k = torch.zeros(4, 3, 128, dtype=BF), torch.zeros(4, 3, 128, dtype=BF)
    for q_out, k_out in ((k, torch.zeros_like(k)), (torch.zeros_like(q), q), (k, q), (torch.zeros_like(q),) * 2):
        a = heads_call(q=B.head_rows(q), k=B.head_rows(k), q_out=q_out, k_out=k_out)
        assert lib.ls_qk_norm_rope(B.C.byref(a), None) == B.LS_ERR_INVALID_ARG
        assert "other operand" in lib.ls_get_error_string().decode()
    x = torch.zeros(5, 128, dtype=BF)
    pool = torch.zeros(8, 64, 128, dtype=BF)
    a = append_call(kv=B.head_rows(x), key=B.head_rows(torch.zeros(5, 128, dtype=BF)), kv_pool=pool, key_pool=pool, key_scale=None)
    assert lib.ls_cache_append(B.C.byref(a), None) == B.LS_ERR_INVALID_ARG
    assert "other pool" in lib.ls_get_error_string().decode()
