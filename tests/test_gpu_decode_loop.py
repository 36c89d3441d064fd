"""A run of the cache operators as a serving loop uses them: new tokens are appended to the paged
caches, the queries of the step are made, the indexer scores the cache they reach, and the attention
reads it.  A selection as long as the context makes the sparse attention a full one, so the two
attentions have to agree; the whole step is captured in a graph whose replays advance the caches."""
import pytest
import torch

from sparse_attention_decode_ls_b200 import binding as B
from test_gpu_prefix_attn import check as check_attention

pytestmark = pytest.mark.gpu

DEV = "cuda"
SCALE = 1 / 24


def test_append_query_score_select_attend_in_a_graph():
    g = torch.Generator(device=DEV).manual_seed(1)
    Bn, shared, own, k = 3, 4, 4, 512
    num_pages, max_pages = shared + Bn * own, shared + own
    perm = torch.randperm(num_pages, generator=g, device=DEV).to(torch.int32)
    table = torch.cat([perm[:shared].expand(Bn, shared), perm[shared:].view(Bn, own)], 1).contiguous()
    prefix = shared * 64
    cs = torch.cat([f(torch.arange(1024, device=DEV, dtype=torch.float64)[:, None] *
                      10000.0 ** (-torch.arange(0, 64, 2, device=DEV, dtype=torch.float64) / 64)) for f in (torch.cos, torch.sin)], 1).float()
    kv_pool = torch.full((num_pages, 64, 576), float("nan"), dtype=torch.bfloat16, device=DEV)
    key_pool = torch.zeros(num_pages, 64, 128, dtype=torch.uint8, device=DEV)
    key_scale = torch.zeros(num_pages, 64, device=DEV)
    w_kv, w_key = torch.ones(512, device=DEV), torch.ones(128, device=DEV)

    def rows(x):
        return dict(kv=B.head_rows(x[:, :576], norm=B.LS_NORM_RMS, norm_dim=512, weight=w_kv, rope_begin=512, rope_layout=B.LS_ROPE_PAIRS),
                    kv_pool=kv_pool, key=B.head_rows(x[:, 576:], norm=B.LS_NORM_LAYER, weight=w_key, rope_begin=0),
                    key_pool=key_pool, key_scale=key_scale)

    def rand(*s):
        return torch.randn(*s, generator=g, device=DEV).to(torch.bfloat16)

    # prefill: the prefix through request 0's table, then what each request has of its own
    B.ls_cache_append(page_table=table[:1].contiguous(), start=torch.zeros(1, dtype=torch.int32, device=DEV),
                      cu_tokens=torch.tensor([0, prefix], dtype=torch.int32, device=DEV), cos_sin=cs, **rows(rand(prefix, 704)))
    counts = [5, 70, 0]
    lens = torch.full((Bn,), prefix, dtype=torch.int32, device=DEV)
    B.ls_cache_append(page_table=table, start=lens, cu_tokens=torch.tensor([0, 5, 75, 75], dtype=torch.int32, device=DEV), cos_sin=cs,
                      **rows(rand(75, 704)))
    lens += torch.tensor(counts, dtype=torch.int32, device=DEV)

    # one step on fixed buffers
    new = rand(Bn, 704)
    proj_i, proj_a = rand(Bn, 64, 128), rand(Bn, 128, 576)
    q8, qs = torch.zeros(Bn, 64, 128, dtype=torch.uint8, device=DEV), torch.zeros(Bn, 64, device=DEV)
    qa = torch.zeros(Bn, 128, 576, dtype=torch.bfloat16, device=DEV)
    w = rand(Bn, 64)
    scores = torch.zeros(Bn, 64 * max_pages, device=DEV)
    idx = torch.zeros(Bn, k, dtype=torch.int32, device=DEV)
    o1, o2 = (torch.zeros(Bn, 128, 512, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    l1, l2 = (torch.zeros(Bn, 128, device=DEV) for _ in range(2))
    append = B.cache_append_args(page_table=table, start=lens, cos_sin=cs, **rows(new))
    query = B.qk_norm_rope_args(pos=lens, cos_sin=cs, q=B.head_rows(proj_i, norm=B.LS_NORM_RMS, rope_begin=0), q_out=q8, q_scale=qs,
                                k=B.head_rows(proj_a, rope_begin=512, rope_layout=B.LS_ROPE_PAIRS), k_out=qa)
    full = B.prefix_attn_args(q=qa, kv_pool=kv_pool, page_table=table, lens=lens, o=o1, lse=l1, scale=SCALE, prefix_len=prefix)
    sparse = B.attn_args(q=qa, k_rows=kv_pool, sel=idx, o=o2, lse=l2, scale=SCALE, page_table=table)
    ws1 = torch.empty(B.ls_prefix_attn_workspace_size(full), dtype=torch.uint8, device=DEV)
    ws2 = torch.empty(max(256, B.ls_sparse_attn_workspace_size(sparse)), dtype=torch.uint8, device=DEV)

    def step():
        B.ls_cache_append(args=append)
        B.ls_qk_norm_rope(args=query)
        lens.add_(1)
        B.ls_index_score(q=q8, w=w, key_pool=key_pool, page_table=table, lens=lens, scores=scores, q_scale=qs, key_scale=key_scale)
        B.ls_topk_select(scores=scores, lens=lens, idx=idx)
        B.ls_prefix_attn_decode(full, ws1)
        B.ls_sparse_attn_decode(sparse, ws2)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for n in range(2, 70):  # over the ends of pages
        new.copy_(rand(Bn, 704))
        proj_a.copy_(rand(Bn, 128, 576))
        graph.replay()
        if n % 13 and n > 3:
            continue
        torch.cuda.synchronize()
        L = [prefix + c + n for c in counts]
        assert lens.tolist() == L
        for b in range(Bn):
            assert idx[b, : L[b]].tolist() == list(range(L[b])) and (idx[b, L[b]:] == -1).all()
            r = kv_pool[table[b].long()].flatten(0, 1)[: L[b]].double()
            assert r.isfinite().all()
            s = SCALE * (qa[b].double() @ r.T)
            ref = torch.softmax(s, 1) @ r[:, :512]
            assert (o1[b].double() - ref).abs().max() <= 2e-2
            assert (l1[b].double() - s.logsumexp(1)).abs().max() <= 1e-4
        # both round P and o to bf16: two roundings each of values below 4
        assert (o1.float() - o2.float()).abs().max() <= 4 * 2.0 ** -7 and (l1 - l2).abs().max() <= 1e-4
    assert B.ls_check_device_status() == 0


@pytest.mark.parametrize("view", ["slice of wider rows", "layer of a stack", "layer between the rows"])
def test_append_to_a_view_and_attend_over_it(view):
    """A pool that is a view: the attention reads the rows that the append wrote, and nothing else changes."""
    g = torch.Generator(device=DEV).manual_seed(2)
    shape, pick = {"slice of wider rows": ((9, 64, 640), lambda t: t[:, :, :576]),
                   "layer of a stack": ((3, 9, 64, 576), lambda t: t[1]),
                   "layer between the rows": ((9, 64, 2, 576), lambda t: t[:, :, 1])}[view]
    whole = torch.full(shape, 7.0, dtype=torch.bfloat16, device=DEV)
    pool = pick(whole)
    table = torch.randperm(9, generator=g, device=DEV)[:8].to(torch.int32).view(2, 4)
    x = torch.randn(300, 576, generator=g, device=DEV).to(torch.bfloat16)
    lens = [130, 170]
    B.ls_cache_append(page_table=table, start=torch.zeros(2, dtype=torch.int32, device=DEV),
                      cu_tokens=torch.tensor([0, 130, 300], dtype=torch.int32, device=DEV), kv=B.head_rows(x), kv_pool=pool)
    q = torch.randn(2, 16, 576, generator=g, device=DEV).to(torch.bfloat16)
    o, lse = torch.zeros(2, 16, 512, dtype=torch.bfloat16, device=DEV), torch.zeros(2, 16, device=DEV)
    a = B.prefix_attn_args(q=q, kv_pool=pool, page_table=table, lens=torch.tensor(lens, dtype=torch.int32, device=DEV), o=o, lse=lse,
                           scale=SCALE)
    B.ls_prefix_attn_decode(a, torch.empty(max(256, B.ls_prefix_attn_workspace_size(a)), dtype=torch.uint8, device=DEV))
    want = torch.full(shape, 7.0, dtype=torch.bfloat16, device=DEV)
    at = 0
    for b, n in enumerate(lens):
        rows = x[at: at + n]
        pos = torch.arange(n, device=DEV)
        pick(want)[table[b, pos // 64].long(), pos % 64] = rows
        at += n
    assert torch.equal(whole, want)
    check_attention(dict(q=q, pool=pick(want), table=table), o, lse, scale=SCALE, lens=lens)
    assert B.ls_check_device_status() == 0


def test_host_tensors_pinned_or_refused():
    """Index arrays may lie in pinned host memory; what the GPU cannot reach is refused before any launch."""
    g = torch.Generator(device=DEV).manual_seed(4)
    x = torch.randn(5, 2, 128, generator=g, device=DEV)
    cs = torch.randn(10, 64, generator=g, device=DEV)
    pos = torch.arange(5, dtype=torch.int32)
    out, want = torch.zeros_like(x), torch.zeros_like(x)
    B.ls_qk_norm_rope(pos=pos.to(DEV), cos_sin=cs, q=B.head_rows(x, rope_begin=0), q_out=want)
    B.ls_qk_norm_rope(pos=pos.pin_memory(), cos_sin=cs, q=B.head_rows(x, rope_begin=0), q_out=out)
    assert torch.equal(out, want)
    for kw in (dict(pos=pos), dict(cos_sin=cs.cpu()), dict(q=B.head_rows(x.cpu(), rope_begin=0)), dict(q_out=torch.zeros(5, 2, 128)),
               dict(q=B.head_rows(x, norm=B.LS_NORM_RMS, weight=torch.ones(128), rope_begin=0))):
        with pytest.raises(B.LsError):
            B.ls_qk_norm_rope(**dict(dict(pos=pos.to(DEV), cos_sin=cs, q=B.head_rows(x, rope_begin=0), q_out=out), **kw))
    d = dict(q=torch.zeros(1, 8, 576, dtype=torch.bfloat16, device=DEV), kv_pool=torch.zeros(9, 64, 576, dtype=torch.bfloat16, device=DEV),
             page_table=torch.zeros(1, 9, dtype=torch.int32, device=DEV), lens=torch.zeros(1, dtype=torch.int32, device=DEV),
             o=torch.zeros(1, 8, 512, device=DEV), lse=torch.zeros(1, 8, device=DEV), scale=SCALE)
    a = B.prefix_attn_args(**d)
    ws = torch.zeros(max(256, B.ls_prefix_attn_workspace_size(a)), dtype=torch.uint8)
    with pytest.raises(B.LsError):
        B.ls_prefix_attn_decode(a, ws)
    for name in ("q", "kv_pool", "page_table", "lens", "o", "lse"):
        with pytest.raises(B.LsError):
            B.ls_prefix_attn_decode(B.prefix_attn_args(**dict(d, **{name: d[name].cpu()})), ws.to(DEV))
    torch.cuda.synchronize()
    assert B.ls_check_device_status() == 0
