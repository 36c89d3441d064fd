"""Cases, plain forms and exact values of three operators around the paged caches of the
sparse-attention decode: the norm and rotation of query and key heads, the append of new rows to
the paged caches, and the decode attention of a batch whose requests share a long prefix.

``own`` chooses between the plain torch form (32-bit arithmetic, one rounding at the end) and the
library's calls.  Both start from what ``prepare`` made and return the same outputs.
"""
import math

import torch

own = False

PAGE = 64
LATENT, KV_DIM, ROPE = 512, 576, 64   # MLA latent row: 512 dims that are also V, 64 rotated dims
INDEX_HEADS, INDEX_DIM = 64, 128
EPS = 1e-6
E4M3_MAX = 448.0


# ----------------------------------------------------------------------------- cases
def listed():
    return [
        # the queries of one decode step at the benchmark's batch: indexer heads to e4m3 with a scale
        # for each, attention heads rotated in place of their last 64 dims; latency counts
        dict(name="queries of a decode step, 8", op="heads", kind="step", tokens=8, pad=0, dtype="bf16", max_pos=131072),
        # the same for the largest batch of the ragged sweep, its last rows padding
        dict(name="queries of a decode step, 256", op="heads", kind="step", tokens=256, pad=13, dtype="bf16", max_pos=16384),
        # a prefill chunk: indexer queries and its one key head (layer norm with a bias), both to e4m3
        dict(name="indexer heads of a prefill chunk", op="heads", kind="indexer", tokens=8192, pad=0, dtype="bf16", max_pos=131072),
        # float32 heads of the small configuration, whole head rotated, an odd number of tokens
        dict(name="float32 heads, 4097 tokens", op="heads", kind="plain", tokens=4097, pad=0, dtype="f32", max_pos=8192,
             q_heads=16, k_heads=1, dim=128, rope=128, pairs=False),
        # one new token for each of 8 requests: latent row and indexer key
        dict(name="append one token, 8 requests", op="append", batch=8, new=1, dtype="bf16", max_start=16384, ragged=False),
        # one new token for each request of the largest sweep batch
        dict(name="append one token, 256 requests", op="append", batch=256, new=1, dtype="bf16", max_start=4096, ragged=False),
        # a ragged prefill chunk: up to 4096 tokens for each request, some requests with none
        dict(name="append ragged prefill chunk", op="append", batch=16, new=4096, dtype="bf16", max_start=8192, ragged=True),
        # the small float32 configuration: 8 requests, chunks of odd lengths
        dict(name="append float32 rows", op="append", batch=8, new=1000, dtype="f32", max_start=4096, ragged=True),
        # one request with a short context and nothing shared: the smallest call, latency
        dict(name="attention, 1 request of 200", op="prefix", batch=1, heads=128, prefix=0, own_len=200),
        # 16 of 128 heads (one rank of eight), many requests behind one system prompt
        dict(name="attention, 64 x 16 heads, 8192", op="prefix", batch=64, heads=16, prefix=8192, own_len=512),
        # a ragged batch, prefix of no whole number of pages, own parts of up to 4096 tokens
        dict(name="attention, 16 requests, 10007", op="prefix", batch=16, heads=128, prefix=10007, own_len=4096),
        # the benchmark's batch over a shared context of 131072 tokens
        dict(name="attention, 8 requests, 131072", op="prefix", batch=8, heads=128, prefix=131072, own_len=1024),
    ]


def _spread(rng, lo, hi):
    """A whole number from lo to hi, spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["heads", "append", "prefix"])
    if op == "heads":
        kind = rng.choice(["step", "indexer", "plain"])
        c = dict(op=op, kind=kind, dtype="bf16", max_pos=_spread(rng, 4096, 131072))
        if kind == "plain":
            c["dtype"] = rng.choice(["bf16", "f32"])
            c["dim"] = rng.choice([64, 80, 96, 128, 192, 256])
            c["rope"] = rng.choice([c["dim"], c["dim"] // 2, 32])
            c["q_heads"] = rng.choice([1, 8, 12, 16, 40, 64])
            c["k_heads"] = rng.choice([1, 2, 4, 8])
            c["pairs"] = rng.random() < 0.5
            per = (c["q_heads"] + c["k_heads"]) * c["dim"] * (4 if c["dtype"] == "f32" else 2)
            c["tokens"] = _spread(rng, 1, max(1, min(16384, (160 << 20) // per)))
        else:
            c["tokens"] = _spread(rng, 1, 1000 if kind == "step" else 8192)
        c["pad"] = rng.choice([0, 0, c["tokens"] // 10])
        return c
    if op == "append":
        ragged = rng.random() < 0.6
        batch = _spread(rng, 1, 256)
        return dict(op=op, batch=batch, new=_spread(rng, 2, max(2, min(8192, 65536 // batch))) if ragged else 1,
                    dtype=rng.choice(["bf16", "bf16", "f32"]), max_start=_spread(rng, 64, max(64, min(16384, 300000 // batch))),
                    ragged=ragged)
    heads = rng.choice([128, 128, 64, 32, 16, 8, 20])
    batch = _spread(rng, 1, max(1, min(128, 8192 // heads)))
    room = 8 * 128 * 131072 // (batch * heads)
    prefix = rng.choice([0, 1, 1, 1]) * _spread(rng, 100, min(131072, room))
    own_len = _spread(rng, 1, max(1, min(8192, (room - prefix) // 2 + 1, 65536 // batch)))
    return dict(op=op, batch=batch, heads=heads, prefix=prefix, own_len=own_len)


def _dtype(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def _parts(c):
    """The two operands of a "heads" case: heads, dim, norm, rotated dims and output type of each."""
    if c["kind"] == "step":
        return (dict(heads=INDEX_HEADS, dim=INDEX_DIM, norm="rms", begin=0, rope=ROPE, pairs=False, out="e4m3"),
                dict(heads=128, dim=KV_DIM, norm="none", begin=LATENT, rope=ROPE, pairs=True, out="same"))
    if c["kind"] == "indexer":
        return (dict(heads=INDEX_HEADS, dim=INDEX_DIM, norm="rms", begin=0, rope=ROPE, pairs=False, out="e4m3"),
                dict(heads=1, dim=INDEX_DIM, norm="layer", begin=0, rope=ROPE, pairs=False, out="e4m3"))
    p = dict(dim=c["dim"], norm="rms", begin=0, rope=c["rope"], pairs=c["pairs"], out="same")
    return dict(p, heads=c["q_heads"]), dict(p, heads=c["k_heads"])


# ----------------------------------------------------------------------------- inputs
def _angles(max_pos, rope, device):
    """[max_pos, rope] float32: the cosines of a position's rope/2 angles, then their sines."""
    inv = 10000.0 ** (-torch.arange(0, rope, 2, dtype=torch.float64, device=device) / rope)
    a = torch.arange(max_pos, dtype=torch.float64, device=device)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float()


def prepare(case, seed):
    c = case
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device=dev)
    uni = lambda lo, hi, n: torch.randint(lo, hi + 1, (n,), generator=g, device=dev, dtype=torch.int32)
    s = dict(case=c)
    if c["op"] == "heads":
        T, dt = c["tokens"], _dtype(c["dtype"])
        parts = _parts(c)
        width = sum(p["heads"] * p["dim"] for p in parts)
        x = (rnd(T, width) * (0.5 + torch.rand(T, 1, generator=g, device=dev))).to(dt)  # one projection's output
        at = 0
        for n, p in zip("qk", parts):
            s[n] = x[:, at: at + p["heads"] * p["dim"]].unflatten(1, (p["heads"], p["dim"]))
            at += p["heads"] * p["dim"]
            s[n + "_weight"] = (1 + 0.1 * rnd(p["dim"])).to(dt) if p["norm"] != "none" else None
            s[n + "_bias"] = (0.1 * rnd(p["dim"])).to(dt) if p["norm"] == "layer" else None
            e = p["out"] == "e4m3"
            s[n + "_out"] = torch.zeros(T, p["heads"], p["dim"], dtype=torch.uint8 if e else dt, device=dev)
            s[n + "_scale"] = torch.zeros(T, p["heads"], device=dev) if e else None
        s["pos"] = uni(0, c["max_pos"] - 1, T)
        if c["pad"]:
            s["pos"][T - c["pad"]:] = -1
        s["cos_sin"] = _angles(c["max_pos"], parts[0]["rope"], dev)
        return s
    if c["op"] == "append":
        Bn, dt = c["batch"], _dtype(c["dtype"])
        n = uni(0, c["new"], Bn) if c["ragged"] else torch.full((Bn,), c["new"], dtype=torch.int32, device=dev)
        s["start"] = uni(0, c["max_start"], Bn)
        s["cu"] = torch.cat([torch.zeros(1, dtype=torch.int32, device=dev), n.cumsum(0, dtype=torch.int32)])
        T = Bn * c["new"] if not c["ragged"] else (Bn * c["new"] + 1) // 2 + c["new"]  # some rows are padding
        s["cu"].clamp_(max=T)
        max_pages = (c["max_start"] + c["new"] + PAGE - 1) // PAGE
        num_pages = Bn * max_pages
        s["page_table"] = torch.randperm(num_pages, generator=g, device=dev).to(torch.int32).view(Bn, max_pages)
        x = (rnd(T, KV_DIM + INDEX_DIM) * (0.5 + torch.rand(T, 1, generator=g, device=dev))).to(dt)
        s["kv"], s["key"] = x[:, :KV_DIM], x[:, KV_DIM:]
        s["kv_weight"] = (1 + 0.1 * rnd(LATENT)).to(dt)
        s["key_weight"], s["key_bias"] = (1 + 0.1 * rnd(INDEX_DIM)).to(dt), (0.1 * rnd(INDEX_DIM)).to(dt)
        s["cos_sin"] = _angles(c["max_start"] + c["new"], ROPE, dev)
        s["kv_pool"] = rnd(num_pages, PAGE, KV_DIM).to(dt)
        e = c["dtype"] != "f32"
        s["key_pool"] = (torch.randint(0, 120, (num_pages, PAGE, INDEX_DIM), generator=g, device=dev, dtype=torch.uint8) if e
                         else rnd(num_pages, PAGE, INDEX_DIM))
        s["key_scale"] = torch.rand(num_pages, PAGE, generator=g, device=dev) if e else None
        return s
    Bn, H, P = c["batch"], c["heads"], c["prefix"]
    shared = P // PAGE  # whole pages that every request's table begins with
    rest = P % PAGE + c["own_len"]
    own_pages = (rest + PAGE - 1) // PAGE
    num_pages = shared + Bn * own_pages
    perm = torch.randperm(num_pages, generator=g, device=dev).to(torch.int32)
    s["page_table"] = torch.cat([perm[:shared].expand(Bn, shared), perm[shared:].view(Bn, own_pages)], 1).contiguous()
    s["lens"] = P + uni(min(1, c["own_len"]), c["own_len"], Bn)
    s["lens"][0] = P + c["own_len"]
    s["q"] = (2 * rnd(Bn, H, KV_DIM)).to(torch.bfloat16)
    s["pool"] = rnd(num_pages, PAGE, KV_DIM).to(torch.bfloat16)
    # what no request has written yet holds anything at all
    at = shared * PAGE + torch.arange(own_pages * PAGE, device=dev)
    unwritten = at[None, :] >= s["lens"][:, None]
    s["pool"][s["page_table"][:, shared:].long()] = torch.where(
        unwritten.view(Bn, own_pages, PAGE, 1), float("nan"), s["pool"][s["page_table"][:, shared:].long()])
    return s


# ----------------------------------------------------------------------------- plain forms
def _norm_rope(x, norm, norm_dim, weight, bias, cos_sin, begin, rope, pairs):
    """Rows [T, heads, dim]: norm of the first norm_dim dims, then the rotation of [begin, begin + rope)."""
    x = x.float()
    if norm != "none":
        y = x[..., :norm_dim]
        if norm == "layer":
            y = y - y.mean(-1, keepdim=True)
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * weight.float()
        if bias is not None:
            y = y + bias.float()
        x = torch.cat([y, x[..., norm_dim:]], -1)
    r = x[..., begin: begin + rope]
    a, b = (r[..., 0::2], r[..., 1::2]) if pairs else r.chunk(2, -1)
    co, si = cos_sin[:, None, :].chunk(2, -1)
    a, b = a * co - b * si, b * co + a * si
    r = torch.stack([a, b], -1).flatten(-2) if pairs else torch.cat([a, b], -1)
    return torch.cat([x[..., :begin], r, x[..., begin + rope:]], -1)


def _to_e4m3(y):
    scale = y.abs().amax(-1).clamp_min(1e-12) / E4M3_MAX
    return (y / scale[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8), scale


def _plain_head(s, n, p, live, cs):
    y = _norm_rope(s[n], p["norm"], p["dim"], s[n + "_weight"], s[n + "_bias"], cs, p["begin"], p["rope"], p["pairs"])
    out, scale = s[n + "_out"], s[n + "_scale"]
    if p["out"] == "e4m3":
        y, sc = _to_e4m3(y)
        scale.copy_(torch.where(live[:, None], sc, scale))
    out.copy_(torch.where(live[:, None, None], y.to(out.dtype), out))


def _plain_heads(s):
    q, k = _parts(s["case"])
    live = s["pos"] >= 0
    cs = s["cos_sin"][s["pos"].clamp_min(0).long()]
    _plain_head(s, "q", q, live, cs)
    _plain_head(s, "k", k, live, cs)


def _rows_of(s):
    """(row, position, pool slot) of every new token that belongs to a request."""
    row = torch.arange(s["kv"].shape[0], device=s["kv"].device)
    row = row[row < s["cu"][-1]]
    req = torch.searchsorted(s["cu"][1:].contiguous(), row.to(torch.int32), right=True)
    pos = (s["start"][req] + row - s["cu"][req]).long()
    return row, pos, s["page_table"][req, pos // PAGE].long() * PAGE + pos % PAGE


def _plain_append(s):
    row, pos, slot = _rows_of(s)
    cs = s["cos_sin"][pos]
    kv = _norm_rope(s["kv"][row, None], "rms", LATENT, s["kv_weight"], None, cs, LATENT, ROPE, True)[:, 0]
    key = _norm_rope(s["key"][row, None], "layer", INDEX_DIM, s["key_weight"], s["key_bias"], cs, 0, ROPE, False)[:, 0]
    s["kv_pool"].view(-1, KV_DIM)[slot] = kv.to(s["kv_pool"].dtype)
    if s["key_scale"] is not None:
        key, scale = _to_e4m3(key)
        s["key_scale"].view(-1)[slot] = scale
    s["key_pool"].view(-1, INDEX_DIM)[slot] = key


def _plain_prefix(s):
    q, lens, table, pool = s["q"].float() / math.sqrt(KV_DIM), s["lens"].long(), s["page_table"].long(), s["pool"]
    Bn, H, _ = q.shape
    shared = s["case"]["prefix"] // PAGE
    n = shared * PAGE
    kp = pool[table[0, :shared]].view(n, KV_DIM).float()
    ko = pool[table[:, shared:]].view(Bn, -1, KV_DIM)
    seen = n + torch.arange(ko.shape[1], device=q.device)[None, :] < lens[:, None]
    ko = torch.where(seen[:, :, None], ko, 0).float()
    sp = (q.view(Bn * H, KV_DIM) @ kp.T).view(Bn, H, n)
    so = torch.where(seen[:, None, :], q @ ko.transpose(1, 2), -math.inf)
    m = torch.cat([sp, so], 2).amax(2, keepdim=True)
    ep, eo = torch.exp(sp - m), torch.exp(so - m)
    total = ep.sum(2, keepdim=True) + eo.sum(2, keepdim=True)
    o = (ep.view(Bn * H, n) @ kp[:, :LATENT]).view(Bn, H, LATENT) + eo @ ko[:, :, :LATENT]
    return (o / total).to(torch.bfloat16), (m + torch.log(total))[..., 0]


# ----------------------------------------------------------------------------- the library's calls
def _own_heads(s):
    from sparse_attention_decode_ls_b200 import binding as B
    norms = {"none": B.LS_NORM_NONE, "rms": B.LS_NORM_RMS, "layer": B.LS_NORM_LAYER}
    rows = [B.head_rows(s[n], norm=norms[p["norm"]], weight=s[n + "_weight"], bias=s[n + "_bias"], eps=EPS, rope_begin=p["begin"],
                        rope_layout=B.LS_ROPE_PAIRS if p["pairs"] else B.LS_ROPE_HALVES) for n, p in zip("qk", _parts(s["case"]))]
    B.ls_qk_norm_rope(pos=s["pos"], cos_sin=s["cos_sin"], q=rows[0], q_out=s["q_out"], q_scale=s["q_scale"],
                      k=rows[1], k_out=s["k_out"], k_scale=s["k_scale"])


def _own_append(s):
    from sparse_attention_decode_ls_b200 import binding as B
    kv = B.head_rows(s["kv"], norm=B.LS_NORM_RMS, norm_dim=LATENT, weight=s["kv_weight"], eps=EPS, rope_begin=LATENT,
                     rope_layout=B.LS_ROPE_PAIRS)
    key = B.head_rows(s["key"], norm=B.LS_NORM_LAYER, weight=s["key_weight"], bias=s["key_bias"], eps=EPS, rope_begin=0,
                      rope_layout=B.LS_ROPE_HALVES)
    B.ls_cache_append(page_table=s["page_table"], start=s["start"], cu_tokens=s["cu"] if s["case"]["ragged"] else None,
                      cos_sin=s["cos_sin"], kv=kv, kv_pool=s["kv_pool"], key=key, key_pool=s["key_pool"], key_scale=s["key_scale"])


def _own_prefix(s):
    from sparse_attention_decode_ls_b200 import binding as B
    q = s["q"]
    o = torch.empty(q.shape[0], q.shape[1], LATENT, dtype=torch.bfloat16, device=q.device)
    lse = torch.empty(q.shape[0], q.shape[1], device=q.device)
    a = B.prefix_attn_args(q=q, kv_pool=s["pool"], page_table=s["page_table"], lens=s["lens"], prefix_len=s["case"]["prefix"], o=o,
                           lse=lse, scale=1 / math.sqrt(KV_DIM))
    ws = torch.empty(B.ls_prefix_attn_workspace_size(a), dtype=torch.uint8, device=q.device)
    B.ls_prefix_attn_decode(a, ws)
    return o, lse


def run(state):
    s = state
    op = s["case"]["op"]
    if op == "prefix":
        o, lse = _own_prefix(s) if own else _plain_prefix(s)
        return {"o": o, "lse": lse}
    if op == "heads":
        if own:
            _own_heads(s)
        else:
            _plain_heads(s)
        out = {}
        for n in "qk":
            e = s[n + "_scale"] is not None
            out[n] = s[n + "_out"].view(torch.float8_e4m3fn) if e else s[n + "_out"]
            if e:
                out[n + "_scale"] = s[n + "_scale"]
        return out
    if own:
        _own_append(s)
    else:
        _plain_append(s)
    out = {"kv_pool": s["kv_pool"], "key_pool": s["key_pool"]}
    if s["key_scale"] is not None:
        out["key_pool"], out["key_scale"] = s["key_pool"].view(torch.float8_e4m3fn), s["key_scale"]
    return out


# ----------------------------------------------------------------------------- work and exact values
def work(case):
    c = case
    if c["op"] == "heads":
        size = 4 if c["dtype"] == "f32" else 2
        T = c["tokens"] - c["pad"]
        values = [p["heads"] * p["dim"] for p in _parts(c)]
        rope = _parts(c)[0]["rope"]
        wide = sum(v * (1 if p["out"] == "e4m3" else size) + (4 * p["heads"] if p["out"] == "e4m3" else 0) for v, p in zip(values, _parts(c)))
        return {"bytes": T * (sum(values) * size + wide + 4 * rope + 4), "flops": 10 * T * sum(values)}
    if c["op"] == "append":
        size = 4 if c["dtype"] == "f32" else 2
        T = c["batch"] * (c["new"] / 2 if c["ragged"] else c["new"])
        key = INDEX_DIM * size if c["dtype"] == "f32" else INDEX_DIM + 4
        return {"bytes": T * ((KV_DIM + INDEX_DIM) * size + KV_DIM * size + key + 4 * ROPE) + 8 * c["batch"],
                "flops": 10 * T * (KV_DIM + INDEX_DIM)}
    tail = c["batch"] * (c["prefix"] % PAGE + c["own_len"] / 2)
    whole = c["prefix"] // PAGE * PAGE
    rows = c["batch"] * c["heads"]
    return {"bytes": (whole + tail) * KV_DIM * 2 + rows * (KV_DIM * 2 + LATENT * 2 + 4) + 4 * (whole + tail) / PAGE,
            "flops": 2 * (KV_DIM + LATENT) * c["heads"] * (c["batch"] * whole + tail)}


def _exact_rows(x, norm, n, weight, bias, pos, rope, begin, pairs):
    """As the definition says, in 64 bits: the rotation as a product of complex numbers, angles from the positions."""
    x = x.double().clone()
    if norm != "none":
        head = x[..., :n]
        if norm == "layer":
            x[..., :n] = (head - head.mean(-1, keepdim=True)) / (head.var(-1, unbiased=False, keepdim=True) + EPS).sqrt()
        else:
            x[..., :n] = head / (head.pow(2).sum(-1, keepdim=True) / n + EPS).sqrt()
        x[..., :n] *= weight.double()
        if bias is not None:
            x[..., :n] += bias.double()
    i = torch.arange(rope // 2, device=x.device)
    first = begin + (2 * i if pairs else i)
    second = first + (1 if pairs else rope // 2)
    angle = pos.double()[:, None] * 10000.0 ** (-2 * i.double() / rope)
    z = torch.complex(x[..., first], x[..., second]) * torch.polar(torch.ones_like(angle), angle)[:, None]
    x[..., first], x[..., second] = z.real, z.imag
    return x


def _exact_scale(y):
    """The scale of each row, and the rows over their scale, before the rounding to e4m3."""
    sc = torch.maximum(y.abs().amax(-1), torch.tensor(1e-12, dtype=torch.float64, device=y.device)) / E4M3_MAX
    return y / sc.unsqueeze(-1), sc


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "heads":
        dead = s["pos"] < 0
        out = {}
        for n, p in zip("qk", _parts(case)):
            y = _exact_rows(s[n], p["norm"], p["dim"], s[n + "_weight"], s[n + "_bias"], s["pos"], p["rope"], p["begin"], p["pairs"])
            if p["out"] == "e4m3":
                y, sc = _exact_scale(y)
                sc[dead] = 0
                out[n + "_scale"] = sc
            y[dead] = 0
            out[n] = y
        return out
    if case["op"] == "append":
        cu, start = s["cu"].tolist(), s["start"].tolist()
        req = torch.tensor([b for b in range(case["batch"]) for _ in range(cu[b + 1] - cu[b])], device="cuda", dtype=torch.int64)
        pos = torch.tensor([start[b] + i for b in range(case["batch"]) for i in range(cu[b + 1] - cu[b])], device="cuda", dtype=torch.int64)
        n = len(pos)
        page, line = s["page_table"][req, pos // PAGE].long(), pos % PAGE
        kv = s["kv_pool"].double()
        kv[page, line] = _exact_rows(s["kv"][:n, None], "rms", LATENT, s["kv_weight"], None, pos, ROPE, LATENT, True)[:, 0]
        y = _exact_rows(s["key"][:n, None], "layer", INDEX_DIM, s["key_weight"], s["key_bias"], pos, ROPE, 0, False)[:, 0]
        if s["key_scale"] is None:
            key = s["key_pool"].double()
            key[page, line] = y
            return {"kv_pool": kv, "key_pool": key}
        key, scale = s["key_pool"].view(torch.float8_e4m3fn).double(), s["key_scale"].double()
        key[page, line], scale[page, line] = _exact_scale(y)
        return {"kv_pool": kv, "key_pool": key, "key_scale": scale}
    o = torch.empty(*s["q"].shape[:2], LATENT, dtype=torch.float64, device="cuda")
    lse = torch.empty(*s["q"].shape[:2], dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["lens"].tolist()):
        rows = s["pool"][s["page_table"][b].long()].flatten(0, 1)[:n].double()
        logits = rows @ s["q"][b].double().T / KV_DIM ** 0.5  # [n, heads]
        lse[b] = logits.logsumexp(0)
        o[b] = (logits - lse[b]).exp().T @ rows[:, :LATENT]
    return {"o": o, "lse": lse}
