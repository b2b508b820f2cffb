"""Workloads of the operators around the 8-bit latent cache: their inputs, their
plain form in elementary torch operations, the library's calls, and the
definition in 64 bits.

Operators (`op` of a case):

* ``rope``   RMS norm of every query and key head and the rotation by position,
             in one pass (``train`` adds the backward pass: gradients of the
             rows and of the norm weights);
* ``write``  quantising the step's new cache rows (attention rows and indexer
             keys) to e4m3 as they are written to their places, and the
             indexer's queries with them;
* ``read``   reading a range of a quantised cache back as BF16 rows;
* ``attn``   attention of all heads over the 8-bit cache (one e4m3 row and one
             scale per token, shared by the heads), over a selection
             (``k`` > 0) or over every visible key (``k`` = 0).

Sequence b holds L_b keys, query t of T sits at position L_b - T + t.  With
``page`` > 0 the caches are pools of pages found through a block table.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
MIN_EXP = -48          # smallest exponent of a power-of-two row scale


# ------------------------------------------------------------------ cases

def _rope(name, B, T, S, Hq, Hk, D, norm, rope, inter=False, train=False, ragged=False):
    c = dict(op="rope", B=B, T=T, S=S, Hq=Hq, Hk=Hk, D=D, norm=norm, rope=rope, inter=inter, train=train,
             ragged=ragged)
    return dict(c, name=name) if name else c


def _write(name, B, T, S, d_k, H_I, D_I, page=0, ragged=False):
    c = dict(op="write", B=B, T=T, S=S, d_k=d_k, H_I=H_I, D_I=D_I, page=page, ragged=ragged)
    return dict(c, name=name) if name else c


def _read(name, B, S, begin, count, d_k, D_I, page=0, ragged=False):
    c = dict(op="read", B=B, T=1, S=S, begin=begin, count=count, d_k=d_k, D_I=D_I, page=page, ragged=ragged)
    return dict(c, name=name) if name else c


def _attn(name, B, T, S, H, k, d_k=576, page=0, ragged=False, decode=False):
    c = dict(op="attn", B=B, T=T, S=S, H=H, k=k, d_k=d_k, page=page, ragged=ragged, decode=decode)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one new token for each of eight sequences at 128K: queries of 128 heads and the one shared key row
        _rope("rope_decode_b8", 8, 1, 131072, 128, 1, 576, 512, 64),
        # the whole query side of an 8K prefill
        _rope("rope_prefill_8k", 1, 8192, 8192, 128, 1, 576, 512, 64),
        # a training pass over two odd-length sequences, MLA rows
        _rope("rope_train_mla", 2, 1031, 1031, 128, 1, 576, 512, 64, train=True),
        # a training pass over the indexer's heads, whole rows normalised, interleaved pairs
        _rope("rope_train_index", 4, 1024, 4096, 64, 1, 128, 128, 64, inter=True, train=True, ragged=True),
        # a decode step of 32 sequences of different lengths appends to a paged cache
        _write("write_decode_b32", 32, 1, 2048, 576, 64, 128, page=64, ragged=True),
        # an 8K prefill fills its cache
        _write("write_prefill_8k", 1, 8192, 8192, 576, 64, 128),
        # a short range of three ragged sequences out of small pages
        _read("read_chunk", 3, 2000, 131, 517, 576, 128, page=16, ragged=True),
        # the whole prefix of four 32K sequences
        _read("read_prefix_32k", 4, 32768, 0, 32768, 576, 128, page=64),
        # the 128K decode step's attention over its selection
        _attn("attn_decode_128k_b8", 8, 1, 131072, 128, 2048, decode=True),
        # a ragged decode batch of 32 over paged caches
        _attn("attn_decode_paged_b32", 32, 1, 32768, 128, 2048, page=64, ragged=True, decode=True),
        # one query block of the 8K prefill over its selection
        _attn("attn_prefill_8k", 1, 2048, 8192, 128, 2048),
        # a short ragged prefill over every visible key
        _attn("attn_dense_short", 2, 769, 1537, 128, 0, ragged=True),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "rope", "write", "read", "attn", "attn", "attn"])
    ragged = rng.random() < 0.5
    page = rng.choice([0, 0, 16, 64, 128])
    if op == "rope":
        D, norm, rope = rng.choice([(576, 512, 64), (576, 576, 64), (80, 64, 16), (128, 128, 64), (128, 0, 64),
                                    (64, 64, 0), (32, 32, 32)])
        tokens = _log(rng, 1, 8192)
        B = min(tokens, _log(rng, 1, 16))
        T = max(1, tokens // B)
        train = rng.random() < 0.5
        if train:
            T = max(1, min(T, 2062 // B))
        S = max(T, _log(rng, max(T, 2), 262144))
        return _rope("", B, T, S, 8 * rng.randint(1, 16), rng.choice([1, 1, 1, 2]), D, norm, rope,
                     rng.random() < 0.5, train, ragged)
    if op == "write":
        tokens = _log(rng, 1, 8192)
        B = min(tokens, _log(rng, 1, 32))
        T = max(1, tokens // B)
        S = max(T, _log(rng, max(T, 16), max(T, 65536 // B)))
        return _write("", B, T, S, rng.choice([576, 576, 80]), rng.choice([4, 8, 16, 32, 64]),
                      rng.choice([32, 64, 128]), page, ragged)
    if op == "read":
        B = _log(rng, 1, 16)
        S = _log(rng, 16, 131072 // B)
        begin = rng.randint(0, S // 2)
        count = _log(rng, 1, S - begin)
        return _read("", B, S, begin, count, rng.choice([576, 576, 80]), rng.choice([32, 64, 128]), page, ragged)
    H = 8 * rng.randint(1, 16)
    d_k = rng.choice([576, 576, 576, 80])
    if rng.random() < 0.5:          # decode
        B = _log(rng, 1, 32)
        if rng.random() < 0.7:
            S = _log(rng, 16, 1048576 // B)
            return _attn("", B, 1, S, H, _log(rng, 1, 2048), d_k, page, ragged, True)
        return _attn("", B, 1, _log(rng, 1, 65536 // B), H, 0, d_k, page, ragged, True)
    B = _log(rng, 1, 4)
    if rng.random() < 0.6:          # a block of queries over a selection
        T = _log(rng, 2, 1024 // B)
        S = max(T, _log(rng, max(T, 64), 32768 // B))
        return _attn("", B, T, S, H, _log(rng, 16, 2048), d_k, page, ragged)
    T = _log(rng, 2, 1024 // B)
    S = max(T, min(2048, _log(rng, T, 2048)))
    return _attn("", B, T, S, H, 0, d_k, page, ragged)


# ------------------------------------------------------------------ inputs

def _dv(d_k):
    return 512 if d_k == 576 else 64


def _pow2_exponent(amax):
    """Smallest e >= MIN_EXP with amax <= 448 * 2^e."""
    m, x = torch.frexp(amax)                     # amax = m * 2^x, m in [0.5, 1); 448 = 0.875 * 2^9
    e = x - 9 + (m > 0.875).int()
    return torch.where(amax > 0, e, torch.full_like(e, MIN_EXP)).clamp(min=MIN_EXP)


def _pow2(e):
    """2^e in float32, exactly (e: int32, a normal number's exponent)."""
    return ((e + 127) << 23).view(torch.float32)


def _quantise(x):
    """Rows of x (float32, over the last axis) as e4m3 values and their power-of-two scales."""
    e = _pow2_exponent(x.abs().amax(-1))
    y = (x * _pow2(-e).unsqueeze(-1)).clamp(-E4M3_MAX, E4M3_MAX)
    return y.to(torch.float8_e4m3fn), _pow2(e)


def _layout(st, c, g):
    """Lengths and the block table of a case, on the GPU."""
    B, T, S, page = c["B"], c["T"], c["S"], c.get("page", 0)
    lens = torch.full((B,), S, dtype=torch.int32, device="cuda")
    if c["ragged"]:
        lo = max(T, S // 2)
        lens = (lo + torch.randint(0, S - lo + 1, (B,), generator=g, device="cuda")).int()
    st["lens"] = lens
    st["pool_rows"] = B * S
    st["table"] = None
    if page:
        per = (S + page - 1) // page
        pages = B * per + 3
        st["pool_rows"] = pages * page
        st["pages"] = pages
        st["table"] = torch.randperm(pages, generator=g, device="cuda")[:B * per].view(B, per).int()


def _cache(n, d, g):
    """n quantised cache rows: N(0, 1) columns, token norms spread by e^(N(0, 1) / 2)."""
    q = torch.empty(n, d, dtype=torch.uint8, device="cuda")
    s = torch.empty(n, dtype=torch.float32, device="cuda")
    for i in range(0, n, 1 << 18):
        x = torch.randn(min(n - i, 1 << 18), d, generator=g, device="cuda")
        x *= torch.exp(0.5 * torch.randn(x.shape[0], 1, generator=g, device="cuda"))
        b, e = _quantise(x)
        q[i:i + x.shape[0]] = b.view(torch.uint8)
        s[i:i + x.shape[0]] = e
    return q, s


def _bf16(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda").bfloat16()


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    st = {"c": c}
    B, T, S = c["B"], c["T"], c["S"]
    _layout(st, c, g)
    if c["op"] == "rope":
        for n, H in (("q", c["Hq"]), ("k", c["Hk"])):
            st[n] = _bf16(g, B, T, H, c["D"])
            st[n + "_w"] = 1 + 0.25 * torch.randn(c["norm"], generator=g, device="cuda") if c["norm"] else None
            st[n + "_out"] = torch.empty_like(st[n])
            if c["train"]:
                st["g" + n] = _bf16(g, B, T, H, c["D"])
                st["d" + n] = torch.empty_like(st[n])
                st["d" + n + "_w"] = torch.zeros(c["norm"], device="cuda")
        i = torch.arange(c["rope"] // 2, device="cuda", dtype=torch.float64)
        st["freq"] = (10000.0 ** (-2 * i / max(1, c["rope"]))).float()
        st["eps"] = 1e-6
    elif c["op"] == "write":
        st["kv"] = _bf16(g, B, T, c["d_k"])
        st["k_I"] = _bf16(g, B, T, c["D_I"])
        st["q_I"] = _bf16(g, B, T, c["H_I"], c["D_I"])
        st["kv8"], st["kv_scale"] = _cache(st["pool_rows"], c["d_k"], g)
        st["kI8"], st["kI_scale"] = _cache(st["pool_rows"], c["D_I"], g)
        st["qI8"] = torch.empty(B, T, c["H_I"], c["D_I"], dtype=torch.uint8, device="cuda")
        st["qI_scale"] = torch.empty(B, T, c["H_I"], device="cuda")
    elif c["op"] == "read":
        st["kv8"], st["kv_scale"] = _cache(st["pool_rows"], c["d_k"], g)
        st["kI8"], st["kI_scale"] = _cache(st["pool_rows"], c["D_I"], g)
        # rows at or past a sequence's length stay as they are
        st["kv_out"] = torch.zeros(B, c["count"], c["d_k"], dtype=torch.bfloat16, device="cuda")
        st["kI_out"] = torch.zeros(B, c["count"], c["D_I"], dtype=torch.bfloat16, device="cuda")
    else:
        H, k = c["H"], c["k"]
        st["q"] = _bf16(g, B, T, H, c["d_k"])
        st["kv8"], st["kv_scale"] = _cache(st["pool_rows"], c["d_k"], g)
        st["out"] = torch.empty(B, T, H, _dv(c["d_k"]), dtype=torch.bfloat16, device="cuda")
        st["lse"] = torch.empty(B, T, H, device="cuda")
        st["tau"] = 1 / math.sqrt(c["d_k"])
        if k:
            pos = st["lens"].view(B, 1, 1) - T + torch.arange(T, device="cuda").view(1, T, 1)
            u = torch.rand(B, T, S, generator=g, device="cuda")
            u.masked_fill_(torch.arange(S, device="cuda").view(1, 1, S) > pos, -1.0)
            v, i = u.topk(min(k, S), dim=-1)
            st["idx"] = torch.full((B, T, k), -1, dtype=torch.int32, device="cuda")
            st["idx"][..., :i.shape[-1]] = torch.where(v >= 0, i, -1).int()
    if own:
        _plan(st)
    return st


# ------------------------------------------------------------------ the library's calls

def _plan(st):
    """What a program keeps between its calls: the shape, the norm's description, workspaces."""
    from long_context_05_b200 import dsa
    c = st["c"]
    f = dict(B=c["B"], T=c["T"], S=c["S"], H_I=c.get("H_I", 4), D_I=c.get("D_I", 32), H=c.get("H", 8),
             d_k=c.get("d_k", 576), d_v=_dv(c.get("d_k", 576)), k=max(1, c.get("k", 1)), q_block=c["T"])
    paged = {}
    if c.get("page"):
        paged = dict(page_size=c["page"], num_pages=st["pages"], block_table=st["table"])
    st["dsa"] = dsa
    st["shape"] = dsa.make_shape(None, mode=dsa.DSA_DECODE if c.get("decode") else dsa.DSA_PREFILL,
                                 seqlens=st["lens"] if c["ragged"] else None, **paged, **f)
    if c["op"] == "rope":
        st["nr"] = dsa.make_norm_rope(Hq=c["Hq"], Hk=c["Hk"], D=c["D"], norm_cols=c["norm"], rope_cols=c["rope"],
                                      interleaved=c["inter"], eps=st["eps"], q_weight=st["q_w"], k_weight=st["k_w"],
                                      inv_freq=st["freq"] if c["rope"] else None)
        if c["train"]:
            st["ws"] = dsa.alloc_norm_rope_workspace(st["shape"], st["nr"])
    elif c["op"] == "attn":
        st["ws"] = dsa.alloc_workspace8(st["shape"])


def _run_own(st):
    c, dsa, sh = st["c"], st["dsa"], st["shape"]
    if c["op"] == "rope":
        dsa.norm_rope(sh, st["nr"], st["q"], st["k"], st["q_out"], st["k_out"])
        if c["train"]:
            dsa.norm_rope_backward(sh, st["nr"], st["q"], st["k"], st["gq"], st["gk"], st["dq"], st["dk"],
                                   st["dq_w"], st["dk_w"], st["ws"])
    elif c["op"] == "write":
        dsa.cache_write(sh, kv=st["kv"], kv8=st["kv8"], kv_scale=st["kv_scale"],
                        k_I=st["k_I"], kI8=st["kI8"], kI_scale=st["kI_scale"],
                        q_I=st["q_I"], qI8=st["qI8"], qI_scale=st["qI_scale"])
    elif c["op"] == "read":
        dsa.cache_read(sh, c["begin"], c["count"], kv8=st["kv8"], kv_scale=st["kv_scale"], kv=st["kv_out"],
                       kI8=st["kI8"], kI_scale=st["kI_scale"], k_I=st["kI_out"])
    elif c["k"]:
        dsa.sparse_attn8(sh, st["q"], st["kv8"], st["kv_scale"], st["idx"], st["out"], st["lse"], st["ws"])
    else:
        dsa.dense_attn8(sh, st["q"], st["kv8"], st["kv_scale"], st["out"], st["lse"], st["ws"])


# ------------------------------------------------------------------ the plain form

def _positions(st):
    c = st["c"]
    return st["lens"].view(-1, 1).long() - c["T"] + torch.arange(c["T"], device="cuda")     # [B, T]


def _cache_rows(st, s):
    """Pool rows of tokens s [B, ...] of each sequence."""
    c = st["c"]
    b = torch.arange(c["B"], device="cuda").view([-1] + [1] * (s.dim() - 1))
    if st["table"] is None:
        return b * c["S"] + s
    return st["table"][b, s // c["page"]].long() * c["page"] + s % c["page"]


def _rotate(st, y, back):
    """Rotate the last `rope` columns of y [B, T, H, D] by position (by the opposite angle when back)."""
    c = st["c"]
    r = c["rope"]
    if not r:
        return y
    a = _positions(st).double().unsqueeze(-1) * st["freq"].double()
    cos, sin = a.cos().float().unsqueeze(2), a.sin().float().unsqueeze(2)
    sin = -sin if back else sin
    head, tail = y[..., :-r], y[..., -r:]
    if c["inter"]:
        u, v = tail[..., 0::2], tail[..., 1::2]
        tail = torch.stack((u * cos - v * sin, u * sin + v * cos), -1).flatten(-2)
    else:
        u, v = tail[..., :r // 2], tail[..., r // 2:]
        tail = torch.cat((u * cos - v * sin, u * sin + v * cos), -1)
    return torch.cat((head, tail), -1)


def _norm_rope(st, n):
    c = st["c"]
    x = st[n].float()
    m = c["norm"]
    if m:
        z = x[..., :m]
        x = torch.cat((z * torch.rsqrt(z.square().mean(-1, keepdim=True) + st["eps"]) * st[n + "_w"], x[..., m:]), -1)
    return _rotate(st, x, False).bfloat16()


def _norm_rope_back(st, n):
    c = st["c"]
    m = c["norm"]
    g = _rotate(st, st["g" + n].float(), True)
    if not m:
        return g.bfloat16(), st["d" + n + "_w"]
    x, gz = st[n].float()[..., :m], g[..., :m]
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + st["eps"])
    wg = gz * st[n + "_w"]
    dx = r * (wg - x * r.square() * (wg * x).mean(-1, keepdim=True))
    return torch.cat((dx, g[..., m:]), -1).bfloat16(), (gz * x * r).sum((0, 1, 2), dtype=torch.float64).float()


def _run_write(st):
    rows = _cache_rows(st, _positions(st)).flatten()
    for src, dst, sc in (("kv", "kv8", "kv_scale"), ("k_I", "kI8", "kI_scale")):
        b, e = _quantise(st[src].float().flatten(0, 1))
        st[dst][rows] = b.view(torch.uint8)
        st[sc][rows] = e
    b, e = _quantise(st["q_I"].float())
    st["qI8"].copy_(b.view(torch.uint8))
    st["qI_scale"].copy_(e)


def _run_read(st):
    c = st["c"]
    s = (c["begin"] + torch.arange(c["count"], device="cuda")).expand(c["B"], -1)
    seen = (s < st["lens"].view(-1, 1)).unsqueeze(-1)
    rows = _cache_rows(st, s)
    for src, sc, dst in (("kv8", "kv_scale", "kv_out"), ("kI8", "kI_scale", "kI_out")):
        x = st[src][rows].view(torch.float8_e4m3fn).float() * st[sc][rows].unsqueeze(-1)
        st[dst].copy_(torch.where(seen, x.bfloat16(), st[dst]))


def _softmax_v(l, v):
    """Outputs and log-sum-exps of logits l [.., H, n] (-inf: not a key) over values v [.., n, d_v]."""
    m = l.amax(-1, keepdim=True)
    p = torch.exp(l - torch.where(m == -math.inf, torch.zeros_like(m), m))
    z = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(z > 0, z, torch.ones_like(z))
    return o.bfloat16(), (m + z.log()).squeeze(-1)


def _run_attn(st):
    c = st["c"]
    B, T, H, dk, dv = c["B"], c["T"], c["H"], c["d_k"], _dv(c["d_k"])
    if c["k"]:
        idx = st["idx"].long()
        rows = _cache_rows(st, idx.clamp(min=0)).view(B * T, -1)
        kv = st["kv8"][rows].view(torch.float8_e4m3fn).float() * st["kv_scale"][rows].unsqueeze(-1)
        l = torch.matmul(st["q"].float().view(B * T, H, dk), kv.transpose(1, 2)) * st["tau"]
        l.masked_fill_((idx < 0).view(B * T, 1, -1), -math.inf)
        o, lse = _softmax_v(l, kv[..., :dv])
    else:
        s = torch.arange(c["S"], device="cuda").expand(B, -1)
        rows = _cache_rows(st, s)
        kv = st["kv8"][rows].view(torch.float8_e4m3fn).float() * st["kv_scale"][rows].unsqueeze(-1)
        l = torch.matmul(st["q"].float().view(B, T * H, dk), kv.transpose(1, 2)).view(B, T, H, -1) * st["tau"]
        l.masked_fill_((s.unsqueeze(1) > _positions(st).unsqueeze(-1)).unsqueeze(2), -math.inf)
        o, lse = _softmax_v(l.view(B, T * H, -1), kv[..., :dv])
    st["out"].copy_(o.view(B, T, H, dv))
    st["lse"].copy_(lse.view(B, T, H))


def _run_rope(st):
    for n in ("q", "k"):
        st[n + "_out"].copy_(_norm_rope(st, n))
        if st["c"]["train"]:
            d, w = _norm_rope_back(st, n)
            st["d" + n].copy_(d)
            st["d" + n + "_w"].copy_(w)


def run(state):
    st = state
    op = st["c"]["op"]
    if own:
        _run_own(st)
    elif op == "rope":
        _run_rope(st)
    elif op == "write":
        _run_write(st)
    elif op == "read":
        _run_read(st)
    else:
        _run_attn(st)
    if op == "rope":
        out = [st["q_out"], st["k_out"]]
        if st["c"]["train"]:
            out += [st["dq"], st["dk"]]
            out += [st["dq_w"], st["dk_w"]] if st["c"]["norm"] else []
        return out
    if op == "write":
        f8 = torch.float8_e4m3fn
        return [st["kv8"].view(f8), st["kv_scale"], st["kI8"].view(f8), st["kI_scale"], st["qI8"].view(f8),
                st["qI_scale"]]
    if op == "read":
        return [st["kv_out"], st["kI_out"]]
    return [st["out"], st["lse"]]


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    c = case
    n = c["B"] * c["T"]
    if c["op"] == "rope":
        e = n * (c["Hq"] + c["Hk"]) * c["D"]
        # forward: rows in, rows out; backward: rows and their gradients in, gradients out
        return {"bytes": 2 * e * (5 if c["train"] else 2), "flops": e * (14 if c["train"] else 5)}
    if c["op"] == "write":
        e = n * (c["d_k"] + c["D_I"] + c["H_I"] * c["D_I"])
        return {"bytes": 3 * e + 4 * n * (2 + c["H_I"]), "flops": 3 * e}
    if c["op"] == "read":
        e = c["B"] * c["count"] * (c["d_k"] + c["D_I"])
        return {"bytes": 3 * e + 8 * c["B"] * c["count"], "flops": e}
    dk, dv, H = c["d_k"], _dv(c["d_k"]), c["H"]
    pos = range(c["S"] - c["T"], c["S"])
    pairs = c["B"] * sum(min(c["k"], p + 1) if c["k"] else p + 1 for p in pos)
    rows = min(pairs, c["B"] * c["S"])
    return {"bytes": n * H * (2 * dk + 2 * dv + 4) + rows * (dk + 4) + (4 * n * c["k"]),
            "flops": 2 * pairs * H * (dk + dv)}


# ------------------------------------------------------------------ the definition in 64 bits

def _exact_rope(st):
    c = st["c"]
    B, T = c["B"], c["T"]
    out, grads, weights = [], [], []
    half = c["rope"] // 2
    for n in ("q", "k"):
        ys, dxs, dw = [], [], 0
        for b in range(B):
            x = st[n][b].double().requires_grad_(c["train"])
            w = None if st[n + "_w"] is None else st[n + "_w"].double().requires_grad_(c["train"])
            y = x
            if c["norm"]:
                z = x[..., :c["norm"]]
                y = torch.cat((w * z / torch.sqrt((z * z).sum(-1, keepdim=True) / c["norm"] + st["eps"]),
                               x[..., c["norm"]:]), -1)
            if half:
                p = (int(st["lens"][b]) - T + torch.arange(T, device="cuda")).double()
                turn = torch.polar(torch.ones(T, half, device="cuda", dtype=torch.float64),
                                   torch.outer(p, st["freq"].double())).unsqueeze(1)
                tail = y[..., c["D"] - c["rope"]:]
                pair = tail.unflatten(-1, (half, 2)) if c["inter"] else tail.unflatten(-1, (2, half)).transpose(-1, -2)
                z = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn)
                z = z.flatten(-2) if c["inter"] else z.transpose(-1, -2).flatten(-2)
                y = torch.cat((y[..., :c["D"] - c["rope"]], z), -1)
            if c["train"]:
                gs = torch.autograd.grad(y, [x] if w is None else [x, w], st["g" + n][b].double())
                dxs.append(gs[0])
                dw = dw + (gs[1] if w is not None else 0)
            ys.append(y.detach())
        out.append(torch.stack(ys))
        if c["train"]:
            grads.append(torch.stack(dxs))
            weights += [dw] if c["norm"] else []
    return out + grads + weights


def _exact_bytes(x):
    """e4m3 values (in 64 bits) and scale of each row, rounded by hand: to even, to the row's grid."""
    x = x.double()
    a = x.abs().amax(-1)
    sizes = torch.tensor([2.0 ** i for i in range(MIN_EXP, 121)], dtype=torch.float64, device="cuda")
    s = sizes[torch.searchsorted(E4M3_MAX * sizes, a.flatten()).clamp(max=sizes.numel() - 1)].view(a.shape)
    y = x / s.unsqueeze(-1)
    step = torch.full_like(y, 2.0 ** -9)                      # the grid of e4m3: 2^-9 below 2^-6, then 8 to an octave
    for i in range(-5, 9):
        step = torch.where(y.abs() >= 2.0 ** i, 2.0 ** (i - 3), step)
    return torch.round(y / step) * step, s


def _exact_write(st):
    c = st["c"]
    res = []
    for src, dst, sc in (("kv", "kv8", "kv_scale"), ("k_I", "kI8", "kI_scale")):
        pool, scales = st[dst].view(torch.float8_e4m3fn).double(), st[sc].double()
        v, s = _exact_bytes(st[src])
        for b in range(c["B"]):
            p0 = int(st["lens"][b]) - c["T"]
            at = [b * c["S"] + p0 + t if st["table"] is None else
                  int(st["table"][b, (p0 + t) // c["page"]]) * c["page"] + (p0 + t) % c["page"] for t in range(c["T"])]
            at = torch.tensor(at, device="cuda")
            pool[at], scales[at] = v[b], s[b]
        res += [pool, scales]
    return res + list(_exact_bytes(st["q_I"]))


def _exact_keys(st, b, src, sc):
    """All of sequence b's cache rows in 64 bits, in token order."""
    c = st["c"]
    if st["table"] is None:
        at = slice(b * c["S"], (b + 1) * c["S"])
        x, s = st[src][at], st[sc][at]
    else:
        pool = st[src].view(-1, c["page"], st[src].shape[-1])
        x = pool[st["table"][b].long()].flatten(0, 1)[:c["S"]]
        s = st[sc].view(-1, c["page"])[st["table"][b].long()].flatten()[:c["S"]]
    return x, s


def _exact_read(st):
    c = st["c"]
    res = []
    for src, sc, dst in (("kv8", "kv_scale", "kv_out"), ("kI8", "kI_scale", "kI_out")):
        out = st[dst].double()
        for b in range(c["B"]):
            x, s = _exact_keys(st, b, src, sc)
            n = max(0, min(c["count"], int(st["lens"][b]) - c["begin"]))
            at = slice(c["begin"], c["begin"] + n)
            out[b, :n] = x[at].view(torch.float8_e4m3fn).double() * s[at].double().unsqueeze(-1)
        res.append(out)
    return res


def _exact_attn(st):
    c = st["c"]
    B, T, H, dv = c["B"], c["T"], c["H"], _dv(c["d_k"])
    out = torch.zeros(B, T, H, dv, dtype=torch.float64, device="cuda")
    lse = torch.full((B, T, H), -math.inf, dtype=torch.float64, device="cuda")
    for b in range(B):
        x, s = _exact_keys(st, b, "kv8", "kv_scale")
        n = int(st["lens"][b])
        if not c["k"]:
            keys = x[:n].view(torch.float8_e4m3fn).double() * s[:n].double().unsqueeze(-1)
        for t0 in range(0, T, 128):
            t1 = min(T, t0 + 128)
            q = st["q"][b, t0:t1].double() * st["tau"]
            if c["k"]:
                i = st["idx"][b, t0:t1].long()
                at = i.clamp(min=0)
                kv = x[at].view(torch.float8_e4m3fn).double() * s[at].double().unsqueeze(-1)
                z = torch.einsum("thd,tkd->thk", q, kv)
                z = z + torch.where(i < 0, -math.inf, 0.0).double().unsqueeze(1)
                lse[b, t0:t1] = torch.logsumexp(z, -1)
                w = torch.exp(z - lse[b, t0:t1].unsqueeze(-1)).nan_to_num(0.0)
                out[b, t0:t1] = torch.einsum("thk,tkv->thv", w, kv[..., :dv])
            else:
                z = torch.einsum("thd,kd->thk", q, keys)
                late = torch.arange(n, device="cuda") > (n - T + torch.arange(t0, t1, device="cuda")).unsqueeze(-1)
                z = z.masked_fill(late.unsqueeze(1), -math.inf)
                lse[b, t0:t1] = torch.logsumexp(z, -1)
                out[b, t0:t1] = torch.einsum("thk,kv->thv", torch.exp(z - lse[b, t0:t1].unsqueeze(-1)), keys[:, :dv])
    return [out, lse]


def exact(case, seed):
    st = prepare(case, seed)
    return {"rope": _exact_rope, "write": _exact_write, "read": _exact_read, "attn": _exact_attn}[case["op"]](st)
