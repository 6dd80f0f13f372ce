"""What is measured of the serving operators: appending to a paged key/value
cache, attention over it and filtered sampling.

Each case runs in a plain form (elementary torch operations, 32 bits, 64 where
a border or an angle needs them) or, with ``own`` set, through the library's
entry points. Sizes are those of the decoders this repository runs: 16 query
heads on 8 key/value heads of 128 (the 0.6B and 1.7B decoders), 16 on 16 of 64
(the code predictor), caches of 512 to 32768 tokens, vocabularies of 151936
(text) and 2048 (codes).
"""
import math

import torch

own = False

BLOCK = 16        # tokens that share one scale of an 8-bit page
EPS = 1e-6
THETA = 1e6
WORKSPACE = 64 << 20


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # one user's next token: what one layer adds to the cache
        dict(name="append int8 1 token", op="append", kv="int8", x="f32", B=1, rows=1, L=512,
             H=16, Hkv=8, D=128, page=64, norm=True),
        # a full batch's next tokens, on a bf16 cache
        dict(name="append bf16 32 tokens", op="append", kv="bf16", x="f32", B=32, rows=32, L=2048,
             H=16, Hkv=8, D=128, page=64, norm=True),
        # prompts of several users in one packed batch, some after a cached prefix
        dict(name="append int8 prompts", op="append", kv="int8", x="bf16", B=5, rows=4099, L=2048,
             H=16, Hkv=8, D=128, page=64, norm=True),
        # one user's next token over a short context: latency
        dict(name="attend int8 1x512", op="attend", kv="int8", x="bf16", out="bf16", B=1, rows=1,
             L=512, H=16, Hkv=8, D=128, page=64),
        # a full batch at the decoder's ordinary context, ragged
        dict(name="attend int8 32x2048", op="attend", kv="int8", x="bf16", out="bf16", B=32,
             rows=32, L=2048, H=16, Hkv=8, D=128, page=64),
        # a full batch at the longest context: the cache's whole rate
        dict(name="attend int8 32x32768", op="attend", kv="int8", x="bf16", out="bf16", B=32,
             rows=32, L=32768, H=16, Hkv=8, D=128, page=128),
        # one user's long context, in fp32 on a bf16 cache
        dict(name="attend bf16 1x32749 f32", op="attend", kv="bf16", x="f32", out="f32", B=1,
             rows=1, L=32749, H=16, Hkv=8, D=128, page=16),
        # small heads, every query head with keys of its own
        dict(name="attend bf16 7x1500 d64", op="attend", kv="bf16", x="bf16", out="bf16", B=7,
             rows=7, L=1500, H=16, Hkv=16, D=64, page=32),
        # prompt rows of several users over their own cached rows
        dict(name="attend int8 prompts", op="attend", kv="int8", x="bf16", out="bf16", B=5,
             rows=2053, L=2048, H=16, Hkv=8, D=128, page=64),
        # one user's next token: top-p over the text vocabulary
        dict(name="sample 1x151936", op="sample", B=1, V=151936, filters="p"),
        # a full batch, every user with filters of their own
        dict(name="sample 32x151936 mixed", op="sample", B=32, V=151936, filters="mixed"),
        # the codes of a batch of frames, unfiltered draws
        dict(name="sample 160x2048 plain", op="sample", B=160, V=2048, filters="none"),
    ]


def _log_between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "sample"])
    if op == "sample":
        V = _log_between(rng, 100, 160000)
        return dict(op=op, B=min(_log_between(rng, 1, 256), max(1, 5000000 // V)), V=V,
                    filters=rng.choice(["none", "k", "p", "m", "mixed"]))
    Hkv = rng.choice([1, 2, 4, 8, 16])
    H = Hkv * rng.choice([1, 2, 3, 4, 5, 8])
    D = rng.choice([64, 128])
    page = rng.choice([16, 32, 48, 64, 128])
    kv = rng.choice(["int8", "bf16"])
    x = rng.choice(["f32", "bf16"])
    B = _log_between(rng, 1, 40)
    if op == "append":
        rows = rng.choice([B, B, B + _log_between(rng, 1, 3000)])
        return dict(op=op, kv=kv, x=x, B=B, rows=rows, L=_log_between(rng, 1, 4000) + rows // B,
                    H=H, Hkv=Hkv, D=D, page=page, norm=rng.random() < 0.5)
    prompt = rng.random() < 0.35
    most = 4000 if prompt else min(32768, (1 << 29) // (B * Hkv * D))
    L = _log_between(rng, 1, max(2, most))
    rows = min(B * L, B + _log_between(rng, 1, 1200)) if prompt else B
    return dict(op=op, kv=kv, x=x, out=rng.choice(["f32", "bf16"]), B=B, rows=rows, L=L, H=H,
                Hkv=Hkv, D=D, page=page)


# ----------------------------------------------------------------- inputs --

def _lengths(case):
    """Rows and cached tokens of each sequence, from the case alone: ragged,
    the first sequence the longest."""
    B, rows, L = case["B"], case["rows"], case["L"]
    if rows == B:
        n = [1] * B
    else:  # shares 1 : 2 : 3 ..., at least one row each
        tot = B * (B + 1) // 2
        n = [1 + (rows - B) * (i + 1) // tot for i in range(B)]
        n[-1] += rows - sum(n)
    lens = [max(n[i], L if i == 0 else L - (i * 7919) % max(1, L // 2)) for i in range(B)]
    if rows != B:  # some prompts start an empty cache
        lens = [n[i] if i % 2 else lens[i] for i in range(B)]
    return n, lens


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _pages(g, case, n_pages):
    """One pool of pages: (values or codes, scales or None)."""
    shape = (n_pages, case["Hkv"], case["page"], case["D"])
    if case["kv"] == "bf16":
        out = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
        for i in range(0, n_pages, 2048):
            out[i:i + 2048] = _normal(g, *out[i:i + 2048].shape)
        return out, None
    codes = torch.empty(shape, dtype=torch.int8, device="cuda")
    scales = torch.empty(shape[:2] + (case["page"] // BLOCK,), device="cuda")
    for i in range(0, n_pages, 2048):
        v = _normal(g, *codes[i:i + 2048].shape).unflatten(2, (-1, BLOCK))
        s = v.abs().amax((-1, -2)) / 127.0
        scales[i:i + 2048] = s
        codes[i:i + 2048] = (v / s[..., None, None]).round_().to(torch.int8).flatten(2, 3)
    return codes, scales


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(int(seed))
    dev = "cuda"
    if case["op"] == "sample":
        B, V = case["B"], case["V"]
        s = dict(case=case, logits=_normal(g, B, V) * 2.5,
                 u=torch.rand(B, generator=g, device=dev), temperature=None, top_k=None,
                 top_p=None, min_p=None, token=torch.empty(B, dtype=torch.int32, device=dev),
                 kept=torch.empty(B, dtype=torch.int32, device=dev),
                 logprob=torch.empty(B, device=dev))
        # a few likely tokens above the rest, as a trained head gives them
        top = torch.randint(0, V // 12, (B, 12), generator=g, device=dev)
        top += torch.arange(12, device=dev) * (V // 12)  # no index twice
        s["logits"].scatter_add_(1, top, _normal(g, B, 12).abs() * 4.0)
        f = case["filters"]
        s["temperature"] = 0.6 + 0.6 * torch.rand(B, generator=g, device=dev)
        if f in ("k", "mixed"):
            s["top_k"] = torch.randint(1, 101, (B,), generator=g, device=dev, dtype=torch.int32)
        if f in ("p", "mixed"):
            s["top_p"] = 0.8 + 0.2 * torch.rand(B, generator=g, device=dev)
        if f in ("m", "mixed"):
            s["min_p"] = 0.1 * torch.rand(B, generator=g, device=dev)
        if f == "mixed":  # every fourth user has one of them off, one is greedy
            s["top_k"][0::4] = 0
            s["top_p"][1::4] = 1.0
            s["min_p"][2::4] = 0.0
            s["temperature"][B // 2] = 0.0 if B > 1 else 1.0
        return s
    n, lens = _lengths(case)
    B, H, Hkv, D, page = case["B"], case["H"], case["Hkv"], case["D"], case["page"]
    T = sum(n)
    need = [(x + page - 1) // page for x in lens]
    n_pages = sum(need) + 2
    order = torch.randperm(n_pages, generator=g, device=dev).tolist()
    table = torch.full((B, max(need) + 1), -1, dtype=torch.int32)  # unused entries are -1
    at = 0
    for b, c in enumerate(need):
        table[b, :c] = torch.tensor(order[at:at + c], dtype=torch.int32)
        at += c
    starts = torch.tensor([0] + n, dtype=torch.int32).cumsum(0, dtype=torch.int32)
    xt = torch.float32 if case["x"] == "f32" else torch.bfloat16
    s = dict(case=case, table=table.to(dev), kv_len=torch.tensor(lens, dtype=torch.int32).to(dev),
             row_start=starts.to(dev), n=n, lens=lens,
             ws=torch.empty(WORKSPACE, dtype=torch.uint8, device=dev))
    s["k_pages"], s["k_scales"] = _pages(g, case, n_pages)
    s["v_pages"], s["v_scales"] = _pages(g, case, n_pages)
    if case["op"] == "attend":
        s["q"] = _normal(g, T, H * D).to(xt)
        s["out"] = torch.empty(T, H * D, device=dev,
                               dtype=torch.float32 if case["out"] == "f32" else torch.bfloat16)
        return s
    # q, k and v as one projection's rows
    s["qkv"] = (_normal(g, T, (H + 2 * Hkv) * D) * 1.5).to(xt)
    s["q_norm"] = (1.0 + 0.1 * _normal(g, D)).bfloat16() if case["norm"] else None
    s["k_norm"] = (1.0 + 0.1 * _normal(g, D)).bfloat16() if case["norm"] else None
    s["q_out"] = torch.empty(T, H * D, device=dev, dtype=torch.bfloat16)
    # what the call may change: the blocks of 16 tokens that its rows fall in
    first = [(lens[b] - n[b]) // BLOCK * BLOCK for b in range(B)]
    back = torch.tensor([0] + [lens[b] - first[b] for b in range(B)], dtype=torch.int32)
    s["first"] = torch.tensor(first, dtype=torch.int32).to(dev)
    s["back_start"] = back.cumsum(0, dtype=torch.int32).to(dev)
    rows = int(back.sum())
    s["k_back"] = torch.empty(rows, Hkv * D, device=dev, dtype=torch.bfloat16)
    s["v_back"] = torch.empty(rows, Hkv * D, device=dev, dtype=torch.bfloat16)
    return s


def work(case):
    if case["op"] == "sample":
        n = case["B"] * case["V"]
        return {"bytes": 4.0 * n + 28.0 * case["B"], "flops": 4.0 * n}
    n, lens = _lengths(case)
    H, Hkv, D = case["H"], case["Hkv"], case["D"]
    xb = 4 if case["x"] == "f32" else 2
    code = 1 + 4 / (BLOCK * D) if case["kv"] == "int8" else 2
    T = sum(n)
    if case["op"] == "attend":
        ob = 4 if case["out"] == "f32" else 2
        keys = sum(n[b] * (lens[b] - n[b]) + n[b] * (n[b] + 1) / 2 for b in range(len(n)))
        return {"bytes": T * H * D * (xb + ob) + 2 * sum(lens) * Hkv * D * code,
                "flops": 4.0 * keys * H * D}
    back = sum(lens[b] - (lens[b] - n[b]) // BLOCK * BLOCK for b in range(len(n)))
    # rows in, q out, pages written and read back as bf16 values
    return {"bytes": T * D * ((H + 2 * Hkv) * xb + 2 * H) + 2 * Hkv * D * (T * code + back * (code + 2)),
            "flops": 10.0 * T * (H + Hkv) * D}


# ---------------------------------------------------------------- one pass --

def run(state):
    op = state["case"]["op"]
    if own:
        import weight_only_quantized_03_b200 as qg
        if op == "append":
            return _own_append(qg, state)
        return _own_attend(qg, state) if op == "attend" else _own_sample(qg, state)
    if op == "append":
        return _plain_append(state)
    return _plain_attend(state) if op == "attend" else _plain_sample(state)


def _own_append(qg, s):
    c = s["case"]
    H, Hkv, D = c["H"], c["Hkv"], c["D"]
    q, k, v = s["qkv"].split((H * D, Hkv * D, Hkv * D), 1)
    kv = qg.PagedKV(s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"])
    qg.qg_paged_kv_append(kv, s["table"], s["kv_len"], k, v, row_start=s["row_start"], q=q,
                          q_out=s["q_out"], q_norm=s["q_norm"], k_norm=s["k_norm"], eps=EPS,
                          theta=THETA)
    qg.qg_paged_kv_gather(kv, s["table"], s["first"], s["back_start"], s["k_back"], s["v_back"])
    return s["q_out"], s["k_back"], s["v_back"]


def _own_attend(qg, s):
    c = s["case"]
    kv = qg.PagedKV(s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"])
    qg.qg_paged_attention(kv, s["table"], s["kv_len"], s["q"], s["out"], c["H"],
                          1.0 / math.sqrt(c["D"]), s["ws"], row_start=s["row_start"])
    return s["out"]


def _own_sample(qg, s):
    qg.qg_sample_filtered(s["logits"], s["u"], s["token"], temperature=s["temperature"],
                          top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"], kept=s["kept"],
                          logprob=s["logprob"])
    return s["token"], s["kept"], s["logprob"]


def _rows(starts, total):
    """Sequence and index within it of each of ``total`` packed rows."""
    r = torch.arange(total, device=starts.device, dtype=torch.int32)
    b = torch.searchsorted(starts, r, right=True) - 1
    return b, r - starts[b]


def _norm_rotate(x, w, pos):
    """fp32 [T, heads, D]: RMSNorm by w (or none), then the rotation."""
    D = x.shape[-1]
    x = x.float()
    if w is not None:
        x = x * (1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)) * w.float()
    i = torch.arange(D // 2, device=x.device, dtype=torch.float64)
    a = pos.double()[:, None] * THETA ** (-2.0 * i / D)
    c, s = a.cos().float()[:, None], a.sin().float()[:, None]
    lo, hi = x[..., :D // 2], x[..., D // 2:]
    return torch.cat((lo * c - hi * s, hi * c + lo * s), -1)


def _store(pages, scales, page, off, x):
    """Rows x [T, Hkv, D] at (page, offset): the pool after it."""
    if scales is None:
        pages[page, :, off] = x.bfloat16()
        return
    P, Hkv, size, D = pages.shape
    per = size // BLOCK
    block = page * per + off // BLOCK
    o = off % BLOCK
    slots = P * per
    first = torch.full((slots,), BLOCK, device=x.device).scatter_reduce(0, block, o, "amin")
    top = torch.zeros(slots, Hkv, device=x.device).scatter_reduce(
        0, block[:, None].expand(-1, Hkv), x.abs().amax(-1), "amax")
    b_page, b_in = block // per, block % per
    old = scales[b_page, :, b_in]
    o1 = first[block]
    kept = torch.where(o1[:, None] > 0, old, 0.0)
    new = torch.maximum(kept, top[block] / 127.0)
    # rows of the block before the first new one: to the new scale
    ratio = torch.where(new > 0, kept / new, 0.0)
    blocks = pages.view(P, Hkv, per, BLOCK, D)
    codes = blocks[b_page, :, b_in]                                     # [T, Hkv, 16, D]
    before = torch.arange(BLOCK, device=x.device) < o1[:, None]
    again = torch.round(codes.float() * ratio[:, :, None, None]).to(torch.int8)
    blocks[b_page, :, b_in] = torch.where(before[:, None, :, None], again, codes)
    scales[b_page, :, b_in] = new
    codes = torch.where(new[..., None] > 0, x / new[..., None], 0.0)
    pages[page, :, off] = torch.round(codes).clamp(-127, 127).to(torch.int8)


def _values(pages, scales, page, off):
    """fp32 values of the rows at (page, offset): [..., Hkv, D]."""
    v = pages[page, :, off].float()
    return v if scales is None else v * scales[page, :, off // BLOCK][..., None]


def _plain_append(s):
    c = s["case"]
    H, Hkv, D, size = c["H"], c["Hkv"], c["D"], c["page"]
    T = s["qkv"].shape[0]
    q, k, v = s["qkv"].split((H * D, Hkv * D, Hkv * D), 1)
    b, i = _rows(s["row_start"], T)
    n = s["row_start"][1:] - s["row_start"][:-1]
    pos = (s["kv_len"] - n)[b] + i
    q_out = _norm_rotate(q.unflatten(1, (H, D)), s["q_norm"], pos)
    page, off = s["table"][b, pos // size].long(), (pos % size).long()
    _store(s["k_pages"], s["k_scales"], page, off,
           _norm_rotate(k.unflatten(1, (Hkv, D)), s["k_norm"], pos))
    _store(s["v_pages"], s["v_scales"], page, off, v.unflatten(1, (Hkv, D)).float())
    b, i = _rows(s["back_start"], s["k_back"].shape[0])
    pos = s["first"][b] + i
    page, off = s["table"][b, pos // size].long(), (pos % size).long()
    return (q_out.flatten(1).bfloat16(),
            _values(s["k_pages"], s["k_scales"], page, off).flatten(1).bfloat16(),
            _values(s["v_pages"], s["v_scales"], page, off).flatten(1).bfloat16())


def _dense(pages, scales, table):
    """fp32 [B, Hkv, max_pages * page, D] of every sequence's pages."""
    v = pages[table].float()
    if scales is not None:
        v = v * scales[table].repeat_interleave(BLOCK, -1)[..., None]
    return v.transpose(1, 2).flatten(2, 3)


def _plain_attend(s):
    c = s["case"]
    H, Hkv, D, B = c["H"], c["Hkv"], c["D"], c["B"]
    G, T, N = H // Hkv, s["q"].shape[0], max(s["n"])
    table = s["table"].clamp(min=0).long()
    k = _dense(s["k_pages"], s["k_scales"], table)
    v = _dense(s["v_pages"], s["v_scales"], table)
    L = k.shape[2]
    b, i = _rows(s["row_start"], T)
    n = s["row_start"][1:] - s["row_start"][:-1]
    q = torch.zeros(B, N, Hkv, G, D, device=k.device)
    q[b, i.long()] = s["q"].float().view(T, Hkv, G, D)
    q = q.permute(0, 2, 1, 3, 4).flatten(2, 3)                          # [B, Hkv, N * G, D]
    p = (q @ k.transpose(2, 3)).mul_(1.0 / math.sqrt(D)).view(B, Hkv, N, G, L)
    last = (s["kv_len"] - n)[:, None] + torch.arange(N, device=k.device)
    hide = torch.arange(L, device=k.device) > last[:, :, None]          # [B, N, L]
    p.masked_fill_(hide[:, None, :, None], -math.inf)
    p.sub_(p.amax(-1, keepdim=True)).exp_()
    l = p.sum(-1, keepdim=True)
    o = ((p.view(B, Hkv, N * G, L) @ v).view(B, Hkv, N, G, D) / l)
    return o.permute(0, 2, 1, 3, 4)[b, i.long()].reshape(T, H * D).to(s["out"].dtype)


def _plain_sample(s):
    x = s["logits"]
    B, V = x.shape
    order, idx = torch.sort(x, dim=1, descending=True, stable=True)
    order = order.double()
    t = s["temperature"].double()[:, None]
    greedy = t <= 0
    w = torch.exp((order - order[:, :1]) / torch.where(greedy, 1.0, t))
    rank = torch.arange(V, device=x.device)[None]
    keep = torch.where(greedy, rank < 1, rank < V)
    if s["top_k"] is not None:
        k = s["top_k"][:, None]
        keep &= (k <= 0) | (rank < k)
    if s["top_p"] is not None:
        p = s["top_p"].double()[:, None]
        run_ = (w * keep).cumsum(1)
        keep &= (p >= 1) | (rank < 1) | (run_ - w < p * run_[:, -1:])
    if s["min_p"] is not None:
        keep &= w >= s["min_p"].double()[:, None]
    w = w * keep
    run_ = w.cumsum(1)
    target = s["u"].double()[:, None] * run_[:, -1:]
    j = (keep & (run_ < target)).sum(1, keepdim=True)
    return (idx.gather(1, j)[:, 0].int(), keep.sum(1).int(),
            torch.log(w.gather(1, j) / run_[:, -1:])[:, 0].float())


# -------------------------------------------------------- exact, in 64 bits --

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(s)
    return _exact_attend(s) if case["op"] == "attend" else _exact_sample(s)


def _where(s, b, pos):
    size = s["case"]["page"]
    return s["table"][b, pos // size].long(), pos % size


def _exact_cached(s, which, b, pos):
    """[Hkv, len(pos), D] in 64 bits of sequence b's cached rows."""
    page, off = _where(s, b, pos)
    x = s[which + "_pages"][page, :, off].double()
    if s[which + "_scales"] is not None:
        x *= s[which + "_scales"][page, :, off // BLOCK].double()[..., None]
    return x.transpose(0, 1)


def _exact_append(s):
    c = s["case"]
    H, Hkv, D = c["H"], c["Hkv"], c["D"]
    half = D // 2
    freq = torch.tensor([THETA ** (-2.0 * i / D) for i in range(half)], dtype=torch.float64,
                        device="cuda")
    q_rows, k_rows, v_rows = [], [], []
    for b, n in enumerate(s["n"]):
        r0, p0 = sum(s["n"][:b]), s["lens"][b] - s["n"][b]
        rows = s["qkv"][r0:r0 + n].double().view(n, H + 2 * Hkv, D)
        pos = torch.arange(p0, p0 + n, device="cuda")
        turn = torch.polar(torch.ones(n, half, dtype=torch.float64, device="cuda"),
                           pos.double()[:, None] * freq)

        def turned(x, weight):
            if weight is not None:
                x = x / (x.pow(2).sum(-1, keepdim=True) / D + EPS).sqrt() * weight.double()
            z = torch.complex(x[..., :half], x[..., half:]) * turn[:, None]
            return torch.cat((z.real, z.imag), -1)

        q_rows.append(turned(rows[:, :H], s["q_norm"]).reshape(n, H * D))
        new = {"k": turned(rows[:, H:H + Hkv], s["k_norm"]), "v": rows[:, H + Hkv:]}
        first = p0 // BLOCK * BLOCK
        for which, out in (("k", k_rows), ("v", v_rows)):
            x = new[which].transpose(0, 1)                               # [Hkv, n, D]
            if s[which + "_scales"] is None:
                old = _exact_cached(s, which, b, torch.arange(first, p0, device="cuda"))
                out.append(torch.cat((old, x), 1).transpose(0, 1).reshape(-1, Hkv * D))
                continue
            for j in range(first, p0 + n, BLOCK):
                lo, hi = max(j, p0), min(j + BLOCK, p0 + n)
                part = x[:, lo - p0:hi - p0]
                scale = part.abs().amax((1, 2)) / 127.0
                got = []
                if lo > j:
                    page, off = _where(s, b, torch.arange(j, lo, device="cuda"))
                    codes = s[which + "_pages"][page, :, off].double().transpose(0, 1)
                    was = s[which + "_scales"][page[0], :, off[0] // BLOCK].double()
                    scale = torch.maximum(scale, was)
                    got.append((codes * (was / scale)[:, None, None]).round())
                got.append((part / scale[:, None, None]).round())
                out.append((torch.cat(got, 1) * scale[:, None, None]).transpose(0, 1)
                           .reshape(-1, Hkv * D))
    return torch.cat(q_rows), torch.cat(k_rows), torch.cat(v_rows)


def _exact_attend(s):
    c = s["case"]
    H, Hkv, D = c["H"], c["Hkv"], c["D"]
    outs = []
    for b, n in enumerate(s["n"]):
        r0, L = sum(s["n"][:b]), s["lens"][b]
        pos = torch.arange(L, device="cuda")
        k, v = _exact_cached(s, "k", b, pos), _exact_cached(s, "v", b, pos)
        q = s["q"][r0:r0 + n].double().view(n, Hkv, H // Hkv, D)
        seen = pos <= torch.arange(L - n, L, device="cuda")[:, None]
        score = torch.einsum("nkgd,kld->kgnl", q, k) / D ** 0.5
        weight = torch.softmax(score.where(seen, torch.tensor(-math.inf, device="cuda",
                                                              dtype=torch.float64)), -1)
        outs.append(torch.einsum("kgnl,kld->nkgd", weight, v).reshape(n, H * D))
    return torch.cat(outs)


def _exact_sample(s):
    import numpy as np
    host = {k: None if s[k] is None else s[k].cpu().numpy() for k in
            ("logits", "u", "temperature", "top_k", "top_p", "min_p")}
    tokens, kept, logprob = [], [], []
    for b, row in enumerate(host["logits"].astype(np.float64)):
        order = np.lexsort((np.arange(row.size), -row))
        temp = float(host["temperature"][b])
        m = 1 if temp <= 0 else row.size
        if temp > 0:
            w = np.exp((row[order] - row[order[0]]) / temp)
            if host["top_k"] is not None and host["top_k"][b] > 0:
                m = min(m, int(host["top_k"][b]))
            if host["top_p"] is not None and host["top_p"][b] < 1:
                before = np.concatenate(([0.0], np.cumsum(w[:m])))
                m = max(1, int(np.searchsorted(before[:m], float(host["top_p"][b]) * before[m])))
            if host["min_p"] is not None:
                m = min(m, int((w >= float(host["min_p"][b])).sum()))
        else:
            w = np.ones(1)
        run_ = np.cumsum(w[:m])
        j = int(np.searchsorted(run_, float(host["u"][b]) * run_[-1]))
        tokens.append(int(order[j]))
        kept.append(m)
        logprob.append(math.log(w[j] / run_[-1]))
    return (torch.tensor(tokens, dtype=torch.int32), torch.tensor(kept, dtype=torch.int32),
            torch.tensor(logprob, dtype=torch.float64))
