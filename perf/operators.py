"""The local attention block's operators as measured work: their inputs, their plain forms in torch, and what each
has to read, write and compute.

  rotate         per-head RMS norms of queries and keys with the position rotation in the same pass; with a cache,
                 the rotated keys and the values also go to their pages
  rotate_train   the same pass and its gradients
  attend         causal attention in a sliding window with a few first tokens that stay visible, grouped heads
  attend_train   the same and its gradients
  decode         attention of one new token per sequence over a paged key-value cache

A case says the operator ("op"), the types and sizes; `prepare` makes the inputs, `run` is one pass.
"""
import math

import torch

own = False  # True: run() calls the framework's kernels; False: the plain forms below

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


# ---------------------------------------------------------------------------------------------- cases
def _rotate(op, name, dtype, B, T, Hq, Hkv, dh, rot, norm=True, cache=False, page=0, far=0):
    return dict(op=op, name=name, dtype=dtype, B=B, T=T, Hq=Hq, Hkv=Hkv, dh=dh, rot=rot, norm=norm, cache=cache,
                page=page, far=far)


def _attend(op, name, B, T, Hq, Hkv, dh, window, sinks, ragged):
    return dict(op=op, name=name, dtype="bf16", B=B, T=T, Hq=Hq, Hkv=Hkv, dh=dh, window=window, sinks=sinks,
                ragged=ragged)


def _decode(name, dtype, N, Hq, Hkv, dh, shortest, longest, window, sinks, page):
    return dict(op="decode", name=name, dtype=dtype, N=N, Hq=Hq, Hkv=Hkv, dh=dh, shortest=shortest, longest=longest,
                window=window, sinks=sinks, page=page)


def listed():
    return [
        # prefill of the 2B-shaped layer's batch: 10 query heads of 256 on one key head, half of each head rotated
        _rotate("rotate", "rotate_prefill_b8_t2048_hq10_dh256", "bf16", 8, 2048, 10, 1, 256, 128),
        # one decoding step of 64 sequences of the 9B-shaped layer, keys and values into the cache, far positions
        _rotate("rotate", "rotate_step_n64_hq16_dh256_cache", "bf16", 64, 1, 16, 1, 256, 128, cache=True, page=64,
                far=1 << 20),
        # a training step of the 2B-shaped layer
        _rotate("rotate_train", "rotate_train_b8_t2048_hq10_dh256", "bf16", 8, 2048, 10, 1, 256, 128),
        # a training step in fp32 with grouped heads, whole heads rotated, odd length
        _rotate("rotate_train", "rotate_train_f32_b3_t1531_hq8_hkv2_dh128", "f32", 3, 1531, 8, 2, 128, 128),
        # a short prompt: latency
        _attend("attend", "attend_b1_t101_hq4_dh64", 1, 101, 4, 1, 64, 32, 4, False),
        # prefill of a padded batch in the 2B-shaped layer, window 1024, four sinks
        _attend("attend", "attend_b8_t2048_hq10_dh256_w1024", 8, 2048, 10, 1, 256, 1024, 4, True),
        # a long document with grouped heads and a wide window
        _attend("attend", "attend_b1_t16384_hq8_hkv2_dh128_w4096", 1, 16384, 8, 2, 128, 4096, 4, False),
        # a training step of the 2B-shaped layer, window 1024
        _attend("attend_train", "attend_train_b4_t2048_hq10_dh256_w1024", 4, 2048, 10, 1, 256, 1024, 0, False),
        # a training step of a padded batch of odd sizes, grouped heads, sinks
        _attend("attend_train", "attend_train_b3_t1111_hq6_hkv2_dh128_w300", 3, 1111, 6, 2, 128, 300, 5, True),
        # one sequence's next token in a local window: latency
        _decode("decode_n1_hq10_dh256_w1024", "bf16", 1, 10, 1, 256, 1500, 1500, 1024, 4, 16),
        # a serving batch of the 9B-shaped layer, lengths from one token on, window 2048
        _decode("decode_n128_hq16_dh256_w2048", "bf16", 128, 16, 1, 256, 1, 6000, 2048, 4, 64),
        # few long sequences, everything visible, grouped heads
        _decode("decode_n4_hq8_hkv2_dh128_131k", "bf16", 4, 8, 2, 128, 65000, 131000, 1 << 30, 0, 32),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _heads(rng, most):
    Hkv = rng.choice([1, 1, 1, 2, 3, 4])
    return Hkv * rng.randint(1, max(1, min(16, most // Hkv))), Hkv


def draw(rng):
    op = rng.choice(["rotate", "rotate_train", "attend", "attend_train", "decode"])
    dh = rng.choice([64, 128, 256])
    if op.startswith("rotate"):
        Hq, Hkv = _heads(rng, 16)
        B = rng.choice([1, 2, 3, 5, 8, 64])
        rows = _spread(rng, 1, (45056 * 1024 // 2) // ((Hq + Hkv) * dh))  # as many values as the listed ones, in fp32
        T = max(1, rows // B)
        cache = op == "rotate" and rng.random() < 0.4
        case = _rotate(op, None, rng.choice(["bf16", "f32"]), min(B, rows), T, Hq, Hkv, dh,
                       rng.choice([dh, dh // 2, dh // 4, dh - 16]), rng.random() < 0.8, cache,
                       rng.choice([1, 16, 17, 64]) if cache else 0, rng.choice([0, 0, 1 << 20]))
    elif op.startswith("attend"):
        Hq, Hkv = _heads(rng, 12)
        B = rng.randint(1, 4)
        T = _spread(rng, 1, min(4096, int((16384 ** 2 / 2 / (B * Hq)) ** 0.5)))  # a training step of dense scores
        case = _attend(op, None, B, T, Hq, Hkv, dh, _spread(rng, 1, 4 * T), rng.choice([0, 0, 1, 4, 7, 70]),
                       rng.random() < 0.5)
    else:
        Hq, Hkv = _heads(rng, 16)
        dtype = rng.choice(["bf16", "bf16", "f32"])
        N = _spread(rng, 1, 200)
        # at most as many bytes of keys and values as the longest listed case has
        most = (384 << 20) // (N * Hkv * dh * 2 * (2 if dtype == "bf16" else 4))
        longest = _spread(rng, 1, min(131072, max(64, most)))
        window = rng.choice([1 << 30, _spread(rng, 1, 2 * longest)])
        case = _decode(None, dtype, N, Hq, Hkv, dh, rng.choice([0, 1, (longest + 1) // 2]), longest, window,
                       rng.choice([0, 0, 1, 4, 50]), rng.choice([1, 7, 16, 32, 64, 128, 256]))
    del case["name"]
    return case


# --------------------------------------------------------------------------------------------- inputs
def _lens(case):
    """Lengths of a padded batch: from the full length down, the last sequence short."""
    B, T = case["B"], case["T"]
    return [max(1, T - (b * T) // (B + 1)) for b in range(B)] if case["ragged"] else [T] * B


def _cache_lens(case):
    """Cached tokens of each sequence (the new one among them), spread evenly over the case's range."""
    N, lo, hi = case["N"], case["shortest"], case["longest"]
    return [hi if N == 1 else lo + (n * (hi - lo)) // (N - 1) for n in range(N)]


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dt = TYPES[case["dtype"]]
    Hq, Hkv, dh = case["Hq"], case["Hkv"], case["dh"]

    def normal(*shape, dtype=dt):
        return torch.randn(*shape, generator=gen, device=dev, dtype=torch.float32).to(dtype)

    s = dict(case=case)
    if case["op"].startswith("rotate"):
        B, T, rot = case["B"], case["T"], case["rot"]
        qkv = normal(B, T, (Hq + 2 * Hkv) * dh)  # the projection's output, queries, keys and values of a token together
        s["q"] = qkv[..., :Hq * dh].unflatten(-1, (Hq, dh))
        s["k"] = qkv[..., Hq * dh:(Hq + Hkv) * dh].unflatten(-1, (Hkv, dh))
        s["v"] = qkv[..., (Hq + Hkv) * dh:].unflatten(-1, (Hkv, dh))
        start = torch.randint(0, case["far"] + 1, (B, 1), generator=gen, device=dev)
        s["positions"] = (start + torch.arange(T, device=dev)).to(torch.int32)
        s["inv_freq"] = (10000.0 ** (-torch.arange(0, rot, 2, device=dev, dtype=torch.float64) / rot)).float()
        s["q_w"] = 1 + 0.1 * normal(dh, dtype=torch.float32) if case["norm"] else None
        s["k_w"] = 1 + 0.1 * normal(dh, dtype=torch.float32) if case["norm"] else None
        if case["cache"]:
            page = case["page"]
            pages = 2 * (B * T + page - 1) // page + 1
            s["k_pages"] = normal(pages, page, Hkv, dh)
            s["v_pages"] = normal(pages, page, Hkv, dh)
            s["slots"] = torch.randperm(pages * page, generator=gen, device=dev)[:B * T].view(B, T)
        if case["op"] == "rotate_train":
            s["dq_out"], s["dk_out"] = normal(B, T, Hq, dh), normal(B, T, Hkv, dh)
    elif case["op"].startswith("attend"):
        B, T = case["B"], case["T"]
        s["q"], s["k"] = normal(B, T, Hq, dh), normal(B, T, Hkv, dh)  # as the norm and rotation leave them
        s["v"] = normal(B, T, (Hq + 2 * Hkv) * dh)[..., (Hq + Hkv) * dh:].unflatten(-1, (Hkv, dh))  # of the projection
        s["lens"] = torch.tensor(_lens(case), dtype=torch.int32, device=dev) if case["ragged"] else None
        if case["op"] == "attend_train":
            s["do"] = normal(B, T, Hq, dh)
    else:
        N, page = case["N"], case["page"]
        lens = torch.tensor(_cache_lens(case), device=dev)[torch.randperm(N, generator=gen, device=dev)]
        held = (lens + page - 1) // page  # pages of each sequence
        width = max(1, (case["longest"] + page - 1) // page)
        pages = int(held.sum()) + 1
        table = torch.zeros(N, width, dtype=torch.int32, device=dev)
        used = torch.arange(width, device=dev)[None] < held[:, None]
        table[used] = torch.randperm(pages, generator=gen, device=dev)[:int(held.sum())].to(torch.int32)
        s["q"] = normal(N, Hq, dh)
        s["k_pages"], s["v_pages"] = normal(pages, page, Hkv, dh), normal(pages, page, Hkv, dh)
        s["block_table"], s["lens"] = table, lens.to(torch.int32)
    return s


# ---------------------------------------------------------------------------------------- plain forms
def _angles(s):
    """cos and sin [B, T, 1, rot/2] of position * inv_freq, the product in 64 bits."""
    phi = s["positions"].double()[..., None] * s["inv_freq"].double()
    return phi.cos().float()[:, :, None], phi.sin().float()[:, :, None]


def _turn(x, cos, sin, rot):
    """The first `rot` values of each head rotated by pairs (i, i + rot/2)."""
    a, b = x[..., :rot // 2], x[..., rot // 2:rot]
    return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., rot:]], -1)


def _rotated(x, w, cos, sin, rot):
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w
    return _turn(x, cos, sin, rot)


def _rotated_back(x, w, g, cos, sin, rot):
    """Gradients of x and w for the gradient g of the rotated x."""
    x, g = x.float(), _turn(g.float(), cos, -sin, rot)
    if w is None:
        return g, None
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    xh, t = x * r, g * w
    return r * (t - xh * (t * xh).mean(-1, keepdim=True)), (g * xh).sum((0, 1, 2))


def _plain_rotate(s):
    dt, rot = s["q"].dtype, s["case"]["rot"]
    cos, sin = _angles(s)
    q = _rotated(s["q"], s["q_w"], cos, sin, rot).to(dt)
    k = _rotated(s["k"], s["k_w"], cos, sin, rot).to(dt)
    out = dict(q=q, k=k)
    if s["case"]["cache"]:
        at = s["slots"].reshape(-1)
        s["k_pages"].flatten(0, 1)[at] = k.flatten(0, 1)
        s["v_pages"].flatten(0, 1)[at] = s["v"].flatten(0, 1)
        out |= dict(k_pages=s["k_pages"], v_pages=s["v_pages"])
    if s["case"]["op"] == "rotate_train":
        dq, dq_w = _rotated_back(s["q"], s["q_w"], s["dq_out"], cos, sin, rot)
        dk, dk_w = _rotated_back(s["k"], s["k_w"], s["dk_out"], cos, sin, rot)
        out |= dict(dq=dq.to(dt), dk=dk.to(dt), dq_w=dq_w, dk_w=dk_w)
    return out


def _by_group(x, Hkv):
    """[B, T, H, dh] -> [B, Hkv, (H / Hkv) T, dh] in fp32: the rows that share a key and value head."""
    B, T, H, dh = x.shape
    return x.float().view(B, T, Hkv, H // Hkv, dh).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, dh)


def _by_token(x, B, T):
    """The way back: [B, Hkv, G T, dh] -> [B, T, Hkv G, dh]."""
    Hkv, dh = x.shape[1], x.shape[3]
    return x.view(B, Hkv, -1, T, dh).permute(0, 3, 1, 2, 4).reshape(B, T, -1, dh)


def _plain_attend(s):
    c = s["case"]
    B, T, Hq, Hkv, dh, W = c["B"], c["T"], c["Hq"], c["Hkv"], c["dh"], c["window"]
    dt, scale = s["q"].dtype, 1 / math.sqrt(dh)
    dev = s["q"].device
    t, u = torch.arange(T, device=dev)[:, None], torch.arange(T, device=dev)[None]
    seen = ((u <= t) & ((u > t - W) | (u < c["sinks"]))).expand(B, T, T)
    if s["lens"] is not None:
        n = s["lens"][:, None, None]
        seen = seen & (t < n) & (u < n)
    q, k, v = (_by_group(s[x], Hkv) for x in "qkv")
    sc = (q @ k.transpose(2, 3).contiguous()).mul_(scale).view(B, Hkv, -1, T, T)
    sc = sc.masked_fill_(~seen[:, None, None], -math.inf)
    m = sc.amax(-1, keepdim=True)
    p = sc.sub_(torch.where(m == -math.inf, 0.0, m)).exp_()
    total = p.sum(-1, keepdim=True)
    p = p.div_(torch.where(total == 0, 1.0, total)).view(B, Hkv, -1, T)
    o = _by_token(p @ v, B, T)
    out = dict(o=o.to(dt))
    if c["op"] == "attend_train":
        do = _by_group(s["do"], Hkv)
        dv = p.transpose(2, 3).contiguous() @ do
        ds = do @ v.transpose(2, 3).contiguous()
        ds = ds.sub_((ds * p).sum(-1, keepdim=True)).mul_(p).mul_(scale)
        out |= dict(dq=_by_token(ds @ k, B, T).to(dt), dk=_by_token(ds.transpose(2, 3).contiguous() @ q, B, T).to(dt),
                    dv=_by_token(dv, B, T).to(dt), lse=(m + total.log()).view(B, Hq, T))
    return out


def _plain_decode(s):
    c = s["case"]
    N, Hq, Hkv, dh, page = c["N"], c["Hq"], c["Hkv"], c["dh"], c["page"]
    S, W = min(c["sinks"], c["longest"]), min(c["window"], max(1, c["longest"]))
    dev, lens = s["q"].device, s["lens"].long()[:, None]
    j = torch.arange(S + W, device=dev)[None]
    u = torch.where(j < S, j, (lens - W).clamp(min=S) + j - S)  # the sinks, then the window behind them
    seen = u < lens
    u = u.clamp(max=s["block_table"].shape[1] * page - 1)
    at = s["block_table"].long().gather(1, u // page) * page + u % page
    k = s["k_pages"].flatten(0, 1)[at].float().transpose(1, 2).contiguous()  # [N, Hkv, S + W, dh]
    v = s["v_pages"].flatten(0, 1)[at].float().transpose(1, 2).contiguous()
    sc = s["q"].float().view(N, Hkv, -1, dh) @ k.transpose(2, 3).contiguous() / math.sqrt(dh)
    sc = sc.masked_fill(~seen[:, None, None], -math.inf)
    m = sc.amax(-1, keepdim=True)
    p = (sc - torch.where(m == -math.inf, 0.0, m)).exp()
    total = p.sum(-1, keepdim=True)
    o = (p @ v) / torch.where(total == 0, 1.0, total)
    return o.view(N, Hq, dh).to(s["q"].dtype)


# ------------------------------------------------------------------------------------------- one pass
def run(s):
    c = s["case"]
    if not own:
        if c["op"].startswith("rotate"):
            return _plain_rotate(s)
        return _plain_decode(s) if c["op"] == "decode" else _plain_attend(s)
    import gated_linear_recurrence_conv1d_amd as rg
    if c["op"].startswith("rotate"):
        cache = dict(v=s["v"], k_pages=s["k_pages"], v_pages=s["v_pages"], slots=s["slots"]) if c["cache"] else {}
        q, k = rg.qk_norm_rope(s["q"], s["k"], s["positions"], s["inv_freq"], s["q_w"], s["k_w"], eps=EPS, **cache)
        out = dict(q=q, k=k)
        if c["cache"]:
            out |= dict(k_pages=s["k_pages"], v_pages=s["v_pages"])
        if c["op"] == "rotate_train":
            out |= rg.qk_norm_rope_backward(s["q"], s["k"], s["positions"], s["inv_freq"], s["dq_out"], s["dk_out"],
                                            s["q_w"], s["k_w"], eps=EPS)
        return out
    if c["op"] == "attend":
        return dict(o=rg.local_attention(s["q"], s["k"], s["v"], c["window"], c["sinks"], lens=s["lens"]))
    if c["op"] == "attend_train":
        o, lse = rg.local_attention(s["q"], s["k"], s["v"], c["window"], c["sinks"], lens=s["lens"], want_lse=True)
        grads = rg.local_attention_backward(s["q"], s["k"], s["v"], o, lse, s["do"], c["window"], c["sinks"],
                                            lens=s["lens"])
        return dict(o=o, lse=lse) | grads
    return rg.paged_attention(s["q"], s["k_pages"], s["v_pages"], s["block_table"], s["lens"], c["window"], c["sinks"])


# ----------------------------------------------------------------------------------------------- work
def _pairs(n, W, S):
    """(query, key) pairs that see each other in a sequence of n tokens."""
    W = min(W, n)
    window = W * (W + 1) // 2 + (n - W) * W
    S = min(S, n)
    past = n - W  # rows t = W .. n-1 have t - W + 1 = 1 .. n - W tokens before their window
    full = max(0, past - S)
    part = past - full
    return window + full * S + part * (part + 1) // 2


def work(case):
    c = case
    e = 2 if c["dtype"] == "bf16" else 4
    Hq, Hkv, dh = c["Hq"], c["Hkv"], c["dh"]
    if c["op"].startswith("rotate"):
        rows, heads = c["B"] * c["T"], Hq + Hkv
        values = 2 * heads + (3 * Hkv if c["cache"] else 0)  # in and out; the cache: values in, keys and values out
        values += 2 * heads if c["op"] == "rotate_train" else 0  # gradients in and out
        flops = rows * heads * dh * (6 if c["op"] == "rotate" else 18)
        return {"bytes": rows * (values * dh * e + 4 + (8 if c["cache"] else 0)) + 4 * (c["rot"] // 2), "flops": flops}
    if c["op"].startswith("attend"):
        lens = _lens(c)
        train = c["op"] == "attend_train"
        flops = sum(_pairs(n, c["window"], c["sinks"]) for n in lens) * Hq * dh * (14 if train else 4)
        read = sum(lens) * (Hq * (2 if train else 1) + 2 * Hkv) * dh * e
        written = c["B"] * c["T"] * ((Hq * 2 + 2 * Hkv if train else Hq) * dh * e + (4 * Hq if train else 0))
        return {"bytes": read + written, "flops": flops}
    keys = sum(min(n, c["window"]) + min(c["sinks"], max(0, n - c["window"])) for n in _cache_lens(c))
    return {"bytes": (2 * keys * Hkv * dh + 2 * c["N"] * Hq * dh) * e, "flops": 4 * keys * Hq * dh}


# ------------------------------------------------------------------------------------ in 64 bits, apart
def _exact_head(x, w, positions, inv_freq, rot):
    """One tensor's heads normed and rotated as complex numbers."""
    x = x.double()
    if w is not None:
        x = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * w.double()
    z = torch.complex(x[..., :rot // 2], x[..., rot // 2:rot])
    turn = torch.exp(1j * (positions.double()[..., None, None] * inv_freq.double()))
    z = z * turn
    return torch.cat([z.real, z.imag, x[..., rot:]], -1)


def _exact_attend_head(q, k, v, W, S):
    """One head of one sequence: o and the log of the softmax's denominator."""
    n = q.shape[0]
    d = torch.arange(n, device=q.device)[:, None] - torch.arange(n, device=q.device)[None]
    hidden = (d < 0) | ((d >= W) & (torch.arange(n, device=q.device)[None] >= S))
    s = (q @ k.T / math.sqrt(q.shape[1])).masked_fill(hidden, -math.inf)
    lse = torch.logsumexp(s, 1)
    return torch.exp(s - lse[:, None]) @ v, lse


def exact(case, seed):
    c, s = case, prepare(case, seed)
    Hq, Hkv, dh = c["Hq"], c["Hkv"], c["dh"]
    if c["op"].startswith("rotate"):
        leaves, out = {}, {}
        train = c["op"] == "rotate_train"
        for x in "qk":
            a = s[x].double().detach().requires_grad_(train)
            w = None if s[x + "_w"] is None else s[x + "_w"].double().detach().requires_grad_(train)
            y = _exact_head(a, w, s["positions"], s["inv_freq"], c["rot"])
            out[x] = y.detach()
            if train:
                y.backward(s["d%s_out" % x].double())
                out["d" + x] = a.grad
                out["d%s_w" % x] = None if w is None else w.grad
        if c["cache"]:
            for x, rows in (("k", out["k"]), ("v", s["v"].double())):
                pool = s[x + "_pages"].double().view(-1, Hkv, dh)
                pool[s["slots"].view(-1)] = rows.reshape(-1, Hkv, dh)
                out[x + "_pages"] = pool.view(s[x + "_pages"].shape)
        return out
    if c["op"].startswith("attend"):
        B, T, train = c["B"], c["T"], c["op"] == "attend_train"
        o = torch.zeros(B, T, Hq, dh, dtype=torch.float64, device="cuda")
        lse = torch.full((B, Hq, T), -math.inf, dtype=torch.float64, device="cuda")
        grads = {x: torch.zeros(s[x].shape, dtype=torch.float64, device="cuda") for x in "qkv"}
        for b, n in enumerate(_lens(c)):
            for h in range(Hq):
                g = h // (Hq // Hkv)
                q, k, v = (x[b, :n, y].double().requires_grad_(train)
                           for x, y in ((s["q"], h), (s["k"], g), (s["v"], g)))
                a, lse_h = _exact_attend_head(q, k, v, c["window"], c["sinks"])
                o[b, :n, h], lse[b, h, :n] = a.detach(), lse_h.detach()
                if train:
                    a.backward(s["do"][b, :n, h].double())
                    for x, y, leaf in (("q", h, q), ("k", g, k), ("v", g, v)):
                        grads[x][b, :n, y] += leaf.grad
        if not train:
            return dict(o=o)
        return dict(o=o, lse=lse, dq=grads["q"], dk=grads["k"], dv=grads["v"])
    o = torch.zeros(c["N"], Hq, dh, dtype=torch.float64, device="cuda")
    for i, n in enumerate(s["lens"].tolist()):
        if not n:
            continue
        at = torch.arange(n, device="cuda")
        at = at[(at >= n - c["window"]) | (at < c["sinks"])]
        page, row = s["block_table"][i, at // c["page"]].long(), at % c["page"]
        k, v = s["k_pages"][page, row].double(), s["v_pages"][page, row].double()
        for h in range(Hq):
            g = h // (Hq // Hkv)
            o[i, h] = torch.softmax(k[:, g] @ s["q"][i, h].double() / math.sqrt(dh), 0) @ v[:, g]
    return o
