"""What a serving process keeps from token to token, and what reads it, as measured work: the operators' inputs, their
plain forms in torch, and what each has to read, write and compute.

  chunk    a chunk of new tokens' keys and values into a paged cache of e4m3 values with a power-of-two scale for each
           (token, head), and each sequence's last tokens read back from it
  step     one new token per sequence: its key and value into that cache, and its attention over the cache
  prefix   attention of one new token per sequence, the sequences sharing a long prefix that the cache holds once
           (bf16 or e4m3)
  linear   causal linear attention with a decay for each head: prompts, from a state and to a state
  token    one token of the same recurrence per sequence

A case says the operator ("op"), the types and sizes; `prepare` makes the inputs, `run` is one pass.
"""
import math

import torch

own = False  # True: run() calls the framework's kernels; False: the plain forms below

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EVERY = 1 << 30  # a window beyond every sequence


# ---------------------------------------------------------------------------------------------- cases
def _chunk(name, dtype, B, new, shortest, longest, span, Hkv, dh, page):
    return dict(op="chunk", name=name, dtype=dtype, B=B, new=new, shortest=shortest, longest=longest, span=span,
                Hkv=Hkv, dh=dh, page=page)


def _step(name, N, Hq, Hkv, dh, shortest, longest, window, sinks, page):
    return dict(op="step", name=name, N=N, Hq=Hq, Hkv=Hkv, dh=dh, shortest=shortest, longest=longest, window=window,
                sinks=sinks, page=page)


def _prefix(name, cache, N, Hq, Hkv, dh, prefix, shortest, longest, window, sinks, page):
    return dict(op="prefix", name=name, cache=cache, N=N, Hq=Hq, Hkv=Hkv, dh=dh, prefix=prefix, shortest=shortest,
                longest=longest, window=window, sinks=sinks, page=page)


def _linear(name, B, T, Hk, H, dk, dv, ragged, gated, start):
    return dict(op="linear", name=name, B=B, T=T, Hk=Hk, H=H, dk=dk, dv=dv, ragged=ragged, gated=gated, start=start)


def _token(name, N, Hk, H, dk, dv, gated):
    return dict(op="token", name=name, N=N, Hk=Hk, H=H, dk=dk, dv=dv, gated=gated)


def listed():
    return [
        # a chunk of 512 prompt tokens in each of 8 sequences of the 2B-shaped layer, which then needs the window of
        # 2048 before the chunk's end
        _chunk("chunk_b8_new512_span2048_dh256", "bf16", 8, 512, 512, 6000, 2048, 1, 256, 64),
        # one long document in fp32 with grouped heads, pages of an odd size: 16384 new tokens, all read back
        _chunk("chunk_f32_b1_new16384_all_hkv2_dh128", "f32", 1, 16384, 65000, 65000, 65000, 2, 128, 17),
        # one sequence's next token in a local window: latency
        _step("step_n1_hq10_dh256_w1024", 1, 10, 1, 256, 1500, 1500, 1024, 4, 16),
        # a serving batch of the 9B-shaped layer, lengths from one token on, window 2048
        _step("step_n128_hq16_dh256_w2048", 128, 16, 1, 256, 1, 6000, 2048, 4, 64),
        # few users of one system prompt: latency
        _prefix("prefix_n6_hq10_dh256_p700", "bf16", 6, 10, 1, 256, 700, 1, 90, 2048, 0, 16),
        # a serving batch of the 9B-shaped layer on one prompt; the longer sequences' windows have left part of it
        _prefix("prefix_n64_hq16_dh256_p1999_w2048", "bf16", 64, 16, 1, 256, 1999, 1, 1500, 2048, 4, 64),
        # many answers to questions about one long document, grouped heads, e4m3 cache
        _prefix("prefix_e4m3_n256_hq8_hkv2_dh128_p32000", "e4m3", 256, 8, 2, 128, 32000, 0, 400, EVERY, 0, 32),
        # prompts of a serving batch, constant decays
        _linear("linear_b8_t2048_h16_dk128_dv128", 8, 2048, 16, 16, 128, 128, False, False, False),
        # one long document, values wider than keys, query and key heads shared by groups, decays of each token
        _linear("linear_b1_t65536_hk2_h8_dk128_dv256", 1, 65536, 2, 8, 128, 256, False, True, False),
        # a short padded batch of odd sizes that goes on from states
        _linear("linear_b5_t301_hk3_h6_dk64_dv64", 5, 301, 3, 6, 64, 64, True, True, True),
        # one sequence's next token: latency
        _token("token_n1_hk2_h8_dk128_dv128", 1, 2, 8, 128, 128, True),
        # a serving batch
        _token("token_n256_h16_dk128_dv256", 256, 16, 16, 128, 256, False),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _heads(rng, most):
    Hkv = rng.choice([1, 1, 1, 2, 3, 4])
    return Hkv * rng.randint(1, max(1, min(16, most // Hkv))), Hkv


def draw(rng):
    op = rng.choice(["chunk", "step", "prefix", "linear", "token"])
    page = rng.choice([1, 7, 16, 32, 64, 128, 256])
    dh = rng.choice([64, 128, 256])
    Hq, Hkv = _heads(rng, 16)
    if op == "chunk":
        B = _spread(rng, 1, 16)
        dtype = rng.choice(["bf16", "bf16", "f32"])
        longest = _spread(rng, 1, max(2, (16 << 20) // (B * Hkv * dh)))  # as many values as the listed ones
        new = _spread(rng, 1, max(1, longest // 2))
        case = _chunk(None, dtype, B, new, rng.choice([new, longest]), longest, _spread(rng, 1, longest), Hkv, dh, page)
    elif op == "step":
        N = _spread(rng, 1, 200)
        most = (384 << 20) // (N * Hkv * dh * 4)  # at most as many values as the listed ones read
        longest = _spread(rng, 1, min(131072, max(64, most)))
        window = rng.choice([EVERY, _spread(rng, 1, 2 * longest)])
        case = _step(None, N, Hq, Hkv, dh, rng.choice([1, (longest + 1) // 2]), longest, window,
                     rng.choice([0, 0, 1, 4, 50]), page)
    elif op == "prefix":
        N = _spread(rng, 1, 300)
        P = _spread(rng, 1, min(40000, (256 * 8 * 32000 * 128) // (N * Hq * dh)))
        longest = _spread(rng, 1, min(2000, max(1, (256 * 400 * 2 * 128) // (N * Hkv * dh))))
        window = rng.choice([EVERY, _spread(rng, 1, 2 * (P + longest))])
        case = _prefix(None, rng.choice(["bf16", "e4m3"]), N, Hq, Hkv, dh, P, rng.choice([0, 1, (longest + 1) // 2]),
                       longest, window, rng.choice([0, 0, 1, 4, 50]), page)
    else:
        Hk = rng.choice([1, 1, 2, 3, 4, 8])
        H = Hk * rng.choice([1, 1, 2, 3, 4])
        dk, dv = rng.choice([64, 128, 128, 256]), rng.choice([64, 128, 128, 256])
        gated = rng.random() < 0.5
        if op == "linear":
            B = _spread(rng, 1, 8)
            T = _spread(rng, 1, min(65536, (65536 * 8 * 128 * 256) // (B * H * dk * dv)))
            case = _linear(None, B, T, Hk, H, dk, dv, rng.random() < 0.5, gated, rng.random() < 0.5)
        else:
            case = _token(None, _spread(rng, 1, max(2, (256 * 16 * 128 * 256) // (H * dk * dv))), Hk, H, dk, dv, gated)
    del case["name"]
    return case


# --------------------------------------------------------------------------------------------- inputs
def _even(n, lo, hi):
    """n lengths spread evenly over lo .. hi."""
    return [hi if n == 1 else lo + (i * (hi - lo)) // (n - 1) for i in range(n)]


def _lens(case):
    """Lengths of a padded batch: from the full length down, the last sequence short."""
    B, T = case["B"], case["T"]
    return [max(1, T - (b * T) // (B + 1)) for b in range(B)] if case["ragged"] else [T] * B


def _quantized(x):
    """e4m3 values of x / s and s as e8m0, s the smallest power of two with max |x| / s <= 448, 2^-117 at least."""
    x = x.float()
    m, e = torch.frexp(x.abs().amax(-1))
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-117)
    y = torch.ldexp(x, -e[..., None])
    return y.to(torch.float8_e4m3fn), (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _values(codes, scales):
    """What the codes and scales stand for, in fp32."""
    e = scales.view(torch.uint8).int() - 127
    return torch.ldexp(codes.float(), e[..., None])


def _table(lens, page, gen, spare=1):
    """A block table for sequences of these lengths, their pages in any order; and how many pages there are."""
    dev = lens.device
    held = (lens + page - 1) // page
    width, total = max(1, int(held.max())), int(held.sum())
    table = torch.zeros(len(lens), width, dtype=torch.int32, device=dev)
    used = torch.arange(width, device=dev)[None] < held[:, None]
    table[used] = torch.randperm(total + spare, generator=gen, device=dev)[:total].to(torch.int32)
    return table, total + spare


def _decays(case, rows, H, normal):
    """Log decays: constant, from quickly forgetting heads to slowly forgetting ones, or of each token."""
    if case["gated"]:
        return -torch.nn.functional.softplus(normal(*rows, H, dtype=torch.float32) - 2)
    h = torch.arange(H, device="cuda", dtype=torch.float64)
    return torch.log1p(-torch.exp2(-4 - 5 * h / H)).float()


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    op, bf = case["op"], torch.bfloat16

    def normal(*shape, dtype=bf):
        return torch.randn(*shape, generator=gen, device=dev, dtype=torch.float32).to(dtype)

    def cache(pages, page, Hkv, dh, quantized=True):
        if not quantized:
            return dict(k_pages=normal(pages, page, Hkv, dh), v_pages=normal(pages, page, Hkv, dh))
        (k, ks), (v, vs) = _quantized(normal(pages, page, Hkv, dh)), _quantized(normal(pages, page, Hkv, dh))
        return dict(k_pages=k, v_pages=v, k_scales=ks, v_scales=vs)

    s = dict(case=case)
    if op == "chunk":
        B, page, Hkv, dh, new = case["B"], case["page"], case["Hkv"], case["dh"], case["new"]
        lens = torch.tensor(_even(B, max(new, case["shortest"]), max(new, case["longest"])), device=dev)
        table, pages = _table(lens, page, gen)
        s |= cache(pages, page, Hkv, dh)
        kv = normal(B, new, 2 * Hkv * dh, dtype=TYPES[case["dtype"]])  # the projection's output, keys and values
        s["k"], s["v"] = (x.unflatten(-1, (Hkv, dh)) for x in (kv[..., :Hkv * dh], kv[..., Hkv * dh:]))
        at = (lens[:, None] - new) + torch.arange(new, device=dev)
        s["slots"] = table.long().gather(1, at // page) * page + at % page
        s["block_table"], s["lens"] = table, lens.int()
        s["starts"] = (lens - case["span"]).clamp(min=0).int()
    elif op == "step":
        N, page, Hq, Hkv, dh = case["N"], case["page"], case["Hq"], case["Hkv"], case["dh"]
        lens = torch.tensor(_even(N, case["shortest"], case["longest"]), device=dev)
        lens = lens[torch.randperm(N, generator=gen, device=dev)]
        table, pages = _table(lens, page, gen)
        s |= cache(pages, page, Hkv, dh)
        qkv = normal(N, (Hq + 2 * Hkv) * dh)
        s["q"] = qkv[:, :Hq * dh].unflatten(-1, (Hq, dh))
        s["k"] = qkv[:, Hq * dh:(Hq + Hkv) * dh].unflatten(-1, (Hkv, dh))
        s["v"] = qkv[:, (Hq + Hkv) * dh:].unflatten(-1, (Hkv, dh))
        at = lens - 1
        s["slots"] = table.long().gather(1, (at // page)[:, None])[:, 0] * page + at % page
        s["block_table"], s["lens"] = table, lens.int()
    elif op == "prefix":
        N, page, Hq, Hkv, dh = case["N"], case["page"], case["Hq"], case["Hkv"], case["dh"]
        lens = torch.tensor(_even(N, case["shortest"], case["longest"]), device=dev)
        lens = lens[torch.randperm(N, generator=gen, device=dev)]
        shared = torch.tensor([case["prefix"]], device=dev)
        held = (case["prefix"] + page - 1) // page
        table, pages = _table(lens, page, gen, spare=held + 1)
        free = torch.ones(pages, dtype=torch.bool, device=dev)
        free[table[torch.arange(table.shape[1], device=dev)[None] < ((lens + page - 1) // page)[:, None]].long()] = False
        s["prefix_table"] = free.nonzero()[:held, 0].flip(0).to(torch.int32).contiguous()
        s["prefix_len"] = shared.int()
        s |= cache(pages, page, Hkv, dh, case["cache"] == "e4m3")
        s["q"], s["block_table"], s["lens"] = normal(N, Hq, dh), table, lens.int()
    else:
        Hk, H, dk, dv = case["Hk"], case["H"], case["dk"], case["dv"]
        rows = (case["B"], case["T"]) if op == "linear" else (case["N"],)
        qkv = normal(*rows, (2 * Hk * dk) + H * dv)
        s["q"] = qkv[..., :Hk * dk].unflatten(-1, (Hk, dk))
        s["k"] = qkv[..., Hk * dk:2 * Hk * dk].unflatten(-1, (Hk, dk))
        s["v"] = qkv[..., 2 * Hk * dk:].unflatten(-1, (H, dv))
        s["log_decay"] = _decays(case, rows, H, normal)
        if op == "token":
            s["state"] = normal(rows[0], H, dk, dv, dtype=torch.float32)
            s["state_out"] = torch.empty_like(s["state"])
        else:
            s["state"] = normal(rows[0], H, dk, dv, dtype=torch.float32) if case["start"] else None
            s["lens"] = torch.tensor(_lens(case), dtype=torch.int32, device=dev) if case["ragged"] else None
    return s


# ---------------------------------------------------------------------------------------- plain forms
def _store(s):
    """The new keys and values into the cache, quantised."""
    at = s["slots"].reshape(-1)
    for x in "kv":
        codes, scales = _quantized(s[x].flatten(0, -3))
        s[x + "_pages"].view(torch.uint8).flatten(0, 1)[at] = codes.view(torch.uint8)
        s[x + "_scales"].view(torch.uint8).flatten(0, 1)[at] = scales.view(torch.uint8)


def _rows(s, x, at):
    """Rows `at` of the cache of x (k or v), in fp32."""
    pool = s[x + "_pages"].flatten(0, 1)
    if "k_scales" not in s:
        return pool[at].float()
    codes = pool.view(torch.uint8)[at].view(torch.float8_e4m3fn)
    return _values(codes, s[x + "_scales"].view(torch.uint8).flatten(0, 1)[at].view(torch.float8_e8m0fnu))


def _span(c):
    return min(c["span"], max(c["new"], c["longest"]))


def _plain_chunk(s):
    c = s["case"]
    _store(s)
    T, page = _span(c), c["page"]
    u = s["starts"].long()[:, None] + torch.arange(T, device="cuda")[None]
    there = (u < s["lens"][:, None])[..., None, None]
    u = u.clamp(max=s["block_table"].shape[1] * page - 1)
    at = s["block_table"].long().gather(1, u // page) * page + u % page
    return {x: torch.where(there, _rows(s, x, at), 0.0).to(TYPES[c["dtype"]]) for x in "kv"}


def _softmax_parts(sc, seen):
    """exp of the scores less their row's maximum (0 where nothing is seen), and that maximum."""
    sc = sc.masked_fill(~seen, -math.inf)
    m = sc.amax(-1, keepdim=True)
    return (sc - torch.where(m == -math.inf, 0.0, m)).exp(), m


def _plain_step(s):
    c = s["case"]
    _store(s)
    N, Hq, Hkv, dh, page = c["N"], c["Hq"], c["Hkv"], c["dh"], c["page"]
    S, W = min(c["sinks"], c["longest"]), min(c["window"], c["longest"])
    lens = s["lens"].long()[:, None]
    j = torch.arange(S + W, device="cuda")[None]
    u = torch.where(j < S, j, (lens - W).clamp(min=S) + j - S)  # the sinks, then the window behind them
    seen = u < lens
    u = u.clamp(max=s["block_table"].shape[1] * page - 1)
    at = s["block_table"].long().gather(1, u // page) * page + u % page
    k, v = (_rows(s, x, at).transpose(1, 2).contiguous() for x in "kv")  # [N, Hkv, S + W, dh]
    sc = s["q"].float().reshape(N, Hkv, -1, dh) @ k.transpose(2, 3).contiguous() / math.sqrt(dh)
    p, _ = _softmax_parts(sc, seen[:, None, None])
    total = p.sum(-1, keepdim=True)
    return ((p @ v) / torch.where(total == 0, 1.0, total)).view(N, Hq, dh).to(s["q"].dtype)


def _plain_prefix(s):
    c = s["case"]
    N, Hq, Hkv, dh, page, P, W, S = (c[x] for x in ("N", "Hq", "Hkv", "dh", "page", "prefix", "window", "sinks"))
    G = Hq // Hkv
    q = s["q"].float().view(N, Hkv, G, dh)
    lens = s["lens"].long()[:, None]
    u = torch.arange(P, device="cuda")
    at = s["prefix_table"].long()[u // page] * page + u % page
    k, v = (_rows(s, x, at).transpose(0, 1).contiguous() for x in "kv")  # [Hkv, P, dh]: once for all
    seen = (u >= P + lens - W) | (u < S)  # [N, P]
    rows = q.transpose(0, 1).reshape(Hkv, N * G, dh)
    sc = (rows @ k.transpose(1, 2).contiguous()).view(Hkv, N, G, P) / math.sqrt(dh)
    p, m = _softmax_parts(sc, seen[None, :, None])
    o, total = (p.view(Hkv, N * G, P) @ v).view(Hkv, N, G, dh), p.sum(-1, keepdim=True)
    j = torch.arange(max(1, c["longest"]), device="cuda")[None]
    seen = (j < lens) & ((j >= lens - W) | (P + j < S))  # [N, longest]
    j = j.clamp(max=s["block_table"].shape[1] * page - 1).expand(N, -1)
    at = s["block_table"].long().gather(1, j // page) * page + j % page
    k, v = (_rows(s, x, at).transpose(1, 2).contiguous() for x in "kv")  # [N, Hkv, longest, dh]
    sc = q @ k.transpose(2, 3).contiguous() / math.sqrt(dh)
    p, m2 = _softmax_parts(sc, seen[:, None, None])
    o2, total2 = p @ v, p.sum(-1, keepdim=True)
    o, total, m = (x.transpose(0, 1) for x in (o, total, m))  # [N, Hkv, G, ..]
    top = torch.maximum(m, m2)
    top = torch.where(top == -math.inf, 0.0, top)
    w, w2 = (m - top).exp(), (m2 - top).exp()
    total = total * w + total2 * w2
    return ((o * w + o2 * w2) / torch.where(total == 0, 1.0, total)).reshape(N, Hq, dh).to(s["q"].dtype)


def _plain_linear(s):
    """Chunks of 128 tokens: inside a chunk by the decayed scores, between chunks by the chunks' own states."""
    c = s["case"]
    B, T, Hk, H, dk, dv, C = c["B"], c["T"], c["Hk"], c["H"], c["dk"], c["dv"], 128
    n = (T + C - 1) // C
    there = torch.arange(n * C, device="cuda")[None] < (T if s["lens"] is None else s["lens"].long()[:, None])

    def chunks(x):  # [B, T, heads, d] -> [B, H, n, C, d], zeros behind the last token
        x = torch.nn.functional.pad(x.float(), (0, 0, 0, 0, 0, n * C - T)) * there[..., None, None]
        x = x.repeat_interleave(H // x.shape[2], 2)
        return x.view(B, n, C, H, -1).permute(0, 3, 1, 2, 4).contiguous()

    q, k, v = (chunks(s[x]) for x in "qkv")
    g = s["log_decay"].double().expand(B, T, H)[..., None]
    g = torch.nn.functional.pad(g, (0, 0, 0, 0, 0, n * C - T)) * there[..., None, None]
    b = g.view(B, n, C, H).permute(0, 3, 1, 2).cumsum(-1)  # [B, H, n, C], each chunk's from its start
    t = torch.arange(C, device="cuda")
    d = (b[..., :, None] - b[..., None, :]).masked_fill(t[:, None] < t[None], -math.inf).exp().float()
    o = ((q @ k.transpose(3, 4).contiguous()) * d) @ v
    kept = (b[..., -1:] - b).exp().float()  # of each token's outer product at its chunk's end
    own_state = (k * kept[..., None]).transpose(3, 4).contiguous() @ v  # [B, H, n, dk, dv]
    end = torch.nn.functional.pad(b[..., -1].cumsum(-1), (1, 0))  # [B, H, n + 1]: up to each chunk's start
    i = torch.arange(n + 1, device="cuda")
    carry = (end[..., :, None] - end[..., None, 1:]).masked_fill(i[:, None] <= i[None, :n], -math.inf).exp().float()
    states = (carry @ own_state.view(B, H, n, dk * dv)).view(B, H, n + 1, dk, dv)
    if s["state"] is not None:
        states = states + end.exp().float()[..., None, None] * s["state"][:, :, None]
    o = o + (q * b.exp().float()[..., None]) @ states[:, :, :n]
    o = o.permute(0, 2, 3, 1, 4).reshape(B, n * C, H, dv)[:, :T] / math.sqrt(dk)
    return dict(o=torch.where(there[:, :T, None, None], o, 0.0).to(s["q"].dtype), state=states[:, :, n].contiguous())


def _plain_token(s):
    c = s["case"]
    q, k, v = (s[x].float().repeat_interleave(c["H"] // s[x].shape[1], 1) for x in "qkv")
    state = s["log_decay"].exp().expand(c["N"], c["H"])[..., None, None] * s["state"] + k[..., None] * v[..., None, :]
    o = (q[..., None, :] @ state)[..., 0, :] / math.sqrt(c["dk"])
    return dict(o=o.to(s["q"].dtype), state=state)


# ------------------------------------------------------------------------------------------- one pass
def run(s):
    c = s["case"]
    if not own:
        return {"chunk": _plain_chunk, "step": _plain_step, "prefix": _plain_prefix, "linear": _plain_linear,
                "token": _plain_token}[c["op"]](s)
    import gated_linear_recurrence_conv1d_amd as rg
    if c["op"] == "linear":
        o, state = rg.linear_attention(s["q"], s["k"], s["v"], s["log_decay"], s["state"], lens=s["lens"])
        return dict(o=o, state=state)
    if c["op"] == "token":
        o = rg.linear_attention_step(s["q"], s["k"], s["v"], s["log_decay"], s["state"], state_out=s["state_out"])
        return dict(o=o, state=s["state_out"])
    if c["op"] == "prefix":
        return rg.prefix_attention(s["q"], s["k_pages"], s["v_pages"], s["prefix_table"], s["prefix_len"],
                                   s["block_table"], s["lens"], c["window"], c["sinks"],
                                   k_scales=s.get("k_scales"), v_scales=s.get("v_scales"))
    cache = s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"]
    rg.cache_quantize(s["k"], s["v"], s["slots"], *cache)
    if c["op"] == "step":
        return rg.paged_attention_e4m3(s["q"], *cache, s["block_table"], s["lens"], c["window"], c["sinks"])
    k, v = rg.cache_dequantize(*cache, s["block_table"], s["lens"], _span(c), s["starts"], dtype=TYPES[c["dtype"]])
    return dict(k=k, v=v)


# ----------------------------------------------------------------------------------------------- work
def work(case):
    c = case
    if c["op"] == "chunk":
        e, head = 2 if c["dtype"] == "bf16" else 4, c["Hkv"] * c["dh"]
        stored = c["dh"] + 1  # bytes of a head's row: codes and a scale
        new = 2 * c["B"] * c["new"] * (head * e + c["Hkv"] * stored)
        read = sum(min(n, c["span"]) for n in _even(c["B"], max(c["new"], c["shortest"]), max(c["new"], c["longest"])))
        back = 2 * (read * c["Hkv"] * stored + c["B"] * _span(c) * head * e)
        return {"bytes": new + back, "flops": 2 * head * (3 * c["B"] * c["new"] + read)}
    if c["op"] in ("step", "prefix"):
        Hq, Hkv, dh = c["Hq"], c["Hkv"], c["dh"]
        row = Hkv * (2 * dh if c.get("cache") == "bf16" else dh + 1)
        lens, W, S = _even(c["N"], c["shortest"], c["longest"]), c["window"], c["sinks"]
        if c["op"] == "step":
            keys = sum(min(n, W) + min(S, max(0, n - W)) for n in lens)
            io = c["N"] * (2 * Hq * dh * 2 + 2 * Hkv * (2 * dh + dh + 1))
            return {"bytes": 2 * keys * row + io, "flops": 4 * keys * Hq * dh}
        P = c["prefix"]
        mine = sum(min(n, W) for n in lens)  # own tokens seen
        shared = [min(P, max(0, W - n)) + min(S, P - min(P, max(0, W - n))) for n in lens]
        return {"bytes": 2 * (mine + max(shared)) * row + 2 * c["N"] * Hq * dh * 2,
                "flops": 4 * (mine + sum(shared)) * Hq * dh}
    Hk, H, dk, dv = c["Hk"], c["H"], c["dk"], c["dv"]
    token = (2 * Hk * dk + 2 * H * dv) * 2 + (4 * H if c["gated"] else 0)  # q, k, v, o and decays
    state = 4 * H * dk * dv
    if c["op"] == "token":
        return {"bytes": c["N"] * (token + 2 * state), "flops": 5 * c["N"] * H * dk * dv}
    tokens = sum(_lens(c))
    return {"bytes": tokens * token + c["B"] * state * (2 if c["start"] else 1), "flops": 4 * tokens * H * dk * dv}


# ------------------------------------------------------------------------------------ in 64 bits, apart
def _exact_stored(x):
    """What a row stands for once it is stored: x to the nearest value n 2^e s, |n| < 16, e >= -9, s as defined."""
    x = x.double()
    top = x.abs().amax(-1, keepdim=True)
    s = torch.exp2(torch.ceil(torch.log2(top.clamp(min=1e-300) / 448)).clamp(min=-117))
    s = torch.where(top / s > 448, 2 * s, torch.where((top / s <= 224) & (s > 2.0 ** -117), s / 2, s))  # log2's rounding
    y = x / s
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step * s


def _exact_pool(s, x):
    """The cache of x (k or v) in 64 bits."""
    pool = s[x + "_pages"].double()
    if "k_scales" in s:
        pool = pool * torch.exp2(s[x + "_scales"].view(torch.uint8).double() - 127)[..., None]
    if "slots" in s:
        pool.view(-1, *pool.shape[2:])[s["slots"].view(-1)] = _exact_stored(s[x]).reshape(-1, *pool.shape[2:])
    return pool


def _exact_attend(q, k, v):
    """One sequence's token: q [Hq, dh] over the keys k and values v [n, Hkv, dh] that it sees."""
    G = q.shape[0] // k.shape[1]
    return torch.stack([torch.softmax(k[:, h // G] @ q[h] / math.sqrt(q.shape[1]), 0) @ v[:, h // G]
                        for h in range(q.shape[0])])


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "chunk":
        out = {}
        for x in "kv":
            pool = _exact_pool(s, x)
            back = torch.zeros(c["B"], _span(c), c["Hkv"], c["dh"], dtype=torch.float64, device="cuda")
            for b, (a, n) in enumerate(zip(s["starts"].tolist(), s["lens"].tolist())):
                u = torch.arange(a, min(n, a + _span(c)), device="cuda")
                back[b, :len(u)] = pool[s["block_table"][b, u // c["page"]].long(), u % c["page"]]
            out[x] = back
        return out
    if c["op"] in ("step", "prefix"):
        kp, vp = _exact_pool(s, "k"), _exact_pool(s, "v")
        P = c.get("prefix", 0)
        o = torch.zeros(c["N"], c["Hq"], c["dh"], dtype=torch.float64, device="cuda")
        for i, n in enumerate(s["lens"].tolist()):
            u = torch.arange(P + n, device="cuda")
            u = u[(u >= P + n - c["window"]) | (u < c["sinks"])]
            if not len(u):
                continue
            before, after = u[u < P], u[u >= P] - P
            pages = s["block_table"][i, after // c["page"]].long()
            if P:
                pages = torch.cat([s["prefix_table"][before // c["page"]].long(), pages])
            row = torch.cat([before, after]) % c["page"]
            o[i] = _exact_attend(s["q"][i].double(), kp[pages, row], vp[pages, row])
        return o
    H, dk, dv = c["H"], c["dk"], c["dv"]
    q, k, v = (s[x].double().unsqueeze(1) if c["op"] == "token" else s[x].double() for x in "qkv")
    N, T = q.shape[:2]
    decay = s["log_decay"].double().exp()
    decay = decay.expand(N, T, H) if decay.dim() == 1 else decay.view(N, T, H)
    state = torch.zeros(N, H, dk, dv, dtype=torch.float64, device="cuda")
    if s["state"] is not None:
        state += s["state"]
    lens = s.get("lens")
    o = torch.zeros(N, T, H, dv, dtype=torch.float64, device="cuda")
    group = torch.arange(H, device="cuda") // (H // c["Hk"])
    for t in range(T):  # the recurrence, token by token
        new = decay[:, t, :, None, None] * state + k[:, t, group][..., None] * v[:, t, :, None]
        if lens is not None:
            on = (t < lens)[:, None, None, None]
            new = torch.where(on, new, state)
        state = new
        ot = (q[:, t, group][..., None, :] @ state)[..., 0, :] / math.sqrt(dk)
        o[:, t] = ot if lens is None else ot * on[..., 0]
    return dict(o=o[:, 0] if c["op"] == "token" else o, state=state)
