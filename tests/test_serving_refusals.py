"""Host-side checks of the serving operators' entry points (no GPU, nothing is launched): every bad argument is refused
with the documented status, and the binding refuses tensors that do not fit before any call. Device addresses are fake
and never dereferenced."""
import pytest
import torch

import gated_linear_recurrence_conv1d_amd as rg

lib = rg._lib
BAD, UNSUP, WS = rg.RGLRU_ERR_INVALID_ARG, rg.RGLRU_ERR_UNSUPPORTED, rg.RGLRU_ERR_WORKSPACE
BASE, STEP = 0x100000000, 0x10000000
BF, F32, I32, I64 = torch.bfloat16, torch.float32, torch.int32, torch.int64
E4, E8 = torch.float8_e4m3fn, torch.float8_e8m0fnu


def at(names):
    return {n: BASE + i * STEP for i, n in enumerate(names)}


W_PTRS = ["k", "v", "slots", "k_pages", "v_pages", "k_scales", "v_scales"]
WA = at(W_PTRS)


def write(**kw):
    a = dict(WA, rows=10, Hkv=2, dh=128, k_stride=256, v_stride=512, n_slots=64, dt=rg.RGLRU_BF16)
    a.update(kw)
    return lib.rglru_cache_quantize(*[a[n] for n in W_PTRS], a["rows"], a["Hkv"], a["dh"], a["k_stride"], a["v_stride"],
                                    a["n_slots"], a["dt"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=0), BAD), (dict(Hkv=0), BAD), (dict(dh=0), BAD), (dict(dt=2), UNSUP), (dict(dh=96), UNSUP),
    (dict(n_slots=0), BAD), (dict(n_slots=0x7FFFFF00), UNSUP), (dict(Hkv=70000, k_stride=1 << 24, v_stride=1 << 24), UNSUP),
    (dict(rows=0x7FFFFFFF, Hkv=60000, k_stride=1 << 23, v_stride=1 << 23), UNSUP),
    *[({n: None}, BAD) for n in W_PTRS],
    (dict(k=WA["k"] + 8), BAD), (dict(k_stride=255), BAD), (dict(k_stride=260), BAD), (dict(v_stride=516), BAD),
    (dict(v_stride=128), BAD), (dict(dt=rg.RGLRU_F32, v_stride=258), BAD), (dict(slots=WA["slots"] + 4), BAD),
    (dict(k_pages=WA["k_pages"] + 4), BAD), (dict(k_pages=WA["v_pages"]), BAD), (dict(k_pages=WA["k"]), BAD),
    (dict(v_scales=WA["k_scales"] + 64), BAD), (dict(k_scales=WA["slots"] + 72), BAD), (dict(v_pages=WA["v"] + 16), BAD),
])
def test_cache_quantize_refusals(kw, status):
    assert write(**kw) == status


R_PTRS = ["k_pages", "v_pages", "k_scales", "v_scales", "block_table", "lens", "starts", "k_out", "v_out"]
RA = at(R_PTRS)


def read(**kw):
    a = dict(RA, B=3, T=20, Hkv=2, dh=128, k_stride=256, v_stride=512, num_pages=9, page=16, max_pages=4, rest=1,
             dt=rg.RGLRU_F32)
    a.update(kw)
    return lib.rglru_cache_dequantize(*[a[n] for n in R_PTRS], a["B"], a["T"], a["Hkv"], a["dh"], a["k_stride"],
                                      a["v_stride"], a["num_pages"], a["page"], a["max_pages"], a["rest"], a["dt"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), BAD), (dict(T=0), BAD), (dict(Hkv=0), BAD), (dict(dt=3), UNSUP), (dict(dh=32), UNSUP),
    (dict(num_pages=0), BAD), (dict(page=0), BAD), (dict(max_pages=0), BAD), (dict(page=1 << 29), UNSUP),
    (dict(max_pages=1 << 27), UNSUP), (dict(T=0x7FFFFF00), UNSUP), (dict(B=1 << 20, T=1 << 20), UNSUP),
    *[({n: None}, BAD) for n in R_PTRS if n != "starts"],
    (dict(k_out=RA["k_out"] + 8), BAD), (dict(k_stride=254), BAD), (dict(v_stride=514), BAD),
    (dict(k_pages=RA["k_pages"] + 8), BAD), (dict(lens=RA["lens"] + 2), BAD), (dict(starts=RA["starts"] + 1), BAD),
    (dict(block_table=RA["block_table"] + 2), BAD), (dict(k_out=RA["v_out"]), BAD), (dict(k_out=RA["k_pages"] + 16), BAD),
    (dict(v_out=RA["v_scales"] - 1024), BAD), (dict(v_out=RA["lens"]), BAD),
])
def test_cache_dequantize_refusals(kw, status):
    assert read(**kw) == status


def test_outputs_may_share_a_row():
    """k_out and v_out as parts of one tensor's rows do not overlap (the call below ends at its missing lengths)."""
    both = dict(k_stride=512, v_stride=512, v_out=RA["k_out"] + 256 * 4)
    assert read(lens=None, **both) == BAD
    assert read(k_stride=512, v_stride=512, v_out=RA["k_out"] + 255 * 4 + 4 - 16) == BAD


P_PTRS = ["q", "k_pages", "v_pages", "k_scales", "v_scales", "block_table", "lens", "o"]
PA = at(P_PTRS)
WSP = BASE + 40 * STEP


def paged(**kw):
    a = dict(PA, N=4, Hq=4, Hkv=2, dh=128, q_stride=512, num_pages=9, page=16, max_pages=100, window=64, sinks=2,
             scale=0.0, ws=WSP, wsb=1 << 26)
    a.update(kw)
    return lib.rglru_paged_attention_e4m3(*[a[n] for n in P_PTRS], a["N"], a["Hq"], a["Hkv"], a["dh"], a["q_stride"],
                                          a["num_pages"], a["page"], a["max_pages"], a["window"], a["sinks"],
                                          a["scale"], a["ws"], a["wsb"], None)


SIZES = [(dict(N=0), BAD), (dict(Hq=0), BAD), (dict(Hkv=0), BAD), (dict(Hkv=3), BAD), (dict(dh=32), UNSUP),
         (dict(window=0), BAD), (dict(sinks=-1), BAD), (dict(num_pages=0), BAD), (dict(page=0), BAD),
         (dict(max_pages=0), BAD), (dict(scale=-1.0), BAD), (dict(scale=float("nan")), BAD),
         (dict(scale=float("inf")), BAD), (dict(num_pages=1 << 28), UNSUP), (dict(max_pages=1 << 28), UNSUP),
         (dict(q_stride=511), BAD), (dict(q_stride=516), BAD), (dict(N=1 << 29), UNSUP)]


@pytest.mark.parametrize("kw,status", SIZES + [
    *[({n: None}, BAD) for n in P_PTRS],
    (dict(q=PA["q"] + 8), BAD), (dict(k_pages=PA["k_pages"] + 8), BAD), (dict(o=PA["o"] + 1), BAD),
    (dict(lens=PA["lens"] + 2), BAD), (dict(block_table=PA["block_table"] + 1), BAD),
    (dict(o=PA["q"]), BAD), (dict(o=PA["k_scales"] - 64), BAD), (dict(o=PA["v_pages"]), BAD),
    (dict(window=1 << 30, ws=None), WS), (dict(window=1 << 30, wsb=16), WS), (dict(window=1 << 30, ws=WSP + 4), BAD),
    (dict(window=1 << 30, ws=PA["v_scales"]), BAD), (dict(window=1 << 30, ws=PA["o"]), BAD),
])
def test_paged_attention_e4m3_refusals(kw, status):
    assert paged(**kw) == status


X_PTRS = ["q", "k_pages", "v_pages", "k_scales", "v_scales", "prefix_table", "prefix_len", "block_table", "lens", "o"]
XA = at(X_PTRS)


def prefix(**kw):
    a = dict(XA, N=4, Hq=4, Hkv=2, dh=128, q_stride=512, num_pages=9, page=16, prefix_pages=5, max_pages=100, window=64,
             sinks=2, scale=0.0, dt=rg.RGLRU_BF16, ws=WSP, wsb=1 << 26)
    a.update(kw)
    return lib.rglru_prefix_attention(*[a[n] for n in X_PTRS], a["N"], a["Hq"], a["Hkv"], a["dh"], a["q_stride"],
                                      a["num_pages"], a["page"], a["prefix_pages"], a["max_pages"], a["window"],
                                      a["sinks"], a["scale"], a["dt"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,status", SIZES + [
    (dict(prefix_pages=0), BAD), (dict(prefix_pages=1 << 28), UNSUP), (dict(dt=rg.RGLRU_F32), UNSUP),
    *[({n: None}, BAD) for n in X_PTRS],  # (one scale without the other among them)
    (dict(q=XA["q"] + 8), BAD), (dict(v_pages=XA["v_pages"] + 8), BAD), (dict(o=XA["o"] + 1), BAD),
    (dict(prefix_table=XA["prefix_table"] + 2), BAD), (dict(prefix_len=XA["prefix_len"] + 2), BAD),
    (dict(o=XA["prefix_len"] - 16), BAD), (dict(o=XA["prefix_table"]), BAD), (dict(o=XA["q"]), BAD),
    (dict(ws=None), WS), (dict(wsb=64), WS), (dict(ws=WSP + 8), BAD), (dict(ws=XA["prefix_table"]), BAD),
    (dict(ws=XA["o"]), BAD), (dict(ws=XA["k_pages"]), BAD),
])
def test_prefix_attention_refusals(kw, status):
    assert prefix(**kw) == status


def test_prefix_workspace():
    size = rg.rglru_prefix_attention_workspace_size
    assert size(4, 4, 2, 128, 16, 5, 100, 64, 2) > 0
    assert size(4, 4, 3, 128, 16, 5, 100, 64, 2) == 0 and size(4, 4, 2, 128, 16, 0, 100, 64, 2) == 0
    need = size(4, 4, 2, 128, 16, 5, 100, 64, 2)
    assert prefix(wsb=need - 1) == WS
    assert prefix(wsb=need, o=XA["q"]) == BAD
    assert prefix(k_scales=None, v_scales=None, wsb=need - 1) == WS  # a bf16 cache: the same


L_PTRS = ["q", "k", "v", "log_decay", "lens", "s0", "o", "s_out"]
LA = at(L_PTRS)


def linear(**kw):
    a = dict(LA, B=1, T=8192, Hk=2, H=4, dk=128, dv=64, q_stride=256, k_stride=512, v_stride=256, gated=1, scale=0.0,
             dt=rg.RGLRU_BF16, ws=WSP, wsb=1 << 30)
    a.update(kw)
    return lib.rglru_linear_attention(*[a[n] for n in L_PTRS], a["B"], a["T"], a["Hk"], a["H"], a["dk"], a["dv"],
                                      a["q_stride"], a["k_stride"], a["v_stride"], a["gated"], a["scale"], a["dt"],
                                      a["ws"], a["wsb"], None)


STATE_SIZES = [
    (dict(Hk=0), BAD), (dict(H=0), BAD), (dict(H=3), BAD), (dict(dk=0), BAD), (dict(dv=0), BAD), (dict(dk=96), UNSUP),
    (dict(dv=32), UNSUP), (dict(dt=rg.RGLRU_F32), UNSUP), (dict(scale=-1.0), BAD), (dict(scale=float("nan")), BAD),
    (dict(scale=float("inf")), BAD), (dict(q_stride=248), BAD), (dict(k_stride=260), BAD), (dict(v_stride=192), BAD),
    (dict(q_stride=(1 << 20) + 8), UNSUP), (dict(H=70000, Hk=1, v_stride=70000 * 64), UNSUP)]


@pytest.mark.parametrize("kw,status", STATE_SIZES + [
    (dict(B=0), BAD), (dict(T=0), BAD), (dict(T=0x7FFFFF00), UNSUP), (dict(B=1 << 24), UNSUP),
    *[({n: None}, BAD) for n in ("q", "k", "v", "log_decay", "o")],
    (dict(q=LA["q"] + 8), BAD), (dict(s0=LA["s0"] + 4), BAD), (dict(s_out=LA["s_out"] + 8), BAD),
    (dict(log_decay=LA["log_decay"] + 2), BAD), (dict(lens=LA["lens"] + 2), BAD), (dict(o=LA["v"]), BAD),
    (dict(o=LA["q"] + 256), BAD), (dict(s_out=LA["s0"] + 16), BAD), (dict(s_out=LA["k"]), BAD), (dict(s_out=LA["o"]), BAD),
    (dict(o=LA["s0"]), BAD), (dict(s_out=LA["log_decay"]), BAD),
    (dict(ws=None), WS), (dict(wsb=100), WS), (dict(ws=WSP + 4), BAD), (dict(ws=LA["s0"]), BAD), (dict(ws=LA["o"]), BAD),
])
def test_linear_attention_refusals(kw, status):
    assert linear(**kw) == status


def test_linear_workspace():
    size = rg.rglru_linear_attention_workspace_size
    need = size(1, 8192, 2, 4, 128, 64)
    assert need > 0 and linear(wsb=need - 1) == WS and linear(wsb=need, o=LA["q"]) == BAD
    assert size(64, 64, 16, 16, 128, 128) == 0  # one segment: none is needed
    assert size(1, 0, 2, 4, 128, 64) == 0 and size(1, 8192, 3, 4, 128, 64) == 0


@pytest.mark.parametrize("B,H", [(64, 16), (1, 256), (1, 1), (3, 1), (2, 8)])
@pytest.mark.parametrize("T", [(1 << 30) + 1, 2_000_000_000, 0x7FFFFEFF])
def test_linear_workspace_of_the_longest_prompts(B, H, T):
    """Segments of more than 2^30 tokens: their number is that of half as many tokens, and a length behind the last one's
    end passes 2^31."""
    size = rg.rglru_linear_attention_workspace_size
    assert size(B, T, 1, H, 64, 128) == size(B, 1 << 30, 1, H, 64, 128) < 1 << 32
    assert size(B, 0x7FFFFF00, 1, H, 64, 128) == 0  # refused


T_PTRS = ["q", "k", "v", "log_decay", "s_in", "s_out", "o"]
TA = at(T_PTRS)


def step(**kw):
    a = dict(TA, N=5, Hk=2, H=4, dk=128, dv=64, q_stride=256, k_stride=512, v_stride=256, gated=1, scale=0.0,
             dt=rg.RGLRU_BF16)
    a.update(kw)
    return lib.rglru_linear_attention_step(*[a[n] for n in T_PTRS], a["N"], a["Hk"], a["H"], a["dk"], a["dv"],
                                           a["q_stride"], a["k_stride"], a["v_stride"], a["gated"], a["scale"], a["dt"],
                                           None)


@pytest.mark.parametrize("kw,status", STATE_SIZES + [
    (dict(N=0), BAD), (dict(N=1 << 24), UNSUP), *[({n: None}, BAD) for n in T_PTRS],
    (dict(v=TA["v"] + 8), BAD), (dict(s_in=TA["s_in"] + 4), BAD), (dict(log_decay=TA["log_decay"] + 1), BAD),
    (dict(o=TA["q"]), BAD), (dict(o=TA["s_in"]), BAD), (dict(s_out=TA["s_in"] + 64), BAD), (dict(s_out=TA["v"]), BAD),
    (dict(o=TA["s_out"] + 16), BAD), (dict(s_in=TA["o"], s_out=TA["o"]), BAD),
])
def test_linear_attention_step_refusals(kw, status):
    assert step(**kw) == status


def test_binding_refuses_what_does_not_fit():
    """Host tensors whose first fault is not their device: each message names its tensor."""
    z = lambda *s, dtype=BF: torch.zeros(*s, dtype=dtype)  # noqa: E731
    k, slots = z(3, 5, 2, 64), z(3, 5, dtype=I64)
    pages, scales = z(9, 16, 2, 64, dtype=torch.uint8).view(E4), z(9, 16, 2, dtype=torch.uint8).view(E8)
    cache = (pages, pages, scales, scales)
    table, lens, q = z(3, 4, dtype=I32), z(3, dtype=I32), z(3, 4, 64)
    no = pytest.raises
    with no(TypeError, match="k: expected a torch.Tensor"):
        rg.cache_quantize(None, k, slots, *cache)
    with no(ValueError, match="k: unsupported dtype torch.float64"):
        rg.cache_quantize(k.double(), k, slots, *cache)
    with no(ValueError, match="slots: expected torch.int64"):
        rg.cache_quantize(k, k, slots.int(), *cache)
    with no(ValueError, match=r"slots: expected shape \(3, 5\)"):
        rg.cache_quantize(k, k, slots.view(-1), *cache)
    with no(ValueError, match="k_pages: expected .* of k's heads"):
        rg.cache_quantize(k[..., :32], k, slots, *cache)
    with no(ValueError, match="k_pages: expected torch.float8_e4m3fn"):
        rg.cache_quantize(k, k, slots, z(9, 16, 2, 64), pages, scales, scales)
    with no(ValueError, match="v_scales: expected torch.float8_e8m0fnu"):
        rg.cache_quantize(k, k, slots, pages, pages, scales, z(9, 16, 2, dtype=F32))
    with no(ValueError, match="k_scales: expected shape"):
        rg.cache_quantize(k, k, slots, pages, pages, scales[:8], scales)
    with no(TypeError, match="v: expected a torch.Tensor"):
        rg.cache_quantize(k, None, slots, *cache)
    with no(TypeError, match="cache: expected a torch.Tensor"):
        rg.cache_quantize(k, k, slots, pages, None, scales, scales)
    with no(ValueError, match="device"):
        rg.cache_quantize(k, k, slots, *cache)
    with no(ValueError, match="k_out: expected .* of the cache's heads"):
        rg.rglru_cache_dequantize(*cache, table, lens, z(3, 5, 1, 64), z(3, 5, 1, 64))
    with no(ValueError, match="v_out: expected torch.bfloat16"):
        rg.rglru_cache_dequantize(*cache, table, lens, k, k.float())
    with no(ValueError, match="starts: expected torch.int32"):
        rg.rglru_cache_dequantize(*cache, table, lens, k, k, lens.long())
    with no(ValueError, match="k_out: unsupported dtype torch.float16"):
        rg.cache_dequantize(*cache, table, lens, 5, dtype=torch.float16)
    with no(ValueError, match="device"):
        rg.cache_dequantize(*cache, table, lens, 5)
    with no(ValueError, match="q: expected torch.bfloat16, got torch.float32"):
        rg.paged_attention_e4m3(q.float(), *cache, table, lens, 10)
    with no(ValueError, match="k_pages: expected torch.float8_e4m3fn"):
        rg.paged_attention_e4m3(q, z(9, 16, 2, 64), pages, scales, scales, table, lens, 10)
    with no(ValueError, match="k_pages: expected shape"):
        rg.paged_attention_e4m3(z(3, 4, 128), *cache, table, lens, 10)
    with no(ValueError, match="device"):
        rg.paged_attention_e4m3(q, *cache, table, lens, 10)
    pt, pl = z(2, dtype=I32), z(1, dtype=I32)
    with no(ValueError, match="both or none"):
        rg.prefix_attention(q, pages, pages, pt, pl, table, lens, 10, k_scales=scales)
    with no(ValueError, match=r"prefix_len: expected shape \(1,\)"):
        rg.prefix_attention(q, pages, pages, pt, z(2, dtype=I32), table, lens, 10, k_scales=scales, v_scales=scales)
    with no(ValueError, match="prefix_table: expected .prefix_pages"):
        rg.prefix_attention(q, pages, pages, table, pl, table, lens, 10, k_scales=scales, v_scales=scales)
    with no(ValueError, match="k_pages: expected torch.bfloat16"):
        rg.prefix_attention(q, pages, pages, pt, pl, table, lens, 10)
    with no(ValueError, match="device"):
        rg.prefix_attention(q, z(9, 16, 2, 64), z(9, 16, 2, 64), pt, pl, table, lens, 10)
    x, v, g = z(2, 7, 2, 64), z(2, 7, 4, 128), z(4, dtype=F32)
    with no(ValueError, match=r"log_decay: expected shape \(2, 7, 4\)"):
        rg.linear_attention(x, x, v, z(2, 7, 2, dtype=F32))
    with no(ValueError, match=r"log_decay: expected shape \(4,\)"):
        rg.linear_attention(x, x, v, z(5, dtype=F32))
    with no(ValueError, match="state: expected shape"):
        rg.linear_attention(x, x, v, g, z(2, 4, 128, 64, dtype=F32))
    with no(ValueError, match="state: expected torch.float32"):
        rg.linear_attention(x, x, v, g, z(2, 4, 64, 128))
    with no(ValueError, match="k: expected shape"):
        rg.linear_attention(x, x[:, :6], v, g)
    with no(ValueError, match="v: expected .B, T, H, dv"):
        rg.linear_attention(x, x, v[0], g)
    with no(ValueError, match="device"):
        rg.linear_attention(x, x, v, g)
    with no(ValueError, match=r"log_decay: expected shape \(2, 4\)"):
        rg.linear_attention_step(x[:, 0], x[:, 0], v[:, 0], z(2, 3, dtype=F32), z(2, 4, 64, 128, dtype=F32))
    with no(TypeError, match="state: expected a torch.Tensor"):
        rg.linear_attention_step(x[:, 0], x[:, 0], v[:, 0], g, 3)
    with no(ValueError, match="device"):
        rg.linear_attention_step(x[:, 0], x[:, 0], v[:, 0], g, z(2, 4, 64, 128, dtype=F32))
