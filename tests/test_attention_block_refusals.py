"""Host-side checks of the attention block's entry points (no GPU, nothing is launched): every bad
argument is refused with the documented status, and the binding refuses tensors that do not fit before
any call. Device addresses are fake and never dereferenced."""
import ctypes

import pytest
import torch

import gated_linear_recurrence_conv1d_amd as rg

lib = rg._lib
BAD, UNSUP, WS = rg.RGLRU_ERR_INVALID_ARG, rg.RGLRU_ERR_UNSUPPORTED, rg.RGLRU_ERR_WORKSPACE
BASE, STEP = 0x100000000, 0x10000000


def at(names):
    return {n: BASE + i * STEP for i, n in enumerate(names)}


ROPE_PTRS = ["q", "k", "v", "q_w", "k_w", "inv_freq", "positions", "slots", "q_out", "k_out", "k_pages", "v_pages"]


def rope(**kw):
    a = at(ROPE_PTRS)
    a.update(rows=10, Hq=4, Hkv=2, dh=128, rot=64, q_stride=512, k_stride=256, v_stride=256, q_out_stride=512,
             k_out_stride=256, n_slots=64, eps=1e-6, dt=rg.RGLRU_BF16)
    a.update(kw)
    return lib.rglru_qk_norm_rope(*[a[n] for n in ROPE_PTRS], a["rows"], a["Hq"], a["Hkv"], a["dh"], a["rot"],
                                  a["q_stride"], a["k_stride"], a["v_stride"], a["q_out_stride"],
                                  a["k_out_stride"], a["n_slots"], a["eps"], a["dt"], None)


A = at(ROPE_PTRS)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=0), BAD), (dict(Hq=0), BAD), (dict(Hkv=-1), BAD), (dict(dh=0), BAD), (dict(dt=5), UNSUP),
    (dict(dh=127, rot=2), UNSUP), (dict(dh=514, q_stride=4000, k_stride=4000, v_stride=4000, q_out_stride=4000,
                                        k_out_stride=4000), UNSUP),
    (dict(rot=63), BAD), (dict(rot=130), BAD), (dict(rot=-2), BAD),
    (dict(eps=0.0), BAD), (dict(eps=float("nan")), BAD), (dict(eps=float("inf")), BAD),
    (dict(q=None), BAD), (dict(k=None), BAD), (dict(positions=None), BAD), (dict(inv_freq=None), BAD),
    (dict(q_out=None), BAD), (dict(k_out=None, slots=None), BAD),
    (dict(q_w=None), BAD), (dict(k_w=None), BAD),                      # one without the other
    (dict(v=None), BAD), (dict(k_pages=None), BAD), (dict(v_pages=None), BAD), (dict(n_slots=0), BAD),
    (dict(q_stride=511), BAD), (dict(k_stride=128), BAD), (dict(v_stride=0), BAD), (dict(k_out_stride=255), BAD),
    (dict(q=A["q"] + 1), BAD), (dict(q_w=A["q_w"] + 2), BAD), (dict(slots=A["slots"] + 4), BAD),
    (dict(q_out=A["q"], q_out_stride=520), BAD),                       # q itself, other stride
    (dict(q_out=A["q"] + 256), BAD), (dict(q_out=A["k"]), BAD), (dict(k_out=A["q"]), BAD),
    (dict(k_pages=A["v"]), BAD), (dict(k_pages=A["v_pages"]), BAD), (dict(k_out=A["k_pages"]), BAD),
    (dict(k_out=A["q_out"] + 16), BAD), (dict(q_out=A["positions"]), BAD), (dict(v_pages=A["slots"]), BAD),
])
def test_norm_rope_refusals(kw, status):
    assert rope(**kw) == status


BWD_PTRS = ["q", "k", "q_w", "k_w", "inv_freq", "positions", "dq_out", "dk_out", "dq", "dk", "dq_w", "dk_w"]
BA = at(BWD_PTRS)
WSP = BASE + 40 * STEP


def rope_bwd(**kw):
    a = dict(BA, rows=10, Hq=4, Hkv=2, dh=128, rot=64, strides=(512, 256, 512, 256, 512, 256), eps=1e-6,
             dt=rg.RGLRU_F32, ws=WSP, wsb=1 << 24)
    a.update(kw)
    return lib.rglru_qk_norm_rope_backward(*[a[n] for n in BWD_PTRS], a["rows"], a["Hq"], a["Hkv"], a["dh"],
                                           a["rot"], *a["strides"], a["eps"], a["dt"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), BAD), (dict(dt=2), UNSUP), (dict(rot=1), BAD), (dict(eps=-1.0), BAD), (dict(q=None), BAD),
    (dict(dq_out=None), BAD), (dict(dk=None), BAD), (dict(dq_w=None), BAD), (dict(dk_w=None), BAD),
    (dict(q_w=None), BAD), (dict(strides=(512, 256, 511, 256, 512, 256)), BAD),
    (dict(strides=(512, 256, 512, 256, 512, 100)), BAD), (dict(dq=BA["dq"] + 2), BAD),
    (dict(ws=None), WS), (dict(wsb=10), WS), (dict(ws=WSP + 4), BAD), (dict(ws=BA["dq"]), BAD),
    (dict(dq=BA["q"]), BAD), (dict(dq=BA["dk_out"]), BAD), (dict(dk=BA["dq_out"]), BAD), (dict(dk=BA["dq"]), BAD),
    (dict(dq_w=BA["q_w"]), BAD), (dict(dq_w=BA["dk_w"]), BAD), (dict(dk_w=BA["dk"]), BAD),
])
def test_norm_rope_backward_refusals(kw, status):
    assert rope_bwd(**kw) == status


FWD_PTRS = ["q", "k", "v", "lens", "o", "lse"]
FA = at(FWD_PTRS)


def attn(**kw):
    a = dict(FA, B=2, T=64, Hq=4, Hkv=2, dh=128, q_stride=512, k_stride=256, v_stride=256, window=16, sinks=2,
             scale=0.0, dt=rg.RGLRU_BF16)
    a.update(kw)
    return lib.rglru_local_attention(*[a[n] for n in FWD_PTRS], a["B"], a["T"], a["Hq"], a["Hkv"], a["dh"],
                                     a["q_stride"], a["k_stride"], a["v_stride"], a["window"], a["sinks"],
                                     a["scale"], a["dt"], None)


SIZES = [
    (dict(B=0), BAD), (dict(T=0), BAD), (dict(Hq=0), BAD), (dict(Hkv=0), BAD), (dict(Hkv=3, k_stride=384, v_stride=384), BAD),
    (dict(window=0), BAD), (dict(sinks=-1), BAD), (dict(scale=-1.0), BAD), (dict(scale=float("nan")), BAD),
    (dict(scale=float("inf")), BAD), (dict(dh=96), UNSUP), (dict(dt=rg.RGLRU_F32), UNSUP), (dict(B=70000), UNSUP),
    (dict(q_stride=508), BAD), (dict(q_stride=516), BAD), (dict(k_stride=248), BAD), (dict(v_stride=260), BAD),
    (dict(q_stride=(1 << 20) + 8), UNSUP), (dict(T=1 << 22), UNSUP), (dict(T=1 << 14, v_stride=1 << 16), UNSUP),
]


@pytest.mark.parametrize("kw,status", SIZES + [
    (dict(q=None), BAD), (dict(k=None), BAD), (dict(v=None), BAD), (dict(o=None), BAD),
    (dict(k=FA["k"] + 8), BAD), (dict(lens=FA["lens"] + 2), BAD), (dict(lse=FA["lse"] + 2), BAD),
    (dict(o=FA["q"]), BAD), (dict(o=FA["v"] + 4096), BAD), (dict(o=FA["lens"] - 64), BAD), (dict(lse=FA["k"]), BAD),
    (dict(lse=FA["o"] + 1024), BAD),
])
def test_attention_refusals(kw, status):
    assert attn(**kw) == status


AB_PTRS = ["q", "k", "v", "lens", "o", "lse", "do", "dq", "dk", "dv"]
AB = at(AB_PTRS)


def attn_bwd(**kw):
    a = dict(AB, B=2, T=64, Hq=4, Hkv=2, dh=128, q_stride=512, k_stride=256, v_stride=256, dq_stride=512,
             dk_stride=256, dv_stride=256, window=16, sinks=2, scale=0.0, dt=rg.RGLRU_BF16, ws=WSP, wsb=1 << 27)
    a.update(kw)
    return lib.rglru_local_attention_backward(
        *[a[n] for n in AB_PTRS], a["B"], a["T"], a["Hq"], a["Hkv"], a["dh"], a["q_stride"], a["k_stride"],
        a["v_stride"], a["dq_stride"], a["dk_stride"], a["dv_stride"], a["window"], a["sinks"], a["scale"], a["dt"],
        a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,status", SIZES + [(dict([(n, None)]), BAD) for n in AB_PTRS if n != "lens"] + [
    (dict(dq_stride=504), BAD), (dict(dk_stride=252), BAD), (dict(dv_stride=8), BAD), (dict(dv=AB["dv"] + 8), BAD),
    (dict(ws=None), WS), (dict(wsb=100), WS), (dict(ws=WSP + 8), BAD),
    (dict(ws=AB["k"] - 1024), BAD),                                   # its 2 KB of delta end in k
    (dict(dq=AB["q"]), BAD), (dict(dq=AB["o"]), BAD), (dict(dk=AB["do"]), BAD), (dict(dk=AB["dv"]), BAD),
    (dict(dv=AB["lse"]), BAD),
    # one tensor with overlapping columns
    (dict(dk=AB["dq"] + 768, dq_stride=1024, dk_stride=1024), BAD),
])
def test_attention_backward_refusals(kw, status):
    assert attn_bwd(**kw) == status


def test_attention_backward_grid_limit():
    """Sizes whose key blocks a launch's grid cannot count are refused, and have no workspace: 65535 blocks
    of 1024 heads at dh / 4 workgroups each are 2147450880 at dh 128, which 2^31 - 1 holds, and twice that at
    dh 256."""
    wide = dict(B=65535, T=1, Hq=1024, Hkv=1024, dh=256, **{n: 1 << 18 for n in (
        "q_stride", "k_stride", "v_stride", "dq_stride", "dk_stride", "dv_stride")})
    assert attn_bwd(**wide) == UNSUP
    assert rg.rglru_local_attention_backward_workspace_size(65535, 1, 1024, 1024, 256, 16) == 0
    assert rg.rglru_local_attention_backward_workspace_size(65535, 1, 1024, 1024, 128, 16) > 0


PG_PTRS = ["q", "k_pages", "v_pages", "block_table", "lens", "o"]
PA = at(PG_PTRS)


def paged(**kw):
    a = dict(PA, N=3, Hq=4, Hkv=2, dh=128, q_stride=512, num_pages=9, page=32, max_pages=20, window=1 << 30, sinks=0,
             scale=0.0, dt=rg.RGLRU_BF16, ws=WSP, wsb=1 << 27)
    a.update(kw)
    return lib.rglru_paged_attention(*[a[n] for n in PG_PTRS], a["N"], a["Hq"], a["Hkv"], a["dh"], a["q_stride"],
                                     a["num_pages"], a["page"], a["max_pages"], a["window"], a["sinks"], a["scale"],
                                     a["dt"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(N=0), BAD), (dict(Hq=3), BAD), (dict(Hkv=0), BAD), (dict(dh=96), UNSUP), (dict(dt=4), UNSUP),
    (dict(page=0), BAD), (dict(max_pages=0), BAD), (dict(num_pages=0), BAD), (dict(window=0), BAD),
    (dict(sinks=-3), BAD), (dict(scale=-0.5), BAD), (dict(scale=float("inf")), BAD), (dict(q_stride=511), BAD),
    (dict(q_stride=516), BAD), (dict(max_pages=1 << 27), UNSUP), (dict(num_pages=1 << 27), UNSUP),
    (dict(N=1 << 29), UNSUP),
    (dict(q=None), BAD), (dict(k_pages=None), BAD), (dict(v_pages=None), BAD), (dict(block_table=None), BAD),
    (dict(lens=None), BAD), (dict(o=None), BAD), (dict(q=PA["q"] + 8), BAD), (dict(v_pages=PA["v_pages"] + 2), BAD),
    (dict(o=PA["o"] + 1), BAD), (dict(lens=PA["lens"] + 1), BAD), (dict(ws=None), WS), (dict(wsb=64), WS),
    (dict(ws=WSP + 4), BAD), (dict(ws=PA["o"]), BAD), (dict(o=PA["q"]), BAD), (dict(o=PA["v_pages"] + 64), BAD),
    (dict(o=PA["block_table"]), BAD),
])
def test_paged_attention_refusals(kw, status):
    assert paged(**kw) == status


def test_workspace_sizes():
    n = rg.rglru_paged_attention_workspace_size(3, 4, 2, 128, 32, 20, 1 << 40, 0, "bf16")
    assert n >= 3 * 5 * 4 * 130 * 4                                    # five chunks of four tiles
    assert rg.rglru_paged_attention_workspace_size(3, 4, 2, 128, 32, 4, 1 << 30, 0, "bf16") == 0  # one chunk
    assert rg.rglru_paged_attention_workspace_size(3, 4, 2, 128, 32, 20, 1, 0, "bf16") == 0
    assert rg.rglru_paged_attention_workspace_size(3, 5, 2, 128, 32, 20, 1 << 30, 0, "bf16") == 0  # refused
    # longer batches need no less, and a longer window no less
    sizes = [rg.rglru_paged_attention_workspace_size(4, 8, 2, 128, 32, 4096, w, 0, "f32") for w in (64, 4096, 1 << 30)]
    assert sizes == sorted(sizes) and sizes[0] < sizes[2]
    assert rg.rglru_qk_norm_rope_backward_workspace_size(10, 128) >= 2 * 128 * 4
    assert rg.rglru_qk_norm_rope_backward_workspace_size(0, 128) == 0
    assert rg.rglru_local_attention_backward_workspace_size(2, 64, 4, 2, 128, 16) >= 2 * 64 * 4 * 4
    assert rg.rglru_local_attention_backward_workspace_size(2, 64, 3, 2, 128, 16) == 0


def test_columns_of_one_tensor_may_be_outputs_together():
    """dq, dk, dv side by side in one gradient tensor pass the overlap check (the call then ends at its
    missing workspace)."""
    assert attn_bwd(dq=AB["dq"], dk=AB["dq"] + 1024, dv=AB["dq"] + 1536, dq_stride=1024, dk_stride=1024,
                    dv_stride=1024, wsb=0) == WS


def test_binding_refuses_what_does_not_fit():
    """Host tensors: the binding stops before any call."""
    bf = torch.bfloat16
    q, k = torch.zeros(2, 5, 4, 64, dtype=bf), torch.zeros(2, 5, 2, 64, dtype=bf)
    pos, freq = torch.zeros(2, 5, dtype=torch.int32), torch.zeros(16)
    with pytest.raises(ValueError, match="device"):
        rg.local_attention(q, k, k, 4)
    with pytest.raises(ValueError, match="device"):
        rg.qk_norm_rope(q, k, pos, freq)
    with pytest.raises(ValueError, match="expected"):
        rg.rglru_local_attention(q[0], k, k, q, 4)
    with pytest.raises(TypeError):
        rg.rglru_local_attention([1], k, k, q, 4)

    class Fake(torch.Tensor):  # a host tensor that says it is on the device, so that shapes are reached
        is_cuda = True

    f = lambda *s, dtype=bf: torch.zeros(*s, dtype=dtype).as_subclass(Fake)  # noqa: E731
    q, k = f(2, 5, 4, 64), f(2, 5, 2, 64)
    with pytest.raises(ValueError, match="v: expected"):
        rg.rglru_local_attention(q, k, f(2, 6, 2, 64), q, 4)
    with pytest.raises(ValueError, match="k: expected torch.bfloat16"):
        rg.rglru_local_attention(q, f(2, 5, 2, 64, dtype=torch.float32), k, q, 4)
    with pytest.raises(ValueError, match="one stride apart"):
        rg.rglru_local_attention(f(2, 9, 4, 64)[:, :5], k, k, q, 4)
    with pytest.raises(ValueError, match="contiguous"):
        rg.rglru_local_attention(f(2, 5, 8, 64)[:, :, ::2], k, k, q, 4)
    with pytest.raises(ValueError, match="overlap"):
        rg.rglru_local_attention(f(1, 1, 4, 64).expand(2, 5, 4, 64), k, k, q, 4)
    with pytest.raises(ValueError, match="lens"):
        rg.rglru_local_attention(q, k, k, f(2, 5, 4, 64), 4, lens=f(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="lens: expected torch.int32"):
        rg.rglru_local_attention(q, k, k, f(2, 5, 4, 64), 4, lens=f(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="o: must be contiguous"):
        rg.rglru_local_attention(q, k, k, f(2, 5, 8, 64)[:, :, :4], 4)
    with pytest.raises(ValueError, match="positions"):
        rg.rglru_qk_norm_rope(q, k, f(2, 4, dtype=torch.int32), f(16, dtype=torch.float32), q, k)
    with pytest.raises(ValueError, match="slots: needs"):
        rg.rglru_qk_norm_rope(q, k, f(2, 5, dtype=torch.int32), f(16, dtype=torch.float32), q, k,
                              slots=f(2, 5, dtype=torch.int64))
    with pytest.raises(ValueError, match="need slots"):
        rg.rglru_qk_norm_rope(q, k, f(2, 5, dtype=torch.int32), f(16, dtype=torch.float32), q, k,
                              k_pages=f(2, 4, 2, 64), v_pages=f(2, 4, 2, 64))
    with pytest.raises(ValueError, match="v_pages"):
        rg.rglru_paged_attention(f(3, 4, 64), f(9, 16, 2, 64), f(9, 16, 2, 32), f(3, 4, dtype=torch.int32),
                                 f(3, dtype=torch.int32), f(3, 4, 64), 10)
    with pytest.raises(ValueError, match="block_table"):
        rg.rglru_paged_attention(f(3, 4, 64), f(9, 16, 2, 64), f(9, 16, 2, 64), f(2, 4, dtype=torch.int32),
                                 f(3, dtype=torch.int32), f(3, 4, 64), 10)


def test_binding_refuses_by_argument():
    """Host tensors whose first fault is not their device: each message names its tensor."""
    bf, i32 = torch.bfloat16, torch.int32
    q, k = torch.zeros(2, 5, 4, 64, dtype=bf), torch.zeros(2, 5, 2, 64, dtype=bf)
    pos, freq = torch.zeros(2, 5, dtype=i32), torch.zeros(16)
    with pytest.raises(ValueError, match="q: unsupported dtype torch.float64"):
        rg.rglru_qk_norm_rope(q.double(), k, pos, freq, q, k)
    with pytest.raises(ValueError, match="q: expected .*heads"):
        rg.rglru_qk_norm_rope(q[0, 0], k, pos, freq, q, k)
    with pytest.raises(TypeError, match="k: expected a torch.Tensor"):
        rg.rglru_qk_norm_rope(q, [1], pos, freq, q, k)
    with pytest.raises(TypeError, match="lens: expected a torch.Tensor"):
        rg.rglru_local_attention(q, k, k, q, 4, lens=[1, 2])
    with pytest.raises(ValueError, match=r"q_w: expected shape \(64,\), got \(32,\)"):
        rg.rglru_qk_norm_rope(q, k, pos, freq, q, k, q_w=torch.zeros(32), k_w=torch.zeros(64))
    with pytest.raises(ValueError, match="inv_freq: expected torch.float32"):
        rg.rglru_qk_norm_rope(q, k, pos, freq.double(), q, k)
    with pytest.raises(ValueError, match="slots: expected torch.int64"):
        rg.rglru_qk_norm_rope(q, k, pos, freq, q, k, v=k, k_pages=torch.zeros(2, 4, 2, 64, dtype=bf),
                              v_pages=torch.zeros(2, 4, 2, 64, dtype=bf), slots=pos)
    with pytest.raises(ValueError, match="workspace: must be contiguous"):
        rg.rglru_local_attention_backward(q, k, k, q, torch.zeros(2, 4, 5), q, q, k, k, 4,
                                          workspace=torch.zeros(4, 8)[:, ::2])
    with pytest.raises(ValueError, match="q: expected .*N, Hq, dh"):
        rg.rglru_paged_attention(q, torch.zeros(9, 16, 2, 64, dtype=bf), torch.zeros(9, 16, 2, 64, dtype=bf),
                                 torch.zeros(3, 4, dtype=i32), torch.zeros(3, dtype=i32), q, 10)
    with pytest.raises(TypeError):
        rg.rglru_local_attention(q, k, k, q, "4")
    with pytest.raises(TypeError):
        rg.rglru_local_attention(q, k, k, q, 4, scale="a")
    # a window that no integer of the entry point holds is the widest one; here the device is what is wrong
    with pytest.raises(ValueError, match="device"):
        rg.rglru_local_attention(q, k, k, q, 1 << 70)


def test_attention_grid_limit():
    """65535 sequences of 16384 heads: their blocks of 128 rows have numbers below 2^31 - 1 up to 256 tokens (the call
    then ends at its missing output), and are refused beyond, with nothing launched."""
    wide = dict(B=65535, Hq=16384, Hkv=1, dh=64, q_stride=1 << 20, k_stride=64, v_stride=64)
    assert attn(T=256, o=None, **wide) == BAD
    assert attn(T=257, **wide) == UNSUP
    assert attn_bwd(T=256, lse=None, dq_stride=1 << 20, dk_stride=64, dv_stride=64, **wide) == BAD
    assert attn_bwd(T=257, dq_stride=1 << 20, dk_stride=64, dv_stride=64, **wide) == UNSUP
    assert rg.rglru_local_attention_backward_workspace_size(65535, 257, 16384, 1, 64, 16) == 0
    assert rg.rglru_local_attention_backward_workspace_size(65535, 256, 16384, 1, 64, 16) > 0


def test_attention_range():
    """k and v of a sequence may span up to 2^31 bytes: 233016 tokens of a projection of 16 + 2 heads of 256 (the
    calls below then end at their missing output)."""
    packed = dict(B=1, Hq=16, Hkv=1, dh=256, q_stride=4608, k_stride=4608, v_stride=4608)
    grads = dict(dq_stride=4608, dk_stride=4608, dv_stride=4608)
    for T, status in ((120000, BAD), (233016, BAD), (233017, UNSUP)):
        assert attn(T=T, o=None, **packed) == status
        assert attn_bwd(T=T, lse=None, **packed, **grads) == status
    assert attn(T=1 << 13, o=None, **dict(packed, v_stride=1 << 17)) == UNSUP


def test_workspace_size_follows_a_window_that_changes():
    """A window given as a tensor is read anew: the size is that of its value now."""
    window = torch.tensor(64)
    args = (4, 8, 2, 128, 32, 4096)
    few = rg.rglru_paged_attention_workspace_size(*args, window, 0, "bf16")
    window.fill_(1 << 20)
    many = rg.rglru_paged_attention_workspace_size(*args, window, 0, "bf16")
    assert few < many == rg.rglru_paged_attention_workspace_size(*args, 1 << 20, 0, "bf16")
