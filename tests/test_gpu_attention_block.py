"""GPU parity of the local attention block's operators through the C ABI against their fp64 oracle
(oracle/attention_block.py): per-head norms with rotation, attention with sinks, the gradients of both,
attention over a paged cache, and runs of them together.

Bounds are elementwise and derived, not fitted. u is the output type's largest relative rounding
(2^-8 bf16, 2^-24 fp32), w = 2^-24 an fp32 operation's. Attention: oracle.attention_bounds. Rotation:
the norm's sum of dh squares is off by dh w at most, half of that in its root, and 8 w for the root,
quotient and products: rn = (dh / 2 + 8) w. Sine and cosine are off by es = 16 w in fp32 (the angle, a
fraction of a turn in fp32, by 2 w; its fp64 product at positions near 2^31 by 8 w; the library's
sincospi by 2 w) and by less than 2^-16 in bf16 (the hardware's sine, about 2^-20). So y is off by
(rn + 4 w + es) (|n_i| + |n_j|), then u |y|."""
import numpy as np
import pytest
import torch

import gated_linear_recurrence_conv1d_amd as rg
from oracle import attention_block as ab

pytestmark = pytest.mark.gpu

DEV = "cuda"
W24 = 2.0 ** -24
U = {torch.bfloat16: 2.0 ** -8, torch.float32: W24}
BF, F32 = torch.bfloat16, torch.float32


def normal(rng, *shape, dtype=BF):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(DEV, dtype)


def num(t):
    return t.detach().double().cpu().numpy()


def check(got, ref, bound, name):
    got = num(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == ref.shape, name
    inf = ~np.isfinite(ref)
    assert np.array_equal(got[inf], ref[inf]), name
    off = np.abs(got[~inf] - ref[~inf])
    lim = np.broadcast_to(bound, ref.shape)[~inf] + 1e-30
    worst = float((off / lim).max()) if off.size else 0.0
    print(f"{name}: at most {worst:.2f} of the bound", flush=True)
    assert worst <= 1.0, name


# ------------------------------------------------------------------------------- norms and rotation
def pair_sum(a, rot):
    """|a_i| + |a_j| of each rotated pair, |a_i| elsewhere."""
    a = np.abs(a)
    s = a[..., :rot // 2] + a[..., rot // 2:rot]
    return np.concatenate([s, s, a[..., rot:]], -1)


def es_of(dtype):
    return 16 * W24 if dtype == F32 else 2.0 ** -16


def rope_bound(y, x, w, dh, rot, eps, dtype):
    n = num(x)
    if w is not None:
        n = n / np.sqrt(np.mean(n * n, -1, keepdims=True) + eps) * num(w)
    rn = (dh / 2 + 8) * W24
    return (1 + 2.0 ** -7) * (rn + 4 * W24 + es_of(dtype)) * pair_sum(n, rot) + U[dtype] * np.abs(y)


def rope_inputs(dtype, lead, Hq, Hkv, dh, rot, norm, seed, packed=True, shift=0, far=0):
    rng = np.random.default_rng(seed)
    H = Hq + 2 * Hkv
    rows = int(np.prod(lead))
    if packed:  # parts of one projection's output, `shift` elements into an allocation
        flat = normal(rng, rows * H * dh + shift, dtype=dtype)[shift:].view(*lead, H, dh)
        q, k, v = flat[..., :Hq, :], flat[..., Hq:Hq + Hkv, :], flat[..., Hq + Hkv:, :]
    else:
        q, k, v = (normal(rng, *lead, h, dh, dtype=dtype) for h in (Hq, Hkv, Hkv))
    pos = torch.from_numpy(rng.integers(far - 1000 if far else 0, (far or 5000) + 1, lead)).to(DEV, torch.int32)
    freq = torch.from_numpy((10000.0 ** (-np.arange(0, rot, 2) / max(rot, 1))).astype(np.float32)).to(DEV)
    qw = 1 + 0.2 * normal(rng, dh, dtype=F32) if norm else None
    kw = 1 + 0.2 * normal(rng, dh, dtype=F32) if norm else None
    return rng, q, k, v, pos, freq, qw, kw


ROPE = [
    # dtype, lead, Hq, Hkv, dh, rot, norm, packed, shift, far
    (BF, (2, 33), 10, 1, 256, 128, True, True, 0, 0),
    (BF, (1, 1), 1, 1, 64, 64, True, False, 0, 0),
    (BF, (3, 65), 5, 2, 128, 96, False, True, 0, 0),
    (BF, (7,), 16, 4, 64, 16, True, True, 0, (1 << 31) - 1),
    (BF, (1500, 3), 3, 1, 64, 32, True, True, 0, 0),       # a wave takes whole rows
    (BF, (2, 33), 3, 1, 128, 24, True, True, 0, 0),        # rot / 2 not whole chunks
    (BF, (2, 33), 3, 1, 128, 64, True, True, 1, 0),        # odd alignment
    (BF, (9,), 3, 2, 80, 40, True, True, 0, 0),            # other head sizes
    (BF, (9,), 3, 1, 2, 2, True, False, 0, 0),
    (BF, (5,), 2, 1, 512, 512, True, True, 0, 0),
    (BF, (5,), 2, 1, 128, 0, True, True, 0, 0),            # no rotation
    (F32, (2, 33), 10, 1, 256, 256, True, True, 0, 1 << 30),
    (F32, (3, 41), 6, 3, 128, 64, True, True, 0, 0),
    (F32, (4, 1), 1, 1, 64, 8, False, False, 0, 0),
    (F32, (11,), 5, 5, 64, 62, True, True, 0, 0),
    (F32, (11,), 3, 2, 34, 10, True, True, 1, -(1 << 31) + 1000),
]


@pytest.mark.parametrize("dtype,lead,Hq,Hkv,dh,rot,norm,packed,shift,far", ROPE)
def test_norm_rope(dtype, lead, Hq, Hkv, dh, rot, norm, packed, shift, far):
    rng, q, k, v, pos, freq, qw, kw = rope_inputs(dtype, lead, Hq, Hkv, dh, rot, norm, dh + rot,
                                                  packed, shift, far)
    q0, k0 = num(q), num(k)
    qo, ko = rg.qk_norm_rope(q, k, pos, freq if rot else None, qw, kw, eps=1e-6)
    assert np.array_equal(num(q), q0) and np.array_equal(num(k), k0)
    for got, x, w, name in ((qo, q, qw, "q"), (ko, k, kw, "k")):
        ref = ab.norm_rope(num(x), None if w is None else num(w), num(pos), num(freq), 1e-6)
        check(got, ref, rope_bound(ref, x, w, dh, rot, 1e-6, dtype), name)
    # in place
    rg.qk_norm_rope(q, k, pos, freq if rot else None, qw, kw, eps=1e-6, q_out=q, k_out=k)
    assert torch.equal(q, qo) and torch.equal(k, ko)


@pytest.mark.parametrize("dtype,lead,Hq,Hkv,dh,rot,norm,packed,shift,far", ROPE)
def test_norm_rope_backward(dtype, lead, Hq, Hkv, dh, rot, norm, packed, shift, far):
    rng, q, k, v, pos, freq, qw, kw = rope_inputs(dtype, lead, Hq, Hkv, dh, rot, norm, dh + rot + 1,
                                                  packed, shift, far)
    dqo, dko = normal(rng, *q.shape, dtype=dtype), normal(rng, *k.shape, dtype=dtype)
    args = (q, k, pos, freq if rot else None, dqo, dko, qw, kw)
    got = rg.qk_norm_rope_backward(*args, eps=1e-6)
    again = rg.qk_norm_rope_backward(*args, eps=1e-6)
    rows = int(np.prod(lead))
    rn, es = (dh / 2 + 8) * W24, es_of(dtype)
    for x, dy, w, H, name in ((q, dqo, qw, Hq, "q"), (k, dko, kw, Hkv, "k")):
        wn = None if w is None else num(w)
        dx, dw = ab.norm_rope_backward(num(x), wn, num(pos), num(freq), 1e-6, num(dy))
        eg = (1 + 2.0 ** -7) * (4 * W24 + es) * pair_sum(num(dy), rot)
        if w is None:
            check(got["d" + name], dx, eg + U[dtype] * np.abs(dx), "d" + name)
            assert got["d" + name + "_w"] is None
        else:
            # t = g w; m = mean(t xh); dx = r (t - xh m): their errors one after the other
            g = ab.rotate(num(dy), num(pos), num(freq), -1.0)
            r = 1 / np.sqrt(np.mean(num(x) ** 2, -1, keepdims=True) + 1e-6)
            xh, t = num(x) * r, g * wn
            et = eg * np.abs(wn) + 2 * W24 * np.abs(t)
            em = np.mean(et * np.abs(xh) + ((dh + 2) * W24 + 2 * rn) * np.abs(t * xh), -1, keepdims=True)
            m = np.abs(np.mean(t * xh, -1, keepdims=True))
            ex = r * (et + np.abs(xh) * em + 2 * rn * np.abs(xh) * m + 4 * W24 * (np.abs(t) + np.abs(xh) * m))
            check(got["d" + name], dx, (1 + 2.0 ** -7) * (ex + 2 * rn * np.abs(dx)) + U[dtype] * np.abs(dx),
                  "d" + name)
            ew = (eg * np.abs(xh) + (rn + (rows * H + 2) * W24) * np.abs(g * xh)).reshape(-1, dh).sum(0)
            check(got["d" + name + "_w"], dw, (1 + 2.0 ** -7) * ew, "d" + name + "_w")
            assert torch.equal(got["d" + name + "_w"], again["d" + name + "_w"])
        assert torch.equal(got["d" + name], again["d" + name])


@pytest.mark.parametrize("dtype,dh", [(BF, 256), (BF, 64), (F32, 128)])
def test_norm_rope_backward_keeps_heads_apart(dtype, dh):
    """Heads of q and of k share a wave: what is not finite in one kind stays out of the other's gradients, which
    are the same to the bit."""
    rng = np.random.default_rng(31)
    q, k = normal(rng, 40, 3, dh, dtype=dtype), normal(rng, 40, 2, dh, dtype=dtype)
    gq, gk = normal(rng, 40, 3, dh, dtype=dtype), normal(rng, 40, 2, dh, dtype=dtype)
    pos, freq = torch.arange(40, device=DEV, dtype=torch.int32), torch.rand(dh // 4, device=DEV)
    w = torch.rand(dh, device=DEV)
    want = rg.qk_norm_rope_backward(q, k, pos, freq, gq, gk, w, w)
    for bad in (float("nan"), float("inf")):
        for mine, grads, other, o_w, hit, h_w in ((k, gk, "dq", "dq_w", "dk", "dk_w"), (q, gq, "dk", "dk_w", "dq", "dq_w")):
            for x in (mine, grads):
                keep = x[5].clone()
                x[5, 1] = bad
                got = rg.qk_norm_rope_backward(q, k, pos, freq, gq, gk, w, w)
                x[5] = keep
                assert torch.equal(got[other], want[other]) and torch.equal(got[o_w], want[o_w])
                assert not torch.isfinite(got[h_w]).all() and not torch.isfinite(got[hit][5, 1].float()).all()
                rest = torch.ones(40, dtype=torch.bool, device=DEV)
                rest[5] = False
                assert torch.equal(got[hit][rest], want[hit][rest])


def test_norm_rope_backward_against_differences():
    """fp32 gradients against fp64 central differences of the oracle's forward, step 1e-4: off by the
    third derivative's h^2 / 6 (below 1e-6 of the gradient's norm) and the kernel's own bound, 1e-5 of
    it altogether."""
    rng, q, k, v, pos, freq, qw, kw = rope_inputs(F32, (2, 9), 3, 1, 64, 32, True, 5)
    dqo, dko = normal(rng, *q.shape, dtype=F32), normal(rng, *k.shape, dtype=F32)
    got = rg.qk_norm_rope_backward(q, k, pos, freq, dqo, dko, qw, kw)
    for x, w, dy, name in ((q, qw, dqo, "q"), (k, kw, dko, "k")):
        sx, sw = rng.standard_normal(x.shape), rng.standard_normal(w.shape)
        f = lambda a, b: np.sum(ab.norm_rope(a, b, num(pos), num(freq), 1e-6) * num(dy))  # noqa: E731
        h = 1e-4
        for diff, g, s in (
                ((f(num(x) + h * sx, num(w)) - f(num(x) - h * sx, num(w))) / (2 * h), got["d" + name], sx),
                ((f(num(x), num(w) + h * sw) - f(num(x), num(w) - h * sw)) / (2 * h), got["d" + name + "_w"], sw)):
            norm = np.linalg.norm(num(g)) * np.linalg.norm(s)
            assert abs(diff - np.sum(num(g) * s)) < 1e-5 * norm, name


@pytest.mark.parametrize("dtype,dh,rot,Hkv,shift", [(BF, 128, 64, 2, 0), (F32, 64, 64, 1, 0), (BF, 80, 80, 3, 0),
                                                    (BF, 256, 128, 1, 3)])
def test_norm_rope_into_the_cache(dtype, dh, rot, Hkv, shift):
    rng, q, k, v, pos, freq, qw, kw = rope_inputs(dtype, (2, 19), 4, Hkv, dh, rot, True, 7, True, shift)
    pages, page = 7, 16
    kp, vp = (normal(rng, pages, page, Hkv, dh, dtype=dtype) for _ in range(2))
    kp0, vp0 = kp.clone(), vp.clone()
    slots = torch.from_numpy(rng.permutation(pages * page)[:38].reshape(2, 19)).to(DEV)
    slots[0, 3], slots[1, 4], slots[1, 18] = -1, pages * page, (1 << 40) + 5  # written nowhere
    qo, ko = rg.qk_norm_rope(q, k, pos, freq, qw, kw, v=v, k_pages=kp, v_pages=vp, slots=slots)
    plain = rg.qk_norm_rope(q, k, pos, freq, qw, kw)
    assert torch.equal(qo, plain[0]) and torch.equal(ko, plain[1])
    ok = (slots >= 0) & (slots < pages * page)
    kp0.view(-1, Hkv, dh)[slots[ok]] = ko[ok]
    vp0.view(-1, Hkv, dh)[slots[ok]] = v[ok]
    assert torch.equal(kp, kp0) and torch.equal(vp, vp0)
    # keys to the cache alone
    kp.zero_()
    rg.rglru_qk_norm_rope(q, k, pos, freq, qo, None, qw, kw, 1e-6, v, kp, vp, slots)
    assert torch.equal(kp.view(-1, Hkv, dh)[slots[ok]], ko[ok])


# ---------------------------------------------------------------------------------------- attention
def packed_qkv(rng, B, T, Hq, Hkv, dh, pad=0):
    x = normal(rng, B, T, (Hq + 2 * Hkv) * dh + pad)
    q = x[..., :Hq * dh].unflatten(-1, (Hq, dh))
    k = x[..., Hq * dh:(Hq + Hkv) * dh].unflatten(-1, (Hkv, dh))
    return q, k, x[..., (Hq + Hkv) * dh:(Hq + 2 * Hkv) * dh].unflatten(-1, (Hkv, dh))


ATTN = [
    # B, T, Hq, Hkv, dh, window, sinks, lens, scale
    (2, 300, 3, 1, 256, 1024, 0, None, 0.0),
    (2, 300, 4, 2, 256, 100, 4, None, 0.0),
    (1, 513, 4, 1, 128, 64, 1, None, 0.0),
    (2, 200, 4, 4, 64, 37, 5, [200, 131], 0.0),
    (3, 1, 2, 2, 64, 5, 0, [1, 0, 1], 0.0),
    (2, 2, 2, 1, 128, 1, 1, None, 0.0),
    (1, 129, 6, 2, 128, 1, 0, None, 0.0),            # every row sees itself alone
    (2, 257, 2, 1, 64, 3, 64, [257, 128], 0.0),      # sinks: exactly one block
    (1, 400, 2, 1, 64, 20, 65, None, 0.0),           # sinks one past a block
    (1, 400, 2, 1, 128, 70, 130, None, 0.0),         # sinks over several blocks
    (2, 130, 2, 1, 256, 10, 999, None, 0.0),         # sinks beyond the sequence: causal
    (4, 70, 5, 1, 128, 1 << 30, 0, [70, 64, 1, 0], 1.0),
    (4, 70, 3, 3, 64, 33, 2, [-5, 1000, 33, 32], 0.05),  # lengths are taken into [0, T]
    (1, 1100, 2, 1, 256, 1024, 4, None, 0.0),
]


@pytest.mark.parametrize("B,T,Hq,Hkv,dh,W,S,lens,scale", ATTN)
def test_attention(B, T, Hq, Hkv, dh, W, S, lens, scale):
    rng = np.random.default_rng(T + W + S)
    q, k, v = packed_qkv(rng, B, T, Hq, Hkv, dh, 8)
    dev_lens = None if lens is None else torch.tensor(lens, dtype=torch.int32, device=DEV)
    if lens is not None:  # what lies past the lengths does not matter
        for b, n in enumerate(lens):
            q[b, max(n, 0):] = float("nan")
            k[b, max(n, 0):] = float("nan")
            v[b, max(n, 0):] = float("inf")
    o, lse = rg.local_attention(q, k, v, W, S, lens=dev_lens, scale=scale, want_lse=True)
    assert torch.equal(o, rg.local_attention(q, k, v, W, S, lens=dev_lens, scale=scale))
    qn, kn, vn = (np.where(np.isfinite(num(x)), num(x), 0) for x in (q, k, v))
    ro, rl = ab.attention(qn, kn, vn, W, S, lens, scale or None)
    el, eo, _, _, _ = ab.attention_bounds(qn, kn, vn, None, W, S, lens, scale or None)
    check(o, ro, eo, "o")
    check(lse, rl, el, "lse")


@pytest.mark.parametrize("B,T,Hq,Hkv,dh,W,S,lens,scale", ATTN)
def test_attention_backward(B, T, Hq, Hkv, dh, W, S, lens, scale):
    rng = np.random.default_rng(T + W + S + 1)
    q, k, v = packed_qkv(rng, B, T, Hq, Hkv, dh)
    do = normal(rng, B, T, Hq, dh)
    dev_lens = None if lens is None else torch.tensor(lens, dtype=torch.int32, device=DEV)
    if lens is not None:
        for b, n in enumerate(lens):
            for x in (q, k, v, do):
                x[b, max(n, 0):] = float("nan")
    o, lse = rg.local_attention(q, k, v, W, S, lens=dev_lens, scale=scale, want_lse=True)
    packed = torch.full((B, T, (Hq + 2 * Hkv) * dh), 7.0, dtype=BF, device=DEV)
    dq = packed[..., :Hq * dh].unflatten(-1, (Hq, dh))
    dk = packed[..., Hq * dh:(Hq + Hkv) * dh].unflatten(-1, (Hkv, dh))
    dv = packed[..., (Hq + Hkv) * dh:].unflatten(-1, (Hkv, dh))
    n = rg.rglru_local_attention_backward_workspace_size(B, T, Hq, Hkv, dh, W, S)
    ws = torch.full((n,), 255, dtype=torch.uint8, device=DEV)  # NaN everywhere
    rg.local_attention_backward(q, k, v, o, lse, do, W, S, dev_lens, scale, dq, dk, dv, ws)
    again = rg.local_attention_backward(q, k, v, o, lse, do, W, S, dev_lens, scale)
    qn, kn, vn, gn = (np.where(np.isfinite(num(x)), num(x), 0) for x in (q, k, v, do))
    refs = ab.attention_backward(qn, kn, vn, gn, W, S, lens, scale or None)
    _, _, eq, ek, ev = ab.attention_bounds(qn, kn, vn, gn, W, S, lens, scale or None)
    for got, ref, e, name in ((dq, refs[0], eq, "dq"), (dk, refs[1], ek, "dk"), (dv, refs[2], ev, "dv")):
        check(got, ref, e, name)
        assert torch.equal(got, again[name]), name
    if W == 1 and S == 0:  # a softmax of one term has no gradient
        assert not dq.any() and not dk.any()


MANY = [  # more workgroups than CUs, and more key blocks in all than 64 and than 64 * 64
    (22, 260, 4, 2, 64, 100, 3, [260 - 11 * (i % 24) for i in range(22)], 0.0),
    (30, 140, 5, 1, 128, 90, 0, None, 0.0),
    (26, 270, 4, 1, 256, 200, 5, [270 if i % 3 else 17 * i % 271 for i in range(26)], 0.0),
    (6, 700, 8, 2, 64, 300, 3, [700, 0, 333, 700, 64, 1], 0.0),
    (4200, 20, 1, 1, 64, 7, 0, None, 0.0),
]


@pytest.mark.parametrize("B,T,Hq,Hkv,dh,W,S,lens,scale", MANY)
def test_attention_of_many(B, T, Hq, Hkv, dh, W, S, lens, scale):
    test_attention(B, T, Hq, Hkv, dh, W, S, lens, scale)
    test_attention_backward(B, T, Hq, Hkv, dh, W, S, lens, scale)


def test_attention_backward_against_differences():
    """The directional derivative along random steps, from fp64 central differences of the oracle's
    forward: within the gradients' own bound, summed along the step (plus 1e-6 for the differences)."""
    rng = np.random.default_rng(11)
    q, k, v = packed_qkv(rng, 1, 90, 4, 2, 64)
    do = normal(rng, 1, 90, 4, 64)
    o, lse = rg.local_attention(q, k, v, 17, 3, want_lse=True)
    got = rg.local_attention_backward(q, k, v, o, lse, do, 17, 3)
    args = [num(x) for x in (q, k, v)]
    bounds = ab.attention_bounds(*args, num(do), 17, 3)[2:]
    for i, (name, e) in enumerate(zip(("dq", "dk", "dv"), bounds)):
        step = rng.standard_normal(args[i].shape)
        lo, hi = ([a + (s * 1e-5 * step if j == i else 0) for j, a in enumerate(args)] for s in (-1, 1))
        diff = (np.sum(ab.attention(*hi, 17, 3)[0] * num(do)) - np.sum(ab.attention(*lo, 17, 3)[0] * num(do))) / 2e-5
        assert abs(diff - np.sum(num(got[name]) * step)) < np.sum(e * np.abs(step)) + 1e-6, name


def test_sinkless_single_head_is_local_mqa():
    """One key/value head and no sinks: the multi-query kernel computes the same, each within the bound."""
    rng = np.random.default_rng(2)
    q, k, v = normal(rng, 2, 300, 4, 128), normal(rng, 2, 300, 1, 128), normal(rng, 2, 300, 1, 128)
    bound = ab.attention_bounds(num(q), num(k), num(v), None, 77)[1]
    check(rg.local_attention(q, k, v, 77), num(rg.local_mqa(q, k[:, :, 0], v[:, :, 0], 77)), 2 * bound, "o")


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_values_out_of_sight_do_not_matter(bad):
    """A value that is not finite reaches the rows that see it and no others."""
    rng = np.random.default_rng(3)
    T, W, S, at = 300, 50, 4, 200
    q, k, v = packed_qkv(rng, 1, T, 2, 1, 128)
    ref = rg.local_attention(q, k, v, W, S)
    v[0, at, 0, 5] = bad
    k2 = k.clone()
    k2[0, at] = float("nan")
    got_v, got_k = rg.local_attention(q, k, v, W, S), rg.local_attention(q, k2, v, W, S)
    sees = torch.zeros(T, dtype=torch.bool, device=DEV)
    sees[at:at + W] = True
    assert torch.isfinite(got_v[0, ~sees].float()).all() and torch.isfinite(got_k[0, ~sees].float()).all()
    assert not torch.isfinite(got_v[0, sees, :, 5].float()).any()
    assert torch.isnan(got_k[0, sees].float()).all()
    # the rows done again are the same up to P's rounding and the sums' order: 2 roundings of o
    bound = ab.attention_bounds(*(np.nan_to_num(num(x), posinf=0, neginf=0) for x in (q, k, v)), None, W, S)[1]
    check(got_v[0, ~sees], num(ref[0, ~sees]), 2 * bound[0, ~sees.cpu().numpy()] + 1e-6, "rows out of sight")


@pytest.mark.parametrize("dh", [64, 256])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_values_out_of_sight_do_not_matter_of_many(bad, dh):
    """The same with more workgroups than CUs, whose waves walk all of their keys: the other sequences and the
    rows before are as they were, to the bit."""
    rng = np.random.default_rng(4)
    B, T, W, S, at = 90, 200, 30, 2, 140
    q, k, v = packed_qkv(rng, B, T, 2, 1, dh)
    ref = rg.local_attention(q, k, v, W, S)
    v[7, at, 0, 5] = bad
    got = rg.local_attention(q, k, v, W, S)
    others = torch.arange(B, device=DEV) != 7
    assert torch.equal(got[others], ref[others]) and torch.equal(got[7, :128], ref[7, :128])
    assert not torch.isfinite(got[7, at:at + W, :, 5].float()).any()
    sees = torch.zeros(T, dtype=torch.bool, device=DEV)
    sees[at:at + W] = True
    bound = ab.attention_bounds(*(np.nan_to_num(num(x[7:8]), posinf=0, neginf=0) for x in (q, k, v)), None, W, S)[1]
    check(got[7, ~sees], num(ref[7, ~sees]), 2 * bound[0, ~sees.cpu().numpy()] + 1e-6, "rows out of sight")


def test_large_scores():
    """Scores down to -1e28 (inputs near the top of bf16's useful range): one key takes all, no NaN, in
    both forms. p of the others is below exp(-1e25) = 0, so o is that key's value, rounded once."""
    T, dh = 140, 64
    q, k, v = (torch.zeros(1, T, 1, dh, dtype=BF, device=DEV) for _ in range(3))
    q[..., 0] = -1e15
    k[0, :, 0, 0] = 1e13 + 1e12 * torch.arange(T, device=DEV)  # the oldest visible key scores highest
    v.copy_(torch.arange(T, device=DEV).view(1, T, 1, 1).expand_as(v))
    o, lse = rg.local_attention(q, k, v, 20, 0, want_lse=True)
    ro, rl = ab.attention(num(q), num(k), num(v), 20, 0)
    assert torch.isfinite(lse).all()
    check(o, ro, 2.0 ** -8 * np.abs(ro), "o")
    table = torch.zeros(1, 1, dtype=torch.int32, device=DEV)
    d = rg.paged_attention(q[:, -1], k, v, table, torch.tensor([T], dtype=torch.int32, device=DEV), 20)
    check(d, ro[:, -1], 2.0 ** -8 * np.abs(ro[:, -1]), "decode")


# -------------------------------------------------------------------------------------- paged cache
def paged_inputs(rng, dtype, lens, Hq, Hkv, dh, page, extra=2, hide=None, W=1 << 30, S=0):
    """A pool with the sequences' pages in random order; table entries nothing may follow are `hide`."""
    N, width = len(lens), max(1, max(-(-n // page) for n in lens) + 1)
    held = [-(-n // page) for n in lens]
    pages = sum(held) + extra
    order = rng.permutation(pages)
    table, at = np.full((N, width), 0 if hide is None else hide, np.int32), 0
    for n, m in enumerate(held):
        table[n, :m] = order[at:at + m]
        if hide is not None:
            for j in range(m):
                u = np.arange(j * page, min((j + 1) * page, lens[n]))
                if not np.any((u >= lens[n] - W) | (u < S)):
                    table[n, j] = hide
        at += m
    q = normal(rng, N, (Hq + 2) * dh, dtype=dtype)[:, dh:(Hq + 1) * dh].unflatten(-1, (Hq, dh))
    kp, vp = (normal(rng, pages, page, Hkv, dh, dtype=dtype) for _ in range(2))
    return q, kp, vp, torch.from_numpy(table).to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV)


def paged_check(got, q, kp, vp, table, lens, W, S, scale=None):
    dtype, dh = q.dtype, q.shape[-1]
    kn, vn = (np.nan_to_num(num(x), nan=0.0, posinf=0.0, neginf=0.0) for x in (kp, vp))
    ref, mag, most = ab.paged_attention(num(q), kn, vn, table.cpu().numpy(), lens.tolist(), W, S, scale)
    n = max(1, int(lens.max()))
    rp = 2 * (dh + 2) * W24 * most + (n + 8) * 2 * W24
    u = U[dtype]
    bound = (rp + (u if dtype == BF else n * W24)) * mag * (1 + 2.0 ** -7) + u * np.abs(ref)
    check(got, ref, bound, "o")


PAGED = [
    # dtype, lens, Hq, Hkv, dh, page, window, sinks
    (BF, [1, 31, 32, 33, 0, 64, 127, 300], 10, 1, 256, 64, 1 << 30, 0),
    (BF, [1, 5, 40, 700], 8, 2, 128, 32, 100, 4),
    (BF, [17, 1, 129], 3, 3, 64, 16, 40, 1),
    (BF, [50, 100, 2], 4, 1, 64, 7, 33, 9),
    (BF, [9, 65], 5, 1, 256, 1, 20, 2),
    (BF, [300], 16, 1, 128, 96, 1, 0),
    (BF, [300, 77], 40, 2, 64, 48, 64, 70),         # more than 16 heads of a group
    (BF, [2500, 3], 2, 1, 256, 128, 1 << 30, 0),    # several chunks
    (BF, [5000], 17, 1, 64, 20, 4999, 40),
    (F32, [1, 15, 16, 17, 0, 200], 10, 1, 256, 16, 1 << 30, 0),
    (F32, [33, 1000, 4], 6, 2, 128, 32, 130, 5),
    (F32, [100, 7], 2, 1, 64, 5, 30, 3),
    (F32, [3000], 20, 1, 64, 64, 1 << 30, 0),
]


@pytest.mark.parametrize("dtype,lens,Hq,Hkv,dh,page,W,S", PAGED)
def test_paged_attention(dtype, lens, Hq, Hkv, dh, page, W, S):
    rng = np.random.default_rng(sum(lens) + dh)
    q, kp, vp, table, dl = paged_inputs(rng, dtype, lens, Hq, Hkv, dh, page, hide=-7, W=W, S=S)
    got = rg.paged_attention(q, kp, vp, table, dl, W, S)
    paged_check(got, q, kp, vp, table, dl, W, S)
    n = rg.rglru_paged_attention_workspace_size(len(lens), Hq, Hkv, dh, page, table.shape[1], W, S, dtype)
    ws = torch.full((max(n, 16),), 255, dtype=torch.uint8, device=DEV)
    assert torch.equal(got, rg.paged_attention(q, kp, vp, table, dl, W, S, workspace=ws))


@pytest.mark.parametrize("dtype,page", [(BF, 32), (BF, 24), (F32, 16), (F32, 10)])
def test_paged_rows_out_of_sight_do_not_matter(dtype, page):
    rng = np.random.default_rng(page)
    lens, W, S = [70, 5, 41], 19, 3
    q, kp, vp, table, dl = paged_inputs(rng, dtype, lens, 4, 2, 64, page, hide=1 << 30, W=W, S=S)
    want = rg.paged_attention(q, kp, vp, table, dl, W, S)
    seen = torch.zeros(kp.shape[:2], dtype=torch.bool, device=DEV)
    for n, ln in enumerate(lens):
        for u in range(ln):
            if u >= ln - W or u < S:
                seen[table[n, u // page].long(), u % page] = True
    kp[~seen], vp[~seen] = float("nan"), float("inf")
    got = rg.paged_attention(q, kp, vp, table, dl, W, S)
    assert torch.equal(got, want)
    paged_check(got, q, kp, vp, table, dl, W, S)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("page,long", [(32, 60), (20, 60), (32, 2000), (20, 2000)])
def test_paged_rows_that_cannot_be_followed_are_nan(dtype, page, long):
    rng = np.random.default_rng(page + long)
    lens = [long, 50, 33, 45, 12]
    q, kp, vp, table, dl = paged_inputs(rng, dtype, lens, 4, 1, 64, page)
    want = rg.paged_attention(q, kp, vp, table, dl, 1 << 30)
    table[1, 1], table[2, 0] = kp.shape[0], -1
    dl[3], dl[4] = -1, table.shape[1] * page + 1
    got = rg.paged_attention(q, kp, vp, table, dl, 1 << 30)
    assert torch.isnan(got[1:].float()).all()
    assert torch.equal(got[0], want[0])


def test_paged_offsets_beyond_32_bits():
    """A pool of more than 2^32 bytes whose last pages are the ones in use."""
    rng = np.random.default_rng(9)
    page, Hkv, dh = 64, 1, 256
    pages = (1 << 32) // (page * Hkv * dh * 2) + 40
    kp = torch.zeros(pages, page, Hkv, dh, dtype=BF, device=DEV)
    vp = torch.zeros_like(kp)
    kp[-40:], vp[-40:] = normal(rng, 40, page, Hkv, dh), normal(rng, 40, page, Hkv, dh)
    table = torch.arange(pages - 20, pages, device=DEV, dtype=torch.int32).view(2, 10)
    lens = torch.tensor([600, 77], dtype=torch.int32, device=DEV)
    q = normal(rng, 2, 10, dh)
    got = rg.paged_attention(q, kp, vp, table, lens, 1 << 30)
    small = rg.paged_attention(q, kp[-40:].clone(), vp[-40:].clone(), table - (pages - 40), lens, 1 << 30)
    assert torch.equal(got, small)
    paged_check(got, q, kp[-40:], vp[-40:], table - (pages - 40), lens, 1 << 30, 0)
    # and the cache write there
    slots = torch.tensor([pages * page - 1, pages * page - 700], device=DEV)
    k = normal(rng, 2, 1, dh)
    pos, freq = torch.tensor([3, 4], dtype=torch.int32, device=DEV), torch.rand(64, device=DEV)
    _, ko = rg.qk_norm_rope(q, k, pos, freq, v=k, k_pages=kp, v_pages=vp, slots=slots)
    assert torch.equal(kp.view(-1, Hkv, dh)[slots], ko) and torch.equal(vp.view(-1, Hkv, dh)[slots], k)


# ----------------------------------------------------------------------------------------- together
def test_prefill_then_decode_over_the_cache():
    """A prompt through the norms (filling the cache) and attention, then token by token through the
    norms and the paged attention: each step within both forms' bounds of attention over the whole
    sequence, window and sinks included."""
    rng = np.random.default_rng(21)
    B, T, n0, Hq, Hkv, dh, rot, W, S, page = 3, 90, 70, 6, 2, 128, 64, 40, 3, 16
    width = -(-T // page)
    q, k, v = packed_qkv(rng, B, T, Hq, Hkv, dh)
    freq = torch.from_numpy((10000.0 ** (-np.arange(0, rot, 2) / rot)).astype(np.float32)).to(DEV)
    qw, kw = 1 + 0.1 * normal(rng, dh, dtype=F32), 1 + 0.1 * normal(rng, dh, dtype=F32)
    table = torch.from_numpy(rng.permutation(B * width).astype(np.int32)).to(DEV).view(B, width)
    kp, vp = (torch.full((B * width, page, Hkv, dh), float("nan"), dtype=BF, device=DEV) for _ in range(2))
    at = torch.arange(T, device=DEV)
    slots = table.long()[:, at // page] * page + at % page  # [B, T]
    pos = at.to(torch.int32).expand(B, T).contiguous()
    q0, k0, v0, pos0, slots0 = (x[:, :n0].contiguous() for x in (q, k, v, pos, slots))
    qr, kr = rg.qk_norm_rope(q0, k0, pos0, freq, qw, kw, v=v0, k_pages=kp, v_pages=vp, slots=slots0)
    full_q, full_k = rg.qk_norm_rope(q, k, pos, freq, qw, kw)
    assert torch.equal(full_q[:, :n0], qr) and torch.equal(full_k[:, :n0], kr)
    whole = rg.local_attention(full_q, full_k, v, W, S)
    assert torch.equal(whole[:, :n0], rg.local_attention(qr, kr, v0, W, S))
    bound = ab.attention_bounds(num(full_q), num(full_k), num(v), None, W, S)[1]
    for t in range(n0, T):
        qt, _ = rg.qk_norm_rope(q[:, t], k[:, t], pos[:, t].contiguous(), freq, qw, kw, v=v[:, t], k_pages=kp,
                                v_pages=vp, slots=slots[:, t].contiguous())
        o = rg.paged_attention(qt, kp, vp, table, torch.full((B,), t + 1, dtype=torch.int32, device=DEV), W, S)
        off = np.abs(num(o) - num(whole[:, t]))
        assert (off <= 2 * bound[:, t]).all(), t


def test_training_step_of_the_block():
    """norms and rotation -> attention -> their gradients down to the packed projection and the norm
    weights, against the oracle's chain on the kernels' own rounded intermediates: 2-norms within 2^-7
    (four roundings of at most 2^-8 each, in random directions over thousands of values, halve)."""
    rng = np.random.default_rng(22)
    B, T, Hq, Hkv, dh, rot, W, S = 2, 150, 4, 2, 128, 64, 60, 2
    lens = [150, 97]
    dl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    q, k, v = packed_qkv(rng, B, T, Hq, Hkv, dh)
    pos = torch.arange(T, device=DEV, dtype=torch.int32).expand(B, T).contiguous()
    freq = torch.from_numpy((10000.0 ** (-np.arange(0, rot, 2) / rot)).astype(np.float32)).to(DEV)
    qw, kw = 1 + 0.1 * normal(rng, dh, dtype=F32), 1 + 0.1 * normal(rng, dh, dtype=F32)
    do = normal(rng, B, T, Hq, dh)
    qr, kr = rg.qk_norm_rope(q, k, pos, freq, qw, kw)
    o, lse = rg.local_attention(qr, kr, v, W, S, lens=dl, want_lse=True)
    packed = torch.empty(B, T, Hq + 2 * Hkv, dh, dtype=BF, device=DEV)
    dq, dk, dv = packed[:, :, :Hq], packed[:, :, Hq:Hq + Hkv], packed[:, :, Hq + Hkv:]
    rg.local_attention_backward(qr, kr, v, o, lse, do, W, S, dl, dq=dq, dk=dk, dv=dv)
    got = rg.qk_norm_rope_backward(q, k, pos, freq, dq, dk, qw, kw, dq=dq, dk=dk)  # in place
    rq, rk, rv = ab.attention_backward(num(qr), num(kr), num(v), num(do), W, S, lens)
    refs = {"dv": (dv, rv)}
    for name, x, w, g, mine in (("q", q, qw, rq, dq), ("k", k, kw, rk, dk)):
        dx, dw = ab.norm_rope_backward(num(x), num(w), num(pos), num(freq), 1e-6, g)
        refs["d" + name], refs["d" + name + "_w"] = (mine, dx), (got["d" + name + "_w"], dw)
    for name, (a, ref) in refs.items():
        rel = np.linalg.norm(num(a) - ref) / np.linalg.norm(ref)
        print(f"{name}: {rel:.2e}", flush=True)
        assert rel < 2.0 ** -7, name
    assert not packed[1, 97:].any()


def test_other_stream_and_graph():
    """A step on a side stream, and the same calls captured into a graph and replayed on changing
    inputs, each replay against the eager result."""
    rng = np.random.default_rng(23)
    N, Hq, Hkv, dh, page, W, S = 5, 4, 1, 128, 32, 500, 4
    lens = [900, 1, 33, 400, 64]
    q, kp, vp, table, dl = paged_inputs(rng, BF, lens, Hq, Hkv, dh, page)
    B, T = 2, 130
    aq, ak, av = packed_qkv(rng, B, T, Hq, Hkv, dh)
    do = normal(rng, B, T, Hq, dh)
    pos, freq = torch.arange(B * T, device=DEV, dtype=torch.int32).view(B, T), torch.rand(32, device=DEV)
    w = torch.rand(dh, device=DEV)

    def step():
        d = rg.paged_attention(q, kp, vp, table, dl, W, S)
        qr, kr = rg.qk_norm_rope(aq, ak, pos, freq, w, w)
        o, lse = rg.local_attention(qr, kr, av, W, S, want_lse=True)
        g = rg.local_attention_backward(qr, kr, av, o, lse, do, W, S)
        r = rg.qk_norm_rope_backward(aq, ak, pos, freq, g["dq"], g["dk"], w, w)
        return [d, o, lse, g["dv"], r["dq"], r["dk"], r["dq_w"], r["dk_w"]]

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    d = rg.paged_attention(q, kp, vp, table, dl, W, S, stream=side)  # given, not current
    o2 = rg.local_attention(aq, ak, av, W, S, stream=side.cuda_stream)
    with torch.cuda.stream(side):
        there = step()
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(d, want[0]) and torch.equal(o2, rg.local_attention(aq, ak, av, W, S))
    assert all(torch.equal(a, b) for a, b in zip(there, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(4):
        for x in (q, aq, ak, do):
            x.mul_(-0.75)
        want = step()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), i


def test_streams_by_number():
    """A stream's number is that stream; 0 is the default stream, whatever stream is current."""
    seen = []

    class Ext:
        @staticmethod
        def local_attention(*args):
            seen.append(args[-1])
            return rg.RGLRU_OK

    q = torch.zeros(1, 3, 1, 64, dtype=BF, device=DEV)
    side, real = torch.cuda.Stream(), rg._ext
    try:
        rg._ext = Ext
        with torch.cuda.stream(side):
            for stream in (None, 0, side.cuda_stream, side, torch.cuda.default_stream()):
                rg.rglru_local_attention(q, q, q, q, 2, stream=stream)
    finally:
        rg._ext = real
    assert seen == [side.cuda_stream, 0, side.cuda_stream, side.cuda_stream, 0]


SHORT = [  # sequences much shorter than T: fewer items of the backward's key side than workgroups
    (1, 2048, 1, 1, 64, 1024, 0, [100], 0.0),
    (1, 2048, 10, 1, 128, 1024, 4, [300], 0.0),
    (4, 2048, 10, 1, 256, 1024, 0, [64] * 4, 0.0),
    (8, 512, 4, 1, 64, 256, 0, [512] + [20] * 7, 0.0),
    (3, 700, 6, 3, 128, 90, 2, [0, 1, 0], 0.0),
    (2, 300, 2, 2, 64, 300, 0, [0, 0], 0.0),
]


@pytest.mark.parametrize("B,T,Hq,Hkv,dh,W,S,lens,scale", SHORT)
def test_attention_backward_of_short_sequences(B, T, Hq, Hkv, dh, W, S, lens, scale):
    test_attention(B, T, Hq, Hkv, dh, W, S, lens, scale)
    test_attention_backward(B, T, Hq, Hkv, dh, W, S, lens, scale)


@pytest.mark.parametrize("B,T,Hq,Hkv,dh,W,S,lens", [
    (1, 1100, 2, 1, 256, 1024, 4, None), (2, 700, 4, 2, 64, 300, 0, [700, 431]), (1, 600, 3, 1, 128, 1 << 30, 0, None),
    (1, 513, 4, 1, 128, 64, 1, None), (4, 2048, 2, 1, 128, 1024, 0, [64] * 4)])
def test_attention_gradients_in_the_norm(B, T, Hq, Hkv, dh, W, S, lens):
    """The gradients' 2-norm, which a factor in all of them cannot hide in: P, dS, o and the result are rounded to
    bf16, at most 2^-8 of the value each and in random directions, so together, over thousands of values, below
    2^-7 of the whole. The rows of dq whose delta comes from o (256 and on, W >= 256) also by themselves."""
    rng = np.random.default_rng(T + W + 5)
    q, k, v = packed_qkv(rng, B, T, Hq, Hkv, dh)
    do = normal(rng, B, T, Hq, dh)
    dev_lens = None if lens is None else torch.tensor(lens, dtype=torch.int32, device=DEV)
    o, lse = rg.local_attention(q, k, v, W, S, lens=dev_lens, want_lse=True)
    got = rg.local_attention_backward(q, k, v, o, lse, do, W, S, dev_lens)
    refs = ab.attention_backward(num(q), num(k), num(v), num(do), W, S, lens)
    pairs = [(name, num(got[name]), ref) for name, ref in zip(("dq", "dk", "dv"), refs)]
    if W >= 256 and T > 256 and (lens is None or max(lens) > 256):
        pairs.append(("dq beyond row 256", pairs[0][1][:, 256:], refs[0][:, 256:]))
    for name, a, ref in pairs:
        rel = np.linalg.norm(a - ref) / np.linalg.norm(ref)
        print(f"{name}: {rel:.2e}", flush=True)
        assert rel < 2.0 ** -7, name


def test_attention_of_more_threads_than_a_dimension_holds():
    """Single tokens of 65535 sequences and 264 heads: 17.3 million workgroups of the forward (256 threads) and of
    dq (512), 277 million of the sum, where one dimension of a launch holds 2^32 threads. A token that sees itself
    alone gives o = v, lse = its score, dv = do and no other gradient, exactly."""
    B, H, dh = 65535, 264, 64
    gen = torch.Generator(device=DEV).manual_seed(1)
    q, k, v, do = (torch.randn(B, 1, H, dh, generator=gen, device=DEV, dtype=BF) for _ in range(4))
    o, lse = rg.local_attention(q, k, v, 5, want_lse=True)
    assert torch.equal(o, v)
    score = torch.stack([(q[b].float() * k[b].float()).sum(-1) / 8 for b in (0, B // 2, B - 1)]).squeeze(1)
    assert torch.allclose(lse[[0, B // 2, B - 1], :, 0], score, rtol=0, atol=(dh + 4) * W24 * 64)
    g = rg.local_attention_backward(q, k, v, o, lse, do, 5)
    assert torch.equal(g["dv"], do)
    assert not g["dq"].any() and not g["dk"].any()


def test_paged_attention_of_more_threads_than_a_dimension_holds():
    """2^24 + 3 sequences of one cached token each: o is its value."""
    N, dh, page = (1 << 24) + 3, 64, 16
    gen = torch.Generator(device=DEV).manual_seed(2)
    q = torch.randn(N, 1, dh, generator=gen, device=DEV, dtype=BF)
    kp, vp = (torch.randn(64, page, 1, dh, generator=gen, device=DEV, dtype=BF) for _ in range(2))
    table = torch.randint(0, 64, (N, 1), generator=gen, device=DEV, dtype=torch.int32)
    got = rg.paged_attention(q, kp, vp, table, torch.ones(N, dtype=torch.int32, device=DEV), 100)
    assert torch.equal(got, vp[:, 0][table[:, 0].long()])


def calls_that_allocate(rng):
    """(name, call taking a stream) for each function that makes its outputs and workspaces, and its inputs."""
    B, T, Hq, Hkv, dh = 2, 300, 4, 2, 128
    q, k, v = packed_qkv(rng, B, T, Hq, Hkv, dh)
    do, w = normal(rng, B, T, Hq, dh), 1 + 0.1 * normal(rng, dh, dtype=F32)
    pos, freq = torch.arange(B * T, device=DEV, dtype=torch.int32).view(B, T), torch.rand(32, device=DEV)
    o, lse = rg.local_attention(q, k, v, 70, 3, want_lse=True)
    pq, kp, vp, table, dl = paged_inputs(rng, BF, [900, 1, 33], Hq, Hkv, dh, 16)
    return [
        ("norm_rope", lambda s: rg.qk_norm_rope(q, k, pos, freq, w, w, stream=s)),
        ("norm_rope_backward", lambda s: rg.qk_norm_rope_backward(q, k, pos, freq, do, k, w, w, stream=s)),
        ("attention", lambda s: rg.local_attention(q, k, v, 70, 3, want_lse=True, stream=s)),
        ("attention_backward", lambda s: rg.local_attention_backward(q, k, v, o, lse, do, 70, 3, stream=s)),
        ("paged_attention", lambda s: rg.paged_attention(pq, kp, vp, table, dl, 1 << 30, stream=s)),
    ]


def tensors(out):
    return list(out.values()) if isinstance(out, dict) else list(out) if isinstance(out, tuple) else [out]


def test_given_stream_owns_what_is_made_for_it(monkeypatch):
    """Outputs and workspaces come from the given stream's pool."""
    calls = calls_that_allocate(np.random.default_rng(41))
    side, real = torch.cuda.Stream(), rg._call
    side.wait_stream(torch.cuda.current_stream())

    def pool_of(t):
        at = t.data_ptr()
        return [s["stream"] for s in torch.cuda.memory_snapshot() if s["address"] <= at < s["address"] + s["total_size"]]

    for name, call in calls:
        want, made = tensors(call(None)), []

        def spy(where, fn, q, stream, *args):
            at = [(a, pool_of(a)) for a in args if isinstance(a, torch.Tensor)]
            made.extend(p for _, p in at if p == [side.cuda_stream])
            return real(where, fn, q, stream, *args)

        monkeypatch.setattr(rg, "_call", spy)
        for given in (side, side.cuda_stream):
            made.clear()
            got = tensors(call(given))
            torch.cuda.synchronize()
            assert all(pool_of(t) == [side.cuda_stream] for t in got), name
            assert len(made) == len(got) + (name in ("norm_rope_backward", "attention_backward", "paged_attention")), name
            assert all(torch.equal(a, b) for a, b in zip(got, want)), name
        monkeypatch.setattr(rg, "_call", real)


def test_given_stream_beside_a_busy_one():
    """The current stream still has to fill memory that it has given back; what a call on another stream makes lies
    elsewhere, and what it made is not reused before the current stream has read it."""
    side = torch.cuda.Stream()
    for name, call in calls_that_allocate(np.random.default_rng(42)):
        want = [t.clone() for t in tensors(call(None))]
        sizes = [(t.shape, t.dtype) for t in want]
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        old = [torch.empty(s, dtype=d, device=DEV) for s, d in sizes]
        torch.cuda._sleep(20_000_000)
        for t in old:
            t.fill_(float("nan"))
        del old, t
        got = tensors(call(side))
        side.synchronize()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), name
        # read by the current stream, then given back and overwritten on the side stream
        torch.cuda._sleep(20_000_000)
        kept = [t.clone() for t in got]
        del got
        with torch.cuda.stream(side):
            new = [torch.full(s, float("nan"), dtype=d, device=DEV) for s, d in sizes]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(kept, want)), name
        del new


@pytest.mark.parametrize("dtype,lens,Hq,Hkv,dh,page,W,S", [c for c in PAGED if c[0] == BF] + [
    (BF, list(range(1, 65)), 10, 1, 256, 16, 1 << 30, 0), (BF, list(range(1, 65)), 4, 2, 64, 5, 1 << 30, 0),
    (BF, [40000, 9000], 8, 2, 128, 32, 1 << 30, 0), (BF, [200, 3000], 17, 1, 256, 7, 1 << 30, 0)])
def test_paged_attention_holds_probabilities_in_16_bits(dtype, lens, Hq, Hkv, dh, page, W, S):
    """P enters its product as bf16 hi + lo: hi is off by at most 2^-8 of P, lo by 2^-8 of that. So o is within
    2^-16 of its terms (and the bound's fp32 part) before its own rounding, at one cached token as at many."""
    rng = np.random.default_rng(len(lens) + dh)
    q, kp, vp, table, dl = paged_inputs(rng, dtype, lens, Hq, Hkv, dh, page)
    got = rg.paged_attention(q, kp, vp, table, dl, W, S)
    ref, mag, most = ab.paged_attention(num(q), num(kp), num(vp), table.cpu().numpy(), lens, W, S)
    rp = 2 * (dh + 2) * W24 * most + (max(lens) + 8) * 2 * W24
    check(got, ref, ((rp + 2.0 ** -16) * mag + 2.0 ** -8 * np.abs(ref)) * (1 + 2.0 ** -7), "o")


def test_attention_beyond_a_gibibyte_of_keys():
    """A prompt whose k and v span more than 2^30 bytes of a packed projection, and its gradients: the last rows
    against the oracle on the last 640 tokens. With a window of 64 what rows (keys) from 64 on give there is what
    they give in the whole."""
    rng = np.random.default_rng(51)
    Hq, Hkv, dh, W, tail = 16, 1, 256, 64, 640
    T = 120000
    gen = torch.Generator(device=DEV).manual_seed(51)
    x = torch.randn(1, T, Hq + 2 * Hkv, dh, generator=gen, device=DEV, dtype=BF)
    q, k, v = x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:]
    assert T * x.stride(1) * 2 > 1 << 30
    do = torch.zeros(1, T, Hq, dh, dtype=BF, device=DEV)
    do[:, -tail:] = normal(rng, 1, tail, Hq, dh)
    o, lse = rg.local_attention(q, k, v, W, want_lse=True)
    g = torch.empty_like(x)
    dq, dk, dv = g[:, :, :Hq], g[:, :, Hq:Hq + Hkv], g[:, :, Hq + Hkv:]
    rg.local_attention_backward(q, k, v, o, lse, do, W, dq=dq, dk=dk, dv=dv)
    args = [num(t[:, -tail:]) for t in (q, k, v)]
    gn = num(do[:, -tail:])
    ro, rl = ab.attention(*args, W)
    refs = ab.attention_backward(*args, gn, W)
    el, eo, eq, ek, ev = ab.attention_bounds(*args, gn, W)
    check(lse[:, :, 64 - tail:], rl[:, :, 64:], el[:, :, 64:], "lse")
    for got, ref, e, name in ((o, ro, eo, "o"), (dq, refs[0], eq, "dq"), (dk, refs[1], ek, "dk"), (dv, refs[2], ev, "dv")):
        check(got[:, 64 - tail:], ref[:, 64:], e[:, 64:], name)
    assert not g[:, :T - tail - W].any()  # no gradient came in there


def test_given_stream_in_a_graph():
    """Calls on a stream that joins a capture, their outputs and workspaces in the graph's own memory: every replay
    against the eager result, with eager work of other sizes between them."""
    rng = np.random.default_rng(43)
    calls = calls_that_allocate(rng)
    want = [[t.clone() for t in tensors(call(None))] for _, call in calls]
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        got = [tensors(call(side)) for _, call in calls]
        here.wait_stream(side)
    for i in range(4):
        for out in got:
            for t in out:
                t.fill_(float("nan"))
        other = [torch.full((100_000 * (i + 1),), float("nan"), device=DEV) for _ in range(4)]
        graph.replay()
        torch.cuda.synchronize()
        del other
        for (name, _), out, ref in zip(calls, got, want):
            assert all(torch.equal(a, b) for a, b in zip(out, ref)), (i, name)
