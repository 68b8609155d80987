"""The serving oracle pinned by other means: e4m3 by torch's conversion and by hand, the prefix by attention over whole
sequences, linear attention by its closed form."""
import numpy as np
import pytest
import torch

from oracle import attention_block as ab
from oracle import serving as sv


def test_e4m3_by_torch():
    rng = np.random.default_rng(0)
    y = np.concatenate([rng.uniform(-448, 448, 4000), rng.standard_normal(4000) * 2.0 ** -7, sv.E4M3, -sv.E4M3,
                        (sv.E4M3[1:] + sv.E4M3[:-1]) / 2]).astype(np.float32)
    got = torch.from_numpy(y).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(sv.codes(y), got)
    assert sv.E4M3[-1] == 448 and sv.E4M3[1] == 2.0 ** -9


def test_scales_by_hand():
    x = np.zeros((8, 4))
    x[:, 1] = [0, 448, 449, 224, 225, -1, 1e-40, 448 * 2.0 ** -117]
    assert sv.scale_exponent(x).tolist() == [-117, 0, 1, -1, 0, -8, -117, -117]
    c, b = sv.quantize(x)
    assert np.array_equal(sv.values(c, b)[1], x[1]) and b[1] == 127
    x[3, 0] = np.inf
    x[4, 0] = np.nan
    c, b = sv.quantize(x)
    assert b[3] == b[4] == 255 and np.isnan(sv.values(c, b)[3]).all()


def test_error_of_a_row():
    """At most half a step, 2^-4 of the value, or half the smallest step of the row's scale."""
    x = np.random.default_rng(1).standard_normal((200, 64)) * np.exp2(np.arange(200) - 100)[:, None]
    c, b = sv.quantize(x)
    s = np.exp2(b.astype(float) - 127)[:, None]
    assert (np.abs(sv.values(c, b) - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * s)).all()


@pytest.mark.parametrize("W,S", [(1 << 30, 0), (9, 0), (9, 4), (25, 30)])
def test_prefix_by_whole_sequences(W, S):
    rng = np.random.default_rng(2)
    P, lens, Hq, Hkv, dh, page = 21, [0, 1, 7, 20], 4, 2, 8, 5
    kp, vp = (rng.standard_normal((40, page, Hkv, dh)) for _ in range(2))
    pages = rng.permutation(40)
    pt, table = pages[:5], pages[5:5 + 16].reshape(4, 4)
    q = rng.standard_normal((4, Hq, dh))
    o, _, _ = sv.prefix_attention(q, kp, vp, pt, P, table, lens, W, S)
    for n, own in enumerate(lens):
        L = P + own
        at = [(pt[u // page], u % page) if u < P else (table[n][(u - P) // page], (u - P) % page) for u in range(L)]
        k, v = (np.stack([x[i, j] for i, j in at])[None] for x in (kp, vp))
        qs = np.zeros((1, L, Hq, dh))
        qs[0, -1] = q[n]
        want, _ = ab.attention(qs, k, v, W, S)
        assert np.allclose(o[n], want[0, -1], rtol=1e-12, atol=1e-14)


def test_linear_by_its_closed_form():
    rng = np.random.default_rng(3)
    B, T, Hk, H, dk, dv = 2, 9, 2, 4, 3, 5
    q, k, v = (rng.standard_normal((B, T, h, d)) for h, d in ((Hk, dk), (Hk, dk), (H, dv)))
    g, s0 = -rng.uniform(0, 2, (B, T, H)), rng.standard_normal((B, H, dk, dv))
    g[0, 4, 1] = -np.inf
    o, s, _, _ = sv.linear_attention(q, k, v, g, s0)
    for b in range(B):
        for h in range(H):
            for t in range(T):
                keep = lambda a: np.exp(np.maximum(g[b, a:t + 1, h], sv.LEAST).sum())  # noqa: E731
                st = keep(0) * s0[b, h] + sum(keep(i + 1) * np.outer(k[b, i, h // 2], v[b, i, h]) for i in range(t + 1))
                assert np.allclose(o[b, t, h], q[b, t, h // 2] @ st / np.sqrt(dk), rtol=1e-12, atol=1e-13)
            assert np.allclose(s[b, h], st, rtol=1e-12, atol=1e-13)
    # a sequence that ends early keeps the state it ended with
    o2, s2, _, _ = sv.linear_attention(q, k, v, g, s0, lens=[4, 0])
    assert np.array_equal(o2[0, :4], o[0, :4]) and not o2[0, 4:].any() and np.array_equal(s2[1], s0[1])
    assert np.array_equal(s2[0], sv.linear_attention(q[:1, :4], k[:1, :4], v[:1, :4], g[:1, :4], s0[:1])[1][0])
