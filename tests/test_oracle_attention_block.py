"""The attention block oracle (oracle/attention_block.py) pinned against independent computations, no
GPU: torch's fp64 autograd for the gradients, central differences, the multi-query oracle, and dense
attention for the paged form. Bound 1e-9: fp64 sums of a few hundred terms; differences 1e-6 (step
1e-5: h^2 of the third derivative and 1e-16 / h)."""
import numpy as np
import pytest
import torch

from oracle import attention_block as ab
from oracle.local_mqa import local_mqa


def torch_norm_rope(x, w, pos, freq, eps):
    if w is not None:
        x = torch.nn.functional.rms_norm(x, x.shape[-1:], w, eps)
    h = len(freq)
    z = torch.view_as_complex(torch.stack([x[..., :h], x[..., h:2 * h]], -1).contiguous())
    z = z * torch.polar(torch.ones(()).double(), pos[..., None, None] * freq)
    return torch.cat([z.real, z.imag, x[..., 2 * h:]], -1)


@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("dh,rot", [(8, 8), (8, 4), (6, 2), (8, 0)])
def test_norm_rope_and_gradient(norm, dh, rot):
    g = torch.Generator().manual_seed(dh + rot)
    x = torch.randn(2, 3, 4, dh, generator=g, dtype=torch.float64, requires_grad=True)
    w = torch.randn(dh, generator=g, dtype=torch.float64, requires_grad=True) if norm else None
    pos = torch.tensor([[0, 5, 100000], [-3, 7, 2]]).double()
    freq = torch.rand(rot // 2, generator=g, dtype=torch.float64)
    y = torch_norm_rope(x, w, pos, freq, 1e-6)
    dy = torch.randn(y.shape, generator=g, dtype=torch.float64)
    y.backward(dy)
    wn = None if w is None else w.detach().numpy()
    args = (wn, pos.numpy(), freq.numpy(), 1e-6)
    assert np.abs(ab.norm_rope(x.detach().numpy(), *args) - y.detach().numpy()).max() < 1e-9
    dx, dw = ab.norm_rope_backward(x.detach().numpy(), *args, dy.numpy())
    assert np.abs(dx - x.grad.numpy()).max() < 1e-9
    if norm:
        assert np.abs(dw - w.grad.numpy()).max() < 1e-9


@pytest.mark.parametrize("W,S,lens", [(4, 0, None), (3, 2, [7, 0]), (1, 0, [7, 3]), (1, 1, None),
                                      (50, 9, [1, 7])])
def test_attention_gradients(W, S, lens):
    rng = np.random.default_rng(W + S)
    B, T, Hq, Hkv, dh = 2, 7, 4, 2, 6
    q, k, v, do = (rng.standard_normal((B, T, h, dh)) for h in (Hq, Hkv, Hkv, Hq))
    leaf = [torch.tensor(x, requires_grad=True) for x in (q, k, v)]
    o = torch.zeros(B, T, Hq, dh, dtype=torch.float64)
    for b in range(B):
        n = T if lens is None else lens[b]
        for h in range(Hq):
            for t in range(n):
                see = [u for u in range(t + 1) if u > t - W or u < S]
                s = leaf[1][b, see, h // 2] @ leaf[0][b, t, h] / np.sqrt(dh)
                o[b, t, h] = torch.softmax(s, 0) @ leaf[2][b, see, h // 2]
    ref, _ = ab.attention(q, k, v, W, S, lens)
    assert np.abs(ref - o.detach().numpy()).max() < 1e-9
    (o * torch.tensor(do)).sum().backward()
    for got, x in zip(ab.attention_backward(q, k, v, do, W, S, lens), leaf):
        assert np.abs(got - (np.zeros(x.shape) if x.grad is None else x.grad.numpy())).max() < 1e-9


def test_attention_against_differences():
    rng = np.random.default_rng(3)
    args = [rng.standard_normal((1, 9, h, 4)) for h in (2, 1, 1)]
    do = rng.standard_normal((1, 9, 2, 4))
    grads = ab.attention_backward(*args, do, 3, 1)
    for i, g in enumerate(grads):
        step = rng.standard_normal(args[i].shape)
        lo, hi = ([a + (s * 1e-5 * step if j == i else 0) for j, a in enumerate(args)] for s in (-1, 1))
        diff = (np.sum(ab.attention(*hi, 3, 1)[0] * do) - np.sum(ab.attention(*lo, 3, 1)[0] * do)) / 2e-5
        assert abs(diff - np.sum(g * step)) < 1e-6


def test_matches_the_multi_query_oracle():
    rng = np.random.default_rng(5)
    q, k, v = (rng.standard_normal((2, 20, h, 8)) for h in (3, 1, 1))
    ref = local_mqa(q, k[:, :, 0], v[:, :, 0], 6)
    assert np.abs(ab.attention(q, k, v, 6)[0] - ref).max() < 1e-9


@pytest.mark.parametrize("W,S", [(100, 0), (4, 0), (3, 2), (1, 0)])
def test_paged_is_the_last_row_of_attention(W, S):
    rng = np.random.default_rng(W + S)
    lens, page, dh = [11, 1, 6, 0], 4, 8
    pool_k, pool_v = rng.standard_normal((2, 9, page, 2, dh))
    table = rng.permutation(9)[:8].reshape(4, 2)
    table = np.concatenate([table, np.array([[8], [0], [0], [0]])], 1)
    q = rng.standard_normal((4, 4, dh))
    o = ab.paged_attention(q, pool_k, pool_v, table, lens, W, S)[0]
    for n, ln in enumerate(lens):
        if not ln:
            assert not o[n].any()
            continue
        u = np.arange(ln)
        k, v = (p[table[n][u // page], u % page][None] for p in (pool_k, pool_v))
        full = np.zeros((1, ln, 4, dh))
        full[0, -1] = q[n]
        assert np.abs(ab.attention(full, k, v, W, S)[0][0, -1] - o[n]).max() < 1e-9
