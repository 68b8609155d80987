"""GPU parity of the serving operators through the C ABI against their fp64 oracle (oracle/serving.py): the e4m3 cache
written, read back and attended over, attention behind a shared prefix, linear attention for prompts and single tokens,
and runs of them together.

What the cache holds is compared bit by bit. Bounds of the rest are elementwise and derived, not fitted; u = 2^-8 is
the largest relative rounding of a bf16 value, w = 2^-24 that of an fp32 operation.
Attention: scores are off by (dh + 2) w |q| |k| scale, so P by rp = 2 (dh + 2) w max + 2 (n + 8) w relatively, and by 2^-16
for its two bf16 terms; then u |o|.
Linear attention, against the same recurrence of absolute values (ao, as): every state element is a sum of n terms with
n / 64 rescalings and 64 more steps of its own chunk's sums, each an operation off by w, its terms' split into three bf16
parts off by w more; decays are exponentials of differences of one chunk's running sum b (in log2 units), each off by 8 w
|b| through the sum's steps, with 4 w for product and exponential: es = (2 n + 200 + 16 max |b|) w. o: es, dk + 64 more
operations, and 2^-16 for the two bf16 terms of S and of the scores; then u |o|."""
import numpy as np
import pytest
import torch

import gated_linear_recurrence_conv1d_amd as rg
from oracle import attention_block as ab
from oracle import serving as sv

pytestmark = pytest.mark.gpu

DEV = "cuda"
W24, U = 2.0 ** -24, 2.0 ** -8
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
E4, E8 = torch.float8_e4m3fn, torch.float8_e8m0fnu
EVERY = 1 << 30


def normal(rng, *shape, dtype=BF):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(DEV, dtype)


def ints(x, dtype=I32):
    return torch.tensor(x, dtype=dtype, device=DEV)


def num(t):
    return t.detach().double().cpu().numpy()


def raw(t):
    return t.view(torch.uint8).cpu().numpy()


def check(got, ref, bound, name):
    got = num(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == ref.shape, name
    assert np.isfinite(got).all(), name
    off = np.abs(got - ref)
    lim = np.broadcast_to(bound, ref.shape) + 1e-30
    worst = float((off / lim).max()) if off.size else 0.0
    print(f"{name}: at most {worst:.2f} of the bound", flush=True)
    assert worst <= 1.0, name


# ------------------------------------------------------------------------------------------ the cache
def empty_cache(pages, page, Hkv, dh, fill=0x5A):
    return [torch.full((pages, page, Hkv, d) if d else (pages, page, Hkv), fill, dtype=torch.uint8, device=DEV).view(t)
            for d, t in ((dh, E4), (dh, E4), (0, E8), (0, E8))]


def wide(rng, *shape, dtype):
    """Rows of all magnitudes, some zero, some of one value, some with an infinity or a NaN."""
    x = rng.standard_normal(shape) * np.exp2(rng.integers(-140, 126, shape[:-1] + (1,)).astype(np.float64))
    flat = x.reshape(-1, shape[-1])
    flat[::7] = rng.standard_normal(flat[::7].shape)
    flat[1::29] = 0
    flat[2::31, 1:] = 0
    flat[3::37, 5] = np.inf
    flat[4::41, 6] = np.nan
    flat[5::43, 7] = -np.inf
    return torch.from_numpy(np.clip(x, -3e38, 3e38) * np.where(np.isinf(x), np.inf, 1)).float().to(DEV, dtype)


WRITE = [(BF, (1,), 1, 64, 1), (BF, (7, 13), 2, 128, 16), (F32, (5, 31), 3, 64, 17), (BF, (300,), 1, 256, 64),
         (F32, (129,), 4, 256, 5), (F32, (3, 2, 9), 1, 128, 32), (BF, (67,), 11, 128, 7)]


@pytest.mark.parametrize("dtype,lead,Hkv,dh,page", WRITE)
def test_quantize_bit_by_bit(dtype, lead, Hkv, dh, page):
    rng = np.random.default_rng(dh + page)
    rows = int(np.prod(lead))
    kv = wide(rng, *lead, 2 * Hkv + 1, dh, dtype=dtype)  # parts of one projection's output
    k, v = kv[..., 1:1 + Hkv, :], kv[..., 1 + Hkv:, :]
    pages = 2 * rows // page + 2
    slots = torch.from_numpy(rng.permutation(pages * page)[:rows].reshape(lead)).to(DEV)
    skipped = rng.random(lead) < 0.2
    outside = torch.from_numpy(np.where(rng.random(lead) < 0.5, -1 - rng.integers(0, 1 << 40, lead),
                                        pages * page + rng.integers(0, 1 << 40, lead))).to(DEV)
    given = torch.where(torch.from_numpy(skipped).to(DEV), outside, slots)
    cache = empty_cache(pages, page, Hkv, dh)
    want = [raw(t).copy() for t in cache]
    rg.cache_quantize(k, v, given, *cache)
    at, on = slots.cpu().numpy().reshape(-1), ~skipped.reshape(-1)
    for x, pool, scales in ((k, 0, 2), (v, 1, 3)):
        c, b = sv.quantize(num(x).reshape(rows, Hkv, dh))
        want[pool].reshape(-1, Hkv, dh)[at[on]] = c[on]
        want[scales].reshape(-1, Hkv)[at[on]] = b[on]
    for got, ref in zip(cache, want):
        assert np.array_equal(raw(got), ref)


def filled(rng, pages, page, Hkv, dh, spread=3):
    """A cache of values of different magnitudes."""
    cache = []
    for _ in range(2):
        x = rng.standard_normal((pages, page, Hkv, dh)) * np.exp2(rng.integers(-spread, spread + 1, (pages, page, Hkv, 1)))
        cache.append(sv.quantize(x))
    (k, ks), (v, vs) = cache
    return [torch.from_numpy(x).to(DEV).view(t) for x, t in ((k, E4), (v, E4), (ks, E8), (vs, E8))]


def read_out(cache):
    return tuple(sv.values(raw(c), raw(s)) for c, s in ((cache[0], cache[2]), (cache[1], cache[3])))


READ = [(BF, 1, 64, 1, [3], [0], 5), (F32, 2, 128, 16, [40, 0, 17], None, 40), (BF, 3, 256, 7, [33, 50, 1], [30, 0, 1], 20),
        (F32, 1, 256, 64, [500], [123], 300), (BF, 5, 64, 32, [64, 31], [0, 40], 64), (BF, 1, 128, 17, [90] * 4, [1, 2, 3, 90], 89)]


@pytest.mark.parametrize("rest", [True, False])
@pytest.mark.parametrize("dtype,Hkv,dh,page,lens,starts,T", READ)
def test_dequantize(dtype, Hkv, dh, page, lens, starts, T, rest):
    rng = np.random.default_rng(T + dh)
    B, width = len(lens), -(-max(lens) // page) or 1
    cache = filled(rng, B * width + 2, page, Hkv, dh, spread=100)
    table = rng.permutation(B * width + 2)[:B * width].reshape(B, width)
    kv = torch.full((B, T, 2 * Hkv, dh), 7.0, dtype=dtype, device=DEV)  # k and v beside each other
    ko, vo = kv[:, :, :Hkv], kv[:, :, Hkv:]
    rg.rglru_cache_dequantize(*cache, ints(table), ints(lens), ko, vo, None if starts is None else ints(starts), rest)
    for got, pool in zip((ko, vo), read_out(cache)):
        want = np.full((B, T, Hkv, dh), 0.0 if rest else 7.0)
        for b, n in enumerate(lens):
            u = np.arange(starts[b] if starts else 0, n)[:T]
            want[b, :len(u)] = pool[table[b][u // page], u % page]
        assert np.array_equal(num(got), want)
    if rest:
        k, v = rg.cache_dequantize(*cache, ints(table), ints(lens), T, None if starts is None else ints(starts), dtype)
        assert torch.equal(k, ko) and torch.equal(v, vo)


def test_dequantize_all_codes_and_scales():
    """Every code under every scale byte, as the format defines it."""
    c = torch.arange(256, dtype=torch.uint8, device=DEV)
    pages = c.view(4, 64).repeat(256, 1, 1).view(256, 4, 1, 64)
    scales = c.view(256, 1, 1).repeat(1, 4, 1).contiguous()
    cache = [pages.view(E4), pages.flip(0).contiguous().view(E4), scales.view(E8), scales.flip(0).contiguous().view(E8)]
    for dtype in (F32, BF):
        k, v = rg.cache_dequantize(*cache, ints([list(range(256))]), ints([1024]), 1024, dtype=dtype)
        want = sv.values(raw(cache[0]), raw(cache[2])).reshape(1, 1024, 1, 64)
        big = np.float64(2.0 ** 128)
        exact = (np.abs(want) < big) & (raw(scales).repeat(64).reshape(want.shape) >= 10)
        got = num(k)
        assert np.array_equal(got[exact], want[exact])
        assert np.array_equal(np.isnan(got), np.isnan(want))
        assert np.isinf(got[np.abs(want) >= big]).all()
        # scales below those that this library writes: products below the least normal number may come as 0, off by
        # less than that number; the others are exact
        tiny = ~exact & (np.abs(want) < big)
        assert (np.abs(got[tiny] - want[tiny]) < 2.0 ** -126).all()
        assert np.array_equal(got[tiny & (np.abs(want) >= 2.0 ** -126)], want[tiny & (np.abs(want) >= 2.0 ** -126)])
        assert torch.equal(v.view(256, 4, 64).flip(0).nan_to_num(1.5), k.view(256, 4, 64).nan_to_num(1.5))


def test_dequantize_what_cannot_be_followed():
    rng = np.random.default_rng(3)
    page, Hkv, dh, T = 8, 2, 64, 20
    cache = filled(rng, 10, page, Hkv, dh)
    table = np.arange(15).reshape(5, 3) % 10
    table[1, 1], table[2, 2] = 10, -1
    lens, starts = [24, 24, 17, 25, -1], [0, 0, -1, 0, 0]
    for rest in (True, False):
        k, v = (torch.full((5, T, Hkv, dh), 7.0, dtype=BF, device=DEV) for _ in range(2))
        rg.rglru_cache_dequantize(*cache, ints(table), ints(lens), k, v, ints(starts), rest)
        for got in (num(k), num(v)):
            assert np.isfinite(got[0]).all()
            assert np.isnan(got[1, 8:16]).all() and np.isfinite(got[1, :8]).all() and np.isfinite(got[1, 16:]).all()
            assert np.isnan(got[2:]).all()
    # a page that no read token lies on may be any
    k, _ = rg.cache_dequantize(*cache, ints(table[2:3]), ints([16]), T)
    assert np.isfinite(num(k)).all()


def test_round_trip_beyond_32_bits():
    """A pool of more than 2^32 bytes whose last pages are the ones in use."""
    rng = np.random.default_rng(5)
    page, Hkv, dh = 64, 1, 256
    pages = (1 << 32) // (page * Hkv * dh) + 40
    cache = [torch.zeros(pages, page, Hkv, dh, dtype=torch.uint8, device=DEV).view(E4) for _ in range(2)]
    cache += [torch.zeros(pages, page, Hkv, dtype=torch.uint8, device=DEV).view(E8) for _ in range(2)]
    table = torch.arange(pages - 20, pages, device=DEV, dtype=I32).view(2, 10)
    lens = ints([600, 77])
    k, v = normal(rng, 2, 600, Hkv, dh), normal(rng, 2, 600, Hkv, dh)
    u = torch.arange(600, device=DEV)
    slots = table.long()[:, u // page] * page + u % page
    rg.cache_quantize(k, v, slots, *cache)
    small = [t[-40:].clone() for t in (x.view(torch.uint8) for x in cache)]
    small = [x.view(t) for x, t in zip(small, (E4, E4, E8, E8))]
    c, b = sv.quantize(num(k))
    kb, _ = rg.cache_dequantize(*cache, table, ints([600, 600]), 600, dtype=F32)
    assert np.array_equal(num(kb), sv.values(c, b))
    q = normal(rng, 2, 10, dh)
    o = rg.paged_attention_e4m3(q, *cache, table, lens, EVERY)
    assert torch.equal(o, rg.paged_attention_e4m3(q, *small, table - (pages - 40), lens, EVERY))
    paged_check(o, q, small, table.cpu().numpy() - (pages - 40), [600, 77], EVERY, 0)
    pt, pl = table[1, :7].contiguous(), ints([433])
    x = rg.prefix_attention(q, cache[0], cache[1], pt, pl, table[:1].expand(2, -1).contiguous(), lens, EVERY, 0, 0.0,
                            cache[2], cache[3])
    y = rg.prefix_attention(q, small[0], small[1], pt - (pages - 40), pl,
                            (table[:1] - (pages - 40)).expand(2, -1).contiguous(), lens, EVERY, 0, 0.0, small[2], small[3])
    assert torch.equal(x, y)


# --------------------------------------------------------------------------- one token over the cache
def attention_bound(o, mag, most, dh, n):
    rp = 2 * (dh + 2) * W24 * most + (n + 8) * 2 * W24
    return ((rp + 2.0 ** -16) * mag + U * np.abs(o)) * (1 + 2.0 ** -7)


def paged_check(got, q, cache, table, lens, W, S, scale=None):
    o, mag, most = ab.paged_attention(num(q), *read_out(cache), table, lens, W, S, scale)
    check(got, o, attention_bound(o, mag, most, q.shape[2], max(lens)), "o")


PAGED = [([1], 1, 1, 64, 16, EVERY, 0, None), ([5, 0, 31, 32, 33], 4, 2, 128, 16, EVERY, 0, None),
         ([700, 1, 200], 10, 1, 256, 64, 128, 4, None), ([300, 77], 17, 1, 128, 7, 100, 3, 0.3),
         ([64, 65], 6, 3, 64, 1, 40, 0, None), ([1000] * 3, 16, 1, 256, 24, EVERY, 0, None),
         ([9000, 40, 3], 8, 2, 128, 32, EVERY, 0, None), ([513], 33, 1, 64, 48, 300, 70, None),
         (list(range(1, 65)), 10, 1, 256, 16, EVERY, 0, None), (list(range(1, 65)), 4, 2, 64, 5, 30, 9, None)]


def paged_inputs(rng, lens, Hq, Hkv, dh, page):
    width = max(1, -(-max(lens) // page))
    cache = filled(rng, len(lens) * width + 2, page, Hkv, dh)
    table = rng.permutation(len(lens) * width + 2)[:len(lens) * width].reshape(len(lens), width)
    q = normal(rng, len(lens), Hq + 2, dh)[:, 1:1 + Hq]
    return q, cache, table


@pytest.mark.parametrize("lens,Hq,Hkv,dh,page,W,S,scale", PAGED)
def test_paged_attention_e4m3(lens, Hq, Hkv, dh, page, W, S, scale):
    rng = np.random.default_rng(sum(lens) + dh)
    q, cache, table = paged_inputs(rng, lens, Hq, Hkv, dh, page)
    got = rg.paged_attention_e4m3(q, *cache, ints(table), ints(lens), W, S, scale or 0.0)
    paged_check(got, q, cache, table, lens, W, S, scale)


@pytest.mark.parametrize("page", [32, 24])
@pytest.mark.parametrize("dh", [64, 256])
def test_paged_e4m3_out_of_sight_does_not_matter(page, dh):
    """NaN codes and scales behind the end, before the window and on pages that are not needed change nothing."""
    rng = np.random.default_rng(8)
    lens, W, S = [100, 41], 50, 3
    q, cache, table = paged_inputs(rng, lens, 6, 2, dh, page)
    want = rg.paged_attention_e4m3(q, *cache, ints(table), ints(lens), W, S)
    seen = np.zeros(raw(cache[0]).shape[:2], bool)
    bad = table.copy()
    for n, L in enumerate(lens):
        u = np.arange(L)
        u = u[(u >= L - W) | (u < S)]
        seen[table[n][u // page], u % page] = True
        unused = np.setdiff1d(np.arange(table.shape[1]), u // page)
        bad[n, unused] = 1 << 20
    for t in cache:
        x = t.view(torch.uint8)
        x[torch.from_numpy(~seen).to(DEV)] = 255
    assert torch.equal(rg.paged_attention_e4m3(q, *cache, ints(bad), ints(lens), W, S), want)
    assert np.isfinite(num(want)).all()


@pytest.mark.parametrize("page,long", [(32, 60), (20, 60), (32, 2000), (20, 2000)])
def test_paged_e4m3_that_cannot_be_followed_is_nan(page, long):
    rng = np.random.default_rng(9)
    lens = [long, long, long, long]
    q, cache, table = paged_inputs(rng, lens, 4, 2, 64, page)
    table = table.copy()
    table[1, 1], table[2, 0] = -1, len(raw(cache[0]))
    got = num(rg.paged_attention_e4m3(q, *cache, ints(table), ints([long, long, long, table.shape[1] * page + 1]), EVERY))
    assert np.isfinite(got[0]).all() and np.isnan(got[1:]).all()
    got = num(rg.paged_attention_e4m3(q, *cache, ints(table), ints([long, 0, -1, 5]), EVERY))
    assert np.isfinite(got[0]).all() and not got[1].any() and np.isnan(got[2]).all() and np.isfinite(got[3]).all()


# ------------------------------------------------------------------------------------- a shared prefix
def prefix_inputs(rng, kind, P, lens, Hq, Hkv, dh, page):
    width, held = max(1, -(-max(lens) // page)), max(1, -(-P // page))
    pages = held + len(lens) * width + 2
    if kind == "e4m3":
        cache = filled(rng, pages, page, Hkv, dh)
        pools = read_out(cache)
    else:
        cache = [normal(rng, pages, page, Hkv, dh) for _ in range(2)]
        pools = tuple(num(x) for x in cache)
    at = rng.permutation(pages)
    pt, table = at[:held], at[held:held + len(lens) * width].reshape(len(lens), width)
    q = normal(rng, len(lens), Hq + 1, dh)[:, :Hq]
    return q, cache, pools, pt, table


def run_prefix(q, cache, pt, P, table, lens, W, S, scale=0.0, **kw):
    scales = dict(k_scales=cache[2], v_scales=cache[3]) if len(cache) == 4 else {}
    return rg.prefix_attention(q, cache[0], cache[1], ints(pt), ints([P]), ints(table), ints(lens), W, S, scale, **scales,
                               **kw)


PREFIX = [(1, [1], 1, 1, 64, 16, EVERY, 0, None), (0, [3, 0, 40], 4, 2, 128, 16, EVERY, 0, None),
          (33, [0, 1, 50], 6, 2, 128, 7, EVERY, 0, None), (700, [1, 20, 90, 33, 64, 5], 10, 1, 256, 16, EVERY, 0, None),
          (500, [1, 200, 450, 300], 4, 1, 256, 64, 300, 4, None), (100, [10, 300, 120], 8, 4, 64, 1, 150, 0, 0.25),
          (90, list(range(0, 130)), 3, 1, 64, 32, 100, 50, None), (300, list(range(1, 40)), 17, 1, 128, 20, 1, 0, None),
          (64, [0] * 5, 16, 1, 256, 32, EVERY, 0, None), (2000, [7] * 50, 8, 2, 128, 16, 1900, 130, None),
          (5000, [600, 0, 31], 2, 2, 64, 128, EVERY, 0, None), (40, [100, 3], 2, 1, 128, 16, 30, 60, None)]


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("P,lens,Hq,Hkv,dh,page,W,S,scale", PREFIX)
def test_prefix_attention(kind, P, lens, Hq, Hkv, dh, page, W, S, scale):
    rng = np.random.default_rng(P + dh)
    q, cache, pools, pt, table = prefix_inputs(rng, kind, P, lens, Hq, Hkv, dh, page)
    got = run_prefix(q, cache, pt, P, table, lens, W, S, scale or 0.0)
    o, mag, most = sv.prefix_attention(num(q), *pools, pt, P, table, lens, W, S, scale)
    check(got, o, attention_bound(o, mag, most, dh, P + max(lens)), "o")
    assert torch.equal(got, run_prefix(q, cache, pt, P, table, lens, W, S, scale or 0.0))  # sums in a fixed order


@pytest.mark.parametrize("bad", [False, True])
@pytest.mark.parametrize("kind,dh,page", [("bf16", 64, 16), ("e4m3", 64, 12), ("bf16", 256, 12), ("e4m3", 256, 16), ("e4m3", 128, 64)])
def test_prefix_of_long_chunks(kind, dh, page, bad):
    """Chunks of 30 blocks of the prefix, the first one with sinks, a gap that no row sees and the rows' windows; bad: what
    nobody sees there is NaN, and a v that some rows see makes the others' go key by key. A lane of a chunk sums 16 values
    of each of 30 blocks, and 32 chunks and two halves are joined: so many operations behind one another."""
    rng = np.random.default_rng(dh)
    P, N, Hq, S, W = 30000, 256, 8, 70, 30000 - 400  # a row with n tokens of its own sees from 400 + n on
    lens = rng.integers(0, 201, N)
    lens[:6] = [0, 5, 10, 11, 200, 97]
    q, cache, pools, pt, table = prefix_inputs(rng, kind, P, lens, Hq, 1, dh, page)
    q = q * 2
    some = np.array([0, 1, 2, 3, 4, 5, 100, 255])
    o, mag, most = sv.prefix_attention(num(q)[some], *pools, pt, P, table[some], lens[some], W, S)
    depth = 16 * 30 + 32 + 64
    if bad:
        for t, which in ((200, (0, 1)), (410, (1,))):  # in the gap; before the windows of more than 10 own tokens
            for i in which:
                if kind == "e4m3":
                    cache[2 + i].view(torch.uint8)[int(pt[t // page]), t % page, 0] = 255
                else:
                    cache[i][int(pt[t // page]), t % page, 0, 3] = float("nan")
    got = run_prefix(q, cache, pt, P, table, lens, W, S)
    assert torch.equal(got.nan_to_num(7.0), run_prefix(q, cache, pt, P, table, lens, W, S).nan_to_num(7.0))
    x, sees = num(got)[some], lens[some] <= 10
    if bad:
        assert np.isnan(x[sees][..., 3]).all() and np.isnan(num(got)[lens <= 10][..., 3]).all()
        assert np.isfinite(num(got)[lens > 10]).all()
        x, o, mag, most = (y[~sees] for y in (x, o, mag, most))
    check(x, o, attention_bound(o, mag, most, dh, depth), "o")


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("P", [31, 700, 2000, 7000, 13000, 20000, 30000, 45000, 52000])  # 1 to 8 blocks a chunk
def test_prefix_of_all_chunk_lengths(kind, P):
    """A lane sums 16 values of each of up to 8 blocks; up to 245 chunks are joined, in four waves."""
    rng = np.random.default_rng(P)
    lens, Hq, dh, page, S, W = [7, 0, 90], 3, 64, 48, 40, P - P // 3
    q, cache, pools, pt, table = prefix_inputs(rng, kind, P, lens, Hq, 1, dh, page)
    q = q * 2
    got = run_prefix(q, cache, pt, P, table, lens, W, S)
    o, mag, most = sv.prefix_attention(num(q), *pools, pt, P, table, lens, W, S)
    check(got, o, attention_bound(o, mag, most, dh, 16 * 8 + 245 // 4 + 64), "o")


def test_prefix_scores_far_apart():
    """A prefix whose scores lie far above or below the own tokens' ones, and rising through it."""
    rng = np.random.default_rng(4)
    P, lens, Hq, dh, page = 200, [50, 3], 4, 128, 16
    q, cache, _, pt, table = prefix_inputs(rng, "bf16", P, lens, Hq, 1, dh, page)
    for f, g in ((40.0, 0.01), (0.01, 40.0), (40.0, 40.0)):
        k = cache[0].clone()
        k[torch.from_numpy(pt).to(DEV)] *= f
        k[torch.from_numpy(table.reshape(-1)).to(DEV)] *= g
        o, mag, most = sv.prefix_attention(num(q), num(k), num(cache[1]), pt, P, table, lens, EVERY)
        got = run_prefix(q, [k, cache[1]], pt, P, table, lens, EVERY, 0)
        check(got, o, attention_bound(o, mag, most, dh, P + 50), "o")


@pytest.mark.parametrize("S", [2 ** 31 - 1, 2 ** 31 - 32, 130])
def test_prefix_all_sinks(S):
    """More sinks than tokens: everything is visible, whatever the window."""
    rng = np.random.default_rng(36)
    P, lens, page = 200, [1, 40, 0], 16
    q, cache, pools, pt, table = prefix_inputs(rng, "bf16", P, lens, 4, 2, 64, page)
    got = run_prefix(q, cache, pt, P, table, lens, 5, S)
    o, mag, most = sv.prefix_attention(num(q), *pools, pt, P, table, lens, 5, S)
    check(got, o, attention_bound(o, mag, most, 64, P + 40), "o")


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("page", [16, 12])
@pytest.mark.parametrize("dh", [64, 128, 256])
def test_prefix_out_of_sight_does_not_matter(kind, page, dh):
    """What no row sees may be anything; what some rows see and others not (an infinite or NaN k or v before some
    rows' windows) reaches the rows that see it and no others."""
    rng = np.random.default_rng(6)
    P, W, S = 170, 120, 2
    lens = [0, 30, 60, 100, 119, 130, 5] * 6
    q, cache, pools, pt, table = prefix_inputs(rng, kind, P, lens, 4, 2, dh, page)
    held = np.zeros(raw(cache[0]).shape[:2], bool)  # some row may see it
    u = np.arange(P)
    first = P - W  # of the row without own tokens
    u = u[(u >= first) | (u < S)]
    held[pt[u // page], u % page] = True
    for n, own in enumerate(lens):
        j = np.arange(max(0, own - W), own)
        held[table[n][j // page], j % page] = True
    far = pt.copy()
    far[np.setdiff1d(np.arange(len(pt)), u // page)] = -5
    dirty = []
    for t in cache:
        x = t.clone() if kind == "bf16" else t.view(torch.uint8).clone()
        x[torch.from_numpy(~held).to(DEV)] = float("nan") if kind == "bf16" else 255
        dirty.append(x if kind == "bf16" else x.view(t.dtype))
    # (not bit by bit: a row whose block has a NaN in sight of none is summed key by key)
    ref, mag, most = sv.prefix_attention(num(q), *pools, pt, P, table, lens, W, S)
    bound = attention_bound(ref, mag, most, dh, P + 130)
    check(run_prefix(q, dirty, far, P, table, lens, W, S), ref, bound, "nothing bad in sight")
    # token 80: seen where 80 >= P + own - W, that is own <= 30
    sees = np.array(lens) <= 80 + W - P
    for which in (0, 1):
        for bad in ([float("inf"), float("nan")] if kind == "bf16" else [None]):
            x = [t.clone() if kind == "bf16" else t.view(torch.uint8).clone().view(t.dtype) for t in dirty]
            if kind == "bf16":
                x[which][int(pt[80 // page]), 80 % page, 0, 3] = bad
            else:
                x[2 + which].view(torch.uint8)[int(pt[80 // page]), 80 % page, 0] = 255
            got = num(run_prefix(q, x, far, P, table, lens, W, S))
            g0 = got[:, :2]  # the heads on key/value head 0
            assert (~np.isfinite(g0[sees]).all(-1)).all() or bad == float("inf") and which == 0
            if which == 1:
                assert not np.isfinite(g0[sees][..., 3]).any()
            check(g0[~sees], ref[:, :2][~sees], bound[:, :2][~sees], "rows that do not see it")
            check(got[:, 2:], ref[:, 2:], bound[:, 2:], "the other key/value head")


def test_prefix_that_cannot_be_followed_is_nan():
    rng = np.random.default_rng(7)
    P, lens, page = 100, [10, 20, 60, 4], 16
    q, cache, _, pt, table = prefix_inputs(rng, "bf16", P, lens, 4, 2, 64, page)
    want = num(run_prefix(q, cache, pt, P, table, lens, EVERY, 0))
    for bad_len in (-1, len(pt) * page + 1):
        assert np.isnan(num(run_prefix(q, cache, pt, bad_len, table, lens, EVERY, 0))).all()
    for own in (-1, table.shape[1] * page + 1):
        got = num(run_prefix(q, cache, pt, P, table, [10, own, 60, 4], EVERY, 0))
        assert np.isnan(got[1]).all() and np.array_equal(got[[0, 2, 3]], want[[0, 2, 3]])
    bad = table.copy()
    bad[2, 1] = 1 << 30
    got = num(run_prefix(q, cache, pt, P, bad, lens, EVERY, 0))
    assert np.isnan(got[2]).all() and np.array_equal(got[[0, 1, 3]], want[[0, 1, 3]])
    for page_no in (-1, 1 << 30):
        bp = pt.copy()
        bp[2] = page_no  # tokens 32 .. 47: in sight of rows with own < 48 + 90 - 100, that is 38
        got = num(run_prefix(q, cache, bp, P, table, lens, 90, 0))
        assert np.isnan(got[[0, 1, 3]]).all() and np.isfinite(got[2]).all()
        assert np.isnan(num(run_prefix(q, cache, bp, P, table, lens, EVERY, 0))).all()


def test_prefix_of_many_sequences():
    """More rows than a dimension of a launch holds threads for: 2^24 + 3 sequences of a prefix token and one of their
    own, whose values are the same: o is that value."""
    N, dh, page = (1 << 24) + 3, 64, 16
    gen = torch.Generator(device=DEV).manual_seed(2)
    q = torch.randn(N, 1, dh, generator=gen, device=DEV, dtype=BF)
    kp = torch.randn(64, page, 1, dh, generator=gen, device=DEV, dtype=BF)
    vp = torch.randn(1, 1, 1, dh, generator=gen, device=DEV, dtype=BF).expand(64, page, 1, dh).contiguous()
    table = torch.randint(0, 64, (N, 1), generator=gen, device=DEV, dtype=I32)
    got = rg.prefix_attention(q, kp, vp, ints([3]), ints([1]), table, torch.ones(N, dtype=I32, device=DEV), 100)
    off = (got - vp[0, 0, 0]).abs()
    assert (off <= 2 * U * vp[0, 0, 0].abs()).all()


# ------------------------------------------------------------------------------------ linear attention
LINEAR = [(1, 1, 1, 1, 64, 64, None, True, False), (2, 63, 1, 2, 64, 128, None, False, True),
          (1, 64, 2, 2, 128, 64, None, True, True), (3, 65, 1, 3, 128, 128, [65, 0, 1], True, True),
          (2, 200, 2, 4, 256, 64, [200, 77], False, False), (1, 130, 1, 1, 64, 256, None, True, True),
          (1, 700, 1, 2, 128, 128, [699], True, True), (2, 400, 2, 2, 256, 256, [300, 400], True, False),
          (5, 301, 3, 6, 64, 64, [301, 250, 129, 64, -3], True, True), (1, 1500, 1, 1, 128, 256, None, False, True)]


def linear_inputs(rng, B, T, Hk, H, dk, dv, gated, start, strong=1.0):
    qkv = normal(rng, B, T, 2 * Hk * dk + H * dv + 8)  # one projection's output
    q = qkv[..., :Hk * dk].unflatten(-1, (Hk, dk))
    k = qkv[..., Hk * dk:2 * Hk * dk].unflatten(-1, (Hk, dk))
    v = qkv[..., 2 * Hk * dk:-8].unflatten(-1, (H, dv))
    g = -strong * np.abs(rng.standard_normal((B, T, H) if gated else H)) * (0.3 if gated else 0.05)
    s0 = normal(rng, B, H, dk, dv, dtype=F32) if start else None
    return q, k, v, torch.from_numpy(g.astype(np.float32)).to(DEV), s0


def chunk_sums(g, B, T, H):
    """The largest |running sum| of log2 decays in a chunk of 64."""
    g = np.maximum(np.broadcast_to(num(g), (B, T, H)), sv.LEAST) / np.log(2)
    pad = np.zeros((B, -T % 64, H))
    return np.abs(np.concatenate([g, pad], 1).reshape(B, -1, 64, H).sum(2)).max()


def linear_check(o, s, q, k, v, g, s0, lens, scale=None):
    B, T, Hk, dk = q.shape
    ro, rs, ao, as_ = sv.linear_attention(num(q), num(k), num(v), num(g), None if s0 is None else num(s0), lens, scale)
    es = (2 * T + 200 + 16 * chunk_sums(g, B, T, v.shape[2])) * W24
    check(s, rs, es * as_, "state")
    check(o, ro, ((es + (dk + 64) * W24 + 2.0 ** -16) * ao + U * np.abs(ro)) * (1 + U), "o")


@pytest.mark.parametrize("B,T,Hk,H,dk,dv,lens,gated,start", LINEAR)
def test_linear_attention(B, T, Hk, H, dk, dv, lens, gated, start):
    rng = np.random.default_rng(T + dk)
    q, k, v, g, s0 = linear_inputs(rng, B, T, Hk, H, dk, dv, gated, start)
    dl = None if lens is None else ints(lens)
    if lens is not None:  # what lies behind a sequence may be anything
        for b, n in enumerate(lens):
            q[b, max(n, 0):] = float("nan")
            k[b, max(n, 0):] = float("inf")
            v[b, max(n, 0):] = float("nan")
            if gated:
                g[b, max(n, 0):] = float("nan")
    o, s = rg.linear_attention(q, k, v, g, s0, dl)
    clean = [x.clone() for x in (q, k, v, g)]
    if lens is not None:
        for x in clean[:3 + gated]:
            for b, n in enumerate(lens):
                x[b, max(n, 0):] = 0
    linear_check(o, s, *clean, s0, lens)
    # in place, and again: sums in a fixed order
    if start:
        mine = s0.clone()
        o2, s2 = rg.linear_attention(q, k, v, g, mine, dl, state_out=mine)
        assert s2 is mine and torch.equal(o, o2) and torch.equal(s, mine)
    rg.rglru_linear_attention(q, k, v, g, o2 := torch.empty_like(o), s0, None, dl, workspace=torch.empty(
        max(1, rg.rglru_linear_attention_workspace_size(B, T, Hk, H, dk, dv)), dtype=torch.uint8, device=DEV))
    assert torch.equal(o, o2)


@pytest.mark.parametrize("T", [250, 512, 520, 800, 1100, 1300, 2500])  # 2 to 20 segments, states of parts
def test_linear_segments(T):
    """Segments whose decays let nothing, a part or all of the ones before them through, and sequences that end in the
    first, in a middle and in the last one."""
    rng = np.random.default_rng(T)
    B, Hk, H, dk, dv = 3, 1, 4, 64, 64
    q, k, v, g, s0 = linear_inputs(rng, B, T, Hk, H, dk, dv, True, True)
    g *= torch.tensor([1e-3, 0.1, 3.0, 60.0], device=DEV)
    g[:, T // 2, 1] = -float("inf")
    lens = [T, T // 2, 40]
    o, s = rg.linear_attention(q, k, v, g, s0, ints(lens))
    linear_check(o, s, q, k, v, g, s0, lens)
    mine = s0.clone()
    o2, _ = rg.linear_attention(q, k, v, g, mine, ints(lens), state_out=mine)
    assert torch.equal(o, o2) and torch.equal(s, mine)


@pytest.mark.parametrize("B,H", [(32, 8), (33, 8)])  # a workgroup a CU, and more of them
def test_linear_of_many_sequences(B, H):
    rng = np.random.default_rng(B)
    T, dk, dv = 70, 128, 128
    q, k, v, g, s0 = linear_inputs(rng, B, T, 1, H, dk, dv, True, True)
    lens = [(37 * b) % (T + 1) for b in range(B)]
    o, s = rg.linear_attention(q, k, v, g, s0, ints(lens))
    linear_check(o, s, q, k, v, g, s0, lens)


@pytest.mark.parametrize("B,T,H,dk,dv", [(8, 1100, 64, 64, 64), (1, 16390, 64, 64, 64), (2, 5000, 32, 128, 128),
                                         (1, 9000, 32, 256, 128), (40, 1300, 8, 128, 128)])
def test_linear_of_many_chunks(B, T, H, dk, dv):
    """18 chunks and more one after another in a workgroup, forming states (but in the first and the last case) and o, with
    decays that let a token, some chunks, or everything through. Against the oracle for some sequences and heads."""
    rng = np.random.default_rng(T)
    q, k, v, g, s0 = linear_inputs(rng, B, T, 1, H, dk, dv, True, True)
    g *= torch.tensor([1e-4, 1e-2, 0.1, 0.4, 3.0] * H, device=DEV)[:H]
    lens = [T - 70 * (b % 3) for b in range(B)]
    o, s = rg.linear_attention(q, k, v, g, s0, ints(lens))
    assert torch.equal(o, rg.linear_attention(q, k, v, g, s0, ints(lens))[0])
    for b in {0, B - 1}:
        h = [0, 1, 2, 3, 4, H - 1]
        part = q[b:b + 1], k[b:b + 1], v[b:b + 1, :, h], g[b:b + 1, :, h], s0[b:b + 1, h]
        n = lens[b]
        ro, rs, ao, as_ = sv.linear_attention(*(num(x) for x in part), [n])
        es = (2 * n + 200) * W24 + decay_error(n)
        check(s[b:b + 1, h], rs, es * as_, "state")
        check(o[b:b + 1][:, :, h], ro, ((es + (dk + 64) * W24 + 2.0 ** -16) * ao + U * np.abs(ro)) * (1 + U), "o")


def test_linear_decays_of_all_strengths():
    """No decay, decays that underflow within a chunk, and tokens that forget the state."""
    rng = np.random.default_rng(11)
    B, T, H, dk, dv = 1, 300, 4, 64, 64
    q, k, v, _, s0 = linear_inputs(rng, B, T, H, H, dk, dv, False, True)
    g = torch.zeros(B, T, H, device=DEV)
    g[..., 1] = -20.0
    g[:, 100, 2] = g[:, 203, 2] = -float("inf")
    g[..., 3] = -1e-6
    g[:, 50, 3] = -300.0
    o, s = rg.linear_attention(q, k, v, g, s0)
    linear_check(o, s, q, k, v, g, s0, None)
    # from the forgetting token on, nothing before it matters
    k2, v2 = k.clone(), v.clone()
    k2[:, :203, 2], v2[:, :203, 2] = 1e3, -1e3
    o2, s2 = rg.linear_attention(q, k2, v2, g, s0 * 5)
    assert torch.allclose(o2[:, 203:, 2].float(), o[:, 203:, 2].float(), rtol=2 * U, atol=1e-6)
    assert torch.allclose(s2[:, 2], s[:, 2], rtol=1e-5, atol=1e-5)


@pytest.mark.parametrize("T", [200, 1100])
def test_linear_forgetting_is_exact(T):
    """Many tokens that forget the state (documents in one row): the others' weights are as exact as without them, so
    the running sums that count are those of the other tokens alone."""
    rng = np.random.default_rng(T)
    B, H, dk, dv = 2, 3, 64, 128
    q, k, v, g, s0 = linear_inputs(rng, B, T, 1, H, dk, dv, True, True)
    others = g.clone()
    for b in range(B):
        for t in rng.choice(T, T // 7, replace=False):
            g[b, t] = torch.tensor([-float("inf"), -1e9, -104.5], device=DEV)
            others[b, t] = 0
    o, s = rg.linear_attention(q, k, v, g, s0)
    ro, rs, ao, as_ = sv.linear_attention(num(q), num(k), num(v), num(g), num(s0))
    es = (2 * T + 200 + 16 * chunk_sums(others, B, T, H)) * W24
    check(s, rs, es * as_, "state")
    check(o, ro, ((es + (dk + 64) * W24 + 2.0 ** -16) * ao + U * np.abs(ro)) * (1 + U), "o")


# What follows holds a decay to its own size, however strong the ones before it are: a weight exp(-x) is 2^b with b = -x
# log2 e from sums in 64 bits, rounded once to fp32 (|b| 2^-24, that is x w of the weight), and an exponential off by 2 w.
# A state is rescaled once a chunk (w more): over c chunks (x + 3 c) w in all, x <= 104 (else the weight is 0, or below
# 2^-149).
def decay_error(T):
    return (104 + 3 * (T // 64 + 2)) * W24


STRONG = {"isolated": (-20.0, 9), "-60": (-60.0, 8), "-103": (-103.0, 30), "resets": (-103.9, 2), "none": (0.0, 1 << 20)}


def strong_decays(rng, B, T, H, kind):
    """Weak decays, and among them strong ones just above those that forget the state: one in so many tokens, and runs of
    48 of them before weak ones."""
    value, every = STRONG[kind]
    g = -0.02 * np.abs(rng.standard_normal((B, T, H)))
    g[rng.random((B, T, H)) < 1.0 / every] = value
    if kind == "resets":
        g[:, (np.arange(T) % 64) >= 48] = -0.01
    return torch.from_numpy(g.astype(np.float32)).to(DEV)


@pytest.mark.parametrize("kind", list(STRONG))
@pytest.mark.parametrize("B,T,H,dk,dv", [(1, 64, 2, 64, 64), (2, 256, 4, 256, 64), (1, 250, 2, 256, 256), (40, 128, 8, 128, 128)])
def test_linear_weights_of_single_tokens(B, T, H, dk, dv, kind):
    """Token t's key is the unit vector t: row t of the state is then v_t times the token's weight alone, off by the
    weight's own error, the product's and the three terms' (4 w with the exact values' conversion)."""
    rng = np.random.default_rng(T + dk)
    assert T <= dk
    q, _, v, _, _ = linear_inputs(rng, B, T, 1, H, dk, dv, True, False)
    k = torch.eye(T, dk, device=DEV, dtype=BF).view(1, T, 1, dk).expand(B, T, 1, dk).contiguous()
    g = strong_decays(rng, B, T, H, kind)
    o, s = rg.linear_attention(q, k, v, g)
    x = num(g)[:, ::-1].cumsum(1)[:, ::-1] - num(g)  # what follows each token
    w = np.exp(x)[..., None] * num(v)  # [B, T, H, dv]
    rel = (-x[..., None] + 3 * (T // 64 + 2) + 4) * W24
    check(s[:, :, :T], w.transpose(0, 2, 1, 3), (rel * np.abs(w)).transpose(0, 2, 1, 3), "state")
    assert not s[:, :, T:].any()


@pytest.mark.parametrize("kind", list(STRONG))
@pytest.mark.parametrize("T,dk,dv", [(64, 64, 64), (333, 128, 128), (1100, 64, 128), (700, 256, 64)])
def test_linear_strong_decays_among_weak(T, dk, dv, kind):
    rng = np.random.default_rng(T + dv)
    B, H = 2, 2
    q, k, v, _, s0 = linear_inputs(rng, B, T, 1, H, dk, dv, True, True)
    g = strong_decays(rng, B, T, H, kind)
    o, s = rg.linear_attention(q, k, v, g, s0)
    ro, rs, ao, as_ = sv.linear_attention(num(q), num(k), num(v), num(g), num(s0))
    es = (2 * T + 200) * W24 + decay_error(T)
    check(s, rs, es * as_, "state")
    check(o, ro, ((es + (dk + 64) * W24 + 2.0 ** -16) * ao + U * np.abs(ro)) * (1 + U), "o")


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 256), (256, 128)])
def test_linear_bad_inputs_reach_later_rows_only(bad, dk, dv):
    rng = np.random.default_rng(12)
    B, T, H = 2, 200, 2
    q, k, v, g, s0 = linear_inputs(rng, B, T, H, H, dk, dv, True, True)
    want, _ = rg.linear_attention(q, k, v, g, s0)
    for which, t in ((0, 70), (1, 70), (2, 70), (2, 0), (2, 63), (1, 32), (2, 97), (3, 45)):
        x = [y.clone() for y in (q, k, v, g)]
        if which == 3:
            x[3][0, t, 1] = float("nan")
        else:
            x[which][0, t, 1, 5] = bad
        o, _ = rg.linear_attention(*x, s0)
        off = (o.float() - want.float()).abs()
        assert torch.equal(o[1], want[1]) and torch.equal(o[0, :, 0], want[0, :, 0]), which
        before = o[0, :t, 1].float()
        assert torch.isfinite(before).all(), (which, t)
        assert (off[0, :t, 1] <= 2 * U * want[0, :t, 1].float().abs() + 1e-3).all(), (which, t)
        if which == 0:
            assert not torch.isfinite(o[0, t, 1]).any() and torch.equal(o[0, t + 1:, 1], want[0, t + 1:, 1])
        elif which == 2:
            assert not torch.isfinite(o[0, t:, 1, 5]).any()
            others = [c for c in range(dv) if c != 5]
            assert torch.isfinite(o[0, :, 1][:, others]).all()
        else:
            assert not torch.isfinite(o[0, t:, 1]).all(-1).any()


def test_linear_in_parts_and_token_by_token():
    """A prompt in two parts, then single tokens, against the oracle over the whole."""
    rng = np.random.default_rng(13)
    B, T, Hk, H, dk, dv, n0, n1 = 3, 150, 2, 4, 128, 64, 70, 140
    q, k, v, g, s0 = linear_inputs(rng, B, T, Hk, H, dk, dv, True, True)
    ro, rs, ao, as_ = sv.linear_attention(num(q), num(k), num(v), num(g), num(s0))
    es = (2 * T + 200 + 16 * chunk_sums(g, B, T, H)) * W24
    state, parts = s0.clone(), []
    for a, b in ((0, n0), (n0, n1)):
        o, _ = rg.linear_attention(q[:, a:b].contiguous(), k[:, a:b].contiguous(), v[:, a:b].contiguous(),
                                   g[:, a:b].contiguous(), state, state_out=state)
        parts.append(o)
    for t in range(n1, T):
        parts.append(rg.linear_attention_step(q[:, t], k[:, t], v[:, t], g[:, t].contiguous(), state)[:, None])
    check(state, rs, es * as_, "state")
    check(torch.cat(parts, 1), ro, ((es + (dk + 64) * W24 + 2.0 ** -16) * ao + U * np.abs(ro)) * (1 + U), "o")


STEP = [(1, 1, 1, 64, 64, True), (3, 2, 4, 128, 64, False), (7, 1, 5, 256, 256, True), (200, 2, 8, 64, 128, True),
        (300, 4, 8, 128, 256, False), (65, 16, 16, 64, 64, True), (1, 2, 8, 128, 128, True)]


@pytest.mark.parametrize("N,Hk,H,dk,dv,gated", STEP)
def test_linear_step(N, Hk, H, dk, dv, gated):
    rng = np.random.default_rng(N + dk)
    q, k, v, g, s0 = (x if x is None or x.dim() < 3 else x for x in linear_inputs(rng, N, 1, Hk, H, dk, dv, gated, True))
    gs = g[:, 0].contiguous() if gated else g
    out = torch.empty_like(s0)
    o = rg.linear_attention_step(q[:, 0], k[:, 0], v[:, 0], gs, s0, state_out=out)
    ro, rs, ao, as_ = sv.linear_attention(num(q), num(k), num(v), num(g), num(s0))
    check(out, rs, 16 * W24 * as_, "state")
    check(o, ro[:, 0], (16 + dk) * W24 * ao[:, 0] + U * np.abs(ro[:, 0]) * (1 + U), "o")
    mine = s0.clone()
    assert torch.equal(rg.linear_attention_step(q[:, 0], k[:, 0], v[:, 0], gs, mine), o) and torch.equal(mine, out)


def test_linear_step_forgets():
    rng = np.random.default_rng(15)
    q, k, v, _, s0 = linear_inputs(rng, 2, 1, 1, 2, 64, 64, False, True)
    g = torch.tensor([[-float("inf"), -1000.0], [0.0, -104.0]], device=DEV)
    s = s0.clone()
    rg.linear_attention_step(q[:, 0], k[:, 0], v[:, 0], g, s)
    kv = k[:, 0, 0].float()[:, None, :, None] * v[:, 0].float()[:, :, None]
    assert torch.equal(s[0], kv[0]) and torch.equal(s[1, 1], kv[1, 1])
    assert torch.allclose(s[1, 0], s0[1, 0] + kv[1, 0], rtol=1e-6, atol=1e-6)


def test_linear_scale_and_zero_state():
    rng = np.random.default_rng(16)
    q, k, v, g, _ = linear_inputs(rng, 2, 90, 1, 2, 128, 128, False, False)
    o, s = rg.linear_attention(q, k, v, g, scale=0.5)
    linear_check(o, s, q, k, v, g, None, None, 0.5)
    o0, s0 = rg.linear_attention(q, k, v, g, torch.zeros_like(s), scale=0.5)
    assert torch.equal(o, o0) and torch.equal(s, s0)


# --------------------------------------------------------------------------------------------- together
def test_prompt_in_chunks_then_tokens_over_an_e4m3_cache():
    """A prompt in two chunks through norm and rotation, its keys and values into the e4m3 cache, the second chunk's
    attention over what it reads back and its own; then token by token over the cache. Each against the oracle over
    what the cache holds."""
    rng = np.random.default_rng(21)
    B, T, n0, n1, Hq, Hkv, dh, rot, W, S, page = 3, 100, 50, 90, 6, 2, 128, 64, 40, 3, 16
    width = -(-T // page)
    qkv = normal(rng, B, T, Hq + 2 * Hkv, dh)
    q, k, v = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:]
    freq = torch.from_numpy((10000.0 ** (-np.arange(0, rot, 2) / rot)).astype(np.float32)).to(DEV)
    pos = torch.arange(T, device=DEV, dtype=I32).expand(B, T).contiguous()
    qr, kr = rg.qk_norm_rope(q, k, pos, freq)
    table = torch.from_numpy(rng.permutation(B * width).astype(np.int32)).to(DEV).view(B, width)
    u = torch.arange(T, device=DEV)
    slots = table.long()[:, u // page] * page + u % page
    cache = empty_cache(B * width, page, Hkv, dh, fill=255)
    rg.cache_quantize(kr[:, :n0].contiguous(), v[:, :n0].contiguous(), slots[:, :n0].contiguous(), *cache)
    stored = [sv.values(*sv.quantize(num(x))) for x in (kr, v)]
    # second chunk: the first one's tokens as the cache holds them, then its own
    ks, vs = (torch.empty(B, n1, Hkv, dh, dtype=BF, device=DEV) for _ in range(2))
    ks[:, n0:], vs[:, n0:] = kr[:, n0:n1], v[:, n0:n1]
    rg.rglru_cache_dequantize(*cache, table, ints([n0] * B), ks, vs)
    assert np.array_equal(num(ks[:, :n0]), stored[0][:, :n0]) and np.array_equal(num(vs[:, :n0]), stored[1][:, :n0])
    assert torch.equal(ks[:, n0:], kr[:, n0:n1])
    o = rg.local_attention(qr[:, :n1].contiguous(), ks, vs, W, S)
    args = num(qr[:, :n1]), num(ks), num(vs)
    check(o[:, n0:], ab.attention(*args, W, S)[0][:, n0:], ab.attention_bounds(*args, None, W, S)[1][:, n0:], "chunk")
    rg.cache_quantize(*(x[:, n0:n1].contiguous() for x in (kr, v, slots)), *cache)
    for t in range(n1, T):
        rg.cache_quantize(kr[:, t], v[:, t], slots[:, t].contiguous(), *cache)
        got = rg.paged_attention_e4m3(qr[:, t], *cache, table, ints([t + 1] * B), W, S)
        paged_check(got, qr[:, t], cache, table.cpu().numpy(), [t + 1] * B, W, S)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_prefix_is_attention_over_the_joined_tables(kind):
    """With a prefix of whole pages the two operators see the same keys: within both bounds of each other."""
    rng = np.random.default_rng(22)
    P, page, W, S, Hq, Hkv, dh = 96, 16, 100, 2, 8, 2, 128
    lens = [1, 17, 40, 33]
    q, cache, pools, pt, table = prefix_inputs(rng, kind, P, lens, Hq, Hkv, dh, page)
    got = run_prefix(q, cache, pt, P, table, lens, W, S)
    joined = np.concatenate([np.broadcast_to(pt, (4, len(pt))), table], 1)
    total = ints([P + n for n in lens])
    paged = rg.paged_attention_e4m3 if kind == "e4m3" else rg.paged_attention
    other = paged(q, *cache, ints(joined), total, W, S)
    o, mag, most = sv.prefix_attention(num(q), *pools, pt, P, table, lens, W, S)
    assert (np.abs(num(got) - num(other)) <= 2 * attention_bound(o, mag, most, dh, P + 40)).all()


# --------------------------------------------------------------------------------- streams and graphs
def calls(rng):
    """(name, call taking a stream, workspaces it makes) of each function, on inputs that stay as they are."""
    lens, Hq, Hkv, dh, page = [900, 1, 33], 4, 2, 128, 16
    q, cache, table = paged_inputs(rng, lens, Hq, Hkv, dh, page)
    dt, dl = ints(table), ints(lens)
    k = normal(rng, 3, Hkv, dh)
    slots = ints([5, 7, 11], torch.int64)
    pools = [t.view(torch.uint8).clone().view(t.dtype) for t in cache]
    pq, pc, _, pt, ptab = prefix_inputs(rng, "e4m3", 300, [5, 40], Hq, Hkv, dh, page)
    dpt, dpl, dptab, dpn = ints(pt), ints([300]), ints(ptab), ints([5, 40])
    lin = linear_inputs(rng, 1, 600, 1, 2, 64, 64, True, True)
    st = linear_inputs(rng, 3, 1, 1, 2, 64, 64, False, True)

    def quantize(s):
        rg.cache_quantize(k, k, slots, *pools, stream=s)
        return tuple(pools)

    return [
        ("quantize", quantize, None),
        ("dequantize", lambda s: rg.cache_dequantize(*cache, dt, dl, 64, stream=s), 0),
        ("paged_e4m3", lambda s: rg.paged_attention_e4m3(q, *cache, dt, dl, EVERY, stream=s), 1),
        ("prefix", lambda s: rg.prefix_attention(pq, pc[0], pc[1], dpt, dpl, dptab, dpn, EVERY, 0, 0.0, pc[2], pc[3],
                                                 stream=s), 1),
        ("linear", lambda s: rg.linear_attention(*lin, stream=s), 1),
        ("step", lambda s: rg.linear_attention_step(st[0][:, 0], st[1][:, 0], st[2][:, 0], st[3], st[4],
                                                    state_out=torch.empty_like(st[4]), stream=s), 0),
    ]


def tensors(out):
    return [t.view(torch.uint8) if t.dtype in (E4, E8) else t for t in (out if isinstance(out, tuple) else (out,))]


def test_given_stream_owns_what_is_made_for_it(monkeypatch):
    made, side = [], torch.cuda.Stream()
    real = rg._ext

    def pool_of(t):
        at = t.data_ptr()
        return [s["stream"] for s in torch.cuda.memory_snapshot() if s["address"] <= at < s["address"] + s["total_size"]]

    class Spy:
        def __getattr__(self, name):
            f = getattr(real, name)
            if name != "empty_bytes":
                return f

            def empty_bytes(*a):
                t = f(*a)
                made.append(pool_of(t))
                return t
            return empty_bytes

    for name, call, spaces in calls(np.random.default_rng(41)):
        want = [t.clone() for t in tensors(call(None))]
        torch.cuda.synchronize()
        monkeypatch.setattr(rg, "_ext", Spy())
        for given in (side, side.cuda_stream):
            made.clear()
            got = tensors(call(given))
            torch.cuda.synchronize()
            if spaces is not None:
                assert all(pool_of(t) == [side.cuda_stream] for t in got), name
                assert made == [[side.cuda_stream]] * spaces, name
            assert all(torch.equal(a, b) for a, b in zip(got, want)), name
        monkeypatch.setattr(rg, "_ext", real)


def test_in_a_graph():
    """Calls on the capturing stream and on one that joins it, outputs and workspaces in the graph's own memory: every
    replay against the eager result, with eager work of other sizes between them."""
    todo = calls(np.random.default_rng(43))
    want = [[t.clone() for t in tensors(call(None))] for _, call, _ in todo]
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        here = torch.cuda.current_stream()
        got = [tensors(call(None)) for _, call, _ in todo]
        side.wait_stream(here)
        again = [tensors(call(side)) for _, call, _ in todo]
        here.wait_stream(side)
    for i in range(4):
        for out in got + again:
            for t in out:
                t.fill_(3)
        other = [torch.full((100_000 * (i + 1),), float("nan"), device=DEV) for _ in range(4)]
        graph.replay()
        torch.cuda.synchronize()
        del other
        for (name, _, spaces), a, b, ref in zip(todo, got, again, want):
            if spaces is None:  # only the named slots are written
                rows = [t.flatten(0, 1)[[5, 7, 11]] for t in a]
                assert all(torch.equal(x, y.flatten(0, 1)[[5, 7, 11]]) for x, y in zip(rows, ref)), (i, name)
                continue
            assert all(torch.equal(x, y) for x, y in zip(a, ref)), (i, name)
            assert all(torch.equal(x, y) for x, y in zip(b, ref)), (i, name)


def test_lengths_that_change_between_replays():
    """Lengths, tables and the prefix's length are read on the device: a captured step follows them."""
    rng = np.random.default_rng(44)
    P, lens, Hq, Hkv, dh, page = 200, [60, 80], 4, 1, 64, 16
    q, cache, pools, pt, table = prefix_inputs(rng, "bf16", P, lens, Hq, Hkv, dh, page)
    dpl, dl, dpt, dtab = ints([P]), ints(lens), ints(pt), ints(table)
    graph = torch.cuda.CUDAGraph()
    rg.prefix_attention(q, *cache, dpt, dpl, dtab, dl, EVERY)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        o = rg.prefix_attention(q, *cache, dpt, dpl, dtab, dl, EVERY)
    for p, n in ((200, [60, 80]), (3, [1, 0]), (0, [5, 0]), (150, [0, 33])):
        dpl.copy_(ints([p]))
        dl.copy_(ints(n))
        graph.replay()
        torch.cuda.synchronize()
        ref, mag, most = sv.prefix_attention(num(q), *pools, pt, p, table, n, EVERY)
        check(o, ref, attention_bound(ref, mag, most, dh, p + max(n)), f"prefix {p}, own {n}")
