"""The quantised cache and its attention at the ends of the number ranges, where streamed rows and tiles have to agree
with the definition and with each other.  Bounds are those of tests/test_gpu_kv.py (u half a unit of the output type, A the
sum of weights times (|floor| + code * step)); where a case needs others they are derived in it."""
import math

import numpy as np
import pytest

from tests import kv_plain as kp
from tests import test_gpu_kv as base
from tests.gpu_common import say

pytestmark = pytest.mark.gpu

TILE_ROWS = 80          # more than 64 rows ...
TILE_WORK = 3 << 23     # ... and more pairs of a row and a key than this, by the bound on the lengths, run in tiles


def one_head(hq, torch, bits, k, v, page=32, g=64, dtype="float16"):
    """Cache with one head and one sequence of the given keys and values, pages in order."""
    f = kp.Fmt(1, k.shape[-1], bits, g, page)
    n = len(k)
    cache = base.make_cache(hq, torch, f, -(-n // page))
    k, v = (kp.to(x.reshape(n, 1, -1), getattr(torch, dtype)) for x in (k, v))
    hq.hqq_kv_write(cache, k.cuda(), v.cuda(), torch.arange(n, device="cuda"))
    kept = [kp.stands_for(*kp.quantise(kp.as_f32(x), bits, g))[:, 0].astype(np.float64) for x in (k, v)]
    return cache, kept


def attend(hq, torch, cache, q, lens, tiles=False, **kw):
    """Every sequence on the same pages; with `tiles` the table is widened until the call runs in tiles."""
    cols = cache.num_pages
    if tiles:
        rows = q.shape[0] // len(lens) * q.shape[1] // cache.num_kv_heads
        assert rows > 64
        cols = max(cols, TILE_WORK // (rows * len(lens) * cache.num_kv_heads * cache.page_size) + 1)
    table = torch.full((1, cols), -1, dtype=torch.int32, device="cuda")
    table[0, :cache.num_pages] = torch.arange(cache.num_pages, dtype=torch.int32)
    return hq.hqq_kv_attention(cache, q, table.expand(len(lens), -1), torch.tensor(lens, dtype=torch.int32, device="cuda"),
                               return_lse=True, **kw)


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("d,bits,g", base.FORMATS)
def test_values_past_the_largest_half(d, bits, g, dtype):
    """Groups that reach +-65504 (by infinities too), whose top code may stand for more: rows that see one such key alone,
    streamed and in tiles, are finite, in fp16 held to 65504; the read-back and the echo are the rounded sum."""
    hq, torch = base.lib()
    dt = getattr(torch, dtype)
    say("kv largest values", d, bits, g, dtype)
    x = np.zeros((4, 1, d), np.float32)
    x[0, 0, ::2], x[0, 0, 1::2] = 65504, -65504
    x[1, 0, ::2], x[1, 0, 1::2] = np.inf, -np.inf
    x[2, 0, ::2] = 65504                            # from 0
    x[3, 0, ::2], x[3, 0, 1::2] = 65504, -60000
    f = kp.Fmt(1, d, bits, g, 16)
    xs = kp.to(x, dt)
    val = kp.stands_for(*kp.quantise(kp.as_f32(xs), bits, g))
    assert (val > 65519).any()
    half = dtype == "float16"
    u = 2.0 ** -11 if half else 2.0 ** -8
    for key in range(4):
        cache = base.make_cache(hq, torch, f, 1)
        at = torch.zeros(1, dtype=torch.int64, device="cuda")
        one = xs[key:key + 1].cuda()
        ke, ve = hq.hqq_kv_write(cache, one, one, at, echo=True)
        kr, vr = hq.hqq_kv_read(cache, at, dtype=dt)
        want = kp.to(val[key:key + 1], torch.float32).to(dt)
        for got in (ke, ve, kr, vr):
            assert torch.equal(got.cpu(), want)
        for t, tiles in ((1, False), (TILE_ROWS, True)):
            q = torch.zeros(t, 1, d, dtype=dt, device="cuda")
            o, lse = attend(hq, torch, cache, q, [1], tiles, causal=False)
            o = o.double().cpu().numpy()
            assert np.isfinite(o).all() and (not half or np.abs(o).max() <= 65504), (key, tiles)
            held = np.clip(val[key, 0].astype(np.float64), -65566, 65504 if half or tiles else 65566)
            # u |o| + 2^-9 A, A at most 65504 + 131072
            assert (np.abs(o - held) <= u * 65566 + 2.0 ** -9 * 196608).all(), (key, tiles)
            assert np.abs(lse.cpu().numpy()).max() == 0


@pytest.mark.parametrize("where", ["low weight", "hidden", "other group", "other group, small floors", "huge, low weight",
                                   "huge, other group"])
@pytest.mark.parametrize("seqs", [1, 130])
@pytest.mark.parametrize("d,bits,g,dtype", [(128, 4, 64, "float16"), (128, 8, 32, "bfloat16"), (64, 4, 32, "bfloat16"), (64, 8, 32, "float16"),
                                            (128, 8, 64, "float16"), (128, 4, 32, "float16")])
def test_small_values_next_to_large_ones(d, bits, g, dtype, seqs, where):
    """Steps of 2 to 5000 next to steps of 1e-4 and less: in other keys (of low weight, or hidden from some rows) and in
    another group of the same keys.  24 rows take two tiles of 16, or where that is more blocks than the GPU runs at
    once, one of 32 (130 sequences)."""
    hq, torch = base.lib()
    say("kv mixed values", d, bits, g, dtype, seqs, where)
    rng = np.random.default_rng(d + bits + seqs)
    n, t, per = 45, 3, 8
    k, v = (rng.normal(size=(n, d)).astype(np.float32) for _ in "kv")
    v *= 1e-3
    large = 1e7 if where.startswith("huge") else 1e6     # (steps of 32 and more in 8 bits too)
    if where.endswith("low weight") or where == "hidden":
        at = n - 1 if where == "hidden" else 7
        v[at] *= large
        if where != "hidden":
            k[at] = -8
    else:
        v[:, :g] *= large
        if where.endswith("floors"):
            v[:, g:] = np.abs(v[:, g:]) + 3e-4
    cache, (ks, vs) = one_head(hq, torch, bits, k, v, g=g, dtype=dtype)
    steps = kp.quantise(kp.as_f32(kp.to(v, getattr(torch, dtype)))[:, None], bits, g)[1]
    assert steps.max() > (32 if large > 1e6 else 2) and steps.min() < 1e-3
    q = kp.to((1 + 0.5 * rng.normal(size=(t, per, d))).astype(np.float32), getattr(torch, dtype))
    o, lse = attend(hq, torch, cache, q.cuda().repeat(seqs, 1, 1), [n] * seqs)
    see = np.arange(n)[None] <= (n - t + np.arange(t))[:, None]
    code, step, floor = kp.quantise(kp.as_f32(kp.to(v, getattr(torch, dtype)))[:, None], bits, g)
    mags = kp.stands_for(code, step, np.abs(floor)).astype(np.float64)
    args = (kp.as_f32(q).astype(np.float64), ks[:, None])
    want, wl, _, _ = kp.attend(*args, vs[:, None], see, d ** -0.5)
    _, _, mag, _ = kp.attend(*args, mags, see, d ** -0.5)
    u = 2.0 ** -11 if dtype == "float16" else 2.0 ** -8
    got = o.double().cpu().numpy().reshape(seqs, t, per, d)
    err = np.abs(got - want) / (u * np.abs(want) + 2.0 ** -9 * mag + 1e-7)
    assert err.max() <= 1, (err.max(), np.unravel_index(err.argmax(), err.shape))


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("what,seqs,t,per,n", [("a block a pair", 1, 1, 1, 1024), ("rows of 32", 130, 3, 8, 1024),
                                               ("shares", 300, 1, 1, 5120), ("shares of rows of 32", 130, 3, 8, 5120),
                                               ("tiles, keys split", 2, 80, 16, 16384), ("tiles", 136, 80, 1, 5120)])
def test_flat_tail_under_one_key(what, seqs, t, per, n, bits):
    """One key whose weight is 2^25 times each other one's, and whose value is 0: the output is the others' part alone, and
    A with it, so every one of them has to be there to 2^-9."""
    hq, torch = base.lib()
    say("kv flat tail", what, bits)
    rng = np.random.default_rng(n + bits)
    d, page = 64, 256
    k = np.zeros((2 * page, d), np.float32)
    v = (30 + 9 * rng.normal(size=(2 * page, d))).astype(np.float32)
    k[5], v[5] = 2.175, 0               # score 17.4 for queries of ones
    cache, (ks, vs) = one_head(hq, torch, bits, k, v, page=page)
    order = np.r_[0, np.ones(n // page - 1, np.int64)]
    rows = t * per
    cols = max(len(order), TILE_WORK // (rows * seqs * page) + 1 if rows > 64 else 0)
    table = torch.full((1, cols), -1, dtype=torch.int32)
    table[0, :len(order)] = torch.from_numpy(order)
    q = torch.ones(seqs * t, per, d, dtype=torch.float16, device="cuda")
    o, lse = hq.hqq_kv_attention(cache, q, table.cuda().expand(seqs, -1), torch.full((seqs,), n, dtype=torch.int32, device="cuda"),
                                 causal=False, return_lse=True)
    at = (order[:, None] * page + np.arange(page)).reshape(-1)
    see, one = np.ones((1, n), bool), np.ones((1, 1, d))
    code, step, floor = kp.quantise(kp.as_f32(kp.to(v, torch.float16))[:, None], bits, 64)
    mags = kp.stands_for(code, step, np.abs(floor)).astype(np.float64)
    want, wl, _, _ = kp.attend(one, ks[at][:, None], vs[at][:, None], see, d ** -0.5)
    _, _, mag, _ = kp.attend(one, ks[at][:, None], mags[at], see, d ** -0.5)
    err = np.abs(o.double().cpu().numpy() - want) / (2.0 ** -11 * np.abs(want) + 2.0 ** -9 * mag + 1e-7)
    assert err.max() <= 1, err.max()
    assert np.abs(lse.double().cpu().numpy() - wl).max() <= 1e-5 * 20


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("seqs", [1, 130])
def test_streamed_rows_that_are_not_finite(seqs, bits, dtype):
    """A streamed query row with NaN or an infinity of either sign is NaN where it sees a key, 0 where it sees none, and touches no
    other row: keys of either sign in the channel, with codes 0 and the largest."""
    hq, torch = base.lib()
    say("kv streamed infinities", seqs, bits, dtype)
    rng = np.random.default_rng(5)
    n, t, per, d = 3, 4, 8, 64
    k, v = (rng.normal(size=(n, d)).astype(np.float32) for _ in "kv")
    k[:, :32] = 2 + rng.uniform(size=(n, 32))       # floors and codes of one sign: every product with an infinity is infinite
    k[:, 7] = 3.5
    cache, _ = one_head(hq, torch, bits, k, v, g=32, dtype=dtype)
    q = kp.to(rng.normal(size=(t, per, d)).astype(np.float32), getattr(torch, dtype)).cuda().repeat(seqs, 1, 1)
    o, lse = attend(hq, torch, cache, q, [n] * seqs)
    odd = q.clone()
    for head, channel, x in ((0, 7, -math.inf), (1, 7, math.inf), (2, 7, math.nan), (3, 50, -math.inf), (4, 50, math.inf)):
        odd[t - 1::t, head, channel] = x
        odd[0::t, head, channel] = x                # (before the sequence's first key)
    o2, lse2 = attend(hq, torch, cache, odd, [n] * seqs)
    assert torch.isnan(o2[t - 1::t, :5]).all() and torch.isnan(lse2[t - 1::t, :5]).all()
    assert not o2[0::t].any() and (lse2[0::t] == -math.inf).all()
    for x, y in ((o2, o), (lse2, lse)):
        x[t - 1::t, :5] = y[t - 1::t, :5]
        assert torch.equal(x, y)


@pytest.mark.parametrize("scale_of_others", [1e-2, 8.0, 3e4])
@pytest.mark.parametrize("what,seqs,t,per", [("rows of 16", 1, 1, 8), ("rows of 32", 130, 3, 8), ("tiles", 2, 30, 8)])
def test_rows_do_not_depend_on_their_neighbours(what, seqs, t, per, scale_of_others):
    """Other queries in half of the rows (flat, peaked, or with scores past 2^20): the other half keeps its bits."""
    hq, torch = base.lib()
    say("kv neighbours", what, scale_of_others)
    rng = np.random.default_rng(9)
    n, d = 400, 128
    k, v = (rng.normal(size=(n, d)).astype(np.float32) for _ in "kv")
    cache, _ = one_head(hq, torch, 4, k * 30, v)
    q = kp.to((0.05 * rng.normal(size=(seqs * t, per, d))).astype(np.float32), torch.float16).cuda()
    o, lse = attend(hq, torch, cache, q, [n] * seqs, tiles=what == "tiles")
    odd = q.clone()
    odd[:, 1::2] = kp.to((scale_of_others * rng.normal(size=(seqs * t, per // 2, d))).astype(np.float32), torch.float16).cuda()
    o2, lse2 = attend(hq, torch, cache, odd, [n] * seqs, tiles=what == "tiles")
    finite = torch.isfinite(odd).all(-1)            # (the largest scale has infinite queries among them)
    assert torch.equal(torch.isfinite(o2).all(-1), finite) and torch.equal(torch.isnan(o2).all(-1), ~finite)
    assert not torch.equal(o2, o)
    assert torch.equal(o2[:, ::2], o[:, ::2]) and torch.equal(lse2[:, ::2], lse[:, ::2])
