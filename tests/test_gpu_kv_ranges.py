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
