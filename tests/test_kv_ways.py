"""The choice of kernels by sizes, on the CPU: both sides of every rule."""
import pytest

import weight_only_quantization_amd as hq  # noqa: F401
from tests.kv_ways import ONCE, SHARES, TILES, WHOLE4, WHOLE8, way_of
from tests.test_kv_abi import FAKE, cache, lib  # noqa: F401
from weight_only_quantization_amd import kv_cache as kc


def way(rows, hkv, seqs, keys, prefix=0, total=None, **kw):
    """Of `seqs` sequences of `rows` query rows a KV head (one head a KV head) over at most `keys` keys."""
    a = dict(cache=cache(num_kv_heads=hkv), dtype=0, q=FAKE, total_q=rows * seqs, num_q_heads=hkv, q_token_stride=1024,
             q_head_stride=128, num_seqs=seqs, page_table=FAKE, table_stride=0, table_cols=1 << 20, seq_lens=FAKE, max_len=keys,
             causal=1, scale=0.1, prefix_table=FAKE if prefix else None, prefix_len=prefix, out=FAKE)
    a.update(kw)
    return way_of(kc.KvAttentionArgs(**a))


@pytest.mark.parametrize("call,rows,mode,splits,join", [
    ((16, 8, 16, 2048), 16, WHOLE8, 1, 0), ((16, 8, 33, 2048), 16, WHOLE4, 1, 0), ((16, 8, 32, 2048), 16, WHOLE8, 1, 0),
    ((16, 8, 16, 2049), 16, ONCE, 1, 1), ((17, 8, 16, 2049), 16, SHARES, 1, 1), ((17, 8, 16, 2048), 16, WHOLE8, 1, 0),
    ((17, 8, 17, 2048), 32, WHOLE8, 1, 0), ((17, 8, 33, 2048), 32, WHOLE4, 1, 0), ((17, 8, 17, 2049), 32, ONCE, 1, 1),
    ((33, 8, 17, 2049), 32, SHARES, 1, 1), ((64, 8, 17, 1 << 20), 32, SHARES, 1, 1),
    # 3 * 2^23 pairs of a row and a key
    ((96, 8, 8, 4096), 32, SHARES, 1, 1), ((96, 8, 8, 4097), 256, TILES, 4, 1), ((128, 8, 17, 1446), 256, TILES, 1, 0),
    ((128, 8, 17, 1445), 32, WHOLE4, 1, 0), ((65, 1, 1, (3 << 23) // 65 + 1), 256, TILES, 253, 1), ((1 << 16, 1, 1, 1), 32, WHOLE4, 1, 0),
    (((1 << 16) + 1, 1, 1, 1), 256, TILES, 1, 0)])
def test_own_keys(lib, call, rows, mode, splits, join):  # noqa: F811
    w = way(*call)
    assert w == (rows, mode, splits, 0, 0, 0, join), w


@pytest.mark.parametrize("call,want", [
    # own keys and prefix in one launch of shares: the same rows a block
    ((1, 8, 16, 200, 300), (16, ONCE, 1, 16, ONCE, 1, 1)), ((2, 8, 16, 200, 300), (16, SHARES, 1, 16, SHARES, 1, 1)),
    # apart: own keys a block a pair, the prefix in shares of 32 rows, or in tiles
    ((16, 8, 33, 200, 300), (16, WHOLE4, 1, 32, SHARES, 1, 1)), ((1, 8, 65, 1000, 1 << 16), (16, WHOLE4, 1, 256, TILES, 32, 1)),
    ((24, 8, 9, 130, 15001), (16, WHOLE8, 1, 256, TILES, 30, 1)),
    # own keys in tiles; the prefix streamed, and in tiles too
    ((128, 8, 17, 2000, 1), (256, TILES, 1, 32, SHARES, 1, 1)), ((128, 8, 17, 2000, 2048), (256, TILES, 1, 256, TILES, 3, 1)),
    ((96, 8, 8, 4097, 16), (256, TILES, 4, 32, SHARES, 1, 1))])
def test_shared(lib, call, want):  # noqa: F811
    w = way(*call)
    assert w == want, w


def test_refused_and_empty(lib):  # noqa: F811
    assert way(16, 8, 16, -1) == hq.HQQ_ERR_INVALID_ARGUMENT
    assert way(0, 8, 16, 100) == (0,) * 7
