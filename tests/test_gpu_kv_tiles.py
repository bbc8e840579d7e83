"""Attention of many rows in tiles, at the sizes and values where it can go wrong.

Calls of more than 64 rows a KV head run in tiles from 3 * 2^23 pairs of a row and a key (of every KV head and sequence) on,
counted with the host's bound on the lengths.  `attend` here widens the page table with columns that lie past every length, so
that short sequences take that way too; bounds and scenes are those of tests/test_gpu_kv.py."""
import numpy as np
import pytest

from tests import kv_plain as kp
from tests import test_gpu_kv as base
from tests.gpu_common import say

pytestmark = pytest.mark.gpu

WORK = 3 << 23
plain_attend = base.attend


def attend(hq, torch, s, shared=False, **kw):
    rows = kw.get("max_q", max(s.new)) * s.per
    if rows <= 64 or shared:
        return plain_attend(hq, torch, s, shared, **kw)
    cols = WORK // (rows * len(s.lens) * s.f.hkv * s.f.page) + 1
    narrow = s.table
    s.table = np.full((len(s.lens), max(cols, narrow.shape[1])), -1, np.int32)
    s.table[:, :narrow.shape[1]] = narrow
    assert rows * len(s.lens) * s.f.hkv * s.table.shape[1] * s.f.page > WORK
    kw["max_len"] = None
    try:
        return plain_attend(hq, torch, s, **kw)
    finally:
        s.table = narrow


@pytest.fixture
def in_tiles(monkeypatch):
    monkeypatch.setattr(base, "attend", attend)


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("d,bits,g", base.FORMATS)
def test_formats(d, bits, g, dtype):
    hq, torch = base.lib()
    for per, t, page in ((5, 13, 16), (1, 270, 256)):
        say("kv tiles", d, bits, g, dtype, per, t, page)
        s = base.Scene(hq, torch, kp.Fmt(2, d, bits, g, page), [t + 140, t, 1], [t] * 3, per, dtype, seed=t + d)
        o, lse = attend(hq, torch, s)
        base.check(torch, o, lse, s.expect(), s.dt, tiles=True, what="formats")


@pytest.mark.parametrize("per,t", [(3, 22), (8, 33), (4, 65), (1, 130), (7, 40)])
def test_several_tokens(per, t, in_tiles):
    base.test_several_tokens(per, t)


@pytest.mark.parametrize("bits,vscale", [(4, 1e-5), (4, 300.0), (4, 9000.0), (8, 9000.0), (8, 1e-4)])
def test_value_ranges(bits, vscale, in_tiles):
    base.test_value_ranges(bits, vscale)


@pytest.mark.parametrize("qscale", [1e3, 6e4])
def test_scores_past_fp32_units(qscale, in_tiles):
    base.test_scores_past_fp32_units(qscale)


@pytest.mark.parametrize("bits", [4, 8])
def test_largest_values(bits, in_tiles):
    base.test_largest_values(bits)


def test_ragged_queries_and_missing_pages():
    hq, torch = base.lib()
    f = kp.Fmt(2, 128, 4, 64, 16)
    s = base.Scene(hq, torch, f, [50, 400, 0, 77, 300, 9], [1, 0, 0, 77, 20, 1], 4, "float16", seed=3, cols=40)
    o, lse = attend(hq, torch, s)
    base.check(torch, o, lse, s.expect(), s.dt, tiles=True, what="ragged")
    s = base.Scene(hq, torch, f, [330, 90, 40], [70, 70, 40], 4, "bfloat16", seed=11)
    s.table[0, 3], s.table[0, 9], s.table[1, :], s.table[2, 0] = -1, 1 << 30, -5, s.cache.num_pages
    hidden = [np.r_[48:64, 144:160], np.r_[0:90], np.r_[0:16]]
    o, lse = attend(hq, torch, s)
    base.check(torch, o, lse, s.expect(hidden=hidden), s.dt, tiles=True, what="missing pages")


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("hkv,n", [(2, 200), (16, 5000)])
def test_rows_that_are_not_finite(dtype, hkv, n):
    """A query row with NaN or an infinity is NaN where it sees a key, 0 where it sees none, and touches no other row;
    with the keys of a pair in one block and split."""
    hq, torch = base.lib()
    s = base.Scene(hq, torch, kp.Fmt(hkv, 64, 8, 32, 32), [n, 30], [80, 80], 2, dtype, seed=31)
    call = attend if hkv == 2 else plain_attend
    assert hkv == 2 or 160 * 2 * hkv * n > WORK
    o, lse = call(hq, torch, s)
    s.q[20, 1], s.q[60, 0, 7], s.q[61, 3, 63], s.q[90, 2] = float("nan"), float("inf"), float("nan"), float("nan")
    o2, lse2 = call(hq, torch, s)
    for at in ((20, 1), (60, 0), (61, 3)):
        assert torch.isnan(o2[at]).all() and torch.isnan(lse2[at]), at
        o2[at], lse2[at] = o[at], lse[at]
    assert not o2[90, 2].any()    # before the sequence's first key
    assert torch.equal(o2, o) and torch.equal(lse2, lse)


@pytest.mark.parametrize("t,per,n", [(300, 8, 2701), (97, 16, 4130)])
def test_key_splits(t, per, n):
    """Sequences long enough by themselves; their keys are split among the blocks and joined."""
    hq, torch = base.lib()
    s = base.Scene(hq, torch, kp.Fmt(4, 128, 4, 64, 64), [n], [t], per, "float16", seed=n)
    assert t * per * 4 * n > WORK
    o, lse = plain_attend(hq, torch, s)
    base.check(torch, o, lse, s.expect(), s.dt, tiles=True, what="splits")
    o2, _ = plain_attend(hq, torch, s)
    assert torch.equal(o, o2)


def test_shared_prefix():
    """A prefix in tiles, the own keys streamed."""
    hq, torch = base.lib()
    s = base.Scene(hq, torch, kp.Fmt(8, 64, 4, 32, 64), [7, 0, 130, 55, 3, 64, 1, 90, 20], [3] * 9, 8, "bfloat16", prefix=15001, seed=9)
    assert 27 * 8 * 8 * 15001 > WORK
    o, lse = plain_attend(hq, torch, s, shared=True)
    base.check(torch, o, lse, s.expect(), s.dt, tiles=True, what="shared")


@pytest.mark.parametrize("rows_of", [64, 65])
def test_both_sides_of_the_rule(rows_of):
    """One row more or less, and a bound on the lengths just below and above the rule: the same outputs to rounding."""
    hq, torch = base.lib()
    s = base.Scene(hq, torch, kp.Fmt(1, 128, 4, 64, 256), [500], [rows_of], 1, "float16", seed=4)
    want = s.expect()
    narrow = s.table
    for cols in (2, WORK // (256 * 65), WORK // (256 * 65) + 1):
        s.table = np.full((1, cols), -1, np.int32)
        s.table[:, :2] = narrow
        o, lse = plain_attend(hq, torch, s, max_len=None)
        base.check(torch, o, lse, want, s.dt, tiles=True, what="rule, %d columns" % cols)
