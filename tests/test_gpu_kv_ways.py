"""Every way that a call of the attention can take (rows of a block, mode, key splits, join), each checked to be taken, against
the plain implementation in 64 bits with the bounds of tests/test_gpu_kv.py: the ones for rounded keys only where a list ran in
tiles.  Sizes that would take too many keys are reached by the bound on the lengths (a wide page table): the lengths themselves
are on the device."""

import numpy as np
import pytest

from tests import kv_plain as kp
from tests import test_gpu_kv as base
from tests import test_gpu_kv_tiles as tiles
from tests.gpu_common import say
from tests.kv_ways import ONCE, SHARES, TILES, WHOLE4, WHOLE8, record

pytestmark = pytest.mark.gpu

PAGES = (16, 32, 64, 128, 256)
FORMATS = [(*f, ("float16", "bfloat16")[i % 2], PAGES[i % 5]) for i, f in enumerate(base.FORMATS)]


@pytest.fixture
def ways(monkeypatch):
    """The calls' ways, and base.check with the bound that the last one's kernels have."""
    base.lib()
    taken = record(monkeypatch)
    plain = base.check

    def check(torch, got, lse, want, dt, tiles=False, what=""):
        plain(torch, got, lse, want, dt, tiles=256 in (taken[-1].rows, taken[-1].prefix_rows), what="%s %s" % (what, taken[-1]))

    monkeypatch.setattr(base, "check", check)
    return taken


def widen(s, keys):
    """A page table for `keys` keys a sequence: columns that lie past every length."""
    wide = np.full((len(s.lens), max(s.table.shape[1], -(-keys // s.f.page))), -1, np.int32)
    wide[:, :s.table.shape[1]] = s.table
    s.table = wide


# ------------------------------------------------------------------------------ the calls of tests/test_gpu_kv.py, with their own bound

@pytest.mark.parametrize("per,t", [(3, 5), (8, 5), (4, 33), (1, 130)])
def test_streamed_drafts(per, t, ways):
    base.test_several_tokens(per, t)
    assert ways and all(w.rows < 256 for w in ways)


@pytest.mark.parametrize("call", ["ragged", "shared ragged", "values 1e-5", "values 300", "values 9000", "values 9000, 8 bits", "values 1e-4, 8 bits",
                                  "largest", "largest, 8 bits"])
def test_streamed_ranges(call, ways):
    {"ragged": base.test_ragged_queries, "shared ragged": base.test_shared_ragged_queries,
     "values 1e-5": lambda: base.test_value_ranges(4, 1e-5), "values 300": lambda: base.test_value_ranges(4, 300.0),
     "values 9000": lambda: base.test_value_ranges(4, 9000.0), "values 9000, 8 bits": lambda: base.test_value_ranges(8, 9000.0),
     "values 1e-4, 8 bits": lambda: base.test_value_ranges(8, 1e-4), "largest": lambda: base.test_largest_values(4),
     "largest, 8 bits": lambda: base.test_largest_values(8)}[call]()
    assert ways and all(max(w.rows, w.prefix_rows) < 256 for w in ways)


@pytest.mark.parametrize("per,batch,t", [(4, 9, 1), (8, 9, 3)])
def test_streamed_prefix(per, batch, t, ways):
    base.test_shared_prefix(per, batch, t)
    assert all(w.rows == 16 for w in ways) and {w.prefix_rows for w in ways} == {0, 16}
    # one launch of shares for both lists, or the own keys a block a pair beside a prefix of other rows
    assert {w.mode for w in ways if w.prefix_rows} <= {SHARES, ONCE}


@pytest.mark.parametrize("what", ["formats", "ragged", "not finite", "splits", "drafts"])
def test_tiles_are_tiles(what, ways, monkeypatch):
    """The tests of the tiles by themselves run in tiles."""
    if what == "drafts":
        monkeypatch.setattr(base, "attend", tiles.attend)
    {"formats": lambda: tiles.test_formats(128, 4, 32, "bfloat16"), "ragged": tiles.test_ragged_queries_and_missing_pages,
     "not finite": lambda: tiles.test_rows_that_are_not_finite("float16", 16, 5000), "splits": lambda: tiles.test_key_splits(300, 8, 2701),
     "drafts": lambda: base.test_several_tokens(7, 40)}[what]()
    assert ways and all(w.rows == 256 for w in ways), ways


# ------------------------------------------------------------------------------ streams

# KV heads, sequences, tokens, heads of a KV head, bound on the keys -> rows of a block, mode
STREAMS = {"16 rows, eight waves": (2, 9, 2, 7, 0, 16, WHOLE8), "16 rows, four waves": (8, 34, 1, 3, 0, 16, WHOLE4),
           "32 rows, eight waves": (2, 65, 3, 8, 0, 32, WHOLE8), "32 rows, four waves": (4, 66, 5, 4, 0, 32, WHOLE4),
           "32 rows, two tiles": (2, 44, 9, 4, 0, 32, WHOLE8), "shares, 16 rows": (2, 70, 2, 6, 2100, 16, ONCE),
           "shares, two tiles of 16": (2, 20, 5, 5, 2100, 16, SHARES), "shares, 32 rows": (2, 66, 3, 7, 2300, 32, ONCE),
           "shares, two tiles of 32": (2, 67, 9, 5, 2300, 32, SHARES)}


def lengths(rng, seqs, most):
    return [0, 1, 15, 17, 33, 129, most][:seqs] + [int(x) for x in rng.integers(0, most // 2, size=max(0, seqs - 7))]


@pytest.mark.parametrize("d,bits,g,dtype,page", FORMATS)
@pytest.mark.parametrize("name", STREAMS)
def test_streams(name, d, bits, g, dtype, page, ways):
    hq, torch = base.lib()
    hkv, seqs, t, per, keys, rows, mode = STREAMS[name]
    say("kv streams", name, d, bits, g, dtype, page)
    rng = np.random.default_rng(seqs + d + bits + g)
    lens = lengths(rng, seqs, 280)
    s = base.Scene(hq, torch, kp.Fmt(hkv, d, bits, g, page), lens, [t] * seqs, per, dtype, seed=g + bits)
    widen(s, keys)
    o, lse = base.attend(hq, torch, s, max_len=None)
    assert ways[-1] == (rows, mode, 1, 0, 0, 0, int(keys > 0)), ways[-1]
    base.check(torch, o, lse, s.expect(), s.dt, what=name)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("name", STREAMS)
def test_ragged_streams(name, causal, ways):
    """Sequences with no, fewer and all query tokens, ones whose range is longer than the bound in between (no output of
    theirs is looked at)."""
    hq, torch = base.lib()
    hkv, seqs, t, per, keys, rows, mode = STREAMS[name]
    say("kv ragged streams", name, causal)
    rng = np.random.default_rng(seqs)
    new = [int(x) for x in rng.choice([0, 1, t], size=seqs)]
    new[:4], new[-2:] = [0, t, 0, t], [t, 0]
    new[seqs // 2] = t + 1
    f = kp.Fmt(hkv, 64 if rows == 32 else 128, 4, 32, 16 if mode in (SHARES, WHOLE8) else 64)
    s = base.Scene(hq, torch, f, lengths(rng, seqs, 200), new, per, "float16", seed=seqs)
    widen(s, keys)
    o, lse = base.attend(hq, torch, s, max_len=None, max_q=t, ragged=True, causal=causal)
    assert (ways[-1].rows, ways[-1].mode) == (rows, mode), ways[-1]
    there = np.repeat(np.array(new) <= t, new)
    base.check(torch, o[there], lse[there], [x[there] for x in s.expect(causal)], s.dt, what=name)


@pytest.mark.parametrize("d,bits,g,dtype,page", FORMATS)
def test_long_sequences(d, bits, g, dtype, page, ways):
    """Thousands of keys in fact: pairs that one, two and many blocks share, between short and empty ones."""
    hq, torch = base.lib()
    say("kv long sequences", d, bits, g, dtype, page)
    s = base.Scene(hq, torch, kp.Fmt(2, d, bits, g, page), [9000, 0, 3000, 1, 2049, 128, 0, 5000], [1] * 8, 3, dtype, seed=d + g)
    for t in (1, 2):
        if t == 2:
            s.new = [2] * 8
            s.q = kp.to((2 * np.random.default_rng(1).normal(size=(16, 6, d))).astype(np.float32), s.dt)
        o, lse = base.attend(hq, torch, s)
        assert ways[-1] == (16, ONCE, 1, 0, 0, 0, 1)
        base.check(torch, o, lse, s.expect(), s.dt, what="long")


def test_prompt_of_many_rows(ways):
    """A prompt's own attention: 2800 rows of 32 on 700 keys, and two tiles of rows that a causal rule cuts at every key."""
    hq, torch = base.lib()
    s = base.Scene(hq, torch, kp.Fmt(2, 128, 4, 64, 64), [700], [700], 4, "float16", seed=6)
    o, lse = base.attend(hq, torch, s)
    assert ways[-1] == (32, WHOLE8, 1, 0, 0, 0, 0)
    base.check(torch, o, lse, s.expect(), s.dt, what="prompt")


# ------------------------------------------------------------------------------ tiles

@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d,bits,g,dtype,page", FORMATS[::2] + FORMATS[1:4:2])
def test_unsplit_tiles(d, bits, g, dtype, page, causal, ways):
    """Tiles that write their rows themselves (136 pairs): rows of no key, queries that are not finite, lengths 0 and 1, ends
    inside a tile, two tiles of rows."""
    hq, torch = base.lib()
    say("kv unsplit tiles", d, bits, g, dtype, page, causal)
    rng = np.random.default_rng(d + g)
    t, per, lens = 35, 2, [0, 1, 34, 35, 127, 128, 129, 300, 16, 17, 255, 257, 2, 33, 64, 100, 5]
    s = base.Scene(hq, torch, kp.Fmt(8, d, bits, g, page), lens, [t] * 17, per, dtype, seed=bits)
    widen(s, tiles.WORK // (t * per * 8 * 17) + 1 + page)
    o, lse = base.attend(hq, torch, s, max_len=None, causal=causal)
    assert ways[-1] == (256, TILES, 1, 0, 0, 0, 0), ways[-1]
    want = s.expect(causal)
    base.check(torch, o, lse, want, s.dt, what="unsplit")
    bad = [(7 * t + 3, 2), (7 * t + 34, 15), (5 * t + 30, 0)]
    for i, at in enumerate(bad):
        s.q[at][5 + i] = (float("nan"), float("inf"), -float("inf"))[i]
    empty = (1, 3)                                  # of the sequence without keys
    s.q[empty][0] = float("inf")
    o2, lse2 = base.attend(hq, torch, s, max_len=None, causal=causal)
    for at in bad:
        assert torch.isnan(o2[at]).all() and torch.isnan(lse2[at]), at
        o2[at], lse2[at] = o[at], lse[at]
    assert torch.equal(o2, o) and torch.equal(lse2, lse)


def test_unsplit_ragged_tiles(ways):
    """Two tiles of rows a sequence, sequences with none, few and many query tokens; one longer than the bound."""
    hq, torch = base.lib()
    new = [70, 0, 1, 33, 70, 71, 64, 5, 70]
    s = base.Scene(hq, torch, kp.Fmt(8, 64, 8, 64, 32), [300, 40, 90, 20, 70, 71, 0, 1, 131], new, 4, "float16", seed=2)
    widen(s, 2100)
    o, lse = base.attend(hq, torch, s, max_len=None, max_q=70)
    assert ways[-1] == (256, TILES, 1, 0, 0, 0, 0), ways[-1]
    there = np.repeat(np.array(new) <= 70, new)
    base.check(torch, o[there], lse[there], [x[there] for x in s.expect()], s.dt, what="ragged tiles")


# own keys: KV heads, sequences, tokens, heads of a KV head, bound on the keys; prefix -> way
SHARED = {"own split, prefix streamed": (2, 3, 20, 4, 60000, 33, (256, TILES, 40, 16, SHARES, 1, 1)),
          "own unsplit, prefix streamed": (8, 17, 10, 8, 2400, 129, (256, TILES, 1, 32, SHARES, 1, 1)),
          "own unsplit, prefix in tiles": (8, 17, 10, 8, 2400, 2600, (256, TILES, 1, 256, TILES, 5, 1)),
          "own split, prefix in tiles": (8, 2, 65, 4, 6400, 6200, (256, TILES, 8, 256, TILES, 10, 1)),
          "both in shares of 16": (4, 40, 2, 8, 0, 70, (16, SHARES, 1, 16, SHARES, 1, 1)),
          "own 32 rows, prefix 16": (4, 45, 5, 4, 0, 70, (32, WHOLE8, 1, 16, SHARES, 1, 1)),
          "both in shares of 16, own long": (2, 70, 1, 8, 2500, 300, (16, SHARES, 1, 16, SHARES, 1, 1)),
          "own 16 rows, prefix 32": (4, 70, 2, 8, 0, 70, (16, WHOLE4, 1, 32, SHARES, 1, 1)),
          "both in shares of 32": (4, 60, 5, 4, 0, 70, (32, SHARES, 1, 32, SHARES, 1, 1)),
          "own long, prefix 32 apart": (4, 70, 2, 8, 2500, 300, (16, ONCE, 1, 32, SHARES, 1, 1))}


@pytest.mark.parametrize("name", SHARED)
@pytest.mark.parametrize("ragged", [False, True])
def test_shared(name, ragged, ways):
    hq, torch = base.lib()
    hkv, seqs, t, per, keys, prefix, way = SHARED[name]
    say("kv shared ways", name, ragged)
    rng = np.random.default_rng(seqs)
    new = [t] * seqs
    if ragged:
        new = [t] + [int(x) for x in rng.choice([0, 1, t], size=seqs - 1)]
    bits, g, dtype = (8, 32, "bfloat16") if seqs % 2 else (4, 64, "float16")
    s = base.Scene(hq, torch, kp.Fmt(hkv, 64, bits, g, 64), lengths(rng, seqs, 150), new, per, dtype, prefix=prefix, seed=seqs)
    widen(s, keys)
    o, lse = base.attend(hq, torch, s, shared=True, max_len=None, ragged=ragged)
    assert ragged or ways[-1] == way, ways[-1]
    base.check(torch, o, lse, s.expect(), s.dt, what=name)


# ------------------------------------------------------------------------------ workspaces

@pytest.mark.parametrize("name", ["shares, two tiles of 16", "shares, 32 rows"] + list(SHARED))
def test_given_workspace(name, ways):
    """A workspace of just the size, filled with NaN, with something behind it that stays: the same bits, twice."""
    hq, torch = base.lib()
    if name in SHARED:
        hkv, seqs, t, per, keys, prefix, _ = SHARED[name]
    else:
        (hkv, seqs, t, per, keys, _, _), prefix = STREAMS[name], 0
    prefix = min(prefix, 400)
    rng = np.random.default_rng(3)
    s = base.Scene(hq, torch, kp.Fmt(hkv, 128, 4, 64, 32), lengths(rng, seqs, 100), [t] * seqs, per, "float16", prefix=prefix, seed=1)
    widen(s, keys)
    o, lse = base.attend(hq, torch, s, shared=prefix > 0, max_len=None)
    assert ways[-1].join
    need = size_of(hq, ways, torch, s, prefix)
    room = torch.full((need + 4096,), 0xFF, dtype=torch.uint8, device="cuda")
    for _ in range(2):
        o2, lse2 = base.attend(hq, torch, s, shared=prefix > 0, max_len=None, workspace=room[:need])
        assert torch.equal(o2, o) and torch.equal(lse2, lse)
        assert (room[need:] == 0xFF).all()
    with pytest.raises(hq.HQQError, match="workspace"):
        base.attend(hq, torch, s, shared=prefix > 0, max_len=None, workspace=room[:need - 16])


def size_of(hq, ways, torch, s, prefix):
    """What hqq_kv_attention_workspace_bytes asks for the call."""
    from weight_only_quantization_amd import kv_cache as kc
    sizes, entry = [], kc._fast["hqq_kv_attention_workspace_bytes"]

    def call(packed):
        sizes.append(entry(packed))
        return sizes[-1]

    kc._fast["hqq_kv_attention_workspace_bytes"] = call
    try:
        base.attend(hq, torch, s, shared=prefix > 0, max_len=None)
    finally:
        kc._fast["hqq_kv_attention_workspace_bytes"] = entry
    assert sizes and sizes[-1] > 0
    return sizes[-1]


def test_bounds_past_the_call(ways):
    """Bounds on query tokens and lengths that are larger than the call itself (a program's fixed ones) are bounds too."""
    hq, torch = base.lib()
    s = base.Scene(hq, torch, kp.Fmt(2, 128, 4, 64, 32), [40, 7, 90], [3, 1, 2], 4, "float16", seed=5)
    o, lse = base.attend(hq, torch, s)
    o2, lse2 = base.attend(hq, torch, s, max_q=64, max_len=1 << 20)
    assert torch.equal(o2, o) and torch.equal(lse2, lse)


def test_graph_of_shares(ways):
    """Shares with a join in a graph, lengths changed between replays: each against the eager call."""
    hq, torch = base.lib()
    s = base.Scene(hq, torch, kp.Fmt(2, 128, 4, 64, 64), [2600, 70, 900], [1] * 3, 4, "float16", seed=8)
    t, q = torch.from_numpy(s.table).cuda(), s.q.cuda()
    lens = torch.tensor(s.lens, dtype=torch.int32, device="cuda")

    def step():
        return hq.hqq_kv_attention(s.cache, q, t, lens)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    assert ways[-1] == (16, ONCE, 1, 0, 0, 0, 1)
    for now in ([2600, 70, 900], [0, 1, 5], [128, 70, 0], [2599, 64, 899]):
        lens.copy_(torch.tensor(now, dtype=torch.int32))
        graph.replay()
        got = out.clone()
        torch.cuda.synchronize()
        assert torch.equal(got, step()), now
        torch.cuda.synchronize()
        s.lens = now
        base_want = s_expect(s, now)
        base.check(torch, got, None, base_want, s.dt, what="graph %s" % now)


def s_expect(s, lens):
    """expect() of a scene whose sequences are cut to `lens` keys."""
    whole = s.kv
    try:
        s.kv = [[tuple(x[:n] for x in part) for part in kv] for kv, n in zip(whole, lens)] + [whole[-1]]
        return s.expect()
    finally:
        s.kv = whole
