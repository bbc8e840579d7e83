"""Attention for drafted trees against the plain implementation in 64 bits, with the bounds of tests/test_gpu_kv.py (the ones for rounded keys
where the call ran in tiles), and the trees' plans against their definition."""
import numpy as np
import pytest

from tests import kv_plain as kp
from tests import test_gpu_kv as base
from tests.gpu_common import say
from tests.kv_ways import ONCE, SHARES, WHOLE4, WHOLE8
from tests.test_gpu_kv_ways import widen

pytestmark = pytest.mark.gpu


def random_parents(rng, new):
    """Parents of each sequence's drafts: any earlier draft, or none."""
    return np.concatenate([[rng.integers(-1, t) if t else -1 for t in range(n)] for n in new] + [[]]).astype(np.int32)


def sees_of(parents, new):
    """Per sequence the drafts [T, T] that each sees: itself and its ancestors."""
    out, at = [], 0
    for n in new:
        m = np.zeros((n, n), bool)
        for t in range(n):
            p = parents[at + t]
            if 0 <= p < t:
                m[t] = m[p]
            m[t, t] = True
        out.append(m)
        at += n
    return out


def words_of(sees, words):
    """Masks as int64 [total, words]."""
    rows = []
    for m in sees:
        for t in range(len(m)):
            w = [0] * words
            for j in np.flatnonzero(m[t]).tolist():
                w[j // 64] |= 1 << (j % 64)
            rows.append([x - (1 << 64) if x >> 63 else x for x in w])
    return np.array(rows, np.int64).reshape(-1, words)


def expect(s, sees, hidden=None):
    """out, lse, sizes as base.Scene.expect, for masks of the drafts."""
    outs, at = [], 0
    pk, _, pv, pa = s.dense(len(s.lens))
    for b, (n, t) in enumerate(zip(s.lens, s.new)):
        q = kp.as_f32(s.q[at:at + t]).astype(np.float64)
        at += t
        k, _, v, a = s.dense(b)
        see = np.ones((t, n), bool)
        for j in range(t):                      # draft j is key n - t + j
            if n - t + j >= 0:
                see[:, n - t + j] = sees[b][:, j]
        if hidden is not None:
            see[:, hidden[b]] = False
        see = np.concatenate([np.ones((t, s.prefix), bool), see], 1)
        k, v, a = (np.concatenate(x) for x in ((pk, k), (pv, v), (pa, a)))
        o, lse, _, terms = kp.attend(q, k, v, see, s.scale)
        _, _, mag, _ = kp.attend(q, k, a, see, s.scale)
        outs.append((o, lse, mag, terms))
    return [np.concatenate(x) for x in zip(*outs)]


def args_of(torch, s, ragged=None):
    t, lens = torch.from_numpy(s.table).cuda(), torch.tensor(s.lens, dtype=torch.int32, device="cuda")
    ragged = len(set(s.new)) > 1 if ragged is None else ragged
    return t, lens, dict(cu_q=base.cu(torch, s.new), max_q=max(s.new)) if ragged else {}


def attend(hq, torch, s, mask, ragged=None, **kw):
    t, lens, more = args_of(torch, s, ragged)
    kw.setdefault("max_len", max(s.lens))
    if s.prefix:
        kw.update(prefix_table=torch.from_numpy(s.prefix_table).cuda(), prefix_len=s.prefix)
    return hq.hqq_kv_attention_tree(s.cache, s.q.cuda(), torch.from_numpy(mask).cuda(), t, lens, scale=s.scale, return_lse=True, **{**more, **kw})


@pytest.fixture
def ways(monkeypatch):
    """The ways (rows, mode, splits, prefix's, join) of the calls of hqq_kv_attention_tree."""
    import ctypes

    from weight_only_quantization_amd import kv_cache as kc
    hq, _ = base.lib()
    fn = hq.load().hqq_kv_attention_tree_way
    fn.argtypes, fn.restype = [ctypes.c_char_p, ctypes.c_int32 * 7], ctypes.c_int
    taken = []
    entry = kc._fast["hqq_kv_attention_tree"]

    def call(packed):
        out = (ctypes.c_int32 * 7)()
        assert fn(packed, out) == 0
        taken.append(tuple(out))
        return entry(packed)

    monkeypatch.setitem(kc._fast, "hqq_kv_attention_tree", call)
    return taken


def run(hq, torch, s, ways, sees, hidden=None, what="", words=None, mask=None, **kw):
    words = words or (max(s.new) + 63) // 64 or 1
    o, lse = attend(hq, torch, s, words_of(sees, words) if mask is None else mask, **kw)
    w = ways[-1]
    base.check(torch, o, lse, expect(s, sees, hidden), s.dt, tiles=max(w[0], w[3]) >= 128, what="%s %s" % (what, w))
    return o, lse


# ------------------------------------------------------------------------------ plans

@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_plan(page):
    hq, torch = base.lib()
    rng = np.random.default_rng(page)
    for new, words in (([1, 5, 0, 64, 13], 1), ([65, 3], 2), ([7] * 9, 1), ([200, 129, 1], 4), ([4096], 64)):
        say("plan", page, new)
        total, ragged = sum(new), len(set(new)) > 1
        lens = [n + int(rng.integers(0, 400)) for n in new]
        lens[-1] = max(0, new[-1] - 2)                                # shorter than its drafts
        cols = -(-max(lens) // page) + 1
        table = rng.permutation(len(new) * cols).reshape(len(new), cols).astype(np.int32)
        table[0, cols - 1] = -1
        parents = random_parents(rng, new)
        if total > 20:
            parents[17] = 5000                                        # no draft in front of it: none
        args = [torch.from_numpy(x).cuda() for x in (parents, table)] + [torch.tensor(lens, dtype=torch.int32, device="cuda")]
        kw = dict(cu_q=base.cu(torch, new), max_q=max(new)) if ragged else {}
        mask, pos, slots = (x.cpu().numpy() for x in hq.hqq_kv_tree_plan(*args, page, **kw))
        sees = sees_of(parents, new)
        assert np.array_equal(mask, words_of(sees, words))
        at = 0
        for b, n in enumerate(new):
            begin = lens[b] - n
            depth = sees[b].sum(1) - 1
            assert np.array_equal(pos[at:at + n], begin + depth)
            for t in range(n):
                p = begin + t
                want = -1 if p < 0 or table[b, p // page] < 0 else int(table[b, p // page]) * page + p % page
                assert slots[at + t] == want
            at += n


def test_plan_edges():
    """No drafts; tokens of no sequence and of one whose range leaves the tensor are left as they are; wide masks; table strides."""
    hq, torch = base.lib()
    i32 = dict(dtype=torch.int32, device="cuda")
    table, lens = torch.arange(12, **i32).view(2, 6), torch.tensor([70, 9], **i32)
    mask, pos, slots = hq.hqq_kv_tree_plan(torch.zeros(0, **i32), table, lens, 16)
    assert mask.shape == (0, 1) and pos.shape == (0,) and slots.shape == (0,)
    from weight_only_quantization_amd import kv_pages as pages
    parents = torch.tensor([-1, 0, 0, -1, 0, 1], **i32)
    cu = torch.tensor([1, 4, 9], **i32)
    full = dict(dtype=torch.int64, device="cuda")
    out = [torch.full((6, 3), 77, **full), torch.full((6,), 77, **full), torch.full((6,), 77, **full)]
    a = pages.KvTreePlanArgs(parents.data_ptr(), 6, 2, cu.data_ptr(), 5, table.data_ptr(), 6, 6, lens.data_ptr(), 16, out[0].data_ptr(), 3,
                             out[1].data_ptr(), out[2].data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert hq.load().hqq_kv_tree_plan(a) == 0
    assert out[0][:, 0].tolist() == [77, 1, 3, 4, 77, 77] and not out[0][1:4, 1:].any() and (out[0][4:] == 77).all()
    assert out[1].tolist() == [77, 67, 68, 67, 77, 77] and out[2].tolist() == [77, 4 * 16 + 3, 4 * 16 + 4, 4 * 16 + 5, 77, 77]
    wide = torch.full((2, 20), -1, **i32)
    wide[:, 3:9] = table
    x, y = hq.hqq_kv_tree_plan(parents, wide[:, 3:9], lens, 16), hq.hqq_kv_tree_plan(parents, table, lens, 16)
    assert all(torch.equal(i, j) for i, j in zip(x, y))


# ------------------------------------------------------------------------------ attention

@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("d,bits,g", base.FORMATS)
def test_trees(d, bits, g, dtype, ways):
    """Ragged trees, sequences of nothing but drafts and shorter than them, drafts across pages, in blocks of 16 and 32 rows."""
    hq, torch = base.lib()
    for per, page, new in ((1, 16, [5, 1, 13, 3]), (4, 64, [26, 26, 2, 7]), (7, 256, [4, 0, 33, 1])):
        say("trees", d, bits, g, dtype, per, page)
        rng = np.random.default_rng(d + bits + per)
        f = kp.Fmt(2, d, bits, g, page)
        s = base.Scene(hq, torch, f, [new[0] + 131, new[1], max(0, new[2] - 2), 700], new, per, dtype, seed=per + d)
        run(hq, torch, s, ways, sees_of(random_parents(rng, new), new), what="trees")
        assert ways[-1][0] < 128


@pytest.mark.parametrize("d,bits,g", base.FORMATS)
@pytest.mark.parametrize("rows", [128, 256])
def test_shares_of_tiles(rows, d, bits, g, ways):
    """Tiles of 128 and of 256 rows in shares: pairs cut and whole, several row tiles, ragged drafts, a partly filled last tile; reached by
    the bound on the lengths (a wide page table), which are on the device."""
    hq, torch = base.lib()
    dtype, page = (("float16", 32), ("bfloat16", 16))[(bits == 8) ^ (g == 32)]
    for per, new, lens in ((5, [25, 3, 17], [700, 140, 17]), (9, [40, 31, 1], [300, 1100, 0]), (3, [130, 0, 43], [131, 500, 41])):
        per, new = (per, new) if rows == 256 or per < 9 else (4, [32, 9, 28])
        if (max(new) * per > 128) != (rows == 256):
            continue
        say("shares", rows, d, bits, g, per, new)
        rng = np.random.default_rng(d + bits + per)
        f = kp.Fmt(2, d, bits, g, page)
        s = base.Scene(hq, torch, f, lens, new, per, dtype, seed=per + d)
        widen(s, 1 << 20)
        run(hq, torch, s, ways, sees_of(random_parents(rng, new), new), what="shares", max_len=1 << 20)
        assert ways[-1][:2] == (rows, SHARES)


@pytest.mark.parametrize("per,t,lens,bound,want", [
    (1, 16, [40, 300, 16], 2048, (16, WHOLE8)), (1, 16, [40, 300, 16], 4096, (16, ONCE)), (4, 8, [40, 300, 16] * 44, 2048, (32, WHOLE4)),
    (4, 8, [40, 300, 16] * 50, 4096, (32, ONCE)), (9, 5, [200, 77, 500], 4096, (16, SHARES)), (4, 30, [30, 222, 900] * 13, 900, (32, WHOLE4)),
    (4, 32, [200, 900, 33], 1 << 20, (128, SHARES)), (8, 32, [200, 900, 33], 1 << 20, (256, SHARES))])
def test_ways(per, t, lens, bound, want, ways):
    """Every way that a call can take."""
    hq, torch = base.lib()
    for d, bits, g, dtype, page in ((128, 4, 64, "float16", 64), (64, 8, 32, "bfloat16", 16)):
        say("ways", per, t, len(lens), bound, d)
        f = kp.Fmt(2, d, bits, g, page)
        new = [t] * len(lens)
        s = base.Scene(hq, torch, f, lens, new, per, dtype, seed=per + t)
        widen(s, bound)
        sees = sees_of(random_parents(np.random.default_rng(t), new), new)
        o, _ = run(hq, torch, s, ways, sees, what="ways", max_len=bound)
        assert ways[-1][:2] == want
        again, _ = attend(hq, torch, s, words_of(sees, 1), max_len=bound)
        assert torch.equal(o, again)


@pytest.mark.parametrize("way", ["streamed", "shares"])
def test_any_mask(way, ways):
    """Masks that are no trees: empty rows, later drafts, bits past the drafts, rows that see nothing at all; masks of several words, for
    drafts of more than 64 and more than 128 tokens."""
    hq, torch = base.lib()
    rng = np.random.default_rng(17)
    for d, bits, g, dtype in ((128, 4, 64, "float16"), (64, 4, 32, "bfloat16")):
        for t, lens, words in ((7, [7, 300, 5], 1), (40, [40, 97, 38], 3), (70, [70, 333, 9], 2), (150, [150, 400, 149], 3)):
            say("any mask", way, d, t)
            per = 4 if way == "streamed" else -(-129 // t) if t < 100 else 1
            f = kp.Fmt(2, d, bits, g, 32)
            s = base.Scene(hq, torch, f, lens, [t] * 3, per, dtype, seed=t)
            sees = [rng.random((t, t)) < p for p in (0.3, 0.03, 0.5)]
            sees[0][:3] = False                                       # with no key in front of them: nothing
            mask = words_of(sees, words)
            past = words_of([np.concatenate([np.zeros((t, t), bool), rng.random((t, 64 * words - t)) < 0.5], 1) for _ in range(3)], words)
            kw = dict(max_len=max(lens))
            if way == "shares":
                widen(s, 1 << 20)
                kw = dict(max_len=1 << 20)
            run(hq, torch, s, ways, sees, what="any", mask=mask | past, **kw)
            assert (ways[-1][0] >= 128) == (way == "shares"), ways[-1]


def test_chain_is_causal(ways):
    """A chain of drafts sees what causal attention sees: the same bits where the rows are streamed."""
    hq, torch = base.lib()
    f = kp.Fmt(2, 128, 4, 64, 64)
    s = base.Scene(hq, torch, f, [900, 5, 33], [5] * 3, 4, "float16", seed=2)
    chain = [np.tril(np.ones((5, 5), bool))] * 3
    o, lse = attend(hq, torch, s, words_of(chain, 1))
    a, b = base.attend(hq, torch, s)
    assert torch.equal(o, a) and torch.equal(lse, b)


@pytest.mark.parametrize("rows", [16, 32, 128, 256])
def test_missing_pages_and_unwritten_memory(rows, ways):
    """Pages outside the cache mask their tokens, drafts' pages too; lengths beyond the table; memory that was never written is NaN."""
    hq, torch = base.lib()
    per, t = {16: (2, 8), 32: (4, 26), 128: (4, 26), 256: (8, 26)}[rows]
    f = kp.Fmt(2, 128, 8, 128, 16)
    new = [t] * 3
    s = base.Scene(hq, torch, f, [200, 64, 40], new, per, "float16", seed=11)
    s.table[0, 3], s.table[0, 12], s.table[1, :], s.table[2, 0] = -1, 1 << 30, -5, s.cache.num_pages
    hidden = [np.r_[48:64, 192:200], np.r_[0:64], np.r_[0:16]]
    sees = sees_of(random_parents(np.random.default_rng(1), new), new)
    kw = dict(max_len=200)
    if rows >= 128:
        widen(s, 1 << 21)
        kw = dict(max_len=1 << 21)
    run(hq, torch, s, ways, sees, hidden=hidden, what="missing", **kw)
    if rows != 32:
        assert ways[-1][0] == rows
    cut = base.Scene(hq, torch, f, [96, 64, 40], new, per, "float16", seed=12)
    mask = words_of(sees, 1)
    want = expect(cut, sees)
    cut.lens = [1000, 64, 40]                                         # the table holds 96
    o, lse = attend(hq, torch, cut, mask, max_len=None)
    base.check(torch, o, lse, want, cut.dt, tiles=ways[-1][0] >= 128, what="length beyond the table")
    cut.lens = [-3, 64, 40]
    o, lse = attend(hq, torch, cut, mask, max_len=64)
    assert not o[:t].any() and torch.isinf(lse[:t]).all()


@pytest.mark.parametrize("case", ["streamed", "apart", "shares", "prefix in tiles"])
def test_prefix(case, ways):
    """With a shared prefix: streamed in one launch, in two, own keys in shares of tiles, the prefix in tiles."""
    hq, torch = base.lib()
    per, t, batch, prefix, bound = {"streamed": (1, 5, 3, 40, None), "apart": (4, 4, 130, 300, None), "shares": (5, 20, 3, 77, 1 << 20),
                                    "prefix in tiles": (4, 33, 5, 20000, 1 << 20)}[case]
    for d, bits, g, dtype in ((128, 4, 64, "float16"), (64, 8, 64, "bfloat16")):
        say("prefix", case, d)
        f = kp.Fmt(2, d, bits, g, 16)
        lens = [max(t, (37 * i) % 190) for i in range(batch)]
        new = [t] * batch
        s = base.Scene(hq, torch, f, lens, new, per, dtype, prefix=prefix, seed=prefix + per)
        if bound:
            widen(s, bound)
        sees = sees_of(random_parents(np.random.default_rng(5), new), new)
        run(hq, torch, s, ways, sees, what=case, max_len=bound or max(lens))
        w = ways[-1]
        assert {"streamed": w[0] == w[3] == 16, "apart": w[0] != w[3] and w[3] <= 32, "shares": w[0] == 128 and w[3] <= 32,
                "prefix in tiles": w[0] == 256 and w[3] == 256}[case], w


def test_queries_not_finite(ways):
    """A query row of NaN or with an infinity touches no other row, in every kernel."""
    hq, torch = base.lib()
    for per, t, bound in ((2, 8, 300), (8, 4, 300), (4, 32, 1 << 20), (8, 32, 1 << 20)):
        f = kp.Fmt(2, 128, 4, 64, 32)
        new = [t] * 2
        s = base.Scene(hq, torch, f, [300, t + 1], new, per, "bfloat16", seed=per)
        widen(s, bound)
        mask = words_of(sees_of(random_parents(np.random.default_rng(8), new), new), 1)
        o, _ = attend(hq, torch, s, mask, max_len=bound)
        s.q[1, 0], s.q[t + 2, 1, 5] = float("nan"), float("-inf")
        o2, _ = attend(hq, torch, s, mask, max_len=bound)
        assert torch.isnan(o2[1, 0]).all() and torch.isnan(o2[t + 2, 1]).all()
        o2[1, 0], o2[t + 2, 1] = o[1, 0], o[t + 2, 1]
        assert torch.equal(o2, o)


def test_many_sequences(ways):
    """More sequences than a scan of lengths takes at once, some without drafts, streamed and in shares."""
    hq, torch = base.lib()
    rng = np.random.default_rng(23)
    f = kp.Fmt(1, 64, 4, 64, 16)
    new = [int(x) for x in rng.integers(0, 20, 150)]
    lens = [n + int(rng.integers(0, 60)) for n in new]
    s = base.Scene(hq, torch, f, lens, new, 6, "float16", seed=4)
    sees = sees_of(random_parents(rng, new), new)
    run(hq, torch, s, ways, sees, what="many")
    widen(s, 1 << 16)
    run(hq, torch, s, ways, sees, what="many", max_len=1 << 16)
    assert ways[-1][:2] == (128, SHARES)


def test_side_stream_and_graph(ways):
    """Plan and attention on a side stream; captured once and replayed with other lengths, trees and queries."""
    hq, torch = base.lib()
    for per, bound in ((4, 960), (5, 1 << 20)):
        f = kp.Fmt(2, 128, 4, 64, 64)
        t = 26
        new = [t] * 3
        s = base.Scene(hq, torch, f, [900, 31, 640], new, per, "float16", seed=61)
        widen(s, bound)
        rng = np.random.default_rng(62)
        table, lens, _ = args_of(torch, s)
        q, parents = s.q.cuda(), torch.from_numpy(random_parents(rng, new)).cuda()

        def step(stream=None):
            mask, pos, slots = hq.hqq_kv_tree_plan(parents, table, lens, 64, stream=stream)
            return hq.hqq_kv_attention_tree(s.cache, q, mask, table, lens, max_len=bound, stream=stream), mask, pos, slots

        want = step()
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        outs = []
        for rep in range(3):
            outs.append(step(side))
            junk = [torch.full((1 << 20,), float(rep), device="cuda") for _ in range(8)]
            del junk
        side.synchronize()
        assert all(torch.equal(x, y) for o in outs for x, y in zip(o, want))
        warm = torch.cuda.Stream()
        warm.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(warm):
            step()
        torch.cuda.current_stream().wait_stream(warm)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
        for rep in range(4):
            lens.copy_(torch.tensor([[900, 31, 640], [26, 0, 601], [333, 28, 27], [899, 30, 77]][rep], dtype=torch.int32))
            parents.copy_(torch.from_numpy(random_parents(rng, new)))
            q.copy_(kp.to(rng.normal(size=tuple(q.shape)).astype(np.float32), s.dt))
            graph.replay()
            got = [x.clone() for x in out]
            torch.cuda.synchronize()
            assert all(torch.equal(x, y) for x, y in zip(got, step()))
            torch.cuda.synchronize()
