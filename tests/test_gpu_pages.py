"""Moving what the cache holds (accepted drafts, forks, compaction) against plain copies of each token's bytes, which the
page layout's index formulas name; everything that is not moved keeps its bytes."""
import numpy as np
import pytest

from tests import kv_plain as kp
from tests import test_gpu_kv as base
from tests.gpu_common import say

pytestmark = pytest.mark.gpu


def token_bytes(f):
    """Byte offsets within a block of everything a token has, [page, bytes]."""
    out = []
    for t in range(f.page):
        at = {f.bit_of(w, t, c) // 8 for w in "kv" for c in range(f.d)}
        at |= {f.meta_of(w, t, g) + i for w in "kv" for g in range(f.d // f.g) for i in range(4)}
        out.append(sorted(at))
    return np.array(out)


class Pool:
    """Layers of random bytes, and their pages in numpy."""

    def __init__(self, hq, torch, f, layers, pages, seed):
        self.rng = np.random.default_rng(seed)
        self.want = self.rng.integers(0, 256, (layers, pages, f.hkv, f.block), np.uint8)
        self.f, self.where = f, token_bytes(f)
        self.pages = torch.from_numpy(self.want.copy()).cuda()
        self.layers = hq.KVLayers([hq.KVCache(p, f.hkv, f.d, f.bits, f.g, f.page) for p in self.pages])

    def token(self, table, pos):
        """Page and bytes of a sequence's token; None outside the cache."""
        p = table[pos // self.f.page]
        return (p, self.where[pos % self.f.page]) if 0 <= p < self.want.shape[1] else None

    def check(self, what=""):
        got = self.pages.cpu().numpy()
        assert np.array_equal(got, self.want), "%s: %d bytes differ" % (what, (got != self.want).sum())


def i32(torch, x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------------------ accepted drafts

def accept_plain(pool, table, lens, new, accepted, counts):
    out = []
    for b, (n, t) in enumerate(zip(lens, new)):
        base_at, count = n - t, min(max(counts[b], 0), len(accepted[b]), t)
        moves = []
        for j in range(count):
            a = accepted[b][j]
            if not 0 <= a < t or base_at + a < 0 or base_at + j < 0:
                continue
            src, dst = pool.token(table[b], base_at + a), pool.token(table[b], base_at + j)
            if src and dst:
                moves.append((dst, pool.want[:, src[0]][:, :, src[1]].copy()))
        for (p, at), data in moves:
            pool.want[:, p, :, at] = np.moveaxis(data, 2, 0)
        out.append(max(base_at + count, 0))
    return out


def paths(rng, new, most):
    """Rising lists of accepted drafts, padded with -1."""
    out, counts = np.full((len(new), most), -1, np.int32), []
    for b, t in enumerate(new):
        c = int(rng.integers(0, min(most, t) + 1))
        out[b, :c] = np.sort(rng.permutation(t)[:c])
        counts.append(c)
    return out, counts


@pytest.mark.parametrize("d,bits,g", base.FORMATS)
def test_accept(d, bits, g):
    hq, torch = base.lib()
    for page, hkv, layers, new, most in ((16, 3, 2, [5, 1, 33, 8], 33), (64, 1, 1, [26], 9), (256, 2, 3, [13, 13, 13], 13), (32, 9, 2, [4, 0, 60, 31], 20)):
        say("accept", d, bits, g, page, hkv, layers, new)
        f = kp.Fmt(hkv, d, bits, g, page)
        rng = np.random.default_rng(d + page)
        lens = [t + int(rng.integers(0, 90)) for t in new]
        cols = -(-max(lens) // page)
        pool = Pool(hq, torch, f, layers, len(new) * cols + 1, seed=page + g)
        table = rng.permutation(len(new) * cols + 1)[:len(new) * cols].reshape(len(new), cols).astype(np.int32)
        accepted, counts = paths(rng, new, most)
        ragged = len(set(new)) > 1
        kw = dict(cu_q=base.cu(torch, new), max_q=max(new)) if ragged else dict(tokens=new[0])
        got = hq.hqq_kv_accept(pool.layers, i32(torch, table), i32(torch, lens), i32(torch, accepted), i32(torch, counts), **kw)
        assert got.tolist() == accept_plain(pool, table, lens, new, accepted, counts)
        pool.check("accept")


def test_accept_edges():
    """Counts out of range, indices outside the draft, sequences shorter than their drafts and without any, missing pages, more
    accepted drafts than one turn of a block takes and than one list of places; a single cache and a list of caches."""
    hq, torch = base.lib()
    f = kp.Fmt(2, 128, 4, 64, 16)
    rng = np.random.default_rng(3)
    new = [10] * 6
    lens = [40, 7, 0, 60, 33, 12]
    pool = Pool(hq, torch, f, 2, 30, seed=1)
    table = rng.permutation(30)[:24].reshape(6, 4).astype(np.int32)
    table[3, 3], table[4, 1] = -1, 30
    accepted = np.tile(np.array([1, 2, 5, 7, 8, 9], np.int32), (6, 1))
    accepted[0, 3], accepted[5] = -4, [0, 3, 4, 10, 11, 1000]
    counts = [6, 4, 3, 5, 99, 6]
    got = hq.hqq_kv_accept(pool.layers, i32(torch, table), i32(torch, lens), i32(torch, accepted), i32(torch, counts), tokens=10)
    assert got.tolist() == accept_plain(pool, table, lens, new, accepted, counts)
    pool.check("edges")
    # none and negative counts move nothing
    got = hq.hqq_kv_accept(pool.layers, i32(torch, table), i32(torch, lens), i32(torch, accepted), i32(torch, [0, -3, 0, 0, -1, 0]), tokens=10)
    assert got.tolist() == [max(n - 10, 0) for n in lens]
    pool.check("none")
    # 600 drafts, 560 of them accepted, 5 heads
    f = kp.Fmt(5, 64, 4, 32, 64)
    pool = Pool(hq, torch, f, 1, 20, seed=2)
    table = rng.permutation(20)[:12].reshape(1, 12).astype(np.int32)
    accepted = np.sort(rng.permutation(600)[:560]).astype(np.int32)[None]
    cache = pool.layers.caches[0]
    for layers in (cache, [cache]):
        got = hq.hqq_kv_accept(layers, i32(torch, table), i32(torch, [700]), i32(torch, accepted), i32(torch, [560]), tokens=600)
        assert got.tolist() == accept_plain(pool, table, [700], [600], accepted, [560])
        pool.check("many")
    # no sequence; no list
    empty = torch.zeros(0, dtype=torch.int32, device="cuda")
    assert hq.hqq_kv_accept(cache, i32(torch, table)[:0], empty, i32(torch, accepted)[:0], empty, tokens=4).shape == (0,)
    assert hq.hqq_kv_accept(cache, i32(torch, table), i32(torch, [30]), i32(torch, accepted)[:, :0], i32(torch, [2]), tokens=4).tolist() == [26]
    pool.check("empty")
    with pytest.raises(ValueError, match="tokens"):
        hq.hqq_kv_accept(cache, i32(torch, table), i32(torch, [30]), i32(torch, accepted), i32(torch, [2]))


# ------------------------------------------------------------------------------ forks

def fork_plain(pool, table, lens, parents, fresh):
    page, count = pool.f.page, pool.want.shape[1]
    out, out_lens, before = [], [], set()
    for c, p in enumerate(parents):
        if not 0 <= p < len(lens):
            out.append([-1] * table.shape[1])
            out_lens.append(0)
            continue
        n = min(max(lens[p], 0), table.shape[1] * page)
        row = list(table[p])
        if p in before:
            last = n // page
            row[last:] = [-1] * (len(row) - last)
            if n % page:
                row[last] = fresh[c]
                src, dst = table[p][last], fresh[c]
                if 0 <= src < count and 0 <= dst < count:
                    for t in range(n % page):
                        at = pool.where[t]
                        pool.want[:, dst][:, :, at] = pool.want[:, src][:, :, at]
        before.add(p)
        out.append(row)
        out_lens.append(n)
    return np.array(out, np.int32).reshape(len(parents), table.shape[1]), out_lens


@pytest.mark.parametrize("d,bits,g", base.FORMATS)
def test_fork(d, bits, g):
    hq, torch = base.lib()
    for page, hkv, layers, batch, new in ((16, 3, 2, 5, 9), (64, 1, 1, 1, 4), (256, 2, 2, 3, 3), (32, 5, 3, 7, 20), (128, 6, 1, 2, 5)):
        say("fork", d, bits, g, page, hkv, layers, batch, new)
        f = kp.Fmt(hkv, d, bits, g, page)
        rng = np.random.default_rng(d + page + new)
        lens = [int(x) for x in rng.integers(0, 3 * page, batch)]
        lens[0] = 2 * page                                     # whole pages
        cols = 4
        pool = Pool(hq, torch, f, layers, batch * cols + new, seed=page + g)
        ids = rng.permutation(batch * cols + new).astype(np.int32)
        table, fresh = ids[:batch * cols].reshape(batch, cols), ids[batch * cols:]
        parents = rng.integers(0, batch, new)
        if new > 6:
            parents[3], parents[5] = -1, batch
        t, n = hq.hqq_kv_fork(pool.layers, i32(torch, table), i32(torch, lens), i32(torch, parents), i32(torch, fresh))
        want, want_lens = fork_plain(pool, table, lens, parents.tolist(), fresh.tolist())
        assert np.array_equal(t.cpu().numpy(), want) and n.tolist() == want_lens
        pool.check("fork")


def test_fork_every_length():
    """Each number of tokens on the partly filled page, children of one parent."""
    hq, torch = base.lib()
    for d, bits, g, page in ((64, 4, 32, 16), (128, 8, 64, 32), (128, 4, 128, 64)):
        f = kp.Fmt(2, d, bits, g, page)
        batch = page + 1
        pool = Pool(hq, torch, f, 1, 2 * batch, seed=d)
        table = np.arange(batch, dtype=np.int32)[:, None]
        parents = np.repeat(np.arange(batch), 2)
        fresh = np.where(np.arange(2 * batch) % 2, batch + np.arange(2 * batch) // 2, -1)
        lens = list(range(batch))
        t, n = hq.hqq_kv_fork(pool.layers, i32(torch, table), i32(torch, lens), i32(torch, parents), i32(torch, fresh))
        want, want_lens = fork_plain(pool, table, lens, parents.tolist(), fresh.tolist())
        assert np.array_equal(t.cpu().numpy(), want) and n.tolist() == want_lens
        pool.check("length")


def test_fork_edges():
    """Lengths past the table and negative ones, missing pages and fresh pages outside the cache, no child, more children than a block has
    threads, wide tables."""
    hq, torch = base.lib()
    f = kp.Fmt(1, 64, 4, 64, 16)
    rng = np.random.default_rng(4)
    pool = Pool(hq, torch, f, 2, 340, seed=8)
    ids = rng.permutation(340).astype(np.int32)
    table = ids[:12].reshape(4, 3).copy()
    table[1, 1] = -1
    lens = [1000, 20, -5, 41]
    parents = rng.integers(0, 4, 320)
    fresh = ids[12:332].copy()
    fresh[[5, 300]] = -1, 340
    t, n = hq.hqq_kv_fork(pool.layers, i32(torch, table), i32(torch, lens), i32(torch, parents), i32(torch, fresh))
    want, want_lens = fork_plain(pool, table, lens, parents.tolist(), fresh.tolist())
    assert np.array_equal(t.cpu().numpy(), want) and n.tolist() == want_lens
    pool.check("edges")
    wide = torch.full((4, 9), 77, dtype=torch.int32, device="cuda")
    wide[:, 2:5] = i32(torch, table)
    t2, n2 = hq.hqq_kv_fork(pool.layers, wide[:, 2:5], i32(torch, lens), i32(torch, parents), i32(torch, fresh))
    assert torch.equal(t, t2) and torch.equal(n, n2)
    pool.check("again")
    t, n = hq.hqq_kv_fork(pool.layers, i32(torch, table), i32(torch, lens), i32(torch, parents[:0]), i32(torch, fresh[:0]))
    assert t.shape == (0, 3) and n.shape == (0,)


# ------------------------------------------------------------------------------ compaction

def compact_plain(pool, table, lens):
    page, count = pool.f.page, pool.want.shape[1]
    held, cols = set(), table.shape[1]
    need = [min(-(-min(max(n, 0), cols * page) // page), cols) for n in lens]
    for row, k in zip(table, need):
        held |= {int(p) for p in row[:k] if 0 <= p < count}
    u = len(held)
    far, holes = sorted(p for p in held if p >= u), sorted(set(range(u)) - held)
    to = dict(zip(far, holes))
    data = pool.want[:, far].copy()
    pool.want[:, holes] = data
    out = np.full(table.shape, -1, np.int32)
    for b, k in enumerate(need):
        for c in range(k):
            p = int(table[b, c])
            if 0 <= p < count:
                out[b, c] = to.get(p, p)
    return out, u


@pytest.mark.parametrize("pages,batch,cols,share", [(1, 1, 1, 0), (31, 3, 5, 2), (32, 4, 8, 0), (33, 5, 4, 1), (64, 8, 8, 0), (257, 9, 20, 3), (1000, 7, 3, 0),
                                                    (4099, 40, 100, 5), (70000, 16, 20, 1)])
def test_compact(pages, batch, cols, share):
    hq, torch = base.lib()
    say("compact", pages, batch, cols, share)
    f = kp.Fmt(1, 64, 4, 64, 16)
    rng = np.random.default_rng(pages)
    pool = Pool(hq, torch, f, 2 if pages < 50000 else 1, pages, seed=pages)
    lens = [int(x) for x in rng.integers(0, cols * 16 + 1, batch)]
    table = rng.choice(pages, (batch, cols), replace=pages < batch * cols).astype(np.int32)
    table[:, :share] = table[0, :share]                      # pages that all sequences hold
    if pages > 100:
        table[1, 0], table[2, 1] = -7, pages
    t, used = hq.hqq_kv_compact(pool.layers, i32(torch, table), i32(torch, lens))
    want, u = compact_plain(pool, table, lens)
    assert np.array_equal(t.cpu().numpy(), want) and used.tolist() == [u]
    pool.check("compact")
    again, used = hq.hqq_kv_compact(pool.layers, t, i32(torch, lens))          # nothing left to move
    assert torch.equal(again, t) and used.tolist() == [u]
    pool.check("again")


@pytest.mark.parametrize("d,bits,g", base.FORMATS)
def test_compact_formats(d, bits, g):
    hq, torch = base.lib()
    for page, hkv, layers in ((16, 1, 5), (256, 3, 2), (64, 8, 3)):
        f = kp.Fmt(hkv, d, bits, g, page)
        rng = np.random.default_rng(d + page)
        pool = Pool(hq, torch, f, layers, 37, seed=g)
        table = rng.permutation(37)[:20].reshape(4, 5).astype(np.int32)
        lens = [5 * page, page + 1, 0, 3 * page - 1]
        t, used = hq.hqq_kv_compact(pool.layers, i32(torch, table), i32(torch, lens))
        want, u = compact_plain(pool, table, lens)
        assert np.array_equal(t.cpu().numpy(), want) and used.tolist() == [u]
        pool.check("formats")


def test_compact_edges():
    """No sequence, nothing held, everything held; a given workspace of any contents; wide tables; the most pages."""
    hq, torch = base.lib()
    f = kp.Fmt(1, 64, 4, 64, 16)
    pool = Pool(hq, torch, f, 2, 64, seed=3)
    t, used = hq.hqq_kv_compact(pool.layers, i32(torch, np.zeros((0, 4))), i32(torch, np.zeros(0)))
    assert t.shape == (0, 4) and used.tolist() == [0]
    t, used = hq.hqq_kv_compact(pool.layers, i32(torch, [[3, 4], [5, 6]]), i32(torch, [0, -9]))
    assert (t == -1).all() and used.tolist() == [0]
    every = np.random.default_rng(1).permutation(64).reshape(4, 16).astype(np.int32)
    ws = torch.full((hq.hqq_kv_compact_workspace_bytes(64),), 0xEE, dtype=torch.uint8, device="cuda")
    t, used = hq.hqq_kv_compact(pool.layers, i32(torch, every), i32(torch, [256] * 4), workspace=ws)
    assert np.array_equal(t.cpu().numpy(), every) and used.tolist() == [64]
    wide = torch.full((4, 30), 9, dtype=torch.int32, device="cuda")
    wide[:, 7:23] = i32(torch, every)
    t, used = hq.hqq_kv_compact(pool.layers, wide[:, 7:23], i32(torch, [16, 17, 0, 40]), workspace=ws)
    want, u = compact_plain(pool, every, [16, 17, 0, 40])
    assert np.array_equal(t.cpu().numpy(), want) and used.tolist() == [u]
    pool.check("edges")
    with pytest.raises(hq.HQQError):
        hq.hqq_kv_compact(pool.layers, wide, i32(torch, [1] * 4), workspace=ws[:64])
    say("compact, 2^20 pages")
    page_bytes = hq.hqq_kv_page_bytes(1, 64, 4, 64, 16)
    pages = torch.zeros((1 << 20, page_bytes), dtype=torch.uint8, device="cuda")
    ids = np.array([[5, (1 << 20) - 1, 1 << 19, 0, 123457]], np.int32)
    pages[torch.from_numpy(ids[0]).long().cuda()] = torch.arange(1, 6, dtype=torch.uint8, device="cuda")[:, None]
    cache = hq.KVCache(pages, 1, 64, 4, 64, 16)
    t, used = hq.hqq_kv_compact(cache, i32(torch, ids), i32(torch, [80]))
    # five pages: 0 stays, 5, 123457, 2^19 and 2^20 - 1 go to 1, 2, 3, 4
    assert t.tolist() == [[1, 4, 3, 0, 2]] and used.tolist() == [5]
    assert pages[:5, 0].tolist() == [4, 1, 5, 3, 2] and bool((pages[:5] == pages[:5, :1]).all())
    with pytest.raises(hq.HQQError):
        hq.hqq_kv_compact(hq.KVCache(torch.zeros(((1 << 20) + 1, page_bytes), dtype=torch.uint8, device="cuda"), 1, 64, 4, 64, 16),
                          i32(torch, ids), i32(torch, [80]))


# ------------------------------------------------------------------------------ streams, graphs, reads

def test_moved_tokens_read_back():
    """What the cache stands for moves along: accepted, forked and compacted tokens read back as they were written."""
    hq, torch = base.lib()
    f = kp.Fmt(2, 128, 4, 64, 16)
    rng = np.random.default_rng(6)
    cache = base.make_cache(hq, torch, f, 40)
    layers = hq.KVLayers([cache])
    table = rng.permutation(40)[:8].reshape(2, 4).astype(np.int32)
    lens, t = [50, 33], 12
    written = []
    for b, n in enumerate(lens):
        k, v = (kp.to(x, torch.float16).cuda() for x in base.values(rng, n, 2, 128))
        slots = torch.tensor([int(table[b, i // 16]) * 16 + i % 16 for i in range(n)], device="cuda")
        written.append(hq.hqq_kv_write(cache, k, v, slots, echo=True))
    accepted = np.array([[0, 2, 3, 7], [1, 5, 0, 0]], np.int32)
    new = hq.hqq_kv_accept(layers, i32(torch, table), i32(torch, lens), i32(torch, accepted), i32(torch, [4, 2]), tokens=t)
    keep = [list(range(38)) + [38 + a for a in (0, 2, 3, 7)], list(range(21)) + [21 + a for a in (1, 5)]]
    assert new.tolist() == [42, 23]
    fresh = np.setdiff1d(np.arange(40), table)[-3:]
    children, child_lens = hq.hqq_kv_fork(layers, i32(torch, table), new, i32(torch, [1, 0, 1]), i32(torch, fresh))
    moved, used = hq.hqq_kv_compact(layers, children, child_lens)
    assert child_lens.tolist() == [23, 42, 23] and used.tolist() == [2 + 3 + 1]
    pages = moved.cpu().numpy()
    assert pages.max() < 6
    for c, p in enumerate((1, 0, 1)):
        slots = torch.tensor([int(pages[c, i // 16]) * 16 + i % 16 for i in range(len(keep[p]))], device="cuda")
        for got, want in zip(hq.hqq_kv_read(cache, slots), written[p]):
            assert torch.equal(got, want[keep[p]])


def test_side_stream_and_graph():
    """All three on a side stream while the current one allocates; captured once and replayed on other tables."""
    hq, torch = base.lib()
    f = kp.Fmt(2, 64, 8, 32, 16)
    rng = np.random.default_rng(12)
    pool = Pool(hq, torch, f, 3, 60, seed=5)
    start = pool.pages.clone()
    ids = rng.permutation(60).astype(np.int32)
    table, fresh = i32(torch, ids[:32].reshape(4, 8)), i32(torch, ids[32:38])
    lens, parents = i32(torch, [100, 37, 64, 90]), i32(torch, [3, 3, 0, 1, 1, 1])
    accepted, counts = i32(torch, [[0, 3, 4, 8]] * 4), i32(torch, [4, 2, 3, 1])

    def step(stream=None):
        n = hq.hqq_kv_accept(pool.layers, table, lens, accepted, counts, tokens=9, stream=stream)
        t, n = hq.hqq_kv_fork(pool.layers, table, n, parents, fresh, stream=stream)
        m, used = hq.hqq_kv_compact(pool.layers, t, n, stream=stream)
        return n, t, m, used

    def eager():
        pool.pages.copy_(start)
        out = step()
        return out, pool.pages.clone()

    want, pages = eager()
    side = torch.cuda.Stream()
    for rep in range(3):
        pool.pages.copy_(start)
        side.wait_stream(torch.cuda.current_stream())
        out = step(side)
        junk = [torch.full((1 << 18,), float(rep), device="cuda") for _ in range(8)]
        del junk
        side.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(out, want)) and torch.equal(pool.pages, pages)
    warm = torch.cuda.Stream()
    warm.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(warm):
        step()
    torch.cuda.current_stream().wait_stream(warm)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for rep in range(4):
        ids = rng.permutation(60).astype(np.int32)
        table.copy_(i32(torch, ids[:32].reshape(4, 8)))
        fresh.copy_(i32(torch, ids[32:38]))
        lens.copy_(i32(torch, rng.integers(9, 129, 4)))
        parents.copy_(i32(torch, rng.integers(0, 4, 6)))
        pool.pages.copy_(start)
        graph.replay()
        got, moved = [x.clone() for x in out], pool.pages.clone()
        torch.cuda.synchronize()
        want, pages = eager()
        assert all(torch.equal(x, y) for x, y in zip(got, want)) and torch.equal(moved, pages)
        torch.cuda.synchronize()


def test_pages_past_32_bits():
    """Pages whose bytes lie past 2^32, moved by each of the three."""
    hq, torch = base.lib()
    f = kp.Fmt(8, 128, 8, 64, 256)
    page_bytes = f.hkv * f.block
    num = (5 << 30) // page_bytes
    say("moves past 32 bits", num, page_bytes)
    pages = torch.empty((num, page_bytes), dtype=torch.uint8, device="cuda")
    cache = hq.KVCache(pages, 8, 128, 8, 64, 256)
    a, b = num - 1, num - 2
    pages[a] = torch.randint(0, 256, (page_bytes,), dtype=torch.uint8, device="cuda")
    pages[b] = 3
    k0, v0 = hq.hqq_kv_read(cache, torch.arange(256, device="cuda") + a * 256)
    bits = [x.view(torch.int16) for x in (k0, v0)]

    def tokens(page, at):
        return [x.view(torch.int16) for x in hq.hqq_kv_read(cache, torch.tensor(at, device="cuda") + page * 256)]

    t, n = hq.hqq_kv_fork(cache, i32(torch, [[a]]), i32(torch, [101]), i32(torch, [0, 0]), i32(torch, [-1, b]))
    assert t.tolist() == [[a], [b]] and n.tolist() == [101, 101]
    assert all(torch.equal(x, y[:101]) for x, y in zip(tokens(b, list(range(101))), bits))
    n = hq.hqq_kv_accept(cache, i32(torch, [[a]]), i32(torch, [200]), i32(torch, [[0, 40, 77]]), i32(torch, [3]), tokens=80)
    assert n.tolist() == [123]
    assert all(torch.equal(x, y[[120, 160, 197]]) for x, y in zip(tokens(a, [120, 121, 122]), bits))
    keep = pages[a].clone()
    t, used = hq.hqq_kv_compact(cache, i32(torch, [[a]]), i32(torch, [256]))
    assert t.tolist() == [[0]] and used.tolist() == [1] and torch.equal(pages[0], keep)
