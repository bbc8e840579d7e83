"""Calls of the drafted step's operators at the borders of what they take: ranges with gaps and without a bound, the most drafts of a
sequence, given outputs and workspaces, two calls at once, broadcast inputs, caches whose pages were replaced."""
import numpy as np
import pytest

from tests import kv_plain as kp
from tests import test_gpu_kv as base
from tests.gpu_common import say
from tests.kv_ways import SHARES
from tests.test_gpu_kv_ways import widen
from tests.test_gpu_pages import Pool, accept_plain, compact_plain, paths
from tests.test_gpu_tree import args_of, expect, random_parents, run, sees_of, ways, words_of  # noqa: F401

pytestmark = pytest.mark.gpu


def i32(torch, x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("way", ["streamed", "streams in shares", "tiles"])
def test_ranges_with_gaps(way, ways):  # noqa: F811
    """Tokens in front of the first range and behind the last stay as they are; sequences of no tokens, of a range that leaves the tensor and
    of a negative one have none."""
    hq, torch = base.lib()
    per, bound = {"streamed": (3, 420), "streams in shares": (3, 1 << 12), "tiles": (5, 1 << 20)}[way]
    f = kp.Fmt(2, 128, 4, 64, 32)
    new = [20, 7, 26]
    s = base.Scene(hq, torch, f, [420, 33, 90], new, per, "float16", seed=9)
    sees = sees_of(random_parents(np.random.default_rng(3), new), new)
    want = expect(s, sees)
    front, behind = 3, 5
    total, heads = front + sum(new) + behind, s.q.shape[1]
    fused = torch.zeros(total, 3 * heads, 128, dtype=s.dt, device="cuda")
    q = fused[:, heads:2 * heads]
    q[front:-behind] = s.q.cuda()
    mask = torch.full((total, 1), -1, dtype=torch.int64)
    mask[front:-behind] = torch.from_numpy(words_of(sees, 1))
    cols = max(s.table.shape[1], -(-bound // f.page))
    for places, cu in (([0, 2, 4], [0, 20, 20, 27, 27, 53]), ([0, 1, 4], [0, 20, 27, total, 27, 53])):
        table, lens = np.full((5, cols), -1, np.int32), [64] * 5
        for i, at in enumerate(places):
            table[at, :s.table.shape[1]], lens[at] = s.table[i], s.lens[i]
        out = torch.full((total, heads, 128), 7.0, dtype=s.dt, device="cuda")
        o, lse = hq.hqq_kv_attention_tree(s.cache, q, mask.cuda(), torch.from_numpy(table).cuda(), i32(torch, lens), scale=s.scale,
                                          cu_q=i32(torch, cu) + front, max_q=26, max_len=bound, out=out, return_lse=True)
        w = ways[-1]
        assert o is out and (w[0] >= 128) == (way == "tiles") and w[6] == (way != "streamed"), w
        base.check(torch, o[front:-behind], lse[front:-behind], want, s.dt, tiles=w[0] >= 128, what=way)
        assert (o[:front] == 7).all() and (o[-behind:] == 7).all()


def test_ranges_without_a_bound(ways):  # noqa: F811
    """cu_q without max_q: the mask's bits bound the drafts; more tokens than 4096 in all."""
    hq, torch = base.lib()
    f = kp.Fmt(1, 64, 4, 64, 16)
    rng = np.random.default_rng(4)
    new = [int(x) for x in rng.integers(1, 65, 140)]
    assert sum(new) > 4096
    s = base.Scene(hq, torch, f, [n + 3 for n in new], new, 1, "float16", seed=4)
    sees = sees_of(random_parents(rng, new), new)
    table, lens, kw = args_of(torch, s, True)
    parents = torch.from_numpy(np.concatenate([[np.flatnonzero(m[t, :t])[-1] if m[t, :t].any() else -1 for t in range(len(m))]
                                               for m in sees]).astype(np.int32)).cuda()
    a = hq.hqq_kv_tree_plan(parents, table, lens, 16, cu_q=kw["cu_q"])
    b = hq.hqq_kv_tree_plan(parents, table, lens, 16, **kw)
    assert a[0].shape[1] == 64 and b[0].shape[1] == 1 and torch.equal(a[0][:, :1], b[0]) and not a[0][:, 1:].any()
    assert torch.equal(a[1], b[1]) and torch.equal(a[2], b[2])
    assert torch.equal(b[0].cpu(), torch.from_numpy(words_of(sees, 1)))
    x = hq.hqq_kv_attention_tree(s.cache, s.q.cuda(), b[0], table, lens, scale=s.scale, cu_q=kw["cu_q"], max_len=67, return_lse=True)
    base.check(torch, *x, expect(s, sees), s.dt, tiles=ways[-1][0] >= 128, what="no bound")
    y = hq.hqq_kv_attention_tree(s.cache, s.q.cuda(), a[0], table, lens, scale=s.scale, cu_q=kw["cu_q"], max_len=67)
    assert y.shape == x[0].shape and torch.isfinite(y.float()).all()


@pytest.mark.parametrize("t", [4095, 4096])
def test_most_drafts(t, ways):  # noqa: F811
    """A sequence of as many drafts as a mask has bits for: random trees, a chain's depth among them."""
    hq, torch = base.lib()
    say("most drafts", t)
    f = kp.Fmt(1, 64, 8, 64, 256)
    rng = np.random.default_rng(t)
    s = base.Scene(hq, torch, f, [t + 130], [t], 1, "float16", seed=1)
    parents = random_parents(rng, [t])
    parents[2048:] = np.arange(2047, t - 1)                              # the second half is a chain
    table, lens, _ = args_of(torch, s)
    mask, pos, slots = hq.hqq_kv_tree_plan(torch.from_numpy(parents).cuda(), table, lens, 256)
    sees = sees_of(parents, [t])
    assert torch.equal(mask.cpu(), torch.from_numpy(words_of(sees, 64)))
    assert pos.tolist() == (129 + sees[0].sum(1)).tolist()
    run(hq, torch, s, ways, sees, what="most", mask=mask.cpu().numpy())
    if t == 4096:
        with pytest.raises(hq.HQQError, match="mask_words"):
            hq.hqq_kv_tree_plan(torch.zeros(4097, dtype=torch.int32, device="cuda"), table, lens, 256)


def test_two_calls_at_once(ways):  # noqa: F811
    """Calls on two streams, each with a workspace and an output of its own, and one workspace for calls one after the other."""
    hq, torch = base.lib()
    rng = np.random.default_rng(8)
    jobs = []
    for i, (per, t, lens) in enumerate(((4, 40, [3000, 70, 4000]), (2, 26, [900, 5000, 26]))):
        f = kp.Fmt(2, 128, 4, 64, 64)
        s = base.Scene(hq, torch, f, lens, [t] * 3, per, "float16", seed=i)
        widen(s, 1 << 18)
        sees = sees_of(random_parents(rng, [t] * 3), [t] * 3)
        table, ln, _ = args_of(torch, s)
        args = (s.cache, s.q.cuda(), torch.from_numpy(words_of(sees, 1)).cuda(), table, ln)
        jobs.append((args, s, hq.hqq_kv_attention_tree(*args, scale=s.scale)))
    assert [w[:2] for w in ways] == [(256, SHARES), (16, SHARES)]       # 160 rows of a KV head, and 52
    need = 512 << 20
    one = torch.empty(need, dtype=torch.uint8, device="cuda")
    own = [torch.empty(need, dtype=torch.uint8, device="cuda") for _ in jobs]
    streams = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()
    for rep in range(5):
        outs = [torch.empty_like(j[2]) for j in jobs]
        torch.cuda.synchronize()
        for j, st, w, o in zip(jobs, streams, own, outs):
            hq.hqq_kv_attention_tree(*j[0], scale=j[1].scale, out=o, workspace=w, stream=st)
        torch.cuda.synchronize()
        assert all(torch.equal(o, j[2]) for o, j in zip(outs, jobs))
        one.fill_(255)                                                   # nothing of a workspace is taken as it was
        for j in jobs:
            assert torch.equal(hq.hqq_kv_attention_tree(*j[0], scale=j[1].scale, workspace=one), j[2])
    with pytest.raises(hq.HQQError, match="workspace"):
        hq.hqq_kv_attention_tree(*jobs[0][0], scale=jobs[0][1].scale, workspace=one[:4096])


def test_broadcast_inputs_of_rope():
    """Inputs that repeat one head or one token; their outputs are new, and in place is refused."""
    hq, torch = base.lib()
    rng = np.random.default_rng(6)
    t = hq.hqq_rope_table(128)
    pos = torch.from_numpy(rng.integers(0, 9000, 13)).cuda()
    x = kp.to(rng.normal(size=(13, 1, 128)).astype(np.float32), torch.bfloat16).cuda()
    for wide in (x.expand(13, 5, 128), x[:1].expand(13, 5, 128), x[:1, :1].expand(13, 1, 128)):
        assert torch.equal(hq.hqq_rope(wide, pos, t), hq.hqq_rope(wide.contiguous(), pos, t))
        with pytest.raises(hq.HQQError, match="overlap"):
            hq.hqq_rope(wide, pos, t, out=wide)
    with pytest.raises(hq.HQQError, match="overlap"):
        hq.hqq_rope(x.expand(13, 5, 128).contiguous(), pos, t, out=torch.empty(13, 1, 128, dtype=x.dtype, device="cuda").expand(13, 5, 128))


def test_replaced_pages():
    """A KVLayers whose caches were given other pages (a pool that grew) works on those; different ones are refused."""
    hq, torch = base.lib()
    caches = [hq.hqq_kv_cache(4, 2, 64, page_size=16) for _ in range(3)]
    layers = hq.KVLayers(caches)
    old = []
    for c in caches:
        c.pages.random_(0, 256)
        old.append(c.pages)
        grown = torch.zeros(9, c.pages.shape[1], dtype=torch.uint8, device="cuda")
        grown[:4] = c.pages
        c.pages = grown
    keep = [x.clone() for x in old]
    t, n = hq.hqq_kv_fork(layers, i32(torch, [[3]]), i32(torch, [16 * 0 + 5]), i32(torch, [0, 0]), i32(torch, [-1, 8]))
    assert t.tolist() == [[3], [8]] and n.tolist() == [5, 5]
    assert all(torch.equal(x, y) for x, y in zip(old, keep)) and all(c.pages[8].any() for c in caches)
    t, used = hq.hqq_kv_compact(layers, t, n)
    assert used.tolist() == [2] and t.tolist() == [[0], [1]]
    assert all(torch.equal(x, y) for x, y in zip(old, keep)) and all(torch.equal(c.pages[0], k[3]) for c, k in zip(caches, keep))
    caches[1].pages = caches[1].pages[:7]
    with pytest.raises(ValueError, match="one format and one number of pages"):
        hq.hqq_kv_compact(layers, t, n)


@pytest.mark.parametrize("pages,batch,cols,layers,hkv", [(4095, 3, 900, 1, 1), (4096, 64, 128, 1, 1), (4096, 1, 8193, 1, 1), (4097, 40, 90, 1, 1), (400, 5, 60, 3, 8),
                                                         (400, 5, 60, 24, 8)])
def test_compact_in_one_launch_and_in_two(pages, batch, cols, layers, hkv):
    """Around the sizes where the blocks stop planning for themselves: pages, entries of the tables, bytes that may move; captured and replayed
    with other tables."""
    hq, torch = base.lib()
    say("compact", pages, batch, cols, layers)
    f = kp.Fmt(hkv, 64, 4, 64, 16)
    rng = np.random.default_rng(pages + cols)
    pool = Pool(hq, torch, f, layers, pages, seed=3)

    def draw():
        table = np.full((batch, cols), -1, np.int32)
        ids = rng.permutation(pages)[:pages // 3].astype(np.int32)
        lens = rng.integers(0, 16 * min(cols, pages // 3 // batch) + 1, batch)
        for b, n in enumerate(lens):
            held = -(-int(n) // 16)
            table[b, :held], ids = ids[:held], ids[held:]
        return table, [int(x) for x in lens]

    table, lens = draw()
    t, n = i32(torch, table), i32(torch, lens)
    m, used = hq.hqq_kv_compact(pool.layers, t, n)
    want, u = compact_plain(pool, table, lens)
    assert np.array_equal(m.cpu().numpy(), want) and used.tolist() == [u] and u > 0
    pool.check("eager")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m, used = hq.hqq_kv_compact(pool.layers, t, n)
    for rep in range(3):
        table, lens = draw()
        t.copy_(i32(torch, table))
        n.copy_(i32(torch, lens))
        graph.replay()
        torch.cuda.synchronize()
        want, u = compact_plain(pool, table, lens)
        assert np.array_equal(m.cpu().numpy(), want) and used.tolist() == [u]
        pool.check("replayed")


@pytest.mark.parametrize("d,bits,g", base.FORMATS)
def test_accept_long_lists(d, bits, g):
    """Accepted drafts of several windows of 256 places, from any place of a page on, among them whole runs that stay; many sequences."""
    hq, torch = base.lib()
    rng = np.random.default_rng(bits + g)
    for page, hkv, layers, new, most in ((16, 5, 3, [700, 513, 260], 600), (256, 3, 2, [600, 37, 900], 900), (32, 2, 40, [9] * 70, 9)):
        say("accept", d, bits, g, page, new[:3])
        f = kp.Fmt(hkv, d, bits, g, page)
        lens = [n + int(rng.integers(0, 50)) for n in new]
        cols = max(-(-n // page) for n in lens)
        pool = Pool(hq, torch, f, layers, cols * len(new) + 3, seed=page)
        table = rng.permutation(cols * len(new)).reshape(len(new), cols).astype(np.int32)
        accepted, counts = paths(rng, new, most)
        for b, c in enumerate(counts):                                  # every other list starts with a run that stays
            if b % 2 == 0:
                accepted[b, :c] = np.sort(np.r_[np.arange(c // 2), c // 2 + np.sort(rng.permutation(new[b] - c // 2)[:c - c // 2])])
        if len(set(new)) > 1:
            kw = dict(cu_q=base.cu(torch, new), max_q=max(new))
        else:
            kw = dict(tokens=new[0])
        n = hq.hqq_kv_accept(pool.layers, i32(torch, table), i32(torch, lens), i32(torch, accepted), i32(torch, counts), **kw)
        want = accept_plain(pool, table.tolist(), lens, new, accepted.tolist(), counts)
        assert n.tolist() == want
        pool.check("accepted")


@pytest.mark.parametrize("inter", [False, True])
def test_outputs_past_the_caches(inter):
    """Outputs of 32 MiB and of one token more, which are stored past the caches: the bits of the same tokens in smaller calls; in place too."""
    hq, torch = base.lib()
    rng = np.random.default_rng(12)
    t = hq.hqq_rope_table(64, interleaved=inter)
    full = 1 << 12                                                       # tokens of 32 heads of 128 channels in 32 MiB
    for n, dtype in ((full, torch.float16), (full + 1, torch.float16), (full + 77, torch.bfloat16)):
        say("past the caches", inter, n)
        pos = torch.from_numpy(rng.integers(0, 1 << 20, n)).cuda()
        q = torch.randn(n, 32, 128, device="cuda").to(dtype)
        k, v = torch.randn(n, 2, 128, device="cuda").to(dtype), torch.randn(n, 2, 128, device="cuda").to(dtype)
        parts = torch.cat([hq.hqq_rope(q[i:i + 1000], pos[i:i + 1000], t) for i in range(0, n, 1000)])
        assert torch.equal(hq.hqq_rope(q, pos, t), parts)
        cache, other = hq.hqq_kv_cache(-(-n // 64), 2, 128), hq.hqq_kv_cache(-(-n // 64), 2, 128)
        cache.pages.zero_(), other.pages.zero_()
        slots = torch.arange(n, device="cuda")
        assert torch.equal(hq.hqq_kv_write_rope(cache, q, k, v, pos, slots, t), parts)
        hq.hqq_kv_write(other, hq.hqq_rope(k, pos, t), v, slots)
        assert torch.equal(cache.pages, other.pages)
        assert hq.hqq_rope(q, pos, t, out=q) is q and torch.equal(q, parts)
