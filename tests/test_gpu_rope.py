"""Rotary positions and the write that takes them into the cache, against 64 bits.

Tolerances, derived before the first run.  Angle and rotation are 64-bit operations and the result is rounded to fp32 and then to
the type: with u the type's half unit (2^-11 fp16, 2^-8 bf16), |error| <= (u + 2^-24)|y|, plus half of fp16's smallest number, 2^-25, and of
the 64-bit operations 2^-50 of the pair (the angle is position * freq, one product, on both sides).  The fused write gives the
bits of the two calls that it stands for."""
import numpy as np
import pytest

from tests import kv_plain as kp
from tests import test_gpu_kv as base
from tests.gpu_common import say

pytestmark = pytest.mark.gpu

HALF_UNIT = {"float16": 2.0 ** -11, "bfloat16": 2.0 ** -8}


def pairs_of(rot, inter):
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)


def turned(x, pos, freqs, m, inter, back):
    """x [n, heads, D] in 64 bits, turned; and the size of each value's pair."""
    a, b = pairs_of(2 * len(freqs), inter)
    ang = pos.astype(np.float64)[:, None] * freqs
    c, s = (m * np.cos(ang))[:, None], (m * np.sin(ang))[:, None]
    s = -s if back else s
    y, size = x.copy(), np.abs(x)
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    size[..., a] = size[..., b] = m * (np.abs(x[..., a]) + np.abs(x[..., b]))
    return y, size


def check(got, want, size, dtype, what):
    got = got.double().cpu().numpy()
    tol = (HALF_UNIT[dtype] + 2.0 ** -24) * np.abs(want) + 2.0 ** -25 + 2.0 ** -50 * size
    err = np.abs(got - want)
    assert (err <= tol).all(), "%s: %.3g of %.3g" % (what, err.flat[(err - tol).argmax()], tol.flat[(err - tol).argmax()])


def table(torch, hq, rot, inter, factor):
    t = hq.hqq_rope_table(rot, 10000.0, inter, "bands" if factor > 1 else "none", factor, original_len=2048)
    return t, t.freqs.cpu().numpy(), t.magnitude


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("d,rot", [(16, 16), (64, 64), (64, 16), (80, 32), (96, 96), (112, 64), (128, 128), (128, 48), (256, 256), (320, 128),
                                   (512, 512), (1024, 1024), (1024, 208)])
def test_rope(d, rot, inter, dtype):
    hq, torch = base.lib()
    dt = getattr(torch, dtype)
    for n, heads, kheads, factor, back in ((1, 1, 0, 1.0, False), (5, 3, 1, 8.0, False), (67, 5, 2, 1.0, True), (9, 33, 17, 4.0, True)):
        say("rope", d, rot, inter, dtype, n, heads, kheads, factor, back)
        rng = np.random.default_rng(d + rot + n)
        t, freqs, m = table(torch, hq, rot, inter, factor)
        pos = rng.integers(0, 200000, n)
        pos[0] = 0 if n == 1 else 1 << 40
        x = kp.to(rng.normal(size=(n, heads + kheads, d)).astype(np.float32) * 3, dt).cuda()
        q, k = x[:, :heads], x[:, heads:]
        p = torch.from_numpy(pos).cuda()
        got = hq.hqq_rope(q, p, t, k=k if kheads else None, backward=back)
        for g, y in zip(got if kheads else (got,), (q, k)):
            want, size = turned(y.double().cpu().numpy(), pos, freqs, m, inter, back)
            assert g.shape == y.shape and g.is_contiguous()
            check(g, want, size, dtype, (n, heads, factor, back))
            assert torch.equal(g[..., rot:], y[..., rot:])


@pytest.mark.parametrize("inter", [False, True])
def test_gradient(inter):
    """The backward call against the formula's Jacobian, taken column by column from the forward call (it is linear: differences
    are exact but for the outputs' roundings): |error| <= u (2 |g| m + |dx|), two terms of a pair."""
    hq, torch = base.lib()
    d, rot = 64, 48
    t, freqs, m = table(torch, hq, rot, inter, 4.0)
    rng = np.random.default_rng(3)
    for pos in (0, 1, 777, 123456):
        p = torch.full((d,), pos, dtype=torch.int64, device="cuda")
        eye = torch.eye(d, dtype=torch.float16, device="cuda")[:, None]
        cols = hq.hqq_rope(eye, p, t)[:, 0].double().cpu().numpy()          # row i: the image of channel i
        g = kp.to(rng.normal(size=(d, 1, d)).astype(np.float32), torch.float16).cuda()
        dx = hq.hqq_rope(g, p, t, backward=True)[:, 0].double().cpu().numpy()
        gg = g[:, 0].double().cpu().numpy()
        want = gg @ cols.T
        tol = 2.0 ** -11 * (2 * m * np.abs(gg).max() + np.abs(want)) + 2.0 ** -24
        assert (np.abs(dx - want) <= tol).all()
        # and back and forth is the magnitude squared, each call rounding once
        y = hq.hqq_rope(hq.hqq_rope(g, p, t), p, t, backward=True)[:, 0].double().cpu().numpy()
        keep = gg * np.where(np.arange(d) < rot, m * m, 1.0)
        assert (np.abs(y - keep) <= 2.0 ** -11 * (4 * m * m * np.abs(gg).max() + np.abs(keep))).all()


def test_strides_places_and_repeats():
    """Slices of a fused projection, [head, token] tensors, outputs in place and into given tensors; the same call twice."""
    hq, torch = base.lib()
    rng = np.random.default_rng(5)
    n = 21
    for d, rot, inter in ((128, 128, False), (128, 64, True), (80, 32, False), (64, 64, True)):
        t, _, _ = table(torch, hq, rot, inter, 1.0)
        pos = torch.from_numpy(rng.integers(0, 5000, n)).cuda()
        qkv = kp.to(rng.normal(size=(n, 12, d)).astype(np.float32), torch.float16).cuda()
        q, k = qkv[:, 1:8], qkv[:, 8:10]
        want_q, want_k = hq.hqq_rope(q.contiguous(), pos, t, k=k.contiguous())
        a, b = hq.hqq_rope(q, pos, t, k=k)
        assert torch.equal(a, want_q) and torch.equal(b, want_k)
        ht = q.transpose(0, 1).contiguous().transpose(0, 1)
        out = torch.empty(7, n, d, dtype=torch.float16, device="cuda").transpose(0, 1)
        assert hq.hqq_rope(ht, pos, t, out=out) is out and torch.equal(out, want_q)
        rest = qkv.clone()
        a, b = hq.hqq_rope(q, pos, t, k=k, out=(q, k))
        assert torch.equal(qkv[:, 1:8], want_q) and torch.equal(qkv[:, 8:10], want_k)
        assert torch.equal(qkv[:, :1], rest[:, :1]) and torch.equal(qkv[:, 10:], rest[:, 10:])
        assert hq.hqq_rope(q[:0], pos[:0], t).shape == (0, 7, d)
    with pytest.raises(ValueError, match="shape"):
        hq.hqq_rope(q, pos, t, out=k)
    with pytest.raises(ValueError, match="strides"):
        hq.hqq_rope(qkv[:, 1:8, ::2], pos, t)


def test_special_values():
    """NaN and infinities stay within their pair; results past fp16 are infinite; copied channels keep their bits."""
    hq, torch = base.lib()
    t, _, _ = table(torch, hq, 32, False, 1.0)
    x = torch.ones(6, 1, 64, dtype=torch.float16, device="cuda")
    x[0, 0, 3], x[1, 0, 17], x[2, 0, 40] = float("nan"), float("inf"), float("nan")
    x[3, 0, 5] = x[3, 0, 21] = 65504.0
    pos = torch.tensor([7, 7, 7, 1, 0, -5], device="cuda")
    y = hq.hqq_rope(x, pos, t)
    clean = hq.hqq_rope(torch.ones_like(x), pos, t)
    for i, pair in ((0, (3, 19)), (1, (1, 17)), (3, (5, 21))):
        keep = [c for c in range(64) if c not in pair]
        assert torch.equal(y[i, 0, keep], clean[i, 0, keep]) and not torch.isfinite(y[i, 0, list(pair)]).all()
    assert torch.isnan(y[0, 0, [3, 19]]).all() and torch.isnan(y[2, 0, 40])
    assert torch.equal(y[4], x[4])                                           # position 0


def test_many_tokens_and_far_offsets():
    """More tokens than one dimension of blocks times a block, and token strides that pass 2^32 elements."""
    hq, torch = base.lib()
    t, freqs, m = table(torch, hq, 64, False, 1.0)
    n = 300001
    pos = torch.arange(n, device="cuda")
    x = torch.randn(n, 1, 64, device="cuda").half()
    y = hq.hqq_rope(x, pos, t)
    at = torch.tensor([0, 1, 65535 * 4, 65536 * 4, n - 1], device="cuda")
    want, size = turned(x[at].double().cpu().numpy(), at.cpu().numpy(), freqs, m, False, False)
    check(y[at], want, size, "float16", "many")
    far = torch.empty((1 << 32) + 4096, dtype=torch.float16, device="cuda")
    q = far.as_strided((3, 2, 64), (1 << 31, 64, 1))
    q.copy_(x[:6].view(3, 2, 64))
    near = hq.hqq_rope(x[:6].view(3, 2, 64), pos[:3], t)
    assert torch.equal(hq.hqq_rope(q, pos[:3], t), near)
    hq.hqq_rope(q, pos[:3], t, out=q)
    assert torch.equal(q, near)


# ------------------------------------------------------------------------------ into the cache

@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("d,bits,g", base.FORMATS)
def test_write_rope(d, bits, g, dtype):
    """The bits of hqq_rope and hqq_kv_write: pages, echo and queries, in every format; slots outside the cache; special values."""
    hq, torch = base.lib()
    dt = getattr(torch, dtype)
    for i, (page, hkv, n, q_heads, rot, inter) in enumerate(((16, 3, 37, 7, d, False), (64, 1, 1, 1, d // 2, True), (256, 2, 70, 16, 32, False),
                                                             (32, 5, 9, 0, 16, False), (128, 4, 33, 9, d, True), (32, 2, 6, 3, 48, False))):
        say("write rope", d, bits, g, dtype, page, hkv, n, q_heads, rot, inter)
        f = kp.Fmt(hkv, d, bits, g, page)
        rng = np.random.default_rng(d + bits + g + n)
        a, b = (base.make_cache(hq, torch, f, 9, fill=0xA5) for _ in range(2))
        k, v = (kp.to(x, dt).cuda() for x in base.values(rng, n, hkv, d, special=True))
        q = kp.to(rng.normal(size=(n, q_heads, d)).astype(np.float32), dt).cuda()
        slots = rng.permutation(9 * page)[:n].astype(np.int64)
        if n > 8:
            slots[6], slots[7], slots[8] = -1, 9 * page, -(1 << 40)
        slots = torch.from_numpy(slots).cuda()
        pos = torch.from_numpy(rng.integers(0, 100000, n)).cuda()
        t, _, _ = table(torch, hq, rot, inter, (1.0, 8.0)[i % 2])
        kr = hq.hqq_rope(k, pos, t)
        want = hq.hqq_kv_write(a, kr, v, slots, echo=True)
        got = hq.hqq_kv_write_rope(b, q, k, v, pos, slots, t, echo=True)
        if q_heads:
            assert torch.equal(got[0], hq.hqq_rope(q, pos, t))
        for x, y in zip(want, got[1:]):
            assert torch.equal(x.view(torch.int16), y.view(torch.int16))
        assert torch.equal(a.pages, b.pages)
        c = base.make_cache(hq, torch, f, 9, fill=0xA5)      # without the echo, q in place
        q0 = q.clone()
        assert hq.hqq_kv_write_rope(c, q0, k, v, pos, slots, t, out=q0) is q0
        assert torch.equal(c.pages, a.pages) and torch.equal(q0, got[0])


def test_write_rope_strides_streams_and_graph():
    """Slices of one projection; a side stream while the current one allocates; captured and replayed with new inputs."""
    hq, torch = base.lib()
    f = kp.Fmt(2, 128, 4, 64, 32)
    n = 18
    t, _, _ = table(torch, hq, 128, False, 1.0)
    rng = np.random.default_rng(9)
    qkv = kp.to(rng.normal(size=(n, 12, 128)).astype(np.float32), torch.float16).cuda()
    q, k, v = qkv[:, :8], qkv[:, 8:10], qkv[:, 10:]
    pos, slots = torch.arange(n, device="cuda") + 500, torch.from_numpy(rng.permutation(96)[:n].astype(np.int64)).cuda()
    a, b = (base.make_cache(hq, torch, f, 3, fill=0) for _ in range(2))
    want = hq.hqq_kv_write_rope(a, q.contiguous(), k.contiguous(), v.contiguous(), pos, slots, t, echo=True)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = []
    for rep in range(4):
        outs.append(hq.hqq_kv_write_rope(b, q, k, v, pos, slots, t, echo=True, stream=side) + (hq.hqq_rope(q, pos, t, stream=side),))
        junk = [torch.full((1 << 18,), float(rep), device="cuda") for _ in range(8)]
        del junk
    side.synchronize()
    for o in outs:
        assert all(torch.equal(x, y) for x, y in zip(o, want)) and torch.equal(o[3], want[0])
    assert torch.equal(a.pages, b.pages)

    def step():
        return hq.hqq_kv_write_rope(a, q, k, v, pos, slots, t, echo=True) + (hq.hqq_rope(k, pos, t, backward=True),)

    warm = torch.cuda.Stream()
    warm.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(warm):
        step()
    torch.cuda.current_stream().wait_stream(warm)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for rep in range(4):
        qkv.copy_(kp.to(rng.normal(size=tuple(qkv.shape)).astype(np.float32), torch.float16))
        pos += 1000 * rep + 1
        graph.replay()
        got = [x.clone() for x in out]
        pages = a.pages.clone()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, step())) and torch.equal(pages, a.pages)
        torch.cuda.synchronize()
