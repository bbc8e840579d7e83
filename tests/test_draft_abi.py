"""Refusals of rotary positions, drafted trees and the cache's moves on the CPU: every check answers before any launch, in the C ABI
(status and message) and in the binding (before a pointer crosses it); and what needs no launch: the frequencies, empty calls, sizes."""
import ctypes
import math

import pytest
import torch

import weight_only_quantization_amd as hq
from tests.kv_ways import ONCE, SHARES, WHOLE8
from tests.test_kv_abi import BAD, CACHE, FAKE, UNSUP, WS, cache, lib  # noqa: F401
from weight_only_quantization_amd import kv_cache as kc
from weight_only_quantization_amd import kv_pages as kp
from weight_only_quantization_amd import rotary as ro


def form(**kw):
    a = dict(freqs=FAKE, rot_dim=128, layout=0, magnitude=1.0)
    a.update(kw)
    return ro.RopeForm(**a)


def rope(lib, f=None, **kw):  # noqa: F811
    a = dict(form=f or form(), dtype=0, head_dim=128, backward=0, n=3, positions=FAKE, q=FAKE, q_token_stride=1024, q_head_stride=128,
             q_heads=8, q_out=FAKE + 4096, q_out_token_stride=1024, q_out_head_stride=128, k=FAKE, k_token_stride=256,
             k_head_stride=128, k_heads=2, k_out=FAKE + 4096, k_out_token_stride=256, k_out_head_stride=128, stream=None)
    a.update(kw)
    return lib.hqq_rope(ro.RopeArgs(**a))


FORMS = [(dict(rot_dim=0), BAD), (dict(rot_dim=144), BAD), (dict(rot_dim=120), UNSUP), (dict(rot_dim=-16), BAD), (dict(layout=2), BAD),
         (dict(magnitude=float("nan")), BAD), (dict(magnitude=float("inf")), BAD), (dict(freqs=None), BAD), (dict(freqs=FAKE + 4), BAD)]


@pytest.mark.parametrize("kw,status", FORMS)
def test_form_refused(lib, kw, status):  # noqa: F811
    assert rope(lib, form(**kw)) == status and hq.last_error()
    assert write_rope(lib, form(**kw)) == status and hq.last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), BAD), (dict(head_dim=0), BAD), (dict(head_dim=136), UNSUP), (dict(head_dim=1040), UNSUP), (dict(backward=2), BAD),
    (dict(n=-1), BAD), (dict(n=1 << 40), UNSUP), (dict(positions=None), BAD), (dict(positions=FAKE + 4), BAD), (dict(q=None), BAD),
    (dict(q=FAKE + 2), BAD), (dict(q_out=None), BAD), (dict(q_out=FAKE + 8), BAD), (dict(q_token_stride=1028), BAD),
    (dict(q_head_stride=-128), BAD), (dict(q_out_head_stride=4), BAD), (dict(k=None), BAD), (dict(k_out=FAKE + 1), BAD),
    (dict(q_heads=-1), BAD), (dict(k_heads=1 << 20), BAD), (dict(q_out=FAKE, q_out_token_stride=2048), BAD),
    (dict(k_out=FAKE, k_out_head_stride=256), BAD)])
def test_rope_refused(lib, kw, status):  # noqa: F811
    assert rope(lib, **kw) == status and hq.last_error()


def write_rope(lib, f=None, c=None, w=None, **kw):  # noqa: F811
    a = dict(cache=c or cache(), dtype=0, k=FAKE, v=FAKE, n=3, k_token_stride=256, k_head_stride=128, v_token_stride=256,
             v_head_stride=128, slots=FAKE, k_echo=None, v_echo=None, stream=None)
    a.update(w or {})
    b = dict(write=kc.KvWriteArgs(**a), form=f or form(), positions=FAKE, q=FAKE, q_token_stride=1024, q_head_stride=128, q_heads=8,
             q_out=FAKE + 4096, q_out_token_stride=1024, q_out_head_stride=128)
    b.update(kw)
    return lib.hqq_kv_write_rope(ro.KvWriteRopeArgs(**b))


@pytest.mark.parametrize("kw,status", CACHE)
def test_cache_refused(lib, kw, status):  # noqa: F811
    assert write_rope(lib, c=cache(**kw)) == status and hq.last_error()
    kw = {k: v for k, v in kw.items() if k != "pages"} or dict(head_dim=96)
    status = UNSUP if kw == dict(head_dim=96) else status
    for call in (accept, fork, compact):
        assert call(lib, c=cache(**kw)) == status and hq.last_error(), call


@pytest.mark.parametrize("w,kw,status", [
    (dict(dtype=3), {}, BAD), (dict(n=-1), {}, BAD), (dict(k=None), {}, BAD), (dict(slots=FAKE + 4), {}, BAD), (dict(k_echo=FAKE), {}, BAD),
    (dict(v_head_stride=4), {}, BAD), ({}, dict(positions=None), BAD), ({}, dict(q=None), BAD), ({}, dict(q_out=FAKE + 8), BAD),
    ({}, dict(q_heads=-1), BAD), ({}, dict(q_token_stride=100), BAD), ({}, dict(q_out=FAKE, q_out_head_stride=256), BAD)])
def test_write_rope_refused(lib, w, kw, status):  # noqa: F811
    assert write_rope(lib, w=w, **kw) == status and hq.last_error()


@pytest.mark.parametrize("args,status", [
    ((0, 1e4, 0, 1.0, 0, 32, 1), BAD), ((24, 1e4, 0, 1.0, 0, 32, 1), UNSUP), ((1040, 1e4, 0, 1.0, 0, 32, 1), BAD), ((64, 1.0, 0, 1.0, 0, 32, 1), BAD),
    ((64, float("inf"), 0, 1.0, 0, 32, 1), BAD), ((64, 1e4, 4, 1.0, 0, 32, 1), BAD), ((64, 1e4, -1, 1.0, 0, 32, 1), BAD),
    ((64, 1e4, 1, 0.5, 0, 32, 1), BAD), ((64, 1e4, 1, float("nan"), 0, 32, 1), BAD), ((64, 1e4, 3, 2.0, 0, 32, 1), BAD),
    ((64, 1e4, 3, 2.0, 4096, 1, 1), BAD), ((64, 1e4, 3, 2.0, 4096, 32, 0), BAD)])
def test_frequencies_refused(lib, args, status):  # noqa: F811
    f = (ctypes.c_double * 512)()
    assert lib.hqq_rope_frequencies(*args, ctypes.addressof(f), None) == status and hq.last_error()
    assert lib.hqq_rope_frequencies(64, 1e4, 0, 1.0, 0, 32, 1, None, None) == BAD


@pytest.mark.parametrize("rot,base", [(128, 1e4), (64, 5e5), (16, 10.0), (1024, 1e6)])
def test_frequencies(lib, rot, base):  # noqa: F811
    """Against the formulas, to a few units of 64 bits (powers and logarithms)."""
    half, factor, length = rot // 2, 7.5, 4096.0
    plain = [base ** (-2 * i / rot) for i in range(half)]

    def close(table, want, magnitude):
        got = table.freqs.tolist()
        assert len(got) == half and table.magnitude == pytest.approx(magnitude, rel=1e-15)
        assert all(abs(a - b) <= 1e-13 * b for a, b in zip(got, want))

    def make(**kw):
        return hq.hqq_rope_table(rot, base, device="cpu", **kw)

    close(make(), plain, 1.0)
    close(make(scaling="linear", factor=factor), [f / factor for f in plain], 1.0)
    raised = base * factor ** (rot / (rot - 2))
    close(make(scaling="base", factor=factor), [raised ** (-2 * i / rot) for i in range(half)], 1.0)
    assert make(scaling="base", factor=factor).freqs[-1] == pytest.approx(plain[-1] / factor, rel=1e-12)
    low, high = (rot * math.log(length / (2 * math.pi * n)) / (2 * math.log(base)) for n in (32.0, 1.0))
    low, high = max(math.floor(low), 0), min(math.ceil(high), rot - 1)
    ramp = [min(max((i - low) / max(high - low, 0.001), 0.0), 1.0) for i in range(half)]
    close(make(scaling="bands", factor=factor, original_len=length), [f * (1 - r) + f / factor * r for f, r in zip(plain, ramp)],
          0.1 * math.log(factor) + 1)
    close(make(scaling="bands", factor=1.0, original_len=length), plain, 1.0)
    with pytest.raises(ValueError, match="scaling"):
        make(scaling="other")
    with pytest.raises(hq.HQQError):
        make(scaling="bands", factor=2.0)


@pytest.mark.parametrize("kw,fits", [
    (dict(q_out_token_stride=0), False), (dict(q_out_head_stride=0), False), (dict(q_out_head_stride=120), False),
    (dict(q_out_token_stride=1016), False), (dict(q_out_token_stride=128, q_out_head_stride=384), True),
    (dict(q_out_token_stride=128, q_out_head_stride=376), False), (dict(q_out_token_stride=120, q_out_head_stride=384), False),
    (dict(q_out_token_stride=128), False), (dict(q_heads=1, q_out_head_stride=0), True), (dict(n=1, q_out_token_stride=0), True),
    (dict(q_heads=1, q_out_token_stride=64), False), (dict(q_heads=0, q_out_token_stride=0), True),
    (dict(q_token_stride=0, q_head_stride=0), True), (dict(k_out_token_stride=128), False)])
def test_outputs_apart(lib, kw, fits):  # noqa: F811
    """Outputs whose heads share memory are refused, broadcast inputs are not (the call then stops at k, which is refused)."""
    kw = dict(kw) if "k_out_token_stride" in kw else dict(k=FAKE + 2, **kw)
    assert rope(lib, **kw) == BAD
    assert ("heads of an output overlap" in hq.last_error()) == (not fits)


# ------------------------------------------------------------------------------ trees

def plan(lib, **kw):  # noqa: F811
    a = dict(parents=FAKE, total_q=8, num_seqs=2, cu_q=None, max_q=0, page_table=FAKE, table_stride=9, table_cols=9, seq_lens=FAKE,
             page_size=64, mask=FAKE, mask_words=1, positions=FAKE, slots=FAKE, stream=None)
    a.update(kw)
    return lib.hqq_kv_tree_plan(kp.KvTreePlanArgs(**a))


@pytest.mark.parametrize("kw,status", [
    (dict(total_q=-1), BAD), (dict(total_q=7), BAD), (dict(num_seqs=0), BAD), (dict(num_seqs=-1), BAD), (dict(num_seqs=70000, total_q=70000), UNSUP),
    (dict(cu_q=FAKE, max_q=9), BAD), (dict(cu_q=FAKE + 2, max_q=4), BAD), (dict(table_cols=-1), BAD), (dict(table_cols=1 << 26), BAD),
    (dict(table_stride=-1), BAD), (dict(page_table=None), BAD), (dict(page_table=FAKE + 2), BAD), (dict(seq_lens=None), BAD),
    (dict(seq_lens=FAKE + 1), BAD), (dict(page_size=0), BAD), (dict(page_size=48), UNSUP), (dict(mask=None), BAD), (dict(mask=FAKE + 4), BAD),
    (dict(mask_words=0), BAD), (dict(mask_words=65), BAD), (dict(total_q=130), BAD), (dict(parents=None), BAD), (dict(parents=FAKE + 2), BAD),
    (dict(positions=FAKE + 4), BAD), (dict(slots=FAKE + 4), BAD)])
def test_plan_refused(lib, kw, status):  # noqa: F811
    assert plan(lib, **kw) == status and hq.last_error()


def tree(lib, c=None, mask=FAKE, mask_words=1, **kw):  # noqa: F811
    a = dict(cache=c or cache(), dtype=0, q=FAKE, total_q=4, q_token_stride=1024, q_head_stride=128, num_q_heads=8,
             num_seqs=2, cu_q=None, max_q=0, page_table=FAKE, table_stride=100, table_cols=100, seq_lens=FAKE, max_len=6400,
             causal=1, scale=0.1, prefix_table=None, prefix_len=0, out=FAKE, lse=None, workspace=FAKE, workspace_bytes=0, stream=None)
    a.update(kw)
    return lib.hqq_kv_attention_tree(kc.KvTreeArgs(attention=kc.KvAttentionArgs(**a), mask=mask, mask_words=mask_words))


@pytest.mark.parametrize("kw,status", [
    (dict(mask=None), BAD), (dict(mask=FAKE + 4), BAD), (dict(mask_words=0), BAD), (dict(mask_words=65), BAD), (dict(total_q=130), BAD),
    (dict(cu_q=FAKE, max_q=4, total_q=4, mask_words=-1), BAD), (dict(dtype=7), BAD), (dict(total_q=5), BAD), (dict(num_q_heads=7), BAD),
    (dict(scale=0.0), BAD), (dict(q=None), BAD), (dict(seq_lens=None), BAD), (dict(page_table=None), BAD), (dict(prefix_len=3), BAD),
    (dict(causal=2), BAD), (dict(workspace=None), WS), (dict(workspace_bytes=64), WS), (dict(total_q=70000, num_seqs=70000), UNSUP)])
def test_tree_refused(lib, kw, status):  # noqa: F811
    assert tree(lib, **kw) == status and hq.last_error()


@pytest.mark.parametrize("kw,status", CACHE)
def test_tree_cache_refused(lib, kw, status):  # noqa: F811
    assert tree(lib, c=cache(**kw)) == status


def tree_way(rows, hkv, seqs, keys, prefix=0):
    """Of drafts of `rows` query rows a KV head (one head a KV head)."""
    out = (ctypes.c_int32 * 7)()
    fn = hq.load().hqq_kv_attention_tree_way
    fn.argtypes, fn.restype = [ctypes.POINTER(kc.KvTreeArgs), ctypes.c_int32 * 7], ctypes.c_int
    a = kc.KvAttentionArgs(cache=cache(num_kv_heads=hkv), dtype=0, q=FAKE, total_q=rows * seqs, num_q_heads=hkv, q_token_stride=1024,
                           q_head_stride=128, num_seqs=seqs, page_table=FAKE, table_stride=0, table_cols=1 << 20, seq_lens=FAKE,
                           max_len=keys, causal=1, scale=0.1, prefix_table=FAKE if prefix else None, prefix_len=prefix, out=FAKE)
    assert fn(kc.KvTreeArgs(attention=a, mask=FAKE, mask_words=8), out) == 0
    return tuple(out)


@pytest.mark.parametrize("call,want", [
    ((16, 8, 16, 2048), (16, WHOLE8, 1, 0, 0, 0, 0)), ((16, 8, 16, 2049), (16, ONCE, 1, 0, 0, 0, 1)), ((64, 8, 17, 1 << 20), (32, SHARES, 1, 0, 0, 0, 1)),
    # shares of tiles: past 3 * 2^23 pairs of a row and a key, up to 2048 keys past 3 * 2^24
    ((96, 8, 8, 4096), (32, SHARES, 1, 0, 0, 0, 1)), ((96, 8, 8, 4097), (128, SHARES, 1, 0, 0, 0, 1)),
    ((129, 8, 8, 4096), (256, SHARES, 1, 0, 0, 0, 1)), ((128, 8, 24, 2048), (32, WHOLE8 + 1, 1, 0, 0, 0, 0)),
    ((128, 8, 25, 2048), (128, SHARES, 1, 0, 0, 0, 1)),
    # with a prefix
    ((1, 8, 16, 200, 300), (16, ONCE, 1, 16, ONCE, 1, 1)), ((128, 8, 25, 2048, 16), (128, SHARES, 1, 32, SHARES, 1, 1)),
    ((129, 8, 25, 2048, 4000), (256, SHARES, 1, 256, -1, 2, 1))])
def test_tree_ways(lib, call, want):  # noqa: F811
    assert tree_way(*call) == want


# ------------------------------------------------------------------------------ moves

def layers(c=None, **kw):
    """hqq_kv_layers of three layers (the host array is kept with it)."""
    pages = (ctypes.c_void_p * 200)(*([FAKE] * 200))
    a = dict(cache=c or cache(pages=None), pages=ctypes.addressof(pages), num_layers=3)
    a.update(kw)
    x = kp.KvLayersArgs(**a)
    x.keep = pages
    return x


TABLE = dict(num_seqs=2, page_table=FAKE, table_stride=9, table_cols=9, seq_lens=FAKE)


def accept(lib, c=None, l=None, **kw):  # noqa: F811
    a = dict(layers=l or layers(c), total_q=8, cu_q=None, max_q=0, accepted=FAKE, accepted_stride=4, max_accepted=4, num_accepted=FAKE,
             new_lens=FAKE, stream=None, **TABLE)
    a.update(kw)
    return lib.hqq_kv_accept(kp.KvAcceptArgs(**a))


def fork(lib, c=None, l=None, **kw):  # noqa: F811
    a = dict(layers=l or layers(c), num_new=3, parents=FAKE, fresh=FAKE, new_table=FAKE, new_stride=9, new_lens=FAKE, stream=None, **TABLE)
    a.update(kw)
    return lib.hqq_kv_fork(kp.KvForkArgs(**a))


def compact(lib, c=None, l=None, **kw):  # noqa: F811
    a = dict(layers=l or layers(c), new_table=FAKE, new_stride=9, used=FAKE, workspace=FAKE, workspace_bytes=1 << 30, stream=None, **TABLE)
    a.update(kw)
    return lib.hqq_kv_compact(kp.KvCompactArgs(**a))


@pytest.mark.parametrize("call", [accept, fork, compact])
@pytest.mark.parametrize("kw,status", [(dict(num_layers=0), BAD), (dict(num_layers=129), BAD), (dict(pages=None), BAD)])
def test_layers_refused(lib, call, kw, status):  # noqa: F811
    assert call(lib, l=layers(**kw)) == status and hq.last_error()


@pytest.mark.parametrize("call", [accept, fork, compact])
def test_layers_pointers(lib, call):  # noqa: F811
    for bad in (0, FAKE + 8):
        x = layers()
        x.keep[2] = bad
        assert call(lib, l=x) == BAD and hq.last_error()


@pytest.mark.parametrize("call", [accept, fork, compact])
@pytest.mark.parametrize("kw,status", [
    (dict(num_seqs=-1), BAD), (dict(num_seqs=70000, total_q=70000), UNSUP), (dict(page_table=None), BAD), (dict(seq_lens=None), BAD),
    (dict(seq_lens=FAKE + 2), BAD), (dict(table_cols=-1), BAD), (dict(table_cols=1 << 26, new_stride=1 << 26), BAD), (dict(table_stride=-1), BAD)])
def test_tables_refused(lib, call, kw, status):  # noqa: F811
    mine = {k: v for k, v in kw.items() if k not in ("total_q", "new_stride") or (k == "total_q") == (call is accept)}
    assert call(lib, **mine) == status and hq.last_error()


@pytest.mark.parametrize("call,kw,status", [
    (accept, dict(total_q=7), BAD), (accept, dict(total_q=-2), BAD), (accept, dict(cu_q=FAKE, max_q=9), BAD), (accept, dict(cu_q=FAKE + 1, max_q=4), BAD),
    (accept, dict(accepted=None), BAD), (accept, dict(accepted=FAKE + 2), BAD), (accept, dict(max_accepted=-1), BAD),
    (accept, dict(accepted_stride=-1), BAD), (accept, dict(num_accepted=None), BAD), (accept, dict(new_lens=None), BAD),
    (accept, dict(new_lens=FAKE + 2), BAD),
    (accept, dict(c=cache(pages=None, num_kv_heads=4096), total_q=1 << 21, max_accepted=1 << 20), UNSUP),
    (fork, dict(num_new=-1), BAD), (fork, dict(num_new=70000), UNSUP), (fork, dict(num_seqs=0), BAD), (fork, dict(parents=None), BAD),
    (fork, dict(fresh=None), BAD), (fork, dict(fresh=FAKE + 2), BAD), (fork, dict(new_table=None), BAD), (fork, dict(new_stride=8), BAD),
    (fork, dict(new_lens=None), BAD),
    (compact, dict(new_table=None), BAD), (compact, dict(new_stride=8), BAD), (compact, dict(used=None), BAD), (compact, dict(used=FAKE + 2), BAD),
    (compact, dict(workspace=None), WS), (compact, dict(workspace_bytes=16), WS), (compact, dict(workspace=FAKE + 8), BAD),
    (compact, dict(c=cache(pages=None, num_pages=(1 << 20) + 1)), UNSUP)])
def test_moves_refused(lib, call, kw, status):  # noqa: F811
    assert call(lib, **kw) == status and hq.last_error()


def test_nothing_to_do(lib):  # noqa: F811
    assert rope(lib, n=0, q=None, k=None, q_out=None, k_out=None, positions=None, f=form(freqs=None)) == hq.HQQ_OK
    assert rope(lib, q_heads=0, k_heads=0, q=None, k=None, q_out=None, k_out=None) == hq.HQQ_OK
    assert write_rope(lib, w=dict(n=0, k=None, v=None, slots=None), q=None, q_out=None, positions=None) == hq.HQQ_OK
    assert plan(lib, total_q=0, num_seqs=0, parents=None, mask=None) == hq.HQQ_OK
    assert plan(lib, cu_q=FAKE, max_q=0, parents=None, mask=None) == hq.HQQ_OK
    assert tree(lib, total_q=0, num_seqs=0, q=None, out=None, mask=None) == hq.HQQ_OK
    assert accept(lib, num_seqs=0, total_q=0, accepted=None, num_accepted=None, new_lens=None) == hq.HQQ_OK
    assert fork(lib, num_new=0, parents=None, fresh=None, new_table=None, new_lens=None) == hq.HQQ_OK
    for f in (lib.hqq_rope, lib.hqq_kv_write_rope, lib.hqq_kv_tree_plan, lib.hqq_kv_attention_tree, lib.hqq_kv_accept, lib.hqq_kv_fork,
              lib.hqq_kv_compact):
        assert f(None) == BAD
    assert lib.hqq_kv_attention_tree_workspace_bytes(None) == 0


def test_sizes(lib):  # noqa: F811
    assert hq.hqq_kv_compact_workspace_bytes(0) == 0 and hq.hqq_kv_compact_workspace_bytes((1 << 20) + 1) == 0
    assert hq.hqq_kv_compact_workspace_bytes(7) == 4 * (4 + 2 * 4 + 7)
    a = kc.KvAttentionArgs(cache=cache(pages=None), total_q=1, num_q_heads=8, num_seqs=1, table_cols=100, table_stride=100, max_len=100,
                           scale=1.0)
    assert lib.hqq_kv_attention_tree_workspace_bytes(kc.KvTreeArgs(attention=a)) == 0
    a.max_len = 6400
    assert lib.hqq_kv_attention_tree_workspace_bytes(kc.KvTreeArgs(attention=a)) > 0


def test_binding_checks(lib):  # noqa: F811
    f16 = torch.float16
    table = hq.RopeTable(torch.ones(64, dtype=torch.float64))
    q, k = torch.zeros(3, 8, 128, dtype=f16), torch.zeros(3, 2, 128, dtype=f16)
    pos = torch.zeros(3, dtype=torch.int64)
    with pytest.raises(ValueError, match="positions must be torch.int64"):
        hq.hqq_rope(q, pos.int(), table)
    with pytest.raises(ValueError, match="positions must be"):
        hq.hqq_rope(q, pos[:2], table)
    with pytest.raises(ValueError, match="float16 or torch.bfloat16"):
        hq.hqq_rope(q.float(), pos, table)
    with pytest.raises(ValueError, match="CUDA"):
        hq.hqq_rope(q, pos, table)
    with pytest.raises(ValueError, match="freqs"):
        hq.RopeTable(torch.ones(64)).args()
    with pytest.raises(ValueError, match="CUDA"):
        table.args()
    c = hq.KVCache(torch.zeros(4, hq.hqq_kv_page_bytes(2, 128), dtype=torch.uint8), 2, 128)
    with pytest.raises(ValueError, match="one dtype"):
        hq.hqq_kv_write_rope(c, q, k, k.bfloat16(), pos, pos, table)
    with pytest.raises(ValueError, match="same number"):
        hq.hqq_kv_write_rope(c, q, k, k[:2], pos, pos, table)
    with pytest.raises(ValueError, match="k must be"):
        hq.hqq_kv_write_rope(c, q, k[:, :1], k, pos, pos, table)
    with pytest.raises(ValueError, match="CUDA"):
        hq.hqq_kv_write_rope(c, q, k, k, pos, pos, table)
    lens, pages = torch.zeros(2, dtype=torch.int32), torch.zeros(2, 5, dtype=torch.int32)
    with pytest.raises(ValueError, match="parents must be torch.int32"):
        hq.hqq_kv_tree_plan(torch.zeros(4, dtype=torch.int64), pages, lens, 64)
    with pytest.raises(ValueError, match="seq_lens must be"):
        hq.hqq_kv_tree_plan(torch.zeros(4, dtype=torch.int32), pages, lens[:1], 64)
    with pytest.raises(ValueError, match="CUDA"):
        hq.hqq_kv_tree_plan(torch.zeros(4, dtype=torch.int32), pages, lens, 64)
    with pytest.raises(ValueError, match="mask must be"):
        hq.hqq_kv_attention_tree(c, q, torch.zeros(2, 1, dtype=torch.int64), pages, lens)
    with pytest.raises(ValueError, match="mask must be torch.int64"):
        hq.hqq_kv_attention_tree(c, q, torch.zeros(3, 1, dtype=torch.int32), pages, lens)
    with pytest.raises(ValueError, match="CUDA"):
        hq.KVLayers([c])
    with pytest.raises(ValueError, match="1 .. 128 layers"):
        hq.KVLayers([])
