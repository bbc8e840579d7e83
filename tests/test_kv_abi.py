"""Refusals of the quantised key/value cache's entry points on the CPU: every check answers before any launch, in
the C ABI (status and message) and in the binding (before a pointer crosses it)."""
import ctypes
import os

import pytest
import torch

import weight_only_quantization_amd as hq
from weight_only_quantization_amd import kv_cache as kc

FAKE = 1 << 20  # aligned, never dereferenced: every case below fails validation
BAD, UNSUP, WS = hq.HQQ_ERR_INVALID_ARGUMENT, hq.HQQ_ERR_UNSUPPORTED, hq.HQQ_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(hq.LIB_PATH):
        from weight_only_quantization_amd import build
        build.build()
    return hq.load()


def cache(**kw):
    a = dict(pages=FAKE, num_pages=8, num_kv_heads=2, head_dim=128, nbits=4, group_size=64, page_size=64)
    a.update(kw)
    return kc.KvCacheArgs(**a)


CACHE = [(dict(pages=None), BAD), (dict(pages=FAKE + 8), BAD), (dict(num_pages=0), BAD), (dict(num_pages=1 << 31), BAD),
         (dict(num_kv_heads=0), BAD), (dict(head_dim=96), UNSUP), (dict(nbits=3), UNSUP), (dict(nbits=9), BAD),
         (dict(group_size=16), UNSUP), (dict(group_size=0), BAD), (dict(head_dim=64, group_size=128), UNSUP),
         (dict(page_size=48), UNSUP), (dict(page_size=0), BAD), (dict(page_size=512), UNSUP)]


def attention(lib, entry="hqq_kv_attention", c=None, **kw):
    a = dict(cache=c or cache(), dtype=0, q=FAKE, total_q=4, q_token_stride=1024, q_head_stride=128, num_q_heads=8,
             num_seqs=2, cu_q=None, max_q=0, page_table=FAKE, table_stride=100, table_cols=100, seq_lens=FAKE, max_len=6400,
             causal=1, scale=0.1, prefix_table=None, prefix_len=0, out=FAKE, lse=None, workspace=FAKE,
             workspace_bytes=0, stream=None)
    a.update(kw)
    return getattr(lib, entry)(kc.KvAttentionArgs(**a))


def write(lib, c=None, **kw):
    a = dict(cache=c or cache(), dtype=0, k=FAKE, v=FAKE, n=3, k_token_stride=256, k_head_stride=128, v_token_stride=256,
             v_head_stride=128, slots=FAKE, k_echo=None, v_echo=None, stream=None)
    a.update(kw)
    return lib.hqq_kv_write(kc.KvWriteArgs(**a))


def read(lib, c=None, **kw):
    a = dict(cache=c or cache(), dtype=0, n=3, slots=FAKE, k=FAKE, v=FAKE, stream=None)
    a.update(kw)
    return lib.hqq_kv_read(kc.KvReadArgs(**a))


@pytest.mark.parametrize("kw,status", CACHE)
def test_cache_refused(lib, kw, status):
    assert write(lib, cache(**kw)) == status and hq.last_error()
    assert read(lib, cache(**kw)) == status
    assert attention(lib, c=cache(**kw)) == status
    assert attention(lib, "hqq_kv_attention_shared", c=cache(**kw)) == status


def test_page_bytes(lib):
    assert hq.hqq_kv_page_bytes(8, 128, 4, 64, 64) == 8 * 64 * 2 * (64 + 8)
    assert hq.hqq_kv_page_bytes(1, 64, 8, 32, 16) == 16 * 2 * (64 + 8)
    for bad in ((8, 80, 4, 16, 64), (0, 128, 4, 64, 64), (8, 128, 2, 64, 64), (8, 128, 4, 64, 20), (5000, 128, 4, 64, 64)):
        assert hq.hqq_kv_page_bytes(*bad) == 0
    with pytest.raises(hq.HQQError):
        hq.hqq_kv_cache(4, 8, 80, device="cpu")


@pytest.mark.parametrize("kw", [dict(dtype=2), dict(n=-1), dict(n=1 << 40), dict(k=None), dict(v=None), dict(slots=None),
                                dict(k=FAKE + 2), dict(slots=FAKE + 4), dict(k_token_stride=257), dict(v_head_stride=4),
                                dict(k_token_stride=-256), dict(k_echo=FAKE), dict(v_echo=FAKE),
                                dict(k_echo=FAKE + 8, v_echo=FAKE)])
def test_write_refused(lib, kw):
    assert write(lib, **kw) == BAD and hq.last_error()


@pytest.mark.parametrize("kw", [dict(dtype=-1), dict(n=-1), dict(k=None), dict(v=FAKE + 4), dict(slots=None)])
def test_read_refused(lib, kw):
    assert read(lib, **kw) == BAD and hq.last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=7), BAD), (dict(total_q=-1), BAD), (dict(total_q=5), BAD), (dict(num_seqs=0), BAD), (dict(num_q_heads=7), BAD),
    (dict(num_q_heads=0), BAD), (dict(cu_q=FAKE, max_q=5), BAD), (dict(cu_q=FAKE, max_q=-1), BAD), (dict(max_len=-1), BAD),
    (dict(max_len=1 << 31), BAD), (dict(prefix_len=-1), BAD), (dict(prefix_len=3), BAD), (dict(prefix_table=FAKE), BAD),
    (dict(table_cols=-1), BAD), (dict(table_cols=1 << 26, table_stride=1 << 26), BAD), (dict(table_stride=-1), BAD), (dict(causal=2), BAD),
    (dict(scale=0.0), BAD), (dict(scale=-1.0), BAD), (dict(scale=float("inf")), BAD), (dict(scale=float("nan")), BAD),
    (dict(q=None), BAD), (dict(q=FAKE + 2), BAD), (dict(out=None), BAD), (dict(q_token_stride=1025), BAD),
    (dict(q_head_stride=-128), BAD), (dict(seq_lens=None), BAD), (dict(page_table=None), BAD), (dict(workspace=None), WS),
    (dict(workspace_bytes=64), WS), (dict(workspace=FAKE + 8, workspace_bytes=1 << 40), BAD),
    (dict(total_q=70000, num_seqs=70000), UNSUP)])
def test_attention_refused(lib, kw, status):
    assert attention(lib, **kw) == status and hq.last_error()


def test_shared_refused(lib):
    e = "hqq_kv_attention_shared"
    assert attention(lib, e, prefix_len=100) == BAD                      # no table
    assert attention(lib, e, prefix_len=-1, prefix_table=FAKE) == BAD
    assert attention(lib, e, prefix_len=100, prefix_table=FAKE) == WS     # the prefix adds its part
    for f in (lib.hqq_kv_write, lib.hqq_kv_read, lib.hqq_kv_attention, lib.hqq_kv_attention_shared):
        assert f(None) == BAD


def test_nothing_to_do(lib):
    assert write(lib, n=0, k=None, v=None, slots=None) == hq.HQQ_OK
    assert read(lib, n=0, k=None, v=None, slots=None) == hq.HQQ_OK
    assert attention(lib, total_q=0, num_seqs=0, q=None, out=None) == hq.HQQ_OK


def test_workspace_bytes(lib):
    a = kc.KvAttentionArgs(cache=cache(pages=None), total_q=1, num_q_heads=8, num_seqs=1, table_cols=100,
                           table_stride=100, max_len=100, scale=1.0)
    assert lib.hqq_kv_attention_workspace_bytes(a) == 0               # one part
    a.max_len = 6400
    one = lib.hqq_kv_attention_workspace_bytes(a)
    assert one > 0
    a.prefix_len = 1
    assert lib.hqq_kv_attention_workspace_bytes(a) > one
    assert lib.hqq_kv_attention_workspace_bytes(None) == 0


def test_binding_checks(lib):
    pb = hq.hqq_kv_page_bytes(2, 128)
    c = hq.KVCache(torch.zeros(4, pb, dtype=torch.uint8), 2, 128)
    k = torch.zeros(3, 2, 128, dtype=torch.float16)
    slots = torch.zeros(3, dtype=torch.int64)
    with pytest.raises(ValueError, match="slots must be torch.int64"):
        hq.hqq_kv_write(c, k, k, slots.int())
    with pytest.raises(ValueError, match="one dtype"):
        hq.hqq_kv_write(c, k, k.bfloat16(), slots)
    with pytest.raises(ValueError, match="float16 or torch.bfloat16"):
        hq.hqq_kv_write(c, k.float(), k.float(), slots)
    with pytest.raises(ValueError, match="same number"):
        hq.hqq_kv_write(c, k, k[:2], slots)
    with pytest.raises(ValueError, match="k must be"):
        hq.hqq_kv_write(c, k[:, :1], k, slots)
    with pytest.raises(ValueError, match="CUDA"):
        hq.hqq_kv_write(c, k, k, slots)
    with pytest.raises(ValueError, match="CUDA"):
        hq.hqq_kv_read(c, slots)
    with pytest.raises(TypeError):
        hq.hqq_kv_read(c, [0, 1])
    q = torch.zeros(3, 8, 128, dtype=torch.float16)
    table, lens = torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="q must be"):
        hq.hqq_kv_attention(c, q[..., :64], table, lens)
    with pytest.raises(ValueError, match="float16 or torch.bfloat16"):
        hq.hqq_kv_attention(c, q.float(), table, lens)
    with pytest.raises(ValueError, match="CUDA"):
        hq.hqq_kv_attention(c, q, table, lens)
    with pytest.raises(ValueError, match="CUDA"):
        c.args()
