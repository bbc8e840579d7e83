"""Which kernels a call of the attention takes (hqq_kv_attention_way of csrc/hqq_kv.h), for tests that have to reach one."""
import collections
import ctypes

import weight_only_quantization_amd as hq
from weight_only_quantization_amd import kv_cache as kc

SHARES, ONCE, WHOLE8, WHOLE4, TILES = 0, 1, 2, 3, -1
# rows of a block (0: no such list), mode, key splits of the own keys and of the prefix; whether a join follows
Way = collections.namedtuple("Way", "rows mode splits prefix_rows prefix_mode prefix_splits join")


def way_of(packed):
    """Way of a call's arguments (packed bytes or a KvAttentionArgs); the status where it would be refused."""
    out = (ctypes.c_int32 * 7)()
    fn = hq.load().hqq_kv_attention_way
    fn.argtypes, fn.restype = [ctypes.c_char_p, ctypes.c_int32 * 7], ctypes.c_int
    status = fn(packed if isinstance(packed, bytes) else bytes(packed), out)
    return Way(*out) if status == 0 else status


def record(monkeypatch):
    """List that every call of the binding's attention appends its way to."""
    ways = []
    hq.load()
    for name in ("hqq_kv_attention", "hqq_kv_attention_shared"):
        def call(packed, entry=kc._fast[name]):
            ways.append(way_of(packed))
            return entry(packed)
        monkeypatch.setitem(kc._fast, name, call)
    return ways
