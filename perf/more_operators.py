"""Measured cases of a drafted decode step on the quantised key/value cache: rotary positions (by themselves and on the
way into the cache), attention for a tree of drafted tokens, and moving cached tokens and pages: accepted drafts, forked
sequences, pools that have become full of holes.

A cache is uint8 [num_pages, Hkv, block] a layer; a block holds one KV head's keys and values of `page` tokens: K codes, V
codes, K metadata, V metadata (b bits a code, groups of g along the D channels).
  K codes      [page][4 h][D/32 i][8 j]         channel 32 i + 8 h + j of the token;  in 4 bits the eight codes of
               a word are its nibbles 0, 4, 1, 5, 2, 6, 3, 7 (j = 0 .. 7), in 8 bits its bytes in order
  V codes      [page/4][16 r][4 t][D/16 j]      channel (D/16) r + j of token 4 * (outer index) + t, lowest bits first
  K, V metadata [D/g][page] pairs of fp16: the step (low half), the floor (high half)
A value is floor + code * step.
"""
import math

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
DEV = "cuda"


def _case(name, op, **kw):
    c = dict(name=name, op=op, dtype="fp16", bits=4, g=64, d=128, page=64, hq=32, hkv=8)
    if op in ("rope", "write"):
        c.update(n=1, rot=128, inter=False, far=4096, factor=1.0)
        if op == "rope":
            c.update(back=False)
    elif op == "tree":
        c.update(batch=1, t=16, ragged=False, len=1024, lo=1024, prefix=0, plan=True)
    else:
        c.update(layers=32, batch=16, len=1000, lo=1000)
        c.update(dict(accept=dict(t=16, acc=4, ragged=False), fork=dict(new=16, kids=4), compact=dict(pool=512, prefix=0))[op])
    c.update(kw)
    return c


def listed():
    return [
        # queries and keys of one decode step of a serving batch (latency)
        _case("rope_step_b64", "rope", n=64, dtype="bf16"),
        # the gradient through the rotation of a training step's packed sequences, half of each head rotated, interleaved
        _case("rope_grad_16411", "rope", n=16411, hkv=32, far=9000, inter=True, rot=64, back=True),
        # a decode step's keys and values rotated on their way into the cache, far into a scaled context (latency)
        _case("write_step_b32", "write", n=32, far=100000, factor=8.0),
        # a batch's prompts of odd length, 64 query heads on 8, 8 bits
        _case("write_prompts_16387", "write", n=16387, hq=64, far=20000, bits=8, dtype="bf16", page=128),
        # one user's draft of 26 tokens, Llama-7B's heads (latency)
        _case("tree_b1", "tree", t=26, hkv=32, len=1049, lo=1049),
        # a serving batch with drafts of up to 32 tokens, grouped heads, ragged lengths
        _case("tree_b16_ragged", "tree", batch=16, t=32, ragged=True, len=4096, lo=200, bits=8, g=128, dtype="bf16"),
        # long contexts with full drafts of 64 tokens, 64 query heads on 8
        _case("tree_b8_long", "tree", batch=8, t=64, hq=64, len=16384, lo=9000, page=256, plan=False),
        # the accepted tokens of one user's draft, 32 layers (latency)
        _case("accept_b1", "accept", batch=1, t=26, acc=5, hkv=32, len=1049, lo=1049),
        # and of a large serving batch's drafts
        _case("accept_b128", "accept", batch=128, t=32, acc=9, ragged=True, len=800, lo=90),
        # beams that go on from a quarter of the sequences
        _case("fork_b64", "fork", batch=64, new=64, kids=4, len=513, lo=70),
        # a small pool of a few sequences with a common prefix, one layer (latency)
        _case("compact_l1", "compact", layers=1, batch=9, len=700, lo=5, pool=211, prefix=3),
        # the pages of a serving batch moved together after two thirds of the sequences have left
        _case("compact_l32", "compact", batch=48, len=2000, lo=300, pool=2600),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "rope", "write", "write", "tree", "tree", "tree", "accept", "accept", "fork", "compact"])
    d = rng.choice([64, 128, 128])
    kw = dict(dtype=rng.choice(["fp16", "bf16"]), bits=rng.choice([4, 4, 8]), d=d, g=rng.choice([x for x in (32, 64, 64, 128) if x <= d]),
              page=rng.choice([16, 32, 64, 128, 256]), hkv=rng.choice([1, 4, 8, 8, 32]))
    kw["hq"] = kw["hkv"] * (1 if kw["hkv"] == 32 else rng.choice([1, 3, 4, 7, 8]))
    if op in ("rope", "write"):
        if op == "rope":
            kw["d"] = rng.choice([64, 80, 96, 128, 128, 256])
            kw["back"] = rng.random() < 0.4
        heads = kw["hq"] + (1 + (op == "write")) * kw["hkv"]
        kw["n"] = _log(rng, 1, 16384 * 64 * 128 // (heads * kw["d"]))
        kw["rot"] = rng.choice([x for x in (kw["d"], kw["d"], kw["d"] // 2 // 16 * 16, 32) if x <= kw["d"]])
        kw["inter"] = rng.random() < 0.4
        kw["far"] = _log(rng, 1, 1000000)
        kw["factor"] = rng.choice([1.0, 1.0, 4.0, 32.0])
    elif op == "tree":
        kw["batch"] = _log(rng, 1, 48)
        kw["t"] = rng.choice([2, 5, 8, 13, 26, 33, 64, 100])
        kw["ragged"] = kw["batch"] > 1 and rng.random() < 0.5
        most = min(8 * 64 * 64 * 16384 // (kw["batch"] * kw["t"] * kw["hq"]), 8 * 16384 * 8 * 4 // (kw["bits"] * kw["batch"] * max(8, kw["hkv"])))
        kw["len"] = kw["t"] + _log(rng, 1, max(2, min(32768, most) - kw["t"])) - 1
        kw["lo"] = rng.randint(kw["t"], kw["len"])
        kw["prefix"] = _log(rng, 30, max(31, min(4096, most // 2))) if rng.random() < 0.25 else 0
        kw["plan"] = rng.random() < 0.6
    else:
        kw["layers"] = rng.choice([1, 2, 16, 32, 40])
        tokens = 48 * 1150 * 32 * 8 * 128 * 4 // (kw["layers"] * kw["hkv"] * kw["d"] * kw["bits"])
        kw["batch"] = _log(rng, 1, min(128, max(1, tokens // 200)))
        kw["len"] = _log(rng, 40, max(41, min(2000, tokens // kw["batch"] - kw["page"])))
        kw["lo"] = rng.randint(1, kw["len"])
        if op == "accept":
            kw["t"] = rng.choice([4, 7, 16, 26, 40])
            kw["acc"] = rng.randint(1, min(kw["t"], 12))
            kw["ragged"] = kw["batch"] > 1 and rng.random() < 0.5
            kw["lo"] = max(kw["lo"], kw["t"])
        elif op == "fork":
            kw["kids"] = rng.choice([1, 2, 3, 4, 8])
            kw["new"] = rng.randint(1, kw["batch"] + 3)
            kw["kids"] = max(kw["kids"], -(-kw["new"] // kw["batch"]))
        else:
            kw["prefix"] = rng.choice([0, 0, 1, 5])
            pages = _own_pages(kw)
            kw["pool"] = pages + _log(rng, 1, 2 * pages + 1)
        kw["hq"] = kw["hkv"]
        kw["dtype"] = "fp16"
    c = _case("", op, **kw)
    del c["name"]
    return c


# ------------------------------------------------------------------------------ sizes that a case fixes

def _lens(case):
    """Cached tokens of each sequence: from `len` down to `lo`, in a fixed mixed order."""
    b = case["batch"]
    span = case["len"] - case["lo"]
    lens = [case["len"] - (span * i) // max(1, b - 1) for i in range(b)]
    step = next(s for s in (7, 5, 3, 1) if math.gcd(s, b) == 1)
    return [lens[(i * step) % b] for i in range(b)]


def _new(case):
    """Drafted tokens of each sequence."""
    b, t = case["batch"], case["t"]
    return [max(1, t - i * t // (2 * b)) for i in range(b)] if case["ragged"] else [t] * b


def _accepted(case):
    return [1 + (i * 5 + case["acc"] - 1) % min(case["acc"], n) for i, n in enumerate(_new(case))]


def _own_pages(case):
    """Distinct pages of all sequences (compact): a common prefix and their own."""
    per = [-(-n // case["page"]) for n in _lens(case)]
    pre = min(case["prefix"], min(per))
    return pre + sum(p - pre for p in per)


def _sizes(case):
    code = case["d"] * case["bits"] // 8
    meta = 4 * case["d"] // case["g"]
    return code, meta, 2 * case["page"] * (code + meta)


def work(case):
    op, hq, hkv, d = case["op"], case["hq"], case["hkv"], case["d"]
    if op == "rope":
        n = case["n"]
        return {"bytes": n * (2 * (hq + hkv) * d * 2 + 8), "flops": 3 * n * (hq + hkv) * case["rot"]}
    code, meta, block = _sizes(case)
    row = 2 * hkv * (code + meta)     # a token's keys and values as they are cached
    if op == "write":
        n = case["n"]
        return {"bytes": n * (2 * (hq + 2 * hkv) * d * 2 + row + 16), "flops": n * (3 * (hq + hkv) * case["rot"] + 12 * hkv * d)}
    lens = _lens(case)
    if op == "tree":
        new = _new(case)
        tokens = sum(lens) + case["prefix"]
        pairs = sum(n * (case["prefix"] + l) for l, n in zip(lens, new))
        return {"bytes": tokens * row + 2 * sum(new) * hq * d * 2, "flops": 4 * pairs * hq * d}
    if op == "accept":
        moved = sum(a - 1 for a in _accepted(case))
        return {"bytes": 2 * moved * row * case["layers"] + 4 * case["batch"], "flops": 0}
    if op == "fork":
        copies = case["new"] - -(-case["new"] // case["kids"])
        used = sum(n % case["page"] for n in lens) / case["batch"]
        return {"bytes": 2 * copies * used * row * case["layers"] + 8 * case["new"] * (1 + -(-case["len"] // case["page"])), "flops": 0}
    used = _own_pages(case)
    moved = used * (1 - used / case["pool"])
    return {"bytes": 2 * moved * hkv * block * case["layers"] + 8 * case["batch"] * -(-case["len"] // case["page"]), "flops": 0}


# ------------------------------------------------------------------------------ inputs

def _freqs(case):
    """Radians per position of each pair (base 10000; scaled for long contexts by bands: pairs that turn often over the
    original 4096 positions are kept, those that turn less than once are slowed by the factor, a ramp between), and the magnitude."""
    r, factor = case["rot"], case["factor"]
    i = torch.arange(0, r, 2, dtype=torch.float64, device=DEV)
    f = 10000.0 ** (-i / r)
    if factor == 1.0:
        return f, 1.0
    pair = [r * math.log(4096 / (turns * 2 * math.pi)) / (2 * math.log(10000.0)) for turns in (32, 1)]
    low, high = max(math.floor(pair[0]), 0), min(math.ceil(pair[1]), r - 1)
    ramp = ((i / 2 - low) / max(high - low, 0.001)).clamp(0, 1)
    return f * (1 - ramp) + f / factor * ramp, 0.1 * math.log(factor) + 1


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEV, dtype=torch.float32)


def _positions(gen, n, far):
    """Positions of packed sequences (or of a step's tokens, each far in its own)."""
    if n <= 256:
        return torch.randint(0, far, (n,), generator=gen, device=DEV)
    begin = torch.randint(0, far, (1,), generator=gen, device=DEV)
    cut = n // 3
    return torch.cat((torch.arange(cut, device=DEV), begin + torch.arange(n - cut, device=DEV)))


def _codes(x, bits, g):
    """Codes (uint8), steps and floors (fp16) of x fp32 [..., D]: min-max over groups of g channels."""
    x = torch.nan_to_num(x, nan=0.0, posinf=65504.0, neginf=-65504.0).clamp(-65504.0, 65504.0)
    x = x.view(*x.shape[:-1], -1, g)
    low, high = x.amin(-1), x.amax(-1)
    m = low.half()
    s = ((high - m.float()) * (1.0 / (2 ** bits - 1))).clamp(min=0).half()
    inv = torch.where(s > 0, torch.reciprocal(s.float()), torch.zeros_like(low))
    c = ((x - m.float()[..., None]) * inv[..., None]).round().clamp(0, 2 ** bits - 1).to(torch.uint8)
    return c.view(*c.shape[:-2], -1), s, m


def _pack(k, v, bits, g):
    """Pages [P, Hkv, block] of dense keys and values, fp32 [P, Hkv, page, D]."""
    p, h, page, d = k.shape
    parts, metas = [], []
    for which, x in (("k", k), ("v", v)):
        c, s, m = _codes(x, bits, g)
        if which == "k":
            c = c.view(p, h, page, d // 32, 4, 8).transpose(3, 4)
            if bits == 4:
                c = c[..., [0, 2, 4, 6, 1, 3, 5, 7]]   # nibble n holds code j: 0 4 1 5 2 6 3 7 inverted
        else:
            c = c.view(p, h, page // 4, 4, 16, d // 16).transpose(3, 4)
        c = c.reshape(p, h, -1)
        parts.append(c if bits == 8 else c[..., 0::2] | (c[..., 1::2] << 4))
        meta = torch.stack((s, m), -1).view(p, h, page, d // g, 2).transpose(2, 3).contiguous()
        metas.append(meta.view(torch.uint8).reshape(p, h, -1))
    return torch.cat(parts + metas, -1)


def _keys_values(gen, d, *lead):
    """Keys whose channels differ in size and offset, as rotary models have them; values plain."""
    chan = torch.exp(0.4 * _randn(gen, d))
    return _randn(gen, *lead, d) * chan + 0.5 * _randn(gen, d) * chan, _randn(gen, *lead, d) * 0.7


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed) * 1000003 + 29)
    s = dict(case=case, dt=DTYPES[case["dtype"]])
    dict(rope=_prepare_rope, write=_prepare_rope, tree=_prepare_tree, accept=_prepare_moves, fork=_prepare_moves,
         compact=_prepare_moves)[case["op"]](s, gen)
    return s


def _prepare_rope(s, gen):
    case, page, hq, hkv, d, n = s["case"], s["case"]["page"], s["case"]["hq"], s["case"]["hkv"], s["case"]["d"], s["case"]["n"]
    s["freqs"], s["magnitude"] = _freqs(case)
    s["positions"] = _positions(gen, n, case["far"])
    k, v = _keys_values(gen, d, n, hkv)
    # slices of one fused projection's output, so with a token stride of their own
    qkv = torch.cat((2.0 * _randn(gen, n, hq, d), k, v), 1).to(s["dt"])
    s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    if case["op"] == "write":
        used = -(-n // page)
        ids = torch.randperm(used + 3, generator=gen, device=DEV)[:used]
        at = torch.arange(n, device=DEV)
        s["slots"] = ids[at // page] * page + at % page
        s["pages"] = torch.zeros(used + 3, hkv, _sizes(case)[2], dtype=torch.uint8, device=DEV)


def _prepare_tree(s, gen):
    case, page, hkv, d = s["case"], s["case"]["page"], s["case"]["hkv"], s["case"]["d"]
    lens, new = _lens(case), _new(case)
    per = -(-max(lens) // page)
    shared = -(-case["prefix"] // page)
    count = case["batch"] * per + shared + 1
    ids = torch.randperm(count, generator=gen, device=DEV).to(torch.int32)
    s["table"] = ids[:case["batch"] * per].view(case["batch"], per).contiguous()
    s["prefix_table"] = ids[case["batch"] * per:case["batch"] * per + shared].contiguous()
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    s["max_len"], s["max_q"], s["cu_q"] = max(lens), max(new), None
    if case["ragged"]:
        s["cu_q"] = torch.tensor([0] + new, dtype=torch.int32, device=DEV).cumsum(0).to(torch.int32)
    # every drafted token hangs on an earlier one; the first is the last token of the answer so far
    t = torch.cat([torch.arange(x, device=DEV) for x in new])
    u = torch.rand(t.shape[0], generator=gen, device=DEV)
    s["parents"] = torch.where(t == 0, -1, (u * t).long().clamp(max=t - 1)).to(torch.int32)
    s["q"] = (2.0 * _randn(gen, sum(new), case["hq"], d)).to(s["dt"])
    s["scale"] = 1.0 / math.sqrt(d)
    if not case["plan"]:
        s["mask"] = _plan_plain(s)[0]
    pages = torch.empty(count, hkv, _sizes(case)[2], dtype=torch.uint8, device=DEV)
    step = max(1, (1 << 25) // (hkv * page * d))
    for i in range(0, count, step):
        n = min(step, count - i)
        k, v = _keys_values(gen, d, n, hkv, page)
        pages[i:i + n] = _pack(k, v, case["bits"], case["g"])
    s["pages"] = pages


def _prepare_moves(s, gen):
    case, page = s["case"], s["case"]["page"]
    lens = _lens(case)
    batch, per = case["batch"], -(-case["len"] // page)
    extra = case["new"] if case["op"] == "fork" else 1
    count = case["pool"] if case["op"] == "compact" else batch * per + extra
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    ids = torch.randperm(count, generator=gen, device=DEV).to(torch.int32)
    if case["op"] == "compact":   # only what the sequences hold; the first pages are common to all
        need = (s["lens"].long() + page - 1) // page
        pre = min(case["prefix"], int(need.min()))
        first = pre + (need - pre).cumsum(0) - (need - pre)
        col = torch.arange(per, device=DEV)
        at = torch.where(col < pre, col, first[:, None] + col - pre)
        s["table"] = torch.where(col < need[:, None], ids[torch.where(col < need[:, None], at, 0)], -1).to(torch.int32)
    else:
        s["table"] = ids[:batch * per].view(batch, per).contiguous()
    if case["op"] == "fork":
        s["fresh"] = ids[batch * per:].contiguous()
        alive = -(-case["new"] // case["kids"])
        some = torch.randperm(batch, generator=gen, device=DEV)[:alive].repeat(case["kids"])[:case["new"]]
        s["parents"] = some[torch.randperm(case["new"], generator=gen, device=DEV)].to(torch.int32)
    if case["op"] == "accept":
        new, acc = _new(case), _accepted(case)
        s["max_q"], s["cu_q"] = max(new), None
        if case["ragged"]:
            s["cu_q"] = torch.tensor([0] + new, dtype=torch.int32, device=DEV).cumsum(0).to(torch.int32)
        # of each draft the first token and an increasing choice of the others
        key = torch.rand(batch, case["t"], generator=gen, device=DEV)
        t = torch.arange(case["t"], device=DEV)
        key = torch.where(t < torch.tensor(new, device=DEV)[:, None], key, 2.0)
        key[:, 0] = -1.0
        s["num_accepted"] = torch.tensor(acc, dtype=torch.int32, device=DEV)
        rank = key.argsort(-1).argsort(-1)
        chosen = torch.where(rank < s["num_accepted"][:, None], t, case["t"]).sort(-1).values[:, :max(acc)]
        s["accepted"] = torch.where(chosen < case["t"], chosen, -1).to(torch.int32).contiguous()
    s["pages"] = torch.randint(0, 256, (case["layers"], count, case["hkv"], _sizes(case)[2]), dtype=torch.uint8, generator=gen, device=DEV)


# ------------------------------------------------------------------------------ one pass

def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    import weight_only_quantization_amd as hq
    case = s["case"]
    op = case["op"]
    if op in ("rope", "write"):
        rope = hq.RopeTable(s["freqs"], interleaved=case["inter"], magnitude=s["magnitude"])
        if op == "rope":
            return hq.hqq_rope(s["q"], s["positions"], rope, k=s["k"], backward=case["back"])
    if op in ("write", "tree"):
        cache = hq.KVCache(s["pages"], case["hkv"], case["d"], case["bits"], case["g"], case["page"])
        if op == "write":
            return hq.hqq_kv_write_rope(cache, s["q"], s["k"], s["v"], s["positions"], s["slots"], rope, echo=True)
        plan = None
        if case["plan"]:
            plan = hq.hqq_kv_tree_plan(s["parents"], s["table"], s["lens"], case["page"], cu_q=s["cu_q"], max_q=s["max_q"])
        mask = plan[0] if plan else s["mask"]
        pre = dict(prefix_table=s["prefix_table"], prefix_len=case["prefix"]) if case["prefix"] else {}
        out = hq.hqq_kv_attention_tree(cache, s["q"], mask, s["table"], s["lens"], scale=s["scale"], cu_q=s["cu_q"],
                                       max_q=s["max_q"], max_len=s["max_len"], **pre)
        return [out, *(plan or ())]
    if "layers" not in s:   # the handle that a program keeps of its layers' caches
        s["layers"] = hq.KVLayers([hq.KVCache(p, case["hkv"], case["d"], case["bits"], case["g"], case["page"]) for p in s["pages"]])
    if op == "accept":
        lens = hq.hqq_kv_accept(s["layers"], s["table"], s["lens"], s["accepted"], s["num_accepted"], tokens=case["t"],
                                cu_q=s["cu_q"], max_q=s["max_q"])
        return [s["pages"], lens]
    if op == "fork":
        return [s["pages"], *hq.hqq_kv_fork(s["layers"], s["table"], s["lens"], s["parents"], s["fresh"])]
    return [s["pages"], *hq.hqq_kv_compact(s["layers"], s["table"], s["lens"])]


def _run_plain(s):
    op = s["case"]["op"]
    if op == "rope":
        return _rotate(s, s["q"]), _rotate(s, s["k"])
    if op == "write":
        return _write_plain(s)
    if op == "tree":
        plan = _plan_plain(s) if s["case"]["plan"] else ()
        return [_attend_plain(s, plan[0] if plan else s["mask"]), *plan]
    return dict(accept=_accept_plain, fork=_fork_plain, compact=_compact_plain)[op](s)


def _rotate(s, x):
    """In 64 bits, rounded once: angles of far positions, and keys that lie next to a code's border."""
    case, r = s["case"], s["case"]["rot"]
    angle = s["positions"].double()[:, None, None] * s["freqs"]
    c, sn = torch.cos(angle) * s["magnitude"], torch.sin(angle) * s["magnitude"]
    if case.get("back"):
        sn = -sn
    y = x.double()
    a, b = (y[..., 0:r:2], y[..., 1:r:2]) if case["inter"] else (y[..., :r // 2], y[..., r // 2:r])
    pair = (a * c - b * sn, b * c + a * sn)
    turned = torch.stack(pair, -1).flatten(-2) if case["inter"] else torch.cat(pair, -1)
    return torch.cat((turned, y[..., r:]), -1).to(x.dtype)


def _stored(x, bits, g):
    c, s, m = _codes(x.float(), bits, g)
    c = c.view(*c.shape[:-1], -1, g).float()
    return (c * s.float()[..., None] + m.float()[..., None]).view(x.shape).to(x.dtype)


def _write_plain(s):
    case, v, slots, pages = s["case"], s["v"], s["slots"], s["pages"]
    page, hkv, d = case["page"], case["hkv"], case["d"]
    q, k = _rotate(s, s["q"]), _rotate(s, s["k"])
    # quantised through a dense page image: the tokens' pages are laid out whole
    used = -(-k.shape[0] // page)
    kv = torch.zeros(2, used * page, hkv, d, device=DEV)
    kv[0, :k.shape[0]], kv[1, :k.shape[0]] = k, v
    kv = kv.view(2, used, page, hkv, d).transpose(2, 3)
    pages[slots[::page] // page] = _pack(kv[0], kv[1], case["bits"], case["g"])
    return q, _stored(k, case["bits"], case["g"]), _stored(v, case["bits"], case["g"])


def _padded(s):
    """Of each sequence's query tokens [B, T]: whether they are there, and their rows."""
    case = s["case"]
    b, tmax = case["batch"], s["max_q"]
    t = torch.arange(tmax, device=DEV)
    if s["cu_q"] is None:
        count = torch.full((b,), tmax, device=DEV)
        first = torch.arange(b, device=DEV) * tmax
    else:
        first = s["cu_q"].long()[:-1]
        count = s["cu_q"].long()[1:] - first
    there = t < count[:, None]
    return t, count, there, torch.where(there, first[:, None] + t, 0)


def _plan_plain(s):
    """Masks (int64 [tokens, words], bit j of a row: the token sees draft j), rotary positions, slots."""
    case, page = s["case"], s["case"]["page"]
    t, count, there, at = _padded(s)
    words = (s["max_q"] + 63) // 64
    parent = s["parents"].long()[at]
    link = (parent[..., None] == t) & there[..., None]
    sees = torch.matrix_power(link.double() + torch.eye(s["max_q"], dtype=torch.float64, device=DEV), s["max_q"]) > 0
    depth = sees.sum(-1) - 1
    bits = torch.zeros(*sees.shape[:2], words * 64, dtype=torch.int64, device=DEV)
    bits[..., :s["max_q"]] = sees.long()
    mask = (bits.view(*sees.shape[:2], words, 64) << torch.arange(64, device=DEV)).sum(-1)
    begin = s["lens"].long()[:, None] - count[:, None]
    place = (begin + t).clamp(min=0)
    slot = s["table"].long().gather(1, (place // page).clamp(max=s["table"].shape[1] - 1)) * page + place % page
    return mask[there], (begin + depth)[there], slot[there]


def _unpack(pages, case):
    """Keys and values, fp32 [..., page, D], of blocks [..., block]."""
    bits, g, d, page = case["bits"], case["g"], case["d"], case["page"]
    lead = pages.shape[:-1]
    nc, nm = page * d * bits // 8, page * 4 * (d // g)
    out = []
    for which in (0, 1):
        c = pages[..., which * nc:(which + 1) * nc]
        if bits == 4:
            c = torch.stack((c & 15, c >> 4), -1)
        if which == 0:
            c = c.reshape(*lead, page, 4, d // 32, 8)
            c = (c[..., [0, 4, 1, 5, 2, 6, 3, 7]] if bits == 4 else c).transpose(-3, -2)
        else:
            c = c.reshape(*lead, page // 4, 16, 4, d // 16).transpose(-3, -2)
        at = 2 * nc + which * nm
        meta = pages[..., at:at + nm].contiguous().view(torch.float16).view(*lead, d // g, page, 2).transpose(-3, -2).float()
        x = c.reshape(*lead, page, d // g, g).float()
        out.append((x * meta[..., 0:1] + meta[..., 1:2]).reshape(*lead, page, d))
    return out


def _by_head(kv, b, hkv, d):
    """[B, P, Hkv, page, D] -> [B, Hkv, P * page, D]."""
    return tuple(x.transpose(1, 2).reshape(b, hkv, -1, d) for x in kv)


def _attend_plain(s, mask):
    case, q = s["case"], s["q"].float()
    hkv, d, b = case["hkv"], case["d"], case["batch"]
    per, tmax, prefix = case["hq"] // hkv, s["max_q"], case["prefix"]
    lens = s["lens"].long()
    t, count, there, at = _padded(s)
    rows = q[at].view(b, tmax, hkv, per, d).permute(0, 2, 1, 3, 4).reshape(b, hkv, tmax * per, d)
    k, v = _by_head(_unpack(s["pages"][s["table"].long()], case), b, hkv, d)
    key = torch.arange(k.shape[2], device=DEV)
    draft = key - (lens - count)[:, None]                               # [B, L]: index among the drafts
    some = draft.clamp(0, 64 * mask.shape[1] - 1)
    sees = (mask[at].gather(2, (some // 64)[:, None].expand(-1, tmax, -1)) >> (some % 64)[:, None]) & 1 != 0
    seen = ((draft < 0)[:, None] | sees) & (key < lens[:, None])[:, None]   # [B, T, L]
    score = torch.matmul(rows, k.transpose(2, 3).contiguous()).view(b, hkv, tmax, per, -1) * s["scale"]
    score = score.masked_fill(~seen[:, None, :, None, :], -math.inf).view(b, hkv, tmax * per, -1)
    top = score.amax(-1, keepdim=True)
    if prefix:
        pk, pv = _by_head(_unpack(s["pages"][s["prefix_table"].long()][None], case), 1, hkv, d)
        pk, pv = pk[0, :, :prefix], pv[0, :, :prefix]                  # [Hkv, prefix, D]
        flat = rows.transpose(0, 1).reshape(hkv, -1, d)
        ps = (torch.matmul(flat, pk.transpose(1, 2).contiguous()) * s["scale"]).view(hkv, b, -1, prefix).transpose(0, 1)
        top = torch.maximum(top, ps.amax(-1, keepdim=True))
        pe = torch.exp(ps - top)
    top = torch.where(top == -math.inf, 0.0, top)
    e = torch.exp(score - top)
    total, o = e.sum(-1, keepdim=True), torch.matmul(e, v)
    if prefix:
        total = total + pe.sum(-1, keepdim=True)
        o = o + torch.matmul(pe.transpose(0, 1).reshape(hkv, -1, prefix), pv.contiguous()).view(hkv, b, -1, d).transpose(0, 1)
    o = torch.where(total > 0, o / total, 0.0).view(b, hkv, tmax, per, d).permute(0, 2, 1, 3, 4).reshape(b, tmax, case["hq"], d)
    return o[there].to(s["dt"])


def _token_bytes(case):
    """Byte offsets within a block of everything a token has there, int64 [page, bytes]."""
    code, meta, _ = _sizes(case)
    page, unit = case["page"], case["d"] * case["bits"] // 128
    t = torch.arange(page, device=DEV)[:, None]
    k = t * code + torch.arange(code, device=DEV)
    u = torch.arange(code, device=DEV)
    v = page * code + (t // 4 * 16 + u // unit) * 4 * unit + t % 4 * unit + u % unit
    w = torch.arange(2 * meta, device=DEV)
    m = 2 * page * code + (w // 4 * page + t) * 4 + w % 4
    return torch.cat((k, v, m), 1)


def _accept_plain(s):
    case, page, pages = s["case"], s["case"]["page"], s["pages"]
    _, count, _, _ = _padded(s)
    acc, base = s["accepted"].long(), s["lens"].long() - count
    j = torch.arange(acc.shape[1], device=DEV)
    on = j < s["num_accepted"].long()[:, None]
    where = _token_bytes(case)
    seq = torch.arange(case["batch"], device=DEV)[:, None].expand_as(acc)[on]
    src, dst = (base[:, None] + acc)[on], (base[:, None] + j)[on]
    table = s["table"].long()
    head = torch.arange(case["hkv"], device=DEV)[None, :, None]
    moved = pages[:, table[seq, src // page][:, None, None], head, where[src % page][:, None]]
    pages[:, table[seq, dst // page][:, None, None], head, where[dst % page][:, None]] = moved
    return [pages, (base + s["num_accepted"]).to(torch.int32)]


def _fork_plain(s):
    case, page, pages = s["case"], s["case"]["page"], s["pages"]
    parents, fresh = s["parents"].long(), s["fresh"]
    lens, table = s["lens"][parents], s["table"][parents]
    child = torch.arange(case["new"], device=DEV)
    first = (parents[:, None] == parents[None, :]).long().argmax(-1) == child
    last = (lens // page).long()
    col = torch.arange(table.shape[1], device=DEV)
    copy = ~first & (lens % page != 0)
    out = torch.where((col[None] > last[:, None]) & ~first[:, None], -1, table)
    out = torch.where((col[None] == last[:, None]) & ~first[:, None], torch.where(copy, fresh, -1)[:, None], out)
    # (the used tokens of the page, as everything of a token that the cache keeps)
    where = _token_bytes(case)
    tok = torch.arange(page, device=DEV)
    on = copy[:, None] & (tok < (lens % page)[:, None])
    c, t = on.nonzero(as_tuple=True)
    head = torch.arange(case["hkv"], device=DEV)[None, :, None]
    src = table.gather(1, last.clamp(max=table.shape[1] - 1)[:, None])[:, 0].long()
    pages[:, fresh.long()[c][:, None, None], head, where[t][:, None]] = pages[:, src[c][:, None, None], head, where[t][:, None]]
    return [pages, out.to(torch.int32), lens]


def _compact_plain(s):
    case, page, pages, table = s["case"], s["case"]["page"], s["pages"], s["table"].long()
    held = torch.arange(table.shape[1], device=DEV) < ((s["lens"].long() + page - 1) // page)[:, None]
    held &= (table >= 0) & (table < pages.shape[1])
    used = torch.zeros(pages.shape[1], dtype=torch.bool, device=DEV)
    used[table[held]] = True
    order = torch.arange(pages.shape[1], device=DEV)
    count = used.sum()
    src, dst = (used & (order >= count)).nonzero()[:, 0], (~used & (order < count)).nonzero()[:, 0]
    to = order.clone()
    to[src] = dst
    pages[:, dst] = pages[:, src]
    return [pages, torch.where(held, to[torch.where(held, table, 0)], -1).to(torch.int32), count.to(torch.int32)[None]]


# ------------------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _turned64(s, s["q"]), _turned64(s, s["k"])
    if case["op"] == "write":
        k = _turned64(s, s["k"]).to(s["dt"])
        return _turned64(s, s["q"]), _stored64(k, case["bits"], case["g"]), _stored64(s["v"], case["bits"], case["g"])
    if case["op"] == "tree":
        return [_tree64(s)] + [None, None, None] * case["plan"]
    return None     # bytes that are moved, and whole numbers


def _turned64(s, x):
    """Pairs as complex numbers, turned by exp(i position freq)."""
    case, r = s["case"], s["case"]["rot"]
    turn = s["magnitude"] * torch.exp(1j * (s["positions"].double()[:, None] * s["freqs"]))[:, None]
    if case.get("back"):
        turn = turn.conj()
    out = x.double()
    i = torch.arange(r // 2, device=DEV)
    re, im = (2 * i, 2 * i + 1) if case["inter"] else (i, i + r // 2)
    z = torch.complex(out[..., re], out[..., im]) * turn
    out = out.clone()
    out[..., re], out[..., im] = z.real, z.imag
    return out


def _stored64(x, bits, g):
    """floor + code * step in 64 bits; step and code are the format's, which defines them by operations of 32 bits (16-bit values
    often lie on the very border of two codes)."""
    y = x.float().unflatten(-1, (-1, g))
    floor = y.min(-1, keepdim=True)[0].half()
    step = ((y.max(-1, keepdim=True)[0] - floor.float()) * torch.tensor(1.0 / (2 ** bits - 1), dtype=torch.float32, device=DEV)).relu().half()
    code = torch.where(step > 0, torch.round((y - floor.float()) * (1.0 / step.float())), 0.0).clamp(0, 2 ** bits - 1)
    return (floor.double() + code.double() * step.double()).flatten(-2)


def _places(case):
    """Bit within a block of the code of K and of V at (token, channel)."""
    bits, d, page = case["bits"], case["d"], case["page"]
    tok = torch.arange(page, device=DEV)[:, None]
    c = torch.arange(d, device=DEV)[None, :]
    i, h, j = c // 32, (c % 32) // 8, c % 8
    kbit = tok * d * bits + (h * (d // 32) + i) * 8 * bits
    kbit = kbit + (4 * (j // 2 + 4 * (j % 2)) if bits == 4 else 8 * j)
    u = d // 16
    vbit = page * d * bits + (((tok // 4) * 16 + c // u) * 4 + tok % 4) * u * bits + (c % u) * bits
    return kbit, vbit


def _dense64(case, pages, ids, length):
    """K and V of a sequence, fp64 [Hkv, length, D], code by code."""
    bits, g, hkv, d, page = case["bits"], case["g"], case["hkv"], case["d"], case["page"]
    out = []
    for which, bit in enumerate(_places(case)):
        parts = [torch.zeros(hkv, 0, d, dtype=torch.float64, device=DEV)]
        for blocks in pages[ids[:-(-length // page)].long()].split(64):
            code = (blocks[..., (bit // 8).reshape(-1)].to(torch.int32) >> (bit % 8).reshape(-1).to(torch.int32)) & (2 ** bits - 1)
            code = code.view(*blocks.shape[:-1], page, d)
            at = 2 * page * d * bits // 8 + which * page * 4 * (d // g)
            half = blocks[..., at:at + page * 4 * (d // g)].contiguous().view(torch.float16).double()
            half = half.view(*blocks.shape[:-1], d // g, page, 2)
            step = half[..., 0].transpose(-1, -2).repeat_interleave(g, -1)
            floor = half[..., 1].transpose(-1, -2).repeat_interleave(g, -1)
            parts.append((floor + code.double() * step).transpose(0, 1).reshape(hkv, -1, d))
        out.append(torch.cat(parts, 1)[:, :length])
    return out


def _tree64(s):
    case, hkv, d = s["case"], s["case"]["hkv"], s["case"]["d"]
    parents, begin, outs = s["parents"].tolist(), 0, []
    pk = _dense64(case, s["pages"], s["prefix_table"], case["prefix"])
    for b, (length, new) in enumerate(zip(_lens(case), _new(case))):
        k, v = _dense64(case, s["pages"], s["table"][b], length)
        k, v = torch.cat((pk[0], k), 1), torch.cat((pk[1], v), 1)      # [Hkv, keys, D]
        hide = torch.zeros(new, new, dtype=torch.bool)
        for t in range(new):
            if t:
                hide[t] = hide[parents[begin + t]]
            else:
                hide[t] = True
            hide[t, t] = False
        hide = torch.cat((torch.zeros(new, k.shape[1] - new, dtype=torch.bool), hide), 1).to(DEV)
        q = s["q"][begin:begin + new].double()
        begin += new
        o = torch.zeros(new, case["hq"], d, dtype=torch.float64, device=DEV)
        for h in range(case["hq"]):
            x = (q[:, h] @ k[h * hkv // case["hq"]].T) * s["scale"]
            o[:, h] = torch.softmax(x.masked_fill(hide, -math.inf), -1) @ v[h * hkv // case["hq"]]
        outs.append(o)
    return torch.cat(outs)
