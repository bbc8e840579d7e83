"""Measured cases of the quantised key/value cache: writing and reading it, attention over each sequence's
own cache, and attention of a batch that shares a long prefix.

A cache is a tensor of pages, uint8 [num_pages, Hkv, block]; a block holds one KV head's keys and values of
`page` tokens: K codes, V codes, K metadata, V metadata (b bits a code, groups of g along the D channels).
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
    c = dict(name=name, op=op, dtype="fp16", bits=4, g=64, d=128, page=64, hq=32, hkv=32, batch=1, t=1, len=0, lo=0,
             prefix=0, n=0, ragged=False)
    c.update(kw)
    return c


def listed():
    return [
        # one decode step of a serving batch: one token a sequence joins the cache (latency)
        _case("write_step_b64", "write", n=64, hkv=8),
        # a prompt of odd length, kept in 8 bits, bfloat16 model
        _case("write_prompt_4099", "write", n=4099, hkv=8, bits=8, g=128, dtype="bf16"),
        # prompts of a whole batch in one call
        _case("write_prompts_32k", "write", n=32768, hkv=8, page=128),
        # a short sequence read back, as for a copy to another layout
        _case("read_777", "read", n=777, hkv=32, g=32, page=16),
        # long contexts read back to dense keys and values
        _case("read_64k", "read", n=65536, hkv=8, bits=8, dtype="bf16"),
        # one user, Llama-7B's heads, a context of about a thousand (latency)
        _case("attn_step_b1", "attn", hq=32, hkv=32, len=1023, lo=1023),
        # an ordinary serving batch with grouped heads and ragged lengths
        _case("attn_step_b32", "attn", batch=32, hq=32, hkv=8, len=4096, lo=65),
        # long contexts, 64 query heads on 8
        _case("attn_step_long", "attn", batch=16, hq=64, hkv=8, len=32768, lo=16384, page=256),
        # a draft of five tokens a sequence to verify, heads of 64, 8 bits, bfloat16
        _case("attn_draft_b16", "attn", batch=16, t=5, hq=32, hkv=8, d=64, bits=8, dtype="bf16", len=2001, lo=3, page=32),
        # a chunk of a long prompt: 2048 new tokens onto 6144 cached ones
        _case("attn_chunk_2048", "attn", t=2048, hq=32, hkv=8, len=8192, lo=8192),
        # sixteen answers to one prompt, Llama-7B's heads
        _case("shared_b16", "shared", batch=16, hq=32, hkv=32, prefix=2048, len=203, lo=1),
        # a long system prompt under a serving batch, 64 query heads on 8
        _case("shared_b64_16k", "shared", batch=64, hq=64, hkv=8, prefix=16384, len=1000, lo=20, page=128),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write", "read", "attn", "attn", "attn", "shared", "shared"])
    d = rng.choice([64, 128, 128])
    kw = dict(dtype=rng.choice(["fp16", "bf16"]), bits=rng.choice([4, 4, 8]), d=d, g=rng.choice([x for x in (32, 64, 64, 128) if x <= d]),
              page=rng.choice([16, 32, 64, 128, 256]), hkv=rng.choice([1, 4, 8, 8, 32]))
    if op in ("write", "read"):
        kw["n"] = _log(rng, 1, 32768 * 8 // max(8, kw["hkv"]))
        kw["hq"] = kw["hkv"]
        return _nameless(op, kw)
    kw["hq"] = kw["hkv"] * (1 if kw["hkv"] == 32 else rng.choice([1, 3, 4, 7, 8]))
    if op == "attn" and rng.random() < 0.35:  # chunks of prompts, the sequences' parts of different lengths
        kw["batch"] = rng.choice([1, 1, 2, 5])
        kw["t"] = _log(rng, 6, 2048 * 32 // (kw["batch"] * max(32, kw["hq"])))
        kw["ragged"] = kw["batch"] > 1
        kw["len"] = kw["t"] + _log(rng, 1, 6144 // kw["batch"]) - 1
        kw["lo"] = rng.randint(kw["t"], kw["len"])
        return _nameless(op, kw)
    kw["batch"] = _log(rng, 1, 96 if op == "shared" else 64)
    kw["t"] = rng.choice([1, 1, 1, 2, 5])
    most = 16 * 24576 * 8 * 4 // (kw["bits"] * kw["batch"] * max(8, kw["hkv"]))
    kw["len"] = _log(rng, kw["t"], min(32768, most) if op == "attn" else min(1024, most))
    kw["lo"] = rng.randint(0 if rng.random() < 0.3 else kw["len"] // 2, kw["len"])
    if op == "shared":
        kw["prefix"] = _log(rng, 100, 16384 * 64 // (max(64, kw["batch"] * kw["t"] * kw["hq"] // 64)))
    return _nameless(op, kw)


def _nameless(op, kw):
    c = _case("", op, **kw)
    del c["name"]
    return c


# ------------------------------------------------------------------------------ sizes that a case fixes

def _lens(case):
    """Cached tokens of each sequence (its own part): from `len` down to `lo`, in a fixed mixed order."""
    b = case["batch"]
    span = case["len"] - case["lo"]
    lens = [case["len"] - (span * i) // max(1, b - 1) for i in range(b)]
    step = next(s for s in (7, 5, 3, 1) if math.gcd(s, b) == 1)
    return [lens[(i * step) % b] for i in range(b)]


def _new(case):
    """New (query) tokens of each sequence."""
    b, t = case["batch"], case["t"]
    return [max(1, t * (i + 1) // b) for i in range(b)] if case["ragged"] else [t] * b


def _sizes(case):
    code = case["d"] * case["bits"] // 8
    meta = 4 * case["d"] // case["g"]
    return code, meta, 2 * case["page"] * (code + meta)


def work(case):
    code, meta, _ = _sizes(case)
    row = 2 * case["hkv"] * (code + meta)     # a token's keys and values as they are cached
    dense = 2 * case["hkv"] * case["d"] * 2   # and in 16 bits
    if case["op"] == "write":
        return {"bytes": case["n"] * (2 * dense + row + 8), "flops": case["n"] * case["hkv"] * case["d"] * 2 * 6}
    if case["op"] == "read":
        return {"bytes": case["n"] * (dense + row + 8), "flops": case["n"] * case["hkv"] * case["d"] * 2 * 2}
    lens, new = _lens(case), _new(case)
    tokens = sum(lens) + case["prefix"]
    pairs = sum(case["prefix"] * n + sum(max(0, min(l, l - n + i + 1)) for i in range(n)) for l, n in zip(lens, new))
    return {"bytes": tokens * row + 2 * sum(new) * case["hq"] * case["d"] * 2, "flops": 4 * pairs * case["hq"] * case["d"]}


# ------------------------------------------------------------------------------ inputs

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


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEV, dtype=torch.float32)


def _keys_values(gen, d, *lead):
    """Keys with a few strong channels and channel offsets, as rotary models have them; values plain."""
    chan = torch.exp(0.4 * _randn(gen, d)) * (1 + 4 * (torch.rand(d, generator=gen, device=DEV) < 0.03))
    k = _randn(gen, *lead, d) * chan + 0.5 * _randn(gen, d) * chan
    return k, _randn(gen, *lead, d) * 0.7


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed) * 1000003 + 17)
    dt, page, hkv, d = DTYPES[case["dtype"]], case["page"], case["hkv"], case["d"]
    block = _sizes(case)[2]
    s = dict(case=case, dt=dt)
    if case["op"] in ("write", "read"):
        n = case["n"]
        used = -(-n // page)
        s["num_pages"] = used + 3
        ids = torch.randperm(used + 3, generator=gen, device=DEV)[:used]
        at = torch.arange(n, device=DEV)
        s["slots"] = ids[at // page] * page + at % page
        if case["op"] == "write":
            k, v = _keys_values(gen, d, n, hkv)
            # slices of one fused projection's output, so with a token stride of their own
            kv = torch.stack((k, v), 1).to(dt)
            s["k"], s["v"] = kv[:, 0], kv[:, 1]
            s["pages"] = torch.zeros(used + 3, hkv, block, dtype=torch.uint8, device=DEV)
            return s
    else:
        lens, new = _lens(case), _new(case)
        per = max(1, -(-max(lens) // page))
        shared = -(-case["prefix"] // page)
        s["num_pages"] = case["batch"] * per + shared + 1
        ids = torch.randperm(s["num_pages"], generator=gen, device=DEV).to(torch.int32)
        s["table"] = ids[:case["batch"] * per].view(case["batch"], per).contiguous()
        s["prefix_table"] = ids[case["batch"] * per:case["batch"] * per + shared].contiguous()
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        total = sum(new)
        s["max_len"], s["max_q"] = max(lens), max(new)
        s["cu_q"] = None
        if case["ragged"]:
            s["cu_q"] = torch.tensor([0] + new, dtype=torch.int32, device=DEV).cumsum(0).to(torch.int32)
        s["q"] = (2.0 * _randn(gen, total, case["hq"], d)).to(dt)
        s["scale"] = 1.0 / math.sqrt(d)
    pages = torch.empty(s["num_pages"], hkv, block, dtype=torch.uint8, device=DEV)
    step = max(1, (1 << 25) // (hkv * page * d))
    for i in range(0, s["num_pages"], step):
        n = min(step, s["num_pages"] - i)
        k, v = _keys_values(gen, d, n, hkv, page)
        pages[i:i + n] = _pack(k, v, case["bits"], case["g"])
    s["pages"] = pages
    return s


# ------------------------------------------------------------------------------ one pass

def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    import weight_only_quantization_amd as hq
    case = s["case"]
    cache = hq.KVCache(s["pages"], case["hkv"], case["d"], case["bits"], case["g"], case["page"])
    if case["op"] == "write":
        return hq.hqq_kv_write(cache, s["k"], s["v"], s["slots"], echo=True)
    if case["op"] == "read":
        return hq.hqq_kv_read(cache, s["slots"], dtype=s["dt"])
    if case["op"] == "attn":
        return hq.hqq_kv_attention(cache, s["q"], s["table"], s["lens"], scale=s["scale"], cu_q=s["cu_q"], max_q=s["max_q"],
                                   max_len=s["max_len"])
    return hq.hqq_kv_attention_shared(cache, s["q"], s["prefix_table"], case["prefix"], s["table"], s["lens"],
                                      scale=s["scale"], cu_q=s["cu_q"], max_q=s["max_q"], max_len=s["max_len"])


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


def _stored(x, bits, g):
    c, s, m = _codes(x.float(), bits, g)
    c = c.view(*c.shape[:-1], -1, g).float()
    return (c * s.float()[..., None] + m.float()[..., None]).view(x.shape).to(x.dtype)


def _run_plain(s):
    case, pages, dt = s["case"], s["pages"], s["dt"]
    page, hkv, d = case["page"], case["hkv"], case["d"]
    if case["op"] == "write":
        k, v, slots = s["k"], s["v"], s["slots"]
        # quantised through a dense page image: the tokens' pages are laid out whole
        used = -(-k.shape[0] // page)
        kv = torch.zeros(2, used * page, hkv, d, device=DEV)
        kv[0, :k.shape[0]], kv[1, :k.shape[0]] = k, v
        kv = kv.view(2, used, page, hkv, d).transpose(2, 3)
        pages[slots[::page] // page] = _pack(kv[0], kv[1], case["bits"], case["g"])
        return _stored(k, case["bits"], case["g"]), _stored(v, case["bits"], case["g"])
    if case["op"] == "read":
        slots = s["slots"]
        k, v = _unpack(pages[slots[::page] // page], case)
        n = slots.shape[0]
        return tuple(x.transpose(1, 2).reshape(-1, hkv, d)[:n].to(dt) for x in (k, v))
    return _attend_plain(s)


def _attend_plain(s):
    case, q = s["case"], s["q"].float()
    page, hkv, d, b = case["page"], case["hkv"], case["d"], case["batch"]
    per = case["hq"] // hkv
    table, lens, prefix = s["table"].long(), s["lens"].long(), case["prefix"]
    tmax = s["max_q"]
    t = torch.arange(tmax, device=DEV)
    if s["cu_q"] is None:
        count = torch.full((b,), tmax, device=DEV)
        first = torch.arange(b, device=DEV) * tmax
    else:
        first = s["cu_q"].long()[:-1]
        count = s["cu_q"].long()[1:] - first
    there = t < count[:, None]                                       # [B, T]
    at = torch.where(there, first[:, None] + t, 0)
    qb = q[at].view(b, tmax, hkv, per, d).permute(2, 0, 1, 3, 4)       # [Hkv, B, T, G, D]
    k, v = _by_head(_unpack(s["pages"][table], case), b, hkv, d)
    key = torch.arange(k.shape[2], device=DEV)
    last = lens[:, None] - count[:, None] + t                        # [B, T]
    seen = (key <= last[..., None]) & (key < lens[:, None, None])       # [B, T, L]
    rows = qb.permute(1, 0, 2, 3, 4).reshape(b, hkv, tmax * per, d)
    score = torch.matmul(rows, k.transpose(2, 3)).view(b, hkv, tmax, per, -1) * s["scale"]
    score = score.masked_fill(~seen[:, None, :, None, :], -math.inf)
    if prefix:
        pk, pv = _by_head(_unpack(s["pages"][s["prefix_table"].long()][None], case), 1, hkv, d)
        pk, pv = pk[0, :, :prefix], pv[0, :, :prefix]                  # [Hkv, prefix, D]
        flat = qb.reshape(hkv, b * tmax * per, d)
        ps = (torch.matmul(flat, pk.transpose(1, 2)) * s["scale"]).view(hkv, b, tmax, per, prefix).transpose(0, 1)
        top = torch.maximum(score.amax(-1, keepdim=True), ps.amax(-1, keepdim=True))
        pe = torch.exp(ps - top)
    else:
        top = score.amax(-1, keepdim=True)
        top = torch.where(top == -math.inf, 0.0, top)
    e = torch.exp(score - top)
    total = e.sum(-1, keepdim=True)
    o = torch.matmul(e.view(b, hkv, tmax * per, -1), v).view(b, hkv, tmax, per, d)
    if prefix:
        total = total + pe.sum(-1, keepdim=True)
        po = torch.matmul(pe.transpose(0, 1).reshape(hkv, b * tmax * per, prefix), pv)
        o = o + po.view(hkv, b, tmax, per, d).transpose(0, 1)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 2, 1, 3, 4).reshape(b, tmax, case["hq"], d)
    out = torch.zeros(q.shape, device=DEV)
    if s["cu_q"] is None:
        return o.reshape(q.shape).to(s["dt"])
    out[at[there]] = o[there]
    return out.to(s["dt"])


def _by_head(kv, b, hkv, d):
    """[B, P, Hkv, page, D] -> [B, Hkv, P * page, D]."""
    return tuple(x.transpose(1, 2).reshape(b, hkv, -1, d) for x in kv)


# ------------------------------------------------------------------------------ in 64 bits

def _places(case):
    """Byte offset and shift within a block of the code of K and of V at (token, channel)."""
    bits, d, page = case["bits"], case["d"], case["page"]
    tok = torch.arange(page, device=DEV)[:, None]
    c = torch.arange(d, device=DEV)[None, :]
    i, h, j = c // 32, (c % 32) // 8, c % 8
    kbit = tok * d * bits + (h * (d // 32) + i) * 8 * bits
    kbit = kbit + (4 * (j // 2 + 4 * (j % 2)) if bits == 4 else 8 * j)
    u = d // 16
    vbit = page * d * bits + (((tok // 4) * 16 + c // u) * 4 + tok % 4) * u * bits + (c % u) * bits
    return kbit, vbit


def _values64(case, blocks):
    """K and V, fp64 [..., page, D], of blocks [..., block], code by code."""
    bits, g, d, page = case["bits"], case["g"], case["d"], case["page"]
    out = []
    for which, bit in enumerate(_places(case)):
        code = (blocks[..., (bit // 8).reshape(-1)].to(torch.int32) >> (bit % 8).reshape(-1).to(torch.int32)) & (2 ** bits - 1)
        code = code.view(*blocks.shape[:-1], page, d)
        at = 2 * page * d * bits // 8 + which * page * 4 * (d // g)
        half = blocks[..., at:at + page * 4 * (d // g)].contiguous().view(torch.float16).double()
        half = half.view(*blocks.shape[:-1], d // g, page, 2)
        step = half[..., 0].transpose(-1, -2).repeat_interleave(g, -1)
        floor = half[..., 1].transpose(-1, -2).repeat_interleave(g, -1)
        out.append(floor + code.double() * step)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    page, hkv, d = case["page"], case["hkv"], case["d"]
    if case["op"] == "write":
        return [_exact_stored(s[x], case["bits"], case["g"]) for x in "kv"]
    if case["op"] == "read":
        n = case["n"]
        ids = s["slots"][::page] // page
        parts = [_values64(case, b) for b in s["pages"][ids].split(64)]
        return [torch.cat([p[w] for p in parts]).transpose(1, 2).reshape(-1, hkv, d)[:n] for w in (0, 1)]
    outs, begin = [], 0
    pk = _dense64(case, s["pages"], s["prefix_table"], case["prefix"])
    for b, (length, new) in enumerate(zip(_lens(case), _new(case))):
        k, v = _dense64(case, s["pages"], s["table"][b], length)
        k, v = torch.cat((pk[0], k), 1), torch.cat((pk[1], v), 1)      # [Hkv, keys, D]
        q = s["q"][begin:begin + new].double()
        begin += new
        o = torch.zeros(new, case["hq"], d, dtype=torch.float64, device=DEV)
        upto = torch.arange(new, device=DEV) + length - new + 1        # keys of its own that a token sees
        hide = torch.arange(k.shape[1], device=DEV)[None] >= case["prefix"] + upto.clamp(min=0)[:, None]
        for h in range(case["hq"]):
            x = (q[:, h] @ k[h * hkv // case["hq"]].T) * s["scale"]
            p = torch.softmax(x.masked_fill(hide, -math.inf), -1)
            o[:, h] = torch.nan_to_num(p, nan=0.0) @ v[h * hkv // case["hq"]]
        outs.append(o)
    return torch.cat(outs)


def _dense64(case, pages, ids, length):
    hkv, d = case["hkv"], case["d"]
    if not length:
        return [torch.zeros(hkv, 0, d, dtype=torch.float64, device=DEV)] * 2
    ids = ids[:-(-length // case["page"])].long()
    parts = [_values64(case, b) for b in pages[ids].split(64)]
    return [torch.cat([p[w] for p in parts]).transpose(0, 1).reshape(hkv, -1, d)[:, :length] for w in (0, 1)]


def _exact_stored(x, bits, g):
    y = x.double().reshape(*x.shape[:-1], -1, g)
    floor = y.amin(-1, keepdim=True).half().double()
    step = ((y.amax(-1, keepdim=True) - floor) / (2 ** bits - 1)).half().double()
    code = torch.where(step > 0, torch.round((y - floor) / step), 0.0).clamp(0, 2 ** bits - 1)
    return (floor + code * step).reshape(x.shape)
