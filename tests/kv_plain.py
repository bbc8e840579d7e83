"""Plain implementation of the quantised key/value cache and its attention for the tests: the page layout
by index formulas, the quantisation in fp32 as the format defines it, attention in 64 bits.  Shares no code
with the package."""
import numpy as np
import torch


class Fmt:
    def __init__(self, hkv=2, d=128, bits=4, g=64, page=16):
        self.hkv, self.d, self.bits, self.g, self.page = hkv, d, bits, g, page
        self.code_bytes = page * d * bits // 8
        self.meta_bytes = 4 * page * (d // g)
        self.block = 2 * (self.code_bytes + self.meta_bytes)

    def bit_of(self, which, t, c):
        """Bit offset within a block of channel c's code of the page's token t."""
        if which == "k":
            i, h, j = c // 32, c % 32 // 8, c % 8
            at = t * self.d * self.bits + (h * (self.d // 32) + i) * 8 * self.bits
            return at + (4 * [0, 4, 1, 5, 2, 6, 3, 7][j] if self.bits == 4 else 8 * j)
        u = self.d // 16
        return 8 * self.code_bytes + (((t // 4) * 16 + c // u) * 4 + t % 4) * u * self.bits + c % u * self.bits

    def meta_of(self, which, t, group):
        """Byte offset within a block of the step of token t's group (the floor follows)."""
        return 2 * self.code_bytes + (0 if which == "k" else self.meta_bytes) + 4 * (group * self.page + t)


def quantise(x, bits, g):
    """Codes (int), steps and floors (fp16 arrays) of x [..., D] fp32, in fp32."""
    x = np.asarray(x, np.float32)
    x = np.clip(np.where(np.isnan(x), np.float32(0), x), np.float32(-65504), np.float32(65504))
    x = x.reshape(*x.shape[:-1], x.shape[-1] // g, g)
    floor = x.min(-1).astype(np.float16)
    f32 = floor.astype(np.float32)
    step = np.maximum((x.max(-1) - f32) * np.float32(1.0 / (2 ** bits - 1)), np.float32(0)).astype(np.float16)
    s32 = step.astype(np.float32)
    inv = np.divide(np.float32(1), s32, out=np.zeros_like(s32), where=s32 > 0)
    code = np.clip(np.rint((x - f32[..., None]) * inv[..., None]), 0, 2 ** bits - 1).astype(np.int64)
    return code.reshape(*code.shape[:-2], code.shape[-2] * g), step, floor


def stands_for(code, step, floor):
    """fp32 floor + code * step, each operation rounded."""
    g = code.shape[-1] // step.shape[-1]
    c = code.reshape(*step.shape, g).astype(np.float32)
    x = c * step.astype(np.float32)[..., None] + floor.astype(np.float32)[..., None]
    return x.reshape(code.shape)


def write(fmt, pages, k, v, slots):
    """Writes fp32 k, v [n, hkv, D] into numpy pages [P, hkv, block]."""
    bits = np.empty((2, fmt.page, fmt.d), np.int64)
    for w, which in enumerate("kv"):
        for t in range(fmt.page):
            for c in range(fmt.d):
                bits[w, t, c] = fmt.bit_of(which, t, c)
    mask = 2 ** fmt.bits - 1
    for w, (which, x) in enumerate((("k", k), ("v", v))):
        code, step, floor = quantise(x, fmt.bits, fmt.g)
        for n, slot in enumerate(slots):
            if slot < 0 or slot // fmt.page >= pages.shape[0]:
                continue
            p, t = slot // fmt.page, slot % fmt.page
            for h in range(fmt.hkv):
                b = pages[p, h]
                at, sh = bits[w, t] // 8, bits[w, t] % 8
                np.bitwise_and.at(b, at, (~(mask << sh) & 255).astype(np.uint8))
                np.bitwise_or.at(b, at, (code[n, h] << sh).astype(np.uint8))
                for q in range(fmt.d // fmt.g):
                    m = fmt.meta_of(which, t, q)
                    b[m:m + 2] = np.frombuffer(step[n, h, q].tobytes(), np.uint8)
                    b[m + 2:m + 4] = np.frombuffer(floor[n, h, q].tobytes(), np.uint8)


def as_f32(t):
    return t.float().cpu().numpy()


def attend(q, keys, vals, bound, scale):
    """Attention in 64 bits of q [T, H, D] over keys, vals [L, hkv, D] (fp64), row t seeing the keys j with
    bound[t, j].  Returns out, lse, the sum of weights times |values| (what roundings scale with), and
    the root sum of squares of the largest score's terms."""
    T, H, D = q.shape
    per = H // keys.shape[1]
    out, lse = np.zeros((T, H, D)), np.full((T, H), -np.inf)
    mag, terms = np.zeros((T, H, D)), np.zeros((T, H))
    for h in range(H):
        k, v = keys[:, h // per], vals[:, h // per]
        s = scale * (q[:, h] @ k.T)
        t2 = scale * np.sqrt((q[:, h] ** 2) @ (k ** 2).T)
        for t in range(T):
            on = bound[t]
            if not on.any():
                continue
            top = s[t, on].max()
            e = np.exp(s[t, on] - top)
            out[t, h] = e @ v[on] / e.sum()
            mag[t, h] = e @ np.abs(v[on]) / e.sum()
            lse[t, h] = top + np.log(e.sum())
            terms[t, h] = t2[t, on].max()
    return out, lse, mag, terms


def to(x, dtype):
    return torch.from_numpy(np.ascontiguousarray(x)).to(dtype)
