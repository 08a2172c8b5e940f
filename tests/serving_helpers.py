"""A filled paged cache and the serving operators' definitions in 64 bits (numpy)."""
from __future__ import annotations

import math

import numpy as np

from oracle import quant as OQ
from tests.gpu_helpers import codebook_for


class Pool:
    """A paged cache on the GPU with every slot written, and its dequantized values here.

    Slots that no sequence owns hold ordinary values too; ``poison`` overwrites the scales of
    given slots with NaN, as memory of an ended request may hold anything."""

    def __init__(self, fmt, D, hkv, page_size, num_pages, seed=0, scale=1.0, device="cuda"):
        import torch
        import quantized_kv_cache_split_b200 as K
        rng = np.random.Generator(np.random.PCG64(seed))
        self.fmt, self.D, self.hkv, self.ps, self.num_pages = fmt, D, hkv, page_size, num_pages
        self.signs = np.where(rng.random(D) < 0.5, -1, 1).astype(np.int8) if fmt == "lut4" else None
        self.cb = codebook_for(D) if fmt == "lut4" else None
        self.cache = K.QuantizedKVCache(fmt, D, hkv, page_size, num_pages, device,
                                        None if self.cb is None else torch.from_numpy(self.cb.view(np.int16).copy()),
                                        None if self.signs is None else torch.from_numpy(self.signs))
        n = num_pages * page_size
        k = (rng.standard_normal((n, hkv, D)) * scale).astype(np.float16)
        v = rng.standard_normal((n, hkv, D)).astype(np.float16)
        u = rng.choice([-1.0, 1.0], D)
        k[rng.random(n) < 0.02] += np.float16(0.8) * u.astype(np.float16)   # some strong keys
        self.u = u
        self.rng = rng
        self.cache.write(torch.from_numpy(k).to(device), torch.from_numpy(v).to(device))
        torch.cuda.synchronize()
        self.k, self.v = self.values("k"), self.values("v")

    def values(self, which):
        """fp64 [slots, heads, D] of a plane pair as the GPU holds it (rotated for lut4)."""
        codes = getattr(self.cache, which + "_codes").cpu().numpy()
        scales = getattr(self.cache, which + "_scales").cpu().numpy()
        if self.fmt == "q8_0":
            codes = codes.view(np.int8)
        else:
            codes = OQ.unpack_nibbles(codes)
        if self.fmt == "nvfp4":
            scales = scales.view(np.uint16)
        x = OQ.dequantize(self.fmt, codes, scales, self.cb)
        return x.transpose(0, 2, 1, 3).reshape(-1, self.hkv, self.D)

    def queries(self, n, hq):
        q = self.rng.standard_normal((n, hq, self.D)) + 0.6 * self.u
        return q.astype(np.float16)

    def slots_of(self, pages, n):
        p = np.arange(n)
        return np.asarray(pages, dtype=np.int64)[p // self.ps] * self.ps + p % self.ps

    def poison(self, slots):
        """NaN scales (nvfp4: NaN block and vector scales) at slots that no result may read."""
        import torch
        for s in np.asarray(slots):
            page, off = int(s) // self.ps, int(s) % self.ps
            for plane in (self.cache.k_scales, self.cache.v_scales):
                plane[page, :, off] = float("nan")
        torch.cuda.synchronize()

    def attend(self, q, slots, sm_scale):
        """One token's heads q [hq, D] (fp16) over `slots`: (out, bound) fp64 [hq, D].

        bound: what the kernels' stated roundings can change at the most.  With u = 2^-11
        (half a step of fp16), a K value is off by cK u relative (cK = 1: code * scale rounded
        once; 2 for nvfp4, whose block scale is rounded first; 2 for lut4, where the rotated
        query is rounded as well), so a score by d <= |sm_scale| cK u sum |q||k|, a weight
        relative to the sum by e^(2d) - 1; the weight itself is rounded to fp16 (u), a V value
        by cV u (1, nvfp4 2), and sums of n fp32 terms by 2^-22 each (the tensor core's
        additions truncate).  Each of these scales the average of |v| under the weights.  The
        smallest fp16 steps add 2^-25 per value and, with the largest weight at 2, 2^-26 of it
        per position."""
        hq, g = q.shape[0], q.shape[0] // self.hkv
        out, bound = np.zeros((hq, self.D)), np.zeros((hq, self.D))
        if len(slots) == 0:
            return out, bound
        u = 2.0 ** -11
        ck, cv = {"q8_0": (1, 1), "q4_0": (1, 1), "lut4": (2, 1), "nvfp4": (2, 2)}[self.fmt]
        qr = q.astype(np.float64)
        if self.fmt == "lut4":
            qr = OQ.rotate_f64(qr, self.signs)
        for h in range(self.hkv):
            qh, k, v = qr[h * g:(h + 1) * g], self.k[slots, h], self.v[slots, h]
            s = sm_scale * (qh @ k.T)
            d = abs(sm_scale) * ((ck * u + 2.0 ** -20) * (np.abs(qh) @ np.abs(k).T)
                                 + 2.0 ** -25 * np.abs(qh).sum(-1, keepdims=True)).max(-1, keepdims=True)
            p = np.exp(s - s.max(-1, keepdims=True))
            p /= p.sum(-1, keepdims=True)
            o = p @ v
            av = p @ np.abs(v)
            e = np.expm1(2 * d) + (1 + cv) * u + len(slots) * 2.0 ** -22
            b = av * e + 2.0 ** -24 + len(slots) * 2.0 ** -26 * np.abs(v).max()
            if self.fmt == "lut4":   # rotated back: each element is a signed mean of all, times sqrt(D)
                o = OQ.unrotate_f64(o, self.signs)
                b = np.repeat(b.sum(-1, keepdims=True) / math.sqrt(self.D), self.D, -1)
            out[h * g:(h + 1) * g], bound[h * g:(h + 1) * g] = o, b
        return out, bound


def check_close(got, want, bound, half):
    """|got - want| <= bound, plus the output's own rounding (fp16: 2^-11 relative, 2^-25 at least)."""
    got = got.astype(np.float64)
    tol = bound + ((np.abs(want) + bound) * 2.0 ** -11 + 2.0 ** -25 if half else 2.0 ** -22 * np.abs(want))
    assert np.isfinite(got).all()
    bad = np.abs(got - want) > tol
    assert not bad.any(), f"{bad.sum()} of {bad.size}, worst {np.max(np.abs(got - want) / np.maximum(tol, 1e-30)):.2f} x the bound"
    norm = np.linalg.norm(want)
    return float(np.linalg.norm(got - want) / norm) if norm else 0.0


def plan_reference(seq_lens, new_lens, free, count, table, page_size, max_tokens):
    """kvq_plan_step in plain Python: the definition, one page and one token at a time."""
    table = table.copy()
    stack = [int(x) for x in free[:count]]
    for b, a in enumerate(new_lens):
        if a == -1:
            stack += [int(x) for x in table[b, :-(-int(seq_lens[b]) // page_size)]]
    slots, pos, offsets, lens = [], [], [0], []
    for b, a in enumerate(new_lens):
        n, a = int(seq_lens[b]), int(a)
        if a >= 0:
            for j in range(-(-n // page_size), -(-(n + a) // page_size)):
                table[b, j] = stack.pop()
            for p in range(n, n + a):
                slots.append(int(table[b, p // page_size]) * page_size + p % page_size)
                pos.append(p)
        offsets.append(len(slots))
        lens.append(n + a if a >= 0 else 0)
    rest = max_tokens - len(slots)
    return dict(table=table, stack=np.array(stack, dtype=np.int32), lens=np.array(lens), offsets=np.array(offsets),
                slots=np.array(slots + [-1] * rest), positions=np.array(pos + [0] * rest))
