"""Inputs, a plain 64-bit form and error bounds for the shared-prefix decode."""
import dataclasses

import numpy as np

from qkv_testutil import bf16_bits, bf16_values


@dataclasses.dataclass
class Batch:
    hq: int
    hkv: int
    prefix: int
    suffix: tuple         # own tokens of each sequence (the query's among them)
    S: int
    W: int
    seed: int = 0
    outliers: float = 0.01
    sm_scale: float = 1 / 16

    def make(self):
        rng = np.random.default_rng(self.seed)
        n, pb = len(self.suffix), self.prefix // 16
        own = [(x + 15) // 16 for x in self.suffix]
        self.n_pool, self.max_pages = pb + sum(own) + 2, pb + max(own) + 1
        perm = rng.permutation(self.n_pool)
        self.block_table = np.full((n, self.max_pages), -5, np.int32)  # entries that must not be read
        self.block_table[0, :pb] = perm[:pb]
        at = pb
        for i, k in enumerate(own):
            self.block_table[i, pb:pb + k] = perm[at:at + k]
            at += k
        shape = (self.n_pool, 16, self.hkv, 256)
        x = rng.standard_normal((2,) + shape).astype(np.float32)
        x *= np.where(rng.random((1,) + shape[:2] + (1, 1)) < self.outliers, 8, 1)
        scale = (np.abs(x).max(-1) / 127).astype(np.float32)
        codes = np.rint(x / scale[..., None]).astype(np.int8)
        # slots of no token: never read, or masked whatever they hold
        used = np.zeros(shape[:2], bool)
        used[perm[:pb]] = True
        for i, (k, m) in enumerate(zip(own, self.suffix)):
            flat = np.zeros(16 * k, bool)
            flat[:m] = True
            used[self.block_table[i, pb:pb + k]] = flat.reshape(k, 16)
        scale[:, ~used] = np.nan
        self.k_pool, self.v_pool = codes
        self.k_scale, self.v_scale = scale
        self.rows = rng.permutation(n + 3)[:n]  # rows of q / out, some of no sequence
        self.q = bf16_bits(rng.standard_normal((n + 3, self.hq, 256)).astype(np.float32))
        ctx = self.prefix + np.array(self.suffix)
        self.seqs = np.stack([self.rows, ctx - 1, np.ones_like(ctx), ctx], 1).astype(np.int32)
        return self

    def visible(self, i):
        t = self.prefix + self.suffix[i] - 1
        j = np.arange(t + 1)
        if self.W > 0:
            j = j[(j // 16 < self.S) | (j // 16 >= max(0, t // 16 + 1 - self.W))]
        return j

    def reference(self, skip_pages=(), only=None):
        """Per sequence (of `only`, if given) (out, bound) float64 [hq, 256].  The bound, per output:
          2^-8 |out|             bf16 rounding of the result
          2^-11 sum p |v|        P' rounded to fp16 (half a step), and where P' is subnormal (below 2^-14 of its
                                 largest) half its fixed step, 2^-25, times the largest V magnitude
          score errors e_j       fp32 sums of 256 products (each addition within 2^-23 of sum |q k|), the scale
                                 products and the exponent's (2^-21 of |score|), 2^-21 for 2^x itself: they move
                                 p_j by a factor 1 + e_j, the output by sum p e |v| + |out| sum p e"""
        pb, G, out = self.prefix // 16, self.hq // self.hkv, []
        for i in range(len(self.suffix)) if only is None else only:
            j = self.visible(i)
            row = np.where(j // 16 < pb, 0, i)
            page = self.block_table[row, j // 16]
            keep = ~np.isin(page, skip_pages)
            j, page = j[keep], page[keep]
            k = self.k_pool[page, j % 16].astype(np.float64) * self.k_scale[page, j % 16][..., None]
            v = self.v_pool[page, j % 16].astype(np.float64) * self.v_scale[page, j % 16][..., None]
            vs = self.v_scale[page, j % 16].astype(np.float64)
            q = bf16_values(self.q[self.rows[i]]).reshape(self.hkv, G, 256)
            o, b = np.empty((self.hq, 256)), np.empty((self.hq, 256))
            for g in range(self.hkv):
                s = q[g] @ k[:, g].T * self.sm_scale
                sabs = np.abs(q[g]) @ np.abs(k[:, g]).T * self.sm_scale
                p = np.exp(s - s.max(-1, keepdims=True))
                rel = p * vs[:, g] / vs[:, g].max()  # P' against its largest possible value
                p /= p.sum(-1, keepdims=True)
                e = 256 * 2.0 ** -23 * sabs + 2.0 ** -21 * (np.abs(s) + np.abs(s).max(-1, keepdims=True) + 2)
                av = np.abs(v[:, g])
                r = p @ v[:, g]
                tiny = (rel < 2.0 ** -13).sum(-1, keepdims=True) * 2.0 ** -25 * 2 * vs[:, g].max() * 127
                heads = slice(g * G, g * G + G)
                o[heads] = r
                b[heads] = (2.0 ** -8 * np.abs(r) + (1 + 2.0 ** -8) * (
                    2.0 ** -11 * (p @ av) + tiny + (p * e) @ av + np.abs(r) * (p * e).sum(-1, keepdims=True)))
            out.append((o, b))
        return np.stack([x[0] for x in out]), np.stack([x[1] for x in out])
