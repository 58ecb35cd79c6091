"""Plain references of the 8-bit cache, the attention over it and the norm, written from the
definitions in include/moe_kv8.h byte by byte (numpy on the CPU; no kernel or package code)."""
import numpy as np
import torch

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
#: half an ulp of a value in [1, 2), relative
HALF_ULP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def k_index(D):
    """[32, D] byte offsets of the key codes in a record."""
    at = np.zeros((32, D), np.int64)
    for t in range(32):
        for d in range(D):
            group, row = (t // 2) % 4, 2 * (t // 8) + t % 2
            at[t, d] = 16 + ((group * (D // 32) + d // 32) * 8 + row) * 32 + d % 32
    return at


def v_index(D):
    at = np.zeros((32, D), np.int64)
    for t in range(32):
        for d in range(D):
            at[t, d] = 16 + 32 * D + d * 32 + t
    return at


class Cache:
    """A host copy of a pool, with the plain write and read."""

    def __init__(self, pool, table):
        self.pool, self.table = pool.copy(), table
        self.P, self.D = pool.shape[2] * 32, (pool.shape[3] - 16) // 64
        self.at = (k_index(self.D), v_index(self.D))

    def block(self, b, j):
        """Records [heads, bytes] of block j of sequence b (a view)."""
        return self.pool[self.table[b, j * 32 // self.P], :, (j * 32 % self.P) // 32]

    def codes(self, b, j, h, w):
        rec = self.block(b, j)[h]
        return rec[self.at[w]].astype(np.int32) - 128, rec[4 * w:4 * w + 4].view(np.float32)[0]

    def write(self, b, start, rows):
        """rows: (k, v) float32 [n, heads, D]."""
        n = rows[0].shape[0]
        with np.errstate(all="ignore"):
            for j in range(start // 32, (start + n + 31) // 32 if n else 0):
                t0, t1 = max(0, start - 32 * j), min(32, start + n - 32 * j)
                for h in range(rows[0].shape[1]):
                    for w in range(2):
                        x = rows[w][32 * j + t0 - start:32 * j + t1 - start, h]
                        c, old = self.codes(b, j, h, w)
                        old = np.float32(old if t0 else 0)
                        amax = np.abs(x).max()
                        scale = np.float32(0) if amax < np.float32(2.0 ** -100) else np.float32(amax) / np.float32(127)
                        scale = np.maximum(old, scale)  # a NaN stays
                        if not np.isfinite(scale):
                            scale = np.float32(np.nan)
                        if scale > 0:
                            c[:t0] = np.rint(c[:t0].astype(np.float32) * (old / scale))
                            c[t0:t1] = np.clip(np.rint(x * (np.float32(1) / scale)), -127, 127)
                        else:
                            c[:t1] = 0
                        rec = self.block(b, j)[h]
                        rec[self.at[w][:t1]] = (c[:t1] + 128).astype(np.uint8)
                        rec[4 * w:4 * w + 4] = np.frombuffer(np.float32(scale).tobytes(), np.uint8)

    def read(self, b, p0, p1):
        """fp32 keys and values [p1 - p0, heads, D]."""
        out = [np.zeros((p1 - p0, self.pool.shape[1], self.D), np.float32) for _ in range(2)]
        for j in range(p0 // 32, (p1 + 31) // 32 if p1 > p0 else 0):
            t0, t1 = max(0, p0 - 32 * j), min(32, p1 - 32 * j)
            for h in range(self.pool.shape[1]):
                for w in range(2):
                    c, s = self.codes(b, j, h, w)
                    out[w][32 * j + t0 - p0:32 * j + t1 - p0, h] = c[t0:t1].astype(np.float32) * s
        return out


def random_pool(rng, n_pages, hkv, D, page, scale=0.03):
    pool = rng.integers(1, 256, (n_pages, hkv, page // 32, 64 * D + 16), dtype=np.uint8)
    s = (scale * np.exp(0.4 * rng.standard_normal((n_pages, hkv, page // 32, 2)))).astype(np.float32)
    pool[..., :8] = s.view(np.uint8).reshape(*s.shape[:3], 8)
    return pool


def page_table(rng, tokens, page, spare=2):
    """A table of distinct pages for sequences of `tokens` positions, unused entries -1; and the pool's pages."""
    need = [-(-t // page) for t in tokens]
    ids = rng.permutation(sum(need) + spare)
    table = np.full((len(need), max(max(need), 1)), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    return table, sum(need) + spare


def attention(q, cache, lens, scale, window=0, tree=None):
    """fp64 out [B, T, hq, D] and lse, and per output the bounds that the error analysis needs:
    reach = max |v| over the positions seen, size = max over them of scale * sum |q| |k|."""
    B, T, hq, D = q.shape
    hkv = cache.pool.shape[1]
    out, lse = np.zeros((B, T, hq, D)), np.full((B, T, hq), -np.inf)
    reach, size = np.zeros((B, T, hq, 1)), np.zeros((B, T, hq))
    for b in range(B):
        n = int(lens[b])
        if n <= 0:
            continue
        k, v = (x.astype(np.float64) for x in cache.read(b, 0, n))
        j = np.arange(n)
        for t in range(T):
            p = n - T + t
            if p < 0:
                continue
            if tree is None:
                see = j <= p
            else:
                see = np.array([i < n - T or bool(int(tree[b, t]) >> (i - n + T) & 1) for i in range(n)])
            if window:
                see &= j > p - window
            if not see.any():
                continue
            for h in range(hq):
                kk, vv = k[see, h // (hq // hkv)], v[see, h // (hq // hkv)]
                s = kk @ q[b, t, h] * scale
                m = s.max()
                e = np.exp(s - m)
                out[b, t, h] = e @ vv / e.sum()
                lse[b, t, h] = m + np.log(e.sum())
                reach[b, t, h], size[b, t, h] = np.abs(vv).max(), (np.abs(kk) @ np.abs(q[b, t, h])).max() * abs(scale)
    return out, lse, reach, size
