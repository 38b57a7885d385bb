"""Plain 64-bit forms of the masked attention, key-mass and eviction calls, and
seeded caches to run them on (imported by their test modules).  Written from
the formulas in include/kvq.h, on numpy arrays; nothing here calls the
library."""
import dataclasses

import numpy as np

INT8, FP8, INT4 = 1, 2, 3
ROW, TENSOR, CHANNEL, GROUP = 1, 2, 3, 4


def e4m3_table():
    """The 256 e4m3 values (NaN for S.1111.111)."""
    t = np.zeros(256)
    for c in range(256):
        s, e, m = c >> 7, (c >> 3) & 15, c & 7
        v = (m / 8) * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        if e == 15 and m == 7:
            v = np.nan
        t[c] = -v if s else v
    return t


E4M3 = e4m3_table()


def bf16(x):
    """fp32 array rounded to bf16 (nearest, ties to even), as fp32."""
    u = np.ascontiguousarray(x, np.float32).view(np.uint32).astype(np.uint64)
    u = (u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000
    return u.astype(np.uint32).view(np.float32)


@dataclasses.dataclass
class Case:
    dtype: int = INT8
    km: int = ROW
    vm: int = ROW
    gs: int = 0
    d: int = 128
    hq: int = 8
    hkv: int = 2
    bs: int = 16
    lens: tuple = (100,)
    c: int = 1                 # query tokens per sequence
    softcap: float = 0.0
    window: int = 0
    latent: bool = False
    dv: int = 0                # LATENT: v_head_size
    slack: int = 3             # unused pages in the pool
    sm_scale: float = 0.0
    seed: int = 0
    amp: float = 1.0           # size of the queries

    @property
    def group(self):
        return self.hq // self.hkv

    @property
    def scale(self):
        return self.sm_scale if self.sm_scale > 0 else self.d ** -0.5


class Cache:
    """Random codes and scales in the cache's layout.  Rows of positions that
    the sequences do not have hold `junk`: NaN scales, e4m3 NaN codes."""

    def __init__(self, case: Case, width=None):
        self.case = case
        r = np.random.default_rng(case.seed + 17)
        bs, hkv, d = case.bs, case.hkv, case.d
        need = [max(1, -(-L // bs)) for L in case.lens]
        self.width = width or max(need)
        self.nb = sum(need) + case.slack
        perm = r.permutation(self.nb)
        self.table = np.full((len(need), self.width), self.nb - 1, np.int32)
        at, used = 0, np.zeros((self.nb, bs), bool)
        for b, n in enumerate(need):
            self.table[b, :n] = perm[at:at + n]
            at += n
            for p in range(case.lens[b]):
                used[self.table[b, p // bs], p % bs] = True
        self.used = used
        dp = d // 2 if case.dtype == INT4 else d

        def side(mode):
            if case.dtype == FP8:
                codes = r.integers(0, 0x7F, (self.nb, hkv, bs, d)).astype(np.uint8)
                codes = np.minimum(codes, 0x7E) | (r.integers(0, 2, codes.shape).astype(np.uint8) << 7)
                top = 60.0  # typical size of a random code's value
            elif case.dtype == INT8:
                codes = r.integers(-127, 128, (self.nb, hkv, bs, d)).astype(np.int8).view(np.uint8)
                top = 73.0
            else:
                lo, hi = r.integers(-7, 8, (2, self.nb, hkv, bs, dp))
                codes = ((lo & 15) | ((hi & 15) << 4)).astype(np.uint8)
                top = 4.3
            shape = {ROW: (self.nb, hkv, bs), TENSOR: (1,), CHANNEL: (hkv, d),
                     GROUP: (self.nb, hkv, bs, d // case.gs if case.gs else 1)}[mode]
            scale = (np.exp(0.4 * r.standard_normal(shape)) / top).astype(np.float32)
            if case.dtype == FP8:
                codes[~np.broadcast_to(used[:, None, :], codes.shape[:3])] = 0x7F
            if mode in (ROW, GROUP):
                scale[~np.broadcast_to(used[:, None, :], scale.shape[:3])] = np.nan
            return codes, scale

        self.k_codes, self.k_scale = side(case.km)
        if case.latent:
            self.v_codes, self.v_scale = self.k_codes, self.k_scale
        else:
            self.v_codes, self.v_scale = side(case.vm)
        self.q = bf16(case.amp * r.standard_normal((len(need), case.c, case.hq, d)))

    def rows(self, b):
        p = np.arange(self.case.lens[b])
        return self.table[b, p // self.case.bs], p % self.case.bs

    def largest(self, b, h, lo, hi):
        """The largest |value| a V row of [lo, hi) could hold: code range times
        the largest scale."""
        c = self.case
        scale, mode = (self.k_scale, c.km) if c.latent else (self.v_scale, c.vm)
        blk, row = self.rows(b)
        s = scale[blk[lo:hi], h, row[lo:hi]] if mode in (ROW, GROUP) else (scale[h] if mode == CHANNEL else scale)
        return {INT8: 128.0, FP8: 448.0, INT4: 8.0}[c.dtype] * float(s.max())

    def values(self, b, h, side):
        """fp64 [L, D] values of sequence b's rows, kv head h."""
        c = self.case
        codes, scale, mode = ((self.k_codes, self.k_scale, c.km) if side == "k" or c.latent else
                              (self.v_codes, self.v_scale, c.vm))
        blk, row = self.rows(b)
        w = codes[blk, h, row]
        if c.dtype == INT8:
            x = w.view(np.int8).astype(np.float64)
        elif c.dtype == FP8:
            x = E4M3[w]
        else:
            x = np.empty((len(blk), c.d))
            x[:, 0::2], x[:, 1::2] = (w & 15).astype(float), (w >> 4).astype(float)
            x = np.where(x > 7, x - 16, x)
        s = scale.astype(np.float64)
        if mode == ROW:
            x = x * s[blk, h, row][:, None]
        elif mode == TENSOR:
            x = x * s[0]
        elif mode == CHANNEL:
            x = x * s[h]
        else:
            x = x * np.repeat(s[blk, h, row], c.gs, axis=1)
        return x[:, :c.dv] if side == "v" and c.latent and c.dv else x


def visible(case, b, c, key_begin=None, key_end=None):
    """[lo, hi) of token c of sequence b."""
    L = case.lens[b]
    pos = L - case.c + c
    lo = 0 if key_begin is None else max(0, int(key_begin[b, c]))
    hi = pos + 1 if key_end is None else int(key_end[b, c])
    if case.window > 0:
        lo = max(lo, pos - case.window + 1)
    return lo, min(hi, L), pos


def attend(cache: Cache, slopes=None, key_begin=None, key_end=None, sink=None):
    """out [B, C, Hq, Dv], lse [B, C, Hq], and what the tolerances need: the
    mean absolute value sum_j p_j |v_j| per channel, the error that the f16 weights leave in out, and the largest
    sum_d |q_d k_d| sm_scale over a row's keys."""
    c = cache.case
    B, dv = len(c.lens), (c.dv or c.d) if c.latent else c.d
    out = np.zeros((B, c.c, c.hq, dv))
    absv, f16 = np.zeros_like(out), np.zeros_like(out)
    lse = np.full((B, c.c, c.hq), -np.inf)
    size = np.zeros((B, c.c, c.hq))
    for b in range(B):
        for h in range(c.hkv):
            k, v = cache.values(b, h, "k"), cache.values(b, h, "v")
            for g in range(c.group):
                hq = h * c.group + g
                for t in range(c.c):
                    lo, hi, pos = visible(c, b, t, key_begin, key_end)
                    if hi <= lo:
                        continue
                    q = cache.q[b, t, hq].astype(np.float64)
                    s = k[lo:hi] @ q * c.scale
                    size[b, t, hq] = (np.abs(k[lo:hi]) @ np.abs(q)).max() * c.scale
                    if c.softcap > 0:
                        s = c.softcap * np.tanh(s / c.softcap)
                    if slopes is not None:
                        s = s - float(slopes[hq]) * np.abs(pos - np.arange(lo, hi))
                    m = s.max()
                    p = np.exp(s - m)
                    lse[b, t, hq] = m + np.log(p.sum())
                    p /= p.sum()
                    f = 1.0
                    if sink is not None:
                        f = 1.0 / (1.0 + np.exp(float(sink[hq]) - lse[b, t, hq]))
                    out[b, t, hq] = p @ v[lo:hi] * f
                    absv[b, t, hq] = p @ np.abs(v[lo:hi]) * f
                    # Weights times V scales enter the product as f16: 2^-11 of
                    # each (twice, for the scaled V tile's own rounding), and
                    # below 2^-14 an absolute 2^-25 in units of the reference
                    # weight (at most the row's sum) and of 2^F, F the power of
                    # two at or above the largest V scale (at most twice it).
                    f16[b, t, hq] = 2.0 ** -10 * absv[b, t, hq] + 2.0 ** -24 * (hi - lo) * cache.largest(b, h, lo, hi)
    return out, lse, absv, f16, size


def key_mass(cache: Cache, lse, mass, decay, fresh, slopes=None, key_begin=None, key_end=None):
    """The new mass array (fp64) and the error bound of each entry."""
    c = cache.case
    new = mass.astype(np.float64).copy()
    tol = np.zeros_like(new)
    for b, L in enumerate(c.lens):
        blk, row = cache.rows(b)
        for h in range(c.hkv):
            k = cache.values(b, h, "k")
            add, err = np.zeros(L), np.zeros(L)
            for g in range(c.group):
                hq = h * c.group + g
                for t in range(c.c):
                    lo, hi, pos = visible(c, b, t, key_begin, key_end)
                    if hi <= lo or lse[b, t, hq] == -np.inf:
                        continue
                    q = cache.q[b, t, hq].astype(np.float64)
                    s = k[lo:hi] @ q * c.scale
                    size = np.abs(k[lo:hi]) @ np.abs(q) * c.scale
                    if c.softcap > 0:
                        s = c.softcap * np.tanh(s / c.softcap)
                    if slopes is not None:
                        s = s - float(slopes[hq]) * np.abs(pos - np.arange(lo, hi))
                    p = np.exp(s - float(lse[b, t, hq]))
                    add[lo:hi] += p
                    # a logit's error: at most 64 fp32 accumulations of partial
                    # sums up to `size` (2^6 * 2^-24) with the split operand's
                    # 2^-22, a few roundings of x and lse (2^-22 of them), and
                    # 2^-20 for exp2 and the fp32 sums of the weights
                    err[lo:hi] += p * (2.0 ** -17.5 * size + 2.0 ** -21 * (np.abs(s) + abs(lse[b, t, hq])) + 2.0 ** -20)
            old = np.where(np.arange(L) >= L - fresh, 0.0, decay * mass[blk, h, row].astype(np.float64))
            if decay == 0:
                old = np.zeros(L)
            new[blk, h, row] = old + add
            tol[blk, h, row] = err + 2.0 ** -22 * np.abs(old)
    return new, tol


def select(mass, table, lens, bs, budget, sinks, recent):
    """keep [B, Hkv, budget], kept_lens [B]."""
    B, hkv = len(lens), mass.shape[1]
    keep = np.full((B, hkv, budget), -1, np.int32)
    for b, L in enumerate(lens):
        n = min(L, budget)
        p = np.arange(L)
        for h in range(hkv):
            m = mass[table[b, p // bs], h, p % bs]
            if L <= budget:
                keep[b, h, :n] = p
                continue
            mid = list(range(sinks, L - recent))
            # NaN last; equal weights (and -0, +0) in index order
            mid.sort(key=lambda i: (1, 0.0, i) if np.isnan(m[i]) else (0, -float(m[i]) + 0.0, i))
            rows = list(range(sinks)) + mid[:budget - sinks - recent] + list(range(L - recent, L))
            keep[b, h] = np.sort(np.array(rows, np.int32))
    return keep, np.minimum(np.array(lens), budget).astype(np.int32)


def compact(arrays, src_table, dst_table, keep, kept_lens, bs):
    """The arrays ([num_blocks, Hkv, block_size, ...] each) after the move."""
    out = [a.copy() for a in arrays]
    for b in range(keep.shape[0]):
        n = int(kept_lens[b])
        i = np.arange(n)
        for h in range(keep.shape[1]):
            k = keep[b, h, :n]
            for a, o in zip(arrays, out):
                o[dst_table[b, i // bs], h, i % bs] = a[src_table[b, k // bs], h, k % bs]
    return out
