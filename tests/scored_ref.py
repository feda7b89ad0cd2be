"""Plain 64-bit restatements of block-scaled quantisation and of scored
attention, and the inputs their tests use (test infrastructure)."""

from __future__ import annotations

import math

import numpy as np
import torch

from paged_kv_cache_68_gb300 import pagedkv

QMAX = {"fp8_e4m3": np.float32(448.0), "int8": np.float32(127.0)}
TINY = np.float32(2.0 ** -126)
TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


# -- 8-bit codes ---------------------------------------------------------------

def e4m3_value(codes):
    """Values of E4M3 codes (uint8), from the format: 4 exponent bits (bias 7),
    3 mantissa bits, no infinity, NaN at 0x7f / 0xff."""
    c = np.asarray(codes, np.uint8).astype(np.int64)
    s, e, m = c >> 7, (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v = np.where((e == 15) & (m == 7), np.nan, v)
    return np.where(s == 1, -v, v)


def e4m3_code(y):
    """Nearest E4M3 code (ties to even, saturating; NaN: 0x7f) of fp32 y."""
    y = np.asarray(y, np.float32).astype(np.float64)
    sign = (np.signbit(y).astype(np.int64)) << 7
    a = np.minimum(np.abs(np.nan_to_num(y, nan=0.0, posinf=1e9, neginf=-1e9)), 448.0)
    e = np.maximum(np.floor(np.log2(np.maximum(a, 1e-30))), -6.0)
    k = np.rint(a / np.exp2(e - 3)).astype(np.int64)      # 0 .. 16 steps of 2^(e - 3)
    code = np.where(e > -6, ((e.astype(np.int64) + 7) << 3) + (k - 8), k)
    code = np.minimum(code, 0x7e)
    return np.where(np.isnan(y), 0x7f, sign | code).astype(np.uint8)


def values(codes, cache):
    if cache == "int8":
        return np.asarray(codes, np.uint8).view(np.int8).astype(np.float64)
    return e4m3_value(codes)


def encode(y, cache):
    if cache == "int8":
        y = np.nan_to_num(np.asarray(y, np.float32), nan=0.0)
        return np.clip(np.rint(y), -127, 127).astype(np.int8).view(np.uint8)
    return e4m3_code(y)


def append_block_scaled(codes, scales, rows, slots, cache):
    """kv_append on a block-scaled pool, block by block (in place).  codes uint8
    [N, bs, H, D], scales fp32 [N, H], rows fp32 [T, H, D]."""
    n, bs = codes.shape[:2]
    blocks = {}
    for i, s in enumerate(slots):                        # the last row of a slot wins
        if 0 <= s < n * bs:
            blocks.setdefault(int(s) // bs, {})[int(s) % bs] = i
    for blk, rowmap in blocks.items():
        off = sorted(rowmap)
        x = rows[[rowmap[o] for o in off]].astype(np.float32)
        for h in range(codes.shape[2]):
            old = np.float32(0) if off[0] == 0 else scales[blk, h]
            fin = np.isfinite(x[:, h])
            a = np.float32(np.abs(np.where(fin, x[:, h], 0)).max())
            new = np.fmax(old, np.float32(a / QMAX[cache]))
            if new < TINY:
                new = np.float32(0)
            if cache == "int8" and (not fin.all() or np.isnan(old)):
                new = np.float32(np.nan)
            if old > 0 and new > old:
                f = np.float32(old / new)
                keep = [r for r in range(bs) if r not in rowmap]
                old_v = values(codes[blk, keep, h], cache).astype(np.float32)
                codes[blk, keep, h] = encode(old_v * f, cache)
            inv = np.float32(np.float32(1) / new) if new > 0 else np.float32(0)
            with np.errstate(invalid="ignore", over="ignore"):
                q = encode(x[:, h] * inv, cache)
            if np.isnan(new):
                q = np.zeros_like(q)
            codes[blk, off, h] = q
            scales[blk, h] = new


# -- attention --------------------------------------------------------------------

def attention(q, k, v, table, L, positions, scale, *, softcap=0.0, slopes=None, window=0,
              first=None, prefix=0):
    """One request, 64-bit: q [n, Hq, D] at `positions`; k, v [N, bs, Hkv, D]."""
    n, hq, d = q.shape
    bs, hkv = k.shape[1], k.shape[2]
    out = np.zeros((n, hq, d))
    if L <= 0:
        return out
    blocks = np.asarray(table[:-(-L // bs)], np.int64)
    kk = k[blocks].reshape(-1, hkv, d)[:L]
    vv = v[blocks].reshape(-1, hkv, d)[:L]
    t = np.arange(L)
    for i in range(n):
        p = int(positions[i])
        if p < 0:
            continue
        ok = (t <= p) | (t < min(prefix, L))
        if window > 0:
            ok &= t > p - window
        if first is not None:
            ok &= t >= first[i]
        if not ok.any():
            continue
        for h in range(hq):
            g = h // (hq // hkv)
            s = scale * (kk[ok, g] @ q[i, h])
            if softcap > 0:
                s = softcap * np.tanh(s / softcap)
            if slopes is not None:
                s = s - slopes[h] * np.abs(p - t[ok])
            w = np.exp(s - s.max())
            out[i, h] = (w / w.sum()) @ vv[ok, g]
    return out


def check(got, ref, dtype, what=""):
    """16-bit: half a step of the output type, eps / 2 relative, and 5e-4 for the
    fp32 arithmetic: scores of |q||k| scale <= 15 summed over 128 products wander
    by sqrt(128) 2^-24 15 = 1e-5, the weights' hi + lo halves and exp2 add 2^-15,
    a cap of 50 adds 50 2^-22 = 1.2e-5; twice their sum (numerator and
    denominator) times |v| <= 5 is 2.5e-4 at most, taken twice.  fp32: the
    library's 1e-5 for inputs of unit variance."""
    got, ref = np.asarray(got, np.float64), np.asarray(ref)
    assert got.shape == ref.shape, (got.shape, ref.shape)
    assert np.isfinite(got).all(), f"{what}: {int((~np.isfinite(got)).sum())} values not finite"
    eps = {"f32": 0.0, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}[dtype]
    lim = (1e-5 if dtype == "f32" else 5e-4) + eps * np.abs(ref)
    err = np.abs(got - ref)
    assert (err <= lim).all(), \
        f"{what}: {int((err > lim).sum())} over the bound, worst {err.max():.3e} of {np.abs(ref).max():.3g}"


class Setup:
    """A pool of one kind over `lens`, with rows outside the sequences, and blocks
    outside the tables, holding NaN (16-bit, fp32, FP8) or a large code (INT8)."""

    def __init__(self, kind, dtype, lens, *, hq, hkv, d=128, bs=16, seed=0):
        rng = np.random.default_rng(seed)
        self.kind, self.dtype, self.lens = kind, dtype, np.asarray(lens, np.int64)
        self.hq, self.hkv, self.d, self.bs = hq, hkv, d, bs
        nb = -(-self.lens // bs)
        used = int(nb.sum())
        n = used + 3
        perm = rng.permutation(n)[:used].astype(np.int32)
        self.tables = np.full((len(lens), max(1, int(nb.max())) + 1), -1, np.int32)
        live = np.zeros((n, bs), bool)
        at = 0
        for b, m in enumerate(nb):
            self.tables[b, :m] = perm[at:at + m]
            for j in range(int(m)):
                live[perm[at + j], :min(bs, int(self.lens[b]) - j * bs)] = True
            at += int(m)
        self.n = n
        shape = (n, bs, hkv, d)
        self.ks = self.vs = None
        self.k_scale = self.v_scale = 1.0
        vals, self.dev = [], []
        if kind == "plain":
            for _ in range(2):
                x = torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(TORCH[dtype])
                vals.append(x.double().numpy())
                x[torch.from_numpy(~live)] = float("nan")
                self.dev.append(x.cuda())
        else:
            cache = "fp8_e4m3" if kind.startswith("fp8") else "int8"
            self.cache = cache
            sshape = (n, hkv) if kind.endswith("_block") else (n, hkv, bs)
            sc = []
            for _ in range(2):
                x = rng.standard_normal(shape)
                if cache == "int8":
                    c = np.clip(np.rint(x * 40), -127, 127).astype(np.int8).view(np.uint8)
                else:
                    c = encode((x * (90 if kind.endswith("_block") else 1)).astype(np.float32), cache)
                unit = 1 / 40 if cache == "int8" else (1 / 90 if kind.endswith("_block") else 1.0)
                s = (unit * np.exp(0.4 * rng.standard_normal(sshape))).astype(np.float32)
                v = values(c, cache)
                if kind == "fp8_e4m3":
                    f = 0.75 if not sc else 1.25
                    v = v * f
                elif kind.endswith("_block"):
                    v = v * s[:, None, :, None].astype(np.float64)
                else:
                    v = v * s.transpose(0, 2, 1)[..., None].astype(np.float64)
                vals.append(v)
                c[~live] = 0x7f
                self.dev.append(torch.from_numpy(c).cuda())
                sc.append(s)
            if kind == "fp8_e4m3":
                self.k_scale, self.v_scale = 0.75, 1.25
            else:
                self.ks, self.vs = (torch.from_numpy(s).cuda() for s in sc)
        self.k, self.v = vals
        self.scale = 1.0 / math.sqrt(d)
        self.rng = rng

    def pool(self):
        dt = TORCH[self.dtype]
        if self.kind == "plain":
            return pagedkv.KVPool(*self.dev)
        kw = dict(cache=self.cache, dtype=dt, k_scales=self.ks, v_scales=self.vs)
        if self.kind.endswith("_block"):
            return pagedkv.KVPool(*self.dev, scale_per="block", **kw)
        return pagedkv.KVPool(*self.dev, k_scale=self.k_scale, v_scale=self.v_scale, **kw)

    def queries(self, n):
        x = torch.from_numpy(self.rng.standard_normal((n, self.hq, self.d)).astype(np.float32))
        return x.to(TORCH[self.dtype])


def cuda_i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()
