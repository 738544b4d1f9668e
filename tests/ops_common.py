"""Plain 64-bit forms of the operators over a paged cache, and caches to test them on.

E4M3 is written out from its definition (sign, 4 exponent bits of bias 7, 3 mantissa bits, no
infinities, codes 0x7f / 0xff are NaN); nothing here calls the library."""
import math

import numpy as np
import torch

HALF_EPS = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


def e4m3_values() -> np.ndarray:
    v = np.empty(256)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v[b] = math.nan if b & 127 == 127 else (-x if b & 128 else x)
    return v


E4M3 = e4m3_values()


def quantise(x: np.ndarray):
    """Rows of float64 values -> (codes, scales): the least power of two s >= 2^-126 with max|x| / s <=
    448 over finite values, then the nearest code, ties to the even code, saturating."""
    a = np.abs(x)
    amax = np.where(np.isfinite(a), a, 0).max(-1)
    s = np.ones_like(amax)
    for i in np.ndindex(amax.shape):
        if amax[i] > 0:
            e = -126
            while amax[i] / 2.0 ** e > 448:
                e += 1
            s[i] = 2.0 ** e
    grid = E4M3[:127]
    with np.errstate(invalid="ignore"):
        y = np.minimum(a / s[..., None], 448.0)
    i = np.clip(np.searchsorted(grid, np.where(np.isnan(y), 0, y)), 1, 126)
    lo, hi = grid[i - 1], grid[i]
    with np.errstate(invalid="ignore"):
        up = (y - lo > hi - y) | ((y - lo == hi - y) & (i % 2 == 0))
    code = np.where(up, i, i - 1).astype(np.uint8)
    code = np.where(np.isnan(x), 127, code) | np.where(np.signbit(x), 128, 0).astype(np.uint8)
    return code.astype(np.uint8), s


def cache(n_pages, page, Hkv, hd, dtype, seed, order="pchd", spread=0.5, device="cuda"):
    """K and V caches of random rows in the given memory order of (page, cell, head, dim) and, for
    uint8 (E4M3 codes), their scales; with their float64 values [cells, Hkv, hd]."""
    rng = np.random.default_rng(seed)
    res = []
    for _ in range(2):
        x = rng.normal(size=(n_pages, page, Hkv, hd)) * np.exp(spread * rng.normal(size=(n_pages, page, Hkv, 1)))
        if dtype == torch.uint8:
            code, s = quantise(x)
            val = E4M3[code] * s[..., None]
            t, sc = torch.from_numpy(code), torch.from_numpy(s.astype(np.float32))
        else:
            t, sc = torch.from_numpy(x).to(dtype), None
            val = t.double().numpy()
        perm = ["pch".index(c) for c in order[:-1]] + [3]
        inv = [perm.index(i) for i in range(4)]
        t = t.permute(perm).contiguous().to(device).permute(inv)
        if sc is not None:
            sc = sc.permute(perm[:3]).contiguous().to(device).permute(inv[:3])
        res.append((t, sc, val.reshape(-1, Hkv, hd)))
    return res


def attention(q, kval, vval, tables, n_new, n_kv, page, window=0, n_sink=0, scale=None):
    """float64 attention and, per output, the sum of |weight * value| (the scale of its errors).
    q [tokens, H, hd]; kval, vval [cells, Hkv, hd]; rows without a visible key are zeros."""
    H, hd = q.shape[1:]
    Hkv = kval.shape[1]
    G = H // Hkv
    scale = hd ** -0.5 if scale is None else scale
    out, mag, smag = np.zeros(q.shape), np.zeros(q.shape), np.zeros(q.shape[:2])
    t0 = 0
    for s in range(len(n_new)):
        j = np.arange(n_kv[s])
        cells = np.asarray(tables[s], dtype=np.int64)[j // page] * page + j % page if n_kv[s] else j
        for t in range(n_new[s]):
            p = n_kv[s] - n_new[s] + t
            vis = j <= p
            if window:
                vis &= (j > p - window) | (j < n_sink)
            idx = cells[vis]
            if len(idx) == 0:
                continue
            for h in range(H):
                K, V = kval[idx, h // G], vval[idx, h // G]
                z = K @ q[t0 + t, h] * scale
                smag[t0 + t, h] = (np.abs(K) @ np.abs(q[t0 + t, h])).max() * abs(scale)
                w = np.exp(z - z.max())
                w /= w.sum()
                out[t0 + t, h] = w @ V
                mag[t0 + t, h] = w @ np.abs(V)
        t0 += n_new[s]
    return out, mag, smag


def attention_tol(out, mag, smag, dtype, n, hd, vmax):
    """How far a kernel may be from the float64 result, term by term:
      - a score is a float32 sum of hd products and three more roundings: an error of (hd + 4) 2^-24
        of sum |q k| scale (smag), the same again for a float32 q held in two 11-bit terms (2^-22 of each
        product); it changes a weight by as much, relatively, and 2^x costs 2^-22 more;
      - p is rounded to 11 bits (half a step 2^-11) for f16 activations and in 256-row bf16 tiles to 8
        bits (2^-9 is half a step of bf16: 2^-8 of the value at most), otherwise held to 2^-17;
      - p below f16's normal range (a second term's too): an absolute error of 2^-25 each, over n keys,
        against a weight sum of at least 2^6 (a row's largest p is 2^6 or more);
      - weights enter numerator and denominator: twice their relative error, of mag = sum w |v|;
      - float32 sums over n keys: n 2^-24 of mag (they are partial sums of positive terms at worst);
      - the output's own rounding."""
    p_err = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -17}[dtype]
    s_err = (hd + 4) * 2.0 ** -24 + (2.0 ** -22 if dtype == torch.float32 else 0)
    rel = 2 * (p_err + 2.0 ** -22 + s_err * smag[..., None] + n * 2.0 ** -24)
    return rel * mag + n * 2.0 ** -31 * vmax + HALF_EPS[dtype] * np.abs(out) + 1e-30
