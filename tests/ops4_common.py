"""Plain 64-bit forms of the 4-bit cache rows (E2M1 codes, an E4M3 number per 16 values, a power-of-two
scale per row) and of the page tables, and caches to test them on; nothing here calls the library."""
import numpy as np
import torch

from tests import ops_common as O

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])


def nearest(grid, y):
    """Index of the value of the ascending grid nearest to y >= 0, ties to the even index."""
    i = np.clip(np.searchsorted(grid, y), 1, len(grid) - 1)
    lo, hi = grid[i - 1], grid[i]
    up = (y - lo > hi - y) | ((y - lo == hi - y) & (i % 2 == 0))
    return np.where(up, i, i - 1)


def quantise(x):
    """Rows of float64 values [..., hd] -> (codes [..., hd], block numbers as E4M3 bytes [..., hd / 16], scales [...])."""
    a = np.where(np.isfinite(x), np.abs(x), 0)
    amax = a.max(-1)
    s = np.ones_like(amax)
    for i in np.ndindex(amax.shape):
        if amax[i] > 0:
            e = -126
            while amax[i] / 2.0 ** e > 2688:
                e += 1
            s[i] = 2.0 ** e
    blocks = x.shape[:-1] + (-1, 16)
    y = (x / s[..., None]).reshape(blocks)
    bmax = (a / s[..., None]).reshape(blocks).max(-1)
    bi = np.maximum(nearest(O.E4M3[:127], bmax / 6), 1)            # (code 1 is 2^-9)
    z = np.abs(y) / O.E4M3[bi][..., None]
    nan = np.isnan(y)
    code = nearest(E2M1[:8], np.where(nan, 0, np.minimum(z, 6)))
    code = code + 8 * np.signbit(y)
    bi = np.where(nan.any(-1), 127, bi)
    return code.reshape(x.shape).astype(np.uint8), bi.astype(np.uint8), s


def values(code, blk, s):
    return (E2M1[code].reshape(code.shape[:-1] + (-1, 16)) * O.E4M3[blk][..., None]).reshape(code.shape) * s[..., None]


def pack(code):
    return code[..., ::2] | code[..., 1::2] << 4


def unpack(byte):
    return np.stack((byte & 15, byte >> 4), -1).reshape(byte.shape[:-1] + (-1,))


def ordered(t, order, device="cuda"):
    """The tensor [n_pages, page, Hkv, ...] laid out in memory as `order` of p(age), c(ell), h(ead) says."""
    perm = ["pch".index(c) for c in order[:3]] + list(range(3, t.dim()))
    return t.permute(perm).contiguous().to(device).permute([perm.index(i) for i in range(t.dim())])


def cache(n_pages, page, Hkv, hd, seed, order="phcd", spread=0.5):
    """K and V caches of random rows: two of ((codes, scales, blocks), float64 values [cells, Hkv, hd])."""
    rng = np.random.default_rng(seed)
    res = []
    for _ in range(2):
        x = rng.normal(size=(n_pages, page, Hkv, hd)) * np.exp(spread * rng.normal(size=(n_pages, page, Hkv, 1)))
        x *= np.exp(rng.normal(size=(n_pages, page, Hkv, hd // 16))).repeat(16, -1)
        code, blk, s = quantise(x)
        t = [ordered(torch.from_numpy(v), order) for v in (pack(code), s.astype(np.float32), blk)]
        res.append((t, values(code, blk, s).reshape(-1, Hkv, hd)))
    return res


def kv_pages(L, k, v):
    return L.KvPages(k[0], v[0], k[1], v[1], k[2], v[2])


def extend(table, n_kv, n_new, free, page, max_tok):
    """A step's pages, one token after the other: the pages go from the stack's end to the sequences that reach a new page."""
    table, stack = np.array(table).copy(), list(free)
    cell, pos, start = [], [], [0]
    for i, (a, b) in enumerate(zip(n_kv, n_new)):
        for p in range(a, a + b):
            if p % page == 0:
                table[i, p // page] = stack.pop()
            cell.append(int(table[i, p // page]) * page + p % page)
            pos.append(p)
        start.append(start[-1] + b)
    pad = [-1] * (max_tok - len(cell))
    return table, cell + pad, pos + pad, start, [int(a + b) for a, b in zip(n_kv, n_new)], stack
