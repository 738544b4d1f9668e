"""kv_store and kv_load over a cache of 4-bit rows on the GPU against the format's definition: every row type and
head_dim, memory orders, padding, the borders of every rounding, non-finite values, cells past the cache,
capture, another stream. Every rounding is to nearest even of an exact number, so results are compared exactly."""
import numpy as np
import pytest
import torch

from tests import ops4_common as F
from tests import ops_common as O

pytestmark = pytest.mark.gpu

ROWS = [torch.float32, torch.float16, torch.bfloat16]


@pytest.fixture(scope="module")
def L():
    import transformer_decode_kv_gb300 as L
    L.lib()
    return L


def empty(n_pages, page, Hkv, hd, order="pchd"):
    full = lambda n, v, t: F.ordered(torch.full((n_pages, page, Hkv) + n, v, dtype=t), order)
    return [[full((hd // 2,), 0x5a, torch.uint8), full((), 7.0, torch.float32), full((hd // 16,), 0x33, torch.uint8)]
            for _ in range(2)]


@pytest.mark.parametrize("order", ["pchd", "phcd", "hpcd"])
@pytest.mark.parametrize("rdt", ROWS)
@pytest.mark.parametrize("hd,Hkv,page,n", [(32, 1, 1, 1), (32, 5, 3, 40), (64, 3, 17, 50), (128, 8, 16, 33), (128, 2, 64, 1)])
def test_store_and_load(L, rdt, order, hd, Hkv, page, n):
    rng = np.random.default_rng(hd + Hkv + n)
    n_pages = n // page + 3
    k, v = empty(n_pages, page, Hkv, hd, order)
    pages = F.kv_pages(L, k, v)
    x = [torch.from_numpy(rng.normal(size=(n, Hkv, hd)) * np.exp(3 * rng.normal(size=(n, Hkv, hd // 16))).repeat(16, -1)).to(rdt)
         for _ in range(2)]
    x[0][0, 0] = 0                                              # a row of zeros
    x[1][0, 0, 16:] = 0                                         # blocks of zeros
    cell = rng.permutation(n_pages * page)[:n].astype(np.int32)
    if n > 3:
        cell[2] = -1
    dcell = torch.from_numpy(cell).cuda()
    L.kv_store(pages, x[0].cuda(), x[1].cuda(), dcell)
    out = [torch.full((n, Hkv, hd), 5.0, dtype=rdt, device="cuda") for _ in range(2)]
    L.kv_load(pages, dcell, *out)
    torch.cuda.synchronize()
    live = cell >= 0
    there = np.zeros(n_pages * page, bool)
    there[cell[live]] = True
    for xi, (c, s, b), o in zip(x, (k, v), out):
        code, blk, scale = F.quantise(xi.double().numpy())
        c, s, b = (t.cpu().reshape((n_pages * page,) + t.shape[2:]).numpy() for t in (c, s, b))
        assert np.array_equal(s[cell[live]], scale[live].astype(np.float32))
        assert np.array_equal(b[cell[live]], blk[live])
        assert np.array_equal(c[cell[live]], F.pack(code)[live])
        assert (c[~there] == 0x5a).all() and (s[~there] == 7.0).all() and (b[~there] == 0x33).all()
        back = torch.from_numpy(F.values(code, blk, scale)).to(rdt)
        assert torch.equal(o.cpu()[torch.from_numpy(live)], back[torch.from_numpy(live)])
        assert (o.cpu()[torch.from_numpy(~live)] == 5.0).all()  # padding rows are left as they were


def round_trip(L, rows):
    n, hd = rows.shape
    k, v = empty(1, n, 1, hd)
    pages = F.kv_pages(L, k, v)
    x = torch.from_numpy(rows).float().view(n, 1, hd).cuda()
    cell = torch.arange(n, dtype=torch.int32, device="cuda")
    L.kv_store(pages, x, x, cell)
    o = torch.empty_like(x)
    L.kv_load(pages, cell, o, torch.empty_like(x))
    return [t.cpu().numpy()[0, :, 0] for t in k] + [o.cpu().numpy()[:, 0]]


def test_borders_of_the_codes(L):
    """Every midpoint between codes, and the float32 numbers next to it, under block numbers of every significand."""
    rows = []
    for b in range(1, 127):                                     # block numbers: the first value of a block sets them
        bv = O.E4M3[b]
        for mid in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0):
            at = np.float32(mid * bv)
            lo, hi = np.nextafter(at, np.float32(0)), np.nextafter(at, np.float32(1e9))
            block = np.zeros(16, np.float32)
            block[:8] = [6 * bv, at, lo, hi, -at, -lo, -hi, 6 * bv]
            top = np.zeros(16, np.float32)
            top[0] = 2688                                       # the row's scale is 1
            rows.append(np.concatenate([top, block]))
    rows = np.stack(rows).astype(np.float64)
    code, blk, s = F.quantise(rows)
    assert (s == 1).all() and len(set(blk[:, 1])) == 126
    c, sc, b, o = round_trip(L, rows)
    assert np.array_equal(sc, s) and np.array_equal(b, blk)
    assert np.array_equal(c, F.pack(code))
    assert np.array_equal(o, F.values(code, blk, s).astype(np.float32))


def test_borders_of_the_block_numbers(L):
    """A block's largest value at 6 times every midpoint between E4M3 numbers, and next to it."""
    rows = []
    for i in range(0, 126):
        at = np.float32(6 * (O.E4M3[i] + O.E4M3[i + 1]) / 2)
        for x in (at, np.nextafter(at, np.float32(0)), np.nextafter(at, np.float32(1e9))):
            row = np.zeros(64, np.float32)
            row[0], row[17], row[18], row[40] = 2688, -x, x / 3, x
            rows.append(row)
    rows = np.stack(rows).astype(np.float64)
    code, blk, s = F.quantise(rows)
    c, sc, b, o = round_trip(L, rows)
    assert np.array_equal(sc, s) and np.array_equal(b, blk) and np.array_equal(c, F.pack(code))


def test_scales_and_values_at_the_edges(L):
    """The scale's step at 2688 * 2^e, tiny, huge and non-finite values."""
    rows = np.zeros((14, 32))
    rows[0, :4] = [2688, 1, -2688, 0.001]                       # s = 1
    rows[1, :4] = [2688.001, 17, 18, 19]                        # just above: s = 2
    rows[2, :3] = [np.inf, 2.0, -np.inf]                        # infinities saturate
    rows[3, :3] = [np.nan, 3.0, -1.0]                           # a block of NaN, the other not
    rows[3, 16:20] = [4, -3, 2, 1]
    rows[4, :] = np.inf                                         # nothing finite: s = 1
    rows[5, :2] = [3e38, -1e30]
    rows[6, :2] = [1e-38, 3e-39]
    rows[7, :2] = [1e-45, 0]                                    # below every scale
    rows[8, :4] = [1344.0, 1345.0, -0.0, 0.0]
    rows[9, :] = -np.linspace(0, 2688, 32)
    rows[10, 0], rows[10, 16:] = 2688, 2.0 ** -11 * np.arange(16)   # the least block number
    rows[11, :] = np.nan
    rows[12, 0] = 2.0 ** -126 * 2688
    rows[13, 0] = 2.0 ** -127 * 2688
    rows = rows.astype(np.float32).astype(np.float64)
    code, blk, s = F.quantise(rows)
    c, sc, b, o = round_trip(L, rows)
    assert np.array_equal(sc, s.astype(np.float32)) and np.array_equal(b, blk)
    nan = np.isnan(F.values(code, blk, s))
    got = F.unpack(c)
    assert np.array_equal(got[~nan], code[~nan])
    want = F.values(code, blk, s).astype(np.float32)
    assert np.array_equal(o[~nan], want[~nan]) and np.isnan(o[nan]).all() and nan[3, :16].all() and not nan[3, 16:].any()


def test_half_precision_rows_read_back_rounded_once(L):
    """An f16 or bf16 read back is the value rounded once (f16: over its range too)."""
    rng = np.random.default_rng(5)
    x = rng.normal(size=(64, 2, 128)) * np.exp(6 * rng.normal(size=(64, 2, 1)))
    code, blk, s = F.quantise(x.astype(np.float32).astype(np.float64))
    k, v = empty(4, 16, 2, 128)
    pages = F.kv_pages(L, k, v)
    cell = torch.arange(64, dtype=torch.int32, device="cuda")
    t = torch.from_numpy(x).float().cuda()
    L.kv_store(pages, t, t, cell)
    for dt in (torch.float16, torch.bfloat16):
        o = torch.zeros(64, 2, 128, dtype=dt, device="cuda")
        L.kv_load(pages, cell, o, torch.zeros_like(o))
        assert torch.equal(o.cpu(), torch.from_numpy(F.values(code, blk, s)).float().to(dt))


def test_cells_past_the_cache_are_reported_and_skipped(L):
    k, v = empty(2, 16, 2, 64)
    pages = F.kv_pages(L, k, v)
    x = torch.randn(4, 2, 64, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    L.kv_store(pages, x, x, torch.tensor([32, 5, 2 ** 31 - 1, -7], dtype=torch.int32, device="cuda"), err=err)
    assert int(err) == 1
    assert (k[1].cpu().reshape(32, 2)[5] != 7.0).all() and int((k[1].cpu() != 7.0).sum()) == 2
    out = torch.full((4, 2, 64), 3.0, device="cuda")
    err.zero_()
    L.kv_load(pages, torch.tensor([32, 5, -1, 5], dtype=torch.int32, device="cuda"), out, out.clone(), err=err)
    assert int(err) == 1 and (out[0] == 3.0).all() and (out[2] == 3.0).all() and torch.equal(out[1], out[3])


def test_capture_and_other_streams(L):
    k, v = empty(4, 16, 2, 128, "hpcd")
    pages = F.kv_pages(L, k, v)
    x = torch.randn(20, 2, 128, device="cuda", dtype=torch.bfloat16)
    cell = torch.arange(20, dtype=torch.int32, device="cuda")
    o = [torch.zeros_like(x) for _ in range(2)]
    L.kv_store(pages, x, x, cell)                               # (the first launch, not captured)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        L.kv_store(pages, x, x, cell)
        L.kv_load(pages, cell, *o)
    for seed in range(2):
        x.copy_(torch.randn(20, 2, 128, generator=torch.Generator().manual_seed(seed)))
        g.replay()
        torch.cuda.synchronize()
        code, blk, s = F.quantise(x.double().cpu().numpy())
        want = torch.from_numpy(F.values(code, blk, s)).to(torch.bfloat16)
        assert torch.equal(o[0].cpu(), want) and torch.equal(o[1].cpu(), want)
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        L.kv_load(pages, cell, *o)
    st.synchronize()
    assert torch.equal(o[0].cpu(), want)


@pytest.mark.parametrize("rdt", ROWS)
def test_rows_below_the_normal_range_are_read_back_rounded_once(L, rdt):
    """Every code times every block number times the least scales: float32 holds the product, whatever its size, and the row's type
    rounds it once."""
    n_pages, page, hd = 4, 32, 128
    k, v = empty(n_pages, page, 1, hd)
    pages = F.kv_pages(L, k, v)
    code = np.broadcast_to(np.arange(hd) % 16, (n_pages, page, 1, hd)).astype(np.uint8)
    blk = np.arange(n_pages * page * 8).reshape(n_pages, page, 1, 8) % 127      # (every number from 0 to 448)
    s = 2.0 ** (-126 + 5 * np.arange(n_pages))[:, None, None] * np.ones((n_pages, page, 1))
    for x in (k, v):
        for t, a in zip(x, (F.pack(code), s.astype(np.float32), blk.astype(np.uint8))):
            t.copy_(torch.from_numpy(a.copy()))
    cell = torch.arange(n_pages * page, dtype=torch.int32, device="cuda")
    o = [torch.full((n_pages * page, 1, hd), 5.0, dtype=rdt, device="cuda") for _ in range(2)]
    L.kv_load(pages, cell, *o)
    want = F.values(code, blk, s).reshape(-1, 1, hd)
    assert np.array_equal(want.astype(np.float32), want) and (np.abs(want[want != 0]) < 2.0 ** -126).any()
    for x in o:
        assert torch.equal(x.cpu(), torch.from_numpy(want).float().to(rdt))
