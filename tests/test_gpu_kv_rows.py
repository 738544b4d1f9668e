"""kv_store and kv_load on the GPU against the formats' definitions: every cache type from every row type,
odd counts, padding, other memory orders, non-finite values, cells past the cache, capture into a
graph, another stream. Casts are roundings to nearest even, so results are compared exactly."""
import numpy as np
import pytest
import torch

from tests import ops_common as O

pytestmark = pytest.mark.gpu

ROWS = [torch.float32, torch.float16, torch.bfloat16]
CACHES = [torch.float16, torch.bfloat16, torch.uint8]


@pytest.fixture(scope="module")
def L():
    import transformer_decode_kv_gb300 as L
    L.lib()
    return L


def empty_cache(n_pages, page, Hkv, hd, dtype, order="pchd"):
    perm = ["pch".index(c) for c in order[:-1]] + [3]
    inv = [perm.index(i) for i in range(4)]
    shape = [(n_pages, page, Hkv, hd)[i] for i in perm]
    fill = (lambda: torch.full(shape, 0x7f, dtype=dtype, device="cuda")) if dtype == torch.uint8 else \
        (lambda: torch.full(shape, float("nan"), dtype=dtype, device="cuda"))
    t = [fill().permute(inv) for _ in range(2)]
    s = [None, None]
    if dtype == torch.uint8:
        s = [torch.full([shape[i] for i in range(3)], 7.0, device="cuda").permute(inv[:3]) for _ in range(2)]
    return t, s


def want_rows(x, cdt):
    """What the cache holds for float rows x (float64), as codes and scales or values."""
    if cdt == torch.uint8:
        return O.quantise(x)
    return torch.from_numpy(x).float().to(cdt), None


@pytest.mark.parametrize("order", ["pchd", "phcd", "hpcd"])
@pytest.mark.parametrize("cdt", CACHES)
@pytest.mark.parametrize("rdt", ROWS)
@pytest.mark.parametrize("hd,Hkv,page,n", [(32, 1, 1, 1), (64, 3, 17, 50), (128, 8, 16, 33), (128, 2, 64, 1)])
def test_store_and_load(L, rdt, cdt, order, hd, Hkv, page, n):
    rng = np.random.default_rng(hd + Hkv + n)
    n_pages = n // page + 3
    (kc, vc), (ks, vs) = empty_cache(n_pages, page, Hkv, hd, cdt, order)
    pages = L.KvPages(kc, vc, ks, vs)
    x = [torch.from_numpy(rng.normal(size=(n, Hkv, hd)) * np.exp(3 * rng.normal(size=(n, Hkv, 1)))).to(rdt) for _ in range(2)]
    x[0][0, 0] = 0                                              # a row of zeros
    cell = rng.permutation(n_pages * page)[:n].astype(np.int32)
    if n > 3:
        cell[2] = -1
    dcell = torch.from_numpy(cell).cuda()
    L.kv_store(pages, x[0].cuda(), x[1].cuda(), dcell)
    out = [torch.full((n, Hkv, hd), 5.0, dtype=rdt, device="cuda") for _ in range(2)]
    L.kv_load(pages, dcell, *out)
    torch.cuda.synchronize()
    for xi, c, s, o in zip(x, (kc, vc), (ks, vs), out):
        flat = c.cpu().reshape(n_pages * page, Hkv, hd)
        code, scale = want_rows(xi.double().numpy(), cdt)
        live = cell >= 0
        if cdt == torch.uint8:
            assert np.array_equal(flat.numpy()[cell[live]], code[live])
            sc = s.cpu().reshape(-1, Hkv).numpy()
            assert np.array_equal(sc[cell[live]], scale[live].astype(np.float32))
            back = torch.from_numpy(O.E4M3[code] * scale[..., None]).to(rdt)
            untouched = np.ones(n_pages * page, bool); untouched[cell[live]] = False
            assert (sc[untouched] == 7.0).all() and (flat.numpy()[untouched] == 0x7f).all()
        else:
            assert torch.equal(flat[cell[live].astype(np.int64)], code[torch.from_numpy(live)])
            back = code.to(torch.float32).to(rdt)
        got = o.cpu()
        assert torch.equal(got[torch.from_numpy(live)], back[torch.from_numpy(live)])
        assert (got[torch.from_numpy(~live)] == 5.0).all()      # padding rows are left as they were


def test_values_at_the_edges_of_e4m3(L):
    """Ties, the scale's step at 448 * 2^e, subnormal codes, tiny, huge and non-finite values."""
    rows = np.zeros((12, 1, 32))
    rows[0, 0, :4] = [448, 1, -448, 0.001]                      # s = 1
    rows[1, 0, :4] = [448.00003, 17, 18, 19]                    # just above: s = 2
    rows[2, 0, :8] = [256, 17, 19, 21, 23, 25, 27, -17]         # ties between codes
    rows[3, 0, :4] = [256, 2.0 ** -10, 3 * 2.0 ** -10, 2.0 ** -11]   # halves of the least code
    rows[4, 0, :3] = [np.inf, 2.0, -np.inf]                     # infinities saturate
    rows[5, 0, :3] = [np.nan, 3.0, -1.0]
    rows[6, 0, :] = np.inf                                      # nothing finite: s = 1
    rows[7, 0, :2] = [3e38, -1e30]
    rows[8, 0, :2] = [1e-38, 3e-39]
    rows[9, 0, :2] = [1e-45, 0]                                 # below every scale
    rows[10, 0, :4] = [224.0, 225.0, -0.0, 0.0]
    rows[11, 0, :] = -np.linspace(0, 448, 32)
    rows = rows.astype(np.float32).astype(np.float64)
    (kc, vc), (ks, vs) = empty_cache(1, 16, 1, 32, torch.uint8)
    x = torch.from_numpy(rows).float().cuda()
    cell = torch.arange(12, dtype=torch.int32, device="cuda")
    L.kv_store(L.KvPages(kc, vc, ks, vs), x, x, cell)
    code, s = O.quantise(rows)
    got, sc = kc.cpu().numpy()[0, :12], ks.cpu().numpy()[0, :12]
    assert np.array_equal(sc, s.astype(np.float32))
    nan = np.isnan(rows)
    assert np.array_equal(got[~nan], code[~nan])
    assert ((got[nan] & 127) == 127).all()
    o = torch.empty_like(x)
    L.kv_load(L.KvPages(kc, vc, ks, vs), cell, o, torch.empty_like(x))
    want = (O.E4M3[code] * s[..., None]).astype(np.float32)
    assert np.array_equal(o.cpu().numpy()[~nan], want[~nan]) and np.isnan(o.cpu().numpy()[nan]).all()


def test_cells_past_the_cache_are_skipped_and_reported(L):
    (kc, vc), (ks, vs) = empty_cache(2, 4, 2, 64, torch.float16)
    pages = L.KvPages(kc, vc, ks, vs)
    x = torch.ones(4, 2, 64, dtype=torch.float16, device="cuda")
    cell = torch.tensor([0, 8, 2 ** 31 - 1, -5], dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    L.kv_store(pages, x, x, cell, err=err)
    assert err.item() == 1
    flat = kc.reshape(8, 2, 64)
    assert (flat[0] == 1).all() and torch.isnan(flat[1:]).all()
    o = [torch.full_like(x, 9) for _ in range(2)]
    err.zero_()
    L.kv_load(pages, cell, *o, err=err)
    assert err.item() == 1
    assert (o[0][0] == 1).all() and (o[0][1:] == 9).all()
    err.zero_()
    L.kv_store(pages, x[:1], x[:1], cell[:1], err=err)
    assert err.item() == 0


def test_strided_and_repeated_rows(L):
    rng = np.random.default_rng(5)
    fused = torch.from_numpy(rng.normal(size=(9, 12, 64))).to(torch.bfloat16).cuda()   # 8 q heads, k, v
    k, v = fused[:, 8:10], fused[:, 10:12]
    (kc, vc), (ks, vs) = empty_cache(3, 4, 2, 64, torch.bfloat16)
    pages = L.KvPages(kc, vc, ks, vs)
    cell = torch.arange(9, dtype=torch.int32, device="cuda")
    L.kv_store(pages, k, v, cell)
    assert torch.equal(kc.reshape(12, 2, 64)[:9], k) and torch.equal(vc.reshape(12, 2, 64)[:9], v)
    # one row for every token, and cells named twice by a load
    L.kv_store(pages, k[:1].expand(9, 2, 64), v[:1].expand(9, 2, 64), cell)
    assert torch.equal(kc.reshape(12, 2, 64)[:9], k[:1].expand(9, 2, 64))
    o = [torch.zeros(6, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    L.kv_load(pages, torch.tensor([3, 3, 0, 8, 8, 3], dtype=torch.int32, device="cuda"), *o)
    assert torch.equal(o[1], v[:1].expand(6, 2, 64))


def test_byte_offsets_past_32_bits(L):
    """Cells whose rows start above 4 GB in the cache."""
    n_pages, page, Hkv, hd = 1 << 17, 16, 8, 128                # 2^21 cells, 4.3 GB each of K and V
    kc = torch.zeros(n_pages, page, Hkv, hd, dtype=torch.float16, device="cuda")
    vc = torch.zeros_like(kc)
    n = 5
    x = torch.randn(n, Hkv, hd, device="cuda", dtype=torch.float16)
    cell = torch.tensor([0, n_pages * page - 1, n_pages * page - 17, 1 << 20, (1 << 20) + 1], dtype=torch.int32, device="cuda")
    pages = L.KvPages(kc, vc)
    L.kv_store(pages, x, -x, cell)
    assert torch.equal(kc.view(-1, Hkv, hd)[cell.long()], x)
    assert int((kc != 0).sum(dtype=torch.int64)) == int((x != 0).sum())
    o = [torch.empty_like(x) for _ in range(2)]
    L.kv_load(pages, cell, *o)
    assert torch.equal(o[0], x) and torch.equal(o[1], -x)


def test_graph_and_stream(L):
    (kc, vc), (ks, vs) = empty_cache(4, 16, 2, 128, torch.uint8)
    pages = L.KvPages(kc, vc, ks, vs)
    x = torch.randn(20, 2, 128, device="cuda")
    cell = torch.arange(20, dtype=torch.int32, device="cuda")
    o = [torch.zeros_like(x) for _ in range(2)]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        L.kv_store(pages, x, x, cell)
        L.kv_load(pages, cell, *o)
    for i in range(2):
        x.normal_()
        cell.copy_((torch.arange(20) * 3 + i).int())
        g.replay()
        torch.cuda.synchronize()
        code, s = O.quantise(x.double().cpu().numpy())
        assert np.array_equal(o[0].cpu().numpy(), (O.E4M3[code] * s[..., None]).astype(np.float32))
    # torch's current stream is the one used
    y = torch.zeros_like(x)
    with torch.cuda.stream(st):
        torch.cuda._sleep(20_000_000)
        y.copy_(x)
        L.kv_store(pages, y, y, cell)
        L.kv_load(pages, cell, *o)
    st.synchronize()
    assert np.array_equal(o[1].cpu().numpy(), (O.E4M3[code] * s[..., None]).astype(np.float32))


def test_host_memory_and_wrong_shapes_are_refused(L):
    (kc, vc), (ks, vs) = empty_cache(2, 4, 2, 64, torch.float16)
    pages = L.KvPages(kc, vc)
    x = torch.zeros(3, 2, 64, dtype=torch.float16)
    cell = torch.zeros(3, dtype=torch.int32, device="cuda")
    with pytest.raises(L.LlmError, match="device memory"):
        L.kv_store(pages, x, x, cell)
    with pytest.raises(L.LlmError, match="device memory"):
        L.kv_store(pages, x.cuda(), x.cuda(), cell.cpu())
    with pytest.raises(ValueError):
        L.kv_store(pages, x.cuda(), x.cuda(), cell.long())
    with pytest.raises(ValueError):
        L.kv_store(pages, x.cuda()[:, :1], x.cuda()[:, :1], cell)
    with pytest.raises(ValueError):
        L.kv_store(pages, x.cuda(), x.cuda(), cell[:2])
    with pytest.raises(ValueError):
        L.KvPages(kc, vc, ks, torch.zeros(2, 4, 2, device="cuda"))


def test_one_row_whose_token_stride_says_nothing(L):
    kc, vc = (torch.zeros(2, 4, 2, 32, device="cuda", dtype=torch.float16) for _ in range(2))
    pages = L.KvPages(kc, vc)
    k = torch.randn(64, device="cuda", dtype=torch.float16).as_strided((1, 2, 32), (5, 32, 1))
    v = torch.randn(64, device="cuda", dtype=torch.float16).as_strided((1, 2, 32), (64, 32, 1))
    cell = torch.tensor([5], dtype=torch.int32, device="cuda")
    L.kv_store(pages, k, v, cell)
    assert torch.equal(kc[1, 1], k[0]) and torch.equal(vc[1, 1], v[0])
    ko = torch.zeros(64, device="cuda", dtype=torch.float16).as_strided((1, 2, 32), (1, 32, 1))
    vo = torch.zeros(2, 1, 32, device="cuda", dtype=torch.float16).transpose(0, 1)
    L.kv_load(pages, cell, ko, vo)
    assert torch.equal(ko, k) and torch.equal(vo, v)
