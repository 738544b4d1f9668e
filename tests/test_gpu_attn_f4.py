"""Attention of new tokens over a paged cache of 4-bit rows on the GPU against the formula in 64 bits (values as the
codes stand for them; tolerances as tests/ops_common.py derives them, where the activations' type bounds the
rounding of the weights): every activation type, head layout, page size, chunk lengths from one token on,
windows and sinks, rows that see nothing, hidden cells that hold NaN, scales far apart, graphs and streams."""
import numpy as np
import pytest
import torch

from tests import ops4_common as F
from tests import ops_common as O

pytestmark = pytest.mark.gpu

ACTS = [torch.float16, torch.bfloat16, torch.float32]


@pytest.fixture(scope="module")
def L():
    import transformer_decode_kv_gb300 as L
    L.lib()
    return L


def tables_of(n_kv, page, rng, spare=2):
    need = [-(-int(n) // page) for n in n_kv]
    n_pages = sum(need) + spare
    perm = rng.permutation(n_pages).astype(np.int32)
    t = np.full((len(n_kv), max(need + [1])), -1, np.int32)       # entries past a sequence are not read
    at = 0
    for i, m in enumerate(need):
        t[i, :m] = perm[at:at + m]
        at += m
    return t, n_pages


def poison(c, tables, n_kv, page, n_pages):
    """NaN scales and block numbers in every cell no sequence uses."""
    used = set()
    for t, n in zip(tables, n_kv):
        used |= {int(t[j // page]) * page + j % page for j in range(int(n))}
    free = [x for x in range(n_pages * page) if x not in used]
    p, a = [x // page for x in free], [x % page for x in free]
    c[0][p, a] = 0x77
    c[1][p, a] = float("nan")
    c[2][p, a] = 0x7f


def check(L, act, hd, Hkv, G, page, n_new, n_kv, window=0, n_sink=0, seed=0, order="phcd", scale=0.0, mutate=None,
          spread=0.5, extra=3, q=None):
    rng = np.random.default_rng(seed)
    tables, n_pages = tables_of(n_kv, page, rng)
    (k, kval), (v, vval) = F.cache(n_pages, page, Hkv, hd, seed + 1, order, spread)
    for c in (k, v):
        poison(c, tables, n_kv, page, n_pages)
    if mutate:
        mutate(k, v, kval, vval, tables)
    T = int(sum(n_new))
    if q is None:
        q = torch.from_numpy(rng.normal(size=(T + extra, Hkv * G, hd))).to(act).cuda()
    out = torch.full_like(q, 77.0)
    pages = F.kv_pages(L, k, v)
    plan = L.AttnPlan(pages, n_head=Hkv * G, dtype=act, max_tok=max(T, 1), max_seq=max(1, len(n_new)),
                      max_table=max(1, tables.size), window=window, n_sink=n_sink, scale=scale)
    plan.set(n_new, n_kv, tables)
    plan.run(q, pages, out)
    assert plan.error() == 0
    got = out.double().cpu().numpy()
    ref, mag, smag = O.attention(q.double().cpu().numpy()[:T], kval, vval, tables, n_new, n_kv, page, window, n_sink,
                                 None if scale == 0 else scale)
    tol = O.attention_tol(ref, mag, smag, act, max(list(n_kv) + [1]), hd, np.abs(vval[np.isfinite(vval)]).max())
    bad = ~(np.abs(got[:T] - ref) <= tol)
    if np.isnan(ref).any():
        bad &= ~(np.isnan(ref) & ~np.isfinite(got[:T]))
    if act == torch.float16:                                      # (65520 and more, half a step past 65504, round to infinity)
        bad &= ~(((ref + tol >= 65520) & (got[:T] == np.inf)) | ((ref - tol <= -65520) & (got[:T] == -np.inf)))
    worst = np.nanmax(np.where(np.isinf(got[:T]), 0, np.abs(got[:T] - ref) / tol), initial=0)
    print(f"form {plan.form} worst error {worst:.3f} of the tolerance")
    assert not bad.any(), (np.argwhere(bad)[:5], got[:T][bad][:5], ref[bad][:5], tol[bad][:5])
    assert (got[T:] == 77.0).all()                                # rows behind the last sequence
    return plan


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("hd", [32, 64, 128])
@pytest.mark.parametrize("n_new,n_kv", [([1], [1]), ([1], [16]), ([1, 1, 1], [17, 64, 301]), ([5, 1, 33], [5, 200, 90]),
                                        ([1] * 9, [31, 32, 33, 191, 192, 193, 400, 1, 2])])
def test_types_and_head_dims(L, act, hd, n_new, n_kv):
    check(L, act, hd, 2, 4, 16, n_new, n_kv, seed=hd)


@pytest.mark.parametrize("Hkv,G", [(1, 1), (1, 32), (8, 1), (2, 3), (3, 7), (2, 16), (1, 20)])
@pytest.mark.parametrize("act,hd", [(torch.float16, 64), (torch.bfloat16, 128), (torch.float32, 32)])
def test_head_layouts(L, act, hd, Hkv, G):
    check(L, act, hd, Hkv, G, 16, [1, 6, 0, 2], [40, 6, 9, 131], seed=G)


@pytest.mark.parametrize("page", [1, 3, 8, 16, 17, 100, 256])
@pytest.mark.parametrize("order", ["pchd", "phcd", "hpcd"])
def test_pages_and_memory_orders(L, page, order):
    check(L, torch.float16, 128, 2, 4, page, [1, 40], [257, 100], order=order, seed=page)
    check(L, torch.bfloat16, 64, 2, 4, page, [1, 9], [257, 100], order=order, seed=page)


@pytest.mark.parametrize("window,n_sink", [(1, 0), (1, 1), (7, 4), (64, 4), (64, 0), (300, 16), (10000, 4), (2 ** 31 - 1, 0),
                                           (50, 2 ** 31 - 1)])
@pytest.mark.parametrize("act", ACTS)
def test_windows_and_sinks(L, act, window, n_sink):
    check(L, act, 64, 2, 4, 16, [1, 70, 3, 1], [500, 80, 3, 66], window, n_sink, seed=7)


@pytest.mark.parametrize("act", ACTS)
def test_rows_that_see_nothing(L, act):
    """No cached rows at all, and more new tokens than rows (negative positions): zeros."""
    check(L, act, 64, 2, 4, 16, [3, 1, 50, 0], [0, 5, 20, 7], seed=3)
    check(L, act, 128, 1, 4, 16, [2], [0], seed=4)
    check(L, act, 32, 2, 4, 16, [], [], seed=5)
    check(L, act, 64, 2, 4, 16, [0, 0], [0, 9], seed=6)
    check(L, act, 64, 2, 4, 16, [40], [25], window=3, n_sink=2, seed=8)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("hd", [32, 128])
def test_long_key_ranges_are_split_and_merged(L, act, hd):
    check(L, act, hd, 1, 4, 16, [1, 2], [9000, 3001], seed=11, spread=0.2)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("hd", [32, 64, 128])
@pytest.mark.parametrize("n_new,n_kv,window,n_sink", [([130], [130], 0, 0), ([200, 1, 64], [700, 900, 64], 0, 0),
                                                      ([150, 33], [500, 300], 100, 5), ([129], [1000], 1, 1),
                                                      ([96], [40], 0, 0)])
def test_chunks(L, act, hd, n_new, n_kv, window, n_sink):
    check(L, act, hd, 2, 4, 16, n_new, n_kv, window, n_sink, seed=hd + 1)


@pytest.mark.parametrize("n_new,n_kv", [([1, 2], [300, 90]), ([200], [300])])
@pytest.mark.parametrize("hd", [32, 128])
def test_rows_of_very_different_scales(L, n_new, n_kv, hd):
    """Row scales from 2^-60 to 2^40, block numbers over their whole range, rows and blocks of zeros."""
    def mutate(k, v, kval, vval, tables):
        rng = np.random.default_rng(1)
        for c, val, top in ((k, kval, -6), (v, vval, 40)):
            n_pages, page, Hkv = c[1].shape
            e = rng.integers(-60, top, (n_pages, page, Hkv))
            s = np.where(rng.random(e.shape) < 0.2, 2.0 ** e, 1.0)
            blk = rng.integers(1, 127, tuple(c[2].shape))
            code = F.unpack(c[0].cpu().numpy())
            code[rng.random(code.shape[:3]) < 0.1] = 0
            code.reshape(blk.shape + (16,))[rng.random(blk.shape) < 0.1] = 0
            if val is kval:
                s /= 2688                                       # scores of ordinary size
                s = 2.0 ** np.round(np.log2(s))
            c[0].copy_(torch.from_numpy(F.pack(code)))
            c[1].copy_(torch.from_numpy(s.astype(np.float32)))
            c[2].copy_(torch.from_numpy(blk.astype(np.uint8)))
            val[:] = F.values(code, blk, s).reshape(val.shape)
    for act in ACTS:
        check(L, act, hd, 2, 4, 16, n_new, n_kv, seed=21, mutate=mutate)


@pytest.mark.parametrize("where", ["scale", "block"])
@pytest.mark.parametrize("n_new", [[1, 1], [3, 90]])
def test_a_visible_nan_reaches_the_rows_that_see_it(L, n_new, where):
    def mutate(k, v, kval, vval, tables):
        p, a = int(tables[1][40 // 16]), 40 % 16                # key 40 of the second sequence
        for c, val in ((k, kval), (v, vval)):
            if where == "scale":
                c[1][p, a, 1] = float("nan")
                val[p * 16 + a, 1] = np.nan
            else:
                c[2][p, a, 1, 2] = 0x7f
                val[p * 16 + a, 1, 32:48] = np.nan
    check(L, torch.float16, 64, 2, 4, 16, n_new, [50, 100], seed=31, mutate=mutate)
    check(L, torch.bfloat16, 128, 2, 4, 16, n_new, [50, 100], seed=32, mutate=mutate)


def test_scales_are_applied_as_given(L):
    """Negative and zero attention scales."""
    for scale in (-0.3, 0.02):
        check(L, torch.float16, 64, 2, 4, 16, [1, 90], [100, 200], scale=scale, seed=41)


def test_strided_rows_other_streams_and_graphs(L):
    rng = np.random.default_rng(3)
    n_new, n_kv, page, Hkv, G, hd = [1, 1, 1], [300, 40, 7], 16, 2, 4, 128
    tables, n_pages = tables_of(n_kv, page, rng)
    (k, kval), (v, vval) = F.cache(n_pages, page, Hkv, hd, 9)
    pages = F.kv_pages(L, k, v)
    big = torch.randn(3, Hkv * G, 3 * hd, device="cuda").half()
    q = big[..., hd:2 * hd]
    out = torch.zeros(3, Hkv * G, 2 * hd, device="cuda").half()[..., :hd]
    plan = L.AttnPlan(pages, n_head=Hkv * G, dtype=torch.float16, max_tok=3, max_seq=3, max_table=tables.size)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        plan.set(n_new, n_kv, tables)
        plan.run(q, pages, out)
    st.synchronize()
    ref, mag, smag = O.attention(q.double().cpu().numpy(), kval, vval, tables, n_new, n_kv, page)
    tol = O.attention_tol(ref, mag, smag, torch.float16, 300, hd, np.abs(vval).max())
    assert (np.abs(out.double().cpu().numpy() - ref) <= tol).all()
    first = out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        plan.run(q, pages, out)
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first)                              # the same bits, launch after launch
    plan.set([1, 1, 0], [299, 40, 0], tables)                   # the graph follows the plan
    g.replay()
    torch.cuda.synchronize()
    ref, mag, smag = O.attention(q.double().cpu().numpy()[:2], kval, vval, tables, [1, 1, 0], [299, 40, 0], page)
    tol = O.attention_tol(ref, mag, smag, torch.float16, 300, hd, np.abs(vval).max())
    assert (np.abs(out.double().cpu().numpy()[:2] - ref) <= tol).all()
    assert torch.equal(out[2], first[2]) and plan.error() == 0


def test_a_page_outside_the_cache_is_refused(L):
    (k, _), (v, _) = F.cache(4, 16, 1, 64, 1)
    pages = F.kv_pages(L, k, v)
    plan = L.AttnPlan(pages, n_head=4, dtype=torch.float16, max_tok=4, max_seq=2, max_table=8)
    with pytest.raises(L.LlmError, match="page"):
        plan.set([1], [20], [[0, 4]])


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("page", [16, 17, 64])
@pytest.mark.parametrize("n_sink", [0, 5, 70])
def test_what_the_window_has_left_behind_may_hold_anything(L, act, page, n_sink):
    """NaN scales, block numbers and codes in cells that no row of the step sees any more, in the same pages and blocks of keys as
    cells that rows see."""
    n_new, n_kv, window = [150, 1, 9], [500, 300, 200], 100

    def mutate(k, v, kval, vval, tables):
        for t, m, n in zip(tables, n_new, n_kv):
            j = np.arange(n_sink, max(n_sink, n - m - window + 1))
            p, a = torch.from_numpy(t[j // page].astype(np.int64)), torch.from_numpy(j % page)
            for c in (k, v):
                c[0][p, a] = 0x77
                c[1][p, a] = float("nan")
                c[2][p, a] = 0x7f
    check(L, act, 64, 2, 4, page, n_new, n_kv, window, n_sink, seed=51, mutate=mutate)
    check(L, act, 128, 1, 4, page, n_new, n_kv, window, n_sink, seed=52, mutate=mutate)
