"""Attention of new tokens over a paged cache on the GPU against the formula in 64 bits
(tests/ops_common.py, which also derives the tolerances): every type pair, head layout, page size,
chunk lengths from one token on, windows and sinks, rows that see nothing, cells that hold NaN where no row
may look, strides, streams, graphs, and the whole step write -> attend -> sample."""
import numpy as np
import pytest
import torch

from tests import ops_common as O

pytestmark = pytest.mark.gpu

PAIRS = [(torch.float16, torch.float16), (torch.bfloat16, torch.bfloat16), (torch.float32, torch.float16),
         (torch.float16, torch.uint8), (torch.bfloat16, torch.uint8), (torch.float32, torch.uint8)]


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
    return t, n_pages, perm[at:]


def poison(c, s, tables, n_kv, page, spare):
    """NaN (code 0x7f and a NaN scale) in every cell no sequence uses."""
    used = set()
    for t, n in zip(tables, n_kv):
        used |= {int(t[j // page]) * page + j % page for j in range(int(n))}
    free = [x for x in range(c.shape[0] * page) if x not in used]
    p, a = [x // page for x in free], [x % page for x in free]
    if c.dtype == torch.uint8:
        c[p, a] = 0x7f
        s[p, a] = float("nan")
    else:
        c[p, a] = float("nan")


def check(L, act, cdt, hd, Hkv, G, page, n_new, n_kv, window=0, n_sink=0, seed=0, order="pchd", scale=0.0, q=None,
          mutate=None, spread=0.5, extra=3):
    rng = np.random.default_rng(seed)
    tables, n_pages, spare = tables_of(n_kv, page, rng)
    (k, ks, kv_), (v, vs, vv) = O.cache(n_pages, page, Hkv, hd, cdt, seed + 1, order, spread)
    for c, s in ((k, ks), (v, vs)):
        poison(c, s, tables, n_kv, page, spare)
    if mutate:
        mutate(k, v, kv_, vv, tables)
    T = int(sum(n_new))
    if q is None:
        q = torch.from_numpy(rng.normal(size=(T + extra, Hkv * G, hd))).to(act).cuda()
    out = torch.full_like(q, 77.0)
    pages = L.KvPages(k, v, ks, vs)
    plan = L.AttnPlan(pages, n_head=Hkv * G, dtype=act, max_tok=max(T, 1), max_seq=max(1, len(n_new)),
                      max_table=max(1, tables.size), window=window, n_sink=n_sink, scale=scale)
    plan.set(n_new, n_kv, tables)
    plan.run(q, pages, out)
    assert plan.error() == 0
    got = out.double().cpu().numpy()
    ref, mag, smag = O.attention(q.double().cpu().numpy()[:T], kv_, vv, tables, n_new, n_kv, page, window, n_sink,
                                 None if scale == 0 else scale)
    tol = O.attention_tol(ref, mag, smag, act, max(list(n_kv) + [1]), hd,
                          np.abs(vv[np.isfinite(vv)]).max())
    bad = ~(np.abs(got[:T] - ref) <= tol)
    if np.isnan(ref).any():
        bad &= ~(np.isnan(ref) & ~np.isfinite(got[:T]))
    worst = np.nanmax(np.abs(got[:T] - ref) / tol, initial=0)
    print(f"form {plan.form} worst error {worst:.3f} of the tolerance")
    assert not bad.any(), (np.argwhere(bad)[:5], got[:T][bad][:5], ref[bad][:5], tol[bad][:5])
    assert (got[T:] == 77.0).all()                                # rows behind the last sequence
    return plan


@pytest.mark.parametrize("act,cdt", PAIRS)
@pytest.mark.parametrize("hd", [32, 64, 128])
@pytest.mark.parametrize("n_new,n_kv", [([1], [1]), ([1], [16]), ([1, 1, 1], [17, 64, 301]), ([5, 1, 33], [5, 200, 90])])
def test_types_and_head_dims(L, act, cdt, hd, n_new, n_kv):
    check(L, act, cdt, hd, 2, 4, 16, n_new, n_kv, seed=hd)


@pytest.mark.parametrize("Hkv,G", [(1, 1), (1, 32), (8, 1), (2, 3), (3, 7), (2, 16), (1, 20)])
@pytest.mark.parametrize("act,cdt", [PAIRS[0], PAIRS[4]])
def test_head_layouts(L, act, cdt, Hkv, G):
    check(L, act, cdt, 64, Hkv, G, 16, [1, 6, 0, 2], [40, 6, 9, 131], seed=G)


@pytest.mark.parametrize("page", [1, 3, 8, 16, 17, 100, 256])
@pytest.mark.parametrize("order", ["pchd", "phcd", "hpcd"])
def test_pages_and_memory_orders(L, page, order):
    check(L, torch.float16, torch.float16, 128, 2, 4, page, [1, 40], [257, 100], order=order, seed=page)
    check(L, torch.bfloat16, torch.uint8, 128, 2, 4, page, [1, 9], [257, 100], order=order, seed=page)


@pytest.mark.parametrize("window,n_sink", [(1, 0), (1, 1), (7, 4), (64, 4), (64, 0), (300, 16), (10000, 4), (2 ** 31 - 1, 0), (50, 2 ** 31 - 1)])
@pytest.mark.parametrize("act,cdt", [PAIRS[0], PAIRS[1], PAIRS[5]])
def test_windows_and_sinks(L, act, cdt, window, n_sink):
    check(L, act, cdt, 64, 2, 4, 16, [1, 70, 3, 1], [500, 80, 3, 66], window, n_sink, seed=7)


@pytest.mark.parametrize("act,cdt", [PAIRS[0], PAIRS[2], PAIRS[4]])
def test_rows_that_see_nothing(L, act, cdt):
    """No cached rows at all, and more new tokens than rows (negative positions): zeros."""
    check(L, act, cdt, 64, 2, 4, 16, [3, 1, 50, 0], [0, 5, 20, 7], seed=3)
    check(L, act, cdt, 128, 1, 4, 16, [2], [0], seed=4)
    check(L, act, cdt, 64, 2, 4, 16, [], [], seed=5)
    check(L, act, cdt, 64, 2, 4, 16, [0, 0], [0, 9], seed=6)
    check(L, act, cdt, 64, 2, 4, 16, [40], [25], window=3, n_sink=2, seed=8)


@pytest.mark.parametrize("act,cdt", PAIRS)
def test_long_key_ranges_are_split_and_merged(L, act, cdt):
    check(L, act, cdt, 128, 1, 4, 16, [1, 2], [9000, 3001], seed=11, spread=0.2)


@pytest.mark.parametrize("act,cdt", [PAIRS[0], PAIRS[1], PAIRS[2], PAIRS[4]])
@pytest.mark.parametrize("hd", [32, 64, 128])
@pytest.mark.parametrize("n_new,n_kv,window,n_sink", [([130], [130], 0, 0), ([200, 1, 64], [700, 900, 64], 0, 0),
                                                      ([150, 33], [500, 300], 100, 5), ([129], [1000], 1, 1),
                                                      ([96], [40], 0, 0)])
def test_chunks(L, act, cdt, hd, n_new, n_kv, window, n_sink):
    check(L, act, cdt, hd, 2, 4, 16, n_new, n_kv, window, n_sink, seed=hd + 1)


@pytest.mark.parametrize("page", [1, 8, 16, 24, 64, 128, 200])
@pytest.mark.parametrize("order", ["pchd", "phcd", "hpcd"])
@pytest.mark.parametrize("hd,Hkv", [(64, 2), (128, 1)])
def test_chunks_over_runs_of_cells(L, page, order, hd, Hkv):
    """Chunks whose key blocks are whole runs of cells, partly so, and not at all."""
    check(L, torch.float16, torch.float16, hd, Hkv, 4, page, [40, 70], [40, 900], order=order, seed=page)
    check(L, torch.bfloat16, torch.bfloat16, hd, Hkv, 4, page, [150], [1300], 500, 5, order=order, seed=page + 1)


def test_chunks_over_pages_in_order(L):
    """A cache whose pages follow each other: runs go on from page to page, as in a cache of single cells."""
    for page in (1, 16):
        n = 700
        (k, _, kv_), (v, _, vv) = O.cache(-(-n // page) + 9, page, 2, 128, torch.float16, 3)
        pages = L.KvPages(k, v)
        q = torch.randn(60, 8, 128, device="cuda", dtype=torch.float16)
        out = torch.zeros_like(q)
        table = (np.arange(-(-n // page)) + 4)[None]
        plan = L.AttnPlan(pages, 8, torch.float16, 60, 1, table.size)
        plan.set([60], [n], table)
        plan.run(q, pages, out)
        ref, mag, smag = O.attention(q.double().cpu().numpy(), kv_, vv, table, [60], [n], page)
        tol = O.attention_tol(ref, mag, smag, torch.float16, n, 128, np.abs(vv).max())
        assert (np.abs(out.double().cpu().numpy() - ref) <= tol).all()


@pytest.mark.parametrize("n_new", [1, 100])
@pytest.mark.parametrize("act,cdt", [PAIRS[0], PAIRS[1], PAIRS[4]])
def test_non_finite_rows_reach_only_the_tokens_that_see_them(L, act, cdt, n_new):
    """NaN and infinities in cells some tokens of a tile see and others do not."""
    n_kv = [max(n_new, 30)]

    def mutate(k, v, kv_, vv, tables):
        for pos, val in ((n_kv[0] - 1, float("nan")), (2, float("inf")), (n_kv[0] // 2, float("nan"))):
            cell = int(tables[0][pos // 16]) * 16 + pos % 16
            for c, x in ((k, kv_), (v, vv)):
                c[cell // 16, cell % 16, 0] = 0x7f if c.dtype == torch.uint8 else val
                x[cell, 0] = np.nan if c.dtype == torch.uint8 else val

    with np.errstate(all="ignore"):
        check(L, act, cdt, 64, 2, 4, 16, [n_new], n_kv, window=5, n_sink=1, seed=21, mutate=mutate)


@pytest.mark.parametrize("n_new", [1, 3, 40])
@pytest.mark.parametrize("act,cdt", [PAIRS[0], PAIRS[1], PAIRS[4]])
def test_a_token_that_sees_only_nan_gives_nan(L, act, cdt, n_new):
    n_kv = [n_new + 20]

    def mutate(k, v, kv_, vv, tables):
        cell = int(tables[0][(n_kv[0] - 1) // 16]) * 16 + (n_kv[0] - 1) % 16
        k[cell // 16, cell % 16] = 0x7f if k.dtype == torch.uint8 else float("nan")
        kv_[cell] = np.nan

    with np.errstate(all="ignore"):
        check(L, act, cdt, 64, 2, 4, 16, [n_new], n_kv, window=1, seed=22, mutate=mutate)


@pytest.mark.parametrize("act,cdt", [PAIRS[0], PAIRS[2], PAIRS[4]])
def test_large_and_small_activations(L, act, cdt):
    """Rows of q far from 1 (their products stay finite) and a scale of its own."""
    rng = np.random.default_rng(9)
    x = rng.normal(size=(6, 8, 64))
    if act == torch.float16:
        x *= 10.0 ** rng.integers(-2, 2, size=(6, 8, 1))
    else:
        x *= 10.0 ** rng.integers(-30, 6, size=(6, 8, 1))
    q = torch.from_numpy(x).to(act).cuda()
    check(L, act, cdt, 64, 2, 4, 16, [6], [50], q=q, scale=1e-3, seed=2)
    check(L, act, cdt, 64, 2, 4, 16, [6], [50], q=q, scale=-1e-4, seed=2)


def test_e4m3_rows_of_very_different_scales(L):
    check(L, torch.float32, torch.uint8, 128, 2, 4, 16, [1, 3], [300, 40], spread=2.5, seed=31)


def test_strided_rows(L):
    rng = np.random.default_rng(1)
    (k, ks, kv_), (v, vs, vv) = O.cache(4, 16, 2, 64, torch.float16, 1)
    fused = torch.from_numpy(rng.normal(size=(5, 12, 64))).to(torch.float16).cuda()
    q = fused[:, :8]
    big = torch.full((8, 5, 64), 3.0, dtype=torch.float16, device="cuda")
    out = big.transpose(0, 1)                                     # [token, head] with the head outermost
    pages = L.KvPages(k, v)
    plan = L.AttnPlan(pages, 8, torch.float16, 5, 2, 8)
    plan.set([4, 1], [30, 3], [[2, 0], [3, -1]])
    plan.run(q, pages, out)
    ref, mag, smag = O.attention(q.double().cpu().numpy(), kv_, vv, [[2, 0], [3]], [4, 1], [30, 3], 16)
    tol = O.attention_tol(ref, mag, smag, torch.float16, 30, 64, np.abs(vv).max())
    assert (np.abs(out.double().cpu().numpy() - ref) <= tol).all()
    # one query row for every token, straight from an expanded tensor
    plan.run(q[:1].expand(5, 8, 64), pages, out)
    ref, mag, smag = O.attention(q[:1].expand(5, 8, 64).double().cpu().numpy(), kv_, vv, [[2, 0], [3]], [4, 1], [30, 3], 16)
    assert (np.abs(out.double().cpu().numpy() - ref) <= O.attention_tol(ref, mag, smag, torch.float16, 30, 64, np.abs(vv).max())).all()


def test_same_result_every_time(L):
    """Merging does not depend on which unit finishes last."""
    (k, _, _), (v, _, _) = O.cache(400, 16, 1, 128, torch.float16, 5)
    pages = L.KvPages(k, v)
    q = torch.randn(2, 4, 128, device="cuda", dtype=torch.float16)
    plan = L.AttnPlan(pages, 4, torch.float16, 2, 2, 800)
    plan.set([1, 1], [6400, 5000], np.tile(np.arange(400), (2, 1)))
    outs = []
    for _ in range(6):
        o = torch.empty_like(q)
        plan.run(q, pages, o)
        outs.append(o.cpu())
    assert all(torch.equal(outs[0], o) for o in outs)


def test_graph_replays_the_plan_as_last_set(L):
    (k, _, kv_), (v, _, vv) = O.cache(64, 16, 2, 64, torch.bfloat16, 5)
    pages = L.KvPages(k, v)
    q = torch.randn(8, 8, 64, device="cuda", dtype=torch.bfloat16)
    out = torch.zeros_like(q)
    plan = L.AttnPlan(pages, 8, torch.bfloat16, 200, 8, 512)
    table = np.arange(64).reshape(8, 8)
    plan.set([1] * 3, [9, 100, 128], table[:3])
    plan.run(q, pages, out)
    st = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        plan.run(q, pages, out)
        with pytest.raises(L.LlmError, match="captured"):
            plan.set([1], [1], table[:1])
    for n_new, n_kv in (([1] * 8, [128, 1, 2, 3, 64, 65, 17, 0]), ([2, 1], [5, 128]), ([1] * 3, [9, 100, 128])):
        plan.set(n_new, n_kv, table[:len(n_new)])
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        T = sum(n_new)
        ref, mag, smag = O.attention(q.double().cpu().numpy()[:T], kv_, vv, table, n_new, n_kv, 16)
        tol = O.attention_tol(ref, mag, smag, torch.bfloat16, 128, 64, np.abs(vv).max())
        assert (np.abs(out.double().cpu().numpy()[:T] - ref) <= tol).all()
        assert plan.error() == 0


def test_a_graph_refuses_steps_it_was_not_captured_for(L):
    (k, _, kv_), (v, _, vv) = O.cache(64, 16, 2, 64, torch.float16, 15)
    pages = L.KvPages(k, v)
    plan = L.AttnPlan(pages, 8, torch.float16, 64, 4, 256)
    q = torch.randn(40, 8, 64, device="cuda", dtype=torch.float16)
    out = torch.zeros_like(q)
    table = np.arange(64).reshape(1, 64)
    st = torch.cuda.Stream()
    plan.set([0], [30], table)
    assert plan.form == 0
    plan.run(q, pages, out)                                  # nothing to do
    with torch.cuda.graph(torch.cuda.CUDAGraph(), stream=st):
        with pytest.raises(L.LlmError, match="empty step"):
            plan.run(q, pages, out)
    plan.set([1], [300], table)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        plan.run(q, pages, out)
    with pytest.raises(ValueError, match="captured run"):
        plan.set([41], [300], table)
    plan.set([40], [300], table)                             # needs kernels that the graph has not
    out.fill_(3)
    g.replay()
    assert plan.error() == 16 and plan.error() == 0
    assert (out == 3).all()
    plan.set([1], [299], table)
    g.replay()
    assert plan.error() == 0
    ref, mag, smag = O.attention(q.double().cpu().numpy()[:1], kv_, vv, table, [1], [299], 16)
    tol = O.attention_tol(ref, mag, smag, torch.float16, 299, 64, np.abs(vv).max())
    assert (np.abs(out.double().cpu().numpy()[:1] - ref) <= tol).all()
    assert (out[1:] == 3).all()


def test_two_plans_on_two_streams(L):
    (k, _, kv_), (v, _, vv) = O.cache(300, 16, 1, 128, torch.float16, 6)
    pages = L.KvPages(k, v)
    table = np.tile(np.arange(300), (2, 1))
    jobs = []
    for i in range(2):
        plan = L.AttnPlan(pages, 4, torch.float16, 2, 2, 600)
        q = torch.randn(2, 4, 128, device="cuda", dtype=torch.float16)
        jobs.append((plan, q, torch.empty_like(q), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(5):
        for i, (plan, q, out, st) in enumerate(jobs):
            with torch.cuda.stream(st):
                plan.set([1, 1], [4800 - 7 * i, 2000], table)
                plan.run(q, pages, out)
    torch.cuda.synchronize()
    for i, (plan, q, out, st) in enumerate(jobs):
        n_kv = [4800 - 7 * i, 2000]
        ref, mag, smag = O.attention(q.double().cpu().numpy(), kv_, vv, table, [1, 1], n_kv, 16)
        tol = O.attention_tol(ref, mag, smag, torch.float16, 4800, 128, np.abs(vv).max())
        assert (np.abs(out.double().cpu().numpy() - ref) <= tol).all()


def test_refusals(L):
    (k, ks, _), (v, vs, _) = O.cache(4, 16, 2, 64, torch.float16, 1)
    pages = L.KvPages(k, v)
    with pytest.raises(L.LlmError):
        L.AttnPlan(pages, 8, torch.bfloat16, 4, 2, 8)
    with pytest.raises(L.LlmError):
        L.AttnPlan(pages, 7, torch.float16, 4, 2, 8)
    plan = L.AttnPlan(pages, 8, torch.float16, 4, 2, 4)
    ok = [[0, 1], [2, 3]]
    plan.set([1, 1], [20, 17], ok)
    for n_new, n_kv, t in (([4, 1], [9, 9], ok), ([1, 1], [33, 9], ok), ([1, 1, 1], [1, 1, 1], [[0], [1], [2]]),
                           ([1, -1], [1, 1], ok), ([1, 1], [1, -1], ok), ([1, 1], [20, 17], [[0, 4], [1, 2]]),
                           ([1, 1], [20, 17], [[0, 1], [-1, 2]])):
        with pytest.raises(L.LlmError):
            plan.set(n_new, n_kv, t)
    q = torch.randn(2, 8, 64, device="cuda", dtype=torch.float16)
    out = torch.empty_like(q)
    plan.run(q, pages, out)                                       # the plan kept what it held
    with pytest.raises(L.LlmError, match="device memory"):
        plan.run(q.cpu(), pages, out)
    with pytest.raises(TypeError):
        plan.run(q.float(), pages, out)
    with pytest.raises(ValueError):
        plan.run(q[:1], pages, out)
    with pytest.raises(L.LlmError, match="apart"):
        plan.run(q, pages, out[:1].expand(2, 8, 64))
    (k2, _, _), (v2, _, _) = O.cache(5, 16, 2, 64, torch.float16, 1)
    with pytest.raises(L.LlmError, match="plan's type and shape"):
        plan.run(q, L.KvPages(k2, v2), out)


def test_a_serving_step(L):
    """Prompt and decode steps of two sequences as a program would run them: rows written in 8 bits, attention
    over the pages with a window and sinks, logits from the outputs, one pick per sequence."""
    Hkv, G, hd, page, V = 2, 4, 64, 16, 500
    rng = np.random.default_rng(0)
    kc = torch.full((8, page, Hkv, hd), 0x7f, dtype=torch.uint8, device="cuda")
    vc = kc.clone()
    ks = torch.full((8, page, Hkv), float("nan"), device="cuda")
    vs = ks.clone()
    pages = L.KvPages(kc, vc, ks, vs)
    plan = L.AttnPlan(pages, Hkv * G, torch.bfloat16, 64, 2, 16, window=20, n_sink=2)
    table = np.array([[5, 1, 7], [0, 3, 2]])
    W = torch.from_numpy(rng.normal(size=(Hkv * G * hd, V)) * 0.2).float().cuda()
    kv_, vv = np.zeros((8 * page, Hkv, hd)), np.zeros((8 * page, Hkv, hd))
    n_kv = [0, 0]
    for n_new in ([33, 14], [1, 1], [1, 1], [1, 2]):
        T = sum(n_new)
        n_kv = [a + b for a, b in zip(n_kv, n_new)]
        cells = np.concatenate([[int(table[s][j // page]) * page + j % page for j in range(n_kv[s] - n_new[s], n_kv[s])]
                                for s in range(2)]).astype(np.int32)
        q, k, v = (torch.from_numpy(rng.normal(size=(T, h, hd))).to(torch.bfloat16).cuda() for h in (Hkv * G, Hkv, Hkv))
        L.kv_store(pages, k, v, torch.from_numpy(cells).cuda())
        plan.set(n_new, n_kv, table)
        out = torch.zeros(T, Hkv * G, hd, dtype=torch.bfloat16, device="cuda")
        plan.run(q, pages, out)
        last = torch.tensor([n_new[0] - 1, T - 1], device="cuda")
        logits = out[last].flatten(1).float() @ W
        token = torch.zeros(2, dtype=torch.int32, device="cuda")
        L.sample_rows(logits, token)                              # greedy
        for x, val in ((k, kv_), (v, vv)):
            code, s = O.quantise(x.double().cpu().numpy())
            val[cells] = O.E4M3[code] * s[..., None]
        ref, mag, smag = O.attention(q.double().cpu().numpy(), kv_, vv, table, n_new, n_kv, page, 20, 2)
        tol = O.attention_tol(ref, mag, smag, torch.bfloat16, max(n_kv), hd, np.abs(vv).max())
        assert (np.abs(out.double().cpu().numpy() - ref) <= tol).all()
        assert token.tolist() == logits.argmax(1).tolist()
    assert plan.error() == 0


def test_a_run_captured_on_a_stream_of_its_own(L):
    """The stream is named in the call and is not torch's current one: the captured run's rows bound later steps all
    the same."""
    (k, _, _), (v, _, _) = O.cache(64, 16, 2, 64, torch.float16, 16)
    pages = L.KvPages(k, v)
    plan = L.AttnPlan(pages, 8, torch.float16, 64, 4, 256)
    q = torch.randn(9, 8, 64, device="cuda", dtype=torch.float16)
    out, want = torch.zeros_like(q), torch.zeros_like(q)
    table = np.arange(64).reshape(1, 64)
    plan.set([1], [300], table)
    plan.run(q, pages, want, stream=0)
    st, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        g.capture_begin()
    plan.run(q, pages, out, stream=st.cuda_stream)
    with torch.cuda.stream(st):
        g.capture_end()
    with pytest.raises(ValueError, match="captured run"):
        plan.set([10], [300], table)
    plan.set([1], [300], table)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_one_token_whose_token_stride_says_nothing(L):
    """A tensor of one token may have any stride along the tokens (a transposed [heads, 1, dim], a column of a larger
    one): it is a step of one token all the same."""
    (k, _, _), (v, _, _) = O.cache(4, 16, 2, 64, torch.float16, 17)
    pages = L.KvPages(k, v)
    plan = L.AttnPlan(pages, 8, torch.float16, 4, 2, 4)
    plan.set([1], [50], [[0, 1, 2, 3]])
    q = torch.randn(1, 8, 64, device="cuda", dtype=torch.float16)
    want = torch.zeros_like(q)
    plan.run(q, pages, want)
    for out in (torch.zeros(8, 1, 64, device="cuda", dtype=torch.float16).transpose(0, 1),
                torch.zeros(512, device="cuda", dtype=torch.float16).as_strided((1, 8, 64), (3, 64, 1))):
        plan.run(q.as_strided((1, 8, 64), (5, 64, 1)), pages, out)
        assert torch.equal(out, want)
    (k1, _, _), (v1, _, _) = O.cache(4, 16, 1, 64, torch.float16, 18)
    plan = L.AttnPlan(L.KvPages(k1, v1), 1, torch.float16, 4, 2, 4)   # one head: its stride says nothing either
    plan.set([1], [50], [[0, 1, 2, 3]])
    out = torch.zeros(64, device="cuda", dtype=torch.float16).as_strided((1, 1, 64), (7, 9, 1))
    plan.run(q[:, :1], L.KvPages(k1, v1), out)
    want = torch.zeros(1, 1, 64, device="cuda", dtype=torch.float16)
    plan.run(q[:, :1].contiguous(), L.KvPages(k1, v1), want)
    assert torch.equal(out, want) and out.abs().sum() > 0
