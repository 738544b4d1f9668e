"""Edges of the operators over 4-bit pages and of the page tables on the GPU: cells past 32-bit offsets, rows and scales on
their least boundaries, many tiles and sequences in a plan set on the device, rows at the ends of a unit's scale range,
equal results launch after launch, several plans at once, one object used from several streams in turn."""
import numpy as np
import pytest
import torch

from tests import ops4_common as F
from tests import ops_common as O

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def L():
    import transformer_decode_kv_gb300 as L
    L.lib()
    return L


def ints(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32)).cuda()


def close(got, q, kval, vval, tables, n_new, n_kv, page, act, window=0, n_sink=0):
    T = int(sum(n_new))
    ref, mag, smag = O.attention(q.double().cpu().numpy()[:T], kval, vval, tables, n_new, n_kv, page, window, n_sink)
    tol = O.attention_tol(ref, mag, smag, act, max(n_kv), q.shape[2], np.abs(vval).max())
    bad = ~(np.abs(got.double().cpu().numpy()[:T] - ref) <= tol)
    assert not bad.any(), np.argwhere(bad)[:5]


@pytest.mark.parametrize("act,order", [(F16, "phcd"), (BF16, "pchd")])
def test_cells_past_32_bit_offsets(L, act, order):
    """Codes, block scales and scales each more than 2^32 bytes apart, by the stride of their pages: store, load, both
    forms of attention, runs of cells and single rows."""
    page, Hkv, hd, n_pages = 16, 2, 128, 4
    far = 2 ** 32 // 3 + 2 ** 28                                # pages 1 .. 3 lie past 1.6, 3.2 and 4.8 GB
    strides = {"phcd": (1, page), "pchd": (Hkv, 1)}[order]      # of cells and heads, in rows

    def wide(row, dtype, size):
        n = far // size // 64 * 64
        buf = torch.zeros(3 * n + page * Hkv * row, dtype=dtype, device="cuda")
        shape = (n_pages, page, Hkv) + ((row,) if row > 1 else ())
        return torch.as_strided(buf, shape, (n, strides[0] * row, strides[1] * row) + ((1,) if row > 1 else ()))
    c = [[wide(hd // 2, torch.uint8, 1), wide(1, F32, 4), wide(hd // 16, torch.uint8, 1)] for _ in range(2)]
    assert c[0][0].stride(0) * 3 > 2 ** 32 and c[0][2].stride(0) * 3 > 2 ** 32
    pages = F.kv_pages(L, *c)
    rng = np.random.default_rng(4)
    x = [torch.from_numpy(rng.normal(size=(n_pages * page, Hkv, hd))).float().cuda() for _ in range(2)]
    cell = torch.arange(n_pages * page, dtype=torch.int32, device="cuda")
    L.kv_store(pages, *x, cell)
    o = [torch.zeros_like(t) for t in x]
    L.kv_load(pages, cell, *o)
    val = [F.values(*F.quantise(t.double().cpu().numpy())) for t in x]
    for a, b in zip(o, val):
        assert np.array_equal(a.double().cpu().numpy(), b)
    table, n_new, n_kv = np.array([[3, 1, 2, 0]] * 2, np.int32), [1, 40], [50, 64]
    q = torch.from_numpy(rng.normal(size=(41, 8, hd))).to(act).cuda()
    out = torch.zeros_like(q)
    plan = L.AttnPlan(pages, 8, act, 41, 2, 8)
    plan.set(n_new, n_kv, table)
    plan.run(q, pages, out)
    assert plan.error() == 0
    close(out, q, *val, table, n_new, n_kv, page, act)


@pytest.mark.parametrize("act", [F16, BF16, F32])
@pytest.mark.parametrize("hd", [32, 64, 128])
@pytest.mark.parametrize("n_new", [1, 5, 70])
def test_rows_on_their_least_boundaries(L, act, hd, n_new):
    """Rows on odd multiples of 16 bytes, block scales on odd multiples of their row, scales on odd words: no run of cells
    can be copied as one, and no dense row takes 32 bytes at once."""
    page, Hkv, n_pages = 8, 2, 20
    rng = np.random.default_rng(hd + n_new)

    def odd(row, dtype, skip):
        shape = (n_pages, Hkv, page) + ((row,) if row > 1 else ())
        buf = torch.zeros(int(np.prod(shape)) + skip, dtype=dtype, device="cuda")
        return buf[skip:].view(shape).transpose(1, 2)
    c = [[odd(hd // 2, torch.uint8, 16), odd(1, F32, 1), odd(hd // 16, torch.uint8, hd // 16)] for _ in range(2)]
    pages = F.kv_pages(L, *c)
    e = 16 // torch.finfo(act).bits * 8 if act != F32 else 4    # elements of 16 bytes
    dense = lambda h: torch.zeros(n_pages * page * h * hd + e, dtype=act, device="cuda")[e:].view(n_pages * page, h, hd)
    x, o = [dense(Hkv) for _ in range(2)], [dense(Hkv) for _ in range(2)]
    for t in x:
        t.copy_(torch.from_numpy(rng.normal(size=tuple(t.shape))))
    cell = ints(rng.permutation(n_pages * page))
    L.kv_store(pages, *x, cell)
    L.kv_load(pages, cell, *o)
    val = []
    for a, b in zip(x, o):
        v = F.values(*F.quantise(a.double().cpu().numpy()))
        assert torch.equal(b.cpu(), torch.from_numpy(v).to(act))
        w = np.zeros_like(v)
        w[cell.cpu().numpy()] = v
        val.append(w)
    table, n_kv = rng.permutation(n_pages).astype(np.int32)[None], [n_pages * page - 3]
    q, out = dense(8)[:n_new], dense(8)[:n_new]
    q.copy_(torch.from_numpy(rng.normal(size=tuple(q.shape))))
    plan = L.AttnPlan(pages, 8, act, n_new, 1, n_pages)
    plan.set([n_new], n_kv, table)
    plan.run(q, pages, out)
    assert plan.error() == 0
    close(out, q, *val, table, [n_new], n_kv, page, act)


@pytest.mark.parametrize("power", [-13, -12, 5, 6, 7, 9])
@pytest.mark.parametrize("which", ["k", "v"])
def test_rows_at_the_ends_of_the_range_of_a_unit(L, power, which):
    """A row far behind a unit's first 128 keys whose scale is 2^power times the largest there, in chunks that take 256-row
    tiles: exact in f16 from 2^-12 to 2^6, done key by key outside."""
    def at(scale):
        rng = np.random.default_rng(power + 20)
        page, hd, n_kv = 16, 64, 400
        x = [rng.uniform(-1, 1, size=(n_kv, 1, hd)) for _ in range(2)]
        x[0 if which == "k" else 1][300] *= scale
        for t in x:
            t[:, 0, 0] = np.abs(t).max((1, 2)) * 1.0               # (a row's largest value where all rows have it)
        return page, hd, n_kv, x
    page, hd, n_kv, x = at(2.0 ** power)
    if which == "k":
        x[0] *= 2.0 ** -3
    got = []
    code = [F.quantise(t) for t in x]
    val = [F.values(*c) for c in code]
    c = [[F.ordered(torch.from_numpy(v).view(-1, page, *v.shape[1:]), "phcd") for v in
          (F.pack(q4), s.astype(np.float32), b)] for q4, b, s in code]
    pages = F.kv_pages(L, *c)
    rng = np.random.default_rng(1)
    for act in (F16, BF16):
        q = torch.from_numpy(rng.normal(size=(200, 4, hd)) * (0.05 if which == "k" else 1)).to(act).cuda()
        out = torch.zeros_like(q)
        plan = L.AttnPlan(pages, 4, act, 200, 1, 25)
        plan.set([200], [n_kv], np.arange(25)[None])
        assert plan.form == 4
        plan.run(q, pages, out)
        assert plan.error() == 0
        close(out, q, *val, [list(range(25))], [200], [n_kv], page, act)


def test_many_tiles_and_sequences_in_a_plan_set_on_the_device(L):
    """More tiles than fit the planner's shared memory, and more sequences, with a window that keeps the keys few."""
    rng = np.random.default_rng(2)
    for n_new, more, window, hd in (([4200], 0, 5, 32), ([1] * 1500, 40, 0, 32), ([3] * 900 + [0] * 50 + [9] * 40, 20, 6, 64)):
        n_kv = [n + int(rng.integers(0, more + 1)) for n in n_new]
        page = 16
        need = [-(-n // page) for n in n_kv]
        table = np.zeros((len(n_kv), max(need)), np.int32)
        perm, at = rng.permutation(sum(need)).astype(np.int32), 0
        for i, m in enumerate(need):
            table[i, :m] = perm[at:at + m]
            at += m
        (k, kval), (v, vval) = F.cache(sum(need), page, 1, hd, 3)
        pages = F.kv_pages(L, k, v)
        act = F32 if len(n_new) == 1 else F16
        q = torch.from_numpy(rng.normal(size=(sum(n_new), 4, hd))).to(act).cuda()
        out = torch.zeros_like(q)
        plan = L.AttnPlan(pages, 4, act, sum(n_new), len(n_new), sum(need), window=window, n_sink=1)
        plan.set_device(ints(np.concatenate([[0], np.cumsum(n_new)])), ints(n_kv), ints(table), max(n_new))
        plan.run(q, pages, out)
        assert plan.error() == 0
        close(out, q, kval, vval, table, n_new, n_kv, page, act, window, 1)


def test_results_do_not_depend_on_the_launch(L):
    """The same bits every time, alone and beside other work, for both forms and cut tiles."""
    rng = np.random.default_rng(6)
    n_new, n_kv, page, hd = [1, 1, 200], [3000, 700, 900], 32, 128
    need = [-(-n // page) for n in n_kv]
    table = np.zeros((3, max(need)), np.int32)
    perm, at = rng.permutation(sum(need)).astype(np.int32), 0
    for i, m in enumerate(need):
        table[i, :m] = perm[at:at + m]
        at += m
    (k, _), (v, _) = F.cache(sum(need), page, 2, hd, 3)
    pages = F.kv_pages(L, k, v)
    q = torch.randn(202, 8, hd, device="cuda").to(BF16)
    plan = L.AttnPlan(pages, 8, BF16, 202, 3, table.size)
    start = ints([0, 1, 2, 202])
    side = torch.cuda.Stream()
    noise = torch.randn(2048, 2048, device="cuda")
    first = None
    for i in range(6):
        out = torch.full_like(q, float("nan"))
        plan.set_device(start, ints(n_kv), ints(table), 200)
        with torch.cuda.stream(side):
            for _ in range(i):
                noise = (noise @ noise).clamp(-1, 1)
        plan.run(q, pages, out)
        torch.cuda.synchronize()
        first = out if first is None else first
        assert torch.equal(out, first)
    assert plan.error() == 0


def test_two_plans_and_two_page_lists_at_once(L):
    """Two serving loops on two streams, each with its own plan and lists, over one cache's disjoint pages."""
    page, Hkv, hd = 16, 2, 64
    (k, kval), (v, vval) = F.cache(40, page, Hkv, hd, 8)
    pages = F.kv_pages(L, k, v)
    loops = []
    for i in range(2):
        own = np.arange(20 * i, 20 * i + 20)
        lists = L.SeqPages(ints(np.zeros((3, 6))), ints([0, 0, 0]), ints(own), ints([20]), page, 40)
        plan = L.AttnPlan(pages, 4, F16, 30, 3, 18)
        loops.append(dict(lists=lists, plan=plan, st=torch.cuda.Stream(), free=own.tolist(), table=np.zeros((3, 6), np.int32), kv=[0, 0, 0]))
    torch.cuda.synchronize()
    rng = np.random.default_rng(9)
    for step in range(5):
        for l in loops:
            add = [int(a) for a in rng.integers(0, 10, 3)]
            l["add"] = add
            x = [torch.from_numpy(rng.normal(size=(30, Hkv, hd))).to(F16).cuda() for _ in range(2)]
            l["q"] = torch.from_numpy(rng.normal(size=(30, 4, hd))).to(F16).cuda()
            l["x"], l["out"] = x, torch.full_like(l["q"], 5.0)
            l["n"], l["cell"], l["pos"], l["start"], l["err"] = ints(add), ints([0] * 30), ints([0] * 30), ints([0] * 4), ints([0])
        torch.cuda.synchronize()
        for l in loops:
            with torch.cuda.stream(l["st"]):
                L.pages_extend(l["lists"], l["n"], l["cell"], l["pos"], l["start"], err=l["err"])
                L.kv_store(pages, *l["x"], l["cell"])
                l["plan"].set_device(l["start"], l["lists"].n_kv, l["lists"].table, 9)
                l["plan"].run(l["q"], pages, l["out"])
        torch.cuda.synchronize()
        for l in loops:
            l["table"], cell, _, _, l["kv"], l["free"] = F.extend(l["table"], l["kv"], l["add"], l["free"], page, 30)
            T = sum(l["add"])
            assert int(l["err"]) == 0 and l["plan"].error() == 0 and l["cell"].tolist() == cell
            for x, val in zip(l["x"], (kval, vval)):
                val[np.array(cell[:T], int)] = F.values(*F.quantise(x.double().cpu().numpy()[:T]))
            if T:
                close(l["out"], l["q"], kval, vval, l["table"], l["add"], l["kv"], page, F16)
            assert (l["out"][T:] == 5.0).all()


def test_infinite_operands(L):
    """Infinities: a value's reach the rows that see it, a query's make its scores infinite or NaN as the formula has it,
    and rows that do not see them keep their results."""
    page, hd = 16, 64
    (k, kval), (v, vval) = F.cache(10, page, 1, hd, 2)
    v[1][3, 5, 0] = float("inf")                                # key 53 of the sequence
    vval[53, 0] = np.inf
    pages = F.kv_pages(L, k, v)
    table = np.arange(10, dtype=np.int32)[None]
    for n_new in (2, 150):
        q = torch.randn(n_new, 4, hd, device="cuda").half()
        out = torch.zeros_like(q)
        plan = L.AttnPlan(pages, 4, F16, n_new, 1, 10)
        for n_kv in (53 + n_new // 2, 160):                     # (rows before key 53 do not see it)
            if n_kv < n_new:
                continue
            plan.set([n_new], [n_kv], table)
            plan.run(q, pages, out)
            assert plan.error() == 0
            seen = np.arange(n_kv - n_new, n_kv) >= 53
            got = out.double().cpu().numpy()
            assert not np.isfinite(got[seen]).any()
            clean = vval.copy()
            clean[53] = 0
            ref, mag, smag = O.attention(q.double().cpu().numpy(), kval, clean, table, [n_new], [n_kv], page)
            tol = O.attention_tol(ref, mag, smag, F16, n_kv, hd, np.abs(clean).max())
            assert (np.abs(got - ref) <= tol)[~seen].all()
