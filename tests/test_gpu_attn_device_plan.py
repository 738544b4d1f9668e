"""Plans set from lengths and page tables on the device: attention results against the formula in 64 bits over every
cache type, head layout and step shape, steps that do not fit, and whole serving steps (pages, rows, plan,
attention) captured once and replayed with other lengths."""
import numpy as np
import pytest
import torch

from tests import ops4_common as F
from tests import ops_common as O

pytestmark = pytest.mark.gpu

PAIRS = [(torch.float16, torch.float16), (torch.bfloat16, torch.bfloat16), (torch.float32, torch.float16),
         (torch.bfloat16, torch.uint8), (torch.float16, "f4"), (torch.bfloat16, "f4")]


@pytest.fixture(scope="module")
def L():
    import transformer_decode_kv_gb300 as L
    L.lib()
    return L


def ints(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32)).cuda()


def caches(L, cdt, n_pages, page, Hkv, hd, seed):
    """(KvPages, float64 keys, float64 values)"""
    if cdt == "f4":
        (k, kval), (v, vval) = F.cache(n_pages, page, Hkv, hd, seed)
        return F.kv_pages(L, k, v), kval, vval
    (k, ks, kval), (v, vs, vval) = O.cache(n_pages, page, Hkv, hd, cdt, seed)
    return L.KvPages(k, v, ks, vs), kval, vval


def tables_of(n_kv, page, rng, ld_more=2):
    need = [-(-int(n) // page) for n in n_kv]
    n_pages = sum(need) + 2
    perm = rng.permutation(n_pages).astype(np.int32)
    t = np.full((len(n_kv), max(need + [0]) + ld_more), 1 << 20, np.int32)   # entries past a sequence are not read
    at = 0
    for i, m in enumerate(need):
        t[i, :m] = perm[at:at + m]
        at += m
    return t, n_pages


def verify(got, q, kval, vval, tables, n_new, n_kv, page, window, n_sink, act):
    T = int(sum(n_new))
    ref, mag, smag = O.attention(q.double().cpu().numpy()[:T], kval, vval, tables, n_new, n_kv, page, window, n_sink)
    tol = O.attention_tol(ref, mag, smag, act, max(list(n_kv) + [1]), q.shape[2], np.abs(vval).max())
    bad = ~(np.abs(got[:T] - ref) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:5], got[:T][bad][:5], ref[bad][:5], tol[bad][:5])


def check(L, act, cdt, hd, Hkv, G, page, n_new, n_kv, window=0, n_sink=0, seed=0, max_new=None, extra=3):
    rng = np.random.default_rng(seed)
    tables, n_pages = tables_of(n_kv, page, rng)
    pages, kval, vval = caches(L, cdt, n_pages, page, Hkv, hd, seed + 1)
    T = int(sum(n_new))
    q = torch.from_numpy(rng.normal(size=(T + extra, Hkv * G, hd))).to(act).cuda()
    out = torch.full_like(q, 77.0)
    plan = L.AttnPlan(pages, n_head=Hkv * G, dtype=act, max_tok=T + extra, max_seq=len(n_new) + 1,
                      max_table=max(1, sum(-(-n // page) for n in n_kv)), window=window, n_sink=n_sink)
    plan.set_device(ints(np.concatenate([[0], np.cumsum(n_new)])), ints(n_kv), ints(tables),
                    max(list(n_new) + [0]) if max_new is None else max_new)
    plan.run(q, pages, out)
    assert plan.error() == 0
    got = out.double().cpu().numpy()
    assert (got[T:] == 77.0).all()
    verify(got, q, kval, vval, tables, n_new, n_kv, page, window, n_sink, act)
    return plan


STEPS = [([1], [1]), ([1], [300]), ([1] * 5, [17, 1, 64, 301, 2000]), ([5, 0, 1, 33], [5, 9, 200, 90]), ([200, 1, 64], [700, 900, 64]),
         ([130], [130])]


@pytest.mark.parametrize("act,cdt", PAIRS)
@pytest.mark.parametrize("hd", [32, 64, 128])
@pytest.mark.parametrize("n_new,n_kv", STEPS)
def test_types_and_steps(L, act, cdt, hd, n_new, n_kv):
    check(L, act, cdt, hd, 2, 4, 16, n_new, n_kv, seed=hd)


@pytest.mark.parametrize("Hkv,G", [(1, 1), (1, 32), (8, 1), (3, 7), (2, 16)])
@pytest.mark.parametrize("page", [1, 17, 64])
def test_heads_and_pages(L, Hkv, G, page):
    check(L, torch.float16, "f4", 64, Hkv, G, page, [1, 6, 0, 2], [40, 6, 9, 131], seed=G)
    check(L, torch.float16, torch.float16, 128, Hkv, G, page, [1, 90], [400, 131], seed=G)


@pytest.mark.parametrize("window,n_sink", [(1, 0), (7, 4), (64, 4), (300, 16), (2 ** 31 - 1, 0), (50, 2 ** 31 - 1)])
@pytest.mark.parametrize("act,cdt", [PAIRS[0], PAIRS[1], PAIRS[5]])
def test_windows_and_sinks(L, act, cdt, window, n_sink):
    check(L, act, cdt, 64, 2, 4, 16, [1, 70, 3, 1], [500, 80, 3, 66], window, n_sink, seed=7)
    check(L, act, cdt, 128, 2, 4, 16, [150, 1], [700, 900], window, n_sink, seed=8)


def test_rows_that_see_nothing_and_empty_steps(L):
    for act, cdt in (PAIRS[0], PAIRS[4]):
        check(L, act, cdt, 64, 2, 4, 16, [3, 1, 50, 0], [0, 5, 20, 7], seed=3)
        check(L, act, cdt, 128, 1, 4, 16, [2], [0], seed=4)
        check(L, act, cdt, 64, 2, 4, 16, [], [], seed=5)
        check(L, act, cdt, 64, 2, 4, 16, [0, 0], [0, 9], seed=6)
        check(L, act, cdt, 64, 2, 4, 16, [0, 0], [0, 9], seed=6, max_new=3)


@pytest.mark.parametrize("act,cdt", [PAIRS[0], PAIRS[3], PAIRS[4]])
def test_long_ranges_and_many_sequences(L, act, cdt):
    check(L, act, cdt, 128, 1, 4, 16, [1, 2], [9000, 3001], seed=11)
    rng = np.random.default_rng(5)
    check(L, act, cdt, 64, 2, 2, 4, [1] * 700, rng.integers(1, 30, 700).tolist(), seed=12)
    n_new = rng.integers(0, 4, 600)
    check(L, act, cdt, 32, 1, 4, 8, n_new.tolist(), (n_new + rng.integers(0, 30, 600)).tolist(), seed=13, max_new=5)


def test_the_same_rows_as_a_plan_set_from_the_host(L):
    """One plan, set either way: the units differ, the results by the order of float32 sums only; a wider max_new
    changes the kernels, not the step."""
    rng = np.random.default_rng(2)
    n_new, n_kv, page = [1, 1, 9], [700, 40, 300], 16
    tables, n_pages = tables_of(n_kv, page, rng)
    pages, kval, vval = caches(L, torch.float16, n_pages, page, 2, 128, 3)
    q = torch.randn(11, 8, 128, device="cuda").half()
    plan = L.AttnPlan(pages, n_head=8, dtype=torch.float16, max_tok=11, max_seq=3, max_table=tables.size)
    start = ints([0, 1, 2, 11])
    for way in ("host", "device", "wide", "host"):
        out = torch.zeros_like(q)
        if way == "host":
            plan.set(n_new, n_kv, tables)
        else:
            plan.set_device(start, ints(n_kv), ints(tables), 9 if way == "device" else 11)
        plan.run(q, pages, out)
        assert plan.error() == 0
        verify(out.double().cpu().numpy(), q, kval, vval, tables, n_new, n_kv, page, 0, 0, torch.float16)


def test_the_planner_of_64_bits_makes_the_same_plan(L):
    """Bounds under which places on the plan's line may pass 32 bits (long table rows, many tokens) select wider sums."""
    rng = np.random.default_rng(4)
    n_new, n_kv, page = [1, 30, 70, 0], [900, 40, 300, 5], 256
    tables, n_pages = tables_of(n_kv, page, rng)
    wide = np.zeros((4, 1 << 20), np.int32)
    wide[:, :tables.shape[1]] = tables
    for act, cdt in (PAIRS[0], PAIRS[5]):
        pages, kval, vval = caches(L, cdt, n_pages, page, 2, 64, 3)
        q = torch.from_numpy(rng.normal(size=(4096, 8, 64))).to(act).cuda()
        outs = []
        for table, max_tok, max_table in ((tables, 101, 16), (wide, 4096, 1 << 22)):
            plan = L.AttnPlan(pages, n_head=8, dtype=act, max_tok=max_tok, max_seq=4, max_table=max_table)
            out = torch.zeros_like(q)
            plan.set_device(ints([0, 1, 31, 101, 101]), ints(n_kv), ints(table), 70)
            plan.run(q, pages, out)
            assert plan.error() == 0
            outs.append(out)
        assert torch.equal(*outs)
        verify(outs[0].double().cpu().numpy(), q, kval, vval, tables, n_new, n_kv, page, 0, 0, act)


@pytest.mark.parametrize("bad", [
    dict(start=[1, 2, 3]), dict(start=[0, 2, 1]), dict(start=[0, 1, 9]), dict(start=[0, 4, 5]), dict(n_kv=[-1, 9]),
    dict(n_kv=[9, 33]), dict(n_kv=[2 ** 31 - 1, 9]), dict(n_kv=[32, 32], max_table=3), dict(start=[0, 2 ** 31 - 1, -2])])
def test_steps_that_do_not_fit_leave_the_output_alone(L, bad):
    (k, kval), (v, vval) = F.cache(8, 16, 1, 64, 1)
    pages = F.kv_pages(L, k, v)
    plan = L.AttnPlan(pages, n_head=4, dtype=torch.float16, max_tok=8, max_seq=2, max_table=bad.get("max_table", 8))
    q = torch.randn(8, 4, 64, device="cuda").half()
    out = torch.full_like(q, 20000.0)
    plan.set_device(ints(bad.get("start", [0, 1, 2])), ints(bad.get("n_kv", [5, 9])), ints([[0, 1], [2, 3]]), 3)
    plan.run(q, pages, out)
    assert plan.error() == 32 and (out == 20000.0).all()
    plan.set_device(ints([0, 1, 2]), ints([5, 9]), ints([[0, 1], [2, 3]]), 3)
    plan.run(q, pages, out)                                     # and the plan goes on
    assert plan.error() == 0 and (out[2:] == 20000.0).all() and not (out[:2] == 20000.0).any()


def test_pages_outside_the_cache_are_not_read(L):
    (k, kval), (v, vval) = F.cache(8, 16, 1, 64, 1)
    pages = F.kv_pages(L, k, v)
    plan = L.AttnPlan(pages, n_head=4, dtype=torch.float16, max_tok=2, max_seq=1, max_table=8)
    q = torch.randn(2, 4, 64, device="cuda").half()
    out = torch.zeros_like(q)
    plan.set_device(ints([0, 1]), ints([40]), ints([[3, 8, -1, 5]]), 1)
    plan.run(q, pages, out)
    assert plan.error() == 1
    plan.set_device(ints([0, 1]), ints([16]), ints([[3, 8, -1, 5]]), 1)
    one = torch.zeros_like(q)
    plan.run(q, pages, one)                                     # the keys of the good page
    assert plan.error() == 0
    assert (out[:1].float() - one[:1].float()).abs().max() < 2e-3


def test_refusals(L):
    (k, _), (v, _) = F.cache(8, 16, 1, 64, 1)
    pages = F.kv_pages(L, k, v)
    plan = L.AttnPlan(pages, n_head=4, dtype=torch.float16, max_tok=8, max_seq=2, max_table=8)
    s, n, t = ints([0, 1, 2]), ints([5, 9]), ints([[0, 1], [2, 3]])
    for args, why in (((ints([0] * 4), ints([1] * 3), ints([[0]] * 3), 1), "max_seq"), ((s, n, t, 9), "max_new"), ((s, n, t, -1), "max_new"),
                      ((s.cpu(), n, t, 1), "not device memory"), ((s, n, t.cpu(), 1), "not device memory")):
        with pytest.raises(L.LlmError, match=why):
            plan.set_device(*args)
    for args in ((s[:2], n, t, 1), (s, n.long(), t, 1), (s, n, t[:1], 1), (s, n, ints([[0, 1, 9], [2, 3, 9]])[:, :2], 1)):
        with pytest.raises(ValueError):
            plan.set_device(*args)
    plan.set_device(s, n, t, 1)
    q = torch.randn(7, 4, 64, device="cuda").half()
    with pytest.raises(ValueError, match="fewer rows"):
        plan.run(q, pages, torch.zeros_like(q))                 # fewer than max_tok rows
    plan.set([1, 1], [5, 9], [[0, 1], [2, 3]])
    g = torch.cuda.CUDAGraph()
    out = torch.zeros_like(q)
    plan.run(q, pages, out)
    with torch.cuda.graph(g):
        plan.run(q, pages, out)
    with pytest.raises(ValueError, match="captured"):
        plan.set_device(s, n, t, 1)                             # a graph holds a run whose rows would not do


@pytest.mark.parametrize("cdt,max_new", [(torch.float16, 1), ("f4", 1), ("f4", 40), (torch.bfloat16, 40)])
def test_serving_steps_in_one_graph(L, cdt, max_new):
    """extend -> store -> plan -> attention -> trim, captured once: steps of other lengths, sequences that end and begin
    again, against the host's books and the formula over the rows as they were stored."""
    act = torch.bfloat16 if cdt == torch.bfloat16 else torch.float16
    rng = np.random.default_rng(3)
    n_seq, page, Hkv, G, hd, ld = 6, 8, 2, 4, 64, 40
    n_pages, tok = 120, 6 * max_new
    pages, kval, vval = caches(L, cdt, n_pages, page, Hkv, hd, 5)
    table, kv, stack = np.full((n_seq, ld), -1, np.int32), [0] * n_seq, rng.permutation(n_pages).tolist()
    lists = L.SeqPages(ints(table), ints(kv), ints(stack), ints([n_pages]), page, n_pages)
    n_new, keep, err = ints([0] * n_seq), ints([-1] * n_seq), ints([0])
    cell, pos, start = ints([0] * tok), ints([0] * tok), ints([0] * (n_seq + 1))
    k, v = (torch.zeros(tok, Hkv, hd, dtype=act, device="cuda") for _ in range(2))
    q = torch.zeros(tok, Hkv * G, hd, dtype=act, device="cuda")
    out = torch.zeros_like(q)
    plan = L.AttnPlan(pages, n_head=Hkv * G, dtype=act, max_tok=tok, max_seq=n_seq, max_table=n_seq * ld)

    def step():
        L.pages_extend(lists, n_new, cell, pos, start, err=err)
        L.kv_store(pages, k, v, cell, err=err)
        plan.set_device(start, lists.n_kv, lists.table, max_new)
        plan.run(q, pages, out)
        L.pages_trim(lists, keep, err=err)

    step()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        step()
    for i in range(12):
        add = [int(x) for x in rng.integers(0, max_new + 1, n_seq)]
        cut = [0 if rng.random() < 0.15 else -1 for _ in range(n_seq)]
        n_new.copy_(ints(add)); keep.copy_(ints(cut))
        for t in (k, v, q):
            t.copy_(torch.from_numpy(rng.normal(size=tuple(t.shape))))
        out.fill_(77.0)
        g.replay()
        torch.cuda.synchronize()
        table, c, p, s, after, stack = F.extend(table, kv, add, stack, page, tok)
        assert int(err) == 0 and plan.error() == 0 and cell.tolist() == c and pos.tolist() == p and start.tolist() == s
        T = sum(add)
        for x, val in ((k, kval), (v, vval)):
            x = x.double().cpu().numpy()[:T]
            val[np.array(c[:T], int)] = F.values(*F.quantise(x)) if cdt == "f4" else x
        got = out.double().cpu().numpy()
        assert (got[T:] == 77.0).all()
        if T:
            verify(got, q, kval, vval, table, add, after, page, 0, 0, act)
        for j, x in enumerate(cut):
            if x == 0:
                stack += [int(table[j, m]) for m in range(-(-after[j] // page))]
                after[j] = 0
        kv = after
        assert lists.n_kv.tolist() == kv and lists.free.tolist()[:len(stack)] == stack


def replayed_plan(L, act, cdt, n_new, n_kv, max_tok, max_new, run_inside=False, seed=21):
    """A plan, and a graph that sets it on the device to this step (and runs it, where asked)."""
    rng = np.random.default_rng(seed)
    tables, n_pages = tables_of(n_kv, 16, rng)
    pages, kval, vval = caches(L, cdt, n_pages, 16, 2, 64, seed + 1)
    q = torch.from_numpy(rng.normal(size=(max_tok, 8, 64))).to(act).cuda()
    out = torch.full_like(q, 77.0)
    plan = L.AttnPlan(pages, n_head=8, dtype=act, max_tok=max_tok, max_seq=len(n_new) + 1, max_table=tables.size)
    args = ints(np.concatenate([[0], np.cumsum(n_new)])), ints(n_kv), ints(tables), max_new
    plan.set_device(*args)                                      # (the first launches, not captured)
    plan.run(q, pages, out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        plan.set_device(*args)
        if run_inside:
            plan.run(q, pages, out)
    out.fill_(77.0)

    def right():
        assert plan.error() == 0
        got = out.double().cpu().numpy()
        assert (got[sum(n_new):] == 77.0).all()
        verify(got, q, kval, vval, tables, n_new, n_kv, 16, 0, 0, act)
    return plan, g, pages, q, out, tables, right, args


@pytest.mark.parametrize("act,cdt", [PAIRS[0], PAIRS[4]])
def test_runs_after_a_replayed_set_need_the_rows_of_its_step(L, act, cdt):
    """set_device captured, a smaller step set by the host, the graph replayed: the plan holds the graph's step again, and a run
    whose q and out would do for the host's is refused."""
    plan, g, pages, q, out, tables, right, _ = replayed_plan(L, act, cdt, [1] * 7, [40, 3, 90, 17, 1, 64, 33], 8, 1)
    plan.set([1], [40], tables[:1])
    g.replay()
    for n in (1, 7):
        with pytest.raises(ValueError, match="fewer rows"):
            plan.run(q[:n], pages, out[:n])
    assert (out == 77.0).all()
    plan.run(q, pages, out)
    right()
    plan.set([1], [40], tables[:1])                             # and the host's step where no replay came after it
    out.fill_(77.0)
    plan.run(q, pages, out)
    assert plan.error() == 0 and (out[1:] == 77.0).all() and not (out[:1] == 77.0).any()


CHUNKS = [1, 40, 0, 1], [30, 90, 5, 17]
SINGLES = [1] * 7, [40, 3, 90, 17, 1, 64, 33]


@pytest.mark.parametrize("n_new,n_kv,max_new,first", [(*SINGLES, 1, []), (*SINGLES, 1, [40]), (*CHUNKS, 40, [1]), (*CHUNKS, 40, [])])
@pytest.mark.parametrize("act,cdt", [PAIRS[0], PAIRS[4]])
def test_runs_after_a_replayed_set_launch_what_its_step_needs(L, act, cdt, n_new, n_kv, max_new, first):
    """The host's step in between is empty, or needs other kernels than the graph's."""
    plan, g, pages, q, out, tables, right, _ = replayed_plan(L, act, cdt, n_new, n_kv, 64, max_new)
    plan.set(first, [n + 3 for n in first], tables[:len(first)])
    g.replay()
    plan.run(q, pages, out)
    right()
    # the same run captured, in a graph without the set, also where the step at hand is empty
    plan.set([], [], tables[:0])
    runs = torch.cuda.CUDAGraph()
    with torch.cuda.graph(runs):
        plan.run(q, pages, out)
    out.fill_(77.0)
    g.replay()
    runs.replay()
    torch.cuda.synchronize()
    right()
    # an empty step, which has not to be taken for the graph's
    plan.set([], [], tables[:0])
    out.fill_(77.0)
    plan.run(q, pages, out)
    assert plan.error() == 0 and (out == 77.0).all()


@pytest.mark.parametrize("act,cdt", [PAIRS[0], PAIRS[4]])
def test_a_captured_set_that_is_not_replayed_changes_no_step(L, act, cdt):
    """Between the capture and its replays the device holds what was set before, from the host or on the device."""
    plan, g, pages, q, out, tables, right, args = replayed_plan(L, act, cdt, *CHUNKS, 64, 40)
    for way in ("host", "device"):
        if way == "host":
            plan.set(*CHUNKS, tables)
        else:
            plan.set_device(*args)
        other = torch.cuda.CUDAGraph()
        with torch.cuda.graph(other):
            plan.set_device(*args[:3], 1)
        out.fill_(77.0)
        plan.run(q, pages, out)
        right()
    other.replay()                                              # more new tokens than its max_new
    out.fill_(77.0)
    plan.run(q, pages, out)
    assert plan.error() == 32 and (out == 77.0).all()


def test_two_graphs_with_other_steps_of_one_plan(L):
    """Decode steps and chunks, each with its own set and run, in turn."""
    act, cdt = PAIRS[5]
    plan, decode, pages, q, out, tables, right, args = replayed_plan(L, act, cdt, *SINGLES, 64, 1, run_inside=True)
    start, kv = ints([0, 0, 0, 40, 40, 40, 40, 40]), ints([40, 3, 90, 17, 1, 64, 33])
    chunks = torch.cuda.CUDAGraph()
    with torch.cuda.graph(chunks):
        plan.set_device(start, kv, args[2], 40)
        plan.run(q, pages, out)
    for _ in range(3):
        out.fill_(77.0)
        decode.replay()
        right()
        out.fill_(77.0)
        chunks.replay()
        assert plan.error() == 0 and (out[40:] == 77.0).all() and not (out[:40] == 77.0).any()
        first = out.clone() if _ == 0 else first
        assert torch.equal(out, first)
    plan.set([0, 0, 40, 0, 0, 0, 0], [40, 3, 90, 17, 1, 64, 33], tables)
    out.fill_(77.0)
    plan.run(q, pages, out)                                     # the same step from the host: sums in another order
    assert plan.error() == 0 and (out[:40].float() - first[:40].float()).abs().max() <= 2 ** -7 * first[:40].float().abs().max()


@pytest.mark.parametrize("act,cdt", [PAIRS[0], PAIRS[1], PAIRS[4]])
def test_plans_made_behind_replays_that_lack_their_kernels(L, act, cdt):
    """A captured run of both tile forms leaves a step of another form alone; the planner behind it, launched early, must not
    begin before both of its kernels have read the plan. Nothing is waited for in between."""
    rng = np.random.default_rng(31)
    mixed, few, one = ([1, 40, 1], [300, 700, 90]), ([3, 0, 2], [300, 9, 90]), ([1, 1, 1], [300, 700, 90])
    tables, n_pages = tables_of(mixed[1], 16, rng)
    pages, kval, vval = caches(L, cdt, n_pages, 16, 2, 64, 32)
    q = torch.from_numpy(rng.normal(size=(42, 8, 64))).to(act).cuda()
    lost = torch.full_like(q, 77.0)
    plan = L.AttnPlan(pages, n_head=8, dtype=act, max_tok=42, max_seq=3, max_table=tables.size)
    plan.set(*mixed, tables)
    assert plan.form == 5
    plan.run(q, pages, lost)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        plan.run(q, pages, lost)
    lost.fill_(77.0)
    table = ints(tables)
    on = [(ints(np.concatenate([[0], np.cumsum(n)])), ints(kv), m) for (n, kv), m in ((few, 3), (one, 1))]
    outs = [[torch.full_like(q, 55.0) for _ in range(20)] for _ in on]
    torch.cuda.synchronize()
    for i in range(20):
        plan.set_device(on[0][0], on[0][1], table, on[0][2])     # 16-row tiles, which the graph has not
        g.replay()
        for (start, kv, m), o in zip(on, outs):
            plan.set_device(start, kv, table, m)
            plan.run(q, pages, o[i])
    assert plan.error() == 16 and (lost == 77.0).all()
    for (n, kv), o in zip((few, one), outs):
        assert all(torch.equal(x, o[0]) for x in o) and (o[0][sum(n):] == 55.0).all()
        verify(o[0].double().cpu().numpy(), q, kval, vval, tables, n, kv, 16, 0, 0, act)


def attention_without(q, kval, vval, table, bad, n_new, n_kv, page, window, n_sink):
    """The formula over the keys whose pages are in the cache, for one sequence: (out, mag, smag, rows without a key)."""
    H, hd = q.shape[1:]
    G = H // kval.shape[1]
    j = np.arange(n_kv)
    good = ~np.isin(j // page, bad)
    cells = np.where(good, table[j // page].astype(np.int64), 0) * page + j % page
    out, mag, smag, none = np.zeros(q.shape), np.zeros(q.shape), np.zeros(q.shape[:2]), np.zeros(n_new, bool)
    for t in range(n_new):
        p = n_kv - n_new + t
        vis = good & (j <= p)
        if window:
            vis &= (j > p - window) | (j < n_sink)
        none[t] = not vis.any()
        if none[t]:
            continue
        for h in range(H):
            K, V = kval[cells[vis], h // G], vval[cells[vis], h // G]
            z = K @ q[t, h] * hd ** -0.5
            smag[t, h] = (np.abs(K) @ np.abs(q[t, h])).max() * hd ** -0.5
            w = np.exp(z - z.max())
            w /= w.sum()
            out[t, h], mag[t, h] = w @ V, w @ np.abs(V)
    return out, mag, smag, none


@pytest.mark.parametrize("act,cdt", [(torch.float16, torch.float16), (torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.uint8),
                                     (torch.float16, "f4"), (torch.bfloat16, "f4"), (torch.float32, torch.uint8)])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("page,window,n_sink", [(16, 0, 0), (64, 0, 0), (17, 0, 0), (16, 200, 40), (64, 300, 70), (1, 0, 0)])
@pytest.mark.parametrize("n_new", [50, 3])
def test_chunks_over_pages_outside_the_cache(L, act, cdt, hd, page, window, n_sink, n_new):
    """Entries past the cache and negative ones among whole runs of good pages, where blocks of keys are brought in bulk: their keys
    have no part, whatever the entry, and the others their full part."""
    rng = np.random.default_rng(41)
    n_kv = 700
    tables, n_pages = tables_of([n_kv], page, rng)
    need = -(-n_kv // page)
    pages, kval, vval = caches(L, cdt, n_pages, page, 2, hd, 42)
    bad = sorted({0, need // 3, need // 2, need // 2 + 2, need - 1})
    shown = tables.copy()
    shown[0, bad] = [-1, n_pages, 2 ** 31 - 1, -2 ** 31, n_pages + 5][:len(bad)]
    q = torch.from_numpy(rng.normal(size=(n_new + 1, 8, hd))).to(act).cuda()
    plan = L.AttnPlan(pages, n_head=8, dtype=act, max_tok=n_new + 1, max_seq=1, max_table=need, window=window, n_sink=n_sink)
    out = torch.full_like(q, 77.0)
    plan.set_device(ints([0, n_new]), ints([n_kv]), ints(shown), n_new)
    plan.run(q, pages, out)
    assert plan.form == (2 | (4 if n_new == 50 and act != torch.float32 else 0)) and plan.error() == 1
    got = out.double().cpu().numpy()
    assert (got[n_new:] == 77.0).all()
    ref, mag, smag, none = attention_without(q.double().cpu().numpy()[:n_new], kval, vval, tables[0], bad, n_new, n_kv, page, window,
                                             n_sink)
    tol = O.attention_tol(ref, mag, smag, act, n_kv, hd, np.abs(vval).max())
    assert not none.any()
    wrong = ~(np.abs(got[:n_new] - ref) <= tol)
    assert not wrong.any(), (np.argwhere(wrong)[:5], got[:n_new][wrong][:5], ref[wrong][:5], tol[wrong][:5])


@pytest.mark.parametrize("act,cdt", [(torch.float16, torch.float16), (torch.bfloat16, torch.uint8), (torch.float16, "f4")])
@pytest.mark.parametrize("n_new", [1, 9, 60])
def test_rows_whose_keys_are_all_on_pages_outside_the_cache(L, act, cdt, n_new):
    """Such a row is NaN, as one of scores without weight is; a row with one key left has that key's value."""
    rng = np.random.default_rng(43)
    pages, kval, vval = caches(L, cdt, 6, 64, 2, 64, 44)
    q = torch.from_numpy(rng.normal(size=(n_new, 8, 64))).to(act).cuda()
    out = torch.full_like(q, 77.0)
    plan = L.AttnPlan(pages, n_head=8, dtype=act, max_tok=n_new, max_seq=1, max_table=2)
    n_kv = 64 + (n_new + 1) // 2                                # the first rows see the bad page only
    if n_new == 1:
        n_kv = 64
    plan.set_device(ints([0, n_new]), ints([n_kv]), ints([[6, 3]]), n_new)
    plan.run(q, pages, out)
    assert plan.error() == 1
    got = out.double().cpu().numpy()
    p = np.arange(n_kv - n_new, n_kv)
    assert np.isnan(got[p < 64]).all() and (p < 64).any()
    if n_new > 1:
        one = got[p == 64][0]
        val = np.repeat(vval[3 * 64], 4, axis=0)
        assert (np.abs(one - val) <= 4 * O.HALF_EPS[act] * np.abs(val) + 1e-30).all()


@pytest.mark.parametrize("act,cdt", [PAIRS[0], PAIRS[5]])
def test_captured_steps_behind_copies_and_other_streams(L, act, cdt):
    """What is launched early has something else than a kernel in front in these graphs: a memset, a copy, two streams that meet; and
    two sets with their runs follow each other in one capture."""
    rng = np.random.default_rng(51)
    page, n_seq, tok = 16, 3, 45
    tables, n_pages = tables_of([700, 90, 33], page, rng)
    pages, kval, vval = caches(L, cdt, n_pages, page, 2, 64, 52)
    before, add = [659, 89, 30], [41, 1, 3]
    stack = [tables[2, 2], tables[0, 43], tables[0, 42]]          # (handed out last first)
    lists = L.SeqPages(ints(tables), ints(before), ints(stack), ints([3]), page, n_pages)
    n_new, cell, pos, start, after, left = ints([0] * 3), ints([0] * tok), ints([0] * tok), ints([0] * 4), ints([0] * 3), ints([0])
    src, err = ints(add), ints([0])
    x = [torch.from_numpy(rng.normal(size=(tok, 2, 64))).to(act).cuda() for _ in range(2)]
    k, v = (torch.zeros_like(t) for t in x)
    q = torch.from_numpy(rng.normal(size=(tok, 8, 64))).to(act).cuda()
    out, small = torch.full_like(q, 77.0), torch.full_like(q, 77.0)
    plan = L.AttnPlan(pages, n_head=8, dtype=act, max_tok=tok, max_seq=n_seq, max_table=tables.size)
    two = ints([0, 0, 1, 4])                                    # the last two sequences' new tokens alone
    side = torch.cuda.Stream()

    def step():
        here = torch.cuda.current_stream()
        n_new.copy_(src)
        L.pages_extend(lists, n_new, cell, pos, start, n_kv_out=after, n_free_out=left, err=err)
        side.wait_stream(here)
        with torch.cuda.stream(side):
            k.copy_(x[0])
        v.copy_(x[1])
        here.wait_stream(side)
        L.kv_store(pages, k, v, cell, err=err)
        out.zero_()
        plan.set_device(start, after, lists.table, 41)
        plan.run(q, pages, out)
        small.copy_(out)
        plan.set_device(two, after, lists.table, 3)
        plan.run(q, pages, small)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    T = sum(add)
    for seed in range(3):
        for t in (*x, q):
            t.copy_(torch.from_numpy(np.random.default_rng(seed).normal(size=tuple(t.shape))))
        n_new.zero_()
        g.replay()
        assert plan.error() == 0 and int(err) == 0 and start.tolist() == [0, 41, 42, 45] and after.tolist() == [700, 90, 33]
        for t, val in zip(x, (kval, vval)):
            t = t.double().cpu().numpy()[:T]
            val[np.array(cell.tolist()[:T])] = F.values(*F.quantise(t)) if cdt == "f4" else t
        verify(out.double().cpu().numpy(), q, kval, vval, tables, add, [700, 90, 33], page, 0, 0, act)
        verify(small.double().cpu().numpy()[:4], q[:4], kval, vval, tables, [0, 1, 3], [700, 90, 33], page, 0, 0, act)
        assert torch.equal(small[4:], out[4:])
