"""Page tables made on the GPU (pages_extend, pages_trim) against a token-by-token form on the host: counts from
none to thousands, page sizes, in place and apart, what does not fit, bad pages, capture, another stream."""
import numpy as np
import pytest
import torch

from tests import ops4_common as F

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    import transformer_decode_kv_gb300 as L
    L.lib()
    return L


def ints(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32)).cuda()


class Lists:
    """n_kv rows per sequence in pages of a random order, `spare` pages left on the stack."""

    def __init__(self, L, n_kv, page, ld, spare, seed=0, room=5):
        rng = np.random.default_rng(seed)
        held = [-(-n // page) for n in n_kv]
        self.n_pages, self.page, self.n_kv = sum(held) + spare + 1, page, list(n_kv)
        perm = rng.permutation(self.n_pages - 1).tolist()
        self.table = np.full((len(n_kv), ld), -9, np.int32)
        for i, m in enumerate(held):
            self.table[i, :m] = [perm.pop() for _ in range(m)]
        self.stack = perm
        self.d_table, self.d_kv = ints(self.table), ints(n_kv)
        self.d_free, self.d_n = ints(self.stack + [-5] * room), ints([len(self.stack)])
        self.max_free = len(self.stack) + room
        self.lists = L.SeqPages(self.d_table, self.d_kv, self.d_free, self.d_n, page, self.n_pages)

    def unchanged(self):
        return (np.array_equal(self.d_table.cpu(), self.table) and self.d_kv.tolist() == self.n_kv and
                self.d_free.tolist()[:len(self.stack)] == self.stack and self.d_n.tolist() == [len(self.stack)])


def extend(L, ls, n_new, max_tok, apart=False, stream=None):
    cell, pos, start = (torch.full((n,), 99, dtype=torch.int32, device="cuda") for n in (max_tok, max_tok, len(n_new) + 1))
    err = ints([0])
    outs = {}
    if apart:
        outs = dict(n_kv_out=torch.full_like(ls.d_kv, 99), n_free_out=ints([99]))
    L.pages_extend(ls.lists, ints(n_new), cell, pos, start, err=err, stream=stream, **outs)
    torch.cuda.synchronize()
    return cell.tolist(), pos.tolist(), start.tolist(), int(err), outs


@pytest.mark.parametrize("apart", [False, True])
@pytest.mark.parametrize("page", [1, 3, 16, 64, 1000])
@pytest.mark.parametrize("n_seq,top,room", [(1, 1, 0), (1, 700, 3), (2, 40, 0), (31, 9, 1), (33, 200, 40), (1024, 3, 0), (1025, 4, 7),
                                            (2500, 2, 0)])
def test_extend(L, n_seq, top, room, page, apart):
    rng = np.random.default_rng(n_seq + page)
    n_kv = rng.integers(0, 3 * page + 2, n_seq).tolist()
    n_new = rng.integers(0, top + 1, n_seq).tolist()
    n_new[-1] = top
    ls = Lists(L, n_kv, page, 4 + -(-top // page), sum(-(-(a + b) // page) - -(-a // page) for a, b in zip(n_kv, n_new)) + 2)
    tok = sum(n_new) + room
    table, cell, pos, start, after, stack = F.extend(ls.table, n_kv, n_new, ls.stack, page, tok)
    got = extend(L, ls, n_new, tok, apart)
    assert got[3] == 0 and got[0] == cell and got[1] == pos and got[2] == start
    assert np.array_equal(ls.d_table.cpu(), table) and ls.d_free.tolist()[:len(ls.stack)] == ls.stack
    if apart:
        assert got[4]["n_kv_out"].tolist() == after and got[4]["n_free_out"].tolist() == [len(stack)]
        assert ls.d_kv.tolist() == n_kv and ls.d_n.tolist() == [len(ls.stack)]
    else:
        assert ls.d_kv.tolist() == after and ls.d_n.tolist() == [len(stack)]


def test_extend_of_many_tokens(L):
    """More tokens than one CTA takes at a time, in few and in many sequences."""
    for n_seq, top in ((3, 12000), (300, 200), (1500, 30)):
        rng = np.random.default_rng(n_seq)
        n_kv, n_new = rng.integers(0, 100, n_seq).tolist(), rng.integers(0, top, n_seq).tolist()
        ls = Lists(L, n_kv, 16, 1000, sum(n_new) // 16 + 2 * n_seq)
        table, cell, pos, start, after, stack = F.extend(ls.table, n_kv, n_new, ls.stack, 16, sum(n_new) + 9)
        got = extend(L, ls, n_new, sum(n_new) + 9)
        assert got[3] == 0 and got[0] == cell and got[1] == pos and got[2] == start
        assert np.array_equal(ls.d_table.cpu(), table) and ls.d_kv.tolist() == after and ls.d_n.tolist() == [len(stack)]


def test_extend_without_sequences_or_tokens(L):
    ls = Lists(L, [], 16, 4, 3)
    assert extend(L, ls, [], 5)[:4] == ([-1] * 5, [-1] * 5, [0], 0) and ls.unchanged()
    ls = Lists(L, [5, 0], 16, 4, 3)
    assert extend(L, ls, [0, 0], 0)[:4] == ([], [], [0, 0, 0], 0) and ls.unchanged()
    ls = Lists(L, [16, 32], 16, 2, 0)                           # an empty stack, no page needed
    assert extend(L, ls, [0, 0], 2)[3] == 0 and ls.unchanged()


BAD = [dict(n_new=[1, 20, 1]),                                  # more pages than are free
       dict(n_new=[1, -1, 1]), dict(n_new=[30, 0, 0]),          # a negative count; more rows than the table row holds
       dict(n_new=[2, 2, 2], max_tok=5), dict(n_new=[2 ** 31 - 1, 0, 0]), dict(n_new=[2 ** 31 - 1] * 3),
       dict(n_kv=[-1, 3, 4]), dict(n_kv=[2 ** 31 - 1, 3, 4]), dict(n_free=-1), dict(n_free=100)]


@pytest.mark.parametrize("apart", [False, True])
@pytest.mark.parametrize("bad", BAD)
def test_a_step_that_does_not_fit_changes_nothing(L, bad, apart):
    ls = Lists(L, [10, 3, 16], 8, 4, 2)
    if "n_kv" in bad:
        ls.n_kv = bad["n_kv"]
        ls.d_kv.copy_(ints(ls.n_kv))
    n_free = bad.get("n_free", 2)
    ls.d_n.fill_(n_free)
    n_new = bad.get("n_new", [1, 1, 1])
    cell, pos, start, err, outs = extend(L, ls, n_new, bad.get("max_tok", 64), apart)
    assert err == 32 and set(cell) == {-1} and set(pos) == {-1} and start == [0] * 4
    assert ls.d_n.tolist() == [n_free]
    ls.d_n.fill_(2)
    assert ls.unchanged()
    if apart:
        assert outs["n_kv_out"].tolist() == ls.n_kv and outs["n_free_out"].tolist() == [n_free]


def test_bad_pages_give_their_tokens_no_cell(L):
    ls = Lists(L, [10, 8], 8, 4, 3)
    ls.d_table[0, 1] = 1000                                     # the first sequence's last page
    ls.d_free[2] = -4                                           # the page that it takes next
    cell, pos, start, err, _ = extend(L, ls, [8, 2], 12)
    want = ls.stack[1] * 8
    assert err == 1 and start == [0, 8, 10] and pos == [10, 11, 12, 13, 14, 15, 16, 17, 8, 9, -1, -1]
    assert cell == [-1] * 6 + [-1, -1] + [want, want + 1] + [-1] * 2


@pytest.mark.parametrize("apart", [False, True])
@pytest.mark.parametrize("n_seq,page", [(1, 16), (40, 1), (40, 7), (1030, 16), (2100, 3)])
def test_trim(L, n_seq, page, apart):
    rng = np.random.default_rng(n_seq)
    n_kv = rng.integers(0, 5 * page, n_seq).tolist()
    keep = [int(k) for k in rng.integers(-1, np.array(n_kv) + 1)]
    keep[0] = 0
    gone = []
    for i, (a, k) in enumerate(zip(n_kv, keep)):
        if k >= 0:
            gone += [(i, j) for j in range(-(-k // page), -(-a // page))]
    ls = Lists(L, n_kv, page, 6, 3, room=len(gone))
    outs = dict(n_kv_out=torch.full_like(ls.d_kv, 99), n_free_out=ints([99])) if apart else {}
    err = ints([0])
    L.pages_trim(ls.lists, ints(keep), err=err, **outs)
    stack = ls.stack + [int(ls.table[i, j]) for i, j in gone]
    left = [a if k < 0 else k for a, k in zip(n_kv, keep)]
    assert int(err) == 0 and ls.d_free.tolist() == stack and np.array_equal(ls.d_table.cpu(), ls.table)
    assert (outs["n_kv_out"] if apart else ls.d_kv).tolist() == left
    assert (outs["n_free_out"] if apart else ls.d_n).tolist() == [len(stack)]
    if apart:
        assert ls.d_kv.tolist() == n_kv and ls.d_n.tolist() == [3]


@pytest.mark.parametrize("bad", [dict(keep=[11, 0, 0]), dict(room=1), dict(n_kv=[-2, 3, 4]), dict(n_kv=[33, 3, 4]), dict(n_free=-1),
                                 dict(n_free=40)])
def test_a_trim_that_does_not_fit_changes_nothing(L, bad):
    ls = Lists(L, [10, 3, 16], 8, 4, 2, room=bad.get("room", 5))
    if "n_kv" in bad:
        ls.n_kv = bad["n_kv"]
        ls.d_kv.copy_(ints(ls.n_kv))
    ls.d_n.fill_(bad.get("n_free", 2))
    err = ints([0])
    L.pages_trim(ls.lists, ints(bad.get("keep", [0, 0, -1])), err=err)
    assert int(err) == 32 and ls.d_n.tolist() == [bad.get("n_free", 2)]
    ls.d_n.fill_(2)
    assert ls.unchanged() and ls.d_free.tolist()[2:] == [-5] * (ls.max_free - 2)


def test_pages_come_back_and_go_out_again_in_a_graph(L):
    """Steps of random lengths, sequences ending and drafts taken back, replayed on another stream: no page is in two
    places, and every token has the cell that the host's books say."""
    rng = np.random.default_rng(7)
    n_seq, page, tok = 20, 4, 90
    ls = Lists(L, rng.integers(0, 9, n_seq).tolist(), page, 8, 60, room=200)
    n_new, keep = ints([0] * n_seq), ints([-1] * n_seq)
    cell, pos, start, err = ints([0] * tok), ints([0] * tok), ints([0] * (n_seq + 1)), ints([0])
    L.pages_extend(ls.lists, n_new, cell, pos, start, err=err)
    L.pages_trim(ls.lists, keep, err=err)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        L.pages_extend(ls.lists, n_new, cell, pos, start, err=err)
        L.pages_trim(ls.lists, keep, err=err)
    st = torch.cuda.Stream()
    table, kv, stack = ls.table, list(ls.n_kv), list(ls.stack)
    for step in range(40):
        add = [int(min(rng.integers(0, 5), 8 * page - n)) for n in kv]
        held = [n + a for n, a in zip(kv, add)]
        cut = [0 if rng.random() < 0.1 else int(rng.integers(0, h + 1)) if rng.random() < 0.2 else -1 for h in held]
        need = sum(-(-h // page) - -(-n // page) for h, n in zip(held, kv))
        n_new.copy_(ints(add)); keep.copy_(ints(cut))
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            g.replay()
        st.synchronize()
        if need > len(stack):                                  # the extension is refused, the cuts may be too
            assert int(err) & 32
            break
        table, c, p, s, after, stack = F.extend(table, kv, add, stack, page, tok)
        for i, k in enumerate(cut):
            if k >= 0:
                stack += [int(table[i, j]) for j in range(-(-k // page), -(-after[i] // page))]
                after[i] = k
        assert cell.tolist() == c and pos.tolist() == p and start.tolist() == s
        assert ls.d_kv.tolist() == after and ls.d_n.tolist() == [len(stack)] and ls.d_free.tolist()[:len(stack)] == stack
        kv = after
        live = [int(table[i, j]) for i in range(n_seq) for j in range(-(-kv[i] // page))]
        assert len(set(live + stack)) == len(live) + len(stack) == ls.n_pages - 1
    assert step > 5


def test_bad_arguments_are_refused(L):
    ls = Lists(L, [10, 3], 8, 4, 2)
    ok = dict(n_new=ints([1, 1]), cell=ints([0] * 4), pos=ints([0] * 4), start=ints([0] * 3))
    for bad in (dict(n_new=ints([1])), dict(pos=ints([0] * 3)), dict(start=ints([0] * 2)), dict(cell=torch.zeros(4, device="cuda")),
                dict(n_kv_out=ints([0])), dict(n_free_out=ints([0, 0])), dict(cell=ints([0] * 8)[::2])):
        with pytest.raises(ValueError):
            L.pages_extend(ls.lists, **{**ok, **bad})
    with pytest.raises(L.LlmError, match="not device memory"):
        L.pages_extend(ls.lists, **{**ok, "pos": torch.zeros(4, dtype=torch.int32)})
    with pytest.raises(L.LlmError, match="cells"):
        L.pages_extend(L.SeqPages(ls.d_table, ls.d_kv, ls.d_free, ls.d_n, 1 << 16, 1 << 15), **ok)
    assert ls.unchanged()


def test_bad_pages_stay_in_the_lists(L):
    """A step over a bad page of the stack is made all the same: the page is entered, lengths and stack advance, and a trim puts
    it back as it is."""
    ls = Lists(L, [10, 8], 8, 4, 3)
    ls.d_free[2] = -4                                           # taken by the first sequence
    ls.d_free[1] = ls.n_pages                                   # by the second
    cell, pos, start, err, _ = extend(L, ls, [8, 2], 12)
    assert err == 1 and start == [0, 8, 10] and cell[6:] == [-1] * 6 and min(cell[:6]) >= 0 and pos[:10] == [*range(10, 18), 8, 9]
    assert ls.d_table[0].tolist() == [*ls.table[0, :2], -4, -9] and ls.d_table[1].tolist() == [ls.table[1, 0], ls.n_pages, -9, -9]
    assert ls.d_kv.tolist() == [18, 10] and ls.d_n.tolist() == [1]
    e = ints([0])
    L.pages_trim(ls.lists, ints([10, 8]), err=e)
    assert int(e) == 1 and ls.d_kv.tolist() == [10, 8] and ls.d_n.tolist() == [3]
    assert ls.d_free.tolist()[:3] == [ls.stack[0], -4, ls.n_pages]


@pytest.mark.parametrize("n_seq,page", [(5000, 1), (300, 4)])
def test_trim_of_many_pages(L, n_seq, page):
    """A stack of more places than one cluster of four takes at a time, in few sequences and in many."""
    rng = np.random.default_rng(n_seq)
    n_kv = rng.integers(0, 80 * page if n_seq < 1000 else 6, n_seq).tolist()
    keep = [int(k) for k in rng.integers(-1, np.array(n_kv) + 1)]
    gone = [(i, j) for i, (a, k) in enumerate(zip(n_kv, keep)) if k >= 0 for j in range(-(-k // page), -(-a // page))]
    ls = Lists(L, n_kv, page, 80, 9000, room=len(gone) + 7)
    assert ls.max_free > 8192 and len(gone) > 4096
    err = ints([0])
    L.pages_trim(ls.lists, ints(keep), err=err)
    stack = ls.stack + [int(ls.table[i, j]) for i, j in gone]
    assert int(err) == 0 and ls.d_free.tolist() == stack + [-5] * 7 and np.array_equal(ls.d_table.cpu(), ls.table)
    assert ls.d_kv.tolist() == [a if k < 0 else k for a, k in zip(n_kv, keep)] and ls.d_n.tolist() == [len(stack)]
