"""The operators over a paged cache and the batched sampler on a machine without a GPU: what their
entry points refuse (before anything touches a device), and the host plan of the attention (every row
meets every key it may see exactly once, within the buffers a plan allocates)."""
import ctypes as C
import os

import numpy as np
import pytest


@pytest.fixture(scope="module")
def B():
    from transformer_decode_kv_gb300 import binding, build
    if not os.path.exists(binding.LIB_PATH):
        build.build()
    return binding


PTR = 0x10000                       # an aligned address that is never read


def desc(B, **kw):
    d = B.KvPagesDesc()
    base = dict(type=B.F16, n_head_kv=2, head_dim=64, page_size=16, n_pages=8, k=PTR, v=PTR,
                stride_page=2048, stride_cell=128, stride_head=64)
    base.update(kw)
    for n, v in base.items():
        setattr(d, n, v)
    return d


BAD_KV = [dict(type=0), dict(type=8), dict(head_dim=96), dict(head_dim=0), dict(n_head_kv=0),
          dict(page_size=0), dict(n_pages=0), dict(page_size=1 << 16, n_pages=1 << 15), dict(k=None),
          dict(v=None), dict(k=PTR + 8), dict(stride_cell=-128), dict(stride_cell=132),
          dict(stride_head=32), dict(stride_page=1024), dict(stride_cell=0),
          dict(type=100), dict(type=100, k_scale=PTR, v_scale=PTR),
          dict(type=100, k_scale=PTR + 2, v_scale=PTR, sstride_page=32, sstride_cell=2, sstride_head=1)]


@pytest.mark.parametrize("bad", BAD_KV)
def test_bad_caches_are_refused(B, bad):
    L = B.lib()
    d = desc(B, **bad)
    for fn in (L.llm_kv_store, L.llm_kv_load):
        assert fn(C.byref(d), B.F16, PTR, PTR, 128, 64, PTR, 4, None, None) == -1
        assert L.llm_op_last_error()


@pytest.mark.parametrize("args", [
    dict(type=B_) for B_ in (8, 100, 7)] + [
    dict(k=None), dict(v=None), dict(cell=None), dict(n=-1), dict(k=PTR + 2), dict(cell=PTR + 1),
    dict(s_tok=-128), dict(s_tok=129), dict(s_head=3)])
def test_bad_rows_are_refused(B, args):
    L = B.lib()
    a = dict(type=1, k=PTR, v=PTR, s_tok=128, s_head=64, cell=PTR, n=4)
    a.update(args)
    d = desc(B)
    for fn in (L.llm_kv_store, L.llm_kv_load):
        assert fn(C.byref(d), a["type"], a["k"], a["v"], a["s_tok"], a["s_head"], a["cell"], a["n"],
                  None, None) == -1


def test_rows_may_repeat_as_inputs_but_not_as_outputs(B):
    d = desc(B)
    # a store may read one row for every token; a load may not write them to one place
    assert B.lib().llm_kv_load(C.byref(d), 1, PTR, PTR, 0, 64, PTR, 4, None, None) == -1
    assert B.lib().llm_kv_store(C.byref(d), 1, PTR, PTR, 0, 64, PTR, 4, None, None) != 0   # no device


def test_zero_rows_are_a_no_op(B):
    d = desc(B)
    assert B.lib().llm_kv_store(C.byref(d), 1, None, None, 0, 0, None, 0, None, None) == 0
    assert B.lib().llm_kv_load(C.byref(d), 1, None, None, 0, 0, None, 0, None, None) == 0
    a = B.SampleRowsArgs(type=0, n_rows=0, n_vocab=10)
    assert B.lib().llm_sample_rows(C.byref(a), None) == 0


GOOD_SHAPE = dict(type=1, n_head=8, scale=0.0, window=0, n_sink=0, max_tok=64, max_seq=8, max_table=64)


@pytest.mark.parametrize("bad", [
    dict(type=2), dict(type=8), dict(n_head=0), dict(n_head=7), dict(n_head=2048), dict(scale=float("nan")),
    dict(scale=float("inf")), dict(window=-1), dict(n_sink=-1), dict(max_tok=0), dict(max_seq=0),
    dict(max_table=0), dict(max_tok=1 << 25), dict(max_seq=1 << 21)])
def test_bad_attention_shapes_are_refused(B, bad):
    s = B.AttnShape(**{**GOOD_SHAPE, **bad})
    d = desc(B)
    assert not B.lib().llm_attn_plan_init(C.byref(s), C.byref(d))
    assert B.lib().llm_debug_attn_units(C.byref(s), C.byref(d), 152, 0, 0, None, None, None, 0, None, None, None) == -1


def test_null_arguments_are_refused(B):
    L = B.lib()
    d = desc(B)
    assert not L.llm_attn_plan_init(None, C.byref(d))
    s = B.AttnShape(**GOOD_SHAPE)
    assert not L.llm_attn_plan_init(C.byref(s), None)
    assert L.llm_attn_plan_set(None, 0, None, None, None, 0, None) == -1
    assert L.llm_attn_run(None, PTR, 1, 1, C.byref(d), PTR, 1, 1, None) == -1
    assert L.llm_attn_plan_form(None) == -1
    assert L.llm_attn_plan_error(None) == 0
    L.llm_attn_plan_free(None)
    assert L.llm_kv_store(None, 1, PTR, PTR, 128, 64, PTR, 4, None, None) == -1
    assert L.llm_sample_rows(None, None) == -1


@pytest.mark.parametrize("bad", [
    dict(type=8), dict(type=100), dict(n_rows=-1), dict(n_vocab=0), dict(n_vocab=400000), dict(logits=None),
    dict(token=None), dict(ld=-1), dict(temperature=PTR), dict(repeat_penalty=PTR),
    dict(repeat_penalty=PTR, penalty_start=PTR, n_penalty_token=3),
    dict(repeat_penalty=PTR, penalty_start=PTR, penalty_token=PTR, n_penalty_token=-1),
    dict(logits=PTR + 2)])
def test_bad_sampler_arguments_are_refused(B, bad):
    a = B.SampleRowsArgs(**{**dict(type=0, n_rows=2, n_vocab=100, logits=PTR, ld=100, token=PTR), **bad})
    assert B.lib().llm_sample_rows(C.byref(a), None) == -1
    assert B.lib().llm_op_last_error()


def units_of(B, shape, kv, n_new, n_kv, n_sm=152, tc=0):
    n_new, n_kv = np.asarray(n_new, np.int32), np.asarray(n_kv, np.int32)
    p = lambda a: a.ctypes.data_as(C.POINTER(C.c_int32))
    n1, caps = C.c_int64(), (C.c_int64 * 7)()
    args = (C.byref(shape), C.byref(kv), n_sm, tc, len(n_new), p(n_new), p(n_kv))
    first = np.zeros((2, 2 * n_sm + 1), np.int32)
    n = B.lib().llm_debug_attn_units(*args, None, 0, C.byref(n1), None, caps)
    assert n >= 0, B.lib().llm_op_last_error()
    out = np.zeros((max(n, 1), 16), np.int32)
    assert B.lib().llm_debug_attn_units(*args, p(out), n, C.byref(n1), p(first), caps) == n
    return out[:n], n1.value, first, list(caps)


@pytest.mark.parametrize("seed", range(60))
def test_plan_covers_every_visible_key_once(B, seed):
    rng = np.random.default_rng(seed)
    Hkv, G = int(rng.choice([1, 2, 8])), int(rng.choice([1, 3, 4, 8]))
    window = int(rng.choice([0, 0, 1, 7, 64, 300]))
    n_sink = int(rng.choice([0, 1, 4, 40]))
    n_seq = int(rng.integers(0, 7))
    n_new = rng.integers(0, 90, n_seq) if seed % 5 else rng.integers(0, 2, n_seq)
    n_kv = np.maximum(0, n_new + rng.integers(-20, 700, n_seq))
    if n_seq and seed % 3 == 0:
        n_kv[0] += 20000                                   # one long sequence
    tok, page = max(1, int(n_new.sum())), 16
    n_sm = [152, 3, 1][seed % 3]
    shape = B.AttnShape(type=1, n_head=Hkv * G, scale=0.0, window=window, n_sink=n_sink, max_tok=tok,
                        max_seq=max(1, n_seq), max_table=max(1, int((n_kv // page + 1).sum())))
    kv = desc(B, n_head_kv=Hkv, n_pages=4096, page_size=page)
    units, n1, first, caps = units_of(B, shape, kv, n_new, n_kv, n_sm=n_sm, tc=seed % 2)
    seen = {}                                              # (sequence, token, query head) -> keys
    starts = np.concatenate([[0], np.cumsum(n_new)])
    tabs = np.concatenate([[0], np.cumsum(-(-n_kv // page))])
    parts, tickets, chunks = [set(), set()], {}, {}
    for i, u in enumerate(units):
        tok0, row0, n_row, p0, tab, ns, lo, v0, v1, n_chunk, chunk, part, ticket, head = u[:14]
        s = [j for j in range(n_seq) if starts[j] == tok0 and n_new[j] > 0][0]
        assert tab == tabs[s] and p0 == n_kv[s] - n_new[s] and 0 <= head < Hkv
        assert 1 <= n_row <= (16 if i < n1 else 256) and 0 <= v0 <= v1 and 0 <= chunk < n_chunk
        tile = (i >= n1, tok0, row0, head)
        chunks.setdefault(tile, []).append((chunk, n_chunk))
        if n_chunk > 1:
            assert part + chunk not in parts[i >= n1]
            parts[i >= n1].add(part + chunk)
            assert i >= n1 or tickets.setdefault(ticket, tile) == tile
        keys = [v if v < ns else v - ns + lo for v in range(v0, v1)]
        assert all(0 <= k < n_kv[s] for k in keys)
        for r in range(row0, row0 + n_row):
            t, h = divmod(r, G)
            p = p0 + t
            got = seen.setdefault((s, t, head * G + h), [])
            got += [k for k in keys if k <= p and (window == 0 or k > p - window or k < n_sink)]
    for s in range(n_seq):
        for t in range(n_new[s]):
            p = n_kv[s] - n_new[s] + t
            want = [k for k in range(p + 1) if window == 0 or k > p - window or k < n_sink]
            for h in range(Hkv * G):
                assert sorted(seen[(s, t, h)]) == want
    for c in chunks.values():
        assert sorted(x[0] for x in c) == list(range(c[0][1]))
    # the CTAs' ranges are the units, each once and in order
    ctas = [2 * n_sm, n_sm]
    for f, n in ((0, n1), (1, len(units) - n1)):
        if n:
            r = first[f][:ctas[f] + 1]
            assert r[0] == 0 and r[-1] == n and (np.diff(r) >= 0).all()
    # and everything fits the plan's buffers
    assert n1 <= caps[0] and len(units) - n1 <= caps[1]
    assert ctas[0] <= caps[2] and (len(units) == n1 or ctas[1] <= caps[3])
    assert all(0 <= t < caps[4] for t in tickets)
    assert max(parts[0], default=-1) < caps[5] and max(parts[1], default=-1) < max(caps[6], 1)


@pytest.mark.parametrize("n_kv", [[300000], [32768 - 1571 * i for i in range(16)], [9, 70000, 5, 2000]])
def test_plan_gives_every_cta_an_even_share(B, n_kv):
    shape = B.AttnShape(**{**GOOD_SHAPE, "max_table": 1 << 20, "max_seq": 64})
    kv = desc(B, n_pages=1 << 16)
    units, _, first, _ = units_of(B, shape, kv, [1] * len(n_kv), n_kv)
    load = [(units[a:b, 8] - units[a:b, 7]).sum() for a, b in zip(first[0][:-1], first[0][1:])]
    fair = sum(n_kv) * 2 / len(load)
    # a share is even up to two blocks (of 192 keys) for the units' own costs and one for rounding
    assert max(load) <= fair + 3 * 192


@pytest.mark.parametrize("n_new,n_kv", [([1] * 9, [1] * 9), ([65], [65]), ([-1], [4]), ([1], [-1]),
                                        ([1], [2 ** 31 - 1]), ([1], [16 * 64 + 1])])
def test_steps_past_the_shape_are_refused(B, n_new, n_kv):
    shape, kv = B.AttnShape(**GOOD_SHAPE), desc(B)
    a, b = np.asarray(n_new, np.int32), np.asarray(n_kv, np.int32)
    p = lambda x: x.ctypes.data_as(C.POINTER(C.c_int32))
    assert B.lib().llm_debug_attn_units(C.byref(shape), C.byref(kv), 152, 0, len(a), p(a), p(b), None, 0,
                                        None, None, None) == -1


def test_rows_past_32_bits_are_refused(B):
    """Rows (token, query head) are numbered in 32 bits: 2^24 tokens of 128 heads or more are too many."""
    L = B.lib()
    n = np.asarray([1], np.int32).ctypes.data_as(C.POINTER(C.c_int32))
    for heads, tok, ok in ((128, 1 << 24, False), (127, 1 << 24, True), (1024, 1 << 21, False), (1024, (1 << 21) - 1, True)):
        kv = desc(B, n_head_kv=1)
        s = B.AttnShape(**{**GOOD_SHAPE, "n_head": heads, "max_tok": tok})
        r = L.llm_debug_attn_units(C.byref(s), C.byref(kv), 152, 0, 1, n, n, None, 0, None, None, None)
        assert (r > 0) == ok
        if not ok:
            assert r == -1 and b"2^31" in L.llm_op_last_error()
            assert not L.llm_attn_plan_init(C.byref(s), C.byref(kv))


def test_sequences_of_almost_2_to_31_keys_are_refused(B):
    """Key numbers run a few blocks past the end of a sequence: they must not wrap."""
    shape, kv = B.AttnShape(**GOOD_SHAPE), desc(B, n_pages=2, page_size=1 << 29)
    p = lambda x: np.asarray([x], np.int32).ctypes.data_as(C.POINTER(C.c_int32))
    for n, ok in ((2 ** 31 - 513, True), (2 ** 31 - 512, False), (2 ** 31 - 128, False), (2 ** 31 - 2, False)):
        r = B.lib().llm_debug_attn_units(C.byref(shape), C.byref(kv), 152, 1, 1, p(64), p(n), None, 0, None, None, None)
        assert (r > 0) == ok


def test_host_integers_are_not_wrapped(B):
    """A page number or length that int32 does not hold must not become another one."""
    plan = B.AttnPlan.__new__(B.AttnPlan)                  # (no device is reached: the arguments are refused first)
    plan.ptr, plan._captured_rows, plan.device = None, None, None
    big = np.array([2 ** 32 + 1])
    for n_new, n_kv, pages in ((big, [1], [[0]]), ([1], big, [[0]]), ([1], [1], big[None]), ([1], [1], [[-2 ** 31 - 1]])):
        with pytest.raises(ValueError, match="int32"):
            plan.set(n_new, n_kv, pages, stream=0)
    for n_new, n_kv, pages in (([1.0], [1], [[0]]), ([1], [1], [[0.5]]), ([1], ["1"], [[0]])):
        with pytest.raises(TypeError, match="integers"):
            plan.set(n_new, n_kv, pages, stream=0)
    with pytest.raises(B.LlmError, match="NULL plan"):     # good ones reach the library
        plan.set(np.array([1], np.int64), [1], np.array([[3]], np.uint8), stream=0)
