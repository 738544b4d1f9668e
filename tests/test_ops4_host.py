"""The 4-bit cache, the page lists and plans set from the device on a machine without a GPU: what the entry points
refuse before anything touches a device."""
import ctypes as C
import os

import pytest
import torch


@pytest.fixture(scope="module")
def B():
    from transformer_decode_kv_gb300 import binding, build
    if not os.path.exists(binding.LIB_PATH):
        build.build()
    return binding


PTR = 0x10000                       # an aligned address that is never read


def desc(B, **kw):
    """A 4-bit cache [8 pages][2 heads][16 cells] of rows of 128 values."""
    d = B.KvPagesDesc()
    base = dict(type=B.F4_E2M1, n_head_kv=2, head_dim=128, page_size=16, n_pages=8, k=PTR, v=PTR, stride_page=2048,
                stride_cell=64, stride_head=1024, k_scale=PTR, v_scale=PTR, sstride_page=32, sstride_cell=1,
                sstride_head=16, k_block=PTR, v_block=PTR, bstride_page=256, bstride_cell=8, bstride_head=128)
    base.update(kw)
    for n, v in base.items():
        setattr(d, n, v)
    return d


@pytest.mark.parametrize("bad,why", [
    (dict(k=PTR + 8), "16-byte"), (dict(v=None), "NULL"), (dict(stride_cell=72), "strides"), (dict(stride_cell=48), "strides"),
    (dict(stride_head=512), "strides"), (dict(k_scale=None), "scales"), (dict(v_scale=PTR + 2), "4-byte"),
    (dict(sstride_cell=0), "scale strides"), (dict(k_block=None), "block scales"), (dict(v_block=None), "block scales"),
    (dict(k_block=PTR + 4), "block scales"), (dict(bstride_cell=4), "block-scale"), (dict(bstride_cell=12), "block-scale"),
    (dict(bstride_cell=-8), "block-scale"), (dict(bstride_head=64), "block-scale"), (dict(bstride_page=1 << 50), "block-scale"),
    (dict(head_dim=96), "head_dim"), (dict(type=102), "paged cache")])
def test_bad_caches_are_refused(B, bad, why):
    L, d = B.lib(), desc(B, **bad)
    for fn in (L.llm_kv_store, L.llm_kv_load):
        assert fn(C.byref(d), B.F16, PTR, PTR, 256, 128, PTR, 4, None, None) == -1
        assert why in L.llm_op_last_error().decode()


def test_good_caches_reach_the_device_check(B):
    L = B.lib()
    one = dict(n_pages=1, stride_page=-1, sstride_page=-1, bstride_page=-1)      # (a stride that is never used)
    for kw in ({}, one, dict(head_dim=32, stride_page=512, stride_cell=16, stride_head=256, k_block=PTR + 2, bstride_cell=2,
                             bstride_head=32, bstride_page=64)):
        d = desc(B, **kw)
        r = L.llm_kv_store(C.byref(d), B.F16, PTR, PTR, 256, 128, PTR, 4, None, None)
        assert r != 0 and not any(w in L.llm_op_last_error() for w in (b"stride", b"boundar", b"scales")), L.llm_op_last_error()


def test_activations_of_a_4_bit_cache(B):
    L, d = B.lib(), desc(B)
    one = (C.c_int32 * 1)(1)
    for t, ok in ((B.F32, True), (B.F16, True), (B.BF16, True), (B.F8_E4M3, False), (B.F4_E2M1, False), (B.Q8_0, False)):
        s = B.AttnShape(type=t, n_head=8, scale=0.0, window=0, n_sink=0, max_tok=64, max_seq=8, max_table=64)
        r = L.llm_debug_attn_units(C.byref(s), C.byref(d), 152, 1, 1, one, one, None, 0, None, None, None)
        assert (r > 0) == ok


def test_a_context_does_not_take_a_4_bit_cache(B):
    cp = B.lib().llm_cparams_default()
    cp.type_k = cp.type_v = B.F4_E2M1
    cp.flags = B.CTX_HOST_ONLY
    hp = B.HParams(2, 64, 2, 1, 32, 128, 100, 10000.0, 1e-5, 0)
    assert not B.lib().llm_ctx_init(C.byref(hp), C.byref(cp))


def test_python_checks_of_the_cache(B):
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)
    k, s, b = u8(4, 16, 2, 64), torch.zeros(4, 16, 2), u8(4, 16, 2, 8)
    d = B.KvPages(k, k, s, s, b, b)
    assert d.desc.type == B.F4_E2M1 and d.dim == 128 and d.desc.stride_cell == 128 and d.desc.bstride_cell == 16
    assert B.KvPages(k, k, s, s).desc.type == B.F8_E4M3          # without block scales: E4M3 codes
    assert B.KvPages(k, k, s, s, b.view(torch.float8_e4m3fn), b.view(torch.float8_e4m3fn)).desc.type == B.F4_E2M1
    for args in ((k, k, s, s, b, None), (k, k, None, None, b, b), (k, k, s, s, u8(4, 16, 2, 4), b),
                 (k, k, s, s, b, u8(4, 2, 16, 8).transpose(1, 2)), (k, k, s, s, u8(4, 16, 2, 16)[..., ::2], u8(4, 16, 2, 16)[..., ::2])):
        with pytest.raises(ValueError):
            B.KvPages(*args)
    with pytest.raises(TypeError):
        B.KvPages(k.half(), k.half(), s, s, b, b)


def lists(B, **kw):
    d = B.SeqPagesDesc()
    base = dict(n_seq=2, page_size=16, n_pages=8, ld_table=4, max_free=8, table=PTR, n_kv=PTR, free_pages=PTR, n_free=PTR)
    base.update(kw)
    for n, v in base.items():
        setattr(d, n, v)
    return d


@pytest.mark.parametrize("bad,why", [
    (dict(n_seq=-1), "n_seq"), (dict(n_seq=(1 << 20) + 1), "n_seq"), (dict(page_size=0), "page_size"), (dict(n_pages=0), "n_pages"),
    (dict(page_size=1 << 16, n_pages=1 << 15), "cells"), (dict(ld_table=-1), "ld_table"), (dict(max_free=-1), "max_free"),
    (dict(table=None), "NULL"), (dict(n_kv=None), "NULL"), (dict(free_pages=None), "NULL"), (dict(n_free=None), "NULL"),
    (dict(n_kv=PTR + 2), "aligned"), (dict(table=PTR + 1), "aligned")])
def test_bad_page_lists_are_refused(B, bad, why):
    L, d = B.lib(), lists(B, **bad)
    assert L.llm_pages_extend(C.byref(d), PTR, PTR, PTR, 4, PTR, PTR, PTR, None, None) == -1
    assert why in L.llm_op_last_error().decode()
    assert L.llm_pages_trim(C.byref(d), PTR, PTR, PTR, None, None) == -1
    assert why in L.llm_op_last_error().decode()


@pytest.mark.parametrize("args", [
    dict(n_new=None), dict(kv_out=None), dict(free_out=None), dict(max_tok=-1), dict(max_tok=(1 << 24) + 1), dict(cell=None),
    dict(pos=None), dict(start=None), dict(cell=PTR + 2), dict(start=PTR + 1), dict(err=PTR + 3)])
def test_bad_extensions_are_refused(B, args):
    a = dict(n_new=PTR, kv_out=PTR, free_out=PTR, max_tok=4, cell=PTR, pos=PTR, start=PTR, err=None)
    a.update(args)
    d = lists(B)
    assert B.lib().llm_pages_extend(C.byref(d), a["n_new"], a["kv_out"], a["free_out"], a["max_tok"], a["cell"], a["pos"], a["start"],
                                    a["err"], None) == -1
    assert B.lib().llm_pages_extend(None, PTR, PTR, PTR, 4, PTR, PTR, PTR, None, None) == -1
    assert B.lib().llm_pages_trim(None, PTR, PTR, PTR, None, None) == -1


def test_numbers_that_int32_does_not_hold_are_refused_not_wrapped(B):
    i = lambda *s: torch.zeros(s, dtype=torch.int32)
    for page_size, n_pages in ((2 ** 32 + 16, 8), (16, 2 ** 32 + 8), (16, -2 ** 32 + 8)):
        with pytest.raises(ValueError, match="int32"):
            B.SeqPages(i(2, 4), i(2), i(8), i(1), page_size, n_pages)
    plan = B.AttnPlan.__new__(B.AttnPlan)                  # (no device is reached: the arguments are refused first)
    plan.ptr, plan._captured_rows, plan.max_tok = None, None, 8
    with pytest.raises(ValueError, match="int32"):
        plan.set_device(i(3), i(2), i(2, 4), 2 ** 32 + 1, stream=0)
    with pytest.raises(B.LlmError, match="NULL plan"):     # good ones reach the library
        plan.set_device(i(3), i(2), i(2, 4), 1, stream=0)


def test_python_checks_of_the_page_lists(B):
    i = lambda *s: torch.zeros(s, dtype=torch.int32)
    ok = dict(table=i(2, 4), n_kv=i(2), free=i(8), n_free=i(1), page_size=16, n_pages=8)
    B.SeqPages(**ok)
    for bad in (dict(table=i(8)), dict(table=i(2, 8)[:, ::2]), dict(table=i(2, 4).long()), dict(n_kv=i(3)), dict(free=i(2, 4)),
                dict(n_free=i(2)), dict(n_free=i(1).float())):
        with pytest.raises(ValueError):
            B.SeqPages(**{**ok, **bad})


@pytest.fixture
def plan_without_a_device(B, monkeypatch):
    """A plan of 8 tokens over a library that accepts everything: what the binding itself keeps count of."""
    class Lib:
        llm_attn_plan_set = llm_attn_plan_set_device = staticmethod(lambda *a: 0)
    monkeypatch.setattr(B, "lib", lambda: Lib)
    plan = B.AttnPlan.__new__(B.AttnPlan)
    plan.ptr, plan.device, plan.dtype, plan.n_head, plan.head_dim = None, None, torch.float16, 2, 64
    plan.n_tok, plan.max_tok, plan._captured_rows, plan._run = 0, 8, None, lambda *a: 0
    plan.capturing = False
    plan._capturing = lambda: plan.capturing
    k = torch.zeros(4, 16, 2, 64, dtype=torch.float16)
    pages, rows = B.KvPages(k, k), lambda n: torch.zeros(n, 2, 64, dtype=torch.float16)
    i = lambda *s: torch.zeros(s, dtype=torch.int32)
    return plan, lambda n, m=None: plan.run(rows(n), pages, rows(n if m is None else m)), lambda: plan.set_device(i(3), i(2), i(2, 4), 1)


def test_a_captured_set_device_asks_every_later_run_for_max_tok_rows(plan_without_a_device):
    """Its replay may come after any other set, and leaves a step of up to max_tok tokens on the device."""
    plan, run, set_device = plan_without_a_device
    plan.capturing = True
    set_device()
    plan.capturing = False
    for _ in range(2):
        plan.set([1], [5], [[0]], stream=0)
        for n, m in ((1, 1), (7, 8), (8, 7)):
            with pytest.raises(ValueError, match="fewer rows"):
                run(n, m)
        run(8)
        plan.capturing = True                              # (a graph that is replayed behind the other)
        with pytest.raises(ValueError, match="fewer rows"):
            run(1)
        run(8)
        plan.capturing = False
        set_device()                                       # an eager one changes nothing about it


def test_an_eager_set_device_asks_the_runs_of_its_step_for_max_tok_rows(plan_without_a_device):
    plan, run, set_device = plan_without_a_device
    set_device()
    with pytest.raises(ValueError, match="fewer rows"):
        run(7)
    plan.set([1], [5], [[0]], stream=0)
    run(1)
    plan.capturing = True
    run(1)
    plan.capturing = False
    with pytest.raises(ValueError, match="captured run"):  # a graph holds a run whose rows would not do
        set_device()
