"""GPU parity of the context's F8_E4M3 KV cache and sliding window, and of its batched sampler.

  - F8_E4M3 rows, bit-exact: the float32 rows the library handed to its cache write (the debug capture)
    quantised by the table of E4M3 values give the library's codes and scales.
  - Layers one by one on the library's own inputs and cache (F8_E4M3), and whole runs (F16 cache with a window)
    against the oracle: 1e-4 for float32 weights, 2e-2 for BF16 weights, the bars of the other cache types.
    (A whole run over an F8_E4M3 cache is not compared with the oracle: a K or V value within float32 rounding of
    the middle between two codes lands a whole step, up to 1/14 of the row's largest value, apart.)
  - The same logits from replayed graphs, defragmented caches and caches without the cells out of sight.
"""
import numpy as np
import pytest

import oracle
import synthetic as S
from oracle.sampling import sample as sample_chain
from synthetic.configs import HParams, Workload
from tests import gpu_common as G
from tests import ops_common as O
from tests.test_gpu_sampler import PARAMS, US, near_edge

pytestmark = pytest.mark.gpu
F8 = 100
KEY = "tiny_f32_8seq"


def _f8_rows(ctx, il, which):
    """Dequantised cache rows [Hkv, n_ctx, hd] and their bytes (codes, scales)."""
    b = ctx.kv_cache(il, which)
    scale = np.ascontiguousarray(b[:, :, :4]).view(np.float32)[:, :, 0]
    code = b[:, :, 4:]
    return O.E4M3[code] * scale[..., None].astype(np.float64), code, scale


def _check_codes(ctx):
    hp, slots = ctx._hp, ctx.last_slots()
    for il in range(hp.n_layer):
        for which, name in ((0, "k_in"), (1, "v_in")):
            rows = ctx.debug_tensor(name, il).reshape(-1, hp.n_head_kv, hp.head_dim)
            T = len(rows)                                     # the last ubatch's
            code, s = O.quantise(rows.astype(np.float64))
            _, gc, gs = _f8_rows(ctx, il, which)
            at = slots[len(slots) - T:]
            assert np.array_equal(gc[:, at].transpose(1, 0, 2), code), (il, name)
            assert np.array_equal(gs[:, at].T, s.astype(np.float32)), (il, name)


def _check_layers(ctx, ow, mirror, rows, tol):
    """Rows of the last ubatch (in its own order, which split_equal may change)."""
    hp, slots = ctx._hp, ctx.last_slots()
    T = ctx.debug_tensor("l_out", 0).size // hp.n_embd
    at = slots[len(slots) - T:][rows]
    pos = mirror.cells.pos[at]
    vis = mirror.mask(pos, [np.nonzero(mirror.cells.seq[s])[0] for s in at], mirror.cells.n_kv())
    worst = 0.0
    for il in range(hp.n_layer):
        x_in, x_out = G.captured_rows(ctx, il, rows)
        e = G.layer_check(ow, hp, il, x_in, x_out, pos, at, vis, _f8_rows(ctx, il, 0)[0], _f8_rows(ctx, il, 1)[0], F8)
        worst = max(worst, e["delta"])
        assert e["delta"] <= tol, (il, e)
    print("layer update", worst)


@pytest.mark.parametrize("unified", [True, False])
@pytest.mark.parametrize("window,n_sink", [(0, 0), (37, 3)])
def test_tiny_f8_cache(unified, window, n_sink):
    w = S.WORKLOADS[KEY]
    kw = dict(n_seq_max=4, type_k=F8, type_v=F8, n_ubatch=64, kv_unified=unified)
    ctx, twin = G.library_ctx(KEY, **kw), G.library_ctx(KEY, **kw)
    mirror = oracle.OracleContext(w.hp, None, n_ctx=w.n_ctx, n_batch=w.n_batch, compute=False, **kw)
    ow = G.oracle_weights(KEY)
    ctx.debug_capture(True)
    for c in (ctx, twin):
        assert c.set_attn_window(window, n_sink) == 0
    mirror.window, mirror.n_sink = window, n_sink
    toks = np.concatenate([S.prompt_tokens(w.prompt_seed_of(s), 90, w.hp.n_vocab).numpy() for s in range(4)])
    seqs = [[s] for s in range(4) for _ in range(90)]

    def step(t, sq):
        fl = [0] * (len(t) - 1) + [1]
        for c in (ctx, twin):
            assert c.decode(t, seq_ids=sq, logits=fl) == 0, c.last_error()
        assert mirror.decode(t, seq_id=sq, n_seq_id=[1] * len(t), logits=fl) == 0
        for k, u in enumerate(mirror.last_ubatches):
            assert np.array_equal(ctx.ubatch_mask(k), u["mask"])
        _check_codes(ctx)
        g, t2 = ctx.get_logits_ith(-1), twin.get_logits_ith(-1)
        assert G.rel_err(g, t2.astype(np.float64)) <= 1e-5

    def check_last(rows):
        _check_layers(ctx, ow, mirror, rows, 1e-4)

    step(toks, seqs)
    n_last = len(mirror.last_ubatches[-1]["pos"])
    check_last([0, n_last // 2, n_last - 1])
    for i in range(3):
        step([i + 1, i + 2, i + 3, i + 4], [[0], [1], [2], [3]])
        check_last([0, 1, 2, 3])
    for c in (ctx, twin, mirror):                            # holes, refilled by later tokens
        c.seq_rm(1, 20, -1)
        c.seq_rm(2, 30, 60)
    step([5, 6, 7], [[1], [2], [0]])
    check_last([0, 1, 2])
    if unified:
        src = mirror.cells.defrag_order()
        before = [ctx.kv_cache(il, x).copy() for il in range(w.hp.n_layer) for x in (0, 1)]
        assert ctx.memory_update(True) == 1 and twin.memory_update(True) == 1 and mirror.memory_update(True)
        after = [ctx.kv_cache(il, x) for il in range(w.hp.n_layer) for x in (0, 1)]
        for b, a in zip(before, after):
            assert np.array_equal(a[:, src >= 0], b[:, src[src >= 0]])
        step([8, 9], [[2], [3]])
        check_last([0, 1])
    assert twin.perf()["n_graph_replays"] >= 1
    for c in (ctx, twin):
        c.free()


def test_tiny_window_f16_whole_run_and_removed_cells():
    w = S.WORKLOADS[KEY]
    ctx, ora, cut = G.library_ctx(KEY), G.oracle_ctx(KEY), G.library_ctx(KEY)
    for c in (ctx, cut):
        assert c.set_attn_window(50, 4) == 0
    ora.window, ora.n_sink = 50, 4
    toks, seqs, flags = G.prompt_batch(KEY)
    for c in (ctx, cut):
        assert c.decode(toks, seq_ids=seqs, logits=flags) == 0, c.last_error()
    assert ora.decode(toks, seq_id=seqs, n_seq_id=[1] * len(toks), logits=flags) == 0
    rows = [(s + 1) * w.n_prompt - 1 for s in range(w.n_seq)]
    rep = G.greedy_compare(ctx, ora, w.n_seq, rows, 8, 1e-4, {})
    print("window:", rep)
    assert rep["tokens_checked"] >= 20
    # a context that drops what no later token sees gives the same logits
    nxt = [int(cut.get_argmax_ith(i)) for i in rows]
    ref = G.library_ctx(KEY)
    assert ref.set_attn_window(50, 4) == 0
    assert ref.decode(toks, seq_ids=seqs, logits=flags) == 0
    for s in range(w.n_seq):
        assert cut.seq_rm(s, 4, w.n_prompt + 1 - 50)
    one = [[s] for s in range(w.n_seq)]
    for _ in range(3):
        assert cut.decode(nxt, seq_ids=one, logits=[1] * w.n_seq) == 0
        assert ref.decode(nxt, seq_ids=one, logits=[1] * w.n_seq) == 0
        for i in range(w.n_seq):
            assert G.rel_err(cut.get_logits_ith(i), ref.get_logits_ith(i).astype(np.float64)) <= 1e-5
    for c in (ctx, cut, ref):
        c.free()


def test_window_switched_between_steps():
    key = "tiny_f32_1seq"
    ctx = G.library_ctx(key, type_k=1, type_v=1, fused_step=True)
    ora = G.oracle_ctx(key, type_k=1, type_v=1)
    toks = G.prompts(key)[0]
    assert ctx.decode(toks) == 0 and ora.decode(toks) == 0
    rows = [len(toks) - 1]
    for win, sink in ((0, 0), (7, 0), (7, 2), (1, 0), (0, 0), (10 ** 9, 10 ** 9), (12, 30)):
        assert ctx.set_attn_window(win, sink) == 0
        ora.window, ora.n_sink = win, sink
        tok = [int(ctx.get_argmax_ith(-1))]
        for _ in range(2):
            assert ctx.decode(tok) == 0, ctx.last_error()
            assert ora.decode(tok) == 0
            assert G.rel_err(ctx.get_logits_ith(-1), ora.get_logits_ith(-1)) <= 1e-4, (win, sink)
    assert rows
    ctx.free()


@pytest.mark.parametrize("tkv,window", [(F8, 0), (F8, 20), (1, 20)])
def test_a_bad_cell_rolls_back_and_resumes(tkv, window):
    """A cell past the cache, planted on the host: the write is skipped and reported, never made."""
    kw = dict(n_seq_max=1, type_k=tkv, type_v=tkv, n_ubatch=32)
    toks = G.prompts(KEY)[0][:96]
    ref, ctx = G.library_ctx(KEY, **kw), G.library_ctx(KEY, **kw)
    for c in (ref, ctx):
        assert c.set_attn_window(window, 2) == 0
    assert ref.decode(toks) == 0, ref.last_error()
    ctx.inject_fault(1, 1)
    assert ctx.decode(toks) == -3
    assert ctx.seq_pos_max(0) == 31 and ctx.get_logits_ith(-1) is None
    assert ctx.decode(toks[32:]) == 0, ctx.last_error()
    for t in (5, 6):
        assert G.rel_err(ctx.get_logits_ith(-1), ref.get_logits_ith(-1).astype(np.float64)) <= 1e-5
        assert ctx.decode([t]) == 0 and ref.decode([t]) == 0
    ctx.free(); ref.free()


def test_sequences_interleaved_at_random():
    w = S.WORKLOADS[KEY]
    kw = dict(n_seq_max=3, n_ubatch=32)
    for unified in (True, False):
        ctx, ora = (mk(KEY, kv_unified=unified, **kw) for mk in (G.library_ctx, G.oracle_ctx))
        for c in (ctx, ora):
            if c is ora:
                c.window, c.n_sink = 9, 2
            else:
                assert c.set_attn_window(9, 2) == 0
        rng = np.random.default_rng(17)
        seq = rng.permutation(np.repeat([0, 1, 2], 30))      # each sequence's tokens in order, among the others'
        toks = rng.integers(0, w.hp.n_vocab, 90).tolist()
        pos = [int(np.sum(seq[:i] == seq[i])) for i in range(90)]
        seqs = [[int(x)] for x in seq]
        ns = [1] * 90
        flags = [1] * 90
        assert ctx.decode(toks, pos=pos, seq_ids=seqs, logits=flags) == 0, ctx.last_error()
        assert ora.decode(toks, pos=pos, seq_id=seqs, n_seq_id=ns, logits=flags) == 0
        for i in range(90):
            assert G.rel_err(ctx.get_logits_ith(i), ora.get_logits_ith(i)) <= 1e-4, (unified, i)
        ctx.free()


SHAPES = {64: HParams(2, 512, 8, 2, 64, 1024, 1024, 10000.0, 1e-5),
          128: HParams(2, 512, 4, 1, 128, 1024, 1024, 10000.0, 1e-5)}


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("tkv,window,n_sink", [(1, 100, 5), (F8, 0, 0), (F8, 33, 1)])
def test_bf16_weights_prefill_and_decode(hd, tkv, window, n_sink):
    wk = f"cache_window_{hd}_{tkv}_{window}"
    S.WORKLOADS[wk] = Workload(wk, SHAPES[hd], {"embd": S.BF16, "linear": S.BF16}, tkv, n_ctx=1024, n_seq=1,
                               n_prompt=300, n_batch=512, n_ubatch=512, n_decode=8, weight_seed=3300 + hd,
                               prompt_seed=4300)
    G.device_model.cache_clear(); G.oracle_weights.cache_clear()
    try:
        ctx = G.library_ctx(wk)
        assert ctx.set_attn_window(window, n_sink) == 0
        toks = G.prompts(wk)[0]
        if tkv == F8:
            mirror = G.mirror_ctx(S.WORKLOADS[wk])
            mirror.window, mirror.n_sink = window, n_sink
            ow = G.oracle_weights(wk)
            ctx.debug_capture(True)
            assert ctx.decode(toks) == 0, ctx.last_error()
            assert mirror.decode(toks) == 0
            _check_codes(ctx)
            rows = [0, 1, 64, 129, 298, 299]
            _check_layers(ctx, ow, mirror, rows, 2e-2)
            for i in range(3):
                assert ctx.decode([i + 3]) == 0, ctx.last_error()
                assert mirror.decode([i + 3]) == 0
                _check_codes(ctx)
                _check_layers(ctx, ow, mirror, [0], 2e-2)
        else:
            ora = G.oracle_ctx(wk)
            ora.window, ora.n_sink = window, n_sink
            assert ctx.decode(toks) == 0, ctx.last_error()
            assert ora.decode(toks) == 0
            rep = G.greedy_compare(ctx, ora, 1, [299], 8, 2e-2, {})
            assert rep.get("tokens_checked", 0) >= 4
        ctx.free()
    finally:
        del S.WORKLOADS[wk]


@pytest.fixture(scope="module")
def rows_ctx():
    key = "tiny_f32_1seq"
    c = G.library_ctx(key)
    toks = G.prompts(key)[0][:24]
    assert c.decode(toks, logits=[1] * len(toks)) == 0, c.last_error()
    yield c
    c.free()


def test_sample_batch_is_the_chain_row_by_row(rows_ctx):
    c = rows_ctx
    rows = [0, 7, 23, -1, -24, 7]                             # (a row may come twice)
    jobs = [(i, p, u) for i in rows for p in PARAMS for u in US]
    got = c.sample_batch([j[0] for j in jobs], [j[2] for j in jobs], [j[1].top_k for j in jobs],
                         [j[1].top_p for j in jobs], [j[1].min_p for j in jobs], [j[1].temperature for j in jobs],
                         [j[1].repeat_penalty for j in jobs], [j[1].penalty_tokens or [] for j in jobs])
    logit = {i: c.get_logits_ith(i).astype(np.float64) for i in rows}
    compared = 0
    for t, (i, p, u) in zip(got, jobs):
        if near_edge(logit[i], p, u):
            continue
        compared += 1
        assert t == sample_chain(logit[i], p, u), (i, p, u)
    assert compared > len(jobs) // 2
    assert c.sample_batch(list(range(24)), [0.5] * 24, temperature=0.0).tolist() == \
        [c.get_argmax_ith(i) for i in range(24)]
    assert c.sample_batch([], []).size == 0
    # beyond llm_sample_ith's limits: any top_k, long penalty lists
    every = list(range(c.n_vocab))
    pick = c.sample_batch([3], [0.3], top_k=c.n_vocab + 5, repeat_penalty=1.5, penalty_tokens=[every])
    assert 0 <= pick[0] < c.n_vocab


def test_sample_batch_refusals(rows_ctx):
    from transformer_decode_kv_gb300 import LlmError
    c = rows_ctx
    bad = [dict(top_k=0), dict(top_p=0.0), dict(top_p=1.5), dict(min_p=1.0), dict(min_p=-0.1),
           dict(repeat_penalty=0.0), dict(rows=[0, 24]), dict(rows=[0, -25]), dict(u=[0.5, 1.0]),
           dict(u=[-0.1, 0.5]), dict(u=[float("nan"), 0.5]), dict(top_p=float("nan"))]
    for kw in bad:
        kw = dict(kw)
        rows, u = kw.pop("rows", [0, 1]), kw.pop("u", [0.5, 0.5])
        with pytest.raises(LlmError):
            c.sample_batch(rows, u, **kw)
    assert c.sample_batch([0], [0.5], temperature=0.0)[0] == c.get_argmax_ith(0)
