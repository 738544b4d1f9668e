"""The sliding window and the F8_E4M3 cache type of a context, as far as they need no GPU: accepted and
refused arguments, the visibility of the cells against the oracle, and the oracle's E4M3 rows against a
table of the type's values."""
import os

import numpy as np
import pytest

import oracle
from oracle import formats as OF
from oracle.context import forward_no_cache
from synthetic.configs import HParams
from tests import ops_common as O
from tests.helpers import MICRO, oracle_weights

HP = HParams(n_layer=2, n_embd=64, n_head=8, n_head_kv=2, head_dim=32, n_ff=96, n_vocab=50,
             rope_freq_base=10000.0, rms_eps=1e-6)


@pytest.fixture(scope="module")
def T():
    from transformer_decode_kv_gb300 import build, binding
    if not os.path.exists(binding.LIB_PATH):
        build.build()
    return binding


def test_cache_types(T):
    T.Context(HP, n_ctx=256, type_k=T.F8_E4M3, type_v=T.F8_E4M3, host_only=True).free()
    for k, v in ((T.F8_E4M3, T.F16), (T.F16, T.F8_E4M3), (T.BF16, T.BF16)):
        with pytest.raises(T.LlmError, match="type_k/type_v"):
            T.Context(HP, n_ctx=256, type_k=k, type_v=v, host_only=True)


def test_window_refusals_leave_it_unchanged(T):
    for t, ok in ((T.F16, True), (T.F8_E4M3, True), (T.F32, False), (T.Q8_0, False)):
        c = T.Context(HP, n_ctx=256, type_k=t, type_v=t, host_only=True)
        c.debug_capture(True)
        assert c.set_attn_window(3, 1) == (0 if ok else -1)
        assert c.set_attn_window(-1, 0) == -1 and c.set_attn_window(4, -1) == -1
        assert c.set_attn_window(2 ** 31 - 1, 2 ** 31 - 1) == (0 if ok else -1)
        assert c.set_attn_window(3, 1) == (0 if ok else -1)
        assert c.decode([1] * 8) == 0
        want = np.tril(np.ones((8, 8), dtype=bool))
        if ok:
            j = np.arange(8)
            want &= (j[None] > j[:, None] - 3) | (j[None] < 1)
        assert np.array_equal(c.ubatch_mask(0)[:, :8], want)
        assert c.set_attn_window(0, 5) == 0                     # off: allowed for every type
        assert c.decode([1]) == 0
        assert c.ubatch_mask(0)[0, :9].all()
        c.free()


@pytest.mark.parametrize("unified", [True, False])
def test_window_masks_match_the_oracle(T, unified):
    rng = np.random.default_rng(5)
    kw = dict(n_ctx=512, n_seq_max=4, n_batch=64, n_ubatch=16)
    lib = T.Context(HP, host_only=True, kv_unified=unified, **kw)
    ora = oracle.OracleContext(HP, None, compute=False, kv_unified=unified, **kw)
    lib.debug_capture(True)
    for step in range(40):
        if step % 7 == 0:
            w, s = int(rng.integers(0, 9)), int(rng.integers(0, 5))
            assert lib.set_attn_window(w, s) == 0
            ora.window, ora.n_sink = w, s
        if step % 5 == 4:
            s, p0 = int(rng.integers(0, 4)), int(rng.integers(0, 6))
            p1 = p0 + int(rng.integers(1, 8))
            assert lib.seq_rm(s, p0, p1) == ora.seq_rm(s, p0, p1)
        n = int(rng.integers(1, 30))
        toks = rng.integers(0, 50, n).tolist()
        seqs = [[int(x)] for x in rng.integers(0, 4, n)]
        r = lib.decode(toks, seq_ids=seqs, logits=[0] * n)
        assert r == ora.decode(toks, seq_id=seqs, n_seq_id=[1] * n, logits=[0] * n)
        if r:
            for s in range(4):
                lib.seq_rm(s, -1, -1), ora.seq_rm(s, -1, -1)
            continue
        for k, u in enumerate(ora.last_ubatches):
            assert np.array_equal(lib.ubatch_mask(k), u["mask"]), (step, k)
    lib.free()


def test_batched_sampler_refuses_a_host_only_context(T):
    c = T.Context(HP, n_ctx=256, host_only=True)
    with pytest.raises(T.LlmError):
        c.sample_batch([0], [0.5])
    c.free()


def test_oracle_e4m3_rows_against_the_table():
    rng = np.random.default_rng(6)
    x = (rng.normal(size=(300, 32)) * np.exp(6 * rng.normal(size=(300, 1)))).astype(np.float32).astype(np.float64)
    x[0] = 0
    x[1, 0], x[2, 0], x[3, 0] = 448, np.nextafter(np.float32(448), np.float32(500)), 1e-42
    x[1, 1:], x[2, 1:], x[3, 1:] = x[1, 1:] % 1, x[2, 1:] % 1, 0
    x[4] = np.arange(32) * 2.0 ** -10                        # ties of the subnormal grid once scaled
    x[4, 0] = 448
    code, s = O.quantise(x)
    v, so = OF.f8_e4m3_rows(x)
    assert np.array_equal(so[..., 0], s)
    assert np.array_equal(v, O.E4M3[code])
    back = OF.round_to_type(x, OF.F8_E4M3)
    # half a step: 2^-4 of a normal value, 2^-10 of the scale below 2^-6 of it
    assert np.all(np.abs(back - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * so))
    assert np.array_equal(OF.round_to_type(back, OF.F8_E4M3), back)


def test_oracle_window_and_f8_cache_equal_the_no_cache_forward():
    w = oracle_weights(MICRO, 9, {"embd": 0, "linear": 0})
    toks = np.arange(12) * 7 % MICRO.n_vocab
    want = forward_no_cache(w, MICRO, toks, OF.F8_E4M3, OF.F8_E4M3)
    for win in (0, 12):
        c = oracle.OracleContext(MICRO, w, n_ctx=256, type_k=OF.F8_E4M3, type_v=OF.F8_E4M3, n_ubatch=5)
        c.window = win
        assert c.decode(toks, logits=[1] * 12) == 0
        assert np.max(np.abs(c.logits - want)) <= 1e-9 * np.max(np.abs(want))
    c = oracle.OracleContext(MICRO, w, n_ctx=256, n_ubatch=5)
    c.window = 1                                             # only the token itself: each row is a one-token forward's
    assert c.decode(toks, logits=[1] * 12) == 0
    one = forward_no_cache(w, MICRO, toks[:1])               # (attention of one key is its value row, at any position)
    assert np.max(np.abs(c.logits[0] - one[0])) <= 1e-9 * np.max(np.abs(one))


def test_a_mask_is_that_of_the_decode_it_belongs_to(T):
    """The window set after a decode does not change what that decode's tokens saw."""
    c = T.Context(HP, n_ctx=256, host_only=True)
    c.debug_capture(True)
    assert c.set_attn_window(3, 1) == 0
    assert c.decode([1] * 8) == 0
    j = np.arange(8)
    want = (j[None] <= j[:, None]) & ((j[None] > j[:, None] - 3) | (j[None] < 1))
    for window, n_sink in ((3, 1), (0, 0), (5, 2)):
        assert c.set_attn_window(window, n_sink) == 0
        assert np.array_equal(c.ubatch_mask(0)[:, :8], want)
    c.free()
