"""Attention over a paged cache where a key's score is infinite. Against the formula in 64 bits, token by token: what a token does
not see has no part in its tolerance.

Tolerances are those of ops_common.attention_tol with the largest |v| that the token itself sees. An E4M3 cache
doubles that term in the small tiles: p * s / E in f16 is off by 2^-25 below its normal range, in units of E * 448,
and E, the largest scale the token sees, belongs to a row whose largest value is above 224 E. An f16 output adds
2^-25, half a step of its subnormal numbers, and one beyond 65504 by half a step (2^4) or more is infinite."""
import math

import numpy as np
import pytest
import torch

from tests import ops_common as O

pytestmark = pytest.mark.gpu

F16, BF16, F32, F8 = torch.float16, torch.bfloat16, torch.float32, torch.uint8
PAGE = 16


@pytest.fixture(scope="module")
def L():
    import transformer_decode_kv_gb300 as L
    L.lib()
    return L


def stored(val, cdt):
    """A cache [pages, PAGE, Hkv, hd] of the rows val [cells, Hkv, hd], its scales, and what it holds."""
    val = val.reshape(-1, PAGE, *val.shape[1:])
    if cdt == F8:
        code, s = O.quantise(val)
        t, sc = torch.from_numpy(code).cuda(), torch.from_numpy(s.astype(np.float32)).cuda()
        held = O.E4M3[code] * s[..., None]
    else:
        t, sc = torch.from_numpy(val).to(cdt), None
        held = t.double().numpy()
        t = t.cuda()
    return t, sc, held.reshape(-1, *val.shape[2:])


def reference(q, k, v, n_new, n_kv, window, n_sink):
    """out, sum |w v|, the largest sum |q k| of a finite score and the largest |v| seen, per (token, head); cell j holds
    position j. (Values are finite in these tests, so a weight of 0 leaves a hidden row out.)"""
    H, hd = q.shape[1:]
    G = H // k.shape[1]
    out, mag = np.zeros(q.shape), np.zeros(q.shape)
    smag, vmax = np.zeros(q.shape[:2]), np.zeros(q.shape[:2])
    if n_kv == 0:
        return out, mag, smag, vmax
    j, p = np.arange(n_kv)[None], np.arange(n_kv - n_new, n_kv)[:, None]
    vis = j <= p
    if window:
        vis &= (j > p - window) | (j < n_sink)
    some = vis.any(1)
    with np.errstate(all="ignore"):
        for h in range(H):
            K, V = k[:n_kv, h // G], v[:n_kv, h // G]
            z = np.where(vis, q[:, h] @ K.T * hd ** -0.5, -np.inf)
            a = np.abs(q[:, h]) @ np.abs(K).T
            smag[:, h] = np.where(vis & np.isfinite(a), a, 0).max(1) * hd ** -0.5
            vmax[:, h] = np.where(vis, np.abs(V).max(1), 0).max(1)
            w = np.exp(z - z.max(1, keepdims=True))
            w /= w.sum(1, keepdims=True)
            out[some, h], mag[some, h] = (w @ V)[some], (w @ np.abs(V))[some]
    return out, mag, smag, vmax


def check(L, act, cdt, k, v, q, n_new, n_kv, window=0, n_sink=0, form=None):
    kc, ks, kh = stored(k, cdt)
    vc, vs, vh = stored(v, cdt)
    pages = L.KvPages(kc, vc, ks, vs)
    H, hd = q.shape[1:]
    qd = torch.from_numpy(q).to(act).cuda()
    out = torch.full_like(qd, 7.0)
    table = np.arange(-(-n_kv // PAGE))[None]
    plan = L.AttnPlan(pages, n_head=H, dtype=act, max_tok=n_new, max_seq=1, max_table=max(1, table.size), window=window, n_sink=n_sink)
    plan.set([n_new], [n_kv], table)
    if form is not None:
        assert plan.form == form
    plan.run(qd, pages, out)
    assert plan.error() == 0
    got = out.double().cpu().numpy()
    ref, mag, smag, vmax = reference(qd.double().cpu().numpy(), kh, vh, n_new, n_kv, window, n_sink)
    tol = O.attention_tol(ref, mag, smag, act, n_kv, hd, (2 if cdt == F8 else 1) * vmax[..., None])
    if act == F16:
        tol = tol + 2.0 ** -25
    with np.errstate(invalid="ignore"):
        bad = np.where(np.isnan(ref), np.isfinite(got), ~(np.abs(got - ref) <= tol))
    if act == F16:                                          # (either rounding where the exact value may be on either side)
        bad &= ~(np.isinf(got) & (np.sign(got) == np.sign(ref)) & (np.abs(ref) + tol >= 65520))
    assert not bad.any(), (bad.sum(), np.argwhere(bad)[:4], got[bad][:4], ref[bad][:4], np.broadcast_to(tol, bad.shape)[bad][:4])
    return ref


def rows(seed, n, Hkv, hd):
    rng = np.random.default_rng(seed)
    return rng, *(rng.normal(size=(-(-n // PAGE) * PAGE, Hkv, hd)) for _ in range(2))


# 8-row, 16-row and (f16, bf16) 256-row tiles; one unit, and cut into many
FORMS = [(1, 60), (1, 9000), (3, 60), (3, 9000), (40, 70), (40, 9000)]


@pytest.mark.parametrize("n_new,n_kv", FORMS)
@pytest.mark.parametrize("act,cdt", [(F16, F16), (BF16, BF16), (F32, F16)])
def test_a_score_of_minus_infinity_has_no_weight(L, act, cdt, n_new, n_kv):
    """The first key is infinite in one dim: heads with a negative q there give it no weight, those with a positive
    one have no result."""
    rng, k, v = rows(5, n_kv, 1, 64)
    k[0, 0, 7] = math.inf
    q = rng.normal(size=(n_new, 4, 64))
    q[:, :, 7] = np.array([-1.0, 1.0, -2.0, -0.5]) * (1 + rng.random(size=(n_new, 1)))
    tc = act != F32 and n_new == 40
    ref = check(L, act, cdt, k, v, q, n_new, n_kv, form=4 if tc else 1 if n_new == 1 else 2)
    assert np.isnan(ref[:, 1]).all() and np.isfinite(ref[:, [0, 2, 3]]).all()
    # the same key as a sink before a window
    check(L, act, cdt, k, v, q, n_new, n_kv, window=20, n_sink=1)


@pytest.mark.parametrize("n_new", [1, 5, 40])
@pytest.mark.parametrize("act,cdt", [(F16, F16), (BF16, BF16), (F32, F16)])
def test_a_first_token_with_an_infinite_key(L, act, cdt, n_new):
    """The first token sees one key of infinite score: 0 / 0 or inf / inf. Those after it see others too."""
    rng, k, v = rows(11, n_new, 1, 64)
    k[0, 0, 7] = math.inf
    q = rng.normal(size=(n_new, 4, 64))
    q[:, :, 7] = [-1.0, 1.0, -2.0, -0.5]
    ref = check(L, act, cdt, k, v, q, n_new, n_new)
    assert np.isnan(ref[0]).all() and np.isfinite(ref[1:, [0, 2, 3]]).all()


@pytest.mark.parametrize("n_new,n_kv", [(1, 50), (3, 50), (40, 60), (40, 9000)])
@pytest.mark.parametrize("act,cdt", [(F16, F16), (BF16, BF16), (F32, F16)])
def test_scores_of_minus_infinity_only(L, act, cdt, n_new, n_kv):
    """Softmax over -infinity alone is 0 / 0, however many keys there are; tokens before the first key see nothing."""
    rng, k, v = rows(6, n_kv, 1, 64)
    k[:, 0, 3] = math.inf                                   # (heads of one sign: no other score sends the tile elsewhere)
    q = rng.normal(size=(n_new, 4, 64))
    q[:, :, 3] = -1.0
    assert np.isnan(check(L, act, cdt, k, v, q, n_new, n_kv)).all()
    ref = check(L, act, cdt, k, v, q, n_new, max(n_new - 2, 0))
    assert (ref[:min(2, n_new)] == 0).all()
