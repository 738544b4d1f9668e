"""Attention over a paged cache where a key's score is infinite, or where rows of an E4M3 cache differ so
much that the tile kernels' 16-bit operands have to be chosen with care: zero rows, rows that only later
tokens see, rows that outgrow the first ones, so that units leave the tile kernels. Against the formula in 64 bits, token by token: what a token does
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


@pytest.mark.parametrize("act", [F16, BF16, F32])
@pytest.mark.parametrize("n_new,n_kv", [(1, 60), (3, 400), (40, 300), (40, 3000)])
def test_e4m3_rows_of_zeros_have_no_say(L, act, n_new, n_kv):
    """A row of zeros has scale 1: beside rows of 1e-5 it must not push the others out of f16's range."""
    rng, k, v = rows(7, n_kv, 2, 128)
    k *= 1e-5
    v *= 1e-5
    for x in (k, v):
        x[rng.random(x.shape[:2]) < 0.2] = 0
        x[[0, 5, n_kv // 2]] = 0
    q = rng.normal(size=(n_new, 8, 128)) * (1e4 if act == F16 else 1e5)
    check(L, act, F8, k, v, q, n_new, n_kv)
    k[:n_kv // 2] = 0                                       # whole blocks of zeros first
    v[:n_kv // 2] = 0
    check(L, act, F8, k, v, q, n_new, n_kv)
    check(L, act, F8, 0 * k, 0 * v, q, n_new, n_kv)


@pytest.mark.parametrize("act", [F16, BF16, F32])
@pytest.mark.parametrize("n_new,n_kv", [(3, 200), (6, 6), (40, 100), (40, 2900), (100, 100)])
@pytest.mark.parametrize("power", [20, 40])
def test_e4m3_rows_of_later_tokens_do_not_reach_earlier_ones(L, act, n_new, n_kv, power):
    """The last tokens' V (then K) rows are 2^power larger than the others: the tokens before them do not see that."""
    rng, k, v = rows(8, n_kv, 2, 64)
    q = rng.normal(size=(n_new, 8, 64))
    late = slice(n_kv - max(1, n_new // 4), n_kv)
    big = v.copy()
    big[late] *= 2.0 ** power
    check(L, act, F8, k, big, q, n_new, n_kv)
    big = k.copy()
    big[late] *= 2.0 ** power
    check(L, act, F8, big, v, q, n_new, n_kv)
    check(L, act, F8, big, v, q, n_new, n_kv, window=3, n_sink=2)


@pytest.mark.parametrize("act", [F16, BF16, F32])
@pytest.mark.parametrize("n_new,n_kv", [(1, 700), (3, 300)])
@pytest.mark.parametrize("power", [-110, -85, -60, 60, 90, 110])
def test_e4m3_values_at_the_ends_of_float32(L, act, n_new, n_kv, power):
    """Value rows of 2^power, alone and among rows of zeros; and beside large scores."""
    if act == F16:
        power //= 8                                         # (outputs that f16 holds)
    rng, k, v = rows(13, n_kv, 2, 64)
    q = rng.normal(size=(n_new, 8, 64))
    check(L, act, F8, k, v * 2.0 ** power, q, n_new, n_kv)
    v[rng.random(v.shape[:2]) < 0.5] = 0
    v[:200] = 0
    check(L, act, F8, k, v * 2.0 ** power, q, n_new, n_kv)
    k[7] *= 2.0 ** 30                                       # one key takes it all, or nothing
    check(L, act, F8, k, v * 2.0 ** power, q, n_new, n_kv)


@pytest.mark.parametrize("act", [BF16, F32])
def test_e4m3_equal_scores_past_2_to_24(L, act):
    """Scores of 2^30 that are equal: every key has the same weight, whatever the scales of its values."""
    rng, k, v = rows(14, 1500, 1, 64)
    k[:] = 0
    k[:, 0, 0] = 2.0 ** 15
    v *= 2.0 ** rng.integers(-30, 30, size=(v.shape[0], 1, 1))
    q = np.zeros((2, 4, 64))
    q[:, :, 0] = 2.0 ** 18
    kc, ks, kh = stored(k, F8)
    vc, vs, vh = stored(v, F8)
    plan = L.AttnPlan(L.KvPages(kc, vc, ks, vs), 4, act, 2, 1, 100)
    plan.set([2], [1500], np.arange(94)[None])
    qd = torch.from_numpy(q).to(act).cuda()
    out = torch.zeros_like(qd)
    plan.run(qd, L.KvPages(kc, vc, ks, vs), out)
    got = out.double().cpu().numpy()
    for t, n in ((0, 1499), (1, 1500)):
        want, mag = vh[:n, 0].mean(0), np.abs(vh[:n, 0]).mean(0)
        tol = O.attention_tol(want, mag, np.zeros(()), act, n, 64, 2 * np.abs(vh[:n]).max())
        assert (np.abs(got[t] - want) <= tol).all()


@pytest.mark.parametrize("act", [F16, BF16])
@pytest.mark.parametrize("n_new,n_kv,at,Hkv", [(16, 700, 400, 1), (64, 700, 690, 1), (150, 5000, 3000, 1),
                                               (150, 5000, 130, 1), (200, 700, 400, 8)])
@pytest.mark.parametrize("power", [7, 8, 12, 30])
def test_e4m3_rows_that_outgrow_the_first_block(L, act, n_new, n_kv, at, Hkv, power):
    """256-row tiles, cut and (8 KV heads, 56 tiles) whole: rows from position `at` on are 2^power larger than the first."""
    rng, k, v = rows(9, n_kv, Hkv, 128)
    q = rng.normal(size=(n_new, 8 * Hkv, 128))
    big = v.copy()
    big[at:at + 40] *= 2.0 ** power
    check(L, act, F8, k, big, q, n_new, n_kv, form=4)
    big = k.copy()
    big[at] *= 2.0 ** power
    check(L, act, F8, big, v, q, n_new, n_kv, form=4)
    small = v.copy()
    small[at:] *= 2.0 ** -power                             # and those that shrink
    check(L, act, F8, k, small, q, n_new, n_kv, window=at // 4, n_sink=3, form=4)


def test_units_done_again_leave_no_trace(L):
    """One plan, captured and not, over caches with and without rows that the tiles cannot do: each run does what its
    own cache needs."""
    n_new, n_kv = [40, 2], [1500, 300]
    rng, k, v = rows(12, 1808, 1, 64)
    sets = []
    for what in ("", "scale", "nan", ""):
        K, V = k.copy(), v.copy()
        if what == "scale":
            V[600:640] *= 2.0 ** 12
        (kc, ks, kh), (vc, vs, vh) = stored(K, F8), stored(V, F8)
        if what == "nan":
            vc.view(-1, 1, 64)[1499, 0, 5] = 0x7f            # the last token alone sees it
            vh[1499, 0, 5] = np.nan
        sets.append((kc, ks, vc, vs, kh, vh))
    cur = [x.clone() for x in sets[0][:4]]
    pages = L.KvPages(cur[0], cur[2], cur[1], cur[3])
    q = torch.from_numpy(rng.normal(size=(42, 4, 64))).to(BF16).cuda()
    out = torch.zeros_like(q)
    table = np.full((2, 94), -1, np.int32)
    table[0], table[1, :19] = np.arange(94), 94 + np.arange(19)
    plan = L.AttnPlan(pages, 4, BF16, 42, 2, table.size)
    plan.set(n_new, n_kv, table)
    assert plan.form == 5
    plan.run(q, pages, out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        plan.run(q, pages, out)
    x = q.double().cpu().numpy()
    for kc, ks, vc, vs, kh, vh in sets * 2:
        for d, s in zip(cur, (kc, ks, vc, vs)):
            d.copy_(s)
        for run in (lambda: plan.run(q, pages, out), g.replay):
            out.fill_(5)
            run()
            got = out.double().cpu().numpy()
            for t0, n, m, c0 in ((0, 40, 1500, 0), (40, 2, 300, 94 * PAGE)):
                bad_v = np.isnan(vh[c0:c0 + m]).any()
                with np.errstate(all="ignore"):
                    ref, mag, smag, vmax = reference(x[t0:t0 + n], kh[c0:], np.nan_to_num(vh[c0:]), n, m, 0, 0)
                tol = O.attention_tol(ref, mag, smag, BF16, m, 64, 2 * vmax[..., None])
                ok = np.abs(got[t0:t0 + n] - ref) <= tol
                if bad_v:
                    assert np.isnan(got[n - 1, :, 5]).all()
                    ok[n - 1, :, 5] = True
                assert ok.all()
    assert plan.error() == 0


@pytest.mark.parametrize("act,cdt,page", [(F16, F16, 64), (BF16, BF16, 17), (F32, F16, 1), (BF16, F8, 64), (F32, F8, 17)])
def test_cells_past_32_bit_offsets(L, act, cdt, page):
    """A cache of more than 2^32 bytes a tensor (E4M3: 2^32 codes), its last pages used: bulk copies, row copies, scales."""
    Hkv, hd = 8, 128
    n_pages = (2 ** 32 + 2 ** 28) // ((1 if cdt == F8 else 2) * page * Hkv * hd)
    n_new, n_kv = [1, 40], [150, 300]
    need = [-(-n // page) for n in n_kv]
    small, spare = sum(need), 3
    rng = np.random.default_rng(19)
    use = np.concatenate([np.arange(n_pages - small + 2, n_pages), [spare, 0]])   # the last pages, and two of the first
    rng.shuffle(use)
    caches = []
    for i in range(2):
        x = rng.normal(size=(small * page, Hkv, hd))
        held, sc = x, None
        if cdt == F8:
            code, s = O.quantise(x)
            held = O.E4M3[code] * s[..., None]
            sc = torch.empty((n_pages, page, Hkv), device="cuda")
            sc[torch.from_numpy(use).cuda()] = torch.from_numpy(s.astype(np.float32)).view(small, page, Hkv).cuda()
            rows_ = torch.from_numpy(code)
        else:
            rows_ = torch.from_numpy(x).to(cdt)
            held = rows_.double().numpy()
        big = torch.empty((n_pages, page, Hkv, hd), dtype=cdt, device="cuda")
        big[torch.from_numpy(use).cuda()] = rows_.view(small, page, Hkv, hd).cuda()
        caches.append((big, sc, held))
    (k, ks, kh), (v, vs, vh) = caches
    assert k.numel() * k.element_size() > 2 ** 32
    pages = L.KvPages(k, v, ks, vs)
    q = torch.from_numpy(rng.normal(size=(41, 16, hd))).to(act).cuda()
    out = torch.zeros_like(q)
    table = np.full((2, max(need)), -1, np.int32)
    table[0, :need[0]], table[1, :need[1]] = use[:need[0]], use[need[0]:]
    plan = L.AttnPlan(pages, 16, act, 41, 2, table.size)
    plan.set(n_new, n_kv, table)
    plan.run(q, pages, out)
    assert plan.error() == 0
    x, got = q.double().cpu().numpy(), out.double().cpu().numpy()
    for t0, n, m, c0 in ((0, 1, 150, 0), (1, 40, 300, need[0] * page)):
        ref, mag, smag, vmax = reference(x[t0:t0 + n], kh[c0:], vh[c0:], n, m, 0, 0)
        tol = O.attention_tol(ref, mag, smag, act, m, hd, 2 * vmax[..., None])
        assert (np.abs(got[t0:t0 + n] - ref) <= tol).all()


@pytest.mark.parametrize("act,cdt", [(F16, F16), (BF16, BF16), (F32, F16), (BF16, F8)])
@pytest.mark.parametrize("n_new", [1, 5, 70])
def test_rows_on_odd_16_byte_boundaries(L, act, cdt, n_new):
    """q and out begin 16 bytes past a 32-byte boundary, and their rows are an odd number of 16 bytes apart."""
    rng, k, v = rows(20, 200, 2, 64)
    kc, ks, kh = stored(k, cdt)
    vc, vs, vh = stored(v, cdt)
    pages = L.KvPages(kc, vc, ks, vs)
    es = 4 if act == F32 else 2
    step = 64 + 16 // es
    buf = [torch.full((n_new * 8 * step + 64,), 9.0, dtype=act, device="cuda") for _ in range(2)]
    q, out = (b[16 // es:].as_strided((n_new, 8, 64), (8 * step, step, 1)) for b in buf)
    assert out.data_ptr() % 32 == 16
    x = rng.normal(size=(n_new, 8, 64))
    q.copy_(torch.from_numpy(x))
    plan = L.AttnPlan(pages, 8, act, n_new, 1, 16)
    plan.set([n_new], [200], np.arange(13)[None])
    plan.run(q, pages, out)
    ref, mag, smag, vmax = reference(q.double().cpu().numpy(), kh, vh, n_new, 200, 0, 0)
    tol = O.attention_tol(ref, mag, smag, act, 200, 64, 2 * vmax[..., None]) + (2.0 ** -25 if act == F16 else 0)
    assert (np.abs(out.double().cpu().numpy() - ref) <= tol).all()
    out.fill_(9.0)
    assert (buf[1] == 9.0).all()                            # nothing was written between the rows
