"""sample_rows on the GPU against the 64-bit chain (oracle/sampling.py), one pick per row: cut-offs on
and off, rows of every length, ties, NaN and infinities, 16-bit logits, penalties, strides, graphs.

The library sums weights in steps of 2^-44 with a relative error of about 2^-42 each; a row is left out
only where the pick, or the prefix of top-p, lies within 1e-9 of a boundary (1e-9 is far above that and, at
4096 boundaries, leaves out a row in 10^5)."""
import math

import numpy as np
import pytest
import torch

from oracle.sampling import SamplerParams, apply_penalty, pick_margin, sample, top_k_order

pytestmark = pytest.mark.gpu
EDGE = 1e-9


@pytest.fixture(scope="module")
def L():
    import transformer_decode_kv_gb300 as L
    L.lib()
    return L


def on_edge(l, p, u):
    lp = apply_penalty(l, p.penalty_tokens, p.repeat_penalty)
    lv = lp[top_k_order(lp, p.top_k)]
    if p.top_p < 1:
        e = np.exp(lv - lv[0])
        if np.min(np.abs(np.cumsum(e) / e.sum() - p.top_p)) < EDGE:
            return True
    if p.min_p > 0 and np.min(np.abs(lv[1:] - lv[0] - math.log(p.min_p)), initial=1.0) < EDGE:
        return True
    return pick_margin(l, p, u) < EDGE


def run(L, logits, ps, us, **kw):
    R, V = logits.shape
    t = lambda v, d: torch.tensor(v, dtype=d, device="cuda")
    pen = {}
    if any(p.repeat_penalty != 1 for p in ps):
        toks = [list(p.penalty_tokens) for p in ps]
        pen = dict(repeat_penalty=t([p.repeat_penalty for p in ps], torch.float32),
                   penalty_start=t(np.concatenate([[0], np.cumsum([len(x) for x in toks])]).tolist(), torch.int32),
                   penalty_token=t(sum(toks, []), torch.int32))
    token = torch.full((R,), -7, dtype=torch.int32, device="cuda")
    L.sample_rows(logits, token, t(us, torch.float32), top_k=t([min(p.top_k, 2 ** 31 - 1) for p in ps], torch.int32),
                  top_p=t([p.top_p for p in ps], torch.float32), min_p=t([p.min_p for p in ps], torch.float32),
                  temperature=t([p.temperature for p in ps], torch.float32), **pen, **kw)
    return token.tolist()


def f32(p):
    """The parameters as the float32 numbers the kernel is given."""
    g = lambda x: float(np.float32(x))
    return SamplerParams(p.top_k, g(p.top_p), g(p.min_p), g(p.temperature), g(p.repeat_penalty), p.penalty_tokens)


def check(L, logits, ps, us):
    host = logits.double().cpu().numpy()
    us = [float(np.float32(u)) for u in us]
    got = run(L, logits, ps, us)
    left_out = 0
    for r, (p, u) in enumerate(zip(ps, us)):
        p = f32(p)
        l = apply_penalty(host[r], p.penalty_tokens, p.repeat_penalty).astype(np.float32).astype(np.float64)
        p = SamplerParams(p.top_k, p.top_p, p.min_p, p.temperature)
        if on_edge(l, p, u):
            left_out += 1
            continue
        assert got[r] == sample(l, p, u), (r, p, u, got[r])
    assert left_out <= 1 + len(us) // 100
    return got


PARAMS = [dict(top_k=1), dict(top_k=40), dict(top_k=40, top_p=0.9, temperature=0.8), dict(top_k=4096, temperature=1.5),
          dict(top_k=4096, top_p=0.5), dict(top_k=100, min_p=0.05, temperature=0.7), dict(top_k=10 ** 9),
          dict(top_k=10 ** 9, top_p=0.95), dict(top_k=10 ** 9, min_p=0.2, top_p=0.99, temperature=0.3),
          dict(top_k=5000, top_p=0.999), dict(top_k=40, temperature=0.0), dict(top_k=40, temperature=100.0),
          dict(top_k=10 ** 9, temperature=0.01), dict(top_k=3, top_p=1e-6), dict(top_k=40, min_p=1.0)]


@pytest.mark.parametrize("V", [1, 2, 31, 1000, 4097, 16384, 16385, 50257, 128256, 151936])
def test_parameters_and_vocabularies(L, V):
    rng = np.random.default_rng(V)
    logits = torch.from_numpy(rng.normal(size=(len(PARAMS), V)) * 2.5).float().cuda()
    for rep in range(3):
        us = rng.random(len(PARAMS))
        us[rep] = [0.0, 0.99999994, 0.5][rep]
        check(L, logits, [SamplerParams(**p) for p in PARAMS], us)


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
def test_16_bit_logits_have_many_ties(L, dt):
    """Rounded logits repeat: ties at the k-th value and at the pick go to the lower id."""
    rng = np.random.default_rng(1)
    logits = torch.from_numpy(rng.normal(size=(40, 32000)) * 2).to(dt).cuda()
    ps = [SamplerParams(**PARAMS[i % len(PARAMS)]) for i in range(40)]
    check(L, logits, ps, rng.random(40))


def test_distributions(L):
    """Rows whose top lies in a few bins, or spread over many: offsets and scales of every size, one outlier, long
    tails, log probabilities, masked vocabularies."""
    rng = np.random.default_rng(2)
    V = 60000
    g = rng.normal(size=V)
    rows = [g * 1e-4, g * 1e4, g + 1000, g - 1e6, np.where(np.arange(V) == 77, 1e4, g), rng.standard_cauchy(V),
            np.log(rng.dirichlet(np.full(V, 0.05)) + 1e-30), np.where(rng.random(V) < 0.999, -np.inf, g), np.exp(3 * g), -np.exp(3 * g),
            np.round(g * 3), np.where(np.arange(V) < 30000, 5.0, g)]
    logits = torch.from_numpy(np.stack(rows)).float().cuda()
    for kw in (dict(top_k=40), dict(top_k=4096, top_p=0.9), dict(top_k=1000, min_p=0.01, temperature=1.3), dict(top_k=59999),
               dict(top_k=513, temperature=0.5)):
        check(L, logits, [SamplerParams(**kw)] * len(rows), rng.random(len(rows)))


def test_flat_and_two_valued_rows(L):
    V = 20000
    x = torch.zeros(6, V, device="cuda")
    x[1] = -3.25
    x[2, ::7] = 1.0
    x[3, 1::2] = -0.0                                            # equal to +0
    x[4, 5:9] = 2.0
    x[5] = torch.where(torch.arange(V, device="cuda") % 3 == 0, 0.5, -60.0)
    ps = [SamplerParams(top_k=k) for k in (10, 10 ** 9, 100, 50, 2, 10 ** 9)]
    for u in (0.0, 0.31, 0.77, 0.999):
        check(L, x, ps, [u] * 6)


def test_nan_and_infinities(L):
    V = 5000
    x = torch.randn(7, V, device="cuda")
    x[0, 10:4000] = float("nan")
    x[1, :] = float("nan")
    x[2, :] = float("-inf")
    x[3, :] = float("-inf"); x[3, 77] = -1e30
    x[4, 123] = float("inf"); x[4, 4000] = float("inf")
    x[5, :] = float("nan"); x[5, 4999] = float("-inf")
    x[6, 0] = float("nan")
    ps = [SamplerParams(top_k=k) for k in (4500, 10, 10, 10 ** 9, 10 ** 9, 3, 1)]
    for u in (0.0, 0.4, 0.9):
        got = run(L, x, ps, [u] * 7)
        l = x.double().cpu().numpy()
        assert got[1] == got[2] == got[5] == -1
        assert got[3] == 77
        assert got[4] == (123 if u < 0.5 else 4000)
        assert got[6] == int(np.nanargmax(l[6]))
        ok = np.where(np.isnan(l[0]), -np.inf, l[0])
        assert got[0] == sample(ok, SamplerParams(top_k=1010 + 3490), float(np.float32(u)))
    # greedy gives the same answers for these rows
    token = torch.zeros(7, dtype=torch.int32, device="cuda")
    L.sample_rows(x, token)
    assert token.tolist()[1:6] == [-1, -1, 77, 123, -1]


def test_extreme_values(L):
    x = torch.tensor([[3e38, -3e38, 3e38, 0.0], [1e-40, 0.0, -1e-40, 5e-41], [100.0, 99.999, 0, -100]], device="cuda")
    ps = [SamplerParams(top_k=4), SamplerParams(top_k=4), SamplerParams(top_k=4, temperature=1e-3)]
    for u in (0.1, 0.6, 0.9):
        check(L, x, ps, [u] * 3)
    # temperatures at the ends of the float range
    assert run(L, x, [SamplerParams(top_k=4, temperature=1e-45)] * 3, [0.9] * 3) == [2, 0, 0]
    assert run(L, x[2:], [SamplerParams(top_k=4, temperature=float("inf"))], [0.6])[0] == 2


def test_parameter_limits(L):
    x = torch.randn(1, 3000, device="cuda")
    best = int(x.argmax())
    nan = float("nan")
    one = lambda **k: run(L, x, [SamplerParams(**{**dict(top_k=10), **k})], [k.pop("u", 0.99)])[0]
    assert one(top_p=0.0) == one(top_p=-1.0) == one(top_p=nan) == best
    assert one(temperature=-1.0) == one(temperature=nan) == best
    assert one(min_p=2.0) == one(min_p=1.0) == best
    assert one(min_p=nan) == one(min_p=0.0) == one(min_p=-1.0)
    assert run(L, x, [SamplerParams(top_k=10)], [1.5]) == run(L, x, [SamplerParams(top_k=10)], [0.99999994])
    assert run(L, x, [SamplerParams(top_k=10)], [-3.0]) == run(L, x, [SamplerParams(top_k=10)], [nan]) == [best]
    assert run(L, x, [SamplerParams(top_k=0)], [0.7]) == run(L, x, [SamplerParams(top_k=3000)], [0.7])


def test_penalties(L):
    rng = np.random.default_rng(3)
    V = 40000
    logits = torch.from_numpy(rng.normal(size=(8, V)) * 2).float().cuda()
    top = logits.topk(60, dim=1).indices.cpu().numpy()
    ps = []
    for r in range(8):
        toks = np.concatenate([top[r][: 5 * r], top[r][:3], rng.integers(0, V, 100 * r), [V - 1, 0]]).tolist()
        ps.append(SamplerParams(top_k=50, temperature=0.9, repeat_penalty=[1.3, 0.7, 1.0, 2.0][r % 4], penalty_tokens=toks))
    check(L, logits, ps, rng.random(8))
    # ids outside the vocabulary are ignored, the logits stay as they were
    before = logits.clone()
    ps = [SamplerParams(top_k=50, repeat_penalty=5.0, penalty_tokens=[-1, V, 2 ** 31 - 1, -2 ** 31]) for _ in range(8)]
    assert run(L, logits, ps, [0.3] * 8) == run(L, logits, [SamplerParams(top_k=50)] * 8, [0.3] * 8)
    assert torch.equal(before, logits)


def test_frequencies(L):
    """Picks over a grid of u reproduce the softmax."""
    l = torch.tensor([1.0, -0.5, 2.0, 0.3, -3.0])
    N = 4096
    token = torch.zeros(N, dtype=torch.int32, device="cuda")
    u = ((torch.arange(N) + 0.5) / N).cuda()
    L.sample_rows(l.cuda()[None].expand(N, 5), token, u, temperature=torch.ones(N, device="cuda"))
    count = torch.bincount(token.cpu(), minlength=5) / N
    assert (count - torch.softmax(l, 0)).abs().max() <= 1.0 / N + 1e-6


def test_strides_graph_and_many_rows(L):
    rng = np.random.default_rng(4)
    base = torch.from_numpy(rng.normal(size=(300, 3 * 2000 + 1))).float().cuda()
    logits = base[:, 2001:4003]                                  # rows not 16-byte aligned
    ps = [SamplerParams(top_k=20, top_p=0.9)] * 300
    check(L, logits, ps, rng.random(300))
    x = torch.randn(4, 30000, device="cuda")
    u = torch.rand(4, device="cuda")
    t = torch.ones(4, device="cuda")
    token = torch.zeros(4, dtype=torch.int32, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        L.sample_rows(x, token, u, temperature=t)
    for _ in range(2):
        x.normal_()
        u.uniform_()
        g.replay()
        torch.cuda.synchronize()
        want = [sample(a, SamplerParams(top_k=10 ** 9), b) for a, b in zip(x.double().cpu().numpy(), u.double().tolist())]
        assert token.tolist() == want
    with pytest.raises(L.LlmError):
        L.sample_rows(torch.zeros(1, 400000, device="cuda"), token[:1])
    with pytest.raises(ValueError):
        L.sample_rows(x.T, token)
    with pytest.raises(ValueError):
        L.sample_rows(x, token.long())
    with pytest.raises(L.LlmError, match="device memory"):
        L.sample_rows(x.cpu(), token)


def test_rows_past_32_bit_offsets(L):
    """Rows 1.5 * 2^30 elements apart: the last begins past 2^32 bytes (and 2^31 elements)."""
    base = torch.empty(3 * 2 ** 30 + 2000, dtype=torch.float16, device="cuda")
    logits = base.as_strided((3, 2000), (3 * 2 ** 29, 1))
    rng = np.random.default_rng(7)
    logits.copy_(torch.from_numpy(rng.normal(size=(3, 2000)) * 2))
    for kw in (dict(top_k=40), dict(top_k=10 ** 9, top_p=0.9)):
        check(L, logits, [SamplerParams(**kw)] * 3, rng.random(3))
