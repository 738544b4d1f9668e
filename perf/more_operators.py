"""Cases that measure attention over a 4-bit paged cache and the page tables and plans made on the GPU.

`run` computes a case either in plain torch (`own` false) or through the library's public calls
(`own` true): kv_store / kv_load and AttnPlan over a cache of 4-bit rows (E2M1 codes, an E4M3 scale per
16 values, a power-of-two scale per row), pages_extend (pages, cells and positions of a step's new
tokens from the sequences' lengths) and AttnPlan.set_device (a step's plan from lengths and a page
table on the device), the last two joined with kv_store and AttnPlan.run as a serving step uses them.
"""
import math

import numpy as np
import torch

own = False

_DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_ES = {"f32": 4, "f16": 2, "bf16": 2}
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------- cases
def _kv(name, act, Hkv, hd, page, n, skip):
    return {"name": name, "op": "kv", "act": act, "cache": "f4", "Hkv": Hkv, "hd": hd, "page": page, "n": n,
            "skip": skip}


def _attn(name, act, H, Hkv, hd, page, n_new, n_kv, window=0, n_sink=0):
    return {"name": name, "op": "attn", "act": act, "cache": "f4", "H": H, "Hkv": Hkv, "hd": hd, "page": page,
            "n_new": " ".join(map(str, n_new)), "n_kv": " ".join(map(str, n_kv)), "window": window, "n_sink": n_sink}


def _step(name, act, cache, H, Hkv, hd, page, n_new, n_kv, window=0, n_sink=0):
    c = _attn(name, act, H, Hkv, hd, page, n_new, n_kv, window, n_sink)
    return {**c, "op": "step", "cache": cache}


def _pages(name, n_seq, page, every, max_new, max_kv, room):
    """n_seq sequences of up to max_kv rows; one of `every` takes up to max_new tokens, the others one or none."""
    return {"name": name, "op": "pages", "n_seq": n_seq, "page": page, "every": every, "max_new": max_new,
            "max_kv": max_kv, "room": room}


def listed():
    dec32 = [1 + (i * 1117) % 2304 for i in range(31)] + [2304]
    dec16 = [32768 - 1571 * i for i in range(16)]
    win32 = [73728 // 32 + 9 + 2003 * i for i in range(32)]
    return [
        # a decode step of 32 sequences writes its rows in 4 bits and reads them back
        _kv("kv_f4_step", "f16", 8, 128, 16, 32, 0),
        # a long prompt's rows, a few of them padding that must not be written
        _kv("kv_f4_prompt", "bf16", 8, 128, 16, 8192, 37),
        # one sequence, one token after a 512-token prompt: latency counts
        _attn("attn_f4_step_1", "f16", 32, 8, 128, 16, [1], [513]),
        # long contexts of 16 sequences, what 4 bits are for: the largest decode step
        _attn("attn_f4_step_long", "bf16", 32, 8, 128, 64, [1] * 16, dec16),
        # long contexts, each token sees four first tokens and a window
        _attn("attn_f4_step_window", "bf16", 32, 8, 128, 16, [1] * 32, win32, 1024, 4),
        # the last 512-token chunk of an 8192-token prompt
        _attn("attn_f4_chunk_512", "f16", 32, 8, 128, 16, [512], [8192]),
        # a large chunk deep in a long context: the largest case
        _attn("attn_f4_chunk_2048", "bf16", 32, 8, 128, 64, [2048], [32768]),
        # prompts and single tokens of a small float32 model (8 heads of 32, 2 KV heads)
        _attn("attn_f4_tiny_f32", "f32", 8, 2, 32, 8, [128, 1, 77, 1, 128, 1, 1, 9], [128, 500, 77, 33, 300, 1, 90, 9]),
        # the pages and cells of a decode step of 64 sequences: latency counts
        _pages("pages_decode_64", 64, 16, 64, 1, 8192, 0),
        # a busy server's step: 512 sequences, prompt chunks among single tokens
        _pages("pages_mixed_512", 512, 16, 16, 1024, 32768, 100),
        # a whole decode step of 32 sequences from lengths on the device: pages, rows, plan, attention
        _step("step_decode_32", "f16", "f16", 32, 8, 128, 16, [1] * 32, dec32),
        # chunks and single tokens of several sequences, 4-bit cache, windowed, likewise
        _step("step_mixed_f4", "bf16", "f4", 32, 8, 128, 16, [700, 1, 333, 1, 64, 129],
              [4096, 8191, 333, 77, 1500, 6000], 1024, 4),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["kv", "attn", "attn", "attn", "pages", "step", "step"])
    hd = rng.choice([32, 64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    page = rng.choice([1, 8, 16, 17, 32, 64, 100, 128])
    if kind == "kv":
        n = _logint(rng, 1, 8192)
        c = _kv("", rng.choice(["f32", "f16", "bf16"]), Hkv, hd, page, n, rng.randint(0, min(n - 1, 40)))
    elif kind == "pages":
        n_seq = _logint(rng, 1, 2048)
        c = _pages("", n_seq, page, rng.choice([1, 4, 16, 64]), _logint(rng, 1, max(1, min(1024, 16384 // n_seq))),
                   _logint(rng, 1, min(32768, (page << 20) // n_seq)), rng.choice([0, 1, 100]))
    else:
        H = Hkv * rng.choice([1, 2, 3, 4, 4, 6, 8])
        window = rng.choice([0, 0, _logint(rng, 1, 4096)])
        n_sink = rng.choice([0, 1, 4, 16]) if window else 0
        if rng.random() < 0.5:                                # single tokens
            n_seq = _logint(rng, 1, 64)
            n_new = [1] * n_seq
            n_kv = [_logint(rng, 1, 32768 if n_seq < 8 else 8192) for _ in range(n_seq)]
        else:                                                 # chunks and single tokens
            n_seq = rng.randint(1, 6)
            n_new = [_logint(rng, 1, 1024) for _ in range(n_seq)]
            n_kv = [n + (0 if rng.random() < 0.3 else _logint(rng, 1, 8192)) for n in n_new]
        if kind == "attn":
            make, types = _attn, (rng.choice(["f16", "bf16", "f32"]),)
        else:
            make, types = _step, rng.choice([("f16", "f16"), ("bf16", "bf16"), ("f16", "f4"), ("bf16", "f4")])
        c = make("", *types, H, Hkv, hd, page, n_new, n_kv, window, n_sink)
        # no dearer than the largest listed cases: drop sequences from the end
        while len(n_kv) > 1 and (work(c)["bytes"] > 4e8 or work(c)["flops"] > 1e12):
            n_new, n_kv = n_new[:-1], n_kv[:-1]
            c = make("", *types, H, Hkv, hd, page, n_new, n_kv, window, n_sink)
    del c["name"]
    return c


# ---------------------------------------------------------------- inputs
def _ints(s):
    return [int(x) for x in s.split()]


def _page_lens(case):
    """(rows held before the step, new tokens) of each sequence."""
    n_kv, n_new = [], []
    for i in range(case["n_seq"]):
        n_kv.append(case["max_kv"] - 1 - (i * 1117) % case["max_kv"])
        n_new.append(1 + (i * 7919 + case["max_new"] - 1) % case["max_new"] if i % case["every"] == 0 else i % 8 != 5)
    return n_kv, [int(n) for n in n_new]


def _rows(shape, gen):
    """K or V rows: normal, with channels and rows of other magnitudes."""
    x = torch.randn(shape, generator=gen, device="cuda")
    x *= 1 + 3 * (torch.rand(shape[-1], generator=gen, device="cuda") > 0.95)
    x *= torch.exp(0.5 * torch.randn(shape[:-1] + (1,), generator=gen, device="cuda"))
    return x


def _quantise(x):
    """Rows of float32 values in 4 bits: (codes 0 .. 15, block scales as float8_e4m3fn, row scales).

    Every step is exact or one rounding: x / s is a change of the exponent, the block scale is the
    E4M3 number nearest to max / 6, and a code is found by comparing with midpoint * b, which float32
    holds (3 and 4 significant bits)."""
    m, e = torch.frexp(x.abs().amax(-1, keepdim=True))     # amax = m 2^e, m in [0.5, 1)
    e = torch.where(m > 0.65625, e - 11, e - 12)           # 2688 = 0.65625 * 2^12
    e = torch.where(m == 0, torch.zeros_like(e), e).clamp(min=-126)
    y = torch.ldexp(x, -e).unflatten(-1, (-1, 16))
    b = (y.abs().amax(-1, keepdim=True) / 6).to(torch.float8_e4m3fn).float().clamp(min=2.0 ** -9)
    a = y.abs()
    code = (a > 0.25 * b).to(torch.uint8)
    for mid, even_above in ((0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        code += (a >= mid * b) if even_above else (a > mid * b)
    code += 8 * torch.signbit(y).to(torch.uint8)
    return code.flatten(-2), b[..., 0].to(torch.float8_e4m3fn), torch.ldexp(torch.ones_like(m), e)[..., 0]


def _cache(n_pages, page, Hkv, hd, cache, gen):
    """A cache of random rows: {"c": rows [n_pages, page, Hkv, ...], "b": block scales, "s": row scales}. A 4-bit cache
    keeps a head's cells of a page together, so that a page's rows and scales of a head are contiguous."""
    d = {"c": torch.empty((n_pages, page, Hkv, hd), dtype=_DT[cache], device="cuda")} if cache != "f4" else {
        "c": torch.empty((n_pages, Hkv, page, hd // 2), dtype=torch.uint8, device="cuda").transpose(1, 2),
        "b": torch.empty((n_pages, Hkv, page, hd // 16), dtype=torch.uint8, device="cuda").transpose(1, 2),
        "s": torch.empty((n_pages, Hkv, page), device="cuda").transpose(1, 2)}
    step = max(1, (1 << 25) // (page * Hkv * hd))
    for p in range(0, n_pages, step):
        x = _rows((min(step, n_pages - p), page, Hkv, hd), gen)
        if cache == "f4":
            code, b, s = _quantise(x)
            d["c"][p:p + step] = code[..., ::2] | code[..., 1::2] << 4
            d["b"][p:p + step] = b.view(torch.uint8)
            d["s"][p:p + step] = s
        else:
            d["c"][p:p + step] = x.to(d["c"].dtype)
    return d


def _kv_pages(st):
    from transformer_decode_kv_gb300 import KvPages
    k, v = st["kc"], st["vc"]
    return KvPages(k["c"], v["c"], k.get("s"), v.get("s"), k.get("b"), v.get("b"))


def _prepare_kv(case, st, gen, rng):
    Hkv, hd, page, n = case["Hkv"], case["hd"], case["page"], case["n"]
    n_pages = -(-n // page) + 3
    st["k"], st["v"] = (_rows((n, Hkv, hd), gen).to(_DT[case["act"]]) for _ in range(2))
    cells = np.concatenate([np.arange(page) + page * p for p in rng.permutation(n_pages)])
    slot = cells[:n].astype(np.int32)
    slot[rng.permutation(n)[:case["skip"]]] = -1              # rows of padding
    st["slot"] = torch.from_numpy(slot).cuda()
    st["kc"], st["vc"] = (_cache(n_pages, page, Hkv, hd, "f4", gen) for _ in range(2))
    st["ko"], st["vo"] = (torch.zeros_like(st["k"]) for _ in range(2))
    if own:
        st["pages"] = _kv_pages(st)


def _prepare_attn(case, st, gen, rng):
    """Attention of new tokens; for a step, the sequences hold the rows before the new ones and the pages of those."""
    H, Hkv, hd, page = case["H"], case["Hkv"], case["hd"], case["page"]
    n_new, n_kv = _ints(case["n_new"]), _ints(case["n_kv"])
    step = case["op"] == "step"
    held = [-(-(n - m if step else n) // page) for m, n in zip(n_new, n_kv)]
    need = [-(-n // page) for n in n_kv]
    n_pages = sum(need) + 2
    perm = rng.permutation(n_pages).astype(np.int32)
    table = np.zeros((len(n_kv), max(need)), dtype=np.int32)
    at = 0
    for i, m in enumerate(held):
        table[i, :m] = perm[at:at + m]
        at += m
    st["n_new"], st["n_kv"] = n_new, n_kv
    st["table"] = torch.from_numpy(table).cuda()
    st["kc"], st["vc"] = (_cache(n_pages, page, Hkv, hd, case["cache"], gen) for _ in range(2))
    tok = sum(n_new)
    st["q"] = torch.randn((tok, H, hd), generator=gen, device="cuda").to(_DT[case["act"]])
    st["out"] = torch.zeros_like(st["q"])
    if step:
        ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
        st["k"], st["v"] = (_rows((tok, Hkv, hd), gen).to(_DT[case["act"]]) for _ in range(2))
        st["add"], st["before"] = ints(n_new), ints([n - m for m, n in zip(n_new, n_kv)])
        st["free"], st["n_free"] = ints(perm[at:].tolist()), ints([n_pages - at])
        st["cell"], st["pos"] = ints([0] * tok), ints([0] * tok)
        st["start"], st["after"], st["left"] = ints([0] * (len(n_kv) + 1)), ints([0] * len(n_kv)), ints([0])
    if own:
        from transformer_decode_kv_gb300 import AttnPlan, SeqPages
        st["pages"] = _kv_pages(st)
        st["plan"] = AttnPlan(st["pages"], n_head=H, dtype=st["q"].dtype, max_tok=tok, max_seq=len(n_kv),
                              max_table=table.size, window=case["window"], n_sink=case["n_sink"])
        if step:
            st["lists"] = SeqPages(st["table"], st["before"], st["free"], st["n_free"], page, n_pages)
        else:
            st["plan"].set(n_new, n_kv, table)


def _prepare_pages(case, st, gen, rng):
    n_kv, n_new = _page_lens(case)
    order = rng.permutation(len(n_kv))
    n_kv, n_new = np.array(n_kv)[order], np.array(n_new)[order]
    page = case["page"]
    held, need = -(-n_kv // page), -(-(n_kv + n_new) // page)
    spare = 50
    n_pages = int(need.sum()) + spare
    perm = rng.permutation(n_pages).astype(np.int32)
    table = np.full((len(n_kv), int(need.max()) + 1), -1, dtype=np.int32)
    at = 0
    for i, m in enumerate(held):
        table[i, :m] = perm[at:at + m]
        at += m
    ints = lambda x: torch.from_numpy(np.asarray(x, dtype=np.int32)).cuda()
    tok = int(n_new.sum()) + case["room"]
    st["before"], st["add"], st["table"] = ints(n_kv), ints(n_new), ints(table)
    st["free"], st["n_free"] = ints(perm[at:]), ints([n_pages - at])
    st["n_pages"] = n_pages
    st["cell"], st["pos"] = ints(np.zeros(tok)), ints(np.zeros(tok))
    st["start"], st["after"], st["left"] = ints(np.zeros(len(n_kv) + 1)), ints(np.zeros(len(n_kv))), ints([0])
    if own:
        from transformer_decode_kv_gb300 import SeqPages
        st["lists"] = SeqPages(st["table"], st["before"], st["free"], st["n_free"], page, n_pages)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    st = {"case": case}
    {"kv": _prepare_kv, "attn": _prepare_attn, "step": _prepare_attn, "pages": _prepare_pages}[case["op"]](
        case, st, gen, np.random.default_rng(seed))
    return st


# ---------------------------------------------------------------- plain forms
def _values(code, b, s):
    """The float32 values of packed codes [..., hd / 2], block scales (bytes) and row scales."""
    grid = torch.tensor(_E2M1 + tuple(-x for x in _E2M1), device=code.device)
    q = grid[torch.stack((code & 15, code >> 4), -1).flatten(-2).long()]
    return (q.unflatten(-1, (-1, 16)) * b.view(torch.float8_e4m3fn).float()[..., None]).flatten(-2) * s[..., None]


def _read(c, page, at):
    """Rows (page, place) of a cache as float32 [n, Hkv, hd]."""
    if "b" not in c:
        return c["c"][page, at].float()
    return _values(c["c"][page, at], c["b"][page, at].contiguous(), c["s"][page, at])


def _write(c, page, at, x):
    if "b" not in c:
        c["c"][page, at] = x.to(c["c"].dtype)
        return
    code, b, s = _quantise(x.float())
    c["c"][page, at] = code[..., ::2] | code[..., 1::2] << 4
    c["b"][page, at] = b.view(torch.uint8)
    c["s"][page, at] = s


def _plain_kv(st):
    """Write the rows of slots >= 0, then read them back (rows of padding stay as they were)."""
    keep = st["slot"] >= 0
    slot = st["slot"][keep].long()
    page, at = slot // st["case"]["page"], slot % st["case"]["page"]
    for x, c, o in ((st["k"], st["kc"], st["ko"]), (st["v"], st["vc"], st["vo"])):
        _write(c, page, at, x[keep])
        o[keep] = _read(c, page, at).to(o.dtype)
    return [st["ko"], st["vo"]]


def _plain_attn(st):
    case = st["case"]
    H, Hkv, hd, page = case["H"], case["Hkv"], case["hd"], case["page"]
    G, W, S = H // Hkv, case["window"], case["n_sink"]
    out, r0 = st["out"], 0
    for i, (nn, nk) in enumerate(zip(st["n_new"], st["n_kv"])):
        j = torch.arange(nk, device="cuda")
        k, v = (_read(c, st["table"][i, j // page].long(), j % page).transpose(0, 1) for c in (st["kc"], st["vc"]))
        p = torch.arange(nk - nn, nk, device="cuda")[:, None]
        vis = j <= p
        if W:
            vis &= (j < S) | (j > p - W)
        q = st["q"][r0:r0 + nn].float().view(nn, Hkv, G, hd)
        for g in range(Hkv):
            s = torch.matmul(q[:, g].reshape(nn * G, hd), k[g].T) / math.sqrt(hd)
            s = s.view(nn, G, nk).masked_fill(~vis[:, None], -math.inf)
            e = torch.exp(s - s.amax(-1, keepdim=True))
            e = e / e.sum(-1, keepdim=True)
            o = torch.matmul(e.view(nn * G, nk), v[g]).view(nn, G, hd)
            out[r0:r0 + nn, g * G:(g + 1) * G] = o.to(out.dtype)
        r0 += nn
    return out


def _plain_pages(st):
    """Pages from the free stack's top for the tokens that need new ones, sequence by sequence; then every
    new token's cell and position."""
    page, table, free = st["case"]["page"], st["table"], st["free"].long()
    before, add = st["before"].long(), st["add"].long()
    held = (before + page - 1) // page
    need = (before + add + page - 1) // page - held
    tok_end, page_end = torch.cumsum(add, 0), torch.cumsum(need, 0)
    # the j-th page taken goes to sequence i
    j = torch.arange(len(free), device="cuda")
    i = torch.searchsorted(page_end, j, right=True).clamp(max=len(add) - 1)
    col = held[i] + j - (page_end - need)[i]
    taken = j < page_end[-1]
    table[i[taken], col[taken]] = free[st["n_free"].long() - 1 - j][taken].int()
    t = torch.arange(len(st["cell"]), device="cuda")
    i = torch.searchsorted(tok_end, t, right=True).clamp(max=len(add) - 1)
    live = t < tok_end[-1]
    p = torch.where(live, before[i] + t - (tok_end - add)[i], 0)
    st["cell"].copy_(torch.where(live, table[i, p // page].long() * page + p % page, -1))
    st["pos"].copy_(torch.where(live, p, -1))
    st["start"][1:] = tok_end
    st["after"].copy_(before + add)
    st["left"].copy_(st["n_free"] - page_end[-1])
    return [st[n] for n in ("table", "cell", "pos", "start", "after", "left")]


def _plain_step(st):
    lists = _plain_pages(st)
    cell, page = st["cell"].long(), st["case"]["page"]
    for x, c in ((st["k"], st["kc"]), (st["v"], st["vc"])):
        _write(c, cell // page, cell % page, x)
    return [_plain_attn(st)] + lists


def run(st):
    op = st["case"]["op"]
    if not own:
        return {"kv": _plain_kv, "attn": _plain_attn, "pages": _plain_pages, "step": _plain_step}[op](st)
    import transformer_decode_kv_gb300 as L
    if op == "kv":
        L.kv_store(st["pages"], st["k"], st["v"], st["slot"])
        L.kv_load(st["pages"], st["slot"], st["ko"], st["vo"])
        return [st["ko"], st["vo"]]
    if op == "attn":
        st["plan"].run(st["q"], st["pages"], st["out"])
        return st["out"]
    L.pages_extend(st["lists"], st["add"], st["cell"], st["pos"], st["start"], n_kv_out=st["after"],
                   n_free_out=st["left"])
    lists = [st[n] for n in ("table", "cell", "pos", "start", "after", "left")]
    if op == "pages":
        return lists
    L.kv_store(st["pages"], st["k"], st["v"], st["cell"])
    st["plan"].set_device(st["start"], st["after"], st["table"], max_new=max(st["n_new"]))
    st["plan"].run(st["q"], st["pages"], st["out"])
    return [st["out"]] + lists


# ---------------------------------------------------------------- work
def _visible(case):
    """Per sequence: (key rows that some new token sees, (token, key) pairs)."""
    W, S = case["window"], case["n_sink"]
    res = []
    for nn, nk in zip(_ints(case["n_new"]), _ints(case["n_kv"])):
        p = np.arange(nk - nn, nk)
        if not W:
            res.append((nk, int((p + 1).sum())))
            continue
        first = max(0, nk - nn - W + 1)                       # the first windowed key of the chunk
        rows = nk - first + min(S, first)
        lo = np.maximum(0, p - W + 1)
        res.append((rows, int((p + 1 - lo + np.minimum(S, lo)).sum())))
    return res


def _row_bytes(case):
    hd = case["hd"]
    return hd // 2 + hd // 16 + 4 if case["cache"] == "f4" else hd * _ES[case["cache"]]


def work(case):
    if case["op"] == "kv":
        m = (case["n"] - case["skip"]) * case["Hkv"] * 2
        # rows in, cells out, cells in, rows out
        return {"bytes": m * 2 * (case["hd"] * _ES[case["act"]] + _row_bytes(case)) + 8 * case["n"],
                "flops": m * case["hd"] * 4}
    if case["op"] == "pages":
        n_kv, n_new = _page_lens(case)
        page, tok = case["page"], sum(n_new) + case["room"]
        taken = sum(-(-(a + b) // page) - -(-a // page) for a, b in zip(n_kv, n_new))
        # lengths in and out, starts, cells and positions, pages from the stack to the table, last pages
        return {"bytes": 20 * len(n_kv) + 8 * tok + 8 * taken, "flops": 4 * tok}
    vis = _visible(case)
    hd, tok = case["hd"], sum(_ints(case["n_new"]))
    n = sum(r for r, _ in vis) * 2 * case["Hkv"] * _row_bytes(case) + 2 * tok * case["H"] * hd * _ES[case["act"]]
    if case["op"] == "step":                                  # the new rows in, their cells, the lengths
        n += 2 * tok * case["Hkv"] * hd * _ES[case["act"]] + 8 * tok + 20 * len(vis)
    return {"bytes": n, "flops": 4 * hd * case["H"] * sum(x for _, x in vis)}


# ---------------------------------------------------------------- 64-bit definitions
def _np(t):
    return t.detach().cpu().numpy()


def _e4m3_table():
    """The value of each of the 256 codes: sign, 4 exponent bits (bias 7), 3 mantissa bits."""
    v = np.empty(256)
    for b in range(256):
        s, e, m = -1.0 if b & 128 else 1.0, (b >> 3) & 15, b & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v[b] = math.nan if (b & 127) == 127 else s * x
    return v


def _nearest(grid, y):
    """The value of the ascending grid (index 0: zero) nearest to y >= 0; ties to the even index."""
    i = np.searchsorted(grid, y).clip(1, len(grid) - 1)
    lo, hi = grid[i - 1], grid[i]
    up = (y - lo > hi - y) | ((y - lo == hi - y) & (i % 2 == 0))
    return np.where(up, hi, lo)


def _round4(x):
    """float64 rows [..., hd] as a 4-bit cache holds them."""
    amax = np.abs(x).max(-1, keepdims=True)
    s = np.where(amax == 0, 1.0, 2.0 ** np.ceil(np.log2(np.maximum(amax, 2.0 ** -300) / 2688.0)))
    y = (x / np.maximum(s, 2.0 ** -126)).reshape(x.shape[:-1] + (-1, 16))
    a = np.abs(y)
    b = np.maximum(_nearest(_e4m3_table()[:127], a.max(-1, keepdims=True) / 6.0), 2.0 ** -9)
    # E2M1: 1 exponent step of halves, then 2 mantissa values to a power of two
    grid = np.array([0, 1, 2, 3, 4, 6, 8, 12]) / 2.0
    q = _nearest(grid, a / b) * b
    return np.copysign(q, y).reshape(x.shape) * np.maximum(s, 2.0 ** -126)


def _exact_kv(case, st):
    keep = _np(st["slot"]) >= 0
    res = []
    for x, o in ((st["k"], st["ko"]), (st["v"], st["vo"])):
        y = _np(o.double()).copy()
        y[keep] = _round4(_np(x.double())[keep])
        res.append(torch.from_numpy(y))
    return res


def _exact_pages(case, st):
    page = case["page"]
    before, add, free = (_np(st[n]).tolist() for n in ("before", "add", "free"))
    table = _np(st["table"]).copy()
    stack = free[:int(_np(st["n_free"])[0])]
    n = len(st["cell"])
    cell, pos, start = [], [], [0]
    for i, (a, b) in enumerate(zip(before, add)):
        for p in range(a, a + b):
            if p % page == 0:
                table[i, p // page] = stack.pop()
            cell.append(int(table[i, p // page]) * page + p % page)
            pos.append(p)
        start.append(start[-1] + b)
    pad = [-1] * (n - len(cell))
    as_int = lambda x: torch.tensor(x, dtype=torch.int32)
    return [torch.from_numpy(table), as_int(cell + pad), as_int(pos + pad), as_int(start),
            as_int([a + b for a, b in zip(before, add)]), as_int([len(stack)])]


def _cells64(c, idx, g, cache, page):
    """Rows idx (cells) of head g as float64."""
    p, at = idx // page, idx % page
    if cache != "f4":
        return c["c"][p, at, g].double()
    grid = torch.tensor([0, 1, 2, 3, 4, 6, 8, 12], dtype=torch.float64, device="cuda") / 2
    e4m3 = torch.from_numpy(_e4m3_table()).cuda()
    raw = c["c"][p, at, g].long()
    x = torch.empty((len(raw), 2 * raw.shape[1]), dtype=torch.float64, device="cuda")
    for half in range(2):
        n = raw >> 4 * half & 15
        x[:, half::2] = torch.where(n > 7, -1.0, 1.0).double() * grid[n & 7]
    x *= e4m3[c["b"][p, at, g].long()].repeat_interleave(16, 1)
    return x * c["s"][p, at, g].double()[:, None]


def _exact_attn(case, st):
    H, Hkv, hd, page = case["H"], case["Hkv"], case["hd"], case["page"]
    G, r0, rows = H // Hkv, 0, []
    for i, (nn, nk) in enumerate(zip(st["n_new"], st["n_kv"])):
        j = torch.arange(nk, device="cuda")
        idx = st["table"][i].long()[j // page] * page + j % page
        o = torch.zeros((nn, H, hd), dtype=torch.float64, device="cuda")
        for g in range(Hkv):
            k, v = (_cells64(st[n], idx, g, case["cache"], page) for n in ("kc", "vc"))
            step = max(1, (1 << 26) // nk)
            for h in range(g * G, g * G + G):
                for a in range(0, nn, step):
                    q = st["q"][r0 + a:r0 + min(nn, a + step), h].double()
                    p = nk - nn + a + torch.arange(len(q), device="cuda")[:, None]
                    hide = j[None, :] > p
                    if case["window"]:
                        hide |= (p - j[None, :] >= case["window"]) & (j[None, :] >= case["n_sink"])
                    z = (q @ k.T) * hd ** -0.5
                    z[hide] = -math.inf
                    o[a:a + len(q), h] = torch.softmax(z, 1) @ v
        rows.append(o)
        r0 += nn
    return torch.cat(rows)


def _exact_step(case, st):
    """The step's pages, its rows as the cache's type holds them, then the attention."""
    lists = _exact_pages(case, st)
    st["table"].copy_(lists[0])
    cell = lists[1]
    page, at = cell.long() // case["page"], cell.long() % case["page"]
    for x, c in ((st["k"], st["kc"]), (st["v"], st["vc"])):
        if case["cache"] == "f4":
            y = _round4(_np(x.double()))                      # back to codes: y is on the grid of these scales
            amax = np.abs(_np(x.double())).max(-1, keepdims=True)
            s = np.where(amax == 0, 1.0, 2.0 ** np.ceil(np.log2(np.maximum(amax, 2.0 ** -300) / 2688.0)))
            z = (_np(x.double()) / s).reshape(x.shape[:-1] + (-1, 16))
            e4m3 = _e4m3_table()[:127]
            b = np.maximum(_nearest(e4m3, np.abs(z).max(-1) / 6.0), 2.0 ** -9)
            q = (y / s).reshape(z.shape) / b[..., None]
            code = np.searchsorted(np.array([0, 1, 2, 3, 4, 6, 8, 12]) / 2.0, np.abs(q)) + 8 * np.signbit(q)
            code = code.reshape(x.shape).astype(np.uint8)
            put = lambda n, v: c[n].__setitem__((page.cuda(), at.cuda()), torch.from_numpy(v).cuda())
            put("c", code[..., ::2] | code[..., 1::2] << 4)
            put("b", np.searchsorted(e4m3, b).astype(np.uint8))
            put("s", s[..., 0].astype(np.float32))
        else:
            c["c"][page.cuda(), at.cuda()] = x.to(c["c"].dtype)
    return [_exact_attn(case, st)] + lists


def exact(case, seed):
    pairs = 0
    if case["op"] in ("attn", "step"):
        pairs = case["H"] * sum(a * b for a, b in zip(_ints(case["n_new"]), _ints(case["n_kv"])))
    if pairs > 4e9:
        return None
    st = prepare(case, seed)
    return {"kv": _exact_kv, "attn": _exact_attn, "pages": _exact_pages, "step": _exact_step}[case["op"]](case, st)
