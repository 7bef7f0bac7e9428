"""Attention operators beside the map compression: what is measured, and their plain forms.

The sender's layers and the receiver's first layers run attention as usual.  Their operators, in the
order in which a serving step uses them:

  rope    per-head RMS norm of q and k and rotary positions, into head-major Q and K or cache pages
  attn    causal attention with a sliding window and first tokens that stay visible (output, lse)
  decode  one query per sequence over a paged cache, optionally adding each key's weight to a sum
  mass    the same accumulated weight of every key of a prompt, from Q, K and lse
  evict   the cache cut to a budget by accumulated weight

``own`` selects between the plain forms (elementary torch operations in 32 bits) and the library.
"""
import math

import numpy as np
import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ES = {"f32": 4, "f16": 2, "bf16": 2}


# ---- cases ------------------------------------------------------------------

def listed():
    return [
        # four sequences' next tokens, written into their cache pages
        dict(name="rope_tokens", op="rope", dtype="bf16", N=4, H=32, Hk=8, d=128, rot=128,
             layout="half", scaling="plain", cache=True, page=64, far=32768),
        # a whole prompt of the 14B-like sender: Q and K for attention and compression
        dict(name="rope_prompt", op="rope", dtype="bf16", N=8192, H=40, Hk=8, d=128, rot=128,
             layout="half", scaling="yarn", cache=False, page=0, far=8192),
        # a packed batch of short ragged prompts, half of each head rotated elsewhere (d = 64)
        dict(name="attn_packed", op="attn", dtype="f16", lens="1 33 250 1000 7 513 129 2047",
             past=0, H=16, Hk=4, d=64, window=256, sinks=4),
        # full precision, a length of no round number
        dict(name="attn_f32", op="attn", dtype="f32", lens="1000", past=24, H=8, Hk=4, d=128,
             window=0, sinks=0),
        # the receiver's prompt under a sliding window with sinks
        dict(name="attn_window", op="attn", dtype="bf16", lens="8192", past=0, H=32, Hk=8, d=128,
             window=1024, sinks=4),
        # a long prompt, every earlier token visible
        dict(name="attn_long", op="attn", dtype="bf16", lens="32768", past=0, H=32, Hk=8, d=128,
             window=0, sinks=0),
        # one conversation's next token over a long cache
        dict(name="decode_one", op="decode", dtype="bf16", S=1, max_len=32768, H=32, Hk=8, d=128,
             window=0, sinks=0, page=64, ragged=False, mass=False),
        # a serving batch of ragged lengths, adding up each key's weight for eviction
        dict(name="decode_batch", op="decode", dtype="f16", S=64, max_len=8192, H=32, Hk=8, d=128,
             window=4096, sinks=64, page=64, ragged=True, mass=True),
        # a short prompt's accumulated weight
        dict(name="mass_short", op="mass", dtype="f16", N=1000, M=1000, H=32, Hk=8, d=128,
             window=0, sinks=0),
        # the 14B-like sender's prompt
        dict(name="mass_prompt", op="mass", dtype="bf16", N=8192, M=8192, H=40, Hk=8, d=128,
             window=0, sinks=0),
        # one long prompt's cache cut to a quarter
        dict(name="evict_one", op="evict", dtype="bf16", S=1, max_len=8192, Hk=8, d=128,
             budget=2048, sinks=4, recent=64, page=8192, ragged=False),
        # a batch of ragged caches cut to one budget
        dict(name="evict_batch", op="evict", dtype="f16", S=32, max_len=16384, Hk=8, d=128,
             budget=4096, sinks=16, recent=256, page=64, ragged=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "attn", "attn", "decode", "decode", "mass", "evict"])
    dtype = rng.choice(["bf16", "f16", "bf16", "f16", "f32"])
    d = rng.choice([64, 128, 128])
    Hk = rng.choice([1, 2, 4, 5, 8])
    H = Hk * rng.choice([1, 2, 3, 4, 5, 8])
    window = rng.choice([0, _log(rng, 1, 4096)])
    sinks = rng.choice([0, 1, 4, rng.randint(0, 100)]) if window else 0
    if op == "rope":
        cache = rng.random() < 0.5
        return dict(op=op, dtype=dtype, N=_log(rng, 1, 256) if cache else _log(rng, 1, 8192),
                    H=H, Hk=Hk, d=d, rot=rng.choice([d, d, d // 2, d // 4, 20]),
                    layout=rng.choice(["half", "interleaved"]),
                    scaling=rng.choice(["plain", "linear", "ntk", "yarn"]), cache=cache,
                    page=rng.choice([16, 24, 64]) if cache else 0, far=_log(rng, 256, 1000000))
    if op == "attn":
        top = 4096 if dtype == "f32" else 16384
        lens = [_log(rng, 1, top)] if rng.random() < 0.5 else \
            [_log(rng, 1, top // 4) for _ in range(rng.randint(2, 12))]
        return dict(op=op, dtype=dtype, lens=" ".join(map(str, lens)), past=rng.choice([0, 0, rng.randint(1, 500)]),
                    H=H, Hk=Hk, d=d, window=window, sinks=sinks)
    if op == "decode":
        return dict(op=op, dtype=dtype, S=_log(rng, 1, 48), max_len=_log(rng, 1, 8192), H=H, Hk=Hk,
                    d=d, window=window, sinks=sinks, page=rng.choice([16, 24, 64, 128]),
                    ragged=rng.random() < 0.7, mass=rng.random() < 0.5)
    if op == "mass":
        N = _log(rng, 1, 2048 if dtype == "f32" else 8192)
        return dict(op=op, dtype=dtype, N=N, M=rng.choice([N, rng.randint(1, N)]), H=H, Hk=Hk, d=d,
                    window=window, sinks=sinks)
    L = _log(rng, 1, 16384)
    budget = rng.randint(1, L)
    s = rng.randint(0, min(budget, 64))
    return dict(op=op, dtype=dtype, S=_log(rng, 1, 16), max_len=L, Hk=Hk, d=d, budget=budget,
                sinks=s, recent=rng.randint(0, min(budget - s, 256)),
                page=rng.choice([16, 24, 64, 128]), ragged=rng.random() < 0.7)


def _prompts(case):
    """Lengths of the packed prompts."""
    return [int(n) for n in case["lens"].split()]


def _lens(case, seed):
    """Cached lengths of a decode or evict batch (host)."""
    r = np.random.default_rng(seed)
    if not case["ragged"]:
        return np.full(case["S"], case["max_len"], dtype=np.int64)
    n = r.integers(1, case["max_len"] + 1, size=case["S"])
    n[r.integers(0, case["S"])] = case["max_len"]
    return n


def _pairs(M, N, window, sinks):
    """Visible (query, key) pairs of M queries at the end of N keys."""
    p = np.arange(N - M, N, dtype=np.int64)
    w = p + 1 if window == 0 else np.minimum(p + 1, window)
    return int((w + np.minimum(sinks, p + 1 - w)).sum())


# ---- inputs -----------------------------------------------------------------

def _randn(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _table(rng_seed, S, max_len, page):
    """A block table that deals shuffled pool pages to the sequences (host)."""
    per = -(-max_len // page)
    t = np.random.default_rng(rng_seed + 1).permutation(S * per).astype(np.int32)
    return t.reshape(S, per)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DT[case["dtype"]]
    op, d, Hk = case["op"], case["d"], case["Hk"]
    st = dict(case=case)
    if op == "rope":
        N, H = case["N"], case["H"]
        # rows of a fused projection: q heads, k heads, v heads side by side
        x = _randn(g, (N, H + 2 * Hk, d), dt, 1.5)
        st["q"], st["k"], st["v"] = x[:, :H], x[:, H:H + Hk], x[:, H + Hk:]
        st["wq"] = (1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(dt)
        st["wk"] = (1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(dt)
        r = np.random.default_rng(seed)
        if case["cache"]:
            pos = r.integers(0, case["far"], size=N)
            page = case["page"]
            pages = -(-N // page) * 2 + 1
            slots = r.permutation(pages * page)[:N]
            st["slots"] = torch.from_numpy(slots.astype(np.int64)).cuda()
            st["K"] = torch.zeros(pages, Hk, page, d, dtype=dt, device="cuda")
            st["V"] = torch.zeros_like(st["K"])
        else:
            pos = np.arange(max(0, case["far"] - N), max(0, case["far"] - N) + N)
        st["pos"] = torch.from_numpy(pos.astype(np.int32)).cuda()
        f, af = _frequencies(case)
        st["freq"], st["af"] = torch.from_numpy(f).cuda(), af
        return st
    if op == "attn":
        H, past, lens = case["H"], case["past"], _prompts(case)
        M, N = sum(lens), sum(lens) + past * len(lens)
        st["Q"] = _randn(g, (H, M, d), dt)
        st["K"] = _randn(g, (Hk, N, d), dt)
        st["V"] = _randn(g, (N, Hk, d), dt)
        st["scale"] = (torch.rand(H, generator=g, device="cuda") + 0.5) / math.sqrt(d)
        cq = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
        ck = np.concatenate([[0], np.cumsum([n + past for n in lens])]).astype(np.int32)
        st["cq"], st["ck"] = torch.from_numpy(cq).cuda(), torch.from_numpy(ck).cuda()
        return st
    if op == "mass":
        H, N, M = case["H"], case["N"], case["M"]
        st["Q"] = _randn(g, (H, M, d), dt)
        st["K"] = _randn(g, (Hk, N, d), dt)
        st["scale"] = (torch.rand(H, generator=g, device="cuda") + 0.5) / math.sqrt(d)
        # the statistic that the attention of the same layer returned
        st["lse"] = torch.empty(H, M, device="cuda")
        for h, i0, i1, s in _scores(st["Q"], st["K"], st["scale"], case["window"], case["sinks"],
                                    torch.float32):
            st["lse"][h, i0:i1] = torch.logsumexp(s, -1)
        st["mass_in"] = torch.rand(Hk, N, generator=g, device="cuda")
        return st
    S, L, page = case["S"], case["max_len"], case["page"]
    lens, table = _lens(case, seed), _table(seed, S, L, page)
    st["lens_h"] = lens
    st["lens"] = torch.from_numpy(lens.astype(np.int32)).cuda()
    st["table"] = torch.from_numpy(table).cuda()
    st["K"] = _randn(g, (table.size, Hk, page, d), dt)
    st["V"] = _randn(g, (table.size, Hk, page, d), dt)
    if op == "decode":
        st["Q"] = _randn(g, (S, case["H"], d), dt, 1.5)
        st["scale"] = (torch.rand(case["H"], generator=g, device="cuda") + 0.5) / math.sqrt(d)
        if case["mass"]:
            st["mass_in"] = torch.rand(S, Hk, L, generator=g, device="cuda") * 4
            st["mass_out"] = torch.zeros(S, Hk, L, device="cuda")
        return st
    # a few heavy keys, many light ones, some that no query ever saw
    m = torch.randn(S, Hk, L, generator=g, device="cuda").mul_(2).exp_()
    m[torch.rand(S, Hk, L, generator=g, device="cuda") < 0.05] = 0
    st["mass"] = m
    cap = case["budget"] + 16
    st["K_out"] = torch.zeros(S, Hk, cap, d, dtype=dt, device="cuda")
    st["V_out"] = torch.zeros_like(st["K_out"])
    st["mass_out"] = torch.zeros(S, Hk, cap, device="cuda")
    return st


def _frequencies(case):
    """Rotary frequencies (radians a position, 64 bits) and the factor on the rotated dims."""
    rot, base, factor, orig = case["rot"], 1e6, 4.0, 4096.0
    i = np.arange(rot // 2, dtype=np.float64)
    f = base ** (-2.0 * i / rot)
    if case["scaling"] == "linear":
        return f / factor, 1.0
    if case["scaling"] == "ntk":
        return (base * factor ** (rot / (rot - 2.0))) ** (-2.0 * i / rot), 1.0
    if case["scaling"] == "yarn":
        def dim(turns):
            return rot * math.log(orig / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo, hi = max(math.floor(dim(32.0)), 0), min(math.ceil(dim(1.0)), rot - 1)
        ramp = np.clip((i - lo) / max(hi - lo, 1e-3), 0, 1)
        return f / factor * ramp + f * (1 - ramp), 0.1 * math.log(factor) + 1.0
    return f, 1.0


# ---- plain forms ------------------------------------------------------------

def _visible(i0, i1, M, N, window, sinks, device):
    p = torch.arange(i0, i1, device=device)[:, None] + (N - M)
    j = torch.arange(N, device=device)[None, :]
    v = j <= p
    if window:
        v &= (j > p - window) | (j < sinks)
    return v


def _scores(Q, K, scale, window, sinks, wide):
    """(head, first row, end row, masked scores) over blocks of query rows."""
    H, M, d = Q.shape
    Hk, N, _ = K.shape
    step = max(1, min(M, (1 << 28) // max(N, 1)))
    for i0 in range(0, M, step):
        i1 = min(M, i0 + step)
        hidden = ~_visible(i0, i1, M, N, window, sinks, Q.device)
        for h in range(H):
            s = Q[h, i0:i1].to(wide) @ K[h // (H // Hk)].to(wide).t().contiguous()
            s *= scale[h].to(wide)
            yield h, i0, i1, s.masked_fill_(hidden, -math.inf)


def _plain_rope(st):
    c = st["case"]
    q, k, v = st["q"].float(), st["k"].float(), st["v"]
    rot, dt = c["rot"], DT[c["dtype"]]
    ang = st["pos"].double()[:, None] * st["freq"][None, :]
    cos, sin = (ang.cos().float() * st["af"])[:, None], (ang.sin().float() * st["af"])[:, None]

    def one(x, w):
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w.float()
        y = x.clone()
        if c["layout"] == "half":
            a, b = x[..., :rot // 2], x[..., rot // 2:rot]
            y[..., :rot // 2], y[..., rot // 2:rot] = a * cos - b * sin, b * cos + a * sin
        else:
            a, b = x[..., 0:rot:2], x[..., 1:rot:2]
            y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
        return y.to(dt)

    qo, ko = one(q, st["wq"]), one(k, st["wk"])
    if not c["cache"]:
        return qo.transpose(0, 1).contiguous(), ko.transpose(0, 1).contiguous()
    pg, r = st["slots"] // c["page"], st["slots"] % c["page"]
    st["K"][pg, :, r] = ko
    st["V"][pg, :, r] = v
    return qo, st["K"], st["V"]


def _plain_attn(st):
    c, dt = st["case"], DT[st["case"]["dtype"]]
    Q, K, V = st["Q"], st["K"], st["V"]
    O = torch.empty(Q.shape[1], c["H"], c["d"], dtype=dt, device=Q.device)
    lse = torch.empty(c["H"], Q.shape[1], device=Q.device)
    G, q0, k0 = c["H"] // c["Hk"], 0, 0
    for n in _prompts(c):
        q1, k1 = q0 + n, k0 + n + c["past"]
        for h, i0, i1, s in _scores(Q[:, q0:q1], K[:, k0:k1], st["scale"], c["window"], c["sinks"],
                                    torch.float32):
            m = s.max(-1, keepdim=True).values
            e = (s - m).exp_()
            l = e.sum(-1, keepdim=True)
            O[q0 + i0:q0 + i1, h] = ((e @ V[k0:k1, h // G].float()) / l).to(dt)
            lse[h, q0 + i0:q0 + i1] = (m + l.log()).squeeze(-1)
        q0, k0 = q1, k1
    return O, lse


def _cache_rows(pool, table, n, page, s):
    """[H_kv][n][d]: the cached rows of sequence s."""
    x = pool[table[s].long()]
    return x.transpose(0, 1).reshape(x.shape[1], -1, x.shape[3])[:, :n]


def _decode_mask(n, window, sinks, device):
    j = torch.arange(n, device=device)
    return (j >= n - window) | (j < sinks) if window else j >= 0


def _plain_decode(st):
    c, dt = st["case"], DT[st["case"]["dtype"]]
    G = c["H"] // c["Hk"]
    O = torch.empty(c["S"], c["H"], c["d"], dtype=dt, device="cuda")
    for s in range(c["S"]):
        n = int(st["lens_h"][s])
        K = _cache_rows(st["K"], st["table"], n, c["page"], s).float()
        V = _cache_rows(st["V"], st["table"], n, c["page"], s).float()
        q = st["Q"][s].float().view(c["Hk"], G, c["d"]) * st["scale"].view(c["Hk"], G, 1)
        x = torch.bmm(q, K.transpose(1, 2).contiguous())
        seen = _decode_mask(n, c["window"], c["sinks"], x.device)
        x = x.masked_fill(~seen, -math.inf)
        e = (x - x.max(-1, keepdim=True).values).exp()
        p = e / e.sum(-1, keepdim=True)
        O[s] = torch.bmm(p, V).reshape(c["H"], c["d"]).to(dt)
        if c["mass"]:
            st["mass_out"][s, :, :n] = st["mass_in"][s, :, :n] + p.sum(1)
    return (O, st["mass_out"]) if c["mass"] else O


def _plain_mass(st):
    c = st["case"]
    out = st["mass_in"].clone()
    for h, i0, i1, s in _scores(st["Q"], st["K"], st["scale"], c["window"], c["sinks"],
                                torch.float32):
        out[h // (c["H"] // c["Hk"])] += (s - st["lse"][h, i0:i1, None]).exp_().sum(0)
    return out


def _choose(mass, n, budget, sinks, recent):
    """Kept rows of one (sequence, head), ascending."""
    if n <= budget:
        return torch.arange(n, device=mass.device)
    j = torch.arange(n, device=mass.device)
    forced = (j < sinks) | (j >= n - recent)
    rest = j[~forced]
    order = torch.sort(mass[rest], descending=True, stable=True).indices
    top = rest[order[:budget - int(min(sinks, n)) - recent]]
    return torch.sort(torch.cat([j[forced], top])).values


def _plain_evict(st):
    c = st["case"]
    kept = torch.full((c["S"], c["Hk"], c["budget"]), -1, dtype=torch.int32, device="cuda")
    left = torch.empty(c["S"], dtype=torch.int32, device="cuda")
    for s in range(c["S"]):
        n = int(st["lens_h"][s])
        K = _cache_rows(st["K"], st["table"], n, c["page"], s)
        V = _cache_rows(st["V"], st["table"], n, c["page"], s)
        m = min(n, c["budget"])
        left[s] = m
        st["mass_out"][s, :, m:] = 0
        for h in range(c["Hk"]):
            idx = _choose(st["mass"][s, h, :n], n, c["budget"], c["sinks"], c["recent"])
            kept[s, h, :m] = idx.int()
            st["K_out"][s, h, :m] = K[h, idx]
            st["V_out"][s, h, :m] = V[h, idx]
            st["mass_out"][s, h, :m] = st["mass"][s, h, idx]
    return kept, left, st["K_out"], st["V_out"], st["mass_out"]


# ---- the library's calls ----------------------------------------------------

def _own(st):
    import cross_model_sparse_amd as mf
    c = st["case"]
    if c["op"] == "rope":
        kw = dict(wq=st["wq"], wk=st["wk"], eps=1e-6, layout=c["layout"], attn_factor=st["af"])
        if c["cache"]:
            Q = mf.qk_norm_rope(st["q"], st["k"], st["freq"], st["pos"], v=st["v"], K=st["K"],
                                V=st["V"], slots=st["slots"], token_major=True, **kw)[0]
            return Q, st["K"], st["V"]
        return mf.qk_norm_rope(st["q"], st["k"], st["freq"], st["pos"], **kw)
    if c["op"] == "attn":
        if len(_prompts(c)) == 1:
            return mf.attention_window(st["Q"], st["K"], st["V"], st["scale"], window=c["window"],
                                       sinks=c["sinks"])
        return mf.attention_window_varlen(st["Q"], st["K"], st["V"], st["scale"], st["cq"], st["ck"],
                                          window=c["window"], sinks=c["sinks"])
    if c["op"] == "decode":
        kw = dict(window=c["window"], sinks=c["sinks"], block_table=st["table"])
        if c["mass"]:
            O, _ = mf.attention_decode(st["Q"], st["K"], st["V"], st["lens"], st["scale"],
                                       c["max_len"], mass_in=st["mass_in"],
                                       mass_out=st["mass_out"], **kw)
            return O, st["mass_out"]
        return mf.attention_decode(st["Q"], st["K"], st["V"], st["lens"], st["scale"],
                                   c["max_len"], **kw)[0]
    if c["op"] == "mass":
        return mf.key_mass_qk(st["Q"], st["K"], st["scale"], st["lse"], window=c["window"],
                              sinks=c["sinks"], mass_in=st["mass_in"])
    kept, left, K, V, m = mf.cache_evict(st["mass"], st["K"], st["V"], st["lens"], c["budget"],
                                         sinks=c["sinks"], recent=c["recent"],
                                         block_table=st["table"], K_out=st["K_out"],
                                         V_out=st["V_out"], mass_out=st["mass_out"])
    return kept, left, K, V, m


def run(state):
    if own:
        return _own(state)
    return dict(rope=_plain_rope, attn=_plain_attn, decode=_plain_decode, mass=_plain_mass,
                evict=_plain_evict)[state["case"]["op"]](state)


# ---- work -------------------------------------------------------------------

def work(case):
    op, e, d, Hk = case["op"], ES[case["dtype"]], case["d"], case["Hk"]
    if op == "rope":
        n = case["N"] * (case["H"] + Hk * (2 if case["cache"] else 1)) * d
        return {"bytes": 2 * n * e + 4 * case["N"], "flops": 8 * n}
    if op == "attn":
        lens, past = _prompts(case), case["past"]
        M, N = sum(lens), sum(lens) + past * len(lens)
        pairs = sum(_pairs(n, n + past, case["window"], case["sinks"]) for n in lens)
        return {"bytes": (2 * M * case["H"] + 2 * N * Hk) * d * e + 4 * M * case["H"],
                "flops": 4 * d * case["H"] * pairs}
    if op == "mass":
        pairs = _pairs(case["M"], case["N"], case["window"], case["sinks"])
        return {"bytes": (case["M"] * case["H"] + case["N"] * Hk) * d * e + 4 * case["M"] * case["H"]
                + 8 * Hk * case["N"], "flops": 2 * d * case["H"] * pairs}
    # ragged lengths are uniform, so a batch caches half of its longest on average
    S, L = case["S"], case["max_len"]
    n = [L * (i + 0.5) / S for i in range(S - 1)] + [L] if case["ragged"] else [L] * S
    if op == "decode":
        seen = sum(_pairs(1, max(1, int(x)), case["window"], case["sinks"]) for x in n)
        extra = 8 * Hk * sum(n) if case["mass"] else 0
        return {"bytes": 2 * seen * Hk * d * e + 2 * S * case["H"] * d * e + extra,
                "flops": 4 * d * case["H"] * seen}
    kept = sum(min(x, case["budget"]) for x in n)
    return {"bytes": 4 * Hk * sum(n) + kept * Hk * (4 * d * e + 12), "flops": 0}


# ---- definitions in 64 bits -------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    f64 = torch.float64
    op, d, Hk = case["op"], case["d"], case["Hk"]
    if op == "rope":
        rot, n = case["rot"], case["rot"] // 2
        ang = torch.outer(st["pos"].to(f64), st["freq"])
        turn = torch.polar(torch.full_like(ang, st["af"]), ang)[:, None]

        def one(x, w):
            x = x.to(f64)
            x = x / (x.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt() * w.to(f64)
            r = x[..., :rot]
            if case["layout"] == "half":
                z = torch.complex(r[..., :n].contiguous(), r[..., n:].contiguous()) * turn
                r = torch.cat([z.real, z.imag], -1)
            else:
                z = torch.complex(r[..., ::2].contiguous(), r[..., 1::2].contiguous()) * turn
                r = torch.view_as_real(z.resolve_conj()).flatten(-2)
            return torch.cat([r, x[..., rot:]], -1)

        q, k = one(st["q"], st["wq"]), one(st["k"], st["wk"])
        if not case["cache"]:
            return q.permute(1, 0, 2).contiguous(), k.permute(1, 0, 2).contiguous()
        P, _, page, _ = st["K"].shape
        flat = [torch.zeros(P * page, Hk, d, dtype=f64, device="cuda") for _ in range(2)]
        flat[0][st["slots"]], flat[1][st["slots"]] = k, st["v"].to(f64)
        K, V = (t.view(P, page, Hk, d).permute(0, 2, 1, 3).contiguous() for t in flat)
        return q, K, V

    if op in ("attn", "mass"):
        H, G = case["H"], case["H"] // Hk
        lens = _prompts(case) if op == "attn" else [case["M"]]
        past = case["past"] if op == "attn" else case["N"] - case["M"]
        M = sum(lens)
        O = torch.empty(M, H, d, dtype=f64, device="cuda") if op == "attn" else None
        lse = torch.empty(H, M, dtype=f64, device="cuda")
        acc = st["mass_in"].to(f64) if op == "mass" else None
        a = b = 0
        for m in lens:
            n = m + past
            for h in range(H):
                K = st["K"][h // G, b:b + n].to(f64).t().contiguous()
                step = max(1, (1 << 27) // n)
                for i in range(0, m, step):
                    rows = torch.arange(i, min(m, i + step), device="cuda")
                    gap = (rows[:, None] + past) - torch.arange(n, device="cuda")[None]
                    ok = gap >= 0
                    if case["window"]:
                        old = gap >= case["window"]
                        old[:, :case["sinks"]] = False
                        ok &= ~old
                    s = (st["Q"][h, a + rows].to(f64) @ K).mul_(float(st["scale"][h]))
                    s = torch.where(ok, s, torch.full((), -math.inf, dtype=f64, device="cuda"))
                    if op == "mass":
                        acc[h // G] += (s - st["lse"][h, rows, None].to(f64)).exp_().sum(0)
                        continue
                    z = torch.logsumexp(s, 1)
                    lse[h, a + rows] = z
                    O[a + rows, h] = (s - z[:, None]).exp_() @ st["V"][b:b + n, h // G].to(f64)
            a, b = a + m, b + n
        return (O, lse) if op == "attn" else acc

    S, page, lens = case["S"], case["page"], st["lens_h"]
    where = [(st["table"][s].long()[:, None] * page + torch.arange(page, device="cuda")).flatten()
             for s in range(S)]
    pool = {x: st[x].transpose(1, 2).reshape(-1, Hk, d) for x in "KV"}
    if op == "decode":
        G = case["H"] // Hk
        O = torch.empty(S, case["H"], d, dtype=f64, device="cuda")
        mass = torch.zeros(S, Hk, case["max_len"], dtype=f64, device="cuda") if case["mass"] else None
        for s in range(S):
            n = int(lens[s])
            K, V = (pool[x][where[s][:n]].to(f64) for x in "KV")
            age = n - 1 - torch.arange(n, device="cuda")
            old = age >= case["window"] if case["window"] else age < 0
            old[:case["sinks"]] = False
            if case["mass"]:
                mass[s, :, :n] = st["mass_in"][s, :, :n].to(f64)
            for h in range(case["H"]):
                x = (K[:, h // G] @ st["Q"][s, h].to(f64)) * float(st["scale"][h])
                x[old] = -math.inf
                p = torch.softmax(x, 0)
                O[s, h] = p @ V[:, h // G]
                if case["mass"]:
                    mass[s, h // G, :n] += p
        return (O, mass) if case["mass"] else O

    cap, B = st["K_out"].shape[2], case["budget"]
    kept = torch.full((S, Hk, B), -1, dtype=torch.int32, device="cuda")
    K2, V2 = (torch.zeros(S, Hk, cap, d, dtype=f64, device="cuda") for _ in range(2))
    m2 = torch.zeros(S, Hk, cap, dtype=f64, device="cuda")
    mh = st["mass"].cpu().numpy().astype(np.float64)
    for s in range(S):
        n = int(lens[s])
        for h in range(Hk):
            w = mh[s, h, :n].copy()
            w[:case["sinks"]] = np.inf
            if case["recent"]:
                w[max(0, n - case["recent"]):] = np.inf
            idx = np.sort(np.lexsort((np.arange(n), -w))[:B])
            i = torch.from_numpy(idx).cuda()
            kept[s, h, :len(idx)] = i.int()
            src = where[s][i]
            K2[s, h, :len(idx)], V2[s, h, :len(idx)] = pool["K"][src, h].to(f64), pool["V"][src, h].to(f64)
            m2[s, h, :len(idx)] = st["mass"][s, h, i].to(f64)
    left = torch.from_numpy(np.minimum(lens, B).astype(np.int32)).cuda()
    return kept, left, K2, V2, m2
