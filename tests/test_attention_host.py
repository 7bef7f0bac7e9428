"""Attention operators, checks that need no GPU: the oracle's pins, the rotary
frequencies, and every refusal (each call below returns before its first HIP call)."""
from __future__ import annotations


import itertools
import math

import numpy as np
import pytest
import torch

import cross_model_sparse_amd as mf
from oracle import attention_ref as ref

FAKE = 0x10000          # never dereferenced: validation fails before any use
INV = mf.MF_ERR_INVALID


@pytest.fixture(scope="module")
def L():
    return mf.load()


def last(L):
    return L.mf_last_error().decode()


# ---- oracle pins ---------------------------------------------------------------

@pytest.mark.parametrize("window,sinks", [(0, 0), (5, 0), (7, 3)])
@pytest.mark.parametrize("M,N", [(12, 12), (4, 20)])
def test_oracle_attention_is_torch_attention(window, sinks, M, N):
    g = torch.Generator().manual_seed(M + window)
    H, Hk, d = 4, 2, 16
    Q, K = (torch.randn(s, generator=g, dtype=torch.float64) for s in ((H, M, d), (Hk, N, d)))
    V = torch.randn(N, Hk, d, generator=g, dtype=torch.float64)
    sc = torch.rand(H, generator=g, dtype=torch.float64)
    keep = torch.tensor(np.stack([ref.visible(N - M + i, N, window, sinks) for i in range(M)]))
    want = torch.nn.functional.scaled_dot_product_attention(
        Q * sc[:, None, None], K.repeat_interleave(H // Hk, 0),
        V.transpose(0, 1).repeat_interleave(H // Hk, 0), attn_mask=keep, scale=1.0)
    r = ref.attention(Q.numpy(), K.numpy(), V.numpy(), sc.numpy(), window, sinks)
    assert np.allclose(r["O"].transpose(1, 0, 2), want.numpy(), atol=1e-12)
    assert np.isclose(r["mass"].sum(), H * M)
    # the mask, by hand: position 9 of 10 keys, window 3, two sinks
    assert np.flatnonzero(ref.visible(9, 10, 3, 2)).tolist() == [0, 1, 7, 8, 9]


def test_oracle_decode_is_the_last_query_of_a_prompt():
    rng = np.random.default_rng(1)
    n, page, Hk, H, d = 11, 4, 2, 4, 8
    K, V = rng.standard_normal((2, 3, Hk, page, d))
    table = np.array([[2, 0, 1]])
    Q, sc = rng.standard_normal((1, H, d)), rng.random(H)
    Ks = K[table[0]].transpose(1, 0, 2, 3).reshape(Hk, -1, d)[:, :n]
    Vs = V[table[0]].transpose(1, 0, 2, 3).reshape(Hk, -1, d)[:, :n]
    a = ref.decode(Q, K, V, [n], table, sc, 6, 1)
    b = ref.attention(Q[0][:, None], Ks, Vs.transpose(1, 0, 2), sc, 6, 1)
    assert np.allclose(a["O"][0], b["O"][0]) and np.allclose(a["lse"][0], b["lse"][:, 0])
    assert np.allclose(a["mass"][0], b["mass"])
    # a page outside the pool takes its rows away
    c = ref.decode(Q, K, V, [n], np.array([[2, 9, 1]]), sc)
    assert (c["mass"][0][:, 4:8] == 0).all() and np.allclose(c["mass"][0].sum(), H)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_oracle_rotation_is_complex_multiplication(layout):
    rng = np.random.default_rng(2)
    x, pos, f = rng.standard_normal((3, 2, 10)), np.array([0, 5, 100000]), rng.random(3)
    y = ref.norm_rope(x, None, 0.0, f, pos, layout, 2.0)
    for i in range(3):
        a, b = (2 * i, 2 * i + 1) if layout == "interleaved" else (i, i + 3)
        z = (x[..., a] + 1j * x[..., b]) * np.exp(1j * pos * f[i])[:, None] * 2.0
        assert np.allclose(y[..., a], z.real) and np.allclose(y[..., b], z.imag)
    assert np.array_equal(y[..., 6:], x[..., 6:])
    n = ref.norm_rope(x, np.ones(10), 0.0, [], pos, layout, 1.0)
    assert np.allclose((n * n).mean(-1), 1)


def test_oracle_eviction_is_the_heaviest_subset():
    rng = np.random.default_rng(3)
    for _ in range(30):
        n, budget = 8, int(rng.integers(1, 8))
        sinks = int(rng.integers(0, budget + 1))
        recent = int(rng.integers(0, budget - sinks + 1))
        m = rng.integers(0, 4, n).astype(float)
        forced = set(range(sinks)) | set(range(n - recent, n))
        best = max((c for c in itertools.combinations(range(n), budget) if forced <= set(c)),
                   key=lambda c: (sum(m[list(c)]), [-j for j in c]))
        got = ref.evict_rows(m, n, budget, sinks, recent)
        # the same mass, and among equals the same rows lowest first
        assert sum(m[got]) == sum(m[list(best)]) and got == sorted(got) and len(got) == budget
        free = [j for j in range(n) if j not in got]
        assert all(m[j] < m[k] or (m[j] == m[k] and j > k)
                   for j in free for k in got if k not in forced)
    assert ref.evict_rows(np.array([np.nan, 0.0, -np.inf, 1.0]), 4, 3, 0, 0) == [0, 1, 3]


# ---- frequencies ---------------------------------------------------------------

def test_rope_frequencies():
    f, a = mf.rope_frequencies(128, 1e6)
    want = 1e6 ** (-np.arange(0, 128, 2) / 128.0)
    assert a == 1.0 and np.allclose(f.numpy(), want, rtol=1e-14)
    f, _ = mf.rope_frequencies(128, 1e6, "linear", 4.0)
    assert np.allclose(f.numpy(), want / 4, rtol=1e-14)
    f, _ = mf.rope_frequencies(128, 1e6, "ntk", 4.0)
    # the slowest pair slows down by the whole factor, the fastest not at all
    assert np.isclose(f[-1], want[-1] / 4, rtol=1e-12) and f[0] == 1.0
    f, a = mf.rope_frequencies(128, 1e6, "yarn", 4.0, orig_len=4096)
    r = f.numpy() / want
    assert np.isclose(a, 0.1 * math.log(4) + 1)
    assert (np.diff(r) <= 1e-15).all() and r[0] == 1.0 and np.isclose(r[-1], 0.25)
    turns = 4096 * want / (2 * np.pi)             # over the original length
    assert np.allclose(r[turns > 40], 1) and np.allclose(r[turns < 0.8], 0.25)


@pytest.mark.parametrize("kw", [dict(rot=0), dict(rot=7), dict(rot=258), dict(base=1.0),
                                dict(base=float("nan")), dict(base=float("inf")), dict(factor=0.5),
                                dict(factor=float("nan")), dict(scaling="other"),
                                dict(scaling="yarn"), dict(scaling="ntk", rot=2),
                                dict(scaling="yarn", orig_len=10.0, beta_fast=1.0),
                                dict(scaling="yarn", orig_len=10.0, beta_slow=0.0)])
def test_rope_frequencies_refusals(kw):
    a = dict(rot=64, base=1e4, factor=2.0)
    a.update(kw)
    with pytest.raises(mf.MapflowError):
        mf.rope_frequencies(**a)


# ---- refusals at the C boundary ------------------------------------------------

def rope(L, cache=False, **kw):
    a = dict(dt=2, N=8, d=128, q=FAKE, Hq=8, ldq=1280, k=FAKE + 16, Hk=2, ldk=1280, v=FAKE + 32, ldv=1280,
             wq=FAKE, wk=FAKE, eps=1e-6, freq=FAKE, rot=128, layout=0, af=1.0, pos=FAKE,
             Q=2 * FAKE, ldQ=1024, hsQ=128, K=3 * FAKE, ldK=256, hsK=128, slots=FAKE, V=4 * FAKE,
             n_pages=4, page=16)
    a.update(kw)
    head = (a["dt"], a["N"], a["d"], a["q"], a["Hq"], a["ldq"], a["k"], a["Hk"], a["ldk"])
    norm = (a["wq"], a["wk"], a["eps"], a["freq"], a["rot"], a["layout"], a["af"], a["pos"], a["Q"],
            a["ldQ"], a["hsQ"])
    if cache:
        return L.mf_qk_norm_rope_cache(*head, a["v"], a["ldv"], *norm, a["slots"], a["K"], a["V"],
                                       a["n_pages"], a["page"], None)
    return L.mf_qk_norm_rope(*head, *norm, a["K"], a["ldK"], a["hsK"], None)


@pytest.mark.parametrize("cache", [False, True])
@pytest.mark.parametrize("kw,frag", [
    (dict(dt=3), "dtype"), (dict(N=-1), "N < 0"), (dict(d=96), "d must"), (dict(Hq=0), "head"),
    (dict(Hk=65), "head"), (dict(rot=130), "rot"), (dict(rot=31), "rot"), (dict(rot=-2), "rot"),
    (dict(layout=2), "layout"), (dict(eps=-1.0), "eps"), (dict(eps=float("nan")), "eps"),
    (dict(ldq=1023), "ldq"), (dict(ldk=255), "ldk"), (dict(ldQ=1000), "overlap"), (dict(hsQ=64), "overlap"),
    (dict(q=None), "null"), (dict(k=None), "null"), (dict(Q=None), "null"), (dict(freq=None), "null"),
    (dict(pos=None), "null"), (dict(K=None), "null"),
    (dict(Q=FAKE, ldQ=1280, hsQ=256, d=128, Hq=4, ldq=1280), "overlaps"),
])
def test_rope_refusals(L, cache, kw, frag):
    assert rope(L, cache, **kw) == INV
    assert frag in last(L)


@pytest.mark.parametrize("kw,frag", [
    (dict(v=None), "null"), (dict(slots=None), "null"), (dict(V=None), "null pool"), (dict(ldv=100), "ldv"),
    (dict(page=0), "page"), (dict(n_pages=-1), "n_pages"), (dict(K=3 * FAKE + 2), "16-byte"),
    (dict(V=3 * FAKE), "one pool")])
def test_rope_cache_refusals(L, kw, frag):
    assert rope(L, True, **kw) == INV
    assert frag in last(L)


def test_rope_of_nothing(L):
    assert rope(L, N=0, q=None, k=None, Q=None, K=None) == mf.MF_OK
    assert rope(L, True, N=0, q=None, k=None, Q=None, v=None) == mf.MF_OK


def attn(L, varlen=False, **kw):
    a = dict(Q=FAKE, K=2 * FAKE, V=3 * FAKE, ldQ=128, hsQ=12800, ldK=128, hsK=12800, ldV=256, hsV=128, dt=2,
             H=8, Hk=2, Nq=100, Nk=100, d=128, scale=FAKE, window=0, sinks=0, O=4 * FAKE, ldO=1024,
             lse=FAKE, S=2, cq=FAKE, ck=FAKE, ws=None, wsb=0)
    a.update(kw)
    body = (a["Q"], a["ldQ"], a["hsQ"], a["K"], a["ldK"], a["hsK"], a["V"], a["ldV"], a["hsV"], a["dt"],
            a["H"], a["Hk"], a["Nq"], a["Nk"], a["d"], a["scale"], a["window"], a["sinks"], a["O"], a["ldO"],
            a["lse"])
    if varlen:
        return L.mf_attention_window_varlen(a["S"], a["cq"], a["ck"], *body, None)
    return L.mf_attention_window(*body, a["ws"], a["wsb"], None)


@pytest.mark.parametrize("varlen", [False, True])
@pytest.mark.parametrize("kw,frag", [
    (dict(dt=-1), "dtype"), (dict(H=0), "head"), (dict(H=66, Hk=2), "head"), (dict(Hk=3), "multiple"),
    (dict(Hk=0), "multiple"), (dict(d=32), "d must"), (dict(Nq=-1), "N_q"), (dict(Nk=-1), "N_k"),
    (dict(window=-1), "window"), (dict(sinks=-1), "sinks"), (dict(ldQ=-1), "stride"), (dict(hsV=-8), "stride"),
    (dict(ldO=1023), "ldO"), (dict(Q=None), "null"), (dict(K=None), "null"), (dict(V=None), "null"),
    (dict(O=None), "null"), (dict(scale=None), "null"), (dict(O=FAKE), "one of the inputs")])
def test_attention_refusals(L, varlen, kw, frag):
    assert attn(L, varlen, **kw) == INV
    assert frag in last(L)


def test_attention_more_refusals(L):
    assert attn(L, True, S=-1) == INV and "S must" in last(L)
    assert attn(L, True, cq=None) == INV and "cu_q" in last(L)
    assert attn(L, ws=FAKE + 4, wsb=1 << 20) == INV and "16 bytes" in last(L)
    # nothing to do
    assert attn(L, Nq=0, Q=None, O=None) == mf.MF_OK
    assert attn(L, True, S=0, cq=None, ck=None) == mf.MF_OK
    for bad in (dict(H=3), dict(d=65), dict(window=-1), dict(dt=9)):
        a = dict(dt=2, H=8, Hk=2, Nq=4, Nk=4096, d=128, window=0, sinks=0)
        a.update(bad)
        assert L.mf_attention_split_workspace_bytes(*a.values()) == 0


def decode(L, **kw):
    a = dict(Q=FAKE, ldQ=1024, K=2 * FAKE, V=3 * FAKE, n_pages=8, page=16, table=FAKE, max_pages=4, lens=FAKE,
             dt=2, S=2, max_len=64, H=8, Hk=2, d=128, scale=FAKE, window=0, sinks=0, O=4 * FAKE, ldO=1024,
             lse=None, mi=None, mo=None, ldm=0, ws=FAKE, wsb=1 << 40)
    a.update(kw)
    return L.mf_attention_decode(*a.values(), None)


@pytest.mark.parametrize("kw,frag", [
    (dict(dt=5), "dtype"), (dict(H=7), "multiple"), (dict(d=256), "d must"), (dict(window=-2), "window"),
    (dict(sinks=-2), "sinks"), (dict(S=-1), "S < 0"), (dict(n_pages=-1), "n_pages"), (dict(page=0), "page"),
    (dict(max_pages=-1), "max_pages"), (dict(max_len=65), "max_len"), (dict(max_len=-1), "max_len"),
    (dict(lens=None), "lens"), (dict(K=None), "pool"), (dict(K=2 * FAKE + 8), "16-byte"), (dict(ldQ=1000), "ldQ"),
    (dict(ldO=1000), "ldO"), (dict(mi=FAKE), "mass_in"), (dict(mo=FAKE, ldm=63), "ldmass"), (dict(Q=None), "null"),
    (dict(O=None), "null"), (dict(scale=None), "null"), (dict(O=2 * FAKE), "one of the inputs"),
    (dict(mo=FAKE, ldm=64, ws=None), "workspace"), (dict(mo=FAKE, ldm=64, wsb=0), "workspace"),
    (dict(ws=FAKE + 8), "16 bytes")])
def test_decode_refusals(L, kw, frag):
    assert decode(L, **kw) == INV
    assert frag in last(L)


def test_decode_of_nothing_and_workspace_sizes(L):
    assert decode(L, S=0, Q=None, O=None, lens=None, K=None, V=None) == mf.MF_OK
    f = mf.attention_decode_workspace_bytes
    assert f(0, 64, 8, 2, 128) == 0 and f(1, -1, 8, 2, 128) == 0 and f(1, 64, 8, 3, 128) == 0
    assert f(4, 64, 8, 2, 128, with_mass=True) >= f(4, 64, 8, 2, 128)


def kmass(L, **kw):
    a = dict(Q=FAKE, ldQ=128, hsQ=12800, K=2 * FAKE, ldK=128, hsK=12800, scale=FAKE, lse=FAKE, dt=2, H=8, Hk=2,
             Nq=100, Nk=100, d=128, window=0, sinks=0, mi=None, mo=FAKE, ws=FAKE, wsb=1 << 40)
    a.update(kw)
    return L.mf_key_mass_qk(*a.values(), None)


@pytest.mark.parametrize("kw,frag", [
    (dict(dt=5), "dtype"), (dict(Hk=5), "multiple"), (dict(d=0), "d must"), (dict(Nq=-1), "N_q"),
    (dict(Nk=-5), "N_k"), (dict(window=-1), "window"), (dict(sinks=-1), "sinks"), (dict(ldK=-1), "stride"),
    (dict(K=None), "null"), (dict(Q=None), "null"), (dict(lse=None), "null"), (dict(scale=None), "null"),
    (dict(mo=None), "null"), (dict(ws=FAKE + 4), "16 bytes")])
def test_key_mass_refusals(L, kw, frag):
    assert kmass(L, **kw) == INV
    assert frag in last(L)
    assert kmass(L, Nk=0, K=None, mo=None) == mf.MF_OK


def evict(L, **kw):
    a = dict(mass=FAKE, ldm=64, K=2 * FAKE, V=3 * FAKE, n_pages=8, page=16, table=FAKE, max_pages=4, lens=FAKE,
             dt=2, S=2, max_len=64, Hk=2, d=128, budget=32, sinks=4, recent=8, Ko=4 * FAKE, Vo=5 * FAKE, cap=32,
             mo=None, kept=FAKE, lo=None)
    a.update(kw)
    return L.mf_cache_evict(*a.values(), None)


@pytest.mark.parametrize("kw,frag", [
    (dict(dt=4), "dtype"), (dict(Hk=0), "head"), (dict(d=100), "d must"), (dict(S=-1), "S < 0"),
    (dict(n_pages=-1), "n_pages"), (dict(page=0), "page"), (dict(max_len=65, ldm=100), "max_len"),
    (dict(budget=0), "budget"), (dict(sinks=-1), "sinks"), (dict(recent=-1), "recent"),
    (dict(sinks=30), "together"), (dict(cap=31), "cap_out"), (dict(ldm=63), "ldmass"), (dict(mass=None), "null"),
    (dict(kept=None), "null"), (dict(Ko=None), "null"), (dict(Vo=None), "null"), (dict(lens=None), "lens"),
    (dict(Ko=2 * FAKE), "source"), (dict(Vo=4 * FAKE), "other output"), (dict(Ko=4 * FAKE + 2), "16-byte"),
    (dict(mo=FAKE), "mass_out is mass")])
def test_evict_refusals(L, kw, frag):
    assert evict(L, **kw) == INV
    assert frag in last(L)
    assert evict(L, S=0, mass=None, kept=None, Ko=None, Vo=None, lens=None, K=None, V=None) == mf.MF_OK


def test_evict_refuses_lengths_written_in_place(L):
    # one head's workgroup would write lens[s] while the others still read it
    assert evict(L, lo=FAKE) == INV
    assert "lens_out is lens" in last(L)


# ---- refusals of the binding ---------------------------------------------------

def test_binding_refuses_host_tensors():
    h, x, f32 = torch.zeros, torch.bfloat16, torch.float32
    Q, K, V, sc = h(4, 8, 64, dtype=x), h(2, 8, 64, dtype=x), h(8, 2, 64, dtype=x), h(4)
    lens = h(1, dtype=torch.int32)
    pool = h(1, 2, 8, 64, dtype=x)
    calls = [
        lambda: mf.attention_window(Q, K, V, sc),
        lambda: mf.attention_window_varlen(Q, K, V, sc, h(2, dtype=torch.int32), h(2, dtype=torch.int32)),
        lambda: mf.attention_decode(h(1, 4, 64, dtype=x), pool, pool, lens, sc, 8),
        lambda: mf.key_mass_qk(Q, K, sc, h(4, 8)),
        lambda: mf.cache_evict(h(1, 2, 8), pool, pool, lens, 4),
        lambda: mf.qk_norm_rope(h(3, 4, 64, dtype=x), h(3, 2, 64, dtype=x), None, None),
    ]
    for c in calls:
        with pytest.raises(mf.MapflowError, match="GPU"):
            c()


def test_binding_refuses_shapes_and_types():
    h, x = torch.zeros, torch.bfloat16
    Q, K, V, sc = h(4, 8, 64, dtype=x), h(2, 8, 64, dtype=x), h(8, 2, 64, dtype=x), h(4)
    pool, lens = h(2, 2, 8, 64, dtype=x), h(2, dtype=torch.int32)
    q3 = h(2, 4, 64, dtype=x)
    bad = [
        lambda: mf.attention_window(Q.double(), K.double(), V.double(), sc),
        lambda: mf.attention_window(Q, K, V.half(), sc),
        lambda: mf.attention_window(Q, K, V.transpose(0, 1), sc),
        lambda: mf.attention_window(Q, K, V, sc.double()),
        lambda: mf.attention_window(Q, K, V, h(5)),
        lambda: mf.attention_window(Q[..., ::2], K[..., ::2], V[..., ::2], sc),
        lambda: mf.attention_window_varlen(Q, K, V, sc, lens.long(), lens),
        lambda: mf.attention_window_varlen(Q, K, V, sc, lens, h(3, dtype=torch.int32)),
        lambda: mf.attention_decode(q3, pool, pool[:1], lens, sc, 8),
        lambda: mf.attention_decode(q3, pool, pool, lens[:1], sc, 8),
        lambda: mf.attention_decode(q3.half(), pool, pool, lens, sc, 8),
        lambda: mf.attention_decode(q3, pool, pool, lens, sc, 8, block_table=lens),
        lambda: mf.attention_decode(q3, pool, pool, lens, sc, 8, mass_in=h(2, 2, 8)),
        lambda: mf.attention_decode(q3, pool, pool, lens, sc, 8, mass_out=h(2, 3, 8)),
        # sizes that an int would cut: 2^32 + 5 is not a window of 5
        lambda: mf.attention_window(Q, K, V, sc, window=(1 << 32) + 5),
        lambda: mf.attention_window_varlen(Q, K, V, sc, lens, lens, sinks=1 << 31),
        lambda: mf.attention_decode(q3, pool, pool, lens, sc, (1 << 32) + 8),
        lambda: mf.attention_decode(q3, pool, pool, lens, sc, 8, window=1 << 40),
        lambda: mf.key_mass_qk(Q, K, sc, h(4, 8), window=1 << 33),
        lambda: mf.cache_evict(h(2, 2, 8), pool, pool, lens, (1 << 32) + 4),
        lambda: mf.cache_evict(h(2, 2, 8), pool, pool, lens, 4, recent=1 << 32),
        lambda: mf.key_mass_qk(Q, K, sc, h(4, 9)),
        lambda: mf.key_mass_qk(Q, K, sc, h(4, 8), mass_in=h(4, 8)),
        lambda: mf.cache_evict(h(2, 3, 8), pool, pool, lens, 4),
        lambda: mf.cache_evict(h(2, 2, 8), pool, pool, lens, 0),
        lambda: mf.cache_evict(h(2, 2, 8), pool, pool, lens, 4, K_out=h(2, 2, 4, 32, dtype=x)),
        lambda: mf.qk_norm_rope(q3, q3[:, :2], None, None, layout="other"),
        lambda: mf.qk_norm_rope(q3, q3[:1], None, None),
        lambda: mf.qk_norm_rope(q3, q3, h(32), lens),
        lambda: mf.qk_norm_rope(q3, q3, h(32, dtype=torch.float64), lens.long()),
        lambda: mf.qk_norm_rope(q3, q3, h(32, dtype=torch.float64), None),
        lambda: mf.qk_norm_rope(q3.transpose(0, 1).contiguous().transpose(0, 1), q3, None, None),
    ]
    for i, c in enumerate(bad):
        with pytest.raises(mf.MapflowError) as e:
            c()
        assert e.value.status == INV, i
