"""Attention operators against the fp64 oracle (MI355X).

Tolerances are derived in _attention.py before any run."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import cross_model_sparse_amd as mf
from oracle import attention_ref as ref
from _attention import (DT, F, close, host, lse_tol, mass_rel, out_tol, randn, score_err,  # noqa: E402
                        u_of)

pytestmark = pytest.mark.gpu

MASK = 1e30        # written where nothing may be written


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def scales(g, H, d, signs=False):
    s = (torch.rand(H, generator=g) + 0.5) / math.sqrt(d)
    if signs and H > 1:
        s[1::2] *= -1
        s[0] = 0.0
    return s


# ---- norm and rotation -------------------------------------------------------

@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("N,Hq,Hk,d,rot,norm", [
    (1, 1, 1, 64, 64, True), (5, 40, 8, 128, 128, True), (33, 6, 2, 128, 20, True),
    (7, 64, 64, 64, 32, False), (3, 5, 1, 128, 0, True), (2, 3, 3, 64, 62, True)])
def test_norm_rope(gpu, dt, layout, N, Hq, Hk, d, rot, norm):
    g = gen(N * 131 + d + rot)
    x = randn(g, (N, Hq + 2 * Hk, d), dt, 2.0)
    w = [randn(g, (d,), dt) if norm else None for _ in range(2)]
    pos = torch.randint(-5, 1 << 20, (N,), generator=g, dtype=torch.int32)
    freq, af = mf.rope_frequencies(rot, 1e6, "yarn", 8.0, orig_len=4096) if rot else (None, 1.0)
    xd = x.to(gpu)
    wd = [None if t is None else t.to(gpu) for t in w]
    Q, K = mf.qk_norm_rope(xd[:, :Hq], xd[:, Hq:Hq + Hk], None if freq is None else freq.to(gpu),
                           pos.to(gpu), wq=wd[0], wk=wd[1], eps=1e-5, layout=layout, attn_factor=af)
    for got, xs, wt, nm in ((Q, x[:, :Hq], w[0], "Q"), (K, x[:, Hq:Hq + Hk], w[1], "K")):
        fr = [] if freq is None else freq.numpy()
        args = (None if wt is None else host(wt), 1e-5)
        want = ref.norm_rope(host(xs), *args, fr, pos.numpy(), layout, af)
        # norm: 12 additions deep (half of it survives the root), root, division, two
        # products; rotation: cos and sin 4 units, two products, a sum; the factor:
        # under 32 fp32 roundings of |a| + |b|, then one to the storage type
        mag = np.abs(ref.norm_rope(host(xs), *args, [], pos.numpy(), layout, 1.0))
        pair = mag.copy()
        for i in range(rot // 2):
            a, b = (2 * i, 2 * i + 1) if layout == "interleaved" else (i, i + rot // 2)
            pair[..., a] = pair[..., b] = (mag[..., a] + mag[..., b]) * af
        tol = 32 * F * pair + u_of(dt) * np.abs(want) + (2.0 ** -25 if dt == "f16" else 0)
        close(host(got).transpose(1, 0, 2), want, tol, nm)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_norm_rope_strides_in_place_and_off_16_bytes(gpu, dt):
    g = gen(5)
    N, H, Hk, d = 9, 4, 2, 64
    freq, _ = mf.rope_frequencies(32, 1e4)
    x = randn(g, (N, (H + Hk) * d), dt)
    pos = torch.arange(N, dtype=torch.int32, device=gpu)
    a = x.to(gpu).view(N, H + Hk, d)
    Q, K = mf.qk_norm_rope(a[:, :H], a[:, H:], freq.to(gpu), pos, token_major=True)
    # in place: Q is q
    b = x.to(gpu).view(N, H + Hk, d)
    mf.qk_norm_rope(b[:, :H], b[:, H:], freq.to(gpu), pos, token_major=True, Q=b[:, :H], K=b[:, H:])
    assert torch.equal(b[:, :H], Q) and torch.equal(b[:, H:], K)
    # one element into a buffer, an odd row stride
    big = torch.zeros(1 + N * ((H + Hk) * d + 3), dtype=DT[dt], device=gpu)
    rows = big[1:].view(N, -1)
    rows[:, :(H + Hk) * d] = x.to(gpu)
    c = rows[:, :(H + Hk) * d].unflatten(1, (H + Hk, d))
    out = torch.full((1 + N * H * d,), 7.0, dtype=DT[dt], device=gpu)
    Q2, K2 = mf.qk_norm_rope(c[:, :H], c[:, H:], freq.to(gpu), pos, token_major=True,
                             Q=out[1:].view(N, H, d))
    assert torch.equal(Q2, Q) and torch.equal(K2, K) and float(out[0]) == 7.0


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("page", [16, 24, 1])
def test_norm_rope_into_cache(gpu, dt, page):
    g = gen(page)
    N, H, Hk, d, P = 7, 8, 2, 128, 9
    x = randn(g, (N, H + 2 * Hk, d), dt).to(gpu)
    freq, _ = mf.rope_frequencies(d, 1e6)
    pos = torch.randint(0, 30000, (N,), generator=g, dtype=torch.int32).to(gpu)
    w = randn(g, (d,), dt).to(gpu)
    slots = torch.randperm(P * page, generator=g)[:N]
    slots[2], slots[5] = -1, P * page              # skipped
    K = torch.full((P, Hk, page, d), MASK if dt == "f32" else 99.0, dtype=DT[dt], device=gpu)
    V = K.clone()
    K0 = K.clone()
    kw = dict(wq=w, wk=w, token_major=True)
    Q, K1, V1 = mf.qk_norm_rope(x[:, :H], x[:, H:H + Hk], freq.to(gpu), pos, v=x[:, H + Hk:], K=K, V=V,
                                slots=slots.to(gpu), **kw)
    Qr, Kr = mf.qk_norm_rope(x[:, :H], x[:, H:H + Hk], freq.to(gpu), pos, **kw)
    assert K1 is K and V1 is V and torch.equal(Q, Qr)
    wantK, wantV = K0.clone(), K0.clone()
    for n in range(N):
        s = int(slots[n])
        if 0 <= s < P * page:
            wantK[s // page, :, s % page] = Kr[n]
            wantV[s // page, :, s % page] = x[n, H + Hk:]
    assert torch.equal(K, wantK) and torch.equal(V, wantV)


# ---- attention of prompts ----------------------------------------------------

def run_attention(gpu, dt, M, N, H, Hk, d, window, sinks, seed=0, signs=False, std=1.0):
    g = gen(seed * 7919 + M * 31 + N)
    Q, K, V = randn(g, (H, M, d), dt, std), randn(g, (Hk, N, d), dt, std), randn(g, (N, Hk, d), dt)
    sc = scales(g, H, d, signs)
    O, lse = mf.attention_window(Q.to(gpu), K.to(gpu), V.to(gpu), sc.to(gpu), window=window, sinks=sinks)
    r = ref.attention(host(Q), host(K), host(V), host(sc), window, sinks)
    check_attention(dt, O, lse, r, N, d, float(V.abs().max()) if N else 0.0)
    return Q, K, V, sc, O, lse, r


def check_attention(dt, O, lse, r, n, d, vmax, what=""):
    close(host(O), r["O"], out_tol(dt, r["O"], r["A"], r["bound"].T, n, d, vmax), what + "O")
    close(host(lse), r["lse"], lse_tol(r["lse"], r["bound"], n, d), what + "lse")


SHAPES = [
    # M, N, H, Hk, d, window, sinks
    (1, 1, 1, 1, 64, 0, 0),
    (1, 300, 4, 2, 128, 0, 0),
    (37, 37, 8, 8, 64, 0, 0),
    (129, 129, 6, 2, 128, 0, 0),
    (64, 200, 5, 1, 128, 16, 3),
    (200, 200, 4, 4, 128, 1, 0),
    (257, 300, 3, 1, 64, 33, 70),
    (150, 150, 2, 2, 128, 64, 1),
    (300, 411, 16, 2, 128, 100, 5),
    (90, 40, 4, 2, 64, 0, 0),          # more queries than keys: the first 50 see nothing
    (70, 65, 2, 1, 128, 8, 2),
    (20, 0, 2, 1, 128, 0, 0),          # no keys at all
]


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,N,H,Hk,d,window,sinks", SHAPES)
def test_attention(gpu, dt, M, N, H, Hk, d, window, sinks):
    run_attention(gpu, dt, M, N, H, Hk, d, window, sinks)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_attention_scales_of_either_sign(gpu, dt):
    run_attention(gpu, dt, 100, 140, 6, 3, 128, 50, 2, seed=3, signs=True)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_attention_large_scores(gpu, dt):
    # scores of hundreds: without the running maximum every exponential overflows
    run_attention(gpu, dt, 130, 130, 2, 1, 64, 0, 0, seed=4, std=12.0)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("fill", [float("nan"), float("inf"), float("-inf"), "lowest"])
def test_masked_keys_reach_nothing(gpu, dt, fill):
    """Keys 10..29 lie outside window and sinks of the queries from 64 on, and the
    last keys are causal for the last queries only: non-finite rows there leave every
    query that does not see them as it was."""
    fill = torch.finfo(DT[dt]).min if fill == "lowest" else fill
    g = gen(11)
    M = N = 200
    H, Hk, d, window, sinks = 4, 2, 128, 32, 4
    Q, K, V = randn(g, (H, M, d), dt), randn(g, (Hk, N, d), dt), randn(g, (N, Hk, d), dt)
    sc = scales(g, H, d)
    r = ref.attention(host(Q), host(K), host(V), host(sc), window, sinks)
    bad = list(range(10, 30)) + [197]
    K[:, bad] = fill
    V[bad] = fill
    O, lse = mf.attention_window(Q.to(gpu), K.to(gpu), V.to(gpu), sc.to(gpu), window=window, sinks=sinks)
    clean = [i for i in range(M) if not any(ref.visible(i, N, window, sinks)[j] for j in bad)]
    assert len(clean) > 120
    tol = out_tol(dt, r["O"], r["A"], r["bound"].T, N, d, float(r["A"].max()) * 4)
    close(host(O)[clean], r["O"][clean], tol[clean], "O")
    close(host(lse)[:, clean], r["lse"][:, clean], lse_tol(r["lse"], r["bound"], N, d)[:, clean], "lse")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_visible_nan_and_infinity_come_through(gpu, dt):
    g = gen(12)
    N, d = 96, 64
    Q, K, V = randn(g, (1, N, d), dt), randn(g, (1, N, d), dt), randn(g, (N, 1, d), dt)
    V[70, 0, 5] = float("inf")
    V[80, 0, 6] = float("nan")
    sc = torch.full((1,), 0.1)
    O, _ = mf.attention_window(Q.to(gpu), K.to(gpu), V.to(gpu), sc.to(gpu))
    O = host(O)[:, 0]
    assert np.isfinite(O[:70]).all()
    assert (O[70:, 5] == np.inf).all() and np.isfinite(O[70:80, [0, 6]]).all()
    assert np.isnan(O[80:, 6]).all() and np.isfinite(O[80:, 7]).all()


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
def test_attention_strided_inputs_and_output(gpu, dt, d):
    g = gen(21)
    N, H, Hk, window = 83, 4, 2, 40
    x = randn(g, (N, H + 2 * Hk, d), dt)
    sc = scales(g, H, d)
    xd = x.to(gpu)
    Q, K, V = xd[:, :H].transpose(0, 1), xd[:, H:H + Hk].transpose(0, 1), xd[:, H + Hk:]
    big = torch.full((N, H + 1, d), 3.0, dtype=DT[dt], device=gpu)
    O, lse = mf.attention_window(Q, K, V, sc.to(gpu), window=window, out=big[:, :H])
    O2, lse2 = mf.attention_window(Q.contiguous(), K.contiguous(), V.contiguous(), sc.to(gpu), window=window)
    assert torch.equal(O, O2) and torch.equal(lse, lse2) and (big[:, H] == 3.0).all()
    # V head-major, K off 16 bytes: another kernel, the same attention
    off = torch.zeros(K.numel() + 1, dtype=DT[dt], device=gpu)
    off[1:] = K.contiguous().flatten()
    Vh = V.transpose(0, 1).contiguous().transpose(0, 1)
    O3, lse3 = mf.attention_window(Q, off[1:].view(Hk, N, d), Vh, sc.to(gpu), window=window)
    r = ref.attention(host(Q), host(K), host(V), host(sc), window, 0)
    check_attention(dt, O, lse, r, N, d, float(x.abs().max()))
    check_attention(dt, O3, lse3, r, N, d, float(x.abs().max()), "off 16 bytes: ")
    # one K and V head shared by stride 0
    O4, _ = mf.attention_window(Q, K[:1].expand(Hk, N, d), V[:, :1].expand(N, Hk, d), sc.to(gpu))
    O5, _ = mf.attention_window(Q, K[:1].repeat(Hk, 1, 1), V[:, :1].repeat(1, Hk, 1), sc.to(gpu))
    assert torch.equal(O4, O5)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (20, 3)])
def test_attention_packed_batch(gpu, dt, window, sinks):
    g = gen(31)
    qn, kn = [0, 1, 70, 0, 33, 5, 129, 2], [0, 1, 70, 9, 200, 0, 140, 1]
    H, Hk, d = 4, 2, 64
    M, N = sum(qn) + 6, sum(kn) + 9                # rows behind the last sequence
    Q, K, V = randn(g, (H, M, d), dt), randn(g, (Hk, N, d), dt), randn(g, (N, Hk, d), dt)
    sc = scales(g, H, d)
    cq, ck = np.concatenate([[0], np.cumsum(qn)]), np.concatenate([[0], np.cumsum(kn)])
    O = torch.full((M, H, d), 5.0, dtype=DT[dt], device=gpu)
    lse = torch.full((H, M), 5.0, device=gpu)
    V2 = V.clone()
    V2[sum(kn):] = float("nan")
    K2 = K.clone()
    K2[:, sum(kn):] = float("nan")
    mf.attention_window_varlen(Q.to(gpu), K2.to(gpu), V2.to(gpu), sc.to(gpu),
                               torch.tensor(cq, dtype=torch.int32, device=gpu),
                               torch.tensor(ck, dtype=torch.int32, device=gpu), window=window, sinks=sinks,
                               out=O, lse=lse)
    for s in range(len(qn)):
        a, b, c, e = cq[s], cq[s + 1], ck[s], ck[s + 1]
        r = ref.attention(host(Q[:, a:b]), host(K[:, c:e]), host(V[c:e]), host(sc), window, sinks)
        check_attention(dt, O[a:b], lse[:, a:b], r, max(1, e - c), d, float(V.abs().max()), f"seq {s} ")
    assert (O[sum(qn):] == 5.0).all() and (lse[:, sum(qn):] == 5.0).all()


def test_attention_table_beyond_the_buffers_stays_inside(gpu):
    """Offsets past the totals are clamped: nothing outside is read or written."""
    g = gen(32)
    Q, K, V = randn(g, (2, 40, 64), "bf16"), randn(g, (2, 40, 64), "bf16"), randn(g, (40, 2, 64), "bf16")
    sc = scales(g, 2, 64).to(gpu)
    cu = torch.tensor([0, 10, 1000], dtype=torch.int32, device=gpu)
    O, lse = mf.attention_window_varlen(Q.to(gpu), K.to(gpu), V.to(gpu), sc, cu, cu)
    ok = torch.tensor([0, 10, 40], dtype=torch.int32, device=gpu)
    O2, lse2 = mf.attention_window_varlen(Q.to(gpu), K.to(gpu), V.to(gpu), sc, ok, ok)
    assert torch.equal(O, O2) and torch.equal(lse, lse2)


def test_attention_lse_feeds_the_compression(gpu):
    g = gen(33)
    N, H, Hk, d = 300, 4, 2, 128
    Q, K, V = (randn(g, s, "bf16").to(gpu) for s in ((H, N, d), (Hk, N, d), (N, Hk, d)))
    sc = scales(g, H, d).to(gpu)
    _, lse = mf.attention_window(Q, K, V, sc)
    # both within (d + 6) 2^-24 sum |q k| scale, and the sums stay below 32
    assert torch.allclose(lse, mf.row_lse(Q, K, sc), rtol=0, atol=2 * (d + 6) * F * 32)
    m1 = mf.block_mass_qk(Q, K, sc, lse, 64)
    # the mass of the map's column blocks is the sum of their keys' masses
    keys = mf.key_mass_qk(Q, K, sc, lse).sum(0)
    cols = torch.stack([c.sum() for c in keys.split(64)])
    assert torch.allclose(m1.sum(0) * H, cols, rtol=8 * (d + 6) * F * 32, atol=1e-3)


# ---- single tokens over a cache ----------------------------------------------

def make_cache(g, dt, lens, Hk, d, page, gpu, spare=3):
    per = [-(-max(n, 1) // page) for n in lens]
    mp, S = max(per), len(lens)
    P = sum(per) + spare
    order = torch.randperm(P, generator=g)
    table = torch.full((S, mp), -7, dtype=torch.int32)
    at = 0
    for s in range(S):
        table[s, :per[s]] = order[at:at + per[s]].int()
        at += per[s]
    K, V = randn(g, (P, Hk, page, d), dt), randn(g, (P, Hk, page, d), dt)
    return K, V, table


DECODE = [
    # lens, H, Hk, d, page, window, sinks
    ([1], 1, 1, 64, 16, 0, 0),
    ([0, 1, 2, 17], 4, 2, 128, 16, 0, 0),
    ([100, 33, 64, 65], 8, 2, 128, 24, 0, 0),
    ([300], 40, 8, 128, 64, 0, 0),
    ([500, 7, 129], 16, 1, 64, 100, 50, 3),
    ([40, 41, 1000], 64, 2, 128, 32, 64, 33),
    ([2500, 31], 6, 2, 128, 64, 0, 0),
    ([3001], 24, 8, 64, 7, 1, 1),
    ([200, 0, 600], 5, 5, 128, 1, 90, 10),
]


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("mass", [False, True])
@pytest.mark.parametrize("lens,H,Hk,d,page,window,sinks", DECODE)
def test_decode(gpu, dt, mass, lens, H, Hk, d, page, window, sinks):
    g = gen(sum(lens) + H)
    S, L = len(lens), max(lens)
    K, V, table = make_cache(g, dt, lens, Hk, d, page, gpu)
    Q = randn(g, (S, H, d), dt, 1.5)
    sc = scales(g, H, d, signs=H == 8)
    r = ref.decode(host(Q), host(K), host(V), lens, table.numpy(), host(sc), window, sinks)
    vmax = float(V.abs().max())
    # rows behind each sequence's end hold NaN
    for s, n in enumerate(lens):
        for j in range(n, table.shape[1] * page):
            pg = int(table[s, j // page])
            if pg >= 0:
                K[pg, :, j % page] = float("nan")
                V[pg, :, j % page] = float("nan")
    mi = torch.rand(S, Hk, L + 5, generator=g) * 3
    mo = torch.full((S, Hk, L + 5), 77.0, device=gpu)
    kw = dict(mass_in=mi.to(gpu), mass_out=mo) if mass else {}
    O, lse = mf.attention_decode(Q.to(gpu), K.to(gpu), V.to(gpu),
                                 torch.tensor(lens, dtype=torch.int32, device=gpu), sc.to(gpu), L,
                                 window=window, sinks=sinks, block_table=table.to(gpu), **kw)
    n = np.array([max(x, 1) for x in lens], dtype=np.float64)[:, None, None]
    close(host(O), r["O"], out_tol(dt, r["O"], r["A"], r["bound"], n, d, vmax), "O")
    close(host(lse), r["lse"], lse_tol(r["lse"], r["bound"], n[..., 0], d), "lse")
    if not mass:
        return
    for s, ln in enumerate(lens):
        want = r["mass"][s] + host(mi)[s, :, :ln]
        ds = score_err(r["bound"][s].max(), d)
        rel = 4 * ds + (2 * ln + 16) * F + H * F
        fin = np.abs(np.where(np.isfinite(r["lse"][s]), r["lse"][s], 0)).max()
        close(host(mo)[s, :, :ln], want, r["mass"][s] * (rel + 4 * F * fin) + 2 * F * np.abs(want) + 1e-30,
              f"mass {s}")
        assert (mo[s, :, ln:] == 77.0).all()


def test_decode_skips_pages_outside_the_pool(gpu):
    g = gen(41)
    K, V, table = make_cache(g, "bf16", [200, 90], 2, 128, 32, gpu)
    table[0, 2], table[1, 0] = 1 << 30, -1
    Q, sc = randn(g, (2, 8, 128), "bf16"), scales(g, 8, 128)
    lens = torch.tensor([200, 90], dtype=torch.int32)
    r = ref.decode(host(Q), host(K), host(V), lens, table.numpy(), host(sc))
    mo = torch.zeros(2, 2, 200, device=gpu)
    O, lse = mf.attention_decode(Q.to(gpu), K.to(gpu), V.to(gpu), lens.to(gpu), sc.to(gpu), 200,
                                 block_table=table.to(gpu), mass_out=mo)
    close(host(O), r["O"], out_tol("bf16", r["O"], r["A"], r["bound"], 200, 128, 5.0), "O")
    assert (mo[0, :, 64:96] == 0).all() and (mo[1, :, :32] == 0).all()
    # a length beyond max_len counts as max_len; mass added in place
    lens2 = torch.tensor([999, -3], dtype=torch.int32, device=gpu)
    O2, lse2 = mf.attention_decode(Q.to(gpu), K.to(gpu), V.to(gpu), lens2, sc.to(gpu), 200,
                                   block_table=table.to(gpu), mass_in=mo, mass_out=mo)
    assert torch.equal(O2[0], O[0]) and (O2[1] == 0).all() and torch.isinf(lse2[1]).all()


def test_decode_contiguous_cache_without_table(gpu):
    g = gen(42)
    S, H, Hk, d, cap = 3, 8, 4, 128, 150
    K, V = randn(g, (S, Hk, cap, d), "f16").to(gpu), randn(g, (S, Hk, cap, d), "f16").to(gpu)
    Q, sc = randn(g, (S, H, d), "f16").to(gpu), scales(g, H, d).to(gpu)
    lens = torch.tensor([150, 3, 77], dtype=torch.int32, device=gpu)
    t = torch.arange(S, dtype=torch.int32, device=gpu)[:, None].contiguous()
    a = mf.attention_decode(Q, K, V, lens, sc, cap)
    b = mf.attention_decode(Q, K, V, lens, sc, cap, block_table=t)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    # the same token as a prompt's last query
    for s in range(S):
        n = int(lens[s])
        O, lse = mf.attention_window(Q[s][:, None].contiguous(), K[s, :, :n].contiguous(),
                                     V[s, :, :n].transpose(0, 1), sc)
        # each within 2^-11 (A + |O|) of the exact row, A and |O| at most max |v| < 5
        assert torch.allclose(O[0].float(), a[0][s].float(), rtol=0, atol=2 * 10 * 2.0 ** -11)
        assert torch.allclose(lse[:, 0], a[1][s], rtol=0, atol=2 * (d + 6) * F * 32)


# ---- accumulated weight of a prompt's keys -----------------------------------

@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,N,H,Hk,d,window,sinks", [s for s in SHAPES if s[1]] + [
    (0, 30, 2, 1, 64, 0, 0), (700, 700, 4, 1, 64, 0, 0), (64, 900, 8, 2, 128, 300, 200)])
def test_key_mass(gpu, dt, M, N, H, Hk, d, window, sinks):
    g = gen(M * 3 + N)
    Q, K, V = randn(g, (H, M, d), dt), randn(g, (Hk, N, d), dt), torch.zeros(N, Hk, d)
    sc = scales(g, H, d, signs=H == 8)
    r = ref.attention(host(Q), host(K), host(V), host(sc), window, sinks)
    lse = torch.tensor(r["lse"], dtype=torch.float32)
    mi = torch.rand(Hk, N, generator=g)
    args = (Q.to(gpu), K.to(gpu), sc.to(gpu), lse.to(gpu))
    got = mf.key_mass_qk(*args, window=window, sinks=sinks, mass_in=mi.to(gpu))
    rel = mass_rel(r, d)
    want = r["mass"] + host(mi)
    close(host(got), want, r["mass"] * rel + 2 * F * np.abs(want), "mass")
    again = mf.key_mass_qk(*args, window=window, sinks=sinks, mass_in=mi.to(gpu))
    assert torch.equal(got, again)
    bare = mf.key_mass_qk(*args, window=window, sinks=sinks)
    close(host(bare), r["mass"], r["mass"] * rel + 2 * F * np.abs(r["mass"]), "mass from zero")


def test_key_mass_masked_nan(gpu):
    """Queries that see nothing, and keys that no given query sees, add nothing."""
    g = gen(52)
    H, Hk, N, M, d = 4, 2, 260, 100, 128
    Q, K = randn(g, (H, M, d), "bf16"), randn(g, (Hk, N, d), "bf16")
    sc = scales(g, H, d)
    r = ref.attention(host(Q), host(K), np.zeros((N, Hk, d)), host(sc), 20, 0)
    K[:, :130] = float("nan")                     # below the first query's window
    lse = torch.tensor(r["lse"], dtype=torch.float32)
    got = host(mf.key_mass_qk(Q.to(gpu), K.to(gpu), sc.to(gpu), lse.to(gpu), window=20))
    assert (got[:, :130] == 0).all()
    close(got[:, 141:], r["mass"][:, 141:], r["mass"][:, 141:] * mass_rel(r, d) + 1e-30, "mass")
    lse[:, 40:] = -math.inf
    Q[:, 40:] = float("nan")
    got = host(mf.key_mass_qk(Q.to(gpu), K.to(gpu), sc.to(gpu), lse.to(gpu), window=20))
    assert np.isfinite(got[:, 141:]).all() and (got[:, 200:] == 0).all()


# ---- eviction ----------------------------------------------------------------

EVICT = [
    # lens, cap of the mass rows, Hk, d, page, budget, sinks, recent
    ([1], 1, 1, 64, 16, 1, 0, 0),
    ([0, 5, 6, 7, 300], 300, 2, 128, 24, 6, 2, 3),
    ([1000, 999], 1003, 3, 64, 64, 100, 0, 0),
    ([2049, 64, 65], 2049, 2, 128, 1, 64, 0, 64),
    ([500], 500, 8, 128, 100, 499, 4, 10),
    ([333, 40], 333, 1, 128, 16, 40, 40, 0),
    ([4100], 4100, 2, 64, 128, 1, 0, 1),
    ([9000, 20000], 20000, 1, 64, 64, 5000, 7, 100),
    ([40001, 300], 40001, 1, 64, 256, 9999, 3, 5),
]


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("kind", ["spread", "ties", "odd"])
@pytest.mark.parametrize("lens,cap,Hk,d,page,budget,sinks,recent", EVICT)
def test_evict(gpu, dt, kind, lens, cap, Hk, d, page, budget, sinks, recent):
    g = gen(cap + budget)
    S = len(lens)
    K, V, table = make_cache(g, dt, lens, Hk, d, page, gpu)
    need = -(-cap // page)
    if table.shape[1] < need:
        table = torch.nn.functional.pad(table, (0, need - table.shape[1]), value=-7).contiguous()
    m = torch.randn(S, Hk, cap, generator=g).mul_(3).exp_()
    if kind == "ties":
        m = torch.randint(0, 4, m.shape, generator=g).float()
    if kind == "odd":
        pick = torch.randint(0, 7, m.shape, generator=g)
        for i, x in enumerate([float("nan"), float("inf"), -float("inf"), -0.0, 0.0, -1e-42]):
            m[pick == i] = x
    co = budget + 3
    Ko = torch.full((S, Hk, co, d), 9.0, dtype=DT[dt], device=gpu)
    Vo = torch.full((S, Hk, co, d), 9.0, dtype=DT[dt], device=gpu)
    mo = torch.full((S, Hk, co), 9.0, device=gpu)
    kept, left, K2, V2, m2 = mf.cache_evict(
        m.to(gpu), K.to(gpu), V.to(gpu), torch.tensor(lens, dtype=torch.int32, device=gpu), budget,
        sinks=sinks, recent=recent, block_table=table.to(gpu), K_out=Ko, V_out=Vo, mass_out=mo)
    kept, left = kept.cpu(), left.cpu()
    for s, n in enumerate(lens):
        assert int(left[s]) == min(n, budget)
        for h in range(Hk):
            want = ref.evict_rows(m[s, h].numpy(), n, budget, sinks, recent)
            c = len(want)
            assert kept[s, h, :c].tolist() == want, (s, h)
            assert (kept[s, h, c:] == -1).all()
            pg = table[s, torch.tensor(want, dtype=torch.long) // page].long()
            rr = torch.tensor(want, dtype=torch.long) % page
            assert torch.equal(K2[s, h, :c].cpu(), K[pg, h, rr]) and torch.equal(V2[s, h, :c].cpu(), V[pg, h, rr])
            assert (K2[s, h, c:] == 9.0).all() and (V2[s, h, c:] == 9.0).all()
            assert np.array_equal(m2[s, h, :c].cpu().numpy(), m[s, h, want].numpy(), equal_nan=True)
            assert (m2[s, h, c:] == 0).all()


def test_evict_rows_off_the_pool_become_zero(gpu):
    g = gen(61)
    K, V, table = make_cache(g, "bf16", [64], 1, 64, 16, gpu)
    table[0, 1] = 1 << 20
    m = torch.rand(1, 1, 64, generator=g)
    kept, left, K2, V2, m2 = mf.cache_evict(m.to(gpu), K.to(gpu), V.to(gpu),
                                            torch.tensor([64], dtype=torch.int32, device=gpu), 40,
                                            block_table=table.to(gpu))
    lost = ((kept[0, 0] >= 16) & (kept[0, 0] < 32)).cpu()
    assert lost.any() and (K2[0, 0].cpu()[lost] == 0).all() and (V2[0, 0].cpu()[lost] == 0).all()
    assert (K2[0, 0].cpu()[~lost] != 0).any(-1).all()


# ---- the operators in a row --------------------------------------------------

@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_prompt_then_eviction_then_tokens(gpu, dt):
    """Projection rows -> Q, K in a cache -> attention and key mass of the prompt ->
    eviction -> three single tokens appended and attended, their weight added up;
    every step against the oracle on the values the step before left."""
    g = gen(71)
    N, H, Hk, d, budget, cap = 333, 8, 2, 128, 100, 112
    freq, _ = mf.rope_frequencies(d, 1e6)
    freq = freq.to(gpu)
    x = randn(g, (N, H + 2 * Hk, d), dt, 1.5).to(gpu)
    wq, wk = (1 + 0.1 * randn(g, (d,), dt)).to(gpu), (1 + 0.1 * randn(g, (d,), dt)).to(gpu)
    sc = scales(g, H, d).to(gpu)
    pos = torch.arange(N, dtype=torch.int32, device=gpu)
    kw = dict(wq=wq, wk=wk)
    Q, K = mf.qk_norm_rope(x[:, :H], x[:, H:H + Hk], freq, pos, **kw)
    V = x[:, H + Hk:]
    O, lse = mf.attention_window(Q, K, V, sc)
    r = ref.attention(host(Q), host(K), host(V), host(sc))
    check_attention(dt, O, lse, r, N, d, 10.0)
    mass = mf.key_mass_qk(Q, K, sc, lse)
    # the lse is the kernel's own: its error comes on top
    close(host(mass), r["mass"], r["mass"] * (mass_rel(r, d) + lse_tol(r["lse"], r["bound"], N, d).max()), "mass")
    Kc, Vc = K[None].contiguous(), V.transpose(0, 1)[None].contiguous()
    lens = torch.tensor([N], dtype=torch.int32, device=gpu)
    K2 = torch.zeros(1, Hk, cap, d, dtype=DT[dt], device=gpu)
    V2, m2 = torch.zeros_like(K2), torch.zeros(1, Hk, cap, device=gpu)
    kept, lens, K2, V2, m2 = mf.cache_evict(mass[None], Kc, Vc, lens, budget, sinks=4, recent=32,
                                            K_out=K2, V_out=V2, mass_out=m2)
    for h in range(Hk):
        want = ref.evict_rows(host(mass)[h], N, budget, 4, 32)
        assert kept[0, h].tolist() == want
    for t in range(3):
        y = randn(g, (1, H + 2 * Hk, d), dt, 1.5).to(gpu)
        n = budget + t
        Qt, _, _ = mf.qk_norm_rope(y[:, :H], y[:, H:H + Hk], freq,
                                   torch.tensor([N + t], dtype=torch.int32, device=gpu), v=y[:, H + Hk:],
                                   K=K2, V=V2, slots=torch.tensor([n], device=gpu), token_major=True, **kw)
        lens = lens + 1
        before = m2.clone()
        Ot, lt = mf.attention_decode(Qt, K2, V2, lens, sc, cap, mass_in=m2, mass_out=m2)
        r = ref.decode(host(Qt), host(K2), host(V2), [n + 1], [[0]], host(sc))
        close(host(Ot), r["O"], out_tol(dt, r["O"], r["A"], r["bound"], n, d, 10.0), f"token {t} O")
        rel = 2 * mass_rel(r, d) + lse_tol(r["lse"], r["bound"], n, d).max()
        close(host(m2 - before)[0, :, :n + 1], r["mass"][0], rel * r["mass"][0] + 2 * F * host(m2).max(),
              f"token {t} mass")
