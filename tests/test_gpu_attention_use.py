"""Attention operators as a serving program uses them (MI355X): long rows, split keys,
captured graphs, side streams, two calls at once, caches past 2^31 elements."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import cross_model_sparse_amd as mf
from oracle import attention_ref as ref
from tests._attention import DT, F, close, host, lse_tol, mass_rel, out_tol, randn, score_err

pytestmark = pytest.mark.gpu


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def rows_of(Q, K, V, sc, window, sinks, rows):
    """The oracle on some queries only: O [R][H][d], lse [H][R], A, bound."""
    Q, K, V, sc = host(Q), host(K), host(V), host(sc)
    H, M, d = Q.shape
    N, G = K.shape[1], H // K.shape[0]
    O, A = np.zeros((len(rows), H, d)), np.zeros((len(rows), H, d))
    lse, bound = np.zeros((H, len(rows))), np.zeros((H, len(rows)))
    for x, i in enumerate(rows):
        seen = ref.visible(N - M + i, N, window, sinks)
        for h in range(H):
            O[x, h], lse[h, x], _, A[x, h], bound[h, x] = ref.attend(Q[h, i], K[h // G], V[:, h // G],
                                                                     sc[h], seen)
    return O, lse, A, bound


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,N,H,Hk,d,window,sinks,split", [
    (2500, 2500, 8, 2, 128, 0, 0, False),
    (2500, 2613, 3, 1, 64, 700, 130, False),
    (1, 6000, 4, 2, 128, 0, 0, True),
    (33, 9001, 2, 1, 128, 0, 0, True),
    (200, 5000, 8, 8, 64, 3500, 9, True),
    (513, 4100, 1, 1, 128, 0, 0, True),
])
def test_long_rows_and_split_keys(gpu, dt, M, N, H, Hk, d, window, sinks, split):
    g = gen(M + N)
    Q, K, V = randn(g, (H, M, d), dt), randn(g, (Hk, N, d), dt), randn(g, (N, Hk, d), dt)
    # keys that grow with their position: the running maximum keeps moving
    K = (K.float() * (0.3 + torch.arange(N)[None, :, None] / N * 2)).to(DT[dt])
    sc = torch.tensor([(0.6 if h % 3 else -0.9) / math.sqrt(d) for h in range(H)])
    need = mf.attention_split_workspace_bytes(DT[dt], H, Hk, M, N, d, window, sinks)
    if H * -(-M // 128) > 256:
        assert need == 0
    if split:
        assert need > 0
    args = [t.to(gpu) for t in (Q, K, V, sc)]
    rows = sorted({0, M - 1, M // 2, *torch.randint(0, M, (12,), generator=g).tolist()})
    Or, lr, A, bound = rows_of(Q, K, V, sc, window, sinks, rows)
    vmax = float(V.abs().max())
    first = None
    # split where it pays, and never (no room for the parts)
    for ws in (None, torch.empty(16, dtype=torch.uint8, device=gpu)):
        O, lse = mf.attention_window(*args, window=window, sinks=sinks, workspace=ws)
        close(host(O)[rows], Or, out_tol(dt, Or, A, bound.T, N, d, vmax), "O")
        close(host(lse)[:, rows], lr, lse_tol(lr, bound, N, d), "lse")
        O2, lse2 = mf.attention_window(*args, window=window, sinks=sinks, workspace=ws)
        assert torch.equal(O, O2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_split_keys_with_non_finite_masked_values(gpu, dt):
    g = gen(3)
    M, N, H, d, window, sinks = 40, 3000, 2, 128, 2000, 3
    Q, K, V = randn(g, (H, M, d), dt), randn(g, (H, N, d), dt), randn(g, (N, H, d), dt)
    sc = torch.full((H,), 0.08)
    O, lse, A, bound = rows_of(Q, K, V, sc, window, sinks, range(M))
    bad = list(range(3, N - window - M + 1)) + [N - 5]
    K[:, bad], V[bad] = float("nan"), float("inf")
    assert mf.attention_split_workspace_bytes(DT[dt], H, H, M, N, d, window, sinks) > 0
    Og, lg = mf.attention_window(*[t.to(gpu) for t in (Q, K, V, sc)], window=window, sinks=sinks)
    clean = [i for i in range(M) if N - M + i < N - 5]
    close(host(Og)[clean], O[clean], out_tol(dt, O, A, bound.T, N, d, 6.0)[clean], "O")
    close(host(lg)[:, clean], lse[:, clean], lse_tol(lse, bound, N, d)[:, clean], "lse")


def test_many_packed_sequences(gpu):
    g = gen(4)
    n = [int(x) for x in torch.randint(0, 9, (300,), generator=g)] + [400]
    N, H, Hk, d = sum(n), 8, 2, 64
    Q, K, V = randn(g, (H, N, d), "bf16"), randn(g, (Hk, N, d), "bf16"), randn(g, (N, Hk, d), "bf16")
    sc = torch.full((H,), 0.1)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32)
    dev = [t.to(gpu) for t in (Q, K, V, sc, cu)]
    O, lse = mf.attention_window_varlen(*dev[:4], dev[4], dev[4], window=5, sinks=1)
    for s in (0, 1, 17, 150, 299, 300):
        a, b = int(cu[s]), int(cu[s + 1])
        one = mf.attention_window(dev[0][:, a:b], dev[1][:, a:b], dev[2][a:b], dev[3], window=5, sinks=1,
                                  workspace=torch.empty(16, dtype=torch.uint8, device=gpu))
        assert torch.equal(O[a:b], one[0]) and torch.equal(lse[:, a:b], one[1])


def test_packed_batch_that_starts_behind_row_0(gpu):
    """Offsets need not start at 0: rows before the first sequence stay as they were."""
    g = gen(14)
    N, H, Hk, d = 700, 2, 1, 64
    Q, K, V = (randn(g, s, "bf16").to(gpu) for s in ((H, N, d), (Hk, N, d), (N, Hk, d)))
    sc = torch.full((H,), 0.1, device=gpu)
    cu = torch.tensor([300, 300, 420, 650], dtype=torch.int32, device=gpu)
    O = torch.full((N, H, d), 5.0, dtype=torch.bfloat16, device=gpu)
    lse = torch.full((H, N), 5.0, device=gpu)
    mf.attention_window_varlen(Q, K, V, sc, cu, cu, out=O, lse=lse)
    for a, b in ((300, 420), (420, 650)):
        one = mf.attention_window(Q[:, a:b], K[:, a:b], V[a:b], sc,
                                  workspace=torch.empty(16, dtype=torch.uint8, device=gpu))
        assert torch.equal(O[a:b], one[0]) and torch.equal(lse[:, a:b], one[1])
    for a, b in ((0, 300), (650, N)):
        assert (O[a:b] == 5.0).all() and (lse[:, a:b] == 5.0).all()


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_decode_masked_rows_hold_anything(gpu, dt):
    g = gen(5)
    S, H, Hk, d, page, L, window, sinks = 2, 8, 2, 128, 48, 500, 77, 5
    P = S * -(-L // page)
    K, V = randn(g, (P, Hk, page, d), dt), randn(g, (P, Hk, page, d), dt)
    table = torch.randperm(P, generator=g).int().view(S, -1)
    Q, sc, lens = randn(g, (S, H, d), dt), torch.full((H,), 0.09), [500, 83]
    r = ref.decode(host(Q), host(K), host(V), lens, table.numpy(), host(sc), window, sinks)
    for s, n in enumerate(lens):
        for j in range(n):
            if j >= sinks and j < n - window:
                pg = int(table[s, j // page])
                K[pg, :, j % page], V[pg, :, j % page] = float("nan"), float("inf")
    mo = torch.zeros(S, Hk, L, device=gpu)
    O, lse = mf.attention_decode(Q.to(gpu), K.to(gpu), V.to(gpu), torch.tensor(lens, dtype=torch.int32, device=gpu),
                                 sc.to(gpu), L, window=window, sinks=sinks, block_table=table.to(gpu),
                                 mass_out=mo)
    close(host(O), r["O"], out_tol(dt, r["O"], r["A"], r["bound"], L, d, 6.0), "O")
    close(host(lse), r["lse"], lse_tol(r["lse"], r["bound"], L, d), "lse")
    for s, n in enumerate(lens):
        want = r["mass"][s]
        close(host(mo)[s, :, :n], want, want * 2 * mass_rel(r, d) + 1e-30, "mass")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_decode_of_a_fused_projection_into_a_wider_buffer(gpu, dt):
    g = gen(15)
    S, H, Hk, d, L = 5, 6, 2, 64, 130
    x = randn(g, (S, H + 3, d), dt).to(gpu)
    K, V = randn(g, (S, Hk, L, d), dt).to(gpu), randn(g, (S, Hk, L, d), dt).to(gpu)
    sc, lens = torch.full((H,), 0.2, device=gpu), torch.tensor([130, 1, 64, 65, 0], dtype=torch.int32, device=gpu)
    big = torch.full((S, H + 1, d), 3.0, dtype=DT[dt], device=gpu)
    a = mf.attention_decode(x[:, 1:1 + H], K, V, lens, sc, L, out=big[:, 1:])
    b = mf.attention_decode(x[:, 1:1 + H].contiguous(), K, V, lens, sc, L)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and (big[:, 0] == 3.0).all()
    # off 16 bytes: queries and outputs need their element's alignment only
    off = torch.zeros(S * H * d + 1, dtype=DT[dt], device=gpu)
    off[1:] = x[:, 1:1 + H].reshape(-1)
    o2 = torch.zeros(S * H * d + 1, dtype=DT[dt], device=gpu)
    c = mf.attention_decode(off[1:].view(S, H, d), K, V, lens, sc, L, out=o2[1:].view(S, H, d))
    assert torch.equal(c[0], b[0]) and float(o2[0]) == 0.0


def test_one_bad_query_or_sequence_stays_alone(gpu):
    """A NaN query, and a sequence full of NaN, leave their neighbours as they were."""
    g = gen(16)
    N, H, Hk, d = 200, 4, 2, 128
    Q, K, V = (randn(g, s, "bf16").to(gpu) for s in ((H, N, d), (Hk, N, d), (N, Hk, d)))
    sc = torch.full((H,), 0.1, device=gpu)
    cu = torch.tensor([0, 70, 130, N], dtype=torch.int32, device=gpu)
    want = mf.attention_window_varlen(Q, K, V, sc, cu, cu)
    Q2, K2, V2 = Q.clone(), K.clone(), V.clone()
    K2[:, 70:130], V2[70:130], Q2[1, 30] = float("nan"), float("nan"), float("nan")
    got = mf.attention_window_varlen(Q2, K2, V2, sc, cu, cu)
    keep = torch.ones(N, H, dtype=torch.bool, device=gpu)
    keep[70:130], keep[30, 1] = False, False
    assert torch.equal(got[0][keep], want[0][keep]) and torch.equal(got[1][keep.t()], want[1][keep.t()])
    assert torch.isnan(got[0][~keep].float()).all()
    pool, vpool = K[None].contiguous(), V.transpose(0, 1)[None].contiguous()
    lens = torch.tensor([N, N], dtype=torch.int32, device=gpu)
    two = torch.cat([pool, pool]), torch.cat([vpool, vpool])
    q = Q[:, -2:].transpose(0, 1).contiguous()
    want = mf.attention_decode(q, *two, lens, sc, N)
    two[0][1], two[1][1], q[0, 2] = float("nan"), float("nan"), float("nan")
    got = mf.attention_decode(q, *two, lens, sc, N)
    ok = [0, 1, 3]
    assert torch.equal(got[0][0, ok], want[0][0, ok]) and torch.isnan(got[0][1].float()).all()
    assert torch.isnan(got[0][0, 2].float()).all()


def test_the_documented_sequence_of_calls(gpu):
    """The README's example."""
    g = gen(17)
    N, H, Hk, d = 2000, 8, 2, 128
    x = randn(g, (N, H + 2 * Hk, d), "bf16").to(gpu)
    q, k, V = x[:, :H], x[:, H:H + Hk], x[:, H + Hk:]
    wq = wk = torch.ones(d, dtype=torch.bfloat16, device=gpu)
    positions = torch.arange(N, dtype=torch.int32, device=gpu)
    scale = torch.full((H,), d ** -0.5, device=gpu)
    lens = torch.tensor([N], dtype=torch.int32, device=gpu)
    freq, af = mf.rope_frequencies(128, 1e6, "yarn", 4.0, orig_len=4096)
    Q, K = mf.qk_norm_rope(q, k, freq.cuda(), positions, wq=wq, wk=wk, attn_factor=af)
    O, lse = mf.attention_window(Q, K, V, scale, window=1024, sinks=4)
    mass = mf.key_mass_qk(Q, K, scale, lse, window=1024, sinks=4)
    kept, lens, Kc, Vc, m = mf.cache_evict(mass[None], K[None], V.transpose(0, 1)[None].contiguous(), lens,
                                           budget=512, sinks=4, recent=64)
    assert O.shape == (N, H, d) and lens.tolist() == [512] and Kc.shape == (1, Hk, 512, d)
    # every query's weights add up to 1
    assert torch.allclose(mass.sum(), torch.tensor(float(H * N), device=gpu), rtol=1e-3)


def test_decode_of_empty_caches(gpu):
    Q = torch.randn(3, 4, 64, device=gpu).half()
    K = torch.zeros(3, 2, 16, 64, device=gpu, dtype=torch.float16)
    sc, lens = torch.ones(4, device=gpu), torch.zeros(3, dtype=torch.int32, device=gpu)
    for n in (0, 16):
        mo = torch.full((3, 2, 16), 5.0, device=gpu)
        O, lse = mf.attention_decode(Q, K, K.clone(), lens, sc, n, mass_out=mo)
        assert (O == 0).all() and torch.isinf(lse).all() and (mo == 5.0).all()
    # no page at all
    none = torch.zeros(0, 2, 16, 64, device=gpu, dtype=torch.float16)
    table = torch.zeros(3, 1, dtype=torch.int32, device=gpu)
    lens = torch.full((3,), 9, dtype=torch.int32, device=gpu)
    mo = torch.full((3, 2, 16), 5.0, device=gpu)
    O, lse = mf.attention_decode(Q, none, none, lens, sc, 16, block_table=table, mass_in=mo, mass_out=mo)
    assert (O == 0).all() and torch.isinf(lse).all() and (mo == 5.0).all()
    # a batch of no sequences
    O, lse = mf.attention_decode(Q[:0], K, K, lens[:0], sc, 0)
    assert O.shape == (0, 4, 64) and lse.shape == (0, 4)


def test_evict_of_empty_caches(gpu):
    K = torch.randn(2, 2, 16, 64, device=gpu)
    m = torch.rand(2, 2, 16, device=gpu)
    lens = torch.tensor([0, 16], dtype=torch.int32, device=gpu)
    kept, left, K2, V2, m2 = mf.cache_evict(m, K, K + 1, lens, 20)
    assert left.tolist() == [0, 16] and (kept[0] == -1).all() and (m2[0] == 0).all() and (K2[0] == 0).all()
    assert torch.equal(K2[1, :, :16], K[1]) and torch.equal(V2[1, :, :16], K[1] + 1)
    kept, left, *_ = mf.cache_evict(m[..., :0].contiguous(), K, K + 1, lens, 3, max_len=0)
    assert left.tolist() == [0, 0] and (kept == -1).all()


def chain(x, st, s=None):
    """Prompt, eviction, one token: every operator once, into the same outputs."""
    H, Hk, d, N = st["H"], st["Hk"], st["d"], x.shape[0]
    Q, K = mf.qk_norm_rope(x[:, :H], x[:, H:H + Hk], st["freq"], st["pos"], wq=st["w"], wk=st["w"], stream=s)
    V = x[:, H + Hk:]
    O, lse = mf.attention_window(Q, K, V, st["sc"], window=st["window"], sinks=4, stream=s)
    Ov, _ = mf.attention_window_varlen(Q, K, V, st["sc"], st["cu"], st["cu"], stream=s)
    mass = mf.key_mass_qk(Q, K, st["sc"], lse, window=st["window"], sinks=4, stream=s)
    Vc = st["Vc"]
    st["Kc"].copy_(K[None])
    Vc.copy_(V.transpose(0, 1)[None])
    kept, left, K2, V2, m2 = mf.cache_evict(mass[None], st["Kc"], Vc, st["len"], 64, sinks=4, recent=16,
                                            K_out=st["K2"], V_out=st["V2"], mass_out=st["m2"], stream=s)
    Qt, _, _ = mf.qk_norm_rope(x[:1, :H], x[:1, H:H + Hk], st["freq"], st["pos"][-1:], v=x[:1, H + Hk:], K=K2,
                               V=V2, slots=st["slot"], token_major=True, stream=s)
    Ot, lt = mf.attention_decode(Qt, K2, V2, st["len2"], st["sc"], 80, mass_in=m2, mass_out=m2, stream=s)
    return [O, lse, Ov, mass, kept, left, K2, V2, m2, Ot, lt]


def chain_state(gpu, seed):
    H, Hk, d, N = 8, 2, 128, 700
    g = gen(seed)
    freq, _ = mf.rope_frequencies(d, 1e6)
    z = lambda *s: torch.zeros(*s, device=gpu, dtype=torch.bfloat16)   # noqa: E731
    return dict(H=H, Hk=Hk, d=d, window=200, freq=freq.to(gpu), pos=torch.arange(N, dtype=torch.int32, device=gpu),
                w=(1 + 0.1 * torch.randn(d, generator=g)).bfloat16().to(gpu),
                sc=torch.full((H,), 1 / math.sqrt(d), device=gpu), Kc=z(1, Hk, N, d), Vc=z(1, Hk, N, d),
                K2=z(1, Hk, 80, d), V2=z(1, Hk, 80, d), m2=torch.zeros(1, Hk, 80, device=gpu),
                len=torch.tensor([N], dtype=torch.int32, device=gpu),
                len2=torch.tensor([65], dtype=torch.int32, device=gpu),
                slot=torch.tensor([64], device=gpu),
                cu=torch.tensor([0, 100, 100, 513, N], dtype=torch.int32, device=gpu))


def test_captured_graph_replays(gpu):
    st = chain_state(gpu, 6)
    xs = [randn(gen(60 + i), (700, 12, 128), "bf16", 1.5).to(gpu) for i in range(3)]
    x = xs[0].clone()
    want = []
    for y in xs:
        x.copy_(y)
        want.append([t.clone() for t in chain(x, st)])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        chain(x, st)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = chain(x, st)
    for r in range(6):
        x.copy_(xs[r % 3])
        graph.replay()
        if r % 2:
            torch.cuda.synchronize()
        got = [t.clone() for t in out]
        for a, b in zip(got, want[r % 3]):
            assert torch.equal(a, b), r
        # the same operators eagerly between replays
        mine = chain_state(gpu, 6)
        for a, b in zip(chain(x, mine), want[r % 3]):
            assert torch.equal(a, b), r


def test_side_streams_and_two_calls_at_once(gpu):
    xs = [randn(gen(70 + i), (700, 12, 128), "bf16", 1.5).to(gpu) for i in range(2)]
    want = [[t.clone() for t in chain(xs[i], chain_state(gpu, i))] for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    states = [chain_state(gpu, i) for i in range(2)]
    torch.cuda.synchronize()
    outs = [None, None]
    for _ in range(3):
        for i, s in enumerate(streams):
            # one by the current stream, one by the argument (its copies follow the stream too)
            if i == 0:
                with torch.cuda.stream(s):
                    outs[i] = chain(xs[i], states[i])
            else:
                with torch.cuda.stream(s):
                    outs[i] = chain(xs[i], states[i], s)
    torch.cuda.synchronize()
    for i in range(2):
        for a, b in zip(outs[i], want[i]):
            assert torch.equal(a, b), i


def test_stream_argument_orders_the_call(gpu):
    """stream= alone: inputs written on that stream are seen, workspaces belong to it."""
    g = gen(8)
    Q, K, V = (randn(g, s, "bf16").to(gpu) for s in ((2, 64, 128), (2, 6000, 128), (6000, 2, 128)))
    sc = torch.full((2,), 0.1, device=gpu)
    want = mf.attention_window(Q, K, V, sc)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    Q2 = torch.zeros_like(Q)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        Q2.copy_(Q)
    got = mf.attention_window(Q2, K, V, sc, stream=s)
    junk = torch.full((1 << 22,), 7, dtype=torch.uint8, device=gpu)   # reuse of freed blocks
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and int(junk[0]) == 7


def test_caches_past_2_31_elements(gpu):
    """Pages at the far end of pools of 2.2e9 elements."""
    g = gen(9)
    Hk, d, page, H, L = 8, 128, 64, 16, 300
    P = 34000                                     # P * Hk * page * d = 2.2e9
    K = torch.zeros(P, Hk, page, d, dtype=torch.float16, device=gpu)
    V = torch.zeros_like(K)
    pages = torch.tensor([P - 1, 3, P - 2, P - 3, 0], dtype=torch.int32)
    kk, vv = randn(g, (5, Hk, page, d), "f16"), randn(g, (5, Hk, page, d), "f16")
    K[pages.long().to(gpu)], V[pages.long().to(gpu)] = kk.to(gpu), vv.to(gpu)
    Q, sc = randn(g, (1, H, d), "f16"), torch.full((H,), 0.1)
    r = ref.decode(host(Q), host(kk), host(vv), [L], [[0, 1, 2, 3, 4]], host(sc))
    lens, table = torch.tensor([L], dtype=torch.int32, device=gpu), pages[None].contiguous().to(gpu)
    O, _ = mf.attention_decode(Q.to(gpu), K, V, lens, sc.to(gpu), L, block_table=table)
    close(host(O), r["O"], out_tol("f16", r["O"], r["A"], r["bound"], L, d, 6.0), "O")
    m = torch.rand(1, Hk, L, generator=g)
    kept, _, K2, V2, _ = mf.cache_evict(m.to(gpu), K, V, lens, 100, block_table=table)
    for h in range(Hk):
        idx = torch.tensor(ref.evict_rows(m[0, h].numpy(), L, 100, 0, 0))
        assert kept[0, h].tolist() == idx.tolist()
        assert torch.equal(K2[0, h].cpu(), kk[idx // page, h, idx % page])
    # a token written to the last row
    x = randn(g, (1, H + 2 * Hk, d), "f16").to(gpu)
    slot = torch.tensor([P * page - 1], device=gpu)
    Qt, _, _ = mf.qk_norm_rope(x[:, :H], x[:, H:H + Hk], None, None, v=x[:, H + Hk:], K=K, V=V, slots=slot,
                               token_major=True)
    assert torch.equal(K[P - 1, :, page - 1], x[0, H:H + Hk]) and torch.equal(V[P - 1, :, page - 1], x[0, H + Hk:])
    del K, V
    # a prompt's keys so far apart that rows lie past 2^31 elements
    N, ld = 70, 1 << 25
    big = torch.zeros(N * ld, dtype=torch.float16, device=gpu)
    view = big.as_strided((1, N, 64), (64, ld, 1))
    k, v, q = randn(g, (1, N, 64), "f16"), randn(g, (N, 1, 64), "f16"), randn(g, (2, N, 64), "f16")
    view.copy_(k.to(gpu))
    s2 = torch.full((2,), 0.1, device=gpu)
    a = mf.attention_window(q.to(gpu), view, v.to(gpu), s2)
    b = mf.attention_window(q.to(gpu), k.to(gpu), v.to(gpu), s2)
    # the far one runs the plain kernel: each within 2^-11 (A + |O|), both below max |v| < 5
    assert torch.allclose(a[0].float(), b[0].float(), rtol=0, atol=2 * 10 * 2.0 ** -11)
    ma, mb = (mf.key_mass_qk(q.to(gpu), t, s2, b[1]) for t in (view, k.to(gpu)))
    assert torch.allclose(ma, mb, rtol=4 * score_err(32.0, 64), atol=0)


def test_scores_accumulate_over_tokens(gpu):
    """mass_in = mass_out over several tokens adds up to the prompt's key mass."""
    g = gen(10)
    N, H, Hk, d = 90, 4, 2, 64
    Q, K, V = randn(g, (H, N, d), "f32"), randn(g, (Hk, N, d), "f32"), randn(g, (N, Hk, d), "f32")
    sc = torch.full((H,), 0.1)
    Qd, Kd, Vd, sd = (t.to(gpu) for t in (Q, K, V, sc))
    O, lse = mf.attention_window(Qd, Kd, Vd, sd)
    want = mf.key_mass_qk(Qd, Kd, sd, lse)
    pool, vpool = Kd[None].contiguous(), Vd.transpose(0, 1)[None].contiguous()
    m = torch.zeros(1, Hk, N, device=gpu)
    for t in range(N):
        o, _ = mf.attention_decode(Qd[:, t][None].contiguous(), pool, vpool,
                                   torch.tensor([t + 1], dtype=torch.int32, device=gpu), sd, N, mass_in=m, mass_out=m)
        assert torch.allclose(o[0], O[t], rtol=0, atol=5 * (4 * score_err(10.0, d) + 4 * N * F))
    assert torch.allclose(m[0], want, rtol=8 * score_err(10.0, d) + 400 * F, atol=N * 2 * F)
