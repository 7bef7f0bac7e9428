"""Python binding of libmapflow's attention operators (argument marshalling only).

The attention around the reuse path: per-head norm and rotary positions of q and
k, windowed attention of prompts, single-token attention over a paged cache, the
accumulated weight of every cached key, and eviction by that weight.  As in
:mod:`.mapflow`, the functions take torch tensors on one GPU, check them on the
host, and call the C boundary of include/mapflow.h; all arithmetic runs in the
library's HIP kernels.

Work goes to `stream`, by default the current stream of the tensors' device
(which need not be the current device).  Outputs and workspaces that a call
allocates belong to that stream.
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

from .mapflow import MF_ERR_INVALID, MapflowError, _check, _DTYPE_CODE, load

__all__ = ["rope_frequencies", "qk_norm_rope", "attention_window", "attention_window_varlen",
           "attention_split_workspace_bytes", "attention_decode",
           "attention_decode_workspace_bytes", "key_mass_qk", "key_mass_qk_workspace_bytes",
           "cache_evict"]

_SCALING = {"plain": 0, "linear": 1, "ntk": 2, "yarn": 3}
_LAYOUT = {"half": 0, "interleaved": 1}


def _bad(msg: str):
    raise MapflowError(MF_ERR_INVALID, msg)


_NULL = contextlib.nullcontext()


def _on(dev: torch.device, stream):
    """(context, handle): the stream that the call runs on, and a context in
    which allocations belong to it."""
    if dev.type != "cuda":
        _bad("tensors must be on the GPU")
    if stream is not None:
        if stream.device != dev:
            _bad(f"stream of {stream.device}, tensors on {dev}")
        return torch.cuda.stream(stream), stream.cuda_stream
    handle = torch._C._cuda_getCurrentRawStream(dev.index)
    return (_NULL if torch._C._cuda_getDevice() == dev.index else torch.cuda.device(dev)), handle


def _same(where: int, dtype, t: torch.Tensor | None, name: str) -> None:
    """t (if given) lives on the device `where` (-1: the host) and holds `dtype`."""
    if t is None:
        return
    if t.get_device() != where:
        _bad(f"{name} is on {t.device}, other tensors elsewhere")
    if dtype is not None and t.dtype is not dtype:
        _bad(f"{name} must be {dtype} (got {t.dtype})")


def _code(t: torch.Tensor) -> int:
    c = _DTYPE_CODE.get(t.dtype)
    if c is None:
        _bad(f"unsupported dtype {t.dtype}")
    return c


def _ints(**xs) -> None:
    """Sizes that the C boundary takes as int (ctypes would cut them silently)."""
    for name, x in xs.items():
        if not -(1 << 31) <= x < 1 << 31:
            _bad(f"{name} = {x} does not fit 32 bits")


def _full(t: torch.Tensor | None, name: str, shape: tuple, dtype, where: int) -> None:
    """t (if given) is a contiguous tensor of that shape, type and device."""
    if t is None:
        return
    if t.shape != shape or t.dtype is not dtype or t.get_device() != where or not t.is_contiguous():
        _same(where, dtype, t, name)
        _bad(f"{name} must be a contiguous {list(shape)} tensor")


def _rows3(t: torch.Tensor, name: str) -> None:
    if t.dim() != 3 or (t.shape[2] > 1 and t.stride(2) != 1):
        _bad(f"{name} must have three dims and contiguous rows")


def _p(t: torch.Tensor | None):
    return None if t is None else t.data_ptr()


def _bytes_of(t: torch.Tensor | None) -> int:
    return 0 if t is None else t.numel() * t.element_size()


def _workspace(t, need: int, dev):
    """The caller's workspace, or a fresh one (None when none is needed)."""
    if t is not None:
        _same(dev.index if dev.type == "cuda" else -1, None, t, "workspace")
        if not t.is_contiguous():
            _bad("workspace must be contiguous")
        return t
    return torch.empty(need, dtype=torch.uint8, device=dev) if need else None


def rope_frequencies(rot: int, base: float, scaling: str = "plain", factor: float = 1.0,
                     orig_len: float = 0.0, beta_fast: float = 32.0, beta_slow: float = 1.0):
    """(freq, attn_factor): rotary frequencies as a host float64 [rot/2] tensor and
    the factor on the rotated dims (mf_rope_frequencies).  scaling: "plain",
    "linear", "ntk" or "yarn" (needs orig_len)."""
    if scaling not in _SCALING:
        _bad(f"unknown scaling {scaling!r}")
    freq = torch.empty(max(int(rot), 2) // 2, dtype=torch.float64)
    af = ctypes.c_double(1.0)
    _check(load().mf_rope_frequencies(int(rot), float(base), _SCALING[scaling], float(factor),
                                      float(orig_len), float(beta_fast), float(beta_slow),
                                      freq.data_ptr(), ctypes.addressof(af)))
    return freq, float(af.value)


def qk_norm_rope(q: torch.Tensor, k: torch.Tensor, freq: torch.Tensor | None,
                 positions: torch.Tensor | None, *, wq: torch.Tensor | None = None,
                 wk: torch.Tensor | None = None, eps: float = 1e-6, layout: str = "half",
                 attn_factor: float = 1.0, Q: torch.Tensor | None = None,
                 K: torch.Tensor | None = None, v: torch.Tensor | None = None,
                 V: torch.Tensor | None = None, slots: torch.Tensor | None = None,
                 token_major: bool = False, stream=None):
    """Per-head RMS norm (weights wq, wk of [d], or None) and rotary positions.

    q [N][H_q][d] and k [N][H_k][d] may be slices of a fused projection; freq is
    the device copy of rope_frequencies' tensor (None: no rotation), positions
    int32 [N].  Returns (Q, K): [H][N][d], or [N][H][d] with token_major=True;
    given Q and K (any strides, of that shape) are written instead.

    With slots (int64 [N]) k goes to row slots[n] of the cache pool K and v to
    that of V, pools [n_pages][H_k][page][d] (mf_qk_norm_rope_cache); slots
    outside the pool are skipped.  Returns (Q, K, V)."""
    if q.dim() != 3 or k.dim() != 3:
        _bad("q and k must have three dims")
    N, H_q, d = q.shape
    H_k = k.shape[1]
    dev, dt, where = q.device, q.dtype, q.get_device()
    code = _code(q)
    if layout not in _LAYOUT:
        _bad(f"unknown layout {layout!r}")

    def source(t, name, H):                      # checked; its stride from row to row
        _same(where, dt, t, name)
        if t.shape != (N, H, d):
            _bad(f"{name} must be [{N}][{H}][{d}]")
        n, h, e = t.stride()
        if N and ((H > 1 and h != d) or e != 1):
            _bad(f"{name}'s heads must lie side by side")
        return n if N > 1 else H * d

    ldq, ldk = source(q, "q", H_q), source(k, "k", H_k)
    ldv = 0 if v is None else source(v, "v", H_k)
    _same(where, dt, Q, "Q")
    _same(where, dt, K, "K")
    rot = 0 if freq is None else 2 * freq.shape[0]
    if rot:
        _full(freq, "freq", (rot // 2,), torch.float64, where)
        if positions is None:
            _bad("positions missing")
        _full(positions, "positions", (N,), torch.int32, where)
    _full(wq, "wq", (d,), dt, where)
    _full(wk, "wk", (d,), dt, where)
    ctx, handle = _on(dev, stream)

    def out(t, H, name):
        shape = (N, H, d) if token_major else (H, N, d)
        if t is None:
            t = torch.empty(shape, dtype=dt, device=dev)
            return (t, H * d, d) if token_major else (t, d, N * d)
        if t.shape != shape or (t.numel() and t.stride(2) != 1):
            _bad(f"{name} must be {list(shape)} with contiguous rows")
        n, h = (0, 1) if token_major else (1, 0)
        return t, (t.stride(n) if N > 1 else H * d), (t.stride(h) if H > 1 else d)

    with ctx:
        Q, ldQ, hsQ = out(Q, H_q, "Q")
        head = (code, N, d, _p(q), H_q, ldq, _p(k), H_k, ldk)
        norm = (_p(wq), _p(wk), float(eps), _p(freq), rot, _LAYOUT[layout], float(attn_factor),
                _p(positions), _p(Q), ldQ, hsQ)
        if slots is None:
            if v is not None or V is not None:
                _bad("v and V need slots")
            K, ldK, hsK = out(K, H_k, "K")
            _check(load().mf_qk_norm_rope(*head, *norm, _p(K), ldK, hsK, handle))
            return Q, K
        if v is None or K is None or V is None:
            _bad("slots need v and the pools K and V")
        _full(slots, "slots", (N,), torch.int64, where)
        if K.dim() != 4 or K.shape[1] != H_k or K.shape[3] != d or not K.is_contiguous():
            _bad("K must be a contiguous [n_pages][H_k][page][d] pool")
        _full(V, "V", K.shape, dt, where)
        _check(load().mf_qk_norm_rope_cache(*head, _p(v), ldv, *norm, _p(slots), _p(K), _p(V),
                                            K.shape[0], K.shape[2], handle))
        return Q, K, V


def attention_split_workspace_bytes(dtype: torch.dtype, H: int, H_kv: int, N_q: int, N_k: int,
                                    d: int, window: int = 0, sinks: int = 0) -> int:
    """Workspace bytes that let attention_window split the keys (0: no split)."""
    return int(load().mf_attention_split_workspace_bytes(_DTYPE_CODE[dtype], H, H_kv, N_q, N_k, d,
                                                         window, sinks))


def _attn_shapes(Q, K, V, scale):
    _rows3(Q, "Q")
    _rows3(K, "K")
    _rows3(V, "V")
    H, N_q, d = Q.shape
    H_kv, N_k, dk = K.shape
    if dk != d or V.shape != (N_k, H_kv, d):
        _bad("K must be [H_kv][N_k][d] and V [N_k][H_kv][d]")
    where = Q.get_device()
    _same(where, Q.dtype, K, "K")
    _same(where, Q.dtype, V, "V")
    _full(scale, "scale", (H,), torch.float32, where)
    rows = (_p(Q), Q.stride(1), Q.stride(0), _p(K), K.stride(1), K.stride(0), _p(V), V.stride(0),
            V.stride(1))
    return rows, H, H_kv, N_q, N_k, d


def _attn_out(Q, H, N_q, d, out, lse):
    dev = Q.device
    if out is None:
        out = torch.empty(N_q, H, d, dtype=Q.dtype, device=dev)
    else:
        _same(Q.get_device(), Q.dtype, out, "out")
        if out.shape != (N_q, H, d) or (N_q and (out.stride(2) != 1 or
                                                        (H > 1 and out.stride(1) != d))):
            _bad("out must be [N_q][H][d] with contiguous rows")
    if lse is None:
        lse = torch.empty(H, N_q, dtype=torch.float32, device=dev)
    else:
        _full(lse, "lse", (H, N_q), torch.float32, Q.get_device())
    return out, lse, (out.stride(0) if N_q > 1 else H * d)


def attention_window(Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, scale: torch.Tensor, *,
                     window: int = 0, sinks: int = 0, out: torch.Tensor | None = None,
                     lse: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                     stream=None):
    """(O, lse) of causal attention (mf_attention_window).

    Q [H][N_q][d], K [H_kv][N_k][d], V [N_k][H_kv][d] (any strides with contiguous
    rows), scale float32 [H]; query i sits at position N_k - N_q + i and sees the
    last `window` keys up to itself (0: all) and the first `sinks`.  O is
    [N_q][H][d], lse float32 [H][N_q] (-inf for a query that sees nothing)."""
    rows, H, H_kv, N_q, N_k, d = _attn_shapes(Q, K, V, scale)
    code = _code(Q)
    _ints(window=window, sinks=sinks, N_q=N_q, N_k=N_k)
    ctx, handle = _on(Q.device, stream)
    with ctx:
        out, lse, ldO = _attn_out(Q, H, N_q, d, out, lse)
        L = load()
        need = 0 if workspace is not None else L.mf_attention_split_workspace_bytes(
            code, H, H_kv, N_q, N_k, d, window, sinks)
        ws = _workspace(workspace, need, Q.device)
        _check(L.mf_attention_window(*rows, code, H, H_kv, N_q, N_k, d, _p(scale), window, sinks,
                                     _p(out), ldO, _p(lse), _p(ws), _bytes_of(ws), handle))
    return out, lse


def attention_window_varlen(Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor,
                            scale: torch.Tensor, cu_q: torch.Tensor, cu_k: torch.Tensor, *,
                            window: int = 0, sinks: int = 0, out: torch.Tensor | None = None,
                            lse: torch.Tensor | None = None, stream=None):
    """attention_window over a packed batch: sequence s holds rows cu_q[s]..cu_q[s+1]-1
    of Q and cu_k[s]..cu_k[s+1]-1 of K and V (int32 [S+1] tensors on the GPU).  Rows
    behind the last sequence are left as they were."""
    rows, H, H_kv, N_q, N_k, d = _attn_shapes(Q, K, V, scale)
    code = _code(Q)
    S = cu_q.shape[0] - 1 if cu_q.dim() == 1 else -1
    if S < 0:
        _bad("cu_q must be an int32 [S+1] tensor")
    _ints(window=window, sinks=sinks, N_q=N_q, N_k=N_k)
    _full(cu_q, "cu_q", (S + 1,), torch.int32, Q.get_device())
    _full(cu_k, "cu_k", (S + 1,), torch.int32, Q.get_device())
    ctx, handle = _on(Q.device, stream)
    with ctx:
        out, lse, ldO = _attn_out(Q, H, N_q, d, out, lse)
        _check(load().mf_attention_window_varlen(S, _p(cu_q), _p(cu_k), *rows, code, H, H_kv, N_q,
                                                 N_k, d, _p(scale), window, sinks, _p(out), ldO,
                                                 _p(lse), handle))
    return out, lse


def _cache(K, V, lens, block_table, S, max_len):
    if K.dim() != 4 or not K.is_contiguous():
        _bad("K must be a contiguous [n_pages][H_kv][page][d] pool")
    _ints(max_len=max_len)
    where = K.get_device()
    _full(V, "V", K.shape, K.dtype, where)
    n_pages, H_kv, page, d = K.shape
    _full(lens, "lens", (S,), torch.int32, where)
    if block_table is not None:
        _same(where, torch.int32, block_table, "block_table")
        if block_table.dim() != 2 or block_table.shape[0] != S or not block_table.is_contiguous():
            _bad(f"block_table must be a contiguous [{S}][max_pages] tensor")
        max_pages = block_table.shape[1]
    else:
        max_pages = n_pages // S if S else 0
    return (_p(K), _p(V), n_pages, page, _p(block_table), max_pages, _p(lens), _code(K), S,
            int(max_len)), H_kv, d


def attention_decode_workspace_bytes(S: int, max_len: int, H: int, H_kv: int, d: int,
                                     window: int = 0, sinks: int = 0,
                                     with_mass: bool = False) -> int:
    return int(load().mf_attention_decode_workspace_bytes(S, max_len, H, H_kv, d, window, sinks,
                                                          int(with_mass)))


def attention_decode(Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, lens: torch.Tensor,
                     scale: torch.Tensor, max_len: int, *, window: int = 0, sinks: int = 0,
                     block_table: torch.Tensor | None = None, out: torch.Tensor | None = None,
                     lse: torch.Tensor | None = None, mass_in: torch.Tensor | None = None,
                     mass_out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                     stream=None):
    """(O, lse): one query per sequence over a cache (mf_attention_decode).

    Q [S][H][d]; K, V pools [n_pages][H_kv][page][d]; lens int32 [S] on the GPU, at
    most max_len (host); block_table int32 [S][max_pages], or None for a pool that
    holds n_pages // S consecutive pages of each sequence.  mass_out float32
    [S][H_kv][>= max_len] receives mass_in (None: 0) plus the weight of every cached
    row summed over the group's heads.  O is [S][H][d], lse float32 [S][H]."""
    _rows3(Q, "Q")
    S, H, d = Q.shape
    cache, H_kv, dk = _cache(K, V, lens, block_table, S, max_len)
    dev, where = K.device, K.get_device()
    _ints(window=window, sinks=sinks)
    _same(where, K.dtype, Q, "Q")
    _full(scale, "scale", (H,), torch.float32, where)
    if dk != d or (S and H > 1 and Q.stride(1) != d):
        _bad("Q must be [S][H][d] with its heads side by side, d as in the cache")
    ldmass = 0
    if mass_out is not None:
        if mass_out.dim() != 3:
            _bad("mass_out must be [S][H_kv][>= max_len]")
        ldmass = mass_out.shape[2]
        _full(mass_out, "mass_out", (S, H_kv, ldmass), torch.float32, where)
        _full(mass_in, "mass_in", (S, H_kv, ldmass), torch.float32, where)
    elif mass_in is not None:
        _bad("mass_in without mass_out")
    ctx, handle = _on(dev, stream)
    with ctx:
        if out is None:
            out = torch.empty(S, H, d, dtype=Q.dtype, device=dev)
        else:
            _same(where, Q.dtype, out, "out")
            if out.shape != (S, H, d) or (S and (out.stride(2) != 1 or
                                                        (H > 1 and out.stride(1) != d))):
                _bad("out must be [S][H][d] with contiguous rows")
        if lse is None:
            lse = torch.empty(S, H, dtype=torch.float32, device=dev)
        else:
            _full(lse, "lse", (S, H), torch.float32, where)
        L = load()
        need = 0 if workspace is not None else L.mf_attention_decode_workspace_bytes(
            S, int(max_len), H, H_kv, d, window, sinks, int(mass_out is not None))
        ws = _workspace(workspace, need, dev)
        _check(L.mf_attention_decode(_p(Q), Q.stride(0) if S > 1 else H * d, *cache, H, H_kv, d,
                                     _p(scale), window, sinks, _p(out),
                                     out.stride(0) if S > 1 else H * d, _p(lse), _p(mass_in),
                                     _p(mass_out), ldmass, _p(ws), _bytes_of(ws), handle))
    return out, lse


def key_mass_qk_workspace_bytes(dtype: torch.dtype, H: int, H_kv: int, N_q: int, N_k: int, d: int,
                                window: int = 0, sinks: int = 0) -> int:
    return int(load().mf_key_mass_qk_workspace_bytes(_DTYPE_CODE[dtype], H, H_kv, N_q, N_k, d,
                                                     window, sinks))


def key_mass_qk(Q: torch.Tensor, K: torch.Tensor, scale: torch.Tensor, lse: torch.Tensor, *,
                window: int = 0, sinks: int = 0, mass_in: torch.Tensor | None = None,
                out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                stream=None) -> torch.Tensor:
    """mass float32 [H_kv][N_k]: mass_in (None: 0) plus the attention weight that every
    key receives from the queries (mf_key_mass_qk).  Q [H][N_q][d], K [H_kv][N_k][d], lse
    [H][N_q] as attention_window returned it for the same mask."""
    _rows3(Q, "Q")
    _rows3(K, "K")
    H, N_q, d = Q.shape
    H_kv, N_k, dk = K.shape
    dev, where = Q.device, Q.get_device()
    code = _code(Q)
    if dk != d:
        _bad("K must match Q in d")
    _ints(window=window, sinks=sinks, N_q=N_q, N_k=N_k)
    _same(where, Q.dtype, K, "K")
    _full(scale, "scale", (H,), torch.float32, where)
    _full(lse, "lse", (H, N_q), torch.float32, where)
    _full(mass_in, "mass_in", (H_kv, N_k), torch.float32, where)
    ctx, handle = _on(dev, stream)
    with ctx:
        if out is None:
            out = torch.empty(H_kv, N_k, dtype=torch.float32, device=dev)
        else:
            _full(out, "out", (H_kv, N_k), torch.float32, where)
        L = load()
        need = 0 if workspace is not None else L.mf_key_mass_qk_workspace_bytes(
            code, H, H_kv, N_q, N_k, d, window, sinks)
        ws = _workspace(workspace, need, dev)
        _check(L.mf_key_mass_qk(_p(Q), Q.stride(1), Q.stride(0), _p(K), K.stride(1), K.stride(0),
                                _p(scale), _p(lse), code, H, H_kv, N_q, N_k, d, window, sinks,
                                _p(mass_in), _p(out), _p(ws), _bytes_of(ws), handle))
    return out


def cache_evict(mass: torch.Tensor, K: torch.Tensor, V: torch.Tensor, lens: torch.Tensor,
                budget: int, *, sinks: int = 0, recent: int = 0, max_len: int | None = None,
                block_table: torch.Tensor | None = None, K_out: torch.Tensor | None = None,
                V_out: torch.Tensor | None = None, mass_out: torch.Tensor | None = None,
                stream=None):
    """(kept, lens, K, V, mass) of a cache cut to `budget` rows a head (mf_cache_evict).

    mass float32 [S][H_kv][>= max_len] (max_len defaults to its last size); the cache as
    in attention_decode.  K_out, V_out [S][H_kv][cap][d] (cap >= budget; allocated with
    cap = budget by default, unused rows then 0) are pools with one page a sequence;
    mass_out [S][H_kv][cap] holds the kept masses, 0 behind them; kept int32
    [S][H_kv][budget], -1 behind the kept rows; lens int32 [S]."""
    if mass.dim() != 3 or not mass.is_contiguous():
        _bad("mass must be a contiguous [S][H_kv][>= max_len] tensor")
    S, _, ldmass = mass.shape
    if max_len is None:
        max_len = ldmass
    cache, H_kv, d = _cache(K, V, lens, block_table, S, max_len)
    dev, where = K.device, K.get_device()
    _full(mass, "mass", (S, H_kv, ldmass), torch.float32, where)
    budget = int(budget)
    given = [t for t in (K_out, V_out, mass_out) if t is not None]
    cap = given[0].shape[2] if given and given[0].dim() >= 3 else budget
    _full(K_out, "K_out", (S, H_kv, cap, d), K.dtype, where)
    _full(V_out, "V_out", (S, H_kv, cap, d), K.dtype, where)
    _full(mass_out, "mass_out", (S, H_kv, cap), torch.float32, where)
    _ints(budget=budget, sinks=sinks, recent=recent)
    if budget < 1:
        _bad(f"budget must be >= 1 (got {budget})")
    ctx, handle = _on(dev, stream)
    with ctx:
        if K_out is None:
            K_out = torch.zeros(S, H_kv, cap, d, dtype=K.dtype, device=dev)
        if V_out is None:
            V_out = torch.zeros(S, H_kv, cap, d, dtype=K.dtype, device=dev)
        if mass_out is None:
            mass_out = torch.empty(S, H_kv, cap, dtype=torch.float32, device=dev)
        kept = torch.empty(S, H_kv, budget, dtype=torch.int32, device=dev)
        left = torch.empty(S, dtype=torch.int32, device=dev)
        _check(load().mf_cache_evict(_p(mass), ldmass, *cache, H_kv, d, budget, int(sinks),
                                     int(recent), _p(K_out), _p(V_out), cap, _p(mass_out),
                                     _p(kept), _p(left), handle))
    return kept, left, K_out, V_out, mass_out
