"""ctypes binding of the full-attention calls of the C ABI (include/kda.h): causal
prompt attention and its gradients, attention of drafted tokens over a paged cache,
and the cache's pages. Argument marshalling only, as in :mod:`.kda`.

Work runs on ``stream`` (default: the current stream of the inputs' device); outputs
and workspaces that a call allocates belong to that stream.
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

from .kda import KdaError, _dt, _f, _i, _need, _p, _sz, _vp, lib

_ready = False


def _lib():
    """The library with the argument types of this module's calls set."""
    global _ready
    L = lib()
    if not _ready:
        sizes = {"kda_attn_fwd_workspace_size": [_i] * 7, "kda_attn_bwd_workspace_size": [_i] * 7,
                 "kda_attn_tree_workspace_size": [_i] * 8,
                 "kda_cache_reserve_workspace_size": [_i] * 3}
        calls = {
            "kda_attn_fwd": [_vp] * 3 + [_i, _vp] + [_i] * 6 + [_f, _vp, _vp, _vp, _sz, _vp],
            "kda_attn_bwd": [_vp] * 6 + [_i, _vp] + [_i] * 6 + [_f] + [_vp] * 4 + [_sz, _vp],
            "kda_attn_status": [_vp, _sz, ctypes.POINTER(_i), _vp],
            "kda_attn_tree": [_vp] * 3 + [_i] + [_vp] * 3 + [_i] * 8 + [_f, _vp, _vp, _vp, _sz,
                                                                     _vp],
            "kda_cache_fork": [_vp] * 4 + [_i] * 4 + [_vp] * 3,
            "kda_cache_reserve": [_vp] * 4 + [_i] * 4 + [_vp, _vp, _vp, _sz, _vp],
            "kda_cache_release": [_vp] * 4 + [_i] * 4 + [_vp],
            "kda_cache_append": [_vp, _vp, _i] + [_vp] * 5 + [_i] * 8 + [_vp],
            "kda_cache_compact": [_vp, _vp, _i] + [_vp] * 3 + [_i] * 7 + [_vp, _vp],
            "kda_cache_copy_pages": [_vp, _vp, _i, _vp] + [_i] * 5 + [_vp],
        }
        for names, res in ((sizes, _sz), (calls, _i)):
            for fn, args in names.items():
                getattr(L, fn).restype = res
                getattr(L, fn).argtypes = args
        _ready = True
    return L


def _same_device(device, **tensors):
    for name, t in tensors.items():
        if t is not None and t.device != device:
            raise ValueError(f"{name} is on {t.device}, expected {device}")


@contextlib.contextmanager
def _stream_of(device, stream):
    with torch.cuda.device(device), torch.cuda.stream(stream):
        yield


def _on(device, stream):
    """The context in which ``device`` and ``stream`` are the current ones (nothing where
    they are): what a call allocates belongs to the stream that its work runs on."""
    if stream is None or stream == torch.cuda.current_stream(device):
        if device.index == torch.cuda.current_device():
            return contextlib.nullcontext()
        return torch.cuda.device(device)
    return _stream_of(device, stream)


def _call(fn, args, device):
    st = getattr(_lib(), fn)(*args, ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream))
    if st != 0:
        raise KdaError(fn, st)


def _ws(workspace, need, device):
    if workspace is None:
        return torch.empty(max(int(need), 16), dtype=torch.uint8, device=device)
    if not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")
    _same_device(device, workspace=workspace)
    return workspace


def _bytes(t):
    return t.numel() * t.element_size()


def _out(t, name, shape, dtype, device):
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    _need(t, name, dtype, shape)
    _same_device(device, **{name: t})
    return t


def _prompt(q, k, v, cu_seqlens, scale):
    """Checks of a prompt call: its sizes (B, T, Hq, Hkv, d), sequences and scale."""
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q and k must be [B, T, heads, d]")
    B, T, Hq, d = q.shape
    Hkv = k.shape[2]
    _dt(q)
    _need(q, "q")
    _need(k, "k", q.dtype, (B, T, Hkv, d))
    _need(v, "v", q.dtype, (B, T, Hkv, d))
    n_seqs = 0
    if cu_seqlens is not None:
        _need(cu_seqlens, "cu_seqlens", torch.int32)
        n_seqs = cu_seqlens.shape[0] - 1
    _same_device(q.device, k=k, v=v, cu_seqlens=cu_seqlens)
    return (B, T, Hq, Hkv, d), n_seqs, float(d ** -0.5 if scale is None else scale)


def kda_attn_fwd(q, k, v, cu_seqlens=None, scale=None, o=None, lse=None, workspace=None,
                 stream=None):
    """Causal softmax attention over whole prompts with grouped heads (C: ``kda_attn_fwd``).

    q [B,T,Hq,d], k and v [B,T,Hkv,d] in bf16 or fp32, Hq a multiple of Hkv, d in
    {32, 64, 128}; cu_seqlens int32 [N+1] (then B = 1) or None; scale defaults to
    d ** -0.5. Returns (o [B,T,Hq,d] in q's dtype, lse [B,T,Hq] fp32, the natural
    logarithm of each row's sum). Tokens outside every sequence are not written.
    """
    (B, T, Hq, Hkv, d), n, scale = _prompt(q, k, v, cu_seqlens, scale)
    dev, dt = q.device, _dt(q)
    with _on(dev, stream):
        o = _out(o, "o", (B, T, Hq, d), q.dtype, dev)
        lse = _out(lse, "lse", (B, T, Hq), torch.float32, dev)
        ws = _ws(workspace, _lib().kda_attn_fwd_workspace_size(B, T, Hq, Hkv, d, n, dt), dev)
        _call("kda_attn_fwd", (_p(q), _p(k), _p(v), dt, _p(cu_seqlens), n, B, T, Hq, Hkv, d,
                               scale, _p(o), _p(lse), _p(ws), _bytes(ws)), dev)
    return o, lse


def kda_attn_bwd(q, k, v, o, lse, dO, cu_seqlens=None, scale=None, workspace=None, stream=None):
    """Gradients of <dO, o> of :func:`kda_attn_fwd` (C: ``kda_attn_bwd``), from its inputs
    and its two results. Returns a dict dq, dk, dv in q's dtype."""
    (B, T, Hq, Hkv, d), n, scale = _prompt(q, k, v, cu_seqlens, scale)
    dev, dt = q.device, _dt(q)
    _need(o, "o", q.dtype, (B, T, Hq, d))
    _need(dO, "dO", q.dtype, (B, T, Hq, d))
    _need(lse, "lse", torch.float32, (B, T, Hq))
    _same_device(dev, o=o, dO=dO, lse=lse)
    with _on(dev, stream):
        g = {"dq": torch.empty_like(q), "dk": torch.empty_like(k), "dv": torch.empty_like(v)}
        ws = _ws(workspace, _lib().kda_attn_bwd_workspace_size(B, T, Hq, Hkv, d, n, dt), dev)
        _call("kda_attn_bwd", (_p(q), _p(k), _p(v), _p(o), _p(lse), _p(dO), dt, _p(cu_seqlens),
                               n, B, T, Hq, Hkv, d, scale, _p(g["dq"]), _p(g["dk"]),
                               _p(g["dv"]), _p(ws), _bytes(ws)), dev)
    return g


def kda_attn_status(workspace, stream=None):
    """Status word of the last prompt call on ``workspace`` (C: ``kda_attn_status``; waits
    for the stream): (0, 0), or (6, code of the first bounded wait that ran out)."""
    code = _i(0)
    s = torch.cuda.current_stream(workspace.device) if stream is None else stream
    st = _lib().kda_attn_status(_p(workspace), _bytes(workspace), ctypes.byref(code),
                                ctypes.c_void_p(s.cuda_stream))
    if st not in (0, 6):
        raise KdaError("kda_attn_status", st)
    return st, code.value


def _pool(k_pages, v_pages):
    if k_pages.dim() != 4:
        raise ValueError("k_pages must be [P, Hkv, page_size, d]")
    _dt(k_pages)
    _need(k_pages, "k_pages")
    _need(v_pages, "v_pages", k_pages.dtype, k_pages.shape)
    _same_device(k_pages.device, v_pages=v_pages)
    return k_pages.shape


def _table(block_table):
    if block_table.dim() != 2:
        raise ValueError("block_table must be [N, M]")
    _need(block_table, "block_table", torch.int32)
    return block_table.shape


def _ints(device, shape, **tensors):
    for name, t in tensors.items():
        if t is not None:
            _need(t, name, torch.int32, shape)
    _same_device(device, **tensors)


def kda_attn_tree(q, k_pages, v_pages, block_table, ctx_lens, parents=None, scale=None, o=None,
                  lse=None, workspace=None, stream=None):
    """Attention of R <= 64 drafted tokens per sequence over a paged cache (C:
    ``kda_attn_tree``); R = 1 is the ordinary decode step.

    q [N,R,Hq,d]; k_pages, v_pages [P,Hkv,page_size,d] in q's dtype; block_table int32
    [N,M]; ctx_lens int32 [N], the tokens cached before the drafts, whose keys and
    values are at the positions that follow; parents int32 [N,R]: the index of each
    draft's parent, -1 for the last cached token, anything else for an absent token;
    None is a chain. Returns (o [N,R,Hq,d], lse [N,R,Hq] fp32); o = 0 and lse = -inf
    where a token sees nothing.
    """
    if q.dim() != 4:
        raise ValueError("q must be [N, R, Hq, d]")
    N, R, Hq, d = q.shape
    P, Hkv, page, _ = _pool(k_pages, v_pages)
    M = _table(block_table)[1]
    dev = q.device
    _need(q, "q", k_pages.dtype, (N, R, Hq, k_pages.shape[3]))
    _ints(dev, (N, M), block_table=block_table)
    _ints(dev, (N,), ctx_lens=ctx_lens)
    _ints(dev, (N, R), parents=parents)
    _same_device(dev, k_pages=k_pages)
    dt = _dt(q)
    scale = float(d ** -0.5 if scale is None else scale)
    with _on(dev, stream):
        o = _out(o, "o", (N, R, Hq, d), q.dtype, dev)
        lse = _out(lse, "lse", (N, R, Hq), torch.float32, dev)
        ws = _ws(workspace, _lib().kda_attn_tree_workspace_size(N, R, Hq, Hkv, d, M, page, dt),
                 dev)
        _call("kda_attn_tree", (_p(q), _p(k_pages), _p(v_pages), dt, _p(block_table),
                                _p(ctx_lens), _p(parents), N, R, Hq, Hkv, d, P, M, page, scale,
                                _p(o), _p(lse), _p(ws), _bytes(ws)), dev)
    return o, lse


def kda_cache_fork(refs, block_table, lens, parents, stream=None):
    """Row n of the new table is row parents[n] of the old one, whose rows end (C:
    ``kda_cache_fork``): a row taken twice is forked, one taken by nobody is freed.
    Updates refs in place; returns (new_table [N_out, M], new_lens [N_out])."""
    N, M = _table(block_table)
    dev, P, n_out = block_table.device, refs.shape[0], parents.shape[0]
    _ints(dev, (P,), refs=refs)
    _ints(dev, (N,), lens=lens)
    _ints(dev, (n_out,), parents=parents)
    with _on(dev, stream):
        table = torch.empty((n_out, M), dtype=torch.int32, device=dev)
        out = torch.empty(n_out, dtype=torch.int32, device=dev)
        _call("kda_cache_fork", (_p(refs), _p(block_table), _p(lens), _p(parents), N, n_out, M,
                                 P, _p(table), _p(out)), dev)
    return table, out


def kda_cache_reserve(refs, block_table, lens, add, page_size, workspace=None, stream=None):
    """Room for add[n] more tokens in every row (C: ``kda_cache_reserve``); updates refs,
    block_table and lens in place. Returns (copies int32 [N, 2], status int32 [1]):
    the pages to copy with :func:`kda_cache_copy_pages`, and 0, the number of missing
    pages, or -1 - n for a row that would be too long (then nothing has changed)."""
    N, M = _table(block_table)
    dev, P = block_table.device, refs.shape[0]
    _ints(dev, (P,), refs=refs)
    _ints(dev, (N,), lens=lens, add=add)
    with _on(dev, stream):
        copies = torch.empty((N, 2), dtype=torch.int32, device=dev)
        status = torch.empty(1, dtype=torch.int32, device=dev)
        ws = _ws(workspace, _lib().kda_cache_reserve_workspace_size(N, M, P), dev)
        _call("kda_cache_reserve", (_p(refs), _p(block_table), _p(lens), _p(add), N, M, P,
                                    int(page_size), _p(copies), _p(status), _p(ws), _bytes(ws)), dev)
    return copies, status


def kda_cache_release(refs, block_table, lens, new_lens, page_size, stream=None):
    """Cut every row to min(lens, new_lens) tokens and let go of the pages behind (C:
    ``kda_cache_release``); updates refs, block_table and lens in place."""
    N, M = _table(block_table)
    dev, P = block_table.device, refs.shape[0]
    _ints(dev, (P,), refs=refs)
    _ints(dev, (N,), lens=lens, new_lens=new_lens)
    with _on(dev, stream):
        _call("kda_cache_release", (_p(refs), _p(block_table), _p(lens), _p(new_lens), N, M, P,
                                    int(page_size)), dev)


def kda_cache_append(k_pages, v_pages, block_table, start, k_new, v_new, cu_seqlens=None,
                     stream=None):
    """Write k_new, v_new [B,T,Hkv,d] (sequences as for the prefill) into the rows' pages,
    sequence n from position start[n] on (C: ``kda_cache_append``)."""
    P, Hkv, page, d = _pool(k_pages, v_pages)
    N, M = _table(block_table)
    B, T = k_new.shape[:2]
    dev = k_pages.device
    for t, name in ((k_new, "k_new"), (v_new, "v_new")):
        _need(t, name, k_pages.dtype, (B, T, Hkv, d))
    n_seqs = 0
    if cu_seqlens is not None:
        _need(cu_seqlens, "cu_seqlens", torch.int32)
        n_seqs = cu_seqlens.shape[0] - 1
    if N != (n_seqs if cu_seqlens is not None else B):
        raise ValueError(f"block_table has {N} rows for {n_seqs or B} sequences")
    _ints(dev, (N,), start=start)
    _same_device(dev, k_new=k_new, v_new=v_new, cu_seqlens=cu_seqlens, block_table=block_table)
    with _on(dev, stream):
        _call("kda_cache_append", (_p(k_pages), _p(v_pages), _dt(k_pages), _p(block_table),
                                   _p(start), _p(k_new), _p(v_new), _p(cu_seqlens), n_seqs, B, T,
                                   Hkv, d, P, M, page), dev)


def kda_cache_compact(k_pages, v_pages, block_table, ctx_lens, path, stream=None):
    """Move the kept drafts path[n, :] (increasing indices, ended by -1) of every row
    together behind its ctx_lens[n] tokens (C: ``kda_cache_compact``). Returns the new
    lengths int32 [N], ctx_lens plus the number kept."""
    P, Hkv, page, d = _pool(k_pages, v_pages)
    N, M = _table(block_table)
    dev = k_pages.device
    if path.dim() != 2:
        raise ValueError("path must be [N, R]")
    R = path.shape[1]
    _ints(dev, (N, R), path=path)
    _ints(dev, (N,), ctx_lens=ctx_lens)
    _same_device(dev, block_table=block_table)
    with _on(dev, stream):
        out = torch.empty(N, dtype=torch.int32, device=dev)
        _call("kda_cache_compact", (_p(k_pages), _p(v_pages), _dt(k_pages), _p(block_table),
                                    _p(ctx_lens), _p(path), N, R, Hkv, d, P, M, page, _p(out)), dev)
    return out


def kda_cache_copy_pages(k_pages, v_pages, copies, stream=None):
    """Copy page copies[c, 0] to page copies[c, 1] in both pools, for every pair with page
    numbers in the pool (C: ``kda_cache_copy_pages``)."""
    P, Hkv, page, d = _pool(k_pages, v_pages)
    dev = k_pages.device
    C = copies.shape[0]
    _ints(dev, (C, 2), copies=copies)
    with _on(dev, stream):
        _call("kda_cache_copy_pages", (_p(k_pages), _p(v_pages), _dt(k_pages), _p(copies), C,
                                       Hkv, d, P, page), dev)
