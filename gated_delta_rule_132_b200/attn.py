"""ctypes binding of the full-attention calls of the C ABI (include/kda.h): causal
prompt attention and its gradients, attention of drafted tokens over a paged cache,
and the cache's pages. Argument marshalling only, as in :mod:`.kda`.

Work runs on ``stream`` (default: the current stream of the inputs' device); outputs
and workspaces that a call allocates belong to that stream.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools

import torch

from .kda import KDA_DTYPE_BF16, KDA_DTYPE_F32, KdaError, _f, _i, _need, _sz, _vp, lib

_SIZES = {"kda_attn_fwd_workspace_size": 7, "kda_attn_bwd_workspace_size": 7,
          "kda_attn_tree_workspace_size": 8, "kda_cache_reserve_workspace_size": 3}
_CALLS = {
    "kda_attn_fwd": [_vp] * 3 + [_i, _vp] + [_i] * 6 + [_f, _vp, _vp, _vp, _sz, _vp],
    "kda_attn_bwd": [_vp] * 6 + [_i, _vp] + [_i] * 6 + [_f] + [_vp] * 4 + [_sz, _vp],
    "kda_attn_status": [_vp, _sz, ctypes.POINTER(_i), _vp],
    "kda_attn_tree": [_vp] * 3 + [_i] + [_vp] * 3 + [_i] * 8 + [_f, _vp, _vp, _vp, _sz, _vp],
    "kda_cache_fork": [_vp] * 4 + [_i] * 4 + [_vp] * 3,
    "kda_cache_reserve": [_vp] * 4 + [_i] * 4 + [_vp, _vp, _vp, _sz, _vp],
    "kda_cache_release": [_vp] * 4 + [_i] * 4 + [_vp],
    "kda_cache_append": [_vp, _vp, _i] + [_vp] * 5 + [_i] * 8 + [_vp],
    "kda_cache_compact": [_vp, _vp, _i] + [_vp] * 3 + [_i] * 7 + [_vp, _vp],
    "kda_cache_copy_pages": [_vp, _vp, _i, _vp] + [_i] * 5 + [_vp],
}
_raw_stream = torch._C._cuda_getCurrentRawStream  # the current stream's handle, by device index
_DTYPES = {torch.float32: KDA_DTYPE_F32, torch.bfloat16: KDA_DTYPE_BF16}
_ready = False


def _lib():
    """The library with the argument types of this module's calls set."""
    global _ready
    L = lib()
    if not _ready:
        for fn, count in _SIZES.items():
            getattr(L, fn).restype = _sz
            getattr(L, fn).argtypes = [_i] * count
        for fn, args in _CALLS.items():
            getattr(L, fn).restype = _i
            getattr(L, fn).argtypes = args
        _ready = True
    return L


@functools.lru_cache(maxsize=4096)
def _size(fn, *args):
    """Workspace bytes: a function of the sizes alone."""
    return max(int(_function(fn)(*args)), 16)


def _dt(t):
    dt = _DTYPES.get(t.dtype)
    if dt is None:
        raise TypeError(f"q/k/v must be bf16 or fp32, got {t.dtype}")
    return dt


def _p(t):
    return None if t is None else t.data_ptr()


def _check(t, name, dtype, shape, device):
    """A contiguous CUDA tensor of this type, shape (None: any) and device."""
    if (t.dtype is dtype and (shape is None or t.shape == shape) and t.is_cuda
            and t.is_contiguous() and t.device == device):
        return
    _need(t, name, dtype, shape)
    raise ValueError(f"{name} is on {t.device}, expected {device}")


@contextlib.contextmanager
def _stream_of(device, stream):
    with torch.cuda.device(device), torch.cuda.stream(stream):
        yield


def _on(device, stream, body, *args):
    """``body(*args)`` with ``device`` and ``stream`` as the current ones: what a call allocates
    belongs to the stream that its work runs on."""
    if stream is not None and stream.device != device:
        raise ValueError(f"stream is on {stream.device}, expected {device}")
    if stream is not None and stream != torch.cuda.current_stream(device):
        with _stream_of(device, stream):
            return body(*args)
    if device.index == torch.cuda.current_device():
        return body(*args)
    with torch.cuda.device(device):
        return body(*args)


@functools.lru_cache(maxsize=None)
def _function(fn):
    return getattr(_lib(), fn)


def _call(fn, device, *args):
    """C call ``fn`` on the device's current stream."""
    st = _function(fn)(*args, _raw_stream(device.index))
    if st:
        raise KdaError(fn, st)


def _ws(workspace, like, fn, *sizes):
    """The caller's workspace, checked, or a new one: the tensor and its bytes."""
    if workspace is None:
        need = _size(fn, *sizes)
        return like.new_empty(need, dtype=torch.uint8), need
    _check(workspace, "workspace", workspace.dtype, None, like.device)
    return workspace, workspace.numel() * workspace.element_size()


def _out(t, name, like, dtype, shape):
    """The caller's output tensor, checked, or a new one on the device of ``like``."""
    if t is None:
        return like.new_empty(shape) if dtype is like.dtype else like.new_empty(shape, dtype=dtype)
    _check(t, name, dtype, shape, like.device)
    return t


def _sequences(cu_seqlens, device):
    """Checks of packed sequences' offsets: their number, 0 without offsets."""
    if cu_seqlens is None:
        return 0
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:  # empty ones have no address to tell them from none
        raise ValueError(f"cu_seqlens must be [N + 1] with N >= 1, got {tuple(cu_seqlens.shape)}")
    _check(cu_seqlens, "cu_seqlens", torch.int32, None, device)
    return cu_seqlens.shape[0] - 1


def _prompt(q, k, v, cu_seqlens, scale):
    """Checks of a prompt call: its sizes (B, T, Hq, Hkv, d), sequences, dtype and scale."""
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q and k must be [B, T, heads, d]")
    B, T, Hq, d = q.shape
    Hkv = k.shape[2]
    dt, dev = _dt(q), q.device
    _check(q, "q", q.dtype, None, dev)
    _check(k, "k", q.dtype, (B, T, Hkv, d), dev)
    _check(v, "v", q.dtype, (B, T, Hkv, d), dev)
    return (B, T, Hq, Hkv, d), _sequences(cu_seqlens, dev), dt, d ** -0.5 if scale is None else float(scale)


def kda_attn_fwd(q, k, v, cu_seqlens=None, scale=None, o=None, lse=None, workspace=None,
                 stream=None):
    """Causal softmax attention over whole prompts with grouped heads (C: ``kda_attn_fwd``).

    q [B,T,Hq,d], k and v [B,T,Hkv,d] in bf16 or fp32, Hq a multiple of Hkv, d in
    {32, 64, 128}; cu_seqlens int32 [N+1] (then B = 1) or None; scale defaults to
    d ** -0.5. Returns (o [B,T,Hq,d] in q's dtype, lse [B,T,Hq] fp32, the natural
    logarithm of each row's sum). Tokens outside every sequence are not written.
    """
    sizes, n, dt, scale = _prompt(q, k, v, cu_seqlens, scale)
    return _on(q.device, stream, _fwd, q, k, v, cu_seqlens, sizes, n, dt, scale, o, lse, workspace)


def _fwd(q, k, v, cu_seqlens, sizes, n, dt, scale, o, lse, workspace):
    o = _out(o, "o", q, q.dtype, q.shape)
    lse = _out(lse, "lse", q, torch.float32, sizes[:3])
    ws, size = _ws(workspace, q, "kda_attn_fwd_workspace_size", *sizes, n, dt)
    _call("kda_attn_fwd", q.device, q.data_ptr(), k.data_ptr(), v.data_ptr(), dt, _p(cu_seqlens), n,
          *sizes, scale, o.data_ptr(), lse.data_ptr(), ws.data_ptr(), size)
    return o, lse


def kda_attn_bwd(q, k, v, o, lse, dO, cu_seqlens=None, scale=None, workspace=None, stream=None):
    """Gradients of <dO, o> of :func:`kda_attn_fwd` (C: ``kda_attn_bwd``), from its inputs
    and its two results. Returns a dict dq, dk, dv in q's dtype; tokens outside every
    sequence are not written."""
    sizes, n, dt, scale = _prompt(q, k, v, cu_seqlens, scale)
    dev = q.device
    _check(o, "o", q.dtype, q.shape, dev)
    _check(dO, "dO", q.dtype, q.shape, dev)
    _check(lse, "lse", torch.float32, q.shape[:3], dev)
    return _on(dev, stream, _bwd, q, k, v, o, lse, dO, cu_seqlens, sizes, n, dt, scale, workspace)


def _bwd(q, k, v, o, lse, dO, cu_seqlens, sizes, n, dt, scale, workspace):
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    ws, size = _ws(workspace, q, "kda_attn_bwd_workspace_size", *sizes, n, dt)
    _call("kda_attn_bwd", q.device, q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
          lse.data_ptr(), dO.data_ptr(), dt, _p(cu_seqlens), n, *sizes, scale, dq.data_ptr(),
          dk.data_ptr(), dv.data_ptr(), ws.data_ptr(), size)
    return {"dq": dq, "dk": dk, "dv": dv}


def kda_attn_status(workspace, stream=None):
    """Status word of the last prompt call on ``workspace`` (C: ``kda_attn_status``; waits
    for the stream): (0, 0), or (6, code of the first bounded wait that ran out)."""
    code = _i(0)
    s = torch.cuda.current_stream(workspace.device) if stream is None else stream
    st = _lib().kda_attn_status(_p(workspace), workspace.numel() * workspace.element_size(),
                                ctypes.byref(code), ctypes.c_void_p(s.cuda_stream))
    if st not in (0, 6):
        raise KdaError("kda_attn_status", st)
    return st, code.value


def _pool(k_pages, v_pages):
    """Checks of a pool: its sizes (P, Hkv, page_size, d) and dtype."""
    if k_pages.dim() != 4:
        raise ValueError("k_pages must be [P, Hkv, page_size, d]")
    dt, dev = _dt(k_pages), k_pages.device
    _check(k_pages, "k_pages", k_pages.dtype, None, dev)
    _check(v_pages, "v_pages", k_pages.dtype, k_pages.shape, dev)
    return k_pages.shape, dt


def _ints(t, name, shape, device):
    _check(t, name, torch.int32, shape, device)


def _table(block_table, device):
    if block_table.dim() != 2:
        raise ValueError("block_table must be [N, M]")
    _ints(block_table, "block_table", None, device)
    return block_table.shape


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
    dev = q.device
    (P, Hkv, page, _), dt = _pool(k_pages, v_pages)
    M = _table(block_table, dev)[1]
    _check(q, "q", k_pages.dtype, (N, R, Hq, k_pages.shape[3]), k_pages.device)
    _ints(block_table, "block_table", (N, M), dev)
    _ints(ctx_lens, "ctx_lens", (N,), dev)
    if parents is not None:
        _ints(parents, "parents", (N, R), dev)
    scale = d ** -0.5 if scale is None else float(scale)
    return _on(dev, stream, _tree, q, k_pages, v_pages, block_table, ctx_lens, parents,
               (N, R, Hq, Hkv, d), P, (M, page), dt, scale, o, lse, workspace)


def _tree(q, k_pages, v_pages, block_table, ctx_lens, parents, sizes, P, table, dt, scale, o, lse,
          workspace):
    o = _out(o, "o", q, q.dtype, q.shape)
    lse = _out(lse, "lse", q, torch.float32, sizes[:3])
    ws, size = _ws(workspace, q, "kda_attn_tree_workspace_size", *sizes, *table, dt)
    _call("kda_attn_tree", q.device, q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), dt,
          block_table.data_ptr(), ctx_lens.data_ptr(), _p(parents), *sizes, P, *table, scale,
          o.data_ptr(), lse.data_ptr(), ws.data_ptr(), size)
    return o, lse


def kda_cache_fork(refs, block_table, lens, parents, stream=None):
    """Row n of the new table is row parents[n] of the old one, whose rows end (C:
    ``kda_cache_fork``): a row taken twice is forked, one taken by nobody is freed.
    Updates refs in place; returns (new_table [N_out, M], new_lens [N_out])."""
    dev = block_table.device
    N, M = _table(block_table, dev)
    n_out = parents.shape[0]
    _ints(refs, "refs", None, dev)
    _ints(lens, "lens", (N,), dev)
    _ints(parents, "parents", (n_out,), dev)

    def body():
        table, out = lens.new_empty((n_out, M)), lens.new_empty(n_out)
        _call("kda_cache_fork", dev, refs.data_ptr(), block_table.data_ptr(), lens.data_ptr(),
              parents.data_ptr(), N, n_out, M, refs.numel(), table.data_ptr(), out.data_ptr())
        return table, out

    return _on(dev, stream, body)


def kda_cache_reserve(refs, block_table, lens, add, page_size, workspace=None, stream=None):
    """Room for add[n] more tokens in every row (C: ``kda_cache_reserve``); updates refs,
    block_table and lens in place. Returns (copies int32 [N, 2], status int32 [1]):
    the pages to copy with :func:`kda_cache_copy_pages`, and 0, the number of missing
    pages, or -1 - n for a row that would be too long (then nothing has changed)."""
    dev = block_table.device
    N, M = _table(block_table, dev)
    P = refs.numel()
    _ints(refs, "refs", None, dev)
    _ints(lens, "lens", (N,), dev)
    _ints(add, "add", (N,), dev)

    def body():
        copies, status = lens.new_empty((N, 2)), lens.new_empty(1)
        ws, size = _ws(workspace, lens, "kda_cache_reserve_workspace_size", N, M, P)
        _call("kda_cache_reserve", dev, refs.data_ptr(), block_table.data_ptr(), lens.data_ptr(),
              add.data_ptr(), N, M, P, int(page_size), copies.data_ptr(), status.data_ptr(),
              ws.data_ptr(), size)
        return copies, status

    return _on(dev, stream, body)


def kda_cache_release(refs, block_table, lens, new_lens, page_size, stream=None):
    """Cut every row to min(lens, new_lens) tokens and let go of the pages behind (C:
    ``kda_cache_release``); updates refs, block_table and lens in place."""
    dev = block_table.device
    N, M = _table(block_table, dev)
    _ints(refs, "refs", None, dev)
    _ints(lens, "lens", (N,), dev)
    _ints(new_lens, "new_lens", (N,), dev)
    _on(dev, stream, _call, "kda_cache_release", dev, refs.data_ptr(), block_table.data_ptr(),
        lens.data_ptr(), new_lens.data_ptr(), N, M, refs.numel(), int(page_size))


def kda_cache_append(k_pages, v_pages, block_table, start, k_new, v_new, cu_seqlens=None,
                     stream=None):
    """Write k_new, v_new [B,T,Hkv,d] (sequences as for the prefill) into the rows' pages,
    sequence n from position start[n] on (C: ``kda_cache_append``)."""
    dev = k_pages.device
    (P, Hkv, page, d), dt = _pool(k_pages, v_pages)
    N, M = _table(block_table, dev)
    B, T = k_new.shape[:2]
    _check(k_new, "k_new", k_pages.dtype, (B, T, Hkv, d), dev)
    _check(v_new, "v_new", k_pages.dtype, (B, T, Hkv, d), dev)
    n_seqs = _sequences(cu_seqlens, dev)
    if N != (n_seqs if cu_seqlens is not None else B):
        raise ValueError(f"block_table has {N} rows for {n_seqs or B} sequences")
    _ints(start, "start", (N,), dev)
    _on(dev, stream, _call, "kda_cache_append", dev, k_pages.data_ptr(), v_pages.data_ptr(), dt,
        block_table.data_ptr(), start.data_ptr(), k_new.data_ptr(), v_new.data_ptr(),
        _p(cu_seqlens), n_seqs, B, T, Hkv, d, P, M, page)


def kda_cache_compact(k_pages, v_pages, block_table, ctx_lens, path, stream=None):
    """Move the kept drafts path[n, :] (increasing indices, ended by -1) of every row
    together behind its ctx_lens[n] tokens (C: ``kda_cache_compact``). Returns the new
    lengths int32 [N], ctx_lens plus the number kept."""
    dev = k_pages.device
    (P, Hkv, page, d), dt = _pool(k_pages, v_pages)
    N, M = _table(block_table, dev)
    if path.dim() != 2:
        raise ValueError("path must be [N, R]")
    R = path.shape[1]
    _ints(path, "path", (N, R), dev)
    _ints(ctx_lens, "ctx_lens", (N,), dev)

    def body():
        out = path.new_empty(N)
        _call("kda_cache_compact", dev, k_pages.data_ptr(), v_pages.data_ptr(), dt,
              block_table.data_ptr(), ctx_lens.data_ptr(), path.data_ptr(), N, R, Hkv, d, P, M,
              page, out.data_ptr())
        return out

    return _on(dev, stream, body)


def kda_cache_copy_pages(k_pages, v_pages, copies, stream=None):
    """Copy page copies[c, 0] to page copies[c, 1] in both pools, for every pair with page
    numbers in the pool (C: ``kda_cache_copy_pages``)."""
    dev = k_pages.device
    (P, Hkv, page, d), dt = _pool(k_pages, v_pages)
    C = copies.shape[0]
    _ints(copies, "copies", (C, 2), dev)
    _on(dev, stream, _call, "kda_cache_copy_pages", dev, k_pages.data_ptr(), v_pages.data_ptr(), dt,
        copies.data_ptr(), C, Hkv, d, P, page)
