"""The serving calls of include/gdn_serve.h: batch tables, the paged 8-bit cache
and its attention, and the delta rule on a pool of states.

The functions carry the C names and only marshal arguments, as the package's
others do; they are reached as gated_delta_rule_linear_amd.gdn_....  A call runs
on the device of its tensors, which all have to be on one device.
"""

from __future__ import annotations

import ctypes

import torch

import gated_delta_rule_linear_amd as _gdn

E4M3 = torch.float8_e4m3fn


def bind(lib):
    """Argument types of the serving calls (called once, when the library is loaded)."""
    P, i32, i64, sz, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
    lib.gdn_batch_tables.argtypes = [P, P, P, i32, i64, i32, P, i32, i32, P, P, i32, P, P, P, P, P, P, sz, P]
    lib.gdn_batch_tables.restype = i32
    lib.gdn_batch_tables_workspace_bytes.argtypes = [i32, i64]
    lib.gdn_batch_tables_workspace_bytes.restype = sz
    lib.gdn_cache_write.argtypes = [P, P, P, i64, P, P, P, P, i64, i32, i32, i32, i32, i32, P]
    lib.gdn_cache_write.restype = i32
    lib.gdn_cache_attention.argtypes = [P, P, P, P, P, P, P, P, P, i32, i64, i64, i64, i64, i32, i32, i32, f32, P, i32,
                                        i32, i32, i32, i32, P, sz, P]
    lib.gdn_cache_attention.restype = i32
    lib.gdn_cache_attention_workspace_bytes.argtypes = [i32, i64, i64, i64, i32, i32, i32, i32, i32, i32]
    lib.gdn_cache_attention_workspace_bytes.restype = sz
    lib.gdn_decode_pool.argtypes = [P, P, P, P, i32, P, P, P, P, P, i32, i64, i32, f32, f32, P, i32, i32, i32, i32, i32,
                                    P]
    lib.gdn_decode_pool.restype = i32


# These calls are made many times per generated token, so a check that passes
# costs a few attribute reads; what is wrong is found out in _refuse.
def _take(t, name, dtype, shape, device):
    """The address of a contiguous tensor of this type and shape on device number `device`."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == device and t.is_contiguous():
        return t.data_ptr()
    _refuse(t, name, dtype, shape)


def _refuse(t, name, dtype, shape):
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} must be on the device of the call's first tensor")


def _device_of(t, name):
    device = t.get_device()
    if device < 0:
        raise ValueError(f"{name} must be a device tensor")
    return device


def _elsewhere(device, stream):
    """Whether a call has to change the current device or stream first."""
    return stream is not None or device != _current_device()


class _On:
    """The device and the stream of a call, while it allocates and enqueues."""

    def __init__(self, device, stream):
        if stream is not None and stream.device_index != device:
            raise ValueError("stream must be of the device of the call's first tensor")
        self.entered = [torch.cuda.device(device)] + ([] if stream is None else [torch.cuda.stream(stream)])

    def __enter__(self):
        for c in self.entered:
            c.__enter__()

    def __exit__(self, *exc):
        for c in reversed(self.entered):
            c.__exit__(*exc)


_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice  # of a process that has device tensors


def _space(t, device):
    """Address and size of a caller's workspace."""
    if t.get_device() != device or not t.is_contiguous():
        raise ValueError("workspace must be contiguous and on the device of the call's first tensor")
    return t.data_ptr(), t.numel() * t.element_size()


def gdn_batch_tables_workspace_bytes(num_seqs: int, T_total: int) -> int:
    return int(_gdn._load().gdn_batch_tables_workspace_bytes(int(num_seqs), int(T_total)))


def gdn_batch_tables(context_lens, new_lens, T_total: int, page_size: int, block_table, page_counts, free_pages,
                     free_state, rows=None, workspace=None, stream=None):
    """Packed offsets, lengths, slots and positions of one step: returns (cu_seqlens [num_seqs + 1], kv_lens
    [num_seqs], slots [T_total], positions [T_total]), all int32, and updates block_table [num_rows, max_blocks],
    page_counts [num_rows], free_pages [num_pages] and free_state [3] (ring head, free pages, refused requests).

    context_lens and new_lens are int32 [num_seqs] on the device (new_lens < 0: the request has ended); rows int32
    [num_seqs] names each request's row (None: row n).  kv_lens - context_lens is the tokens that were taken: 0 for a
    request that found no pages, whose tokens stay in cu_seqlens; as `commit` of gdn_decode_pool it keeps their states
    as they are."""
    lib, dev, i32 = _gdn._load(), _device_of(context_lens, "context_lens"), torch.int32
    if _elsewhere(dev, stream):
        with _On(dev, stream):
            return gdn_batch_tables(context_lens, new_lens, T_total, page_size, block_table, page_counts, free_pages,
                                    free_state, rows, workspace)
    (n,), (num_rows, max_blocks), (pages,) = context_lens.shape, block_table.shape, free_pages.shape
    cp, np = _take(context_lens, "context_lens", i32, (n,), dev), _take(new_lens, "new_lens", i32, (n,), dev)
    rp = None if rows is None else _take(rows, "rows", i32, (n,), dev)
    table = _take(block_table, "block_table", i32, (num_rows, max_blocks), dev)
    counts = _take(page_counts, "page_counts", i32, (num_rows,), dev)
    ring, state = _take(free_pages, "free_pages", i32, (pages,), dev), _take(free_state, "free_state", i32, (3,), dev)
    T = int(T_total)
    if T < 0:
        raise ValueError("T_total must be >= 0")
    need = lib.gdn_batch_tables_workspace_bytes(n, T) // 4 if workspace is None else 0
    # one block for the four results and the workspace
    cu, kv, slots, pos, own = torch.split_with_sizes(context_lens.new_empty(2 * n + 1 + 2 * T + need),
                                                     (n + 1, n, T, T, need))
    base = cu.data_ptr()
    wp, wb = (own.data_ptr(), 4 * need) if workspace is None else _space(workspace, dev)
    st = lib.gdn_batch_tables(cp, np, rp, n, T, page_size, table, num_rows, max_blocks, counts, ring, pages, state, base,
                              base + 4 * (n + 1), base + 4 * (2 * n + 1), base + 4 * (2 * n + 1 + T), wp, wb, _stream(dev))
    if st:
        _gdn._check(st, "gdn_batch_tables")
    return cu, kv, slots, pos


def _cache(k_cache, v_cache, k_scale, v_scale, dev):
    (pages, hkv, page, dk), (_, _, _, dv, _) = k_cache.shape, v_cache.shape
    return (pages, page, hkv, dk, dv, _take(k_cache, "k_cache", E4M3, (pages, hkv, page, dk), dev),
            _take(v_cache, "v_cache", E4M3, (pages, hkv, page // 16, dv, 16), dev),
            _take(k_scale, "k_scale", torch.float32, (pages, hkv), dev),
            _take(v_scale, "v_scale", torch.float32, (pages, hkv), dev))


def gdn_cache_write(k, v, slots, k_cache, v_cache, k_scale, v_scale, stream=None) -> None:
    """New keys k [T, H_kv, dk] and values v [T, H_kv, dv] (bf16 or fp32) to their slots (int32 [T]) of the paged cache:
    k_cache [pages, H_kv, page, dk] and v_cache [pages, H_kv, page / 16, dv, 16] (torch.float8_e4m3fn), k_scale and
    v_scale [pages, H_kv] (fp32 powers of two), updated in place."""
    lib, dt, dev = _gdn._load(), _gdn._dtype_code(k), _device_of(k, "k")
    if _elsewhere(dev, stream):
        with _On(dev, stream):
            return gdn_cache_write(k, v, slots, k_cache, v_cache, k_scale, v_scale)
    pages, page, hkv, dk, dv, kc, vc, ks, vs = _cache(k_cache, v_cache, k_scale, v_scale, dev)
    T = k.shape[0]
    kp, vp = _take(k, "k", k.dtype, (T, hkv, dk), dev), _take(v, "v", k.dtype, (T, hkv, dv), dev)
    sp = _take(slots, "slots", torch.int32, (T,), dev)
    st = lib.gdn_cache_write(kp, vp, sp, T, kc, vc, ks, vs, pages, page, hkv, dk, dv, dt, _stream(dev))
    if st:
        _gdn._check(st, "gdn_cache_write")


def gdn_cache_attention_workspace_bytes(num_seqs: int, T_total: int, max_new: int, max_kv: int, page_size: int,
                                        max_blocks: int, H: int, H_kv: int, dk: int, dv: int) -> int:
    return int(_gdn._load().gdn_cache_attention_workspace_bytes(num_seqs, T_total, int(max_new), int(max_kv), page_size,
                                                                max_blocks, H, H_kv, dk, dv))


def gdn_cache_attention(q, k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, cu_seqlens, rows=None, scale=None,
                        max_new: int = 0, max_kv: int = 0, o=None, workspace=None, stream=None):
    """Causal attention of the step's queries q [T, H, dk] (bf16 or fp32) over the paged cache (see gdn_cache_write);
    returns o [T, H, dv].  Request n's queries are rows cu_seqlens[n] .. cu_seqlens[n + 1] - 1 and the last of the
    kv_lens[n] tokens that row rows[n] (None: row n) of block_table holds.  scale: 1 / sqrt(dk) by default.  max_new
    and max_kv, host-side bounds on a request's new tokens and on kv_lens, help to plan (0: unknown).  Rows behind
    cu_seqlens[-1] are not written: they keep what a given o holds, and of an o made here they are uninitialised."""
    lib, dt, dev, i32 = _gdn._load(), _gdn._dtype_code(q), _device_of(q, "q"), torch.int32
    if _elsewhere(dev, stream):
        with _On(dev, stream):
            return gdn_cache_attention(q, k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, cu_seqlens, rows, scale,
                                       max_new, max_kv, o, workspace)
    pages, page, hkv, dk, dv, kc, vc, ks, vs = _cache(k_cache, v_cache, k_scale, v_scale, dev)
    (T, H, _), (n,), (num_rows, max_blocks) = q.shape, kv_lens.shape, block_table.shape
    qp = _take(q, "q", q.dtype, (T, H, dk), dev)
    table = _take(block_table, "block_table", i32, (num_rows, max_blocks), dev)
    rp = None if rows is None else _take(rows, "rows", i32, (n,), dev)
    kv, cu = _take(kv_lens, "kv_lens", i32, (n,), dev), _take(cu_seqlens, "cu_seqlens", i32, (n + 1,), dev)
    if o is None:
        o = torch.empty_like(q) if dv == dk else q.new_empty((T, H, dv))
        op = o.data_ptr()
    else:
        op = _take(o, "o", q.dtype, (T, H, dv), dev)
    if workspace is None:
        wp, wb = None, lib.gdn_cache_attention_workspace_bytes(n, T, max_new, max_kv, page, max_blocks, H, hkv, dk, dv)
        if wb:
            workspace = k_scale.new_empty((wb + 3) // 4)  # fp32
            wp = workspace.data_ptr()
    else:
        wp, wb = _space(workspace, dev)
    st = lib.gdn_cache_attention(qp, kc, vc, ks, vs, table, rp, kv, cu, n, T, max_new, max_kv, pages, page, num_rows,
                                 max_blocks, dk ** -0.5 if scale is None else scale, op, H, hkv, dk, dv, dt, wp, wb,
                                 _stream(dev))
    if st:
        _gdn._check(st, "gdn_cache_attention")
    return o


def gdn_decode_pool(q, k, v, g, beta, states, slots, cu_seqlens=None, commit=None, q_scale: float = 1.0,
                    l2_eps: float = 0.0, o=None, stream=None):
    """The delta rule on a pool of states [num_slots, H, dk, dv] (fp32, updated in place), one or a few tokens for each
    request; returns o [T, H, dv].  q, k [T, H_k, dk] and v [T, H, dv] in bf16 or fp32 (head h reads key head
    h // (H // H_k)); g [T, H, dk] or [T, H] and beta [T, H] in fp32; slots int32 [num_seqs]; cu_seqlens int32
    [num_seqs + 1] (None: one token each); commit int32 [num_seqs]: the tokens whose update is kept (None: all);
    l2_eps > 0: q and k are L2-normalised in the kernel.  Rows behind cu_seqlens[-1] and those of requests whose slot is
    outside the pool are not written: they keep what a given o holds, and of an o made here they are uninitialised."""
    lib, dt, dev, i32, f32 = _gdn._load(), _gdn._dtype_code(q), _device_of(q, "q"), torch.int32, torch.float32
    if _elsewhere(dev, stream):
        with _On(dev, stream):
            return gdn_decode_pool(q, k, v, g, beta, states, slots, cu_seqlens, commit, q_scale, l2_eps, o)
    (T, hk, dk), (num_slots, H, _, dv), (n,) = q.shape, states.shape, slots.shape
    head_gate = g.dim() == 2
    qp, kp = _take(q, "q", q.dtype, (T, hk, dk), dev), _take(k, "k", q.dtype, (T, hk, dk), dev)
    vp = _take(v, "v", q.dtype, (T, H, dv), dev)
    gp, bp = _take(g, "g", f32, (T, H) if head_gate else (T, H, dk), dev), _take(beta, "beta", f32, (T, H), dev)
    sp, lp = _take(states, "states", f32, (num_slots, H, dk, dv), dev), _take(slots, "slots", i32, (n,), dev)
    cp = None if cu_seqlens is None else _take(cu_seqlens, "cu_seqlens", i32, (n + 1,), dev)
    mp = None if commit is None else _take(commit, "commit", i32, (n,), dev)
    if o is None:
        o = torch.empty_like(v)
        op = o.data_ptr()
    else:
        op = _take(o, "o", q.dtype, (T, H, dv), dev)
    st = lib.gdn_decode_pool(qp, kp, vp, gp, head_gate, bp, sp, lp, cp, mp, n, T, num_slots, q_scale, l2_eps, op, H, hk, dk,
                             dv, dt, _stream(dev))
    if st:
        _gdn._check(st, "gdn_decode_pool")
    return o


__all__ = ["gdn_batch_tables", "gdn_batch_tables_workspace_bytes", "gdn_cache_write", "gdn_cache_attention",
           "gdn_cache_attention_workspace_bytes", "gdn_decode_pool"]
