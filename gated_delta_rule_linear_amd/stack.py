"""The calls of include/gdn_stack.h: queries and keys normalised and rotated, the
gated linear recurrence, and attention behind a common prefix.

The functions carry the C names and only marshal arguments, as the package's
others do; they are reached as gated_delta_rule_linear_amd.gdn_....  A call runs
on the device of its tensors, which all have to be on one device.
"""

from __future__ import annotations

import ctypes

import torch

import gated_delta_rule_linear_amd as _gdn

from .serve import _cache, _device_of, _elsewhere, _On, _space, _stream, _take

GDN_NORM_NONE, GDN_NORM_L2, GDN_NORM_RMS = range(3)
_DENSE = torch.contiguous_format


def bind(lib):
    """Argument types of these calls (called once, when the library is loaded)."""
    P, i32, i64, sz, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
    lib.gdn_qk_norm.argtypes = [P, i64, P, i64, i64, i32, i32, i32, i32, f32, P, P, P, P, i32, i32, f32, P, P, i32, P]
    lib.gdn_qk_norm.restype = i32
    lib.gdn_qk_norm_backward.argtypes = [P, i64, P, i64, P, P, i64, i32, i32, i32, i32, f32, P, P, P, P, i32, i32, f32, P,
                                         i64, P, i64, P, P, i32, P, sz, P]
    lib.gdn_qk_norm_backward.restype = i32
    lib.gdn_qk_norm_backward_workspace_bytes.argtypes = [i64, i32, i32, i32]
    lib.gdn_qk_norm_backward_workspace_bytes.restype = sz
    for name in ("gdn_scan_checkpoint_bytes", "gdn_scan_workspace_bytes", "gdn_scan_backward_workspace_bytes"):
        getattr(lib, name).argtypes = [i64, i32]
        getattr(lib, name).restype = sz
    lib.gdn_scan.argtypes = [P, P, P, i32, i64, i32, i32, P, P, P, P, i32, P, sz, P]
    lib.gdn_scan.restype = i32
    lib.gdn_scan_backward.argtypes = [P, P, P, i32, i64, i32, i32, P, P, P, P, P, P, P, i32, P, sz, P]
    lib.gdn_scan_backward.restype = i32
    lib.gdn_scan_pool.argtypes = [P, P, P, P, P, P, i32, i64, i32, i32, i32, P, i32, P]
    lib.gdn_scan_pool.restype = i32
    lib.gdn_cache_attention_prefix.argtypes = [P, P, P, P, P, P, P, P, P, P, P, i32, i32, i64, i64, i64, i64, i64, i32, i32,
                                               i32, f32, P, i32, i32, i32, i32, i32, P, sz, P]
    lib.gdn_cache_attention_prefix.restype = i32
    lib.gdn_cache_attention_prefix_workspace_bytes.argtypes = [i32, i32, i64, i64, i64, i64, i32, i32, i32, i32, i32, i32]
    lib.gdn_cache_attention_prefix_workspace_bytes.restype = sz


# ---------------------------------------------------------------- norm and rotation


def _heads(t, name, dtype, tokens, d, device):
    """Address, token stride and heads of a [tokens, heads, d] tensor whose heads lie side by side."""
    if t.dim() == 3:
        (n, heads, channels), (stride, head, channel) = t.shape, t.stride()
        if n == tokens and channels == d and channel == 1 and (head == d or heads < 2) and t.dtype is dtype \
                and t.get_device() == device:
            return t.data_ptr(), stride if n > 1 else heads * d, heads
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 3 or t.shape[0] != tokens or t.shape[2] != d:
        raise ValueError(f"{name} must be [{tokens}, heads, {d}], got {list(t.shape)}")
    if t.get_device() != device:
        raise ValueError(f"{name} must be on the device of the call's first tensor")
    raise ValueError(f"the heads of a token of {name} must lie side by side")


def _norm_arguments(q, k, q_weight, k_weight, positions, inv_freq, dev):
    if q.dim() != 3:
        raise ValueError("q must have 3 dimensions")
    T, _, d = q.shape
    qp, qs, H = _heads(q, "q", q.dtype, T, d, dev)
    kp, ks, hk = (None, 0, 0) if k is None else _heads(k, "k", q.dtype, T, d, dev)
    f32 = torch.float32
    wq = None if q_weight is None else _take(q_weight, "q_weight", f32, (d,), dev)
    wk = None if k_weight is None else _take(k_weight, "k_weight", f32, (d,), dev)
    pos = freq = None
    rotary = 0
    if positions is not None and inv_freq is not None:
        (pairs,) = inv_freq.shape
        pos = _take(positions, "positions", torch.int32, (T,), dev)
        freq = _take(inv_freq, "inv_freq", f32, (pairs,), dev)
        rotary = 2 * pairs
    elif positions is not None or inv_freq is not None:
        raise ValueError("positions and inv_freq go together")
    return T, H, hk, d, qp, qs, kp, ks, wq, wk, pos, freq, rotary


def gdn_qk_norm(q, k=None, norm: int = GDN_NORM_RMS, eps: float = 1e-6, q_weight=None, k_weight=None, positions=None,
                inv_freq=None, interleaved: bool = False, q_scale: float = 1.0, q_out=None, k_out=None, stream=None):
    """Queries q [T, H, d] and keys k [T, H_k, d] (bf16 or fp32; None: no keys), normalised for each head (GDN_NORM_NONE,
    GDN_NORM_L2 or GDN_NORM_RMS), times q_weight and k_weight (fp32 [d], None: 1), rotated by positions (int32 [T]) times
    inv_freq (fp32 [rotary / 2]; both None: no rotation), queries times q_scale; returns (q_out, k_out).  q and k may be
    slices of one tensor [T, heads, d]: a token's heads have to lie side by side, tokens may be any multiple of 16 bytes
    apart.  Channels are paired (i, i + rotary / 2), or (2 i, 2 i + 1) with `interleaved`.  q_out and k_out are contiguous;
    they may be q and k themselves where those are."""
    lib, dt, dev = _gdn._load(), _gdn._dtype_code(q), _device_of(q, "q")
    if _elsewhere(dev, stream):
        with _On(dev, stream):
            return gdn_qk_norm(q, k, norm, eps, q_weight, k_weight, positions, inv_freq, interleaved, q_scale, q_out, k_out)
    T, H, hk, d, qp, qs, kp, ks, wq, wk, pos, freq, rotary = _norm_arguments(q, k, q_weight, k_weight, positions, inv_freq,
                                                                             dev)
    if q_out is None:
        q_out = torch.empty_like(q, memory_format=_DENSE)
        qo = q_out.data_ptr()
    else:
        qo = _take(q_out, "q_out", q.dtype, (T, H, d), dev)
    ko = None
    if k is None:
        if k_out is not None:
            raise ValueError("k_out without k")
    elif k_out is None:
        k_out = torch.empty_like(k, memory_format=_DENSE)
        ko = k_out.data_ptr()
    else:
        ko = _take(k_out, "k_out", q.dtype, (T, hk, d), dev)
    st = lib.gdn_qk_norm(qp, qs, kp, ks, T, H, hk, d, norm, eps, wq, wk, pos, freq, rotary, interleaved, q_scale, qo, ko, dt,
                         _stream(dev))
    if st:
        _gdn._check(st, "gdn_qk_norm")
    return q_out, k_out


def gdn_qk_norm_backward_workspace_bytes(T_total: int, H: int, H_k: int, d: int) -> int:
    return int(_gdn._load().gdn_qk_norm_backward_workspace_bytes(int(T_total), int(H), int(H_k), int(d)))


def gdn_qk_norm_backward(q, k, d_q_out, d_k_out, norm: int = GDN_NORM_RMS, eps: float = 1e-6, q_weight=None,
                         k_weight=None, positions=None, inv_freq=None, interleaved: bool = False, q_scale: float = 1.0,
                         dq=None, dk=None, want_d_weights: bool = True, workspace=None, stream=None):
    """Gradients of gdn_qk_norm for its inputs q and k (k None: no keys) and the gradients d_q_out [T, H, d] and d_k_out
    [T, H_k, d] of its outputs; returns (dq, dk, d_q_weight, d_k_weight).  The weights' gradients are fp32 [d], None for a
    weight that is None or without want_d_weights.  dq and dk may be slices of one tensor, as q and k may."""
    lib, dt, dev = _gdn._load(), _gdn._dtype_code(q), _device_of(q, "q")
    if _elsewhere(dev, stream):
        with _On(dev, stream):
            return gdn_qk_norm_backward(q, k, d_q_out, d_k_out, norm, eps, q_weight, k_weight, positions, inv_freq,
                                        interleaved, q_scale, dq, dk, want_d_weights, workspace)
    T, H, hk, d, qp, qs, kp, ks, wq, wk, pos, freq, rotary = _norm_arguments(q, k, q_weight, k_weight, positions, inv_freq,
                                                                             dev)
    if k is None and (d_k_out is not None or dk is not None):
        raise ValueError("d_k_out or dk without k")
    gq = _take(d_q_out, "d_q_out", q.dtype, (T, H, d), dev)
    gk = None if k is None else _take(d_k_out, "d_k_out", q.dtype, (T, hk, d), dev)
    if dq is None:
        dq = torch.empty_like(q, memory_format=_DENSE)
    dqp, dqs, h2 = _heads(dq, "dq", q.dtype, T, d, dev)
    dkp, dks, h3 = None, 0, 0
    if k is not None:
        if dk is None:
            dk = torch.empty_like(k, memory_format=_DENSE)
        dkp, dks, h3 = _heads(dk, "dk", q.dtype, T, d, dev)
    if h2 != H or h3 != hk:
        raise ValueError("dq and dk must have the heads of q and k")
    dwq = dwk = None
    wp, wb = None, 0
    if want_d_weights and (q_weight is not None or k_weight is not None):
        if q_weight is not None:
            dwq = torch.empty_like(q_weight)
        if k_weight is not None:
            dwk = torch.empty_like(k_weight)
        if workspace is None:
            wb = lib.gdn_qk_norm_backward_workspace_bytes(T, H, hk, d)
            workspace = (q_weight if q_weight is not None else k_weight).new_empty((wb + 3) // 4)
            wp = workspace.data_ptr()
        else:
            wp, wb = _space(workspace, dev)
    st = lib.gdn_qk_norm_backward(qp, qs, kp, ks, gq, gk, T, H, hk, d, norm, eps, wq, wk, pos, freq, rotary, interleaved,
                                  q_scale, dqp, dqs, dkp, dks, None if dwq is None else dwq.data_ptr(),
                                  None if dwk is None else dwk.data_ptr(), dt, wp, wb, _stream(dev))
    if st:
        _gdn._check(st, "gdn_qk_norm_backward")
    return dq, dk, dwq, dwk


# ---------------------------------------------------------------- the recurrence


def gdn_scan_checkpoint_bytes(T_total: int, C: int) -> int:
    return int(_gdn._load().gdn_scan_checkpoint_bytes(int(T_total), int(C)))


def gdn_scan_workspace_bytes(T_total: int, C: int) -> int:
    return int(_gdn._load().gdn_scan_workspace_bytes(int(T_total), int(C)))


def gdn_scan_backward_workspace_bytes(T_total: int, C: int) -> int:
    return int(_gdn._load().gdn_scan_backward_workspace_bytes(int(T_total), int(C)))


def gdn_scan_checkpoints(x):
    """A tensor for the checkpoints of gdn_scan over x [T, C], which gdn_scan_backward takes."""
    T, C = x.shape
    return torch.empty(gdn_scan_checkpoint_bytes(T, C) // 4, dtype=torch.float32, device=x.device)


def _scan_arguments(x, g, cu_seqlens, initial_state, checkpoints, lib, dev):
    if x.dim() != 2 or cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1:
        raise ValueError("x must have 2 dimensions, cu_seqlens 1 and at least one entry")
    (T, C), n, f32 = x.shape, cu_seqlens.shape[0] - 1, torch.float32
    xp, gp = _take(x, "x", x.dtype, (T, C), dev), _take(g, "g", f32, (T, C), dev)
    cu = _take(cu_seqlens, "cu_seqlens", torch.int32, (n + 1,), dev)
    s0 = None if initial_state is None else _take(initial_state, "initial_state", f32, (n, C), dev)
    kept = None
    if checkpoints is not None:
        kept = _take(checkpoints, "checkpoints", f32, (lib.gdn_scan_checkpoint_bytes(T, C) // 4,), dev)
    return T, C, n, xp, gp, cu, s0, kept


def _scratch(g, workspace, need, dev):
    if workspace is not None:
        return workspace, *_space(workspace, dev)
    workspace = g.new_empty((need + 3) // 4)
    return workspace, workspace.data_ptr(), need


def gdn_scan(x, g, cu_seqlens, mix: bool = False, initial_state=None, final_state=None, h=None, checkpoints=None,
             output_final_state: bool = True, workspace=None, stream=None):
    """The gated linear recurrence h_t = e^g_t h_{t-1} + x_t of every channel (with `mix`: + (1 - e^g_t) x_t) over packed
    sequences; returns (h, final_state or None).  x [T, C] in bf16 or fp32, C a multiple of 4; g [T, C] in fp32, at most 0;
    cu_seqlens int32 [num_seqs + 1]; initial_state and final_state fp32 [num_seqs, C], which must not overlap.  checkpoints,
    from gdn_scan_checkpoints(x), receives what gdn_scan_backward takes.  h may be x.  Rows behind cu_seqlens[-1] are not
    written."""
    lib, dt, dev = _gdn._load(), _gdn._dtype_code(x), _device_of(x, "x")
    if _elsewhere(dev, stream):
        with _On(dev, stream):
            return gdn_scan(x, g, cu_seqlens, mix, initial_state, final_state, h, checkpoints, output_final_state, workspace)
    T, C, n, xp, gp, cu, s0, kept = _scan_arguments(x, g, cu_seqlens, initial_state, checkpoints, lib, dev)
    if h is None:
        h = torch.empty_like(x)
        hp = h.data_ptr()
    else:
        hp = _take(h, "h", x.dtype, (T, C), dev)
    if final_state is None and output_final_state:
        final_state = g.new_empty((n, C))
    sp = None if final_state is None else _take(final_state, "final_state", torch.float32, (n, C), dev)
    workspace, wp, wb = _scratch(g, workspace, lib.gdn_scan_workspace_bytes(T, C), dev)
    st = lib.gdn_scan(xp, gp, cu, n, T, C, mix, s0, sp, hp, kept, dt, wp, wb, _stream(dev))
    if st:
        _gdn._check(st, "gdn_scan")
    return h, final_state


def gdn_scan_backward(x, g, cu_seqlens, d_h, mix: bool = False, initial_state=None, d_final_state=None, checkpoints=None,
                      want_d_initial_state: bool = True, workspace=None, stream=None):
    """Gradients of gdn_scan: given d_h [T, C] (of x's type) and d_final_state (fp32 [num_seqs, C], None: 0) returns
    (dx, dg, d_initial_state); dx has the type of x, the others are fp32.  checkpoints: what gdn_scan wrote for the same
    inputs; without them the states are computed again.  Rows behind cu_seqlens[-1] are not written."""
    lib, dt, dev = _gdn._load(), _gdn._dtype_code(x), _device_of(x, "x")
    if _elsewhere(dev, stream):
        with _On(dev, stream):
            return gdn_scan_backward(x, g, cu_seqlens, d_h, mix, initial_state, d_final_state, checkpoints,
                                     want_d_initial_state, workspace)
    T, C, n, xp, gp, cu, s0, kept = _scan_arguments(x, g, cu_seqlens, initial_state, checkpoints, lib, dev)
    hp = _take(d_h, "d_h", x.dtype, (T, C), dev)
    fp = None if d_final_state is None else _take(d_final_state, "d_final_state", torch.float32, (n, C), dev)
    dx, dg = torch.empty_like(x), torch.empty_like(g)
    d_initial_state = g.new_empty((n, C)) if want_d_initial_state else None
    workspace, wp, wb = _scratch(g, workspace, lib.gdn_scan_backward_workspace_bytes(T, C), dev)
    st = lib.gdn_scan_backward(xp, gp, cu, n, T, C, mix, s0, kept, hp, fp, dx.data_ptr(), dg.data_ptr(),
                               None if d_initial_state is None else d_initial_state.data_ptr(), dt, wp, wb, _stream(dev))
    if st:
        _gdn._check(st, "gdn_scan_backward")
    return dx, dg, d_initial_state


def gdn_scan_pool(x, g, states, slots, cu_seqlens=None, commit=None, mix: bool = False, h=None, stream=None):
    """The recurrence of gdn_scan on a pool of states [num_slots, C] (fp32, updated in place), one or a few tokens for each
    request; returns h [T, C].  x [T, C] in bf16 or fp32, g [T, C] in fp32; slots int32 [num_seqs]; cu_seqlens int32
    [num_seqs + 1] (None: one token each); commit int32 [num_seqs]: the tokens whose update is kept (None: all).  Rows
    behind cu_seqlens[-1] and those of requests whose slot is outside the pool are not written: they keep what a given h
    holds, and of an h made here they are uninitialised."""
    lib, dt, dev, i32, f32 = _gdn._load(), _gdn._dtype_code(x), _device_of(x, "x"), torch.int32, torch.float32
    if _elsewhere(dev, stream):
        with _On(dev, stream):
            return gdn_scan_pool(x, g, states, slots, cu_seqlens, commit, mix, h)
    (T, C), (num_slots, _), (n,) = x.shape, states.shape, slots.shape
    xp, gp = _take(x, "x", x.dtype, (T, C), dev), _take(g, "g", f32, (T, C), dev)
    sp, lp = _take(states, "states", f32, (num_slots, C), dev), _take(slots, "slots", i32, (n,), dev)
    cp = None if cu_seqlens is None else _take(cu_seqlens, "cu_seqlens", i32, (n + 1,), dev)
    mp = None if commit is None else _take(commit, "commit", i32, (n,), dev)
    if h is None:
        h = torch.empty_like(x)
        hp = h.data_ptr()
    else:
        hp = _take(h, "h", x.dtype, (T, C), dev)
    st = lib.gdn_scan_pool(xp, gp, sp, lp, cp, mp, n, T, num_slots, C, mix, hp, dt, _stream(dev))
    if st:
        _gdn._check(st, "gdn_scan_pool")
    return h


# ---------------------------------------------------------------- attention behind a common beginning


def gdn_cache_attention_prefix_workspace_bytes(num_seqs: int, num_groups: int, T_total: int, max_new: int, max_kv: int,
                                               max_prefix: int, page_size: int, max_blocks: int, H: int, H_kv: int, dk: int,
                                               dv: int) -> int:
    return int(_gdn._load().gdn_cache_attention_prefix_workspace_bytes(num_seqs, num_groups, T_total, int(max_new),
                                                                       int(max_kv), int(max_prefix), page_size, max_blocks, H,
                                                                       H_kv, dk, dv))


def gdn_cache_attention_prefix(q, k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, cu_seqlens, group_offsets,
                               prefix_lens, rows=None, scale=None, max_new: int = 0, max_kv: int = 0, max_prefix: int = 0,
                               o=None, workspace=None, stream=None):
    """gdn_cache_attention for requests of which groups share the pages of a long beginning, which their queries then read
    once; returns o [T, H, dv].  Group i is requests group_offsets[i] .. group_offsets[i + 1] - 1 (int32 [num_groups + 1]);
    its first prefix_lens[i] tokens (int32 [num_groups]) lie in the same pages, that is, the rows of block_table of its
    requests agree in those blocks.  The other arguments are gdn_cache_attention's; max_prefix, a host-side bound on
    prefix_lens, helps to plan as max_new and max_kv do (0: unknown)."""
    lib, dt, dev, i32 = _gdn._load(), _gdn._dtype_code(q), _device_of(q, "q"), torch.int32
    if _elsewhere(dev, stream):
        with _On(dev, stream):
            return gdn_cache_attention_prefix(q, k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, cu_seqlens,
                                              group_offsets, prefix_lens, rows, scale, max_new, max_kv, max_prefix, o,
                                              workspace)
    pages, page, hkv, dk, dv, kc, vc, ks, vs = _cache(k_cache, v_cache, k_scale, v_scale, dev)
    (T, H, _), (n,), (num_rows, max_blocks), (groups,) = q.shape, kv_lens.shape, block_table.shape, prefix_lens.shape
    qp = _take(q, "q", q.dtype, (T, H, dk), dev)
    table = _take(block_table, "block_table", i32, (num_rows, max_blocks), dev)
    rp = None if rows is None else _take(rows, "rows", i32, (n,), dev)
    kv, cu = _take(kv_lens, "kv_lens", i32, (n,), dev), _take(cu_seqlens, "cu_seqlens", i32, (n + 1,), dev)
    go = _take(group_offsets, "group_offsets", i32, (groups + 1,), dev)
    pl = _take(prefix_lens, "prefix_lens", i32, (groups,), dev)
    if o is None:
        o = torch.empty_like(q) if dv == dk else q.new_empty((T, H, dv))
        op = o.data_ptr()
    else:
        op = _take(o, "o", q.dtype, (T, H, dv), dev)
    if workspace is None:
        wp, wb = None, lib.gdn_cache_attention_prefix_workspace_bytes(n, groups, T, max_new, max_kv, max_prefix, page,
                                                                      max_blocks, H, hkv, dk, dv)
        if wb:
            workspace = k_scale.new_empty((wb + 3) // 4)  # fp32
            wp = workspace.data_ptr()
    else:
        wp, wb = _space(workspace, dev)
    st = lib.gdn_cache_attention_prefix(qp, kc, vc, ks, vs, table, rp, kv, cu, go, pl, n, groups, T, max_new, max_kv,
                                        max_prefix, pages, page, num_rows, max_blocks, dk ** -0.5 if scale is None else scale,
                                        op, H, hkv, dk, dv, dt, wp, wb, _stream(dev))
    if st:
        _gdn._check(st, "gdn_cache_attention_prefix")
    return o


__all__ = ["GDN_NORM_NONE", "GDN_NORM_L2", "GDN_NORM_RMS", "gdn_qk_norm", "gdn_qk_norm_backward",
           "gdn_qk_norm_backward_workspace_bytes", "gdn_scan", "gdn_scan_backward", "gdn_scan_pool", "gdn_scan_checkpoints",
           "gdn_scan_checkpoint_bytes", "gdn_scan_workspace_bytes", "gdn_scan_backward_workspace_bytes",
           "gdn_cache_attention_prefix", "gdn_cache_attention_prefix_workspace_bytes"]
