"""Torch-facing calls of libychee: the hybrid-head sparse decode-attention step.

    out, idx_out = hybrid_decode_attn(q, k_cache, v_cache, seqlens, head_role, idx_in, k)
    out, idx_final, idx_layers = decode_stack(q, k_caches, v_caches, seqlens, head_roles, k)

Method: page "LycheeDecode: Accelerating Long-Context LLM Inference via
Hybrid-Head Sparse Decoding" (paper.rainbus.top/paper/2602.04541), steps (1),
(3), (4), (7).  Shapes and conventions are those of include/lychee.h; this module
only checks that tensors live on a CUDA device with the expected dtype and
layout, allocates outputs/workspace with torch when the caller does not pass
them, and hands raw pointers to the library on the current (or given) stream.

With stream=, what a call allocates belongs to that stream: a workspace is reused
behind the call's kernels only, and outputs are also kept until the stream that was
current at the call is done with them.  Tensors that the caller passes have to be
ready on the stream and kept until its kernels are done, as torch has it everywhere.
"""
from __future__ import annotations

import contextlib
import ctypes
from typing import NamedTuple

import torch

from . import _native as N

_DT = {torch.bfloat16: N.BF16, torch.float32: N.FP32}
_CODE = {torch.float8_e4m3fn: N.E4M3, torch.int8: N.INT8}


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream_handle(stream, device=None):
    """The raw handle of `stream` (default: the current stream of `device`); a
    given stream must belong to `device`."""
    s = stream if stream is not None else torch.cuda.current_stream(device)
    if device is not None and s.device != device:
        raise ValueError(f"stream is on {s.device}, but the call runs on {device}")
    return ctypes.c_void_p(s.cuda_stream)


def _on(stream):
    """The context in which a call on `stream` (None: the current one) allocates."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _empty_out(shape, dtype, device, stream):
    """An output of a call on `stream`, which the caller's stream may read after it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream(device))
    return t


def _need_cuda(name, t, dtype=None, shape=None, device=None):
    """t must be a contiguous CUDA tensor (of dtype / shape when given, and on
    `device` when given: the library launches on one device per call, the one
    of q, so every tensor of a call must live there)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device (there is no CPU path)")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, but the call runs on {device} (the device of q)")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def make_shape(B, Hq, Hkv, d, N_max, k, dtype, block=0) -> N.Shape:
    """block: 0 (token-level argsTopK) or the positions per selected block of a
    retrieval head's set (a multiple of 32, at most k)."""
    code = _DT.get(dtype, dtype)
    return N.Shape(int(B), int(Hq), int(Hkv), int(d), int(N_max), int(code), int(k), int(block))


def workspace_size(B, Hq, Hkv, d, N_max, k, dtype, block=0) -> int:
    """Bytes of workspace that serve both hybrid_decode_attn and decode_stack."""
    sh = make_shape(B, Hq, Hkv, d, N_max, k, dtype, block)
    n = N.load().lychee_workspace_size(ctypes.byref(sh))
    if n == 0:
        raise N.LycheeError(N.ERR_INVALID_ARG, "workspace_size")
    return int(n)


def layer_workspace_size(B, Hq, Hkv, d, N_max, k, dtype, block=0) -> int:
    """Bytes of workspace that hybrid_decode_attn alone needs."""
    sh = make_shape(B, Hq, Hkv, d, N_max, k, dtype, block)
    n = N.load().lychee_layer_workspace_size(ctypes.byref(sh))
    if n == 0:
        raise N.LycheeError(N.ERR_INVALID_ARG, "layer_workspace_size")
    return int(n)


def alloc_workspace(B, Hq, Hkv, d, N_max, k, dtype, device=None, block=0) -> torch.Tensor:
    n = workspace_size(B, Hq, Hkv, d, N_max, k, dtype, block)
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def _roles_host(role, n_expected):
    r = torch.as_tensor(role, dtype=torch.uint8).contiguous().cpu()
    if r.numel() != n_expected:
        raise ValueError(f"head_role must have {n_expected} entries")
    return r


def _check(st, what):
    if st != N.OK:
        raise N.LycheeError(st, what)


def _check_swa(swa, B, Hkv, d, dt, dev, gate_shape):
    """swa = (k_ring, v_ring, gate): rings [B,Hkv,window,d] of the caches' dtype,
    gate logits fp32 of gate_shape.  Returns the window length."""
    if len(swa) != 3:
        raise ValueError("swa must be (k_ring, v_ring, gate)")
    kr, vr, gate = swa
    _need_cuda("swa k_ring", kr, dt, device=dev)
    if kr.dim() != 4 or kr.shape[0] != B or kr.shape[1] != Hkv or kr.shape[3] != d:
        raise ValueError(f"swa k_ring must be [B, Hkv, window, d] = [{B}, {Hkv}, *, {d}]")
    _need_cuda("swa v_ring", vr, dt, tuple(kr.shape), device=dev)
    _need_cuda("swa gate", gate, torch.float32, gate_shape, device=dev)
    return int(kr.shape[2])


def hybrid_decode_attn(q, k_cache, v_cache, seqlens, head_role, idx_in, k, *, k_per_seq=None,
                       out=None, idx_out=None, workspace=None, stream=None, block=0, swa=None):
    """One hybrid-head layer.  q [B,Hq,d]; caches [B,Hkv,N_max,d] (bf16 or fp32);
    seqlens [B] int32 (device); head_role [Hq] (host, 1 = retrieval);
    idx_in [B,Hq,k] int32 (device, or None when every head is retrieval);
    block: 0 for argsTopK sets, else positions per selected block;
    swa: None, or (k_ring [B,Hkv,window,d], v_ring, gate [B,Hq] fp32) to fuse a
    sliding-window branch into every sparse head's output through a sigmoid gate.
    Returns (out [B,Hq,d], idx_out [B,Hq,k])."""
    B, Hq, d = q.shape
    _, Hkv, N_max, _ = k_cache.shape
    _need_cuda("q", q)
    dev = q.device
    dt = q.dtype
    _need_cuda("k_cache", k_cache, dt, (B, Hkv, N_max, d), device=dev)
    _need_cuda("v_cache", v_cache, dt, (B, Hkv, N_max, d), device=dev)
    _need_cuda("seqlens", seqlens, torch.int32, (B,), device=dev)
    if k_per_seq is not None:
        _need_cuda("k_per_seq", k_per_seq, torch.int32, (B,), device=dev)
    if idx_in is not None:
        _need_cuda("idx_in", idx_in, torch.int32, (B, Hq, k), device=dev)
    role = _roles_host(head_role, Hq)
    if out is None:
        out = _empty_out((B, Hq, d), dt, q.device, stream)
    _need_cuda("out", out, dt, (B, Hq, d), device=dev)
    if idx_out is None:
        idx_out = _empty_out((B, Hq, k), torch.int32, q.device, stream)
    _need_cuda("idx_out", idx_out, torch.int32, (B, Hq, k), device=dev)
    sh = make_shape(B, Hq, Hkv, d, N_max, k, dt, block)
    if workspace is None:
        with _on(stream):
            workspace = alloc_workspace(B, Hq, Hkv, d, N_max, k, dt, q.device, block)
    _need_cuda("workspace", workspace, torch.uint8, device=dev)
    if swa is not None:
        window = _check_swa(swa, B, Hkv, d, dt, dev, (B, Hq))
        with torch.cuda.device(dev):
            st = N.load().lychee_hybrid_decode_attn_swa(
                ctypes.byref(sh), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(seqlens),
                _ptr(k_per_seq), ctypes.c_void_p(role.data_ptr()), _ptr(idx_in), _ptr(swa[0]),
                _ptr(swa[1]), ctypes.c_int32(window), _ptr(swa[2]), _ptr(out), _ptr(idx_out),
                _ptr(workspace), ctypes.c_size_t(workspace.numel()), _stream_handle(stream, dev))
        _check(st, "lychee_hybrid_decode_attn_swa")
        return out, idx_out
    with torch.cuda.device(dev):
        st = N.load().lychee_hybrid_decode_attn(
            ctypes.byref(sh), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(seqlens), _ptr(k_per_seq),
            ctypes.c_void_p(role.data_ptr()), _ptr(idx_in), _ptr(out), _ptr(idx_out),
            _ptr(workspace), ctypes.c_size_t(workspace.numel()), _stream_handle(stream, dev))
    _check(st, "lychee_hybrid_decode_attn")
    return out, idx_out


def hybrid_decode_attn_noalloc(q, k_cache, v_cache, seqlens, head_role, idx_in, k, *,
                               k_per_seq=None, out=None, idx_out=None, device_error=None,
                               stream=None, block=0):
    """hybrid_decode_attn served from the library's static device scratch: no
    workspace argument and no device allocation by the library (out / idx_out
    are allocated here only when not given).  device_error: optional device
    int32 tensor [1] that receives the call's device error bits.  Calls on one device
    share the scratch, so they must not overlap; the first call on a device must
    precede any stream capture."""
    B, Hq, d = q.shape
    _, Hkv, N_max, _ = k_cache.shape
    _need_cuda("q", q)
    dev = q.device
    dt = q.dtype
    _need_cuda("k_cache", k_cache, dt, (B, Hkv, N_max, d), device=dev)
    _need_cuda("v_cache", v_cache, dt, (B, Hkv, N_max, d), device=dev)
    _need_cuda("seqlens", seqlens, torch.int32, (B,), device=dev)
    if k_per_seq is not None:
        _need_cuda("k_per_seq", k_per_seq, torch.int32, (B,), device=dev)
    if idx_in is not None:
        _need_cuda("idx_in", idx_in, torch.int32, (B, Hq, k), device=dev)
    need = layer_workspace_size(B, Hq, Hkv, d, N_max, k, dt, block)
    if need > N.NOALLOC_SCRATCH_BYTES:
        raise ValueError(f"this layer needs {need} bytes of scratch; the static scratch holds "
                         f"{N.NOALLOC_SCRATCH_BYTES} (use hybrid_decode_attn with a workspace)")
    role = _roles_host(head_role, Hq)
    if out is None:
        out = _empty_out((B, Hq, d), dt, q.device, stream)
    _need_cuda("out", out, dt, (B, Hq, d), device=dev)
    if idx_out is None:
        idx_out = _empty_out((B, Hq, k), torch.int32, q.device, stream)
    _need_cuda("idx_out", idx_out, torch.int32, (B, Hq, k), device=dev)
    if device_error is not None:
        _need_cuda("device_error", device_error, torch.int32, (1,), device=dev)
    sh = make_shape(B, Hq, Hkv, d, N_max, k, dt, block)
    with torch.cuda.device(dev):
        st = N.load().lychee_hybrid_decode_attn_noalloc(
            ctypes.byref(sh), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(seqlens), _ptr(k_per_seq),
            ctypes.c_void_p(role.data_ptr()), _ptr(idx_in), _ptr(out), _ptr(idx_out),
            _ptr(device_error), _stream_handle(stream, dev))
    _check(st, "lychee_hybrid_decode_attn_noalloc")
    return out, idx_out


def decode_stack(q, k_caches, v_caches, seqlens, head_roles, k, *, k_per_seq=None, out=None,
                 idx_final=None, idx_layers=None, want_layers=False, workspace=None, stream=None,
                 block=0, swa=None):
    """L chained layers of one decode step.  q [L,B,Hq,d]; k_caches / v_caches:
    sequences of L tensors [B,Hkv,N_max,d]; head_roles [L,Hq] (host, row 0 all
    retrieval); block as in hybrid_decode_attn; swa: None, or (k_rings, v_rings,
    gate): L window rings [B,Hkv,window,d] each and gate logits [L,B,Hq] fp32.
    Returns (out [L,B,Hq,d], idx_final [B,Hq,k], idx_layers or None)."""
    L, B, Hq, d = q.shape
    if len(k_caches) != L or len(v_caches) != L:
        raise ValueError("need one K and one V cache per layer")
    _need_cuda("q", q)
    dev = q.device
    dt = q.dtype
    _, Hkv, N_max, _ = k_caches[0].shape
    for l in range(L):
        _need_cuda(f"k_caches[{l}]", k_caches[l], dt, (B, Hkv, N_max, d), device=dev)
        _need_cuda(f"v_caches[{l}]", v_caches[l], dt, (B, Hkv, N_max, d), device=dev)
    _need_cuda("seqlens", seqlens, torch.int32, (B,), device=dev)
    if k_per_seq is not None:
        _need_cuda("k_per_seq", k_per_seq, torch.int32, (B,), device=dev)
    roles = _roles_host(head_roles, L * Hq)
    if out is None:
        out = _empty_out((L, B, Hq, d), dt, q.device, stream)
    _need_cuda("out", out, dt, (L, B, Hq, d), device=dev)
    if idx_final is None:
        idx_final = _empty_out((B, Hq, k), torch.int32, q.device, stream)
    _need_cuda("idx_final", idx_final, torch.int32, (B, Hq, k), device=dev)
    if idx_layers is None and want_layers:
        idx_layers = _empty_out((L, B, Hq, k), torch.int32, q.device, stream)
    if idx_layers is not None:
        _need_cuda("idx_layers", idx_layers, torch.int32, (L, B, Hq, k), device=dev)
    sh = make_shape(B, Hq, Hkv, d, N_max, k, dt, block)
    if workspace is None:
        with _on(stream):
            workspace = alloc_workspace(B, Hq, Hkv, d, N_max, k, dt, q.device, block)
    _need_cuda("workspace", workspace, torch.uint8, device=dev)
    kp = (ctypes.c_void_p * L)(*[t.data_ptr() for t in k_caches])
    vp = (ctypes.c_void_p * L)(*[t.data_ptr() for t in v_caches])
    if swa is not None:
        kr, vr, gate = swa
        if len(kr) != L or len(vr) != L:
            raise ValueError("swa needs one window ring of K and one of V per layer")
        window = None
        for l in range(L):
            w = _check_swa((kr[l], vr[l], gate[l]), B, Hkv, d, dt, dev, (B, Hq))
            if window not in (None, w):
                raise ValueError("every layer's window ring must have the same length")
            window = w
        _need_cuda("swa gate", gate, torch.float32, (L, B, Hq), device=dev)
        krp = (ctypes.c_void_p * L)(*[t.data_ptr() for t in kr])
        vrp = (ctypes.c_void_p * L)(*[t.data_ptr() for t in vr])
        with torch.cuda.device(dev):
            st = N.load().lychee_decode_stack_swa(
                ctypes.byref(sh), ctypes.c_int32(L), _ptr(q), ctypes.cast(kp, ctypes.c_void_p),
                ctypes.cast(vp, ctypes.c_void_p), _ptr(seqlens), _ptr(k_per_seq),
                ctypes.c_void_p(roles.data_ptr()), ctypes.cast(krp, ctypes.c_void_p),
                ctypes.cast(vrp, ctypes.c_void_p), ctypes.c_int32(window), _ptr(gate), _ptr(out),
                _ptr(idx_final), _ptr(idx_layers), _ptr(workspace),
                ctypes.c_size_t(workspace.numel()), _stream_handle(stream, dev))
        _check(st, "lychee_decode_stack_swa")
        return out, idx_final, idx_layers
    with torch.cuda.device(dev):
        st = N.load().lychee_decode_stack(
            ctypes.byref(sh), ctypes.c_int32(L), _ptr(q), ctypes.cast(kp, ctypes.c_void_p),
            ctypes.cast(vp, ctypes.c_void_p), _ptr(seqlens), _ptr(k_per_seq),
            ctypes.c_void_p(roles.data_ptr()), _ptr(out), _ptr(idx_final), _ptr(idx_layers),
            _ptr(workspace), ctypes.c_size_t(workspace.numel()), _stream_handle(stream, dev))
    _check(st, "lychee_decode_stack")
    return out, idx_final, idx_layers


def append_kv(k_new, v_new, k_cache, v_cache, seqlens, stream=None):
    """The current token's K/V rows [B,Hkv,d] into the caches [B,Hkv,N_max,d] at
    row seqlens[b] - 1 (in place).  Returns (k_cache, v_cache)."""
    B, Hkv, N_max, d = k_cache.shape
    dt = k_cache.dtype
    dev = k_cache.device
    _need_cuda("k_cache", k_cache, dt, (B, Hkv, N_max, d), device=dev)
    _need_cuda("v_cache", v_cache, dt, (B, Hkv, N_max, d), device=dev)
    _need_cuda("k_new", k_new, dt, (B, Hkv, d), device=dev)
    _need_cuda("v_new", v_new, dt, (B, Hkv, d), device=dev)
    _need_cuda("seqlens", seqlens, torch.int32, (B,), device=dev)
    sh = make_shape(B, Hkv, Hkv, d, N_max, 1, dt)
    with torch.cuda.device(dev):
        st = N.load().lychee_append_kv(ctypes.byref(sh), _ptr(k_new), _ptr(v_new), _ptr(k_cache),
                                       _ptr(v_cache), _ptr(seqlens), _stream_handle(stream, dev))
    _check(st, "lychee_append_kv")
    return k_cache, v_cache


class Q8Cache(NamedTuple):
    """One layer's 8-bit paged cache.  k, v: codes [num_pages, Hkv, page, d] (torch.float8_e4m3fn
    or torch.int8); k_scale, v_scale [num_pages, Hkv] fp32: a page's rows of one head hold
    code * scale."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor


def alloc_q8_cache(num_pages, Hkv, page, d, code=torch.float8_e4m3fn, device=None) -> Q8Cache:
    """An uninitialised cache (a page is written before it is read)."""
    if code not in _CODE:
        raise TypeError(f"code must be torch.float8_e4m3fn or torch.int8, got {code}")
    dev = device or "cuda"
    k, v = (torch.empty((num_pages, Hkv, page, d), dtype=code, device=dev) for _ in range(2))
    ks, vs = (torch.ones((num_pages, Hkv), dtype=torch.float32, device=dev) for _ in range(2))
    return Q8Cache(k, v, ks, vs)


def make_q8_shape(B, Hq, Hkv, d, page, num_pages, max_pages, dtype, code) -> N.Q8Shape:
    return N.Q8Shape(int(B), int(Hq), int(Hkv), int(d), int(page), int(num_pages), int(max_pages),
                     int(_DT.get(dtype, dtype)), int(_CODE.get(code, code)))


def q8_workspace_size(B, Hq, Hkv, d, page, num_pages, max_pages, dtype, code, k=0) -> int:
    """Bytes of workspace of decode_attn_q8 (k = 0) or of hybrid_decode_attn_q8 with sets of
    capacity k."""
    sh = make_q8_shape(B, Hq, Hkv, d, page, num_pages, max_pages, dtype, code)
    n = N.load().lychee_q8_workspace_size(ctypes.byref(sh), int(k))
    if n == 0:
        raise N.LycheeError(N.ERR_INVALID_ARG, "q8_workspace_size")
    return int(n)


def alloc_q8_workspace(B, Hq, Hkv, d, page, num_pages, max_pages, dtype, code, k=0,
                       device=None) -> torch.Tensor:
    """A workspace of that size, its error word (check_device_error) zero."""
    n = q8_workspace_size(B, Hq, Hkv, d, page, num_pages, max_pages, dtype, code, k)
    ws = torch.empty(n, dtype=torch.uint8, device=device or "cuda")
    ws[:4].zero_()
    return ws


# The calls below run once a layer and token, so what they do on the host counts: a
# tensor that is as it must be passes one short test, and only another one goes
# through the checks that name what is wrong.

def _need(name, t, dtype, shape, dev, index):
    """_need_cuda, quick where there is nothing to report."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and
            t.get_device() == index and t.is_contiguous()):
        _need_cuda(name, t, dtype, shape, device=dev)


def _device_index(name, t):
    """The index of a CUDA tensor's device."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device (there is no CPU path)")
    return t.get_device()


# The current stream of a device as a raw handle (without the Stream object where torch has a call for it).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _q8_launch(what, fn, dev, index, stream, args):
    """Call the library on device `index` with the raw stream as the last argument."""
    if stream is not None and stream.device != dev:
        raise ValueError(f"stream is on {stream.device}, but the call runs on {dev}")
    raw = _raw_stream(index) if stream is None else stream.cuda_stream
    if torch.cuda.current_device() == index:
        st = fn(*args, raw)
    else:
        with torch.cuda.device(index):
            st = fn(*args, raw)
    if st != N.OK:
        raise N.LycheeError(st, what)


def _q8_cache(cache, block_table, seqlens, Hq, d, dt, dev, index):
    """The checked cache of a call: its shape and pointers for the library."""
    if not isinstance(cache, Q8Cache):
        raise TypeError("cache must be a Q8Cache")
    k, v, ks, vs = cache
    if not isinstance(k, torch.Tensor):
        raise TypeError("cache.k must be a torch.Tensor")
    code = _CODE.get(k.dtype)
    if code is None:
        raise TypeError(f"cache.k must be torch.float8_e4m3fn or torch.int8, got {k.dtype}")
    shape = k.shape
    if len(shape) != 4 or shape[3] != d:
        raise ValueError(f"cache.k must be [num_pages, Hkv, page, {d}], got {tuple(shape)}")
    P, Hkv, page, _ = shape
    if not isinstance(block_table, torch.Tensor) or block_table.dim() != 2:
        raise ValueError("block_table must be a tensor [B, max_pages]")
    B, max_pages = block_table.shape
    try:
        fine = (k.get_device() == index and v.get_device() == index and ks.get_device() == index and
                vs.get_device() == index and block_table.get_device() == index and
                seqlens.get_device() == index and v.dtype is k.dtype and ks.dtype is torch.float32 and
                vs.dtype is torch.float32 and block_table.dtype is torch.int32 and
                seqlens.dtype is torch.int32 and v.shape == shape and ks.shape == (P, Hkv) and
                vs.shape == (P, Hkv) and seqlens.shape == (B,) and k.is_contiguous() and
                v.is_contiguous() and ks.is_contiguous() and vs.is_contiguous() and
                block_table.is_contiguous() and seqlens.is_contiguous())
    except AttributeError:
        fine = False
    if not fine:
        _need_cuda("cache.k", k, device=dev)
        _need_cuda("cache.v", v, k.dtype, shape, device=dev)
        _need_cuda("cache.k_scale", ks, torch.float32, (P, Hkv), device=dev)
        _need_cuda("cache.v_scale", vs, torch.float32, (P, Hkv), device=dev)
        _need_cuda("block_table", block_table, torch.int32, device=dev)
        _need_cuda("seqlens", seqlens, torch.int32, (B,), device=dev)
    return (N.Q8Shape(B, Hq, Hkv, d, page, P, max_pages, _DT[dt], code),
            N.Q8CachePtrs(k.data_ptr(), v.data_ptr(), ks.data_ptr(), vs.data_ptr(),
                          block_table.data_ptr()), B, Hkv)


def _need_rows(name, t, dt, shape, dev, index):
    """Rows [T, heads, d] of dtype dt whose tokens may lie further apart than a row's end (a part
    of a projection's output).  Returns the elements from one token to the next."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.get_device() != index:
        _need_cuda(name, t, device=dev)
    if t.dtype is not dt:
        raise TypeError(f"{name} must be {dt}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    T, heads, d = shape
    s0, s1, s2 = t.stride()
    if T <= 1:
        s0 = heads * d
    if s2 != 1 or (heads > 1 and s1 != d) or s0 < heads * d:
        raise ValueError(f"{name}: the rows of one token must be contiguous")
    if s0 * (2 if dt is torch.bfloat16 else 4) % 16 != 0 or t.data_ptr() % 16 != 0:
        raise ValueError(f"{name}: tokens must begin on 16-byte boundaries")
    return s0


def append_rope_q8(k_new, v_new, cache, block_table, seqlens, cos_sin=None, *, q=None, cu_new=None,
                   interleaved=False, q_out=None, device_error=None, stream=None):
    """New keys and values [T, Hkv, d] (bf16 or fp32) into the 8-bit paged cache, in place, rotated
    by their positions on the way; the queries q [T, Hq, d] (or None) rotated beside them.

    cu_new [B + 1] int32: sequence b's tokens are cu_new[b] .. cu_new[b + 1] - 1 (None: token b).
    seqlens [B] int32 counts the new tokens.  cos_sin [n_pos, rot] fp32: cosines, then sines, of
    every position's rot / 2 angles (None: no rotation); interleaved: pairs (2i, 2i + 1) instead of
    (i, i + rot / 2).  Rows of k_new, v_new and q may be parts of one projection output.
    device_error [1] int32: error bits are OR-ed into it (1 bad page, 2 bad length, 16 a value that is
    not finite; None: nothing tells of them, but the rotated queries of a sequence whose numbers do
    not fit are NaN).  q_out may be q itself (contiguous).  Returns the rotated queries
    [T, Hq, d], or None without q."""
    if not isinstance(k_new, torch.Tensor) or k_new.dim() != 3:
        raise ValueError("k_new must be a tensor [T, Hkv, d]")
    shape, dt, dev = k_new.shape, k_new.dtype, k_new.device
    T, Hkv, d = shape
    if dt not in _DT:
        raise TypeError(f"k_new must be torch.bfloat16 or torch.float32, got {dt}")
    index = _device_index("k_new", k_new)
    k_stride = _need_rows("k_new", k_new, dt, shape, dev, index)
    v_stride = _need_rows("v_new", v_new, dt, shape, dev, index)
    Hq, q_stride, q_ptr, q_out_ptr = Hkv, 0, None, None
    if q is not None:
        if not isinstance(q, torch.Tensor) or q.dim() != 3:
            raise ValueError("q must be a tensor [T, Hq, d]")
        Hq = q.shape[1]
        q_stride = _need_rows("q", q, dt, (T, Hq, d), dev, index)
        if q_out is None:
            q_out = _empty_out((T, Hq, d), dt, dev, stream)
        else:
            _need("q_out", q_out, dt, (T, Hq, d), dev, index)
        q_ptr, q_out_ptr = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out without q")
    sh, ptrs, B, cache_heads = _q8_cache(cache, block_table, seqlens, Hq, d, dt, dev, index)
    if cache_heads != Hkv:
        raise ValueError(f"k_new has {Hkv} heads, the cache {cache_heads}")
    cu_ptr = cs_ptr = err = None
    if cu_new is not None:
        _need("cu_new", cu_new, torch.int32, (B + 1,), dev, index)
        cu_ptr = cu_new.data_ptr()
    elif T != B:
        raise ValueError(f"without cu_new there is one token a sequence: got {T} for {B}")
    n_pos = rot = 0
    if cos_sin is not None:
        if not isinstance(cos_sin, torch.Tensor) or cos_sin.dim() != 2:
            raise ValueError("cos_sin must be a tensor [n_pos, rot]")
        n_pos, rot = cos_sin.shape
        _need("cos_sin", cos_sin, torch.float32, (n_pos, rot), dev, index)
        cs_ptr = cos_sin.data_ptr()
    if device_error is not None:
        _need("device_error", device_error, torch.int32, (1,), dev, index)
        err = device_error.data_ptr()
    if T > 0:
        tok = N.Q8Tokens(k_new.data_ptr(), v_new.data_ptr(), q_ptr, q_out_ptr, k_stride, v_stride,
                         q_stride, cs_ptr, cu_ptr, T, n_pos, rot, 1 if interleaved else 0)
        _q8_launch("lychee_append_rope_q8", N.load().lychee_append_rope_q8, dev, index, stream,
                   (sh, ptrs, tok, seqlens.data_ptr(), err))
    return q_out


def _q8_call(q, cache, block_table, seqlens, out, workspace, device_error, k, stream):
    """What both attention calls check and make: (shape, pointers, B, Hq, device, its index, out,
    workspace, device_error's pointer)."""
    index = _device_index("q", q)
    if q.dim() != 3:
        raise ValueError("q must be [B, Hq, d]")
    shape, dt, dev = q.shape, q.dtype, q.device
    if dt not in _DT:
        raise TypeError(f"q must be torch.bfloat16 or torch.float32, got {dt}")
    _need("q", q, dt, shape, dev, index)
    if out is None:
        out = torch.empty_like(q) if stream is None else _empty_out(shape, dt, dev, stream)
    else:
        _need("out", out, dt, shape, dev, index)
    sh, ptrs, B, _ = _q8_cache(cache, block_table, seqlens, shape[1], shape[2], dt, dev, index)
    if B != shape[0]:
        raise ValueError(f"q has {shape[0]} sequences, block_table {B}")
    if workspace is None:
        n = N.load().lychee_q8_workspace_size(sh, k)
        with _on(stream):
            workspace = torch.empty(max(n, 256), dtype=torch.uint8, device=dev)
    elif not (isinstance(workspace, torch.Tensor) and workspace.dtype is torch.uint8 and
              workspace.get_device() == index and workspace.is_contiguous()):
        _need_cuda("workspace", workspace, torch.uint8, device=dev)
    err = None
    if device_error is not None:
        _need("device_error", device_error, torch.int32, (1,), dev, index)
        err = device_error.data_ptr()
    return sh, ptrs, B, shape[1], dev, index, out, workspace, err


def decode_attn_q8(q, cache, block_table, seqlens, *, out=None, workspace=None, device_error=None,
                   stream=None):
    """Attention of one query token a sequence over every position of the 8-bit paged cache.
    q [B, Hq, d] (bf16 or fp32), block_table [B, max_pages] int32, seqlens [B] int32.
    workspace: uint8, q8_workspace_size(...) bytes (calls that share one must be ordered on one
    stream; None: a fresh one).  device_error as in append_rope_q8; without it the bits go to the
    workspace (check_device_error reads and clears them; one of alloc_q8_workspace begins with none).
    out must not overlap q.  Returns out [B, Hq, d]."""
    sh, ptrs, _, _, dev, index, out, workspace, err = _q8_call(q, cache, block_table, seqlens, out,
                                                               workspace, device_error, 0, stream)
    _q8_launch("lychee_decode_attn_q8", N.load().lychee_decode_attn_q8, dev, index, stream,
               (sh, q.data_ptr(), ptrs, seqlens.data_ptr(), out.data_ptr(), workspace.data_ptr(),
                workspace.numel(), err))
    return out


def hybrid_decode_attn_q8(q, cache, block_table, seqlens, head_role, idx_in, k, *, k_per_seq=None,
                          out=None, idx_out=None, workspace=None, device_error=None, stream=None,
                          block=0):
    """hybrid_decode_attn over the 8-bit paged cache: one hybrid-head layer.  q, head_role, idx_in,
    k, k_per_seq and block as there; cache, block_table, seqlens, workspace (q8_workspace_size(...,
    k) bytes), device_error and out as in decode_attn_q8; idx_out may be idx_in.
    Returns (out [B, Hq, d], idx_out [B, Hq, k])."""
    k = int(k)
    sh, ptrs, B, Hq, dev, index, out, workspace, err = _q8_call(q, cache, block_table, seqlens, out,
                                                                workspace, device_error, max(k, 0),
                                                                stream)
    kps = idx = None
    if k_per_seq is not None:
        _need("k_per_seq", k_per_seq, torch.int32, (B,), dev, index)
        kps = k_per_seq.data_ptr()
    if idx_in is not None:
        _need("idx_in", idx_in, torch.int32, (B, Hq, k), dev, index)
        idx = idx_in.data_ptr()
    role = head_role
    if not (isinstance(role, torch.Tensor) and role.dtype is torch.uint8 and role.shape == (Hq,) and
            not role.is_cuda and role.is_contiguous()):
        role = _roles_host(head_role, Hq)
    if idx_out is None:
        idx_out = _empty_out((B, Hq, max(k, 0)), torch.int32, dev, stream)
    else:
        _need("idx_out", idx_out, torch.int32, (B, Hq, k), dev, index)
    _q8_launch("lychee_hybrid_decode_attn_q8", N.load().lychee_hybrid_decode_attn_q8, dev, index,
               stream, (sh, k, int(block), q.data_ptr(), ptrs, seqlens.data_ptr(), kps,
                        role.data_ptr(), idx, out.data_ptr(), idx_out.data_ptr(),
                        workspace.data_ptr(), workspace.numel(), err))
    return out, idx_out


def hardkuma_roles(alpha, beta, p=-0.1, q=1.1, layer0_retrieval=True, stream=None):
    """Head roles from HardKuma gate parameters: alpha, beta [L, Hq] float64 on
    one CUDA device.  Returns (roles [L, Hq] uint8 on that device, 1 = retrieval
    when E[z] > 0.5 or in layer 0; E[z] [L, Hq] float64; the expected L0 norm of
    the gated heads, a float64 tensor [1])."""
    _need_cuda("alpha", alpha, torch.float64)
    dev = alpha.device
    if alpha.dim() != 2:
        raise ValueError("alpha must be [L, Hq]")
    L, Hq = alpha.shape
    _need_cuda("beta", beta, torch.float64, (L, Hq), device=dev)
    roles = _empty_out((L, Hq), torch.uint8, dev, stream)
    ez = _empty_out((L, Hq), torch.float64, dev, stream)
    l0 = _empty_out((1,), torch.float64, dev, stream)
    with torch.cuda.device(dev):
        st = N.load().lychee_hardkuma_roles(_ptr(alpha), _ptr(beta), int(L), int(Hq), float(p),
                                            float(q), int(bool(layer0_retrieval)), _ptr(roles),
                                            _ptr(ez), _ptr(l0), _stream_handle(stream, dev))
    _check(st, "lychee_hardkuma_roles")
    return roles, ez, l0


def check_device_error(workspace, stream=None):
    """Synchronise, read and clear the device error word.  Returns (status, bits)."""
    _need_cuda("workspace", workspace, torch.uint8)
    dev = workspace.device
    bits = ctypes.c_uint32(0)
    with torch.cuda.device(dev):
        st = N.load().lychee_check_device_error(_ptr(workspace), _stream_handle(stream, dev),
                                                ctypes.byref(bits))
    return int(st), int(bits.value)


def workspace_views(workspace, B, Hq, Hkv, d, N_max, k, dtype):
    """Views into the documented workspace regions (for inspection in tests):
    logits [B,Hq,N_max] fp32 (raw q.k of the most recent layer's retrieval
    heads) and bitmaps [B,Hq,ceil(N_max/32)] int32 (bit patterns of the sets)."""
    sh = make_shape(B, Hq, Hkv, d, N_max, k, dtype)
    lo, bo, nw = ctypes.c_size_t(0), ctypes.c_size_t(0), ctypes.c_int32(0)
    _check(N.load().lychee_workspace_offsets(ctypes.byref(sh), ctypes.byref(lo), ctypes.byref(bo),
                                             ctypes.byref(nw)), "lychee_workspace_offsets")
    lo, bo, nw = lo.value, bo.value, nw.value
    logits = workspace[lo: lo + B * Hq * N_max * 4].view(torch.float32).view(B, Hq, N_max)
    bitmaps = workspace[bo: bo + B * Hq * nw * 4].view(torch.int32).view(B, Hq, nw)
    return logits, bitmaps


class Profile:
    """Context manager around lychee_profile_begin / lychee_profile_end.
    After exit, ``records`` is a list of (kind, ms) per library launch.  With
    spans=True (lychee_profile_spans_begin) there is one ("attn_span", ms)
    record per stack call instead, and no event between its launches."""
    KINDS = {0: "attn", 1: "topk", 2: "combine", 3: "build_bits", 4: "export",
             5: "topk+combine", 6: "attn_span", 7: "append"}

    def __init__(self, max_launches=4096, spans=False):
        self.max_launches = int(max_launches)
        self.spans = bool(spans)
        self.records = []

    def __enter__(self):
        if self.spans:
            _check(N.load().lychee_profile_spans_begin(self.max_launches),
                   "lychee_profile_spans_begin")
        else:
            _check(N.load().lychee_profile_begin(self.max_launches), "lychee_profile_begin")
        return self

    def __exit__(self, *exc):
        cap = self.max_launches
        kinds = (ctypes.c_int32 * cap)()
        ms = (ctypes.c_float * cap)()
        n = ctypes.c_int32(0)
        _check(N.load().lychee_profile_end(cap, ctypes.cast(kinds, ctypes.c_void_p),
                                           ctypes.cast(ms, ctypes.c_void_p), ctypes.byref(n)),
               "lychee_profile_end")
        self.records = [(self.KINDS.get(kinds[i], str(kinds[i])), float(ms[i]))
                        for i in range(min(n.value, cap))]
        return False
