"""Torch-tensor front end of the C ABI: builds the ``ttt_desc``, allocates outputs and the
workspace with torch, and calls the library. No arithmetic of the layer happens here.

Shapes (see include/ttt.h): q, k, v [B,H,N,h] (bf16 or fp32, contiguous, on the GPU);
eta [B,H,N] fp32; W0, W2 [H,h,m] fp32 ([H,m,h] with w_in_layout=1); W1 [H,m,h] fp32
([H,h,m] with w1_layout=1).

The token-mixer operators (short_conv_*, head_norm_rope_*, selective_scan_*) take token-major
inputs [B,N,...] that may be slices of a wider projection (one stride between all tokens);
they run on the device of their first tensor, on its current stream unless ``stream`` is given.
A caller who gives one orders it behind the streams that made the inputs, and keeps the inputs
until it is done; the outputs belong to it.
"""
from __future__ import annotations

import functools

import torch

from . import abi

ORDERS = {"update_apply": abi.TTT_ORDER_UPDATE_APPLY, "apply_update": abi.TTT_ORDER_APPLY_UPDATE}


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return abi.TTT_DTYPE_BF16
    if t.dtype == torch.float32:
        return abi.TTT_DTYPE_FP32
    raise TypeError(f"q/k/v must be bfloat16 or float32, got {t.dtype}")


def _need(t, name, dtype=None):
    if t is None:
        return
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")


def workspace(nbytes: int, device) -> torch.Tensor:
    """A device byte buffer of at least ``nbytes`` (torch allocations are 512-byte aligned)."""
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def parallel_desc(q, W1, chunk, order="update_apply", sign=1, w_in_layout=0, w1_layout=0):
    B, H, N, h = q.shape
    m = W1.shape[1] if w1_layout == 0 else W1.shape[2]
    return abi.ttt_desc(B=B, H=H, N=N, h=h, m=m, chunk=chunk, dtype=_dtype_code(q),
                        order=ORDERS[order], sign=sign, w_in_layout=w_in_layout,
                        w1_layout=w1_layout)


def la_parallel_fwd(q, k, v, eta, W0, W2, W1, chunk, *, order="update_apply", sign=1,
                    w_in_layout=0, w1_layout=0, return_state=True, out=None, ws=None,
                    stream=None):
    """Parallel last-layer-only form. Returns (out [B,H,N,h], final state or None)."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n, q.dtype)
    _need(eta, "eta", torch.float32)
    for t, n in ((W0, "W0"), (W2, "W2"), (W1, "W1")):
        _need(t, n, torch.float32)
    desc = parallel_desc(q, W1, chunk, order, sign, w_in_layout, w1_layout)
    B, H, N, h = q.shape
    m = desc.m
    if out is None:
        out = torch.empty_like(q)
    S = None
    if return_state:
        shape = (B, H, m, h) if w1_layout == 0 else (B, H, h, m)
        S = torch.empty(shape, dtype=torch.float32, device=q.device)
    if ws is None:
        ws = workspace(abi.ttt_workspace_bytes(desc, abi.TTT_PATH_PARALLEL), q.device)
    abi.ttt_la_parallel_fwd(desc, q, k, v, eta, W0, W2, W1, out, S, ws, stream=stream)
    return out, S


def la_parallel_fwd_shard(q, k, v, eta, W0, W2, W1, chunk, *, prior=None, state_only=False,
                          order="update_apply", sign=1, w_in_layout=0, w1_layout=0, m=None,
                          out=None, ws=None, stream=None):
    """One contiguous shard of a sequence (context parallelism): the parallel form from the
    initial state W1 (zeros when None) plus the sum of ``prior`` [n, B, H, m, h] (W1's
    layout per entry) along its first axis. ``state_only`` skips the outputs. Returns
    (out or None, final state). ``m`` is needed when W1 is None."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n, q.dtype)
    _need(eta, "eta", torch.float32)
    for t, n in ((W0, "W0"), (W2, "W2"), (W1, "W1"), (prior, "prior")):
        _need(t, n, torch.float32)
    B, H, N, h = q.shape
    if m is None:
        m = W1.shape[1] if w1_layout == 0 else W1.shape[2]
    desc = abi.ttt_desc(B=B, H=H, N=N, h=h, m=m, chunk=chunk, dtype=_dtype_code(q),
                        order=ORDERS[order], sign=sign, w_in_layout=w_in_layout,
                        w1_layout=w1_layout)
    if out is None and not state_only:
        out = torch.empty_like(q)
    S = torch.empty((B, H, m, h) if w1_layout == 0 else (B, H, h, m), dtype=torch.float32,
                    device=q.device)
    if ws is None:
        ws = workspace(abi.ttt_workspace_bytes(desc, abi.TTT_PATH_PARALLEL), q.device)
    n_prior = 0 if prior is None else prior.shape[0]
    abi.ttt_la_parallel_fwd_shard(desc, q, k, v, eta, W0, W2, W1, prior if n_prior else None,
                                  n_prior, None if state_only else out, S, ws, stream=stream)
    return (None if state_only else out), S


def la_parallel_fwd_shard_outputs(q, W1, chunk, ws, *, prior=None, order="update_apply",
                                  sign=1, w_in_layout=0, w1_layout=0, m=None, out=None,
                                  stream=None):
    """The outputs pass of a shard after its state-only pass ``la_parallel_fwd_shard(...,
    state_only=True, ws=ws)`` on this thread: reuses that call's chunk deltas (left in
    ``ws``) and forms the states from W1 (zeros when None) plus the sum of ``prior``, then
    the outputs. Returns (out, final state). ``m`` is needed when W1 is None."""
    _need(q, "q", q.dtype)
    for t, n in ((W1, "W1"), (prior, "prior")):
        _need(t, n, torch.float32)
    B, H, N, h = q.shape
    if m is None:
        m = W1.shape[1] if w1_layout == 0 else W1.shape[2]
    desc = abi.ttt_desc(B=B, H=H, N=N, h=h, m=m, chunk=chunk, dtype=_dtype_code(q),
                        order=ORDERS[order], sign=sign, w_in_layout=w_in_layout,
                        w1_layout=w1_layout)
    if out is None:
        out = torch.empty_like(q)
    S = torch.empty((B, H, m, h) if w1_layout == 0 else (B, H, h, m), dtype=torch.float32,
                    device=q.device)
    n_prior = 0 if prior is None else prior.shape[0]
    abi.ttt_la_parallel_fwd_shard_outputs(desc, q, W1, prior if n_prior else None, n_prior,
                                          out, S, ws, stream=stream)
    return out, S


def la_parallel_momentum_fwd(q, k, v, eta, W0, W2, W1, chunk, *, order="update_apply", sign=1,
                             alpha=None, ns_steps=0, w_in_layout=0, return_state=True,
                             out=None, ws=None, stream=None):
    """Parallel form with W1 momentum (when ``alpha`` [B,H,C] is given) and Newton-Schulz.
    Returns (out [B,H,N,h], final state [B,H,m,h] or None)."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n, q.dtype)
    _need(eta, "eta", torch.float32)
    _need(alpha, "alpha", torch.float32)
    desc = parallel_desc(q, W1, chunk, order, sign, w_in_layout, 0)
    desc.momentum = int(alpha is not None)
    desc.ns_steps = ns_steps
    B, H, N, h = q.shape
    if out is None:
        out = torch.empty_like(q)
    S = torch.empty((B, H, desc.m, h), dtype=torch.float32, device=q.device) if return_state else None
    if ws is None:
        ws = workspace(abi.ttt_workspace_bytes(desc, abi.TTT_PATH_PARALLEL_MOMENTUM), q.device)
    abi.ttt_la_parallel_momentum_fwd(desc, q, k, v, eta, alpha, W0, W2, W1, out, S, ws,
                                     stream=stream)
    return out, S


def la_parallel_bwd(q, k, v, eta, W0, W2, W1, dout, chunk, *, order="update_apply", sign=1,
                    dS_final=None, ws=None, stream=None):
    """Backward of la_parallel_fwd. Returns dq, dk, dv (q's dtype), deta, dW0, dW2, dW1
    (fp32; weight gradients per head, summed over the batch)."""
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (dout, "dout")):
        _need(t, n, q.dtype)
    _need(eta, "eta", torch.float32)
    _need(dS_final, "dS_final", torch.float32)
    desc = parallel_desc(q, W1, chunk, order, sign)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    deta = torch.empty_like(eta)
    dW0, dW2, dW1 = torch.empty_like(W0), torch.empty_like(W2), torch.empty_like(W1)
    if ws is None:
        ws = workspace(abi.ttt_workspace_bytes(desc, abi.TTT_PATH_PARALLEL_BWD), q.device)
    abi.ttt_la_parallel_bwd(desc, q, k, v, eta, W0, W2, W1, dout, dS_final, dq, dk, dv, deta,
                            dW0, dW2, dW1, ws, stream=stream)
    return dq, dk, dv, deta, dW0, dW2, dW1


def linear_attn_fwd(q, k, v, eta, S0, chunk, *, order="update_apply", sign=1, s_layout=0,
                    return_state=True, out=None, ws=None, stream=None):
    """Parallel form with identity features (plain chunked linear attention with per-token
    eta). S0 [H,h,h] fp32. Returns (out [B,H,N,h], final state [B,H,h,h] or None)."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n, q.dtype)
    _need(eta, "eta", torch.float32)
    _need(S0, "S0", torch.float32)
    B, H, N, h = q.shape
    desc = abi.ttt_desc(B=B, H=H, N=N, h=h, m=h, chunk=chunk, dtype=_dtype_code(q),
                        order=ORDERS[order], sign=sign, w1_layout=s_layout)
    if out is None:
        out = torch.empty_like(q)
    S = torch.empty((B, H, h, h), dtype=torch.float32, device=q.device) if return_state else None
    if ws is None:
        ws = workspace(abi.ttt_workspace_bytes(desc, abi.TTT_PATH_LINEAR), q.device)
    abi.ttt_linear_attn_fwd(desc, q, k, v, eta, S0, out, S, ws, stream=stream)
    return out, S


def recurrent_desc(q, W1, chunk, order="update_apply", sign=1, update_mask=abi.TTT_UPDATE_ALL,
                   renorm=False, momentum=False, ns_steps=0):
    B, H, N, h = q.shape
    return abi.ttt_desc(B=B, H=H, N=N, h=h, m=W1.shape[1], chunk=chunk, dtype=_dtype_code(q),
                        order=ORDERS[order], sign=sign, update_mask=update_mask,
                        renorm=int(renorm), momentum=int(momentum), ns_steps=ns_steps)


def lact_recurrent_fwd(q, k, v, eta, W0, W2, W1, chunk, *, order="update_apply", sign=1,
                       update_mask=abi.TTT_UPDATE_ALL, renorm=False, alpha=None, ns_steps=0,
                       M_init=None, return_weights=True, return_momentum=False, out=None,
                       ws=None, stream=None):
    """Recurrent LaCT form. Returns (out, (W0, W2, W1) finals or None, momentum or None).
    Momentum is on when ``alpha`` [B,H,C] is given; ``M_init`` [B,H,3hm] resumes it."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n, q.dtype)
    _need(eta, "eta", torch.float32)
    _need(alpha, "alpha", torch.float32)
    for t, n in ((W0, "W0"), (W2, "W2"), (W1, "W1")):
        _need(t, n, torch.float32)
    momentum = alpha is not None
    desc = recurrent_desc(q, W1, chunk, order, sign, update_mask, renorm, momentum, ns_steps)
    B, H, N, h = q.shape
    m = desc.m
    dev = q.device
    if out is None:
        out = torch.empty_like(q)
    Wf = None
    if return_weights:
        Wf = (torch.empty((B, H, h, m), dtype=torch.float32, device=dev),
              torch.empty((B, H, h, m), dtype=torch.float32, device=dev),
              torch.empty((B, H, m, h), dtype=torch.float32, device=dev))
    M = None
    if momentum and (return_momentum or M_init is not None):
        M = torch.zeros((B, H, 3 * h * m), dtype=torch.float32, device=dev)
        if M_init is not None:
            M.copy_(M_init)
    if ws is None:
        ws = workspace(abi.ttt_workspace_bytes(desc, abi.TTT_PATH_RECURRENT), dev)
    abi.ttt_lact_recurrent_fwd(desc, q, k, v, eta, alpha, W0, W2, W1, out,
                               Wf[0] if Wf else None, Wf[1] if Wf else None,
                               Wf[2] if Wf else None, M, ws, stream=stream)
    return out, Wf, M


def lm_target(X0, conv_w, W_target, *, out=None, ws=None, stream=None):
    """LM-aligned target Vbar = Conv1D(X0) W_target (bf16 [N,d])."""
    _need(X0, "X0", torch.bfloat16)
    _need(conv_w, "conv_w", torch.float32)
    _need(W_target, "W_target", torch.bfloat16)
    N, d = X0.shape
    if out is None:
        out = torch.empty_like(X0)
    if ws is None:
        ws = workspace(abi.ttt_lm_target_workspace_bytes(N, d), X0.device)
    abi.ttt_lm_target(N, d, X0, conv_w, W_target, out, ws, stream=stream)
    return out


# ----------------------------------------------------------------- the token mixer's operators
ACTS = {None: abi.TTT_ACT_NONE, "silu": abi.TTT_ACT_SILU}
NORMS = {None: abi.TTT_NORM_NONE, "rms": abi.TTT_NORM_RMS, "l2": abi.TTT_NORM_L2}
PAIRS = {"halves": abi.TTT_PAIRS_HALVES, "interleaved": abi.TTT_PAIRS_INTERLEAVED}


def _on_device(fn):
    """Runs ``fn`` with the device of its first tensor as the current one, on that device's
    current stream, or on ``stream`` with what the call allocates belonging to it (memory of
    another stream could be handed out again while the kernels still run)."""
    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        first = args[0] if args else None
        if not isinstance(first, torch.Tensor):
            first = next((t for t in (*args, *kw.values()) if isinstance(t, torch.Tensor)), None)
        if first is None or not first.is_cuda:
            return fn(*args, stream=stream, **kw)
        index = first.device.index
        if stream is not None:
            if isinstance(stream, int):
                stream = torch.cuda.ExternalStream(stream, device=first.device)
            if stream.device_index != index:
                raise ValueError(f"stream is of device {stream.device_index}, the tensors of {index}")
            with torch.cuda.stream(stream):
                return fn(*args, stream=stream.cuda_stream, **kw)
        raw = torch._C._cuda_getCurrentRawStream(index)
        if index == torch._C._cuda_getDevice():
            return fn(*args, stream=raw, **kw)
        with torch.cuda.device(index):
            return fn(*args, stream=raw, **kw)
    return call


def _choice(table, key, name):
    if key not in table:
        raise ValueError(f"{name} must be one of {list(table)}, got {key!r}")
    return table[key]


def _dense(t, name, shape, dtype, device):
    """A contiguous tensor of exactly this shape and type, or None."""
    if t is None or t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous():
        return
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _rows(t, name, lead, width, dtype, device):
    """Elements between the tokens of ``t`` [*lead, *width] (lead: B, N or B); 0 when None."""
    if t is None or t.dtype is dtype and t.is_contiguous() and t.shape == lead + width and t.device == device:
        return 0
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != lead + width:
        raise ValueError(f"{name} must be {lead + width}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if t.is_contiguous():
        return 0
    n, strides, outer = 1, t.stride(), len(lead)
    for i in range(len(strides) - 1, outer - 1, -1):
        size = width[i - outer]
        if size > 1 and strides[i] != n:
            raise ValueError(f"{name}: the elements of a token must be contiguous")
        n *= size
    row = tokens = None      # the innermost of the leading sizes above 1 sets the stride
    for i in range(outer - 1, -1, -1):
        if lead[i] <= 1:
            continue
        if row is None:
            row, tokens = strides[i], lead[i]
        elif strides[i] != row * tokens:
            raise ValueError(f"{name}: all tokens must be one stride apart")
    if row is None:
        return 0
    if row < n:
        raise ValueError(f"{name}: tokens overlap (stride {row}, {n} elements)")
    return row


def _scratch(ws, nbytes, device):
    """The caller's workspace, or a new one of ``nbytes`` (None when none is needed)."""
    if ws is None:
        return workspace(nbytes, device) if nbytes else None
    if ws.device != device:
        raise ValueError(f"ws must be on {device}, got {ws.device}")
    if not ws.is_contiguous():
        raise ValueError("ws must be contiguous")
    return ws


def _sizes(*sizes):
    """The sizes as they are, refused where the descriptor's 32 bits would wrap them."""
    if max(sizes) > 2**31 - 1:
        raise ValueError(f"sizes must be below 2^31, got {sizes}")
    return sizes


def _new(t):
    """A dense tensor like ``t``, or None."""
    if t is None:
        return None
    return torch.empty_like(t, memory_format=torch.contiguous_format)


def _first(t, name, dims):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions, got {tuple(t.shape)}")
    return t.device


def _conv_desc(x, w, bias, act, state, lens, lead):
    device = x.device
    D = x.shape[-1]
    if w.dim() != 2:
        raise ValueError(f"w must be [width, {D}], got {tuple(w.shape)}")
    width = w.shape[0]
    _dense(w, "w", (width, D), torch.float32, device)
    _dense(bias, "bias", (D,), torch.float32, device)
    _dense(state, "state", (lead[0], width - 1, D), x.dtype, device)
    _dense(lens, "lens", (lead[0],), torch.int32, device)
    return abi.ttt_conv_desc(*_sizes(lead[0], lead[1] if len(lead) > 1 else 1, D, width), _dtype_code(x),
                             _choice(ACTS, act, "act"), _rows(x, "x", lead, (D,), x.dtype, device))


@_on_device
def short_conv_fwd(x, w, *, bias=None, act="silu", state=None, lens=None, return_state=True,
                   out=None, state_out=None, stream=None):
    """Short causal depthwise convolution of x [B,N,D] with taps w [width,D] (tap j multiplies
    x[t-j]), after the inputs in ``state`` [B,width-1,D] (zeros when None). ``act`` is "silu" or
    None; ``lens`` [B] int32 gives the tokens of padded sequences. Returns (y, the state after
    the last token or None). ``state_out`` may be ``state``."""
    device = _first(x, "x", 3)
    desc = _conv_desc(x, w, bias, act, state, lens, tuple(x.shape[:2]))
    B, N, D = x.shape
    shape = (B, desc.width - 1, D)
    if out is None:
        out = _new(x)
    else:
        _dense(out, "out", (B, N, D), x.dtype, device)
    if state_out is None and return_state:
        state_out = x.new_empty(shape)
    else:
        _dense(state_out, "state_out", shape, x.dtype, device)
    abi.ttt_short_conv_fwd(desc, x, w, bias, state, lens, out, state_out, stream=stream)
    return out, state_out


@_on_device
def short_conv_step(x, w, state, *, bias=None, act="silu", out=None, stream=None):
    """The next token x [B,D] of B sequences; ``state`` [B,width-1,D] is shifted in place.
    Returns y [B,D]."""
    device = _first(x, "x", 2)
    desc = _conv_desc(x, w, bias, act, state, None, (x.shape[0],))
    if out is None:
        out = _new(x)
    else:
        _dense(out, "out", x.shape, x.dtype, device)
    abi.ttt_short_conv_step(desc, x, w, bias, state, out, stream=stream)
    return out


@_on_device
def short_conv_bwd(x, w, dy, *, bias=None, act="silu", state=None, lens=None, dstate=None,
                   ws=None, stream=None):
    """Backward of short_conv_fwd for dy [B,N,D] and ``dstate``, the gradient of the returned
    state (or None). Returns dx, dw, dbias (None without bias), the gradient of ``state`` (None
    without it)."""
    device = _first(x, "x", 3)
    desc = _conv_desc(x, w, bias, act, state, lens, tuple(x.shape[:2]))
    B, N, D = x.shape
    _dense(dy, "dy", (B, N, D), x.dtype, device)
    _dense(dstate, "dstate", (B, desc.width - 1, D), x.dtype, device)
    dx, dw, dbias, dstate_in = _new(x), _new(w), _new(bias), _new(state)
    ws = _scratch(ws, abi.ttt_short_conv_bwd_workspace_bytes(desc), device)
    abi.ttt_short_conv_bwd(desc, x, w, bias, state, lens, dy, dstate, dx, dw, dbias, dstate_in,
                           ws, stream=stream)
    return dx, dw, dbias, dstate_in


def _heads_desc(q, k, v, wq, wk, norm, eps, inv_freq, positions, pos0, pairs):
    if not 0 <= pos0 < 2**31:       # the descriptor's 32 bits would wrap it
        raise ValueError(f"pos0 must be in 0..2^31-1, got {pos0}")
    some = next((t for t in (q, k, v) if t is not None), None)
    if some is None:
        raise ValueError("one of q, k and v must be given")
    device = _first(some, "q, k and v", 4)
    B, N, _, h = some.shape
    row, H = [], []
    for t, name in ((q, "q"), (k, "k"), (v, "v")):
        if t is not None and t.dim() != 4:
            raise ValueError(f"{name} must be [B, N, heads, h], got {tuple(t.shape)}")
        n = 0 if t is None else t.shape[2]
        H.append(n)
        row.append(_rows(t, name, (B, N), (n, h), some.dtype, device))
    _dense(wq, "wq", (h,), torch.float32, device)
    _dense(wk, "wk", (h,), torch.float32, device)
    _dense(positions, "positions", (B, N), torch.int32, device)
    rot = 0
    if inv_freq is not None:
        rot, = _sizes(2 * inv_freq.numel())
        _dense(inv_freq, "inv_freq", (rot // 2,), torch.float32, device)
    return abi.ttt_heads_desc(*_sizes(B, N, H[0], H[1], H[2], h), _dtype_code(some),
                              _choice(NORMS, norm, "norm"), rot, _choice(PAIRS, pairs, "pairs"),
                              eps, pos0, row[0], row[1], row[2]), some


@_on_device
def head_norm_rope_fwd(q, k, v=None, *, wq=None, wk=None, norm="l2", eps=1e-6, inv_freq=None,
                       positions=None, pos0=0, pairs="halves", stream=None):
    """The layer's q, k, v [B,H,N,h] from the projection's token-major q, k, v [B,N,H,h] (any
    of them None): every query and key head normed ("l2", "rms" or None) and scaled by wq / wk
    [h], its first 2 * len(inv_freq) elements rotated by position * inv_freq (positions [B,N]
    int32, or pos0 + t), and v laid out. Returns (q, k, v)."""
    desc, some = _heads_desc(q, k, v, wq, wk, norm, eps, inv_freq, positions, pos0, pairs)
    B, N, _, h = some.shape
    out = [None if t is None else t.new_empty((B, t.shape[2], N, h)) for t in (q, k, v)]
    abi.ttt_head_norm_rope_fwd(desc, q, k, v, wq, wk, inv_freq, positions, *out, stream=stream)
    return tuple(out)


@_on_device
def head_norm_rope_bwd(q, k, v, dq, dk, dv, *, wq=None, wk=None, norm="l2", eps=1e-6,
                       inv_freq=None, positions=None, pos0=0, pairs="halves", ws=None,
                       stream=None):
    """Backward of head_norm_rope_fwd for the gradients dq, dk, dv [B,H,N,h] of its outputs.
    Returns the gradients of q, k, v [B,N,H,h] and of wq, wk (None for what was None)."""
    desc, some = _heads_desc(q, k, v, wq, wk, norm, eps, inv_freq, positions, pos0, pairs)
    B, N, _, h = some.shape
    device = some.device
    for t, g, name in ((q, dq, "dq"), (k, dk, "dk"), (v, dv, "dv")):
        if (t is None) != (g is None):
            raise ValueError(f"{name} must be given exactly when its tensor is")
        if g is not None:
            _dense(g, name, (B, t.shape[2], N, h), some.dtype, device)
    out = [_new(t) for t in (q, k, v)]
    dwq, dwk = _new(wq), _new(wk)
    sums = wq is not None or wk is not None
    ws = _scratch(ws, abi.ttt_head_norm_rope_bwd_workspace_bytes(desc) if sums else 0, device)
    abi.ttt_head_norm_rope_bwd(desc, q, k, wq, wk, inv_freq, positions, dq, dk, dv, *out, dwq,
                               dwk, ws, stream=stream)
    return (*out, dwq, dwk)


def _scan_desc(u, dt, A, Bm, Cm, D, z, dt_bias, softplus, state, lens, lead):
    device, dtype = u.device, u.dtype
    d = u.shape[-1]
    if A.dim() != 2:
        raise ValueError(f"A must be [{d}, S], got {tuple(A.shape)}")
    if Bm.dim() != len(lead) + 2:
        raise ValueError(f"Bm must be {lead} + (G, S), got {tuple(Bm.shape)}")
    S, G = A.shape[1], Bm.shape[-2]
    f32 = torch.float32
    _dense(A, "A", (d, S), f32, device)
    _dense(D, "D", (d,), f32, device)
    _dense(dt_bias, "dt_bias", (d,), f32, device)
    _dense(state, "state", (lead[0], d, S), f32, device)
    _dense(lens, "lens", (lead[0],), torch.int32, device)
    return abi.ttt_scan_desc(*_sizes(lead[0], lead[1] if len(lead) > 1 else 1, d, S, G), _dtype_code(u),
                             int(bool(softplus)), 0, _rows(u, "u", lead, (d,), dtype, device),
                             _rows(dt, "dt", lead, (d,), dtype, device),
                             _rows(z, "z", lead, (d,), dtype, device),
                             _rows(Bm, "Bm", lead, (G, S), dtype, device),
                             _rows(Cm, "Cm", lead, (G, S), dtype, device))


@_on_device
def selective_scan_fwd(u, dt, A, Bm, Cm, *, D=None, z=None, dt_bias=None, softplus=True,
                       state=None, lens=None, return_state=True, out=None, state_out=None, ws=None,
                       stream=None):
    """Selective state space scan of u, dt [B,N,D] with A [D,S], Bm, Cm [B,N,G,S], the skip D
    [D], the gate z [B,N,D] and dt_bias [D], from ``state`` [B,D,S] fp32 (zeros when None);
    ``lens`` [B] int32 gives the tokens of padded sequences. Returns (y [B,N,D], the state after
    the last token or None). ``state_out`` may be ``state``."""
    device = _first(u, "u", 3)
    desc = _scan_desc(u, dt, A, Bm, Cm, D, z, dt_bias, softplus, state, lens, tuple(u.shape[:2]))
    shape = (desc.B, desc.D, desc.S)
    if out is None:
        out = _new(u)
    else:
        _dense(out, "out", u.shape, u.dtype, device)
    if state_out is None and return_state:
        state_out = A.new_empty(shape)
    else:
        _dense(state_out, "state_out", shape, torch.float32, device)
    ws = _scratch(ws, abi.ttt_selective_scan_workspace_bytes(desc, 0), device)
    abi.ttt_selective_scan_fwd(desc, u, dt, A, Bm, Cm, D, z, dt_bias, state, lens, out,
                               state_out, ws, stream=stream)
    return out, state_out


@_on_device
def selective_scan_step(u, dt, A, Bm, Cm, state, *, D=None, z=None, dt_bias=None, softplus=True,
                        out=None, stream=None):
    """The next token of B sequences: u, dt, z [B,D], Bm, Cm [B,G,S]; ``state`` [B,D,S] fp32 is
    updated in place. Returns y [B,D]."""
    device = _first(u, "u", 2)
    desc = _scan_desc(u, dt, A, Bm, Cm, D, z, dt_bias, softplus, state, None, (u.shape[0],))
    if out is None:
        out = _new(u)
    else:
        _dense(out, "out", u.shape, u.dtype, device)
    abi.ttt_selective_scan_step(desc, u, dt, A, Bm, Cm, D, z, dt_bias, state, out,
                                stream=stream)
    return out


@_on_device
def selective_scan_bwd(u, dt, A, Bm, Cm, dy, *, D=None, z=None, dt_bias=None, softplus=True,
                       state=None, lens=None, dstate=None, ws=None, stream=None):
    """Backward of selective_scan_fwd for dy [B,N,D] and ``dstate``, the gradient of the
    returned state (or None). Returns du, ddt, dA, dBm, dCm, dD, dz, ddt_bias, dstate_in (None
    for what was None)."""
    device = _first(u, "u", 3)
    desc = _scan_desc(u, dt, A, Bm, Cm, D, z, dt_bias, softplus, state, lens, tuple(u.shape[:2]))
    _dense(dy, "dy", u.shape, u.dtype, device)
    _dense(dstate, "dstate", (desc.B, desc.D, desc.S), torch.float32, device)

    du, ddt, dA, dB, dC = _new(u), _new(dt), _new(A), _new(Bm), _new(Cm)
    dD, dz, dbias, dstate_in = _new(D), _new(z), _new(dt_bias), _new(state)
    ws = _scratch(ws, abi.ttt_selective_scan_workspace_bytes(desc, 1), device)
    abi.ttt_selective_scan_bwd(desc, u, dt, A, Bm, Cm, D, z, dt_bias, state, lens, dy, dstate,
                               du, ddt, dA, dB, dC, dD, dz, dbias, dstate_in, ws,
                               stream=stream)
    return du, ddt, dA, dB, dC, dD, dz, dbias, dstate_in
