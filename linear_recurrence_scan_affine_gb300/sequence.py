"""Sequence operators of ``librlcs.so`` (the C ABI in include/rlcs_seq.h).

The mixing layers of a policy and critic over rollouts: a gated linear
recurrence, the head norm with rotary positions, and causal attention over
packed episodes, each with its gradient and its form for single steps.
Argument marshalling only, as in ``binding``: PyTorch supplies device memory
and the stream, every step runs in the CUDA library, and a status other than
OK raises ``RlcsError``. Outputs and temporary copies are allocated on the
stream the call runs on.
"""
import ctypes

import torch

from . import binding as _b

_lib = _b.lib()
_DTYPES = {torch.float32: 0, torch.bfloat16: 1}
ROPE_SCALINGS = {"plain": 0, "linear": 1, "base": 2, "parts": 3}
EXPORTED = ("rlcs_gated_scan", "rlcs_gated_scan_backward", "rlcs_gated_step", "rlcs_rope_table",
            "rlcs_qk_norm_rope", "rlcs_qk_norm_rope_scratch_bytes", "rlcs_qk_norm_rope_backward",
            "rlcs_attention_scratch_bytes", "rlcs_attention", "rlcs_attention_backward",
            "rlcs_attention_step_scratch_bytes", "rlcs_attention_step")


def _declare():
    P, I64, F, SZ, I = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_double, ctypes.c_size_t,
                        ctypes.c_int)
    view = [P, I64, I64]
    sig = {
        "rlcs_gated_scan": ([P] * 6 + [I64] * 3 + [I, P], I),
        "rlcs_gated_scan_backward": ([P] * 10 + [I64] * 3 + [I, P], I),
        "rlcs_gated_step": ([P] * 6 + [I64] * 2 + [I, P], I),
        "rlcs_rope_table": ([P, P, I64, I64, F, I] + [F] * 5 + [P], I),
        "rlcs_qk_norm_rope": (view * 2 + [P] * 7 + [I64] * 6 + [I, F, I, P], I),
        "rlcs_qk_norm_rope_scratch_bytes": ([I64], SZ),
        "rlcs_qk_norm_rope_backward": ([P, P] + view * 2 + [P] * 9 + [I64] * 6
                                       + [I, F, I, P, SZ, P], I),
        "rlcs_attention_scratch_bytes": ([I64, I64], SZ),
        "rlcs_attention": (view * 3 + [P] * 3 + [I64] * 5 + [F, I, P, SZ, P], I),
        "rlcs_attention_backward": ([P] + view * 3 + [P] * 6 + [I64] * 5 + [F, I, P, SZ, P], I),
        "rlcs_attention_step_scratch_bytes": ([I64] * 5, SZ),
        "rlcs_attention_step": ([P] + [P, I64, I64, I64] * 2 + [P, P] + [I64] * 5
                                + [F, I, P, SZ, P], I),
    }
    for name, (args, res) in sig.items():
        f = getattr(_lib, name)
        f.argtypes = args
        f.restype = res


_declare()

# One scratch buffer per (device, stream), apart from the estimators'
# workspaces: these operators leave sums in it, which would break the chunk
# records a look-back relies on. Its first 64 bytes hold a status word and are
# zeroed when it is made.
_scratch_cache = {}


def _scratch(need, device, stream):
    key = (device.index, stream.cuda_stream)
    with _b._ws_lock:
        ws = _scratch_cache.get(key)
        if ws is None or ws.numel() < need:
            with torch.cuda.stream(stream):
                ws = torch.empty(max(need, 1 << 20), dtype=torch.uint8, device=device)
                ws[:64].zero_()
            _scratch_cache[key] = ws
    return ws, ws.numel()


def check_scratch():
    """Synchronise and check the status word of every scratch buffer."""
    with _b._ws_lock:
        items = list(_scratch_cache.values())
    for ws in items:
        _b._check(_lib.rlcs_check_status(_b._ptr(ws), None), "rlcs_check_status")


def _need(t, name, dim, dtypes):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dim() != dim:
        raise ValueError("%s must have %d dimensions, got %d" % (name, dim, t.dim()))
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if t.dtype not in dtypes:
        raise TypeError("%s must be %s, got %s"
                        % (name, " or ".join(str(d) for d in dtypes), t.dtype))
    return t


def _like(t, name, shape, dtype):
    _need(t, name, len(shape), (dtype,))
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s" % (name, tuple(shape)))
    return t.contiguous()


def _mask(t, name, shape):
    if t is None:
        return None
    _need(t, name, len(shape), (torch.bool, torch.uint8))
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s" % (name, tuple(shape)))
    t = t.contiguous()
    return t.view(torch.uint8) if t.dtype == torch.bool else t


def _on(main, stream):
    if not isinstance(main, torch.Tensor) or not main.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if stream is None:
        return torch.cuda.current_stream(main.device)
    return stream


def _heads(t, name, dtypes, multiple):
    """A [tokens, heads, D] tensor the library can read in place, or a copy:
    its last dimension contiguous, and where `multiple` is 8 its strides
    multiples of 8 elements and its base 16-byte aligned. Returns the tensor,
    token stride and head stride."""
    _need(t, name, 3, dtypes)
    n, H, D = t.shape
    ts, hs = t.stride(0), t.stride(1)
    if H == 1:
        hs = D
    if n <= 1:
        ts = max(1, H) * hs
    bad = (D > 1 and t.stride(2) != 1) or ts <= 0 or hs <= 0
    if multiple > 1:
        bad = bad or ts % multiple or hs % multiple or t.data_ptr() % 16
    if bad:
        t, ts, hs = t.contiguous(), H * D, D
        if multiple > 1 and t.data_ptr() % 16:  # contiguous already, but off a 16-byte boundary
            t = t.clone()
    return t, ts, hs


def rlcs_gated_scan(x, gate, reset=None, h0=None, out=None, stream=None):
    """h_t = keep_t sigmoid(gate_t) h_{t-1} + (1 - sigmoid(gate_t)) x_t over
    [B, T, D] (float32 or bfloat16). `reset` [B, T] (bool or uint8) starts a
    new episode at each set step; `h0` [B, D] float32 is the state before the
    first. Returns (h, h_last): the states in x's dtype, and the last one in
    float32."""
    s = _on(x, stream)
    with torch.cuda.stream(s):
        x = _need(x, "x", 3, tuple(_DTYPES)).contiguous()
        B, T, D = x.shape
        gate = _like(gate, "gate", x.shape, x.dtype)
        reset = _mask(reset, "reset", (B, T))
        h0 = None if h0 is None else _like(h0, "h0", (B, D), torch.float32)
        h = torch.empty_like(x) if out is None else _b._out(out, "out", x)
        last = torch.empty((B, D), dtype=torch.float32, device=x.device)
        _b._devices(x, gate, reset, h0, h, stream=stream)
    _b._check(_lib.rlcs_gated_scan(_b._ptr(x), _b._ptr(gate), _b._ptr(reset), _b._ptr(h0),
                                   _b._ptr(h), _b._ptr(last), B, T, D, _DTYPES[x.dtype],
                                   _b._stream(s)), "rlcs_gated_scan")
    return h.view(x.shape), last


def rlcs_gated_scan_backward(dh, x, gate, h, reset=None, h0=None, dh_last=None, stream=None):
    """Gradients (dx, dgate, dh0) of rlcs_gated_scan from the gradients of its
    states (and of its last state, if given); `h` is the forward output. dh0
    [B, D] float32 is the gradient of the state before the first step."""
    s = _on(x, stream)
    with torch.cuda.stream(s):
        x = _need(x, "x", 3, tuple(_DTYPES)).contiguous()
        B, T, D = x.shape
        dh, gate, h = (_like(t, n, x.shape, x.dtype)
                       for t, n in ((dh, "dh"), (gate, "gate"), (h, "h")))
        reset = _mask(reset, "reset", (B, T))
        h0 = None if h0 is None else _like(h0, "h0", (B, D), torch.float32)
        dh_last = None if dh_last is None else _like(dh_last, "dh_last", (B, D), torch.float32)
        dx, dgate = torch.empty_like(x), torch.empty_like(x)
        dh0 = torch.empty((B, D), dtype=torch.float32, device=x.device)
        _b._devices(x, dh, gate, h, reset, h0, dh_last, stream=stream)
    _b._check(_lib.rlcs_gated_scan_backward(
        _b._ptr(dh), _b._ptr(x), _b._ptr(gate), _b._ptr(h), _b._ptr(reset), _b._ptr(h0),
        _b._ptr(dh_last), _b._ptr(dx), _b._ptr(dgate), _b._ptr(dh0), B, T, D, _DTYPES[x.dtype],
        _b._stream(s)), "rlcs_gated_scan_backward")
    return dx, dgate, dh0


def rlcs_gated_step(x, gate, state, reset=None, new_state=None, stream=None):
    """One step of the recurrence for B states: x, gate [B, D]; state [B, D]
    float32; reset [B]. Returns (h, new_state). Pass `new_state=state` to
    update the states in place."""
    s = _on(x, stream)
    with torch.cuda.stream(s):
        x = _need(x, "x", 2, tuple(_DTYPES)).contiguous()
        B, D = x.shape
        gate = _like(gate, "gate", x.shape, x.dtype)
        in_place = new_state is state
        old = _like(state, "state", (B, D), torch.float32)
        reset = _mask(reset, "reset", (B,))
        if new_state is None:
            new_state = torch.empty_like(old)
        elif in_place:  # written through its own memory, so it must be contiguous
            _b._out(new_state, "new_state", x, dtype=torch.float32)
        else:
            _b._out(new_state, "new_state", x, dtype=torch.float32)
        h = torch.empty_like(x)
        _b._devices(x, gate, old, new_state, reset, stream=stream)
    _b._check(_lib.rlcs_gated_step(_b._ptr(x), _b._ptr(gate), _b._ptr(reset), _b._ptr(old),
                                   _b._ptr(new_state), _b._ptr(h), B, D, _DTYPES[x.dtype],
                                   _b._stream(s)), "rlcs_gated_step")
    return h, new_state


def rlcs_rope_table(max_pos, rotary_dim, base=10000.0, scaling="plain", factor=1.0,
                    trained_len=0.0, slow=1.0, fast=32.0, scale=1.0, device=None, stream=None):
    """Rotary tables (cos, sin), each [max_pos, rotary_dim // 2] float32.
    `scaling`: "plain", "linear" (positions interpolated by `factor`), "base"
    (the base raised so that the slowest pair is) or "parts" (pairs that turn
    more than `fast` times over `trained_len` kept, those under `slow`
    interpolated, linear in between). `scale` multiplies both tables."""
    if scaling not in ROPE_SCALINGS:
        raise ValueError("scaling must be one of %s" % sorted(ROPE_SCALINGS))
    device = torch.device("cuda", torch.cuda.current_device()) if device is None \
        else torch.device(device)
    s = torch.cuda.current_stream(device) if stream is None else stream
    with torch.cuda.stream(s):
        cos, sin = (torch.empty((max(0, max_pos), max(0, rotary_dim // 2)), dtype=torch.float32,
                                device=device) for _ in range(2))
        _b._devices(cos, sin, stream=stream)
    _b._check(_lib.rlcs_rope_table(_b._ptr(cos), _b._ptr(sin), max_pos, rotary_dim, base,
                                   ROPE_SCALINGS[scaling], factor, trained_len, slow, fast, scale,
                                   _b._stream(s)), "rlcs_rope_table")
    return cos, sin


def _norm_args(q, k, q_weight, k_weight, cos, sin, positions):
    q, qts, qhs = _heads(q, "q", tuple(_DTYPES), 1)
    k, kts, khs = _heads(k, "k", (q.dtype,), 1)
    n, Hq, D = q.shape
    Hk = k.shape[1]
    if k.shape[0] != n or k.shape[2] != D:
        raise ValueError("k must have shape (%d, heads, %d)" % (n, D))
    qw, kw = (_like(w, name, (D,), torch.float32)
              for w, name in ((q_weight, "q_weight"), (k_weight, "k_weight")))
    cos = _need(cos, "cos", 2, (torch.float32,)).contiguous()
    sin = _like(sin, "sin", cos.shape, torch.float32)
    positions = _like(positions, "positions", (n,), torch.int32)
    arrays = [_b._ptr(q), qts, qhs, _b._ptr(k), kts, khs, _b._ptr(qw), _b._ptr(kw), _b._ptr(cos),
              _b._ptr(sin), _b._ptr(positions)]
    keep = (q, k, qw, kw, cos, sin, positions)
    return (n, Hq, Hk, D, 2 * cos.shape[1], cos.shape[0]), arrays, keep


def rlcs_qk_norm_rope(q, k, q_weight, k_weight, cos, sin, positions, eps=1e-6, interleaved=False,
                      stream=None):
    """RMS norm of every head of q [tokens, Hq, D] and k [tokens, Hk, D]
    (float32 or bfloat16; strided views are read in place), then rotary
    positions on the first 2 * cos.shape[1] elements: pairs (i, i + half), or
    (2i, 2i + 1) with `interleaved`. `positions` [tokens] int32 selects the
    tables' rows. Returns contiguous (q_out, k_out)."""
    s = _on(q, stream)
    with torch.cuda.stream(s):
        sizes, arrays, keep = _norm_args(q, k, q_weight, k_weight, cos, sin, positions)
        n, Hq, Hk, D = sizes[:4]
        qo = torch.empty((n, Hq, D), dtype=q.dtype, device=q.device)
        ko = torch.empty((n, Hk, D), dtype=q.dtype, device=q.device)
        _b._devices(*keep, stream=stream)
    _b._check(_lib.rlcs_qk_norm_rope(*arrays, _b._ptr(qo), _b._ptr(ko), *sizes,
                                     1 if interleaved else 0, eps, _DTYPES[q.dtype],
                                     _b._stream(s)), "rlcs_qk_norm_rope")
    return qo, ko


def rlcs_qk_norm_rope_backward(dq_out, dk_out, q, k, q_weight, k_weight, cos, sin, positions,
                               eps=1e-6, interleaved=False, stream=None):
    """Gradients (dq, dk, dq_weight, dk_weight) of rlcs_qk_norm_rope; the
    weights' gradients are float32 and summed in a fixed order."""
    s = _on(q, stream)
    with torch.cuda.stream(s):
        sizes, arrays, keep = _norm_args(q, k, q_weight, k_weight, cos, sin, positions)
        n, Hq, Hk, D = sizes[:4]
        dq_out = _like(dq_out, "dq_out", (n, Hq, D), q.dtype)
        dk_out = _like(dk_out, "dk_out", (n, Hk, D), q.dtype)
        dq, dk = torch.empty_like(dq_out), torch.empty_like(dk_out)
        dqw, dkw = (torch.empty(D, dtype=torch.float32, device=q.device) for _ in range(2))
        _b._devices(*keep, dq_out, dk_out, stream=stream)
    ws, wsb = _scratch(_lib.rlcs_qk_norm_rope_scratch_bytes(D) + 64, q.device, s)
    _b._check(_lib.rlcs_qk_norm_rope_backward(
        _b._ptr(dq_out), _b._ptr(dk_out), *arrays, _b._ptr(dq), _b._ptr(dk), _b._ptr(dqw),
        _b._ptr(dkw), *sizes, 1 if interleaved else 0, eps, _DTYPES[q.dtype],
        ctypes.c_void_p(ws.data_ptr() + 64), wsb - 64, _b._stream(s)),
        "rlcs_qk_norm_rope_backward")
    return dq, dk, dqw, dkw


def _attention_args(q, k, v, cu_seqlens):
    views = [_heads(t, name, (torch.bfloat16,), 8) for t, name in ((q, "q"), (k, "k"), (v, "v"))]
    n, Hq, D = q.shape
    Hk = k.shape[1]
    if tuple(k.shape) != (n, Hk, D) or tuple(v.shape) != (n, Hk, D):
        raise ValueError("k and v must have shape (%d, heads, %d)" % (n, D))
    if Hk == 0 or Hq % Hk:
        raise ValueError("the query heads (%d) must be a multiple of the key/value heads (%d)"
                         % (Hq, Hk))
    cu = _need(cu_seqlens, "cu_seqlens", 1, (torch.int32,)).contiguous()
    if cu.numel() < 1:
        raise ValueError("cu_seqlens must hold the sequences' bounds (one more than sequences)")
    arrays = []
    for t, ts, hs in views:
        arrays += [_b._ptr(t), ts, hs]
    keep = tuple(t for t, _, _ in views) + (cu,)
    return (cu.numel() - 1, n, Hq, Hk, D), arrays, keep


def rlcs_attention(q, k, v, cu_seqlens, scale=None, return_lse=False, stream=None):
    """Causal attention over packed sequences: q [tokens, Hq, D], k and v
    [tokens, Hk, D] bfloat16, D a multiple of 8 up to 128, Hq a multiple of
    Hk; sequence s holds tokens cu_seqlens[s] to cu_seqlens[s+1] (int32).
    `scale` defaults to D ** -0.5. Views whose strides are multiples of 8
    elements on a 16-byte boundary are read in place, others copied. Returns
    out [tokens, Hq, D], or (out, lse [Hq, tokens] float32) with
    `return_lse`. Tokens that no sequence holds are left unwritten."""
    s = _on(q, stream)
    with torch.cuda.stream(s):
        sizes, arrays, keep = _attention_args(q, k, v, cu_seqlens)
        _, n, Hq, _, D = sizes
        out = torch.empty((n, Hq, D), dtype=q.dtype, device=q.device)
        lse = torch.empty((Hq, n), dtype=torch.float32, device=q.device) if return_lse else None
        _b._devices(*keep, stream=stream)
    ws, wsb = _scratch(_lib.rlcs_attention_scratch_bytes(n, Hq), q.device, s)
    _b._check(_lib.rlcs_attention(*arrays, _b._ptr(keep[3]), _b._ptr(out), _b._ptr(lse), *sizes,
                                  D ** -0.5 if scale is None else scale, _DTYPES[q.dtype],
                                  _b._ptr(ws), wsb, _b._stream(s)), "rlcs_attention")
    return (out, lse) if return_lse else out


def rlcs_attention_backward(dout, q, k, v, out, lse, cu_seqlens, scale=None, stream=None):
    """Gradients (dq, dk, dv) of rlcs_attention from the gradient of its
    output; `out` and `lse` are the forward call's. The gradients of a shared
    key/value head sum over its query heads."""
    s = _on(q, stream)
    with torch.cuda.stream(s):
        sizes, arrays, keep = _attention_args(q, k, v, cu_seqlens)
        _, n, Hq, Hk, D = sizes
        dout, out = (_like(t, name, (n, Hq, D), q.dtype)
                     for t, name in ((dout, "dout"), (out, "out")))
        dout, out = (t.clone() if t.data_ptr() % 16 else t for t in (dout, out))
        lse = _like(lse, "lse", (Hq, n), torch.float32)
        dq = torch.empty((n, Hq, D), dtype=q.dtype, device=q.device)
        dk, dv = (torch.empty((n, Hk, D), dtype=q.dtype, device=q.device) for _ in range(2))
        _b._devices(*keep, dout, out, lse, stream=stream)
    ws, wsb = _scratch(_lib.rlcs_attention_scratch_bytes(n, Hq), q.device, s)
    _b._check(_lib.rlcs_attention_backward(
        _b._ptr(dout), *arrays, _b._ptr(out), _b._ptr(lse), _b._ptr(keep[3]), _b._ptr(dq),
        _b._ptr(dk), _b._ptr(dv), *sizes, D ** -0.5 if scale is None else scale,
        _DTYPES[q.dtype], _b._ptr(ws), wsb, _b._stream(s)), "rlcs_attention_backward")
    return dq, dk, dv


def _cache(t, name, B, D):
    _need(t, name, 4, (torch.bfloat16,))
    if t.shape[0] != B or t.shape[3] != D:
        raise ValueError("%s must have shape (%d, positions, heads, %d)" % (name, B, D))
    strides = list(t.stride()[:3])
    # a dimension of one element has no stride to speak of
    for i in (2, 1, 0):
        if t.shape[i] <= 1:
            strides[i] = 8 if i == 2 else max(8, strides[i + 1] * t.shape[i + 1])
    if (D > 1 and t.stride(3) != 1) or t.data_ptr() % 16 or any(x <= 0 or x % 8 for x in strides):
        raise ValueError("%s must be read in place: its last dimension contiguous, its strides "
                         "multiples of 8 elements, its base on a 16-byte boundary" % name)
    return strides


def rlcs_attention_step(q, k_cache, v_cache, lengths, scale=None, out=None, stream=None):
    """Attention of one new token per sequence over its cache: q [B, Hq, D],
    k_cache and v_cache [B, S, Hk, D] bfloat16 (strided views are read in
    place; a cache is never copied), lengths [B] int32, the entries to attend
    to (0 gives a zero output). Returns out [B, Hq, D]."""
    s = _on(q, stream)
    with torch.cuda.stream(s):
        q = _need(q, "q", 3, (torch.bfloat16,)).contiguous()
        if q.data_ptr() % 16:
            q = q.clone()
        B, Hq, D = q.shape
        ks, vs = _cache(k_cache, "k_cache", B, D), _cache(v_cache, "v_cache", B, D)
        S, Hk = k_cache.shape[1], k_cache.shape[2]
        if v_cache.shape != k_cache.shape:
            raise ValueError("v_cache must have k_cache's shape")
        if Hk == 0 or Hq % Hk:
            raise ValueError("the query heads (%d) must be a multiple of the key/value heads (%d)"
                             % (Hq, Hk))
        lengths = _like(lengths, "lengths", (B,), torch.int32)
        o = torch.empty_like(q) if out is None else _b._out(out, "out", q)
        _b._devices(q, k_cache, v_cache, lengths, o, stream=stream)
    ws, wsb = _scratch(_lib.rlcs_attention_step_scratch_bytes(B, S, Hq, Hk, D) + 64, q.device, s)
    _b._check(_lib.rlcs_attention_step(
        _b._ptr(q), _b._ptr(k_cache), *ks, _b._ptr(v_cache), *vs, _b._ptr(lengths), _b._ptr(o), B,
        S, Hq, Hk, D, D ** -0.5 if scale is None else scale, _DTYPES[q.dtype],
        ctypes.c_void_p(ws.data_ptr() + 64), wsb - 64, _b._stream(s)), "rlcs_attention_step")
    return o.view(q.shape)
