"""Sequence operators of ``librlcs.so`` (the C ABI in include/rlcs_seq.h).

The mixing layers of a policy and critic over rollouts: a gated linear
recurrence, the head norm with rotary positions, causal attention and linear
attention over packed episodes, each with its gradient and its form for single
steps.
Argument marshalling only, as in ``binding``: PyTorch supplies device memory
and the stream, every step runs in the CUDA library, and a status other than
OK raises ``RlcsError``. Each function takes a `stream` (default: the current
one); outputs and temporary copies are allocated on it.

Nothing is recorded for automatic differentiation: results are detached, and
the gradients come from the ``_backward`` calls (examples/sequence_policy.py
wraps them in ``torch.autograd.Function``). Calls may come from any thread.
"""
import ctypes
import functools

import torch

from . import binding as _b

_lib = _b.lib()
_DTYPES = {torch.float32: 0, torch.bfloat16: 1}
ROPE_SCALINGS = {"plain": 0, "linear": 1, "base": 2, "parts": 3}
EXPORTED = ("rlcs_gated_scan", "rlcs_gated_scan_backward", "rlcs_gated_step", "rlcs_rope_table",
            "rlcs_qk_norm_rope", "rlcs_qk_norm_rope_scratch_bytes", "rlcs_qk_norm_rope_backward",
            "rlcs_attention_status", "rlcs_attention_scratch_bytes", "rlcs_attention",
            "rlcs_attention_backward", "rlcs_attention_step_scratch_bytes", "rlcs_attention_step",
            "rlcs_linear_attention_scratch_bytes", "rlcs_linear_attention",
            "rlcs_linear_attention_backward", "rlcs_linear_attention_step")


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
        "rlcs_attention_status": ([], I),
        "rlcs_attention_scratch_bytes": ([I64, I64], SZ),
        "rlcs_attention": (view * 3 + [P] * 3 + [I64] * 5 + [F, I, P, SZ, P], I),
        "rlcs_attention_backward": ([P] + view * 3 + [P] * 6 + [I64] * 5 + [F, I, P, SZ, P], I),
        "rlcs_attention_step_scratch_bytes": ([I64] * 5, SZ),
        "rlcs_attention_step": ([P] + [P, I64, I64, I64] * 2 + [P, P] + [I64] * 5
                                + [F, I, P, SZ, P], I),
        "rlcs_linear_attention_scratch_bytes": ([I64] * 5, SZ),
        "rlcs_linear_attention": (view * 3 + [P] * 5 + [I64] * 5 + [F, I, P, SZ, P], I),
        "rlcs_linear_attention_backward": ([P] + view * 3 + [P] * 8 + [I64] * 5
                                           + [F, I, P, SZ, P], I),
        "rlcs_linear_attention_step": (view * 3 + [P] * 5 + [I64] * 4 + [F, I, P], I),
    }
    for name, (args, res) in sig.items():
        f = getattr(_lib, name)
        f.argtypes = args
        f.restype = res


_declare()


def _call(name, *args):
    """Call the library with addresses and numbers; raise on any other status."""
    st = _fn[name](*args)
    if st:
        raise _b.RlcsError(st, name)


_fn = {name: getattr(_lib, name) for name in EXPORTED}
_raw_stream = torch._C._cuda_getCurrentRawStream

# Some calls are several launches that pass values through a scratch, and the
# interpreter lock is released while one is issued. So a scratch is the call's
# own: taken from PyTorch's allocator (in a capture, from the graph's memory)
# and given back once the launches are issued, since what the allocator hands
# it to next on this stream runs after them.
_alloc = torch._C._cuda_cudaCachingAllocator_raw_alloc
_free = torch._C._cuda_cudaCachingAllocator_raw_delete
_attended = set()  # devices with calls that may record a status
_statuses = ["rlcs_attention_status"]  # and the functions that read it


@functools.lru_cache(maxsize=256)
def _scratch_bytes(name, *sizes):
    return _fn[name](*sizes)


def _call_with_scratch(name, need, stream, *args):
    """_call with `need` bytes of scratch and the stream as last arguments."""
    ws = _alloc(need, stream)
    try:
        _call(name, *args, ws, need, stream)
    finally:
        _free(ws)


def check_scratch():
    """Wait for every device with calls of attention, linear attention or the
    losses, and raise what they recorded there since the last check."""
    for dev in sorted(_attended):
        with torch.cuda.device(dev):
            for name in _statuses:
                _b._check(_fn[name](), name)


def _streamed(f):
    """Give `f` a `stream` argument: with one, the call runs with that stream
    (and its device) current, so its outputs and copies belong to it."""
    @functools.wraps(f)
    def call(*args, stream=None, **kw):
        if stream is None:
            return f(*args, **kw)
        with torch.cuda.stream(stream):
            return f(*args, **kw)
    return call


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


def _main(t, name, dim, dtypes=_DTYPES):
    """The call's leading tensor and its device, which must be the current
    one: the library launches there."""
    _need(t, name, dim, dtypes)
    dev = t.get_device()
    if dev != torch.cuda.current_device():
        _b._devices(t)  # raises
    return t, dev


def _like(t, name, shape, dtype, dev):
    """`t` as a contiguous tensor of this shape, dtype and device."""
    if (not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.shape != shape
            or t.get_device() != dev):
        _need(t, name, len(shape), (dtype,))
        if t.shape != shape:
            raise ValueError("%s must have shape %s, got %s"
                             % (name, tuple(shape), tuple(t.shape)))
        raise ValueError("%s must be on cuda:%d, got %s" % (name, dev, t.device))
    return t if t.is_contiguous() else t.contiguous()


def _mask(t, name, shape, dev):
    if t is None:
        return None
    return _like(t, name, shape, torch.uint8 if isinstance(t, torch.Tensor)
                 and t.dtype is torch.uint8 else torch.bool, dev)


def _maybe(t, name, shape, dtype, dev):
    return None if t is None else _like(t, name, shape, dtype, dev)


def _at(t):
    return None if t is None else t.data_ptr()


def _heads(t, name, dtypes, dev, multiple):
    """A [tokens, heads, D] tensor the library can read in place, or a copy:
    its last dimension contiguous, and where `multiple` is 8 its strides
    multiples of 8 elements and its base 16-byte aligned. Returns the tensor,
    token stride and head stride."""
    _need(t, name, 3, dtypes)
    if t.get_device() != dev:
        raise ValueError("%s must be on cuda:%d, got %s" % (name, dev, t.device))
    n, H, D = t.shape
    ts, hs, ds = t.stride()
    if H == 1:
        hs = D
    if n <= 1:
        ts = max(1, H) * hs
    bad = (D > 1 and ds != 1) or ts <= 0 or hs <= 0
    if multiple > 1:
        bad = bad or ts % multiple or hs % multiple or t.data_ptr() % 16
    if bad:
        t, ts, hs = t.contiguous(), H * D, D
        if multiple > 1 and t.data_ptr() % 16:  # contiguous already, but off a 16-byte boundary
            t = t.clone()
    return t, ts, hs


@_streamed
def rlcs_gated_scan(x, gate, reset=None, h0=None, out=None):
    """h_t = keep_t sigmoid(gate_t) h_{t-1} + (1 - sigmoid(gate_t)) x_t over
    [B, T, D] (float32 or bfloat16). `reset` [B, T] (bool or uint8) starts a
    new episode at each set step; `h0` [B, D] float32 is the state before the
    first. Returns (h, h_last): the states in x's dtype, and the last one in
    float32."""
    x, dev = _main(x, "x", 3)
    B, T, D = x.shape
    x = x.contiguous()
    gate = _like(gate, "gate", x.shape, x.dtype, dev)
    reset = _mask(reset, "reset", (B, T), dev)
    h0 = _maybe(h0, "h0", (B, D), torch.float32, dev)
    h = torch.empty_like(x) if out is None else _b._out(out, "out", x)
    last = torch.empty((B, D), dtype=torch.float32, device=x.device)
    _call("rlcs_gated_scan", x.data_ptr(), gate.data_ptr(), _at(reset), _at(h0), h.data_ptr(),
          last.data_ptr(), B, T, D, _DTYPES[x.dtype], _raw_stream(dev))
    return (h if out is None else h.view(x.shape)), last


@_streamed
def rlcs_gated_scan_backward(dh, x, gate, h, reset=None, h0=None, dh_last=None):
    """Gradients (dx, dgate, dh0) of rlcs_gated_scan from the gradients of its
    states (and of its last state, if given); `h` is the forward output. dh0
    [B, D] float32 is the gradient of the state before the first step."""
    x, dev = _main(x, "x", 3)
    B, T, D = x.shape
    x = x.contiguous()
    dh = _like(dh, "dh", x.shape, x.dtype, dev)
    gate = _like(gate, "gate", x.shape, x.dtype, dev)
    h = _like(h, "h", x.shape, x.dtype, dev)
    reset = _mask(reset, "reset", (B, T), dev)
    h0 = _maybe(h0, "h0", (B, D), torch.float32, dev)
    dh_last = _maybe(dh_last, "dh_last", (B, D), torch.float32, dev)
    dx, dgate = torch.empty_like(x), torch.empty_like(x)
    dh0 = torch.empty((B, D), dtype=torch.float32, device=x.device)
    _call("rlcs_gated_scan_backward", dh.data_ptr(), x.data_ptr(), gate.data_ptr(), h.data_ptr(),
          _at(reset), _at(h0), _at(dh_last), dx.data_ptr(), dgate.data_ptr(), dh0.data_ptr(), B, T,
          D, _DTYPES[x.dtype], _raw_stream(dev))
    return dx, dgate, dh0


@_streamed
def rlcs_gated_step(x, gate, state, reset=None, new_state=None):
    """One step of the recurrence for B states: x, gate [B, D]; state [B, D]
    float32; reset [B]. Returns (h, new_state). Pass `new_state=state` to
    update the states in place."""
    x, dev = _main(x, "x", 2)
    B, D = x.shape
    x = x.contiguous()
    gate = _like(gate, "gate", x.shape, x.dtype, dev)
    old = _like(state, "state", x.shape, torch.float32, dev)
    reset = _mask(reset, "reset", (B,), dev)
    # written through its own memory, so a caller's buffer must be contiguous
    new_state = (torch.empty_like(old) if new_state is None
                 else _b._out(new_state, "new_state", x, dtype=torch.float32))
    h = torch.empty_like(x)
    _call("rlcs_gated_step", x.data_ptr(), gate.data_ptr(), _at(reset), old.data_ptr(),
          new_state.data_ptr(), h.data_ptr(), B, D, _DTYPES[x.dtype], _raw_stream(dev))
    return h, new_state


@_streamed
def rlcs_rope_table(max_pos, rotary_dim, base=10000.0, scaling="plain", factor=1.0,
                    trained_len=0.0, slow=1.0, fast=32.0, scale=1.0, device=None):
    """Rotary tables (cos, sin), each [max_pos, rotary_dim // 2] float32.
    `scaling`: "plain", "linear" (positions interpolated by `factor`), "base"
    (the base raised so that the slowest pair is) or "parts" (pairs that turn
    more than `fast` times over `trained_len` kept, those under `slow`
    interpolated, linear in between). `scale` multiplies both tables."""
    if scaling not in ROPE_SCALINGS:
        raise ValueError("scaling must be one of %s" % sorted(ROPE_SCALINGS))
    device = torch.device("cuda", torch.cuda.current_device()) if device is None \
        else torch.device(device)
    cos, sin = (torch.empty((max(0, max_pos), max(0, rotary_dim // 2)), dtype=torch.float32,
                            device=device) for _ in range(2))
    _b._devices(cos, sin)
    _call("rlcs_rope_table", cos.data_ptr(), sin.data_ptr(), max_pos, rotary_dim, base,
          ROPE_SCALINGS[scaling], factor, trained_len, slow, fast, scale,
          _raw_stream(cos.get_device()))
    return cos, sin


def _norm_args(q, k, q_weight, k_weight, cos, sin, positions):
    q, dev = _main(q, "q", 3)
    q, qts, qhs = _heads(q, "q", _DTYPES, dev, 1)
    k, kts, khs = _heads(k, "k", (q.dtype,), dev, 1)
    n, Hq, D = q.shape
    Hk = k.shape[1]
    if k.shape[0] != n or k.shape[2] != D:
        raise ValueError("k must have shape (%d, heads, %d)" % (n, D))
    qw = _like(q_weight, "q_weight", (D,), torch.float32, dev)
    kw = _like(k_weight, "k_weight", (D,), torch.float32, dev)
    cos = _need(cos, "cos", 2, (torch.float32,))
    cos = _like(cos, "cos", cos.shape, torch.float32, dev)
    sin = _like(sin, "sin", cos.shape, torch.float32, dev)
    positions = _like(positions, "positions", (n,), torch.int32, dev)
    arrays = (q.data_ptr(), qts, qhs, k.data_ptr(), kts, khs, qw.data_ptr(), kw.data_ptr(),
              cos.data_ptr(), sin.data_ptr(), positions.data_ptr())
    keep = (q, k, qw, kw, cos, sin, positions)
    return dev, (n, Hq, Hk, D, 2 * cos.shape[1], cos.shape[0]), arrays, keep


@_streamed
def rlcs_qk_norm_rope(q, k, q_weight, k_weight, cos, sin, positions, eps=1e-6, interleaved=False):
    """RMS norm of every head of q [tokens, Hq, D] and k [tokens, Hk, D]
    (float32 or bfloat16; strided views are read in place), then rotary
    positions on the first 2 * cos.shape[1] elements: pairs (i, i + half), or
    (2i, 2i + 1) with `interleaved`. `positions` [tokens] int32 selects the
    tables' rows. Returns contiguous (q_out, k_out)."""
    dev, sizes, arrays, keep = _norm_args(q, k, q_weight, k_weight, cos, sin, positions)
    n, Hq, Hk, D = sizes[:4]
    qo = torch.empty((n, Hq, D), dtype=q.dtype, device=q.device)
    ko = torch.empty((n, Hk, D), dtype=q.dtype, device=q.device)
    _call("rlcs_qk_norm_rope", *arrays, qo.data_ptr(), ko.data_ptr(), *sizes,
          1 if interleaved else 0, eps, _DTYPES[q.dtype], _raw_stream(dev))
    return qo, ko


@_streamed
def rlcs_qk_norm_rope_backward(dq_out, dk_out, q, k, q_weight, k_weight, cos, sin, positions,
                               eps=1e-6, interleaved=False):
    """Gradients (dq, dk, dq_weight, dk_weight) of rlcs_qk_norm_rope; the
    weights' gradients are float32 and summed in a fixed order."""
    dev, sizes, arrays, keep = _norm_args(q, k, q_weight, k_weight, cos, sin, positions)
    n, Hq, Hk, D = sizes[:4]
    dq_out = _like(dq_out, "dq_out", (n, Hq, D), q.dtype, dev)
    dk_out = _like(dk_out, "dk_out", (n, Hk, D), q.dtype, dev)
    dq, dk = torch.empty_like(dq_out), torch.empty_like(dk_out)
    dqw = torch.empty(D, dtype=torch.float32, device=q.device)
    dkw = torch.empty(D, dtype=torch.float32, device=q.device)
    _call_with_scratch("rlcs_qk_norm_rope_backward",
                       _scratch_bytes("rlcs_qk_norm_rope_scratch_bytes", D), _raw_stream(dev),
                       dq_out.data_ptr(), dk_out.data_ptr(), *arrays, dq.data_ptr(), dk.data_ptr(),
                       dqw.data_ptr(), dkw.data_ptr(), *sizes, 1 if interleaved else 0, eps,
                       _DTYPES[q.dtype])
    return dq, dk, dqw, dkw


def _attention_args(q, k, v, cu_seqlens):
    q, dev = _main(q, "q", 3, (torch.bfloat16,))
    q, qts, qhs = _heads(q, "q", (torch.bfloat16,), dev, 8)
    k, kts, khs = _heads(k, "k", (torch.bfloat16,), dev, 8)
    v, vts, vhs = _heads(v, "v", (torch.bfloat16,), dev, 8)
    n, Hq, D = q.shape
    Hk = k.shape[1]
    if k.shape != (n, Hk, D) or v.shape != (n, Hk, D):
        raise ValueError("k and v must have shape (%d, heads, %d)" % (n, D))
    if Hk == 0 or Hq % Hk:
        raise ValueError("the query heads (%d) must be a multiple of the key/value heads (%d)"
                         % (Hq, Hk))
    cu = _need(cu_seqlens, "cu_seqlens", 1, (torch.int32,))
    cu = _like(cu, "cu_seqlens", cu.shape, torch.int32, dev)
    if cu.numel() < 1:
        raise ValueError("cu_seqlens must hold the sequences' bounds (one more than sequences)")
    arrays = (q.data_ptr(), qts, qhs, k.data_ptr(), kts, khs, v.data_ptr(), vts, vhs)
    return dev, (cu.numel() - 1, n, Hq, Hk, D), arrays, (q, k, v, cu)


def _scale(scale, D):
    return max(D, 1) ** -0.5 if scale is None else scale  # (the library refuses D = 0)


def _rows_out(sequences, shape, like):
    """An array the library writes whole, where there are sequences at all."""
    make = torch.empty if sequences else torch.zeros
    return make(shape, dtype=like.dtype, device=like.device)


@_streamed
def rlcs_attention(q, k, v, cu_seqlens, scale=None, return_lse=False):
    """Causal attention over packed sequences: q [tokens, Hq, D], k and v
    [tokens, Hk, D] bfloat16, D a multiple of 8 up to 128, Hq a multiple of
    Hk; sequence s holds tokens cu_seqlens[s] to cu_seqlens[s+1] (int32).
    `scale` (positive) defaults to D ** -0.5. Views whose strides are multiples of
    8 elements on a 16-byte boundary are read in place, others copied. Returns
    out [tokens, Hq, D], or (out, lse [Hq, tokens] float32) with
    `return_lse`. Tokens that no sequence holds (before the first bound, from
    the last on) get zeros, and -inf in lse."""
    dev, sizes, arrays, keep = _attention_args(q, k, v, cu_seqlens)
    sequences, n, Hq, _, D = sizes
    out = _rows_out(sequences, (n, Hq, D), q)
    lse = torch.empty((Hq, n), dtype=torch.float32, device=q.device) if return_lse else None
    if return_lse and sequences == 0:
        lse.fill_(-float("inf"))
    _attended.add(dev)
    _call_with_scratch("rlcs_attention", _scratch_bytes("rlcs_attention_scratch_bytes", n, Hq),
                       _raw_stream(dev), *arrays, keep[3].data_ptr(), out.data_ptr(), _at(lse),
                       *sizes, _scale(scale, D), _DTYPES[q.dtype])
    return (out, lse) if return_lse else out


@_streamed
def rlcs_attention_backward(dout, q, k, v, out, lse, cu_seqlens, scale=None):
    """Gradients (dq, dk, dv) of rlcs_attention from the gradient of its
    output; `out` and `lse` are the forward call's. The gradients of a shared
    key/value head sum over its query heads; those of tokens that no sequence
    holds are zeros."""
    dev, sizes, arrays, keep = _attention_args(q, k, v, cu_seqlens)
    sequences, n, Hq, Hk, D = sizes
    dout = _like(dout, "dout", (n, Hq, D), q.dtype, dev)
    out = _like(out, "out", (n, Hq, D), q.dtype, dev)
    dout, out = (t.clone() if t.data_ptr() % 16 else t for t in (dout, out))
    lse = _like(lse, "lse", (Hq, n), torch.float32, dev)
    dq = _rows_out(sequences, (n, Hq, D), q)
    dk, dv = (_rows_out(sequences, (n, Hk, D), q) for _ in range(2))
    _attended.add(dev)
    _call_with_scratch("rlcs_attention_backward",
                       _scratch_bytes("rlcs_attention_scratch_bytes", n, Hq), _raw_stream(dev),
                       dout.data_ptr(), *arrays, out.data_ptr(), lse.data_ptr(),
                       keep[3].data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), *sizes,
                       _scale(scale, D), _DTYPES[q.dtype])
    return dq, dk, dv


def _cache(t, name, B, D, dev):
    _need(t, name, 4, (torch.bfloat16,))
    if t.get_device() != dev:
        raise ValueError("%s must be on cuda:%d, got %s" % (name, dev, t.device))
    batch, positions, heads, width = t.shape
    if batch != B or width != D:
        raise ValueError("%s must have shape (%d, positions, heads, %d)" % (name, B, D))
    b, s, h, d = t.stride()
    # a dimension of one element has no stride to speak of
    if heads == 1:
        h = 8
    if positions <= 1:
        s = 8
    if B <= 1:
        b = 8
    if ((D > 1 and d != 1) or t.data_ptr() % 16 or b <= 0 or s <= 0 or h <= 0
            or b % 8 or s % 8 or h % 8):
        raise ValueError("%s must be read in place: its last dimension contiguous, its strides "
                         "multiples of 8 elements, its base on a 16-byte boundary" % name)
    return t.data_ptr(), b, s, h


@_streamed
def rlcs_attention_step(q, k_cache, v_cache, lengths, scale=None, out=None):
    """Attention of one new token per sequence over its cache: q [B, Hq, D],
    k_cache and v_cache [B, S, Hk, D] bfloat16 (strided views are read in
    place; a cache is never copied), lengths [B] int32, the entries to attend
    to (0 gives a zero output). Returns out [B, Hq, D]."""
    q, dev = _main(q, "q", 3, (torch.bfloat16,))
    q = q.contiguous()
    if q.data_ptr() % 16:
        q = q.clone()
    B, Hq, D = q.shape
    ks = _cache(k_cache, "k_cache", B, D, dev)
    vs = _cache(v_cache, "v_cache", B, D, dev)
    S, Hk = k_cache.shape[1], k_cache.shape[2]
    if v_cache.shape != k_cache.shape:
        raise ValueError("v_cache must have k_cache's shape")
    if Hk == 0 or Hq % Hk:
        raise ValueError("the query heads (%d) must be a multiple of the key/value heads (%d)"
                         % (Hq, Hk))
    lengths = _like(lengths, "lengths", (B,), torch.int32, dev)
    o = torch.empty_like(q) if out is None else _b._out(out, "out", q)
    _call_with_scratch("rlcs_attention_step",
                       _scratch_bytes("rlcs_attention_step_scratch_bytes", B, S, Hq, Hk, D),
                       _raw_stream(dev), q.data_ptr(), *ks, *vs, lengths.data_ptr(), o.data_ptr(),
                       B, S, Hq, Hk, D, _scale(scale, D), _DTYPES[q.dtype])
    return o if out is None else o.view(q.shape)


def _linear_args(q, k, v, log_decay, cu_seqlens, state):
    dev, sizes, arrays, keep = _attention_args(q, k, v, cu_seqlens)
    sequences, _, _, Hk, D = sizes
    decay = _like(log_decay, "log_decay", (Hk,), torch.float32, dev)
    state = _matrices(state, "state", sequences, Hk, D, dev)
    return dev, sizes, arrays + (decay.data_ptr(), keep[3].data_ptr()), keep + (decay, state)


def _matrices(t, name, B, H, D, dev):
    """A [B, H, D, D] float32 array on a 16-byte boundary, or None."""
    t = _maybe(t, name, (B, H, D, D), torch.float32, dev)
    return t.clone() if t is not None and t.data_ptr() % 16 else t


@_streamed
def rlcs_linear_attention(q, k, v, log_decay, cu_seqlens, state=None, scale=None,
                          return_state=False):
    """Linear attention over packed sequences: S_t = exp(log_decay) S_{t-1} +
    k_t v_t^T per key/value head, out_t = scale q_t S_t. q [tokens, Hq, D], k
    and v [tokens, Hk, D], cu_seqlens and `scale` as for rlcs_attention;
    log_decay [Hk] float32 (0 keeps everything, -inf nothing but the token,
    positive values grow); `state` [sequences, Hk, D, D] float32,
    the states before the first tokens, defaults to zeros. Returns out
    [tokens, Hq, D], or (out, states after the last tokens) with
    `return_state`. Tokens that no sequence holds get zeros."""
    dev, sizes, arrays, keep = _linear_args(q, k, v, log_decay, cu_seqlens, state)
    sequences, n, Hq, Hk, D = sizes
    out = _rows_out(sequences, (n, Hq, D), q)
    last = (torch.empty((sequences, Hk, D, D), dtype=torch.float32, device=q.device)
            if return_state else None)
    _attended.add(dev)
    _call_with_scratch("rlcs_linear_attention",
                       _scratch_bytes("rlcs_linear_attention_scratch_bytes", *sizes),
                       _raw_stream(dev), *arrays, _at(keep[5]), out.data_ptr(), _at(last), *sizes,
                       _scale(scale, D), _DTYPES[q.dtype])
    return (out, last) if return_state else out


@_streamed
def rlcs_linear_attention_backward(dout, q, k, v, log_decay, cu_seqlens, state=None, dlast=None,
                                   scale=None):
    """Gradients (dq, dk, dv, dstate) of rlcs_linear_attention from those of
    its output and (`dlast` [sequences, Hk, D, D] float32) of its last states.
    The gradients of a shared key/value head sum over its query heads; dstate
    is None where no `state` was given; the decays are constants."""
    dev, sizes, arrays, keep = _linear_args(q, k, v, log_decay, cu_seqlens, state)
    sequences, n, Hq, Hk, D = sizes
    dout = _like(dout, "dout", (n, Hq, D), q.dtype, dev)
    dout = dout.clone() if dout.data_ptr() % 16 else dout
    dlast = _matrices(dlast, "dlast", sequences, Hk, D, dev)
    dq = _rows_out(sequences, (n, Hq, D), q)
    dk, dv = (_rows_out(sequences, (n, Hk, D), q) for _ in range(2))
    dstate = None if state is None else torch.empty_like(keep[5])
    _attended.add(dev)
    _call_with_scratch("rlcs_linear_attention_backward",
                       _scratch_bytes("rlcs_linear_attention_scratch_bytes", *sizes),
                       _raw_stream(dev), dout.data_ptr(), *arrays, _at(keep[5]), _at(dlast),
                       dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), _at(dstate), *sizes,
                       _scale(scale, D), _DTYPES[q.dtype])
    return dq, dk, dv, dstate


@_streamed
def rlcs_linear_attention_step(q, k, v, log_decay, state, reset=None, scale=None, new_state=None):
    """One step of linear attention for B states: q [B, Hq, D], k and v [B, Hk,
    D] bfloat16 (strided views are read in place), state [B, Hk, D, D]
    float32; `reset` [B] (bool or uint8) drops the old state where it is set.
    Returns (out [B, Hq, D], new_state). Pass `new_state=state` to update the
    states in place."""
    q, dev = _main(q, "q", 3, (torch.bfloat16,))
    q, qbs, qhs = _heads(q, "q", (torch.bfloat16,), dev, 1)
    k, kbs, khs = _heads(k, "k", (torch.bfloat16,), dev, 1)
    v, vbs, vhs = _heads(v, "v", (torch.bfloat16,), dev, 1)
    B, Hq, D = q.shape
    Hk = k.shape[1]
    if k.shape != (B, Hk, D) or v.shape != (B, Hk, D):
        raise ValueError("k and v must have shape (%d, heads, %d)" % (B, D))
    if Hk == 0 or Hq % Hk:
        raise ValueError("the query heads (%d) must be a multiple of the key/value heads (%d)"
                         % (Hq, Hk))
    decay = _like(log_decay, "log_decay", (Hk,), torch.float32, dev)
    old = _matrices(state, "state", B, Hk, D, dev)
    reset = _mask(reset, "reset", (B,), dev)
    # written through its own memory, so a caller's buffer must be contiguous
    new_state = torch.empty_like(old) if new_state is None else _b._out(new_state, "new_state", old)
    out = torch.empty((B, Hq, D), dtype=q.dtype, device=q.device)
    _call("rlcs_linear_attention_step", q.data_ptr(), qbs, qhs, k.data_ptr(), kbs, khs,
          v.data_ptr(), vbs, vhs, decay.data_ptr(), _at(reset), old.data_ptr(),
          new_state.data_ptr(), out.data_ptr(), B, Hq, Hk, D, _scale(scale, D), _DTYPES[q.dtype],
          _raw_stream(dev))
    return out, new_state
