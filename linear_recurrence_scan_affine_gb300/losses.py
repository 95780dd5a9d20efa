"""Losses of a policy's logits in ``librlcs.so`` (the C ABI in include/rlcs_loss.h).

The clipped policy loss that takes the estimators' advantages, and distillation
from a teacher's top logits, each with its gradient. Argument marshalling only,
as in ``sequence``: the same checks, errors, streams and threads, and nothing
recorded for automatic differentiation.
"""
import collections
import ctypes

import torch

from . import binding as _b
from . import sequence as _s

_lib = _b.lib()
EXPORTED = ("rlcs_loss_status", "rlcs_policy_loss", "rlcs_policy_loss_backward",
            "rlcs_distill_loss", "rlcs_distill_loss_backward")

#: A token's loss, log probability of its action, entropy and (given a
#: reference) KL term, each [tokens] float32; `kl` is None without ref_logp.
PolicyLoss = collections.namedtuple("PolicyLoss", "loss logp entropy kl")


def _declare():
    P, I64, F, I = ctypes.c_void_p, ctypes.c_int64, ctypes.c_double, ctypes.c_int
    row = [P, I64]
    sig = {
        "rlcs_loss_status": [],
        "rlcs_policy_loss": row + [P] * 9 + [I64] * 2 + [F] * 4 + [I, P],
        "rlcs_policy_loss_backward": [P] + row + [P] * 10 + [I64] * 2 + [F] * 4 + [I, P],
        "rlcs_distill_loss": row + [P] * 5 + [I64] * 3 + [F, I, P],
        "rlcs_distill_loss_backward": [P] + row + [P] * 6 + [I64] * 3 + [F, I, P],
    }
    for name, args in sig.items():
        f = getattr(_lib, name)
        f.argtypes = args
        f.restype = I


_declare()
_s._fn.update((name, getattr(_lib, name)) for name in EXPORTED)
_s._statuses.append("rlcs_loss_status")


def _rows(logits):
    """Logits the library can read in place, or a copy, with their row stride
    and device."""
    x, dev = _s._main(logits, "logits", 2)
    n, V = x.shape
    _s._attended.add(dev)
    stride = V if n <= 1 else x.stride(0)
    if (V > 1 and x.stride(1) != 1) or stride < V:
        x, stride = x.contiguous(), V
    return x, stride, dev


def _dlogits(out, x):
    if out is not None:
        return _b._out(out, "out", x)
    return torch.empty(x.shape, dtype=x.dtype, device=x.device)


def _policy_args(logits, actions, old_logp, advantages, ref_logp, mask):
    x, stride, dev = _rows(logits)
    one = (x.shape[0],)
    actions = _s._like(actions, "actions", one, torch.int32, dev)
    old = _s._like(old_logp, "old_logp", one, torch.float32, dev)
    adv = _s._like(advantages, "advantages", one, torch.float32, dev)
    ref = _s._maybe(ref_logp, "ref_logp", one, torch.float32, dev)
    mask = _s._mask(mask, "mask", one, dev)
    keep = (x, actions, old, adv, ref, mask)
    return dev, keep, (x.data_ptr(), stride, actions.data_ptr(), old.data_ptr(), adv.data_ptr(),
                       _s._at(ref), _s._at(mask))


def _policy_results(x, ref):
    """A PolicyLoss of new arrays: rows of one allocation."""
    rows = torch.empty((3 if ref is None else 4, x.shape[0]), dtype=torch.float32,
                       device=x.device).unbind(0)
    return PolicyLoss(*rows) if ref is not None else PolicyLoss(*rows, None)


@_s._streamed
def rlcs_policy_loss(logits, actions, old_logp, advantages, ref_logp=None, mask=None,
                     clip_low=0.2, clip_high=0.2, kl_coef=0.0, entropy_coef=0.0):
    """Clipped policy loss of every token: logits [tokens, V] (float32 or
    bfloat16; rows that lie apart are read in place), actions [tokens] int32,
    old_logp and advantages [tokens] float32. With r = exp(logp - old_logp),
      loss = -min(r A, clip(r, 1 - clip_low, 1 + clip_high) A)
             + kl_coef (exp(d) - d - 1) - entropy_coef H,   d = ref_logp - logp.
    `mask` [tokens] (bool or uint8) leaves tokens out: zeros, nothing of them
    read. Logits of -inf are actions that cannot be taken. Returns a
    PolicyLoss."""
    dev, keep, arrays = _policy_args(logits, actions, old_logp, advantages, ref_logp, mask)
    x = keep[0]
    out = _policy_results(x, keep[4])
    _s._call("rlcs_policy_loss", *arrays, *(_s._at(t) for t in out), x.shape[0], x.shape[1],
             clip_low, clip_high, kl_coef, entropy_coef, _s._DTYPES[x.dtype], _s._raw_stream(dev))
    return out


@_s._streamed
def rlcs_policy_loss_backward(dloss, logits, actions, old_logp, advantages, ref_logp=None,
                              mask=None, clip_low=0.2, clip_high=0.2, kl_coef=0.0,
                              entropy_coef=0.0, out=None, return_loss=False):
    """Gradient in the logits of sum(dloss * loss), loss that of
    rlcs_policy_loss: dlogits [tokens, V] in the logits' dtype. `out` may be
    the logits themselves, which are then overwritten. With `return_loss`,
    (dlogits, PolicyLoss) from the same reading of the logits: the whole loss
    of a step whose weights dloss [tokens] float32 are known beforehand."""
    dev, keep, arrays = _policy_args(logits, actions, old_logp, advantages, ref_logp, mask)
    x = keep[0]
    dloss = _s._like(dloss, "dloss", (x.shape[0],), torch.float32, dev)
    dx = _dlogits(out, x)
    stats = _policy_results(x, keep[4]) if return_loss else (None,) * 4
    _s._call("rlcs_policy_loss_backward", dloss.data_ptr(), *arrays, dx.data_ptr(),
             *(_s._at(t) for t in stats), x.shape[0], x.shape[1], clip_low, clip_high, kl_coef,
             entropy_coef, _s._DTYPES[x.dtype], _s._raw_stream(dev))
    dx = dx if out is None else dx.view(x.shape)
    return (dx, stats) if return_loss else dx


def _distill_args(logits, top_ids, top_logits, teacher_lse, mask):
    x, stride, dev = _rows(logits)
    n = x.shape[0]
    ids = _s._need(top_ids, "top_ids", 2, (torch.int32,))
    ids = _s._like(ids, "top_ids", torch.Size((n, ids.shape[1])), torch.int32, dev)
    top = _s._like(top_logits, "top_logits", ids.shape, torch.float32, dev)
    lse = _s._maybe(teacher_lse, "teacher_lse", (n,), torch.float32, dev)
    mask = _s._mask(mask, "mask", (n,), dev)
    keep = (x, ids, top, lse, mask)
    return dev, keep, (x.data_ptr(), stride, ids.data_ptr(), top.data_ptr(), _s._at(lse),
                       _s._at(mask))


@_s._streamed
def rlcs_distill_loss(logits, top_ids, top_logits, teacher_lse=None, mask=None, temperature=1.0):
    """Distillation from a teacher's K top logits: logits [tokens, V] (float32
    or bfloat16), top_ids [tokens, K] int32, top_logits [tokens, K] float32.
    loss [tokens] = sum_j q_j (log q_j - log p[top_ids_j]) with p = softmax(
    logits / temperature), q the softmax of top_logits / temperature, or
    exp(top_logits / temperature - teacher_lse) where teacher_lse [tokens],
    the log sum over all of the teacher's logits, is given. Entries whose id
    lies outside [0, V) or whose logit is -inf are absent. `mask` as in
    rlcs_policy_loss."""
    dev, keep, arrays = _distill_args(logits, top_ids, top_logits, teacher_lse, mask)
    x = keep[0]
    loss = torch.empty(x.shape[0], dtype=torch.float32, device=x.device)
    _s._call("rlcs_distill_loss", *arrays, loss.data_ptr(), x.shape[0], x.shape[1],
             keep[1].shape[1], temperature, _s._DTYPES[x.dtype], _s._raw_stream(dev))
    return loss


@_s._streamed
def rlcs_distill_loss_backward(dloss, logits, top_ids, top_logits, teacher_lse=None, mask=None,
                               temperature=1.0, out=None, return_loss=False):
    """Gradient in the logits of sum(dloss * loss), loss that of
    rlcs_distill_loss: dlogits [tokens, V] in the logits' dtype. `out` may be
    the logits themselves. With `return_loss`, (dlogits, loss) from the same
    reading of the logits."""
    dev, keep, arrays = _distill_args(logits, top_ids, top_logits, teacher_lse, mask)
    x = keep[0]
    dloss = _s._like(dloss, "dloss", (x.shape[0],), torch.float32, dev)
    dx = _dlogits(out, x)
    loss = (torch.empty(x.shape[0], dtype=torch.float32, device=x.device) if return_loss
            else None)
    _s._call("rlcs_distill_loss_backward", dloss.data_ptr(), *arrays, dx.data_ptr(), _s._at(loss),
             x.shape[0], x.shape[1], keep[1].shape[1], temperature, _s._DTYPES[x.dtype],
             _s._raw_stream(dev))
    dx = dx if out is None else dx.view(x.shape)
    return (dx, loss) if return_loss else dx
