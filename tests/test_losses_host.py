"""Host-side checks of the losses' C ABI and of linear attention's: every
declared function is exported and bad arguments are refused with the
documented status before anything is launched (fake device addresses)."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

from linear_recurrence_scan_affine_gb300 import binding, losses, sequence

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, MISALIGNED, WORKSPACE = 0, 1, 2, 3
F32, BF16 = 0, 1
lib = binding.lib()


def fake(i, off=0):
    return ctypes.c_void_p(0x7f0000000000 + (i << 36) + off)


def test_header_binding_and_library_agree():
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "rlcs_loss.h")).read(),
                 flags=re.S)
    names = sorted(set(re.findall(r"\b(rlcs_[a-z_]+)\s*\(", src)))
    assert names == sorted(losses.EXPORTED)
    assert all(hasattr(lib, n) for n in names)


def test_header_compiles_as_c(tmp_path):
    prog = tmp_path / "h.c"
    prog.write_text('#include "rlcs_loss.h"\nint main(void) { return 0; }\n')
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-c", "-I",
                    os.path.join(ROOT, "include"), str(prog), "-o", str(tmp_path / "h.o")],
                   check=True)


def policy(x=fake(0), stride=8, a=fake(1), old=fake(2), adv=fake(3), ref=None, mask=None,
           loss=fake(4), logp=fake(5), H=fake(6), kl=None, n=4, V=8, low=0.2, high=0.2, klc=0.0,
           ent=0.0, dtype=F32):
    return lib.rlcs_policy_loss(x, stride, a, old, adv, ref, mask, loss, logp, H, kl, n, V, low,
                                high, klc, ent, dtype, None)


def policy_back(w=fake(7), x=fake(0), stride=8, dx=fake(8), loss=None, logp=None, n=4, V=8,
                dtype=F32, a=fake(1)):
    return lib.rlcs_policy_loss_backward(w, x, stride, a, fake(2), fake(3), None, None, dx, loss,
                                         logp, None, None, n, V, 0.2, 0.2, 0.0, 0.0, dtype, None)


def test_policy_refusals():
    nan, inf = float("nan"), float("inf")
    for bad in (dict(x=None), dict(a=None), dict(old=None), dict(adv=None), dict(loss=None),
                dict(n=-1), dict(V=0), dict(V=1 << 31), dict(n=1 << 40, V=1 << 30), dict(stride=7),
                dict(stride=-8), dict(stride=1 << 60), dict(dtype=2), dict(low=-0.01),
                dict(low=1.01), dict(low=nan), dict(high=-0.1), dict(high=inf), dict(klc=inf),
                dict(klc=0.1), dict(kl=fake(9)), dict(ent=nan), dict(loss=fake(0)),
                dict(loss=fake(0, 124)), dict(logp=fake(4)), dict(H=fake(3)), dict(H=fake(5, 8))):
        assert policy(**bad) == INVALID, bad
    for bad in (dict(w=None), dict(dx=None), dict(x=None), dict(dx=fake(0, 4)), dict(stride=7),
                dict(dx=fake(0), stride=9), dict(dx=fake(7)), dict(loss=fake(8)),
                dict(loss=fake(0)), dict(dx=fake(0), loss=fake(0, 16)),
                dict(loss=fake(9), logp=fake(9))):
        assert policy_back(**bad) == INVALID, bad
    assert policy(x=fake(0, 2)) == MISALIGNED and policy(x=fake(0, 1), dtype=BF16) == MISALIGNED
    assert policy_back(dx=fake(8, 2)) == MISALIGNED
    assert policy(n=0, x=None, a=None, loss=None) == OK
    assert policy_back(n=0, w=None, dx=None) == OK


def distill(x=fake(0), stride=8, ids=fake(1), top=fake(2), lse=None, mask=None, loss=fake(3), n=4,
            V=8, K=2, t=1.0, dtype=F32):
    return lib.rlcs_distill_loss(x, stride, ids, top, lse, mask, loss, n, V, K, t, dtype, None)


def distill_back(w=fake(4), x=fake(0), dx=fake(5), loss=None, stride=8, n=4, K=2):
    return lib.rlcs_distill_loss_backward(w, x, stride, fake(1), fake(2), None, None, dx, loss, n,
                                          8, K, 1.0, F32, None)


def test_distill_refusals():
    for bad in (dict(x=None), dict(ids=None), dict(top=None), dict(loss=None), dict(n=-1),
                dict(V=0), dict(K=0), dict(K=1025), dict(t=0.0), dict(t=-1.0),
                dict(t=float("nan")), dict(t=float("inf")), dict(stride=5), dict(dtype=-1),
                dict(loss=fake(2)), dict(loss=fake(0, 32)), dict(loss=fake(1, 16)),
                dict(lse=fake(3, 8))):
        assert distill(**bad) == INVALID, bad
    for bad in (dict(w=None), dict(dx=None), dict(dx=fake(0, 16)), dict(dx=fake(1)),
                dict(dx=fake(0), stride=16), dict(loss=fake(5, 8)), dict(K=0),
                dict(dx=fake(0), loss=fake(0))):
        assert distill_back(**bad) == INVALID, bad
    assert distill(n=0, x=None, loss=None) == OK and distill_back(n=0, dx=None) == OK


def linear(q=fake(0), k=fake(1), v=fake(2), ld=fake(3), cu=fake(4), state=None, out=fake(5),
           last=None, seqs=1, n=4, Hq=2, Hk=1, D=64, scale=0.125, dtype=BF16, qs=(128, 64),
           ks=(64, 64), scratch=fake(6), size=1 << 30):
    return lib.rlcs_linear_attention(q, *qs, k, *ks, v, *ks, ld, cu, state, out, last, seqs, n, Hq,
                                     Hk, D, scale, dtype, scratch, size, None)


def linear_back(dout=fake(7), state=None, dlast=None, dq=fake(8), dk=fake(9), dv=fake(10),
                dstate=None, n=4, seqs=1, scratch=fake(6), size=1 << 30, qs=(128, 64)):
    return lib.rlcs_linear_attention_backward(
        dout, fake(0), *qs, fake(1), 64, 64, fake(2), 64, 64, fake(3), fake(4), state, dlast, dq,
        dk, dv, dstate, seqs, n, 2, 1, 64, 0.125, BF16, scratch, size, None)


def test_linear_attention_refusals():
    for bad in (dict(n=-1), dict(seqs=-1), dict(Hq=0), dict(Hq=3, Hk=2), dict(Hk=0), dict(D=0),
                dict(D=12), dict(D=136), dict(dtype=F32), dict(scale=float("nan")),
                dict(scale=0.0), dict(scale=1e31), dict(q=None), dict(k=None), dict(v=None),
                dict(ld=None), dict(cu=None), dict(out=None), dict(qs=(-128, 64)),
                dict(out=fake(0)), dict(out=fake(2, 16)), dict(last=fake(5)), dict(out=fake(3)),
                dict(state=fake(11), last=fake(11)), dict(scratch=fake(1)), dict(n=1 << 31),
                dict(state=fake(5, 64))):
        assert linear(**bad) == INVALID, bad
    for bad in (dict(qs=(132, 64)), dict(ks=(64, 60)), dict(q=fake(0, 8)), dict(out=fake(5, 2)),
                dict(state=fake(11, 4)), dict(last=fake(11, 8))):
        assert linear(**bad) == MISALIGNED, bad
    need = lib.rlcs_linear_attention_scratch_bytes(1, 4, 2, 1, 64)
    assert need >= 64
    for bad in ((-1, 4, 2, 1, 64), (1, -4, 2, 1, 64), (1, 4, 3, 2, 64), (1, 4, 2, 1, 130)):
        assert lib.rlcs_linear_attention_scratch_bytes(*bad) == 0
    for bad in (dict(scratch=None, size=0), dict(size=need - 1), dict(scratch=fake(6, 8))):
        assert linear(**bad) == WORKSPACE, bad
    assert linear(seqs=0, q=None) == OK
    for bad in (dict(dout=None), dict(dq=None), dict(dk=None), dict(dv=None),
                dict(dk=fake(9), dv=fake(9)), dict(dq=fake(7)), dict(dstate=fake(8)),
                dict(dlast=fake(11), dstate=fake(11)), dict(scratch=fake(7))):
        assert linear_back(**bad) == INVALID, bad
    assert linear_back(dout=fake(7, 2)) == MISALIGNED and linear_back(qs=(128, 68)) == MISALIGNED
    assert linear_back(dlast=fake(11, 4)) == MISALIGNED
    assert linear_back(size=8) == WORKSPACE
    assert linear_back(seqs=0) == OK


def linear_step(q=fake(0), qs=(128, 64), k=fake(1), ks=(64, 64), v=fake(2), ld=fake(3), reset=None,
                state=fake(4), new=fake(5), out=fake(6), B=2, Hq=2, Hk=1, D=64, scale=0.125,
                dtype=BF16):
    return lib.rlcs_linear_attention_step(q, *qs, k, *ks, v, *ks, ld, reset, state, new, out, B, Hq,
                                          Hk, D, scale, dtype, None)


def test_linear_step_refusals():
    for bad in (dict(B=-1), dict(Hq=3, Hk=2), dict(D=20), dict(D=0), dict(dtype=F32),
                dict(q=None), dict(k=None), dict(v=None), dict(ld=None), dict(state=None),
                dict(new=None), dict(out=None), dict(qs=(-128, 64)), dict(ks=(64, -1)),
                dict(out=fake(0)), dict(out=fake(4)), dict(new=fake(4, 16)),
                dict(new=fake(4), out=fake(4)), dict(reset=fake(5)), dict(scale=0.0),
                dict(B=1 << 31)):
        assert linear_step(**bad) == INVALID, bad
    for bad in (dict(q=fake(0, 1)), dict(state=fake(4, 8)), dict(new=fake(5, 4)),
                dict(out=fake(6, 2))):
        assert linear_step(**bad) == MISALIGNED, bad
    assert linear_step(B=0, q=None, state=None) == OK


def test_binding_refuses_host_tensors():
    x = torch.zeros(2, 3, 4)
    i, one = torch.zeros(3, dtype=torch.int32), torch.zeros(3)
    for call in (lambda: losses.rlcs_policy_loss(x[0], i, one, one),
                 lambda: losses.rlcs_policy_loss_backward(one, x[0], i, one, one),
                 lambda: losses.rlcs_distill_loss(x[0], i[:, None], one[:, None]),
                 lambda: losses.rlcs_distill_loss_backward(one, x[0], i[:, None], one[:, None]),
                 lambda: sequence.rlcs_linear_attention(x, x, x, one, i),
                 lambda: sequence.rlcs_linear_attention_backward(x, x, x, x, one, i),
                 lambda: sequence.rlcs_linear_attention_step(x, x, x, one, x)):
        with pytest.raises((ValueError, TypeError)):
            call()
