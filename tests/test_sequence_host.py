"""Host-side checks of the sequence operators' C ABI and binding: every
declared function is exported, and bad arguments are refused with the
documented status before anything is launched (fake device addresses)."""
import ctypes
import os
import re

import pytest
import torch

from linear_recurrence_scan_affine_gb300 import binding, sequence

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, MISALIGNED, WORKSPACE = 0, 1, 2, 3
F32, BF16 = 0, 1
lib = binding.lib()


def fake(i, off=0):
    return ctypes.c_void_p(0x7f0000000000 + (i << 32) + off)


def test_header_binding_and_library_agree():
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "rlcs_seq.h")).read(),
                 flags=re.S)
    names = sorted(set(re.findall(r"\b(rlcs_[a-z_]+)\s*\(", src)))
    assert names == sorted(sequence.EXPORTED)
    assert all(hasattr(lib, n) for n in names)


def test_header_compiles_as_c(tmp_path):
    import subprocess
    prog = tmp_path / "h.c"
    prog.write_text('#include "rlcs_seq.h"\nint main(void) { return 0; }\n')
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-c", "-I",
                    os.path.join(ROOT, "include"), str(prog), "-o", str(tmp_path / "h.o")],
                   check=True)


def scan(B=2, T=4, D=8, dtype=F32, x=fake(0), gate=fake(1), reset=None, h0=None, h=fake(2),
         last=fake(3)):
    return lib.rlcs_gated_scan(x, gate, reset, h0, h, last, B, T, D, dtype, None)


def back(B=2, T=4, D=8, dtype=F32, dh=fake(0), x=fake(1), gate=fake(2), h=fake(3), dx=fake(4),
         dgate=fake(5), dh0=fake(6), dh_last=None):
    return lib.rlcs_gated_scan_backward(dh, x, gate, h, None, None, dh_last, dx, dgate, dh0, B, T,
                                        D, dtype, None)


def test_scan_refusals():
    for size in (dict(B=0), dict(T=0), dict(D=-1), dict(B=1 << 30, T=1 << 30, D=1 << 30),
                 dict(B=1 << 40, T=1, D=1)):
        assert scan(**size) == INVALID and back(**size) == INVALID
    assert scan(dtype=7) == INVALID
    for name in ("x", "gate", "h"):
        assert scan(**{name: None}) == INVALID
    for name in ("dh", "x", "gate", "h", "dx", "dgate"):
        assert back(**{name: None}) == INVALID
    assert scan(h=fake(0)) == INVALID                # an output on an input
    assert scan(h=fake(1, 2 * 4 * 8 * 4 - 4)) == INVALID
    assert scan(last=fake(2, 16)) == INVALID         # outputs on one another
    assert scan(reset=fake(2, 8)) == INVALID
    assert back(dgate=fake(4)) == INVALID
    assert back(dh0=fake(3)) == INVALID


def step(state=fake(2), new=fake(3), h=fake(4), B=2, D=8, dtype=F32):
    return lib.rlcs_gated_step(fake(0), fake(1), None, state, new, h, B, D, dtype, None)


def test_step_refusals():
    assert step(state=None) == INVALID and step(new=None) == INVALID
    assert step(B=0) == INVALID and step(dtype=2) == INVALID
    assert step(new=fake(2, 4)) == INVALID           # neither the same states nor apart
    assert step(h=fake(3)) == INVALID


def table(cos=fake(0), sin=fake(1), n=16, R=8, base=1e4, scaling=0, factor=1.0, trained=0.0,
          slow=1.0, fast=32.0, scale=1.0):
    return lib.rlcs_rope_table(cos, sin, n, R, base, scaling, factor, trained, slow, fast, scale,
                               None)


def test_table_refusals():
    nan = float("nan")
    for bad in (dict(cos=None), dict(sin=None), dict(n=0), dict(R=7), dict(R=0), dict(base=0.0),
                dict(base=nan), dict(scaling=4), dict(scaling=1, factor=0.0), dict(scale=nan),
                dict(scaling=2, factor=2.0, R=2), dict(scaling=3, factor=2.0),
                dict(scaling=3, factor=2.0, trained=64.0, fast=1.0), dict(sin=fake(0, 4))):
        assert table(**bad) == INVALID, bad


def norm(q=fake(0), k=fake(1), qw=fake(2), kw=fake(3), cos=fake(4), sin=fake(5), pos=fake(6),
         qo=fake(7), ko=fake(8), n=4, Hq=2, Hk=1, D=8, R=8, max_pos=16, eps=1e-6, dtype=F32,
         qs=(16, 8), ks=(8, 8)):
    return lib.rlcs_qk_norm_rope(q, *qs, k, *ks, qw, kw, cos, sin, pos, qo, ko, n, Hq, Hk, D, R,
                                 max_pos, 0, eps, dtype, None)


def norm_back(scratch=fake(13), size=None, dq=fake(9), dqw=fake(11), dkw=fake(12), n=4, D=8):
    size = lib.rlcs_qk_norm_rope_scratch_bytes(D) if size is None else size
    return lib.rlcs_qk_norm_rope_backward(
        fake(7), fake(8), fake(0), 16, 8, fake(1), 8, 8, fake(2), fake(3), fake(4), fake(5),
        fake(6), dq, fake(10), dqw, dkw, n, 2, 1, D, 8, 16, 0, 1e-6, F32, scratch, size, None)


def test_norm_refusals():
    for bad in (dict(n=-1), dict(Hq=0), dict(Hk=-1), dict(D=0), dict(D=1025), dict(R=10),
                dict(R=3), dict(eps=-1.0), dict(dtype=9), dict(q=None), dict(k=None),
                dict(qw=None), dict(cos=None), dict(pos=None), dict(qo=None), dict(ko=None),
                dict(qs=(-16, 8)), dict(qo=fake(0)), dict(ko=fake(7, 8)), dict(max_pos=-1),
                dict(qo=fake(4, 4))):
        assert norm(**bad) == INVALID, bad
    assert norm(n=0, q=None) == OK                   # nothing to do
    assert lib.rlcs_qk_norm_rope_scratch_bytes(0) == 0
    assert norm_back(dqw=None) == INVALID and norm_back(dkw=None) == INVALID
    assert norm_back(dq=fake(7)) == INVALID
    assert norm_back(scratch=fake(7)) == INVALID
    assert norm_back(scratch=None, size=0) == WORKSPACE
    assert norm_back(size=64) == WORKSPACE
    assert norm_back(scratch=fake(13, 4)) == WORKSPACE


def attn(q=fake(0), k=fake(1), v=fake(2), cu=fake(3), out=fake(4), lse=fake(5), seqs=1, n=4, Hq=2,
         Hk=1, D=64, scale=0.125, dtype=BF16, qs=(128, 64), ks=(64, 64), scratch=fake(6),
         size=1 << 20):
    return lib.rlcs_attention(q, *qs, k, *ks, v, *ks, cu, out, lse, seqs, n, Hq, Hk, D, scale,
                              dtype, scratch, size, None)


def attn_back(dout=fake(7), out=fake(4), lse=fake(5), dq=fake(8), dk=fake(9), dv=fake(10), n=4,
              scratch=fake(6), size=1 << 20, qs=(128, 64)):
    return lib.rlcs_attention_backward(dout, fake(0), *qs, fake(1), 64, 64, fake(2), 64, 64, out,
                                       lse, fake(3), dq, dk, dv, 1, n, 2, 1, 64, 0.125, BF16,
                                       scratch, size, None)


def test_attention_refusals():
    for bad in (dict(n=-1), dict(seqs=-1), dict(Hq=0), dict(Hq=3, Hk=2), dict(Hk=0), dict(D=0),
                dict(D=12), dict(D=136), dict(dtype=F32), dict(scale=float("nan")), dict(q=None),
                dict(k=None), dict(v=None), dict(cu=None), dict(out=None), dict(qs=(-128, 64)),
                dict(out=fake(0)), dict(out=fake(2, 16)), dict(lse=fake(4)), dict(scratch=fake(1)),
                dict(n=1 << 31)):
        assert attn(**bad) == INVALID, bad
    for bad in (dict(qs=(132, 64)), dict(ks=(64, 60)), dict(q=fake(0, 8)), dict(out=fake(4, 2))):
        assert attn(**bad) == MISALIGNED, bad
    need = lib.rlcs_attention_scratch_bytes(4, 2)
    assert need >= 64 and lib.rlcs_attention_scratch_bytes(-1, 2) == 0
    for bad in (dict(scratch=None, size=0), dict(size=need - 1), dict(scratch=fake(6, 8))):
        assert attn(**bad) == WORKSPACE, bad
    assert attn(n=0, q=None) == OK and attn(seqs=0, q=None) == OK
    for bad in (dict(dout=None), dict(out=None), dict(lse=None), dict(dq=None), dict(dk=None),
                dict(dv=None), dict(dk=fake(9), dv=fake(9)), dict(dq=fake(7)),
                dict(scratch=fake(5))):
        assert attn_back(**bad) == INVALID, bad
    assert attn_back(dout=fake(7, 2)) == MISALIGNED and attn_back(qs=(128, 68)) == MISALIGNED
    assert attn_back(size=8) == WORKSPACE
    assert attn_back(n=0) == OK


def attn_step(q=fake(0), k=fake(1), v=fake(2), lens=fake(3), out=fake(4), B=2, S=16, Hq=2, Hk=1,
              D=64, ks=(1024, 64, 64), dtype=BF16, scratch=fake(5), size=1 << 24):
    return lib.rlcs_attention_step(q, k, *ks, v, *ks, lens, out, B, S, Hq, Hk, D, 0.125, dtype,
                                   scratch, size, None)


def test_attention_step_refusals():
    for bad in (dict(B=-1), dict(S=-1), dict(Hq=3, Hk=2), dict(D=20), dict(dtype=F32),
                dict(q=None), dict(k=None), dict(v=None), dict(lens=None), dict(out=None),
                dict(ks=(-1024, 64, 64)), dict(out=fake(0)), dict(out=fake(1, 32)),
                dict(scratch=fake(2))):
        assert attn_step(**bad) == INVALID, bad
    for bad in (dict(ks=(1028, 64, 64)), dict(ks=(1024, 60, 64)), dict(k=fake(1, 2)),
                dict(q=fake(0, 4))):
        assert attn_step(**bad) == MISALIGNED, bad
    assert attn_step(scratch=None, size=0) == WORKSPACE
    assert attn_step(B=0, q=None) == OK


def test_binding_refuses_host_tensors_and_wrong_kinds():
    x = torch.zeros(2, 3, 4)
    for call in (lambda: sequence.rlcs_gated_scan(x, x),
                 lambda: sequence.rlcs_gated_scan_backward(x, x, x, x),
                 lambda: sequence.rlcs_gated_step(x[0], x[0], x[0]),
                 lambda: sequence.rlcs_attention(x, x, x, torch.zeros(2, dtype=torch.int32)),
                 lambda: sequence.rlcs_attention_step(x, x, x, x),
                 lambda: sequence.rlcs_qk_norm_rope(x, x, x, x, x, x, x)):
        with pytest.raises((ValueError, TypeError)):
            call()
    with pytest.raises(ValueError):
        sequence.rlcs_rope_table(4, 4, scaling="none such")


def test_attention_scale_range():
    # scale * log2(e) is held in float32: outside this range it would be zero,
    # subnormal or infinite
    for scale in (0.0, -0.125, 1e-31, 1e-320, 1e31, 3e38, float("inf"), float("nan")):
        assert attn(scale=scale) == INVALID, scale
