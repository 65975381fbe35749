"""Refusals and sizes of the decayed attention and state-pool entry points, without a GPU:
every call here returns before any device work."""
import ctypes as C

import pytest

from kernelized_linear_attention_unit_b200 import binding as bd

P = 1 << 20            # an aligned address that no call here dereferences
OK, BAD, NO = bd.SLAY_OK, bd.SLAY_ERR_INVALID_ARG, bd.SLAY_ERR_UNSUPPORTED


def _ws(op, dt, B, H, L, F):
    return bd.slay_workspace_bytes(op, dt, B, H, L, 64, 64, 1, F)


def _fwd(**kw):
    a = dict(phq=P, phk=P, v=P, log_decay=P, lengths=None, S_in=None, z_in=None, out=P, den=P, S_out=None, z_out=None,
             B=2, H=3, L=100, F=64, Dv=64, dt=bd.SLAY_BF16, normalize=1, eps=1e-6, ws=P, ws_bytes=1 << 40, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return bd.lib().slay_decay_attn_fwd(*a.values())


def _bwd(**kw):
    a = dict(phq=P, phk=P, v=P, log_decay=P, lengths=None, S_in=None, z_in=None, out=P, den=P, dout=P, dS_out=None,
             dz_out=None, dphq=P, dphk=P, dv=P, dS_in=None, dz_in=None, B=2, H=3, L=100, F=64, Dv=64, dt=bd.SLAY_BF16,
             normalize=1, eps=1e-6, ws=P, ws_bytes=1 << 40, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return bd.lib().slay_decay_attn_bwd(*a.values())


def _decode(**kw):
    a = dict(phq=P, phk=P, v=P, log_decay=P, S=P, z=P, slots=P, out=P, Bt=2, H=3, F=64, Dv=64, n_slots=4,
             dt=bd.SLAY_BF16, normalize=1, eps=1e-6, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return bd.lib().slay_decay_decode_step(*a.values())


def _copy(**kw):
    a = dict(S_src=P, z_src=P, src=P, n_src=4, S_dst=P, z_dst=P, dst=P, n_dst=4, n=2, H=3, F=64, Dv=64, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return bd.lib().slay_state_copy(*a.values())


SIZES = [(dict(B=-1), BAD), (dict(L=-1), BAD), (dict(F=0), BAD), (dict(F=1025), NO), (dict(Dv=128), NO), (dict(dt=2), BAD),
         (dict(eps=0.0), BAD), (dict(eps=float("nan")), BAD), (dict(B=22000, H=1), NO), (dict(log_decay=None), BAD),
         (dict(log_decay=P + 2), BAD), (dict(lengths=P + 1), BAD), (dict(phq=None), BAD), (dict(phk=P + 8), BAD),
         (dict(v=None), BAD), (dict(S_in=P), BAD), (dict(z_in=P), BAD), (dict(S_in=P, z_in=P + 4), BAD),
         (dict(S_in=P, z_in=P, normalize=0, den=None), BAD), (dict(ws=None), BAD), (dict(ws=P + 128), BAD),
         (dict(ws_bytes=100), BAD), (dict(B=0), OK), (dict(H=0), OK), (dict(L=0), OK)]


@pytest.mark.parametrize("kw,want", SIZES + [(dict(out=None), BAD), (dict(den=P + 1), BAD), (dict(normalize=0), BAD),
                                             (dict(S_out=P), BAD), (dict(z_out=P), BAD)])
def test_forward_refusals(kw, want):
    assert _fwd(**kw) == want


@pytest.mark.parametrize("kw,want", [s for s in SIZES if s[0].get("den", 0) is not None] + [
    (dict(out=None), BAD), (dict(den=None), BAD), (dict(dout=None), BAD), (dict(dphq=None), BAD), (dict(dphk=P + 8), BAD),
    (dict(dv=None), BAD), (dict(dS_out=P), BAD), (dict(dz_out=P), BAD), (dict(dS_in=P), BAD),
    (dict(dS_in=P, dz_in=P, normalize=0), BAD)])
def test_backward_refusals(kw, want):
    assert _bwd(**kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(Bt=-1), BAD), (dict(F=0), BAD), (dict(F=1025), NO), (dict(Dv=32), NO), (dict(dt=7), BAD), (dict(eps=-1.0), BAD),
    (dict(n_slots=-1), BAD), (dict(slots=None, Bt=5), BAD), (dict(slots=P + 2), BAD), (dict(log_decay=None), BAD),
    (dict(phq=None), BAD), (dict(phk=P + 4), BAD), (dict(v=None), BAD), (dict(out=None), BAD), (dict(S=None), BAD),
    (dict(z=None), BAD), (dict(normalize=0), BAD), (dict(S=P + 4), BAD), (dict(Bt=0), OK), (dict(H=0), OK)])
def test_decode_refusals(kw, want):
    assert _decode(**kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(n=-1), BAD), (dict(n=4097), NO), (dict(H=0), BAD), (dict(F=1025), NO), (dict(Dv=65), NO), (dict(n_src=-1), BAD),
    (dict(src=None), BAD), (dict(dst=P + 1), BAD), (dict(S_src=None), BAD), (dict(S_dst=P + 8), BAD), (dict(z_src=None), BAD),
    (dict(z_dst=None), BAD), (dict(S_dst=P + 3 * 64 * 64 * 4), BAD),        # a pool that starts inside the other
    (dict(z_dst=P + 3 * 64 * 4), BAD), (dict(n=0), OK), (dict(n_dst=0), OK)])
def test_copy_refusals(kw, want):
    assert _copy(**kw) == want


def test_workspace_sizes():
    for op in (bd.OP_DECAY_FWD, bd.OP_DECAY_BWD):
        for dt in (bd.SLAY_F32, bd.SLAY_BF16):
            a, b = _ws(op, dt, 1, 2, 1000, 256), _ws(op, dt, 1, 2, 4000, 256)
            assert 0 < a <= b and a % 256 == 0
        assert _ws(op, bd.SLAY_BF16, 1, 2, 0, 256) == 0
        with pytest.raises(bd.SlayError):
            _ws(op, bd.SLAY_BF16, 1, 2, 100, 1025)
    # one block short is refused, whatever the pointers
    need = _ws(bd.OP_DECAY_FWD, bd.SLAY_BF16, 2, 3, 100, 64)
    assert _fwd(ws_bytes=need - 256) == BAD
    need = _ws(bd.OP_DECAY_BWD, bd.SLAY_BF16, 2, 3, 100, 64)
    assert _bwd(ws_bytes=need - 256) == BAD


@pytest.mark.parametrize("dt,F,want", [("BF16", 256, 2), ("BF16", 8, 2), ("BF16", 512, 2), ("BF16", 520, 0), ("BF16", 100, 0),
                                       ("F32", 256, 0)])
def test_path(dt, F, want):
    for op in (bd.OP_DECAY_FWD, bd.OP_DECAY_BWD):
        assert bd.slay_path(op, getattr(bd, "SLAY_" + dt), 1, 2, 100, 64, 64, 1, F) == want
        assert bd.slay_path(op, getattr(bd, "SLAY_" + dt), 0, 2, 100, 64, 64, 1, F) == 0
    with pytest.raises(bd.SlayError):
        bd.slay_path(bd.OP_DECAY_FWD, bd.SLAY_BF16, 1, 2, 100, 64, 32, 1, F)


def test_binding_checks():
    import torch
    x = torch.zeros(1, 1, 4, 8)
    with pytest.raises(ValueError):
        bd.slay_decay_attn_fwd(x, x, x, torch.zeros(1), x)            # not on a GPU
    with pytest.raises(ValueError):
        bd.slay_decay_decode_step(x, x, x, torch.zeros(1), x, None, x)
    with pytest.raises(ValueError):
        bd.slay_state_copy(x, None, None, x, None, None)
    assert C.sizeof(C.c_void_p) == 8
