"""A workspace that a call allocates for itself belongs to the stream the call runs on.

torch's allocator hands out a block while the last kernels that use it are still queued on the
stream it was allocated for, so a block taken on the current stream and used on another would be
written by both at once.  On the CPU every entry point is called with stand-ins for the library
and the allocator; on the GPU a freed block of the current stream is the bait.
"""
import contextlib
import types

import pytest
import torch

import kernelized_linear_attention_unit_b200.binding as bd

B, H, L, R, m = 1, 2, 8, 2, 4
F = R * m
x, s, z, d = torch.zeros(B, H, L, 64), torch.zeros(B, H, F, 64), torch.zeros(B, H, F), torch.zeros(B, H, L)
ph, ld = torch.zeros(B, H, L, F), torch.zeros(H)
KEY = (R, m, 1, 1e-6)
CALLS = {
    "slay_attn_causal_fwd": lambda **k: bd.slay_attn_causal_fwd(x, x, x, x, d, *KEY, **k),
    "slay_attn_bidir_fwd": lambda **k: bd.slay_attn_bidir_fwd(x, x, x, x, d, *KEY, **k),
    "slay_attn_causal_bwd": lambda **k: bd.slay_attn_causal_bwd(x, x, x, x, d, x, x, x, x, *KEY, **k),
    "slay_attn_bidir_bwd": lambda **k: bd.slay_attn_bidir_bwd(x, x, x, x, d, x, x, x, x, *KEY, **k),
    "slay_linear_attn_fwd": lambda **k: bd.slay_linear_attn_fwd(ph, ph, x, x, d, 1e-6, True, **k),
    "slay_attn_causal_fwd_state": lambda **k: bd.slay_attn_causal_fwd_state(x, x, x, x, d, *KEY, **k),
    "slay_causal_state": lambda **k: bd.slay_causal_state(x, x, s, z, *KEY, **k),
    "slay_attn_causal_fwd_begin": lambda **k: bd.slay_attn_causal_fwd_begin(x, x, s, z, *KEY, **k),
    "slay_attn_causal_bwd_state": lambda **k: bd.slay_attn_causal_bwd_state(x, x, x, x, d, x, x, x, x, *KEY, **k),
    "slay_causal_bwd_state": lambda **k: bd.slay_causal_bwd_state(x, x, d, x, s, z, *KEY, **k),
    "slay_attn_causal_bwd_begin": lambda **k: bd.slay_attn_causal_bwd_begin(x, x, d, x, s, z, *KEY, **k),
    "slay_decay_attn_fwd": lambda **k: bd.slay_decay_attn_fwd(ph, ph, x, ld, x, **k),
    "slay_decay_attn_bwd": lambda **k: bd.slay_decay_attn_bwd(ph, ph, x, ld, x, ph, ph, x, out=x, den=d, **k),
}


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("given", [True, False])
def test_block_comes_from_the_calls_stream(monkeypatch, name, given):
    current, taken = ["current"], []

    @contextlib.contextmanager
    def on(stream):
        current.append(stream)
        yield
        current.pop()

    def block(*_, **__):
        taken.append(current[-1])
        return types.SimpleNamespace(numel=lambda: 4096, element_size=lambda: 1, data_ptr=lambda: 256,
                                     record_stream=lambda stream: None)

    class Library:   # every call succeeds; any size needs 4096 bytes
        def __getattr__(self, call):
            return lambda *a: 4096 if call == "slay_workspace_bytes" else bd.SLAY_OK

    monkeypatch.setattr(bd, "lib", lambda: Library())
    monkeypatch.setattr(bd, "_check", lambda *a, **k: None)
    monkeypatch.setattr(bd, "_check_on", lambda *a, **k: None)
    monkeypatch.setattr(bd, "_stream", lambda stream=None: None)
    monkeypatch.setattr(bd, "_call_on", lambda *a: None)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch, "empty", block)
    monkeypatch.setattr(torch, "zeros", block)
    mine = types.SimpleNamespace(device=x.device, cuda_stream=0)
    CALLS[name](stream=mine if given else None)
    assert taken == [mine if given else "current"]


@pytest.mark.gpu
def test_another_streams_call_takes_no_block_of_this_one():
    Bg, Hg, Lg, Fg = 2, 4, 1500, 128
    ph, v = torch.rand(Bg, Hg, Lg, Fg, device="cuda").bfloat16(), torch.randn(Bg, Hg, Lg, 64, device="cuda").bfloat16()
    ld, out, side = torch.full((Hg,), -0.01, device="cuda"), torch.empty_like(v), torch.cuda.Stream()
    want = torch.empty_like(v)
    bait = bd.slay_decay_attn_fwd(ph, ph, v, ld, want)   # a block of this call's size, of the current stream
    at = bait.data_ptr()
    del bait
    torch.cuda.synchronize()
    ws = bd.slay_decay_attn_fwd(ph, ph, v, ld, out, stream=side)
    side.synchronize()
    assert ws.data_ptr() != at
    assert torch.equal(out, want)


def test_current_stream_without_torchs_own_shortcut(monkeypatch):
    """The handle comes from torch's public stream where its private shortcut is missing."""
    asked = []
    monkeypatch.setattr(bd, "_raw_stream", None)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev: asked.append(dev) or types.SimpleNamespace(cuda_stream=77))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    got = []
    dev = torch.device("cuda", 3)
    bd._call_on(dev, None, lambda *a: got.append(a) or bd.SLAY_OK, "call", (1, 2))
    assert asked == [dev] and got == [(1, 2, 77)]


@pytest.mark.gpu
def test_current_stream_handles_agree(monkeypatch):
    dev, side = torch.device("cuda", torch.cuda.current_device()), torch.cuda.Stream()
    for stream in (torch.cuda.current_stream(), side):
        with torch.cuda.stream(stream):
            assert bd._current_handle(dev) == stream.cuda_stream
            with monkeypatch.context() as m:
                m.setattr(bd, "_raw_stream", None)
                assert bd._current_handle(dev) == stream.cuda_stream
