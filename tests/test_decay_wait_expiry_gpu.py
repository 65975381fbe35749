"""The bounded waits of the decayed sweeps, without a fault: under the library's test hook the
first CTA of each sweep of one call issues none of its loads.  The waits for them run out after
the 2 s that the header states, the call reports SLAY_ERR_TIMEOUT and leaves the context usable;
the same call again is what it was before."""
import time

import pytest
import torch

import test_decay_gpu as base
from kernelized_linear_attention_unit_b200 import binding as bd

pytestmark = pytest.mark.gpu


def _expired(call, sweeps):
    """call() runs its sweeps' waits out: 2 s each, or twice that where a thread goes from one to the next."""
    torch.cuda.synchronize()
    assert bd.lib().slay_debug_expire_wait(2) == bd.SLAY_OK
    t0 = time.monotonic()
    ws = call()
    with pytest.raises(bd.SlayError) as e:
        bd.slay_kernel_status(ws)
    assert 2.0 * sweeps - 0.1 < time.monotonic() - t0 < 5.0 * sweeps
    assert e.value.status == bd.SLAY_ERR_TIMEOUT and "bounded wait ran out" in str(e.value)


# one sweep, and one after its segments' sums
@pytest.mark.parametrize("B,H,L,F,norm,sweeps", [(2, 2, 200, 128, True, 1), (8, 4, 1000, 128, False, 2)])
def test_forward(B, H, L, F, norm, sweeps):
    c, _ = base._case(B, H, L, F, "bf16", norm, False, False)
    out = torch.empty_like(c["v"])
    bd.slay_kernel_status(bd.slay_decay_attn_fwd(out=out, **c))
    _expired(lambda: bd.slay_decay_attn_fwd(out=torch.empty_like(out), **c), sweeps)
    again = torch.empty_like(out)
    bd.slay_kernel_status(bd.slay_decay_attn_fwd(out=again, **c))
    assert torch.equal(out, again)


# the sweeps side by side, and one after the other
@pytest.mark.parametrize("B,H,L,F,norm,sweeps", [(2, 2, 200, 128, True, 1), (100, 1, 400, 64, True, 3)])
def test_backward(B, H, L, F, norm, sweeps):
    c, g = base._case(B, H, L, F, "bf16", norm, False, False)
    out, den, _, _ = base._forward(c, "bf16")
    c["dout"] = base._randn(g, B, H, L, 64).bfloat16()
    if norm:
        c["out"], c["den"] = out, den

    def call():
        got = {k: torch.empty_like(c[x]) for k, x in (("dphq", "phq"), ("dphk", "phk"), ("dv", "v"))}
        return got, bd.slay_decay_attn_bwd(**c, **got)

    want, ws = call()
    bd.slay_kernel_status(ws)
    _expired(lambda: call()[1], sweeps)
    got, ws = call()
    bd.slay_kernel_status(ws)
    assert all(torch.equal(want[k], got[k]) for k in want)


def test_disarmed():
    c, _ = base._case(1, 1, 100, 64, "bf16", True, False, False)
    bd.lib().slay_debug_expire_wait(2)
    bd.lib().slay_debug_expire_wait(0)
    bd.slay_kernel_status(bd.slay_decay_attn_fwd(out=torch.empty_like(c["v"]), **c))
