"""Ways through the decayed calls that depend on how a sequence is cut, against the fp64
definition: a few segments whose sums the sweeps add up themselves, a state updated in place
while other segments still read it, a sequence run in pieces; the limbs that the sums and the
normalized dphq are made of; the calls between the feature map and its backward; gradients on
two streams at once.  Tolerances as in test_decay_gpu, but where a test says otherwise."""
import contextlib
import math

import numpy as np
import pytest
import torch

import decay_reference as ref
import oracle as O
import test_decay_gpu as base
from kernelized_linear_attention_unit_b200 import binding as bd
from kernelized_linear_attention_unit_b200 import workloads as W
from parity_check import check

gpu = pytest.mark.gpu


@contextlib.contextmanager
def _launches():
    """The names of the library's launches inside the block, once it is left."""
    names = []
    bd.slay_trace_enable(True)
    try:
        bd.slay_trace_read()
        yield names
        torch.cuda.synchronize()
        names.extend(n for n, _ in bd.slay_trace_read())
    finally:
        bd.slay_trace_enable(False)


def _summed(names):
    return "tc_decay_state" in names and "decay_seg_scan" not in names


# two to four segments and no state carried in: no scan between the segments' sums and the sweeps
@gpu
@pytest.mark.parametrize("B,H,L,F,norm,ragged", [
    (4, 9, 900, 320, True, True), (40, 1, 1100, 256, True, False), (10, 1, 512, 512, False, False), (8, 4, 1000, 128, False, True),
    (4, 8, 1100, 64, True, True)])
def test_forward_sums_of_few_segments(B, H, L, F, norm, ragged):
    with _launches() as names:
        base.test_forward(B, H, L, F, "bf16", norm, ragged, False)
    assert _summed(names), names


# the reverse walk of dphk and dv: four segments in two launches of dv's features, two in one launch of all sweeps
@gpu
@pytest.mark.parametrize("B,H,L,F,norm,ragged", [
    (4, 9, 900, 320, True, True), (4, 9, 900, 320, False, False), (10, 1, 512, 512, False, False), (12, 1, 400, 320, True, True)])
def test_backward_sums_of_few_segments(B, H, L, F, norm, ragged):
    with _launches() as names:
        base.test_backward(B, H, L, F, "bf16", norm, ragged, False)
    assert _summed(names), names


# two segments and a carried state: the sweeps add it up, so one that is updated in place is read from a copy
@gpu
@pytest.mark.parametrize("norm,ragged", [(True, False), (True, True), (False, False)])
def test_forward_state_in_place_of_two_segments(norm, ragged):
    B, H, L, F = 40, 1, 512, 64
    c, _ = base._case(B, H, L, F, "bf16", norm, ragged, True, seed=31, kind="slow")
    want, mag = ref.forward(**c)
    apart = base._forward(c, "bf16")
    for _ in range(4):
        with _launches() as names:
            here = base._forward(c, "bf16", inplace=True)
        assert _summed(names), names
        assert all(x is None or torch.equal(x, y) for x, y in zip(apart, here))
    base._ok("out", base._valid_only(here[0], c["lengths"]), want["out"], mag["out"], "bf16", L + F)
    base._ok("S_out", here[2], want["S_out"], mag["S_out"], "bf16", L)
    if norm:
        base._ok("z_out", here[3], want["z_out"], mag["z_out"], "bf16", L)


@gpu
@pytest.mark.parametrize("B,L,F,norm,ragged", [(10, 512, 512, False, False), (10, 400, 320, True, True)])
def test_backward_state_in_place_of_two_segments(B, L, F, norm, ragged):
    c, g = base._case(B, 1, L, F, "bf16", norm, ragged, True, seed=32, kind="slow")
    c["dout"] = base._randn(g, B, 1, L, 64).bfloat16()
    fwd, _ = ref.forward(**{k: x for k, x in c.items() if k != "dout"})
    c["out"], c["den"] = (fwd["out"].bfloat16(), fwd["den"].float()) if norm else (torch.zeros_like(c["v"]), torch.ones(B, 1, L, device="cuda"))
    dS, dz = base._randn(g, B, 1, F, 64), base._randn(g, B, 1, F) if norm else None
    want, mag = ref.backward(**c, dS_out=dS, dz_out=dz)
    if not norm:
        c["out"] = c["den"] = None

    def run(in_place):
        got = {k: torch.full_like(c[x], base.MARK) for k, x in (("dphq", "phq"), ("dphk", "phk"), ("dv", "v"))}
        dS_out, dz_out = dS.clone(), dz.clone() if norm else None
        got["dS_in"] = dS_out if in_place else torch.empty_like(dS)
        got["dz_in"] = None if not norm else dz_out if in_place else torch.empty_like(dz)
        bd.slay_kernel_status(bd.slay_decay_attn_bwd(**c, **got, dS_out=dS_out, dz_out=dz_out))
        return {k: x for k, x in got.items() if x is not None}

    apart = run(False)
    for _ in range(4):
        with _launches() as names:
            here = run(True)
        assert _summed(names), names
        assert all(torch.equal(apart[k], here[k]) for k in apart)
    for k, x in here.items():
        base._ok(k, x if k[-3:] == "_in" else base._valid_only(x, c["lengths"]), want[k], mag[k], "bf16", L + F)


# ------------------------------------------------------------------------------ limbs
# One rounding to bf16 is off by at most 2^-8 of a value, evenly spread: an rms of at most 2^-8 / sqrt(3) = 2.26e-3.
# Two limbs of the scores and of the state add 2^-16 to that; 2% more than covers them and the fp32 sums.
ONE_ROUNDING = 1.02 * 2.0 ** -8 / math.sqrt(3.0)


def sum_bar(L):
    """Relative L2 of a cut sequence's state: the products of a 128-token chunk are added in eight
    steps and the chunks one by one, each addition off by at most 2^-23 of its partial sum; the
    weights' third limb leaves 2^-24."""
    return (8 + -(-L // 128)) * 2.0 ** -23


LIMBS = [(5, 4, 600, 256, -1.0 / 512), (2, 3, 300, 128, -1.0 / 64), (1, 2, 700, 320, -1.0 / 512)]
SUMS = [(40, 1, 512, 64, False), (1, 4, 640, 256, True), (4, 8, 512, 128, False)]   # B, H, L, F, whether a scan joins the segments


def _limbs(x, n):
    got = torch.zeros_like(x)
    x = x.float().double()
    for _ in range(n):
        part = x.to(torch.bfloat16).double()
        got, x = got + part, x - part
    return got


@pytest.mark.parametrize("B,H,L,F,g", LIMBS)
def test_bar_of_dphq_tells_one_limb_from_two(B, H, L, F, g):
    """The definition with the scores and the state of each chunk rounded to one limb, and to two."""
    gen = torch.Generator().manual_seed(7)
    new = lambda *s: torch.randn(*s, generator=gen).bfloat16().double()  # noqa: E731
    q, k = (torch.exp(0.7 * new(L, F)).div(F ** 0.5).bfloat16().double() for _ in range(2))
    v, do = new(L, 64), new(L, 64)
    t = torch.arange(L)
    Wd = torch.tril(torch.exp(g * (t[:, None] - t).clamp(min=0).double()))
    A = (q @ k.T) * Wd
    rz = 1.0 / (A.sum(-1) + 1e-3)
    r = ((A @ v * rz[:, None]).bfloat16().double() * do).sum(-1)
    scores = (do @ v.T - r[:, None]) * rz[:, None] * Wd
    want = scores @ k
    err = []
    for n in (1, 2):
        got = torch.zeros_like(want)
        for a in range(0, L, 128):
            s, before = slice(a, min(a + 128, L)), slice(0, a)
            w = torch.exp(g * (a - 1 - t[before]).double())[:, None] * k[before]
            up = (torch.exp(g * (t[s] + 1 - a).double()) * rz[s])[:, None]
            got[s] = _limbs(scores[s, s], n) @ k[s] + up * (do[s] @ _limbs(w.T @ v[before], n).T - r[s, None] * w.sum(0))
        err.append(float((got.bfloat16().double() - want).norm() / want.norm()))
    assert err[0] > ONE_ROUNDING > err[1], err


@pytest.mark.parametrize("B,H,L,F,scan", SUMS)
def test_bar_of_the_sums_tells_two_limbs_from_three(B, H, L, F, scan):
    gen = torch.Generator().manual_seed(8)
    k = torch.exp(0.7 * torch.randn(L, F, generator=gen)).div(F ** 0.5).bfloat16().double()
    v = torch.randn(L, 64, generator=gen).bfloat16().double()
    for g in (-1.0 / 512, -1.0 / 64):
        to_end = torch.arange(L - 1, -1, -1)
        chunk = torch.exp(g * (to_end % 128).double())[:, None]
        rest = torch.exp(g * (to_end // 128 * 128).double())[:, None]
        want = (rest * chunk * k).T @ v
        err = [float(((rest * k).T @ _limbs(chunk * v, n) - want).norm() / want.norm()) for n in (2, 3)]
        assert err[0] > sum_bar(L) > 10 * err[1], err


@gpu
@pytest.mark.parametrize("B,H,L,F,g", LIMBS)
def test_normalized_dphq_is_off_by_its_own_rounding(B, H, L, F, g):
    c, gen = base._case(B, H, L, F, "bf16", True, False, False, seed=33)
    c["log_decay"] = torch.full((H,), g, device="cuda")
    c["dout"] = base._randn(gen, B, H, L, 64).bfloat16()
    out, den, _, _ = base._forward({k: x for k, x in c.items() if k != "dout"}, "bf16")
    c["out"], c["den"] = out, den
    want, _ = ref.backward(**c)
    got = {k: torch.empty_like(c[x]) for k, x in (("dphq", "phq"), ("dphk", "phk"), ("dv", "v"))}
    bd.slay_decay_attn_bwd(**c, **got)
    rel = float((got["dphq"].double() - want["dphq"]).norm() / want["dphq"].norm())
    assert rel <= ONE_ROUNDING, rel


@gpu
@pytest.mark.parametrize("B,H,L,F,scan", SUMS)
def test_state_of_a_cut_sequence_keeps_three_limbs(B, H, L, F, scan):
    c, _ = base._case(B, H, L, F, "bf16", True, False, False, seed=34, kind="slow")
    want, _ = ref.forward(**c)
    with _launches() as names:
        _, _, S, z = base._forward(c, "bf16")
    assert "tc_decay_state" in names and ("decay_seg_scan" in names) == scan, names
    for got, k in ((S, "S_out"), (z, "z_out")):
        rel = float((got.double() - want[k]).norm() / want[k].norm())
        assert rel <= sum_bar(L), (k, rel)


# ----------------------------------------------------------------------------- pieces
@gpu
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("cuts", [(77,), (128, 1), (300, 211)])
def test_a_sequence_in_pieces(dt, norm, cuts):
    """Forwards joined by their states, the state updated in place, are one forward."""
    B, H, L, F = 2, 3, 640, 128
    c, _ = base._case(B, H, L, F, dt, norm, False, True, seed=35, kind="slow")
    want, mag = ref.forward(**c)
    S, z = c["S_in"].clone(), c["z_in"].clone() if norm else None
    outs, dens, at = [], [], 0
    for n in (*cuts, L - sum(cuts)):
        part = [c[k][:, :, at:at + n].contiguous() for k in ("phq", "phk", "v")]
        out = torch.empty_like(part[2])
        den = torch.empty(B, H, n, device="cuda") if norm else None
        bd.slay_decay_attn_fwd(*part, c["log_decay"], out, den=den, normalize=norm, eps=c["eps"], S_in=S, z_in=z, S_out=S, z_out=z)
        outs.append(out)
        dens.append(den)
        at += n
    base._ok("out", torch.cat(outs, 2), want["out"], mag["out"], dt, L + F)
    base._ok("S_out", S, want["S_out"], mag["S_out"], dt, L)
    if norm:
        base._ok("den", torch.cat(dens, 2), want["den"], mag["den"], dt, L + F)
        base._ok("z_out", z, want["z_out"], mag["z_out"], dt, L)


# -------------------------------------------------------- between the feature map's calls
@gpu
@pytest.mark.parametrize("dt,tol", [("bf16", 1.5e-2), ("f32", 1e-5)])
def test_feature_map_to_its_backward(dt, tol):
    """Features of the library's map through the decayed forward and backward into the map's
    backward; each step against its definition on the values that it was given."""
    w = W.Workload("decay chain", B=2, H=2, L=300, R=4, m=64, dtype=dt, data_seed=61)
    q, k, v = W.gen_qkv(w)
    key = (w.R, w.m, w.sketch_seed, float(np.float32(w.eps)))
    P = O.sketch_params(w.D, *key)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.float32)).cuda().to(base.TDT[dt])  # noqa: E731
    host = lambda t: t.double().cpu().numpy()  # noqa: E731
    x = {"phq": dev(q), "phk": dev(k)}
    c = {"v": dev(v), "log_decay": base._decays(w.H, "slow"), "normalize": True, "eps": key[3]}
    for name in x:
        c[name] = torch.empty(w.B, w.H, w.L, w.F, device="cuda", dtype=base.TDT[dt])
        bd.slay_feature_map(x[name], c[name], *key)
        check("decay chain %s %s" % (dt, name), host(c[name]), O.feature_map(host(x[name]), P), tol)
    out, den = torch.empty_like(c["v"]), torch.empty(w.B, w.H, w.L, device="cuda")
    bd.slay_decay_attn_fwd(out=out, den=den, **c)
    want, mag = ref.forward(**c)
    base._ok("out", out, want["out"], mag["out"], dt, w.L + w.F)
    c["dout"] = dev(W.gen_dout(w))
    got = {"d" + name: torch.empty_like(c[name]) for name in ("phq", "phk", "v")}
    bd.slay_decay_attn_bwd(**c, **got, out=out, den=den)
    want, mag = ref.backward(**c, out=out, den=den)
    for name in got:
        base._ok(name, got[name], want[name], mag[name], dt, w.L + w.F)
    for name in x:
        dx = torch.empty(x[name].shape, device="cuda")
        bd.slay_feature_map_bwd(x[name], got["d" + name], dx, *key)
        check("decay chain %s d%s" % (dt, name), host(dx), O.feature_map_bwd(host(x[name]), host(got["d" + name]), P), tol)


# ---------------------------------------------------------------------------- streams
@gpu
def test_gradients_on_two_streams_with_blocks_of_their_own():
    """Calls in flight on two streams, each allocating its workspace, while this stream frees blocks of that size."""
    shape = (2, 4, 1500, 128)
    calls = []
    for seed in (41, 42):
        c, g = base._case(*shape, "bf16", True, False, True, seed=seed, kind="slow")
        fwd = base._forward(c, "bf16")
        c["out"], c["den"], c["dout"] = fwd[0], fwd[1], base._randn(g, *shape[:3], 64).bfloat16()
        calls.append(c)

    def run(c, stream):
        got = {k: torch.empty_like(c[x]) for k, x in (("dphq", "phq"), ("dphk", "phk"), ("dv", "v"))}
        bd.slay_decay_attn_bwd(**c, **got, stream=stream)
        return got

    alone = [run(c, None) for c in calls]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        both = [run(c, s) for c, s in zip(calls, streams)]
        run(calls[0], None)
        torch.cuda.synchronize()
        for a, b in zip(alone, both):
            assert all(torch.equal(a[k], b[k]) for k in a)


# ------------------------------------------------------------------------------- pool
@gpu
@pytest.mark.parametrize("with_z,F", [(True, 64), (True, 33), (False, 64)])
def test_copy_from_a_pool_of_no_slots_clears(with_z, F):
    g = base._gen(51)
    S, z = base._randn(g, 5, 2, F, 64), base._randn(g, 5, 2, F)
    S0, z0 = S.clone(), z.clone()
    i = lambda *x: torch.tensor(x, device="cuda", dtype=torch.int32)  # noqa: E731
    none_S, none_z = torch.empty(0, 2, F, 64, device="cuda"), torch.empty(0, 2, F, device="cuda")
    bd.slay_state_copy(none_S, none_z if with_z else None, i(-1, 0, -1), S, z if with_z else None, i(3, 1, 0))
    for pool, old, cleared in ((S, S0, True), (z, z0, with_z)):
        for slot in range(5):
            assert torch.equal(pool[slot], torch.zeros_like(old[slot]) if cleared and slot in (0, 3) else old[slot])


# ----------------------------------------------------------------- long and slow decays
def _slow_decay(chunk, L):
    """A decay over some 2^18 tokens whose factor of a chunk is about as far from a float as it can be."""
    g = np.float32(-3e-6) - np.arange(512, dtype=np.float32) * np.float32(1e-9)
    exact = np.exp(g.astype(np.float64) * chunk)
    off = np.abs(exact.astype(np.float32).astype(np.float64) - exact)
    return float(g[off.argmax()]), float(off.max()) * (L // chunk)


@pytest.mark.parametrize("chunk", [64, 128])
def test_a_fixed_factor_of_a_chunk_would_not_do(chunk):
    """The state of 2^18 tokens, chunk by chunk in fp64, with the chunk's factor rounded once."""
    L = 1 << 18
    g, worst = _slow_decay(chunk, L)
    own = np.exp(g * np.arange(chunk, dtype=np.float64)).sum()
    off = []
    for lam in (np.exp(g * chunk), float(np.float32(np.exp(g * chunk)))):
        off.append(own * (1.0 - lam ** (L // chunk)) / (1.0 - lam))
    assert worst > 2e-5 and abs(off[1] / off[0] - 1.0) > 1e-5, (worst, off)


@gpu
@pytest.mark.parametrize("dt,H", [("f32", 1), ("bf16", 80), ("bf16", 1)])
def test_long_slow_decays_keep_their_states(dt, H):
    """States, denominators and gradients of states over 2^18 tokens, at the bar of fp32 outputs:
    the sequence in one walk on either path, and cut."""
    L, F = 1 << 18, 8
    g, _ = _slow_decay(64 if dt == "f32" else 128, L)
    gen = base._gen(61)
    one = lambda *s: base._randn(gen, 1, 1, L, *s)  # noqa: E731
    q, k = (torch.exp(0.7 * one(F)).to(base.TDT[dt]) for _ in range(2))
    v, do = ((1.0 + one(64)).to(base.TDT[dt]) for _ in range(2))
    many = lambda x: x.expand(1, H, *x.shape[2:]).contiguous()  # noqa: E731
    ld, out, den = torch.full((H,), g, device="cuda"), torch.empty_like(many(v)), torch.empty(1, H, L, device="cuda")
    S, z = torch.empty(1, H, F, 64, device="cuda"), torch.empty(1, H, F, device="cuda")
    bd.slay_kernel_status(bd.slay_decay_attn_fwd(many(q), many(k), many(v), ld, out, den=den, S_out=S, z_out=z))
    t = torch.arange(L, device="cuda").double()
    w = torch.exp(g * (L - 1 - t))[:, None] * k[0, 0].double()
    up = torch.exp(g * (t + 1))[:, None] * q[0, 0].double()
    want = {"S_out": w.T @ v[0, 0].double(), "z_out": w.sum(0), "dS_in": up.T @ do[0, 0].double()}
    want["den"] = q[0, 0, -1].double() @ want["z_out"]
    dS = torch.empty_like(S)
    grads = [torch.empty_like(many(x)) for x in (q, k, v)]
    bd.slay_kernel_status(bd.slay_decay_attn_bwd(many(q), many(k), many(v), ld, many(do), *grads, normalize=False, dS_in=dS))
    for name, got in (("S_out", S[0, -1]), ("z_out", z[0, -1]), ("den", den[0, -1, -1]), ("dS_in", dS[0, -1])):
        rel = float((got.double() - want[name]).norm() / want[name].norm())
        assert rel <= 1e-5, (name, rel)


def _slow_step():
    """A decay over some thousand tokens whose factor of one step is about as far from a float as it can be."""
    g = np.float32(-1.0 / 1024) - np.arange(512, dtype=np.float32) * np.float32(1e-8)
    exact = np.exp(g.astype(np.float64))
    return float(g[np.abs(exact.astype(np.float32).astype(np.float64) - exact).argmax()])


def test_a_fixed_factor_of_a_step_would_not_do():
    g, n = _slow_step(), 4096
    sums = [(1.0 - lam ** n) / (1.0 - lam) for lam in (np.exp(g), float(np.float32(np.exp(g))))]
    assert abs(sums[1] / sums[0] - 1.0) > 2e-5


@gpu
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_thousands_of_decode_steps_keep_their_states(dt):
    """The states after 4096 steps, at the bar of fp32 outputs; heads without decay, with a slow one and with none left."""
    H, F, n = 4, 32, 4096
    gen = base._gen(62)
    q, k = (torch.exp(0.7 * base._randn(gen, n, 1, H, F)).to(base.TDT[dt]) for _ in range(2))
    v = (1.0 + base._randn(gen, n, 1, H, 64)).to(base.TDT[dt])
    ld = torch.tensor([0.0, _slow_step(), -0.5, -math.inf], device="cuda")
    S, z, out = torch.zeros(1, H, F, 64, device="cuda"), torch.zeros(1, H, F, device="cuda"), torch.empty_like(v[0])
    for t in range(n):
        bd.slay_decay_decode_step(q[t], k[t], v[t], ld, S, z, out, eps=1e-3)
    w = torch.stack([ref.powers(g, torch.arange(n - 1, -1, -1, device="cuda")) for g in ld])[..., None]
    kk, vv = k[:, 0].transpose(0, 1).double(), v[:, 0].transpose(0, 1).double()
    want, want_z = (w * kk).transpose(1, 2) @ vv, (w * kk).sum(1)
    for h in range(H):
        assert float((S[0, h] - want[h]).norm() / want[h].norm()) <= 1e-5, h
        assert float((z[0, h] - want_z[h]).norm() / want_z[h].norm()) <= 1e-5, h
