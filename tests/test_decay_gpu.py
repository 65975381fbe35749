"""Decayed linear attention and the state pool on the GPU against their definition in fp64.

Tolerances.  u is the output type's half step (2^-8 bf16, 2^-24 fp32).
  - Every element: |got - want| <= k u M, M the sum of the absolute terms of the value.  In
    bf16 mode a value sees at most four roundings to bf16 (the score, the state's operand, the
    weighted row that enters the state, the output), so k = 4; den and the states are fp32 sums of exact
    products of bf16 values whose weights are split into three bf16 limbs (8 bits each: 2^-24),
    at most n + F terms added in fp32 and two exponentials, 2^-22 relative each: 16 u sqrt(n) with u = 2^-24
    covers them for the lengths here (n <= 2049: 2^-24 * 16 * 45 = 4.3e-5 of M).  In fp32 mode
    the same 16 u sqrt(n).
  - Whole tensors of more than a few tokens, relative L2: independent roundings of at most a
    half step have an rms of u / sqrt(3); four of them 2 u / sqrt(3) < 1.2 u -> 1.5 u in bf16;
    1e-5 for fp32 outputs, the library's bar.
"""
import concurrent.futures
import math

import pytest
import torch

import decay_reference as ref
from kernelized_linear_attention_unit_b200 import binding as bd

pytestmark = pytest.mark.gpu
TDT = {"f32": torch.float32, "bf16": torch.bfloat16}
U = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
MARK = 7.5     # what rows that must not be written hold


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _decays(H, kind="mixed"):
    lists = {"mixed": [-0.01, 0.0, -0.3, -math.inf, -2.5, -1e-3], "none": [0.0], "slow": [-1.0 / 512, -1.0 / 64]}[kind]
    return torch.tensor([lists[h % len(lists)] for h in range(H)], device="cuda")


def _features(g, dt, norm, *shape):
    x = _randn(g, *shape)
    x = torch.exp(0.7 * x) if norm else x
    return (x / shape[-1] ** 0.5).to(TDT[dt])


def _case(B, H, L, F, dt, norm, ragged, state, seed=0, kind="mixed"):
    g = _gen(seed)
    c = {"phq": _features(g, dt, norm, B, H, L, F), "phk": _features(g, dt, norm, B, H, L, F),
         "v": _randn(g, B, H, L, 64).to(TDT[dt]), "log_decay": _decays(H, kind), "normalize": norm, "eps": 1e-3,
         "lengths": None, "S_in": None, "z_in": None}
    if ragged:
        n = [L, 0, 1, L // 2, max(L - 1, 0), L // 3 + 1, 200000, -3]
        c["lengths"] = torch.tensor([n[b % len(n)] for b in range(B)], device="cuda", dtype=torch.int32)
    if state:
        c["S_in"] = _randn(g, B, H, F, 64)
        c["z_in"] = torch.exp(_randn(g, B, H, F)) if norm else None
    return c, g


def _poison(c, *names):
    """NaN and infinities in the rows behind each sequence."""
    if c["lengths"] is None:
        return
    for b, n in enumerate(c["lengths"].tolist()):
        n = min(max(n, 0), c["v"].shape[2])
        for k in names:
            c[k][b, :, n:] = float("nan")
            c[k][b, :, n::2] = float("inf")


def _ok(name, got, want, mag, dt, n, l2=True):
    got = got.double()
    assert torch.isfinite(got).all(), name
    low = dt == "bf16" and name not in ("den", "S_out", "z_out", "dS_in", "dz_in")
    k = 4 * U["bf16"] if low else 16 * U["f32"] * math.sqrt(max(n, 1))
    err = (got - want).abs()
    assert (err <= k * mag + 1e-30).all(), (name, float((err / (mag + 1e-30)).max()) / k)
    if l2 and float(want.norm()) > 0:
        rel = float((got - want).norm() / want.norm())
        assert rel <= (1.5 * U["bf16"] if low else 1e-5), (name, rel)


def _untouched(x, lengths):
    if lengths is None:
        return
    for b, n in enumerate(lengths.tolist()):
        assert (x[b, :, min(max(n, 0), x.shape[2]):] == MARK).all()


def _valid_only(x, lengths):
    if lengths is None:
        return x
    x = x.clone()
    for b, n in enumerate(lengths.tolist()):
        x[b, :, min(max(n, 0), x.shape[2]):] = 0
    return x


SHAPES = [  # B, H, L, F, dtype, normalize, ragged, state
    (1, 1, 1, 64, "bf16", True, False, False),
    (1, 2, 1, 40, "f32", True, False, True),
    (3, 2, 70, 8, "bf16", True, True, True),
    (1, 1, 129, 1, "bf16", False, False, True),
    (1, 2, 90, 1024, "bf16", True, False, True),
    (2, 3, 2, 128, "bf16", False, False, True),
    (2, 6, 63, 64, "bf16", True, False, True),
    (1, 6, 64, 33, "f32", True, False, True),
    (2, 2, 65, 96, "f32", False, False, False),
    (1, 6, 127, 256, "bf16", True, False, True),
    (2, 3, 128, 64, "bf16", False, False, True),
    (1, 6, 129, 128, "bf16", True, False, True),
    (1, 2, 200, 200, "bf16", True, False, False),
    (1, 2, 257, 30, "bf16", True, False, True),
    (2, 2, 300, 320, "bf16", True, False, True),
    (1, 3, 300, 512, "bf16", False, False, True),
    (1, 2, 130, 600, "bf16", True, False, False),
    (8, 3, 300, 128, "bf16", True, True, True),
    (8, 2, 200, 72, "bf16", False, True, True),
    (8, 2, 150, 72, "f32", True, True, True),
    (8, 1, 513, 256, "bf16", True, True, False),
    (1, 2, 2049, 256, "bf16", True, False, True),
    (1, 2, 2048, 64, "bf16", False, False, False),
    (1, 2, 2000, 512, "bf16", True, False, True),
    (1, 1, 1500, 256, "f32", False, False, True),
    (160, 1, 140, 64, "bf16", True, False, True),
    # segments of several chunks (the sequences cut in three, four and eight)
    (40, 1, 1100, 256, "bf16", True, False, True),
    (37, 1, 1000, 128, "bf16", False, True, True),
    (4, 9, 900, 320, "bf16", True, True, True),
    (2, 9, 3000, 64, "bf16", True, False, True),
]


def _forward(c, dt, den=True, state_out=True, inplace=False):
    B, H, L, F = c["phq"].shape
    out = torch.full((B, H, L, 64), MARK, device="cuda", dtype=TDT[dt])
    d = torch.full((B, H, L), MARK, device="cuda") if c["normalize"] and den else None
    S = z = None
    if state_out:
        S = c["S_in"].clone() if inplace else torch.full((B, H, F, 64), MARK, device="cuda")
        if c["normalize"]:
            z = c["z_in"].clone() if inplace else torch.full((B, H, F), MARK, device="cuda")
    kw = dict(c)
    if inplace:
        kw["S_in"], kw["z_in"] = S, z
    ws = bd.slay_decay_attn_fwd(out=out, den=d, S_out=S, z_out=z, **kw)
    bd.slay_kernel_status(ws)
    return out, d, S, z


@pytest.mark.parametrize("B,H,L,F,dt,norm,ragged,state", SHAPES)
def test_forward(B, H, L, F, dt, norm, ragged, state):
    c, _ = _case(B, H, L, F, dt, norm, ragged, state)
    want, mag = ref.forward(**c)
    _poison(c, "phq", "phk", "v")
    out, den, S, z = _forward(c, dt)
    l2 = L > 16
    _untouched(out, c["lengths"])
    _ok("out", _valid_only(out, c["lengths"]), want["out"], mag["out"], dt, L + F, l2)
    _ok("S_out", S, want["S_out"], mag["S_out"], dt, L, l2)
    if norm:
        _untouched(den, c["lengths"])
        _ok("den", _valid_only(den, c["lengths"]), want["den"], mag["den"], dt, L + F, l2)
        _ok("z_out", z, want["z_out"], mag["z_out"], dt, L, l2)


@pytest.mark.parametrize("B,H,L,F,dt,norm,ragged,state", SHAPES)
def test_backward(B, H, L, F, dt, norm, ragged, state):
    c, g = _case(B, H, L, F, dt, norm, ragged, state, seed=1)
    c["dout"] = _randn(g, B, H, L, 64).to(TDT[dt])
    fwd, _ = ref.forward(**{k: x for k, x in c.items() if k != "dout"})
    c["out"], c["den"] = fwd["out"].to(TDT[dt]), fwd["den"].float()
    c["dS_out"] = _randn(g, B, H, F, 64) if state else None
    c["dz_out"] = _randn(g, B, H, F) if state and norm else None
    want, mag = ref.backward(**c)
    _poison(c, "phq", "phk", "v", "dout", "out", "den")
    new = lambda x: torch.full_like(x, MARK)  # noqa: E731
    got = {"dphq": new(c["phq"]), "dphk": new(c["phk"]), "dv": new(c["v"]),
           "dS_in": torch.full((B, H, F, 64), MARK, device="cuda"),
           "dz_in": torch.full((B, H, F), MARK, device="cuda") if norm else None}
    if not norm:
        c["out"] = c["den"] = None
    ws = bd.slay_decay_attn_bwd(**c, **got)
    bd.slay_kernel_status(ws)
    for k in ("dphq", "dphk", "dv"):
        _untouched(got[k], c["lengths"])
        # a first token's normalized gradient of its own scores cancels exactly: elementwise only
        _ok(k, _valid_only(got[k], c["lengths"]), want[k], mag[k], dt, L + F, L > 16)
    for k in ("dS_in", "dz_in"):
        if got[k] is not None:
            _ok(k, got[k], want[k], mag[k], dt, L, L > 16 and not (norm and dt == "f32"))


# CUDA cores: half chunks and whole ones a block, one and several blocks of features, grouped and not
@pytest.mark.parametrize("B,H,L,F,dt,norm,ragged,state", [
    (8, 3, 700, 96, "f32", True, True, True), (8, 3, 500, 36, "f32", False, True, True),
    (1, 2, 1000, 200, "f32", True, False, True), (1, 1, 200, 64, "f32", True, False, True),
    (1, 1, 97, 130, "bf16", True, False, True), (3, 5, 400, 70, "bf16", False, True, True)])
def test_cuda_cores_few_and_many_chunks(B, H, L, F, dt, norm, ragged, state):
    test_forward(B, H, L, F, dt, norm, ragged, state)
    test_backward(B, H, L, F, dt, norm, ragged, state)


def test_gradients_against_differences():
    """The fp64 definition's gradients, which the kernels are held to, against central
    differences of its forward (the normalized form at its own out and den)."""
    B, H, L, F = 1, 2, 9, 8
    for norm in (True, False):
        c, g = _case(B, H, L, F, "f32", norm, False, True, seed=3)
        c = {k: x.double() if torch.is_tensor(x) else x for k, x in c.items()}
        do, dS, dz = (_randn(g, *s).double() for s in ((B, H, L, 64), (B, H, F, 64), (B, H, F)))

        def loss(**kw):
            v, _ = ref.forward(**{**c, **kw})
            return float((v["out"] * do).sum() + (v["S_out"] * dS).sum() + (v["z_out"] * dz).sum() * norm)

        f, _ = ref.forward(**c)
        want, _ = ref.backward(**c, out=f["out"], den=f["den"], dout=do, dS_out=dS, dz_out=dz if norm else None)
        for name, grad in (("phq", "dphq"), ("phk", "dphk"), ("v", "dv"), ("S_in", "dS_in"), ("z_in", "dz_in")):
            if c[name] is None:
                continue
            for at in ((0, 0, 0), (0, 1, 4), (0, 0, 7)):
                at = at + (3,) if c[name].dim() == 4 else at
                x0, x1 = c[name].clone(), c[name].clone()
                x0[at] -= 1e-6
                x1[at] += 1e-6
                diff = (loss(**{name: x1}) - loss(**{name: x0})) / 2e-6
                assert abs(diff - float(want[grad][at])) <= 1e-6 * (1 + abs(diff)), (name, at)


def test_no_decay_is_the_plain_contraction():
    c, _ = _case(2, 2, 300, 256, "f32", True, False, False, kind="none")
    out, den, _, _ = _forward(c, "f32")
    o2, d2 = torch.empty_like(out), torch.empty_like(den)
    bd.slay_linear_attn_fwd(c["phq"], c["phk"], c["v"], o2, d2, c["eps"], True)
    assert float((out - o2).norm() / o2.norm()) <= 1e-5 and float((den - d2).norm() / d2.norm()) <= 1e-5


def test_optional_outputs_change_nothing():
    c, _ = _case(3, 2, 700, 256, "bf16", True, True, True, kind="slow")
    a = _forward(c, "bf16")[0]
    b = _forward(c, "bf16", den=False, state_out=False)[0]
    # (the state that leaves is summed from three limbs, the one inside from two: 2^-17)
    assert float((a - b).float().norm() / a.float().norm()) <= 2.0 ** -9


def test_larger_workspace_and_reuse():
    """One workspace, larger than any of the calls needs, for calls of several sizes in a row."""
    ws = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
    for shape in ((1, 4, 900, 128), (2, 3, 257, 512), (40, 1, 300, 64), (1, 1, 5000, 256)):
        c, _ = _case(*shape, "bf16", True, False, False, kind="slow")
        want = _forward(c, "bf16")[0]
        out = torch.empty_like(want)
        assert bd.slay_decay_attn_fwd(out=out, workspace=ws, **c) is ws
        bd.slay_kernel_status(ws)
        assert float((out - want).float().norm() / want.float().norm()) <= 2.0 ** -9


def test_path_is_what_runs():
    for dt, F, tc in (("bf16", 256, True), ("bf16", 8, True), ("bf16", 512, True), ("bf16", 520, False), ("bf16", 36, False),
                      ("f32", 256, False)):
        c, g = _case(1, 2, 300, F, dt, True, False, False)
        bd.slay_trace_enable(True)
        try:
            bd.slay_trace_read()
            out, den, _, _ = _forward(c, dt)
            fwd = [n for n, _ in bd.slay_trace_read()]
            grads = [torch.empty_like(c[k]) for k in ("phq", "phk", "v")]
            bd.slay_decay_attn_bwd(c["phq"], c["phk"], c["v"], c["log_decay"], torch.ones_like(out), *grads, out=out, den=den)
            torch.cuda.synchronize()
            bwd = [n for n, _ in bd.slay_trace_read()]
        finally:
            bd.slay_trace_enable(False)
        for op, names in ((bd.OP_DECAY_FWD, fwd), (bd.OP_DECAY_BWD, bwd)):
            assert any(n.startswith("tc_decay") for n in names) == tc, names
            assert bd.slay_path(op, TDT[dt], 1, 2, 300, 64, 64, 1, F) == (bd.PATH_TC_CONTRACTION if tc else 0)


@pytest.mark.parametrize("L", [0, 1, 300, 2500])
def test_state_in_place(L):
    c, _ = _case(2, 3, L, 128, "bf16", True, False, True)
    _, _, S, z = _forward(c, "bf16")
    _, _, S2, z2 = _forward(c, "bf16", inplace=True)
    assert torch.equal(S, S2) and torch.equal(z, z2)
    if L == 0:
        assert torch.equal(S, c["S_in"]) and torch.equal(z, c["z_in"])


def test_bwd_state_in_place_and_empty():
    for L in (0, 260):
        c, g = _case(2, 2, L, 64, "bf16", False, False, True)
        dout = _randn(g, 2, 2, L, 64).bfloat16()
        dS = _randn(g, 2, 2, 64, 64)
        grads = [torch.empty_like(c[k]) for k in ("phq", "phk", "v")]
        keep = dS.clone()
        a = torch.empty_like(dS)
        bd.slay_decay_attn_bwd(c["phq"], c["phk"], c["v"], c["log_decay"], dout, *grads, normalize=False, S_in=c["S_in"],
                               dS_out=dS, dS_in=a)
        bd.slay_decay_attn_bwd(c["phq"], c["phk"], c["v"], c["log_decay"], dout, *grads, normalize=False, S_in=c["S_in"],
                               dS_out=dS, dS_in=dS)
        assert torch.equal(a, dS)
        if L == 0:
            assert torch.equal(a, keep)


# The backward's launches: sums of both walks together or not, its sweeps in one launch (with dv
# or without) or one after the other; a final state's gradient updated in place makes no difference.
@pytest.mark.parametrize("B,H,L,F,norm,ragged,states,one", [
    (8, 3, 300, 128, True, True, 0, True), (160, 1, 140, 64, False, True, 0, True), (100, 1, 400, 64, True, False, 0, False),
    (40, 1, 1100, 256, True, False, 0, True), (2, 3, 520, 400, False, True, 1, True), (1, 2, 700, 512, True, False, 1, True),
    (1, 18, 4500, 128, False, False, 2, False), (170, 1, 130, 512, False, True, 0, True), (1, 4, 900, 256, True, False, 1, True),
    (2, 9, 1800, 320, True, False, 2, False), (32, 1, 1100, 512, True, False, 1, False)])
def test_backward_launches(B, H, L, F, norm, ragged, states, one):
    test_backward(B, H, L, F, "bf16", norm, ragged, True)
    c, g = _case(B, H, L, F, "bf16", norm, ragged, True, seed=4)
    out, den, _, _ = _forward(c, "bf16")
    c["dout"] = _randn(g, B, H, L, 64).bfloat16()
    if norm:
        c["out"], c["den"] = out, den
    dS, dz = _randn(g, B, H, F, 64), _randn(g, B, H, F) if norm else None

    def run(in_place):
        grads = {k: torch.full_like(c[x], MARK) for k, x in (("dphq", "phq"), ("dphk", "phk"), ("dv", "v"))}
        dS_out, dz_out = dS.clone(), dz.clone() if norm else None
        dS_in, dz_in = (dS_out, dz_out) if in_place else (torch.empty_like(dS), torch.empty_like(dz) if norm else None)
        bd.slay_decay_attn_bwd(**c, **grads, dS_out=dS_out, dz_out=dz_out, dS_in=dS_in, dz_in=dz_in)
        return [x for x in (*grads.values(), dS_in, dz_in) if x is not None]

    bd.slay_trace_enable(True)
    try:
        bd.slay_trace_read()
        apart = run(False)
        torch.cuda.synchronize()
        names = [n for n, _ in bd.slay_trace_read()]
    finally:
        bd.slay_trace_enable(False)
    assert names.count("tc_decay_state") == states and ("tc_decay_grads" in names) == one, names
    assert all(torch.equal(x, y) for x, y in zip(apart, run(True)))


def test_runs_are_bit_identical():
    c, g = _case(2, 3, 1000, 256, "bf16", True, True, True, kind="slow")
    a, b = _forward(c, "bf16"), _forward(c, "bf16")
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_two_streams_at_once():
    """Two calls in flight, each with its own workspace, and the caller's stream argument."""
    c1, _ = _case(2, 4, 1500, 128, "bf16", True, False, True, seed=5)
    c2, _ = _case(2, 4, 1500, 128, "bf16", True, False, True, seed=6)
    alone = [_forward(c, "bf16")[0] for c in (c1, c2)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [torch.empty_like(x) for x in alone]
    ws = [bd.alloc_workspace(bd.OP_DECAY_FWD, torch.bfloat16, 2, 4, 1500, 64, 64, 1, 128) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, o, w, s in zip((c1, c2), outs, ws, streams):
            bd.slay_decay_attn_fwd(out=o, workspace=w, stream=s, **c)
    torch.cuda.synchronize()
    assert all(torch.equal(a, o) for a, o in zip(alone, outs))


def test_graph_replay_with_new_inputs():
    """Forward and backward captured once, replayed on other values and other lengths."""
    c, g = _case(4, 2, 700, 128, "bf16", False, True, True, kind="slow")
    B, H, L, F = c["phq"].shape
    dout = _randn(g, B, H, L, 64).bfloat16()
    out = torch.zeros_like(c["v"])
    S = torch.empty_like(c["S_in"])
    grads = [torch.zeros_like(c[k]) for k in ("phq", "phk", "v")]
    wf = bd.alloc_workspace(bd.OP_DECAY_FWD, torch.bfloat16, B, H, L, 64, 64, 1, F)
    wb = bd.alloc_workspace(bd.OP_DECAY_BWD, torch.bfloat16, B, H, L, 64, 64, 1, F)

    def step():
        bd.slay_decay_attn_fwd(out=out, S_out=S, workspace=wf, **c)
        bd.slay_decay_attn_bwd(c["phq"], c["phk"], c["v"], c["log_decay"], dout, *grads, normalize=False,
                               lengths=c["lengths"], S_in=c["S_in"], workspace=wb)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    new, _ = _case(4, 2, 700, 128, "bf16", False, True, True, seed=9, kind="slow")
    for k in ("phq", "phk", "v", "S_in"):
        c[k].copy_(new[k])
    c["lengths"].copy_(torch.tensor([3, 700, 129, 0], device="cuda", dtype=torch.int32))
    for x in [out] + grads:
        x.zero_()
    graph.replay()
    torch.cuda.synchronize()
    got = [x.clone() for x in [out, S] + grads]
    for x in [out] + grads:
        x.zero_()
    step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, [out, S] + grads))


# ------------------------------------------------------------------------------ decode
def _decode_want(c, S, z, slots):
    S, z = S.double().clone(), None if z is None else z.double().clone()
    out = torch.full((slots.numel(), S.shape[1], 64), MARK, dtype=torch.float64, device="cuda")
    lam = torch.exp(c["log_decay"].double())
    seen = set()
    for b, s in enumerate(slots.tolist()):
        if s < 0 or s >= S.shape[0] or s in seen:
            continue
        seen.add(s)
        q, k, v = (c[x][b].double() for x in ("phq", "phk", "v"))
        S[s] = lam[:, None, None] * S[s] + k[:, :, None] * v[:, None, :]
        num = torch.einsum("hf,hfe->he", q, S[s])
        if z is not None:
            z[s] = lam[:, None] * z[s] + k
            num = num / ((q * z[s]).sum(-1)[:, None] + c["eps"])
        out[b] = num
    return out, S, z


@pytest.mark.parametrize("Bt,H,F,n,dt,norm", [
    (1, 1, 8, 1, "bf16", True), (1, 3, 33, 2, "f32", True), (3, 2, 256, 5, "bf16", False), (1, 16, 256, 4, "bf16", True),
    (40, 4, 512, 64, "bf16", True), (7, 6, 1000, 9, "f32", True), (300, 2, 64, 320, "bf16", False), (5, 1, 1, 7, "f32", True)])
def test_decode(Bt, H, F, n, dt, norm):
    g = _gen(Bt)
    c = {"phq": _features(g, dt, norm, Bt, H, F), "phk": _features(g, dt, norm, Bt, H, F),
         "v": _randn(g, Bt, H, 64).to(TDT[dt]), "log_decay": _decays(H), "eps": 1e-3}
    S = _randn(g, n, H, F, 64)
    z = torch.exp(_randn(g, n, H, F)) if norm else None
    slots = torch.randperm(n, generator=g, device="cuda")[:Bt].to(torch.int32)
    if Bt >= 3:
        slots[1] = -1
        slots[2] = n            # outside the pool
    if Bt >= 5:
        slots[4] = slots[3]     # named twice: the first row has it
    want, wS, wz = _decode_want(c, S, z, slots)
    out = torch.full((Bt, H, 64), MARK, device="cuda", dtype=TDT[dt])
    bd.slay_decay_decode_step(c["phq"], c["phk"], c["v"], c["log_decay"], S, z, out, slots=slots, normalize=norm, eps=1e-3)
    left = want == MARK
    assert (out.double()[left] == MARK).all()
    # numerators are sums of F terms, each with three fp32 roundings
    mag = want.abs() + F ** 0.5
    assert ((out.double() - want).abs() <= (U[dt] * want.abs() + 8 * 2.0 ** -24 * F ** 0.5 * mag)).all()
    assert ((S.double() - wS).abs() <= 4 * 2.0 ** -24 * (wS.abs() + 1)).all()
    if norm:
        assert ((z.double() - wz).abs() <= 4 * 2.0 ** -24 * (wz.abs() + 1)).all()


def test_decode_without_slots_is_row_order():
    g = _gen(2)
    q, k, v = _features(g, "bf16", True, 3, 2, 128), _features(g, "bf16", True, 3, 2, 128), _randn(g, 3, 2, 64).bfloat16()
    S, z = _randn(g, 4, 2, 128, 64), torch.exp(_randn(g, 4, 2, 128))
    S2, z2 = S.clone(), z.clone()
    a, b = torch.empty_like(v), torch.empty_like(v)
    ld = _decays(2)
    bd.slay_decay_decode_step(q, k, v, ld, S, z, a)
    bd.slay_decay_decode_step(q, k, v, ld, S2, z2, b, slots=torch.arange(3, device="cuda", dtype=torch.int32))
    assert torch.equal(a, b) and torch.equal(S, S2) and torch.equal(z, z2)


# -------------------------------------------------------------------------------- pool
def _copy_want(src_pool, src, dst_pool, dst):
    out = dst_pool.clone()
    for a, b in zip(src, dst):
        if 0 <= b < dst_pool.shape[0] and -1 <= a < src_pool.shape[0]:
            out[b] = src_pool[a] if a >= 0 else 0.0
    return out


@pytest.mark.parametrize("slots,H,F,n,z,seed", [
    (4, 1, 8, 3, True, 0), (9, 3, 33, 9, True, 1), (64, 2, 256, 64, True, 2), (300, 1, 40, 700, True, 3),
    (40, 4, 64, 25, False, 4), (3, 16, 512, 8, True, 5), (5000, 1, 1, 4096, True, 6), (2, 1, 1, 1, True, 7)])
def test_state_copy(slots, H, F, n, z, seed):
    g = _gen(seed)
    S, Z = _randn(g, slots, H, F, 64), _randn(g, slots, H, F)
    src = torch.randint(-2, slots + 2, (n,), generator=g, device="cuda", dtype=torch.int32)
    dst = torch.randint(-1, slots + 1, (n,), generator=g, device="cuda", dtype=torch.int32)   # repeats: the last wins
    wS, wZ = _copy_want(S, src.tolist(), S, dst.tolist()), _copy_want(Z, src.tolist(), Z, dst.tolist())
    other, otherZ = _randn(g, slots + 3, H, F, 64), _randn(g, slots + 3, H, F)
    wO, wOZ = _copy_want(S, src.tolist(), other, dst.tolist()), _copy_want(Z, src.tolist(), otherZ, dst.tolist())
    bd.slay_state_copy(S, Z if z else None, src, other, otherZ if z else None, dst)
    bd.slay_state_copy(S, Z if z else None, src, S, Z if z else None, dst)
    assert torch.equal(other, wO) and torch.equal(S, wS)
    if z:
        assert torch.equal(otherZ, wOZ) and torch.equal(Z, wZ)


def test_copies_of_two_host_threads():
    """Calls of different sizes from two threads, each on its own pools and stream."""
    def work(seed, n, slots, H, F):
        g = _gen(seed)
        S, Z = _randn(g, slots, H, F, 64), _randn(g, slots, H, F)
        src = torch.randint(0, slots, (n,), generator=g, device="cuda", dtype=torch.int32)
        dst = torch.randperm(slots, generator=g, device="cuda")[:n].int()
        want, wantZ = _copy_want(S, src.tolist(), S, dst.tolist()), _copy_want(Z, src.tolist(), Z, dst.tolist())
        S2, Z2, st = torch.empty_like(S), torch.empty_like(Z), torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            for _ in range(200):
                S2.copy_(S), Z2.copy_(Z)
                bd.slay_state_copy(S2, Z2, src, S2, Z2, dst)
        st.synchronize()
        return torch.equal(S2, want) and torch.equal(Z2, wantZ)

    with concurrent.futures.ThreadPoolExecutor(2) as ex:
        runs = [ex.submit(work, 31, 3, 8, 2, 64), ex.submit(work, 32, 2000, 2000, 1, 16)]
        assert all(r.result() for r in runs)


def test_swap_cycle_and_clear():
    g = _gen(11)
    S, Z = _randn(g, 5, 2, 64, 64), _randn(g, 5, 2, 64)
    S0, Z0 = S.clone(), Z.clone()
    i = lambda *x: torch.tensor(x, device="cuda", dtype=torch.int32)  # noqa: E731
    bd.slay_state_copy(S, Z, i(1, 2, 0, -1), S, Z, i(0, 1, 2, 4))
    for pool, old in ((S, S0), (Z, Z0)):
        assert torch.equal(pool[:3], old[[1, 2, 0]]) and torch.equal(pool[3], old[3]) and not pool[4].any()


# ------------------------------------------------------------------ past 32 bits
def test_pool_offsets_past_32_bits():
    """Slots that start beyond 2^31 elements of a pool step and move as those of a small one."""
    H, F, n = 16, 512, 4200
    g = _gen(21)
    small, small_z = _randn(g, 3, H, F, 64), torch.exp(_randn(g, 3, H, F))
    pool, pool_z = torch.zeros(n, H, F, 64, device="cuda"), torch.zeros(n, H, F, device="cuda")
    assert (n - 2) * H * F * 64 > 2 ** 31
    i32 = lambda *x: torch.tensor(x, device="cuda", dtype=torch.int32)  # noqa: E731
    bd.slay_state_copy(small, small_z, i32(0, 1, 2), pool, pool_z, i32(n - 1, 0, n - 2))
    q, k = _features(g, "bf16", True, 2, H, F), _features(g, "bf16", True, 2, H, F)
    v, ld = _randn(g, 2, H, 64).bfloat16(), _decays(H, "slow")
    a, b = torch.empty_like(v), torch.empty_like(v)
    bd.slay_decay_decode_step(q, k, v, ld, pool, pool_z, a, slots=i32(n - 1, n - 2))
    bd.slay_decay_decode_step(q, k, v, ld, small, small_z, b, slots=i32(0, 2))
    bd.slay_state_copy(pool, pool_z, i32(n - 2, -1), pool, pool_z, i32(n - 3, 0))
    assert torch.equal(a, b)
    assert torch.equal(pool[n - 1], small[0]) and torch.equal(pool[n - 2], small[2]) and torch.equal(pool[n - 3], small[2])
    assert torch.equal(pool_z[n - 1], small_z[0]) and torch.equal(pool_z[n - 3], small_z[2])
    assert not pool[0].any() and not pool[1].any() and not pool[n - 4].any()


@pytest.mark.parametrize("B,H,L,F,dt", [(2100, 1, 2048, 512, "bf16"), (1100, 4, 1024, 512, "f32")])
def test_batch_offsets_past_32_bits(B, H, L, F, dt):
    """A batch of more than 2^31 feature elements, every sequence the same: so are its results."""
    assert B * H * L * F > 2 ** 31
    c, g = _case(1, H, L, F, dt, False, False, False, seed=22, kind="slow")
    dout = _randn(g, 1, H, L, 64).to(TDT[dt])
    many = lambda x: x.expand(B, *x.shape[1:]).contiguous()  # noqa: E731
    q, k, v, do = many(c["phq"]), many(c["phk"]), many(c["v"]), many(dout)
    out, dq, dk, dv = torch.zeros_like(v), torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    bd.slay_decay_attn_fwd(q, k, v, c["log_decay"], out, normalize=False)
    bd.slay_decay_attn_bwd(q, k, v, c["log_decay"], do, dq, dk, dv, normalize=False)
    want, mag = ref.forward(**c)
    _ok("out", out[:1], want["out"], mag["out"], dt, L + F)
    for x in (out, dq, dk, dv):
        assert x[0].any() and all(torch.equal(x[b], x[0]) for b in range(1, B))
    del q, k, v, do, out, dq, dk, dv, x
    torch.cuda.empty_cache()


# ------------------------------------------------------------- as a server would use them
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_prefill_fork_decode_compact(dt):
    """Prompts of unequal length into the pool, a fork, decode steps through slots, a move in
    between: every sequence's outputs are those of one forward over its whole token list."""
    H, F, T, steps = 3, 128, 150, 6
    g = _gen(21)
    c, _ = _case(3, H, T + steps, F, dt, True, False, False, seed=21, kind="slow")
    prompt = [150, 1, 77]
    seqs = [0, 1, 2, 1]                       # the running sequences: the fourth is a fork of the second
    q, k, v = (c[x] for x in ("phq", "phk", "v"))
    ext = [tuple(_features(g, dt, True, H, steps, F) for _ in range(2)) + (_randn(g, H, steps, 64).to(TDT[dt]),) for _ in seqs]
    lens = torch.tensor(prompt, device="cuda", dtype=torch.int32)
    S, z = torch.empty(3, H, F, 64, device="cuda"), torch.empty(3, H, F, device="cuda")
    pq, pk, pv = (x[:, :, :T].contiguous() for x in (q, k, v))
    bd.slay_decay_attn_fwd(pq, pk, pv, c["log_decay"], torch.empty_like(pv), eps=c["eps"], lengths=lens, S_out=S, z_out=z)
    pool, pz = torch.full((8, H, F, 64), MARK, device="cuda"), torch.full((8, H, F), MARK, device="cuda")
    i = lambda *x: torch.tensor(x, device="cuda", dtype=torch.int32)  # noqa: E731
    bd.slay_state_copy(S, z, i(0, 1, 2), pool, pz, i(6, 2, 4))        # prompts into their slots
    bd.slay_state_copy(pool, pz, i(2), pool, pz, i(7))                # fork
    slots = i(6, 2, 4, 7)
    got = []
    for t in range(steps):
        if t == 3:                                                    # compaction to the front
            bd.slay_state_copy(pool, pz, i(6, 2, 4, 7, -1, -1), pool, pz, i(0, 1, 2, 3, 6, 7))
            slots = i(0, 1, 2, 3)
        qs, ks, vs = (torch.stack([e[j][:, t] for e in ext]) for j in range(3))
        out = torch.empty_like(vs)
        bd.slay_decay_decode_step(qs, ks, vs, c["log_decay"], pool, pz, out, slots=slots, eps=c["eps"])
        got.append(out)
    got = torch.stack(got, 2)                                         # [4, H, steps, 64]
    for b, s in enumerate(seqs):
        n = prompt[s]
        full = [torch.cat([x[s, :, :n], e], 1)[None] for x, e in zip((q, k, v), ext[b])]
        want, mag = ref.forward(*full, c["log_decay"], c["eps"], True)
        _ok("out", got[b][None], want["out"][:, :, n:], mag["out"][:, :, n:], dt, n + F)
    assert not pool[6:].any() and not pz[6:].any()
