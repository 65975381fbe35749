"""Measured cases of the decayed linear-attention operators and the state pool they share.

Operators (entry points of kernelized_linear_attention_unit_b200.binding):

  fwd     slay_decay_attn_fwd     the chunked causal contraction with a decay for each head
  bwd     slay_decay_attn_bwd     its gradients
  decode  slay_decay_decode_step  one token per sequence on states kept in the slots of a pool
  copy    slay_state_copy         copying, forking, moving and clearing slots of such a pool

Per head, with lambda = exp(log_decay) and lambda^0 = 1, over the tokens of one sequence:

  num_i = sum_{j<=i} lambda^(i-j) (phq_i . phk_j) v_j + lambda^(i+1) phq_i^T S_in
  den_i = sum_{j<=i} lambda^(i-j) (phq_i . phk_j)     + lambda^(i+1) phq_i . z_in
  out_i = num_i / (den_i + eps) (normalized) or num_i
  S_out = sum_j lambda^(n-1-j) phk_j v_j^T + lambda^n S_in,   z_out likewise with v = 1

`run` with `own` false is the plain form of each (torch products, sums and exponentials in
fp32, decay factors from fp64 exponents); with `own` true it calls the framework.  `exact`
is the definition in fp64, one head at a time, over all pairs of tokens.
"""
import torch

own = False

EPS = 1e-6
C = 128          # chunk of the plain form
DV = 64          # value width of the framework's attention
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ----------------------------------------------------------------------------- cases
def listed():
    return [
        # fp32 reference run of a small model with odd sizes, continued from a state
        dict(name="fwd_f32_odd", op="fwd", B=2, H=3, L=333, F=96, dtype="f32", norm=True, ragged=False, state=True),
        # the 2k-token causal workload of the benchmark, with decay
        dict(name="fwd_2k", op="fwd", B=4, H=8, L=2048, F=256, dtype="bf16", norm=True, ragged=False, state=False),
        # the 16k-token causal workload of the benchmark: a long prompt whose state is kept
        dict(name="fwd_16k", op="fwd", B=1, H=16, L=16384, F=256, dtype="bf16", norm=True, ragged=False, state=True),
        # a training batch of short sequences, more heads than SMs, plain sums
        dict(name="fwd_batch", op="fwd", B=32, H=12, L=1024, F=256, dtype="bf16", norm=False, ragged=False, state=False),
        # prompts of unequal length in one padded batch, each continued from its state
        dict(name="fwd_prompts", op="fwd", B=8, H=16, L=1500, F=128, dtype="bf16", norm=False, ragged=True, state=True),
        # fp32 gradients of a small model
        dict(name="bwd_f32", op="bwd", B=1, H=8, L=1024, F=64, dtype="f32", norm=True, ragged=False, state=False),
        # the 8k-token backward workload of the benchmark (F = 512), with decay
        dict(name="bwd_8k", op="bwd", B=2, H=16, L=8192, F=512, dtype="bf16", norm=True, ragged=False, state=False),
        # a padded training batch whose sequences start from carried states
        dict(name="bwd_ragged", op="bwd", B=8, H=8, L=1111, F=128, dtype="bf16", norm=False, ragged=True, state=True),
        # one conversation: latency
        dict(name="decode_1", op="decode", B=1, H=16, F=256, dtype="bf16", norm=True, slots=4),
        # the decode workload of the benchmark (256 sequences), states in a larger pool
        dict(name="decode_256", op="decode", B=256, H=16, F=512, dtype="bf16", norm=True, slots=288),
        # two prompts forked into eight continuations
        dict(name="copy_fork", op="copy", n=8, sources=2, clear=0, slots=64, H=16, F=256),
        # compaction of a serving pool: slots moved to its front, freed ones cleared
        dict(name="copy_compact", op="copy", n=96, sources=96, clear=32, slots=256, H=16, F=512),
    ]


def _log_int(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["fwd", "fwd", "bwd", "bwd", "decode", "copy"])
    F = 8 * _log_int(rng, 4, 64)
    H = _log_int(rng, 1, 24)
    if op == "decode":
        B = max(1, min(_log_int(rng, 1, 256), 2 ** 21 // (H * F)))
        return dict(op=op, B=B, H=H, F=F, dtype=rng.choice(["bf16", "bf16", "f32"]),
                    norm=rng.random() < 0.5, slots=B + _log_int(rng, 1, 32))
    if op == "copy":
        slots = max(3, min(_log_int(rng, 4, 256), 2 ** 21 // (H * F)))
        n = rng.randint(1, slots - 1)
        return dict(op=op, n=n, sources=rng.randint(1, n), clear=rng.randint(0, slots - n) // 2,
                    slots=slots, H=H, F=F)
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    # tokens x heads x features: up to the largest listed backward in bf16, less in fp32
    most = 2 ** 26 if dtype == "bf16" else 2 ** 22
    L = _log_int(rng, 1 if op == "fwd" else 64, 16384)
    H = max(1, min(H, most // (L * F)))
    L = min(L, most // (H * F))
    B = max(1, min(_log_int(rng, 1, 32), most // (H * L * F)))
    return dict(op=op, B=B, H=H, L=L, F=F, dtype=dtype, norm=rng.random() < 0.5,
                ragged=rng.random() < 0.4, state=rng.random() < 0.5)


# ---------------------------------------------------------------------------- inputs
def _decays(H):
    """log(1 - 2^-x), x from 5 to 10 over the heads: memories of 32 to 1024 tokens."""
    x = 5.0 + 5.0 * torch.arange(H, dtype=torch.float64) / max(H - 1, 1)
    return torch.log1p(-torch.exp2(-x)).float().cuda()


def _inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    return g, normal


def _features(case, normal, *shape):
    """Positive random features for the normalized form, signed rows for the plain sums."""
    F = shape[-1]
    x = normal(*shape)
    x = torch.exp(0.7 * x) if case["norm"] else x
    return (x / F ** 0.5).to(DT[case["dtype"]])


def _attn_inputs(case, seed):
    g, normal = _inputs(case, seed)
    B, H, L, F, dt = case["B"], case["H"], case["L"], case["F"], DT[case["dtype"]]
    s = {"case": case, "log_decay": _decays(H)}
    s["phq"] = _features(case, normal, B, H, L, F)
    s["phk"] = _features(case, normal, B, H, L, F)
    s["v"] = normal(B, H, L, DV).to(dt)
    s["lengths"] = None
    if case["ragged"]:
        s["lengths"] = torch.randint(0, L + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
        s["lengths"][int(torch.randint(0, B, (1,), generator=g, device="cuda"))] = L
    s["S_in"] = s["z_in"] = None
    if case["state"]:
        s["S_in"] = normal(B, H, F, DV)
        if case["norm"]:
            s["z_in"] = 8.0 * torch.exp(0.5 * normal(B, H, F))
    return s, g, normal


def prepare(case, seed):
    op = case["op"]
    if op == "fwd":
        s, _, _ = _attn_inputs(case, seed)
        s["out"] = torch.zeros_like(s["v"])
        B, H, L, F = case["B"], case["H"], case["L"], case["F"]
        s["den"] = torch.zeros(B, H, L, device="cuda") if case["norm"] else None
        s["S_out"] = torch.empty(B, H, F, DV, device="cuda") if case["state"] else None
        s["z_out"] = torch.empty(B, H, F, device="cuda") if case["state"] and case["norm"] else None
        s["workspace"] = None
        return s
    if op == "bwd":
        s, _, normal = _attn_inputs(case, seed)
        B, H, L, F, dt = case["B"], case["H"], case["L"], case["F"], DT[case["dtype"]]
        s["dout"] = normal(B, H, L, DV).to(dt)
        s["out"] = s["den"] = None
        if case["norm"]:       # what the forward call left for the backward
            f = _fwd_plain(s)
            s["out"], s["den"] = f["out"], f["den"]
        s["dS_out"] = s["dz_out"] = s["dS_in"] = s["dz_in"] = None
        if case["state"]:
            s["dS_out"] = 0.1 * normal(B, H, F, DV)
            s["dS_in"] = torch.empty_like(s["S_in"])
            if case["norm"]:
                s["dz_out"] = 0.1 * normal(B, H, F)
                s["dz_in"] = torch.empty_like(s["z_in"])
        s["dphq"] = torch.zeros_like(s["phq"])
        s["dphk"] = torch.zeros_like(s["phk"])
        s["dv"] = torch.zeros_like(s["v"])
        s["workspace"] = None
        return s
    if op == "decode":
        g, normal = _inputs(case, seed)
        B, H, F, n, dt = case["B"], case["H"], case["F"], case["slots"], DT[case["dtype"]]
        s = {"case": case, "log_decay": _decays(H)}
        s["phq"] = _features(case, normal, B, H, F)
        s["phk"] = _features(case, normal, B, H, F)
        s["v"] = normal(B, H, DV).to(dt)
        s["S"] = normal(n, H, F, DV)
        s["z"] = 8.0 * torch.exp(0.5 * normal(n, H, F)) if case["norm"] else None
        slots = torch.randperm(n, generator=g, device="cuda")[:B].to(torch.int32)
        if B >= 8:             # rows of the batch that serve no sequence at present
            slots[:: max(8, B // 8)] = -1
        s["slots"] = slots
        s["rows"] = torch.nonzero(slots >= 0).reshape(-1)
        s["out"] = torch.zeros(B, H, DV, device="cuda", dtype=dt)
        return s
    if op == "copy":
        g, normal = _inputs(case, seed)
        n, H, F, slots, clear = case["n"], case["H"], case["F"], case["slots"], case["clear"]
        s = {"case": case, "S": normal(slots, H, F, DV), "z": normal(slots, H, F)}
        perm = torch.randperm(slots, generator=g, device="cuda")
        src = perm[torch.arange(n, device="cuda") % case["sources"]]
        dst = torch.randperm(slots, generator=g, device="cuda")[: n + clear]
        s["src"] = torch.cat([src, torch.full((clear,), -1, device="cuda")]).to(torch.int32)
        s["dst"] = dst.to(torch.int32)
        return s
    raise ValueError(op)


# ------------------------------------------------------------------------ plain forms
def _powers(log_decay, e):
    """lambda^e per head, fp32 [H, *e.shape], from fp64 exponents; lambda^0 = 1."""
    g = log_decay.double().reshape(-1, *([1] * e.dim()))
    return torch.exp(torch.where(e == 0, 0.0, g * e.double())).float()


def _chunked(x, nc):
    B, H, L = x.shape[:3]
    x = torch.nn.functional.pad(x.float(), (0, 0, 0, nc * C - L))
    return x.reshape(B, H, nc, C, x.shape[-1])


def _valid(s):
    """[B,1,L,1] whether a token lies inside its sequence, and the lengths [B]."""
    B, L = s["v"].shape[0], s["v"].shape[2]
    n = s["lengths"].long() if s["lengths"] is not None else torch.full((B,), L, device="cuda")
    return (torch.arange(L, device="cuda") < n[:, None])[:, None, :, None], n


def _to_end(s, n):
    """lambda^(n-1-j) for every token j of a sequence of n tokens, [B,H,L,1] (0 behind it)."""
    L = s["v"].shape[2]
    e = n[:, None] - 1 - torch.arange(L, device="cuda")
    w = _powers(s["log_decay"], e.clamp(min=0)).transpose(0, 1)
    return torch.where(e[:, None] >= 0, w, 0.0)[..., None]


def _with_ones(v, norm):
    return torch.cat([v, torch.ones_like(v[..., :1])], -1) if norm else v


def _joined(S, z):
    return torch.cat([S, z[..., None]], -1) if z is not None else S


def _states(s, k, v, nc, first, reverse):
    """Decayed sums of k v^T over the chunks before (after) each chunk, from `first`."""
    g = s["log_decay"]
    r = torch.arange(C, device="cuda")
    c = torch.arange(nc, device="cuda")
    w = _powers(g, r + 1 if reverse else C - 1 - r)[None, :, None, :, None]
    local = (k * w).transpose(-1, -2) @ v
    e = c[None, :] - c[:, None] - 1 if reverse else c[:, None] - c[None, :] - 1
    D = torch.where(e >= 0, _powers(g, C * e.clamp(min=0)), 0.0)
    B, H, _, F, E = local.shape
    S = (D @ local.reshape(B, H, nc, F * E)).reshape(B, H, nc, F, E)
    if first is not None:
        S = S + _powers(g, C * c)[None, :, :, None, None] * first[:, :, None]
    return S


def _fwd_plain(s):
    case = s["case"]
    B, H, L, F = s["phq"].shape
    g, norm = s["log_decay"], case["norm"]
    nc = -(-L // C)
    ok, n = _valid(s)
    q, k, v = (torch.where(ok, s[x].float(), 0.0) for x in ("phq", "phk", "v"))
    v1 = torch.where(ok, _with_ones(v, norm), 0.0)
    first = _joined(s["S_in"], s["z_in"]) if s["S_in"] is not None else None
    qc, kc, vc = (_chunked(x, nc) for x in (q, k, v1))
    r = torch.arange(C, device="cuda")
    W = torch.tril(_powers(g, (r[:, None] - r[None, :]).clamp(min=0)))
    y = ((qc @ kc.transpose(-1, -2)) * W[None, :, None]) @ vc
    y = y + _powers(g, r + 1)[None, :, None, :, None] * (qc @ _states(s, kc, vc, nc, first, False))
    y = y.reshape(B, H, nc * C, -1)[:, :, :L]
    got = {}
    num = y[..., :DV]
    if norm:
        got["den"] = torch.where(ok[..., 0], y[..., DV], 0.0)
        num = num / (y[..., DV:] + EPS)
    got["out"] = torch.where(ok, num, 0.0).to(s["v"].dtype)
    if case["state"]:
        S = (k * _to_end(s, n)).transpose(-1, -2) @ v1 \
            + _powers(g, n).transpose(0, 1)[..., None, None] * first
        got["S_out"] = S[..., :DV].contiguous()
        if norm:
            got["z_out"] = S[..., DV].contiguous()
    return got


def _bwd_plain(s):
    case = s["case"]
    B, H, L, F = s["phq"].shape
    g, norm, dt = s["log_decay"], case["norm"], s["v"].dtype
    nc = -(-L // C)
    ok, n = _valid(s)
    q, k, v, go = (torch.where(ok, s[x].float(), 0.0) for x in ("phq", "phk", "v", "dout"))
    v1 = torch.where(ok, _with_ones(v, norm), 0.0)
    if norm:
        rz = 1.0 / (s["den"] + EPS)[..., None]
        delta = (go * s["out"].float()).sum(-1, keepdim=True)
        go = torch.where(ok, torch.cat([go * rz, -delta * rz], -1), 0.0)
    first = _joined(s["S_in"], s["z_in"]) if s["S_in"] is not None else None
    qc, kc, vc, gc = (_chunked(x, nc) for x in (q, k, v1, go))
    r = torch.arange(C, device="cuda")
    W = torch.tril(_powers(g, (r[:, None] - r[None, :]).clamp(min=0)))[None, :, None]
    A = (qc @ kc.transpose(-1, -2)) * W
    P = (gc @ vc.transpose(-1, -2)) * W
    S = _states(s, kc, vc, nc, first, False)
    G = _states(s, qc, gc, nc, None, True)
    up = _powers(g, r + 1)[None, :, None, :, None]
    down = _powers(g, C - 1 - r)[None, :, None, :, None]
    dq = P @ kc + up * (gc @ S.transpose(-1, -2))
    dk = P.transpose(-1, -2) @ qc + down * (vc @ G.transpose(-1, -2))
    dv = A.transpose(-1, -2) @ gc[..., :DV] + down * (kc @ G[..., :DV])
    dq, dk, dv = (x.reshape(B, H, nc * C, -1)[:, :, :L] for x in (dq, dk, dv))
    got = {}
    if case["state"]:
        last = _joined(s["dS_out"], s["dz_out"])
        w = _to_end(s, n)
        dk = dk + w * (v1 @ last.transpose(-1, -2))
        dv = dv + w * (k @ s["dS_out"])
        e = torch.arange(L, device="cuda") + 1
        dS = (q * _powers(g, e)[None, ..., None]).transpose(-1, -2) @ go \
            + _powers(g, n).transpose(0, 1)[..., None, None] * last
        got["dS_in"] = dS[..., :DV].contiguous()
        if norm:
            got["dz_in"] = dS[..., DV].contiguous()
    for name, x in (("dphq", dq), ("dphk", dk), ("dv", dv)):
        got[name] = torch.where(ok, x, 0.0).to(dt)
    return got


def _decode_plain(s):
    case, rows = s["case"], s["rows"]
    slots = s["slots"][rows].long()
    lam = torch.exp(s["log_decay"].double()).float()[None, :, None]
    q, k, v = (s[x][rows].float() for x in ("phq", "phk", "v"))
    S = lam[..., None] * s["S"][slots] + k[..., None] * v[..., None, :]
    num = (q[..., None, :] @ S)[..., 0, :]
    s["S"][slots] = S
    if case["norm"]:
        z = lam * s["z"][slots] + k
        s["z"][slots] = z
        num = num / ((q * z).sum(-1, keepdim=True) + EPS)
    s["out"][rows] = num.to(s["out"].dtype)
    return {"out": s["out"], "S": s["S"], **({"z": s["z"]} if case["norm"] else {})}


def _copy_plain(s):
    src, dst = s["src"].long(), s["dst"].long()
    for x in (s["S"], s["z"]):
        y = x[src.clamp(min=0)]
        x[dst] = torch.where((src < 0).reshape(-1, *([1] * (x.dim() - 1))), 0.0, y)
    return {"S": s["S"], "z": s["z"]}


def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        return {"fwd": _fwd_plain, "bwd": _bwd_plain, "decode": _decode_plain, "copy": _copy_plain}[op](s)
    from kernelized_linear_attention_unit_b200 import binding as bd
    if op == "fwd":
        s["workspace"] = bd.slay_decay_attn_fwd(
            s["phq"], s["phk"], s["v"], s["log_decay"], s["out"], den=s["den"], normalize=case["norm"],
            eps=EPS, lengths=s["lengths"], S_in=s["S_in"], z_in=s["z_in"], S_out=s["S_out"],
            z_out=s["z_out"], workspace=s["workspace"])
        return {x: s[x] for x in ("out", "den", "S_out", "z_out") if s[x] is not None}
    if op == "bwd":
        s["workspace"] = bd.slay_decay_attn_bwd(
            s["phq"], s["phk"], s["v"], s["log_decay"], s["dout"], s["dphq"], s["dphk"], s["dv"],
            out=s["out"], den=s["den"], normalize=case["norm"], eps=EPS, lengths=s["lengths"],
            S_in=s["S_in"], z_in=s["z_in"], dS_out=s["dS_out"], dz_out=s["dz_out"], dS_in=s["dS_in"],
            dz_in=s["dz_in"], workspace=s["workspace"])
        return {x: s[x] for x in ("dphq", "dphk", "dv", "dS_in", "dz_in") if s[x] is not None}
    if op == "decode":
        bd.slay_decay_decode_step(s["phq"], s["phk"], s["v"], s["log_decay"], s["S"], s["z"], s["out"],
                                  slots=s["slots"], normalize=case["norm"], eps=EPS)
        return {x: s[x] for x in ("out", "S", "z") if s[x] is not None}
    bd.slay_state_copy(s["S"], s["z"], s["src"], s["S"], s["z"], s["dst"])
    return {"S": s["S"], "z": s["z"]}


# --------------------------------------------------------------------------- the floor
def work(case):
    op, H, F = case["op"], case["H"], case["F"]
    z = 1 if case.get("norm", True) else 0
    if op == "copy":
        slot = 4 * H * F * (DV + 1)
        return {"bytes": slot * (case["sources"] + case["n"] + case["clear"]), "flops": 0}
    e = 2 if case["dtype"] == "bf16" else 4
    B = case["B"]
    if op == "decode":
        rows = B - (-(-B // max(8, B // 8)) if B >= 8 else 0)
        return {"bytes": rows * H * (2 * 4 * F * (DV + z) + e * (2 * F + 2 * DV)),
                "flops": rows * H * F * DV * 5}
    L = case["L"]
    t = B * H * L * (0.5 if case["ragged"] else 1.0)
    st = 4 * B * H * F * (DV + z) if case["state"] else 0
    if op == "fwd":       # phq, phk, v, out and den; the recurrent form's products
        return {"bytes": t * (e * (2 * F + 2 * DV) + 4 * z) + 2 * st, "flops": 4 * t * F * (DV + z)}
    return {"bytes": t * (e * (4 * F + (3 + z) * DV) + 4 * z) + 3 * st, "flops": 10 * t * F * (DV + z)}


# ------------------------------------------------------------------- the definition, fp64
def _pairs(g, n, rows):
    """lambda^(i-j) for i in rows, j < n, zero where j > i."""
    d = rows[:, None] - torch.arange(n, device="cuda")
    return torch.where(d >= 0, torch.exp(torch.where(d == 0, 0.0, g * d.clamp(min=0).double())), 0.0)


def _pow(g, e):
    return torch.exp(torch.where(e == 0, 0.0, g * e.double()))


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "copy":
        S, z = s["S"].clone(), s["z"].clone()
        for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
            S[b] = s["S"][a] if a >= 0 else 0.0
            z[b] = s["z"][a] if a >= 0 else 0.0
        return {"S": S, "z": z}
    norm = case["norm"]
    gs = s["log_decay"].double()
    if op == "decode":
        S, z = s["S"].double(), s["z"].double() if norm else None
        out = s["out"].double()
        for b, slot in enumerate(s["slots"].tolist()):
            if slot < 0:
                continue
            q, k, v = (s[x][b].double() for x in ("phq", "phk", "v"))
            S[slot] = torch.exp(gs)[:, None, None] * S[slot] + torch.einsum("hf,he->hfe", k, v)
            num = torch.einsum("hf,hfe->he", q, S[slot])
            if norm:
                z[slot] = torch.exp(gs)[:, None] * z[slot] + k
                num = num / (torch.einsum("hf,hf->h", q, z[slot])[:, None] + EPS)
            out[b] = num
        return {"out": out, "S": S, **({"z": z} if norm else {})}
    B, H, L, F = s["phq"].shape
    lens = s["lengths"].tolist() if s["lengths"] is not None else [L] * B
    names = ("out", "den", "S_out", "z_out") if op == "fwd" else ("dphq", "dphk", "dv", "dS_in", "dz_in")
    got = {x: torch.zeros_like(s[x], dtype=torch.float64) for x in names if s[x] is not None}
    for b in range(B):
        n = lens[b]
        for h in range(H):
            g = gs[h]
            q, k, v = (s[x][b, h, :n].double() for x in ("phq", "phk", "v"))
            t = torch.arange(n, device="cuda")
            S0 = s["S_in"][b, h].double() if s["S_in"] is not None else None
            z0 = s["z_in"][b, h].double() if s["z_in"] is not None else None
            if op == "fwd":
                for a in range(0, n, 4096):
                    i = t[a:a + 4096]
                    A = (q[i] @ k.T) * _pairs(g, n, i)
                    num, den = A @ v, A.sum(-1)
                    if S0 is not None:
                        num += _pow(g, i + 1)[:, None] * (q[i] @ S0)
                    if norm:
                        if z0 is not None:
                            den += _pow(g, i + 1) * (q[i] @ z0)
                        got["den"][b, h, a:a + len(i)] = den
                        num = num / (den[:, None] + EPS)
                    got["out"][b, h, a:a + len(i)] = num
                if S0 is not None:
                    w = _pow(g, n - 1 - t)[:, None]
                    got["S_out"][b, h] = (w * k).T @ v + _pow(g, torch.tensor(n, device="cuda")) * S0
                    if norm:
                        got["z_out"][b, h] = (w * k).sum(0) + _pow(g, torch.tensor(n, device="cuda")) * z0
                continue
            go = s["dout"][b, h, :n].double()
            delta = torch.zeros(n, dtype=torch.float64, device="cuda")
            if norm:
                go = go / (s["den"][b, h, :n].double()[:, None] + EPS)
                delta = -(go * s["out"][b, h, :n].double()).sum(-1)
            one = 1.0 if norm else 0.0
            dq, dk = torch.zeros(n, F, dtype=torch.float64, device="cuda"), torch.zeros(n, F, dtype=torch.float64, device="cuda")
            dv = torch.zeros(n, DV, dtype=torch.float64, device="cuda")
            for a in range(0, n, 4096):
                i = t[a:a + 4096]
                W = _pairs(g, n, i)
                P = (go[i] @ v.T + delta[i][:, None]) * W
                dq[i] = P @ k
                dk += P.T @ q[i]
                dv += ((q[i] @ k.T) * W).T @ go[i]
            if S0 is not None:
                up, end = _pow(g, t + 1)[:, None], _pow(g, n - 1 - t)[:, None]
                all_ = _pow(g, torch.tensor(n, device="cuda"))
                dS = s["dS_out"][b, h].double()
                dq += up * (go @ S0.T)
                dk += end * (v @ dS.T)
                dv += end * (k @ dS)
                got["dS_in"][b, h] = (up * q).T @ go + all_ * dS
                if norm:
                    dz = s["dz_out"][b, h].double()
                    dq += up * delta[:, None] * z0
                    dk += end * one * dz
                    got["dz_in"][b, h] = ((up * q) * delta[:, None]).sum(0) + all_ * dz
            got["dphq"][b, h, :n], got["dphk"][b, h, :n], got["dv"][b, h, :n] = dq, dk, dv
    return got
