"""The decayed linear-attention operators in fp64 over all pairs of tokens, for their tests.

Every function returns, beside each value, the same sum over absolute values: the size that
the roundings inside a kernel are relative to, whatever cancels in the value itself.
"""
import torch


def powers(g, e):
    """exp(g)^e elementwise, fp64, with lambda^0 = 1 also for g = -inf."""
    return torch.where(e == 0, 1.0, torch.exp(torch.where(e == 0, 0.0, g * e.clamp(min=1).double())))


def _pairs(g, n, dev):
    t = torch.arange(n, device=dev)
    d = t[:, None] - t[None, :]
    return torch.where(d >= 0, powers(g, d.clamp(min=0)), 0.0)


def _lens(lengths, B, L):
    return [L] * B if lengths is None else [min(max(int(x), 0), L) for x in lengths.tolist()]


def forward(phq, phk, v, log_decay, eps, normalize, lengths=None, S_in=None, z_in=None):
    B, H, L, F = phq.shape
    dev = phq.device
    new = lambda *s: torch.zeros(*s, dtype=torch.float64, device=dev)  # noqa: E731
    val = {"out": new(B, H, L, 64), "den": new(B, H, L), "S_out": new(B, H, F, 64), "z_out": new(B, H, F)}
    mag = {k: x.clone() for k, x in val.items()}
    for b, n in enumerate(_lens(lengths, B, L)):
        for h in range(H):
            g = log_decay[h].double()
            q, k, u = (x[b, h, :n].double() for x in (phq, phk, v))
            t = torch.arange(n, device=dev)
            W, up, end = _pairs(g, n, dev), powers(g, t + 1)[:, None], powers(g, n - 1 - t)[:, None]
            whole = powers(g, torch.tensor(n, device=dev))
            S = S_in[b, h].double() if S_in is not None else new(F, 64)
            z = z_in[b, h].double() if z_in is not None else new(F)
            for d, f in ((val, lambda x: x), (mag, torch.abs)):
                fq, fk, fu, fS, fz = f(q), f(k), f(u), f(S), f(z)
                A = (fq @ fk.T) * W
                num, den = A @ fu + up * (fq @ fS), A.sum(-1) + up[:, 0] * (fq @ fz)
                d["den"][b, h, :n] = den
                d["S_out"][b, h] = (end * fk).T @ fu + whole * fS
                d["z_out"][b, h] = (end * fk).sum(0) + whole * fz
                if normalize:
                    num = num / (val["den"][b, h, :n, None] + eps).abs()
                d["out"][b, h, :n] = num
            if normalize:
                val["out"][b, h, :n] *= torch.sign(val["den"][b, h, :n, None] + eps)
    return val, mag


def backward(phq, phk, v, log_decay, out, den, dout, eps, normalize, lengths=None, S_in=None, z_in=None,
             dS_out=None, dz_out=None):
    B, H, L, F = phq.shape
    dev = phq.device
    new = lambda *s: torch.zeros(*s, dtype=torch.float64, device=dev)  # noqa: E731
    val = {"dphq": new(B, H, L, F), "dphk": new(B, H, L, F), "dv": new(B, H, L, 64), "dS_in": new(B, H, F, 64),
           "dz_in": new(B, H, F)}
    mag = {k: x.clone() for k, x in val.items()}
    for b, n in enumerate(_lens(lengths, B, L)):
        for h in range(H):
            g = log_decay[h].double()
            q, k, u, do = (x[b, h, :n].double() for x in (phq, phk, v, dout))
            t = torch.arange(n, device=dev)
            W, up, end = _pairs(g, n, dev), powers(g, t + 1)[:, None], powers(g, n - 1 - t)[:, None]
            whole = powers(g, torch.tensor(n, device=dev))
            pick = lambda x, *s: x[b, h].double() if x is not None else new(*s)  # noqa: E731
            S, z, dS, dz = pick(S_in, F, 64), pick(z_in, F), pick(dS_out, F, 64), pick(dz_out, F)
            rz = 1.0 / (den[b, h, :n].double() + eps) if normalize else torch.ones(n, dtype=torch.float64, device=dev)
            o = out[b, h, :n].double() if normalize else torch.zeros_like(do)
            one = 1.0 if normalize else 0.0
            for d, f, sign in ((val, lambda x: x, -1.0), (mag, torch.abs, 1.0)):
                fq, fk, fu, fdo, fS, fz, fdS, fdz, fr = (f(x) for x in (q, k, u, do, S, z, dS, dz, rz))
                delta = sign * (fdo * f(o)).sum(-1)
                P = ((fdo @ fu.T) + delta[:, None]) * fr[:, None] * W
                A = (fq @ fk.T) * fr[:, None] * W
                d["dphq"][b, h, :n] = P @ fk + up * fr[:, None] * (fdo @ fS.T + one * delta[:, None] * fz)
                d["dphk"][b, h, :n] = P.T @ fq + end * (fu @ fdS.T + one * fdz)
                d["dv"][b, h, :n] = A.T @ fdo + end * (fk @ fdS)
                wq = up * fr[:, None] * fq
                d["dS_in"][b, h] = wq.T @ fdo + whole * fdS
                d["dz_in"][b, h] = one * ((wq * delta[:, None]).sum(0) + whole * fdz)
    return val, mag
