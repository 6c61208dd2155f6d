"""The sequence operators' definitions in 64 bits, with the sums of absolute
terms that the tolerances are made of. Dense, on the CPU, for small sizes."""
from __future__ import annotations

import math

import torch


def unit(dtype):
    """Half a step of the type, relative to the value."""
    return torch.finfo(dtype).eps / 2


def visible(nq, nk, window, sinks):
    p = (nk - nq + torch.arange(nq)).view(-1, 1)
    j = torch.arange(nk).view(1, -1)
    return (j <= p) & ((j > p - window) | (j < sinks))


def lengths(lens, B, most):
    return [most] * B if lens is None else [min(max(int(n), 0), most) for n in lens]


def attention(q, k, v, window, sinks, scale, q_lens=None, kv_lens=None, dout=None):
    """dict of out, lse (and dq, dk, dv) with the bounds' sums beside them:
    out_abs[b, i, h, d] = sum_j p_ij |v_jd| and so on."""
    B, Lq, Hq, D = q.shape
    Lk, Hkv = k.shape[1:3]
    G = Hq // Hkv
    q, k, v = q.double().cpu(), k.double().cpu(), v.double().cpu()
    new = lambda *s: torch.zeros(s, dtype=torch.float64)  # noqa: E731
    r = {"out": new(B, Lq, Hq, D), "out_abs": new(B, Lq, Hq, D),
         "lse": torch.full((B, Hq, Lq), -math.inf, dtype=torch.float64)}
    if dout is not None:
        dout = dout.double().cpu()
        for n, like in (("dq", q), ("dk", k), ("dv", v)):
            r[n], r[n + "_abs"] = torch.zeros_like(like), torch.zeros_like(like)
    for b, (m, n) in enumerate(zip(lengths(q_lens, B, Lq), lengths(kv_lens, B, Lk))):
        if m == 0 or n == 0:
            continue
        seen = visible(m, n, window, sinks)
        for h in range(Hq):
            Q, K, V = q[b, :m, h], k[b, :n, h // G], v[b, :n, h // G]
            s = torch.where(seen, scale * (Q @ K.T), -math.inf)
            lse = torch.logsumexp(s, 1)
            P = torch.where(seen, torch.exp(s - lse.view(-1, 1)), 0.0)
            o, oa = P @ V, P @ V.abs()
            r["out"][b, :m, h], r["out_abs"][b, :m, h], r["lse"][b, h, :m] = o, oa, lse
            if dout is None:
                continue
            dO = dout[b, :m, h]
            dP, dPa = dO @ V.T, dO.abs() @ V.abs().T
            delta, da = (dO * o).sum(1, keepdim=True), (dO * o).abs().sum(1, keepdim=True)
            dS, dSa = P * (dP - delta), P * (dPa + da)
            r["dq"][b, :m, h] = scale * (dS @ K)
            r["dq_abs"][b, :m, h] = abs(scale) * (dSa @ K.abs())
            r["dk"][b, :n, h // G] += scale * (dS.T @ Q)
            r["dk_abs"][b, :n, h // G] += abs(scale) * (dSa.T @ Q.abs())
            r["dv"][b, :n, h // G] += P.T @ dO
            r["dv_abs"][b, :n, h // G] += P.T @ dO.abs()
    return r


def linear(q, k, v, log_decay, scale, state=None, lens=None, dout=None, dstate=None):
    """out, state (and dq, dk, dv, dstate_in), each with its sums of absolute
    terms, token by token."""
    B, L, H, Dk = q.shape
    Dv = v.shape[3]
    q, k, v, g = (x.double().cpu().movedim(-1, -1) for x in (q, k, v, log_decay))
    a = torch.exp(g).view(1, H, 1, 1)
    new = lambda *s: torch.zeros(s, dtype=torch.float64)  # noqa: E731
    S0 = new(B, H, Dk, Dv) if state is None else state.double().cpu()
    live = torch.tensor(lengths(lens, B, L)).view(B, 1)
    at = lambda x, t: torch.where((t < live).view(B, 1, 1), x[:, t], 0.0)  # noqa: E731
    keep = lambda t: (t < live).view(B, 1, 1, 1)  # noqa: E731
    r = {"out": new(B, L, H, Dv), "out_abs": new(B, L, H, Dv)}
    S, Sa, before, before_abs = S0.clone(), S0.abs(), [], []
    for t in range(L):
        Q, K, V = at(q, t), at(k, t), at(v, t)
        S = torch.where(keep(t), a * S + K.unsqueeze(3) * V.unsqueeze(2), S)
        Sa = torch.where(keep(t), a * Sa + K.abs().unsqueeze(3) * V.abs().unsqueeze(2), Sa)
        before.append(S), before_abs.append(Sa)
        r["out"][:, t] = scale * (Q.unsqueeze(2) @ S).squeeze(2)
        r["out_abs"][:, t] = abs(scale) * (Q.abs().unsqueeze(2) @ Sa).squeeze(2)
    r["state"], r["state_abs"] = S, Sa
    if dout is None:
        return r
    dout = dout.double().cpu()
    for n, like in (("dq", q), ("dk", k), ("dv", v)):
        r[n], r[n + "_abs"] = torch.zeros_like(like), torch.zeros_like(like)
    # R: gradient of the state after token t.
    R = new(B, H, Dk, Dv) if dstate is None else dstate.double().cpu()
    Ra = R.abs()
    for t in reversed(range(L)):
        Q, K, V, dO = at(q, t), at(k, t), at(v, t), at(dout, t)
        R = torch.where(keep(t), R + scale * Q.unsqueeze(3) * dO.unsqueeze(2), R)
        Ra = torch.where(keep(t), Ra + abs(scale) * Q.abs().unsqueeze(3) * dO.abs().unsqueeze(2), Ra)
        r["dq"][:, t] = scale * (before[t] @ dO.unsqueeze(3)).squeeze(3)
        r["dq_abs"][:, t] = abs(scale) * (before_abs[t] @ dO.abs().unsqueeze(3)).squeeze(3)
        r["dk"][:, t] = (R @ V.unsqueeze(3)).squeeze(3)
        r["dk_abs"][:, t] = (Ra @ V.abs().unsqueeze(3)).squeeze(3)
        r["dv"][:, t] = (K.unsqueeze(2) @ R).squeeze(2)
        r["dv_abs"][:, t] = (K.abs().unsqueeze(2) @ Ra).squeeze(2)
        R, Ra = torch.where(keep(t), a * R, R), torch.where(keep(t), a * Ra, Ra)
    r["dstate"], r["dstate_abs"] = R, Ra
    return r


def assert_close(got, want, bound, what):
    """|got - want| <= bound everywhere; NaN never passes, nor do shapes that differ."""
    got = got.double().cpu()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    over = ~((got - want).abs() <= bound)
    if bool(over.any()):
        at = [tuple(i) for i in over.nonzero()[:4].tolist()]
        raise AssertionError(f"{what}: {int(over.sum())} of {over.numel()} out of bounds; " + ", ".join(
            f"{i}: {got[i].item():.6g} for {want[i].item():.6g} +- {bound[i].item():.2g}" for i in at))
