"""Linear attention with a decay for each head from its definition, in 64 bits on the
CPU: the recurrence over the tokens and its adjoint. With `magnitude` every input is
replaced by its absolute value, which gives the sum of the terms' absolute values that
the tests' error bounds are relative to."""
from __future__ import annotations

import torch


def reference(q, k, v, log_decay, scale, h0=None, lengths=None, dy=None, dh_final=None, magnitude=False):
    d = lambda t: None if t is None else (t.double().cpu().abs() if magnitude else t.double().cpu())
    q, k, v, h0, dy, dh_final = d(q), d(k), d(v), d(h0), d(dy), d(dh_final)
    scale = abs(scale) if magnitude else scale
    b, L, H, N = q.shape
    per = H // k.shape[2]
    P = v.shape[-1]
    kf, vf = k.repeat_interleave(per, 2), v.repeat_interleave(per, 2)
    a = torch.exp(log_decay.double().cpu())[:, None, None]
    out = {"y": torch.zeros(b, L, H, P, dtype=torch.float64), "h": torch.zeros(b, H, P, N, dtype=torch.float64)}
    back = dy is not None
    if back:
        z = lambda *s: torch.zeros(*s, dtype=torch.float64)
        out.update(q=z(b, L, H, N), log_decay=z(H), h0=z(b, H, P, N))
        dk, dv = z(b, L, H, N), z(b, L, H, P)
    for i in range(b):
        n = L if lengths is None else max(0, min(L, int(lengths[i])))
        S = h0[i].clone() if h0 is not None else torch.zeros(H, P, N, dtype=torch.float64)
        U = torch.zeros_like(S)
        for t in range(n):
            U = a * (U + S)
            S = a * S + vf[i, t][:, :, None] * kf[i, t][:, None, :]
            out["y"][i, t] = scale * (S @ q[i, t][:, :, None])[..., 0]
            if back:
                g = scale * dy[i, t][:, :, None]
                out["q"][i, t] = (S * g).sum(1)
                out["log_decay"] += ((U @ q[i, t][:, :, None]) * g).sum((1, 2))
        out["h"][i] = S
        if not back:
            continue
        D = dh_final[i].clone() if dh_final is not None else torch.zeros_like(S)
        out["log_decay"] += (D * U).sum((1, 2))
        for t in reversed(range(n)):
            D = D + scale * dy[i, t][:, :, None] * q[i, t][:, None, :]
            dk[i, t] = (D * vf[i, t][:, :, None]).sum(1)
            dv[i, t] = (D * kf[i, t][:, None, :]).sum(2)
            D = a * D
        out["h0"][i] = D
    if back:
        out["k"] = dk.reshape(b, L, H // per, per, N).sum(3)
        out["v"] = dv.reshape(b, L, H // per, per, P).sum(3)
    return out
