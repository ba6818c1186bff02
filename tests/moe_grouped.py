"""moe_oracle's layer and bound with the slots of an expert taken together: the same
arithmetic in 64 bits, quick enough for layers of usual sizes (on any device)."""
import math

import torch

import moe_oracle
from moe_oracle import U


def layer(p, bits, act, product=moe_oracle._product):
    """(y, bound) of the layer in 64 bits, y not rounded."""
    ids, weights = p["ids"], p["weights"].double()
    T, k = ids.shape
    x, I, N, dtype = p["x"].double(), p["I"], p["down"][0].shape[2], p["x"].dtype
    y, mag, err = (torch.zeros((T, N), dtype=torch.float64, device=x.device) for _ in range(3))
    for e in range(p["E"]):
        t, j = (ids == e).nonzero(as_tuple=True)
        if not len(t):
            continue
        gu, dgu = product(x[t], torch.zeros_like(x[t]), *(v[e] for v in p["up"]), bits)
        gate, up, dg, du = gu[:, :I], gu[:, I:], dgu[:, :I], dgu[:, I:]
        if act == "silu":
            a = gate * torch.sigmoid(gate)
        else:
            a = gate * 0.5 * torch.special.erfc(-gate / math.sqrt(2.0))
        h = a * up
        dh = 1.13 * dg * up.abs() + a.abs() * du + 1.13 * dg * du + 16 * U * h.abs() + 1e-37
        part, dpart = product(h, dh, *(v[e] for v in p["down"]), bits)
        c = weights[t, j][:, None]
        y.index_add_(0, t, c * part)
        err.index_add_(0, t, c.abs() * dpart)
        mag.index_add_(0, t, c.abs() * part.abs())
    err += (k + 34) * U * mag
    info = torch.finfo(dtype)
    return y, err + (y.abs() + err) * info.eps / 2 + info.smallest_normal * info.eps / 2
