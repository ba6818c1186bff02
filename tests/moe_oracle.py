"""A mixture-of-experts layer in 64 bits from the definition, with a bound of the
fixed-point and fp32 arithmetic that the kernels are allowed.

Error terms, u = 2^-24 (half a step of fp32):
  * x, and h, are held in fixed point: at most 1.02 * 2^-15 of the largest magnitude of
    their block of 128, for each value;
  * a block's integer sums are exact; with w' = |x| (q + |z|) s the magnitude that it is
    folded at, the conversion, the zero point, the step and s round 5 times, the additions
    of up to K / 32 folds and 8 warps once each: (13 + K / 32) u sum(w');
  * h: |act'| <= 1.13 for both activations; exp, erfc, the division and the product a few
    u (taken as 16 u);
  * DOWN sums the same way over h, its K splits and the slots (up to 32 + top_k + 2 roundings);
  * y rounds once: half a step of its type, relative to the value (and half the smallest
    subnormal step).
"""
import math

import torch

U = 2.0 ** -24


def problem(T, E, k, K, I, N, bits, G, dtype, seed, frac=False):
    """Random layer on the CPU: codes (E, K, 2 I) and (E, I, N), s, z, x, ids, weights."""
    g = torch.Generator().manual_seed(seed)
    top = 2 ** bits - 1

    def weight(rows, cols):
        groups = 1 if G == -1 else rows // G
        codes = torch.randint(0, top + 1, (E, rows, cols), generator=g, dtype=torch.uint8)
        s = (0.5 + torch.rand((E, groups, cols), generator=g)) / (0.29 * top * math.sqrt(rows))
        z = (top + 1) / 2 + torch.randn((E, groups, cols), generator=g) * top / 8
        return codes, s.to(dtype), (z if frac else z.round()).to(dtype)

    x = torch.randn((T, K), generator=g).to(dtype)
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).to(torch.int32)
    weights = torch.softmax(torch.randn((T, k), generator=g), 1)
    return {"x": x, "ids": ids, "weights": weights, "up": weight(K, 2 * I), "down": weight(I, N), "E": E, "I": I}


def _product(a, da, codes, s, z, bits):
    """a @ W in 64 bits and a bound of the kernels' error, given a's own error da."""
    K, groups = codes.shape[0], s.shape[0]
    G = K // groups
    q, grp = codes.double(), torch.arange(K) // G
    sd, zd = s.double()[grp], z.double()[grp]
    w = (q - zd) * sd
    mag = a.abs() @ ((q + zd.abs()) * sd.abs())
    top = torch.nn.functional.pad(a.abs() + da, (0, -K % 128)).view(len(a), -1, 128).amax(2)
    da = da + 1.02 * 2.0 ** -15 * top.repeat_interleave(128, 1)[:, :K]
    err = (13 + K / 32) * U * mag + da @ w.abs()
    return a @ w, err


def layer(p, bits, act, ids=None):
    """(y, bound) of the layer in 64 bits, y not rounded."""
    ids = p["ids"] if ids is None else ids
    T, k = ids.shape
    x, I, N = p["x"].double(), p["I"], p["down"][0].shape[2]
    dtype = p["x"].dtype
    y, mag, err = (torch.zeros((T, N), dtype=torch.float64) for _ in range(3))
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            if not 0 <= e < p["E"]:
                continue
            gu, dgu = _product(x[t:t + 1], torch.zeros_like(x[t:t + 1]), *(v[e] for v in p["up"]), bits)
            gate, up, dg, du = gu[:, :I], gu[:, I:], dgu[:, :I], dgu[:, I:]
            if act == "silu":
                a = gate * torch.sigmoid(gate)
            else:
                a = gate * 0.5 * torch.special.erfc(-gate / math.sqrt(2.0))
            h = a * up
            dh = 1.13 * dg * up.abs() + a.abs() * du + 1.13 * dg * du + 16 * U * h.abs() + 1e-37
            part, dpart = _product(h, dh, *(v[e] for v in p["down"]), bits)
            c = float(p["weights"][t, j])
            y[t] += c * part[0]
            err[t] += abs(c) * dpart[0]
            mag[t] += abs(c) * part[0].abs()
    err += (k + 34) * U * mag
    info = torch.finfo(dtype)
    return y, err + (y.abs() + err) * info.eps / 2 + info.smallest_normal * info.eps / 2


def to_gpu(wq, p, bits, dev):
    """x, ids, weights and the six weight tensors as the layer takes them."""
    out = []
    for codes, s, z in (p["up"], p["down"]):
        E, K, N = codes.shape
        w, _ = wq.pack_kmajor(codes.reshape(E * K, N).contiguous().to(dev), bits)
        out += [w.view(E, -1, N), s.to(dev), z.to(dev)]
    return (p["x"].to(dev), p["ids"].to(dev), p["weights"].to(dev)), out


def assert_close(y, ref, tol, what=""):
    d = (y.double().cpu() - ref).abs()
    bad = ~(d <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outside the bound, worst ratio "
                           f"{float((d / tol).nan_to_num(posinf=1e30, nan=1e30).max()):.3g}, first at {bad.nonzero()[0].tolist()}")
    return float((d / tol).max())
