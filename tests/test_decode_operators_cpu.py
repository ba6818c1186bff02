"""The router, the expert layer and the log probabilities refuse bad arguments on the
host, before any launch, and the 64-bit oracle of the layer agrees with worked cases."""
import ctypes
import math

import pytest

import moe_oracle

P = 0x10000  # an aligned fake device address: never dereferenced on the host path
INV, UNS, ALI, CUDA = 1, 2, 3, 6


def no_device():
    import torch
    return not torch.cuda.is_available()


def test_route_argument_checks(libwq):
    L = libwq.lib()

    def call(l=P, type=2, T=3, E=64, ld=64, k=8, norm=1, scale=1.0, ids=P, w=P, flags=0):
        return L.wq_moe_route(l, type, T, E, ld, k, norm, ctypes.c_float(scale), ids, w, flags, None)
    assert call(type=3) == UNS and call(type=-1) == UNS
    for bad in (dict(T=0), dict(E=0), dict(E=513, ld=513), dict(ld=63), dict(k=0), dict(k=17), dict(E=4, k=5),
                dict(norm=2), dict(scale=math.nan), dict(scale=math.inf), dict(l=None), dict(ids=None),
                dict(w=None), dict(flags=2), dict(flags=4), dict(T=-1)):
        assert call(**bad) == INV, bad
    assert call(l=P + 2) == ALI and call(l=P + 1, type=0) == ALI and call(ids=P + 2) == ALI and call(w=P + 1) == ALI
    if no_device():
        assert call() == CUDA and call(l=P + 2, type=1, flags=1) == CUDA


def test_moe_argument_checks(libwq):
    L = libwq.lib()
    need = L.wq_moe_workspace_size(4, 2, 128, 256)
    assert need >= 4 * 2 * 128 * 2
    assert L.wq_moe_workspace_size(0, 2, 128, 256) == 0 and L.wq_moe_workspace_size(65, 2, 128, 256) == 0
    assert L.wq_moe_workspace_size(4, 17, 128, 256) == 0

    def call(T=4, K=256, I=128, N=256, E=8, k=2, bits=4, G=64, act=0, flags=0, ws=P, nbytes=None, **ptr):
        names = ("x", "ids", "weights", "w_up", "s_up", "z_up", "w_down", "s_down", "z_down", "y")
        a = [ptr.get(n, P) for n in names]
        return L.wq_moe(*a, T, K, I, N, E, k, bits, G, act, flags, ws,
                        ctypes.c_size_t(need if nbytes is None else nbytes), None)
    assert call(bits=3) == UNS and call(bits=5) == UNS and call(act=2) == UNS and call(G=16) == UNS
    assert call(K=24576 + 64) == UNS and call(bits=8, G=16) == UNS
    assert call(T=64, k=16, I=1 << 20, G=-1, nbytes=1 << 50) == UNS       # h of all slots passes 2^31 bytes
    for bad in (dict(T=0), dict(T=65, nbytes=1 << 40), dict(K=0), dict(K=252, G=-1), dict(I=0), dict(I=-8), dict(N=0),
                dict(E=0), dict(E=513), dict(k=0), dict(k=17, nbytes=1 << 40), dict(G=0), dict(G=96), dict(flags=2),
                dict(flags=8), dict(ws=None), dict(nbytes=need - 1), dict(I=1 << 30)):
        assert call(**bad) == INV, bad
    for name in ("x", "ids", "weights", "w_up", "s_up", "z_up", "w_down", "s_down", "z_down", "y"):
        assert call(**{name: None}) == INV
        assert call(**{name: P + 2}) == ALI
    assert call(N=252) == ALI and call(I=132, G=-1, bits=8) == ALI and call(ws=P + 16) == ALI
    if no_device():
        assert call() == CUDA and call(G=-1, flags=4) == CUDA and call(bits=8, G=32, flags=5) == CUDA


def test_logprobs_argument_checks(libwq):
    L = libwq.lib()

    def call(l=P, type=0, R=2, V=1000, ld=1000, tok=P, k=5, lp=P, ent=P, tlp=P, tid=P, flags=0):
        return L.wq_logprobs(l, type, R, V, ld, tok, k, lp, ent, tlp, tid, flags, None)
    assert call(type=3) == UNS
    for bad in (dict(R=0), dict(R=(1 << 24) + 1), dict(V=0), dict(V=1 << 30, ld=1 << 30), dict(ld=999), dict(k=-1),
                dict(k=33), dict(V=4, ld=4), dict(l=None), dict(ent=None), dict(tok=None), dict(lp=None),
                dict(k=0), dict(tid=None), dict(tlp=None), dict(flags=2), dict(flags=4)):
        assert call(**bad) == INV, bad
    assert call(l=P + 1) == ALI and call(l=P + 2, type=2) == ALI and call(tok=P + 4) == ALI
    assert call(tid=P + 4) == ALI and call(ent=P + 2) == ALI and call(lp=P + 2) == ALI and call(tlp=P + 1) == ALI
    if no_device():
        assert call() == CUDA and call(tok=None, lp=None, k=0, tlp=None, tid=None) == CUDA
        assert call(l=P + 2, V=3, ld=1 << 33, k=3) == CUDA


def test_binding_refuses_host_tensors(libwq):
    torch = pytest.importorskip("torch")
    with pytest.raises(ValueError):
        libwq.moe_route(torch.zeros(2, 4), 1)
    with pytest.raises(ValueError):
        libwq.logprobs(torch.zeros(2, 4))
    with pytest.raises(TypeError):
        libwq.logprobs([[1.0]])
    p = moe_oracle.problem(2, 2, 1, 32, 32, 8, 4, 32, torch.float16, seed=0)
    w = [torch.zeros((2, 4, 64), dtype=torch.int32), p["up"][1], p["up"][2],
         torch.zeros((2, 4, 8), dtype=torch.int32), p["down"][1], p["down"][2]]
    with pytest.raises(ValueError):
        libwq.MoePlan(*w, 4, 32, 2, 1)
    with pytest.raises(ValueError):
        libwq.MoePlan(*w, 3, 32, 2, 1)
    with pytest.raises(TypeError):
        libwq.MoePlan(*w[:1], w[1].float(), *w[2:], 4, 32, 2, 1)


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_oracle_worked_case(act):
    """One token, one expert, one nonzero path: y = c * act(g) u d by hand; an empty slot gives 0."""
    torch = pytest.importorskip("torch")
    p = moe_oracle.problem(2, 2, 1, 8, 8, 8, 4, -1, torch.float16, seed=0)
    for name in ("up", "down"):
        p[name][0].zero_(), p[name][2].zero_(), p[name][1].fill_(1.0)
    p["x"].zero_()
    p["x"][0, 3] = 2.0
    p["up"][0][1, 3, 5], p["up"][0][1, 3, 8 + 5], p["down"][0][1, 5, 2] = 1, 3, 4
    p["weights"].fill_(0.5)
    ids = torch.tensor([[1], [-1]], dtype=torch.int32)
    y, tol = moe_oracle.layer(p, 4, act, ids)
    a = 2 / (1 + math.exp(-2)) if act == "silu" else 2 * 0.5 * (1 + math.erf(2 / math.sqrt(2)))
    want = torch.zeros((2, 8), dtype=torch.float64)
    want[0, 2] = 0.5 * a * 6 * 4
    assert torch.allclose(y, want, rtol=1e-12, atol=0) and (tol[1] < 1e-7).all()


def test_oracle_bound_is_tight_enough():
    """A small mistake in the zero points is outside the bound nearly everywhere."""
    torch = pytest.importorskip("torch")
    p = moe_oracle.problem(2, 3, 2, 64, 32, 16, 4, 32, torch.float16, seed=3)
    y, tol = moe_oracle.layer(p, 4, "silu")
    q = dict(p, up=(p["up"][0], p["up"][1], p["up"][2] + 0.25))
    y2, _ = moe_oracle.layer(q, 4, "silu")
    assert ((y - y2).abs() > tol).float().mean() > 0.9
