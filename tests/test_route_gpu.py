"""The expert router against the 64-bit softmax.

Ids are compared exactly.  A weight is exp(l - m) / sum: l - m rounds once (|l - m| u in
the exponent, u = 2^-24), expf is within 2 units (2u each), the sum of E values in 32
lanes rounds at most E / 32 + 5 times, the division, the scale and the comparison's own
widening add 3: relative (2 (|l - m| + 4) + E / 32 + 12) u, twice over for a margin of 1."""
import pytest

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _dtype(name):
    import torch
    return {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}[name]


def check(libwq, logits, k, renormalize=True, scale=1.0):
    import torch
    ids, w = libwq.moe_route(logits, k, renormalize=renormalize, scale=scale)
    l = logits.double().cpu()
    order = torch.sort(l.nan_to_num(nan=-float("inf"), posinf=float("inf"), neginf=-float("inf")), dim=1,
                       descending=True, stable=True)[1][:, :k]
    top = l.gather(1, order)
    empty = ~(top > -float("inf"))
    assert torch.equal(ids.cpu().long(), torch.where(empty, -1, order))
    m = top[:, :1]
    e = torch.exp(top - m)
    rest = l if not renormalize else top
    total = torch.where(rest > -float("inf"), torch.exp(rest - m), 0.0).sum(1, keepdim=True)
    ref = torch.where(empty, 0.0, scale * e / total)
    ref[torch.isnan(l).any(1, keepdim=True) & ~empty] = float("nan")
    got = w.double().cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(ref))
    fine = ~torch.isnan(ref)
    tol = ref.abs() * (2 * ((top - m).abs() + 4) + l.shape[1] / 32 + 12) * 2 * U + 1e-38
    d = (got - ref).abs()
    assert (d[fine] <= tol.nan_to_num(nan=1e-38)[fine]).all(), float((d / tol)[fine].max())
    return ids, w


@pytest.mark.parametrize("dt", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 2, 2), (1, 64, 8), (7, 31, 5), (8, 32, 16), (9, 33, 16),
                                   (100, 65, 6), (257, 128, 8), (3, 200, 1), (1000, 512, 16)])
def test_random(cuda, libwq, T, E, k, dt):
    import torch
    g = torch.Generator(device=cuda).manual_seed(T + E)
    logits = (2 * torch.randn((T, E), generator=g, device=cuda)).to(_dtype(dt))
    check(libwq, logits, k)
    check(libwq, logits, k, renormalize=False, scale=2.5)


def test_ties_take_the_lowest_index(cuda, libwq):
    import torch
    logits = torch.zeros((4, 96), device=cuda)
    logits[1, ::2] = -0.0
    logits[2, 40:44] = 1.0
    logits[3] = torch.finfo(torch.float32).min
    ids, w = check(libwq, logits, 6)
    assert ids[0].tolist() == ids[1].tolist() == ids[3].tolist() == [0, 1, 2, 3, 4, 5]
    assert ids[2].tolist() == [40, 41, 42, 43, 0, 1]


def test_masked_rows(cuda, libwq):
    """-inf is never chosen; a row of nothing else has empty slots."""
    import torch
    logits = torch.randn((5, 40), device=cuda)
    logits[0] = -float("inf")
    logits[1, 3:] = -float("inf")
    logits[2, 5] = float("nan")
    logits[3, :] = float("nan")
    logits[4, 39] = 60000.0
    for renormalize in (True, False):
        ids, w = check(libwq, logits, 8, renormalize)
        assert (ids[0] == -1).all() and (w[0] == 0).all()
        assert (ids[1, 3:] == -1).all() and (w[1, 3:] == 0).all()
        assert (ids[3] == -1).all()


def test_row_stride_and_infinity(cuda, libwq):
    import torch
    wide = torch.randn((6, 77), device=cuda).half()
    check(libwq, wide[:, 3:70], 4)
    check(libwq, wide[::2, :10], 4)
    wide[:, 20] = float("inf")
    ids, w = libwq.moe_route(wide, 2)
    assert (ids[:, 0] == 20).all() and torch.isnan(w).all()


def test_stream_and_graph(cuda, libwq):
    import torch
    logits = torch.randn((16, 64), device=cuda)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ids, w = libwq.moe_route(logits, 4, pdl=True)
    logits.copy_(torch.randn((16, 64), device=cuda))
    graph.replay()
    torch.cuda.synchronize()
    ids2, w2 = check(libwq, logits, 4)
    assert torch.equal(ids, ids2) and torch.equal(w, w2)


def test_refusals(cuda, libwq):
    import torch
    l = torch.randn((4, 16), device=cuda)
    for bad in (l.double(), l.cpu(), l[0], l.t(), l.int()):
        with pytest.raises((TypeError, ValueError)):
            libwq.moe_route(bad, 2)
    for k in (0, 17):
        with pytest.raises((RuntimeError, ValueError)):
            libwq.moe_route(l, k)
    with pytest.raises(libwq.WQError):
        libwq.moe_route(l, 2, scale=float("nan"))
    with pytest.raises(libwq.WQError):
        libwq.moe_route(torch.zeros((2, 513), device=cuda), 2)
    with pytest.raises(libwq.WQError):
        libwq.moe_route(l[:0], 2)
