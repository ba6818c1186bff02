"""Token log probabilities, entropy and top entries against 64 bits.

Bounds, u = 2^-24, d = l - ref with ref at most 8 below the maximum, p the softmax:
a term e^d has relative error 2u (ex2) + (|d| + 2) 2u (its argument); the sums round at
most V / 256 + 32 times per thread, warp, CTA and cluster together.  So
  r      = 2u + 2u (sum p |d| + 10) + (V / 256 + 32) u      (ln S1, absolute)
  log p  : r + u (|l - ref| + |ln S1| + |log p|) (the subtractions, logf)
  entropy: r + (2u + (V / 256 + 34) u) D + 2u (sum p d^2 + 10 D) + r D + 2u (H + D),  D = sum p |d|
with |d| <= |l - max| + 8.  Ids are exact."""
import pytest

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
INF = float("inf")


def _dtype(name):
    import torch
    return {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}[name]


def reference(logits, tokens, k):
    import torch
    l = logits.double().cpu()
    V = l.shape[1]
    m = l.amax(1, keepdim=True)
    logp = torch.log_softmax(l, 1)
    p = logp.exp()
    d = torch.where(p > 0, (l - m).abs() + 8, 0.0)
    D, D2 = (p * d).sum(1), (p * d * d).sum(1)
    H = torch.where(p > 0, -p * logp, 0.0).sum(1)
    H[torch.isnan(logp).any(1)] = float("nan")
    steps = V / 256 + 34
    r = (2 + 2 * (D + 10) + steps) * U
    tol_h = r + ((2 + steps) * D + 2 * (D2 + 10 * D) + 2 * (H + D)) * U + r * D

    def tol(at):  # of log p at columns `at`
        lp = logp.gather(1, at)
        dd = (l.gather(1, at) - m).abs() + 8
        return r[:, None] + U * (dd + 8 + (dd + lp.abs()) + lp.abs())
    inside = (tokens >= 0) & (tokens < V)
    at = torch.where(inside, tokens, 0)[:, None]
    lp = torch.where(inside, logp.gather(1, at)[:, 0], torch.tensor(-INF, dtype=torch.float64))
    order = torch.sort(l.nan_to_num(nan=-INF, posinf=INF, neginf=-INF), dim=1, descending=True, stable=True)[1][:, :k]
    return {"entropy": (H, tol_h), "logprob": (lp, tol(at)[:, 0]), "top_id": order,
            "top_logprob": (logp.gather(1, order), tol(order))}


def check(libwq, logits, tokens, k):
    import torch
    got = libwq.logprobs(logits, tokens, k)
    ref = reference(logits, tokens.cpu(), k)
    if k:
        assert torch.equal(got["top_id"].cpu(), ref["top_id"])
    else:
        assert "top_id" not in got
    for name in ("entropy", "logprob") + (("top_logprob",) if k else ()):
        (want, tol), have = ref[name], got[name].double().cpu()
        assert torch.equal(torch.isnan(have), torch.isnan(want)), name
        odd = ~torch.isfinite(want)
        assert torch.equal(have[odd].nan_to_num(nan=7.0), want[odd].nan_to_num(nan=7.0)), name
        d = (have - want).abs()[~odd]
        assert (d <= tol[~odd]).all(), (name, float((d / tol[~odd]).max()))
    return got


def draw(R, V, dt, seed, dev):
    import torch
    g = torch.Generator(device=dev).manual_seed(seed)
    l = (2.5 * torch.randn((R, V), generator=g, device=dev)).to(_dtype(dt))
    return l, torch.randint(0, V, (R,), generator=g, device=dev)


@pytest.mark.parametrize("dt", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("R,V", [(1, 1), (3, 2), (2, 7), (5, 8), (4, 9), (3, 31), (2, 255), (9, 257), (70, 1000),
                                 (3, 2049), (2, 4097), (1, 8192), (700, 3001), (40, 16384), (1, 50001), (3, 131071),
                                 (300, 20000)])
def test_random(cuda, libwq, R, V, dt):
    logits, tokens = draw(R, V, dt, R * 7 + V, cuda)
    for k in sorted({0, 1, min(5, V), min(32, V)}):
        check(libwq, logits, tokens, k)


@pytest.mark.parametrize("dt", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("R", [2, 320])
def test_row_strides(cuda, libwq, dt, R):
    """Rows that start at any element, inside a wider array, and columns cut off a padded vocabulary."""
    wide, tokens = draw(R, 5003, dt, 3, cuda)
    for lo, hi in ((0, 5000), (1, 4000), (3, 5), (7, 4999), (5, 1030)):
        check(libwq, wide[:, lo:hi], tokens % (hi - lo), 2)
    check(libwq, wide[::2, :2000], (tokens % 2000)[::2].contiguous(), 4)


@pytest.mark.parametrize("dt", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("R,V", [(3, 20000), (320, 5000)])
def test_masks(cuda, libwq, dt, R, V):
    """-inf and the type's lowest value, with fewer entries left than top_k; whole rows of either."""
    import torch
    logits, tokens = draw(R, V, dt, 5, cuda)
    low = torch.finfo(logits.dtype).min
    logits[0, 10:] = -INF
    logits[1, :V - 3] = low
    logits[2] = low
    tokens[0], tokens[1] = 3, V - 1
    check(libwq, logits, tokens, 32)
    logits[0] = -INF
    logits[1] = -INF
    logits[1, 777] = 1.5
    tokens[1] = 777
    got = check(libwq, logits, tokens, 32)
    assert torch.isnan(got["entropy"][0]) and got["top_id"][0].tolist() == list(range(32))
    assert got["logprob"][1] == 0 and got["entropy"][1] == 0 and got["top_id"][1, 0] == 777


@pytest.mark.parametrize("dt", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("R,V", [(3, 20000), (320, 5000)])
def test_not_finite(cuda, libwq, dt, R, V):
    import torch
    logits, tokens = draw(R, V, dt, 6, cuda)
    logits[0, 100] = float("nan")
    logits[1, 101] = INF
    logits[2] = float("nan")
    check(libwq, logits, tokens, 5)


@pytest.mark.parametrize("dt", ["fp16", "fp32"])
@pytest.mark.parametrize("R,V", [(1, 65536), (2, 9000), (320, 33000)])
def test_ties_and_order(cuda, libwq, dt, R, V):
    """Constant rows, ramps, and patterns that put a row's large values on one thread."""
    import torch
    i = torch.arange(V, device=cuda)
    tokens = torch.full((R,), V - 1, device=cuda)
    per = 2048 if dt == "fp16" else 1024   # entries that one round of a CTA's loads covers
    for row in (torch.zeros(V, device=cuda), i / V, -i / V, (i % per) / per, ((i // 8) % 256 == 77).float() * 3,
                (i % per < 5 * 8) * (1 + (i // per) / 100.0), (i % 3).float(), -0.0 * (i % 2)):
        check(libwq, row.expand(R, V).to(_dtype(dt)).contiguous(), tokens, 32)


def test_large_logits(cuda, libwq):
    """Differences of large values are taken before they are scaled."""
    import torch
    logits, tokens = draw(4, 6000, "fp32", 8, cuda)
    logits[0] += 60000
    logits[1] *= 1e30
    logits[2] = 1.5e38 * torch.sign(logits[2])
    check(libwq, logits, tokens, 3)


def test_tokens_outside_and_none(cuda, libwq):
    import torch
    logits, tokens = draw(5, 3000, "bf16", 9, cuda)
    tokens[0], tokens[1], tokens[2] = -1, 3000, -2 ** 62
    got = check(libwq, logits, tokens, 0)
    assert (got["logprob"][:3] == -INF).all()
    only = libwq.logprobs(logits)
    assert set(only) == {"entropy"} and torch.equal(only["entropy"], got["entropy"])


def test_top_agrees_with_tokens_and_repeats(cuda, libwq):
    """The log probability of a top entry is that of the token itself, and a call repeats its bits."""
    import torch
    for R in (1, 400):
        logits, _ = draw(R, 30000, "bf16", 10, cuda)
        a = libwq.logprobs(logits, top_k=8)
        for j in (0, 7):
            b = libwq.logprobs(logits, a["top_id"][:, j].contiguous(), top_k=8)
            assert torch.equal(b["logprob"], a["top_logprob"][:, j])
            assert all(torch.equal(a[n], b[n]) for n in a)


def test_stream_and_graph(cuda, libwq):
    import torch
    logits, tokens = draw(12, 9000, "fp16", 11, cuda)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = libwq.logprobs(logits, tokens, 4, pdl=True)
    logits.copy_(draw(12, 9000, "fp16", 12, cuda)[0])
    graph.replay()
    torch.cuda.synchronize()
    now = check(libwq, logits, tokens, 4)
    assert all(torch.equal(now[n], got[n]) for n in now)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = libwq.logprobs(logits, tokens, 4)
    torch.cuda.synchronize()
    assert all(torch.equal(now[n], other[n]) for n in now)


def test_refusals(cuda, libwq):
    import torch
    logits, tokens = draw(4, 100, "fp32", 1, cuda)
    for bad in (logits.double(), logits.cpu(), logits[0], logits.t(), logits[:, ::2]):
        with pytest.raises((TypeError, ValueError)):
            libwq.logprobs(bad, tokens)
    for bad in (tokens.int(), tokens.cpu(), tokens[:3], tokens[:, None]):
        with pytest.raises((TypeError, ValueError)):
            libwq.logprobs(logits, bad)
    for k in (-1, 33, 101):
        with pytest.raises(ValueError):
            libwq.logprobs(logits, tokens, k)
    with pytest.raises(libwq.WQError):
        libwq.logprobs(logits[:0], tokens[:0])


@pytest.mark.parametrize("M", [2, 40])
def test_decode_step(cuda, libwq, M):
    """Router, experts, quantised LM head and its log probabilities in one captured step: every
    operator against the 64-bit result of what it was given, and the replay against the eager run."""
    import moe_oracle
    import torch
    from test_route_gpu import check as check_route
    D, V, E = 128, 3000, 8
    p = moe_oracle.problem(M, E, 2, D, 96, D, 4, 32, torch.bfloat16, seed=31)
    (x, _, _), w = moe_oracle.to_gpu(libwq, p, 4, cuda)
    g = torch.Generator(device=cuda).manual_seed(3)
    router = torch.randn((D, E), generator=g, device=cuda, dtype=torch.bfloat16)
    head, _ = libwq.pack_kmajor(torch.randint(0, 16, (D, V), generator=g, device=cuda, dtype=torch.uint8), 4)
    s = torch.full((4, V), 0.02, dtype=torch.bfloat16, device=cuda)
    z = torch.full((4, V), 8.0, dtype=torch.bfloat16, device=cuda)
    tokens = torch.randint(0, V, (M,), generator=g, device=cuda)
    plan = libwq.MoePlan(*w, 4, 32, M, 2, pdl=True)

    def step():
        scores = x @ router
        ids, weights = libwq.moe_route(scores, 2, pdl=True)
        y = x + plan(x, ids, weights)
        return scores, ids, weights, y, libwq.matmul_logprobs(y, head, None, s, z, 4, 32, tokens, top_k=4)
    eager = step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    graph.replay()
    torch.cuda.synchronize()
    scores, ids, weights, y, out = eager
    check_route(libwq, scores, 2)
    p["weights"] = weights.cpu()
    ref, tol = moe_oracle.layer(p, 4, "silu", ids.cpu())
    half = torch.finfo(torch.bfloat16).eps / 2
    total = x.double().cpu() + ref
    moe_oracle.assert_close(y, total, tol + (total.abs() + tol) * half)
    logits = libwq.matmul(y, head, None, s, z, 4, 32)
    again = check(libwq, logits, tokens, 4)
    assert all(torch.equal(again[n], out[n]) for n in again)
    for a, b in zip(eager[:4], captured[:4]):
        assert torch.equal(a, b)
    assert all(torch.equal(out[n], captured[4][n]) for n in out)


@pytest.mark.parametrize("R,V", [(17, 16384), (20, 9000), (40, 9001), (100, 9000), (64, 50003), (128, 50000), (300, 49200)])
def test_rows_split_over_ctas(cuda, libwq, R, V):
    """Numbers of rows on both sides of every split of a row: 8, 4, 2 CTAs and one, and more CTAs than SMs."""
    l, tok = draw(R, V, "bf16", R + V, cuda)
    check(libwq, l, tok, 7)
    assert libwq.device_status() == 0
