"""The mixture-of-experts layer against the 64-bit definition (moe_oracle.py has the bound)."""
import subprocess
import sys
from pathlib import Path

import pytest

import moe_oracle
from guard import Guarded

pytestmark = pytest.mark.gpu
ROOT = Path(__file__).resolve().parents[1]

# T, E, k, K, I, N, bits, G, dtype, act, frac
CASES = [
    (1, 1, 1, 8, 8, 8, 4, -1, "fp16", "silu", False),            # one word row
    (1, 3, 2, 4, 8, 16, 8, -1, "bf16", "silu", False),           # one 8-bit word row
    (1, 4, 2, 256, 128, 64, 4, 128, "fp16", "silu", False),
    (1, 8, 8, 512, 384, 520, 4, 128, "bf16", "gelu", False),
    (2, 5, 3, 288, 96, 72, 4, 32, "fp16", "gelu", True),
    (3, 6, 2, 96, 64, 136, 8, 32, "fp16", "silu", True),
    (4, 4, 4, 256, 256, 64, 8, 128, "bf16", "silu", True),       # 4 slots on every expert
    (5, 12, 3, 1112, 744, 1000, 4, -1, "bf16", "gelu", False),   # K ends inside a tile
    (5, 7, 2, 20, 24, 40, 8, -1, "fp16", "silu", False),         # K = 5 word rows
    (8, 2, 2, 320, 160, 96, 4, 32, "fp16", "silu", False),       # 8 slots on every expert
    (9, 3, 3, 384, 128, 64, 4, 128, "bf16", "silu", False),      # 9: a second token tile
    (16, 2, 2, 256, 192, 104, 4, 64, "fp16", "silu", True),      # 16: full blocks
    (17, 1, 1, 128, 64, 64, 4, 64, "bf16", "gelu", False),       # 17 tokens on one expert: two blocks
    (33, 40, 1, 64, 64, 64, 8, 64, "fp16", "silu", False),       # more than 32 slots
    (48, 32, 4, 256, 192, 128, 8, 32, "bf16", "silu", True),
    (64, 16, 16, 64, 32, 64, 4, 32, "fp16", "silu", False),      # 1024 slots, 64 tokens on every expert
    (64, 512, 2, 32, 32, 8, 4, 32, "bf16", "silu", False),       # as many experts as there can be
    (3, 4, 2, 192, 96, 72, 4, 96, "fp16", "silu", True),         # groups of 3 steps, across stages
    (6, 3, 2, 480, 320, 64, 4, 160, "bf16", "gelu", False),      # and of 5
    (20, 4, 2, 192, 96, 72, 8, 96, "fp16", "silu", False),       # more tokens than the warps keep sums for
    (15, 5, 4, 224, 32, 200, 4, 32, "bf16", "silu", False),
    (40, 6, 3, 96, 352, 328, 4, -1, "fp16", "gelu", True),
    (2, 2, 1, 64, 32, 20008, 4, 32, "fp16", "silu", False),      # a column tile per CTA: no cluster
    (24, 3, 1, 32, 64, 12296, 8, 32, "bf16", "silu", False),
    (4, 3, 2, 64, 2080, 136, 8, 32, "bf16", "gelu", False),
    (7, 3, 2, 8256, 32, 16, 4, 32, "bf16", "silu", False),       # a long K: two slots per block
    (2, 2, 1, 20000, 16, 8, 8, -1, "fp16", "silu", False),       # one slot per block
    (6, 2, 1, 64, 6176, 24, 4, 32, "fp16", "silu", True),        # a long inner length: K splits
    (1, 2, 2, 32, 8776, 16, 8, -1, "bf16", "gelu", False),
    (20, 2, 1, 64, 6176, 24, 4, 32, "bf16", "silu", False),      # a block's rows from many warps
    (18, 3, 2, 64, 352, 72, 8, -1, "fp16", "silu", True),
    (40, 16, 16, 32, 32, 19208, 8, 32, "fp16", "silu", False),   # no cluster: the rows are summed a few tokens at a time
]


def _dtype(name):
    import torch
    return {"fp16": torch.float16, "bf16": torch.bfloat16}[name]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "T{}E{}k{}_{}x{}x{}_{}b_G{}_{}_{}".format(*c[:10]))
def test_layer(cuda, libwq, case):
    import torch
    T, E, k, K, I, N, bits, G, dt, act, frac = case
    p = moe_oracle.problem(T, E, k, K, I, N, bits, G, _dtype(dt), seed=T * 1000 + K + N, frac=frac)
    ref, tol = moe_oracle.layer(p, bits, act)
    (x, ids, weights), w = moe_oracle.to_gpu(libwq, p, bits, cuda)
    out = Guarded((T, N), x.dtype, cuda)
    y = libwq.moe(x, ids, weights, *w, bits, G, activation=act, out=out.view)
    torch.cuda.synchronize()
    assert out.intact()
    moe_oracle.assert_close(y, ref, tol, str(case))
    plan = libwq.MoePlan(*w, bits, G, T, k, activation=act, pdl=True)
    assert torch.equal(plan(x, ids, weights), y)                 # the same bits, and again
    assert libwq.device_status() == 0


def test_fewer_tokens_than_the_plan(cuda, libwq):
    """A plan for 64 tokens takes any smaller batch; a token's row does not depend on the others."""
    import torch
    p = moe_oracle.problem(20, 6, 2, 128, 64, 72, 4, 32, torch.float16, seed=5)
    ref, tol = moe_oracle.layer(p, 4, "silu")
    (x, ids, weights), w = moe_oracle.to_gpu(libwq, p, 4, cuda)
    plan = libwq.MoePlan(*w, 4, 32, 64, 2)
    for T in (1, 4, 5, 8, 9, 16, 17, 20):
        y = plan(x[:T], ids[:T], weights[:T])
        moe_oracle.assert_close(y, ref[:T], tol[:T], f"T={T}")


@pytest.mark.parametrize("T", [6, 40])
def test_empty_slots(cuda, libwq, T):
    """Ids outside the experts add nothing; a token without slots, and a batch without any, give zeros."""
    import torch
    p = moe_oracle.problem(T, 5, 3, 96, 64, 40, 4, 32, torch.bfloat16, seed=8)
    ids = p["ids"].clone()
    ids[0] = -1
    ids[1, 1] = 5
    ids[2, 0] = 2 ** 31 - 1
    ids[3, 2] = -2 ** 31
    ids[-1] = torch.tensor([-1, 7, -3])
    ref, tol = moe_oracle.layer(p, 4, "silu", ids)
    (x, _, weights), w = moe_oracle.to_gpu(libwq, p, 4, cuda)
    weights[0] = float("nan")                                    # an empty slot's weight is not read
    y = libwq.moe(x, ids.to(cuda), weights, *w, 4, 32)
    moe_oracle.assert_close(y, ref, tol)
    assert (y[0] == 0).all() and (y[-1] == 0).all()
    none = libwq.moe(x, torch.full_like(ids, -1).to(cuda), weights, *w, 4, 32, out=torch.ones_like(y))
    assert (none == 0).all()


@pytest.mark.parametrize("T", [4, 12, 24])
def test_the_same_expert_twice(cuda, libwq, T):
    import torch
    p = moe_oracle.problem(T, 4, 3, 64, 32, 64, 8, 32, torch.float16, seed=9)
    ids = p["ids"].clone()
    ids[:, 2] = ids[:, 0]
    ids[1] = 3
    ref, tol = moe_oracle.layer(p, 8, "silu", ids)
    (x, _, weights), w = moe_oracle.to_gpu(libwq, p, 8, cuda)
    moe_oracle.assert_close(libwq.moe(x, ids.to(cuda), weights, *w, 8, 32), ref, tol)


def test_extreme_zero_points_and_scales(cuda, libwq):
    """Zero points far outside the codes, negative and zero scales, and codes equal to z."""
    import torch
    p = moe_oracle.problem(3, 3, 2, 128, 96, 48, 4, 32, torch.float16, seed=11)
    for name in ("up", "down"):
        codes, s, z = p[name]
        z[0, 0] = 300.0
        z[1, 1] = -77.5
        s[1] = -s[1]
        s[2, 0] = 0.0
    ref, tol = moe_oracle.layer(p, 4, "gelu")
    (x, ids, weights), w = moe_oracle.to_gpu(libwq, p, 4, cuda)
    moe_oracle.assert_close(libwq.moe(x, ids, weights, *w, 4, 32, activation="gelu"), ref, tol)


@pytest.mark.parametrize("dt", ["fp16", "bf16"])
def test_values_of_very_different_size(cuda, libwq, dt):
    """Blocks with one large value, tiny blocks, zeros, and the type's own limits."""
    import torch
    p = moe_oracle.problem(5, 3, 2, 512, 64, 48, 4, 32, _dtype(dt), seed=14)
    info = torch.finfo(p["x"].dtype)
    p["x"][0, 7] = 2000.0
    p["x"][1, 128:256] *= 2.0 ** -12
    p["x"][2] = 0
    p["x"][3, ::3] = 0
    p["x"][4] = (p["x"][4].float() * (info.max / 1e6 if dt == "fp16" else 1e-30)).to(p["x"].dtype)
    ref, tol = moe_oracle.layer(p, 4, "silu")
    (x, ids, weights), w = moe_oracle.to_gpu(libwq, p, 4, cuda)
    y = libwq.moe(x, ids, weights, *w, 4, 32)
    moe_oracle.assert_close(y, ref, tol)
    assert (y[2] == 0).all()


def test_the_largest_values(cuda, libwq):
    """bf16 values next to the type's maximum: the fixed-point step has the next exponent.  With
    s = 2^-75 gate and up stay below 32 * 16 * 2^128 * 2^-75 = 2^62, so h below 2^124 is in fp32's
    range (with 2^-70 it is not: the 64-bit h of these inputs reaches 1.36e39)."""
    import torch
    p = moe_oracle.problem(2, 1, 1, 32, 32, 8, 4, 32, torch.bfloat16, seed=15)
    p["x"][:] = torch.finfo(torch.bfloat16).max
    p["x"][1] *= -1
    for name in ("up", "down"):
        p[name][1].fill_(2.0 ** -75)
    ref, tol = moe_oracle.layer(p, 4, "gelu")
    (x, ids, weights), w = moe_oracle.to_gpu(libwq, p, 4, cuda)
    y = libwq.moe(x, ids, weights, *w, 4, 32, activation="gelu")
    assert torch.isfinite(y).all()
    moe_oracle.assert_close(y, ref, tol)


def test_hidden_values_beyond_fp16(cuda, libwq):
    """h above 65504 in an fp16 layer: the values between the two products keep fp32's range."""
    import torch
    p = moe_oracle.problem(2, 2, 1, 64, 32, 32, 4, 32, torch.float16, seed=12)
    p["x"] *= 300
    p["down"] = (p["down"][0], (p["down"][1].float() * 2 ** -8).half(), p["down"][2])
    ref, tol = moe_oracle.layer(p, 4, "silu")
    (x, ids, weights), w = moe_oracle.to_gpu(libwq, p, 4, cuda)
    y = libwq.moe(x, ids, weights, *w, 4, 32)
    assert torch.isfinite(y).all()
    moe_oracle.assert_close(y, ref, tol)


@pytest.mark.parametrize("T", [5, 20])
def test_a_row_that_is_not_finite_stays_alone(cuda, libwq, T):
    import torch
    p = moe_oracle.problem(T, 2, 2, 64, 32, 64, 4, 32, torch.bfloat16, seed=13)
    ref, tol = moe_oracle.layer(p, 4, "silu")
    (x, ids, weights), w = moe_oracle.to_gpu(libwq, p, 4, cuda)
    x[1, 3] = float("nan")
    x[3, 0] = float("inf")
    y = libwq.moe(x, ids, weights, *w, 4, 32)
    keep = [t for t in range(T) if t not in (1, 3)]
    assert torch.isnan(y[1]).all() and torch.isnan(y[3]).all()
    moe_oracle.assert_close(y[keep], ref[keep], tol[keep])


def test_streams_and_graphs(cuda, libwq):
    """Calls on two streams at once, and two captured graphs replayed at once, do not share a workspace."""
    import torch
    ps = [moe_oracle.problem(16, 8, 2, 256, 128, 256, 4, 64, torch.float16, seed=s) for s in (21, 22)]
    refs = [moe_oracle.layer(p, 4, "silu") for p in ps]
    runs = []
    for p in ps:
        (x, ids, weights), w = moe_oracle.to_gpu(libwq, p, 4, cuda)
        runs.append((libwq.MoePlan(*w, 4, 64, 16, 2, pdl=True), x, ids, weights))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    ys = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                plan, *a = runs[i]
                ys[i].append(plan(*a))
    torch.cuda.synchronize()
    graphs, outs = [], []
    for plan, *a in runs:
        gph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gph):
            outs.append(plan(*a))
        graphs.append(gph)
    runs[0][1].mul_(0.5)                                         # a replay reads the inputs anew
    ps[0]["x"] = ps[0]["x"] * 0.5
    refs.append(moe_oracle.layer(ps[0], 4, "silu"))
    torch.cuda.synchronize()
    for _ in range(10):
        for gph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                gph.replay()
    torch.cuda.synchronize()
    for i in range(2):
        for y in ys[i]:
            assert torch.equal(y, ys[i][0])
        moe_oracle.assert_close(ys[i][0], *refs[i])
    moe_oracle.assert_close(outs[0], *refs[2])
    moe_oracle.assert_close(outs[1], *refs[1])


@pytest.mark.parametrize("T", [1, 12, 24])
def test_first_call_is_captured(cuda, T):
    """A process whose first call of the layer is recorded in a graph; the replays give the eager bits."""
    code = f"""
import sys
sys.path.insert(0, "tests")
import torch, moe_oracle
import gemm_wq_gemv_b200 as wq
p = moe_oracle.problem({T}, 6, 2, 256, 128, 136, 4, 64, torch.bfloat16, seed=31)
ref, tol = moe_oracle.layer(p, 4, "silu")
dev = torch.device("cuda:0")
a, w = moe_oracle.to_gpu(wq, p, 4, dev)
plan = wq.MoePlan(*w, 4, 64, {T}, 2, pdl=True)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    y = plan(*a)
for _ in range(3):
    y.zero_()
    g.replay()
    torch.cuda.synchronize()
    moe_oracle.assert_close(y, ref, tol)
assert torch.equal(y, plan(*a)) and wq.device_status() == 0
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout + r.stderr


def test_two_graphs_of_one_plan(cuda, libwq):
    """More tokens than the warps keep sums for: two graphs of one plan, replayed at once on two streams, leave
    their rows in workspaces of their own."""
    import torch
    p = moe_oracle.problem(24, 6, 3, 128, 352, 136, 8, 32, torch.bfloat16, seed=41)
    ref, tol = moe_oracle.layer(p, 8, "silu")
    (x, ids, weights), w = moe_oracle.to_gpu(libwq, p, 8, cuda)
    plan = libwq.MoePlan(*w, 8, 32, 24, 3, pdl=True)
    want = plan(x, ids, weights)
    flipped = plan(x.flip(0).contiguous(), ids.flip(0).contiguous(), weights.flip(0).contiguous())
    moe_oracle.assert_close(want, ref, tol)
    runs = []
    for a in ((x, ids, weights), (x.flip(0).contiguous(), ids.flip(0).contiguous(), weights.flip(0).contiguous())):
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(4):
                y = plan(*a)
        runs.append((g, y, a, torch.cuda.Stream()))
    for _ in range(10):
        for g, _, _, s in runs:
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert torch.equal(runs[0][1], want) and torch.equal(runs[1][1], flipped)
    assert libwq.device_status() == 0


def test_refusals(cuda, libwq):
    import torch
    p = moe_oracle.problem(2, 4, 2, 64, 32, 32, 4, 32, torch.float16, seed=1)
    (x, ids, weights), w = moe_oracle.to_gpu(libwq, p, 4, cuda)
    plan = libwq.MoePlan(*w, 4, 32, 2, 2)
    bad = [(x.bfloat16(), ids, weights), (x, ids.long(), weights), (x, ids, weights.half()), (x.cpu(), ids, weights),
           (x[:, :32].contiguous(), ids, weights), (x, ids[:, :1].contiguous(), weights),
           (torch.cat([x, x]), torch.cat([ids, ids]), torch.cat([weights, weights])),
           (x[:0], ids[:0], weights[:0]), (x.t(), ids, weights)]
    for a in bad:
        with pytest.raises((TypeError, ValueError)):
            plan(*a)
    with pytest.raises(ValueError):
        plan(x, ids, weights, out=torch.empty((2, 40), dtype=x.dtype, device=cuda))
    for bits, G in ((3, 32), (4, 24), (4, 0), (8, 32), (4, 64)):
        with pytest.raises((ValueError, libwq.WQError)):
            libwq.moe(x, ids, weights, *w, bits, G)
    with pytest.raises(ValueError):
        libwq.moe(x, ids, weights, *w, 4, 32, activation="relu")
    with pytest.raises(ValueError):
        libwq.moe(x, ids, weights, w[0], w[1], w[2], w[3][:3].contiguous(), w[4], w[5], 4, 32)
    with pytest.raises(ValueError):
        libwq.moe(x, ids, weights, w[0], w[1][:, :1].contiguous(), w[2], *w[3:], 4, 32)
    with pytest.raises(ValueError):
        libwq.MoePlan(*w, 4, 32, 65, 2)
    with pytest.raises(libwq.WQError) as e:                       # groups of 16: four word rows cover two groups
        p16 = moe_oracle.problem(2, 4, 2, 64, 32, 32, 4, 16, torch.float16, seed=1)
        a16, w16 = moe_oracle.to_gpu(libwq, p16, 4, cuda)
        libwq.moe(*a16, *w16, 4, 16)
    assert e.value.status == 2
