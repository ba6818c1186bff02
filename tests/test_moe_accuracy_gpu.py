"""What the expert layer loses of x and h, against a bound that leaves fp32's share only.

Bound of a product with row a, |a| <= A in a block of 128 values, u = 2^-24, w = (q - z) s.  A value is held in fixed
point to half of 2^-22 of the power of two below A (the next one from 1.984 of it on): 1.02 * 2^-23 A at most.  It is
256 (256 hi + mid) + lo with |256^2 hi| + |256 mid| + |lo| <= 3 |value| (128 = 256 - 128 is the worst).  The three sums
over q, and the sum X of the values, are exact integers; joining the three rounds twice (3 u and 1 u of sum |a| q), X
and D - z X once each, the product with s and the step once, the additions of up to K / 32 folds and 8 warps once each,
and the fixed-point values stand for those of a: 4 u sum |a| (q + |z|) s + (12 + K / 32) u sum |a w|.  The rest as
moe_oracle has it.

An outlier in x (or h) whose codes equal their zero point, or whose group's scale is 0, adds nothing to the output: the
rest of its block is the output, and has to come out as in fp32."""
import pytest

import moe_grouped
import moe_oracle
from moe_oracle import U

pytestmark = pytest.mark.gpu


def product(a, da, codes, s, z, bits):
    """moe_oracle's product with fp32's share alone."""
    import torch
    K, groups = codes.shape[0], s.shape[0]
    q, grp = codes.double(), torch.arange(K, device=a.device) // (K // groups)
    sd, zd = s.double()[grp], z.double()[grp]
    w = (q - zd) * sd
    top = torch.nn.functional.pad(a.abs() + da, (0, -K % 128)).view(len(a), -1, 128).amax(2)
    da = da + 1.02 * 2.0 ** -23 * top.repeat_interleave(128, 1)[:, :K]
    mag = a.abs() @ ((q + zd.abs()) * sd.abs())
    return a @ w, U * (4 * mag + (12 + K / 32) * (a.abs() @ w.abs())) + da @ w.abs()


def _dtype(name):
    import torch
    return {"fp16": torch.float16, "bf16": torch.bfloat16}[name]


def outliers(T, K, I, N, bits, G, dt, ratio, seed, silent):
    """A layer with one value of every 128 of x `ratio` times the rest; silent: its codes at the zero point, and each
    column of the second product takes one hidden value (all other codes at the zero point)."""
    import torch
    p = moe_oracle.problem(T, 4, 2, K, I, N, bits, G, _dtype(dt), seed=seed)
    g = torch.Generator().manual_seed(seed)
    for b in range(0, K, 128):
        at = b + int(torch.randint(0, min(128, K - b), (1,), generator=g))
        p["x"][:, at] = (p["x"][:, at].float().sign() * ratio).to(p["x"].dtype)
        if silent:
            codes, s, z = p["up"]
            grp = at // (K // s.shape[1])
            z[:, grp] = z[:, grp].clamp(0, 2 ** bits - 1)
            codes[:, at] = z[:, grp].to(codes.dtype)
    if silent:
        codes, s, z = p["down"]
        z.clamp_(0, 2 ** bits - 1)
        one = torch.arange(N) % I
        keep = codes[:, one, torch.arange(N)]
        codes[:] = z.repeat_interleave(I // s.shape[1], 1).to(codes.dtype)
        codes[:, one, torch.arange(N)] = keep
    return p


def run(libwq, p, bits, G, act, cuda):
    import torch
    (x, ids, weights), w = moe_oracle.to_gpu(libwq, p, bits, cuda)
    y = libwq.moe(x, ids, weights, *w, bits, G, activation=act)
    torch.cuda.synchronize()
    assert libwq.device_status() == 0
    return y


SHAPES = [(1, 512, 256, 136, 4, 128), (4, 1112, 744, 72, 4, -1), (6, 512, 256, 264, 4, 64), (9, 384, 352, 104, 8, 32),
          (16, 640, 384, 128, 8, 128), (20, 256, 512, 72, 4, 32), (48, 512, 128, 136, 8, -1),
          (33, 480, 320, 64, 4, 160), (3, 576, 192, 72, 4, 96), (12, 320, 448, 136, 8, 64), (22, 288, 96, 64, 8, 96), (2, 64, 40, 2056, 8, -1)]


@pytest.mark.parametrize("ratio", [1, 300, 3000, 60000])
@pytest.mark.parametrize("dt", ["fp16", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "T{}_{}x{}x{}_{}b_G{}".format(*s))
def test_a_large_value_that_adds_nothing(cuda, libwq, shape, dt, ratio):
    T, K, I, N, bits, G = shape
    p = outliers(T, K, I, N, bits, G, dt, ratio, seed=T + K + ratio, silent=True)
    ref, tol = moe_grouped.layer(p, bits, "silu", product)
    moe_oracle.assert_close(run(libwq, p, bits, G, "silu", cuda), ref, tol, str(shape))


@pytest.mark.parametrize("dt", ["fp16", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "T{}_{}x{}x{}_{}b_G{}".format(*s))
def test_large_values_that_add(cuda, libwq, shape, dt):
    T, K, I, N, bits, G = shape
    p = outliers(T, K, I, N, bits, G, dt, 40, seed=3 * T + K, silent=False)
    ref, tol = moe_grouped.layer(p, bits, "gelu", product)
    moe_oracle.assert_close(run(libwq, p, bits, G, "gelu", cuda), ref, tol, str(shape))


@pytest.mark.parametrize("T", [2, 7, 24])
def test_a_large_hidden_value_in_a_silent_group(cuda, libwq, T):
    """One hidden value of a block is about 3000 times the rest, and its group of the down product has scale 0."""
    import torch
    p = moe_oracle.problem(T, 3, 2, 256, 256, 104, 4, 32, torch.float16, seed=60 + T)
    p["up"][1][:, :, 256 + 37] *= 60                              # the up column of hidden value 37
    p["up"][1][:, :, 37] *= 50
    p["down"][1][:, 1] = 0                                        # group of 32 .. 63
    ref, tol = moe_grouped.layer(p, 4, "silu", product)
    moe_oracle.assert_close(run(libwq, p, 4, 32, "silu", cuda), ref, tol)


@pytest.mark.parametrize("T,K,I,bits,G", [(3, 24576, 32, 4, 32), (20, 24576, 32, 4, 32), (2, 24572, 8, 8, -1),
                                         (9, 12288, 64, 8, 64), (1, 8192, 64, 4, 64), (6, 64, 12320, 4, 32),
                                         (3, 64, 12296, 8, -1)])
def test_long_rows(cuda, libwq, T, K, I, bits, G):
    """The longest K there can be (few slots per block, 8 warps with one CTA per SM), and long inner lengths."""
    import torch
    p = moe_oracle.problem(T, 3, 2, K, I, 40, bits, G, torch.bfloat16, seed=T + K + I)
    ref, tol = moe_grouped.layer(p, bits, "silu", product)
    moe_oracle.assert_close(run(libwq, p, bits, G, "silu", cuda), ref, tol)


@pytest.mark.parametrize("bits,G", [(4, 32), (8, -1)])
def test_the_longest_rows_and_the_most_slots(cuda, libwq, bits, G):
    import torch
    p = moe_oracle.problem(64, 16, 16, 24576, 32, 8, bits, G, torch.float16, seed=77)
    y = run(libwq, p, bits, G, "silu", cuda)
    on = {n: tuple(t.to(cuda) for t in v) if isinstance(v, tuple) else v.to(cuda) if isinstance(v, torch.Tensor) else v
          for n, v in p.items()}
    ref, tol = moe_grouped.layer(on, bits, "silu", product)
    moe_oracle.assert_close(y, ref.cpu(), tol.cpu())


@pytest.mark.parametrize("dt", ["fp16", "bf16"])
@pytest.mark.parametrize("T,E,k,K,I,N,bits,G", [
    (1, 64, 8, 2048, 1024, 2048, 4, 128), (12, 8, 2, 2048, 1408, 2048, 4, 128), (40, 16, 4, 2048, 768, 2048, 8, 128),
    (64, 16, 8, 4096, 512, 8192, 4, 128), (5, 4, 2, 8192, 1024, 4096, 4, 64), (3, 6, 2, 4096, 2048, 4096, 8, -1)])
def test_layers_of_usual_sizes(cuda, libwq, T, E, k, K, I, N, bits, G, dt):
    import torch
    p = moe_oracle.problem(T, E, k, K, I, N, bits, G, _dtype(dt), seed=T + K + I)
    y = run(libwq, p, bits, G, "silu", cuda)
    on = {n: tuple(t.to(cuda) for t in v) if isinstance(v, tuple) else v.to(cuda) if isinstance(v, torch.Tensor) else v
          for n, v in p.items()}
    ref, tol = moe_grouped.layer(on, bits, "silu", product)
    moe_oracle.assert_close(y, ref.cpu(), tol.cpu())
    # rounding y is all that shows: nearly every value is the nearest one
    same = (y.cpu() == ref.cpu().to(y.dtype)).float().mean()
    assert same > (0.99 if dt == "fp16" else 0.998), float(same)
