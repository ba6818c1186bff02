"""The expert layer for more than 16 tokens and many output columns: few CTAs per tile
of columns, each of which stages up to 192 rows (tests/test_moe_smem_cpu.py has the bytes)."""
import pytest

import moe_grouped
import moe_oracle
from guard import Guarded

pytestmark = pytest.mark.gpu

# T, E, k, K, I, N, bits, G, dtype, act, frac: 4-bit words with groups of 128 or per column, 8-bit words with groups of
# 64 or more have the smallest rings, which the staged rows outgrow
WIDE = [
    (48, 16, 8, 128, 128, 8192, 4, 128, "fp16", "silu", False),
    (48, 8, 4, 128, 256, 16384, 4, 128, "bf16", "gelu", True),
    (64, 12, 6, 96, 160, 8192, 4, -1, "bf16", "silu", False),
    (64, 7, 3, 64, 64, 19208, 8, 64, "fp16", "silu", False),
    (24, 9, 8, 32, 64, 18952, 8, 32, "fp16", "gelu", False),
    (17, 11, 11, 40, 72, 24000, 8, -1, "bf16", "silu", True),
]


def _dtype(name):
    import torch
    return {"fp16": torch.float16, "bf16": torch.bfloat16}[name]


@pytest.mark.parametrize("case", WIDE, ids=lambda c: "T{}E{}k{}_{}x{}x{}_{}b_G{}_{}_{}".format(*c[:10]))
def test_staged_rows(cuda, libwq, case):
    import torch
    T, E, k, K, I, N, bits, G, dt, act, frac = case
    p = moe_oracle.problem(T, E, k, K, I, N, bits, G, _dtype(dt), seed=T + K + N, frac=frac)
    ref, tol = moe_grouped.layer(p, bits, act)
    (x, ids, weights), w = moe_oracle.to_gpu(libwq, p, bits, cuda)
    out = Guarded((T, N), x.dtype, cuda)
    y = libwq.moe(x, ids, weights, *w, bits, G, activation=act, out=out.view)
    torch.cuda.synchronize()
    assert out.intact() and libwq.device_status() == 0
    moe_oracle.assert_close(y, ref, tol, str(case))
    assert torch.equal(libwq.moe(x, ids, weights, *w, bits, G, activation=act, pdl=True), y)


@pytest.mark.parametrize("T,E,k,K,I,N,bits,G", [(1, 2, 16, 256, 128, 72, 4, 128), (4, 2, 16, 64, 64, 40, 8, 32),
                                               (3, 1, 5, 96, 96, 64, 4, 96), (64, 1, 2, 8192, 32, 16, 4, 32),
                                               (64, 3, 16, 128, 64, 136, 8, -1), (7, 2, 16, 4096, 64, 520, 4, 64)])
def test_more_slots_than_experts(cuda, libwq, T, E, k, K, I, N, bits, G):
    """An expert several times among a token's slots, and empty ones between them: blocks of any length."""
    import torch
    p = moe_oracle.problem(T, E, 1, K, I, N, bits, G, torch.float16, seed=T + K + k)
    g = torch.Generator().manual_seed(T + k)
    p["ids"] = torch.randint(-1, E, (T, k), generator=g).to(torch.int32)
    p["weights"] = torch.softmax(torch.randn((T, k), generator=g), 1)
    ref, tol = moe_grouped.layer(p, bits, "silu")
    (x, ids, weights), w = moe_oracle.to_gpu(libwq, p, bits, cuda)
    out = Guarded((T, N), x.dtype, cuda)
    y = libwq.moe(x, ids, weights, *w, bits, G, out=out.view)
    torch.cuda.synchronize()
    assert out.intact() and libwq.device_status() == 0
    moe_oracle.assert_close(y, ref, tol)
