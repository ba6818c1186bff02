"""Rows so long that a thread's sums in fp32 would lose digits to their length.

Two values in turn, so that every addition of a sum rounds the same way for a long stretch: one chain of V / 2048
additions is off by 4e-4 at V = 2^28 and 1e-3 at 2^29 (added up in fp32 on the host).  Bound, u = 2^-24, as in
test_logprobs_gpu.py with other counts of additions: a thread adds at most 1024 terms into a sum, that into its total
(V / 2^18 of them with a CTA per row), then 64 more over warps, CTA and cluster:
  r = (2 + 2 (D + 10) + 1088 + V / 2^18) u for ln S1,  D = sum p |d|, |d| <= |l - max| + 8."""
import math

import pytest

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.mark.parametrize("R,V,dt,lo", [(1, 1 << 29, "bf16", -1.0), (1, 1 << 28, "fp16", -0.5),
                                       (2, (1 << 28) + 1, "bf16", -1.0), (1, (1 << 28) - 3, "fp32", -1.0),
                                       (5, 1 << 24, "fp32", -3.0)])
def test_long_rows(cuda, libwq, R, V, dt, lo):
    import torch
    dtype = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}[dt]
    logits = torch.zeros((R, V), dtype=dtype, device=cuda)
    logits[:, 1::2] = lo
    tokens = torch.tensor([V - 1] * R, device=cuda)
    out = libwq.logprobs(logits, tokens, top_k=2)
    n1 = V // 2
    Z = (V - n1) + n1 * math.exp(lo)
    p1 = n1 * math.exp(lo) / Z
    H = math.log(Z) - p1 * lo
    D, D2 = p1 * (8 - lo) + (1 - p1) * 8, p1 * (8 - lo) ** 2 + (1 - p1) * 64
    steps = 1088 + V / 2 ** 18
    r = (2 + 2 * (D + 10) + steps) * U
    tol = r + U * (3 * 8 - 2 * lo + 8 + 2 * math.log(Z))
    tol_h = r + ((2 + steps) * D + 2 * (D2 + 10 * D) + 2 * (H + D)) * U + r * D
    want = (lo if (V - 1) % 2 else 0.0) - math.log(Z)
    assert (out["logprob"].double() - want).abs().max().item() <= tol
    assert (out["entropy"].double() - H).abs().max().item() <= tol_h
    assert out["top_id"].tolist() == [[0, 2]] * R
    assert (out["top_logprob"].double() + math.log(Z)).abs().max().item() <= tol
