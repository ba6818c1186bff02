"""The router, the expert layer and the log probabilities allocate nothing: with every output and the workspace
given, calls leave the device's free memory as it was, and two streams can make them at once."""
import ctypes

import pytest

import moe_grouped
import moe_oracle

pytestmark = pytest.mark.gpu


class Step:
    """One decode step through the C calls, into buffers of its own."""

    def __init__(self, wq, dev, T, seed):
        import torch
        self.E, self.k, self.K, self.I, self.N, self.V, self.T = 8, 3, 256, 128, 264, 5003, T
        self.p = moe_oracle.problem(T, self.E, self.k, self.K, self.I, self.N, 4, 64, torch.float16, seed)
        (self.x, _, _), self.w = moe_oracle.to_gpu(wq, self.p, 4, dev)
        g = torch.Generator().manual_seed(seed)
        self.gate = torch.randn((T, self.E), generator=g).to(dev)
        self.logits = torch.randn((T, self.V), generator=g).to(dev)
        self.tokens = torch.randint(0, self.V, (T,), generator=g).to(dev)
        self.ids = torch.empty((T, self.k), dtype=torch.int32, device=dev)
        self.weights = torch.empty((T, self.k), device=dev)
        self.y = torch.empty((T, self.N), dtype=torch.float16, device=dev)
        self.lp, self.ent = torch.empty(T, device=dev), torch.empty(T, device=dev)
        self.top, self.top_id = torch.empty((T, 4), device=dev), torch.empty((T, 4), dtype=torch.int64, device=dev)
        self.nbytes = wq.lib().wq_moe_workspace_size(T, self.k, self.I, self.N)
        self.ws = torch.empty(self.nbytes, dtype=torch.uint8, device=dev)

    def run(self, L, stream):
        T, a = self.T, [t.data_ptr() for t in (self.x, self.ids, self.weights, *self.w, self.y)]
        assert L.wq_moe_route(self.gate.data_ptr(), 2, T, self.E, self.E, self.k, 1, ctypes.c_float(1.0),
                              self.ids.data_ptr(), self.weights.data_ptr(), 0, stream) == 0
        assert L.wq_moe(*a, T, self.K, self.I, self.N, self.E, self.k, 4, 64, 0, 1, self.ws.data_ptr(),
                        ctypes.c_size_t(self.nbytes), stream) == 0
        assert L.wq_logprobs(self.logits.data_ptr(), 2, T, self.V, self.V, self.tokens.data_ptr(), 4,
                             self.lp.data_ptr(), self.ent.data_ptr(), self.top.data_ptr(), self.top_id.data_ptr(),
                             1, stream) == 0

    def outputs(self):
        return [t.clone() for t in (self.ids, self.weights, self.y, self.lp, self.ent, self.top, self.top_id)]


def test_no_device_memory_taken_per_call(cuda, libwq):
    import torch
    L, steps = libwq.lib(), [Step(libwq, cuda, T, seed=T) for T in (1, 6, 20)]
    stream = torch.cuda.current_stream().cuda_stream
    for s in steps:
        s.run(L, stream)
    torch.cuda.synchronize()
    free = torch.cuda.mem_get_info(cuda)[0]
    for _ in range(3):
        for s in steps:
            s.run(L, stream)
    torch.cuda.synchronize()
    assert torch.cuda.mem_get_info(cuda)[0] == free
    for s in steps:
        ref = moe_grouped.layer(dict(s.p, ids=s.ids.cpu(), weights=s.weights.cpu()), 4, "silu")
        moe_oracle.assert_close(s.y, *ref)
    assert libwq.device_status() == 0


def test_two_streams_at_once(cuda, libwq):
    import torch
    L, steps = libwq.lib(), [Step(libwq, cuda, 20, seed=5), Step(libwq, cuda, 20, seed=6)]
    want = []
    for s in steps:
        s.run(L, torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        want.append(s.outputs())
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        for s, t in zip(steps, streams):
            s.run(L, t.cuda_stream)
    torch.cuda.synchronize()
    for s, w in zip(steps, want):
        assert all(torch.equal(a, b) for a, b in zip(s.outputs(), w))
    assert libwq.device_status() == 0
