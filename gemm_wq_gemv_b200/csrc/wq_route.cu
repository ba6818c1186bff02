// wq_route.cu -- expert router: the top_k of a row of logits and their softmax weights.
//
// What is computed: for row l over E experts, the top_k experts in the order
// (logit descending, index ascending) and w = scale * exp(l_e - max) / sum, the
// sum over the chosen experts or over all of them; -inf and NaN are never
// chosen.
//
// How.  One warp per row, its E <= 512 logits in registers (lane + 32 r), so a
// row is read once and nothing is shared.  top_k rounds: each lane offers its
// best remaining entry, one redux finds the largest key and a second the lowest
// index that holds it.  The row is a few hundred bytes: a call is bound by
// launch latency for a few tokens, and by the rounds (two reductions each, which
// wait for each other) for many.  Measured (B200, device time): 1 row of 64 fp32
// logits, 8 chosen, 2.2 us; 8192 rows of 128 bf16, 8 chosen, 6.7 us for 2.6 MB
// (0.4 us at copy rate); 1000 rows of 500 fp16, 10 chosen, 5.5 us.
#include <cuda_runtime.h>

#include "wq_internal.h"
#include "wq_logits.cuh"
#include "wq_ptx.cuh"

namespace wq {
namespace {

constexpr int RW = 8;  // rows (warps) per CTA

struct RouteParams {
    const void* logits;
    int T, E, top_k, renormalize;
    long long ld;
    float scale;
    int32_t* ids;
    float* weights;
};

// R: logits per lane (E <= 32 R).
template <int TYPE, int R>
__global__ void __launch_bounds__(RW * 32) route_kernel(const RouteParams p) {
    using L = Logit<TYPE>;
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int row = blockIdx.x * RW + (threadIdx.x >> 5);
    if (row >= p.T) return;
    const typename L::raw* src = static_cast<const typename L::raw*>(p.logits) + (size_t)row * p.ld;
    float v[R];
    uint32_t key[R];
    bool nan = false;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int e = lane + 32 * r;
        v[r] = e < p.E ? L::load(src + e) : -INFINITY;
        nan |= v[r] != v[r];
        const uint32_t k = order_key(v[r]);
        key[r] = k > KEY_NEG_INF ? k : 0u;  // 0: not to be chosen
    }
    nan = __any_sync(0xffffffffu, nan);
    // the lane's best entry: largest key, lowest index
    uint32_t best;
    int at;
    auto offer = [&]() {
        best = key[0];
        at = 0;
#pragma unroll
        for (int r = 1; r < R; ++r)
            if (key[r] > best) {
                best = key[r];
                at = r;
            }
    };
    offer();
    float m = 0.0f, mine = 0.0f;  // the row's maximum; lane j: exp(l - m) of choice j
    int my_id = -1;
    for (int j = 0; j < p.top_k; ++j) {
        const uint32_t top = __reduce_max_sync(0xffffffffu, best);
        if (top == 0) break;
        const int e = lane + 32 * at;
        const int id = __reduce_min_sync(0xffffffffu, best == top ? (unsigned)e : 0xFFFFFFFFu);
        const float val = key_value(top);
        if (j == 0) m = val;
        if (lane == j) {
            my_id = id;
            mine = expf(val - m);
        }
        if (best == top && e == id) {
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (r == at) key[r] = 0;
            offer();
        }
    }
    float sum = mine;
    if (!p.renormalize) {
        sum = 0.0f;
#pragma unroll
        for (int r = 0; r < R; ++r) sum += v[r] > -INFINITY ? expf(v[r] - m) : 0.0f;
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if (lane < p.top_k) {
        const size_t o = (size_t)row * p.top_k + lane;
        p.ids[o] = my_id;
        p.weights[o] = my_id < 0 ? 0.0f : nan ? NAN : __fdiv_rn(mine, sum) * p.scale;
    }
}

template <int TYPE>
wq_status run_route(const RouteParams& p, bool pdl, cudaStream_t s) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((p.T + (long long)RW - 1) / RW));
    cfg.blockDim = dim3(RW * 32);
    cfg.stream = s;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = pdl ? 1 : 0;
    if (p.E <= 32) return from_cuda(cudaLaunchKernelEx(&cfg, route_kernel<TYPE, 1>, p));
    if (p.E <= 64) return from_cuda(cudaLaunchKernelEx(&cfg, route_kernel<TYPE, 2>, p));
    if (p.E <= 128) return from_cuda(cudaLaunchKernelEx(&cfg, route_kernel<TYPE, 4>, p));
    if (p.E <= 256) return from_cuda(cudaLaunchKernelEx(&cfg, route_kernel<TYPE, 8>, p));
    return from_cuda(cudaLaunchKernelEx(&cfg, route_kernel<TYPE, 16>, p));
}

}  // namespace

wq_status launch_moe_route(const void* logits, int type, int T, int E, long long ld, int top_k, int renormalize,
                           float scale, int32_t* ids, float* weights, unsigned flags, cudaStream_t s) {
    const RouteParams p{logits, T, E, top_k, renormalize, ld, scale, ids, weights};
    const bool pdl = (flags & WQ_FLAG_PDL) != 0;
    if (type == WQ_TYPE_F32) return run_route<WQ_TYPE_F32>(p, pdl, s);
    if (type == WQ_TYPE_F16) return run_route<WQ_TYPE_F16>(p, pdl, s);
    return run_route<WQ_TYPE_BF16>(p, pdl, s);
}

}  // namespace wq
