// wq_logprobs.cu -- log probabilities of given tokens, entropy and top alternatives.
//
// What is computed, per row of V logits l: M = max l, S1 = sum e^(l - M),
// S2 = sum e^(l - M) (l - M);
//   logprob(t) = (l_t - M) - ln S1,  entropy = ln S1 - S2 / S1,
// and the top_k entries in the order (logit descending, index ascending).
//
// How.  Bound by HBM: a row is read once, in 16-byte loads, whatever its
// alignment (elements before the first and after the last full vector are read
// one by one).  A CTA takes a row, or, when there are few rows, a cluster of up
// to 8 CTAs splits it and joins through distributed shared memory.
//  * Each thread keeps its own reference m, S1 and S2 and moves m only when a
//    vector's maximum exceeds it by 8: e^8 times the count stays far inside
//    fp32, and the rescaling branch becomes rare.  After 1024 terms the sums go
//    to a total, so that a row's length does not cost digits.
//  * Top entries without a second pass.  A thread also keeps the largest value
//    it met and the first vector that held it.  The k-th largest of these
//    (value, vector) pairs over the CTA is a floor: k elements are at or above
//    it, so each of the row's top k lies in a vector of one of those k threads
//    and is itself at or above it.  Those threads' vectors alone (k of 256) are
//    read again, from L2, and the few entries at or above the floor are
//    ranked by counting.  Keys (value, index) are unique, so the result does not
//    depend on the order in which entries are collected.  Where more than 1024
//    entries lie above the floor (large logits that repeat with the period of the
//    threads' vectors) the chosen vectors are read again once per alternative: 64
//    rows of 128000 made so, 28 us with 5 alternatives and 73 with 32, against 9 and
//    16 of random ones; 2048 rows 129 and 1056 against 99 and 147.
// Measured (B200, device time): 2048 rows of 128000 bf16, 1 alternative, 524 MB: 92 us,
// 5.7 TB/s, 87 % of the copy rate; what is left is the rows' ends (the joins and the
// re-read, about 1 us per row, overlap with other CTAs' streams only).  Five CTAs of 256
// threads per SM: 4 take 98.6 us (94 with 8 vectors in flight per thread instead of 4), 6
// take 103 (registers), CTAs of 128 threads 100.  64 rows of 50001 bf16, 20 alternatives,
// 6.4 MB: 11.5 us; 32 rows of 128000 fp32, 16 MB: 9.3 us; one row of 32000 fp16: 6.4 us --
// chains of loads, joins and ranking, not bytes.
#include <cuda_runtime.h>

#include <algorithm>

#include "wq_internal.h"
#include "wq_logits.cuh"
#include "wq_ptx.cuh"

namespace wq {
namespace {

constexpr int LT = 256;        // threads per CTA
constexpr int LW = LT / 32;
constexpr int CAP = 1024;      // entries at or above the floor that are ranked at once
constexpr int MAXK = 32;
// Steps of the main loop (4 vectors: 32 or 16 terms) that a thread adds into one sum; then it goes to the thread's total
// in shared memory, so that a sum's error does not grow with the row: at most 1024 + V / 2^18 additions in a chain.  (One
// chain of a row of 2^29 was off by 1e-3.)
constexpr int CHAIN = 32;
constexpr float LOWEST = -1000.0f;  // e^-1000 = 0 in fp32: stands in for l - M = -inf, whose product with 0 is NaN

struct LpParams {
    const void* logits;
    long long ld;
    int V, top_k;
    const int64_t* tokens;
    float* logprob;
    float* entropy;
    float* top_logprob;
    int64_t* top_id;
};

struct Sums {
    float m, s1, s2;
};

__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// The same sums with reference M >= m.
__device__ __forceinline__ void rebase(Sums& s, float M) {
    const float dm = fmaxf(s.m - M, LOWEST);  // -inf (no finite value yet) and NaN: LOWEST
    const float f = ex2(dm * LOG2E);
    s.s2 = f * fmaf(dm, s.s1, s.s2);
    s.s1 *= f;
    s.m = M;
}

// 16 bytes as floats.
template <int TYPE> struct Vec;
template <> struct Vec<WQ_TYPE_F32> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void unpack(uint4 v, float (&f)[4]) {
        f[0] = __uint_as_float(v.x); f[1] = __uint_as_float(v.y);
        f[2] = __uint_as_float(v.z); f[3] = __uint_as_float(v.w);
    }
    static __device__ __forceinline__ float max(uint4 v) {
        return fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)),
                     fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
    }
};
template <> struct Vec<WQ_TYPE_F16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ float2 two(uint32_t u) {
        return __half22float2(*reinterpret_cast<const __half2*>(&u));
    }
    static __device__ __forceinline__ void unpack(uint4 v, float (&f)[8]) {
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 t = two(u[i]);
            f[2 * i] = t.x;
            f[2 * i + 1] = t.y;
        }
    }
    static __device__ __forceinline__ float max(uint4 v) {
        const float2 t = two(hmax2_u32(hmax2_u32(v.x, v.y), hmax2_u32(v.z, v.w)));
        return fmaxf(t.x, t.y);
    }
};
template <> struct Vec<WQ_TYPE_BF16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
        uint32_t r;
        asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    static __device__ __forceinline__ void unpack(uint4 v, float (&f)[8]) {
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(u[i] << 16);
            f[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
        }
    }
    static __device__ __forceinline__ float max(uint4 v) {
        const uint32_t t = max2(max2(v.x, v.y), max2(v.z, v.w));
        return fmaxf(__uint_as_float(t << 16), __uint_as_float(t & 0xFFFF0000u));
    }
};

__device__ __forceinline__ unsigned long long ld_cluster_u64(uint32_t addr) {
    unsigned long long v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
    return v;
}

struct LpShared {
    unsigned long long best[LT];    // threads' (key, ~vector); 0: a thread without vectors
    unsigned long long cand[CAP];   // entries at or above the floor: (key, ~index)
    unsigned long long top[MAXK];   // this CTA's top entries, best first; 0: none
    unsigned long long floor_;
    Sums warp[LW];
    Sums all;
    int chosen[MAXK];
    int nchosen, ncand;
};

__device__ __forceinline__ unsigned long long pack_key(uint32_t key, uint32_t index) {
    return ((unsigned long long)key << 32) | (0xFFFFFFFFu - index);
}

template <int TYPE, int CS>
__global__ void __launch_bounds__(LT, 5) logprobs_kernel(const LpParams p) {
    using L = Logit<TYPE>;
    using VT = Vec<TYPE>;
    constexpr int VN = VT::N;
    constexpr int U = 4;  // vectors in flight per thread
    __shared__ LpShared sh;
    grid_dependency_wait();
    grid_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long row = blockIdx.x / CS;
    const int rank = blockIdx.x % CS;
    const typename L::raw* src = static_cast<const typename L::raw*>(p.logits) + (size_t)row * p.ld;
    // aligned vectors over the row: vector v holds elements v * VN - mis ...
    const int mis = (int)((reinterpret_cast<uintptr_t>(src) & 15u) / sizeof(typename L::raw));
    const int nv = (mis + p.V + VN - 1) / VN;
    const int per = (nv + CS - 1) / CS;
    const int v0 = min(nv, rank * per), v1 = min(nv, v0 + per);
    const uint4* vecs = reinterpret_cast<const uint4*>(src - mis);
    const int full0 = mis ? 1 : 0, full1 = (mis + p.V) / VN;  // vectors that lie inside the row

    Sums s{-INFINITY, 0.0f, 0.0f};
    float ref = 0.0f, limit = -INFINITY;  // s.m once it is finite; the maximum that moves it
    float best = -INFINITY;
    int bvec = v0 + tid;
    auto add = [&](int v, float vmax, const float* f, int n) {
        if (vmax > best) {
            best = vmax;
            bvec = v;
        }
        if (vmax > limit) {
            if (limit > -INFINITY) rebase(s, vmax);
            s.m = ref = vmax;
            limit = vmax + 8.0f;
        }
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const float d = max_nan(f[i] - ref, LOWEST);
            const float e = ex2(d * LOG2E);
            s.s1 += e;
            s.s2 = fmaf(e, d, s.s2);
        }
    };
    auto partial = [&](int v) {  // a vector that reaches over the row's ends
        float f[VN], m = -INFINITY;
#pragma unroll
        for (int i = 0; i < VN; ++i) {
            const int e = v * VN - mis + i;
            f[i] = e >= 0 && e < p.V ? L::load(src + e) : -INFINITY;
            m = fmaxf(m, f[i]);
        }
        add(v, m, f, VN);
    };
    auto vector = [&](int v, uint4 r) {
        float f[VN];
        VT::unpack(r, f);
        add(v, VT::max(r), f, VN);
    };
    int v = v0 + tid;
    if (v < v1 && v < full0) {
        partial(v);
        v += LT;
    }
    const int vend = min(v1, full1);
    Sums* const total = reinterpret_cast<Sums*>(sh.cand) + tid;   // this thread's, where its row is long
    auto join = [&]() {   // s and the total
        Sums t = *total;
        const float M = fmaxf(s.m, t.m);
        rebase(s, M);
        rebase(t, M);
        s.s1 += t.s1;
        s.s2 += t.s2;
    };
    const int last = vend - (U - 1) * LT;   // a step begins below it
    int stop = min(last, v + CHAIN * U * LT);
    bool lengthy = false;
    while (true) {
        for (; v < stop; v += U * LT) {
            uint4 r[U];
#pragma unroll
            for (int j = 0; j < U; ++j) r[j] = __ldg(vecs + v + j * LT);
#pragma unroll
            for (int j = 0; j < U; ++j) vector(v + j * LT, r[j]);
        }
        if (v >= last) break;
        // into the total, and a new chain with the same reference
        const float m = s.m;
        if (lengthy) join();
        *total = s;
        s = Sums{m, 0.0f, 0.0f};
        lengthy = true;
        stop = min(last, v + CHAIN * U * LT);
    }
    for (; v < vend; v += LT) vector(v, __ldg(vecs + v));
    if (v < v1) partial(v);
    if (lengthy) join();

    // ---- the CTA's sums
    {
        float M = s.m;
#pragma unroll
        for (int d = 16; d; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
        rebase(s, M);
#pragma unroll
        for (int d = 16; d; d >>= 1) {
            s.s1 += __shfl_xor_sync(0xffffffffu, s.s1, d);
            s.s2 += __shfl_xor_sync(0xffffffffu, s.s2, d);
        }
        if (lane == 0) sh.warp[warp] = s;
    }
    const int k = p.top_k;
    if (k > 0) {
        sh.best[tid] = v0 + tid < v1 ? pack_key(order_key(best), (uint32_t)bvec) : 0ull;
        if (tid < MAXK) sh.top[tid] = 0ull;
        if (tid == 0) sh.ncand = 0;
    }
    __syncthreads();
    if (warp == 0) {
        Sums w = lane < LW ? sh.warp[lane] : Sums{-INFINITY, 0.0f, 0.0f};
        float M = w.m;
#pragma unroll
        for (int d = LW / 2; d; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
        rebase(w, M);
#pragma unroll
        for (int d = LW / 2; d; d >>= 1) {
            w.s1 += __shfl_xor_sync(0xffffffffu, w.s1, d);
            w.s2 += __shfl_xor_sync(0xffffffffu, w.s2, d);
        }
        if (lane == 0) sh.all = w;
    }
    if (k > 0) {
        // ---- the floor: the k best threads, by k rounds of one warp
        if (warp == LW - 1) {
            unsigned long long mine[LW], top = 0ull;
#pragma unroll
            for (int i = 0; i < LW; ++i) {
                mine[i] = sh.best[lane + 32 * i];
                top = max(top, mine[i]);
            }
            unsigned long long fl = 0ull;
            int n = 0;
            for (int j = 0; j < k; ++j) {
                const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(top >> 32));
                const uint32_t lo =
                    __reduce_max_sync(0xffffffffu, (uint32_t)(top >> 32) == hi ? (uint32_t)top : 0u);
                const unsigned long long win = ((unsigned long long)hi << 32) | lo;
                fl = win;
                if (win == 0ull) break;  // fewer threads with vectors than k: every entry counts
                if (lane == 0) sh.chosen[j] = (int)((0xFFFFFFFFu - lo) - (uint32_t)v0) % LT;
                ++n;
                if (top == win) {
                    top = 0ull;
#pragma unroll
                    for (int i = 0; i < LW; ++i) {
                        if (mine[i] == win) mine[i] = 0ull;
                        top = max(top, mine[i]);
                    }
                }
            }
            if (lane == 0) {
                sh.floor_ = fl;
                sh.nchosen = n;
            }
        }
        __syncthreads();
        // ---- entries at or above the floor, from the chosen threads' vectors
        const unsigned long long fl = sh.floor_;
        const int nvt = (v1 - v0 + LT - 1) / LT, total = sh.nchosen * nvt;
        auto each = [&](auto&& use) {
            for (int i = tid; i < total; i += LT) {
                const int c = i / nvt, vv = v0 + sh.chosen[c] + LT * (i - c * nvt);
                if (vv >= v1) continue;
                if (vv >= full0 && vv < full1) {
                    float f[VN];
                    VT::unpack(__ldg(vecs + vv), f);
#pragma unroll
                    for (int j = 0; j < VN; ++j) use(vv, vv * VN - mis + j, f[j]);
                } else {
                    for (int j = 0; j < VN; ++j) {
                        const int e = vv * VN - mis + j;
                        if (e >= 0 && e < p.V) use(vv, e, L::load(src + e));
                    }
                }
            }
        };
        each([&](int vv, int e, float x) {
            const uint32_t key = order_key(x);
            if (pack_key(key, (uint32_t)vv) >= fl) {
                const int at = atomicAdd(&sh.ncand, 1);
                if (at < CAP) sh.cand[at] = pack_key(key, (uint32_t)e);
            }
        });
        __syncthreads();
        const int n = sh.ncand;
        if (n <= CAP) {
            for (int i = tid; i < n; i += LT) {
                const unsigned long long me = sh.cand[i];
                int above = 0;
                for (int j = 0; j < n; ++j) above += sh.cand[j] > me;
                if (above < k) sh.top[above] = me;
            }
        } else {  // logits that repeat with the period of the threads: one entry per round
            unsigned long long below = ~0ull;
            for (int j = 0; j < k; ++j) {
                unsigned long long top = 0ull;
                each([&](int, int e, float x) {
                    const unsigned long long c = pack_key(order_key(x), (uint32_t)e);
                    if (c < below) top = max(top, c);
                });
                sh.best[tid] = top;
                __syncthreads();
#pragma unroll
                for (int d = LT / 2; d; d >>= 1) {
                    if (tid < d) sh.best[tid] = max(sh.best[tid], sh.best[tid + d]);
                    __syncthreads();
                }
                below = sh.best[0];
                if (tid == 0) sh.top[j] = below;
                __syncthreads();
            }
        }
    }
    __syncthreads();

    // ---- join the cluster's CTAs, write
    if constexpr (CS > 1) {
        cluster_sync();
        if (rank != 0) {
            cluster_sync();  // keep the shared memory until rank 0 has read it
            return;
        }
    }
    Sums a = sh.all;
    unsigned long long mine = 0ull;
    if constexpr (CS > 1) {
        const uint32_t base = smem_u32(&sh.all), tops = smem_u32(sh.top);
        Sums q[CS];
        float M = a.m;
#pragma unroll
        for (int r = 0; r < CS; ++r) {
            const uint32_t at = map_shared_rank(base, r);
            q[r].m = ld_shared_cluster_f32(at);
            q[r].s1 = ld_shared_cluster_f32(at + 4);
            q[r].s2 = ld_shared_cluster_f32(at + 8);
            M = fmaxf(M, q[r].m);
        }
        a.s1 = a.s2 = 0.0f;
#pragma unroll
        for (int r = 0; r < CS; ++r) {
            rebase(q[r], M);
            a.s1 += q[r].s1;
            a.s2 += q[r].s2;
        }
        a.m = M;
        if (tid < CS * k) mine = ld_cluster_u64(map_shared_rank(tops + 8u * (tid % k), tid / k));
        __syncwarp();
        cluster_sync();
        if (k > 0) {
            sh.cand[tid] = mine;
            __syncthreads();
        }
    } else if (tid < k) {
        mine = sh.top[tid];
    }
    const float ln = logf(a.s1);
    if (tid == 0) {
        p.entropy[row] = ln - a.s2 / a.s1;
        if (p.tokens) {
            const int64_t tok = p.tokens[row];
            p.logprob[row] = tok >= 0 && tok < p.V ? (L::load(src + tok) - a.m) - ln : -INFINITY;
        }
    }
    if (mine != 0ull) {
        int at = tid;
        if constexpr (CS > 1) {
            at = 0;
            for (int j = 0; j < CS * k; ++j) at += sh.cand[j] > mine;
        }
        if (at < k) {
            const size_t o = (size_t)row * k + at;
            p.top_logprob[o] = (key_value((uint32_t)(mine >> 32)) - a.m) - ln;
            p.top_id[o] = (int64_t)(0xFFFFFFFFu - (uint32_t)mine);
        }
    }
}

template <int TYPE, int CS>
wq_status launch_lp(const LpParams& p, int R, bool pdl, cudaStream_t s) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)R * CS);
    cfg.blockDim = dim3(LT);
    cfg.stream = s;
    cudaLaunchAttribute attrs[2];
    int na = 0;
    if (CS > 1) {
        attrs[na].id = cudaLaunchAttributeClusterDimension;
        attrs[na].val.clusterDim.x = CS;
        attrs[na].val.clusterDim.y = 1;
        attrs[na].val.clusterDim.z = 1;
        ++na;
    }
    if (pdl) {
        attrs[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attrs[na].val.programmaticStreamSerializationAllowed = 1;
        ++na;
    }
    cfg.attrs = attrs;
    cfg.numAttrs = na;
    return from_cuda(cudaLaunchKernelEx(&cfg, logprobs_kernel<TYPE, CS>, p));
}

template <int TYPE>
wq_status run_lp(const LpParams& p, int R, bool pdl, cudaStream_t s) {
    // A row is split while there is an SM for every CTA and each keeps a vector per thread, and on to four CTAs per SM
    // where each keeps 12 (bf16, 128 rows: of 128000, 4 CTAs per row 14.7 us, 2 15.9, 1 20.4; of 32000, 1 6.5 us, 2 7.7,
    // 4 8.4; 64 rows of 128000: 4 11.3 us, 8 12.8, 2 13.8).
    const int nv = p.V / Vec<TYPE>::N;
    int cs = 1;
    while (cs < 8) {
        const long long ctas = (long long)R * cs * 2;
        if (ctas > 4ll * sm_count() || nv < cs * 2 * LT * (ctas > sm_count() ? 12 : 1)) break;
        cs *= 2;
    }
    switch (cs) {
        case 8: return launch_lp<TYPE, 8>(p, R, pdl, s);
        case 4: return launch_lp<TYPE, 4>(p, R, pdl, s);
        case 2: return launch_lp<TYPE, 2>(p, R, pdl, s);
        default: return launch_lp<TYPE, 1>(p, R, pdl, s);
    }
}

}  // namespace

wq_status launch_logprobs(const void* logits, int type, int R, int V, long long ld, const int64_t* tokens, int top_k,
                          float* logprob, float* entropy, float* top_logprob, int64_t* top_id, unsigned flags,
                          cudaStream_t s) {
    const LpParams p{logits, ld, V, top_k, tokens, logprob, entropy, top_logprob, top_id};
    const bool pdl = (flags & WQ_FLAG_PDL) != 0;
    if (type == WQ_TYPE_F32) return run_lp<WQ_TYPE_F32>(p, R, pdl, s);
    if (type == WQ_TYPE_F16) return run_lp<WQ_TYPE_F16>(p, R, pdl, s);
    return run_lp<WQ_TYPE_BF16>(p, R, pdl, s);
}

}  // namespace wq
