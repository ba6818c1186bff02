// wq_moe.cu -- a mixture-of-experts layer on packed weights, for a few tokens.
//
// What is computed: for token t and its top_k slots (t, j) with expert
// e = ids[t][j] and weight a = weights[t][j],
//   h = act(x[t] @ Wg[e]) * (x[t] @ Wu[e])           (gate and up: one packed array, 2 I columns)
//   y[t] = sum_j a * (h[t][j] @ Wd[e])
// with W = (q - z) * s as everywhere in this library.  A slot whose id lies
// outside 0 .. E-1 is empty and adds nothing.
//
// Two launches of one kernel template.  UP turns x into h (one row per slot), DOWN
// turns h into y.  The layer reads each chosen expert's words once and is meant to
// be bound by HBM.
//  * Work split.  Slots are grouped by expert into blocks of bt slots (up to 8;
//    fewer when K is very long), so an expert's words are read once for them.  Every
//    CTA derives the blocks from the ids.  UP (one CTA per SM): the
//    (block, column tile) pairs, all of K each, are dealt out over the SMs in runs of
//    equal weight; its warps split K and the tile's columns, 64 columns each (32 gate and
//    the matching 32 up columns, so the activation needs no second pass), and their
//    partials meet in shared memory while the loads of the next item run.  DOWN (two CTAs
//    per SM): a tile of 64 columns belongs to a cluster of up to 8 CTAs, among whose warps
//    the tile's (block, part of K) line is dealt out; a warp works alone on its run.  Up
//    to 16 tokens every warp sums y, weighted, in its own copy in shared memory, and the
//    copies are joined at the end, across the cluster through distributed shared memory.
//    With more, the copies do not fit: a warp leaves the rows of its (block, part) in
//    global memory (L2), and the cluster sums them at its end.  Both in a fixed order.
//    (On an earlier form, instead of rows, 32 tokens: 85 us; a split of K over the CTA's warps
//    with two barriers per item 95 us, one copy per CTA with the warps adding in turn 97 us; a
//    last CTA to arrive that sums rows cost 1 us per item for the fence, up to 17 us at the end.)
//  * Products on integers.  Unpacking codes to fp16 or bf16 costs 7 instructions
//    per word of 8 codes, and with m16n8k16 (2.1 clocks per SM on B200) that held
//    a first version to 2.4 TB/s.  So the codes stay integers: 4-bit codes become
//    bytes with 3 instructions per word, 8-bit codes are used as they are, and
//    m16n8k32 on u8 x s8 (2.1 clocks too, twice the work) sums them exactly in int32.
//  * x (or h) becomes 24-bit fixed point: per token and block of 128 values
//    (aligned in K; 64 where UP's tiles are) a power-of-two step that puts the largest
//    value at 2^22 to 2^23, held as three signed bytes, x = step * (256 (256 hi + mid) +
//    lo).  Error: half a step, at most 1.02 * 2^-23 of the block's largest value, which is
//    what fp32 sums lose to a value of that size; none for values whose own last bit is at
//    or above the step (a bf16 within 2^-15 of the largest, an fp16 within 2^-12).  (Two
//    bytes were not enough: next to a value 3000 times the rest of its block, as single
//    channels have them, the rest kept 4 %, and where that value's codes lie at z it is
//    the rest that is the output.)  hi and mid of a slot are two adjacent columns of the
//    MMA, the lo of all slots a tile of their own.  UP converts x once per block of slots,
//    while its first words arrive, and leaves h converted (a tile's 128 values of a slot,
//    or 64, are one block), so that DOWN only reads bytes.  A block with a value that is
//    not finite gets the step NaN.
//  * The sums X of the values, which a zero point of any value needs, are taken when they
//    are converted, per unit: the 1, 2 or 4 steps of 32, as many as a group and a block
//    hold.  At the end of a unit: acc += s * step * (D - z X) in fp32,
//    D = 256 (256 D_hi + D_mid) + D_lo.  The unit's length is a template parameter: with
//    all three in one kernel, and a path for the rest of K, registers spilled and 16
//    tokens took 160 us instead of 128.
//  * Loads.  A warp's words come by TMA, 128 values of K x 64 columns (8-bit: 32, the
//    halves in turn) per stage (4 KB) with the s and z rows of its groups, into a private ring of two stages: 96 to
//    128 KB in flight per SM.  The 128-byte swizzle and the column order of the lanes
//    (chunk cg) keep the 16-byte reads free of bank conflicts.  (cp.async by every
//    lane, which this replaced, cost 19 instructions per step of 32 values, a quarter
//    of all.)
//  * DOWN is a programmatic dependent of UP: it finds its blocks and requests its
//    first words while UP drains, and waits only before it reads h.
// Measured (B200, device time): 16 tokens, 2 of 8 experts of 4096 x 11008, 4-bit, 569 MB:
// 119 us, 4.8 TB/s; 48 tokens, 4 of 32 experts of 2048 x 1408, 8-bit, 285 MB: 79 us, 3.6 TB/s;
// 1 token, 8 of 64 experts of 2048 x 1024, 4-bit, 27 MB: 14.2 us.  With 16 tokens neither DRAM
// (65 % of the copy rate in UP, 59 % in DOWN), the issue slots (46 and 41 %) nor the tensor pipe
// (36 %) is full: three warps per scheduler wait for their own chains (stage, unpacking, MMAs,
// fold), and UP's SMs end at different times (a part of the line is 2 to 6 items of 12 to
// 20 us); 1 token is the two starts (blocks, first loads, the join: 9 of 14.2 us).
// Every mbarrier wait is bounded; on time-out the kernel records it in its status
// word and skips the rest of the warp's work.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

#include "wq_dequant.cuh"
#include "wq_internal.h"
#include "wq_ptx.cuh"

namespace wq {

// Device status of these kernels: bit 0 once a bounded wait ran out, bit 1 once a
// check of the checked build failed.
__device__ unsigned int g_moe_status = 0;

namespace {

constexpr int MCOLS = 64;       // weight columns per warp (two halves of 32)
constexpr int MAXBT = 8;        // slots per block
// Most tokens for which every warp of DOWN keeps sums of y of its own; with more it leaves rows in global memory.  (Rows
// against sums, 16 tokens of 64 experts: 58.1 us against 55.1; 5 tokens, small: 19.0 against 14.5.  32 tokens of 64
// experts: rows 84.2, sums 80.6; of 128 experts of 7168 x 512 164 and 156: with a copy of 32 tokens the shared memory
// fills to 2 KB.)
constexpr int SUMS_T = 16;
constexpr int SK = 32;          // values of K per step (one MMA)
constexpr int XBLK = 4;         // steps per block of fixed-point values
// A stage: 4 KB of words.  4-bit: 16 word rows (128 values of K) of both halves; 8-bit: 32 (128 again) of one half, the
// halves in turn.  So a block of fixed-point values is multiplied with one half of the columns after the other, and the
// sums of one half alone are in registers.
constexpr int STAGE = 4096;
template <int BITS> constexpr int stage_rows() { return BITS == 4 ? 16 : 32; }
// Space for a stage's s rows and its z rows (64 or 32 columns), each at a multiple of 128 bytes.
__host__ __device__ constexpr int sz_space(int bits, int rows) { return bits == 4 ? 256 * rows : (rows + 1) / 2 * 256; }
constexpr int NST = 2;          // ring stages per warp (DOWN with 3: the same time)
// Warps of a CTA with NT token tiles.  Two tiles need about 160 registers: with 16 warps per SM, and 128, some spill, and
// 16 warps' rings leave fewer slots per block.  So 12 per SM, UP 12 in one CTA, DOWN 6 in each of two (DOWN with 8:
// 16 tokens, 2 of 8 experts, 131.3 us against 128.0; 8 tokens, top 4 of 16 of 7168 x 2048, 83.1 against 81.9; its sums do
// not fit groups of 32.  UP with 16: 16 tokens, 2 of 8, 130.9 against 128.0, 64 tokens, 2 of 8 of 4096 x 4096, 142.6
// against 132.5, 24 tokens of 8192 x 2048 91.6 against 85.8; but 48 tokens, 8-bit, 75.9 against 78.6, 16 tokens with
// groups of 32 44.1 against 50.1).  One tile: 16 per SM (1 token: 14.6 us; DOWN with 6 in a CTA 15.7).
constexpr int up_warps(int nt) { return nt == 1 ? 16 : 12; }
constexpr int down_warps(int nt) { return nt == 1 ? 8 : 6; }
constexpr int along_k(int warps) { return warps == 12 ? 3 : 4; }   // warps of a CTA of UP along K
constexpr uint64_t WAIT_NS = 2000000000ull;
// DOWN, many tokens, at its end: the slots' tables, then up to PART_ROWS weighted rows of a tile's columns, in the
// place of the rings (and beyond them: cut_smem counts the rows).
constexpr int PART_AT = 8192, PART_ROWS = 192;
__host__ __device__ constexpr int tokens_at_once(int top_k) { return PART_ROWS / top_k; }
static_assert((8 * down_warps(2) + 1) * 4 + 3 * WQ_MOE_MAX_TOKENS * 16 * 2 <= PART_AT, "starts, place, first, last");

template <int BITS> constexpr int step_rows() { return SK * BITS / 32; }   // word rows per step: 4 or 8

struct MoeParams {
    const uint16_t* x;      // UP: (T, K)
    int8_t* hq;             // (S, 3, Qh * SK): h in fixed point, hi, mid and lo bytes, in the byte order of DOWN's MMA
    // (S, Qh >> hlog): its units, the sum of the values and the step's bits.  A unit is the 1, 2 or 4 steps, as many as
    // no group ends inside, of a block of fixed-point values.
    uint2* hunit;
    const int32_t* ids;     // (T, top_k)
    const float* weights;   // (T, top_k)
    uint16_t* y;            // (T, N)
    float* rows;            // DOWN, many tokens: (tiles, S + bt * warps of a cluster, 64), the items' rows; else NULL
    int T, top_k, S, E, bt; // bt: slots per block
    int nblk;               // most blocks there can be
    int K;                  // inner length of this product (UP: K of x, DOWN: I)
    int NW;                 // weight columns (UP: 2 I, DOWN: N)
    int I;
    int ntiles;             // column tiles
    int Kw, Q;              // word rows, steps
    int spg;                // steps per group (large when one group spans K)
    int groups;
    int sz_rows;            // s (and z) rows per stage
    int act;
    int xcol;               // UP: bytes between two columns of x's fixed-point values
    int nunits;             // UP: units of x
    int Qh, hlog;           // steps of K in a row of h (whole stages); steps per unit of h, log2
    int cluster;            // DOWN: CTAs per column tile
};

__device__ __forceinline__ void sts64(uint32_t dst, uint32_t a, uint32_t b) {
    asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(dst), "r"(a), "r"(b) : "memory");
}
__device__ __forceinline__ void sts32(uint32_t dst, uint32_t a) {
    asm volatile("st.shared.u32 [%0], %1;" ::"r"(dst), "r"(a) : "memory");
}

// 3-D tiled bulk tensor load into this CTA's shared memory, completing on `bar`.
__device__ __forceinline__ void tma_load_3d_u32(uint32_t dst, const void* tmap, uint64_t* bar, int c0, int c1, int c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], "
        "[%2];" ::"r"(dst),
        "l"(tmap), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}

// Dynamic shared memory of this launch.
__device__ __forceinline__ uint32_t dynamic_smem_bytes() {
    uint32_t n;
    asm("mov.u32 %0, %%dynamic_smem_size;" : "=r"(n));
    return n;
}

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// D(16x8, s32) = A(16x32, u8) * B(32x8, s8) + D, or + c in every element (first).
__device__ __forceinline__ void mma_u8s8(bool first, int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint2 b, int c) {
    if (first)   // a constant where this is called
        asm("mma.sync.aligned.m16n8k32.row.col.s32.u8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%10,%10,%10,%10};"
            : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b.x), "r"(b.y), "r"(c));
    else
        asm("mma.sync.aligned.m16n8k32.row.col.s32.u8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b.x), "r"(b.y));
}

// Two floats at once (one instruction each: the folds below are bound by instruction issue).
__device__ __forceinline__ uint64_t pack2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// The blocks of a launch: experts in the order of their first slot (S <= 32) or of their
// number, up to bt slots each, in the order of the slots.
struct Blocks {         // in shared memory
    int* n;             // blocks
    int* start;         // sum of the weights of the blocks before u, and of all
    int16_t* e;         // expert of block u
    int16_t* first;     // its first slot's place in `order`
    int16_t* order;     // the slots, block by block
    // slots of block u
    __device__ __forceinline__ int count(int u) const { return first[u + 1] - first[u]; }
};
// More blocks than these cannot be: e experts with m slots each take the sum of ceil(m / bt) <= (S + e (bt - 1)) / bt.
__host__ __device__ constexpr int most_blocks(int S, int E, int bt) {
    return (S + (E < S ? E : S) * (bt - 1)) / bt;
}
__host__ __device__ constexpr int table_bytes(int S, int nblk) {
    return ((nblk + 1) * 4 + (2 * nblk + 1 + S) * 2 + 15) / 16 * 16;
}

// Weight of a block of m slots: two token tiles take more instructions, the same loads.  (16 tokens, 2 of 8 experts,
// 4-bit | 48 tokens, 8-bit: with 4 : 5 128.0 | 78.7 us, 3 : 4 128.2 | 82.2, 2 : 3 125.4 | 81.7, 1 : 1 139.8 | 78.2.)
__device__ __forceinline__ int block_weight(int m) { return m <= 4 ? 4 : 5; }

// Work is dealt out along a line: block u takes `units` of it (UP: its column tiles, DOWN: its fixed-point
// blocks of K), each as heavy as the block's weight.  The first unit at or after part i of n.
__device__ __forceinline__ int share(const Blocks& b, int units, int i, int n) {
    const int nb = *b.n;
    if (nb == 0) return 0;
    const int C = b.start[nb] * units;                           // below 2^31 (checked by the host)
    const int c = C / n * i + C % n * i / n, q = c / units;      // c = floor(C i / n) in 32 bits
    int lo = 0, hi = nb;                                         // start[lo] <= q < start[hi], but for q = start[nb]
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (b.start[mid] <= q) lo = mid;
        else hi = mid;
    }
    const int w = b.start[lo + 1] - b.start[lo];
    return lo * units + (c - b.start[lo] * units + w - 1) / w;
}

// Fills the table; every thread returns after it is complete.  cnt: scratch, E ints and S shorts.
template <int MT>
__device__ __forceinline__ void find_blocks(const MoeParams& p, const Blocks& b, int* cnt) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const unsigned lt = (1u << lane) - 1u;
    if (p.S <= 32) {   // one slot per lane of one warp
        if (warp == 0) {
            int id = lane < p.S ? p.ids[lane] : -1;
            if (id >= p.E || id < 0) id = -1;
            const unsigned same = __match_any_sync(0xffffffffu, id < 0 ? -1 - lane : id);
            const bool leader = id >= 0 && (same & lt) == 0;
            const int nb = leader ? (__popc(same) + p.bt - 1) / p.bt : 0;
            const int m = leader ? __popc(same) : 0;
            const int wt = leader ? (nb - 1) * block_weight(p.bt) + block_weight(m - (nb - 1) * p.bt) : 0;
            int pre = nb, cost = wt, place = m;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, pre, d), c = __shfl_up_sync(0xffffffffu, cost, d);
                const int l = __shfl_up_sync(0xffffffffu, place, d);
                if (lane >= d) {
                    pre += v;
                    cost += c;
                    place += l;
                }
            }
            if (lane == 31) {
                *b.n = pre;
                b.start[pre] = cost;
                b.first[pre] = (int16_t)place;
            }
            pre -= nb;
            cost -= wt;
            place -= m;
            for (int i = 0; i < nb; ++i) {
                b.e[pre + i] = (int16_t)id;
                b.first[pre + i] = (int16_t)(place + i * p.bt);
                b.start[pre + i] = cost + i * block_weight(p.bt);
            }
            const int at = __shfl_sync(0xffffffffu, place, __ffs(same) - 1) + __popc(same & lt);
            if (id >= 0) b.order[at] = (int16_t)lane;
        }
        __syncthreads();
        return;
    }
    for (int e = threadIdx.x; e < p.E; e += MT) cnt[e] = 0;
    __syncthreads();
    int16_t* const of = reinterpret_cast<int16_t*>(cnt + p.E);   // the slots' experts
    for (int i = threadIdx.x; i < p.S; i += MT) {
        const int id = p.ids[i];
        const bool in = id >= 0 && id < p.E;
        of[i] = in ? (int16_t)id : (int16_t)-1;
        if (in) atomicAdd(&cnt[id], 1);
    }
    __syncthreads();
    if (warp == 0) {
        const int per = (p.E + 31) / 32;
        int mine = 0, wt = 0, m = 0;
        for (int j = 0; j < per; ++j) {
            const int e = lane * per + j;
            if (e >= p.E) break;
            m += cnt[e];
            for (int r = 0; r < cnt[e]; r += p.bt) {
                ++mine;
                wt += block_weight(min(p.bt, cnt[e] - r));
            }
        }
        int pre = mine, cost = wt, place = m;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, pre, d), c = __shfl_up_sync(0xffffffffu, cost, d);
            const int l = __shfl_up_sync(0xffffffffu, place, d);
            if (lane >= d) {
                pre += v;
                cost += c;
                place += l;
            }
        }
        if (lane == 31) {
            *b.n = pre;
            b.start[pre] = cost;
            b.first[pre] = (int16_t)place;
        }
        pre -= mine;
        cost -= wt;
        place -= m;
        for (int j = 0; j < per; ++j) {
            const int e = lane * per + j;
            if (e >= p.E) break;
            const int c = cnt[e];
            for (int r = 0; r < c; r += p.bt, ++pre) {
                b.e[pre] = (int16_t)e;
                b.first[pre] = (int16_t)(place + r);
                b.start[pre] = cost;
                cost += block_weight(min(p.bt, c - r));
            }
            cnt[e] = place;   // from here on: where the expert's next slot goes
            place += c;
        }
        __syncwarp();
        for (int i0 = 0; i0 < p.S; i0 += 32) {   // the slots in ascending order
            const int i = i0 + lane;
            const int id = i < p.S ? of[i] : -1;
            const unsigned same = __match_any_sync(0xffffffffu, id < 0 ? -1 - lane : id);
            const int at = id < 0 ? 0 : cnt[id] + __popc(same & lt);
            __syncwarp();
            if (id >= 0) {
                b.order[at] = (int16_t)i;
                if ((same & lt) == 0) cnt[id] = at + __popc(same);
            }
            __syncwarp();
        }
    }
    fence_proxy_async_smem();   // cnt lies where the copies will land
    __syncthreads();
}

__device__ __forceinline__ float activate(float g, int act) {
    if (act == WQ_ACT_SILU) return g / (1.0f + __expf(-g));
    return 0.5f * g * erfcf(-0.70710678118654752f * g);  // gelu
}

// 8 values as 24-bit fixed point with step 2^(E - 149), `inv` = 2^(149 - E): the integer plus 0x808080 has the bytes
// hi, mid and lo plus 128: x = 256^2 hi + 256 mid + lo, all in -128 .. 127.
// Byte order: 4-bit words, the codes 0 2 4 6 and 1 3 5 7 of a word row; 8-bit, as they come.
struct Bytes {
    uint2 hi, mid, lo;
};
template <int BITS>
__device__ __forceinline__ Bytes to_fixed(const float (&v)[8], float inv) {
    uint32_t u[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] = (uint32_t)__float2int_rn(v[i] * inv) + 0x808080u;
    auto four = [&](int a, int b, int c, int d, uint32_t& h, uint32_t& m, uint32_t& l) {
        const uint32_t p = prmt(u[a], u[b], 0x5140u), q = prmt(u[c], u[d], 0x5140u);  // bytes a0 b0 a1 b1
        l = prmt(p, q, 0x5410u) ^ 0x80808080u;
        m = prmt(p, q, 0x7632u) ^ 0x80808080u;
        h = prmt(prmt(u[a], u[b], 0x0062u), prmt(u[c], u[d], 0x0062u), 0x5410u) ^ 0x80808080u;
    };
    Bytes r;
    if constexpr (BITS == 4) {
        four(0, 2, 4, 6, r.hi.x, r.mid.x, r.lo.x);
        four(1, 3, 5, 7, r.hi.y, r.mid.y, r.lo.y);
    } else {
        four(0, 1, 2, 3, r.hi.x, r.mid.x, r.lo.x);
        four(4, 5, 6, 7, r.hi.y, r.mid.y, r.lo.y);
    }
    return r;
}

// Exponent E of a block whose largest magnitude has the bits `top`: |x| 2^(149 - E) <= 1.984375 * 2^22 < 0x7F7F80, one
// more from 1.984375 * 2^n up (at least 23: a step is no subnormal); and its step 2^(E - 149), NaN where a value is not
// finite.
__device__ __forceinline__ uint32_t block_exponent(uint32_t top) {
    return min(max((top + 0x00020000u) >> 23, 23u), 255u);
}
__device__ __forceinline__ float block_inverse(uint32_t E) { return __uint_as_float((276u - E) << 23); }
__device__ __forceinline__ uint32_t block_step(uint32_t top, uint32_t E) {
    return top >= 0x7F800000u ? 0x7FC00000u : (E - 22u) << 23;
}

// The sum of 8 values, from their bytes.
__device__ __forceinline__ int value_sum(const Bytes& b) {
    auto sum = [](uint2 v) { return __dp4a((int)v.y, 0x01010101, __dp4a((int)v.x, 0x01010101, 0)); };
    return 256 * (256 * sum(b.hi) + sum(b.mid)) + sum(b.lo);
}

// Shared memory behind the rings: the warps' partials, the blocks; UP: x's fixed-point values and their units; DOWN:
// the sums of y.
__host__ __device__ constexpr int table_at(int W, int bt) { return W * bt * MCOLS * 4; }
__host__ __device__ constexpr int values_at(int W, int bt, int S, int nblk) {
    return table_at(W, bt) + table_bytes(S, nblk);
}
__host__ __device__ constexpr int units_at(int W, int bt, int S, int nblk, int xcol) {
    return values_at(W, bt, S, nblk) + 3 * bt * xcol;
}

// NT: token tiles of 4 slots (8 MMA columns).  MW: warps.  U: steps per unit (XBLK but for groups that are no multiple of
// 128, and for blocks of h of 64 values).
template <int BITS, bool BF, int NT, bool UP, int MW, int U>
__global__ void __launch_bounds__(MW * 32, UP ? 16 / MW : 2)
moe_kernel(const __grid_constant__ CUtensorMap tm, const __grid_constant__ CUtensorMap tm_s,
           const __grid_constant__ CUtensorMap tm_z, const MoeParams p) {
    constexpr int MT = MW * 32;
    using T16 = Dt<BF>;
    constexpr int RPS = step_rows<BITS>();       // 4 or 8
    constexpr int RL = RPS / 4;                  // word rows per lane and step
    constexpr int SPS = XBLK;                    // steps per stage
    constexpr int WK = UP ? along_k(MW) : 1;               // UP: warps along K
    constexpr int WC = UP ? MW / WK : 1;         // and along the columns.  DOWN: every warp works alone
    constexpr int TC = MCOLS * WC;               // weight columns per tile
    extern __shared__ uint8_t smem_raw[];
    // the 128-byte swizzle of the TMA boxes repeats every 1024 bytes
    uint8_t* const smem = smem_raw + (((smem_u32(smem_raw) + 1023u) & ~1023u) - smem_u32(smem_raw));
    __shared__ int nblocks;
    __shared__ uint64_t bars[MW * NST], free_bar;   // free_bar (UP): the partials have been read

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    // 16-byte column chunk of this lane (columns 4 cg .. 4 cg + 3 of each half): with the lines of a
    // stage below, the eight lanes of a quarter-warp meet eight different bank groups
    const int cg = UP && BITS == 4 ? g : ((g & 1) << 2) | (g >> 1);
    const int wk = warp / WC, wc = warp % WC;   // UP
    uint64_t* const bar = bars + warp * NST;
    if (lane == 0) {
        for (int i = 0; i < NST; ++i) mbar_init(&bar[i], 1);
        if (UP && warp == 0) mbar_init(&free_bar, MW);
        fence_mbarrier_init();
        if (warp == 1) prefetch_tmap(&tm);
        if (warp == 2) prefetch_tmap(&tm_s);
        if (warp == 3) prefetch_tmap(&tm_z);
    }
    if constexpr (UP) grid_dependency_wait();   // ids, weights and x may be the previous kernel's output
    grid_launch_dependents();
    const int Q4 = (p.Q + XBLK - 1) / XBLK;
    const int rank = UP ? 0 : (int)blockIdx.x % p.cluster;
    const uint32_t sz_bytes = sz_space(BITS, p.sz_rows);    // a stage's s rows, then its z rows
    const uint32_t roff = MW * NST * (STAGE + sz_bytes);    // behind the rings
    constexpr int RW = UP ? MW : 0;   // warps with partials in shared memory
    uint8_t* const tab = smem + roff + table_at(RW, p.bt);
    int16_t* const tab16 = reinterpret_cast<int16_t*>(tab + 4 * (p.nblk + 1));
    const Blocks blk{&nblocks, reinterpret_cast<int*>(tab), tab16, tab16 + p.nblk, tab16 + 2 * p.nblk + 1};
    find_blocks<MT>(p, blk, reinterpret_cast<int*>(smem));
    // this CTA's part of the line (UP) or this warp's (DOWN): lane 0 finds where it starts, the others where it ends
    const int part = UP ? (int)blockIdx.x : rank * MW + warp, parts = UP ? (int)gridDim.x : p.cluster * MW;
    const int mine = share(blk, UP ? p.ntiles : Q4, part + (lane != 0), parts);
    const int at0 = __shfl_sync(0xffffffffu, mine, 0), end = __shfl_sync(0xffffffffu, mine, 1);
    // ---- the items.  UP, the CTA's: (block, tile) pairs, all steps of K; DOWN, the warp's: one tile, runs of a
    // block's steps
    struct Item {
        int at, u, tile, s0, ns;   // position on the line, block, column tile; this warp's first step and steps
    };
    Item it;                       // (divisions here alone, none per item)
    it.at = at0;
    it.u = at0 / (UP ? p.ntiles : Q4);
    if constexpr (UP) {            // the warps along K: whole fixed-point blocks
        it.tile = at0 - it.u * p.ntiles;
        const int per = ((p.Q + WK - 1) / WK + XBLK - 1) / XBLK * XBLK;
        it.s0 = min(p.Q, wk * per);
        it.ns = min(p.Q, it.s0 + per) - it.s0;
    } else {
        it.tile = (int)blockIdx.x / p.cluster;
        it.s0 = (at0 - it.u * Q4) * XBLK;
        it.ns = min(p.Q - it.s0, (end - at0) * XBLK);
    }
    auto next = [&](Item& it) {
        if constexpr (UP) {
            ++it.at;
            if (++it.tile == p.ntiles) {
                it.tile = 0;
                ++it.u;
            }
        } else {
            it.at += (it.ns + XBLK - 1) / XBLK;
            ++it.u;
            it.s0 = 0;
            it.ns = min(p.Q, (end - it.at) * XBLK);
        }
    };
    // first column of this warp in a tile (UP: of the gate; the up columns are the map's second plane)
    auto col = [&](int tile) { return UP ? tile * (TC / 2) + 32 * wc : tile * TC; };
    // ---- loads: a cursor over the (item, stage) sequence of this warp
    const uint32_t ring = smem_u32(smem) + (uint32_t)warp * (NST * STAGE);
    const uint32_t sz_ring = smem_u32(smem) + MW * NST * STAGE + (uint32_t)warp * (NST * sz_bytes);
    Item wit = it;                          // the item whose stages are being requested
    const int g0 = it.s0 / p.spg, gp0 = it.s0 - g0 * p.spg;   // UP: of every item; DOWN: of the first, then 0
    int wleft = 0, whalf = 0;               // stages left in it; 8-bit: the half of the next one
    int row = 0, grow = 0, gpos = 0;        // the next stage: word row, s row, steps into its group
    bool ok = true, first = true;
    auto issue = [&](uint32_t slot) {
        if (wleft == 0) {
            // (an item of UP has no steps for a warp past the end of K: nor has any other)
            if (!first) next(wit);
            if (wit.at >= end || wit.ns == 0) return;
            wleft = (wit.ns + SPS - 1) / SPS * (BITS == 4 ? 1 : 2);
            const int e = blk.e[wit.u];
            row = e * p.Kw + wit.s0 * RPS;
            grow = e * p.groups + (UP || first ? g0 : 0);
            gpos = UP || first ? gp0 : 0;
            first = false;
        }
        if (lane == 0) {
            uint64_t* const b = &bar[slot];
            mbar_arrive_expect_tx(b, STAGE + (BITS == 4 ? 256u : 128u) * (uint32_t)p.sz_rows);
            const int wcol = col(wit.tile);
            const uint32_t dst = ring + slot * STAGE, sz = sz_ring + slot * sz_bytes;
            if constexpr (UP) {
                tma_load_3d_u32(dst, &tm, b, wcol, whalf, row);
                tma_load_3d_u32(sz, &tm_s, b, wcol, whalf, grow);
                tma_load_3d_u32(sz + sz_bytes / 2, &tm_z, b, wcol, whalf, grow);
            } else {
                tma_load_2d_u32(dst, &tm, b, wcol + 32 * whalf, row);
                if constexpr (BITS == 4) tma_load_2d_u32(dst + STAGE / 2, &tm, b, wcol + 32, row);
                tma_load_2d_u32(sz, &tm_s, b, wcol + 32 * whalf, grow);
                tma_load_2d_u32(sz + sz_bytes / 2, &tm_z, b, wcol + 32 * whalf, grow);
            }
        }
        --wleft;
        if constexpr (BITS == 8) {
            whalf ^= 1;
            if (whalf) return;
        }
        row += stage_rows<BITS>();
        for (gpos += SPS; gpos >= p.spg; gpos -= p.spg) ++grow;
    };
    issue(0);
    issue(1);

    if constexpr (!UP) grid_dependency_wait();   // h
    float* const red = reinterpret_cast<float*>(smem + roff);   // [wk][slot][TC]
    const uint32_t xoff = roff + values_at(RW, p.bt, p.S, p.nblk), xbase = smem_u32(smem) + xoff;          // UP
    // UP: x's units, [slot][unit]; DOWN: the sums of y, [warp][T][TC]
    uint2* const units = reinterpret_cast<uint2*>(smem + roff + units_at(MW, p.bt, p.S, p.nblk, p.xcol));
    float* const ys = reinterpret_cast<float*>(smem + xoff);
    // This lane's 16-byte vectors of word row t (and t + 4): line r of 128 bytes holds them at chunk
    // cg ^ (r & 7).  4-bit UP: the lines of a word row's two halves follow each other; 4-bit DOWN: 16 lines each.
    constexpr bool PAIRED = UP && BITS == 4;
    constexpr uint32_t HALF = PAIRED ? 128u : BITS == 4 ? STAGE / 2 : 0u;   // to the other half
    constexpr uint32_t LINE = PAIRED ? 256u : 128u;                          // to the next row
    // (paired: rows 4 apart have the same swizzle; else: the two halves have)
    const uint32_t off0 = t * LINE + (((uint32_t)cg ^ ((PAIRED ? 2 * t : t) & 7u)) << 4);
    const uint32_t off1 = PAIRED ? t * LINE + HALF + (((uint32_t)cg ^ ((2 * t + 1) & 7u)) << 4)
                                 : (t + 4) * LINE + (((uint32_t)cg ^ (t + 4u)) << 4);
    auto off = [&](int odd, int hf) {   // constants
        if constexpr (PAIRED) return (hf ? off1 : off0) + 4 * LINE * odd;
        else return (odd ? off1 : off0) + HALF * hf;
    };
    uint32_t slot = 0, phase = 0;   // ring position of the next stage to read
    auto advance = [&]() {
        slot ^= 1u;
        phase ^= slot ^ 1u;
    };

    if constexpr (!UP)
        if (p.rows == nullptr) {
            for (int i = lane; i < p.T * TC; i += 32) ys[warp * p.T * TC + i] = 0.0f;
            __syncwarp();
        }

    // UP: the column of slot m's lo bytes (full blocks: the four that a load phase reads, slots 0 4 1 5 and 2 6 3 7, lie
    // in different banks)
    auto lo_col = [&](int m) { return 2 * p.bt + (p.bt == 8 ? m ^ ((m >> 1) & 2) : m); };
    int block = -1;   // UP: the block whose values are in shared memory
    int done = 0;     // items finished
    for (; it.at < end; next(it)) {
        const int q0 = it.s0, nq = it.ns;
        const int16_t* const slots = blk.order + blk.first[it.u];
        const int bm = blk.count(it.u);
        if (UP && it.u != block) {
            // ---- another block: x of its slots as fixed point.  Column 2 m holds hi of the block's slot m, 2 m + 1
            // its mid, and lo_col(m) its lo: 32 bytes per step, 8 for each word row t.
            block = it.u;
            // (the previous block's were last read before the barrier behind the partials)
            // (slot, 8 steps) pairs of this warp, XU at a time so that their loads overlap; a lane has 8 values
            const int rounds = (nq + 7) / 8, pairs = bm > wc ? (bm - wc + WC - 1) / WC * rounds : 0;
            constexpr int XU = 4;
#pragma unroll 1
            for (int p0 = 0; p0 < pairs; p0 += XU) {
                uint4 raw[XU];
#pragma unroll
                for (int u = 0; u < XU; ++u) {
                    const int pr = min(p0 + u, pairs - 1), m = wc + pr / rounds * WC;
                    const int q = q0 + pr % rounds * 8 + g, k = q * SK + 8 * t, slot = slots[m];
                    check(slot >= 0 && slot < p.S, &g_moe_status);
                    const bool in = q < q0 + nq;
                    raw[u] = make_uint4(0u, 0u, 0u, 0u);
                    const uint16_t* const src = p.x + (size_t)(slot / p.top_k) * p.K + k;
                    if constexpr (BITS == 4) {                // K is a multiple of 8
                        if (in && k < p.K) raw[u] = *reinterpret_cast<const uint4*>(src);   // (else 0)
                    } else {                                  // K is a multiple of 4
                        uint2 a = make_uint2(0u, 0u), c = a;
                        if (in && k < p.K) a = *reinterpret_cast<const uint2*>(src);
                        if (in && k + 4 < p.K) c = *reinterpret_cast<const uint2*>(src + 4);
                        raw[u] = make_uint4(a.x, a.y, c.x, c.y);
                    }
                }
#pragma unroll
                for (int u = 0; u < XU; ++u) {
                    if (p0 + u >= pairs) break;
                    const int pr = p0 + u, m = wc + pr / rounds * WC, qo = pr % rounds * 8 + g, q = q0 + qo;
                    const bool in = qo < (nq + U - 1) / U * U;   // the last unit is filled up with zeros
                    float v[8];
                    const uint32_t r0[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 f = T16::pair(r0[i]);
                        v[2 * i] = f.x;
                        v[2 * i + 1] = f.y;
                    }
                    uint32_t top = 0;   // bits of the block's largest magnitude, over its 16 lanes
#pragma unroll
                    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
#pragma unroll
                    for (int d = 8; d; d >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
                    const uint32_t E = block_exponent(top);
                    const Bytes b = to_fixed<BITS>(v, block_inverse(E));
                    const uint32_t at = xbase + (uint32_t)(2 * m) * p.xcol + (uint32_t)q * 32u;
                    const uint32_t at_lo = xbase + (uint32_t)lo_col(m) * p.xcol + (uint32_t)q * 32u;
                    if (in && check(q * 32 + 32 <= p.xcol && lo_col(m) < 3 * p.bt, &g_moe_status)) {
                        if constexpr (BITS == 4) {
                            sts64(at + 8u * t, b.hi.x, b.hi.y);
                            sts64(at + p.xcol + 8u * t, b.mid.x, b.mid.y);
                            sts64(at_lo + 8u * t, b.lo.x, b.lo.y);
                        } else {   // word row j of the step (4 values each): bytes 8 (j % 4) + 4 (j / 4)
                            const uint32_t j = 2u * t, o = 8u * (j & 3u) + 4u * (j >> 2);
                            sts32(at + o, b.hi.x);
                            sts32(at + o + 8u, b.hi.y);
                            sts32(at + p.xcol + o, b.mid.x);
                            sts32(at + p.xcol + o + 8u, b.mid.y);
                            sts32(at_lo + o, b.lo.x);
                            sts32(at_lo + o + 8u, b.lo.y);
                        }
                    }
                    int sum = value_sum(b);   // of the lane, its step (4 lanes) and its unit (4, 8 or 16)
#pragma unroll
                    for (int d = 1; d < 16; d <<= 1)
                        if (d < 4 * U) sum += __shfl_xor_sync(0xffffffffu, sum, d);
                    if (lane % (4 * U) == 0 && in && check(q / U < p.nunits, &g_moe_status))
                        units[m * p.nunits + q / U] = make_uint2((uint32_t)sum, block_step(top, E));
                }
            }
            __syncthreads();
        }

        // ---- one item.  AT: token tiles that hold slots of this block
        auto run = [&](auto at_tag) {
            constexpr int AT = decltype(at_tag)::value;
            uint64_t acc[2][2][AT];   // two columns each
#pragma unroll
            for (int hf = 0; hf < 2; ++hf)
#pragma unroll
                for (int n = 0; n < AT; ++n) acc[hf][0][n] = acc[hf][1][n] = 0ull;
            // B column g of token tile n: hi and mid of slots 4 n + g / 2; of the last one, lo of slots g / 2 (g even)
            // and 4 + g / 2 (odd).  UP from shared memory; DOWN straight from global memory, a stage ahead (every CTA
            // reads the same bytes: L2).  Columns beyond the block's slots: any bytes, the results are not used.
            uint32_t at[AT + 1], unit[AT];         // offsets of values and units
            [[maybe_unused]] uint2 ux[AT];
            uint2 bx[SPS][AT + 1];                 // this stage's values; DOWN: its units, that of step g % 4
            [[maybe_unused]] float wt[AT];         // DOWN: weights of the slots 4 n + t and their rows of y's sums
            [[maybe_unused]] uint32_t yrow[AT];
            const int third = (g >> 1) + (AT > 1 ? 4 * (g & 1) : 0);
#pragma unroll
            for (int n = 0; n < AT; ++n) {
                if constexpr (UP) {
                    at[n] = xoff + (uint32_t)min(8 * n + g, 2 * p.bt - 1) * p.xcol + (uint32_t)q0 * 32u + 8u * t;
                    unit[n] = smem_u32(units + min(4 * n + t, p.bt - 1) * p.nunits + q0 / U);
                } else {
                    const int col = 3 * slots[min(4 * n + (g >> 1), bm - 1)] + (g & 1);
                    at[n] = (uint32_t)(col * p.Qh + q0) * SK + 8 * t;   // (wq_moe keeps it below 3 * 2^30)
                    const int sl = slots[min(4 * n + t, bm - 1)];
                    unit[n] = (sl * p.Qh + q0) / U;         // (Qh is a multiple of XBLK)
                    wt[n] = p.weights[sl];
                    yrow[n] = (uint32_t)(warp * p.T + sl / p.top_k) * TC + 4 * cg;
                    check(col < 3 * p.S, &g_moe_status);
                }
            }
            at[AT] = UP ? xoff + (uint32_t)lo_col(min(third, p.bt - 1)) * p.xcol + (uint32_t)q0 * 32u + 8u * t
                        : (uint32_t)((3 * slots[min(third, bm - 1)] + 2) * p.Qh + q0) * SK + 8 * t;
            auto request = [&](int i) {            // the values of the stage from step i; DOWN: and its units
#pragma unroll
                for (int j = 0; j < SPS; ++j)
#pragma unroll
                    for (int n = 0; n <= AT; ++n)
                        bx[j][n] = UP ? *reinterpret_cast<const uint2*>(smem + at[n] + 32 * (i + j))
                                      : *reinterpret_cast<const uint2*>(p.hq + at[n] + (uint32_t)((i + j) * SK));
                if constexpr (!UP) {
#pragma unroll
                    for (int n = 0; n < AT; ++n) ux[n] = p.hunit[unit[n] + (i + (g & (SPS - 1))) / U];
                }
            };
            if constexpr (!UP) request(0);         // (an item has a step; rows of values hold whole stages)
            struct Sums {           // of one half of the columns: products with hi and mid, and with lo
                int d[2][AT][4], lo[2][4];
            };
            struct Unit {           // sum of the values, step
                int X[AT];
                uint32_t step[AT];
            };
            // The sums start at the bits of 1.5 * 2^23: an integer of at most 22 bits added to them is, read
            // as a float, that much more (128 * 255 * 128 < 2^22), so no conversion is needed.
            constexpr int BIAS = 0x4B400000;
            auto value2 = [](int a, int b) {
                return unpack2(add2(pack2(__int_as_float(a), __int_as_float(b)), pack2(-12582912.0f, -12582912.0f)));
            };
            auto read_unit = [&](int i, int j) {   // step j of the stage, i of the range
                Unit un;
#pragma unroll
                for (int n = 0; n < AT; ++n) {
                    uint2 w;
                    if constexpr (UP) {
                        w = lds64_u32(unit[n] + 8u * (i / U));
                    } else {                       // (lanes 4 j .. 4 j + 3 have it)
                        w.x = U == SPS ? ux[n].x : __shfl_sync(0xffffffffu, ux[n].x, 4 * j + t);
                        w.y = U == SPS ? ux[n].y : __shfl_sync(0xffffffffu, ux[n].y, 4 * j + t);
                    }
                    un.X[n] = (int)w.x;
                    un.step[n] = w.y;
                }
                return un;
            };
            // step j of the stage with one half of the columns
            // (st: the stage; plain loads, whose constant offsets fold).  first: a new sum, from BIAS
            auto mult = [&](Sums& m, bool first, int hf, const uint8_t* st, int j) {
                uint4 w[RL];
#pragma unroll
                for (int r = 0; r < RL; ++r) {   // rows 4 j + t (4-bit), 8 j + t and 8 j + t + 4 (8-bit)
                    const int row8 = BITS == 4 ? j >> 1 : j, odd = BITS == 4 ? j & 1 : r;
                    w[r] = *reinterpret_cast<const uint4*>(st + off(odd, hf) + 8 * LINE * row8);
                }
                uint32_t a[2][4];   // k 0-15 and 16-31 of the lane's four columns
                const uint32_t v0[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
                if constexpr (BITS == 4) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        a[0][c] = v0[c] & 0x0F0F0F0Fu;
                        a[1][c] = (v0[c] >> 4) & 0x0F0F0F0Fu;
                    }
                } else {
                    const uint32_t v1[4] = {w[RL - 1].x, w[RL - 1].y, w[RL - 1].z, w[RL - 1].w};
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        a[0][c] = v0[c];
                        a[1][c] = v1[c];
                    }
                }
#pragma unroll
                for (int T = 0; T < 2; ++T) {
#pragma unroll
                    for (int n = 0; n < AT; ++n)
                        mma_u8s8(first, m.d[T][n], a[0][2 * T], a[0][2 * T + 1], a[1][2 * T], a[1][2 * T + 1], bx[j][n],
                                 BIAS);
                    mma_u8s8(first, m.lo[T], a[0][2 * T], a[0][2 * T + 1], a[1][2 * T], a[1][2 * T + 1], bx[j][AT],
                             BIAS);
                }
            };
            // the unit ends: acc += s step (D - z X), D = 256 (256 D_hi + D_mid) + D_lo
            // (sz: the group's s row)
            auto fold = [&](const Sums& m, const Unit& un, int hf, uint32_t sz) {
                uint64_t st[AT], x[AT];   // twice each; X negated
#pragma unroll
                for (int n = 0; n < AT; ++n) {
                    const float f = __uint_as_float(un.step[n]), v = -(float)un.X[n];
                    st[n] = pack2(f, f);
                    x[n] = pack2(v, v);
                }
                const uint2 sv = lds64_u32(sz), zv = lds64_u32(sz + sz_bytes / 2);
#pragma unroll
                for (int T = 0; T < 2; ++T) {   // columns 2 T and 2 T + 1
                    const float2 sf = T16::pair(T ? sv.y : sv.x), zf = T16::pair(T ? zv.y : zv.x);
                    const uint64_t s2 = pack2(sf.x, sf.y), z2 = pack2(zf.x, zf.y);
                    const float2 l0 = value2(m.lo[T][0], m.lo[T][1]), l1 = value2(m.lo[T][2], m.lo[T][3]);
#pragma unroll
                    for (int n = 0; n < AT; ++n) {
                        const int(&v)[4] = m.d[T][n];
                        const float2 h0 = value2(v[0], v[1]), h1 = value2(v[2], v[3]);
                        const uint64_t D = pack2(fmaf(256.0f, fmaf(256.0f, h0.x, h0.y), n ? l0.y : l0.x),
                                                 fmaf(256.0f, fmaf(256.0f, h1.x, h1.y), n ? l1.y : l1.x));
                        // (s step first: the other product can pass fp32's range where the result does not)
                        acc[hf][T][n] = fma2(mul2(s2, st[n]), fma2(z2, x[n], D), acc[hf][T][n]);
                    }
                }
            };
            // the halves h0 .. h1 - 1 of the stage from step i, unit by unit
            auto stage = [&](int h0, int h1, int i, int gleft) {
                const uint8_t* const st = smem + (warp * NST + slot) * STAGE;
                uint32_t sz = sz_ring + slot * sz_bytes + 8u * cg;   // the stage's first group
#pragma unroll
                for (int j0 = 0; j0 < SPS; j0 += U) {
                    if (j0 > 0 && i + j0 >= nq) break;
                    const Unit un = read_unit(i + j0, j0);
#pragma unroll
                    for (int hf = h0; hf < h1; ++hf) {
                        Sums m;
#pragma unroll
                        for (int j = 0; j < U; ++j) mult(m, j == 0, hf, st, j0 + j);
                        fold(m, un, hf, sz + (BITS == 4 ? 64u * hf : 0u));
                    }
                    if (U < SPS && (gleft -= U) == 0) {
                        gleft = p.spg;
                        sz += BITS == 4 ? 128u : 64u;
                    }
                }
            };
            auto wait = [&]() {
                if (ok) {
                    const bool good = mbar_wait_bounded(&bar[slot], phase, WAIT_NS);
                    if (!good) atomicOr(&g_moe_status, 1u);
                    ok = __all_sync(0xffffffffu, good);
                }
                return ok;
            };
            auto release = [&]() {   // every lane has read the stage: refill it
                __syncwarp();
                fence_proxy_async_smem();
                issue(slot);
                advance();
            };
            int gleft = p.spg - q0 % p.spg;   // steps left in the current group
#pragma unroll 1
            for (int i = 0; i < nq; i += SPS) {
                if constexpr (UP) request(i);
                if (!wait()) break;
                if constexpr (BITS == 4) {
                    stage(0, 2, i, gleft);
                } else {
                    stage(0, 1, i, gleft);
                    release();
                    if (!wait()) break;
                    stage(1, 2, i, gleft);
                }
                if (!UP && i + SPS < nq) request(i + SPS);
                release();
                if constexpr (U < SPS) {
                    gleft -= SPS;
                    while (gleft <= 0) gleft += p.spg;
                }
            }
            if constexpr (!UP) {
                if (p.rows != nullptr) {   // the rows of this (warp, block), to be summed at the end
                    if (!check(blk.first[it.u] + bm + p.bt * (rank * MW + warp) <= p.S + p.bt * MW * p.cluster,
                               &g_moe_status))
                        return;
                    float* const to = p.rows + ((size_t)it.tile * (p.S + p.bt * MW * p.cluster) + blk.first[it.u] +
                                                p.bt * (rank * MW + warp)) * TC + 4 * cg;
#pragma unroll
                    for (int n = 0; n < AT; ++n)
                        if (const int pos = 4 * n + t; pos < bm)
#pragma unroll
                            for (int hf = 0; hf < 2; ++hf)
                                *reinterpret_cast<ulonglong2*>(to + pos * TC + 32 * hf) =
                                    make_ulonglong2(acc[hf][0][n], acc[hf][1][n]);
                    return;
                }
                // y += weight * row, in the warp's own sums; slots that share a token lie in different lanes t or n,
                // which take turns
#pragma unroll
                for (int n = 0; n < AT; ++n)
#pragma unroll 1
                    for (int tt = 0; tt < 4; ++tt) {
                        if (4 * n + tt < bm && t == tt) {
                            float* const row = ys + yrow[n];
                            const uint64_t a = pack2(wt[n], wt[n]);
#pragma unroll
                            for (int hf = 0; hf < 2; ++hf) {
                                ulonglong2 v = *reinterpret_cast<ulonglong2*>(row + 32 * hf);
                                v.x = fma2(a, acc[hf][0][n], v.x);
                                v.y = fma2(a, acc[hf][1][n], v.y);
                                *reinterpret_cast<ulonglong2*>(row + 32 * hf) = v;
                            }
                        }
                        __syncwarp();
                    }
                return;
            }
            // ---- the warps' partials meet in shared memory, once every warp has read the last item's
            if (ok && done > 0) {
                const bool good = mbar_wait_bounded(&free_bar, (uint32_t)(done - 1) & 1u, WAIT_NS);
                if (!good) atomicOr(&g_moe_status, 1u);
                ok = __all_sync(0xffffffffu, good);
            }
#pragma unroll
            for (int n = 0; n < AT; ++n) {
                const int pos = 4 * n + t;
                if (pos < bm)
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf)
                        *reinterpret_cast<ulonglong2*>(red + (wk * p.bt + pos) * TC + MCOLS * wc + 32 * hf + 4 * cg) =
                            make_ulonglong2(acc[hf][0][n], acc[hf][1][n]);
            }
        };
        if (NT == 1 || bm <= 4) run(std::integral_constant<int, 1>{});
        else run(std::integral_constant<int, NT>{});
        if constexpr (UP) {
            __syncthreads();
            // The tile's TC / 2 values of h of one slot are one fixed-point block (128 or 64): LPS lanes, 4 each
            constexpr int LPS = TC / 8, SPW = 32 / LPS;
            const int c = 4 * (lane % LPS), cc = it.tile * (TC / 2) + c;
            // (by the warps in turn: the others go on to the next item)
            for (int pos0 = (warp + MW / 2 * done) % MW * SPW; pos0 < bm; pos0 += MW * SPW) {
                const int pos = min(pos0 + lane / LPS, bm - 1);
                const bool mine = pos0 + lane / LPS < bm;
                const float* const src = red + pos * TC + MCOLS * (c / 32) + c % 32;   // gate; its up column 32 on
                float4 ga = make_float4(0.0f, 0.0f, 0.0f, 0.0f), ua = ga;
#pragma unroll
                for (int w = 0; w < WK; ++w) {   // over the warps along K, in their order
                    const float4 a = *reinterpret_cast<const float4*>(src + w * p.bt * TC);
                    const float4 b = *reinterpret_cast<const float4*>(src + w * p.bt * TC + 32);
                    ga.x += a.x; ga.y += a.y; ga.z += a.z; ga.w += a.w;
                    ua.x += b.x; ua.y += b.y; ua.z += b.z; ua.w += b.w;
                }
                const float gv[4] = {ga.x, ga.y, ga.z, ga.w}, uv[4] = {ua.x, ua.y, ua.z, ua.w};
                float v[8] = {};
                uint32_t top = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (cc < p.I) v[i] = activate(gv[i], p.act) * uv[i];   // I is a multiple of 4
                    top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
                }
#pragma unroll
                for (int d = LPS / 2; d; d >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
                const uint32_t E = block_exponent(top);
                const Bytes b = to_fixed<8>(v, block_inverse(E));   // bytes 0 1 2 3 in .x
                int sum = value_sum(b);                             // of 8 lanes, a step, and of its unit (8, 16 or 32)
#pragma unroll
                for (int d = 1; d < 32; d <<= 1)
                    if (d < 8 << p.hlog) sum += __shfl_xor_sync(0xffffffffu, sum, d);
                const int slot = slots[pos], q = cc / SK;
                const size_t plane = (size_t)p.Qh * SK;
                int8_t* const row = p.hq + ((size_t)(3 * slot) * p.Qh + q) * SK;   // hi, then mid and lo, a plane each
                const bool in = mine && q < p.Qh && check(slot >= 0 && slot < p.S, &g_moe_status);
                if constexpr (BITS == 4) {
                    // a word row's 8 values are two lanes': the even one stores hi and lo, the odd one mid, as 0 2 4 6
                    // 1 3 5 7
                    const bool odd = lane & 1;
                    const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? b.hi.x : b.mid.x, 1);
                    const uint32_t lo2 = __shfl_xor_sync(0xffffffffu, b.lo.x, 1);
                    const uint32_t u0 = odd ? got : b.hi.x, u1 = odd ? b.mid.x : got;   // values 0-3 and 4-7
                    int8_t* const to = row + 8 * (c % SK / 8);
                    if (in) {
                        *reinterpret_cast<uint2*>(to + (odd ? plane : 0)) =
                            make_uint2(prmt(u0, u1, 0x6420u), prmt(u0, u1, 0x7531u));
                        if (!odd)
                            *reinterpret_cast<uint2*>(to + 2 * plane) =
                                make_uint2(prmt(b.lo.x, lo2, 0x6420u), prmt(b.lo.x, lo2, 0x7531u));
                    }
                } else if (in) {   // word row j of the step: bytes 8 (j % 4) + 4 (j / 4)
                    const int j = c % SK / 4, o = 8 * (j & 3) + 4 * (j >> 2);
                    *reinterpret_cast<uint32_t*>(row + o) = b.hi.x;
                    *reinterpret_cast<uint32_t*>(row + plane + o) = b.mid.x;
                    *reinterpret_cast<uint32_t*>(row + 2 * plane + o) = b.lo.x;
                }
                if (in && (lane & ((8 << p.hlog) - 1)) == 0)
                    p.hunit[(size_t)((slot * p.Qh + q) >> p.hlog)] =
                        make_uint2((uint32_t)sum, block_step(top, E));
            }
            ++done;
            __syncwarp();
            if (lane == 0) mbar_arrive(&free_bar);
        }
    }
    if (!ok)   // gave up a wait: give the copies still in flight as long again
        for (int i = 0; i < NST; ++i) {
            mbar_wait_bounded(&bar[slot], phase, WAIT_NS);
            advance();
        }
    if constexpr (!UP) {
        const int tl = (int)blockIdx.x / p.cluster;
        auto write = [&](int tok, int c, float4 v) {   // y[tok], columns c to c + 3 of the tile
            const int cc = tl * TC + c;
            if (cc >= p.NW) return;                    // N is a multiple of 4
            uint2 o;
            o.x = (uint32_t)T16::store(v.x) | ((uint32_t)T16::store(v.y) << 16);
            o.y = (uint32_t)T16::store(v.z) | ((uint32_t)T16::store(v.w) << 16);
            *reinterpret_cast<uint2*>(p.y + (size_t)tok * p.NW + cc) = o;
        };
        auto add = [](float4& v, const float4& o) {
            v.x += o.x;
            v.y += o.y;
            v.z += o.z;
            v.w += o.w;
        };
        const float4 zero = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (p.rows != nullptr) {
            // ---- the tile's rows are complete: every CTA sums those of its tokens (rank, rank + cluster, ..)
            if (p.cluster > 1) cluster_sync();
            else __syncthreads();
            // in the rings' place: where each warp's run starts; per slot its place in `order` and its block's warps
            const int nw = p.cluster * MW, ns = p.S + p.bt * nw;
            int* const starts = reinterpret_cast<int*>(smem);                        // nw + 1
            int16_t* const place = reinterpret_cast<int16_t*>(starts + 8 * MW + 1);  // S; then the first and the last warp
            int16_t* const wfirst = place + p.S;
            int16_t* const wlast = wfirst + p.S;
            float* const part = reinterpret_cast<float*>(smem + PART_AT);            // [slots of a few tokens][TC]
            const uint32_t part_at = smem_u32(part) - smem_u32(smem_raw);
            for (int i = threadIdx.x; i < p.S; i += MT) place[i] = -1;
            for (int w = threadIdx.x; w <= nw; w += MT) starts[w] = share(blk, Q4, w, nw);
            __syncthreads();
            for (int u = threadIdx.x; u < nblocks; u += MT) {
                int w0 = 0, w1 = nw;
                while (w0 < nw - 1 && starts[w0 + 1] <= u * Q4) ++w0;
                while (w1 > w0 + 1 && starts[w1 - 1] >= (u + 1) * Q4) --w1;
                for (int i = blk.first[u]; i < blk.first[u + 1]; ++i) {
                    place[blk.order[i]] = (int16_t)i;
                    wfirst[blk.order[i]] = (int16_t)w0;
                    wlast[blk.order[i]] = (int16_t)w1;
                }
            }
            __syncthreads();
            const int step = tokens_at_once(p.top_k);
            for (int k0 = 0; rank + k0 * p.cluster < p.T; k0 += step) {
                const int nt = min(step, (p.T - rank - k0 * p.cluster + p.cluster - 1) / p.cluster);
                for (int i = threadIdx.x; i < nt * p.top_k * (TC / 4); i += MT) {
                    const int r = i / (TC / 4), c = 4 * (i % (TC / 4));
                    const int sl = (rank + (k0 + r / p.top_k) * p.cluster) * p.top_k + r % p.top_k;
                    float4 v = zero;
                    if (check(sl < p.S, &g_moe_status) && place[sl] >= 0 &&
                        check(place[sl] + p.bt * (wlast[sl] - 1) < ns && wlast[sl] <= nw, &g_moe_status)) {
                        const float a = p.weights[sl];
                        const float* const from = p.rows + ((size_t)tl * ns + place[sl]) * TC + c;
                        for (int w = wfirst[sl]; w < wlast[sl]; w += 2) {   // (a run may be empty)
                            float4 o0 = zero, o1 = zero;
                            if (starts[w] < starts[w + 1])
                                o0 = __ldcg(reinterpret_cast<const float4*>(from + (size_t)p.bt * w * TC));
                            if (w + 1 < wlast[sl] && starts[w + 1] < starts[w + 2])
                                o1 = __ldcg(reinterpret_cast<const float4*>(from + (size_t)p.bt * (w + 1) * TC));
                            add(v, o0);
                            add(v, o1);
                        }
                        v = make_float4(a * v.x, a * v.y, a * v.z, a * v.w);
                    }
                    if (check(part_at + 16u * i + 16u <= dynamic_smem_bytes(), &g_moe_status))
                        *reinterpret_cast<float4*>(part + 4 * i) = v;
                }
                __syncthreads();
                for (int i = threadIdx.x; i < nt * (TC / 4); i += MT) {
                    const int k = i / (TC / 4), c = 4 * (i % (TC / 4));
                    float4 v = zero;
                    for (int j = 0; j < p.top_k; ++j)
                        add(v, *reinterpret_cast<const float4*>(part + (k * p.top_k + j) * TC + c));
                    write(rank + (k0 + k) * p.cluster, c, v);
                }
                __syncthreads();
            }
            return;
        }
        // ---- the warps join their sums, then the tile's CTAs, each in their order; each CTA writes its share of y
        __syncthreads();
        for (int i = threadIdx.x; i < p.T * (TC / 4); i += MT) {
            float4 v = *reinterpret_cast<const float4*>(ys + 4 * i);
#pragma unroll
            for (int w = 1; w < MW; ++w) add(v, *reinterpret_cast<const float4*>(ys + w * p.T * TC + 4 * i));
            *reinterpret_cast<float4*>(ys + 4 * i) = v;
        }
        if (p.cluster > 1) cluster_sync();
        else __syncthreads();
        const uint32_t at = smem_u32(ys);
        for (int i = rank + p.cluster * (int)threadIdx.x; i < p.T * (TC / 4); i += p.cluster * MT) {
            float4 v = zero;
            if (p.cluster == 1) v = *reinterpret_cast<const float4*>(ys + 4 * i);
            else
                for (int r = 0; r < p.cluster; ++r) add(v, ld_cluster_f4(map_shared_rank(at + 16u * i, r)));
            write(i / (TC / 4), 4 * (i % (TC / 4)), v);
        }
        __syncwarp();
        if (p.cluster > 1) cluster_sync();   // peers keep their shared memory until every read is done
    }
}

// Dynamic shared memory a CTA of 12 or 16 warps (one per SM), or of 6 or 8 (two), can have.  (227 KB, less 320 bytes for
// the static part.)
constexpr int WHOLE_SM = 227 * 1024 - 320;
constexpr int max_smem(int W) { return W > 8 ? WHOLE_SM : 112 * 1024; }
constexpr int ring_bytes(int W, int bits, int sz_rows) { return 1024 + W * NST * (STAGE + sz_space(bits, sz_rows)); }
// s rows of the groups that a stage of `sps` steps, starting at a multiple of them, can touch.
int stage_groups(int spg, int sps) { return spg % sps == 0 ? 1 : std::min(sps, (sps - 1) / spg + 2); }

int xcol_bytes(int steps) {   // 32 mod 128: the four columns of a load phase lie in different banks
    const int b = (steps + XBLK - 1) / XBLK * XBLK * 32;
    return b + (160 - b % 128) % 128;
}
// How a product of inner length K is cut.
struct Cut {
    int bits, spg, sz_rows;   // steps per group, s rows per stage
    int bt;               // slots per block
    int W, cluster;       // warps; CTAs per column tile (DOWN)
    bool rows;            // DOWN: rows in global memory instead of the warps' own sums
    int xcol, nunits, nblk, smem;
    int ulog;             // steps per unit, log2: the most, up to a fixed-point block, that no group ends inside
};
int unit_log(int spg) { return spg % 4 == 0 ? 2 : spg % 2 == 0 ? 1 : 0; }

// DOWN with rows: the most that a CTA stages at a time, its tokens' slots.
int staged_rows(int T, int top_k, int cluster) {
    return std::min(tokens_at_once(top_k), (T + cluster - 1) / cluster) * top_k;
}

void cut_smem(Cut& c, bool up, int T, int S, int E, int Q) {
    c.xcol = up ? xcol_bytes(Q) : 0;
    c.nunits = up ? (Q + (1 << c.ulog) - 1) >> c.ulog : 0;
    c.nblk = most_blocks(S, E, c.bt);
    c.smem = ring_bytes(c.W, c.bits, c.sz_rows) + (up ? units_at(c.W, c.bt, S, c.nblk, c.xcol) + c.bt * c.nunits * 8
                                              : values_at(0, c.bt, S, c.nblk) + (c.rows ? 0 : c.W * T * MCOLS * 4));
    if (!up && c.rows) c.smem = std::max(c.smem, 1024 + PART_AT + staged_rows(T, S / T, c.cluster) * MCOLS * 4);
}

// UP: blocks take as many slots, at most 8 and no more than the tokens can fill, as their fixed-point values
// leave room for (bt = 0: K is too long).
//  * Few tokens, and no more tiles of 64 values of h than SMs: CTAs of 8 warps, beside which DOWN's start while
//    they run (1 token, 8 experts of 2048 x 1024: 14.7 us against 18.7 us with 16, of 7168 x 512 27.2 against 32.7; on
//    an earlier form, with 344 tiles, 2 experts of 4096 x 11008, 54 us against 41.5 us; 4 tokens, 32 experts of
//    2048 x 1024, 36.6 us against 30.2 us).
//  * Else one CTA per SM and tiles of 128 values, 3 or 4 warps along K.  (Tiles of 64, where that fills the SMs' last
//    round better, measured slower on an earlier form: DOWN's shorter fixed-point blocks cost more.  16 tokens, 64
//    experts of 2048 x 1024: 96 us against 81 us.  So did pairs of CTAs that halve the odd item of their part of the
//    line: 48 tokens, 8-bit, 99 us against 88 us, though 1 token, 2 experts of 4096 x 11008, took 40 us against 42 us.)
//  * Very long K with few tokens and short groups, where 16 warps' rings leave no room: 8 warps, one CTA per SM.
Cut cut_up(int T, int S, int E, int K, int I, int group_size, int bits) {
    const int Q = (K + SK - 1) / SK;
    Cut c{};
    c.spg = group_size == -1 || group_size == K ? 1 << 29 : group_size / SK;
    c.bits = bits;
    c.sz_rows = stage_groups(c.spg, XBLK);
    c.ulog = unit_log(c.spg);
    c.cluster = 1;
    if (T <= 4 && (long long)((I + 63) / 64) * std::min(S, E) <= sm_count()) {
        c.W = 8;
        c.bt = T;
        cut_smem(c, true, T, S, E, Q);
        if (c.smem <= max_smem(8)) return c;
    }
    c.W = up_warps(T <= 4 ? 1 : 2);
    for (c.bt = std::min(T, MAXBT); c.bt > 0; --c.bt) {
        cut_smem(c, true, T, S, E, Q);
        if (c.smem <= max_smem(c.W)) return c;
    }
    c.W = T <= 4 ? 8 : c.W;
    c.bt = 1;
    cut_smem(c, true, T, S, E, Q);
    if (c.smem > WHOLE_SM) c.bt = 0;
    return c;
}

// Clusters of cs CTAs of DOWN, two per SM, that the device holds at once (a GPC's SMs are not a multiple of
// every size: 15 clusters of 8 with one CTA per SM on a B200, not 148 / 8 = 18).  Asked once per device.
int clusters_that_fit(int cs) {
    static std::atomic<int> known[MAX_DEVICES][9];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= MAX_DEVICES) return 2 * sm_count() / cs;
    int n = known[dev][cs].load(std::memory_order_relaxed);
    if (n > 0) return n;
    n = 2 * sm_count() / cs;
    if (cs > 1) {
        auto kern = moe_kernel<4, false, 1, false, down_warps(1), XBLK>;
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(cs, 1, 1);
        cfg.blockDim = dim3(down_warps(1) * 32, 1, 1);
        cfg.dynamicSmemBytes = max_smem(8);
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = cs;
        attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        int found = 0;
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, max_smem(8)) == cudaSuccess &&
            cudaOccupancyMaxActiveClusters(&found, kern, &cfg) == cudaSuccess && found > 0)
            n = found;
        else
            cudaGetLastError();
    }
    known[dev][cs].store(n, std::memory_order_relaxed);
    return n;
}

// DOWN with clusters of a given size.
Cut cut_down(int T, int S, int E, int I, int group_size, int bits, int cluster) {
    Cut c{};
    c.W = down_warps(T <= 4 ? 1 : 2);
    c.spg = group_size == -1 || group_size == I ? 1 << 29 : group_size / SK;
    c.bits = bits;
    c.sz_rows = stage_groups(c.spg, XBLK);
    c.bt = T <= 4 ? 4 : MAXBT;
    c.ulog = unit_log(c.spg);
    c.cluster = cluster;
    c.rows = T > SUMS_T;
    cut_smem(c, false, T, S, E, 0);   // (at most 92 KB)
    return c;
}

// DOWN: a column tile is worked on by a cluster, of the size that leaves the fewest places of the SMs without a CTA:
// two per SM, or one when there is little to do and UP still holds the other.  (A sixteenth of the clusters that fit
// an empty device is kept back: 32 clusters of 8 where 33 fit ran in two waves behind UP.)
Cut cut_down(int T, int S, int E, int I, int N, int group_size, int bits, bool few) {
    const int places = few ? sm_count() : 2 * sm_count();
    const int tiles = (N + MCOLS - 1) / MCOLS;
    int best = -1, cluster = 1;   // places taken, in percent
    for (int cs = 1; cs <= 8; ++cs) {
        const int held = clusters_that_fit(cs), all = held - (cs > 1 ? (held + 15) / 16 : 0);
        const int fit = std::max(1, few ? all / 2 : all);
        const int waves = (tiles + fit - 1) / fit, use = (int)(100ll * tiles * cs / ((long long)waves * places));
        if (use > best + 2) {
            best = use;
            cluster = cs;
        }
    }
    return cut_down(T, S, E, I, group_size, bits, cluster);
}

template <int BITS, bool BF, int NT, bool UP, int W, int U>
wq_status launch_kernel(const CUtensorMap (&tm)[3], const MoeParams& p, int smem, bool pdl, cudaStream_t stream) {
    auto kern = moe_kernel<BITS, BF, NT, UP, W, U>;
    static std::atomic<uint64_t> attr_ctx[MAX_DEVICES];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return WQ_ERR_CUDA;
    if (const wq_status st = ensure_smem_attr((const void*)kern, UP ? WHOLE_SM : max_smem(W), attr_ctx, dev); st != WQ_OK) return st;
    cudaLaunchConfig_t cfg{};
    const long long ctas = UP ? std::min<long long>(sm_count() * (16 / W), (long long)p.nblk * p.ntiles)
                              : (long long)p.ntiles * p.cluster;
    cfg.gridDim = dim3((unsigned)ctas, 1, 1);
    cfg.blockDim = dim3(W * 32, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attrs[2];
    int na = 0;
    if (!UP && p.cluster > 1) {
        attrs[na].id = cudaLaunchAttributeClusterDimension;
        attrs[na].val.clusterDim.x = p.cluster;
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
    return from_cuda(cudaLaunchKernelEx(&cfg, kern, tm[0], tm[1], tm[2], p));
}

template <int BITS, bool BF, int NT, bool UP, int W>
wq_status launch_one(const CUtensorMap (&tm)[3], const MoeParams& p, const Cut& c, bool pdl, cudaStream_t stream) {
    switch (UP ? c.ulog : p.hlog) {
        case 2: return launch_kernel<BITS, BF, NT, UP, W, 4>(tm, p, c.smem, pdl, stream);
        case 1: return launch_kernel<BITS, BF, NT, UP, W, 2>(tm, p, c.smem, pdl, stream);
        default: return launch_kernel<BITS, BF, NT, UP, W, 1>(tm, p, c.smem, pdl, stream);
    }
}

// One product: its shape, its launch.
template <int BITS, bool BF, bool UP>
wq_status run_product(MoeParams& p, const uint32_t* w, const uint16_t* s, const uint16_t* z, int K, int group_size,
                      const Cut& c, bool pdl, cudaStream_t stream) {
    p.K = K;
    p.Kw = K * BITS / 32;
    p.Q = (K + SK - 1) / SK;
    p.bt = c.bt; p.spg = c.spg; p.sz_rows = c.sz_rows;
    p.cluster = c.cluster; p.xcol = c.xcol; p.nunits = c.nunits; p.nblk = c.nblk;
    p.groups = group_size == -1 ? 1 : K / group_size;
    // UP: planes of I columns, gate and up; DOWN: rows of N columns (words in boxes of 32; 4-bit: s and z of both halves)
    CUtensorMap tm[3];
    const uint64_t cols = UP ? p.I : p.NW, planes = UP ? 2 : 1, wrows = (uint64_t)p.E * p.Kw;
    const uint64_t srows = (uint64_t)p.E * p.groups;
    const uint32_t sc = UP || BITS == 8 ? 32 : 64, bp = UP && BITS == 4 ? 2 : 1;
    const int dims = UP ? 3 : 2;
    if (!make_map_rows(&tm[0], CU_TENSOR_MAP_DATA_TYPE_UINT32, w, 4, dims, cols, planes, wrows, 32, bp,
                       stage_rows<BITS>(),
                       CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_map_rows(&tm[1], CU_TENSOR_MAP_DATA_TYPE_UINT16, s, 2, dims, cols, planes, srows, sc, bp, p.sz_rows,
                       CU_TENSOR_MAP_SWIZZLE_NONE) ||
        !make_map_rows(&tm[2], CU_TENSOR_MAP_DATA_TYPE_UINT16, z, 2, dims, cols, planes, srows, sc, bp, p.sz_rows,
                       CU_TENSOR_MAP_SWIZZLE_NONE))
        return WQ_ERR_CUDA;
    const int tc = UP ? MCOLS / 2 * (c.W / along_k(c.W)) : MCOLS;   // columns of h or y per tile
    p.ntiles = ((UP ? p.I : p.NW) + tc - 1) / tc;
    if constexpr (UP) {
        if (c.W == 8) return launch_one<BITS, BF, 1, UP, 8>(tm, p, c, pdl, stream);
        return c.W == up_warps(1) ? launch_one<BITS, BF, 1, UP, up_warps(1)>(tm, p, c, pdl, stream)
                         : launch_one<BITS, BF, 2, UP, up_warps(2)>(tm, p, c, pdl, stream);
    } else {
        return c.bt <= 4 ? launch_one<BITS, BF, 1, UP, down_warps(1)>(tm, p, c, pdl, stream)
                         : launch_one<BITS, BF, 2, UP, down_warps(2)>(tm, p, c, pdl, stream);
    }
}

// Workspace: h's three bytes per value, then its units (at most one per step of K); then DOWN's rows.
int h_steps(int I) { return (I + SK * XBLK - 1) / (SK * XBLK) * XBLK; }   // whole stages
size_t h_bytes(int S, int I) {
    const size_t rows = (size_t)S * h_steps(I);
    return (rows * (3 * SK + 8) + 255) & ~(size_t)255;
}

template <int BITS, bool BF>
wq_status run_moe(const MoeProblem& m, cudaStream_t stream) {
    MoeParams p{};
    p.x = m.x; p.ids = m.ids; p.weights = m.weights; p.y = m.y;
    p.T = m.T; p.top_k = m.top_k; p.S = m.T * m.top_k; p.E = m.E; p.I = m.I; p.act = m.act;
    // the cuts of this thread's last shape: a decode loop asks for the same ones again (per device: two with the same SMs
    // may hold different numbers of clusters)
    struct Plan {
        int T, S, E, K, I, N, group_size, dev;
        Cut up, down;
    };
    static thread_local Plan last{};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return WQ_ERR_CUDA;
    if (last.T != p.T || last.S != p.S || last.E != p.E || last.K != m.K || last.I != m.I || last.N != m.N ||
        last.group_size != m.group_size || last.dev != dev) {
        last = Plan{p.T, p.S, p.E, m.K, m.I, m.N, m.group_size, dev, {}, {}};
        last.up = cut_up(m.T, p.S, p.E, m.K, m.I, m.group_size, BITS);
        last.down = cut_down(m.T, p.S, m.E, m.I, m.N, m.group_size, BITS, last.up.W == 8);
    }
    const Cut up = last.up, down = last.down;
    p.Qh = h_steps(m.I);
    const int hb = MCOLS * (up.W / along_k(up.W)) / 2 / SK;   // a tile of UP, steps of h: 4, or 2
    p.hlog = std::min(down.ulog, hb / 2);                     // (4 steps: 2, 2 steps: 1)
    // (before anything is launched: what must fit 31 bits -- the weighted line of work, word rows, CTAs)
    const long long units = std::max((m.I + 31) / 32, (p.Qh + XBLK - 1) / XBLK), most = 1ll << 31;
    if (up.bt == 0 || down.bt == 0 || p.S * 5 * units >= most || (long long)p.E * (m.K * BITS / 32) >= most ||
        (long long)p.E * ((long long)m.I * BITS / 32) >= most || (m.N + 63ll) / 64 * 8 >= most)
        return WQ_ERR_UNSUPPORTED;
    p.hq = static_cast<int8_t*>(m.ws);
    p.hunit = reinterpret_cast<uint2*>(p.hq + (size_t)3 * p.S * p.Qh * SK);
    if (down.rows) p.rows = reinterpret_cast<float*>(static_cast<uint8_t*>(m.ws) + h_bytes(p.S, m.I));
    p.NW = 2 * m.I;
    const wq_status st = run_product<BITS, BF, true>(p, m.w_up, m.s_up, m.z_up, m.K, m.group_size, up,
                                                     (m.flags & WQ_FLAG_PDL) != 0, stream);
    if (st != WQ_OK) return st;
    p.NW = m.N;
    return run_product<BITS, BF, false>(p, m.w_down, m.s_down, m.z_down, m.I, m.group_size, down, true, stream);
}

}  // namespace

size_t moe_workspace_bytes(int T, int top_k, int I, int N) {
    const size_t tiles = (N + MCOLS - 1) / MCOLS, rows = (size_t)T * top_k + MAXBT * 64;   // 64 warps in the largest cluster
    return h_bytes(T * top_k, I) + (T > SUMS_T ? tiles * rows * MCOLS * 4 : 0);
}

// What DOWN asks for with clusters of the given size, and the end of what it touches (the round-up of the rings to 1024
// bytes among it).
size_t moe_down_smem(int T, int top_k, int I, int bits, int group_size, int cluster, size_t* used) {
    const Cut c = cut_down(T, T * top_k, WQ_MOE_MAX_EXPERTS, I, group_size, bits, cluster);
    const int tables = ring_bytes(c.W, bits, c.sz_rows) - 1 + values_at(0, c.bt, T * top_k, c.nblk);
    *used = c.rows ? std::max(tables, 1023 + PART_AT + staged_rows(T, top_k, cluster) * MCOLS * 4)
                   : tables + c.W * T * MCOLS * 4;
    return c.smem;
}

wq_status launch_moe(const MoeProblem& m, cudaStream_t stream) {
    const bool bf = (m.flags & WQ_FLAG_BF16) != 0;
    if (m.bits == 4) return bf ? run_moe<4, true>(m, stream) : run_moe<4, false>(m, stream);
    return bf ? run_moe<8, true>(m, stream) : run_moe<8, false>(m, stream);
}

wq_status moe_device_status(int reset) {
    unsigned int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_moe_status, sizeof(v)) != cudaSuccess) return WQ_ERR_CUDA;
    if (reset) {
        const unsigned int zero = 0;
        if (cudaMemcpyToSymbol(g_moe_status, &zero, sizeof(zero)) != cudaSuccess) return WQ_ERR_CUDA;
    }
    return (v & 1u) ? WQ_ERR_TIMEOUT : (v & 2u) ? WQ_ERR_CHECK : WQ_OK;
}

}  // namespace wq
