// wq_moe.cu -- a mixture-of-experts layer on packed weights, for a few tokens.
//
// What is computed: for token t and its top_k slots (t, j) with expert
// e = ids[t][j] and weight a = weights[t][j],
//   h = act(x[t] @ Wg[e]) * (x[t] @ Wu[e])           (gate and up: one packed array, 2 I columns)
//   y[t] = sum_j a * (h[t][j] @ Wd[e])
// with W = (q - z) * s as everywhere in this library.  A slot whose id lies
// outside 0 .. E-1 is empty and adds nothing.
//
// Two launches of one kernel template.  UP turns x into h; DOWN turns h into
// one fp32 row per slot, and the last CTA of a column tile to finish sums the
// slots of each token, in slot order, and writes y.  Both are bound by HBM: the
// layer reads each chosen expert's words once.
//  * Work split.  Slots are grouped by expert into blocks of BT slots, so an
//    expert's words are read once for all its tokens.  The grid is (column
//    tiles, an upper bound of the number of blocks); every CTA derives its block
//    from the ids and the surplus CTAs leave.  A CTA owns 64 columns (UP: 32
//    gate and the matching 32 up columns, so the activation needs no second
//    pass) and its 8 warps split K; partials meet in shared memory.
//  * Loads.  A warp walks its K range in quads (4 word rows) through a private
//    ring of stages filled by cp.async: lane (g, t) (g = lane / 4, t = lane % 4)
//    copies the 16 bytes (4 columns of word row 4 q + t) that it will itself
//    convert, so words need no barrier and meet no bank conflict; only s and z,
//    copied where a group starts, are read across lanes.
//  * Products (m16n8k16 warp MMA, fp32 accumulators): A holds codes, B the
//    tokens.  A code needs only AND / OR to become an operand: in fp16 the code
//    bits are the subnormal q 2^-24, which the tensor core multiplies exactly; in
//    bf16 4-bit codes are ORed into 128 (0x4300) and 8-bit ones go through fp32.
//    One more MMA per k step with A = 1 gives X, the tokens' sums over the group,
//    so a zero point of any value costs nothing per code: with D the group's
//    product, acc += s (D - (128 + z) X) in fp32 (no 128 in fp16).
//  * h is kept as two bf16 values, h = hi + lo (16 significant bits: 2^-17
//    relative, far below the output's own rounding, and fp32's range, so an fp16
//    layer cannot overflow between the products).  hi and lo of a token are two
//    adjacent columns of the MMA, whose sum the fold takes.
//  * DOWN is a programmatic dependent of UP: it finds its block and requests its
//    first words while UP drains, and waits only before it reads h.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

#include "wq_dequant.cuh"
#include "wq_internal.h"
#include "wq_ptx.cuh"

namespace wq {

// Device status of these kernels: bit 1 once a check of the checked build failed.
__device__ unsigned int g_moe_status = 0;

namespace {

constexpr int MW = 8;           // warps per CTA, split along K
constexpr int MT = MW * 32;
constexpr int MCOLS = 64;       // weight columns per CTA (two halves of 32)
constexpr int SZ_BYTES = 256;   // s and z of the 64 columns, one group
constexpr int W_BYTES = 1024;   // one quad: 4 word rows x 64 columns

struct MoeParams {
    const uint16_t* x;      // UP: (T, K); DOWN: null
    uint16_t* h;            // (2, S, I) bf16: hi, then lo
    const int32_t* ids;     // (T, top_k)
    const float* weights;   // (T, top_k)
    const uint32_t* w;      // (E, Kw, NW) words of this product
    const uint16_t* s;      // (E, groups, NW)
    const uint16_t* z;
    float* part;            // (S, N): DOWN's rows per slot
    unsigned int* count;    // arrivals per DOWN column tile
    uint16_t* y;            // (T, N)
    int T, top_k, S, E;
    int K;                  // inner length of this product (UP: K of x, DOWN: I)
    int NW;                 // weight columns (UP: 2 I, DOWN: N)
    int NC;                 // columns the tiles cover (UP: I, DOWN: N)
    int I;
    int Kw, Q, QW;          // word rows, quads, quads per warp
    int qpg;                // quads per group (large when one group spans K)
    int groups;
    int act;
    int ntiles_down;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The block of a CTA: up to BT slots of one expert.
struct Block {
    int e, m, nblocks;  // expert, slots in the block, blocks in the whole launch
};

struct Lists {
    int slots[MW][16];   // per warp: the block's slots (S <= 32), or row 0 for the whole CTA
    int found[2];        // expert and slot count of the block
    int total;
};
// Scratch of find_block while the ring holds nothing yet: slots per expert, the ids.
struct Counts {
    int cnt[WQ_MOE_MAX_EXPERTS];
    int ids[WQ_MOE_MAX_SLOTS];
};

// Block u of the launch: experts in the order of their first slot (S <= 32) or
// of their number, slots in ascending order, BT per block.  Every warp gets
// the result; the slots are in l.slots[warp] or, S > 32, l.slots[0].
template <int BT>
__device__ __forceinline__ Block find_block(const MoeParams& p, int u, Lists& l, Counts& c) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const unsigned lt = (1u << lane) - 1u;
    Block b;
    if (p.S <= 32) {  // one slot per lane: no shared counts and no CTA barrier
        const int id = lane < p.S ? p.ids[lane] : -1;
        const bool valid = id >= 0 && id < p.E;
        const unsigned same = __match_any_sync(0xffffffffu, valid ? id : -1 - lane);
        const bool leader = valid && (same & lt) == 0;
        const int nb = leader ? (__popc(same) + BT - 1) / BT : 0;
        int pre = nb;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, pre, d);
            if (lane >= d) pre += v;
        }
        b.nblocks = __shfl_sync(0xffffffffu, pre, 31);
        pre -= nb;
        const unsigned hit = __ballot_sync(0xffffffffu, u >= pre && u < pre + nb);
        if (hit == 0) {
            b.e = b.m = 0;
            return b;
        }
        const int src = __ffs(hit) - 1;
        b.e = __shfl_sync(0xffffffffu, id, src);
        const unsigned mine = __shfl_sync(0xffffffffu, same, src);
        const int first = BT * (u - __shfl_sync(0xffffffffu, pre, src));
        b.m = min(BT, __popc(mine) - first);
        const int r = __popc(mine & lt) - first;
        if (((mine >> lane) & 1u) && r >= 0 && r < BT) l.slots[warp][r] = lane;
        __syncwarp();
        return b;
    }
    for (int e = threadIdx.x; e < p.E; e += MT) c.cnt[e] = 0;
    if (threadIdx.x < 2) l.found[threadIdx.x] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < p.S; i += MT) {
        const int id = p.ids[i];
        c.ids[i] = id;
        if (id >= 0 && id < p.E) atomicAdd(&c.cnt[id], 1);
    }
    __syncthreads();
    if (warp == 0) {
        const int per = (p.E + 31) / 32;
        int mine = 0;
        for (int j = 0; j < per; ++j) {
            const int e = lane * per + j;
            mine += e < p.E ? (c.cnt[e] + BT - 1) / BT : 0;
        }
        int pre = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, pre, d);
            if (lane >= d) pre += v;
        }
        if (lane == 31) l.total = pre;
        pre -= mine;
        int e0 = -1, first = 0, m = 0;
        if (u >= pre && u < pre + mine) {
            for (int j = 0; j < per; ++j) {
                const int e = lane * per + j;
                const int nb = e < p.E ? (c.cnt[e] + BT - 1) / BT : 0;
                if (u < pre + nb) {
                    e0 = e;
                    first = BT * (u - pre);
                    m = min(BT, c.cnt[e] - first);
                    break;
                }
                pre += nb;
            }
        }
        const unsigned hit = __ballot_sync(0xffffffffu, e0 >= 0);
        if (hit != 0) {
            const int src = __ffs(hit) - 1;
            e0 = __shfl_sync(0xffffffffu, e0, src);
            first = __shfl_sync(0xffffffffu, first, src);
            m = __shfl_sync(0xffffffffu, m, src);
            int base = -first;
            for (int i0 = 0; i0 < p.S && base < BT; i0 += 32) {
                const bool is = i0 + lane < p.S && c.ids[i0 + lane] == e0;
                const unsigned mask = __ballot_sync(0xffffffffu, is);
                const int r = base + __popc(mask & lt);
                if (is && r >= 0 && r < BT) l.slots[0][r] = i0 + lane;
                base += __popc(mask);
            }
            if (lane == 0) {
                l.found[0] = e0;
                l.found[1] = m;
            }
        }
    }
    __syncthreads();
    b.e = l.found[0];
    b.m = l.found[1];
    b.nblocks = l.total;
    return b;
}

// Code pair j of a word as an MMA operand register (codes j and j + EPS / 2).
template <int BITS, bool BF>
__device__ __forceinline__ uint32_t code_pair(uint32_t w, int j) {
    if constexpr (BITS == 4) {
        return BF ? and_or(w >> (4 * j), 0x000F000Fu, 0x43004300u) : (w >> (4 * j)) & 0x000F000Fu;
    } else if constexpr (!BF) {
        return prmt(w, 0u, j == 0 ? 0x4240u : 0x4341u);
    } else {
        const float lo = __uint_as_float(prmt(w, 0x4B000000u, 0x7440u + j)) - 8388608.0f;
        const float hi = __uint_as_float(prmt(w, 0x4B000000u, 0x7442u + j)) - 8388608.0f;
        const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&v);
    }
}

__device__ __forceinline__ float activate(float g, int act) {
    if (act == WQ_ACT_SILU) return g / (1.0f + __expf(-g));
    return 0.5f * g * erfcf(-0.70710678118654752f * g);  // gelu
}

// Ring stages per warp: two CTAs of 8 warps fit an SM and keep 96 KB of words
// in flight with one token tile (80 KB with two, 64 KB with four, whose rows
// take twice the shared memory of the words).
template <int NT> constexpr int stages() { return NT > 2 ? 4 : 5 + (NT == 1); }
template <int BITS> constexpr int xt_bytes() { return BITS == 4 ? 512 : 256; }  // one token tile of a quad
template <int BITS, int NT> constexpr int stage_bytes() { return W_BYTES + SZ_BYTES + NT * xt_bytes<BITS>(); }

// NT: token tiles of 8 MMA columns (UP: 8 slots each, DOWN: 4 slots as hi, lo).
template <int BITS, bool BF, int NT, bool UP>
__global__ void __launch_bounds__(MT, NT > 2 ? 1 : 2) moe_kernel(const MoeParams p) {
    using T16 = Dt<BF>;
    constexpr bool MBF = UP ? BF : true;        // MMA operand type: x's, or bf16 for h
    constexpr int EPS = 32 / BITS;
    constexpr int MMAS = EPS / 4;               // k steps per quad
    constexpr int TPT = UP ? 8 : 4;             // slots per token tile
    constexpr int BT = TPT * NT;
    constexpr int NE = UP ? 2 : 1;              // slots per lane and tile
    constexpr int ST = stages<NT>();
    constexpr int SB = stage_bytes<BITS, NT>();
    constexpr float DSCALE = MBF ? 1.0f : 16777216.0f;              // fp16 operands are q 2^-24
    constexpr float ZOFF = (MBF && BITS == 4) ? 128.0f : 0.0f;      // bf16 4-bit operands are 128 + q
    static_assert(BT <= 16 && BT * MCOLS * 4 <= ST * SB, "partials reuse the ring");
    static_assert(sizeof(Counts) <= MW * ST * SB, "the counts lie in the ring before its first load");
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ Lists lists;
    __shared__ int last;

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int tile = blockIdx.x;
    if constexpr (UP) {
        grid_dependency_wait();   // ids, weights and x may be the previous kernel's output
        if (blockIdx.y == 0 && tile == 0)
            for (int i = threadIdx.x; i < p.ntiles_down; i += MT) p.count[i] = 0;
    }
    grid_launch_dependents();
    const Block b = find_block<BT>(p, blockIdx.y, lists, *reinterpret_cast<Counts*>(smem));
    if ((int)blockIdx.y >= b.nblocks && !(!UP && blockIdx.y == 0)) return;
    const int* slots = lists.slots[p.S <= 32 ? warp : 0];

    // ---- this warp's quads
    const int q0 = min(p.Q, warp * p.QW), nq = b.m > 0 ? min(p.Q, q0 + p.QW) - q0 : 0;
    const uint32_t ring = smem_u32(smem) + (uint32_t)warp * (ST * SB);
    // first column of half hf, clamped so that the ragged last tile reads inside the row
    auto col = [&](int hf, int c) {
        if constexpr (UP) return hf * p.I + min(tile * 32 + c, p.I - 4);
        else return min(tile * MCOLS + 32 * hf + c, p.NW - 4);
    };
    const uint32_t* wp[2];
    const size_t wexp = (size_t)b.e * p.Kw * p.NW, szexp = (size_t)b.e * p.groups * p.NW;
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) wp[hf] = p.w + wexp + col(hf, 4 * g);
    // lane (g, t): t = 0, 1 copies s, z of half 0, t = 2, 3 of half 1
    const uint16_t* szp = ((t & 1) ? p.z : p.s) + szexp + col(t >> 1, 4 * g);
    // B operand rows: UP slot g of each tile; DOWN slot g / 2, hi (even g) or lo (odd g)
    const uint16_t* xp[NT];
    bool xon[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int pos = n * TPT + (UP ? g : g >> 1);
        xon[n] = pos < b.m;
        const int slot = xon[n] ? slots[pos] : 0;
        if constexpr (UP) xp[n] = p.x + (size_t)(slot / p.top_k) * p.K;
        else xp[n] = p.h + (size_t)(g & 1) * p.S * p.I + (size_t)slot * p.I;
        check(slot >= 0 && slot < p.S, &g_moe_status);
    }
    auto issue_w = [&](int i) {   // words (and s, z where a group starts) of quad i
        if (i < nq) {
            const int q = q0 + i;
            const uint32_t st = ring + (uint32_t)(i % ST) * SB;
            const size_t row = (size_t)min(4 * q + t, p.Kw - 1) * p.NW;
#pragma unroll
            for (int hf = 0; hf < 2; ++hf)
                if (check(b.e < p.E && row + col(hf, 4 * g) + 4 <= (size_t)p.Kw * p.NW, &g_moe_status))
                    cp_async16(st + 512u * hf + 16u * lane, wp[hf] + row);
            if (i == 0 || q % p.qpg == 0) {
                const int grp = q / p.qpg;
                if (check(grp < p.groups, &g_moe_status))
                    cp_async8(st + W_BYTES + 64u * t + 8u * g, szp + (size_t)grp * p.NW);
            }
        }
    };
    auto issue_x = [&](int i) {   // the tokens' values of quad i
        if (i < nq) {
            const int r = 4 * (q0 + i) + t;
            const uint32_t st = ring + (uint32_t)(i % ST) * SB + W_BYTES + SZ_BYTES;
#pragma unroll
            for (int n = 0; n < NT; ++n)
                if (xon[n] && r < p.Kw) {
                    if constexpr (BITS == 4) cp_async16(st + 512u * n + 16u * lane, xp[n] + (size_t)r * EPS);
                    else cp_async8(st + 256u * n + 8u * lane, xp[n] + (size_t)r * EPS);
                }
        }
    };
    // words of the first ST quads before h exists; then their x, one group each
    for (int i = 0; i < ST; ++i) {
        issue_w(i);
        if constexpr (UP) issue_x(i);
        cp_commit();
    }
    if constexpr (!UP) {
        grid_dependency_wait();
        for (int i = 0; i < ST; ++i) {
            issue_x(i);
            cp_commit();
        }
    }

    float acc[2][4][NT][NE], d[2][2][NT][4], xs[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int k = 0; k < 4; ++k) xs[n][k] = 0.0f;
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int e = 0; e < NE; ++e) acc[hf][c][n][e] = 0.0f;
#pragma unroll
            for (int T = 0; T < 2; ++T)
#pragma unroll
                for (int k = 0; k < 4; ++k) d[hf][T][n][k] = 0.0f;
        }
    }
    const int nt = NT == 1 ? 1 : (b.m + TPT - 1) / TPT;   // tiles that hold slots
    uint2 sv[2], zv[2];
    int left = p.qpg - (nq > 0 ? q0 % p.qpg : 0);
    bool start = true;
    constexpr uint32_t ONE = MBF ? 0x3F803F80u : 0x3C003C00u;
    const uint32_t ones[4] = {ONE, ONE, ONE, ONE};
    for (int i = 0; i < nq; ++i) {
        cp_wait<ST - 1>();
        __syncwarp();  // the s and z that other lanes copied
        const uint32_t st = ring + (uint32_t)(i % ST) * SB;
        const uint4 wa = lds128_u32(st + 16u * lane), wb = lds128_u32(st + 512u + 16u * lane);
        if (start) {
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                sv[hf] = lds64_u32(st + W_BYTES + 128u * hf + 8u * g);
                zv[hf] = lds64_u32(st + W_BYTES + 128u * hf + 64u + 8u * g);
            }
            start = false;
        }
        uint32_t bx[NT][EPS / 2];
        const bool in = 4 * (q0 + i) + t < p.Kw;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const uint32_t a = st + W_BYTES + SZ_BYTES;
            if constexpr (BITS == 4) {
                uint4 v = make_uint4(0u, 0u, 0u, 0u);
                if (xon[n] && in) v = lds128_u32(a + 512u * n + 16u * lane);
                bx[n][0] = prmt(v.x, v.z, 0x5410u);   // pairs (0, 4), (1, 5), (2, 6), (3, 7)
                bx[n][1] = prmt(v.x, v.z, 0x7632u);
                bx[n][2] = prmt(v.y, v.w, 0x5410u);
                bx[n][3] = prmt(v.y, v.w, 0x7632u);
            } else {
                uint2 v = make_uint2(0u, 0u);
                if (xon[n] && in) v = lds64_u32(a + 256u * n + 8u * lane);
                bx[n][0] = prmt(v.x, v.y, 0x5410u);   // pairs (0, 2), (1, 3)
                bx[n][1] = prmt(v.x, v.y, 0x7632u);
            }
        }
        __syncwarp();  // every lane has read the stage: refill it
        issue_w(i + ST);
        issue_x(i + ST);
        cp_commit();
        const uint32_t wv[2][4] = {{wa.x, wa.y, wa.z, wa.w}, {wb.x, wb.y, wb.z, wb.w}};
#pragma unroll
        for (int k = 0; k < MMAS; ++k) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
                if (n < nt) mma_16816<MBF>(xs[n], ones, bx[n][2 * k], bx[n][2 * k + 1]);
#pragma unroll
            for (int hf = 0; hf < 2; ++hf)
#pragma unroll
                for (int T = 0; T < 2; ++T) {
                    const uint32_t a[4] = {
                        code_pair<BITS, MBF>(wv[hf][2 * T], 2 * k), code_pair<BITS, MBF>(wv[hf][2 * T + 1], 2 * k),
                        code_pair<BITS, MBF>(wv[hf][2 * T], 2 * k + 1),
                        code_pair<BITS, MBF>(wv[hf][2 * T + 1], 2 * k + 1)};
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        if (n < nt) mma_16816<MBF>(d[hf][T][n], a, bx[n][2 * k], bx[n][2 * k + 1]);
                }
        }
        if (--left == 0 || i + 1 == nq) {   // the group (or the warp's part of it) ends: fold
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const float2 s01 = T16::pair(sv[hf].x), s23 = T16::pair(sv[hf].y);
                const float2 z01 = T16::pair(zv[hf].x), z23 = T16::pair(zv[hf].y);
                const float sc[4] = {s01.x, s01.y, s23.x, s23.y};
                const float zc[4] = {z01.x + ZOFF, z01.y + ZOFF, z23.x + ZOFF, z23.y + ZOFF};
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < NE; ++e) {
                            const int k = 2 * (c & 1) + e;
                            float D = d[hf][c >> 1][n][k], X = xs[n][e];
                            if constexpr (!UP) {
                                D += d[hf][c >> 1][n][k + 1];
                                X += xs[n][1];
                            }
                            acc[hf][c][n][e] = fmaf(sc[c], fmaf(D, DSCALE, -zc[c] * X), acc[hf][c][n][e]);
                        }
#pragma unroll
                for (int T = 0; T < 2; ++T)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int k = 0; k < 4; ++k) d[hf][T][n][k] = 0.0f;
            }
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int k = 0; k < 4; ++k) xs[n][k] = 0.0f;
            left = p.qpg;
            start = true;
        }
    }

    // ---- the warps' partials meet in shared memory: [slot][64], in each warp's own ring
    cp_wait<0>();
    __syncwarp();
    {
        float* red = reinterpret_cast<float*>(smem + (size_t)warp * (ST * SB));
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < NE; ++e) {
                const int pos = n * TPT + (UP ? 2 * t + e : t);
                if (pos < b.m)
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf)
                        *reinterpret_cast<float4*>(red + pos * MCOLS + 32 * hf + 4 * g) =
                            make_float4(acc[hf][0][n][e], acc[hf][1][n][e], acc[hf][2][n][e], acc[hf][3][n][e]);
            }
    }
    __syncthreads();
    auto total = [&](int i) {   // over the warps, in their order
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < MW; ++w) v += reinterpret_cast<const float*>(smem + (size_t)w * (ST * SB))[i];
        return v;
    };
    if constexpr (UP) {
        for (int i = threadIdx.x; i < b.m * 32; i += MT) {
            const int pos = i >> 5, c = i & 31, cc = tile * 32 + c;
            if (cc >= p.I) continue;
            const float v = activate(total(pos * MCOLS + c), p.act) * total(pos * MCOLS + 32 + c);
            const __nv_bfloat16 hi = __float2bfloat16_rn(v);
            const __nv_bfloat16 lo = __float2bfloat16_rn(v - __bfloat162float(hi));
            uint16_t* dst = p.h + (size_t)slots[pos] * p.I + cc;
            dst[0] = __bfloat16_as_ushort(hi);
            dst[(size_t)p.S * p.I] = __bfloat16_as_ushort(lo);
        }
    } else {
        for (int i = threadIdx.x; i < b.m * MCOLS; i += MT) {
            const int pos = i / MCOLS, cc = tile * MCOLS + i % MCOLS;
            if (cc < p.NW) p.part[(size_t)slots[pos] * p.NW + cc] = total(i);
        }
        // the last of the tile's blocks to arrive sums the slots of each token
        __threadfence();
        __syncthreads();
        if (threadIdx.x == 0)
            last = b.nblocks == 0 || atomicAdd(&p.count[tile], 1u) == (unsigned)b.nblocks - 1u;
        __syncthreads();
        if (!last) return;
        __threadfence();
        for (int i = threadIdx.x; i < p.T * (MCOLS / 4); i += MT) {
            const int tok = i / (MCOLS / 4), cc = tile * MCOLS + 4 * (i % (MCOLS / 4));
            if (cc >= p.NW) continue;
            float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            for (int j = 0; j < p.top_k; ++j) {
                const int slot = tok * p.top_k + j, id = p.ids[slot];
                if (id < 0 || id >= p.E) continue;
                const float a = p.weights[slot];
                const float4 r = __ldcg(reinterpret_cast<const float4*>(p.part + (size_t)slot * p.NW + cc));
                v.x = fmaf(a, r.x, v.x);
                v.y = fmaf(a, r.y, v.y);
                v.z = fmaf(a, r.z, v.z);
                v.w = fmaf(a, r.w, v.w);
            }
            uint2 o;
            o.x = (uint32_t)T16::store(v.x) | ((uint32_t)T16::store(v.y) << 16);
            o.y = (uint32_t)T16::store(v.z) | ((uint32_t)T16::store(v.w) << 16);
            *reinterpret_cast<uint2*>(p.y + (size_t)tok * p.NW + cc) = o;
        }
    }
}

template <int BITS, bool BF, int NT, bool UP>
wq_status launch_one(const MoeParams& p, int tiles, bool pdl, cudaStream_t stream) {
    auto kern = moe_kernel<BITS, BF, NT, UP>;
    static std::atomic<uint64_t> attr_ctx[MAX_DEVICES];
    constexpr int smem = MW * stages<NT>() * stage_bytes<BITS, NT>();
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return WQ_ERR_CUDA;
    if (const wq_status st = ensure_smem_attr((const void*)kern, smem, attr_ctx, dev); st != WQ_OK) return st;
    constexpr int BT = (UP ? 8 : 4) * NT;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(tiles, std::min(p.S, std::min(p.E, p.S) + p.S / BT), 1);
    cfg.blockDim = dim3(MT, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return from_cuda(cudaLaunchKernelEx(&cfg, kern, p));
}

void set_product(MoeParams& p, int K, int G, int eps) {
    p.K = K;
    p.Kw = K / eps;
    p.Q = (p.Kw + 3) / 4;
    p.QW = (p.Q + MW - 1) / MW;
    p.qpg = G == K ? (1 << 29) : G / (4 * eps);
    p.groups = G == K ? 1 : K / G;
}

template <int BITS, bool BF>
wq_status run_moe(const MoeProblem& m, cudaStream_t stream) {
    constexpr int EPS = 32 / BITS;
    MoeParams p{};
    p.x = m.x; p.ids = m.ids; p.weights = m.weights; p.y = m.y;
    p.T = m.T; p.top_k = m.top_k; p.S = m.T * m.top_k; p.E = m.E; p.I = m.I; p.act = m.act;
    p.ntiles_down = (m.N + MCOLS - 1) / MCOLS;
    uint8_t* ws = static_cast<uint8_t*>(m.ws);
    const MoeLayout lay = moe_layout(m.T, m.top_k, m.I, m.N);
    p.count = reinterpret_cast<unsigned int*>(ws);
    p.h = reinterpret_cast<uint16_t*>(ws + lay.off_h);
    p.part = reinterpret_cast<float*>(ws + lay.off_part);

    p.w = m.w_up; p.s = m.s_up; p.z = m.z_up;
    p.NW = 2 * m.I; p.NC = m.I;
    set_product(p, m.K, m.group_size == -1 ? m.K : m.group_size, EPS);
    const bool pdl = (m.flags & WQ_FLAG_PDL) != 0;
    const int up_tiles = (m.I + 31) / 32;
    wq_status st = m.T <= 8 ? launch_one<BITS, BF, 1, true>(p, up_tiles, pdl, stream)
                            : launch_one<BITS, BF, 2, true>(p, up_tiles, pdl, stream);
    if (st != WQ_OK) return st;

    p.w = m.w_down; p.s = m.s_down; p.z = m.z_down;
    p.NW = p.NC = m.N;
    set_product(p, m.I, m.group_size == -1 ? m.I : m.group_size, EPS);
    if (m.T <= 4) return launch_one<BITS, BF, 1, false>(p, p.ntiles_down, true, stream);
    if (m.T <= 8) return launch_one<BITS, BF, 2, false>(p, p.ntiles_down, true, stream);
    return launch_one<BITS, BF, 4, false>(p, p.ntiles_down, true, stream);
}

}  // namespace

// Workspace: arrival counters, h (two bf16 planes), the fp32 rows per slot.
MoeLayout moe_layout(int T, int top_k, int I, int N) {
    const size_t S = (size_t)T * top_k;
    auto up = [](size_t v) { return (v + 255) & ~(size_t)255; };
    MoeLayout l;
    l.off_h = up((size_t)((N + MCOLS - 1) / MCOLS) * 4);
    l.off_part = l.off_h + up(S * I * 4);
    l.bytes = l.off_part + up(S * N * 4);
    return l;
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
    return (v & 2u) ? WQ_ERR_CHECK : WQ_OK;
}

}  // namespace wq
