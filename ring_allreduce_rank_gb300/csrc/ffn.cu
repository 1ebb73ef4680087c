// ffn.cu -- gated feed-forward block, forward and backward.
//
//   g = x Wg^T, u = x Wu^T, h = act(g) * u, y = h Wd^T
//   dh = dy Wd, du = dh * act(g), dg = dh * u * act'(g)
//   dx = dg Wg + du Wu, dWg = dg^T x, dWu = du^T x, dWd = dy^T h
//
// Every product is one kernel, ffn_gemm_kernel: a persistent grid of CTA pairs,
// each pair computing 256 x 256 fp32 accumulators in tensor memory with
// tcgen05.mma (cta_group::2, bf16 operands), operands brought by TMA into a
// ring of shared-memory stages, two accumulators in turn so that one tile's
// epilogue runs under the next tile's products.  The operands are used where
// they lie, whichever of their dimensions is contiguous (K-major or MN-major
// descriptors), so nothing is transposed.  The epilogues carry the activation
// and its derivative: the forward's first product makes g and u of the same
// 128 columns side by side in one accumulator (one CTA of the pair loads Wg's
// rows, the other Wu's), and the backward's first product turns dh into dg,
// du and h without dh reaching memory.  dx's two products are one longer sum,
// and the three weight gradients are one launch.
//
// h, dg and du are rounded to bf16: they are operands of the next products.
// g and u are kept in fp32 for the backward pass, since rounding them would
// add a rounding to every factor of every gradient.
//
// Bound by the tensor cores for many tokens, by reading the weights for few.
// At 4096 x 11008: forward of 4096 tokens 678-692 us (1.60-1.63 PFLOP/s; cuBLAS
// sustains 1.71 on plain products at this card's power limit), forward and
// backward of 2048 tokens 1077-1103 us (1.51-1.54 PFLOP/s), forward of one
// token 53 us (5.1 TB/s of weights, 0.75 of the copy bandwidth), of 48 60 us.
// Cutting the last, partly filled round of tiles along K to fill it made each
// product shorter alone and the whole longer: at the power limit a fuller GPU
// runs at a lower clock, and the partial sums' join is not free.
#include <algorithm>
#include <atomic>
#include <vector>

#include "../../include/ccl.h"
#include "ccl_internal.h"
#include "step_ops.cuh"
#include "tensor_core.cuh"

namespace ccl {
namespace {

constexpr int kTileM = 256, kTileN = 256, kTileK = 64; // a CTA pair's tile
constexpr int kOperandBytes = 128 * kTileK * 2;        // one CTA's part of A or B in a stage
constexpr int kStageBytes = 2 * kOperandBytes;
constexpr int kStages = 6;
constexpr int kMaxStages = 6; // ffn_few_kernel's
// Products that ffn_few_kernel takes: few tokens.  Forward in us, this kernel
// against CTA pairs' 256-row tiles: 488 x 2584 with 48 tokens 16.8 against 17.3,
// with 64 equal, with 128 22.0 against 19.7; 4096 x 11008 with 64 tokens 61
// against 73, with 128 69 against 79, with 198 84 against 82 (kManyWeights lies
// between the two widths, where nothing was measured).  Backward to the
// inputs, 1000 x 3000: with 64 tokens 19.5 against 31.4, with 128 24.4 against
// 34.4, with 198 54.5 against 34.5.
constexpr uint64_t kFewTokens = 64, kFewTokensMost = 128; // the latter for many weights, and backward
constexpr uint64_t kManyWeights = 1 << 24;
constexpr int kFewBytes = 200 * 1024; // its stages', at most
constexpr int kGemmThreads = 384; // producer, issuer, tensor memory, one idle warp, eight epilogue warps
constexpr int kEpiWarps = 8;
constexpr int kTurnFloats = 32 * 33; // an epilogue warp's 32 x 32 values, rows padded against bank conflicts
constexpr int kGemmSmem = kStages * kStageBytes + 1024 /* alignment */ + kEpiWarps * kTurnFloats * 4;
constexpr int kGroupM = 8; // row tiles walked before the next column tile
constexpr int kMaxProblems = 3;
std::atomic<unsigned long long> g_wait_ns{4000000000ull}; // the bounded waits' limit, for calls made from now on

enum Epilogue { EPI_GATED = 0, EPI_STORE = 1, EPI_BACKWARD = 2 };

// One product C[M, N] = sum over segments of A_s[M, K] B_s[N, K]^T.
struct Problem {
    CUtensorMap a[2], b[2];
    void *out;        // EPI_STORE: bf16, row stride N
    float *partial;   // split sums: [splits][M][column tiles * 256]
    uint32_t m, n;    // n: output columns (EPI_GATED: of h)
    uint32_t mt, nt;  // tiles
    uint32_t kblocks; // of one segment
    uint32_t segs;
    uint32_t units;   // mt * nt * splits
};

struct GemmParams {
    Problem prob[kMaxProblems];
    uint32_t nprob, splits;
    int act, accumulate;
    // EPI_GATED writes h and, if kept, g and u; EPI_BACKWARD reads those and writes h, dg and du
    uint16_t *h, *dg, *du;
    float *g, *u;
    uint32_t ldh; // row stride of h, dg and du (g and u: n)
    int vectors;  // every row that the epilogue touches is 16-byte aligned (fp32: 32) and whole vectors of 8 columns
    int early;    // the weights may be read before the kernel before this one has ended
    unsigned long long wait_ns; // how long a role waits for another; 0: no role begins
};

// ffn_few_kernel's: the same products with the weights as rows.
struct FewParams {
    GemmParams p;
    uint32_t npad;   // tokens, rounded up to 16
    uint32_t stages; // of 32 KiB of weights and npad * 128 bytes of activations
};

__device__ unsigned long long g_ffn_timeouts;

__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, volatile int *gave_up, unsigned long long limit)
{
    return ccl::mbar_wait(bar, parity, gave_up, limit, &g_ffn_timeouts);
}

template <bool MN> __device__ __forceinline__ void load_operand(uint32_t dst, const CUtensorMap *map, int mn, int k, uint32_t bar)
{
    if (MN) {
        tma_load(dst, map, mn, k, bar);
        tma_load(dst + kOperandBytes / 2, map, mn + 64, k, bar);
    } else {
        tma_load(dst, map, k, mn, bar);
    }
}

template <bool MN> __device__ __forceinline__ void load_weights(uint32_t dst, const CUtensorMap *map, int mn, int k, uint32_t bar)
{
    if (MN) {
        tma_load_own(dst, map, mn, k, bar);
        tma_load_own(dst + kOperandBytes / 2, map, mn + 64, k, bar);
    } else {
        tma_load_own(dst, map, k, mn, bar);
    }
}

// ------------------------------------------------------------------ epilogues

// What the epilogue reads of one column: the saved g and u, or the old value.
template <int EPI> struct Ahead1 {
    float g, u;
    __device__ __forceinline__ void load(const GemmParams &p, const Problem &q, uint64_t at, bool in)
    {
        if (EPI == EPI_BACKWARD && in) {
            g = gload<float>(p.g + at);
            u = gload<float>(p.u + at);
        }
        if (EPI == EPI_STORE && p.accumulate && in)
            g = ld_value<DT_BF16>(q.out, at);
    }
};

// One finished sum: v, and for EPI_GATED g = v and u = w; at: its place in
// rows of n columns, ath: in rows of ldh.
template <int EPI>
__device__ __forceinline__ void finish1(const GemmParams &p, const Problem &q, uint64_t at, uint64_t ath,
                                        const Ahead1<EPI> &ahead, float v, float w)
{
    float a, da;
    if (EPI == EPI_GATED) {
        if (p.g) {
            gstore<float>(p.g + at, v);
            gstore<float>(p.u + at, w);
        }
        activation(p.act, v, a, da);
        st_value<DT_BF16>(p.h, ath, a * w);
    } else if (EPI == EPI_BACKWARD) {
        activation(p.act, ahead.g, a, da);
        st_value<DT_BF16>(p.h, ath, a * ahead.u);
        st_value<DT_BF16>(p.dg, ath, v * ahead.u * da);
        st_value<DT_BF16>(p.du, ath, v * a);
    } else {
        st_value<DT_BF16>(q.out, at, p.accumulate ? __fadd_rn(ahead.g, v) : v);
    }
}

// The result of one column of one row whose products never came, as NaN: a
// kernel that gave up leaves nothing that could pass for a result.
template <int EPI> __device__ __forceinline__ void finish_nan(const GemmParams &p, const Problem &q, uint32_t row, uint32_t col)
{
    const float nan = __uint_as_float(0x7fffffffu);
    const uint64_t at = (uint64_t)row * q.n + col;
    Ahead1<EPI> old;
    old.load(p, q, at, true);
    finish1<EPI>(p, q, at, (uint64_t)row * p.ldh + col, old, nan, nan);
}

// What the epilogue reads of sixteen columns, asked for before it is needed.
template <int EPI> struct Ahead16 {
    Vals16 g, u;
    __device__ __forceinline__ void load(const GemmParams &p, const Problem &q, uint32_t row, uint32_t col)
    {
        if (row >= q.m || col >= q.n)
            return;
        const uint64_t at = (uint64_t)row * q.n + col;
        if (EPI == EPI_BACKWARD) {
            g.load(p.g + at, col + 8 < q.n);
            u.load(p.u + at, col + 8 < q.n);
        }
        if (EPI == EPI_STORE && p.accumulate)
            g.load(static_cast<const uint16_t *>(q.out) + at, col + 8 < q.n);
    }
};

// Sixteen finished sums of one row (p.vectors).
template <int EPI>
__device__ __forceinline__ void finish16(const GemmParams &p, const Problem &q, uint32_t row, uint32_t col,
                                         const Ahead16<EPI> &ahead, float *v, float *w)
{
    if (row >= q.m || col >= q.n)
        return;
    const bool both = col + 8 < q.n;
    const uint64_t at = (uint64_t)row * q.n + col, ath = (uint64_t)row * p.ldh + col;
    float a[16], da;
    if (EPI == EPI_GATED) {
        if (p.g) {
            store16(p.g + at, v, both);
            store16(p.u + at, w, both);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            activation(p.act, v[i], a[i], da);
            a[i] *= w[i];
        }
        store16(p.h + ath, a, both);
    } else if (EPI == EPI_BACKWARD) {
        float g[16], u[16];
        ahead.g.get(g);
        ahead.u.get(u);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            activation(p.act, g[i], a[i], da);
            g[i] = v[i] * u[i] * da; // dg
            v[i] = v[i] * a[i];      // du
            a[i] = a[i] * u[i];      // h
        }
        store16(p.h + ath, a, both);
        store16(p.dg + ath, g, both);
        store16(p.du + ath, v, both);
    } else {
        if (p.accumulate) {
            unpack<DT_BF16>(ahead.g.v[0], a);
            unpack<DT_BF16>(ahead.g.v[1], a + 8);
#pragma unroll
            for (int i = 0; i < 16; ++i)
                v[i] = __fadd_rn(a[i], v[i]);
        }
        store16(static_cast<uint16_t *>(q.out) + at, v, both);
    }
}

// ------------------------------------------------------------------ the product

struct Unit {
    uint32_t prob, split, m, n, kb0, kb1;
};

__device__ __forceinline__ Unit unit_at(const GemmParams &p, uint32_t i)
{
    Unit u;
    u.prob = 0;
    while (i >= p.prob[u.prob].units)
        i -= p.prob[u.prob++].units;
    const Problem &q = p.prob[u.prob];
    const uint32_t tiles = q.mt * q.nt;
    u.split = i / tiles;
    const uint32_t t = i % tiles, per = kGroupM * q.nt, grp = t / per, in = t % per;
    const uint32_t gm = min(q.mt - grp * kGroupM, (uint32_t)kGroupM);
    u.m = grp * kGroupM + in % gm;
    u.n = in / gm;
    const uint32_t kb = q.kblocks * q.segs;
    u.kb0 = (uint32_t)((uint64_t)kb * u.split / p.splits);
    u.kb1 = (uint32_t)((uint64_t)kb * (u.split + 1) / p.splits);
    return u;
}

template <int EPI, bool A_MN, bool B_MN>
__global__ void __launch_bounds__(kGemmThreads, 1) ffn_gemm_kernel(const __grid_constant__ GemmParams p)
{
    extern __shared__ uint8_t raw[];
    __shared__ uint64_t bars[2 * kStages + 4];
    __shared__ uint32_t tmem_slot;
    __shared__ volatile int gave_up;
    const uint32_t stages = (smem_u32(raw) + 1023) & ~1023u;
    const uint32_t full = smem_u32(&bars[0]), empty = smem_u32(&bars[kStages]);
    const uint32_t acc_full = smem_u32(&bars[2 * kStages]), acc_empty = smem_u32(&bars[2 * kStages + 2]);
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const uint32_t pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(acc_full + 8 * i, 1);
            mbar_init(acc_empty + 8 * i, 2 * kEpiWarps);
        }
        if ((gave_up = p.wait_ns == 0))
            atomicAdd(&g_ffn_timeouts, 1ull);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 3 && lane / 4 < p.nprob) {
        const Problem &q = p.prob[lane / 4];
        const int i = lane & 1;
        if (lane & 2 ? i < (EPI == EPI_GATED ? 2 : q.segs) : i < q.segs)
            prefetch_map(lane & 2 ? &q.b[i] : &q.a[i]);
    }
    if (warp == 2) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&tmem_slot)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    cluster_sync();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t tmem = tmem_slot;
    chain_entry();

    uint32_t total = 0;
    for (uint32_t i = 0; i < p.nprob; ++i)
        total += p.prob[i].units;

    if (warp == 0 && lane == 0) {
        // producer: this CTA's halves of A and B, stage by stage
        const uint32_t leader_full = in_cta(full, 0);
        uint32_t s = 0, phase = 0;
        bool ok = p.wait_ns != 0;
        for (uint32_t i = pair; ok && i < total; i += pairs) {
            const Unit u = unit_at(p, i);
            const Problem &q = p.prob[u.prob];
            const int am = (int)(u.m * kTileM + rank * 128);
            const int bn = EPI == EPI_GATED ? (int)(u.n * 128) : (int)(u.n * kTileN + rank * 128);
            for (uint32_t kb = u.kb0; kb < u.kb1; ++kb) {
                if (!(ok = mbar_wait(empty + 8 * s, phase ^ 1, &gave_up, p.wait_ns)))
                    break;
                if (rank == 0)
                    mbar_expect(full + 8 * s, 2 * kStageBytes);
                const uint32_t seg = kb >= q.kblocks ? 1 : 0;
                const int k = (int)((kb - seg * q.kblocks) * kTileK);
                const uint32_t at = stages + s * kStageBytes;
                const CUtensorMap *b = EPI == EPI_GATED ? &q.b[rank] : &q.b[seg];
                load_operand<A_MN>(at, &q.a[seg], am, k, leader_full + 8 * s);
                load_operand<B_MN>(at + kOperandBytes, b, bn, k, leader_full + 8 * s);
                if (++s == kStages) {
                    s = 0;
                    phase ^= 1;
                }
            }
        }
        // the issuer's last arrivals reach both CTAs while they are here
        for (int i = 0; ok && i < kStages; ++i) {
            ok = mbar_wait(empty + 8 * s, phase ^ 1, &gave_up, p.wait_ns);
            if (++s == kStages) {
                s = 0;
                phase ^= 1;
            }
        }
    } else if (warp == 1 && lane == 0 && rank == 0) {
        // issuer: fp32 accumulator, bf16 operands, their majorness, N, M
        const uint32_t idesc = 1u << 4 | 1u << 7 | 1u << 10 | (A_MN ? 1u << 15 : 0) | (B_MN ? 1u << 16 : 0) |
                               (kTileN >> 3) << 17 | (kTileM >> 4) << 24;
        uint32_t s = 0, phase = 0, t = 0;
        bool ok = p.wait_ns != 0;
        for (uint32_t i = pair; ok && i < total; i += pairs, ++t) {
            const Unit u = unit_at(p, i);
            const uint32_t buf = t & 1;
            if (!(ok = mbar_wait(acc_empty + 8 * buf, ((t >> 1) & 1) ^ 1, &gave_up, p.wait_ns)))
                break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            for (uint32_t kb = u.kb0; kb < u.kb1; ++kb) {
                if (!(ok = mbar_wait(full + 8 * s, phase, &gave_up, p.wait_ns)))
                    break;
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                const uint32_t at = stages + s * kStageBytes;
#pragma unroll
                for (int k = 0; k < kTileK / 16; ++k)
                    tc_mma(tmem + buf * kTileN, operand_desc<A_MN>(at + k * k_step<A_MN>()),
                           operand_desc<B_MN>(at + kOperandBytes + k * k_step<B_MN>()), idesc, kb > u.kb0 || k > 0);
                tc_commit(empty + 8 * s);
                if (++s == kStages) {
                    s = 0;
                    phase ^= 1;
                }
            }
            if (ok)
                tc_commit(acc_full + 8 * buf);
        }
    } else if (warp >= 4) {
        // epilogue: warp w reads lanes 32 (w % 4) .. + 32 and half of the
        // columns.  Vectors: a lane keeps its row, sixteen columns at a time,
        // what it reads asked for one step ahead.  Otherwise the values are
        // turned in shared memory, so that a warp's accesses run along a row.
        const uint32_t half = (warp - 4) / 4;
        const uint32_t lanes = (uint32_t)(warp & 3) * 32;
        const uint32_t leader_empty = in_cta(acc_empty, 0);
        float *turn = reinterpret_cast<float *>(raw + (stages - smem_u32(raw)) + kStages * kStageBytes) + (warp - 4) * kTurnFloats;
        constexpr uint32_t kCols = EPI == EPI_GATED ? 64 : 128;
        uint32_t t = 0, i = pair;
        for (; p.wait_ns && i < total; i += pairs, ++t) {
            const Unit u = unit_at(p, i);
            const Problem &q = p.prob[u.prob];
            const uint32_t buf = t & 1;
            const uint32_t row0 = u.m * kTileM + rank * 128 + lanes, row = row0 + lane;
            const uint32_t c0 = half * kCols, col0 = u.n * (2 * kCols) + c0;
            Ahead16<EPI> ahead;
            if (p.vectors && p.splits == 1)
                ahead.load(p, q, row, col0);
            if (!__all_sync(0xffffffffu, mbar_wait(acc_full + 8 * buf, (t >> 1) & 1, &gave_up, p.wait_ns)))
                break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            const uint32_t acc = tmem + buf * kTileN + (lanes << 16);
            if (p.splits > 1) {
                const uint64_t width = (uint64_t)q.nt * kTileN;
                float *out = q.partial + ((uint64_t)u.split * q.m + row) * width + u.n * kTileN;
                for (uint32_t c = half * 128; c < half * 128 + 128; c += 16) {
                    float v[16];
                    tc_load16(acc + c, v);
                    if (row < q.m)
                        store16(out + c, v, true);
                }
            } else if (p.vectors) {
#pragma unroll 2
                for (uint32_t c = 0; c < kCols; c += 16) {
                    float v[16], w[16];
                    tc_load16(acc + c0 + c, v);
                    if (EPI == EPI_GATED)
                        tc_load16(acc + 128 + c0 + c, w);
                    Ahead16<EPI> next;
                    if (c + 16 < kCols)
                        next.load(p, q, row, col0 + c + 16);
                    finish16<EPI>(p, q, row, col0 + c, ahead, v, w);
                    ahead = next;
                }
            } else {
                // rows of 32 columns, or of 16 columns of g and the same of u
                constexpr uint32_t kWide = EPI == EPI_GATED ? 16 : 32, kRows = 32 / kWide;
                for (uint32_t c = 0; c < kCols; c += kWide) {
                    float v[32];
                    if (EPI == EPI_GATED) {
                        tc_load16(acc + c0 + c, v);
                        tc_load16(acc + 128 + c0 + c, v + 16);
                    } else {
                        tc_load32(acc + c0 + c, v);
                    }
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        turn[lane * 33 + j] = v[j];
                    __syncwarp();
                    const uint32_t cc = lane % kWide, col = col0 + c + cc;
                    for (uint32_t r0 = lane / kWide; r0 < 32; r0 += 8 * kRows) { // eight rows' reads in flight
                        Ahead1<EPI> old[8];
                        const uint64_t at = (uint64_t)(row0 + r0) * q.n + col, ath = (uint64_t)(row0 + r0) * p.ldh + col;
                        const uint32_t step = kRows * q.n, steph = kRows * p.ldh;
                        const uint32_t rows = col >= q.n || row0 + r0 >= q.m ? 0 : (q.m - row0 - r0 + kRows - 1) / kRows;
#pragma unroll
                        for (uint32_t r = 0; r < 8; ++r)
                            old[r].load(p, q, at + (uint64_t)r * step, r < rows);
#pragma unroll
                        for (uint32_t r = 0; r < 8; ++r) {
                            const float *from = turn + (r0 + r * kRows) * 33 + cc;
                            if (r < rows)
                                finish1<EPI>(p, q, at + (uint64_t)r * step, ath + (uint64_t)r * steph, old[r], from[0],
                                             EPI == EPI_GATED ? from[16] : 0.0f);
                        }
                    }
                    __syncwarp();
                }
            }
            asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
            __syncwarp();
            if (lane == 0)
                mbar_arrive_cluster(leader_empty + 8 * buf);
        }
        for (; i < total; i += pairs) { // after a wait that gave up
            const Unit u = unit_at(p, i);
            const Problem &q = p.prob[u.prob];
            const uint32_t row0 = u.m * kTileM + rank * 128 + lanes, col0 = u.n * (2 * kCols) + half * kCols;
            for (uint32_t row = row0; row < min(row0 + 32, q.m); ++row)
                if (p.splits > 1) {
                    float *out = q.partial + ((uint64_t)u.split * q.m + row) * q.nt * kTileN + u.n * kTileN + half * 128;
                    for (uint32_t c = lane; c < 128; c += 32)
                        gstore<float>(out + c, __uint_as_float(0x7fffffffu));
                } else {
                    for (uint32_t col = col0 + lane; col < min(col0 + kCols, q.n); col += 32)
                        finish_nan<EPI>(p, q, row, col);
                }
        }
    }
    __syncwarp();
    if (gave_up) // copies still in flight land before the CTA's memory is given back
        for (int i = 0; i < 1000; ++i)
            __nanosleep(1000);
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    cluster_sync();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    if (warp == 2)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

// ------------------------------------------------------------------ few tokens

// The same products for at most 128 tokens, with the weights as the
// accumulator's rows and the tokens as its columns, so that the tensor cores
// work on the tokens there are and not on a 256-row tile of them: one CTA a
// unit of two 128-row blocks of weights (EPI_GATED: the same rows of Wg and
// Wu), which share the tokens' stage.  Bound by reading the weights: one
// token's g and u at 4096 x 11008 take 34 us (5.3 TB/s); on the 256-row tile
// they took 52, half of a tensor core's time spent on absent tokens.  Its 86
// units are cut in 7 along K, 602 on 152 CTAs; other cuts, into 2 to 14, made
// the call 52-61 us.  With 48 tokens they stay whole, on 86 CTAs: cutting them
// cost 4-7 us, because the partial sums weigh.
template <int EPI, bool A_MN> __global__ void __launch_bounds__(kGemmThreads, 1) ffn_few_kernel(const __grid_constant__ FewParams fp)
{
    extern __shared__ uint8_t raw[];
    __shared__ uint64_t bars[2 * kMaxStages + 4];
    __shared__ uint32_t tmem_slot;
    __shared__ volatile int gave_up;
    const GemmParams &p = fp.p;
    const Problem &q = p.prob[0];
    const uint32_t stages = (smem_u32(raw) + 1023) & ~1023u;
    const uint32_t stage_bytes = 2 * kOperandBytes + fp.npad * 128;
    const uint32_t full = smem_u32(&bars[0]), empty = smem_u32(&bars[kMaxStages]);
    const uint32_t acc_full = smem_u32(&bars[2 * kMaxStages]), acc_empty = smem_u32(&bars[2 * kMaxStages + 2]);
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kMaxStages; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(acc_full + 8 * i, 1);
            mbar_init(acc_empty + 8 * i, kEpiWarps);
        }
        if ((gave_up = p.wait_ns == 0))
            atomicAdd(&g_ffn_timeouts, 1ull);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 3 && lane < (EPI == EPI_GATED ? 2 : q.segs))
        prefetch_map(&q.a[lane]);
    else if (warp == 3 && lane >= 16 && lane - 16 < q.segs)
        prefetch_map(&q.b[lane - 16]);
    if (warp == 2) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&tmem_slot)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t tmem = tmem_slot;
    if (!p.early)
        chain_entry();

    if (warp == 0 && lane == 0) {
        uint32_t s = 0, phase = 0;
        bool ok = p.wait_ns != 0;
        // a: the weights (EPI_GATED: Wg and Wu; else one per segment); b: the tokens
        auto load_a = [&](const Unit &u, uint32_t kb, uint32_t stage) {
            mbar_expect(full + 8 * stage, stage_bytes);
            const uint32_t seg = kb >= q.kblocks ? 1 : 0, at = stages + stage * stage_bytes;
            const int k = (int)((kb - seg * q.kblocks) * kTileK);
            const int r0 = EPI == EPI_GATED ? (int)(u.n * 128) : (int)(u.n * 256);
            load_weights<A_MN>(at, EPI == EPI_GATED ? &q.a[0] : &q.a[seg], r0, k, full + 8 * stage);
            load_weights<A_MN>(at + kOperandBytes, EPI == EPI_GATED ? &q.a[1] : &q.a[seg], EPI == EPI_GATED ? r0 : r0 + 128, k, full + 8 * stage);
        };
        auto load_b = [&](uint32_t kb, uint32_t stage) {
            const uint32_t seg = kb >= q.kblocks ? 1 : 0;
            tma_load_own(stages + stage * stage_bytes + 2 * kOperandBytes, &q.b[seg], (int)((kb - seg * q.kblocks) * kTileK), 0, full + 8 * stage);
        };
        // the first stages' weights before the tokens' values are ready
        uint32_t ahead = 0;
        if (p.early) {
            const Unit u = unit_at(p, blockIdx.x);
            ahead = ok ? min(fp.stages, u.kb1 - u.kb0) : 0;
            for (uint32_t i = 0; i < ahead; ++i)
                load_a(u, u.kb0 + i, i);
            chain_entry();
        }
        auto next = [&] {
            if (++s == fp.stages) {
                s = 0;
                phase ^= 1;
            }
        };
        for (uint32_t i = blockIdx.x; ok && i < q.units; i += gridDim.x) {
            const Unit u = unit_at(p, i);
            for (uint32_t kb = u.kb0; kb < u.kb1; ++kb) {
                if (ahead) {
                    --ahead; // the ring's first round: this stage is free and its weights are on the way
                } else {
                    if (!(ok = mbar_wait(empty + 8 * s, phase ^ 1, &gave_up, p.wait_ns)))
                        break;
                    load_a(u, kb, s);
                }
                load_b(kb, s);
                next();
            }
        }
        // the issuer's last arrivals come while the CTA is here
        for (uint32_t i = 0; ok && i < fp.stages; ++i) {
            ok = mbar_wait(empty + 8 * s, phase ^ 1, &gave_up, p.wait_ns);
            next();
        }
    } else if (warp == 1 && lane == 0) {
        const uint32_t idesc = 1u << 4 | 1u << 7 | 1u << 10 | (A_MN ? 1u << 15 : 0) | (fp.npad >> 3) << 17 | (128u >> 4) << 24;
        uint32_t s = 0, phase = 0, t = 0;
        bool ok = p.wait_ns != 0;
        for (uint32_t i = blockIdx.x; ok && i < q.units; i += gridDim.x, ++t) {
            const Unit u = unit_at(p, i);
            const uint32_t buf = t & 1;
            if (!(ok = mbar_wait(acc_empty + 8 * buf, ((t >> 1) & 1) ^ 1, &gave_up, p.wait_ns)))
                break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            for (uint32_t kb = u.kb0; kb < u.kb1; ++kb) {
                if (!(ok = mbar_wait(full + 8 * s, phase, &gave_up, p.wait_ns)))
                    break;
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                const uint32_t at = stages + s * stage_bytes;
#pragma unroll
                for (int k = 0; k < kTileK / 16; ++k)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        tc_mma_own(tmem + (buf * 2 + j) * fp.npad, operand_desc<A_MN>(at + j * kOperandBytes + k * k_step<A_MN>()),
                                   operand_desc<false>(at + 2 * kOperandBytes + k * k_step<false>()), idesc, kb > u.kb0 || k > 0);
                tc_commit_own(empty + 8 * s);
                if (++s == fp.stages) {
                    s = 0;
                    phase ^= 1;
                }
            }
            if (ok)
                tc_commit_own(acc_full + 8 * buf);
        }
    } else if (warp >= 4) {
        if (p.early)
            chain_entry();
        // a lane is a weight row, so that a warp's accesses run along a token's
        // row.  EPI_GATED: the two halves of the warps take the tokens in turn,
        // else one block of rows each.
        const uint32_t half = (warp - 4) / 4, lanes = (uint32_t)(warp & 3) * 32;
        uint32_t t = 0, i = blockIdx.x;
        for (; p.wait_ns && i < q.units; i += gridDim.x, ++t) {
            const Unit u = unit_at(p, i);
            const uint32_t buf = t & 1;
            if (!__all_sync(0xffffffffu, mbar_wait(acc_full + 8 * buf, (t >> 1) & 1, &gave_up, p.wait_ns)))
                break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            const uint32_t acc = tmem + buf * 2 * fp.npad + (lanes << 16);
            const uint32_t col = EPI == EPI_GATED ? u.n * 128 + lanes + lane : u.n * 256 + half * 128 + lanes + lane;
            const uint64_t width = (uint64_t)q.nt * kTileN;
            for (uint32_t c = EPI == EPI_GATED ? half * 16 : 0; c < fp.npad; c += EPI == EPI_GATED ? 32 : 16) {
                float v[16], w[16];
                tc_load16(acc + (EPI == EPI_GATED ? 0 : half * fp.npad) + c, v);
                if (EPI == EPI_GATED)
                    tc_load16(acc + fp.npad + c, w);
                const uint32_t rows = min(16u, q.m - min(q.m, c)); // tokens of these columns
                if (p.splits > 1) {
                    float *out = q.partial + ((uint64_t)u.split * q.m + c) * width + u.n * kTileN + (EPI == EPI_GATED ? 0 : half * 128) + lanes + lane;
#pragma unroll
                    for (uint32_t j = 0; j < 16; ++j, out += width)
                        if (j < rows) {
                            gstore<float>(out, v[j]);
                            if (EPI == EPI_GATED)
                                gstore<float>(out + 128, w[j]);
                        }
                } else if (col < q.n) {
                    uint64_t at = (uint64_t)c * q.n + col, ath = (uint64_t)c * p.ldh + col;
                    Ahead1<EPI> old[16];
#pragma unroll
                    for (uint32_t j = 0; j < 16; ++j)
                        old[j].load(p, q, at + (uint64_t)j * q.n, j < rows);
#pragma unroll
                    for (uint32_t j = 0; j < 16; ++j, at += q.n, ath += p.ldh)
                        if (j < rows)
                            finish1<EPI>(p, q, at, ath, old[j], v[j], EPI == EPI_GATED ? w[j] : 0.0f);
                }
            }
            asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
            __syncwarp();
            if (lane == 0)
                mbar_arrive(acc_empty + 8 * buf);
        }
        for (; i < q.units; i += gridDim.x) { // after a wait that gave up
            const Unit u = unit_at(p, i);
            const uint32_t c0 = (EPI == EPI_GATED ? 0 : half * 128) + lanes + lane, col = u.n * (EPI == EPI_GATED ? 128 : 256) + c0;
            for (uint32_t row = 0; row < q.m; ++row) {
                if (EPI == EPI_GATED && (row / 16 & 1) != half)
                    continue; // the other half's token
                if (p.splits > 1) {
                    float *out = q.partial + ((uint64_t)u.split * q.m + row) * q.nt * kTileN + u.n * kTileN + c0;
                    gstore<float>(out, __uint_as_float(0x7fffffffu));
                    if (EPI == EPI_GATED)
                        gstore<float>(out + 128, __uint_as_float(0x7fffffffu));
                } else if (col < q.n) {
                    finish_nan<EPI>(p, q, row, col);
                }
            }
        }
    }
    __syncwarp();
    if (gave_up) // copies still in flight land before the CTA's memory is given back
        for (int i = 0; i < 1000; ++i)
            __nanosleep(1000);
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    if (warp == 2)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

// ------------------------------------------------------------------ split sums

// The splits' sums of one product, added in order, a column a thread.
template <int EPI> __global__ void __launch_bounds__(256) ffn_join_kernel(const __grid_constant__ GemmParams p)
{
    chain_entry();
    for (uint32_t i = 0; i < p.nprob; ++i) {
        const Problem &q = p.prob[i];
        const uint64_t width = (uint64_t)q.nt * kTileN, slab = (uint64_t)q.m * width;
        const uint32_t blocks = (q.n + 255) / 256; // of 256 columns
        for (uint64_t e = blockIdx.x; e < (uint64_t)q.m * blocks; e += gridDim.x) {
            const uint32_t row = (uint32_t)(e / blocks), col = (uint32_t)(e % blocks) * 256 + threadIdx.x;
            if (col >= q.n)
                continue;
            // EPI_GATED: 128 columns of g, then the same of u, in each tile
            const float *at = q.partial + row * width + (EPI == EPI_GATED ? col / 128 * 256 + col % 128 : col);
            float v = 0.0f, w = 0.0f, f[4], h[4];
            Ahead1<EPI> old;
            const uint64_t place = (uint64_t)row * q.n + col;
            old.load(p, q, place, true);
            for (uint32_t s0 = 0; s0 < p.splits; s0 += 4) { // four loads in flight
#pragma unroll
                for (int s = 0; s < 4; ++s)
                    if (s0 + s < p.splits) {
                        f[s] = gload<float>(at + (s0 + s) * slab);
                        if (EPI == EPI_GATED)
                            h[s] = gload<float>(at + (s0 + s) * slab + 128);
                    }
#pragma unroll
                for (int s = 0; s < 4; ++s)
                    if (s0 + s < p.splits) {
                        v = __fadd_rn(v, f[s]);
                        if (EPI == EPI_GATED)
                            w = __fadd_rn(w, h[s]);
                    }
            }
            finish1<EPI>(p, q, place, (uint64_t)row * p.ldh + col, old, v, w);
        }
    }
}

// ------------------------------------------------------------------ host side

// A map whose boxes are 64 columns wide: as K-major operand tiles (128 rows of
// 64 k values) or as MN-major ones (64 k rows of 64 values).  What lies
// outside the matrix reads as zero.
bool encode(CUtensorMap *map, const Matrix &m, bool mn, uint32_t box_rows = 128)
{
    const cuuint64_t dim[2] = {m.cols, m.rows}, stride[1] = {m.ld * 2};
    const cuuint32_t box[2] = {64, mn ? 64u : box_rows}, step[2] = {1, 1};
    return encode_fn() &&
           encode_fn()(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(m.ptr), dim, stride, box, step,
                       CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

uint32_t tiles_of(uint64_t n, uint32_t t) { return (uint32_t)((n + t - 1) / t); }

constexpr uint32_t kMaxSplits = 16;

// How many parts the sum over K is cut into: the number that minimises the
// rounds of CTA pairs (CTAs, for few tokens), each as long as the longer of a
// part's products and a unit's epilogue, which overlap, plus the join.  A block
// of K takes a pair about 0.35 us; a CTA with few tokens reads its 32 KiB of
// weights in 0.5 us alone, and at the memory's rate with the others.  An
// epilogue takes a pair about 3 us, or 15 us on rows that no 16-byte vector
// divides, and a CTA with few tokens 0.5 us; a join about 3 us and its bytes
// at 6 TB/s.  Without it a product of few tiles (few tokens, narrow layers)
// would leave most SMs idle.
uint32_t choose_splits(uint64_t tiles, uint64_t kblocks, uint64_t partial_bytes, bool few, bool odd)
{
    uint32_t best = 1;
    double cost = 0;
    const uint64_t slots = few ? kSms : kPairs;
    for (uint32_t s = 1; s <= kMaxSplits && s <= kblocks; ++s) {
        const double rounds = (double)((tiles * s + slots - 1) / slots);
        const double block = few ? std::max(0.5, 0.005 * (double)std::min(slots, tiles * s)) : 0.35;
        const double products = (double)kblocks / s * block, epilogue = few ? 0.5 : odd && s == 1 ? 15.0 : 3.0;
        const double c = rounds * std::max(products, epilogue) + std::min(products, epilogue) +
                         (s > 1 ? 3.0 + 2.0 * s * (double)partial_bytes / 6e6 : 0.0);
        if (s == 1 || c < cost * 0.97) {
            best = s;
            cost = c;
        }
    }
    return best;
}

// The products of a pass: problem sizes, splits and partial sums.
struct Shape {
    uint64_t m, n, k;
    uint32_t segs;
};
struct Launch {
    Shape s[kMaxProblems];
    int n;
    bool gated, few, odd; // few: by ffn_few_kernel; odd: the epilogue's rows are no 16-byte vectors
    uint32_t splits;
    size_t partial; // bytes of all splits
    void plan()
    {
        uint64_t tiles = 0, kb = 0;
        size_t bytes = 0;
        for (int i = 0; i < n; ++i) {
            tiles += (few ? 1 : (uint64_t)tiles_of(s[i].m, kTileM)) * tiles_of(s[i].n, gated ? 128 : kTileN);
            kb = std::max<uint64_t>(kb, (uint64_t)tiles_of(s[i].k, kTileK) * s[i].segs);
            bytes += up(s[i].m * (size_t)tiles_of(s[i].n, gated ? 128 : kTileN) * kTileN * 4);
        }
        splits = choose_splits(tiles, kb, bytes, few, odd);
        partial = splits > 1 ? bytes * splits : 0;
    }
};

struct FfnPlan {
    uint64_t t, d, f, dp, fp; // tokens, model width, inner width, padded widths
    Launch up_, down, dh, dx, dw;
    // offsets into the work buffer
    size_t h, dg, du, x, wg, wu, wd, dy, partial, bytes;
};

constexpr uint64_t kMaxTokens = 0x7fffff00, kMaxWidth = 1 << 24;

bool make_plan(size_t t, size_t d, size_t f, bool backward, bool aligned, FfnPlan *p)
{
    if (t > kMaxTokens || d > kMaxWidth || f > kMaxWidth || t * std::max(d, f) > (1ull << 44) || (uint64_t)d * f > (1ull << 44))
        return false;
    *p = FfnPlan{};
    p->t = t;
    p->d = d;
    p->f = f;
    p->dp = (d + 7) / 8 * 8;
    p->fp = (f + 15) / 16 * 16; // h, dg and du in rows of whole 32-byte vectors
    const bool pd = p->dp != d || !aligned, pf = f % 8 || !aligned, few = t <= kFewTokens || (t <= kFewTokensMost && (uint64_t)d * f >= kManyWeights),
               few_b = t <= kFewTokensMost,
               od = d % 8 != 0, of = f % 8 != 0;
    p->up_ = Launch{{{t, f, d, 1}}, 1, true, few, of, 1, 0};
    p->down = Launch{{{t, d, f, 1}}, 1, false, few, od, 1, 0};
    p->dh = Launch{{{t, f, d, 1}}, 1, false, few_b, of, 1, 0};
    p->dx = Launch{{{t, d, f, 2}}, 1, false, few_b, od, 1, 0};
    p->dw = Launch{{{f, d, t, 1}, {f, d, t, 1}, {d, f, t, 1}}, 3, false, false, od || of, 1, 0};
    size_t at = 0, partial = 0;
    auto take = [&](size_t n) {
        const size_t o = at;
        at += up(n);
        return o;
    };
    p->h = take(t * p->fp * 2);
    if (backward) {
        p->dg = take(t * p->fp * 2);
        p->du = take(t * p->fp * 2);
    }
    if (pd) {
        p->x = take(t * p->dp * 2);
        p->wg = take(f * p->dp * 2);
        p->wu = take(f * p->dp * 2);
        if (backward)
            p->dy = take(t * p->dp * 2);
    }
    if (pf)
        p->wd = take(d * p->fp * 2);
    for (Launch *l : {&p->up_, &p->down, &p->dh, &p->dx, &p->dw}) {
        l->plan();
        if (backward || l == &p->up_ || l == &p->down) // a backward pass's buffer serves the forward too
            partial = std::max(partial, l->partial);
    }
    p->partial = take(partial);
    p->bytes = at;
    return true;
}

// Fills in what the launch's problems share; the maps are the caller's.
cudaError_t set_problems(GemmParams &p, const Launch &l, char *partial, uint64_t *units)
{
    *units = 0;
    p.nprob = (uint32_t)l.n;
    p.splits = l.splits;
    for (int i = 0; i < l.n; ++i) {
        Problem &q = p.prob[i];
        const Shape &s = l.s[i];
        q.m = (uint32_t)s.m;
        q.n = (uint32_t)s.n;
        q.mt = l.few ? 1 : tiles_of(s.m, kTileM);
        q.nt = tiles_of(s.n, l.gated ? 128 : kTileN);
        q.kblocks = tiles_of(s.k, kTileK);
        q.segs = s.segs;
        if ((uint64_t)q.mt * q.nt * l.splits > 0x3fffffff)
            return cudaErrorInvalidValue;
        q.units = q.mt * q.nt * l.splits;
        q.partial = reinterpret_cast<float *>(partial);
        partial += up(s.m * (size_t)q.nt * kTileN * 4) * l.splits;
        *units += q.units;
    }
    return cudaSuccess;
}

template <int EPI> cudaError_t launch_join(const GemmParams &p, cudaStream_t stream)
{
    if (p.splits == 1)
        return cudaSuccess;
    uint64_t blocks = 0;
    for (uint32_t i = 0; i < p.nprob; ++i)
        blocks = std::max<uint64_t>(blocks, (uint64_t)p.prob[i].m * ((p.prob[i].n + 255) / 256));
    const cudaError_t e = launch_chained(ffn_join_kernel<EPI>, dim3((unsigned)std::min<uint64_t>(blocks, 8 * kSms)), dim3(256), 0, stream, p);
    if (e == cudaSuccess)
        count_launches(1);
    return e;
}

// A product (A rows: tokens, or for weight gradients units) on CTA pairs.
template <int EPI, bool A_MN, bool B_MN> cudaError_t launch_gemm(GemmParams &p, const Launch &l, char *partial, cudaStream_t stream)
{
    uint64_t units;
    cudaError_t e = set_problems(p, l, partial, &units);
    static std::atomic<unsigned long long> ready{0};
    if (e != cudaSuccess ||
        (e = large_smem_once(reinterpret_cast<const void *>(ffn_gemm_kernel<EPI, A_MN, B_MN>), kGemmSmem, ready)) != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * (unsigned)std::min<uint64_t>(units, kPairs));
    cfg.blockDim = dim3(kGemmThreads);
    cfg.dynamicSmemBytes = kGemmSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if ((e = cudaLaunchKernelEx(&cfg, ffn_gemm_kernel<EPI, A_MN, B_MN>, p)) != cudaSuccess)
        return e;
    count_launches(1);
    return launch_join<EPI>(p, stream);
}

// A product of few tokens: weights w[0], w[1] (EPI_GATED: of g and u, else of
// each segment; MN: their columns are the product's rows), tokens' rows x[].
template <int EPI, bool A_MN>
ccl_status_t launch_few(GemmParams &p, const Launch &l, const Matrix *w, const Matrix *x, char *partial, cudaStream_t stream)
{
    FewParams fp;
    fp.npad = (uint32_t)(l.s[0].m + 15) / 16 * 16;
    fp.stages = std::min<uint32_t>(kMaxStages, kFewBytes / (2 * kOperandBytes + fp.npad * 128));
    uint64_t units;
    cudaError_t e = set_problems(p, l, partial, &units);
    static std::atomic<unsigned long long> ready{0};
    if (e != cudaSuccess ||
        (e = large_smem_once(reinterpret_cast<const void *>(ffn_few_kernel<EPI, A_MN>), kFewBytes + 1024, ready)) != cudaSuccess)
        return from_cuda(e);
    Problem &q = p.prob[0];
    for (uint32_t i = 0; i < (l.gated ? 2 : q.segs); ++i)
        if (!encode(&q.a[i], w[i], A_MN) || (i < q.segs && !encode(&q.b[i], x[i], false, fp.npad)))
            return CCL_ERR_CUDA;
    fp.p = p;
    if ((e = launch_chained(ffn_few_kernel<EPI, A_MN>, dim3((unsigned)std::min<uint64_t>(units, kSms)), dim3(kGemmThreads), kFewBytes + 1024, stream, fp)) != cudaSuccess)
        return from_cuda(e);
    count_launches(1);
    return from_cuda(launch_join<EPI>(p, stream));
}

struct FfnArgs {
    const void *x, *wg, *wu, *wd;
    size_t t, d, f;
    ccl_dtype_t dtype;
    ccl_act_t act;
    float *saved;
    void *work;
    size_t work_bytes;
};

// The checks that both directions share; on CCL_OK `plan` is ready.
ccl_status_t check_ffn(const FfnArgs &a, bool backward, bool aligned, FfnPlan *plan)
{
    if (!valid_dtype(a.dtype) || (a.act != CCL_ACT_SILU && a.act != CCL_ACT_GELU_TANH))
        return CCL_ERR_INVALID_ARG;
    if (a.dtype != CCL_BF16)
        return CCL_ERR_UNSUPPORTED;
    if (!make_plan(a.t, a.d, a.f, backward, aligned, plan))
        return CCL_ERR_INVALID_ARG;
    return CCL_OK;
}

bool aligned_all(std::initializer_list<const void *> ps)
{
    for (const void *p : ps)
        if ((uintptr_t)p % 16)
            return false;
    return true;
}

#ifdef CCL_DEBUG_BOUNDS
cudaError_t dbg_ffn(const std::vector<Range> &w, const std::vector<Range> &r, cudaStream_t stream)
{
    std::vector<DbgRange> v;
    for (const std::vector<Range> *s : {&w, &r})
        for (const Range &x : *s)
            v.push_back(DbgRange{reinterpret_cast<const void *>(x.lo), (size_t)(x.hi - x.lo)});
    return dbg_set_ranges(v, stream);
}
#define CCL_DBG_FFN(w, r, st)                                                                                          \
    do {                                                                                                               \
        if (cudaError_t e_ = dbg_ffn(w, r, st))                                                                        \
            return from_cuda(e_);                                                                                      \
    } while (0)
#else
#define CCL_DBG_FFN(w, r, st)                                                                                          \
    do {                                                                                                               \
    } while (0)
#endif

ccl_status_t gated_ffn_impl(const FfnArgs &a, void *out, cudaStream_t stream)
{
    FfnPlan pl;
    if (ccl_status_t st = check_ffn(a, false, aligned_all({a.x, a.wg, a.wu, a.wd}), &pl))
        return st;
    if (a.t == 0 || a.d == 0)
        return CCL_OK;
    if (!a.x || !out || (a.f && (!a.wg || !a.wu || !a.wd)) || !element_aligned(2, {a.x, a.wg, a.wu, a.wd, out}) ||
        !element_aligned(4, {a.saved}))
        return CCL_ERR_INVALID_ARG;
    if (a.f == 0)
        return from_cuda(cudaMemsetAsync(out, 0, a.t * a.d * 2, stream));
    if (!a.work || (uintptr_t)a.work % 256 || a.work_bytes < pl.bytes)
        return CCL_ERR_INVALID_ARG;
    std::vector<Range> w{range_of(out, a.t * a.d * 2, 0), range_of(a.work, pl.bytes, 0)};
    if (a.saved)
        w.push_back(range_of(a.saved, 2 * a.t * a.f * 4, 0));
    const std::vector<Range> r{range_of(a.x, a.t * a.d * 2, 0), range_of(a.wg, a.f * a.d * 2, 0),
                               range_of(a.wu, a.f * a.d * 2, 0), range_of(a.wd, a.d * a.f * 2, 0)};
    if (ccl_status_t st = check_overlaps(w, r, [](const Range &, const Range &) { return false; }))
        return st;
    CCL_DBG_FFN(w, r, stream);
    char *work = static_cast<char *>(a.work);
    Operands ops(work);
    const Matrix x = ops.add(a.x, a.t, a.d, pl.x), wd = ops.add(a.wd, a.d, a.f, pl.wd);
    const Matrix w2[2] = {ops.add(a.wg, a.f, a.d, pl.wg), ops.add(a.wu, a.f, a.d, pl.wu)};
    const Matrix h{work + pl.h, a.t, a.f, pl.fp};
    if (cudaError_t e = ops.copy(stream))
        return from_cuda(e);
    GemmParams p{};
    p.act = (int)a.act;
    p.wait_ns = g_wait_ns.load(std::memory_order_relaxed);
    p.h = reinterpret_cast<uint16_t *>(work + pl.h);
    p.g = a.saved;
    p.u = a.saved ? a.saved + a.t * a.f : nullptr;
    p.ldh = (uint32_t)pl.fp;
    char *partial = work + pl.partial;
    p.vectors = a.f % 8 == 0 && (uintptr_t)a.saved % 32 == 0;
    Problem &q = p.prob[0];
    if (pl.up_.few) {
        if (ccl_status_t st = launch_few<EPI_GATED, false>(p, pl.up_, w2, &x, partial, stream))
            return st;
        q.out = out;
        p.early = wd.ptr == a.wd; // not a copy made within this call
        return launch_few<EPI_STORE, false>(p, pl.down, &wd, &h, partial, stream);
    }
    if (!encode(&q.a[0], x, false) || !encode(&q.b[0], w2[0], false) || !encode(&q.b[1], w2[1], false))
        return CCL_ERR_CUDA;
    if (cudaError_t e = launch_gemm<EPI_GATED, false, false>(p, pl.up_, partial, stream))
        return from_cuda(e);
    q.out = out;
    p.vectors = a.d % 8 == 0 && (uintptr_t)out % 16 == 0;
    if (!encode(&q.a[0], h, false) || !encode(&q.b[0], wd, false))
        return CCL_ERR_CUDA;
    return from_cuda(launch_gemm<EPI_STORE, false, false>(p, pl.down, partial, stream));
}

ccl_status_t gated_ffn_grad_impl(const FfnArgs &a, const void *dy, void *dx, void *dwg, void *dwu, void *dwd,
                                 int accumulate, cudaStream_t stream)
{
    FfnPlan pl;
    if (ccl_status_t st = check_ffn(a, true, aligned_all({a.x, a.wg, a.wu, a.wd, dy}), &pl))
        return st;
    if (a.d == 0 || (a.t == 0 && accumulate))
        return CCL_OK;
    const size_t tb = a.t * a.d * 2, wb = a.f * a.d * 2;
    if ((a.t && (!a.x || !dy || (a.f && (!a.wg || !a.wu || !a.wd || !a.saved)))) ||
        !element_aligned(2, {a.x, a.wg, a.wu, a.wd, dy, dx, dwg, dwu, dwd}) || !element_aligned(4, {a.saved}))
        return CCL_ERR_INVALID_ARG;
    const bool empty = a.t == 0 || a.f == 0;
    if (!empty && (!a.work || (uintptr_t)a.work % 256 || a.work_bytes < pl.bytes))
        return CCL_ERR_INVALID_ARG;
    std::vector<Range> w, r;
    if (!empty) {
        w.push_back(range_of(a.work, pl.bytes, 0));
        r = {range_of(a.x, tb, 0), range_of(dy, tb, 0), range_of(a.wg, wb, 0), range_of(a.wu, wb, 0),
             range_of(a.wd, wb, 0), range_of(a.saved, 2 * a.t * a.f * 4, 0)};
    }
    if (dx)
        w.push_back(range_of(dx, tb, 0));
    for (void *g : {dwg, dwu, dwd})
        if (g)
            w.push_back(range_of(g, wb, 0));
    if (ccl_status_t st = check_overlaps(w, r, [](const Range &, const Range &) { return false; }))
        return st;
    if (!dx && !dwg && !dwu && !dwd)
        return CCL_OK;
    cudaError_t e;
    if (empty) { // empty sums
        if (dx && tb && (e = cudaMemsetAsync(dx, 0, tb, stream)))
            return from_cuda(e);
        for (void *g : {dwg, dwu, dwd})
            if (g && wb && !accumulate && (e = cudaMemsetAsync(g, 0, wb, stream)))
                return from_cuda(e);
        return CCL_OK;
    }
    CCL_DBG_FFN(w, r, stream);
    char *work = static_cast<char *>(a.work);
    Operands ops(work);
    const Matrix x = ops.add(a.x, a.t, a.d, pl.x), y = ops.add(dy, a.t, a.d, pl.dy), wd = ops.add(a.wd, a.d, a.f, pl.wd);
    const Matrix w2[2] = {ops.add(a.wg, a.f, a.d, pl.wg), ops.add(a.wu, a.f, a.d, pl.wu)};
    const Matrix h{work + pl.h, a.t, a.f, pl.fp};
    const Matrix d2[2] = {{work + pl.dg, a.t, a.f, pl.fp}, {work + pl.du, a.t, a.f, pl.fp}};
    if ((e = ops.copy(stream)))
        return from_cuda(e);
    GemmParams p{};
    p.act = (int)a.act;
    p.wait_ns = g_wait_ns.load(std::memory_order_relaxed);
    p.h = reinterpret_cast<uint16_t *>(work + pl.h);
    p.dg = reinterpret_cast<uint16_t *>(work + pl.dg);
    p.du = reinterpret_cast<uint16_t *>(work + pl.du);
    p.g = a.saved;
    p.u = a.saved + a.t * a.f;
    p.ldh = (uint32_t)pl.fp;
    char *partial = work + pl.partial;
    p.vectors = a.f % 8 == 0 && (uintptr_t)a.saved % 32 == 0;
    Problem &q = p.prob[0];
    if (pl.dh.few) {
        if (ccl_status_t st = launch_few<EPI_BACKWARD, true>(p, pl.dh, &wd, &y, partial, stream))
            return st;
    } else {
        if (!encode(&q.a[0], y, false) || !encode(&q.b[0], wd, true))
            return CCL_ERR_CUDA;
        if ((e = launch_gemm<EPI_BACKWARD, false, true>(p, pl.dh, partial, stream)))
            return from_cuda(e);
    }
    if (dx) {
        q.out = dx;
        p.vectors = a.d % 8 == 0 && (uintptr_t)dx % 16 == 0;
        if (pl.dx.few) {
            p.early = w2[0].ptr == a.wg && w2[1].ptr == a.wu; // not copies made within this call
            if (ccl_status_t st = launch_few<EPI_STORE, true>(p, pl.dx, w2, d2, partial, stream))
                return st;
        } else {
            for (int i = 0; i < 2; ++i)
                if (!encode(&q.a[i], d2[i], false) || !encode(&q.b[i], w2[i], true))
                    return CCL_ERR_CUDA;
            if ((e = launch_gemm<EPI_STORE, false, true>(p, pl.dx, partial, stream)))
                return from_cuda(e);
        }
    }
    if (!dwg && !dwu && !dwd)
        return CCL_OK;
    // the weight gradients asked for, in one launch
    p.accumulate = accumulate != 0;
    p.vectors = a.d % 8 == 0 && a.f % 8 == 0;
    Launch l = pl.dw;
    l.n = 0;
    const Matrix *am[3] = {&d2[0], &d2[1], &y}, *bm[3] = {&x, &x, &h};
    void *out[3] = {dwg, dwu, dwd};
    for (int i = 0; i < 3; ++i)
        if (out[i]) {
            l.s[l.n] = pl.dw.s[i];
            p.prob[l.n].out = out[i];
            p.vectors = p.vectors && (uintptr_t)out[i] % 16 == 0;
            if (!encode(&p.prob[l.n].a[0], *am[i], true) || !encode(&p.prob[l.n].b[0], *bm[i], true))
                return CCL_ERR_CUDA;
            ++l.n;
        }
    return from_cuda(launch_gemm<EPI_STORE, true, true>(p, l, partial, stream));
}

} // namespace

unsigned long long feed_forward_wait_ns() { return g_wait_ns.load(std::memory_order_relaxed); }

} // namespace ccl

using namespace ccl;

extern "C" {

ccl_status_t ccl_plan_gated_ffn_work_bytes(size_t ntokens, size_t dim, size_t ffn, int backward, int aligned, size_t *bytes)
{
    FfnPlan p;
    if (!bytes || !make_plan(ntokens, dim, ffn, backward != 0, aligned != 0, &p))
        return CCL_ERR_INVALID_ARG;
    *bytes = p.bytes;
    return CCL_OK;
}

ccl_status_t ccl_gated_ffn(const void *x, const void *w_gate, const void *w_up, const void *w_down, size_t ntokens,
                           size_t dim, size_t ffn, ccl_dtype_t dtype, ccl_act_t act, void *out, float *saved, void *work,
                           size_t work_bytes, cudaStream_t stream)
{
    TraceScope tr("gated_ffn", 1, ntokens, (int)dtype, -1, (int)act, stream);
    return tr.done(guarded([&] {
        return gated_ffn_impl(FfnArgs{x, w_gate, w_up, w_down, ntokens, dim, ffn, dtype, act, saved, work, work_bytes},
                              out, stream);
    }));
}

ccl_status_t ccl_gated_ffn_grad(const void *grad_out, const void *x, const void *w_gate, const void *w_up,
                                const void *w_down, const float *saved, size_t ntokens, size_t dim, size_t ffn,
                                ccl_dtype_t dtype, ccl_act_t act, int accumulate, void *grad_x, void *grad_w_gate,
                                void *grad_w_up, void *grad_w_down, void *work, size_t work_bytes, cudaStream_t stream)
{
    TraceScope tr("gated_ffn_grad", 1, ntokens, (int)dtype, -1, (int)act, stream);
    return tr.done(guarded([&] {
        return gated_ffn_grad_impl(FfnArgs{x, w_gate, w_up, w_down, ntokens, dim, ffn, dtype, act,
                                           const_cast<float *>(saved), work, work_bytes},
                                   grad_out, grad_x, grad_w_gate, grad_w_up, grad_w_down, accumulate, stream);
    }));
}

ccl_status_t ccl_set_gated_ffn_wait_limit(unsigned long long ns)
{
    g_wait_ns.store(ns, std::memory_order_relaxed);
    return CCL_OK;
}

ccl_status_t ccl_gated_ffn_timeouts(unsigned long long *count)
{
    if (!count)
        return CCL_ERR_INVALID_ARG;
    const cudaError_t e = cudaMemcpyFromSymbol(count, g_ffn_timeouts, sizeof *count);
    return from_cuda(e == cudaSuccess ? expert_timeouts(count) : e);
}

} // extern "C"
