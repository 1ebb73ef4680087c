// experts.cu -- the gated feed-forward blocks of a layer's experts over rows in
// expert order, forward and backward, with the activations kept in 8 bits.
//
// The products are ffn.cu's, expert by expert, and so is the machinery: CTA
// pairs with 256 x 256 fp32 accumulators in tensor memory (tcgen05.mma), a ring
// of stages filled by TMA, epilogues that carry the activation and its
// derivative.  What is its own:
//   - The experts' row counts stay on the device.  Every CTA makes a table of
//     the experts' first rows and row tiles from the offsets, and the persistent
//     grid walks (expert, tile) units of one launch for all experts.  The
//     weights' tensor maps have the expert as third dimension, so that a tile
//     past an expert's units reads zeros and not the next one's.
//   - A row tile that begins in one expert's rows may read the next one's: rows
//     of a product do not meet, and the epilogue writes an expert's own rows.
//     Only in the weight gradients are rows summed over.  There every expert's
//     rows begin at a multiple of 64 (a K block) in a padded layout of the work
//     buffer, zeros behind them: h, dg and du are written there by the epilogue
//     that makes them, and of x and the incoming gradient the last, partial
//     block of each expert is copied there (all rows, where TMA cannot address
//     them or x is kept in 8 bits), so that no row, finite or not, reaches
//     another expert's sums.
//   - g and u are kept in 8 bits (act8.cuh): an epilogue thread holds 32
//     consecutive columns of a row, which is a block.  The codes' rows are whole
//     blocks, and zeros behind the last column come from the tensor maps.
//   - Few rows an expert: the weights are the accumulator's rows and a tile of
//     16 to 128 tokens its columns (expert_few_kernel), the sums cut along K when
//     that leaves SMs idle.  (Cutting them on pairs was slower: 35 -> 41 us and
//     the join for the gradient by 4026 rows of 320.)
//
// Bound by the tensor cores for many rows an expert, by reading the weights (and
// writing their gradients) for few.  Two experts of eight for each of 4096
// tokens at 4096 x 11008, forward: 1.31-1.37 ms, at the power limit 1.45-1.55
// (1.45-1.69 PFLOP/s; cuBLAS sustains 1.72 there), an eighth of the products
// being of row tiles that an expert does not fill; the same for one token 94 us
// (5.7 TB/s of weights, 0.85 of the copy bandwidth).  Forward and backward of
// 32768 rows over 32 experts of 2048 x 1408: 1.36-1.5 ms, 1.1-1.25 PFLOP/s.
#include <algorithm>
#include <vector>

#include "../../include/ccl.h"
#include "act8.cuh"
#include "ccl_internal.h"
#include "step_ops.cuh"
#include "tensor_core.cuh"

namespace ccl {
namespace {

constexpr int kTileM = 256, kTileN = 256, kTileK = 64; // a CTA pair's tile
constexpr int kOperandBytes = 128 * kTileK * 2;        // one CTA's part of A or B in a stage
constexpr int kStageBytes = 2 * kOperandBytes;
constexpr int kStages = 6, kStagedStages = 4; // the latter beside the room that outputs are staged in
constexpr int kEpiWarps = 8, kFewThreads = 128 + 32 * kEpiWarps; // expert_few_kernel's: beside them producer, issuer, tensor memory, an idle warp
// Staging: 32 rows of 128 bf16 columns for each of the epilogue warps.  The
// pitch puts eight rows' 16 bytes in different banks.
constexpr uint32_t kPitch = 272, kStaging = 32 * kPitch;
constexpr int kTableBytes = 3 * (CCL_MAX_EXPERTS + 2) * 4;
constexpr int kGemmSmem = 1024 /* alignment */ + kTableBytes + std::max(kStages * kStageBytes, kStagedStages * kStageBytes + kEpiWarps * (int)kStaging);
constexpr int kGroupM = 8; // row tiles walked before the next column tile
constexpr uint32_t kPad = kTileK; // an expert's rows in the padded layout are a multiple of this
constexpr int kFewStages = 6;
constexpr int kFewBytes = 190 * 1024; // its stages', at most
constexpr uint32_t kFewMost = 128;    // tokens of one tile

enum Epilogue { EPI_GATED = 0, EPI_STORE = 1, EPI_BACKWARD = 2, EPI_WEIGHTS = 3 };
// Epilogue warps of expert_gemm_kernel.  dh's epilogue has the most to do: over a
// short K twelve are faster (the gradient by 4000 rows of 320, ffn 2944: 66.3 us
// with eight, 63.9), over a long one equal (435).  The others' hide behind their
// products, which sixteen slowed down by 5 %.
template <int EPI> constexpr int kWarpsOf = EPI == EPI_BACKWARD ? 12 : kEpiWarps;
template <int EPI> constexpr int kThreadsOf = 128 + 32 * kWarpsOf<EPI>;

// An epilogue warp's lane has a row of the accumulator and writes 32 bytes of it
// at a time.  Rows that no 16-byte vector divides are staged in shared memory
// (STAGED), so that the warp writes words along a row (weight gradients of 73
// experts of 530 x 1809: a value a lane 760 us, staged 220); for whole vectors
// staging costs more than full lines gain (44 -> 60 us).  Launches with staged
// outputs neither begin before the kernel before them has ended nor let the next
// one begin.

// Division of numbers below 2^31 by a number that the host knows: the multiplier
// and shift of Granlund and Montgomery, "Division by invariant integers using
// multiplication" (1994).  Each role of a CTA works out every unit it takes part
// in, which the divider's chain made most of for the shortest products.
struct Divisor {
    uint32_t mul, shift, by;
    __device__ __forceinline__ uint32_t operator()(uint32_t n) const { return (__umulhi(n, mul) + n) >> shift; }
};

Divisor divisor(uint32_t by)
{
    uint32_t shift = 0;
    while (shift < 31 && (1u << shift) < by)
        ++shift;
    return Divisor{(uint32_t)((((1ull << shift) - by) << 32) / by + 1), shift, by};
}

// C[M, N] = sum over segments of A_s[M, K] B_s[N, K]^T for each expert: M its
// rows, or for EPI_WEIGHTS K its rows.
struct Problem {
    CUtensorMap a[2], b[2];
    void *out;      // EPI_STORE: row stride n; EPI_WEIGHTS: [experts][m][n]
    uint32_t m, n;  // m: EPI_WEIGHTS only
    uint32_t mt, nt; // tiles (mt: EPI_WEIGHTS only)
    Divisor by_nt, by_group; // nt, kGroupM * nt
    uint32_t kblocks, segs;
    // EPI_WEIGHTS: a[1], b[1] are the rows as they lie, which full blocks of K
    // are read from; the last, partial one is in the padded layout (a[0], b[0])
    int direct_a, direct_b;
};

struct ExpertParams {
    Problem prob[3];
    uint32_t nprob;
    Divisor by_expert; // EPI_WEIGHTS: an expert's units
    const int32_t *offsets;
    uint32_t experts, rows;
    int act, accumulate;
    uint16_t *h, *dg, *du; // rows of ldh columns
    int8_t *codes[2];      // of g and u: rows of ldh columns
    uint8_t *scales[2];
    uint32_t ldh;
    int padded;  // A's rows are those of the padded layout
    uint32_t half; // columns of B that a CTA of the pair brings: half a tile's
    unsigned long long wait_ns;
    // expert_few_kernel
    float *partial; // [splits][rows][column tiles * 256]
    uint32_t splits, npad, stages;
    int early; // the weights and the offsets may be read before the kernel before this one has ended
};

__device__ unsigned long long g_expert_timeouts;

__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, volatile int *gave_up, unsigned long long limit)
{
    return ccl::mbar_wait(bar, parity, gave_up, limit, &g_expert_timeouts);
}

// ------------------------------------------------------------------ the experts' rows

// [experts + 1] each: an expert's first row, its first row tile, its first row
// in the padded layout.
struct Table {
    int32_t *row0, *tile0, *pad0;
};

// The offset as any CTA sees it, whatever its L1 held.
__device__ __forceinline__ int32_t load_offset(const int32_t *p)
{
    int32_t v = 0;
    if (dbg_ok(p, 4))
        asm volatile("ld.relaxed.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}

// All threads of the CTA; complete when it returns.
__device__ __forceinline__ void make_table(const ExpertParams &p, const Table &t, uint32_t tile)
{
    const uint32_t E = p.experts, lane = threadIdx.x & 31;
    for (uint32_t e = threadIdx.x; e <= E; e += blockDim.x)
        t.row0[e] = min(max(load_offset(p.offsets + e), 0), (int32_t)p.rows);
    __syncthreads();
    if (threadIdx.x < 32) {
        int32_t top = 0;
        for (uint32_t e0 = 0; e0 <= E; e0 += 32) {
            int32_t v = e0 + lane <= E ? t.row0[e0 + lane] : 0;
            v = max(v, top);
#pragma unroll
            for (int d = 1; d < 32; d *= 2) {
                const int32_t o = __shfl_up_sync(0xffffffffu, v, d);
                if (lane >= (uint32_t)d)
                    v = max(v, o);
            }
            if (e0 + lane <= E)
                t.row0[e0 + lane] = v;
            top = __shfl_sync(0xffffffffu, v, 31);
        }
        __syncwarp();
        int32_t tiles = 0, pads = 0;
        for (uint32_t e0 = 0; e0 <= E; e0 += 32) {
            const uint32_t e = e0 + lane;
            const int32_t n = e < E ? t.row0[e + 1] - t.row0[e] : 0;
            const int32_t mine = (int32_t)((n + tile - 1) / tile), pad = (int32_t)((n + kPad - 1) / kPad);
            int32_t a = mine, b = pad;
#pragma unroll
            for (int d = 1; d < 32; d *= 2) {
                const int32_t oa = __shfl_up_sync(0xffffffffu, a, d), ob = __shfl_up_sync(0xffffffffu, b, d);
                if (lane >= (uint32_t)d) {
                    a += oa;
                    b += ob;
                }
            }
            if (e <= E) {
                t.tile0[e] = tiles + a - mine;
                t.pad0[e] = (pads + b - pad) * (int32_t)kPad;
            }
            tiles += __shfl_sync(0xffffffffu, a, 31);
            pads += __shfl_sync(0xffffffffu, b, 31);
        }
    }
    __syncthreads();
}

// The last expert whose entry is at most x (the entries rise, x is below the last).
__device__ __forceinline__ uint32_t expert_at(const int32_t *first, uint32_t experts, int32_t x)
{
    uint32_t lo = 0, hi = experts;
    while (hi - lo > 1) {
        const uint32_t mid = (lo + hi) / 2;
        if (first[mid] <= x)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

struct Unit {
    uint32_t prob, expert, m, n, kblocks, split;
    uint32_t half; // columns of B that each CTA of the pair brings: p.half, or fewer in the last column tile
    uint32_t row0, rows, pad0; // the expert's
};

template <int EPI> __device__ __forceinline__ uint32_t units_of(const ExpertParams &p, const Table &t)
{
    if (EPI != EPI_WEIGHTS)
        return (uint32_t)t.tile0[p.experts] * p.prob[0].nt;
    return p.by_expert.by * p.experts;
}

template <int EPI> __device__ __forceinline__ Unit unit_at(const ExpertParams &p, const Table &tb, uint32_t i)
{
    Unit u;
    u.prob = u.split = 0;
    uint32_t t, mt;
    if (EPI == EPI_WEIGHTS) {
        u.expert = p.by_expert(i);
        t = i - u.expert * p.by_expert.by;
        while (t >= p.prob[u.prob].mt * p.prob[u.prob].nt) {
            t -= p.prob[u.prob].mt * p.prob[u.prob].nt;
            ++u.prob;
        }
        mt = p.prob[u.prob].mt;
    } else {
        const uint32_t nt = p.prob[0].nt;
        u.expert = expert_at(tb.tile0, p.experts, (int32_t)p.prob[0].by_nt(i));
        t = i - (uint32_t)tb.tile0[u.expert] * nt;
        mt = (uint32_t)(tb.tile0[u.expert + 1] - tb.tile0[u.expert]);
    }
    const Problem &q = p.prob[u.prob];
    const uint32_t grp = q.by_group(t), in = t - grp * kGroupM * q.nt, gm = mt - grp * kGroupM;
    if (gm >= kGroupM) {
        u.n = in / kGroupM;
        u.m = grp * kGroupM + in % kGroupM;
    } else if (gm == 1) {
        u.n = in;
        u.m = grp * kGroupM;
    } else {
        u.n = in / gm;
        u.m = grp * kGroupM + in % gm;
    }
    u.row0 = (uint32_t)tb.row0[u.expert];
    u.rows = (uint32_t)tb.row0[u.expert + 1] - u.row0;
    u.pad0 = (uint32_t)tb.pad0[u.expert];
    u.kblocks = EPI == EPI_WEIGHTS ? (u.rows + kTileK - 1) / kTileK : q.kblocks * q.segs;
    const uint32_t left = EPI == EPI_GATED ? q.n - u.n * p.half : (q.n - u.n * 2 * p.half + 1) / 2;
    u.half = min(p.half, EPI == EPI_GATED ? (left + 31) / 32 * 32 : (left + 15) / 16 * 16);
    return u;
}

// ------------------------------------------------------------------ copies

// A 3-D box (one expert's) of a tensor map, counted at `bar` of the pair's first CTA.
__device__ __forceinline__ void tma_load3(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint32_t bar)
{
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 "
                 "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
                 "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
                 : "memory");
}

__device__ __forceinline__ void tma_load3_own(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint32_t bar)
{
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
                 "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
                 : "memory");
}

template <bool MN> __device__ __forceinline__ void load_rows(uint32_t dst, const CUtensorMap *map, int mn, int k, uint32_t bar)
{
    if (MN) {
        tma_load(dst, map, mn, k, bar);
        tma_load(dst + kOperandBytes / 2, map, mn + 64, k, bar);
    } else {
        tma_load(dst, map, k, mn, bar);
    }
}

template <bool MN> __device__ __forceinline__ void load_expert(uint32_t dst, const CUtensorMap *map, int mn, int k, int e, uint32_t bar)
{
    if (MN) {
        tma_load3(dst, map, mn, k, e, bar);
        tma_load3(dst + kOperandBytes / 2, map, mn + 64, k, e, bar);
    } else {
        tma_load3(dst, map, k, mn, e, bar);
    }
}

// ------------------------------------------------------------------ epilogues

__device__ __forceinline__ void tc_load64(uint32_t addr, float *f)
{
    uint32_t r[64];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x64.b32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
                 "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, "
                 "%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, "
                 "%48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%64];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
                   "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
                   "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
                   "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]),
                   "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]),
                   "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]),
                   "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
                 : "r"(addr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 64; ++i)
        f[i] = __uint_as_float(r[i]);
}

constexpr uint32_t kNanBits = 0x7fffffffu;

// act(g) and act'(g) as activation() has them, in fewer instructions: the
// epilogues of products over a short K are bound by these.  With a = g s,
// SiLU' = s + a (1 - s), and GELU's (tanh form) the same times the inner
// derivative of its second term.
__device__ __forceinline__ void gate(int act, float g, float &a, float &da)
{
    constexpr float c2 = 1.5957691216057308f; // 2 sqrt(2/pi)
    if (act == CCL_ACT_SILU) {
        const float s = sigmoid(g);
        a = __fmul_rn(g, s);
        da = __fmaf_rn(a, __fadd_rn(1.0f, -s), s);
    } else {
        const float gg = __fmul_rn(g, g);
        const float s = sigmoid(__fmul_rn(g, __fmaf_rn(0.044715f * c2, gg, c2)));
        const float t = __fadd_rn(1.0f, -s), as = __fmul_rn(g, s);
        a = as;
        da = t == 0.0f ? s : __fmaf_rn(__fmul_rn(as, t), __fmaf_rn(3 * 0.044715f * c2, gg, c2), s);
        da = s == 0.0f ? 0.0f : da; // where the polynomial has overflowed
    }
}

__device__ __forceinline__ void store32(uint16_t *q, const float *f)
{
    st32(q, pack<DT_BF16>(f), pack<DT_BF16>(f + 8));
    st32(q + 16, pack<DT_BF16>(f + 16), pack<DT_BF16>(f + 24));
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

__device__ __forceinline__ void shared_store16(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

__device__ __forceinline__ uint4 shared_load16(uint32_t at)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}

__device__ __forceinline__ uint32_t shared_load4(uint32_t at)
{
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    return v;
}

// A warp's staged rows (at most 32, of `cols` <= 128 columns) to out, rows `ld`
// apart: as words, with single values at the ends.  `step` 2 takes every second
// row where rows of an odd length change their parity.
__device__ __forceinline__ void staged_out(uint32_t staging, uint16_t *out, uint64_t ld, uint32_t rows, uint32_t cols)
{
    const uint32_t lane = threadIdx.x & 31, step = ld % 2 ? 2 : 1;
    for (uint32_t r0 = 0; r0 < step && r0 < rows && cols; ++r0) {
        uint16_t *dst = out + r0 * ld;
        uint32_t src = staging + r0 * kPitch;
        const uint32_t odd = ((uintptr_t)dst & 2) / 2, n = (rows - r0 + step - 1) / step; // words begin at column `odd`
        const bool first = 2 * lane + odd + 1 < cols, second = 2 * lane + 64 + odd + 1 < cols;
        const bool edge = lane == 0 ? odd : lane == 1 ? cols > odd && (cols - odd) % 2 : false; // the columns that no word holds
        const uint32_t at = lane == 0 ? 0 : cols - 1, shift = odd * 16;
#pragma unroll 4
        for (uint32_t r = 0; r < n; ++r, dst += step * ld, src += step * kPitch) {
            uint32_t a = shared_load4(src + 4 * lane), b = shared_load4(src + 4 * lane + 128);
            if (odd) {
                a = __funnelshift_r(a, shared_load4(src + 4 * lane + 4), shift);
                b = __funnelshift_r(b, shared_load4(src + 4 * lane + 132), shift);
            }
            if (first)
                gstore<uint32_t>(dst + 2 * lane + odd, a);
            if (second)
                gstore<uint32_t>(dst + 2 * lane + 64 + odd, b);
            if (edge)
                gstore<uint16_t>(dst + at, (uint16_t)(shared_load4(src + at / 2 * 4) >> at % 2 * 16));
        }
    }
}

// The other way: what the rows hold now.
__device__ __forceinline__ void staged_in(uint32_t staging, const uint16_t *out, uint64_t ld, uint32_t rows, uint32_t cols)
{
    const uint32_t lane = threadIdx.x & 31;
#pragma unroll 2
    for (uint32_t r = 0; r < rows; ++r)
#pragma unroll
        for (uint32_t k = 0; k < 4; ++k) {
            const uint32_t c = lane + 32 * k;
            const uint16_t v = c < cols ? gload<uint16_t>(out + r * ld + c) : (uint16_t)0;
            asm volatile("st.shared.u16 [%0], %1;" ::"r"(staging + r * kPitch + 2 * c), "h"(v) : "memory");
        }
}

// A block of g (k = 0) or u (k = 1) of a row in 8 bits.
__device__ __forceinline__ void keep(const ExpertParams &p, int k, uint64_t at, const float *f)
{
    uint4 lo, hi;
    const uint32_t b = act8_encode(f, lo, hi);
    st32(p.codes[k] + at, lo, hi);
    gstore<uint8_t>(p.scales[k] + at / kActBlock, (uint8_t)b);
}

// h of sixteen columns of a row.  What would lie past the last column is zero.
__device__ __forceinline__ void finish_gated(const ExpertParams &p, uint64_t at, float *g, const float *u)
{
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        float a, da;
        gate(p.act, g[i], a, da);
        g[i] = __fmul_rn(a, u[i]);
    }
    st32(p.h + at, pack<DT_BF16>(g), pack<DT_BF16>(g + 8));
}

// What the backward epilogue reads of a block: the codes of g and u, and steps.
struct Saved {
    uint4 g[2], u[2];
    float sg, su;
    __device__ __forceinline__ void load(const ExpertParams &p, uint64_t at, bool in)
    {
        if (!in)
            return;
        ld32(p.codes[0] + at, g[0], g[1]);
        ld32(p.codes[1] + at, u[0], u[1]);
        sg = act8_step(gload<uint8_t>(p.scales[0] + at / kActBlock));
        su = act8_step(gload<uint8_t>(p.scales[1] + at / kActBlock));
    }
};

// dh to dg, du and h, sixteen columns of a row: the first or second half of a block.
__device__ __forceinline__ void finish_backward(const ExpertParams &p, uint64_t to, const Saved &s, uint32_t second, const float *v)
{
    const uint4 cg = s.g[second], cu = s.u[second];
    const uint32_t wg[4] = {cg.x, cg.y, cg.z, cg.w}, wu[4] = {cu.x, cu.y, cu.z, cu.w};
    float h[16], dg[16], du[16];
#pragma unroll
    for (int j = 0; j < 16; j += 4) {
        float g[4], u[4];
        act8_decode4(wg[j / 4], s.sg, g);
        act8_decode4(wu[j / 4], s.su, u);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float a, da;
            gate(p.act, g[k], a, da);
            const float d = v[j + k];
            h[j + k] = __fmul_rn(a, u[k]);
            dg[j + k] = __fmul_rn(__fmul_rn(d, u[k]), da);
            du[j + k] = __fmul_rn(d, a);
        }
    }
    st32(p.h + to, pack<DT_BF16>(h), pack<DT_BF16>(h + 8));
    st32(p.dg + to, pack<DT_BF16>(dg), pack<DT_BF16>(dg + 8));
    st32(p.du + to, pack<DT_BF16>(du), pack<DT_BF16>(du + 8));
}

__device__ __forceinline__ void backward_zeros(const ExpertParams &p, uint64_t to)
{
    const uint4 z = make_uint4(0, 0, 0, 0);
    st32(p.h + to, z, z);
    st32(p.dg + to, z, z);
    st32(p.du + to, z, z);
}

// Sixteen (or eight) finished sums of one row of an output, added to what is
// there when accumulating.
__device__ __forceinline__ void finish_store(const ExpertParams &p, uint16_t *out, bool both, const Vals16 &old, float *v)
{
    if (p.accumulate) {
        float a[16];
        unpack<DT_BF16>(old.v[0], a);
        unpack<DT_BF16>(old.v[1], a + 8);
#pragma unroll
        for (int i = 0; i < 16; ++i)
            v[i] = __fadd_rn(a[i], v[i]);
    }
    store16(out, v, both);
}

// The unit's output rows: how many of its 256, and the first one's address.
template <int EPI> __device__ __forceinline__ uint16_t *unit_out(const ExpertParams &p, const Unit &u, uint32_t &rows)
{
    const Problem &q = p.prob[u.prob];
    uint16_t *out = static_cast<uint16_t *>(q.out);
    if (EPI == EPI_WEIGHTS) {
        rows = q.m;
        return out + (uint64_t)u.expert * q.m * q.n;
    }
    rows = u.rows;
    return out + (uint64_t)u.row0 * q.n;
}

// ------------------------------------------------------------------ the product on CTA pairs

// A warp loads, a lane of the pair's first CTA issues, eight or twelve warps work
// on the accumulator before this one's.  8192 rows over 8 experts of 4096 x 11008: g, u
// and h 908 us and y 466 (tensor pipe 89 and 91 % busy).  32768 rows over 32 of
// 2048 x 1408: g, u, h and their 8 bits 255, y 137, dh with dg, du and h 172 (60 %:
// its epilogue reads 0.10 GB and writes 0.28), dx 252 (84 %), weight gradients 379 (74 %).
template <int EPI, bool A_MN, bool B_MN, bool STAGED>
__global__ void __launch_bounds__(kThreadsOf<EPI>, 1) expert_gemm_kernel(const __grid_constant__ ExpertParams p)
{
    extern __shared__ uint8_t raw[];
    __shared__ uint64_t bars[2 * kStages + 4];
    __shared__ uint32_t tmem_slot;
    __shared__ volatile int gave_up;
    const uint32_t stages = (smem_u32(raw) + 1023) & ~1023u;
    constexpr uint32_t nstages = STAGED ? kStagedStages : kStages;
    uint8_t *behind = raw + (stages - smem_u32(raw)) + nstages * kStageBytes + (STAGED ? kEpiWarps * kStaging : 0);
    const Table table{reinterpret_cast<int32_t *>(behind), reinterpret_cast<int32_t *>(behind) + CCL_MAX_EXPERTS + 2,
                      reinterpret_cast<int32_t *>(behind) + 2 * (CCL_MAX_EXPERTS + 2)};
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
            mbar_init(acc_empty + 8 * i, 2 * kWarpsOf<EPI>);
        }
        if ((gave_up = p.wait_ns == 0))
            atomicAdd(&g_expert_timeouts, 1ull);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 3 && lane / 4 < p.nprob) {
        const Problem &q = p.prob[lane / 4];
        const int i = lane & 1;
        if (lane & 2 ? i < (EPI == EPI_GATED ? 2 : q.segs + q.direct_b) : i < q.segs + q.direct_a)
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
    if (!STAGED)
        chain_entry();
    make_table(p, table, kTileM);
    const uint32_t total = units_of<EPI>(p, table);

    if (warp == 0 && lane == 0) {
        // producer: this CTA's halves of A and B, stage by stage
        const uint32_t leader_full = in_cta(full, 0);
        uint32_t s = 0, phase = 0;
        bool ok = p.wait_ns != 0;
        for (uint32_t i = pair; ok && i < total; i += pairs) {
            const Unit u = unit_at<EPI>(p, table, i);
            const Problem &q = p.prob[u.prob];
            // a half tile behind the expert's rows: from past the matrix, zeros that cost neither traffic nor much power
            const uint32_t in = u.m * kTileM + rank * 128;
            const int am = EPI == EPI_WEIGHTS ? (int)in : in >= u.rows ? 0x7fffff00 : (int)(in + (p.padded ? u.pad0 : u.row0));
            const int bn = (int)(EPI == EPI_GATED ? u.n * p.half : u.n * 2 * p.half + rank * u.half);
            for (uint32_t kb = 0; kb < u.kblocks; ++kb) {
                if (!(ok = mbar_wait(empty + 8 * s, phase ^ 1, &gave_up, p.wait_ns)))
                    break;
                if (rank == 0)
                    mbar_expect(full + 8 * s, 2 * kStageBytes);
                const uint32_t at = stages + s * kStageBytes;
                if (EPI == EPI_WEIGHTS) {
                    const int padded = (int)(u.pad0 + kb * kTileK), lies = (int)(u.row0 + kb * kTileK);
                    const bool whole = (kb + 1) * kTileK <= u.rows;
                    const bool da = q.direct_a && whole, db = q.direct_b && whole;
                    load_rows<A_MN>(at, &q.a[da], am, da ? lies : padded, leader_full + 8 * s);
                    load_rows<B_MN>(at + kOperandBytes, &q.b[db], bn, db ? lies : padded, leader_full + 8 * s);
                } else {
                    const uint32_t seg = kb >= q.kblocks ? 1 : 0;
                    const int k = (int)((kb - seg * q.kblocks) * kTileK);
                    load_rows<A_MN>(at, &q.a[seg], am, k, leader_full + 8 * s);
                    load_expert<B_MN>(at + kOperandBytes, EPI == EPI_GATED ? &q.b[rank] : &q.b[seg], bn, k, (int)u.expert, leader_full + 8 * s);
                }
                if (++s == nstages) {
                    s = 0;
                    phase ^= 1;
                }
            }
        }
        // the issuer's last arrivals reach both CTAs while they are here
        for (uint32_t i = 0; ok && i < nstages; ++i) {
            ok = mbar_wait(empty + 8 * s, phase ^ 1, &gave_up, p.wait_ns);
            if (++s == nstages) {
                s = 0;
                phase ^= 1;
            }
        }
    } else if (warp == 1 && lane == 0 && rank == 0) {
        // issuer: fp32 accumulator, bf16 operands, their majorness, N, M
        constexpr uint32_t form = 1u << 4 | 1u << 7 | 1u << 10 | (A_MN ? 1u << 15 : 0) | (B_MN ? 1u << 16 : 0) | (kTileM >> 4) << 24;
        uint32_t s = 0, phase = 0, t = 0;
        bool ok = p.wait_ns != 0;
        auto products = [&](uint32_t buf, uint32_t kblocks, uint32_t idesc) {
            for (uint32_t kb = 0; kb < kblocks; ++kb) {
                if (!(ok = mbar_wait(full + 8 * s, phase, &gave_up, p.wait_ns)))
                    break;
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                const uint32_t at = stages + s * kStageBytes;
#pragma unroll
                for (int k = 0; k < kTileK / 16; ++k)
                    tc_mma(tmem + buf * kTileN, operand_desc<A_MN>(at + k * k_step<A_MN>()),
                           operand_desc<B_MN>(at + kOperandBytes + k * k_step<B_MN>()), idesc, kb > 0 || k > 0);
                tc_commit(empty + 8 * s);
                if (++s == nstages) {
                    s = 0;
                    phase ^= 1;
                }
            }
        };
        for (uint32_t i = pair; ok && i < total; i += pairs) {
            const Unit u = unit_at<EPI>(p, table, i);
            if (u.kblocks == 0)
                continue; // an expert without rows: the epilogue needs no accumulator
            const uint32_t buf = t & 1;
            if (!(ok = mbar_wait(acc_empty + 8 * buf, ((t >> 1) & 1) ^ 1, &gave_up, p.wait_ns)))
                break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            // a tile of full width by a constant: a descriptor that is not costs the products 3 %
            if (u.half == 128)
                products(buf, u.kblocks, form | (kTileN >> 3) << 17);
            else
                products(buf, u.kblocks, form | (2 * u.half >> 3) << 17);
            if (ok)
                tc_commit(acc_full + 8 * buf);
            ++t;
        }
    } else if (warp >= 4) {
        // epilogue: warp w reads lanes 32 (w % 4) .. + 32 and every second 32
        // columns (EPI_BACKWARD: third), or of an output one half of the columns
        constexpr uint32_t kStride = 32 * kWarpsOf<EPI> / 4;
        const uint32_t c0 = (warp - 4) / 4 * 32;
        const uint32_t lanes = (uint32_t)(warp & 3) * 32;
        const uint32_t leader_empty = in_cta(acc_empty, 0);
        const uint32_t staging = stages + nstages * kStageBytes + (warp - 4) * kStaging;
        uint32_t t = 0, i = pair;
        for (; p.wait_ns && i < total; i += pairs) {
            const Unit u = unit_at<EPI>(p, table, i);
            const Problem &q = p.prob[u.prob];
            const uint32_t buf = t & 1;
            const uint32_t in0 = u.m * kTileM + rank * 128 + lanes, in = in0 + lane; // rows within the expert's
            const uint32_t cols = EPI == EPI_GATED ? u.half : 2 * u.half, col0 = u.n * (EPI == EPI_GATED ? 1 : 2) * p.half;
            const bool some = EPI != EPI_WEIGHTS || u.kblocks;
            if (!some && p.accumulate)
                continue; // nothing is added
            Saved ahead;
            if (EPI == EPI_BACKWARD)
                ahead.load(p, (uint64_t)(u.row0 + in) * p.ldh + col0 + c0, in < u.rows && c0 < cols);
            bool ok = true;
            if (some)
                ok = __all_sync(0xffffffffu, mbar_wait(acc_full + 8 * buf, (t >> 1) & 1, &gave_up, p.wait_ns));
            if (!ok)
                break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            const uint32_t acc = tmem + buf * kTileN + (lanes << 16);
            auto release = [&] { // the accumulator has been read
                asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
                __syncwarp();
                if (lane == 0)
                    mbar_arrive_cluster(leader_empty + 8 * buf);
                ++t;
            };
            if (EPI == EPI_GATED) {
                for (uint32_t c = c0; c < cols && in0 < u.rows; c += kStride) {
                    const uint64_t at = (uint64_t)(u.row0 + in) * p.ldh + col0 + c;
                    if (p.codes[0]) {
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            float f[32];
                            tc_load32(acc + k * u.half + c, f);
                            if (in < u.rows)
                                keep(p, k, at, f);
                        }
                    }
#pragma unroll
                    for (int k = 0; k < 2; ++k) { // read again, which costs less than the registers
                        float g[16], v[16];
                        tc_load16(acc + c + 16 * k, g);
                        tc_load16(acc + u.half + c + 16 * k, v);
                        if (in < u.rows)
                            finish_gated(p, at + 16 * k, g, v);
                    }
                }
                release();
            } else if (EPI == EPI_BACKWARD) {
                const bool behind = in < (u.rows + kPad - 1) / kPad * kPad; // the padding's zeros
                for (uint32_t c = c0; c < cols && __any_sync(0xffffffffu, behind); c += kStride) {
                    Saved next;
                    next.load(p, (uint64_t)(u.row0 + in) * p.ldh + col0 + c + kStride, in < u.rows && c + kStride < cols);
                    const uint64_t to = (uint64_t)(u.pad0 + in) * p.ldh + col0 + c;
#pragma unroll
                    for (uint32_t k = 0; k < 2; ++k) {
                        float v[16];
                        tc_load16(acc + c + 16 * k, v);
                        if (in < u.rows)
                            finish_backward(p, to + 16 * k, ahead, k, v);
                        else if (behind)
                            backward_zeros(p, to + 16 * k);
                    }
                    ahead = next;
                }
                release();
            } else {
                // one half of the tile's columns, 64 at a time
                uint32_t rows;
                const uint32_t c1 = (warp - 4) / 4 * u.half;
                uint16_t *out = unit_out<EPI>(p, u, rows) + (uint64_t)in0 * q.n + col0 + c1; // the warp's first row
                rows = rows > in0 ? min(rows - in0, 32u) : 0;
                const uint32_t wide = col0 + c1 < q.n ? min(q.n - col0 - c1, u.half) : 0; // columns that there are
                if (STAGED && p.accumulate) {
                    staged_in(staging, out, q.n, rows, wide);
                    __syncwarp();
                }
                const uint32_t n = lane < rows ? wide : 0; // of this lane's row
                uint16_t *at = out + (uint64_t)lane * q.n;
                for (uint32_t c = 0; c < u.half && rows; c += 64) { // the last columns read may be the other half's
                    Vals16 old[4];
#pragma unroll
                    for (uint32_t k = 0; k < 4; ++k)
                        if (!STAGED && p.accumulate && c + 16 * k < n)
                            old[k].load(at + c + 16 * k, c + 16 * k + 8 < n);
                    float v[64];
                    if (some) {
                        tc_load64(acc + c1 + c, v);
                    } else {
#pragma unroll
                        for (int j = 0; j < 64; ++j)
                            v[j] = 0.0f;
                    }
#pragma unroll
                    for (uint32_t k = 0; k < 4; ++k) {
                        if (STAGED) {
                            const uint32_t to = staging + lane * kPitch + 2 * (c + 16 * k); // 64 columns: inside the row of 128
                            uint32_t w[8];
#pragma unroll
                            for (int j = 0; j < 8; j += 4) {
                                uint4 x = make_uint4(0, 0, 0, 0);
                                if (p.accumulate)
                                    x = shared_load16(to + 4 * j);
                                const uint32_t was[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                                for (int l = 0; l < 4; ++l) {
                                    const float *f = v + 16 * k + 2 * (j + l);
                                    w[j + l] = p.accumulate ? pack2(__fadd_rn(__uint_as_float(was[l] << 16), f[0]),
                                                                    __fadd_rn(__uint_as_float(was[l] & 0xffff0000u), f[1]))
                                                            : pack2(f[0], f[1]);
                                }
                                shared_store16(to + 4 * j, w[j], w[j + 1], w[j + 2], w[j + 3]);
                            }
                        } else if (c + 16 * k < n) {
                            finish_store(p, at + c + 16 * k, c + 16 * k + 8 < n, old[k], v + 16 * k);
                        }
                    }
                }
                if (some)
                    release();
                if (STAGED) {
                    __syncwarp();
                    staged_out(staging, out, q.n, rows, wide);
                    __syncwarp();
                }
            }
        }
        // after a wait that gave up: NaN in everything that could not be computed
        const float nan = __uint_as_float(kNanBits);
        for (; i < total; i += pairs) {
            const Unit u = unit_at<EPI>(p, table, i);
            const Problem &q = p.prob[u.prob];
            const uint32_t in = u.m * kTileM + rank * 128 + lanes + lane;
            const uint32_t cols = EPI == EPI_GATED ? u.half : 2 * u.half, col0 = u.n * (EPI == EPI_GATED ? 1 : 2) * p.half;
            const bool none = EPI == EPI_WEIGHTS && u.kblocks == 0; // no sum to give up
            for (uint32_t c = c0; c < cols; c += kStride) {
                float v[32];
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    v[j] = nan;
                if (EPI == EPI_GATED) {
                    const uint64_t at = (uint64_t)(u.row0 + in) * p.ldh + col0 + c;
                    if (in < u.rows) {
                        store32(p.h + at, v);
                        for (int k = 0; k < 2 && p.codes[0]; ++k)
                            keep(p, k, at, v);
                    }
                } else if (EPI == EPI_BACKWARD) {
                    const uint64_t to = (uint64_t)(u.pad0 + in) * p.ldh + col0 + c;
                    if (in < u.rows) {
                        store32(p.h + to, v);
                        store32(p.dg + to, v);
                        store32(p.du + to, v);
                    } else if (in < (u.rows + kPad - 1) / kPad * kPad) {
                        backward_zeros(p, to);
                        backward_zeros(p, to + 16);
                    }
                } else {
                    uint32_t rows;
                    uint16_t *out = unit_out<EPI>(p, u, rows);
                    for (uint32_t k = col0 + c; in < rows && k < min(col0 + c + 32, q.n) && !(none && p.accumulate); ++k)
                        st_value<DT_BF16>(out, (uint64_t)in * q.n + k, none ? 0.0f : nan);
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
    cluster_sync();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    if (warp == 2)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

// ------------------------------------------------------------------ few rows an expert

// One finished sum of a token (row of the call) and a column, a lane a column:
// v, and for EPI_GATED g = v and u = w, whose block of 32 columns is the warp.
// All lanes call; `in` says whether the column exists (EPI_GATED: in rows of ldh).
template <int EPI> __device__ __forceinline__ void finish_lane(const ExpertParams &p, uint32_t row, uint32_t col, bool in, float v, float w)
{
    if (EPI == EPI_GATED) {
        const uint64_t at = (uint64_t)row * p.ldh + col;
        if (p.codes[0]) {
            const float x[2] = {v, w};
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const uint32_t b = act8_byte(__reduce_max_sync(0xffffffffu, __float_as_uint(x[k]) & 0x7fffffffu));
                if (in) {
                    gstore<int8_t>(p.codes[k] + at, b == kActNan ? (int8_t)0 : (int8_t)(act8_code(act8_clamp(x[k]), act8_inverse(b)) & 0xff));
                    if (col % kActBlock == 0)
                        gstore<uint8_t>(p.scales[k] + at / kActBlock, (uint8_t)b);
                }
            }
        }
        float a, da;
        gate(p.act, v, a, da);
        if (in)
            st_value<DT_BF16>(p.h, at, __fmul_rn(a, w));
    } else if (in) {
        st_value<DT_BF16>(p.prob[0].out, (uint64_t)row * p.prob[0].n + col, v);
    }
}

// Units of expert_few_kernel: a tile of npad tokens, two blocks of 128 weight
// rows (EPI_GATED: the same of gate and up), a part of K.
template <int EPI> __device__ __forceinline__ Unit few_unit_at(const ExpertParams &p, const Table &tb, uint32_t i, uint32_t &kb0)
{
    Unit u;
    const Problem &q = p.prob[0];
    u.prob = 0;
    u.split = i % p.splits;
    i /= p.splits;
    const uint32_t t = q.by_nt(i);
    u.n = i - t * q.nt;
    u.expert = expert_at(tb.tile0, p.experts, (int32_t)t);
    u.m = t - (uint32_t)tb.tile0[u.expert];
    u.row0 = (uint32_t)tb.row0[u.expert] + u.m * p.npad;
    u.rows = min((uint32_t)tb.row0[u.expert + 1] - u.row0, p.npad); // of the tile
    u.pad0 = 0;
    kb0 = (uint32_t)((uint64_t)q.kblocks * u.split / p.splits);
    u.kblocks = (uint32_t)((uint64_t)q.kblocks * (u.split + 1) / p.splits) - kb0;
    return u;
}

// A CTA by itself: the roles of expert_gemm_kernel, 128 weight rows an
// accumulator.  Bound by reading the weights, each once for a tile of tokens: one
// token by two experts of 4096 x 11008 61 us for g and u and 37 for y (5.9 and 4.9
// TB/s).
template <int EPI> __global__ void __launch_bounds__(kFewThreads, 1) expert_few_kernel(const __grid_constant__ ExpertParams p)
{
    extern __shared__ uint8_t raw[];
    __shared__ uint64_t bars[2 * kFewStages + 4];
    __shared__ uint32_t tmem_slot;
    __shared__ volatile int gave_up;
    const Problem &q = p.prob[0];
    const uint32_t stages = (smem_u32(raw) + 1023) & ~1023u;
    const uint32_t stage_bytes = 2 * kOperandBytes + p.npad * 128;
    uint8_t *behind = raw + (stages - smem_u32(raw)) + p.stages * stage_bytes;
    const Table table{reinterpret_cast<int32_t *>(behind), reinterpret_cast<int32_t *>(behind) + CCL_MAX_EXPERTS + 2,
                      reinterpret_cast<int32_t *>(behind) + 2 * (CCL_MAX_EXPERTS + 2)};
    const uint32_t full = smem_u32(&bars[0]), empty = smem_u32(&bars[kFewStages]);
    const uint32_t acc_full = smem_u32(&bars[2 * kFewStages]), acc_empty = smem_u32(&bars[2 * kFewStages + 2]);
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kFewStages; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(acc_full + 8 * i, 1);
            mbar_init(acc_empty + 8 * i, kEpiWarps);
        }
        if ((gave_up = p.wait_ns == 0))
            atomicAdd(&g_expert_timeouts, 1ull);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 3 && lane < 2)
        prefetch_map(lane ? &q.b[0] : &q.a[0]);
    if (warp == 3 && lane == 2 && EPI == EPI_GATED)
        prefetch_map(&q.a[1]);
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
    make_table(p, table, p.npad);
    const uint32_t total = (uint32_t)table.tile0[p.experts] * q.nt * p.splits;

    if (warp == 0 && lane == 0) {
        uint32_t s = 0, phase = 0;
        bool ok = p.wait_ns != 0;
        // a: the weights (EPI_GATED: of gate and up); b: the tokens
        auto load_a = [&](const Unit &u, uint32_t kb, uint32_t stage) {
            mbar_expect(full + 8 * stage, stage_bytes);
            const uint32_t at = stages + stage * stage_bytes;
            const int k = (int)(kb * kTileK), r0 = EPI == EPI_GATED ? (int)(u.n * 128) : (int)(u.n * 256);
            tma_load3_own(at, &q.a[0], k, r0, (int)u.expert, full + 8 * stage);
            tma_load3_own(at + kOperandBytes, EPI == EPI_GATED ? &q.a[1] : &q.a[0], k, EPI == EPI_GATED ? r0 : r0 + 128, (int)u.expert, full + 8 * stage);
        };
        auto load_b = [&](const Unit &u, uint32_t kb, uint32_t stage) {
            tma_load_own(stages + stage * stage_bytes + 2 * kOperandBytes, &q.b[0], (int)(kb * kTileK), (int)u.row0, full + 8 * stage);
        };
        // the first stages' weights before the tokens' values are ready
        uint32_t ahead = 0, kb0;
        if (p.early) {
            if (ok && blockIdx.x < total) {
                const Unit u = few_unit_at<EPI>(p, table, blockIdx.x, kb0);
                ahead = min(p.stages, u.kblocks);
                for (uint32_t i = 0; i < ahead; ++i)
                    load_a(u, kb0 + i, i);
            }
            chain_entry();
        }
        auto next = [&] {
            if (++s == p.stages) {
                s = 0;
                phase ^= 1;
            }
        };
        for (uint32_t i = blockIdx.x; ok && i < total; i += gridDim.x) {
            const Unit u = few_unit_at<EPI>(p, table, i, kb0);
            for (uint32_t kb = kb0; kb < kb0 + u.kblocks; ++kb) {
                if (ahead) {
                    --ahead; // the ring's first round: this stage is free and its weights are on the way
                } else {
                    if (!(ok = mbar_wait(empty + 8 * s, phase ^ 1, &gave_up, p.wait_ns)))
                        break;
                    load_a(u, kb, s);
                }
                load_b(u, kb, s);
                next();
            }
        }
        // the issuer's last arrivals come while the CTA is here
        for (uint32_t i = 0; ok && i < p.stages; ++i) {
            ok = mbar_wait(empty + 8 * s, phase ^ 1, &gave_up, p.wait_ns);
            next();
        }
    } else if (warp == 1 && lane == 0) {
        uint32_t s = 0, phase = 0, t = 0, kb0;
        bool ok = p.wait_ns != 0;
        for (uint32_t i = blockIdx.x; ok && i < total; i += gridDim.x, ++t) {
            const Unit u = few_unit_at<EPI>(p, table, i, kb0);
            const uint32_t idesc = 1u << 4 | 1u << 7 | 1u << 10 | ((u.rows + 15) / 16 * 16 >> 3) << 17 | (128u >> 4) << 24;
            const uint32_t buf = t & 1;
            if (!(ok = mbar_wait(acc_empty + 8 * buf, ((t >> 1) & 1) ^ 1, &gave_up, p.wait_ns)))
                break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            for (uint32_t kb = 0; kb < u.kblocks; ++kb) {
                if (!(ok = mbar_wait(full + 8 * s, phase, &gave_up, p.wait_ns)))
                    break;
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                const uint32_t at = stages + s * stage_bytes;
#pragma unroll
                for (int k = 0; k < kTileK / 16; ++k)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        tc_mma_own(tmem + (buf * 2 + j) * p.npad, operand_desc<false>(at + j * kOperandBytes + k * k_step<false>()),
                                   operand_desc<false>(at + 2 * kOperandBytes + k * k_step<false>()), idesc, kb > 0 || k > 0);
                tc_commit_own(empty + 8 * s);
                if (++s == p.stages) {
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
        const uint64_t width = (uint64_t)q.nt * kTileN, cols = EPI == EPI_GATED ? p.ldh : q.n;
        uint32_t t = 0, i = blockIdx.x, kb0;
        for (; p.wait_ns && i < total; i += gridDim.x, ++t) {
            const Unit u = few_unit_at<EPI>(p, table, i, kb0);
            const uint32_t buf = t & 1;
            if (!__all_sync(0xffffffffu, mbar_wait(acc_full + 8 * buf, (t >> 1) & 1, &gave_up, p.wait_ns)))
                break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            const uint32_t acc = tmem + buf * 2 * p.npad + (lanes << 16);
            const uint32_t col = (EPI == EPI_GATED ? u.n * 128 : u.n * 256 + half * 128) + lanes + lane;
            for (uint32_t c = EPI == EPI_GATED ? half * 16 : 0; c < u.rows; c += EPI == EPI_GATED ? 32 : 16) {
                float v[16], w[16];
                tc_load16(acc + (EPI == EPI_GATED ? 0 : half * p.npad) + c, v);
                if (EPI == EPI_GATED)
                    tc_load16(acc + p.npad + c, w);
                const uint32_t rows = min(16u, u.rows - c); // tokens of these columns
                if (p.splits > 1) {
                    float *out = p.partial + ((uint64_t)u.split * p.rows + u.row0 + c) * width + u.n * kTileN + (EPI == EPI_GATED ? 0 : half * 128) + lanes + lane;
#pragma unroll
                    for (uint32_t j = 0; j < 16; ++j, out += width)
                        if (j < rows) {
                            gstore<float>(out, v[j]);
                            if (EPI == EPI_GATED)
                                gstore<float>(out + 128, w[j]);
                        }
                } else {
#pragma unroll
                    for (uint32_t j = 0; j < 16; ++j)
                        if (j < rows)
                            finish_lane<EPI>(p, u.row0 + c + j, col, col < cols, v[j], EPI == EPI_GATED ? w[j] : 0.0f);
                }
            }
            asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
            __syncwarp();
            if (lane == 0)
                mbar_arrive(acc_empty + 8 * buf);
        }
        const float nan = __uint_as_float(kNanBits);
        for (; i < total; i += gridDim.x) { // after a wait that gave up
            const Unit u = few_unit_at<EPI>(p, table, i, kb0);
            const uint32_t c0 = (EPI == EPI_GATED ? 0 : half * 128) + lanes + lane, col = u.n * (EPI == EPI_GATED ? 128 : 256) + c0;
            for (uint32_t r = 0; r < u.rows; ++r) {
                if (EPI == EPI_GATED && (r / 16 & 1) != half)
                    continue; // the other half's token
                if (p.splits > 1) {
                    float *out = p.partial + ((uint64_t)u.split * p.rows + u.row0 + r) * width + u.n * kTileN + c0;
                    gstore<float>(out, nan);
                    if (EPI == EPI_GATED)
                        gstore<float>(out + 128, nan);
                } else {
                    finish_lane<EPI>(p, u.row0 + r, col, col < cols, nan, nan);
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

// The splits' sums, added in order, a column a lane; bound by its launch (one
// token, 11008 columns of g and u: 6 us with a cold cache).
template <int EPI> __global__ void __launch_bounds__(256) expert_join_kernel(const __grid_constant__ ExpertParams p)
{
    chain_entry();
    // the rows that some expert has: from the first offset to the largest
    __shared__ int32_t tops[8];
    int32_t top = 0;
    for (uint32_t e = threadIdx.x; e <= p.experts; e += 256)
        top = max(top, min(load_offset(p.offsets + e), (int32_t)p.rows));
    top = __reduce_max_sync(0xffffffffu, top);
    if ((threadIdx.x & 31) == 0)
        tops[threadIdx.x >> 5] = top;
    __syncthreads();
    for (int i = 0; i < 8; ++i)
        top = max(top, tops[i]);
    const uint32_t first = (uint32_t)min(max(load_offset(p.offsets), 0), (int32_t)p.rows);
    const Problem &q = p.prob[0];
    const uint64_t width = (uint64_t)q.nt * kTileN, slab = (uint64_t)p.rows * width;
    const uint32_t cols = EPI == EPI_GATED ? p.ldh : q.n, blocks = (cols + 255) / 256; // of 256 columns
    const uint64_t all = (uint64_t)((uint32_t)top - min(first, (uint32_t)top)) * blocks;
    for (uint64_t i = blockIdx.x; i < all; i += gridDim.x) {
        const uint32_t row = first + (uint32_t)(i / blocks), col = (uint32_t)(i % blocks) * 256 + threadIdx.x;
        if ((col & ~31u) >= cols)
            continue; // the whole warp
        // EPI_GATED: 128 columns of g, then the same of u, in each tile
        const float *at = p.partial + row * width + (EPI == EPI_GATED ? col / 128 * 256 + col % 128 : col);
        float v = 0.0f, w = 0.0f, f[4], h[4];
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
        finish_lane<EPI>(p, row, col, col < cols, v, w);
    }
}

// ------------------------------------------------------------------ the padded layout

struct PadParams {
    ExpertParams p; // offsets, experts, rows
    struct {
        const uint16_t *src;   // rows of `cols`, or NULL:
        const int8_t *codes;   // rows of `width`
        const uint8_t *scales;
        uint16_t *dst; // rows of ld
        int tails;     // only the last, partial block of 64 rows of each expert
    } m[2];
    uint32_t nrows; // matrices of rows (m); then those of `weights`
    uint32_t cols, ld, width;
    int vector; // src: 16-byte aligned rows of whole vectors
    PackParams weights;
};

// Every expert's rows at their place in the padded layout and zeros behind them,
// a warp a row; in the same launch the weights that TMA cannot address, to rows
// of a padded stride.  blockIdx.y is the matrix.  32768 rows of 2048 from their 8
// bits: 50 us, 4 TB/s (two blocks in flight a lane took as long).
__global__ void __launch_bounds__(256) expert_pad_kernel(const __grid_constant__ PadParams q)
{
    chain_entry();
    __shared__ int32_t tables[3 * (CCL_MAX_EXPERTS + 2)];
    if (blockIdx.y >= q.nrows) {
        pack_operand(q.weights, blockIdx.y - q.nrows);
        return;
    }
    const ExpertParams &p = q.p;
    const Table t{tables, tables + CCL_MAX_EXPERTS + 2, tables + 2 * (CCL_MAX_EXPERTS + 2)};
    make_table(p, t, kTileM);
    const auto &m = q.m[blockIdx.y];
    const uint32_t lane = threadIdx.x & 31, total = m.tails ? p.experts * kPad : (uint32_t)t.pad0[p.experts];
    for (uint32_t i = blockIdx.x * 8 + (threadIdx.x >> 5); i < total; i += gridDim.x * 8) {
        uint32_t e, in; // row `in` of expert e
        if (m.tails) {
            e = i / kPad;
            const uint32_t n = (uint32_t)(t.row0[e + 1] - t.row0[e]);
            if (n % kPad == 0)
                continue;
            in = n / kPad * kPad + i % kPad;
        } else {
            e = expert_at(t.pad0, p.experts, (int32_t)i);
            in = i - (uint32_t)t.pad0[e];
        }
        const uint32_t r = (uint32_t)t.pad0[e] + in, row = (uint32_t)t.row0[e] + in;
        const bool has = row < (uint32_t)t.row0[e + 1];
        uint16_t *dst = m.dst + (uint64_t)r * q.ld;
        if (!has) {
            for (uint32_t c = lane * 8; c < q.ld; c += 256)
                st16(dst + c, make_uint4(0, 0, 0, 0));
        } else if (!m.src) {
            for (uint32_t c = lane * 32; c < q.ld; c += 1024) {
                uint4 lo, hi;
                float f[32];
                const uint64_t at = (uint64_t)row * q.width + c;
                ld32(m.codes + at, lo, hi);
                act8_decode(lo, hi, act8_step(gload<uint8_t>(m.scales + at / kActBlock)), f);
#pragma unroll
                for (int j = 0; j < 32; j += 8)
                    if (c + j < q.ld)
                        st16(dst + c + j, pack<DT_BF16>(f + j));
            }
        } else if (q.vector) {
            const uint16_t *src = m.src + (uint64_t)row * q.cols;
            for (uint32_t c0 = lane * 8; c0 < q.ld; c0 += 4 * 256) {
                uint4 v[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (c0 + j * 256 < q.ld)
                        v[j] = ld16(src + c0 + j * 256);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (c0 + j * 256 < q.ld)
                        st16(dst + c0 + j * 256, v[j]);
            }
        } else {
            const uint16_t *src = m.src + (uint64_t)row * q.cols;
            for (uint32_t c0 = lane; c0 < q.ld; c0 += 4 * 32) {
                uint16_t v[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    v[j] = c0 + j * 32 < q.cols ? gload<uint16_t>(src + c0 + j * 32) : (uint16_t)0;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (c0 + j * 32 < q.ld)
                        gstore<uint16_t>(dst + c0 + j * 32, v[j]);
            }
        }
    }
}

// ------------------------------------------------------------------ host side

// A map of rows (as in ffn.cu), and one with the expert as third dimension.
bool encode_rows(CUtensorMap *map, const Matrix &m, bool mn, uint32_t box_rows = 128)
{
    const cuuint64_t dim[2] = {m.cols, m.rows}, stride[1] = {m.ld * 2};
    const cuuint32_t box[2] = {64, mn ? 64u : box_rows}, step[2] = {1, 1};
    return encode_fn() &&
           encode_fn()(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(m.ptr), dim, stride, box, step,
                       CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool encode_experts(CUtensorMap *map, const Matrix &m, uint64_t experts, bool mn)
{
    const uint64_t rows = m.rows / experts; // of one expert
    const cuuint64_t dim[3] = {m.cols, rows, experts}, stride[2] = {m.ld * 2, rows * m.ld * 2};
    const cuuint32_t box[3] = {64, mn ? 64u : 128u, 1}, step[3] = {1, 1, 1};
    return encode_fn() &&
           encode_fn()(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(m.ptr), dim, stride, box, step,
                       CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

uint32_t tiles_of(uint64_t n, uint32_t t) { return (uint32_t)((n + t - 1) / t); }

constexpr uint64_t kMaxRows = 0x7fff0000, kMaxWidth = 1 << 24;
constexpr uint32_t kMaxSplits = 16;
// Rows an expert, on average, up to which a forward pass has the weights as the
// accumulator's rows (expert_few_kernel).  Forward in us, so and on pairs: eight
// experts of 4096 x 11008 with 16 rows each 333 and 362, with 64 372 and 371, with
// 96 459 and 392; one of 4096 x 4096 with 64 36.5 and 47.4; three of 2048 x 2816
// with 32 34.5 and 35.1; 32 of 512 x 1376 with 16 37.8 and 35.4, with 64 47.6 and
// 36.8.
constexpr uint64_t kFewRows = 64;

// Parts that the sum over K is cut into, in expert_few_kernel: as ffn.cu's rule,
// the number that minimises the rounds of CTAs (each as long as a part's weights
// take) and the join; tiles: those of the experts that can have rows.  One token
// by two experts of 4096 x 11008 94 us, without cuts 154; 64 rows over four of
// 2048 x 2816 39.0 and 45.5.
// The parts' sums have to fit into `room` bytes.
uint32_t choose_splits(uint64_t tiles, uint64_t kblocks, uint64_t partial_bytes, size_t room)
{
    uint32_t best = 1;
    double cost = 0;
    for (uint32_t s = 1; s <= kMaxSplits && s <= kblocks && (s == 1 || s * partial_bytes <= room); ++s) {
        const double rounds = (double)((tiles * s + kSms - 1) / kSms);
        const double block = std::max(0.5, 0.005 * (double)std::min<uint64_t>(kSms, tiles * s));
        const double products = (double)kblocks / s * block;
        const double c = rounds * std::max(products, 0.5) + std::min(products, 0.5) + (s > 1 ? 3.0 + 2.0 * s * (double)partial_bytes / 6e6 : 0.0);
        if (s == 1 || c < cost * 0.97) {
            best = s;
            cost = c;
        }
    }
    return best;
}

struct ExpertPlan {
    uint64_t r, rp, dp, fp, fw; // rows, padded rows; widths to 8, and of the codes
    bool few;
    uint32_t npad, up_splits, down_splits;
    // offsets into the work buffer
    size_t h, dg, du, x, y, wg, wu, wd, partial, bytes;
};

// room: the bytes that there are.  The sums over K are the only part of the buffer
// that fewer bytes can do with: fewer rows have more parts, and a buffer that was
// planned for a larger batch serves them with the parts that fit.
bool make_plan(size_t r, size_t e, size_t d, size_t f, bool backward, bool aligned, size_t room, ExpertPlan *p)
{
    if (r > kMaxRows || e > CCL_MAX_EXPERTS || d > kMaxWidth || f > kMaxWidth || r * std::max(d, f) > (1ull << 44) ||
        (uint64_t)d * f > (1ull << 38) /* an expert's stride in its tensor map */ || (uint64_t)e * d * f > (1ull << 44))
        return false;
    const uint64_t pads = r + (kPad - 1) * std::min(r, e);
    if (pads > kMaxRows) // rows are 32-bit
        return false;
    *p = ExpertPlan{};
    p->r = r;
    p->rp = (pads + kPad - 1) / kPad * kPad;
    p->dp = (d + 7) / 8 * 8;
    p->fp = (f + 7) / 8 * 8;
    p->fw = (f + kActBlock - 1) / kActBlock * kActBlock;
    const bool pd = p->dp != d || !aligned, pf = p->fp != f || !aligned;
    const uint64_t active = std::min(r, e);
    // units are counted in 32 bits
    const uint64_t most = ((r + kTileM - 1) / kTileM + active) * std::max(tiles_of(f, 32), tiles_of(d, 64));
    const uint64_t weights = (uint64_t)e * 3 * (tiles_of(f, 64) + 1) * (tiles_of(d, 64) + 1);
    if (most > 0x3fffffff || weights > 0x3fffffff)
        return false;
    p->few = !backward && e && r <= kFewRows * e;
    size_t at = 0;
    auto take = [&](size_t n) {
        const size_t o = at;
        at += up(n);
        return o;
    };
    const uint64_t rows = backward ? p->rp : r;
    p->h = take(rows * p->fw * 2);
    if (backward) {
        p->dg = take(rows * p->fw * 2);
        p->du = take(rows * p->fw * 2);
        p->x = take(rows * p->dp * 2);
        p->y = take(rows * p->dp * 2);
    } else if (pd) {
        p->x = take(r * p->dp * 2);
    }
    if (pd) {
        p->wg = take(e * f * p->dp * 2);
        p->wu = take(e * f * p->dp * 2);
    }
    if (pf)
        p->wd = take(e * d * p->fp * 2);
    if (p->few) {
        // tokens a tile: four times the mean, since experts are not chosen evenly
        // (64 tokens, four of 16 experts of 2048 x 2816: 102.1 us, the mean 126.1,
        // eight times it 102.5)
        const uint64_t mean = (r + e - 1) / e;
        p->npad = (uint32_t)std::min<uint64_t>({kFewMost, (r + 15) / 16 * 16, std::max<uint64_t>(16, (4 * mean + 15) / 16 * 16)});
        p->npad = std::max(p->npad, 16u);
        const uint64_t tiles = std::max<uint64_t>(active, r / p->npad);
        const size_t up_bytes = r * (size_t)tiles_of(f, 128) * kTileN * 4, down_bytes = r * (size_t)tiles_of(d, kTileN) * kTileN * 4;
        room = room > at ? (room - at) / kAlign * kAlign : 0;
        p->up_splits = choose_splits(tiles * tiles_of(f, 128), tiles_of(d, kTileK), up_bytes, room);
        p->down_splits = choose_splits(tiles * tiles_of(d, kTileN), tiles_of(f, kTileK), down_bytes, room);
        p->partial = take(std::max(p->up_splits > 1 ? p->up_splits * up_bytes : 0, p->down_splits > 1 ? p->down_splits * down_bytes : 0));
    }
    p->bytes = at;
    return true;
}

cudaLaunchConfig_t pair_launch(cudaLaunchAttribute *attr, unsigned pairs, unsigned threads, bool chained, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * pairs);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = kGemmSmem;
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = chained ? 2 : 1;
    return cfg;
}

// units: the most that the launch can have.
template <int EPI, bool A_MN, bool B_MN, bool STAGED = false> cudaError_t launch_gemm(const ExpertParams &p, uint64_t units, cudaStream_t stream)
{
    static std::atomic<unsigned long long> ready{0};
    cudaError_t e = large_smem_once(reinterpret_cast<const void *>(expert_gemm_kernel<EPI, A_MN, B_MN, STAGED>), kGemmSmem, ready);
    if (e != cudaSuccess)
        return e;
    cudaLaunchAttribute attr[2];
    const cudaLaunchConfig_t cfg = pair_launch(attr, (unsigned)std::max<uint64_t>(1, std::min<uint64_t>(units, kPairs)), kThreadsOf<EPI>, !STAGED, stream);
    if ((e = cudaLaunchKernelEx(&cfg, expert_gemm_kernel<EPI, A_MN, B_MN, STAGED>, p)) == cudaSuccess)
        count_launches(1);
    return e;
}

// Outputs whose every row is 16-byte aligned and whole vectors of 8 columns are
// written directly.
template <int EPI, bool A_MN, bool B_MN> cudaError_t launch_out(const ExpertParams &p, bool vectors, uint64_t units, cudaStream_t stream)
{
    return vectors ? launch_gemm<EPI, A_MN, B_MN, false>(p, units, stream) : launch_gemm<EPI, A_MN, B_MN, true>(p, units, stream);
}

template <int EPI> cudaError_t launch_few(ExpertParams &p, uint64_t tiles, cudaStream_t stream)
{
    static std::atomic<unsigned long long> ready{0};
    constexpr int smem = kFewBytes + 1024 + kTableBytes;
    cudaError_t e = large_smem_once(reinterpret_cast<const void *>(expert_few_kernel<EPI>), smem, ready);
    if (e != cudaSuccess)
        return e;
    p.stages = std::min<uint32_t>(kFewStages, kFewBytes / (2 * kOperandBytes + p.npad * 128));
    const uint64_t units = tiles * p.prob[0].nt * p.splits;
    if (units > 0x3fffffff)
        return cudaErrorInvalidValue;
    if ((e = launch_chained(expert_few_kernel<EPI>, dim3((unsigned)std::min<uint64_t>(units, kSms)), dim3(kFewThreads), smem, stream, p)) != cudaSuccess)
        return e;
    count_launches(1);
    if (p.splits > 1) {
        const uint64_t blocks = (uint64_t)p.rows * (((EPI == EPI_GATED ? p.ldh : p.prob[0].n) + 255) / 256);
        if ((e = launch_chained(expert_join_kernel<EPI>, dim3((unsigned)std::min<uint64_t>(blocks, 8 * kSms)), dim3(256), 0, stream, p)) == cudaSuccess)
            count_launches(1);
    }
    return e;
}

struct ExpertArgs {
    const void *x;
    const int8_t *x_codes;
    const uint8_t *x_scales;
    const int32_t *offsets;
    const void *wg, *wu, *wd;
    int8_t *codes;
    uint8_t *scales;
    size_t r, e, d, f;
    ccl_dtype_t dtype;
    ccl_act_t act;
    void *work;
    size_t work_bytes;
};

bool all_aligned(std::initializer_list<const void *> ps)
{
    for (const void *p : ps)
        if ((uintptr_t)p % 16)
            return false;
    return true;
}

// The checks that both directions share; on CCL_OK `plan` is ready.
ccl_status_t check_experts(const ExpertArgs &a, bool backward, bool aligned, ExpertPlan *plan)
{
    if (!valid_dtype(a.dtype) || (a.act != CCL_ACT_SILU && a.act != CCL_ACT_GELU_TANH))
        return CCL_ERR_INVALID_ARG;
    if (a.dtype != CCL_BF16)
        return CCL_ERR_UNSUPPORTED;
    if (a.f == 0 || !make_plan(a.r, a.e, a.d, a.f, backward, aligned, a.work_bytes, plan))
        return CCL_ERR_INVALID_ARG;
    return CCL_OK;
}

ccl_status_t dbg_ranges(const std::vector<Range> &w, const std::vector<Range> &r, cudaStream_t stream)
{
#ifdef CCL_DEBUG_BOUNDS
    std::vector<DbgRange> v;
    for (const std::vector<Range> *s : {&w, &r})
        for (const Range &x : *s)
            v.push_back(DbgRange{reinterpret_cast<const void *>(x.lo), (size_t)(x.hi - x.lo)});
    return from_cuda(dbg_set_ranges(v, stream));
#else
    (void)w, (void)r, (void)stream;
    return CCL_OK;
#endif
}

ExpertParams params_of(const ExpertArgs &a, const ExpertPlan &pl)
{
    ExpertParams p{};
    p.nprob = 1;
    p.offsets = a.offsets;
    p.experts = (uint32_t)a.e;
    p.rows = (uint32_t)a.r;
    p.act = (int)a.act;
    p.ldh = (uint32_t)pl.fw;
    p.wait_ns = feed_forward_wait_ns();
    p.splits = 1;
    if (a.codes) {
        p.codes[0] = a.codes;
        p.codes[1] = a.codes + a.r * pl.fw;
        p.scales[0] = a.scales;
        p.scales[1] = a.scales + a.r * (pl.fw / kActBlock);
    }
    char *work = static_cast<char *>(a.work);
    p.h = reinterpret_cast<uint16_t *>(work + pl.h);
    p.dg = reinterpret_cast<uint16_t *>(work + pl.dg);
    p.du = reinterpret_cast<uint16_t *>(work + pl.du);
    p.partial = reinterpret_cast<float *>(work + pl.partial);
    p.npad = pl.npad;
    return p;
}

// Half the columns of a pair's tile: 128, whose products reuse what they read
// most, or fewer where that shortens the rounds of tiles (row tiles x columns).
// A block of K takes a pair about 0.35 us, and little less at half and quarter
// width; an epilogue, which runs beside the next tile's products, `epilogue` us
// at full width.  Backward of 300 rows over five experts of 1000 x 736: 39.6 us,
// with full tiles 43.4.
uint32_t half_tile(uint64_t row_tiles, uint64_t columns, uint64_t kblocks, double epilogue)
{
    uint32_t best = 128;
    double cost = 0;
    for (uint32_t half = 128; half >= 32; half /= 2) {
        const double rounds = (double)((row_tiles * ((columns + 2 * half - 1) / (2 * half)) + kPairs - 1) / kPairs);
        const double products = (double)kblocks * (half == 128 ? 0.35 : half == 64 ? 0.33 : 0.31), after = 0.7 + epilogue * half / 128;
        const double c = rounds * std::max(products, after) + std::min(products, after);
        if (half == 128 || c < cost * 0.95) {
            best = half;
            cost = c;
        }
    }
    return best;
}

void set_problem(Problem &q, uint64_t n, uint32_t tile, uint64_t k, uint32_t segs)
{
    q.n = (uint32_t)n;
    q.nt = tiles_of(n, tile);
    q.by_nt = divisor(q.nt);
    q.by_group = divisor(kGroupM * q.nt);
    q.kblocks = tiles_of(k, kTileK);
    q.segs = segs;
}

ccl_status_t expert_ffn_impl(const ExpertArgs &a, void *out, cudaStream_t stream)
{
    ExpertPlan pl;
    if (ccl_status_t st = check_experts(a, false, all_aligned({a.x, a.wg, a.wu, a.wd}), &pl))
        return st;
    if (a.r == 0 || a.e == 0 || a.d == 0)
        return CCL_OK;
    const uint64_t saved = 2 * a.r * pl.fw;
    if (!a.x || !out || !a.offsets || !a.wg || !a.wu || !a.wd || !a.codes != !a.scales || !element_aligned(2, {a.x, a.wg, a.wu, a.wd, out}) ||
        !element_aligned(4, {a.offsets}) || !element_aligned(32, {a.codes}) || !a.work || (uintptr_t)a.work % 256 || a.work_bytes < pl.bytes)
        return CCL_ERR_INVALID_ARG;
    const size_t wb = a.e * a.f * a.d * 2;
    const std::vector<Range> w{range_of(out, a.r * a.d * 2, 0), range_of(a.work, pl.bytes, 0), range_of(a.codes, a.codes ? saved : 0, 0),
                               range_of(a.scales, a.codes ? saved / kActBlock : 0, 0)},
        r{range_of(a.x, a.r * a.d * 2, 0), range_of(a.wg, wb, 0), range_of(a.wu, wb, 0), range_of(a.wd, wb, 0), range_of(a.offsets, (a.e + 1) * 4, 0)};
    if (ccl_status_t st = check_overlaps(w, r, [](const Range &, const Range &) { return false; }))
        return st;
    if (ccl_status_t st = dbg_ranges(w, r, stream))
        return st;
    char *work = static_cast<char *>(a.work);
    Operands ops(work);
    const Matrix x = ops.add(a.x, a.r, a.d, pl.x), wd = ops.add(a.wd, a.e * a.d, a.f, pl.wd);
    const Matrix w2[2] = {ops.add(a.wg, a.e * a.f, a.d, pl.wg), ops.add(a.wu, a.e * a.f, a.d, pl.wu)};
    const Matrix h{work + pl.h, a.r, a.f, pl.fw};
    if (cudaError_t e = ops.copy(stream))
        return from_cuda(e);
    ExpertParams p = params_of(a, pl);
    Problem &q = p.prob[0];
    const uint64_t active = std::min<uint64_t>(a.r, a.e);
    if (pl.few) {
        const uint64_t tiles = a.r / pl.npad + active; // at most
        set_problem(q, a.f, 128, a.d, 1);
        p.splits = pl.up_splits;
        if (!encode_experts(&q.a[0], w2[0], a.e, false) || !encode_experts(&q.a[1], w2[1], a.e, false) || !encode_rows(&q.b[0], x, false, p.npad))
            return CCL_ERR_CUDA;
        if (cudaError_t e = launch_few<EPI_GATED>(p, tiles, stream))
            return from_cuda(e);
        set_problem(q, a.d, kTileN, a.f, 1);
        q.out = out;
        p.splits = pl.down_splits;
        p.early = wd.ptr == a.wd; // not a copy made within this call
        if (!encode_experts(&q.a[0], wd, a.e, false) || !encode_rows(&q.b[0], h, false, p.npad))
            return CCL_ERR_CUDA;
        return from_cuda(launch_few<EPI_STORE>(p, tiles, stream));
    }
    const uint64_t tiles = a.r / kTileM + active; // at most
    const uint64_t likely = std::max(active, a.r / kTileM + active / 2);
    p.half = half_tile(likely, 2 * a.f, tiles_of(a.d, kTileK), a.codes ? 5.0 : 3.5);
    set_problem(q, a.f, p.half, a.d, 1);
    if (!encode_rows(&q.a[0], x, false) || !encode_experts(&q.b[0], w2[0], a.e, false) || !encode_experts(&q.b[1], w2[1], a.e, false))
        return CCL_ERR_CUDA;
    if (cudaError_t e = launch_gemm<EPI_GATED, false, false>(p, tiles * q.nt, stream))
        return from_cuda(e);
    const bool vectors = a.d % 8 == 0 && (uintptr_t)out % 16 == 0;
    p.half = half_tile(likely, a.d, tiles_of(a.f, kTileK), vectors ? 2.5 : 4.0);
    set_problem(q, a.d, 2 * p.half, a.f, 1);
    q.out = out;
    if (!encode_rows(&q.a[0], h, false) || !encode_experts(&q.b[0], wd, a.e, false))
        return CCL_ERR_CUDA;
    return from_cuda(launch_out<EPI_STORE, false, false>(p, vectors, tiles * q.nt, stream));
}

ccl_status_t expert_ffn_grad_impl(const ExpertArgs &a, const void *dy, void *dx, void *dwg, void *dwu, void *dwd, int accumulate, cudaStream_t stream)
{
    ExpertPlan pl;
    if (ccl_status_t st = check_experts(a, true, all_aligned({a.wg, a.wu, a.wd}), &pl))
        return st;
    if (a.d == 0 || a.e == 0 || (!dx && !dwg && !dwu && !dwd))
        return CCL_OK;
    const size_t rb = a.r * a.d * 2, wb = a.e * a.f * a.d * 2;
    const uint64_t saved = 2 * a.r * pl.fw, xw = (a.d + kActBlock - 1) / kActBlock * kActBlock;
    const bool need_x = dwg || dwu, eight = !a.x;
    if ((a.r && (!a.offsets || !dy || (need_x && eight && (!a.x_codes || !a.x_scales)) || !a.wg || !a.wu || !a.wd || !a.codes || !a.scales)) ||
        !element_aligned(2, {a.x, a.wg, a.wu, a.wd, dy, dx, dwg, dwu, dwd}) || !element_aligned(4, {a.offsets}) ||
        !element_aligned(32, {a.codes, a.x_codes}))
        return CCL_ERR_INVALID_ARG;
    const bool empty = a.r == 0;
    if (!empty && (!a.work || (uintptr_t)a.work % 256 || a.work_bytes < pl.bytes))
        return CCL_ERR_INVALID_ARG;
    std::vector<Range> w, r;
    if (!empty) {
        w.push_back(range_of(a.work, pl.bytes, 0));
        r = {range_of(dy, rb, 0), range_of(a.wg, wb, 0), range_of(a.wu, wb, 0), range_of(a.wd, wb, 0), range_of(a.codes, saved, 0),
             range_of(a.scales, saved / kActBlock, 0), range_of(a.offsets, (a.e + 1) * 4, 0)};
        if (need_x && !eight)
            r.push_back(range_of(a.x, rb, 0));
        if (need_x && eight) {
            r.push_back(range_of(a.x_codes, a.r * xw, 0));
            r.push_back(range_of(a.x_scales, a.r * (xw / kActBlock), 0));
        }
    }
    if (dx)
        w.push_back(range_of(dx, rb, 0));
    for (void *g : {dwg, dwu, dwd})
        if (g)
            w.push_back(range_of(g, wb, 0));
    if (ccl_status_t st = check_overlaps(w, r, [](const Range &, const Range &) { return false; }))
        return st;
    cudaError_t e;
    if (empty) { // empty sums
        for (void *g : {dwg, dwu, dwd})
            if (g && wb && !accumulate && (e = cudaMemsetAsync(g, 0, wb, stream)))
                return from_cuda(e);
        return CCL_OK;
    }
    if (ccl_status_t st = dbg_ranges(w, r, stream))
        return st;
    char *work = static_cast<char *>(a.work);
    Operands ops(work);
    const Matrix wd = ops.add(a.wd, a.e * a.d, a.f, pl.wd);
    const Matrix w2[2] = {ops.add(a.wg, a.e * a.f, a.d, pl.wg), ops.add(a.wu, a.e * a.f, a.d, pl.wu)};
    const Matrix x{work + pl.x, pl.rp, a.d, pl.dp}, y{work + pl.y, pl.rp, a.d, pl.dp};
    const Matrix h{work + pl.h, pl.rp, a.f, pl.fw};
    const Matrix d2[2] = {{work + pl.dg, pl.rp, a.f, pl.fw}, {work + pl.du, pl.rp, a.f, pl.fw}};
    ExpertParams p = params_of(a, pl);
    PadParams pad{};
    pad.weights = ops.params();
    pad.nrows = need_x ? 2 : 1;
    pad.p = p;
    pad.m[0].src = static_cast<const uint16_t *>(dy);
    pad.m[0].dst = reinterpret_cast<uint16_t *>(work + pl.y);
    // rows that TMA can address are read where they lie, but for the partial blocks
    const bool direct_y = a.d % 8 == 0 && all_aligned({dy}), direct_x = need_x && !eight && a.d % 8 == 0 && all_aligned({a.x});
    const Matrix ly{dy, a.r, a.d, a.d}, lx{a.x, a.r, a.d, a.d};
    pad.m[0].tails = direct_y;
    pad.m[1].tails = direct_x;
    pad.m[1].src = static_cast<const uint16_t *>(a.x);
    pad.m[1].codes = a.x_codes;
    pad.m[1].scales = a.x_scales;
    pad.m[1].dst = reinterpret_cast<uint16_t *>(work + pl.x);
    pad.cols = (uint32_t)a.d;
    pad.ld = (uint32_t)pl.dp;
    pad.width = (uint32_t)xw;
    pad.vector = a.d % 8 == 0 && all_aligned({dy, need_x ? a.x : nullptr});
    const uint64_t most = std::max((pl.rp + 7) / 8, (ops.most() + 255) / 256);
    if ((e = launch_chained(expert_pad_kernel, dim3((unsigned)std::min<uint64_t>(most, 8 * kSms), pad.nrows + (unsigned)pad.weights.n), dim3(256), 0, stream, pad)))
        return from_cuda(e);
    count_launches(1);
    const uint64_t active = std::min<uint64_t>(a.r, a.e), tiles = a.r / kTileM + active; // at most
    const uint64_t likely = std::max(active, a.r / kTileM + active / 2);
    Problem &q = p.prob[0];
    p.half = half_tile(likely, a.f, tiles_of(a.d, kTileK), 7.0);
    set_problem(q, a.f, 2 * p.half, a.d, 1);
    p.padded = !direct_y;
    if (!encode_rows(&q.a[0], direct_y ? ly : y, false) || !encode_experts(&q.b[0], wd, a.e, true))
        return CCL_ERR_CUDA;
    if ((e = launch_gemm<EPI_BACKWARD, false, true>(p, tiles * q.nt, stream)))
        return from_cuda(e);
    p.padded = 1;
    if (dx) {
        const bool vectors = a.d % 8 == 0 && (uintptr_t)dx % 16 == 0;
        p.half = half_tile(likely, a.d, 2 * tiles_of(a.f, kTileK), vectors ? 2.5 : 4.0);
        set_problem(q, a.d, 2 * p.half, a.f, 2);
        q.out = dx;
        for (int i = 0; i < 2; ++i)
            if (!encode_rows(&q.a[i], d2[i], false) || !encode_experts(&q.b[i], w2[i], a.e, true))
                return CCL_ERR_CUDA;
        if ((e = launch_out<EPI_STORE, false, true>(p, vectors, tiles * q.nt, stream)))
            return from_cuda(e);
    }
    if (!need_x && !dwd)
        return CCL_OK;
    // the weight gradients asked for, in one launch
    p.accumulate = accumulate != 0;
    bool vectors = a.d % 8 == 0 && a.f % 8 == 0;
    p.nprob = 0;
    uint64_t units = 0;
    for (void *g : {dwg, dwu, dwd})
        vectors = vectors && (uintptr_t)g % 16 == 0;
    p.half = half_tile(a.e * ((dwg != nullptr) + (dwu != nullptr) + (dwd != nullptr)) * tiles_of(a.f, kTileM), a.d,
                       tiles_of(a.r / active, kTileK), vectors ? 2.5 : 4.0);
    const Matrix *am[3] = {&d2[0], &d2[1], &y}, *bm[3] = {&x, &x, &h};
    void *out[3] = {dwg, dwu, dwd};
    for (int i = 0; i < 3; ++i)
        if (out[i]) {
            Problem &o = p.prob[p.nprob++];
            o.m = (uint32_t)am[i]->cols;
            o.mt = tiles_of(o.m, kTileM);
            set_problem(o, bm[i]->cols, 2 * p.half, 0, 1);
            o.out = out[i];
            o.direct_a = i == 2 && direct_y;
            o.direct_b = i < 2 && direct_x;
            if (!encode_rows(&o.a[0], *am[i], true) || !encode_rows(&o.b[0], *bm[i], true) || (o.direct_a && !encode_rows(&o.a[1], ly, true)) ||
                (o.direct_b && !encode_rows(&o.b[1], lx, true)))
                return CCL_ERR_CUDA;
            units += (uint64_t)o.mt * o.nt;
        }
    p.by_expert = divisor((uint32_t)units);
    return from_cuda(launch_out<EPI_WEIGHTS, true, true>(p, vectors, units * a.e, stream));
}

} // namespace

cudaError_t expert_timeouts(unsigned long long *count)
{
    unsigned long long n = 0;
    const cudaError_t e = cudaMemcpyFromSymbol(&n, g_expert_timeouts, sizeof n);
    *count += n;
    return e;
}

} // namespace ccl

using namespace ccl;

extern "C" {

ccl_status_t ccl_plan_expert_ffn_work_bytes(size_t nrows, size_t experts, size_t dim, size_t ffn, int backward, int aligned, size_t *bytes)
{
    ExpertPlan f, b;
    if (!bytes || ffn == 0 || !make_plan(nrows, experts, dim, ffn, false, aligned != 0, SIZE_MAX, &f) ||
        !make_plan(nrows, experts, dim, ffn, true, aligned != 0, SIZE_MAX, &b))
        return CCL_ERR_INVALID_ARG;
    *bytes = backward ? std::max(f.bytes, b.bytes) : f.bytes; // a backward pass's buffer serves the forward too
    return CCL_OK;
}

ccl_status_t ccl_expert_ffn(const void *x, const int32_t *offsets, const void *w_gate, const void *w_up, const void *w_down, size_t nrows,
                            size_t experts, size_t dim, size_t ffn, ccl_dtype_t dtype, ccl_act_t act, void *out, int8_t *saved_codes,
                            uint8_t *saved_scales, void *work, size_t work_bytes, cudaStream_t stream)
{
    TraceScope tr("expert_ffn", 1, nrows, (int)dtype, -1, (int)act, stream);
    return tr.done(guarded([&] {
        return expert_ffn_impl(ExpertArgs{x, nullptr, nullptr, offsets, w_gate, w_up, w_down, saved_codes, saved_scales, nrows, experts, dim, ffn,
                                          dtype, act, work, work_bytes},
                               out, stream);
    }));
}

ccl_status_t ccl_expert_ffn_grad(const void *grad_out, const void *x, const int8_t *x_codes, const uint8_t *x_scales, const int32_t *offsets,
                                 const void *w_gate, const void *w_up, const void *w_down, const int8_t *saved_codes, const uint8_t *saved_scales,
                                 size_t nrows, size_t experts, size_t dim, size_t ffn, ccl_dtype_t dtype, ccl_act_t act, int accumulate, void *grad_x,
                                 void *grad_w_gate, void *grad_w_up, void *grad_w_down, void *work, size_t work_bytes, cudaStream_t stream)
{
    TraceScope tr("expert_ffn_grad", 1, nrows, (int)dtype, -1, (int)act, stream);
    return tr.done(guarded([&] {
        return expert_ffn_grad_impl(ExpertArgs{x, x_codes, x_scales, offsets, w_gate, w_up, w_down, const_cast<int8_t *>(saved_codes),
                                               const_cast<uint8_t *>(saved_scales), nrows, experts, dim, ffn, dtype, act, work, work_bytes},
                                    grad_out, grad_x, grad_w_gate, grad_w_up, grad_w_down, accumulate, stream);
    }));
}

} // extern "C"
