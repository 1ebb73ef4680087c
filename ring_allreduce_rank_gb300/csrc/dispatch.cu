// dispatch.cu -- tokens to their experts and back: the order of the tokens'
// copies by expert, the rows of the exchange's send buffer, the weighted sum
// of the experts' rows, and its gradients.
//
// Order: a stable counting sort of the ntokens * top choices by expert.  Up to
// 4096 of them one CTA counts, scans and places, each warp a run of its own, up
// to 16384 a cluster of eight does, in half the host's time of the three chained
// launches that more take (6 us against 11, which is what a call of that size
// costs; on the device 32768 take the cluster 10.3 us and the three 8.4): the
// runs' counts, one scan per expert over the runs, the places.  A choice's rank within its run comes from match.any of a
// warp's 32, so that no atomic decides an order.
//
// Dispatch: rows[place[t][s]] = x[t]: every token's row is read once and
// written top times.  Combine: out[t] = sum over s of w[t][s] rows[place[t][s]],
// in fp32, in the order of s, one rounding.  Its gradients: grad_rows[place] =
// w grad_out[t], grad_w = <grad_out[t], rows[place]>, in one pass over a
// token's rows.  All three are bound by memory bandwidth; a group of threads
// takes a token, each 32-byte vector (16 where a row is no multiple of it) of
// its rows with every row's load in flight before the first sum.  8192 tokens of
// 7168 bf16, 4 choices: dispatch 84.7 us (6.9 TB/s; in 16-byte vectors 87.0, in
// elements 91.6), combine 82.0 (7.2 TB/s; 86.6, 230.6), its gradients 148.6 (7.1
// TB/s; 151.6, 217.1).
#include <cooperative_groups.h>

#include <vector>

#include "../../include/ccl.h"
#include "ccl_internal.h"
#include "step_ops.cuh"

namespace cg = cooperative_groups;

namespace ccl {
namespace {

constexpr size_t kMaxChoices = 0x7fffffff, kMaxDim = (size_t)1 << 24;
constexpr uint32_t kFewChoices = 4096, kClusterChoices = 16384;
constexpr int kOrderCtas = 8; // one portable cluster
constexpr int kOrderThreads = 256, kOrderWarps = kOrderThreads / 32;
constexpr uint32_t kFewCounters = 10240; // one CTA's counters, warps x experts

// ------------------------------------------------------------------ order

struct OrderParams {
    const int32_t *ids;
    int32_t *offsets, *place;
    int32_t *counts; // [experts][runs], then their exclusive sums along the runs
    int32_t *totals; // [experts]
    int32_t first;
    uint32_t n, experts, runs, run; // choices, runs and the length of one
};

// A choice's expert, or p.experts.
__device__ __forceinline__ uint32_t expert_of(const OrderParams &p, uint32_t i, uint32_t end)
{
    const int64_t e = i < end ? (int64_t)gload<int32_t>(p.ids + i) - p.first : -1;
    return e >= 0 && e < p.experts ? (uint32_t)e : p.experts;
}

// Adds a warp's 32 choices to its counters; each choice's rank among its
// expert's so far.
__device__ __forceinline__ uint32_t count32(int32_t *counters, uint32_t e, uint32_t experts, uint32_t lane)
{
    const uint32_t same = __match_any_sync(0xffffffffu, e);
    uint32_t at = 0;
    if (e < experts)
        at = (uint32_t)counters[e] + __popc(same & ((1u << lane) - 1));
    __syncwarp();
    if (e < experts && lane == (uint32_t)__ffs(same) - 1)
        counters[e] += __popc(same);
    __syncwarp();
    return at;
}

// The exclusive sum over a warp, and the total.
__device__ __forceinline__ uint32_t warp_scan(uint32_t v, uint32_t lane, uint32_t &total)
{
    uint32_t s = v;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const uint32_t o = __shfl_up_sync(0xffffffffu, s, d);
        if (lane >= (uint32_t)d)
            s += o;
    }
    total = __shfl_sync(0xffffffffu, s, 31);
    return s - v;
}

// Everything in one launch, by one CTA or a cluster of them: counters[warp][expert]
// in shared memory, a warp a run, and the CTAs' counts from one another's.
template <int CTAS> __global__ void __launch_bounds__(1024) order_few_kernel(const __grid_constant__ OrderParams p)
{
    chain_entry();
    __shared__ int32_t counters[kFewCounters], mine[CCL_MAX_EXPERTS];
    __shared__ uint32_t sums[32];
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5, rank = blockIdx.x;
    for (uint32_t i = threadIdx.x; i < warps * p.experts; i += blockDim.x)
        counters[i] = 0;
    __syncthreads();
    const uint32_t i0 = min((rank * warps + warp) * p.run, p.n), i1 = min(i0 + p.run, p.n);
    int32_t *own = counters + warp * p.experts;
    // the run's experts, eight loads in flight; the first 256 choices' stay for the places
    constexpr uint32_t kHeld = 8;
    uint32_t held[kHeld], more[kHeld];
    auto fetch = [&](uint32_t *e, uint32_t i) {
#pragma unroll
        for (uint32_t j = 0; j < kHeld; ++j)
            e[j] = expert_of(p, i + 32 * j + lane, i1);
    };
    auto count = [&](const uint32_t *e, uint32_t i, bool place) {
#pragma unroll
        for (uint32_t j = 0; j < kHeld; ++j)
            if (i + 32 * j < i1) {
                const uint32_t at = count32(own, e[j], p.experts, lane);
                if (place && i + 32 * j + lane < i1)
                    gstore<int32_t>(p.place + i + 32 * j + lane, e[j] < p.experts ? (int32_t)at : -1);
            }
    };
    fetch(held, i0);
    count(held, i0, false);
    for (uint32_t i = i0 + 32 * kHeld; i < i1; i += 32 * kHeld) {
        fetch(more, i);
        count(more, i, false);
    }
    __syncthreads();
    if (CTAS > 1) {
        for (uint32_t e = threadIdx.x; e < p.experts; e += blockDim.x) {
            int32_t n = 0;
#pragma unroll 8
            for (uint32_t w = 0; w < warps; ++w)
                n += counters[w * p.experts + e];
            mine[e] = n;
        }
        cg::this_cluster().sync();
    }
    // experts in order, within one the CTAs, within those the warps: a thread takes an expert
    uint32_t before = 0;
    for (uint32_t e0 = 0; e0 < p.experts; e0 += blockDim.x) {
        const uint32_t e = e0 + threadIdx.x;
        uint32_t n = 0, lower = 0, all;
        if (e < p.experts) {
            if (CTAS > 1) {
                uint32_t c[CTAS];
#pragma unroll
                for (int k = 0; k < CTAS; ++k)
                    c[k] = (uint32_t)cg::this_cluster().map_shared_rank(mine, k)[e];
#pragma unroll
                for (int k = 0; k < CTAS; ++k) {
                    n += c[k];
                    lower += (uint32_t)k < rank ? c[k] : 0;
                }
            } else {
#pragma unroll 8
                for (uint32_t w = 0; w < warps; ++w)
                    n += (uint32_t)counters[w * p.experts + e];
            }
        }
        uint32_t at = warp_scan(n, lane, all);
        if (lane == 31)
            sums[warp] = all;
        __syncthreads();
        if (warp == 0) {
            uint32_t rest;
            const uint32_t s = warp_scan(lane < warps ? sums[lane] : 0, lane, rest);
            sums[lane] = s;
        }
        __syncthreads();
        at += before + sums[warp];
        const uint32_t past = at + n;
        if (e < p.experts) {
            if (rank == 0) {
                gstore<int32_t>(p.offsets + e, (int32_t)at);
                if (e + 1 == p.experts)
                    gstore<int32_t>(p.offsets + p.experts, (int32_t)past);
            }
            at += lower;
            for (uint32_t w0 = 0; w0 < warps; w0 += 8) {
                uint32_t c[8];
#pragma unroll
                for (uint32_t w = 0; w < 8; ++w)
                    c[w] = w0 + w < warps ? (uint32_t)counters[(w0 + w) * p.experts + e] : 0;
#pragma unroll
                for (uint32_t w = 0; w < 8; ++w) {
                    if (w0 + w < warps)
                        counters[(w0 + w) * p.experts + e] = (int32_t)at;
                    at += c[w];
                }
            }
        }
        __syncthreads();
        if (e0 + blockDim.x < p.experts) { // fewer threads than experts: a rare second round
            if (threadIdx.x == blockDim.x - 1)
                sums[0] = past;
            __syncthreads();
            before = sums[0];
            __syncthreads();
        }
    }
    if (CTAS > 1)
        cg::this_cluster().sync(); // the counts have been read before any of the CTAs goes
    count(held, i0, true);
    for (uint32_t i = i0 + 32 * kHeld; i < i1; i += 32 * kHeld) {
        fetch(more, i);
        count(more, i, true);
    }
}

// The runs' counts, a warp a run.
__global__ void __launch_bounds__(kOrderThreads) order_count_kernel(const __grid_constant__ OrderParams p)
{
    chain_entry();
    extern __shared__ int32_t counters[];
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int32_t *mine = counters + warp * p.experts;
    for (uint32_t e = lane; e < p.experts; e += 32)
        mine[e] = 0;
    __syncwarp();
    const uint32_t run = blockIdx.x * kOrderWarps + warp;
    const uint64_t start = (uint64_t)run * p.run;
    const uint32_t i0 = (uint32_t)umin64(start, p.n), i1 = (uint32_t)umin64(start + p.run, p.n);
    for (uint32_t i = i0; i < i1; i += 32) {
        const uint32_t e = expert_of(p, i + lane, i1), same = __match_any_sync(0xffffffffu, e);
        if (e < p.experts && lane == (uint32_t)__ffs(same) - 1)
            mine[e] += __popc(same);
        __syncwarp();
    }
    if (run < p.runs)
        for (uint32_t e = lane; e < p.experts; e += 32)
            gstore<int32_t>(p.counts + (uint64_t)e * p.runs + run, mine[e]);
}

// Each expert's counts to their exclusive sums along the runs, a warp an expert.
__global__ void __launch_bounds__(kOrderThreads) order_scan_kernel(const __grid_constant__ OrderParams p)
{
    chain_entry();
    const uint32_t e = blockIdx.x * kOrderWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (e >= p.experts)
        return;
    int32_t *row = p.counts + (uint64_t)e * p.runs;
    uint32_t before = 0;
    for (uint32_t r0 = 0; r0 < p.runs; r0 += 128) { // four loads in flight
        uint32_t v[4], all;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            v[j] = r0 + 32 * j + lane < p.runs ? (uint32_t)gload<int32_t>(row + r0 + 32 * j + lane) : 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t s = warp_scan(v[j], lane, all);
            if (r0 + 32 * j + lane < p.runs)
                gstore<int32_t>(row + r0 + 32 * j + lane, (int32_t)(before + s));
            before += all;
        }
    }
    if (lane == 0)
        gstore<int32_t>(p.totals + e, (int32_t)before);
}

// The places, a warp a run; every CTA sums the experts' totals for itself.
__global__ void __launch_bounds__(kOrderThreads) order_place_kernel(const __grid_constant__ OrderParams p)
{
    chain_entry();
    extern __shared__ int32_t counters[]; // [warps][experts], then [experts + 1] first rows
    int32_t *first = counters + kOrderWarps * p.experts;
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp == 0) {
        uint32_t before = 0;
        for (uint32_t e0 = 0; e0 < p.experts; e0 += 32) {
            uint32_t all;
            const uint32_t s = warp_scan(e0 + lane < p.experts ? (uint32_t)gload<int32_t>(p.totals + e0 + lane) : 0, lane, all);
            if (e0 + lane < p.experts)
                first[e0 + lane] = (int32_t)(before + s);
            before += all;
        }
        if (lane == 0)
            first[p.experts] = (int32_t)before;
    }
    __syncthreads();
    if (blockIdx.x == 0)
        for (uint32_t e = threadIdx.x; e <= p.experts; e += kOrderThreads)
            gstore<int32_t>(p.offsets + e, first[e]);
    const uint32_t run = blockIdx.x * kOrderWarps + warp;
    if (run >= p.runs)
        return;
    int32_t *mine = counters + warp * p.experts;
    for (uint32_t e = lane; e < p.experts; e += 32)
        mine[e] = first[e] + gload<int32_t>(p.counts + (uint64_t)e * p.runs + run);
    __syncwarp();
    const uint64_t start = (uint64_t)run * p.run;
    const uint32_t i0 = (uint32_t)umin64(start, p.n), i1 = (uint32_t)umin64(start + p.run, p.n);
    for (uint32_t i = i0; i < i1; i += 32) {
        const uint32_t e = expert_of(p, i + lane, i1), at = count32(mine, e, p.experts, lane);
        if (i + lane < i1)
            gstore<int32_t>(p.place + i + lane, e < p.experts ? (int32_t)at : -1);
    }
}

// ------------------------------------------------------------------ rows

// A group of threads (x) takes a token (blockIdx.x * blockDim.y + y); `items`
// are the vectors (elements) of a row.
struct RowsParams {
    const char *in; // dispatch: x; else the experts' rows
    char *out;      // dispatch: the experts' rows; combine: out
    const char *dy;
    char *grad_rows;
    float *grad_weights;
    const int32_t *place;
    const float *weights;
    uint64_t ntokens, nrows;
    uint64_t in_pitch, out_pitch, dy_pitch, grad_pitch; // bytes
    uint32_t top, items;
};

// A vector of W bytes of a row: 32, 16, or one element (W = 0).
template <int DT, int W> struct Vec {
    static constexpr int N = W == 0 ? 1 : W / DType<DT>::kSize;
    uint4 v[W == 32 ? 2 : 1];
    __device__ __forceinline__ void load(const char *row, uint32_t i)
    {
        if (W == 32)
            ld32(row + (uint64_t)i * 32, v[0], v[W == 32 ? 1 : 0]);
        else if (W == 16)
            v[0] = ld16(row + (uint64_t)i * 16);
        else
            v[0].x = ld_elem<DT>(row, i);
    }
    __device__ __forceinline__ void store(char *row, uint32_t i) const
    {
        if (W == 32)
            st32(row + (uint64_t)i * 32, v[0], v[W == 32 ? 1 : 0]);
        else if (W == 16)
            st16(row + (uint64_t)i * 16, v[0]);
        else
            st_elem<DT>(row, i, v[0].x);
    }
    __device__ __forceinline__ void get(float *f) const
    {
        if (W == 0) {
            f[0] = __uint_as_float(DT == DT_BF16 ? v[0].x << 16 : v[0].x);
        } else {
            unpack<DT>(v[0], f);
            if (W == 32)
                unpack<DT>(v[W == 32 ? 1 : 0], f + 16 / DType<DT>::kSize);
        }
    }
    __device__ __forceinline__ void set(const float *f)
    {
        if (W == 0) {
            const __nv_bfloat16 h = __float2bfloat16_rn(f[0]);
            v[0].x = DT == DT_BF16 ? *reinterpret_cast<const uint16_t *>(&h) : __float_as_uint(f[0]);
        } else {
            v[0] = pack<DT>(f);
            if (W == 32)
                v[W == 32 ? 1 : 0] = pack<DT>(f + 16 / DType<DT>::kSize);
        }
    }
};

template <int DT, int W> __global__ void __launch_bounds__(128) dispatch_kernel(const __grid_constant__ RowsParams p)
{
    chain_entry();
    const uint64_t t = (uint64_t)blockIdx.x * blockDim.y + threadIdx.y;
    if (t >= p.ntokens)
        return;
    constexpr int AHEAD = 4;
    const char *src = p.in + t * p.in_pitch;
    const int32_t *place = p.place + t * p.top;
    for (uint32_t i0 = threadIdx.x; i0 < p.items; i0 += AHEAD * blockDim.x) {
        Vec<DT, W> v[AHEAD];
#pragma unroll
        for (int j = 0; j < AHEAD; ++j)
            if (i0 + j * blockDim.x < p.items)
                v[j].load(src, i0 + j * blockDim.x);
        for (uint32_t s = 0; s < p.top; ++s) {
            const uint32_t row = (uint32_t)gload<int32_t>(place + s);
            if (row >= p.nrows)
                continue;
            char *dst = p.out + row * p.out_pitch;
#pragma unroll
            for (int j = 0; j < AHEAD; ++j)
                if (i0 + j * blockDim.x < p.items)
                    v[j].store(dst, i0 + j * blockDim.x);
        }
    }
}

constexpr int kSlots = 4; // rows of a token whose loads are in flight together

// kSlots of a token's rows and weights.
struct Slots {
    uint32_t row[kSlots];
    float w[kSlots];
    __device__ __forceinline__ void load(const RowsParams &p, uint64_t t, uint32_t s0)
    {
#pragma unroll
        for (int s = 0; s < kSlots; ++s) {
            row[s] = s0 + s < p.top ? (uint32_t)gload<int32_t>(p.place + t * p.top + s0 + s) : 0xffffffffu;
            w[s] = p.weights && s0 + s < p.top ? gload<float>(p.weights + t * p.top + s0 + s) : 1.0f;
        }
    }
};

template <int DT, int W> __global__ void __launch_bounds__(128) combine_kernel(const __grid_constant__ RowsParams p)
{
    chain_entry();
    const uint64_t t = (uint64_t)blockIdx.x * blockDim.y + threadIdx.y;
    if (t >= p.ntokens)
        return;
    constexpr int N = Vec<DT, W>::N, AHEAD = W == 0 ? 4 : 1; // single elements: four of a row in flight
    char *dst = p.out + t * p.out_pitch;
    Slots slots;
    slots.load(p, t, 0);
    for (uint32_t i0 = threadIdx.x; i0 < p.items; i0 += AHEAD * blockDim.x) {
        float acc[AHEAD][N], f[N];
#pragma unroll
        for (int j = 0; j < AHEAD; ++j)
#pragma unroll
            for (int k = 0; k < N; ++k)
                acc[j][k] = 0.0f;
        for (uint32_t s0 = 0; s0 < p.top; s0 += kSlots) {
            if (p.top > kSlots)
                slots.load(p, t, s0);
            Vec<DT, W> v[AHEAD][kSlots];
#pragma unroll
            for (int j = 0; j < AHEAD; ++j)
#pragma unroll
                for (int s = 0; s < kSlots; ++s)
                    if (slots.row[s] < p.nrows && i0 + j * blockDim.x < p.items)
                        v[j][s].load(p.in + slots.row[s] * p.in_pitch, i0 + j * blockDim.x);
#pragma unroll
            for (int j = 0; j < AHEAD; ++j)
#pragma unroll
                for (int s = 0; s < kSlots; ++s)
                    if (slots.row[s] < p.nrows && i0 + j * blockDim.x < p.items) {
                        v[j][s].get(f);
#pragma unroll
                        for (int k = 0; k < N; ++k)
                            acc[j][k] = __fmaf_rn(slots.w[s], f[k], acc[j][k]);
                    }
        }
#pragma unroll
        for (int j = 0; j < AHEAD; ++j)
            if (i0 + j * blockDim.x < p.items) {
                Vec<DT, W> o;
                o.set(acc[j]);
                o.store(dst, i0 + j * blockDim.x);
            }
    }
}

// One CTA a token.  The weights' gradients of kSlots rows at a time are sums
// over the row in a fixed order: a thread's vectors, the lanes, the warps.
template <int DT, int W, bool DOTS> __global__ void __launch_bounds__(256) combine_grad_kernel(const __grid_constant__ RowsParams p)
{
    chain_entry();
    __shared__ float sums[8][kSlots];
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (uint64_t t = blockIdx.x; t < p.ntokens; t += gridDim.x) {
        const char *dy = p.dy + t * p.dy_pitch;
        for (uint32_t s0 = 0; s0 < p.top; s0 += kSlots) {
            Slots slots;
            slots.load(p, t, s0);
            const uint32_t(&row)[kSlots] = slots.row;
            const float(&w)[kSlots] = slots.w;
            float dot[kSlots];
#pragma unroll
            for (int s = 0; s < kSlots; ++s)
                dot[s] = 0.0f;
            for (uint32_t i = threadIdx.x; i < p.items; i += blockDim.x) {
                constexpr int N = Vec<DT, W>::N;
                Vec<DT, W> y, v[kSlots], o;
                float g[N], f[N];
                y.load(dy, i);
                if (DOTS) {
#pragma unroll
                    for (int s = 0; s < kSlots; ++s)
                        if (row[s] < p.nrows)
                            v[s].load(p.in + row[s] * p.in_pitch, i);
                }
                y.get(g);
#pragma unroll
                for (int s = 0; s < kSlots; ++s)
                    if (row[s] < p.nrows) {
                        if (DOTS) {
                            v[s].get(f);
#pragma unroll
                            for (int k = 0; k < N; ++k)
                                dot[s] = __fmaf_rn(g[k], f[k], dot[s]);
                        }
                        if (p.grad_rows) {
#pragma unroll
                            for (int k = 0; k < N; ++k)
                                f[k] = __fmul_rn(w[s], g[k]);
                            o.set(f);
                            o.store(p.grad_rows + row[s] * p.grad_pitch, i);
                        }
                    }
            }
            if (DOTS) {
#pragma unroll
                for (int s = 0; s < kSlots; ++s) {
#pragma unroll
                    for (int d = 16; d; d /= 2)
                        dot[s] = __fadd_rn(dot[s], __shfl_xor_sync(0xffffffffu, dot[s], d));
                    if (lane == 0)
                        sums[warp][s] = dot[s];
                }
                __syncthreads();
                if (threadIdx.x < kSlots && s0 + threadIdx.x < p.top) {
                    float v = 0.0f;
                    for (uint32_t k = 0; k < blockDim.x / 32; ++k)
                        v = __fadd_rn(v, sums[k][threadIdx.x]);
                    gstore<float>(p.grad_weights + t * p.top + s0 + threadIdx.x, v); // 0 where there is no row
                }
                __syncthreads();
            }
        }
    }
}

// ------------------------------------------------------------------ host side

struct OrderPlan {
    uint32_t n, run, runs, warps, ctas; // warps: of a CTA of the one launch, 0 where there are several
    size_t counts, bytes;
};

bool plan_order(size_t ntokens, size_t top, size_t experts, OrderPlan *p)
{
    if (ntokens > kMaxChoices || top > CCL_MAX_EXPERT_TOP || experts > CCL_MAX_EXPERTS || ntokens * top > kMaxChoices)
        return false;
    *p = OrderPlan{};
    p->n = (uint32_t)(ntokens * top);
    if (p->n <= kClusterChoices) {
        p->ctas = p->n <= kFewChoices ? 1 : kOrderCtas;
        p->warps = std::max<uint32_t>(1, std::min<uint32_t>({32, (p->n + 31) / 32, kFewCounters / (uint32_t)std::max<size_t>(experts, 1)}));
        p->run = ((p->n + p->ctas * p->warps - 1) / (p->ctas * p->warps) + 31) / 32 * 32;
        return true;
    }
    // a run a warp, eight of them on every SM, but no fewer choices than experts whose counts it writes
    constexpr size_t most = 8 * 152;
    const uint32_t least = (uint32_t)((std::max<size_t>(experts, 64) + 31) / 32 * 32);
    p->run = std::max(least, (uint32_t)((p->n + most - 1) / most + 31) / 32 * 32);
    p->runs = (p->n + p->run - 1) / p->run;
    // room for the most runs that so many choices or fewer are cut into: the
    // length's steps of 32 make runs fewer again as the choices grow, and a buffer
    // serves every call that is smaller than the one it was planned for
    p->counts = up(experts * std::min(most, ((size_t)p->n + least - 1) / least) * 4);
    p->bytes = p->counts + up(experts * 4);
    return true;
}

ccl_status_t order_impl(const int32_t *ids, size_t ntokens, size_t top, int32_t first, size_t experts, int32_t *offsets, int32_t *place, void *work,
                        size_t work_bytes, cudaStream_t stream)
{
    OrderPlan pl;
    if (!plan_order(ntokens, top, experts, &pl))
        return CCL_ERR_INVALID_ARG;
    if (!offsets || (pl.n && (!ids || !place)) || !element_aligned(4, {ids, offsets, place}) ||
        (pl.bytes && (!work || (uintptr_t)work % 256 || work_bytes < pl.bytes)))
        return CCL_ERR_INVALID_ARG;
    const std::vector<Range> w{range_of(offsets, (experts + 1) * 4, 0), range_of(place, (size_t)pl.n * 4, 0), range_of(work, pl.bytes, 0)},
        r{range_of(ids, (size_t)pl.n * 4, 0)};
    if (ccl_status_t st = check_overlaps(w, r, [](const Range &, const Range &) { return false; }))
        return st;
    if (pl.n == 0 || experts == 0) { // no choice has a row
        cudaError_t e = cudaMemsetAsync(offsets, 0, (experts + 1) * 4, stream);
        if (e == cudaSuccess && pl.n)
            e = cudaMemsetAsync(place, 0xff, (size_t)pl.n * 4, stream);
        return from_cuda(e);
    }
#ifdef CCL_DEBUG_BOUNDS
    if (cudaError_t e = dbg_set_ranges({{offsets, (experts + 1) * 4}, {place, (size_t)pl.n * 4}, {work, pl.bytes}, {ids, (size_t)pl.n * 4}}, stream))
        return from_cuda(e);
#endif
    OrderParams p{};
    p.ids = ids;
    p.offsets = offsets;
    p.place = place;
    p.counts = static_cast<int32_t *>(work);
    p.totals = reinterpret_cast<int32_t *>(static_cast<char *>(work) + pl.counts);
    p.first = first;
    p.n = pl.n;
    p.experts = (uint32_t)experts;
    p.runs = pl.runs;
    p.run = pl.run;
    cudaError_t e;
    if (pl.warps) {
        if (pl.ctas == 1) {
            e = launch_chained(order_few_kernel<1>, dim3(1), dim3(32 * pl.warps), 0, stream, p);
        } else {
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(kOrderCtas);
            cfg.blockDim = dim3(32 * pl.warps);
            cfg.stream = stream;
            cudaLaunchAttribute attr[2];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = kOrderCtas;
            attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
            attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
            attr[1].val.programmaticStreamSerializationAllowed = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 2;
            e = cudaLaunchKernelEx(&cfg, order_few_kernel<kOrderCtas>, p);
        }
        if (e == cudaSuccess)
            count_launches(1);
        return from_cuda(e);
    }
    const unsigned ctas = (pl.runs + kOrderWarps - 1) / kOrderWarps;
    const size_t smem = kOrderWarps * experts * 4;
    if ((e = launch_chained(order_count_kernel, dim3(ctas), dim3(kOrderThreads), smem, stream, p)) != cudaSuccess)
        return from_cuda(e);
    count_launches(1);
    if ((e = launch_chained(order_scan_kernel, dim3((p.experts + kOrderWarps - 1) / kOrderWarps), dim3(kOrderThreads), 0, stream, p)) != cudaSuccess)
        return from_cuda(e);
    count_launches(1);
    if ((e = launch_chained(order_place_kernel, dim3(ctas), dim3(kOrderThreads), smem + (experts + 1) * 4, stream, p)) != cudaSuccess)
        return from_cuda(e);
    count_launches(1);
    return CCL_OK;
}

// The widest vector that all the rows are whole multiples of, in bytes (0: an element).
int width_of(std::initializer_list<uintptr_t> all)
{
    uintptr_t x = 0;
    for (uintptr_t v : all)
        x |= v;
    return x % 32 == 0 ? 32 : x % 16 == 0 ? 16 : 0;
}

// kernel<DT, W> of the call's type and width
#define CCL_ROWS_KERNEL(kernel, dtype, width, ...)                                                                     \
    ((dtype) == CCL_FP32 ? ((width) == 32 ? kernel<DT_FP32, 32 __VA_ARGS__>                                            \
                                          : (width) == 16 ? kernel<DT_FP32, 16 __VA_ARGS__> : kernel<DT_FP32, 0 __VA_ARGS__>) \
                         : ((width) == 32 ? kernel<DT_BF16, 32 __VA_ARGS__>                                            \
                                          : (width) == 16 ? kernel<DT_BF16, 16 __VA_ARGS__> : kernel<DT_BF16, 0 __VA_ARGS__>))

struct RowsArgs {
    const void *in;
    size_t in_rows, in_stride;
    void *out;
    size_t out_rows, out_stride;
    size_t dim;
    ccl_dtype_t dtype;
    const int32_t *place;
    const float *weights;
    size_t ntokens, top;
    bool combine;
};

ccl_status_t rows_impl(const RowsArgs &a, cudaStream_t stream)
{
    if (!valid_dtype(a.dtype) || a.in_stride < a.dim || a.out_stride < a.dim || a.dim > kMaxDim || a.top > CCL_MAX_EXPERT_TOP ||
        a.ntokens > kMaxChoices || a.ntokens * a.top > kMaxChoices || a.in_rows > kMaxChoices || a.out_rows > kMaxChoices)
        return CCL_ERR_INVALID_ARG;
    const size_t es = elem_size(a.dtype), choices = a.ntokens * a.top;
    size_t ib, ob;
    if (!extent(a.in_rows, a.dim, a.in_stride, es, &ib) || !extent(a.out_rows, a.dim, a.out_stride, es, &ob))
        return CCL_ERR_INVALID_ARG;
    if (a.ntokens == 0 || a.dim == 0 || (!a.combine && (choices == 0 || a.out_rows == 0)))
        return CCL_OK;
    if ((a.in_rows && !a.in) || !a.out || (choices && !a.place) || !element_aligned(es, {a.in, a.out}) || !element_aligned(4, {a.place, a.weights}))
        return CCL_ERR_INVALID_ARG;
    const std::vector<Range> w{range_of(a.out, ob, 0)},
        r{range_of(a.in, ib, 0), range_of(a.place, choices * 4, 0), range_of(a.weights, a.weights ? choices * 4 : 0, 0)};
    if (ccl_status_t st = check_overlaps(w, r, [](const Range &, const Range &) { return false; }))
        return st;
#ifdef CCL_DEBUG_BOUNDS
    if (cudaError_t e = dbg_set_ranges({{a.out, ob}, {a.in, ib}, {a.place, choices * 4}, {a.weights, a.weights ? choices * 4 : 0}}, stream))
        return from_cuda(e);
#endif
    RowsParams p{};
    p.in = static_cast<const char *>(a.in);
    p.out = static_cast<char *>(a.out);
    p.place = a.place;
    p.weights = a.weights;
    p.ntokens = a.ntokens;
    p.nrows = a.combine ? a.in_rows : a.out_rows;
    p.in_pitch = a.in_stride * es;
    p.out_pitch = a.out_stride * es;
    p.top = (uint32_t)a.top;
    const int width = width_of({(uintptr_t)a.in, (uintptr_t)a.out, p.in_pitch, p.out_pitch, a.dim * es});
    p.items = (uint32_t)(width ? a.dim * es / width : a.dim);
    unsigned tx = 1;
    while (tx < 128 && tx < p.items)
        tx *= 2;
    const dim3 block(tx, 128 / tx), grid((unsigned)((a.ntokens + block.y - 1) / block.y));
    const auto k = a.combine ? CCL_ROWS_KERNEL(combine_kernel, a.dtype, width) : CCL_ROWS_KERNEL(dispatch_kernel, a.dtype, width);
    const cudaError_t e = launch_chained(k, grid, block, 0, stream, p);
    if (e == cudaSuccess)
        count_launches(1);
    return from_cuda(e);
}

struct GradArgs {
    const void *dy;
    size_t dy_stride;
    const void *rows;
    size_t nrows, rows_stride, dim;
    ccl_dtype_t dtype;
    const int32_t *place;
    const float *weights;
    size_t ntokens, top;
    void *grad_rows;
    size_t grad_stride;
    float *grad_weights;
};

#define CCL_COMMA_TRUE , true
#define CCL_COMMA_FALSE , false

ccl_status_t combine_grad_impl(const GradArgs &a, cudaStream_t stream)
{
    if (!valid_dtype(a.dtype) || a.dy_stride < a.dim || (a.grad_weights && a.rows_stride < a.dim) || (a.grad_rows && a.grad_stride < a.dim) ||
        a.dim > kMaxDim || a.top > CCL_MAX_EXPERT_TOP || a.ntokens > kMaxChoices || a.ntokens * a.top > kMaxChoices || a.nrows > kMaxChoices)
        return CCL_ERR_INVALID_ARG;
    const size_t es = elem_size(a.dtype), choices = a.ntokens * a.top;
    size_t yb, rb = 0, gb = 0;
    if (!extent(a.ntokens, a.dim, a.dy_stride, es, &yb) || (a.grad_weights && !extent(a.nrows, a.dim, a.rows_stride, es, &rb)) ||
        (a.grad_rows && !extent(a.nrows, a.dim, a.grad_stride, es, &gb)))
        return CCL_ERR_INVALID_ARG;
    if (choices == 0 || (!a.grad_rows && !a.grad_weights))
        return CCL_OK;
    if (!a.place || (a.dim && (!a.dy || (a.grad_weights && a.nrows && !a.rows))) || !element_aligned(es, {a.dy, a.rows, a.grad_rows}) ||
        !element_aligned(4, {a.place, a.weights, a.grad_weights}))
        return CCL_ERR_INVALID_ARG;
    // in place: the rows' gradients may take the rows' place, vector by vector
    const bool in_place = a.grad_rows && a.grad_rows == a.rows && a.grad_stride == a.rows_stride;
    const std::vector<Range> w{range_of(a.grad_rows, gb, 1), range_of(a.grad_weights, a.grad_weights ? choices * 4 : 0, 0)},
        r{range_of(a.dy, yb, 0), range_of(a.rows, rb, 1), range_of(a.place, choices * 4, 0), range_of(a.weights, a.weights ? choices * 4 : 0, 0)};
    if (ccl_status_t st = check_overlaps(w, r, [&](const Range &x, const Range &y) { return in_place && x.rank == 1 && y.rank == 1; }))
        return st;
#ifdef CCL_DEBUG_BOUNDS
    std::vector<DbgRange> rg;
    for (const std::vector<Range> *v : {&w, &r})
        for (const Range &x : *v)
            rg.push_back(DbgRange{reinterpret_cast<const void *>(x.lo), (size_t)(x.hi - x.lo)});
    if (cudaError_t e = dbg_set_ranges(rg, stream))
        return from_cuda(e);
#endif
    RowsParams p{};
    p.in = static_cast<const char *>(a.rows);
    p.dy = static_cast<const char *>(a.dy);
    p.grad_rows = static_cast<char *>(a.grad_rows);
    p.grad_weights = a.grad_weights;
    p.place = a.place;
    p.weights = a.weights;
    p.ntokens = a.ntokens;
    p.nrows = a.nrows;
    p.in_pitch = a.rows_stride * es;
    p.dy_pitch = a.dy_stride * es;
    p.grad_pitch = a.grad_stride * es;
    p.top = (uint32_t)a.top;
    const int width = width_of({(uintptr_t)a.dy, p.dy_pitch, a.dim * es, a.grad_weights ? (uintptr_t)a.rows | p.in_pitch : 0,
                                a.grad_rows ? (uintptr_t)a.grad_rows | p.grad_pitch : 0});
    p.items = (uint32_t)(width ? a.dim * es / width : a.dim);
    unsigned threads = 32;
    while (threads < 256 && threads < p.items)
        threads *= 2;
    const dim3 grid((unsigned)a.ntokens);
    const auto k = a.grad_weights ? CCL_ROWS_KERNEL(combine_grad_kernel, a.dtype, width, CCL_COMMA_TRUE)
                                  : CCL_ROWS_KERNEL(combine_grad_kernel, a.dtype, width, CCL_COMMA_FALSE);
    const cudaError_t e = launch_chained(k, grid, dim3(threads), 0, stream, p);
    if (e == cudaSuccess)
        count_launches(1);
    return from_cuda(e);
}

} // namespace
} // namespace ccl

using namespace ccl;

extern "C" {

ccl_status_t ccl_plan_expert_order_work_bytes(size_t ntokens, size_t top, size_t experts, size_t *bytes)
{
    OrderPlan p;
    if (!bytes || !plan_order(ntokens, top, experts, &p))
        return CCL_ERR_INVALID_ARG;
    *bytes = p.bytes;
    return CCL_OK;
}

ccl_status_t ccl_expert_order(const int32_t *ids, size_t ntokens, size_t top, int32_t first_expert, size_t experts, int32_t *offsets, int32_t *place,
                              void *work, size_t work_bytes, cudaStream_t stream)
{
    TraceScope tr("expert_order", 1, ntokens, -1, -1, 0, stream);
    return tr.done(guarded([&] { return order_impl(ids, ntokens, top, first_expert, experts, offsets, place, work, work_bytes, stream); }));
}

ccl_status_t ccl_dispatch(const void *x, size_t ntokens, size_t dim, size_t x_stride, ccl_dtype_t dtype, const int32_t *place, size_t top, void *rows,
                          size_t nrows, size_t rows_stride, cudaStream_t stream)
{
    TraceScope tr("dispatch", 1, ntokens, (int)dtype, -1, 0, stream);
    return tr.done(guarded([&] {
        return rows_impl(RowsArgs{x, ntokens, x_stride, rows, nrows, rows_stride, dim, dtype, place, nullptr, ntokens, top, false}, stream);
    }));
}

ccl_status_t ccl_combine(const void *rows, size_t nrows, size_t dim, size_t rows_stride, ccl_dtype_t dtype, const int32_t *place, const float *weights,
                         size_t ntokens, size_t top, void *out, size_t out_stride, cudaStream_t stream)
{
    TraceScope tr("combine", 1, ntokens, (int)dtype, -1, 0, stream);
    return tr.done(guarded([&] {
        return rows_impl(RowsArgs{rows, nrows, rows_stride, out, ntokens, out_stride, dim, dtype, place, weights, ntokens, top, true}, stream);
    }));
}

ccl_status_t ccl_combine_grad(const void *grad_out, size_t grad_out_stride, const void *rows, size_t nrows, size_t dim, size_t rows_stride,
                              ccl_dtype_t dtype, const int32_t *place, const float *weights, size_t ntokens, size_t top, void *grad_rows,
                              size_t grad_rows_stride, float *grad_weights, cudaStream_t stream)
{
    TraceScope tr("combine_grad", 1, ntokens, (int)dtype, -1, 0, stream);
    return tr.done(guarded([&] {
        return combine_grad_impl(GradArgs{grad_out, grad_out_stride, rows, nrows, rows_stride, dim, dtype, place, weights, ntokens, top, grad_rows,
                                          grad_rows_stride, grad_weights},
                                 stream);
    }));
}

} // extern "C"
