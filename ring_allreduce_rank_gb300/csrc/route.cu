// route.cu -- the router of a mixture of experts: the top choices of every
// token's softmax over the experts, the experts' counts, the balance and z
// losses, and the gradient by the logits.
//
//   p = softmax(z), ids = the top largest z (ties: the lower expert), w = p_ids
//   or p_ids / sum p_ids, load_e = choices of e / choices, importance_e = mean
//   of p_e, balance = E sum_e load_e importance_e, zloss = mean of lse^2.
//   dz_j = p_j (G_j - sum_i G_i p_i + 2 c_z lse / n),
//   G_j = c_b E load_j / n + [j chosen] g_j, with g = grad_w, or for normalised
//   weights g_i = (grad_w_i - sum_m grad_w_m w_m) / sum_top p.
//
// A group of 8 or 32 lanes holds a row in registers, reads it once, takes its
// maximum, sum and choices from there, and adds its p to sums of its own
// columns, so that the importance costs no further pass.  A choice is a
// reduction of (ordered bits, expert) over the group, and its holder looks for
// its next best only then.  Sums over the tokens are the groups' rows in order,
// the groups of a CTA in order, the CTAs in order: no float is added by an
// atomic.  Bound by memory bandwidth for many tokens, by the launch and one
// row's chain of reductions for few.
#include <cooperative_groups.h>

#include <vector>

#include "../../include/ccl.h"
#include "ccl_internal.h"
#include "step_ops.cuh"

namespace cg = cooperative_groups;

namespace ccl {
namespace {

constexpr int kJoinCtas = 8; // one portable cluster
constexpr size_t kMaxTokens = 0x7fffffff;
constexpr int kRouteThreads = 256; // route_grad_kernel's
constexpr size_t kSms = 152;
// route_kernel's, at most: one CTA an SM with eight or sixteen values a lane, so
// that 152 rows of partial sums are left; two with 32.  Lanes take 64 to 128
// registers.  (16384 tokens, forward: 256 experts 22.9 us, with 608 CTAs of 256
// threads 26.1; 64 experts 9.0 and 9.5; 4096 x 512 15.2 and 19.8.)  Fewer tokens
// are spread over CTAs of 256 (50 x 256 in one CTA of 1024, two rounds, 11.0 us,
// in seven and a join 6.7; 256 x 64 9.4 and 6.4), but those that one CTA takes at
// once stay in it (128 x 64 5.4 us, spread 6.1).
constexpr int route_threads(int values) { return values <= 8 ? 1024 : values <= 16 ? 512 : 256; }
constexpr size_t kFewRouteThreads = 256;

struct RouteParams {
    const char *logits;
    char *grad;
    uint64_t pitch, grad_pitch; // bytes
    const uint8_t *valid;
    int32_t *ids;
    float *weights, *lse;
    int32_t *counts;
    float *load, *importance, *loss;
    float *sums;     // partial: [ctas][experts + 1], the last one of lse^2
    int32_t *hits;   // partial: [ctas][experts + 2], the last ones routed tokens and choices
    const float *grad_weights;
    float balance, z; // the losses' coefficients
    uint32_t ntokens, experts, top, ctas;
    int normalize;
};

constexpr uint32_t kNothing = 0x007fffffu, kNaN = 0xffffffffu; // ordered(-inf); any NaN

// A float's bits in an order of unsigned numbers: both zeros equal, any NaN
// above +inf.
__device__ __forceinline__ uint32_t ordered(float f)
{
    const uint32_t b = __float_as_uint(__fadd_rn(f, 0.0f)); // -0 + 0 = 0
    if ((b & 0x7fffffffu) > 0x7f800000u)
        return kNaN;
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float from_ordered(uint32_t k)
{
    return __uint_as_float(k == kNaN ? 0x7fffffffu : k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

// e^x for x <= 0, to 2 + 1.2 |x| units in the last place: 1.4e-6 of a probability
// e^-8 of the largest.  x, the rounded difference of two fp32 logits, is itself
// good to |x| / 2 such units; of two bf16 logits it is often exact, and the error is
// this function's.  expf, good to 2 units, takes 3 % more (131072 x 256 bf16 119 us
// for 116, 16384 x 256 fp32 23.2 for 22.5, its gradient 10.8 for 10.2).
__device__ __forceinline__ float exp_of(float x) { return __expf(x); }

template <int L> __device__ __forceinline__ float group_sum(float v)
{
#pragma unroll
    for (int d = L / 2; d; d /= 2)
        v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, d));
    return v;
}

template <int L> __device__ __forceinline__ uint32_t group_max(uint32_t v)
{
    if constexpr (L == 32) {
        return __reduce_max_sync(0xffffffffu, v);
    } else {
#pragma unroll
        for (int d = L / 2; d; d /= 2)
            v = max(v, __shfl_xor_sync(0xffffffffu, v, d));
        return v;
    }
}

template <int L> __device__ __forceinline__ uint32_t group_min(uint32_t v)
{
    if constexpr (L == 32) {
        return __reduce_min_sync(0xffffffffu, v);
    } else {
#pragma unroll
        for (int d = L / 2; d; d /= 2)
            v = min(v, __shfl_xor_sync(0xffffffffu, v, d));
        return v;
    }
}

// Column of a lane's i-th value: vectors of N side by side, so that a group's
// loads run along the row.
template <int L, int N> __device__ __forceinline__ uint32_t column(uint32_t lane, int i) { return (i / N) * (L * N) + lane * N + i % N; }

// A lane's V values of a row; columns past the experts are -inf.
template <int DT, int L, int V, int N> __device__ __forceinline__ void load_row(const RouteParams &p, const char *row, uint32_t lane, float *f)
{
    if (N > 1) {
#pragma unroll
        for (int i = 0; i < V; i += N) {
            const uint32_t c = column<L, N>(lane, i);
            const bool in = c < p.experts;
            const char *at = row + (uint64_t)c * DType<DT>::kSize;
            uint4 v = make_uint4(0, 0, 0, 0);
            if (in && N * DType<DT>::kSize == 16) {
                v = ld16(at);
            } else if (in && N * DType<DT>::kSize == 8) {
                const uint2 w = gload<uint2>(at);
                v.x = w.x;
                v.y = w.y;
            } else if (in) {
                v.x = gload<uint32_t>(at);
            }
            float h[DType<DT>::kVec];
            unpack<DT>(v, h);
#pragma unroll
            for (int k = 0; k < N; ++k)
                f[i + k] = h[k];
#pragma unroll
            for (int k = 0; k < N; ++k)
                f[i + k] = in ? f[i + k] : -INFINITY;
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const uint32_t c = column<L, 1>(lane, i);
            f[i] = c < p.experts ? ld_value<DT>(row, c) : -INFINITY;
        }
    }
}

// What the partial sums' last reader makes of them: sums [experts + 1], hits
// [experts + 2] in shared memory, complete and visible.
__device__ __forceinline__ void finish_losses(const RouteParams &p, float *sums, const int32_t *hits)
{
    const uint32_t E = p.experts;
    const float n = fmaxf((float)hits[E], 1.0f), inv = __fdiv_rn(1.0f, fmaxf((float)hits[E + 1], 1.0f));
    for (uint32_t e = threadIdx.x; e < E; e += blockDim.x) {
        const float load = __fmul_rn((float)hits[e], inv), importance = __fdiv_rn(sums[e], n);
        gstore<int32_t>(p.counts + e, hits[e]);
        gstore<float>(p.load + e, load);
        gstore<float>(p.importance + e, importance);
        sums[e] = __fmul_rn(load, importance);
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        float b = 0.0f;
        for (uint32_t e = threadIdx.x; e < E; e += 32)
            b = __fadd_rn(b, sums[e]);
        b = group_sum<32>(b);
        if (threadIdx.x == 0) {
            gstore<int32_t>(p.counts + E, hits[E]);
            gstore<float>(p.loss, __fmul_rn((float)E, b));
            gstore<float>(p.loss + 1, __fdiv_rn(sums[E], n));
        }
    }
}

// L lanes a row, V values a lane, loads of N values; the block has whole warps.
// 16384 x 256 fp32, 8 choices: 22.8 us, bound by the choices' instructions (two
// reductions and a pass over a lane's values each); 8 x 64 3.3 us.
template <int DT, int L, int V, int N> __global__ void __launch_bounds__(route_threads(V)) route_kernel(const __grid_constant__ RouteParams p)
{
    chain_entry();
    extern __shared__ float shared[]; // sums [warps][experts + 1], hits [experts + 2]
    const uint32_t E = p.experts, warps = blockDim.x / 32, groups = blockDim.x / L;
    int32_t *hits = reinterpret_cast<int32_t *>(shared + warps * (E + 1));
    const uint32_t lane = threadIdx.x % L, group = threadIdx.x / L, warp = threadIdx.x / 32;
    for (uint32_t e = threadIdx.x; e < E + 2; e += blockDim.x)
        hits[e] = 0;
    __syncthreads();
    float acc[V], square = 0.0f;
    int32_t routed = 0, choices = 0;
#pragma unroll
    for (int i = 0; i < V; ++i)
        acc[i] = 0.0f;
    const uint32_t stride = p.ctas * groups;
    // whole warps go round together: rows past the last are rows without experts
    const uint32_t rounds = (p.ntokens + stride - 1) / stride;
    auto fetch = [&](uint32_t round, float *v) {
        const uint64_t t = (uint64_t)round * stride + group * p.ctas + blockIdx.x; // a partly filled last round falls on every CTA
        if (round < rounds && t < p.ntokens && (!p.valid || gload<uint8_t>(p.valid + t))) {
            load_row<DT, L, V, N>(p, p.logits + t * p.pitch, lane, v);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i)
                v[i] = -INFINITY;
        }
    };
    constexpr bool kAhead = V <= 16; // the next row's values fit beside this one's
    float f[V], next[kAhead ? V : 1];
    if (kAhead)
        fetch(0, f);
    for (uint32_t round = 0; round < rounds; ++round) {
        const uint64_t t = (uint64_t)round * stride + group * p.ctas + blockIdx.x; // a partly filled last round falls on every CTA
        if (kAhead)
            fetch(round + 1, next);
        else
            fetch(round, f);
        uint32_t key[V], best = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            key[i] = ordered(f[i]);
            best = max(best, key[i]);
        }
        const uint32_t top = group_max<L>(best);
        const bool live = top > kNothing;
        // a NaN in the row makes its sum NaN whatever is taken off
        const float m = live && top != kNaN ? from_ordered(top) : 0.0f;
        float total = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            f[i] = exp_of(__fsub_rn(f[i], m)); // 0 for -inf
            total = __fadd_rn(total, f[i]);
        }
        total = group_sum<L>(total);
        const float inv = live ? __fdiv_rn(1.0f, total) : 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i)
            acc[i] = __fmaf_rn(f[i], inv, acc[i]);
        const float lse = live ? __fadd_rn(m, logf(total)) : 0.0f;
        // the choices, one a step: the largest key, at its lowest column; lane s
        // keeps the s-th (and s + L, ...)
        constexpr int kMine = (CCL_MAX_EXPERT_TOP + L - 1) / L;
        uint32_t mine[kMine];
        int32_t id[kMine];
        uint32_t k = top;
#pragma unroll
        for (int s0 = 0; s0 < kMine; ++s0) {
            mine[s0] = kNothing;
            id[s0] = -1;
            if (s0 * L < p.top)
                for (uint32_t s = 0; s < L && s0 * L + s < p.top; ++s) {
                    uint32_t c = 0xffffffffu;
#pragma unroll
                    for (int i = V - 1; i >= 0; --i) // columns rise with i: the first of equals stays
                        c = key[i] == k ? column<L, N>(lane, i) : c;
                    c = group_min<L>(c);
                    if (lane == s && k > kNothing) {
                        mine[s0] = k;
                        id[s0] = (int32_t)c;
                    }
                    best = 0;
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        key[i] = column<L, N>(lane, i) == c ? 0 : key[i]; // out of the running
                        best = max(best, key[i]);
                    }
                    k = group_max<L>(best);
                }
        }
        float w[kMine], kept = 0.0f;
#pragma unroll
        for (int s0 = 0; s0 < kMine; ++s0) {
            w[s0] = id[s0] >= 0 ? exp_of(__fsub_rn(from_ordered(mine[s0]), m)) : 0.0f;
            kept = __fadd_rn(kept, w[s0]);
        }
        const float by = p.normalize ? __fdiv_rn(1.0f, group_sum<L>(kept)) : inv;
        if (t < p.ntokens) {
#pragma unroll
            for (int s0 = 0; s0 < kMine; ++s0) {
                const uint32_t s = s0 * L + lane;
                if (s < p.top) {
                    gstore<int32_t>(p.ids + t * p.top + s, id[s0]);
                    gstore<float>(p.weights + t * p.top + s, id[s0] < 0 ? 0.0f : __fmul_rn(w[s0], by));
                    if (id[s0] >= 0) {
                        atomicAdd(&hits[id[s0]], 1); // whole numbers: any order gives the same count
                        ++choices;
                    }
                }
            }
            if (lane == 0)
                gstore<float>(p.lse + t, lse);
        }
        square = __fmaf_rn(lse, lse, square);
        routed += live;
        if (kAhead) {
#pragma unroll
            for (int i = 0; i < V; ++i)
                f[i] = next[kAhead ? i : 0];
        }
    }
    // the warp's sums, its groups pairwise
#pragma unroll
    for (int d = L; d < 32; d *= 2) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            acc[i] = __fadd_rn(acc[i], __shfl_xor_sync(0xffffffffu, acc[i], d));
        square = __fadd_rn(square, __shfl_xor_sync(0xffffffffu, square, d));
        routed += __shfl_xor_sync(0xffffffffu, routed, d);
    }
    choices = __reduce_add_sync(0xffffffffu, choices);
    float *mine = shared + warp * (E + 1);
    if (threadIdx.x % 32 < L) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const uint32_t c = column<L, N>(lane, i);
            if (c < E)
                mine[c] = acc[i];
        }
    }
    if (threadIdx.x % 32 == 0) {
        mine[E] = square;
        atomicAdd(&hits[E], routed);
        atomicAdd(&hits[E + 1], choices);
    }
    __syncthreads();
    // the CTA's, its warps in order; each column is one thread's from here on
    for (uint32_t e = threadIdx.x; e <= E; e += blockDim.x) {
        float v = shared[e];
        for (uint32_t k = 1; k < warps; ++k)
            v = __fadd_rn(v, shared[k * (E + 1) + e]);
        if (p.ctas == 1)
            shared[e] = v;
        else
            gstore<float>(p.sums + (uint64_t)blockIdx.x * (E + 1) + e, v);
    }
    if (p.ctas == 1) {
        __syncthreads();
        finish_losses(p, shared, hits);
    } else {
        for (uint32_t e = threadIdx.x; e < E + 2; e += blockDim.x)
            gstore<int32_t>(p.hits + (uint64_t)blockIdx.x * (E + 2) + e, hits[e]);
    }
}

// The CTAs' partial sums, by one cluster: each of its CTAs takes a run of rows,
// 1024 / columns threads a column take parts of it, eight loads in flight, and
// the parts, then the runs, are joined in order.
__global__ void __cluster_dims__(kJoinCtas) __launch_bounds__(1024) route_join_kernel(const __grid_constant__ RouteParams p)
{
    chain_entry();
    cg::cluster_group cluster = cg::this_cluster();
    extern __shared__ float shared[]; // sums [parts][columns], hits [parts][columns]
    const uint32_t n = p.experts + 2, parts = max(1024u / n, 1u), per = (p.ctas + kJoinCtas - 1) / kJoinCtas, run = (per + parts - 1) / parts;
    const uint32_t first = min(cluster.block_rank() * per, p.ctas), past = min(first + per, p.ctas);
    float *sums = shared;
    int32_t *hits = reinterpret_cast<int32_t *>(shared + parts * n);
    for (uint32_t i = threadIdx.x; i < parts * n; i += 1024) {
        const uint32_t part = i / n, c = i - part * n, b1 = min(first + (part + 1) * run, past);
        float s = 0.0f;
        int32_t h = 0;
        for (uint32_t b0 = first + part * run; b0 < b1; b0 += 8) {
            float x[8];
            int32_t y[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                x[j] = b0 + j < b1 && c + 1 < n ? gload<float>(p.sums + (uint64_t)(b0 + j) * (n - 1) + c) : 0.0f;
                y[j] = b0 + j < b1 ? gload<int32_t>(p.hits + (uint64_t)(b0 + j) * n + c) : 0;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                s = __fadd_rn(s, x[j]);
                h += y[j];
            }
        }
        sums[i] = s;
        hits[i] = h;
    }
    __syncthreads();
    for (uint32_t c = threadIdx.x; c < n; c += 1024) {
        float s = sums[c];
        int32_t h = hits[c];
        for (uint32_t k = 1; k < parts; ++k) {
            s = __fadd_rn(s, sums[k * n + c]);
            h += hits[k * n + c];
        }
        sums[c] = s;
        hits[c] = h;
    }
    cluster.sync();
    if (cluster.block_rank() == 0)
        for (uint32_t c = threadIdx.x; c < n; c += 1024) {
            float s[kJoinCtas];
            int32_t h[kJoinCtas];
#pragma unroll
            for (int k = 0; k < kJoinCtas; ++k) {
                s[k] = cluster.map_shared_rank(sums, k)[c];
                h[k] = cluster.map_shared_rank(hits, k)[c];
            }
#pragma unroll
            for (int k = 1; k < kJoinCtas; ++k) {
                s[0] = __fadd_rn(s[0], s[k]);
                h[0] += h[k];
            }
            sums[c] = s[0];
            hits[c] = h[0];
        }
    cluster.sync(); // the others' memory has been read
    if (cluster.block_rank() == 0)
        finish_losses(p, sums, hits);
}

// A group of L lanes a row, which it reads once; `pull` in registers, since the
// lanes' vectors of columns meet in the same banks (131072 x 256 bf16: 79 -> 56
// us, single elements 65, with exp(z - lse) for p).  More rows' loads in flight
// (the row's before its ids are there) gained nothing.  p is made as the forward
// pass makes it, exp(z - m) over its sum: exp(z - lse) carries the rounding of
// lse, |lse| 2^-24 of p, and is 1 for every expert of a row of -1e9.  The sums of
// a row are reduced side by side (calls in a graph, with exp(z - lse), with the
// maximum and the sums one after another, and as it is: 131072 x 256 bf16 62.3,
// 68.7, 66.8 us; 131072 x 64 25.9, 26.8, 24.7; 16384 x 256 fp32 10.4, 10.5, 10.2;
// 8 x 64 2.5, 2.5, 2.4).
template <int DT, int L, int V, int N> __global__ void __launch_bounds__(kRouteThreads) route_grad_kernel(const __grid_constant__ RouteParams p)
{
    chain_entry();
    extern __shared__ float pull[]; // balance * experts / n * load
    constexpr int kGroups = kRouteThreads / L;
    const uint32_t lane = threadIdx.x % L, group = threadIdx.x / L, E = p.experts;
    const float n = fmaxf((float)gload<int32_t>(p.counts + E), 1.0f);
    const float b = __fdiv_rn(__fmul_rn(p.balance, (float)E), n);
    for (uint32_t e = threadIdx.x; e < E; e += kRouteThreads)
        pull[e] = __fmul_rn(b, gload<float>(p.load + e));
    __syncthreads();
    float own[V]; // of this lane's columns
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const uint32_t c = column<L, N>(lane, i);
        own[i] = c < E ? pull[c] : 0.0f;
    }
    const float cz = __fdiv_rn(__fmul_rn(2.0f, p.z), n);
    const uint32_t stride = gridDim.x * kGroups, rounds = (p.ntokens + stride - 1) / stride;
    for (uint32_t round = 0; round < rounds; ++round) {
        const uint64_t t = (uint64_t)round * stride + blockIdx.x * kGroups + group;
        const bool in = t < p.ntokens;
        constexpr int kMine = (CCL_MAX_EXPERT_TOP + L - 1) / L;
        int32_t id[kMine];
        float g[kMine], q[kMine];
        bool any = false;
#pragma unroll
        for (int s0 = 0; s0 < kMine; ++s0) {
            const uint32_t s = s0 * L + lane;
            id[s0] = in && s < p.top ? gload<int32_t>(p.ids + t * p.top + s) : -1;
            if ((uint32_t)id[s0] >= E)
                id[s0] = -1;
            g[s0] = id[s0] >= 0 ? gload<float>(p.grad_weights + t * p.top + s) : 0.0f;
            any |= id[s0] >= 0;
        }
        const bool live = group_max<L>(any ? 1u : 0u);
        const float lse = live ? gload<float>(p.lse + t) : 0.0f;
        const char *row = p.logits + (live ? t : 0) * p.pitch;
        float f[V], best = -INFINITY;
#pragma unroll
        for (int i = 0; i < V; ++i)
            f[i] = -INFINITY;
        if (live)
            load_row<DT, L, V, N>(p, row, lane, f);
#pragma unroll
        for (int i = 0; i < V; ++i)
            best = fmaxf(best, f[i]); // a NaN makes the sum one
        const uint32_t most = group_max<L>(ordered(best));
        const float m = most > kNothing ? from_ordered(most) : 0.0f;
        // the row's sums side by side, of exp(z - m): of all, with the balance
        // loss's pull, of the chosen, with their weights' gradients
        float total = 0.0f, pulled = 0.0f, kept = 0.0f, gw = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            f[i] = exp_of(__fsub_rn(f[i], m));
            total = __fadd_rn(total, f[i]);
            pulled = __fmaf_rn(own[i], f[i], pulled);
        }
#pragma unroll
        for (int s0 = 0; s0 < kMine; ++s0) {
            q[s0] = id[s0] >= 0 ? exp_of(__fsub_rn(ld_value<DT>(row, (uint32_t)id[s0]), m)) : 0.0f;
            kept = __fadd_rn(kept, q[s0]);
            gw = __fmaf_rn(g[s0], q[s0], gw);
        }
        total = group_sum<L>(total);
        pulled = group_sum<L>(pulled);
        kept = group_sum<L>(kept);
        gw = group_sum<L>(gw);
        const float by = total != 0.0f ? __fdiv_rn(1.0f, total) : 0.0f;
        // sum_i G_i p_i: the normalised weights' part is 0, their sum being constant
        // (times 0, so that a gradient that is NaN or infinite shows in the whole row)
        const float inner = __fmaf_rn(gw, p.normalize ? 0.0f : by, __fmul_rn(pulled, by));
        if (p.normalize && live) {
            const float inv = __fdiv_rn(1.0f, kept), mean = __fmul_rn(gw, inv), each = __fmul_rn(total, inv);
#pragma unroll
            for (int s0 = 0; s0 < kMine; ++s0)
                g[s0] = id[s0] >= 0 ? __fmul_rn(__fsub_rn(g[s0], mean), each) : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < V; ++i)
            f[i] = column<L, N>(lane, i) < E ? __fmul_rn(f[i], by) : 0.0f;
#pragma unroll
        for (int s0 = 0; s0 < kMine; ++s0)
            q[s0] = __fmul_rn(q[s0], by);
        const float off = __fmaf_rn(cz, lse, -inner);
        if (in) {
            char *out = p.grad + t * p.grad_pitch;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const uint32_t c = column<L, N>(lane, i);
                f[i] = c < E ? __fmul_rn(f[i], __fadd_rn(own[i], off)) : 0.0f;
            }
            if (N > 1) {
#pragma unroll
                for (int i = 0; i < V; i += N) {
                    const uint32_t c = column<L, N>(lane, i);
                    if (c < E) {
                        char *at = out + (uint64_t)c * DType<DT>::kSize;
                        float h[DType<DT>::kVec];
#pragma unroll
                        for (int k = 0; k < DType<DT>::kVec; ++k)
                            h[k] = k < N ? f[i + (k < N ? k : 0)] : 0.0f;
                        const uint4 v = pack<DT>(h);
                        if (N * DType<DT>::kSize == 16)
                            st16(at, v);
                        else if (N * DType<DT>::kSize == 8)
                            gstore<uint2>(at, make_uint2(v.x, v.y));
                        else
                            gstore<uint32_t>(at, v.x);
                    }
                }
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const uint32_t c = column<L, 1>(lane, i);
                    if (c < E)
                        st_value<DT>(out, c, f[i]);
                }
            }
        }
        __syncwarp();
        // the chosen experts' entries again, with what their weights' gradients add
        if (in) {
            char *out = p.grad + t * p.grad_pitch;
#pragma unroll
            for (int s0 = 0; s0 < kMine; ++s0)
                if (id[s0] >= 0)
                    st_value<DT>(out, (uint32_t)id[s0], __fmul_rn(q[s0], __fadd_rn(__fadd_rn(pull[id[s0]], g[s0]), off)));
        }
    }
}

// ------------------------------------------------------------------ host side

struct RoutePlan {
    uint32_t lanes, threads, ctas;
    size_t sums, bytes;
};

bool plan_route(size_t ntokens, size_t experts, RoutePlan *p)
{
    if (ntokens > kMaxTokens || experts == 0 || experts > CCL_MAX_EXPERTS)
        return false;
    *p = RoutePlan{};
    p->lanes = experts <= 64 ? 8 : 32; // 16384 x 64: 8 lanes 9.0 us, 32 lanes 12.1
    const size_t most = route_threads(experts <= 256 ? 8 : experts <= 512 ? 16 : 32);
    if (ntokens * p->lanes <= most) { // one CTA, which needs no second launch
        p->ctas = 1;
        p->threads = (uint32_t)std::max<size_t>(ntokens * p->lanes + 31, 32) / 32 * 32;
    } else {
        const size_t rows = kFewRouteThreads / p->lanes; // that the smallest CTA takes at a time
        p->ctas = (uint32_t)std::min<size_t>((ntokens + rows - 1) / rows, experts <= 512 ? kSms : 2 * kSms);
        p->threads = (uint32_t)std::min(most, std::max(kFewRouteThreads, ((ntokens + p->ctas - 1) / p->ctas * p->lanes + 31) / 32 * 32));
    }
    if (p->ctas > 1) {
        p->sums = up(p->ctas * (experts + 1) * 4);
        p->bytes = p->sums + up(p->ctas * (experts + 2) * 4);
    }
    return true;
}

template <int DT, int L, int V, bool GRAD> cudaError_t launch_route3(const RouteParams &p, unsigned ctas, unsigned threads, cudaStream_t stream)
{
    constexpr int N = V < DType<DT>::kVec ? V : DType<DT>::kVec;
    const size_t smem = GRAD ? p.experts * 4 : (threads / 32 * (p.experts + 1) + p.experts + 2) * 4;
    void (*const vec)(RouteParams) = GRAD ? route_grad_kernel<DT, L, V, N> : route_kernel<DT, L, V, N>;
    void (*const one)(RouteParams) = GRAD ? route_grad_kernel<DT, L, V, 1> : route_kernel<DT, L, V, 1>;
    const uintptr_t all = (uintptr_t)p.logits | p.pitch | p.experts * DType<DT>::kSize | (GRAD ? (uintptr_t)p.grad | p.grad_pitch : 0);
    return launch_chained(all % (N * DType<DT>::kSize) == 0 ? vec : one, dim3(ctas), dim3(threads), smem, stream, p);
}

template <int DT, bool GRAD> cudaError_t launch_route2(const RouteParams &p, unsigned ctas, unsigned threads, cudaStream_t stream)
{
    if (p.experts <= 16)
        return launch_route3<DT, 8, 2, GRAD>(p, ctas, threads, stream);
    if (p.experts <= 64)
        return launch_route3<DT, 8, 8, GRAD>(p, ctas, threads, stream);
    if (p.experts <= 256)
        return launch_route3<DT, 32, 8, GRAD>(p, ctas, threads, stream);
    if (p.experts <= 512)
        return launch_route3<DT, 32, 16, GRAD>(p, ctas, threads, stream);
    return launch_route3<DT, 32, 32, GRAD>(p, ctas, threads, stream);
}

template <bool GRAD> cudaError_t launch_route(ccl_dtype_t dtype, const RouteParams &p, unsigned ctas, unsigned threads, cudaStream_t stream)
{
    const cudaError_t e = dtype == CCL_FP32 ? launch_route2<DT_FP32, GRAD>(p, ctas, threads, stream) : launch_route2<DT_BF16, GRAD>(p, ctas, threads, stream);
    if (e == cudaSuccess)
        count_launches(1);
    return e;
}

ccl_status_t route_impl(const void *logits, size_t ntokens, size_t experts, size_t stride, ccl_dtype_t dtype, const uint8_t *valid, size_t top,
                        int normalize, int32_t *ids, float *weights, float *lse, int32_t *counts, float *load, float *importance, float *loss,
                        void *work, size_t work_bytes, cudaStream_t stream)
{
    RoutePlan pl;
    size_t lb;
    if (!valid_dtype(dtype) || !plan_route(ntokens, experts, &pl) || stride < experts || top == 0 || top > experts || top > CCL_MAX_EXPERT_TOP ||
        !extent(ntokens, experts, stride, elem_size(dtype), &lb))
        return CCL_ERR_INVALID_ARG;
    if (ntokens * top > kMaxTokens) // choices are counted in 32 bits
        return CCL_ERR_INVALID_ARG;
    if (!counts || !load || !importance || !loss || (ntokens && (!logits || !lse || !ids || !weights)) ||
        !element_aligned(elem_size(dtype), {logits}) || !element_aligned(4, {ids, weights, lse, counts, load, importance, loss}) ||
        (pl.bytes && (!work || (uintptr_t)work % 256 || work_bytes < pl.bytes)))
        return CCL_ERR_INVALID_ARG;
    const size_t choices = ntokens * top;
    const std::vector<Range> w{range_of(ids, choices * 4, 0), range_of(weights, choices * 4, 0), range_of(lse, ntokens * 4, 0),
                               range_of(counts, (experts + 1) * 4, 0), range_of(load, experts * 4, 0), range_of(importance, experts * 4, 0),
                               range_of(loss, 8, 0), range_of(work, pl.bytes, 0)},
        r{range_of(logits, lb, 0), range_of(valid, valid ? ntokens : 0, 0)};
    if (ccl_status_t st = check_overlaps(w, r, [](const Range &, const Range &) { return false; }))
        return st;
#ifdef CCL_DEBUG_BOUNDS
    std::vector<DbgRange> rg;
    for (const std::vector<Range> *v : {&w, &r})
        for (const Range &x : *v)
            rg.push_back(DbgRange{reinterpret_cast<const void *>(x.lo), (size_t)(x.hi - x.lo)});
    if (cudaError_t e = dbg_set_ranges(rg, stream))
        return from_cuda(e);
#endif
    RouteParams p{};
    p.logits = static_cast<const char *>(logits);
    p.pitch = stride * elem_size(dtype);
    p.valid = valid;
    p.ids = ids;
    p.weights = weights;
    p.lse = lse;
    p.counts = counts;
    p.load = load;
    p.importance = importance;
    p.loss = loss;
    p.sums = static_cast<float *>(work);
    p.hits = reinterpret_cast<int32_t *>(static_cast<char *>(work) + pl.sums);
    p.ntokens = (uint32_t)ntokens;
    p.experts = (uint32_t)experts;
    p.top = (uint32_t)top;
    p.ctas = pl.ctas;
    p.normalize = normalize != 0;
    cudaError_t e = launch_route<false>(dtype, p, pl.ctas, pl.threads, stream);
    if (e == cudaSuccess && pl.ctas > 1) {
        const size_t n = experts + 2, parts = std::max<size_t>(1024 / n, 1);
        e = launch_chained(route_join_kernel, dim3(kJoinCtas), dim3(1024), parts * n * 8, stream, p);
        if (e == cudaSuccess)
            count_launches(1);
    }
    return from_cuda(e);
}

ccl_status_t route_grad_impl(const void *logits, size_t ntokens, size_t experts, size_t stride, ccl_dtype_t dtype, const int32_t *ids, size_t top,
                             int normalize, const float *lse, const int32_t *counts, const float *load, const float *grad_weights, float balance,
                             float z, void *grad, size_t grad_stride, cudaStream_t stream)
{
    RoutePlan pl;
    size_t lb, gb;
    const size_t es = elem_size(dtype);
    if (!valid_dtype(dtype) || !plan_route(ntokens, experts, &pl) || stride < experts || grad_stride < experts || top == 0 || top > experts ||
        top > CCL_MAX_EXPERT_TOP || !extent(ntokens, experts, stride, es, &lb) || !extent(ntokens, experts, grad_stride, es, &gb) ||
        balance != balance || z != z)
        return CCL_ERR_INVALID_ARG;
    if (ntokens * top > kMaxTokens)
        return CCL_ERR_INVALID_ARG;
    if (ntokens == 0)
        return CCL_OK;
    if (!logits || !grad || !lse || !counts || !load || !ids || !grad_weights || !element_aligned(es, {logits, grad}) ||
        !element_aligned(4, {ids, lse, counts, load, grad_weights}))
        return CCL_ERR_INVALID_ARG;
    const size_t choices = ntokens * top;
    // in place: the gradient may take the logits' place, row by row
    const bool in_place = grad == logits && grad_stride == stride;
    const std::vector<Range> w{range_of(grad, gb, 1)},
        r{range_of(logits, lb, 1), range_of(ids, choices * 4, 0), range_of(lse, ntokens * 4, 0), range_of(counts, (experts + 1) * 4, 0),
          range_of(load, experts * 4, 0), range_of(grad_weights, choices * 4, 0)};
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
    RouteParams p{};
    p.logits = static_cast<const char *>(logits);
    p.pitch = stride * es;
    p.grad = static_cast<char *>(grad);
    p.grad_pitch = grad_stride * es;
    p.ids = const_cast<int32_t *>(ids);
    p.lse = const_cast<float *>(lse);
    p.counts = const_cast<int32_t *>(counts);
    p.load = const_cast<float *>(load);
    p.grad_weights = grad_weights;
    p.balance = balance;
    p.z = z;
    p.ntokens = (uint32_t)ntokens;
    p.experts = (uint32_t)experts;
    p.top = (uint32_t)top;
    p.normalize = normalize != 0;
    const size_t groups = kRouteThreads / pl.lanes;
    return from_cuda(launch_route<true>(dtype, p, (unsigned)std::min<size_t>((ntokens + groups - 1) / groups, 8 * 152), kRouteThreads, stream));
}

} // namespace
} // namespace ccl

using namespace ccl;

extern "C" {

ccl_status_t ccl_plan_route_work_bytes(size_t ntokens, size_t experts, size_t *bytes)
{
    RoutePlan p;
    if (!bytes || !plan_route(ntokens, experts, &p))
        return CCL_ERR_INVALID_ARG;
    *bytes = p.bytes;
    return CCL_OK;
}

ccl_status_t ccl_route(const void *logits, size_t ntokens, size_t experts, size_t logits_stride, ccl_dtype_t dtype, const uint8_t *valid, size_t top,
                       int normalize, int32_t *ids, float *weights, float *lse, int32_t *counts, float *load, float *importance, float *losses,
                       void *work, size_t work_bytes, cudaStream_t stream)
{
    TraceScope tr("route", 1, ntokens, (int)dtype, -1, 0, stream);
    return tr.done(guarded([&] {
        return route_impl(logits, ntokens, experts, logits_stride, dtype, valid, top, normalize, ids, weights, lse, counts, load, importance, losses,
                          work, work_bytes, stream);
    }));
}

ccl_status_t ccl_route_grad(const void *logits, size_t ntokens, size_t experts, size_t logits_stride, ccl_dtype_t dtype, const int32_t *ids, size_t top,
                            int normalize, const float *lse, const int32_t *counts, const float *load, const float *grad_weights, float balance,
                            float z, void *grad_logits, size_t grad_stride, cudaStream_t stream)
{
    TraceScope tr("route_grad", 1, ntokens, (int)dtype, -1, 0, stream);
    return tr.done(guarded([&] {
        return route_grad_impl(logits, ntokens, experts, logits_stride, dtype, ids, top, normalize, lse, counts, load, grad_weights, balance, z,
                               grad_logits, grad_stride, stream);
    }));
}

} // extern "C"
