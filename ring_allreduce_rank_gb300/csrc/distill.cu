// distill.cu -- distillation loss from a teacher's top logits, and its
// gradient.
//
// Per row: p = softmax over the teacher's K listed logits / tau, q = softmax
// of the student's whole row / tau,
//     loss  = w * sum_j p_j (log p_j - log q_{i_j}),
//     ds_v  = w / tau * (q_v - sum_{j: i_j = v} p_j).
// With m the row's maximum and Z = sum_v exp((s_v - m) / tau), both need one
// pass over the row for (m, Z); the gradient needs the row's values again.
// Bound by memory bandwidth: a CTA streams its row once for (m, Z), with the
// next vectors' loads in flight under the current ones' exponentials, and reads
// it again from the L2 cache for the gradient, so that memory sees one read of
// the logits and one write of the gradient.  Where there are few rows, a
// cluster of CTAs shares each one and joins (m, Z) through distributed shared
// memory.
#include <cooperative_groups.h>

#include <vector>

#include "../../include/ccl.h"
#include "ccl_internal.h"
#include "step_ops.cuh"

namespace cg = cooperative_groups;

namespace ccl {
namespace {

constexpr int kDThreads = 256;
constexpr int kDWarps = kDThreads / 32;
constexpr int kDCtas = 4;        // resident CTAs per SM
constexpr int kVecs = 4;         // 16-byte vectors a thread loads at a time
constexpr int kMaxCluster = 8;   // portable cluster size
constexpr int kMaxTop = CCL_MAX_TEACHER_TOP;
constexpr float kLog2e = 1.4426950408889634f;

enum DistillMode { DISTILL_LOSS = 0, DISTILL_FUSED = 1, DISTILL_GRAD = 2 };

struct DistillParams {
    const char *logits;
    char *grad;
    const int64_t *ids;
    const float *teacher;
    const float *weights;
    float *loss;
    float *stats;         // (m, Z) of every row: written by the loss, read by DISTILL_GRAD
    uint64_t vocab;
    uint64_t pitch, grad_pitch; // bytes
    uint64_t top;
    float scale;          // log2(e) / tau
    float inv_tau;
};

__device__ __forceinline__ float exp2_approx(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// exp((s - m) / tau): the difference first, so that a row of one value, the
// type's lowest included, gives 1 and not an overflow of s * scale.
__device__ __forceinline__ float row_exp(float s, float m, float scale)
{
    return exp2_approx(__fmul_rn(__fsub_rn(s, m), scale));
}

struct Stat {
    float m, z;
};

// ------------------------------------------------------------------ two fp32 values at a time

__device__ __forceinline__ float2 add2(const float2 &a, const float2 &b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(reinterpret_cast<const uint64_t &>(a)), "l"(reinterpret_cast<const uint64_t &>(b)));
    return reinterpret_cast<const float2 &>(r);
}

__device__ __forceinline__ float2 mul2(const float2 &a, const float2 &b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(reinterpret_cast<const uint64_t &>(a)), "l"(reinterpret_cast<const uint64_t &>(b)));
    return reinterpret_cast<const float2 &>(r);
}

// row_exp of a pair; neg_m holds -m twice, scale the scale twice
__device__ __forceinline__ float2 row_exp2(const float2 &s, const float2 &neg_m, const float2 &scale)
{
    const float2 x = mul2(add2(s, neg_m), scale);
    return make_float2(exp2_approx(x.x), exp2_approx(x.y));
}

// The pairs of a 16-byte vector.
template <int DT> __device__ __forceinline__ void unpack2(const uint4 &v, float2 *f)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < DType<DT>::kVec / 2; ++i)
        f[i] = DT == DT_FP32 ? make_float2(__uint_as_float(w[(2 * i) & 3]), __uint_as_float(w[(2 * i + 1) & 3]))
                             : make_float2(__uint_as_float(w[i & 3] << 16), __uint_as_float(w[i & 3] & 0xffff0000u));
}

// The largest value of kVecs vectors; a NaN does not count (it reaches the sum).
template <int DT> __device__ __forceinline__ float max_of(const uint4 *x)
{
    if (DT == DT_FP32) {
        float m = -INFINITY;
#pragma unroll
        for (int i = 0; i < kVecs; ++i)
            m = fmaxf(m, fmaxf(fmaxf(__uint_as_float(x[i].x), __uint_as_float(x[i].y)),
                               fmaxf(__uint_as_float(x[i].z), __uint_as_float(x[i].w))));
        return m;
    }
    uint32_t m = 0xff80ff80u; // -inf twice
    auto up = [&](uint32_t w) { asm("max.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(w)); };
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        up(x[i].x);
        up(x[i].y);
        up(x[i].z);
        up(x[i].w);
    }
    return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
}

// The statistics of two parts of a row.
__device__ __forceinline__ Stat join(const Stat &a, const Stat &b, float scale)
{
    Stat r;
    r.m = fmaxf(a.m, b.m);
    const float za = a.m == r.m ? a.z : __fmul_rn(a.z, row_exp(a.m, r.m, scale));
    const float zb = b.m == r.m ? b.z : __fmul_rn(b.z, row_exp(b.m, r.m, scale));
    r.z = __fadd_rn(za, zb);
    return r;
}

__device__ __forceinline__ Stat warp_join(Stat s, float scale)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        Stat t;
        t.m = __shfl_xor_sync(0xffffffffu, s.m, o);
        t.z = __shfl_xor_sync(0xffffffffu, s.z, o);
        s = join(s, t, scale);
    }
    return s;
}

template <bool MAX> __device__ __forceinline__ float block_reduce(float v, float *buf)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const float u = __shfl_xor_sync(0xffffffffu, v, o);
        v = MAX ? fmaxf(v, u) : __fadd_rn(v, u);
    }
    __syncthreads(); // the buffer's last use
    if (lane == 0)
        buf[warp] = v;
    __syncthreads();
    v = buf[lane & (kDWarps - 1)];
#pragma unroll
    for (int o = kDWarps / 2; o; o >>= 1) {
        const float u = __shfl_xor_sync(0xffffffffu, v, o);
        v = MAX ? fmaxf(v, u) : __fadd_rn(v, u);
    }
    return v;
}

// One cluster per row.  The row's 16-byte vectors are shared out over the
// cluster's CTAs in contiguous parts; the elements before the first 16-byte
// boundary and after the last one (fewer than a vector each) are CTA 0's.
template <int DT, int MODE>
__global__ void __launch_bounds__(kDThreads, kDCtas) distill_kernel(const __grid_constant__ DistillParams p)
{
    constexpr int VEC = DType<DT>::kVec, ES = DType<DT>::kSize;
    constexpr uint32_t kNone = 0xffffffffu;
    constexpr uint32_t kStep = kVecs * kDThreads; // vectors of one load by the CTA
    __shared__ uint32_t id[kMaxTop];
    __shared__ float prob[kMaxTop];  // p_j, 0 for entries that do not count
    __shared__ float logit[kMaxTop]; // the student's logit at id j
    __shared__ float red[kDWarps];
    __shared__ Stat wstat[kDWarps];
    __shared__ Stat cstat; // this CTA's part of the row, read by the cluster
    cg::cluster_group cluster = cg::this_cluster();
    const uint32_t ctas = cluster.num_blocks(), cta = cluster.block_rank();
    const uint64_t t = blockIdx.x / ctas;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int top = (int)p.top;

    const float w = p.weights ? gload<float>(p.weights + t) : 1.0f;
    const char *row = p.logits + t * p.pitch;
    char *grow = MODE == DISTILL_LOSS ? nullptr : p.grad + t * p.grad_pitch;
    const uint32_t nh = (uint32_t)umin64(p.vocab, ((16 - ((uintptr_t)row & 15)) & 15) / ES);
    const uint32_t nv = ((uint32_t)p.vocab - nh) / VEC, nt = (uint32_t)p.vocab - nh - nv * VEC;
    const uint32_t per = (nv + ctas - 1) / ctas, v0 = min(nv, per * cta), v1 = min(nv, v0 + per);
    const uint32_t loads = (v1 - v0 + kStep - 1) / kStep;
    const char *body = row + (uint64_t)nh * ES;
    // an edge element: head, then tail
    const bool edge = cta == 0 && tid < (int)(nh + nt);
    const uint32_t ei = tid < (int)nh ? tid : (uint32_t)p.vocab - nt + (tid - nh);
    // a row whose weight is 0 has loss 0 and gradient 0 whatever it holds
    // (its statistics are still wanted where the caller keeps them)
    const bool skip = w == 0.0f && (MODE == DISTILL_GRAD || !p.stats);

    // the vectors of one load; past the part's end -inf, which adds nothing
    auto load = [&](uint4 *x, uint32_t l) {
        const uint32_t b = v0 + l * kStep + tid;
        constexpr uint32_t kNinf = DT == DT_FP32 ? 0xff800000u : 0xff80ff80u;
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            x[i] = make_uint4(kNinf, kNinf, kNinf, kNinf);
            if (b + i * kDThreads < v1)
                x[i] = ld16(body + (uint64_t)(b + i * kDThreads) * 16);
        }
    };
    uint4 xa[kVecs], xb[kVecs];
    float xe = 0.0f;
    if (!skip) {
        load(xa, 0);
        if (edge)
            xe = ld_value<DT>(row, ei);
    }
    // whether element i of the row is in this CTA's part
    auto mine = [&](uint32_t i) {
        if (i < nh || i >= nh + nv * VEC)
            return cta == 0;
        const uint32_t v = (i - nh) / VEC;
        return v >= v0 && v < v1;
    };

    // the teacher's probabilities; the loss is CTA 0's
    const bool listed = !skip && (MODE != DISTILL_LOSS || cta == 0);
    float tm = -INFINITY;
    if (listed)
        for (int j = tid; j < top; j += kDThreads) {
            const int64_t i = gload<int64_t>(p.ids + t * p.top + j);
            const bool ok = (uint64_t)i < p.vocab;
            const float l = ok ? gload<float>(p.teacher + t * p.top + j) : -INFINITY;
            id[j] = ok ? (uint32_t)i : kNone;
            prob[j] = l;
            // CTA 0 needs every listed logit for the loss, the others their own
            if (ok && (mine((uint32_t)i) || (MODE != DISTILL_GRAD && cta == 0)))
                logit[j] = ld_value<DT>(row, (uint64_t)i);
            // a NaN counts as present, so that it reaches the result
            tm = l != l ? INFINITY : fmaxf(tm, l);
        }
    tm = block_reduce<true>(tm, red);
    const bool some = tm > -INFINITY;
    float tz = 0.0f;
    if (some)
        for (int j = tid; j < top; j += kDThreads) {
            const float e = id[j] != kNone ? exp2f(__fmul_rn(__fsub_rn(prob[j], tm), p.scale)) : 0.0f;
            prob[j] = e;
            tz = __fadd_rn(tz, e);
        }
    tz = block_reduce<false>(tz, red);
    if (some)
        for (int j = tid; j < top; j += kDThreads)
            prob[j] = __fdiv_rn(prob[j], tz);

    Stat st{-INFINITY, 0.0f};
    const float2 scale2 = make_float2(p.scale, p.scale);
    if (MODE == DISTILL_GRAD) {
        st.m = gload<float>(p.stats + 2 * t);
        st.z = gload<float>(p.stats + 2 * t + 1);
        __syncthreads();
    } else {
        // (m, Z): this thread's vectors, then warp, CTA and cluster
        if (!skip) {
            float2 z = make_float2(0.0f, 0.0f);
            auto fold = [&](const uint4 *x) {
                const float bm = max_of<DT>(x);
                if (bm > st.m) { // the sum so far, relative to the new maximum
                    const float r = row_exp(st.m, bm, p.scale);
                    z = mul2(z, make_float2(r, r));
                    st.m = bm;
                }
                if (st.m == -INFINITY) { // nothing yet but -inf, and perhaps a NaN
#pragma unroll
                    for (int i = 0; i < kVecs; ++i) {
                        float f[VEC];
                        unpack<DT>(x[i], f);
#pragma unroll
                        for (int k = 0; k < VEC; ++k)
                            z.x = f[k] != f[k] ? f[k] : z.x;
                    }
                    return;
                }
                const float2 neg = make_float2(-st.m, -st.m);
#pragma unroll
                for (int i = 0; i < kVecs; ++i) {
                    float2 f[VEC / 2];
                    unpack2<DT>(x[i], f);
#pragma unroll
                    for (int k = 0; k < VEC / 2; ++k)
                        f[k] = row_exp2(f[k], neg, scale2);
#pragma unroll
                    for (int o = VEC / 4; o; o >>= 1)
#pragma unroll
                        for (int k = 0; k < o; ++k)
                            f[k] = add2(f[k], f[k + o]);
                    z = add2(z, f[0]);
                }
            };
            for (uint32_t l = 0; l < loads; l += 2) {
                if (l + 1 < loads)
                    load(xb, l + 1);
                fold(xa);
                if (l + 2 < loads)
                    load(xa, l + 2);
                if (l + 1 < loads)
                    fold(xb);
            }
            st.z = __fadd_rn(z.x, z.y);
            if (edge)
                st = join(st, Stat{xe, xe == -INFINITY ? 0.0f : row_exp(xe, xe, p.scale)}, p.scale);
        }
        st = warp_join(st, p.scale);
        if (lane == 0)
            wstat[warp] = st;
        __syncthreads();
        if (warp == 0) {
            st = lane < kDWarps ? wstat[lane] : Stat{-INFINITY, 0.0f};
            st = warp_join(st, p.scale);
            if (lane == 0)
                cstat = st;
        }
        // from here on a CTA may overwrite its part of the logits (in place):
        // every read of another CTA's part is above
        cluster.sync();
        st = *cluster.map_shared_rank(&cstat, 0);
        for (uint32_t c = 1; c < ctas; ++c)
            st = join(st, *cluster.map_shared_rank(&cstat, c), p.scale);
        if (cta == 0) {
            if (p.stats && tid == 0) {
                gstore<float>(p.stats + 2 * t, st.m);
                gstore<float>(p.stats + 2 * t + 1, st.z);
            }
            float sum = 0.0f;
            if (some) {
                const float lz = logf(st.z);
                for (int j = tid; j < top; j += kDThreads)
                    if (!(prob[j] == 0.0f)) {
                        const float logq = __fsub_rn(__fmul_rn(__fsub_rn(logit[j], st.m), p.inv_tau), lz);
                        sum = __fadd_rn(sum, __fmul_rn(prob[j], __fsub_rn(logf(prob[j]), logq)));
                    }
            }
            sum = block_reduce<false>(sum, red);
            if (tid == 0)
                gstore<float>(p.loss + t, w == 0.0f ? 0.0f : __fmul_rn(w, sum));
        }
    }

    if (MODE != DISTILL_LOSS) {
        const float a = __fmul_rn(w, p.inv_tau);
        const bool zero = w == 0.0f || !some;
        const float c = zero ? 0.0f : __fdiv_rn(a, st.z);
        const float2 c2 = make_float2(c, c), neg = make_float2(-st.m, -st.m);
        const bool vec_store = (((uintptr_t)grow ^ (uintptr_t)row) & 15) == 0;
        char *gbody = grow + (uint64_t)nh * ES;
        auto emit = [&](const uint4 *x, uint32_t l) {
            const uint32_t b = v0 + l * kStep + tid;
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                const uint32_t v = b + i * kDThreads;
                float2 f[VEC / 2];
                unpack2<DT>(x[i], f);
#pragma unroll
                for (int k = 0; k < VEC / 2; ++k)
                    f[k] = zero ? make_float2(0.0f, 0.0f) : mul2(row_exp2(f[k], neg, scale2), c2);
                if (v < v1) {
                    const float *g = reinterpret_cast<const float *>(f);
                    if (vec_store) {
                        st16(gbody + (uint64_t)v * 16, pack<DT>(g));
                    } else {
#pragma unroll
                        for (int k = 0; k < VEC; ++k)
                            st_value<DT>(grow, nh + (uint64_t)v * VEC + k, g[k]);
                    }
                }
            }
        };
        const bool again = !skip && (MODE != DISTILL_GRAD ? loads > 1 : false);
        if (again)
            load(xa, 0);
        for (uint32_t l = 0; l < loads; l += 2) {
            if (!skip && l + 1 < loads)
                load(xb, l + 1);
            emit(xa, l);
            if (!skip && l + 2 < loads)
                load(xa, l + 2);
            if (l + 1 < loads)
                emit(xb, l + 1);
        }
        if (edge)
            st_value<DT>(grow, ei, zero ? 0.0f : __fmul_rn(row_exp(xe, st.m, p.scale), c));
        __syncthreads(); // before the listed ids' gradients replace what was written
        // `part` neighbouring threads share an entry's search for its id's other places
        int part = 1;
        while (part < 32 && 2 * part * top <= kDThreads)
            part *= 2;
        if (!zero)
            for (int j0 = 0; j0 < top; j0 += kDThreads / part) {
                const int j = j0 + tid / part;
                const uint32_t i = j < top ? id[j] : kNone;
                const bool own = i != kNone && mine(i);
                float sum = 0.0f;
                int first = top;
                if (own)
                    for (int k = tid % part; k < top; k += part)
                        if (id[k] == i) {
                            first = min(first, k);
                            sum = __fadd_rn(sum, prob[k]);
                        }
                for (int o = 1; o < part; o *= 2) {
                    sum = __fadd_rn(sum, __shfl_xor_sync(0xffffffffu, sum, o));
                    first = min(first, __shfl_xor_sync(0xffffffffu, first, o));
                }
                if (own && first == j && tid % part == 0) {
                    const float q = __fdiv_rn(row_exp(logit[j], st.m, p.scale), st.z);
                    st_value<DT>(grow, i, __fmul_rn(a, __fsub_rn(q, sum)));
                }
            }
    }
    if (MODE != DISTILL_GRAD)
        cluster.sync(); // no CTA leaves while another may read its statistics
}

// ------------------------------------------------------------------ host side

template <int DT, int MODE>
cudaError_t launch_distill(const DistillParams &p, uint64_t rows, uint32_t ctas, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(rows * ctas));
    cfg.blockDim = dim3(kDThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ctas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, distill_kernel<DT, MODE>, p);
    if (e == cudaSuccess)
        count_launches(1);
    return e;
}

struct DistillArgs {
    const void *logits;
    size_t nrows, vocab, stride;
    ccl_dtype_t dtype;
    const int64_t *ids;
    const float *teacher;
    size_t top;
    float temperature;
    const float *weights;
    float *loss, *stats;
    void *grad;
    size_t grad_stride;
};

ccl_status_t distill_impl(int mode, const DistillArgs &a, cudaStream_t stream)
{
    if (!valid_dtype(a.dtype) || a.stride < a.vocab || a.top > kMaxTop || !(a.temperature > 0.0f) ||
        a.temperature == INFINITY || a.nrows > 0x0fffffff || a.vocab > 0x7fffffff ||
        (mode != DISTILL_LOSS && a.grad_stride < a.vocab))
        return CCL_ERR_INVALID_ARG;
    const float inv_tau = 1.0f / a.temperature;
    if (!(inv_tau > 0.0f) || inv_tau * kLog2e == INFINITY)
        return CCL_ERR_INVALID_ARG; // a temperature whose reciprocal fp32 does not hold
    const size_t es = elem_size(a.dtype);
    size_t lb, gb = 0;
    if (!extent(a.nrows, a.vocab, a.stride, es, &lb) ||
        (mode != DISTILL_LOSS && !extent(a.nrows, a.vocab, a.grad_stride, es, &gb)))
        return CCL_ERR_INVALID_ARG;
    if (a.nrows == 0)
        return CCL_OK;
    if ((a.vocab && !a.logits) || (a.top && (!a.ids || !a.teacher)) || (mode != DISTILL_GRAD && !a.loss) ||
        (mode == DISTILL_GRAD && !a.stats) || (mode != DISTILL_LOSS && a.vocab && !a.grad))
        return CCL_ERR_INVALID_ARG;
    // in place: the gradient may take the logits' place, row by row
    const bool in_place = a.grad == a.logits && a.grad_stride == a.stride;
    std::vector<Range> w, r;
    r.push_back(range_of(a.logits, lb, 1));
    r.push_back(range_of(a.ids, a.nrows * a.top * 8, 0));
    r.push_back(range_of(a.teacher, a.nrows * a.top * 4, 0));
    r.push_back(range_of(a.weights, a.weights ? a.nrows * 4 : 0, 0));
    if (mode != DISTILL_LOSS)
        w.push_back(range_of(a.grad, gb, 1));
    if (mode != DISTILL_GRAD)
        w.push_back(range_of(a.loss, a.nrows * 4, 0));
    if (a.stats)
        (mode == DISTILL_GRAD ? r : w).push_back(range_of(a.stats, a.nrows * 8, 0));
    if (ccl_status_t st = check_overlaps(w, r, [&](const Range &x, const Range &y) {
            return in_place && x.rank == 1 && y.rank == 1;
        }))
        return st;
#ifdef CCL_DEBUG_BOUNDS
    std::vector<DbgRange> rg;
    for (const std::vector<Range> *v : {&w, &r})
        for (const Range &x : *v)
            rg.push_back(DbgRange{reinterpret_cast<const void *>(x.lo), (size_t)(x.hi - x.lo)});
    if (cudaError_t e = dbg_set_ranges(rg, stream))
        return from_cuda(e);
#endif
    DistillParams p{};
    p.logits = static_cast<const char *>(a.logits);
    p.grad = static_cast<char *>(a.grad);
    p.ids = a.ids;
    p.teacher = a.teacher;
    p.weights = a.weights;
    p.loss = a.loss;
    p.stats = a.stats;
    p.vocab = a.vocab;
    p.pitch = a.stride * es;
    p.grad_pitch = a.grad_stride * es;
    p.top = a.top;
    p.inv_tau = inv_tau;
    p.scale = inv_tau * kLog2e;
    // one CTA a row; where that leaves CTAs' places on the GPU empty, up to
    // eight, as long as each has a full load of vectors
    const uint64_t bytes = a.vocab * es;
    uint32_t ctas = 1;
    while (ctas < kMaxCluster && a.nrows * ctas < 152 * kDCtas && bytes >= 2 * ctas * kVecs * kDThreads * 16)
        ctas *= 2;
    const bool f = a.dtype == CCL_FP32;
    cudaError_t e;
    if (mode == DISTILL_LOSS)
        e = f ? launch_distill<DT_FP32, DISTILL_LOSS>(p, a.nrows, ctas, stream)
              : launch_distill<DT_BF16, DISTILL_LOSS>(p, a.nrows, ctas, stream);
    else if (mode == DISTILL_FUSED)
        e = f ? launch_distill<DT_FP32, DISTILL_FUSED>(p, a.nrows, ctas, stream)
              : launch_distill<DT_BF16, DISTILL_FUSED>(p, a.nrows, ctas, stream);
    else
        e = f ? launch_distill<DT_FP32, DISTILL_GRAD>(p, a.nrows, ctas, stream)
              : launch_distill<DT_BF16, DISTILL_GRAD>(p, a.nrows, ctas, stream);
    return from_cuda(e);
}

} // namespace
} // namespace ccl

using namespace ccl;

extern "C" {

ccl_status_t ccl_distill_loss(const void *logits, size_t nrows, size_t vocab, size_t logits_stride, ccl_dtype_t dtype,
                              const int64_t *teacher_ids, const float *teacher_logits, size_t top, float temperature,
                              const float *weights, float *loss, float *stats, void *grad, size_t grad_stride,
                              cudaStream_t stream)
{
    TraceScope tr("distill_loss", 1, nrows, (int)dtype, -1, 0, stream);
    return tr.done(guarded([&] {
        return distill_impl(grad ? DISTILL_FUSED : DISTILL_LOSS,
                            DistillArgs{logits, nrows, vocab, logits_stride, dtype, teacher_ids, teacher_logits, top,
                                        temperature, weights, loss, stats, grad, grad_stride},
                            stream);
    }));
}

ccl_status_t ccl_distill_grad(const void *logits, size_t nrows, size_t vocab, size_t logits_stride, ccl_dtype_t dtype,
                              const int64_t *teacher_ids, const float *teacher_logits, size_t top, float temperature,
                              const float *weights, const float *stats, void *grad, size_t grad_stride,
                              cudaStream_t stream)
{
    TraceScope tr("distill_grad", 1, nrows, (int)dtype, -1, 0, stream);
    return tr.done(guarded([&] {
        return distill_impl(DISTILL_GRAD,
                            DistillArgs{logits, nrows, vocab, logits_stride, dtype, teacher_ids, teacher_logits, top,
                                        temperature, weights, nullptr, const_cast<float *>(stats), grad, grad_stride},
                            stream);
    }));
}

} // extern "C"
