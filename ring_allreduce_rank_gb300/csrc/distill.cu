// distill.cu -- distillation loss from a teacher's top logits, and its
// gradient.
//
// Per row: p = softmax over the teacher's K listed logits / tau, q = softmax
// of the student's whole row / tau,
//     loss  = w * sum_j p_j (log p_j - log q_{i_j}),
//     ds_v  = w / tau * (q_v - sum_{j: i_j = v} p_j).
// With m the row's maximum and Z = sum_v exp((s_v - m) / tau), both need one
// pass over the row for (m, Z); the gradient needs the row's values again.
// Bound by memory bandwidth: the row is read once and the gradient written
// once, so a cluster of CTAs keeps the row in registers between the two uses
// (kVecs 16-byte vectors a thread; 64 KiB a CTA, so that three CTAs' loads and
// stores overlap on an SM), joins (m, Z) through distributed shared memory,
// and reads a row again only where it exceeds eight CTAs' registers.
#include <cooperative_groups.h>

#include <vector>

#include "../../include/ccl.h"
#include "ccl_internal.h"
#include "step_ops.cuh"

namespace cg = cooperative_groups;

namespace ccl {
namespace {

constexpr int kDThreads = 512;
constexpr int kDWarps = kDThreads / 32;
constexpr int kVecs = 8;         // 16-byte vectors a thread holds
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
__global__ void __launch_bounds__(kDThreads, 2) distill_kernel(const __grid_constant__ DistillParams p)
{
    constexpr int VEC = DType<DT>::kVec, ES = DType<DT>::kSize;
    __shared__ int64_t id[kMaxTop];
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
    const uint64_t nh = umin64(p.vocab, ((16 - ((uintptr_t)row & 15)) & 15) / ES);
    const uint64_t nv = (p.vocab - nh) / VEC, nt = p.vocab - nh - nv * VEC;
    const uint64_t per = (nv + ctas - 1) / ctas, v0 = umin64(nv, per * cta), v1 = umin64(nv, v0 + per);
    const char *body = row + nh * ES;
    // an edge element: head, then tail
    const bool edge = cta == 0 && tid < (int)(nh + nt);
    const uint64_t ei = tid < (int)nh ? tid : p.vocab - nt + (tid - nh);
    // a row whose weight is 0 has loss 0 and gradient 0 whatever it holds
    // (its statistics are still wanted where the caller keeps them)
    const bool skip = w == 0.0f && (MODE != DISTILL_LOSS || !p.stats) && !(MODE == DISTILL_FUSED && p.stats);
    const bool vec_store = MODE != DISTILL_LOSS && (((uintptr_t)grow ^ (uintptr_t)row) & 15) == 0;

    uint4 x[kVecs];
    float xe = 0.0f;
    const uint64_t rounds = (v1 - v0 + (uint64_t)kVecs * kDThreads - 1) / ((uint64_t)kVecs * kDThreads);
    auto load = [&](uint64_t round) {
        const uint64_t b = v0 + round * kVecs * kDThreads + tid;
#pragma unroll
        for (int i = 0; i < kVecs; ++i)
            if (b + (uint64_t)i * kDThreads < v1)
                x[i] = ld16(body + (b + (uint64_t)i * kDThreads) * 16);
    };
    Stat st{-INFINITY, 0.0f};
    if (!skip) {
        load(0);
        if (edge)
            xe = ld_value<DT>(row, ei);
    }

    // whether element i of the row is in this CTA's part
    auto mine = [&](uint64_t i) {
        if (i < nh || i >= nh + nv * VEC)
            return cta == 0;
        const uint64_t v = (i - nh) / VEC;
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
            id[j] = ok ? i : -1;
            prob[j] = l;
            // a NaN counts as present, so that it reaches the result
            tm = l != l ? INFINITY : fmaxf(tm, l);
        }
    tm = block_reduce<true>(tm, red);
    const bool some = tm > -INFINITY;
    float tz = 0.0f;
    if (some)
        for (int j = tid; j < top; j += kDThreads) {
            const float e = id[j] >= 0 ? exp2f(__fmul_rn(__fsub_rn(prob[j], tm), p.scale)) : 0.0f;
            prob[j] = e;
            tz = __fadd_rn(tz, e);
        }
    tz = block_reduce<false>(tz, red);
    if (some)
        for (int j = tid; j < top; j += kDThreads) {
            prob[j] = __fdiv_rn(prob[j], tz);
            // CTA 0 needs every listed logit for the loss, the others their own
            if (id[j] >= 0 && (mine((uint64_t)id[j]) || (MODE != DISTILL_GRAD && cta == 0)))
                logit[j] = ld_value<DT>(row, (uint64_t)id[j]);
        }

    if (MODE == DISTILL_GRAD) {
        st.m = gload<float>(p.stats + 2 * t);
        st.z = gload<float>(p.stats + 2 * t + 1);
        __syncthreads();
    } else {
        // (m, Z): this thread's vectors, then warp, CTA and cluster
        if (!skip) {
            for (uint64_t r = 0; r < rounds; ++r) {
                if (r)
                    load(r);
                const uint64_t b = v0 + r * kVecs * kDThreads + tid;
                Stat part{-INFINITY, 0.0f};
#pragma unroll
                for (int i = 0; i < kVecs; ++i)
                    if (b + (uint64_t)i * kDThreads < v1) {
                        float f[VEC];
                        unpack<DT>(x[i], f);
#pragma unroll
                        for (int k = 0; k < VEC; ++k)
                            part.m = fmaxf(part.m, f[k]);
                    }
#pragma unroll
                for (int i = 0; i < kVecs; ++i)
                    if (b + (uint64_t)i * kDThreads < v1) {
                        float f[VEC];
                        unpack<DT>(x[i], f);
#pragma unroll
                        for (int k = 0; k < VEC; ++k)
                            part.z = __fadd_rn(part.z, f[k] == -INFINITY ? 0.0f : row_exp(f[k], part.m, p.scale));
                    }
                st = join(st, part, p.scale);
            }
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
            if (some && !skip) {
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
        char *gbody = grow + nh * ES;
        for (uint64_t r = 0; r < rounds; ++r) {
            if (!skip && (MODE == DISTILL_GRAD ? r > 0 : rounds > 1))
                load(r);
            const uint64_t b = v0 + r * kVecs * kDThreads + tid;
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                const uint64_t v = b + (uint64_t)i * kDThreads;
                if (v < v1) {
                    float f[VEC];
                    if (zero) {
#pragma unroll
                        for (int k = 0; k < VEC; ++k)
                            f[k] = 0.0f;
                    } else {
                        unpack<DT>(x[i], f);
#pragma unroll
                        for (int k = 0; k < VEC; ++k)
                            f[k] = __fmul_rn(row_exp(f[k], st.m, p.scale), c);
                    }
                    if (vec_store) {
                        st16(gbody + v * 16, pack<DT>(f));
                    } else {
#pragma unroll
                        for (int k = 0; k < VEC; ++k)
                            st_value<DT>(grow, nh + v * VEC + k, f[k]);
                    }
                }
            }
        }
        if (edge)
            st_value<DT>(grow, ei, zero ? 0.0f : __fmul_rn(row_exp(xe, st.m, p.scale), c));
        __syncthreads(); // before the listed ids' gradients replace what was written
        if (!zero)
            for (int j = tid; j < top; j += kDThreads) {
                if (id[j] < 0)
                    continue;
                const uint64_t i = (uint64_t)id[j];
                if (!mine(i))
                    continue;
                float sum = 0.0f;
                bool firstj = true;
                for (int k = 0; k < top; ++k)
                    if (id[k] == id[j]) {
                        firstj = firstj && k >= j;
                        sum = __fadd_rn(sum, prob[k]);
                    }
                if (firstj) {
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
    // the fewest CTAs whose registers hold a row; more, down to one vector a
    // thread, while there are fewer of them than SMs
    const uint64_t bytes = a.vocab * es, cap = (uint64_t)kVecs * kDThreads * 16;
    uint32_t ctas = 1;
    while (ctas < kMaxCluster && (bytes > ctas * cap || (a.nrows * ctas < 152 && bytes > ctas * cap / kVecs)))
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
