// distill.cu -- distillation loss from a teacher's top logits, and its
// gradient.
//
// Per row: p = softmax over the teacher's K listed logits / tau, q = softmax
// of the student's whole row / tau,
//     loss  = w * sum_j p_j (log p_j - log q_{i_j}),
//     ds_v  = w / tau * (q_v - sum_{j: i_j = v} p_j).
// With m the row's maximum and Z = sum_v exp((s_v - m) / tau), both need one
// pass over the row for (m, Z); the gradient needs the row's values again.
// Bound by memory bandwidth.  The loss alone uses a row once: a CTA streams it
// through its registers, eight vectors a thread in flight (4096 rows of 128000
// bf16: 161-163 us, 0.95-0.96 of the measured copy bandwidth).  For loss and gradient
// in one call memory sees one read of the logits and one write of the gradient:
// a cluster of CTAs takes a row, each CTA asks for its whole part at once (up to
// 64 KiB: half to registers, half to shared memory by asynchronous copies) and
// keeps it there between the two uses, and the CTAs join (m, Z) through
// distributed shared memory.  Four CTAs an SM are at different places of this,
// so that loads, exponentials and stores overlap: 406 us for the same rows,
// 0.76 of the copy bandwidth (reading a row a second time from the L2 cache
// missed it, 608 CTAs' rows of 250 KiB, and took 471).  Four CTAs leave a thread
// 56 registers and 100-160 bytes of spills; three, without spills, took 427.
// The gradient from kept statistics asks for its part in the same way, 345 us,
// 0.90 (streaming it like the loss, stores between the loads, took 409).
#include <cooperative_groups.h>

#include <atomic>
#include <vector>

#include "../../include/ccl.h"
#include "ccl_internal.h"
#include "step_ops.cuh"

namespace cg = cooperative_groups;

namespace ccl {
namespace {

constexpr int kDThreads = 256;   // that hold a row's vectors; a further warp works on the teacher's entries
constexpr int kDWarps = kDThreads / 32;
constexpr int kDCtas = 4;        // resident CTAs per SM, for loss and gradient in one call; one less for either alone
constexpr int kVecs = 2;         // 16-byte vectors a thread folds at a time
constexpr int kHeld = 8;         // vectors a thread keeps in registers, and as many in shared memory
constexpr uint32_t kPart = 2 * kHeld * kDThreads; // vectors a CTA keeps
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
    uint32_t slot_bits;   // the hash table of the listed ids has 2^slot_bits places
    float scale;          // log2(e) / tau
    float inv_tau;
    uint32_t cluster_bits; // 2^cluster_bits CTAs take a row
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

__device__ __forceinline__ void copy16_async(uint4 *dst, const void *src)
{
    if (dbg_ok(src, 16))
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src) : "memory");
}

__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

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
    float m = s.m;
#pragma unroll
    for (int o = 16; o; o >>= 1)
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (s.m != m) // not where both are -inf
        s.z = __fmul_rn(s.z, row_exp(s.m, m, scale));
#pragma unroll
    for (int o = 16; o; o >>= 1)
        s.z = __fadd_rn(s.z, __shfl_xor_sync(0xffffffffu, s.z, o));
    s.m = m;
    return s;
}

template <bool MAX> __device__ __forceinline__ float warp_reduce(float v)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const float u = __shfl_xor_sync(0xffffffffu, v, o);
        v = MAX ? fmaxf(v, u) : __fadd_rn(v, u);
    }
    return v;
}

// One cluster per row.  The row's 16-byte vectors are shared out over the
// cluster's CTAs in contiguous parts; the elements before the first 16-byte
// boundary and after the last one (fewer than a vector each) are CTA 0's.
template <int DT, int MODE>
__global__ void __launch_bounds__(kDThreads + 32, MODE == DISTILL_FUSED ? kDCtas : kDCtas - 1) distill_kernel(const __grid_constant__ DistillParams p)
{
    constexpr int VEC = DType<DT>::kVec, ES = DType<DT>::kSize;
    constexpr uint32_t kNone = 0xffffffffu, kEntry = 0x7fffffffu;
    extern __shared__ uint4 held[]; // [kHeld][kDThreads]: each thread reads back its own vectors
    __shared__ uint32_t id[kMaxTop];
    __shared__ float prob[kMaxTop];  // p_j, 0 for entries that do not count
    __shared__ float logit[kMaxTop]; // the student's logit at id j
    __shared__ uint32_t slot[MODE == DISTILL_LOSS ? 1 : 2 * kMaxTop]; // an entry of each id, hashed
    __shared__ int present; // whether the row has a teacher
    __shared__ Stat wstat[kMaxCluster * kDWarps]; // every warp of the cluster's part of the row
    cg::cluster_group cluster = cg::this_cluster();
    const uint32_t ctas = 1u << p.cluster_bits, cta = blockIdx.x & (ctas - 1); // its rank in the cluster
    if (MODE != DISTILL_GRAD)
        cluster_arrive(); // waited for before the first write to another CTA
    const uint64_t t = blockIdx.x >> p.cluster_bits;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int top = (int)p.top;

    const float w = p.weights ? gload<float>(p.weights + t) : 1.0f;
    const char *row = p.logits + t * p.pitch;
    char *grow = MODE == DISTILL_LOSS ? nullptr : p.grad + t * p.grad_pitch;
    const uint32_t nh = (uint32_t)umin64(p.vocab, ((16 - ((uintptr_t)row & 15)) & 15) / ES);
    const uint32_t nv = ((uint32_t)p.vocab - nh) / VEC, nt = (uint32_t)p.vocab - nh - nv * VEC;
    const uint32_t per = (nv + ctas - 1) >> p.cluster_bits, v0 = min(nv, per * cta), v1 = min(nv, v0 + per);
    const char *body = row + (uint64_t)nh * ES;
    // an edge element: head, then tail
    const bool edge = cta == 0 && tid < (int)(nh + nt); // (fewer than 16 threads)
    const uint32_t ei = tid < (int)nh ? tid : (uint32_t)p.vocab - nt + (tid - nh);
    // a row whose weight is 0 has loss 0 and gradient 0 whatever it holds
    // (its statistics are still wanted where the caller keeps them)
    const bool skip = w == 0.0f && (MODE == DISTILL_GRAD || !p.stats);

    // kVecs vectors from vector b on; past the part's end -inf, which adds nothing
    constexpr uint32_t kNinf = DT == DT_FP32 ? 0xff800000u : 0xff80ff80u;
    const uint4 ninf = make_uint4(kNinf, kNinf, kNinf, kNinf);
    auto load = [&](uint4 *x, uint32_t b) {
        const char *q = body + (uint64_t)b * 16;
        if (b - tid + kVecs * kDThreads <= v1) { // the whole CTA's vectors
#pragma unroll
            for (int i = 0; i < kVecs; ++i)
                x[i] = ld16(q + i * kDThreads * 16);
            return;
        }
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            x[i] = ninf;
            if (b + i * kDThreads < v1)
                x[i] = ld16(q + i * kDThreads * 16);
        }
    };
    auto from_held = [&](uint4 *x, int i0) {
#pragma unroll
        for (int i = 0; i < kVecs; ++i)
            x[i] = held[(i0 + i) * kDThreads + tid];
    };
    // vectors a thread has to work on (some threads one less): registers
    // first, then shared memory, then what does not fit
    const int mine_n = (int)((v1 - v0 + kDThreads - 1) / kDThreads);
    const bool holds = warp < kDWarps; // else the warp of the teacher's entries
    uint4 x[kHeld];
    float xe = 0.0f;
    if (!skip && holds) {
#pragma unroll
        for (int i = 0; MODE != DISTILL_LOSS && i < kHeld; ++i)
            if (kHeld + i / kVecs * kVecs < mine_n) {
                if (v0 + tid + (kHeld + i) * kDThreads < v1)
                    copy16_async(&held[i * kDThreads + tid], body + (uint64_t)(v0 + tid) * 16 + (kHeld + i) * kDThreads * 16);
                else
                    held[i * kDThreads + tid] = ninf;
            }
#pragma unroll
        for (int i = 0; i < kHeld; i += kVecs)
            load(x + i, v0 + tid + i * kDThreads);
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

    // The teacher's entries: a warp of their own, beside the sums of the row.
    // The loss is CTA 0's.
    const bool listed = !holds && !skip && (MODE != DISTILL_LOSS || cta == 0);
    float tm = -INFINITY;
    if (!holds) {
        constexpr int kBatch = 4;
        if (MODE != DISTILL_LOSS)
            for (uint32_t i = lane; i < 1u << p.slot_bits; i += 32)
                slot[i] = kNone;
        if (listed)
            for (int j0 = lane; j0 < top; j0 += 32 * kBatch) {
                int64_t i[kBatch];
                float l[kBatch], student[kBatch];
#pragma unroll
                for (int b = 0; b < kBatch; ++b)
                    if (j0 + 32 * b < top) {
                        i[b] = gload<int64_t>(p.ids + t * p.top + j0 + 32 * b);
                        l[b] = gload<float>(p.teacher + t * p.top + j0 + 32 * b);
                    }
#pragma unroll
                for (int b = 0; b < kBatch; ++b) {
                    // CTA 0 needs every listed logit for the loss, the others their own
                    student[b] = 0.0f;
                    if (j0 + 32 * b < top && (uint64_t)i[b] < p.vocab && (mine((uint32_t)i[b]) || (MODE != DISTILL_GRAD && cta == 0)))
                        student[b] = ld_value<DT>(row, (uint64_t)i[b]);
                }
#pragma unroll
                for (int b = 0; b < kBatch; ++b)
                    if (j0 + 32 * b < top) {
                        const bool ok = (uint64_t)i[b] < p.vocab;
                        const float v = ok ? l[b] : -INFINITY;
                        id[j0 + 32 * b] = ok ? (uint32_t)i[b] : kNone;
                        prob[j0 + 32 * b] = v;
                        logit[j0 + 32 * b] = student[b];
                        // a NaN counts as present, so that it reaches the result
                        tm = v != v ? INFINITY : fmaxf(tm, v);
                    }
            }
        tm = warp_reduce<true>(tm);
        if (lane == 0)
            present = tm > -INFINITY;
    }
    auto probabilities = [&] {
        float tz = 0.0f;
        if (!(tm > -INFINITY))
            return;
        for (int j = lane; j < top; j += 32) {
            const float e = id[j] != kNone ? exp2f(__fmul_rn(__fsub_rn(prob[j], tm), p.scale)) : 0.0f;
            prob[j] = e;
            tz = __fadd_rn(tz, e);
            if (MODE != DISTILL_LOSS && id[j] != kNone) {
                // one entry stands for each id in an open hash table at most
                // half full; the top bit says that the id has others
                const uint32_t mask = (1u << p.slot_bits) - 1;
                for (uint32_t h = id[j] * 2654435761u >> (32 - p.slot_bits);; h = (h + 1) & mask) {
                    const uint32_t was = atomicCAS(&slot[h], kNone, (uint32_t)j);
                    if (was == kNone)
                        break;
                    if (id[was & kEntry] == id[j]) {
                        atomicOr(&slot[h], ~kEntry);
                        break;
                    }
                }
            }
        }
        tz = warp_reduce<false>(tz);
        for (int j = lane; j < top; j += 32)
            prob[j] = __fdiv_rn(prob[j], tz);
        __syncwarp();
    };

    Stat st{-INFINITY, 0.0f};
    const float2 scale2 = make_float2(p.scale, p.scale);
    uint4 y[kVecs];
    if (MODE == DISTILL_GRAD) {
        st.m = gload<float>(p.stats + 2 * t);
        st.z = gload<float>(p.stats + 2 * t + 1);
        copies_wait();
        __syncthreads();
        if (!holds)
            probabilities();
    } else {
        // (m, Z): this thread's vectors, then warp, CTA and cluster
        if (!skip && holds) {
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
            if (MODE == DISTILL_LOSS) {
                // nothing is needed again: the registers take the next vectors
#pragma unroll 1
                for (int n = 0; n < mine_n; n += kHeld)
#pragma unroll
                    for (int i = 0; i < kHeld; i += kVecs) {
                        fold(x + i);
                        load(x + i, v0 + tid + (uint32_t)(n + kHeld + i) * kDThreads);
                    }
            } else {
#pragma unroll
                for (int i = 0; i < kHeld; i += kVecs)
                    if (i < mine_n)
                        fold(x + i);
                copies_wait();
#pragma unroll 1
                for (int i = 0; i < kHeld && kHeld + i < mine_n; i += kVecs) {
                    from_held(y, i);
                    fold(y);
                }
#pragma unroll 1
                for (uint32_t b = v0 + kPart; b < v1; b += kVecs * kDThreads) {
                    load(y, b + tid);
                    fold(y);
                }
            }
            st.z = __fadd_rn(z.x, z.y);
            if (edge)
                st = join(st, Stat{xe, xe == -INFINITY ? 0.0f : row_exp(xe, xe, p.scale)}, p.scale);
        }
        if (holds)
            st = warp_join(st, p.scale);
        cluster_wait(); // every CTA of the cluster has begun
        if (holds && lane < (int)ctas)
            cluster.map_shared_rank(wstat, lane)[cta * kDWarps + warp] = st;
        // from here on a CTA may overwrite its part of the logits (in place):
        // every read of another CTA's part is above
        cluster_arrive();
        if (listed)
            probabilities();
        cluster_wait();
        st = Stat{-INFINITY, 0.0f};
#pragma unroll
        for (int i = 0; i < kMaxCluster * kDWarps; i += 32)
            if (i + lane < (int)ctas * kDWarps)
                st = join(st, wstat[i + lane], p.scale);
        st = warp_join(st, p.scale);
        if (cta == 0 && !holds) {
            if (p.stats && lane == 0) {
                gstore<float>(p.stats + 2 * t, st.m);
                gstore<float>(p.stats + 2 * t + 1, st.z);
            }
            float sum = 0.0f;
            if (tm > -INFINITY) {
                const float lz = logf(st.z);
                for (int j = lane; j < top; j += 32)
                    if (!(prob[j] == 0.0f)) {
                        const float logq = __fsub_rn(__fmul_rn(__fsub_rn(logit[j], st.m), p.inv_tau), lz);
                        sum = __fadd_rn(sum, __fmul_rn(prob[j], __fsub_rn(logf(prob[j]), logq)));
                    }
            }
            sum = warp_reduce<false>(sum);
            if (lane == 0) // without a teacher 0 whatever the weight is
                gstore<float>(p.loss + t, w == 0.0f || !(tm > -INFINITY) ? 0.0f : __fmul_rn(w, sum));
        }
    }

    if (MODE != DISTILL_LOSS) {
        const float a = __fmul_rn(w, p.inv_tau);
        const bool zero = w == 0.0f || !present;
        const float c = zero ? 0.0f : __fdiv_rn(a, st.z);
        const float2 c2 = make_float2(c, c), neg = make_float2(-st.m, -st.m);
        const bool vec_store = (((uintptr_t)grow ^ (uintptr_t)row) & 15) == 0;
        char *gbody = grow + (uint64_t)nh * ES;
        auto emit = [&](const uint4 *x, uint32_t b) {
            char *q = gbody + (uint64_t)b * 16;
            const bool whole = vec_store && b - tid + kVecs * kDThreads <= v1;
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                uint4 o = make_uint4(0, 0, 0, 0);
                float2 f[VEC / 2];
                if (!zero) {
                    unpack2<DT>(x[i], f);
#pragma unroll
                    for (int k = 0; k < VEC / 2; ++k)
                        f[k] = mul2(row_exp2(f[k], neg, scale2), c2);
                    o = pack<DT>(reinterpret_cast<const float *>(f));
                }
                if (whole) {
                    st16(q + i * kDThreads * 16, o);
                } else if (b + i * kDThreads < v1) {
                    if (vec_store) {
                        st16(q + i * kDThreads * 16, o);
                    } else {
                        const uint32_t e[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
                        for (int k = 0; k < VEC; ++k)
                            st_elem<DT>(grow, nh + (uint64_t)(b + i * kDThreads) * VEC + k,
                                        DT == DT_FP32 ? e[k & 3] : e[k / 2] >> 16 * (k & 1) & 0xffff);
                    }
                }
            }
        };
        if (holds) {
#pragma unroll
            for (int i = 0; i < kHeld; i += kVecs)
                if (i < mine_n)
                    emit(x + i, v0 + tid + i * kDThreads);
#pragma unroll 1
            for (int i = 0; i < kHeld && kHeld + i < mine_n; i += kVecs) {
                from_held(y, i);
                emit(y, v0 + tid + (kHeld + i) * kDThreads);
            }
#pragma unroll 1
            for (uint32_t b = v0 + kPart; b < v1; b += kVecs * kDThreads) {
                if (!skip)
                    load(y, b + tid);
                emit(y, b + tid);
            }
        }
        if (edge)
            st_value<DT>(grow, ei, zero ? 0.0f : __fmul_rn(row_exp(xe, st.m, p.scale), c));
        __syncthreads(); // before the listed ids' gradients replace what was written
        if (!zero)
            for (uint32_t h = tid; h < 1u << p.slot_bits; h += kDThreads + 32) {
                const uint32_t e = slot[h];
                if (e == kNone)
                    continue;
                const uint32_t j = e & kEntry, i = id[j];
                if (!mine(i))
                    continue;
                float sum = prob[j];
                if (e != j) { // the id's entries, in order
                    sum = 0.0f;
                    for (int k = 0; k < top; ++k)
                        if (id[k] == i)
                            sum = __fadd_rn(sum, prob[k]);
                }
                const float q = __fdiv_rn(row_exp(logit[j], st.m, p.scale), st.z);
                st_value<DT>(grow, i, __fmul_rn(a, __fsub_rn(q, sum)));
            }
    }
}

// ------------------------------------------------------------------ host side

template <int DT, int MODE>
cudaError_t launch_distill(const DistillParams &p, uint64_t rows, uint32_t ctas, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(rows * ctas));
    cfg.blockDim = dim3(kDThreads + 32);
    cfg.dynamicSmemBytes = MODE == DISTILL_LOSS ? 0 : kHeld * kDThreads * 16;
    cfg.stream = stream;
    static std::atomic<unsigned long long> ready{0};
    if (MODE != DISTILL_LOSS)
        if (cudaError_t e = large_smem_once(reinterpret_cast<const void *>(distill_kernel<DT, MODE>), (int)cfg.dynamicSmemBytes, ready))
            return e;
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
        (mode == DISTILL_GRAD && !a.stats) || (mode != DISTILL_LOSS && a.vocab && !a.grad) ||
        !element_aligned(es, {a.logits, a.grad}) || !element_aligned(8, {a.ids}) ||
        !element_aligned(4, {a.teacher, a.weights, a.loss, a.stats}))
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
    p.slot_bits = 5;
    while (1u << p.slot_bits < 2 * a.top)
        ++p.slot_bits;
    // the fewest CTAs that hold a row (for the loss alone: one); more, as long
    // as each thread has a batch of vectors, while they leave places on the
    // GPU empty (counted as loss and gradient in one call have them; the other
    // two have 456 of these 608: 333 rows of 50257 fp32 take 1.5 and 2.9 rounds)
    const uint64_t bytes = a.vocab * es;
    uint32_t ctas = 1;
    p.cluster_bits = 0;
    while (ctas < kMaxCluster && ((mode != DISTILL_LOSS && bytes > (uint64_t)ctas * kPart * 16) ||
                                  (a.nrows * ctas < 152 * kDCtas && bytes >= (uint64_t)2 * ctas * kVecs * kDThreads * 16))) {
        ctas *= 2;
        ++p.cluster_bits;
    }
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
