// tensor_core.cuh -- what the feed-forward kernels (ffn.cu, experts.cu) share:
// the tensor cores', tensor memory's, copies' and barriers' instructions, the
// activations, and the epilogues' vectors.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include "../../include/ccl.h"
#include "ccl_internal.h"
#include "step_ops.cuh"

namespace ccl {

// ------------------------------------------------------------------ PTX

__device__ __forceinline__ uint32_t smem_u32(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

__device__ __forceinline__ uint32_t in_cta(uint32_t addr, uint32_t rank)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}

__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}

__device__ __forceinline__ void mbar_expect(uint32_t bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar)
{
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ unsigned long long now_ns()
{
    unsigned long long t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

// Waits for the phase of the given parity; false (and the CTA's flag set, and
// the counter raised) after `limit` ns, or once another role gave up.
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, volatile int *gave_up, unsigned long long limit,
                                          unsigned long long *timeouts)
{
    unsigned long long t0 = 0;
    for (uint32_t n = 0;; ++n) {
        uint32_t done;
        asm volatile("{\n\t.reg .pred p;\n\t"
                     "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
                     "selp.u32 %0, 1, 0, p;\n\t}"
                     : "=r"(done)
                     : "r"(bar), "r"(parity)
                     : "memory");
        if (done)
            return true;
        if ((n & 255) == 255) {
            if (*gave_up)
                return false;
            const unsigned long long t = now_ns();
            if (!t0) {
                t0 = t;
            } else if (t - t0 > limit) {
                *gave_up = 1;
                atomicAdd(timeouts, 1ull);
                return false;
            }
        }
    }
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap *map)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// A 2-D box of a tensor map into this CTA's shared memory; its bytes are
// counted at `bar`, a barrier of the pair's first CTA.
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar)
{
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 "
                 "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
                 "l"(map), "r"(x), "r"(y), "r"(bar)
                 : "memory");
}

// The same within one CTA.
__device__ __forceinline__ void tma_load_own(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar)
{
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
                 "l"(map), "r"(x), "r"(y), "r"(bar)
                 : "memory");
}

__device__ __forceinline__ void tc_commit_own(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void tc_mma_own(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
                 "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
                 : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void tc_commit(uint32_t bar) // arrives at `bar` in both CTAs
{
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
                 "h"((uint16_t)3)
                 : "memory");
}

__device__ __forceinline__ void tc_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
                 "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
                 : "memory");
}

__device__ __forceinline__ void tc_load16(uint32_t addr, float *f)
{
    uint32_t r[16];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(addr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i)
        f[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ void tc_load32(uint32_t addr, float *f)
{
    uint32_t r[32];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
                 "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
                   "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
                   "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
                   "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
                 : "r"(addr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i)
        f[i] = __uint_as_float(r[i]);
}

// Shared-memory descriptor of a 128-byte-swizzled operand tile.  K-major: rows
// of 64 k values (128 bytes), eight rows a swizzle atom (1024 bytes apart).
// MN-major: for each 64 rows or columns of the operand, 64 k rows of 128
// bytes; the next 64 follow 8192 bytes later.
template <bool MN> __device__ __forceinline__ uint64_t operand_desc(uint32_t addr)
{
    const uint64_t lead = MN ? 8192 >> 4 : 1, stride = 1024 >> 4;
    return (uint64_t)((addr & 0x3ffff) >> 4) | lead << 16 | stride << 32 | (uint64_t)1 << 46 | (uint64_t)2 << 61;
}

// Bytes from one 16-deep step of K to the next within a tile.
template <bool MN> __device__ __forceinline__ constexpr uint32_t k_step() { return MN ? 16 * 128 : 32; }

// ------------------------------------------------------------------ activations

__device__ __forceinline__ float sigmoid(float x)
{
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(__fmul_rn(x, -1.4426950408889634f)));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(__fadd_rn(1.0f, e)));
    return r;
}

// act(g) and act'(g).  SiLU: g s(g).  GELU (tanh form): 0.5 g (1 + tanh y) =
// g s(2y), y = sqrt(2/pi) (g + 0.044715 g^3), which keeps its small values.
__device__ __forceinline__ void activation(int act, float g, float &a, float &da)
{
    if (act == CCL_ACT_SILU) {
        const float s = sigmoid(g);
        a = g * s;
        da = s * __fmaf_rn(g, 1.0f - s, 1.0f);
    } else {
        constexpr float c2 = 1.5957691216057308f; // 2 sqrt(2/pi)
        const float gg = g * g;
        const float s = sigmoid(c2 * g * __fmaf_rn(0.044715f, gg, 1.0f));
        const float d = s * (1.0f - s);
        a = g * s;
        da = d == 0.0f ? s : __fmaf_rn(g * d, c2 * __fmaf_rn(3 * 0.044715f, gg, 1.0f), s);
    }
}

// ------------------------------------------------------------------ epilogue vectors

// Sixteen values of one row, eight at a time: `both` says whether the second
// eight are columns of the matrix.
struct Vals16 {
    uint4 v[4];
    __device__ __forceinline__ void load(const float *q, bool both)
    {
        ld32(q, v[0], v[1]);
        if (both)
            ld32(q + 8, v[2], v[3]);
    }
    __device__ __forceinline__ void load(const uint16_t *q, bool both)
    {
        v[0] = ld16(q);
        if (both)
            v[1] = ld16(q + 8);
    }
    __device__ __forceinline__ void get(float *f) const
    {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            unpack<DT_FP32>(v[i], f + 4 * i);
    }
};

__device__ __forceinline__ void store16(float *q, const float *f, bool both)
{
    st32(q, pack<DT_FP32>(f), pack<DT_FP32>(f + 4));
    if (both)
        st32(q + 8, pack<DT_FP32>(f + 8), pack<DT_FP32>(f + 12));
}

__device__ __forceinline__ void store16(uint16_t *q, const float *f, bool both)
{
    if (both && ((uintptr_t)q & 31) == 0) {
        st32(q, pack<DT_BF16>(f), pack<DT_BF16>(f + 8));
    } else {
        st16(q, pack<DT_BF16>(f));
        if (both)
            st16(q + 8, pack<DT_BF16>(f + 8));
    }
}

// ------------------------------------------------------------------ operands TMA cannot address

struct PackParams {
    struct {
        const uint16_t *src;
        uint16_t *dst;
        uint32_t cols, ld;
        uint64_t vectors; // rows * ld / 8
    } m[5];
    int n;
};

// Rows of `cols` elements of the i-th matrix to rows `ld` apart (ld a multiple
// of 8), the rest of a row zero; a thread (of 256) writes a vector of eight.
__device__ __forceinline__ void pack_operand(const PackParams &p, uint32_t i)
{
    const auto &m = p.m[i];
    const uint32_t per = m.ld / 8;
    for (uint64_t e = (uint64_t)blockIdx.x * 256 + threadIdx.x; e < m.vectors; e += (uint64_t)gridDim.x * 256) {
        const uint64_t r = m.vectors >> 32 ? e / per : (uint32_t)e / per;
        const uint32_t c = (uint32_t)(e - r * per) * 8;
        const uint16_t *src = m.src + r * m.cols + c;
        if (c && c + 9 <= m.cols) {
            // inside a row: the words around the eight values
            const uint32_t odd = (uintptr_t)src & 2;
            const uint16_t *word = src - odd / 2;
            uint32_t x[5];
#pragma unroll
            for (int i = 0; i < 5; ++i)
                x[i] = i < 4 || odd ? gload<uint32_t>(word + 2 * i) : 0;
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                o[i] = __funnelshift_r(x[i], x[i + 1], odd * 8);
            st16(m.dst + e * 8, make_uint4(o[0], o[1], o[2], o[3]));
            continue;
        }
        uint32_t h[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            h[i] = c + i < m.cols ? gload<uint16_t>(src + i) : 0;
        st16(m.dst + e * 8, make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16));
    }
}

static __global__ void __launch_bounds__(256) pack_operands_kernel(const __grid_constant__ PackParams p)
{
    chain_entry();
    pack_operand(p, blockIdx.y); // the matrix
}

// ------------------------------------------------------------------ host side

inline PFN_cuTensorMapEncodeTiled_v12000 encode_fn()
{
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) != cudaSuccess ||
            r != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            f = nullptr;
        }
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    }();
    return fn;
}

constexpr int kPairs = 76, kSms = 152; // CTA pairs and SMs of the GPU

struct Matrix { // a row-major bf16 operand as TMA sees it
    const void *ptr;
    uint64_t rows, cols, ld;
};

// The operands as they lie where TMA can address them (16-byte aligned base
// and rows), else copied to rows of a padded stride, all in one launch.
class Operands {
  public:
    explicit Operands(char *work) : work_(work) {}
    Matrix add(const void *src, uint64_t rows, uint64_t cols, size_t at)
    {
        const uint64_t ld = (cols + 7) / 8 * 8;
        if ((uintptr_t)src % 16 == 0 && cols == ld)
            return Matrix{src, rows, cols, cols};
        auto &m = p_.m[p_.n++];
        m.src = static_cast<const uint16_t *>(src);
        m.dst = reinterpret_cast<uint16_t *>(work_ + at);
        m.cols = (uint32_t)cols;
        m.ld = (uint32_t)ld;
        m.vectors = rows * ld / 8;
        most_ = std::max(most_, m.vectors);
        return Matrix{m.dst, rows, cols, ld};
    }
    cudaError_t copy(cudaStream_t stream)
    {
        if (p_.n == 0)
            return cudaSuccess;
        const cudaError_t e = launch_chained(pack_operands_kernel, dim3((unsigned)std::min<uint64_t>((most_ + 255) / 256, 8 * kSms), (unsigned)p_.n), dim3(256), 0, stream, p_);
        if (e == cudaSuccess)
            count_launches(1);
        return e;
    }

    // for a kernel that makes the copies beside its own work
    const PackParams &params() const { return p_; }
    uint64_t most() const { return most_; } // vectors of the largest one

  private:
    PackParams p_{};
    char *work_;
    uint64_t most_ = 0;
};

// How long a role of a feed-forward kernel waits for another, in ns, in calls made from now on.
unsigned long long feed_forward_wait_ns();
// Adds the expert kernels' waits that ran out on the current device.
cudaError_t expert_timeouts(unsigned long long *count);

} // namespace ccl
