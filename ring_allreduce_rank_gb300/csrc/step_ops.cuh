// step_ops.cuh -- what the training-step operators (embed.cu, distill.cu,
// ffn.cu) share besides ccl_device.cuh: values of both types as fp32, and the
// host side's extents.
#pragma once

#include <atomic>
#include <initializer_list>
#include <new>

#include "ccl_internal.h"

namespace ccl {

// ------------------------------------------------------------------ 16-byte vectors as fp32 values

template <int DT> __device__ __forceinline__ void unpack(const uint4 &v, float *f)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if (DT == DT_FP32) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            f[i] = __uint_as_float(w[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
}

template <int DT> __device__ __forceinline__ uint4 pack(const float *f)
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (DT == DT_FP32) {
            w[i] = __float_as_uint(f[i]);
        } else {
            __nv_bfloat162 p = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<uint32_t *>(&p);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int DT> __device__ __forceinline__ float ld_value(const void *base, uint64_t i)
{
    const uint32_t v = ld_elem<DT>(base, i);
    return __uint_as_float(DT == DT_BF16 ? v << 16 : v);
}

template <int DT> __device__ __forceinline__ void st_value(void *base, uint64_t i, float f)
{
    if (DT == DT_FP32) {
        st_elem<DT>(base, i, __float_as_uint(f));
    } else {
        const __nv_bfloat16 h = __float2bfloat16_rn(f);
        st_elem<DT>(base, i, *reinterpret_cast<const uint16_t *>(&h));
    }
}

// 32-byte vectors (32-byte aligned): a full memory sector per lane.
__device__ __forceinline__ void ld32(const void *p, uint4 &a, uint4 &b)
{
    a = b = make_uint4(0, 0, 0, 0);
    if (dbg_ok(p, 32))
        asm volatile("ld.global.L1::no_allocate.v8.u32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
                     : "l"(p));
}

__device__ __forceinline__ void st32(void *p, const uint4 &a, const uint4 &b)
{
    if (dbg_ok(p, 32))
        asm volatile("st.global.L1::no_allocate.v8.u32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(a.x), "r"(a.y),
                     "r"(a.z), "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
                     : "memory");
}

// ------------------------------------------------------------------ host side

// Runs an entry point's body; an exception (the host vectors of the argument
// checks) becomes a status, so that none leaves a C entry.
template <class F> inline ccl_status_t guarded(F f)
{
    try {
        return f();
    } catch (...) {
        return CCL_ERR_NO_MEMORY;
    }
}

// Opts a kernel in to `bytes` of dynamic shared memory on the current device,
// once per device (`ready`: the kernel's own bits; doing it twice is harmless).
inline cudaError_t large_smem_once(const void *kernel, int bytes, std::atomic<unsigned long long> &ready)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (ready.load(std::memory_order_relaxed) & bit)
        return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
    if (e == cudaSuccess)
        ready.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

constexpr size_t kAlign = 256;
inline size_t up(size_t n) { return (n + kAlign - 1) / kAlign * kAlign; }

// Whether every pointer is a multiple of `size` bytes (NULL is): the kernels
// read elements with loads of their own size, which fault elsewhere.
inline bool element_aligned(size_t size, std::initializer_list<const void *> ps)
{
    for (const void *p : ps)
        if ((uintptr_t)p % size)
            return false;
    return true;
}

// Bytes from the first to past the last of n rows of `dim` elements, `stride`
// apart; false where that overflows.
inline bool extent(size_t n, size_t dim, size_t stride, size_t es, size_t *bytes)
{
    if (n == 0 || dim == 0) {
        *bytes = 0;
        return true;
    }
    if (mul_overflows(stride, es) || mul_overflows(n, stride * es) || dim > stride)
        return false;
    *bytes = ((n - 1) * stride + dim) * es;
    return true;
}

} // namespace ccl
