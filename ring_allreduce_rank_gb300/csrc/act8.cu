// act8.cu -- activations kept in 8 bits for the backward pass, and brought back.
//
// 8.25 bits a value instead of 16 or 32: codes [rows][width], a byte a value, and
// bytes [rows][width / 32], a power of two a block (act8.cuh), width being the
// columns rounded up to 32, so that every row of codes is whole 32-byte
// vectors.  Bound by memory bandwidth: each value is read once and written
// once.  A thread takes a whole block, so that no value crosses lanes; where
// the rows are no whole vectors, values pass a warp's 32 x 32 in shared memory,
// so that its accesses still run along a row.  8192 x 11008 bf16: pack 43.8 us
// (6.2 TB/s; in 16-byte vectors 45.3, turned 105.7), unpack 40.1 (6.8 TB/s; 55.0,
// 79.3).
#include <vector>

#include "../../include/ccl.h"
#include "act8.cuh"
#include "ccl_internal.h"
#include "step_ops.cuh"

namespace ccl {
namespace {

constexpr uint32_t kActThreads = 256;

struct Act8Params {
    char *x; // the values' rows, read or written
    uint8_t *codes, *bytes;
    uint64_t pitch, blocks; // bytes from row to row; blocks of all rows
    uint32_t cols, per;     // columns, blocks a row
};

__device__ __forceinline__ uint64_t row_of(const Act8Params &p, uint64_t i)
{
    return p.blocks >> 32 ? i / p.per : (uint32_t)i / p.per;
}

// 32 consecutive values of a row in vectors of W bytes; those past the row are 0.
template <int DT, int W> __device__ __forceinline__ void load_block(const char *src, uint32_t n, float *f)
{
    constexpr int V = DType<DT>::kVec;
    uint4 v[32 / V];
#pragma unroll
    for (int i = 0; i < 32 / V; i += W == 32 ? 2 : 1) {
        v[i] = v[W == 32 ? i + 1 : i] = make_uint4(0, 0, 0, 0);
        if ((uint32_t)(i * V) < n) {
            if (W == 32)
                ld32(src + i * 16, v[i], v[W == 32 ? i + 1 : i]);
            else
                v[i] = ld16(src + i * 16);
        }
    }
#pragma unroll
    for (int i = 0; i < 32 / V; ++i)
        unpack<DT>(v[i], f + i * V);
}

template <int DT, int W> __global__ void __launch_bounds__(kActThreads) act8_pack_kernel(Act8Params p)
{
    chain_entry();
    constexpr int es = DType<DT>::kSize;
    if (W) {
        const uint64_t i = (uint64_t)blockIdx.x * kActThreads + threadIdx.x;
        if (i >= p.blocks)
            return;
        const uint64_t r = row_of(p, i);
        const uint32_t c = (uint32_t)(i - r * p.per) * kActBlock;
        const char *src = p.x + r * p.pitch + (uint64_t)c * es;
        float f[32];
        uint4 lo, hi;
        load_block<DT, W>(src, p.cols - c, f);
        const uint32_t byte = act8_encode(f, lo, hi);
        st32(p.codes + i * kActBlock, lo, hi);
        gstore<uint8_t>(p.bytes + i, (uint8_t)byte);
    } else {
        // a warp takes 32 blocks: their values a block at a time, a lane a value,
        // turned in shared memory so that a lane then has a block
        __shared__ float turned[kActThreads / 32][32][33];
        const uint32_t lane = threadIdx.x & 31;
        float(*mine)[33] = turned[threadIdx.x / 32];
        const uint64_t i0 = ((uint64_t)blockIdx.x * (kActThreads / 32) + threadIdx.x / 32) * 32;
        if (i0 >= p.blocks)
            return;
        uint64_t r = row_of(p, i0);
        uint32_t b = (uint32_t)(i0 - r * p.per);
        const uint32_t n = (uint32_t)umin64(32, p.blocks - i0);
#pragma unroll
        for (uint32_t j0 = 0; j0 < 32; j0 += 8) {
            float v[8];
#pragma unroll
            for (uint32_t j = 0; j < 8; ++j) {
                const uint32_t c = b * kActBlock + lane;
                v[j] = j0 + j < n && c < p.cols ? ld_value<DT>(p.x + r * p.pitch, c) : 0.0f;
                if (++b == p.per) {
                    b = 0;
                    ++r;
                }
            }
#pragma unroll
            for (uint32_t j = 0; j < 8; ++j)
                mine[j0 + j][lane] = v[j];
        }
        __syncwarp();
        if (lane < n) {
            float f[32];
            uint4 lo, hi;
#pragma unroll
            for (int j = 0; j < 32; ++j)
                f[j] = mine[lane][j];
            const uint32_t byte = act8_encode(f, lo, hi);
            st32(p.codes + (i0 + lane) * kActBlock, lo, hi);
            gstore<uint8_t>(p.bytes + i0 + lane, (uint8_t)byte);
        }
    }
}

template <int DT, int W> __global__ void __launch_bounds__(kActThreads) act8_unpack_kernel(Act8Params p)
{
    chain_entry();
    constexpr int es = DType<DT>::kSize, V = DType<DT>::kVec;
    if (W) {
        const uint64_t i = (uint64_t)blockIdx.x * kActThreads + threadIdx.x;
        if (i >= p.blocks)
            return;
        const uint64_t r = row_of(p, i);
        const uint32_t c = (uint32_t)(i - r * p.per) * kActBlock;
        char *dst = p.x + r * p.pitch + (uint64_t)c * es;
        uint4 lo, hi;
        ld32(p.codes + i * kActBlock, lo, hi);
        float f[32];
        act8_decode(lo, hi, act8_step(gload<uint8_t>(p.bytes + i)), f);
#pragma unroll
        for (int j = 0; j < 32 / V; j += W == 32 ? 2 : 1)
            if ((uint32_t)(j * V) < p.cols - c) {
                if (W == 32)
                    st32(dst + j * 16, pack<DT>(f + j * V), pack<DT>(f + (W == 32 ? j + 1 : j) * V));
                else
                    st16(dst + j * 16, pack<DT>(f + j * V));
            }
    } else {
        __shared__ float turned[kActThreads / 32][32][33];
        const uint32_t lane = threadIdx.x & 31;
        float(*mine)[33] = turned[threadIdx.x / 32];
        const uint64_t i0 = ((uint64_t)blockIdx.x * (kActThreads / 32) + threadIdx.x / 32) * 32;
        if (i0 >= p.blocks)
            return;
        uint64_t r = row_of(p, i0);
        uint32_t b = (uint32_t)(i0 - r * p.per);
        const uint32_t n = (uint32_t)umin64(32, p.blocks - i0);
        if (lane < n) {
            uint4 lo, hi;
            float f[32];
            ld32(p.codes + (i0 + lane) * kActBlock, lo, hi);
            act8_decode(lo, hi, act8_step(gload<uint8_t>(p.bytes + i0 + lane)), f);
#pragma unroll
            for (int j = 0; j < 32; ++j)
                mine[lane][j] = f[j];
        }
        __syncwarp();
#pragma unroll 8
        for (uint32_t j = 0; j < n; ++j) {
            const uint32_t c = b * kActBlock + lane;
            if (c < p.cols)
                st_value<DT>(p.x + r * p.pitch, c, mine[j][lane]);
            if (++b == p.per) {
                b = 0;
                ++r;
            }
        }
    }
}

constexpr size_t kMaxRows = 0x7fffffff, kMaxCols = (size_t)1 << 24;

ccl_status_t act8_impl(bool pack, const void *x, size_t rows, size_t cols, size_t stride, ccl_dtype_t dtype, const void *codes, const void *bytes,
                       cudaStream_t stream)
{
    if (!valid_dtype(dtype) || stride < cols || rows > kMaxRows || cols > kMaxCols)
        return CCL_ERR_INVALID_ARG;
    const size_t es = elem_size(dtype), per = (cols + kActBlock - 1) / kActBlock;
    size_t xb;
    if (!extent(rows, cols, stride, es, &xb))
        return CCL_ERR_INVALID_ARG;
    if (rows == 0 || cols == 0)
        return CCL_OK;
    if (!x || !codes || !bytes || !element_aligned(es, {x}) || !element_aligned(32, {codes}))
        return CCL_ERR_INVALID_ARG;
    const Range a = range_of(x, xb, 0), b = range_of(codes, rows * per * kActBlock, 0), c = range_of(bytes, rows * per, 0);
    const std::vector<Range> w = pack ? std::vector<Range>{b, c} : std::vector<Range>{a}, r = pack ? std::vector<Range>{a} : std::vector<Range>{b, c};
    if (ccl_status_t st = check_overlaps(w, r, [](const Range &, const Range &) { return false; }))
        return st;
#ifdef CCL_DEBUG_BOUNDS
    if (cudaError_t e = dbg_set_ranges({{x, xb}, {codes, rows * per * kActBlock}, {bytes, rows * per}}, stream))
        return from_cuda(e);
#endif
    Act8Params p{};
    p.x = static_cast<char *>(const_cast<void *>(x));
    p.codes = static_cast<uint8_t *>(const_cast<void *>(codes));
    p.bytes = static_cast<uint8_t *>(const_cast<void *>(bytes));
    p.pitch = stride * es;
    p.blocks = (uint64_t)rows * per;
    p.cols = (uint32_t)cols;
    p.per = (uint32_t)per;
    const uintptr_t all = (uintptr_t)x | p.pitch | cols * es;
    const int width = all % 32 == 0 ? 32 : all % 16 == 0 ? 16 : 0;
    // a thread a block: the grid's 2^31 CTAs hold 2^39 of them, and 2^31 rows of 2^24 columns have 2^50
    if (p.blocks > (uint64_t)0x7fffffff * kActThreads)
        return CCL_ERR_INVALID_ARG;
    const dim3 grid((unsigned)((p.blocks + kActThreads - 1) / kActThreads)), block(kActThreads);
    void (*k)(Act8Params);
#define CCL_ACT8_KERNEL(kernel)                                                                                        \
    (dtype == CCL_FP32 ? (width == 32 ? kernel<DT_FP32, 32> : width == 16 ? kernel<DT_FP32, 16> : kernel<DT_FP32, 0>)  \
                       : (width == 32 ? kernel<DT_BF16, 32> : width == 16 ? kernel<DT_BF16, 16> : kernel<DT_BF16, 0>))
    k = pack ? CCL_ACT8_KERNEL(act8_pack_kernel) : CCL_ACT8_KERNEL(act8_unpack_kernel);
    const cudaError_t e = launch_chained(k, grid, block, 0, stream, p);
    if (e == cudaSuccess)
        count_launches(1);
    return from_cuda(e);
}

} // namespace
} // namespace ccl

using namespace ccl;

extern "C" {

ccl_status_t ccl_plan_act8_width(size_t cols, size_t *width)
{
    if (!width || cols > kMaxCols)
        return CCL_ERR_INVALID_ARG;
    *width = (cols + kActBlock - 1) / kActBlock * kActBlock;
    return CCL_OK;
}

ccl_status_t ccl_act8_pack(const void *x, size_t rows, size_t cols, size_t x_stride, ccl_dtype_t dtype, int8_t *codes, uint8_t *scales,
                           cudaStream_t stream)
{
    TraceScope tr("act8_pack", 1, rows, (int)dtype, -1, 0, stream);
    return tr.done(guarded([&] { return act8_impl(true, x, rows, cols, x_stride, dtype, codes, scales, stream); }));
}

ccl_status_t ccl_act8_unpack(const int8_t *codes, const uint8_t *scales, size_t rows, size_t cols, ccl_dtype_t dtype, void *x, size_t x_stride,
                             cudaStream_t stream)
{
    TraceScope tr("act8_unpack", 1, rows, (int)dtype, -1, 0, stream);
    return tr.done(guarded([&] { return act8_impl(false, x, rows, cols, x_stride, dtype, codes, scales, stream); }));
}

} // extern "C"
