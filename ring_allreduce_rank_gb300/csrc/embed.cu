// embed.cu -- embedding lookup with scaling and its gradient.
//
// Forward: out[t] = round(scale * table[id_t - first_row]); an id outside the
// table's rows gives a row of zeros.  One read of each looked-up row and one
// write of each output row: bound by memory bandwidth, by launch latency for
// a few tokens.
//
// Gradient: dE[v] = round([dE[v] +] scale * sum over {t: id_t = v} of dY[t]),
// the sum in fp32.  Launches, chained so that each starts under the one before:
//   0. embed_zero_kernel (dense gradient): zeros to the rows that no token
//      names, which need no sort to be found; a few further CTAs of it rank
//      the tokens where they are at most 4096.
//   1. embed_sort_kernel, for more: the tokens' (row, position) pairs sorted by
//      row, stably, by a radix sort that one cluster of eight CTAs runs (the
//      digits' counts cross the cluster through distributed shared memory).  It
//      need not wait for the zeros, but its CTAs take all the registers of an
//      SM each, so it begins once eight SMs have finished theirs.
//   2. embed_sum_kernel: the sorted tokens in pieces of 8 to 32, each summed in
//      order; a row whose tokens lie in one piece is finished here, a row that
//      crosses pieces leaves one fp32 partial sum per piece.
//   3. embed_join_kernel: those partial sums, added in order.
// No value is added by an atomic, so the same ids give the same bits each
// time, and a row that takes every token is still summed by all SMs.
// 16384 Zipf-distributed tokens of 4096 bf16 values over 32000 rows: lookup
// 31 us (the repeated rows come from the L2 cache), dense gradient 84 us
// against 58 us for its bytes at the copy bandwidth: zeros 40 us, sort 16,
// sums 30, join 12 (each alone); 94 us where the sort begins after the last
// zero.  Added to a table that is there (no zeros, old rows read): 73 us.
#include <cooperative_groups.h>

#include <vector>

#include "../../include/ccl.h"
#include "ccl_internal.h"
#include "step_ops.cuh"

namespace cg = cooperative_groups;

namespace ccl {
namespace {

constexpr int kSortCtas = 8;       // one portable cluster
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kDigits = 256;       // bins of one radix pass
constexpr int kZeroThreads = 512;
constexpr int kMinPiece = 8, kMaxPiece = 32; // sorted tokens summed by one warp
constexpr int kAhead = 8;          // rows' loads a warp has in flight; pieces are multiples of it
constexpr int kFewIds = 4096;      // so many tokens are ranked by counting instead of sorted
constexpr int kRanked = 128;       // tokens that a CTA ranks
constexpr int kSumThreads = 128;

// ------------------------------------------------------------------ lookup

struct EmbedParams {
    const char *table;
    char *out;
    const int64_t *ids;
    uint64_t ntokens, rows;
    uint64_t dim;                // elements
    uint64_t table_pitch, out_pitch; // bytes
    int64_t first_row;
    float scale;
};

// Thread (x, y) of a block covers row blockIdx.x * blockDim.y + y, every
// blockDim.x-th vector (element) of it.
template <int DT, bool VECTOR> __global__ void __launch_bounds__(128) embed_kernel(EmbedParams p)
{
    const uint64_t t = (uint64_t)blockIdx.x * blockDim.y + threadIdx.y;
    if (t >= p.ntokens)
        return;
    const uint64_t row = (uint64_t)gload<int64_t>(p.ids + t) - (uint64_t)p.first_row;
    const bool has = row < p.rows;
    const char *src = p.table + (has ? row : 0) * p.table_pitch;
    char *dst = p.out + t * p.out_pitch;
    if (VECTOR) {
        constexpr int V = DType<DT>::kVec;
        const uint32_t n = (uint32_t)(p.dim / V);
        for (uint32_t i0 = threadIdx.x; i0 < n; i0 += 4 * blockDim.x) {
            uint4 v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (has && i0 + j * blockDim.x < n)
                    v[j] = gload<uint4>(src + (uint64_t)(i0 + j * blockDim.x) * 16);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (i0 + j * blockDim.x < n) {
                    float f[V];
                    uint4 o = make_uint4(0, 0, 0, 0);
                    if (has) {
                        unpack<DT>(v[j], f);
#pragma unroll
                        for (int k = 0; k < V; ++k)
                            f[k] = __fmul_rn(f[k], p.scale);
                        o = pack<DT>(f);
                    }
                    st16(dst + (uint64_t)(i0 + j * blockDim.x) * 16, o);
                }
        }
    } else {
        for (uint64_t i0 = threadIdx.x; i0 < p.dim; i0 += 4 * blockDim.x) {
            float f[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (has && i0 + j * blockDim.x < p.dim)
                    f[j] = ld_value<DT>(src, i0 + j * blockDim.x);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (i0 + j * blockDim.x < p.dim)
                    st_value<DT>(dst, i0 + j * blockDim.x, has ? __fmul_rn(f[j], p.scale) : 0.0f);
        }
    }
}

// ------------------------------------------------------------------ gradient: sort and zero rows

struct SortParams {
    const int64_t *ids;
    uint64_t ntokens;
    int64_t first_row;
    uint32_t rows;
    uint2 *buf[2]; // (row, position) pairs, written in turn by the passes
    int passes, bits;
    char *grad; // the dense gradient, for its zero rows
    uint64_t pitch, row_bytes;
    int elem;
    uint32_t zero_ctas, rank_ctas; // embed_zero_kernel's CTAs that zero, and those before them that rank
};

__device__ __forceinline__ uint32_t row_key(const SortParams &p, uint64_t t)
{
    const uint64_t row = (uint64_t)gload<int64_t>(p.ids + t) - (uint64_t)p.first_row;
    return row < p.rows ? (uint32_t)row : p.rows; // ids outside the table sort last
}

// Zeros to the n bytes at q (a whole number of elements), one warp.
__device__ __forceinline__ void warp_zero(char *q, uint64_t n, int elem, int lane)
{
    const uint64_t head = umin64(n, (16 - ((uintptr_t)q & 15)) & 15);
    const uint64_t body = (n - head) / 16, tail = n - head - body * 16;
    for (uint64_t i = lane * elem; i < head; i += 32 * elem)
        if (elem == 2)
            gstore<uint16_t>(q + i, 0);
        else
            gstore<uint32_t>(q + i, 0);
    for (uint64_t i = lane; i < body; i += 32)
        st16(q + head + i * 16, make_uint4(0, 0, 0, 0));
    char *e = q + head + body * 16;
    for (uint64_t i = lane * elem; i < tail; i += 32 * elem)
        if (elem == 2)
            gstore<uint16_t>(e + i, 0);
        else
            gstore<uint32_t>(e + i, 0);
}

// A range of rows per CTA: the rows that tokens name marked from all the ids,
// the others zeroed.  The first p.rank_ctas CTAs make the sorted list of at
// most kFewIds tokens.
__global__ void __launch_bounds__(kZeroThreads, 2) embed_zero_kernel(const __grid_constant__ SortParams p)
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); // the sort needs no zeros, only room
    constexpr uint32_t kRows = 16384; // marked at a time
    constexpr int kIds = 16;
    // a byte a row, set by plain stores of one value: an atomic per token of a
    // frequent row took longer than the zeros
    __shared__ uint32_t mark_words[kRows / 4];
    uint8_t *mark = reinterpret_cast<uint8_t *>(mark_words);
    __shared__ uint4 row4[kFewIds / 4]; // rows of the tokens
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (blockIdx.x < p.rank_ctas) {
        // a token's place is the number of tokens of smaller rows and of
        // earlier ones of its own; four threads count for each, in segments of
        // an odd number of vectors so that they read different banks
        uint32_t *row = reinterpret_cast<uint32_t *>(row4);
        const uint32_t n = (uint32_t)p.ntokens, n4 = (n + 3) / 4, seg = (n4 + 3) / 4 | 1;
        uint32_t key[kFewIds / kZeroThreads]; // all the loads in flight
#pragma unroll
        for (int j = 0; j < kFewIds / kZeroThreads; ++j)
            key[j] = tid + j * kZeroThreads < n ? row_key(p, tid + j * kZeroThreads) : 0xffffffffu;
#pragma unroll
        for (int j = 0; j < kFewIds / kZeroThreads; ++j)
            row[tid + j * kZeroThreads] = key[j]; // past the end: larger than any row
        __syncthreads();
        const uint32_t t = blockIdx.x * kRanked + tid / 4;
        const uint32_t lo = min(n4, (tid & 3) * seg), hi = min(n4, lo + seg);
        const uint32_t own = t < n ? row[t] : 0;
        uint32_t place = 0;
        // all lanes walk the segment in step: before the warp's tokens (<=), the
        // vectors around them (both), after them (<)
        const uint32_t first4 = (t & ~7u) / 4, last4 = first4 + 2; // a warp's eight tokens
        uint32_t v = lo;
        const uint32_t a = max(lo, min(hi, first4)), b = max(lo, min(hi, last4));
#pragma unroll 8
        for (; v < a; ++v) {
            const uint4 r = row4[v];
            place += (r.x <= own) + (r.y <= own) + (r.z <= own) + (r.w <= own);
        }
        for (; v < b; ++v)
            for (uint32_t i = 4 * v; i < 4 * v + 4; ++i)
                place += row[i] < own || (row[i] == own && i < t);
#pragma unroll 8
        for (; v < hi; ++v) {
            const uint4 r = row4[v];
            place += (r.x < own) + (r.y < own) + (r.z < own) + (r.w < own);
        }
        place += __shfl_xor_sync(0xffffffffu, place, 1);
        place += __shfl_xor_sync(0xffffffffu, place, 2);
        if (t < n && (tid & 3) == 0)
            gstore<uint2>(p.buf[0] + place, make_uint2(own, t));
        return;
    }
    const uint32_t zero_cta = blockIdx.x - p.rank_ctas;
    const uint32_t per = (p.rows + p.zero_ctas - 1) / p.zero_ctas;
    const uint64_t end = umin64(p.rows, (uint64_t)(zero_cta + 1) * per);
    for (uint64_t lo = (uint64_t)zero_cta * per; lo < end; lo += kRows) {
        const uint32_t n = (uint32_t)umin64(kRows, end - lo);
        for (uint32_t i = tid; i < (n + 3) / 4; i += kZeroThreads)
            mark_words[i] = 0;
        __syncthreads();
        for (uint64_t t0 = tid; t0 < p.ntokens; t0 += kIds * kZeroThreads) {
            uint32_t key[kIds]; // as many loads in flight
#pragma unroll
            for (int j = 0; j < kIds; ++j)
                key[j] = t0 + j * kZeroThreads < p.ntokens ? row_key(p, t0 + j * kZeroThreads) : 0xffffffffu;
#pragma unroll
            for (int j = 0; j < kIds; ++j) {
                const uint64_t r = (uint64_t)key[j] - lo;
                if (r < n)
                    mark[r] = 1;
            }
        }
        __syncthreads();
        for (uint32_t r = warp; r < n; r += kZeroThreads / 32)
            if (!mark[r])
                warp_zero(p.grad + (lo + r) * p.pitch, p.row_bytes, p.elem, lane);
        __syncthreads();
    }
}

__global__ void __launch_bounds__(kSortThreads) embed_sort_kernel(const __grid_constant__ SortParams p)
{
    __shared__ uint32_t cnt[kSortWarps][kDigits];
    __shared__ uint32_t total[kDigits];
    __shared__ uint32_t wsum[kDigits / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    cg::cluster_group cluster = cg::this_cluster();
    // each warp owns a contiguous run of positions, so that the order within
    // a bin is the order of the positions
    const uint64_t slice = (p.ntokens + (uint64_t)kSortCtas * kSortThreads - 1) / (kSortCtas * kSortThreads) * 32;
    const uint64_t lo = ((uint64_t)blockIdx.x * kSortWarps + warp) * slice;
    const uint64_t hi = umin64(p.ntokens, lo + slice);
    const uint32_t below = (1u << lane) - 1;

    for (int pass = 0; pass < p.passes; ++pass) {
        const int shift = pass * p.bits;
        const uint32_t dmask = (1u << p.bits) - 1;
        const uint2 *in = pass ? p.buf[(pass - 1) & 1] : nullptr;
        uint2 *out = p.buf[pass & 1];
        auto pair = [&](uint64_t i) {
            return pass ? gload<uint2>(in + i) : make_uint2(row_key(p, i), (uint32_t)i);
        };
        for (int i = lane; i < kDigits; i += 32)
            cnt[warp][i] = 0;
        __syncwarp();
        for (uint64_t i = lo + lane; i - lane < hi; i += 32) {
            const unsigned act = __ballot_sync(0xffffffffu, i < hi);
            if (i < hi) {
                const uint32_t d = pair(i).x >> shift & dmask;
                const unsigned same = __match_any_sync(act, d);
                if ((same & below) == 0)
                    cnt[warp][d] += __popc(same);
            }
            __syncwarp();
        }
        __syncthreads();
        if (tid < kDigits) { // exclusive over the warps
            uint32_t run = 0;
            for (int w = 0; w < kSortWarps; ++w) {
                const uint32_t c = cnt[w][tid];
                cnt[w][tid] = run;
                run += c;
            }
            total[tid] = run;
        }
        cluster.sync();
        uint32_t before = 0, all = 0, inc = 0;
        if (tid < kDigits) { // over the CTAs, then exclusive over the bins
            for (int c = 0; c < kSortCtas; ++c) {
                const uint32_t v = cluster.map_shared_rank(total, c)[tid];
                all += v;
                if (c < (int)blockIdx.x)
                    before += v;
            }
            inc = all;
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t v = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o)
                    inc += v;
            }
            if (lane == 31)
                wsum[warp] = inc;
        }
        __syncthreads();
        if (tid < kDigits) {
            uint32_t base = inc - all + before;
            for (int w = 0; w < warp; ++w)
                base += wsum[w];
            for (int w = 0; w < kSortWarps; ++w)
                cnt[w][tid] += base;
        }
        __syncthreads();
        for (uint64_t i = lo + lane; i - lane < hi; i += 32) {
            const unsigned act = __ballot_sync(0xffffffffu, i < hi);
            if (i < hi) {
                const uint2 v = pair(i);
                const uint32_t d = v.x >> shift & dmask;
                const unsigned same = __match_any_sync(act, d);
                const uint32_t at = cnt[warp][d] + __popc(same & below);
                gstore<uint2>(out + at, v);
                __syncwarp(act);
                if ((same & below) == 0)
                    cnt[warp][d] += __popc(same);
            }
            __syncwarp();
        }
        // the pairs written here are read by the whole cluster, and no CTA
        // leaves or reuses its totals while another may read them
        cluster.sync();
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

// ------------------------------------------------------------------ gradient: sums

struct SumParams {
    const uint2 *sorted;
    uint64_t ntokens, dim, dim_pad;
    const char *dy;
    uint64_t dy_pitch;
    char *grad;
    uint64_t pitch;
    float *head, *tail; // [piece][dim_pad] partial sums of rows that cross pieces
    uint32_t rows, piece;
    float scale;
    int accumulate;
};

// The columns of one lane: VECTOR, the DType<DT>::kVec neighbours of one
// 16-byte vector; else four columns 32 apart (coalesced element accesses).
template <int DT, bool VECTOR> struct Columns {
    static constexpr int N = VECTOR ? DType<DT>::kVec : 4;
    uint64_t c0, dim;
    __device__ __forceinline__ Columns(uint64_t dim_, int lane)
        : c0(VECTOR ? (uint64_t)(blockIdx.y * (kSumThreads / 32) + threadIdx.x / 32) * 32 * N + lane * N
                    : (uint64_t)(blockIdx.y * (kSumThreads / 32) + threadIdx.x / 32) * 32 * N + lane),
          dim(dim_)
    {
    }
    __device__ __forceinline__ uint64_t col(int j) const { return VECTOR ? c0 + j : c0 + 32 * j; }
    // a row's values as loaded (nothing waits for them), and as fp32
    __device__ __forceinline__ uint4 fetch(const char *row) const
    {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (VECTOR) {
            if (c0 < dim)
                v = ld16(row + c0 * DType<DT>::kSize);
        } else {
            uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (col(j) < dim)
                    w[j] = ld_elem<DT>(row, col(j));
            v = make_uint4(w[0], w[1], w[2], w[3]);
        }
        return v;
    }
    __device__ __forceinline__ void values(const uint4 &v, float *f) const
    {
        if (VECTOR) {
            unpack<DT>(v, f);
        } else {
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                f[j] = __uint_as_float(DT == DT_BF16 ? w[j] << 16 : w[j]);
        }
    }
    __device__ __forceinline__ void load(const char *row, float *f) const { values(fetch(row), f); }
    __device__ __forceinline__ void store(char *row, float *f, float scale, bool accumulate) const
    {
        float old[N];
#pragma unroll
        for (int j = 0; j < N; ++j)
            f[j] = __fmul_rn(f[j], scale);
        if (accumulate) {
            load(row, old);
#pragma unroll
            for (int j = 0; j < N; ++j)
                f[j] = __fadd_rn(old[j], f[j]);
        }
        if (VECTOR) {
            if (c0 < dim)
                st16(row + c0 * DType<DT>::kSize, pack<DT>(f));
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j)
                if (col(j) < dim)
                    st_value<DT>(row, col(j), f[j]);
        }
    }
    __device__ __forceinline__ void load_partial(const float *row, float *f) const
    {
        if (VECTOR) {
#pragma unroll
            for (int j = 0; j < N; j += 4) {
                const uint4 v = c0 < dim ? ld16(row + c0 + j) : make_uint4(0, 0, 0, 0);
                unpack<DT_FP32>(v, f + j);
            }
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j)
                f[j] = col(j) < dim ? gload<float>(row + col(j)) : 0.0f;
        }
    }
    __device__ __forceinline__ void store_partial(float *row, const float *f) const
    {
        if (VECTOR) {
#pragma unroll
            for (int j = 0; j < N; j += 4)
                if (c0 < dim)
                    st16(row + c0 + j, pack<DT_FP32>(f + j));
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j)
                if (col(j) < dim)
                    gstore<float>(row + col(j), f[j]);
        }
    }
};

// The row of sorted token i, or ~0 outside the list (no row has that number).
__device__ __forceinline__ uint32_t row_at(const SumParams &p, uint64_t i)
{
    return i < p.ntokens ? gload<uint2>(p.sorted + i).x : 0xffffffffu;
}

// One warp sums one piece for its columns, kAhead rows' loads in flight.
template <int DT, bool VECTOR> __global__ void __launch_bounds__(kSumThreads) embed_sum_kernel(SumParams p)
{
    chain_entry();
    const int lane = threadIdx.x & 31;
    const Columns<DT, VECTOR> cols(p.dim, lane);
    constexpr int N = Columns<DT, VECTOR>::N;
    const uint64_t first = (uint64_t)blockIdx.x * p.piece;
    const int n = (int)umin64(p.piece, p.ntokens - first);
    // lane l holds token l of the piece
    static_assert(kMaxPiece <= 32, "a lane holds one token");
    const uint2 a = lane < n ? gload<uint2>(p.sorted + first + lane) : make_uint2(0xffffffffu, 0);
    const uint32_t prev = first ? row_at(p, first - 1) : 0xffffffffu;
    const uint32_t next = row_at(p, first + n);
    float acc[N];
    uint32_t row = __shfl_sync(0xffffffffu, a.x, 0);
    bool begins = row != prev;
#pragma unroll
    for (int j = 0; j < N; ++j)
        acc[j] = 0.0f;
    for (int i0 = 0; i0 < n; i0 += kAhead) {
        uint32_t r[kAhead];
        uint4 v[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            r[i] = __shfl_sync(0xffffffffu, a.x, i0 + i);
            const uint32_t t = __shfl_sync(0xffffffffu, a.y, i0 + i);
            if (r[i] < p.rows)
                v[i] = cols.fetch(p.dy + (uint64_t)t * p.dy_pitch);
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (r[i] != row) {
                // the run of `row` ends before token i0 + i
                if (row < p.rows) {
                    if (begins)
                        cols.store(p.grad + (uint64_t)row * p.pitch, acc, p.scale, p.accumulate);
                    else
                        cols.store_partial(p.head + blockIdx.x * p.dim_pad, acc);
                }
                row = r[i];
                begins = true;
#pragma unroll
                for (int j = 0; j < N; ++j)
                    acc[j] = 0.0f;
            }
            if (r[i] < p.rows) {
                float f[N];
                cols.values(v[i], f);
#pragma unroll
                for (int j = 0; j < N; ++j)
                    acc[j] = __fadd_rn(acc[j], f[j]);
            }
        }
    }
    if (row < p.rows) { // the piece's last run (a full piece: it did not end above)
        if (!begins)
            cols.store_partial(p.head + blockIdx.x * p.dim_pad, acc);
        else if (row == next)
            cols.store_partial(p.tail + blockIdx.x * p.dim_pad, acc);
        else
            cols.store(p.grad + (uint64_t)row * p.pitch, acc, p.scale, p.accumulate);
    }
}

// The rows that begin in piece blockIdx.x and go on in the next one: their
// partial sums, in order, four at a time in flight.
template <int DT, bool VECTOR> __global__ void __launch_bounds__(kSumThreads) embed_join_kernel(SumParams p)
{
    chain_entry();
    const int lane = threadIdx.x & 31;
    const Columns<DT, VECTOR> cols(p.dim, lane);
    constexpr int N = Columns<DT, VECTOR>::N;
    const uint64_t first = (uint64_t)blockIdx.x * p.piece;
    if (first + p.piece >= p.ntokens)
        return; // the last piece
    const uint32_t row = row_at(p, first + p.piece - 1);
    const uint32_t next = row_at(p, first + p.piece), begin = row_at(p, first);
    const uint32_t prev = first ? row_at(p, first - 1) : 0xffffffffu;
    if (row >= p.rows || next != row)
        return;
    // it goes on; it began here unless the whole piece and the token before are its own
    if (begin == row && prev == row)
        return;
    float acc[N];
    cols.load_partial(p.tail + blockIdx.x * p.dim_pad, acc);
    for (uint64_t q = blockIdx.x + 1;;) {
        // the pieces that begin with this row, 32 looked at together
        const unsigned go = __ballot_sync(0xffffffffu, row_at(p, (q + lane) * p.piece) == row);
        const int n = go == 0xffffffffu ? 32 : __ffs(~go) - 1;
        for (int i0 = 0; i0 < n; i0 += 4) {
            float f[4][N];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i0 + i < n)
                    cols.load_partial(p.head + (q + i0 + i) * p.dim_pad, f[i]);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i0 + i < n)
#pragma unroll
                    for (int j = 0; j < N; ++j)
                        acc[j] = __fadd_rn(acc[j], f[i][j]);
        }
        if (n < 32)
            break;
        q += 32;
    }
    cols.store(p.grad + (uint64_t)row * p.pitch, acc, p.scale, p.accumulate);
}

// ------------------------------------------------------------------ host side

bool aligned16(const void *p, size_t pitch, size_t row_bytes)
{
    return ((uintptr_t)p | pitch | row_bytes) % 16 == 0;
}

// Tokens a piece: eight, doubled up to 32 while that
// still leaves more warps than the GPU holds about half full (152 SMs x 32
// warps; a warp covers at least 128 columns).
uint32_t piece_of(size_t ntokens, size_t dim)
{
    uint32_t n = kMinPiece;
    while (n < kMaxPiece && (ntokens / n) * ((dim + 127) / 128) > 152 * 32)
        n *= 2;
    return n;
}

constexpr size_t kMaxRows = 0x7fffffff; // rows and tokens are 32-bit in the sorted list
constexpr size_t kMaxDim = (size_t)1 << 24; // columns: the second dimension of the sums' grid

template <int DT>
cudaError_t launch_sums(const SumParams &p, bool vector, uint32_t npieces, cudaStream_t stream)
{
    const uint64_t per = (uint64_t)kSumThreads * (vector ? DType<DT>::kVec : 4);
    const dim3 grid(npieces, (unsigned)((p.dim + per - 1) / per));
    cudaError_t e;
    if ((e = launch_chained(vector ? embed_sum_kernel<DT, true> : embed_sum_kernel<DT, false>, grid, dim3(kSumThreads), 0,
                            stream, p)) != cudaSuccess)
        return e;
    count_launches(1);
    if (npieces > 1) {
        if ((e = launch_chained(vector ? embed_join_kernel<DT, true> : embed_join_kernel<DT, false>, grid,
                                dim3(kSumThreads), 0, stream, p)) != cudaSuccess)
            return e;
        count_launches(1);
    }
    return cudaSuccess;
}

ccl_status_t embedding_impl(const void *table, size_t rows, size_t dim, size_t table_stride, ccl_dtype_t dtype,
                            const int64_t *ids, size_t ntokens, int64_t first_row, float scale, void *out,
                            size_t out_stride, cudaStream_t stream)
{
    if (!valid_dtype(dtype) || table_stride < dim || out_stride < dim || rows > kMaxRows || ntokens > kMaxRows ||
        dim > kMaxDim)
        return CCL_ERR_INVALID_ARG;
    const size_t es = elem_size(dtype);
    size_t tb, ob;
    if (!extent(rows, dim, table_stride, es, &tb) || !extent(ntokens, dim, out_stride, es, &ob))
        return CCL_ERR_INVALID_ARG;
    if (ntokens == 0 || dim == 0)
        return CCL_OK;
    if ((!table && rows) || !ids || !out || !element_aligned(es, {table, out}) || !element_aligned(8, {ids}))
        return CCL_ERR_INVALID_ARG;
    const std::vector<Range> w{range_of(out, ob, 0)}, r{range_of(table, tb, 0), range_of(ids, ntokens * 8, 0)};
    if (ccl_status_t st = check_overlaps(w, r, [](const Range &, const Range &) { return false; }))
        return st;
#ifdef CCL_DEBUG_BOUNDS
    if (cudaError_t e = dbg_set_ranges({{table, tb}, {ids, ntokens * 8}, {out, ob}}, stream))
        return from_cuda(e);
#endif
    EmbedParams p{static_cast<const char *>(table), static_cast<char *>(out), ids, ntokens, rows, dim,
                  table_stride * es, out_stride * es, first_row, scale};
    const bool vec = aligned16(table, p.table_pitch, dim * es) && aligned16(out, p.out_pitch, dim * es);
    const uint64_t items = vec ? dim * es / 16 : dim;
    unsigned tx = 1;
    while (tx < 128 && tx < items)
        tx *= 2;
    const dim3 block(tx, 128 / tx), grid((unsigned)((ntokens + block.y - 1) / block.y));
    if (dtype == CCL_FP32)
        (vec ? embed_kernel<DT_FP32, true> : embed_kernel<DT_FP32, false>)<<<grid, block, 0, stream>>>(p);
    else
        (vec ? embed_kernel<DT_BF16, true> : embed_kernel<DT_BF16, false>)<<<grid, block, 0, stream>>>(p);
    count_launches(1);
    return from_cuda(cudaGetLastError());
}

struct GradWork {
    size_t sorted, partial, bytes; // one list of pairs, one array of partial sums, everything
};

bool grad_work(size_t ntokens, size_t dim, GradWork *w)
{
    const size_t pad = (dim + 3) / 4 * 4, np = (ntokens + piece_of(ntokens, dim) - 1) / piece_of(ntokens, dim);
    if (mul_overflows(np, pad * 16))
        return false;
    w->sorted = up(ntokens * sizeof(uint2));
    w->partial = np > 1 ? up(np * pad * 4) : 0; // one piece leaves no partial sums
    w->bytes = 2 * (w->sorted + w->partial);
    return true;
}

ccl_status_t embedding_grad_impl(const void *grad_out, size_t grad_out_stride, const int64_t *ids, size_t ntokens,
                                 int64_t first_row, size_t rows, size_t dim, ccl_dtype_t dtype, float scale,
                                 int accumulate, void *grad_table, size_t grad_table_stride, void *work,
                                 size_t work_bytes, cudaStream_t stream)
{
    if (!valid_dtype(dtype) || grad_out_stride < dim || grad_table_stride < dim || rows > kMaxRows ||
        ntokens > kMaxRows || dim > kMaxDim)
        return CCL_ERR_INVALID_ARG;
    const size_t es = elem_size(dtype);
    size_t yb, gb;
    GradWork gw;
    if (!extent(ntokens, dim, grad_out_stride, es, &yb) || !extent(rows, dim, grad_table_stride, es, &gb) ||
        !grad_work(ntokens, dim, &gw))
        return CCL_ERR_INVALID_ARG;
    if (rows == 0 || dim == 0 || (ntokens == 0 && accumulate))
        return CCL_OK;
    if (!grad_table || (ntokens && (!grad_out || !ids || !work || (uintptr_t)work % 16 || work_bytes < gw.bytes)))
        return CCL_ERR_INVALID_ARG;
    if (!element_aligned(es, {grad_out, grad_table}) || !element_aligned(8, {ids}))
        return CCL_ERR_INVALID_ARG;
    std::vector<Range> w{range_of(grad_table, gb, 0)}, r;
    if (ntokens) {
        w.push_back(range_of(work, gw.bytes, 0));
        r = {range_of(grad_out, yb, 0), range_of(ids, ntokens * 8, 0)};
    }
    if (ccl_status_t st = check_overlaps(w, r, [](const Range &, const Range &) { return false; }))
        return st;
#ifdef CCL_DEBUG_BOUNDS
    if (cudaError_t e = dbg_set_ranges({{grad_table, gb}, {work, gw.bytes}, {grad_out, yb}, {ids, ntokens * 8}}, stream))
        return from_cuda(e);
#endif
    char *wp = static_cast<char *>(work);
    SortParams s{};
    s.ids = ids;
    s.ntokens = ntokens;
    s.first_row = first_row;
    s.rows = (uint32_t)rows;
    s.buf[0] = reinterpret_cast<uint2 *>(wp);
    s.buf[1] = reinterpret_cast<uint2 *>(wp + gw.sorted);
    int bits = 1;
    while (rows >> bits) // keys are 0 .. rows
        ++bits;
    s.passes = (bits + 7) / 8;
    s.bits = (bits + s.passes - 1) / s.passes;
    s.grad = static_cast<char *>(grad_table);
    s.pitch = grad_table_stride * es;
    s.row_bytes = dim * es;
    s.elem = (int)es;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = stream;
    s.rank_ctas = ntokens <= kFewIds ? (uint32_t)((ntokens + kRanked - 1) / kRanked) : 0;
    if (!accumulate) {
        int sms = 0, dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return CCL_ERR_CUDA;
        s.zero_ctas = (uint32_t)std::min<size_t>(rows, 2 * (size_t)sms); // all resident
    }
    if (s.zero_ctas + s.rank_ctas) {
        cfg.gridDim = dim3(s.zero_ctas + s.rank_ctas);
        cfg.blockDim = dim3(kZeroThreads);
        if (cudaError_t e = cudaLaunchKernelEx(&cfg, embed_zero_kernel, s))
            return from_cuda(e);
        count_launches(1);
    }
    if (ntokens == 0)
        return CCL_OK;
    if (!s.rank_ctas) {
        cfg.gridDim = dim3(kSortCtas);
        cfg.blockDim = dim3(kSortThreads);
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = kSortCtas;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[1].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = accumulate ? 1 : 2; // under the zeros' tail, when there are any
        if (cudaError_t e = cudaLaunchKernelEx(&cfg, embed_sort_kernel, s))
            return from_cuda(e);
        count_launches(1);
    }
    SumParams p{};
    p.sorted = s.buf[s.rank_ctas ? 0 : (s.passes - 1) & 1];
    p.ntokens = ntokens;
    p.dim = dim;
    p.dim_pad = (dim + 3) / 4 * 4;
    p.dy = static_cast<const char *>(grad_out);
    p.dy_pitch = grad_out_stride * es;
    p.grad = s.grad;
    p.pitch = s.pitch;
    p.head = reinterpret_cast<float *>(wp + 2 * gw.sorted);
    p.tail = reinterpret_cast<float *>(wp + 2 * gw.sorted + gw.partial);
    p.rows = s.rows;
    p.piece = piece_of(ntokens, dim);
    p.scale = scale;
    p.accumulate = accumulate != 0;
    const bool vec = aligned16(grad_out, p.dy_pitch, dim * es) && aligned16(grad_table, p.pitch, dim * es);
    const uint32_t np = (uint32_t)((ntokens + p.piece - 1) / p.piece);
    return from_cuda(dtype == CCL_FP32 ? launch_sums<DT_FP32>(p, vec, np, stream)
                                       : launch_sums<DT_BF16>(p, vec, np, stream));
}

} // namespace
} // namespace ccl

using namespace ccl;

extern "C" {

ccl_status_t ccl_plan_embedding_grad_work_bytes(size_t ntokens, size_t rows, size_t dim, size_t *bytes)
{
    GradWork w;
    if (!bytes || ntokens > kMaxRows || rows > kMaxRows || dim > kMaxDim || !grad_work(ntokens, dim, &w))
        return CCL_ERR_INVALID_ARG;
    *bytes = w.bytes;
    return CCL_OK;
}

ccl_status_t ccl_embedding(const void *table, size_t rows, size_t dim, size_t table_stride, ccl_dtype_t dtype,
                           const int64_t *ids, size_t ntokens, int64_t first_row, float scale, void *out,
                           size_t out_stride, cudaStream_t stream)
{
    TraceScope tr("embedding", 1, ntokens, (int)dtype, -1, 0, stream);
    return tr.done(guarded([&] {
        return embedding_impl(table, rows, dim, table_stride, dtype, ids, ntokens, first_row, scale, out,
                  out_stride, stream);
    }));
}

ccl_status_t ccl_embedding_grad(const void *grad_out, size_t grad_out_stride, const int64_t *ids, size_t ntokens,
                                int64_t first_row, size_t rows, size_t dim, ccl_dtype_t dtype, float scale,
                                int accumulate, void *grad_table, size_t grad_table_stride, void *work,
                                size_t work_bytes, cudaStream_t stream)
{
    TraceScope tr("embedding_grad", 1, ntokens, (int)dtype, -1, 0, stream);
    return tr.done(guarded([&] {
        return embedding_grad_impl(grad_out, grad_out_stride, ids, ntokens, first_row, rows, dim, dtype, scale,
                       accumulate, grad_table, grad_table_stride, work, work_bytes, stream);
    }));
}

} // extern "C"
