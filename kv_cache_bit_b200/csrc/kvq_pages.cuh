// kvq_pages.cuh -- paged 4-bit cache: writing rows into their slots and
// reading them back.
//
// One vector (a row's head of K or V) belongs to a quad of lanes; lane t of
// the quad holds its channels [t D/4, (t + 1) D/4), so that a lane's codes are
// one 16-byte (D = 128) or 8-byte store and a vector's codes one contiguous
// run.  Butterflies of strides below D/4 stay in the lane's registers, the
// last two exchange with lanes t ^ 1 and t ^ 2.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "kvq_device.cuh"

namespace kvq {

constexpr uint32_t kErrRange = 4u;  // a page number or token outside its range was left out

// The batch descriptor as the kernels use it.
struct Batch {
    const int* start;
    const int* len;
    const int* table;
    int n_seqs, max_pages, table_stride;
};

struct Pool {
    uint8_t* codes[2];
    __half* tok[2];
    int n_pages, H, page_log2;
};

// Staged part of start[]: batches of more sequences search it in global memory.
constexpr int kStartStage = 1024;

// Copies start[0 .. n_seqs] to shared memory where it fits; returns where to
// search.  The caller synchronizes the block.
__device__ __forceinline__ const int* stage_start(const Batch& b, int (&sm)[kStartStage]) {
    if (b.n_seqs >= kStartStage) return b.start;
    for (int i = threadIdx.x; i <= b.n_seqs; i += blockDim.x) sm[i] = b.start[i];
    return sm;
}

// The sequence whose rows start[s] .. start[s + 1] - 1 hold `row`, or -1.
__device__ __forceinline__ int owner_of(const int* start, int n_seqs, int row) {
    int lo = 0, hi = n_seqs;  // start[lo] <= row < start[hi] where there is an owner
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (start[mid] <= row) lo = mid;
        else hi = mid;
    }
    return start[lo] <= row && row < start[lo + 1] ? lo : -1;
}

// Index of token `pos` of sequence s in the pool's [page][H][slot] order, head
// 0; -1 where the page is refused (the error bit is set).  pos >= 0.
__device__ __forceinline__ long long slot_of(const Batch& b, const Pool& p, int s, int pos) {
    const int col = pos >> p.page_log2;
    if (col < b.max_pages) {
        const int page = b.table[(long long)s * b.table_stride + col];
        if (page >= 0 && page < p.n_pages)
            return (((long long)page * p.H) << p.page_log2) + (pos & ((1 << p.page_log2) - 1));
    }
    report_error(kErrRange);
    return -1;
}

template <typename T>
struct Elem;
template <>
struct Elem<__half> {
    static constexpr uint32_t kSpecial = 0x7C00u;  // magnitudes from here on are infinite or NaN
    __device__ static float2 wide(uint32_t u) { return __half22float2(*reinterpret_cast<__half2*>(&u)); }
    __device__ static uint32_t pack(float a, float b) {
        uint32_t r;  // a in the low half; saturates, and keeps NaN
        asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
        return r;
    }
};
template <>
struct Elem<__nv_bfloat16> {
    static constexpr uint32_t kSpecial = 0x4780u;  // 65536: past the range that is kept
    __device__ static float2 wide(uint32_t u) {
        return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
    }
    __device__ static uint32_t pack(float a, float b) {
        __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<uint32_t*>(&h);
    }
};

__device__ __forceinline__ float clean(float x) { return x != x ? 0.0f : fminf(fmaxf(x, -65504.0f), 65504.0f); }

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Butterflies of strides H, 2H, .. below N on a lane's own values.
template <int H, int N>
__device__ __forceinline__ void lane_stages(float (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N; i += 2 * H) {
#pragma unroll
        for (int j = 0; j < H; ++j) {
            const float a = v[i + j], b = v[i + j + H];
            v[i + j] = __fadd_rn(a, b);
            v[i + j + H] = __fsub_rn(a, b);
        }
    }
    if constexpr (2 * H < N) lane_stages<2 * H, N>(v);
}

struct WriteArgs {
    Batch b;
    Pool p;
    const void* x[2];
    long long row_stride[2], head_stride[2];  // elements
    const int8_t* signs;
    int rows;
    float rsqd;
};

constexpr int kWriteThreads = 256;

// blockIdx.y: K or V; a quad of lanes per (row, head) vector.
template <int D, typename T, bool HAD>
__global__ void __launch_bounds__(kWriteThreads) pages_write_kernel(WriteArgs a) {
    constexpr int N = D / 4;  // channels a lane
    __shared__ int s_start[kStartStage];
    const int i = blockIdx.y, t = threadIdx.x & 3;
    const int* start = stage_start(a.b, s_start);
    const int vec = (int)((blockIdx.x * (unsigned)kWriteThreads + threadIdx.x) >> 2);
    const int row = vec / a.p.H, h = vec - row * a.p.H;
    uint32_t u[N / 2];
    if (row < a.rows) {
        const T* src = static_cast<const T*>(a.x[i]) + row * a.row_stride[i] + h * a.head_stride[i] + t * N;
#pragma unroll
        for (int k = 0; k < N / 8; ++k) {
            const uint4 w = reinterpret_cast<const uint4*>(src)[k];
            u[4 * k] = w.x, u[4 * k + 1] = w.y, u[4 * k + 2] = w.z, u[4 * k + 3] = w.w;
        }
    }
    __syncthreads();
    int s = -1;
    if (row < a.rows) s = owner_of(start, a.b.n_seqs, row);
    long long slot = -1;
    if (s >= 0) {
        const int pos = a.b.len[s] - (start[s + 1] - start[s]) + (row - start[s]);
        if (pos >= 0) slot = slot_of(a.b, a.p, s, pos);
    }
    if (slot < 0) return;  // the four lanes of a quad agree

    const uint32_t quad = 0xFu << (threadIdx.x & 28);
    uint32_t big = 0;
#pragma unroll
    for (int k = 0; k < N / 2; ++k) big = max_u16x2(big, u[k] & 0x7FFF7FFFu);
    float v[N];
#pragma unroll
    for (int k = 0; k < N / 2; ++k) {
        const float2 f = Elem<T>::wide(u[k]);
        v[2 * k] = f.x, v[2 * k + 1] = f.y;
    }
    if ((big & 0xFFFFu) >= Elem<T>::kSpecial || (big >> 16) >= Elem<T>::kSpecial) {
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] = clean(v[k]);
    }
    if constexpr (HAD) {
        if (a.signs != nullptr) {
#pragma unroll
            for (int k = 0; k < N / 4; ++k) {
                const char4 c = reinterpret_cast<const char4*>(a.signs + t * N)[k];
                v[4 * k] *= c.x, v[4 * k + 1] *= c.y, v[4 * k + 2] *= c.z, v[4 * k + 3] *= c.w;
            }
        }
        lane_stages<1, N>(v);
#pragma unroll
        for (int x = 1; x <= 2; x <<= 1) {
            const float sg = (t & x) ? -1.0f : 1.0f;
#pragma unroll
            for (int k = 0; k < N; ++k) v[k] = __fmaf_rn(v[k], sg, __shfl_xor_sync(quad, v[k], x));
        }
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] = __fmul_rn(v[k], a.rsqd);
    }
    float m = 0.0f;
#pragma unroll
    for (int k = 0; k < N; ++k) m = fmaxf(m, fabsf(v[k]));
    m = fmaxf(m, __shfl_xor_sync(quad, m, 1));
    m = fmaxf(m, __shfl_xor_sync(quad, m, 2));
    const __half sigma = __float2half_rn(fminf(__fdiv_rn(m, 7.0f), 65504.0f));
    const float sf = __half2float(sigma);
    const float r = sf > 0.0f ? __frcp_rn(sf) : 0.0f;
    // Codes from the low mantissa bits of fma(y, r, 1.5 2^23 + 8): the FMA
    // rounds the exact product once, half to even.  Only a subnormal or
    // saturated scale can send a product past 7.5.
    if (__fmul_rn(m, r) > 7.25f) {
        const float top = 7.0f / r;  // any |y| in [7 sigma, 7.5 sigma) has the code 7
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] = fminf(fmaxf(v[k], -top), top);
    }
    constexpr float kMagic = 12582912.0f + 8.0f;
    uint32_t w[N / 8];
#pragma unroll
    for (int k = 0; k < N / 8; ++k) {
        uint32_t x = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) x |= (__float_as_uint(__fmaf_rn(v[8 * k + j], r, kMagic)) & 15u) << (4 * j);
        w[k] = x;
    }
    slot += (long long)h << a.p.page_log2;
    store_words(a.p.codes[i] + slot * (D / 2) + t * (N / 2), w);
    if (t == 0) a.p.tok[i][slot] = sigma;
}

struct ReadArgs {
    Batch b;
    Pool p;
    void* out[2];
    long long row_stride[2], head_stride[2];  // elements
    const int8_t* signs;
    int rows;
    int only;  // 0 or 1: that tensor alone; -1: both (blockIdx.y)
    float rsqd;
};

// Stores N consecutive values of type T at a 16-byte aligned place.
template <typename T, int N>
__device__ __forceinline__ void store_values(T* dst, const float (&v)[N]) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int k = 0; k < N / 4; ++k)
            reinterpret_cast<float4*>(dst)[k] = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
    } else {
#pragma unroll
        for (int k = 0; k < N / 8; ++k)
            reinterpret_cast<uint4*>(dst)[k] =
                make_uint4(Elem<T>::pack(v[8 * k], v[8 * k + 1]), Elem<T>::pack(v[8 * k + 2], v[8 * k + 3]),
                           Elem<T>::pack(v[8 * k + 4], v[8 * k + 5]), Elem<T>::pack(v[8 * k + 6], v[8 * k + 7]));
    }
}

template <int D, typename T, bool HAD>
__global__ void __launch_bounds__(kWriteThreads) pages_read_kernel(ReadArgs a) {
    constexpr int N = D / 4;
    __shared__ int s_start[kStartStage];
    const int i = a.only >= 0 ? a.only : blockIdx.y, t = threadIdx.x & 3;
    const int* start = stage_start(a.b, s_start);
    __syncthreads();
    const int vec = (int)((blockIdx.x * (unsigned)kWriteThreads + threadIdx.x) >> 2);
    const int row = vec / a.p.H, h = vec - row * a.p.H;
    if (row >= a.rows) return;
    const int s = owner_of(start, a.b.n_seqs, row);
    if (s < 0) return;
    const int pos = a.b.len[s] - (start[s + 1] - start[s]) + (row - start[s]);
    const long long slot = pos >= 0 ? slot_of(a.b, a.p, s, pos) : -1;
    float v[N];
    if (slot >= 0) {
        const long long at = slot + ((long long)h << a.p.page_log2);
        uint32_t w[N / 8];
        load_words(a.p.codes[i] + at * (D / 2) + t * (N / 2), w);
        const float sf = __half2float(a.p.tok[i][at]);
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] = (float)((int)((w[k >> 3] >> (4 * (k & 7))) & 15u) - 8);
        if constexpr (HAD) {
            const uint32_t quad = 0xFu << (threadIdx.x & 28);
            lane_stages<1, N>(v);  // sums of at most 128 codes: exact
#pragma unroll
            for (int x = 1; x <= 2; x <<= 1) {
                const float sg = (t & x) ? -1.0f : 1.0f;
#pragma unroll
                for (int k = 0; k < N; ++k) v[k] = __fmaf_rn(v[k], sg, __shfl_xor_sync(quad, v[k], x));
            }
            const float f = __fmul_rn(sf, a.rsqd);
            if (a.signs != nullptr) {
#pragma unroll
                for (int k = 0; k < N / 4; ++k) {
                    const char4 c = reinterpret_cast<const char4*>(a.signs + t * N)[k];
                    v[4 * k] *= c.x, v[4 * k + 1] *= c.y, v[4 * k + 2] *= c.z, v[4 * k + 3] *= c.w;
                }
            }
#pragma unroll
            for (int k = 0; k < N; ++k) v[k] *= f;
        } else {
#pragma unroll
            for (int k = 0; k < N; ++k) v[k] *= sf;
        }
    } else {
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] = 0.0f;
    }
    store_values(static_cast<T*>(a.out[i]) + row * a.row_stride[i] + h * a.head_stride[i] + t * N, v);
}

}  // namespace kvq
