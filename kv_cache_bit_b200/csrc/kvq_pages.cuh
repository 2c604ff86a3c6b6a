// kvq_pages.cuh -- paged 4-bit cache: writing rows into their slots and
// reading them back.
//
// One vector (a row's head of K or V) belongs to a quad of lanes; lane t of
// the quad holds its eight-channel pieces t, t + 4, .., so that a quad's loads
// and stores of 16-bit values are 64 bytes in a row.  Butterflies of strides
// 1, 2, 4 and 32, 64 stay in the lane's registers, those of strides 8 and 16
// exchange with lanes t ^ 1 and t ^ 2.  Where there are enough vectors to fill
// the GPU a quad takes several heads of its row: the search for the row's
// sequence and page, about as many instructions as half a vector, is then made
// once for them.
//
// A warp's instructions for eight vectors (D = 128, rotated): 517 writing, in
// packed fp32 pairs, 66 of them shuffles; 387 reading, whose butterflies are
// exact in fp16 pairs (sums of codes stay below 1024).  32 x 4096 rows, 8 kv
// heads: 177 us to write (HBM would take 103), 126 us to read back (103).
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

// Packed fp32 pairs.
__device__ __forceinline__ uint64_t pair2(float x, float y) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ void unpair2(uint64_t v, float& x, float& y) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
}
__device__ __forceinline__ uint64_t fma_f2(uint64_t x, uint64_t y, uint64_t z) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
    return r;
}
__device__ __forceinline__ uint64_t mul_f2(uint64_t x, uint64_t y) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
    return r;
}
__device__ __forceinline__ uint64_t add_f2(uint64_t x, uint64_t y) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
    return r;
}
// Packed fp16 pairs.
__device__ __forceinline__ uint32_t add_h2(uint32_t x, uint32_t y) {
    uint32_t r;
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
    return r;
}
__device__ __forceinline__ uint32_t sub_h2(uint32_t x, uint32_t y) {
    uint32_t r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
    return r;
}
__device__ __forceinline__ uint32_t fma_h2(uint32_t x, uint32_t y, uint32_t z) {
    uint32_t r;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(y), "r"(z));
    return r;
}
template <uint32_t MASK, uint32_t BASE>
__device__ __forceinline__ uint32_t in_mantissa(uint32_t w) {  // (w & MASK) | BASE: one lop3
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w), "n"(MASK), "r"(BASE));
    return r;
}
// The codes of nibbles 0 and 4 of a word as two fp16, exactly.
__device__ __forceinline__ uint32_t codes_low(uint32_t w) {  // (1024 + e) - 1032
    return add_h2(in_mantissa<0x000F000Fu, 0x64006400u>(w), 0xE408E408u);
}
// Those of nibbles 1 and 5: (1024 + 16 e) / 16 - 72.
__device__ __forceinline__ uint32_t codes_upper(uint32_t w) {
    return fma_h2(in_mantissa<0x00F000F0u, 0x64006400u>(w), 0x2C002C00u, 0xD480D480u);
}

// A row's sequence, page and slot (head 0), or -1.
__device__ __forceinline__ long long slot_of_row(const Batch& b, const Pool& p, const int* start, int row, int* seq) {
    const int s = owner_of(start, b.n_seqs, row);
    *seq = s;
    if (s < 0) return -1;
    const int pos = b.len[s] - (start[s + 1] - start[s]) + (row - start[s]);
    return pos >= 0 ? slot_of(b, p, s, pos) : -1;
}

struct WriteArgs {
    Batch b;
    Pool p;
    const void* x[2];
    long long row_stride[2], head_stride[2];  // elements
    const int8_t* signs;
    int rows;
    int per;  // heads a quad takes
    float rsqd;
};

constexpr int kWriteThreads = 128;

// blockIdx.y: K or V.
template <int D, typename T, bool HAD>
__global__ void __launch_bounds__(kWriteThreads) pages_write_kernel(WriteArgs a) {
    constexpr int KC = D / 32;  // pieces a lane
    __shared__ int s_start[kStartStage];
    __shared__ alignas(16) uint32_t s_sign[D / 2];  // sign bits of two neighbouring channels' signs
    const int i = blockIdx.y, t = threadIdx.x & 3, H = a.p.H;
    grid_dep_wait();
    grid_dep_launch();
    const int* start = stage_start(a.b, s_start);
    if (HAD && threadIdx.x < D / 2)
        s_sign[threadIdx.x] = a.signs == nullptr ? 0u
                                                 : (a.signs[2 * threadIdx.x] < 0 ? 0x8000u : 0u) |
                                                       (a.signs[2 * threadIdx.x + 1] < 0 ? 0x80000000u : 0u);
    const int groups = (H + a.per - 1) / a.per;
    const int quad = (int)((blockIdx.x * (unsigned)kWriteThreads + threadIdx.x) >> 2);
    const int row = quad / groups, h0 = (quad - row * groups) * a.per, h1 = min(h0 + a.per, H);
    const T* src = static_cast<const T*>(a.x[i]) + row * a.row_stride[i] + t * 8;
    uint4 next[KC];
    const auto load = [&](int h) {
#pragma unroll
        for (int k = 0; k < KC; ++k)
            next[k] = *reinterpret_cast<const uint4*>(src + h * a.head_stride[i] + 32 * k);
    };
    if (row < a.rows) load(h0);
    __syncthreads();
    if (row >= a.rows) return;
    int seq;
    const long long slot0 = slot_of_row(a.b, a.p, start, row, &seq);
    if (slot0 < 0) return;  // the four lanes of a quad agree

    const uint32_t lanes = 0xFu << (threadIdx.x & 28);
#pragma unroll 1
    for (int h = h0; h < h1; ++h) {
        uint32_t u[4 * KC], big = 0;
#pragma unroll
        for (int k = 0; k < KC; ++k) {
            u[4 * k] = next[k].x, u[4 * k + 1] = next[k].y, u[4 * k + 2] = next[k].z, u[4 * k + 3] = next[k].w;
#pragma unroll
            for (int j = 0; j < 4; ++j) big = max_u16x2(big, u[4 * k + j] & 0x7FFF7FFFu);
            if constexpr (HAD) {  // signs, on the inputs' own bits
                const uint4 sg = *reinterpret_cast<const uint4*>(&s_sign[(4 * k + t) * 4]);
                u[4 * k] ^= sg.x, u[4 * k + 1] ^= sg.y, u[4 * k + 2] ^= sg.z, u[4 * k + 3] ^= sg.w;
            }
        }
        if (h + 1 < h1) load(h + 1);
        float v[8 * KC];  // piece k's channels at 8 k
#pragma unroll
        for (int k = 0; k < 4 * KC; ++k) {
            const float2 f = Elem<T>::wide(u[k]);
            v[2 * k] = f.x, v[2 * k + 1] = f.y;
        }
        if ((big & 0xFFFFu) >= Elem<T>::kSpecial || (big >> 16) >= Elem<T>::kSpecial) {
#pragma unroll
            for (int k = 0; k < 8 * KC; ++k) v[k] = clean(v[k]);
        }
        // pairs of pieces KC / 2 apart, so that all strides but the last are whole pairs'
        constexpr int NP = 4 * KC, KH = KC / 2;
        uint64_t p[NP];
#pragma unroll
        for (int k = 0; k < KH; ++k)
#pragma unroll
            for (int e = 0; e < 8; ++e) p[8 * k + e] = pair2(v[8 * k + e], v[8 * (k + KH) + e]);
        if constexpr (HAD) {
            const uint64_t minus = pair2(-1.0f, -1.0f);
            const auto stage = [&](int x) {
#pragma unroll
                for (int k = 0; k < NP; ++k)
                    if (!(k & x)) {
                        const uint64_t lo = p[k], hi = p[k + x];
                        p[k] = add_f2(lo, hi);
                        p[k + x] = fma_f2(hi, minus, lo);
                    }
            };
            stage(1);
            stage(2);
            stage(4);
#pragma unroll
            for (int x = 1; x <= 2; x <<= 1) {
                const float sg = (t & x) ? -1.0f : 1.0f;
                const uint64_t sg2 = pair2(sg, sg);
#pragma unroll
                for (int k = 0; k < NP; ++k) {
                    float f, g;
                    unpair2(p[k], f, g);
                    p[k] = fma_f2(p[k], sg2,
                                  pair2(__shfl_xor_sync(lanes, f, x), __shfl_xor_sync(lanes, g, x)));
                }
            }
            if constexpr (KH == 2) stage(8);
            const uint64_t rs = pair2(a.rsqd, a.rsqd);
#pragma unroll
            for (int k = 0; k < NP; ++k) {
                float f, g;
                unpair2(p[k], f, g);
                p[k] = mul_f2(pair2(__fadd_rn(f, g), __fsub_rn(f, g)), rs);
            }
        }
        float m = 0.0f;
#pragma unroll
        for (int k = 0; k < NP; ++k) {
            float f, g;
            unpair2(p[k], f, g);
            m = fmaxf(m, fmaxf(fabsf(f), fabsf(g)));
        }
        m = fmaxf(m, __shfl_xor_sync(lanes, m, 1));
        m = fmaxf(m, __shfl_xor_sync(lanes, m, 2));
        const __half sigma = __float2half_rn(fminf(__fdiv_rn(m, 7.0f), 65504.0f));
        const float sf = __half2float(sigma);
        const float r = sf > 0.0f ? __frcp_rn(sf) : 0.0f;
        // Codes from the low mantissa bits of fma(y, r, 1.5 2^23 + 8): the FMA
        // rounds the exact product once, half to even.  Only a subnormal or
        // saturated scale can send a product past 7.5.
        if (__fmul_rn(m, r) > 7.25f) {
            const float top = 7.0f / r;  // any |y| in [7 sigma, 7.5 sigma) has the code 7
#pragma unroll
            for (int k = 0; k < NP; ++k) {
                float f, g;
                unpair2(p[k], f, g);
                p[k] = pair2(fminf(fmaxf(f, -top), top), fminf(fmaxf(g, -top), top));
            }
        }
        const uint64_t r2 = pair2(r, r), magic = pair2(12582912.0f + 8.0f, 12582912.0f + 8.0f);
        const long long slot = slot0 + ((long long)h << a.p.page_log2);
        uint32_t* dst = reinterpret_cast<uint32_t*>(a.p.codes[i] + slot * (D / 2)) + t;
#pragma unroll
        for (int k = 0; k < KH; ++k) {
            // sum of 16^e times the bits, 0x4B400000 + code each, modulo 2^32
            uint32_t lo = 0, hi = 0;
#pragma unroll
            for (int e = 7; e >= 0; --e) {
                float f, g;
                unpair2(fma_f2(p[8 * k + e], r2, magic), f, g);
                lo = lo * 16u + __float_as_uint(f);
                hi = hi * 16u + __float_as_uint(g);
            }
            constexpr uint32_t kBase = 0x4B400000u * 0x11111111u;
            dst[4 * k] = lo - kBase;
            dst[4 * (k + KH)] = hi - kBase;
        }
        if (t == 0) a.p.tok[i][slot] = sigma;
    }
}

struct ReadArgs {
    Batch b;
    Pool p;
    void* out[2];
    long long row_stride[2], head_stride[2];  // elements
    const int8_t* signs;
    int rows;
    int per;   // heads a quad takes
    int only;  // 0 or 1: that tensor alone; -1: both (blockIdx.y)
    float rsqd;
};

// Eight values at a 16-byte aligned place.
template <typename T>
__device__ __forceinline__ void store8(T* dst, const float (&v)[8]) {
    if constexpr (sizeof(T) == 4) {
        reinterpret_cast<float4*>(dst)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4*>(dst)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        *reinterpret_cast<uint4*>(dst) = make_uint4(Elem<T>::pack(v[0], v[1]), Elem<T>::pack(v[2], v[3]),
                                                    Elem<T>::pack(v[4], v[5]), Elem<T>::pack(v[6], v[7]));
    }
}

template <int D, typename T, bool HAD>
__global__ void __launch_bounds__(kWriteThreads) pages_read_kernel(ReadArgs a) {
    constexpr int KC = D / 32, NP = 4 * KC;
    __shared__ int s_start[kStartStage];
    __shared__ alignas(16) uint32_t s_sign[D / 2];  // sign bits of the signs of channels e and e + 4 of a piece
    const int i = a.only >= 0 ? a.only : blockIdx.y, t = threadIdx.x & 3, H = a.p.H;
    grid_dep_wait();
    grid_dep_launch();
    const int* start = stage_start(a.b, s_start);
    if (HAD && threadIdx.x < D / 2) {
        const int c = (threadIdx.x >> 2) * 8 + (threadIdx.x & 3);
        s_sign[threadIdx.x] = a.signs == nullptr
                                  ? 0u : (a.signs[c] < 0 ? 0x8000u : 0u) | (a.signs[c + 4] < 0 ? 0x80000000u : 0u);
    }
    __syncthreads();
    const int groups = (H + a.per - 1) / a.per;
    const int quad = (int)((blockIdx.x * (unsigned)kWriteThreads + threadIdx.x) >> 2);
    const int row = quad / groups, h0 = (quad - row * groups) * a.per, h1 = min(h0 + a.per, H);
    if (row >= a.rows) return;
    int seq;
    const long long slot0 = slot_of_row(a.b, a.p, start, row, &seq);
    if (seq < 0) return;
    T* dst = static_cast<T*>(a.out[i]) + row * a.row_stride[i] + t * 8;
    if (slot0 < 0) {
        const float zero[8] = {};
        for (int h = h0; h < h1; ++h)
#pragma unroll
            for (int k = 0; k < KC; ++k) store8<T>(dst + h * a.head_stride[i] + 32 * k, zero);
        return;
    }
    const uint32_t lanes = 0xFu << (threadIdx.x & 28);
    uint32_t next[KC];
    __half next_sigma;
    const auto load = [&](int h) {
        const long long at = slot0 + ((long long)h << a.p.page_log2);
#pragma unroll
        for (int k = 0; k < KC; ++k)
            next[k] = reinterpret_cast<const uint32_t*>(a.p.codes[i] + at * (D / 2))[4 * k + t];
        next_sigma = a.p.tok[i][at];
    };
    load(h0);
#pragma unroll 1
    for (int h = h0; h < h1; ++h) {
        uint32_t p[NP];  // channels e and e + 4 of piece k at 4 k + e
#pragma unroll
        for (int k = 0; k < KC; ++k) {
            const uint32_t w = next[k], w8 = w >> 8;
            p[4 * k] = codes_low(w);
            p[4 * k + 1] = codes_upper(w);
            p[4 * k + 2] = codes_low(w8);
            p[4 * k + 3] = codes_upper(w8);
        }
        const float sf = __half2float(next_sigma);
        if (h + 1 < h1) load(h + 1);
        float f = sf;
        if constexpr (HAD) {
            f = __fmul_rn(sf, a.rsqd);
            const auto stage = [&](int x) {
#pragma unroll
                for (int k = 0; k < NP; ++k)
                    if (!(k & x)) {
                        const uint32_t lo = p[k], hi = p[k + x];
                        p[k] = add_h2(lo, hi);
                        p[k + x] = sub_h2(lo, hi);
                    }
            };
            stage(1);
            stage(2);
#pragma unroll
            for (int k = 0; k < NP; ++k)  // (x, y) to (x + y, x - y)
                p[k] = fma_h2(p[k], 0xBC003C00u, __byte_perm(p[k], p[k], 0x1032));
#pragma unroll
            for (int x = 1; x <= 2; x <<= 1) {
                const uint32_t sg = (t & x) ? 0xBC00BC00u : 0x3C003C00u;
#pragma unroll
                for (int k = 0; k < NP; ++k) p[k] = fma_h2(p[k], sg, __shfl_xor_sync(lanes, p[k], x));
            }
            stage(4);
            if constexpr (KC == 4) stage(8);
#pragma unroll
            for (int k = 0; k < KC; ++k) {
                const uint4 sg = *reinterpret_cast<const uint4*>(&s_sign[(4 * k + t) * 4]);
                p[4 * k] ^= sg.x, p[4 * k + 1] ^= sg.y, p[4 * k + 2] ^= sg.z, p[4 * k + 3] ^= sg.w;
            }
        }
#pragma unroll
        for (int k = 0; k < KC; ++k) {
            float v[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&p[4 * k + e]));
                v[e] = x.x * f, v[e + 4] = x.y * f;
            }
            store8<T>(dst + h * a.head_stride[i] + 32 * k, v);
        }
    }
}

}  // namespace kvq
