// kvq_pages_attn.cuh -- attention over the paged 4-bit cache: what the kernels
// share (arguments, ranges of rows, the softmax's scaling, the last steps of a
// row), and the merge of partial states.
//
// The softmax with the value scale inside.  With x_t the score of token t in
// the log2 domain and sigma_t its value scale, the generation-step kernel forms
//   y_t = x_t + log2 sigma_t,   w_t = 2^(y_t - M + kBias),   M >= max y_t
//   o = sum_t w_t q^V_t,        l = sum_t w_t / sigma_t
// so that o / l is the softmax average and M + log2 l - kBias its logarithm
// (base 2).  w is the only value that is rounded to fp16, at most 2^kBias and
// normal down to 2^-29 of the largest, whatever the scales are; one addition
// replaces the product with sigma.  A scale of 0 (a zero vector) counts as
// 2^-24 in y and 1 / sigma: its codes are all 0.  (The tile kernel's form
// stands there; it leaves the same M, l and o.)
#pragma once

#include "kvq_pages.cuh"

namespace kvq {

constexpr float kBias = 15.0f;
constexpr float kLowest = -3.0e38f;  // M before any token: finite, so that M - M is 0
constexpr float kLn2 = 0.693147180559945f;

struct AttnArgs {
    Batch b;
    Pool p;
    const void* q;
    void* out;
    float* lse;
    long long q_row, q_head, o_row, o_head;  // strides, elements
    const int8_t* signs;
    int rows, Hq, G, bf16;
    int causal, window;
    float scale2, rsqd;  // scale * log2 e; 1 / sqrt(d)
    float* ml;           // partial states: M, l [slot][query][2]
    float* part;         // and o [slot][query][D]
    float* left;         // o of warps' first items [warp][query][D]
    int4* meta;          // [CTA]: sequence, head, first query, merged slots (0: nothing to merge)
};

// Tokens [t0, t1) that rows lo .. hi - 1 of a sequence see between them; its
// rows end before row `end` (hi <= end) and it has len >= 0 tokens.
struct Range {
    int t0, t1;
};
__device__ __forceinline__ Range seen_by(const AttnArgs& a, int len, int first, int last) {  // rows' tokens
    const int t1 = a.causal ? min(last + 1, len) : len;
    const int t0 = a.causal && a.window > 0 && first >= a.window ? first - a.window + 1 : 0;
    return t0 < t1 ? Range{t0, t1} : Range{0, 0};
}
__device__ __forceinline__ Range range_of(const AttnArgs& a, int len, int end, int lo, int hi) {
    Range r = seen_by(a, len, len + (lo - end), len + (hi - 1 - end));
    const int cap = a.b.max_pages << a.p.page_log2;  // below 2^31
    if (r.t1 > cap) {
        report_error(kErrRange);
        r.t1 = cap;
        if (r.t0 >= cap) r = Range{0, 0};
    }
    return r;
}

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float lg2(float x) {
    float r;
    asm("lg2.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// 2^k with k such that m 2^k is in [2^14, 2^15); for infinite or NaN m, NaN
// (the row's result is then NaN whatever its codes are).
__device__ __forceinline__ float query_scale(float m) {
    if (!(m < INFINITY)) return NAN;
    const int e = (int)(__float_as_uint(m) >> 23) - 127;
    return __uint_as_float((uint32_t)(min(max(14 - e, -126), 127) + 127) << 23);
}

// Channel of place `pos` in the order in which the generation-step kernel keeps o:
// pos = (nibble, word of a pair, row of the tensor core's tile).
template <int D>
__device__ __forceinline__ int channel_of(int pos) {
    const int g = pos & 7, w = (pos >> 3) & 1, j = pos >> 4;
    return D == 128 ? 16 * g + 8 * w + j : 8 * g + 4 * w + j;
}

// A warp's last steps for one row: o / l, the rotation back, out and lse.
// v[i] is o at place lane + 32 i.
template <int D, bool HAD>
__device__ __forceinline__ void finish_row(const AttnArgs& a, int row, int head, float (&v)[D / 32], float M, float l) {
    const int lane = threadIdx.x & 31;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) v[i] *= inv;
    if constexpr (HAD) {
        lane_stages<1, D / 32>(v);
#pragma unroll
        for (int x = 1; x < 32; x <<= 1) {
            const float sg = (lane & x) ? -1.0f : 1.0f;
#pragma unroll
            for (int i = 0; i < D / 32; ++i) v[i] = __fmaf_rn(v[i], sg, __shfl_xor_sync(~0u, v[i], x));
        }
    }
    uint16_t* dst = static_cast<uint16_t*>(a.out) + row * a.o_row + head * a.o_head;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
        const int c = channel_of<D>(lane + 32 * i);
        float x = v[i];
        if constexpr (HAD) x *= a.signs ? (float)a.signs[c] * a.rsqd : a.rsqd;
        dst[c] = (uint16_t)(a.bf16 ? Elem<__nv_bfloat16>::pack(x, x) : Elem<__half>::pack(x, x));
    }
    if (lane == 0 && a.lse) a.lse[(long long)row * a.Hq + head] = (M - kBias + lg2(l)) * kLn2;
}

// Merges the partial states of an item that several CTAs worked on.  One CTA a
// main-kernel CTA: those of CTAs that no split item starts in return at once.
// Slot 2b + 1 is the state of an item that CTA b began and did not end, slot
// 2b of one that it did not begin.  Warps beyond one a query share its states; the order of the sums is fixed.
constexpr int kMergeWarps = 16;

// Queries a block (blockIdx.y): items of many rows are merged of few states, those of few rows of up to one a CTA.
constexpr int merge_queries(int nq) { return nq > 16 ? 16 : 4; }

template <int D, int NQ, bool HAD>
__global__ void __launch_bounds__(kMergeWarps * 32) pages_merge_kernel(AttnArgs a) {
    constexpr int NB = merge_queries(NQ), W = kMergeWarps / NB;
    __shared__ float s_o[NB][W][D], s_l[NB][W];
    const int b = blockIdx.x, qb = (threadIdx.x >> 5) / W, part = (threadIdx.x >> 5) % W, lane = threadIdx.x & 31;
    const int qi = blockIdx.y * NB + qb;
    grid_dep_wait();
    grid_dep_launch();
    const int4 meta = a.meta[b];
    const int n = meta.w;
    if (n == 0) return;
    const int s = meta.x, h = meta.y, i = meta.z + qi;
    const int end = a.b.start[s + 1], lo = max(a.b.start[s], 0);
    const int row = lo + i / a.G, head = h * a.G + i % a.G;
    const auto slot = [&](int k) { return ((long long)(k == 0 ? 2 * b + 1 : 2 * (b + k)) * NQ + qi); };
    float M = kLowest;
    for (int k = lane; k < n; k += 32) M = fmaxf(M, a.ml[2 * slot(k)]);
#pragma unroll
    for (int x = 16; x; x >>= 1) M = fmaxf(M, __shfl_xor_sync(~0u, M, x));
    float v[D / 32] = {}, l = 0.0f;
#pragma unroll 4
    for (int k = part; k < n; k += W) {
        const long long at = slot(k);
        const float2 ml = reinterpret_cast<const float2*>(a.ml)[at];
        const float f = ex2(ml.x - M);
        l = __fmaf_rn(ml.y, f, l);
#pragma unroll
        for (int c = 0; c < D / 32; ++c) v[c] = __fmaf_rn(a.part[at * D + lane + 32 * c], f, v[c]);
    }
#pragma unroll
    for (int c = 0; c < D / 32; ++c) s_o[qb][part][lane + 32 * c] = v[c];
    if (lane == 0) s_l[qb][part] = l;
    __syncthreads();
    if (part != 0 || row >= min(end, a.rows)) return;
#pragma unroll
    for (int w = 1; w < W; ++w) {
        l += s_l[qb][w];
#pragma unroll
        for (int c = 0; c < D / 32; ++c) v[c] += s_o[qb][w][lane + 32 * c];
    }
    finish_row<D, HAD>(a, row, head, v, M, l);
}

}  // namespace kvq
