// kvq_pages_attn.cuh -- attention over the paged 4-bit cache.
#pragma once

#include "kvq_pages.cuh"

namespace kvq {

struct AttnArgs {
    Batch b;
    Pool p;
    const void* q;
    void* out;
    float* lse;
    long long q_row, q_head, o_row, o_head;  // strides, elements
    const int8_t* signs;
    int rows, Hq, G;
    int causal, window;
    float scale, rsqd;
};

// The plainest form: one CTA per (row, query head), one token a thread for
// the scores, one channel a thread for the values, online softmax.
template <int D, typename T, bool HAD>
__global__ void __launch_bounds__(128) pages_attn_simple_kernel(AttnArgs a) {
    __shared__ float sq[D], sp[128], red[4];
    __shared__ long long sslot[128];
    const int row = blockIdx.x, j = blockIdx.y, g = j / a.G, tid = threadIdx.x;
    const int s = owner_of(a.b.start, a.b.n_seqs, row);
    if (s < 0) return;
    const int len = max(a.b.len[s], 0), pos = a.b.len[s] - a.b.start[s + 1] + row;
    int t1 = a.causal ? min(pos + 1, len) : len;
    const int t0 = a.causal && a.window > 0 ? max(pos - a.window + 1, 0) : 0;
    if (tid < D) {
        const T x = static_cast<const T*>(a.q)[row * a.q_row + j * a.q_head + tid];
        sq[tid] = (float)x * (HAD && a.signs ? (float)a.signs[tid] : 1.0f);
    }
    __syncthreads();
    auto turn = [&]() {
        for (int h = 1; h < D; h <<= 1) {
            float v = 0;
            if (tid < D) v = (tid & h) ? sq[tid ^ h] - sq[tid] : sq[tid] + sq[tid ^ h];
            __syncthreads();
            if (tid < D) sq[tid] = v;
            __syncthreads();
        }
        if (tid < D) sq[tid] *= a.rsqd;
        __syncthreads();
    };
    if (HAD) turn();
    float m = -INFINITY, l = 0, acc = 0;
    for (int base = t0; base < t1; base += 128) {
        const int tok = base + tid;
        long long slot = -1;
        float x = -INFINITY;
        if (tok < t1) slot = slot_of(a.b, a.p, s, tok);
        if (slot >= 0) {
            slot += (long long)g << a.p.page_log2;
            const uint8_t* c = a.p.codes[0] + slot * (D / 2);
            float d = 0;
            for (int k = 0; k < D / 2; ++k)
                d += sq[2 * k] * (float)((c[k] & 15) - 8) + sq[2 * k + 1] * (float)((c[k] >> 4) - 8);
            x = d * __half2float(a.p.tok[0][slot]) * a.scale;
        }
        sslot[tid] = slot;
        float mm = x;
        for (int o = 16; o; o >>= 1) mm = fmaxf(mm, __shfl_xor_sync(~0u, mm, o));
        if ((tid & 31) == 0) red[tid >> 5] = mm;
        __syncthreads();
        mm = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
        const float m2 = fmaxf(m, mm);
        const float keep = m2 == -INFINITY ? 1.0f : expf(m - m2);
        const float p = slot < 0 ? 0.0f : expf(x - m2);
        sp[tid] = slot < 0 ? 0.0f : p * __half2float(a.p.tok[1][slot]);
        float ps = p;
        for (int o = 16; o; o >>= 1) ps += __shfl_xor_sync(~0u, ps, o);
        __syncthreads();
        if ((tid & 31) == 0) red[tid >> 5] = ps;
        __syncthreads();
        l = l * keep + red[0] + red[1] + red[2] + red[3];
        m = m2;
        acc *= keep;
        if (tid < D)
            for (int k = 0; k < min(128, t1 - base); ++k)
                if (sslot[k] >= 0) {
                    const int b = a.p.codes[1][sslot[k] * (D / 2) + (tid >> 1)];
                    acc += sp[k] * (float)(((tid & 1 ? b >> 4 : b) & 15) - 8);
                }
        __syncthreads();
    }
    if (tid < D) sq[tid] = l == 0.0f ? 0.0f : acc / l;
    __syncthreads();
    if (HAD) turn();
    if (tid < D) {
        float o = sq[tid] * (HAD && a.signs ? (float)a.signs[tid] : 1.0f);
        const uint32_t u = Elem<T>::pack(o, o);
        static_cast<T*>(a.out)[row * a.o_row + j * a.o_head + tid] = *reinterpret_cast<const T*>(&u);
    }
    if (tid == 0 && a.lse) a.lse[(long long)row * a.Hq + j] = m + logf(l);
}

}  // namespace kvq
