// kvq_pages_step.cuh -- attention of few query rows a kv head (generation
// steps, a few drafted tokens): the paged cache is read once, straight into
// the registers of mma.m16n8k16.
//
// Work: an item is (sequence, kv head, up to NQ of the head's query rows); its
// cost is the number of 32-token units that the sequence's rows see.  All
// items laid end to end are cut into equal ranges, one a warp of a single-wave
// grid, whatever the lengths are: one long sequence is spread over the whole
// GPU, many short ones share warps.  pages_queries_kernel has rotated, scaled
// and split the queries once, in the order of the tensor core's fragments; it
// runs while this kernel looks for its ranges.  A warp works alone -- its own
// ring in shared memory is filled by cp.async that runs ahead over item
// borders -- and finishes the items that lie whole in its range.  What is left
// of items at the ends of the ranges is merged per CTA once all its warps are
// done, and what goes past a CTA by pages_merge_kernel.  (With ranges a CTA
// and its warps taking units in turn, each item's end stopped all warps: 105 us
// instead of 89 at 64 sequences of 500 .. 8192 tokens.)
//
// Per 16 tokens, channels and tokens permuted so that unpacking is cheap:
//   scores  A = K codes, exact in fp16: a nibble pair ORed into the mantissas of
//           1024 and less 1032 (or, from the upper nibbles, times 1 / 16 less
//           72).
//           B = the query, times a power of two for its row so that its
//           largest element is near 2^15.  A rotated query is split into fp16
//           high and low parts in neighbouring columns (22 bits of it are
//           kept); an input that is not rotated fits fp16 exactly.
//   values  A = V codes transposed (byte permutes pair two tokens' words), exact
//           as K's; B = w from the score fragments by movmatrix.  (Codes with a
//           bias, which save the addition, are no good: the sum of w (q + 72)
//           grows with the number of tokens, that of w q with its root, and the
//           72 sum w taken away at the end leaves the accumulator's rounding,
//           3e-2 of the outputs after 4800 tokens of equal weights.  The bits
//           taken as subnormals e 2^-24 need no arithmetic at all, but the
//           tensor core aligns products by their exponent fields and drops what
//           falls below: errors of 7e-4 of the values.)
// Measured at 64 x 500 .. 8192 tokens, 32 query heads over 8, rotated, D = 128:
// 303 warp instructions a 16-token tile, set-up and merging included (the
// block cache's kernel: 332), 81 us; the loop itself reads at 5.8 TB/s.
#pragma once

#include "kvq_pages_attn.cuh"

namespace kvq {

constexpr int kUnit = 32;  // tokens of a ring slot: one a lane
constexpr int kRingPages = 2;
// What an item costs a warp besides its units (queries, the state's way out), in units: the kernel ends with
// the warps that have two items.
constexpr int kStepCost = 2;

template <int D>
constexpr int slot_bytes() { return kUnit * (D + 4); }  // K codes, V codes, K scales, V scales

struct StepArgs {
    AttnArgs a;
    int many;  // sequences of more query rows a kv head than this are not this kernel's (0: all are)
    // Prepared queries: fragments [place][head][part][D] and per query the factor of its scores.  A row's place is
    // its number, or, with `many`, its number in its sequence behind a stretch of `stretch` places a sequence.
    __half* frag;
    float* scal;
    int stretch;
    // Short caches and few items: a CTA takes one item whole, its warps equal parts of it, and nothing is left
    // for pages_merge_kernel, which is not launched.
    int whole;
};

// A sequence's share of the work.
struct Item {
    int s, lo, nq, chunks, units, u0, t0, t1;
    int len, base;  // tokens of the sequence; token of row r: base + r
    long long cost;
};

template <int NQ>
__device__ __forceinline__ Item item_of(const StepArgs& g, int s, int H) {
    Item it;
    const int from = g.a.b.start[s], end = g.a.b.start[s + 1], len = max(g.a.b.len[s], 0);
    const int hi = min(end, g.a.rows);
    it.s = s;
    it.lo = max(from, 0);
    it.nq = max(hi - it.lo, 0) * g.a.G;
    it.len = len;
    it.base = len - end;
    it.cost = 0;
    if (it.nq == 0 || (g.many > 0 && it.nq > g.many)) return it;
    const Range r = range_of(g.a, len, end, it.lo, hi);
    it.t0 = r.t0;
    it.t1 = r.t1;
    it.u0 = r.t0 / kUnit;
    it.units = max((r.t1 + kUnit - 1) / kUnit - it.u0, 1);  // rows that see nothing need an owner too
    it.chunks = (it.nq + NQ - 1) / NQ;
    it.cost = (long long)(H * it.chunks) * (it.units + kStepCost);
    return it;
}

// What the ranges are cut from: positions, or items where CTAs take them whole.
template <int NQ>
__device__ __forceinline__ long long share_of(const StepArgs& g, const Item& it, int H) {
    return g.whole && it.cost > 0 ? H * it.chunks : it.cost;
}

// x / y of non-negative numbers; 64-bit division only where 32 do not hold them.
__device__ __forceinline__ long long quotient(long long x, long long y) {
    return (x | y) >> 32 ? x / y : (long long)((uint32_t)x / (uint32_t)y);
}

// A walk over the segments of [x, end) of the work.  An item takes
// kStepCost + units positions, of which the first kStepCost hold no unit.
template <int NQ>
struct Walk {
    long long x, end;  // the current segment begins at x
    Item it;
    int h, c, u, n;    // head, chunk, first unit and units of the segment; n = 0: the end
    int pos, span;     // where in the item the segment begins, and its positions

    __device__ __forceinline__ void cut() {
        span = (int)min((long long)(it.units + kStepCost - pos), end - x);
        u = max(pos - kStepCost, 0);
        n = max(pos + span - kStepCost, 0) - u;
    }
    // x, inside sequence it.s at offset `off` from its first item.
    __device__ __forceinline__ void place(const StepArgs& g, int H, long long off) {
        const int all = it.units + kStepCost;
        const long long k = quotient(off, all), kh = quotient(k, it.chunks);
        pos = (int)(off - k * all);
        c = (int)(k - kh * it.chunks);
        h = (int)kh;
        cut();
        if (n == 0) next(g, H);
    }
    __device__ __forceinline__ void next(const StepArgs& g, int H) {
        do {
            x += span;
            n = 0;
            if (x >= end) return;
            pos = 0;
            if (++c == it.chunks) {
                c = 0;
                if (++h == H) {
                    h = 0;
                    do {
                        if (it.s + 1 >= g.a.b.n_seqs) {
                            end = x;
                            return;
                        }
                        it = item_of<NQ>(g, it.s + 1, H);
                    } while (it.cost == 0);
                }
            }
            cut();
        } while (n == 0);
    }
};

// What a warp leaves of an item whose other parts are elsewhere.
struct Part {
    int lo, nq, h, c, s;  // the item
    int there, begins, ends;
    int ctas;  // where it begins: how many CTAs the item goes over
};

// NW warps; NQ query rows an item.
template <int D, int NQ, bool HAD, int NW>
struct StepSmem {
    static constexpr int kQT = HAD ? NQ / 4 : NQ / 8;   // score tiles of 8 columns
    static constexpr int kNV = HAD ? kQT : 2 * kQT;     // query rows a lane holds scores of
    static constexpr int kNP = (kNV + 1) / 2;           // value tiles of 8 columns
    static constexpr int kStride = D + 4;               // floats of a query's o: lanes of one store in 32 banks
    static constexpr int kMQ = NQ < 8 ? NQ : 8;         // query rows staged at a time
    struct Warp {
        union {
            alignas(128) uint8_t ring[kRingPages][slot_bytes<D>()];
            float last[NQ][kStride];  // o of the range's end, once the ring is done with
        };
        union {
            alignas(16) uint32_t q[kQT][D / 32][32][4];
            float o[kMQ][kStride];
        };
        alignas(16) float4 par[kUnit];  // a token's K scale, log2 and inverse of its V scale
        float m[2][NQ], l[2][NQ];
        Walk<NQ> own, ahead;  // the place in the work: what is computed, what is fetched
        Part part[2];         // of the range's first item and of its last
    };
    Warp warp[NW];
    long long sums[NW], before[NW * 32];
};

__device__ __forceinline__ float max_or_nan(float x, float y) { return x != x || y <= x ? x : y; }

__device__ __forceinline__ float rcp(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// 16 bytes to shared memory: `n` (16 or 0) of them from src, zeros for the rest.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int n) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint32_t perm(uint32_t a, uint32_t b, uint32_t sel) {
    uint32_t r;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
    return r;
}
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}
// D += A B, m16n8k16
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&x)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(b0), "r"(b1));
}

// Query qi's index in the lanes' values: lane t of a quad, value v.
template <bool HAD>
__device__ __forceinline__ int query_of(int v, int t) {
    return HAD ? 4 * v + t : 8 * (v >> 1) + 2 * t + (v & 1);
}

// Tokens that a row of an item sees, the r-th of the sequence's.
__device__ __forceinline__ Range row_range(const AttnArgs& a, const Item& it, int r) {
    const int pos = it.base + it.lo + r;
    Range see = seen_by(a, it.len, pos, pos);
    see.t1 = min(see.t1, it.t1);
    return see;
}

template <int D, int NQ, bool HAD, int NW, int PER_SM>
__global__ void __launch_bounds__(NW * 32, PER_SM) pages_step_kernel(StepArgs g) {
    using S = StepSmem<D, NQ, HAD, NW>;
    constexpr int QT = S::kQT, NV = S::kNV, NP = S::kNP, NJ = D / 16;
    extern __shared__ __align__(128) uint8_t raw[];
    S& sh = *reinterpret_cast<S*>(raw);
    const AttnArgs& a = g.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, t = lane & 3, r8 = lane >> 2;
    const int H = a.p.H;
    typename S::Warp& sm = sh.warp[warp];
    Walk<NQ>&wk = sm.own, &pw = sm.ahead;

    if (lane < 2) sm.part[lane].there = 0;
    grid_dep_launch();
    // pages_queries_kernel let this kernel start once all before it was done; what it writes itself is
    // waited for below

    // ---- the warps' ranges: prefix sums of the sequences' costs, a run of `per` sequences a thread; up to two a
    // lane, every warp by itself
    const bool alone = a.b.n_seqs <= 64;
    const int runs = alone ? 32 : NW * 32, run = alone ? lane : threadIdx.x;
    const int per = (a.b.n_seqs + runs - 1) / runs, s0 = run * per;
    Item mine0;  // of the run's first sequence
    mine0.cost = 0;
    long long mine = 0;
    for (int s = min(s0 + per, a.b.n_seqs) - 1; s >= s0; --s) {
        mine0 = item_of<NQ>(g, s, H);
        mine += share_of<NQ>(g, mine0, H);
    }
    long long sum = mine;
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) {
        const long long o = __shfl_up_sync(~0u, sum, x);
        if (lane >= x) sum += o;
    }
    long long before = sum - mine, total = __shfl_sync(~0u, sum, 31);
    if (!alone) {
        if (lane == 31) sh.sums[warp] = sum;
        __syncthreads();
        total = 0;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            if (w < warp) before += sh.sums[w];
            total += sh.sums[w];
        }
    }
    const int me = blockIdx.x * NW + warp;
    const int workers = g.whole ? (int)min((long long)gridDim.x, total) * NW : (int)min((long long)gridDim.x * NW, total);
    if (!g.whole && threadIdx.x == 0) a.meta[blockIdx.x] = make_int4(0, 0, 0, 0);
    if ((int)blockIdx.x * NW >= workers) {
        grid_dep_wait();  // this grid's end stands for that of the kernels before it
        return;
    }
    const long long share = g.whole ? 1 : quotient(total, workers);  // the first `extra` warps have one unit more
    const int extra = g.whole ? 0 : (int)(total - share * workers);
    const auto begin_of = [&](int worker) { return share * worker + min(worker, extra); };
    if (!alone) {
        sh.before[threadIdx.x] = before;
        __syncthreads();
    }
    {
        Walk<NQ> w;
        w.n = 0;
        if (me < workers) {
            const long long first = g.whole ? blockIdx.x : begin_of(me);
            long long off;
            if (alone) {  // the lane whose run holds the first position (or the item)
                const uint32_t owner = __ballot_sync(~0u, before <= first && first < before + mine);
                const int src = max(__ffs(owner) - 1, 0);
                off = first - __shfl_sync(~0u, before, src);
                constexpr int kWords = sizeof(Item) / 4;
                static_assert(sizeof(Item) % 4 == 0);
                int words[kWords];
                memcpy(words, &mine0, sizeof(Item));
#pragma unroll
                for (int k = 0; k < kWords; ++k) words[k] = __shfl_sync(~0u, words[k], src);
                memcpy(&w.it, words, sizeof(Item));
            } else {
                int lo = 0, hi = NW * 32;
                while (hi - lo > 1) {
                    const int mid = (lo + hi) >> 1;
                    if (sh.before[mid] <= first) lo = mid;
                    else hi = mid;
                }
                off = first - sh.before[lo];
                w.it = item_of<NQ>(g, lo * per, H);
            }
            while (w.it.s + 1 < a.b.n_seqs) {
                const long long of_seq = share_of<NQ>(g, w.it, H);
                if (off < of_seq) break;
                off -= of_seq;
                w.it = item_of<NQ>(g, w.it.s + 1, H);
            }
            if (g.whole) {
                const int part = (w.it.units + NW - 1) / NW;
                w.h = (int)off / w.it.chunks;
                w.c = (int)off - w.h * w.it.chunks;
                w.pos = kStepCost + warp * part;
                w.x = w.pos;
                w.end = min(w.pos + part, kStepCost + w.it.units);
                if (w.x < w.end) w.cut();
            } else {
                w.x = first;
                w.end = begin_of(me + 1);
                w.place(g, H, off);
            }
        }
        if (lane == 0) wk = w;
        if (lane == 1) pw = w;
    }
    __syncwarp();

    // ---- the copies' side of the ring
    int pk = 0, pg0 = -1, pg1 = -1;  // the warp's next unit of the segment; pages of 32 of them, one a lane
    uint32_t held = 0;               // two bits a ring slot: which 16-token halves hold tokens
    const int plog = a.p.page_log2;
    const auto page_of = [&](int tok) {
        if (tok >= pw.it.t1 || tok + 16 <= pw.it.t0) return -1;
        const int col = tok >> plog;  // below max_pages, as t1 is
        const int page = a.b.table[(long long)pw.it.s * a.b.table_stride + col];
        if (page >= 0 && page < a.p.n_pages) return page;
        report_error(kErrRange);
        return -1;
    };
    const auto produce = [&](int slot) {
        if (pk == pw.n && pk > 0) {
            __syncwarp();
            if (lane == 0) pw.next(g, H);
            __syncwarp();
            pk = 0;
        }
        if (pw.n > 0) {
            const int tok = (pw.it.u0 + pw.u + pk) * kUnit;
            if ((pk & 31) == 0) {
                const int at = tok + kUnit * lane;
                pg0 = pk + lane < pw.n ? page_of(at) : -1;
                pg1 = pk + lane < pw.n ? page_of(at + 16) : -1;
            }
            const int p0 = __shfl_sync(~0u, pg0, pk & 31), p1 = __shfl_sync(~0u, pg1, pk & 31);
            ++pk;
            held = (held & ~(3u << (2 * slot))) | ((p0 >= 0 ? 1u : 0u) | (p1 >= 0 ? 2u : 0u)) << (2 * slot);
            constexpr int RB = D / 2, PER = 16 * RB / 512;  // bytes of a token's codes; copies a lane makes of a half
            const uint32_t dst = smem_u32(sm.ring[slot]);
            const int in_page = tok & ((1 << plog) - 1) & ~31;
            // first token of the halves; a half that is not there is filled with zeros
            const long long at0 = (((long long)max(p0, 0) * H + pw.h) << plog) + in_page;
            const long long at1 = (((long long)max(p1, 0) * H + pw.h) << plog) + in_page + (plog > 4 ? 16 : 0);
            const int n0 = p0 >= 0 ? 16 : 0, n1 = p1 >= 0 ? 16 : 0;
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int k = 0; k < PER; ++k) {
                    const int byte = lane * 16 + k * 512;
                    copy16(dst + i * kUnit * RB + byte, a.p.codes[i] + at0 * RB + byte, n0);
                    copy16(dst + i * kUnit * RB + 16 * RB + byte, a.p.codes[i] + at1 * RB + byte, n1);
                }
            if (lane < 8) {  // 64 bytes of scales a tensor: lanes 0 .. 3 (K) and 4 .. 7 (V)
                const __half* src = (lane & 4 ? a.p.tok[1] : a.p.tok[0]) + (lane & 2 ? at1 : at0) + (lane & 1) * 8;
                copy16(dst + kUnit * D + lane * 16, src, lane & 2 ? n1 : n0);
            }
        }
        copies_commit();
    };
    grid_dep_wait();
    bool primed = false;

    int slot = 0;

    // ---- segments
    while (wk.n > 0) {
        const bool begins = wk.u == 0, ends = wk.u + wk.n == wk.it.units;
        const int units = wk.n, unit0 = wk.it.u0 + wk.u, seen0 = wk.it.t0, seen1 = wk.it.t1;
        const bool final = wk.x + wk.span >= wk.end;  // the range's last segment
        float M[NV], l[NV], cq[NV];
        float o[NP][NJ][4];
        const int i0 = wk.c * NQ, lo = wk.it.lo, nq = wk.it.nq;
        // index of query i of the item among the prepared ones
        const int query0 = (g.many > 0 ? wk.it.s * g.stretch : lo) * a.Hq + wk.h * a.G;
        const auto prepared = [&](int i, int r) { return query0 + r * a.Hq + i - r * a.G; };
        constexpr bool kHold = QT * (D / 32) <= 4;  // few enough fragments to stay in registers
        uint4 qf[QT][D / 32];
#pragma unroll
        for (int n = 0; n < QT; ++n) {  // column r8 of tile n
            const int i = i0 + (HAD ? 4 * n + (r8 >> 1) : 8 * n + r8);
#pragma unroll
            for (int k = 0; k < D / 32; ++k) qf[n][k] = make_uint4(0, 0, 0, 0);
            if (i < nq) {
                const long long at = prepared(i, i / a.G);
                const uint4* src = reinterpret_cast<const uint4*>(g.frag + (HAD ? 2 * at + (r8 & 1) : at) * D) + t;
#pragma unroll
                for (int k = 0; k < D / 32; ++k) qf[n][k] = src[4 * k];
            }
        }
        if (!primed) {  // (behind the loads of the first queries)
            primed = true;
            for (int i = 0; i < kRingPages; ++i) produce(i);
        }
        int lo_max = 0, hi_min = 0x7FFFFFFF;  // tokens that all of the chunk's rows see
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            M[v] = kLowest;
            l[v] = 0.0f;
            const int i = i0 + query_of<HAD>(v, t);
            cq[v] = 0.0f;
            if (i < nq) {
                const int r = i / a.G;
                cq[v] = g.scal[prepared(i, r)];
                const Range see = row_range(a, wk.it, r);
                lo_max = max(lo_max, see.t0);
                hi_min = min(hi_min, see.t1);
            }
        }
        lo_max = __reduce_max_sync(~0u, lo_max);
        hi_min = __reduce_min_sync(~0u, hi_min);
#pragma unroll
        for (int n = 0; n < NP; ++n)
#pragma unroll
            for (int j = 0; j < NJ; ++j)
#pragma unroll
                for (int k = 0; k < 4; ++k) o[n][j][k] = 0.0f;
        if constexpr (!kHold) {
#pragma unroll
            for (int n = 0; n < QT; ++n)
#pragma unroll
                for (int k = 0; k < D / 32; ++k) *reinterpret_cast<uint4*>(sm.q[n][k][lane]) = qf[n][k];
            __syncwarp();
        }

        for (int off = 0; off < units; ++off) {
            const int tok0 = (unit0 + off) * kUnit;
            copies_wait<kRingPages - 1>();
            __syncwarp();
            const uint8_t* ring = sm.ring[slot];
            {   // one token a lane: scales of K, log2 and inverse of V's
                const __half* sc = reinterpret_cast<const __half*>(ring + kUnit * D);
                const float sk = __half2float(sc[lane]), sv = fmaxf(__half2float(sc[kUnit + lane]), 0x1p-24f);
                const bool there = (held >> (2 * slot + (lane >> 4)) & 1) && tok0 + lane < seen1 && tok0 + lane >= seen0;
                sm.par[lane] = there ? make_float4(sk, lg2(sv), rcp(sv), 0.0f)
                                           : make_float4(0.0f, -INFINITY, 0.0f, 0.0f);
            }
            __syncwarp();
            float y[2][NV][2];  // [tile][value][token r8 or r8 + 8]
            float4 par[2][2];
#pragma unroll
            for (int mt = 0; mt < 2; ++mt) {
                uint32_t kw[2][D / 32];
#pragma unroll
                for (int hf = 0; hf < 2; ++hf)
                    load_words(ring + (mt * 16 + hf * 8 + r8) * (D / 2) + t * (D / 8), kw[hf]);
                float s[QT][4];
#pragma unroll
                for (int n = 0; n < QT; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.0f;
#pragma unroll
                for (int i = 0; i < D / 32; ++i) {
                    uint32_t x[2][4];
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        const uint32_t w = kw[hf][i], w8 = w >> 8;
                        x[0][hf] = codes_low(w);
                        x[1][hf] = codes_upper(w);
                        x[0][2 + hf] = codes_low(w8);
                        x[1][2 + hf] = codes_upper(w8);
                    }
#pragma unroll
                    for (int n = 0; n < QT; ++n) {
                        const uint4 f = kHold ? qf[n][i]
                                              : *reinterpret_cast<const uint4*>(sm.q[n][i][lane]);
                        mma(s[n], x[0], f.x, f.y);
                        mma(s[n], x[1], f.z, f.w);
                    }
                }
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    par[mt][hf] = sm.par[mt * 16 + hf * 8 + r8];
#pragma unroll
                    for (int v = 0; v < NV; ++v) {
                        const float score = HAD ? s[v][2 * hf] + s[v][2 * hf + 1] : s[v >> 1][2 * hf + (v & 1)];
                        y[mt][v][hf] = __fmaf_rn(score, cq[v] * par[mt][hf].x, par[mt][hf].y);
                    }
                }
            }
            if (tok0 < lo_max || tok0 + kUnit > hi_min) {
#pragma unroll
                for (int v = 0; v < NV; ++v) {
                    const int i = i0 + query_of<HAD>(v, t);
                    const Range see = i < nq ? row_range(a, wk.it, i / a.G) : Range{0, 0};
#pragma unroll
                    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf) {
                            const int tok = tok0 + mt * 16 + hf * 8 + r8;
                            if (tok < see.t0 || tok >= see.t1) y[mt][v][hf] = -INFINITY;
                        }
                }
            }
            float top[NV];
            bool more = false;
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                top[v] = fmaxf(fmaxf(y[0][v][0], y[0][v][1]), fmaxf(y[1][v][0], y[1][v][1]));
                more |= top[v] > M[v];
            }
            if (__any_sync(~0u, more)) {
#pragma unroll
                for (int v = 0; v < NV; ++v) {
#pragma unroll
                    for (int x = 4; x < 32; x <<= 1) top[v] = fmaxf(top[v], __shfl_xor_sync(~0u, top[v], x));
                    const float m2 = fmaxf(M[v], top[v]), f = ex2(M[v] - m2);
                    M[v] = m2;
                    l[v] *= f;
#pragma unroll
                    for (int j = 0; j < NJ; ++j) {
                        o[v >> 1][j][v & 1] *= f;
                        o[v >> 1][j][2 + (v & 1)] *= f;
                    }
                }
            }
#pragma unroll
            for (int mt = 0; mt < 2; ++mt) {
                uint32_t bw[NP][2];
#pragma unroll
                for (int hf = 0; hf < 2; ++hf)
#pragma unroll
                    for (int n = 0; n < NP; ++n) {
                        float w[2] = {0.0f, 0.0f};
#pragma unroll
                        for (int k = 0; k < 2 && 2 * n + k < NV; ++k) {
                            w[k] = ex2(y[mt][2 * n + k][hf] - (M[2 * n + k] - kBias));
                            l[2 * n + k] = __fmaf_rn(w[k], par[mt][hf].z, l[2 * n + k]);
                        }
                        bw[n][hf] = transposed(Elem<__half>::pack(w[0], w[1]));
                    }
                // tokens 2t, 2t + 1 and 2t + 8, 2t + 9; words of channels r8 (and, at D = 128, its neighbour's)
                constexpr int NWD = D / 64;
                uint32_t vw[2][2][NWD];
#pragma unroll
                for (int hf = 0; hf < 2; ++hf)
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        load_words(ring + kUnit * (D / 2) + (mt * 16 + hf * 8 + 2 * t + k) * (D / 2) + r8 * (D / 16),
                                   vw[hf][k]);
#pragma unroll
                for (int j0 = 0; j0 < NJ; j0 += 4) {  // four tiles: nibbles 0 .. 3 or 4 .. 7 of the words
                    uint32_t z[4][4];
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf)
#pragma unroll
                        for (int k = 0; k < 2; ++k) {  // row r8, or r8 + 8: the other word, or half of the word
                            const int wd = D == 128 ? k : 0;
                            const bool up = D == 128 ? j0 != 0 : k != 0;
                            const uint32_t p = perm(vw[hf][0][wd], vw[hf][1][wd], up ? 0x7632u : 0x5410u), p8 = p >> 8;
                            z[0][2 * hf + k] = codes_low(p);
                            z[1][2 * hf + k] = codes_upper(p);
                            z[2][2 * hf + k] = codes_low(p8);
                            z[3][2 * hf + k] = codes_upper(p8);
                        }
#pragma unroll
                    for (int n = 0; n < NP; ++n)
#pragma unroll
                        for (int j = 0; j < 4; ++j) mma(o[n][j0 + j], z[j], bw[n][0], bw[n][1]);
                }
            }
            __syncwarp();  // the slot has been read
            produce(slot);
            if (++slot == kRingPages) slot = 0;
        }

        // ---- the segment's state: finished, or left for the merge
        const bool whole = begins && ends;
        const int which = final || whole ? 1 : 0;  // (0 is kept for the range's first item)
#pragma unroll
        for (int v = 0; v < NV; ++v) {
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) l[v] += __shfl_xor_sync(~0u, l[v], x);
            if (r8 == 0) {
                sm.m[which][query_of<HAD>(v, t)] = M[v];
                sm.l[which][query_of<HAD>(v, t)] = l[v];
            }
        }
        if (!whole && lane == 0) {
            int ctas = 1;
            if (begins) {
                const long long last = wk.x - wk.pos + wk.it.units + kStepCost - 1, longer = (share + 1) * extra;
                const int worker = (int)(last < longer ? quotient(last, share + 1) : extra + quotient(last - longer, share));
                ctas = worker / NW - (int)blockIdx.x + 1;
            }
            sm.part[which] = Part{wk.it.lo, wk.it.nq, wk.h, wk.c, wk.it.s, 1, begins, ends, ctas};
        }
        const int queries = min(NQ, wk.it.nq - wk.c * NQ);
        float* left = a.left + (long long)me * NQ * D;
#pragma unroll
        for (int n = 0; n < NP; ++n) {
            __syncwarp();
#pragma unroll
            for (int k = 0; k < 2 && 2 * n + k < NV; ++k) {
                const int q = query_of<HAD>(2 * n + k, t);
                float* dst = final && !whole ? sm.last[q] : sm.o[q - 8 * n];
#pragma unroll
                for (int j = 0; j < NJ; ++j)
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf)
                        dst[(2 * j + hf) * 8 + r8] = o[n][j][2 * hf + k];
            }
            __syncwarp();
            if (whole || !final) {
#pragma unroll 1
                for (int q = 8 * n; q < min(8 * n + S::kMQ, queries); ++q) {
                    float v[D / 32];
#pragma unroll
                    for (int k = 0; k < D / 32; ++k) v[k] = sm.o[q - 8 * n][lane + 32 * k];
                    if (whole) {
                        const int i = wk.c * NQ + q, r = i / a.G;
                        finish_row<D, HAD>(a, wk.it.lo + r, wk.h * a.G + i - r * a.G, v, sm.m[which][q],
                                           sm.l[which][q]);
                    } else {
#pragma unroll
                        for (int k = 0; k < D / 32; ++k) left[q * D + lane + 32 * k] = v[k];
                    }
                }
            }
        }
        __syncwarp();
        if (lane == 0) wk.next(g, H);
        __syncwarp();
    }

    // ---- items whose parts lie at the ends of the warps' ranges: part 2 warp + which, in order
    __syncthreads();
    const Part& mine_p = sh.warp[min(lane >> 1, NW - 1)].part[lane & 1];
    const bool there = lane < 2 * NW && mine_p.there;
    const uint32_t all = __ballot_sync(~0u, there), closed = __ballot_sync(~0u, there && mine_p.ends);
    int ch = 0;
    for (uint32_t rest = all; rest;) {
        // the first part's item goes on to the first part that ends it
        const uint32_t close = closed & rest;
        const uint32_t set = close ? rest & ((close & (0u - close)) * 2 - 1) : rest;
        const int p0 = __ffs(set) - 1;
        const bool ends = close != 0;
        rest &= ~set;
        const Part& x = sh.warp[p0 >> 1].part[p0 & 1];
        const int queries = min(NQ, x.nq - x.c * NQ);
        for (int q = (warp + NW - ch++ % NW) % NW; q < queries; q += NW) {  // (items begin with different warps)
            const bool in = set >> lane & 1;
            const float m = in ? sh.warp[lane >> 1].m[lane & 1][q] : kLowest;
            float top = m;
#pragma unroll
            for (int k = 16; k; k >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, k));
            const float f = ex2(m - top);
            float sum_l = in ? sh.warp[lane >> 1].l[lane & 1][q] * f : 0.0f;
#pragma unroll
            for (int k = 16; k; k >>= 1) sum_l += __shfl_xor_sync(~0u, sum_l, k);
            float v[D / 32] = {};
            for (uint32_t parts = set; parts; parts &= parts - 1) {
                const int p = __ffs(parts) - 1;
                const float fp = __shfl_sync(~0u, f, p);
                const float* src = p & 1 ? sh.warp[p >> 1].last[q]
                                         : a.left + ((long long)(blockIdx.x * NW + (p >> 1)) * NQ + q) * D;
#pragma unroll
                for (int c = 0; c < D / 32; ++c) v[c] = __fmaf_rn(src[lane + 32 * c], fp, v[c]);
            }
            if (x.begins && ends) {
                const int i = x.c * NQ + q, r = i / a.G;
                finish_row<D, HAD>(a, x.lo + r, x.h * a.G + i - r * a.G, v, top, sum_l);
                continue;
            }
            const long long at = (2ll * blockIdx.x + (x.begins ? 1 : 0)) * NQ + q;
            if (lane == 0) reinterpret_cast<float2*>(a.ml)[at] = make_float2(top, sum_l);
#pragma unroll
            for (int c = 0; c < D / 32; ++c) a.part[at * D + lane + 32 * c] = v[c];
            if (x.begins && q == 0 && lane == 0) a.meta[blockIdx.x] = make_int4(x.s, x.h, x.c * NQ, x.ctas);
        }
    }
}

}  // namespace kvq
