// kvq_pages_tile.cuh -- attention of many query rows a kv head (prompts, parts
// of prompts): tcgen05 products on tiles of 256 rows and 64 tokens.
//
// Rows: row r and query head j of a kv head's group are tile row r G + j, so
// that a kv head's codes are unpacked once for all its heads.  An item is
// (sequence, 256 such rows, kv head); its cost is the number of 64-token
// tiles that its rows see.  pages_plan lays all items end to end and cuts them
// into one range a CTA; parts of items at the ends are merged by
// pages_merge_kernel.
//
// A CTA (one an SM):
//   warps 0 .. 3, 4 .. 7   softmax of the lower and the upper 128 rows, one row a
//                          thread; they also bring in the queries and finish rows
//   warps 8 .. 13          codes from global memory to the fp16 tiles of K and V,
//                          32 tokens at a time in turn; scales
//   warps 14, 15           issue the products of a half each
// Products a step of 64 tokens, rows X: S_X = Q_X K^T (for rotated queries
// twice, the high and the low fp16 part: 22 bits of the query are kept), then
// O_X += W_X V with W_X, fp16, taken from tensor memory, where it lies over
// S_X.  Each half has two S, so that the scores of the next step are there
// when a softmax ends one; with one S of 128 tokens a half, which the tensor
// core fills faster, softmax and products waited for each other in turn (9000
// cycles for 128 tokens).  Tiles of K and V go through a ring of six buffers.
// With the reference R of a row (its largest score + the largest exponent of the
// V scales that it sees of a tile, over the tiles so far, up to 2^kSlack), p = 2^(x - R + kTileBias),
//   W = fp16(p sigma_V),  O = sum W q,  l = sum p,
// so W is the only rounding here too, and stays in fp16's range; what is below
// its normal range is kept to 2^-31 of the largest V scale.  (V tiles of
// sigma q, rounded, with W = p, need no scale in the softmax threads: the same
// time, but 3.0e-4 of the values instead of 2.3e-4.)  The scales are read in
// fp16: a number that all lanes read from shared memory takes it as long as 32
// different ones, and three fp32 numbers a token took as long as the products.
// O stays in tensor memory; a row whose maximum rose by more than 2^kSlack
// scales it there, once the step before is in it.
// Measured (8192 rows and tokens, 32 query heads over 8, rotated, D = 128):
// 1000 us, 550 TFLOP/s of 4 D a (row, token, head); the products and their
// reads of shared memory (a 64-token product of 128 rows reads 6 KB in the 32
// cycles that it computes) are busy 60% of it, the exponentials a third.
#pragma once

#include "kvq_pages_attn.cuh"
#include "kvq_pages_step.cuh"

namespace kvq {

constexpr int kRowsM = 128, kItemRows = 256, kTileTokens = 64;
// What an item costs besides its tiles (queries in, rows out), in tiles: with 0, the CTA of a prompt's first
// rows, whose items are short, took twice the time of the others.
constexpr int kItemCost = 8;
constexpr int kTileThreads = 512;
constexpr int kRingTiles = 6, kParStages = 4;
constexpr int kUnitTokens = 32, kUnits = kTileTokens / kUnitTokens;  // units of a tile
constexpr float kSlack = 8.0f;               // how far a row's maximum may pass its reference
constexpr float kTileBias = 6.0f;            // W < 2^(kSlack + kTileBias + 1), in fp16's range
constexpr uint32_t kTileWait = 1u << 22;  // polls, of a second at most together
// Registers a thread; the launch gives 128.
constexpr int kLaunchRegs = 128, kSoftmaxRegs = 160, kProducerRegs = 96;
static_assert(256 * (kSoftmaxRegs + kProducerRegs) <= kTileThreads * kLaunchRegs);
constexpr int kProducers = 6;

struct TileArgs {
    AttnArgs a;
    int many;             // sequences of more query rows a kv head than this are this kernel's
    int4* plan;           // [CTA]: sequence, chunk, head, first tile
    long long* seq_cost;  // [sequence] tiles, then the total
};

// One item's place among the tokens and rows.
struct TileItem {
    int s, lo, nq, len, base;  // the sequence: first row, query rows a kv head, tokens, token of row 0
    int chunks, c, h;
    int u0, units;  // tiles that the item's rows see
    int t0, t1;
};

__device__ __forceinline__ bool tile_seq(const TileArgs& g, int s, TileItem& it) {
    const int end = g.a.b.start[s + 1], lo = max(g.a.b.start[s], 0), hi = min(end, g.a.rows);
    it.s = s;
    it.lo = lo;
    it.nq = max(hi - lo, 0) * g.a.G;
    it.chunks = 0;
    if (it.nq <= g.many) return false;
    const int len = max(g.a.b.len[s], 0);
    it.len = len;
    it.base = len - end;
    it.chunks = (it.nq + kItemRows - 1) / kItemRows;
    return true;
}
__device__ __forceinline__ void tile_chunk(const TileArgs& g, TileItem& it, int c) {
    it.c = c;
    const int r0 = c * kItemRows / g.a.G, r1 = (min((c + 1) * kItemRows, it.nq) - 1) / g.a.G + 1;
    const Range r = range_of(g.a, it.len, it.len - it.base, it.lo + r0, it.lo + r1);
    it.t0 = r.t0;
    it.t1 = r.t1;
    it.u0 = r.t0 / kTileTokens;
    it.units = max((r.t1 + kTileTokens - 1) / kTileTokens - it.u0, 1);
}

// The first position of range b when `total` positions are cut into `ctas` ranges.
struct Cut {
    long long share, extra;
    __device__ __forceinline__ Cut(long long total, int ctas) {
        share = quotient(total, ctas);
        extra = total - share * ctas;
    }
    __device__ __forceinline__ long long begin(long long b) const { return share * b + min(b, extra); }
    // the range that position x lies in
    __device__ __forceinline__ long long of(long long x) const {
        const long long longer = (share + 1) * extra;
        return x < longer ? quotient(x, share + 1) : extra + quotient(x - longer, share);
    }
};

// The ranges of the tile kernel's CTAs, by one block of 256 threads: a warp
// a sequence sums its items' costs; then, with the sequences' running sums,
// every chunk of rows writes the plans of the ranges that begin in its items.
__device__ __forceinline__ void pages_plan(const TileArgs& g, int ctas_max) {
    __shared__ long long sums[8];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, H = g.a.p.H, n_seqs = g.a.b.n_seqs;
    TileItem it;
    for (int s = warp; s < n_seqs; s += 8) {
        long long cost = 0;
        if (tile_seq(g, s, it))
            for (int c = lane; c < it.chunks; c += 32) {
                tile_chunk(g, it, c);
                cost += it.units + kItemCost;
            }
#pragma unroll
        for (int x = 16; x; x >>= 1) cost += __shfl_xor_sync(~0u, cost, x);
        if (lane == 0) g.seq_cost[s] = cost * H;
    }
    __syncthreads();
    const int per = (n_seqs + 255) / 256, s0 = threadIdx.x * per, s1 = min(s0 + per, n_seqs);
    long long mine = 0;
    for (int s = s0; s < s1; ++s) mine += g.seq_cost[s];
    long long sum = mine;
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) {
        const long long o = __shfl_up_sync(~0u, sum, x);
        if (lane >= x) sum += o;
    }
    if (lane == 31) sums[warp] = sum;
    __syncthreads();
    long long before = sum - mine, total = 0;
    for (int w = 0; w < 8; ++w) {
        if (w < warp) before += sums[w];
        total += sums[w];
    }
    for (int s = s0; s < s1; ++s) {  // costs to running sums
        const long long cost = g.seq_cost[s];
        g.seq_cost[s] = before;
        before += cost;
    }
    if (threadIdx.x == 0) g.seq_cost[n_seqs] = total;
    __syncthreads();
    if (total == 0) return;
    const int ctas = (int)min((long long)ctas_max, total);
    const Cut cut(total, ctas);
    for (int s = warp; s < n_seqs; s += 8) {
        if (!tile_seq(g, s, it)) continue;
        long long at = g.seq_cost[s];
        for (int c0 = 0; c0 < it.chunks; c0 += 32) {
            long long cost = 0;
            if (c0 + lane < it.chunks) {
                tile_chunk(g, it, c0 + lane);
                cost = (long long)(it.units + kItemCost) * H;
            }
            long long upto = cost;
#pragma unroll
            for (int x = 1; x < 32; x <<= 1) {
                const long long o = __shfl_up_sync(~0u, upto, x);
                if (lane >= x) upto += o;
            }
            const long long lo = at + upto - cost, hi = at + upto;
            if (cost > 0) {
                long long b = cut.of(lo);
                if (cut.begin(b) < lo) ++b;
                for (; b < ctas && cut.begin(b) < hi; ++b) {
                    const long long in = cut.begin(b) - lo, h = quotient(in, it.units + kItemCost);
                    g.plan[b] = make_int4(s, c0 + lane, (int)h, (int)(in - h * (it.units + kItemCost)));
                }
            }
            at += __shfl_sync(~0u, upto, 31);
        }
    }
}

// Loads, rotates, scales and splits the queries: a warp each, D / 32
// neighbouring channels a lane.  Where the tile kernel runs too, the last block
// plans it.
constexpr int kQueryWarps = 8;

template <int D, bool HAD>
__global__ void __launch_bounds__(kQueryWarps * 32) pages_queries_kernel(StepArgs g, TileArgs tiles, int plan_ctas) {
    constexpr int N = D / 32, C = D / 4;  // channels a lane; channels a fragment lane
    const AttnArgs& a = g.a;
    const int lane = threadIdx.x & 31;
    const long long at = (long long)blockIdx.x * kQueryWarps + (threadIdx.x >> 5);
    const long long place = at / a.Hq;
    const int head = (int)(at - place * a.Hq);
    grid_dep_wait();
    grid_dep_launch();
    if (plan_ctas > 0 && blockIdx.x == gridDim.x - 1) {  // the last block cuts the tile kernel's work
        pages_plan(tiles, plan_ctas);
        return;
    }
    long long row = place;
    if (g.many > 0) {
        const int s = (int)(place / g.stretch);
        if (s >= a.b.n_seqs) return;
        const int lo = max(a.b.start[s], 0), hi = min(a.b.start[s + 1], a.rows);
        row = lo + (place - (long long)s * g.stretch);
        if (row >= hi || (long long)(hi - lo) * a.G > g.many) return;
    }
    if (row >= a.rows) return;
    const uint16_t* src = static_cast<const uint16_t*>(a.q) + row * a.q_row + head * a.q_head + lane * N;
    uint32_t u[N / 2];
    load_words(reinterpret_cast<const uint8_t*>(src), u);
    float v[N];
#pragma unroll
    for (int k = 0; k < N / 2; ++k) {
        const float2 f = a.bf16 ? Elem<__nv_bfloat16>::wide(u[k]) : Elem<__half>::wide(u[k]);
        v[2 * k] = f.x, v[2 * k + 1] = f.y;
    }
    if constexpr (HAD) {
        if (a.signs) {
            if constexpr (N == 4) {
                const char4 x = reinterpret_cast<const char4*>(a.signs)[lane];
                v[0] *= x.x, v[1] *= x.y, v[2] *= x.z, v[3] *= x.w;
            } else {
                const char2 x = reinterpret_cast<const char2*>(a.signs)[lane];
                v[0] *= x.x, v[1] *= x.y;
            }
        }
        lane_stages<1, N>(v);
#pragma unroll
        for (int x = 1; x < 32; x <<= 1) {
            const float flip = (lane & x) ? -1.0f : 1.0f;
#pragma unroll
            for (int k = 0; k < N; ++k) v[k] = __fmaf_rn(v[k], flip, __shfl_xor_sync(~0u, v[k], x));
        }
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] *= a.rsqd;
    }
    float m = 0.0f;
#pragma unroll
    for (int k = 0; k < N; ++k) m = max_or_nan(m, fabsf(v[k]));
#pragma unroll
    for (int x = 16; x; x >>= 1) m = max_or_nan(m, __shfl_xor_sync(~0u, m, x));
    const float f = m > 0.0f || m != m ? query_scale(m) : 1.0f;
    __half* dst = g.frag + at * (HAD ? 2 : 1) * D;
#pragma unroll
    for (int k = 0; k < N; ++k) {
        // fragment lane t holds channels C t .. ; of eight of them, channel c8 is half c8 / 4 of word
        // (tile's nibble parity, register)
        const int ch = lane * N + k, t = ch / C, i8 = (ch % C) >> 3, c8 = ch & 7;
        const int place8 = (i8 * 4 + t) * 8 + ((c8 & 1) * 2 + ((c8 >> 1) & 1)) * 2 + (c8 >> 2);
        const float x = v[k] * f;
        const __half hi = __float2half_rn(x);
        dst[place8] = hi;
        if constexpr (HAD) dst[D + place8] = __float2half_rn(x - __half2float(hi));
    }
    if (lane == 0) g.scal[at] = a.scale2 / f;
}

// A walk over a CTA's segments; every warp has its own.  An item takes
// kItemCost + units positions, of which the first kItemCost hold no tile.
struct TileWalk {
    TileItem it;
    int u, n;        // first tile (of the item's) and tiles of the segment; n = 0: the end
    long long left;  // positions of the range from the segment's first on
    int from, span;  // where in the item they begin, and how many are the segment's

    __device__ __forceinline__ void cut_at(const TileArgs& g, int position) {
        from = position;
        while (true) {
            const int all = it.units + kItemCost;
            span = (int)min((long long)(all - from), left);
            u = max(from - kItemCost, 0);
            n = max(from + span - kItemCost, 0) - u;
            if (n > 0) return;
            left -= span;
            if (left <= 0) return;
            step(g);
            if (left <= 0) return;
            from = 0;
        }
    }
    __device__ __forceinline__ void step(const TileArgs& g) {  // to the next item
        if (++it.h < g.a.p.H) return;
        it.h = 0;
        if (it.c + 1 < it.chunks) {
            tile_chunk(g, it, it.c + 1);
            return;
        }
        int s = it.s + 1;
        while (s < g.a.b.n_seqs && !tile_seq(g, s, it)) ++s;
        if (s >= g.a.b.n_seqs) left = 0, n = 0;
        else tile_chunk(g, it, 0);
    }
    __device__ __forceinline__ void begin(const TileArgs& g, int b, const Cut& cut) {
        const int4 p = g.plan[b];
        left = cut.begin(b + 1) - cut.begin(b);
        tile_seq(g, p.x, it);
        tile_chunk(g, it, p.y);
        it.h = p.z;
        cut_at(g, p.w);
    }
    __device__ __forceinline__ void next(const TileArgs& g) {
        left -= span;
        n = 0;
        if (left <= 0) return;
        step(g);
        if (left > 0) cut_at(g, 0);
    }
};

template <int D, bool HAD>
struct TileSmem {
    static constexpr int kTile = kTileTokens * D * 2;  // bytes of a K or V tile
    static constexpr int kQuery = kRowsM * D * 2;      // of a part of a half's queries
    alignas(1024) uint8_t q[2][HAD ? 2 : 1][kQuery];   // [half][high, low][64 channels][row]
    alignas(1024) uint8_t ring[kRingTiles][kTile];
    alignas(16) __half par[kParStages][2][kTileTokens];  // K and V scales
    alignas(8) int expo[kParStages][kUnits];           // largest exponent of a unit's V scales
    alignas(8) uint32_t absent[kParStages][kUnits];    // tokens of the tile that are not there, a bit each
    alignas(16) uint32_t signs[D / 2];                 // sign bits of two channels' signs
    uint64_t full[kRingTiles], empty[kRingTiles];
    uint64_t par_full[kParStages], par_empty[kParStages];
    uint64_t q_full[2], s_full[2][2], w_full[2][2], o_full[2][2];  // [half], [half][tile's parity]
    uint64_t drained[2];
    uint32_t tmem;
    TileWalk walk[kTileThreads / 32];                  // each warp's place in the work
};

// ---------------------------------------------------------------- tcgen05

__device__ __forceinline__ void mbar_arrive(uint64_t* bar, uint32_t n = 1) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(n) : "memory");
}
// mbar_wait that also gives up once a second has passed (a poll's suspension is the hardware's choice).
__device__ __forceinline__ bool mbar_wait_1s(uint64_t* bar, uint32_t parity, uint32_t max_iter) {
    uint64_t t0 = 0, t;
    for (uint32_t left = max_iter; left > 0;) {
        const uint32_t n = min(left, 64u);
        if (mbar_wait(bar, parity, n)) return true;
        left -= n;
        asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
        if (t0 == 0) t0 = t;
        else if (t - t0 > 1000000000ull) break;
    }
    return false;
}
// The tensor core's arrival once all products issued so far are done.
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}
__device__ __forceinline__ void tc_before_sync() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after_sync() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// One lane of a warp that is together.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
    return p != 0;
}

// Shared-memory descriptor of a 128-byte-swizzled operand.  K-major (queries,
// K): 8-row groups 1024 bytes apart (stride offset); the other offset is not
// used.  MN-major (V, channels contiguous): 8-token groups 1024 bytes apart,
// the next 64 channels kTile / (D / 64) on (leading offset).
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t leading) {
    return (uint64_t)((addr & 0x3FFFF) >> 4) | (uint64_t)(leading >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 |
           (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
// fp16 operands, fp32 sums, M = 128.
__host__ __device__ constexpr uint32_t mma_desc(int n, bool b_mn_major) {
    return 1u << 4 | (b_mn_major ? 1u << 16 : 0u) | (uint32_t)(n >> 3) << 17 | (uint32_t)(kRowsM >> 4) << 24;
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t desc, bool add) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
        "l"(a), "l"(b), "r"(desc), "r"((uint32_t)add)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t desc, bool add) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
        "r"(a), "l"(b), "r"(desc), "r"((uint32_t)add)
        : "memory");
}

// 32 columns of the thread's row.
__device__ __forceinline__ void tmem_load32(uint32_t (&r)[32], uint32_t at) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
        "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(at)
        : "memory");
}
__device__ __forceinline__ void tmem_store32(uint32_t at, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
        "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(at),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void tmem_wait_load() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_store() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Four 16-byte pieces of a 128-byte-swizzled tile from 32 codes of one token:
// channels 32 quarter .. + 31 of row `row`.  Of eight channels the halves are
// in the order 0 4 1 5 2 6 3 7, as the queries' and O's are.  Lanes of the
// second 64 channels take their pieces in another order: the same places of
// the two 64-channel halves lie in the same banks.
__device__ __forceinline__ void store_codes(uint8_t* tile, int row, int quarter, const uint4& w) {
    const bool upper = quarter & 2;
    const uint32_t words[4] = {upper ? w.y : w.x, upper ? w.x : w.y, upper ? w.w : w.z, upper ? w.z : w.w};
    uint8_t* base = tile + (upper ? kTileTokens * 128 : 0) + row * 128;
    const int swizzle = (quarter & 1) * 4 ^ (upper ? 1 : 0) ^ (row & 7);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint32_t x = words[k], x8 = x >> 8;
        *reinterpret_cast<uint4*>(base + (k ^ swizzle) * 16) =
            make_uint4(codes_low(x), codes_upper(x), codes_low(x8), codes_upper(x8));
    }
}
// Order of eight channels in a 16-byte piece: place p holds channel place8(p).
__host__ __device__ constexpr int place8(int p) { return (p >> 1) + 4 * (p & 1); }

// 32 tokens of a tile of K or V, by one warp: codes into registers, and from
// there, as fp16, into the tile; with K's also the scales of both.  K and V
// share the code: the instruction cache holds the loops of all roles, and
// hardly more.
template <int D>
struct Unit {
    static constexpr int kPieces = D / 32, kLoads = kPieces;  // 16-byte pieces of a token; loads of a lane
    uint4 w[kLoads];
    __half scale[2];  // K's and V's of the token that is this lane's
    bool absent;      // which is not there

    // pg: the pages of the two halves as the table has them.
    __device__ __forceinline__ void fetch(const TileArgs& g, int h, int t0, int t1, int tok, int is_v, int pg0, int pg1) {
        const Pool& p = g.a.p;
        const int lane = threadIdx.x & 31;
        absent = tok + lane < t0 || tok + lane >= t1;
        scale[0] = scale[1] = __ushort_as_half(0);
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            const int t = tok + 16 * hf, pg = hf ? pg1 : pg0;
            const bool needed = t + 16 > t0 && t < t1, there = needed && pg >= 0 && pg < p.n_pages;
#pragma unroll
            for (int k = 0; k < kLoads / 2; ++k)
                w[hf * (kLoads / 2) + k] = make_uint4(0x88888888u, 0x88888888u, 0x88888888u, 0x88888888u);  // zeros
            if (there) {  // the 16 tokens lie in a row, and all may be read
                const uint32_t at = (uint32_t)((pg * p.H + h) << p.page_log2) + (t & ((1 << p.page_log2) - 1));
                const uint4* src = reinterpret_cast<const uint4*>(p.codes[is_v]) + at * (uint64_t)kPieces + lane;
#pragma unroll
                for (int k = 0; k < kLoads / 2; ++k) w[hf * (kLoads / 2) + k] = src[32 * k];
                if (!is_v && (lane >> 4) == hf && !absent)
                    scale[0] = p.tok[0][at + (lane & 15)], scale[1] = p.tok[1][at + (lane & 15)];
            } else {
                absent |= (lane >> 4) == hf;
                if (needed) report_error(kErrRange);
            }
        }
    }
    __device__ __forceinline__ void store(uint8_t* tile, int first_row) const {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int k = 0; k < kLoads; ++k)
            store_codes(tile, first_row + k * (32 / kPieces) + lane / kPieces, lane % kPieces, w[k]);
    }
};

template <int D, bool HAD>
__global__ void __launch_bounds__(kTileThreads, 1) pages_tile_kernel(TileArgs g) {
    using S = TileSmem<D, HAD>;
    constexpr int kTile = S::kTile, kSlab = kTileTokens * 128, kQSlab = kRowsM * 128;  // 64 channels of a tile, of queries
    extern __shared__ __align__(1024) uint8_t tile_raw[];
    S& sm = *reinterpret_cast<S*>(tile_raw);
    const AttnArgs& a = g.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kRingTiles; ++i) mbar_init(&sm.full[i], kUnits), mbar_init(&sm.empty[i], 2);
        for (int i = 0; i < kParStages; ++i) mbar_init(&sm.par_full[i], kUnits), mbar_init(&sm.par_empty[i], 8);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.q_full[i], 4), mbar_init(&sm.drained[i], 1);
            for (int j = 0; j < 2; ++j)
                mbar_init(&sm.s_full[i][j], 1), mbar_init(&sm.w_full[i][j], 4), mbar_init(&sm.o_full[i][j], 1);
        }
        fence_mbar_init();
    }
    if (warp == 15) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&sm.tmem))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    grid_dep_wait();
    grid_dep_launch();
    const long long total = g.seq_cost[a.b.n_seqs];
    const int ctas = (int)min((long long)gridDim.x, max(total, 1ll));
    const Cut cut(total, ctas);
    if (threadIdx.x < D / 2)
        sm.signs[threadIdx.x] = HAD && a.signs ? (a.signs[2 * threadIdx.x] < 0 ? 0x8000u : 0u) |
                                                     (a.signs[2 * threadIdx.x + 1] < 0 ? 0x80000000u : 0u)
                                               : 0u;
    if (threadIdx.x == 0) a.meta[blockIdx.x] = make_int4(0, 0, 0, 0);
    tc_before_sync();
    __syncthreads();
    tc_after_sync();
    const uint32_t tmem = sm.tmem;
    const bool works = (int)blockIdx.x < ctas && total > 0;
    // Waits give up after a while: results are void then, and every warp leaves its loop.
    const auto wait_one = [&](uint64_t* bar, uint32_t parity) {
        if (mbar_wait_1s(bar, parity, KVQ_WAIT_LIMIT(kTileWait))) return true;
        report_error(kErrBarrierTimeout);
        return false;
    };
    TileWalk& wk = sm.walk[warp];
    const auto advance = [&] {
        __syncwarp();
        if (lane == 0) wk.next(g);
        __syncwarp();
    };
    if (works && lane == 0) wk.begin(g, blockIdx.x, cut);
    __syncwarp();
    const auto wait = [&](uint64_t* bar, uint32_t parity) { return __all_sync(~0u, wait_one(bar, parity)) != 0; };

    // All warps of a warpgroup (0 .. 3, 4 .. 7, 8 .. 11, 12 .. 15) have to run one and the same setmaxnreg: the
    // roles part behind it, since producers and issuers share a warpgroup.
    if (works) {
        if (warp < 8) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
        else asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kProducerRegs));
    }
    if (works && warp < 8) {
        // ------------------------------------------------ softmax
        const int half = warp >> 2, r = threadIdx.x & 127;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // this warp's 32 lanes of tensor memory
        const uint32_t ts0 = tmem + lanes + half * 128, to = tmem + lanes + 256 + half * 128;
        uint32_t tile = 0;
        bool ok = true;
        const auto o_done = [&](uint32_t x) { return wait(&sm.o_full[half][x & 1], x >> 1 & 1); };  // O has tile x
        for (uint32_t item = 0; ok && wk.n > 0; advance(), ++item) {
            const TileItem& it = wk.it;
            Range see{0, 0x7FFFFFFF};  // rows that are not there count as seeing all
            float factor = 1.0f;
            {   // the query: rotated, split, into the tile
                const int i = it.c * kItemRows + half * kRowsM + r;  // row of the kv head's queries
                const bool there = i < it.nq;
                const int qr = i / a.G, row = it.lo + qr, head = it.h * a.G + i - qr * a.G;
                uint64_t v[D / 2];
                const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + row * a.q_row +
                                                                  head * a.q_head);
                if (there) {
                    see = seen_by(a, it.len, it.base + row, it.base + row);
                    see.t1 = min(see.t1, it.t1);
                }
#pragma unroll
                for (int k = 0; k < D / 8; ++k) {
                    uint4 u = there ? src[k] : make_uint4(0, 0, 0, 0);
                    if constexpr (HAD) {
                        const uint4 sg = *reinterpret_cast<const uint4*>(&sm.signs[4 * k]);
                        u.x ^= sg.x, u.y ^= sg.y, u.z ^= sg.z, u.w ^= sg.w;
                    }
                    const uint32_t word[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 f = a.bf16 ? Elem<__nv_bfloat16>::wide(word[j]) : Elem<__half>::wide(word[j]);
                        v[4 * k + j] = pair2(f.x, f.y);
                    }
                }
                if constexpr (HAD) {
                    const uint64_t minus = pair2(-1.0f, -1.0f);
#pragma unroll
                    for (int x = 1; x < D / 2; x <<= 1)
#pragma unroll
                        for (int k = 0; k < D / 2; ++k)
                            if (!(k & x)) {
                                const uint64_t p = v[k], q = v[k + x];
                                v[k] = add_f2(p, q);
                                v[k + x] = fma_f2(q, minus, p);
                            }
                }
                float m = 0.0f, bad = 0.0f;  // bad: NaN if anything is infinite or NaN
#pragma unroll
                for (int k = 0; k < D / 2; ++k) {
                    float x, y;
                    unpair2(v[k], x, y);
                    if constexpr (HAD) {
                        const float p = (x + y) * a.rsqd, q = (x - y) * a.rsqd;
                        x = p, y = q;
                        v[k] = pair2(x, y);
                    }
                    bad = __fmaf_rn(x, 0.0f, __fmaf_rn(y, 0.0f, bad));
                    m = fmaxf(m, fmaxf(fabsf(x), fabsf(y)));
                }
                if (bad != 0.0f) m = NAN;
                // Rows in this range keep 22 bits in the two fp16 parts as they are; others are scaled.
                if (!(m == 0.0f || (m >= 0x1p-4f && m <= 0x1p14f))) factor = query_scale(m);
                uint8_t* hi = sm.q[half][0] + r * 128;
#pragma unroll
                for (int k8 = 0; k8 < D / 8; ++k8) {
                    uint32_t wh[4], wl[4];
                    float x[8];
#pragma unroll
                    for (int k = 0; k < 4; ++k) unpair2(v[4 * k8 + k], x[2 * k], x[2 * k + 1]);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float p = x[place8(2 * k)] * factor, q = x[place8(2 * k + 1)] * factor;
                        const __half2 h = __floats2half2_rn(p, q);
                        wh[k] = *reinterpret_cast<const uint32_t*>(&h);
                        if constexpr (HAD) {
                            const float2 b = __half22float2(h);
                            const __half2 l = __floats2half2_rn(p - b.x, q - b.y);
                            wl[k] = *reinterpret_cast<const uint32_t*>(&l);
                        }
                    }
                    const int at = (k8 >> 3) * kQSlab + ((k8 & 7) ^ (r & 7)) * 16;
                    *reinterpret_cast<uint4*>(hi + at) = make_uint4(wh[0], wh[1], wh[2], wh[3]);
                    if constexpr (HAD) *reinterpret_cast<uint4*>(hi + S::kQuery + at) = make_uint4(wl[0], wl[1], wl[2], wl[3]);
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.q_full[half]);
            const bool scaled = __any_sync(~0u, factor != 1.0f);
            const float back = 1.0f / factor;
            const int see_lo = __reduce_max_sync(~0u, see.t0), see_hi = __reduce_min_sync(~0u, see.t1);  // all rows of the warp

            const int tiles = wk.n, first = (it.u0 + wk.u) * kTileTokens;
            float M = kLowest;
            uint64_t l2[2] = {pair2(0.0f, 0.0f), pair2(0.0f, 0.0f)};
            for (int n = 0; n < tiles; ++n, ++tile) {
                const int tok0 = first + n * kTileTokens;
                const uint32_t stage = tile % kParStages, ts = ts0 + (tile & 1) * kTileTokens;
                if (!(ok = wait(&sm.par_full[stage], tile / kParStages & 1)) ||
                    !(ok = wait(&sm.s_full[half][tile & 1], tile >> 1 & 1)) ||
                    !(ok = n < 2 || o_done(tile - 2)))  // (done when S is; a barrier's phases are waited for in turn)
                    break;
                tc_after_sync();
                const __half* par = sm.par[stage][0];
                const int2 ex = *reinterpret_cast<const int2*>(sm.expo[stage]);
                const uint2 gone = *reinterpret_cast<const uint2*>(sm.absent[stage]);
                const bool plain = !(scaled || tok0 < see_lo || tok0 + kTileTokens > see_hi || (gone.x | gone.y));
                int expo = max(ex.x, ex.y);  // of the largest V scale that the row sees
                if (!plain) {
                    // a huge one that it does not see would push the row's W below fp16's range (tokens that are not
                    // there have 0).  A short loop ahead of the scores: among them its registers cost a prompt 9%.
                    uint32_t most = 0;
#pragma unroll 1
                    for (int c = 0; c < kTileTokens; c += 8) {
                        const uint4 sv = *reinterpret_cast<const uint4*>(&par[kTileTokens + c]);
                        const uint32_t two[4] = {sv.x, sv.y, sv.z, sv.w};
                        const int t = tok0 + c;
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            most = max_u16x2(most, two[j] & ((t + 2 * j >= see.t0 && t + 2 * j < see.t1 ? 0xFFFFu : 0u) |
                                                             (t + 2 * j + 1 >= see.t0 && t + 2 * j + 1 < see.t1
                                                                  ? 0xFFFF0000u : 0u)));
                    }
                    expo = (int)max(max(most & 0xFFFFu, most >> 16) >> 10, 1u) - 15;
                }
                uint32_t s[2][32];
                tmem_load32(s[0], ts);
                tmem_load32(s[1], ts + 32);
                tmem_wait_load();
                if (!plain) {
                    // scores that are not plain: scaled rows, tokens that a row does not see
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int from = see.t0 - tok0 - 32 * e, to_ = see.t1 - tok0 - 32 * e;  // of these 32 tokens
                        const uint32_t sees = (to_ >= 32 ? ~0u : to_ > 0 ? (1u << to_) - 1 : 0u) &
                                              (from <= 0 ? ~0u : from < 32 ? ~0u << from : 0u) & ~(e ? gone.y : gone.x);
#pragma unroll
                        for (int c = 0; c < 32; ++c)
                            s[e][c] = sees >> c & 1 ? __float_as_uint(__uint_as_float(s[e][c]) * back)
                                                    : 0xFF800000u;  // -inf
                    }
                }
                float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int c = 0; c < 32; c += 8) {  // S sigma (a scale of 0 counts as the smallest: -inf stays)
                        const uint4 sk = *reinterpret_cast<const uint4*>(&par[32 * e + c]);
                        const uint32_t two[4] = {sk.x, sk.y, sk.z, sk.w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&two[j]));
                            uint32_t* x = &s[e][c + 2 * j];
                            float x0, x1;
                            unpair2(mul_f2(pair2(__uint_as_float(x[0]), __uint_as_float(x[1])), pair2(f.x, f.y)), x0, x1);
                            x[0] = __float_as_uint(x0), x[1] = __float_as_uint(x1);
                            tops[j] = fmaxf(tops[j], fmaxf(x0, x1));
                        }
                    }
                const float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3])) * a.scale2 + (float)expo;
                if (__any_sync(~0u, top > M + kSlack)) {
                    const float m2 = top > M + kSlack ? top : M, f = ex2(M - m2);  // (other rows as they were)
                    const uint64_t ff = pair2(f, f);
                    M = m2;
                    l2[0] = mul_f2(l2[0], ff);
                    l2[1] = mul_f2(l2[1], ff);
                    if (n > 0) {  // O, once the tile before is in it
                        if (!(ok = o_done(tile - 1))) break;
                        tc_after_sync();
#pragma unroll 1
                        for (int k = 0; k < D; k += 32) {
                            uint32_t o[32];
                            tmem_load32(o, to + k);
                            tmem_wait_load();
#pragma unroll
                            for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * f);
                            tmem_store32(to + k, o);
                        }
                    }
                }
                const uint64_t ref = pair2(kTileBias - M, kTileBias - M), scale2 = pair2(a.scale2, a.scale2);
                uint32_t w[32];
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int c = 0; c < 32; c += 8) {
                        const uint4 sv = *reinterpret_cast<const uint4*>(&par[kTileTokens + 32 * e + c]);
                        const uint32_t two[4] = {sv.x, sv.y, sv.z, sv.w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const uint32_t* x = &s[e][c + 2 * j];
                            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&two[j]));
                            float p0, p1;
                            unpair2(fma_f2(pair2(__uint_as_float(x[0]), __uint_as_float(x[1])), scale2, ref), p0, p1);
                            const uint64_t p = pair2(ex2(p0), ex2(p1));
                            l2[j & 1] = add_f2(l2[j & 1], p);
                            unpair2(mul_f2(p, pair2(f.x, f.y)), p0, p1);
                            w[16 * e + c / 2 + j] = Elem<__half>::pack(p0, p1);
                        }
                    }
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.par_empty[stage]);
                tmem_store32(ts, w);
                tmem_wait_store();
                tc_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.w_full[half][tile & 1]);
            }
            if (!ok || !(ok = (tiles < 2 || o_done(tile - 2)) && o_done(tile - 1))) break;
            tc_after_sync();
            const int i = it.c * kItemRows + half * kRowsM + r;
            const bool there = i < it.nq;
            const int row = it.lo + i / a.G, head = it.h * a.G + i % a.G;
            float la, lb;
            unpair2(add_f2(l2[0], l2[1]), la, lb);
            const float l = la + lb;
            const bool begins = wk.u == 0, ends = wk.u + wk.n == it.units, whole = begins && ends;
            float o[D];
#pragma unroll
            for (int k = 0; k < D; k += 32) {
                uint32_t x[32];
                tmem_load32(x, to + k);
                tmem_wait_load();
#pragma unroll
                for (int c = 0; c < 32; ++c) o[k + (c & ~7) + place8(c & 7)] = __uint_as_float(x[c]);
            }
            tc_before_sync();
            if (whole) {
                const float inv = l == 0.0f ? 0.0f : 1.0f / l;
                if constexpr (HAD) lane_stages<1, D>(o);
                const float unit = HAD ? inv * a.rsqd : inv;
                uint16_t* dst = static_cast<uint16_t*>(a.out) + row * a.o_row + head * a.o_head;
#pragma unroll
                for (int k = 0; k < D; k += 8) {
                    uint32_t w[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const float x = o[k + 2 * c] * unit, y = o[k + 2 * c + 1] * unit;
                        w[c] = a.bf16 ? Elem<__nv_bfloat16>::pack(x, y) : Elem<__half>::pack(x, y);
                        if constexpr (HAD) w[c] ^= sm.signs[k / 2 + c];
                    }
                    if (there) *reinterpret_cast<uint4*>(dst + k) = make_uint4(w[0], w[1], w[2], w[3]);
                }
                if (there && a.lse) a.lse[(long long)row * a.Hq + head] = (M - kTileBias + lg2(l)) * kLn2;
            } else if (there) {
                const long long at = (2ll * blockIdx.x + (begins ? 1 : 0)) * kItemRows + half * kRowsM + r;
                reinterpret_cast<float2*>(a.ml)[at] = make_float2(M + (kBias - kTileBias), l);
                float4* dst = reinterpret_cast<float4*>(a.part + at * D);
#pragma unroll
                for (int p = 0; p < D; p += 4)
                    dst[p / 4] = make_float4(o[channel_of<D>(p)], o[channel_of<D>(p + 1)], o[channel_of<D>(p + 2)],
                                             o[channel_of<D>(p + 3)]);
            }
            if (begins && !ends && threadIdx.x == 0) {
                // CTAs from this one to that of the item's last tile
                const long long item = cut.begin(blockIdx.x + 1) - wk.left - wk.from;  // its first position
                a.meta[blockIdx.x] = make_int4(it.s, it.h, it.c * kItemRows,
                                               (int)(cut.of(item + kItemCost + it.units - 1) - blockIdx.x) + 1);
            }
        }
    } else if (works && warp >= 14) {
        // ------------------------------------------------ products
        // All lanes walk along, so that addresses and descriptors stay in uniform registers; one issues.  (With
        // one lane in the loop an issue took 80 cycles, longer than the product itself.)
        constexpr uint32_t kS = mma_desc(kTileTokens, false), kO = mma_desc(D, true);
        const uint32_t tm = __shfl_sync(~0u, tmem, 0);
        const uint64_t ring = smem_desc(smem_u32(sm.ring[0]), 16), ring_v = smem_desc(smem_u32(sm.ring[0]), kSlab);
        const uint64_t q = smem_desc(smem_u32(sm.q[0][0]), 16);
        const uint32_t half = __shfl_sync(~0u, warp & 1, 0);
        uint32_t tile = 0;  // the item's first, of all the CTA's
        bool ok = true;
        // S of tile x: K is number 2 x of the ring's tiles
        const auto scores = [&](uint32_t x) {
            const uint32_t buf = 2 * x % kRingTiles;
            if (!(ok = wait(&sm.full[buf], 2 * x / kRingTiles & 1))) return;
            tc_after_sync();
            const uint32_t d = tm + half * 128 + (x & 1) * kTileTokens;
            const uint64_t qd = q + half * ((HAD ? 2 : 1) * S::kQuery >> 4), kd = ring + buf * (kTile >> 4);
            if (elect_one()) {
#pragma unroll
                for (int part = 0; part < (HAD ? 2 : 1); ++part)
#pragma unroll
                    for (int k = 0; k < D / 16; ++k)
                        mma_ss(d, qd + ((part * S::kQuery + (k >> 2) * kQSlab + (k & 3) * 32) >> 4),
                               kd + (((k >> 2) * kSlab + (k & 3) * 32) >> 4), kS, part + k > 0);
                mma_commit(&sm.s_full[half][x & 1]);
                mma_commit(&sm.empty[buf]);
            }
            __syncwarp();
        };
        // O of tile x: V is number 2 x + 1
        const auto values = [&](uint32_t x, bool add) {
            const uint32_t buf = (2 * x + 1) % kRingTiles;
            if (!(ok = wait(&sm.full[buf], (2 * x + 1) / kRingTiles & 1))) return;
            if (!(ok = wait(&sm.w_full[half][x & 1], x >> 1 & 1))) return;
            tc_after_sync();
            const uint32_t d = tm + 256 + half * 128, w = tm + half * 128 + (x & 1) * kTileTokens;
            const uint64_t vd = ring_v + buf * (kTile >> 4);
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < kTileTokens / 16; ++k) mma_ts(d, w + 8 * k, vd + (k * 2048 >> 4), kO, add || k > 0);
                mma_commit(&sm.o_full[half][x & 1]);
                mma_commit(&sm.empty[buf]);
            }
            __syncwarp();
        };
        for (uint32_t item = 0; ok; ++item) {
            const int tiles = __shfl_sync(~0u, wk.n, 0);
            if (tiles == 0) break;
            ok = wait(&sm.q_full[half], item & 1);
            for (int n = -2; n < tiles && ok; ++n) {  // O of tile n, S of tile n + 2
                if (n >= 0) values(tile + n, n > 0);
                if (ok && n + 2 < tiles) scores(tile + n + 2);
            }
            tile += tiles;
            advance();
        }
        if (!ok && elect_one()) {  // products in flight end before tensor memory is given back
            mma_commit(&sm.drained[half]);
            mbar_wait_1s(&sm.drained[half], 0, kTileWait);
        }
        __syncwarp();
    } else if (works) {
        // ------------------------------------------------ tiles of K and V
        // units of 32 tokens: those of a step's K tile, of its V tile, of the next step's, ..; this warp
        // takes every kProducers-th
        uint32_t step = 0, unit = warp - 8;
        int n = 0;  // the step's tile in the segment
        const auto seek = [&] {  // the walk to the unit's step; false at the end
            for (; step < unit / (2 * kUnits) && wk.n > 0; ++step)
                if (++n == wk.n) {
                    advance();
                    n = 0;
                }
            return wk.n > 0;
        };
        const auto token = [&] { return (wk.it.u0 + wk.u + n) * kTileTokens + kUnitTokens * (int)(unit % kUnits); };
        int page0 = 0, page1 = 0;
        const auto look_up = [&] {  // a unit ahead of the codes
            const int tok = token(), t0 = wk.it.t0, t1 = wk.it.t1;
            const int* row = a.b.table + (long long)wk.it.s * a.b.table_stride;
            page0 = tok + 16 > t0 && tok < t1 ? row[tok >> a.p.page_log2] : 0;
            page1 = tok + 32 > t0 && tok + 16 < t1 ? row[(tok + 16) >> a.p.page_log2] : 0;
        };
        bool more = seek();
        if (more) look_up();
        while (more) {
            const uint32_t is_v = unit / kUnits & 1, rows = kUnitTokens * (unit % kUnits);
            const uint32_t stage = step % kParStages, turn = step / kParStages;
            const uint32_t seq = 2 * step + is_v, buf = seq % kRingTiles, round = seq / kRingTiles;
            Unit<D> un;
            un.fetch(g, wk.it.h, wk.it.t0, wk.it.t1, token(), is_v, page0, page1);
            unit += kProducers;
            more = seek();
            if (more) look_up();
            if (round > 0 && !wait(&sm.empty[buf], (round - 1) & 1)) break;
            if (!is_v) {
                if (turn > 0 && !wait(&sm.par_empty[stage], (turn - 1) & 1)) break;
                const uint32_t absent = __ballot_sync(~0u, un.absent);
                const uint32_t expo = __reduce_max_sync(~0u, (uint32_t)__half_as_ushort(un.scale[1]) >> 10);
                sm.par[stage][0][rows + lane] = __hmax(un.scale[0], __ushort_as_half(1));
                sm.par[stage][1][rows + lane] = un.scale[1];
                if (lane == 0) {
                    sm.absent[stage][rows / kUnitTokens] = absent;
                    sm.expo[stage][rows / kUnitTokens] = (int)max(expo, 1u) - 15;
                }
            }
            un.store(sm.ring[buf], rows);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&sm.full[buf]);
                if (!is_v) mbar_arrive(&sm.par_full[stage]);
            }
        }
    }
    tc_before_sync();
    __syncthreads();
    if (warp == 15) {
        tc_after_sync();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
    }
}

}  // namespace kvq
