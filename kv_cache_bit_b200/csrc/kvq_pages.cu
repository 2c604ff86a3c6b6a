// kvq_pages.cu -- host side of the paged 4-bit cache (kvq_pages_* of
// include/kvq.h): argument checks and launches.  A translation unit of its
// own, with its own copy of the device error word of kvq_device.cuh, which
// kvq_pages_read_errors reads.
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>

#include <nvtx3/nvToolsExt.h>

#include "kvq.h"
#include "kvq_pages.cuh"
#include "kvq_pages_attn.cuh"
#include "kvq_pages_step.cuh"
#include "kvq_pages_tile.cuh"

namespace kvq {
namespace {

constexpr int64_t kMaxIndex = int64_t(1) << 31;
constexpr int64_t kMaxVectors = int64_t(1) << 29;  // rows x heads of a write or read: lanes, four each, are counted in 32 bits
constexpr int kMaxGroup = 256;  // query heads per kv head
// Which of the two kernels a sequence goes to, by its query rows a kv head.  The generation-step kernel reads the
// cache once for 16 of them at most (four or eight where the call's single rows ask for no more), the tile kernel
// once for 256, with half the multiprocessor idle below 129.
//   A call whose sequences all have up to kFewRows is the step kernel's alone.  Step and tile kernel, us, at about
//   64, 80 and 112 rows, rotated, 16 x 300 .. 3001 tokens: 28 over 4 heads, D = 128: 48 62, 64 62, 83 63; 32 over 32:
//   302 394, 370 388, 504 386; 32 over 8, D = 64: 72 82, 78 82, 102 83; 64 x 500 .. 4000, 32 over 8, D = 64: 234 300,
//   291 301, 394 301.
//   Beside sequences of more, and where the host does not know, those of up to kFewBeside: two of 500 rows and 14 of
//   24, 32 and 48 rows, 600 .. 3001 tokens, D = 128, 32 over 8: 140 144, 151 145, 174 147; of 32 x 2000 .. 4000 four and
//   28 of these: 332 369, 367 370, 438 369; D = 64: 264 325, 287 323, 336 325.
constexpr int kFewRows = 80, kFewBeside = 32;

struct NvtxRange {
    explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
    ~NvtxRange() { nvtxRangePop(); }
    NvtxRange(const NvtxRange&) = delete;
    NvtxRange& operator=(const NvtxRange&) = delete;
};

// a * b >= limit, for a, b >= 0 and b < 2^31.
bool reaches(int64_t a, int64_t b, int64_t limit) { return a >= kMaxIndex || a * b >= limit; }

bool ok_ptr(const void* p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool ok_ints(const void* p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

kvq_status launch_status() { return cudaGetLastError() == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA; }

// Configuration, pool and batch; the checks every paged call shares.
kvq_status check_paged(const kvq_config* cfg, const kvq_pages* p, const kvq_batch* b, int64_t rows) {
    if (cfg == nullptr || p == nullptr || b == nullptr) return KVQ_ERR_INVALID_ARG;
    if (cfg->reserved != 0 || rows < 0) return KVQ_ERR_INVALID_ARG;
    if (cfg->signs != nullptr && !ok_ptr(cfg->signs)) return KVQ_ERR_INVALID_ARG;
    if (cfg->bits != 4 || (cfg->head_dim != 64 && cfg->head_dim != 128)) return KVQ_ERR_UNSUPPORTED;
    if (cfg->flags != 0 && cfg->flags != KVQ_HADAMARD) return KVQ_ERR_UNSUPPORTED;
    if (p->n_pages < 1 || p->kv_heads < 1 || p->head_dim != cfg->head_dim) return KVQ_ERR_INVALID_ARG;
    const int t = p->page_tokens;
    if (t != 16 && t != 32 && t != 64 && t != 128) return KVQ_ERR_UNSUPPORTED;
    for (int i = 0; i < 2; ++i)
        if (!ok_ptr(p->codes[i]) || !ok_ptr(p->tok[i])) return KVQ_ERR_INVALID_ARG;
    if ((int64_t)p->n_pages * p->kv_heads >= kMaxIndex / t) return KVQ_ERR_UNSUPPORTED;
    if (b->n_seqs < 0 || b->max_rows < 0) return KVQ_ERR_INVALID_ARG;
    if (b->n_seqs > 0) {
        if (b->max_pages < 1 || b->table_stride < b->max_pages) return KVQ_ERR_INVALID_ARG;
        if (!ok_ints(b->start) || !ok_ints(b->len) || !ok_ints(b->table)) return KVQ_ERR_INVALID_ARG;
        // tokens are rounded up to units of 64 in 32 bits
        if ((int64_t)b->max_pages * t > kMaxIndex - 256) return KVQ_ERR_UNSUPPORTED;
    }
    return KVQ_OK;
}

// From the first to the last element of a rows tensor at most: far above what
// a GPU holds, and sums of its offsets are far from 64 bits.
constexpr int64_t kMaxExtent = int64_t(1) << 42;

// A rows tensor; strides of dimensions of one element are not looked at.
kvq_status check_rows(const kvq_rows* x, int64_t rows, int heads, int d, bool output, bool f32) {
    if (x == nullptr || !ok_ptr(x->data) || x->reserved != 0) return KVQ_ERR_INVALID_ARG;
    if (x->dtype != KVQ_F16 && x->dtype != KVQ_BF16 && !(f32 && x->dtype == KVQ_F32)) return KVQ_ERR_UNSUPPORTED;
    const int64_t unit = x->dtype == KVQ_F32 ? 4 : 8;  // elements of 16 bytes
    const int64_t rs = rows > 1 ? x->row_stride : 0, hs = heads > 1 ? x->head_stride : 0;
    if (rs % unit != 0 || hs % unit != 0) return KVQ_ERR_INVALID_ARG;
    const int64_t most = kMaxExtent / (x->dtype == KVQ_F32 ? 4 : 2);  // elements
    if (rs > most || rs < -most || hs > most || hs < -most) return KVQ_ERR_INVALID_ARG;
    const __int128 span = (__int128)(rs < 0 ? -rs : rs) * (rows - 1) + (__int128)(hs < 0 ? -hs : hs) * (heads - 1) + d;
    if (rows > 0 && span > most) return KVQ_ERR_INVALID_ARG;
    if (output) {  // no two elements in one place: rows inside heads or heads inside rows
        if ((rows > 1 && rs < d) || (heads > 1 && hs < d)) return KVQ_ERR_INVALID_ARG;
        if (rows > 1 && heads > 1 && rs < (heads - 1) * hs + d && hs < (rows - 1) * rs + d) return KVQ_ERR_INVALID_ARG;
    }
    return KVQ_OK;
}

// Bytes [lo, hi) from the first to the last element.
void extent(const kvq_rows* x, int64_t rows, int heads, int d, intptr_t* lo, intptr_t* hi) {
    const int64_t size = x->dtype == KVQ_F32 ? 4 : 2;
    const int64_t r = (rows - 1) * x->row_stride * (rows > 1), h = (heads - 1) * x->head_stride * (heads > 1);
    const intptr_t at = reinterpret_cast<intptr_t>(x->data);
    *lo = at + size * ((r < 0 ? r : 0) + (h < 0 ? h : 0));
    *hi = at + size * ((r > 0 ? r : 0) + (h > 0 ? h : 0) + d);
}

// Whether x and outputs y share an element.  Slices of one buffer (of the same
// strides) are looked at element by element; what others are taken for, where
// their extents meet, is the caller's choice.
bool overlap(const kvq_rows* x, const kvq_rows* y, int64_t rows, int heads, int d, bool others) {
    intptr_t xl, xh, yl, yh;
    extent(x, rows, heads, d, &xl, &xh);
    extent(y, rows, heads, d, &yl, &yh);
    if (xl >= yh || yl >= xh) return false;
    const int64_t rs = rows > 1 ? y->row_stride : 0, hs = heads > 1 ? y->head_stride : 0;  // of an output: positive
    if ((rows > 1 && x->row_stride != rs) || (heads > 1 && x->head_stride != hs)) return others;
    // vectors u rows and w heads apart share one iff |at + u rs| < d
    const int64_t size = x->dtype == KVQ_F32 ? 4 : 2;
    const int64_t delta = (reinterpret_cast<intptr_t>(y->data) - reinterpret_cast<intptr_t>(x->data)) / size;
    for (int64_t w = 1 - (int64_t)heads; w < heads; ++w) {
        const int64_t at = delta + w * hs;
        int64_t u = 0, rest = at;  // rest = at + u rs, the last below rs
        if (rs > 0) {
            u = -(at / rs);
            rest = at % rs;
            if (rest < 0) rest += rs, ++u;
        }
        const auto hit = [&](int64_t n, int64_t v) { return n > -rows && n < rows && v < d && v > -d; };
        if (hit(u, rest) || (rs > 0 && hit(u - 1, rest - rs))) return true;
    }
    return false;
}

Batch batch_of(const kvq_batch* b) {
    return Batch{b->start, b->len, b->table, b->n_seqs, b->max_pages, b->table_stride};
}

Pool pool_of(const kvq_pages* p) {
    Pool o;
    for (int i = 0; i < 2; ++i) {
        o.codes[i] = p->codes[i];
        o.tok[i] = reinterpret_cast<__half*>(p->tok[i]);
    }
    o.n_pages = p->n_pages;
    o.H = p->kv_heads;
    o.page_log2 = p->page_tokens == 16 ? 4 : p->page_tokens == 32 ? 5 : p->page_tokens == 64 ? 6 : 7;
    return o;
}

float rsqd_of(int d) { return (float)(1.0 / std::sqrt((double)d)); }

// SMs of the current device.
int sm_count() {
    static std::atomic<int> known[64];
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
        cudaGetLastError();
        return 148;
    }
    if ((n = known[dev].load(std::memory_order_relaxed)) > 0) return n;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) {
        cudaGetLastError();
        return 148;
    }
    known[dev].store(n, std::memory_order_relaxed);
    return n;
}

// Heads of a row that a quad of lanes takes in turn: one while that leaves quads for every SM's schedulers
// (a generation step), eight at most.
int heads_a_quad(int64_t rows, int H) {
    int per = 1;
    while (per < 8 && per * 2 <= H && rows * H >= (int64_t)per * 2 * sm_count() * 128) per *= 2;
    return per;
}

// Compile-time dispatch over (head_dim, element type, rotation).
template <int D, typename T, typename Fn>
kvq_status dispatch_had(bool had, Fn& fn) {
    return had ? fn.template run<D, T, true>() : fn.template run<D, T, false>();
}

template <typename Fn>
kvq_status dispatch(int d, int dtype, bool had, Fn& fn) {
    if (dtype == KVQ_F16) return d == 64 ? dispatch_had<64, __half>(had, fn) : dispatch_had<128, __half>(had, fn);
    return d == 64 ? dispatch_had<64, __nv_bfloat16>(had, fn) : dispatch_had<128, __nv_bfloat16>(had, fn);
}

// Launch as a programmatic dependent of the kernel ahead of it in the stream:
// the kernels wait for that one (grid_dep_wait) before they read anything.
template <typename... A>
kvq_status launch(void (*kernel)(A...), dim3 grid, int threads, int smem, cudaStream_t st, const A&... args) {
    cudaLaunchConfig_t c = {};
    c.gridDim = grid;
    c.blockDim = dim3(threads);
    c.dynamicSmemBytes = smem;
    c.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    c.attrs = at;
    c.numAttrs = 1;
    if (cudaLaunchKernelEx(&c, kernel, args...) != cudaSuccess) {
        cudaGetLastError();
        return KVQ_ERR_CUDA;
    }
    return launch_status();
}

struct WriteLaunch {
    WriteArgs a;
    unsigned grid;
    cudaStream_t st;
    template <int D, typename T, bool HAD>
    kvq_status run() {
        return launch(pages_write_kernel<D, T, HAD>, dim3(grid, 2), kWriteThreads, 0, st, a);
    }
};

struct ReadLaunch {
    ReadArgs a;
    unsigned grid;
    cudaStream_t st;
    template <int D, typename T, bool HAD>
    kvq_status run() {
        return launch(pages_read_kernel<D, T, HAD>, dim3(grid, a.only >= 0 ? 1 : 2), kWriteThreads, 0, st, a);
    }
};

// Dynamic shared memory and the largest carveout, once per kernel and device
// (racing callers set the same attributes, which is harmless).  regs: what the
// kernel's register split needs the launch to give a thread.
template <auto Kernel>
bool allow_smem(int bytes, int regs = 0) {
    static std::atomic<uint64_t> done{0};  // one bit a device
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
    const uint64_t bit = uint64_t(1) << dev;
    if (done.load(std::memory_order_acquire) & bit) return true;
    if (cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess ||
        cudaFuncSetAttribute(Kernel, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared) !=
            cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    if (regs > 0) {
        cudaFuncAttributes at;
        if (cudaFuncGetAttributes(&at, Kernel) != cudaSuccess || at.numRegs < regs) {
            cudaGetLastError();
            return false;
        }
    }
    done.fetch_or(bit, std::memory_order_release);
    return true;
}

// Generation-step kernel: CTAs of a single wave, and query rows an item.
template <int NQ>
struct StepShape {
    static constexpr int kWarps = NQ == 16 ? 8 : 4, kPerSm = NQ == 16 ? 1 : 3;
};

// Which kernels a call needs, from what the host knows of it.
struct AttnPlan {
    bool tiles;        // some sequence may have more than kFewRows query rows a kv head
    int stretch;       // with tiles: rows of a sequence of up to kFewBeside
    long long places;  // rows that the step kernel's queries are prepared for
    long long queries; // query rows a kv head of the sequences that are the step kernel's
};
AttnPlan attn_plan(const kvq_batch* b, long long rows, int G) {
    AttnPlan p;
    const long long most = (long long)G * b->max_rows;
    p.tiles = b->max_rows == 0 || most > kFewRows;
    p.stretch = p.tiles ? kFewBeside / G : 0;
    p.places = p.tiles ? (long long)b->n_seqs * p.stretch : rows;
    p.queries = p.tiles ? G : most;
    return p;
}

struct AttnWorkspace {
    size_t meta, ml, part, left, frag, scal;                 // step kernel
    size_t tile_meta, tile_ml, tile_part, plan, seq_cost;    // tile kernel
    size_t bytes;
};
AttnWorkspace attn_workspace(const AttnPlan& p, int sms, int d, bool had, int q_heads, int n_seqs) {
    size_t ctas = 0, queries = 0, warps = 0;  // the most of any shape: CTAs, and query rows over all CTAs and warps
    const auto shape = [&](int per_sm, int nw, int nq) {
        const size_t n = size_t(sms) * per_sm;
        if (n > ctas) ctas = n;
        if (n * nq > queries) queries = n * nq;
        if (n * nq * nw > warps) warps = n * nq * nw;
    };
    shape(StepShape<8>::kPerSm, StepShape<8>::kWarps, 8);
    shape(StepShape<16>::kPerSm, StepShape<16>::kWarps, 16);
    AttnWorkspace w;
    size_t at = 0;
    const auto take = [&](size_t bytes) {
        const size_t here = at;
        at += (bytes + 255) / 256 * 256;
        return here;
    };
    w.meta = take(ctas * 16);
    w.ml = take(2 * queries * 8);
    w.part = take(2 * queries * d * 4);
    w.left = take(warps * d * 4);
    w.frag = take(size_t(p.places) * q_heads * d * (had ? 4 : 2));
    w.scal = take(size_t(p.places) * q_heads * 4);
    const size_t tiles = p.tiles ? size_t(sms) : 0;
    w.tile_meta = take(tiles * 16);
    w.tile_ml = take(2 * tiles * kItemRows * 8);
    w.tile_part = take(2 * tiles * kItemRows * d * 4);
    w.plan = take(tiles * 16);
    w.seq_cost = take(p.tiles ? (size_t(n_seqs) + 1) * 8 : 0);
    w.bytes = at;
    return w;
}

// Caches of up to this many tokens (by the table's width) are taken whole where there is a CTA for every item.
// In ranges with a merge, and whole, us, at tables of 256, 512 and 768 tokens: 1 sequence, 8 heads, D = 64: 9.0 7.3,
// 9.1 8.8, 9.4 9.8; 4 of a quarter of that up to it, 32 over 8 heads, D = 128: 10.8 8.2, 11.3 9.8, 11.4 11.8; 1
// sequence, 28 over 4 heads: 11.2 9.8, 11.9 12.0, 12.1 13.9; 12, 28 over 4: 12.9 10.1, 13.1 12.1, 13.6 13.9.
constexpr long long kWholeTokens = 512;

template <int D, int NQ, bool HAD>
kvq_status launch_step(StepArgs g, long long tokens, int sms, cudaStream_t st) {
    using Sh = StepShape<NQ>;
    constexpr int smem = (int)sizeof(StepSmem<D, NQ, HAD, Sh::kWarps>);
    static_assert(smem * Sh::kPerSm + Sh::kPerSm * 1024 <= 228 * 1024, "shared memory of the CTAs on one SM");
    constexpr auto kernel = pages_step_kernel<D, NQ, HAD, Sh::kWarps, Sh::kPerSm>;
    if (!allow_smem<kernel>(smem)) return KVQ_ERR_CUDA;
    const int grid = sms * Sh::kPerSm;
    // at most: whatever the rows are, a sequence has one chunk that is not full
    const long long items = (long long)g.a.p.H * (g.a.rows * (long long)g.a.G / NQ + g.a.b.n_seqs);
    g.whole = tokens <= kWholeTokens && items <= grid;
    const kvq_status s = launch(kernel, dim3(g.whole ? (int)items : grid), Sh::kWarps * 32, smem, st, g);
    if (s != KVQ_OK || g.whole) return s;
    return launch(pages_merge_kernel<D, NQ, HAD>, dim3(grid, NQ / merge_queries(NQ)), kMergeWarps * 32, 0, st, g.a);
}

template <int D, bool HAD>
kvq_status launch_tiles(const TileArgs& t, int sms, cudaStream_t st) {
    constexpr auto kernel = pages_tile_kernel<D, HAD>;
    constexpr int smem = (int)sizeof(TileSmem<D, HAD>);
    static_assert(smem <= 227 * 1024, "shared memory of a CTA");
    if (!allow_smem<kernel>(smem, kLaunchRegs)) return KVQ_ERR_CUDA;
    const kvq_status s = launch(kernel, dim3(sms), kTileThreads, smem, st, t);
    if (s != KVQ_OK) return s;
    return launch(pages_merge_kernel<D, kItemRows, HAD>, dim3(sms, kItemRows / merge_queries(kItemRows)), kMergeWarps * 32, 0,
                  st, t.a);
}

template <int D, bool HAD>
kvq_status launch_attn(const StepArgs& g, const TileArgs& t, const AttnPlan& p, int sms, cudaStream_t st) {
    const unsigned ctas = (unsigned)((p.places * g.a.Hq + kQueryWarps - 1) / kQueryWarps) + (p.tiles ? 1 : 0);
    kvq_status s = launch(pages_queries_kernel<D, HAD>, dim3(ctas), kQueryWarps * 32, 0, st, g, t, p.tiles ? sms : 0);
    if (s == KVQ_OK && p.places > 0) {
        const long long tokens = (long long)g.a.b.max_pages << g.a.p.page_log2;
        if (HAD && p.queries <= 4) s = launch_step<D, HAD ? 4 : 8, HAD>(g, tokens, sms, st);
        else if (p.queries <= 8) s = launch_step<D, 8, HAD>(g, tokens, sms, st);
        else s = launch_step<D, 16, HAD>(g, tokens, sms, st);
    }
    if (s == KVQ_OK && p.tiles) s = launch_tiles<D, HAD>(t, sms, st);
    return s;
}

kvq_status check_attention(const kvq_config* cfg, const kvq_pages* p, const kvq_batch* b, int64_t rows, int q_heads) {
    const kvq_status s = check_paged(cfg, p, b, rows);
    if (s != KVQ_OK) return s;
    if (q_heads < p->kv_heads || q_heads % p->kv_heads != 0) return KVQ_ERR_INVALID_ARG;
    if (q_heads / p->kv_heads > kMaxGroup || q_heads > 65535 || reaches(rows, q_heads, kMaxIndex) ||
        reaches(b->n_seqs, kFewRows * (int64_t)q_heads, kMaxIndex))  // prepared queries are counted in 32 bits
        return KVQ_ERR_UNSUPPORTED;
    return KVQ_OK;
}

}  // namespace
}  // namespace kvq

using namespace kvq;

extern "C" {

kvq_status kvq_pages_write(const kvq_config* cfg, const kvq_pages* pages, const kvq_batch* batch, const kvq_rows* k,
                           const kvq_rows* v, int64_t rows, void* stream) {
    NvtxRange nvtx_range("kvq_pages_write");
    kvq_status s = check_paged(cfg, pages, batch, rows);
    if (s != KVQ_OK) return s;
    const int H = pages->kv_heads, d = cfg->head_dim;
    if (reaches(rows, H, kMaxVectors)) return KVQ_ERR_UNSUPPORTED;
    if ((s = check_rows(k, rows, H, d, false, false)) != KVQ_OK) return s;
    if ((s = check_rows(v, rows, H, d, false, false)) != KVQ_OK) return s;
    if (k->dtype != v->dtype) return KVQ_ERR_INVALID_ARG;
    if (rows == 0 || batch->n_seqs == 0) return KVQ_OK;
    WriteLaunch L;
    L.a.b = batch_of(batch);
    L.a.p = pool_of(pages);
    const kvq_rows* x[2] = {k, v};
    for (int i = 0; i < 2; ++i) {
        L.a.x[i] = x[i]->data;
        L.a.row_stride[i] = rows > 1 ? x[i]->row_stride : 0;
        L.a.head_stride[i] = H > 1 ? x[i]->head_stride : 0;
    }
    L.a.signs = cfg->signs;
    L.a.rows = (int)rows;
    L.a.rsqd = rsqd_of(d);
    L.a.per = heads_a_quad(rows, H);
    L.grid = (unsigned)((rows * ((H + L.a.per - 1) / L.a.per) * 4 + kWriteThreads - 1) / kWriteThreads);
    L.st = static_cast<cudaStream_t>(stream);
    return dispatch(d, k->dtype, cfg->flags == KVQ_HADAMARD, L);
}

kvq_status kvq_pages_read(const kvq_config* cfg, const kvq_pages* pages, const kvq_batch* batch, const kvq_rows* k_out,
                          const kvq_rows* v_out, int64_t rows, void* stream) {
    NvtxRange nvtx_range("kvq_pages_read");
    kvq_status s = check_paged(cfg, pages, batch, rows);
    if (s != KVQ_OK) return s;
    const int H = pages->kv_heads, d = cfg->head_dim;
    if (reaches(rows, H, kMaxVectors)) return KVQ_ERR_UNSUPPORTED;
    if (k_out == nullptr && v_out == nullptr) return KVQ_ERR_INVALID_ARG;
    const kvq_rows* x[2] = {k_out, v_out};
    for (int i = 0; i < 2; ++i)
        if (x[i] != nullptr && (s = check_rows(x[i], rows, H, d, true, true)) != KVQ_OK) return s;
    if (k_out != nullptr && v_out != nullptr && (k_out->dtype != v_out->dtype || k_out->data == v_out->data))
        return KVQ_ERR_INVALID_ARG;
    if (rows == 0 || batch->n_seqs == 0) return KVQ_OK;
    if (k_out != nullptr && v_out != nullptr && overlap(k_out, v_out, rows, H, d, false)) return KVQ_ERR_INVALID_ARG;
    ReadLaunch L;
    L.a.b = batch_of(batch);
    L.a.p = pool_of(pages);
    for (int i = 0; i < 2; ++i) {
        L.a.out[i] = x[i] ? x[i]->data : nullptr;
        L.a.row_stride[i] = x[i] && rows > 1 ? x[i]->row_stride : 0;
        L.a.head_stride[i] = x[i] && H > 1 ? x[i]->head_stride : 0;
    }
    L.a.signs = cfg->signs;
    L.a.rows = (int)rows;
    L.a.only = k_out == nullptr ? 1 : v_out == nullptr ? 0 : -1;
    L.a.rsqd = rsqd_of(d);
    L.a.per = heads_a_quad(rows, H);
    L.grid = (unsigned)((rows * ((H + L.a.per - 1) / L.a.per) * 4 + kWriteThreads - 1) / kWriteThreads);
    L.st = static_cast<cudaStream_t>(stream);
    const bool had = cfg->flags == KVQ_HADAMARD;
    const int dtype = (k_out ? k_out : v_out)->dtype;
    if (dtype == KVQ_F32) return d == 64 ? dispatch_had<64, float>(had, L) : dispatch_had<128, float>(had, L);
    return dispatch(d, dtype, had, L);
}

size_t kvq_pages_attention_workspace_bytes(const kvq_config* cfg, const kvq_pages* pages, const kvq_batch* batch,
                                           int64_t rows, int32_t q_heads) {
    if (check_attention(cfg, pages, batch, rows, q_heads) != KVQ_OK) return 0;
    const AttnPlan p = attn_plan(batch, rows, q_heads / pages->kv_heads);
    return attn_workspace(p, sm_count(), cfg->head_dim, cfg->flags == KVQ_HADAMARD, q_heads, batch->n_seqs).bytes;
}

kvq_status kvq_pages_attention(const kvq_config* cfg, const kvq_pages* pages, const kvq_batch* batch,
                               const kvq_rows* q, int32_t q_heads, int64_t rows, float scale, int32_t causal,
                               int32_t window, const kvq_rows* out, float* lse, void* ws, size_t ws_bytes,
                               void* stream) {
    NvtxRange nvtx_range("kvq_pages_attention");
    kvq_status s = check_attention(cfg, pages, batch, rows, q_heads);
    if (s != KVQ_OK) return s;
    const int d = cfg->head_dim;
    if ((s = check_rows(q, rows, q_heads, d, false, false)) != KVQ_OK) return s;
    if ((s = check_rows(out, rows, q_heads, d, true, false)) != KVQ_OK) return s;
    if (q->dtype != out->dtype || window < 0 || (window > 0 && causal == 0)) return KVQ_ERR_INVALID_ARG;
    if (lse != nullptr && !ok_ints(lse)) return KVQ_ERR_INVALID_ARG;
    if (!(scale <= 2.0e38f)) return KVQ_ERR_INVALID_ARG;  // infinite or NaN, or times log2 e infinite
    if (rows == 0 || batch->n_seqs == 0) return KVQ_OK;
    if (overlap(q, out, rows, q_heads, d, true)) return KVQ_ERR_INVALID_ARG;
    const size_t need = kvq_pages_attention_workspace_bytes(cfg, pages, batch, rows, q_heads);
    if (!ok_ptr(ws) || ws_bytes < need) return KVQ_ERR_WORKSPACE;
    const int sms = sm_count();
    const bool had = cfg->flags == KVQ_HADAMARD;
    const AttnPlan p = attn_plan(batch, rows, q_heads / pages->kv_heads);
    const AttnWorkspace w = attn_workspace(p, sms, d, had, q_heads, batch->n_seqs);
    uint8_t* base = static_cast<uint8_t*>(ws);
    StepArgs g;
    AttnArgs& a = g.a;
    a.b = batch_of(batch);
    a.p = pool_of(pages);
    a.q = q->data;
    a.out = out->data;
    a.lse = lse;
    a.q_row = rows > 1 ? q->row_stride : 0;
    a.q_head = q_heads > 1 ? q->head_stride : 0;
    a.o_row = rows > 1 ? out->row_stride : 0;
    a.o_head = q_heads > 1 ? out->head_stride : 0;
    a.signs = cfg->signs;
    a.rows = (int)rows;
    a.Hq = q_heads;
    a.G = q_heads / pages->kv_heads;
    a.bf16 = q->dtype == KVQ_BF16;
    a.causal = causal != 0;
    a.window = window;
    a.scale2 = (scale > 0.0f ? scale : rsqd_of(d)) * 1.4426950408889634f;
    a.rsqd = rsqd_of(d);
    a.meta = reinterpret_cast<int4*>(base + w.meta);
    a.ml = reinterpret_cast<float*>(base + w.ml);
    a.part = reinterpret_cast<float*>(base + w.part);
    a.left = reinterpret_cast<float*>(base + w.left);
    g.many = p.tiles ? kFewBeside : 0;
    g.stretch = p.stretch;
    g.whole = 0;
    g.frag = reinterpret_cast<__half*>(base + w.frag);
    g.scal = reinterpret_cast<float*>(base + w.scal);
    TileArgs t;
    t.a = a;
    t.a.meta = reinterpret_cast<int4*>(base + w.tile_meta);
    t.a.ml = reinterpret_cast<float*>(base + w.tile_ml);
    t.a.part = reinterpret_cast<float*>(base + w.tile_part);
    t.many = kFewBeside;
    t.plan = reinterpret_cast<int4*>(base + w.plan);
    t.seq_cost = reinterpret_cast<long long*>(base + w.seq_cost);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (d == 64) return had ? launch_attn<64, true>(g, t, p, sms, st) : launch_attn<64, false>(g, t, p, sms, st);
    return had ? launch_attn<128, true>(g, t, p, sms, st) : launch_attn<128, false>(g, t, p, sms, st);
}

kvq_status kvq_pages_read_errors(uint32_t* host_out, int32_t clear) {
    if (host_out == nullptr) return KVQ_ERR_INVALID_ARG;
    return read_error_word(host_out, clear != 0) ? KVQ_OK : KVQ_ERR_CUDA;
}

#ifdef KVQ_WAIT_TEST
// Test build only: scale of the poll limits of the paged kernels' waits (0: give up at once).
int kvq_test_set_pages_wait_scale(uint32_t scale) {
    return cudaMemcpyToSymbol(g_wait_scale, &scale, sizeof(scale)) == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}
#endif

}  // extern "C"
