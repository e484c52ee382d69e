// Attention of drafted token trees over the paged K/V caches, on the
// 5th-generation tensor cores (tcgen05).
//
//   out[t,h] = sum_s softmax_s(sm q[t,h].K[s]) V[s],  s in prefix, ancestors, self
//
// Every drafted token of a sequence reads the same prefix, so the tokens times the
// query heads of one K/V head are the rows of one product: tiles of 128 rows (the
// UMMA M), two at a time where there are more than 128, against blocks of 128 cache
// rows.  With few rows (n H_q / H_kv below about 130 for bf16) the cache's bytes bound
// the kernel, with many the tensor pipe and the exponentials, which take as long: 128 x 128
// exponentials at 16 a clock are 1024 clocks, the two products of a block at head
// dim 128 also 1024.
//
// The work of a launch is one list: sequence by sequence, K/V head by head, pair of
// row tiles by pair, its blocks of cache rows, each at the cost that was measured for
// it.  Each CTA (one per SM) takes an equal share of the list, wherever it begins and
// ends: no length or batch leaves SMs idle, and a single long sequence spreads over all
// of them.  An item (row tiles of one sequence and head) that is cut leaves partial
// results (fp32 O / l and log-sum-exp), which a second, chained kernel merges; the
// others are written at once.
//
// Roles of a CTA, bf16:
//   warp 0  brings Q and the K and V tiles by TMA through the page table, one box
//           of gcd(page_size, 128) rows a page, into a ring of 32 KB slots; boxes behind the
//           context (and pages out of range) start behind the cache's last row, which
//           TMA fills with zeros;
//   warp 1  issues S_x = Q_x K^T into TMEM, x = 0, 1, 64 cache rows at a time;
//   warp 2  issues O_x += P_x V, P_x from TMEM;
//   warp 3  walks the list of work, and the tree of each sequence: each token's ancestors
//           as 128 bits;
//   warps 4-7 and 8-11 are softmax sets, a thread a row: set x takes tile x of a pair
//           (both halves of each block) or half x of each block of a single tile (merged at
//           the end).  Each set has two score buffers in TMEM, so that the next scores
//           are made while it works; P takes the place of S.  O is rescaled only where the
//           maximum grows by more than 2^8, which is exact up to rounding.
// With FP8 caches warp 0 brings codes, and eight more warps (12-15: K, 16-19: V) widen
// them to bf16, exactly, into the ring; the scales stay in fp32 and multiply the logits
// and the weights.
// Every wait of one role for another is on an mbarrier and bounded (DSA_ERR_TIMEOUT on expiry):
// roles leave their loops one by one then, so a wait for all threads stands only behind the loops.
//
// Measured on one B200 (6.55 TB/s and 1.40 PFLOP/s sustained), over a second of calls and "at first", in the
// milliseconds before the power limit takes the SM clock down from 1.97 GHz to what is given here.
// 16 x 64K contexts, 8-16 drafts, 128 heads on one K/V head: 0.65 ms at 1.5 GHz (0.89 PFLOP/s, 63 % of the
// sustained rate), 0.55 ms at first (half of the exponentials on the FMA pipe took 15 % fewer clocks but more power,
// and so more time).  64 x 32K, one draft, pages of 64 or 128 rows: 164 us (4.85 TB/s, 74 %), 147 at first; with
// pages of 16 rows, whose boxes are 2 KB, 204 and 185.  FP8 64 x 32K x 2-3 drafts: 0.36 ms at 1.80 GHz, 0.33 at
// first, bound by the widening and by shared memory, which the products, the widening and the scales share.  The
// code of the hot roles has to fit the instruction cache: one copy of each product's code instead of four took the
// FP8 kernel from 450 to 358 us (these and the next at first).  128-row steps over one score buffer: bf16 585, FP8
// 432 us.
#include <algorithm>
#include <atomic>
#include <limits>
#include <numeric>

#include <cuda_fp8.h>

#include "kernels.h"
#include "sm100.cuh"

namespace dsa {
namespace {

using namespace sm100;

constexpr int TA_M = 128;              // rows of a tile
constexpr int TA_BLK = 128;            // cache rows of a block
constexpr int TA_MAX_CTAS = 160;       // CTAs a workspace has room for (148 SMs)
constexpr int TA_SEGS = 4;             // segments in the ring
constexpr int TA_HALF = 64;            // cache rows of a step of a softmax set
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNaN = std::numeric_limits<float>::quiet_NaN();
constexpr float kRescaleThreshold = 8.f;   // log2 units
// A padding row's log2 sum in the workspace.  No other row has it: an infinite logit makes the sum a NaN.
constexpr float kPadding = INFINITY;

// Register splits: they add up to the launch's registers only for kernels built with
// exactly these counts (checked by the build and before every launch).
constexpr int TA_THREADS = 384, TA_REGS = 168, TA_REGS_LOW = 96, TA_REGS_HIGH = 200;
constexpr int TA8_THREADS = 640, TA8_REGS = 96, TA8_REGS_LOW = 56, TA8_REGS_HIGH = 152;
static_assert(128 * TA_REGS_LOW + 256 * TA_REGS_HIGH <= TA_THREADS * TA_REGS, "register split");
static_assert(384 * TA8_REGS_LOW + 256 * TA8_REGS_HIGH <= TA8_THREADS * TA8_REGS, "register split");

struct TreeArgs {
    const uint16_t *q;
    const int32_t *block_table, *context_lens, *token_start, *parents;
    const float *ks, *vs;              // KV8: scales
    int64_t num_pages, N, max_context;
    int max_pages, page_size, box;     // box: cache rows of one TMA box
    int B, max_tree, H, Hkv;
    int group;                         // query heads of a K/V head
    int rows_tok;                      // rows of a tile that one token takes: min(group, 128)
    int tile_tok;                      // tokens of a tile (1 when group > 128)
    int head_tiles;                    // tiles of one token (1 when group <= 128)
    int cost_pair, cost_one;           // of a block of cache rows for a pair of tiles and for a single one
    uint32_t stall_at;                 // test hook: CTA 0 stops before its K or V tile stall_at (~0: off)
    float scale_log2;
    uint16_t *out;
    float *lse;
    int4 *desc;                        // [CTAs] first item of each CTA: sequence, head, tile, bits (1: cut, 2: pair)
    uint32_t *err;                     // [CTAs] dsa_status
    float *part;                       // [2 CTAs][d / 4][256][4] O / l: slot, columns, row
    float *part_lse;                   // [2 CTAs][256] log2 sum, kPadding for a padding row
    WsHeader *hdr;
};

// Shared memory (byte offsets; the dynamic block starts on a 1024-byte boundary).
template <bool KV8, int D> struct Smem {
    static constexpr int halves = D / 64;
    static constexpr int half = 128 * 128;                     // 64 columns of 128 rows
    static constexpr int tile = halves * half;                 // one bf16 tile
    static constexpr int slots = KV8 ? (D == 128 ? 3 : 4) : (D == 128 ? 5 : 10);
    static constexpr int codes = KV8 ? (D == 128 ? 3 : 6) : 0; // KV8: staged E4M3 tiles
    static constexpr int code_tile = 128 * D;
    static constexpr int q_off = 0;                            // two tiles
    // The (m, l) of both sets lie in Q's second tile, which a single tile leaves free; the
    // next pair's Q waits until they are read.
    static constexpr int ml_off = q_off + tile;                // [item % 2][set][m, l][128]
    static constexpr int kv_off = q_off + 2 * tile;
    static constexpr int code_off = kv_off + slots * tile;
    static constexpr int scale_off = code_off + codes * code_tile;       // KV8: [block % 4][K, V][128]
    static constexpr int mask_off = scale_off + (KV8 ? 4 * 2 * 128 * 4 : 0);
    static constexpr int parent_off = mask_off + DSA_MAX_TREE * 16;
    static constexpr int seg_off = parent_off + DSA_MAX_TREE * 2;        // ring of segments
    static constexpr int bar_off = seg_off + TA_SEGS * 48;
    static constexpr int n_bars = 2 + 2 * slots + 12 + 5 + 2 * TA_SEGS + 2 * codes;
    static constexpr int ctl_off = bar_off + 8 * n_bars;
    static constexpr int total = ctl_off + 256;
};
static_assert(Smem<false, 128>::total <= 232448 && Smem<false, 64>::total <= 232448, "shared memory of a CTA");
static_assert(Smem<true, 128>::total <= 232448 && Smem<true, 64>::total <= 232448, "shared memory of a CTA");

// Control words of a CTA.
struct Ctl {
    uint32_t tmem;
    volatile int abort;
    int err;                           // dsa_status
    int start_b;                       // sequence of the CTA's first unit of work, -1: none
    long long start_base;              // work before that sequence
    long long c0, c1;                  // the CTA's share of the work
    int kv_issued, q_issued, code_issued, s_issued[2], pv_issued[2];
    long long sums[20];
};
static_assert(sizeof(Ctl) <= 256, "control words");

__device__ __forceinline__ bool wait_or_abort(uint64_t *bar, uint32_t parity, volatile int *abort)
{
    uint64_t t0 = 0;
#pragma unroll 1
    for (uint32_t i = 1; !mbar_try_wait(bar, parity); ++i) {
        if (i & 255) continue;         // reading the timer takes longer than most waits
        const uint64_t t = globaltimer_ns();
        if (t0 == 0) t0 = t;
        if (*abort) return false;
        if (t - t0 > kWaitLimitNs) {
            *abort = 1;
            return false;
        }
    }
    return true;
}

// 2^x by the SFU (2 ulp; results below 2^-126 flush to zero, which a sum that holds a term near 1 does not notice).
__device__ __forceinline__ float ex2_sfu(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two fp32 values in registers times two others.
__device__ __forceinline__ void f2_scale(uint32_t &a, uint32_t &b, float fa, float fb)
{
    float x, y;
    f2_unpack(f2_mul(f2_pack(__uint_as_float(a), __uint_as_float(b)), f2_pack(fa, fb)), x, y);
    a = __float_as_uint(x);
    b = __float_as_uint(y);
}

// The largest of three (sm_100's three-operand form).
__device__ __forceinline__ float max3(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// Sixteen E4M3 codes as eight bf16 pairs, exactly.
__device__ __forceinline__ void e4m3x16_to_bf16(const uint4 &raw, uint32_t (&out)[8])
{
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const __nv_fp8x2_storage_t two = (__nv_fp8x2_storage_t)((w[i >> 1] >> (16 * (i & 1))) & 0xffffu);
        const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2(two, __NV_E4M3);
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&hr));
        out[i] = pack_bf16x2(f.x, f.y);
    }
}

// A sequence's tokens and context.  Returns its row tiles per K/V head x blocks of cache
// rows (0: nothing to do), and reports what it may not be.
struct Seq {
    int n, ctx, tok0, tiles, nblk;
    __device__ __forceinline__ int64_t load(const TreeArgs &a, int b, bool &bad)
    {
        const int64_t t0 = a.token_start[b], t1 = a.token_start[b + 1];
        const int64_t c = a.context_lens[b], m = t1 - t0;
        bad = false;
        n = 0;
        if (m == 0) return 0;
        const int64_t room = min(a.max_context, (int64_t)a.max_pages * a.page_size);
        if (t0 < 0 || m < 0 || t1 > a.N || m > a.max_tree || c < m || c > room) {
            bad = true;
            return 0;
        }
        n = (int)m;
        ctx = (int)c;
        tok0 = (int)t0;
        tiles = a.head_tiles > 1 ? n * a.head_tiles : (n + a.tile_tok - 1) / a.tile_tok;
        nblk = (ctx + TA_BLK - 1) / TA_BLK;
        return (int64_t)((tiles >> 1) * a.cost_pair + (tiles & 1) * a.cost_one) * nblk;
    }
};

// The CTA's part of one item: blocks [blk0, blk1) for row tile `tile` (and the next, if `pair`).
struct alignas(16) Segment {
    int b, hk, tile, blk0;             // b: sequence, -1: no more
    int blk1, pair, n, ctx;            // n, ctx, tok0, nblk: the sequence's tokens, context, first token, blocks
    int tok0, nblk, pad0, pad1;
};

// Walks the CTA's share [c0, c1) of the list of work.  One warp does, and leaves the
// segments in a ring in shared memory for the others (the walk's code in every role would not fit the
// instruction cache).
struct Walker {
    const TreeArgs &a;
    int64_t c0, c1, item;              // item: work before the current item
    Seq s;
    int b, hk, rg;                     // rg: pair of row tiles
    __device__ __forceinline__ Walker(const TreeArgs &args, const Ctl *ctl) : a(args)
    {
        c0 = ctl->c0;
        c1 = ctl->c1;
        b = ctl->start_b;
        item = ctl->start_base;
        hk = rg = 0;
        if (b < 0) {
            b = a.B;
            return;
        }
        bool bad;
        const int64_t per_head = s.load(a, b, bad);    // work of a K/V head
        const int64_t rel = c0 - item;
        hk = (int)(rel / per_head);
        item += hk * per_head;
        const int64_t per_pair = (int64_t)a.cost_pair * s.nblk;
        rg = (int)min((rel - hk * per_head) / per_pair, (int64_t)(s.tiles - 1) / 2);
        item += rg * per_pair;
    }
    __device__ __forceinline__ bool next(Segment &g)
    {
        while (true) {
            if (b >= a.B || item >= c1) return false;
            if (s.n == 0 || hk == a.Hkv) {
                // The next sequence with tokens: 32 at a time (a call over 60 000 idle ones 4.0 ms one at a time, 0.3 so).
                for (++b;; b += 32) {
                    if (b >= a.B) return false;
                    const int c = b + (int)(threadIdx.x & 31);
                    const unsigned any = __ballot_sync(0xffffffffu, c < a.B && a.token_start[c] != a.token_start[c + 1]);
                    if (any) {
                        b += __ffs(any) - 1;
                        break;
                    }
                }
                bool bad;
                s.load(a, b, bad);
                hk = rg = 0;
                continue;
            }
            const bool pair = 2 * rg + 1 < s.tiles;
            const int w = pair ? a.cost_pair : a.cost_one;
            const int64_t cost = (int64_t)w * s.nblk;
            const int64_t lo = max(c0 - item, (int64_t)0), hi = min(c1 - item, cost);
            g.b = b;
            g.n = s.n;
            g.ctx = s.ctx;
            g.tok0 = s.tok0;
            g.nblk = s.nblk;
            g.hk = hk;
            g.tile = 2 * rg;
            g.pair = pair;
            g.blk0 = (int)((lo + w - 1) / w);
            g.blk1 = (int)((hi + w - 1) / w);
            item += cost;
            if (2 * ++rg >= s.tiles) {
                rg = 0;
                ++hk;
            }
            if (g.blk0 < g.blk1) return true;
        }
    }
};

// Cache row of position p, or the row behind the last one (TMA fills it with zeros).
__device__ __forceinline__ int cache_row(const TreeArgs &a, int b, int ctx, int p, Ctl *ctl)
{
    const int64_t rows = a.num_pages * a.page_size;
    if (p >= ctx) return (int)rows;
    const int page = a.block_table[(int64_t)b * a.max_pages + p / a.page_size];
    if (page < 0 || page >= a.num_pages) {
        ctl->err = DSA_ERR_INVALID_ARG;
        return (int)rows;
    }
    return page * a.page_size + p % a.page_size;
}

template <bool KV8, int D>
__device__ __forceinline__ void tree_attn_body(const CUtensorMap &qmap, const CUtensorMap &kmap,
                                               const CUtensorMap &vmap, const TreeArgs &a)
{
    using S = Smem<KV8, D>;
    constexpr int SLOTS = S::slots, CODES = KV8 ? S::codes : 1;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + S::bar_off);
    uint64_t *qfull = bars, *qempty = bars + 1, *kvfull = bars + 2, *kvempty = kvfull + SLOTS;
    uint64_t *sfull = kvempty + SLOTS, *pfull = sfull + 4, *pvdone = pfull + 4, *oempty = pvdone + 4;   // [set][buffer]
    uint64_t *mfull = oempty + 2, *mempty = mfull + 1, *mlfull = mempty + 1, *gfull = mlfull + 1, *gempty = gfull + TA_SEGS;
    uint64_t *cfull = gempty + TA_SEGS, *cempty = cfull + CODES;
    Ctl *ctl = reinterpret_cast<Ctl *>(smem + S::ctl_off);
    uint32_t *masks = reinterpret_cast<uint32_t *>(smem + S::mask_off);
    int16_t *par = reinterpret_cast<int16_t *>(smem + S::parent_off);
    float *scales = reinterpret_cast<float *>(smem + S::scale_off);
    Segment *segs = reinterpret_cast<Segment *>(smem + S::seg_off);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int threads = blockDim.x;

    if (warp == 0) {
        tmem_alloc(&ctl->tmem, 512);
        tmem_relinquish();
    }
    if (tid == 32) {
        tma_prefetch_desc(&qmap);
        tma_prefetch_desc(&kmap);
        tma_prefetch_desc(&vmap);
    }
    if (tid == 0) {
        mbar_init(qfull, 1);
        mbar_init(qempty, 1);
        for (int i = 0; i < SLOTS; ++i) { mbar_init(&kvfull[i], KV8 ? 4 : 1); mbar_init(&kvempty[i], 1); }
        for (int i = 0; i < 4; ++i) { mbar_init(&sfull[i], 1); mbar_init(&pfull[i], 4); mbar_init(&pvdone[i], 1); }
        mbar_init(&oempty[0], 8);
        mbar_init(&oempty[1], 8);
        mbar_init(mfull, 1);
        mbar_init(mempty, 8);
        mbar_init(mlfull, 8);
        for (int i = 0; i < TA_SEGS; ++i) { mbar_init(&gfull[i], 1); mbar_init(&gempty[i], KV8 ? 19 : 11); }
        if (KV8)
            for (int i = 0; i < CODES; ++i) { mbar_init(&cfull[i], 1); mbar_init(&cempty[i], 4); }
        ctl->abort = 0;
        ctl->err = DSA_OK;
        ctl->start_b = -1;
        ctl->kv_issued = ctl->q_issued = ctl->code_issued = 0;
        ctl->s_issued[0] = ctl->s_issued[1] = ctl->pv_issued[0] = ctl->pv_issued[1] = 0;
        fence_mbar_init();
    }

    grid_dep_wait();                   // what came before on the stream

    // ---- the CTA's share of the work: a sum over the sequences, then a search
    int64_t all = 0, mine = 0;
    bool any_bad = false;
#pragma unroll 1
    for (int b = tid; b < a.B; b += threads) {
        Seq s;
        bool bad;
        const int64_t c = s.load(a, b, bad) * a.Hkv;
        if (b == tid) mine = c;
        all += c;
        any_bad |= bad;
    }
    {
        int64_t v = all;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (lane == 0) ctl->sums[warp] = v;
    }
    __syncthreads();
    all = 0;
    for (int w = 0; w < threads / 32; ++w) all += ctl->sums[w];
    // at least two blocks a CTA: shorter shares cost more to merge than they save
    const int64_t ctas = min((int64_t)gridDim.x, max((int64_t)1, all / (2 * a.cost_one)));
    const bool works = (int64_t)blockIdx.x < ctas && all > 0;
    const int64_t c0 = works ? all * blockIdx.x / ctas : 0, c1 = works ? all * (blockIdx.x + 1) / ctas : 0;
    if (blockIdx.x == 0 && any_bad) ctl->err = DSA_ERR_INVALID_ARG;
    int64_t before = 0;
#pragma unroll 1
    for (int b0 = 0; b0 < a.B && works; b0 += threads) {
        const int b = b0 + tid;
        int64_t c = mine;
        if (b0 > 0) {
            Seq s;
            bool bad;
            c = b < a.B ? s.load(a, b, bad) * a.Hkv : 0;
        }
        int64_t v = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t t = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += t;
        }
        __syncthreads();
        if (lane == 31) ctl->sums[warp] = v;
        __syncthreads();
        int64_t total = 0;
        for (int w = 0; w < threads / 32; ++w) {
            if (w < warp) v += ctl->sums[w];
            total += ctl->sums[w];
        }
        const int64_t base = before + v - c;
        if (c > 0 && base <= c0 && c0 < base + c) {
            ctl->start_b = b;
            ctl->start_base = base;
        }
        before += total;
        if (before > c0) break;        // the same in every thread
    }
    if (tid == 0) {
        ctl->c0 = c0;
        ctl->c1 = c1;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctl->tmem;
    const uint32_t tS = tmem, tO = tmem + 256;     // S_x (and P_x in its first 64 columns), O_x

    // The next segment of the ring (whole warps); false: there is none, or a wait ran out.
    uint32_t seg_i = 0;
    auto next = [&](Segment &g) -> bool {
        const uint32_t st = seg_i % TA_SEGS;
        if (!__all_sync(0xffffffffu, wait_or_abort(&gfull[st], (seg_i / TA_SEGS) & 1, &ctl->abort))) return false;
        g = segs[st];
        __syncwarp();
        if (lane == 0) mbar_arrive(&gempty[st]);
        ++seg_i;
        return g.b >= 0;
    };

    if (warp < 4 || warp >= 12) {
        regs_dec<KV8 ? TA8_REGS_LOW : TA_REGS_LOW>();
        if (warp == 0) {
            // ------------------------------------------------ Q, K and V by TMA
            Segment g;
            const int nbox = TA_BLK / a.box;
            const int halves = KV8 ? 1 : S::halves;
            const int box = lane % nbox, half = lane / nbox;
            const bool loads = half < halves;
            uint32_t t = 0;                        // tiles issued
            int item = 0;
            bool was_single = false, ok = true;
            const uint32_t stall_at = blockIdx.x == 0 ? a.stall_at : ~0u;
            for (; ok && next(g); ++item) {
                int row = cache_row(a, g.b, g.ctx, g.blk0 * TA_BLK + box * a.box, ctl);
                if (lane == 0) {
                    ok = wait_or_abort(qempty, (item & 1) ^ 1, &ctl->abort);
                    // the last item's end only where its (m, l) lie in the second tile's place; the one before
                    // it always, so that no end goes by unseen (a parity tells two phases apart, not three)
                    if (ok && item >= 2) ok = wait_or_abort(&oempty[item & 1], ((item >> 1) & 1) ^ 1, &ctl->abort);
                    if (ok && g.pair && was_single)
                        ok = wait_or_abort(&oempty[(item - 1) & 1], ((item - 1) >> 1) & 1, &ctl->abort);
                    if (ok) {
                        const int tiles = g.pair ? 2 : 1;
                        const int bytes = a.tile_tok * a.rows_tok * 128 * S::halves;
                        mbar_arrive_expect_tx(qfull, tiles * bytes);
                        ctl->q_issued = item + 1;
                        for (int x = 0; x < tiles; ++x) {
                            const int tl = g.tile + x;
                            const int tok = a.head_tiles > 1 ? tl / a.head_tiles : tl * a.tile_tok;
                            const int head = a.head_tiles > 1 ? (tl % a.head_tiles) * TA_M : 0;
                            for (int h = 0; h < S::halves; ++h)
                                tma_load_4d(smem + S::q_off + x * S::tile + h * S::half, &qmap, qfull, h * 64, head, g.hk,
                                            g.tok0 + tok);
                        }
                    }
                }
                ok = __shfl_sync(0xffffffffu, ok, 0);
                was_single = !g.pair;
                for (int blk = g.blk0; ok && blk < g.blk1; ++blk) {
                    const int here = row;
                    if (blk + 1 < g.blk1) row = cache_row(a, g.b, g.ctx, (blk + 1) * TA_BLK + box * a.box, ctl);
                    for (int kv = 0; kv < 2 && ok; ++kv, ++t) {
                        const int st = KV8 ? t % CODES : t % SLOTS;
                        const uint32_t ph = KV8 ? t / CODES : t / SLOTS;
                        ok = wait_or_abort(KV8 ? &cempty[st] : &kvempty[st], (ph & 1) ^ 1, &ctl->abort);
                        ok = __all_sync(0xffffffffu, ok);
                        if (t == stall_at) ok = false;         // test hook: leave the copies unissued
                        if (!ok) break;
                        uint64_t *full = KV8 ? &cfull[st] : &kvfull[st];
                        if (lane == 0) {
                            mbar_arrive_expect_tx(full, KV8 ? S::code_tile : S::tile);
                            if (KV8) ctl->code_issued = (int)t + 1; else ctl->kv_issued = (int)t + 1;
                        }
                        __syncwarp();
                        if (loads) {
                            uint8_t *dst = KV8 ? smem + S::code_off + st * S::code_tile + box * a.box * D
                                               : smem + S::kv_off + st * S::tile + half * S::half + box * a.box * 128;
                            tma_load_3d(dst, kv ? &vmap : &kmap, full, half * 64, g.hk, here);
                        }
                    }
                }
            }
        } else if (warp == 1) {
            // ------------------------------------------------ S_x = Q_x K^T
            // (the whole warp keeps step, so that addresses stay in uniform registers; one lane issues)
            constexpr uint32_t idesc = umma_idesc_bf16_f32(TA_M, TA_HALF, false);
            constexpr uint64_t upper = TA_HALF * 128 >> 4;     // the second half's rows of a tile
            const uint64_t qd0 = umma_desc_k_sw128(smem_u32(smem + S::q_off));
            const uint64_t kd0 = umma_desc_k_sw128(smem_u32(smem + S::kv_off));
            Segment g;
            uint32_t st = 0, ph = 0, cnt = 0;          // slot and its phase; steps of each set
            int item = 0;
            bool ok = true;
            auto product = [&](int x, uint32_t k, uint64_t qd, uint64_t kd) {
                const uint32_t buf = k & 1;
                // P lies in S: the P V of two steps ago must have read it
                ok = __all_sync(0xffffffffu, ok && wait_or_abort(&pvdone[2 * x + buf], ((k >> 1) & 1) ^ 1, &ctl->abort));
                if (!ok) return;
                tc_fence_after();
                if (elect_sync()) {
                    const uint32_t d = tS + x * 128 + buf * TA_HALF;
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        constexpr int h = S::half >> 4;
                        umma_f16(d, qd + (kk >> 2) * h + (kk & 3) * 2, kd + (kk >> 2) * h + (kk & 3) * 2, idesc,
                                 kk > 0 ? 1u : 0u);
                    }
                    umma_commit(&sfull[2 * x + buf]);
                    ctl->s_issued[x] = (int)k + 1;
                }
                __syncwarp();
            };
            for (; ok && next(g); ++item) {
                ok = __all_sync(0xffffffffu, wait_or_abort(qfull, item & 1, &ctl->abort));
                for (int blk = g.blk0; ok && blk < g.blk1; ++blk) {
                    ok = __all_sync(0xffffffffu, wait_or_abort(&kvfull[st], ph, &ctl->abort));
                    const uint64_t kd = kd0 + (uint64_t)(st * (S::tile >> 4));
                    // a pair: both tiles by each half of the rows; a single tile: its set for each half
#pragma unroll 1
                    for (int u = 0; u < (g.pair ? 4 : 2); ++u) {
                        const int x = u & 1, h = g.pair ? u >> 1 : u;
                        product(x, cnt + (g.pair ? h : 0), qd0 + (g.pair && x ? S::tile >> 4 : 0), kd + (h ? upper : 0));
                    }
                    cnt += g.pair ? 2 : 1;
                    if (ok && elect_sync()) umma_commit(&kvempty[st]);
                    __syncwarp();
                    st += 2;
                    if (st >= SLOTS) { st -= SLOTS; ph ^= 1; }
                }
                if (ok && elect_sync()) umma_commit(qempty);
                __syncwarp();
            }
        } else if (warp == 2) {
            // ------------------------------------------------ O_x += P_x V
            constexpr uint32_t idesc = umma_idesc_bf16_f32(TA_M, D, true);
            const uint64_t vd0 = umma_desc_mn_sw128(smem_u32(smem + S::kv_off), S::half, 1024);
            Segment g;
            uint32_t st = 1, ph = 0, cnt = 0;
            int item = 0;
            bool ok = true;
            constexpr uint64_t upper = TA_HALF * 128 >> 4;
            auto product = [&](int x, uint32_t k, uint64_t vd, bool first) {
                const uint32_t buf = k & 1;
                ok = __all_sync(0xffffffffu, ok && wait_or_abort(&pfull[2 * x + buf], (k >> 1) & 1, &ctl->abort));
                if (!ok) return;
                tc_fence_after();
                if (elect_sync()) {
                    const uint32_t pa = tS + x * 128 + buf * TA_HALF;
#pragma unroll
                    for (int kk = 0; kk < TA_HALF / 16; ++kk)
                        umma_f16_ts(tO + x * 128, pa + kk * 8, vd + kk * 128, idesc, (first && kk == 0) ? 0u : 1u);
                    umma_commit(&pvdone[2 * x + buf]);
                    ctl->pv_issued[x] = (int)k + 1;
                }
                __syncwarp();
            };
            for (; ok && next(g); ++item) {
                // the item before has read its O
                if (item > 0)
                    ok = __all_sync(0xffffffffu, wait_or_abort(&oempty[(item - 1) & 1], ((item - 1) >> 1) & 1, &ctl->abort));
                for (int blk = g.blk0; ok && blk < g.blk1; ++blk) {
                    ok = __all_sync(0xffffffffu, wait_or_abort(&kvfull[st], ph, &ctl->abort));
                    const uint64_t vd = vd0 + (uint64_t)(st * (S::tile >> 4));
                    const bool first = blk == g.blk0;
#pragma unroll 1
                    for (int u = 0; u < (g.pair ? 4 : 2); ++u) {
                        const int x = u & 1, h = g.pair ? u >> 1 : u;
                        product(x, cnt + (g.pair ? h : 0), vd + (h ? upper : 0), first && u < 2);
                    }
                    cnt += g.pair ? 2 : 1;
                    if (ok && elect_sync()) umma_commit(&kvempty[st]);
                    __syncwarp();
                    st += 2;
                    if (st >= SLOTS) { st -= SLOTS; ph ^= 1; }
                }
            }
        } else if (warp == 3) {
            // ------------------------------------------------ segments, and each token's ancestors
            // Bit j of token i: j is i or above it.  0 for a padding row (and under one).
            Walker w(a, ctl);
            Segment g;
            int cur = -1, seq = 0;
            bool ok = true;
            while (ok) {
                const bool more = w.next(g);
                const uint32_t st = seg_i % TA_SEGS;
                ok = __all_sync(0xffffffffu, wait_or_abort(&gempty[st], ((seg_i / TA_SEGS) & 1) ^ 1, &ctl->abort));
                if (!ok) break;
                if (!more) g.b = -1;
                if (lane == 0) {
                    if (seg_i == 0)
                        a.desc[blockIdx.x] = make_int4(g.b, g.hk, g.tile, (g.blk0 > 0 ? 1 : 0) | (g.pair ? 2 : 0));
                    segs[st] = g;
                    mbar_arrive(&gfull[st]);
                }
                __syncwarp();
                ++seg_i;
                if (!more) break;
                if (g.b == cur) continue;
                cur = g.b;
                const Segment &s = g;
                int p[DSA_MAX_TREE / 32];
#pragma unroll
                for (int j = 0; j < DSA_MAX_TREE / 32; ++j) {
                    const int i = j * 32 + lane;
                    p[j] = i < s.n ? a.parents[s.tok0 + i] : -2;
                    if (i < s.n && p[j] >= i) {
                        p[j] = -2;
                        ctl->err = DSA_ERR_INVALID_ARG;
                    }
                    p[j] = max(p[j], -2);
                }
                ok = __all_sync(0xffffffffu, wait_or_abort(mempty, (seq & 1) ^ 1, &ctl->abort));
                if (!ok) break;
#pragma unroll
                for (int j = 0; j < DSA_MAX_TREE / 32; ++j) par[j * 32 + lane] = (int16_t)p[j];
                __syncwarp();
                for (int i = lane; i < s.n; i += 32) {
                    uint32_t m[4] = {0u, 0u, 0u, 0u};
                    int j = par[i] == -2 ? -2 : i;
                    while (j >= 0) {               // parents come before their children: at most i steps
                        m[0] |= j < 32 ? 1u << j : 0u;
                        m[1] |= (j >> 5) == 1 ? 1u << (j & 31) : 0u;
                        m[2] |= (j >> 5) == 2 ? 1u << (j & 31) : 0u;
                        m[3] |= (j >> 5) == 3 ? 1u << (j & 31) : 0u;
                        j = par[j];
                    }
                    if (j == -2) m[0] = m[1] = m[2] = m[3] = 0u;
                    *reinterpret_cast<uint4 *>(masks + 4 * i) = make_uint4(m[0], m[1], m[2], m[3]);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(mfull);
                ++seq;
            }
        } else if (KV8) {
            // ------------------------------------------------ E4M3 -> bf16 (warps 12-15: K, 16-19: V)
            // Every E4M3 value is a bf16 value.  Thread i of the V warps brings the two scales of
            // row i of a block, a block ahead (their addresses go through the page table).
            const int ct = tid & 127, kv = (warp >> 2) - 3;
            Segment g;
            uint32_t t = kv, i = 0;
            bool ok = true;
            while (ok && next(g)) {
                const int none = (int)(a.num_pages * a.page_size);
                auto row_of = [&](int blk) {
                    return kv && blk < g.blk1 ? cache_row(a, g.b, g.ctx, blk * TA_BLK + ct, ctl) : none;
                };
                auto scale_of = [&](const float *p, int r) { return r < none ? p[(int64_t)r * a.Hkv + g.hk] : 0.f; };
                int r1 = row_of(g.blk0);
                float ksc = scale_of(a.ks, r1), vsc = scale_of(a.vs, r1);
                r1 = row_of(g.blk0 + 1);
#pragma unroll 1
                for (int blk = g.blk0; blk < g.blk1; ++blk, ++i, t += 2) {
                    const float k_now = ksc, v_now = vsc;
                    ksc = scale_of(a.ks, r1);
                    vsc = scale_of(a.vs, r1);
                    r1 = row_of(blk + 2);
                    const uint32_t cs = t % CODES, st = t % SLOTS;
                    ok = wait_or_abort(&cfull[cs], (t / CODES) & 1, &ctl->abort) &&
                         wait_or_abort(&kvempty[st], ((t / SLOTS) & 1) ^ 1, &ctl->abort);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    if (kv) {
                        scales[(i & 3) * 256 + ct] = k_now;
                        scales[(i & 3) * 256 + 128 + ct] = v_now;
                    }
                    const uint8_t *src = smem + S::code_off + cs * S::code_tile;
                    uint8_t *dst = smem + S::kv_off + st * S::tile;
#pragma unroll 1
                    for (int j0 = 0; j0 < D / 16; j0 += 2) {
                        // reads before writes: the compiler cannot know that they are apart
                        uint4 raw[2];
#pragma unroll
                        for (int j = 0; j < 2; ++j) raw[j] = *reinterpret_cast<const uint4 *>(src + ((ct + 128 * (j0 + j)) << 4));
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const int q = ct + 128 * (j0 + j), row = q / (D / 16), c = q % (D / 16);
                            // rows behind the context count as zeros, whatever they hold
                            if (blk * TA_BLK + row >= g.ctx) raw[j] = make_uint4(0u, 0u, 0u, 0u);
                            uint32_t o[8];
                            e4m3x16_to_bf16(raw[j], o);
                            uint8_t *p = dst + (c >> 2) * S::half + row * 128;
                            const int c0 = (c & 3) * 2;
                            // the two halves of a row start on the same banks: the upper one's threads
                            // write their chunks in the other order
                            const int f = c >> 2;
                            const uint4 lo = make_uint4(o[0], o[1], o[2], o[3]), hi = make_uint4(o[4], o[5], o[6], o[7]);
                            *reinterpret_cast<uint4 *>(p + (((c0 + f) ^ (row & 7)) << 4)) = f ? hi : lo;
                            *reinterpret_cast<uint4 *>(p + (((c0 + 1 - f) ^ (row & 7)) << 4)) = f ? lo : hi;
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&kvfull[st]);
                        mbar_arrive(&cempty[cs]);
                    }
                }
            }
        }
    } else {
        regs_inc<KV8 ? TA8_REGS_HIGH : TA_REGS_HIGH>();
        // ------------------------------------------------ softmax sets
        const int x = (warp >> 2) - 1;             // warps 4-7: set 0, 8-11: set 1
        const int r = tid & 127;                   // row of the tile
        const uint32_t trow = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tSx = tS + x * 128 + trow, tOx = tO + x * 128 + trow;
        const int tr = r / a.rows_tok, hr = r - tr * a.rows_tok;
        Segment g;
        uint32_t cnt = 0, i0 = 0;                  // steps of each set and blocks, before this segment
        uint32_t items = 0;                        // segments before this one
        uint32_t singles = 0;                      // items of a single tile before this one
        int cur = -1, seqs = 0;                    // sequence, and how many before it
        bool masked = false;                       // its masks are there
        bool dead = false;
        auto need_masks = [&]() {
            if (masked || dead) return;
            if (!__all_sync(0xffffffffu, wait_or_abort(mfull, seqs & 1, &ctl->abort))) dead = true;
            masked = true;
        };
        auto leave = [&]() {                       // the masks may be overwritten
            if (cur < 0) return;
            need_masks();
            __syncwarp();
            if (lane == 0) mbar_arrive(mempty);
            ++seqs;
            masked = false;
        };
        while (next(g)) {
            if (g.b != cur) {
                leave();
                cur = g.b;
            }
            const Segment &s = g;
            const int prefix = s.ctx - s.n;
            const int tile = g.tile + (g.pair ? x : 0);
            const int tok = (a.head_tiles > 1 ? tile / a.head_tiles : tile * a.tile_tok) + tr;
            const int head = (a.head_tiles > 1 ? (tile % a.head_tiles) * TA_M : 0) + hr;
            const bool valid = tr < a.tile_tok && tok < s.n && head < a.group;
            const int node = valid ? tok : 0;
            const int nb = g.blk1 - g.blk0;
            // a pair: both halves of every block; a single tile: the set's own half
            const int steps = g.pair ? 2 * nb : nb;
            float m = -INFINITY, l = 0.f;
            for (int t = 0; t < steps && !dead; ++t) {
                const uint32_t k = cnt + t, buf = k & 1;
                const int nth = g.pair ? t >> 1 : t, half = g.pair ? t & 1 : x;
                const int pos = (g.blk0 + nth) * TA_BLK + half * TA_HALF;      // the step's first position
                const uint32_t i = i0 + nth, tv = 2 * i + 1, stv = tv % SLOTS;
                const uint32_t tSb = tSx + buf * TA_HALF;
                bool ok = wait_or_abort(&sfull[2 * x + buf], (k >> 1) & 1, &ctl->abort);
                // V's tile (and the scales of K and V with it)
                const bool tail = pos + TA_HALF > s.ctx;
                if (KV8 || tail) ok = ok && wait_or_abort(&kvfull[stv], (tv / SLOTS) & 1, &ctl->abort);
                if (!__all_sync(0xffffffffu, ok)) { dead = true; break; }
                tc_fence_after();
                uint32_t v[2][32];
                tmem_ld32(tSb, v[0]);
                tmem_ld32(tSb + 32, v[1]);
                tmem_wait_ld_dep32(v[0]);
                tmem_wait_ld_dep32(v[1]);
                const float4 *sc = reinterpret_cast<const float4 *>(scales + (i & 3) * 256 + half * TA_HALF);
                if (KV8) {
#pragma unroll
                    for (int c = 0; c < 16; ++c) {
                        const float4 f = sc[c];
                        uint32_t *u = &v[c >> 3][(c & 7) * 4];
                        f2_scale(u[0], u[1], f.x, f.y);
                        f2_scale(u[2], u[3], f.z, f.w);
                    }
                }
                if (pos + TA_HALF > prefix) {
                    // the drafts (and what lies behind them): column c is draft j = pos + c - prefix
                    need_masks();
                    if (dead) break;
                    const uint32_t *mw = masks + 4 * node;
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const int j0 = pos + c * 32 - prefix;
                        uint32_t bits;
                        if (j0 <= -32) bits = 0xffffffffu;
                        else if (j0 < 0) bits = (mw[0] << -j0) | ((1u << -j0) - 1u);
                        else if (j0 >= DSA_MAX_TREE) bits = 0u;
                        else bits = __funnelshift_r(mw[j0 >> 5], j0 + 32 < DSA_MAX_TREE ? mw[(j0 >> 5) + 1] : 0u, j0 & 31);
#pragma unroll
                        for (int q = 0; q < 32; ++q)
                            if (!((bits >> q) & 1u)) v[c][q] = 0xff800000u;
                    }
                    if (!KV8 && tail) {
                        // V's rows behind the context, up to the end of their box, may hold anything:
                        // their weights are 0, but 0 times an infinity is not
                        const int ctx_row = s.ctx - (g.blk0 + nth) * TA_BLK;
                        const int lo = max(ctx_row, half * TA_HALF);
                        const int hi = min((ctx_row + a.box - 1) / a.box * a.box, (half + 1) * TA_HALF);
                        uint8_t *vt = smem + S::kv_off + stv * S::tile;
                        for (int q = r; q < (hi - lo) * S::halves * 8; q += 128) {
                            const int row = lo + q / (S::halves * 8), c = q % (S::halves * 8);
                            *reinterpret_cast<uint4 *>(vt + (c >> 3) * S::half + row * 128 + (c & 7) * 16) =
                                make_uint4(0u, 0u, 0u, 0u);
                        }
                        fence_proxy_async_smem();
                    }
                }
                float mx[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) mx[c] = __uint_as_float(v[c >> 1][(c & 1) * 16]);
#pragma unroll
                for (int q = 1; q < 15; q += 2)
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        mx[c] = max3(mx[c], __uint_as_float(v[c >> 1][(c & 1) * 16 + q]),
                                     __uint_as_float(v[c >> 1][(c & 1) * 16 + q + 1]));
#pragma unroll
                for (int c = 0; c < 4; ++c) mx[c] = fmaxf(mx[c], __uint_as_float(v[c >> 1][(c & 1) * 16 + 15]));
                const float mr = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]);
                const float mb = mr * a.scale_log2;            // the scale is positive
                const bool grows = mb > m + kRescaleThreshold || (m == -INFINITY && mb != -INFINITY);
                if (__any_sync(0xffffffffu, grows)) {
                    const float f = grows ? (m == -INFINITY ? 0.f : exp2f(m - mb)) : 1.f;
                    if (t > 0) {
                        // the last step's P V must be done; tcgen05.ld/st take the whole warp
                        ok = wait_or_abort(&pvdone[2 * x + (buf ^ 1)], ((k - 1) >> 1) & 1, &ctl->abort);
                        if (!__all_sync(0xffffffffu, ok)) { dead = true; break; }
                        tc_fence_after();
#pragma unroll 1
                        for (int c = 0; c < D / 32; ++c) {
                            uint32_t o[32];
                            tmem_ld32(tOx + c * 32, o);
                            tmem_wait_ld_dep32(o);
#pragma unroll
                            for (int q = 0; q < 32; ++q) o[q] = __float_as_uint(__uint_as_float(o[q]) * f);
                            tmem_st32(tOx + c * 32, o);
                        }
                    }
                    l *= f;
                    if (grows) m = mb;
                }
                const float base = m == -INFINITY ? 0.f : m;
                const uint64_t sc2 = f2_pack(a.scale_log2, a.scale_log2), nb2 = f2_pack(-base, -base);
                const uint64_t one2 = f2_pack(1.f, 1.f);
                uint64_t rs2[4] = {0ull, 0ull, 0ull, 0ull};
                uint32_t pk[32];
#pragma unroll
                for (int q = 0; q < 32; ++q) {
                    const uint32_t *u = &v[q >> 4][(2 * q) & 31];
                    float p0, p1;
                    f2_unpack(f2_fma(f2_pack(__uint_as_float(u[0]), __uint_as_float(u[1])), sc2, nb2), p0, p1);
                    p0 = ex2_sfu(p0);
                    p1 = ex2_sfu(p1);
                    rs2[q & 3] = f2_fma(f2_pack(p0, p1), one2, rs2[q & 3]);
                    if (KV8) {
                        const float4 f = sc[32 + (q >> 1)];
                        f2_unpack(f2_mul(f2_pack(p0, p1), (q & 1) ? f2_pack(f.z, f.w) : f2_pack(f.x, f.y)), p0, p1);
                    }
                    pk[q] = pack_bf16x2(p0, p1);               // the products' precision: one rounding of each weight
                }
                tmem_st32(tSb, pk);
                float rsum = 0.f;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float lo, hi;
                    f2_unpack(rs2[q], lo, hi);
                    rsum += lo + hi;
                }
                l += rsum;
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&pfull[2 * x + buf]);
            }
            // ---- the item's end (or this CTA's part of it)
            cnt += steps;
            i0 += nb;
            need_masks();
            const uint32_t *mw = masks + 4 * node;
            const bool lives = valid && !dead && ((mw[node >> 5] >> (node & 31)) & 1u);
            // A padding row: zeros and -inf.  A row that lives has at least its own logit, so a sum of 0 over all
            // of it says that every logit is -inf, and its softmax is 0 / 0; a sum that is a NaN (of logits that
            // are: the maximum may still be -inf, from masked columns) stays one.
            if (!lives) l = 0.f;
            float m_o = -INFINITY, l_o = 0.f;      // the other set's part of the row
            if (!g.pair) {
                // two copies in turn: a set may be an item ahead of the other, which still reads
                float *ml = reinterpret_cast<float *>(smem + S::ml_off) + (singles & 1) * 512;
                ml[x * 256 + r] = m;
                ml[x * 256 + 128 + r] = l;
                __syncwarp();
                if (!dead) {                       // (a warp that gave up does not meet the others: their wait ends too)
                    if (lane == 0) mbar_arrive(mlfull);
                    if (!__all_sync(0xffffffffu, wait_or_abort(mlfull, singles & 1, &ctl->abort))) dead = true;
                }
                ++singles;
                m_o = ml[(x ^ 1) * 256 + r];
                l_o = ml[(x ^ 1) * 256 + 128 + r];
                // (both sets have taken the same steps)
                if (!dead && !wait_or_abort(&pvdone[2 * (x ^ 1) + ((cnt - 1) & 1)], ((cnt - 1) >> 1) & 1, &ctl->abort)) dead = true;
            }
            if (!dead && !wait_or_abort(&pvdone[2 * x + ((cnt - 1) & 1)], ((cnt - 1) >> 1) & 1, &ctl->abort)) dead = true;
            dead = __any_sync(0xffffffffu, dead);
            if (dead) {
                __syncwarp();
                continue;                          // outputs stay; the status word tells
            }
            tc_fence_after();
            const float mt = fmaxf(l > 0.f ? m : -INFINITY, l_o > 0.f ? m_o : -INFINITY);
            const float f_own = l != 0.f ? exp2f(m - mt) : 0.f, f_oth = l_o != 0.f ? exp2f(m_o - mt) : 0.f;
            const float lt = l * f_own + l_o * f_oth;
            const bool whole = g.blk0 == 0 && g.blk1 == s.nblk;
            const float inv = lt != 0.f || (whole && lives) ? 1.f / lt : 0.f;
            const float g_own = f_own * inv, g_oth = f_oth * inv;
            // slot 0: an item that began in an earlier CTA, 1: one that ends in a later CTA
            const int64_t pslot = (int64_t)blockIdx.x * 2 + (g.blk0 > 0 ? 0 : 1);
            const int prow = (g.pair ? x * 128 : 0) + r;
            const int64_t orow = (int64_t)(s.tok0 + tok) * a.H + g.hk * a.group + head;
            // a single tile: set x takes half of the columns of both parts
            const int col0 = g.pair ? 0 : x * (D / 2), cols = g.pair ? D : D / 2;
            const uint32_t tOo = tO + (x ^ 1) * 128 + trow;
#pragma unroll 1
            for (int c = col0; c < col0 + cols; c += 32) {
                uint32_t o[32];
                float acc[32];
                tmem_ld32(tOx + c, o);
                tmem_wait_ld_dep32(o);
#pragma unroll
                for (int q = 0; q < 32; ++q) acc[q] = __uint_as_float(o[q]) * g_own;
                if (!g.pair) {
                    tmem_ld32(tOo + c, o);
                    tmem_wait_ld_dep32(o);
#pragma unroll
                    for (int q = 0; q < 32; ++q) acc[q] += __uint_as_float(o[q]) * g_oth;
                }
                if (!lives) {
#pragma unroll
                    for (int q = 0; q < 32; ++q) acc[q] = 0.f;
                }
                if (whole) {
                    if (valid) {
                        uint4 *p = reinterpret_cast<uint4 *>(a.out + orow * D + c);
#pragma unroll
                        for (int u = 0; u < 4; ++u)
                            p[u] = make_uint4(pack_bf16x2(acc[8 * u], acc[8 * u + 1]), pack_bf16x2(acc[8 * u + 2], acc[8 * u + 3]),
                                              pack_bf16x2(acc[8 * u + 4], acc[8 * u + 5]), pack_bf16x2(acc[8 * u + 6], acc[8 * u + 7]));
                    }
                } else if (valid) {
                    // four columns of all 256 rows lie side by side: a warp stores 512 bytes at a time
                    float4 *p = reinterpret_cast<float4 *>(a.part) + pslot * (D / 4 * 256) + (c / 4) * 256 + prow;
#pragma unroll
                    for (int u = 0; u < 8; ++u)
                        p[u * 256] = make_float4(acc[4 * u], acc[4 * u + 1], acc[4 * u + 2], acc[4 * u + 3]);
                }
            }
            if (valid && (g.pair || x == 0)) {
                if (!whole) a.part_lse[pslot * 256 + prow] = !lives ? kPadding : lt != 0.f ? mt + log2f(lt) : -INFINITY;
                else if (a.lse) a.lse[orow] = !lives ? -INFINITY : lt != 0.f ? mt * kLn2 + logf(lt) : kNaN;
            }
            tc_fence_before();
            fence_proxy_async_smem();              // ml, before TMA may write Q there
            __syncwarp();
            if (lane == 0) mbar_arrive(&oempty[items & 1]);
            ++items;
        }
    }

    tc_fence_before();
    __syncthreads();
    if (tid == 0) {
        if (ctl->abort) {
            ctl->err = DSA_ERR_TIMEOUT;
            // let copies and products in flight land before shared and tensor memory go
            const int n_kv = KV8 ? ctl->code_issued : ctl->kv_issued, ring = KV8 ? CODES : SLOTS;
            for (int j = max(0, n_kv - ring); j < n_kv; ++j)
                mbar_wait(KV8 ? &cfull[j % ring] : &kvfull[j % ring], (j / ring) & 1);
            if (ctl->q_issued > 0) mbar_wait(qfull, (ctl->q_issued - 1) & 1);
            for (int y = 0; y < 2; ++y) {
                const int ns = ctl->s_issued[y] - 1, np = ctl->pv_issued[y] - 1;
                if (ns >= 0) mbar_wait(&sfull[2 * y + (ns & 1)], (ns >> 1) & 1);
                if (np >= 0) mbar_wait(&pvdone[2 * y + (np & 1)], (np >> 1) & 1);
            }
        }
        a.err[blockIdx.x] = (uint32_t)ctl->err;
    }
    __syncthreads();
    tc_fence_after();
    grid_dep_trigger();
    if (warp == 0) tmem_dealloc(tmem, 512);
}

template <int D>
__global__ void __launch_bounds__(TA_THREADS, 1)
tree_attn_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                 const __grid_constant__ CUtensorMap vmap, const __grid_constant__ TreeArgs a)
{
    tree_attn_body<false, D>(qmap, kmap, vmap, a);
}

template <int D>
__global__ void __launch_bounds__(TA8_THREADS, 1)
tree_attn_kv8_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap, const __grid_constant__ TreeArgs a)
{
    tree_attn_body<true, D>(qmap, kmap, vmap, a);
}

// ---------------------------------------------------------------- merge of cut items

// Parts of a cut item: the last of the CTA where it began (slot 1), and the first
// (slot 0) of every CTA behind it up to its end.
//   out = sum_i 2^(L_i - M) O_i / sum_i 2^(L_i - M),  L_i the parts' log2 sums.
constexpr int TM_THREADS = 256;        // rows of two tiles
constexpr int TM_QUADS = 4;            // sixteen columns: 32 bytes of output, a sector
constexpr int TM_PARTS = 4;            // parts in flight

template <int D>
__global__ void __launch_bounds__(TM_THREADS)
tree_merge_kernel(const __grid_constant__ TreeArgs a, int ctas)
{
    grid_dep_wait();
    __shared__ int4 desc[TA_MAX_CTAS];
    __shared__ int first[TA_MAX_CTAS];         // CTAs in whose share a cut item continues for the first time
    __shared__ int n_items;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int c = tid; c < ctas; c += TM_THREADS) desc[c] = a.desc[c];
    if (tid == 0) n_items = 0;
    if (blockIdx.x == 0 && warp == 0) {        // the call's status word: the worst of the CTAs'
        uint32_t e = 0;
        for (int c = lane; c < ctas; c += 32) e = max(e, a.err[c]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) e = max(e, __shfl_xor_sync(0xffffffffu, e, o));
        if (lane == 0) {
            a.hdr->status = e;
            a.hdr->detail = 0;
        }
    }
    __syncthreads();
    auto same = [&](int c, int d) { return desc[c].x == desc[d].x && desc[c].y == desc[d].y && desc[c].z == desc[d].z; };
    if (warp == 0) {                           // in order
        for (int c0 = 0; c0 < ctas; c0 += 32) {
            const int c = c0 + lane;
            const bool f = c > 0 && c < ctas && desc[c].x >= 0 && (desc[c].w & 1) && !((desc[c - 1].w & 1) && same(c, c - 1));
            const unsigned fs = __ballot_sync(0xffffffffu, f);
            if (f) first[n_items + __popc(fs & ((1u << lane) - 1u))] = c;
            __syncwarp();
            if (lane == 0) n_items += __popc(fs);
            __syncwarp();
        }
    }
    __syncthreads();
    // a block per item and TM_QUADS column quads, a thread per row; a single tile has 128 rows, and the
    // threads behind them take every other part
    constexpr int groups = D / 4 / TM_QUADS;
    __shared__ float4 half_acc[TM_QUADS][128];
    __shared__ float2 half_ml[128];
    for (int u = blockIdx.x; u < n_items * groups; u += gridDim.x) {
        const int c = first[u / groups], quad = (u % groups) * TM_QUADS;
        const int4 d = desc[c];
        Seq s;
        bool bad;
        s.load(a, d.x, bad);
        const bool pair = d.w & 2;
        const int x = pair ? tid >> 7 : 0, r = tid & 127, row = x * 128 + r;
        const int step = pair ? 1 : 2, begin = pair ? 0 : tid >> 7;
        const int tile = d.z + x, tr = r / a.rows_tok;
        const int tok = (a.head_tiles > 1 ? tile / a.head_tiles : tile * a.tile_tok) + tr;
        const int head = (a.head_tiles > 1 ? (tile % a.head_tiles) * TA_M : 0) + r - tr * a.rows_tok;
        const bool valid = tr < a.tile_tok && tok < s.n && head < a.group;
        int parts = 1;
        while (c + parts - 1 < ctas && (desc[c + parts - 1].w & 1) && same(c, c + parts - 1)) ++parts;
        // part 0: slot 1 of CTA c - 1; part p: slot 0 of CTA c - 1 + p
        auto at = [&](int p) -> int64_t { return (int64_t)(c - 1 + p) * 2 + (p == 0 ? 1 : 0); };
        const float4 *part = reinterpret_cast<const float4 *>(a.part) + quad * 256 + row;
        // one pass: sums relative to the largest part so far
        float M = -INFINITY, sum = 0.f;
        bool padding = false;                  // (all parts say the same; the thread that writes has part 0)
        float4 acc[TM_QUADS];
#pragma unroll
        for (int e = 0; e < TM_QUADS; ++e) acc[e] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int p0 = begin; valid && p0 < parts; p0 += TM_PARTS * step) {
            float L[TM_PARTS];
            float4 o[TM_PARTS][TM_QUADS];
            float top = M;
            bool any = false;                  // a part that holds something, if only a NaN
#pragma unroll
            for (int q = 0; q < TM_PARTS; ++q) {
                L[q] = -INFINITY;
                const int p = p0 + q * step;
                if (p >= parts) continue;
                L[q] = a.part_lse[at(p) * 256 + row];
                padding |= L[q] == kPadding;
#pragma unroll
                for (int e = 0; e < TM_QUADS; ++e) o[q][e] = part[at(p) * (D / 4 * 256) + e * 256];
            }
            if (padding) break;
#pragma unroll
            for (int q = 0; q < TM_PARTS; ++q) {
                top = fmaxf(top, L[q]);
                any |= L[q] != -INFINITY;
            }
            if (!any) continue;
            const float f = sum != 0.f ? exp2f(M - top) : 0.f;
            M = top;
            sum *= f;
#pragma unroll
            for (int e = 0; e < TM_QUADS; ++e) {
                acc[e].x *= f;
                acc[e].y *= f;
                acc[e].z *= f;
                acc[e].w *= f;
            }
#pragma unroll
            for (int q = 0; q < TM_PARTS; ++q) {
                if (p0 + q * step >= parts) continue;
                const float wt = L[q] != -INFINITY ? exp2f(L[q] - M) : 0.f;
                sum += wt;
#pragma unroll
                for (int e = 0; e < TM_QUADS; ++e) {
                    acc[e].x += wt * o[q][e].x;
                    acc[e].y += wt * o[q][e].y;
                    acc[e].z += wt * o[q][e].z;
                    acc[e].w += wt * o[q][e].w;
                }
            }
        }
        if (!pair) {
            if (begin == 1) {
#pragma unroll
                for (int e = 0; e < TM_QUADS; ++e) half_acc[e][r] = acc[e];
                half_ml[r] = make_float2(M, sum);
            }
            __syncthreads();
            if (begin == 0) {
                const float2 other = half_ml[r];
                const float top = fmaxf(M, other.x);
                const float f0 = sum != 0.f ? exp2f(M - top) : 0.f, f1 = other.y != 0.f ? exp2f(other.x - top) : 0.f;
                M = top;
                sum = sum * f0 + other.y * f1;
#pragma unroll
                for (int e = 0; e < TM_QUADS; ++e) {
                    const float4 b = half_acc[e][r];
                    acc[e] = make_float4(acc[e].x * f0 + b.x * f1, acc[e].y * f0 + b.y * f1, acc[e].z * f0 + b.z * f1,
                                         acc[e].w * f0 + b.w * f1);
                }
            }
            __syncthreads();                   // half_acc may be written again
            if (begin == 1) continue;
        }
        if (!valid) continue;
        const float inv = padding ? 0.f : 1.f / sum;           // 0 / 0 where no part has any weight
        const int64_t orow = (int64_t)(s.tok0 + tok) * a.H + d.y * a.group + head;
        uint4 *out = reinterpret_cast<uint4 *>(a.out + orow * D + quad * 4);
#pragma unroll
        for (int e = 0; e < TM_QUADS; e += 2)
            out[e / 2] = make_uint4(pack_bf16x2(acc[e].x * inv, acc[e].y * inv), pack_bf16x2(acc[e].z * inv, acc[e].w * inv),
                                    pack_bf16x2(acc[e + 1].x * inv, acc[e + 1].y * inv),
                                    pack_bf16x2(acc[e + 1].z * inv, acc[e + 1].w * inv));
        if (quad == 0 && a.lse) a.lse[orow] = padding ? -INFINITY : sum != 0.f ? M * kLn2 + logf(sum) : kNaN;
    }
}

template <bool KV8, int D>
cudaError_t launch_tree_t(const CUtensorMap &qmap, const CUtensorMap &kmap, const CUtensorMap &vmap, const TreeArgs &a,
                          int ctas, cudaStream_t st)
{
    auto kernel = KV8 ? tree_attn_kv8_kernel<D> : tree_attn_kernel<D>;
    constexpr int smem = Smem<KV8, D>::total;
    // once a device
    static std::atomic<uint64_t> ready{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0ull;
    if (!(ready.load(std::memory_order_acquire) & bit)) {
        cudaFuncAttributes fa;
        e = cudaFuncGetAttributes(&fa, kernel);
        if (e != cudaSuccess) return e;
        // the register split assumes it: an error, not a wait that never ends
        if (fa.numRegs != (KV8 ? TA8_REGS : TA_REGS)) return cudaErrorInvalidKernelImage;
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        ready.fetch_or(bit, std::memory_order_release);
    }
    e = launch_chained(kernel, dim3((unsigned)ctas), dim3(KV8 ? TA8_THREADS : TA_THREADS), smem, st, qmap, kmap, vmap, a);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    e = launch_chained(tree_merge_kernel<D>, dim3((unsigned)std::max(1, (ctas - 1) * (D / 4 / TM_QUADS))), dim3(TM_THREADS), 0, st, a, ctas);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

// Workspace: header, then these.
struct TreeWs {
    size_t desc, err, lse, part, end;
    explicit TreeWs(int d)
    {
        desc = kWsHeader;
        err = desc + sizeof(int4) * TA_MAX_CTAS;
        lse = err + align_up(sizeof(uint32_t) * TA_MAX_CTAS, 256);
        part = lse + sizeof(float) * 2 * 256 * TA_MAX_CTAS;
        end = part + sizeof(float) * 2 * 256 * (size_t)d * TA_MAX_CTAS;
    }
};

}  // namespace

size_t tree_attn_ws_bytes(int d) { return TreeWs(d).end; }

cudaError_t launch_tree_attn(const uint16_t *q, const void *k, const float *ks, const void *v, const float *vs,
                             const int32_t *block_table, const int32_t *context_lens, const int32_t *token_start,
                             const int32_t *parents, int64_t num_pages, int max_pages, int page_size, int B, int64_t N,
                             int max_tree, int64_t max_context, int H, int Hkv, int d, float sm_scale, uint16_t *out,
                             float *lse, void *ws, cudaStream_t st)
{
    uint8_t *w = static_cast<uint8_t *>(ws);
    const TreeWs L(d);
    TreeArgs a{};
    a.q = q;
    a.block_table = block_table;
    a.context_lens = context_lens;
    a.token_start = token_start;
    a.parents = parents;
    a.ks = ks;
    a.vs = vs;
    a.num_pages = num_pages;
    a.N = N;
    a.max_context = max_context;
    a.max_pages = max_pages;
    a.page_size = page_size;
    a.box = std::gcd(page_size, TA_BLK);
    a.B = B;
    a.max_tree = max_tree;
    a.H = H;
    a.Hkv = Hkv;
    a.group = H / Hkv;
    a.rows_tok = std::min(a.group, TA_M);
    a.tile_tok = TA_M / a.rows_tok;
    a.head_tiles = (int)ceil_div(a.group, TA_M);
    // measured a block: bf16 2.1 us for a pair and 1.3 for one, FP8 3.1 and 2.2 (the conversion is the same)
    a.cost_pair = ks ? 7 : 5;
    a.cost_one = ks ? 5 : 3;
    a.stall_at = consume_test_stall(2 /* tree attention */) ? 4 : ~0u;
    a.scale_log2 = sm_scale * kLog2e;
    a.out = out;
    a.lse = lse;
    a.desc = reinterpret_cast<int4 *>(w + L.desc);
    a.err = reinterpret_cast<uint32_t *>(w + L.err);
    a.part_lse = reinterpret_cast<float *>(w + L.lse);
    a.part = reinterpret_cast<float *>(w + L.part);
    a.hdr = reinterpret_cast<WsHeader *>(w);

    int dev = 0, sms = 148;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    // one CTA per SM, and no more than the largest possible list of work feeds
    const int64_t tiles = a.head_tiles > 1 ? N * a.head_tiles : ceil_div(N, a.tile_tok) + B;
    const int64_t most = tiles * Hkv * ceil_div(std::min(max_context, (int64_t)max_pages * page_size), TA_BLK);
    const int ctas = (int)std::max<int64_t>(1, std::min<int64_t>({(int64_t)sms, (int64_t)TA_MAX_CTAS, ceil_div(most, 2)}));

    CUtensorMap qmap, kmap, vmap;
    const uint64_t rows = (uint64_t)num_pages * page_size;
    const uint64_t qd[4] = {(uint64_t)d, (uint64_t)a.group, (uint64_t)Hkv, (uint64_t)N};
    const uint64_t qs[3] = {2ull * d, 2ull * d * a.group, 2ull * d * H};
    const uint32_t qb[4] = {64, (uint32_t)a.rows_tok, 1, (uint32_t)a.tile_tok};
    if (!make_tmap_bf16(&qmap, q, 4, qd, qs, qb)) return cudaErrorNotSupported;
    const uint64_t kd[3] = {(uint64_t)d, (uint64_t)Hkv, rows};
    const uint64_t size = ks ? 1 : 2;
    const uint64_t kst[2] = {size * d, size * d * Hkv};
    const uint32_t kb[3] = {ks ? (uint32_t)d : 64u, 1, (uint32_t)a.box};
    const bool maps = ks ? make_tmap_u8_linear(&kmap, k, 3, kd, kst, kb) && make_tmap_u8_linear(&vmap, v, 3, kd, kst, kb)
                         : make_tmap_bf16(&kmap, k, 3, kd, kst, kb) && make_tmap_bf16(&vmap, v, 3, kd, kst, kb);
    if (!maps) return cudaErrorNotSupported;
    if (ks) return d == 128 ? launch_tree_t<true, 128>(qmap, kmap, vmap, a, ctas, st)
                            : launch_tree_t<true, 64>(qmap, kmap, vmap, a, ctas, st);
    return d == 128 ? launch_tree_t<false, 128>(qmap, kmap, vmap, a, ctas, st)
                    : launch_tree_t<false, 64>(qmap, kmap, vmap, a, ctas, st);
}

}  // namespace dsa
