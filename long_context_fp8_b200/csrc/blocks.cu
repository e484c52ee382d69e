// Block tables and slot maps of the paged caches, built on the GPU from request
// lengths, and the cache rows of accepted drafts moved together.
//
// Pages are handed out by two running sums over the sequences (pages needed,
// tokens granted): one block scans them, 1024 sequences at a time, and gives the
// fresh pages out, one thread a page.  The token maps are then written by a
// second, chained launch, 16 bytes a token at HBM rate; up to BL_SMALL tokens the
// first block writes them itself and the second launch is saved.  At the sizes of
// a decode step all of this is latency: two scans, one table write, one read.
#include <cooperative_groups.h>

#include "kernels.h"

namespace dsa {
namespace {

namespace cg = cooperative_groups;

constexpr int BL_THREADS = 1024;
// Tokens that the scanning block maps itself.
constexpr int64_t BL_SMALL = 4096;
// Blocks that share the pages out where there may be many.
constexpr int BL_CLUSTER = 8;

__device__ __forceinline__ void report(uint32_t *status, dsa_status s)
{
    if (status) atomicCAS(status, (uint32_t)DSA_OK, (uint32_t)s);
}

struct Two { int64_t a, b; };

__device__ __forceinline__ Two warp_scan(Two v, int lane)
{
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t a = __shfl_up_sync(0xffffffffu, v.a, o), b = __shfl_up_sync(0xffffffffu, v.b, o);
        if (lane >= o) { v.a += a; v.b += b; }
    }
    return v;
}

// Inclusive sums of two values over the block (BL_THREADS threads); *total gets the block's.
__device__ __forceinline__ Two block_scan(Two v, Two *warp_sums, Two *total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    v = warp_scan(v, lane);
    if (lane == 31) warp_sums[warp] = v;
    __syncthreads();
    // every warp sums the warps' totals for itself: one barrier less
    const Two w = warp_scan(warp_sums[lane], lane);
    total->a = __shfl_sync(0xffffffffu, w.a, 31);
    total->b = __shfl_sync(0xffffffffu, w.b, 31);
    const int64_t ba = __shfl_sync(0xffffffffu, w.a, (warp + 31) & 31), bb = __shfl_sync(0xffffffffu, w.b, (warp + 31) & 31);
    if (warp > 0) { v.a += ba; v.b += bb; }
    __syncthreads();                   // warp_sums may be written again
    return v;
}

// First i in [0, n) with ends[i] > x (ends ascending; n if none).
template <typename I>
__device__ __forceinline__ int upper(const I *ends, int n, int64_t x)
{
    int lo = 0, hi = n;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if ((int64_t)ends[mid] > x) hi = mid; else lo = mid + 1;
    }
    return lo;
}

struct Maps {
    const int32_t *token_start, *context_lens, *block_table;
    int B, max_pages, ps;
    int64_t num_pages, max_tokens;
    int32_t *seq_ids, *positions;
    int64_t *slots;
    uint32_t *status;
};

// The maps of four tokens t .. t + 3 (t a multiple of 4).  `ends` and `lens`: token_start + 1 and context_lens,
// or copies of them.
__device__ __forceinline__ void write_maps(const Maps &m, const int32_t *ends, const int32_t *lens, int64_t t)
{
    int b = upper(ends, m.B, t);
    int32_t sid[4], pos[4];
    int64_t slot[4];
    int32_t stop = 0, ctx = 0;
    int have = -1;
    int32_t at = -1, page = -1;        // column of the table and the page there
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        sid[j] = pos[j] = -1;
        slot[j] = -1;
        if (b < m.B && (have == b ? stop : ends[b]) <= t + j) {
            ++b;                       // mostly the next one; any number without tokens may lie between (a step each
                                       // is 90 ns: 18 ms over 200 000 of them, 0.5 with the search)
            if (b < m.B && ends[b] <= t + j) b += upper(ends + b, m.B - b, t + j);
        }
        if (b >= m.B) continue;
        if (have != b) {
            stop = ends[b];
            ctx = lens[b];             // already the new length
            have = b;
            at = -1;
        }
        sid[j] = b;
        const int p = ctx - stop + (int)(t + j), col = p / m.ps;
        pos[j] = p;
        if (col != at) {
            at = col;
            page = m.block_table[(int64_t)b * m.max_pages + col];
        }
        if (page >= 0 && page < m.num_pages) slot[j] = (int64_t)page * m.ps + (p - col * m.ps);
        else report(m.status, DSA_ERR_INVALID_ARG);
    }
    if (t + 4 <= m.max_tokens) {
        *reinterpret_cast<int4 *>(m.seq_ids + t) = make_int4(sid[0], sid[1], sid[2], sid[3]);
        *reinterpret_cast<int4 *>(m.positions + t) = make_int4(pos[0], pos[1], pos[2], pos[3]);
        if (m.slots) {
            *reinterpret_cast<longlong2 *>(m.slots + t) = make_longlong2(slot[0], slot[1]);
            *reinterpret_cast<longlong2 *>(m.slots + t + 2) = make_longlong2(slot[2], slot[3]);
        }
    } else {
        for (int j = 0; j < 4 && t + j < m.max_tokens; ++j) {
            m.seq_ids[t + j] = sid[j];
            m.positions[t + j] = pos[j];
            if (m.slots) m.slots[t + j] = slot[j];
        }
    }
}

// Every block of the cluster runs the same sums over the same lengths; the first one
// writes the new ones, when all have read, and the pages are shared out among them.
__global__ void __launch_bounds__(BL_THREADS)
blocks_extend_kernel(const int32_t *new_lens, int32_t *context_lens, int32_t *pages_held, int32_t *block_table,
                     const int32_t *free_pages, int64_t free_capacity, int32_t *free_count, int32_t *token_start,
                     const Maps m, bool small)
{
    cg::cluster_group cluster = cg::this_cluster();
    __shared__ Two sums[32];
    __shared__ int64_t ends[BL_THREADS];       // pages handed out up to and with each sequence of the chunk
    __shared__ int first_page[BL_THREADS];     // a sequence's pages before
    __shared__ int32_t t_ends[BL_THREADS], lens[BL_THREADS];
    const int tid = threadIdx.x, blocks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const bool writer = rank == 0;
    grid_dep_wait();
    const int64_t count = free_count[0];
    const bool count_ok = count >= 0 && count <= free_capacity;
    if (!count_ok && tid == 0) report(m.status, DSA_ERR_INVALID_ARG);
    int64_t asked = 0, offered = 0, served = 0, tokens = 0;    // sums over the chunks before
    for (int b0 = 0; b0 < m.B; b0 += BL_THREADS) {
        const int b = b0 + tid;
        int64_t ctx = 0, grow = 0, held = 0, need = 0;
        if (b < m.B) {
            ctx = context_lens[b];
            grow = new_lens[b];
            held = pages_held[b];
            const int64_t room = (int64_t)m.max_pages * m.ps;
            if (grow != 0) {
                if (grow < 0 || ctx < 0 || held < 0 || held > m.max_pages || held * m.ps < ctx || ctx + grow > room) {
                    report(m.status, DSA_ERR_INVALID_ARG);
                    grow = 0;
                } else {
                    need = max((int64_t)0, (ctx + grow + m.ps - 1) / m.ps - held);
                }
            }
        }
        // one pass of sums where no sequence is refused
        Two total, upto = block_scan({need, grow}, sums, &total);
        int64_t got = grow, pages = need;
        bool ok = grow > 0;
        const bool tight = (need > 0 && (!count_ok || asked + upto.a > count)) || (ok && offered + upto.b > m.max_tokens);
        if (__syncthreads_or(tight)) {
            if (ok && need > 0 && (!count_ok || asked + upto.a > count)) {
                ok = false;
                report(m.status, DSA_ERR_WORKSPACE);
            }
            asked += total.a;
            const int64_t t_upto = offered + block_scan({ok ? grow : 0, 0}, sums, &total).a;
            offered += total.a;
            if (ok && t_upto > m.max_tokens) {
                ok = false;
                report(m.status, DSA_ERR_WORKSPACE);
            }
            got = ok ? grow : 0;
            pages = ok ? need : 0;
            upto = block_scan({pages, got}, sums, &total);
        } else {
            asked += total.a;
            offered += total.b;
        }
        const int64_t t_end = tokens + upto.b;
        tokens += total.b;
        ends[tid] = upto.a;
        first_page[tid] = (int)held;
        t_ends[tid] = (int32_t)t_end;
        lens[tid] = (int32_t)(ctx + got);
        cluster.sync();                // all have read the lengths; and the block its shared arrays
        if (writer) {
            if (b < m.B) {
                token_start[b + 1] = (int32_t)t_end;
                if (ok) {
                    context_lens[b] = (int32_t)(ctx + got);
                    pages_held[b] = (int32_t)(held + pages);
                }
            }
            if (b == 0) token_start[0] = 0;
        }
        // served sequences take their pages from the top of the stack in order: the
        // refused ones come behind the last that needs any, so the sums are dense
        const int64_t top = count - 1 - served;
        for (int64_t i = (int64_t)rank * BL_THREADS + tid; i < total.a; i += (int64_t)blocks * BL_THREADS) {
            const int s = upper(ends, BL_THREADS, i);
            const int64_t j = i - (s > 0 ? ends[s - 1] : 0);
            int32_t page = free_pages[top - i];
            if (page < 0 || page >= m.num_pages) page = -1;    // reported where its tokens are mapped
            block_table[(int64_t)(b0 + s) * m.max_pages + first_page[s] + j] = page;
        }
        served += total.a;
        __syncthreads();               // the shared arrays may be written; this block's table is visible to it
    }
    if (writer && tid == 0 && count_ok && served > 0) free_count[0] = (int32_t)(count - served);
    if (small) {
        const bool copied = m.B <= BL_THREADS;
        for (int64_t t = 4 * (int64_t)tid; t < m.max_tokens; t += 4 * BL_THREADS)
            write_maps(m, copied ? t_ends : m.token_start + 1, copied ? lens : m.context_lens, t);
    }
}

constexpr int BM_THREADS = 256;

__global__ void __launch_bounds__(BM_THREADS)
blocks_maps_kernel(const Maps m)
{
    grid_dep_wait();                   // the tables and lengths of blocks_extend_kernel
    const int64_t step = 4 * (int64_t)gridDim.x * BM_THREADS;
    for (int64_t t = 4 * ((int64_t)blockIdx.x * BM_THREADS + threadIdx.x); t < m.max_tokens; t += step)
        write_maps(m, m.token_start + 1, m.context_lens, t);
}

__global__ void __launch_bounds__(BL_THREADS)
blocks_trim_kernel(const int32_t *keep_lens, int32_t *context_lens, int32_t *pages_held, int32_t *block_table,
                   int32_t *free_pages, int64_t free_capacity, int32_t *free_count, int B, int max_pages,
                   int64_t num_pages, int ps, uint32_t *status)
{
    cg::cluster_group cluster = cg::this_cluster();
    __shared__ Two sums[32];
    __shared__ int64_t ends[BL_THREADS];
    __shared__ int first_page[BL_THREADS];
    const int tid = threadIdx.x, blocks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const bool writer = rank == 0;
    grid_dep_wait();
    const int64_t count = free_count[0];
    const bool count_ok = count >= 0 && count <= free_capacity;
    if (!count_ok && tid == 0) report(status, DSA_ERR_INVALID_ARG);
    const int64_t room = count_ok ? free_capacity - count : 0;
    // pages of one sequence to give back, 0 .. held; -1: the sequence is left alone
    auto freed_of = [&](int b, int &stay) -> int64_t {
        const int64_t ctx = context_lens[b], keep = keep_lens[b], held = pages_held[b];
        if (keep < 0 || keep > ctx || held < 0 || held > max_pages) return -1;
        stay = (int)min(held, (keep + ps - 1) / ps);
        return held - stay;
    };
    // first round: how many pages come back in all (the first of them goes on top); a single chunk
    // knows it when it has summed
    int64_t asked = 0, all = 0;
    const bool one = B <= BL_THREADS;
    for (int b0 = 0; b0 < B && !one; b0 += BL_THREADS) {
        const int b = b0 + tid;
        int stay = 0;
        const int64_t freed = b < B ? max((int64_t)0, freed_of(b, stay)) : 0;
        Two total;
        const int64_t upto = asked + block_scan({freed, 0}, sums, &total).a;
        asked += total.a;
        if (asked > room) block_scan({upto > room ? 0 : freed, 0}, sums, &total);
        all += total.a;
    }
    if (!one) cluster.sync();          // all have read free_count
    asked = 0;
    int64_t before = 0;
    for (int b0 = 0; b0 < B; b0 += BL_THREADS) {
        const int b = b0 + tid;
        int stay = 0;
        int64_t freed = -1;
        if (b < B) {
            freed = freed_of(b, stay);
            if (freed < 0) report(status, DSA_ERR_INVALID_ARG);
        }
        Two total;
        int64_t end = block_scan({max((int64_t)0, freed), 0}, sums, &total).a;
        const int64_t upto = asked + end;
        asked += total.a;
        if (asked > room) {
            if (freed > 0 && upto > room) {
                freed = -1;
                report(status, DSA_ERR_WORKSPACE);
            }
            end = block_scan({max((int64_t)0, freed), 0}, sums, &total).a;
        }
        if (one) all = total.a;
        ends[tid] = end;
        first_page[tid] = stay;
        cluster.sync();                // all have read this chunk's lengths; and the block its shared arrays
        if (writer && freed >= 0) {
            context_lens[b] = keep_lens[b];
            pages_held[b] = stay;
        }
        for (int64_t i = (int64_t)rank * BL_THREADS + tid; i < total.a; i += (int64_t)blocks * BL_THREADS) {
            const int s = upper(ends, BL_THREADS, i);
            const int64_t j = i - (s > 0 ? ends[s - 1] : 0);
            int32_t *entry = block_table + (int64_t)(b0 + s) * max_pages + first_page[s] + j;
            int32_t page = *entry;
            if (page < 0 || page >= num_pages) {
                page = -1;
                report(status, DSA_ERR_INVALID_ARG);
            }
            *entry = -1;
            free_pages[count + all - 1 - before - i] = page;
        }
        before += total.a;
        __syncthreads();
    }
    if (writer && tid == 0 && count_ok && all > 0) free_count[0] = (int32_t)(count + all);
}

// ---------------------------------------------------------------- compaction

constexpr int CP_THREADS = 128;
constexpr int CP_BATCH = 8;

struct CompactArgs {
    const int32_t *block_table, *context_lens, *token_start, *path, *accept_len;
    int B;
    int64_t N;
    int max_path, max_pages;
    int64_t num_pages;
    int ps;
    uint8_t *rows[3];                  // index keys, K, V (null: none)
    int row_bytes[3];                  // multiples of 8
    float *scale[3];                   // null: none
    int32_t *keep_lens;
    uint32_t *status;
};

// One block per sequence.  A thread owns one 8-byte column of a cache's rows
// (or one scale) and moves it row by row along the path, CP_BATCH rows read
// before they are written.  path[i] >= i, so a row is overwritten only after
// it was read: by this thread, earlier or in the same batch.  No thread touches
// another's columns, so no barrier orders them.
__global__ void __launch_bounds__(CP_THREADS)
cache_compact_kernel(const CompactArgs a)
{
    __shared__ int64_t src[DSA_MAX_TREE], dst[DSA_MAX_TREE];
    __shared__ int bad;
    const int b = blockIdx.x, tid = threadIdx.x;
    if (tid == 0) bad = 0;
    __syncthreads();
    grid_dep_wait();
    const int64_t t0 = a.token_start[b], t1 = a.token_start[b + 1];
    const int64_t n = t1 - t0, ctx = a.context_lens[b], first = ctx - n;
    const int len = a.accept_len[b];
    const bool sane = t0 >= 0 && n >= 0 && t1 <= a.N && n <= DSA_MAX_TREE && first >= 0 &&
                      ctx <= (int64_t)a.max_pages * a.ps && len >= 0 && len <= n && len <= a.max_path;
    if (sane) {
        for (int i = tid; i < len; i += CP_THREADS) {
            const int p = a.path[(int64_t)b * a.max_path + i];
            const int prev = i > 0 ? a.path[(int64_t)b * a.max_path + i - 1] : -1;
            if (p <= prev || p >= n) { bad = 1; continue; }
            const int32_t *table = a.block_table + (int64_t)b * a.max_pages;
            const int64_t from = first + p, to = first + i;
            const int64_t pf = table[from / a.ps], pt = table[to / a.ps];
            if (pf < 0 || pf >= a.num_pages || pt < 0 || pt >= a.num_pages) { bad = 1; continue; }
            src[i] = pf * a.ps + from % a.ps;
            dst[i] = pt * a.ps + to % a.ps;
        }
    }
    __syncthreads();
    if (!sane || bad) {
        if (tid == 0) {
            if (a.keep_lens) a.keep_lens[b] = (int32_t)ctx;
            report(a.status, DSA_ERR_INVALID_ARG);
        }
        return;
    }
    if (tid == 0 && a.keep_lens) a.keep_lens[b] = (int32_t)(first + len);
    // rows that stay where they are need no move
    int i0 = 0;
    while (i0 < len && src[i0] == dst[i0]) ++i0;
    int columns = 0;
#pragma unroll
    for (int x = 0; x < 3; ++x) columns += (a.rows[x] ? a.row_bytes[x] / 8 : 0) + (a.scale[x] ? 1 : 0);
    for (int c = tid; c < columns; c += CP_THREADS) {
        int k = c;
        bool is_scale = false;
        uint8_t *base = nullptr;
        int64_t pitch = 0;
#pragma unroll
        for (int x = 0; x < 3; ++x) {
            if (base) break;
            const int w = a.rows[x] ? a.row_bytes[x] / 8 : 0;
            if (k < w) {
                base = a.rows[x] + 8 * (int64_t)k;
                pitch = a.row_bytes[x];
                break;
            }
            k -= w;
            if (a.scale[x]) {
                if (k == 0) {
                    base = reinterpret_cast<uint8_t *>(a.scale[x]);
                    pitch = 4;
                    is_scale = true;
                    break;
                }
                --k;
            }
        }
        for (int i = i0; i < len; i += CP_BATCH) {
            uint2 v[CP_BATCH];
#pragma unroll
            for (int j = 0; j < CP_BATCH; ++j) {
                if (i + j >= len) break;
                const uint8_t *p = base + src[i + j] * pitch;
                if (is_scale) v[j].x = *reinterpret_cast<const uint32_t *>(p);
                else v[j] = *reinterpret_cast<const uint2 *>(p);
            }
#pragma unroll
            for (int j = 0; j < CP_BATCH; ++j) {
                if (i + j >= len) break;
                uint8_t *p = base + dst[i + j] * pitch;
                if (is_scale) *reinterpret_cast<uint32_t *>(p) = v[j].x;
                else *reinterpret_cast<uint2 *>(p) = v[j];
            }
        }
    }
}

}  // namespace

cudaError_t launch_blocks_extend(const int32_t *new_lens, int32_t *context_lens, int32_t *pages_held,
                                 int32_t *block_table, const int32_t *free_pages, int64_t free_capacity,
                                 int32_t *free_count, int B, int max_pages, int64_t num_pages, int ps,
                                 int64_t max_tokens, int32_t *token_start, int32_t *seq_ids, int32_t *positions,
                                 int64_t *slots, uint32_t *status, cudaStream_t st)
{
    Maps m{token_start, context_lens, block_table, B, max_pages, ps, num_pages, max_tokens,
           seq_ids, positions, slots, status};
    const bool small = max_tokens <= BL_SMALL;
    cudaError_t e = launch_cluster(blocks_extend_kernel, 1, small ? 1 : BL_CLUSTER, BL_THREADS, 0, st, new_lens, context_lens,
                                   pages_held, block_table, free_pages, free_capacity, free_count, token_start, m, small);
    if (e != cudaSuccess || small) return e;
    const int64_t need = ceil_div(max_tokens, 4 * BM_THREADS);
    e = launch_chained(blocks_maps_kernel, dim3((unsigned)(need < 148 * 8 ? need : 148 * 8)), dim3(BM_THREADS), 0, st, m);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

cudaError_t launch_blocks_trim(const int32_t *keep_lens, int32_t *context_lens, int32_t *pages_held,
                               int32_t *block_table, int32_t *free_pages, int64_t free_capacity, int32_t *free_count,
                               int B, int max_pages, int64_t num_pages, int ps, uint32_t *status, cudaStream_t st)
{
    const int blocks = (int64_t)B * max_pages <= BL_THREADS ? 1 : BL_CLUSTER;
    return launch_cluster(blocks_trim_kernel, 1, blocks, BL_THREADS, 0, st, keep_lens, context_lens, pages_held, block_table,
                          free_pages, free_capacity, free_count, B, max_pages, num_pages, ps, status);
}

cudaError_t launch_cache_compact(const int32_t *block_table, const int32_t *context_lens, const int32_t *token_start,
                                 const int32_t *path, const int32_t *accept_len, int B, int64_t N, int max_path,
                                 int max_pages, int64_t num_pages, int ps, int d_I, int d, void *kidx_cache,
                                 float *kscale_cache, void *k_cache, float *k_scale, void *v_cache, float *v_scale,
                                 int32_t *keep_lens, uint32_t *status, cudaStream_t st)
{
    CompactArgs a{block_table, context_lens, token_start, path, accept_len, B, N, max_path, max_pages, num_pages, ps,
                  {(uint8_t *)kidx_cache, (uint8_t *)k_cache, (uint8_t *)v_cache},
                  {d_I, k_scale ? d : 2 * d, v_scale ? d : 2 * d},
                  {kscale_cache, k_scale, v_scale},
                  keep_lens, status};
    const cudaError_t e = launch_chained(cache_compact_kernel, dim3((unsigned)B), dim3(CP_THREADS), 0, st, a);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace dsa
