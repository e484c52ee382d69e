// Block tables and slot maps of the paged caches, built on the GPU from request
// lengths, and the cache rows of accepted drafts moved together.
//
// Pages are handed out by two running sums over the sequences (pages needed,
// tokens granted): one block scans them, 1024 sequences at a time, and gives the
// fresh pages out, one thread a page.  The token maps are then written by a
// second, chained launch, 16 bytes a token at HBM rate; up to BL_SMALL tokens the
// first block writes them itself and the second launch is saved.  At the sizes of
// a decode step all of this is latency: two scans, one table write, one read.
#include "kernels.h"

namespace dsa {
namespace {

constexpr int BL_THREADS = 1024;
// Tokens that the scanning block maps itself.
constexpr int64_t BL_SMALL = 4096;

__device__ __forceinline__ void report(uint32_t *status, dsa_status s)
{
    if (status) atomicCAS(status, (uint32_t)DSA_OK, (uint32_t)s);
}

// Inclusive sum over the block (BL_THREADS threads); *total gets the block's.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t *warp_sums, int64_t *total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t t = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += t;
    }
    if (lane == 31) warp_sums[warp] = v;
    __syncthreads();
    if (warp == 0) {
        int64_t w = warp_sums[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t t = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += t;
        }
        warp_sums[lane] = w;
    }
    __syncthreads();
    if (warp > 0) v += warp_sums[warp - 1];
    *total = warp_sums[31];
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

// The maps of four tokens t .. t + 3 (t a multiple of 4).
__device__ __forceinline__ void write_maps(const Maps &m, int64_t t)
{
    int b = upper(m.token_start + 1, m.B, t);
    int32_t sid[4], pos[4];
    int64_t slot[4];
    int32_t stop = 0, ctx = 0;
    int have = -1;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        sid[j] = pos[j] = -1;
        slot[j] = -1;
        while (b < m.B && (have == b ? stop : m.token_start[b + 1]) <= t + j) ++b;
        if (b >= m.B) continue;
        if (have != b) {
            stop = m.token_start[b + 1];
            ctx = m.context_lens[b];   // already the new length
            have = b;
        }
        sid[j] = b;
        const int p = ctx - stop + (int)(t + j);
        pos[j] = p;
        const int64_t page = m.block_table[(int64_t)b * m.max_pages + p / m.ps];
        if (page >= 0 && page < m.num_pages) slot[j] = page * m.ps + p % m.ps;
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

__global__ void __launch_bounds__(BL_THREADS)
blocks_extend_kernel(const int32_t *new_lens, int32_t *context_lens, int32_t *pages_held, int32_t *block_table,
                     const int32_t *free_pages, int64_t free_capacity, int32_t *free_count, int32_t *token_start,
                     Maps m, bool small)
{
    __shared__ int64_t sums[32];
    __shared__ int64_t ends[BL_THREADS];       // pages handed out up to and with each sequence of the chunk
    __shared__ int first_page[BL_THREADS];     // a sequence's pages before
    const int tid = threadIdx.x;
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
        int64_t total;
        const int64_t upto = asked + block_scan(need, sums, &total);
        asked += total;
        bool ok = grow > 0;
        if (ok && need > 0 && (!count_ok || upto > count)) {
            ok = false;
            report(m.status, DSA_ERR_WORKSPACE);
        }
        const int64_t t_upto = offered + block_scan(ok ? grow : 0, sums, &total);
        offered += total;
        if (ok && t_upto > m.max_tokens) {
            ok = false;
            report(m.status, DSA_ERR_WORKSPACE);
        }
        const int64_t got = ok ? grow : 0, pages = ok ? need : 0;
        const int64_t t_end = tokens + block_scan(got, sums, &total);
        tokens += total;
        const int64_t p_end = block_scan(pages, sums, &total);
        ends[tid] = p_end;
        first_page[tid] = (int)held;
        if (b < m.B) {
            token_start[b + 1] = (int32_t)t_end;
            if (ok) {
                context_lens[b] = (int32_t)(ctx + got);
                pages_held[b] = (int32_t)(held + pages);
            }
        }
        if (b == 0) token_start[0] = 0;
        __syncthreads();
        // served sequences take their pages from the top of the stack in order: the
        // refused ones come behind the last that needs any, so the sums are dense
        const int64_t top = count - 1 - served;
        for (int64_t i = tid; i < total; i += BL_THREADS) {
            const int s = upper(ends, BL_THREADS, i);
            const int64_t j = i - (s > 0 ? ends[s - 1] : 0);
            int32_t page = free_pages[top - i];
            if (page < 0 || page >= m.num_pages) page = -1;    // reported where its tokens are mapped
            block_table[(int64_t)(b0 + s) * m.max_pages + first_page[s] + j] = page;
        }
        served += total;
        __syncthreads();
    }
    if (tid == 0 && count_ok) free_count[0] = (int32_t)(count - served);
    if (small) {
        __syncthreads();               // this block's global writes are visible to its threads
        for (int64_t t = 4 * (int64_t)tid; t < m.max_tokens; t += 4 * BL_THREADS) write_maps(m, t);
    }
}

constexpr int BM_THREADS = 256;

__global__ void __launch_bounds__(BM_THREADS)
blocks_maps_kernel(Maps m)
{
    grid_dep_wait();                   // the tables and lengths of blocks_extend_kernel
    const int64_t step = 4 * (int64_t)gridDim.x * BM_THREADS;
    for (int64_t t = 4 * ((int64_t)blockIdx.x * BM_THREADS + threadIdx.x); t < m.max_tokens; t += step)
        write_maps(m, t);
}

__global__ void __launch_bounds__(BL_THREADS)
blocks_trim_kernel(const int32_t *keep_lens, int32_t *context_lens, int32_t *pages_held, int32_t *block_table,
                   int32_t *free_pages, int64_t free_capacity, int32_t *free_count, int B, int max_pages,
                   int64_t num_pages, int ps, uint32_t *status)
{
    __shared__ int64_t sums[32];
    __shared__ int64_t ends[BL_THREADS];
    __shared__ int first_page[BL_THREADS];
    const int tid = threadIdx.x;
    const int64_t count = free_count[0];
    const bool count_ok = count >= 0 && count <= free_capacity;
    if (!count_ok && tid == 0) report(status, DSA_ERR_INVALID_ARG);
    const int64_t room = count_ok ? free_capacity - count : 0;
    int64_t all = 0;                   // pages given back by all sequences
    // pages of one sequence to give back, 0 .. held; -1: the sequence is left alone
    auto freed_of = [&](int b, int &stay) -> int64_t {
        const int64_t ctx = context_lens[b], keep = keep_lens[b], held = pages_held[b];
        if (keep < 0 || keep > ctx || held < 0 || held > max_pages) return -1;
        stay = (int)min(held, (keep + ps - 1) / ps);
        return held - stay;
    };
    // first round: how many pages come back in all (the first of them goes on top)
    int64_t asked = 0;
    for (int b0 = 0; b0 < B; b0 += BL_THREADS) {
        const int b = b0 + tid;
        int stay = 0;
        int64_t freed = b < B ? max((int64_t)0, freed_of(b, stay)) : 0;
        int64_t total;
        const int64_t upto = asked + block_scan(freed, sums, &total);
        asked += total;
        if (upto > room) freed = 0;
        block_scan(freed, sums, &total);
        all += total;
    }
    asked = 0;
    int64_t before = 0;
    for (int b0 = 0; b0 < B; b0 += BL_THREADS) {
        const int b = b0 + tid;
        int stay = 0;
        int64_t freed = -1, total;
        if (b < B) {
            freed = freed_of(b, stay);
            if (freed < 0) report(status, DSA_ERR_INVALID_ARG);
        }
        const int64_t upto = asked + block_scan(max((int64_t)0, freed), sums, &total);
        asked += total;
        if (freed > 0 && upto > room) {
            freed = -1;
            report(status, DSA_ERR_WORKSPACE);
        }
        ends[tid] = block_scan(max((int64_t)0, freed), sums, &total);
        first_page[tid] = stay;
        if (freed >= 0) {
            context_lens[b] = keep_lens[b];
            pages_held[b] = stay;
        }
        __syncthreads();
        for (int64_t i = tid; i < total; i += BL_THREADS) {
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
        before += total;
        __syncthreads();
    }
    if (tid == 0 && count_ok) free_count[0] = (int32_t)(count + all);
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
    blocks_extend_kernel<<<1, BL_THREADS, 0, st>>>(new_lens, context_lens, pages_held, block_table, free_pages,
                                                   free_capacity, free_count, token_start, m, small);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || small) return e;
    const int64_t need = ceil_div(max_tokens, 4 * BM_THREADS);
    e = launch_chained(blocks_maps_kernel, dim3((unsigned)(need < 148 * 8 ? need : 148 * 8)), dim3(BM_THREADS), 0, st, m);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

cudaError_t launch_blocks_trim(const int32_t *keep_lens, int32_t *context_lens, int32_t *pages_held,
                               int32_t *block_table, int32_t *free_pages, int64_t free_capacity, int32_t *free_count,
                               int B, int max_pages, int64_t num_pages, int ps, uint32_t *status, cudaStream_t st)
{
    blocks_trim_kernel<<<1, BL_THREADS, 0, st>>>(keep_lens, context_lens, pages_held, block_table, free_pages,
                                                 free_capacity, free_count, B, max_pages, num_pages, ps, status);
    return cudaGetLastError();
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
    cache_compact_kernel<<<(unsigned)B, CP_THREADS, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace dsa
