// Verification of drafted token trees against the target's probabilities.
//
// Along the walk almost nothing is read: a child is accepted or rejected on one
// entry of its parent's target and draft rows, and these are read all at once. Only a
// rejection sums a whole row (Z = sum_v max(R(v) / Z - Q(v), 0)), and the last one is
// drawn from.  So a sequence reads, besides single entries, one pair of rows for each
// rejection, or the last node's target row alone if no child was left to reject; with point
// masses one row for the first rejection and one for the draw, since the others change one entry (and one more
// each time that less than an eighth of the last sum is left).
//
// A cluster of thread blocks takes a sequence.  Every block runs the same walk from
// the same values; a row is cut into contiguous spans, one a warp, and each warp
// sums its span in 64 bits.  The warps' sums are kept: the draw finds the span by
// their running sum, the block goes through that span again in chunks, and one warp
// through the chunk that holds the value.  Sums have a fixed order, so a call repeats bit
// for bit.  R is never stored: it is made again from P and Q, rejection by rejection, in
// registers (a node has few rejections, and the second row pass finds P and Q in L2).
//
// Measured on one B200: a chain of 5 over 32 000 tokens 7.8 us; 64 trees of 16 over
// 128 001 tokens 44 us (121 at first, with 125 registers: one block an SM, four waves of
// clusters), of which the sequence with four rejections takes 8 us a pass: 100
// instructions for four elements a lane, most of them the 64-bit arithmetic, bind it on its four
// SMs, not the bytes (32 in flight a thread or 192 made no difference there).
#include <atomic>

#include <cooperative_groups.h>

#include "kernels.h"

namespace dsa {
namespace {

namespace cg = cooperative_groups;

constexpr int VF_THREADS = 512;
constexpr int VF_WARPS = VF_THREADS / 32;
constexpr int VF_DEPTH = 6;            // groups of four elements of a lane in the ring
constexpr int VF_RING = VF_DEPTH * 2 * VF_THREADS * 16;        // bytes: 96 KB, two blocks an SM
constexpr int VF_CHUNKS = 64;          // parts of a warp's span that the draw looks through

struct VerifyArgs {
    const float *target, *draft;       // draft null: point masses
    const int32_t *tokens, *parents, *token_start;
    const float *u_accept, *u_sample;
    int64_t N, V;
    int max_path;
    int32_t *path, *accept_len, *next_token;
    uint32_t *status;
};

// max(x, 0) that keeps a NaN, so that a sum over it shows it.
__device__ __forceinline__ double positive(double x) { return x < 0.0 ? 0.0 : x; }

// Residual weights of the current node after its rejections.
struct Residual {
    const float *p, *q;                // target and draft row (q null: point masses)
    const double *inv;                 // 1 / Z before each rejection
    const int32_t *gone;               // rejected tokens
    int n;                             // rejections
    __device__ __forceinline__ double of(float pv, float qv, int v) const
    {
        double r = pv;
        for (int k = 0; k < n; ++k) r = positive(r * inv[k] - (q ? (double)qv : gone[k] == v ? 1.0 : 0.0));
        return r;
    }
    // Four elements v .. v + 3, from their target and draft values.
    __device__ __forceinline__ void of4(const float4 &pv, const float4 &qv, int v, double (&r)[4]) const
    {
        r[0] = pv.x; r[1] = pv.y; r[2] = pv.z; r[3] = pv.w;
        if (n == 0) return;
        double qd[4] = {qv.x, qv.y, qv.z, qv.w};
        double f = inv[0];
#pragma unroll 1
        for (int k = 0;;) {
            if (!q) {
                const int x = gone[k] - v;
#pragma unroll
                for (int j = 0; j < 4; ++j) qd[j] = x == j ? 1.0 : 0.0;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) r[j] = positive(r[j] * f - qd[j]);
            if (++k == n) break;
            f = inv[k];
        }
    }
    // Target and draft values of the four elements 4 c - skew .. (0 outside the row).  `skew`
    // aligns the 16-byte loads: a row starts at any element.
    __device__ __forceinline__ void load(int c, int skew, int groups, int V, float4 &pv, float4 &qv) const
    {
        const int v = 4 * c - skew;
        qv = make_float4(0.f, 0.f, 0.f, 0.f);
        if (c > 0 && c + 1 < groups) {
            pv = *reinterpret_cast<const float4 *>(p + v);
            if (q && n > 0) qv = *reinterpret_cast<const float4 *>(q + v);
            return;
        }
        float a[4], b[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const bool in = v + j >= 0 && v + j < V;
            a[j] = in ? p[v + j] : 0.f;
            b[j] = in && q && n > 0 ? q[v + j] : 0.f;
        }
        pv = make_float4(a[0], a[1], a[2], a[3]);
        qv = make_float4(b[0], b[1], b[2], b[3]);
    }
    __device__ __forceinline__ void four(int c, int skew, int groups, int V, double (&r)[4]) const
    {
        float4 pv, qv;
        load(c, skew, groups, V, pv, qv);
        of4(pv, qv, 4 * c - skew, r);
    }
};

__device__ __forceinline__ double warp_sum_of(double s)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}

__global__ void __launch_bounds__(VF_THREADS, 2)
verify_tree_kernel(const VerifyArgs a)
{
    extern __shared__ float4 ring[];           // [place][target, draft][thread]
    cg::cluster_group cluster = cg::this_cluster();
    __shared__ int32_t parent[DSA_MAX_TREE], token[DSA_MAX_TREE], gone[DSA_MAX_TREE];
    __shared__ float chance[DSA_MAX_TREE], p_at[DSA_MAX_TREE], q_at[DSA_MAX_TREE];
    __shared__ double inv[DSA_MAX_TREE];
    __shared__ double warp_sum[VF_WARPS];
    __shared__ double chunk_sum[VF_CHUNKS];
    __shared__ double block_sum[2][8];         // of every block of the cluster, written by them
    __shared__ int pick;                       // chunk that holds the drawn element, -1: none
    __shared__ double pick_before;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int blocks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int b = blockIdx.x / blocks;
    grid_dep_wait();
    const int64_t t0 = a.token_start[b], t1 = a.token_start[b + 1];
    const int64_t n64 = t1 - t0;
    const bool sane = t0 >= 0 && n64 >= 0 && t1 <= a.N && n64 <= DSA_MAX_TREE;
    int32_t *path = a.path + (int64_t)b * a.max_path;
    const bool writer = rank == 0;
    if (!sane || n64 == 0) {                   // the same in every block of the cluster
        if (writer) {
            for (int i = tid; i < a.max_path; i += VF_THREADS) path[i] = -1;
            if (tid == 0) {
                a.accept_len[b] = 0;
                a.next_token[b] = -1;
                if (!sane && a.status) atomicCAS(a.status, (uint32_t)DSA_OK, (uint32_t)DSA_ERR_INVALID_ARG);
            }
        }
        return;
    }
    const int n = (int)n64, V = (int)a.V;
    if (tid < n) {
        // the entries that acceptance looks at, all at once: each child's own in its parent's rows
        const int par = a.parents[t0 + tid], x = a.tokens[t0 + tid];
        parent[tid] = par;
        token[tid] = x;
        chance[tid] = a.u_accept[t0 + tid];
        const bool seen = par >= 0 && par < tid && x >= 0 && x < V;
        const int64_t at = (t0 + par) * V + x;
        p_at[tid] = seen ? a.target[at] : 0.f;
        q_at[tid] = seen && a.draft ? a.draft[at] : 1.f;
    }
    const double u_sample = a.u_sample[b];
    cluster.sync();                            // every block of the cluster runs: its shared memory may be written

    int parity = 0;
    Residual R{};
    R.inv = inv;
    R.gone = gone;
    int skew = 0, groups = 0;
    int c_begin = 0, c_end = 0;                // this warp's span, in groups of four
    auto move_to = [&](int node) {
        const int64_t at = (t0 + node) * V;
        R.p = a.target + at;
        R.q = a.draft ? a.draft + at : nullptr;
        R.n = 0;
        skew = (int)(at & 3);
        groups = (int)(((int64_t)V + skew + 3) / 4);
        const int spans = blocks * VF_WARPS;
        const int span = (groups + spans - 1) / spans;
        c_begin = min(groups, (rank * VF_WARPS + warp) * span);
        c_end = min(groups, c_begin + span);
    };
    // Sum of R over the row, the same in every thread of the cluster.
    auto sum_row = [&]() -> double {
        double s0 = 0.0;
        // The first and last group of the row may be cut: the ring takes the others.  Each lane brings its own
        // groups into its own places, VF_DEPTH - 1 ahead.
        const int lo = max(c_begin, 1), hi = min(c_end, groups - 1);
        const bool two = R.q && R.n > 0;
        const float *pp = R.p + (4 * (lo + lane) - skew), *qp = two ? R.q + (4 * (lo + lane) - skew) : pp;
        int left = hi - lo - lane;             // this lane has a group while above 0, and the next every 32
        constexpr int kPlace = 2 * VF_THREADS; // float4s from one place to the next
        float4 *const mine = ring + tid;
#pragma unroll
        for (int d = 0; d < VF_DEPTH - 1; ++d) {
            if (left > 32 * d) {
                cp_async_16(mine + d * kPlace, pp + 128 * d, true);
                if (two) cp_async_16(mine + d * kPlace + VF_THREADS, qp + 128 * d, true);
            }
            cp_async_commit();
        }
        int v = 4 * (lo + lane) - skew;
        float4 *now = mine, *then = mine + (VF_DEPTH - 1) * kPlace;    // `then`: read a turn ago
#pragma unroll 1
        for (; left > 0; left -= 32, v += 128, pp += 128, qp += 128) {
            cp_async_wait<VF_DEPTH - 2>();
            const float4 pv = now[0], qv = now[VF_THREADS];
            if (left > 32 * (VF_DEPTH - 1)) {
                cp_async_16(then, pp + 128 * (VF_DEPTH - 1), true);
                if (two) cp_async_16(then + VF_THREADS, qp + 128 * (VF_DEPTH - 1), true);
            }
            cp_async_commit();
            then = now;
            now = now == mine + (VF_DEPTH - 1) * kPlace ? mine : now + kPlace;
            double r[4];
            R.of4(pv, qv, v, r);
            s0 += (r[0] + r[1]) + (r[2] + r[3]);
        }
        cp_async_wait<0>();
        if (lane < 2) {
            const int c = lane == 0 ? 0 : groups - 1;
            if (c >= c_begin && c < c_end && (lane == 0 || groups > 1)) {
                double r[4];
                R.four(c, skew, groups, V, r);
                s0 += (r[0] + r[1]) + (r[2] + r[3]);
            }
        }
        const double s = warp_sum_of(s0);
        if (lane == 0) warp_sum[warp] = s;
        __syncthreads();
        if (tid < blocks) {
            double t = 0.0;
            for (int w = 0; w < VF_WARPS; ++w) t += warp_sum[w];
            *cluster.map_shared_rank(&block_sum[parity][rank], tid) = t;
        }
        cluster.sync();
        double t = 0.0;
        for (int r = 0; r < blocks; ++r) t += block_sum[parity][r];
        parity ^= 1;                           // the other copy: a slow block may still read this one
        return t;
    };

    int cur = 0, kept = 1;
    bool summed = false;                       // warp_sum and block_sum belong to R
    bool known = false;                        // Z is the sum of R
    double Z = 1.0, total = 0.0;
    double left = 1.0;                         // of the last sum over the row, since then
    move_to(0);
    if (writer && tid == 0) path[0] = 0;
    for (int i = 1; i < n && kept < a.max_path; ++i) {
        if (parent[i] != cur) continue;
        const int x = token[i];
        if (x < 0 || x >= V) {
            if (writer && tid == 0 && a.status)
                atomicCAS(a.status, (uint32_t)DSA_OK, (uint32_t)DSA_ERR_INVALID_ARG);
            continue;
        }
        if ((double)chance[i] * (double)q_at[i] * Z < R.of(p_at[i], q_at[i], x)) {
            cur = i;
            move_to(i);
            Z = 1.0;
            summed = known = false;
            if (writer && tid == 0) path[kept] = i;
            ++kept;
            continue;
        }
        const double f = 1.0 / Z, r_x = R.of(p_at[i], q_at[i], x);
        __syncthreads();                       // every thread has read inv and gone
        if (tid == 0) {
            inv[R.n] = f;
            gone[R.n] = x;
        }
        __syncthreads();
        ++R.n;
        if (!R.q && known) {
            // A point mass changes one entry, and the sum follows from it without a pass.  That takes a part of
            // the sum away and scales the rest back to one, the sum's error with it: each rejection multiplies the
            // relative error by 1 / s.  So it is the product since the last pass that has to stay near one, and
            // where less than an eighth is left the row is summed again: a rounding since then counts up to eight
            // times in the sum.
            const double s = (Z - r_x) * f + fmax(r_x * f - 1.0, 0.0);
            if (left * s >= 0.125) {
                left *= s;
                Z = s;
                summed = false;
                continue;
            }
        }
        const double s = sum_row();
        if (s > 0.0) {
            Z = total = s;
            left = 1.0;
            summed = known = true;
        } else {
            --R.n;                             // nothing would be left: R stays
            summed = false;
        }
    }
    if (!summed) total = sum_row();

    // ---- draw: the block, the warp's span, then the chunk of it that holds the target value
    const double goal = u_sample * total;
    const bool drawable = total > 0.0 && total <= 1.7976931348623157e308;
    const int pr = parity ^ 1;
    if (writer) {
        for (int i = kept + tid; i < a.max_path; i += VF_THREADS) path[i] = -1;
        if (tid == 0) {
            a.accept_len[b] = kept;
            if (!drawable) {
                a.next_token[b] = -1;
                if (a.status) atomicCAS(a.status, (uint32_t)DSA_OK, (uint32_t)DSA_ERR_INVALID_ARG);
            }
        }
    }
    // The first of `count` sums that takes the running sum past the goal; if rounding leaves none, the
    // last with weight.  `before`: the running sum in front of it.
    auto find = [&](const double *sums, int count, double &before) {
        int at = -1, last = -1;
        double t = before, t_at = before, t_last = before;
        for (int r = 0; r < count && at < 0; ++r) {
            const double s = sums[r];
            if (s > 0.0) { last = r; t_last = t; }
            if (t + s > goal) { at = r; t_at = t; }
            t += s;
        }
        before = at >= 0 ? t_at : t_last;
        return at >= 0 ? at : last;
    };
    if (drawable) {
        double before = 0.0;
        if (find(block_sum[pr], blocks, before) == rank) {     // the same in the whole block
            const int w = find(warp_sum, VF_WARPS, before);
            const int spans = blocks * VF_WARPS, span = (groups + spans - 1) / spans;
            const int first = min(groups, (rank * VF_WARPS + w) * span), stop = min(groups, first + span);
            // its span again, by all warps: sums of chunks of whole warps
            const int step = 32 * ((span + 32 * VF_CHUNKS - 1) / (32 * VF_CHUNKS));
            const int chunks = (stop - first + step - 1) / step;
            for (int k = warp; k < chunks; k += VF_WARPS) {
                double s = 0.0;
                for (int c = first + k * step + lane; c < min(stop, first + (k + 1) * step); c += 32) {
                    double r[4];
                    R.four(c, skew, groups, V, r);
                    s += (r[0] + r[1]) + (r[2] + r[3]);
                }
                s = warp_sum_of(s);
                if (lane == 0) chunk_sum[k] = s;
            }
            __syncthreads();
            if (tid == 0) {
                pick = find(chunk_sum, chunks, before);
                pick_before = before;
            }
            __syncthreads();
            if (warp == 0) {
                int found = -1, heaviest = -1;                 // heaviest: the last element with weight
                double run = pick_before;
                const int from = first + pick * step, to = min(stop, from + step);
                for (int c0 = from; c0 < to && found < 0; c0 += 32) {
                    double r[4] = {0.0, 0.0, 0.0, 0.0};
                    if (c0 + lane < to) R.four(c0 + lane, skew, groups, V, r);
                    const double mine = (r[0] + r[1]) + (r[2] + r[3]);
                    double upto = mine;
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const double p = __shfl_up_sync(0xffffffffu, upto, o);
                        if (lane >= o) upto += p;
                    }
                    // the first weight in this lane that passes the goal, and the last one at all
                    int hit = -1, any = -1;
                    double at = run + (upto - mine);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        at += r[j];
                        const int v = 4 * (c0 + lane) - skew + j;
                        if (hit < 0 && r[j] > 0.0 && at > goal) hit = v;
                        if (r[j] > 0.0) any = v;
                    }
                    const unsigned hits = __ballot_sync(0xffffffffu, hit >= 0);
                    if (hits) found = __shfl_sync(0xffffffffu, hit, __ffs(hits) - 1);
                    const unsigned some = __ballot_sync(0xffffffffu, any >= 0);
                    if (some) heaviest = __shfl_sync(0xffffffffu, any, 31 - __clz(some));
                    run += __shfl_sync(0xffffffffu, upto, 31);
                }
                if (lane == 0) a.next_token[b] = found >= 0 ? found : heaviest;
            }
        }
    }
    cluster.sync();                            // no block leaves while another may write its sums
}

}  // namespace

cudaError_t launch_verify_tree(const float *target, const float *draft, const int32_t *tokens, const int32_t *parents,
                               const int32_t *token_start, const float *u_accept, const float *u_sample, int B,
                               int64_t N, int64_t V, int max_path, int32_t *path, int32_t *accept_len,
                               int32_t *next_token, uint32_t *status, cudaStream_t st)
{
    const VerifyArgs a{target, draft, tokens, parents, token_start, u_accept, u_sample, N, V, max_path,
                       path, accept_len, next_token, status};
    // blocks of a sequence: so many that all fill the GPU one and a half times (two of 512 threads are
    // resident on an SM).  Most sequences need one pass over their rows and leave early: 40 trees of 16
    // over 128001 tokens 64 us with one filling at most, 47 with one and a half or two; 64 such trees with two
    // fillings 54 instead of 46
    int blocks = 8;
    while (blocks > 1 && (int64_t)B * blocks > 148 * 3) blocks /= 2;
    static std::atomic<uint64_t> ready{0};     // devices whose kernel may use the ring
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0ull;
    if (!(ready.load(std::memory_order_acquire) & bit)) {
        e = cudaFuncSetAttribute(verify_tree_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, VF_RING);
        if (e != cudaSuccess) return e;
        ready.fetch_or(bit, std::memory_order_release);
    }
    return launch_cluster(verify_tree_kernel, (unsigned)B, (unsigned)blocks, VF_THREADS, VF_RING, st, a);
}

}  // namespace dsa
