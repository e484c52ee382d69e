// Verification of drafted token trees against the target's probabilities.
//
// Along the walk almost nothing is read: a child is accepted or rejected on one
// entry of its parent's target and draft rows.  Only a rejection sums a whole row
// (Z = sum_v max(R(v) / Z - Q(v), 0)), and the last one is drawn from.  So a
// sequence reads, besides single entries, one pair of rows for each rejection, or
// the last node's target row alone if no child was left to reject.
//
// A cluster of thread blocks takes a sequence.  Every block runs the same walk from
// the same values; a row is cut into contiguous spans, one a warp, and each warp
// sums its span in 64 bits.  The warps' sums are kept: the draw finds the span by
// their running sum and only that warp goes through its span again.  Sums have a
// fixed order, so a call repeats bit for bit.  R is never stored: it is made again
// from P and Q, rejection by rejection, in registers (a node has few rejections, and
// the second row pass finds P and Q in L2).
#include <cooperative_groups.h>

#include "kernels.h"

namespace dsa {
namespace {

namespace cg = cooperative_groups;

constexpr int VF_THREADS = 512;
constexpr int VF_WARPS = VF_THREADS / 32;
constexpr int VF_STEP = 128;           // elements a warp takes at a time (four a lane)

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
    __device__ __forceinline__ double of(float pv, float qv, int64_t v) const
    {
        double r = pv;
        if (q) {
            for (int k = 0; k < n; ++k) r = positive(r * inv[k] - (double)qv);
        } else {
            for (int k = 0; k < n; ++k) r = positive(r * inv[k] - (gone[k] == v ? 1.0 : 0.0));
        }
        return r;
    }
    __device__ __forceinline__ double at(int64_t v) const { return of(p[v], q ? q[v] : 0.f, v); }
    // Weights of elements 4 c - skew .. 4 c - skew + 3 (0 outside the row).  `skew`
    // aligns the 16-byte loads: a row starts at any element.
    __device__ __forceinline__ void four(int64_t c, int skew, int64_t V, double (&r)[4]) const
    {
        const int64_t v = 4 * c - skew;
        float pv[4] = {0.f, 0.f, 0.f, 0.f}, qv[4] = {0.f, 0.f, 0.f, 0.f};
        if (v >= 0 && v + 4 <= V) {
            const float4 a = *reinterpret_cast<const float4 *>(p + v);
            pv[0] = a.x; pv[1] = a.y; pv[2] = a.z; pv[3] = a.w;
            if (q && n > 0) {
                const float4 b = *reinterpret_cast<const float4 *>(q + v);
                qv[0] = b.x; qv[1] = b.y; qv[2] = b.z; qv[3] = b.w;
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (v + j < 0 || v + j >= V) continue;
                pv[j] = p[v + j];
                if (q && n > 0) qv[j] = q[v + j];
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) r[j] = of(pv[j], qv[j], v + j);
    }
};

__global__ void __launch_bounds__(VF_THREADS)
verify_tree_kernel(const VerifyArgs a)
{
    cg::cluster_group cluster = cg::this_cluster();
    __shared__ int32_t parent[DSA_MAX_TREE], token[DSA_MAX_TREE], gone[DSA_MAX_TREE];
    __shared__ float chance[DSA_MAX_TREE];
    __shared__ double inv[DSA_MAX_TREE];
    __shared__ double warp_sum[VF_WARPS];
    __shared__ double block_sum[2][8];         // of every block of the cluster, written by them
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
    const int n = (int)n64;
    if (tid < n) {
        parent[tid] = a.parents[t0 + tid];
        token[tid] = a.tokens[t0 + tid];
        chance[tid] = a.u_accept[t0 + tid];
    }
    cluster.sync();                            // every block of the cluster runs: its shared memory may be written

    const int64_t V = a.V;
    int parity = 0;
    Residual R{};
    R.inv = inv;
    R.gone = gone;
    int skew = 0;
    int64_t c_begin = 0, c_end = 0;            // this warp's span, in groups of four
    auto move_to = [&](int node) {
        const int64_t at = (t0 + node) * V;
        R.p = a.target + at;
        R.q = a.draft ? a.draft + at : nullptr;
        R.n = 0;
        skew = (int)(at & 3);
        const int64_t groups = (V + skew + 3) / 4;
        const int64_t span = ceil_div(groups, (int64_t)blocks * VF_WARPS * (VF_STEP / 4)) * (VF_STEP / 4);
        c_begin = min(groups, ((int64_t)rank * VF_WARPS + warp) * span);
        c_end = min(groups, c_begin + span);
    };
    // Sum of R over the row, the same in every thread of the cluster.
    auto sum_row = [&]() -> double {
        double s0 = 0.0, s1 = 0.0, s2 = 0.0, s3 = 0.0;
        int64_t c = c_begin + lane;
        for (; c + 96 < c_end; c += 128) {     // four groups a lane in flight
            double r0[4], r1[4], r2[4], r3[4];
            R.four(c, skew, V, r0);
            R.four(c + 32, skew, V, r1);
            R.four(c + 64, skew, V, r2);
            R.four(c + 96, skew, V, r3);
            s0 += (r0[0] + r0[1]) + (r0[2] + r0[3]);
            s1 += (r1[0] + r1[1]) + (r1[2] + r1[3]);
            s2 += (r2[0] + r2[1]) + (r2[2] + r2[3]);
            s3 += (r3[0] + r3[1]) + (r3[2] + r3[3]);
        }
        for (; c < c_end; c += 32) {
            double r[4];
            R.four(c, skew, V, r);
            s0 += (r[0] + r[1]) + (r[2] + r[3]);
        }
        double s = (s0 + s1) + (s2 + s3);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (lane == 0) warp_sum[warp] = s;
        __syncthreads();
        if (tid == 0) {
            double t = 0.0;
            for (int w = 0; w < VF_WARPS; ++w) t += warp_sum[w];
            for (int r = 0; r < blocks; ++r) *cluster.map_shared_rank(&block_sum[parity][rank], r) = t;
        }
        cluster.sync();
        double t = 0.0;
        for (int r = 0; r < blocks; ++r) t += block_sum[parity][r];
        parity ^= 1;                           // the other copy: a slow block may still read this one
        return t;
    };

    int cur = 0, kept = 1;
    bool summed = false;                       // warp_sum and block_sum belong to R
    double Z = 1.0, total = 0.0;
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
        const double qx = R.q ? (double)R.q[x] : 1.0;
        if ((double)chance[i] * qx * Z < R.at(x)) {
            cur = i;
            move_to(i);
            Z = 1.0;
            summed = false;
            if (writer && tid == 0) path[kept] = i;
            ++kept;
            continue;
        }
        __syncthreads();                       // every thread has read inv and gone
        if (tid == 0) {
            inv[R.n] = 1.0 / Z;
            gone[R.n] = x;
        }
        __syncthreads();
        ++R.n;
        const double s = sum_row();
        if (s > 0.0) {
            Z = total = s;
            summed = true;
        } else {
            --R.n;                             // nothing would be left: R stays
            summed = false;
        }
    }
    if (!summed) total = sum_row();

    // ---- draw: the block, then the warp, whose span holds the target value
    const double goal = (double)a.u_sample[b] * total;
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
    if (drawable) {
        // the first block whose running sum passes the goal; if rounding leaves none, the last with weight
        int blk = -1, last = 0;
        double before = 0.0, last_before = 0.0, t = 0.0;
        for (int r = 0; r < blocks; ++r) {
            const double s = block_sum[pr][r];
            if (s > 0.0) { last = r; last_before = t; }
            if (blk < 0 && t + s > goal) { blk = r; before = t; }
            t += s;
        }
        if (blk < 0) { blk = last; before = last_before; }
        if (blk == rank) {
            int w = -1;
            last = 0;
            t = last_before = before;
            double w_before = before;
            for (int k = 0; k < VF_WARPS; ++k) {
                const double s = warp_sum[k];
                if (s > 0.0) { last = k; last_before = t; }
                if (w < 0 && t + s > goal) { w = k; w_before = t; }
                t += s;
            }
            if (w < 0) { w = last; w_before = last_before; }
            if (w == warp) {
                int64_t found = -1, heaviest = -1;     // heaviest: the last element with weight
                double run = w_before;
                for (int64_t c0 = c_begin; c0 < c_end && found < 0; c0 += 32) {
                    double r[4] = {0.0, 0.0, 0.0, 0.0};
                    if (c0 + lane < c_end) R.four(c0 + lane, skew, V, r);
                    const double mine = (r[0] + r[1]) + (r[2] + r[3]);
                    double upto = mine;
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const double p = __shfl_up_sync(0xffffffffu, upto, o);
                        if (lane >= o) upto += p;
                    }
                    // the first weight in this lane that passes the goal, and the last one at all
                    int64_t hit = -1, any = -1;
                    double at = run + (upto - mine);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        at += r[j];
                        const int64_t v = 4 * (c0 + lane) - skew + j;
                        if (hit < 0 && r[j] > 0.0 && at > goal) hit = v;
                        if (r[j] > 0.0) any = v;
                    }
                    const unsigned hits = __ballot_sync(0xffffffffu, hit >= 0);
                    if (hits) found = __shfl_sync(0xffffffffu, hit, __ffs(hits) - 1);
                    const unsigned some = __ballot_sync(0xffffffffu, any >= 0);
                    if (some) heaviest = __shfl_sync(0xffffffffu, any, 31 - __clz(some));
                    run += __shfl_sync(0xffffffffu, upto, 31);
                }
                if (lane == 0) a.next_token[b] = (int32_t)(found >= 0 ? found : heaviest);
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
    // blocks of a sequence: as many as let all of them be resident at once (four of
    // 512 threads an SM), so that a row is read by as many SMs as there are
    int blocks = 8;
    while (blocks > 1 && (int64_t)B * blocks > 148 * 4) blocks /= 2;
    return launch_cluster(verify_tree_kernel, (unsigned)B, (unsigned)blocks, VF_THREADS, st, a);
}

}  // namespace dsa
