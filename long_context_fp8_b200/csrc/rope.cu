// Rotary positions of queries and keys.
//
// Pair i of a head is turned by angle = 2 pi * frac(p * t_i), t_i the turns per
// position.  The host gives t_i as a 64-bit fixed-point fraction of a turn, so
// p * t_i mod 1 is one wrapping 64-bit product: exact for any position (a
// product in fp32 is off by 0.06 rad at position 2^20).  Its upper 32 bits
// are the angle in units of 2^-32 turns: the nearest quarter turn, taken out
// exactly, and a rest that sincospif takes in half turns.
//
// One pass: every element is read and written once, 16 bytes a thread (bf16),
// so HBM bounds it.  A block takes the heads of a few tokens: it first puts the
// cosines and sines of those tokens in shared memory (rot_dim / 2 pairs a token,
// shared by all heads), then works through units of eight elements (or of two
// groups of eight that belong together, in the half layout), four a thread in
// flight.
// Measured on one B200: see the launch function.
#include "kernels.h"

namespace dsa {
namespace {

constexpr int RP_THREADS = 256;
constexpr int RP_TABLE = 4096;         // (cos, sin) pairs of a block: 32 KB of shared memory

struct RopeTensor {
    const void *in;
    void *out;
    int64_t in_stride, out_stride;     // elements between tokens
    int H;
};

struct RopeArgs {
    RopeTensor x[2];                   // q, k
    const int32_t *positions;
    int64_t rows;
    int d, begin, half;                // half: pairs of a head
    int copy_units;                    // copied units of one head
    int rot_all, head_units;           // rotated units of all heads, and all units, of one token
    // i / n = i * mul >> 32 for n units of a head (all, rotated, copied), exact while i * n < 2^32
    uint64_t head_mul, rot_mul, copy_mul;
    int tokens;                        // tokens of a block
    int per_block;                     // units of one token that one block takes
    float factor;                      // attn_factor
    float sign;                        // -1: inverse
    uint64_t turns[128];
};

// Eight elements as fp32.
template <typename T> struct Vec8;
template <> struct Vec8<uint16_t> {
    uint4 a;
    __device__ __forceinline__ void load(const uint16_t *p) { a = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ void store(uint16_t *p) const { *reinterpret_cast<uint4 *>(p) = a; }
    __device__ __forceinline__ void get(float (&f)[8]) const
    {
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f[2 * j] = __uint_as_float(w[j] << 16);
            f[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
        }
    }
    __device__ __forceinline__ void set(const float (&f)[8])
    {
        a = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                       pack_bf16x2(f[6], f[7]));
    }
};
template <> struct Vec8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *p)
    {
        a = reinterpret_cast<const float4 *>(p)[0];
        b = reinterpret_cast<const float4 *>(p)[1];
    }
    __device__ __forceinline__ void store(float *p) const
    {
        reinterpret_cast<float4 *>(p)[0] = a;
        reinterpret_cast<float4 *>(p)[1] = b;
    }
    __device__ __forceinline__ void get(float (&f)[8]) const
    {
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    }
    __device__ __forceinline__ void set(const float (&f)[8])
    {
        a = make_float4(f[0], f[1], f[2], f[3]);
        b = make_float4(f[4], f[5], f[6], f[7]);
    }
};

// One unit: where it lies, what it has read.
template <typename T> struct RopeUnit {
    const T *in;                       // its first eight elements
    T *out;
    const float2 *cs;                  // cosine and sine of its first pair, or null: copied
    bool live;
    Vec8<T> lo, hi;
};

// INTERLEAVED: a unit is eight elements, four pairs (or a copied eight).  Half
// layout: a rotated unit is elements i .. i + 7 of both halves, eight pairs.
// Within a head the rotated part comes first, then the elements before and behind it; the half layout
// takes all rotated units before the copied ones (8192 x 129 heads bf16: 119 us head by head, 108 so; the
// interleaved layout 13.0 and 16.2 at 1024 x 129).
template <typename T, bool INTERLEAVED, bool COPY>
__global__ void __launch_bounds__(RP_THREADS)
rope_kernel(const __grid_constant__ RopeArgs a)
{
    constexpr int U = 4;
    extern __shared__ float2 table[];  // [tokens][half]
    const int64_t row0 = (int64_t)blockIdx.x * a.tokens;
    const int rows = (int)min((int64_t)a.tokens, a.rows - row0);
    const int rot_units = INTERLEAVED ? a.half / 4 : a.half / 8;
    grid_dep_wait();
    // A thread keeps to one pair: its turns are read once (from constant memory, where lanes that read
    // different words take turns).
    const int at_once = RP_THREADS / a.half, pair = threadIdx.x % a.half;
    const uint64_t turns = a.turns[pair];
    for (int r = threadIdx.x / a.half; r < rows; r += at_once) {
        if ((int)threadIdx.x >= at_once * a.half) break;
        const uint64_t phase = (uint64_t)(int64_t)a.positions[row0 + r] * turns;
        // the nearest quarter turn, and the rest (at most 1/8 turn, 2^-27 half turns as a float)
        const uint32_t angle = (uint32_t)(phase >> 32), quarter = (angle + 0x20000000u) >> 30;
        float s0, c0;
        sincospif((float)(int32_t)(angle - (quarter << 30)) * 0x1p-31f, &s0, &c0);
        float s = quarter & 1 ? c0 : s0, c = quarter & 1 ? -s0 : c0;
        if (quarter & 2) { s = -s; c = -c; }
        table[r * a.half + pair] = make_float2(c * a.factor, s * a.factor * a.sign);
    }
    __syncthreads();
    const int begin = blockIdx.y * a.per_block, end = min(a.head_units, begin + a.per_block);
    const int per = end - begin, total = rows * per;
    for (int i0 = threadIdx.x; i0 < total; i0 += RP_THREADS * U) {
        RopeUnit<T> u[U];
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const int i = i0 + j * RP_THREADS;
            u[j].live = i < total;
            if (!u[j].live) continue;
            const int r = a.tokens == 1 ? 0 : i / per;
            int w = begin + i - r * per;
            bool rot = true;
            int h, c;
            if (INTERLEAVED) {         // head by head: all units are alike
                h = (int)(((uint64_t)(uint32_t)w * a.head_mul) >> 32);
                c = w - h * (rot_units + a.copy_units);
                if (COPY && c >= rot_units) { rot = false; c -= rot_units; }
            } else {                   // rotated units of all heads, then copied ones: a warp seldom has both
                rot = !COPY || w < a.rot_all;
                if (!rot) w -= a.rot_all;
                h = (int)(((uint64_t)(uint32_t)w * (rot ? a.rot_mul : a.copy_mul)) >> 32);
                c = w - h * (rot ? rot_units : a.copy_units);
            }
            int e = a.begin + c * 8;
            u[j].cs = table + r * a.half + c * (INTERLEAVED ? 4 : 8);
            if (!rot) {
                u[j].cs = nullptr;
                e = c * 8;
                if (e >= a.begin) e += 2 * a.half;
            }
            const bool is_k = h >= a.x[0].H;
            if (is_k) h -= a.x[0].H;
            const int64_t at = (int64_t)h * a.d + e;
            u[j].in = static_cast<const T *>(is_k ? a.x[1].in : a.x[0].in) +
                      (row0 + r) * (is_k ? a.x[1].in_stride : a.x[0].in_stride) + at;
            u[j].out = static_cast<T *>(is_k ? a.x[1].out : a.x[0].out) +
                       (row0 + r) * (is_k ? a.x[1].out_stride : a.x[0].out_stride) + at;
            u[j].lo.load(u[j].in);
            if (!INTERLEAVED && u[j].cs) u[j].hi.load(u[j].in + a.half);
        }
#pragma unroll
        for (int j = 0; j < U; ++j) {
            if (!u[j].live) continue;
            if (!COPY || u[j].cs) {
                float x[8], y[8];
                u[j].lo.get(x);
                if (INTERLEAVED) {
#pragma unroll
                    for (int p = 0; p < 4; ++p) {
                        const float2 t = u[j].cs[p];
                        y[2 * p] = x[2 * p] * t.x - x[2 * p + 1] * t.y;
                        y[2 * p + 1] = x[2 * p + 1] * t.x + x[2 * p] * t.y;
                    }
                } else {
                    float z[8];
                    u[j].hi.get(y);
#pragma unroll
                    for (int p = 0; p < 8; ++p) {
                        const float2 t = u[j].cs[p];
                        z[p] = y[p] * t.x + x[p] * t.y;
                        y[p] = x[p] * t.x - y[p] * t.y;
                    }
                    u[j].hi.set(z);
                    u[j].hi.store(u[j].out + a.half);
                }
                u[j].lo.set(y);
            }
            u[j].lo.store(u[j].out);
        }
    }
}

template <typename T>
cudaError_t launch_rope_t(const RopeArgs &a, bool interleaved, bool copy, dim3 grid, size_t smem, cudaStream_t st)
{
    auto kernel = interleaved ? (copy ? rope_kernel<T, true, true> : rope_kernel<T, true, false>)
                              : (copy ? rope_kernel<T, false, true> : rope_kernel<T, false, false>);
    const cudaError_t e = launch_chained(kernel, grid, dim3(RP_THREADS), smem, st, a);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace

cudaError_t launch_rope(const void *q, int64_t q_stride, int H_q, const void *k, int64_t k_stride, int H_k,
                        const int32_t *positions, int64_t rows, int d, int rot_begin, int rot_dim, bool interleaved,
                        const uint64_t *turns, float factor, bool inverse, void *q_out, int64_t q_out_stride,
                        void *k_out, int64_t k_out_stride, bool bf16, cudaStream_t st)
{
    RopeArgs a{};
    a.x[0] = {q, q_out, q_stride, q_out_stride, H_q};
    a.x[1] = {k, k_out, k_stride, k_out_stride, H_k};
    a.positions = positions;
    a.rows = rows;
    a.d = d;
    a.begin = rot_begin;
    a.half = rot_dim / 2;
    a.factor = factor;
    a.sign = inverse ? -1.f : 1.f;
    for (int i = 0; i < rot_dim / 2; ++i) a.turns[i] = turns[i];
    // in place, the elements that are not rotated need no pass
    const bool copy = rot_dim < d && !(q_out == q && (H_k == 0 || k_out == k));
    const int rot_units = interleaved ? rot_dim / 8 : rot_dim / 16, heads = H_q + H_k;
    a.copy_units = copy ? (d - rot_dim) / 8 : 0;
    a.head_mul = ((uint64_t)1 << 32) / (rot_units + a.copy_units) + 1;
    a.rot_mul = ((uint64_t)1 << 32) / rot_units + 1;
    a.copy_mul = copy ? ((uint64_t)1 << 32) / a.copy_units + 1 : 0;
    a.rot_all = rot_units * heads;
    a.head_units = a.rot_all + a.copy_units * heads;
    // a block takes about 4096 units (four rounds of 4 a thread; 16K x 65 heads fp32 194 us with 2048, 177
    // with 4096, 181 with 8192, whose few large blocks cost 1024 x 129 heads 4 us more): the tokens that
    // make them up, or a part of one token
    constexpr int kUnits = 4096;
    int tokens = kUnits / a.head_units;
    tokens = tokens < RP_TABLE / a.half ? tokens : RP_TABLE / a.half;
    a.tokens = tokens > 1 ? tokens : 1;
    a.per_block = a.head_units;
    if (a.head_units > kUnits) a.per_block = (int)ceil_div(a.head_units, ceil_div(a.head_units, kUnits));
    // few tokens: smaller blocks, so that every SM has some
    while (a.tokens > 1 && ceil_div(rows, a.tokens) < 2 * 148) a.tokens = (a.tokens + 1) / 2;
    while (a.tokens == 1 && a.per_block > RP_THREADS && rows * ceil_div(a.head_units, a.per_block) < 4 * 148)
        a.per_block = (a.per_block + 1) / 2;
    const int64_t blocks = ceil_div(rows, a.tokens);
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    const dim3 grid((unsigned)blocks, (unsigned)ceil_div(a.head_units, a.per_block));
    const size_t smem = sizeof(float2) * (size_t)a.tokens * a.half;
    return bf16 ? launch_rope_t<uint16_t>(a, interleaved, copy, grid, smem, st)
                : launch_rope_t<float>(a, interleaved, copy, grid, smem, st);
}

}  // namespace dsa
