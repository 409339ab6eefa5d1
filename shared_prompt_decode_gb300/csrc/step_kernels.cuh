// Device code of the steps around the cache: block tables and slot maps from
// the request lengths, the return of finished requests' blocks, and rotary
// positions with several axes.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "relay_kernels.cuh"

namespace relay {

enum : unsigned { FLAG_POOL = 32u };

constexpr int CTRL_STEP_TICKET = 6;      // ctrl word: CTAs that have read the free count
constexpr int kStepThreads = kMaxB;      // one thread per request in the scans

// ----------------------------------------------------------------------------- block plan
// The blocks of a growing batch, from one exclusive scan over the requests:
// request b holds ceil((n - q) / 16) blocks and needs ceil(n / 16) of them;
// the missing ones come from the top of the free list in request order.  Every
// CTA repeats the scan (two loads a request, no traffic between CTAs) and
// then covers its share of the B x Lq row slots.  A new block always starts
// with a new token, so the thread of that token writes the table entry, and a
// slot never waits on an entry that another thread writes: what the scan says
// is new is read from the free list.  One launch and three dependent reads
// bound it: 3.1 us for a decode step of 32 requests, 5.3 us for 512 requests of
// up to 1024 rows.
struct BlockPlan {
    int B, Lq, max_blocks, num_blocks;
    const int *ctx_lens, *q_lens, *free_blocks, *n_free;
    int *block_tables, *slot_map, *n_free_out;
    unsigned *flags, *ticket;
};

// Inclusive scan of one value per thread of a kStepThreads CTA.
__device__ __forceinline__ long long step_scan(long long v, long long *warp_sum)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const long long t = __shfl_up_sync(0xffffffffu, v, off);
        if (lane >= off) v += t;
    }
    if (lane == 31) warp_sum[warp] = v;
    __syncthreads();
    long long base = 0;
    for (int j = 0; j < warp; j++) base += warp_sum[j];
    return base + v;
}

// The free count, which one CTA may replace once every CTA has read it: the
// last CTA to pass here writes it (the caller may give one word for both).
__device__ __forceinline__ void publish_free(int *out, int value, unsigned *ticket)
{
    if (threadIdx.x == 0) {
        __threadfence();      // this CTA's read of the old count comes before its ticket
        // atomicInc wraps to zero after the last CTA: the word is ready for the next call
        if (gridDim.x == 1 || atomicInc(ticket, gridDim.x - 1) == gridDim.x - 1) *out = value;
    }
}

__global__ void __launch_bounds__(kStepThreads) block_plan_kernel(const __grid_constant__ BlockPlan a)
{
    __shared__ long long warp_sum[kStepThreads / 32];
    __shared__ int pos0[kMaxB], rows[kMaxB], held[kMaxB], top[kMaxB];
    __shared__ int total;
    const int tid = threadIdx.x;
    int n = 0, ql = 0, h = 0, need = 0;
    unsigned flags = 0;
    int nf = *a.n_free;
    if (nf < 0 || nf > a.num_blocks) {
        flags |= FLAG_POOL;
        nf = 0;
    }
    if (tid < a.B) {
        ql = a.q_lens ? a.q_lens[tid] : a.Lq;
        n = a.ctx_lens[tid];
        if (ql < 0 || ql > a.Lq) { flags |= FLAG_BAD_Q_LEN; ql = n = 0; }
        if (n < ql || n > (long long)a.max_blocks * kBlock) { flags |= FLAG_BAD_CTX_LEN; ql = n = 0; }
        h = (n - ql + kBlock - 1) / kBlock;
        need = (n + kBlock - 1) / kBlock - h;
    }
    if (tid == 0) total = 0;
    const long long end = step_scan(need, warp_sum);      // (a barrier: total is zero for everybody)
    const bool granted = end <= nf;
    if (!granted && need > 0) flags |= FLAG_POOL;
    if (tid < a.B) {
        pos0[tid] = n - ql;
        rows[tid] = granted || need == 0 ? ql : 0;
        held[tid] = h;
        top[tid] = (int)(nf - 1 - (granted ? end - need : 0));
        // needs are not negative: the granted requests are the first ones
        if (granted) atomicMax(&total, (int)end);
    }
    __syncthreads();
    if (flags && blockIdx.x == 0) atomicOr(a.flags, flags);
    publish_free(a.n_free_out, nf - total, a.ticket);

    const long long slots = (long long)a.B * a.Lq;
    for (long long idx = (long long)blockIdx.x * kStepThreads + tid; idx < slots;
         idx += (long long)gridDim.x * kStepThreads) {
        const int b = (int)(idx / a.Lq), i = (int)(idx - (long long)b * a.Lq);
        int slot = -1;
        if (i < rows[b]) {
            const int pos = pos0[b] + i, page = pos / kBlock;
            int *entry = a.block_tables + (size_t)b * a.max_blocks + page;
            int blk;
            if (page < held[b]) {
                blk = *entry;
            } else {
                blk = a.free_blocks[top[b] - (page - held[b])];
                if (pos % kBlock == 0) *entry = blk;
            }
            if (blk >= 0 && blk < a.num_blocks) slot = blk * kBlock + pos % kBlock;
            else atomicOr(a.flags, FLAG_BAD_BLOCK);
        }
        if (a.slot_map) a.slot_map[idx] = slot;
    }
}

// ----------------------------------------------------------------------------- block release
// The blocks of finished requests, appended to the free list in request
// order: the same scan, then one warp per 256 table entries (a few of a long
// table keep many lanes' loads in flight).  3.1 us for three of 32 requests,
// 4.8 us for 400 of 512 with up to 1024 blocks each.
struct BlockRelease {
    int B, max_blocks, num_blocks;
    const int *done, *ctx_lens, *block_tables, *n_free;
    int *free_blocks, *n_free_out;
    unsigned *flags, *ticket;
};
constexpr int kReleaseChunk = 256;

__global__ void __launch_bounds__(kStepThreads) block_release_kernel(const __grid_constant__ BlockRelease a)
{
    __shared__ long long warp_sum[kStepThreads / 32];
    __shared__ int count[kMaxB], first[kMaxB];
    __shared__ int total;
    const int tid = threadIdx.x, lane = tid & 31;
    unsigned flags = 0;
    int nf = *a.n_free, cnt = 0;
    const bool bad = nf < 0 || nf > a.num_blocks;
    if (bad) flags |= FLAG_POOL;
    if (tid < a.B && a.done[tid] != 0) {
        const int n = a.ctx_lens[tid];
        if (n < 0 || n > (long long)a.max_blocks * kBlock) flags |= FLAG_BAD_CTX_LEN;
        else cnt = (n + kBlock - 1) / kBlock;
    }
    if (tid == 0) total = 0;
    const long long end = step_scan(cnt, warp_sum);
    const bool fits = !bad && nf + end <= a.num_blocks;
    if (!fits && cnt > 0) flags |= FLAG_POOL;      // more blocks than the pool has
    if (tid < a.B) {
        count[tid] = fits ? cnt : 0;
        first[tid] = fits ? (int)(nf + end - cnt) : 0;
        if (fits) atomicMax(&total, (int)end);
    }
    __syncthreads();
    if (flags && blockIdx.x == 0) atomicOr(a.flags, flags);
    publish_free(a.n_free_out, nf + total, a.ticket);

    const int chunks = (a.max_blocks + kReleaseChunk - 1) / kReleaseChunk;
    const long long units = (long long)a.B * chunks;
    constexpr int kPer = kStepThreads / 32;
    for (long long u = (long long)blockIdx.x * kPer + (tid >> 5); u < units; u += (long long)gridDim.x * kPer) {
        const int b = (int)(u / chunks), j0 = (int)(u % chunks) * kReleaseChunk;
        const int *row = a.block_tables + (size_t)b * a.max_blocks;
#pragma unroll
        for (int k = 0; k < kReleaseChunk / 32; k++) {
            const int j = j0 + k * 32 + lane;
            if (j >= count[b]) continue;
            int blk = row[j];
            if (blk < 0 || blk >= a.num_blocks) {
                atomicOr(a.flags, FLAG_BAD_BLOCK);
                blk = -1;      // no block: the plan that would draw it reports it again
            }
            a.free_blocks[first[b] + j] = blk;
        }
    }
}

// ----------------------------------------------------------------------------- rotary positions, several axes
// Pair j of a head turns by (Ls + pos[axis(j)]) * base^(-2j / D).  The angle
// is formed in turns, as a 64-bit fixed-point fraction: turn[j] is base^(-2j
// / D) / (2 pi) times 2^64, and position times turn[j] modulo 2^64 is the
// fraction of a turn with no range reduction and no fp64 (positions are
// integers, so the wrap-around drops whole turns exactly).  A warp takes one
// token and `hpw` of its heads: it forms the D / 2 sines and cosines once,
// passes them through shared memory, and a lane then holds the eight pairs
// that it turns in every head (D / 16 lanes a head, two 16-byte loads each,
// kUnroll heads in flight).  Bound by memory: 45 us for 6872 tokens of 64 + 8
// heads (265 MB, 39.6 us at the copy rate); a decode step is a launch and two
// dependent reads.
struct RopeAxes {
    int B, Lq, H, Hkv, Ls, hpw;       // Hkv = 0 without k; hpw: heads of a warp
    unsigned long long turn[kMaxRopePairs];
    unsigned char axis[kMaxRopePairs];
    const __half *q, *k;
    __half *q_out, *k_out;
    const int *pos, *q_lens;          // pos [n_axes, B, Lq]
    unsigned *flags;
    int inverse;
};

constexpr int kRopeWarps = 4;

// two products and sums at a time (32-bit each, IEEE)
__device__ __forceinline__ float2 mul2(float2 a, float2 b)
{
    unsigned long long r, x = *reinterpret_cast<unsigned long long *>(&a), y = *reinterpret_cast<unsigned long long *>(&b);
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
    return *reinterpret_cast<float2 *>(&r);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    unsigned long long r, x = *reinterpret_cast<unsigned long long *>(&a), y = *reinterpret_cast<unsigned long long *>(&b);
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
    return *reinterpret_cast<float2 *>(&r);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    unsigned long long r, x = *reinterpret_cast<unsigned long long *>(&a), y = *reinterpret_cast<unsigned long long *>(&b),
                          z = *reinterpret_cast<unsigned long long *>(&c);
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
    return *reinterpret_cast<float2 *>(&r);
}

template <int D>
__global__ void __launch_bounds__(kRopeWarps * 32) rope_axes_kernel(const __grid_constant__ RopeAxes a)
{
    constexpr int kLanes = D / 16, kHeads = 32 / kLanes;      // lanes of a head, heads of a warp's pass
    constexpr int kUnroll = 3;
    __shared__ float2 cs[kRopeWarps][D / 2];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int tokens = a.B * a.Lq, tok = blockIdx.x * kRopeWarps + warp;
    if (tok >= tokens) return;
    const int nh = a.H + a.Hkv, h0 = blockIdx.y * a.hpw, h1 = min(h0 + a.hpw, nh);
    if (a.q_lens) {
        const int b = tok / a.Lq, i = tok - b * a.Lq;
        const int ql = a.q_lens[b];
        if (ql < 0 || ql > a.Lq) {
            if (lane == 0 && i == 0 && h0 == 0) atomicOr(a.flags, FLAG_BAD_Q_LEN);
            return;
        }
        if (i >= ql) return;
    }
#pragma unroll
    for (int j = lane; j < D / 2; j += 32) {
        const long long pos = (long long)a.Ls + a.pos[(size_t)a.axis[j] * tokens + tok];
        const unsigned long long f = (unsigned long long)pos * a.turn[j];
        float s, c;
        sincospif((float)(int)(f >> 32) * 0x1p-31f, &s, &c);      // half turns in [-1, 1)
        cs[warp][j] = make_float2(c, a.inverse ? -s : s);
    }
    __syncwarp();
    const int c = lane % kLanes;
    float2 co[4], si[4], ni[4];      // cosines, sines and negative sines of the lane's pairs, two by two
#pragma unroll
    for (int e = 0; e < 4; e++) {
        const float2 t0 = cs[warp][8 * c + 2 * e], t1 = cs[warp][8 * c + 2 * e + 1];
        co[e] = make_float2(t0.x, t1.x);
        si[e] = make_float2(t0.y, t1.y);
        ni[e] = make_float2(-t0.y, -t1.y);
    }
    for (int hb = h0 + lane / kLanes; hb < h1; hb += kUnroll * kHeads) {
        uint4 x[kUnroll], y[kUnroll];
        size_t off[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; u++) {
            const int h = hb + u * kHeads;
            if (h >= h1) continue;
            const bool isq = h < a.H;
            off[u] = (isq ? (size_t)tok * a.H + h : (size_t)tok * a.Hkv + (h - a.H)) * D + 8 * c;
            const __half *src = (isq ? a.q : a.k) + off[u];
            x[u] = *reinterpret_cast<const uint4 *>(src);
            y[u] = *reinterpret_cast<const uint4 *>(src + D / 2);
        }
#pragma unroll
        for (int u = 0; u < kUnroll; u++) {
            const int h = hb + u * kHeads;
            if (h >= h1) continue;
            __half *dst = (h < a.H ? a.q_out : a.k_out) + off[u];
            const unsigned xs[4] = {x[u].x, x[u].y, x[u].z, x[u].w}, ys[4] = {y[u].x, y[u].y, y[u].z, y[u].w};
            unsigned xo[4], yo[4];
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const float2 p = __half22float2(*reinterpret_cast<const __half2 *>(&xs[e]));
                const float2 r = __half22float2(*reinterpret_cast<const __half2 *>(&ys[e]));
                const float2 px = fma2(p, co[e], mul2(r, ni[e])), py = fma2(r, co[e], mul2(p, si[e]));
                xo[e] = pack_half2(px.x, px.y);
                yo[e] = pack_half2(py.x, py.y);
            }
            *reinterpret_cast<uint4 *>(dst) = make_uint4(xo[0], xo[1], xo[2], xo[3]);
            *reinterpret_cast<uint4 *>(dst + D / 2) = make_uint4(yo[0], yo[1], yo[2], yo[3]);
        }
    }
}

}  // namespace relay
