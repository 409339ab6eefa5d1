// Device code of the 4-bit context pool: the quantising append and the
// attention that reads it.
//
// One token of one KV head is D codes of 4 bits (two to a byte, the even
// dimension in the low half) in groups of GROUP dimensions; a group stands
// for s * code + z with an fp16 pair (s, z).
//
// The products never see s * code + z.  With the codes c_t of key t,
//     q . k_t     = sum_groups  s_t (q . c_t) + z_t sum(q)
//     sum p_t v_t = sum (p_t s_t) c_t + (sum p_t z_t),
// and a 4-bit code needs no conversion for the tensor cores: the bits of a
// code in the low bits of an fp16 word are the subnormal number code * 2^-24,
// and four bits higher code * 2^-20, both exact.  One AND makes two operand
// elements (one shift for every second pair of them), and the powers of two
// come off in fp32 at the end.  What is rounded below 32 bits is p_t s_t
// alone (fp16, like the weights of the fp16 path).  So that this rounding
// meets the value's distance from the middle of its range and not from the
// range's end, the sum is taken as
//     sum w_t (c_t - 8) + sum p_t (z_t + 8 s_t),   w_t = fp16(p_t s_t),
// whose - 8 sum w_t is one more product with the same weights (a row of
// codes 8).  Without it the error is three times as large on normal data.
// (Prompt chunks on the tensor cores are the exception: rows_kernel.)
#pragma once

#include <cuda_fp16.h>
#include <stddef.h>
#include <stdint.h>

#include "relay_kernels.cuh"
#include "step_kernels.cuh"
#include "sys_tc.cuh"

namespace relay {
namespace q4 {

struct Pool {
    const unsigned char *k, *v;      // codes [num_blocks, Hkv, 16, D / 2]
    const __half2 *ksz, *vsz;        // (s, z) [num_blocks, Hkv, 16, D / GROUP]
};

// ----------------------------------------------------------------------------- append
// s = fp16((max - min) / 15), z = min, code = rint((x - z) / s) clamped to
// 0..15, in fp32 with IEEE divisions; s = 0 has code 0, and a group with a NaN
// or an infinity stores s = z = NaN.  D / 32 lanes take one row of one KV
// head, K or V: with the instructions of a row's address, group and scale
// spread over 32 elements the kernel takes 39.6 us for K and V of 6872 rows of
// 32 heads (D = 128, groups of 64; 149 MB, 22 us at the copy rate): what is
// left is the codes' arithmetic, ten instructions an element pair.  A row of
// 8 elements a lane took 112 us.  A decode step's 32 rows are one launch.
//
// The quotient's code comes from a product with 1 / s: t = (x - z) * (1 / s)
// is off by less than 1e-5 (15 times a few roundings of 2^-24), so unless t
// is that near to a half its nearest whole number c is the quotient's too.
// Exact halves are common (x - z and s are short fractions): there x - z - c
// s is s / 2 to the bit, and c goes to the even side.  Only what is near a
// half without being one is divided.
struct Append {
    int B, Lq, Hkv, num_blocks, max_blocks;
    unsigned magic;                   // (2^32 - 1) / Lq
    const __half *k_new, *v_new;      // [B, Lq, Hkv, D]
    const int *block_tables, *ctx_lens, *q_lens;
    const int *slot_map;              // [B, Lq] or null: the slots from the block tables
    unsigned char *k, *v;
    __half2 *ksz, *vsz;
    unsigned *flags;
};
constexpr int kAppendDims = 32;       // elements of a lane: 64 bytes in, 16 bytes of codes out

// Codes of eight elements.  r: 1 / s; clamp: a code may come out above 15.
__device__ __forceinline__ unsigned codes_of(uint4 x, float lo, float s, float r, bool clamp)
{
    constexpr float kMagic = 12582912.f;      // 1.5 * 2^23: t + kMagic has rint(t) in its low bits
    const unsigned xs[4] = {x.x, x.y, x.z, x.w};
    float2 t[4], m[4];
    float far = 0.f;
#pragma unroll
    for (int e = 0; e < 4; e++) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&xs[e]));
        t[e] = mul2(add2(f, make_float2(-lo, -lo)), make_float2(r, r));
        m[e] = add2(t[e], make_float2(kMagic, kMagic));
        const float2 d = fma2(add2(m[e], make_float2(-kMagic, -kMagic)), make_float2(-1.f, -1.f), t[e]);
        far = fmaxf(far, fmaxf(fabsf(d.x), fabsf(d.y)));
    }
    if (far > 0.49999f) {
        const float half = 0.5f * s;
        auto settle = [&](float d, float t1, float &m1) {
            const float c1 = m1 - kMagic, rest = fmaf(-c1, s, d);
            if (fabsf(rest) == half) {
                if (__float_as_uint(m1) & 1u) m1 += copysignf(1.f, rest);
            } else if (fabsf(t1 - c1) > 0.49999f) {
                m1 = __fdiv_rn(d, s) + kMagic;
            }
        };
#pragma unroll
        for (int e = 0; e < 4; e++) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&xs[e]));
            settle(f.x - lo, t[e].x, m[e].x);
            settle(f.y - lo, t[e].y, m[e].y);
        }
    }
    if (clamp) {
#pragma unroll
        for (int e = 0; e < 4; e++) m[e] = make_float2(fminf(m[e].x, kMagic + 15.f), fminf(m[e].y, kMagic + 15.f));
    }
    // the codes are the low bits of eight equal words plus 0..15: shifted
    // together, less what the eight words come to (x - z >= 0: none below 0)
    unsigned word = 0;
#pragma unroll
    for (int e = 3; e >= 0; e--) word = (((word << 4) + __float_as_uint(m[e].y)) << 4) + __float_as_uint(m[e].x);
    return word - 0x4b400000u * 0x11111111u;
}

template <int D, int GROUP>
__global__ void __launch_bounds__(256) append_kernel(const __grid_constant__ Append a)
{
    constexpr int kLanes = D / kAppendDims, kGroupLanes = GROUP / kAppendDims, kRows = 256 / kLanes;
    const int b = blockIdx.y, c = threadIdx.x % kLanes;
    const unsigned unit = blockIdx.x * kRows + threadIdx.x / kLanes;
    // rows do not straddle warps and all lanes of one take the same way: the
    // shuffles below name the row's own lanes
    const unsigned lanes = ((1u << kLanes) - 1u) << ((threadIdx.x & 31) / kLanes * kLanes);
    const int ql = a.q_lens ? a.q_lens[b] : a.Lq;
    const bool first = blockIdx.x == 0 && threadIdx.x == 0;
    if (ql < 0 || ql > a.Lq) {
        if (first) atomicOr(a.flags, FLAG_BAD_Q_LEN);
        return;
    }
    // consecutive rows of one head are neighbours, as they are in their page.
    // unit / Lq: the product with the rounded-down reciprocal is the quotient
    // or one less
    int hv = (int)__umulhi(unit, a.magic), i = (int)unit - hv * a.Lq;
    if (i >= a.Lq) {
        hv++;
        i -= a.Lq;
    }
    if (hv >= 2 * a.Hkv || i >= ql) return;
    const bool is_v = hv & 1;
    const int hk = hv >> 1;
    const size_t row = (size_t)b * a.Lq + i;
    const uint4 *src = reinterpret_cast<const uint4 *>((is_v ? a.v_new : a.k_new) + (row * a.Hkv + hk) * D) + 4 * c;
    uint4 x[4];
#pragma unroll
    for (int k = 0; k < 4; k++) x[k] = __ldg(src + k);
    int blk, at;
    if (a.slot_map) {
        const int slot = a.slot_map[row];
        if (slot < 0) return;
        blk = slot / kBlock;
        at = slot % kBlock;
    } else {
        const int n = a.ctx_lens[b];
        if (n < ql || n > (long long)a.max_blocks * kBlock) {
            if (first) atomicOr(a.flags, FLAG_BAD_CTX_LEN);
            return;
        }
        const int pos = n - ql + i;
        blk = a.block_tables[(size_t)b * a.max_blocks + pos / kBlock];
        at = pos % kBlock;
    }
    if (blk < 0 || blk >= a.num_blocks) {
        if (hv == 0 && c == 0) atomicOr(a.flags, FLAG_BAD_BLOCK);
        return;
    }
    // (lowest, minus the highest) of the group: two minima in one, which a NaN
    // goes through
    __half2 mn = *reinterpret_cast<const __half2 *>(&x[0].x), mx = mn;
#pragma unroll
    for (int k = 0; k < 4; k++) {
        const unsigned xs[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
#pragma unroll
        for (int e = 0; e < 4; e++) {
            const __half2 h = *reinterpret_cast<const __half2 *>(&xs[e]);
            mn = __hmin2_nan(mn, h);
            mx = __hmax2_nan(mx, h);
        }
    }
    mx = __hneg2(mx);
    __half2 lh = __hmin2_nan(__lows2half2(mn, mx), __highs2half2(mn, mx));
#pragma unroll
    for (int off = 1; off < kGroupLanes; off <<= 1) lh = __hmin2_nan(lh, __shfl_xor_sync(lanes, lh, off));
    const float lo = __low2float(lh), range = -__high2float(lh) - lo;
    __half s16 = __float2half_rn(__fdiv_rn(range, 15.f)), z16 = __low2half(lh);
    const float s = __half2float(s16);
    uint4 codes = make_uint4(0u, 0u, 0u, 0u);
    if (!(range < __int_as_float(0x7f800000))) {      // a NaN, or an infinity
        s16 = z16 = __ushort_as_half(0x7fff);
    } else if (s > 0.f) {
        float r;
        asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(s));
        // a scale that was rounded down by a large part of itself (a subnormal one)
        const bool clamp = range * r > 15.4f;
        codes.x = codes_of(x[0], lo, s, r, clamp);
        codes.y = codes_of(x[1], lo, s, r, clamp);
        codes.z = codes_of(x[2], lo, s, r, clamp);
        codes.w = codes_of(x[3], lo, s, r, clamp);
    }
    const size_t to = ((size_t)blk * a.Hkv + hk) * kBlock + at;
    *reinterpret_cast<uint4 *>((is_v ? a.v : a.k) + to * (D / 2) + 16 * c) = codes;
    if (c % kGroupLanes == 0) (is_v ? a.vsz : a.ksz)[to * (D / GROUP) + c / kGroupLanes] = __halves2half2(s16, z16);
}

// ----------------------------------------------------------------------------- attention: layout of a staged page
// A page of one KV head is staged as 16 rows of D / 2 bytes, K then V, in
// 16-byte chunks permuted within 128-byte lines so that the operand reads
// below (rows g or 2t, word or chunk of the other lane index) meet no bank
// twice; then the (s, z) pairs of K and of V.  Pages start on a line, so a
// chunk's place is an exclusive or away from its row's.
template <int D, int GROUP>
struct PageQ {
    static constexpr int kRow = D / 2;               // bytes of a row of codes
    static constexpr int kCodes = kBlock * kRow;
    static constexpr int NG = D / GROUP;             // groups of a row
    static constexpr int kSz = kBlock * NG * 4;      // bytes of the (s, z) pairs of K or V
    static constexpr int kPage = 2 * kCodes + 2 * kSz;
    static_assert(kPage % 128 == 0 && kCodes % 512 == 0 && 2 * kSz <= 512, "a page starts on a line; copies of a warp");
};

template <int D>
__device__ __forceinline__ int row_off(int row)
{
    constexpr int kPerLine = 256 / D;                // rows of a 128-byte line
    const int line = row / kPerLine, pos = (row % kPerLine) * (D / 32);
    return line * 128 + ((pos ^ ((line & 3) << 1)) << 4);
}
// byte `byte` of the row at row_off `row`
__device__ __forceinline__ int byte_off(int row, int byte) { return (row ^ (byte & 0x70)) + (byte & 15); }

// What a lane reads and copies in every page.  Its further rows are fixed
// steps away: 8 rows are an exclusive or and a sum, the next row is an
// exclusive or (D = 128: row 2t + 1 is the other half of row 2t's line).
template <int D, int GROUP>
struct Lane {
    using P = PageQ<D, GROUP>;
    static constexpr int kXor8 = D == 128 ? 0 : 64, kAdd8 = D == 128 ? 512 : 256, kXor1 = D == 128 ? 64 : 32;
    int lane;
    unsigned k0;                    // its K words of key g
    unsigned v0;                    // its V words of key 2t
    unsigned sz;                    // the pairs of key g
    unsigned to;                    // its first copied chunk
    unsigned long long at;          // that chunk's place among the block's codes
    const unsigned char *szc;       // its chunk of the pairs of block 0

    __device__ __forceinline__ void init(const Pool &pool)
    {
        asm volatile("mov.u32 %0, %%laneid;" : "=r"(lane));      // (kept, not read again)
        const int g = lane >> 2, t = lane & 3;
        k0 = byte_off(row_off<D>(g), t * (GROUP / 8));
        v0 = P::kCodes + byte_off(row_off<D>(2 * t), 4 * (GROUP == 32 ? (g & 3) : g));
        sz = 2 * P::kCodes + g * P::NG * 4;
        constexpr int kPerRow = P::kRow / 16, kChunks = P::kSz / 16;
        to = byte_off(row_off<D>(lane / kPerRow), 16 * (lane % kPerRow));
        at = 16 * lane;
        szc = reinterpret_cast<const unsigned char *>(lane < kChunks ? pool.ksz : pool.vsz) + 16 * (lane % kChunks);
    }
    // address of its K words of key g + 8 r, of its V words of key 2t + (k & 1) + 8 (k >> 1), x bytes into the row
    __device__ __forceinline__ unsigned k(unsigned st, int r, int x) const
    {
        return ((st + k0) ^ (unsigned)(r * kXor8 ^ x)) + r * kAdd8;
    }
    __device__ __forceinline__ unsigned v(unsigned st, int k, int x) const
    {
        return ((st + v0) ^ (unsigned)((k & 1) * kXor1 ^ (k >> 1) * kXor8 ^ x)) + (k >> 1) * kAdd8;
    }
};

__device__ __forceinline__ unsigned lds32(unsigned a)
{
    unsigned x;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(x) : "r"(a));
    return x;
}
__device__ __forceinline__ uint2 lds64(unsigned a)
{
    uint2 x;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(x.x), "=r"(x.y) : "r"(a));
    return x;
}
__device__ __forceinline__ uint4 lds128(unsigned a)
{
    uint4 x;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(a));
    return x;
}
// 16 bytes from global to shared memory, the first n of them (the others
// zero), where `go` is set: no branch
__device__ __forceinline__ void copy16(unsigned to, const void *from, int n, bool go)
{
    asm volatile("{ .reg .pred p; setp.ne.u32 p, %3, 0;\n @p cp.async.cg.shared.global [%0], [%1], 16, %2; }" ::"r"(to),
                 "l"(from), "r"(n), "r"((unsigned)go)
                 : "memory");
}
// A lane's pieces of one page's codes: N of K and N of V, 512 bytes apart
// (V's behind the page's K codes), n bytes each.
template <int N, int CODES, bool ALWAYS>
__device__ __forceinline__ void copy_codes(unsigned to, const void *k, const void *v, int n, bool go)
{
    static_assert(N == 1 || N == 2, "D = 64, 128");
    if constexpr (ALWAYS) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %3;\n cp.async.cg.shared.global [%0 + %4], [%2], 16, %3;" ::"r"(to),
                     "l"(k), "l"(v), "r"(n), "n"(CODES)
                     : "memory");
        if constexpr (N == 2)
            asm volatile("cp.async.cg.shared.global [%0 + 512], [%1 + 512], 16, %3;\n"
                         " cp.async.cg.shared.global [%0 + %4], [%2 + 512], 16, %3;" ::"r"(to),
                         "l"(k), "l"(v), "r"(n), "n"(CODES + 512)
                         : "memory");
    } else if constexpr (N == 2) {
        asm volatile("{ .reg .pred p; setp.ne.u32 p, %4, 0;\n"
                     " @p cp.async.cg.shared.global [%0], [%1], 16, %3;\n @p cp.async.cg.shared.global [%0 + %5], [%2], 16, %3;\n"
                     " @p cp.async.cg.shared.global [%0 + 512], [%1 + 512], 16, %3;\n"
                     " @p cp.async.cg.shared.global [%0 + %6], [%2 + 512], 16, %3; }" ::"r"(to),
                     "l"(k), "l"(v), "r"(n), "r"((unsigned)go), "n"(CODES), "n"(CODES + 512)
                     : "memory");
    } else {
        asm volatile("{ .reg .pred p; setp.ne.u32 p, %4, 0;\n"
                     " @p cp.async.cg.shared.global [%0], [%1], 16, %3;\n @p cp.async.cg.shared.global [%0 + %5], [%2], 16, %3; }" ::"r"(to),
                     "l"(k), "l"(v), "r"(n), "r"((unsigned)go), "n"(CODES)
                     : "memory");
    }
}

// ----------------------------------------------------------------------------- attention: work
// The context work as one line of pages: for every request, KV head and tile
// of columns (a sequence) the pages of the context, one after the other.  The
// line is cut into chunks of Q pages, a chunk is one warp's work, and a
// sequence inside a chunk leaves one partial result.  Chunk c and sequence s
// have partial c + s: along the line either number grows at every cut, so no
// two partials meet, and those of one sequence are neighbours.
struct Args {
    Params p;
    Pool pool;
    int nc;                   // columns kept per partial
    int q_min;                // pages of a chunk, at least
    int queue;                // every chunk from the queue (a grid in front has some of the SMs), else the first static
    long long part0;          // first partial row of the contexts
    float slack;              // kSlack in units of q . k
    long long rows0;          // first partial row of the prompt chunks: (split * max_q_total + row) * H + head
    int rows_max;             // columns of a request on the line, at most
};

// Handed to the merge kernel (the words of Sched's header: bad, Q, the pages
// of a prompt chunk's split).
struct Sched {
    long long *pre;           // [B + 1] pages of the line before request b
    int *qo, *seq;            // [B + 1] query rows and sequences before it
};
__host__ __device__ inline size_t sched_bytes(int B) { return 16 + 8 * (size_t)(B + 1) + 4 * (size_t)(2 * B + 2); }
__device__ __forceinline__ Sched sched_at(int *base, int B)
{
    Sched s;
    s.pre = reinterpret_cast<long long *>(base + 4);
    s.qo = reinterpret_cast<int *>(s.pre + B + 1);
    s.seq = s.qo + B + 1;
    return s;
}

// Requests of more than Args::rows_max columns are not on the line: they have
// CTAs of their own (rows_kernel).
constexpr int kRowsTile = 128, kRowsKeys = 64;
constexpr int CTRL_Q4_ROWS = 7;      // ctrl word: row items taken

// Columns of a request: query row i and head c of the group are column i G +
// c, in tiles of 8 * nt: one, two or four tensor-core tiles, as many as they
// fill.
struct Cols {
    int cols, nt, tiles;
};
__host__ __device__ inline Cols cols_of(int ql, int G)
{
    Cols c;
    c.cols = ql * G;
    const int lg = c.cols > 16 ? 2 : c.cols > 8 ? 1 : 0;
    c.nt = 1 << lg;
    c.tiles = (c.cols + 8 * c.nt - 1) >> (3 + lg);
    return c;
}

// One sequence, and a page of it.
struct Seq {
    int b, hk, tile, id;      // id: over the whole batch
    int page, pages;
    int n, ql, tiles;
};
// A place in a chunk: the sequence, and the pages of the chunk from its page on.
struct alignas(16) Walk {
    Seq q;
    int left;
    __device__ __forceinline__ int take() const { return min(left, q.pages - q.page); }
};
// A sequence's share of a chunk, as its loads were opened.
struct alignas(16) Share {
    int b, hk, tile, part;
    int page, end;            // pages to read
    int n, ql;
};
constexpr int kMaxWarps = 16, kShares = 3;

struct Smem4 {
    long long pre[kMaxB + 1];
    long long warp_pre[16];
    int qo[kMaxB + 1], seq[kMaxB + 1];
    int warp_qo[16], warp_seq[16];
    int bad;
    Walk walk[kMaxWarps];                     // where a warp's loads are
    Share share[kMaxWarps][kShares];          // its shares that are open, oldest first
    alignas(128) unsigned char ring[16];      // (the launch gives it its size)
};

// Shape of a CTA: warps, pages of a step (their keys share one round of the
// softmax), steps in a warp's ring.  One CTA per SM.  (12 warps: 10, 14 and 16
// were no faster at D = 128; nor were three or four pages a step.)
constexpr size_t kMaxSmem = 227 * 1024;
template <int D, int GROUP, int NT>
struct Geo {
    static constexpr int kPer = 2;
    static constexpr int kW = NT > 1 ? 8 : D == 128 ? 12 : 16;
    static constexpr int kStep = kPer * PageQ<D, GROUP>::kPage;
    static constexpr int kQ = NT > 1 ? NT * (D / 32) * 512 : 0;      // a warp's query operands in shared memory
    static constexpr int kFit = (int)((kMaxSmem - offsetof(Smem4, ring) - kW * kQ) / (kW * kStep));
    static constexpr int kStages = kFit < 6 ? kFit : 6;
    static_assert(kStages >= 2, "ring");
    static constexpr size_t kSmem = offsetof(Smem4, ring) + (size_t)kW * (kStages * kStep + kQ);
};

__device__ __forceinline__ void set_request(const Params &p, const Smem4 &s, Seq &q, int b)
{
    q.b = b;
    q.n = p.ctx_lens[b];      // (in range, or the call has ended)
    q.ql = s.qo[b + 1] - s.qo[b];
    q.tiles = cols_of(q.ql, p.G).tiles;
    q.pages = (q.n + kBlock - 1) / kBlock;
}
// the sequence at position f of the line
__device__ __forceinline__ Seq locate(const Params &p, const Smem4 &s, long long f)
{
    Seq q;
    int lo = 0, hi = p.B - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s.pre[mid] <= f) lo = mid; else hi = mid - 1;
    }
    set_request(p, s, q, lo);
    const unsigned rem = (unsigned)(f - s.pre[lo]);      // the host keeps a request below 2^31 pages
    const int at = (int)(rem / (unsigned)q.pages);
    q.page = (int)rem - at * q.pages;
    q.hk = q.tiles == 1 ? at : at / q.tiles;
    q.tile = at - q.hk * q.tiles;
    q.id = s.seq[lo] + at;
    return q;
}
// the next one of the line (there is one)
__device__ __forceinline__ void advance(const Params &p, const Smem4 &s, Seq &q)
{
    q.page = 0;
    q.id++;
    if (++q.tile < q.tiles) return;
    q.tile = 0;
    if (++q.hk < p.Hkv) return;
    q.hk = 0;
    int b = q.b + 1;
    while (s.pre[b + 1] == s.pre[b]) b++;      // requests without pages
    set_request(p, s, q, b);
    q.id = s.seq[b];
}
// Keys that row i of a request sees.
__device__ __forceinline__ int keys_seen(int n, int ql, int i) { return max(0, min(n, n - ql + 1 + i)); }
// Pages that any column of the sequence sees.
__device__ __forceinline__ int pages_seen(const Params &p, const Seq &q)
{
    if (q.ql == 1) return q.pages;
    const Cols c = cols_of(q.ql, p.G);
    const int last = min(c.cols, (q.tile + 1) * 8 * c.nt) - 1;
    return (keys_seen(q.n, q.ql, last / p.G) + kBlock - 1) / kBlock;
}

// The line of the batch, built by the whole CTA (W warps).
template <int W>
__device__ void build_line(const Params &p, Smem4 &s, int rows_max)
{
    constexpr int PER = (kMaxB + 32 * W - 1) / (32 * W);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int ql[PER], n[PER], sq[PER], sum_q = 0, sum_s = 0;
    long long pg[PER], sum_p = 0;
    unsigned flags = 0;
    if (tid == 0) s.bad = 0;
#pragma unroll
    for (int k = 0; k < PER; k++) {
        const int b = tid * PER + k;
        ql[k] = n[k] = 0;
        if (b < p.B) {
            ql[k] = p.q_lens ? p.q_lens[b] : p.Lq;
            n[k] = p.ctx_lens[b];
            if (ql[k] < 0 || ql[k] > p.Lq) { flags |= FLAG_BAD_Q_LEN; ql[k] = 0; }
            if (n[k] < 0 || n[k] > p.max_blocks * kBlock) { flags |= FLAG_BAD_CTX_LEN; ql[k] = n[k] = 0; }
        }
        sq[k] = ql[k] * p.G > rows_max ? 0 : p.Hkv * cols_of(ql[k], p.G).tiles;
        pg[k] = (long long)sq[k] * ((n[k] + kBlock - 1) / kBlock);
        sum_q += ql[k];
        sum_s += sq[k];
        sum_p += pg[k];
    }
    int iq = sum_q, is = sum_s;
    long long ip = sum_p;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int tq = __shfl_up_sync(0xffffffffu, iq, off), ts = __shfl_up_sync(0xffffffffu, is, off);
        const long long tp = __shfl_up_sync(0xffffffffu, ip, off);
        if (lane >= off) { iq += tq; is += ts; ip += tp; }
    }
    if (lane == 31) {
        s.warp_qo[warp] = iq;
        s.warp_seq[warp] = is;
        s.warp_pre[warp] = ip;
    }
    __syncthreads();
    if (flags) atomicOr(&s.bad, (int)flags);
    int bq = iq - sum_q, bs = is - sum_s;
    long long bp = ip - sum_p;
    for (int j = 0; j < warp; j++) {
        bq += s.warp_qo[j];
        bs += s.warp_seq[j];
        bp += s.warp_pre[j];
    }
#pragma unroll
    for (int k = 0; k < PER; k++) {
        const int b = tid * PER + k;
        if (b < p.B) {
            s.qo[b] = bq;
            s.seq[b] = bs;
            s.pre[b] = bp;
        }
        bq += ql[k];
        bs += sq[k];
        bp += pg[k];
    }
    if (tid == 32 * W - 1) {
        s.qo[p.B] = bq;
        s.seq[p.B] = bs;
        s.pre[p.B] = bp;
    }
    __syncthreads();
}

// ----------------------------------------------------------------------------- attention: one step
// The lane's E columns of a tile, one or two.
template <int E>
struct Vec {
    float x[E];
    __device__ __forceinline__ float &operator[](int e) { return x[e]; }
    __device__ __forceinline__ float operator[](int e) const { return x[e]; }
    static __device__ __forceinline__ Vec all(float v)
    {
        Vec r;
#pragma unroll
        for (int e = 0; e < E; e++) r[e] = v;
        return r;
    }
    // a row (0: keys g, 1: keys g + 8) of an accumulator tile
    static __device__ __forceinline__ Vec row(const float (&c)[4], int i)
    {
        Vec r;
#pragma unroll
        for (int e = 0; e < E; e++) r[e] = c[2 * i + e];
        return r;
    }
};
template <int E>
__device__ __forceinline__ Vec<E> vfma(Vec<E> a, float b, Vec<E> c)
{
    Vec<E> r;
#pragma unroll
    for (int e = 0; e < E; e++) r[e] = fmaf(a[e], b, c[e]);
    return r;
}
template <int E>
__device__ __forceinline__ Vec<E> vmul(Vec<E> a, float b)
{
    Vec<E> r;
#pragma unroll
    for (int e = 0; e < E; e++) r[e] = a[e] * b;
    return r;
}

// the first product of a sum: no accumulator to clear
__device__ __forceinline__ void mma16816_first(float c[4], const unsigned a[4], unsigned b0, unsigned b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
                 "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};\n"
                 : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// the NG pairs of a token
template <int NG>
__device__ __forceinline__ void load_pairs(unsigned at, __half2 (&h)[NG])
{
    unsigned w[NG];
    if constexpr (NG == 1) {
        w[0] = lds32(at);
    } else if constexpr (NG == 2) {
        const uint2 x = lds64(at);
        w[0] = x.x; w[1] = x.y;
    } else {
        const uint4 x = lds128(at);
        w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
    }
#pragma unroll
    for (int i = 0; i < NG; i++) h[i] = *reinterpret_cast<const __half2 *>(&w[i]);
}

// Softmax state of a warp's columns, E of them in a lane (8 nt + 2t, + 1; a
// batch of single columns has E = 1: column 0, in the lanes of t = 0).  O^T in
// units of (code * 2^-24 or 2^-20) * 2^-down.
template <int D, int GROUP, int NT, int E>
struct State {
    float o[NT][D / 16][4];
    float c[NT][D / GROUP][4];      // the same for a code of 8 in every dimension
    Vec<E> z[NT][D / GROUP];        // sum of p (z + 8 s) over the lane's keys
    Vec<E> m[NT], l[NT];
    int e;                          // scale_exp of the largest V scale so far
};

constexpr float kSlack = 8.f;
constexpr unsigned kLoCodes = 0x000f000fu, kHiCodes = 0x00f000f0u;

// Biased exponent of a scale, plus one; 0 for an infinite or NaN scale, which
// must not move the others' power (it may belong to a key no row sees).
__device__ __forceinline__ int scale_exp(__half2 sz) { return ((__half_as_ushort(__low2half(sz)) >> 10) + 1) & 31; }
// 2^(15 - e): brings a scale of that exponent at most to below 1
__device__ __forceinline__ float scale_down(int e) { return __int_as_float((15 - e + 127) << 23); }

template <int D, int GROUP, int NT>
__device__ __forceinline__ void load_q(const Params &p, int lane, const Share &s, int cols, unsigned (&qb)[NT][D / 16][2])
{
    constexpr int WPG = GROUP / 32;
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int nt = 0; nt < NT; nt++) {
        const int v = s.tile * 8 * NT + 8 * nt + g;
        const bool has = v < cols;
        const int i = s.ql == 1 || !has ? 0 : v / p.G, c = has ? v - i * p.G : 0;
        const __half *q = p.q + (((size_t)s.b * p.Lq + i) * p.H + s.hk * p.G + c) * D;
#pragma unroll
        for (int w = 0; w < D / 32; w++) {
            // dimensions of word w of the lane: the K words are read the same way
            const int d0 = (w / WPG) * GROUP + t * (GROUP / 4) + 8 * (w % WPG);
            uint4 x = make_uint4(0u, 0u, 0u, 0u);
            if (has) x = *reinterpret_cast<const uint4 *>(q + d0);
            qb[nt][2 * w][0] = __byte_perm(x.x, x.z, 0x5410);          // dimensions 0, 4
            qb[nt][2 * w][1] = __byte_perm(x.y, x.w, 0x5410);          // 2, 6
            qb[nt][2 * w + 1][0] = __byte_perm(x.x, x.z, 0x7632);      // 1, 5
            qb[nt][2 * w + 1][1] = __byte_perm(x.y, x.w, 0x7632);      // 3, 7
        }
    }
}

// Sums of q over each group, for the lane's columns of every tile: the product
// with rows of ones.
template <int D, int GROUP, int NT, int E>
__device__ __forceinline__ void q_sums(const unsigned (&qb)[NT][D / 16][2], Vec<E> (&qs)[NT][D / GROUP])
{
    constexpr int WPG = GROUP / 32;
    const unsigned ones[4] = {0x3c003c00u, 0x3c003c00u, 0x3c003c00u, 0x3c003c00u};
#pragma unroll
    for (int nt = 0; nt < NT; nt++)
#pragma unroll
        for (int gi = 0; gi < D / GROUP; gi++) {
            float x[4];
            mma16816_first(x, ones, qb[nt][gi * 2 * WPG][0], qb[nt][gi * 2 * WPG][1]);
#pragma unroll
            for (int w = gi * 2 * WPG + 1; w < (gi + 1) * 2 * WPG; w++) mma16816(x, ones, qb[nt][w][0], qb[nt][w][1]);
            qs[nt][gi] = Vec<E>::row(x, 0);
        }
}

// One lane's share of staging one page (where `go` is set): `rows` valid
// tokens.  The codes are copied whole (what lies behind the last token is a
// number either way); the pairs of further tokens read as zero, so that
// nothing of them is left.  A block id of -1 (block_ids) reads as zero.
template <int D, int GROUP, bool ALWAYS>
__device__ __forceinline__ void load_page(const Params &p, const Pool &pool, const Lane<D, GROUP> &ln, unsigned st, int blk,
                                          int hk, int rows, bool go)
{
    using P = PageQ<D, GROUP>;
    const int all = blk >= 0 ? 16 : 0;
    const unsigned page = max(blk, 0) * p.Hkv + hk;      // the host keeps the pool below 2^31 of them
    const unsigned long long off = (unsigned long long)page * P::kCodes + ln.at;
    const unsigned char *kc = pool.k + off, *vc = pool.v + off;
    copy_codes<P::kCodes / 512, P::kCodes, ALWAYS>(st + ln.to, kc, vc, all, go);
    constexpr int kChunks = P::kSz / 16;      // of K, then of V
    const int n = min(all, max(0, rows * P::NG * 4 - 16 * (ln.lane % kChunks)));
    copy16(st + 2 * P::kCodes + 16 * ln.lane, ln.szc + (unsigned long long)page * P::kSz, n, go && ln.lane < 2 * kChunks);
}
// Lane j's entry of a table, one outside the pool flagged and -1.
__device__ __forceinline__ int block_id(const Params &p, const int *table, int at, int end)
{
    int blk = 0;
    if (at < end) {
        blk = table[at];
        if ((unsigned)blk >= (unsigned)p.num_blocks) {
            atomicOr(&p.ctrl[CTRL_FLAGS], FLAG_BAD_BLOCK);
            blk = -1;
        }
    }
    return blk;
}

// S^T = K q of one staged page, a group at a time: keys g, g + 8.
template <int D, int GROUP, int NT, int E>
__device__ __forceinline__ void page_scores(unsigned st, const Lane<D, GROUP> &ln, const unsigned (&qb)[NT][D / 16][2],
                                            const Vec<E> (&qs)[NT][D / GROUP], Vec<E> (&sc)[NT][2])
{
    using P = PageQ<D, GROUP>;
    constexpr int NG = P::NG, WPG = GROUP / 32;
    __half2 h0[NG], h1[NG];
    load_pairs<NG>(st + ln.sz, h0);
    load_pairs<NG>(st + ln.sz + 8 * NG * 4, h1);
#pragma unroll
    for (int gi = 0; gi < NG; gi++) {
        unsigned w0[WPG], w1[WPG];
        const unsigned r0 = ln.k(st, 0, gi * (GROUP / 2)), r1 = ln.k(st, 1, gi * (GROUP / 2));
        if constexpr (WPG == 4) {
            const uint4 x = lds128(r0), y = lds128(r1);
            w0[0] = x.x; w0[1] = x.y; w0[2] = x.z; w0[3] = x.w;
            w1[0] = y.x; w1[1] = y.y; w1[2] = y.z; w1[3] = y.w;
        } else if constexpr (WPG == 2) {
            const uint2 x = lds64(r0), y = lds64(r1);
            w0[0] = x.x; w0[1] = x.y;
            w1[0] = y.x; w1[1] = y.y;
        } else {
            w0[0] = lds32(r0);
            w1[0] = lds32(r1);
        }
        float lo[NT][4], hi[NT][4];
#pragma unroll
        for (int j = 0; j < WPG; j++) {
            const unsigned x0 = w0[j] >> 8, x1 = w1[j] >> 8;
            const unsigned a0[4] = {w0[j] & kLoCodes, w1[j] & kLoCodes, x0 & kLoCodes, x1 & kLoCodes};
            const unsigned a1[4] = {w0[j] & kHiCodes, w1[j] & kHiCodes, x0 & kHiCodes, x1 & kHiCodes};
            const int w = 2 * (gi * WPG + j);
#pragma unroll
            for (int nt = 0; nt < NT; nt++) {
                if (j == 0) {
                    mma16816_first(lo[nt], a0, qb[nt][w][0], qb[nt][w][1]);
                    mma16816_first(hi[nt], a1, qb[nt][w + 1][0], qb[nt][w + 1][1]);
                } else {
                    mma16816(lo[nt], a0, qb[nt][w][0], qb[nt][w][1]);
                    mma16816(hi[nt], a1, qb[nt][w + 1][0], qb[nt][w + 1][1]);
                }
            }
        }
        const float2 k0 = __half22float2(h0[gi]), k1 = __half22float2(h1[gi]);
#pragma unroll
        for (int nt = 0; nt < NT; nt++)
#pragma unroll
            for (int r = 0; r < 2; r++) {
                const float2 k = r ? k1 : k0;
                const Vec<E> dot = vfma(Vec<E>::row(lo[nt], r), 16.f, Vec<E>::row(hi[nt], r));
                const Vec<E> z = gi ? vfma(qs[nt][gi], k.y, sc[nt][r]) : vmul(qs[nt][gi], k.y);
                sc[nt][r] = vfma(dot, k.x * 0x1p20f, z);
            }
    }
}

// O^T += V^T P of one staged page.  A lane's operand rows are dimensions, its
// columns keys 2t, 2t + 1, 2t + 8, 2t + 9: two keys' words are interleaved by
// halves, and a tile is one code position of the words.  Rows of a tile share
// their group, so with GROUP = 32 (four words) the two halves of the rows take
// the same word at positions 8 bits apart.
template <int D, int GROUP, int NT>
__device__ __forceinline__ void page_values(unsigned st, const Lane<D, GROUP> &ln, const unsigned (&pb)[NT][D / GROUP][2],
                                            float (&o)[NT][D / 16][4], float (&c8)[NT][D / GROUP][4])
{
    using P = PageQ<D, GROUP>;
    constexpr unsigned kEight = 0x00080008u;
    const unsigned eights[4] = {kEight, kEight, kEight, kEight};
#pragma unroll
    for (int nt = 0; nt < NT; nt++)
#pragma unroll
        for (int gi = 0; gi < P::NG; gi++) mma16816(c8[nt][gi], eights, pb[nt][gi][0], pb[nt][gi][1]);
    constexpr int kHalf = GROUP == 32 ? 32 : 64;      // dimensions of a set of tiles
#pragma unroll
    for (int h = 0; h < D / kHalf; h++) {
        unsigned w[4];
#pragma unroll
        for (int k = 0; k < 4; k++) w[k] = lds32(ln.v(st, k, h * (kHalf / 2)));
        unsigned x0 = __byte_perm(w[0], w[1], 0x5410), y0 = __byte_perm(w[0], w[1], 0x7632);
        unsigned x1 = __byte_perm(w[2], w[3], 0x5410), y1 = __byte_perm(w[2], w[3], 0x7632);
        const int gi = h * kHalf / GROUP;
        if constexpr (GROUP == 32) {
            const int sh = (ln.lane >> 4) * 8;
            x0 >>= sh; y0 >>= sh; x1 >>= sh; y1 >>= sh;
            const unsigned a0[4] = {x0 & kLoCodes, y0 & kLoCodes, x1 & kLoCodes, y1 & kLoCodes};
            const unsigned a1[4] = {x0 & kHiCodes, y0 & kHiCodes, x1 & kHiCodes, y1 & kHiCodes};
#pragma unroll
            for (int nt = 0; nt < NT; nt++) {
                mma16816(o[nt][2 * h], a0, pb[nt][gi][0], pb[nt][gi][1]);
                mma16816(o[nt][2 * h + 1], a1, pb[nt][gi][0], pb[nt][gi][1]);
            }
        } else {
#pragma unroll
            for (int r = 0; r < 2; r++) {
                const unsigned x = r ? y0 : x0, y = r ? y1 : x1;
                const unsigned xs = x >> 8, ys = y >> 8;
                const unsigned a0[4] = {x & kLoCodes, xs & kLoCodes, y & kLoCodes, ys & kLoCodes};
                const unsigned a1[4] = {x & kHiCodes, xs & kHiCodes, y & kHiCodes, ys & kHiCodes};
#pragma unroll
                for (int nt = 0; nt < NT; nt++) {
                    mma16816(o[nt][4 * h + 2 * r], a0, pb[nt][gi][0], pb[nt][gi][1]);
                    mma16816(o[nt][4 * h + 2 * r + 1], a1, pb[nt][gi][0], pb[nt][gi][1]);
                }
            }
        }
    }
}

// One warp, KP staged pages of one sequence that every column sees whole
// (FULL), or np <= KP of which the lane's columns see end[nt][e] keys.
template <int D, int GROUP, int NT, int E, int KP, bool FULL>
__device__ __forceinline__ void step(unsigned st, const Lane<D, GROUP> &ln, int np,
                                     const unsigned (&qb)[NT][D / 16][2], const Vec<E> (&qs)[NT][D / GROUP],
                                     State<D, GROUP, NT, E> &s, const int (&end)[NT][E], float scale_log2, float slack)
{
    using P = PageQ<D, GROUP>;
    constexpr int NG = P::NG;
    const int g = ln.lane >> 2;

    Vec<E> sc[KP][NT][2];      // rows: keys g, g + 8
#pragma unroll
    for (int j = 0; j < KP; j++) {
        if (FULL || j == 0 || j < np) {
            page_scores<D, GROUP, NT, E>(st + j * P::kPage, ln, qb, qs, sc[j]);
        } else {
#pragma unroll
            for (int nt = 0; nt < NT; nt++) sc[j][nt][0] = sc[j][nt][1] = Vec<E>::all(kNegInf);
        }
    }
    // Online softmax per column (keys over the lanes' g).  The reference of the
    // weights moves only when some score is past it by more than 2^kSlack (up
    // to that the weights are as exact), and the V scales' common power of
    // two, which makes p s / 2^e fill fp16 from the top, only when a scale is
    // past it: the lanes look at their own keys, and one vote in most steps
    // finds that nothing has moved.  (m is in units of q . k; the softmax scale
    // is positive.)
    if (!FULL) {
#pragma unroll
        for (int j = 0; j < KP; j++)
#pragma unroll
            for (int nt = 0; nt < NT; nt++)
#pragma unroll
                for (int e = 0; e < E; e++) {
                    if (16 * j + g >= end[nt][e]) sc[j][nt][0][e] = kNegInf;
                    if (16 * j + g + 8 >= end[nt][e]) sc[j][nt][1][e] = kNegInf;
                }
    }
    Vec<E> mx[NT];
    bool moved = false;
#pragma unroll
    for (int nt = 0; nt < NT; nt++)
#pragma unroll
        for (int e = 0; e < E; e++) {
            float x = kNegInf;
#pragma unroll
            for (int j = 0; j < KP; j++) x = fmaxf(x, fmaxf(sc[j][nt][0][e], sc[j][nt][1][e]));
            mx[nt][e] = x;
            moved = moved || x > s.m[nt][e] + slack;      // (any number is past minus infinity)
        }
    __half2 h[KP][2][NG];
    int em = 0;
#pragma unroll
    for (int j = 0; j < KP; j++)
        if (FULL || j == 0 || j < np) {
#pragma unroll
            for (int r = 0; r < 2; r++) {
                load_pairs<NG>(st + j * P::kPage + P::kSz + ln.sz + r * 8 * NG * 4, h[j][r]);
#pragma unroll
                for (int gi = 0; gi < NG; gi++)
                    if (!FULL) em = max(em, scale_exp(h[j][r][gi]));
            }
        }
    if (FULL) {      // the keys are all seen: their largest scale as it is
        __half2 top = __habs2(h[0][0][0]);
#pragma unroll
        for (int i = 1; i < KP * 2 * NG; i++) top = __hmax2(top, __habs2(h[i / (2 * NG)][i / NG % 2][i % NG]));
        em = scale_exp(top);
    }
    if (__any_sync(0xffffffffu, moved || em > s.e)) {
        em = max(s.e, (int)__reduce_max_sync(0xffffffffu, (unsigned)em));
        const float ae = __int_as_float((s.e - em + 127) << 23);
        s.e = em;
#pragma unroll
        for (int nt = 0; nt < NT; nt++)
#pragma unroll
            for (int e = 0; e < E; e++) {
                float x = mx[nt][e];
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, off));
                const float old = s.m[nt][e], m = fmaxf(old, x);
                s.m[nt][e] = m;
                const float al = m == kNegInf ? 1.f : ex2((old - m) * scale_log2), ao = al * ae;
                s.l[nt][e] *= al;
#pragma unroll
                for (int gi = 0; gi < NG; gi++) {
                    s.z[nt][gi][e] *= al;
                    s.c[nt][gi][e] *= ao;
                }
#pragma unroll
                for (int d = 0; d < D / 16; d++) {
                    s.o[nt][d][e] *= ao;
                    s.o[nt][d][2 + e] *= ao;
                }
            }
    }
    Vec<E> mu[NT];      // minus the reference, in powers of two
#pragma unroll
    for (int nt = 0; nt < NT; nt++)
#pragma unroll
        for (int e = 0; e < E; e++) mu[nt][e] = s.m[nt][e] == kNegInf ? 0.f : -s.m[nt][e] * scale_log2;
    em = s.e;
    const float down = scale_down(em);
#pragma unroll
    for (int j = 0; j < KP; j++) {
        if (!FULL && j > 0 && j >= np) break;
        unsigned pb[NT][NG][2];
#pragma unroll
        for (int nt = 0; nt < NT; nt++)
#pragma unroll
            for (int r = 0; r < 2; r++) {
                sc[j][nt][r] = vfma(sc[j][nt][r], scale_log2, mu[nt]);
#pragma unroll
                for (int e = 0; e < E; e++) {
                    sc[j][nt][r][e] = ex2(sc[j][nt][r][e]);
                    s.l[nt][e] += sc[j][nt][r][e];
                }
            }
#pragma unroll
        for (int gi = 0; gi < NG; gi++)
#pragma unroll
            for (int r = 0; r < 2; r++) {
                const float2 v = __half22float2(h[j][r][gi]);
                const float vs = v.x * down, vz = fmaf(8.f, v.x, v.y);
#pragma unroll
                for (int nt = 0; nt < NT; nt++) {
                    Vec<E> w;
                    if (FULL) {
                        w = vmul(sc[j][nt][r], vs);
                        s.z[nt][gi] = vfma(sc[j][nt][r], vz, s.z[nt][gi]);
                    } else {
                        // a NaN behind the mask must not meet its zero weight
#pragma unroll
                        for (int e = 0; e < E; e++) {
                            const bool seen = 16 * j + g + 8 * r < end[nt][e];
                            w[e] = seen ? sc[j][nt][r][e] * vs : 0.f;
                            s.z[nt][gi][e] += seen ? sc[j][nt][r][e] * vz : 0.f;
                        }
                    }
                    pb[nt][gi][r] = movmatrix_t(pack_half2(w[0], E > 1 ? w[E - 1] : 0.f));
                }
            }
        page_values<D, GROUP, NT>(st + j * P::kPage, ln, pb, s.o, s.c);
    }
}

// ----------------------------------------------------------------------------- attention: many columns
// The same step for NT = 2 or 4 tiles of columns, a page at a time, where the
// tensor cores and the arithmetic per column count for more than the unpacking
// that the tiles share:
//  - the query operands stay in shared memory (a lane's fragments of word w of
//    tile nt side by side), the accumulators take the registers;
//  - all four code positions of a K word are shifted to the bottom, so that
//    one accumulator takes them all;
//  - V's operands are c - 8 (1024 + c as fp16 bits, less 1032: exact), so no
//    product with eights is needed;
//  - sum(q) z and sum p (z + 8 s) are products too, over the groups and over
//    the keys, with sum(q) and z + 8 s as an fp16 number and its remainder.
template <int D, int GROUP, int NT>
struct Wide {
    float o[NT][D / 16][4];         // tiles of code positions 0 (units of 2^-down) and 1 (of 16 times that)
    float z[NT][4];                 // row i < NG: sum p hi(z + 8 s) of group i, row NG + i: of the remainders
    Vec<2> m[NT], l[NT];
    int e;
};
constexpr float kQsScale = 1.f / 128.f;      // a group's sum of q fits fp16

// The share's query operands: fragments to shared memory, sums to registers.
template <int D, int GROUP, int NT>
__device__ __forceinline__ void wide_q(const Params &p, int lane, const Share &s, int cols, unsigned qsm, unsigned (&qz)[NT])
{
    constexpr int WPG = GROUP / 32, NG = D / GROUP;
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int nt = 0; nt < NT; nt++) {
        const int v = s.tile * 8 * NT + 8 * nt + g;
        const bool has = v < cols;
        const int i = s.ql == 1 || !has ? 0 : v / p.G, c = has ? v - i * p.G : 0;
        const __half *q = p.q + (((size_t)s.b * p.Lq + i) * p.H + s.hk * p.G + c) * D;
        float sum[NG];
#pragma unroll
        for (int gi = 0; gi < NG; gi++) sum[gi] = 0.f;
#pragma unroll
        for (int w = 0; w < D / 32; w++) {
            const int d0 = (w / WPG) * GROUP + t * (GROUP / 4) + 8 * (w % WPG);
            uint4 x = make_uint4(0u, 0u, 0u, 0u);
            if (has) x = *reinterpret_cast<const uint4 *>(q + d0);
            const unsigned xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int k = 0; k < 4; k++) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&xs[k]));
                sum[w / WPG] += f.x + f.y;
            }
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(qsm + ((nt * (D / 32) + w) * 32 + lane) * 16),
                         "r"(__byte_perm(x.x, x.z, 0x5410)), "r"(__byte_perm(x.y, x.w, 0x5410)),
                         "r"(__byte_perm(x.x, x.z, 0x7632)), "r"(__byte_perm(x.y, x.w, 0x7632))
                         : "memory");
        }
        // row k of the operand: sums of groups k 2^-7 of themselves, then their
        // remainders as they are (2^-7 of them would fall below fp16 where q is small)
        __half v16[2 * NG];
#pragma unroll
        for (int gi = 0; gi < NG; gi++) {
            float f = sum[gi];
            f += __shfl_xor_sync(0xffffffffu, f, 1);
            f += __shfl_xor_sync(0xffffffffu, f, 2);
            v16[gi] = __float2half_rn(f * kQsScale);
            v16[NG + gi] = __float2half_rn(f - __half2float(v16[gi]) * (1.f / kQsScale));
        }
        unsigned w = 0;
#pragma unroll
        for (int k = 0; k < NG; k++)
            if (t == k) {
                const __half2 h = __halves2half2(v16[2 * k], v16[2 * k + 1]);
                w = *reinterpret_cast<const unsigned *>(&h);
            }
        qz[nt] = w;
    }
    __syncwarp();
}

// One staged page.  FULL: every column sees all of it.
template <int D, int GROUP, int NT, bool FULL>
__device__ __forceinline__ void wide_page(unsigned st, const Lane<D, GROUP> &ln, unsigned qsm, const unsigned (&qz)[NT],
                                          Wide<D, GROUP, NT> &s, const int (&end)[NT][2], float scale_log2, float slack)
{
    using P = PageQ<D, GROUP>;
    constexpr int NG = P::NG, WPG = GROUP / 32;
    const int g = ln.lane >> 2, t = ln.lane & 3;
    const __half2 zero = __floats2half2_rn(0.f, 0.f);
    float sc[NT][4];
    {
        // z sum(q): rows keys, columns of the operand groups (z for the sums, 2^-7 z for their remainders)
        const __half2 by = __floats2half2_rn(2 * t < NG ? 1.f : kQsScale, 2 * t + 1 < NG ? 1.f : kQsScale);
        __half2 h[2][NG];
        load_pairs<NG>(st + ln.sz, h[0]);
        load_pairs<NG>(st + ln.sz + 8 * NG * 4, h[1]);
        unsigned a[4] = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int r = 0; r < 2; r++) {
            __half2 z = NG == 1 ? __highs2half2(h[r][0], h[r][0]) : __highs2half2(h[r][0], h[r][NG > 1 ? 1 : 0]);
            if (NG == 4 && (t & 1)) z = __highs2half2(h[r][NG > 2 ? 2 : 0], h[r][NG > 2 ? 3 : 0]);
            z = __hmul2(z, by);
            a[r] = *reinterpret_cast<const unsigned *>(&z);
        }
#pragma unroll
        for (int nt = 0; nt < NT; nt++) {
            mma16816_first(sc[nt], a, qz[nt], 0u);
#pragma unroll
            for (int e = 0; e < 4; e++) sc[nt][e] *= 1.f / kQsScale;
        }
#pragma unroll
        for (int gi = 0; gi < NG; gi++) {
            unsigned w[2][WPG];
#pragma unroll
            for (int r = 0; r < 2; r++) {
                const unsigned at = ln.k(st, r, gi * (GROUP / 2));
                if constexpr (WPG == 4) {
                    const uint4 x = lds128(at);
                    w[r][0] = x.x; w[r][1] = x.y; w[r][2] = x.z; w[r][3] = x.w;
                } else if constexpr (WPG == 2) {
                    const uint2 x = lds64(at);
                    w[r][0] = x.x; w[r][1] = x.y;
                } else {
                    w[r][0] = lds32(at);
                }
            }
            float acc[NT][4];
#pragma unroll
            for (int j = 0; j < WPG; j++) {
                const unsigned x0 = w[0][j], x1 = w[1][j];
                const unsigned a0[4] = {x0 & kLoCodes, x1 & kLoCodes, (x0 >> 8) & kLoCodes, (x1 >> 8) & kLoCodes};
                const unsigned a1[4] = {(x0 >> 4) & kLoCodes, (x1 >> 4) & kLoCodes, (x0 >> 12) & kLoCodes, (x1 >> 12) & kLoCodes};
#pragma unroll
                for (int nt = 0; nt < NT; nt++) {
                    const uint4 b = lds128(qsm + ((nt * (D / 32) + gi * WPG + j) * 32 + ln.lane) * 16);
                    if (j == 0) mma16816_first(acc[nt], a0, b.x, b.y);
                    else mma16816(acc[nt], a0, b.x, b.y);
                    mma16816(acc[nt], a1, b.z, b.w);
                }
            }
            const float f[2] = {__low2float(h[0][gi]) * 0x1p24f, __low2float(h[1][gi]) * 0x1p24f};
#pragma unroll
            for (int nt = 0; nt < NT; nt++)
#pragma unroll
                for (int e = 0; e < 4; e++) sc[nt][e] = fmaf(f[e >> 1], acc[nt][e], sc[nt][e]);
        }
    }
    bool moved = false;
    Vec<2> mn[NT], mu[NT];
#pragma unroll
    for (int nt = 0; nt < NT; nt++)
#pragma unroll
        for (int e = 0; e < 2; e++) {
            if (!FULL) {
                if (g >= end[nt][e]) sc[nt][e] = kNegInf;
                if (g + 8 >= end[nt][e]) sc[nt][2 + e] = kNegInf;
            }
            float mx = fmaxf(sc[nt][e], sc[nt][2 + e]);
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
            const float m = s.m[nt][e];
            const bool move = mx > m + slack;
            mn[nt][e] = move ? mx : m;
            mu[nt][e] = mn[nt][e] == kNegInf ? 0.f : -mn[nt][e] * scale_log2;
            moved = moved || move;
        }
    // V's pairs of keys g, g + 8 (the weights) and of the operand's keys (z + 8 s)
    const unsigned vsz = st + 2 * P::kCodes + P::kSz;
    __half2 h[2][NG];
    load_pairs<NG>(vsz + g * NG * 4, h[0]);
    load_pairs<NG>(vsz + (g + 8) * NG * 4, h[1]);
    int em = 0;
#pragma unroll
    for (int i = 0; i < 2 * NG; i++) em = max(em, scale_exp(h[i / NG][i % NG]));
    em = max(s.e, (int)__reduce_max_sync(0xffffffffu, (unsigned)em));
    if (__any_sync(0xffffffffu, moved || em != s.e)) {
        const float ae = __int_as_float((s.e - em + 127) << 23);
        s.e = em;
#pragma unroll
        for (int nt = 0; nt < NT; nt++)
#pragma unroll
            for (int e = 0; e < 2; e++) {
                const float al = ex2(fmaf(s.m[nt][e], scale_log2, mu[nt][e])), ao = al * ae;
                s.m[nt][e] = mn[nt][e];
                s.l[nt][e] *= al;
                s.z[nt][e] *= al;
                s.z[nt][2 + e] *= al;
#pragma unroll
                for (int d = 0; d < D / 16; d++) {
                    s.o[nt][d][e] *= ao;
                    s.o[nt][d][2 + e] *= ao;
                }
            }
    }
    const float down = scale_down(em);
#pragma unroll
    for (int nt = 0; nt < NT; nt++)
#pragma unroll
        for (int e = 0; e < 4; e++) {
            sc[nt][e] = ex2(fmaf(sc[nt][e], scale_log2, mu[nt][e & 1]));
            s.l[nt][e & 1] += sc[nt][e];
        }
    {
        // rows: group i's z + 8 s as fp16, row NG + i: what that leaves
        unsigned a[4] = {0u, 0u, 0u, 0u};
        const int gi = g % NG;
        const bool hi = g < NG, lo = !hi && g < 2 * NG;
#pragma unroll
        for (int k = 0; k < 2; k++) {
            float z[2];
#pragma unroll
            for (int i = 0; i < 2; i++) {
                const unsigned w = lds32(vsz + ((2 * t + i + 8 * k) * NG + gi) * 4);
                const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&w));
                z[i] = fmaf(8.f, v.x, v.y);
                // (of a key that some column does not see: it must not meet a zero weight)
                if (!FULL && !(fabsf(z[i]) < __int_as_float(0x7f800000))) z[i] = 0.f;
            }
            __half2 h16 = __floats2half2_rn(z[0], z[1]);
            if (lo) {
                const float2 b = __half22float2(h16);
                h16 = __floats2half2_rn(z[0] - b.x, z[1] - b.y);
            }
            if (!hi && !lo) h16 = zero;
            a[2 * k] = *reinterpret_cast<const unsigned *>(&h16);
        }
#pragma unroll
        for (int nt = 0; nt < NT; nt++)
            mma16816(s.z[nt], a, movmatrix_t(pack_half2(sc[nt][0], sc[nt][1])), movmatrix_t(pack_half2(sc[nt][2], sc[nt][3])));
    }
    constexpr int kHalf = GROUP == 32 ? 32 : 64;
    const __half2 bias0 = __floats2half2_rn(-1032.f, -1032.f), bias1 = __floats2half2_rn(-1152.f, -1152.f);
    auto lo_code = [&](unsigned x) {
        const unsigned b = (x & kLoCodes) | 0x64006400u;
        const __half2 r = __hadd2(*reinterpret_cast<const __half2 *>(&b), bias0);
        return *reinterpret_cast<const unsigned *>(&r);
    };
    auto hi_code = [&](unsigned x) {
        const unsigned b = (x & kHiCodes) | 0x64006400u;
        const __half2 r = __hadd2(*reinterpret_cast<const __half2 *>(&b), bias1);
        return *reinterpret_cast<const unsigned *>(&r);
    };
    unsigned pb[NT][2];
#pragma unroll
    for (int hf = 0; hf < D / kHalf; hf++) {
        const int gi = hf * kHalf / GROUP;
        if (hf * kHalf % GROUP == 0) {
#pragma unroll
            for (int r = 0; r < 2; r++) {
                float2 v = __half22float2(h[r][gi]);
                // (a bad z has left the operand above: the weights carry it)
                if (!FULL && !(fabsf(fmaf(8.f, v.x, v.y)) < __int_as_float(0x7f800000))) v.x = __int_as_float(0x7fffffff);
                const float vs = v.x * down;
#pragma unroll
                for (int nt = 0; nt < NT; nt++) {
                    float w[2];
#pragma unroll
                    for (int e = 0; e < 2; e++) {
                        const bool seen = FULL || g + 8 * r < end[nt][e];
                        w[e] = seen ? sc[nt][2 * r + e] * vs : 0.f;
                    }
                    pb[nt][r] = movmatrix_t(pack_half2(w[0], w[1]));
                }
            }
        }
        unsigned w[4];
#pragma unroll
        for (int k = 0; k < 4; k++) w[k] = lds32(ln.v(st, k, hf * (kHalf / 2)));
        unsigned x0 = __byte_perm(w[0], w[1], 0x5410), y0 = __byte_perm(w[0], w[1], 0x7632);
        unsigned x1 = __byte_perm(w[2], w[3], 0x5410), y1 = __byte_perm(w[2], w[3], 0x7632);
        if constexpr (GROUP == 32) {
            const int sh = (ln.lane >> 4) * 8;
            x0 >>= sh; y0 >>= sh; x1 >>= sh; y1 >>= sh;
            const unsigned a0[4] = {lo_code(x0), lo_code(y0), lo_code(x1), lo_code(y1)};
            const unsigned a1[4] = {hi_code(x0), hi_code(y0), hi_code(x1), hi_code(y1)};
#pragma unroll
            for (int nt = 0; nt < NT; nt++) {
                mma16816(s.o[nt][2 * hf], a0, pb[nt][0], pb[nt][1]);
                mma16816(s.o[nt][2 * hf + 1], a1, pb[nt][0], pb[nt][1]);
            }
        } else {
#pragma unroll
            for (int r = 0; r < 2; r++) {
                const unsigned x = r ? y0 : x0, y = r ? y1 : x1;
                const unsigned a0[4] = {lo_code(x), lo_code(x >> 8), lo_code(y), lo_code(y >> 8)};
                const unsigned a1[4] = {hi_code(x), hi_code(x >> 8), hi_code(y), hi_code(y >> 8)};
#pragma unroll
                for (int nt = 0; nt < NT; nt++) {
                    mma16816(s.o[nt][4 * hf + 2 * r], a0, pb[nt][0], pb[nt][1]);
                    mma16816(s.o[nt][4 * hf + 2 * r + 1], a1, pb[nt][0], pb[nt][1]);
                }
            }
        }
    }
}

// The group term of the lane's column 2t + e, from the operand's rows.
template <int D, int GROUP, int NT>
__device__ __forceinline__ float wide_z(const Wide<D, GROUP, NT> &s, int lane, int nt, int gi, int e)
{
    constexpr int NG = D / GROUP;
    const int t = lane & 3;
    return __shfl_sync(0xffffffffu, s.z[nt][e], 4 * gi + t) + __shfl_sync(0xffffffffu, s.z[nt][e], 4 * (NG + gi) + t);
}

// Writes a column's partial: normalised output (o times f0, in tiles of code
// position 1 times f1, plus its group's term) and log2-sum-exp.
template <int D, int GROUP>
__device__ __forceinline__ void write_column(const Args &a, int lane, size_t pr, const float (&o)[D / 16][4], int e, float f0,
                                             float f1, const float (&z)[D / GROUP], float lse)
{
    const int g = lane >> 2;
    float *po = a.p.part_o + pr * D;
    if constexpr (GROUP == 32) {
#pragma unroll
        for (int gi = 0; gi < D / GROUP; gi++)
#pragma unroll
            for (int r = 0; r < 2; r++)
                __stcg(reinterpret_cast<float2 *>(po + 32 * gi + 8 * (g & 3) + 2 * (g >> 2) + 4 * r),
                       make_float2(o[2 * gi][2 * r + e] * f0 + z[gi], o[2 * gi + 1][2 * r + e] * f1 + z[gi]));
    } else {
#pragma unroll
        for (int hf = 0; hf < D / 64; hf++) {
            const float zg = z[hf * 64 / GROUP];
            // tiles: code positions 0, 1, 4, 5 (rows g) and 2, 3, 6, 7 (rows g + 8)
#pragma unroll
            for (int r = 0; r < 2; r++) {
                const float(&x)[4] = o[4 * hf + 2 * r], (&y)[4] = o[4 * hf + 2 * r + 1];
                __stcg(reinterpret_cast<float4 *>(po + 64 * hf + 8 * g + 4 * r),
                       make_float4(x[e] * f0 + zg, y[e] * f1 + zg, x[2 + e] * f0 + zg, y[2 + e] * f1 + zg));
            }
        }
    }
    if (g == 0) __stcg(a.p.part_lse + pr, lse);
}

// Takes the product with eights off the output, as the end does.  The tensor
// cores cut what falls below the accumulator's last bit, and codes that are
// all positive grow it with the number of keys: taken off every kCentre pages
// the error against fp64 is 3.0e-4 of the result for 32 x 16384 keys, 4.2e-4
// without it (a result rounded once: 2.1e-4), for 1 us in 84.
constexpr int kCentre = 32;
template <int D, int GROUP, int E>
__device__ __forceinline__ void centre(State<D, GROUP, 1, E> &s)
{
#pragma unroll
    for (int d = 0; d < D / 16; d++)
#pragma unroll
        for (int i = 0; i < 4; i++) s.o[0][d][i] = fmaf(s.c[0][d * 16 / GROUP][i & 1], d & 1 ? -16.f : -1.f, s.o[0][d][i]);
#pragma unroll
    for (int gi = 0; gi < D / GROUP; gi++)
#pragma unroll
        for (int i = 0; i < 4; i++) s.c[0][gi][i] = 0.f;
}

// Writes the partial of a share, rows pr0 + column.
template <int D, int GROUP, int NT, int E>
__device__ __forceinline__ void write_partial(const Args &a, int lane, int nv, State<D, GROUP, NT, E> &s, size_t pr0)
{
    constexpr int NG = D / GROUP;
    const int t = lane & 3;
    const float up = __int_as_float((24 + s.e - 15 + 127) << 23);      // 2^24 / scale_down
#pragma unroll
    for (int nt = 0; nt < NT; nt++)
#pragma unroll
        for (int e = 0; e < E; e++) {
            float z[NG];
#pragma unroll
            for (int gi = 0; gi < NG; gi++) z[gi] = s.z[nt][gi][e];
            float L = s.l[nt][e];
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) {
                L += __shfl_xor_sync(0xffffffffu, L, off);
#pragma unroll
                for (int gi = 0; gi < NG; gi++) z[gi] += __shfl_xor_sync(0xffffffffu, z[gi], off);
            }
            const float inv = L == 0.f ? 0.f : __fdividef(1.f, L), f0 = up * inv;      // (a NaN goes on)
#pragma unroll
            for (int gi = 0; gi < NG; gi++) z[gi] = z[gi] * inv - s.c[nt][gi][e] * f0;
            const int c = 8 * nt + 2 * t + e;
            if (c < nv)
                write_column<D, GROUP>(a, lane, pr0 + c, s.o[nt], e, f0, f0 * 0.0625f, z,
                                       L == 0.f ? kNegInf : fmaf(s.m[nt][e], a.p.scale_log2, lg2(L)));
        }
}
template <int D, int GROUP, int NT>
__device__ __forceinline__ void write_partial(const Args &a, int lane, int nv, Wide<D, GROUP, NT> &s, size_t pr0)
{
    constexpr int NG = D / GROUP;
    const int t = lane & 3;
    const float up = __int_as_float((s.e - 15 + 127) << 23);      // 1 / scale_down
#pragma unroll
    for (int nt = 0; nt < NT; nt++)
#pragma unroll
        for (int e = 0; e < 2; e++) {
            float L = s.l[nt][e], z[NG];
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) L += __shfl_xor_sync(0xffffffffu, L, off);
            const float inv = L == 0.f ? 0.f : __fdividef(1.f, L), f0 = up * inv;
#pragma unroll
            for (int gi = 0; gi < NG; gi++) z[gi] = wide_z<D, GROUP, NT>(s, lane, nt, gi, e) * inv;
            const int c = 8 * nt + 2 * t + e;
            if (c < nv)
                write_column<D, GROUP>(a, lane, pr0 + c, s.o[nt], e, f0, f0 * 0.0625f, z,
                                       L == 0.f ? kNegInf : fmaf(s.m[nt][e], a.p.scale_log2, lg2(L)));
        }
}

// ----------------------------------------------------------------------------- attention: one chunk
// The chunks of a warp: the first one is static (spread over the SMs) where
// all CTAs start together, the others come from a queue and are asked for one
// ahead.
struct Chunks {
    long long total, count, queue0;      // queue0: the queue's first chunk
    int Q;
    unsigned ticket;

    __device__ __forceinline__ void ask(const Params &p)
    {
        ticket = 0x7fffffffu;
        if (count > queue0 && (threadIdx.x & 31) == 0) ticket = atomicAdd(&p.ctrl[CTRL_DEC_ITEMS], 1u);
    }
    __device__ __forceinline__ long long take() const { return queue0 + __shfl_sync(0xffffffffu, ticket, 0); }
};

// The pages in the order of the line, fetched a few steps ahead of the
// arithmetic, across the ends of sequences and chunks.  What only the end of a
// share needs is kept in shared memory.
template <int D, int GROUP, int KP, int STAGES>
struct Loader {
    using P = PageQ<D, GROUP>;
    int page, end, hk, n;       // the open share: next page, its end, KV head, tokens
    int blk, window;            // lane j: block of page window + j
    const int *table;
    unsigned at;                // ring place of the next step
    int issued;                 // steps staged so far
    int opened;                 // shares opened so far
    long long chunk;            // (its number, for the partials)

    // Opens the warp's next share, if there is one and room for it.
    __device__ __forceinline__ bool open(const Args &a, Smem4 &s, int lane, int warp, Chunks &ch, int closed)
    {
        if (opened - closed >= kShares) return false;
        Walk w = s.walk[warp];
        if (w.left <= 0) {
            chunk = ch.take();
            if (chunk >= ch.count) return false;
            ch.ask(a.p);
            w.q = locate(a.p, s, chunk * ch.Q);
            w.left = (int)min((long long)ch.Q, ch.total - chunk * ch.Q);
        }
        Share sh;
        sh.b = w.q.b;
        sh.hk = w.q.hk;
        sh.tile = w.q.tile;
        sh.part = (int)(chunk + w.q.id);
        sh.n = w.q.n;
        sh.ql = w.q.ql;
        const int take = w.take();
        sh.page = w.q.page;
        sh.end = min(sh.page + take, pages_seen(a.p, w.q));
        page = sh.page;
        end = sh.end;
        hk = sh.hk;
        n = w.q.n;
        table = a.p.block_tables + (size_t)sh.b * a.p.max_blocks;
        window = page;
        blk = block_id(a.p, table, page + lane, end);
        w.left -= take;
        if (w.left > 0) advance(a.p, s, w.q);
        __syncwarp();
        if (lane == 0) {
            s.walk[warp] = w;
            s.share[warp][opened % kShares] = sh;
        }
        __syncwarp();
        opened++;
        return true;
    }
    // Stages the warp's next steps, a cp.async group each, until the ring is
    // full (`done` steps have left it) or nothing is left to stage (`closed`
    // shares are done).
    __device__ __forceinline__ void fill(const Args &a, Smem4 &s, const Lane<D, GROUP> &ln, int warp, Chunks &ch, unsigned ring,
                                         int done, int closed)
    {
        while (issued - done < STAGES - 1) {
            if (page >= end) {
                if (!open(a, s, ln.lane, warp, ch, closed)) return;
                continue;      // (it may have no page to read)
            }
            static_assert(32 % KP == 0, "a step's blocks are in one window");
            if (page >= window + 32) {
                window = page;
                blk = block_id(a.p, table, window + ln.lane, end);
            }
            load_page<D, GROUP, true>(a.p, a.pool, ln, at, __shfl_sync(0xffffffffu, blk, page - window), hk, n - page * kBlock,
                                      true);
#pragma unroll
            for (int j = 1; j < KP; j++)
                load_page<D, GROUP, false>(a.p, a.pool, ln, at + j * P::kPage, __shfl_sync(0xffffffffu, blk, page + j - window),
                                           hk, n - (page + j) * kBlock, page + j < end);
            page += KP;
            at = at + KP * P::kPage == ring + STAGES * KP * P::kPage ? ring : at + KP * P::kPage;
            issued++;
            cp_async_commit();
        }
    }
};

// One share: its steps are in the ring or come.
template <int D, int GROUP, int E, int KP, int STAGES>
__device__ __forceinline__ void run_share(const Args &a, Smem4 &sm, const Lane<D, GROUP> &ln, int warp, Chunks &ch, unsigned ring,
                                          Loader<D, GROUP, KP, STAGES> &ld, unsigned &at, int &done, int closed, const Share sh)
{
    using P = PageQ<D, GROUP>;
    constexpr int NT = 1;
    const Params &p = a.p;
    const int n = sh.n, ql = sh.ql, cols = ql * p.G;
    unsigned qb[NT][D / 16][2];
    Vec<E> qs[NT][D / GROUP];
    load_q<D, GROUP, NT>(p, ln.lane, sh, cols, qb);
    q_sums<D, GROUP, NT, E>(qb, qs);
    const int v0 = sh.tile * 8 * NT;
    const int all = ql == 1 ? n : keys_seen(n, ql, v0 / p.G);      // the first row sees least
    State<D, GROUP, NT, E> s;
    s.e = 0;
#pragma unroll
    for (int nt = 0; nt < NT; nt++) {
        s.m[nt] = Vec<E>::all(kNegInf);
        s.l[nt] = Vec<E>::all(0.f);
#pragma unroll
        for (int gi = 0; gi < P::NG; gi++) s.z[nt][gi] = Vec<E>::all(0.f);
#pragma unroll
        for (int e = 0; e < 4; e++) {
#pragma unroll
            for (int gi = 0; gi < P::NG; gi++) s.c[nt][gi][e] = 0.f;
#pragma unroll
            for (int d = 0; d < D / 16; d++) s.o[nt][d][e] = 0.f;
        }
    }
    // pages that end below this are seen whole by every column
    const int full_end = min(sh.end, all / kBlock);
    for (int page = sh.page; page < sh.end; page += KP) {
        // the ring is full but at the end of the warp's work
        if (ld.issued - done == STAGES - 1) cp_async_wait<STAGES - 2>();
        else cp_async_wait<0>();
        __syncwarp();
        int end[NT][E];
        if (page + KP <= full_end) {
            step<D, GROUP, NT, E, KP, true>(at, ln, KP, qb, qs, s, end, p.scale_log2, a.slack);
        } else {
            const int t = ln.lane & 3, vlast = min(cols, v0 + 8 * NT) - 1;
#pragma unroll
            for (int nt = 0; nt < NT; nt++)
#pragma unroll
                for (int e = 0; e < E; e++)
                    end[nt][e] = (ql == 1 ? n : keys_seen(n, ql, min(v0 + 8 * nt + 2 * t + e, vlast) / p.G)) - page * kBlock;
            step<D, GROUP, NT, E, KP, false>(at, ln, sh.end - page, qb, qs, s, end, p.scale_log2, a.slack);
        }
        if ((page - sh.page) % kCentre == kCentre - KP) centre<D, GROUP, E>(s);
        __syncwarp();
        at = at + KP * P::kPage == ring + STAGES * KP * P::kPage ? ring : at + KP * P::kPage;
        ld.fill(a, sm, ln, warp, ch, ring, ++done, closed);
    }
    write_partial<D, GROUP, NT, E>(a, ln.lane, min(8 * NT, cols - v0), s, a.part0 + (long long)sh.part * a.nc);
}

// One share of a sequence of many columns.
template <int D, int GROUP, int NT, int KP, int STAGES>
__device__ __forceinline__ void run_wide(const Args &a, Smem4 &sm, const Lane<D, GROUP> &ln, int warp, Chunks &ch, unsigned ring,
                                         unsigned qsm, Loader<D, GROUP, KP, STAGES> &ld, unsigned &at, int &done, int closed,
                                         const Share sh)
{
    using P = PageQ<D, GROUP>;
    const Params &p = a.p;
    const int n = sh.n, ql = sh.ql, cols = ql * p.G;
    unsigned qz[NT];
    wide_q<D, GROUP, NT>(p, ln.lane, sh, cols, qsm, qz);
    const int v0 = sh.tile * 8 * NT, vlast = min(cols, v0 + 8 * NT) - 1;
    const int all = ql == 1 ? n : keys_seen(n, ql, v0 / p.G);      // the first row sees least
    Wide<D, GROUP, NT> s;
    s.e = 0;
#pragma unroll
    for (int nt = 0; nt < NT; nt++) {
        s.m[nt] = Vec<2>::all(kNegInf);
        s.l[nt] = Vec<2>::all(0.f);
#pragma unroll
        for (int e = 0; e < 4; e++) {
            s.z[nt][e] = 0.f;
#pragma unroll
            for (int d = 0; d < D / 16; d++) s.o[nt][d][e] = 0.f;
        }
    }
    const int full_end = min(sh.end, all / kBlock);
    for (int page = sh.page; page < sh.end; page += KP) {
        if (ld.issued - done == STAGES - 1) cp_async_wait<STAGES - 2>();
        else cp_async_wait<0>();
        __syncwarp();
#pragma unroll 1
        for (int j = 0; j < KP && page + j < sh.end; j++) {
            int end[NT][2];
            if (page + j < full_end) {
                wide_page<D, GROUP, NT, true>(at + j * P::kPage, ln, qsm, qz, s, end, p.scale_log2, a.slack);
            } else {
                const int t = ln.lane & 3;
#pragma unroll
                for (int nt = 0; nt < NT; nt++)
#pragma unroll
                    for (int e = 0; e < 2; e++)
                        end[nt][e] =
                            (ql == 1 ? n : keys_seen(n, ql, min(v0 + 8 * nt + 2 * t + e, vlast) / p.G)) - (page + j) * kBlock;
                wide_page<D, GROUP, NT, false>(at + j * P::kPage, ln, qsm, qz, s, end, p.scale_log2, a.slack);
            }
        }
        __syncwarp();
        at = at + KP * P::kPage == ring + STAGES * KP * P::kPage ? ring : at + KP * P::kPage;
        ld.fill(a, sm, ln, warp, ch, ring, ++done, closed);
    }
    write_partial<D, GROUP, NT>(a, ln.lane, min(8 * NT, cols - v0), s, a.part0 + (long long)sh.part * a.nc);
}

// ----------------------------------------------------------------------------- attention: kernels
// The context kernel: one CTA per SM, every warp on its own through chunks of
// the line.  Bound by memory on long contexts: 64 requests x 4096 keys x 32
// heads (D = 128, groups of 128, 1.14 GB) take 197 us with the merge, 5.8 TB/s
// of 6.7 for a copy; a call has about 12 us besides (the line, the first
// loads, the last partials and their merge), which is what remains of short
// ones: 16 us at the copy rate and 37 us for 32 requests of 64 to 1024 keys with
// a prompt of 2048.  With eight query heads a KV head and groups of 64 the
// arithmetic comes near: 85 us, 49 at the copy rate (32 requests, 1000 to 16384 keys).
//  NT: tensor-core tiles of columns that a sequence may have; E as
// in State.  It starts beside a grid in front of it that computes the prompt's
// partials (whichever SMs that leaves) and ends only after it.
template <int D, int GROUP, int NT, int E>
__global__ void __launch_bounds__(Geo<D, GROUP, NT>::kW * 32, 1) ctx_kernel(const __grid_constant__ Args a)
{
    using G = Geo<D, GROUP, NT>;
    extern __shared__ __align__(128) unsigned char smem_raw[];
    Smem4 &s = *reinterpret_cast<Smem4 *>(smem_raw);
    const Params &p = a.p;
    const int warp = threadIdx.x >> 5;
    Chunks ch;
    ch.count = 1;      // (asked for before the number of chunks is known)
    ch.queue0 = 0;
    if (a.queue) ch.ask(p);
    build_line<G::kW>(p, s, a.rows_max);
    const long long total = s.pre[p.B], workers = (long long)gridDim.x * G::kW;
    // Pages of a chunk: one chunk a warp where the warps start together (two
    // only cost partials and starts: 32 x 32768 keys of 8 heads 69 -> 77 us, 64 x
    // 4096 of 32 heads 197 -> 199), four where the CTAs follow a grid in front
    // of them as its CTAs leave (prompt chunks beside twelve decode requests:
    // 236, 204, 196, 193 and 194 us with one, two, three, four and six)
    const int parts = a.queue ? 4 : 1;
    const int Q = (int)max((long long)a.q_min, (total + workers * parts - 1) / (workers * parts));
    const unsigned bad = (unsigned)s.bad | (s.qo[p.B] > p.max_q_total ? FLAG_Q_TOTAL : 0u);
    if (blockIdx.x == 0) {
        const Sched sc = sched_at(p.sched, p.B);
        for (int k = threadIdx.x; k <= p.B; k += G::kW * 32) {
            sc.pre[k] = s.pre[k];
            sc.qo[k] = s.qo[k];
            sc.seq[k] = s.seq[k];
        }
        if (threadIdx.x == 0) {
            p.sched[0] = bad ? -1 : 0;
            p.sched[1] = Q;
            if (bad) atomicOr(&p.ctrl[CTRL_FLAGS], bad);
        }
    }
    ch.total = total;
    ch.count = (total + Q - 1) / Q;
    const long long first = a.queue ? ch.take() : (long long)warp * gridDim.x + blockIdx.x;
    ch.queue0 = a.queue ? 0 : workers;
    ch.Q = Q;
    if (!bad && first < ch.count) {
        const unsigned ring = smem_u32(s.ring) + warp * (G::kStages * G::kStep);
        const unsigned qsm = smem_u32(s.ring) + G::kW * (G::kStages * G::kStep) + warp * G::kQ;
        Lane<D, GROUP> ln;
        ln.init(a.pool);
        ch.ask(p);
        if (ln.lane == 0) {
            Walk w;
            w.q = locate(p, s, first * Q);
            w.left = (int)min((long long)Q, total - first * Q);
            s.walk[warp] = w;
        }
        __syncwarp();
        Loader<D, GROUP, G::kPer, G::kStages> ld;
        ld.chunk = first;
        ld.page = ld.end = ld.issued = ld.opened = 0;
        ld.at = ring;
        unsigned at = ring;
        for (int done = 0, closed = 0;; closed++) {
            ld.fill(a, s, ln, warp, ch, ring, done, closed);
            if (ld.opened == closed) break;      // no share is left
            const Share sh = s.share[warp][closed % kShares];
            const int cols = sh.ql * p.G;
            if constexpr (NT == 4) {
                if (cols > 16) {
                    run_wide<D, GROUP, 4>(a, s, ln, warp, ch, ring, qsm, ld, at, done, closed, sh);
                    continue;
                }
            }
            if constexpr (NT > 1) {
                if (cols > 8) {
                    run_wide<D, GROUP, 2>(a, s, ln, warp, ch, ring, qsm, ld, at, done, closed, sh);
                    continue;
                }
            }
            run_share<D, GROUP, E>(a, s, ln, warp, ch, ring, ld, at, done, closed, sh);
        }
        cp_async_wait<0>();
    }
    __syncthreads();
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
}

// ----------------------------------------------------------------------------- attention: prompt chunks
// Requests of more columns than the line takes: a dense contraction, on the
// 5th-generation tensor cores.  A CTA takes 128 columns of one KV head (a TMEM
// lane each) against a range of the context, 64 keys a stage.  Its warps:
//   0-3, 4-7   softmax of the even and of the odd stages, each with a reference,
//              a sum and an O of its own (joined at the item's end): thread t of
//              them has column t, so a maximum needs no other lane.  One thread
//              of each issues the products: a stage's P V, then, when P has been
//              read, the Q K^T of the stage after the next in its place.
//   8-15       unpack: codes and pairs come from global memory to registers a
//              stage ahead, and go to shared memory as fp16 tiles (128-byte
//              swizzle), three stages of them.
// With c the codes and s = s' + s" a scale cut after 7 bits, c s' and c s" are
// exact in fp16, and so is S but for its fp32 sums:
//     S = Q (c s')^T + sum(q) z^T, and Q (c s")^T   (M 128, N 2 x 64, K D and 16; the softmax adds them)
//     O += P V                                      (V = fma(c, s, z), one fp16 rounding; P in two halves, which
//                                                    have 22 bits of it: with P in one, too, the error of the
//                                                    results would be half as large again)
// sum(q) of a group is two halves, the first 2^-7 of itself against 2^7 z, the
// second what that leaves.  P takes the place of its S in TMEM.
// What fp16 does not hold is kept out of the tiles: a key whose K or V would
// leave its range is stored 2^-11 or 2^-5 of itself, with a bit for the softmax,
// and a V pair that is no number as zeros, with a bit of its group that makes
// NaNs of the columns that see the key, and of no other.
// The tiles hold a word's eight dimensions in the order of the unpacking, 0 4
// 1 5 2 6 3 7; Q is stored in that order and the output written back from it.

struct RowItems {
    int qo[kMaxB + 1];        // query rows before request b
    int it[kMaxB + 1];        // items before request b
    long long sum[16];
    int sum_q[16], most[16];
    int bad, next[2];
};
// An item, in shared memory (what a role uses of it would cost registers).
struct RowsItem {
    int b, hk, n, ql, v0, vlast, page0, end_page, n_st, part;
};

constexpr int kRowsThreads = 512;
template <int D, int GROUP>
struct RowsSmem {
    static constexpr int NG = D / GROUP, KH = D / 64;      // KH: 64-dimension halves of a row
    static constexpr int kQHalf = kRowsTile * 128, kKHalf = kRowsKeys * 128;
    unsigned char q[KH * kQHalf];
    static constexpr int kStages = 3;
    unsigned char k[kStages][KH][2 * kKHalf];      // 64 keys c s', 64 keys c s"
    unsigned char v[kStages][KH * kKHalf];
    unsigned char qz[kRowsTile * 32];        // [16][2][8] pieces of 16 bytes: row, half of the 16 terms
    unsigned char kz[kStages][kRowsKeys * 32];
    unsigned long long bar[16];
    // stage i mod 4: a bit a key (a byte eight of them); v_odd: 1 scaled, 2 no number
    unsigned char kbig[4][8], vbig[4][8], vnan[4][NG][8], v_odd[4][8];
    float2 ml[2][kRowsTile];                 // a column's reference and sum
    unsigned nan[2][kRowsTile];              // its groups of V that are no numbers
    RowItems s;
    RowsItem r[2];
    unsigned tmem;
    int abort;
};
template <int D, int GROUP>
constexpr size_t kRowsSmem = sizeof(RowsSmem<D, GROUP>) + 1024;      // (from a 1024-byte boundary on)
// full, free: of a stage's tiles; the others of the even and the odd stages
enum { ROWS_QFULL, ROWS_FIN, ROWS_SFULL, ROWS_PREADY = ROWS_SFULL + 2, ROWS_PVDONE = ROWS_PREADY + 2, ROWS_FULL = ROWS_PVDONE + 2,
       ROWS_FREE = ROWS_FULL + 3 };
constexpr unsigned kRowsTmem = 512, kRowsColS = 0, kRowsColO = 256;      // S (its two parts; or P) of stage i: 128 (i & 1); O: 128 (i & 1)

// descriptor of 8 x 16-byte pieces without swizzle: the row's next 16 bytes
// 128 bytes on, the next eight rows 256
__device__ __forceinline__ uint64_t plain_desc(unsigned saddr)
{
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (uint64_t)(128u >> 4) << 16 | (uint64_t)(256u >> 4) << 32 | (uint64_t)1 << 46;
}
// a descriptor that is made where it is used (the many of a stage would be
// kept in registers, and those in local memory)
__device__ __forceinline__ uint64_t pinned(uint64_t d)
{
    uint64_t r;
    asm volatile("mov.b64 %0, %1;" : "=l"(r) : "l"(d));
    return r;
}

// Pages of a split, from the batch's pages of all items and of its longest
// context: about two items an SM (an item costs 7 us apart from its stages; with
// three or four 7 and 15 us more for 482 rows over 3700 keys, 40 heads), at
// most kRowsParts of a context, whole stages.
constexpr int kRowsParts = 8, kRowsPages = 32;
__device__ __forceinline__ int split_pages(long long work, int most, int grid)
{
    const long long even = min(256ll, (work + 2 * grid - 1) / (2 * grid));
    return ((int)max((long long)max(kRowsPages, (most + kRowsParts - 1) / kRowsParts), even) + 3) / 4 * 4;
}
__device__ __forceinline__ int rows_tiles(int cols) { return (cols + kRowsTile - 1) / kRowsTile; }

// The items of the batch (at least 256 threads): items prefix, and the split.
__device__ __forceinline__ int build_rows(const Params &p, RowItems &s, int rows_max)
{
    constexpr int PER = kMaxB / 256;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int ql[PER], pages[PER], sum_q = 0, most = 0, bad = 0;
    long long work = 0;
    if (tid == 0) s.bad = 0;
#pragma unroll
    for (int k = 0; k < PER; k++) {
        const int b = tid * PER + k;
        ql[k] = pages[k] = 0;
        if (b < p.B) {
            ql[k] = p.q_lens ? p.q_lens[b] : p.Lq;
            const int n = p.ctx_lens[b];
            if (ql[k] < 0 || ql[k] > p.Lq || n < 0 || n > p.max_blocks * kBlock) bad = 1;      // (the context kernel reports it)
            else pages[k] = (n + kBlock - 1) / kBlock;
        }
        sum_q += ql[k];
        if (ql[k] * p.G > rows_max) {
            work += (long long)p.Hkv * rows_tiles(ql[k] * p.G) * pages[k];
            most = max(most, pages[k]);
        }
    }
    int iq = sum_q;
    long long iw = work;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, iq, off);
        const long long tw = __shfl_up_sync(0xffffffffu, iw, off);
        if (lane >= off) { iq += t; iw += tw; }
    }
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 31) {
        s.sum_q[warp] = iq;
        s.sum[warp] = iw;
        s.most[warp] = most;
    }
    __syncthreads();
    if (bad) s.bad = 1;
    int bq = iq - sum_q;
    long long total = 0;
    for (int j = 0; j < 8; j++) {
        if (j < warp) bq += s.sum_q[j];
        total += s.sum[j];
        most = max(most, s.most[j]);
    }
    const int split = split_pages(total, most, gridDim.x);
    int n_it[PER], sum_i = 0;
#pragma unroll
    for (int k = 0; k < PER; k++) {
        const int b = tid * PER + k;
        if (b < p.B) s.qo[b] = bq;
        bq += ql[k];
        n_it[k] = ql[k] * p.G > rows_max ? p.Hkv * rows_tiles(ql[k] * p.G) * ((pages[k] + split - 1) / split) : 0;
        sum_i += n_it[k];
    }
    if (tid == 255) s.qo[p.B] = bq;
    __syncthreads();      // (the sums have been read)
    int ii = sum_i;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, ii, off);
        if (lane >= off) ii += t;
    }
    if (lane == 31) s.sum_q[warp] = ii;
    __syncthreads();
    int bi = ii - sum_i;
    for (int j = 0; j < warp; j++) bi += s.sum_q[j];
#pragma unroll
    for (int k = 0; k < PER; k++) {
        const int b = tid * PER + k;
        if (b < p.B) s.it[b] = bi;
        bi += n_it[k];
    }
    if (tid == 255) s.it[p.B] = bi;
    __syncthreads();
    return split;
}

__device__ __forceinline__ void sts128(unsigned a, unsigned x, unsigned y, unsigned z, unsigned w)
{
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ void tmem_st8(unsigned taddr, const unsigned (&r)[8])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

// What is rare stays out of the loops: four roles' code passes through a
// scheduler's instruction cache, and what it does not hold runs at a tenth of
// the rate.
__device__ __noinline__ bool rows_wait_long(unsigned bar, unsigned parity, volatile int *abort)
{
    if constexpr (tc::kWaitNs > 0) {
        return tc::mbar_wait(bar, parity, abort);
    } else {
        *abort = 1;
        return false;
    }
}
// (a limit of 0: a wait that is not met at once gives up)
__device__ __forceinline__ bool rows_wait(unsigned bar, unsigned parity, volatile int *abort)
{
    if constexpr (tc::kWaitNs > 0) return tc::mbar_try(bar, parity) || rows_wait_long(bar, parity, abort);
    return tc::mbar_test(bar, parity) || rows_wait_long(bar, parity, abort);
}
// All ones in the bytes of x that have bit `b`.
__device__ __forceinline__ unsigned rows_bytes(unsigned x, unsigned b) { return (x & 0x01010101u * b) / b * 255u; }
// Scores in TMEM, two parts: the keys of `big` times 2048, those from `seen` on
// hidden.
__device__ __noinline__ void rows_fix_scores(unsigned tS, unsigned long long big, int seen)
{
#pragma unroll 1
    for (int c = 0; c < 128; c += 32) {
        const int key = c & 63;
        unsigned x[32];
        tc::tmem_ld32(tS + c, x);
        tc::tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < 32; k++) {
            if (big >> key >> k & 1) x[k] = __float_as_uint(__uint_as_float(x[k]) * 2048.f);
            if (key + k >= seen) x[k] = c < 64 ? __float_as_uint(kNegInf) : 0u;
        }
        tc::tmem_st32(tS + c, x);
    }
    tc::tmem_wait_st();
}
// Weights in TMEM, two halves each: the keys of `big` times 32.
__device__ __noinline__ void rows_fix_weights(unsigned tP, unsigned long long big)
{
    tc::tmem_wait_st();
#pragma unroll 1
    for (int c = 0; c < 64; c += 32) {
        unsigned x[32];
        tc::tmem_ld32(tP + c, x);
        tc::tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < 32; k++) {
            const __half2 f = __floats2half2_rn(big >> (2 * k) & 1 ? 32.f : 1.f, big >> (2 * k + 1) & 1 ? 32.f : 1.f);
            const __half2 y = __hmul2(*reinterpret_cast<const __half2 *>(&x[k]), f);
            x[k] = *reinterpret_cast<const unsigned *>(&y);
        }
        tc::tmem_st32(tP + c, x);
    }
}
// An O of W columns times f.
template <int W>
__device__ __noinline__ void rows_scale(unsigned tO, float f)
{
#pragma unroll 1
    for (int c = 0; c < W; c += 32) {
        unsigned o[32];
        tc::tmem_ld32(tO + c, o);
        tc::tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < 32; k++) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
        tc::tmem_st32(tO + c, o);
    }
}

// A thread's part of a stage on its way: 32 dimensions of a key, of K and of V
// (D = 128; D = 64: the first four warps have K, the others V).  Eight lanes
// that store together are four keys and two neighbouring pieces: no bank twice.
template <int D, int GROUP>
struct Pieces {
    using S = RowsSmem<D, GROUP>;
    static constexpr int NG = S::NG;
    static constexpr int kBytes = D == 128 ? 1 : 2;      // a warp's keys are eight, or 16
    uint4 k, v;
    unsigned ksz, vsz;

    static __device__ __forceinline__ bool has_k(int u) { return D == 128 || u < 128; }
    static __device__ __forceinline__ bool has_v(int u) { return D == 128 || u >= 128; }
    static __device__ __forceinline__ int piece(int u) { return D == 128 ? (u & 1) | (u >> 2 & 2) : u & 1; }
    static __device__ __forceinline__ int key(int u)
    {
        return D == 128 ? (u >> 5) * 8 + (u >> 1 & 3) + (u >> 2 & 4) : u >> 1 & 63;
    }
    static __device__ __forceinline__ unsigned key_lanes(int first) { return (D == 128 ? 0x303u : 3u) << first; }
    // the warp's keys of a ballot: byte `lane` of them
    static __device__ __noinline__ unsigned char keys_of(unsigned b, int lane)
    {
        unsigned r = 0;
#pragma unroll
        for (int i = 0; i < 8 * kBytes; i++) r |= (b & key_lanes(D == 128 ? (i & 3) << 1 | (i & 4) << 2 : 2 * i)) ? 1u << i : 0u;
        return (unsigned char)(r >> (8 * lane & 31));
    }
    static __device__ __forceinline__ bool of_key(unsigned b, int lane) { return b & key_lanes(lane & (D == 128 ? ~9 : ~1)); }

    static __device__ __forceinline__ int id(const int *table, int u, int page0, int end)
    {
        const int page = page0 + key(u) / kBlock;
        return page < end ? __ldg(table + page) : -1;
    }
    // places of the thread's key and piece in a block
    static __device__ __forceinline__ unsigned codes_at(int u, int hk)
    {
        return ((unsigned)hk * kBlock + key(u) % kBlock) * (D / 2) + 16 * piece(u);
    }
    static __device__ __forceinline__ unsigned pairs_at(int u, int hk)
    {
        return ((unsigned)hk * kBlock + key(u) % kBlock) * NG + piece(u) * 32 / GROUP;
    }
    __device__ __forceinline__ void load(const Params &p, const Pool &pool, unsigned codes, unsigned pairs, int u, int page0, int end,
                                         int n, int blk)
    {
        k = v = make_uint4(0u, 0u, 0u, 0u);
        ksz = vsz = 0u;
        if ((unsigned)blk >= (unsigned)p.num_blocks) {
            if (page0 + key(u) / kBlock < end) atomicOr(&p.ctrl[CTRL_FLAGS], FLAG_BAD_BLOCK);
        } else {
            const size_t at = (size_t)blk * (unsigned)(p.Hkv * kBlock * (D / 2)) + codes;
            const size_t at_sz = (size_t)blk * (unsigned)(p.Hkv * kBlock * NG) + pairs;
            // pairs of tokens behind the last one are zero
            const bool in = page0 * kBlock + key(u) < n;
            if (has_k(u)) {
                k = __ldg(reinterpret_cast<const uint4 *>(pool.k + at));
                if (in) ksz = __ldg(reinterpret_cast<const unsigned *>(pool.ksz) + at_sz);
            }
            if (has_v(u)) {
                v = __ldg(reinterpret_cast<const uint4 *>(pool.v + at));
                if (in) vsz = __ldg(reinterpret_cast<const unsigned *>(pool.vsz) + at_sz);
            }
        }
    }
    // Codes of word w, dimensions k and k + 4, as halves 1024 + c (k even) and 64 + c.
    static __device__ __forceinline__ void raised(unsigned w, __half2 (&c)[4])
    {
#pragma unroll
        for (int k = 0; k < 4; k += 2) {
            const unsigned x = w >> (4 * k), lo = (x & kLoCodes) | 0x64006400u, hi = (x & kHiCodes) | 0x54005400u;
            c[k] = *reinterpret_cast<const __half2 *>(&lo);
            c[k + 1] = *reinterpret_cast<const __half2 *>(&hi);
        }
    }
    // Its first store into a tile at `tile`.
    template <int HALF>      // bytes of a tile of 64 dimensions
    static __device__ __forceinline__ unsigned first(unsigned tile, int u)
    {
        const int ch = piece(u);
        unsigned x;      // (not kept through the loop in 24 addresses)
        asm volatile("add.u32 %0, %1, %2;" : "=r"(x) : "r"(tile), "r"((ch >> 1) * HALF + tc::sw_off(key(u), 4 * (ch & 1))));
        return x;
    }
    static __device__ __forceinline__ void put(unsigned at, int j, const __half2 (&x)[4])
    {
        const unsigned *w = reinterpret_cast<const unsigned *>(x);
        sts128(at ^ (j << 4), w[0], w[1], w[2], w[3]);
    }
    static __device__ __forceinline__ float2 pair(unsigned w) { return __half22float2(*reinterpret_cast<const __half2 *>(&w)); }
    static __device__ __forceinline__ __half2 both(unsigned w, unsigned sel)
    {
        const unsigned x = __byte_perm(w, 0u, sel);
        return *reinterpret_cast<const __half2 *>(&x);
    }
    static __device__ __forceinline__ bool number(unsigned w) { return (w & 0x7c00u) != 0x7c00u && (w & 0x7c000000u) != 0x7c000000u; }
    static __device__ __forceinline__ void times(unsigned &w, float f)
    {
        const float2 x = pair(w);
        const __half2 h = __floats2half2_rn(x.x * f, x.y * f);
        w = *reinterpret_cast<const unsigned *>(&h);
    }
    // c s = (1024 + c) s - 1024 s, exact for a scale of at most seven bits
    // whose 1024 s is a half, and the same with 64.
    __device__ __forceinline__ void unpack_k(S &sm, int at, int slot, int u)
    {
        const int lane = u & 31, ch = piece(u), kk = key(u);
        const unsigned to = first<2 * S::kKHalf>(smem_u32(sm.k[at][0]), u);
        const float2 f = pair(ksz);
        const unsigned any = __ballot_sync(0xffffffffu, fabsf(f.x) >= 60.f || fabsf(f.y) >= 511.f);
        unsigned char bits = 0;
        if (any) {
            bits = keys_of(any, lane);
            if (of_key(any, lane)) times(ksz, 0x1p-11f);
        }
        if (lane < kBytes) sm.kbig[slot][kk / 8 + lane] = bits;
        const unsigned s1 = __byte_perm(ksz, 0u, 0x1010), s1h = s1 & 0xfff0fff0u;
        const __half2 sh = *reinterpret_cast<const __half2 *>(&s1h), sl = __hsub2(*reinterpret_cast<const __half2 *>(&s1), sh);
        const __half2 k0 = __floats2half2_rn(-1024.f, -1024.f), k1 = __floats2half2_rn(-64.f, -64.f);
        const __half2 sh0 = __hmul2(sh, k0), sh1 = __hmul2(sh, k1), sl0 = __hmul2(sl, k0), sl1 = __hmul2(sl, k1);
        const unsigned w[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
        for (int j = 0; j < 4; j++) {
            __half2 x[4], h[4], l[4];
            raised(w[j], x);
#pragma unroll
            for (int i = 0; i < 4; i++) {
                h[i] = __hfma2(x[i], sh, i & 1 ? sh1 : sh0);
                l[i] = __hfma2(x[i], sl, i & 1 ? sl1 : sl0);
            }
            put(to, j, h);
            put(to + S::kKHalf, j, l);
        }
        if (ch * 32 % GROUP == 0) {
            const int gi = ch * 32 / GROUP;
            const __half z = __ushort_as_half((unsigned short)(ksz >> 16));
            __half *terms = reinterpret_cast<__half *>(sm.kz[at] + kk / 8 * 256 + kk % 8 * 16);
            terms[gi] = __hmul(z, __float2half_rn(1.f / kQsScale));
            terms[NG + gi] = z;      // (at most eight terms: the first 16 bytes)
        }
    }
    __device__ __forceinline__ void unpack_v(S &sm, int at, int slot, int u)
    {
        const int lane = u & 31, ch = piece(u), byte = key(u) / 8 + lane;
        const unsigned to = first<S::kKHalf>(smem_u32(sm.v[at]), u);
        const float2 f = pair(vsz);
        const bool odd = !(fmaf(15.f, fabsf(f.x), fabsf(f.y)) < 65504.f);
        unsigned char bits = 0;
        if (__any_sync(0xffffffffu, odd)) {
            const bool num = number(vsz);
            const unsigned any = __ballot_sync(0xffffffffu, num && odd), none = __ballot_sync(0xffffffffu, !num);
            const unsigned char b = keys_of(any, lane);
            if (lane < kBytes) sm.vbig[slot][byte] = b;
#pragma unroll 1
            for (int gi = 0; gi < NG; gi++) {
                const unsigned char g = keys_of(__ballot_sync(0xffffffffu, !num && ch * 32 / GROUP == gi), lane);
                if (lane < kBytes) sm.vnan[slot][gi][byte] = g;
            }
            bits = (any ? 1 : 0) | (none ? 2 : 0);
            if (!num) vsz = 0u;
            if (of_key(any, lane)) times(vsz, 0x1p-5f);
        }
        if (lane < kBytes) sm.v_odd[slot][byte] = bits;
        const __half2 s = both(vsz, 0x1010), z = both(vsz, 0x3232);
        const __half2 k0 = __floats2half2_rn(-1024.f, -1024.f), k1 = __floats2half2_rn(-64.f, -64.f);
        const unsigned w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; j++) {
            __half2 x[4];
            raised(w[j], x);
#pragma unroll
            for (int i = 0; i < 4; i++) x[i] = __hfma2(__hadd2(x[i], i & 1 ? k1 : k0), s, z);
            put(to, j, x);
        }
    }
};

__device__ __forceinline__ RowsItem rows_item(const Params &p, const RowItems &s, int item, int split)
{
    RowsItem r;
    r.b = find_owner(s.it, p.B, item);
    r.n = p.ctx_lens[r.b];
    r.ql = s.qo[r.b + 1] - s.qo[r.b];
    const int cols = r.ql * p.G, pages = (r.n + kBlock - 1) / kBlock, tiles = rows_tiles(cols);
    int j = item - s.it[r.b];
    r.hk = j % p.Hkv;      // (KV heads next to each other: they share the split's length)
    j /= p.Hkv;
    const int tile = j % tiles;
    r.part = j / tiles;
    r.v0 = tile * kRowsTile;
    r.vlast = min(cols, r.v0 + kRowsTile) - 1;
    r.page0 = r.part * split;
    r.end_page = min(min(r.page0 + split, pages), (keys_seen(r.n, r.ql, r.vlast / p.G) + kBlock - 1) / kBlock);
    r.n_st = r.end_page > r.page0 ? (r.end_page - r.page0 + 3) / 4 : 0;
    return r;
}

// Partial row of a column.
__device__ __forceinline__ size_t rows_slot(const Args &a, const RowItems &s, const RowsItem &r, int v)
{
    const int i = v / a.p.G;
    return (size_t)a.rows0 + ((size_t)r.part * a.p.max_q_total + s.qo[r.b] + i) * a.p.H + r.hk * a.p.G + v - i * a.p.G;
}

// What bounds it: 482 rows against 3300 to 4100 keys of 40 heads (D = 128, groups
// of 32) are 24 us of products at the measured dense rate, and take 95 us of
// the SMs.  A stage is 1.2 us: unpacking (12 stores of 16 bytes and their
// arithmetic a thread, 0.9 us), the softmax (0.6) and the products
// (0.6) overlap, but a scheduler's instruction cache passes three kinds of code,
// and an item has 7 us apart from its stages.  The form before it (mma.sync,
// eight warps of 16 columns over codes in shared memory) was bound by the
// shared-memory reads of its operands and took 215 us.
template <int D, int GROUP>
__global__ void __launch_bounds__(kRowsThreads, 1) rows_kernel(const __grid_constant__ Args a)
{
    using S = RowsSmem<D, GROUP>;
    using X = Pieces<D, GROUP>;
    constexpr int NG = S::NG;
    constexpr uint32_t id_s = tc::idesc_f16(kRowsTile, 2 * kRowsKeys), id_z = tc::idesc_f16(kRowsTile, kRowsKeys), id_o = tc::idesc_f16(kRowsTile, D, true);
    extern __shared__ unsigned char smem_rows[];
    S &sm = *reinterpret_cast<S *>(smem_rows + (-smem_u32(smem_rows) & 1023u));
    const Params &p = a.p;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    auto bar = [&](int i) { return smem_u32(sm.bar) + 8u * (unsigned)i; };
    volatile int *abort_p = &sm.abort;
    const int split = build_rows(p, sm.s, a.rows_max);
    if (blockIdx.x == 0 && tid == 0) p.sched[2] = split;
    const bool run = !sm.s.bad && sm.s.qo[p.B] <= p.max_q_total;
    const int n_items = run ? sm.s.it[p.B] : 0;
    if ((int)blockIdx.x >= n_items) {
        asm volatile("griddepcontrol.wait;\n" ::: "memory");
        return;
    }
    if (warp == 8) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(smem_u32(&sm.tmem)), "n"(kRowsTmem)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
    }
    if (tid == 0) {
        sm.abort = 0;
        tc::mbar_init(bar(ROWS_QFULL), 8);
        tc::mbar_init(bar(ROWS_FIN), 2);
        for (int i = 0; i < S::kStages; i++) {
            tc::mbar_init(bar(ROWS_FULL + i), 8);
            tc::mbar_init(bar(ROWS_FREE + i), 1);
        }
        for (int i = 0; i < 2; i++) {
            tc::mbar_init(bar(ROWS_SFULL + i), 1);
            tc::mbar_init(bar(ROWS_PREADY + i), 4);
            tc::mbar_init(bar(ROWS_PVDONE + i), 1);
        }
        sm.r[0] = rows_item(p, sm.s, blockIdx.x, split);
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    }
    // terms that no group has
    for (int i = tid; i < (int)sizeof(sm.kz) / 4; i += kRowsThreads) reinterpret_cast<unsigned *>(sm.kz)[i] = 0u;
    for (int i = tid; i < (int)sizeof(sm.qz) / 4; i += kRowsThreads) reinterpret_cast<unsigned *>(sm.qz)[i] = 0u;
    tc::fence_async_smem();
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const unsigned tmem = sm.tmem;
    // Both halves of the CTA go through the same items; J: stages before the item.
    if (warp < 8) {
        unsigned q_items = 0;      // items with stages before it
        for (int item = blockIdx.x, turn = 0, J = 0; item < n_items; turn ^= 1) {
            const RowsItem &r = sm.r[turn];
            bool ok = true;
            // ------------------------------------------------------------ softmax, Q and the output
            const int e = warp >> 2, row = tid & 127;
            const bool have = r.v0 + row <= r.vlast;
            const unsigned lane_off = (unsigned)((warp & 3) * 32) << 16;
            // keys that the row sees, of the range (rows that are none hide
            // nothing: what they come to is not written)
            int end = r.end_page * kBlock;
            if (have) end = min(end, keys_seen(r.n, r.ql, (r.v0 + row) / p.G));
            if (r.n_st > 0) {
                // Q: a warp has kR rows at a time, 16 bytes a lane
                constexpr int kL = D / 8, kR = 32 / kL, kT = kRowsTile / (8 * kR);
                const int c = lane % kL;
                uint4 x[kT];
#pragma unroll
                for (int k = 0; k < kT; k++) {
                    const int v = r.v0 + (warp * kT + k) * kR + lane / kL, i = v / p.G;
                    x[k] = make_uint4(0u, 0u, 0u, 0u);
                    if (v <= r.vlast)
                        x[k] = __ldg(reinterpret_cast<const uint4 *>(p.q + (((size_t)r.b * p.Lq + i) * p.H + r.hk * p.G + v - i * p.G) * D) + c);
                }
#pragma unroll
                for (int k = 0; k < kT; k++) {
                    const int at = (warp * kT + k) * kR + lane / kL;
                    sts128(smem_u32(sm.q) + (c >> 3) * S::kQHalf + tc::sw_off(at, c & 7), __byte_perm(x[k].x, x[k].z, 0x5410),
                           __byte_perm(x[k].x, x[k].z, 0x7632), __byte_perm(x[k].y, x[k].w, 0x5410), __byte_perm(x[k].y, x[k].w, 0x7632));
                    // the groups' sums, then their remainders
                    const float2 y0 = X::pair(x[k].x), y1 = X::pair(x[k].y), y2 = X::pair(x[k].z), y3 = X::pair(x[k].w);
                    float f = ((y0.x + y0.y) + (y1.x + y1.y)) + ((y2.x + y2.y) + (y3.x + y3.y));
#pragma unroll
                    for (int off = 1; off < GROUP / 8; off <<= 1) f += __shfl_xor_sync(0xffffffffu, f, off);
                    if (c % (GROUP / 8) == 0) {
                        const __half hi = __float2half_rn(f * kQsScale);
                        __half *terms = reinterpret_cast<__half *>(sm.qz + at / 8 * 256 + at % 8 * 16) + c / (GROUP / 8);
                        terms[0] = hi;
                        terms[NG] = __float2half_rn(f - __half2float(hi) * (1.f / kQsScale));
                    }
                }
                tc::fence_async_smem();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(bar(ROWS_QFULL));
            }
            auto issue_s = [&](int j) {      // S = Q K^T, by one thread
                const int at = j % S::kStages;
                ok = rows_wait(bar(ROWS_FULL + at), (j / S::kStages) & 1, abort_p);
                if (!ok) return;
                tc::tc_fence_after();
                const unsigned d0 = tmem + kRowsColS + 128 * e;
                const uint64_t qd = pinned(tc::sw128_desc(smem_u32(sm.q))), kd = pinned(tc::sw128_desc(smem_u32(sm.k[at][0])));
#pragma unroll
                for (int kk = 0; kk < D / 16; kk++)
                    tc::umma_ss(d0, qd + (((kk >> 2) * S::kQHalf + (kk & 3) * 32) >> 4),
                                kd + (((kk >> 2) * 2 * S::kKHalf + (kk & 3) * 32) >> 4), id_s, kk > 0);
                tc::umma_ss(d0, pinned(plain_desc(smem_u32(sm.qz))), pinned(plain_desc(smem_u32(sm.kz[at]))), id_z, 1);
                tc::umma_commit(bar(ROWS_SFULL + e));
            };
            const int st0 = (J + e) & 1;      // its first stage of the item
            if ((warp & 3) == 0 && lane == 0 && st0 < r.n_st) {
                ok = rows_wait(bar(ROWS_QFULL), q_items & 1, abort_p);
                if (ok) issue_s(J + st0);
            }
            __syncwarp();
            float m = kNegInf, l = 0.f;
            unsigned nan = 0;
            const unsigned tS = tmem + kRowsColS + 128 * e + lane_off, tO = tmem + kRowsColO + 128 * e + lane_off;
            for (int st = st0; st < r.n_st; st += 2) {
                const int j = J + st, key0 = (r.page0 + 4 * st) * kBlock;
                ok = ok && rows_wait(bar(ROWS_SFULL + e), (j >> 1) & 1, abort_p);
                if (!__all_sync(0xffffffffu, ok)) break;
                tc::tc_fence_after();
                const unsigned *flags = reinterpret_cast<const unsigned *>(sm.kbig[j & 3]);
                const unsigned k0 = flags[0], k1 = flags[1];
                flags = reinterpret_cast<const unsigned *>(sm.v_odd[j & 3]);
                const unsigned v0 = flags[0], v1 = flags[1], v_odd = v0 | v1;
                const int seen = end - key0;
                if (__any_sync(0xffffffffu, seen < kRowsKeys || (k0 | k1))) rows_fix_scores(tS, (unsigned long long)k1 << 32 | k0, seen);
                if (v_odd & 0x02020202u) {
                    const unsigned long long odd = (unsigned long long)rows_bytes(v1, 2) << 32 | rows_bytes(v0, 2);
                    const unsigned long long mask = seen >= 64 ? ~0ull : seen <= 0 ? 0ull : (1ull << seen) - 1ull;
#pragma unroll 1
                    for (int gi = 0; gi < NG; gi++)
                        if (*reinterpret_cast<const unsigned long long *>(sm.vnan[j & 3][gi]) & mask & odd) nan |= 1u << gi;
                }
                float x[64];
#pragma unroll
                for (int h = 0; h < 2; h++) {      // the two parts together
                    unsigned y[2][32];
                    tc::tmem_ld32(tS + 32 * h, y[0]);
                    tc::tmem_ld32(tS + 32 * h + 64, y[1]);
                    tc::tmem_wait_ld();
#pragma unroll
                    for (int k = 0; k < 32; k += 2)
                        tc::f2_unpack(tc::f2_add(tc::f2_pack(__uint_as_float(y[0][k]), __uint_as_float(y[0][k + 1])),
                                                 tc::f2_pack(__uint_as_float(y[1][k]), __uint_as_float(y[1][k + 1]))),
                                      x[32 * h + k], x[32 * h + k + 1]);
                }
                float mx[4];
#pragma unroll
                for (int k = 0; k < 4; k++) {
                    mx[k] = fmaxf(x[k], x[4 + k]);
#pragma unroll
                    for (int c = 8; c < 64; c += 8) mx[k] = tc::max3f(mx[k], x[c + k], x[c + 4 + k]);
                }
                const float top = fmaxf(tc::max3f(mx[0], mx[1], mx[2]), mx[3]);
                const bool move = top > m + a.slack;
                const bool moved = __any_sync(0xffffffffu, move);
                float al = 1.f;
                if (moved) {
                    const float mn = move ? top : m;
                    al = move ? ex2((m - mn) * p.scale_log2) : 1.f;
                    m = mn;
                    l *= al;
                }
                const float mu = m == kNegInf ? 0.f : -m * p.scale_log2;
                const unsigned long long sc2 = tc::f2_pack(p.scale_log2, p.scale_log2), mu2 = tc::f2_pack(mu, mu);
                unsigned long long ls[2] = {0ull, 0ull};
#pragma unroll
                for (int i = 0; i < 64; i += 16) {
                    unsigned pk[8], rest[8];
#pragma unroll
                    for (int k = 0; k < 16; k += 2) {
                        float y0, y1;
                        tc::f2_unpack(tc::f2_fma(tc::f2_pack(x[i + k], x[i + k + 1]), sc2, mu2), y0, y1);
                        y0 = ex2(y0);
                        y1 = ex2(y1);
                        ls[k / 2 & 1] = tc::f2_add(ls[k / 2 & 1], tc::f2_pack(y0, y1));
                        pk[k / 2] = pack_half2(y0, y1);
                        const float2 y = X::pair(pk[k / 2]);
                        rest[k / 2] = pack_half2(y0 - y.x, y1 - y.y);
                    }
                    tmem_st8(tS + i / 2, pk);
                    tmem_st8(tS + 32 + i / 2, rest);
                }
                float l0, l1;
                tc::f2_unpack(tc::f2_add(ls[0], ls[1]), l0, l1);
                l += l0 + l1;
                if (v_odd & 0x01010101u)
                    rows_fix_weights(tS, *reinterpret_cast<const unsigned long long *>(sm.vbig[j & 3]) &
                                             ((unsigned long long)rows_bytes(v1, 1) << 32 | rows_bytes(v0, 1)));
                if (moved && st > 1) {      // O holds the stages before
                    ok = rows_wait(bar(ROWS_PVDONE + e), ((j - 2) >> 1) & 1, abort_p);
                    if (!__all_sync(0xffffffffu, ok)) break;
                    tc::tc_fence_after();
                    rows_scale<D>(tO, al);
                }
                tc::tmem_wait_st();
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) {      // (the warp's others wait for the next S)
                    tc::mbar_arrive(bar(ROWS_PREADY + e));
                    if ((warp & 3) == 0) {      // O (+)= P V
                        ok = rows_wait(bar(ROWS_PREADY + e), (j >> 1) & 1, abort_p);
                        if (ok) {
                            tc::tc_fence_after();
                            const uint64_t vd = pinned(tc::sw128_desc(smem_u32(sm.v[j % S::kStages]), S::kKHalf));
#pragma unroll
                            for (int kk = 0; kk < 2 * kRowsKeys / 16; kk++)
                                tc::umma_ts(tmem + kRowsColO + 128 * e, tmem + kRowsColS + 128 * e + 8 * kk,
                                            vd + kk % (kRowsKeys / 16) * (2048 >> 4), id_o, st > 1 || kk > 0);
                            tc::umma_commit(bar(ROWS_PVDONE + e));
                            tc::umma_commit(bar(ROWS_FREE + j % S::kStages));
                        }
                        if (ok && st + 2 < r.n_st) {
                            ok = rows_wait(bar(ROWS_PVDONE + e), (j >> 1) & 1, abort_p);
                            if (ok) issue_s(j + 2);
                        }
                    }
                }
            }
            // the two halves of the stages together: half of the dimensions each
            sm.ml[e][row] = make_float2(m, l);
            sm.nan[e][row] = nan;
            asm volatile("bar.sync 1, 256;\n" ::: "memory");
            const int first = J & 1;      // (the half that has the item's first stage)
            if (r.n_st > 0) ok = ok && rows_wait(bar(ROWS_PVDONE + ((J + r.n_st - 1) & 1)), ((J + r.n_st - 1) >> 1) & 1, abort_p);
            if (r.n_st > 1) ok = ok && rows_wait(bar(ROWS_PVDONE + ((J + r.n_st) & 1)), ((J + r.n_st - 2) >> 1) & 1, abort_p);
            if (!__all_sync(0xffffffffu, ok)) sm.abort = 1;      // (set, or about to be: all eight warps take the same way)
            asm volatile("bar.sync 1, 256;\n" ::: "memory");
            if (!*abort_p) {
                tc::tc_fence_after();
                const float2 x0 = sm.ml[first][row], x1 = sm.ml[first ^ 1][row];
                const float M = fmaxf(x0.x, x1.x), mu = M == kNegInf ? 0.f : M;
                float f0 = ex2((x0.x - mu) * p.scale_log2), f1 = ex2((x1.x - mu) * p.scale_log2);
                const float L = fmaf(x0.y, f0, x1.y * f1), inv = L == 0.f ? 0.f : __fdividef(1.f, L);      // (a NaN goes on)
                f0 *= inv;
                f1 *= inv;
                nan = sm.nan[0][row] | sm.nan[1][row];
                // rows through the K tiles (every product has been taken), so that a
                // warp writes whole rows
                constexpr int kRow = D * 4 + 16;
                static_assert(kRowsTile * kRow <= (int)sizeof(sm.k), "room for the output");
                const unsigned to = smem_u32(sm.k) + row * kRow;
                const unsigned t0 = tmem + kRowsColO + 128 * first + lane_off, t1 = tmem + kRowsColO + 128 * (first ^ 1) + lane_off;
#pragma unroll 1
                for (int c = e * (D / 2); c < (e + 1) * (D / 2); c += 32) {
                    float y[32];
#pragma unroll
                    for (int k = 0; k < 32; k++) y[k] = 0.f;
                    unsigned o[32];
                    if (r.n_st > 0) {
                        tc::tmem_ld32(t0 + c, o);
                        tc::tmem_wait_ld();
#pragma unroll
                        for (int k = 0; k < 32; k++) y[k] = __uint_as_float(o[k]) * f0;
                    }
                    if (r.n_st > 1) {
                        tc::tmem_ld32(t1 + c, o);
                        tc::tmem_wait_ld();
#pragma unroll
                        for (int k = 0; k < 32; k++) y[k] = fmaf(__uint_as_float(o[k]), f1, y[k]);
                    }
                    if (nan >> (c / GROUP) & 1) {
#pragma unroll
                        for (int k = 0; k < 32; k++) y[k] = __int_as_float(0x7fffffff);
                    }
                    const unsigned *z = reinterpret_cast<const unsigned *>(y);
#pragma unroll
                    for (int k = 0; k < 32; k += 8) {
                        sts128(to + 4 * (c + k), z[k], z[k + 2], z[k + 4], z[k + 6]);
                        sts128(to + 4 * (c + k) + 16, z[k + 1], z[k + 3], z[k + 5], z[k + 7]);
                    }
                }
                if (have && e == 0) __stcg(p.part_lse + rows_slot(a, sm.s, r, r.v0 + row), L == 0.f ? kNegInf : fmaf(M, p.scale_log2, lg2(L)));
                asm volatile("bar.sync 1, 256;\n" ::: "memory");
                constexpr int kL = D / 4, kR = 32 / kL;      // lanes of a row, rows at a time
#pragma unroll 4
                for (int k = warp * kR + lane / kL; k < kRowsTile && r.v0 + k <= r.vlast; k += 8 * kR) {
                    const uint4 x = lds128(smem_u32(sm.k) + k * kRow + lane % kL * 16);
                    __stcg(reinterpret_cast<uint4 *>(p.part_o + rows_slot(a, sm.s, r, r.v0 + k) * D) + lane % kL, x);
                }
            }
            __syncwarp();
            J += r.n_st;      // (before the barrier: behind it r may become another item)
            q_items += r.n_st > 0;
            tc::tc_fence_before();
            __syncthreads();
            tc::tc_fence_after();
            item = sm.s.next[turn];
        }
    } else {
        // ------------------------------------------------------------ unpack
        const int u = tid - 256;
        X next;           // a stage on its way
        int blk;          // the block of the one behind it
        auto begin = [&](const RowsItem &r) {
            const int *table = p.block_tables + (size_t)r.b * p.max_blocks;
            next.load(p, a.pool, X::codes_at(u, r.hk), X::pairs_at(u, r.hk), u, r.page0, r.end_page, r.n,
                      X::id(table, u, r.page0, r.end_page));
            blk = X::id(table, u, r.page0 + 4, r.end_page);
        };
        begin(sm.r[0]);
        for (int item = blockIdx.x, turn = 0, J = 0; item < n_items; turn ^= 1) {
            const RowsItem &r = sm.r[turn];
            bool ok = true;
            const int *table = p.block_tables + (size_t)r.b * p.max_blocks;
            const unsigned codes = X::codes_at(u, r.hk), pairs = X::pairs_at(u, r.hk);
#pragma unroll 1
            for (int st = 0; st < r.n_st; st++) {
                const int j = J + st, at = j % S::kStages, page = r.page0 + 4 * (st + 1);
                X x = next;      // (asked for a stage ago)
                next.load(p, a.pool, codes, pairs, u, page, r.end_page, r.n, blk);
                blk = X::id(table, u, page + 4, r.end_page);
                if (j >= S::kStages) ok = rows_wait(bar(ROWS_FREE + at), (j / S::kStages - 1) & 1, abort_p);
                if (!__all_sync(0xffffffffu, ok)) break;
                if (X::has_k(u)) x.unpack_k(sm, at, j & 3, u);
                if (X::has_v(u)) x.unpack_v(sm, at, j & 3, u);
                tc::fence_async_smem();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(bar(ROWS_FULL + at));
            }
            // the next item, and its first stage, beside the end of this one
            if (u == 0) {
                const int to = *abort_p ? n_items : (int)(gridDim.x + atomicAdd(&p.ctrl[CTRL_Q4_ROWS], 1u));
                sm.s.next[turn] = to;
                if (to < n_items) sm.r[turn ^ 1] = rows_item(p, sm.s, to, split);
            }
            asm volatile("bar.sync 2, 256;\n" ::: "memory");
            if (sm.s.next[turn] < n_items) begin(sm.r[turn ^ 1]);
            __syncwarp();
            J += r.n_st;      // (before the barrier: behind it r may become another item)
            tc::tc_fence_before();
            __syncthreads();
            tc::tc_fence_after();
            item = sm.s.next[turn];
        }
    }
    // after a wait that gave up: the MMAs in flight, of the two threads that issue them
    if (*abort_p && lane == 0 && (warp == 0 || warp == 4)) tc::umma_commit(bar(ROWS_FIN));
    if (warp == 8) {
        if (lane == 0 && *abort_p) {
            atomicOr(&p.ctrl[CTRL_FLAGS], RELAY_FLAG_WAIT_TIMEOUT);
            tc::mbar_drain(bar(ROWS_FIN), 0);
        }
        __syncwarp();
        tc::tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "n"(kRowsTmem) : "memory");
    }
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
}

// The prompt's partials beside it: the system items of the fp16 path (row
// teams, the prompt read once per batch), in a grid of their own that lets the
// context kernel start at once.
template <int D, int KGF>
__global__ void __launch_bounds__(kThreads, 1) prompt_kernel(const __grid_constant__ Params p)
{
    extern __shared__ __align__(128) unsigned char smem_raw[];
    Smem<D> &s = *reinterpret_cast<Smem<D> *>(smem_raw);
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    constexpr int PER = (kMaxB + kThreads - 1) / kThreads;
    int ql[PER];
#pragma unroll
    for (int k = 0; k < PER; k++) {
        const int b = threadIdx.x * PER + k;
        ql[k] = 0;
        if (b < p.B) {
            // a bad length fails the whole call (the context kernel reports it)
            ql[k] = p.q_lens ? p.q_lens[b] : p.Lq;
            if (ql[k] < 0 || ql[k] > p.Lq) ql[k] = 0;
        }
    }
    block_scan<D, PER>(ql, s.qo, p.B, s);
    const int Mtot = s.qo[p.B];
    if (Mtot > p.max_q_total) return;
    const int n_sys = p.Hkv * ((Mtot * p.G + kTileM - 1) / kTileM) * p.seg_R[0];
    const int team = team_of();
    const bool leader = (threadIdx.x % kRowThreads) == 0;
    for (int item = blockIdx.x + team * gridDim.x; item < n_sys;) {
        sys_item<D, KGF>(p, s, item, Mtot);
        if (leader) s.item[team] = (int)(kTeams * gridDim.x + atomicAdd(&p.ctrl[CTRL_ROW_ITEMS], 1u));
        team_sync();
        item = s.item[team];
        team_sync();
    }
}

// The fusion: WPR warps per (row, head) combine the prompt's ranges and the
// context's partials by their log-sum-exps, as merge_kernel of the fp16 path
// does.  With few rows it is one memory round trip after another, so four
// warps share a row's parts; with many rows one warp a row moves the bytes.
// About 5 us of a decode step, 27 us for 494 rows of 40 heads.
template <int D, int WPR, int CH>
__global__ void __launch_bounds__(256, CH > 8 ? 2 : 3) merge_kernel(const __grid_constant__ Args a)
{
    constexpr int V = D / 32, kRows = 8 / WPR;      // CH: partial rows in flight per warp
    constexpr float kLn2 = 0.69314718055994531f;
    __shared__ int qo[kMaxB + 1];
    __shared__ float sm_m[8], sm_w[8];
    __shared__ float sm_acc[WPR > 1 ? 8 : 1][D];
    const Params &p = a.p;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = warp % WPR, d0 = lane * V;
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        p.ctrl[CTRL_ROW_ITEMS] = 0u;
        p.ctrl[CTRL_DEC_ITEMS] = 0u;
        p.ctrl[CTRL_Q4_ROWS] = 0u;
    }
    const Sched sc = sched_at(p.sched, p.B);
    const int w = blockIdx.x * kRows + warp / WPR, r = w / p.H, h = w - r * p.H;
    int b = 0, i = 0, ql = p.Lq;
    bool live = true;
    if (p.q_lens) {
        for (int k = threadIdx.x; k <= p.B; k += 256) qo[k] = sc.qo[k];
        __syncthreads();
        live = p.sched[0] >= 0 && r < qo[p.B];
        if (live) {
            b = find_owner(qo, p.B, r);
            i = r - qo[b];
            ql = qo[b + 1] - qo[b];
        }
    } else {
        b = r / p.Lq;
        i = r - b * p.Lq;
        live = b < p.B;
        if (!live) b = 0;
    }
    const int bad = __ldcg(p.sched), Q = __ldcg(p.sched + 1), n = __ldg(p.ctx_lens + b), seq = __ldcg(sc.seq + b);
    const long long pre = __ldcg(sc.pre + b);
    live = live && bad >= 0;
    float M = kNegInf, W = 0.f, acc[V];
#pragma unroll
    for (int k = 0; k < V; k++) acc[k] = 0.f;
    if (live) {
        const Cols c = cols_of(ql, p.G);
        const int hk = h / p.G, v = i * p.G + h - hk * p.G, tile = v / (8 * c.nt), col = v - tile * 8 * c.nt;
        const int pages = (n + kBlock - 1) / kBlock, at = hk * c.tiles + tile;
        const long long f = pre + (long long)at * pages;
        long long c0, c1;      // its chunks
        if (f + pages <= 0xffffffffll) {
            c0 = (unsigned)f / (unsigned)Q;
            c1 = (unsigned)(f + pages - 1) / (unsigned)Q;
        } else {
            c0 = f / Q;
            c1 = (f + pages - 1) / Q;
        }
        const int n_sys = has_sys(p.mode) ? p.R_sys : 0;
        int n_parts = n_sys + (pages > 0 ? (int)(c1 - c0) + 1 : 0);
        const size_t sys0 = sys_slot(p, 0, r, h), sys_st = (size_t)p.max_q_total * p.H;
        size_t ctx0 = (size_t)a.part0 + (size_t)(c0 + seq + at) * a.nc + col, ctx_st = a.nc;
        if (c.cols > a.rows_max) {
            const int split = __ldcg(p.sched + 2);
            n_parts = n_sys + (pages + split - 1) / split;
            ctx0 = (size_t)a.rows0 + (size_t)r * p.H + h;
            ctx_st = sys_st;
        }
        auto slot = [&](int j) { return j < n_sys ? sys0 + j * sys_st : ctx0 + (size_t)(j - n_sys) * ctx_st; };
        // this warp's parts: part, part + WPR, ...
        const int mine = (n_parts - part + WPR - 1) / WPR;
        for (int j0 = 0; j0 < mine; j0 += 32) {
            const int cnt = min(32, mine - j0);
            const float lk = lane < cnt ? __ldcg(p.part_lse + slot((j0 + lane) * WPR + part)) : kNegInf;
            float x[CH][V];
            auto load = [&](int k0) {
#pragma unroll
                for (int k = 0; k < CH; k++) {
                    if (k0 + k < cnt) {
                        const float *src = p.part_o + slot((j0 + k0 + k) * WPR + part) * D + d0;
                        if constexpr (V == 4) {
                            const float4 t = __ldcg(reinterpret_cast<const float4 *>(src));
                            x[k][0] = t.x; x[k][1] = t.y; x[k][2] = t.z; x[k][3] = t.w;
                        } else {
                            const float2 t = __ldcg(reinterpret_cast<const float2 *>(src));
                            x[k][0] = t.x; x[k][1] = t.y;
                        }
                    }
                }
            };
            load(0);      // with the log-sum-exps: one round trip
            float mk = lk;
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) mk = fmaxf(mk, __shfl_xor_sync(0xffffffffu, mk, off));
            const float Mn = fmaxf(M, mk), mu = Mn == kNegInf ? 0.f : Mn, al = ex2(M - mu), wk = ex2(lk - mu);
            M = Mn;
            W *= al;
#pragma unroll
            for (int k = 0; k < V; k++) acc[k] *= al;
            for (int k0 = 0; k0 < cnt; k0 += CH) {
                if (k0 > 0) load(k0);
#pragma unroll
                for (int k = 0; k < CH; k++) {
                    const float wt = __shfl_sync(0xffffffffu, wk, (k0 + k) & 31);
                    if (k0 + k < cnt) {
                        W += wt;
#pragma unroll
                        for (int e = 0; e < V; e++) acc[e] += wt * x[k][e];
                    }
                }
            }
        }
    }
    if constexpr (WPR > 1) {
        if (lane == 0) {
            sm_m[warp] = M;
            sm_w[warp] = W;
        }
#pragma unroll
        for (int k = 0; k < V; k++) sm_acc[warp][d0 + k] = acc[k];
        __syncthreads();
        if (part > 0) return;
        float top = M;
#pragma unroll
        for (int k = 1; k < WPR; k++) top = fmaxf(top, sm_m[warp + k]);
        const float mu = top == kNegInf ? 0.f : top, al = ex2(M - mu);
        W *= al;
#pragma unroll
        for (int e = 0; e < V; e++) acc[e] *= al;
#pragma unroll
        for (int k = 1; k < WPR; k++) {
            const float ak = ex2(sm_m[warp + k] - mu);
            W += sm_w[warp + k] * ak;
#pragma unroll
            for (int e = 0; e < V; e++) acc[e] += sm_acc[warp + k][d0 + e] * ak;
        }
        M = top;
    }
    if (!live) return;
    const float inv = W == 0.f ? 0.f : 1.f / W;
    const float lse = W == 0.f ? kNegInf : (M + lg2(W)) * kLn2;
    const size_t orow = ((size_t)b * p.Lq + i) * p.H + h;
    if (p.mode == MODE_FUSED) {
        __half *dst = p.out + orow * D + d0;
        if constexpr (V == 4)
            *reinterpret_cast<uint2 *>(dst) =
                make_uint2(pack_half2(acc[0] * inv, acc[1] * inv), pack_half2(acc[2] * inv, acc[3] * inv));
        else
            *reinterpret_cast<unsigned *>(dst) = pack_half2(acc[0] * inv, acc[1] * inv);
        if (p.lse_out && lane == 0) p.lse_out[orow] = lse;
    } else {
        float *dst = p.o_f32 + orow * D + d0;
#pragma unroll
        for (int k = 0; k < V; k++) dst[k] = acc[k] * inv;
        if (lane == 0) p.lse_f32[orow] = lse;
    }
}

}  // namespace q4
}  // namespace relay
