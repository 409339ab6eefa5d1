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
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "relay_kernels.cuh"
#include "step_kernels.cuh"

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
// spread over 32 elements the kernel is [APPEND].
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
// twice; then the (s, z) pairs of K and of V.
template <int D, int GROUP>
struct PageQ {
    static constexpr int kRow = D / 2;               // bytes of a row of codes
    static constexpr int kCodes = kBlock * kRow;
    static constexpr int NG = D / GROUP;             // groups of a row
    static constexpr int kSz = kBlock * NG * 4;      // bytes of the (s, z) pairs of K or V
    static constexpr int kStage = 2 * kCodes + 2 * kSz;
    static constexpr int kRing = kRingBytes / kWarps;
    static constexpr int kStages = kRing / kStage < 8 ? kRing / kStage : 8;
};

template <int D>
__device__ __forceinline__ int chunk_off(int row, int ch)
{
    constexpr int kPerLine = 256 / D;                // rows of a 128-byte line
    const int line = row / kPerLine, pos = (row % kPerLine) * (D / 32) + ch;
    return line * 128 + ((pos ^ ((line & 3) << 1)) << 4);
}
template <int D>
__device__ __forceinline__ int byte_off(int row, int byte) { return chunk_off<D>(row, byte >> 4) + (byte & 15); }

// ----------------------------------------------------------------------------- attention: items
// A warp's item: the keys of one KV head in a range of one request's pages
// against up to 8 * NT columns.  Column v is query row v / G with head
// hk * G + v % G (one row: the heads of the group).
template <int D, int NT>
struct Item {
    int b, hk, v0, nv;      // first column and columns of the item
    int ql, row0;           // query rows of the request; its first compact row
    int split, p0, np;      // partial index; first page and pages
    int n_ctx;
    unsigned qb[NT][D / 16][2];
};

// Row state: O^T in units of (code * 2^-24 or 2^-20) * 2^e, softmax statistics
// of the lane's columns 8 nt + 2t, + 1.
template <int D, int GROUP, int NT>
struct State {
    float o[NT][D / 16][4];
    float c[NT][D / GROUP][4];      // the same for a code of 8 in every dimension
    float z[NT][D / GROUP][2];      // sum of p (z + 8 s) over the lane's keys
    float m[NT][2], l[NT][2];
    int e;                          // scale_exp of the largest V scale so far
};

constexpr unsigned kLoCodes = 0x000f000fu, kHiCodes = 0x00f000f0u;

// Biased exponent of a scale, plus one; 0 for an infinite or NaN scale, which
// must not move the others' power (it may belong to a key no row sees).
__device__ __forceinline__ int scale_exp(__half2 sz) { return ((__half_as_ushort(__low2half(sz)) >> 10) + 1) & 31; }
// 2^(15 - e): brings a scale of that exponent at most to below 1
__device__ __forceinline__ float scale_down(int e) { return __int_as_float((15 - e + 127) << 23); }

template <int D, int GROUP, int NT>
__device__ __forceinline__ void load_q(const Params &p, Item<D, NT> &it)
{
    constexpr int WPG = GROUP / 32;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int nt = 0; nt < NT; nt++) {
        const int v = it.v0 + 8 * nt + g;
        const bool has = 8 * nt + g < it.nv;
        const int i = has ? v / p.G : 0, c = has ? v % p.G : 0;
        const __half *q = p.q + (((size_t)it.b * p.Lq + i) * p.H + it.hk * p.G + c) * D;
#pragma unroll
        for (int w = 0; w < D / 32; w++) {
            // dimensions of word w of the lane: the K words are read the same way
            const int d0 = (w / WPG) * GROUP + t * (GROUP / 4) + 8 * (w % WPG);
            uint4 x = make_uint4(0u, 0u, 0u, 0u);
            if (has) x = *reinterpret_cast<const uint4 *>(q + d0);
            it.qb[nt][2 * w][0] = __byte_perm(x.x, x.z, 0x5410);          // dimensions 0, 4
            it.qb[nt][2 * w][1] = __byte_perm(x.y, x.w, 0x5410);          // 2, 6
            it.qb[nt][2 * w + 1][0] = __byte_perm(x.x, x.z, 0x7632);      // 1, 5
            it.qb[nt][2 * w + 1][1] = __byte_perm(x.y, x.w, 0x7632);      // 3, 7
        }
    }
}

// Sums of q over each group, for the lane's two columns of every tile.
template <int D, int GROUP, int NT>
__device__ __forceinline__ void q_sums(const Item<D, NT> &it, float (&qs)[NT][D / GROUP][2])
{
    constexpr int WPG = GROUP / 32;
    const int t = threadIdx.x & 3;
#pragma unroll
    for (int nt = 0; nt < NT; nt++)
#pragma unroll
        for (int gi = 0; gi < D / GROUP; gi++) {
            float x = 0.f;
#pragma unroll
            for (int w = gi * 2 * WPG; w < (gi + 1) * 2 * WPG; w++)
#pragma unroll
                for (int r = 0; r < 2; r++) {
                    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&it.qb[nt][w][r]));
                    x += f.x + f.y;
                }
            x += __shfl_xor_sync(0xffffffffu, x, 1);
            x += __shfl_xor_sync(0xffffffffu, x, 2);
            qs[nt][gi][0] = __shfl_sync(0xffffffffu, x, 8 * t);
            qs[nt][gi][1] = __shfl_sync(0xffffffffu, x, 8 * t + 4);
        }
}

// One lane's share of staging one page: `rows` valid tokens.  The codes are
// copied whole (what lies behind the last token is a number either way); the
// pairs of further tokens read as zero, so that nothing of them is left.
template <int D, int GROUP>
__device__ __forceinline__ void load_page(const Params &p, const Pool &pool, unsigned char *st, int blk, int hk, int rows,
                                          int lane)
{
    using P = PageQ<D, GROUP>;
    const bool ok = blk >= 0 && blk < p.num_blocks;
    if (!ok && lane == 0) atomicOr(&p.ctrl[CTRL_FLAGS], FLAG_BAD_BLOCK);
    const size_t page = (size_t)(ok ? blk : 0) * p.Hkv + hk;
    const unsigned char *kc = pool.k + page * P::kCodes, *vc = pool.v + page * P::kCodes;
#pragma unroll
    for (int k = 0; k < P::kCodes / 512; k++) {
        const int c = lane + 32 * k;
        const int dst = chunk_off<D>(c / (D / 32), c % (D / 32));
        cp_async16(st + dst, kc + 16 * c, ok);
        cp_async16(st + P::kCodes + dst, vc + 16 * c, ok);
    }
    constexpr int kChunks = P::kSz / 16;      // of K, then of V
#pragma unroll
    for (int c0 = 0; c0 < 2 * kChunks; c0 += 32) {
        const int c = c0 + lane;
        if (c < 2 * kChunks) {
            const int cc = c % kChunks;
            const unsigned char *src =
                reinterpret_cast<const unsigned char *>(c < kChunks ? pool.ksz : pool.vsz) + page * P::kSz + 16 * cc;
            const int n = ok ? min(16, max(0, rows * P::NG * 4 - 16 * cc)) : 0;
            asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;\n" ::"r"(
                             smem_u32(st + 2 * P::kCodes + 16 * c)),
                         "l"(src), "r"(n));
        }
    }
}

// One warp, one page.  end[nt][e]: keys of this page that column e sees.
template <int D, int GROUP, int NT, bool MASK>
__device__ __forceinline__ void page_step(const unsigned char *st, const Item<D, NT> &it, const float (&qs)[NT][D / GROUP][2],
                                          State<D, GROUP, NT> &s, const int (&end)[NT][2], float scale_log2)
{
    using P = PageQ<D, GROUP>;
    constexpr int NG = P::NG, WPG = GROUP / 32;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const float2 zero2 = make_float2(0.f, 0.f);

    // S^T = K q, a group at a time
    float sc[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; nt++)
#pragma unroll
        for (int e = 0; e < 4; e++) sc[nt][e] = 0.f;
    const __half2 *ksz = reinterpret_cast<const __half2 *>(st + 2 * P::kCodes);
#pragma unroll
    for (int gi = 0; gi < NG; gi++) {
        unsigned w0[WPG], w1[WPG];
        const int byte = gi * (GROUP / 2) + t * (GROUP / 8);
        if constexpr (WPG == 4) {
            const uint4 x = *reinterpret_cast<const uint4 *>(st + byte_off<D>(g, byte));
            const uint4 y = *reinterpret_cast<const uint4 *>(st + byte_off<D>(g + 8, byte));
            w0[0] = x.x; w0[1] = x.y; w0[2] = x.z; w0[3] = x.w;
            w1[0] = y.x; w1[1] = y.y; w1[2] = y.z; w1[3] = y.w;
        } else if constexpr (WPG == 2) {
            const uint2 x = *reinterpret_cast<const uint2 *>(st + byte_off<D>(g, byte));
            const uint2 y = *reinterpret_cast<const uint2 *>(st + byte_off<D>(g + 8, byte));
            w0[0] = x.x; w0[1] = x.y;
            w1[0] = y.x; w1[1] = y.y;
        } else {
            w0[0] = *reinterpret_cast<const unsigned *>(st + byte_off<D>(g, byte));
            w1[0] = *reinterpret_cast<const unsigned *>(st + byte_off<D>(g + 8, byte));
        }
        float lo[NT][4], hi[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; nt++)
#pragma unroll
            for (int e = 0; e < 4; e++) lo[nt][e] = hi[nt][e] = 0.f;
#pragma unroll
        for (int j = 0; j < WPG; j++) {
            const unsigned x0 = w0[j] >> 8, x1 = w1[j] >> 8;
            const unsigned a0[4] = {w0[j] & kLoCodes, w1[j] & kLoCodes, x0 & kLoCodes, x1 & kLoCodes};
            const unsigned a1[4] = {w0[j] & kHiCodes, w1[j] & kHiCodes, x0 & kHiCodes, x1 & kHiCodes};
            const int w = 2 * (gi * WPG + j);
#pragma unroll
            for (int nt = 0; nt < NT; nt++) {
                mma16816(lo[nt], a0, it.qb[nt][w][0], it.qb[nt][w][1]);
                mma16816(hi[nt], a1, it.qb[nt][w + 1][0], it.qb[nt][w + 1][1]);
            }
        }
        const float2 k0 = __half22float2(ksz[g * NG + gi]), k1 = __half22float2(ksz[(g + 8) * NG + gi]);
#pragma unroll
        for (int nt = 0; nt < NT; nt++)
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const float2 k = e < 2 ? k0 : k1;
                sc[nt][e] += k.x * (lo[nt][e] * 0x1p24f + hi[nt][e] * 0x1p20f) + k.y * qs[nt][gi][e & 1];
            }
    }
    // online softmax per column (keys over the lanes' g)
    bool moved = false;
    float mu[NT][2], mn[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; nt++)
#pragma unroll
        for (int e = 0; e < 2; e++) {
            float x0 = sc[nt][e] * scale_log2, x1 = sc[nt][2 + e] * scale_log2;
            if (MASK) {
                x0 = g < end[nt][e] ? x0 : kNegInf;
                x1 = g + 8 < end[nt][e] ? x1 : kNegInf;
            }
            sc[nt][e] = x0;
            sc[nt][2 + e] = x1;
            float mx = fmaxf(x0, x1);
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
            mn[nt][e] = fmaxf(s.m[nt][e], mx);
            mu[nt][e] = mn[nt][e] == kNegInf ? 0.f : mn[nt][e];
            moved = moved || mn[nt][e] != s.m[nt][e];
        }
    if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int nt = 0; nt < NT; nt++)
#pragma unroll
            for (int e = 0; e < 2; e++) {
                const float al = ex2(s.m[nt][e] - mu[nt][e]);
                s.m[nt][e] = mn[nt][e];
                s.l[nt][e] *= al;
#pragma unroll
                for (int gi = 0; gi < NG; gi++) {
                    s.z[nt][gi][e] *= al;
                    s.c[nt][gi][e] *= al;
                    s.c[nt][gi][2 + e] *= al;
                }
#pragma unroll
                for (int d = 0; d < D / 16; d++) {
                    s.o[nt][d][e] *= al;
                    s.o[nt][d][2 + e] *= al;
                }
            }
    }
#pragma unroll
    for (int nt = 0; nt < NT; nt++)
#pragma unroll
        for (int e = 0; e < 4; e++) {
            sc[nt][e] = ex2(sc[nt][e] - mu[nt][e & 1]);
            s.l[nt][e & 1] += sc[nt][e];
        }
    // the V scales' common power of two: p s / 2^e fills fp16 from the top
    const __half2 *vsz = ksz + kBlock * NG;
    float2 v0[NG], v1[NG];
    int em = 0;
#pragma unroll
    for (int gi = 0; gi < NG; gi++) {
        const __half2 h0 = vsz[g * NG + gi], h1 = vsz[(g + 8) * NG + gi];
        em = max(em, max(scale_exp(h0), scale_exp(h1)));
        v0[gi] = __half22float2(h0);
        v1[gi] = __half22float2(h1);
    }
    em = max(s.e, (int)__reduce_max_sync(0xffffffffu, (unsigned)em));
    if (em != s.e) {      // warp-uniform
        const float al = __int_as_float((s.e - em + 127) << 23);
        s.e = em;
#pragma unroll
        for (int nt = 0; nt < NT; nt++)
#pragma unroll
            for (int e = 0; e < 4; e++) {
#pragma unroll
                for (int d = 0; d < D / 16; d++) s.o[nt][d][e] *= al;
#pragma unroll
                for (int gi = 0; gi < NG; gi++) s.c[nt][gi][e] *= al;
            }
    }
    const float down = scale_down(em);
    unsigned pb[NT][NG][2];
#pragma unroll
    for (int nt = 0; nt < NT; nt++)
#pragma unroll
        for (int gi = 0; gi < NG; gi++) {
            float w[4];
#pragma unroll
            for (int e = 0; e < 4; e++) {
                float2 v = e < 2 ? v0[gi] : v1[gi];
                // a NaN behind the mask must not meet its zero weight
                if (MASK) v = g + (e < 2 ? 0 : 8) < end[nt][e & 1] ? v : zero2;
                w[e] = sc[nt][e] * (v.x * down);
                s.z[nt][gi][e & 1] += sc[nt][e] * fmaf(8.f, v.x, v.y);
            }
            pb[nt][gi][0] = movmatrix_t(pack_half2(w[0], w[1]));
            pb[nt][gi][1] = movmatrix_t(pack_half2(w[2], w[3]));
            constexpr unsigned kEight = 0x00080008u;
            const unsigned a[4] = {kEight, kEight, kEight, kEight};
            mma16816(s.c[nt][gi], a, pb[nt][gi][0], pb[nt][gi][1]);
        }
    // O^T += V^T P.  A lane's operand rows are dimensions, its columns keys 2t,
    // 2t + 1, 2t + 8, 2t + 9: two keys' words are interleaved by halves, and
    // a tile is one code position of the words.  Rows of a tile share their
    // group, so with GROUP = 32 (four words) the two halves of the rows take
    // the same word at positions 8 bits apart.
    const unsigned char *vc = st + P::kCodes;
    constexpr int kHalf = GROUP == 32 ? 32 : 64;      // dimensions of a set of tiles
#pragma unroll
    for (int h = 0; h < D / kHalf; h++) {
        const int byte = h * (kHalf / 2) + 4 * (GROUP == 32 ? (g & 3) : g);
        unsigned w[4];
#pragma unroll
        for (int k = 0; k < 4; k++)
            w[k] = *reinterpret_cast<const unsigned *>(vc + byte_off<D>(2 * t + (k & 1) + 8 * (k >> 1), byte));
        unsigned x0 = __byte_perm(w[0], w[1], 0x5410), y0 = __byte_perm(w[0], w[1], 0x7632);
        unsigned x1 = __byte_perm(w[2], w[3], 0x5410), y1 = __byte_perm(w[2], w[3], 0x7632);
        const int gi = h * kHalf / GROUP;
        if constexpr (GROUP == 32) {
            const int sh = (g >> 2) * 8;
            x0 >>= sh; y0 >>= sh; x1 >>= sh; y1 >>= sh;
            const unsigned a0[4] = {x0 & kLoCodes, y0 & kLoCodes, x1 & kLoCodes, y1 & kLoCodes};
            const unsigned a1[4] = {x0 & kHiCodes, y0 & kHiCodes, x1 & kHiCodes, y1 & kHiCodes};
#pragma unroll
            for (int nt = 0; nt < NT; nt++) {
                mma16816(s.o[nt][2 * h], a0, pb[nt][gi][0], pb[nt][gi][1]);
                mma16816(s.o[nt][2 * h + 1], a1, pb[nt][gi][0], pb[nt][gi][1]);
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
                    mma16816(s.o[nt][4 * h + 2 * r], a0, pb[nt][gi][0], pb[nt][gi][1]);
                    mma16816(s.o[nt][4 * h + 2 * r + 1], a1, pb[nt][gi][0], pb[nt][gi][1]);
                }
            }
        }
    }
}

// Writes the item's partials: normalised output and log2-sum-exp per column.
template <int D, int GROUP, int NT>
__device__ __forceinline__ void write_item(const Params &p, const Item<D, NT> &it, State<D, GROUP, NT> &s)
{
    constexpr int NG = D / GROUP;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const float up = __int_as_float((24 + s.e - 15 + 127) << 23);      // 2^24 / scale_down
#pragma unroll
    for (int nt = 0; nt < NT; nt++)
#pragma unroll
        for (int e = 0; e < 2; e++) {
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) {
                s.l[nt][e] += __shfl_xor_sync(0xffffffffu, s.l[nt][e], off);
#pragma unroll
                for (int gi = 0; gi < NG; gi++) s.z[nt][gi][e] += __shfl_xor_sync(0xffffffffu, s.z[nt][gi][e], off);
            }
            const int c = 8 * nt + 2 * t + e;
            if (c >= it.nv) continue;
            const int v = it.v0 + c, i = v / p.G, h = it.hk * p.G + v % p.G;
            const size_t pr = it.ql == 1 ? dec_slot(p, it.split, it.b, h) : mq_slot(p, it.split, it.row0 + i, h);
            const float L = s.l[nt][e], inv = L > 0.f ? 1.f / L : 0.f;
            const float f0 = up * inv, f1 = f0 * 0.0625f;
            float *po = p.part_o + pr * D;
            if constexpr (GROUP == 32) {
#pragma unroll
                for (int gi = 0; gi < NG; gi++)
#pragma unroll
                    for (int r = 0; r < 2; r++) {
                        const float z = s.z[nt][gi][e] * inv - s.c[nt][gi][e] * f0;
                        __stcg(reinterpret_cast<float2 *>(po + 32 * gi + 8 * (g & 3) + 2 * (g >> 2) + 4 * r),
                               make_float2(s.o[nt][2 * gi][2 * r + e] * f0 + z, s.o[nt][2 * gi + 1][2 * r + e] * f1 + z));
                    }
            } else {
#pragma unroll
                for (int hf = 0; hf < D / 64; hf++) {
                    const float z = s.z[nt][hf * 64 / GROUP][e] * inv - s.c[nt][hf * 64 / GROUP][e] * f0;
                    // tiles: code positions 0, 1, 4, 5 (rows g) and 2, 3, 6, 7 (rows g + 8)
#pragma unroll
                    for (int r = 0; r < 2; r++) {
                        const float(&a)[4] = s.o[nt][4 * hf + 2 * r], (&b)[4] = s.o[nt][4 * hf + 2 * r + 1];
                        __stcg(reinterpret_cast<float4 *>(po + 64 * hf + 8 * g + 4 * r),
                               make_float4(a[e] * f0 + z, b[e] * f1 + z, a[2 + e] * f0 + z, b[2 + e] * f1 + z));
                    }
                }
            }
            if (g == 0) __stcg(p.part_lse + pr, L > 0.f ? s.m[nt][e] + lg2(L) : kNegInf);
        }
}

// ----------------------------------------------------------------------------- attention: schedule
// Shared memory: that of the row items, and the item prefix of this queue.
template <int D>
struct SmemQ {
    Smem<D> row;
    int it[kMaxB + 1];      // items before request b
};

// Context work of request b with ql rows and n tokens: columns, tiles of
// columns, splits and keys per split.  One row: the pages of the context in
// ns nearly equal runs of at most tps pages; several rows: ranges of ri.split
// keys (the merge kernel reads both the same way).
struct Work {
    ReqInfo ri;
    int cols, nt, tiles;
};
__device__ __forceinline__ Work work_of(const Params &p, int n, int ql, int tps, int max_nt)
{
    Work w;
    w.ri = req_info(p, n, ql, tps);
    w.cols = ql * p.G;
    w.nt = w.cols > 8 && max_nt > 1 ? 2 : 1;
    w.tiles = (w.cols + 8 * w.nt - 1) / (8 * w.nt);
    return w;
}

template <int D>
__device__ void build_schedule_q4(const Params &p, SmemQ<D> &sq, int max_nt, int items_per_warp)
{
    constexpr int PER = (kMaxB + kThreads - 1) / kThreads;
    Smem<D> &s = sq.row;
    const int tid = threadIdx.x;
    int vq[PER], pages[PER], nn[PER], items[PER];
    unsigned flags = 0;
    if (tid == 0) s.bad = 0;
#pragma unroll
    for (int k = 0; k < PER; k++) {
        const int b = tid * PER + k;
        int ql = 0, n = 0;
        if (b < p.B) {
            ql = p.q_lens ? p.q_lens[b] : p.Lq;
            n = p.ctx_lens[b];
            s.segm[b] = ~0u;
            if (ql < 0 || ql > p.Lq) { flags |= FLAG_BAD_Q_LEN; ql = 0; }
            if (n < 0 || n > p.max_blocks * kBlock) { flags |= FLAG_BAD_CTX_LEN; ql = n = 0; }
            s.nctx[b] = n;
        }
        vq[k] = ql;
        nn[k] = n;
        pages[k] = ql == 1 ? p.HQ * ((n + kBlock - 1) / kBlock) : 0;
    }
    __syncthreads();
    if (flags) atomicOr(&s.bad, (int)flags);
    block_scan<D, PER>(vq, s.qo, p.B, s);
    block_scan<D, PER>(pages, s.dec, p.B, s);
    if (tid == 0) {
        const long long want = (long long)gridDim.x * kWarps * items_per_warp;
        s.tps = max(p.tps_min, min(p.tps_max, (int)((s.dec[p.B] + want - 1) / want)));
        if (s.qo[p.B] > p.max_q_total) s.bad |= FLAG_Q_TOTAL;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < PER; k++) {
        items[k] = 0;
        if (vq[k] > 0) {
            const Work w = work_of(p, nn[k], vq[k], s.tps, max_nt);
            items[k] = p.Hkv * w.tiles * w.ri.ns;
        }
    }
    block_scan<D, PER>(items, sq.it, p.B, s);
}

// ----------------------------------------------------------------------------- attention: one item
template <int D, int GROUP, int NT>
__device__ void run_item(const Params &p, const Pool &pool, SmemQ<D> &sq, int b, int local, const Work &w)
{
    using P = PageQ<D, GROUP>;
    constexpr int S = P::kStages;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, t = lane & 3;
    unsigned char *ring = sq.row.ring + warp * P::kRing;
    Item<D, NT> it;
    it.b = b;
    it.n_ctx = w.ri.n_ctx;
    it.ql = w.ri.ql;
    it.row0 = sq.row.qo[b];
    it.split = local % w.ri.ns;
    const int r = local / w.ri.ns, tile = r % w.tiles;
    it.hk = r / w.tiles;
    it.v0 = tile * 8 * NT;
    it.nv = min(8 * NT, w.cols - it.v0);
    // keys that column v sees: max(0, n - ql + 1 + i), and none past the split
    auto sees = [&](int v) { return max(0, min(it.n_ctx, it.n_ctx - it.ql + 1 + v / p.G)); };
    const int all = sees(it.v0), most = sees(it.v0 + it.nv - 1);      // first and last row of the item
    if (it.ql == 1) {
        it.p0 = (int)((long long)it.split * w.ri.pages / w.ri.ns);
        it.np = (int)((long long)(it.split + 1) * w.ri.pages / w.ri.ns) - it.p0;
    } else {
        it.p0 = it.split * (w.ri.split / kBlock);
        it.np = (min(most, (it.split + 1) * w.ri.split) + kBlock - 1) / kBlock - it.p0;
    }
    const int *table = p.block_tables + (size_t)b * p.max_blocks;
    int blk = 0, window = -32;      // lane j: block of page `window` + j
    int issued = 0;
    auto issue = [&]() {
        if (issued >= window + 32) {
            window = issued;
            blk = issued + lane < it.np ? table[it.p0 + issued + lane] : 0;
        }
        load_page<D, GROUP>(p, pool, ring + (issued % S) * P::kStage, __shfl_sync(0xffffffffu, blk, issued - window), it.hk,
                            min(kBlock, it.n_ctx - (it.p0 + issued) * kBlock), lane);
        issued++;
    };
    for (int k = 0; k < S - 1; k++) {
        if (issued < it.np) issue();
        cp_async_commit();
    }
    load_q<D, GROUP, NT>(p, it);
    float qs[NT][D / GROUP][2];
    q_sums<D, GROUP, NT>(it, qs);
    int see[NT][2];
    State<D, GROUP, NT> s;
    s.e = 0;
#pragma unroll
    for (int nt = 0; nt < NT; nt++)
#pragma unroll
        for (int e = 0; e < 2; e++) {
            see[nt][e] = sees(min(it.v0 + 8 * nt + 2 * t + e, it.v0 + it.nv - 1));
            s.m[nt][e] = kNegInf;
            s.l[nt][e] = 0.f;
#pragma unroll
            for (int gi = 0; gi < P::NG; gi++) s.z[nt][gi][e] = s.c[nt][gi][e] = s.c[nt][gi][2 + e] = 0.f;
#pragma unroll
            for (int d = 0; d < D / 16; d++) s.o[nt][d][e] = s.o[nt][d][2 + e] = 0.f;
        }
    for (int j = 0; j < it.np; j++) {
        cp_async_wait<S - 2>();
        __syncwarp();
        const int key0 = (it.p0 + j) * kBlock;
        int end[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; nt++)
#pragma unroll
            for (int e = 0; e < 2; e++) end[nt][e] = see[nt][e] - key0;
        const unsigned char *st = ring + (j % S) * P::kStage;
        if (key0 + kBlock <= all)
            page_step<D, GROUP, NT, false>(st, it, qs, s, end, p.scale_log2);
        else
            page_step<D, GROUP, NT, true>(st, it, qs, s, end, p.scale_log2);
        __syncwarp();
        if (issued < it.np) issue();
        cp_async_commit();
    }
    cp_async_wait<0>();
    __syncwarp();
    write_item<D, GROUP, NT>(p, it, s);
}

// ----------------------------------------------------------------------------- attention: kernel
// One CTA of 8 warps per SM, in the two phases of relay_kernel: row teams take
// the system items (the fp16 prompt, read once per batch), then every warp on
// its own takes items of the 4-bit contexts from one queue.  Partials and
// schedule are handed to merge_kernel exactly as relay_kernel does.
template <int D, int GROUP, int MAXNT>
__global__ void __launch_bounds__(kThreads, 1) q4_kernel(const __grid_constant__ Params p, const __grid_constant__ Pool pool)
{
    extern __shared__ __align__(128) unsigned char smem_raw[];
    SmemQ<D> &sq = *reinterpret_cast<SmemQ<D> *>(smem_raw);
    Smem<D> &s = sq.row;
    build_schedule_q4<D>(p, sq, MAXNT, 2);
    if (blockIdx.x == 0) {
        for (int k = threadIdx.x; k <= p.B; k += kThreads) p.sched[1 + k] = s.qo[k];
        for (int k = threadIdx.x; k < p.B; k += kThreads) p.sched[2 + p.B + k] = s.nctx[k];
        if (threadIdx.x == 0) p.sched[0] = s.bad ? -1 : s.tps;
    }
    if (s.bad) {
        if (threadIdx.x == 0) atomicOr(&p.ctrl[CTRL_FLAGS], (unsigned)s.bad);
        return;
    }
    const int Mtot = s.qo[p.B];
    const int T = (Mtot * p.G + kTileM - 1) / kTileM;
    const int n_sys = has_sys(p.mode) && !p.skip_sys ? p.Hkv * T * p.seg_R[0] : 0;
    {
        const int team = team_of();
        const bool leader = (threadIdx.x % kRowThreads) == 0;
        for (int item = blockIdx.x + team * gridDim.x; item < n_sys;) {
            sys_item<D, 0>(p, s, item, Mtot);
            if (leader) s.item[team] = (int)(kTeams * gridDim.x + atomicAdd(&p.ctrl[CTRL_ROW_ITEMS], 1u));
            team_sync();
            item = s.item[team];
            team_sync();
        }
    }
    const int n_items = sq.it[p.B];
    const int lane = threadIdx.x & 31;
    for (;;) {
        int id = 0;
        if (lane == 0) id = (int)atomicAdd(&p.ctrl[CTRL_DEC_ITEMS], 1u);
        id = __shfl_sync(0xffffffffu, id, 0);
        if (id >= n_items) break;
        const int b = find_owner(sq.it, p.B, id);
        const Work w = work_of(p, s.nctx[b], s.qo[b + 1] - s.qo[b], s.tps, MAXNT);
        if (MAXNT > 1 && w.nt > 1) run_item<D, GROUP, MAXNT>(p, pool, sq, b, id - sq.it[b], w);
        else run_item<D, GROUP, 1>(p, pool, sq, b, id - sq.it[b], w);
    }
    __syncthreads();
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
}

}  // namespace q4
}  // namespace relay
