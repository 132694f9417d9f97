// The 4-bit pool's tile format and the device code that reads it into tensor
// core fragments.
//
// Blocks of 16 consecutive dims of a row share one E4M3 scale; a code is an
// E2M1 value (0, .5, 1, 1.5, 2, 3, 4, 6 and a sign).  code * scale has at
// most 6 significant bits and lies between 2^-10 and 2688, so it is exact in
// fp16: the products below are those of an fp16 pool holding these values.
//
// One chunk of one key/value head is a contiguous tile
//     K codes [c x D/2 B] | V codes [c x D/2 B] | K scales [c x D/16 B] | V scales [c x D/16 B]
// (9216 bytes at c = 64, D = 128) fetched by one bulk copy.  Inside it every
// array is laid out for m16n8k16 fragments, so that a lane's operands come
// with few wide shared-memory loads and no bank conflicts.  With lane
// (g, t) = (lane / 4, lane % 4), tokens taken 16 at a time:
//  * K (operand A of S = K q: rows tokens, columns dims).  Storage row
//    m = f4_row(token) is fragment row m.  In a row, dim 16 kk + 4t + j is
//    byte t * D/8 + 2 kk + j / 2, nibble j % 2: a lane's codes of all steps
//    kk are D/8 consecutive bytes, each byte a pair of adjacent columns (the
//    columns are permuted inside a step; the query fragments take the same
//    order).
//  * V (operand A of O^T += V^T p: rows dims, columns tokens).  Fragment
//    columns 2t, 2t + 1, 2t + 8, 2t + 9 are tokens t, t + 4, t + 8, t + 12 (the
//    order in which S^T's rows reach the operand p), so tokens x and x + 4 of
//    each 8 share bytes, low and high nibble: a byte converts to a fragment
//    register's pair.  Row = pair of tokens, D bytes; in it unit g holds dims
//    16 db + 2g of all db, then dims 16 db + 2g + 1: a lane's dims of both
//    tokens are D/8 consecutive bytes.  Unit g of a row sits at
//    f4_v_unit(row, g), which keeps the loads of four rows apart.
//  * K scales: row m, one byte per step kk.
//  * V scales: tokens x and x + 4 (and x + 8, x + 12) paired, [pair][db][2],
//    so that 16 bits convert to the pair of scales that a fragment register's
//    two tokens need.
#pragma once

#include "device.cuh"

namespace ca {
namespace dev {

template <int C, int D>
struct F4Tile {
    static constexpr int kCodes = C * D / 2;
    static constexpr int kScales = C * D / 16;
    static constexpr int kVCodes = kCodes;
    static constexpr int kKScales = 2 * kCodes;
    static constexpr int kVScales = 2 * kCodes + kScales;
    static constexpr int kBytes = 2 * (kCodes + kScales);
};

// Storage row of a token's keys inside its block of 16 (and back).
__host__ __device__ constexpr int f4_row(int tok) {
    return (tok & ~7) | ((tok & 3) << 1) | ((tok >> 2) & 1);
}
__host__ __device__ constexpr int f4_token(int row) {
    return (row & ~7) | ((row & 1) << 2) | ((row >> 1) & 3);
}
// Byte offsets inside the four arrays.  Keys: the pair of dims d, d + 1 (d even).
template <int D>
__host__ __device__ constexpr int f4_k_byte(int tok, int d) {
    return f4_row(tok) * (D / 2) + ((d & 15) >> 2) * (D / 8) + (d >> 4) * 2 + ((d & 3) >> 1);
}
// Values: the row of a token's pair, and the byte of its dim d in the array.
__host__ __device__ constexpr int f4_pair(int tok) { return (tok >> 3) * 4 + (tok & 3); }
template <int D>
__host__ __device__ constexpr int f4_v_unit(int pair, int g) {
    return D == 128 ? (g ^ ((pair & 3) << 1)) : (g ^ ((pair & 2) << 1));
}
template <int D>
__host__ __device__ constexpr int f4_v_byte(int pair, int d) {
    return pair * D + f4_v_unit<D>(pair, (d & 15) >> 1) * (D / 8) + (d & 1) * (D / 16) + (d >> 4);
}
template <int D>
__host__ __device__ constexpr int f4_k_scale(int tok, int blk) {
    return f4_row(tok) * (D / 16) + blk;
}
template <int D>
__host__ __device__ constexpr int f4_v_scale(int tok, int blk) {
    return (f4_pair(tok) * (D / 16) + blk) * 2 + ((tok >> 2) & 1);
}

// Two E2M1 codes (low nibble first) as an fp16 pair.
__device__ __forceinline__ uint32_t f16x2_from_e2m1x2(uint32_t v8) {
    uint32_t r;
    asm("{\n\t.reg .b8 t;\n\tcvt.u8.u32 t, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, t;\n\t}" : "=r"(r) : "r"(v8));
    return r;
}
// The four code pairs of a word, and the two scale pairs of one.  Unpacking the
// register as bytes lets the conversion pick its byte itself: shifting each
// byte down first took 14.5 issue cycles a word where this takes 10.5 (8 of
// them the fp16 multiplies of the loop it was timed in).
__device__ __forceinline__ void f16x2_from_e2m1x8(uint32_t w, uint32_t (&r)[4]) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
        : "r"(w));
}
__device__ __forceinline__ void f16x2_from_e2m1x4(uint16_t w, uint32_t (&r)[2]) {
    asm("{\n\t.reg .b8 a, b;\n\tmov.b16 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t}"
        : "=r"(r[0]), "=r"(r[1])
        : "h"(w));
}
__device__ __forceinline__ void f16x2_from_e4m3x4(uint32_t w, uint32_t (&r)[2]) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(r[0]), "=r"(r[1])
        : "r"(w));
}
// E2M1 codes of two fp32 values (nearest even, saturating): lo in the low nibble.
__device__ __forceinline__ uint32_t e2m1x2_from_f32(float lo, float hi) {
    uint32_t r;
    asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n\tcvt.u32.u8 %0, t;\n\t}"
        : "=r"(r)
        : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
}
// mbar_wait by a whole warp: its lanes agree on whether the wait ran out.  (A
// vote on the first try, before any loop: 64 sequences of fp4 tiles under a
// shared prompt 58.7 us, with the one vote behind the loop 59.5.)
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity) {
    if (__all_sync(kFull, mbar_try_wait(bar, parity))) return true;
    return __all_sync(kFull, mbar_wait(bar, parity));
}
template <int N>
__device__ __forceinline__ void lds_words(const uint8_t* p, uint32_t (&w)[N]) {
    static_assert(N == 1 || N == 2 || N == 4, "one load");
    if constexpr (N == 4) {
        const uint4 v = *reinterpret_cast<const uint4*>(p);
        w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
    } else if constexpr (N == 2) {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        w[0] = v.x; w[1] = v.y;
    } else {
        w[0] = *reinterpret_cast<const uint32_t*>(p);
    }
}

// Scores of the 16 tokens of block `blk` against NB groups of 8 query rows:
// s[nb] is the accumulator tile (rows g and g + 8 = tokens f4_token(g) and
// f4_token(g + 8) of the block, columns 2t and 2t + 1 = query rows).  The
// E4M3 scale of a row differs from step to step, so each step's product is
// taken from zero and added times the scale in fp32 (two FMAs per row and
// column pair instead of scaling four operand registers, and no rounding).
// FEW: columns 2t and 2t + 1 are the same row (only the first of s is formed).
// qb[nb][kk]: query dims 16 kk + 4t, + 1 and 16 kk + 4t + 2, + 3.
template <int C, int D, int NB, bool FEW>
__device__ __forceinline__ void f4_scores(const uint8_t* tile, int blk, const uint32_t (&qb)[NB][D / 16][2],
                                          float (&s)[NB][4], int lane) {
    using T = F4Tile<C, D>;
    const int g = lane >> 2, t = lane & 3;
    const uint8_t* kc = tile + (blk * 16 + g) * (D / 2) + t * (D / 8);
    const uint8_t* ks = tile + T::kKScales + (blk * 16 + g) * (D / 16);
    uint32_t w0[D / 32], w1[D / 32], c0[D / 64], c1[D / 64];
    lds_words<D / 32>(kc, w0);
    lds_words<D / 32>(kc + 8 * (D / 2), w1);
    lds_words<D / 64>(ks, c0);
    lds_words<D / 64>(ks + 8 * (D / 16), c1);
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) s[nb][0] = s[nb][1] = s[nb][2] = s[nb][3] = 0.f;
#pragma unroll
    for (int sp = 0; sp < D / 64; ++sp) {                 // four steps: one word of scales per row
        uint32_t h0[2], h1[2];
        f16x2_from_e4m3x4(c0[sp], h0);
        f16x2_from_e4m3x4(c1[sp], h1);
#pragma unroll
        for (int kp = 2 * sp; kp < 2 * sp + 2; ++kp) {    // two steps: one word of codes per row
            const float2 f0 = __half22float2(*reinterpret_cast<const __half2*>(&h0[kp & 1]));
            const float2 f1 = __half22float2(*reinterpret_cast<const __half2*>(&h1[kp & 1]));
            uint32_t x0[4], x1[4];
            f16x2_from_e2m1x8(w0[kp], x0);
            f16x2_from_e2m1x8(w1[kp], x1);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const uint32_t a[4] = {x0[2 * e], x1[2 * e], x0[2 * e + 1], x1[2 * e + 1]};
                const float r0 = e ? f0.y : f0.x, r1 = e ? f1.y : f1.x;
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                    float acc[4] = {0.f, 0.f, 0.f, 0.f};
                    mma16816(acc, a, qb[nb][2 * kp + e][0], qb[nb][2 * kp + e][1]);
                    s[nb][0] = fmaf(acc[0], r0, s[nb][0]);
                    s[nb][2] = fmaf(acc[2], r1, s[nb][2]);
                    if constexpr (!FEW) {
                        s[nb][1] = fmaf(acc[1], r0, s[nb][1]);
                        s[nb][3] = fmaf(acc[3], r1, s[nb][3]);
                    }
                }
            }
        }
    }
}

// O^T += V^T p for the 16 tokens of block `blk`: o[nb][db] holds dims
// 16 db + 2g (c0, c1: query rows 2t, 2t + 1) and 16 db + 2g + 1 (c2, c3).
// pb[nb]: p's operand, token pairs (t, t + 4) and (t + 8, t + 12).  The values
// are scaled before the product (exact in fp16): a scale moved onto p would
// round p, whose small weights are near fp16's smallest already.
template <int C, int D, int NB>
__device__ __forceinline__ void f4_pv(const uint8_t* tile, int blk, const uint32_t (&pb)[NB][2],
                                      float (&o)[NB][D / 16][4], int lane) {
    using T = F4Tile<C, D>;
    const int g = lane >> 2, t = lane & 3;
    // pairs (t, t + 4) and (t + 8, t + 12) of the block: rows 8 blk + t and 4 on
    const uint8_t* vc = tile + T::kVCodes + (blk * 8 + t) * D + f4_v_unit<D>(t, g) * (D / 8);
    const uint8_t* vs = tile + T::kVScales + (blk * 8 + t) * (D / 8);
    constexpr int NW = D / 64;
    uint32_t ab[2 * NW], cd[2 * NW], sab[D / 32], scd[D / 32];
    lds_words<2 * NW>(vc, ab);                            // dims 16 db + 2g: words 0 .. NW - 1, then + 1
    lds_words<2 * NW>(vc + 4 * D, cd);
    lds_words<D / 32>(vs, sab);
    lds_words<D / 32>(vs + 4 * (D / 8), scd);
#pragma unroll
    for (int i = 0; i < NW; ++i) {                        // four blocks of dims per word
        uint32_t v0[4], v1[4], v2[4], v3[4];
        f16x2_from_e2m1x8(ab[i], v0);
        f16x2_from_e2m1x8(ab[NW + i], v1);
        f16x2_from_e2m1x8(cd[i], v2);
        f16x2_from_e2m1x8(cd[NW + i], v3);
#pragma unroll
        for (int j2 = 0; j2 < 2; ++j2) {
            uint32_t x[2], y[2];
            f16x2_from_e4m3x4(sab[2 * i + j2], x);
            f16x2_from_e4m3x4(scd[2 * i + j2], y);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int j = 2 * j2 + e;
                const uint32_t a[4] = {mul_f16x2(v0[j], x[e]), mul_f16x2(v1[j], x[e]), mul_f16x2(v2[j], y[e]),
                                       mul_f16x2(v3[j], y[e])};
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) mma16816(o[nb][4 * i + j], a, pb[nb][0], pb[nb][1]);
            }
        }
    }
}

}  // namespace dev
}  // namespace ca
