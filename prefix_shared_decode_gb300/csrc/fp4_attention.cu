// The two-phase decode attention kernel of a 4-bit pool.  It runs the same
// work plan as the kernels of the other pools (kernels.cu: units, the static
// lists and the tail queue, partial triples, the merge kernel after it); what
// differs is how a tile reaches the tensor cores.
//
//  * A chunk-head tile is one bulk copy (9216 bytes at 64 tokens x 128 dims).
//  * All products are taken transposed, tokens on the rows and query rows on
//    the columns (S^T = K Q^T, O^T += V^T P^T), 16 tokens at a time: the
//    tile's bytes widen straight into operand registers (fp4.cuh).
//  * Units of up to 8 query rows (every sequence-first unit of head groups up
//    to 8, chunk-first ones of few sharers): each of the four warps takes its
//    own 16 tokens of a tile and nothing is exchanged until the head ends.  Up
//    to 4 rows lie twice in the 8 columns, which halves a lane's softmax (four
//    query tokens over 2048 tokens of their own: 71.4 -> 66.7 us).
//  * Units of more rows: 64 tokens at a time, the warps split the tokens for the
//    scores and the dims for the outputs, so that each code is widened once;
//    the weights pass through shared memory.
//
// What bounds it: the widening (two ALU cycles for each pair of values, and a
// multiply for its scale), not the bytes: a single-row tile costs its four
// warps about 250 instructions each.  So the path is written for issue slots:
// a vote decides whether the softmax reference must rise, sums stay per lane
// until the head ends, queries of the next head are fetched a head ahead, and
// three CTAs per SM cover the latencies (at their 128 registers a thread the
// instances of 128 dims spill 196 to 288 bytes, those of 64 dims 16 to 28).
// 65536 tiles of single rows alone take 114 us, 79% of the copy rate; 64
// sequences of 512 tokens of their own under 4096 shared ones, 32 heads of 128
// dims, 55 us, where the own tiles by themselves take 38: the shared ones' 13.5
// steps of 64 rows an SM are the other 17, and their 544 products a step, at the
// 0.5 a cycle that an SM issues, some 7.5 of these.  (Widening shared tiles into
// fp16 in shared memory first, 16 rows a warp: 61 us.)
#include <cuda.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <climits>

#include "ca_internal.h"
#include "fp4.cuh"
#include "row_blocks.cuh"

namespace ca {
namespace dev {

constexpr int kF4Warps = 4, kF4Threads = 32 * (kF4Warps + 1);
constexpr int kF4Stages = 8, kF4Ring = 16;
// The softmax reference is kept kLift below a running maximum and raised only
// when a score passes it by kLift + kSlack: the weights stay below 2^13 in
// their fp16 operand and normal numbers down to 2^-19 (or less) of the largest.
constexpr float kLift = 5.f, kSlack = 8.f;

// Shared memory: the ring, two areas, (m, s) per warp and row.  For units of up
// to 8 rows the areas hold the warps' outputs at the end of a head, in turn;
// for others the weights of 64 tokens with their tables, and the queries.
constexpr int kWideTok = 64;                                    // tokens of a step
struct WideTables {
    float ref[kQRows], thr[kQRows], fall[kQRows];               // softmax references; scores that raise them; 2^(old - new)
    float top[kF4Warps][kQRows];                                // largest scores of each warp's tokens
    int32_t qrow[kQRows], lim[kQRows], pid[kQRows];             // rows of q (of head 0); causal limits; partial ids
};
template <int C, int D>
struct F4Smem {
    static constexpr int kStage = F4Tile<C, D>::kBytes;
    static constexpr int kOut8 = kF4Warps * 8 * D * 4;          // 8 rows of each warp
    static constexpr int kP = kQRows * kWideTok * 2;            // weights [row][token]
    static constexpr int kWide = kP + (int)sizeof(WideTables);
    static constexpr int kExch = kOut8 > kWide ? kOut8 : (kWide + 127) / 128 * 128;
    static constexpr int kMs = 2 * kF4Warps * 8 * 2 * 4;
    static constexpr int kQ = kQRows * D * 2;                   // query rows of a shared tile (= kOut8)
    static_assert(kQ >= kOut8, "the second area");
    static constexpr int kTail = kMs + 2 * kF4Stages * 8 + kF4Ring * 4 + 2 * kF4Stages * 4 + kQRows * 4;
    static size_t bytes(int stages) { return (size_t)stages * kStage + kExch + kQ + kTail; }
};

__device__ __forceinline__ void f4_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kF4Warps * 32) : "memory"); }
__device__ __forceinline__ bool f4_sync_any(bool x) {      // the same barrier: does x hold anywhere?
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, 1, %2, p;\n\t"
                 "selp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(r)
                 : "r"((uint32_t)x), "n"(kF4Warps * 32)
                 : "memory");
    return r != 0u;
}

// A wait for a tile that runs out: the warp reports it, takes no tile any more
// and goes on to the next barrier, which is a vote (at a unit's begin, where a
// small head's warps meet, where a wide step raises its references): the
// consumers leave together.  (A warp that left alone would have the others stand
// at a barrier that has no limit: a tile that lands at the end of the limit is
// seen by some warps only.)  So each warp gives up once at most, and the
// producer, which gets no slot back from it, after its own limit; the call's
// outputs are undefined.

// What the consumers' loops share.
struct F4Ctx {
    const uint8_t* stages;
    uint8_t *exch, *qreg;
    float* ms;
    uint32_t full0, empty0;
    const volatile int32_t *ntok, *tok0;
    int S, st, it;            // ring slots, the next one, tiles taken
    uint32_t ph;
    int w, lane, flush;       // flush: heads ended (exchange parity)
    // The test hook's other half, in CTAs of odd number: warp 0 behaves as if its
    // wait had run out while the tiles come, at a unit's first (in CTAs 4i + 1) or
    // inside a head (4i + 3).
    __device__ __forceinline__ bool gives_up(const AttnParams& p, uint32_t cta) const {
        return p.test_stall && (blockIdx.x & 3u) == cta && w == 0;
    }
    __device__ __forceinline__ void next() {
        ++it;
        if (++st == S) {
            st = 0;
            ph ^= 1u;
        }
    }
};

template <int D, int NB>
struct F4State {
    float o[NB][D / 16][4], m[NB][2], s[NB][2];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            m[nb][0] = m[nb][1] = -INFINITY;
            s[nb][0] = s[nb][1] = 0.f;
#pragma unroll
            for (int db = 0; db < D / 16; ++db) o[nb][db][0] = o[nb][db][1] = o[nb][db][2] = o[nb][db][3] = 0.f;
        }
    }
};

// Scaled and masked scores x of a 16-token block -> the operand p and the
// state's sums.  The weights are rounded to fp16 for the product with the values
// alone, as in the other pools' kernels (mma takes 16-bit operands; half a step,
// 2^-11 of each weight, so at most 2^-11 * sum p|v| of an output); their sum is
// of the unrounded ones, in fp32.  FEW (up to 4 rows): row r is in columns 2r and 2r + 1, so that a
// lane's two columns are one row and half the work is left.
template <int D, int NB, bool FEW>
__device__ __forceinline__ void f4_softmax(float (&x)[NB][4], F4State<D, NB>& a, uint32_t (&pb)[NB][2]) {
    bool grow = false;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int e = 0; e < 4; e += FEW ? 2 : 1) grow = grow || x[nb][e] > a.m[nb][e & 1] + (kLift + kSlack);
    if (__any_sync(kFull, grow)) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int r = 0; r < (FEW ? 1 : 2); ++r) {
                float mx = fmaxf(x[nb][r], x[nb][r + 2]);
#pragma unroll
                for (int d = 4; d <= 16; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, d));
                const float mn = fmaxf(a.m[nb][r], mx - kLift);
                const float al = mn == -INFINITY ? 1.f : ex2(a.m[nb][r] - mn);
                a.m[nb][r] = mn;
                a.s[nb][r] *= al;
#pragma unroll
                for (int db = 0; db < D / 16; ++db) {
                    a.o[nb][db][r] *= al;
                    a.o[nb][db][r + 2] *= al;
                }
            }
    }
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
        const float u0 = a.m[nb][0] == -INFINITY ? 0.f : a.m[nb][0];
        const float p0 = ex2(x[nb][0] - u0), p2 = ex2(x[nb][2] - u0);
        a.s[nb][0] += p0 + p2;                 // the lane's tokens; summed over the lanes at the end
        if constexpr (FEW) {
            pb[nb][0] = movm_trans(pack_half2(p0, p0));
            pb[nb][1] = movm_trans(pack_half2(p2, p2));
        } else {
            const float u1 = a.m[nb][1] == -INFINITY ? 0.f : a.m[nb][1];
            const float p1 = ex2(x[nb][1] - u1), p3 = ex2(x[nb][3] - u1);
            a.s[nb][1] += p1 + p3;
            pb[nb][0] = movm_trans(pack_half2(p0, p1));
            pb[nb][1] = movm_trans(pack_half2(p2, p3));
        }
    }
}

// Scale, the chunk's token count and (lim: per row) the causal limit.
template <int NB, bool FEW>
__device__ __forceinline__ void f4_mask(float (&x)[NB][4], int tok, int ntok, int ctx0, bool causal,
                                        const int (&lim)[NB][2], float scale_log2) {
    const bool in0 = tok < ntok, in1 = tok + 8 < ntok;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int e = 0; e < 4; e += FEW ? 2 : 1)
            x[nb][e] = ((e >> 1) ? in1 : in0) ? x[nb][e] * scale_log2 : -INFINITY;
    if (causal) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int e = 0; e < 4; e += FEW ? 2 : 1)
                if (ctx0 + tok + 8 * (e >> 1) > lim[nb][e & 1]) x[nb][e] = -INFINITY;
    }
}

// One head's `tiles` tiles, each warp taking 16 tokens of its own; false where
// its wait ran out.
template <int C, int D, int NB, bool FEW>
__device__ __forceinline__ bool f4_tiles_own(F4Ctx& c, const AttnParams& p, int tiles,
                                             const uint32_t (&qb)[NB][D / 16][2], const int (&lim)[NB][2],
                                             int first_lim, F4State<D, NB>& a) {
    constexpr int NBLK = C / 16;
    const int tg = f4_token(c.lane >> 2);
    if (c.gives_up(p, 3)) {
        set_status(p.status, CA_ERR_TIMEOUT);
        return false;
    }
    for (; tiles > 0; --tiles) {
        if (!warp_wait(c.full0 + 8 * c.st, c.ph)) {
            set_status(p.status, CA_ERR_TIMEOUT);
            return false;
        }
        const int ntok = c.ntok[c.st];
        // a tile's blocks go to the warps in turn, tile after tile
        const int blk = NBLK == 4 ? c.w : (c.w - c.it * NBLK) & 3;
        if (blk < NBLK && blk * 16 < ntok) {
            const uint8_t* tile = c.stages + (size_t)c.st * F4Tile<C, D>::kBytes;
            float x[NB][4];
            uint32_t pb[NB][2];
            f4_scores<C, D, NB, FEW>(tile, blk, qb, x, c.lane);
            const int tok0 = c.tok0[c.st];
            f4_mask<NB, FEW>(x, blk * 16 + tg, ntok, tok0, tok0 + (C - 1) > first_lim, lim, p.scale_log2);
            f4_softmax<D, NB, FEW>(x, a, pb);
            f4_pv<C, D, NB>(tile, blk, pb, a.o, c.lane);
        }
        __syncwarp();
        if (c.lane == 0) mbar_arrive(c.empty0 + 8 * c.st);
        c.next();
    }
    return true;
}

// Units of more than 8 rows (to 64).  A step takes 64 tokens: warp w the scores
// of 16 of them for all rows, then, with the weights of all 64 in shared
// memory, 16 D / 64 dims of all rows' outputs.  So every code is widened by one
// warp only, straight into its operand (code * scale is exact in fp16), and a
// row's output needs no meeting of warps at the end.  A row's softmax reference
// is the same for all warps: a barrier that is also a vote tells whether any
// score passes it by more than the slack.  The weights are rounded to fp16 for
// the product (half a step, 2^-11 of each), and summed in fp32 as rounded, by the
// tensor cores too: an output stays an average of its values exactly.
template <int C, int D, int NP>
__device__ __forceinline__ void f4_wide_scores(const uint8_t* tile, int blk, uint32_t qa, float (&s)[2 * NP][4],
                                               int lane) {
    using T = F4Tile<C, D>;
    const int g = lane >> 2, t = lane & 3, i = lane >> 3, j = lane & 7;
    const uint8_t* kc = tile + (blk * 16 + g) * (D / 2) + t * (D / 8);
    const uint8_t* ks = tile + T::kKScales + (blk * 16 + g) * (D / 16);
    const uint32_t row = qa + ((i >> 1) * 8 + j) * (2 * D), at = (uint32_t)((i & 1) ^ j);
#pragma unroll
    for (int nb = 0; nb < 2 * NP; ++nb) s[nb][0] = s[nb][1] = s[nb][2] = s[nb][3] = 0.f;
#pragma unroll
    for (int sp = 0; sp < D / 64; ++sp) {                 // four steps of 16 dims
        uint32_t w0[2], w1[2], c0[1], c1[1], h0[2], h1[2];
        lds_words<2>(kc + sp * 8, w0);
        lds_words<2>(kc + 8 * (D / 2) + sp * 8, w1);
        lds_words<1>(ks + sp * 4, c0);
        lds_words<1>(ks + 8 * (D / 16) + sp * 4, c1);
        f16x2_from_e4m3x4(c0[0], h0);
        f16x2_from_e4m3x4(c1[0], h1);
#pragma unroll
        for (int kp = 0; kp < 2; ++kp) {
            uint32_t x0[4], x1[4];
            f16x2_from_e2m1x8(w0[kp], x0);
            f16x2_from_e2m1x8(w1[kp], x1);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int kk = 4 * sp + 2 * kp + e;
                const uint32_t s0 = __byte_perm(h0[kp], 0u, e ? 0x3232 : 0x1010);
                const uint32_t s1 = __byte_perm(h1[kp], 0u, e ? 0x3232 : 0x1010);
                const uint32_t a[4] = {mul_f16x2(x0[2 * e], s0), mul_f16x2(x1[2 * e], s1),
                                       mul_f16x2(x0[2 * e + 1], s0), mul_f16x2(x1[2 * e + 1], s1)};
                const uint32_t col = row + ((at ^ (uint32_t)(2 * kk)) << 4);
#pragma unroll
                for (int n = 0; n < NP; ++n) {            // 16 rows at a time
                    uint32_t b[4];
                    ldsm_x4(col + n * 16 * 2 * D, b[0], b[1], b[2], b[3]);
                    mma16816(s[2 * n], a, b[0], b[1]);
                    mma16816(s[2 * n + 1], a, b[2], b[3]);
                }
            }
        }
    }
}

// Address of 16 rows' weights for the 16 tokens of block b of the step, as
// four 8 x 8 matrices (rows 0-7 and 8-15 of the first, then the next 8 tokens
// of each: the order of two operands); lane l addresses row l % 8 of matrix l / 8.
__device__ __forceinline__ uint32_t f4_p_addr(uint32_t pa, int n, int b, int lane) {
    const int i = lane >> 3, j = lane & 7;
    return pa + (uint32_t)((n * 16 + (i >> 1) * 8 + j) * (kWideTok * 2)) +
           (uint32_t)(((2 * b + (i & 1)) ^ j) << 4);
}
__device__ __forceinline__ void stsm_x4_t(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b),
                 "r"(c), "r"(d)
                 : "memory");
}

// O^T += V^T p for block b of the step (block `blk` of its tile): warp w's dims,
// all rows.  o[nb][d] as f4_pv's, d-th of the warp's groups of 16 dims.
template <int C, int D, int NP>
__device__ __forceinline__ void f4_wide_pv(const uint8_t* tile, int blk, int b, uint32_t pa,
                                           float (&o)[2 * NP][D / 64][4], int w, int lane) {
    using T = F4Tile<C, D>;
    constexpr int N = D / 64;
    const int g = lane >> 2, t = lane & 3;
    const uint8_t* vc = tile + T::kVCodes + (blk * 8 + t) * D + f4_v_unit<D>(t, g) * (D / 8) + N * w;
    const uint8_t* vs = tile + T::kVScales + (blk * 8 + t) * (D / 8) + 2 * N * w;
    uint32_t a[N][4];
    if constexpr (N == 2) {
        uint32_t v0[2], v1[2], v2[2], v3[2], x[2], y[2];
        f16x2_from_e2m1x4(*reinterpret_cast<const uint16_t*>(vc), v0);
        f16x2_from_e2m1x4(*reinterpret_cast<const uint16_t*>(vc + D / 16), v1);
        f16x2_from_e2m1x4(*reinterpret_cast<const uint16_t*>(vc + 4 * D), v2);
        f16x2_from_e2m1x4(*reinterpret_cast<const uint16_t*>(vc + 4 * D + D / 16), v3);
        f16x2_from_e4m3x4(*reinterpret_cast<const uint32_t*>(vs), x);
        f16x2_from_e4m3x4(*reinterpret_cast<const uint32_t*>(vs + 4 * (D / 8)), y);
#pragma unroll
        for (int d = 0; d < N; ++d) {
            a[d][0] = mul_f16x2(v0[d], x[d]);
            a[d][1] = mul_f16x2(v1[d], x[d]);
            a[d][2] = mul_f16x2(v2[d], y[d]);
            a[d][3] = mul_f16x2(v3[d], y[d]);
        }
    } else {
        const uint32_t x = f16x2_from_e4m3x2(*reinterpret_cast<const uint16_t*>(vs));
        const uint32_t y = f16x2_from_e4m3x2(*reinterpret_cast<const uint16_t*>(vs + 4 * (D / 8)));
        a[0][0] = mul_f16x2(f16x2_from_e2m1x2(vc[0]), x);
        a[0][1] = mul_f16x2(f16x2_from_e2m1x2(vc[D / 16]), x);
        a[0][2] = mul_f16x2(f16x2_from_e2m1x2(vc[4 * D]), y);
        a[0][3] = mul_f16x2(f16x2_from_e2m1x2(vc[4 * D + D / 16]), y);
    }
#pragma unroll
    for (int n = 0; n < NP; ++n) {
        uint32_t pb[4];
        ldsm_x4(f4_p_addr(pa, n, b, lane), pb[0], pb[1], pb[2], pb[3]);
#pragma unroll
        for (int d = 0; d < N; ++d) {
            mma16816(o[2 * n][d], a[d], pb[0], pb[1]);
            mma16816(o[2 * n + 1][d], a[d], pb[2], pb[3]);
        }
    }
}

// One head of such a unit: its `tiles` tiles over NP blocks of 16 rows (a loop
// to a number known at run time would wait for every load of operands), whose
// queries lie in qreg (word 2t of a row's 16 dims before word 2t + 1 of all t:
// the operand order of the widened keys), to the partials of its rows.
// scale_log2 > 0.  False, for all warps, where a wait ran out.
template <int C, int D, int NP>
__device__ __forceinline__ bool f4_wide_head(F4Ctx& c, const AttnParams& p, WideTables* tab, int tiles, int rows,
                                             float scale_log2) {
    constexpr int N = D / 64, NBLK = C / 16, TP = 4 / NBLK;     // tiles of a step
    const int lane = c.lane, g = lane >> 2, t = lane & 3, w = c.w;
    const uint32_t qa = smem_u32(c.qreg), pa = smem_u32(c.exch);
    float o[2 * NP][N][4], sum[2][4];
#pragma unroll
    for (int nb = 0; nb < 2 * NP; ++nb)
#pragma unroll
        for (int d = 0; d < N; ++d) o[nb][d][0] = o[nb][d][1] = o[nb][d][2] = o[nb][d][3] = 0.f;
#pragma unroll
    for (int k = 0; k < 2; ++k) sum[k][0] = sum[k][1] = sum[k][2] = sum[k][3] = 0.f;
    // (tiles up to the first of the rows' causal limits need no mask)
    const int first_lim = p.causal ? __reduce_min_sync(kFull, min(tab->lim[lane], tab->lim[lane + 32])) : 0;
    bool first = true;
#pragma unroll 1
    for (; tiles > 0; tiles -= TP, first = false) {
        const int nt = min(tiles, TP);
        auto slot_of = [&](int k) { return c.st + k < c.S ? c.st + k : c.st + k - c.S; };
        bool late = c.gives_up(p, 3);          // a wait ran out: on to the vote
        for (int k = 0; k < nt && !late; ++k) {
            const int sl = slot_of(k);
            late = !warp_wait(c.full0 + 8 * sl, c.st + k < c.S ? c.ph : c.ph ^ 1u);
        }
        if (late) set_status(p.status, CA_ERR_TIMEOUT);
        float s[2 * NP][4];
        {
            const int k = w / NBLK, blk = w % NBLK, sl = slot_of(k);
            const int left = k < nt && !late ? c.ntok[sl] - blk * 16 : 0;      // tokens of the warp's block
            if (left > 0) {
                f4_wide_scores<C, D, NP>(c.stages + (size_t)sl * F4Tile<C, D>::kBytes, blk, qa, s, lane);
                const int tg = f4_token(g);
                if (left < 16) {
#pragma unroll
                    for (int nb = 0; nb < 2 * NP; ++nb)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (tg + 8 * (e >> 1) >= left) s[nb][e] = -INFINITY;
                }
                if (p.causal && c.tok0[sl] + C - 1 > first_lim) {
                    const int tok = c.tok0[sl] + blk * 16 + tg;
#pragma unroll
                    for (int nb = 0; nb < 2 * NP; ++nb) {
                        const int2 lim = *reinterpret_cast<const int2*>(tab->lim + nb * 8 + 2 * t);
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (tok + 8 * (e >> 1) > ((e & 1) ? lim.y : lim.x)) s[nb][e] = -INFINITY;
                    }
                }
            } else {
#pragma unroll
                for (int nb = 0; nb < 2 * NP; ++nb) s[nb][0] = s[nb][1] = s[nb][2] = s[nb][3] = -INFINITY;
            }
        }
        bool grow = late;
        if (!first) {
#pragma unroll
            for (int nb = 0; nb < 2 * NP; ++nb) {
                const float2 thr = *reinterpret_cast<const float2*>(&tab->thr[nb * 8 + 2 * t]);
                grow = grow | (fmaxf(s[nb][0], s[nb][2]) > thr.x) | (fmaxf(s[nb][1], s[nb][3]) > thr.y);
            }
        }
        // (past the vote every warp has read the last step's weights, too)
        if (first || f4_sync_any(grow)) {
#pragma unroll
            for (int nb = 0; nb < 2 * NP; ++nb) {
                float2 mx = make_float2(fmaxf(s[nb][0], s[nb][2]), fmaxf(s[nb][1], s[nb][3]));
#pragma unroll
                for (int d = 4; d <= 16; d <<= 1) {
                    mx.x = fmaxf(mx.x, __shfl_xor_sync(kFull, mx.x, d));
                    mx.y = fmaxf(mx.y, __shfl_xor_sync(kFull, mx.y, d));
                }
                if (g == 0) *reinterpret_cast<float2*>(&tab->top[w][nb * 8 + 2 * t]) = mx;
            }
            if (f4_sync_any(late)) return false;
            if (const int row = threadIdx.x; row < NP * 16) {
                const float old = first ? -FLT_MAX : tab->ref[row];      // (any finite score raises it)
                const float mx = fmaxf(fmaxf(tab->top[0][row], tab->top[1][row]),
                                       fmaxf(tab->top[2][row], tab->top[3][row]));
                const float ref = fmaxf(old, mx * scale_log2 - kLift);
                tab->ref[row] = ref;
                tab->thr[row] = (ref + (kLift + kSlack)) / scale_log2;
                tab->fall[row] = ex2(old - ref);
            }
            f4_sync();
            if (!first) {
#pragma unroll
                for (int nb = 0; nb < 2 * NP; ++nb) {
                    const float2 f = *reinterpret_cast<const float2*>(&tab->fall[nb * 8 + 2 * t]);
#pragma unroll
                    for (int d = 0; d < N; ++d) {
                        o[nb][d][0] *= f.x;
                        o[nb][d][1] *= f.y;
                        o[nb][d][2] *= f.x;
                        o[nb][d][3] *= f.y;
                    }
                    if (nb >> 1 == w) {
                        sum[nb & 1][0] *= f.x;
                        sum[nb & 1][1] *= f.y;
                    }
                }
            }
        }
#pragma unroll
        for (int n = 0; n < NP; ++n) {
            uint32_t pk[4];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int nb = 2 * n + k;
                const float2 ref = *reinterpret_cast<const float2*>(&tab->ref[nb * 8 + 2 * t]);
                pk[2 * k] = pack_half2(ex2(fmaf(s[nb][0], scale_log2, -ref.x)),
                                       ex2(fmaf(s[nb][1], scale_log2, -ref.y)));
                pk[2 * k + 1] = pack_half2(ex2(fmaf(s[nb][2], scale_log2, -ref.x)),
                                           ex2(fmaf(s[nb][3], scale_log2, -ref.y)));
            }
            stsm_x4_t(f4_p_addr(pa, n, w, lane), pk[0], pk[1], pk[2], pk[3]);
        }
        f4_sync();
        // A tile is zero past its tokens, so one test for each is enough, and the
        // loads of its four blocks need not wait for one another.
#pragma unroll
        for (int k = 0; k < TP; ++k) {
            const int sl = slot_of(k);
            if (k < nt && c.ntok[sl] > 0) {
                const uint8_t* tile = c.stages + (size_t)sl * F4Tile<C, D>::kBytes;
#pragma unroll
                for (int blk = 0; blk < NBLK; ++blk)
                    f4_wide_pv<C, D, NP>(tile, blk, k * NBLK + blk, pa, o, w, lane);
                if (w < NP) {                              // the sums of 16 rows: a product with ones
                    const uint32_t ones[4] = {0x3c003c00u, 0x3c003c00u, 0x3c003c00u, 0x3c003c00u};
#pragma unroll
                    for (int blk = 0; blk < NBLK; ++blk) {
                        uint32_t pb[4];
                        ldsm_x4(f4_p_addr(pa, w, k * NBLK + blk, lane), pb[0], pb[1], pb[2], pb[3]);
                        mma16816(sum[0], ones, pb[0], pb[1]);
                        mma16816(sum[1], ones, pb[2], pb[3]);
                    }
                }
            }
        }
        __syncwarp();
        for (int k = 0; k < nt; ++k) {
            if (lane == 0) mbar_arrive(c.empty0 + 8 * c.st);
            c.next();
        }
    }
#pragma unroll
    for (int nb = 0; nb < 2 * NP; ++nb)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int row = nb * 8 + 2 * t + r;
            if (row < rows) {
                const int id = tab->pid[row];
#pragma unroll
                for (int d = 0; d < N; ++d)
                    *reinterpret_cast<float2*>(p.part_o + (size_t)id * D + 16 * (N * w + d) + 2 * g) =
                        make_float2(o[nb][d][r], o[nb][d][r + 2]);
                if (nb >> 1 == w && g == 0) {
                    const float all = sum[nb & 1][r];      // 0: no token of the unit is the row's
                    p.part_ms[id] = make_float2(all == 0.f ? -INFINITY : tab->ref[row], all);
                }
            }
        }
    return true;
}

// The end of a head of at most 8 rows: the warps' states meet in the exchange
// area (two buffers in turn, so that a head's stores never meet the last head's
// loads) and warp w writes the partials of rows w and w + 4.  Lane j holds the
// first partial id of row w + 4 j's pieces, this one is `part` further: added
// here, so that the id's load, begun with the head, is first waited for here.
template <int C, int D, bool FEW>
__device__ __forceinline__ bool f4_finish(F4Ctx& c, const AttnParams& p, F4State<D, 1>& a, int rows, int pid, int part,
                                          bool late) {
    const int g = c.lane >> 2, t = c.lane & 3;
    float* ob = reinterpret_cast<float*>((c.flush & 1) ? c.qreg : c.exch);
    // column of a row's dim: the fragments' stores of four rows stay apart
    auto col = [](int row, int d) { return d ^ ((row >> 1 & 3) << 3); };
    float* ms = c.ms + (c.flush & 1) * kF4Warps * 8 * 2;
    ++c.flush;
#pragma unroll
    for (int r = 0; r < (FEW ? 1 : 2); ++r) {
        float s = a.s[0][r];
#pragma unroll
        for (int d = 4; d <= 16; d <<= 1) s += __shfl_xor_sync(kFull, s, d);
        const int row = FEW ? t : 2 * t + r;
        if (!FEW || t < rows) {
            if (g == 0) *reinterpret_cast<float2*>(ms + (c.w * 8 + row) * 2) = make_float2(a.m[0][r], s);
#pragma unroll
            for (int db = 0; db < D / 16; ++db)
                *reinterpret_cast<float2*>(ob + (c.w * 8 + row) * D + col(row, 16 * db + 2 * g)) =
                    make_float2(a.o[0][db][r], a.o[0][db][r + 2]);
        }
    }
    if (f4_sync_any(late)) return false;
    for (int row = c.w, j = 0; row < rows; row += kF4Warps, ++j) {
        const int id = __shfl_sync(kFull, pid, j) + part;
        float2 q[kF4Warps];
        float M = -INFINITY, sum = 0.f;
#pragma unroll
        for (int k = 0; k < kF4Warps; ++k) {
            q[k] = *reinterpret_cast<const float2*>(ms + (k * 8 + row) * 2);
            M = fmaxf(M, q[k].x);
        }
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < kF4Warps; ++k) {
            const float wt = q[k].x == -INFINITY ? 0.f : ex2(q[k].x - M);
            sum += wt * q[k].y;
            if (c.lane < D / 4) {
                const float4 v = *reinterpret_cast<const float4*>(ob + (k * 8 + row) * D + col(row, 4 * c.lane));
                acc.x += wt * v.x; acc.y += wt * v.y; acc.z += wt * v.z; acc.w += wt * v.w;
            }
        }
        if (c.lane < D / 4) reinterpret_cast<float4*>(p.part_o + (size_t)id * D)[c.lane] = acc;
        if (c.lane == 0) p.part_ms[id] = make_float2(M, sum);
    }
    return true;
}

template <int C, int D>
__global__ void __launch_bounds__(kF4Threads, 3)
fp4_attention_kernel(const __grid_constant__ CUtensorMap, const AttnParams p) {
    using SM = F4Smem<C, D>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int S = p.n_stages;
    uint8_t* stages = smem;
    uint8_t* exch = smem + (size_t)S * SM::kStage;
    uint8_t* qreg = exch + SM::kExch;
    float* ms = reinterpret_cast<float*>(qreg + SM::kQ);
    uint64_t* bars = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(ms) + SM::kMs);
    volatile int32_t* ring = reinterpret_cast<volatile int32_t*>(bars + 2 * kF4Stages);
    volatile int32_t* stage_ntok = ring + kF4Ring;
    volatile int32_t* stage_tok0 = stage_ntok + kF4Stages;
    // row r of a unit: its position (from q_lo), query token and head of the group
    int32_t* row_tab = const_cast<int32_t*>(stage_tok0) + kF4Stages;
    const uint32_t full0 = smem_u32(bars), empty0 = smem_u32(bars + kF4Stages);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int H = p.n_heads, HK = p.n_kv_heads, G = p.group, QL = p.q_len, RW = QL * G;
    // The merge kernel may be scheduled now; it waits for this grid itself.
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (S < 64 / C || S > kF4Stages) {                     // uniform across the CTA
        if (threadIdx.x == 0) set_status(p.status, CA_ERR_INVALID);
        return;
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(full0 + 8 * i, 1);
            mbar_init(empty0 + 8 * i, kF4Warps);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (threadIdx.x < kQRows) {
        const int r = threadIdx.x;
        row_tab[r] = (r / RW) << 16 | (r % RW / G) << 8 | r % G;
    }
    __syncthreads();
    const CtaHead* hd = p.cta_head + blockIdx.x;
    const int2 range = *reinterpret_cast<const int2*>(hd);
    const int u_begin = range.x, u_end = range.y;

    if (warp == kF4Warps) {
        // ------------------------------ producer ------------------------------
        // The walk of kernels.cu's producer (static units, then the tail queue,
        // one claim ahead; the pool before the dependency wait only where
        // kv_stable says so); a step is one bulk copy.
        if (lane != 0) return;
        if (p.test_stall && !(blockIdx.x & 1)) {
            if (!mbar_wait(full0, 0u)) set_status(p.status, CA_ERR_TIMEOUT);
            return;
        }
        const uint64_t pol = policy_evict_first();
        auto lin_n = [](const Unit& X) { return X.kind == UNIT_SF ? X.n_per_head : X.c_end - X.c_begin; };
        auto lin_base = [](const Unit& X) { return X.kind == UNIT_SF ? X.base : X.c_begin; };
        auto lin_begin = [&](const Unit& X) { return X.kind == UNIT_SF ? X.c_begin : X.head * lin_n(X); };
        auto lin_end = [&](const Unit& X) {
            return X.kind == UNIT_SF ? X.c_end : (X.head + X.n_per_head) * lin_n(X);
        };
        auto first_chunk = [&](const Unit& X) { return lin_base(X) + lin_begin(X) % lin_n(X); };
        bool dep_done = false;
        auto dep_wait = [&]() {
            if (!dep_done) {
                asm volatile("griddepcontrol.wait;" ::: "memory");
                dep_done = true;
            }
        };
        int s_next = u_begin;
        auto claim = [&]() -> int {
            if (s_next < u_end) return s_next++;
            dep_wait();
            const int k = atomicAdd(p.dyn_counter, 1);
            return (p.dyn_begin + k < p.dyn_end) ? p.dyn_begin + k : -1;
        };
        int cur = (u_begin < u_end) ? s_next++ : -1;
        bool from_head = cur >= 0;
        Unit Un = from_head ? hd->first : Unit{};
        ChunkRef chn = from_head ? hd->refs[0] : ChunkRef{0, 0};
        int tkn = (from_head && p.causal) ? p.chunk_tok0[first_chunk(Un)] : 0;
        if (!p.kv_stable) dep_wait();
        if (cur < 0) {
            cur = claim();
            if (cur >= 0) {
                Un = p.units[cur];
                chn = p.chunks[first_chunk(Un)];
                if (p.causal) tkn = p.chunk_tok0[first_chunk(Un)];
            }
        }
        int it = 0, seq = 0;
        bool ok = true;
        for (; cur >= 0 && ok; ++seq) {
            const Unit U = Un;
            ring[seq % kF4Ring] = cur;
            int nxt = -1;
            bool have_next = false;
            const int n = lin_n(U), base = lin_base(U), L0 = lin_begin(U), L1 = lin_end(U);
            const int claim_at = max(L0, L1 - 2);
            int h = L0 / n, j = L0 - h * n;
            for (int L = L0; L < L1; ++L, ++it) {
                if (!have_next && L >= claim_at) {
                    nxt = claim();
                    if (nxt >= 0) Un = p.units[nxt];
                    have_next = true;
                }
                const ChunkRef ch = chn;
                const int tok0 = tkn, head = h;
                const bool slot_ok = ch.slot >= 0 && ch.slot < p.capacity;
                const int ntok = slot_ok ? p.slot_ntok[ch.slot] : 0;
                if (++j == n) { j = 0; ++h; }
                if (L + 1 < L1) {
                    chn = (from_head && L + 1 - L0 < kHeadRefs) ? hd->refs[L + 1 - L0] : p.chunks[base + j];
                    if (p.causal) tkn = p.chunk_tok0[base + j];
                } else if (nxt >= 0) {
                    chn = p.chunks[first_chunk(Un)];
                    if (p.causal) tkn = p.chunk_tok0[first_chunk(Un)];
                }
                const int st = it % S;
                if (!mbar_wait(empty0 + 8 * st, ((uint32_t)(it / S) & 1u) ^ 1u)) {
                    set_status(p.status, CA_ERR_TIMEOUT);
                    ok = false;
                    break;
                }
                const uint32_t fb = full0 + 8 * st;
                if (!slot_ok || head < 0 || head >= HK) {
                    set_status(p.status, CA_ERR_DEVICE_BOUNDS);
                    stage_ntok[st] = 0;
                    mbar_arrive(fb);                       // release the consumers without data
                    continue;
                }
                mbar_expect_tx_only(fb, SM::kStage);
                bulk_load(smem_u32(stages + (size_t)st * SM::kStage),
                          p.kv + (((long long)ch.slot * p.n_layers + p.layer) * HK + head) * SM::kStage, SM::kStage,
                          fb, pol);
                stage_ntok[st] = min(max(ntok, 0), C);
                stage_tok0[st] = tok0;
                mbar_arrive(fb);
            }
            if (!have_next) nxt = -1;                      // left early on a timeout
            from_head = false;
            cur = nxt;
        }
        if (ok) {
            // end of work: one more stage, without data, carries the id -1
            const int st = it % S;
            if (mbar_wait(empty0 + 8 * st, ((uint32_t)(it / S) & 1u) ^ 1u)) {
                ring[seq % kF4Ring] = -1;
                mbar_arrive(full0 + 8 * st);
            } else {
                set_status(p.status, CA_ERR_TIMEOUT);
                ok = false;
            }
        }
        if (!ok) {
            // Give the copies already issued a bounded chance to land before
            // the CTA can exit.
            for (int k = (it > S ? it - S : 0); k < it; ++k)
                mbar_wait(full0 + 8 * (k % S), (uint32_t)(k / S) & 1u);
        }
        return;
    }

    // ------------------------------ consumers ------------------------------
    enum { F_KIND = 0, F_HEAD, F_QLO, F_QHI, F_CB, F_CE, F_PART, F_QROW, F_N, F_BASE, F_PNEXT };
    auto load_desc = [&](int u) -> int32_t {
        return lane < kUnitInts ? reinterpret_cast<const int32_t*>(p.units + u)[lane] : 0;
    };
    auto fld = [&](int32_t d, int i) -> int32_t { return __shfl_sync(kFull, d, i); };
    F4Ctx c{stages, exch, qreg, ms, full0, empty0, stage_ntok, stage_tok0, S, 0, 0, 0u, warp, lane, 0};
    const int w = warp, g = lane >> 2, t = lane & 3;
    auto tab_pos = [](int32_t e) { return e >> 16; };
    auto tab_tok = [](int32_t e) { return e >> 8 & 0xff; };
    auto tab_head = [](int32_t e) { return e & 0xff; };
    const bool few = RW <= 4;                  // rows of a position twice over, see f4_softmax
    const int gr = few ? g >> 1 : g;           // the row in column g of a position's rows
    const int gt = tab_tok(row_tab[gr]), gh = tab_head(row_tab[gr]);

    // Query rows in operand order.  One position's rows g < RW (its row of q
    // known from the unit), and any unit's rows.
    using Q1 = uint32_t[1][D / 16][2];
    auto put_row = [&](uint32_t (&dst)[D / 16][2], const uint16_t* q, bool there) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            uint2 x = make_uint2(0u, 0u);
            if (there) x = *reinterpret_cast<const uint2*>(q + 16 * kk + 4 * t);
            dst[kk][0] = x.x;
            dst[kk][1] = x.y;
        }
    };
    auto load_own = [&](Q1& dst, int qrow, int kvh) {
        const bool there = gr < RW;
        put_row(dst[0], p.q + (((size_t)qrow * QL + (there ? gt : 0)) * H + kvh * G + (there ? gh : 0)) * D, there);
    };
    Q1 qn;                                     // the next head's queries ...
    int qn_row = -1, qn_head = -1;             // ... and which they are
    auto prefetch = [&](int qrow, int kvh) {
        load_own(qn, qrow, kvh);
        qn_row = qrow;
        qn_head = kvh;
    };

    const int n_static = u_end - u_begin;
    int32_t dn = (n_static > 0) ? load_desc(u_begin) : 0;
    // What a unit of more rows asks of the plan: its rows' places in q, causal
    // limits and partial ids.
    WideTables* const tab = reinterpret_cast<WideTables*>(exch + SM::kP);
    auto wide_rows = [&](int q_lo, int rows, int kvh, int upart) {
        if (threadIdx.x >= kQRows) return;
        const int r = threadIdx.x, e = row_tab[r], at = q_lo + tab_pos(e);
        if (r < rows) {
            tab->qrow[r] = (p.seq_perm[at] * QL + tab_tok(e)) * H + tab_head(e);
            tab->pid[r] = p.pbase[((size_t)at * QL + tab_tok(e)) * H + kvh * G + tab_head(e)] + upart;
        }
        tab->lim[r] = p.causal && r < rows ? p.ctx_len[at] - QL + tab_tok(e) : INT_MAX;
    };
    asm volatile("griddepcontrol.wait;" ::: "memory");     // q and the pool after this
    if (n_static > 0 && RW <= 8 && fld(dn, F_KIND) == UNIT_SF) prefetch(fld(dn, F_QROW), fld(dn, F_HEAD));
    for (int seq = 0;; ++seq) {
        // The unit's first stage (or the closing one) carries its id.
        const bool in = !c.gives_up(p, 1) && warp_wait(full0 + 8 * c.st, c.ph);
        if (!in) set_status(p.status, CA_ERR_TIMEOUT);
        const int cur = ring[seq % kF4Ring];   // (anything, if that ran out)
        const int32_t dc = (seq < n_static) ? dn : (in && cur >= 0) ? load_desc(cur) : 0;
        const bool next_static = seq + 1 < n_static;
        if (next_static) dn = load_desc(u_begin + seq + 1);
        const bool next_own = next_static && RW <= 8 && fld(dn, F_KIND) == UNIT_SF;
        if (f4_sync_any(!in)) return;          // (the previous unit's exchange has been read, too)
        if (cur < 0) break;
        const bool is_sf = fld(dc, F_KIND) == UNIT_SF;
        const int q_lo = fld(dc, F_QLO), q_hi = fld(dc, F_QHI), cb = fld(dc, F_CB), ce = fld(dc, F_CE);
        const int qrow = fld(dc, F_QROW);
        const int n = is_sf ? fld(dc, F_N) : ce - cb;
        int L = is_sf ? cb : fld(dc, F_HEAD) * n;
        const int L_end = is_sf ? ce : (fld(dc, F_HEAD) + fld(dc, F_N)) * n;
        int upart = fld(dc, F_PART);
        const int part_rest = is_sf ? fld(dc, F_PNEXT) : upart;
        const int rows = (q_hi - q_lo) * RW;   // rows of the unit: position, query token, head of the group
        // The partial of row r for key/value head kvh.
        auto pid_of = [&](int r, int kvh) {
            const int32_t e = row_tab[r];
            return p.pbase[((size_t)(q_lo + tab_pos(e)) * QL + tab_tok(e)) * H + kvh * G + tab_head(e)];
        };
        auto limit_of = [&](int r) {
            if (!p.causal || r >= rows) return INT_MAX;
            return p.ctx_len[q_lo + tab_pos(row_tab[r])] - QL + tab_tok(row_tab[r]);
        };
        // q of row r (key/value head 0)
        auto q_of = [&](int r) {
            const int32_t e = row_tab[r];
            return p.q + (((size_t)p.seq_perm[q_lo + tab_pos(e)] * QL + tab_tok(e)) * H + tab_head(e)) * D;
        };
        int kvh = L / n;
        if (rows <= 8) {
            const bool half = rows <= 4;
            int lim[1][2] = {{limit_of(half ? t : 2 * t), limit_of(half ? t : 2 * t + 1)}};
            // (tiles up to the first of the rows' causal limits need no mask)
            const int first_lim = p.causal ? __reduce_min_sync(kFull, min(lim[0][0], lim[0][1])) : INT_MAX;
            for (; L < L_end; ++kvh, upart = part_rest) {
                const int seg_end = min(L_end, (kvh + 1) * n);
                Q1 qb;
                if (is_sf) {
                    if (qn_row != qrow || qn_head != kvh) prefetch(qrow, kvh);
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        qb[0][kk][0] = qn[0][kk][0];
                        qb[0][kk][1] = qn[0][kk][1];
                    }
                    if (seg_end < L_end) prefetch(qrow, kvh + 1);
                    else if (next_own) prefetch(fld(dn, F_QROW), fld(dn, F_HEAD));
                } else {
                    const int r = half ? g >> 1 : g;
                    put_row(qb[0], q_of(r < rows ? r : 0) + (size_t)kvh * G * D, r < rows);
                }
                const int pid = (lane < 2 && w + 4 * lane < rows) ? pid_of(w + 4 * lane, kvh) : 0;
                F4State<D, 1> a;
                a.clear();
                if (half) {
                    const bool all = f4_tiles_own<C, D, 1, true>(c, p, seg_end - L, qb, lim, first_lim, a);
                    if (!f4_finish<C, D, true>(c, p, a, rows, pid, upart, !all)) return;
                } else {
                    const bool all = f4_tiles_own<C, D, 1, false>(c, p, seg_end - L, qb, lim, first_lim, a);
                    if (!f4_finish<C, D, false>(c, p, a, rows, pid, upart, !all)) return;
                }
                L = seg_end;
            }
        } else {
            qn_row = -1;                       // (its registers are wanted here)
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) qn[0][kk][0] = qn[0][kk][1] = 0u;
            // The scale's sign goes to the queries, and a scale of zero makes
            // them zero, so that larger products are larger scores below.
            const uint32_t flip = p.scale_log2 < 0.f ? 0x80008000u : 0u, keep = p.scale_log2 == 0.f ? 0u : 0xffffffffu;
            const float scale_log2 = p.scale_log2 == 0.f ? 1.f : fabsf(p.scale_log2);
            const int np = rows <= 16 ? 1 : rows <= 32 ? 2 : 4;
            for (; L < L_end; ++kvh, upart = part_rest) {
                const int seg_end = min(L_end, (kvh + 1) * n);
                f4_sync();                     // the last head's queries and tables have been read
                wide_rows(q_lo, rows, kvh, upart);
                f4_sync();
                constexpr int M = kQRows * (D / 16) / (kF4Warps * 32);   // 16 dims of a row at a time
                uint4 a[M], b[M];
#pragma unroll
                for (int k = 0; k < M; ++k) {
                    const int i = threadIdx.x + k * kF4Warps * 32, r = i / (D / 16), kk = i % (D / 16);
                    a[k] = b[k] = make_uint4(0u, 0u, 0u, 0u);
                    if (r < rows) {
                        const uint4* q =
                            reinterpret_cast<const uint4*>(p.q + ((size_t)tab->qrow[r] + kvh * G) * D + kk * 16);
                        a[k] = q[0];
                        b[k] = q[1];
                    }
                }
#pragma unroll
                for (int k = 0; k < M; ++k) {
                    const int i = threadIdx.x + k * kF4Warps * 32, r = i / (D / 16), kk = i % (D / 16);
                    auto put = [&](int x, uint4 v) {
                        *reinterpret_cast<uint4*>(qreg + r * (2 * D) + (((2 * kk + x) ^ (r & 7)) << 4)) =
                            make_uint4((v.x ^ flip) & keep, (v.y ^ flip) & keep, (v.z ^ flip) & keep,
                                       (v.w ^ flip) & keep);
                    };
                    if (r < np * 16) {
                        put(0, make_uint4(a[k].x, a[k].z, b[k].x, b[k].z));
                        put(1, make_uint4(a[k].y, a[k].w, b[k].y, b[k].w));
                    }
                }
                f4_sync();
                const int tiles = seg_end - L;
                if (!(np == 1   ? f4_wide_head<C, D, 1>(c, p, tab, tiles, rows, scale_log2)
                      : np == 2 ? f4_wide_head<C, D, 2>(c, p, tab, tiles, rows, scale_log2)
                                : f4_wide_head<C, D, 4>(c, p, tab, tiles, rows, scale_log2)))
                    return;
                L = seg_end;
            }
        }
    }
}

}  // namespace dev

namespace {
template <int C, int D>
void* f4_ptr() {
    return reinterpret_cast<void*>(&dev::fp4_attention_kernel<C, D>);
}
}  // namespace

void* fp4_kernel(const PoolCfg& c) {
    if (c.head_dim == 128)
        return c.chunk == 64 ? f4_ptr<64, 128>() : c.chunk == 32 ? f4_ptr<32, 128>() : f4_ptr<16, 128>();
    if (c.head_dim == 64) return c.chunk == 64 ? f4_ptr<64, 64>() : c.chunk == 32 ? f4_ptr<32, 64>() : f4_ptr<16, 64>();
    return nullptr;
}

size_t fp4_smem_bytes(const PoolCfg& c, int stages) {
    if (c.head_dim == 128)
        return c.chunk == 64   ? dev::F4Smem<64, 128>::bytes(stages)
               : c.chunk == 32 ? dev::F4Smem<32, 128>::bytes(stages)
                               : dev::F4Smem<16, 128>::bytes(stages);
    return c.chunk == 64   ? dev::F4Smem<64, 64>::bytes(stages)
           : c.chunk == 32 ? dev::F4Smem<32, 64>::bytes(stages)
                           : dev::F4Smem<16, 64>::bytes(stages);
}

}  // namespace ca
