// A chunk-head tile against 16-row blocks of a query tile, on the tensor cores
// (shared by the two-phase kernels of all pool types).
#pragma once

#include "device.cuh"

namespace ca {
namespace dev {

constexpr int kQRows = 64;                 // query rows per tensor-core unit, max (D <= 128)
// Query rows of the Q tile: 32 at head_dim 256 (the tile stays 16 KiB).
template <int D>
__host__ __device__ constexpr int q_rows() { return D == 256 ? 32 : kQRows; }

// ---------------------------------------------------------------------------
// Tensor-core path (chunk-first units, and sequence-first units with several
// query rows): one chunk-head tile against a 16-row block of the Q tile with
// mma.sync m16n8k16 (fp16 in, fp32 accumulate).  The warp takes tokens
// [tok0, tok0 + NT) of the chunk.  Row state per thread: rows g = lane/4 and
// g + 8 of the block.
// ---------------------------------------------------------------------------
// Scores of a 16-row block against NT tokens [tok0, tok0 + NT) of a chunk
// tile, over the head dims [16 kk0, 16 kk1): S = Q K^T with the Q fragments
// read from the swizzled Q tile (row lane%16, 16-byte chunk 2kk + lane/16).
template <int C, int D, int NT, bool F8 = false>
__device__ __forceinline__ void cf_scores(uint32_t kt, int tok0, uint32_t qrow_addr_base, int kk0, int kk1,
                                          float (&sacc)[NT / 8][4], int lane) {
#pragma unroll
    for (int i = 0; i < NT / 8; ++i) sacc[i][0] = sacc[i][1] = sacc[i][2] = sacc[i][3] = 0.f;
    if constexpr (F8) {
        // E4M3 keys (128-byte rows, 16-byte chunk kk of row r at chunk
        // kk ^ (r % 8)).  Inside each 16-dim step the fragment columns are
        // permuted, 2t (+1) <-> dim 16kk + 4t (+1) and 2t + 8 (+9) <->
        // 16kk + 4t + 2 (+3), on both operands: one 32-bit load gives a
        // lane's four key bytes of token g, one 64-bit load its four query
        // dims of a row.  The scores come out in the usual layout.
        const int g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int kk = kk0; kk < kk1; ++kk) {
            uint32_t qa[4];
            lds64(qrow_addr_base + swz(g, 2 * kk + (t >> 1), q_rows<D>()) + 8 * (t & 1), qa[0], qa[2]);
            lds64(qrow_addr_base + swz(g + 8, 2 * kk + (t >> 1), q_rows<D>()) + 8 * (t & 1), qa[1], qa[3]);
#pragma unroll
            for (int j = 0; j < NT / 8; ++j) {
                const int row = tok0 + 8 * j + g;
                const uint32_t wd = lds32(kt + row * 128 + ((kk ^ (row & 7)) << 4) + 4 * t);
                mma16816(sacc[j], qa, f16x2_from_e4m3x2(wd & 0xffffu), f16x2_from_e4m3x2(wd >> 16));
            }
        }
        return;
    }
#pragma unroll
    for (int kk = kk0; kk < kk1; ++kk) {
        uint32_t qa[4];
        {
            const int qr = (lane & 15), qc = 2 * kk + (lane >> 4);
            ldsm_x4(qrow_addr_base + swz(qr, qc, q_rows<D>()), qa[0], qa[1], qa[2], qa[3]);
        }
#pragma unroll
        for (int np = 0; np < NT / 16; ++np) {
            const int tok = tok0 + np * 16 + (lane & 7) + ((lane >> 4) << 3);
            const int kc = 2 * kk + ((lane >> 3) & 1);
            uint32_t b0, b1, b2, b3;
            ldsm_x4(kt + swz(tok, kc, C), b0, b1, b2, b3);
            mma16816(sacc[2 * np], qa, b0, b1);
            mma16816(sacc[2 * np + 1], qa, b2, b3);
        }
    }
}

// Online softmax of a scored 16-row block (log2 units; columns past ntok,
// and under the causal mask past each row's limit, are masked), then
// O += P V for the OD output dims [16 dp0, 16 dp0 + OD).
template <int C, int NT, int OD, bool F8 = false>
__device__ __forceinline__ void cf_softmax_pv(uint32_t vt, int ntok, int tok0, int ctx0, int lim0, int lim1,
                                              float scale_log2, float (&sacc)[NT / 8][4], int dp0,
                                              float (&m)[2], float (&s)[2], float (&o)[OD / 8][4], int lane) {
    float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int nt = 0; nt < NT / 8; ++nt) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int col = tok0 + nt * 8 + 2 * (lane & 3) + (e & 1);
            // a column counts if it holds a token and, under the causal
            // mask, that token is at or before the row's limit
            const bool ok = col < ntok && ctx0 + col <= ((e >> 1) ? lim1 : lim0);
            const float x = ok ? sacc[nt][e] * scale_log2 : -INFINITY;
            sacc[nt][e] = x;
            mx[e >> 1] = fmaxf(mx[e >> 1], x);
        }
    }
    // The row's reference maximum m is raised lazily: only when the chunk's
    // maximum exceeds it by more than 2^8 (P then stays below 256, exact in
    // fp16), so most chunks leave O unscaled; o and s always refer to the
    // same m, which the partial carries.
    float alpha[2], mu[2];
    bool grow = false;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        mx[r] = fmaxf(mx[r], __shfl_xor_sync(kFull, mx[r], 1));
        mx[r] = fmaxf(mx[r], __shfl_xor_sync(kFull, mx[r], 2));
        alpha[r] = 1.f;
        if (mx[r] > m[r] + 8.f) {                   // also the first finite maximum
            alpha[r] = ex2(m[r] - mx[r]);           // 0 while m is -inf
            m[r] = mx[r];
            s[r] *= alpha[r];
            grow = true;
        }
        mu[r] = (m[r] == -INFINITY) ? 0.f : m[r];
    }
    uint32_t pa[NT / 16][4];
#pragma unroll
    for (int nt = 0; nt < NT / 8; ++nt) {
        const float p0 = ex2(sacc[nt][0] - mu[0]), p1 = ex2(sacc[nt][1] - mu[0]);
        const float p2 = ex2(sacc[nt][2] - mu[1]), p3 = ex2(sacc[nt][3] - mu[1]);
        s[0] += p0 + p1;
        s[1] += p2 + p3;
        // accumulator layout of n-tile nt == A-operand layout of k-step nt/2
        pa[nt >> 1][(nt & 1) * 2 + 0] = pack_half2(p0, p1);
        pa[nt >> 1][(nt & 1) * 2 + 1] = pack_half2(p2, p3);
    }
    if (__any_sync(kFull, grow)) {
#pragma unroll
        for (int dt = 0; dt < OD / 8; ++dt) {
            o[dt][0] *= alpha[0]; o[dt][1] *= alpha[0];
            o[dt][2] *= alpha[1]; o[dt][3] *= alpha[1];
        }
    }
    if constexpr (F8) {
        // E4M3 values: n-tile 4dq + i holds output dims 32dq + 4n + i
        // (n = the fragment column), so a lane's B operand for dims
        // 32dq + 4g .. + 3 of its four tokens (16j + 2t, + 1, + 8, + 9) is
        // four 32-bit loads paired per dim by byte permutes.  The
        // accumulator of lane (g, t) then holds dims 32dq + 8t .. + 7 of its
        // rows: o[4dq + i][c] <-> dim 32dq + 8t + 4c' + i (c' = c % 2).
        static_assert(OD == 128, "fp8 pools have head_dim 128");
        const int g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int j = 0; j < NT / 16; ++j) {
            const int r0 = tok0 + 16 * j + 2 * t;
#pragma unroll
            for (int dq = 0; dq < 4; ++dq) {
                const int kc = 2 * dq + (g >> 2);
                const uint32_t off = 4 * (g & 3);
                const uint32_t wa = lds32(vt + r0 * 128 + ((kc ^ (r0 & 7)) << 4) + off);
                const uint32_t wb = lds32(vt + (r0 + 1) * 128 + ((kc ^ ((r0 + 1) & 7)) << 4) + off);
                const uint32_t wc = lds32(vt + (r0 + 8) * 128 + ((kc ^ (r0 & 7)) << 4) + off);
                const uint32_t wd = lds32(vt + (r0 + 9) * 128 + ((kc ^ ((r0 + 1) & 7)) << 4) + off);
                const uint32_t x01 = __byte_perm(wa, wb, 0x5140), x23 = __byte_perm(wa, wb, 0x7362);
                const uint32_t y01 = __byte_perm(wc, wd, 0x5140), y23 = __byte_perm(wc, wd, 0x7362);
                mma16816(o[4 * dq + 0], pa[j], f16x2_from_e4m3x2(x01 & 0xffffu), f16x2_from_e4m3x2(y01 & 0xffffu));
                mma16816(o[4 * dq + 1], pa[j], f16x2_from_e4m3x2(x01 >> 16), f16x2_from_e4m3x2(y01 >> 16));
                mma16816(o[4 * dq + 2], pa[j], f16x2_from_e4m3x2(x23 & 0xffffu), f16x2_from_e4m3x2(y23 & 0xffffu));
                mma16816(o[4 * dq + 3], pa[j], f16x2_from_e4m3x2(x23 >> 16), f16x2_from_e4m3x2(y23 >> 16));
            }
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < NT / 16; ++j) {
#pragma unroll
        for (int dq = 0; dq < OD / 16; ++dq) {
            const int tok = tok0 + 16 * j + (lane & 7) + (((lane >> 3) & 1) << 3);
            const int kc = 2 * (dp0 + dq) + (lane >> 4);
            uint32_t b0, b1, b2, b3;
            ldsm_x4_t(vt + swz(tok, kc, C), b0, b1, b2, b3);
            mma16816(o[2 * dq], pa[j], b0, b1);
            mma16816(o[2 * dq + 1], pa[j], b2, b3);
        }
    }
}

// One warp, one 16-row block, NT tokens, every head dim.
// F8: K and V are the stage's E4M3 bytes (head_dim 128), and o comes out
// with its dims permuted as cf_softmax_pv describes.
template <int C, int D, int NT, bool F8 = false>
__device__ __forceinline__ void cf_chunk(uint32_t kt, uint32_t vt, int ntok, int tok0, int ctx0, int lim0,
                                         int lim1, uint32_t qrow_addr_base, float scale_log2,
                                         float (&m)[2], float (&s)[2], float (&o)[D / 8][4], int lane) {
    float sacc[NT / 8][4];
    cf_scores<C, D, NT, F8>(kt, tok0, qrow_addr_base, 0, D / 16, sacc, lane);
    cf_softmax_pv<C, NT, D, F8>(vt, ntok, tok0, ctx0, lim0, lim1, scale_log2, sacc, 0, m, s, o, lane);
}

}  // namespace dev
}  // namespace ca
