// A decode step's attention weights, added to running sums per token:
//     out[i][h][t] = in[i][h][t] + sum over the rows r of sequence i and
//     key/value head h of  exp(x_rt) / sum_t' exp(x_rt'),  x_rt = scale q_r . k_t.
// Keys alone are read, once for all sharers of a chunk: the first kernel walks
// the two-phase plan of the schedule (units of shared chunks against the
// queries of all their sharers, then each sequence's own chunks) and leaves the
// scores, fp32 in log2 units, and each unit's (maximum, sum) of each row; the
// second joins those per row and adds the weights up.
//
// Bound by DRAM where contexts have nothing in common (eight of 128 K tokens, 4
// rows a key/value head: 345 us for 2.28 GB, 97% of the copy rate, then 37 us for
// the sums).  Shorter stretches of single rows are bound by the first kernel's
// latency: 64 sequences of 4096 shared and 512 own tokens 65 us for 309 MB (two
// CTAs an SM, eight warps; a stage of 64 tokens takes one 1100 clocks), 22 us for the
// sums.  Stages of 128 tokens leave one CTA an SM (128 us in all instead of 87).
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>

#include "ca_internal.h"
#include "fp4.cuh"
#include "row_blocks.cuh"

namespace ca {
namespace dev {

constexpr int kWtWarps = 4, kWtThreads = 32 * (kWtWarps + 1);
constexpr int kWtTokens = 64;             // tokens of a stage: 16 a warp
constexpr int kAddThreads = 128, kAddPer = 2, kAddTokens = 4 * kAddPer * kAddThreads;

struct WeightParams {
    AttnParams a;                 // the schedule's plan, the pool, q (part_ms: the units' (m, s))
    const int32_t* tok_base;      // [b + 1] chunks of the positions before each one
    float* scores;                // position by position: [Hkv][rows][its chunks' tokens]
    const float* in;
    float* out;
    int32_t room;                 // tokens per row of in and out
    int32_t chunk;
    int32_t blocks, block_tokens; // second kernel: blocks per row, tokens of each
};

template <int C, int D, int EB>
struct WtSmem {
    static constexpr int kPer = kWtTokens / C;            // chunk tiles of a stage
    static constexpr int kTile = EB == 0 ? F4Tile<C, D>::kBytes : C * D * EB;
    static constexpr int kStage = kPer * kTile;
    static constexpr int kStages = EB == 2 && D == 256 ? 4 : EB == 2 && D == 128 ? 5 : 8;   // two CTAs an SM (D 256: one)
    static constexpr int kQ = q_rows<D>() * D * 2;
    static constexpr int kRows = kStages * kStage + kQ;              // score rows' addresses, of two pieces
    static constexpr int kMs = kRows + 2 * kQRows * 8;               // (m, s) of each warp's rows
    static constexpr int kInfo = kMs + kWtWarps * kQRows * 8;        // ntok and first token of each chunk tile
    static constexpr int kBars = kInfo + kStages * kPer * 8;
    static constexpr int kBytes = kBars + 2 * kStages * 8;
};

// Fragments for m16n8k16 over the dims [128 part, 128 part + 16 KK): of 16 rows of
// the query tile, and of the keys [tok0, tok0 + 16) of a chunk tile.  All loads of
// a stage go out together: one after the other between the products (8 of them in
// a chain) a stage of 64 tokens took 0.7 us, whatever the memory did.
template <int D, int KK, bool F8>
__device__ __forceinline__ void query_frags(uint32_t rows, int part, uint32_t (&q)[KK][4], int lane) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int k = 0; k < KK; ++k) {
        const int kk = 8 * part + k;
        if constexpr (F8) {               // (dims permuted inside each step, as the keys are below)
            lds64(rows + swz(g, 2 * kk + (t >> 1), q_rows<D>()) + 8 * (t & 1), q[k][0], q[k][2]);
            lds64(rows + swz(g + 8, 2 * kk + (t >> 1), q_rows<D>()) + 8 * (t & 1), q[k][1], q[k][3]);
        } else {
            ldsm_x4(rows + swz(lane & 15, 2 * kk + (lane >> 4), q_rows<D>()), q[k][0], q[k][1], q[k][2], q[k][3]);
        }
    }
}
template <int C, int KK, bool F8>
__device__ __forceinline__ void key_frags(uint32_t tile, int tok0, int part, uint32_t (&b)[KK][4], int lane) {
    const int g = lane >> 2, t = lane & 3;
    if constexpr (F8) {
        // a lane's four bytes of a step, dims 16 kk + 4 t + 0 .. 3: columns 2t, 2t + 1 and 2t + 8, 2t + 9
        uint32_t w[KK][2];
#pragma unroll
        for (int k = 0; k < KK; ++k)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int row = tok0 + 8 * j + g;
                w[k][j] = lds32(tile + row * 128 + (((8 * part + k) ^ (row & 7)) << 4) + 4 * t);
            }
#pragma unroll
        for (int k = 0; k < KK; ++k)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                b[k][2 * j] = f16x2_from_e4m3x2(w[k][j] & 0xffffu);
                b[k][2 * j + 1] = f16x2_from_e4m3x2(w[k][j] >> 16);
            }
    } else {
#pragma unroll
        for (int k = 0; k < KK; ++k)
            ldsm_x4(tile + swz(tok0 + (lane & 7) + ((lane >> 4) << 3), 2 * (8 * part + k) + ((lane >> 3) & 1), C), b[k][0], b[k][1],
                    b[k][2], b[k][3]);
    }
}

__device__ __forceinline__ void wt_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kWtWarps * 32) : "memory"); }

// One head's stretch of a unit: its chunks are chunk base + L % n for L in
// [begin, end).
struct Piece {
    int head, begin, end, n, base, part, q_lo, positions;
};
// The pieces of a CTA's units: its static ones, then every grid-th of the tail.
struct PieceWalk {
    const AttnParams& p;
    int u, u_end, tail;
    Unit U;
    int L, L1, n;
    __device__ __forceinline__ explicit PieceWalk(const AttnParams& p_) : p(p_), tail(p_.dyn_begin + blockIdx.x), L(0), L1(0), n(1) {
        const int2 range = *reinterpret_cast<const int2*>(p.cta_head + blockIdx.x);
        u = range.x;
        u_end = range.y;
    }
    __device__ __forceinline__ bool next(Piece& x) {
        while (L >= L1) {
            int at;
            if (u < u_end) at = u++;
            else if (tail < p.dyn_end) {
                at = tail;
                tail += gridDim.x;
            } else return false;
            U = p.units[at];
            const bool sf = U.kind == UNIT_SF;
            n = sf ? U.n_per_head : U.c_end - U.c_begin;
            L = sf ? U.c_begin : U.head * n;
            L1 = sf ? U.c_end : (U.head + U.n_per_head) * n;
            first = true;
        }
        const bool sf = U.kind == UNIT_SF;
        x.head = L / n;
        x.begin = L;
        x.end = L = min(L1, (x.head + 1) * n);
        x.n = n;
        x.base = sf ? U.base : U.c_begin;
        x.part = first || !sf ? U.part : U.part_next;
        x.q_lo = U.q_lo;
        x.positions = U.q_hi - U.q_lo;
        first = false;
        return true;
    }
    bool first = true;
};

// Rows of the query tile are (position, query token, query head) as in the
// two-phase kernel; a warp takes 16 tokens of a stage against every 16 of them.  A
// thread keeps the running maximum and sum of its own columns of each of its
// rows; they meet at the end of a piece.  Pieces of at most half the tile's rows
// use its halves in turn, so that the next one's queries come meanwhile.
template <int C, int D, int EB>
__global__ void __launch_bounds__(kWtThreads, D == 256 ? 1 : 2) weight_scores_kernel(const __grid_constant__ CUtensorMap tmap,
                                                                   const WeightParams wp) {
    using SM = WtSmem<C, D, EB>;
    constexpr int kPer = SM::kPer, kN = SM::kStages;
    extern __shared__ __align__(1024) uint8_t smem[];
    const AttnParams& p = wp.a;
    uint8_t* qt = smem + kN * SM::kStage;
    float** row_at = reinterpret_cast<float**>(smem + SM::kRows);
    float2* ms = reinterpret_cast<float2*>(smem + SM::kMs);
    volatile int2* info = reinterpret_cast<volatile int2*>(smem + SM::kInfo);
    const uint32_t full0 = smem_u32(smem + SM::kBars), empty0 = full0 + 8 * kN;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (threadIdx.x == 0) {
        for (int i = 0; i < kN; ++i) {
            mbar_init(full0 + 8 * i, 1);
            mbar_init(empty0 + 8 * i, kWtWarps);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    __syncthreads();
    const int HK = p.n_kv_heads, G = p.group, QL = p.q_len, RW = QL * G, H = p.n_heads;
    // the plan may be read before the dependency wait; q and the pool after it
    PieceWalk walk(p);
    Piece cur, nxt;
    bool have = walk.next(cur);
    asm volatile("griddepcontrol.wait;" ::: "memory");

    if (warp == kWtWarps) {
        // ------------------------------ producer ------------------------------
        // A lane per chunk, 32 chunks of a head at a time: slots, token counts and
        // offsets of all of them come in one round trip (chunk after chunk, each
        // stage waited for two dependent loads: 391 us where these take 341 for
        // eight contexts of 128 K tokens).
        if (p.test_stall) {               // test hook: a wait that nothing ends
            if (lane == 0 && !mbar_wait(full0, 0u)) set_status(p.status, CA_ERR_TIMEOUT);
            return;
        }
        const uint64_t pol = policy_evict_first();
        constexpr uint32_t kCopy = EB == 0 ? C * D / 2 + C * D / 16 : C * D * EB;
        struct Refs { int slot, ntok, tok0; };
        auto fetch = [&](const Piece& x, int L) {
            Refs r{-1, 0, 0};
            if (L + lane < x.end) {
                const int at = x.base + (L + lane) % x.n;
                r.slot = p.chunks[at].slot;
                r.tok0 = p.chunk_tok0[at];
                if (r.slot < 0 || r.slot >= p.capacity || x.head >= HK) {
                    set_status(p.status, CA_ERR_DEVICE_BOUNDS);
                    r.slot = -1;
                }
                if (r.slot >= 0) r.ntok = min(max(p.slot_ntok[r.slot], 0), C);
            }
            return r;
        };
        int it = 0;
        bool ok = true;
        Refs next{-1, 0, 0};
        if (have) next = fetch(cur, cur.begin);
        while (have && ok) {
            const bool more = walk.next(nxt);
            for (int L = cur.begin; L < cur.end && ok; L += 32) {
                const int batch = min(32, cur.end - L);
                const Refs r = next;
                if (L + 32 < cur.end) next = fetch(cur, L + 32);
                else if (more) next = fetch(nxt, nxt.begin);
                for (int x0 = 0; x0 < batch; x0 += kPer, ++it) {   // (32 is a multiple of kPer)
                    const int st = it % kN;
                    const uint32_t fb = full0 + 8 * st;
                    if (!__all_sync(kFull, mbar_wait(empty0 + 8 * st, ((uint32_t)(it / kN) & 1u) ^ 1u))) {
                        if (lane == 0) set_status(p.status, CA_ERR_TIMEOUT);
                        ok = false;
                        break;
                    }
                    const int x = lane - x0;
                    const bool mine = x >= 0 && x < kPer && lane < batch, there = mine && r.slot >= 0;
                    const uint32_t copies = __popc(__ballot_sync(kFull, there));
                    if (lane == 0 && copies) mbar_expect_tx_only(fb, copies * kCopy);
                    if (mine) {
                        info[st * kPer + x].x = r.ntok;
                        info[st * kPer + x].y = r.tok0;
                    }
                    __syncwarp();
                    if (there) {
                        const uint32_t dst = smem_u32(smem + st * SM::kStage + x * SM::kTile);
                        if constexpr (EB == 0) {
                            using T = F4Tile<C, D>;
                            const uint8_t* src =
                                p.kv + (((long long)r.slot * p.n_layers + p.layer) * HK + cur.head) * T::kBytes;
                            bulk_load(dst, src, T::kCodes, fb, pol);
                            bulk_load(dst + T::kKScales, src + T::kKScales, T::kScales, fb, pol);
                        } else {
                            const int row = ((r.slot * p.n_layers + p.layer) * 2 * HK + cur.head) * C;
#pragma unroll
                            for (int bx = 0; bx < D * EB / 128; ++bx)
                                tma_load_2d(dst + bx * C * 128, &tmap, bx * (128 / (EB == 0 ? 1 : EB)), row, fb, pol);
                        }
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(fb);
                }
            }
            cur = nxt;
            have = more;
        }
        if (!ok)                          // let the copies in flight land before the CTA can end
            for (int k = max(0, it - kN); k < it; ++k) mbar_wait(full0 + 8 * (k % kN), (uint32_t)(k / kN) & 1u);
        return;
    }

    // ------------------------------ consumers --------------------------------
    constexpr int RS = EB == 0 ? 4 : 2;               // rows of a 16-row block that a thread holds columns of
    constexpr int RB = q_rows<D>() / 16;
    const int g = lane >> 2, t = lane & 3;
    const int sub = warp * 16 / C, tok0 = warp * 16 % C;
    auto row_of = [&](int rb, int k) { return rb * 16 + (EB == 0 ? (k >> 1) * 8 + 2 * t + (k & 1) : g + 8 * k); };
    // a piece's queries into the tile from row `at` on, and where its rows' scores go
    auto fetch_queries = [&](const Piece& x, int at, int which) {
        const int rows = x.positions * RW;
        for (int i = threadIdx.x; i < rows * (D / 8); i += kWtWarps * 32) {
            const int r = i / (D / 8), k = i % (D / 8);
            const size_t tok = (size_t)p.seq_perm[x.q_lo + r / RW] * QL + (r % RW) / G;
            cp_async16(smem_u32(qt + swz(at + r, k, q_rows<D>())), p.q + (tok * H + x.head * G + r % G) * D + k * 8);
        }
        for (int r = threadIdx.x; r < rows; r += kWtWarps * 32) {
            const int pos = x.q_lo + r / RW;
            const long long c0 = wp.tok_base[pos], tokens = (wp.tok_base[pos + 1] - c0) * C;
            row_at[which * kQRows + r] = wp.scores + c0 * C * ((long long)QL * H) + (long long)(x.head * RW + r % RW) * tokens;
        }
    };
    constexpr int kHalf = q_rows<D>() / 2;
    int it = 0, which = 0;
    bool ok = true, fetched = false;                  // (a warp whose wait ran out still meets the others at their barriers)
    for (; have; cur = nxt, which ^= 1) {
        const bool more = walk.next(nxt);
        const int head = cur.head, part = cur.part, m_rows = cur.positions * RW;
        const int at = m_rows <= kHalf ? which * kHalf : 0;
        if (!fetched) fetch_queries(cur, at, which);
        cp_async_wait_all();
        wt_sync();
        fetched = more && m_rows <= kHalf && nxt.positions * RW <= kHalf;
        if (fetched) fetch_queries(nxt, (which ^ 1) * kHalf, which ^ 1);
        have = more;
        int lim[RB][RS];                              // causal mask: the last token that a row sees
#pragma unroll
        for (int rb = 0; rb < RB; ++rb)
#pragma unroll
            for (int k = 0; k < RS; ++k) {
                const int row = row_of(rb, k);
                lim[rb][k] = p.causal && row < m_rows ? p.ctx_len[cur.q_lo + row / RW] - QL + (row % RW) / G : INT_MAX;
            }
        // (up to 16 rows: their fragments stay in registers for the whole piece)
        constexpr bool kKeep = EB != 0 && D <= 128;
        uint32_t qf[EB == 0 ? 1 : D / 16 < 8 ? D / 16 : 8][4];
        if constexpr (kKeep)
            if (m_rows <= 16) query_frags<D, D / 16 < 8 ? D / 16 : 8, EB == 1>(smem_u32(qt) + at * 128, 0, qf, lane);
        float m[RB][RS], s[RB][RS];
#pragma unroll
        for (int rb = 0; rb < RB; ++rb)
#pragma unroll
            for (int k = 0; k < RS; ++k) {
                m[rb][k] = -INFINITY;
                s[rb][k] = 0.f;
            }
        for (int L = cur.begin; L < cur.end; ++it) {
            const int st = it % kN, cnt = min(kPer, cur.end - L);
            if (ok && !mbar_wait(full0 + 8 * st, (uint32_t)(it / kN) & 1u)) {
                set_status(p.status, CA_ERR_TIMEOUT);
                ok = false;
            }
            ok = __all_sync(kFull, ok);
            L += cnt;
            if (!ok) continue;
            if (sub < cnt) {
                const uint8_t* tile = smem + st * SM::kStage + sub * SM::kTile;
                const int ntok = info[st * kPer + sub].x, ctx0 = info[st * kPer + sub].y;
                constexpr int KK = D / 16 < 8 ? D / 16 : 8;
                uint32_t kf[EB == 0 ? 1 : KK][4];
                if constexpr (EB != 0 && D <= 128) key_frags<C, KK, EB == 1>(smem_u32(tile), tok0, 0, kf, lane);
#pragma unroll
                for (int rb = 0; rb < RB; ++rb) {
                    if (rb * 16 >= m_rows) break;
                    float acc[2][4];
                    if constexpr (EB == 0) {
                        uint32_t qb[2][D / 16][2];
#pragma unroll
                        for (int nb = 0; nb < 2; ++nb)
#pragma unroll
                            for (int kk = 0; kk < D / 16; ++kk)
                                lds64(smem_u32(qt) + swz(at + rb * 16 + nb * 8 + g, 2 * kk + (t >> 1), q_rows<D>()) + 8 * (t & 1),
                                      qb[nb][kk][0], qb[nb][kk][1]);
                        f4_scores<C, D, 2, false>(tile, tok0 / 16, qb, acc, lane);
                    } else {
#pragma unroll
                        for (int j = 0; j < 8; ++j) acc[j >> 2][j & 3] = 0.f;
#pragma unroll
                        for (int part = 0; part < D / 16 / KK; ++part) {
                            if constexpr (D > 128) key_frags<C, KK, EB == 1>(smem_u32(tile), tok0, part, kf, lane);
                            if (!kKeep || m_rows > 16) query_frags<D, KK, EB == 1>(smem_u32(qt) + (at + rb * 16) * 128, part, qf, lane);
#pragma unroll
                            for (int k = 0; k < KK; ++k) {
                                mma16816(acc[0], qf[k], kf[k][0], kf[k][1]);
                                mma16816(acc[1], qf[k], kf[k][2], kf[k][3]);
                            }
                        }
                    }
#pragma unroll
                    for (int k = 0; k < RS; ++k) {
                        const int row = row_of(rb, k);
                        if (row >= m_rows) continue;
                        // this thread's columns of the row, in the order of x
                        constexpr int N = 8 / RS;
                        float x[N], top = m[rb][k];
#pragma unroll
                        for (int j = 0; j < N; ++j) {
                            const int col = tok0 + (EB == 0 ? f4_token(g) + 8 * j : (j >> 1) * 8 + 2 * t + (j & 1));
                            const float v = (EB == 0 ? acc[k >> 1][2 * j + (k & 1)] : acc[j >> 1][2 * k + (j & 1)]) * p.scale_log2;
                            x[j] = col < ntok && ctx0 + col <= lim[rb][k] ? v : -INFINITY;
                            top = fmaxf(top, x[j]);
                        }
                        const float mu = top == -INFINITY ? 0.f : top;
                        float sum = s[rb][k] * ex2(m[rb][k] - mu);
#pragma unroll
                        for (int j = 0; j < N; ++j) sum += ex2(x[j] - mu);
                        m[rb][k] = top;
                        s[rb][k] = sum;
                        float* dst = row_at[which * kQRows + row] + ctx0 + tok0;
                        if constexpr (EB == 0) {
                            dst[f4_token(g)] = x[0];
                            dst[f4_token(g) + 8] = x[1];
                        } else {
                            *reinterpret_cast<float2*>(dst + 2 * t) = make_float2(x[0], x[1]);
                            *reinterpret_cast<float2*>(dst + 8 + 2 * t) = make_float2(x[2], x[3]);
                        }
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(empty0 + 8 * st);
        }
        // the row's columns of the other lanes, then of the other warps
#pragma unroll
        for (int rb = 0; rb < RB; ++rb)
#pragma unroll
            for (int k = 0; k < RS; ++k) {
                float mk = m[rb][k], sk = s[rb][k];
#pragma unroll
                for (int off = EB == 0 ? 4 : 1; off <= (EB == 0 ? 16 : 2); off <<= 1) {
                    const float m2 = __shfl_xor_sync(kFull, mk, off), s2 = __shfl_xor_sync(kFull, sk, off);
                    const float M = fmaxf(mk, m2), mu = M == -INFINITY ? 0.f : M;
                    sk = sk * ex2(mk - mu) + s2 * ex2(m2 - mu);
                    mk = M;
                }
                const int row = row_of(rb, k);
                if (row < m_rows && (EB == 0 ? g : t) == 0) ms[warp * kQRows + row] = make_float2(mk, sk);
            }
        wt_sync();
        for (int row = threadIdx.x; row < m_rows; row += kWtWarps * 32) {
            float M = -INFINITY, S = 0.f;
#pragma unroll
            for (int w = 0; w < kWtWarps; ++w) M = fmaxf(M, ms[w * kQRows + row].x);
            const float mu = M == -INFINITY ? 0.f : M;
#pragma unroll
            for (int w = 0; w < kWtWarps; ++w) S += ms[w * kQRows + row].y * ex2(ms[w * kQRows + row].x - mu);
            const int pos = cur.q_lo + row / RW, jq = (row % RW) / G;
            p.part_ms[p.pbase[((size_t)pos * QL + jq) * H + head * G + row % G] + part] = make_float2(M, S);
        }
    }
}

// Joins the units' (m, s) of each row of a position and head, then adds the
// rows' weights.  A thread has four tokens of each kAddPer-th part of the block's
// range; a row's scores and the sums are on their way before the join is through.
__global__ void __launch_bounds__(kAddThreads) add_weights_kernel(const WeightParams wp) {
    __shared__ float lse[kQRows];                     // log2 of each row's sum
    const AttnParams& p = wp.a;
    const int blk = blockIdx.x % wp.blocks, pair = blockIdx.x / wp.blocks;
    const int pos = pair / p.n_kv_heads, h = pair % p.n_kv_heads;
    const int G = p.group, QL = p.q_len, RW = QL * G, H = p.n_heads;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long c0 = wp.tok_base[pos], tokens = (wp.tok_base[pos + 1] - c0) * wp.chunk;
    const bool apart = wp.in != wp.out;
    const long long last = apart ? max(tokens, (long long)wp.room) : tokens;
    const size_t row = ((size_t)p.seq_perm[pos] * p.n_kv_heads + h) * wp.room;
    const float* scores = wp.scores + c0 * wp.chunk * ((long long)QL * H) + (long long)h * RW * tokens;
    auto token = [&](int k) { return blk * wp.block_tokens + k * (4 * kAddThreads) + 4 * (int)threadIdx.x; };
    // this warp's first row's partials: on their way with all the rest (the plan may
    // be read before the dependency wait)
    auto row_id = [&](int r) { return ((size_t)pos * QL + r / G) * H + h * G + r % G; };
    const int part0 = warp < RW ? p.pbase[row_id(warp)] : 0, part1 = warp < RW ? p.pbase[row_id(warp) + 1] : 0;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const long long end = min(last, (long long)(blk + 1) * wp.block_tokens);    // of this block
    if ((long long)blk * wp.block_tokens >= last) return;
    const bool wide = (wp.room & 3) == 0 && ((reinterpret_cast<uintptr_t>(wp.in) | reinterpret_cast<uintptr_t>(wp.out)) & 15u) == 0;
    float4 x[kAddPer], sum[kAddPer];
    auto load_row = [&](int r) {
#pragma unroll
        for (int k = 0; k < kAddPer; ++k)             // (a position's tokens are a multiple of 16)
            x[k] = token(k) < min(tokens, end) ? __ldcg(reinterpret_cast<const float4*>(scores + r * tokens + token(k)))
                                     : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
    };
    load_row(0);
#pragma unroll
    for (int k = 0; k < kAddPer; ++k) {
        const int t = token(k);
        sum[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (t >= end) continue;
        if (wide) {
            if (t < wp.room) sum[k] = *reinterpret_cast<const float4*>(wp.in + row + t);
        } else {
            if (t < wp.room) sum[k].x = wp.in[row + t];
            if (t + 1 < wp.room) sum[k].y = wp.in[row + t + 1];
            if (t + 2 < wp.room) sum[k].z = wp.in[row + t + 2];
            if (t + 3 < wp.room) sum[k].w = wp.in[row + t + 3];
        }
    }
    for (int r = warp; r < RW; r += kAddThreads / 32) {
        const int a = r == warp ? part0 : p.pbase[row_id(r)], n = (r == warp ? part1 : p.pbase[row_id(r) + 1]) - a;
        float M = -INFINITY, S = 0.f;
        for (int j = lane; j < n; j += 32) {
            const float2 v = __ldcg(&p.part_ms[a + j]);
            const float top = fmaxf(M, v.x), mu = top == -INFINITY ? 0.f : top;
            S = S * ex2(M - mu) + v.y * ex2(v.x - mu);
            M = top;
        }
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) {
            const float m2 = __shfl_xor_sync(kFull, M, off), s2 = __shfl_xor_sync(kFull, S, off);
            const float top = fmaxf(M, m2), mu = top == -INFINITY ? 0.f : top;
            // (the same order in both lanes, so that they agree)
            const float a1 = S * ex2(M - mu), a2 = s2 * ex2(m2 - mu);
            S = (lane & off) ? a2 + a1 : a1 + a2;
            M = top;
        }
        if (lane == 0) lse[r] = S > 0.f || S != S ? M + log2f(S) : INFINITY;   // (a row that sees nothing weighs nothing)
    }
    __syncthreads();
    // a context that has outgrown its row
    bool over = false;
#pragma unroll
    for (int k = 0; k < kAddPer; ++k) {
        const int t = token(k);
        over |= (t >= wp.room && x[k].x != -INFINITY) || (t + 1 >= wp.room && x[k].y != -INFINITY) ||
                (t + 2 >= wp.room && x[k].z != -INFINITY) || (t + 3 >= wp.room && x[k].w != -INFINITY);
    }
    if (over) set_status(p.status, CA_ERR_DEVICE_BOUNDS);
    float4 w[kAddPer];
#pragma unroll
    for (int k = 0; k < kAddPer; ++k) w[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    // (not earlier: the next kernel's CTAs would take this one's registers while
    // they wait, 64 sequences back to back 111 us)
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // (a token that a row does not see, or past the context, gets nothing of it even
    // where the row's sum is not a number)
    auto weight = [](float x, float l) { return x == -INFINITY ? 0.f : ex2(x - l); };
    for (int r = 0; r < RW; ++r) {
        const float l = lse[r];
        float4 y[kAddPer];
#pragma unroll
        for (int k = 0; k < kAddPer; ++k) y[k] = x[k];
        if (r + 1 < RW) load_row(r + 1);
#pragma unroll
        for (int k = 0; k < kAddPer; ++k) {
            w[k].x += weight(y[k].x, l);
            w[k].y += weight(y[k].y, l);
            w[k].z += weight(y[k].z, l);
            w[k].w += weight(y[k].w, l);
        }
    }
    // (a weight of 0 leaves the bits of the sum: past the context they are the caller's)
    auto add = [](float s, float x) { return x == 0.f ? s : s + x; };
#pragma unroll
    for (int k = 0; k < kAddPer; ++k) {
        const int t = token(k);
        if (t >= end) continue;
        const float4 v = make_float4(add(sum[k].x, w[k].x), add(sum[k].y, w[k].y), add(sum[k].z, w[k].z), add(sum[k].w, w[k].w));
        if (wide) {
            if (t < wp.room) *reinterpret_cast<float4*>(wp.out + row + t) = v;
        } else {
            if (t < wp.room) wp.out[row + t] = v.x;
            if (t + 1 < wp.room) wp.out[row + t + 1] = v.y;
            if (t + 2 < wp.room) wp.out[row + t + 2] = v.z;
            if (t + 3 < wp.room) wp.out[row + t + 3] = v.w;
        }
    }
}

}  // namespace dev

namespace {

template <int C, int D, int EB>
int run_scores(const CUtensorMap* map, const dev::WeightParams& w, unsigned grid, cudaLaunchAttribute* attr, cudaStream_t s) {
    constexpr int bytes = dev::WtSmem<C, D, EB>::kBytes;
    if (cudaFuncSetAttribute(dev::weight_scores_kernel<C, D, EB>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
        return CA_ERR_CUDA;
    cudaLaunchConfig_t c = {};
    c.gridDim = dim3(grid);
    c.blockDim = dim3(dev::kWtThreads);
    c.dynamicSmemBytes = bytes;
    c.stream = s;
    c.attrs = attr;
    c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, dev::weight_scores_kernel<C, D, EB>, *map, w) == cudaSuccess ? CA_OK : CA_ERR_CUDA;
}

template <int D, int EB>
int pick_scores(int chunk, const CUtensorMap* map, const dev::WeightParams& w, unsigned grid, cudaLaunchAttribute* attr,
                cudaStream_t s) {
    if (chunk == 16) return run_scores<16, D, EB>(map, w, grid, attr, s);
    if (chunk == 32) return run_scores<32, D, EB>(map, w, grid, attr, s);
    if constexpr (D <= 128)
        if (chunk == 64) return run_scores<64, D, EB>(map, w, grid, attr, s);
    return CA_ERR_UNSUPPORTED;
}

}  // namespace

int launch_weights(const Pool& p, const Sched& s, int32_t layer, const void* q, const float* in, float* out, int32_t room,
                   float scale, void* ws, void* stream) {
    const PoolCfg& c = p.cfg;
    unsigned char* w8 = static_cast<unsigned char*>(ws);
    dev::WeightParams w{};
    w.a = attn_params(p, s, layer, q, nullptr, scale, ws);
    w.a.part_o = nullptr;
    w.a.part_ms = reinterpret_cast<float2*>(w8 + s.ws.weights_ms);
    w.tok_base = reinterpret_cast<const int32_t*>(static_cast<unsigned char*>(s.dev) + s.layout.tok_base);
    w.scores = reinterpret_cast<float*>(w8 + s.ws.weights_scores);
    w.in = in;
    w.out = out;
    w.room = room;
    w.chunk = c.chunk;
    int64_t most = in == out ? 0 : room;
    for (int32_t pos = 0; pos < s.t.b; ++pos)
        most = std::max<int64_t>(most, (int64_t)(s.t.tok_base[pos + 1] - s.t.tok_base[pos]) * c.chunk);
    // blocks of about equal length, whole rounds of the threads
    constexpr int64_t round = 4 * dev::kAddThreads;
    w.blocks = (int32_t)((most + dev::kAddTokens - 1) / dev::kAddTokens);
    w.block_tokens = (int32_t)(((most + w.blocks - 1) / w.blocks + round - 1) / round * round);
    const int64_t adds = (int64_t)w.blocks * s.t.b * kv_heads(c);
    if (adds > INT32_MAX) return CA_ERR_UNSUPPORTED;
    w.a.test_stall = 0;
    if (s.stall_calls > 0) {
        w.a.test_stall = 1;
        --s.stall_calls;
    }
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    // Both are programmatic dependents of what precedes them in the stream.
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    const CUtensorMap* map = reinterpret_cast<const CUtensorMap*>(p.tmap);
    const unsigned grid = (unsigned)s.plan.grid;
    int st = CA_ERR_UNSUPPORTED;
    if (c.flags & CA_KV_FP4) {
        if (c.head_dim == 64) st = pick_scores<64, 0>(c.chunk, map, w, grid, attr, cs);
        else if (c.head_dim == 128) st = pick_scores<128, 0>(c.chunk, map, w, grid, attr, cs);
    } else if (c.flags & CA_KV_FP8) {
        if (c.head_dim == 128) st = pick_scores<128, 1>(c.chunk, map, w, grid, attr, cs);
    } else {
        if (c.head_dim == 64) st = pick_scores<64, 2>(c.chunk, map, w, grid, attr, cs);
        else if (c.head_dim == 128) st = pick_scores<128, 2>(c.chunk, map, w, grid, attr, cs);
        else if (c.head_dim == 256) st = pick_scores<256, 2>(c.chunk, map, w, grid, attr, cs);
    }
    if (st) return st;
    count_launch();
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3((unsigned)adds);
    lc.blockDim = dim3(dev::kAddThreads);
    lc.stream = cs;
    lc.attrs = attr;
    lc.numAttrs = 1;
    if (cudaLaunchKernelEx(&lc, dev::add_weights_kernel, w) != cudaSuccess) return CA_ERR_CUDA;
    count_launch();
    return CA_OK;
}

}  // namespace ca
