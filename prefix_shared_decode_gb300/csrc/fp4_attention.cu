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
//    own 16 tokens of a tile and nothing is exchanged until the head ends.
//  * Units of more rows: the warps widen the tile once into fp16 tiles in
//    shared memory, 32 tokens at a time, and take a 16-row block each (with
//    fewer than four blocks also a share of the tokens).
//
// What bounds it: the widening (two ALU cycles for each pair of values, and a
// multiply for its scale), not the bytes: a single-row tile costs its four
// warps about 250 instructions each.  So the path is written for issue slots:
// a vote decides whether the softmax reference must rise, sums stay per lane
// until the head ends, queries of the next head are fetched a head ahead, and
// three CTAs per SM (128 registers a thread) cover the latencies.  65536 tiles
// of single rows alone take 114 us, 80% of the copy rate; 64 sequences of 512
// tokens of their own under 4096 shared ones, 32 heads of 128 dims, 61 us (50%
// of the issue slots, 43% of the ALU, 36% of DRAM), where the shared tiles'
// trip through shared memory and its waits take the rest.
#include <cuda.h>
#include <cuda_runtime.h>

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
// to 8 rows the areas hold the warps' outputs at the end of a head, in turn; for
// others a shared tile widened to fp16 (32 tokens at a time: with all 64 the
// ring had two slots instead of four, and single-row tiles took 1.91 ns each
// over the card instead of 1.73) and the queries.
template <int C, int D>
struct F4Smem {
    static constexpr int kStage = F4Tile<C, D>::kBytes;
    static constexpr int kTok = C < 32 ? C : 32;                // tokens widened at a time
    static constexpr int kImage = kTok * D * 2;                 // their keys (and their values)
    static constexpr int kOut8 = kF4Warps * 8 * D * 4;          // 8 rows of each warp
    static constexpr int kExch = 2 * kImage > kOut8 ? 2 * kImage : kOut8;
    static constexpr int kMs = 2 * kF4Warps * 8 * 2 * 4;
    static constexpr int kQ = kQRows * D * 2;                   // query rows of a shared tile (= kOut8)
    static_assert(kQ >= kOut8, "the second area");
    static constexpr int kTail = kMs + 2 * kF4Stages * 8 + kF4Ring * 4 + 2 * kF4Stages * 4 + kQRows * 4;
    static size_t bytes(int stages) { return (size_t)stages * kStage + kExch + kQ + kTail; }
};

__device__ __forceinline__ void f4_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kF4Warps * 32) : "memory"); }

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
// state's sums (ONE: a single query in every column).
template <int D, int NB, bool ONE>
__device__ __forceinline__ void f4_softmax(float (&x)[NB][4], F4State<D, NB>& a, uint32_t (&pb)[NB][2]) {
    bool grow = false;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int e = 0; e < 4; e += ONE ? 2 : 1) grow = grow || x[nb][e] > a.m[nb][e & 1] + (kLift + kSlack);
    if (__any_sync(kFull, grow)) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int r = 0; r < (ONE ? 1 : 2); ++r) {
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
        if constexpr (ONE) {
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
template <int NB>
__device__ __forceinline__ void f4_mask(float (&x)[NB][4], int tok, int ntok, int ctx0, bool causal,
                                        const int (&lim)[NB][2], float scale_log2) {
    const bool in0 = tok < ntok, in1 = tok + 8 < ntok;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[nb][e] = ((e >> 1) ? in1 : in0) ? x[nb][e] * scale_log2 : -INFINITY;
    if (causal) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (ctx0 + tok + 8 * (e >> 1) > lim[nb][e & 1]) x[nb][e] = -INFINITY;
    }
}

// One head's `tiles` tiles, each warp taking 16 tokens of its own; false on a
// timeout.
template <int C, int D, int NB, bool ONE>
__device__ __forceinline__ bool f4_tiles_own(F4Ctx& c, int tiles, const uint32_t (&qb)[NB][D / 16][2],
                                             const int (&lim)[NB][2], bool causal, float scale_log2, int32_t* status,
                                             F4State<D, NB>& a) {
    constexpr int NBLK = C / 16;
    const int tg = f4_token(c.lane >> 2);
    for (; tiles > 0; --tiles) {
        if (!mbar_wait(c.full0 + 8 * c.st, c.ph)) {
            set_status(status, CA_ERR_TIMEOUT);
            return false;
        }
        const int ntok = c.ntok[c.st];
        // a tile's blocks go to the warps in turn, tile after tile
        const int blk = NBLK == 4 ? c.w : (c.w - c.it * NBLK) & 3;
        if (blk < NBLK && blk * 16 < ntok) {
            const uint8_t* tile = c.stages + (size_t)c.st * F4Tile<C, D>::kBytes;
            float x[NB][4];
            uint32_t pb[NB][2];
            f4_scores<C, D, NB, ONE>(tile, blk, qb, x, c.lane);
            f4_mask<NB>(x, blk * 16 + tg, ntok, causal ? c.tok0[c.st] : 0, causal, lim, scale_log2);
            f4_softmax<D, NB, ONE>(x, a, pb);
            f4_pv<C, D, NB>(tile, blk, pb, a.o, c.lane);
        }
        __syncwarp();
        if (c.lane == 0) mbar_arrive(c.empty0 + 8 * c.st);
        c.next();
    }
    return true;
}

// Tokens [base, base + N) of a tile widened once for all warps, into the fp16 K
// and V tiles that the 16-row blocks read (code * scale is exact in fp16).  A
// thread takes 16 bytes (8 at D = 64) of a row's key codes: four dims of every
// 16, and as many of a pair's value codes: two dims of every 16 of both tokens;
// consecutive threads take rows whose swizzled 16-byte columns differ.
template <int C, int D, int N>
__device__ __forceinline__ void f4_tile_to_f16(const uint8_t* src, int base, uint8_t* kd, uint8_t* vd, int tid) {
    using T = F4Tile<C, D>;
    constexpr int NK = D / 16;
    for (int i = tid; i < N * 4; i += kF4Warps * 32) {
        const int t = i & 3, r = i >> 2;
        // rows of 8 in the order 0 1 4 5 2 3 6 7: tokens 0 4 2 6, then 1 5 3 7
        const int m = (r & ~7) | (r & 1) | ((r & 2) << 1) | ((r & 4) >> 1);
        const int tok = f4_token(m);
        uint32_t w[D / 32], sc[D / 64];
        lds_words<D / 32>(src + (base + m) * (D / 2) + t * (D / 8), w);
        lds_words<D / 64>(src + T::kKScales + (base + m) * (D / 16), sc);
#pragma unroll
        for (int kp = 0; kp < NK / 2; ++kp) {             // two steps: one word of codes, two scales
            uint32_t x[4], h[2];
            f16x2_from_e2m1x8(w[kp], x);
            f16x2_from_e4m3x4(sc[kp >> 1], h);
            const uint32_t sa = __byte_perm(h[kp & 1], 0u, 0x1010), sb = __byte_perm(h[kp & 1], 0u, 0x3232);
            *reinterpret_cast<uint2*>(kd + swz(tok, 4 * kp + (t >> 1), N) + 8 * (t & 1)) =
                make_uint2(mul_f16x2(x[0], sa), mul_f16x2(x[1], sa));
            *reinterpret_cast<uint2*>(kd + swz(tok, 4 * kp + 2 + (t >> 1), N) + 8 * (t & 1)) =
                make_uint2(mul_f16x2(x[2], sb), mul_f16x2(x[3], sb));
        }
    }
    for (int i = tid; i < N * 4; i += kF4Warps * 32) {
        // four pairs of tokens a warp: (0, 4), (1, 5), ... of each 8; their rows
        // two apart in turn
        const int g = i & 7, q = i >> 3, pair = (q & ~3) | ((q & 1) << 1) | ((q >> 1) & 1);
        const int tok = (pair >> 2) * 8 + (pair & 3);
        uint32_t w[D / 32], sc[D / 32];
        lds_words<D / 32>(src + T::kVCodes + (base / 2 + pair) * D + f4_v_unit<D>(pair, g) * (D / 8), w);
        lds_words<D / 32>(src + T::kVScales + (base / 2 + pair) * (D / 8), sc);
#pragma unroll
        for (int i4 = 0; i4 < D / 64; ++i4) {
            uint32_t x[4], y[4];
            f16x2_from_e2m1x8(w[i4], x);
            f16x2_from_e2m1x8(w[D / 64 + i4], y);
#pragma unroll
            for (int j2 = 0; j2 < 2; ++j2) {
                uint32_t h[2];
                f16x2_from_e4m3x4(sc[2 * i4 + j2], h);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int k = 2 * j2 + e, kc = 2 * (4 * i4 + k) + (g >> 2), off = 4 * (g & 3);
                    const uint32_t a = mul_f16x2(x[k], h[e]), b = mul_f16x2(y[k], h[e]);   // (tok, tok + 4)
                    *reinterpret_cast<uint32_t*>(vd + swz(tok, kc, N) + off) = __byte_perm(a, b, 0x5410);
                    *reinterpret_cast<uint32_t*>(vd + swz(tok + 4, kc, N) + off) = __byte_perm(a, b, 0x7632);
                }
            }
        }
    }
}

// The end of a head of at most 8 rows: the warps' states meet in the exchange
// area (two buffers in turn, so that a head's stores never meet the last head's
// loads) and warp w writes the partials of rows w and w + 4.  Lane j holds the
// first partial id of row w + 4 j's pieces, this one is `part` further: added
// here, so that the id's load, begun with the head, is first waited for here.
template <int C, int D, bool ONE>
__device__ __forceinline__ void f4_finish(F4Ctx& c, const AttnParams& p, F4State<D, 1>& a, int rows, int pid, int part) {
    const int g = c.lane >> 2, t = c.lane & 3;
    float* ob = reinterpret_cast<float*>((c.flush & 1) ? c.qreg : c.exch);
    // column of a row's dim: the fragments' stores of four rows stay apart
    auto col = [](int row, int d) { return d ^ ((row >> 1 & 3) << 3); };
    float* ms = c.ms + (c.flush & 1) * kF4Warps * 8 * 2;
    ++c.flush;
#pragma unroll
    for (int r = 0; r < (ONE ? 1 : 2); ++r) {
        float s = a.s[0][r];
#pragma unroll
        for (int d = 4; d <= 16; d <<= 1) s += __shfl_xor_sync(kFull, s, d);
        const int row = ONE ? 0 : 2 * t + r;
        if (!ONE || t == 0) {
            if (g == 0) *reinterpret_cast<float2*>(ms + (c.w * 8 + row) * 2) = make_float2(a.m[0][r], s);
#pragma unroll
            for (int db = 0; db < D / 16; ++db)
                *reinterpret_cast<float2*>(ob + (c.w * 8 + row) * D + col(row, 16 * db + 2 * g)) =
                    make_float2(a.o[0][db][r], a.o[0][db][r + 2]);
        }
    }
    f4_sync();
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
    if (S < 1 || S > kF4Stages) {                          // uniform across the CTA
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
        if (p.test_stall) {
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
    const int gt = tab_tok(row_tab[g]), gh = tab_head(row_tab[g]);   // of row g of one position

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
    const bool one = RW == 1;                  // a single row: in every column
    auto load_own = [&](Q1& dst, int qrow, int kvh) {
        const bool there = one || g < RW;
        const int tk = one ? 0 : gt, hh = one ? 0 : gh;
        put_row(dst[0], p.q + (((size_t)qrow * QL + tk) * H + kvh * G + hh) * D, there);
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
    asm volatile("griddepcontrol.wait;" ::: "memory");     // q and the pool after this
    if (n_static > 0 && RW <= 8 && fld(dn, F_KIND) == UNIT_SF) prefetch(fld(dn, F_QROW), fld(dn, F_HEAD));
    for (int seq = 0;; ++seq) {
        // The unit's first stage (or the closing one) carries its id.
        if (!mbar_wait(full0 + 8 * c.st, c.ph)) {
            set_status(p.status, CA_ERR_TIMEOUT);
            return;
        }
        const int cur = ring[seq % kF4Ring];
        if (cur < 0) break;
        const int32_t dc = (seq < n_static) ? dn : load_desc(cur);
        const bool next_static = seq + 1 < n_static;
        if (next_static) dn = load_desc(u_begin + seq + 1);
        const bool next_own = next_static && RW <= 8 && fld(dn, F_KIND) == UNIT_SF;
        f4_sync();                             // the previous unit's exchange has been read
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
            int lim[1][2] = {{limit_of(one ? 0 : 2 * t), limit_of(one ? 0 : 2 * t + 1)}};
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
                    const bool there = g < rows;
                    put_row(qb[0], q_of(there ? g : 0) + (size_t)kvh * G * D, there);
                }
                const int pid = (lane < 2 && w + 4 * lane < rows) ? pid_of(w + 4 * lane, kvh) : 0;
                F4State<D, 1> a;
                a.clear();
                if (one && is_sf) {
                    if (!f4_tiles_own<C, D, 1, true>(c, seg_end - L, qb, lim, false, p.scale_log2, p.status, a)) return;
                    f4_finish<C, D, true>(c, p, a, rows, pid, upart);
                } else {
                    if (!f4_tiles_own<C, D, 1, false>(c, seg_end - L, qb, lim, p.causal, p.scale_log2, p.status, a))
                        return;
                    f4_finish<C, D, false>(c, p, a, rows, pid, upart);
                }
                L = seg_end;
            }
        } else {
            qn_row = -1;                       // (its registers are wanted here)
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) qn[0][kk][0] = qn[0][kk][1] = 0u;
            // More rows: the tile widened once for all warps, each taking a
            // 16-row block and (fewer than 4 blocks) a share of the tokens.
            const int rblocks = rows <= 16 ? 1 : rows <= 32 ? 2 : 4;
            constexpr int N = SM::kTok;
            const int T = min(kF4Warps / rblocks, N / 16), rb = w / T, tp = w % T;
            const bool act = rb < rblocks && rb * 16 < rows;
            int lim[2] = {INT_MAX, INT_MAX};
            if (p.causal) {
                lim[0] = limit_of(rb * 16 + g);
                lim[1] = limit_of(rb * 16 + g + 8);
            }
            const uint32_t kt = smem_u32(exch), vt = kt + SM::kImage, qblock = smem_u32(qreg) + rb * 16 * 128;
            for (; L < L_end; ++kvh, upart = part_rest) {
                const int seg_end = min(L_end, (kvh + 1) * n);
                f4_sync();                     // the last head's exchange has been read
                // Rows past `rows` are left as they are: every mma row is
                // independent and such rows are never written out.
                for (int i = threadIdx.x; i < rows * (D / 8); i += kF4Warps * 32) {
                    const int r = i / (D / 8), k = i % (D / 8);
                    cp_async16(smem_u32(qreg + swz(r, k, kQRows)), q_of(r) + (size_t)kvh * G * D + k * 8);
                }
                cp_async_wait_all();
                float o[D / 8][4], m[2] = {-INFINITY, -INFINITY}, s[2] = {0.f, 0.f};
#pragma unroll
                for (int dt = 0; dt < D / 8; ++dt) o[dt][0] = o[dt][1] = o[dt][2] = o[dt][3] = 0.f;
                for (; L < seg_end; ++L) {
                    if (!mbar_wait(full0 + 8 * c.st, c.ph)) {
                        set_status(p.status, CA_ERR_TIMEOUT);
                        return;
                    }
                    const int ntok = c.ntok[c.st], ctx0 = c.tok0[c.st];
                    const uint8_t* tile = stages + (size_t)c.st * SM::kStage;
#pragma unroll 1
                    for (int base = 0; base < C && (base == 0 || base < ntok); base += N) {
                        f4_sync();             // the last tokens have been read (and the queries are there)
                        f4_tile_to_f16<C, D, N>(tile, base, exch, exch + SM::kImage, threadIdx.x);
                        f4_sync();
                        if (lane == 0 && (base + N >= C || base + N >= ntok)) mbar_arrive(empty0 + 8 * c.st);
                        if (!act) continue;
                        if (T * 16 == N)
                            cf_chunk<N, D, 16>(kt, vt, ntok - base, tp * 16, ctx0 + base, lim[0], lim[1], qblock,
                                               p.scale_log2, m, s, o, lane);
                        else
                            cf_chunk<N, D, N>(kt, vt, ntok - base, 0, ctx0 + base, lim[0], lim[1], qblock,
                                              p.scale_log2, m, s, o, lane);
                    }
                    c.next();
                }
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    s[r] += __shfl_xor_sync(kFull, s[r], 1);
                    s[r] += __shfl_xor_sync(kFull, s[r], 2);
                }
                // The T warps of a block meet two by two in the exchange area
                // (the last tile's place): warps [half, 2 half) hand over.
                float* xo = reinterpret_cast<float*>(exch);
                for (int half = T / 2; half >= 1; half /= 2) {
                    f4_sync();
                    if (act && tp >= half && tp < 2 * half) {
                        const int slot = rb * (T / 2) + tp - half;
                        float* dst = xo + (size_t)slot * (16 * D);
#pragma unroll
                        for (int dt = 0; dt < D / 8; ++dt)
                            reinterpret_cast<float4*>(dst)[dt * 32 + lane] =
                                make_float4(o[dt][0], o[dt][1], o[dt][2], o[dt][3]);
                        if (t == 0)
                            reinterpret_cast<float4*>(ms)[slot * 8 + g] = make_float4(m[0], s[0], m[1], s[1]);
                    }
                    f4_sync();
                    if (act && tp < half) {
                        const int slot = rb * (T / 2) + tp;
                        const float4* so = reinterpret_cast<const float4*>(xo + (size_t)slot * (16 * D));
                        const float4 q = reinterpret_cast<const float4*>(ms)[slot * 8 + g];
                        float a1[2], a2[2];
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            const float m2 = r ? q.z : q.x, s2 = r ? q.w : q.y;
                            const float M = fmaxf(m[r], m2), Mu = M == -INFINITY ? 0.f : M;
                            a1[r] = ex2(m[r] - Mu);
                            a2[r] = ex2(m2 - Mu);
                            s[r] = s[r] * a1[r] + s2 * a2[r];
                            m[r] = M;
                        }
#pragma unroll
                        for (int dt = 0; dt < D / 8; ++dt) {
                            const float4 v = so[dt * 32 + lane];
                            o[dt][0] = o[dt][0] * a1[0] + v.x * a2[0];
                            o[dt][1] = o[dt][1] * a1[0] + v.y * a2[0];
                            o[dt][2] = o[dt][2] * a1[1] + v.z * a2[1];
                            o[dt][3] = o[dt][3] * a1[1] + v.w * a2[1];
                        }
                    }
                }
                if (act && tp == 0) {
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const int row = rb * 16 + g + 8 * r;
                        if (row >= rows) continue;
                        const int id = pid_of(row, kvh) + upart;
                        float* dst = p.part_o + (size_t)id * D;
#pragma unroll
                        for (int dt = 0; dt < D / 8; ++dt)
                            *reinterpret_cast<float2*>(dst + dt * 8 + 2 * t) = make_float2(o[dt][2 * r], o[dt][2 * r + 1]);
                        if (t == 0) p.part_ms[id] = make_float2(m[r], s[r]);
                    }
                }
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
