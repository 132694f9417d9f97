// Query blocks on the 5th-generation tensor cores: tiles of 256 rows (128 at
// head_dim 256) against 128 (64) keys at a time.
//
// One CTA per SM walks its items.  Its warps:
//   0-3, 4-7  the softmax of the tile's two halves of 128 rows, one thread a row
//   8         issues every product: S = Q K^T and O += P V
//   9         brings chunks' keys and values in (TMA)
//   10, 11    bring the next tile's queries in
//   12-15     pools of 8 and 4 bits: widen the chunks to fp16 (values in units of
//             the pool's scales, exact), from a ring of their own
// S, P and O stay in tensor memory; P takes the place of the scores it came from.
// While one half is in its softmax, the other half's products run: a step of 128
// keys and a half takes the tensor cores 8 D clocks (4096 multiply-adds each) and
// its softmax 512 of exponentials (32 a clock), some 1000 with all the rest.  So 128
// dims and many rows are bound by the products, fed one tile's worth at a time (a
// product of 128 x 128 x 16 takes 60 to 75 clocks where 64 are ideal, and the hand-over
// from half to half some 200); 64 dims by the hand-overs themselves (2048 queries of 32
// heads over 8192 tokens: 148 us, 113 if the softmax's warps only pass scores on and
// 133 with half the products; steps of 192 keys 141, but 2% more over some 1200
// tokens, whose last step is then emptier); few rows by DRAM.
// 4096 queries of 32 heads over 32768 tokens (8 key/value heads): 1469 us, 1.40
// PFLOP/s at 1670 MHz under the power limit; of 8-bit pools 20% more a step.
#include <cuda.h>
#include <cuda_runtime.h>

#include <climits>

#include "cross.cuh"
#include "fp4.cuh"
#include "tcgen05.cuh"

namespace ca {
namespace dev {

constexpr int kTmemColumns = 512;
constexpr int kMmaWarp = 8, kChunkWarp = 9, kQueryWarp = 10, kQueryWarps = 2, kWidenWarp = 12, kWidenWarps = 4;
// EB: bytes of a stored element (0: the 4-bit codes).
template <int D, int EB>
struct TileShape {
    static constexpr bool kWiden = EB != 2;
    static constexpr int kThreads = kWiden ? 512 : 384;
    // Registers: 128 a thread at launch (168 with 12 warps); the softmax's warps take
    // what the others give.
    static constexpr int kLaunchRegs = kWiden ? 128 : 168, kSoftmaxRegs = kWiden ? 168 : 200, kOtherRegs = kWiden ? 88 : 104;
    static_assert(256 * kSoftmaxRegs + (kThreads - 256) * kOtherRegs == kThreads * kLaunchRegs, "as many as at launch");
    static constexpr int kHalves = D == 256 ? 1 : 2;
    static constexpr int kKeys = D == 256 ? 64 : 128;             // of a step
    static constexpr int kSlab = kKeys * 128, kStage = D / 64 * kSlab;   // K or V of a step, fp16
    static constexpr int kQSlab = 128 * 128, kQHalf = D / 64 * kQSlab;
    static constexpr int kQBuffers = D == 64 ? 2 : 1;             // the next tile's queries beside this one's
    static constexpr int kQBytes = kHalves * kQHalf;
    static constexpr int kStages = D == 64 ? 8 : kWiden ? 4 : 5;
    // as the pool holds them: E4M3 rows, swizzled; codes, then scales
    static constexpr int kRaw = EB == 1 ? kKeys * D : EB == 0 ? kKeys * (D / 2 + D / 16) : 0;
    static constexpr int kRawStages = EB == 1 ? 2 : EB == 0 ? 3 : 0;
    static constexpr int kO = 0, kS = kHalves * D;                // columns: outputs, then scores, half by half
    static constexpr int kBytes = kQBuffers * kQBytes + kStages * kStage + kRawStages * kRaw + 512;
    static_assert(kS + kHalves * kKeys <= kTmemColumns && kBytes <= 227 * 1024, "fits an SM");
};

struct TileBars {
    uint64_t full[8], empty[8];           // a stage's K or V
    uint64_t raw_full[4], raw_empty[4];   // the same as the pool holds it
    uint64_t q_full[2], q_empty[2];
    uint64_t s_full[2], p_full[2];        // a half's scores are there; its weights are
    uint64_t o_full[2];
    uint64_t drain;
    uint32_t tmem;
};
static_assert(sizeof(TileBars) <= 512, "room behind the stages");

// What every role reads of an item.
struct TileItem {
    BlockItem b;
    int n, steps;                         // tokens up to the item's last chunk, steps from c_begin on
};
template <int C, int KEYS>
__device__ __forceinline__ TileItem tile_item(const CrossParams& p, int idx) {
    TileItem t;
    t.b = p.items[idx];
    t.n = min(tokens_now(p, t.b, C), t.b.c_end * C);
    t.steps = max(0, (t.n - t.b.c_begin * C + KEYS - 1) / KEYS);
    return t;
}

// A CTA's items in turn; what there is to know of the next one is on its way
// beforehand.
template <int C, int KEYS>
struct ItemWalk {
    const CrossParams& p;
    int idx, end;
    TileItem t, next;
    __device__ __forceinline__ explicit ItemWalk(const CrossParams& p_)
        : p(p_), idx(p_.cta_begin[blockIdx.x]), end(p_.cta_begin[blockIdx.x + 1]) {
        if (idx < end) t = tile_item<C, KEYS>(p, idx);
        if (idx + 1 < end) next = tile_item<C, KEYS>(p, idx + 1);
    }
    __device__ __forceinline__ bool more() const { return idx < end; }
    __device__ __forceinline__ void advance() {
        t = next;
        if (++idx + 1 < end) next = tile_item<C, KEYS>(p, idx + 1);
    }
};

// A stage as the pool holds it, widened into swizzled fp16 slabs by the threads
// of kWidenWarps warps.  Which lane has which piece keeps loads and stores of
// 8-bit rows free of bank conflicts (rows r and r ^ 5 beside each other) and those
// of 4-bit ones two to a bank at most.
template <int D, int EB, int KEYS>
__device__ __forceinline__ void widen(const uint8_t* raw, uint8_t* dst, bool values, int warp, int lane) {
    if constexpr (EB == 1) {
        const int r0 = (lane >> 3) ^ ((lane >> 2 & 1) * 5), k0 = lane & 3;
#pragma unroll 4
        for (int i = warp; i < KEYS / 8 * (D / 64); i += kWidenWarps) {
            const int r = i / (D / 64) * 8 + r0, k = i % (D / 64) * 4 + k0;     // 16 dims of a row
            const uint4 x = *reinterpret_cast<const uint4*>(raw + swz(r, k, KEYS));
            uint32_t w[8];
            const uint32_t in[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t y[2];
                f16x2_from_e4m3x4(in[j], y);
                w[2 * j] = y[0];
                w[2 * j + 1] = y[1];
            }
            *reinterpret_cast<uint4*>(dst + swz(r, 2 * k, KEYS)) = make_uint4(w[0], w[1], w[2], w[3]);
            *reinterpret_cast<uint4*>(dst + swz(r, 2 * k + 1, KEYS)) = make_uint4(w[4], w[5], w[6], w[7]);
        }
    } else if (!values) {
        // codes of a row: its dims 16 b + 4 t + 0 .. 3 of all blocks b are D / 8 bytes
        const int t = lane & 3;
#pragma unroll 2
        for (int m = warp * 8 + (lane >> 2); m < KEYS; m += 8 * kWidenWarps) {
            const int r = f4_token(m);
            uint32_t c[D / 32], s[D / 64];
            lds_words<D / 32>(raw + m * (D / 2) + t * (D / 8), c);
            lds_words<D / 64>(raw + KEYS * (D / 2) + m * (D / 16), s);
#pragma unroll
            for (int b4 = 0; b4 < D / 64; ++b4) {
                uint32_t h[2];
                f16x2_from_e4m3x4(s[b4], h);
#pragma unroll
                for (int b2 = 0; b2 < 2; ++b2) {          // two blocks: a word of codes
                    uint32_t x[4];
                    f16x2_from_e2m1x8(c[2 * b4 + b2], x);
                    const uint32_t lo = __byte_perm(h[b2], h[b2], 0x1010), hi = __byte_perm(h[b2], h[b2], 0x3232);
                    const int k = 2 * (4 * b4 + 2 * b2) + (t >> 1);
                    *reinterpret_cast<uint2*>(dst + swz(r, k, KEYS) + 8 * (t & 1)) = make_uint2(mul_f16x2(x[0], lo), mul_f16x2(x[1], lo));
                    *reinterpret_cast<uint2*>(dst + swz(r, k + 2, KEYS) + 8 * (t & 1)) =
                        make_uint2(mul_f16x2(x[2], hi), mul_f16x2(x[3], hi));
                }
            }
        }
    } else {
        // pairs of tokens r, r + 4 to a byte: dims 16 b + 2 g of all blocks b, then 16 b + 2 g + 1
        const int u = lane & 7;
#pragma unroll 2
        for (int pair = warp * 4 + (lane >> 3); pair < KEYS / 2; pair += 4 * kWidenWarps) {
            const int g = f4_v_unit<D>(pair, u), r = (pair >> 2) * 8 + (pair & 3);
            constexpr int NW = D / 64;
            uint32_t c[2 * NW], s[D / 32];
            lds_words<2 * NW>(raw + pair * D + u * (D / 8), c);
            lds_words<D / 32>(raw + KEYS * (D / 2) + pair * (D / 8), s);
#pragma unroll
            for (int i = 0; i < NW; ++i) {                // four blocks to a word
                uint32_t a[4], b[4];
                f16x2_from_e2m1x8(c[i], a);
                f16x2_from_e2m1x8(c[NW + i], b);
#pragma unroll
                for (int j2 = 0; j2 < 2; ++j2) {
                    uint32_t h[2];
                    f16x2_from_e4m3x4(s[2 * i + j2], h);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int j = 2 * j2 + e, k = 2 * (4 * i + j) + (g >> 2);
                        const uint32_t x = mul_f16x2(a[j], h[e]), y = mul_f16x2(b[j], h[e]);
                        *reinterpret_cast<uint32_t*>(dst + swz(r, k, KEYS) + 4 * (g & 3)) = __byte_perm(x, y, 0x5410);
                        *reinterpret_cast<uint32_t*>(dst + swz(r + 4, k, KEYS) + 4 * (g & 3)) = __byte_perm(x, y, 0x7632);
                    }
                }
            }
        }
    }
}

template <int C, int D, int EB>
__global__ void __launch_bounds__(TileShape<D, EB>::kThreads, 1)
cross_tiles_kernel(const __grid_constant__ CUtensorMap tmap, const CrossParams p) {
    using T = TileShape<D, EB>;
    using Walk = ItemWalk<C, T::kKeys>;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t* stages = smem + T::kQBuffers * T::kQBytes;
    uint8_t* raw = stages + T::kStages * T::kStage;
    TileBars* bars = reinterpret_cast<TileBars*>(raw + T::kRawStages * T::kRaw);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if ((smem_u32(smem) & 1023u) != 0) {                  // (the same for the whole CTA)
        if (threadIdx.x == 0) set_status(p.status, CA_ERR_INVALID);
        return;
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < T::kStages; ++i) {
            mbar_init(smem_u32(&bars->full[i]), T::kWiden ? kWidenWarps : 1);
            mbar_init(smem_u32(&bars->empty[i]), 1);
        }
        for (int i = 0; i < T::kRawStages; ++i) {
            mbar_init(smem_u32(&bars->raw_full[i]), 1);
            mbar_init(smem_u32(&bars->raw_empty[i]), kWidenWarps);
        }
        for (int i = 0; i < T::kQBuffers; ++i) {
            mbar_init(smem_u32(&bars->q_full[i]), kQueryWarps);
            mbar_init(smem_u32(&bars->q_empty[i]), 1);
        }
        for (int h = 0; h < 2; ++h) {
            mbar_init(smem_u32(&bars->s_full[h]), 1);
            mbar_init(smem_u32(&bars->p_full[h]), 4);
            mbar_init(smem_u32(&bars->o_full[h]), 1);
        }
        mbar_init(smem_u32(&bars->drain), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == kMmaWarp) tmem_alloc(smem_u32(&bars->tmem), kTmemColumns);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem;
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // Every wait is bounded; a role whose wait runs out says so and ends, and
    // the others' waits for it then run out too.
    auto timed_out = [&]() { set_status(p.status, CA_ERR_TIMEOUT); };

    constexpr int kPer = T::kKeys / C;                    // chunks of a step

    if (warp >= kMmaWarp) {
        give_registers<T::kOtherRegs>();
        if (warp == kChunkWarp) {
            // ------------------------------ keys and values ------------------------------
            constexpr int N = T::kWiden ? T::kRawStages : T::kStages;
            uint64_t* const full = T::kWiden ? bars->raw_full : bars->full;
            uint64_t* const empty = T::kWiden ? bars->raw_empty : bars->empty;
            int it = 0;
            bool ok = true;
            if (p.test_stall) {                               // test hook: a wait that nothing ends
                if (lane == 0 && !mbar_wait(smem_u32(&full[0]), 0u)) timed_out();
                ok = false;
            }
            for (Walk walk(p); ok && walk.more(); walk.advance()) {
                const TileItem& t = walk.t;
                const int32_t* slots = p.list_slots + t.b.list0;
                // A lane per chunk.  Past the item's last chunk that one comes again: its
                // keys are masked, and its values, whose weights are 0, are finite.
                auto slot_at = [&](int step) {
                    return lane < kPer && step < t.steps ? slots[min(t.b.c_begin + step * kPer + lane, t.b.c_end - 1)] : 0;
                };
                int slot = slot_at(0);
                for (int x = 0; x < 2 * t.steps; ++x, ++it) { // K and V of each step
                    const int st = it % N;
                    if (!mbar_wait(smem_u32(&empty[st]), ((uint32_t)(it / N) & 1u) ^ 1u)) ok = false;
                    ok = __all_sync(kFull, ok);
                    if (!ok) {
                        if (lane == 0) timed_out();
                        break;
                    }
                    if (slot < 0 || slot >= p.capacity) {
                        set_status(p.status, CA_ERR_DEVICE_BOUNDS);
                        slot = 0;
                    }
                    const uint32_t fb = smem_u32(&full[st]);
                    if (lane == 0) mbar_expect_tx_only(fb, T::kWiden ? T::kRaw : T::kStage);
                    __syncwarp();
                    if (lane < kPer) {
                        if constexpr (EB == 0) {
                            using F = F4Tile<C, D>;
                            const uint8_t* src =
                                p.kv + (((long long)slot * p.n_layers + p.layer) * p.n_kv_heads + t.b.head) * F::kBytes;
                            const uint32_t dst = smem_u32(raw) + st * T::kRaw;
                            bulk_load(dst + lane * F::kCodes, src + (x & 1) * F::kCodes, F::kCodes, fb);
                            bulk_load(dst + T::kKeys * (D / 2) + lane * F::kScales, src + F::kKScales + (x & 1) * F::kScales,
                                      F::kScales, fb);
                        } else {
                            const int row =
                                ((slot * p.n_layers + p.layer) * 2 * p.n_kv_heads + (x & 1) * p.n_kv_heads + t.b.head) * C;
                            const uint32_t dst =
                                (T::kWiden ? smem_u32(raw) + st * T::kRaw : smem_u32(stages) + st * T::kStage) + lane * C * 128;
#pragma unroll
                            for (int s = 0; s < D * EB / 128; ++s) tma_load_2d(dst + s * T::kSlab, &tmap, s * (128 / EB), row, fb);
                        }
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(fb);
                    if (x & 1) slot = slot_at((x >> 1) + 1);
                }
            }
            if (!ok)                                          // copies in flight land before the CTA can end
                for (int k = max(0, it - N); k < it; ++k) mbar_wait(smem_u32(&full[k % N]), (uint32_t)(k / N) & 1u);
        } else if (T::kWiden && warp >= kWidenWarp) {
            // ------------------------------ widening ------------------------------
            if constexpr (T::kWiden) {
                int st = 0, rs = 0;
                uint32_t st_ph = 0u, rs_ph = 0u;
                bool ok = true;
                for (Walk walk(p); ok && walk.more(); walk.advance()) {
                    const int steps = walk.t.steps;
                    for (int x = 0; x < 2 * steps; ++x) {
                        ok = __all_sync(kFull, mbar_wait(smem_u32(&bars->empty[st]), st_ph ^ 1u) &&
                                                   mbar_wait(smem_u32(&bars->raw_full[rs]), rs_ph));
                        if (!ok) {
                            if (lane == 0) timed_out();
                            break;
                        }
                        widen<D, EB, T::kKeys>(raw + rs * T::kRaw, stages + st * T::kStage, (x & 1) != 0, warp - kWidenWarp, lane);
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                        __syncwarp();
                        if (lane == 0) {
                            mbar_arrive(smem_u32(&bars->full[st]));
                            mbar_arrive(smem_u32(&bars->raw_empty[rs]));
                        }
                        if (++st == T::kStages) { st = 0; st_ph ^= 1u; }
                        if (++rs == T::kRawStages) { rs = 0; rs_ph ^= 1u; }
                    }
                }
            }
        } else if (warp >= kQueryWarp && warp < kQueryWarp + kQueryWarps) {
            // ------------------------------ queries ------------------------------
            int qb = 0;
            uint32_t ph = 0u;
            for (Walk walk(p); walk.more(); walk.advance()) {
                const TileItem& t = walk.t;
                if (t.steps == 0) continue;
                if (!__all_sync(kFull, mbar_wait(smem_u32(&bars->q_empty[qb]), ph ^ 1u))) {
                    if (lane == 0) timed_out();
                    break;
                }
                // A lane has one 16-byte piece of every kStep-th row of the halves that have
                // any.  Row r is token (x0 + r) / group behind the tile's first; that quotient
                // of a number below 320 by one up to 64 is exact in 16 fraction bits, and
                // every row's address is on its own (a running one took 15000 clocks a tile).
                constexpr int kPieces = D / 8, kStep = 32 * kQueryWarps / kPieces;
                const int id = threadIdx.x - 32 * kQueryWarp, k = id % kPieces, rows = t.b.rows > 128 ? 256 : 128;
                const uint32_t x0 = t.b.row0 % p.group, inverse = (65535u + p.group) / p.group;
                const uint16_t* src = p.q + ((size_t)(t.b.q0 + t.b.row0 / p.group) * p.n_heads + (size_t)t.b.head * p.group) * D + k * 8;
                const uint32_t dst = smem_u32(smem) + qb * T::kQBytes;
#pragma unroll 8
                for (int r = id / kPieces; r < rows; r += kStep) {
                    const uint32_t tok = (x0 + r) * inverse >> 16, x = x0 + r - tok * p.group;
                    const bool there = r < t.b.rows;
                    cp_async16_or_zero(dst + r / 128 * T::kQHalf + swz(r % 128, k, 128),
                                       src + (there ? ((size_t)tok * p.n_heads + x) * D : 0), there);
                }
                cp_async_wait_all();
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&bars->q_full[qb]));
                if constexpr (T::kQBuffers == 1) {            // the next tile's into L2 meanwhile
                    if (walk.idx + 1 < walk.end) {
                        const BlockItem& n = walk.next.b;
                        constexpr int kLines = D / 64;        // 128 bytes each
                        for (int i = id; i < n.rows * kLines; i += 32 * kQueryWarps)
                            asm volatile("prefetch.global.L2 [%0];" ::"l"(p.q + block_row(p, n, i / kLines, D) + i % kLines * 64));
                    }
                }
                if (++qb == T::kQBuffers) { qb = 0; ph ^= 1u; }
            }
        } else if (warp == kMmaWarp) {
            // ------------------------------ products ------------------------------
            // (the whole warp runs this: mma_ss)
            constexpr uint32_t kShapeS = f16_shape(T::kKeys, false), kShapeO = f16_shape(D, true);
            const uint32_t q_desc = desc_along_row(smem_u32(smem)), k_desc = desc_along_row(smem_u32(stages)),
                           v_desc = desc_along_rows(smem_u32(stages), T::kSlab);
            int st = 0;                                       // the stage whose turn it is, and its parity
            int qb = 0;                                       // the same of the queries' buffers
            uint32_t st_ph = 0u, q_ph = 0u, p_ph = 0u;        // (p_ph: a bit for each half)
            bool ok = true;
            auto wait = [&](uint64_t* bar, uint32_t parity) {
                ok = warp_wait(smem_u32(bar), parity);
                if (!ok && lane == 0) timed_out();
                return ok;
            };
            auto next_stage = [&]() {
                if (++st == T::kStages) { st = 0; st_ph ^= 1u; }
            };
            auto scores = [&](int h, int stage) {
                const uint32_t a = q_desc + qb * (T::kQBytes >> 4) + h * (T::kQHalf >> 4), b = k_desc + stage * (T::kStage >> 4);
                const uint32_t d = tmem + T::kS + h * T::kKeys;
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
                    mma_ss<kShapeS>(d, a + k / 4 * (T::kQSlab >> 4) + k % 4 * 2, b + k / 4 * (T::kSlab >> 4) + k % 4 * 2, k > 0);
                mma_commit(smem_u32(&bars->s_full[h]));
            };
            for (Walk walk(p); ok && walk.more(); walk.advance()) {
                const TileItem& t = walk.t;
                if (t.steps == 0) continue;
                const int halves = t.b.rows > 128 ? 2 : 1;
                if (!wait(&bars->q_full[qb], q_ph)) break;
                if (!wait(&bars->full[st], st_ph)) break;
                for (int h = 0; h < halves; ++h) scores(h, st);
                // Each step: its values, then the next one's keys.  What a step waits for is
                // asked for while products are still queued: a wait takes some 150 clocks
                // even where nothing is missing, and the queue is not deep.
                next_stage();
                int sv = st;
                if (!wait(&bars->full[st], st_ph)) break;
                for (int j = 0; j < t.steps; ++j) {
                    const bool more = j + 1 < t.steps;
                    if (more) {
                        next_stage();
                        if (!wait(&bars->full[st], st_ph)) break;
                    }
                    const int sk = st;
                    for (int h = 0; h < halves; ++h) {
                        if (!wait(&bars->p_full[h], (p_ph >> h) & 1u)) break;
                        tc_fence_after();
                        p_ph ^= 1u << h;
                        const uint32_t b = v_desc + sv * (T::kStage >> 4);
                        const uint32_t a = tmem + T::kS + h * T::kKeys, d = tmem + T::kO + h * D;
#pragma unroll
                        for (int k = 0; k < T::kKeys / 16; ++k) mma_ts<kShapeO>(d, a + 8 * k, b + k * (2048 >> 4), j > 0 || k > 0);
                        if (more) scores(h, sk);
                        else mma_commit(smem_u32(&bars->o_full[h]));
                        if (h == 0 && more) {                 // the next step's values
                            next_stage();
                            if (!wait(&bars->full[st], st_ph)) break;
                        }
                    }
                    if (!ok) break;
                    sv = st;
                }
                if (ok) next_stage();
                if (++qb == T::kQBuffers) { qb = 0; q_ph ^= 1u; }
            }
            // everything issued is done before the CTA can end
            mma_commit(smem_u32(&bars->drain));
            mbar_wait(smem_u32(&bars->drain), 0u);
            __syncwarp();
        }
    } else {
        take_registers<T::kSoftmaxRegs>();
        if (warp < 4 * T::kHalves) {
            // ------------------------------ softmax ------------------------------
            const int h = warp >> 2;
            const uint32_t lanes = (uint32_t)(warp & 3) << 21;          // 32 (warp % 4), in an address's upper half
            const uint32_t s_at = tmem + lanes + T::kS + h * T::kKeys, o_at = tmem + lanes + T::kO + h * D;
            const int r = threadIdx.x & (128 * T::kHalves - 1);
            // a negative scale turns the scores' signs; with 0 all scores are alike
            const float scale = fmaxf(fabsf(p.scale_log2), 1e-37f);
            const bool turned = p.scale_log2 < 0.f;
            const bool wide = (reinterpret_cast<uintptr_t>(p.out) & 31u) == 0;
            const uint64_t scale2 = pair_of(__float_as_uint(scale), __float_as_uint(scale));
            auto largest = [](const uint32_t (&x)[32]) {
                float a[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int e = 0; e < 32; e += 2)
                    a[(e >> 1) & 3] = fmaxf(a[(e >> 1) & 3], fmaxf(__uint_as_float(x[e]), __uint_as_float(x[e + 1])));
                return fmaxf(fmaxf(a[0], a[1]), fmaxf(a[2], a[3]));
            };
            // The scores of the tile's last half being there says that every product before
            // them is done: its first thread then gives the stages and queries back.  (A
            // commit of the products' warp for each of them cost it 100 clocks.)
            int first = 0, qb = 0;                            // the item's first stage, its queries' buffer
            auto release = [&](int x) { mbar_arrive(smem_u32(&bars->empty[(first + x) % T::kStages])); };
            uint32_t s_ph = 0u, o_ph = 0u;
            bool ok = true;
            auto wait = [&](uint64_t* bar, uint32_t parity) {
                ok = __all_sync(kFull, mbar_wait(smem_u32(bar), parity));
                if (!ok && lane == 0) timed_out();
                tc_fence_after();
                return ok;
            };
            for (Walk walk(p); ok && walk.more(); walk.advance()) {
                const TileItem& t = walk.t;
                auto pass_by = [&]() {
                    first = (first + 2 * t.steps) % T::kStages;
                    if (t.steps > 0 && ++qb == T::kQBuffers) qb = 0;
                };
                const bool releases = (warp & 3) == 0 && lane == 0 && (128 * (h + 1) >= t.b.rows) && 128 * h < t.b.rows;
                if (128 * h >= t.b.rows) {
                    pass_by();
                    continue;
                }
                // the last token that the row sees (a row past the tile's last: all)
                int last = t.n - 1;
                if (p.causal && r < t.b.rows) last = min(last, t.b.ctx - t.b.m + (t.b.row0 + r) / p.group);
                const int all_see = __reduce_min_sync(kFull, last);
                float m = -INFINITY, sum = 0.f;
                for (int j = 0; j < t.steps; ++j) {
                    if (!wait(&bars->s_full[h], s_ph)) break;
                    s_ph ^= 1u;
                    if (releases) {                           // K of this step, V of the one before
                        if (j > 0) release(2 * j - 1);
                        release(2 * j);
                        if (j + 1 == t.steps) mbar_arrive(smem_u32(&bars->q_empty[qb]));
                    }
                    constexpr int NC = T::kKeys / 32;         // 32 columns at a time
                    if (turned || t.b.c_begin * C + (j + 1) * T::kKeys - 1 > all_see) {
                        // few steps need it: signs turned and hidden tokens masked in place
                        // (from the first column on that some row of the warp does not see)
                        const int at = t.b.c_begin * C + j * T::kKeys, see = last - at;
#pragma unroll 1
                        for (int c = turned ? 0 : max(0, all_see + 1 - at) / 32; c < NC; ++c) {
                            uint32_t x[32];
                            tmem_ld32(s_at + 32 * c, x);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; ++e) x[e] = 32 * c + e > see ? 0xff800000u : turned ? x[e] ^ 0x80000000u : x[e];
                            tmem_st32(s_at + 32 * c, x);
                        }
                        tmem_wait_st();
                    }
                    // The weights 2^(x - m), with the reference m that the steps before have
                    // left, and beside them the largest score.  m is set 8 below a largest
                    // score (rounded up), and rises only where one exceeds it by more than 15:
                    // weights in fp16 stay below 2^15, and those that lose bits below 2^-14 are
                    // at most 2^-21 of the largest.  It rises by whole numbers, so that scaling
                    // the outputs rounds nothing; the step's weights are then taken again (the
                    // scores are overwritten after this check).
                    if (j == 0) {                             // (from the first 32: what exceeds them by 7 is rare)
                        uint32_t x[32];
                        tmem_ld32(s_at, x);
                        tmem_wait_ld();
                        const float top = largest(x) * scale;
                        if (top > -INFINITY) m = ceilf(top) - 8.f;
                    }
                    uint64_t add[2] = {0ull, 0ull};
                    auto weigh = [&](const uint32_t (&x)[32], uint32_t* w) {
                        const float mu = m == -INFINITY ? 0.f : m;
                        const uint64_t mu2 = pair_of(__float_as_uint(-mu), __float_as_uint(-mu));
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            uint32_t lo, hi;
                            halves_of(fma2(pair_of(x[2 * e], x[2 * e + 1]), scale2, mu2), lo, hi);
                            const float a = ex2(__uint_as_float(lo)), b = ex2(__uint_as_float(hi));
                            w[e] = pack_half2(a, b);
                            add[e & 1] = add2(add[e & 1], pair_of(__float_as_uint(a), __float_as_uint(b)));
                        }
                    };
                    uint32_t w[NC / 2][32];
                    float top = -INFINITY;
                    {
                        uint32_t x[2][32];
                        tmem_ld32(s_at, x[0]);
#pragma unroll
                        for (int c = 0; c < NC; ++c) {
                            tmem_wait_ld();
                            if (c + 1 < NC) tmem_ld32(s_at + 32 * (c + 1), x[(c + 1) & 1]);
                            top = fmaxf(top, largest(x[c & 1]));
                            weigh(x[c & 1], &w[c / 2][c % 2 * 16]);
                        }
                    }
                    top *= scale;
                    const bool rise = top > m + 15.f;
                    if (!__any_sync(kFull, rise)) {
#pragma unroll
                        for (int c = 0; c < NC / 2; ++c) tmem_st32(s_at + 32 * c, w[c]);
                    } else {
                        const float up = ceilf(top) - 8.f, a = rise ? ex2(m - up) : 1.f;
                        if (rise) m = up;
                        sum *= a;
                        if (j > 0) {                          // (the scores' barrier says that the step before is in)
#pragma unroll 1
                            for (int d = 0; d < D / 32; ++d) {
                                uint32_t o[32];
                                tmem_ld32(o_at + 32 * d, o);
                                tmem_wait_ld();
#pragma unroll
                                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * a);
                                tmem_st32(o_at + 32 * d, o);
                            }
                        }
                        add[0] = add[1] = 0ull;
#pragma unroll 1
                        for (int c = 0; c < NC; ++c) {        // (P's columns 16 c .. + 15 held scores that have been read)
                            uint32_t x[32], y[16];
                            tmem_ld32(s_at + 32 * c, x);
                            tmem_wait_ld();
                            weigh(x, y);
                            tmem_st16(s_at + 16 * c, y);
                        }
                    }
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&bars->p_full[h]));
                    uint32_t lo, hi;
                    halves_of(add2(add[0], add[1]), lo, hi);
                    sum += __uint_as_float(lo) + __uint_as_float(hi);
                }
                if (!ok) break;
                if (t.steps > 0) {
                    if (!wait(&bars->o_full[h], o_ph)) break;
                    o_ph ^= 1u;
                    if (releases) release(2 * t.steps - 1);
                }
                const float inv = sum == 0.f ? 0.f : p.out_scale / sum;
                const size_t id = (size_t)t.b.part * p.tile_rows + r;
                const size_t at = r < t.b.rows ? block_row(p, t.b, r, D) : 0;
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t o[32];
                    if (t.steps > 0) {
                        tmem_ld32(o_at + 32 * c, o);
                        tmem_wait_ld();
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = 0u;
                    }
                    // (32 bytes a store where the rows allow it: whole sectors, half as many)
                    if (r >= t.b.rows) {
                    } else if (t.b.part >= 0) {
                        float* dst = p.part_o + id * D + 32 * c;
#pragma unroll
                        for (int e = 0; e < 32; e += 8)
                            st_32b(dst + e, o[e], o[e + 1], o[e + 2], o[e + 3], o[e + 4], o[e + 5], o[e + 6], o[e + 7]);
                    } else {
                        uint16_t* dst = p.out + at + 32 * c;
                        uint32_t w[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            w[e] = pack_half2(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv);
                        if (wide) {
#pragma unroll
                            for (int e = 0; e < 16; e += 8)
                                st_32b(dst + 2 * e, w[e], w[e + 1], w[e + 2], w[e + 3], w[e + 4], w[e + 5], w[e + 6],
                                       w[e + 7]);
                        } else {
#pragma unroll
                            for (int e = 0; e < 16; e += 4)
                                *reinterpret_cast<uint4*>(dst + 2 * e) = make_uint4(w[e], w[e + 1], w[e + 2], w[e + 3]);
                        }
                    }
                    __syncwarp();
                }
                if (t.b.part >= 0 && r < t.b.rows) p.part_ms[id] = make_float2(m, sum);
                pass_by();
                tc_fence_before();                            // (the next tile's first product overwrites the outputs)
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp) tmem_free(tmem, kTmemColumns);
}

}  // namespace dev

namespace {

template <int C, int D, int EB>
int run(const Pool& p, const dev::CrossParams& a, cudaStream_t s) {
    using T = dev::TileShape<D, EB>;
    if (cudaFuncSetAttribute(dev::cross_tiles_kernel<C, D, EB>, cudaFuncAttributeMaxDynamicSharedMemorySize, T::kBytes) != cudaSuccess)
        return CA_ERR_CUDA;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t c = {};
    c.gridDim = dim3((unsigned)a.n_places);
    c.blockDim = dim3(T::kThreads);
    c.dynamicSmemBytes = T::kBytes;
    c.stream = s;
    c.attrs = attr;
    c.numAttrs = 1;
    if (cudaLaunchKernelEx(&c, dev::cross_tiles_kernel<C, D, EB>, *reinterpret_cast<const CUtensorMap*>(p.tmap), a) != cudaSuccess)
        return CA_ERR_CUDA;
    count_launch();
    return CA_OK;
}

template <int D, int EB>
int pick(const Pool& p, const dev::CrossParams& a, cudaStream_t s) {
    if (p.cfg.chunk == 16) return run<16, D, EB>(p, a, s);
    if (p.cfg.chunk == 32) return run<32, D, EB>(p, a, s);
    if constexpr (D <= 128)
        if (p.cfg.chunk == 64) return run<64, D, EB>(p, a, s);
    return CA_ERR_UNSUPPORTED;
}

}  // namespace

int cross_tile_rows(const PoolCfg& c) { return c.head_dim == 256 ? 128 : 256; }
int cross_places(const Pool& p) { return p.sms > 0 ? p.sms : 152; }

int launch_cross_tiles(const Pool& p, const dev::CrossParams& a, cudaStream_t s) {
    const int D = p.cfg.head_dim;
    if (p.cfg.flags & CA_KV_FP4) return D == 64 ? pick<64, 0>(p, a, s) : D == 128 ? pick<128, 0>(p, a, s) : CA_ERR_UNSUPPORTED;
    if (p.cfg.flags & CA_KV_FP8) return D == 128 ? pick<128, 1>(p, a, s) : CA_ERR_UNSUPPORTED;
    return D == 64 ? pick<64, 2>(p, a, s) : D == 128 ? pick<128, 2>(p, a, s) : D == 256 ? pick<256, 2>(p, a, s) : CA_ERR_UNSUPPORTED;
}

}  // namespace ca
