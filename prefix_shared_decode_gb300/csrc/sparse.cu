// Attention over selected chunks: choosing each context's chunks by an upper
// bound on their scores, and decode attention over listed chunks alone, for
// every pool type.  Contexts of 10^5 tokens and more spend a decode step
// reading keys and values that the softmax weights at nothing; the bounds are
// 1 / (chunk length) of the keys and the lists a few of the chunks.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "ca_internal.h"
#include "fp4.cuh"

namespace ca {
namespace dev {

// ---------------------------------------------------------------------------
// Clusters: the CTAs that score one context's chunks leave their scores in
// the first one's shared memory.
// ---------------------------------------------------------------------------
__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync_all() {
    cluster_arrive();
    cluster_wait();
}
__device__ __forceinline__ uint32_t peer_addr(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ void st_peer(uint32_t addr, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
// What both kernels read of the schedule and the pool.
struct ListParams {
    const uint16_t* q;            // fp16 [b][H][D]
    const int32_t* list_off;      // chunk slots of batch row i: list_slots[list_off[i] ..)
    const int32_t* list_slots;
    const int32_t* slot_ntok;
    const uint8_t* kv;
    const uint16_t* bounds;       // [slot][L][Hkv][largest, smallest][D]
    int32_t* status;
    int32_t* lists;               // [b][Hkv][top_k] (read by the attention)
    uint16_t* out;
    int32_t n_layers, n_kv_heads, n_heads, group, layer, capacity, top_k;
    int32_t sink, recent;         // selection
    int32_t splits;               // selection: CTAs per cluster
    int32_t n_stages, n_units;    // attention: ring stages, units
    int32_t* counters;            // pieces of each unit that have arrived (0 between calls)
    float* parts;                 // [2 per CTA] (m, s) of the rows, then their outputs
    float scale_log2, out_scale;
    int32_t test_stall;           // attention, test hook: waits that run out (below)
};

// ---------------------------------------------------------------------------
// Selection.  score(chunk) = max over the group's rows of
//     sum_d max(q_d hi_d, q_d lo_d) = sum_d q_d^+ hi_d + q_d^- lo_d,
// a product of the bounds [chunks x 2D] with the rows' positive and negative
// parts: tensor cores take it 16 chunks by 8 rows at a time, with the dims
// permuted so that a lane's operand of a bounds row is 16 contiguous bytes
// from global memory (nothing is staged; the kernel is bound by reading the
// bounds once).  The CTAs of a cluster score their blocks of 16 chunks and
// leave the scores, as order-preserving integers, in the first CTA's shared
// memory; that CTA finds the top_k-th.
//
// Exact order: a 32-bit score is off by at most E (below), so with T the
// top_k-th largest of them, a chunk above T + 2E is among the exact top_k, one
// below T - 2E is not.  Where more chunks lie in between than places are left
// (a handful as a rule), those are summed again to 48 bits and ranked by
// (score, lower number).
// ---------------------------------------------------------------------------
constexpr int kSelThreads = 256, kSelWarps = kSelThreads / 32;
constexpr uint32_t kSure = 0xffffffffu;   // key of a chunk that is taken
constexpr uint32_t kTie = 0xfffffffeu;    // key of one that ties for the last places
constexpr int kFewTies = 256;             // chunks ranked pairwise in 64 bits

__device__ __forceinline__ uint32_t order_key(float x) {   // monotone; 0 for a NaN, never as much as kTie
    if (x != x) return 0u;
    const uint32_t u = __float_as_uint(x + 0.f);           // -0 counts as 0
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ unsigned long long order_key(double x) {
    if (x != x) return 0ull;
    const unsigned long long u = (unsigned long long)__double_as_longlong(x + 0.0);
    return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}
__device__ __forceinline__ uint32_t part_f16x2(uint32_t x, bool positive) {   // max(x, 0) or min(x, 0)
    const __half2 h = *reinterpret_cast<const __half2*>(&x), z = __float2half2_rn(0.f);
    const __half2 r = positive ? __hmax2(h, z) : __hmin2(h, z);
    return *reinterpret_cast<const uint32_t*>(&r);
}

constexpr int kBins = 2048, kPerBin = kBins / kSelThreads;
struct SelShared {
    uint32_t hist[kBins];
    uint32_t top_abs[8][128];             // largest |bound| of each pair of dims: per warp, then per CTA of the cluster
    uint32_t red[kSelWarps][2];
    float qsum[kSelWarps];
    uint32_t bin, left, in_bin, T;        // histogram step: the digit, places left inside it, its count
    uint32_t n_list;
    uint32_t list[kFewTies];
    unsigned long long key64[kFewTies];
};

// s + e <- s + e + x, s the rounded sum and e what rounding lost.
__device__ __forceinline__ void add_pair(float& s, float& e, float x, float y) {
    const float t = __fadd_rn(s, x), z = __fsub_rn(t, s);
    const float lost = __fadd_rn(__fsub_rn(s, __fsub_rn(t, z)), __fsub_rn(x, z));
    s = t;
    e = __fadd_rn(__fadd_rn(e, y), lost);
}
// The largest of N rows' products with a chunk's bounds, each to 48 bits
// (a warp; every lane gets it), as an ordered key.  Products of fp16 are exact
// in fp32 and their sums are held as pairs of fp32: on the card's fp64 pipe (2
// FMAs a clock and SM) five chunks of four rows took 8 us; 8 sequences of 2048
// chunks lose some 3.5 us to all of the exact ranking now.  The order of a sum is
// fixed: equal bounds tie.  (Four rows share the chunk's loads and overlap their
// sums: 0.5 us less there than row by row.)
constexpr int kExactRows = 4;
template <int D, int N>
__device__ __forceinline__ unsigned long long exact_rows(const uint16_t* q, const uint16_t* bounds, int lane) {
    float s[N], e[N];
#pragma unroll
    for (int r = 0; r < N; ++r) s[r] = e[r] = 0.f;
#pragma unroll
    for (int j = 0; j < D / 64; ++j) {
        const int d = 64 * j + 2 * lane;
        const float2 hi = __half22float2(*reinterpret_cast<const __half2*>(bounds + d));
        const float2 lo = __half22float2(*reinterpret_cast<const __half2*>(bounds + D + d));
#pragma unroll
        for (int r = 0; r < N; ++r) {
            const float2 x = __half22float2(*reinterpret_cast<const __half2*>(q + r * D + d));
            add_pair(s[r], e[r], __fmul_rn(x.x, x.x > 0.f ? hi.x : lo.x), 0.f);
            add_pair(s[r], e[r], __fmul_rn(x.y, x.y > 0.f ? hi.y : lo.y), 0.f);
        }
    }
    unsigned long long k = 0ull;
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1)
#pragma unroll
        for (int r = 0; r < N; ++r) {
            const float s2 = __shfl_xor_sync(kFull, s[r], off), e2 = __shfl_xor_sync(kFull, e[r], off);
            // the same pair order in both lanes, so that every lane ends with the same sum
            const bool up = (threadIdx.x & off) != 0;
            float a = up ? s2 : s[r], ae = up ? e2 : e[r];
            add_pair(a, ae, up ? s[r] : s2, up ? e[r] : e2);
            s[r] = a;
            e[r] = ae;
        }
#pragma unroll
    for (int r = 0; r < N; ++r) k = max(k, order_key((double)s[r] + (double)e[r]));
    return k;
}

// The same over rows [0, n) of q.
template <int D>
__device__ __forceinline__ unsigned long long exact_key(const uint16_t* q, int n, const uint16_t* bounds, int lane) {
    unsigned long long k = 0ull;
    int r = 0;
    for (; r + kExactRows <= n; r += kExactRows) k = max(k, exact_rows<D, kExactRows>(q + r * D, bounds, lane));
    for (; r < n; ++r) k = max(k, exact_rows<D, 1>(q + r * D, bounds, lane));
    return k;
}

// Block-wide sums of two counts (every thread gets them).
__device__ __forceinline__ uint2 sum2(SelShared& sh, uint32_t a, uint32_t b) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    a = __reduce_add_sync(kFull, a);
    b = __reduce_add_sync(kFull, b);
    __syncthreads();                      // earlier reads of red are done
    if (lane == 0) { sh.red[warp][0] = a; sh.red[warp][1] = b; }
    __syncthreads();
    uint2 t = make_uint2(0u, 0u);
#pragma unroll
    for (int w = 0; w < kSelWarps; ++w) { t.x += sh.red[w][0]; t.y += sh.red[w][1]; }
    return t;
}

// After a histogram: the bin that holds the `left`-th largest, its count and
// how many places are left inside it.
__device__ __forceinline__ void pick_bin(SelShared& sh, uint32_t left) {
    __syncthreads();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t c[kPerBin], sum = 0;         // thread 0 takes the largest bins
#pragma unroll
    for (int j = 0; j < kPerBin; ++j) {
        c[j] = sh.hist[kBins - 1 - (threadIdx.x * kPerBin + j)];
        sum += c[j];
    }
    uint32_t at = sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const uint32_t o = __shfl_up_sync(kFull, at, off);
        if (lane >= off) at += o;
    }
    if (lane == 31) sh.red[warp][0] = at;
    __syncthreads();
    for (int w = 0; w < warp; ++w) at += sh.red[w][0];
    at -= sum;                            // the larger bins' count
    if (at < left && at + sum >= left) {
#pragma unroll
        for (int j = 0; j < kPerBin; ++j) {
            if (at < left && at + c[j] >= left) {
                sh.bin = kBins - 1 - (threadIdx.x * kPerBin + j);
                sh.left = left - at;
                sh.in_bin = c[j];
            }
            at += c[j];
        }
    }
    __syncthreads();
}

// The `left`-th largest of the keys that are not kSure (at least `left` of them).
__device__ __forceinline__ uint32_t kth_key(SelShared& sh, const uint32_t* keys, int n, uint32_t left) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t lo = 0xffffffffu, hi = 0u;
    for (int j = threadIdx.x; j < n; j += kSelThreads)
        if (keys[j] != kSure) {
            lo = min(lo, keys[j]);
            hi = max(hi, keys[j]);
        }
    lo = __reduce_min_sync(kFull, lo);
    hi = __reduce_max_sync(kFull, hi);
    __syncthreads();
    if (lane == 0) { sh.red[warp][0] = lo; sh.red[warp][1] = hi; }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kSelWarps; ++w) { lo = min(lo, sh.red[w][0]); hi = max(hi, sh.red[w][1]); }
    uint32_t some = (uint32_t)n;          // keys within [lo, hi], at most
    while (lo != hi && some > (uint32_t)kFewTies) {
        // 2048 bins over [lo, hi]
        const int shift = max(0, 32 - __clz(hi - lo) - 11);
        __syncthreads();
        for (int j = threadIdx.x; j < kBins; j += kSelThreads) sh.hist[j] = 0u;
        __syncthreads();
        for (int j = threadIdx.x; j < n; j += kSelThreads) {
            const uint32_t k = keys[j];
            if (k != kSure && k >= lo && k <= hi) atomicAdd(&sh.hist[(k - lo) >> shift], 1u);
        }
        pick_bin(sh, left);
        left = sh.left;
        some = sh.in_bin;
        lo += sh.bin << shift;
        hi = min(hi, lo + ((1u << shift) - 1u));
    }
    if (lo == hi) return lo;
    // few keys left: their order by pairs
    if (threadIdx.x == 0) sh.n_list = 0u;
    __syncthreads();
    for (int j = threadIdx.x; j < n; j += kSelThreads) {
        const uint32_t k = keys[j];
        if (k != kSure && k >= lo && k <= hi) sh.list[atomicAdd(&sh.n_list, 1u)] = k;
    }
    __syncthreads();
    const uint32_t m = sh.n_list;
    for (uint32_t x = threadIdx.x; x < m; x += kSelThreads) {
        const uint32_t k = sh.list[x];
        uint32_t above = 0, same = 0;
        for (uint32_t y = 0; y < m; ++y) {
            above += sh.list[y] > k;
            same += sh.list[y] == k;
        }
        if (above < left && above + same >= left) sh.T = k;
    }
    __syncthreads();
    return sh.T;
}

template <int D>
__global__ void __launch_bounds__(kSelThreads) select_chunks_kernel(const ListParams p) {
    extern __shared__ __align__(16) uint32_t keys[];      // the first CTA's: one key per chunk
    __shared__ SelShared sh;
    __shared__ uint32_t wtop[kSelWarps][D / 2];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int cs = p.splits, rank = blockIdx.x % cs, pair = blockIdx.x / cs;
    const int i = pair / p.n_kv_heads, h = pair % p.n_kv_heads;
    // (the schedule's lists may be read before the dependency wait, as its plan is)
    const int off = p.list_off[i], n = p.list_off[i + 1] - off, K = p.top_k, G = p.group;
    if (cs > 1) cluster_arrive();                         // waited for before the first remote store
    asm volatile("griddepcontrol.wait;" ::: "memory");
    int32_t* out = p.lists + (size_t)pair * K;
    if (n <= K) {                                         // (the whole cluster: same n)
        if (rank == 0)
            for (int j = threadIdx.x; j < K; j += kSelThreads) out[j] = j < n ? j : -1;
        if (cs > 1) cluster_wait();
        return;
    }
    const uint16_t* q = p.q + ((size_t)i * p.n_heads + (size_t)h * G) * D;
    const int32_t* slots = p.list_slots + off;
    auto bounds_of = [&](int slot) {
        return p.bounds + (((size_t)slot * p.n_layers + p.layer) * p.n_kv_heads + h) * 2 * D;
    };
    const uint32_t keys0 = cs > 1 ? peer_addr(smem_u32(keys), 0) : 0u;
    const uint32_t abs0 = cs > 1 ? peer_addr(smem_u32(sh.top_abs), 0) : 0u;

    // each warp's own row of the largest |bound| per pair of dims (for E)
    for (int d = lane; d < D / 2; d += 32) wtop[warp][d] = 0u;
    __syncwarp();
    // scores of blocks of 16 chunks
    bool met = cs == 1;                                   // the first CTA's shared memory exists
    bool bad = false;
    for (int blk = rank * kSelWarps + warp; blk * 16 < n; blk += cs * kSelWarps) {
        const int c0 = blk * 16 + g, c1 = c0 + 8;
        int s0 = slots[min(c0, n - 1)], s1 = slots[min(c1, n - 1)];
        if (s0 < 0 || s0 >= p.capacity) { s0 = 0; bad = true; }
        if (s1 < 0 || s1 >= p.capacity) { s1 = 0; bad = true; }
        const uint4* b0 = reinterpret_cast<const uint4*>(bounds_of(s0)) + t;
        const uint4* b1 = reinterpret_cast<const uint4*>(bounds_of(s1)) + t;
        float best0 = __uint_as_float(0x7fffffffu), best1 = best0;   // NaN: a row that is not a number is passed over
        constexpr int J = D / 32;                         // 64-byte groups of a bounds row
        uint4 x0[2][J], x1[2][J];
#pragma unroll
        for (int part = 0; part < 2; ++part)
#pragma unroll
            for (int j = 0; j < J; ++j) {
                x0[part][j] = __ldg(b0 + part * (D / 8) + j * 4);
                x1[part][j] = __ldg(b1 + part * (D / 8) + j * 4);
            }
        for (int r0 = 0; r0 < G; r0 += 8) {
            float acc[4] = {0.f, 0.f, 0.f, 0.f};
            const uint4* qr = reinterpret_cast<const uint4*>(q + (size_t)min(r0 + g, G - 1) * D) + t;
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const uint4 y = __ldg(qr + j * 4);
#pragma unroll
                for (int part = 0; part < 2; ++part) {
                    const uint4 u = x0[part][j], w = x1[part][j];
                    const uint32_t a[4] = {u.x, w.x, u.y, w.y}, b[4] = {u.z, w.z, u.w, w.w};
                    mma16816(acc, a, part_f16x2(y.x, part == 0), part_f16x2(y.y, part == 0));
                    mma16816(acc, b, part_f16x2(y.z, part == 0), part_f16x2(y.w, part == 0));
                }
            }
            // rows past the group repeat its last one: they change no maximum
            best0 = fmaxf(best0, fmaxf(acc[0], acc[1]));
            best1 = fmaxf(best1, fmaxf(acc[2], acc[3]));
        }
        auto larger = [](uint32_t a, uint32_t b) {        // max(|a|, |b|) of fp16 pairs
            const __half2 m = __hmax2(__habs2(*reinterpret_cast<const __half2*>(&a)),
                                      __habs2(*reinterpret_cast<const __half2*>(&b)));
            return *reinterpret_cast<const uint32_t*>(&m);
        };
#pragma unroll
        for (int j = 0; j < J; ++j) {
            uint32_t m[4] = {larger(x0[0][j].x, x1[0][j].x), larger(x0[0][j].y, x1[0][j].y),
                             larger(x0[0][j].z, x1[0][j].z), larger(x0[0][j].w, x1[0][j].w)};
            m[0] = larger(m[0], larger(x0[1][j].x, x1[1][j].x));
            m[1] = larger(m[1], larger(x0[1][j].y, x1[1][j].y));
            m[2] = larger(m[2], larger(x0[1][j].z, x1[1][j].z));
            m[3] = larger(m[3], larger(x0[1][j].w, x1[1][j].w));
#pragma unroll
            for (int k = 0; k < 4; ++k) {
#pragma unroll
                for (int d = 4; d <= 16; d <<= 1) m[k] = larger(m[k], __shfl_xor_sync(kFull, m[k], d));
                uint32_t* to = &wtop[warp][j * 16 + t * 4 + k];
                if (g == 0) *to = larger(*to, m[k]);
            }
        }
#pragma unroll
        for (int d = 1; d <= 2; d <<= 1) {
            best0 = fmaxf(best0, __shfl_xor_sync(kFull, best0, d));
            best1 = fmaxf(best1, __shfl_xor_sync(kFull, best1, d));
        }
        if (!met) {
            cluster_wait();
            met = true;
        }
        if (t < 2) {
            const int c = t ? c1 : c0;
            const bool forced = c < p.sink || c >= n - p.recent;
            const uint32_t k = forced ? kSure : order_key(t ? best1 : best0);
            if (c < n) {
                if (cs > 1) st_peer(keys0 + 4u * (uint32_t)c, k);
                else keys[c] = k;
            }
        }
    }
    if (bad) set_status(p.status, CA_ERR_DEVICE_BOUNDS);
    if (!met) cluster_wait();
    __syncthreads();
    for (int d = threadIdx.x; d < D / 2; d += kSelThreads) {
        __half2 m = *reinterpret_cast<const __half2*>(&wtop[0][d]);
#pragma unroll
        for (int w = 1; w < kSelWarps; ++w) m = __hmax2(m, *reinterpret_cast<const __half2*>(&wtop[w][d]));
        const uint32_t bits = *reinterpret_cast<const uint32_t*>(&m);
        if (cs > 1) st_peer(abs0 + 4u * (uint32_t)(rank * 128 + d), bits);
        else sh.top_abs[0][d] = bits;
    }
    uint32_t q0[D / 64];                                  // the bound's first row (below), on its way meanwhile
#pragma unroll
    for (int j = 0; j < D / 64; ++j)
        q0[j] = *reinterpret_cast<const uint32_t*>(q + (size_t)min(warp, G - 1) * D + 64 * j + 2 * lane);
    if (cs > 1) {
        cluster_sync_all();
        if (rank != 0) return;
    } else {
        __syncthreads();
    }

    const uint32_t places = (uint32_t)(K - p.sink - p.recent);   // n > K >= sink + recent: they do not overlap
    uint32_t cut = kTie, ties = 0;                        // taken: keys above `cut`, and the first `ties` of kTie
    if (places > 0) {
        // E: with A the sum of |terms|, at most max over rows of sum_d |q_d| * (the largest |bound| of
        // dim d), each of the D / 8 steps of mma (16 exact products and the running sum, aligned and cut
        // at 2^-23 of the largest each, rounded once) is off by at most 18 * 2^-23 * A.  (A bound by the
        // largest |bound| of all dims would count a channel of large keys in every dim.)
        {
            __half2 m[D / 64];
#pragma unroll
            for (int j = 0; j < D / 64; ++j) {
                m[j] = *reinterpret_cast<const __half2*>(&sh.top_abs[0][j * 32 + lane]);
                for (int r = 1; r < cs; ++r)
                    m[j] = __hmax2(m[j], *reinterpret_cast<const __half2*>(&sh.top_abs[r][j * 32 + lane]));
            }
            float qs = 0.f;
            for (int r = warp; r < G; r += kSelWarps) {
                float s = 0.f;
#pragma unroll
                for (int j = 0; j < D / 64; ++j) {
                    if (r != warp)
                        q0[j] = *reinterpret_cast<const uint32_t*>(q + (size_t)r * D + 64 * j + 2 * lane);
                    const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&q0[j]));
                    const float2 b = __half22float2(m[j]);
                    s += fabsf(x.x) * b.x + fabsf(x.y) * b.y;
                }
#pragma unroll
                for (int o = 16; o >= 1; o >>= 1) s += __shfl_xor_sync(kFull, s, o);
                qs = s > qs || s != s ? s : qs;          // a NaN stays: no bound then
            }
            if (lane == 0) sh.qsum[warp] = qs;
        }
        const uint32_t kth = kth_key(sh, keys, n, places);
        float A = 0.f;
#pragma unroll
        for (int w = 0; w < kSelWarps; ++w) A = sh.qsum[w] > A || sh.qsum[w] != sh.qsum[w] ? sh.qsum[w] : A;
        const float E = A * ((D / 8) * 18.2f / 8388608.f);
        const float T = key_value(kth);
        uint32_t low = 0u, high = kTie - 1u;              // a band without bounds where E or T is not finite
        if (kth != 0u && E < 1e37f && fabsf(T) < 1e37f) {
            const float w = 2.01f * E + fabsf(T) * 1e-6f;
            low = max(order_key(T - w), 1u);
            high = order_key(T + w);
        }
        uint32_t above = 0, band = 0;
        for (int j = threadIdx.x; j < n; j += kSelThreads) {
            const uint32_t k = keys[j];
            above += k > high && k != kSure;
            band += k >= low && k <= high;
        }
        const uint2 c = sum2(sh, above, band);
        const uint32_t open = places - c.x;               // places left for the band
        cut = high;
        if (c.y == open) {
            // (low is at least 1 here: an unbounded band holds every chunk that is
            // not forced, and those are more than the places, as n > K)
            cut = low - 1u;
        } else if (E == 0.f) {                            // every score in the band is the same
            for (int j = threadIdx.x; j < n; j += kSelThreads)
                if (keys[j] >= low && keys[j] <= high) keys[j] = kTie;
            ties = open;
            cut = high;
        } else if (c.y <= (uint32_t)kFewTies) {
            if (threadIdx.x == 0) sh.n_list = 0u;
            for (int x = threadIdx.x; x < kFewTies; x += kSelThreads) sh.key64[x] = 0ull;
            __syncthreads();
            for (int j = threadIdx.x; j < n; j += kSelThreads)
                if (keys[j] >= low && keys[j] <= high) sh.list[atomicAdd(&sh.n_list, 1u)] = (uint32_t)j;
            __syncthreads();
            const uint32_t RB = (uint32_t)(G + kExactRows - 1) / kExactRows;
            for (uint32_t x = warp; x < c.y * RB; x += kSelWarps) {            // (rows, chunk) by (rows, chunk)
                const uint32_t e = x / RB, r = x % RB * kExactRows;
                const int s = slots[sh.list[e]];
                const unsigned long long k = exact_key<D>(q + (size_t)r * D, min(kExactRows, G - (int)r),
                                                          bounds_of(s >= 0 && s < p.capacity ? s : 0), lane);
                if (lane == 0) atomicMax(&sh.key64[e], k);
            }
            __syncthreads();
            for (uint32_t x = threadIdx.x; x < c.y; x += kSelThreads) {
                uint32_t before = 0;
                for (uint32_t y = 0; y < c.y; ++y)
                    before += sh.key64[y] > sh.key64[x] || (sh.key64[y] == sh.key64[x] && sh.list[y] < sh.list[x]);
                keys[sh.list[x]] = before < open ? kSure : 0u;
            }
        } else {
            // Many near-equal scores (contexts of equal chunks): a radix
            // selection over the 64-bit keys, computed anew for each digit.
            unsigned long long pre = 0;
            uint32_t rest = open;
            auto key_of = [&](int j) {
                const int s = slots[j];
                return exact_key<D>(q, G, bounds_of(s >= 0 && s < p.capacity ? s : 0), lane);
            };
            for (int shift = 56; shift >= 0; shift -= 8) {
                __syncthreads();
                for (int j = threadIdx.x; j < kBins; j += kSelThreads) sh.hist[j] = 0u;
                __syncthreads();
                for (int j = warp; j < n; j += kSelWarps) {
                    if (keys[j] < low || keys[j] > high) continue;
                    const unsigned long long k = key_of(j);
                    if (lane == 0 && (shift == 56 || (k >> (shift + 8)) == pre))
                        atomicAdd(&sh.hist[(k >> shift) & 255u], 1u);
                }
                pick_bin(sh, rest);
                pre = (pre << 8) | sh.bin;
                rest = sh.left;
            }
            for (int j = warp; j < n; j += kSelWarps) {
                const uint32_t k32 = keys[j];
                __syncwarp();
                if (k32 < low || k32 > high) continue;
                const unsigned long long k = key_of(j);
                if (lane == 0) keys[j] = k > pre ? kSure : k == pre ? kTie : 0u;
            }
            ties = rest;
        }
    }
    __syncthreads();

    // The taken chunks in ascending order: a thread counts its stretch, a scan
    // over the threads gives its first place, and it writes them.
    const int per = (n + kSelThreads - 1) / kSelThreads, j0 = min(n, (int)threadIdx.x * per), j1 = min(n, j0 + per);
    uint32_t took = 0, tied = 0;
    for (int j = j0; j < j1; ++j) {
        const uint32_t k = keys[j];
        tied += k == kTie;
        took += k > cut && k != kTie;
    }
    uint32_t a = took, b = tied;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const uint32_t x = __shfl_up_sync(kFull, a, d), y = __shfl_up_sync(kFull, b, d);
        if (lane >= d) { a += x; b += y; }
    }
    if (lane == 31) { sh.red[warp][0] = a; sh.red[warp][1] = b; }
    __syncthreads();
    a -= took;
    b -= tied;
    for (int w = 0; w < warp; ++w) { a += sh.red[w][0]; b += sh.red[w][1]; }
    for (int j = j0; j < j1; ++j) {
        const uint32_t k = keys[j];
        const bool tie = k == kTie, take = tie ? b < ties : k > cut;
        const uint32_t at = a + min(b, ties);
        if (take && at < (uint32_t)K) out[at] = j;
        a += take && !tie;
        b += tie;
    }
}

// ---------------------------------------------------------------------------
// Tiles of the three pool types as tensor core fragments, the products taken
// transposed (tokens on the rows, up to 8 NB query rows on the columns).
// `tok(g)`: the token of the block in fragment row g (g + 8: 8 further).
// `qdim(kk, t)`: first of a lane's dims of step kk, held in two registers
// (kPair: four consecutive dims, else two and the two 8 further).
// ---------------------------------------------------------------------------
template <int EB, int C, int D, int NB, bool FEW>
struct Frag;

template <int C, int D, int NB>
struct Frag<2, C, D, NB, false> {                       // fp16: ldmatrix from the swizzled tiles
    static constexpr int kStage = 4 * C * D;
    static constexpr bool kPair = false;
    __device__ static int tok(int g) { return g; }
    __device__ static int dim(int db, int half, int g) { return 16 * db + 8 * half + g; }
    __device__ static void scores(const uint8_t* st, int blk, const uint32_t (&qb)[NB][D / 16][2], float (&s)[NB][4],
                                  int lane) {
        const uint32_t kt = smem_u32(st);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) s[nb][0] = s[nb][1] = s[nb][2] = s[nb][3] = 0.f;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            uint32_t a[4];
            ldsm_x4(kt + swz(blk * 16 + (lane & 15), 2 * kk + (lane >> 4), C), a[0], a[1], a[2], a[3]);
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) mma16816(s[nb], a, qb[nb][kk][0], qb[nb][kk][1]);
        }
    }
    __device__ static void pv(const uint8_t* st, int blk, const uint32_t (&pb)[NB][2], float (&o)[NB][D / 16][4],
                              int lane) {
        const uint32_t vt = smem_u32(st) + 2 * C * D;
#pragma unroll
        for (int db = 0; db < D / 16; ++db) {
            uint32_t a[4];
            ldsm_x4_t(vt + swz(blk * 16 + (lane & 7) + ((lane >> 4) << 3), 2 * db + ((lane >> 3) & 1), C), a[0], a[1],
                      a[2], a[3]);
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) mma16816(o[nb][db], a, pb[nb][0], pb[nb][1]);
        }
    }
};

template <int C, int D, int NB>
struct Frag<1, C, D, NB, false> {                       // fp8: bytes widened into the fragments
    static_assert(D == 128, "fp8 pools have head_dim 128");
    static constexpr int kStage = 2 * C * D;
    static constexpr bool kPair = true;
    __device__ static int tok(int g) { return f4_token(g); }
    // O^T rows: dims 32 qd + 4g + 2e (row g) and one further (row g + 8), db = 2 qd + e
    __device__ static int dim(int db, int half, int g) { return 32 * (db >> 1) + 4 * g + 2 * (db & 1) + half; }
    __device__ static uint32_t word(const uint8_t* tile, int row, int chunk, int off) {
        return *reinterpret_cast<const uint32_t*>(tile + swz(row, chunk, C) + off);
    }
    __device__ static void scores(const uint8_t* st, int blk, const uint32_t (&qb)[NB][D / 16][2], float (&s)[NB][4],
                                  int lane) {
        const int g = lane >> 2, t = lane & 3, r0 = blk * 16 + tok(g), r1 = r0 + 8;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) s[nb][0] = s[nb][1] = s[nb][2] = s[nb][3] = 0.f;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t w0 = word(st, r0, kk, 4 * t), w1 = word(st, r1, kk, 4 * t);
            const uint32_t a[4] = {f16x2_from_e4m3x2(w0 & 0xffffu), f16x2_from_e4m3x2(w1 & 0xffffu),
                                   f16x2_from_e4m3x2(w0 >> 16), f16x2_from_e4m3x2(w1 >> 16)};
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) mma16816(s[nb], a, qb[nb][kk][0], qb[nb][kk][1]);
        }
    }
    __device__ static void pv(const uint8_t* st, int blk, const uint32_t (&pb)[NB][2], float (&o)[NB][D / 16][4],
                              int lane) {
        const int g = lane >> 2, t = lane & 3, t0 = blk * 16 + t;
        const uint8_t* vt = st + C * D;
#pragma unroll
        for (int qd = 0; qd < D / 32; ++qd) {
            const int kc = 2 * qd + (g >> 2), off = 4 * (g & 3);
            const uint32_t a = word(vt, t0, kc, off), b = word(vt, t0 + 4, kc, off);
            const uint32_t c = word(vt, t0 + 8, kc, off), d = word(vt, t0 + 12, kc, off);
            const uint32_t ab0 = __byte_perm(a, b, 0x5140), cd0 = __byte_perm(c, d, 0x5140);
            const uint32_t ab1 = __byte_perm(a, b, 0x7362), cd1 = __byte_perm(c, d, 0x7362);
            const uint32_t x[4] = {f16x2_from_e4m3x2(ab0 & 0xffffu), f16x2_from_e4m3x2(ab0 >> 16),
                                   f16x2_from_e4m3x2(cd0 & 0xffffu), f16x2_from_e4m3x2(cd0 >> 16)};
            const uint32_t y[4] = {f16x2_from_e4m3x2(ab1 & 0xffffu), f16x2_from_e4m3x2(ab1 >> 16),
                                   f16x2_from_e4m3x2(cd1 & 0xffffu), f16x2_from_e4m3x2(cd1 >> 16)};
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                mma16816(o[nb][2 * qd], x, pb[nb][0], pb[nb][1]);
                mma16816(o[nb][2 * qd + 1], y, pb[nb][0], pb[nb][1]);
            }
        }
    }
};

template <int C, int D, int NB, bool FEW>
struct Frag<0, C, D, NB, FEW> {                  // fp4
    static constexpr int kStage = F4Tile<C, D>::kBytes;
    static constexpr bool kPair = true;
    __device__ static int tok(int g) { return f4_token(g); }
    __device__ static int dim(int db, int half, int g) { return 16 * db + 2 * g + half; }
    __device__ static void scores(const uint8_t* st, int blk, const uint32_t (&qb)[NB][D / 16][2], float (&s)[NB][4],
                                  int lane) {
        f4_scores<C, D, NB, FEW>(st, blk, qb, s, lane);
    }
    __device__ static void pv(const uint8_t* st, int blk, const uint32_t (&pb)[NB][2], float (&o)[NB][D / 16][4],
                              int lane) {
        f4_pv<C, D, NB>(st, blk, pb, o, lane);
    }
};

// ---------------------------------------------------------------------------
// Attention over listed chunks.  A unit is one (sequence, key/value head, up to
// 8 NB rows of its group) with its top_k list entries; the units' entries are
// laid end to end and cut into equal stretches, one per resident CTA, so every
// CTA streams the same number of tiles whatever the batch.  (Clusters of up to
// eight CTAs per unit took 75 us where the stretches took 69, with the same
// code for a tile: 512 units of 64 fp4 tiles on 456 resident CTAs.)  A producer warp looks 32 entries up at once (list ->
// slot -> token count) and keeps a ring of tiles in flight, across units; the
// consumer warps take the tiles' blocks of 16 tokens with an online softmax.
// Each ring slot belongs to the warps of one group, a warp per block of a tile.
// Units of 64 tiles of 64 tokens, head_dim 128: 128 of fp16 46 us, 88% of the
// copy rate, bound by DRAM; 128 of fp8 30 us (67%), two CTAs per SM at 162
// registers, whose word loads and byte permutes bring two tokens beside each
// other for every 32 dims; 512 of fp4 59 us (77%),
// bound by the instructions that widen a tile (55% of the issue slots, 50% of
// the ALU) in the shadow of its loads: three CTAs per SM hide most of them
// (three of four warps and two of eight 69 us before the values' codes lay in
// pairs, four of four 70, one of twelve 83).
// A unit cut between CTAs leaves its pieces' partial triples in the schedule's
// buffer, and the CTA that finishes its last piece (a counter per unit, which
// it clears again) merges them in the order of the pieces: nothing waits, and
// results do not depend on the order of arrival.  One warp sees to that while
// the others go on with the next unit; all four at the end of the stretch.
//
// A consumer whose wait for a tile runs out reports it and waits for no tile
// any more, but goes through the rest of its CTA's pieces with the others: the
// named barriers at a piece's end count all four warps and have no limit of
// their own.  So each warp gives up once at most, the CTA ends within a few of
// the waits' limits, and the units' counters end at 0 as always; the outputs
// of its units are undefined.
// ---------------------------------------------------------------------------
constexpr int kSpWarps = 4, kSpThreads = 32 * (kSpWarps + 1), kSpStages = 12;
// The softmax reference is kept 5 below a running maximum and raised only when
// a score passes it by 13: the weights stay below 2^13 in their fp16 operand
// and normal numbers down to 2^-19 (or less) of the largest.  They are rounded for
// the product with the values alone (2^-11 of each, so at most 2^-11 * sum p|v| of
// an output); their sum is of the unrounded ones, in fp32.
constexpr float kSpLift = 5.f, kSpSlack = 8.f;

template <int EB, int C, int D, int NB, bool FEW>
struct SpShared {
    using F = Frag<EB, C, D, NB, FEW>;
    static constexpr int kGroups = kSpWarps / (C / 16);           // of warps; the ring is a multiple of them
    static constexpr int kPerSm = EB == 0 && NB == 1 ? 3 : 2;     // resident CTAs
    static constexpr int kRows = 8 * NB;
    static constexpr int kRow = D + 4;                            // floats: no bank conflicts between rows
    static constexpr int kExch = (kSpWarps - 1) * kRows * kRow * 4;   // outputs of warps 1, 2, 3
    // stage bars, token counts, (m, s) of the warps, a flag
    static constexpr int kTail = 2 * kSpStages * 8 + kSpStages * 4 + kSpWarps * kRows * 2 * 4 + 16;
    static constexpr size_t bytes(int stages) { return (size_t)stages * F::kStage + kExch + kTail; }
};

__device__ __forceinline__ void sp_consumers() { asm volatile("bar.sync 1, %0;" ::"n"(kSpWarps * 32) : "memory"); }

// Entries [first, last) of CTA c when `total` are cut into `grid` stretches.
__device__ __forceinline__ long long cut_at(long long total, int grid, int c) { return total * c / grid; }

template <int EB, int C, int D, int NB, bool FEW>
__global__ void __launch_bounds__(kSpThreads, SpShared<EB, C, D, NB, FEW>::kPerSm)
sparse_attention_kernel(const __grid_constant__ CUtensorMap tmap, const ListParams p) {
    using F = Frag<EB, C, D, NB, FEW>;
    using SM = SpShared<EB, C, D, NB, FEW>;
    // FEW (up to 4 rows): row r is in columns 2r and 2r + 1, one row for a lane
    constexpr int NR = FEW ? 1 : 2;                        // query rows among a lane's two columns
    constexpr int R = SM::kRows, NBLK = C / 16, RS = SM::kRow, W = kSpWarps, NG = SM::kGroups;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int S = p.n_stages;
    float* exch = reinterpret_cast<float*>(smem + (size_t)S * F::kStage);
    uint64_t* bars = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(exch) + SM::kExch);
    volatile int32_t* stage_ntok = reinterpret_cast<volatile int32_t*>(bars + 2 * kSpStages);
    float* wms = const_cast<float*>(reinterpret_cast<volatile float*>(stage_ntok + kSpStages));   // [warp][row][m, s]
    volatile int32_t* flag = reinterpret_cast<volatile int32_t*>(wms + W * R * 2);
    const uint32_t full0 = smem_u32(bars), empty0 = smem_u32(bars + kSpStages);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if ((smem_u32(smem) & 1023u) != 0 || S < NG || S > kSpStages || S % NG) {   // the same in every CTA
        asm volatile("griddepcontrol.wait;" ::: "memory");
        if (threadIdx.x == 0) set_status(p.status, CA_ERR_INVALID);
        return;
    }
    if (threadIdx.x == 0) {
        for (int k = 0; k < S; ++k) {
            mbar_init(full0 + 8 * k, 1);
            mbar_init(empty0 + 8 * k, NBLK);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    __syncthreads();
    const int G = p.group, RB = (G + R - 1) / R, K = p.top_k, HK = p.n_kv_heads, grid = gridDim.x;
    const long long total = (long long)p.n_units * K;
    const long long e0 = cut_at(total, grid, blockIdx.x), e1 = cut_at(total, grid, blockIdx.x + 1);
    // unit u: row block u % RB of head (u / RB) % HK of batch row u / (RB * HK)

    if (warp == W) {
        // ------------------------------ producer ------------------------------
        const uint64_t pol = policy_evict_first();
        if (p.test_stall && !(blockIdx.x & 1)) {
            // Test hook (ca_sched_inject_stall): no tile is copied, and of several
            // groups the first alone is told that its piece ends, so that it stands
            // at the piece's barriers while the others' waits run out.
            asm volatile("griddepcontrol.wait;" ::: "memory");
            if (lane == 0) {
                if (NG > 1) {
                    stage_ntok[0] = -1;
                    mbar_arrive(full0);
                }
                if (!mbar_wait(full0 + 8 * (NG > 1), 0u)) set_status(p.status, CA_ERR_TIMEOUT);
            }
            return;
        }
        int st = 0, done = 0;                              // ring slot; slots filled so far
        uint32_t ph = 1u;                                  // the empty barriers' phase: free at first
        bool ok = true;
        auto take = [&](int slot, uint32_t phase) -> bool {
            if (mbar_wait(empty0 + 8 * slot, phase)) return true;
            set_status(p.status, CA_ERR_TIMEOUT);
            return false;
        };
        auto step = [&](int n) {
            done += n;
            if ((st += n) >= S) {
                st -= S;
                ph ^= 1u;
            }
        };
        for (long long e = e0; e < e1 && ok;) {
            const int u = (int)(e / K), pair = u / RB, h = pair % HK, i = pair / HK;
            const int j1 = (int)min((long long)K, e1 - (long long)u * K);
            const int off = p.list_off[i], n = p.list_off[i + 1] - off;
            const int32_t* list = p.lists + (size_t)pair * K;
            // Only a context's last chunk can be partial.  (The schedule's
            // lists may be read before the dependency wait, as its plan is;
            // token counts, the caller's lists and the pool after it.)
            const int end_slot = p.list_slots[off + n - 1];
            if (e == e0) asm volatile("griddepcontrol.wait;" ::: "memory");
            const int end_ntok = end_slot >= 0 && end_slot < p.capacity ? min(max(p.slot_ntok[end_slot], 0), C) : 0;
            for (int j0 = (int)(e - (long long)u * K); j0 < j1 && ok; j0 += 32) {
                int slot = -1, ntok = 0;
                if (j0 + lane < j1) {
                    const int j = list[j0 + lane];
                    if (j >= n) {
                        set_status(p.status, CA_ERR_DEVICE_BOUNDS);
                    } else if (j >= 0) {
                        slot = p.list_slots[off + j];
                        if (slot < 0 || slot >= p.capacity) set_status(p.status, CA_ERR_DEVICE_BOUNDS);
                        else ntok = j == n - 1 ? end_ntok : C;
                    }
                }
                // The lanes that hold a tile take the next ring slots in their
                // order, a third of the ring at a time (one lane at a time was
                // too slow for 16-token tiles), each waiting for its own.
                uint32_t todo = __ballot_sync(kFull, ntok > 0);
                while (todo && ok) {
                    const int r = __popc(todo & ((1u << lane) - 1u)), some = min(__popc(todo), max(1, S / 3));
                    const bool mine = (todo >> lane & 1u) && r < some;
                    bool good = true;
                    if (mine) {
                        const int sl = st + r < S ? st + r : st + r - S;
                        good = take(sl, st + r < S ? ph : ph ^ 1u);
                        if (good) {
                            const uint32_t fb = full0 + 8 * sl, dst = smem_u32(smem) + sl * F::kStage;
                            mbar_expect_tx_only(fb, F::kStage);
                            if constexpr (EB == 0) {
                                bulk_load(dst, p.kv + (((long long)slot * p.n_layers + p.layer) * HK + h) * F::kStage,
                                          F::kStage, fb, pol);
                            } else {
                                const int rowK = (((slot * p.n_layers + p.layer) * 2) * HK + h) * C;
                                const int rowV = rowK + HK * C;
#pragma unroll
                                for (int bx = 0; bx < D * EB / 128; ++bx) {
                                    tma_load_2d(dst + bx * C * 128, &tmap, bx * (128 / EB), rowK, fb, pol);
                                    tma_load_2d(dst + F::kStage / 2 + bx * C * 128, &tmap, bx * (128 / EB), rowV, fb,
                                                pol);
                                }
                            }
                            stage_ntok[sl] = ntok;
                            mbar_arrive(fb);
                        }
                    }
                    ok = __all_sync(kFull, good);
                    todo &= ~__ballot_sync(kFull, mine);
                    step(some);
                }
            }
            for (int k = 0; k < NG && ok; ++k) {           // the piece ends: a slot without data for each group
                if (lane == 0) {
                    ok = take(st, ph);
                    if (ok) {
                        stage_ntok[st] = -1;
                        mbar_arrive(full0 + 8 * st);
                    }
                }
                ok = __shfl_sync(kFull, (int)ok, 0) != 0;
                step(1);
            }
            e = (long long)u * K + j1;
        }
        if (!ok && lane == 0)                              // copies in flight get a bounded chance to land
            for (int k = max(0, done - S); k < done; ++k)
                mbar_wait(full0 + 8 * (k % S), (uint32_t)(k / S) & 1u);
        return;
    }

    // ------------------------------ consumers ------------------------------
    asm volatile("griddepcontrol.wait;" ::: "memory");
    int st = warp / NBLK;                                  // the warp's next slot: its group's
    const int blk = warp % NBLK;                           // its block of that group's tiles
    uint32_t ph = 0u;
    // (the test hook's other half, in CTAs of odd number: one warp of the four
    // gives up while its tiles come)
    bool alive = !(p.test_stall && (blockIdx.x & 1) && warp == 0);
    if (!alive) set_status(p.status, CA_ERR_TIMEOUT);
    // (every piece moves the ring on by its tiles and a slot for each group, so
    // the groups' turns shift from piece to piece; a group's own slots do not)
    for (long long e = e0; e < e1;) {
        const int u = (int)(e / K), pair = u / RB, rb = u % RB, h = pair % HK, i = pair / HK;
        const long long u0 = (long long)u * K, end = min(u0 + K, e1);
        const bool whole = e == u0 && end == u0 + K;
        const int rows = min(R, G - rb * R);
        const size_t row0 = (size_t)i * p.n_heads + h * G + rb * R;      // the unit's first row of q and out
        uint32_t qb[NB][D / 16][2];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            const int r = FEW ? g >> 1 : nb * 8 + g;
            const bool there = r < rows;
            const uint16_t* q = p.q + (row0 + (there ? r : 0)) * D;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                uint2 x = make_uint2(0u, 0u);
                if (there) {
                    if constexpr (F::kPair) {
                        x = *reinterpret_cast<const uint2*>(q + 16 * kk + 4 * t);
                    } else {
                        x.x = *reinterpret_cast<const uint32_t*>(q + 16 * kk + 2 * t);
                        x.y = *reinterpret_cast<const uint32_t*>(q + 16 * kk + 2 * t + 8);
                    }
                }
                qb[nb][kk][0] = x.x;
                qb[nb][kk][1] = x.y;
            }
        }
        float o[NB][D / 16][4], m[NB][2], s[NB][2];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            m[nb][0] = m[nb][1] = -INFINITY;
            s[nb][0] = s[nb][1] = 0.f;
#pragma unroll
            for (int db = 0; db < D / 16; ++db) o[nb][db][0] = o[nb][db][1] = o[nb][db][2] = o[nb][db][3] = 0.f;
        }
        for (bool more = alive; more;) {
            if (!warp_wait(full0 + 8 * st, ph)) {
                set_status(p.status, CA_ERR_TIMEOUT);
                alive = false;
                break;
            }
            const int ntok = stage_ntok[st];
            more = ntok >= 0;
            if (blk * 16 < ntok) {
                const uint8_t* tile = smem + (size_t)st * F::kStage;
                float x[NB][4];
                F::scores(tile, blk, qb, x, lane);
                const int tk = blk * 16 + F::tok(g);
                const bool in0 = tk < ntok, in1 = tk + 8 < ntok;
                bool grow = false;
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
                    for (int k = 0; k < 4; k += 3 - NR) {
                        x[nb][k] = ((k >> 1) ? in1 : in0) ? x[nb][k] * p.scale_log2 : -INFINITY;
                        grow = grow || x[nb][k] > m[nb][k & 1] + (kSpLift + kSpSlack);
                    }
                }
                if (__any_sync(kFull, grow)) {
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                        for (int r = 0; r < NR; ++r) {
                            float mx = fmaxf(x[nb][r], x[nb][r + 2]);
#pragma unroll
                            for (int d = 4; d <= 16; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, d));
                            const float mn = fmaxf(m[nb][r], mx - kSpLift);
                            const float al = mn == -INFINITY ? 1.f : ex2(m[nb][r] - mn);
                            m[nb][r] = mn;
                            s[nb][r] *= al;
#pragma unroll
                            for (int db = 0; db < D / 16; ++db) {
                                o[nb][db][r] *= al;
                                o[nb][db][r + 2] *= al;
                            }
                        }
                }
                uint32_t pb[NB][2];
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                    // (the sums are of the lane's tokens, until the piece ends)
                    const float u0_ = m[nb][0] == -INFINITY ? 0.f : m[nb][0];
                    const float p0 = ex2(x[nb][0] - u0_), p2 = ex2(x[nb][2] - u0_);
                    float p1 = p0, p3 = p2;
                    s[nb][0] += p0 + p2;
                    if constexpr (!FEW) {
                        const float u1_ = m[nb][1] == -INFINITY ? 0.f : m[nb][1];
                        p1 = ex2(x[nb][1] - u1_);
                        p3 = ex2(x[nb][3] - u1_);
                        s[nb][1] += p1 + p3;
                    }
                    pb[nb][0] = movm_trans(pack_half2(p0, p1));
                    pb[nb][1] = movm_trans(pack_half2(p2, p3));
                }
                F::pv(tile, blk, pb, o, lane);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(empty0 + 8 * st);
            if ((st += NG) >= S) {
                st -= S;
                ph ^= 1u;
            }
        }
        // The warps' states meet: warps 1 to 3 hand theirs to warp 0, which
        // leaves the sum in the exchange area for all of them to write out
        // (three copies there leave room for a third tile of 32 KB).
        auto row_of = [&](int nb, int r) { return FEW ? t : nb * 8 + 2 * t + r; };
        auto put = [&](float* dst) {                       // [row][D] with the rows' stride
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int db = 0; db < D / 16; ++db)
#pragma unroll
                    for (int k = 0; k < 4; k += 3 - NR)
                        dst[row_of(nb, k & 1) * RS + F::dim(db, k >> 1, g)] = o[nb][db][k];
        };
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int r = 0; r < NR; ++r)
#pragma unroll
                for (int d = 4; d <= 16; d <<= 1) s[nb][r] += __shfl_xor_sync(kFull, s[nb][r], d);
        sp_consumers();                                 // the last piece has been written out
        if (warp > 0) {
            put(exch + (size_t)(warp - 1) * R * RS);
            if (g == 0)
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int r = 0; r < NR; ++r)
                        *reinterpret_cast<float2*>(wms + (warp * R + row_of(nb, r)) * 2) =
                            make_float2(m[nb][r], s[nb][r]);
        }
        sp_consumers();
        if (warp == 0) {
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int r = 0; r < NR; ++r) {
                    const int row = row_of(nb, r);
                    float2 q[W - 1];
                    float M = m[nb][r];
#pragma unroll
                    for (int k = 1; k < W; ++k) {
                        q[k - 1] = *reinterpret_cast<const float2*>(wms + (k * R + row) * 2);
                        M = fmaxf(M, q[k - 1].x);
                    }
                    const float a0 = m[nb][r] == -INFINITY ? 0.f : ex2(m[nb][r] - M);
                    float sum = s[nb][r] * a0;
#pragma unroll
                    for (int db = 0; db < D / 16; ++db) {
                        o[nb][db][r] *= a0;
                        o[nb][db][r + 2] *= a0;
                    }
#pragma unroll
                    for (int k = 1; k < W; ++k) {
                        const float ak = q[k - 1].x == -INFINITY ? 0.f : ex2(q[k - 1].x - M);
                        sum += q[k - 1].y * ak;
                        const float* src = exch + ((size_t)(k - 1) * R + row) * RS;
#pragma unroll
                        for (int db = 0; db < D / 16; ++db) {
                            o[nb][db][r] += ak * src[F::dim(db, 0, g)];
                            o[nb][db][r + 2] += ak * src[F::dim(db, 1, g)];
                        }
                    }
                    if (g == 0) *reinterpret_cast<float2*>(wms + row * 2) = make_float2(M, sum);
                }
            __syncwarp();
            put(exch);
        }
        sp_consumers();
        const int c = blockIdx.x;
        float* part = p.parts + (size_t)(2 * c + (e != e0)) * R * (D + 2);
        for (int idx = threadIdx.x; idx < rows * (D / 4); idx += W * 32) {
            const int row = idx / (D / 4), d4 = idx % (D / 4);
            const float4 v = reinterpret_cast<const float4*>(exch + row * RS)[d4];
            const float2 q = *reinterpret_cast<const float2*>(wms + row * 2);
            if (whole) {
                const float inv = q.y > 0.f ? p.out_scale / q.y : 0.f;
                *reinterpret_cast<uint2*>(p.out + (row0 + row) * D + d4 * 4) =
                    make_uint2(pack_half2(v.x * inv, v.y * inv), pack_half2(v.z * inv, v.w * inv));
            } else {
                reinterpret_cast<float4*>(part + R * 2)[row * (D / 4) + d4] = v;
                if (d4 == 0) reinterpret_cast<float2*>(part)[row] = q;
            }
        }
        // The last warp sees to a piece that is not a whole unit (the others have
        // arrived when their stores are out; the ring's slack covers its
        // detour), with all the others where nothing follows.
        if (!whole) {
            const bool over = end == e1;
            if (warp < W - 1) {
                asm volatile("bar.arrive 2, %0;" ::"n"(W * 32) : "memory");
                if (!over) {
                    e = end;
                    continue;
                }
            } else {
                asm volatile("bar.sync 2, %0;" ::"n"(W * 32) : "memory");
            }
            // the unit's pieces lie in CTAs c0 .. c1; the last to arrive merges
            int c0 = (int)((u0 * grid) / total), c1 = (int)(((u0 + K - 1) * grid) / total), last = 0;
            while (cut_at(total, grid, c0 + 1) <= u0) ++c0;
            while (cut_at(total, grid, c1 + 1) <= u0 + K - 1) ++c1;
            if (warp == W - 1) {
                if (lane == 0) {
                    __threadfence();
                    last = atomicAdd(p.counters + u, 1) == c1 - c0;
                    if (last) p.counters[u] = 0;
                    __threadfence();
                    *flag = last;
                }
                last = __shfl_sync(kFull, last, 0);
            }
            if (over) {
                sp_consumers();
                last = *flag;
            }
            if (last) {
                const int first = over ? threadIdx.x : lane, stride = over ? W * 32 : 32;
                for (int idx = first; idx < rows * (D / 4); idx += stride) {
                    const int row = idx / (D / 4), d4 = idx % (D / 4);
                    float M = -INFINITY, sum = 0.f;
                    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
                    constexpr int KB = 4;                  // pieces whose loads are in flight together
                    for (int k0 = c0; k0 <= c1; k0 += KB) {
                        float2 q[KB];
                        float4 v[KB];
                        float mn = M;
#pragma unroll
                        for (int k = 0; k < KB; ++k) {
                            const int cc = min(k0 + k, c1);
                            const float* src =
                                p.parts + (size_t)(2 * cc + (cut_at(total, grid, cc) < u0)) * R * (D + 2);
                            q[k] = __ldcg(reinterpret_cast<const float2*>(src) + row);
                            v[k] = __ldcg(reinterpret_cast<const float4*>(src + R * 2) + row * (D / 4) + d4);
                        }
#pragma unroll
                        for (int k = 0; k < KB; ++k) mn = fmaxf(mn, q[k].x);
                        const float mu = mn == -INFINITY ? 0.f : mn, wa = ex2(M - mu);
                        M = mn;
                        sum *= wa;
                        acc.x *= wa; acc.y *= wa; acc.z *= wa; acc.w *= wa;
#pragma unroll
                        for (int k = 0; k < KB; ++k) {
                            const float w = k0 + k <= c1 ? ex2(q[k].x - mu) : 0.f;
                            sum += q[k].y * w;
                            acc.x += v[k].x * w; acc.y += v[k].y * w; acc.z += v[k].z * w; acc.w += v[k].w * w;
                        }
                    }
                    const float inv = sum > 0.f ? p.out_scale / sum : 0.f;
                    *reinterpret_cast<uint2*>(p.out + (row0 + row) * D + d4 * 4) =
                        make_uint2(pack_half2(acc.x * inv, acc.y * inv), pack_half2(acc.z * inv, acc.w * inv));
                }
            }
        }
        e = end;
    }
}

}  // namespace dev

namespace {

constexpr int32_t kMostChunks = 49152;    // keys of one context in a CTA's shared memory (192 KB)

dev::ListParams list_params(const Pool& p, const Sched& s, int32_t layer, const void* q, int32_t top_k) {
    unsigned char* dev = static_cast<unsigned char*>(s.dev);
    const PoolCfg& c = p.cfg;
    dev::ListParams a{};
    a.q = static_cast<const uint16_t*>(q);
    a.list_off = reinterpret_cast<const int32_t*>(dev + s.layout.list_off);
    a.list_slots = reinterpret_cast<const int32_t*>(dev + s.layout.list_slots);
    a.kv = static_cast<const uint8_t*>(p.kv);
    a.slot_ntok = reinterpret_cast<const int32_t*>(a.kv + pool_tile_bytes(c));
    a.bounds = reinterpret_cast<const uint16_t*>(a.kv + pool_bounds_offset(c));
    a.status = reinterpret_cast<int32_t*>(dev + s.layout.status);
    a.n_layers = c.n_layers;
    a.n_kv_heads = kv_heads(c);
    a.n_heads = c.n_heads;
    a.group = c.n_heads / a.n_kv_heads;
    a.layer = layer;
    a.capacity = c.capacity_slots;
    a.top_k = top_k;
    return a;
}

// One launch of `blocks` clusters of `cs` CTAs, a programmatic dependent of
// the work before it (the kernels wait for that before they read or write what
// it may have written).
int launch(const void* fn, unsigned blocks, int cs, int threads, size_t smem, void** args, cudaStream_t stream) {
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cs;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks * (unsigned)cs);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = cs > 1 ? 2 : 1;
    if (cudaLaunchKernelExC(&cfg, fn, args) != cudaSuccess) return CA_ERR_CUDA;
    count_launch();
    return CA_OK;
}

struct SparseKernel {
    const void* fn = nullptr;
    int rows = 0, stage = 0, fixed = 0;      // rows of a unit; bytes of a stage, of the rest
    int groups = 0, per_sm = 0;              // the ring's slots come in multiples of `groups`; CTAs per SM
};
template <int EB, int C, int D, int NB, bool FEW = false>
SparseKernel sparse_of() {
    using SM = dev::SpShared<EB, C, D, NB, FEW>;
    return {reinterpret_cast<const void*>(&dev::sparse_attention_kernel<EB, C, D, NB, FEW>), SM::kRows, SM::F::kStage,
            (int)SM::bytes(0), SM::kGroups, SM::kPerSm};
}
// Rows of a group per CTA: 8, or 16 for groups of more (at head_dim 256 the
// accumulators of 16 rows do not fit the registers).  In an fp4 pool, which is
// bound by instructions, up to 4 rows lie twice in the 8 columns and a lane's
// softmax is of one row, not two: 512 units of 64 tiles 58.8 us for 62.3 with
// one row, 57.8 for 62.3 with four (an fp8 pool gains 1%, and has no such form).
template <int EB, int C, int D>
SparseKernel pick_rows(int group) {
    if constexpr (D <= 128) {
        if (group > 8) return sparse_of<EB, C, D, 2>();
    }
    if constexpr (EB == 0) {
        if (group <= 4) return sparse_of<EB, C, D, 1, true>();
    }
    return sparse_of<EB, C, D, 1>();
}
template <int EB, int D>
SparseKernel pick_sparse(const PoolCfg& c) {
    const int G = c.n_heads / kv_heads(c);
    if (c.chunk == 16) return pick_rows<EB, 16, D>(G);
    if (c.chunk == 32) return pick_rows<EB, 32, D>(G);
    if constexpr (D <= 128) {
        if (c.chunk == 64) return pick_rows<EB, 64, D>(G);
    }
    return {};
}
SparseKernel pick_sparse(const PoolCfg& c) {
    switch (kv_elem_bytes(c)) {
        case 0: return c.head_dim == 64 ? pick_sparse<0, 64>(c) : pick_sparse<0, 128>(c);
        case 1: return pick_sparse<1, 128>(c);
        default:
            return c.head_dim == 64 ? pick_sparse<2, 64>(c) : c.head_dim == 128 ? pick_sparse<2, 128>(c)
                                                                               : pick_sparse<2, 256>(c);
    }
}

// The ring: what the resident CTAs (two or three per SM) leave room for.
int sparse_stages(const SparseKernel& k, size_t* smem) {
    const size_t room = (size_t)(k.per_sm == 2 ? 113 : 75) * 1024;
    int st = dev::kSpStages / k.groups * k.groups;
    while (st > k.groups && (size_t)st * k.stage + k.fixed > room) st -= k.groups;
    *smem = (size_t)st * k.stage + k.fixed;
    return st;
}

const void* select_fn(const PoolCfg& c) {
    return c.head_dim == 64    ? reinterpret_cast<const void*>(&dev::select_chunks_kernel<64>)
           : c.head_dim == 128 ? reinterpret_cast<const void*>(&dev::select_chunks_kernel<128>)
                               : reinterpret_cast<const void*>(&dev::select_chunks_kernel<256>);
}

}  // namespace

int launch_select(const Pool& p, const Sched& s, int32_t layer, const void* q, int32_t top_k, int32_t sink,
                  int32_t recent, int32_t* lists, void* stream) {
    if (s.t.list_max > kMostChunks) return CA_ERR_UNSUPPORTED;
    dev::ListParams a = list_params(p, s, layer, q, top_k);
    a.lists = lists;
    a.sink = sink;
    a.recent = recent;
    const int pairs = s.t.b * a.n_kv_heads, sms = p.sms;
    // More CTAs per pair while all are resident at once (two per SM) and each warp still has a block of 16 chunks.
    int cs = 1;
    while (cs < 8 && pairs * cs * 2 <= 2 * sms && cs * dev::kSelWarps * 16 < s.t.list_max) cs *= 2;
    a.splits = cs;
    const size_t smem = (size_t)s.t.list_max * 4;
    void* args[] = {&a};
    return launch(select_fn(p.cfg), (unsigned)pairs, cs, dev::kSelThreads, smem, args, static_cast<cudaStream_t>(stream));
}

int launch_sparse(const Pool& p, const Sched& s, int32_t layer, const void* q, const int32_t* lists, int32_t top_k,
                  void* out, float scale, void* stream) {
    const SparseKernel k = pick_sparse(p.cfg);
    if (!k.fn) return CA_ERR_UNSUPPORTED;
    dev::ListParams a = list_params(p, s, layer, q, top_k);
    a.lists = const_cast<int32_t*>(lists);
    a.out = static_cast<uint16_t*>(out);
    const bool quant = (p.cfg.flags & (CA_KV_FP8 | CA_KV_FP4)) != 0;
    a.scale_log2 = scale * 1.4426950408889634f * (quant ? kv_scale_of(p.cfg.k_scale) : 1.f);
    a.out_scale = quant ? kv_scale_of(p.cfg.v_scale) : 1.f;
    a.n_units = s.t.b * a.n_kv_heads * ((a.group + k.rows - 1) / k.rows);
    a.counters = reinterpret_cast<int32_t*>(static_cast<unsigned char*>(s.dev) + s.layout.list_count);
    a.parts = static_cast<float*>(s.list_parts);
    size_t smem;
    a.n_stages = sparse_stages(k, &smem);
    if (s.stall_calls > 0) {
        a.test_stall = 1;
        --s.stall_calls;
    }
    // Two entries per CTA at least: a piece costs its queries, a partial and a place in the merge.
    const int64_t entries = (int64_t)a.n_units * top_k;
    const int grid = (int)std::min<int64_t>((int64_t)k.per_sm * p.sms, (entries + 1) / 2);
    void* args[] = {const_cast<unsigned char*>(p.tmap), &a};
    return launch(k.fn, (unsigned)grid, 1, dev::kSpThreads, smem, args, static_cast<cudaStream_t>(stream));
}

// Once per pool, when a schedule is built with chunk lists (outside stream
// capture): the kernels' shared-memory limits, which load them too.  Every pool
// asks the same of a kernel.
int prepare_lists(Pool& p) {
    if (p.lists_ready) return CA_OK;
    const SparseKernel k = pick_sparse(p.cfg);
    if (!k.fn) return CA_ERR_UNSUPPORTED;
    size_t smem;
    sparse_stages(k, &smem);
    if (cudaFuncSetAttribute(k.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess ||
        cudaFuncSetAttribute(select_fn(p.cfg), cudaFuncAttributeMaxDynamicSharedMemorySize, kMostChunks * 4) !=
            cudaSuccess)
        return CA_ERR_CUDA;
    p.lists_ready = true;
    return CA_OK;
}

size_t list_parts_bytes(const Pool& p) {
    const int rows = p.cfg.head_dim <= 128 && p.cfg.n_heads / kv_heads(p.cfg) > 8 ? 16 : 8;
    return (size_t)3 * p.sms * 2 * rows * (p.cfg.head_dim + 2) * sizeof(float);
}

}  // namespace ca
