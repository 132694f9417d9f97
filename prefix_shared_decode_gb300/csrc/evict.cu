// Eviction by accumulated attention weight: which tokens of each layer,
// sequence and key/value head stay, and their rows moved into chunks of their
// own.  The first sink and last recent tokens always stay; between them the
// largest sums do, ties to the lower position, NaN last.
//
// The bytes that count are the kept rows', in and out: 64 rows of 65536 tokens cut
// to 8192 (268 MB of keys and values) move in 83 us, 6.4 TB/s or 95% of the copy
// rate; their choice takes 39 us more, latency of four digits and a barrier of the
// cluster for each, where reading the sums would take 5.
#include <cuda_runtime.h>

#include <algorithm>

#include "ca_internal.h"
#include "cluster.cuh"
#include "fp4.cuh"

namespace ca {
namespace dev {

// ---------------------------------------------------------------------------
// Choice: a cluster of CTAs per (layer, sequence, head), each with a stretch of
// the row's sums in shared memory.  The number to take from the middle is known, so
// the smallest key taken is found digit by digit (8 bits) from the
// cluster's histograms; then each CTA takes, in token order, what is above it and
// the first of what ties with it, and writes positions and sums behind those of
// the CTAs before it.  (One CTA a row that reads it five times from L2: 64 rows
// of 65536 took 75 us, 1024 rows of 2560 29 us.)
// ---------------------------------------------------------------------------
constexpr int kPickThreads = 256, kPickWarps = kPickThreads / 32, kPickPer = 16;   // a thread per digit
constexpr int kPickCache = 53248;         // sums that fit a CTA's shared memory

struct PickParams {
    const float* in;              // [L][b][Hkv][room]
    float* out;                   // the same or apart
    int32_t* kept;                // [L][b][Hkv][budget]
    const int32_t* list_off;
    const int32_t* list_slots;
    const int32_t* slot_ntok;
    int32_t* status;
    int32_t room, budget, sink, recent, chunk, b, n_heads, capacity;
    int32_t splits, cache;        // CTAs a cluster; sums that a CTA has room for
};

// Context tokens of batch row i (every chunk but its last is full).
__device__ __forceinline__ int context_tokens(const int32_t* list_off, const int32_t* list_slots, const int32_t* slot_ntok,
                                              int i, int chunk, int capacity) {
    const int a = list_off[i], n = list_off[i + 1] - a;
    const int last = n > 0 ? list_slots[a + n - 1] : -1;
    if (last < 0 || last >= capacity) return 0;
    return (n - 1) * chunk + min(max(slot_ntok[last], 0), chunk);
}

// Exclusive sums over the block's threads (red: one word a warp); all: the total.
__device__ __forceinline__ uint32_t sum_before(uint32_t mine, uint32_t* red, uint32_t& all) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t at = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const uint32_t o = __shfl_up_sync(kFull, at, off);
        if (lane >= off) at += o;
    }
    __syncthreads();                      // earlier reads of red are done
    if (lane == 31) red[warp] = at;
    __syncthreads();
    all = 0u;
#pragma unroll
    for (int x = 0; x < kPickWarps; ++x) {
        if (x == warp) at += all;
        all += red[x];
    }
    return at - mine;
}

// CACHED: the CTA holds its sums (else the only CTA of a row reads them each time).
template <bool CACHED>
__global__ void __launch_bounds__(kPickThreads, 6) pick_tokens_kernel(const PickParams p) {
    extern __shared__ __align__(16) float held[];
    __shared__ uint32_t hist[4][256];
    __shared__ uint32_t red[kPickWarps];
    __shared__ uint32_t found[2];                     // the digit, places left inside it
    __shared__ uint32_t count[1];                     // this CTA's tokens that are taken, those that tie above
    const int cs = p.splits, rank = blockIdx.x % cs;
    const size_t row = blockIdx.x / cs;
    const int i = (int)(row / p.n_heads % p.b);
    const float* in = p.in + row * p.room;
    float* out = p.out + row * p.room;
    int32_t* kept = p.kept + row * p.budget;
    const int n = min(context_tokens(p.list_off, p.list_slots, p.slot_ntok, i, p.chunk, p.capacity), p.room);
    const int first = rank * kPickThreads + threadIdx.x, stride = cs * kPickThreads;
    if (n <= p.budget) {                              // (the whole cluster: the same n)
        for (int j = first; j < p.budget; j += stride) kept[j] = j < n ? j : -1;
        if (in != out)
            for (int j = first; j < n; j += stride) out[j] = in[j];
        for (int j = n + first; j < p.room; j += stride) out[j] = 0.f;
        return;
    }
    // this CTA's tokens [t0, t1), a multiple of 4 but for the last one's
    const int per = ((n + cs - 1) / cs + 3) & ~3, t0 = min(n, rank * per), t1 = min(n, t0 + per);
    if (CACHED && per > p.cache) {                    // a context longer than the host knew of (the same for the cluster)
        if (threadIdx.x == 0) set_status(p.status, CA_ERR_DEVICE_BOUNDS);
        return;
    }
    const int lo = p.sink, hi = n - p.recent;         // the middle
    uint32_t left = (uint32_t)(p.budget - p.sink - p.recent), T = 0u, above = 0xffffffffu;   // keys > above are taken
    for (int j = threadIdx.x; j < 4 * 256; j += kPickThreads) hist[j >> 8][j & 255] = 0u;
    if (CACHED) {
        // (8 loads a thread on their way together)
        if (((reinterpret_cast<uintptr_t>(in + t0)) & 15u) == 0) {
            for (int from = t0 + 4 * threadIdx.x; from < t1; from += 32 * kPickThreads) {
                float4 w[8];
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    const int t = from + 4 * x * kPickThreads;
                    w[x] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (t + 3 < t1) w[x] = *reinterpret_cast<const float4*>(in + t);
                    else if (t < t1) {
                        w[x].x = in[t];
                        if (t + 1 < t1) w[x].y = in[t + 1];
                        if (t + 2 < t1) w[x].z = in[t + 2];
                    }
                }
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    const int t = from + 4 * x * kPickThreads;
                    if (t < t1) *reinterpret_cast<float4*>(held + (t - t0)) = w[x];
                }
            }
        } else {
            for (int from = t0 + threadIdx.x; from < t1; from += 8 * kPickThreads) {
                float w[8];
#pragma unroll
                for (int x = 0; x < 8; ++x) w[x] = from + x * kPickThreads < t1 ? in[from + x * kPickThreads] : 0.f;
#pragma unroll
                for (int x = 0; x < 8; ++x)
                    if (from + x * kPickThreads < t1) held[from + x * kPickThreads - t0] = w[x];
            }
        }
    }
    __syncthreads();
    // four sums from token t on (those from t1 on are anything)
    auto four = [&](int t, float (&w)[4]) {
        if constexpr (CACHED) {
            const float4 v = *reinterpret_cast<const float4*>(held + (t - t0));
            w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
        } else {
#pragma unroll
            for (int x = 0; x < 4; ++x) w[x] = t + x < t1 ? in[t + x] : 0.f;
        }
    };
    uint32_t known = 0u;                              // bits of T that are found
    uint32_t larger = 0u, equal = 0u;                 // of this CTA's keys: above T (this thread's part), equal to it
#pragma unroll 1
    for (int pass = 0; pass < 4 && left > 0u; ++pass) {
        const int shift = 24 - 8 * pass, m0 = max(lo, t0), m1 = min(hi, t1);
#pragma unroll 2
        for (int t = t0 + 4 * threadIdx.x; t < m1; t += 4 * kPickThreads) {
            float w[4];
            four(t, w);
#pragma unroll
            for (int x = 0; x < 4; ++x) {             // of the keys whose digits so far are T's
                const uint32_t k = order_key(w[x]);
                if (t + x >= m0 && t + x < m1 && (k & known) == T) atomicAdd(&hist[pass][k >> shift & 255u], 1u);
            }
        }
        if (cs > 1) cluster_sync_all();
        else __syncthreads();
        const uint32_t bin = 255u - threadIdx.x;      // thread 0 has the largest digit
        uint32_t c = 0u, all;
        if (cs == 1) c = hist[pass][bin];
        else
            for (int r = 0; r < cs; ++r) c += ld_peer(peer_addr(smem_u32(&hist[pass][bin]), r));
        const uint32_t at = sum_before(c, red, all);  // keys of larger digits
        if (at < left && at + c >= left) {
            found[0] = bin;
            found[1] = left - at;
        }
        __syncthreads();
        if (bin > found[0]) larger += hist[pass][bin];
        equal = hist[pass][found[0]];
        T |= found[0] << shift;
        known |= 255u << shift;
        left = found[1];                              // (at least 1 once there is any)
    }
    if (left > 0u) above = T;
    // left of the keys that equal T are taken, the first ones
    auto kinds = [&](int t, const float (&w)[4], uint32_t& sure, uint32_t& tie, int bit) {
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const uint32_t k = order_key(w[x]);
            if (t + x >= t1) continue;
            if (t + x < lo || t + x >= hi || k > above) sure |= 1u << (bit + x);
            else if (left > 0u && k == T) tie |= 1u << (bit + x);
        }
    };
    uint32_t sure0 = 0u, tie0 = 0u;                   // before this CTA's tokens, then before each stretch's
    if (cs > 1) {
        uint32_t all;
        sum_before(larger, red, all);
        all += max(0, min(t1, lo) - t0) + max(0, t1 - max(t0, hi));      // and the forced ones
        if (left > 0u) all |= equal << 16;            // (53248 sums a CTA at most: 16 bits each)
        if (threadIdx.x == 0) count[0] = all;
        cluster_sync_all();                           // (all of the cluster's sums are held by now: in place from here on)
        for (int r = 0; r < rank; ++r) {
            const uint32_t v = ld_peer(peer_addr(smem_u32(&count[0]), r));
            sure0 += v & 0xffffu;
            tie0 += v >> 16;
        }
    }
    for (int from = t0; from < t1; from += kPickThreads * kPickPer) {
        const int t = from + kPickPer * threadIdx.x;
        float w[kPickPer / 4][4];
        uint32_t sure = 0u, tie = 0u, all;            // bit masks
#pragma unroll
        for (int x = 0; x < kPickPer / 4; ++x) {
            if (t + 4 * x >= t1) break;
            four(t + 4 * x, w[x]);
            kinds(t + 4 * x, w[x], sure, tie, 4 * x);
        }
        // both counts of the threads before, in one scan (4096 tokens a stretch: 16 bits each);
        // its barriers also part this stretch's reads from its writes
        const uint32_t at = sum_before(__popc(sure) | (__popc(tie) << 16), red, all);
        uint32_t s = sure0 + (at & 0xffffu), e = tie0 + (at >> 16);
#pragma unroll
        for (int x = 0; x < kPickPer; ++x) {
            if ((sure >> x & 1u) || ((tie >> x & 1u) && e < left)) {
                const uint32_t to = s + min(e, left);
                kept[to] = t + x;
                out[to] = w[x / 4][x % 4];            // (to <= t + x: in place, a place that has been read)
            }
            s += sure >> x & 1u;
            e += tie >> x & 1u;
        }
        sure0 += all & 0xffffu;
        tie0 += all >> 16;
    }
    if (!CACHED) __syncthreads();
    for (int j = p.budget + first; j < p.room; j += stride) out[j] = 0.f;
    if (cs > 1) cluster_sync_all();                   // the others have read this one's counts
}

// ---------------------------------------------------------------------------
// Move: one CTA per (new chunk, layer, head).  Rows [pos0, pos0 + rows) of the
// kept ones of a batch row go to `slot`, as the pool holds them (codes and scales
// of 8 and 4 bits are not requantised); rows past them are zeros.
// ---------------------------------------------------------------------------
constexpr int kMoveThreads = 256;
constexpr int kFewMoves = 16, kSomeMoves = 248, kManyMoves = 1024;   // (as the lists of the row copies)

struct EvictChunk {
    int32_t seq, pos0, rows, slot;
};
template <int N>
struct MoveArgs {
    uint8_t* pool;
    int32_t* slot_ntok;
    const int32_t* kept;
    const int32_t* list_off;
    const int32_t* list_slots;
    int32_t* status;
    int32_t budget, n_chunks, n_layers, n_heads, b, capacity;
    EvictChunk ch[N];
};
static_assert(sizeof(MoveArgs<kSomeMoves>) <= 4096 && sizeof(MoveArgs<kManyMoves>) <= 32764, "launch parameters");

template <int C, int D, int EB, int N>
__global__ void __launch_bounds__(kMoveThreads) move_rows_kernel(const __grid_constant__ MoveArgs<N> a) {
    __shared__ int2 from[C];                          // slot and row of each new row; slot -1: zeros
    const int h = blockIdx.x % a.n_heads, rest = blockIdx.x / a.n_heads;
    const EvictChunk c = a.ch[rest % a.n_chunks];
    const int l = rest / a.n_chunks;
    if (h == 0 && l == 0 && threadIdx.x == 0) a.slot_ntok[c.slot] = c.rows;
    const int off = a.list_off[c.seq], n = a.list_off[c.seq + 1] - off;
    const int32_t* kept = a.kept + (((size_t)l * a.b + c.seq) * a.n_heads + h) * a.budget + c.pos0;
    for (int r = threadIdx.x; r < C; r += kMoveThreads) {
        int2 x = make_int2(-1, 0);
        if (r < c.rows) {
            const int pos = kept[r];
            if (pos >= 0 && pos / C < n) x = make_int2(a.list_slots[off + pos / C], pos % C);
            if (x.x < 0 || x.x >= a.capacity) {
                x.x = -1;
                set_status(a.status, CA_ERR_DEVICE_BOUNDS);
            }
        }
        from[r] = x;
    }
    __syncthreads();
    if constexpr (EB != 0) {
        constexpr int NV = D * EB / 16;               // 16-byte pieces of a row
        const long long tile = (long long)C * NV;
        uint4* pool = reinterpret_cast<uint4*>(a.pool);
        auto at = [&](long long slot, int kv) { return (((slot * a.n_layers + l) * 2 + kv) * a.n_heads + h) * tile; };
        for (int i = threadIdx.x; i < 2 * C * NV; i += kMoveThreads) {
            const int kv = i / (C * NV), r = i / NV % C, x = i % NV;
            const int2 f = from[r];
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (f.x >= 0) v = __ldcs(pool + at(f.x, kv) + f.y * NV + x);
            pool[at(c.slot, kv) + r * NV + x] = v;
        }
    } else {
        using T = F4Tile<C, D>;
        auto at = [&](long long slot) { return ((slot * a.n_layers + l) * a.n_heads + h) * T::kBytes; };
        uint8_t* dst = a.pool + at(c.slot);
        // keys: rows of codes and of scales, each in the same order within the row
        for (int i = threadIdx.x; i < C * (D / 32); i += kMoveThreads) {
            const int r = i / (D / 32), x = i % (D / 32);
            const int2 f = from[r];
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (f.x >= 0) v = *reinterpret_cast<const uint4*>(a.pool + at(f.x) + f4_row(f.y) * (D / 2) + 16 * x);
            *reinterpret_cast<uint4*>(dst + f4_row(r) * (D / 2) + 16 * x) = v;
        }
        for (int i = threadIdx.x; i < C * (D / 64); i += kMoveThreads) {
            const int r = i / (D / 64), x = i % (D / 64);
            const int2 f = from[r];
            uint32_t v = 0u;
            if (f.x >= 0) v = *reinterpret_cast<const uint32_t*>(a.pool + at(f.x) + T::kKScales + f4_row(f.y) * (D / 16) + 4 * x);
            *reinterpret_cast<uint32_t*>(dst + T::kKScales + f4_row(r) * (D / 16) + 4 * x) = v;
        }
        // values: two tokens to a byte
        for (int i = threadIdx.x; i < C / 2 * D; i += kMoveThreads) {
            const int pair = i / D, d = i % D, tok = (pair >> 2) * 8 + (pair & 3);
            uint32_t v = 0u;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int2 f = from[tok + 4 * x];
                if (f.x < 0) continue;
                const uint32_t byte = a.pool[at(f.x) + T::kVCodes + f4_v_byte<D>(f4_pair(f.y), d)];
                v |= (byte >> (f.y & 4) & 15u) << (4 * x);
            }
            dst[T::kVCodes + f4_v_byte<D>(pair, d)] = (uint8_t)v;
        }
        for (int i = threadIdx.x; i < C * (D / 16); i += kMoveThreads) {
            const int r = i / (D / 16), blk = i % (D / 16);
            const int2 f = from[r];
            dst[T::kVScales + f4_v_scale<D>(r, blk)] =
                f.x >= 0 ? a.pool[at(f.x) + T::kVScales + f4_v_scale<D>(f.y, blk)] : (uint8_t)0;
        }
    }
}

}  // namespace dev

namespace {

// CTAs per row: enough that the card is full twice over, as long as each has some
// 2048 sums, and so many that a row's sums fit their shared memories (if 8 hold
// them; else one CTA reads them from memory).
int run_pick(const Pool& p, dev::PickParams& a, size_t rows, const std::vector<EvictSeq>& seqs, cudaStream_t s) {
    int64_t most = 1;
    for (const EvictSeq& e : seqs) most = std::max<int64_t>(most, e.n);
    int cs = 1;
    auto share = [&](int k) { return (most + k - 1) / k; };
    while (cs < 8 && ((rows * cs < (size_t)2 * p.sms && share(2 * cs) >= 2048) || share(cs) + 4 > dev::kPickCache)) cs *= 2;
    const bool cached = share(cs) + 4 <= dev::kPickCache;
    if (!cached) cs = 1;
    a.splits = cs;
    a.cache = cached ? (int32_t)share(cs) + 4 : 0;
    const size_t bytes = (size_t)a.cache * sizeof(float);
    if (rows * cs > (size_t)INT32_MAX) return CA_ERR_UNSUPPORTED;
    if (cached && cudaFuncSetAttribute(dev::pick_tokens_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       dev::kPickCache * (int)sizeof(float)) != cudaSuccess)
        return CA_ERR_CUDA;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)cs;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t c = {};
    c.gridDim = dim3((unsigned)(rows * cs));
    c.blockDim = dim3(dev::kPickThreads);
    c.dynamicSmemBytes = bytes;
    c.stream = s;
    c.attrs = attr;
    c.numAttrs = 1;
    if ((cached ? cudaLaunchKernelEx(&c, dev::pick_tokens_kernel<true>, a) : cudaLaunchKernelEx(&c, dev::pick_tokens_kernel<false>, a)) !=
        cudaSuccess)
        return CA_ERR_CUDA;
    count_launch();
    return CA_OK;
}

template <int D, int EB, int N>
bool pick_chunk(int chunk, unsigned blocks, const dev::MoveArgs<N>& a, cudaStream_t s) {
    if (chunk == 16) dev::move_rows_kernel<16, D, EB, N><<<blocks, dev::kMoveThreads, 0, s>>>(a);
    else if (chunk == 32) dev::move_rows_kernel<32, D, EB, N><<<blocks, dev::kMoveThreads, 0, s>>>(a);
    else if (chunk == 64 && D <= 128)
        dev::move_rows_kernel<64, D <= 128 ? D : 128, EB, N><<<blocks, dev::kMoveThreads, 0, s>>>(a);
    else return false;
    return true;
}

template <int N>
int run_moves(const Pool& p, dev::MoveArgs<N>& a, const dev::EvictChunk* ch, size_t n, cudaStream_t s) {
    const PoolCfg& c = p.cfg;
    a.n_chunks = (int32_t)n;
    std::copy(ch, ch + n, a.ch);
    const unsigned blocks = (unsigned)(n * c.n_layers * kv_heads(c));
    const int D = c.head_dim;
    bool ok = false;
    if (c.flags & CA_KV_FP4) {
        if (D == 64) ok = pick_chunk<64, 0>(c.chunk, blocks, a, s);
        else if (D == 128) ok = pick_chunk<128, 0>(c.chunk, blocks, a, s);
    } else if (c.flags & CA_KV_FP8) {
        if (D == 128) ok = pick_chunk<128, 1>(c.chunk, blocks, a, s);
    } else {
        if (D == 64) ok = pick_chunk<64, 2>(c.chunk, blocks, a, s);
        else if (D == 128) ok = pick_chunk<128, 2>(c.chunk, blocks, a, s);
        else if (D == 256) ok = pick_chunk<256, 2>(c.chunk, blocks, a, s);
    }
    if (!ok) return CA_ERR_UNSUPPORTED;
    if (cudaGetLastError() != cudaSuccess) return CA_ERR_CUDA;
    count_launch();
    return CA_OK;
}

template <int N>
int moves(const Pool& p, const Sched& s, const dev::EvictChunk* ch, size_t n, int32_t budget, const int32_t* kept,
          cudaStream_t stream) {
    unsigned char* dev8 = static_cast<unsigned char*>(s.dev);
    dev::MoveArgs<N> a;
    a.pool = static_cast<uint8_t*>(p.kv);
    a.slot_ntok = reinterpret_cast<int32_t*>(a.pool + pool_tile_bytes(p.cfg));
    a.kept = kept;
    a.list_off = reinterpret_cast<const int32_t*>(dev8 + s.layout.list_off);
    a.list_slots = reinterpret_cast<const int32_t*>(dev8 + s.layout.list_slots);
    a.status = reinterpret_cast<int32_t*>(dev8 + s.layout.status);
    a.budget = budget;
    a.n_layers = p.cfg.n_layers;
    a.n_heads = kv_heads(p.cfg);
    a.b = s.t.b;
    a.capacity = p.cfg.capacity_slots;
    return run_moves(p, a, ch, n, stream);
}

}  // namespace

int launch_evict(const Pool& p, const Sched& s, const std::vector<EvictSeq>& seqs, const float* weights, int32_t room,
                 int32_t budget, int32_t sink, int32_t recent, int32_t* kept, float* weights_out, void* stream) {
    const PoolCfg& c = p.cfg;
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    const size_t per = (size_t)c.n_layers * kv_heads(c);
    if (per * s.t.b > (size_t)INT32_MAX) return CA_ERR_UNSUPPORTED;
    // the new chunks
    std::vector<dev::EvictChunk> ch;
    std::vector<ScatterChunk> rows;
    for (size_t i = 0; i < seqs.size(); ++i) {
        const EvictSeq& e = seqs[i];
        if (!e.changed) continue;
        for (int32_t k = e.stay; k < (int32_t)e.next.path.size(); ++k) {
            const Node* x = e.next.path[k];
            alloc_point(p);
            ch.push_back({(int32_t)i, k * c.chunk, x->ntok, x->slot});
            if (c.flags & CA_CHUNK_BOUNDS) rows.push_back({0, x->ntok, x->slot, 0});
        }
    }
    p.kv_written = true;
    unsigned char* dev8 = static_cast<unsigned char*>(s.dev);
    dev::PickParams a{};
    a.in = weights;
    a.out = weights_out;
    a.kept = kept;
    a.list_off = reinterpret_cast<const int32_t*>(dev8 + s.layout.list_off);
    a.list_slots = reinterpret_cast<const int32_t*>(dev8 + s.layout.list_slots);
    a.slot_ntok = reinterpret_cast<const int32_t*>(static_cast<const unsigned char*>(p.kv) + pool_tile_bytes(c));
    a.status = reinterpret_cast<int32_t*>(dev8 + s.layout.status);
    a.room = room;
    a.budget = budget;
    a.sink = sink;
    a.recent = recent;
    a.chunk = c.chunk;
    a.b = s.t.b;
    a.n_heads = kv_heads(c);
    a.capacity = c.capacity_slots;
    int st = run_pick(p, a, per * s.t.b, seqs, cs);
    if (st) return st;
    const size_t most = std::max<size_t>(1, std::min<size_t>(dev::kManyMoves, (size_t)INT32_MAX / per));
    for (size_t i = 0; i < ch.size();) {
        const size_t n = std::min(most, ch.size() - i);
        st = n <= dev::kFewMoves    ? moves<dev::kFewMoves>(p, s, ch.data() + i, n, budget, kept, cs)
             : n <= dev::kSomeMoves ? moves<dev::kSomeMoves>(p, s, ch.data() + i, n, budget, kept, cs)
                                    : moves<dev::kManyMoves>(p, s, ch.data() + i, n, budget, kept, cs);
        if (st) return st;
        i += n;
    }
    return rows.empty() ? CA_OK : launch_key_bounds(p, rows, stream);
}

}  // namespace ca
