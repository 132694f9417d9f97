// Eviction by accumulated attention weight: which tokens of each layer,
// sequence and key/value head stay, and their rows moved into chunks of their
// own.  The first sink and last recent tokens always stay; between them the
// largest sums do, ties to the lower position, NaN last.  Both kernels are bound
// by DRAM bytes: the sums once, the kept rows in and out.
#include <cuda_runtime.h>

#include <algorithm>

#include "ca_internal.h"
#include "fp4.cuh"

namespace ca {
namespace dev {

// ---------------------------------------------------------------------------
// Choice: one CTA per (layer, sequence, head).  The number to take from the
// middle is known, so the smallest key taken is found digit by digit from
// histograms; a pass in token order then takes what is above it and the first
// of what ties with it, and writes positions and sums behind one another.
// ---------------------------------------------------------------------------
constexpr int kPickThreads = 512, kPickWarps = kPickThreads / 32, kPickPer = 4;
constexpr int kPickBins = 2048;

struct PickParams {
    const float* in;              // [L][b][Hkv][room]
    float* out;                   // the same or apart
    int32_t* kept;                // [L][b][Hkv][budget]
    const int32_t* list_off;
    const int32_t* list_slots;
    const int32_t* slot_ntok;
    int32_t* status;
    int32_t room, budget, sink, recent, chunk, b, n_heads, capacity;
};

// Context tokens of batch row i (every chunk but its last is full).
__device__ __forceinline__ int context_tokens(const int32_t* list_off, const int32_t* list_slots, const int32_t* slot_ntok,
                                              int i, int chunk, int capacity) {
    const int a = list_off[i], n = list_off[i + 1] - a;
    const int last = n > 0 ? list_slots[a + n - 1] : -1;
    if (last < 0 || last >= capacity) return 0;
    return (n - 1) * chunk + min(max(slot_ntok[last], 0), chunk);
}

__global__ void __launch_bounds__(kPickThreads) pick_tokens_kernel(const PickParams p) {
    __shared__ uint32_t hist[kPickBins];
    __shared__ uint32_t sums[kPickWarps];
    __shared__ uint32_t found[2];                     // the digit, places left inside it
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const size_t row = blockIdx.x;
    const int i = (int)(row / p.n_heads % p.b);
    const float* in = p.in + row * p.room;
    float* out = p.out + row * p.room;
    int32_t* kept = p.kept + row * p.budget;
    const int n = min(context_tokens(p.list_off, p.list_slots, p.slot_ntok, i, p.chunk, p.capacity), p.room);
    if (n <= p.budget) {
        for (int j = threadIdx.x; j < p.budget; j += kPickThreads) kept[j] = j < n ? j : -1;
        if (in != out)
            for (int j = threadIdx.x; j < n; j += kPickThreads) out[j] = in[j];
        for (int j = n + threadIdx.x; j < p.room; j += kPickThreads) out[j] = 0.f;
        return;
    }
    const int lo = p.sink, hi = n - p.recent;         // the middle
    uint32_t left = (uint32_t)(p.budget - p.sink - p.recent), T = 0u, above = 0xffffffffu;   // keys > above are taken
    if (left > 0) {
        // the left-th largest key of the middle (which has more than left)
        uint32_t known = 0u;                          // bits of T that are found
#pragma unroll 1
        for (int shift = 21; shift >= 0; shift = shift == 21 ? 10 : shift == 10 ? 0 : -1) {
            const int bits = shift == 0 ? 10 : 11;
            for (int j = threadIdx.x; j < kPickBins; j += kPickThreads) hist[j] = 0u;
            __syncthreads();
            for (int j = lo + threadIdx.x; j < hi; j += kPickThreads) {
                const uint32_t k = order_key(in[j]);
                if ((k & known) == T) atomicAdd(&hist[(k >> shift) & ((1u << bits) - 1u)], 1u);
            }
            __syncthreads();
            // thread 0 has the largest digits
            constexpr int kPer = kPickBins / kPickThreads;
            uint32_t c[kPer], mine = 0u;
#pragma unroll
            for (int x = 0; x < kPer; ++x) mine += c[x] = hist[kPickBins - 1 - (threadIdx.x * kPer + x)];
            uint32_t at = mine;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const uint32_t o = __shfl_up_sync(kFull, at, off);
                if (lane >= off) at += o;
            }
            if (lane == 31) sums[warp] = at;
            __syncthreads();
            for (int w = 0; w < warp; ++w) at += sums[w];
            at -= mine;                               // keys of larger digits
            if (at < left && at + mine >= left) {
#pragma unroll
                for (int x = 0; x < kPer; ++x) {
                    if (at < left && at + c[x] >= left) {
                        found[0] = kPickBins - 1 - (threadIdx.x * kPer + x);
                        found[1] = left - at;
                    }
                    at += c[x];
                }
            }
            __syncthreads();
            T |= found[0] << shift;
            left = found[1];
            known |= ((1u << bits) - 1u) << shift;
            __syncthreads();
        }
        above = T;
    }
    // left of the keys that equal T are taken, the first ones
    uint32_t sure0 = 0u, tie0 = 0u;                   // before this round's tokens
    for (int t0 = 0; t0 < n; t0 += kPickThreads * kPickPer) {
        const int t = t0 + kPickPer * threadIdx.x;
        float w[kPickPer];
        uint32_t sure = 0u, tie = 0u;                 // bit masks
#pragma unroll
        for (int x = 0; x < kPickPer; ++x) {
            w[x] = t + x < n ? in[t + x] : 0.f;
            const uint32_t k = order_key(w[x]);
            const bool forced = t + x < lo || t + x >= hi;
            if (t + x < n && (forced || k > above)) sure |= 1u << x;
            else if (t + x < n && left > 0u && k == T) tie |= 1u << x;
        }
        // both counts of the threads before, in one scan (2048 tokens a round: 16 bits each)
        const uint32_t mine = __popc(sure) | (__popc(tie) << 16);
        uint32_t at = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const uint32_t o = __shfl_up_sync(kFull, at, off);
            if (lane >= off) at += o;
        }
        if (lane == 31) sums[warp] = at;
        __syncthreads();                              // (this round's reads of the sums are done too)
        uint32_t all = 0u;
        for (int x = 0; x < kPickWarps; ++x) {
            if (x == warp) at += all;
            all += sums[x];
        }
        at -= mine;
        uint32_t s = sure0 + (at & 0xffffu), e = tie0 + (at >> 16);
#pragma unroll
        for (int x = 0; x < kPickPer; ++x) {
            const bool take = (sure >> x & 1u) || ((tie >> x & 1u) && e < left);
            if (take) {
                const uint32_t to = s + min(e, left);
                kept[to] = t + x;
                out[to] = w[x];                       // (to <= t + x: in place, a place that has been read)
            }
            s += sure >> x & 1u;
            e += tie >> x & 1u;
        }
        sure0 += all & 0xffffu;
        tie0 += all >> 16;
        __syncthreads();
    }
    for (int j = p.budget + threadIdx.x; j < p.room; j += kPickThreads) out[j] = 0.f;
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
    dev::pick_tokens_kernel<<<(unsigned)(per * s.t.b), dev::kPickThreads, 0, cs>>>(a);
    if (cudaGetLastError() != cudaSuccess) return CA_ERR_CUDA;
    count_launch();
    const size_t most = std::max<size_t>(1, std::min<size_t>(dev::kManyMoves, (size_t)INT32_MAX / per));
    for (size_t i = 0; i < ch.size();) {
        const size_t n = std::min(most, ch.size() - i);
        const int st = n <= dev::kFewMoves    ? moves<dev::kFewMoves>(p, s, ch.data() + i, n, budget, kept, cs)
                       : n <= dev::kSomeMoves ? moves<dev::kSomeMoves>(p, s, ch.data() + i, n, budget, kept, cs)
                                              : moves<dev::kManyMoves>(p, s, ch.data() + i, n, budget, kept, cs);
        if (st) return st;
        i += n;
    }
    return rows.empty() ? CA_OK : launch_key_bounds(p, rows, stream);
}

}  // namespace ca
