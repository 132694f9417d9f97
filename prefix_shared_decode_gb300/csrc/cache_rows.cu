// Moving rows between packed fp16 tensors and the pool's tiles, where the
// pool is more than a copy: quantising inserts of an fp4 pool, the key
// bounds of a pool with chunk bounds, and reading rows back (every pool).
// All three are bound by DRAM bytes; a CTA takes one chunk of one key/value
// head and layer, and goes through shared memory where the tile's order is
// not the rows'.  1024 chunks of 64 tokens, 32 heads of 128 dims: 215 us to
// store as fp4 (1.32 GB moved, 6.1 TB/s), 225 us to read back (5.8 TB/s), 91% and
// 87% of the copy rate; bounds read the rows just written from L2.
#include <cuda_runtime.h>

#include <algorithm>

#include "ca_internal.h"
#include "fp4.cuh"

namespace ca {
namespace dev {

constexpr int kRowThreads = 256;
// Chunk lists travel in the launch parameters: short lists for decode-time
// appends, longer ones for prompts.  Parameters above 4 KB cost the host some
// 10 us a launch, so the longest list is taken only where several launches of
// the next one would cost it as much and the card a tail each (1024 chunks of
// 32 heads stored and read back: 59 us less in one launch each than in five).
constexpr int kFewChunks = 16, kSomeChunks = 248, kManyChunks = 1024;

template <int N>
struct RowArgs {
    const uint16_t *k, *v;        // packed rows [L][total_rows][Hkv][D] (written by the read kernel)
    uint8_t* pool;
    int32_t* slot_ntok;
    uint16_t* bounds;             // [slot][L][Hkv][2][D], or null
    int32_t total_rows, n_chunks, n_layers, n_heads;
    float k_mul, v_mul;           // stores: 1 / scale; reads: scale
    ScatterChunk ch[N];
};

static_assert(sizeof(RowArgs<kSomeChunks>) <= 4096 && sizeof(RowArgs<kManyChunks>) <= 32764, "launch parameters");

struct Where {
    ScatterChunk c;
    int h, l;
};
template <int N>
__device__ __forceinline__ Where where(const RowArgs<N>& a) {
    const int h = blockIdx.x % a.n_heads, rest = blockIdx.x / a.n_heads;
    return {a.ch[rest % a.n_chunks], h, rest / a.n_chunks};
}

// ---------------------------------------------------------------------------
// fp4 store.  A thread takes one block of 16 dims of a row (32 bytes):
//   y = fp32(x) * fp32(1 / S), scale = E4M3(max|y| * fp32(1/6)),
//   code = E2M1(y * fp32(1 / scale)), nearest even, saturating; all codes 0
// where the scale is 0.  The codes are placed in a shared-memory tile and
// written out in 16-byte pieces: the whole tile of a new chunk (zeros past
// its tokens, whose weight is 0 and must not meet a NaN), the new rows'
// bytes of one that grows.
// ---------------------------------------------------------------------------
template <int C, int D, int N>
__global__ void __launch_bounds__(kRowThreads) fp4_store_kernel(const __grid_constant__ RowArgs<N> a) {
    using T = F4Tile<C, D>;
    __shared__ __align__(16) uint8_t tile[T::kBytes];
    const Where at = where(a);
    const ScatterChunk c = at.c;
    if (at.h == 0 && at.l == 0 && threadIdx.x == 0) a.slot_ntok[c.slot] = c.dst_row + c.n_rows;
    if (c.dst_row == 0 && c.n_rows < C) {
        for (int i = threadIdx.x; i < T::kBytes / 16; i += kRowThreads)
            reinterpret_cast<uint4*>(tile)[i] = make_uint4(0u, 0u, 0u, 0u);
        __syncthreads();
    }
    constexpr int NB = D / 16;                       // blocks per row
    uint8_t* dst = a.pool + (((long long)c.slot * a.n_layers + at.l) * a.n_heads + at.h) * T::kBytes;
    // A thread takes one block of two tokens that share value bytes (x and
    // x + 4), keys and values: all 128 bytes are on their way before the first
    // is looked at.
    struct Block { uint4 a, b; };
    auto fetch = [&](const uint16_t* rows, int r, int blk) -> Block {
        const long long src = (((long long)at.l * a.total_rows + c.src_row + r) * a.n_heads + at.h) * D + blk * 16;
        const uint4* p = reinterpret_cast<const uint4*>(rows + src);
        return {__ldcs(p), __ldcs(p + 1)};
    };
    // its codes, two to a byte, and its scale
    auto quantise = [&](const Block& x, float mul, uint32_t (&b)[8]) -> uint32_t {
        const uint32_t w[8] = {x.a.x, x.a.y, x.a.z, x.a.w, x.b.x, x.b.y, x.b.z, x.b.w};
        float y[16], top = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
            y[2 * j] = f.x * mul;
            y[2 * j + 1] = f.y * mul;
            top = fmaxf(top, fmaxf(fabsf(y[2 * j]), fabsf(y[2 * j + 1])));
        }
        const uint32_t sc = e4m3x2_from_f32(top * (1.f / 6.f), 0.f) & 0xffu;
        const uint32_t sh = f16x2_from_e4m3x2(sc);
        const float s = __low2float(*reinterpret_cast<const __half2*>(&sh));
        const float inv = s > 0.f ? __frcp_rn(s) : 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) b[j] = e2m1x2_from_f32(y[2 * j] * inv, y[2 * j + 1] * inv);
        return sc;
    };
    auto put_key = [&](const Block& x, int tok, int blk) {
        uint32_t b[8];
        tile[T::kKScales + f4_k_scale<D>(tok, blk)] = (uint8_t)quantise(x, a.k_mul, b);
#pragma unroll
        for (int t = 0; t < 4; ++t)
            *reinterpret_cast<uint16_t*>(tile + f4_k_byte<D>(tok, blk * 16 + 4 * t)) =
                (uint16_t)(b[2 * t] | (b[2 * t + 1] << 8));
    };
    const int z = c.dst_row + c.n_rows;
    for (int i = threadIdx.x; i < C / 2 * NB; i += kRowThreads) {
        const int pair = i / NB, blk = i % NB, tok = (pair >> 2) * 8 + (pair & 3);
        const bool has0 = tok >= c.dst_row && tok < z, has1 = tok + 4 >= c.dst_row && tok + 4 < z;
        if (!has0 && !has1) continue;
        Block k0, k1, v0, v1;
        if (has0) { k0 = fetch(a.k, tok - c.dst_row, blk); v0 = fetch(a.v, tok - c.dst_row, blk); }
        if (has1) { k1 = fetch(a.k, tok + 4 - c.dst_row, blk); v1 = fetch(a.v, tok + 4 - c.dst_row, blk); }
        if (has0) put_key(k0, tok, blk);
        if (has1) put_key(k1, tok + 4, blk);
        uint32_t b0[8], b1[8];
        if (has0) tile[T::kVScales + f4_v_scale<D>(tok, blk)] = (uint8_t)quantise(v0, a.v_mul, b0);
        if (has1) tile[T::kVScales + f4_v_scale<D>(tok + 4, blk)] = (uint8_t)quantise(v1, a.v_mul, b1);
        // The token that is not among the new rows keeps what the pool holds
        // (nothing, in a new chunk).
#pragma unroll
        for (int g = 0; g < 8; ++g) {
            const int at0 = T::kVCodes + f4_v_byte<D>(pair, blk * 16 + 2 * g), at1 = at0 + D / 16;
            uint32_t x, y;                            // dims 2g, 2g + 1: (tok, tok + 4)
            if (has0 && has1) {
                x = (b0[g] & 15u) | (b1[g] << 4);
                y = (b0[g] >> 4) | (b1[g] & 0xf0u);
            } else {
                const uint32_t ox = c.dst_row ? dst[at0] : 0u, oy = c.dst_row ? dst[at1] : 0u;
                x = has0 ? (b0[g] & 15u) | (ox & 0xf0u) : (ox & 15u) | (b1[g] << 4);
                y = has0 ? (b0[g] >> 4) | (oy & 0xf0u) : (oy & 15u) | (b1[g] & 0xf0u);
            }
            tile[at0] = (uint8_t)x;
            tile[at1] = (uint8_t)y;
        }
    }
    __syncthreads();
    if (c.dst_row == 0) {
        for (int i = threadIdx.x; i < T::kBytes / 16; i += kRowThreads)
            reinterpret_cast<uint4*>(dst)[i] = reinterpret_cast<const uint4*>(tile)[i];
        return;
    }
    // the new rows alone: key rows and pairs of value rows in 16-byte pieces,
    // then the scales
    for (int i = threadIdx.x; i < c.n_rows * (D / 32); i += kRowThreads) {
        const int off = f4_row(c.dst_row + i / (D / 32)) * (D / 2) + i % (D / 32) * 16;
        *reinterpret_cast<uint4*>(dst + off) = *reinterpret_cast<const uint4*>(tile + off);
    }
    for (int i = threadIdx.x; i < C / 2 * (D / 16); i += kRowThreads) {
        const int pair = i / (D / 16), tok = (pair >> 2) * 8 + (pair & 3);
        if (!(tok >= c.dst_row && tok < z) && !(tok + 4 >= c.dst_row && tok + 4 < z)) continue;
        const int off = T::kVCodes + i * 16;
        *reinterpret_cast<uint4*>(dst + off) = *reinterpret_cast<const uint4*>(tile + off);
    }
    for (int i = threadIdx.x; i < 2 * c.n_rows * NB; i += kRowThreads) {
        const int r = i / NB % c.n_rows, blk = i % NB;
        const int off = (i < c.n_rows * NB) ? T::kKScales + f4_k_scale<D>(c.dst_row + r, blk)
                                            : T::kVScales + f4_v_scale<D>(c.dst_row + r, blk);
        dst[off] = tile[off];
    }
}

// ---------------------------------------------------------------------------
// Stored keys as pairs of dims, in units of the key scale: fp16 values of an
// fp16 pool, the E4M3 values of an fp8 pool, code * scale of an fp4 pool.
// EB: bytes per element (0: fp4).  tile: the key tile of one chunk and head.
// ---------------------------------------------------------------------------
template <int C, int D, int EB>
__device__ __forceinline__ uint32_t key_pair(const uint8_t* tile, int tok, int d) {
    if constexpr (EB == 2) {
        return *reinterpret_cast<const uint32_t*>(tile + ((size_t)tok * D + d) * 2);
    } else if constexpr (EB == 1) {
        return f16x2_from_e4m3x2(*reinterpret_cast<const uint16_t*>(tile + (size_t)tok * D + d));
    } else {
        const uint32_t s = f16x2_from_e4m3x2(tile[F4Tile<C, D>::kKScales + f4_k_scale<D>(tok, d >> 4)] * 0x101u);
        return mul_f16x2(f16x2_from_e2m1x2(tile[f4_k_byte<D>(tok, d)]), s);
    }
}

// Byte offset of the tile of (slot, layer, head): K's of an fp16 or fp8 pool
// (V's lies n_heads tiles on), the joint one of an fp4 pool.
template <int C, int D, int EB>
__device__ __forceinline__ long long tile_at(long long slot, int n_layers, int l, int n_heads, int h) {
    if constexpr (EB == 0) return ((slot * n_layers + l) * n_heads + h) * F4Tile<C, D>::kBytes;
    return ((slot * n_layers + l) * 2 * n_heads + h) * (long long)(C * D * EB);
}

// ---------------------------------------------------------------------------
// Chunk bounds: the largest and smallest stored key of each dim over the
// chunk's tokens.  Maxima of stored values are stored values, so the bounds
// are exact and an append only joins its rows to the old ones.  Runs after
// the store in stream order and reads back the rows just written (in L2).
// ---------------------------------------------------------------------------
template <int C, int D, int EB, int N>
__global__ void __launch_bounds__(kRowThreads) key_bounds_kernel(const __grid_constant__ RowArgs<N> a) {
    constexpr int P = D / 2, G = kRowThreads / P;    // pairs of dims; groups of rows
    __shared__ uint32_t part[2][G][P];
    const Where at = where(a);
    const ScatterChunk c = at.c;
    const uint8_t* tile = a.pool + tile_at<C, D, EB>(c.slot, a.n_layers, at.l, a.n_heads, at.h);
    const int p = threadIdx.x % P, g = threadIdx.x / P;
    __half2 hi = __float2half2_rn(-INFINITY), lo = __float2half2_rn(INFINITY);
    for (int r = c.dst_row + g; r < c.dst_row + c.n_rows; r += G) {
        const uint32_t x = key_pair<C, D, EB>(tile, r, 2 * p);
        hi = __hmax2(hi, *reinterpret_cast<const __half2*>(&x));
        lo = __hmin2(lo, *reinterpret_cast<const __half2*>(&x));
    }
    part[0][g][p] = *reinterpret_cast<const uint32_t*>(&hi);
    part[1][g][p] = *reinterpret_cast<const uint32_t*>(&lo);
    __syncthreads();
    if (g != 0) return;
    uint32_t* out = reinterpret_cast<uint32_t*>(
        a.bounds + (((long long)c.slot * a.n_layers + at.l) * a.n_heads + at.h) * 2 * D);
#pragma unroll
    for (int j = 1; j < G; ++j) {
        hi = __hmax2(hi, *reinterpret_cast<const __half2*>(&part[0][j][p]));
        lo = __hmin2(lo, *reinterpret_cast<const __half2*>(&part[1][j][p]));
    }
    if (c.dst_row > 0) {
        const uint32_t oh = out[p], ol = out[P + p];
        hi = __hmax2(hi, *reinterpret_cast<const __half2*>(&oh));
        lo = __hmin2(lo, *reinterpret_cast<const __half2*>(&ol));
    }
    out[p] = *reinterpret_cast<const uint32_t*>(&hi);
    out[P + p] = *reinterpret_cast<const uint32_t*>(&lo);
}

// ---------------------------------------------------------------------------
// Read back: rows [dst_row, dst_row + n_rows) of a slot to rows [src_row, ...)
// of the packed tensors, as fp16(value * S).  fp16 and fp8 rows are read in
// 16 bytes of output per thread and step; an fp4 tile is staged in shared
// memory (its rows are permuted) and a thread takes a block of 16 dims.
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t scaled(uint32_t h, float mul) {
    if (mul == 1.f) return h;                          // (the same for the whole launch)
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    return pack_half2(f.x * mul, f.y * mul);
}

template <int C, int D, int EB, int N>
__global__ void __launch_bounds__(kRowThreads) read_rows_kernel(const __grid_constant__ RowArgs<N> a) {
    const Where at = where(a);
    const ScatterChunk c = at.c;
    const uint8_t* src = a.pool + tile_at<C, D, EB>(c.slot, a.n_layers, at.l, a.n_heads, at.h);
    const long long row0 = (long long)at.l * a.total_rows + c.src_row;
    uint16_t* const ok = const_cast<uint16_t*>(a.k);
    uint16_t* const ov = const_cast<uint16_t*>(a.v);
    if constexpr (EB != 0) {
        constexpr int NV = D / 8;
        const long long vofs = (long long)a.n_heads * C * D * EB;
        const int half = c.n_rows * NV;
        for (int i = threadIdx.x; i < 2 * half; i += kRowThreads) {
            const bool isv = i >= half;
            const int r = (isv ? i - half : i) / NV, x = i % NV;
            const uint8_t* s = src + (isv ? vofs : 0) + ((c.dst_row + r) * D + x * 8) * EB;
            uint4 o;
            if constexpr (EB == 2) {
                o = __ldcs(reinterpret_cast<const uint4*>(s));
            } else {
                const uint2 b = __ldcs(reinterpret_cast<const uint2*>(s));
                const float mul = isv ? a.v_mul : a.k_mul;
                o = make_uint4(scaled(f16x2_from_e4m3x2(b.x & 0xffffu), mul), scaled(f16x2_from_e4m3x2(b.x >> 16), mul),
                               scaled(f16x2_from_e4m3x2(b.y & 0xffffu), mul), scaled(f16x2_from_e4m3x2(b.y >> 16), mul));
            }
            __stcs(reinterpret_cast<uint4*>((isv ? ov : ok) + ((row0 + r) * a.n_heads + at.h) * D + x * 8), o);
        }
    } else {
        using T = F4Tile<C, D>;
        __shared__ __align__(16) uint8_t tile[T::kBytes];
        for (int i = threadIdx.x; i < T::kBytes / 16; i += kRowThreads)
            reinterpret_cast<uint4*>(tile)[i] = __ldcs(reinterpret_cast<const uint4*>(src) + i);
        __syncthreads();
        constexpr int NB = D / 16;
        const int z = c.dst_row + c.n_rows;
        auto write = [&](uint16_t* rows, int tok, int blk, const uint32_t (&w)[8]) {
            if (tok < c.dst_row || tok >= z) return;
            uint4* o = reinterpret_cast<uint4*>(rows + ((row0 + tok - c.dst_row) * a.n_heads + at.h) * D + blk * 16);
            __stcs(o, make_uint4(w[0], w[1], w[2], w[3]));
            __stcs(o + 1, make_uint4(w[4], w[5], w[6], w[7]));
        };
        // keys token by token, values by the pairs of tokens that share bytes
        for (int i = threadIdx.x; i < c.n_rows * NB; i += kRowThreads) {
            const int blk = i % NB, tok = c.dst_row + i / NB;
            const uint32_t s2 = f16x2_from_e4m3x2(tile[T::kKScales + f4_k_scale<D>(tok, blk)] * 0x101u);
            uint32_t w[8];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const uint32_t b = *reinterpret_cast<const uint16_t*>(tile + f4_k_byte<D>(tok, blk * 16 + 4 * t));
                w[2 * t] = scaled(mul_f16x2(f16x2_from_e2m1x2(b), s2), a.k_mul);
                w[2 * t + 1] = scaled(mul_f16x2(f16x2_from_e2m1x2(b >> 8), s2), a.k_mul);
            }
            write(ok, tok, blk, w);
        }
        for (int i = threadIdx.x; i < C / 2 * NB; i += kRowThreads) {
            const int pair = i / NB, blk = i % NB, tok = (pair >> 2) * 8 + (pair & 3);
            if ((tok < c.dst_row || tok >= z) && (tok + 4 < c.dst_row || tok + 4 >= z)) continue;
            const uint32_t s2 = f16x2_from_e4m3x2(
                *reinterpret_cast<const uint16_t*>(tile + T::kVScales + f4_v_scale<D>(tok, blk)));
            uint32_t w0[8], w1[8];
#pragma unroll
            for (int g = 0; g < 8; ++g) {
                const uint8_t* b = tile + T::kVCodes + f4_v_byte<D>(pair, blk * 16 + 2 * g);
                const uint32_t x = mul_f16x2(f16x2_from_e2m1x2(b[0]), s2), y = mul_f16x2(f16x2_from_e2m1x2(b[D / 16]), s2);
                w0[g] = scaled(__byte_perm(x, y, 0x5410), a.v_mul);
                w1[g] = scaled(__byte_perm(x, y, 0x7632), a.v_mul);
            }
            write(ov, tok, blk, w0);
            write(ov, tok + 4, blk, w1);
        }
    }
}

}  // namespace dev

namespace {

enum class RowOp { kStore4, kBounds, kRead };

template <int C, int D, int EB, int N>
void launch_rows(RowOp op, unsigned blocks, const dev::RowArgs<N>& a, cudaStream_t s) {
    if (op == RowOp::kStore4) {
        if constexpr (EB == 0) dev::fp4_store_kernel<C, D, N><<<blocks, dev::kRowThreads, 0, s>>>(a);
    } else if (op == RowOp::kBounds) {
        dev::key_bounds_kernel<C, D, EB, N><<<blocks, dev::kRowThreads, 0, s>>>(a);
    } else {
        dev::read_rows_kernel<C, D, EB, N><<<blocks, dev::kRowThreads, 0, s>>>(a);
    }
}

template <int D, int EB, int N>
bool pick_chunk(int chunk, RowOp op, unsigned blocks, const dev::RowArgs<N>& a, cudaStream_t s) {
    if (chunk == 16) launch_rows<16, D, EB, N>(op, blocks, a, s);
    else if (chunk == 32) launch_rows<32, D, EB, N>(op, blocks, a, s);
    else if (chunk == 64 && D <= 128) launch_rows<64, D <= 128 ? D : 128, EB, N>(op, blocks, a, s);
    else return false;
    return true;
}

template <int N>
int run_rows(const Pool& p, RowOp op, const void* k, const void* v, int32_t total_rows, const ScatterChunk* ch,
             size_t n, cudaStream_t s) {
    const PoolCfg& c = p.cfg;
    dev::RowArgs<N> a;
    a.k = static_cast<const uint16_t*>(k);
    a.v = static_cast<const uint16_t*>(v);
    a.pool = static_cast<uint8_t*>(p.kv);
    a.slot_ntok = reinterpret_cast<int32_t*>(a.pool + pool_tile_bytes(c));
    a.bounds = (c.flags & CA_CHUNK_BOUNDS) ? reinterpret_cast<uint16_t*>(a.pool + pool_bounds_offset(c)) : nullptr;
    a.total_rows = total_rows;
    a.n_chunks = (int32_t)n;
    a.n_layers = c.n_layers;
    a.n_heads = kv_heads(c);
    const bool quant = (c.flags & (CA_KV_FP8 | CA_KV_FP4)) != 0;
    const float ks = quant ? kv_scale_of(c.k_scale) : 1.f, vs = quant ? kv_scale_of(c.v_scale) : 1.f;
    a.k_mul = op == RowOp::kRead ? ks : 1.f / ks;
    a.v_mul = op == RowOp::kRead ? vs : 1.f / vs;
    std::copy(ch, ch + n, a.ch);
    const unsigned blocks = (unsigned)(n * c.n_layers * a.n_heads);
    const int D = c.head_dim;
    bool ok = false;
    if (c.flags & CA_KV_FP4) {
        if (D == 64) ok = pick_chunk<64, 0>(c.chunk, op, blocks, a, s);
        else if (D == 128) ok = pick_chunk<128, 0>(c.chunk, op, blocks, a, s);
    } else if (c.flags & CA_KV_FP8) {
        if (D == 128) ok = pick_chunk<128, 1>(c.chunk, op, blocks, a, s);
    } else {
        if (D == 64) ok = pick_chunk<64, 2>(c.chunk, op, blocks, a, s);
        else if (D == 128) ok = pick_chunk<128, 2>(c.chunk, op, blocks, a, s);
        else if (D == 256) ok = pick_chunk<256, 2>(c.chunk, op, blocks, a, s);
    }
    if (!ok) return CA_ERR_UNSUPPORTED;
    if (cudaGetLastError() != cudaSuccess) return CA_ERR_CUDA;
    count_launch();
    return CA_OK;
}

int rows(const Pool& p, RowOp op, const void* k, const void* v, int32_t total_rows,
         const std::vector<ScatterChunk>& chunks, void* stream) {
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    // grid.x holds chunks x layers x heads
    const size_t per = (size_t)p.cfg.n_layers * kv_heads(p.cfg);
    if (per > (size_t)INT32_MAX) return CA_ERR_UNSUPPORTED;
    const size_t most = std::max<size_t>(1, std::min<size_t>(dev::kManyChunks, (size_t)INT32_MAX / per));
    for (size_t i = 0; i < chunks.size();) {
        const size_t n = std::min(most, chunks.size() - i);
        const ScatterChunk* c = chunks.data() + i;
        const int st = n <= dev::kFewChunks    ? run_rows<dev::kFewChunks>(p, op, k, v, total_rows, c, n, s)
                       : n <= dev::kSomeChunks ? run_rows<dev::kSomeChunks>(p, op, k, v, total_rows, c, n, s)
                                               : run_rows<dev::kManyChunks>(p, op, k, v, total_rows, c, n, s);
        if (st) return st;
        i += n;
    }
    return CA_OK;
}

}  // namespace

int launch_fp4_store(const Pool& p, const void* k, const void* v, int32_t total_rows,
                     const std::vector<ScatterChunk>& chunks, void* stream) {
    return rows(p, RowOp::kStore4, k, v, total_rows, chunks, stream);
}

int launch_key_bounds(const Pool& p, const std::vector<ScatterChunk>& chunks, void* stream) {
    return rows(p, RowOp::kBounds, nullptr, nullptr, 0, chunks, stream);
}

int launch_read_rows(const Pool& p, void* k, void* v, int32_t total_rows, const std::vector<ScatterChunk>& chunks,
                     void* stream) {
    return rows(p, RowOp::kRead, k, v, total_rows, chunks, stream);
}

}  // namespace ca
