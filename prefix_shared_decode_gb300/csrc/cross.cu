// Attention of query blocks over the pool (cross attention to other states, and
// the rest of a prompt behind what the pool already holds): blocks of any
// number of rows, each over its sequence's whole context, causal or not.
//     out[r] = sum_t p_rt v_t / sum_t p_rt,  p_rt = exp(scale q_r . k_t - m_r)
// over the tokens t that row r sees, in one pass over the context with the
// running maximum m_r; a row that sees none gives zeros.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>

#include "cross.cuh"
#include "fp4.cuh"
#include "row_blocks.cuh"

namespace ca {
namespace dev {

constexpr int kCrossRows = 64, kCrossKeys = 64, kCrossThreads = 128;

// 64 tokens from t0 on of a head's keys and values as fp16 tiles (in units of
// the pool's scales), swizzled; tokens from n on are zeros.
template <int C, int D, int EB>
__device__ __forceinline__ void load_tiles(const CrossParams& p, const int32_t* slots, int head, int t0, int n, uint8_t* kt,
                                           uint8_t* vt) {
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    auto put = [](uint8_t* tile, int r, int k, const uint4& v) {
        *reinterpret_cast<uint4*>(tile + swz(r, k, kCrossKeys)) = v;
    };
    auto slot_of = [&](int t) {
        const int s = slots[t / C];
        if (s >= 0 && s < p.capacity) return s;
        set_status(p.status, CA_ERR_DEVICE_BOUNDS);
        return -1;
    };
    if constexpr (EB != 0) {
        for (int i = threadIdx.x; i < kCrossKeys * (D / 8); i += kCrossThreads) {
            const int r = i / (D / 8), x = i % (D / 8), t = t0 + r;
            const int slot = t < n ? slot_of(t) : -1;
            uint4 k = zero, v = zero;
            if (slot >= 0) {
                const long long row = (((long long)slot * p.n_layers + p.layer) * 2 * p.n_kv_heads + head) * C + t % C;
                const uint8_t* src = p.kv + (row * D + x * 8) * EB;
                const long long vofs = (long long)p.n_kv_heads * C * D * EB;
                if constexpr (EB == 2) {
                    k = *reinterpret_cast<const uint4*>(src);
                    v = *reinterpret_cast<const uint4*>(src + vofs);
                } else {
                    const uint2 a = *reinterpret_cast<const uint2*>(src), b = *reinterpret_cast<const uint2*>(src + vofs);
                    k = make_uint4(f16x2_from_e4m3x2(a.x & 0xffffu), f16x2_from_e4m3x2(a.x >> 16),
                                   f16x2_from_e4m3x2(a.y & 0xffffu), f16x2_from_e4m3x2(a.y >> 16));
                    v = make_uint4(f16x2_from_e4m3x2(b.x & 0xffffu), f16x2_from_e4m3x2(b.x >> 16),
                                   f16x2_from_e4m3x2(b.y & 0xffffu), f16x2_from_e4m3x2(b.y >> 16));
                }
            }
            put(kt, r, x, k);
            put(vt, r, x, v);
        }
    } else {
        using T = F4Tile<C, D>;
        constexpr int NB = D / 16;
        for (int i = threadIdx.x; i < kCrossKeys * NB; i += kCrossThreads) {
            const int r = i / NB, blk = i % NB, t = t0 + r;
            const int slot = t < n ? slot_of(t) : -1;
            uint32_t w[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
            if (slot >= 0) {
                const uint8_t* tile = p.kv + (((long long)slot * p.n_layers + p.layer) * p.n_kv_heads + head) * T::kBytes;
                const uint32_t s2 = f16x2_from_e4m3x2(tile[T::kKScales + f4_k_scale<D>(t % C, blk)] * 0x101u);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t b = *reinterpret_cast<const uint16_t*>(tile + f4_k_byte<D>(t % C, blk * 16 + 4 * j));
                    w[2 * j] = mul_f16x2(f16x2_from_e2m1x2(b & 0xffu), s2);
                    w[2 * j + 1] = mul_f16x2(f16x2_from_e2m1x2(b >> 8), s2);
                }
            }
            put(kt, r, 2 * blk, make_uint4(w[0], w[1], w[2], w[3]));
            put(kt, r, 2 * blk + 1, make_uint4(w[4], w[5], w[6], w[7]));
        }
        for (int i = threadIdx.x; i < kCrossKeys / 2 * NB; i += kCrossThreads) {
            const int pair = i / NB, blk = i % NB, r = (pair >> 2) * 8 + (pair & 3), t = t0 + r;
            const int slot = t < n ? slot_of(t) : -1;
            uint32_t w0[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u}, w1[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
            if (slot >= 0) {
                const uint8_t* tile = p.kv + (((long long)slot * p.n_layers + p.layer) * p.n_kv_heads + head) * T::kBytes;
                const int pr = f4_pair(t % C);
                const uint32_t s2 = f16x2_from_e4m3x2(
                    *reinterpret_cast<const uint16_t*>(tile + T::kVScales + f4_v_scale<D>(t % C, blk)));
#pragma unroll
                for (int g = 0; g < 8; ++g) {
                    const uint8_t* b = tile + T::kVCodes + f4_v_byte<D>(pr, blk * 16 + 2 * g);
                    const uint32_t x = mul_f16x2(f16x2_from_e2m1x2(b[0]), s2), y = mul_f16x2(f16x2_from_e2m1x2(b[D / 16]), s2);
                    w0[g] = __byte_perm(x, y, 0x5410);
                    w1[g] = __byte_perm(x, y, 0x7632);
                }
            }
            put(vt, r, 2 * blk, make_uint4(w0[0], w0[1], w0[2], w0[3]));
            put(vt, r, 2 * blk + 1, make_uint4(w0[4], w0[5], w0[6], w0[7]));
            put(vt, r + 4, 2 * blk, make_uint4(w1[0], w1[1], w1[2], w1[3]));
            put(vt, r + 4, 2 * blk + 1, make_uint4(w1[4], w1[5], w1[6], w1[7]));
        }
    }
}

// One item per CTA; a warp has 16 of its rows.
template <int C, int D, int EB>
__global__ void __launch_bounds__(kCrossThreads) cross_rows_kernel(const CrossParams p) {
    extern __shared__ __align__(1024) uint8_t smem[];
    constexpr int kTile = kCrossKeys * D * 2, QR = q_rows<D>();
    uint8_t* kt = smem;
    uint8_t* vt = smem + kTile;
    uint8_t* qt = smem + 2 * kTile;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const BlockItem it = p.items[blockIdx.x];
    const int G = p.group;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int n = min(tokens_now(p, it, C), it.c_end * C);
    const int32_t* slots = p.list_slots + it.list0;
    auto row_at = [&](int r) { return block_row(p, it, r, D); };
    for (int i = threadIdx.x; i < kCrossRows * (D / 8); i += kCrossThreads) {
        const int r = i / (D / 8), k = i % (D / 8);
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (r < it.rows) v = *reinterpret_cast<const uint4*>(p.q + row_at(r) + k * 8);
        *reinterpret_cast<uint4*>(qt + r / QR * (QR * D * 2) + swz(r % QR, k, QR)) = v;
    }
    const int r0 = warp * 16;
    const uint32_t qblock = smem_u32(qt) + r0 / QR * (QR * D * 2) + r0 % QR * 128;
    int lim[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) lim[k] = p.causal ? it.ctx - it.m + (it.row0 + r0 + g + 8 * k) / G : INT_MAX;
    float o[D / 8][4], mx[2] = {-INFINITY, -INFINITY}, s[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    for (int t0 = it.c_begin * C; t0 < n; t0 += kCrossKeys) {
        __syncthreads();
        load_tiles<C, D, EB>(p, slots, it.head, t0, n, kt, vt);
        __syncthreads();
        if (r0 < it.rows)
            cf_chunk<kCrossKeys, D, kCrossKeys>(smem_u32(kt), smem_u32(vt), min(kCrossKeys, n - t0), 0, t0, lim[0], lim[1],
                                                qblock, p.scale_log2, mx, s, o, lane);
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        s[k] += __shfl_xor_sync(kFull, s[k], 1);
        s[k] += __shfl_xor_sync(kFull, s[k], 2);
        const int r = r0 + g + 8 * k;
        if (r >= it.rows) continue;
        if (it.part >= 0) {
            float* dst = p.part_o + ((size_t)it.part * p.tile_rows + r) * D;
#pragma unroll
            for (int i = 0; i < D / 8; ++i) *reinterpret_cast<float2*>(dst + i * 8 + 2 * t4) = make_float2(o[i][2 * k], o[i][2 * k + 1]);
            if (t4 == 0) p.part_ms[(size_t)it.part * p.tile_rows + r] = make_float2(mx[k], s[k]);
        } else {
            const float inv = s[k] == 0.f ? 0.f : p.out_scale / s[k];
            uint16_t* dst = p.out + row_at(r);
#pragma unroll
            for (int i = 0; i < D / 8; ++i)
                *reinterpret_cast<uint32_t*>(dst + i * 8 + 2 * t4) = pack_half2(o[i][2 * k] * inv, o[i][2 * k + 1] * inv);
        }
    }
}

// A tile's pieces joined: one warp per row.
template <int D>
__global__ void __launch_bounds__(256) cross_join_kernel(const CrossParams p) {
    constexpr int DPL = D / 32;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int per = (p.tile_rows + 7) / 8;
    const BlockJoin j = p.joins[blockIdx.x / per];
    const int r = blockIdx.x % per * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (r >= j.rows) return;
    const int row = j.row0 + r;
    const size_t at = ((size_t)(p.q_off[j.seq] + row / p.group) * p.n_heads + j.head * p.group + row % p.group) * D;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    float M = -INFINITY, S = 0.f, acc[DPL];
#pragma unroll
    for (int d = 0; d < DPL; ++d) acc[d] = 0.f;
    for (int x = 0; x < j.n_parts; ++x) {
        const size_t id = (size_t)(j.part + x) * p.tile_rows + r;
        const float2 ms = __ldcg(&p.part_ms[id]);
        float o[DPL];
        ldcg_f<DPL>(p.part_o + id * D + lane * DPL, o);
        const float top = fmaxf(M, ms.x), mu = top == -INFINITY ? 0.f : top;
        const float a = ex2(M - mu), w = ms.x == -INFINITY ? 0.f : ex2(ms.x - mu);
        S = S * a + ms.y * w;
#pragma unroll
        for (int d = 0; d < DPL; ++d) acc[d] = acc[d] * a + o[d] * w;
        M = top;
    }
    const float inv = S == 0.f ? 0.f : p.out_scale / S;
    uint32_t h[DPL / 2];
#pragma unroll
    for (int i = 0; i < DPL / 2; ++i) h[i] = pack_half2(acc[2 * i] * inv, acc[2 * i + 1] * inv);
    uint16_t* dst = p.out + at + lane * DPL;
    if constexpr (DPL == 8) *reinterpret_cast<uint4*>(dst) = make_uint4(h[0], h[1], h[2], h[3]);
    else if constexpr (DPL == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(h[0], h[1]);
    else *reinterpret_cast<uint32_t*>(dst) = h[0];
}

}  // namespace dev

// fp16 pools: tiles for the 5th-generation tensor cores, an SM each.
static bool on_tiles(const PoolCfg& c) { return !(c.flags & (CA_KV_FP8 | CA_KV_FP4)); }
int cross_tile_rows(const PoolCfg& c) { return !on_tiles(c) ? dev::kCrossRows : c.head_dim == 256 ? 128 : 256; }
int cross_places(const Pool& p) { return (p.sms > 0 ? p.sms : 152) * (on_tiles(p.cfg) ? 1 : 2); }

namespace {

template <class K>
int run(K kernel, unsigned grid, unsigned threads, int smem, const dev::CrossParams& a, cudaStream_t s) {
    if (smem > 48 * 1024 &&
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
        return CA_ERR_CUDA;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t c = {};
    c.gridDim = dim3(grid);
    c.blockDim = dim3(threads);
    c.dynamicSmemBytes = (size_t)smem;
    c.stream = s;
    c.attrs = attr;
    c.numAttrs = 1;
    if (cudaLaunchKernelEx(&c, kernel, a) != cudaSuccess) return CA_ERR_CUDA;
    count_launch();
    return CA_OK;
}

template <int D, int EB>
int pick(int chunk, unsigned grid, const dev::CrossParams& a, cudaStream_t s) {
    constexpr int smem = (2 * dev::kCrossKeys + dev::kCrossRows) * D * 2;
    if (chunk == 16) return run(dev::cross_rows_kernel<16, D, EB>, grid, dev::kCrossThreads, smem, a, s);
    if (chunk == 32) return run(dev::cross_rows_kernel<32, D, EB>, grid, dev::kCrossThreads, smem, a, s);
    if constexpr (D <= 128)
        if (chunk == 64) return run(dev::cross_rows_kernel<64, D, EB>, grid, dev::kCrossThreads, smem, a, s);
    return CA_ERR_UNSUPPORTED;
}

}  // namespace

int launch_cross(const Pool& p, const Sched& s, int32_t layer, const void* q, void* out, float scale, void* ws, void* stream) {
    const PoolCfg& c = p.cfg;
    unsigned char* dev8 = static_cast<unsigned char*>(s.dev);
    unsigned char* w8 = static_cast<unsigned char*>(ws);
    const bool quant = (c.flags & (CA_KV_FP8 | CA_KV_FP4)) != 0;
    dev::CrossParams a{};
    a.q = static_cast<const uint16_t*>(q);
    a.out = static_cast<uint16_t*>(out);
    a.items = reinterpret_cast<const BlockItem*>(dev8 + s.layout.items);
    a.joins = reinterpret_cast<const BlockJoin*>(dev8 + s.layout.joins);
    a.q_off = reinterpret_cast<const int32_t*>(dev8 + s.layout.q_off);
    a.list_slots = reinterpret_cast<const int32_t*>(dev8 + s.layout.list_slots);
    a.slot_ntok = reinterpret_cast<const int32_t*>(static_cast<const unsigned char*>(p.kv) + pool_tile_bytes(c));
    a.kv = static_cast<const uint8_t*>(p.kv);
    a.status = reinterpret_cast<int32_t*>(dev8 + s.layout.status);
    a.part_o = reinterpret_cast<float*>(w8 + s.ws.part_o);
    a.part_ms = reinterpret_cast<float2*>(w8 + s.ws.part_ms);
    a.n_layers = c.n_layers;
    a.n_heads = c.n_heads;
    a.n_kv_heads = kv_heads(c);
    a.group = c.n_heads / a.n_kv_heads;
    a.layer = layer;
    a.capacity = c.capacity_slots;
    a.causal = (s.flags & CA_SCHED_CAUSAL) ? 1 : 0;
    a.tile_rows = s.tile_rows;
    a.scale_log2 = scale * 1.4426950408889634f * (quant ? kv_scale_of(c.k_scale) : 1.f);
    a.out_scale = quant ? kv_scale_of(c.v_scale) : 1.f;
    a.cta_begin = reinterpret_cast<const int32_t*>(dev8 + s.layout.cta_begin);
    a.n_places = s.n_places;
    if (s.items.empty()) return CA_OK;
    if (s.stall_calls > 0) {
        a.test_stall = 1;
        --s.stall_calls;
    }
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    const unsigned grid = (unsigned)s.items.size();
    int st = CA_ERR_UNSUPPORTED;
    if (c.flags & CA_KV_FP4) {
        if (c.head_dim == 64) st = pick<64, 0>(c.chunk, grid, a, cs);
        else if (c.head_dim == 128) st = pick<128, 0>(c.chunk, grid, a, cs);
    } else if (c.flags & CA_KV_FP8) {
        if (c.head_dim == 128) st = pick<128, 1>(c.chunk, grid, a, cs);
    } else {
        st = launch_cross_tiles(p, a, cs);
    }
    if (st || s.joins.empty()) return st;
    const unsigned jg = (unsigned)(s.joins.size() * ((s.tile_rows + 7) / 8));
    if (c.head_dim == 256) return run(dev::cross_join_kernel<256>, jg, 256, 0, a, cs);
    if (c.head_dim == 128) return run(dev::cross_join_kernel<128>, jg, 256, 0, a, cs);
    return run(dev::cross_join_kernel<64>, jg, 256, 0, a, cs);
}

}  // namespace ca
