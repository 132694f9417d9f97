// Attention of query blocks over the pool (cross attention to other states, and
// the rest of a prompt behind what the pool already holds): blocks of any
// number of rows, each over its sequence's whole context, causal or not.
//     out[r] = sum_t p_rt v_t / sum_t p_rt,  p_rt = exp(scale q_r . k_t - m_r)
// over the tokens t that row r sees, in one pass over the context with the
// running maximum m_r; a row that sees none gives zeros.
#include <cuda.h>
#include <cuda_runtime.h>

#include "cross.cuh"

namespace ca {
namespace dev {

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

namespace {

template <class K>
int join(K kernel, unsigned grid, const dev::CrossParams& a, cudaStream_t s) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t c = {};
    c.gridDim = dim3(grid);
    c.blockDim = dim3(256);
    c.stream = s;
    c.attrs = attr;
    c.numAttrs = 1;
    if (cudaLaunchKernelEx(&c, kernel, a) != cudaSuccess) return CA_ERR_CUDA;
    count_launch();
    return CA_OK;
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
    const int st = launch_cross_tiles(p, a, cs);
    if (st || s.joins.empty()) return st;
    const unsigned jg = (unsigned)(s.joins.size() * ((s.tile_rows + 7) / 8));
    if (c.head_dim == 256) return join(dev::cross_join_kernel<256>, jg, a, cs);
    if (c.head_dim == 128) return join(dev::cross_join_kernel<128>, jg, a, cs);
    return join(dev::cross_join_kernel<64>, jg, a, cs);
}

}  // namespace ca
