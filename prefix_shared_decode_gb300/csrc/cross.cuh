// What the kernels over query blocks share.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "ca_internal.h"
#include "device.cuh"

namespace ca {
namespace dev {

struct CrossParams {
    const uint16_t* q;            // [rows of all blocks][H][D]
    uint16_t* out;
    const BlockItem* items;
    const BlockJoin* joins;
    const int32_t* cta_begin;     // [places + 1] items of each place
    const int32_t* q_off;         // [b + 1] first row of each block
    const int32_t* list_slots;
    const int32_t* slot_ntok;
    const uint8_t* kv;
    int32_t* status;
    float* part_o;                // [parts][tile rows][D]
    float2* part_ms;              // [parts][tile rows]
    int32_t n_layers, n_heads, n_kv_heads, group, layer, capacity, causal, tile_rows, n_places;
    int32_t test_stall;           // test hook: waits that run out (kernels that wait)
    float scale_log2, out_scale;
};

// Context tokens of an item's sequence as the pool holds it now.
__device__ __forceinline__ int tokens_now(const CrossParams& p, const BlockItem& it, int chunk) {
    if (it.last_slot < 0 || it.last_slot >= p.capacity) return 0;
    return (it.n_chunks - 1) * chunk + min(max(p.slot_ntok[it.last_slot], 0), chunk);
}
// The element of q and out where row r of an item begins.
__device__ __forceinline__ size_t block_row(const CrossParams& p, const BlockItem& it, int r, int D) {
    const int row = it.row0 + r;
    return ((size_t)(it.q0 + row / p.group) * p.n_heads + it.head * p.group + row % p.group) * D;
}

}  // namespace dev

// cross_tiles.cu
int launch_cross_tiles(const Pool& p, const dev::CrossParams& a, cudaStream_t s);

}  // namespace ca
