// qc_lds.hpp -- loads from memory straight into LDS, for the tiled products.
#pragma once
#include "qc_matrix.hpp"

namespace qc {

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void* base, int bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, bytes, 0x00020000);
}

// 16 bytes a lane from rsrc + voff + soff straight into LDS, lane i at lds +
// 16 i.  Written as asm because the compiler takes every LDS access after
// the builtin as dependent on it and waits for the load before the next
// fragment read; it returns nothing in registers, and lds_landed() is the
// wait that its readers need.  (m0, which holds the address in LDS, is a
// reserved register: clang warns against naming it as clobbered, sets it right
// before each use of its own, and has none in the kernels that include this.)
__device__ __forceinline__ void load_lds16(__amdgpu_buffer_rsrc_t rsrc, uint32_t lds, int voff, int soff) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                 :
                 : "s"(__builtin_amdgcn_readfirstlane((int)lds)), "v"(voff), "s"(rsrc), "s"(soff)
                 : "memory");
}
// The same with 4 bytes a lane, lane i at lds + 4 i.
__device__ __forceinline__ void load_lds4(__amdgpu_buffer_rsrc_t rsrc, uint32_t lds, int voff, int soff) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, %3 offen lds"
                 :
                 : "s"(__builtin_amdgcn_readfirstlane((int)lds)), "v"(voff), "s"(rsrc), "s"(soff)
                 : "memory");
}
// This wave's loads into LDS have landed and its LDS accesses are done; then
// every wave's are.
__device__ __forceinline__ void lds_landed() {
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
}
// As lds_landed, but the wave's N newest loads may still be on their way.
template <int N>
__device__ __forceinline__ void lds_landed_but() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" : : "n"(N) : "memory");
}
__device__ __forceinline__ uint32_t lds_addr(const void* p) {
    return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)p;
}

// Block b of `blocks` to tile (x, y) of a tx x ty grid.  Consecutive blocks go
// to the eight XCDs in turn; each XCD gets a contiguous run of tiles, walked in
// columns of G tiles in y, so that the tiles an XCD works on at one time (32
// compute units) share rows and columns in its L2.
struct Tile2 {
    int x, y;
};
template <int G>
__device__ __forceinline__ Tile2 tile_of(uint32_t b, uint32_t tx, uint32_t ty) {
    const uint32_t total = tx * ty, q = total / 8, r = total % 8, xcd = b % 8;
    const uint32_t id = xcd * q + min(xcd, r) + b / 8;
    const uint32_t band = id / (G * tx), first = band * G, rows = min(ty - first, (uint32_t)G);
    const uint32_t in = id - band * G * tx;
    return Tile2{(int)(in / rows), (int)(first + in % rows)};
}

}  // namespace qc
