// Shared by the ragged grouped products: the checked group layout in shared memory,
// the tile schedule, and the masked store of an accumulator chunk.
#pragma once

#include <type_traits>

#include "moe_internal.h"
#include "sm100.cuh"

namespace moe {

// Expert e owns `count[e]` rows from `start[e]` on. `tiles[e]` is the first row tile
// of expert e and `tiles[E]` their number.
struct RaggedGroups {
  int32_t start[kMaxExperts];
  int32_t count[kMaxExperts];
  int32_t tiles[kMaxExperts + 1];
};

// Reads the layout (all threads of the CTA; it ends with a block barrier). A group
// that does not lie inside [0, rows) is recorded and treated as empty, so that no
// later access depends on a bad offset. TILE_ROWS: rows a tile.
template <int TILE_ROWS>
__device__ __forceinline__ void load_groups(RaggedGroups* g, const int32_t* group_start, const int32_t* offsets,
                                            int E, int64_t rows, int32_t* status) {
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    const int64_t lo = offsets[e], hi = offsets[e + 1];
    const int64_t s = group_start != nullptr ? group_start[e] : lo;
    int64_t c = hi - lo;
    if (c < 0 || s < 0 || s + c > rows) {
      report(status, DEV_BAD_GROUP);
      c = 0;
    }
    g->start[e] = c > 0 ? static_cast<int32_t>(s) : 0;
    g->count[e] = static_cast<int32_t>(c);
  }
  __syncthreads();
  if (threadIdx.x < 32) {  // one warp: a prefix sum over 32 experts a turn
    int carry = 0;
    for (int base = 0; base < E; base += 32) {
      const int e = base + static_cast<int>(threadIdx.x);
      const int mine = e < E ? (g->count[e] + TILE_ROWS - 1) / TILE_ROWS : 0;
      int incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, incl, o);
        if (static_cast<int>(threadIdx.x) >= o) incl += up;
      }
      if (e < E) g->tiles[e] = carry + incl - mine;
      carry += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (threadIdx.x == 0) g->tiles[E] = carry;
  }
  __syncthreads();
}

// The expert of row tile `mt`: the largest e with tiles[e] <= mt (an expert without
// rows owns no tile and is never found).
__device__ __forceinline__ int tile_expert(const RaggedGroups& g, int E, int mt) {
  int lo = 0, hi = E - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (g.tiles[mid] <= mt) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// 3-D tiled load global -> shared, completion counted on `bar`; c0 is the innermost coordinate.
__device__ __forceinline__ void tma_load_3d(const CUtensorMap* map, uint64_t* bar, void* dst, int32_t c0, int32_t c1,
                                            int32_t c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}

// One warp writes a 32 x 32 chunk whose row `lane` this thread holds in v, through
// a staging buffer of 32 rows of PITCH bytes so that each store instruction covers
// whole row pieces. Only the first `rows` rows and `cols` columns (a multiple of 8)
// are written; rows past a group's end belong to another group or to nobody.
template <typename T, int PITCH>
__device__ __forceinline__ void store_chunk_masked(unsigned char* stg, const float (&v)[32], T* g, int64_t ld, int rows,
                                                   int cols, int lane) {
  constexpr int CPP = ((PITCH - 16) / static_cast<int>(sizeof(T))) < 32 ? 16 : 32;  // columns a pass
  constexpr int RB = CPP * static_cast<int>(sizeof(T));
  constexpr int LPR = RB / 16;   // lanes a row on the way out
  constexpr int RPI = 32 / LPR;  // rows a store instruction
  constexpr int EPS = 16 / static_cast<int>(sizeof(T));  // elements of a 16-byte piece
  unsigned char* mine = stg + lane * PITCH;
#pragma unroll
  for (int p = 0; p < 32 / CPP; ++p) {
    if constexpr (std::is_same_v<T, float>) {
#pragma unroll
      for (int i = 0; i < CPP / 4; ++i)
        *reinterpret_cast<float4*>(mine + 16 * i) =
            make_float4(v[p * CPP + 4 * i], v[p * CPP + 4 * i + 1], v[p * CPP + 4 * i + 2], v[p * CPP + 4 * i + 3]);
    } else {
#pragma unroll
      for (int i = 0; i < CPP / 8; ++i) {
        const int b = p * CPP + 8 * i;
        uint4 w;
        w.x = pack_bf16x2(v[b], v[b + 1]);
        w.y = pack_bf16x2(v[b + 2], v[b + 3]);
        w.z = pack_bf16x2(v[b + 4], v[b + 5]);
        w.w = pack_bf16x2(v[b + 6], v[b + 7]);
        *reinterpret_cast<uint4*>(mine + 16 * i) = w;
      }
    }
    __syncwarp();
#pragma unroll
    for (int it = 0; it < 32 / RPI; ++it) {
      const int r = it * RPI + lane / LPR;
      const int seg = lane % LPR;
      const uint4 val = *reinterpret_cast<const uint4*>(stg + r * PITCH + seg * 16);
      if (r < rows && p * CPP + seg * EPS < cols)
        *reinterpret_cast<uint4*>(reinterpret_cast<unsigned char*>(g + r * ld + p * CPP) + seg * 16) = val;
    }
    __syncwarp();
  }
}

}  // namespace moe
