// Shared by the ragged grouped products: the checked group layout in shared memory,
// the tile schedule, the issue of MMAs, and the masked store of an accumulator chunk.
#pragma once

#include <type_traits>

#include "moe_internal.h"
#include "sm100.cuh"

namespace moe {

// Expert e owns `count[e]` rows from `start[e]` on, cut into row tiles, each with the
// same number of column tiles. Experts come in the order `order[0..E)`; `tiles[j]` is the
// number of the j-th one's first tile and `tiles[E]` their sum.
struct RaggedGroups {
  int32_t start[kMaxExperts];
  int32_t count[kMaxExperts];
  int32_t order[kMaxExperts];
  int32_t per[kMaxExperts];  // rows of a row tile
  int32_t tiles[kMaxExperts + 1];
};

// Every warp works out each of its tiles by itself, so divisions go by multiplication
// and the search is one of the whole warp (131072 rows of 4-bit values over 64 experts:
// 283 us with plain divisions and a binary search, 274 so).

// x / d for 0 <= x < 2^31 by a multiplication.
struct FastDiv {
  uint32_t d, m;
  __device__ explicit FastDiv(int divisor)
      : d(static_cast<uint32_t>(divisor)), m(divisor > 1 ? 0xFFFFFFFFu / static_cast<uint32_t>(divisor) + 1u : 0u) {}
  __device__ int operator()(int x) const {
    const uint32_t u = static_cast<uint32_t>(x);
    const uint32_t q = d == 1u ? u : __umulhi(u, m);  // exact or one too large
    return static_cast<int>(q * d > u ? q - 1u : q);
  }
};

// A group's row tiles: as few as tiles of at most MOST rows allow, all of one size, a
// multiple of UNIT, but the last.
template <int MOST, int UNIT>
__device__ __forceinline__ int rows_a_tile(int count) {
  const int least = max(1, (count + MOST - 1) / MOST);
  return min(MOST, max(UNIT, ((count + least - 1) / least + UNIT - 1) / UNIT * UNIT));
}

// The rows of group e. A group that does not lie inside [0, rows) is recorded and treated
// as empty, so that no later access depends on a bad offset.
__device__ __forceinline__ void checked_group(const int32_t* group_start, const int32_t* offsets, int e, int64_t rows,
                                              int32_t* start, int32_t* count, int32_t* status) {
  const int64_t lo = offsets[e], hi = offsets[e + 1];
  const int64_t s = group_start != nullptr ? group_start[e] : lo;
  int64_t c = hi - lo;
  if (c < 0 || (c > 0 && (s < 0 || s + c > rows))) {  // (an empty group may start anywhere)
    report(status, DEV_BAD_GROUP);
    c = 0;
  }
  *start = c > 0 ? static_cast<int32_t>(s) : 0;
  *count = static_cast<int32_t>(c);
}

// Reads the layout (all threads of the CTA; it ends with a block barrier). cols: column
// tiles of a row tile. SORTED: the experts come by falling row count (equal counts in
// order of e).
template <int MOST, int UNIT, bool SORTED>
__device__ __forceinline__ void load_groups(RaggedGroups* g, const int32_t* group_start, const int32_t* offsets, int E,
                                            int64_t rows, int cols, int32_t* status) {
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    checked_group(group_start, offsets, e, rows, &g->start[e], &g->count[e], status);
    g->per[e] = rows_a_tile<MOST, UNIT>(g->count[e]);
    if constexpr (!SORTED) g->order[e] = e;
  }
  __syncthreads();
  if constexpr (SORTED) {
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
      int rank = 0;
      const int mine = g->count[e];
      for (int o = 0; o < E; ++o) rank += g->count[o] > mine || (g->count[o] == mine && o < e);
      g->order[rank] = e;
    }
    __syncthreads();
  }
  if (threadIdx.x < 32) {  // one warp: a prefix sum over 32 experts a turn
    const int lane = static_cast<int>(threadIdx.x);
    int carry = 0;
    for (int base = 0; base < E; base += 32) {
      const int j = base + lane;
      int mine = 0;
      if (j < E) {
        const int e = g->order[j], per = g->per[e];
        mine = (g->count[e] + per - 1) / per * cols;
      }
      int incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
      }
      if (j < E) g->tiles[j] = carry + incl - mine;
      carry += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) g->tiles[E] = carry;
  }
  __syncthreads();
}

// The place in `order` of the expert of tile L: the largest j with tiles[j] <= L (an
// expert without rows owns no tile and is never found). The whole warp.
__device__ __forceinline__ int tile_place(const RaggedGroups& g, int E, int L) {
  const int lane = static_cast<int>(threadIdx.x & 31u);
  int n = 0;
  for (int base = 0; base < E; base += 32)
    n += __popc(__ballot_sync(0xffffffffu, base + lane < E && g.tiles[base + lane] <= L));
  return n - 1;
}

// Issuing MMAs. One thread feeds the tensor core, and its own instructions bound the rate
// when each MMA's operands are put together by divergent code: 230 cycles an MMA of 256 x
// 256 x 16 that the tensor cores take 128 for (measured with the loads taken out). So
//  - the high word of a descriptor is a constant, the low word (address and leading
//    offset) is carried from stage to stage, and a step adds a constant to it (195);
//  - the whole warp runs the loop on values that the compiler can see to be the same in
//    every lane (uniform()), and one lane is elected around the instructions alone, so
//    that their operands live in uniform registers (150).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(p));
  return p != 0;
}

__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(0xffffffffu, v, 0); }
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }

struct DescLo {
  uint32_t a, b;
};

constexpr uint32_t kDescHiSw128 = (1024u >> 4) | (1u << 14) | (2u << 29);

__device__ __forceinline__ uint32_t desc_lo_sw128(uint32_t saddr, uint32_t lbo_bytes) {
  return ((saddr >> 4) & 0x3FFFu) | ((lbo_bytes >> 4) << 16);
}

template <bool PAIR>
__device__ __forceinline__ void umma_bf16_lo(uint32_t d, uint32_t alo, uint32_t blo, uint32_t idesc,
                                             uint32_t accumulate) {
  if constexpr (PAIR)
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 ad, bd;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 ad, {%1, %5};\n\tmov.b64 bd, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], ad, bd, %3, p;\n\t}\n" ::"r"(d),
        "r"(alo), "r"(blo), "r"(idesc), "r"(accumulate), "r"(kDescHiSw128)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 ad, bd;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 ad, {%1, %5};\n\tmov.b64 bd, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], ad, bd, %3, p;\n\t}\n" ::"r"(d),
        "r"(alo), "r"(blo), "r"(idesc), "r"(accumulate), "r"(kDescHiSw128)
        : "memory");
}

// The MMAs of a stage of four steps, `steps` of them (fewer at a reduction's end).
// A_STEP, B_STEP: bytes between the steps' operands.
template <bool PAIR, int A_STEP, int B_STEP>
__device__ __forceinline__ void umma_stage(uint32_t d, DescLo lo, uint32_t idesc, bool first, int steps) {
  umma_bf16_lo<PAIR>(d, lo.a, lo.b, idesc, first ? 0u : 1u);
  if (steps == 4) {
#pragma unroll
    for (int kk = 1; kk < 4; ++kk)
      umma_bf16_lo<PAIR>(d, lo.a + kk * (A_STEP >> 4), lo.b + kk * (B_STEP >> 4), idesc, 1u);
  } else {
    for (int kk = 1; kk < steps; ++kk)
      umma_bf16_lo<PAIR>(d, lo.a + kk * (A_STEP >> 4), lo.b + kk * (B_STEP >> 4), idesc, 1u);
  }
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

// tma_load_3d by a CTA of a pair, its bytes counted on the leader's barrier (see tma_load_2d_pair).
__device__ __forceinline__ void tma_load_3d_pair(const CUtensorMap* map, uint64_t* bar, void* dst, int32_t c0,
                                                 int32_t c1, int32_t c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar) & 0xFEFFFFFFu), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}

// Arrival on another CTA's barrier by an epilogue warp that has read its accumulator. It
// orders TMEM reads only (tcgen05.wait::ld and the fence before it do), so it is relaxed:
// a releasing one waits until the warp's stores to global memory have been performed
// (131072 rows over 64 experts: gradients 1.70 -> 1.65 ms, the 4-bit product 274 -> 266 us).
__device__ __forceinline__ void mbar_arrive_cluster_relaxed(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

__device__ __forceinline__ void mbar_arrive_relaxed(uint64_t* bar) {
  asm volatile("mbarrier.arrive.relaxed.cta.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// One warp writes a 32 x 32 chunk whose COLUMN `lane` this thread holds in v: v[j] is
// the element of row j. fp32 rows leave as 128 bytes a store; bf16 neighbours swap one
// of every two rows, packed, and two rows of 64 bytes leave a store. Only the first
// `rows` rows and `cols` columns (a multiple of 8) are written. Short reductions are
// bound by this (54425 rows of 120 over 51 experts, 1432 wide: 59 us with values swapped
// before they are packed and every store predicated, 57 so).
template <typename T, bool WHOLE>
__device__ __forceinline__ void store_columns(const float (&v)[32], T* g, int64_t ld, int rows, int cols, int lane) {
  if constexpr (std::is_same_v<T, float>) {
    float* p = g + lane;
    const int mine = lane < cols ? rows : 0;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      if (WHOLE || j < mine) *p = v[j];
      p += ld;
    }
  } else {
    const bool odd = (lane & 1) != 0;
    T* p = g + (lane & ~1) + (odd ? ld : 0);
    const int mine = lane < cols ? rows - (odd ? 1 : 0) : 0;
    const uint32_t pick = odd ? 0x3276u : 0x5410u;  // (other.hi, own.hi) or (own.lo, other.lo)
#pragma unroll
    for (int j = 0; j < 32; j += 2) {
      const uint32_t own = pack_bf16x2(v[j], v[j + 1]);
      const uint32_t w = __byte_perm(own, __shfl_xor_sync(0xffffffffu, own, 1), pick);
      if (WHOLE || j < mine) *reinterpret_cast<uint32_t*>(p) = w;
      p += 2 * ld;
    }
  }
}

template <typename T>
__device__ __forceinline__ void store_chunk_turned(const float (&v)[32], T* g, int64_t ld, int rows, int cols,
                                                   int lane) {
  if (rows >= 32 && cols >= 32)
    store_columns<T, true>(v, g, ld, rows, cols, lane);
  else
    store_columns<T, false>(v, g, ld, rows, cols, lane);
}

}  // namespace moe
