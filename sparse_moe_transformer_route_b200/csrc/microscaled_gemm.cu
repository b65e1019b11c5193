// The grouped product on microscaled 4-bit operands (MXFP4 or NVFP4):
//   y[r] = g_x g_w[e] * sum_k (code_x s_x)(code_w s_w)      for the rows r of expert e
// with the block-scaled form of tcgen05.mma: 64 terms an instruction, codes packed
// two to a byte in shared memory, block scales in TMEM, fp32 accumulation. The
// products of scaled elements are exact there; the two tensor scales multiply the
// finished sum. As in ragged_gemm.cu the weight is the MMA's M operand and the rows its
// N operand, of any multiple of 16 rows.
//
// Scales. The instruction reads the scale bytes of row r (of either operand) from
// TMEM lane r % 32, column r / 32, four bytes a column: with NVFP4 the four blocks of
// one 64-term step, with MXFP4 the four blocks of two steps. One tcgen05.cp
// (32x128b.warpx4) brings 128 rows' column set from 512 bytes of shared memory whose
// 16-byte line i holds the words of rows i, i + 32, i + 64, i + 96. In global memory
// scales are plain row-major bytes, so that a group may start at any row. TMA brings
// 32 bytes of each row, the scales of two stages of 256 terms (NVFP4) or four (MXFP4),
// and a warp per 128 rows turns its 4 KB round in place: 16-byte reads and stores, no
// bank conflicts (32-byte swizzle; 16 bytes at a time TMA's own rate, about a row a
// clock, was the bound). Only widths whose scale rows are no multiple of 16 bytes, which
// TMA cannot address, go through registers (64 experts, 32768 rows of 2016: 127 us; of
// 2048: 90): the fence in front of the tensor core's reads waits for every load that a
// warp has in flight, so four sets of warps take the slots in turn (one set: 289).
//
// Structure per CTA (persistent, one an SM): warp 0 TMA of codes, warp 1 MMA issue,
// warps 2..9 epilogue, the rest scales. A 256-column accumulator pair and the
// scales do not fit TMEM's 512 columns side by side, so the two accumulators share
// 64 columns: the epilogue reads those first and then lets the next tile start.
// PAIR: a tile of 256 output columns on the two CTAs of a cluster, each with its 128 rows
// of the weight and half of the tile's rows in shared memory and the scales of its own
// 128 weight rows and of all the tile's rows; the leader issues cta_group::2 copies and
// MMAs for both (131072 rows, 64 experts: 338 us with one CTA a tile, 283 on pairs, 258
// with the accumulator's release relaxed, shorter tile lookups and scales looked up in
// shared memory; replayed graphs with a cold L2, in a loop of calls of some seconds 332 at
// the power cap). What bounds it is the
// operands' way into shared memory: 38 KB a stage whose MMAs take 512 cycles, five
// stages in flight, about 2 us from a stage's release to its next use.
// The scale warps arrive on the leader's barrier without a cluster-scope release: each
// CTA's lines are read from its own shared memory by its own tensor core (with one,
// 32768 rows of 2048 x 2048 took 141 us instead of 86).
// Every wait is bounded; a timeout is recorded in the status word.
#include <cudaTypedefs.h>

#include "ragged.cuh"

namespace moe {
namespace {

template <bool NV_, int BN_, bool O32_, bool PAIR_>
struct QCfg {
  static constexpr bool NV = NV_;
  static constexpr int BN = BN_;
  static constexpr bool O32 = O32_;
  static constexpr bool PAIR = PAIR_;
  using OutT = std::conditional_t<O32, float, __nv_bfloat16>;
  static constexpr int CTAS = PAIR ? 2 : 1;
  static constexpr int BM = 128 * CTAS;          // M: output columns a tile; BN: at most so many rows
  static constexpr int UNIT = 16 * CTAS;         // N is a multiple of this
  static constexpr int BK = 256;                 // terms a stage: one 128-byte swizzle row of codes
  static constexpr int UK = 64;                  // terms a tcgen05.mma
  static constexpr int SCALE_BYTES = NV ? 16 : 8;  // scale bytes of a row and stage
  static constexpr int WORDS = SCALE_BYTES / 4;  // TMEM column sets a stage
  static constexpr int SF_STAGES_PER = NV ? 2 : 4;  // stages whose scales fill a slot
  static constexpr int SF_BLOCK = 4096;          // 128 rows' scales of a slot: 8 words a row
  static constexpr int BBLK = (BN + 127) / 128;  // 128-row blocks of B
  static constexpr int B_ROWS = BN / CTAS;       // rows of B in this CTA's shared memory
  static constexpr int A_BYTES = 128 * 128;
  static constexpr int B_BYTES = B_ROWS * 128;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int SF_BYTES = (1 + BBLK) * SF_BLOCK;  // a slot
  static constexpr bool OVERLAP = BN == 256;
  // The tensor core's fp32 sum loses up to an ulp a step towards zero (terms of one sign,
  // against 64 bits: 6e-7 of the result after the 128 steps of k = 8192, 8e-6 after 512).
  // Where the result is fp32, the accumulator is therefore handed over every SUM_BLOCKS
  // stages (128 steps) and the parts are added in the result's own place, rounded to
  // nearest: the registers do not hold a tile's sums beside the rest. (Parts of 32 steps
  // would make 32768 rows of 4096 in 16 groups 40% slower.)
  static constexpr bool PARTS = O32;
  static constexpr int SUM_BLOCKS = 32;
  static constexpr uint32_t ACC1 = OVERLAP ? 192 : BN;  // first column of the second accumulator
  static constexpr uint32_t SFA_COL = 448;
  static constexpr uint32_t SFB_COL = SFA_COL + WORDS * 4;
  static constexpr uint32_t TMEM_COLS = 512;
  static constexpr int EPI_WARPS = 8;
  // scale warps: one for each 128 rows, in sets that take the slots in turn, so that the
  // loads of some are in flight while others write
  static constexpr int SF_WARPS = 1 + BBLK;
  static constexpr int SF_SETS = 4;
  static constexpr int THREADS = 64 + 32 * (EPI_WARPS + SF_SETS * SF_WARPS + 1);
  static constexpr int CHUNKS = (BN + 63) / 64;  // 32-column chunks of an epilogue warp
  static constexpr int MISC_BYTES = 1024 + static_cast<int>(sizeof(RaggedGroups)) + 4 * kMaxExperts;
  static constexpr int ROOM = 227 * 1024 - 1024 - MISC_BYTES;
  static constexpr int STAGES_FIT = (ROOM - 4 * SF_BYTES) / STAGE_BYTES;
  static constexpr int STAGES = STAGES_FIT > 8 ? 8 : STAGES_FIT;
  // the scales' way is longer by a pass through registers: their ring reaches further
  static constexpr int SF_FIT = (ROOM - STAGES * STAGE_BYTES) / SF_BYTES;
  // (a multiple of the sets: a slot is always the same set's, which has then seen every
  // phase of its barriers)
  static constexpr int SF_SLOTS = (SF_FIT > 8 ? 8 : SF_FIT) / SF_SETS * SF_SETS;
  static constexpr size_t SMEM_BYTES =
      1024 + static_cast<size_t>(STAGES) * STAGE_BYTES + static_cast<size_t>(SF_SLOTS) * SF_BYTES + MISC_BYTES;
  static_assert(STAGES >= 3 && SF_SLOTS >= 4 && SF_SLOTS % SF_SETS == 0 && (2 * STAGES + 3 * SF_SLOTS + 6) * 8 <= 1024 && THREADS >= kMaxExperts, "rings");
  static_assert(SMEM_BYTES > 114 * 1024, "one CTA an SM");
  static_assert(SFB_COL + WORDS * 4 * BBLK <= 512, "TMEM columns");
  static_assert(BN == 256 || (!PAIR && (BN == 128 || BN == 64 || BN == 32)), "tile N");
};

struct QArgs {
  const int32_t* group_start;
  const int32_t* offsets;
  const uint8_t* xs;
  const uint8_t* ws;
  const float* x_scale;
  const float* w_scale;
  int64_t rows;
  int E, n, k;
  bool tma_scales;  // scale rows are multiples of 16 bytes
  void* out;
  int32_t* status;
};

// Instruction descriptor of the block-scaled kinds, both operands E2M1 and K-major:
//   bits 4-5 B scale id; 7-9 A format, 10-11 B format (1 = E2M1); 17-22 N >> 3;
//   bit 23 scale format (0 = UE4M3, 1 = UE8M0); 27-28 M >> 7; 29-30 A scale id.
// A scale id picks the first byte used of each column's four.
__host__ __device__ constexpr uint32_t micro_idesc(bool nv, int M, int N, uint32_t sf_id) {
  return (sf_id << 4) | (1u << 7) | (1u << 10) | ((static_cast<uint32_t>(N) >> 3) << 17) | ((nv ? 0u : 1u) << 23) |
         ((static_cast<uint32_t>(M) >> 7) << 27) | (sf_id << 29);
}

// 128 rows' words from shared memory to TMEM. Descriptor of a scale block: no swizzle,
// 8-row groups of 16-byte lines 128 bytes apart; `lo` is its address >> 4.
template <bool PAIR>
__device__ __forceinline__ void scales_to_tmem(uint32_t taddr, uint32_t lo) {
  constexpr uint32_t hi = (128u >> 4) | (1u << 14);
  if constexpr (PAIR)
    asm volatile(
        "{\n\t.reg .b64 d;\n\tmov.b64 d, {%1, %2};\n\t"
        "tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], d;\n\t}\n" ::"r"(taddr),
        "r"(lo), "r"(hi)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .b64 d;\n\tmov.b64 d, {%1, %2};\n\t"
        "tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], d;\n\t}\n" ::"r"(taddr),
        "r"(lo), "r"(hi)
        : "memory");
}

#define MOE_UMMA_MICRO(GROUP, VEC)                                                                            \
  asm volatile(                                                                                               \
      "{\n\t.reg .pred p;\n\t.reg .b64 ad, bd;\n\t"                                                           \
      "setp.ne.b32 p, %6, 0;\n\t"                                                                             \
      "mov.b64 ad, {%1, %7};\n\tmov.b64 bd, {%2, %7};\n\t"                                                    \
      "tcgen05.mma.cta_group::" GROUP ".kind::mxf4nvf4.block_scale.scale_vec::" VEC                           \
      " [%0], ad, bd, %3, [%4], [%5], p;\n\t}\n" ::"r"(d),                                                    \
      "r"(alo), "r"(blo), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate), "r"(kDescHiSw128)                  \
      : "memory")

template <bool NV, bool PAIR>
__device__ __forceinline__ void umma_micro(uint32_t d, uint32_t alo, uint32_t blo, uint32_t idesc, uint32_t sfa,
                                           uint32_t sfb, uint32_t accumulate) {
  if constexpr (PAIR) {
    if constexpr (NV) MOE_UMMA_MICRO("2", "4X");
    else MOE_UMMA_MICRO("2", "2X");
  } else {
    if constexpr (NV) MOE_UMMA_MICRO("1", "4X");
    else MOE_UMMA_MICRO("1", "2X");
  }
}
#undef MOE_UMMA_MICRO

struct QTile {
  int e;
  int m0;    // first output column
  int n0;    // first row of the buffer
  int left;  // rows, of the group
  int N;     // the MMA's N
};

template <class C>
__device__ __forceinline__ QTile q_tile(const QArgs& a, const RaggedGroups& g, const FastDiv& by_m, int L) {
  QTile t;
  const int place = tile_place(g, a.E, L);
  t.e = g.order[place];
  const int in = L - g.tiles[place];
  const int rt = by_m(in);
  t.m0 = (in - rt * static_cast<int>(by_m.d)) * C::BM;
  const int count = g.count[t.e], per = g.per[t.e];
  t.n0 = g.start[t.e] + rt * per;
  t.left = min(per, count - rt * per);
  t.N = (t.left + C::UNIT - 1) / C::UNIT * C::UNIT;
  return t;
}

// The product of the two tensor scales as shift * lead, which multiply a sum in this order.
// Each scale may be anywhere in [2^-100, 2^117], so their product may leave fp32's normal
// range although its product with a sum does not (a sum of products of 4-bit values and
// block scales is 0 or at least 2^-20). It is then split in the middle, shift a power of
// two: sum * shift is exact, or overflows where the whole does, and * lead rounds once.
// Elsewhere lead is the rounded product and shift is 1.
struct TensorScales {
  float shift, lead;
};

__device__ __forceinline__ TensorScales tensor_scales(float gx, float gw) {
  const float m = fabsf(gx * gw);
  const bool normal = m >= 0x1p-126f && m <= 0x1.fffffep127f;
  if (normal || gx == 0.0f || gw == 0.0f || !isfinite(gx) || !isfinite(gw)) return {1.0f, gx * gw};
  int ex, ew;
  const float f = frexpf(gx, &ex) * frexpf(gw, &ew);  // rounded once, as the product above
  const int half = (ex + ew) / 2;
  return {ldexpf(1.0f, ex + ew - half), ldexpf(f, half)};
}

// Multiplies this warp's chunks of an accumulator by `shift` where they are, in TMEM. A
// second product for every element instead costs large products 3% (131072 rows of 2048 x
// 2048 over 64 experts: 268 and 276 us), a second loop for such tiles needs more registers
// than there are, and forming both factors a tile at a time costs 1.7%; every expert's
// lead is formed once a CTA and lies in shared memory (0.8%).
__device__ __forceinline__ void shift_chunks(uint32_t tb, int csel, int N, float shift) {
#pragma unroll 1
  for (int c = csel * 32; c < N; c += 64) {
#pragma unroll 1
    for (int h = 0; h < 32; h += 16) {
      uint32_t r[16];
      tmem_ld16(tb + c + h, r);
      tmem_ld_wait();
#pragma unroll
      for (int x = 0; x < 16; ++x) r[x] = __float_as_uint(__uint_as_float(r[x]) * shift);
      tmem_st16(tb + c + h, r);
    }
  }
  tmem_st_wait();
}

// r += shift * what store_chunk_turned has left of the parts before at the same place (this
// thread's own stores).
__device__ __forceinline__ void add_stored(uint32_t (&r)[32], const float* at, int64_t ld, int rows, int cols,
                                           float shift, int lane) {
  const volatile float* p = at + lane;  // (loads in this order, a few in flight: there are no more registers)
  const int mine = lane < cols ? rows : 0;
#pragma unroll
  for (int j0 = 0; j0 < 32; j0 += 4) {
    float had[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      had[j] = j0 + j < mine ? *p : 0.0f;
      p += ld;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) r[j0 + j] = __float_as_uint(fmaf(had[j], shift, __uint_as_float(r[j0 + j])));
  }
}

// Eight words of a scale row from byte `at` on, zero past the row's end. The row starts
// at any address: the (up to three) 16-byte pieces that cover the words are read whole
// and shifted together, but for one that would leave the buffer at `end`, which is read
// byte by byte.
__device__ __forceinline__ void load_scale_words(uint32_t (&w)[8], const uint8_t* row, int at, int row_bytes,
                                                 const uint8_t* end) {
  const uint8_t* p = row + at;
  const int bytes = min(32, row_bytes - at);
  const uint32_t off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p) & 15u);
  const uint8_t* base = p - off;
  uint32_t v[12];
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    uint4 q = make_uint4(0u, 0u, 0u, 0u);
    if (16 * i < bytes + static_cast<int>(off)) {
      if (base + 16 * i + 16 <= end) {
        q = __ldg(reinterpret_cast<const uint4*>(base) + i);
      } else {
        for (int b = 0; base + 16 * i + b < end; ++b) {
          const uint32_t byte = static_cast<uint32_t>(__ldg(base + 16 * i + b)) << (8 * (b & 3));
          if (b < 4) q.x |= byte;
          else if (b < 8) q.y |= byte;
          else if (b < 12) q.z |= byte;
          else q.w |= byte;
        }
      }
    }
    v[4 * i] = q.x;
    v[4 * i + 1] = q.y;
    v[4 * i + 2] = q.z;
    v[4 * i + 3] = q.w;
  }
  if (off & 8u) {
#pragma unroll
    for (int i = 0; i < 10; ++i) v[i] = v[i + 2];
  }
  if (off & 4u) {
#pragma unroll
    for (int i = 0; i < 9; ++i) v[i] = v[i + 1];
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    w[i] = __funnelshift_r(v[i], v[i + 1], 8 * (off & 3u));
    const int have = bytes - 4 * i;  // bytes of this word that belong to the row
    if (have < 4) w[i] &= have <= 0 ? 0u : (1u << (8 * have)) - 1u;
  }
}

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1)
    microscaled_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                            const __grid_constant__ CUtensorMap tmB32, const __grid_constant__ CUtensorMap tmSA,
                            const __grid_constant__ CUtensorMap tmSB, const __grid_constant__ CUtensorMap tmSB32,
                            const QArgs a) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  unsigned char* sf_base = smem + static_cast<size_t>(C::STAGES) * C::STAGE_BYTES;
  unsigned char* misc = sf_base + static_cast<size_t>(C::SF_SLOTS) * C::SF_BYTES;
  uint64_t* full = reinterpret_cast<uint64_t*>(misc);
  uint64_t* empty = full + C::STAGES;
  uint64_t* sf_raw = empty + C::STAGES;  // a stage's scales have landed as they lie in global memory
  uint64_t* sf_full = sf_raw + C::SF_SLOTS;
  uint64_t* sf_empty = sf_full + C::SF_SLOTS;
  uint64_t* acc_full = sf_empty + C::SF_SLOTS;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* drain = acc_empty + 2;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain + 1);
  uint32_t* far_flag = tmem_holder + 1;  // some expert's tensor scales have a shift
  RaggedGroups* groups = reinterpret_cast<RaggedGroups*>(misc + 1024);
  float* lead = reinterpret_cast<float*>(groups + 1);  // of every expert's tensor scales

  constexpr int CTAS = C::CTAS;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rank = C::PAIR ? static_cast<int>(cluster_ctarank()) : 0;
  const bool leader = rank == 0;

  pdl_trigger();
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < C::SF_SLOTS; ++s) {
      mbar_init(&sf_raw[s], 1);
      mbar_init(&sf_full[s], CTAS * C::SF_WARPS);
      mbar_init(&sf_empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], CTAS * C::EPI_WARPS);
    }
    mbar_init(drain, 1);
    fence_mbar_init();
    *far_flag = 0;
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
    tma_prefetch_desc(&tmB32);
    if (a.tma_scales) {
      tma_prefetch_desc(&tmSA);
      tma_prefetch_desc(&tmSB);
      tma_prefetch_desc(&tmSB32);
    }
  }
  if (warp == 1) {
    if constexpr (C::PAIR) {
      tmem_alloc_pair(tmem_holder, C::TMEM_COLS);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(tmem_holder, C::TMEM_COLS);
      tmem_relinquish();
    }
  }
  __syncwarp();
  pdl_wait();
  const FastDiv by_m((a.n + C::BM - 1) / C::BM);
  float gx = 1.0f, gw = 1.0f;  // a thread an expert, asked for ahead of the groups
  if constexpr (C::NV) {
    if (a.x_scale != nullptr) gx = __ldg(a.x_scale);
    if (a.w_scale != nullptr && threadIdx.x < static_cast<unsigned>(a.E)) gw = __ldg(a.w_scale + threadIdx.x);
  }
  load_groups<C::BN, C::UNIT, false>(groups, a.group_start, a.offsets, a.E, a.rows, static_cast<int>(by_m.d), a.status);
  if (C::NV && threadIdx.x < static_cast<unsigned>(a.E)) {
    const TensorScales by = tensor_scales(gx, gw);
    lead[threadIdx.x] = by.lead;
    if (by.shift != 1.0f) *far_flag = 1;
  }
  tc_fence_before();
  if constexpr (C::PAIR)
    cluster_sync_all();
  else
    __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = uniform(*tmem_holder);
  const bool any_far = C::NV && uniform(*far_flag) != 0;
  const int n_tiles = uniform(groups->tiles[a.E]);
  const int nk = (a.k + C::BK - 1) / C::BK;
  const int first_tile = static_cast<int>(blockIdx.x) / CTAS;
  const int grid = static_cast<int>(gridDim.x) / CTAS;
  // barriers that the leader's MMA warp waits on
  const uint32_t sf_full_leader = C::PAIR ? mapa_shared(smem_u32(sf_full), 0) : smem_u32(sf_full);
  const uint32_t acc_empty_leader = C::PAIR ? mapa_shared(smem_u32(acc_empty), 0) : smem_u32(acc_empty);

  if (warp == 0) {
    // ------------------------------------------------ TMA producer of codes
    int stage = 0;
    uint32_t phase = 0;
    int issued = 0;
    bool ok = true;
    for (int L = first_tile; L < n_tiles && ok; L += grid) {
      const QTile t = q_tile<C>(a, *groups, by_m, L);
      // few rows: 32-row boxes over those that count
      const int need = uniform(t.N) / CTAS;
      const int boxes = need > C::B_ROWS - 32 ? 0 : (need + 31) / 32;
      const uint32_t bytes = C::A_BYTES + (boxes == 0 ? C::B_BYTES : boxes * 32 * 128);
      const int row = uniform(t.n0) + need * rank;
      const int col = uniform(t.m0) + 128 * rank;
      const int e = uniform(t.e);
      for (int kb = 0; kb < nk; ++kb) {
        if (!__all_sync(0xffffffffu, mbar_wait(&empty[stage], phase ^ 1u))) {
          if (lane == 0) report(a.status, DEV_WAIT_TIMEOUT_PRODUCER);
          ok = false;
          break;
        }
        if (elect_one()) {
          unsigned char* sa = smem + static_cast<size_t>(stage) * C::STAGE_BYTES;
          if (leader) mbar_arrive_expect_tx(&full[stage], CTAS * bytes);
          auto load = [&](const CUtensorMap* map, unsigned char* dst, int c1, int c2) {
            if constexpr (C::PAIR)
              tma_load_3d_pair(map, &full[stage], dst, kb * 128, c1, c2);
            else
              tma_load_3d(map, &full[stage], dst, kb * 128, c1, c2);
          };
          load(&tmA, sa, col, e);
          if (boxes == 0) {
            load(&tmB, sa + C::A_BYTES, row, 0);
          } else {
            for (int q = 0; q < boxes; ++q) load(&tmB32, sa + C::A_BYTES + q * (32 * 128), row + 32 * q, 0);
          }
        }
        ++issued;
        if (++stage == C::STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    // every copy has landed before the CTA may end (a pair's are counted by the
    // leader; its peer waits at the cluster barrier)
    if (leader) {
      for (int s = 0; s < C::STAGES && s < issued; ++s) {
        const int last = (issued - 1 - s) / C::STAGES;
        if (!mbar_wait(&full[s], static_cast<uint32_t>(last & 1))) report(a.status, DEV_WAIT_TIMEOUT_DRAIN);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------ MMA issuer
    if (leader) {
      const uint32_t sf_lo = smem_u32(sf_base) >> 4;
      const DescLo desc0{desc_lo_sw128(smem_u32(smem), 16), desc_lo_sw128(smem_u32(smem) + C::A_BYTES, 16)};
      int stage = 0;
      uint32_t phase = 0;
      int slot = 0;
      uint32_t sf_phase = 0;
      int part = 0;  // accumulators handed to the epilogues: one a tile, or one every SUM_BLOCKS stages
      bool ok = true;
      for (int L = first_tile; L < n_tiles && ok; L += grid) {
        const uint32_t n_bits = uniform(static_cast<uint32_t>(q_tile<C>(a, *groups, by_m, L).N) >> 3 << 17);
        for (int kb = 0; kb < nk; ++kb) {
          const int sub = kb % C::SF_STAGES_PER;
          const int acc = part & 1;
          const bool first = kb == 0 || (C::PARTS && kb % C::SUM_BLOCKS == 0);
          if (first) {
            // the accumulator is free: with shared columns once the part before has let
            // go of them (its epilogue is then past the part before that)
            bool free = true;
            if constexpr (C::OVERLAP) {
              if (part > 0) free = mbar_wait(&acc_empty[0], static_cast<uint32_t>((part - 1) & 1));
            } else {
              free = mbar_wait(&acc_empty[acc], static_cast<uint32_t>(((part >> 1) & 1) ^ 1));
            }
            if (!__all_sync(0xffffffffu, free)) {
              if (lane == 0) report(a.status, DEV_WAIT_TIMEOUT_MMA);
              ok = false;
              break;
            }
          }
          if (!__all_sync(0xffffffffu,
                          (sub != 0 || mbar_wait(&sf_full[slot], sf_phase)) && mbar_wait(&full[stage], phase))) {
            if (lane == 0) report(a.status, DEV_WAIT_TIMEOUT_MMA);
            ok = false;
            break;
          }
          tc_fence_after();
          const bool slot_done = sub == C::SF_STAGES_PER - 1 || kb + 1 == nk;
          const bool part_done = kb + 1 == nk || (C::PARTS && (kb + 1) % C::SUM_BLOCKS == 0);
          if (elect_one()) {
            const uint32_t d_tmem = tmem_base + (acc ? C::ACC1 : 0u);
            const uint32_t off = static_cast<uint32_t>(stage) * (C::STAGE_BYTES >> 4);
            const uint32_t sfa =
                (sf_lo + static_cast<uint32_t>(slot) * (C::SF_BYTES >> 4) + sub * (C::WORDS * 512 >> 4)) & 0x3FFFu;
            const uint32_t sfb = sfa + (C::SF_BLOCK >> 4);
            // copies and MMAs of one thread run in the order of their issue, so the
            // columns can be written again for every stage
#pragma unroll
            for (int w = 0; w < C::WORDS; ++w) {
              scales_to_tmem<C::PAIR>(tmem_base + C::SFA_COL + w * 4, sfa + w * 32);
#pragma unroll
              for (int b = 0; b < C::BBLK; ++b)
                scales_to_tmem<C::PAIR>(tmem_base + C::SFB_COL + (w * C::BBLK + b) * 4, sfb + b * (C::SF_BLOCK >> 4) + w * 32);
            }
            const int steps = min(C::BK / C::UK, (a.k - kb * C::BK + C::UK - 1) / C::UK);
#pragma unroll
            for (int kk = 0; kk < C::BK / C::UK; ++kk) {
              if (kk < steps) {
                const int w = C::NV ? kk : kk >> 1;
                constexpr uint32_t even = micro_idesc(C::NV, C::BM, 0, 0);
                constexpr uint32_t odd = micro_idesc(C::NV, C::BM, 0, 2);
                umma_micro<C::NV, C::PAIR>(d_tmem, desc0.a + off + kk * 2, desc0.b + off + kk * 2,
                                           (C::NV || (kk & 1) == 0 ? even : odd) | n_bits, tmem_base + C::SFA_COL + w * 4,
                                           tmem_base + C::SFB_COL + w * C::BBLK * 4, (first && kk == 0) ? 0u : 1u);
              }
            }
            if constexpr (C::PAIR) {
              umma_commit_pair(&empty[stage], 0x3);
              if (slot_done) umma_commit_pair(&sf_empty[slot], 0x3);
              if (part_done) umma_commit_pair(&acc_full[acc], 0x3);
            } else {
              umma_commit(&empty[stage]);
              if (slot_done) umma_commit(&sf_empty[slot]);
              if (part_done) umma_commit(&acc_full[acc]);
            }
          }
          if (part_done) ++part;
          if (slot_done && ++slot == C::SF_SLOTS) {
            slot = 0;
            sf_phase ^= 1u;
          }
          if (++stage == C::STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (elect_one()) {
        if constexpr (C::PAIR)
          umma_commit_pair(drain, 0x1);
        else
          umma_commit(drain);
        if (!mbar_wait(drain, 0)) report(a.status, DEV_WAIT_TIMEOUT_DRAIN);
        // a pair's epilogues have released every accumulator, so that no remote arrival
        // reaches this CTA after it has ended
        if (C::PAIR && part > 0 && !mbar_wait(&acc_empty[0], static_cast<uint32_t>((part - 1) & 1)))
          report(a.status, DEV_WAIT_TIMEOUT_DRAIN);
      }
    }
  } else if (warp < 2 + C::EPI_WARPS) {
    // ------------------------------------------------ epilogue
    using OutT = typename C::OutT;
    const int q = warp & 3;
    const int csel = (warp - 2) >> 2;
    const int parts = C::PARTS ? (nk + C::SUM_BLOCKS - 1) / C::SUM_BLOCKS : 1;
    int part = 0;
    bool ok = true;
    for (int L = first_tile; L < n_tiles && ok; L += grid) {
      const QTile t = q_tile<C>(a, *groups, by_m, L);
      const float alpha = C::NV ? lead[t.e] : 1.0f;
      for (int p = 0; p < parts; ++p, ++part) {
        const int acc = part & 1;
        if (!__all_sync(0xffffffffu, mbar_wait(&acc_full[acc], static_cast<uint32_t>((part >> 1) & 1)))) {
          if (lane == 0) report(a.status, DEV_WAIT_TIMEOUT_EPILOGUE);
          ok = false;
          break;
        }
        tc_fence_after();
        const bool last = p + 1 == parts;
        const int mrow = t.m0 + 128 * rank + q * 32;  // first output column of this warp
        OutT* out = static_cast<OutT*>(a.out) + static_cast<int64_t>(t.n0) * a.n + mrow;
        const uint32_t tb = tmem_base + (acc ? C::ACC1 : 0u) + (static_cast<uint32_t>(q * 32) << 16);
        float shift = 1.0f;
        if (C::NV && any_far && last) {
          shift = tensor_scales(a.x_scale != nullptr ? __ldg(a.x_scale) : 1.0f,
                                a.w_scale != nullptr ? __ldg(a.w_scale + t.e) : 1.0f).shift;
          if (__any_sync(0xffffffffu, shift != 1.0f)) shift_chunks(tb, csel, t.N, shift);
        }
#pragma unroll 1
        for (int i = 0; i < C::CHUNKS; ++i) {
          // the two warps of a lane quarter take alternate chunks of 32 rows; the
          // accumulator columns shared with the other accumulator come first: the upper
          // end of the first accumulator, the lower end of the second
          const int j = C::OVERLAP && acc == 0 ? C::CHUNKS - 1 - i : i;
          const int c = (2 * j + csel) * 32;
          uint32_t r[32];
          if (c < t.N) {
            tmem_ld32(tb + c, r);
            tmem_ld_wait();
          }
          if (i == (C::OVERLAP ? 0 : C::CHUNKS - 1)) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
              if constexpr (C::PAIR)
                mbar_arrive_cluster_relaxed(acc_empty_leader);
              else
                mbar_arrive_relaxed(&acc_empty[C::OVERLAP ? 0 : acc]);
            }
          }
          if (c < t.N) {
            float v[32];
            OutT* at = out + static_cast<int64_t>(c) * a.n;
            int ld = a.n;
            if constexpr (C::PARTS) {
              // (opaque: the rows' addresses are not kept from part to part, in registers that there are not)
              asm volatile("" : "+l"(at), "+r"(ld));
              if (p > 0) add_stored(r, at, ld, t.left - c, a.n - mrow, shift, lane);
            }
            const float by = last ? alpha : 1.0f;
#pragma unroll
            for (int x = 0; x < 32; ++x) v[x] = __uint_as_float(r[x]) * by;
            store_chunk_turned<OutT>(v, at, ld, t.left - c, a.n - mrow, lane);
          }
        }
      }
    }
  } else {
    // ------------------------------------------------ scale warps: warp 0 of a set the
    // rows of A, then a 128-row block of B each; after the sets the TMA producer
    const int sf_warp = warp - 2 - C::EPI_WARPS;
    const bool producer = sf_warp == C::SF_SETS * C::SF_WARPS;
    const int set = sf_warp / C::SF_WARPS, who = sf_warp % C::SF_WARPS;
    const int my_tiles = first_tile < n_tiles ? (n_tiles - 1 - first_tile) / grid + 1 : 0;
    unsigned char* const block0 = sf_base + who * C::SF_BLOCK;
    const int stride = producer ? 1 : C::SF_SETS;
    int slot = producer ? 0 : set;
    uint32_t phase = 0;
    auto step = [&]() {
      slot += stride;
      if (slot >= C::SF_SLOTS) {
        slot -= C::SF_SLOTS;
        phase ^= 1u;
      }
    };
    // writes the lines of a slot's block, this lane's rows being lane + 32 i: the tensor
    // core may read them
    auto hand_over = [&](const uint32_t (&r)[4][8]) {
      uint4* block = reinterpret_cast<uint4*>(block0 + static_cast<size_t>(slot) * C::SF_BYTES);
#pragma unroll
      for (int w = 0; w < 8; ++w) block[lane + 32 * w] = make_uint4(r[0][w], r[1][w], r[2][w], r[3][w]);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        if constexpr (C::PAIR)
          mbar_arrive_cluster(sf_full_leader + static_cast<uint32_t>(slot * sizeof(uint64_t)));
        else
          mbar_arrive(&sf_full[slot]);
      }
      step();
    };
    const int slots = (nk + C::SF_STAGES_PER - 1) / C::SF_STAGES_PER;  // of a tile
    if (producer) {
      if (a.tma_scales) {
        int issued = 0;
        bool ok = true;
        for (int L = first_tile; L < n_tiles && ok; L += grid) {
          const QTile t = q_tile<C>(a, *groups, by_m, L);
          const int rows = uniform(t.N);
          const int boxes = rows > C::BN - 32 ? 0 : (rows + 31) / 32;
          const uint32_t bytes = static_cast<uint32_t>(32 * (128 + (boxes == 0 ? C::BN : 32 * boxes)));
          const int row = uniform(t.n0);
          const int col = uniform(t.m0) + 128 * rank;
          const int e = uniform(t.e);
          for (int j = 0; j < slots; ++j) {
            if (!__all_sync(0xffffffffu, mbar_wait(&sf_empty[slot], phase ^ 1u))) {
              if (lane == 0) report(a.status, DEV_WAIT_TIMEOUT_PRODUCER);
              ok = false;
              break;
            }
            if (elect_one()) {
              unsigned char* sf = sf_base + static_cast<size_t>(slot) * C::SF_BYTES;
              mbar_arrive_expect_tx(&sf_raw[slot], bytes);
              tma_load_3d(&tmSA, &sf_raw[slot], sf, j * 32, col, e);
              if (boxes == 0) {
                tma_load_3d(&tmSB, &sf_raw[slot], sf + C::SF_BLOCK, j * 32, row, 0);
              } else {
                for (int q = 0; q < boxes; ++q)
                  tma_load_3d(&tmSB32, &sf_raw[slot], sf + C::SF_BLOCK + q * 1024, j * 32, row + 32 * q, 0);
              }
            }
            ++issued;
            step();
          }
        }
        for (int s = 0; s < C::SF_SLOTS && s < issued; ++s) {
          const int last = (issued - 1 - s) / C::SF_SLOTS;
          if (!mbar_wait(&sf_raw[s], static_cast<uint32_t>(last & 1))) report(a.status, DEV_WAIT_TIMEOUT_DRAIN);
        }
      }
    } else if (a.tma_scales) {
      for (int i = set; i < my_tiles * slots; i += C::SF_SETS) {
        if (!__all_sync(0xffffffffu, mbar_wait(&sf_raw[slot], phase))) {
          if (lane == 0) report(a.status, DEV_WAIT_TIMEOUT_PRODUCER);
          break;
        }
        const uint4* raw = reinterpret_cast<const uint4*>(block0 + static_cast<size_t>(slot) * C::SF_BYTES);
        uint32_t r[4][8];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int row = lane + 32 * q;
          const int flip = (row >> 2) & 1;  // 32-byte swizzle: which 16-byte half comes first
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint4 v = raw[2 * row + (h ^ flip)];
            r[q][4 * h] = v.x;
            r[q][4 * h + 1] = v.y;
            r[q][4 * h + 2] = v.z;
            r[q][4 * h + 3] = v.w;
          }
        }
        __syncwarp();
        hand_over(r);
      }
    } else {
      // through registers
      const int row_bytes = a.k / (C::NV ? 16 : 32);
      const uint8_t* end = who == 0 ? a.ws + static_cast<int64_t>(a.E) * a.n * row_bytes : a.xs + a.rows * row_bytes;
      int lL = first_tile, lj = set;
      const uint8_t* src[4];
      bool live[4];
      auto aim = [&]() {
        if (lL >= n_tiles) return;
        const QTile t = q_tile<C>(a, *groups, by_m, lL);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = lane + 32 * i;
          if (who == 0) {
            const int m = t.m0 + 128 * rank + r;
            live[i] = m < a.n;
            src[i] = a.ws + (static_cast<int64_t>(t.e) * a.n + m) * row_bytes;
          } else {
            const int x = (who - 1) * 128 + r;
            live[i] = x < t.left;
            src[i] = a.xs + (static_cast<int64_t>(t.n0) + x) * row_bytes;
          }
        }
      };
      bool aimed = false;
      for (int i = set; i < my_tiles * slots; i += C::SF_SETS) {
        while (lj >= slots) {
          lj -= slots;
          lL += grid;
          aimed = false;
        }
        if (!aimed) aim();
        aimed = true;
        uint32_t r[4][8];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if (live[q]) {
            load_scale_words(r[q], src[q], lj * 32, row_bytes, end);
          } else {
#pragma unroll
            for (int w = 0; w < 8; ++w) r[q][w] = 0u;
          }
        }
        lj += C::SF_SETS;
        if (!__all_sync(0xffffffffu, mbar_wait(&sf_empty[slot], phase ^ 1u))) {
          if (lane == 0) report(a.status, DEV_WAIT_TIMEOUT_PRODUCER);
          break;
        }
        hand_over(r);
      }
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if constexpr (C::PAIR) cluster_sync_all();
  if (warp == 1) {
    tc_fence_after();
    if constexpr (C::PAIR)
      tmem_dealloc_pair(tmem_base, C::TMEM_COLS);
    else
      tmem_dealloc(tmem_base, C::TMEM_COLS);
  }
}

// -------------------------------------------------------------- host side

template <class C>
cudaError_t launch_q(const void* x, const void* w, const QArgs& a, cudaStream_t st) {
  static std::atomic<size_t> smem_set[kMaxDevices];
  cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(microscaled_gemm_kernel<C>), C::SMEM_BYTES, smem_set);
  if (e != cudaSuccess) return e;
  const uint64_t row_bytes = static_cast<uint64_t>(a.k) / 2;
  const uint64_t rows = static_cast<uint64_t>(a.rows), n = static_cast<uint64_t>(a.n), E = static_cast<uint64_t>(a.E);
  CUtensorMap ta, tb, tb32;
  if (!make_map_bytes(&ta, w, E, n, row_bytes, 128) || !make_map_bytes(&tb, x, 1, rows, row_bytes, C::B_ROWS) ||
      !make_map_bytes(&tb32, x, 1, rows, row_bytes, 32))
    return cudaErrorInvalidValue;
  CUtensorMap tsa = ta, tsb = tb, tsb32 = tb32;
  if (a.tma_scales) {
    const uint64_t sf_bytes = static_cast<uint64_t>(a.k) / (C::NV ? 16 : 32);
    if (!make_map_scales(&tsa, a.ws, E, n, sf_bytes, 128) || !make_map_scales(&tsb, a.xs, 1, rows, sf_bytes, C::BN) ||
        !make_map_scales(&tsb32, a.xs, 1, rows, sf_bytes, 32))
      return cudaErrorInvalidValue;
  }
  // row tiles: at most one more than full ones for every group that has rows
  const int64_t tiles = (a.rows / C::BN + (a.rows < a.E ? a.rows : a.E)) * ((a.n + C::BM - 1) / C::BM);
  const int64_t most = device_sm_count() / C::CTAS;
  const unsigned units = static_cast<unsigned>(tiles < most ? tiles : most);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  return launch_dependent(microscaled_gemm_kernel<C>, dim3(C::CTAS * units), dim3(C::THREADS), C::SMEM_BYTES, st, attr,
                          C::PAIR ? 1 : 0, ta, tb, tb32, tsa, tsb, tsb32, a);
}

template <bool NV, bool O32>
cudaError_t run_q(const void* x, const void* w, QArgs& a, cudaStream_t st) {
  a.tma_scales = a.k / (NV ? 16 : 32) % 16 == 0;
  // a stage of 256 terms takes about 1.75 times one of 64 bf16 terms
  switch (pick_row_tile(a.rows, a.E, a.n, (a.k + 255) / 256, 175)) {
    case kTilePair: return launch_q<QCfg<NV, 256, O32, true>>(x, w, a, st);
    case kTile256: return launch_q<QCfg<NV, 256, O32, false>>(x, w, a, st);
    case kTile128: return launch_q<QCfg<NV, 128, O32, false>>(x, w, a, st);
    case kTile64: return launch_q<QCfg<NV, 64, O32, false>>(x, w, a, st);
    default: return launch_q<QCfg<NV, 32, O32, false>>(x, w, a, st);
  }
}

}  // namespace

cudaError_t launch_ragged_microscaled(bool nv, int64_t rows, int E, int n, int k, bool out32, const uint8_t* xc,
                                      const uint8_t* xs, const float* xg, const int32_t* gs, const int32_t* off,
                                      const uint8_t* wc, const uint8_t* ws, const float* wg, void* y, int32_t* status,
                                      cudaStream_t st) {
  QArgs a{gs, off, xs, ws, xg, wg, rows, E, n, k, false, y, status};
  if (nv) return out32 ? run_q<true, true>(xc, wc, a, st) : run_q<true, false>(xc, wc, a, st);
  return out32 ? run_q<false, true>(xc, wc, a, st) : run_q<false, false>(xc, wc, a, st);
}

}  // namespace moe
