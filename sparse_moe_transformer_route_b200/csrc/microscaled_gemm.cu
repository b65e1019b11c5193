// The grouped product on microscaled 4-bit operands (MXFP4 or NVFP4):
//   y[r] = g_x g_w[e] * sum_k (code_x s_x)(code_w s_w)      for the rows r of expert e
// with the block-scaled form of tcgen05.mma: 64 terms an instruction, codes packed
// two to a byte in shared memory, block scales in TMEM, fp32 accumulation. The
// products of scaled elements are exact there; the two tensor scales multiply the
// finished sum.
//
// Scales. The instruction reads the scale bytes of row r (of either operand) from
// TMEM lane r % 32, column r / 32, four bytes a column: with NVFP4 the four blocks of
// one 64-term step, with MXFP4 the four blocks of two steps. One tcgen05.cp
// (32x128b.warpx4) brings 128 rows' column set from 512 bytes of shared memory whose
// 16-byte line i holds the words of rows i, i + 32, i + 64, i + 96. In global memory
// scales are plain row-major bytes, so that a group may start at any row: loader
// warps read 16 (NVFP4) or 8 (MXFP4) bytes of four rows per thread, which is one
// stage of 256 terms, and write the lines as they are: 16-byte loads and stores, no
// bank conflicts. The loads run several stages ahead in registers.
//
// Structure per CTA (persistent, one an SM): warp 0 TMA of codes, warp 1 MMA issue,
// warps 2..9 epilogue, the rest scale loaders. A 256-column accumulator pair and the
// scales do not fit TMEM's 512 columns side by side, so the two accumulators share
// 64 columns: the epilogue reads those first and then lets the next tile start.
// Every wait is bounded; a timeout is recorded in the status word.
#include <cudaTypedefs.h>

#include "ragged.cuh"

namespace moe {
namespace {

template <bool NV_, int BN_, bool O32_>
struct QCfg {
  static constexpr bool NV = NV_;
  static constexpr int BN = BN_;
  static constexpr bool O32 = O32_;
  using OutT = std::conditional_t<O32, float, __nv_bfloat16>;
  static constexpr int BM = 128;
  static constexpr int BK = 256;                 // terms a stage: one 128-byte swizzle row of codes
  static constexpr int UK = 64;                  // terms a tcgen05.mma
  static constexpr int SCALE_BYTES = NV ? 16 : 8;  // scale bytes of a row and stage
  static constexpr int WORDS = SCALE_BYTES / 4;  // TMEM column sets a stage
  static constexpr int BBLK = (BN + 127) / 128;  // 128-row blocks of B
  static constexpr int A_BYTES = BM * 128;
  static constexpr int B_BYTES = BN * 128;
  static constexpr int SFA_BYTES = WORDS * 512;
  static constexpr int SFB_BYTES = WORDS * 512 * BBLK;
  static constexpr int STAGE_BYTES = (A_BYTES + B_BYTES + SFA_BYTES + SFB_BYTES + 1023) / 1024 * 1024;
  static constexpr bool OVERLAP = BN == 256;
  static constexpr uint32_t ACC1 = OVERLAP ? 192 : BN;  // first column of the second accumulator
  static constexpr uint32_t SFA_COL = 448;
  static constexpr uint32_t SFB_COL = SFA_COL + WORDS * 4;
  static constexpr uint32_t TMEM_COLS = 512;
  static constexpr int EPI_WARPS = 8;
  static constexpr int SF_WARPS = 1 + BBLK;
  static constexpr int THREADS = 64 + 32 * (EPI_WARPS + SF_WARPS);
  static constexpr int CHUNKS = BN / 64;  // 32-column chunks of an epilogue warp
  static constexpr int MISC_BYTES = 1024 + static_cast<int>(sizeof(RaggedGroups));
  static constexpr int STAGES_FIT = (227 * 1024 - 1024 - MISC_BYTES) / STAGE_BYTES;
  static constexpr int STAGES = STAGES_FIT > 8 ? 8 : STAGES_FIT;
  static constexpr size_t SMEM_BYTES = 1024 + static_cast<size_t>(STAGES) * STAGE_BYTES + MISC_BYTES;
  static constexpr int AHEAD = 4;  // stages whose scales are in flight in registers
  static_assert(STAGES >= 3, "ring");
  static_assert(SMEM_BYTES > 114 * 1024, "one CTA an SM");
  static_assert(SFB_COL + WORDS * 4 * BBLK <= 512, "TMEM columns");
  static_assert(BN == 256 || BN == 128 || BN == 64, "tile N");
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

// Descriptor of a scale block in shared memory: no swizzle, 8-row groups of 16-byte
// lines 128 bytes apart.
__device__ __forceinline__ uint64_t scale_desc(uint32_t saddr) {
  return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (static_cast<uint64_t>(128 >> 4) << 32) | (1ull << 46);
}

__device__ __forceinline__ void scales_to_tmem(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

template <bool NV>
__device__ __forceinline__ void umma_micro(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t sfa,
                                           uint32_t sfb, uint32_t accumulate) {
  if constexpr (NV)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}\n" ::"r"(
            d),
        "l"(ad), "l"(bd), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}\n" ::"r"(
            d),
        "l"(ad), "l"(bd), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}

struct QTile {
  int e, m0, n0, valid;
};

template <class C>
__device__ __forceinline__ QTile q_tile(const QArgs& a, const RaggedGroups& g, int nN, int L) {
  QTile t;
  const int mt = L / nN;
  t.n0 = (L - mt * nN) * C::BN;
  t.e = tile_expert(g, a.E, mt);
  const int in = (mt - g.tiles[t.e]) * C::BM;
  t.m0 = g.start[t.e] + in;
  t.valid = min(C::BM, g.count[t.e] - in);
  return t;
}

// The scale words of one row for one stage: bytes [at, at + 4 WORDS) of its scale
// row, zero past the row's end. `whole`: every stage of a row is a full, aligned piece.
template <int WORDS>
__device__ __forceinline__ void load_scale_words(uint32_t (&w)[WORDS], const uint8_t* row, int at, int row_bytes,
                                                 bool whole) {
  if (whole) {
    if constexpr (WORDS == 4) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(row + at));
      w[0] = v.x;
      w[1] = v.y;
      w[2] = v.z;
      w[3] = v.w;
    } else {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(row + at));
      w[0] = v.x;
      w[1] = v.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < WORDS; ++i) {
      uint32_t v = 0;
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const int c = at + 4 * i + b;
        if (c < row_bytes) v |= static_cast<uint32_t>(__ldg(row + c)) << (8 * b);
      }
      w[i] = v;
    }
  }
}

// 32 consecutive columns of one row, this thread's, scaled and stored in pieces of 16
// bytes; `cols` (a multiple of 8) bounds them.
template <typename T>
__device__ __forceinline__ void store_row32(T* dst, const uint32_t (&r)[32], float alpha, int cols) {
  constexpr int EPS = 16 / static_cast<int>(sizeof(T));
#pragma unroll
  for (int i = 0; i < 32 / EPS; ++i) {
    uint4 w;
    if constexpr (sizeof(T) == 4) {
      w.x = __float_as_uint(__uint_as_float(r[4 * i]) * alpha);
      w.y = __float_as_uint(__uint_as_float(r[4 * i + 1]) * alpha);
      w.z = __float_as_uint(__uint_as_float(r[4 * i + 2]) * alpha);
      w.w = __float_as_uint(__uint_as_float(r[4 * i + 3]) * alpha);
    } else {
      w.x = pack_bf16x2(__uint_as_float(r[(8 * i) & 31]) * alpha, __uint_as_float(r[(8 * i + 1) & 31]) * alpha);
      w.y = pack_bf16x2(__uint_as_float(r[(8 * i + 2) & 31]) * alpha, __uint_as_float(r[(8 * i + 3) & 31]) * alpha);
      w.z = pack_bf16x2(__uint_as_float(r[(8 * i + 4) & 31]) * alpha, __uint_as_float(r[(8 * i + 5) & 31]) * alpha);
      w.w = pack_bf16x2(__uint_as_float(r[(8 * i + 6) & 31]) * alpha, __uint_as_float(r[(8 * i + 7) & 31]) * alpha);
    }
    if (i * EPS < cols) reinterpret_cast<uint4*>(dst)[i] = w;
  }
}

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1)
    microscaled_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmA32,
                            const __grid_constant__ CUtensorMap tmB, const QArgs a) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + static_cast<size_t>(C::STAGES) * C::STAGE_BYTES);
  uint64_t* empty = full + C::STAGES;
  uint64_t* acc_full = empty + C::STAGES;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* drain = acc_empty + 2;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain + 1);
  RaggedGroups* groups =
      reinterpret_cast<RaggedGroups*>(smem + static_cast<size_t>(C::STAGES) * C::STAGE_BYTES + 1024);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  pdl_trigger();
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&full[s], 1 + C::SF_WARPS);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], C::EPI_WARPS);
    }
    mbar_init(drain, 1);
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmA32);
    tma_prefetch_desc(&tmB);
  }
  if (warp == 1) {
    tmem_alloc(tmem_holder, C::TMEM_COLS);
    tmem_relinquish();
  }
  __syncwarp();
  pdl_wait();
  load_groups<C::BM>(groups, a.group_start, a.offsets, a.E, a.rows, a.status);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  const int nN = (a.n + C::BN - 1) / C::BN;
  const int n_tiles = groups->tiles[a.E] * nN;
  const int nk = (a.k + C::BK - 1) / C::BK;
  const int grid = static_cast<int>(gridDim.x);

  if (warp == 0) {
    // ------------------------------------------------ TMA producer of codes
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      int issued = 0;
      bool ok = true;
      for (int L = blockIdx.x; L < n_tiles && ok; L += grid) {
        const QTile t = q_tile<C>(a, *groups, nN, L);
        const int boxes = t.valid > 96 ? 0 : (t.valid + 31) / 32;
        const uint32_t bytes = C::B_BYTES + (boxes == 0 ? C::A_BYTES : boxes * 32 * 128);
        for (int kb = 0; kb < nk; ++kb) {
          if (!mbar_wait(&empty[stage], phase ^ 1u)) {
            report(a.status, DEV_WAIT_TIMEOUT_PRODUCER);
            ok = false;
            break;
          }
          unsigned char* sa = smem + static_cast<size_t>(stage) * C::STAGE_BYTES;
          mbar_arrive_expect_tx(&full[stage], bytes);
          if (boxes == 0) {
            tma_load_3d(&tmA, &full[stage], sa, kb * 128, t.m0, 0);
          } else {
            for (int q = 0; q < boxes; ++q)
              tma_load_3d(&tmA32, &full[stage], sa + q * (32 * 128), kb * 128, t.m0 + 32 * q, 0);
          }
          tma_load_3d(&tmB, &full[stage], sa + C::A_BYTES, kb * 128, t.n0, t.e);
          ++issued;
          if (++stage == C::STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      // every copy this thread issued has landed before the CTA may end
      for (int s = 0; s < C::STAGES && s < issued; ++s) {
        const int last = (issued - 1 - s) / C::STAGES;
        if (!mbar_wait(&full[s], static_cast<uint32_t>(last & 1))) report(a.status, DEV_WAIT_TIMEOUT_DRAIN);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------ MMA issuer
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      int tile = 0;
      bool ok = true;
      for (int L = blockIdx.x; L < n_tiles && ok; L += grid, ++tile) {
        const int acc = tile & 1;
        // the accumulator is free: with shared columns once the tile before has let
        // go of them (its epilogue is then past the tile before that)
        bool free = true;
        if constexpr (C::OVERLAP) {
          if (tile > 0) free = mbar_wait(&acc_empty[0], static_cast<uint32_t>((tile - 1) & 1));
        } else {
          free = mbar_wait(&acc_empty[acc], static_cast<uint32_t>(((tile >> 1) & 1) ^ 1));
        }
        if (!free) {
          report(a.status, DEV_WAIT_TIMEOUT_MMA);
          break;
        }
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + (acc ? C::ACC1 : 0u);
        for (int kb = 0; kb < nk; ++kb) {
          if (!mbar_wait(&full[stage], phase)) {
            report(a.status, DEV_WAIT_TIMEOUT_MMA);
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sa = smem_u32(smem + static_cast<size_t>(stage) * C::STAGE_BYTES);
          const uint32_t sb = sa + C::A_BYTES;
          const uint32_t sfa = sb + C::B_BYTES;
          const uint32_t sfb = sfa + C::SFA_BYTES;
          // copies and MMAs of one thread run in the order of their issue, so the
          // columns can be written again for every stage
#pragma unroll
          for (int w = 0; w < C::WORDS; ++w) {
            scales_to_tmem(tmem_base + C::SFA_COL + w * 4, scale_desc(sfa + w * 512));
#pragma unroll
            for (int b = 0; b < C::BBLK; ++b)
              scales_to_tmem(tmem_base + C::SFB_COL + (w * C::BBLK + b) * 4, scale_desc(sfb + (w * C::BBLK + b) * 512));
          }
          const int steps = min(C::BK / C::UK, (a.k - kb * C::BK + C::UK - 1) / C::UK);
          for (int kk = 0; kk < steps; ++kk) {
            const int w = C::NV ? kk : kk >> 1;
            const uint32_t idesc =
                C::NV || (kk & 1) == 0 ? micro_idesc(C::NV, C::BM, C::BN, 0) : micro_idesc(C::NV, C::BM, C::BN, 2);
            umma_micro<C::NV>(d_tmem, smem_desc_sw128(sa + kk * 32, 16, 1024), smem_desc_sw128(sb + kk * 32, 16, 1024),
                              idesc, tmem_base + C::SFA_COL + w * 4, tmem_base + C::SFB_COL + w * C::BBLK * 4,
                              (kb > 0 || kk > 0) ? 1u : 0u);
          }
          umma_commit(&empty[stage]);
          if (++stage == C::STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        umma_commit(&acc_full[acc]);
      }
      umma_commit(drain);
      if (!mbar_wait(drain, 0)) report(a.status, DEV_WAIT_TIMEOUT_DRAIN);
    }
  } else if (warp < 2 + C::EPI_WARPS) {
    // ------------------------------------------------ epilogue
    using OutT = typename C::OutT;
    const int q = warp & 3;
    const int csel = (warp - 2) >> 2;
    int tile = 0;
    for (int L = blockIdx.x; L < n_tiles; L += grid, ++tile) {
      const QTile t = q_tile<C>(a, *groups, nN, L);
      const int acc = tile & 1;
      float alpha = 1.0f;
      if (a.x_scale != nullptr) alpha = __ldg(a.x_scale);
      if (a.w_scale != nullptr) alpha *= __ldg(a.w_scale + t.e);
      if (!__all_sync(0xffffffffu, mbar_wait(&acc_full[acc], static_cast<uint32_t>((tile >> 1) & 1)))) {
        if (lane == 0) report(a.status, DEV_WAIT_TIMEOUT_EPILOGUE);
        break;
      }
      tc_fence_after();
      const bool row_ok = q * 32 + lane < t.valid;
      OutT* row = static_cast<OutT*>(a.out) + (static_cast<int64_t>(t.m0) + q * 32 + lane) * a.n + t.n0;
      const uint32_t tb = tmem_base + (acc ? C::ACC1 : 0u) + (static_cast<uint32_t>(q * 32) << 16);
#pragma unroll 1
      for (int i = 0; i < C::CHUNKS; ++i) {
        // the two warps of a lane quarter take alternate 32-column chunks; the
        // columns shared with the other accumulator come first: the upper end of
        // the first accumulator, the lower end of the second
        const int j = C::OVERLAP && acc == 0 ? C::CHUNKS - 1 - i : i;
        const int c = (2 * j + csel) * 32;
        uint32_t r[32];
        tmem_ld32(tb + c, r);
        tmem_ld_wait();
        if (i == (C::OVERLAP ? 0 : C::CHUNKS - 1)) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&acc_empty[C::OVERLAP ? 0 : acc]);
        }
        if (row_ok) store_row32<OutT>(row + c, r, alpha, a.n - t.n0 - c);
      }
    }
  } else {
    // ------------------------------------------------ scale loaders: warp 0 of these
    // the rows of A, the others a 128-row block of B each
    const int who = warp - 2 - C::EPI_WARPS;
    const int row_bytes = a.k / (C::NV ? 16 : 32);
    const bool whole = a.k % C::BK == 0;
    const uint32_t dst = (who == 0 ? C::A_BYTES + C::B_BYTES : C::A_BYTES + C::B_BYTES + C::SFA_BYTES + (who - 1) * 512);
    const int word_step = who == 0 ? 512 : 512 * C::BBLK;
    // the load side runs AHEAD stages before the store side
    int lL = blockIdx.x, lkb = 0;
    const uint8_t* src[4];
    bool live[4];
    auto aim = [&]() {
      if (lL >= n_tiles) return;
      const QTile t = q_tile<C>(a, *groups, nN, lL);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = lane + 32 * i;
        if (who == 0) {
          live[i] = r < t.valid;
          src[i] = a.xs + (static_cast<int64_t>(t.m0) + r) * row_bytes;
        } else {
          const int n = t.n0 + (who - 1) * 128 + r;
          live[i] = n < a.n && (C::BN >= 128 || r < C::BN);
          src[i] = a.ws + (static_cast<int64_t>(t.e) * a.n + n) * row_bytes;
        }
      }
    };
    aim();
    uint32_t buf[C::AHEAD][4][C::WORDS];
    auto fetch = [&](uint32_t (&b)[4][C::WORDS]) {
      if (lL >= n_tiles) return;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (live[i]) {
          load_scale_words<C::WORDS>(b[i], src[i], lkb * C::SCALE_BYTES, row_bytes, whole);
        } else {
#pragma unroll
          for (int w = 0; w < C::WORDS; ++w) b[i][w] = 0u;
        }
      }
      if (++lkb == nk) {
        lkb = 0;
        lL += grid;
        aim();
      }
    };
#pragma unroll
    for (int s = 0; s < C::AHEAD; ++s) fetch(buf[s]);
    const int my_tiles = blockIdx.x < n_tiles ? (n_tiles - 1 - static_cast<int>(blockIdx.x)) / grid + 1 : 0;
    const int64_t total = static_cast<int64_t>(my_tiles) * nk;
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int64_t it = 0; it < total && ok; it += C::AHEAD) {
#pragma unroll
      for (int s = 0; s < C::AHEAD; ++s) {
        if (it + s < total && ok) {
          if (!__all_sync(0xffffffffu, mbar_wait(&empty[stage], phase ^ 1u))) {
            if (lane == 0) report(a.status, DEV_WAIT_TIMEOUT_PRODUCER);
            ok = false;
          } else {
            unsigned char* line = smem + static_cast<size_t>(stage) * C::STAGE_BYTES + dst + lane * 16;
#pragma unroll
            for (int w = 0; w < C::WORDS; ++w)
              *reinterpret_cast<uint4*>(line + w * word_step) =
                  make_uint4(buf[s][0][w], buf[s][1][w], buf[s][2][w], buf[s][3][w]);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&full[stage]);
            if (++stage == C::STAGES) {
              stage = 0;
              phase ^= 1u;
            }
            fetch(buf[s]);
          }
        }
      }
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, C::TMEM_COLS);
  }
}

// -------------------------------------------------------------- host side

template <class C>
cudaError_t launch_q(const void* x, const void* w, const QArgs& a, int64_t max_tiles, cudaStream_t st) {
  static std::atomic<size_t> smem_set[kMaxDevices];
  cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(microscaled_gemm_kernel<C>), C::SMEM_BYTES, smem_set);
  if (e != cudaSuccess) return e;
  const uint64_t row_bytes = static_cast<uint64_t>(a.k) / 2;
  CUtensorMap ta, ta32, tb;
  if (!make_map_bytes(&ta, x, 1, static_cast<uint64_t>(a.rows), row_bytes, 128) ||
      !make_map_bytes(&ta32, x, 1, static_cast<uint64_t>(a.rows), row_bytes, 32) ||
      !make_map_bytes(&tb, w, static_cast<uint64_t>(a.E), static_cast<uint64_t>(a.n), row_bytes, C::BN))
    return cudaErrorInvalidValue;
  const int64_t sms = device_sm_count();
  const unsigned grid = static_cast<unsigned>(max_tiles < sms ? max_tiles : sms);
  return launch_dependent(microscaled_gemm_kernel<C>, dim3(grid), dim3(C::THREADS), C::SMEM_BYTES, st, nullptr, 0, ta,
                          ta32, tb, a);
}

template <bool NV, bool O32>
cudaError_t run_q(const void* x, const void* w, const QArgs& a, cudaStream_t st) {
  const int64_t row_tiles = a.rows / 128 + (a.rows < a.E ? a.rows : a.E);
  const int bn = pick_tile_width(row_tiles, a.n);
  const int64_t max_tiles = row_tiles * ((a.n + bn - 1) / bn);
  if (bn == 256) return launch_q<QCfg<NV, 256, O32>>(x, w, a, max_tiles, st);
  if (bn == 128) return launch_q<QCfg<NV, 128, O32>>(x, w, a, max_tiles, st);
  return launch_q<QCfg<NV, 64, O32>>(x, w, a, max_tiles, st);
}

}  // namespace

cudaError_t launch_ragged_microscaled(bool nv, int64_t rows, int E, int n, int k, bool out32, const uint8_t* xc,
                                      const uint8_t* xs, const float* xg, const int32_t* gs, const int32_t* off,
                                      const uint8_t* wc, const uint8_t* ws, const float* wg, void* y, int32_t* status,
                                      cudaStream_t st) {
  const QArgs a{gs, off, xs, ws, xg, wg, rows, E, n, k, y, status};
  if (nv) return out32 ? run_q<true, true>(xc, wc, a, st) : run_q<true, false>(xc, wc, a, st);
  return out32 ? run_q<false, true>(xc, wc, a, st) : run_q<false, false>(xc, wc, a, st);
}

}  // namespace moe
