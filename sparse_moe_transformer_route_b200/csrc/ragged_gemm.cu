// Matrix products grouped by expert with ragged sizes, and their gradients.
//
// Expert e owns count_e rows (any number) of row buffers X [rows, k], Y [rows, n]
// and a weight W_e [n, k]:
//   forward   y[r]  = W_e x[r]                        Y_e  = X_e  W_e^T
//   dgrad     dx[r] = W_e^T dy[r]                     dX_e = dY_e W_e
//   wgrad     dW_e  = sum over rows r of dy[r] x[r]^T dW_e = dY_e^T X_e
// bf16 operands, fp32 sums, bf16 or fp32 results. Groups start at any row: a tile's
// operand box simply starts at the group's row (only the innermost TMA coordinate
// has an alignment rule), reads into the next group where the group ends inside the
// tile, and the rows past the end are not stored. Widths are multiples of 8 (16-byte
// row strides); TMA fills what lies past a width with zeros, so a reduction's tail
// adds nothing. The weights are mapped in three dimensions, so that a tile that
// leaves an expert's matrix reads zeros and not the next expert's rows. In wgrad the
// reduction runs over a group's rows: the rows past its end in the last box belong
// to another group (or hold anything at all), so the MMA warp overwrites them with
// zeros in shared memory before it issues that step.
//
// Structure per CTA (persistent, one an SM): warp 0 issues TMA loads into a ring of
// stages, warp 1 issues tcgen05.mma (128 x BN x 16), warps 2..9 read the fp32
// accumulator from TMEM and store; two accumulators, so that a tile's epilogue runs
// under the next tile's MMAs. Every wait is bounded; a timeout is recorded in the
// status word and the CTA unwinds.
#include <cudaTypedefs.h>

#include "ragged.cuh"

namespace moe {
namespace {

enum class Op { Fwd, Dgrad, Wgrad };

template <Op OP_, int BN_, bool O32_>
struct RCfg {
  static constexpr Op OP = OP_;
  static constexpr bool A_MN = OP == Op::Wgrad;                    // A read as [reduction][row of the tile]
  static constexpr bool B_MN = OP != Op::Fwd;
  static constexpr int BN = BN_;
  static constexpr bool O32 = O32_;
  using OutT = std::conditional_t<O32, float, __nv_bfloat16>;
  static constexpr int BM = 128;
  static constexpr int BK = 64;  // one 128-byte swizzle row when K-major
  static constexpr int UK = 16;
  static constexpr int A_BYTES = BM * BK * 2;
  static constexpr int B_BYTES = BN * BK * 2;
  static constexpr int CHUNK_BYTES = BK * 128;  // MN-major: 64 reduction rows of one 64-column piece
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int A_STEP = A_MN ? UK * 128 : UK * 2;  // bytes between the operands of two steps
  static constexpr int B_STEP = B_MN ? UK * 128 : UK * 2;
  // The tensor core's fp32 sum over a long reduction loses about half an ulp a step
  // towards zero. Where the result is fp32, or the reduction may be as long as the
  // buffer (wgrad), the accumulator is handed over every SUM_BLOCKS stages (512
  // terms) and the parts are added in fp32 registers, rounded to nearest.
  static constexpr bool PARTS = O32 || OP == Op::Wgrad;
  static constexpr int SUM_BLOCKS = 8;
  static constexpr uint32_t IDESC = make_idesc(false, A_MN, B_MN, BM, BN);
  static constexpr uint32_t TMEM_COLS = 2 * BN;
  static constexpr int EPI_WARPS = 8;
  static constexpr int THREADS = 64 + 32 * EPI_WARPS;
  static constexpr int WCOLS = BN / 2;  // columns of an epilogue warp
  static constexpr int STG_PITCH = 32 * 2 + 16;  // fp32 leaves in two passes
  static constexpr int STG_WARP_BYTES = 32 * STG_PITCH;
  static constexpr int STG_BYTES = EPI_WARPS * STG_WARP_BYTES;
  static constexpr int MISC_BYTES = 1024 + static_cast<int>(sizeof(RaggedGroups)) + kMaxExperts * 4;
  static constexpr int STAGES_FIT = (227 * 1024 - 1024 - MISC_BYTES - STG_BYTES) / STAGE_BYTES;
  static constexpr int STAGES = STAGES_FIT > 12 ? 12 : STAGES_FIT;
  static constexpr size_t SMEM_BYTES = 1024 + static_cast<size_t>(STAGES) * STAGE_BYTES + STG_BYTES + MISC_BYTES;
  static_assert(STAGES >= 3 && (2 * STAGES + 6) * 8 <= 1024, "ring");
  static_assert(BN == 256 || BN == 128 || BN == 64, "tile N");
  // no two CTAs of such kernels share an SM: one that is launched early (as a dependent)
  // never holds the TMEM that a CTA of the kernel before it is still to allocate
  static_assert(SMEM_BYTES > 114 * 1024, "one CTA an SM");
};

struct RArgs {
  const int32_t* group_start;
  const int32_t* offsets;
  int64_t rows;
  int E, n, k;
  void* out;
  int32_t* status;
};

struct RTile {
  int e;
  int m0;     // first row of the tile: of the buffer (fwd, dgrad) or of dW_e
  int n0;     // first output column
  int valid;  // rows of the tile that exist
  int red;    // length of the reduction
  int row0;   // wgrad: first row of the group
};

template <class C>
struct Schedule {
  int n_tiles, nN, out_cols;
  __device__ Schedule(const RArgs& a, const RaggedGroups& g) {
    out_cols = C::OP == Op::Fwd ? a.n : a.k;
    nN = (out_cols + C::BN - 1) / C::BN;
    n_tiles = (C::OP == Op::Wgrad ? a.E * ((a.n + C::BM - 1) / C::BM) : g.tiles[a.E]) * nN;
  }
  // Tile of this CTA's turn i, or -1. wgrad's tiles cost their group's rows and come
  // largest group first: every other turn runs backwards over the CTAs, which evens
  // out what a turn's first and last CTA get.
  __device__ int at(int i) const {
    const int G = static_cast<int>(gridDim.x), c = static_cast<int>(blockIdx.x);
    const int64_t L = static_cast<int64_t>(i) * G + ((C::OP == Op::Wgrad && (i & 1)) ? G - 1 - c : c);
    return L < n_tiles ? static_cast<int>(L) : -1;
  }
  // turns of any CTA: at() may be -1 in the last one only
  __device__ int turns() const { return (n_tiles + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x); }
  __device__ RTile tile(const RArgs& a, const RaggedGroups& g, const int32_t* by_size, int L) const {
    RTile t;
    const int mt = L / nN;
    t.n0 = (L - mt * nN) * C::BN;
    if constexpr (C::OP == Op::Wgrad) {
      const int mT = (a.n + C::BM - 1) / C::BM;
      t.e = by_size[mt / mT];
      t.m0 = (mt % mT) * C::BM;
      t.valid = min(C::BM, a.n - t.m0);
      t.red = g.count[t.e];
      t.row0 = g.start[t.e];
    } else {
      t.e = tile_expert(g, a.E, mt);
      const int in = (mt - g.tiles[t.e]) * C::BM;
      t.m0 = g.start[t.e] + in;
      t.valid = min(C::BM, g.count[t.e] - in);
      t.red = C::OP == Op::Fwd ? a.k : a.n;
      t.row0 = 0;
    }
    return t;
  }
};

// by_size: experts by falling row count (equal counts in order of e). All threads; the
// caller's block barrier follows.
__device__ __forceinline__ void rank_by_size(const RaggedGroups* g, int32_t* by_size, int E) {
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    int rank = 0;
    const int mine = g->count[e];
    for (int o = 0; o < E; ++o) rank += g->count[o] > mine || (g->count[o] == mine && o < e);
    by_size[rank] = e;
  }
}

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1)
    ragged_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmA32,
                       const __grid_constant__ CUtensorMap tmB, const RArgs a) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  unsigned char* stg_base = smem + static_cast<size_t>(C::STAGES) * C::STAGE_BYTES;
  uint64_t* full = reinterpret_cast<uint64_t*>(stg_base + C::STG_BYTES);
  uint64_t* empty = full + C::STAGES;
  uint64_t* acc_full = empty + C::STAGES;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* drain = acc_empty + 2;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain + 1);
  RaggedGroups* groups = reinterpret_cast<RaggedGroups*>(stg_base + C::STG_BYTES + 1024);
  int32_t* by_size = reinterpret_cast<int32_t*>(groups + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  pdl_trigger();
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&full[s], 1);
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
    if constexpr (!C::A_MN) tma_prefetch_desc(&tmA32);
    tma_prefetch_desc(&tmB);
  }
  if (warp == 1) {
    tmem_alloc(tmem_holder, C::TMEM_COLS);
    tmem_relinquish();
  }
  __syncwarp();
  pdl_wait();
  load_groups<C::BM>(groups, a.group_start, a.offsets, a.E, a.rows, a.status);
  if constexpr (C::OP == Op::Wgrad) rank_by_size(groups, by_size, a.E);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = uniform(*tmem_holder);
  const Schedule<C> sched(a, *groups);
  const int turns = sched.turns();

  if (warp == 0) {
    // ------------------------------------------------ TMA producer
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      int issued = 0;
      bool ok = true;
      for (int i = 0; i < turns && ok; ++i) {
        const int L = sched.at(i);
        if (L < 0) continue;
        const RTile t = sched.tile(a, *groups, by_size, L);
        const int nk = (t.red + C::BK - 1) / C::BK;
        // K-major A: a 128-row box, or 32-row boxes over the rows that exist when
        // these are few (the accumulator rows of the others are never stored)
        const int boxes = t.valid > 96 ? 0 : (t.valid + 31) / 32;
        const uint32_t bytes =
            C::B_BYTES + (C::A_MN || boxes == 0 ? C::A_BYTES : static_cast<uint32_t>(boxes) * 32 * 128);
        for (int kb = 0; kb < nk; ++kb) {
          if (!mbar_wait(&empty[stage], phase ^ 1u)) {
            report(a.status, DEV_WAIT_TIMEOUT_PRODUCER);
            ok = false;
            break;
          }
          unsigned char* sa = smem + static_cast<size_t>(stage) * C::STAGE_BYTES;
          unsigned char* sb = sa + C::A_BYTES;
          mbar_arrive_expect_tx(&full[stage], bytes);
          const int k0 = kb * C::BK;
          if constexpr (C::A_MN) {
#pragma unroll
            for (int ch = 0; ch < C::BM / 64; ++ch)
              tma_load_2d(&tmA, &full[stage], sa + ch * C::CHUNK_BYTES, t.m0 + ch * 64, t.row0 + k0);
          } else if (boxes == 0) {
            tma_load_2d(&tmA, &full[stage], sa, k0, t.m0);
          } else {
            for (int q = 0; q < boxes; ++q)
              tma_load_2d(&tmA32, &full[stage], sa + q * (32 * 128), k0, t.m0 + 32 * q);
          }
          if constexpr (C::OP == Op::Fwd) {
            tma_load_3d(&tmB, &full[stage], sb, k0, t.n0, t.e);
          } else if constexpr (C::OP == Op::Dgrad) {
#pragma unroll
            for (int ch = 0; ch < C::BN / 64; ++ch)
              tma_load_3d(&tmB, &full[stage], sb + ch * C::CHUNK_BYTES, t.n0 + ch * 64, k0, t.e);
          } else {
#pragma unroll
            for (int ch = 0; ch < C::BN / 64; ++ch)
              tma_load_2d(&tmB, &full[stage], sb + ch * C::CHUNK_BYTES, t.n0 + ch * 64, t.row0 + k0);
          }
          ++issued;
          if (++stage == C::STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      // every copy this thread issued has landed before the CTA may end
      for (int s = 0; s < C::STAGES && s < issued; ++s) {
        const int last = (issued - 1 - s) / C::STAGES;  // uses of stage s, less one
        if (!mbar_wait(&full[s], static_cast<uint32_t>(last & 1))) report(a.status, DEV_WAIT_TIMEOUT_DRAIN);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------ MMA issuer (the whole warp;
    // it also clears the rows past a group's end)
    const uint32_t smem_a = smem_u32(smem);
    const DescLo desc0{desc_lo_sw128(smem_a, C::A_MN ? C::CHUNK_BYTES : 16),
                       desc_lo_sw128(smem_a + C::A_BYTES, C::B_MN ? C::CHUNK_BYTES : 16)};
    int stage = 0;
    uint32_t phase = 0;
    int acc = 0;
    uint32_t acc_phase = 0;
    bool ok = true;
    for (int i = 0; i < turns && ok; ++i) {
      const int L = sched.at(i);
      if (L < 0) continue;
      const RTile t = sched.tile(a, *groups, by_size, L);
      const int nk = uniform((t.red + C::BK - 1) / C::BK);
      for (int kb = 0; kb < nk; ++kb) {
        const bool first = kb == 0 || (C::PARTS && kb % C::SUM_BLOCKS == 0);
        if (first && !__all_sync(0xffffffffu, mbar_wait(&acc_empty[acc], acc_phase ^ 1u))) ok = false;
        if (ok && !__all_sync(0xffffffffu, mbar_wait(&full[stage], phase))) ok = false;
        if (!ok) {
          if (lane == 0) report(a.status, DEV_WAIT_TIMEOUT_MMA);
          break;
        }
        unsigned char* stage_ptr = smem + static_cast<size_t>(stage) * C::STAGE_BYTES;
        const int terms = min(C::BK, t.red - kb * C::BK);
        const int steps = (terms + C::UK - 1) / C::UK;
        if constexpr (C::OP == Op::Wgrad) {
          const int pad = steps * C::UK - terms;
          if (pad > 0) {  // rows [terms, terms + pad) of every 64-column piece: 128 bytes each
            constexpr int PIECES = (C::BM + C::BN) / 64;
            for (int j = lane; j < PIECES * pad * 8; j += 32) {
              const int piece = j / (pad * 8), w = j - piece * (pad * 8);
              *reinterpret_cast<uint4*>(stage_ptr + piece * C::CHUNK_BYTES + terms * 128 + w * 16) =
                  make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();
            __syncwarp();
          }
        }
        tc_fence_after();
        if (elect_one()) {
          const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * C::BN);
          const uint32_t off = static_cast<uint32_t>(stage) * (C::STAGE_BYTES >> 4);
          umma_stage<false, C::A_STEP, C::B_STEP>(d_tmem, DescLo{desc0.a + off, desc0.b + off}, C::IDESC,
                                                      first, steps);
          umma_commit(&empty[stage]);
        }
        if (++stage == C::STAGES) {
          stage = 0;
          phase ^= 1u;
        }
        if (kb + 1 == nk || (C::PARTS && (kb + 1) % C::SUM_BLOCKS == 0)) {
          if (elect_one()) umma_commit(&acc_full[acc]);
          if (++acc == 2) {
            acc = 0;
            acc_phase ^= 1u;
          }
        }
        __syncwarp();
      }
    }
    if (elect_one()) {
      umma_commit(drain);
      if (!mbar_wait(drain, 0)) report(a.status, DEV_WAIT_TIMEOUT_DRAIN);
    }
  } else {
    // ------------------------------------------------ epilogue
    using OutT = typename C::OutT;
    const int q = warp & 3;               // TMEM lane quarter of this warp
    const int cw = ((warp - 2) >> 2) * C::WCOLS;
    unsigned char* stg = stg_base + (warp - 2) * C::STG_WARP_BYTES;
    int acc = 0;
    uint32_t acc_phase = 0;
    bool ok = true;
    for (int i = 0; i < turns && ok; ++i) {
      const int L = sched.at(i);
      if (L < 0) continue;
      const RTile t = sched.tile(a, *groups, by_size, L);
      const int nk = (t.red + C::BK - 1) / C::BK;
      const int rows = min(32, t.valid - q * 32);
      const int64_t row = (C::OP == Op::Wgrad ? static_cast<int64_t>(t.e) * a.n : 0) + t.m0 + q * 32;
      OutT* out = static_cast<OutT*>(a.out) + row * sched.out_cols + t.n0 + cw;
      const int cols = sched.out_cols - t.n0 - cw;  // may be past the width (<= 0)
      const uint32_t lane_base = static_cast<uint32_t>(q * 32) << 16;
      if constexpr (C::PARTS) {
        float sum[C::WCOLS];
#pragma unroll
        for (int c = 0; c < C::WCOLS; ++c) sum[c] = 0.f;
        const int parts = (nk + C::SUM_BLOCKS - 1) / C::SUM_BLOCKS;  // 0: an expert without rows
        for (int p = 0; p < parts; ++p) {
          if (!__all_sync(0xffffffffu, mbar_wait(&acc_full[acc], acc_phase))) {
            if (lane == 0) report(a.status, DEV_WAIT_TIMEOUT_EPILOGUE);
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t tb = tmem_base + static_cast<uint32_t>(acc * C::BN + cw) + lane_base;
#pragma unroll
          for (int c = 0; c < C::WCOLS; c += 16) {
            uint32_t r[16];
            tmem_ld16(tb + c, r);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 16; ++j) sum[c + j] += __uint_as_float(r[j]);
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&acc_empty[acc]);
          if (++acc == 2) {
            acc = 0;
            acc_phase ^= 1u;
          }
        }
        if (!ok) break;
#pragma unroll
        for (int c = 0; c < C::WCOLS; c += 32) {
          float v[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = sum[c + j];
          store_chunk_masked<OutT, C::STG_PITCH>(stg, v, out + c, sched.out_cols, rows, cols - c, lane);
        }
      } else {
        if (!__all_sync(0xffffffffu, mbar_wait(&acc_full[acc], acc_phase))) {
          if (lane == 0) report(a.status, DEV_WAIT_TIMEOUT_EPILOGUE);
          break;
        }
        tc_fence_after();
        const uint32_t tb = tmem_base + static_cast<uint32_t>(acc * C::BN + cw) + lane_base;
#pragma unroll 1
        for (int c = 0; c < C::WCOLS; c += 32) {
          uint32_t r[32];
          tmem_ld32(tb + c, r);
          tmem_ld_wait();
          float v[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]);
          store_chunk_masked<OutT, C::STG_PITCH>(stg, v, out + c, sched.out_cols, rows, cols - c, lane);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&acc_empty[acc]);
        if (++acc == 2) {
          acc = 0;
          acc_phase ^= 1u;
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

// -------------------------------------------------------------- pairs of CTAs
//
// The same products on two CTAs of a cluster (the SMs of one TPC): a tile is 256 x 256,
// each CTA loads its 128 rows of A and half of B's 256 columns and holds its 128
// accumulator rows, and the leader (rank 0) issues cta_group::2 MMAs that read both
// shared memories. Per SM a 64-term stage is then 32 KB for the MMA work that takes
// 48 KB with one CTA a tile; one CTA a tile is bound by what shared memory takes in and
// gives out (192 bytes a clock at the tensor cores' full rate).
// A row tile of which at most 128 rows exist is a tail tile: an M = 128 MMA, 64 rows a
// CTA. There TMEM lanes 0..63 hold output columns 0..127 of the CTA's 64 rows and lanes
// 64..127 columns 128..255, both at TMEM columns 0..127.
// wgrad's rows past a group's end: each CTA clears its own shared memory. The peer's
// last, ragged stage arrives on a barrier of its own, its second warp clears the rows
// and only then arrives on the leader's barrier, which counts one arrival a CTA.
template <Op OP_, bool O32_>
struct PCfg {
  static constexpr Op OP = OP_;
  static constexpr bool A_MN = OP == Op::Wgrad;
  static constexpr bool B_MN = OP != Op::Fwd;
  static constexpr bool O32 = O32_;
  using OutT = std::conditional_t<O32, float, __nv_bfloat16>;
  static constexpr int BM = 256, BN = 256, BK = 64, UK = 16;
  static constexpr int CHUNK_BYTES = BK * 128;
  static constexpr int A_BYTES = 2 * CHUNK_BYTES;  // this CTA's 128 rows; half of them in a tail tile
  static constexpr int B_BYTES = 2 * CHUNK_BYTES;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int A_STEP = A_MN ? UK * 128 : UK * 2;  // bytes between the operands of two steps
  static constexpr int B_STEP = B_MN ? UK * 128 : UK * 2;
  static constexpr bool PARTS = O32 || OP == Op::Wgrad;
  static constexpr int SUM_BLOCKS = 8;
  static constexpr uint32_t IDESC = make_idesc(false, A_MN, B_MN, 256, BN);
  static constexpr uint32_t IDESC_TAIL = make_idesc(false, A_MN, B_MN, 128, BN);
  static constexpr uint32_t TMEM_COLS = 512;
  static constexpr int EPI_WARPS = 8;
  static constexpr int THREADS = 64 + 32 * EPI_WARPS;
  static constexpr int WCOLS = 128;
  static constexpr int STG_PITCH = 32 * 2 + 16;
  static constexpr int STG_WARP_BYTES = 32 * STG_PITCH;
  static constexpr int STG_BYTES = EPI_WARPS * STG_WARP_BYTES;
  static constexpr int MISC_BYTES = 1024 + static_cast<int>(sizeof(RaggedGroups)) + kMaxExperts * 4;
  static constexpr int STAGES = (227 * 1024 - 1024 - MISC_BYTES - STG_BYTES) / STAGE_BYTES;
  static constexpr size_t SMEM_BYTES = 1024 + static_cast<size_t>(STAGES) * STAGE_BYTES + STG_BYTES + MISC_BYTES;
  static_assert(STAGES >= 4 && (3 * STAGES + 7) * 8 <= 1024, "ring");
  static_assert(SMEM_BYTES > 114 * 1024, "one CTA an SM (see RCfg)");
};

struct PairTile {
  int e, m0, n0, red, row0;
  int tail;   // 1: at most 128 rows
  int share;  // rows a CTA: 128, or 64 in a tail tile
  int left;   // rows of the tile that exist (up to 256)
};

template <class C>
struct PairSchedule {
  int n_tiles, nN, out_cols, c, G;
  __device__ PairSchedule(const RArgs& a, const RaggedGroups& g) {
    c = static_cast<int>(blockIdx.x >> 1);
    G = static_cast<int>(gridDim.x >> 1);
    out_cols = C::OP == Op::Fwd ? a.n : a.k;
    nN = (out_cols + C::BN - 1) / C::BN;
    n_tiles = (C::OP == Op::Wgrad ? a.E * ((a.n + C::BM - 1) / C::BM) : g.tiles[a.E]) * nN;
  }
  __device__ int at(int i) const {  // as in Schedule
    const int64_t L = static_cast<int64_t>(i) * G + ((C::OP == Op::Wgrad && (i & 1)) ? G - 1 - c : c);
    return L < n_tiles ? static_cast<int>(L) : -1;
  }
  __device__ int turns() const { return (n_tiles + G - 1) / G; }
  __device__ PairTile tile(const RArgs& a, const RaggedGroups& g, const int32_t* by_size, int L) const {
    PairTile t;
    const int mt = L / nN;
    t.n0 = (L - mt * nN) * C::BN;
    if constexpr (C::OP == Op::Wgrad) {
      const int mT = (a.n + C::BM - 1) / C::BM;
      t.e = by_size[mt / mT];
      t.m0 = (mt % mT) * C::BM;
      t.left = min(C::BM, a.n - t.m0);
      t.red = g.count[t.e];
      t.row0 = g.start[t.e];
    } else {
      t.e = tile_expert(g, a.E, mt);
      const int in = (mt - g.tiles[t.e]) * C::BM;
      t.m0 = g.start[t.e] + in;
      t.left = min(C::BM, g.count[t.e] - in);
      t.red = C::OP == Op::Fwd ? a.k : a.n;
      t.row0 = 0;
    }
    t.tail = t.left <= 128 ? 1 : 0;
    t.share = t.tail ? 64 : 128;
    return t;
  }
};

// Zeroes reduction rows [from, from + count) of every 64-column piece of a stage: `a_pieces`
// of A and both of B. One warp.
template <class C>
__device__ __forceinline__ void clear_stage_rows(unsigned char* stage, int a_pieces, int from, int count, int lane) {
  const int per = count * 8;
  for (int j = lane; j < (a_pieces + 2) * per; j += 32) {
    const int piece = j / per, w = j - piece * per;
    unsigned char* base =
        stage + (piece < a_pieces ? piece * C::CHUNK_BYTES : C::A_BYTES + (piece - a_pieces) * C::CHUNK_BYTES);
    *reinterpret_cast<uint4*>(base + from * 128 + w * 16) = make_uint4(0u, 0u, 0u, 0u);
  }
  fence_proxy_async_smem();
  __syncwarp();
}

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1)
    ragged_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmA64,
                       const __grid_constant__ CUtensorMap tmB, const RArgs a) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  unsigned char* stg_base = smem + static_cast<size_t>(C::STAGES) * C::STAGE_BYTES;
  uint64_t* full = reinterpret_cast<uint64_t*>(stg_base + C::STG_BYTES);
  uint64_t* empty = full + C::STAGES;
  uint64_t* acc_full = empty + C::STAGES;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* drain = acc_empty + 2;
  uint64_t* ragged_full = drain + 1;  // per stage: the peer's copies of a group's last, ragged stage (wgrad)
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(ragged_full + C::STAGES);
  RaggedGroups* groups = reinterpret_cast<RaggedGroups*>(stg_base + C::STG_BYTES + 1024);
  int32_t* by_size = reinterpret_cast<int32_t*>(groups + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const bool leader = rank == 0;

  pdl_trigger();
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&full[s], C::OP == Op::Wgrad ? 2 : 1);  // (the leader's copies are the ones used)
      mbar_init(&empty[s], 1);
      mbar_init(&ragged_full[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 2 * C::EPI_WARPS);
    }
    mbar_init(drain, 1);
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmA);
    if constexpr (!C::A_MN) tma_prefetch_desc(&tmA64);
    tma_prefetch_desc(&tmB);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_holder, C::TMEM_COLS);
    tmem_relinquish_pair();
  }
  __syncwarp();
  pdl_wait();
  load_groups<C::BM>(groups, a.group_start, a.offsets, a.E, a.rows, a.status);
  if constexpr (C::OP == Op::Wgrad) rank_by_size(groups, by_size, a.E);
  tc_fence_before();
  cluster_sync_all();  // both CTAs' barriers are initialised before the other's copies or commits reach them
  tc_fence_after();
  const uint32_t tmem_base = uniform(*tmem_holder);
  const PairSchedule<C> sched(a, *groups);
  const int turns = sched.turns();

  if (warp == 0) {
    // ------------------------------------------------ TMA producer (both CTAs)
    if (lane == 0) {
      const uint32_t full_leader = mapa_shared(smem_u32(full), 0);
      int stage = 0;
      uint32_t phase = 0;
      int issued = 0;
      bool ok = true;
      for (int i = 0; i < turns && ok; ++i) {
        const int L = sched.at(i);
        if (L < 0) continue;
        const PairTile t = sched.tile(a, *groups, by_size, L);
        const int nk = (t.red + C::BK - 1) / C::BK;
        const int am = t.m0 + t.share * rank;
        const int bn = t.n0 + 128 * rank;
        const uint32_t bytes = (t.tail ? C::A_BYTES / 2 : C::A_BYTES) + C::B_BYTES;
        for (int kb = 0; kb < nk; ++kb) {
          if (!mbar_wait(&empty[stage], phase ^ 1u)) {
            report(a.status, DEV_WAIT_TIMEOUT_PRODUCER);
            ok = false;
            break;
          }
          unsigned char* sa = smem + static_cast<size_t>(stage) * C::STAGE_BYTES;
          unsigned char* sb = sa + C::A_BYTES;
          const int k0 = kb * C::BK;
          const bool ragged = C::OP == Op::Wgrad && kb + 1 == nk && t.red % C::UK != 0;
          if (leader) {
            mbar_arrive_expect_tx(&full[stage], ragged ? bytes : 2 * bytes);
          } else if constexpr (C::OP == Op::Wgrad) {
            if (ragged)
              mbar_arrive_expect_tx(&ragged_full[stage], bytes);
            else
              mbar_arrive_cluster(full_leader + static_cast<uint32_t>(stage * sizeof(uint64_t)));
          }
          if constexpr (C::OP == Op::Wgrad) {
            auto load = [&](const CUtensorMap* map, unsigned char* dst, int col) {
              if (ragged)
                tma_load_2d(map, leader ? &full[stage] : &ragged_full[stage], dst, col, t.row0 + k0);
              else
                tma_load_2d_pair(map, &full[stage], dst, col, t.row0 + k0);
            };
            load(&tmA, sa, am);
            if (!t.tail) load(&tmA, sa + C::CHUNK_BYTES, am + 64);
            load(&tmB, sb, bn);
            load(&tmB, sb + C::CHUNK_BYTES, bn + 64);
          } else {
            tma_load_2d_pair(t.tail ? &tmA64 : &tmA, &full[stage], sa, k0, am);
            if constexpr (C::OP == Op::Fwd) {
              tma_load_3d_pair(&tmB, &full[stage], sb, k0, bn, t.e);
            } else {
              tma_load_3d_pair(&tmB, &full[stage], sb, bn, k0, t.e);
              tma_load_3d_pair(&tmB, &full[stage], sb + C::CHUNK_BYTES, bn + 64, k0, t.e);
            }
          }
          ++issued;
          if (++stage == C::STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      // every copy of the pair has landed before the CTAs may end (the leader's
      // barriers count both CTAs' bytes; the peer waits at the cluster barrier)
      if (leader) {
        for (int s = 0; s < C::STAGES && s < issued; ++s) {
          const int last = (issued - 1 - s) / C::STAGES;
          if (!mbar_wait(&full[s], static_cast<uint32_t>(last & 1))) report(a.status, DEV_WAIT_TIMEOUT_DRAIN);
        }
      }
    }
  } else if (warp == 1) {
    if (leader) {
      // ---------------------------------------------- MMA issuer
      const uint32_t smem_a = smem_u32(smem);
      const DescLo desc0{desc_lo_sw128(smem_a, C::A_MN ? C::CHUNK_BYTES : 16),
                         desc_lo_sw128(smem_a + C::A_BYTES, C::B_MN ? C::CHUNK_BYTES : 16)};
      int stage = 0;
      uint32_t phase = 0;
      int acc = 0;
      uint32_t acc_phase = 0;
      int handed = 0;  // accumulators handed to the epilogues
      bool ok = true;
      for (int i = 0; i < turns && ok; ++i) {
        const int L = sched.at(i);
        if (L < 0) continue;
        const PairTile t = sched.tile(a, *groups, by_size, L);
        const int nk = uniform((t.red + C::BK - 1) / C::BK);
        const uint32_t idesc = uniform(t.tail ? C::IDESC_TAIL : C::IDESC);
        for (int kb = 0; kb < nk; ++kb) {
          const bool first = kb == 0 || (C::PARTS && kb % C::SUM_BLOCKS == 0);
          if (first && !__all_sync(0xffffffffu, mbar_wait(&acc_empty[acc], acc_phase ^ 1u))) ok = false;
          if (ok && !__all_sync(0xffffffffu, C::OP == Op::Wgrad ? mbar_wait_cluster(&full[stage], phase)
                                                                : mbar_wait(&full[stage], phase)))
            ok = false;
          if (!ok) {
            if (lane == 0) report(a.status, DEV_WAIT_TIMEOUT_MMA);
            break;
          }
          unsigned char* stage_ptr = smem + static_cast<size_t>(stage) * C::STAGE_BYTES;
          const int terms = min(C::BK, t.red - kb * C::BK);
          const int steps = (terms + C::UK - 1) / C::UK;
          if constexpr (C::OP == Op::Wgrad) {
            if (terms % C::UK != 0)
              clear_stage_rows<C>(stage_ptr, t.tail ? 1 : 2, terms, steps * C::UK - terms, lane);
          }
          tc_fence_after();
          if (elect_one()) {
            const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * C::BN);
            const uint32_t off = static_cast<uint32_t>(stage) * (C::STAGE_BYTES >> 4);
            umma_stage<true, C::A_STEP, C::B_STEP>(d_tmem, DescLo{desc0.a + off, desc0.b + off}, idesc,
                                                        first, steps);
            umma_commit_pair(&empty[stage], 0x3);
          }
          if (++stage == C::STAGES) {
            stage = 0;
            phase ^= 1u;
          }
          if (kb + 1 == nk || (C::PARTS && (kb + 1) % C::SUM_BLOCKS == 0)) {
            if (elect_one()) umma_commit_pair(&acc_full[acc], 0x3);
            ++handed;
            if (++acc == 2) {
              acc = 0;
              acc_phase ^= 1u;
            }
          }
          __syncwarp();
        }
      }
      if (elect_one()) {
        umma_commit_pair(drain, 0x1);
        if (!mbar_wait(drain, 0)) report(a.status, DEV_WAIT_TIMEOUT_DRAIN);
        // both epilogues have released every accumulator, so that no remote arrival
        // reaches this CTA after it has ended
        for (int b = 0; b < 2; ++b) {
          const int uses = handed > b ? (handed - 1 - b) / 2 + 1 : 0;
          if (uses > 0 && !mbar_wait(&acc_empty[b], static_cast<uint32_t>((uses - 1) & 1)))
            report(a.status, DEV_WAIT_TIMEOUT_DRAIN);
        }
      }
    } else if constexpr (C::OP == Op::Wgrad) {
      // ---------------------------------------------- the peer's ragged stages
      const uint32_t full_leader = mapa_shared(smem_u32(full), 0);
      int stage = 0;        // of the tile's first block
      uint32_t parity = 0;  // bit s: parity of ragged_full[s]'s next phase
      for (int i = 0; i < turns; ++i) {
        const int L = sched.at(i);
        if (L < 0) continue;
        const PairTile t = sched.tile(a, *groups, by_size, L);
        const int nk = (t.red + C::BK - 1) / C::BK;
        if (t.red % C::UK != 0) {
          const int last = (stage + nk - 1) % C::STAGES;
          // the stage is loaded after the whole group before it: one bounded wait for
          // every 2^18 rows, each a small part of a second's work
          bool in = false;
          for (int w = 0; w <= nk / 4096 && !in; ++w)
            in = __all_sync(0xffffffffu, mbar_wait(&ragged_full[last], (parity >> last) & 1u));
          if (!in) {
            if (lane == 0) report(a.status, DEV_WAIT_TIMEOUT_MMA);
            break;
          }
          parity ^= 1u << last;
          const int terms = t.red - (nk - 1) * C::BK;
          const int steps = (terms + C::UK - 1) / C::UK;
          clear_stage_rows<C>(smem + static_cast<size_t>(last) * C::STAGE_BYTES, t.tail ? 1 : 2, terms,
                              steps * C::UK - terms, lane);
          if (lane == 0) mbar_arrive_release_cluster(full_leader + static_cast<uint32_t>(last * sizeof(uint64_t)));
        }
        stage = (stage + nk) % C::STAGES;
      }
    }
  } else {
    // ------------------------------------------------ epilogue (both CTAs)
    using OutT = typename C::OutT;
    const int q = warp & 3;
    const int csel = (warp - 2) >> 2;
    const uint32_t acc_empty_leader = mapa_shared(smem_u32(&acc_empty[0]), 0);
    unsigned char* stg = stg_base + (warp - 2) * C::STG_WARP_BYTES;
    int acc = 0;
    uint32_t acc_phase = 0;
    bool ok = true;
    for (int i = 0; i < turns && ok; ++i) {
      const int L = sched.at(i);
      if (L < 0) continue;
      const PairTile t = sched.tile(a, *groups, by_size, L);
      const int nk = (t.red + C::BK - 1) / C::BK;
      const int rq = t.tail ? (q & 1) : q;              // 32-row block of the CTA's share
      const int wc = t.tail ? 64 : 128;                 // columns of this warp
      const int oc = (t.tail ? (q >> 1) * 128 : 0) + csel * wc;
      const int first_row = t.share * rank + rq * 32;   // of the tile
      const int rows = min(32, t.left - first_row);
      const int64_t row = (C::OP == Op::Wgrad ? static_cast<int64_t>(t.e) * a.n : 0) + t.m0 + first_row;
      OutT* out = static_cast<OutT*>(a.out) + row * sched.out_cols + t.n0 + oc;
      const int cols = sched.out_cols - t.n0 - oc;
      const uint32_t lane_base = (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(csel * wc);
      if constexpr (C::PARTS) {
        float sum[C::WCOLS];
#pragma unroll
        for (int c = 0; c < C::WCOLS; ++c) sum[c] = 0.f;
        const int parts = (nk + C::SUM_BLOCKS - 1) / C::SUM_BLOCKS;
        for (int p = 0; p < parts; ++p) {
          if (!__all_sync(0xffffffffu, mbar_wait(&acc_full[acc], acc_phase))) {
            if (lane == 0) report(a.status, DEV_WAIT_TIMEOUT_EPILOGUE);
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t tb = tmem_base + static_cast<uint32_t>(acc * C::BN) + lane_base;
#pragma unroll
          for (int c = 0; c < C::WCOLS; c += 16) {
            if (c < wc) {
              uint32_t r[16];
              tmem_ld16(tb + c, r);
              tmem_ld_wait();
#pragma unroll
              for (int j = 0; j < 16; ++j) sum[c + j] += __uint_as_float(r[j]);
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(acc_empty_leader + static_cast<uint32_t>(acc * sizeof(uint64_t)));
          if (++acc == 2) {
            acc = 0;
            acc_phase ^= 1u;
          }
        }
        if (!ok) break;
#pragma unroll
        for (int c = 0; c < C::WCOLS; c += 32) {
          if (c < wc) {
            float v[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = sum[c + j];
            store_chunk_masked<OutT, C::STG_PITCH>(stg, v, out + c, sched.out_cols, rows, cols - c, lane);
          }
        }
      } else {
        if (!__all_sync(0xffffffffu, mbar_wait(&acc_full[acc], acc_phase))) {
          if (lane == 0) report(a.status, DEV_WAIT_TIMEOUT_EPILOGUE);
          break;
        }
        tc_fence_after();
        const uint32_t tb = tmem_base + static_cast<uint32_t>(acc * C::BN) + lane_base;
#pragma unroll 1
        for (int c = 0; c < wc; c += 32) {
          uint32_t r[32];
          tmem_ld32(tb + c, r);
          tmem_ld_wait();
          float v[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]);
          store_chunk_masked<OutT, C::STG_PITCH>(stg, v, out + c, sched.out_cols, rows, cols - c, lane);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(acc_empty_leader + static_cast<uint32_t>(acc * sizeof(uint64_t)));
        if (++acc == 2) {
          acc = 0;
          acc_phase ^= 1u;
        }
      }
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, C::TMEM_COLS);
  }
}

// -------------------------------------------------------------- host side

template <class C>
cudaError_t launch_cfg(const CUtensorMap& ta, const CUtensorMap& ta32, const CUtensorMap& tb, const RArgs& a,
                       int64_t max_tiles, cudaStream_t st) {
  static std::atomic<size_t> smem_set[kMaxDevices];
  cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(ragged_gemm_kernel<C>), C::SMEM_BYTES, smem_set);
  if (e != cudaSuccess) return e;
  const int64_t sms = device_sm_count();
  const unsigned grid = static_cast<unsigned>(max_tiles < sms ? max_tiles : sms);
  return launch_dependent(ragged_gemm_kernel<C>, dim3(grid), dim3(C::THREADS), C::SMEM_BYTES, st, nullptr, 0, ta, ta32,
                          tb, a);
}

bool use_pairs(bool wgrad, const RArgs& a, int cols) {
  if (cols <= 128) return false;
  if (wgrad) return a.n > 128 && a.rows >= 64 * static_cast<int64_t>(a.E);
  return a.rows >= 192 * static_cast<int64_t>(a.E);
}

template <class C>
cudaError_t launch_pair(const CUtensorMap& ta, const CUtensorMap& ta64, const CUtensorMap& tb, const RArgs& a,
                        int64_t max_tiles, cudaStream_t st) {
  static std::atomic<size_t> smem_set[kMaxDevices];
  cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(ragged_pair_kernel<C>), C::SMEM_BYTES, smem_set);
  if (e != cudaSuccess) return e;
  const int64_t most = device_sm_count() / 2;
  const unsigned clusters = static_cast<unsigned>(max_tiles < most ? max_tiles : most);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  return launch_dependent(ragged_pair_kernel<C>, dim3(2 * clusters), dim3(C::THREADS), C::SMEM_BYTES, st, attr, 1, ta,
                          ta64, tb, a);
}

template <Op OP, bool O32>
cudaError_t run(const void* A, int64_t a_cols, const void* B, int64_t b_cols, const RArgs& a, cudaStream_t st) {
  const int64_t row_tiles = OP == Op::Wgrad ? static_cast<int64_t>(a.E) * ((a.n + 127) / 128)
                                            : a.rows / 128 + (a.rows < a.E ? a.rows : a.E);
  const int cols = OP == Op::Fwd ? a.n : a.k;
  const int bn = pick_tile_width(row_tiles, cols);
  CUtensorMap ta, ta32, tb;
  if (use_pairs(OP == Op::Wgrad, a, cols)) {
    const uint64_t rows = static_cast<uint64_t>(a.rows);
    CUtensorMap ta64;
    if (!make_map(&ta64, A, false, rows, a_cols, 64, 64)) return cudaErrorInvalidValue;
    ta = ta64;
    if (OP == Op::Wgrad) {
      if (!make_map(&tb, B, false, rows, b_cols, 64, 64)) return cudaErrorInvalidValue;
    } else if (!make_map(&ta, A, false, rows, a_cols, 64, 128) ||
               !make_map_3d(&tb, B, static_cast<uint64_t>(a.E), static_cast<uint64_t>(a.n), static_cast<uint64_t>(a.k),
                            64, OP == Op::Fwd ? 128 : 64)) {
      return cudaErrorInvalidValue;
    }
    const int64_t pair_rows = OP == Op::Wgrad ? static_cast<int64_t>(a.E) * ((a.n + 255) / 256)
                                              : a.rows / 256 + (a.rows < a.E ? a.rows : a.E);
    return launch_pair<PCfg<OP, O32>>(ta, ta64, tb, a, pair_rows * ((cols + 255) / 256), st);
  }
  const uint64_t rows = static_cast<uint64_t>(a.rows);
  if (OP == Op::Wgrad) {
    if (!make_map(&ta, A, false, rows, a_cols, 64, 64)) return cudaErrorInvalidValue;
    ta32 = ta;
    if (!make_map(&tb, B, false, rows, b_cols, 64, 64)) return cudaErrorInvalidValue;
  } else {
    if (!make_map(&ta, A, false, rows, a_cols, 64, 128)) return cudaErrorInvalidValue;
    if (!make_map(&ta32, A, false, rows, a_cols, 64, 32)) return cudaErrorInvalidValue;
    if (!make_map_3d(&tb, B, static_cast<uint64_t>(a.E), static_cast<uint64_t>(a.n), static_cast<uint64_t>(a.k), 64,
                     OP == Op::Fwd ? bn : 64))
      return cudaErrorInvalidValue;
  }
  const int64_t max_tiles = row_tiles * ((cols + bn - 1) / bn);
  if (bn == 256) return launch_cfg<RCfg<OP, 256, O32>>(ta, ta32, tb, a, max_tiles, st);
  if (bn == 128) return launch_cfg<RCfg<OP, 128, O32>>(ta, ta32, tb, a, max_tiles, st);
  return launch_cfg<RCfg<OP, 64, O32>>(ta, ta32, tb, a, max_tiles, st);
}

}  // namespace

// Tile width: 256 columns feed the tensor cores best; when that leaves SMs without a
// tile, 128 or 64 columns spread the weights' stream over more of them. A width that
// one narrower tile covers takes that tile.
int pick_tile_width(int64_t row_tiles, int cols) {
  const int sms = device_sm_count();
  for (int bn = 256; bn > 64; bn /= 2)
    if (cols > bn / 2 && row_tiles * ((cols + bn - 1) / bn) >= sms) return bn;
  return 64;
}

cudaError_t launch_ragged_forward(int64_t rows, int E, int n, int k, bool out32, const void* x, const int32_t* gs,
                                  const int32_t* off, const void* w, void* y, int32_t* status, cudaStream_t st) {
  const RArgs a{gs, off, rows, E, n, k, y, status};
  return out32 ? run<Op::Fwd, true>(x, k, w, 0, a, st) : run<Op::Fwd, false>(x, k, w, 0, a, st);
}

cudaError_t launch_ragged_dgrad(int64_t rows, int E, int n, int k, bool out32, const void* dy, const int32_t* gs,
                                const int32_t* off, const void* w, void* dx, int32_t* status, cudaStream_t st) {
  const RArgs a{gs, off, rows, E, n, k, dx, status};
  return out32 ? run<Op::Dgrad, true>(dy, n, w, 0, a, st) : run<Op::Dgrad, false>(dy, n, w, 0, a, st);
}

cudaError_t launch_ragged_wgrad(int64_t rows, int E, int n, int k, bool out32, const void* dy, const void* x,
                                const int32_t* gs, const int32_t* off, void* dw, int32_t* status, cudaStream_t st) {
  const RArgs a{gs, off, rows, E, n, k, dw, status};
  return out32 ? run<Op::Wgrad, true>(dy, n, x, k, a, st) : run<Op::Wgrad, false>(dy, n, x, k, a, st);
}

}  // namespace moe
