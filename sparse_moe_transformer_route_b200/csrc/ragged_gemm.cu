// Matrix products grouped by expert with ragged sizes, and their gradients.
//
// Expert e owns count_e rows (any number) of row buffers X [rows, k], Y [rows, n]
// and a weight W_e [n, k]:
//   forward   y[r]  = W_e x[r]                        Y_e^T  = W_e   X_e^T
//   dgrad     dx[r] = W_e^T dy[r]                     dX_e^T = W_e^T dY_e^T
//   wgrad     dW_e  = sum over rows r of dy[r] x[r]^T dW_e^T = X_e^T dY_e
// bf16 operands, fp32 sums, bf16 or fp32 results.
//
// Sizes. Forward and dgrad make the weight the MMA's M operand (128 output columns a
// CTA) and the rows its N operand, which may be any multiple of 16 (a pair's 32): a
// group's rows are cut into equal tiles of at most BN rows, and one costs what its rows
// cost. (With the rows as M, every group pays for 128 or 256 at a time, and an M = 128
// MMA on a pair takes as long as an M = 256 one: 64 groups of about 512 rows, 2048 x
// 2048, took 217 us, 205 this way.) Groups start at any row: a tile's operand box simply starts
// there (only the innermost TMA coordinate has an alignment rule), reads into the next
// group where the group ends inside the tile, and rows past the end are not stored.
// Widths are multiples of 8 (16-byte row strides); TMA fills what lies past a width with
// zeros, so a reduction's tail adds nothing. The weights are mapped in three dimensions,
// so that a tile that leaves an expert's matrix reads zeros and not the next expert's
// rows. In wgrad the reduction runs over a group's rows: the rows past its end in the
// last box belong to another group (or hold anything at all), so they are overwritten
// with zeros in shared memory before that step is issued.
//
// Structure per CTA (persistent, one an SM): warp 0 issues TMA loads into a ring of
// stages, warp 1 issues tcgen05.mma, warps 2..9 read the fp32 accumulator from TMEM and
// store; two accumulators, so that a tile's epilogue runs under the next tile's MMAs.
// Every wait is bounded; a timeout is recorded in the status word and the CTA unwinds.
// What bounds it: few rows, the stream of weights (64 rows over 64 experts of 2048 x
// 2048: 55 us, 92% of the measured HBM rate); many, the tensor cores (one expert of
// 32768 rows 164 us, 1,680 TFLOP/s; 131072 rows over 64 experts: dgrad and wgrad,
// which also writes 1 GB of fp32, 1.65 ms together). These and the figures below are
// replayed graphs with a cold L2; in a loop of calls of some seconds the power cap bounds
// the large ones (32768 rows over 64 experts 274 us instead of 213, the gradients 2.0 ms).
//
// PAIR: a tile is 256 x BN on the two CTAs of a cluster (the SMs of one TPC), each with
// its 128 rows of the M operand, half of the N operand and its 128 accumulator rows;
// the leader (rank 0) issues cta_group::2 MMAs that read both shared memories. Per SM a
// 64-term stage is then 32 KB for the MMA work that takes 48 KB with one CTA a tile.
// wgrad's rows past a group's end: each CTA clears its own shared memory. The peer's
// last, ragged stage arrives on a barrier of its own, its second warp clears the rows
// and only then arrives on the leader's barrier, which counts one arrival a CTA. (The
// rows are cleared in the peer's own shared memory, made visible to the tensor core's
// reads by the proxy fence and read by the peer's own tensor core, so the arrival needs
// no cluster-scope release; one costs 2% of the whole product.)
#include <cudaTypedefs.h>

#include <cmath>

#include "ragged.cuh"

namespace moe {
namespace {

enum class Op { Fwd, Dgrad, Wgrad };

template <Op OP_, int BN_, bool PAIR_, bool O32_>
struct RCfg {
  static constexpr Op OP = OP_;
  static constexpr bool W = OP == Op::Wgrad;
  static constexpr bool PAIR = PAIR_;
  // largest groups first, so that the last turn's tiles are short (64 groups by Zipf's
  // law, 32768 rows: 217 us in order of the experts, 213 sorted); a small call does not
  // get back what sorting takes
  static constexpr bool SORTED = PAIR || W;
  static constexpr int CTAS = PAIR ? 2 : 1;
  static constexpr bool A_MN = OP != Op::Fwd;  // operand read as [reduction][row of the operand]
  static constexpr bool B_MN = W;
  static constexpr int BM = 128 * CTAS;        // M: columns of the result
  static constexpr int BN = BN_;               // N: at most so many of its rows
  static constexpr int UNIT = 16 * CTAS;       // N is a multiple of this
  static constexpr int B_ROWS = BN / CTAS;     // of the N operand in this CTA's shared memory
  static constexpr bool O32 = O32_;
  using OutT = std::conditional_t<O32, float, __nv_bfloat16>;
  static constexpr int BK = 64;  // one 128-byte swizzle row when K-major
  static constexpr int UK = 16;
  static constexpr int CHUNK_BYTES = BK * 128;  // MN-major: 64 reduction rows of one 64-column piece
  static constexpr int A_BYTES = 128 * BK * 2;
  static constexpr int B_BYTES = B_ROWS * BK * 2;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int A_STEP = A_MN ? UK * 128 : UK * 2;  // bytes between the operands of two steps
  static constexpr int B_STEP = B_MN ? UK * 128 : UK * 2;
  // The tensor core's fp32 sum over a long reduction loses about half an ulp a step
  // towards zero. Where the result is fp32, or the reduction may be as long as the
  // buffer (wgrad), the accumulator is handed over every SUM_BLOCKS stages (512
  // terms) and the parts are added in fp32 registers, rounded to nearest. dW over 8192
  // rows is then off by 4.8e-7 of its norm, 1.0e-6 with parts of 1024 and 9.1e-6 as one
  // sum (an fp32 library product: 9.5e-7), for less than 1% of the time. A bf16 result's
  // one sum over the width is off by about 2e-6 of itself after 2048 terms, a thousandth of
  // the rounding that follows; parts would cost it 1 to 4% (32768 rows over 64 experts
  // 213 -> 219 us).
  static constexpr bool PARTS = O32 || W;
  static constexpr int SUM_BLOCKS = 8;
  static constexpr uint32_t IDESC0 = make_idesc(false, A_MN, B_MN, BM, 0);  // N is added by the tile
  static constexpr uint32_t TMEM_COLS = 2 * BN;
  static constexpr int EPI_WARPS = 8;
  static constexpr int THREADS = 64 + 32 * EPI_WARPS;
  static constexpr int CHUNKS = (BN + 63) / 64;  // 32-column accumulator chunks of an epilogue warp
  static constexpr int MISC_BYTES = 1024 + static_cast<int>(sizeof(RaggedGroups));
  static constexpr int STAGES_FIT = (227 * 1024 - 1024 - MISC_BYTES) / STAGE_BYTES;
  static constexpr int STAGES = STAGES_FIT > 12 ? 12 : STAGES_FIT;
  static constexpr size_t SMEM_BYTES = 1024 + static_cast<size_t>(STAGES) * STAGE_BYTES + MISC_BYTES;
  static_assert(STAGES >= 4 && (3 * STAGES + 7) * 8 <= 1024, "ring");
  static_assert(BN == 256 || (!PAIR && (BN == 128 || BN == 64 || (BN == 32 && !W))), "tile N");
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
  int m0;   // first column of the result
  int n0;   // its first row: of the buffer (fwd, dgrad) or of dW_e
  int N;    // the MMA's N
  int red;  // length of the reduction
  int row0; // wgrad: first row of the group
  int left; // rows that exist (fwd, dgrad: of the group, at most N)
};

template <class C>
struct Schedule {
  int n_tiles, nM, m_size, c, G;
  FastDiv by_m, by_n;  // (by_n: wgrad)
  __device__ static int m_tiles(const RArgs& a) { return ((C::OP == Op::Fwd ? a.n : a.k) + C::BM - 1) / C::BM; }
  __device__ Schedule(const RArgs& a, const RaggedGroups& g)
      : by_m(m_tiles(a)), by_n(C::W ? (a.n + C::BN - 1) / C::BN : 1) {
    c = static_cast<int>(blockIdx.x) / C::CTAS;
    G = static_cast<int>(gridDim.x) / C::CTAS;
    m_size = C::OP == Op::Fwd ? a.n : a.k;
    nM = m_tiles(a);
    n_tiles = C::W ? a.E * nM * ((a.n + C::BN - 1) / C::BN) : g.tiles[a.E];
  }
  // Tile of this CTA's (pair's) turn i, or -1. wgrad's tiles cost their group's rows and
  // come largest group first: every other turn runs backwards over the CTAs, which evens
  // out what a turn's first and last CTA get.
  __device__ int at(int i) const {
    const int64_t L = static_cast<int64_t>(i) * G + ((C::W && (i & 1)) ? G - 1 - c : c);
    return L < n_tiles ? static_cast<int>(L) : -1;
  }
  // turns of any CTA: at() may be -1 in the last one only
  __device__ int turns() const { return (n_tiles + G - 1) / G; }
  __device__ RTile tile(const RArgs& a, const RaggedGroups& g, int L) const {
    RTile t;
    if constexpr (C::W) {
      const int mt = by_n(L);
      t.n0 = (L - mt * static_cast<int>(by_n.d)) * C::BN;
      const int place = by_m(mt);
      t.e = g.order[place];
      t.m0 = (mt - place * nM) * C::BM;
      t.N = C::BN;
      t.red = g.count[t.e];
      t.row0 = g.start[t.e];
      t.left = a.n - t.n0;
    } else {
      const int place = tile_place(g, a.E, L);
      t.e = g.order[place];
      const int in = L - g.tiles[place];
      const int rt = by_m(in);
      t.m0 = (in - rt * nM) * C::BM;
      const int count = g.count[t.e], per = g.per[t.e];
      t.n0 = g.start[t.e] + rt * per;
      t.left = min(per, count - rt * per);
      t.N = (t.left + C::UNIT - 1) / C::UNIT * C::UNIT;
      t.red = C::OP == Op::Fwd ? a.k : a.n;
      t.row0 = 0;
    }
    return t;
  }
};

// wgrad: zeroes reduction rows [from, from + count) of every 64-column piece of a stage.
// One warp.
template <class C>
__device__ __forceinline__ void clear_stage_rows(unsigned char* stage, int from, int count, int lane) {
  const int per = count * 8;
  for (int j = lane; j < C::STAGE_BYTES / C::CHUNK_BYTES * per; j += 32) {
    const int piece = j / per, w = j - piece * per;
    *reinterpret_cast<uint4*>(stage + piece * C::CHUNK_BYTES + from * 128 + w * 16) = make_uint4(0u, 0u, 0u, 0u);
  }
  fence_proxy_async_smem();
  __syncwarp();
}

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1)
    ragged_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                       const __grid_constant__ CUtensorMap tmB32, const RArgs a) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  unsigned char* misc = smem + static_cast<size_t>(C::STAGES) * C::STAGE_BYTES;
  uint64_t* full = reinterpret_cast<uint64_t*>(misc);
  uint64_t* empty = full + C::STAGES;
  uint64_t* acc_full = empty + C::STAGES;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* drain = acc_empty + 2;
  uint64_t* ragged_full = drain + 1;  // per stage: the peer's copies of a group's last, ragged stage (wgrad)
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(ragged_full + C::STAGES);
  volatile uint32_t* loads = tmem_holder + 1;  // stages that this CTA's producer has asked for (wgrad on a pair)
  RaggedGroups* groups = reinterpret_cast<RaggedGroups*>(misc + 1024);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rank = C::PAIR ? static_cast<int>(cluster_ctarank()) : 0;
  const bool leader = rank == 0;

  pdl_trigger();
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&full[s], C::W && C::PAIR ? 2 : 1);  // (of a pair the leader's copies are the ones used)
      mbar_init(&empty[s], 1);
      mbar_init(&ragged_full[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], C::CTAS * C::EPI_WARPS);
    }
    mbar_init(drain, 1);
    fence_mbar_init();
    *loads = 0;
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
    if constexpr (!C::W) tma_prefetch_desc(&tmB32);
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
  load_groups<C::BN, C::UNIT, C::SORTED>(groups, a.group_start, a.offsets, a.E, a.rows, Schedule<C>::m_tiles(a), a.status);
  tc_fence_before();
  if constexpr (C::PAIR)
    cluster_sync_all();  // both CTAs' barriers are initialised before the other's copies or commits reach them
  else
    __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = uniform(*tmem_holder);
  const Schedule<C> sched(a, *groups);
  const int turns = sched.turns();
  // barriers that the leader's MMA warp waits on
  const uint32_t full_leader = C::PAIR ? mapa_shared(smem_u32(full), 0) : smem_u32(full);
  const uint32_t acc_empty_leader = C::PAIR ? mapa_shared(smem_u32(acc_empty), 0) : smem_u32(acc_empty);

  if (warp == 0) {
    // ------------------------------------------------ TMA producer
    int stage = 0;
    uint32_t phase = 0;
    int issued = 0;
    bool ok = true;
    for (int i = 0; i < turns && ok; ++i) {
      const int L = sched.at(i);
      if (L < 0) continue;
      const RTile t = sched.tile(a, *groups, L);
      const int red = uniform(t.red);
      const int nk = (red + C::BK - 1) / C::BK;
      const int need = uniform(t.N) / C::CTAS;
      const int am = uniform(t.m0) + 128 * rank;
      const int bn = uniform(t.n0) + need * rank;
      const int e = uniform(t.e);
      const int row0 = uniform(t.row0);
      // rows (K-major B): the whole box, or 32-row boxes over the rows that count when
      // these are few
      const int boxes = C::W || need > C::B_ROWS - 32 ? 0 : (need + 31) / 32;
      const uint32_t bytes = C::A_BYTES + (boxes == 0 ? C::B_BYTES : boxes * 32 * 128);
      for (int kb = 0; kb < nk; ++kb) {
        if (!__all_sync(0xffffffffu, mbar_wait(&empty[stage], phase ^ 1u))) {
          if (lane == 0) report(a.status, DEV_WAIT_TIMEOUT_PRODUCER);
          ok = false;
          break;
        }
        if (elect_one()) {
          unsigned char* sa = smem + static_cast<size_t>(stage) * C::STAGE_BYTES;
          unsigned char* sb = sa + C::A_BYTES;
          const int k0 = kb * C::BK;
          // a pair's ragged last stage counts on each CTA's own barrier
          const bool own = C::PAIR && C::W && kb + 1 == nk && red % C::UK != 0;
          if (leader) {
            mbar_arrive_expect_tx(&full[stage], own ? bytes : C::CTAS * bytes);
          } else if constexpr (C::W) {
            if (own)
              mbar_arrive_expect_tx(&ragged_full[stage], bytes);
            else
              mbar_arrive_cluster(full_leader + static_cast<uint32_t>(stage * sizeof(uint64_t)));
          }
          if constexpr (C::W) {
            auto load = [&](const CUtensorMap* map, unsigned char* dst, int col) {
              if (!C::PAIR || own)
                tma_load_2d(map, leader ? &full[stage] : &ragged_full[stage], dst, col, row0 + k0);
              else
                tma_load_2d_pair(map, &full[stage], dst, col, row0 + k0);
            };
            load(&tmA, sa, am);
            load(&tmA, sa + C::CHUNK_BYTES, am + 64);
#pragma unroll
            for (int ch = 0; ch < C::B_ROWS / 64; ++ch) load(&tmB, sb + ch * C::CHUNK_BYTES, bn + ch * 64);
            if constexpr (C::PAIR) *loads = static_cast<uint32_t>(issued + 1);
          } else {
            auto load_w = [&](unsigned char* dst, int c0, int c1) {
              if constexpr (C::PAIR)
                tma_load_3d_pair(&tmA, &full[stage], dst, c0, c1, e);
              else
                tma_load_3d(&tmA, &full[stage], dst, c0, c1, e);
            };
            if constexpr (C::OP == Op::Fwd) {
              load_w(sa, k0, am);
            } else {
              load_w(sa, am, k0);
              load_w(sa + C::CHUNK_BYTES, am + 64, k0);
            }
            auto load_x = [&](const CUtensorMap* map, unsigned char* dst, int row) {
              if constexpr (C::PAIR)
                tma_load_2d_pair(map, &full[stage], dst, k0, row);
              else
                tma_load_2d(map, &full[stage], dst, k0, row);
            };
            if (boxes == 0) {
              load_x(&tmB, sb, bn);
            } else {
              for (int q = 0; q < boxes; ++q) load_x(&tmB32, sb + q * (32 * 128), bn + 32 * q);
            }
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
        const int last = (issued - 1 - s) / C::STAGES;  // uses of stage s, less one
        if (!mbar_wait(&full[s], static_cast<uint32_t>(last & 1))) report(a.status, DEV_WAIT_TIMEOUT_DRAIN);
      }
    }
  } else if (warp == 1) {
    if (leader) {
      // ---------------------------------------------- MMA issuer (the whole warp; it
      // also clears the rows past a group's end)
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
        const RTile t = sched.tile(a, *groups, L);
        const int nk = uniform((t.red + C::BK - 1) / C::BK);
        const uint32_t idesc = uniform(C::IDESC0 | (static_cast<uint32_t>(t.N) >> 3) << 17);
        for (int kb = 0; kb < nk; ++kb) {
          const bool first = kb == 0 || (C::PARTS && kb % C::SUM_BLOCKS == 0);
          if (first && !__all_sync(0xffffffffu, mbar_wait(&acc_empty[acc], acc_phase ^ 1u))) ok = false;
          if (ok && !__all_sync(0xffffffffu, mbar_wait(&full[stage], phase))) ok = false;
          if (!ok) {
            if (lane == 0) report(a.status, DEV_WAIT_TIMEOUT_MMA);
            break;
          }
          const int terms = min(C::BK, t.red - kb * C::BK);
          const int steps = (terms + C::UK - 1) / C::UK;
          if constexpr (C::W) {
            if (terms % C::UK != 0)
              clear_stage_rows<C>(smem + static_cast<size_t>(stage) * C::STAGE_BYTES, terms, steps * C::UK - terms,
                                  lane);
          }
          tc_fence_after();
          const bool part_done = kb + 1 == nk || (C::PARTS && (kb + 1) % C::SUM_BLOCKS == 0);
          if (elect_one()) {
            const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * C::BN);
            const uint32_t off = static_cast<uint32_t>(stage) * (C::STAGE_BYTES >> 4);
            umma_stage<C::PAIR, C::A_STEP, C::B_STEP>(d_tmem, DescLo{desc0.a + off, desc0.b + off}, idesc, first, steps);
            if constexpr (C::PAIR) {
              umma_commit_pair(&empty[stage], 0x3);
              if (part_done) umma_commit_pair(&acc_full[acc], 0x3);
            } else {
              umma_commit(&empty[stage]);
              if (part_done) umma_commit(&acc_full[acc]);
            }
          }
          if (++stage == C::STAGES) {
            stage = 0;
            phase ^= 1u;
          }
          if (part_done) {
            ++handed;
            if (++acc == 2) {
              acc = 0;
              acc_phase ^= 1u;
            }
          }
        }
      }
      __syncwarp();
      if (elect_one()) {
        if constexpr (C::PAIR)
          umma_commit_pair(drain, 0x1);
        else
          umma_commit(drain);
        if (!mbar_wait(drain, 0)) report(a.status, DEV_WAIT_TIMEOUT_DRAIN);
        // a pair's epilogues have released every accumulator, so that no remote arrival
        // reaches this CTA after it has ended
        for (int b = 0; C::PAIR && b < 2; ++b) {
          const int uses = handed > b ? (handed - 1 - b) / 2 + 1 : 0;
          if (uses > 0 && !mbar_wait(&acc_empty[b], static_cast<uint32_t>((uses - 1) & 1)))
            report(a.status, DEV_WAIT_TIMEOUT_DRAIN);
        }
      }
    } else if constexpr (C::W) {
      // ---------------------------------------------- the peer's ragged stages
      int stage = 0;        // of the tile's first block
      uint32_t parity = 0;  // bit s: parity of ragged_full[s]'s next phase
      for (int i = 0; i < turns; ++i) {
        const int L = sched.at(i);
        if (L < 0) continue;
        const RTile t = sched.tile(a, *groups, L);
        const int nk = (t.red + C::BK - 1) / C::BK;
        if (t.red % C::UK != 0) {
          const int last = (stage + nk - 1) % C::STAGES;
          // The stage is loaded after everything before it, any number of tiles: the wait
          // goes on for as long as this CTA's producer does, each of whose own waits is
          // bounded, and gives up when it has asked for nothing new in a whole bounded wait.
          bool in = false;
          uint32_t before, now = uniform(*loads);
          do {
            before = now;
            in = __all_sync(0xffffffffu, mbar_wait(&ragged_full[last], (parity >> last) & 1u));
            now = uniform(*loads);
          } while (!in && now != before);
          if (!in) {
            if (lane == 0) report(a.status, DEV_WAIT_TIMEOUT_MMA);
            break;
          }
          parity ^= 1u << last;
          const int terms = t.red - (nk - 1) * C::BK;
          clear_stage_rows<C>(smem + static_cast<size_t>(last) * C::STAGE_BYTES, terms,
                              (terms + C::UK - 1) / C::UK * C::UK - terms, lane);
          if (lane == 0) mbar_arrive_cluster(full_leader + static_cast<uint32_t>(last * sizeof(uint64_t)));
        }
        stage = (stage + nk) % C::STAGES;
      }
    }
  } else {
    // ------------------------------------------------ epilogue
    using OutT = typename C::OutT;
    const int q = warp & 3;               // TMEM lane quarter of this warp
    const int csel = (warp - 2) >> 2;     // it takes every other 32-column chunk
    int acc = 0;
    uint32_t acc_phase = 0;
    bool ok = true;
    auto release = [&]() {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (C::PAIR)
          mbar_arrive_cluster_relaxed(acc_empty_leader + static_cast<uint32_t>(acc * sizeof(uint64_t)));
        else
          mbar_arrive_relaxed(&acc_empty[acc]);
      }
      if (++acc == 2) {
        acc = 0;
        acc_phase ^= 1u;
      }
    };
    for (int i = 0; i < turns && ok; ++i) {
      const int L = sched.at(i);
      if (L < 0) continue;
      const RTile t = sched.tile(a, *groups, L);
      const int nk = (t.red + C::BK - 1) / C::BK;
      const int mrow = t.m0 + 128 * rank + q * 32;  // first M row of this warp
      const int m_left = sched.m_size - mrow;       // of those that exist (may be <= 0)
      const uint32_t lane_base = static_cast<uint32_t>(q * 32) << 16;
      // one 32 x 32 chunk, accumulator columns [c, c + 32)
      auto store = [&](const float (&v)[32], int c) {
        const int64_t row = (C::W ? static_cast<int64_t>(t.e) * a.n : 0) + t.n0 + c;
        OutT* out = static_cast<OutT*>(a.out) + row * sched.m_size + mrow;
        store_chunk_turned<OutT>(v, out, sched.m_size, t.left - c, m_left, lane);
      };
      if constexpr (C::PARTS) {
        float sum[C::CHUNKS * 32];
#pragma unroll
        for (int c = 0; c < C::CHUNKS * 32; ++c) sum[c] = 0.f;
        const int parts = (nk + C::SUM_BLOCKS - 1) / C::SUM_BLOCKS;  // 0: an expert without rows
        for (int p = 0; p < parts; ++p) {
          if (!__all_sync(0xffffffffu, mbar_wait(&acc_full[acc], acc_phase))) {
            if (lane == 0) report(a.status, DEV_WAIT_TIMEOUT_EPILOGUE);
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t tb = tmem_base + static_cast<uint32_t>(acc * C::BN) + lane_base;
#pragma unroll
          for (int ch = 0; ch < C::CHUNKS; ++ch) {
            const int c = (2 * ch + csel) * 32;
            if (c < t.N) {
#pragma unroll
              for (int h = 0; h < 32; h += 16) {
                uint32_t r[16];
                tmem_ld16(tb + c + h, r);
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 16; ++j) sum[ch * 32 + h + j] += __uint_as_float(r[j]);
              }
            }
          }
          release();
        }
        if (!ok) break;
#pragma unroll
        for (int ch = 0; ch < C::CHUNKS; ++ch) {
          const int c = (2 * ch + csel) * 32;
          if (c < t.N) {
            float v[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = sum[ch * 32 + j];
            store(v, c);
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
        for (int c = csel * 32; c < t.N; c += 64) {
          uint32_t r[32];
          tmem_ld32(tb + c, r);
          tmem_ld_wait();
          float v[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]);
          store(v, c);
        }
        release();
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

template <Op OP, int BN, bool PAIR, bool O32>
cudaError_t launch(const void* A, const void* B, const RArgs& a, cudaStream_t st) {
  using C = RCfg<OP, BN, PAIR, O32>;
  static std::atomic<size_t> smem_set[kMaxDevices];
  cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(ragged_gemm_kernel<C>), C::SMEM_BYTES, smem_set);
  if (e != cudaSuccess) return e;
  const uint64_t rows = static_cast<uint64_t>(a.rows), n = static_cast<uint64_t>(a.n), k = static_cast<uint64_t>(a.k);
  CUtensorMap ta, tb, tb32;
  int64_t tiles;
  if (OP == Op::Wgrad) {
    if (!make_map(&ta, A, false, rows, k, 64, 64) || !make_map(&tb, B, false, rows, n, 64, 64))
      return cudaErrorInvalidValue;
    tb32 = tb;
    tiles = static_cast<int64_t>(a.E) * ((a.k + C::BM - 1) / C::BM) * ((a.n + BN - 1) / BN);
  } else {
    const uint64_t width = OP == Op::Fwd ? k : n;
    if (!make_map_3d(&ta, A, static_cast<uint64_t>(a.E), n, k, 64, OP == Op::Fwd ? 128 : 64) ||
        !make_map(&tb, B, false, rows, width, 64, C::B_ROWS) || !make_map(&tb32, B, false, rows, width, 64, 32))
      return cudaErrorInvalidValue;
    // row tiles: at most one more than full ones for every group that has rows
    tiles = (a.rows / BN + (a.rows < a.E ? a.rows : a.E)) * (((OP == Op::Fwd ? a.n : a.k) + C::BM - 1) / C::BM);
  }
  const int64_t most = device_sm_count() / C::CTAS;
  const unsigned units = static_cast<unsigned>(tiles < most ? tiles : most);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  return launch_dependent(ragged_gemm_kernel<C>, dim3(C::CTAS * units), dim3(C::THREADS), C::SMEM_BYTES, st, attr,
                          PAIR ? 1 : 0, ta, tb, tb32, a);
}

// y and dx (A: the weights, B: the rows).
template <Op OP, bool O32>
cudaError_t run_rows(const void* w, const void* x, const RArgs& a, cudaStream_t st) {
  const int red = OP == Op::Fwd ? a.k : a.n;
  switch (pick_row_tile(a.rows, a.E, OP == Op::Fwd ? a.n : a.k, (red + 63) / 64, 100)) {
    case kTilePair: return launch<OP, 256, true, O32>(w, x, a, st);
    case kTile256: return launch<OP, 256, false, O32>(w, x, a, st);
    case kTile128: return launch<OP, 128, false, O32>(w, x, a, st);
    case kTile64: return launch<OP, 64, false, O32>(w, x, a, st);
    default: return launch<OP, 32, false, O32>(w, x, a, st);
  }
}

// Nanoseconds of a 64-term stage in a full grid, per kind of tile (32, 64, 128 or 256 rows
// by 128 columns, 256 by 256 on a pair): fitted to 64 groups of 1 to 1024 rows, 2048 x
// 2048, where the tiles took 1954, 1032, 598, 422 and 373 us for 65536 rows.
constexpr int64_t kStageNs[kTileKinds] = {270, 290, 340, 475, 420};
constexpr int64_t kPairStartNs = 2000;  // a cluster launch and its barriers

int64_t turns_of(int kind, int64_t units, int64_t sms) {
  const int64_t slots = sms / (kind == kTilePair ? 2 : 1);
  return (units + slots - 1) / slots;
}

// dW: the kind of tile (256 columns of dW by 256 rows on a pair, or 128 columns by 256, 128
// or 64 rows) that ends first: its turns times a turn's stages and its stores.
template <bool O32>
cudaError_t run_weights(const void* dy, const void* x, const RArgs& a, cudaStream_t st) {
  const int64_t stages = (a.rows / a.E + 63) / 64, sms = device_sm_count();
  int best = kTile64;
  int64_t least = INT64_MAX;
  for (int kind = kTile64; kind < kTileKinds; ++kind) {
    const int bm = kind == kTilePair ? 256 : 128, bn = kind == kTile64 ? 64 : kind == kTile128 ? 128 : 256;
    const int64_t units = static_cast<int64_t>(a.E) * ((a.k + bm - 1) / bm) * ((a.n + bn - 1) / bn);
    const int64_t ns = turns_of(kind, units, sms) * (stages * kStageNs[kind] + 700 + 8 * bn) +
                       (kind == kTilePair ? kPairStartNs : 0);
    if (ns < least) {
      least = ns;
      best = kind;
    }
  }
  switch (best) {
    case kTilePair: return launch<Op::Wgrad, 256, true, O32>(x, dy, a, st);
    case kTile256: return launch<Op::Wgrad, 256, false, O32>(x, dy, a, st);
    case kTile128: return launch<Op::Wgrad, 128, false, O32>(x, dy, a, st);
    default: return launch<Op::Wgrad, 64, false, O32>(x, dy, a, st);
  }
}

}  // namespace

// The kind of tile that ends first: its turns over the SMs times a turn's stages. The host
// does not know the groups: it takes the buffer's rows as their sum, equal groups, and each
// two standard deviations of a random split taller, so that most groups fit the tile that
// it picks. A buffer that is mostly padding gets taller tiles than its groups need: 64 rows
// over 64 experts of 2048 x 2048 in moe_dispatch's buffer of 8192 rows take 66.5 us, back
// to back 62.4 (4-bit: 28.7 and 27.3). The times a stage were fitted to one width. For 64
// groups of 2048 x 2048 the fastest kind is 32 rows at 1 a group, 64 at up to 32 (90 against 100 us
// with 32 rows), 128 at 64 to 96 (96 against 139 and 100) and a pair from 128 on (102
// against 106 with 256 rows); a single group of 96 rows takes 32 so that more SMs read
// its weight.
int pick_row_tile(int64_t rows, int E, int out_cols, int64_t stages, int stage_percent) {
  const int64_t groups = rows < E ? rows : E, sms = device_sm_count();
  const int64_t mean = (rows + groups - 1) / groups;
  const int64_t tall = mean + 2 * static_cast<int64_t>(std::sqrt(static_cast<double>(mean)));
  int best = kTile32;
  int64_t least = INT64_MAX;
  for (int kind = kTile32; kind < kTileKinds; ++kind) {
    const int bm = kind == kTilePair ? 256 : 128, most = kind == kTilePair ? 256 : 32 << kind;
    const int64_t units = groups * ((tall + most - 1) / most) * ((out_cols + bm - 1) / bm);
    const int64_t ns = turns_of(kind, units, sms) * (stages * kStageNs[kind] * stage_percent / 100 + 600) +
                       (kind == kTilePair ? kPairStartNs : 0);
    if (ns < least) {
      least = ns;
      best = kind;
    }
  }
  return best;
}

cudaError_t launch_ragged_forward(int64_t rows, int E, int n, int k, bool out32, const void* x, const int32_t* gs,
                                  const int32_t* off, const void* w, void* y, int32_t* status, cudaStream_t st) {
  const RArgs a{gs, off, rows, E, n, k, y, status};
  return out32 ? run_rows<Op::Fwd, true>(w, x, a, st) : run_rows<Op::Fwd, false>(w, x, a, st);
}

cudaError_t launch_ragged_dgrad(int64_t rows, int E, int n, int k, bool out32, const void* dy, const int32_t* gs,
                                const int32_t* off, const void* w, void* dx, int32_t* status, cudaStream_t st) {
  const RArgs a{gs, off, rows, E, n, k, dx, status};
  return out32 ? run_rows<Op::Dgrad, true>(w, dy, a, st) : run_rows<Op::Dgrad, false>(w, dy, a, st);
}

cudaError_t launch_ragged_wgrad(int64_t rows, int E, int n, int k, bool out32, const void* dy, const void* x,
                                const int32_t* gs, const int32_t* off, void* dw, int32_t* status, cudaStream_t st) {
  const RArgs a{gs, off, rows, E, n, k, dw, status};
  return out32 ? run_weights<true>(dy, x, a, st) : run_weights<false>(dy, x, a, st);
}

}  // namespace moe
