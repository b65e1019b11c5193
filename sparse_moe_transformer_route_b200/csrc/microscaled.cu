// Microscaled 4-bit floating point: a tensor's scale, quantisation and the way back.
//
// An element holds one of 0, .5, 1, 1.5, 2, 3, 4, 6 and a sign (E2M1) and a block
// of elements shares a scale:
//   MXFP4  32 elements, scale s = 2^(floor(log2 amax) - 2), at least 2^-127, held as
//          its biased exponent (E8M0);
//   NVFP4  16 elements, scale s = amax / (6 g) rounded to E4M3 (nearest, ties to
//          even, at most 448), g the fp32 scale of the whole tensor (1 when absent).
// The element is the representable number nearest to x / (s g), ties to the even
// code, saturating at 6. Both roundings are those of the real quotients, not of
// an fp32 approximation of them, so the codes do not depend on how they are
// computed. A block that holds an infinity or a NaN gets the NaN scale and zero
// codes, and so reads back as NaN.
//
// All three kernels are bound by memory: quantisation reads 2 (bf16) or 4 (fp32)
// bytes an element and writes 1/2 + 1/16 (NVFP4) or 1/2 + 1/32 (MXFP4); the way
// back is the reverse. A thread takes 32 bytes of the wide side in one access, so that
// a warp covers 1 KB of it in whole sectors (two 16-byte accesses a thread instead:
// dequantisation of 32768 x 2048 took 46 us, 29 this way), and four such pieces, all
// loads before the first use, in CTAs that end with them: 64 weights of 2048 x 2048 to
// bf16 take 107 us, 117 with CTAs that stay and loop, 135 with one piece at a time. Small
// tensors take one piece a thread, which reaches four times as many SMs. A block's
// threads (1 to 4) find amax with shuffles. Quantisation goes from the end of a group to
// its start: of one group about as large as L2, what the tensor scale's pass has read last
// is still there (128 MB: both passes 69.6 us, 70.7 from the start on; smaller groups and
// many groups, which both passes take in the same order: no difference).
#include "ragged.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr float kMinTensorScale = 0x1p-100f;
constexpr float kMaxTensorScale = 0x1p117f;  // within both, 1 / (6 g) and 1 / (s g) are normal; amax / 2688 is below it

template <typename T>
constexpr int elems_per_thread() {
  return 32 / static_cast<int>(sizeof(T));
}

// 32 bytes, one access.
__device__ __forceinline__ void load32(const void* p, uint32_t (&w)[8]) {
  asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
               : "l"(p));
}

__device__ __forceinline__ void store32(void* p, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// Those of buffers that start at a multiple of 16 only.
__device__ __forceinline__ void load16x2(const void* p, uint32_t (&w)[8]) {
  const uint4 a = __ldg(static_cast<const uint4*>(p)), b = __ldg(static_cast<const uint4*>(p) + 1);
  w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
  w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
}

__device__ __forceinline__ void store16x2(void* p, const uint32_t (&w)[8]) {
  static_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
  static_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
}

__device__ __forceinline__ bool aligned32(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }

// 32 bytes of input as fp32 values.
template <typename T>
__device__ __forceinline__ void widen(const uint32_t (&w)[8], float (&v)[elems_per_thread<T>()]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (sizeof(T) == 4) {
      v[i] = __uint_as_float(w[i]);
    } else {
      const float2 f = bf16x2_to_float2(w[i]);
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
}

// Eight values to eight E2M1 codes, the first in the lowest nibble (nearest, ties
// to the even code, saturating).
__device__ __forceinline__ uint32_t cvt_e2m1x8(const float* v) {
  uint32_t r;
  asm("{\n\t.reg .b8 t0, t1, t2, t3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 t0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 t1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 t2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 t3, %8, %7;\n\t"
      "mov.b32 %0, {t0, t1, t2, t3};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// Two values to E4M3 (nearest even, saturating): `lo` in the low byte.
__device__ __forceinline__ uint32_t cvt_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// The value of a non-negative E4M3 byte other than NaN.
__device__ __forceinline__ float e4m3_value(uint32_t b) {
  const uint32_t e = b >> 3, m = b & 7u;
  return e == 0 ? static_cast<float>(m) * 0x1p-9f : __uint_as_float(((e + 120u) << 23) | (m << 20));
}

// The magnitude that E2M1 code m (0..7) stands for: fields at the top of an fp32's
// exponent and mantissa give the value times 2^-126, m = 1 as a subnormal.
__device__ __forceinline__ float e2m1_value(uint32_t m) { return __uint_as_float(m << 22) * 0x1p126f; }

// fp32 approximations of a quotient are off by less than 2^-22 of it, so when the
// quotient times 1 - 2^-20 and times 1 + 2^-20 round alike, that is the rounding
// of the real quotient. Otherwise the one border between the two candidates is
// compared exactly: the sign of a fused multiply-add is that of the unrounded sum.
constexpr float kBelow = 1.0f - 0x1p-20f;
constexpr float kAbove = 1.0f + 0x1p-20f;

// amax / (6 g) in E4M3; inv6g is 1 / (6 g) to fp32.
__device__ __forceinline__ uint32_t nv_scale(float amax, float g, float inv6g) {
  const float q = amax * inv6g;
  const uint32_t both = cvt_e4m3x2(q * kBelow, q * kAbove);
  const uint32_t lo = both & 0xFFu, hi = both >> 8;
  if (lo == hi) return lo;
  const float mid = 0.5f * (e4m3_value(lo) + e4m3_value(hi));  // 5 significant bits; times 6 still exact
  const float d = fmaf(-6.0f * mid, g, amax);
  if (d != 0.0f) return d > 0.0f ? hi : lo;
  return (lo & 1u) ? hi : lo;
}

// Codes of eight values whose rounding is in doubt somewhere: `lo` and `hi` are the
// candidates of every value.
__device__ __noinline__ uint32_t nv_settle(const float (&v)[8], uint32_t lo, uint32_t hi, float s, float g) {
  uint32_t out = lo;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t a = (lo >> (4 * i)) & 7u, b = (hi >> (4 * i)) & 7u;
    if (a != b) {
      const float border = 0.5f * (e2m1_value(a) + e2m1_value(b));
      const float d = fmaf(-border * s, g, fabsf(v[i]));  // border * s is exact: 3 + 4 bits
      const bool up = d > 0.0f || (d == 0.0f && (a & 1u));
      if (up) out = (out & ~(15u << (4 * i))) | (hi & (15u << (4 * i)));
    }
  }
  return out;
}

// The codes (EPT / 8 words) and the scale byte of one piece of a block; all lanes of the
// warp together.
template <typename T, bool NV>
__device__ __forceinline__ void quantize_piece(const float (&v)[elems_per_thread<T>()], float g, float inv6g, bool g_ok,
                                               uint32_t (&word)[elems_per_thread<T>() / 8], uint32_t& sbyte) {
  constexpr int EPT = elems_per_thread<T>();
  constexpr int TPB = (NV ? 16 : 32) / EPT;  // threads that share a block
  // magnitudes compare as integers; an infinity or a NaN is above every number
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < EPT; ++i) top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
#pragma unroll
  for (int o = 1; o < TPB; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
  const bool bad = top >= 0x7F800000u || !g_ok;
  float s, inv;
  if constexpr (NV) {
    sbyte = bad ? 0x7Fu : nv_scale(__uint_as_float(top), g, inv6g);
    s = e4m3_value(sbyte);
    inv = sbyte == 0 ? 0.0f : 1.0f / (s * g);
  } else {
    const uint32_t e = top >> 23;
    sbyte = bad ? 0xFFu : (e < 2u ? 0u : e - 2u);
    s = 0.0f;
    inv = __uint_as_float((254u - (bad ? 127u : sbyte)) << 23);  // 2^(127 - sbyte): the products below are exact
  }
#pragma unroll
  for (int h = 0; h < EPT / 8; ++h) {
    float q[8], t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = v[8 * h + i] * inv;
    if constexpr (NV) {
      float u[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        t[i] = q[i] * kBelow;
        u[i] = q[i] * kAbove;
      }
      const uint32_t lo = cvt_e2m1x8(t), hi = cvt_e2m1x8(u);
      word[h] = lo;
      if (lo != hi) {
        float w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = v[8 * h + i];
        word[h] = nv_settle(w, lo, hi, s, g);
      }
    } else {
      word[h] = cvt_e2m1x8(q);
    }
    if (bad) word[h] = 0u;
  }
}

// NV: NVFP4, else MXFP4. kPieces: pieces of a thread, kThreads apart.
template <typename T, bool NV, int kPieces>
__global__ void __launch_bounds__(kThreads)
    quantize_kernel(const T* __restrict__ x, const float* __restrict__ tensor_scale, uint8_t* __restrict__ codes,
                    uint8_t* __restrict__ scales, int64_t groups, int64_t pieces_per_group) {
  constexpr int EPT = elems_per_thread<T>();
  constexpr int TPB = (NV ? 16 : 32) / EPT;
  pdl_trigger();
  pdl_wait();
  const bool wide = aligned32(x);
  for (int64_t grp = blockIdx.y; grp < groups; grp += gridDim.y) {
    float g = 1.0f, inv6g = 0.0f;
    bool g_ok = true;
    if constexpr (NV) {
      if (tensor_scale != nullptr) g = tensor_scale[grp];
      g_ok = g >= kMinTensorScale && g <= kMaxTensorScale;  // false for a NaN
      inv6g = 1.0f / (6.0f * g);
    }
    const int64_t first = grp * pieces_per_group;
    // (whole warps come here together: quantize_piece's shuffles are warp-wide)
    const int64_t p0 = static_cast<int64_t>(gridDim.x - 1 - blockIdx.x) * (kPieces * kThreads) + threadIdx.x;
    uint32_t raw[kPieces][8];
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
      const int64_t p = p0 + j * kThreads;
      if (p < pieces_per_group) {
        if (wide)
          load32(x + (first + p) * EPT, raw[j]);
        else
          load16x2(x + (first + p) * EPT, raw[j]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) raw[j][i] = 0u;
      }
    }
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
      const int64_t p = p0 + j * kThreads;
      float v[EPT];
      widen<T>(raw[j], v);
      uint32_t word[EPT / 8], sbyte;
      quantize_piece<T, NV>(v, g, inv6g, g_ok, word, sbyte);
      if (p < pieces_per_group) {
        if constexpr (EPT == 16)
          *reinterpret_cast<uint2*>(codes + (first + p) * 8) = make_uint2(word[0], word[EPT / 8 - 1]);
        else
          *reinterpret_cast<uint32_t*>(codes + (first + p) * 4) = word[0];
        if (TPB == 1 || (threadIdx.x & (TPB - 1)) == 0) scales[(first + p) / TPB] = static_cast<uint8_t>(sbyte);
      }
    }
  }
}

// Eight E2M1 codes (first in the lowest nibble) to fp32, times 2^-126: each field
// is moved to the top of an fp32's exponent and mantissa, the sign to bit 31.
__device__ __forceinline__ void e2m1x8_scaled(uint32_t w, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t n = w >> (4 * i);
    v[i] = __uint_as_float(((n & 7u) << 22) | ((n & 8u) << 28));
  }
}

template <typename T, bool NV, int kPieces>
__global__ void __launch_bounds__(kThreads)
    dequantize_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                      const float* __restrict__ tensor_scale, T* __restrict__ out, int64_t groups,
                      int64_t pieces_per_group) {
  constexpr int EPT = elems_per_thread<T>();
  constexpr int TPB = (NV ? 16 : 32) / EPT;
  pdl_trigger();
  pdl_wait();
  const bool wide = aligned32(out);
  for (int64_t grp = blockIdx.y; grp < groups; grp += gridDim.y) {
    float g = 1.0f;
    if (NV && tensor_scale != nullptr) g = tensor_scale[grp];
    const int64_t first = grp * pieces_per_group;
    const int64_t p0 = static_cast<int64_t>(blockIdx.x) * (kPieces * kThreads) + threadIdx.x;
    uint32_t w[kPieces][EPT / 8], sbyte[kPieces];
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
      const int64_t at = first + p0 + j * kThreads;
      if (p0 + j * kThreads < pieces_per_group) {
        if constexpr (EPT == 16) {
          const uint2 c = __ldg(reinterpret_cast<const uint2*>(codes + at * 8));
          w[j][0] = c.x;
          w[j][EPT / 8 - 1] = c.y;
        } else {
          w[j][0] = __ldg(reinterpret_cast<const uint32_t*>(codes + at * 4));
        }
        sbyte[j] = __ldg(scales + at / TPB) & (NV ? 0x7Fu : 0xFFu);
      }
    }
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
      if (p0 + j * kThreads >= pieces_per_group) break;
      const uint32_t b = sbyte[j];
      float s;
      if constexpr (NV)
        s = b == 0x7Fu ? __uint_as_float(0x7FC00000u) : e4m3_value(b);
      else
        s = b == 255u ? __uint_as_float(0x7FC00000u) : (b == 0u ? 0x1p-127f : __uint_as_float(b << 23));
      float v[EPT];
#pragma unroll
      for (int h = 0; h < EPT / 8; ++h) {
        float t[8];
        e2m1x8_scaled(w[j][h], t);
        // the first two products are exact (6 significant bits), so a value is rounded once
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float e = t[i] * 0x1p126f * s;
          v[8 * h + i] = NV ? e * g : e;
        }
      }
      uint32_t o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if constexpr (sizeof(T) == 4)
          o[i] = __float_as_uint(v[i]);
        else
          o[i] = pack_bf16x2(v[(2 * i) % EPT], v[(2 * i + 1) % EPT]);
      }
      T* dst = out + (first + p0 + j * kThreads) * EPT;
      if (wide)
        store32(dst, o);
      else
        store16x2(dst, o);
    }
  }
}

// scale[group] = max(amax / 2688, 2^-100) over the finite elements: 2688 = 6 * 448
// puts the largest block scale at E4M3's largest number. Division and the lower
// bound keep the order of their arguments, so each CTA divides its own amax and the
// largest result is the group's; non-negative fp32 numbers order as integers. The CTAs
// of a group are a cluster, whose first gathers the others' results in its shared
// memory; a few large groups have more CTAs each than a cluster holds and combine by an
// integer atomic maximum (whose order does not matter) over a zeroed array.
constexpr int kMaxCluster = 8;

constexpr int kTurnPieces = 4 * kThreads;  // of a CTA at a time

// The largest finite magnitude (as an integer) of a thread's four pieces p0, p0 + kThreads,
// ... of the `pieces` at `src`.
template <typename T>
__device__ __forceinline__ uint32_t top_of_turn(const T* src, int64_t p0, int64_t pieces, bool wide) {
  constexpr int EPT = elems_per_thread<T>();
  constexpr int U = kTurnPieces / kThreads;
  uint32_t raw[U][8];
#pragma unroll
  for (int j = 0; j < U; ++j) {
    const int64_t p = p0 + j * kThreads;
    if (p < pieces) {
      if (wide)
        load32(src + p * EPT, raw[j]);
      else
        load16x2(src + p * EPT, raw[j]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) raw[j][i] = 0u;
    }
  }
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < U; ++j) {
    float v[EPT];
    widen<T>(raw[j], v);
#pragma unroll
    for (int i = 0; i < EPT; ++i) {
      const uint32_t m = __float_as_uint(v[i]) & 0x7FFFFFFFu;
      top = max(top, m < 0x7F800000u ? m : 0u);
    }
  }
  return top;
}

// The scale's bits of the CTA's largest magnitude, in thread 0; ends behind a block barrier.
__device__ __forceinline__ uint32_t cta_scale(uint32_t top, uint32_t (&warp_top)[kThreads / 32]) {
  top = __reduce_max_sync(0xffffffffu, top);
  if ((threadIdx.x & 31) == 0) warp_top[threadIdx.x >> 5] = top;
  __syncthreads();
  if (threadIdx.x != 0) return 0;
#pragma unroll
  for (int i = 1; i < kThreads / 32; ++i) top = max(top, warp_top[i]);
  return __float_as_uint(fmaxf(__uint_as_float(top) / 2688.0f, kMinTensorScale));
}

template <typename T, bool CLUSTER>
__global__ void __launch_bounds__(kThreads)
    tensor_scale_kernel(const T* __restrict__ x, float* __restrict__ scale, int64_t groups, int64_t pieces_per_group) {
  constexpr int EPT = elems_per_thread<T>();
  __shared__ uint32_t warp_top[kThreads / 32];
  __shared__ uint32_t cta_top[kMaxCluster];
  pdl_trigger();
  // A CTA's shared memory may be written by another only once it is known to have
  // started: each tells the cluster here and waits for the others before its first result
  // leaves, after the loads (a CTA whose share of the group is empty gets there at once).
  if constexpr (CLUSTER) cluster_arrive();
  pdl_wait();
  const bool wide = aligned32(x);
  for (int64_t grp = blockIdx.y; grp < groups; grp += gridDim.y) {
    const T* src = x + grp * pieces_per_group * EPT;
    uint32_t top = 0;
    for (int64_t p0 = static_cast<int64_t>(blockIdx.x) * kTurnPieces + threadIdx.x; p0 < pieces_per_group;
         p0 += static_cast<int64_t>(gridDim.x) * kTurnPieces)
      top = max(top, top_of_turn(src, p0, pieces_per_group, wide));
    uint32_t mine = cta_scale(top, warp_top);
    if constexpr (CLUSTER) {
      if (grp == blockIdx.y) {  // the first of this cluster's groups
        __syncwarp();
        cluster_wait();
      }
      if (threadIdx.x == 0) {
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(mapa_shared(smem_u32(&cta_top[blockIdx.x]), 0)), "r"(mine)
                     : "memory");
      }
      __syncwarp();
      cluster_sync_all();
      if (blockIdx.x == 0 && threadIdx.x == 0) {
        for (unsigned i = 1; i < gridDim.x; ++i) mine = max(mine, cta_top[i]);
        scale[grp] = __uint_as_float(mine);
      }
      __syncwarp();
      cluster_sync_all();  // read before the next group's results come
    } else if (threadIdx.x == 0) {
      if (gridDim.x == 1)
        scale[grp] = __uint_as_float(mine);
      else
        atomicMax(reinterpret_cast<unsigned int*>(scale + grp), mine);
    }
    __syncthreads();
  }
}

// One scale over the rows that some expert owns: group e is pieces_per_row * count_e pieces in
// a row, and the groups' turns are dealt to the CTAs one after the other. The rows between
// and behind the groups hold whatever the buffer held before (moe_dispatch zeroes the pads
// of a group, and leaves the rows behind the last one) and are not read. A thread works
// out one group, and a turn finds its group in the sums (walking over 64 groups in every
// warp took 25 us).
template <typename T>
__global__ void __launch_bounds__(kThreads)
    tensor_scale_owned_kernel(const T* __restrict__ x, const int32_t* __restrict__ group_start,
                              const int32_t* __restrict__ offsets, int E, int64_t rows, int pieces_per_row,
                              float* __restrict__ scale, int32_t* status) {
  constexpr int EPT = elems_per_thread<T>();
  static_assert(kThreads >= kMaxExperts, "a thread a group");
  __shared__ uint32_t warp_top[kThreads / 32];
  __shared__ int32_t start[kMaxExperts], count[kMaxExperts];
  __shared__ int64_t first[kThreads], warp_sum[kThreads / 32];  // number of a group's first turn
  const int lane = static_cast<int>(threadIdx.x & 31u), warp = static_cast<int>(threadIdx.x >> 5);
  pdl_trigger();
  pdl_wait();
  int64_t turns = 0;
  if (static_cast<int>(threadIdx.x) < E) {
    const int e = static_cast<int>(threadIdx.x);
    checked_group(group_start, offsets, e, rows, &start[e], &count[e], status);
    turns = (static_cast<int64_t>(count[e]) * pieces_per_row + kTurnPieces - 1) / kTurnPieces;
  }
  int64_t upto = turns;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t up = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += up;
  }
  if (lane == 31) warp_sum[warp] = upto;
  __syncthreads();
  int64_t total = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w == warp) first[threadIdx.x] = total + upto - turns;
    total += warp_sum[w];
  }
  __syncthreads();
  const bool wide = aligned32(x);
  uint32_t top = 0;
  for (int64_t turn = blockIdx.x; turn < total; turn += gridDim.x) {
    int e = -1;  // the last group that starts at this turn or before (those without rows start with the next)
    for (int base = 0; base < E; base += 32)
      e += __popc(__ballot_sync(0xffffffffu, base + lane < E && first[base + lane] <= turn));
    top = max(top, top_of_turn(x + static_cast<int64_t>(start[e]) * pieces_per_row * EPT,
                               (turn - first[e]) * kTurnPieces + threadIdx.x,
                               static_cast<int64_t>(count[e]) * pieces_per_row, wide));
  }
  const uint32_t mine = cta_scale(top, warp_top);
  if (threadIdx.x == 0) atomicMax(reinterpret_cast<unsigned int*>(scale), mine);
}

// A CTA for every per_turn pieces of a group, a group each in y.
dim3 piece_grid(int64_t groups, int64_t pieces_per_group, int64_t per_turn) {
  const int64_t gy = groups < 65535 ? groups : 65535;
  const int64_t gx = (pieces_per_group + per_turn - 1) / per_turn;
  return dim3(static_cast<unsigned>(gx < 1 ? 1 : gx), static_cast<unsigned>(gy));
}

// Pieces of a thread: four once that fills the device's threads.
bool four_pieces(int64_t groups, int64_t pieces_per_group) {
  return groups * pieces_per_group >= static_cast<int64_t>(device_sm_count()) * 8 * kThreads;
}

template <typename T>
cudaError_t run_tensor_scale(int64_t groups, int64_t pieces, const void* x, float* scale, cudaStream_t st) {
  dim3 grid = piece_grid(groups, pieces, 4 * kThreads);
  const T* typed = static_cast<const T*>(x);
  // A cluster a group saves the launch that zeroes `scale` (about 2 us): where its CTAs
  // take at most eight turns (of 32 KB).
  if (grid.x > 1 && pieces <= 8 * 4 * kThreads * kMaxCluster) {
    if (grid.x > kMaxCluster) grid.x = kMaxCluster;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = grid.x;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    return launch_dependent(tensor_scale_kernel<T, true>, grid, dim3(kThreads), 0, st, attr, 1, typed, scale, groups,
                            pieces);
  }
  if (grid.x > 1) {
    const cudaError_t e = cudaMemsetAsync(scale, 0, static_cast<size_t>(groups) * 4, st);
    if (e != cudaSuccess) return e;
  }
  return launch_dependent(tensor_scale_kernel<T, false>, grid, dim3(kThreads), 0, st, nullptr, 0, typed, scale, groups,
                          pieces);
}

template <typename T>
cudaError_t run_tensor_scale_owned(int64_t rows, int E, int k, const void* x, const int32_t* gs, const int32_t* off,
                                   float* scale, int32_t* status, cudaStream_t st) {
  const int pieces_per_row = k / elems_per_thread<T>();
  const int64_t turns = (rows * pieces_per_row + kTurnPieces - 1) / kTurnPieces + E;  // at most
  const int64_t most = 4 * static_cast<int64_t>(device_sm_count());
  const cudaError_t e = cudaMemsetAsync(scale, 0, 4, st);
  if (e != cudaSuccess) return e;
  return launch_dependent(tensor_scale_owned_kernel<T>, dim3(static_cast<unsigned>(turns < most ? turns : most)),
                          dim3(kThreads), 0, st, nullptr, 0, static_cast<const T*>(x), gs, off, E, rows, pieces_per_row,
                          scale, status);
}

}  // namespace

cudaError_t launch_tensor_scale_owned(int64_t rows, int E, int k, bool fp32, const void* x, const int32_t* gs,
                                      const int32_t* off, float* scale, int32_t* status, cudaStream_t st) {
  return fp32 ? run_tensor_scale_owned<float>(rows, E, k, x, gs, off, scale, status, st)
              : run_tensor_scale_owned<__nv_bfloat16>(rows, E, k, x, gs, off, scale, status, st);
}

cudaError_t launch_tensor_scale(int64_t groups, int64_t per_group, bool fp32, const void* x, float* scale,
                                cudaStream_t st) {
  const int64_t pieces = per_group / (fp32 ? 8 : 16);
  return fp32 ? run_tensor_scale<float>(groups, pieces, x, scale, st)
              : run_tensor_scale<__nv_bfloat16>(groups, pieces, x, scale, st);
}

cudaError_t launch_quantize(bool nv, int64_t groups, int64_t per_group, bool fp32, const void* x,
                            const float* tensor_scale, uint8_t* codes, uint8_t* scales, cudaStream_t st) {
  const int64_t pieces = per_group / (fp32 ? 8 : 16);
  const bool four = four_pieces(groups, pieces);
  const dim3 grid = piece_grid(groups, pieces, (four ? 4 : 1) * kThreads);
  auto go = [&](auto kern, auto* typed) {
    return launch_dependent(kern, grid, dim3(kThreads), 0, st, nullptr, 0, typed, tensor_scale, codes, scales, groups,
                            pieces);
  };
  const float* xf = static_cast<const float*>(x);
  const __nv_bfloat16* xb = static_cast<const __nv_bfloat16*>(x);
  using bf16 = __nv_bfloat16;
  if (nv) {
    if (fp32) return four ? go(quantize_kernel<float, true, 4>, xf) : go(quantize_kernel<float, true, 1>, xf);
    return four ? go(quantize_kernel<bf16, true, 4>, xb) : go(quantize_kernel<bf16, true, 1>, xb);
  }
  if (fp32) return four ? go(quantize_kernel<float, false, 4>, xf) : go(quantize_kernel<float, false, 1>, xf);
  return four ? go(quantize_kernel<bf16, false, 4>, xb) : go(quantize_kernel<bf16, false, 1>, xb);
}

cudaError_t launch_dequantize(bool nv, int64_t groups, int64_t per_group, bool fp32, const uint8_t* codes,
                              const uint8_t* scales, const float* tensor_scale, void* out, cudaStream_t st) {
  const int64_t pieces = per_group / (fp32 ? 8 : 16);
  const bool four = four_pieces(groups, pieces);
  const dim3 grid = piece_grid(groups, pieces, (four ? 4 : 1) * kThreads);
  auto go = [&](auto kern, auto* typed) {
    return launch_dependent(kern, grid, dim3(kThreads), 0, st, nullptr, 0, codes, scales, tensor_scale, typed, groups,
                            pieces);
  };
  float* of = static_cast<float*>(out);
  __nv_bfloat16* ob = static_cast<__nv_bfloat16*>(out);
  using bf16 = __nv_bfloat16;
  if (nv) {
    if (fp32) return four ? go(dequantize_kernel<float, true, 4>, of) : go(dequantize_kernel<float, true, 1>, of);
    return four ? go(dequantize_kernel<bf16, true, 4>, ob) : go(dequantize_kernel<bf16, true, 1>, ob);
  }
  if (fp32) return four ? go(dequantize_kernel<float, false, 4>, of) : go(dequantize_kernel<float, false, 1>, of);
  return four ? go(dequantize_kernel<bf16, false, 4>, ob) : go(dequantize_kernel<bf16, false, 1>, ob);
}

}  // namespace moe
