// 4-bit weights with group scales: the format, the dense product and the
// sparse FFN over 4-bit rows (include/asffn.h, "4-bit weights").
//
//   asf_w4_quantize / asf_w4_dequantize   k_w4_quantize, k_w4_dequantize
//   asf_w4_matmul       y = act(W x + b)  k_w4_dot, or k_w4_matmul_tc for fp16 x and many rows
//   asf_w4_sparse_ffn   gate/up rows      k_w4_dot over the list
//                       down projection   k_w4_down
//
// Mathematics.  With w = (c - 8) s_G, G = i / group, a row's product is
//   sum_G s_G * sum_{i in G} (c_i - 8) x_i .
// The inner sum has small whole numbers on one side.  They are exact in fp16
// and in bf16, so the tensor cores (mma.sync m16n8k16, fp32 accumulators) take
// them as they are, straight from registers, and the group scale multiplies
// the fp32 sum once per group: no weight is ever rounded.  x in fp16 is the
// other operand as it is; x in fp32 is the exact sum of three bf16 parts
// (8 + 8 + 8 mantissa bits, by truncation; below 2^-110 the last ones are lost),
// multiplied in three instructions into the same accumulators.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "asffn.h"
#include "common.cuh"
#include "host.cuh"

using namespace asf;

namespace {

constexpr int kBlk = 128;              // weights per format block: 16 words of 8 codes
constexpr int kSuper = 512;            // weights per scale superblock, and the unit of a split of k
constexpr int kDotWarps = 16;
constexpr int kDownWarps = 8;
constexpr int kDownCols = 256;         // columns per down-projection CTA (two blocks)
constexpr int kTicketBytes = kMaxTiles * 4;   // one byte a ticket: more than the splits a row tile has
constexpr size_t kDotSmem = 226 * 1024;
constexpr int kPartsPerCta = 64;       // see dot_per
constexpr float kFp16Max = 65504.f;

__host__ __device__ inline int ceil_div(int a, int b) { return (a + b - 1) / b; }
__host__ __device__ inline int w4_kp(int k) { return ceil_div(k, kBlk) * kBlk; }
__host__ __device__ inline int w4_scale_bytes(int k, int group) {
  return ceil_div(ceil_div(w4_kp(k), kSuper) * (kSuper / group) * 2, 16) * 16;
}
inline int64_t w4_row_bytes(int k, int group) { return (int64_t)w4_kp(k) / 2 + w4_scale_bytes(k, group); }

// ------------------------------------------------------------- quantize --
// A CTA takes 1, 2, 4 or 8 rows, so that its eight warps have a superblock of
// 512 weights each; a lane has 8 weights of each half of it, the group maximum
// comes from group / 8 neighbouring lanes.  A code is the rounding of the IEEE
// quotient v / s.  v (1/s) is within 2^-23 of it, relatively, and |v / s| < 8,
// so wherever that product is 1e-5 or more off a half its rounding is the same;
// the few others divide.  (Dividing always: 72 us for 11008 x 4096 in fp16.)
// 11008 x 4096 in fp16 with the way back: 55 us, 4.1 TB/s of the four passes;
// issue slots bound the quantizer (0.85 instructions a scheduler and cycle).
__device__ __forceinline__ void rows_of_cta(int nsb, int warp, int &lsh, int &sb, int64_t &row) {
  lsh = nsb > 4 ? 3 : nsb > 2 ? 2 : nsb > 1 ? 1 : 0;           // log2 of the warps of a row
  sb = warp & ((1 << lsh) - 1);
  row = (int64_t)blockIdx.x * (8 >> lsh) + (warp >> lsh);
}

template <typename T>
__global__ void __launch_bounds__(256)
k_w4_quantize(const T *__restrict__ src, int rows, int k, int group, unsigned char *__restrict__ dst, int64_t stride) {
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int nsb = ceil_div(k, kSuper), kp = w4_kp(k);
  int lsh, sb0;
  int64_t row;
  rows_of_cta(nsb, threadIdx.x >> 5, lsh, sb0, row);
  if (row >= rows) return;
  const T *in = src + row * k;
  unsigned char *out = dst + row * stride;
  const int gsh = group == 32 ? 2 : group == 64 ? 3 : 4;       // log2 of a group's lanes
  for (int sb = sb0; sb < nsb; sb += 1 << lsh) {
    uint4 raw[2][sizeof(T) / 2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int i0 = sb * kSuper + h * 256 + lane * 8;
#pragma unroll
      for (int q = 0; q < (int)sizeof(T) / 2; ++q)
        raw[h][q] = i0 < k ? __ldcs(reinterpret_cast<const uint4 *>(in + i0) + q) : make_uint4(0, 0, 0, 0);   // k % 8 == 0
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int i0 = sb * kSuper + h * 256 + lane * 8;
      float v[8];
      // the largest magnitude by its bits: a NaN counts as more than an infinity
      uint32_t m = 0;
      if constexpr (sizeof(T) == 2) {
        Vec<__half>::to_float(raw[h][0], v);
        const uint32_t w[4] = {raw[h][0].x, raw[h][0].y, raw[h][0].z, raw[h][0].w};
        uint32_t m2 = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) m2 = __vmaxu2(m2, w[i] & 0x7fff7fffu);
        m = max(m2 >> 16, m2 & 0xffffu);
      } else {
        const uint32_t w[8] = {raw[h][0].x, raw[h][0].y, raw[h][0].z, raw[h][0].w,
                               raw[h][sizeof(T) / 2 - 1].x, raw[h][sizeof(T) / 2 - 1].y, raw[h][sizeof(T) / 2 - 1].z,
                               raw[h][sizeof(T) / 2 - 1].w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          v[i] = __uint_as_float(w[i]);
          m = max(m, w[i] & 0x7fffffffu);
        }
      }
#pragma unroll
      for (int o = 0; o < 4; ++o) {
        if (o >= gsh) break;
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1 << o));
      }
      float top;
      if constexpr (sizeof(T) == 2) top = __half2float(__ushort_as_half((unsigned short)m));
      else top = __uint_as_float(m);
      const __half sh = __float2half_rn(__fdiv_rn(top, 7.f));
      const float s = __half2float(sh);
      const bool good = s <= kFp16Max;             // a group that fp16 scales cannot hold reads back as NaN
      // From fp16's normal range on |v / s| <= 7 (1 + 2^-11): no code is clamped.
      const bool plain = good && s >= 6.103515625e-05f;
      const float r = plain ? __frcp_rn(s) : 0.f;
      constexpr float kMagic = 12582912.f;         // 1.5 * 2^23: adding it rounds to whole numbers, half to even
      uint32_t word = 0;
      float off = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float t = fmaf(v[i], r, kMagic);
        off = fmaxf(off, fabsf(fmaf(v[i], r, kMagic - t)));
        // t's bits are kMagic's plus the whole number: shifted sums of them are
        // the codes' plus a constant, modulo 2^32
        word += __float_as_uint(t) << (16 * (i & 1) + 4 * (i >> 1));
      }
      word += 0x88888888u - 0x4b400000u * 0x1111u - ((0x4b400000u * 0x1111u) << 16);
      if (!good || s == 0.f) {
        word = 0x88888888u;
      } else if (off > 0.5f - 1e-5f || !plain) {
        word = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float c = fminf(fmaxf(rintf(__fdiv_rn(v[i], s)), -8.f), 7.f);
          word |= (uint32_t)((int)c + 8) << (16 * (i & 1) + 4 * (i >> 1));
        }
      }
      const int wi = (i0 % kBlk) / 8;              // word j*4 + t of the block is stored at t*4 + j
      if (i0 < kp) *reinterpret_cast<uint32_t *>(out + (i0 / kBlk) * 64 + ((wi & 3) * 4 + (wi >> 2)) * 4) = word;
      if ((lane & ((1 << gsh) - 1)) == 0) {        // past kp the maximum is 0: zero padding
        const __half w = good ? sh : __ushort_as_half((unsigned short)0x7fff);
        *reinterpret_cast<__half *>(out + kp / 2 + (i0 >> (gsh + 3)) * 2) = w;
      }
    }
  }
  const int used = nsb * (kSuper / group) * 2;     // rest of the scale area, up to 16 bytes
  if (sb0 == 0 && lane * 2 < w4_scale_bytes(k, group) - used)
    *reinterpret_cast<uint16_t *>(out + kp / 2 + used + lane * 2) = 0;
}

// ---------------------------------------------------- codes to operands --
// The four pairs (weights 2p, 2p+1 of a word) as fp16 or bf16 whole numbers
// -8..7.  Or-ing a nibble into the mantissa of 1024 (fp16: pair 0, and pair 1
// as 1024 + 16 q) or of 128 (bf16) is exact, and so is what follows: the method
// of Kim, Henry, Fahim and Awadalla, "Who Says Elephants Can't Run: Bringing Large
// Scale MoE Models into Cloud Scale Production" (2022), with this format's zero
// point and order of weights.
__device__ __forceinline__ uint32_t lop_or(uint32_t w, uint32_t mask, uint32_t magic) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w), "r"(mask), "r"(magic));   // (w & mask) | magic
  return r;
}
__device__ __forceinline__ uint32_t hsub2(uint32_t a, uint32_t b) {
  const __half2 r = __hsub2(*reinterpret_cast<__half2 *>(&a), *reinterpret_cast<__half2 *>(&b));
  return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
  const __half2 r =
      __hfma2(*reinterpret_cast<__half2 *>(&a), *reinterpret_cast<__half2 *>(&b), *reinterpret_cast<__half2 *>(&c));
  return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ uint32_t bsub2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hsub2(*reinterpret_cast<__nv_bfloat162 *>(&a), *reinterpret_cast<__nv_bfloat162 *>(&b));
  return *reinterpret_cast<const uint32_t *>(&r);
}
template <bool BF>
__device__ __forceinline__ void unpack8(uint32_t w, uint32_t (&h)[4]) {
  if constexpr (BF) {
#pragma unroll
    for (int p = 0; p < 4; ++p) h[p] = bsub2(lop_or(w >> (4 * p), 0x000f000fu, 0x43004300u), 0x43084308u);
  } else {
    const uint32_t w8 = w >> 8;
    h[0] = hsub2(lop_or(w, 0x000f000fu, 0x64006400u), 0x64086408u);                    // (1024 + q) - 1032
    h[1] = hfma2(lop_or(w, 0x00f000f0u, 0x64006400u), 0x2c002c00u, 0xd480d480u);       // (1024 + 16 q) / 16 - 72
    h[2] = hsub2(lop_or(w8, 0x000f000fu, 0x64006400u), 0x64086408u);
    h[3] = hfma2(lop_or(w8, 0x00f000f0u, 0x64006400u), 0x2c002c00u, 0xd480d480u);
  }
}
// D += A B, A 16x16 and B 16x8 in the registers of a warp.
template <bool BF>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  if constexpr (BF)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// one of the two fp16 values of a word
__device__ __forceinline__ float half_of(uint32_t w, int hi) {
  return __half2float(__ushort_as_half((unsigned short)(hi ? w >> 16 : w & 0xffffu)));
}
// 4-, 8- or 16-byte asynchronous copy global -> shared
template <int BYTES>
__device__ __forceinline__ void cp_async_small(void *dst, const void *src, bool in = true) {
  if constexpr (BYTES == 16)
    cp_async16(dst, src, in ? 16u : 0u);
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(smem_u32(dst)), "l"(src), "n"(BYTES),
                 "r"(in ? BYTES : 0)
                 : "memory");
}
// D = A B
template <bool BF>
__device__ __forceinline__ void mma16816_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
  if constexpr (BF)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ float trunc_bf16(float v) { return __uint_as_float(__float_as_uint(v) & 0xffff0000u); }
// the upper halves of two floats as one pair (lo first)
__device__ __forceinline__ uint32_t upper2(float lo, float hi) {
  return __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x7632);
}

// ----------------------------------------------------------- dequantize --
// fp16: (c - 8) is exact in fp16, and its product with the scale rounds once.
// HBM bounds it: 11008 x 4096 alone 22.6 us, 5.0 TB/s.
template <typename T>
__global__ void __launch_bounds__(256)
k_w4_dequantize(const unsigned char *__restrict__ src, int64_t stride, int rows, int k, int group, T *__restrict__ dst) {
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int nsb = ceil_div(k, kSuper);
  int lsh, sb0;
  int64_t row;
  rows_of_cta(nsb, threadIdx.x >> 5, lsh, sb0, row);
  if (row >= rows) return;
  const unsigned char *in = src + row * stride;
  const __half *sc = reinterpret_cast<const __half *>(in + w4_kp(k) / 2);
  T *out = dst + row * k;
  const int gsh = group == 32 ? 5 : group == 64 ? 6 : 7;
  for (int sb = sb0; sb < nsb; sb += 1 << lsh) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int at = sb * kSuper + h * 256 + lane * 8;
      if (at >= k) continue;
      const int wi = (at % kBlk) / 8;
      const uint32_t w = *reinterpret_cast<const uint32_t *>(in + (at / kBlk) * 64 + ((wi & 3) * 4 + (wi >> 2)) * 4);
      uint32_t c[4];
      unpack8<false>(w, c);
      if constexpr (sizeof(T) == 2) {
        const __half2 s = __half2half2(sc[at >> gsh]);
        uint4 u;
        uint32_t *p = &u.x;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const __half2 v = __hmul2(*reinterpret_cast<const __half2 *>(&c[q]), s);
          p[q] = *reinterpret_cast<const uint32_t *>(&v);
        }
        __stcs(reinterpret_cast<uint4 *>(out + at), u);
      } else {
        const float s = __half2float(sc[at >> gsh]);
        float v[8];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&c[q]));
          v[2 * q] = f.x * s;
          v[2 * q + 1] = f.y * s;
        }
        __stcs(reinterpret_cast<float4 *>(out + at), make_float4(v[0], v[1], v[2], v[3]));
        __stcs(reinterpret_cast<float4 *>(out + at) + 1, make_float4(v[4], v[5], v[6], v[7]));
      }
    }
  }
}

// ------------------------------------------------------- row products --
struct DotArgs {
  const unsigned char *data;   // first row (gate rows of the list form)
  int64_t stride;              // bytes from row to row (neuron to neuron)
  int64_t up;                  // bytes from a neuron's gate row to its up row
  int rows;                    // rows, or neurons the list may name
  int k;
  const void *x;
  int B;
  const float *bias;           // per row, or null
  int relu;
  const int32_t *idx, *count;  // list form; null: all rows
  float *y;                    // dense: [B][rows]; list form: a [positions][8 * NT]
  int y16;                     // dense: y is fp16
  float *part;                 // partial tiles of a split k
  int most;                    // superblocks of k whose x fits a CTA
  Header *hdr;
};

// Stages of two blocks (256 weights of 16 rows, and their scales) that a warp
// keeps in shared memory, all but one of them in flight.
__host__ __device__ constexpr int dot_stages(int NT) { return NT == 1 ? 4 : 3; }
__host__ __device__ constexpr int dot_stage_bytes(int GS) { return 2048 + 16 * (4 << GS); }
__host__ __device__ constexpr size_t dot_ring_bytes(int NT, int GS) { return (size_t)kDotWarps * dot_stages(NT) * dot_stage_bytes(GS); }

// Superblocks of k per CTA (k is split into ceil(nsb / per) parts): the least
// of (row tiles of a CTA, in whole rounds of its four schedulers, and 8 at
// least, about what keeps enough loads in flight) x per, where a split costs a
// CTA as much as 12 superblocks for its last ticket and an eighth of one per
// tile and 8 tokens for the partial sums.  At most 64 tile parts an SM, or
// twice the parts that x forces, are made, which bounds the workspace.
__device__ __forceinline__ int dot_per(int tiles, int nsb, int most, int ctas, int NT, int lane) {
  const int64_t room = max((int64_t)kPartsPerCta * ctas, 2 * (int64_t)tiles * ceil_div(nsb, most));
  uint32_t best = 0xffffffffu;
  for (int p0 = 0; p0 < most; p0 += 32) {
    const int per = p0 + lane + 1;
    uint32_t key = 0xffffffffu;
    if (per <= most) {
      const int S = ceil_div(nsb, per);
      if (S <= ctas && (per == most || (int64_t)tiles * S <= room)) {
        const int c = ceil_div(tiles, ctas / S), w = c <= kDotWarps ? 4 : kDotWarps;
        const int u = max(8, ceil_div(c, w) * w);
        const int64_t cost = 8 * (int64_t)u * per + (S > 1 ? 8 * (12 + S) + (int64_t)u * NT : 0);
        key = (uint32_t)min(cost, (int64_t)(1 << 23)) * 256u + (uint32_t)(255 - per);
      }
    }
    best = min(best, __reduce_min_sync(0xffffffffu, key));
  }
  return 255 - (int)(best & 255u);
}

// Each warp owns row tiles of 16 rows (8 neurons' gate rows over their 8 up
// rows in the gated form: a thread then holds a neuron's gate and up sums of
// the same tokens side by side) over its CTA's part of k.  It streams them
// through a ring of its own in shared memory by 16-byte cp.async, whole
// 128-byte lines of a row, across tile ends, without meeting the other warps.
// x's part sits in shared memory for the CTA's life.  With k split, a tile's
// partial sums meet in the workspace and the warp that takes the tile's last
// ticket adds them in the order of the splits.
// What bounds it: start, first rows and ticket (4 us of the 6.8 us of 4096 x 4096
// for one token; L2 holds its 9 MB); on long streams the unpacking and waits for
// rows, 28672 x 8192 for one token 41.5 us, 2.9 TB/s.  The three forms are compiled
// apart: one body for all took 7.25 us for 4096 x 4096, and 96 us instead of 88 for
// the OPT-shaped layer of 16 tokens.
enum { kDense = 0, kListUp = 1, kListGated = 2 };   // gated: tiles of 8 gate rows over their 8 up rows

template <bool BF, int NT, int GS, int MODE>
__global__ void __launch_bounds__(kDotWarps * 32, 1) k_w4_dot(DotArgs A) {
  extern __shared__ __align__(128) unsigned char sm[];
  constexpr bool LIST = MODE != kDense, gated = MODE == kListGated;
  constexpr int P = BF ? 3 : 1;                    // parts of x
  constexpr int AC = NT == 1 ? 2 : 1;              // accumulators of a group: a shorter chain where one token tile is all
  constexpr int NS = dot_stages(NT), SB = dot_stage_bytes(GS), SCB = 4 << GS;
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  int total = A.rows;
  if (LIST && A.count) {
    total = ld_cg_i32(A.count);
    if (total < 0 || total > A.rows) {
      if (blockIdx.x == 0 && threadIdx.x == 0) flag_error(&A.hdr->err, kErrIndex);
      total = total < 0 ? 0 : A.rows;
    }
  }
  constexpr int per = gated ? 8 : 16;
  const int tiles = ceil_div(total, per);
  const int nblk = w4_kp(A.k) / kBlk, nsb = ceil_div(nblk, 4);
  const int sb_per = dot_per(tiles, nsb, A.most, gridDim.x, NT, lane);
  const int S = ceil_div(nsb, sb_per);
  const int ctas = gridDim.x / S;                  // CTAs of one part of k
  const int s = blockIdx.x / ctas, p = blockIdx.x % ctas;
  if (s >= S) return;
  const int b0 = s * sb_per * 4, b1 = min(nblk, b0 + sb_per * 4);   // blocks of this part
  // a warp's unit: tpu consecutive tiles under one ticket
  const int tpu = S > 1 ? ceil_div(tiles, kTicketBytes) : 1;
  const int units = ceil_div(tiles, tpu);
  if (p >= units) return;

  unsigned char *ring = sm + (size_t)warp * NS * SB;
  unsigned char *sx = sm + dot_ring_bytes(NT, GS);
  const int stages = ceil_div(b1 - b0, 2);
  const int step = ctas * kDotWarps;

  // x's part: [P][B][b1-b0 blocks], rows 64 bytes past a multiple of 128 apart
  // (eight lanes of a 16-byte read then touch every bank once)
  const int kw = stages * 2 * kBlk;                // a last stage of one block multiplies zeros
  const int xrow = kw * 2 + 64;
  for (int i = threadIdx.x; i < kw / 8; i += blockDim.x)
    *reinterpret_cast<uint4 *>(sx + (size_t)P * A.B * xrow + i * 16) = make_uint4(0, 0, 0, 0);
  if constexpr (!BF) {                             // all of it in flight ahead of the rings (waiting for it: OPT shape, 16 tokens, 2 us more)
    for (int i = threadIdx.x; i < A.B * (kw / 8); i += blockDim.x) {
      const int b = i / (kw / 8), c = (i % (kw / 8)) * 8, kk = b0 * kBlk + c;
      const __half *src = static_cast<const __half *>(A.x) + (int64_t)b * A.k + kk;
      cp_async16(sx + (size_t)b * xrow + c * 2, kk < A.k ? src : A.x, kk < A.k ? 16u : 0u);
    }
    cp_async_commit();
  }

  // ---- the copying side, ahead of the computing side
  struct {
    int unit, tile, stage;
  } pr{p + ctas * warp, 0, 0}, co;
  pr.tile = pr.unit * tpu;
  co = pr;
  auto advance = [&](auto &c) {                    // to the next stage; true at a tile's end
    if (++c.stage < stages) return false;
    c.stage = 0;
    if (++c.tile >= min(tiles, (c.unit + 1) * tpu)) {
      c.unit += step;
      c.tile = c.unit * tpu;
    }
    return true;
  };
  const int mine = lane & (per - 1);               // this lane's place in a tile's list
  auto id_of = [&](int tile) {
    const int pos = min(tile * per + mine, total - 1);
    return LIST && A.idx ? ld_cg_i32(A.idx + pos) : pos;
  };
  const unsigned char *rp[4], *sp;
  int next_id = 0;
  auto point = [&]() {                             // at pr.tile's rows; next_id holds its list entry
    int id = next_id;
    if ((unsigned)id >= (unsigned)A.rows) {
      flag_error(&A.hdr->err, kErrIndex);
      id = 0;
    }
    {                                              // the entry of the tile after this one
      int nu = pr.unit, nt = pr.tile + 1;
      if (nt >= min(tiles, (nu + 1) * tpu)) nt = (nu + step) * tpu;
      if (nt < tiles) next_id = id_of(nt);
    }
    const int part = lane & 7;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 4 * i + (lane >> 3);
      const unsigned char *row = A.data + (int64_t)__shfl_sync(0xffffffffu, id, r & (per - 1)) * A.stride;
      if (gated && r >= 8) row += A.up;
      rp[i] = row + (int64_t)b0 * 64 + part * 16;
    }
    sp = A.data + (int64_t)id * A.stride + (gated && (lane & 8) ? A.up : 0) + w4_kp(A.k) / 2 +
         (int64_t)b0 * (2 << GS);
  };
  auto copy = [&](int slot) {                      // stage pr.stage of pr.tile
    if (pr.unit < units) {
      unsigned char *to = ring + slot * SB;
      const int part = lane & 7;
      const bool in = b0 + pr.stage * 2 + (part >> 2) < b1;
#pragma unroll
      for (int i = 0; i < 4; ++i)
      {
        cp_async16(to + (part >> 2) * 1024 + (4 * i + (lane >> 3)) * 64 + (part & 3) * 16, rp[i], in ? 16u : 0u);
        rp[i] += 128;
      }
      // the scale area is padded to whole superblocks: a stage's scales are inside it
      if (lane < 16) cp_async_small<SCB>(to + 2048 + lane * SCB, sp);
      sp += SCB;
      if (advance(pr) && pr.unit < units) point();
    }
    cp_async_commit();
  };
  if (pr.unit < units) {
    next_id = id_of(pr.tile);
    point();
  }
#pragma unroll
  for (int i = 0; i < NS - 1; ++i) copy(i);

  if constexpr (BF) {
    for (int i = threadIdx.x; i < A.B * (kw / 8); i += blockDim.x) {
      const int b = i / (kw / 8), c = (i % (kw / 8)) * 8, kk = b0 * kBlk + c;
      float f[8] = {};
      if (kk < A.k) {
        const float4 *src = reinterpret_cast<const float4 *>(static_cast<const float *>(A.x) + (int64_t)b * A.k + kk);
        const float4 u = src[0], w = src[1];
        f[0] = u.x; f[1] = u.y; f[2] = u.z; f[3] = u.w; f[4] = w.x; f[5] = w.y; f[6] = w.z; f[7] = w.w;
      }
#pragma unroll
      for (int q = 0; q < 3; ++q) {
        uint4 v;
        v.x = upper2(f[0], f[1]); v.y = upper2(f[2], f[3]); v.z = upper2(f[4], f[5]); v.w = upper2(f[6], f[7]);
        *reinterpret_cast<uint4 *>(sx + ((size_t)q * A.B + b) * xrow + c * 2) = v;
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] -= trunc_bf16(f[e]);
      }
    }
  } else {
    cp_async_wait<NS - 1>();                       // x, the oldest group
  }
  __syncthreads();

  // ---- the computing side
  float tot[NT][4];
  auto clear = [&]() {
#pragma unroll
    for (int n = 0; n < NT; ++n) tot[n][0] = tot[n][1] = tot[n][2] = tot[n][3] = 0.f;
  };
  // this lane's token of each tile; columns past the batch read a row of zeros
  uint32_t xo[NT], xpart[NT];                      // and from part to part
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    xo[n] = (8 * n + g < A.B ? 8 * n + g : P * A.B) * xrow;
    xpart[n] = 8 * n + g < A.B ? A.B * xrow : 0;
  }
  auto compute = [&](const unsigned char *st, int stage) {
    uint32_t sa[1 << GS], sb[1 << GS];             // scales of rows g and g + 8
#pragma unroll
    for (int i = 0; i < (1 << GS); ++i) {
      sa[i] = *reinterpret_cast<const uint32_t *>(st + 2048 + g * SCB + 4 * i);
      sb[i] = *reinterpret_cast<const uint32_t *>(st + 2048 + (g + 8) * SCB + 4 * i);
    }
    uint4 ca[2], cb[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      ca[u] = *reinterpret_cast<const uint4 *>(st + u * 1024 + g * 64 + t * 16);
      cb[u] = *reinterpret_cast<const uint4 *>(st + u * 1024 + (g + 8) * 64 + t * 16);
    }
    const unsigned char *xb = sx + t * 16 + stage * 512;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const uint32_t wa[4] = {ca[u].x, ca[u].y, ca[u].z, ca[u].w}, wb[4] = {cb[u].x, cb[u].y, cb[u].z, cb[u].w};
      float acc[NT][AC][4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bool fresh = j % (4 >> GS) == 0, last = (j + 1) % (4 >> GS) == 0;   // of a group
        uint32_t ha[4], hb[4];
        unpack8<BF>(wa[j], ha);
        unpack8<BF>(wb[j], hb);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int q = 0; q < P; ++q) {
            const uint4 xv = *reinterpret_cast<const uint4 *>(xb + xo[n] + q * xpart[n] + u * 256 + j * 64);
            if (fresh && q == 0) mma16816_first<BF>(acc[n][0], ha[0], hb[0], ha[1], hb[1], xv.x, xv.y);
            else mma16816<BF>(acc[n][0], ha[0], hb[0], ha[1], hb[1], xv.x, xv.y);
            if (fresh && q == 0 && AC == 2) mma16816_first<BF>(acc[n][AC - 1], ha[2], hb[2], ha[3], hb[3], xv.z, xv.w);
            else mma16816<BF>(acc[n][AC - 1], ha[2], hb[2], ha[3], hb[3], xv.z, xv.w);
          }
        if (last) {                                // scale the group's sum
          const int i = (u << GS) + (j >> (2 - GS));
          const float fa = half_of(sa[i >> 1], i & 1), fb = half_of(sb[i >> 1], i & 1);
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              tot[n][e] = fmaf(e < 2 ? fa : fb, AC == 2 ? acc[n][0][e] + acc[n][AC - 1][e] : acc[n][0][e], tot[n][e]);
        }
      }
    }
  };
  // List form: the entry and bias of rows g and g + 8 of a tile, read during its
  // first and its last stage, so that the sums do not wait for two loads (list of
  // 1100, d 4096: 14.5 -> 14.0 us; the dense form, with one load, loses 0.1 to 0.3).
  int nrn[2] = {0, 0};
  float bias[2] = {0.f, 0.f};
  auto name_rows = [&](int tile) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int pos = tile * per + g + 8 * h;
      nrn[h] = -1;
      if (pos < total && !(h == 1 && gated)) nrn[h] = A.idx ? ld_cg_i32(A.idx + pos) : pos;
    }
  };
  auto read_bias = [&]() {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      bias[h] = 0.f;
      if ((unsigned)nrn[h] < (unsigned)A.rows) bias[h] = __ldg(A.bias + nrn[h]);
    }
  };
  auto finish = [&](int tile) {                    // tot holds the whole sums
    if constexpr (!LIST) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = tile * 16 + g + 8 * h;
        if (r >= total) continue;
        const float row_bias = A.bias ? __ldg(A.bias + r) : 0.f;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int b = 8 * n + 2 * t + c;
            float v = tot[n][2 * h + c] + row_bias;
            if (A.relu) v = v > 0.f ? v : (v != v ? v : 0.f);
            if (b >= A.B) continue;
            if (A.y16) reinterpret_cast<__half *>(A.y)[(int64_t)b * A.rows + r] = __float2half_rn(v);
            else A.y[(int64_t)b * A.rows + r] = v;
          }
      }
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (h == 1 && gated) continue;
        const int pos = tile * per + g + 8 * h;
        if (pos >= total) continue;
        const bool ok = (unsigned)nrn[h] < (unsigned)A.rows;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float v[2];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float a = tot[n][2 * h + c] + bias[h];
            a = a > 0.f ? a : (a != a ? a : 0.f);
            if (gated) a *= tot[n][2 + c];
            v[c] = ok && 8 * n + 2 * t + c < A.B ? a : 0.f;
          }
          *reinterpret_cast<float2 *>(A.y + ((int64_t)pos * NT + n) * 8 + 2 * t) = make_float2(v[0], v[1]);
        }
      }
    }
  };
  // the tile's partial sums, and with the unit's last ticket its whole sums
  auto share = [&](int tile, int unit) {
    float4 *to = reinterpret_cast<float4 *>(A.part) + ((int64_t)tile * S + s) * NT * 32 + lane;
#pragma unroll
    for (int n = 0; n < NT; ++n) __stcg(to + n * 32, make_float4(tot[n][0], tot[n][1], tot[n][2], tot[n][3]));
    if (tile + 1 < min(tiles, (unit + 1) * tpu)) return;
    __syncwarp();                                  // the warp's sums, then lane 0's release
    const int sh = 8 * (unit & 3);
    uint32_t *word = &A.hdr->tile_done[unit >> 2];
    uint32_t old = 0;
    if (lane == 0) old = (ticket_acq_rel(word, 1u << sh) >> sh) & 255u;
    old = __shfl_sync(0xffffffffu, old, 0);
    if (old != (uint32_t)(S - 1)) return;
    __syncwarp();                                  // lane 0's acquire, then every lane's reads of the parts
    for (int tl = unit * tpu; tl <= tile; ++tl) {
      clear();
      if (LIST && unit * tpu != tile) {  // a unit of several tiles: the registers hold the last one's
        name_rows(tl);
        read_bias();
      }
      const float4 *from = reinterpret_cast<const float4 *>(A.part) + (int64_t)tl * S * NT * 32 + lane;
#pragma unroll 4
      for (int q = 0; q < S; ++q)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float4 v = __ldcg(from + (q * NT + n) * 32);
          tot[n][0] += v.x; tot[n][1] += v.y; tot[n][2] += v.z; tot[n][3] += v.w;
        }
      finish(tl);
    }
    if (lane == 0) atomicSub(word, (uint32_t)S << sh);                 // the ticket is zero again for the next call
  };

  clear();
  for (int i = 0; co.unit < units; i = i + 1 == NS ? 0 : i + 1) {
    cp_async_wait<NS - 2>();
    __syncwarp();
    copy(i == 0 ? NS - 1 : i - 1);                 // the slot that the last step has read
    if (LIST) {
      if (co.stage == 0) name_rows(co.tile);
      if (co.stage == stages - 1) read_bias();
    }
    compute(ring + i * SB, co.stage);
    const int unit = co.unit, tile = co.tile;
    if (advance(co)) {
      if (S == 1) finish(tile);
      else share(tile, unit);
      clear();
    }
  }
}

// ------------------------------------------------ fp16 x: tcgen05 -------
// The dense product for fp16 x.  A row of the tile is a lane of tensor memory:
// its thread reads the row's codes from shared memory, turns them into fp16
// whole numbers and stores them to tensor memory as the MMA's A operand (M 128,
// K 16); x is the B operand, N = 16 or 32 tokens.  What is left per weight is
// the unpacking: nothing is read again for the tokens, and the products cost no
// issue slots.  Each group's product has an accumulator of its own, which the
// row's thread scales into its fp32 totals.
//   one warp    loads stages of 256 weights of 128 rows, their scales
//               and x's columns by TMA (rows and columns past the end as zeros)
//   four sets of four warps unpack, each one half of every other stage into an A
//               operand of its own, so that a set unpacks while the others'
//               blocks are multiplied (two sets, each with two operands and one
//               half of every stage, where 32 tokens x 4 groups of 32 weights
//               leave room for two accumulators only)
//   two warps   issue the MMAs, one for each half of a stage
// The (row tile, stage) pairs are dealt out in one run of equal lengths per
// CTA; tiles that fall to several CTAs meet in the workspace, where the one that
// takes a tile's last ticket adds the parts in the order of the CTAs.
// 28672 x 8192 (121 MB): 37.5 us for one token, 3.2 TB/s, 47 us for 32 tokens.
// No unit is full (issue slots 58% used, DRAM 37%, tensor pipe 9%): the unpacking
// warps wait for their stages and for their own chain of unpacking and stores, and
// with many tokens for the passes over the accumulators (32 tokens, groups of 64:
// 50.8 us).
constexpr int kTcStageK = 256;
template <int N, int GS>
struct MatTc {
  static constexpr int W = 128 * kTcStageK / 2;
  static constexpr int SC = 128 * 16;              // a 16-byte piece of each row's scales
  static constexpr int X = N * kTcStageK * 2;
  static constexpr int STAGE = W + SC + X;
  static constexpr int SETS = (N << GS) <= 64 ? 4 : 2;
  static constexpr int NS = N == 16 ? 7 : SETS == 4 ? 5 : 6;
  static constexpr int THREADS = SETS * 128 + 96;
  static constexpr int BAR = 1024;
  static constexpr int RED = (SETS - 1) * 128 * (N + 1) * 4;
  static constexpr size_t SMEM = 1024 + BAR + RED + 1024 + (size_t)NS * STAGE;
  static constexpr uint32_t COLS = 512;            // A: 4 x 64 columns, then D: SETS x (N << GS)
  static_assert(STAGE % 1024 == 0, "stages must keep the 1024-byte swizzle alignment");
  static_assert(256 + SETS * (N << GS) <= 512, "tensor memory");
  static_assert(SMEM <= 227 * 1024, "shared memory");
};
constexpr uint64_t kTcWaitNs = 200ull * 1000 * 1000;           // bound on any mbarrier wait

struct MatTcArgs {
  int rows, k, nst;            // weights [rows][k]; stages of a row
  int B;
  const float *bias;
  int relu;
  void *y;
  int y16;
  float *part;                 // [CTA][2][N][128]
  Header *hdr;
};

// columns c .. c+31 of this lane
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

template <int N, int GS>
__global__ void __launch_bounds__(MatTc<N, GS>::THREADS, 1)
    k_w4_matmul_tc(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_s,
                   const __grid_constant__ CUtensorMap map_x, MatTcArgs A) {
  using Lc = MatTc<N, GS>;
  constexpr int NS = Lc::NS, SETS = Lc::SETS, DC = N << GS, kLoad = 4 * SETS, kMma = 4 * SETS + 1;
  extern __shared__ unsigned char smem_raw[];
  __shared__ uint32_t s_last;
  unsigned char *smem = align_1024(smem_raw);
  uint64_t *full = reinterpret_cast<uint64_t *>(smem), *empty = full + NS;
  uint64_t *a_full = empty + NS, *d_full = a_full + 4;         // of the A operands
  uint32_t *tslot = reinterpret_cast<uint32_t *>(d_full + 4);
  float *red = reinterpret_cast<float *>(smem + Lc::BAR);      // [128][N + 1]
  unsigned char *stages = align_1024(smem + Lc::BAR + Lc::RED);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 8 + 2);                 // the warps that unpack it, and its halves' products
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&a_full[i], 128);
      mbar_init(&d_full[i], 1);
    }
    fence_mbar_init();
    prefetch_map(&map_w);
    prefetch_map(&map_s);
    prefetch_map(&map_x);
  }
  if (warp == kMma) {
    tmem_alloc(tslot, Lc::COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tslot;
  pdl_wait();
  pdl_trigger();

  const int tiles = ceil_div(A.rows, 128);
  const int64_t total = (int64_t)tiles * A.nst;
  const int G = (int)min((int64_t)gridDim.x, total);           // a stage at least for each CTA that takes part
  auto start_of = [&](int c) { return total * min(c, G) / G; };
  const int64_t u0 = start_of(blockIdx.x), u1 = start_of(blockIdx.x + 1);
  const int n = (int)(u1 - u0);                    // this CTA's stages
  int32_t *err = &A.hdr->err;

  if (warp == kLoad) {
    // ------------------------------------------------------------------ loads --
    if (lane == 0) {
      int tile = (int)(u0 / A.nst), st = (int)(u0 % A.nst);
      for (int i = 0; i < n; ++i) {
        const int sl = i % NS;
        if (i >= NS && !mbar_wait(&empty[sl], (uint32_t)((i / NS) - 1) & 1u, kTcWaitNs)) {
          flag_error(err, kErrTimeout);
          // what is on its way lands before the shared memory is given back
          for (int e = i - NS; e < i; ++e) mbar_wait(&full[e % NS], (uint32_t)(e / NS) & 1u, kTcWaitNs);
          break;
        }
        unsigned char *to = stages + (size_t)sl * Lc::STAGE;
        mbar_arrive_expect_tx(&full[sl], Lc::STAGE);
        tma_load_2d(to, &map_w, st * (kTcStageK / 2), tile * 128, &full[sl]);
        tma_load_2d(to + Lc::W, &map_s, (st * (4 << GS)) & ~15, tile * 128, &full[sl]);
#pragma unroll
        for (int q = 0; q < kTcStageK / 64; ++q)
          tma_load_2d(to + Lc::W + Lc::SC + q * (N * 128), &map_x, st * kTcStageK + 64 * q, 0, &full[sl]);
        if (++st == A.nst) {
          st = 0;
          ++tile;
        }
      }
    }
    __syncwarp();
  } else if (warp >= kMma) {
    // -------------------------------------------------------------------- MMA --
    constexpr uint32_t idesc = umma_idesc_f16(128, N, 0, 0);
    const int e = warp - kMma;                     // half of the stages
    const uint64_t dx = umma_desc(stages + Lc::W + Lc::SC + e * (2 * N * 128), 16, 1024, kSwz128);
    bool ok = true;
    for (int i = 0; i < n && ok; ++i) {
      const int sl = i % NS, op = 2 * (i & 1) + e; // A operand (and set, where there are four)
      const uint64_t d = dx + (uint64_t)(sl * (Lc::STAGE >> 4));
      const uint32_t a = tbase + op * 64, acc = tbase + 256 + (SETS == 4 ? op : e) * DC;
      ok = warp_wait(&full[sl], (uint32_t)(i / NS) & 1u, kTcWaitNs) && warp_wait(&a_full[op], (uint32_t)(i >> 1) & 1u, kTcWaitNs);
      if (!ok) break;
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < 8; ++k)                // 16 weights; a group's first product starts its accumulator
          umma_f16_ta(acc + (k >> (3 - GS)) * N, a + 8 * k, d + (uint64_t)(((k >> 2) * (N * 128) + (k & 3) * 32) >> 4), idesc,
                      (k & ((8 >> GS) - 1)) != 0);
        umma_commit(&d_full[op]);
        umma_commit(&empty[sl]);
      }
      __syncwarp();
    }
    if (!ok && lane == 0) flag_error(err, kErrTimeout);
  } else {
    // ----------------------------------------------------------------- unpack --
    const int set = warp >> 2, e = set & 1, par = set >> 1, row = tid & 127;
    const uint32_t tl = tbase + ((uint32_t)(32 * (warp & 3)) << 16);
    const uint32_t acc = tl + 256 + set * DC;
    float tot[N];
#pragma unroll
    for (int b = 0; b < N; ++b) tot[b] = 0.f;
    uint32_t sc[2] = {0, 0};                       // a block's scales, kept until its products are there
    int tile = (int)(u0 / A.nst), st = (int)(u0 % A.nst);      // of the stage settled next
    const int first_tile = tile;
    int begun = st;                                // first stage of the tile in this CTA
    int here = st;                                 // stage within its row tile, of the one unpacked
    bool ok = true;

    // the sets' sums of `tile` meet in set 0, whole or this CTA's part
    auto finish = [&](bool whole) {
      if (set != 0) {
        float *to = red + ((set - 1) * 128 + row) * (N + 1);
        named_sync(3, SETS * 128);                 // the buffer is free
#pragma unroll
        for (int b = 0; b < N; ++b) to[b] = tot[b];
        named_arrive(2, SETS * 128);
      } else {
        named_arrive(3, SETS * 128);
        named_sync(2, SETS * 128);
#pragma unroll
        for (int q = 0; q < SETS - 1; ++q)
#pragma unroll
          for (int b = 0; b < N; ++b) tot[b] += red[(q * 128 + row) * (N + 1) + b];
        bool mine = whole;
        if (!whole) {
          const int64_t t0 = (int64_t)tile * A.nst;
          const int c0 = (int)(((t0 + 1) * G - 1) / total), c1 = (int)(((t0 + A.nst) * G - 1) / total);
          float *to = A.part + ((int64_t)blockIdx.x * 2 + (tile != first_tile)) * (N * 128) + row;
#pragma unroll
          for (int b = 0; b < N; ++b)
            if (b < A.B) __stcg(to + b * 128, tot[b]);
          named_sync(4, 128);
          if (tid == 0) s_last = ticket_acq_rel(&A.hdr->tile_done[c0]);
          named_sync(4, 128);
          mine = s_last == (uint32_t)(c1 - c0);
          if (mine) {
#pragma unroll
            for (int b = 0; b < N; ++b) tot[b] = 0.f;
            for (int c = c0; c <= c1; ++c) {
              const float *from = A.part + ((int64_t)c * 2 + (start_of(c) / A.nst != tile)) * (N * 128) + row;
#pragma unroll
              for (int b = 0; b < N; ++b)
                if (b < A.B) tot[b] += __ldcg(from + b * 128);
            }
            if (tid == 0) A.hdr->tile_done[c0] = 0;            // zero again for the next call
          }
        }
        const int r = tile * 128 + row;
        if (mine && r < A.rows) {
          const float bias = A.bias ? __ldg(A.bias + r) : 0.f;
#pragma unroll
          for (int b = 0; b < N; ++b) {
            float v = tot[b] + bias;
            if (A.relu) v = v > 0.f ? v : (v != v ? v : 0.f);
            if (b >= A.B) continue;
            if (A.y16) static_cast<__half *>(A.y)[(int64_t)b * A.rows + r] = __float2half_rn(v);
            else static_cast<float *>(A.y)[(int64_t)b * A.rows + r] = v;
          }
        }
      }
#pragma unroll
      for (int b = 0; b < N; ++b) tot[b] = 0.f;
    };
    // the products of stage q, if they are this set's, into its sums; at a tile's end they meet
    auto settle = [&](int q) {
      if (SETS == 2 || (q & 1) == par) {
        const int op = 2 * (q & 1) + e;
        if (ok) ok = warp_wait(&d_full[op], (uint32_t)(q >> 1) & 1u, kTcWaitNs);
        if (ok) {
          tc_fence_after();
#pragma unroll
          for (int g = 0; g < (1 << GS); ++g) {
            const float s = half_of(sc[g >> 1], g & 1);
#pragma unroll
            for (int c = 0; c < N; c += 16) {
              if (c >= A.B) continue;
              float v[16];
              tmem_ld16w(acc + g * N + c, v);
#pragma unroll
              for (int b = 0; b < 16; ++b) tot[c + b] = fmaf(s, v[b], tot[c + b]);
            }
          }
          tc_fence_before();
        }
      }
      if (++st == A.nst || q == n - 1) {
        finish(begun == 0 && st == A.nst);
        if (st == A.nst) {
          st = 0;
          ++tile;
        }
        begun = st;
      }
    };
    int settled = 0;
    for (int i = 0; i < n; ++i) {
      if (SETS == 2 || (i & 1) == par) {
        const int sl = i % NS, op = 2 * (i & 1) + e;
        if (SETS == 4)
          while (settled < i) settle(settled++);   // frees the set's operand and accumulator
        if (ok) ok = warp_wait(&full[sl], (uint32_t)(i / NS) & 1u, kTcWaitNs);
        uint32_t next[2] = {0, 0};
        if (ok) {
          const unsigned char *w = stages + (size_t)sl * Lc::STAGE;
          // the 2 << GS bytes of this block in the 16-byte piece of its row
          const unsigned char *ps = w + Lc::W + row * 16 + (((here * (4 << GS)) & 15) + e * (2 << GS));
          if constexpr (GS == 0) {
            next[0] = *reinterpret_cast<const unsigned short *>(ps);
          } else {
            next[0] = *reinterpret_cast<const uint32_t *>(ps);
            if constexpr (GS == 2) next[1] = *reinterpret_cast<const uint32_t *>(ps + 4);
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {            // weights 64 h .. 64 h + 63: words j = 2h, 2h + 1
            uint32_t r[32];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
              const uint2 v = *reinterpret_cast<const uint2 *>(w + row * 128 + (((4 * e + t) ^ (row & 7)) << 4) + 8 * h);
              uint32_t p[4];
              unpack8<false>(v.x, p);
#pragma unroll
              for (int q = 0; q < 4; ++q) r[4 * t + q] = p[q];
              unpack8<false>(v.y, p);
#pragma unroll
              for (int q = 0; q < 4; ++q) r[16 + 4 * t + q] = p[q];
            }
            __syncwarp();
            tmem_st32(tl + op * 64 + 32 * h, r);
          }
          tmem_wait_st();
        }
        if (SETS == 2)
          while (settled < i) settle(settled++);   // its accumulator is the next one's too
        sc[0] = next[0];
        sc[1] = next[1];
        if (ok) {
          tc_fence_before();
          mbar_arrive(&a_full[op]);
          __syncwarp();
          if (lane == 0) mbar_arrive(&empty[sl]);
        }
      }
      if (++here == A.nst) here = 0;
    }
    while (settled < n) settle(settled++);
    if (!ok && lane == 0) flag_error(err, kErrTimeout);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMma) {
    tc_fence_after();
    tmem_dealloc(tbase, Lc::COLS);
  }
}

// two floats as an fp16 pair (lo first), an infinity as the largest finite value
__device__ __forceinline__ uint32_t half2_finite(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// ---------------------------------------------------- down projection --
// y[b][c] = sum_j a[j][b] s[j][c / group] (q[j][c] - 8): the neurons are the
// contracted dimension, so the scale, which changes with the neuron, joins the
// activation: v = a s in fp32, times a power of two, split into two fp16 parts,
// hi = fp16(v) and lo = fp16(v - hi): v to 2^-22, as the products' fp32 sums.  An
// infinite v has the largest fp16 as hi and itself as lo, so that it gives infinities
// of the weights' signs, and NaN where a weight is 0.
// The power of two keeps the parts in fp16's range.  Each warp has one for each
// token, so that a token's sums do not depend on the others': its largest |v| so
// far lies below 2^15, and what is 2^20 below it still has 16 bits.  When a
// larger one comes, the token's sums are rescaled (exactly) to the new power.
// D is 16 columns x 8 tokens.  Two neurons' words give one operand register by
// a byte permutation of the packed codes, before they are unpacked: a word's
// low half holds its even weights, its high half the odd ones.
struct DownArgs {
  const unsigned char *data;   // first down row
  int64_t stride;
  int n, d;
  const int32_t *idx, *count;
  const float *a;              // [positions][8 * NT]
  int B, R;                    // tokens, list splits
  float *part;                 // [R][B][d]
  float *y;
  Header *hdr;
};

// A warp's stage: 32 neurons' codes of one block of 128 columns, their scales
// and their activations.
constexpr int kDownTile = 32;
__host__ __device__ constexpr int down_stages(int NT) { return NT == 2 ? 3 : 4; }
__host__ __device__ constexpr int down_scale_bytes(int GS) { return GS == 2 ? 8 : 4; }
__host__ __device__ constexpr int down_stage_bytes(int NT, int GS) {
  return kDownTile * (64 + down_scale_bytes(GS) + 32 * NT);
}
__host__ __device__ constexpr size_t down_smem(int NT, int GS) {
  const size_t ring = (size_t)kDownWarps * down_stages(NT) * down_stage_bytes(NT, GS);
  const size_t red = (size_t)(kDownWarps / 2) * kDownCols * (8 * NT + 1) * 4;
  return ring > red ? ring : red;
}

// A CTA is 256 columns x a share of the list: four shares of neurons, two
// blocks of columns, a warp each with its own ring of cp.async stages.  The
// 64 bytes of codes of neurons 2i and 2i+1 share 128 bytes of shared memory,
// chunk (part, odd) at (2 part + odd) ^ x(i), so that the eight lanes of a
// 16-byte read touch every bank once.  Codes and scales do not depend on the
// gate/up kernel: the first stages are on their way while it still runs (it
// passed its own wait before this grid could start, so the list and the rows
// are complete).  With PC (up to four tokens) the two parts of an activation
// are two columns of one product instead of two products.
// What bounds it: for one token its chain of loads and the ticket (3440 neurons of
// d 8192, 14.5 MB: 17.9 us alone with cold rows, 26.3 us together with gate/up);
// for 16 tokens the splitting, unpacking and products share the issue slots with
// 16 warps an SM, all that the accumulators leave (13000 neurons of d 12288, 84 MB:
// 60 us alone, tensor pipe 37%).
template <int NT, int GS, bool PC>
__global__ void __launch_bounds__(kDownWarps * 32, NT <= 2 ? 2 : 1) k_w4_down(DownArgs A) {
  extern __shared__ __align__(128) unsigned char sm[];
  constexpr int NS = down_stages(NT), SB = down_stage_bytes(NT, GS), SCB = down_scale_bytes(GS);
  constexpr int kScales = kDownTile * 64, kActs = kScales + kDownTile * SCB;
  constexpr int RS = 8 * NT + 1;
  constexpr int P = PC ? 1 : 2;
  __shared__ uint32_t s_last;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  int total = A.n;
  if (A.count) total = max(0, min(A.n, ld_cg_i32(A.count)));   // out of range: flagged by the gate/up kernel
  const int ntile = ceil_div(total, kDownTile);
  // a warp takes two stages before the list is split further: a split costs its ticket
  const int R = max(1, min(A.R, ceil_div(ntile, kDownWarps)));
  const int cu = blockIdx.x / A.R, r = blockIdx.x % A.R;
  if (r >= R) return;
  const int kp = w4_kp(A.d);
  const int col0 = cu * kDownCols + (warp & 1) * kBlk;         // this warp's block
  const int sub = g & 3;                                       // word column of this lane's rows
  const uint32_t sel = (g >> 2) ? 0x7632u : 0x5410u;           // odd or even weights of two words

  unsigned char *ring = sm + (size_t)warp * NS * SB;
  const int first = r * (kDownWarps / 2) + (warp >> 1), step = R * (kDownWarps / 2);
  const int tiles = col0 < kp && first < ntile ? (ntile - first + step - 1) / step : 0;
  auto id_of = [&](int i) {                                    // this lane's neuron of stage i
    const int pos = (first + i * step) * kDownTile + lane;
    int id = -1;
    if (pos < total) id = A.idx ? ld_cg_i32(A.idx + pos) : pos;
    return (unsigned)id < (unsigned)A.n ? id : -1;
  };
  int id = tiles > 0 ? id_of(0) : -1;
  const unsigned char *codes = A.data + col0 / 2 + (lane & 3) * 16;
  // one block's scales; a single one comes with its neighbour (4 bytes at least)
  const unsigned char *scales = A.data + kp / 2 + (GS == 0 ? (col0 / kBlk) & ~1 : (col0 / kBlk) << GS) * 2;
  auto copy_rows = [&](int i, int slot) {                      // stage i's codes and scales
    if (i >= tiles) return;
    const int now = id;
    if (i + 1 < tiles) id = id_of(i + 1);
    unsigned char *to = ring + slot * SB;
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      const int row = h * 8 + (lane >> 2);
      const int nrn = __shfl_sync(0xffffffffu, now, row);
      const int x = ((row >> 1) & 1) | (row & 4);
      cp_async16(to + (row >> 1) * 128 + ((((lane & 3) * 2 + (row & 1)) ^ x) * 16), codes + (int64_t)max(nrn, 0) * A.stride,
                 nrn >= 0 ? 16u : 0u);
    }
    cp_async_small<SCB>(to + kScales + lane * SCB, scales + (int64_t)max(now, 0) * A.stride, now >= 0);
  };
  auto copy_act = [&](int i, int slot) {
    if (i < tiles) {
      unsigned char *to = ring + slot * SB + kActs;
      const int64_t pos0 = (int64_t)(first + i * step) * kDownTile;
#pragma unroll
      for (int q = 0; q < 2 * NT; ++q) {
        const int c = q * 32 + lane;
        const bool in = pos0 + c / (2 * NT) < total;
        cp_async16(to + c * 16, in ? A.a + pos0 * 8 * NT + c * 4 : A.a, in ? 16u : 0u);
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < NS - 1; ++i) copy_rows(i, i);
  pdl_wait();
  pdl_trigger();
#pragma unroll
  for (int i = 0; i < NS - 1; ++i) copy_act(i, i);

  float acc[8][NT][4];                             // [group of 32][half] x tokens
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[i][n][0] = acc[i][n][1] = acc[i][n][2] = acc[i][n][3] = 0.f;
  // PC: column g is part g & 1 of token g / 2
  const int act0 = PC ? g >> 1 : g;
  constexpr float kMostUp = 1.7014118e38f;         // 2^127
  float up[NT];                                    // the power of two of column g of each token tile
#pragma unroll
  for (int n = 0; n < NT; ++n) up[n] = kMostUp;
  const int hi0 = GS == 0 ? (col0 / kBlk) & 1 : 0;

  int slot = 0;
  for (int i = 0; i < tiles; ++i) {
    cp_async_wait<NS - 2>();
    __syncwarp();
    copy_rows(i + NS - 1, slot == 0 ? NS - 1 : slot - 1);      // into the slot that the last step has read
    copy_act(i + NS - 1, slot == 0 ? NS - 1 : slot - 1);
    const unsigned char *st = ring + slot * SB;
    slot = slot + 1 == NS ? 0 : slot + 1;
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {               // 16 neurons
      uint4 c[4];
      uint32_t sc[4][GS == 2 ? 2 : 1];
      float av[4][NT];
#pragma unroll
      for (int q = 0; q < 4; ++q) {                // this lane's: 2t, 2t+1, 2t+8, 2t+9
        const int row = 16 * kk + 2 * t + (q & 1) + 8 * (q >> 1);
        const int x = (t & 1) | ((t & 2) << 1);
        c[q] = *reinterpret_cast<const uint4 *>(st + (row >> 1) * 128 + (((sub * 2 + (q & 1)) ^ x) * 16));
#pragma unroll
        for (int w = 0; w < (GS == 2 ? 2 : 1); ++w)
          sc[q][w] = *reinterpret_cast<const uint32_t *>(st + kScales + row * SCB + 4 * w);
#pragma unroll
        for (int n = 0; n < NT; ++n) av[q][n] = *reinterpret_cast<const float *>(st + kActs + ((row * NT + n) * 8 + act0) * 4);
      }
      uint32_t bp[NT][P][2];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (j % (4 >> GS) == 0) {                  // a new group of columns: a * s
          float v[NT][4], most = 0.f;
          auto values = [&](int n) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const float s = half_of(sc[q][GS == 2 ? j >> 1 : 0], GS == 2 ? j & 1 : GS == 1 ? j >> 1 : hi0);
              v[n][q] = av[q][n] * s * up[n];      // (a s) first: s times the power alone can overflow
            }
          };
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            values(n);
#pragma unroll
            for (int q = 0; q < 4; ++q) most = fmaxf(most, fabsf(v[n][q]));
          }
          if (__any_sync(0xffffffffu, most >= 32768.f)) {      // past the parts' range: smaller powers
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              uint32_t top = 0;                    // the column's largest finite |a s|
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const float s = half_of(sc[q][GS == 2 ? j >> 1 : 0], GS == 2 ? j & 1 : GS == 1 ? j >> 1 : hi0);
                const uint32_t u = __float_as_uint(av[q][n] * s) & 0x7fffffffu;
                if (u < 0x7f800000u) top = max(top, u);        // an infinity or NaN is its token's own affair
              }
              top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
              top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
              float f = 1.f;
              if (__uint_as_float(top) * up[n] >= 32768.f) {   // 2^11 <= the largest < 2^12 from here on
                const float now = __uint_as_float((uint32_t)max(127 + 11 - (int)(top >> 23) + 127, 1) << 23);
                f = fmaxf(now / up[n], 1.17549435e-38f);       // never 0, which an infinite sum would turn into NaN
                up[n] = now;
              }
              const float f0 = __shfl_sync(0xffffffffu, f, 8 * t), f1 = __shfl_sync(0xffffffffu, f, 8 * t + 4);
#pragma unroll
              for (int e = 0; e < 8; ++e) {        // columns 2t and 2t + 1
                acc[e][n][0] *= f0;
                acc[e][n][1] *= f1;
                acc[e][n][2] *= f0;
                acc[e][n][3] *= f1;
              }
              values(n);
            }
          }
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const float v0 = v[n][2 * q], v1 = v[n][2 * q + 1];
              const uint32_t hw = half2_finite(v0, v1);
              const float2 back = __half22float2(*reinterpret_cast<const __half2 *>(&hw));
              const __half2 lo = __floats2half2_rn(v0 - back.x, v1 - back.y);
              const uint32_t lw = *reinterpret_cast<const uint32_t *>(&lo);
              if constexpr (PC) {
                bp[n][0][q] = g & 1 ? lw : hw;
              } else {
                bp[n][0][q] = hw;
                bp[n][1][q] = lw;
              }
            }
        }
        const uint32_t w[4] = {j == 0 ? c[0].x : j == 1 ? c[0].y : j == 2 ? c[0].z : c[0].w,
                               j == 0 ? c[1].x : j == 1 ? c[1].y : j == 2 ? c[1].z : c[1].w,
                               j == 0 ? c[2].x : j == 1 ? c[2].y : j == 2 ? c[2].z : c[2].w,
                               j == 0 ? c[3].x : j == 1 ? c[3].y : j == 2 ? c[3].z : c[3].w};
        uint32_t lo[4], hi[4];
        unpack8<false>(__byte_perm(w[0], w[1], sel), lo);      // [p] = weight 2p + (g >> 2) of neurons 2t, 2t+1
        unpack8<false>(__byte_perm(w[2], w[3], sel), hi);      // of neurons 2t+8, 2t+9
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int q = 0; q < P; ++q) {
            mma16816<false>(acc[2 * j][n], lo[0], lo[1], hi[0], hi[1], bp[n][q][0], bp[n][q][1]);
            mma16816<false>(acc[2 * j + 1][n], lo[2], lo[3], hi[2], hi[3], bp[n][q][0], bp[n][q][1]);
          }
      }
    }
  }
  // the four shares of a column, added in order
  cp_async_wait<0>();
  __syncthreads();
  float *red = reinterpret_cast<float *>(sm);                  // [share][256 columns][8 * NT + 1]
  float down[NT][2];                               // of columns 2t and 2t + 1
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    down[n][0] = 1.f / __shfl_sync(0xffffffffu, up[n], 8 * t);
    down[n][1] = 1.f / __shfl_sync(0xffffffffu, up[n], 8 * t + 4);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        // row g of half h is weight 2p + (g >> 2) of word 4j + (g & 3), p = 2h (+1 for row g + 8)
        const int p = 2 * (i & 1) + (e >> 1);
        const int col = (warp & 1) * kBlk + (i >> 1) * 32 + sub * 8 + 2 * p + (g >> 2);
        red[((warp >> 1) * kDownCols + col) * RS + 8 * n + 2 * t + (e & 1)] = acc[i][n][e] * down[n][e & 1];
      }
  __syncthreads();
  for (int i = threadIdx.x; i < A.B * kDownCols; i += blockDim.x) {
    const int b = i / kDownCols, c = cu * kDownCols + i % kDownCols;
    if (c >= A.d) continue;
    float v = 0.f;
#pragma unroll
    for (int q = 0; q < kDownWarps / 2; ++q) {
      const float *from = red + (q * kDownCols + i % kDownCols) * RS;
      v += PC ? from[2 * b + 1] + from[2 * b] : from[b];
    }
    if (R == 1) A.y[(int64_t)b * A.d + c] = v;
    else __stcg(A.part + ((int64_t)r * A.B + b) * A.d + c, v);
  }
  if (R == 1) return;
  __syncthreads();
  if (threadIdx.x == 0) s_last = ticket_acq_rel(&A.hdr->tile_done[cu]);
  __syncthreads();
  if (s_last != (uint32_t)(R - 1)) return;
  // the list's parts in order; a thread has four columns of four tokens at a
  // time, 16 loads in flight (one value at a time: 36 us for 32 tokens x 18 parts)
  const int c4 = cu * kDownCols + 4 * (threadIdx.x & 63);
  if (c4 < A.d) {
    for (int k0 = threadIdx.x >> 6; k0 < A.B; k0 += 16) {
      float4 v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int q = 0; q < R; ++q)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (k0 + 4 * k < A.B) {
            const float4 u = __ldcg(reinterpret_cast<const float4 *>(A.part + ((int64_t)q * A.B + k0 + 4 * k) * A.d + c4));
            v[k].x += u.x; v[k].y += u.y; v[k].z += u.z; v[k].w += u.w;
          }
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (k0 + 4 * k < A.B) {
          float *to = A.y + (int64_t)(k0 + 4 * k) * A.d + c4;
          to[0] = v[k].x; to[1] = v[k].y; to[2] = v[k].z; to[3] = v[k].w;
        }
    }
  }
  if (threadIdx.x == 0) A.hdr->tile_done[cu] = 0;
}

// ------------------------------------------------------------------ host --
asf_status check_w4(const asf_w4_matrix *m) {
  if (!m || !m->data) return ASF_ERR_INVALID_ARG;
  if (m->group != 32 && m->group != 64 && m->group != 128) return ASF_ERR_UNSUPPORTED;
  if (m->rows <= 0 || m->k <= 0) return ASF_ERR_INVALID_ARG;
  if (m->k % 8 || m->row_stride % 16 || !al16(m->data)) return ASF_ERR_MISALIGNED;
  if (m->k > ASF_W4_MAX_K || m->rows > ASF_W4_MAX_ROWS) return ASF_ERR_UNSUPPORTED;
  if (m->row_stride < w4_row_bytes(m->k, m->group)) return ASF_ERR_INVALID_ARG;
  return ASF_OK;
}
// whether contiguous [rows][k] values share memory with the matrix: warps of a row read and write at their own pace
bool rows_overlap(const asf_w4_matrix *m, const void *dense, asf_dtype dtype) {
  return overlap(dense, (size_t)m->rows * m->k * (dtype == ASF_F16 ? 2 : 4), m->data,
                 (size_t)(m->rows - 1) * m->row_stride + w4_row_bytes(m->k, m->group));
}
// CTAs of the row-wise kernels (rows_of_cta)
unsigned row_ctas(const asf_w4_matrix *m) {
  const int nsb = ceil_div(m->k, kSuper), per = nsb > 4 ? 1 : nsb > 2 ? 2 : nsb > 1 ? 4 : 8;
  return (unsigned)ceil_div(m->rows, per);
}
int ffn_mats(const asf_w4_ffn *f) { return f->act == ASF_ACT_REGLU ? 3 : 2; }
asf_status check_w4_ffn(const asf_w4_ffn *f) {
  if (!f || !f->data || !f->bias) return ASF_ERR_INVALID_ARG;
  if (f->act != ASF_ACT_RELU && f->act != ASF_ACT_REGLU) return ASF_ERR_UNSUPPORTED;
  if (f->group != 32 && f->group != 64 && f->group != 128) return ASF_ERR_UNSUPPORTED;
  if (f->d <= 0 || f->n <= 0) return ASF_ERR_INVALID_ARG;
  if (f->d % 8 || f->neuron_stride % 16 || !al16(f->data) || !al4(f->bias)) return ASF_ERR_MISALIGNED;
  if (f->d > ASF_W4_MAX_K || f->n > ASF_W4_MAX_ROWS) return ASF_ERR_UNSUPPORTED;
  if (f->neuron_stride < ffn_mats(f) * w4_row_bytes(f->d, f->group)) return ASF_ERR_INVALID_ARG;
  return ASF_OK;
}

int nt_of(int B) { return B <= 8 ? 1 : B <= 16 ? 2 : 4; }
int gs_of(int group) { return group == 32 ? 2 : group == 64 ? 1 : 0; }
int dot_ctas() { return sm_count(); }
size_t x_bytes(int B, int parts, int superblocks) { return ((size_t)B * parts + 1) * ((size_t)superblocks * kSuper * 2 + 64); }
// superblocks of k whose x fits a CTA beside the rings
int dot_most(int k, int group, int B, int parts) {
  const int nsb = ceil_div(w4_kp(k), kSuper);
  const size_t room = kDotSmem - dot_ring_bytes(nt_of(B), gs_of(group));
  int n = nsb;
  while (n > 1 && x_bytes(B, parts, n) > room) --n;
  return n;
}
// partial sums of a split k (the most that dot_per makes of it)
size_t dot_part_bytes(int tiles, int k, int group, int B) {
  const int nsb = ceil_div(w4_kp(k), kSuper);
  const size_t forced = (size_t)tiles * ceil_div(nsb, dot_most(k, group, B, 3));
  // (the tensor-memory product needs two parts of 16 or 32 x 512 bytes a CTA: less)
  return r256(std::max<size_t>((size_t)kPartsPerCta * dot_ctas(), 2 * forced) * nt_of(B) * 512);
}
int down_units(int d) { return ceil_div(w4_kp(d), kDownCols); }
int down_w4_splits(int d, int B) {
  const int per_sm = nt_of(B) <= 2 ? 2 : 1;
  return std::max(1, sm_count() * per_sm / down_units(d));
}
size_t ffn_w4_scratch(const asf_w4_ffn *f, int B) {
  const int tiles = ceil_div(f->n, f->act == ASF_ACT_REGLU ? 8 : 16);
  return r256((size_t)f->n * nt_of(B) * 32) + dot_part_bytes(tiles, f->d, f->group, B) +
         r256((size_t)down_w4_splits(f->d, B) * B * f->d * 4);
}

template <bool BF, int NT, int MODE>
cudaError_t run_dot_nt(const DotArgs &a, int group, cudaStream_t st) {
  const size_t smem = dot_ring_bytes(NT, gs_of(group)) + x_bytes(a.B, BF ? 3 : 1, a.most);
  const dim3 grid(dot_ctas()), block(kDotWarps * 32);
  return group == 128  ? launch(k_w4_dot<BF, NT, 0, MODE>, grid, block, smem, st, a)
         : group == 64 ? launch(k_w4_dot<BF, NT, 1, MODE>, grid, block, smem, st, a)
                       : launch(k_w4_dot<BF, NT, 2, MODE>, grid, block, smem, st, a);
}
template <int MODE>
cudaError_t run_dot(DotArgs a, int group, asf_dtype xdtype, cudaStream_t st) {
  const bool bf = xdtype == ASF_F32;
  a.most = dot_most(a.k, group, a.B, bf ? 3 : 1);
  switch (nt_of(a.B)) {
    case 1: return bf ? run_dot_nt<true, 1, MODE>(a, group, st) : run_dot_nt<false, 1, MODE>(a, group, st);
    case 2: return bf ? run_dot_nt<true, 2, MODE>(a, group, st) : run_dot_nt<false, 2, MODE>(a, group, st);
    default: return bf ? run_dot_nt<true, 4, MODE>(a, group, st) : run_dot_nt<false, 4, MODE>(a, group, st);
  }
}

// Byte map of `rows` rows `stride` apart, in boxes of cols x box_rows bytes.
bool byte_map(CUtensorMap *tm, const void *base, int64_t width, int64_t rows, int64_t stride, int cols, int box_rows,
              CUtensorMapSwizzle swz) {
  TmapEncodeFn enc = tmap_encoder();
  if (!enc) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)width, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)stride};
  const cuuint32_t box[2] = {(cuuint32_t)cols, (cuuint32_t)box_rows}, one[2] = {1, 1};
  return enc(tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box, one,
             CU_TENSOR_MAP_INTERLEAVE_NONE, swz, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
bool x_map(CUtensorMap *tm, const void *x, int k, int B, int box_rows) {
  TmapEncodeFn enc = tmap_encoder();
  if (!enc) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)k, (cuuint64_t)B}, strides[1] = {(cuuint64_t)k * 2};
  const cuuint32_t box[2] = {64, (cuuint32_t)box_rows}, one[2] = {1, 1};
  return enc(tm, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, const_cast<void *>(x), dims, strides, box, one,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int N>
cudaError_t run_matmul_tc_n(const asf_w4_matrix *m, const CUtensorMap &w, const CUtensorMap &s, const CUtensorMap &x,
                            const MatTcArgs &a, cudaStream_t st) {
  const dim3 grid(dot_ctas());
  return m->group == 128 ? launch(k_w4_matmul_tc<N, 0>, grid, dim3(MatTc<N, 0>::THREADS), MatTc<N, 0>::SMEM, st, w, s, x, a)
         : m->group == 64
             ? launch(k_w4_matmul_tc<N, 1>, grid, dim3(MatTc<N, 1>::THREADS), MatTc<N, 1>::SMEM, st, w, s, x, a)
             : launch(k_w4_matmul_tc<N, 2>, grid, dim3(MatTc<N, 2>::THREADS), MatTc<N, 2>::SMEM, st, w, s, x, a);
}
// false: no maps for these operands
bool run_matmul_tc(const asf_w4_matrix *m, const void *x, MatTcArgs a, cudaStream_t st, cudaError_t &e) {
  CUtensorMap mw, ms, mx;
  const int N = a.B <= 16 ? 16 : 32, half = w4_kp(m->k) / 2;
  a.nst = ceil_div(w4_kp(m->k), kTcStageK);
  if (!byte_map(&mw, m->data, half, m->rows, m->row_stride, kTcStageK / 2, 128, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !byte_map(&ms, static_cast<const unsigned char *>(m->data) + half, w4_scale_bytes(m->k, m->group), m->rows,
                m->row_stride, 16, 128, CU_TENSOR_MAP_SWIZZLE_NONE) ||
      !x_map(&mx, x, m->k, a.B, N))
    return false;
  e = N == 16 ? run_matmul_tc_n<16>(m, mw, ms, mx, a, st) : run_matmul_tc_n<32>(m, mw, ms, mx, a, st);
  return true;
}
template <int GS>
cudaError_t run_down(const DownArgs &a, cudaStream_t st) {
  const dim3 grid(down_units(a.d) * a.R), block(kDownWarps * 32);
  if (a.B <= 4) return launch(k_w4_down<1, GS, true>, grid, block, down_smem(1, GS), st, a);
  switch (nt_of(a.B)) {
    case 1: return launch(k_w4_down<1, GS, false>, grid, block, down_smem(1, GS), st, a);
    case 2: return launch(k_w4_down<2, GS, false>, grid, block, down_smem(2, GS), st, a);
    default: return launch(k_w4_down<4, GS, false>, grid, block, down_smem(4, GS), st, a);
  }
}

}  // namespace

extern "C" {

int64_t asf_w4_row_bytes(int32_t k, int32_t group) {
  if (k <= 0 || k % 8 || k > ASF_W4_MAX_K || (group != 32 && group != 64 && group != 128)) return 0;
  return w4_row_bytes(k, group);
}

size_t asf_w4_workspace_bytes(const asf_w4_matrix *mat, const asf_w4_ffn *ffn, int32_t max_batch) {
  if (max_batch < 1 || max_batch > ASF_MAX_BATCH || (!mat && !ffn)) return 0;
  if (mat && check_w4(mat) != ASF_OK) return 0;
  if (ffn && check_w4_ffn(ffn) != ASF_OK) return 0;
  size_t need = 0;
  for (int b : {1, 8, 16, 32}) {                   // the need grows with each of the token tiles, and within one
    const int B = std::min<int>(b, max_batch);
    if (mat) need = std::max(need, dot_part_bytes(ceil_div(mat->rows, 16), mat->k, mat->group, B));
    if (ffn) need = std::max(need, ffn_w4_scratch(ffn, B));
  }
  return kHeaderBytes + need;
}

asf_status asf_w4_quantize(const void *src, asf_dtype dtype, const asf_w4_matrix *mat, asf_stream_t stream) {
  asf_status s = check_w4(mat);
  if (s != ASF_OK) return s;
  if (!src) return ASF_ERR_INVALID_ARG;
  if (dtype != ASF_F16 && dtype != ASF_F32) return ASF_ERR_UNSUPPORTED;
  if (!al16(src)) return ASF_ERR_MISALIGNED;
  if (rows_overlap(mat, src, dtype)) return ASF_ERR_INVALID_ARG;
  const dim3 grid(row_ctas(mat)), block(256);
  unsigned char *dst = static_cast<unsigned char *>(const_cast<void *>(mat->data));
  cudaStream_t st = (cudaStream_t)stream;
  return cuda_status(dtype == ASF_F16
                         ? launch(k_w4_quantize<__half>, grid, block, 0, st, static_cast<const __half *>(src), mat->rows,
                                  mat->k, mat->group, dst, mat->row_stride)
                         : launch(k_w4_quantize<float>, grid, block, 0, st, static_cast<const float *>(src), mat->rows,
                                  mat->k, mat->group, dst, mat->row_stride));
}

asf_status asf_w4_dequantize(const asf_w4_matrix *mat, void *dst, asf_dtype dtype, asf_stream_t stream) {
  asf_status s = check_w4(mat);
  if (s != ASF_OK) return s;
  if (!dst) return ASF_ERR_INVALID_ARG;
  if (dtype != ASF_F16 && dtype != ASF_F32) return ASF_ERR_UNSUPPORTED;
  if (!al16(dst)) return ASF_ERR_MISALIGNED;
  if (rows_overlap(mat, dst, dtype)) return ASF_ERR_INVALID_ARG;
  const dim3 grid(row_ctas(mat)), block(256);
  const unsigned char *src = static_cast<const unsigned char *>(mat->data);
  cudaStream_t st = (cudaStream_t)stream;
  return cuda_status(dtype == ASF_F16 ? launch(k_w4_dequantize<__half>, grid, block, 0, st, src, mat->row_stride,
                                               mat->rows, mat->k, mat->group, static_cast<__half *>(dst))
                                      : launch(k_w4_dequantize<float>, grid, block, 0, st, src, mat->row_stride,
                                               mat->rows, mat->k, mat->group, static_cast<float *>(dst)));
}

asf_status asf_w4_matmul(const asf_w4_matrix *mat, const void *x, asf_dtype xdtype, int32_t B, const float *bias,
                         int32_t relu, void *y, asf_dtype ydtype, void *ws, size_t ws_bytes, asf_stream_t stream) {
  asf_status s = check_w4(mat);
  if (s != ASF_OK) return s;
  if (!x || !y || B < 1 || B > ASF_MAX_BATCH || (relu != 0 && relu != 1)) return ASF_ERR_INVALID_ARG;
  if (xdtype != ASF_F16 && xdtype != ASF_F32) return ASF_ERR_UNSUPPORTED;
  if (ydtype != ASF_F16 && ydtype != ASF_F32) return ASF_ERR_UNSUPPORTED;
  if (!al16(x) || (reinterpret_cast<uintptr_t>(y) & (ydtype == ASF_F16 ? 1u : 3u)) || !al4(bias)) return ASF_ERR_MISALIGNED;
  s = check_ws(ws, ws_bytes, kHeaderBytes + dot_part_bytes(ceil_div(mat->rows, 16), mat->k, mat->group, B));
  if (s != ASF_OK) return s;
  if (overlap(x, (size_t)B * mat->k * (xdtype == ASF_F16 ? 2 : 4), y, (size_t)B * mat->rows * (ydtype == ASF_F16 ? 2 : 4)))
    return ASF_ERR_INVALID_ARG;
  // A part of k whose x fits a CTA is a CTA's at least: never so on a whole B200.
  if (ceil_div(ceil_div(mat->k, kSuper), dot_most(mat->k, mat->group, B, xdtype == ASF_F32 ? 3 : 1)) > dot_ctas())
    return ASF_ERR_UNSUPPORTED;
  // k_w4_matmul_tc from so many stages (of 128 rows x 256 weights) a CTA on: it
  // costs 4 us more to start and end, and less per stage, the more so the more
  // tokens share the unpacked weights.  us of k_w4_dot and of it, one token:
  // 8192 x 8192 (14 stages) 13.7 and 16.9, 28672 x 8192 (48) 41.5 and 37.6;
  // 16 tokens: 11008 x 4096 (9) 13.9 and 15.2, 8192 x 8192 18.3 and 19.3, 28672 x
  // 8192 56 and 39; 32 tokens: 8192 x 4096 (7) 16.5 and 19.4, 11008 x 4096 21.8
  // and 19.9, 28672 x 8192 93 and 47.
  const int64_t stages = (int64_t)ceil_div(mat->rows, 128) * ceil_div(w4_kp(mat->k), kTcStageK);
  if (xdtype == ASF_F16 && stages >= (int64_t)(B <= 8 ? 28 : B <= 16 ? 16 : 10) * dot_ctas()) {
    MatTcArgs t{};
    t.rows = mat->rows;
    t.k = mat->k;
    t.B = B;
    t.bias = bias;
    t.relu = relu;
    t.y = y;
    t.y16 = ydtype == ASF_F16;
    t.part = reinterpret_cast<float *>(static_cast<unsigned char *>(ws) + kHeaderBytes);
    t.hdr = static_cast<Header *>(ws);
    cudaError_t e = cudaSuccess;
    if (run_matmul_tc(mat, x, t, (cudaStream_t)stream, e)) return cuda_status(e);
  }
  DotArgs a{};
  a.data = static_cast<const unsigned char *>(mat->data);
  a.stride = mat->row_stride;
  a.rows = mat->rows;
  a.k = mat->k;
  a.x = x;
  a.B = B;
  a.bias = bias;
  a.relu = relu;
  a.y = static_cast<float *>(y);
  a.y16 = ydtype == ASF_F16;
  a.part = reinterpret_cast<float *>(static_cast<unsigned char *>(ws) + kHeaderBytes);
  a.hdr = static_cast<Header *>(ws);
  return cuda_status(run_dot<kDense>(a, mat->group, xdtype, (cudaStream_t)stream));
}

asf_status asf_w4_sparse_ffn(const asf_w4_ffn *f, const void *x, asf_dtype xdtype, int32_t B, const int32_t *idx,
                             const int32_t *count, float *y, void *ws, size_t ws_bytes, asf_stream_t stream) {
  asf_status s = check_w4_ffn(f);
  if (s != ASF_OK) return s;
  if (!x || !y || (!idx != !count) || B < 1 || B > ASF_MAX_BATCH) return ASF_ERR_INVALID_ARG;
  if (xdtype != ASF_F16 && xdtype != ASF_F32) return ASF_ERR_UNSUPPORTED;
  if (!al16(x) || !al4(y) || !al4(idx) || !al4(count)) return ASF_ERR_MISALIGNED;
  s = check_ws(ws, ws_bytes, kHeaderBytes + ffn_w4_scratch(f, B));
  if (s != ASF_OK) return s;
  if (ceil_div(ceil_div(f->d, kSuper), dot_most(f->d, f->group, B, xdtype == ASF_F32 ? 3 : 1)) > dot_ctas())
    return ASF_ERR_UNSUPPORTED;
  const bool gated = f->act == ASF_ACT_REGLU;
  unsigned char *base = static_cast<unsigned char *>(ws) + kHeaderBytes;
  const int64_t rb = w4_row_bytes(f->d, f->group);
  DotArgs a{};
  a.data = static_cast<const unsigned char *>(f->data);
  a.stride = f->neuron_stride;
  a.up = rb;
  a.rows = f->n;
  a.k = f->d;
  a.x = x;
  a.B = B;
  a.bias = f->bias;
  a.idx = idx;
  a.count = count;
  a.y = reinterpret_cast<float *>(base);
  base += r256((size_t)f->n * nt_of(B) * 32);
  a.part = reinterpret_cast<float *>(base);
  base += dot_part_bytes(ceil_div(f->n, gated ? 8 : 16), f->d, f->group, B);
  a.hdr = static_cast<Header *>(ws);
  cudaStream_t st = (cudaStream_t)stream;
  const cudaError_t e = gated ? run_dot<kListGated>(a, f->group, xdtype, st) : run_dot<kListUp>(a, f->group, xdtype, st);
  if (e != cudaSuccess) return ASF_ERR_CUDA;
  DownArgs w{};
  w.data = a.data + (ffn_mats(f) - 1) * rb;
  w.stride = f->neuron_stride;
  w.n = f->n;
  w.d = f->d;
  w.idx = idx;
  w.count = count;
  w.a = a.y;
  w.B = B;
  w.R = down_w4_splits(f->d, B);
  w.part = reinterpret_cast<float *>(base);
  w.y = y;
  w.hdr = a.hdr;
  return cuda_status(f->group == 128  ? run_down<0>(w, st)
                     : f->group == 64 ? run_down<1>(w, st)
                                      : run_down<2>(w, st));
}

}  // extern "C"
