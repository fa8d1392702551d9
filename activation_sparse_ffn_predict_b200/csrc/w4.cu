// 4-bit weights with group scales: the format, the dense product and the
// sparse FFN over 4-bit rows (include/asffn.h, "4-bit weights").
//
//   asf_w4_quantize / asf_w4_dequantize   k_w4_quantize, k_w4_dequantize
//   asf_w4_matmul       y = act(W x + b)  k_w4_dot
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
// (8 + 8 + 8 mantissa bits, by truncation), multiplied in three instructions
// into the same accumulators.
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
constexpr size_t kDotSmem = 200 * 1024;
constexpr float kFp16Max = 65504.f;

__host__ __device__ inline int ceil_div(int a, int b) { return (a + b - 1) / b; }
__host__ __device__ inline int w4_kp(int k) { return ceil_div(k, kBlk) * kBlk; }
__host__ __device__ inline int w4_scale_bytes(int k, int group) {
  return ceil_div(ceil_div(w4_kp(k), kSuper) * (kSuper / group) * 2, 16) * 16;
}
inline int64_t w4_row_bytes(int k, int group) { return (int64_t)w4_kp(k) / 2 + w4_scale_bytes(k, group); }

// ------------------------------------------------------------- quantize --
// One warp per superblock of 512 weights of a row, 8 weights a lane at a
// time: the group maximum over group / 8 neighbouring lanes, one division per
// weight (IEEE, so that codes are the formula's own), one word of codes.
template <typename T>
__global__ void __launch_bounds__(256)
k_w4_quantize(const T *__restrict__ src, int rows, int k, int group, unsigned char *__restrict__ dst, int64_t stride) {
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int nsb = ceil_div(k, kSuper), kp = w4_kp(k);
  const int64_t unit = (int64_t)blockIdx.x * (blockDim.x / 32) + (threadIdx.x >> 5);
  if (unit >= (int64_t)rows * nsb) return;
  const int64_t row = unit / nsb;
  const int sb = (int)(unit % nsb);
  const T *in = src + row * k;
  unsigned char *out = dst + row * stride;
  const int per = group / 8;                       // lanes of a group
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int i0 = sb * kSuper + h * 256 + lane * 8;
    float v[8] = {};
    if (i0 < k) {                                  // k is a multiple of 8
      if constexpr (sizeof(T) == 2) {
        const uint4 u = *reinterpret_cast<const uint4 *>(in + i0);
        Vec<__half>::to_float(u, v);
      } else {
        const float4 a = *reinterpret_cast<const float4 *>(in + i0), b = *reinterpret_cast<const float4 *>(in + i0 + 4);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
      }
    }
    // NaN counts as infinite: the maximum of fmaxf would drop it
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, v[i] != v[i] ? INFINITY : fabsf(v[i]));
    for (int o = 1; o < per; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const __half sh = __float2half_rn(__fdiv_rn(m, 7.f));
    const float s = __half2float(sh);
    const bool good = s <= kFp16Max;               // a group that fp16 scales cannot hold reads back as NaN
    uint32_t word = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float c = good && s > 0.f ? rintf(__fdiv_rn(v[i], s)) : 0.f;
      c = fminf(fmaxf(c, -8.f), 7.f);
      word |= (uint32_t)((int)c + 8) << (16 * (i & 1) + 4 * (i >> 1));
    }
    const int wi = (i0 % kBlk) / 8;                // word j*4 + t of the block is stored at t*4 + j
    if (i0 < kp) *reinterpret_cast<uint32_t *>(out + (i0 / kBlk) * 64 + ((wi & 3) * 4 + (wi >> 2)) * 4) = word;
    if (lane % per == 0) {                         // past kp the maximum is 0: zero padding
      __half w = good ? sh : __ushort_as_half((unsigned short)0x7fff);
      *reinterpret_cast<__half *>(out + kp / 2 + (i0 / group) * 2) = w;
    }
  }
  const int used = nsb * (kSuper / group) * 2;     // rest of the scale area, up to 16 bytes
  if (sb == nsb - 1 && lane * 2 < w4_scale_bytes(k, group) - used)
    *reinterpret_cast<uint16_t *>(out + kp / 2 + used + lane * 2) = 0;
}

template <typename T>
__global__ void __launch_bounds__(256)
k_w4_dequantize(const unsigned char *__restrict__ src, int64_t stride, int rows, int k, int group, T *__restrict__ dst) {
  pdl_wait();
  const int words = k / 8;
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= (int64_t)rows * words) return;
  const int64_t row = i / words;
  const int at = (int)(i % words) * 8;
  const unsigned char *in = src + row * stride;
  const int wi = (at % kBlk) / 8;
  const uint32_t w = *reinterpret_cast<const uint32_t *>(in + (at / kBlk) * 64 + ((wi & 3) * 4 + (wi >> 2)) * 4);
  const float s = __half2float(*reinterpret_cast<const __half *>(in + w4_kp(k) / 2 + (at / group) * 2));
  float v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = (float)((int)((w >> (16 * (e & 1) + 4 * (e >> 1))) & 15u) - 8) * s;
  T *out = dst + row * k + at;
  if constexpr (sizeof(T) == 2) {
    uint4 u;
    uint32_t *p = &u.x;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const __half2 h2 = __floats2half2_rn(v[2 * q], v[2 * q + 1]);
      p[q] = *reinterpret_cast<const uint32_t *>(&h2);
    }
    *reinterpret_cast<uint4 *>(out) = u;
  } else {
    *reinterpret_cast<float4 *>(out) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4 *>(out + 4) = make_float4(v[4], v[5], v[6], v[7]);
  }
}

// ---------------------------------------------------- codes to operands --
// The four pairs (weights 2p, 2p+1 of a word) as fp16 or bf16 whole numbers
// -8..7.  Or-ing a nibble into the mantissa of 1024 (fp16: pair 0, and pair 1
// as 1024 + 16 q) or of 128 (bf16) is exact, and so is what follows.
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

__device__ __forceinline__ float trunc_bf16(float v) { return __uint_as_float(__float_as_uint(v) & 0xffff0000u); }
// the upper halves of two floats as one pair (lo first)
__device__ __forceinline__ uint32_t upper2(float lo, float hi) {
  return __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x7632);
}

// ------------------------------------------------------- row products --
// Splits S of k (in superblocks) such that tiles * S fills the warps that keep
// enough loads in flight (8 an SM); smin splits at least, so that a CTA's part
// of x fits its shared memory.  Even shares.
__host__ __device__ inline int w4_splits(int tiles, int nsb, int smin, int ctas) {
  int S = ceil_div(8 * ctas, tiles > 0 ? tiles : 1);
  if (S < smin) S = smin;
  if (S > nsb) S = nsb;
  if (S > ctas) S = ctas;
  return ceil_div(nsb, ceil_div(nsb, S));
}

struct DotArgs {
  const unsigned char *data;   // first row (gate rows of the list form)
  int64_t stride;              // bytes from row to row (neuron to neuron)
  int64_t up;                  // bytes from a neuron's gate row to its up row (REGLU), else 0
  int rows;                    // rows, or neurons the list may name
  int k, group;
  const void *x;
  int B;
  const float *bias;           // per row, or null
  int relu;
  const int32_t *idx, *count;  // list form; null count: all rows
  float *y;                    // dense: [B][rows]; list form: a [positions][8 * NT]
  int y16;                     // dense: y is fp16
  float *part;                 // partial tiles of a split k
  int smin;
  Header *hdr;
};

enum { kDense = 0, kListUp = 1, kListGated = 2 };

// Each warp owns row tiles of 16 rows (8 neurons' gate rows over their 8 up
// rows in the gated form: a thread then holds a neuron's gate and up sums of
// the same tokens side by side) over its CTA's part of k.  A stage is UB
// blocks of 128 weights of each row, loaded one stage ahead into registers
// (16-byte loads; four lanes share a row, so 64 bytes of a row in a row), also
// across the tile's end.  x's part sits in shared memory for the CTA's life.
// With k split, a tile's partial sums meet in the workspace and the warp that
// takes the tile's last ticket adds them in the order of the splits.
template <bool BF, int NT, int UB>
__global__ void __launch_bounds__(kDotWarps * 32, 1) k_w4_dot(DotArgs A, int mode) {
  extern __shared__ __align__(16) unsigned char sm[];
  constexpr int P = BF ? 3 : 1;                    // parts of x
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  int total = A.rows;
  if (mode != kDense) {
    if (A.count) {
      total = ld_cg_i32(A.count);
      if (total < 0 || total > A.rows) {
        if (blockIdx.x == 0 && threadIdx.x == 0) flag_error(&A.hdr->err, kErrIndex);
        total = total < 0 ? 0 : A.rows;
      }
    }
  }
  const int per = mode == kListGated ? 8 : 16;
  const int tiles = ceil_div(total, per);
  const int nblk = w4_kp(A.k) / kBlk, nsb = ceil_div(nblk, 4);
  const int S = w4_splits(tiles, nsb, A.smin, gridDim.x);
  const int ctas = gridDim.x / S;                  // CTAs of one part of k
  const int s = blockIdx.x / ctas, p = blockIdx.x % ctas;
  if (s >= S) return;
  const int sb_per = ceil_div(nsb, S);
  const int b0 = s * sb_per * 4, b1 = min(nblk, b0 + sb_per * 4);   // blocks of this part
  // a warp's unit: tpu consecutive tiles under one ticket
  const int tpu = S > 1 ? ceil_div(tiles, kTicketBytes) : 1;
  const int units = ceil_div(tiles, tpu);
  if (p >= units) return;

  // x's part: [P][B][b1-b0 blocks], rows 64 bytes past a multiple of 128 apart
  // (eight lanes of a 16-byte read then touch every bank once)
  const int kw = (b1 - b0) * kBlk;
  const int xrow = kw * 2 + 64;
  for (int i = threadIdx.x; i < A.B * (kw / 8); i += blockDim.x) {
    const int b = i / (kw / 8), c = (i % (kw / 8)) * 8, kk = b0 * kBlk + c;
    if constexpr (!BF) {
      uint4 v = make_uint4(0, 0, 0, 0);
      if (kk < A.k) v = *reinterpret_cast<const uint4 *>(static_cast<const __half *>(A.x) + (int64_t)b * A.k + kk);
      *reinterpret_cast<uint4 *>(sm + (size_t)b * xrow + c * 2) = v;
    } else {
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
        *reinterpret_cast<uint4 *>(sm + ((size_t)q * A.B + b) * xrow + c * 2) = v;
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] -= trunc_bf16(f[e]);
      }
    }
  }
  __syncthreads();

  const int stages = ceil_div(b1 - b0, UB);
  const int kp2 = w4_kp(A.k) / 2;
  const int gsh = A.group == 32 ? 2 : A.group == 64 ? 1 : 0;         // log2 of the groups of a block
  constexpr int SB = UB * 4;                                         // most scales of a stage

  // rows of a tile: this lane's two row pointers
  auto rows_of = [&](int tile, const unsigned char *&ra, const unsigned char *&rb) {
    int pa = tile * per + g, pb = pa + 8;
    if (mode == kListGated) pb = pa;
    pa = min(pa, total - 1);
    pb = min(pb, total - 1);
    if (mode != kDense && A.idx) {
      pa = ld_cg_i32(A.idx + pa);
      pb = ld_cg_i32(A.idx + pb);
      if ((unsigned)pa >= (unsigned)A.rows) { flag_error(&A.hdr->err, kErrIndex); pa = 0; }
      if ((unsigned)pb >= (unsigned)A.rows) { flag_error(&A.hdr->err, kErrIndex); pb = 0; }
    }
    ra = A.data + (int64_t)pa * A.stride;
    rb = A.data + (int64_t)pb * A.stride + (mode == kListGated ? A.up : 0);
  };
  struct Stage {
    uint4 c[UB][2];
    uint32_t sc[2][SB / 2];
  };
  auto load = [&](Stage &st, const unsigned char *ra, const unsigned char *rb, int stage) {
    const int b = b0 + stage * UB;
#pragma unroll
    for (int u = 0; u < UB; ++u) {
      const bool in = b + u < b1;
      st.c[u][0] = in ? ld_stream(ra + (int64_t)(b + u) * 64 + t * 16) : make_uint4(0, 0, 0, 0);
      st.c[u][1] = in ? ld_stream(rb + (int64_t)(b + u) * 64 + t * 16) : make_uint4(0, 0, 0, 0);
    }
    // UB << gsh scales of each row; the scale area is padded to whole
    // superblocks, so the reads past the last block stay inside it
    const unsigned char *pa = ra + kp2 + ((b << gsh) * 2), *pb = rb + kp2 + ((b << gsh) * 2);
#pragma unroll
    for (int q = 0; q < SB / 2; ++q) {
      const bool in = 2 * q < (UB << gsh);
      st.sc[0][q] = in ? __ldg(reinterpret_cast<const uint32_t *>(pa) + q) : 0u;
      st.sc[1][q] = in ? __ldg(reinterpret_cast<const uint32_t *>(pb) + q) : 0u;
    }
  };

  float tot[NT][4];
  auto compute = [&](const Stage &st, int stage) {
#pragma unroll
    for (int u = 0; u < UB; ++u) {
      if (b0 + stage * UB + u >= b1) break;
      float acc[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
      const unsigned char *xb = sm + (size_t)(stage * UB + u) * 256 + t * 16;
      const uint32_t wa[4] = {st.c[u][0].x, st.c[u][0].y, st.c[u][0].z, st.c[u][0].w};
      const uint32_t wb[4] = {st.c[u][1].x, st.c[u][1].y, st.c[u][1].z, st.c[u][1].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t ha[4], hb[4];
        unpack8<BF>(wa[j], ha);
        unpack8<BF>(wb[j], hb);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const int b = 8 * n + g;
#pragma unroll
          for (int q = 0; q < P; ++q) {
            uint4 xv = make_uint4(0, 0, 0, 0);
            if (b < A.B) xv = *reinterpret_cast<const uint4 *>(xb + ((size_t)q * A.B + b) * xrow + j * 64);
            mma16816<BF>(acc[n], ha[0], hb[0], ha[1], hb[1], xv.x, xv.y);
            mma16816<BF>(acc[n], ha[2], hb[2], ha[3], hb[3], xv.z, xv.w);
          }
        }
        // end of a group: scale its sum (all lanes alike)
        if (j == 3 || gsh == 2 || (gsh == 1 && j == 1)) {
          const int i = (u << gsh) + (j >> (2 - gsh));
          float sa, sb;
          {
            // i is not a constant: pick the half without indexing registers
            uint32_t va = 0, vb = 0;
#pragma unroll
            for (int q = 0; q < SB / 2; ++q)
              if (q == (i >> 1)) { va = st.sc[0][q]; vb = st.sc[1][q]; }
            sa = __half2float(__ushort_as_half((unsigned short)((i & 1) ? va >> 16 : va & 0xffffu)));
            sb = __half2float(__ushort_as_half((unsigned short)((i & 1) ? vb >> 16 : vb & 0xffffu)));
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            tot[n][0] = fmaf(sa, acc[n][0], tot[n][0]);
            tot[n][1] = fmaf(sa, acc[n][1], tot[n][1]);
            tot[n][2] = fmaf(sb, acc[n][2], tot[n][2]);
            tot[n][3] = fmaf(sb, acc[n][3], tot[n][3]);
            acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
          }
        }
      }
    }
  };
  auto finish = [&](int tile) {                    // tot holds the whole sums
    if (mode == kDense) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = tile * 16 + g + 8 * h;
        if (r >= total) continue;
        const float bias = A.bias ? __ldg(A.bias + r) : 0.f;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int b = 8 * n + 2 * t + c;
            float v = tot[n][2 * h + c] + bias;
            if (A.relu) v = v > 0.f ? v : (v != v ? v : 0.f);
            if (b >= A.B) continue;
            if (A.y16) reinterpret_cast<__half *>(A.y)[(int64_t)b * A.rows + r] = __float2half_rn(v);
            else A.y[(int64_t)b * A.rows + r] = v;
          }
      }
      return;
    }
#pragma unroll
    for (int h = 0; h < (mode == kListGated ? 1 : 2); ++h) {
      const int pos = tile * per + g + 8 * h;
      if (pos >= total) continue;
      const int nrn = A.idx ? ld_cg_i32(A.idx + pos) : pos;
      const bool ok = (unsigned)nrn < (unsigned)A.rows;
      const float bias = ok ? __ldg(A.bias + nrn) : 0.f;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float2 v;
        float *pv = &v.x;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float a = tot[n][2 * h + c] + bias;
          a = a > 0.f ? a : (a != a ? a : 0.f);
          if (mode == kListGated) a *= tot[n][2 + c];
          pv[c] = ok && 8 * n + 2 * t + c < A.B ? a : 0.f;
        }
        *reinterpret_cast<float2 *>(A.y + ((int64_t)pos * NT + n) * 8 + 2 * t) = v;
      }
    }
  };

  const int step = ctas * kDotWarps;
  Stage cur, nxt;
  int unit = p + ctas * warp;
  if (unit >= units) return;
  int tile = unit * tpu, stage = 0;
  const unsigned char *ra, *rb;
  rows_of(tile, ra, rb);
  load(cur, ra, rb, 0);
#pragma unroll
  for (int n = 0; n < NT; ++n) tot[n][0] = tot[n][1] = tot[n][2] = tot[n][3] = 0.f;
  while (true) {
    // where the next stage is
    int nu = unit, nt = tile, ns = stage + 1;
    if (ns == stages) {
      ns = 0;
      nt = tile + 1;
      if (nt == min(tiles, (unit + 1) * tpu)) {
        nu = unit + step;
        nt = nu * tpu;
      }
    }
    const bool more = nu < units;
    if (more) {
      if (ns == 0) rows_of(nt, ra, rb);
      load(nxt, ra, rb, ns);
    }
    compute(cur, stage);
    if (stage == stages - 1) {
      if (S == 1) {
        finish(tile);
      } else {
        float4 *to = reinterpret_cast<float4 *>(A.part) + ((int64_t)tile * S + s) * NT * 32 + lane;
#pragma unroll
        for (int n = 0; n < NT; ++n) __stcg(to + n * 32, make_float4(tot[n][0], tot[n][1], tot[n][2], tot[n][3]));
        if (nu != unit) {                          // the unit's last tile
          __syncwarp();
          uint32_t old = 0;
          const int sh = 8 * (unit & 3);
          uint32_t *word = &A.hdr->tile_done[unit >> 2];
          if (lane == 0) {
            __threadfence();
            old = (atomicAdd(word, 1u << sh) >> sh) & 255u;
            __threadfence();
          }
          old = __shfl_sync(0xffffffffu, old, 0);
          if (old == (uint32_t)(S - 1)) {
            for (int tl = unit * tpu; tl < min(tiles, (unit + 1) * tpu); ++tl) {
#pragma unroll
              for (int n = 0; n < NT; ++n) tot[n][0] = tot[n][1] = tot[n][2] = tot[n][3] = 0.f;
              for (int q = 0; q < S; ++q) {
                const float4 *from = reinterpret_cast<const float4 *>(A.part) + ((int64_t)tl * S + q) * NT * 32 + lane;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                  const float4 v = __ldcg(from + n * 32);
                  tot[n][0] += v.x; tot[n][1] += v.y; tot[n][2] += v.z; tot[n][3] += v.w;
                }
              }
              finish(tl);
            }
            if (lane == 0) atomicSub(word, (uint32_t)S << sh);       // the ticket is zero again for the next call
          }
        }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) tot[n][0] = tot[n][1] = tot[n][2] = tot[n][3] = 0.f;
    }
    if (!more) break;
    cur = nxt;
    unit = nu;
    tile = nt;
    stage = ns;
  }
}

// ---------------------------------------------------- down projection --
// y[b][c] = sum_j a[j][b] s[j][c / group] (q[j][c] - 8): the neurons are the
// contracted dimension, so the scale, which changes with the neuron, joins the
// activation: v = a s in fp32, split exactly into three bf16 parts as x above.
// D is 16 columns x 8 tokens.  Two neurons' words give one operand register by
// a byte permutation of the packed codes, before they are unpacked: a word's
// low half holds its even weights, its high half the odd ones.
struct DownArgs {
  const unsigned char *data;   // first down row
  int64_t stride;
  int n, d, group;
  const int32_t *idx, *count;
  const float *a;              // [positions][8 * NT]
  int B, R;                    // tokens, list splits
  float *part;                 // [R][B][d]
  float *y;
  Header *hdr;
};

template <int NT>
__global__ void __launch_bounds__(kDownWarps * 32, NT <= 2 ? 2 : 1) k_w4_down(DownArgs A) {
  extern __shared__ __align__(16) float red[];     // [256 columns][8 * NT + 1]
  constexpr int RS = 8 * NT + 1;
  __shared__ uint32_t s_last;
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  int total = A.n;
  if (A.count) total = max(0, min(A.n, ld_cg_i32(A.count)));   // out of range: flagged by the gate/up kernel
  const int ntile = ceil_div(total, 16);
  const int R = max(1, min(A.R, ceil_div(ntile, kDownWarps / 2)));
  const int cu = blockIdx.x / A.R, r = blockIdx.x % A.R;
  if (r >= R) return;
  const int kp = w4_kp(A.d);
  const int col0 = cu * kDownCols + (warp & 1) * kBlk;         // this warp's block
  const bool live = col0 < kp;
  const int gsh = A.group == 32 ? 2 : A.group == 64 ? 1 : 0;
  const int sub = g & 3;                                       // word column of this lane's rows
  const uint32_t sel = (g >> 2) ? 0x7632u : 0x5410u;           // odd or even weights of two words

  float acc[8][NT][4];                             // [group of 32][half] x tokens
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[i][n][0] = acc[i][n][1] = acc[i][n][2] = acc[i][n][3] = 0.f;

  struct Stage {
    uint4 c[4];
    uint2 sc[4];
    int pos[4];                                    // -1: no such position, or not a neuron
  };
  // the four neurons of this lane: 2t, 2t+1, 2t+8, 2t+9 of the tile
  auto load = [&](Stage &st, int tile) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int pos = tile * 16 + 2 * t + (i & 1) + 8 * (i >> 1);
      int nrn = -1;
      if (pos < total) nrn = A.idx ? ld_cg_i32(A.idx + pos) : pos;
      const bool ok = (unsigned)nrn < (unsigned)A.n;
      st.pos[i] = ok ? pos : -1;
      const unsigned char *row = A.data + (int64_t)(ok ? nrn : 0) * A.stride;
      st.c[i] = ok ? ld_stream(row + col0 / 2 + sub * 16) : make_uint4(0, 0, 0, 0);
      st.sc[i] = make_uint2(0, 0);
      if (ok) {
        const unsigned char *ps = row + kp / 2 + (((col0 / kBlk) << gsh) * 2);
        if (gsh == 0) st.sc[i].x = __ldg(reinterpret_cast<const unsigned short *>(ps));
        else if (gsh == 1) st.sc[i].x = __ldg(reinterpret_cast<const uint32_t *>(ps));
        else st.sc[i] = __ldg(reinterpret_cast<const uint2 *>(ps));
      }
    }
  };
  auto compute = [&](const Stage &st) {
    uint32_t bp[NT][3][2];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j == 0 || gsh == 2 || (gsh == 1 && j == 2)) {        // a new group of columns: a * s
        float s[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t w = (gsh == 2 && j >= 2) ? st.sc[i].y : st.sc[i].x;
          const bool hi = gsh == 2 ? (j & 1) : (gsh == 1 && j == 2);
          s[i] = __half2float(__ushort_as_half((unsigned short)(hi ? w >> 16 : w & 0xffffu)));
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float v[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            v[i] = st.pos[i] >= 0 ? ld_cg_f32(A.a + ((int64_t)st.pos[i] * NT + n) * 8 + g) * s[i] : 0.f;
#pragma unroll
          for (int q = 0; q < 3; ++q) {
            bp[n][q][0] = upper2(v[0], v[1]);
            bp[n][q][1] = upper2(v[2], v[3]);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] -= trunc_bf16(v[i]);
          }
        }
      }
      const uint32_t w[4] = {(&st.c[0].x)[j], (&st.c[1].x)[j], (&st.c[2].x)[j], (&st.c[3].x)[j]};
      uint32_t lo[4], hi[4];
      unpack8<true>(__byte_perm(w[0], w[1], sel), lo);         // [p] = weight 2p + (g >> 2) of neurons 2t, 2t+1
      unpack8<true>(__byte_perm(w[2], w[3], sel), hi);         // of neurons 2t+8, 2t+9
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int q = 0; q < 3; ++q) {
          mma16816<true>(acc[2 * j][n], lo[0], lo[1], hi[0], hi[1], bp[n][q][0], bp[n][q][1]);
          mma16816<true>(acc[2 * j + 1][n], lo[2], lo[3], hi[2], hi[3], bp[n][q][0], bp[n][q][1]);
        }
    }
  };
  const int first = r * (kDownWarps / 2) + (warp >> 1), stride = R * (kDownWarps / 2);
  if (live && first < ntile) {
    Stage cur, nxt;
    load(cur, first);
    for (int tile = first; tile < ntile; tile += stride) {
      if (tile + stride < ntile) load(nxt, tile + stride);
      compute(cur);
      cur = nxt;
    }
  }
  // sum the four warps of a column block, in order
  for (int q = 0; q < kDownWarps / 2; ++q) {
    if ((warp >> 1) == q) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            // row g of half h is weight 2p + (g >> 2) of word 4j + (g & 3), p = 2h (+1 for row g + 8)
            const int p = 2 * (i & 1) + (c >> 1);
            const int col = (warp & 1) * kBlk + (i >> 1) * 32 + sub * 8 + 2 * p + (g >> 2);
            float *to = red + col * RS + 8 * n + 2 * t + (c & 1);
            *to = q == 0 ? acc[i][n][c] : *to + acc[i][n][c];
          }
    }
    __syncthreads();
  }
  float *out = R == 1 ? A.y : A.part + (int64_t)r * A.B * A.d;
  for (int i = threadIdx.x; i < A.B * kDownCols; i += blockDim.x) {
    const int b = i / kDownCols, c = cu * kDownCols + i % kDownCols;
    if (c < A.d) {
      if (R == 1) out[(int64_t)b * A.d + c] = red[(i % kDownCols) * RS + b];
      else __stcg(out + (int64_t)b * A.d + c, red[(i % kDownCols) * RS + b]);
    }
  }
  if (R == 1) return;
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    s_last = ticket_acq_rel(&A.hdr->tile_done[cu]);
    __threadfence();
  }
  __syncthreads();
  if (s_last != (uint32_t)(R - 1)) return;
  for (int i = threadIdx.x; i < A.B * kDownCols; i += blockDim.x) {
    const int b = i / kDownCols, c = cu * kDownCols + i % kDownCols;
    if (c >= A.d) continue;
    float v = 0.f;
    for (int q = 0; q < R; ++q) v += __ldcg(A.part + ((int64_t)q * A.B + b) * A.d + c);
    A.y[(int64_t)b * A.d + c] = v;
  }
  if (threadIdx.x == 0) A.hdr->tile_done[cu] = 0;
}

// ------------------------------------------------------------------ host --
asf_status check_w4(const asf_w4_matrix *m) {
  if (!m || !m->data) return ASF_ERR_INVALID_ARG;
  if (m->group != 32 && m->group != 64 && m->group != 128) return ASF_ERR_UNSUPPORTED;
  if (m->rows <= 0 || m->k <= 0) return ASF_ERR_INVALID_ARG;
  if (m->k % 8 || m->row_stride % 16 || !al16(m->data)) return ASF_ERR_MISALIGNED;
  if (m->k > ASF_W4_MAX_K) return ASF_ERR_UNSUPPORTED;
  if (m->row_stride < w4_row_bytes(m->k, m->group)) return ASF_ERR_INVALID_ARG;
  return ASF_OK;
}
int ffn_mats(const asf_w4_ffn *f) { return f->act == ASF_ACT_REGLU ? 3 : 2; }
asf_status check_w4_ffn(const asf_w4_ffn *f) {
  if (!f || !f->data || !f->bias) return ASF_ERR_INVALID_ARG;
  if (f->act != ASF_ACT_RELU && f->act != ASF_ACT_REGLU) return ASF_ERR_UNSUPPORTED;
  if (f->group != 32 && f->group != 64 && f->group != 128) return ASF_ERR_UNSUPPORTED;
  if (f->d <= 0 || f->n <= 0) return ASF_ERR_INVALID_ARG;
  if (f->d % 8 || f->neuron_stride % 16 || !al16(f->data) || !al4(f->bias)) return ASF_ERR_MISALIGNED;
  if (f->d > ASF_W4_MAX_K) return ASF_ERR_UNSUPPORTED;
  if (f->neuron_stride < ffn_mats(f) * w4_row_bytes(f->d, f->group)) return ASF_ERR_INVALID_ARG;
  return ASF_OK;
}

// superblocks of x that fit a CTA, for B tokens
int dot_smin(int k, int B, int parts) {
  const int nsb = ceil_div(w4_kp(k), kSuper);
  const size_t row = (size_t)B * parts;
  const int fit = (int)std::max<size_t>(1, (kDotSmem - row * 64) / (row * kSuper * 2));
  return ceil_div(nsb, fit);
}
int dot_ctas() { return sm_count(); }
int nt_of(int B) { return B <= 8 ? 1 : B <= 16 ? 2 : 4; }

// partial sums of a split k: at most max(8 CTAs-worth of tiles + tiles, tiles * smin) row tiles
size_t dot_part_bytes(int tiles, int k, int B) {
  const size_t most = std::max<size_t>((size_t)8 * dot_ctas() + tiles, (size_t)tiles * (dot_smin(k, B, 3) + 1));
  return r256(most * nt_of(B) * 512);
}
int down_units(int d) { return ceil_div(w4_kp(d), kDownCols); }
int down_w4_splits(int d, int B) {
  const int per_sm = nt_of(B) <= 2 ? 2 : 1;
  return std::max(1, sm_count() * per_sm / down_units(d));
}
size_t ffn_w4_scratch(const asf_w4_ffn *f, int B) {
  const int tiles = ceil_div(f->n, f->act == ASF_ACT_REGLU ? 8 : 16);
  return r256((size_t)f->n * nt_of(B) * 32) + dot_part_bytes(tiles, f->d, B) +
         r256((size_t)down_w4_splits(f->d, B) * B * f->d * 4);
}

template <bool BF>
cudaError_t run_dot(const DotArgs &a, int mode, cudaStream_t st) {
  const int parts = BF ? 3 : 1;
  const int nsb = ceil_div(w4_kp(a.k), kSuper);
  const int sb = ceil_div(nsb, a.smin);
  const size_t smem = (size_t)a.B * parts * ((size_t)sb * kSuper * 2 + 64);
  const dim3 grid(dot_ctas()), block(kDotWarps * 32);
  switch (nt_of(a.B)) {
    case 1: return launch(k_w4_dot<BF, 1, 2>, grid, block, smem, st, a, mode);
    case 2: return launch(k_w4_dot<BF, 2, 2>, grid, block, smem, st, a, mode);
    default: return launch(k_w4_dot<BF, 4, 2>, grid, block, smem, st, a, mode);
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
    if (mat) need = std::max(need, dot_part_bytes(ceil_div(mat->rows, 16), mat->k, B));
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
  const int64_t units = (int64_t)mat->rows * ceil_div(mat->k, kSuper);
  const dim3 grid((unsigned)((units + 7) / 8)), block(256);
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
  const int64_t words = (int64_t)mat->rows * (mat->k / 8);
  const dim3 grid((unsigned)((words + 255) / 256)), block(256);
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
  if (!al16(x) || !al4(y) || !al4(bias)) return ASF_ERR_MISALIGNED;
  s = check_ws(ws, ws_bytes, kHeaderBytes + dot_part_bytes(ceil_div(mat->rows, 16), mat->k, B));
  if (s != ASF_OK) return s;
  DotArgs a{};
  a.data = static_cast<const unsigned char *>(mat->data);
  a.stride = mat->row_stride;
  a.rows = mat->rows;
  a.k = mat->k;
  a.group = mat->group;
  a.x = x;
  a.B = B;
  a.bias = bias;
  a.relu = relu;
  a.y = static_cast<float *>(y);
  a.y16 = ydtype == ASF_F16;
  a.part = reinterpret_cast<float *>(static_cast<unsigned char *>(ws) + kHeaderBytes);
  a.smin = dot_smin(mat->k, B, xdtype == ASF_F32 ? 3 : 1);
  a.hdr = static_cast<Header *>(ws);
  return cuda_status(xdtype == ASF_F32 ? run_dot<true>(a, kDense, (cudaStream_t)stream)
                                       : run_dot<false>(a, kDense, (cudaStream_t)stream));
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
  const bool gated = f->act == ASF_ACT_REGLU;
  unsigned char *base = static_cast<unsigned char *>(ws) + kHeaderBytes;
  const int64_t rb = w4_row_bytes(f->d, f->group);
  DotArgs a{};
  a.data = static_cast<const unsigned char *>(f->data);
  a.stride = f->neuron_stride;
  a.up = gated ? rb : 0;
  a.rows = f->n;
  a.k = f->d;
  a.group = f->group;
  a.x = x;
  a.B = B;
  a.bias = f->bias;
  a.idx = idx;
  a.count = count;
  a.y = reinterpret_cast<float *>(base);
  base += r256((size_t)f->n * nt_of(B) * 32);
  a.part = reinterpret_cast<float *>(base);
  base += dot_part_bytes(ceil_div(f->n, gated ? 8 : 16), f->d, B);
  a.smin = dot_smin(f->d, B, xdtype == ASF_F32 ? 3 : 1);
  a.hdr = static_cast<Header *>(ws);
  const int mode = gated ? kListGated : kListUp;
  cudaStream_t st = (cudaStream_t)stream;
  cudaError_t e = xdtype == ASF_F32 ? run_dot<true>(a, mode, st) : run_dot<false>(a, mode, st);
  if (e != cudaSuccess) return ASF_ERR_CUDA;
  DownArgs w{};
  w.data = a.data + (ffn_mats(f) - 1) * rb;
  w.stride = f->neuron_stride;
  w.n = f->n;
  w.d = f->d;
  w.group = f->group;
  w.idx = idx;
  w.count = count;
  w.a = a.y;
  w.B = B;
  w.R = down_w4_splits(f->d, B);
  w.part = reinterpret_cast<float *>(base);
  w.y = y;
  w.hdr = a.hdr;
  const dim3 grid(down_units(f->d) * w.R), block(kDownWarps * 32);
  const int nt = nt_of(B);
  const size_t smem = (size_t)kDownCols * (8 * nt + 1) * 4;
  return cuda_status(nt == 1   ? launch(k_w4_down<1>, grid, block, smem, st, w)
                     : nt == 2 ? launch(k_w4_down<2>, grid, block, smem, st, w)
                               : launch(k_w4_down<4>, grid, block, smem, st, w));
}

}  // extern "C"
