// What the kernels of tree attention and of its scores share: the call's
// arguments, the plan that every kernel makes of the requests, and matrix steps.
#pragma once

#include <cuda.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "asffn.h"
#include "common.cuh"
#include "host.cuh"
#include "paged.cuh"

namespace asf {

constexpr int kTile = 64;              // keys per tile
constexpr int kMinChunk = 4;           // key tiles per split, at least
constexpr uint64_t kTcWaitNs = 200ull * 1000 * 1000;   // bound on any mbarrier wait

struct AttnArgs {
  const __half *k, *v;
  int64_t page_stride, token_stride, head_stride;
  int pages, page, hkv, D;
  const int32_t *table;
  int max_pages, R, T, grp;
  const int32_t *lens, *begin;
  const __half *q;
  const int32_t *anc;
  float scale;                         // times log2(e)
  __half *o;
  float *part;                         // [unit < target][MT][DP]
  float2 *ml;                          // [unit][MT]: reference (log2) and sum
  int4 *plan;                          // per request, for the merge: first token, tokens, splits, first unit
  int target;                          // CTAs to aim at
  int whole;                           // key tiles up to which nothing is split
  int cluster;                         // CTAs that share a unit
  int box;                             // keys of a TMA load, or 0
  int32_t *err;
  float2 *stats;                       // scored: per row (token, query head) its reference (log2) and sum
  int mt;                              // rows of the attention's row tiles
  bool beside;                         // the scores are summed beside the merge, from the splits' references and sums
  float *z;                            // [row][zs]: every row's scores (log2, -inf where it sees nothing), or null
  int64_t zs;
  float *scores;                       // [R][hkv][S]
  int S;
};

// One request, as every kernel here sees it.
struct Req {
  int t0, n;                           // its tokens
  int len, L;                          // keys before them, and with them
  int nkt, rt;                         // key tiles, row tiles
  int splits, base;                    // splits of the keys, first unit
};

// The requests: lane r holds request r, all but splits and base.  Bad inputs are
// clamped; the flag says so.
__device__ __forceinline__ Req req_lane(const AttnArgs &A, int MT, int lane, bool &bad) {
  Req q{};
  bad = false;
  if (lane < A.R) {
    int t0 = ld_cg_i32(A.begin + lane), t1 = ld_cg_i32(A.begin + lane + 1);
    bad = t0 < 0 || t1 < t0 || t1 > A.T;
    t0 = min(max(t0, 0), A.T);
    t1 = min(max(t1, t0), A.T);
    q.t0 = t0;
    q.n = t1 - t0;
  }
  int end = q.t0 + q.n;                // ranges stay apart whatever `begin` holds: the units then fit the grid
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, end, o);
    if (lane >= o) end = max(end, v);
  }
  int before = __shfl_up_sync(0xffffffffu, end, 1);
  if (lane == 0) before = 0;
  if (lane < A.R) {
    const int t1 = q.t0 + q.n, t0 = max(q.t0, min(before, t1));
    int len = ld_cg_i32(A.lens + lane);
    const int64_t cap = (int64_t)A.max_pages * A.page;
    bad |= len < 0 || (int64_t)len + (t1 - t0) > cap;
    len = (int)min((int64_t)max(len, 0), cap);
    q.t0 = t0;
    q.n = t1 - t0;
    q.len = len;
    q.L = (int)min((int64_t)len + q.n, cap);
    q.nkt = max(1, (q.L + kTile - 1) / kTile);
    q.rt = (q.n * A.grp + MT - 1) / MT;
  }
  return q;
}
// The plan: C key tiles per unit, the fewest for which the units (request, kv
// head, row tile, split) fit `target` CTAs (one split each where even that is more).
__device__ __forceinline__ Req plan_lane(const AttnArgs &A, int MT, int lane, int &C, int &units, bool &bad) {
  Req q = req_lane(A, MT, lane, bad);
  int64_t W = (int64_t)q.rt * q.nkt;
  int most = q.rt ? q.nkt : 0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    W += __shfl_xor_sync(0xffffffffu, W, o);
    most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
  }
  C = max(most <= A.whole ? A.whole : kMinChunk, (int)((W * A.hkv + A.target - 1) / A.target));
  while (true) {
    q.splits = (q.nkt + C - 1) / C;
    int u = q.rt * q.splits * A.hkv;
    const int own = u;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, u, o);
      if (lane >= o) u += v;
    }
    q.base = u - own;
    units = __shfl_sync(0xffffffffu, u, 31);
    if (units <= A.target || C >= most) break;
    C += max(1, C / 16);
  }
  return q;
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_h2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ float exp2_fast(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// Map of a cache's keys or values: columns, tokens of a page, heads, pages; a
// box is `box` tokens of one head and page by 64 columns, swizzled as the MMA
// reads it.  Columns past head_dim and pages past the last read as zeros.
inline bool cache_map(CUtensorMap *tm, const void *base, const AttnArgs &a) {
  TmapEncodeFn enc = tmap_encoder();
  if (!enc) return false;
  const cuuint64_t dims[4] = {(cuuint64_t)a.D, (cuuint64_t)a.page, (cuuint64_t)a.hkv, (cuuint64_t)a.pages};
  // the stride of a dimension of one is never used, but has to be legal
  const cuuint64_t strides[3] = {(cuuint64_t)a.token_stride * 2, (cuuint64_t)std::max<int64_t>(a.head_stride, 8) * 2,
                                 (cuuint64_t)std::max<int64_t>(a.page_stride, 8) * 2};
  const cuuint32_t box[4] = {64, (cuuint32_t)a.box, 1, 1}, one[4] = {1, 1, 1, 1};
  return enc(tm, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, const_cast<void *>(base), dims, strides, box, one,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Keys of a TMA load where a tile of 64 keys is whole pages or lies in one, else 0.
inline int tma_box(int page) { return page >= kTile ? (page % kTile ? 0 : kTile) : page >= 8 && kTile % page == 0 ? page : 0; }

// scores of a call whose attention has left a.stats (score.cu)
cudaError_t run_scores(AttnArgs a, cudaStream_t st);

}  // namespace asf
