// Attention of a tree of drafted tokens over a paged key/value cache, and the
// append that fills it (include/asffn.h, "Tree attention").
//
//   asf_kv_append        k_kv_append
//   asf_tree_attention   k_tree_attn, then k_tree_merge over split requests
//
// Mathematics.  For a query row q (token t of request r, one query head) over
// the keys p that t sees: z_p = scale q.k_p, o = sum_p e^(z_p - m) v_p / l with
// m = max z_p and l = sum_p e^(z_p - m).  One pass over the keys keeps the
// running m, l and the unnormalised sum; parts over disjoint keys merge by
// rescaling to the larger m, which is how warps and splits of the keys meet.
// All of it in fp32 in units of log2 (scale log2(e) joins the score); the
// weights e^(z - m) are rounded to fp16 for the product with v, half a step of
// 2^-11 each, as much as the output's own rounding and averaged over the keys.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "asffn.h"
#include "common.cuh"
#include "host.cuh"

using namespace asf;

namespace {

constexpr int kTile = 64;              // keys per tile
constexpr int kStages = 3;             // tiles in shared memory
constexpr int kMinChunk = 4;           // key tiles per split, at least
constexpr int kWhole = 8;              // key tiles up to which nothing is split (no merge to launch)

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
  float *part;                         // [unit][MT][DP]
  float2 *ml;                          // [unit][MT]: maximum (log2) and sum
  int4 *plan;                          // per request, for the merge: first token, tokens, splits, first unit
  int target;                          // CTAs to aim at
  int32_t *err;
};

// One request, as every kernel here sees it.
struct Req {
  int t0, n;                           // its tokens
  int len, L;                          // keys before them, and with them
  int nkt, rt;                         // key tiles, row tiles
  int splits, base;                    // splits of the keys, first unit
};

// The plan: lane r holds request r.  C key tiles per unit, the fewest for
// which the units (request, kv head, row tile, split) fit `target` CTAs (one
// split each where even that is more).  Bad inputs are clamped; the flag says so.
__device__ __forceinline__ Req plan_lane(const AttnArgs &A, int MT, int lane, int &C, int &units, bool &bad) {
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
  int64_t W = (int64_t)q.rt * q.nkt;
  int most = q.rt ? q.nkt : 0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    W += __shfl_xor_sync(0xffffffffu, W, o);
    most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
  }
  C = max(most <= kWhole ? kWhole : kMinChunk, (int)((W * A.hkv + A.target - 1) / A.target));
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

// CTAs of an SM: what their stages (48 or 96 KB) and registers leave.
__host__ __device__ constexpr int attn_resident(int DP, int WM) { return DP == 64 ? (WM == 8 ? 2 : 3) : (WM == 8 ? 1 : 2); }

// A CTA is one unit: WM groups of 16 query rows x KG groups of keys, a warp
// each.  Keys and values of a tile go to shared memory by 16-byte cp.async, two
// tiles ahead; 16-byte chunk c of row i sits at c ^ (i & 7), so that the
// 8 x 8 matrix loads touch every bank once.
template <int DP, int WM>
__global__ void __launch_bounds__((WM > 4 ? WM : 4) * 32, attn_resident(DP, WM)) k_tree_attn(AttnArgs A) {
  constexpr int NW = WM > 4 ? WM : 4;
  constexpr int KG = NW / WM;          // key groups
  constexpr int KW = kTile / KG;       // keys of a warp
  constexpr int MT = WM * 16;
  constexpr int CH = DP / 8;           // 16-byte chunks of a row
  extern __shared__ __align__(128) unsigned char sm[];
  __shared__ int64_t s_off[4][kTile];  // element offset of a key's row, -1: no such key
  __shared__ int s_special[4];         // a tile with a key that some row does not see
  __shared__ int s_unit[10];
  __shared__ uint32_t s_nonfin[2];     // drafted values of a tile that are not finite
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  pdl_wait();
  pdl_trigger();
  if (warp == 0) {
    int C, units;
    bool bad;
    const Req q = plan_lane(A, MT, lane, C, units, bad);
    if (bad && blockIdx.x == 0) flag_error(A.err, kErrIndex);
    if (blockIdx.x == 0) A.plan[lane] = make_int4(q.t0, q.n, q.splits, q.base);
    const int mine = q.rt * q.splits * A.hkv, u = (int)blockIdx.x - q.base;
    if (lane == 0) s_unit[0] = -1;
    __syncwarp();
    if (u >= 0 && u < mine) {
      const int tile = u % q.rt, s = u / q.rt % q.splits;
      s_unit[0] = lane;
      s_unit[1] = u / q.rt / q.splits;              // kv head
      s_unit[2] = tile;
      s_unit[3] = s * C;
      s_unit[4] = min(q.nkt, (s + 1) * C);
      s_unit[5] = q.t0;
      s_unit[6] = q.n;
      s_unit[7] = q.len;
      s_unit[8] = q.L;
      s_unit[9] = q.splits;
    }
  }
  __syncthreads();
  const int req = s_unit[0];
  if (req < 0) return;
  const int head = s_unit[1], row0 = s_unit[2] * MT, kt0 = s_unit[3], kt1 = s_unit[4];
  const int t0 = s_unit[5], n = s_unit[6], len = s_unit[7], L = s_unit[8], splits = s_unit[9];
  const int rows = n * A.grp;
  const int wm = warp % WM, kg = warp / WM;

  // offsets of a tile's keys
  auto offsets = [&](int j) {
    if (tid >= kTile) return;
    const int slot = j & 3, pos = (kt0 + j) * kTile + tid;
    int64_t off = -1;
    if (kt0 + j < kt1 && pos < L) {
      const int pi = pos / A.page;
      const int id = __ldg(A.table + (int64_t)req * A.max_pages + pi);
      if ((unsigned)id < (unsigned)A.pages)
        off = (int64_t)id * A.page_stride + (int64_t)(pos - pi * A.page) * A.token_stride + (int64_t)head * A.head_stride;
      else
        flag_error(A.err, kErrIndex);
    }
    s_off[slot][tid] = off;
    const bool sp = off < 0 || pos >= len;
    if (tid == 0) s_special[slot] = 0;
    asm volatile("bar.sync 1, 64;" ::: "memory");
    if (sp) s_special[slot] = 1;
  };
  auto copy = [&](int j) {             // 8 lanes a row: whole 128-byte lines
    if (kt0 + j < kt1) {
      unsigned char *kb = sm + (size_t)(j % kStages) * (2 * kTile * DP * 2), *vb = kb + kTile * DP * 2;
#pragma unroll
      for (int i = tid >> 3; i < kTile; i += NW * 4) {
        const int64_t off = s_off[j & 3][i];
#pragma unroll
        for (int c = tid & 7; c < CH; c += 8) {
          const bool in = off >= 0 && c * 8 < A.D;
          const uint32_t at = i * DP * 2 + ((c ^ (i & 7)) * 16);
          cp_async16(kb + at, A.k + (in ? off + c * 8 : 0), in ? 16u : 0u);
          cp_async16(vb + at, A.v + (in ? off + c * 8 : 0), in ? 16u : 0u);
        }
      }
    }
    cp_async_commit();
  };
  offsets(0);
  offsets(1);
  offsets(2);

  // this lane's two rows, their masks and their queries
  uint32_t see[2];
  uint32_t qf[DP / 16][4];
  const __half *qp[2];
  bool live[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int m = row0 + wm * 16 + g + 8 * h;
    live[h] = m < rows;
    const int tok = t0 + (live[h] ? m / A.grp : 0), hq = head * A.grp + (live[h] ? m % A.grp : 0);
    see[h] = live[h] ? (uint32_t)__ldg(A.anc + tok) : 0u;
    qp[h] = A.q + ((int64_t)tok * A.hkv * A.grp + hq) * A.D;
  }
#pragma unroll
  for (int s = 0; s < DP / 16; ++s)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = s * 16 + 2 * t + 8 * (i >> 1);
      qf[s][i] = live[i & 1] && c < A.D ? __ldg(reinterpret_cast<const uint32_t *>(qp[i & 1] + c)) : 0u;
    }
  __syncthreads();
  copy(0);
  copy(1);

  float acc[DP / 8][4], mx[2] = {-INFINITY, -INFINITY}, sum[2] = {0.f, 0.f};
#pragma unroll
  for (int i = 0; i < DP / 8; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
  const uint32_t smb = smem_u32(sm);
  const int tiles = kt1 - kt0;
  for (int j = 0; j < tiles; ++j) {
    cp_async_wait<kStages - 2>();
    __syncthreads();
    copy(j + 2);
    const uint32_t kb = smb + (uint32_t)(j % kStages) * (2 * kTile * DP * 2), vb = kb + kTile * DP * 2;
    const bool special = s_special[j & 3];
    const int key0 = kg * KW;
    const int pos0 = (kt0 + j) * kTile;
    uint32_t nonfin[2] = {0u, 0u};
    if (special && pos0 + kTile > len) {
      // A drafted value that is not finite would reach rows that do not see it
      // as 0 * NaN: take such rows of v out of the product, add them below.
      if (tid < 2) s_nonfin[tid] = 0u;
      __syncthreads();
      unsigned char *vp = sm + (size_t)(j % kStages) * (2 * kTile * DP * 2) + kTile * DP * 2;
      for (int i = tid; i < kTile * CH; i += NW * 32) {
        if (pos0 + i / CH < len) continue;
        const uint4 u = *reinterpret_cast<const uint4 *>(vp + i * 16);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
        bool bad = false;
#pragma unroll
        for (int e = 0; e < 4; ++e) bad |= (w[e] & 0x7c00u) == 0x7c00u || (w[e] & 0x7c000000u) == 0x7c000000u;
        if (bad) atomicOr(&s_nonfin[i / CH / 32], 1u << (i / CH % 32));
      }
      __syncthreads();
      nonfin[0] = s_nonfin[0];
      nonfin[1] = s_nonfin[1];
      if (nonfin[0] | nonfin[1]) {
        for (int i = tid; i < kTile * CH; i += NW * 32)
          if (((i / CH & 32 ? nonfin[1] : nonfin[0]) >> (i / CH % 32)) & 1u) *reinterpret_cast<uint4 *>(vp + i * 16) = make_uint4(0, 0, 0, 0);
        __syncthreads();
      }
    }
    float z[KW / 8][4];
#pragma unroll
    for (int i = 0; i < KW / 8; ++i) z[i][0] = z[i][1] = z[i][2] = z[i][3] = 0.f;
#pragma unroll
    for (int s = 0; s < DP / 16; ++s)
#pragma unroll
      for (int i = 0; i < KW / 16; ++i) {
        uint32_t b[4];
        const int row = key0 + i * 16 + (lane >> 4) * 8 + (lane & 7), c = s * 2 + ((lane >> 3) & 1);
        ldsm4(b, kb + row * DP * 2 + ((c ^ (row & 7)) * 16));
        mma_f16(z[2 * i], qf[s], b[0], b[1]);
        mma_f16(z[2 * i + 1], qf[s], b[2], b[3]);
      }
    float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int i = 0; i < KW / 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) z[i][e] *= A.scale;
    if (special) {
#pragma unroll
      for (int i = 0; i < KW / 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int key = key0 + i * 8 + 2 * t + (e & 1), d = pos0 + key - len;
          const bool ok = s_off[j & 3][key] >= 0 && (d < 0 || ((see[e >> 1] >> ((t0 + d) & 31)) & 1u));
          if (!ok) z[i][e] = -INFINITY;
        }
    }
#pragma unroll
    for (int i = 0; i < KW / 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) top[e >> 1] = fmaxf(top[e >> 1], z[i][e]);
    float fix[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 1));
      top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 2));
      top[h] = fmaxf(top[h], mx[h]);
      const float ref = top[h] == -INFINITY ? 0.f : top[h];   // nothing seen yet: every weight is 2^-inf = 0
      fix[h] = exp2_fast(mx[h] - ref);
      mx[h] = top[h];
      top[h] = ref;
      sum[h] *= fix[h];
    }
    uint32_t pf[KW / 16][4];
#pragma unroll
    for (int i = 0; i < KW / 8; ++i) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        z[i][e] = exp2_fast(z[i][e] - top[e >> 1]);
        sum[e >> 1] += z[i][e];
      }
      pf[i / 2][2 * (i & 1)] = pack_h2(z[i][0], z[i][1]);
      pf[i / 2][2 * (i & 1) + 1] = pack_h2(z[i][2], z[i][3]);
    }
    if (fix[0] != 1.f || fix[1] != 1.f) {
#pragma unroll
      for (int i = 0; i < DP / 8; ++i) {
        acc[i][0] *= fix[0];
        acc[i][1] *= fix[0];
        acc[i][2] *= fix[1];
        acc[i][3] *= fix[1];
      }
    }
#pragma unroll
    for (int i = 0; i < KW / 16; ++i)
#pragma unroll
      for (int s = 0; s < DP / 16; ++s) {
        uint32_t b[4];
        const int row = key0 + i * 16 + ((lane >> 3) & 1) * 8 + (lane & 7), c = s * 2 + (lane >> 4);
        ldsm4_t(b, vb + row * DP * 2 + ((c ^ (row & 7)) * 16));
        mma_f16(acc[2 * s], pf[i], b[0], b[1]);
        mma_f16(acc[2 * s + 1], pf[i], b[2], b[3]);
      }
    if (nonfin[0] | nonfin[1]) {       // rows of v left out above: only where they are seen
#pragma unroll
      for (int i = 0; i < KW / 8; ++i)
#pragma unroll 1
        for (int c = 0; c < 8; ++c) {
          const int key = key0 + i * 8 + c;
          if (!(((key & 32 ? nonfin[1] : nonfin[0]) >> (key & 31)) & 1u)) continue;
          const int from = (lane & 28) | (c >> 1), d = pos0 + key - len;
          float p[2];
          p[0] = __shfl_sync(0xffffffffu, c & 1 ? z[i][1] : z[i][0], from);
          p[1] = __shfl_sync(0xffffffffu, c & 1 ? z[i][3] : z[i][2], from);
          const __half *vr = A.v + s_off[j & 3][key];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (!((see[h] >> ((t0 + d) & 31)) & 1u)) continue;
#pragma unroll
            for (int e = 0; e < DP / 8; ++e)
              if (e * 8 + 2 * t < A.D) {
                acc[e][2 * h] = fmaf(p[h], __half2float(__ldg(vr + e * 8 + 2 * t)), acc[e][2 * h]);
                acc[e][2 * h + 1] = fmaf(p[h], __half2float(__ldg(vr + e * 8 + 2 * t + 1)), acc[e][2 * h + 1]);
              }
          }
        }
    }
    __syncwarp();
    offsets(j + 3);                    // its slot was last read before this iteration's barrier
  }
  cp_async_wait<0>();
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    sum[h] += __shfl_xor_sync(0xffffffffu, sum[h], 1);
    sum[h] += __shfl_xor_sync(0xffffffffu, sum[h], 2);
  }
  if constexpr (KG > 1) {              // the key groups' parts meet in shared memory
    __syncthreads();
    float *so = reinterpret_cast<float *>(sm);                           // [KG][MT][DP]
    float *sml = so + KG * MT * DP;                                      // [KG][MT][2]
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int m = wm * 16 + g + 8 * h;
      if (t == 0) {
        sml[(kg * MT + m) * 2] = mx[h];
        sml[(kg * MT + m) * 2 + 1] = sum[h];
      }
#pragma unroll
      for (int i = 0; i < DP / 8; ++i)
        *reinterpret_cast<float2 *>(so + (kg * MT + m) * DP + i * 8 + 2 * t) = make_float2(acc[i][2 * h], acc[i][2 * h + 1]);
    }
    __syncthreads();
    if (kg != 0) return;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int m = wm * 16 + g + 8 * h;
      float M = -INFINITY;
#pragma unroll
      for (int k = 0; k < KG; ++k) M = fmaxf(M, sml[(k * MT + m) * 2]);
      const float ref = M == -INFINITY ? 0.f : M;
      float l = 0.f;
#pragma unroll
      for (int i = 0; i < DP / 8; ++i) acc[i][2 * h] = acc[i][2 * h + 1] = 0.f;
#pragma unroll
      for (int k = 0; k < KG; ++k) {
        const float f = exp2_fast(sml[(k * MT + m) * 2] - ref);
        l += f * sml[(k * MT + m) * 2 + 1];
#pragma unroll
        for (int i = 0; i < DP / 8; ++i) {
          const float2 v = *reinterpret_cast<const float2 *>(so + (k * MT + m) * DP + i * 8 + 2 * t);
          acc[i][2 * h] += f * v.x;
          acc[i][2 * h + 1] += f * v.y;
        }
      }
      mx[h] = M;
      sum[h] = l;
    }
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (!live[h]) continue;
    const int m = row0 + wm * 16 + g + 8 * h;
    if (splits == 1) {
      const float inv = sum[h] == 0.f ? 0.f : 1.f / sum[h];              // nothing seen: zeros
      __half *op = A.o + ((int64_t)(t0 + m / A.grp) * A.hkv * A.grp + head * A.grp + m % A.grp) * A.D;
#pragma unroll
      for (int i = 0; i < DP / 8; ++i)
        if (i * 8 + 2 * t < A.D)
          *reinterpret_cast<uint32_t *>(op + i * 8 + 2 * t) = pack_h2(acc[i][2 * h] * inv, acc[i][2 * h + 1] * inv);
    } else {
      const int64_t at = (int64_t)blockIdx.x * MT + wm * 16 + g + 8 * h;
      if (t == 0) __stcg(A.ml + at, make_float2(mx[h], sum[h]));
#pragma unroll
      for (int i = 0; i < DP / 8; ++i)
        __stcg(reinterpret_cast<float2 *>(A.part + at * DP + i * 8 + 2 * t), make_float2(acc[i][2 * h], acc[i][2 * h + 1]));
    }
  }
}

// The splits of a row, in order: one warp per (token, query head).
template <int DP>
__global__ void __launch_bounds__(128) k_tree_merge(AttnArgs A, int MT) {
  constexpr int V = DP / 32;
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int4 q = __ldcg(A.plan + lane);
  const int row = blockIdx.x * 4 + (threadIdx.x >> 5);
  const int hq = A.hkv * A.grp, tok = row / hq, hd = row % hq;
  if (tok >= A.T) return;
  const uint32_t who = __ballot_sync(0xffffffffu, tok >= q.x && tok < q.x + q.y);   // ranges do not overlap
  if (!who) return;
  const int r = __ffs(who) - 1;
  const int t0 = __shfl_sync(0xffffffffu, q.x, r), rt = (__shfl_sync(0xffffffffu, q.y, r) * A.grp + MT - 1) / MT;
  const int splits = __shfl_sync(0xffffffffu, q.z, r), base = __shfl_sync(0xffffffffu, q.w, r);
  if (splits == 1) return;
  const int m = (tok - t0) * A.grp + hd % A.grp, head = hd / A.grp;
  const int64_t first = ((int64_t)base + (int64_t)head * splits * rt + m / MT) * MT + m % MT, step = (int64_t)rt * MT;
  float M = -INFINITY;
  for (int s = lane; s < splits; s += 32) M = fmaxf(M, __ldcg(&A.ml[first + s * step].x));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  const float ref = M == -INFINITY ? 0.f : M;
  float l = 0.f, o[V] = {};
#pragma unroll 8
  for (int s = 0; s < splits; ++s) {
    const int64_t at = first + s * step;
    const float2 ml = __ldcg(A.ml + at);
    const float f = exp2_fast(ml.x - ref);
    const float *p = A.part + at * DP + lane * V;
    float v[V];
    if constexpr (V == 4) {
      const float4 u = __ldcg(reinterpret_cast<const float4 *>(p));
      v[0] = u.x; v[1] = u.y; v[2] = u.z; v[3] = u.w;
    } else {
      const float2 u = __ldcg(reinterpret_cast<const float2 *>(p));
      v[0] = u.x; v[1] = u.y;
    }
    l = fmaf(f, ml.y, l);
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] = fmaf(f, v[i], o[i]);
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  __half *op = A.o + (int64_t)row * A.D + lane * V;
#pragma unroll
  for (int i = 0; i < V; i += 2)
    if (lane * V + i < A.D) *reinterpret_cast<uint32_t *>(op + i) = pack_h2(o[i] * inv, o[i + 1] * inv);
}

// One 16-byte chunk of a token's keys and values per thread.
struct AppendArgs {
  __half *k, *v;
  int64_t page_stride, token_stride, head_stride;
  int pages, page, hkv, D;
  const int32_t *table;
  int max_pages, R, T;
  const int32_t *lens, *begin;
  const __half *kn, *vn;
  int32_t *err;
};
__global__ void __launch_bounds__(128) k_kv_append(AppendArgs A) {
  pdl_wait();
  pdl_trigger();
  const int per = A.hkv * (A.D / 8);
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= A.T * per) return;
  const int tok = i / per, head = i % per / (A.D / 8), c = i % (A.D / 8);
  int r = 0;                           // the request whose range holds the token
#pragma unroll 8
  for (int q = 1; q <= A.R; ++q) r += tok >= ld_cg_i32(A.begin + q);
  if (r >= A.R) return;                // behind the last range: nothing is written
  const int t0 = ld_cg_i32(A.begin + r);
  if (tok < t0) return;
  const int len = ld_cg_i32(A.lens + r);
  const int64_t pos = (int64_t)len + (tok - t0);
  const int64_t pi = pos / A.page;
  int id = -1;
  if (t0 >= 0 && len >= 0 && pi < A.max_pages) id = __ldg(A.table + (int64_t)r * A.max_pages + pi);
  if ((unsigned)id >= (unsigned)A.pages) {
    flag_error(A.err, kErrIndex);
    return;
  }
  const int64_t at = (int64_t)id * A.page_stride + (pos - pi * A.page) * A.token_stride + (int64_t)head * A.head_stride + c * 8;
  const int64_t from = ((int64_t)tok * A.hkv + head) * A.D + c * 8;
  *reinterpret_cast<uint4 *>(A.k + at) = *reinterpret_cast<const uint4 *>(A.kn + from);
  *reinterpret_cast<uint4 *>(A.v + at) = *reinterpret_cast<const uint4 *>(A.vn + from);
}

// ------------------------------------------------------------------ host --
asf_status check_cache(const asf_kv_cache *c) {
  if (!c || !c->k || !c->v) return ASF_ERR_INVALID_ARG;
  if (c->pages <= 0 || c->page <= 0 || c->heads <= 0 || c->head_dim <= 0) return ASF_ERR_INVALID_ARG;
  if (c->head_dim > 128 || c->heads > ASF_MAX_KV_HEADS) return ASF_ERR_UNSUPPORTED;
  if (c->head_dim % 8 || c->page_stride % 8 || c->token_stride % 8 || c->head_stride % 8) return ASF_ERR_MISALIGNED;
  if (!al16(c->k) || !al16(c->v)) return ASF_ERR_MISALIGNED;
  if (c->page_stride < 0 || c->token_stride < c->head_dim || c->head_stride < 0 ||
      (c->heads > 1 && c->head_stride < c->head_dim))
    return ASF_ERR_INVALID_ARG;
  return ASF_OK;
}
asf_status check_requests(const int32_t *table, int max_pages, int R, const int32_t *lens, const int32_t *begin, int T) {
  if (!table || !lens || !begin) return ASF_ERR_INVALID_ARG;
  if (max_pages < 1 || R < 1 || R > ASF_MAX_BATCH || T < 1 || T > ASF_MAX_BATCH) return ASF_ERR_INVALID_ARG;
  return ASF_OK;
}
asf_status check_tables(const int32_t *table, int max_pages, int page, const int32_t *lens, const int32_t *begin) {
  if ((int64_t)max_pages * page > ASF_MAX_KEYS) return ASF_ERR_UNSUPPORTED;
  if (!al4(table) || !al4(lens) || !al4(begin)) return ASF_ERR_MISALIGNED;
  return ASF_OK;
}

// Groups of 16 rows a CTA takes: enough for a request's rows where the tokens
// are shared out evenly (any number is right, the rest become row tiles).
int row_groups(int grp, int R, int T) {
  const int rows = (T + R - 1) / R * grp;
  return rows <= 16 ? 1 : rows <= 32 ? 2 : rows <= 64 ? 4 : 8;
}
int row_tiles_most(int grp, int R, int T, int wm) { return T * grp / (16 * wm) + R; }
int attn_dp(const asf_kv_cache *c) { return c->head_dim <= 64 ? 64 : 128; }
int attn_target(const asf_kv_cache *c, int wm) { return sm_count() * attn_resident(attn_dp(c), wm); }
int attn_units_most(const asf_kv_cache *c, int grp, int R, int T, int wm) {
  return attn_target(c, wm) + c->heads * row_tiles_most(grp, R, T, wm);
}
size_t attn_scratch(const asf_kv_cache *c, int grp, int R, int T) {
  const int wm = row_groups(grp, R, T);
  const size_t rows = (size_t)attn_units_most(c, grp, R, T, wm) * 16 * wm;
  return 512 + r256(rows * attn_dp(c) * 4) + r256(rows * 8);
}

template <int DP, int WM>
cudaError_t run_attn(const AttnArgs &a, int units, cudaStream_t st) {
  constexpr int NW = WM > 4 ? WM : 4;
  const size_t smem = (size_t)kStages * 2 * kTile * DP * 2;
  return launch(k_tree_attn<DP, WM>, dim3(units), dim3(NW * 32), smem, st, a);
}
template <int DP>
cudaError_t run_attn_any(const AttnArgs &a, int wm, int units, cudaStream_t st) {
  cudaError_t e = wm == 1   ? run_attn<DP, 1>(a, units, st)
                  : wm == 2 ? run_attn<DP, 2>(a, units, st)
                  : wm == 4 ? run_attn<DP, 4>(a, units, st)
                            : run_attn<DP, 8>(a, units, st);
  if (e != cudaSuccess) return e;
  if ((int64_t)a.max_pages * a.page <= kWhole * kTile) return e;
  const int rows = a.T * a.hkv * a.grp;
  return launch(k_tree_merge<DP>, dim3((rows + 3) / 4), dim3(128), 0, st, a, 16 * wm);
}

}  // namespace

extern "C" {

size_t asf_attention_workspace_bytes(const asf_kv_cache *cache, int32_t q_heads, int32_t R, int32_t T) {
  if (check_cache(cache) != ASF_OK || q_heads < 1 || q_heads % cache->heads) return 0;
  if (R < 1 || R > ASF_MAX_BATCH || T < 1 || T > ASF_MAX_BATCH || q_heads / cache->heads > ASF_MAX_HEAD_GROUP) return 0;
  size_t need = 0;
  for (int r = 1; r <= R; ++r)
    for (int t = 1; t <= T; ++t) need = std::max(need, attn_scratch(cache, q_heads / cache->heads, r, t));
  return kHeaderBytes + need;
}

asf_status asf_kv_append(const asf_kv_cache *cache, const int32_t *table, int32_t max_pages, int32_t R,
                         const int32_t *lens, const int32_t *begin, int32_t T, const void *k, const void *v, void *ws,
                         size_t ws_bytes, asf_stream_t stream) {
  asf_status s = check_cache(cache);
  if (s == ASF_OK) s = check_requests(table, max_pages, R, lens, begin, T);
  if (s == ASF_OK) s = check_tables(table, max_pages, cache->page, lens, begin);
  if (s != ASF_OK) return s;
  if (!k || !v) return ASF_ERR_INVALID_ARG;
  if (!al16(k) || !al16(v)) return ASF_ERR_MISALIGNED;
  s = check_ws(ws, ws_bytes, kHeaderBytes);
  if (s != ASF_OK) return s;
  AppendArgs a{static_cast<__half *>(cache->k), static_cast<__half *>(cache->v), cache->page_stride, cache->token_stride,
               cache->head_stride, cache->pages, cache->page, cache->heads, cache->head_dim, table, max_pages, R, T, lens,
               begin, static_cast<const __half *>(k), static_cast<const __half *>(v), &static_cast<Header *>(ws)->err};
  const int chunks = T * cache->heads * (cache->head_dim / 8);
  return cuda_status(launch(k_kv_append, dim3((chunks + 127) / 128), dim3(128), 0, (cudaStream_t)stream, a));
}

asf_status asf_tree_attention(const asf_kv_cache *cache, const int32_t *table, int32_t max_pages, int32_t R,
                              const int32_t *lens, const int32_t *begin, int32_t T, int32_t q_heads, const void *q,
                              const int32_t *anc, float scale, void *o, void *ws, size_t ws_bytes, asf_stream_t stream) {
  asf_status s = check_cache(cache);
  if (s == ASF_OK) s = check_requests(table, max_pages, R, lens, begin, T);
  if (s == ASF_OK) s = check_tables(table, max_pages, cache->page, lens, begin);
  if (s != ASF_OK) return s;
  if (!q || !anc || !o || q_heads < 1 || q_heads % cache->heads || !std::isfinite(scale)) return ASF_ERR_INVALID_ARG;
  const int grp = q_heads / cache->heads;
  if (grp > ASF_MAX_HEAD_GROUP) return ASF_ERR_UNSUPPORTED;
  if (!al16(q) || !al16(o) || !al4(anc)) return ASF_ERR_MISALIGNED;
  s = check_ws(ws, ws_bytes, kHeaderBytes + attn_scratch(cache, grp, R, T));
  if (s != ASF_OK) return s;
  const int wm = row_groups(grp, R, T);
  const int units = attn_units_most(cache, grp, R, T, wm);
  unsigned char *base = static_cast<unsigned char *>(ws) + kHeaderBytes;
  AttnArgs a{};
  a.k = static_cast<const __half *>(cache->k);
  a.v = static_cast<const __half *>(cache->v);
  a.page_stride = cache->page_stride;
  a.token_stride = cache->token_stride;
  a.head_stride = cache->head_stride;
  a.pages = cache->pages;
  a.page = cache->page;
  a.hkv = cache->heads;
  a.D = cache->head_dim;
  a.table = table;
  a.max_pages = max_pages;
  a.R = R;
  a.T = T;
  a.grp = grp;
  a.lens = lens;
  a.begin = begin;
  a.q = static_cast<const __half *>(q);
  a.anc = anc;
  a.scale = (float)((double)scale * 1.4426950408889634);
  a.o = static_cast<__half *>(o);
  a.plan = reinterpret_cast<int4 *>(base);
  base += 512;
  a.part = reinterpret_cast<float *>(base);
  a.ml = reinterpret_cast<float2 *>(base + r256((size_t)units * 16 * wm * attn_dp(cache) * 4));
  a.target = attn_target(cache, wm);
  a.err = &static_cast<Header *>(ws)->err;
  cudaStream_t st = (cudaStream_t)stream;
  return cuda_status(attn_dp(cache) == 64 ? run_attn_any<64>(a, wm, units, st) : run_attn_any<128>(a, wm, units, st));
}

}  // extern "C"
