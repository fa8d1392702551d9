// Attention of a tree of drafted tokens over a paged key/value cache, and the
// append that fills it (include/asffn.h, "Tree attention").
//
//   asf_kv_append        k_kv_append
//   asf_tree_attention   k_tree_attn, or k_tree_tc for more than 32 query rows of
//                        a request and kv head; then k_tree_merge over split requests
//
// Mathematics.  For a query row q (token t of request r, one query head) over
// the keys p that t sees: z_p = scale q.k_p, o = sum_p e^(z_p - m) v_p / l with
// m = max z_p and l = sum_p e^(z_p - m).  One pass over the keys keeps the
// running m, l and the unnormalised sum; parts over disjoint keys merge by
// rescaling to the larger m, which is how warps and splits of the keys meet.
// All of it in fp32 in units of log2 (scale log2(e) joins the score).
//
// The weights are rounded to fp16 for the product with v, as much as the output's
// own rounding.  Any reference in the place of m is right, since it cancels in
// o, so m is lowered by kLift (k_tree_attn; kLiftTc in k_tree_tc) to put the
// largest weights near the top of fp16's range.  A weight then has an error of
// 2^-12 of itself (half a step of 2^-11) down to 2^-29 (2^-25) of the row's
// largest, and of 2^-40 (2^-36) of the largest below that.  (Without kLift what
// lay 2^-25 below the largest was lost to o, yet counted in l.)
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "asffn.h"
#include "common.cuh"
#include "host.cuh"

using namespace asf;

namespace {

constexpr int kTile = 64;              // keys per tile
constexpr int kStages = 3;             // tiles in shared memory (k_tree_attn)
constexpr int kClusterTiles = 4;       // key tiles that each CTA of a cluster takes at most
constexpr int kMinChunk = 4;           // key tiles per split, at least
constexpr int kWhole = 8;              // key tiles up to which nothing is split (no merge to launch)
constexpr float kTopLog2 = 15.99f;     // of a weight at most: below fp16's largest, 65504
constexpr float kLift = 15.f;
// k_tree_tc lets a row outgrow its reference by the rest, 2^5.  8 ragged requests, and 16
// tokens over 65500 keys, us of the call with a lift of 0 to 9: 33.9, 71.0; 11: 34.1,
// 71.2; 12: 34.9, 72.2, since rows outgrow their references more often.
constexpr float kLiftTc = 11.f;

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

// shared memory of CTA `rank` of the cluster, at the address of this CTA's p
__device__ __forceinline__ uint32_t peer_smem(const void *p, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ float2 ld_peer2(const void *p, int rank) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(peer_smem(p, rank)) : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_peer4(const void *p, int rank) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(peer_smem(p, rank))
               : "memory");
  return v;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// CTAs of an SM: what their stages (48 or 96 KB), registers and, for k_tree_tc
// (8 groups of 16 rows), tensor memory leave.
__host__ __device__ constexpr int attn_resident(int DP, int WM) { return DP == 64 && WM < 8 ? 3 : 2; }

// A CTA is one unit: WM (1 or 2) groups of 16 query rows x KG groups of keys, a
// warp each.  Keys and values of a tile go to shared memory by 16-byte cp.async, two
// tiles ahead; 16-byte chunk c of row i sits at c ^ (i & 7), so that the
// 8 x 8 matrix loads touch every bank once.  With CL > 1 a cluster of CTAs shares
// the unit's tiles, CTA c every CL-th from c on, and adds its parts over
// distributed shared memory: the form for few units of few tiles, which
// otherwise leave most SMs idle and yet are not worth a merge of their own.
// Latency bounds it below some MB of keys (32 heads of 333 keys, 5.5 MB: 10.8 us
// with the append, and 15.9 where the table has room for 4096 keys, which takes the
// form without clusters and the merge's launch), the loads in flight above: 32
// requests of 4096 keys (8 kv heads, 537 MB) 98.8 us, 5.4 TB/s.
template <int DP, int WM, int CL>
__global__ void __launch_bounds__(128, attn_resident(DP, WM)) k_tree_attn(AttnArgs A) {
  constexpr int NW = 4;
  constexpr int KG = NW / WM;          // key groups
  constexpr int KW = kTile / KG;       // keys of a warp
  constexpr int MT = WM * 16;
  constexpr int CH = DP / 8;           // 16-byte chunks of a row
  extern __shared__ __align__(128) unsigned char sm[];
  constexpr int NST = kStages, SLOTS = 4;   // NST + 1 at least
  __shared__ int64_t s_off[SLOTS][kTile];   // element offset of a key's row, -1: no such key
  __shared__ int s_special[SLOTS];     // a tile with a key that some row does not see
  __shared__ int s_unit[10];
  __shared__ uint32_t s_nonfin[2];     // drafted values of a tile that are not finite
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  if (tid >= 32 && tid < 32 + SLOTS) s_special[tid - 32] = 0;
  pdl_wait();
  pdl_trigger();
  if (warp == 0) {
    int C, units;
    bool bad;
    const Req q = plan_lane(A, MT, lane, C, units, bad);
    if (bad && blockIdx.x == 0) flag_error(A.err, kErrIndex);
    if (blockIdx.x == 0) A.plan[lane] = make_int4(q.t0, q.n, q.splits, q.base);
    const int mine = q.rt * q.splits * A.hkv, u = (int)blockIdx.x / CL - q.base;
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
  // this CTA's tiles: kt0, kt0 + CL, ...
  const int head = s_unit[1], row0 = s_unit[2] * MT, kt0 = s_unit[3] + (int)blockIdx.x % CL, kt1 = s_unit[4];
  const int t0 = s_unit[5], n = s_unit[6], len = s_unit[7], L = s_unit[8], splits = s_unit[9];
  const int rows = n * A.grp;
  const int wm = warp % WM, kg = warp / WM;

  // a key's page, as the table has it
  auto page_of = [&](int pos) { return A.table[(int64_t)req * A.max_pages + pos / A.page]; };
  auto offset_of = [&](int pos, int id) -> int64_t {
    if ((unsigned)id >= (unsigned)A.pages) {
      flag_error(A.err, kErrIndex);
      return -1;
    }
    return (int64_t)id * A.page_stride + (int64_t)(pos % A.page) * A.token_stride + (int64_t)head * A.head_stride;
  };
  // offsets of a tile's keys
  auto offsets = [&](int j) {
    if (tid >= kTile) return;
    const int slot = j & (SLOTS - 1), pos = (kt0 + j * CL) * kTile + tid;
    const int64_t off = kt0 + j * CL < kt1 && pos < L ? offset_of(pos, page_of(pos)) : -1;
    s_off[slot][tid] = off;
    const bool sp = off < 0 || pos >= len;
    if (tid == 0) s_special[slot] = 0;
    asm volatile("bar.sync 1, 64;" ::: "memory");
    if (sp) s_special[slot] = 1;
  };
  {
    // of the first NST tiles, their table entries all at once (tile by tile: 2 us more)
    int id[(NST + 1) / 2];
#pragma unroll
    for (int i = 0; i < (NST + 1) / 2; ++i) {
      const int j = 2 * i + (tid >> 6), pos = (kt0 + j * CL) * kTile + (tid & 63);
      id[i] = j < NST && kt0 + j * CL < kt1 && pos < L ? page_of(pos) : 0;
    }
#pragma unroll
    for (int i = 0; i < (NST + 1) / 2; ++i) {
      const int j = 2 * i + (tid >> 6), pos = (kt0 + j * CL) * kTile + (tid & 63);
      if (j >= NST) continue;
      const int64_t off = kt0 + j * CL < kt1 && pos < L ? offset_of(pos, id[i]) : -1;
      s_off[j][tid & 63] = off;
      if (off < 0 || pos >= len) s_special[j] = 1;
    }
  }
  auto copy = [&](int j) {             // 8 lanes a row: whole 128-byte lines
    if (kt0 + j * CL < kt1) {
      unsigned char *kb = sm + (size_t)(j % NST) * (2 * kTile * DP * 2), *vb = kb + kTile * DP * 2;
#pragma unroll
      for (int i = tid >> 3; i < kTile; i += NW * 4) {
        const int64_t off = s_off[j & (SLOTS - 1)][i];
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
    see[h] = live[h] ? (uint32_t)A.anc[tok] : 0u;
    qp[h] = A.q + ((int64_t)tok * A.hkv * A.grp + hq) * A.D;
  }
#pragma unroll
  for (int s = 0; s < DP / 16; ++s)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = s * 16 + 2 * t + 8 * (i >> 1);
      qf[s][i] = live[i & 1] && c < A.D ? *reinterpret_cast<const uint32_t *>(qp[i & 1] + c) : 0u;
    }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < NST - 1; ++j) copy(j);

  float acc[DP / 8][4], mx[2] = {-INFINITY, -INFINITY}, sum[2] = {0.f, 0.f};   // mx: the rows' references
#pragma unroll
  for (int i = 0; i < DP / 8; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
  const uint32_t smb = smem_u32(sm);
  const int tiles = (kt1 - kt0 + CL - 1) / CL;
  for (int j = 0; j < tiles; ++j) {
    cp_async_wait<NST - 2>();
    __syncthreads();
    copy(j + NST - 1);
    const uint32_t kb = smb + (uint32_t)(j % NST) * (2 * kTile * DP * 2), vb = kb + kTile * DP * 2;
    const bool special = s_special[j & (SLOTS - 1)];
    const int key0 = kg * KW;
    const int pos0 = (kt0 + j * CL) * kTile;
    uint32_t nonfin[2] = {0u, 0u};
    if (special && pos0 + kTile > len) {
      // A drafted value that is not finite would reach rows that do not see it
      // as 0 * NaN: take such rows of v out of the product, add them below.
      if (tid < 2) s_nonfin[tid] = 0u;
      __syncthreads();
      unsigned char *vp = sm + (size_t)(j % NST) * (2 * kTile * DP * 2) + kTile * DP * 2;
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
          if (((i / CH & 32 ? nonfin[1] : nonfin[0]) >> (i / CH % 32)) & 1u)
            *reinterpret_cast<uint4 *>(vp + i * 16) = make_uint4(0, 0, 0, 0);
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
          const bool ok = s_off[j & (SLOTS - 1)][key] >= 0 && (d < 0 || ((see[e >> 1] >> ((t0 + d) & 31)) & 1u));
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
      float low = top[h] - kLift;
      if (!(top[h] - low <= kTopLog2)) low = top[h];             // scores so large that this rounds, and infinities
      low = fmaxf(low, mx[h]);
      const float ref = low == -INFINITY ? 0.f : low;         // nothing seen yet: every weight is 2^-inf = 0
      fix[h] = exp2_fast(mx[h] - ref);
      mx[h] = low;
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
          const __half *vr = A.v + s_off[j & (SLOTS - 1)][key];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (!((see[h] >> ((t0 + d) & 31)) & 1u)) continue;
#pragma unroll
            for (int e = 0; e < DP / 8; ++e)
              if (e * 8 + 2 * t < A.D) {
                acc[e][2 * h] = fmaf(p[h], __half2float(vr[e * 8 + 2 * t]), acc[e][2 * h]);
                acc[e][2 * h + 1] = fmaf(p[h], __half2float(vr[e * 8 + 2 * t + 1]), acc[e][2 * h + 1]);
              }
          }
        }
    }
    __syncwarp();
    offsets(j + NST);                  // its slot was last read before this iteration's barrier
  }
  cp_async_wait<0>();
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    sum[h] += __shfl_xor_sync(0xffffffffu, sum[h], 1);
    sum[h] += __shfl_xor_sync(0xffffffffu, sum[h], 2);
  }
  if constexpr (KG > 1 || CL > 1) {    // the key groups' parts meet in shared memory
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
    if constexpr (CL > 1) {
      // all CL x KG parts of a row, MT / CL rows a CTA, four columns a thread
      cluster_sync();
      const int rank = (int)blockIdx.x % CL;
      for (int i = tid; i < MT / CL * (DP / 4); i += 128) {
        const int row = rank * (MT / CL) + i / (DP / 4), c = i % (DP / 4) * 4, m = row0 + row;
        float M = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
        float2 ml[CL * KG];
        float4 v[CL * KG];
#pragma unroll
        for (int p = 0; p < CL * KG; ++p) {
          ml[p] = ld_peer2(sml + ((p % KG) * MT + row) * 2, p / KG);
          v[p] = ld_peer4(so + ((p % KG) * MT + row) * DP + c, p / KG);
          M = fmaxf(M, ml[p].x);
        }
        const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll
        for (int p = 0; p < CL * KG; ++p) {
          const float f = exp2_fast(ml[p].x - ref);
          l = fmaf(f, ml[p].y, l);
          o[0] = fmaf(f, v[p].x, o[0]); o[1] = fmaf(f, v[p].y, o[1]); o[2] = fmaf(f, v[p].z, o[2]); o[3] = fmaf(f, v[p].w, o[3]);
        }
        const float inv = l == 0.f ? 0.f : 1.f / l;                      // nothing seen: zeros
        if (m < rows && c < A.D) {
          __half *op = A.o + ((int64_t)(t0 + m / A.grp) * A.hkv * A.grp + head * A.grp + m % A.grp) * A.D + c;
          *reinterpret_cast<uint2 *>(op) = make_uint2(pack_h2(o[0] * inv, o[1] * inv), pack_h2(o[2] * inv, o[3] * inv));
        }
      }
      __syncwarp();
      cluster_sync();                  // nobody leaves while its parts are read
      return;
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

// ------------------------------------------- many rows: tcgen05 ----------
// For tiles of more than 32 query rows mma.sync's rate (a quarter of
// tcgen05's) bounds the kernel above, not HBM.  Here a CTA takes 128 rows:
//   warps 4, 5 copy tiles of 64 keys (warp 4) and of their values (warp 5) into
//              the 128-byte swizzled layout that the MMA reads;
//   warp 6     one thread issues S = Q K^T (M 128, N 64) into one of two
//              accumulators in tensor memory, and O += P V with P read from
//              tensor memory (V as it lies: keys are its K, so it is MN-major);
//   warps 0-3  a thread per row copies its row of Q, then per tile reads S, masks it, takes the running maximum
//              and sum, and writes P in fp16 over the accumulator it has read.
// S of the next tile is computed while this one's weights are, and keys and
// values have slots of their own: the keys' are free as soon as S is there, so
// only their copy has to be ahead, and a tile's values arrive under its
// exponentials.  O is rescaled
// only when the weights of some row of a warp would pass fp16's range, 2^5 above where
// its last reference put the largest: that spares a pass over O in tensor memory per
// tile.  Two CTAs share an SM,
// one's products under the other's exponentials.
//
// 16 tokens x 64 heads over 65500 keys (8 kv heads, 268 MB): 54.9 us alone, 4.9
// TB/s; what is left is the exponentials and the passes between registers and
// tensor memory (issue slots 39% used, tensor pipe 34%).  The kernel above with
// eight row groups took 150 us for the call, this one 64.
template <int DP>
struct TreeTc {
  static constexpr int Q = 128 * DP * 2;
  static constexpr int KV = kTile * DP * 2;        // keys, or values, of a tile
  static constexpr int NS = DP == 128 ? 2 : 4;     // slots of keys, and of values
  static constexpr int BAR = 1024;
  static constexpr size_t SMEM = 1024 + BAR + Q + (size_t)NS * 2 * KV;
  static constexpr uint32_t COLS = 256;            // O: DP columns at 0; S and P: 64 each at 128 and 192
};
constexpr int kTcThreads = 7 * 32;
constexpr uint64_t kTcWaitNs = 200ull * 1000 * 1000;   // bound on any mbarrier wait

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const float (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(v[8]), "f"(v[9]),
      "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15])
      : "memory");
}

//
// Copies: where a tile is whole pages or lies in one (pages of 8, 16, 32 or a
// multiple of 64 tokens), one TMA load per page and 64 columns; else 16-byte
// cp.async, whose rate is what an SM's load path takes (about 25 bytes a
// clock).
template <int DP, bool TMA>
__global__ void __launch_bounds__(kTcThreads, 2)
    k_tree_tc(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v, AttnArgs A) {
  using Lc = TreeTc<DP>;
  constexpr int NS = Lc::NS, MT = 128, CH = DP / 8;
  extern __shared__ unsigned char smem_raw[];
  __shared__ int s_unit[10];
  __shared__ int64_t s_off[2][2][kTile];           // of keys, of values: element offset of a row, -1: no such key
  __shared__ uint32_t s_valid[8][2];               // keys of a tile that exist
  __shared__ uint32_t s_nonfin[NS][kTile];         // 16-byte chunks of drafted values left out of the product
  __shared__ int s_any[NS];
  unsigned char *smem = align_1024(smem_raw);
  uint64_t *full_k = reinterpret_cast<uint64_t *>(smem), *empty_k = full_k + NS;
  uint64_t *full_v = empty_k + NS, *empty_v = full_v + NS;
  uint64_t *bs = empty_v + NS, *bp = bs + 2, *bo = bp + 2, *bq = bo + 2, *land = bq + 1;
  uint32_t *tslot = reinterpret_cast<uint32_t *>(land + 1);
  unsigned char *sq = smem + Lc::BAR, *sk = sq + Lc::Q, *sv = sk + NS * Lc::KV;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(&full_k[i], TMA ? 1 : 32);
      mbar_init(&full_v[i], TMA ? 1 : 32);
      mbar_init(&empty_k[i], 1);
      mbar_init(&empty_v[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bs[i], 2);                        // the products, and the thread that issued them
      mbar_init(&bp[i], 4 * 32);
      mbar_init(&bo[i], 1);
    }
    mbar_init(bq, 128);
    mbar_init(land, 1);
    fence_mbar_init();
    if (TMA) {
      prefetch_map(&map_k);
      prefetch_map(&map_v);
    }
  }
  if (warp == 6) {
    tmem_alloc(tslot, Lc::COLS);
    tmem_relinquish();
  }
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
      s_unit[1] = u / q.rt / q.splits;
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
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tslot;
  const int req = s_unit[0];
  if (req < 0) {
    if (warp == 6) tmem_dealloc(tbase, Lc::COLS);
    return;
  }
  const int head = s_unit[1], row0 = s_unit[2] * MT, kt0 = s_unit[3], tiles = s_unit[4] - kt0;
  const int t0 = s_unit[5], n = s_unit[6], len = s_unit[7], L = s_unit[8], splits = s_unit[9];
  const int rows = n * A.grp;

  if (warp == 4 || warp == 5) {
    // ---------------------------------------------------------------- copies --
    const bool is_k = warp == 4;
    const __half *base = is_k ? A.k : A.v;
    unsigned char *slots = is_k ? sk : sv;
    uint64_t *full = is_k ? full_k : full_v, *empty = is_k ? empty_k : empty_v;
    int64_t(*off)[kTile] = s_off[warp - 4];
    auto offsets = [&](int j) {                    // two keys a lane
      if (j >= tiles) return;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int pos = (kt0 + j) * kTile + 32 * h + lane;
        int64_t o = -1;
        if (pos < L) {
          const int pi = pos / A.page;
          const int id = A.table[(int64_t)req * A.max_pages + pi];
          if ((unsigned)id < (unsigned)A.pages)
            o = (int64_t)id * A.page_stride + (int64_t)(pos - pi * A.page) * A.token_stride + (int64_t)head * A.head_stride;
          else
            flag_error(A.err, kErrIndex);
        }
        off[j & 1][32 * h + lane] = o;
        const uint32_t have = __ballot_sync(0xffffffffu, o >= 0);
        if (is_k && lane == 0) s_valid[j & 7][h] = have;
      }
    };
    // this lane's 16-byte chunk of every RP-th row
    constexpr int RP = 32 / CH, ROWS = kTile / RP;
    const int r0 = lane / CH, c = lane % CH;
    const bool col = c * 8 < A.D;
    if (!TMA) offsets(0);
    // tile j has landed; drafted values are looked over first
    auto hand_on = [&](int j) {
      const int sl = j % NS, pos0 = (kt0 + j) * kTile;
      if (!is_k && pos0 + kTile > len) {
#pragma unroll 4
        for (int i = 0; i < ROWS; ++i) {           // (cp.async: the chunks that this lane has copied)
          const int r = r0 + i * RP;
          uint4 *at = reinterpret_cast<uint4 *>(slots + (size_t)sl * Lc::KV + (c >> 3) * (kTile * 128) + r * 128 +
                                                (((c & 7) ^ (r & 7)) << 4));
          const uint4 u = *at;
          const uint32_t w[4] = {u.x, u.y, u.z, u.w};
          bool bad = false;
#pragma unroll
          for (int e = 0; e < 4; ++e) bad |= (w[e] & 0x7c00u) == 0x7c00u || (w[e] & 0x7c000000u) == 0x7c000000u;
          if (TMA && pos0 + r >= L) {
            *at = make_uint4(0, 0, 0, 0);          // what lies behind the last key
          } else if (bad && pos0 + r >= len) {
            // 0 * NaN would reach rows that do not see the key: out of the
            // product, added by the rows that do
            *at = make_uint4(0, 0, 0, 0);
            atomicOr(&s_nonfin[sl][r], 1u << c);
            s_any[sl] = 1;
          }
        }
      }
      fence_proxy_async_smem();
      if (TMA) __syncwarp();
      if (!TMA || lane == 0) mbar_arrive(&full[sl]);
    };
    bool ok = true;
    int marked = 0;                                // tiles that had to be looked over
    if (TMA) {
      const int nb = kTile / A.box;
      // lane b: box b of tile j, as the table's entry (looked at a tile later, when it
      // has come) and a token of that page, -1: no such box
      auto page_of = [&](int j, int &tok) {
        const int pos = (kt0 + j) * kTile + lane * A.box;
        tok = -1;
        if (j >= tiles || lane >= nb || pos >= L) return -1;
        const int pi = pos / A.page;
        tok = pos - pi * A.page;
        return (int)A.table[(int64_t)req * A.max_pages + pi];
      };
      int tok, id = page_of(0, tok);
      const uint32_t bytes = kTile * DP * 2;
      for (int j = 0; j < tiles; ++j) {
        const int sl = j % NS, pos0 = (kt0 + j) * kTile;
        const int at = tok, now = tok >= 0 && (unsigned)id < (unsigned)A.pages ? id : -1;
        if (at >= 0 && now < 0) flag_error(A.err, kErrIndex);
        id = page_of(j + 1, tok);
        if (j >= NS) {
          ok = warp_wait(&empty[sl], (uint32_t)((j / NS) - 1) & 1u, kTcWaitNs);
          if (!ok) {
            // what is on its way lands before the shared memory is given back
            for (int e = j - NS; e < j; ++e) warp_wait(&full[e % NS], (uint32_t)(e / NS) & 1u, kTcWaitNs);
            break;
          }
        }
        if (is_k) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int key = 32 * h + lane;
            const bool there = __shfl_sync(0xffffffffu, now, key / A.box) >= 0 && pos0 + key < L;
            const uint32_t have = __ballot_sync(0xffffffffu, there);
            if (lane == 0) s_valid[j & 7][h] = have;
          }
        } else {
          s_nonfin[sl][lane] = s_nonfin[sl][32 + lane] = 0;
          if (lane == 0) s_any[sl] = 0;
        }
        const bool look = !is_k && pos0 + kTile > len;
        uint64_t *bar = look ? land : &full[sl];
        __syncwarp();
        if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
        __syncwarp();
        if (lane < nb) {
          // a page that is not there: outside the map, zeros
#pragma unroll
          for (int h = 0; h < DP / 64; ++h)
            tma_load_4d(slots + (size_t)sl * Lc::KV + h * (kTile * 128) + lane * A.box * 128, is_k ? &map_k : &map_v, 64 * h,
                        now >= 0 ? at : 0, head, now >= 0 ? now : A.pages, bar);
        }
        __syncwarp();
        if (look) {
          ok = warp_wait(land, (uint32_t)(marked++) & 1u, kTcWaitNs);
          __syncwarp();
          if (!ok) break;
          hand_on(j);
        }
      }
      if (!ok) flag_error(A.err, kErrTimeout);
    }
    for (int j = 0; j < (TMA ? 0 : tiles); ++j) {
      const int sl = j % NS;
      bool behind = j > 0;                         // tile j - 1 is not handed on yet
      __syncwarp();                                // off[j & 1] is written
      if (j >= NS) {
        const uint32_t parity = (uint32_t)((j / NS) - 1) & 1u;
        if (!__all_sync(0xffffffffu, mbar_test(&empty[sl], parity))) {
          cp_async_wait<0>();                      // the slot may need tile j - 1
          hand_on(j - 1);
          behind = false;
          ok = warp_wait(&empty[sl], parity, kTcWaitNs);
          if (!ok) break;
        }
      }
      if (!is_k) {
        s_nonfin[sl][lane] = s_nonfin[sl][32 + lane] = 0;
        if (lane == 0) s_any[sl] = 0;
        __syncwarp();
      }
      unsigned char *to = slots + (size_t)sl * Lc::KV + (c >> 3) * (kTile * 128);
#pragma unroll
      for (int i0 = 0; i0 < ROWS; i0 += 16) {
        int64_t o[16];                             // read ahead: a copy is a barrier to the compiler
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i] = off[j & 1][r0 + (i0 + i) * RP];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int r = r0 + (i0 + i) * RP;
          const bool in = o[i] >= 0 && col;
          cp_async16(to + r * 128 + (((c & 7) ^ (r & 7)) << 4), in ? base + o[i] + c * 8 : base, in ? 16u : 0u);
        }
      }
      cp_async_commit();
      if (behind) {
        cp_async_wait<1>();
        hand_on(j - 1);
      }
      offsets(j + 1);
    }
    if (!TMA) {
      cp_async_wait<0>();                          // nothing lands in shared memory that is given back
      if (ok) hand_on(tiles - 1);
      else flag_error(A.err, kErrTimeout);
    }
  } else if (warp == 6) {
    // ------------------------------------------------------------------- MMA --
    constexpr uint32_t id_s = umma_idesc_f16(128, kTile, 0, 0), id_o = umma_idesc_f16(128, DP, 0, 1);
    const uint64_t dq = umma_desc(sq, 16, 1024, kSwz128), dk = umma_desc(sk, 16, 1024, kSwz128);
    // 16 keys of V: two groups of 8 rows (1024 apart), 64-column atoms half a slot apart
    const uint64_t dv = umma_desc(sv, kTile * 128, 1024, kSwz128);
    bool ok = warp_wait(bq, 0, kTcWaitNs);
    auto pv = [&](int i) {
      const int sl = i % NS;
      if (!warp_wait(&bp[i & 1], (uint32_t)(i >> 1) & 1u, kTcWaitNs)) return false;
      if (!warp_wait(&full_v[sl], (uint32_t)(i / NS) & 1u, kTcWaitNs)) return false;
      tc_fence_after();
      const uint64_t d = dv + (uint64_t)(sl * (Lc::KV >> 4));
      const uint32_t p = tbase + 128 + 64 * (i & 1);
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < kTile / 16; ++k) umma_f16_ta(tbase, p + 8 * k, d + k * (2048 >> 4), id_o, 1);
        umma_commit(&empty_v[sl]);
        umma_commit(&bo[i & 1]);
      }
      __syncwarp();
      return true;
    };
    for (int j = 0; j < tiles && ok; ++j) {
      const int sl = j % NS;
      if (!(ok = warp_wait(&full_k[sl], (uint32_t)(j / NS) & 1u, kTcWaitNs))) break;
      tc_fence_after();
      const uint64_t d = dk + (uint64_t)(sl * (Lc::KV >> 4));
      const uint32_t z = tbase + 128 + 64 * (j & 1);
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < DP / 16; ++k)
          umma_f16(z, dq + ((k >> 2) * (128 * 128) + (k & 3) * 32) / 16, d + ((k >> 2) * (kTile * 128) + (k & 3) * 32) / 16, id_s,
                   k != 0);
        umma_commit(&empty_k[sl]);
        umma_commit(&bs[j & 1]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bs[j & 1]);      // passes on what the copying threads have written
      if (j > 0) ok = pv(j - 1);
    }
    if (ok) ok = pv(tiles - 1);
    if (!ok && lane == 0) flag_error(A.err, kErrTimeout);
  } else {
    // ---------------------------------------------------------------- softmax --
    const int m = row0 + tid;
    const bool live = m < rows;
    const int tok = t0 + (live ? m / A.grp : 0);
    // drafted tokens that the row sees, by their place in the request
    const uint32_t see = live ? ((uint32_t)A.anc[tok] >> t0) & (n >= 32 ? 0xffffffffu : (1u << n) - 1u) : 0u;
    const uint32_t tl = tbase + ((uint32_t)(32 * warp) << 16);
    {
      // the row of Q; a row past the request's is zeros
      const __half *src = live ? A.q + ((int64_t)tok * A.hkv * A.grp + head * A.grp + m % A.grp) * A.D : A.q;
#pragma unroll
      for (int c = 0; c < CH; ++c)
        cp_async16(sq + (c >> 3) * (128 * 128) + tid * 128 + (((c & 7) ^ (tid & 7)) << 4), live && c * 8 < A.D ? src + c * 8 : A.q,
                   live && c * 8 < A.D ? 16u : 0u);
      cp_async_commit();
      float zero[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) zero[i] = 0.f;
#pragma unroll
      for (int c = 0; c < DP; c += 16) tmem_st16(tl + c, zero);
      tmem_wait_st();
      cp_async_wait<0>();
      fence_proxy_async_smem();
      mbar_arrive(bq);
    }
    float ref = 0.f, sum = 0.f;
    bool ok = true;                                // sum: 0 until a key is seen (2^11 at least from then on; NaN stays)
    for (int j = 0; j < tiles; ++j) {
      const uint32_t sc = tl + 128 + 64 * (j & 1);
      const int pos0 = (kt0 + j) * kTile, sl = j % NS;
      ok = warp_wait(&bs[j & 1], (uint32_t)(j >> 1) & 1u, kTcWaitNs);
      if (ok && pos0 + kTile > len) ok = warp_wait(&full_v[sl], (uint32_t)(j / NS) & 1u, kTcWaitNs);   // the marks of its values
      if (!ok) break;
      tc_fence_after();
      __syncwarp();                                // tensor-memory accesses are warp-synchronous
      // which of the tile's keys the row sees
      uint64_t sees = (uint64_t)s_valid[j & 7][0] | (uint64_t)s_valid[j & 7][1] << 32;
      const int d = len - pos0;                    // keys of the tile in front of the drafted ones
      if (d < kTile) {
        uint64_t w = 0;
        if (d > 0) w = ((uint64_t)1 << d) - 1 | (uint64_t)see << d;
        else if (d > -32) w = (uint64_t)(see >> -d);
        sees &= w;
      }
      float top = -INFINITY;
      const bool all = __all_sync(0xffffffffu, sees == ~(uint64_t)0);
      float z[kTile];
      tmem_ld64(sc, z);
      if (!all) {
#pragma unroll
        for (int i = 0; i < kTile; ++i) z[i] = (sees >> i) & 1 ? z[i] * A.scale : -INFINITY;
      } else {
#pragma unroll
        for (int i = 0; i < kTile; ++i) z[i] *= A.scale;
      }
#pragma unroll
      for (int i = 0; i < kTile; ++i) top = fmaxf(top, z[i]);
      // a new reference for the warp's rows where some row needs one
      const bool grow = top != -INFINITY && (sum == 0.f || top - ref > kTopLog2);
      const bool redo = __any_sync(0xffffffffu, grow);
      const bool extra = d < kTile && s_any[sl];
      if ((redo || extra) && j > 0) {              // O must rest: the product of the last tile is done
        ok = warp_wait(&bo[(j - 1) & 1], (uint32_t)((j - 1) >> 1) & 1u, kTcWaitNs);
        if (!ok) break;
        tc_fence_after();
        __syncwarp();
      }
      if (redo) {
        float now = grow ? top - kLiftTc : ref;
        if (grow && !(top - now <= kTopLog2)) now = top;       // scores so large that this rounds, and infinities
        const float f = sum != 0.f ? exp2_fast(ref - now) : 0.f;
        if (j > 0) {
#pragma unroll
          for (int c = 0; c < DP; c += 16) {
            float o[16];
            tmem_ld16w(tl + c, o);
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = sum != 0.f ? o[i] * f : 0.f;
            tmem_st16(tl + c, o);
          }
          tmem_wait_st();
        }
        sum = sum != 0.f ? sum * f : 0.f;
        ref = now;
      }
      if (extra) {
        // the chunks of v left out, for the rows that see their keys
#pragma unroll 1
        for (int i = max(0, d); i < kTile && pos0 + i < L; ++i) {
          const uint32_t bad = s_nonfin[sl][i];
          if (!bad) continue;                      // the same for every lane
          const int pos = pos0 + i, pi = pos / A.page, id = A.table[(int64_t)req * A.max_pages + pi];
          const __half *v = A.v + (int64_t)id * A.page_stride + (int64_t)(pos - pi * A.page) * A.token_stride +
                            (int64_t)head * A.head_stride;
          const bool on = (sees >> i) & 1;
          const float w = exp2_fast(tmem_ld1(sc + i) * A.scale - ref);
#pragma unroll 1
          for (int h = 0; h < CH; h += 2) {
            if (!((bad >> h) & 3u)) continue;
            float o[16];
            __syncwarp();
            tmem_ld16w(tl + 8 * h, o);
#pragma unroll
            for (int q = 0; q < 16; ++q)
              if (on && ((bad >> (h + (q >> 3))) & 1u)) o[q] = fmaf(w, __half2float(v[8 * h + q]), o[q]);
            __syncwarp();
            tmem_st16(tl + 8 * h, o);
            tmem_wait_st();
          }
        }
        __syncwarp();
      }
#pragma unroll
      for (int i = 0; i < kTile; ++i) {
        z[i] = exp2_fast(z[i] - ref);
        sum += z[i];
      }
#pragma unroll
      for (int c = 0; c < kTile; c += 16) {        // over scores that are in registers
        uint32_t p[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = pack_h2(z[c + 2 * i], z[c + 2 * i + 1]);
        tmem_st8(sc + c / 2, p);
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&bp[j & 1]);
    }
    if (ok) {
      ok = warp_wait(&bo[(tiles - 1) & 1], (uint32_t)((tiles - 1) >> 1) & 1u, kTcWaitNs);
      tc_fence_after();
    }
    if (!ok && lane == 0) flag_error(A.err, kErrTimeout);
    const float inv = sum == 0.f ? 0.f : 1.f / sum;                      // nothing seen: zeros
    const int64_t at = (int64_t)blockIdx.x * MT + tid;
    if (splits > 1 && live) __stcg(A.ml + at, make_float2(sum != 0.f ? ref : -INFINITY, sum));
    __half *op = A.o + ((int64_t)tok * A.hkv * A.grp + head * A.grp + (live ? m % A.grp : 0)) * A.D;
#pragma unroll
    for (int c = 0; c < DP; c += 16) {
      float o[16];
      __syncwarp();
      tmem_ld16w(tl + c, o);
      if (live && splits == 1) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (c + 8 * h < A.D) {
            uint4 u;
            u.x = pack_h2(o[8 * h] * inv, o[8 * h + 1] * inv);
            u.y = pack_h2(o[8 * h + 2] * inv, o[8 * h + 3] * inv);
            u.z = pack_h2(o[8 * h + 4] * inv, o[8 * h + 5] * inv);
            u.w = pack_h2(o[8 * h + 6] * inv, o[8 * h + 7] * inv);
            *reinterpret_cast<uint4 *>(op + c + 8 * h) = u;
          }
      } else if (live) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          __stcg(reinterpret_cast<float4 *>(A.part + at * DP + c) + q, make_float4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]));
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 6) {
    tc_fence_after();
    tmem_dealloc(tbase, Lc::COLS);
  }
}

// The splits of a row (token, query head): W warps take every W-th split each,
// with up to AHEAD in flight, and their sums meet in a fixed order.  What bounds
// it is latency: plan, then maxima and sums beside the first parts.
template <int DP, int W, int AHEAD>
__global__ void __launch_bounds__(128) k_tree_merge(AttnArgs A, int MT) {
  constexpr int V = DP / 32;
  __shared__ float s_m[4], s_l[4], s_o[4][DP];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int4 q = __ldcg(A.plan + lane);
  const int row = blockIdx.x * (4 / W) + warp / W, hq = A.hkv * A.grp, tok = row / hq, hd = row % hq;
  const uint32_t who = __ballot_sync(0xffffffffu, tok >= q.x && tok < q.x + q.y);   // ranges do not overlap
  if (!who) return;
  const int r = __ffs(who) - 1;
  const int t0 = __shfl_sync(0xffffffffu, q.x, r), rt = (__shfl_sync(0xffffffffu, q.y, r) * A.grp + MT - 1) / MT;
  const int splits = __shfl_sync(0xffffffffu, q.z, r), base = __shfl_sync(0xffffffffu, q.w, r);
  if (splits == 1) return;
  const int m = (tok - t0) * A.grp + hd % A.grp, head = hd / A.grp;
  const int64_t first = ((int64_t)base + (int64_t)head * splits * rt + m / MT) * MT + m % MT, step = (int64_t)rt * MT;
  float M = -INFINITY, l = 0.f, o[V] = {};
  for (int s0 = warp % W; s0 < splits; s0 += 32 * W) {         // this warp's: s0, s0 + W, ..., 32 of them at most
    const int n = min(32, (splits - s0 + W - 1) / W);
    auto part = [&](int i, float (&v)[V]) {
      const float *p = A.part + (first + (int64_t)(s0 + W * i) * step) * DP + lane * V;
      if constexpr (V == 4) {
        const float4 u = __ldcg(reinterpret_cast<const float4 *>(p));
        v[0] = u.x; v[1] = u.y; v[2] = u.z; v[3] = u.w;
      } else {
        const float2 u = __ldcg(reinterpret_cast<const float2 *>(p));
        v[0] = u.x; v[1] = u.y;
      }
    };
    float v[AHEAD][V] = {};
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
      if (i < n) part(i, v[i]);
    float2 ml = make_float2(-INFINITY, 0.f);
    if (lane < n) ml = __ldcg(A.ml + first + (int64_t)(s0 + W * lane) * step);
    float top = ml.x;
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
    top = fmaxf(top, M);
    const float ref = top == -INFINITY ? 0.f : top, fix = exp2_fast(M - ref), f = exp2_fast(ml.x - ref);
    M = top;
    l = fmaf(l, fix, f * ml.y);                    // a lane's share
#pragma unroll
    for (int k = 0; k < V; ++k) o[k] *= fix;
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const float w = __shfl_sync(0xffffffffu, f, i);
      if (i < n) {
#pragma unroll
        for (int k = 0; k < V; ++k) o[k] = fmaf(w, v[i][k], o[k]);
      }
    }
#pragma unroll 8
    for (int i = AHEAD; i < n; ++i) {
      const float w = __shfl_sync(0xffffffffu, f, i);
      part(i, v[0]);
#pragma unroll
      for (int k = 0; k < V; ++k) o[k] = fmaf(w, v[0][k], o[k]);
    }
  }
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) l += __shfl_xor_sync(0xffffffffu, l, k);
  if (lane == 0) {
    s_m[warp] = M;
    s_l[warp] = l;
  }
#pragma unroll
  for (int k = 0; k < V; ++k) s_o[warp][lane * V + k] = o[k];
  if (W == 1) __syncwarp();
  else named_sync(1 + warp / W, 32 * W);
  const int w0 = warp / W * W;
  float top = s_m[w0], sum = 0.f;
#pragma unroll
  for (int w = 1; w < W; ++w) top = fmaxf(top, s_m[w0 + w]);
  const float ref = top == -INFINITY ? 0.f : top;
  float f[W];
#pragma unroll
  for (int w = 0; w < W; ++w) {
    f[w] = exp2_fast(s_m[w0 + w] - ref);
    sum = fmaf(f[w], s_l[w0 + w], sum);
  }
  for (int d = 2 * (threadIdx.x % (32 * W)); d < A.D; d += 64 * W) {
    float x = 0.f, y = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      x = fmaf(f[w], s_o[w0 + w][d], x);
      y = fmaf(f[w], s_o[w0 + w][d + 1], y);
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    *reinterpret_cast<uint32_t *>(A.o + (int64_t)row * A.D + d) = pack_h2(x * inv, y * inv);
  }
}

// One 16-byte chunk of a token's keys and values per thread.  A lane of every
// warp reads one request's range and length, all at once: the chain to the first
// store is two loads (these, then the table) instead of four.
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
  const int lane = threadIdx.x & 31;
  const int per = A.hkv * (A.D / 8), total = A.T * per;
  const int i = blockIdx.x * blockDim.x + threadIdx.x, at = min(i, total - 1);
  const int tok = at / per, head = at % per / (A.D / 8), c = at % (A.D / 8);
  const int64_t from = ((int64_t)tok * A.hkv + head) * A.D + c * 8;
  const uint4 key = *reinterpret_cast<const uint4 *>(A.kn + from), val = *reinterpret_cast<const uint4 *>(A.vn + from);
  int b0 = 0, b1 = A.T, n = 0;
  if (lane < A.R) {
    b0 = ld_cg_i32(A.begin + lane);
    b1 = ld_cg_i32(A.begin + lane + 1);
    n = ld_cg_i32(A.lens + lane);
  }
  const bool bad = __any_sync(0xffffffffu, b0 < 0 || b1 < b0 || b1 > A.T);
  if (bad && i == 0) flag_error(A.err, kErrIndex);
  int r = 0;                           // the request whose range holds the token
  for (int q = 0; q < A.R; ++q) r += tok >= __shfl_sync(0xffffffffu, b1, q);
  const int t0 = __shfl_sync(0xffffffffu, b0, r & 31), len = __shfl_sync(0xffffffffu, n, r & 31);
  if (i >= total || r >= A.R || tok < t0) return;   // behind the last range: nothing is written
  const int64_t pos = (int64_t)len + (tok - t0);
  const int64_t pi = pos / A.page;
  int id = -1;
  if (t0 >= 0 && len >= 0 && pi < A.max_pages) id = A.table[(int64_t)r * A.max_pages + pi];
  if ((unsigned)id >= (unsigned)A.pages) {
    flag_error(A.err, kErrIndex);
    return;
  }
  const int64_t to = (int64_t)id * A.page_stride + (pos - pi * A.page) * A.token_stride + (int64_t)head * A.head_stride + c * 8;
  *reinterpret_cast<uint4 *>(A.k + to) = key;
  *reinterpret_cast<uint4 *>(A.v + to) = val;
}

// ------------------------------------------------------------------ host --
asf_status check_cache(const asf_kv_cache *c) {
  if (!c || !c->k || !c->v) return ASF_ERR_INVALID_ARG;
  if (c->pages <= 0 || c->page <= 0 || c->heads <= 0 || c->head_dim <= 0) return ASF_ERR_INVALID_ARG;
  if (c->head_dim > 128 || c->heads > ASF_MAX_KV_HEADS) return ASF_ERR_UNSUPPORTED;
  if (c->head_dim % 8 || c->page_stride % 8 || c->token_stride % 8 || c->head_stride % 8) return ASF_ERR_MISALIGNED;
  if (!al16(c->k) || !al16(c->v)) return ASF_ERR_MISALIGNED;
  if (c->page_stride < 0 || c->token_stride < c->head_dim || c->head_stride < 0 ||
      (c->heads > 1 && c->head_stride < c->head_dim) || (c->pages > 1 && c->page_stride < c->head_dim))
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
  return rows <= 16 ? 1 : rows <= 32 ? 2 : 8;
}
int row_tiles_most(int grp, int R, int T, int wm) { return T * grp / (16 * wm) + R; }
int attn_dp(const asf_kv_cache *c) { return c->head_dim <= 64 ? 64 : 128; }
int attn_target(const asf_kv_cache *c, int wm) { return sm_count() * attn_resident(attn_dp(c), wm); }
size_t attn_scratch(const asf_kv_cache *c, int grp, int R, int T) {
  const int wm = row_groups(grp, R, T);
  const size_t rows = (size_t)attn_target(c, wm) * 16 * wm;   // more units than that: nothing is split
  return 512 + r256(rows * attn_dp(c) * 4) + r256(rows * 8);
}

// CTAs that share a unit (k_tree_attn), 1: no cluster, and splits with a merge
// from kWhole tiles on.  `keys` is what a request's table has room for, all that the
// host knows: a short request in a wide table takes no cluster.  A cluster where its CTAs find room at once and have
// few tiles each; eight CTAs where that leaves an SM to each.  us of the call
// with 1, 4 and 8: 8 heads x 200 keys 11.4, 9.4, 10.1; 500 keys 15.0, 10.2, 9.9;
// 1000 keys 13.8, 12.4, 10.9; 2000 keys 14.0, 16.8, 13.0; 32 heads x 333 keys
// 13.2, 10.7, 12.6; 1000 keys 15.3, 12.4, 13.2; 2000 keys 17.4, 17.9, 16.9.
int cluster_of(int64_t keys, int units, int target) {
  if (keys <= kTile) return 1;
  if (keys > 4 * kTile && keys <= 8 * kClusterTiles * kTile && units * 8 <= sm_count()) return 8;
  return keys <= 4 * kClusterTiles * kTile && units * 4 <= target ? 4 : 1;
}
template <int DP, int WM>
cudaError_t run_attn(const AttnArgs &a, int units, cudaStream_t st) {
  const size_t smem = (size_t)kStages * 2 * kTile * DP * 2;
  if (a.cluster == 8) return launch_clusters(k_tree_attn<DP, WM, 8>, dim3(units * 8), dim3(128), smem, st, 8, a);
  if (a.cluster == 4) return launch_clusters(k_tree_attn<DP, WM, 4>, dim3(units * 4), dim3(128), smem, st, 4, a);
  return launch(k_tree_attn<DP, WM, 1>, dim3(units), dim3(128), smem, st, a);
}
// Map of a cache's keys or values: columns, tokens of a page, heads, pages; a
// box is `box` tokens of one head and page by 64 columns, swizzled as the MMA
// reads it.  Columns past head_dim and pages past the last read as zeros.
bool cache_map(CUtensorMap *tm, const void *base, const AttnArgs &a) {
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

template <int DP>
cudaError_t run_tc(AttnArgs a, int units, cudaStream_t st) {
  CUtensorMap mk, mv;
  std::memset(&mk, 0, sizeof(mk));
  std::memset(&mv, 0, sizeof(mv));
  a.box = a.page >= kTile ? (a.page % kTile ? 0 : kTile) : a.page >= 8 && kTile % a.page == 0 ? a.page : 0;
  if (a.box && cache_map(&mk, a.k, a) && cache_map(&mv, a.v, a))
    return launch(k_tree_tc<DP, true>, dim3(units), dim3(kTcThreads), TreeTc<DP>::SMEM, st, mk, mv, a);
  return launch(k_tree_tc<DP, false>, dim3(units), dim3(kTcThreads), TreeTc<DP>::SMEM, st, mk, mv, a);
}

template <int DP>
cudaError_t run_attn_any(const AttnArgs &a, int wm, int units, cudaStream_t st) {
  const cudaError_t e = wm == 1   ? run_attn<DP, 1>(a, units, st)
                        : wm == 2 ? run_attn<DP, 2>(a, units, st)
                                  : run_tc<DP>(a, units, st);
  if (e != cudaSuccess) return e;
  if ((int64_t)a.max_pages * a.page <= a.whole * kTile) return e;       // no request can have splits
  const int rows = a.T * a.hkv * a.grp;
  // Four warps a row where that is a few CTAs an SM at most, else one.  us of the
  // whole call, one and four warps: 64 rows x 55 splits 42.9 and 35.8, 1024 rows
  // 69.9 and 64.2; 2048 rows x 6 splits 65.6 and 70.1, 4096 rows 32.8 and 36.5.
  return rows <= 8 * sm_count() ? launch(k_tree_merge<DP, 4, 16>, dim3(rows), dim3(128), 0, st, a, 16 * wm)
                                : launch(k_tree_merge<DP, 1, 8>, dim3((rows + 3) / 4), dim3(128), 0, st, a, 16 * wm);
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
  const size_t bytes = (size_t)T * q_heads * cache->head_dim * 2;
  if (overlap(q, bytes, o, bytes)) return ASF_ERR_INVALID_ARG;
  const int wm = row_groups(grp, R, T);
  const int64_t keys = (int64_t)max_pages * cache->page;
  int units = cache->heads * row_tiles_most(grp, R, T, wm);
  const int cluster = wm <= 2 ? cluster_of(keys, units, attn_target(cache, wm)) : 1;
  const int whole = cluster > 1 ? kClusterTiles * cluster : kWhole;
  if (keys > whole * kTile) units += attn_target(cache, wm);
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
  if (!std::isfinite(a.scale)) return ASF_ERR_INVALID_ARG;
  a.o = static_cast<__half *>(o);
  a.plan = reinterpret_cast<int4 *>(base);
  base += 512;
  a.part = reinterpret_cast<float *>(base);
  a.ml = reinterpret_cast<float2 *>(base + r256((size_t)attn_target(cache, wm) * 16 * wm * attn_dp(cache) * 4));
  a.target = attn_target(cache, wm);
  a.whole = whole;
  a.cluster = cluster;
  a.err = &static_cast<Header *>(ws)->err;
  cudaStream_t st = (cudaStream_t)stream;
  return cuda_status(attn_dp(cache) == 64 ? run_attn_any<64>(a, wm, units, st) : run_attn_any<128>(a, wm, units, st));
}

}  // extern "C"
