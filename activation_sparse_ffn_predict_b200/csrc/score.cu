// The attention weight that each cached key receives (include/asffn.h,
// asf_tree_attention_scored), after the attention itself.
//
// Mathematics.  scores[r][head][p] gains (is, for the call's own tokens) the sum over the
// request's rows of softmax_p.  The attention leaves every row's reference M and sum l
// (in units of log2, over scores that carry log2(e)); the weight of a score z is then
// 2^(z - M) / l, in fp32, and a key's rows are added in a fixed order.  Rows that saw
// nothing have l = 0 and add nothing.
//
// The kernels start while the attention's last kernel runs.  That one has passed its own
// dependency wait before it let them start, so what the call was given (requests, table,
// queries, keys, scores) is complete, and is read from L2; what it writes is read after
// the wait.  With `beside` the last kernel is the merge, and the sum reads only what is
// in front of that.  The wait comes before the end in any case: a grid's end is
// its predecessors' end, too.
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstring>

#include "asffn.h"
#include "attn.cuh"

using namespace asf;

namespace {

// What the attention has left for a row: for each split, or in stats where there is one.
struct Left {
  const float2 *first;
  int64_t step;
  int splits;
};
__device__ __forceinline__ Left left_of(const AttnArgs &A, int4 plan, int head, int m, int64_t row) {
  if (plan.z == 1) return {A.stats + row, 0, 1};
  const int rt = (plan.y * A.grp + A.mt - 1) / A.mt;
  return {A.ml + ((int64_t)plan.w + (int64_t)head * plan.z * rt + m / A.mt) * A.mt + m % A.mt, (int64_t)rt * A.mt, plan.z};
}
// (reference, 1 / sum) of parts (reference, sum)
__device__ __forceinline__ float2 join(float2 a, float2 b) {
  const float M = fmaxf(a.x, b.x), ref = M == -INFINITY ? 0.f : M;
  return make_float2(M, fmaf(exp2_fast(a.x - ref), a.y, exp2_fast(b.x - ref) * b.y));
}

// ---------------------------------------- the attention's own scores ----
// k_tree_attn has kept its scores: each is read once, a thread four keys, every row in turn.
// Latency bounds it, and HBM where the keys have pushed the scores out of L2: 8 requests
// of up to 16000 keys, 64 query heads, 62 us with the attention, 49.5 without (the keys
// read again by mma.sync: 139); one token, 32 heads, 333 keys 12.4 and 9.5.
constexpr int kSumKeys = 512;          // of a unit
constexpr int kSumThreads = 128;
constexpr int kSumRows = 64;           // whose references are in shared memory

__global__ void __launch_bounds__(kSumThreads) k_score_sum(AttnArgs A) {
  __shared__ float2 s_stat[kSumRows];  // reference, 1 / sum
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31;
  bool bad;
  const Req q = req_lane(A, 16, lane, bad);        // bad requests have been flagged
  const int parts = (q.L + kSumKeys - 1) / kSumKeys;
  int end = q.n ? parts * A.hkv : 0;
  const int own = end;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, end, o);
    if (lane >= o) end += v;
  }
  const int total = __shfl_sync(0xffffffffu, end, 31);
  if (!A.beside) pdl_wait();
  const int4 plans = __ldcg(A.plan + lane);
  for (int u = blockIdx.x; u < total; u += gridDim.x) {
    const int req = __popc(__ballot_sync(0xffffffffu, end <= u));
    const int in = u - __shfl_sync(0xffffffffu, end - own, req), np = __shfl_sync(0xffffffffu, parts, req);
    const int t0 = __shfl_sync(0xffffffffu, q.t0, req), rows = __shfl_sync(0xffffffffu, q.n, req) * A.grp;
    const int len = __shfl_sync(0xffffffffu, q.len, req), L = __shfl_sync(0xffffffffu, q.L, req);
    const int4 plan = make_int4(0, __shfl_sync(0xffffffffu, plans.y, req), __shfl_sync(0xffffffffu, plans.z, req),
                                __shfl_sync(0xffffffffu, plans.w, req));
    const int head = in / np, p0 = (in - head * np) * kSumKeys + 4 * tid;
    const bool there = p0 < L;                     // then its tile of 64 keys has scores, to the end
    float *scores = A.scores + ((int64_t)req * A.hkv + head) * A.S;
    float old[4], acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < 4; ++k) old[k] = p0 + k < len && p0 + k < A.S ? __ldcg(scores + p0 + k) : 0.f;
    const int64_t hop = (int64_t)(A.hkv - 1) * A.grp * A.zs;             // from a token's last row to the next token's first
    for (int m0 = 0; m0 < rows; m0 += kSumRows) {
      const int n = min(kSumRows, rows - m0);
      __syncthreads();
      auto put = [&](int i, float2 st) { s_stat[i] = st.y == 0.f ? make_float2(0.f, 0.f) : make_float2(st.x, 1.f / st.y); };
      auto row_of = [&](int m) { return (int64_t)(t0 + m / A.grp) * A.hkv * A.grp + head * A.grp + m % A.grp; };
      if (!A.beside) {
        if (tid < n) put(tid, __ldcg(A.stats + row_of(m0 + tid)));
      } else {
        // a warp a row, a lane a split (or every 32nd)
        for (int i = tid >> 5; i < n; i += kSumThreads / 32) {
          const Left left = left_of(A, plan, head, m0 + i, row_of(m0 + i));
          float2 st = make_float2(-INFINITY, 0.f);
          for (int p = lane; p < left.splits; p += 32) st = join(st, __ldcg(left.first + p * left.step));
#pragma unroll
          for (int o = 16; o > 0; o >>= 1)
            st = join(st, make_float2(__shfl_xor_sync(0xffffffffu, st.x, o), __shfl_xor_sync(0xffffffffu, st.y, o)));
          if (lane == 0) put(i, st);
        }
      }
      int tok = m0 / A.grp, g = m0 - tok * A.grp;
      const float *z = A.z + ((int64_t)(t0 + tok) * A.hkv * A.grp + head * A.grp + g) * A.zs + p0;
      constexpr int U = 8;                         // rows in flight
      for (int i = 0; i < n; i += U) {
        float4 v[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
          v[k] = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
          if (i + k < n && there) v[k] = __ldcg(reinterpret_cast<const float4 *>(z));
          z += A.zs;
          if (++g == A.grp) {
            g = 0;
            z += hop;
          }
        }
        if (i == 0) __syncthreads();               // the references are there
#pragma unroll
        for (int k = 0; k < U; ++k) {
          const float2 st = s_stat[min(i + k, n - 1)];
          const float w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float x = exp2_fast(w[e] - st.x);
            acc[e] = w[e] != -INFINITY ? fmaf(x, st.y, acc[e]) : acc[e];
          }
        }
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int p = p0 + k;
      if (p >= L) continue;
      if (p >= A.S) flag_error(A.err, kErrIndex);
      else scores[p] = old[k] + acc[k];
    }
  }
  if (A.beside) pdl_wait();
}

// ------------------------------------- keys again, any page size: mma.sync --
// For pages that TMA does not take in whole tiles.  A tile of 64 keys is multiplied with
// all of the request's rows, 16 at a time, a warp every fourth group of them.  16 tokens x 64 heads over 65500 keys
// in pages of 20: 302 us with the attention, 82 without (in pages of 64, k_score_tc, 97): the exponentials and
// one tile in flight a CTA, whose loads nothing overlaps.
template <int DP>
__global__ void __launch_bounds__(128) k_tree_score(AttnArgs A) {
  constexpr int CH = DP / 8;
  __shared__ __align__(128) unsigned char sk[kTile * DP * 2];
  __shared__ float s_sum[4][kTile];
  __shared__ int64_t s_off[kTile];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  bool bad;
  const Req q = req_lane(A, 16, lane, bad);                              // bad requests have been flagged
  int64_t end = q.n ? (int64_t)q.nkt * A.hkv : 0;                        // this request's tiles, all heads
  const int64_t own = end;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, end, o);
    if (lane >= o) end += v;
  }
  const int64_t total = __shfl_sync(0xffffffffu, end, 31);
  for (int64_t u = blockIdx.x; u < total; u += gridDim.x) {
    const int req = __popc(__ballot_sync(0xffffffffu, end <= u));
    const int64_t in = u - __shfl_sync(0xffffffffu, end - own, req);
    const int nkt = __shfl_sync(0xffffffffu, q.nkt, req);
    const int t0 = __shfl_sync(0xffffffffu, q.t0, req), n = __shfl_sync(0xffffffffu, q.n, req);
    const int len = __shfl_sync(0xffffffffu, q.len, req), L = __shfl_sync(0xffffffffu, q.L, req);
    const int head = (int)(in / nkt), pos0 = (int)(in - (int64_t)head * nkt) * kTile, rows = n * A.grp;
    if (tid < kTile) {
      const int pos = pos0 + tid;
      int64_t off = -1;
      if (pos < L) {
        const int id = A.table[(int64_t)req * A.max_pages + pos / A.page];
        if ((unsigned)id < (unsigned)A.pages)
          off = (int64_t)id * A.page_stride + (int64_t)(pos % A.page) * A.token_stride + (int64_t)head * A.head_stride;
      }
      s_off[tid] = off;
    }
    __syncthreads();
    for (int i = tid >> 3; i < kTile; i += 16) {
      const int64_t off = s_off[i];
#pragma unroll
      for (int c = tid & 7; c < CH; c += 8) {
        const bool in_row = off >= 0 && c * 8 < A.D;
        cp_async16(sk + i * DP * 2 + ((c ^ (i & 7)) * 16), A.k + (in_row ? off + c * 8 : 0), in_row ? 16u : 0u);
      }
    }
    cp_async_commit();
    cp_async_wait<0>();
    __syncthreads();
    const bool special = pos0 + kTile > len;
    float acc[kTile / 8][2];
#pragma unroll
    for (int i = 0; i < kTile / 8; ++i) acc[i][0] = acc[i][1] = 0.f;
    const uint32_t kb = smem_u32(sk);
    for (int m0 = warp * 16; m0 < rows; m0 += 64) {
      uint32_t qf[DP / 16][4], see[2];
      float M[2], inv[2];
      const __half *qp[2];
      bool live[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int m = m0 + g + 8 * h;
        live[h] = m < rows;
        const int tok = t0 + (live[h] ? m / A.grp : 0);
        const int64_t row = (int64_t)tok * A.hkv * A.grp + head * A.grp + (live[h] ? m % A.grp : 0);
        see[h] = live[h] ? (uint32_t)A.anc[tok] : 0u;
        qp[h] = A.q + row * A.D;
        const float2 st = __ldcg(A.stats + row);
        const bool none = !live[h] || st.y == 0.f;
        M[h] = none ? INFINITY : st.x;
        inv[h] = none ? 0.f : 1.f / st.y;
      }
#pragma unroll
      for (int s = 0; s < DP / 16; ++s)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c = s * 16 + 2 * t + 8 * (i >> 1);
          qf[s][i] = live[i & 1] && c < A.D ? *reinterpret_cast<const uint32_t *>(qp[i & 1] + c) : 0u;
        }
      float z[kTile / 8][4];
#pragma unroll
      for (int i = 0; i < kTile / 8; ++i) z[i][0] = z[i][1] = z[i][2] = z[i][3] = 0.f;
#pragma unroll
      for (int s = 0; s < DP / 16; ++s)
#pragma unroll
        for (int i = 0; i < kTile / 16; ++i) {
          uint32_t b[4];
          const int row = i * 16 + (lane >> 4) * 8 + (lane & 7), c = s * 2 + ((lane >> 3) & 1);
          ldsm4(b, kb + row * DP * 2 + ((c ^ (row & 7)) * 16));
          mma_f16(z[2 * i], qf[s], b[0], b[1]);
          mma_f16(z[2 * i + 1], qf[s], b[2], b[3]);
        }
#pragma unroll
      for (int i = 0; i < kTile / 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int key = i * 8 + 2 * t + (e & 1), d = pos0 + key - len, h = e >> 1;
          const bool ok = live[h] && (!special || (s_off[key] >= 0 && (d < 0 || ((see[h] >> ((t0 + d) & 31)) & 1u))));
          const float w = exp2_fast(fmaf(z[i][e], A.scale, -M[h]));
          acc[i][e & 1] = ok ? fmaf(w, inv[h], acc[i][e & 1]) : acc[i][e & 1];
        }
    }
#pragma unroll
    for (int i = 0; i < kTile / 8; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) acc[i][e] += __shfl_xor_sync(0xffffffffu, acc[i][e], o);
        if (g == 0) s_sum[warp][i * 8 + 2 * t + e] = acc[i][e];
      }
    __syncthreads();
    if (tid < kTile && pos0 + tid < L) {
      const int pos = pos0 + tid;
      if (pos >= A.S) {
        flag_error(A.err, kErrIndex);
      } else {
        float *to = A.scores + ((int64_t)req * A.hkv + head) * A.S + pos;
        const float w = s_sum[0][tid] + s_sum[1][tid] + s_sum[2][tid] + s_sum[3][tid];
        if (pos >= len) *to = w;
        else if (s_off[tid] >= 0) *to += w;
      }
    }
  }
}

// --------------------------------------------- keys again, tcgen05 ---------
// For many rows.  S^T = K Q^T: a tile of 128 keys is the M of the product and the
// request's rows are its N, 64 at a time, so that a thread of the softmax warps has a key
// and adds its rows up without meeting another thread.
//   warp 4     copies tiles of 128 keys by TMA, a load per page and 64 columns
//   warps 6, 7 a thread a row: its query, reference, 1 / sum and mask, into one of two
//              slots; up to 128 rows stay there, more go round for every two tiles
//   warp 5     one thread issues the products into one of four accumulators
//   warps 0-3  read the accumulators of two tiles, hand them back, and add up 2^(z - M) / l:
//              with two keys a thread, a reference read from shared memory serves both
// A CTA takes a run of tiles of one kv head; two CTAs share an SM.  16 tokens x 64 heads
// over 65500 keys (134 MB of keys): 97 us with the attention, 63 without (276 with
// mma.sync).  From 16000 keys on a key costs what HBM takes for it (6.2 TB/s); what bounds
// it below, and adds to it above, are 10 us of start, merge and end.
// 32 columns of this thread's tensor-memory lane, and the wait that makes them usable
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, "
      "[%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]),
        "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]),
        "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(taddr)
      : "memory");
}

template <int DP>
struct ScoreTc {
  static constexpr int KEYS = 128, ROWS = 64;
  static constexpr int K = KEYS * DP * 2, Q = ROWS * DP * 2;
  static constexpr int NS = DP == 128 ? 2 : 4;     // slots of keys
  static constexpr int BAR = 1024, STAT = 2 * ROWS * 12;
  static constexpr size_t SMEM = 1024 + BAR + STAT + 512 + 2 * Q + NS * K;
  static constexpr int NB = 4;                     // accumulators, ROWS columns each
  static constexpr uint32_t COLS = NB * ROWS;
};
constexpr int kScoreThreads = 8 * 32;

template <int DP>
__global__ void __launch_bounds__(kScoreThreads, 2) k_score_tc(const __grid_constant__ CUtensorMap map_k, AttnArgs A) {
  using Lc = ScoreTc<DP>;
  constexpr int NS = Lc::NS, KEYS = Lc::KEYS, ROWS = Lc::ROWS, NB = Lc::NB, CH = DP / 8;
  extern __shared__ unsigned char smem_raw[];
  __shared__ int s_unit[9];
  unsigned char *smem = align_1024(smem_raw);
  uint64_t *full_k = reinterpret_cast<uint64_t *>(smem), *empty_k = full_k + NS;
  uint64_t *full_q = empty_k + NS, *empty_q = full_q + 2, *bs = empty_q + 2, *be = bs + NB;
  uint32_t *tslot = reinterpret_cast<uint32_t *>(be + NB);
  unsigned char *sq = smem + Lc::BAR, *sk = sq + 2 * Lc::Q;
  float4 *s_stat = reinterpret_cast<float4 *>(sk + NS * Lc::K);           // [2][ROWS / 2]: two rows' references and 1 / sums
  uint32_t *s_see = reinterpret_cast<uint32_t *>(s_stat + ROWS);          // [2][ROWS]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(&full_k[i], 1);
      mbar_init(&empty_k[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&full_q[i], 64);
      mbar_init(&empty_q[i], 1 + 128);             // the products, and the threads that read the references
    }
    for (int i = 0; i < NB; ++i) {
      mbar_init(&bs[i], 1);
      mbar_init(&be[i], 128);
    }
    fence_mbar_init();
    prefetch_map(&map_k);
  }
  if (warp == 5) {
    tmem_alloc(tslot, Lc::COLS);
    tmem_relinquish();
  }
  pdl_trigger();
  if (warp == 0) {
    // C tiles a unit, the fewest for which the units fit `target` CTAs (one unit a kv head where even that is more)
    bool bad;
    const Req q = req_lane(A, ROWS, lane, bad);
    const int nkt = q.n ? (q.L + KEYS - 1) / KEYS : 0;
    int64_t W = nkt;
    int most = nkt;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      W += __shfl_xor_sync(0xffffffffu, W, o);
      most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
    }
    int C = max(1, (int)((W * A.hkv + A.target - 1) / A.target)), base, splits, mine;
    while (true) {
      splits = (nkt + C - 1) / C;
      mine = splits * A.hkv;
      int u = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, u, o);
        if (lane >= o) u += v;
      }
      base = u - mine;
      if (__shfl_sync(0xffffffffu, u, 31) <= A.target || C >= most) break;
      C += max(1, C / 16);
    }
    const int u = (int)blockIdx.x - base;
    if (lane == 0) s_unit[0] = -1;
    __syncwarp();
    if (u >= 0 && u < mine) {
      const int s = u % splits;
      s_unit[0] = lane;
      s_unit[1] = u / splits;                      // kv head
      s_unit[2] = s * C;
      s_unit[3] = min(nkt, (s + 1) * C);
      s_unit[4] = q.t0;
      s_unit[5] = q.n;
      s_unit[6] = q.len;
      s_unit[7] = q.L;
      s_unit[8] = q.rt;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tslot;
  const int req = s_unit[0];
  if (req < 0) {
    if (warp == 5) tmem_dealloc(tbase, Lc::COLS);
    pdl_wait();
    return;
  }
  const int head = s_unit[1], kt1 = s_unit[3], tiles = kt1 - s_unit[2];   // from the last tile on: the attention read it last
  const int t0 = s_unit[4], n = s_unit[5], len = s_unit[6], L = s_unit[7], rt = s_unit[8];
  const int rows = n * A.grp;
  const bool stay = rt <= 2;                       // the rows stay in their slots
  // step i: the i / rt-th two tiles with the rows of group i % rt; the rows' slot and the parity of its filling
  auto slot_of = [&](int i, int g) { return stay ? g : i & 1; };
  auto fill_of = [&](int i) { return stay ? 0u : (uint32_t)(i >> 1) & 1u; };
  const int twos = (tiles + 1) / 2;

  if (warp == 4) {
    // ------------------------------------------------------------------ keys --
    const int nb = KEYS / A.box;
    auto page_of = [&](int j, int &tok) {          // lane b: box b of tile j
      const int pos = (kt1 - 1 - j) * KEYS + lane * A.box;
      tok = -1;
      if (j >= tiles || lane >= nb || pos >= L) return -1;
      const int pi = pos / A.page;
      tok = pos - pi * A.page;
      return __ldcg(A.table + (int64_t)req * A.max_pages + pi);
    };
    bool ok = true;
    int tok, id = page_of(0, tok);
    for (int j = 0; j < tiles; ++j) {
      const int sl = j % NS, at = tok, now = tok >= 0 && (unsigned)id < (unsigned)A.pages ? id : -1;
      id = page_of(j + 1, tok);
      if (j >= NS) {
        ok = warp_wait(&empty_k[sl], (uint32_t)((j / NS) - 1) & 1u, kTcWaitNs);
        if (!ok) {
          // what is on its way lands before the shared memory is given back
          for (int e = j - NS; e < j; ++e) warp_wait(&full_k[e % NS], (uint32_t)(e / NS) & 1u, kTcWaitNs);
          break;
        }
      }
      if (lane == 0) mbar_arrive_expect_tx(&full_k[sl], Lc::K);
      __syncwarp();
      if (lane < nb) {
#pragma unroll
        for (int h = 0; h < DP / 64; ++h)          // a page that is not there: outside the map, zeros
          tma_load_4d(sk + (size_t)sl * Lc::K + h * (KEYS * 128) + lane * A.box * 128, &map_k, 64 * h, now >= 0 ? at : 0, head,
                      now >= 0 ? now : A.pages, &full_k[sl]);
      }
      __syncwarp();
    }
    if (!ok) flag_error(A.err, kErrTimeout);
  } else if (warp >= 6) {
    // ------------------------------------------------------------------ rows --
    const int r = tid - 6 * 32;
    bool ok = true;
    const int fills = stay ? rt : twos * rt;
    for (int i = 0, g = 0; i < fills; ++i) {
      const int sl = slot_of(i, g), m = g * ROWS + r;
      if (!stay && i >= 2) {
        ok = warp_wait(&empty_q[sl], (uint32_t)((i >> 1) - 1) & 1u, kTcWaitNs);
        if (!ok) break;
      }
      const bool live = m < rows;
      const int tok = t0 + (live ? m / A.grp : 0);
      const int64_t row = (int64_t)tok * A.hkv * A.grp + head * A.grp + (live ? m % A.grp : 0);
      const __half *src = A.q + row * A.D;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const bool in = live && c * 8 < A.D;
        cp_async16(sq + (size_t)sl * Lc::Q + (c >> 3) * (ROWS * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4), in ? src + c * 8 : A.q,
                   in ? 16u : 0u);
      }
      cp_async_commit();
      const uint32_t see = live ? (uint32_t)__ldcg(A.anc + tok) >> t0 : 0u;
      if (i == 0) pdl_wait();
      const float2 st = __ldcg(A.stats + row);
      const bool none = !live || st.y == 0.f;
      reinterpret_cast<float2 *>(s_stat + sl * (ROWS / 2))[r] = make_float2(none ? INFINITY : st.x, none ? 0.f : 1.f / st.y);
      s_see[sl * ROWS + r] = see;
      cp_async_wait<0>();
      fence_proxy_async_smem();
      mbar_arrive(&full_q[sl]);
      if (++g == rt) g = 0;
    }
    if (!ok) flag_error(A.err, kErrTimeout);
  } else if (warp == 5) {
    // ------------------------------------------------------------------- MMA --
    constexpr uint32_t idesc = umma_idesc_f16(KEYS, ROWS, 0, 0);
    const uint64_t dk = umma_desc(sk, 16, 1024, kSwz128), dq = umma_desc(sq, 16, 1024, kSwz128);
    bool ok = true;
    for (int two = 0, i = 0; two < twos && ok; ++two) {
      const int there = min(2, tiles - 2 * two);
      for (int g = 0; g < rt && ok; ++g, ++i) {
        const int qs = slot_of(i, g);
        ok = warp_wait(&full_q[qs], fill_of(i), kTcWaitNs);
        for (int h = 0; h < there && ok; ++h) {
          const int j = 2 * two + h, ks = j % NS, use = 2 * i + h, b = use % NB;
          if (g == 0) ok = warp_wait(&full_k[ks], (uint32_t)(j / NS) & 1u, kTcWaitNs);
          if (ok && use >= NB) ok = warp_wait(&be[b], (uint32_t)((use / NB) - 1) & 1u, kTcWaitNs);
          if (!ok) break;
          tc_fence_after();
          const uint64_t ak = dk + (uint64_t)(ks * (Lc::K >> 4)), bq = dq + (uint64_t)(qs * (Lc::Q >> 4));
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < DP / 16; ++k)
              umma_f16(tbase + b * ROWS, ak + ((k >> 2) * (KEYS * 128) + (k & 3) * 32) / 16,
                       bq + ((k >> 2) * (ROWS * 128) + (k & 3) * 32) / 16, idesc, k != 0);
            umma_commit(&bs[b]);
            if (!stay && h == there - 1) umma_commit(&empty_q[qs]);
            if (g == rt - 1) umma_commit(&empty_k[ks]);
          }
          __syncwarp();
        }
      }
    }
    if (!ok && lane == 0) flag_error(A.err, kErrTimeout);
  } else {
    // --------------------------------------------------------------- weights --
    const uint32_t tl = tbase + ((uint32_t)(32 * warp) << 16);
    float *scores = A.scores + ((int64_t)req * A.hkv + head) * A.S;
    bool ok = true;
    for (int two = 0, i = 0; two < twos && ok; ++two) {
      const int there = min(2, tiles - 2 * two);
      int pos[2], d[2], id[2] = {-1, -1};
      float old[2] = {0.f, 0.f}, acc[2][2] = {{0.f, 0.f}, {0.f, 0.f}};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        pos[h] = (kt1 - 1 - 2 * two - h) * KEYS + tid;
        d[h] = pos[h] - len;
        if (h >= there) pos[h] = L;                // the other accumulator holds what it held
        if (pos[h] < L) {
          id[h] = __ldcg(A.table + (int64_t)req * A.max_pages + pos[h] / A.page);
          if (d[h] < 0 && pos[h] < A.S) old[h] = __ldcg(scores + pos[h]);
        }
      }
      const bool special = (kt1 - 2 * two) * KEYS > len;
      for (int g = 0; g < rt; ++g, ++i) {
        const int b = 2 * i % NB, sl = slot_of(i, g), live = rows - g * ROWS;
        const uint32_t done = (uint32_t)(2 * i / NB) & 1u;
        ok = warp_wait(&full_q[sl], fill_of(i), kTcWaitNs);
        if (ok) ok = warp_wait(&bs[b], done, kTcWaitNs);
        if (ok && there == 2) ok = warp_wait(&bs[b + 1], done, kTcWaitNs);
        if (!ok) break;
        tc_fence_after();
        __syncwarp();
#pragma unroll
        for (int c = 0; c < ROWS; c += 32) {
          float z[2][32];
          tmem_ld32(tl + b * ROWS + c, z[0]);
          tmem_ld32(tl + (b + 1) * ROWS + c, z[1]);
          if (c + 32 == ROWS) {
            tc_fence_before();
            mbar_arrive(&be[b]);
            mbar_arrive(&be[b + 1]);
          }
          const float4 *st = s_stat + sl * (ROWS / 2) + c / 2;
          if (!special && live >= c + 32) {
#pragma unroll
            for (int m = 0; m < 32; m += 2) {
              const float4 u = st[m / 2];
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                acc[h][0] = fmaf(exp2_fast(fmaf(z[h][m], A.scale, -u.x)), u.y, acc[h][0]);
                acc[h][1] = fmaf(exp2_fast(fmaf(z[h][m + 1], A.scale, -u.z)), u.w, acc[h][1]);
              }
            }
          } else {
            const uint32_t *see = s_see + sl * ROWS + c;
#pragma unroll
            for (int m = 0; m < 32; ++m) {
              const float2 u = reinterpret_cast<const float2 *>(st)[m];
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const float w = exp2_fast(fmaf(z[h][m], A.scale, -u.x));
                const bool sees = d[h] < 0 || (d[h] < 32 && (see[m] >> d[h]) & 1u);
                if (c + m < live && sees) acc[h][m & 1] = fmaf(w, u.y, acc[h][m & 1]);
              }
            }
          }
          __syncwarp();
        }
        if (!stay) mbar_arrive(&empty_q[sl]);
      }
      if (!ok) break;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (pos[h] >= L) continue;
        const float w = acc[h][0] + acc[h][1];
        if (pos[h] >= A.S) flag_error(A.err, kErrIndex);
        else if (d[h] >= 0) scores[pos[h]] = (unsigned)id[h] < (unsigned)A.pages ? w : 0.f;
        else if ((unsigned)id[h] < (unsigned)A.pages) scores[pos[h]] = old[h] + w;
      }
    }
    if (!ok && lane == 0) flag_error(A.err, kErrTimeout);
  }
  pdl_wait();
  tc_fence_before();
  __syncthreads();
  if (warp == 5) {
    tc_fence_after();
    tmem_dealloc(tbase, Lc::COLS);
  }
}

template <int DP>
cudaError_t run_scores_dp(AttnArgs a, cudaStream_t st) {
  const int64_t keys = (int64_t)a.max_pages * a.page, heads = (int64_t)a.R * a.hkv;
  if (a.z) {
    const int64_t parts = heads * ((keys + kSumKeys - 1) / kSumKeys);
    return launch(k_score_sum, dim3((unsigned)std::min<int64_t>(parts, 8 * sm_count())), dim3(kSumThreads), 0, st, a);
  }
  a.box = tma_box(a.page);
  a.target = 2 * sm_count();
  CUtensorMap mk;
  std::memset(&mk, 0, sizeof(mk));
  if (a.box && cache_map(&mk, a.k, a))
    return launch(k_score_tc<DP>, dim3((unsigned)std::max<int64_t>(std::min<int64_t>(a.target, heads * ((keys + 127) / 128)), heads)),
                  dim3(kScoreThreads), ScoreTc<DP>::SMEM, st, mk, a);
  const int64_t tiles = heads * ((keys + kTile - 1) / kTile);
  return launch(k_tree_score<DP>, dim3((unsigned)std::min<int64_t>(tiles, 8 * sm_count())), dim3(128), 0, st, a);
}

}  // namespace

namespace asf {
cudaError_t run_scores(AttnArgs a, cudaStream_t st) { return a.D <= 64 ? run_scores_dp<64>(a, st) : run_scores_dp<128>(a, st); }
}  // namespace asf
