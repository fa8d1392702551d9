// Low-rank adapters of many tokens beside a 4-bit product that they share
// (include/asffn.h, "Adapters").
//
//   asf_w4_matmul_lora    k_lora_down, the product of asf_w4_matmul, k_lora_up
//
// Mathematics.  y = act(W x + bias + s_a B_a (A_a x)) with a token's own adapter a:
// h = s_a A_a x has `rank` values, kept in fp32, and so is W x, so that y is rounded
// once.  Both steps read each adapter in use once: the first token of the call that
// has it (its leader) takes all of its tokens along, four at a time.  A token's sums
// are added in the same order whoever comes along, and however many.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "asffn.h"
#include "common.cuh"
#include "host.cuh"

using namespace asf;

namespace {

constexpr int kDownThreads = 128;
constexpr int kUpThreads = 128;
constexpr int kUpCtas = 3;             // of an SM, where its shared memory holds them
constexpr int kUpStages = 4, kUpStage = 16 * 1024;
constexpr int kUpRows = 256;           // of a stage at most
// Dynamic shared memory with which kUpCtas of them are on an SM: beside it each has its static part and 1 KB that
// the system keeps (28672 x 8192, 22 tokens of as many adapters of rank 128, 75 KB: 99 us with two CTAs an SM,
// 111 with three, of which the third waits).
constexpr size_t kUpShared = 228 * 1024 / kUpCtas - 1024 - 512;
constexpr int kAlong = 4;              // tokens at a time
constexpr uint64_t kUpWaitNs = 200ull * 1000 * 1000;   // bound on any mbarrier wait

struct LoraArgs {
  int adapters, rank, k, rows, B;
  const void *A, *Bm;                  // [adapters][rank][k], [adapters][rows][rank]
  const float *scale;                  // [adapters], or null: 1
  const int32_t *which;                // [B]
  const void *x;
  float *h;                            // [B][rank]
  const float *base;                   // [B][rows]: W x + bias
  void *y;
  int y16, relu;
  int32_t *err;
};

// The tokens that use token b's adapter, if b is the first of them; 0 else.  a: the
// adapter, -1 without one.  Whole warps call it.
__device__ __forceinline__ uint32_t led_by(const LoraArgs &A, int b, int &a) {
  const int lane = threadIdx.x & 31;
  int w = -1;
  if (lane < A.B) {
    w = ld_cg_i32(A.which + lane);
    if (w >= A.adapters) {
      flag_error(A.err, kErrIndex);
      w = -1;
    }
    w = max(w, -1);
  }
  a = __shfl_sync(0xffffffffu, w, b);
  const uint32_t all = __ballot_sync(0xffffffffu, lane < A.B && w == a);
  return __ffs(all) - 1 == b ? all : 0u;
}
// the next (up to) NB tokens of a set, the last one again where there are fewer
template <int NB>
__device__ __forceinline__ int take(uint32_t &set, int (&tok)[NB]) {
  int n = 0;
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    if (set) {
      tok[i] = __ffs(set) - 1;
      set &= set - 1;
      ++n;
    } else {
      tok[i] = i ? tok[i - 1] : 0;
    }
  }
  return n;
}

// v[i] summed over the warp; lane l is left with the sum of v[i] for i = l / (32 / N)
// in the order 16, 8, 4, 2, 1 of lanes, which is every N's.
template <int N>
__device__ __forceinline__ float warp_sums(float (&v)[N]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int n = N / 2, o = 16; n > 0; n /= 2, o /= 2) {
    const bool hi = lane & o;
#pragma unroll
    for (int i = 0; i < N / 2; ++i)
      if (i < n) {
        const float keep = hi ? v[i + n] : v[i], give = hi ? v[i] : v[i + n];
        v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
      }
  }
#pragma unroll
  for (int o = 16 / N; o > 0; o >>= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
  return v[0];
}

template <typename T, int RW, int NB>
__device__ __forceinline__ void down_rows(const LoraArgs &A, int a, int row0, uint32_t &set, float *s_red) {
  constexpr int E = Vec<T>::N;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int tok[NB];
  const int n = take<NB>(set, tok);
  const T *w = static_cast<const T *>(A.A) + ((int64_t)a * A.rank + row0) * A.k;
  const T *x = static_cast<const T *>(A.x);
  float acc[RW * NB];
#pragma unroll
  for (int i = 0; i < RW * NB; ++i) acc[i] = 0.f;
#pragma unroll(NB == 1 ? 4 : NB == 2 && RW == 4 ? 2 : NB == 2 ? 4 : RW == 4 ? 2 : 1)
  for (int i = tid * E; i < A.k; i += kDownThreads * E) {
    uint4 wv[RW], xv[NB];
#pragma unroll
    for (int r = 0; r < RW; ++r) wv[r] = __ldcg(reinterpret_cast<const uint4 *>(w + (int64_t)r * A.k + i));
#pragma unroll
    for (int b = 0; b < NB; ++b) xv[b] = __ldcg(reinterpret_cast<const uint4 *>(x + (int64_t)tok[b] * A.k + i));
#pragma unroll
    for (int r = 0; r < RW; ++r)
#pragma unroll
      for (int b = 0; b < NB; ++b) acc[r * NB + b] = Vec<T>::dot(wv[r], xv[b], acc[r * NB + b]);
  }
  constexpr int N = RW * NB, SPAN = 32 / N;
  const float v = warp_sums<N>(acc);
  __syncthreads();                     // the last sums have been read
  if (lane % SPAN == 0) s_red[warp * N + lane / SPAN] = v;
  __syncthreads();
  if (tid < N && tid % NB < n) {
    float sum = 0.f;
#pragma unroll
    for (int q = 0; q < kDownThreads / 32; ++q) sum += s_red[q * N + tid];
    const float s = A.scale ? __ldcg(A.scale + a) : 1.f;
    int t = tok[0];
#pragma unroll
    for (int b = 1; b < NB; ++b) t = tid % NB == b ? tok[b] : t;
    __stcg(A.h + (int64_t)t * A.rank + row0 + tid / NB, s * sum);
  }
}

// h = s A x: a CTA is RW rows of the adapter that its token leads, over all of k.  Four
// rows where those are a CTA an SM (x is read once for them), else one, in few registers, so
// that it finds room beside a product that leaves some (k_w4_dot).  24 adapters of rank 64 over
// 8192 columns, 25 MB: 12 us alone, 2.0 TB/s: the loads of 2.6 CTAs an SM in flight.
template <typename T, int RW>
__global__ void __launch_bounds__(kDownThreads, RW == 1 ? 8 : 4) k_lora_down(LoraArgs A) {
  __shared__ float s_red[kDownThreads / 32 * RW * kAlong];
  pdl_trigger();
  int a;
  uint32_t set = led_by(A, blockIdx.y, a);
  const int row0 = blockIdx.x * RW;    // rank is a multiple of 8
  while (set && a >= 0) {
    const int left = __popc(set);
    if (left > 2) down_rows<T, RW, 4>(A, a, row0, set, s_red);
    else if (left > 1) down_rows<T, RW, 2>(A, a, row0, set, s_red);
    else down_rows<T, RW, 1>(A, a, row0, set, s_red);
  }
  pdl_wait();
}

__device__ __forceinline__ void put(const LoraArgs &A, int64_t at, float v) {
  if (A.relu) v = v > 0.f ? v : (v != v ? v : 0.f);
  if (A.y16) static_cast<__half *>(A.y)[at] = __float2half_rn(v);
  else static_cast<float *>(A.y)[at] = v;
}
__device__ __forceinline__ void eight(const __half *p, float (&v)[8]) {
  Vec<__half>::to_float(*reinterpret_cast<const uint4 *>(p), v);
}
__device__ __forceinline__ void eight(const float *p, float (&v)[8]) {
  const float4 a = *reinterpret_cast<const float4 *>(p), b = *(reinterpret_cast<const float4 *>(p) + 1);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

// The next NB of the leader's tokens (`set`) over `rows` rows of B in
// shared memory, a thread a row.  s_h: [token][2][rank / 2], the first four values of each
// eight ranks and the last four.  A thread begins with its own eight ranks, so that eight
// neighbours' 16 bytes of rows that lie a multiple of 128 bytes apart are in different banks;
// which they are goes by the row of the matrix, so that a row's sum has one order in every tiling.
template <typename T, int NB>
__device__ __forceinline__ void up_tokens(const LoraArgs &A, const T *w, int row0, int rows, const float *s_h, uint32_t &set) {
  int tok[NB];
  const int n = take<NB>(set, tok), eights = A.rank / 8;
  const int g = eights & -eights, rot = ((row0 + threadIdx.x) & 7) * min(g, 8) >> 3;
  static_assert(kUpThreads % 8 == 0, "a thread's rows begin alike");
  for (int row = threadIdx.x; row < rows; row += kUpThreads) {
    float base[NB], acc[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      base[b] = b < n ? __ldcg(A.base + (int64_t)tok[b] * A.rows + row0 + row) : 0.f;   // on its way while the sum is made
      acc[b] = 0.f;
    }
    const T *wr = w + row * A.rank;
    int c = rot;
#pragma unroll 4
    for (int i = 0; i < eights; ++i) {
      float v[8];
      eight(wr + c * 8, v);
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const float *h = s_h + (b < n ? b : 0) * A.rank + c * 4;
        const float4 p = *reinterpret_cast<const float4 *>(h), q = *reinterpret_cast<const float4 *>(h + A.rank / 2);
        float d = v[0] * p.x;
        d = fmaf(v[1], p.y, d);
        d = fmaf(v[2], p.z, d);
        d = fmaf(v[3], p.w, d);
        d = fmaf(v[4], q.x, d);
        d = fmaf(v[5], q.y, d);
        d = fmaf(v[6], q.z, d);
        d = fmaf(v[7], q.w, d);
        acc[b] += d;
      }
      if (++c == eights) c = 0;
    }
#pragma unroll
    for (int b = 0; b < NB; ++b)
      if (b < n) put(A, (int64_t)tok[b] * A.rows + row0 + row, base[b] + acc[b]);
  }
}

// y = act(base + B h).  The (adapter in use, tile of its rows) pairs are dealt out in one
// run of equal lengths per CTA, which streams its tiles, whole runs of memory, through a
// ring of bulk copies; the first of them are issued before the wait.  24 adapters of rank
// 64 over 28672 rows, 88 MB: 24 us alone, 3.7 TB/s; with the product and k_lora_down 77
// (lanes along a row of B, whose sums meet by shuffles: 99; fewer tiles in flight: 82).
template <typename T>
__global__ void __launch_bounds__(kUpThreads, kUpCtas) k_lora_up(LoraArgs A, int tile) {
  extern __shared__ __align__(128) unsigned char sm[];
  __shared__ uint64_t full[kUpStages];
  __shared__ int s_adapter[32];
  __shared__ uint32_t s_set[32];
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < kUpStages; ++i) mbar_init(&full[i], 1);
    fence_mbar_init();
  }
  int w = -1;
  if (lane < A.B) w = ld_cg_i32(A.which + lane);
  if (w >= A.adapters) {
    if (blockIdx.x == 0) flag_error(A.err, kErrIndex);
    w = -1;
  }
  w = max(w, -1);
  const uint32_t same = __match_any_sync(0xffffffffu, w), tokens = A.B >= 32 ? 0xffffffffu : (1u << A.B) - 1u;
  const bool leads = w >= 0 && __ffs(same) - 1 == lane;
  const uint32_t leaders = __ballot_sync(0xffffffffu, leads), none = __ballot_sync(0xffffffffu, w < 0) & tokens;
  if (tid < 32 && leads) {
    const int at = __popc(leaders & ((1u << lane) - 1u));
    s_adapter[at] = w;
    s_set[at] = same;
  }
  __syncthreads();
  const int tiles = (A.rows - 1) / tile + 1;
  const int64_t total = (int64_t)__popc(leaders) * tiles, u0 = total * blockIdx.x / gridDim.x, u1 = total * (blockIdx.x + 1) / gridDim.x;
  const int n = (int)(u1 - u0);
  int lead = (int)(u0 / tiles), t = (int)(u0 - (int64_t)lead * tiles);   // of the copies, then of the sums
  int next_lead = lead, next_t = t;
  auto copy = [&](int i) {             // thread 0: pair i of the run
    const int rows = min(tile, A.rows - next_t * tile);
    const uint32_t bytes = (uint32_t)(rows * A.rank * (int)sizeof(T));
    mbar_arrive_expect_tx(&full[i % kUpStages], bytes);
    bulk_g2s(sm + (i % kUpStages) * kUpStage,
             static_cast<const T *>(A.Bm) + ((int64_t)s_adapter[next_lead] * A.rows + (int64_t)next_t * tile) * A.rank, bytes,
             &full[i % kUpStages]);
    if (++next_t == tiles) {
      next_t = 0;
      ++next_lead;
    }
  };
  if (tid == 0)
    for (int i = 0; i < min(n, kUpStages); ++i) copy(i);
  pdl_wait();
  float *s_h = reinterpret_cast<float *>(sm + kUpStages * kUpStage);   // of the tokens that `there` leads
  int there = -1;
  bool ok = true;
  for (int i = 0; i < n && ok; ++i) {
    uint32_t set = s_set[lead];
    if (lead != there) {
      const int quads = A.rank / 4, all = __popc(set) * quads;
      for (int j = tid; j < all; j += kUpThreads) {
        const int b = j / quads, q = j - b * quads, tok = __fns(set, 0, b + 1);
        *reinterpret_cast<float4 *>(s_h + b * A.rank + (q & 1) * (A.rank / 2) + (q >> 1) * 4) =
            __ldcg(reinterpret_cast<const float4 *>(A.h + (int64_t)tok * A.rank) + q);
      }
      there = lead;
    }
    ok = mbar_wait(&full[i % kUpStages], (uint32_t)(i / kUpStages) & 1u, kUpWaitNs);
    ok = __syncthreads_and(ok);
    if (!ok) {
      if (tid == 0) {
        flag_error(A.err, kErrTimeout);
        // what is on its way lands before the shared memory is given back
        for (int e = i; e < min(n, i + kUpStages); ++e) mbar_wait(&full[e % kUpStages], (uint32_t)(e / kUpStages) & 1u, kUpWaitNs);
      }
      break;
    }
    const T *rows_of_b = reinterpret_cast<const T *>(sm + (i % kUpStages) * kUpStage);
    const int row0 = t * tile, rows = min(tile, A.rows - row0);
    for (const float *h = s_h; set; h += kAlong * A.rank) {
      const int left = __popc(set);
      if (left > 2) up_tokens<T, 4>(A, rows_of_b, row0, rows, h, set);
      else if (left > 1) up_tokens<T, 2>(A, rows_of_b, row0, rows, h, set);
      else up_tokens<T, 1>(A, rows_of_b, row0, rows, h, set);
    }
    __syncthreads();                   // the stage and the values of h have been read
    if (tid == 0 && i + kUpStages < n) copy(i + kUpStages);
    if (++t == tiles) {
      t = 0;
      ++lead;
    }
  }
  // tokens without an adapter: the activation and the rounding are left to do
  if (none && (A.relu || static_cast<const void *>(A.base) != A.y))
    for (int64_t row = (int64_t)blockIdx.x * kUpThreads + tid; row < A.rows; row += (int64_t)gridDim.x * kUpThreads)
      for (uint32_t set = none; set; set &= set - 1) {
        const int64_t at = (int64_t)(__ffs(set) - 1) * A.rows + row;
        put(A, at, __ldcg(A.base + at));
      }
}

// ------------------------------------------------------------------ host --
asf_status check_lora(const asf_lora *l) {
  if (!l || !l->A || !l->B || l->adapters < 1 || l->rank < 1 || l->k < 1 || l->rows < 1) return ASF_ERR_INVALID_ARG;
  if (l->dtype != ASF_F16 && l->dtype != ASF_F32) return ASF_ERR_UNSUPPORTED;
  if (l->rank % 8 || l->k % 8 || !al16(l->A) || !al16(l->B) || !al4(l->scale)) return ASF_ERR_MISALIGNED;
  if (l->rank > ASF_MAX_LORA_RANK || l->k > ASF_W4_MAX_K || l->rows > ASF_W4_MAX_ROWS) return ASF_ERR_UNSUPPORTED;
  return ASF_OK;
}
size_t lora_scratch(const asf_lora *l, int B) { return r256((size_t)B * l->rank * 4) + r256((size_t)B * l->rows * 4); }

template <typename T>
cudaError_t run_down(const LoraArgs &a, cudaStream_t st) {
  // four rows a CTA where that still is a CTA an SM, for adapters as many as may be
  return a.rank / 4 * std::min(a.B, a.adapters) >= sm_count()
             ? launch(k_lora_down<T, 4>, dim3(a.rank / 4, a.B), dim3(kDownThreads), 0, st, a)
             : launch(k_lora_down<T, 1>, dim3(a.rank, a.B), dim3(kDownThreads), 0, st, a);
}

}  // namespace

extern "C" {

size_t asf_w4_lora_workspace_bytes(const asf_w4_matrix *mat, const asf_lora *lora, int32_t max_batch) {
  const size_t need = asf_w4_workspace_bytes(mat, nullptr, max_batch);
  if (need == 0 || check_lora(lora) != ASF_OK || lora->k != mat->k || lora->rows != mat->rows) return 0;
  return r256(need) + lora_scratch(lora, max_batch);
}

asf_status asf_w4_matmul_lora(const asf_w4_matrix *mat, const asf_lora *lora, const int32_t *which, const void *x,
                              asf_dtype xdtype, int32_t B, const float *bias, int32_t relu, void *y, asf_dtype ydtype,
                              void *ws, size_t ws_bytes, asf_stream_t stream) {
  asf_status s = check_lora(lora);
  if (s != ASF_OK) return s;
  if (!mat || !which || !x || !y || lora->k != mat->k || lora->rows != mat->rows || B < 1 || B > ASF_MAX_BATCH ||
      (relu != 0 && relu != 1))
    return ASF_ERR_INVALID_ARG;
  if ((ydtype != ASF_F16 && ydtype != ASF_F32) || xdtype != lora->dtype) return ASF_ERR_UNSUPPORTED;
  if (!al4(which) || !al16(x) || (reinterpret_cast<uintptr_t>(y) & (ydtype == ASF_F16 ? 1u : 3u))) return ASF_ERR_MISALIGNED;
  const size_t plain = r256(w4_product_bytes(mat, B));                  // at most what the workspace was sized with
  if (plain) {
    s = check_ws(ws, ws_bytes, plain + lora_scratch(lora, B));
    if (s != ASF_OK) return s;
  }
  if (overlap(x, (size_t)B * mat->k * (xdtype == ASF_F16 ? 2 : 4), y, (size_t)B * mat->rows * (ydtype == ASF_F16 ? 2 : 4)))
    return ASF_ERR_INVALID_ARG;
  unsigned char *at = static_cast<unsigned char *>(ws) + plain;
  LoraArgs a{};
  a.adapters = lora->adapters;
  a.rank = lora->rank;
  a.k = lora->k;
  a.rows = lora->rows;
  a.B = B;
  a.A = lora->A;
  a.Bm = lora->B;
  a.scale = lora->scale;
  a.which = which;
  a.x = x;
  a.h = reinterpret_cast<float *>(at);
  a.y = y;
  a.y16 = ydtype == ASF_F16;
  float *base = a.y16 ? reinterpret_cast<float *>(at + r256((size_t)B * lora->rank * 4)) : static_cast<float *>(y);
  a.base = base;
  a.relu = relu;
  a.err = plain ? &static_cast<Header *>(ws)->err : nullptr;
  // the product first: it refuses what is wrong with the matrix before anything is enqueued
  s = asf_w4_matmul(mat, x, xdtype, B, bias, 0, base, ASF_F32, ws, plain, stream);
  if (s != ASF_OK) return s;
  cudaStream_t st = (cudaStream_t)stream;
  cudaError_t e = xdtype == ASF_F16 ? run_down<__half>(a, st) : run_down<float>(a, st);
  if (e != cudaSuccess) return ASF_ERR_CUDA;
  // 16 KB a tile, or as much as leaves an SM one
  const int64_t even = ((int64_t)a.rows * std::min(B, a.adapters) / sm_count() + 31) / 32 * 32;
  const int tile = (int)std::min<int64_t>({kUpRows, kUpStage / (a.rank * (xdtype == ASF_F16 ? 2 : 4)), std::max<int64_t>(32, even)});
  const int64_t pairs = ((int64_t)a.rows + tile - 1) / tile * std::min(B, a.adapters);
  const size_t smem = (size_t)kUpStages * kUpStage + (size_t)B * a.rank * 4;
  const int ctas = smem <= kUpShared ? kUpCtas : 2;                      // as many as an SM's shared memory holds
  const dim3 grid((unsigned)std::min<int64_t>(std::max<int64_t>(pairs, 1), (int64_t)ctas * sm_count()));
  e = xdtype == ASF_F16 ? launch(k_lora_up<__half>, grid, dim3(kUpThreads), smem, st, a, tile)
                        : launch(k_lora_up<float>, grid, dim3(kUpThreads), smem, st, a, tile);
  return cuda_status(e);
}

}  // extern "C"
