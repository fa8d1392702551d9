// Eviction from a paged key/value cache by the weight that keys have received
// (include/asffn.h, "Eviction").
//
//   asf_kv_evict    k_evict_select, then k_evict_move
//
// Selection is exact: scores become 32-bit keys whose order as whole numbers is the
// scores' (NaN below everything, the zeros equal), and the value of the last key to
// stay is found digit by digit (11, 11 and 10 bits) from counts of each digit's
// values; of the keys equal to it the lowest positions stay.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "asffn.h"
#include "common.cuh"
#include "host.cuh"
#include "paged.cuh"

using namespace asf;

namespace {

constexpr int kSelThreads = 512;
constexpr int kBins = 2048;
constexpr int kMoveThreads = 256;
constexpr int kMoveKeys = 32, kMoveHeads = 8;    // of a CTA: a row's offsets by a thread each
static_assert(kMoveKeys * kMoveHeads == kMoveThreads, "a row a thread");
constexpr uint32_t kHeld = 0xffffffffu;          // above every score
constexpr int kStageMost = 40 * 1024;            // keys of a CTA in shared memory

struct EvictArgs {
  asf_kv_cache c;
  const int32_t *table, *table_out;
  int max_pages, max_pages_out, R;
  const int32_t *lens;
  int32_t *lens_out;
  const float *scores;
  float *scores_out;
  int S, S_out;
  int32_t *kept;                                 // [R][heads][keep]
  int keep, first, recent;
  int staged;                                    // keys of a CTA that fit its shared memory
  int32_t *err;
};

__device__ __forceinline__ uint32_t order_of(float v) {
  const uint32_t b = __float_as_uint(v);
  if ((b & 0x7fffffffu) > 0x7f800000u) return 0u;
  if ((b & 0x7fffffffu) == 0u) return 0x80000000u;
  return b >> 31 ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// a word of CTA `rank`'s shared memory, at the address of this CTA's p
__device__ __forceinline__ uint32_t ld_peer(const uint32_t *p, int rank) {
  uint32_t at, v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}

// exclusive sum over the CTA's threads, and the total; `part` holds a word per warp
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t *part, uint32_t &total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t u = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += u;
  }
  __syncthreads();
  if (lane == 31) part[warp] = s;
  __syncthreads();
  uint32_t before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kSelThreads / 32; ++w) {
    const uint32_t u = part[w];
    if (w < warp) before += u;
    total += u;
  }
  return before + s - v;
}

// A cluster of CL CTAs is one kv head of one request, each of them a run of its
// positions, kept in shared memory as keys where it fits.  Per digit: counts of the
// keys that agree with the digits found so far, summed over distributed shared
// memory by every CTA, and a scan from the largest value down.  Then each thread
// walks a run of its own twice: how many stay, and where they go.
template <int CL>
__global__ void __launch_bounds__(kSelThreads) k_evict_select(EvictArgs A) {
  extern __shared__ uint32_t s_keys[];
  __shared__ uint32_t s_hist[kBins], s_part[kSelThreads / 32], s_found[2], s_count[2];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, rank = CL > 1 ? (int)blockIdx.x % CL : 0, unit = blockIdx.x / CL;
  const int r = unit / A.c.heads, head = unit % A.c.heads;
  int n = ld_cg_i32(A.lens + r);
  const int cap = (int)min((int64_t)A.S, (int64_t)A.max_pages * A.c.page);
  if (n < 0 || n > cap) {
    if (head == 0 && rank == 0 && tid == 0) flag_error(A.err, kErrIndex);
    n = n < 0 ? 0 : cap;
  }
  const int stay = min(n, A.keep);
  if (head == 0 && rank == 0 && tid == 0) A.lens_out[r] = stay;
  const float *scores = A.scores + (int64_t)unit * A.S;
  float *scores_out = A.scores_out + (int64_t)unit * A.S_out;
  int32_t *kept = A.kept + (int64_t)unit * A.keep;
  if (n <= A.keep) {                             // everything stays; the whole cluster is here
    for (int p = rank * kSelThreads + tid; p < n; p += CL * kSelThreads) {
      kept[p] = p;
      scores_out[p] = scores[p];
    }
    return;
  }
  const int run = (n + CL - 1) / CL, p0 = min(n, rank * run), mine = min(n, p0 + run) - p0;
  auto fresh = [&](int i) {
    const int p = p0 + i;
    return p < A.first || p >= n - A.recent ? kHeld : order_of(__ldcg(scores + p));
  };
  const bool staged = run <= A.staged;
  if (staged)
    for (int i = tid; i < mine; i += kSelThreads) s_keys[i] = fresh(i);
  auto key = [&](int i) { return staged ? s_keys[i] : fresh(i); };

  uint32_t want = (uint32_t)A.keep, prefix = 0;  // of the keys that agree with prefix, the want-th largest
  int shift = 21;
#pragma unroll 1
  for (int digit = 0; digit < 3; ++digit) {
    const int bits = digit == 2 ? 10 : 11, upper = shift + bits;
    for (int i = tid; i < kBins; i += kSelThreads) s_hist[i] = 0;
    __syncthreads();
#pragma unroll 4
    for (int i = tid; i < mine; i += kSelThreads) {
      const uint32_t k = key(i);
      if (digit == 0 || k >> upper == prefix) atomicAdd(&s_hist[(k >> shift) & ((1u << bits) - 1u)], 1u);
    }
    if (CL > 1) cluster_barrier();
    else __syncthreads();
    // four bins a thread, from the largest down
    constexpr int PER = kBins / kSelThreads;
    uint32_t c[PER], sum = 0;
#pragma unroll
    for (int b = 0; b < PER; ++b) {
      const int bin = kBins - 1 - (tid * PER + b);
      c[b] = 0;
      if (CL > 1) {
#pragma unroll
        for (int q = 0; q < CL; ++q) c[b] += ld_peer(&s_hist[bin], q);
      } else {
        c[b] = s_hist[bin];
      }
      sum += c[b];
    }
    uint32_t total;
    uint32_t above = block_scan(sum, s_part, total);
#pragma unroll
    for (int b = 0; b < PER; ++b) {
      if (above < want && above + c[b] >= want) {
        s_found[0] = kBins - 1 - (tid * PER + b);
        s_found[1] = want - above;
      }
      above += c[b];
    }
    if (CL > 1) cluster_barrier();               // counts are read before they are cleared
    else __syncthreads();
    prefix = prefix << bits | s_found[0];
    want = s_found[1];
    shift -= digit == 1 ? 10 : 11;
    __syncthreads();
  }
  // larger keys than prefix stay, and the first `want` of those equal to it
  const int per = ((mine + kSelThreads - 1) / kSelThreads) | 1;          // odd: threads' runs begin in different banks
  const int i0 = min(mine, tid * per), i1 = min(mine, i0 + per);
  uint32_t more = 0, same = 0;
  for (int i = i0; i < i1; ++i) {
    const uint32_t k = key(i);
    more += k > prefix;
    same += k == prefix;
  }
  uint32_t all_more, all_same;
  uint32_t m = block_scan(more, s_part, all_more), e = block_scan(same, s_part, all_same);
  if (CL > 1) {
    if (tid == 0) {
      s_count[0] = all_more;
      s_count[1] = all_same;
    }
    cluster_barrier();
    for (int q = 0; q < rank; ++q) {
      m += ld_peer(&s_count[0], q);
      e += ld_peer(&s_count[1], q);
    }
    cluster_barrier();                           // nobody leaves while its counts are read
  }
  for (int i = i0; i < i1; ++i) {
    const uint32_t k = key(i);
    if (k > prefix || (k == prefix && e < want)) {
      const uint32_t to = m + min(e, want);
      kept[to] = p0 + i;
      scores_out[to] = __ldcg(scores + p0 + i);
    }
    m += k > prefix;
    e += k == prefix;
  }
}

// The kept rows to their new places: offsets of 32 keys x 8 heads by a thread
// each, then 16 bytes of keys and of values a thread at a time.
__global__ void __launch_bounds__(kMoveThreads) k_evict_move(EvictArgs A) {
  __shared__ int64_t s_from[kMoveThreads], s_to[kMoveThreads];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, r = blockIdx.z, j0 = blockIdx.x * kMoveKeys, h0 = blockIdx.y * kMoveHeads;
  const int stay = ld_cg_i32(A.lens_out + r), page = A.c.page;
  if (j0 >= stay) return;
  const int heads = min(kMoveHeads, A.c.heads - h0), keys = min(kMoveKeys, stay - j0);
  {
    const int j = j0 + (tid & 31), h = tid >> 5;
    int64_t from = -1, to = -1;
    if (h < heads && j < stay) {
      const int p = ld_cg_i32(A.kept + ((int64_t)r * A.c.heads + h0 + h) * A.keep + j);
      const int pi = p / page, ji = j / page;
      const int a = A.table[(int64_t)r * A.max_pages + pi];
      const int b = ji < A.max_pages_out ? A.table_out[(int64_t)r * A.max_pages_out + ji] : -1;
      if ((unsigned)a < (unsigned)A.c.pages && (unsigned)b < (unsigned)A.c.pages) {
        from = (int64_t)a * A.c.page_stride + (int64_t)(p - pi * page) * A.c.token_stride + (int64_t)(h0 + h) * A.c.head_stride;
        to = (int64_t)b * A.c.page_stride + (int64_t)(j - ji * page) * A.c.token_stride + (int64_t)(h0 + h) * A.c.head_stride;
      } else {
        flag_error(A.err, kErrIndex);
      }
    }
    const int at = (tid & 31) * heads + h;       // a key's heads side by side
    if (h < heads) {
      s_from[at] = from;
      s_to[at] = to;
    }
  }
  __syncthreads();
  const int ch = A.c.head_dim / 8, rows = keys * heads;
  const int lanes = kMoveThreads / ch;           // rows at a time
  const int c = tid % ch;
  __half *k = static_cast<__half *>(A.c.k), *v = static_cast<__half *>(A.c.v);
  constexpr int U = 4;
  for (int row = tid / ch; row < rows; row += lanes * U) {
    uint4 a[U], b[U];
    int64_t to[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int at = row + i * lanes;
      to[i] = at < rows && tid < lanes * ch ? s_to[at] : -1;
      if (to[i] >= 0) {
        a[i] = __ldcs(reinterpret_cast<const uint4 *>(k + s_from[at]) + c);
        b[i] = __ldcs(reinterpret_cast<const uint4 *>(v + s_from[at]) + c);
      }
    }
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (to[i] >= 0) {
        reinterpret_cast<uint4 *>(k + to[i])[c] = a[i];
        reinterpret_cast<uint4 *>(v + to[i])[c] = b[i];
      }
  }
}

}  // namespace

extern "C" {

asf_status asf_kv_evict(const asf_kv_cache *cache, const int32_t *table, int32_t max_pages, int32_t R, const int32_t *lens,
                        const float *scores, int32_t S, int32_t keep, int32_t first, int32_t recent, const int32_t *table_out,
                        int32_t max_pages_out, int32_t *lens_out, float *scores_out, int32_t S_out, int32_t *kept, void *ws,
                        size_t ws_bytes, asf_stream_t stream) {
  asf_status s = check_cache(cache);
  if (s != ASF_OK) return s;
  if (!table || !lens || !scores || !table_out || !lens_out || !scores_out || !kept || table == table_out)
    return ASF_ERR_INVALID_ARG;
  if (max_pages < 1 || max_pages_out < 1 || R < 1 || R > ASF_MAX_BATCH || S < 1 || keep < 1 || first < 0 || recent < 0 ||
      (int64_t)first + recent > keep || S_out < keep)
    return ASF_ERR_INVALID_ARG;
  if ((int64_t)max_pages * cache->page > ASF_MAX_KEYS || (int64_t)max_pages_out * cache->page > ASF_MAX_KEYS ||
      S > ASF_MAX_KEYS || S_out > ASF_MAX_KEYS)
    return ASF_ERR_UNSUPPORTED;
  if (!al4(table) || !al4(lens) || !al4(scores) || !al4(table_out) || !al4(lens_out) || !al4(scores_out) || !al4(kept))
    return ASF_ERR_MISALIGNED;
  s = check_ws(ws, ws_bytes, kHeaderBytes);
  if (s != ASF_OK) return s;
  const size_t rows = (size_t)R * cache->heads * 4, in = rows * S, out = rows * S_out, list = rows * keep;
  if (overlap(scores, in, scores_out, out) || overlap(scores, in, kept, list) || overlap(scores_out, out, kept, list) ||
      overlap(lens, (size_t)R * 4, lens_out, (size_t)R * 4))
    return ASF_ERR_INVALID_ARG;
  EvictArgs a{*cache, table, table_out, max_pages, max_pages_out, R, lens, lens_out, scores, scores_out, S, S_out, kept,
              keep, first, recent, 0, &static_cast<Header *>(ws)->err};
  cudaStream_t st = (cudaStream_t)stream;
  const int most = (int)std::min<int64_t>(S, (int64_t)max_pages * cache->page), units = R * cache->heads;
  const int cl = most > 4096 ? 8 : 1;
  a.staged = std::min((most + cl - 1) / cl, kStageMost);
  const size_t smem = (size_t)a.staged * 4;
  cudaError_t e = cl == 8 ? launch_clusters(k_evict_select<8>, dim3(units * 8), dim3(kSelThreads), smem, st, 8, a)
                          : launch(k_evict_select<1>, dim3(units), dim3(kSelThreads), smem, st, a);
  if (e != cudaSuccess) return ASF_ERR_CUDA;
  const int last = std::min(keep, most);
  const dim3 grid((last + kMoveKeys - 1) / kMoveKeys, (cache->heads + kMoveHeads - 1) / kMoveHeads, R);
  return cuda_status(launch(k_evict_move, grid, dim3(kMoveThreads), 0, st, a));
}

}  // extern "C"
