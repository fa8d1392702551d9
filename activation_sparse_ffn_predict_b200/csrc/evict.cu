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
// Rows of a CTA, a row's places by a thread each.  4 requests of up to 65500 keys to 16384, us
// of the call: 32 x 8 rows and four steps in flight 127, 16 x 8 117 (a shorter tail),
// without the streaming hint on loads 110, with two steps in flight 107 (eight: 129).
constexpr int kMoveThreads = 256;
constexpr int kMoveKeys = 16, kMoveHeads = 8;
constexpr int kMoveRows = kMoveKeys * kMoveHeads;
static_assert(kMoveRows <= kMoveThreads, "a row a thread");
constexpr uint32_t kHeld = 0xffffffffu;          // above every score
constexpr int kStageMost = 40 * 1024;            // scores of a CTA in shared memory

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
  int staged;                                    // scores of a CTA that fit its shared memory
  int32_t *err;
};

__device__ __forceinline__ uint32_t order_of(float v) {
  const uint32_t b = __float_as_uint(v);
  if ((b & 0x7fffffffu) > 0x7f800000u) return 0u;
  if ((b & 0x7fffffffu) == 0u) return 0x80000000u;
  return b >> 31 ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ void cluster_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// a word of CTA `rank`'s shared memory, at the address of this CTA's p
__device__ __forceinline__ uint32_t ld_peer(const uint32_t *p, int rank) {
  uint32_t at, v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}

// adds to it
__device__ __forceinline__ void add_peer(uint32_t *p, int rank, uint32_t v) {
  uint32_t at;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
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
// positions, whose scores it keeps in shared memory where they fit.  Per digit: counts
// of the keys that agree with the digits found so far, which every CTA adds to the
// CTAs that own a share of the digit's values (distributed shared memory), and a scan of
// all of them from the largest value down.  Then each warp walks a stretch of positions
// twice: how many stay, and where they go.  Latency bounds it, above all the barriers
// of the cluster: five of them, a microsecond and more each (with nine, counts fetched and
// shares' sums published, 26 us at 65500 keys).
template <int CL>
__global__ void __launch_bounds__(kSelThreads) k_evict_select(EvictArgs A) {
  constexpr int NW = kSelThreads / 32, SHARE = kBins / CL, PER = kBins / kSelThreads;
  extern __shared__ float s_score[];
  __shared__ uint32_t s_hist[kBins], s_part[NW], s_found[2];
  __shared__ uint32_t s_share[3][CL > 1 ? SHARE : 1], s_count[2];   // other CTAs add to these: a digit's counts, what is before this CTA
  __shared__ uint32_t s_more[NW], s_same[NW];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = CL > 1 ? (int)blockIdx.x % CL : 0, unit = blockIdx.x / CL;
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
  if constexpr (CL > 1) {
    for (int i = tid; i < 3 * SHARE; i += kSelThreads) s_share[i / SHARE][i % SHARE] = 0;
    if (tid < 2) s_count[tid] = 0;
    cluster_arrive();
  }
  const int run = (n + CL - 1) / CL, p0 = min(n, rank * run), mine = min(n, p0 + run) - p0;
  const bool staged = run <= A.staged;
  if (staged) {
    constexpr int U = 8;                         // loads in flight
    for (int i0 = tid; i0 < mine; i0 += U * kSelThreads) {
      float v[U];
#pragma unroll
      for (int k = 0; k < U; ++k) v[k] = i0 + k * kSelThreads < mine ? __ldcg(scores + p0 + i0 + k * kSelThreads) : 0.f;
#pragma unroll
      for (int k = 0; k < U; ++k)
        if (i0 + k * kSelThreads < mine) s_score[i0 + k * kSelThreads] = v[k];
    }
  }
  auto score = [&](int i) { return staged ? s_score[i] : __ldcg(scores + p0 + i); };
  auto key_of = [&](int i, float v) {
    const int p = p0 + i;
    return p < A.first || p >= n - A.recent ? kHeld : order_of(v);
  };

  uint32_t want = (uint32_t)A.keep, prefix = 0;  // of the keys that agree with prefix, the want-th largest
  int shift = 21;
#pragma unroll 1
  for (int digit = 0; digit < 3; ++digit) {
    const int bits = digit == 2 ? 10 : 11, upper = shift + bits;
    for (int i = tid; i < kBins; i += kSelThreads) s_hist[i] = 0;
    __syncthreads();
#pragma unroll 4
    for (int i = tid; i < mine; i += kSelThreads) {
      const uint32_t k = key_of(i, score(i));
      if (digit == 0 || k >> upper == prefix) atomicAdd(&s_hist[(k >> shift) & ((1u << bits) - 1u)], 1u);
    }
    __syncthreads();
    if constexpr (CL > 1) {
      if (digit == 0) cluster_wait();            // every CTA's shares are clear
      for (int i = tid; i < kBins; i += kSelThreads)
        if (s_hist[i]) add_peer(&s_share[digit][i % SHARE], i / SHARE, s_hist[i]);
      cluster_arrive();
      cluster_wait();
    }
    // PER values a thread, from the largest down
    uint32_t c[PER], sum = 0, total;
#pragma unroll
    for (int b = 0; b < PER; ++b) {
      const int value = kBins - 1 - (tid * PER + b);
      c[b] = CL > 1 ? ld_peer(&s_share[digit][value % SHARE], value / SHARE) : s_hist[value];
    }
#pragma unroll
    for (int b = 0; b < PER; ++b) sum += c[b];
    uint32_t above = block_scan(sum, s_part, total);
#pragma unroll
    for (int b = 0; b < PER; ++b) {
      if (above < want && above + c[b] >= want) {
        s_found[0] = kBins - 1 - (tid * PER + b);
        s_found[1] = want - above;
      }
      above += c[b];
    }
    __syncthreads();
    prefix = prefix << bits | s_found[0];
    want = s_found[1];
    shift -= digit == 1 ? 10 : 11;
  }
  // larger keys than prefix stay, and the first `want` of those equal to it
  const int stretch = ((mine + NW - 1) / NW + 31) & ~31, i0 = warp * stretch, i1 = min(mine, i0 + stretch);
  uint32_t more = 0, same = 0;
  for (int i = i0; i < i1; i += 32) {
    const uint32_t k = i + lane < i1 ? key_of(i + lane, score(i + lane)) : 0u;
    more += __popc(__ballot_sync(0xffffffffu, i + lane < i1 && k > prefix));
    same += __popc(__ballot_sync(0xffffffffu, i + lane < i1 && k == prefix));
  }
  if (lane == 0) {
    s_more[warp] = more;
    s_same[warp] = same;
  }
  __syncthreads();
  uint32_t m = 0, e = 0, all_more = 0, all_same = 0;
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    const uint32_t a = s_more[w], b = s_same[w];
    if (w < warp) {
      m += a;
      e += b;
    }
    all_more += a;
    all_same += b;
  }
  if constexpr (CL > 1) {
    if (tid > rank && tid < CL) {
      add_peer(&s_count[0], tid, all_more);
      add_peer(&s_count[1], tid, all_same);
    }
    cluster_arrive();
    cluster_wait();                              // nothing reaches into another CTA from here on
    m += s_count[0];
    e += s_count[1];
  }
  const uint32_t below = (1u << lane) - 1u;
  for (int i = i0; i < i1; i += 32) {
    const bool in = i + lane < i1;
    const float v = in ? score(i + lane) : 0.f;
    const uint32_t k = in ? key_of(i + lane, v) : 0u;
    const uint32_t bm = __ballot_sync(0xffffffffu, in && k > prefix), be = __ballot_sync(0xffffffffu, in && k == prefix);
    const uint32_t mm = m + __popc(bm & below), ee = e + __popc(be & below);
    if (in && (k > prefix || (k == prefix && ee < want))) {
      const uint32_t to = mm + min(ee, want);
      kept[to] = p0 + i + lane;
      scores_out[to] = v;
    }
    m += __popc(bm);
    e += __popc(be);
  }
}

// The kept rows to their new places: a row's two places by a thread each, then 16
// bytes of keys and of values a thread at a time.  HBM bounds it: 402 MB in 71 us, 5.7 TB/s.
__global__ void __launch_bounds__(kMoveThreads) k_evict_move(EvictArgs A) {
  __shared__ int64_t s_from[kMoveRows], s_to[kMoveRows];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, r = blockIdx.z, j0 = blockIdx.x * kMoveKeys, h0 = blockIdx.y * kMoveHeads;
  const int stay = ld_cg_i32(A.lens_out + r), page = A.c.page;
  if (j0 >= stay) return;
  const int heads = min(kMoveHeads, A.c.heads - h0), keys = min(kMoveKeys, stay - j0);
  if (tid < kMoveRows) {
    const int j = j0 + tid % kMoveKeys, h = tid / kMoveKeys;
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
    const int at = tid % kMoveKeys * heads + h;    // a key's heads side by side
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
  constexpr int U = 2;
  for (int row = tid / ch; row < rows; row += lanes * U) {
    uint4 a[U], b[U];
    int64_t to[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int at = row + i * lanes;
      to[i] = at < rows && tid < lanes * ch ? s_to[at] : -1;
      if (to[i] >= 0) {
        a[i] = __ldcg(reinterpret_cast<const uint4 *>(k + s_from[at]) + c);
        b[i] = __ldcg(reinterpret_cast<const uint4 *>(v + s_from[at]) + c);
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
  const size_t rows = (size_t)R * cache->heads * 4;
  struct Range {
    const void *p;
    size_t bytes;
  };
  const Range in[] = {{table, (size_t)R * max_pages * 4}, {table_out, (size_t)R * max_pages_out * 4}, {lens, (size_t)R * 4}, {scores, rows * S}};
  const Range out[] = {{lens_out, (size_t)R * 4}, {scores_out, rows * S_out}, {kept, rows * keep}};
  for (int i = 0; i < 3; ++i) {
    if (in_cache(cache, out[i].p, out[i].bytes)) return ASF_ERR_INVALID_ARG;
    for (const Range &u : in)
      if (overlap(u.p, u.bytes, out[i].p, out[i].bytes)) return ASF_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (overlap(out[j].p, out[j].bytes, out[i].p, out[i].bytes)) return ASF_ERR_INVALID_ARG;
  }
  EvictArgs a{*cache, table, table_out, max_pages, max_pages_out, R, lens, lens_out, scores, scores_out, S, S_out, kept,
              keep, first, recent, 0, &static_cast<Header *>(ws)->err};
  cudaStream_t st = (cudaStream_t)stream;
  const int most = (int)std::min<int64_t>(S, (int64_t)max_pages * cache->page), units = R * cache->heads;
  // A cluster per kv head as large as leaves every CTA an SM, or half of one where its run is
  // long (tables of requests of different lengths leave some CTAs idle), and in any case so
  // large that its shared memory holds the scores.  us of the call, keeping 200 keys, with 8, 4, 2
  // and 1 CTAs: 8 heads x 4000 keys 13.9, 14.1, 15.5, 12.9; 20000 keys 16.7, 19.6, 26.2,
  // 34.2; 32 heads x 20000 27.0, 21.9, 26.5, 34.4; 64 heads x 10000 43.2, 26.0, 20.8, 22.9;
  // 128 heads x 10000 76.8, 44.3, 28.5, 24.5; 32 heads x 65500 keys 37.9 and 37.0 (8 and 4), and
  // with a request in two of them short 104 and 113.
  int cl = 1;
  for (; cl < 8 && most > 4096; cl *= 2) {
    const int run = (most + cl - 1) / cl, room = sm_count() * (run > 12 * 1024 ? 2 : 1);
    if (units * cl * 2 > room && run <= kStageMost) break;
  }
  a.staged = std::min((most + cl - 1) / cl, kStageMost);
  // Beside the static part (21 KB at most) more than 48 KB have to be asked for, which a launch does from 40 KB on.
  const size_t keys = (size_t)a.staged * 4, smem = keys <= 24 * 1024 ? keys : std::max<size_t>(keys, 41 * 1024);
  const dim3 ctas(units * cl), block(kSelThreads);
  const cudaError_t e = cl == 8   ? launch_clusters(k_evict_select<8>, ctas, block, smem, st, 8, a)
                        : cl == 4 ? launch_clusters(k_evict_select<4>, ctas, block, smem, st, 4, a)
                        : cl == 2 ? launch_clusters(k_evict_select<2>, ctas, block, smem, st, 2, a)
                                  : launch(k_evict_select<1>, ctas, block, smem, st, a);
  if (e != cudaSuccess) return ASF_ERR_CUDA;
  const int last = std::min(keep, most);
  const dim3 grid((last + kMoveKeys - 1) / kMoveKeys, (cache->heads + kMoveHeads - 1) / kMoveHeads, R);
  return cuda_status(launch(k_evict_move, grid, dim3(kMoveThreads), 0, st, a));
}

}  // extern "C"
