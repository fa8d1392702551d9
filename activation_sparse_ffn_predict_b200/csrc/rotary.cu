// Rotary positions: the turn of queries and keys in front of tree attention
// (include/asffn.h, "Rotary positions").
//
//   asf_rotary_frequencies, asf_rotary_turns   host
//   asf_rotary_apply                           k_rotary, k_rotary_odd
//   asf_rotary_append                          k_rotary_append
//
// Mathematics.  Pair j of a head at position p turns by p f_j radians,
// (u, w) -> m (u cos - w sin, w cos + u sin).  A position reaches 2^31, and
// fp32 has lost the angle long before.  So f_j is kept as a whole number of 2^-64
// turns: p f_j modulo a turn is the low 64 bits of one product of whole numbers,
// off by less than p 2^-64 turns, and only the fraction of a turn that is left goes
// to fp32 (2^-25 of a half turn) and to sincospi.  The turn is fp32, rounded once.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "asffn.h"
#include "common.cuh"
#include "host.cuh"
#include "paged.cuh"

using namespace asf;

namespace {

constexpr int kRotThreads = 128;
// Places of a head that a thread has in flight, of 32 bytes (halves) or 16 (pairs): more are
// slower, the threads of an SM are enough (8192 tokens x 72 heads of 128 columns in fp16,
// halves, us with 4, 2 and 1: 79, 60, 57).
constexpr int kAheadHalf = 1, kAheadPairs = 2;
static_assert(ASF_MAX_ROTARY_DIM / 4 <= kRotThreads, "a head's places are a CTA's");
// Chunks of a thread where there is work for every SM: more share the cosines, fewer leave more
// CTAs to hide loads.  8192 tokens, us with 3, 6, 9 and 18: 72 heads of 128 in halves 54.2, 53.5, 55.0,
// 61.0, 40 heads 31.0, 31.6, 32.8, 34.9, 128 heads 93.0, 92.1, 93.0, 98.0; 72 heads in pairs 68.3, 63.3, 61.0, 65.3,
// 126 of 128 columns in halves 103, 91, 81, 78, 24 of 96 columns 96, 81, 71, 65.
constexpr int kItems = 9;

// The fraction of a turn is rounded to fp32 as it is: fp32 heads come out 3.7e-8 of their norm from the definition
// (2.9e-8 with the angle in 64 bits).  Rounding only what is left of the nearest quarter turn, or a step of the derivative
// for what the rounding leaves, takes 8 registers more where pairs are in flight: 8192 tokens x 72 heads 60.3 -> 65.4 us.
__device__ __forceinline__ float2 cos_sin(int pos, uint64_t turns, float mul) {
  const uint64_t phase = (uint64_t)(int64_t)pos * turns;
  const int half_turns = (int)(uint32_t)((phase + 0x80000000ull) >> 32);     // of 2^-31
  float s, c;
  sincospif((float)half_turns * 4.656612873077393e-10f, &s, &c);
  return make_float2(c * mul, s * mul);
}

// N elements of T, N a power of two and 16 bytes at most
template <typename T, int N>
struct alignas(sizeof(T) * N) Pack {
  T v[N];
};
__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
__device__ __forceinline__ void from_f(float v, float &to) { to = v; }
__device__ __forceinline__ void from_f(float v, __half &to) { to = __float2half_rn(v); }

// (k_rotary_append) VEC pairs of a head, 4 at most: halves are `half` columns apart, neighbours side by side in one access.
template <int VEC, bool PAIRS>
struct Pairs {
  static constexpr int kPass = 2 * VEC;            // columns of an access to what passes
  Pack<__half, VEC> a, b;
  __device__ __forceinline__ void load(const __half *row, int j, int half) {
    if constexpr (PAIRS) {
      load_pass(row + j * kPass);
    } else {
      a = *reinterpret_cast<const Pack<__half, VEC> *>(row + j * VEC);
      b = *reinterpret_cast<const Pack<__half, VEC> *>(row + half + j * VEC);
    }
  }
  __device__ __forceinline__ void store(__half *row, int j, int half) const {
    if constexpr (PAIRS) {
      store_pass(row + j * kPass);
    } else {
      *reinterpret_cast<Pack<__half, VEC> *>(row + j * VEC) = a;
      *reinterpret_cast<Pack<__half, VEC> *>(row + half + j * VEC) = b;
    }
  }
  // kPass columns, as they are
  __device__ __forceinline__ void load_pass(const __half *p) {
    const Pack<__half, kPass> u = *reinterpret_cast<const Pack<__half, kPass> *>(p);
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      a.v[i] = u.v[i];
      b.v[i] = u.v[VEC + i];
    }
  }
  __device__ __forceinline__ void store_pass(__half *p) const {
    Pack<__half, kPass> u;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      u.v[i] = a.v[i];
      u.v[VEC + i] = b.v[i];
    }
    *reinterpret_cast<Pack<__half, kPass> *>(p) = u;
  }
  // cs[i]: cos and sin of the i-th pair
  __device__ __forceinline__ void turn(const float2 *cs) {
    const Pack<__half, VEC> x = a, y = b;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      // element 2i and 2i + 1 of the 2 VEC where neighbours are paired
      __half &u = PAIRS ? (2 * i < VEC ? a.v[(2 * i) % VEC] : b.v[(2 * i) % VEC]) : a.v[i];
      __half &w = PAIRS ? (2 * i + 1 < VEC ? a.v[(2 * i + 1) % VEC] : b.v[(2 * i + 1) % VEC]) : b.v[i];
      const float fu = to_f(PAIRS ? (2 * i < VEC ? x.v[(2 * i) % VEC] : y.v[(2 * i) % VEC]) : x.v[i]);
      const float fw = to_f(PAIRS ? (2 * i + 1 < VEC ? x.v[(2 * i + 1) % VEC] : y.v[(2 * i + 1) % VEC]) : y.v[i]);
      const float c = cs[i].x, s = cs[i].y;
      from_f(fmaf(fu, c, -(fw * s)), u);
      from_f(fmaf(fw, c, fu * s), w);
    }
  }
};

struct RotArgs {
  const void *x;
  void *y;
  int64_t xt, xh, yt, yh;              // elements from token to token, head to head
  int T, heads;
  int D, half;
  const uint64_t *turns;
  float mul;
  const int32_t *pos;
  int tb, hs;                          // tokens and heads of a CTA
  bool copy;                           // the columns from rot_dim on, too
};

template <typename T>
using Chunk = Pack<T, 16 / (int)sizeof(T)>;

// Where a token's pair is, among its cosines and sines: those of every P-th pair side
// by side, since neighbouring threads read pairs P apart (together in different banks;
// two neighbouring pairs are 16 bytes in any case).
template <int P>
__host__ __device__ constexpr int pitch(int half) { return (half + P - 1) / P; }
template <int P>
__device__ __forceinline__ int place_in(int half, int pair) { return P > 2 ? pair % P * pitch<P>(half) + pair / P : pair; }
// cosines and sines of the CTA's tokens
template <int P>
__device__ __forceinline__ void all_angles(const RotArgs &A, int t0, int nt, float2 *cs) {
  for (int i = threadIdx.x; i < nt * A.half; i += kRotThreads) {
    const int k = i / A.half, j = i - k * A.half;
    cs[k * P * pitch<P>(A.half) + place_in<P>(A.half, j)] = cos_sin(A.pos[t0 + k], A.turns[j], A.mul);
  }
  __syncthreads();
}

// A CTA takes tb tokens and hs of their heads: each token's cosines and sines
// are computed once a CTA, into shared memory, while the first chunks are on
// their way; then a thread keeps one place in a head, and steps from head to head.
// A place is 16 bytes of neighbours (those behind rot_dim keep their bits), or 16 of
// each half where the halves are whole 16 bytes; k_rotary_odd takes the others.
// HBM bounds it on long prompts: 8192 tokens x 72 heads of 128 columns in fp16, 302 MB
// in 55 us, 5.5 TB/s.
template <typename T, bool PAIRS>
__global__ void __launch_bounds__(kRotThreads) k_rotary(RotArgs A) {
  constexpr int U = 16 / (int)sizeof(T), kAhead = PAIRS ? kAheadPairs : kAheadHalf, P = PAIRS ? U / 2 : U;   // pairs of a place
  extern __shared__ float2 s_cs[];     // [tb][P][pitch]
  pdl_wait();
  pdl_trigger();
  const int t0 = blockIdx.x * A.tb, nt = min(A.tb, A.T - t0);
  const int h0 = blockIdx.y * A.hs, nh = min(A.hs, A.heads - h0);
  const int turned = PAIRS ? (2 * A.half + U - 1) / U : A.half / U;
  const int per = !A.copy ? turned : PAIRS ? A.D / U : turned + (A.D - 2 * A.half) / U;   // at most kRotThreads
  const int step = kRotThreads / per, rows = nt * nh;
  const int row0 = threadIdx.x / per, c = threadIdx.x - row0 * per;
  const bool turns = c < turned;
  const int at = PAIRS || turns ? c * U : 2 * A.half + (c - turned) * U;
  const T *x = static_cast<const T *>(A.x) + t0 * A.xt + h0 * A.xh + at;
  T *y = static_cast<T *>(A.y) + t0 * A.yt + h0 * A.yh + at;
  const int dt = step / nh, dh = step - dt * nh;
  int t = row0 / nh, h = row0 - t * nh, row = row0 < step ? row0 : rows;
  bool fresh = true;
  do {
    Chunk<T> a[kAhead], b[PAIRS ? 1 : kAhead];
    int64_t to[kAhead];
    int tok[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      to[i] = -1;
      if (row < rows) {
        to[i] = t * A.yt + h * A.yh;
        tok[i] = t;
        const T *from = x + (t * A.xt + h * A.xh);
        a[i] = *reinterpret_cast<const Chunk<T> *>(from);
        if constexpr (!PAIRS)
          if (turns) b[i] = *reinterpret_cast<const Chunk<T> *>(from + A.half);
      }
      row += step;
      h += dh;
      t += dt;
      if (h >= nh) {
        h -= nh;
        ++t;
      }
    }
    if (fresh) all_angles<P>(A, t0, nt, s_cs);     // every thread is here once at least
    fresh = false;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (to[i] < 0) continue;
      if (turns) {
        const int apart = P > 2 ? pitch<P>(A.half) : 1;
        const float2 *cs = s_cs + tok[i] * P * pitch<P>(A.half) + (P > 2 ? c : c * P);
#pragma unroll
        for (int j = 0; j < P; ++j) {
          if (PAIRS && c * P + j >= A.half) break;
          T &u = a[i].v[PAIRS ? 2 * j : j], &w = PAIRS ? a[i].v[(2 * j + 1) % U] : b[PAIRS ? 0 : i].v[j];
          const float fu = to_f(u), fw = to_f(w), cv = cs[j * apart].x, sv = cs[j * apart].y;
          from_f(fmaf(fu, cv, -(fw * sv)), u);
          from_f(fmaf(fw, cv, fu * sv), w);
        }
        if constexpr (!PAIRS) *reinterpret_cast<Chunk<T> *>(y + to[i] + A.half) = b[i];
      }
      *reinterpret_cast<Chunk<T> *>(y + to[i]) = a[i];
    }
  } while (row < rows);
}

// Halves that are not whole 16 bytes: a thread has 16 bytes of a head, and finds the
// other halves of its pairs in shared memory, where the CTA lays out a group of heads
// (two buffers: a barrier a group), the next group's chunk in flight meanwhile.
// 8192 tokens x 72 heads, 126 of 128 columns in fp16: 81 us (a pair a thread in 2-byte
// accesses 171), 24 of 96 columns 71: 3.7 and 3.2 TB/s, the barrier a group of heads and two reads of shared
// memory a pair.
template <typename T>
__global__ void __launch_bounds__(kRotThreads) k_rotary_odd(RotArgs A) {
  constexpr int U = 16 / (int)sizeof(T);
  extern __shared__ float2 s_cs[];     // [tb][U][pitch]
  __shared__ Chunk<T> s_row[2][kRotThreads];
  pdl_wait();
  pdl_trigger();
  const int t0 = blockIdx.x * A.tb, nt = min(A.tb, A.T - t0);
  const int h0 = blockIdx.y * A.hs, nh = min(A.hs, A.heads - h0);
  const int per = A.copy ? A.D / U : (2 * A.half + U - 1) / U;           // at most kRotThreads
  const int step = kRotThreads / per, rows = nt * nh;
  const int row0 = threadIdx.x / per, c = threadIdx.x - row0 * per;
  const T *x = static_cast<const T *>(A.x) + t0 * A.xt + h0 * A.xh + c * U;
  T *y = static_cast<T *>(A.y) + t0 * A.yt + h0 * A.yh + c * U;
  const int dt = step / nh, dh = step - dt * nh;
  int t = row0 / nh, h = row0 - t * nh;
  auto load = [&](int row) {
    Chunk<T> v;
    if (row < rows && row0 < step) v = *reinterpret_cast<const Chunk<T> *>(x + (t * A.xt + h * A.xh));
    return v;
  };
  Chunk<T> now = load(row0);
  all_angles<U>(A, t0, nt, s_cs);
  for (int first = 0, buf = 0; first < rows; first += step, buf ^= 1) {
    const bool there = first + row0 < rows && row0 < step;
    const int tok = t;
    const int64_t to = t * A.yt + h * A.yh;
    s_row[buf][threadIdx.x] = now;
    Chunk<T> v = now;
    h += dh;
    t += dt;
    if (h >= nh) {
      h -= nh;
      ++t;
    }
    now = load(first + step + row0);
    __syncthreads();
    if (!there) continue;
    const T *own = reinterpret_cast<const T *>(s_row[buf] + row0 * per);
    const float2 *cs = s_cs + tok * U * pitch<U>(A.half);
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int col = c * U + j;
      if (col >= 2 * A.half) break;
      const bool upper = col >= A.half;
      const int pair = upper ? col - A.half : col;
      const float2 p = cs[place_in<U>(A.half, pair)];
      const float fu = to_f(v.v[j]), fw = to_f(own[upper ? col - A.half : col + A.half]) * p.y;
      from_f(upper ? fmaf(fu, p.x, fw) : fmaf(fu, p.x, -fw), v.v[j]);
    }
    *reinterpret_cast<Chunk<T> *>(y + to) = v;
  }
}

struct RotAppendArgs {
  asf_kv_cache c;
  const int32_t *table;
  int max_pages, R, T;
  const int32_t *lens, *begin, *pos;
  int q_heads, half;
  const uint64_t *turns;
  float mul;
  const __half *q, *k, *v;
  int64_t qt, kt, vt;                  // elements from token to token
  __half *qo;
  int32_t *err;
};

// A thread takes VEC pairs, or as many columns that pass, of a token's query or key
// head, or 16 bytes of its value head.  Latency bounds it: positions and ranges,
// then the table, then the store; 32 requests of 72 heads 3.6 us (9.8 where the host has
// to call it each time).
template <int VEC, bool PAIRS>
__global__ void __launch_bounds__(128) k_rotary_append(RotAppendArgs A) {
  pdl_wait();
  pdl_trigger();
  const int D = A.c.head_dim, turned = A.half / VEC, kPass = 2 * VEC, per = turned + (D - 2 * A.half) / kPass;
  const int qk = (A.q_heads + A.c.heads) * per, each = qk + A.c.heads * (D / 8), total = A.T * each;
  const int i = blockIdx.x * blockDim.x + threadIdx.x, at = min(i, total - 1);
  const int tok = at / each, in = at - tok * each;
  const bool value = in >= qk;
  const int unit = value ? D / 8 : per, item = value ? in - qk : in;
  int head = item / unit;
  const int c = item - head * unit;
  const bool query = !value && head < A.q_heads;
  if (!value && !query) head -= A.q_heads;
  const __half *from = (value ? A.v + tok * A.vt : query ? A.q + tok * A.qt : A.k + tok * A.kt) + (int64_t)head * D;
  Pairs<VEC, PAIRS> x;
  uint4 whole = make_uint4(0, 0, 0, 0);
  const int col = value ? c * 8 : 2 * A.half + (c - turned) * kPass;
  const bool turns = !value && c < turned;
  if (value) whole = *reinterpret_cast<const uint4 *>(from + col);
  else if (turns) x.load(from, c, A.half);
  else x.load_pass(from + col);
  const Place w = place_of(A.lens, A.begin, A.R, A.T, tok, A.err, i == 0);
  if (i >= total || w.r < 0) return;   // behind the last range: nothing is written
  __half *to = A.qo + ((int64_t)tok * A.q_heads + head) * D;
  if (!query) {
    const int64_t pi = w.pos / A.c.page;
    int id = -1;
    if (w.pos >= 0 && pi < A.max_pages) id = A.table[(int64_t)w.r * A.max_pages + pi];
    if ((unsigned)id >= (unsigned)A.c.pages) {
      flag_error(A.err, kErrIndex);
      return;
    }
    to = static_cast<__half *>(value ? A.c.v : A.c.k) + (int64_t)id * A.c.page_stride +
         (w.pos - pi * A.c.page) * A.c.token_stride + (int64_t)head * A.c.head_stride;
  }
  if (value) {
    *reinterpret_cast<uint4 *>(to + col) = whole;
  } else if (turns) {
    float2 cs[VEC];
    const int pos = A.pos[tok];
#pragma unroll
    for (int j = 0; j < VEC; ++j) cs[j] = cos_sin(pos, A.turns[c * VEC + j], A.mul);
    x.turn(cs);
    x.store(to, c, A.half);
  } else {
    x.store_pass(to + col);
  }
}

// ------------------------------------------------------------------ host --
asf_status check_rotary(const asf_rotary *r) {
  if (!r || !r->turns || r->head_dim <= 0 || r->rot_dim <= 0 || r->rot_dim > r->head_dim || r->rot_dim % 2 ||
      !std::isfinite(r->scale))
    return ASF_ERR_INVALID_ARG;
  if (r->head_dim > ASF_MAX_ROTARY_DIM || (r->layout != ASF_ROTARY_HALF && r->layout != ASF_ROTARY_PAIRS))
    return ASF_ERR_UNSUPPORTED;
  if (reinterpret_cast<uintptr_t>(r->turns) & 7u) return ASF_ERR_MISALIGNED;
  return ASF_OK;
}
// pairs of an access: what divides the turned half, 16 bytes at most
int pairs_of(int half, int most) {
  int v = most;
  while (half % v) v /= 2;
  return v;
}
// one past the last element of [T][heads][D]
int64_t extent(int T, int heads, int64_t ts, int64_t hs, int D) { return (T - 1) * ts + (heads - 1) * hs + D; }
// whether no two heads of [T][heads][D] meet
bool apart(int T, int heads, int64_t ts, int64_t hs, int D) {
  return (heads == 1 || hs >= D) && (T == 1 || ts >= D) &&
         (heads == 1 || T == 1 || ts >= (heads - 1) * hs + D || hs >= (T - 1) * ts + D);
}

// f / 2 pi modulo 1 in units of 2^-64, rounded to the nearest: |f| < 2^100 is a whole number
// below 2^53 times a power of two, 1 / 2 pi is taken to 192 bits, and their product is
// exact, so that what is rounded is off by less than 2^-28 units.
void turns_of(double f, uint64_t &out) {
  static const uint64_t inv[3] = {0x36d8a5664f10e410ull, 0x7f09d5f47d4d3770ull, 0x28be60db9391054aull};
  int e;
  const uint64_t whole = (uint64_t)std::ldexp(std::frexp(std::fabs(f), &e), 53);   // |f| = whole 2^(e - 53)
  uint64_t p[4];                       // whole / 2 pi in units of 2^-192
  unsigned __int128 carry = 0;
  for (int i = 0; i < 3; ++i) {
    carry += (unsigned __int128)whole * inv[i];
    p[i] = (uint64_t)carry;
    carry >>= 64;
  }
  p[3] = (uint64_t)carry;
  auto bits = [&](int at) {            // 64 of them
    const int w = at / 64, o = at % 64;
    uint64_t v = w < 4 ? p[w] >> o : 0;
    if (o && w + 1 < 4) v |= p[w + 1] << (64 - o);
    return v;
  };
  const int from = 192 - 64 + 53 - e;  // of the unit; 81 at least
  const uint64_t t = bits(from) + (bits(from - 1) & 1);
  out = f < 0. ? 0 - t : t;
}

template <typename T>
cudaError_t run_rotary(const RotArgs &a, int layout, dim3 grid, size_t smem, cudaStream_t st) {
  return layout == ASF_ROTARY_PAIRS          ? launch(k_rotary<T, true>, grid, dim3(kRotThreads), smem, st, a)
         : a.half % (16 / (int)sizeof(T)) == 0 ? launch(k_rotary<T, false>, grid, dim3(kRotThreads), smem, st, a)
                                               : launch(k_rotary_odd<T>, grid, dim3(kRotThreads), smem, st, a);
}
template <int VEC>
cudaError_t run_append(const RotAppendArgs &a, int layout, int64_t items, cudaStream_t st) {
  const dim3 grid((unsigned)((items + 127) / 128));
  return layout == ASF_ROTARY_PAIRS ? launch(k_rotary_append<VEC, true>, grid, dim3(128), 0, st, a)
                                    : launch(k_rotary_append<VEC, false>, grid, dim3(128), 0, st, a);
}

}  // namespace

extern "C" {

asf_status asf_rotary_frequencies(int32_t rot_dim, double base, int32_t scaling, double factor, double original,
                                  double *freq_out, float *scale_out) {
  if (rot_dim <= 0 || rot_dim % 2 || !(base > 1.) || !std::isfinite(base) || !freq_out || !scale_out) return ASF_ERR_INVALID_ARG;
  if (rot_dim > ASF_MAX_ROTARY_DIM || scaling < ASF_ROTARY_PLAIN || scaling > ASF_ROTARY_YARN) return ASF_ERR_UNSUPPORTED;
  if (scaling != ASF_ROTARY_PLAIN && (!(factor >= 1.) || !std::isfinite(factor))) return ASF_ERR_INVALID_ARG;
  if (scaling == ASF_ROTARY_YARN && (!(original >= 1.) || !std::isfinite(original))) return ASF_ERR_INVALID_ARG;
  const int n = rot_dim / 2;
  if (scaling == ASF_ROTARY_NTK && rot_dim > 2) base *= std::pow(factor, (double)rot_dim / (rot_dim - 2));
  *scale_out = scaling == ASF_ROTARY_YARN ? (float)(0.1 * std::log(factor) + 1.) : 1.f;
  // YaRN: the pairs that make 32 turns in the original context, and one
  auto pair_of = [&](double turns) {
    return rot_dim * std::log(original / (2. * 3.14159265358979323846 * turns)) / (2. * std::log(base));
  };
  const double low = scaling == ASF_ROTARY_YARN ? std::max(std::floor(pair_of(32.)), 0.) : 0.;
  const double high = scaling == ASF_ROTARY_YARN ? std::min(std::ceil(pair_of(1.)), rot_dim - 1.) : 0.;
  for (int i = 0; i < n; ++i) {
    const double f = std::pow(base, -2. * i / rot_dim);
    const double ramp = std::min(std::max((i - low) / std::max(high - low, 0.001), 0.), 1.);
    freq_out[i] = scaling == ASF_ROTARY_LINEAR ? f / factor
                  : scaling == ASF_ROTARY_YARN ? f * (1. - ramp) + f / factor * ramp
                                               : f;
  }
  return ASF_OK;
}

asf_status asf_rotary_turns(const double *freq, int32_t n, uint64_t *turns_out) {
  if (!freq || !turns_out || n < 1) return ASF_ERR_INVALID_ARG;
  for (int i = 0; i < n; ++i)
    if (!(std::fabs(freq[i]) < 0x1p100)) return ASF_ERR_INVALID_ARG;
  for (int i = 0; i < n; ++i) turns_of(freq[i], turns_out[i]);
  return ASF_OK;
}

asf_status asf_rotary_apply(const asf_rotary *rot, const void *x, asf_dtype dtype, int32_t T, int32_t heads,
                            int64_t x_token_stride, int64_t x_head_stride, const int32_t *pos, void *y,
                            int64_t y_token_stride, int64_t y_head_stride, asf_stream_t stream) {
  const asf_status s = check_rotary(rot);
  if (s != ASF_OK) return s;
  if (!x || !y || !pos || T < 1 || heads < 1 || x_token_stride < 0 || x_head_stride < 0 || y_token_stride < 0 || y_head_stride < 0)
    return ASF_ERR_INVALID_ARG;
  if (dtype != ASF_F16 && dtype != ASF_F32) return ASF_ERR_UNSUPPORTED;
  const int D = rot->head_dim, size = dtype == ASF_F16 ? 2 : 4, per16 = 16 / size;
  if (!al16(x) || !al16(y) || !al4(pos) || D % per16 || x_token_stride % per16 || x_head_stride % per16 ||
      y_token_stride % per16 || y_head_stride % per16)
    return ASF_ERR_MISALIGNED;
  if (heads > ASF_MAX_ROTARY_HEADS) return ASF_ERR_UNSUPPORTED;
  if (!apart(T, heads, y_token_stride, y_head_stride, D)) return ASF_ERR_INVALID_ARG;
  const bool in_place = x == y && (T == 1 || x_token_stride == y_token_stride) && (heads == 1 || x_head_stride == y_head_stride);
  if (!in_place && overlap(x, (size_t)extent(T, heads, x_token_stride, x_head_stride, D) * size, y,
                           (size_t)extent(T, heads, y_token_stride, y_head_stride, D) * size))
    return ASF_ERR_INVALID_ARG;
  const int half = rot->rot_dim / 2;
  RotArgs a{x, y, x_token_stride, x_head_stride, y_token_stride, y_head_stride, T, heads, D, half, rot->turns, rot->scale,
            pos, 1, heads, !in_place};
  // places of a head: ASF_MAX_ROTARY_DIM / 4 = kRotThreads at most
  const bool wide = rot->layout == ASF_ROTARY_HALF && half % per16 == 0;
  const int64_t per = wide ? half / per16 + (in_place ? 0 : (D - 2 * half) / per16) : in_place ? (2 * half + per16 - 1) / per16 : D / per16;
  const int64_t chunks = (int64_t)T * heads * per, wave = (int64_t)sm_count() * 2048 * 2;
  a.hs = (int)std::min<int64_t>(heads, std::max<int64_t>(1, kRotThreads * (chunks < wave ? 1 : kItems) / per));
  if (a.hs == heads)
    a.tb = (int)std::max<int64_t>(1, std::min<int64_t>({8, (int64_t)kRotThreads * kItems / (heads * per), chunks / wave}));
  const dim3 grid((unsigned)(((int64_t)T + a.tb - 1) / a.tb), (unsigned)((heads + a.hs - 1) / a.hs));
  const size_t smem = (size_t)a.tb * (half + per16) * sizeof(float2);     // pitches round up
  cudaStream_t st = (cudaStream_t)stream;
  return cuda_status(dtype == ASF_F16 ? run_rotary<__half>(a, rot->layout, grid, smem, st)
                                      : run_rotary<float>(a, rot->layout, grid, smem, st));
}

asf_status asf_rotary_append(const asf_rotary *rot, const asf_kv_cache *cache, const int32_t *table, int32_t max_pages,
                             int32_t R, const int32_t *lens, const int32_t *begin, int32_t T, const int32_t *pos,
                             int32_t q_heads, const void *q, int64_t q_stride, void *q_out, const void *k, int64_t k_stride,
                             const void *v, int64_t v_stride, void *ws, size_t ws_bytes, asf_stream_t stream) {
  asf_status s = check_rotary(rot);
  if (s == ASF_OK) s = check_cache(cache);
  if (s == ASF_OK) s = check_requests(table, max_pages, R, lens, begin, T);
  if (s == ASF_OK) s = check_tables(table, max_pages, cache->page, lens, begin);
  if (s != ASF_OK) return s;
  const int D = cache->head_dim;
  if (!pos || !q || !q_out || !k || !v || rot->head_dim != D || q_heads < 1) return ASF_ERR_INVALID_ARG;
  if (q_heads > ASF_MAX_KV_HEADS * ASF_MAX_HEAD_GROUP) return ASF_ERR_UNSUPPORTED;
  if (!al16(q) || !al16(q_out) || !al16(k) || !al16(v) || !al4(pos) || q_stride % 8 || k_stride % 8 || v_stride % 8)
    return ASF_ERR_MISALIGNED;
  const int64_t qw = (int64_t)q_heads * D, kw = (int64_t)cache->heads * D;
  if (T > 1 && (q_stride < qw || k_stride < kw || v_stride < kw)) return ASF_ERR_INVALID_ARG;
  s = check_ws(ws, ws_bytes, kHeaderBytes);
  if (s != ASF_OK) return s;
  // q may be turned in place; a thread that has not read yet is in nobody's way otherwise
  const size_t out = (size_t)T * qw * 2;
  const bool in_place = q == q_out && (T == 1 || q_stride == qw);
  if (!in_place && overlap(q, ((size_t)(T - 1) * q_stride + qw) * 2, q_out, out)) return ASF_ERR_INVALID_ARG;
  if (overlap(k, ((size_t)(T - 1) * k_stride + kw) * 2, q_out, out) ||
      overlap(v, ((size_t)(T - 1) * v_stride + kw) * 2, q_out, out) || in_cache(cache, q_out, out))
    return ASF_ERR_INVALID_ARG;
  RotAppendArgs a{*cache, table, max_pages, R, T, lens, begin, pos, q_heads, rot->rot_dim / 2, rot->turns, rot->scale,
                  static_cast<const __half *>(q), static_cast<const __half *>(k), static_cast<const __half *>(v),
                  q_stride, k_stride, v_stride, static_cast<__half *>(q_out), &static_cast<Header *>(ws)->err};
  const int vec = pairs_of(a.half, 4);
  const int64_t items = T * ((q_heads + cache->heads) * (int64_t)(a.half / vec + (D - 2 * a.half) / (2 * vec)) + cache->heads * (D / 8));
  if (items > INT32_MAX) return ASF_ERR_UNSUPPORTED;
  cudaStream_t st = (cudaStream_t)stream;
  return cuda_status(vec == 4   ? run_append<4>(a, rot->layout, items, st)
                     : vec == 2 ? run_append<2>(a, rot->layout, items, st)
                                : run_append<1>(a, rot->layout, items, st));
}

}  // extern "C"
