// Token log probabilities with entropy, log-sum-exp and top alternatives from
// logits, their gradient, and the scoring head that calls them
// (rdt_token_logprobs, rdt_token_logprobs_backward, rdt_head_logprobs).
//
// Bound by DRAM where rows are many: the logits are read once, in the gradient
// written once. Measured, of the copy bandwidth: 4096 bf16 rows of 151,936
// 193 us (0.95), 1024 fp32 rows with 20 alternatives 101 us (0.91), gradient of
// 4096 bf16 rows 366 us (1.00). One row is bound by latency and the host: 9 us;
// rows of a few thousand logits by each CTA's start, joins and selection (8192
// bf16 rows of 4096: 17 us, 40 with 20 alternatives, 9.9 for the bytes).
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdio>
#include <cuda_fp16.h>

#include "../../include/rdt.h"
#include "common.cuh"
#include "internal.h"

namespace rdt {

namespace {

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(bf16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
template <typename T> __device__ __forceinline__ T from_f(float x);
template <> __device__ __forceinline__ float from_f<float>(float x) { return x; }
template <> __device__ __forceinline__ bf16 from_f<bf16>(float x) { return __float2bfloat16_rn(x); }
template <> __device__ __forceinline__ __half from_f<__half>(float x) { return __float2half_rn(x); }

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.693147180559945309417f;
// Exponents of 2 are kept above this (2^-1000 is 0 in fp32): -inf would make
// the products p ln p of masked tokens NaN.
constexpr float kLowest = -1000.f;

// 2^x, relative error below 2^-21, 0 for x < -126.
__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// max(x, kLowest), NaN if x is (fmaxf would drop it).
__device__ __forceinline__ float keep_finite(float x) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(kLowest));
  return r;
}
// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float nan_f() { return __int_as_float(0x7fffffff); }

// Larger value first, equal values in order of index: a whole number whose
// order is that order; 0 for -inf (never an alternative). NaN must not come here.
__device__ __forceinline__ uint64_t order_key(float z, uint32_t idx) {
  if (z == -INFINITY) return 0;
  uint32_t b = __float_as_uint(z + 0.0f);  // both zeros are one value
  b = (b & 0x80000000u) ? ~b : (b | 0x80000000u);
  return (static_cast<uint64_t>(b) << 32) | (0xffffffffu - idx);
}
__device__ __forceinline__ float key_value(uint64_t key) {
  const uint32_t b = static_cast<uint32_t>(key >> 32);
  return __uint_as_float((b & 0x80000000u) ? (b & 0x7fffffffu) : ~b);
}
__device__ __forceinline__ uint32_t key_index(uint64_t key) {
  return 0xffffffffu - static_cast<uint32_t>(key);
}

// ------------------------------------------------------------ 16-byte vectors
// kPer elements of a row, as loaded; filled with -inf where the row has none.
//
// kFloor: in a row whose maximum is `near`, a logit of kFloor or less has
// probability 0; raised to it, masked tokens need no case of their own.
template <typename T> struct Vec;
// The maximum of n vectors of 16-bit elements, two elements to an instruction.
template <typename H2, int n>
__device__ __forceinline__ float max_of_halves(const uint4* r) {
  const H2* h = reinterpret_cast<const H2*>(r);
  H2 m = h[0];
#pragma unroll
  for (int i = 1; i < 4 * n; ++i) m = __hmax2(m, h[i]);
  return fmaxf(__low2float(m), __high2float(m));
}
template <> struct Vec<float> {
  static constexpr float kFloor = -0x1p100f;
  // For every logit_scale; c (z - m) stays finite.
  static __device__ __forceinline__ bool near(float m, float) { return m > kFloor && m <= -kFloor; }
  static constexpr int kPer = 4;
  static constexpr uint32_t kNone = 0xff800000u;
  static __device__ __forceinline__ void unpack(const uint4& r, float* x) {
    x[0] = __uint_as_float(r.x); x[1] = __uint_as_float(r.y);
    x[2] = __uint_as_float(r.z); x[3] = __uint_as_float(r.w);
  }
  template <int n = 1>
  static __device__ __forceinline__ float max(const uint4* r) {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < n; ++i)
      m = fmaxf(m, fmaxf(fmaxf(__uint_as_float(r[i].x), __uint_as_float(r[i].y)),
                         fmaxf(__uint_as_float(r[i].z), __uint_as_float(r[i].w))));
    return m;
  }
  // The elements, raised to kFloor (NaN stays).
  static __device__ __forceinline__ void raised(const uint4& r, float* x) {
    unpack(r, x);
#pragma unroll
    for (int i = 0; i < kPer; ++i) x[i] = max_nan(x[i], kFloor);
  }
};
template <> struct Vec<bf16> {
  static constexpr float kFloor = -0x1p100f;
  static __device__ __forceinline__ bool near(float m, float) { return m > kFloor && m <= -kFloor; }
  static constexpr int kPer = 8;
  static constexpr uint32_t kNone = 0xff80ff80u;
  static __device__ __forceinline__ void unpack(const uint4& r, float* x) {
    x[0] = bf16lo(r.x); x[1] = bf16hi(r.x); x[2] = bf16lo(r.y); x[3] = bf16hi(r.y);
    x[4] = bf16lo(r.z); x[5] = bf16hi(r.z); x[6] = bf16lo(r.w); x[7] = bf16hi(r.w);
  }
  template <int n = 1>
  static __device__ __forceinline__ float max(const uint4* r) {
    return max_of_halves<__nv_bfloat162, n>(r);
  }
  // kFloor is a bf16 value: two elements are raised at once.
  static __device__ __forceinline__ void raised(const uint4& r, float* x) {
    const __nv_bfloat162 low = __float2bfloat162_rn(kFloor);
    uint4 q = r;
    __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&q);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __hmax2_nan(h[i], low);
    unpack(q, x);
  }
};
template <> struct Vec<__half> {
  static constexpr float kFloor = -65504.f;  // the lowest finite one
  static __device__ __forceinline__ bool near(float m, float c) { return (m - kFloor) * c > 160.f; }
  static constexpr int kPer = 8;
  static constexpr uint32_t kNone = 0xfc00fc00u;
  static __device__ __forceinline__ void unpack(const uint4& r, float* x) {
    const __half2* h = reinterpret_cast<const __half2*>(&r);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(h[i]);
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
  template <int n = 1>
  static __device__ __forceinline__ float max(const uint4* r) {
    return max_of_halves<__half2, n>(r);
  }
  static __device__ __forceinline__ void raised(const uint4& r, float* x) {
    const __half2 low = __float2half2_rn(kFloor);
    uint4 q = r;
    __half2* h = reinterpret_cast<__half2*>(&q);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __hmax2_nan(h[i], low);
    unpack(q, x);
  }
};

// A row as 16-byte vectors of memory: vector v holds elements v kPer - head to
// that + kPer - 1. The first and the last may reach outside the row; only
// their elements inside it are read.
template <typename T>
struct Row {
  const T* z;      // element 0
  const uint4* v0; // the vector that holds it
  int head, vocab;
  int vectors;
  int whole0, whole1;  // the vectors that lie in the row as a whole: [whole0, whole1)
  __device__ __forceinline__ Row(const T* row, int n) : z(row), vocab(n) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(row);
    v0 = reinterpret_cast<const uint4*>(at & ~static_cast<uintptr_t>(15));
    head = static_cast<int>((at & 15) / sizeof(T));
    vectors = static_cast<int>((static_cast<int64_t>(head) + n + Vec<T>::kPer - 1) / Vec<T>::kPer);
    whole0 = head > 0;
    whole1 = (head + n) / Vec<T>::kPer;
  }
  __device__ __forceinline__ int first_of(int v) const { return v * Vec<T>::kPer - head; }
  __device__ __forceinline__ bool whole(int v) const { return v >= whole0 && v < whole1; }
  // v in [0, vectors)
  __device__ __forceinline__ uint4 load(int v) const {
    return whole(v) ? v0[v] : load_part(first_of(v));
  }
  // Starts to copy whole vector v to shared memory; the thread that called finds it there
  // after a wait for its copies.
  __device__ __forceinline__ void fetch(int v, uint4* to) const {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(smem_u32(to)),
                 "l"(v0 + v)
                 : "memory");
  }
  __device__ __noinline__ uint4 load_part(int j) const {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 4) {
        w[i] = static_cast<unsigned>(j + i) < static_cast<unsigned>(vocab)
                   ? __float_as_uint(to_f(z[j + i])) : Vec<T>::kNone;
      } else {
        const uint16_t* h = reinterpret_cast<const uint16_t*>(z);
        const int e = j + 2 * i;
        const uint32_t none = Vec<T>::kNone & 0xffffu;
        const uint32_t lo = static_cast<unsigned>(e) < static_cast<unsigned>(vocab) ? h[e] : none;
        const uint32_t hi =
            static_cast<unsigned>(e + 1) < static_cast<unsigned>(vocab) ? h[e + 1] : none;
        w[i] = lo | (hi << 16);
      }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  static __device__ __forceinline__ uint4 none() {
    return make_uint4(Vec<T>::kNone, Vec<T>::kNone, Vec<T>::kNone, Vec<T>::kNone);
  }
};

// ------------------------------------------------------------ running softmax
// Of a set of logits z, with c = logit_scale log2 e and t = c (z - m):
// m the maximum (-inf for none; a NaN is not seen), s0 = sum 2^t, s1 = sum
// 2^t t. A NaN or +inf in the set makes s0 NaN.
struct Sums {
  float m, s0, s1;
};
__device__ __forceinline__ float base_of(float m) { return m == -INFINITY ? 0.f : m; }
// The same sums with the larger reference m.
__device__ __forceinline__ void rebase(Sums& a, float m, float c) {
  const float t = keep_finite((a.m - base_of(m)) * c);
  const float f = exp2_fast(t);
  a.s1 = f * fmaf(t, a.s0, a.s1);
  a.s0 = f * a.s0;
  a.m = m;
}
// ------------------------------------------------------- lists of 32, by lane
// A warp holds a list of 32 keys, one per lane, largest in lane 0.
constexpr unsigned kAll = 0xffffffffu;
__device__ __forceinline__ uint64_t keep_of(uint64_t a, uint64_t b, bool larger) {
  return (a > b) == larger ? a : b;
}
// The 32 largest of two ordered lists, in order; `back` holds the second one's
// keys in reverse (its lane i the key of place 31 - i).
__device__ __forceinline__ uint64_t merge32(uint64_t k, uint64_t back) {
  const int lane = threadIdx.x & 31;
  k = k > back ? k : back;
#pragma unroll
  for (int step = 16; step > 0; step >>= 1) {
    const uint64_t other = __shfl_xor_sync(kAll, k, step);
    k = keep_of(k, other, (lane & step) == 0);
  }
  return k;
}
// Puts one key (the same in every lane, in the list nowhere yet) in its place.
__device__ __forceinline__ uint64_t insert32(uint64_t k, uint64_t x) {
  const int lane = threadIdx.x & 31;
  const int place = __popc(__ballot_sync(kAll, k > x));
  const uint64_t up = __shfl_up_sync(kAll, k, 1);
  return lane < place ? k : lane == place ? x : up;
}

// Stores to shared memory of a CTA of the cluster (address from mapa_shared).
__device__ __forceinline__ void st_cluster_f32(uint32_t at, float x) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at), "f"(x) : "memory");
}
__device__ __forceinline__ void st_cluster_u64(uint32_t at, uint64_t x) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(at), "l"(x) : "memory");
}

// Each kernel of this file may be launched while the one before it in the
// stream still runs, and waits here for its end before it touches memory: of
// two calls in a row the second's launch is hidden (programmatic launch; after
// a kernel that does not take part the launch is an ordinary one). Nothing is
// read through the read-only path (__ldg, const __restrict__): that is for
// memory nobody writes while the kernel is there, and this one may be there
// while the kernel before it writes.
__device__ __forceinline__ void after_previous_kernel() {
  asm volatile("griddepcontrol.wait;\n\tgriddepcontrol.launch_dependents;" ::: "memory");
}
inline cudaLaunchAttribute overlapping_launch(bool yes = true) {
  cudaLaunchAttribute at = {};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = yes;
  return at;
}

struct LogprobArgs {
  const void* logits;
  int64_t ld;
  int rows, vocab;
  float scale;
  const int32_t* targets;
  float *logp, *entropy, *lse;
  float2* stats;
  int top;
  int32_t* top_ids;
  float* top_logp;
  bool early;
};

constexpr int kMaxSplit = 8;  // CTAs that share a row (a cluster of the portable size)
// A group: the vectors a thread works on at once. A thread holds kStages
// groups in shared memory, all but one of them under way.
constexpr int kUnroll = 4;
template <int kThreads, int kStages>
constexpr int kRingBytes = kUnroll * kStages * kThreads * 16;
// A thread's first groups, whose maxima are all kept (8 for 256 threads: 16 would leave an SM a
// CTA less; rows for 64 threads have at most 5).
constexpr int first_of(int threads) { return threads == 128 ? 16 : 8; }
constexpr int kSample = 64;  // sets of threads whose maxima bound the row's alternatives
// Later groups that reached the bound of their time, at most (for 64 threads there are none).
constexpr int seen_of(int threads) { return threads == 64 ? 1 : threads == 256 ? 160 : 320; }
constexpr int kKeys = 256;   // candidates that are ranked by counting

template <int kThreads, bool kTop>
struct Shared {
  Sums warp_sums[kThreads / 32];
  Sums part[kMaxSplit];  // of the cluster's CTAs, in its first CTA
};
template <int kThreads>
struct Shared<kThreads, true> {
  Sums warp_sums[kThreads / 32];
  Sums part[kMaxSplit];
  unsigned long long parts[kThreads < 256 ? 1 : kMaxSplit][32];  // smaller CTAs share no row
  unsigned long long best[32], merged[32];
  bf16 first[first_of(kThreads)][kThreads];  // maxima, rounded up
  bf16 seen_max[seen_of(kThreads)];          // the same of the groups in seen_group
  uint32_t seen_group[seen_of(kThreads)];                // group kThreads + thread
  float sample[kSample];
  float bound;
  int seen, items, keys;
};
// What lies in the ring once the loop is through.
template <int kThreads>
struct Lists {
  unsigned long long list[kThreads / 32][32];
  unsigned long long key[kKeys];
  uint32_t item[first_of(kThreads) * kThreads + seen_of(kThreads)];  // group kThreads + thread
};

// The sums of kLanes (a power of 2) neighbouring lanes, in each of them.
template <int kLanes>
__device__ __forceinline__ Sums join_lanes(Sums s, float c) {
  float m = s.m;
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
  rebase(s, m, c);
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) {
    s.s0 += __shfl_xor_sync(kAll, s.s0, o);
    s.s1 += __shfl_xor_sync(kAll, s.s1, o);
  }
  return s;
}

// Notes the threads' maxima for the bound below.
template <int kThreads>
__device__ __forceinline__ void put_sample(float m, float* sample) {
#pragma unroll
  for (int o = 1; o < kThreads / kSample; o <<= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
  if (threadIdx.x % (kThreads / kSample) == 0) sample[threadIdx.x / (kThreads / kSample)] = m;
}
// The `top`-th largest of the samples: a lower bound of the `top`-th largest
// logit so far, for each set holds one at least as large. Called by all
// threads after a barrier; the bound is there after the next one.
__device__ __forceinline__ void put_bound(const float* sample, int top, float* bound) {
  if (threadIdx.x < kSample) {
    const float x = sample[threadIdx.x];
    int rank = 0;
#pragma unroll 16
    for (int j = 0; j < kSample; ++j) {
      const float y = sample[j];
      rank += y > x || (y == x && j < static_cast<int>(threadIdx.x));
    }
    if (rank == top - 1) *bound = x;
  }
}

// The CTA's sums from its threads', in every thread: the maximum first, one
// rebase, then plain sums, within warps and then between them.
template <int kWarps>
__device__ __forceinline__ Sums join_sums(Sums s, float c, Sums* warp_sums) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  rebase(s, warp_max(s.m), c);
  s.s0 = warp_sum(s.s0);
  s.s1 = warp_sum(s.s1);
  if (lane == 0) warp_sums[warp] = s;
  __syncthreads();
  return join_lanes<kWarps>(warp_sums[lane % kWarps], c);
}

// A thread's vectors v, v + kThreads, ... below v1, whatever they hold.
template <typename T, int kThreads>
__device__ __noinline__ Sums sums_of_any(const Row<T>& row, int v, int v1, float c) {
  constexpr int kPer = Vec<T>::kPer;
  constexpr int kAhead = 4;
  Sums s{-INFINITY, 0.f, 0.f};
  for (; v < v1; v += kAhead * kThreads) {
    uint4 r[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      r[u] = v + u * kThreads < v1 ? row.load(v + u * kThreads) : Row<T>::none();
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const float m = Vec<T>::max(&r[u]);
      if (m > s.m) rebase(s, m, c);
      const float base = base_of(s.m);
      float x[kPer];
      Vec<T>::unpack(r[u], x);
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const float t = keep_finite((x[i] - base) * c);
        const float e = exp2_fast(t);
        s.s0 += e;
        s.s1 = fmaf(e, t, s.s1);
      }
    }
  }
  return s;
}

// Starts the copies of a thread's group at vector g, below v1, to its part of a
// ring's stage.
template <typename T, int kThreads>
__device__ __forceinline__ void fetch_group(const Row<T>& row, int g, int v1, uint4* to) {
  if (g >= row.whole0 && g + (kUnroll - 1) * kThreads < min(v1, row.whole1)) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) row.fetch(g + u * kThreads, to + u * kThreads);
  } else {
#pragma unroll 1
    for (int u = 0; u < kUnroll; ++u) {
      const int at = g + u * kThreads;
      if (at >= v1) break;
      if (row.whole(at))
        row.fetch(at, to + u * kThreads);
      else
        to[u * kThreads] = row.load_part(row.first_of(at));
    }
  }
  asm volatile("cp.async.commit_group;" ::: "memory");
}
// The first groups, before sums_of.
template <typename T, int kThreads, int kStages>
__device__ __forceinline__ void fetch_first(const Row<T>& row, int v, int v1, uint4* ring) {
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i)
    fetch_group<T, kThreads>(row, v + i * kUnroll * kThreads, v1,
                             ring + i * kUnroll * kThreads + threadIdx.x);
}

// The same for values whose maximum (over the CTA) is `near`, without special
// values but NaN and with two elements to an instruction (256 us for 4096 bf16
// rows with one, at 0.7 of the issue slots). A thread with nothing above
// kFloor returns m = kFloor, with nothing but -inf what an empty set has. t is
// 0 and 2^t 1 at the maximum itself, so a row with one token left has ln p = 0.
//
// The loads run kStages - 1 groups ahead (fetch_first), each thread's into its own part of
// `ring` (no barrier: a thread reads only what it copied). `raw` receives the
// thread's maximum (-inf for none, NaN not seen).
//
// For alternatives the maxima of the first groups are kept; then, and at each
// doubling of the groups, the row so far bounds its `top`-th largest logit, and
// later groups are kept if they reach that bound: some 24 for 20 alternatives
// and doubling of a row of random logits. All threads make `groups` turns.
template <typename T, int kThreads, int kStages, bool kTop>
__device__ __forceinline__ Sums sums_of(const Row<T>& row, int v, int v1, int groups, float c,
                                        uint4* ring, Shared<kThreads, kTop>& sh, int alternatives,
                                        float& raw) {
  constexpr int kPer = Vec<T>::kPer;
  constexpr int kStep = kUnroll * kThreads;
  ring += threadIdx.x;
  float m = Vec<T>::kFloor, bound = INFINITY;
  int renew = first_of(kThreads);
  uint64_t s0 = 0, s1 = 0;
  const uint64_t cc = pack2(c, c);
  for (int group = 0, stage = 0; group < groups; ++group, v += kStep) {
    if constexpr (kTop) {
      if (group == renew) {
        put_sample<kThreads>(raw, sh.sample);
        __syncthreads();
        put_bound(sh.sample, alternatives, &sh.bound);
        __syncthreads();
        bound = sh.bound;
        renew *= 2;
      }
    }
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
    uint4 r[kUnroll];
    if (v + (kUnroll - 1) * kThreads < v1) {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) r[u] = ring[(stage * kUnroll + u) * kThreads];
    } else {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)
        r[u] = v + u * kThreads < v1 ? ring[(stage * kUnroll + u) * kThreads] : Row<T>::none();
    }
    fetch_group<T, kThreads>(row, v + (kStages - 1) * kStep, v1,
                             ring + (stage == 0 ? kStages - 1 : stage - 1) * kStep);
    stage = stage == kStages - 1 ? 0 : stage + 1;
    const float top = Vec<T>::template max<kUnroll>(r);
    raw = fmaxf(raw, top);
    if (top > m) {
      const float t = keep_finite((m - top) * c), f = exp2_fast(t);
      const uint64_t ff = pack2(f, f), tt = pack2(t, t);
      s1 = mul2(ff, fma2(tt, s0, s1));
      s0 = mul2(ff, s0);
      m = top;
    }
    if constexpr (kTop) {
      if (group < first_of(kThreads)) {
        sh.first[group][threadIdx.x] = __float2bfloat16_ru(top);
      } else if (top >= bound && top > -INFINITY) {
        const int at = atomicAdd(&sh.seen, 1);
        if (at < seen_of(kThreads)) {
          sh.seen_group[at] = static_cast<uint32_t>(group) * kThreads + threadIdx.x;
          sh.seen_max[at] = __float2bfloat16_ru(top);
        }
      }
    }
    const uint64_t mm = pack2(-m, -m);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      float x[kPer];
      Vec<T>::raised(r[u], x);
#pragma unroll
      for (int i = 0; i < kPer; i += 2) {
        const uint64_t t = mul2(add2(pack2(x[i], x[i + 1]), mm), cc);
        const float2 f = unpack2(t);
        const uint64_t e = pack2(exp2_fast(f.x), exp2_fast(f.y));
        s0 = add2(s0, e);
        s1 = fma2(e, t, s1);
      }
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  const float2 a = unpack2(s0), b = unpack2(s1);
  const float sum = a.x + a.y;
  if (raw == -INFINITY && sum == sum) return Sums{-INFINITY, 0.f, 0.f};
  return Sums{m, sum, b.x + b.y};
}

// f(element, index) for the elements of the listed groups that are at least
// `low` (all groups where item is null); the vectors are spread over the
// threads, kReread of each under way. With kWhole f is called by whole warps,
// with -inf where a lane has no such element.
template <typename T, int kThreads, bool kWhole, typename F>
__device__ __forceinline__ void for_each_candidate(const Row<T>& row, int v0, int v1,
                                                   const uint32_t* item, int items, float low,
                                                   F f) {
  constexpr int kPer = Vec<T>::kPer;
  constexpr int kReread = 2;
  const int lane = threadIdx.x & 31;
  const int pairs = items * kUnroll;
  for (int q = threadIdx.x; q - lane < pairs; q += kReread * kThreads) {
    uint4 r[kReread];
    int at[kReread];
#pragma unroll
    for (int u = 0; u < kReread; ++u) {
      const int pair = q + u * kThreads;
      r[u] = Row<T>::none();
      at[u] = v0;
      if (pair < pairs) {
        const int id = item ? static_cast<int>(item[pair / kUnroll]) : pair / kUnroll;
        at[u] = v0 + id % kThreads + (id / kThreads * kUnroll + pair % kUnroll) * kThreads;
        if (at[u] < v1) r[u] = row.load(at[u]);
      }
    }
#pragma unroll
    for (int u = 0; u < kReread; ++u) {
      const bool some = Vec<T>::max(&r[u]) >= low;
      if (kWhole ? !__any_sync(kAll, some) : !some) continue;
      float x[kPer];
      Vec<T>::unpack(r[u], x);
#pragma unroll
      for (int e = 0; e < kPer; ++e) f(x[e] >= low ? x[e] : -INFINITY, row.first_of(at[u]) + e);
    }
  }
}

// The CTA's 32 largest elements among the candidates, to best[]: for any
// number of them (ties, or few finite logits). list: scratch, 32 keys a warp.
template <typename T, int kThreads>
__device__ __noinline__ void select_any(const Row<T>& row, int v0, int v1, const uint32_t* item,
                                        int items, float low, int top,
                                        unsigned long long (*list)[32], unsigned long long* best) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint64_t mine = 0;
  for_each_candidate<T, kThreads, true>(
      row, v0, v1, item, items, low, [&](float x, int index) {
        const uint64_t k = order_key(x, index);
        const uint64_t least = __shfl_sync(kAll, mine, top - 1);
        unsigned who = __ballot_sync(kAll, k > least);
        while (who) {
          const int l = __ffs(who) - 1;
          who &= who - 1;
          mine = insert32(mine, __shfl_sync(kAll, k, l));
        }
      });
  list[warp][lane] = mine;
  for (int step = kThreads / 64; step > 0; step >>= 1) {
    __syncthreads();
    if (warp < step) {
      mine = merge32(mine, list[warp + step][31 - lane]);
      list[warp][lane] = mine;
    }
  }
  if (warp == 0) best[lane] = mine;
}

// A row (or, in a cluster of `split` CTAs, 1 / split of it) per CTA, read once.
// Each thread keeps the running maximum and sums of its vectors in registers;
// warps, the CTA and the cluster join them in a fixed order.
//
// Alternatives: the groups that the loop kept and whose maximum reaches the
// whole row's bound are read again (of random logits about 64 ln(64 / (64 -
// top)) elements are above it, 24 for 20), and what reaches it there is ranked
// by counting.
template <typename T, int kThreads, int kStages, bool kTop>
__global__ void __launch_bounds__(kThreads) logprobs_kernel(const LogprobArgs a, int split) {
  constexpr int kWarps = kThreads / 32;
  extern __shared__ uint4 ring[];  // kRingBytes; after the loop, lists
  __shared__ Shared<kThreads, kTop> sh;
  after_previous_kernel();
  const int row_i = split == 1 ? blockIdx.x : blockIdx.x / split;
  const int part = split == 1 ? 0 : blockIdx.x % split;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const float inf = INFINITY;
  const Row<T> row(static_cast<const T*>(a.logits) + static_cast<int64_t>(row_i) * a.ld, a.vocab);
  const int v0 = static_cast<int>(static_cast<int64_t>(row.vectors) * part / split);
  const int v1 = static_cast<int>(static_cast<int64_t>(row.vectors) * (part + 1) / split);
  // few rows: their loads start before it is known whether they are scored
  if (a.early) fetch_first<T, kThreads, kStages>(row, v0 + tid, v1, ring);
  const int target = a.targets ? a.targets[row_i] : 0;
  if (target < 0) {  // not scored (the same in every CTA of the cluster)
    if (part == 0 && tid == 0) {
      if (a.logp) a.logp[row_i] = 0.f;
      if (a.entropy) a.entropy[row_i] = 0.f;
      if (a.lse) a.lse[row_i] = 0.f;
      if (a.stats) a.stats[row_i] = make_float2(0.f, 0.f);
    }
    if (kTop && part == 0 && tid < a.top) {
      a.top_ids[static_cast<int64_t>(row_i) * a.top + tid] = -1;
      a.top_logp[static_cast<int64_t>(row_i) * a.top + tid] = 0.f;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    return;
  }
  if (!a.early) fetch_first<T, kThreads, kStages>(row, v0 + tid, v1, ring);
  // shared memory of another CTA may be written once that CTA runs: every CTA says so here and
  // waits for the others only before its stores
  if (kThreads >= 256 && split > 1) asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
  const float c = a.scale * kLog2e;
  float target_z = 0.f;  // long before it is needed
  if (tid == 0 && part == 0 && a.logp && target < a.vocab) target_z = to_f(row.z[target]);

  const int groups = (v1 - v0 + kUnroll * kThreads - 1) / (kUnroll * kThreads);
  float raw = -inf;
  if constexpr (kTop) {
    if (tid == 0) sh.seen = sh.items = sh.keys = 0;
    if (tid < 32) sh.best[tid] = sh.merged[tid] = 0;
    __syncthreads();
  }
  Sums s = sums_of<T, kThreads, kStages, kTop>(row, v0 + tid, v1, groups, c, ring, sh, a.top, raw);
  if constexpr (kTop) put_sample<kThreads>(raw, sh.sample);
  Sums all = join_sums<kWarps>(s, c, sh.warp_sums);
  if (!Vec<T>::near(all.m, c) && all.m > -inf) {  // a maximum outside the fast range
    s = sums_of_any<T, kThreads>(row, v0 + tid, v1, c);
    __syncthreads();
    all = join_sums<kWarps>(s, c, sh.warp_sums);
  }

  uint64_t list = 0;
  if constexpr (kTop) if (all.s0 == all.s0 && all.m > -inf) {  // the same in every thread
    put_bound(sh.sample, a.top, &sh.bound);
    __syncthreads();
    const float low = sh.bound;  // -inf: fewer than `top` sets hold anything
    Lists<kThreads>& lists = *reinterpret_cast<Lists<kThreads>*>(ring);
    static_assert(sizeof(Lists<kThreads>) <= kRingBytes<kThreads, kStages>, "fits the ring");
    const int seen = sh.seen;
    const bool lost = seen > seen_of(kThreads);  // rising rows: every group is looked at again
    if (!lost) {
      unsigned mask = 0;  // the thread's first groups that reach the bound
      if (raw >= low && raw > -inf) {
#pragma unroll
        for (int i = 0; i < first_of(kThreads); ++i) {
          const float m = i < groups ? bf16_to_f(sh.first[i][tid]) : -inf;
          mask |= static_cast<unsigned>(m >= low && m > -inf) << i;
        }
      }
      if (__any_sync(kAll, mask)) {  // one place for the warp's
        const int n = __popc(mask);
        int before = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int x = __shfl_up_sync(kAll, before, o);
          if (lane >= o) before += x;
        }
        int at = 0;
        if (lane == 31) at = atomicAdd(&sh.items, before);
        at = __shfl_sync(kAll, at, 31) + before - n;
        while (mask) {
          const int i = __ffs(mask) - 1;
          mask &= mask - 1;
          lists.item[at++] = static_cast<uint32_t>(i * kThreads + tid);
        }
      }
      for (int i = tid; i < seen; i += kThreads)
        if (bf16_to_f(sh.seen_max[i]) >= low)
          lists.item[atomicAdd(&sh.items, 1)] = sh.seen_group[i];
    }
    __syncthreads();
    // the order of items and keys varies, what is chosen among them does not
    const uint32_t* item = lost ? nullptr : lists.item;
    const int items = lost ? groups * kThreads : sh.items;
    for_each_candidate<T, kThreads, false>(
        row, v0, v1, item, items, low, [&](float x, int index) {
          const uint64_t k = order_key(x, index);
          if (k == 0) return;
          const int n = atomicAdd(&sh.keys, 1);
          if (n < kKeys) lists.key[n] = k;
        });
    __syncthreads();
    const int keys = sh.keys;
    if (keys <= kKeys) {
      for (int i = tid; i < keys; i += kThreads) {
        const unsigned long long k = lists.key[i];
        int rank = 0;
#pragma unroll 8
        for (int j = 0; j < keys; ++j) rank += lists.key[j] > k;
        if (rank < a.top) sh.best[rank] = k;
      }
    } else {
      select_any<T, kThreads>(row, v0, v1, item, items, low, a.top, lists.list, sh.best);
    }
    __syncthreads();
    list = sh.best[lane];
  }

  if constexpr (kThreads >= 256) if (split > 1) {
    // every part to the cluster's first CTA; it joins them in order
    asm volatile("barrier.cluster.wait;" ::: "memory");
    if (warp == 0) {
      const uint32_t p = mapa_shared(smem_u32(&sh.part[part]), 0);
      if (lane == 0) {
        st_cluster_f32(p, all.m);
        st_cluster_f32(p + 4, all.s0);
        st_cluster_f32(p + 8, all.s1);
      }
      if constexpr (kTop) st_cluster_u64(mapa_shared(smem_u32(&sh.parts[part][lane]), 0), list);
    }
    cluster_sync();
    if (part != 0) return;
    if constexpr (kTop) {
      // a key's place: its place in its own list, and in the others by halving them
      for (int i = tid; i < split * 32; i += kThreads) {
        const unsigned long long k = sh.parts[i >> 5][i & 31];
        int rank = i & 31;
        int n[kMaxSplit] = {};  // keys of list q above k, the lists side by side
#pragma unroll
        for (int step = 16; step > 0; step >>= 1)
#pragma unroll
          for (int q = 0; q < kMaxSplit; ++q)
            if (q < split && sh.parts[q][n[q] + step - 1] > k) n[q] += step;
#pragma unroll
        for (int q = 0; q < kMaxSplit; ++q) {
          if (q < split && n[q] == 31 && sh.parts[q][31] > k) n[q] = 32;
          if (q != i >> 5) rank += n[q];
        }
        if (k != 0 && rank < 32) sh.merged[rank] = k;
      }
      __syncthreads();
      list = sh.merged[lane];
    }
    if (warp == 0) {
      all = lane % kMaxSplit < split ? sh.part[lane % kMaxSplit] : Sums{-inf, 0.f, 0.f};
      all = join_lanes<kMaxSplit>(all, c);
    }
  }
  if (warp != 0) return;
  const bool live = all.s0 == all.s0, some = live && all.m > -inf;
  const float log_sum = some ? logf(all.s0) : 0.f;
  if (lane == 0) {
    if (a.logp) {
      float lp = nan_f();
      if (live && target < a.vocab)
        lp = some ? (target_z - all.m) * a.scale - log_sum : -inf;
      a.logp[row_i] = lp;
    }
    if (a.entropy)
      a.entropy[row_i] = some ? log_sum - kLn2 * (all.s1 / all.s0) : live ? 0.f : nan_f();
    if (a.lse) a.lse[row_i] = some ? fmaf(all.m, a.scale, log_sum) : live ? -inf : nan_f();
    if (a.stats)
      a.stats[row_i] = live ? make_float2(all.m, log_sum) : make_float2(nan_f(), nan_f());
  }
  if (kTop && lane < a.top) {
    const int64_t at = static_cast<int64_t>(row_i) * a.top + lane;
    const bool there = some && list != 0;
    a.top_ids[at] = there ? static_cast<int32_t>(key_index(list)) : -1;
    a.top_logp[at] = there  ? (key_value(list) - all.m) * a.scale - log_sum
                     : live ? -inf
                            : nan_f();
  }
}

template <typename T, int kThreads, int kStages, bool kTop>
cudaError_t launch_logprobs(const LogprobArgs& a, int split, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.rows) * split, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = s;
  cfg.dynamicSmemBytes = kRingBytes<kThreads, kStages>;
  static std::atomic<uint64_t> allowed{0};  // devices where the kernel may use that much
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev > 63 || !(allowed.load() >> dev & 1)) {
    e = cudaFuncSetAttribute(logprobs_kernel<T, kThreads, kStages, kTop>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(cfg.dynamicSmemBytes));
    if (e != cudaSuccess) return e;
    if (dev < 64) allowed.fetch_or(uint64_t(1) << dev);
  }
  cudaLaunchAttribute at[2];
  // CTAs that wait already sit where there was room, some SMs full and some not; long rows in
  // one or two waves lose by that (1024 rows of 151,936, 20 alternatives: fp32 105 us for 101,
  // bf16 71 for 64) what small calls and many waves win (2 us). Some that the rule leaves out
  // would win as well (2048 bf16 rows of 32,000: 35 us for 38).
  const int64_t bytes = static_cast<int64_t>(a.rows) * a.vocab * sizeof(T);
  at[0] = overlapping_launch(bytes <= (64 << 20) || a.rows >= 24 * num_sms());
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = static_cast<unsigned>(split);
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = split > 1 ? 2 : 1;
  note_launch();
  return cudaLaunchKernelEx(&cfg, logprobs_kernel<T, kThreads, kStages, kTop>, a, split);
}

// Threads by the row's vectors (a thread should have a few), CTAs per row by
// how many rows there are to fill the GPU with.
template <typename T>
cudaError_t logprobs_of(LogprobArgs a, cudaStream_t s) {
  const int vectors = a.vocab / Vec<T>::kPer;
  // Short rows: 64 threads, and two groups in shared memory so that more CTAs fit (8192 bf16
  // rows of 4096, 20 alternatives: 39 us, 44 with three).
  if (vectors <= 1024)
    return a.top ? launch_logprobs<T, 64, 2, true>(a, 1, s) : launch_logprobs<T, 64, 2, false>(a, 1, s);
  // At most a row an SM: a cluster a row, as long as each thread has four vectors (152 fp32
  // rows of 151,936, 20 alternatives: 27 us with 256 threads, 33 with 512, 39 with 128 and no
  // cluster; without alternatives 21 us with 512, 23 with 256).
  const int sms = num_sms();
  if (a.rows <= sms) {
    int split = 1;
    while (split < kMaxSplit && a.rows * split <= sms && vectors >= 4 * 1024 * split) split *= 2;
    a.early = true;
    return a.top ? launch_logprobs<T, 256, 4, true>(a, split, s)
                 : launch_logprobs<T, 512, 2, false>(a, split, s);
  }
  if (!a.top) return launch_logprobs<T, 256, 3, false>(a, 1, s);
  // Alternatives leave a CTA without loads under way for some microseconds a row; smaller and
  // more CTAs hide more of it once there are rows for them (20 alternatives, 151,936 logits: 608
  // fp32 rows 66 us with 128 threads, 75 with 256, but 304 rows 47 and 39; 4096 bf16 rows 221 and
  // 232, without alternatives 204 and 197).
  if (a.rows <= 2 * sms) return launch_logprobs<T, 256, 3, true>(a, 1, s);
  // Of 128 threads an SM holds 7 CTAs with three groups in shared memory and 9 with two. Up to 6
  // rows an SM want the three (760 fp32 rows: 81 us, 86 with two), one wave of more the two (1024
  // rows: 106, 113 with three; 1216 rows: 121 and 153), and several waves whichever leaves less of
  // the last one empty (2048 rows: 226 and 205; 2432 rows: 234 and 252). bf16 rows of 151,936, two
  // and three: 760 rows 51 and 48, 1024 rows 63 and 67, 1216 rows 72 and 86, 2048 rows 122 and 116,
  // 2432 rows 132 and 135, but 4096 rows 212 and 204; of 32,000: 760 rows 22 and 19, 1216 rows 24
  // and 29, but 1024 rows 23 and 20.
  const int deep = (a.rows - 1) / sms + 1;  // rows an SM
  const bool two = deep > 6 && (deep <= 9 || (deep + 8) / 9 * 9 <= (deep + 6) / 7 * 7);
  return two ? launch_logprobs<T, 128, 2, true>(a, 1, s) : launch_logprobs<T, 128, 3, true>(a, 1, s);
}

cudaError_t logprobs(const LogprobArgs& a, int dtype, cudaStream_t s) {
  return dtype == RDT_F32    ? logprobs_of<float>(a, s)
         : dtype == RDT_BF16 ? logprobs_of<bf16>(a, s)
                             : logprobs_of<__half>(a, s);
}

// ------------------------------------------------------------------ gradient
struct GradArgs {
  const void* logits;
  int64_t ld;
  int rows, vocab;
  float scale;
  const int32_t* targets;
  const float2* stats;
  const float *entropy, *d_logp, *d_entropy, *d_lse;
  void* out;
  int64_t ld_out;
  int pieces;  // CTAs per row
};

constexpr int kGradThreads = 256;
constexpr int kGradPer = 8;  // elements of a thread's piece: 16 bytes of a 16-bit type

// Eight elements; inside: all of them in the row and p 16-byte aligned.
template <typename T>
__device__ __forceinline__ void load_piece(const T* p, int j, int vocab, bool inside, float* x) {
  if (inside) {
    if constexpr (sizeof(T) == 4) {
      Vec<T>::unpack(*reinterpret_cast<const uint4*>(p + j), x);
      Vec<T>::unpack(*reinterpret_cast<const uint4*>(p + j + 4), x + 4);
    } else {
      Vec<T>::unpack(*reinterpret_cast<const uint4*>(p + j), x);
    }
  } else {
#pragma unroll
    for (int i = 0; i < kGradPer; ++i)
      x[i] = static_cast<unsigned>(j + i) < static_cast<unsigned>(vocab) ? to_f(p[j + i]) : 0.f;
  }
}
template <typename T>
__device__ __forceinline__ void store_piece(T* p, int j, int vocab, bool inside, const float* x) {
  if (inside) {
    if constexpr (sizeof(T) == 4) {
      *reinterpret_cast<float4*>(p + j) = make_float4(x[0], x[1], x[2], x[3]);
      *reinterpret_cast<float4*>(p + j + 4) = make_float4(x[4], x[5], x[6], x[7]);
    } else {
      uint4 r;
      T* h = reinterpret_cast<T*>(&r);
#pragma unroll
      for (int i = 0; i < kGradPer; ++i) h[i] = from_f<T>(x[i]);
      *reinterpret_cast<uint4*>(p + j) = r;
    }
  } else {
#pragma unroll
    for (int i = 0; i < kGradPer; ++i)
      if (static_cast<unsigned>(j + i) < static_cast<unsigned>(vocab)) p[j + i] = from_f<T>(x[i]);
  }
}

// With t = log2 p, A = logit_scale (d_lse - d_logp - d_entropy entropy) and
// B = logit_scale d_entropy ln 2 a row's gradient is p (A - B t), plus
// logit_scale d_logp at the target. Pieces of eight elements start where the
// output is 16-byte aligned, so the stores are whole; a row whose logits have
// another phase there loads them one by one.
template <typename T, typename O>
__global__ void __launch_bounds__(kGradThreads) logprobs_grad_kernel(const GradArgs a) {
  after_previous_kernel();
  const int row = blockIdx.x / a.pieces, part = blockIdx.x % a.pieces;
  const T* z = static_cast<const T*>(a.logits) + static_cast<int64_t>(row) * a.ld;
  O* out = static_cast<O*>(a.out) + static_cast<int64_t>(row) * a.ld_out;
  const int target = a.targets ? a.targets[row] : 0;
  const float2 st = a.stats[row];
  const float g = a.d_logp ? a.d_logp[row] : 0.f, h = a.d_entropy ? a.d_entropy[row] : 0.f;
  float coef = (a.d_lse ? a.d_lse[row] : 0.f) - g;
  if (a.d_entropy) coef -= h * a.entropy[row];
  const bool none = target < 0 || st.x == -INFINITY;
  const bool wrong = target >= a.vocab;
  const float c = a.scale * kLog2e, shift = st.y * kLog2e;
  const float big_a = wrong ? nan_f() : a.scale * coef, big_b = a.scale * h * kLn2;
  const int head = static_cast<int>((reinterpret_cast<uintptr_t>(out) / sizeof(O)) % kGradPer);
  const int pieces = static_cast<int>((static_cast<int64_t>(head) + a.vocab + kGradPer - 1) / kGradPer);
  const bool same = (reinterpret_cast<uintptr_t>(z - head) & 15) == 0;
  const int stride = a.pieces * kGradThreads;
  int q = part * kGradThreads + threadIdx.x;
  if (none) {
    const float zero[kGradPer] = {};
    for (; q < pieces; q += stride) {
      const int j = q * kGradPer - head;
      store_piece(out, j, a.vocab, j >= 0 && j <= a.vocab - kGradPer, zero);
    }
    return;
  }
  const uint64_t mm = pack2(-st.x, -st.x), cc = pack2(c, c), ss = pack2(-shift, -shift),
                 aa = pack2(big_a, big_a), bb = pack2(-big_b, -big_b);
  for (; q < pieces; q += stride) {
    const int j = q * kGradPer - head, hit = target - j;
    const bool inside = j >= 0 && j <= a.vocab - kGradPer;
    float x[kGradPer];
    load_piece(z, j, a.vocab, same && inside, x);
#pragma unroll
    for (int i = 0; i < kGradPer; i += 2) {
      const float2 t = unpack2(fma2(add2(pack2(x[i], x[i + 1]), mm), cc, ss));
      const float2 k = make_float2(keep_finite(t.x), keep_finite(t.y));
      const uint64_t e = pack2(exp2_fast(k.x), exp2_fast(k.y));
      const float2 r = unpack2(mul2(e, fma2(bb, pack2(k.x, k.y), aa)));
      x[i] = r.x;
      x[i + 1] = r.y;
    }
    if (a.d_logp && static_cast<unsigned>(hit) < static_cast<unsigned>(kGradPer)) {
#pragma unroll
      for (int i = 0; i < kGradPer; ++i)
        if (i == hit) x[i] = fmaf(a.scale, g, x[i]);
    }
    store_piece(out, j, a.vocab, inside, x);
  }
}

template <typename T>
cudaError_t launch_grad(GradArgs a, int d_dtype, cudaStream_t s) {
  const int pieces = (a.vocab + kGradPer - 1) / kGradPer;
  a.pieces = (pieces + 2 * kGradThreads - 1) / (2 * kGradThreads);  // two pieces a thread
  // ... while there are few rows, else four CTAs a row: its stats and gradients are read by
  // each (4096 bf16 rows of 151,936: 370 us; with two pieces of a thread under way at once
  // 410, the bytes in flight do not need it and the window of rows grows)
  const int64_t enough = 16LL * num_sms();
  if (static_cast<int64_t>(a.rows) * a.pieces > enough)
    a.pieces = static_cast<int>(std::max<int64_t>(
        std::min<int64_t>(a.pieces, 4), enough / a.rows));
  if (static_cast<int64_t>(a.rows) * a.pieces > INT32_MAX) a.pieces = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.rows) * a.pieces, 1, 1);
  cfg.blockDim = dim3(kGradThreads, 1, 1);
  cfg.stream = s;
  cudaLaunchAttribute at = overlapping_launch();
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  note_launch();
  return d_dtype == RDT_F32    ? cudaLaunchKernelEx(&cfg, logprobs_grad_kernel<T, float>, a)
         : d_dtype == RDT_BF16 ? cudaLaunchKernelEx(&cfg, logprobs_grad_kernel<T, bf16>, a)
                               : cudaLaunchKernelEx(&cfg, logprobs_grad_kernel<T, __half>, a);
}

constexpr int kMaxVocab = 1 << 30;  // indexes of a row's elements stay inside 32 bits

bool dtype_ok(int dtype) { return dtype == RDT_F32 || dtype == RDT_BF16 || dtype == RDT_F16; }
int dtype_bytes(int dtype) { return dtype == RDT_F32 ? 4 : 2; }

rdt_status refuse(const char* msg) {
  set_last_error(msg);
  return RDT_EINVAL;
}
rdt_status launched(cudaError_t e) {
  if (e == cudaSuccess) return RDT_OK;
  cudaGetLastError();  // not left for the next call to find
  set_last_error(cudaGetErrorString(e));
  return RDT_ECUDA;
}

// What both calls check of their logits.
const char* logits_problem(const void* logits, int dtype, int64_t ld, int rows, int vocab,
                           float scale) {
  if (!dtype_ok(dtype)) return "dtype must be RDT_F32, RDT_BF16 or RDT_F16";
  if (rows < 0 || vocab < 1 || vocab > kMaxVocab)
    return "rows must be >= 0 and vocab in [1, 2^30]";
  if (ld < vocab) return "ld must be >= vocab";
  if (!(scale >= 1e-6f && scale <= 1e6f)) return "logit_scale must be in [1e-6, 1e6]";
  if (rows > 0 && !logits) return "null pointer";
  if (reinterpret_cast<uintptr_t>(logits) % dtype_bytes(dtype))
    return "logits must be aligned to their type";
  return nullptr;
}

const char* top_problem(int top, const void* ids, const void* lp) {
  if (top < 0 || top > RDT_MAX_TOP) return "top must be in [0, RDT_MAX_TOP]";
  if ((top > 0) != (ids != nullptr) || (top > 0) != (lp != nullptr))
    return "top_ids and top_logp are given exactly when top >= 1";
  return nullptr;
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }

constexpr int64_t kHeadLogitBytes = int64_t(1) << 30;

// Rows of fp32 logits rdt_head_logprobs holds at a time.
int head_rows(int64_t tokens, int64_t vocab) {
  int64_t r = kHeadLogitBytes / (4 * vocab) / 128 * 128;
  r = std::max<int64_t>(r, 128);
  return static_cast<int>(std::min(r, tokens));
}

struct HeadScratch {
  bf16* hn;
  float *rstd, *logits;
  size_t bytes;
};
HeadScratch head_scratch(const rdt_config* c, int tokens, void* ws) {
  HeadScratch h;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    void* p = ws ? static_cast<uint8_t*>(ws) + off : nullptr;
    off = (off + bytes + 255) / 256 * 256;
    return p;
  };
  h.hn = static_cast<bf16*>(take(static_cast<size_t>(tokens) * c->hidden * 2));
  h.rstd = static_cast<float*>(take(static_cast<size_t>(tokens) * 4));
  h.logits = static_cast<float*>(
      take(static_cast<size_t>(head_rows(tokens, c->vocab)) * c->vocab * 4));
  h.bytes = off;
  return h;
}

}  // namespace

}  // namespace rdt

using namespace rdt;

extern "C" {

rdt_status rdt_token_logprobs(const void* logits, int32_t dtype, int64_t ld, int32_t rows,
                              int32_t vocab, float logit_scale, const int32_t* targets,
                              float* logp, float* entropy, float* lse, float* stats, int32_t top,
                              int32_t* top_ids, float* top_logp, void* stream) {
  if (const char* why = logits_problem(logits, dtype, ld, rows, vocab, logit_scale))
    return refuse(why);
  if (rows == 0) return RDT_OK;
  if (const char* why = top_problem(top, top_ids, top_logp)) return refuse(why);
  if (logp && !targets) return refuse("logp needs targets");
  if (!logp && !entropy && !lse && !stats && top == 0) return refuse("null pointer: no output");
  if (!aligned4(targets) || !aligned4(logp) || !aligned4(entropy) || !aligned4(lse) ||
      (reinterpret_cast<uintptr_t>(stats) & 7) || !aligned4(top_ids) || !aligned4(top_logp))
    return refuse("targets and outputs must be 4-byte aligned (stats 8-byte)");
  LogprobArgs a{logits,  ld,   rows,    vocab, logit_scale,
                targets, logp, entropy, lse,   reinterpret_cast<float2*>(stats),
                top,     top_ids, top_logp, false};
  return launched(rdt::logprobs(a, dtype, static_cast<cudaStream_t>(stream)));
}

rdt_status rdt_token_logprobs_backward(const void* logits, int32_t dtype, int64_t ld,
                                       int32_t rows, int32_t vocab, float logit_scale,
                                       const int32_t* targets, const float* stats,
                                       const float* entropy, const float* d_logp,
                                       const float* d_entropy, const float* d_lse, void* d_logits,
                                       int32_t d_dtype, int64_t ld_d, void* stream) {
  if (const char* why = logits_problem(logits, dtype, ld, rows, vocab, logit_scale))
    return refuse(why);
  if (!dtype_ok(d_dtype)) return refuse("d_dtype must be RDT_F32, RDT_BF16 or RDT_F16");
  if (ld_d < vocab) return refuse("ld_d must be >= vocab");
  if (rows == 0) return RDT_OK;
  if (!d_logp && !d_entropy && !d_lse) return refuse("null pointer: no upstream gradient");
  if (d_logp && !targets) return refuse("d_logp needs targets");
  if (d_entropy && !entropy) return refuse("d_entropy needs entropy");
  if (!stats || !d_logits) return refuse("null pointer");
  if (!aligned4(targets) || !aligned4(entropy) || !aligned4(d_logp) || !aligned4(d_entropy) ||
      !aligned4(d_lse) || (reinterpret_cast<uintptr_t>(stats) & 7))
    return refuse("row arrays must be 4-byte aligned (stats 8-byte)");
  if (reinterpret_cast<uintptr_t>(d_logits) % dtype_bytes(d_dtype))
    return refuse("d_logits must be aligned to its type");
  const uintptr_t z0 = reinterpret_cast<uintptr_t>(logits);
  const uintptr_t z1 = z0 + (static_cast<int64_t>(rows - 1) * ld + vocab) * dtype_bytes(dtype);
  const uintptr_t d0 = reinterpret_cast<uintptr_t>(d_logits);
  const uintptr_t d1 = d0 + (static_cast<int64_t>(rows - 1) * ld_d + vocab) * dtype_bytes(d_dtype);
  if (z0 < d1 && d0 < z1 && !(z0 == d0 && dtype == d_dtype && ld == ld_d))
    return refuse("d_logits overlaps logits without being them");
  GradArgs a{logits,  ld,     rows,      vocab, logit_scale, targets,
             reinterpret_cast<const float2*>(stats),
             entropy, d_logp, d_entropy, d_lse, d_logits,    ld_d, 1};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return launched(dtype == RDT_F32    ? launch_grad<float>(a, d_dtype, s)
                  : dtype == RDT_BF16 ? launch_grad<bf16>(a, d_dtype, s)
                                      : launch_grad<__half>(a, d_dtype, s));
}

size_t rdt_head_logprobs_workspace_bytes(const rdt_config* cfg, int32_t tokens) {
  if (rdt_check_config(cfg) != RDT_OK || tokens < 1) return 0;
  return head_scratch(cfg, tokens, nullptr).bytes;
}

rdt_status rdt_head_logprobs(const rdt_config* cfg, int32_t tokens, const float* h,
                             const float* gamma_f, const rdt_bf16* w_lm, float logit_scale,
                             const int32_t* targets, float* logp, float* entropy, float* lse,
                             int32_t top, int32_t* top_ids, float* top_logp, void* ws,
                             size_t ws_bytes, void* stream) {
  if (rdt_check_config(cfg) != RDT_OK) return RDT_EINVAL;
  if (tokens < 1) return refuse("tokens must be >= 1");
  if (!h || !gamma_f || !w_lm || !ws) return refuse("null pointer");
  if ((reinterpret_cast<uintptr_t>(h) | reinterpret_cast<uintptr_t>(gamma_f) |
       reinterpret_cast<uintptr_t>(w_lm)) & 15 || (reinterpret_cast<uintptr_t>(ws) & 255))
    return refuse("pointers must be 16-byte (ws 256-byte) aligned");
  if (const char* why = top_problem(top, top_ids, top_logp)) return refuse(why);
  if (logp && !targets) return refuse("logp needs targets");
  if (!logp && !entropy && !lse && top == 0) return refuse("null pointer: no output");
  if (!(logit_scale >= 1e-6f && logit_scale <= 1e6f))
    return refuse("logit_scale must be in [1e-6, 1e6]");
  const HeadScratch k = head_scratch(cfg, tokens, ws);
  if (ws_bytes < k.bytes) return refuse("workspace too small");
  const int H = cfg->hidden, V = cfg->vocab, step = head_rows(tokens, V);
  cudaError_t e = rmsnorm_fwd(h, gamma_f, k.hn, k.rstd, tokens, H, cfg->rms_eps,
                              static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return launched(e);
  for (int t = 0; t < tokens; t += step) {
    const int n = std::min(step, tokens - t);
    rdt_status st = rdt_gemm(reinterpret_cast<const rdt_bf16*>(k.hn + static_cast<int64_t>(t) * H),
                             0, H, w_lm, 0, H, n, V, H, k.logits, V, nullptr, 0, stream);
    if (st != RDT_OK) return st;
    auto row = [&](float* p) { return p ? p + t : nullptr; };
    const int64_t at = static_cast<int64_t>(t) * top;
    st = rdt_token_logprobs(k.logits, RDT_F32, V, n, V, logit_scale,
                            targets ? targets + t : nullptr, row(logp), row(entropy), row(lse),
                            nullptr, top, top_ids ? top_ids + at : nullptr,
                            top_logp ? top_logp + at : nullptr, stream);
    if (st != RDT_OK) return st;
  }
  return RDT_OK;
}

}  // extern "C"
