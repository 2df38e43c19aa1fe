// Squared sum and AdamW over many tensors at once (rdt_tensors_sq_sum,
// rdt_tensors_adamw): the tensors' addresses and sizes travel as kernel
// parameters, every tensor is cut into tiles, and the tiles of all tensors
// make one launch (one per kMaxTensors tensors).
//
// Both are bound by DRAM: each value is read and written once. Measured, of the
// copy bandwidth: squared sum of 490 M fp32 gradients 275 us (1.05), AdamW with
// 32-bit states of a 101 M block 437 us (1.02), with 8-bit states of 490 M
// 1326 us rounded at random (0.98; 0.88 with bf16 gradients, where the 91
// instructions an element weigh more), 1360 us with the step on the device.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cuda_fp8.h>
#include <new>
#include <type_traits>
#include <utility>
#include <vector>

#include "../../include/rdt.h"
#include "common.cuh"
#include "internal.h"

namespace rdt {

namespace {

constexpr int kRun = 256;            // elements that share one scale of an 8-bit state
constexpr int kThreads = 256;
constexpr int kTile = 8 * kThreads;  // elements of a CTA's tile: one run per warp, 8 per lane
// Tensors per launch: the table stays inside the 32,764 bytes of parameters a
// kernel may have. Short lists take the short table, whose launch copies less.
constexpr int kMaxTensors = 400;
constexpr int kFewTensors = 32;

struct Tensor {
  float* w;
  const void* g;
  void* m;
  void* v;
  float* m_scale;
  float* v_scale;
  bf16* wb;
  int64_t n;
  float lr, wd;
};

template <int kMax>
struct Table {
  Tensor t[kMax];
  int32_t end[kMax];  // tiles up to and including tensor i
  int32_t first;      // index of t[0] in the caller's list
  int32_t count;
};
static_assert(sizeof(Table<kMaxTensors>) + 128 <= 32764, "the table must fit the parameters");

// The CTA's way through the tiles: chunks of `chunk` neighbours, a grid apart,
// so that the whole grid works in one window of each array (a contiguous share
// per CTA, a thousand windows, read DRAM at 0.8 of the speed), and so that
// only every chunk needs a search of the table.
struct Walk {
  int tile, end_of_chunk, o, begin, end;  // tensor o has the tiles [begin, end)
};
template <int kMax>
__device__ __forceinline__ void find_owner(const Table<kMax>& tab, Walk& w) {
  int lo = w.o, hi = tab.count - 1;  // the first tensor whose end is above the tile
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (tab.end[mid] > w.tile) hi = mid; else lo = mid + 1;
  }
  w.o = lo;
  w.begin = lo ? tab.end[lo - 1] : 0;
  w.end = tab.end[lo];
}
template <int kMax>
__device__ __forceinline__ Walk first_tile(const Table<kMax>& tab, int tiles, int chunk) {
  Walk w{static_cast<int>(blockIdx.x) * chunk, 0, 0, 0, 0};
  w.end_of_chunk = min(w.tile + chunk, tiles);
  if (w.tile < tiles) find_owner(tab, w);
  return w;
}
// The next tile; at or behind `tiles` there is none.
template <int kMax>
__device__ __forceinline__ void next_tile(const Table<kMax>& tab, int tiles, int chunk, Walk& w) {
  if (++w.tile == w.end_of_chunk) {
    w.tile += chunk * (static_cast<int>(gridDim.x) - 1);
    w.end_of_chunk = min(w.tile + chunk, tiles);
  }
  if (w.tile >= w.end && w.tile < tiles) find_owner(tab, w);
}

// Launches overlap (programmatic launch: one may start when all CTAs of the
// one before it have come here). Each waits for the end of what is before it
// in the stream ahead of its first access to memory, the later launches of one
// call as well as its first: nothing but that wait orders their reads after
// the writes of earlier kernels. What overlaps is a launch's own start and its
// first look at the table. For the same reason nothing is read through the
// read-only path (__ldg, const __restrict__), which is for memory nobody writes
// while the kernel is there.
__device__ __forceinline__ void after_previous_kernel() {
  asm volatile("griddepcontrol.wait;\n\tgriddepcontrol.launch_dependents;" ::: "memory");
}

// Two fp32 operations, each rounded to nearest, in one instruction.
__device__ __forceinline__ uint64_t bits2(float2 a) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a.x), "f"(a.y));
  return r;
}
__device__ __forceinline__ float2 floats2(uint64_t a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a));
  return r;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)));
  return floats2(r);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)), "l"(bits2(c)));
  return floats2(r);
}
__device__ __forceinline__ float2 both(float a) { return make_float2(a, a); }
// A pair's product and the sum it goes into would be contracted to one fma,
// the .rn of both notwithstanding; a sum that is an fma itself, with a 1 the
// compiler does not know, is not.
__device__ __forceinline__ float2 add2(float2 a, float2 b, float one) {
  return fma2(a, both(one), b);
}
__device__ __forceinline__ float2 sub2(float2 a, float2 b, float one) {
  return fma2(b, both(-one), a);
}

// A lane's eight elements of its warp's run are two groups of four, 128
// elements apart, so that every access of the warp is one contiguous piece.
// `have` counts the run's elements from the lane's first on; the masked forms
// serve the run that ends a tensor.
__device__ __forceinline__ int group_have(int have, int h) {
  return have - 128 * h > 4 ? 4 : have - 128 * h;
}

template <bool kFull>
__device__ __forceinline__ void load8(const float* p, int have, float* x) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (kFull) {
      const float4 a = *reinterpret_cast<const float4*>(p + 128 * h);
      x[4 * h] = a.x; x[4 * h + 1] = a.y; x[4 * h + 2] = a.z; x[4 * h + 3] = a.w;
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) x[4 * h + k] = k < group_have(have, h) ? p[128 * h + k] : 0.f;
    }
  }
}
template <bool kFull>
__device__ __forceinline__ void load8(const bf16* p, int have, float* x) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (kFull) {
      const uint2 a = *reinterpret_cast<const uint2*>(p + 128 * h);
      x[4 * h] = bf16lo(a.x); x[4 * h + 1] = bf16hi(a.x);
      x[4 * h + 2] = bf16lo(a.y); x[4 * h + 3] = bf16hi(a.y);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        x[4 * h + k] = k < group_have(have, h) ? bf16_to_f(p[128 * h + k]) : 0.f;
    }
  }
}
template <bool kFull>
__device__ __forceinline__ void store8(float* p, int have, const float* x) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (kFull) {
      *reinterpret_cast<float4*>(p + 128 * h) =
          make_float4(x[4 * h], x[4 * h + 1], x[4 * h + 2], x[4 * h + 3]);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (k < group_have(have, h)) p[128 * h + k] = x[4 * h + k];
    }
  }
}
template <bool kFull>
__device__ __forceinline__ void store8(bf16* p, int have, const float* x) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (kFull) {
      *reinterpret_cast<uint2*>(p + 128 * h) =
          make_uint2(pack_bf16x2(x[4 * h], x[4 * h + 1]), pack_bf16x2(x[4 * h + 2], x[4 * h + 3]));
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (k < group_have(have, h)) p[128 * h + k] = __float2bfloat16_rn(x[4 * h + k]);
    }
  }
}
// Eight one-byte codes, four to a word.
template <bool kFull>
__device__ __forceinline__ void load8(const uint8_t* p, int have, uint32_t* c) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (kFull) {
      c[h] = *reinterpret_cast<const uint32_t*>(p + 128 * h);
    } else {
      c[h] = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (k < group_have(have, h)) c[h] |= static_cast<uint32_t>(p[128 * h + k]) << (8 * k);
    }
  }
}
template <bool kFull>
__device__ __forceinline__ void store8(uint8_t* p, int have, const uint32_t* c) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (kFull) {
      *reinterpret_cast<uint32_t*>(p + 128 * h) = c[h];
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (k < group_have(have, h)) p[128 * h + k] = static_cast<uint8_t>(c[h] >> (8 * k));
    }
  }
}

// hi + lo += x x for two elements at once, with the rounding errors of the
// product and of the sum kept in lo. (fp64 has 1/64 of fp32's rate here: the
// same sum in fp64 took 1.82 ms for 490 M fp32 values.) kExact: x x has no
// rounding error (bf16).
//
// lo is a plain fp32 sum that grows with the number n of additions: with u =
// 2^-24 its own roundings come to (n^2 / 2) u^2 of the sum, and equal values
// give them all one sign. So after every 8 additions lo is taken into hi
// (tidy; 52 u^2 for the eight), and after every 24 the pairs go into an fp64
// sum. Adding up every rounding that can occur, with the joins of a thread's
// pairs (25 u^2) and of a warp's lanes (41 u^2, or 80 u^2 where there was no
// fp64 sum to start from), the result is within 270 u^2 = 9.6e-13 of the sum
// for any number of values.
template <bool kExact>
__device__ __forceinline__ void add_squares(float2 x, float2& hi, float2& lo, float one) {
  const float2 p = mul2(x, x);
  const float2 t = add2(hi, p, one);
  const float2 b = sub2(t, hi, one);
  float2 c = add2(sub2(hi, sub2(t, b, one), one), sub2(p, b, one), one);
  if (!kExact) c = add2(c, fma2(x, x, make_float2(-p.x, -p.y)), one);
  hi = t;
  lo = add2(lo, c, one);
}

// hi + lo += h + l, the rounding error of hi + h kept in lo.
__device__ __forceinline__ void add_pair(float& hi, float& lo, float h, float l) {
  const float t = __fadd_rn(hi, h), b = __fsub_rn(t, hi);
  lo += l + __fadd_rn(__fsub_rn(hi, __fsub_rn(t, b)), __fsub_rn(h, b));
  hi = t;
}

// The same for two pairs at once.
__device__ __forceinline__ void add_pair2(float2& hi, float2& lo, float2 h, float2 l, float one) {
  const float2 t = add2(hi, h, one), b = sub2(t, hi, one);
  const float2 e = add2(sub2(hi, sub2(t, b, one), one), sub2(h, b, one), one);
  lo = add2(lo, add2(l, e, one), one);
  hi = t;
}

// Sixteen bytes of gradients to fp32.
template <bool kBf16>
__device__ __forceinline__ void unpack16(const uint4& r, float* x) {
  if constexpr (!kBf16) {
    x[0] = __uint_as_float(r.x); x[1] = __uint_as_float(r.y);
    x[2] = __uint_as_float(r.z); x[3] = __uint_as_float(r.w);
  } else {
    x[0] = bf16lo(r.x); x[1] = bf16hi(r.x); x[2] = bf16lo(r.y); x[3] = bf16hi(r.y);
    x[4] = bf16lo(r.z); x[5] = bf16hi(r.z); x[6] = bf16lo(r.w); x[7] = bf16hi(r.w);
  }
}

// A CTA's step is one chunk of two tiles: two (bf16) or four (fp32) 16-byte
// loads of a thread, those of the next step under way with them. 268 M values,
// 4 CTAs an SM: fp32 152 us (1.04 of the copy bandwidth; 173 with 6 CTAs), bf16
// 100 us (0.79: the additions bound it; without the next step's loads 4 to 9 us
// more). Left to itself the compiler takes 48 registers for bf16 and spills.
template <bool kBf16> constexpr int kSqLoads = kBf16 ? 2 : 4;
template <bool kBf16>
constexpr int kSqTiles = kSqLoads<kBf16> * (kBf16 ? 8 : 4) * kThreads / kTile;
// A chunk makes two additions to each pair of a thread: chunks before a tidy, and tidies before
// the pairs go to fp64. 490 M bf16 values: 176 us; 189 with fp64 every 4 chunks, 165 with neither.
constexpr int kSqTidy = 4, kSqFold = 3;
template <bool kBf16, int kMax>
__global__ void __launch_bounds__(kThreads, 4) tensors_sq_sum_kernel(
    const __grid_constant__ Table<kMax> tab, int tiles, float one, double* partials) {
  __shared__ double red[kThreads / 32];
  using G = typename std::conditional<kBf16, bf16, float>::type;
  constexpr int kPer = 16 / sizeof(G), kStep = kPer * kThreads;  // elements of a load
  constexpr int kLoads = kSqLoads<kBf16>, kSqChunk = kSqTiles<kBf16>;
  static_assert(kLoads * kPer / 2 == 2 * 4 && kLoads * kStep == kSqChunk * kTile,
                "two additions to each pair a chunk");
  float2 hi[4] = {}, lo[4] = {};
  double total = 0.0;
  bool folded = false;
  // the u-th of a thread's loads of a chunk
  auto add = [&](const float* x, int u) {
#pragma unroll
    for (int k = 0; k < kPer / 2; ++k) {
      const int i = (u * (kPer / 2) + k) & 3;
      add_squares<kBf16>(make_float2(x[2 * k], x[2 * k + 1]), hi[i], lo[i], one);
    }
  };
  auto tidy = [&]() {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 t = add2(hi[k], lo[k], one);
      lo[k] = sub2(lo[k], sub2(t, hi[k], one), one);
      hi[k] = t;
    }
  };
  // The thread's pairs joined to one.
  auto join = [&]() {
    float2 h2 = hi[0], l2 = lo[0];
#pragma unroll
    for (int k = 1; k < 4; ++k) add_pair2(h2, l2, hi[k], lo[k], one);
    float h = h2.x, l = l2.x;
    add_pair(h, l, h2.y, l2.y);
    return make_float2(h, l);
  };
  auto fold = [&]() {
    const float2 a = join();
    total += static_cast<double>(a.x) + a.y;
#pragma unroll
    for (int k = 0; k < 4; ++k) hi[k] = lo[k] = make_float2(0.f, 0.f);
    folded = true;
  };
  // The tiles of the walk's tensor and chunk from its tile on, and whether they are a whole
  // chunk of whole tiles.
  auto count_of = [&](const Walk& w) { return min(w.end, w.end_of_chunk) - w.tile; };
  auto whole = [&](const Walk& w) {
    return w.tile < tiles && count_of(w) == kSqChunk &&
           static_cast<int64_t>(w.tile - w.begin + kSqChunk) * kTile <= tab.t[w.o].n;
  };
  auto first_of = [&](const Walk& w) {
    return static_cast<const G*>(tab.t[w.o].g) + static_cast<int64_t>(w.tile - w.begin) * kTile;
  };
  auto load = [&](const Walk& w, uint4* r) {
    const uint4* g = reinterpret_cast<const uint4*>(first_of(w)) + threadIdx.x;
#pragma unroll
    for (int u = 0; u < kLoads; ++u) r[u] = __ldcg(g + u * kThreads);  // (plain: 352 us for 275)
  };
  Walk w = first_tile(tab, tiles, kSqChunk);
  uint4 r[kLoads];
  bool full = whole(w);
  after_previous_kernel();
  if (full) load(w, r);
  while (w.tile < tiles) {
    for (int f = 0; f < kSqFold && w.tile < tiles; ++f) {
      for (int c = 0; c < kSqTidy && w.tile < tiles; ++c) {
        // the next chunk is looked up and its loads started before this one is added
        Walk n = w;
        n.tile += count_of(w) - 1;
        next_tile(tab, tiles, kSqChunk, n);
        uint4 next_r[kLoads];
        const bool next_full = whole(n);
        if (next_full) load(n, next_r);
        if (full) {
#pragma unroll
          for (int u = 0; u < kLoads; ++u) {
            float x[kPer];
            unpack16<kBf16>(r[u], x);
            add(x, u);
          }
        } else {
          const G* g = first_of(w);
          const int left =
              static_cast<int>(min(tab.t[w.o].n - static_cast<int64_t>(w.tile - w.begin) * kTile,
                                   static_cast<int64_t>(count_of(w)) * kTile));
#pragma unroll 1
          for (int u = 0, e = threadIdx.x * kPer; e < left; e += kStep, ++u) {
            float x[kPer];
            if (e + kPer <= left) {
              unpack16<kBf16>(__ldcg(reinterpret_cast<const uint4*>(g + e)), x);
            } else {
#pragma unroll
              for (int k = 0; k < kPer; ++k) x[k] = e + k < left ? static_cast<float>(g[e + k]) : 0.f;
            }
            if (kBf16 || u & 1) add(x, 1); else add(x, 0);
          }
        }
        w = n;
        full = next_full;
#pragma unroll
        for (int u = 0; u < kLoads; ++u) r[u] = next_r[u];
      }
      tidy();
    }
    if (w.tile < tiles) fold();  // short lists do without fp64 (1.2 us)
  }
  const float2 rest = join();
  float h = rest.x, l = rest.y;
  if (folded) {
    total += static_cast<double>(h) + l;
    h = static_cast<float>(total);
    l = static_cast<float>(total - h);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    add_pair(h, l, __shfl_xor_sync(0xffffffffu, h, o), __shfl_xor_sync(0xffffffffu, l, o));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = static_cast<double>(h) + l;
  __syncthreads();
  if (threadIdx.x == 0) {
    double s = 0.0;
    for (int w = 0; w < kThreads / 32; ++w) s += red[w];
    partials[blockIdx.x] = s;
  }
}

__global__ void __launch_bounds__(kThreads) tensors_sq_final_kernel(
    const double* partials, int n, double* out) {
  after_previous_kernel();
  __shared__ double red[kThreads / 32];
  double s = 0.0;
  for (int i = threadIdx.x; i < n; i += kThreads) s += partials[i];
  s = warp_sum_d(s);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    double t = 0.0;
    for (int w = 0; w < kThreads / 32; ++w) t += red[w];
    *out = t;
  }
}

struct AdamArgs {
  float b1, b2, omb1, omb2, inv_bc1, inv_root_bc2, eps, one;
  double log_b1, log_b2;  // for a step on the device
  const float* scale;
  const int32_t* skip;
  const int32_t* step_dev;
  int32_t step;
  uint32_t seed;
};

constexpr float kE4m3Max = 448.f;
constexpr float kE4m3Tiny = 0x1p-9f;
constexpr float kAbsmaxTiny = 0x1p-100f;

// Four e4m3 codes of a word to fp32 and back (round to nearest even, saturating).
__device__ __forceinline__ void e4m3_decode4(uint32_t c, float* x) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(c >> (16 * h)),
                                                     __NV_E4M3);
    const float2 f = __half22float2(__half2(r));
    x[2 * h] = f.x;
    x[2 * h + 1] = f.y;
  }
}
__device__ __forceinline__ uint32_t e4m3_encode4(const float* x) {
  const uint32_t a = __nv_cvt_float2_to_fp8x2(make_float2(x[0], x[1]), __NV_SATFINITE, __NV_E4M3);
  const uint32_t b = __nv_cvt_float2_to_fp8x2(make_float2(x[2], x[3]), __NV_SATFINITE, __NV_E4M3);
  return a | (b << 16);
}

// A 32-bit number from another, each bit of the result depending on every bit
// of x: two rounds of an odd multiplier (the fraction bits of the square roots
// of 5 and 3, the last bit set) and a fold of high bits onto low ones. With
// these shifts numbers of consecutive x, and of x 2^k apart, show no
// correlation (below 3 / sqrt(n) for lags to 2048; sqrt 2 with a fold by 15
// left 1 % at lag 256).
__device__ __forceinline__ uint32_t mix(uint32_t x) {
  x ^= x >> 16;
  x *= 0x3C6EF373u;
  x ^= x >> 14;
  x *= 0xBB67AE85u;
  return x ^ (x >> 16);
}

// |x| <= 448 up or down to a neighbouring e4m3 value with the probability of
// the distance: 20 of fp32's 23 mantissa bits go, so a number of 20 bits (16
// random ones, then 1000) is added and the 20 are cut. Below 2^-6 e4m3 has the
// steps of [2^-6, 2^-5), hence the shift by 2^-6. Not for NaN; what is rounded
// beyond 448 saturates when it is encoded.
template <bool kSigned>
__device__ __forceinline__ float round_random(float x, uint32_t bits20) {
  const float a = kSigned ? fabsf(x) : x;
  const float low = a < 0x1p-6f ? 0x1p-6f : 0.f;
  const uint32_t b = __float_as_uint(__fadd_rn(a, low)) + bits20;
  const float r = __fsub_rn(__uint_as_float(b & 0xfff00000u), low);
  return kSigned ? __uint_as_float(__float_as_uint(r) | (__float_as_uint(x) & 0x80000000u)) : r;
}
// 1 / x to 1 ulp.
__device__ __forceinline__ float reciprocal(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// The run's scale from its largest magnitude, and the factor to code units.
__device__ __forceinline__ void run_scale(float big, float& scale, float& unit) {
  const bool there = big >= kAbsmaxTiny;
  scale = there ? __fdiv_rn(big, kE4m3Max) : 0.f;
  unit = there ? __fmul_rn(__frcp_rn(big), kE4m3Max) : 0.f;
}

// A thread's share of a run with 8-bit states in shared memory, 16 bytes or
// less a piece; each thread copies and reads only its own. (32-bit states are
// loaded directly: their arithmetic is short enough beside their bytes, and
// 479 us a q4b block through shared memory stood against 466.)
template <bool kBf16>
struct Stage {
  static constexpr int kG = kBf16 ? 8 : 16, kS = 4;  // bytes of four elements
  static constexpr int kW = 0, kGAt = 2 * 16 * kThreads, kM = kGAt + 2 * kG * kThreads,
                       kV = kM + 2 * kS * kThreads, kBytes = kV + 2 * kS * kThreads;
};
template <int kBytes>
__device__ __forceinline__ void copy_async(uint32_t to, const void* from) {
  if constexpr (kBytes == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to), "l"(from), "n"(kBytes)
                 : "memory");
}
// Starts the copies of the whole run at `first`.
template <bool kBf16>
__device__ __forceinline__ void fetch_run(const Tensor& t, int64_t first, uint32_t stage,
                                          float& ms, float& vs) {
  using S = Stage<kBf16>;
  const int tid = threadIdx.x;
  const int64_t i = first + (tid & 31) * 4;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int at = h * kThreads + tid;
    const int64_t e = i + 128 * h;
    copy_async<16>(stage + S::kW + at * 16, t.w + e);
    copy_async<S::kG>(stage + S::kGAt + at * S::kG, static_cast<const uint8_t*>(t.g) + e * (S::kG / 4));
    copy_async<S::kS>(stage + S::kM + at * S::kS, static_cast<uint8_t*>(t.m) + e * (S::kS / 4));
    copy_async<S::kS>(stage + S::kV + at * S::kS, static_cast<uint8_t*>(t.v) + e * (S::kS / 4));
  }
  ms = t.m_scale[first / kRun];
  vs = t.v_scale[first / kRun];
}

// One run of 256 elements of tensor t, `first` its first element's index; the
// lane's own elements start at first + 4 lane. A full run of 8 bits is in `stage`.
template <int kBits, bool kBf16, bool kRandom, bool kFull>
__device__ __forceinline__ void adamw_run(const Tensor& t, int64_t first, const uint8_t* stage,
                                          float ms, float vs, const AdamArgs& p, float sc,
                                          float inv_bc1, float inv_root_bc2, uint32_t key) {
  using G = typename std::conditional<kBf16, bf16, float>::type;
  using S = Stage<kBf16>;
  const int tid = threadIdx.x, lane = tid & 31;
  const int64_t i = first + lane * 4;
  const int have = kFull ? kRun : static_cast<int>(t.n - i);
  const int64_t run = first / kRun;
  float w[8], g[8], m[8], r[8];
  uint32_t mc[2], vc[2];
  if constexpr (kFull && kBits == 8) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int at = h * kThreads + tid;
      auto four = [&](int where, float* x) {
        const float4 a = *reinterpret_cast<const float4*>(stage + where + at * 16);
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
      };
      four(S::kW, w + 4 * h);
      if constexpr (kBf16) {
        const uint2 a = *reinterpret_cast<const uint2*>(stage + S::kGAt + at * 8);
        g[4 * h] = bf16lo(a.x); g[4 * h + 1] = bf16hi(a.x);
        g[4 * h + 2] = bf16lo(a.y); g[4 * h + 3] = bf16hi(a.y);
      } else {
        four(S::kGAt, g + 4 * h);
      }
      mc[h] = *reinterpret_cast<const uint32_t*>(stage + S::kM + at * 4);
      vc[h] = *reinterpret_cast<const uint32_t*>(stage + S::kV + at * 4);
    }
  } else {
    load8<kFull>(t.w + i, have, w);
    load8<kFull>(static_cast<const G*>(t.g) + i, have, g);
    if constexpr (kBits == 32) {
      load8<kFull>(static_cast<const float*>(t.m) + i, have, m);
      load8<kFull>(static_cast<const float*>(t.v) + i, have, r);
    } else {
      load8<false>(static_cast<const uint8_t*>(t.m) + i, have, mc);
      load8<false>(static_cast<const uint8_t*>(t.v) + i, have, vc);
      ms = t.m_scale[run];
      vs = t.v_scale[run];
    }
  }
  if constexpr (kBits == 8) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      e4m3_decode4(mc[h], m + 4 * h);
      e4m3_decode4(vc[h], r + 4 * h);
    }
#pragma unroll
    for (int k = 0; k < 8; k += 2) {
      const float2 a = mul2(make_float2(m[k], m[k + 1]), both(ms));
      const float2 b = mul2(make_float2(r[k], r[k + 1]), both(vs));
      const float2 q = mul2(b, b);
      m[k] = a.x; m[k + 1] = a.y;
      r[k] = q.x; r[k + 1] = q.y;
    }
  }
  const float rate = __fmul_rn(t.lr, inv_bc1), keep = __fsub_rn(1.f, __fmul_rn(t.lr, t.wd));
  float big_m = 0.f, big_r = 0.f;
#pragma unroll
  for (int k = 0; k < 8; k += 2) {
    const float2 gs = mul2(make_float2(g[k], g[k + 1]), both(sc));
    const float2 mm = add2(mul2(make_float2(m[k], m[k + 1]), both(p.b1)),
                           mul2(gs, both(p.omb1)), p.one);
    const float2 v = add2(mul2(make_float2(r[k], r[k + 1]), both(p.b2)),
                          mul2(mul2(gs, both(p.omb2)), gs), p.one);
    const float2 root = make_float2(__fsqrt_rn(v.x), __fsqrt_rn(v.y));
    const float2 den = add2(mul2(root, both(inv_root_bc2)), both(p.eps), p.one);
    const float2 u = mul2(mm, make_float2(reciprocal(den.x), reciprocal(den.y)));
    const float2 x = sub2(mul2(make_float2(w[k], w[k + 1]), both(keep)), mul2(u, both(rate)),
                          p.one);
    w[k] = x.x; w[k + 1] = x.y;
    m[k] = mm.x; m[k + 1] = mm.y;
    r[k] = kBits == 32 ? v.x : root.x;
    r[k + 1] = kBits == 32 ? v.y : root.y;
    big_m = fmaxf(big_m, fmaxf(fabsf(mm.x), fabsf(mm.y)));
    big_r = fmaxf(big_r, fmaxf(root.x, root.y));
  }
  store8<kFull>(t.w + i, have, w);
  if (t.wb) store8<kFull>(t.wb + i, have, w);
  if constexpr (kBits == 32) {
    store8<kFull>(static_cast<float*>(t.m) + i, have, m);
    store8<kFull>(static_cast<float*>(t.v) + i, have, r);
  } else {
    float um, uv;
    run_scale(warp_max(big_m), ms, um);
    run_scale(warp_max(big_r), vs, uv);
    if (lane == 0) {
      t.m_scale[run] = ms;
      t.v_scale[run] = vs;
    }
    // no sqrt(v) > 0 becomes 0, but in a run that is stored as zeros
    const float least = uv > 0.f ? kE4m3Tiny : 0.f;
    float q[8], lowest = kE4m3Max;
    auto codes = [&](auto careful) {
#pragma unroll
      for (int k = 0; k < 8; k += 2) {
        float2 qm = mul2(make_float2(m[k], m[k + 1]), both(um));
        float2 qr = mul2(make_float2(r[k], r[k + 1]), both(uv));
        if constexpr (kRandom) {
          const uint32_t at = static_cast<uint32_t>(i + (k & 3) + 32 * (k & 4));
          const uint32_t x = mix(at ^ key), y = mix((at + 1) ^ key);
          auto up = [&](float& q, float& p, uint32_t z) {
            if (!careful.value || q == q) q = round_random<true>(q, (z << 4 & 0xffff0u) | 8u);
            if (!careful.value || p == p) p = round_random<false>(p, (z >> 12 & 0xffff0u) | 8u);
          };
          up(qm.x, qr.x, x);
          up(qm.y, qr.y, y);
        }
        m[k] = qm.x; m[k + 1] = qm.y;
        q[k] = qr.x; q[k + 1] = qr.y;
        lowest = fminf(lowest, fminf(qr.x, qr.y));
      }
    };
    if constexpr (kRandom) {
      // NaN must not go through round_random; a sum shows it (so does one that leaves fp32's
      // range, which only costs the careful way)
      float2 sum = make_float2(0.f, 0.f);
#pragma unroll
      for (int k = 0; k < 8; k += 2)
        sum = fma2(make_float2(m[k], m[k + 1]), make_float2(r[k], r[k + 1]), sum);
      if (fabsf(sum.x + sum.y) < INFINITY)
        codes(std::false_type{});
      else
        codes(std::true_type{});
    } else {
      codes(std::false_type{});
    }
    if (lowest < least) {  // looked at element by element where one of the eight is so low
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (r[k] > 0.f) q[k] = fmaxf(q[k], least);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      mc[h] = e4m3_encode4(m + 4 * h);
      vc[h] = e4m3_encode4(q + 4 * h);
    }
    store8<kFull>(static_cast<uint8_t*>(t.m) + i, have, mc);
    store8<kFull>(static_cast<uint8_t*>(t.v) + i, have, vc);
  }
}

// The bias corrections of a step on the device: two threads form them, in double and rounded
// once, from the logarithms that the host took, while the CTA's first copies are under way. (Two
// powers in every thread: 490 M parameters in 8 bits took 3.69 ms, 1.28 this way; 1.25 with a
// step from the host, whose kernel is another one so that it has none of this.)
__device__ __forceinline__ void corrections_of(int step, const AdamArgs& p, float& inv_bc1,
                                               float& inv_root_bc2) {
  __shared__ float both[2];
  if (threadIdx.x < 2) {
    const double left = 1.0 - exp(step * (threadIdx.x ? p.log_b2 : p.log_b1));
    both[threadIdx.x] = static_cast<float>(1.0 / (threadIdx.x ? sqrt(left) : left));
  }
  __syncthreads();
  inv_bc1 = both[0];
  inv_root_bc2 = both[1];
}

constexpr int kChunk = 2;  // tiles of a CTA's step of tensors_adamw_kernel
template <int kBits, bool kBf16, bool kRandom, bool kStepDev, int kMax>
__global__ void __launch_bounds__(kThreads) tensors_adamw_kernel(
    const __grid_constant__ Table<kMax> tab, int tiles, const AdamArgs p) {
  Walk w = first_tile(tab, tiles, kChunk);
  after_previous_kernel();
  if (p.skip && *p.skip) return;
  const float sc = p.scale ? *p.scale : 1.f;
  float inv_bc1 = p.inv_bc1, inv_root_bc2 = p.inv_root_bc2;
  const int step = kStepDev ? *p.step_dev : p.step;
  const uint32_t key0 = mix(mix(static_cast<uint32_t>(step)) + p.seed) + tab.first;
  const int part = (threadIdx.x >> 5) * kRun;
  auto place = [&](const Walk& w) { return static_cast<int64_t>(w.tile - w.begin) * kTile + part; };
  auto key_of = [&](const Walk& w) {
    return mix(key0 + w.o) ^ static_cast<uint32_t>(place(w) >> 32) * 0x9E3779B1u;
  };
  if constexpr (kBits == 32) {
    if constexpr (kStepDev) corrections_of(step, p, inv_bc1, inv_root_bc2);
    while (w.tile < tiles) {
      const Tensor& t = tab.t[w.o];
      const int64_t first = place(w);
      next_tile(tab, tiles, kChunk, w);
      if (first + kRun <= t.n)
        adamw_run<32, kBf16, false, true>(t, first, nullptr, 0.f, 0.f, p, sc, inv_bc1, inv_root_bc2, 0);
      else if (first < t.n)
        adamw_run<32, kBf16, false, false>(t, first, nullptr, 0.f, 0.f, p, sc, inv_bc1, inv_root_bc2, 0);
    }
  } else {
    // the next run's copies are under way while one is computed
    extern __shared__ __align__(16) uint8_t stages[];
    constexpr int kBytes = Stage<kBf16>::kBytes;
    const uint32_t at = smem_u32(stages);
    float ms = 0.f, vs = 0.f;
    if (w.tile < tiles && place(w) + kRun <= tab.t[w.o].n)
      fetch_run<kBf16>(tab.t[w.o], place(w), at, ms, vs);
    asm volatile("cp.async.commit_group;" ::: "memory");
    if constexpr (kStepDev) corrections_of(step, p, inv_bc1, inv_root_bc2);
    for (int s = 0; w.tile < tiles; s ^= 1) {
      Walk n = w;
      next_tile(tab, tiles, kChunk, n);
      float next_ms = 0.f, next_vs = 0.f;
      if (n.tile < tiles && place(n) + kRun <= tab.t[n.o].n)
        fetch_run<kBf16>(tab.t[n.o], place(n), at + (s ^ 1) * kBytes, next_ms, next_vs);
      asm volatile("cp.async.commit_group;" ::: "memory");
      asm volatile("cp.async.wait_group 1;" ::: "memory");
      const Tensor& t = tab.t[w.o];
      const int64_t first = place(w);
      if (first + kRun <= t.n)
        adamw_run<8, kBf16, kRandom, true>(t, first, stages + s * kBytes, ms, vs, p, sc, inv_bc1,
                                           inv_root_bc2, key_of(w));
      else if (first < t.n)
        adamw_run<8, kBf16, kRandom, false>(t, first, nullptr, 0.f, 0.f, p, sc, inv_bc1,
                                            inv_root_bc2, key_of(w));
      w = n;
      ms = next_ms;
      vs = next_vs;
    }
  }
}

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

constexpr int kMaxCount = 1000000;
// Tiles of a launch: a CTA's next tile, up to a grid's chunks further on, stays inside 32 bits.
// More than memory holds, but a list for the squared sum may name a tensor again and again.
constexpr int64_t kMaxTiles = int64_t(1) << 30;

int64_t tiles_of(int64_t n) { return (n + kTile - 1) / kTile; }

const char* list_problem(const rdt_opt_tensor* t, int count, int g_dtype) {
  if (count < 0 || count > kMaxCount) return "count must be in [0, 1000000]";
  if (count > 0 && !t) return "null pointer: tensors";
  if (g_dtype != RDT_F32 && g_dtype != RDT_BF16) return "g_dtype must be RDT_F32 or RDT_BF16";
  for (int i = 0; i < count; ++i) {
    if (t[i].n < 0 || t[i].n > (int64_t(1) << 40)) return "n of a tensor must be in [0, 2^40]";
    if (t[i].n > 0 && !t[i].g) return "null pointer: g of a tensor";
    if (reinterpret_cast<uintptr_t>(t[i].g) & 15) return "g of a tensor must be 16-byte aligned";
  }
  return nullptr;
}

// Calls f(table, tiles) for each launch's share of the list.
template <int kMax, typename F>
cudaError_t each_launch(const rdt_opt_tensor* list, int count, F f) {
  Table<kMax> tab;
  int64_t tiles = 0;
  tab.count = 0;
  tab.first = 0;
  for (int i = 0; i <= count; ++i) {
    const int64_t more = i < count ? tiles_of(list[i].n) : 0;
    if (tab.count && (i == count || tab.count == kMax || tiles + more > kMaxTiles)) {
      if (tiles > 0) {
        const cudaError_t e = f(tab, static_cast<int>(tiles));
        if (e != cudaSuccess) return e;
      }
      tab.count = 0;
      tiles = 0;
    }
    if (i == count) break;
    // entries with n == 0 keep their place: the random bits go by the index in the list
    if (tab.count == 0) tab.first = i;
    tiles += more;
    const rdt_opt_tensor& t = list[i];
    tab.t[tab.count] = Tensor{t.w, t.g, t.m, t.v, t.m_scale, t.v_scale,
                              reinterpret_cast<bf16*>(t.w_bf16), t.n, t.lr, t.weight_decay};
    tab.end[tab.count++] = static_cast<int32_t>(tiles);
  }
  return cudaSuccess;
}

// CTAs for `tiles`: a resident wave at most, or, with `share`, one per `share`
// tiles if that is more. CTAs that come and go in order keep the grid's
// window of the arrays narrow: 268 M parameters with 8-bit states took 823 us
// in one wave, 702 with 12 tiles a CTA, 693 with 6 and 685 with 2 (776 for
// random rounding, against 730 with 6, by each CTA's start). The squared sum,
// one array, loses: 166 us in a wave, 168 with 16 tiles a CTA.
int ctas(int tiles, int chunk, int per_sm, int share = INT32_MAX) {
  const int all = (tiles + chunk - 1) / chunk;
  return std::min(all, std::max(per_sm * num_sms(), tiles / share));
}

constexpr int kMaxPartials = 2048;  // of one launch

template <typename K, typename... A>
cudaError_t launch(K kernel, int grid, size_t smem, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  note_launch();
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int kMax>
cudaError_t sq_sum_launches(const rdt_opt_tensor* list, int count, bool half, double* parts,
                            int64_t room, int64_t* used, cudaStream_t s) {
  return each_launch<kMax>(list, count, [&](const Table<kMax>& tab, int tiles) {
    const int blocks = std::min(ctas(tiles, half ? kSqTiles<true> : kSqTiles<false>, 4), kMaxPartials);
    if (*used + blocks > room) return cudaErrorInvalidValue;
    auto kernel = half ? tensors_sq_sum_kernel<true, kMax> : tensors_sq_sum_kernel<false, kMax>;
    double* to = parts + *used;
    *used += blocks;
    return launch(kernel, blocks, 0, s, tab, tiles, 1.f, to);
  });
}

template <int kBits, bool kBf16, bool kRandom, bool kStepDev, int kMax>
cudaError_t launch_adamw(const Table<kMax>& tab, int tiles, const AdamArgs& a, cudaStream_t s) {
  constexpr int kBytes = kBits == 8 ? 2 * Stage<kBf16>::kBytes : 0;
  auto kernel = tensors_adamw_kernel<kBits, kBf16, kRandom, kStepDev, kMax>;
  static std::atomic<uint64_t> allowed{0};  // devices where the kernel may use kBytes
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev > 63 || !(allowed.load() >> dev & 1)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
    if (e != cudaSuccess) return e;
    if (dev < 64) allowed.fetch_or(uint64_t(1) << dev);
  }
  return launch(kernel, ctas(tiles, kChunk, kBits == 32 ? 8 : 4, 6), kBytes, s, tab,
                tiles, a);
}

template <bool kStepDev, int kMax>
cudaError_t adamw_launches(const rdt_opt_tensor* list, int count, bool half, int bits, bool random,
                           const AdamArgs& a, cudaStream_t s) {
  return each_launch<kMax>(list, count, [&](const Table<kMax>& tab, int tiles) {
    if (bits == 32)
      return half ? launch_adamw<32, true, false, kStepDev>(tab, tiles, a, s)
                  : launch_adamw<32, false, false, kStepDev>(tab, tiles, a, s);
    if (random)
      return half ? launch_adamw<8, true, true, kStepDev>(tab, tiles, a, s)
                  : launch_adamw<8, false, true, kStepDev>(tab, tiles, a, s);
    return half ? launch_adamw<8, true, false, kStepDev>(tab, tiles, a, s)
                : launch_adamw<8, false, false, kStepDev>(tab, tiles, a, s);
  });
}

}  // namespace

}  // namespace rdt

using namespace rdt;

extern "C" {

size_t rdt_tensors_sq_sum_workspace_bytes(const rdt_opt_tensor* tensors, int32_t count) {
  if (list_problem(tensors, count, RDT_F32)) return 0;
  // one partial sum for each block of each launch (no device is asked how many there are); two
  // launches that end for their tiles have more than kMaxTiles together
  int64_t tiles = 0;
  for (int i = 0; i < count; ++i) tiles += tiles_of(tensors[i].n);
  const size_t launches = count / kMaxTensors + 1 + 2 * (tiles / kMaxTiles);
  return launches * kMaxPartials * sizeof(double);
}

rdt_status rdt_tensors_sq_sum(const rdt_opt_tensor* tensors, int32_t count, int32_t g_dtype,
                              double* sumsq, void* ws, size_t ws_bytes, void* stream) {
  if (const char* why = list_problem(tensors, count, g_dtype)) return refuse(why);
  if (!sumsq || !ws) return refuse("null pointer");
  if ((reinterpret_cast<uintptr_t>(sumsq) | reinterpret_cast<uintptr_t>(ws)) & 7)
    return refuse("sumsq and ws must be 8-byte aligned");
  if (ws_bytes < rdt_tensors_sq_sum_workspace_bytes(tensors, count))
    return refuse("workspace too small");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  double* parts = static_cast<double*>(ws);
  int64_t used = 0;
  const int64_t room = static_cast<int64_t>(ws_bytes / sizeof(double));
  const bool half = g_dtype == RDT_BF16;
  cudaError_t e =
      count <= kFewTensors
          ? sq_sum_launches<kFewTensors>(tensors, count, half, parts, room, &used, s)
          : sq_sum_launches<kMaxTensors>(tensors, count, half, parts, room, &used, s);
  if (e != cudaSuccess) return launched(e);
  return launched(launch(tensors_sq_final_kernel, 1, 0, s, parts, static_cast<int>(used), sumsq));
}

rdt_status rdt_tensors_adamw(const rdt_opt_tensor* tensors, int32_t count, int32_t g_dtype,
                             int32_t state_bits, int64_t seed, const float* scale,
                             const int32_t* skip_flag, int32_t step, const int32_t* step_dev,
                             float beta1, float beta2, float eps, void* stream) {
  if (const char* why = list_problem(tensors, count, g_dtype)) return refuse(why);
  if (state_bits != 32 && state_bits != 8) return refuse("state_bits must be 32 or 8");
  if (seed >= (int64_t(1) << 32)) return refuse("seed must be below 2^32");
  if (!step_dev && step < 1) return refuse("step must be >= 1 (bias correction)");
  if (!(beta1 >= 0.f && beta1 < 1.f) || !(beta2 >= 0.f && beta2 < 1.f) ||
      !(eps >= 1e-30f && eps <= 1e30f))
    return refuse("beta1 and beta2 must be in [0, 1) and eps in [1e-30, 1e30]");
  if ((reinterpret_cast<uintptr_t>(scale) | reinterpret_cast<uintptr_t>(skip_flag) |
       reinterpret_cast<uintptr_t>(step_dev)) & 3)
    return refuse("scale, skip_flag and step_dev must be 4-byte aligned");
  bool sorted = true;
  uintptr_t last = 0;
  for (int i = 0; i < count; ++i) {
    const rdt_opt_tensor& t = tensors[i];
    if (t.n == 0) continue;
    if (!t.w || !t.m || !t.v) return refuse("null pointer: w, m or v of a tensor");
    if ((reinterpret_cast<uintptr_t>(t.w) | reinterpret_cast<uintptr_t>(t.m) |
         reinterpret_cast<uintptr_t>(t.v) | reinterpret_cast<uintptr_t>(t.w_bf16)) & 15)
      return refuse("w, m, v and w_bf16 of a tensor must be 16-byte aligned");
    if (state_bits == 8) {
      if (!t.m_scale || !t.v_scale) return refuse("null pointer: m_scale or v_scale of a tensor");
      if ((reinterpret_cast<uintptr_t>(t.m_scale) | reinterpret_cast<uintptr_t>(t.v_scale)) & 3)
        return refuse("m_scale and v_scale of a tensor must be 4-byte aligned");
    }
    const uintptr_t at = reinterpret_cast<uintptr_t>(t.w);
    sorted = sorted && at >= last;
    last = at + static_cast<uintptr_t>(t.n) * 4;
  }
  if (!sorted) {
    // the same tensor twice would be updated twice at once
    try {
      std::vector<std::pair<uintptr_t, uintptr_t>> spans;
      for (int i = 0; i < count; ++i)
        if (tensors[i].n > 0) {
          const uintptr_t at = reinterpret_cast<uintptr_t>(tensors[i].w);
          spans.emplace_back(at, at + static_cast<uintptr_t>(tensors[i].n) * 4);
        }
      std::sort(spans.begin(), spans.end());
      for (size_t i = 1; i < spans.size(); ++i)
        if (spans[i].first < spans[i - 1].second) return refuse("two tensors' w overlap");
    } catch (const std::bad_alloc&) {
      return refuse("out of host memory");
    }
  }
  AdamArgs a;
  a.b1 = beta1;
  a.b2 = beta2;
  a.omb1 = static_cast<float>(1.0 - static_cast<double>(beta1));
  a.omb2 = static_cast<float>(1.0 - static_cast<double>(beta2));
  a.step = step_dev ? 1 : step;
  a.inv_bc1 = static_cast<float>(1.0 / (1.0 - std::pow(static_cast<double>(beta1), a.step)));
  a.inv_root_bc2 =
      static_cast<float>(1.0 / std::sqrt(1.0 - std::pow(static_cast<double>(beta2), a.step)));
  a.log_b1 = std::log(static_cast<double>(beta1));
  a.log_b2 = std::log(static_cast<double>(beta2));
  a.eps = eps;
  a.one = 1.f;
  a.scale = scale;
  a.skip = skip_flag;
  a.step_dev = step_dev;
  a.seed = seed < 0 ? 0u : static_cast<uint32_t>(seed);
  const bool random = seed >= 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool half = g_dtype == RDT_BF16;
  auto launches = step_dev ? (count <= kFewTensors ? adamw_launches<true, kFewTensors>
                                                   : adamw_launches<true, kMaxTensors>)
                           : (count <= kFewTensors ? adamw_launches<false, kFewTensors>
                                                   : adamw_launches<false, kMaxTensors>);
  return launched(launches(tensors, count, half, state_bits, random, a, s));
}

}  // extern "C"
