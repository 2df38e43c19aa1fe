// Squared sum and AdamW over many tensors at once (rdt_tensors_sq_sum,
// rdt_tensors_adamw): the tensors' addresses and sizes travel as kernel
// parameters, every tensor is cut into tiles, and the tiles of all tensors
// make one launch (one per kMaxTensors tensors).
#include <algorithm>
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
// Tensors per launch: the table stays inside the 32,764 bytes of parameters a kernel may have.
constexpr int kMaxTensors = 400;

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

struct Table {
  Tensor t[kMaxTensors];
  int32_t end[kMaxTensors];  // tiles up to and including tensor i
  int32_t first;             // index of t[0] in the caller's list
  int32_t count;
};
static_assert(sizeof(Table) + 128 <= 32764, "the table must fit the kernel parameters");

// The tensor that owns a tile: the first whose end is above it.
__device__ __forceinline__ int owner_of(const Table& tab, int tile) {
  int lo = 0, hi = tab.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (tab.end[mid] > tile) hi = mid; else lo = mid + 1;
  }
  return lo;
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

// hi + lo += x x, with the rounding errors of the product and of the sum kept
// in lo: a sum of n squares is right to about n 2^-48. (fp64 has 1/64 of
// fp32's rate here: the same sum in fp64 took 1.82 ms for 490 M fp32 values.)
__device__ __forceinline__ void add_square(float x, float& hi, float& lo) {
  const float p = __fmul_rn(x, x);
  const float e = __fmaf_rn(x, x, -p);
  const float t = __fadd_rn(hi, p);
  const float b = __fsub_rn(t, hi);
  const float c = __fadd_rn(__fsub_rn(hi, __fsub_rn(t, b)), __fsub_rn(p, b));
  hi = t;
  lo = __fadd_rn(lo, __fadd_rn(c, e));
}

template <bool kBf16>
__global__ void __launch_bounds__(kThreads) tensors_sq_sum_kernel(
    const __grid_constant__ Table tab, int tiles, double* __restrict__ partials) {
  __shared__ double red[kThreads / 32];
  using G = typename std::conditional<kBf16, bf16, float>::type;
  const int at = (threadIdx.x >> 5) * kRun + (threadIdx.x & 31) * 4;
  float hi[4] = {0.f, 0.f, 0.f, 0.f}, lo[4] = {0.f, 0.f, 0.f, 0.f};
  for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int o = owner_of(tab, tile);
    const Tensor& t = tab.t[o];
    const int64_t first = static_cast<int64_t>(tile - (o ? tab.end[o - 1] : 0)) * kTile;
    const G* g = static_cast<const G*>(t.g) + first + at;
    const int64_t left = t.n - first;
    float x[8];
    if (left >= kTile)
      load8<true>(g, 0, x);
    else
      load8<false>(g, static_cast<int>(left) - at, x);
#pragma unroll
    for (int k = 0; k < 8; ++k) add_square(x[k], hi[k & 3], lo[k & 3]);
  }
  double acc = 0.0;
#pragma unroll
  for (int k = 0; k < 4; ++k) acc += static_cast<double>(hi[k]) + static_cast<double>(lo[k]);
  acc = warp_sum_d(acc);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = acc;
  __syncthreads();
  if (threadIdx.x == 0) {
    double s = 0.0;
    for (int w = 0; w < kThreads / 32; ++w) s += red[w];
    partials[blockIdx.x] = s;
  }
}

__global__ void __launch_bounds__(kThreads) tensors_sq_final_kernel(
    const double* __restrict__ partials, int n, double* __restrict__ out) {
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
  float b1, b2, omb1, omb2, inv_bc1, inv_root_bc2, eps;
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
// the distance: 20 of fp32's 23 mantissa bits go, so a number of 20 bits, the
// upper 16 random, is added and the 20 are cut. Below 2^-6 e4m3 has the steps
// of [2^-6, 2^-5), hence the shift by 2^-6.
__device__ __forceinline__ float round_random(float x, uint32_t half) {
  const float a = fabsf(x);
  const float low = a < 0x1p-6f ? 0x1p-6f : 0.f;
  const uint32_t b = __float_as_uint(__fadd_rn(a, low)) + half * 16u + 8u;
  const float r = __fsub_rn(__uint_as_float(b & 0xfff00000u), low);
  return copysignf(fminf(r, kE4m3Max), x);
}

// The run's scale from its largest magnitude, and the factor to code units.
__device__ __forceinline__ void run_scale(float big, float& scale, float& unit) {
  const bool there = big >= kAbsmaxTiny;
  scale = there ? __fdiv_rn(big, kE4m3Max) : 0.f;
  unit = there ? __fmul_rn(__frcp_rn(big), kE4m3Max) : 0.f;
}

// One run of 256 elements of tensor t, `first` its first element's index; the
// lane's own elements start at first + 4 lane.
template <int kBits, bool kBf16, bool kRandom, bool kFull>
__device__ __forceinline__ void adamw_run(const Tensor& t, int64_t first, const AdamArgs& p,
                                          float sc, float inv_bc1, float inv_root_bc2,
                                          uint32_t key) {
  using G = typename std::conditional<kBf16, bf16, float>::type;
  const int lane = threadIdx.x & 31;
  const int64_t i = first + lane * 4;
  const int have = kFull ? kRun : static_cast<int>(t.n - i);
  const int64_t run = first / kRun;
  float w[8], g[8], m[8], r[8];
  load8<kFull>(t.w + i, have, w);
  load8<kFull>(static_cast<const G*>(t.g) + i, have, g);
  if constexpr (kBits == 32) {
    load8<kFull>(static_cast<const float*>(t.m) + i, have, m);
    load8<kFull>(static_cast<const float*>(t.v) + i, have, r);
  } else {
    uint32_t mc[2], vc[2];
    load8<kFull>(static_cast<const uint8_t*>(t.m) + i, have, mc);
    load8<kFull>(static_cast<const uint8_t*>(t.v) + i, have, vc);
    const float ms = t.m_scale[run], vs = t.v_scale[run];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      e4m3_decode4(mc[h], m + 4 * h);
      e4m3_decode4(vc[h], r + 4 * h);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      m[k] = __fmul_rn(m[k], ms);
      r[k] = __fmul_rn(r[k], vs);
      r[k] = __fmul_rn(r[k], r[k]);
    }
  }
  const float rate = __fmul_rn(t.lr, inv_bc1), keep = __fsub_rn(1.f, __fmul_rn(t.lr, t.wd));
  float big_m = 0.f, big_r = 0.f;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float gs = __fmul_rn(g[k], sc);
    m[k] = __fadd_rn(__fmul_rn(m[k], p.b1), __fmul_rn(gs, p.omb1));
    const float v = __fadd_rn(__fmul_rn(r[k], p.b2), __fmul_rn(__fmul_rn(gs, p.omb2), gs));
    const float root = __fsqrt_rn(v);
    const float u = __fdiv_rn(m[k], __fadd_rn(__fmul_rn(root, inv_root_bc2), p.eps));
    w[k] = __fsub_rn(__fmul_rn(w[k], keep), __fmul_rn(u, rate));
    r[k] = kBits == 32 ? v : root;
    big_m = fmaxf(big_m, fabsf(m[k]));
    big_r = fmaxf(big_r, root);
  }
  store8<kFull>(t.w + i, have, w);
  if (t.wb) store8<kFull>(t.wb + i, have, w);
  if constexpr (kBits == 32) {
    store8<kFull>(static_cast<float*>(t.m) + i, have, m);
    store8<kFull>(static_cast<float*>(t.v) + i, have, r);
  } else {
    float ms, vs, um, uv;
    run_scale(warp_max(big_m), ms, um);
    run_scale(warp_max(big_r), vs, uv);
    if (lane == 0) {
      t.m_scale[run] = ms;
      t.v_scale[run] = vs;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      float qm = __fmul_rn(m[k], um), qr = __fmul_rn(r[k], uv);
      if constexpr (kRandom) {
        const uint32_t x = mix(static_cast<uint32_t>(i + (k & 3) + 32 * (k & 4)) ^ key);
        qm = qm != qm ? qm : round_random(fminf(fmaxf(qm, -kE4m3Max), kE4m3Max), x & 0xffffu);
        qr = qr != qr ? qr : round_random(fminf(qr, kE4m3Max), x >> 16);
      }
      if (r[k] > 0.f && uv > 0.f && qr < kE4m3Tiny) qr = kE4m3Tiny;
      m[k] = qm;
      r[k] = qr;
    }
    uint32_t mc[2] = {e4m3_encode4(m), e4m3_encode4(m + 4)};
    uint32_t vc[2] = {e4m3_encode4(r), e4m3_encode4(r + 4)};
    store8<kFull>(static_cast<uint8_t*>(t.m) + i, have, mc);
    store8<kFull>(static_cast<uint8_t*>(t.v) + i, have, vc);
  }
}

template <int kBits, bool kBf16, bool kRandom>
__global__ void __launch_bounds__(kThreads) tensors_adamw_kernel(
    const __grid_constant__ Table tab, int tiles, const AdamArgs p) {
  if (p.skip && *p.skip) return;
  const float sc = p.scale ? *p.scale : 1.f;
  float inv_bc1 = p.inv_bc1, inv_root_bc2 = p.inv_root_bc2;
  int step = p.step;
  if (p.step_dev) {
    step = *p.step_dev;
    inv_bc1 = static_cast<float>(1.0 / (1.0 - pow(static_cast<double>(p.b1), static_cast<double>(step))));
    inv_root_bc2 = static_cast<float>(
        1.0 / sqrt(1.0 - pow(static_cast<double>(p.b2), static_cast<double>(step))));
  }
  const uint32_t key0 = mix(mix(static_cast<uint32_t>(step)) + p.seed) + tab.first;
  for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int o = owner_of(tab, tile);
    const Tensor& t = tab.t[o];
    const int64_t first = static_cast<int64_t>(tile - (o ? tab.end[o - 1] : 0)) * kTile +
                          (threadIdx.x >> 5) * kRun;
    const uint32_t key = mix(key0 + o) ^ static_cast<uint32_t>(first >> 32) * 0x9E3779B1u;
    if (first + kRun <= t.n)
      adamw_run<kBits, kBf16, kRandom, true>(t, first, p, sc, inv_bc1, inv_root_bc2, key);
    else if (first < t.n)
      adamw_run<kBits, kBf16, kRandom, false>(t, first, p, sc, inv_bc1, inv_root_bc2, key);
  }
}

rdt_status refuse(const char* msg) {
  set_last_error(msg);
  return RDT_EINVAL;
}
rdt_status launched(cudaError_t e) {
  if (e == cudaSuccess) return RDT_OK;
  set_last_error(cudaGetErrorString(e));
  return RDT_ECUDA;
}

constexpr int kMaxCount = 1000000;

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
template <typename F>
cudaError_t each_launch(const rdt_opt_tensor* list, int count, F f) {
  Table tab;
  int64_t tiles = 0;
  tab.count = 0;
  tab.first = 0;
  for (int i = 0; i <= count; ++i) {
    const int64_t more = i < count ? tiles_of(list[i].n) : 0;
    if (tab.count && (i == count || tab.count == kMaxTensors || tiles + more > INT32_MAX)) {
      const cudaError_t e = f(tab, static_cast<int>(tiles));
      if (e != cudaSuccess) return e;
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

int sq_blocks(int64_t tiles) {
  return static_cast<int>(std::min<int64_t>(std::max<int64_t>(tiles, 1), 4LL * num_sms()));
}

}  // namespace

}  // namespace rdt

using namespace rdt;

extern "C" {

size_t rdt_tensors_sq_sum_workspace_bytes(const rdt_opt_tensor* tensors, int32_t count) {
  if (list_problem(tensors, count, RDT_F32)) return 0;
  // one partial sum for each block of each launch (num_sms() is not asked: no device needed)
  return (static_cast<size_t>(count) / kMaxTensors + 2) * 1024 * sizeof(double);
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
  cudaError_t e = each_launch(tensors, count, [&](const Table& tab, int tiles) {
    if (tiles == 0) return cudaSuccess;
    const int blocks = static_cast<int>(std::min<int64_t>(sq_blocks(tiles), 1024));
    if (used + blocks > room) return cudaErrorInvalidValue;
    note_launch();
    if (g_dtype == RDT_BF16)
      tensors_sq_sum_kernel<true><<<blocks, kThreads, 0, s>>>(tab, tiles, parts + used);
    else
      tensors_sq_sum_kernel<false><<<blocks, kThreads, 0, s>>>(tab, tiles, parts + used);
    used += blocks;
    return cudaGetLastError();
  });
  if (e != cudaSuccess) return launched(e);
  note_launch();
  tensors_sq_final_kernel<<<1, kThreads, 0, s>>>(parts, static_cast<int>(used), sumsq);
  return launched(cudaGetLastError());
}

rdt_status rdt_tensors_adamw(const rdt_opt_tensor* tensors, int32_t count, int32_t g_dtype,
                             int32_t state_bits, int64_t seed, const float* scale,
                             const int32_t* skip_flag, int32_t step, const int32_t* step_dev,
                             float beta1, float beta2, float eps, void* stream) {
  if (const char* why = list_problem(tensors, count, g_dtype)) return refuse(why);
  if (state_bits != 32 && state_bits != 8) return refuse("state_bits must be 32 or 8");
  if (seed >= (int64_t(1) << 32)) return refuse("seed must be below 2^32");
  if (!step_dev && step < 1) return refuse("step must be >= 1 (bias correction)");
  if (!(beta1 >= 0.f && beta1 < 1.f) || !(beta2 >= 0.f && beta2 < 1.f) || !(eps >= 0.f))
    return refuse("beta1 and beta2 must be in [0, 1) and eps >= 0");
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
  a.eps = eps;
  a.scale = scale;
  a.skip = skip_flag;
  a.step_dev = step_dev;
  a.seed = seed < 0 ? 0u : static_cast<uint32_t>(seed);
  const bool random = seed >= 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return launched(each_launch(tensors, count, [&](const Table& tab, int tiles) {
    if (tiles == 0) return cudaSuccess;
    const int blocks = static_cast<int>(std::min<int64_t>(tiles, 8LL * num_sms()));
    note_launch();
    const bool half = g_dtype == RDT_BF16;
    auto kernel = state_bits == 32 ? (half ? tensors_adamw_kernel<32, true, false>
                                           : tensors_adamw_kernel<32, false, false>)
                  : random ? (half ? tensors_adamw_kernel<8, true, true>
                                   : tensors_adamw_kernel<8, false, true>)
                           : (half ? tensors_adamw_kernel<8, true, false>
                                   : tensors_adamw_kernel<8, false, false>);
    kernel<<<blocks, kThreads, 0, s>>>(tab, tiles, a);
    return cudaGetLastError();
  }));
}

}  // extern "C"
