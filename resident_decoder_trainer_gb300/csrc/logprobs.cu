// Token log probabilities with entropy, log-sum-exp and top alternatives from
// logits, their gradient, and the scoring head that calls them
// (rdt_token_logprobs, rdt_token_logprobs_backward, rdt_head_logprobs).
#include <algorithm>
#include <cmath>
#include <cstdio>
#include <cuda_fp16.h>

#include "../../include/rdt.h"
#include "common.cuh"
#include "internal.h"

namespace rdt {

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(bf16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
template <typename T> __device__ __forceinline__ T from_f(float x);
template <> __device__ __forceinline__ float from_f<float>(float x) { return x; }
template <> __device__ __forceinline__ bf16 from_f<bf16>(float x) { return __float2bfloat16_rn(x); }
template <> __device__ __forceinline__ __half from_f<__half>(float x) { return __float2half_rn(x); }

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
};

template <typename V, typename F>
__device__ __forceinline__ V block_reduce(V v, V* red, F f) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = f(v, __shfl_xor_sync(0xffffffffu, v, o));
  __syncthreads();
  if (lane == 0) red[warp] = v;
  __syncthreads();
  v = red[0];
  for (int w = 1; w < kThreads / 32; ++w) v = f(v, red[w]);
  return v;
}

// One CTA per row: maximum, then sums, then one pass per alternative.
template <typename T>
__global__ void __launch_bounds__(kThreads) logprobs_kernel(const LogprobArgs a) {
  __shared__ float redf[kThreads / 32];
  __shared__ unsigned long long redk[kThreads / 32];
  const int row = blockIdx.x, tid = threadIdx.x;
  const T* z = static_cast<const T*>(a.logits) + static_cast<int64_t>(row) * a.ld;
  const int target = a.targets ? a.targets[row] : 0;
  const float inf = INFINITY;
  float m = -inf, bad = 0.f, s0 = 0.f, s1 = 0.f;
  const bool scored = target >= 0;
  if (scored) {
    for (int j = tid; j < a.vocab; j += kThreads) {
      const float x = to_f(z[j]);
      m = fmaxf(m, x);
      if (!(x < inf)) bad = 1.f;
    }
    auto fmx = [](float x, float y) { return fmaxf(x, y); };
    auto fad = [](float x, float y) { return x + y; };
    m = block_reduce(m, redf, fmx);
    bad = block_reduce(bad, redf, fmx);
    if (bad == 0.f && m > -inf) {
      for (int j = tid; j < a.vocab; j += kThreads) {
        const float d = (to_f(z[j]) - m) * a.scale;
        const float e = expf(d);
        s0 += e;
        s1 += e > 0.f ? e * d : 0.f;
      }
      s0 = block_reduce(s0, redf, fad);
      s1 = block_reduce(s1, redf, fad);
    }
  }
  const bool live = scored && bad == 0.f, some = live && m > -inf;
  const float log_sum = some ? logf(s0) : 0.f;
  const float nan = __int_as_float(0x7fffffff);
  if (tid == 0) {
    const float dead = scored ? nan : 0.f;  // for rows that are not live
    if (a.logp) {
      float lp = dead;
      if (live) {
        lp = target >= a.vocab ? nan
             : some            ? (to_f(z[target]) - m) * a.scale - log_sum
                               : -inf;
      }
      a.logp[row] = lp;
    }
    if (a.entropy) a.entropy[row] = some ? log_sum - s1 / s0 : live ? 0.f : dead;
    if (a.lse) a.lse[row] = some ? m * a.scale + log_sum : live ? -inf : dead;
    if (a.stats) a.stats[row] = live ? make_float2(m, log_sum) : make_float2(dead, dead);
  }
  uint64_t last = ~0ull;
  for (int i = 0; i < a.top; ++i) {
    unsigned long long best = 0;
    if (some && last) {
      for (int j = tid; j < a.vocab; j += kThreads) {
        const uint64_t k = order_key(to_f(z[j]), j);
        if (k < last && k > best) best = k;
      }
      best = block_reduce(best, redk, [](unsigned long long x, unsigned long long y) {
        return x > y ? x : y;
      });
      last = best;
    }
    if (tid == 0) {
      const int64_t at = static_cast<int64_t>(row) * a.top + i;
      a.top_ids[at] = best ? static_cast<int32_t>(0xffffffffu - static_cast<uint32_t>(best)) : -1;
      a.top_logp[at] = best    ? (key_value(best) - m) * a.scale - log_sum
                       : live  ? -inf
                       : scored ? nan
                                : 0.f;
    }
  }
}

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
};

template <typename T, typename O>
__global__ void __launch_bounds__(kThreads) logprobs_grad_kernel(const GradArgs a) {
  const int row = blockIdx.x;
  const T* z = static_cast<const T*>(a.logits) + static_cast<int64_t>(row) * a.ld;
  O* out = static_cast<O*>(a.out) + static_cast<int64_t>(row) * a.ld_out;
  const int target = a.targets ? a.targets[row] : 0;
  const float2 st = a.stats[row];
  const float g = a.d_logp ? a.d_logp[row] : 0.f, h = a.d_entropy ? a.d_entropy[row] : 0.f;
  float c = (a.d_lse ? a.d_lse[row] : 0.f) - g;
  if (a.d_entropy) c -= h * a.entropy[row];
  const bool none = target < 0 || st.x == -INFINITY;
  const bool wrong = target >= a.vocab;
  for (int j = threadIdx.x; j < a.vocab; j += kThreads) {
    float r = 0.f;
    if (wrong) {
      r = __int_as_float(0x7fffffff);
    } else if (!none) {
      const float lp = (to_f(z[j]) - st.x) * a.scale - st.y;
      const float p = expf(lp);
      r = p == 0.f ? 0.f : p * (c - h * lp);
      if (a.targets && j == target) r += g;
      r *= a.scale;
    }
    out[j] = from_f<O>(r);
  }
}

bool dtype_ok(int dtype) { return dtype == RDT_F32 || dtype == RDT_BF16 || dtype == RDT_F16; }
int dtype_bytes(int dtype) { return dtype == RDT_F32 ? 4 : 2; }

rdt_status refuse(const char* msg) {
  set_last_error(msg);
  return RDT_EINVAL;
}
rdt_status launched(cudaError_t e) {
  if (e == cudaSuccess) return RDT_OK;
  set_last_error(cudaGetErrorString(e));
  return RDT_ECUDA;
}

cudaError_t logprobs(const LogprobArgs& a, int dtype, cudaStream_t s) {
  note_launch();
  if (dtype == RDT_F32)
    logprobs_kernel<float><<<a.rows, kThreads, 0, s>>>(a);
  else if (dtype == RDT_BF16)
    logprobs_kernel<bf16><<<a.rows, kThreads, 0, s>>>(a);
  else
    logprobs_kernel<__half><<<a.rows, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

template <typename T>
void launch_grad(const GradArgs& a, int d_dtype, cudaStream_t s) {
  if (d_dtype == RDT_F32)
    logprobs_grad_kernel<T, float><<<a.rows, kThreads, 0, s>>>(a);
  else if (d_dtype == RDT_BF16)
    logprobs_grad_kernel<T, bf16><<<a.rows, kThreads, 0, s>>>(a);
  else
    logprobs_grad_kernel<T, __half><<<a.rows, kThreads, 0, s>>>(a);
}

// What both calls check of their logits.
const char* logits_problem(const void* logits, int dtype, int64_t ld, int rows, int vocab,
                           float scale) {
  if (!dtype_ok(dtype)) return "dtype must be RDT_F32, RDT_BF16 or RDT_F16";
  if (rows < 0 || vocab < 1) return "rows must be >= 0 and vocab >= 1";
  if (ld < vocab) return "ld must be >= vocab";
  if (!(scale > 0.f) || !std::isfinite(scale)) return "logit_scale must be finite and > 0";
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
  float *rstd, *logits, *split;
  int64_t split_floats;
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
  LogprobArgs a{logits,  ld,  rows, vocab, logit_scale, targets, logp,
                entropy, lse, reinterpret_cast<float2*>(stats), top, top_ids, top_logp};
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
             entropy, d_logp, d_entropy, d_lse, d_logits,    ld_d};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  note_launch();
  if (dtype == RDT_F32)
    launch_grad<float>(a, d_dtype, s);
  else if (dtype == RDT_BF16)
    launch_grad<bf16>(a, d_dtype, s);
  else
    launch_grad<__half>(a, d_dtype, s);
  return launched(cudaGetLastError());
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
  if (!(logit_scale > 0.f) || !std::isfinite(logit_scale))
    return refuse("logit_scale must be finite and > 0");
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
