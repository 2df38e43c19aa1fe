// RMSNorm of every query and key head with the rotation at given positions in
// the same pass, and the backward pass of both (rdt_qk_norm_rope,
// rdt_qk_norm_rope_backward).
//
//   n = x rsqrt(mean x^2 + eps) gain;  (n_i, n_{i + d/2}) turned by the angle
//   positions[axis of i][t] theta^(-2i/d)
// backward: dn = the gradient turned back; d_gain = sum dn x r;
//   dx = r (dn gain - x r mean(dn gain x r)), r = rsqrt(mean x^2 + eps).
//
// Bound by DRAM: every value is read once and written once. A lane holds
// eight neighbouring pairs (two 16-byte loads of a 16-bit type), so a head of
// 128 is eight lanes and a warp takes four heads at a time, several such
// passes' loads under way at once; all heads of a token share the lane's eight
// cosines and sines.
//
// Angles: a full turn is 2^64. A pair's rate is kept as a 64-bit fraction of a
// turn, the product with the position is taken modulo 2^64, and its upper 32
// bits are the angle, exact to 2^-32 turns beside the rate's own rounding
// (2^-53), however far the position.
#include <algorithm>
#include <cmath>

#include "heads.cuh"

namespace rdt {

namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kMaxHalf = 128;  // pairs of a head of 256

struct Rates {
  uint64_t turn[kMaxHalf];  // turns a position, in 2^-64
  int end[3];               // first pair of axis 1, 2, 3
};

struct NormArgs {
  const void *q, *k;
  int64_t q_ts, q_hs, k_ts, k_hs;
  const float *gain_q, *gain_k;  // null: no norm
  float eps;
  const int32_t* positions;  // null: no rotation
  int axes;
  void *q_out, *k_out;
  int64_t qo_ts, qo_hs, ko_ts, ko_hs;
  int out_dtype;
  int tokens, nh, nkv, d;
  int lanes;       // lanes of a head, a power of two; those past d / 16 have nothing
  int lanes_log2;
  int passes;      // of a warp over a token's heads
  int slices;      // warps that share a token's passes
};

// Where a lane stands: head slot within the pass and chunk of eight pairs.
struct Lane {
  int slot, chunk, per_pass;
  bool has;
  __device__ __forceinline__ explicit Lane(const NormArgs& a) {
    const int lane = threadIdx.x & 31;
    slot = lane >> a.lanes_log2;
    chunk = lane & (a.lanes - 1);
    per_pass = 32 >> a.lanes_log2;
    has = 16 * chunk < a.d;
  }
};

// A lane's rates and axes (two bits each), read once.
struct Turning {
  uint64_t turn[8];
  uint32_t axis;
  __device__ __forceinline__ Turning(const NormArgs& a, const Rates& r, int chunk) {
    axis = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int pair = min(8 * chunk + i, kMaxHalf - 1);
      turn[i] = r.turn[pair];
      const int which = (pair >= r.end[0]) + (pair >= r.end[1]) + (pair >= r.end[2]);
      axis |= static_cast<uint32_t>(which) << (2 * i);
    }
  }
  __device__ __forceinline__ void at(const NormArgs& a, int token, float (&cos)[8],
                                     float (&sin)[8]) const {
    if (!a.positions) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        cos[i] = 1.f;
        sin[i] = 0.f;
      }
      return;
    }
    const int p0 = a.positions[token];
    int p1 = p0, p2 = p0, p3 = p0;
    if (a.axes > 1) p1 = a.positions[static_cast<int64_t>(a.tokens) + token];
    if (a.axes > 2) p2 = a.positions[2 * static_cast<int64_t>(a.tokens) + token];
    if (a.axes > 3) p3 = a.positions[3 * static_cast<int64_t>(a.tokens) + token];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t w = (axis >> (2 * i)) & 3;
      const int64_t p = w == 0 ? p0 : w == 1 ? p1 : w == 2 ? p2 : p3;
      const int32_t half_turns = static_cast<int32_t>((static_cast<uint64_t>(p) * turn[i]) >> 32);
      sincospif(static_cast<float>(half_turns) * 0x1p-31f, &sin[i], &cos[i]);
    }
  }
};

__device__ __forceinline__ float head_sum(float v, int lanes) {
  for (int o = lanes >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// kBatch passes' loads are under way at once.
template <typename T, int kBatch>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const NormArgs a,
                                                             const __grid_constant__ Rates rates) {
  __shared__ float gain[2][2 * kMaxHalf];
  after_previous_kernel();
  const Lane at(a);
  const int half = a.d >> 1, heads = a.nh + a.nkv;
  for (int i = threadIdx.x; i < 2 * a.d; i += kThreads) {
    const int which = i >= a.d, c = which ? i - a.d : i;
    const float* g = which ? a.gain_k : a.gain_q;
    gain[which][c] = g ? g[c] : 1.f;
  }
  const Turning turning(a, rates, at.chunk);
  __syncthreads();
  const int64_t units = static_cast<int64_t>(a.tokens) * a.slices;
  const int per_slice = (a.passes + a.slices - 1) / a.slices;
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); u < units;
       u += static_cast<int64_t>(gridDim.x) * kWarps) {
    const int token = static_cast<int>(u / a.slices), slice = static_cast<int>(u % a.slices);
    const int last = min(a.passes, (slice + 1) * per_slice);
    float cos[8], sin[8];
    for (int first = slice * per_slice; first < last; first += kBatch) {
      Eight<T> lo[kBatch], hi[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int h = (first + b) * at.per_pass + at.slot;
        if (at.has && first + b < last && h < heads) {
          const T* x = h < a.nh
                           ? static_cast<const T*>(a.q) + token * a.q_ts + h * a.q_hs
                           : static_cast<const T*>(a.k) + token * a.k_ts + (h - a.nh) * a.k_hs;
          lo[b].load(x + 8 * at.chunk);
          hi[b].load(x + half + 8 * at.chunk);
        } else {
          lo[b].zero();
          hi[b].zero();
        }
      }
      if (first == slice * per_slice) turning.at(a, token, cos, sin);
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        if (first + b >= last) break;
        const int h = (first + b) * at.per_pass + at.slot;
        const bool key = h >= a.nh;
        float x[8], y[8];
        lo[b].get(x);
        hi[b].get(y);
        float sq = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) sq = fmaf(x[i], x[i], fmaf(y[i], y[i], sq));
        sq = head_sum(sq, a.lanes);
        const float r = (key ? a.gain_k : a.gain_q) ? rsqrtf(sq / a.d + a.eps) : 1.f;
        if (!at.has || h >= heads) continue;
        const float* g = gain[key] + 8 * at.chunk;
        float u0[8], u1[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float p = x[i] * r * g[i], q = y[i] * r * g[half + i];
          u0[i] = p * cos[i] - q * sin[i];
          u1[i] = q * cos[i] + p * sin[i];
        }
        void* out = key ? a.k_out : a.q_out;
        const int64_t o = key ? token * a.ko_ts + (h - a.nh) * a.ko_hs
                              : token * a.qo_ts + h * a.qo_hs;
        store_eight(out, a.out_dtype, o + 8 * at.chunk, u0);
        store_eight(out, a.out_dtype, o + half + 8 * at.chunk, u1);
      }
    }
  }
}

struct GradArgs {
  NormArgs n;  // q_out and k_out are dq and dk
  const void *d_q, *d_k;
  int64_t dq_ts, dq_hs, dk_ts, dk_hs;
  float* partial;  // [CTAs][2][d]: sums of the gains' gradients
};

// G: type of the incoming gradient, T: type of q and k.
template <typename G, typename T, int kBatch>
__global__ void __launch_bounds__(kThreads)
    norm_rope_grad_kernel(const GradArgs ga, const __grid_constant__ Rates rates) {
  const NormArgs& a = ga.n;
  __shared__ float gain[2][2 * kMaxHalf];
  __shared__ float sums[kWarps][2 * kMaxHalf];
  after_previous_kernel();
  const Lane at(a);
  const int half = a.d >> 1, heads = a.nh + a.nkv;
  for (int i = threadIdx.x; i < 2 * a.d; i += kThreads) {
    const int which = i >= a.d, c = which ? i - a.d : i;
    const float* g = which ? a.gain_k : a.gain_q;
    gain[which][c] = g ? g[c] : 1.f;
  }
  const Turning turning(a, rates, at.chunk);
  __syncthreads();
  const int64_t units = static_cast<int64_t>(a.tokens) * a.slices;
  const int per_slice = (a.passes + a.slices - 1) / a.slices;
  float acc[2][16] = {};  // [query, key][lower half, upper half]
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); u < units;
       u += static_cast<int64_t>(gridDim.x) * kWarps) {
    const int token = static_cast<int>(u / a.slices), slice = static_cast<int>(u % a.slices);
    const int last = min(a.passes, (slice + 1) * per_slice);
    float cos[8], sin[8];
    for (int first = slice * per_slice; first < last; first += kBatch) {
      Eight<T> xlo[kBatch], xhi[kBatch];
      Eight<G> glo[kBatch], ghi[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int h = (first + b) * at.per_pass + at.slot;
        if (at.has && first + b < last && h < heads) {
          const bool key = h >= a.nh;
          const T* x = !key ? static_cast<const T*>(a.q) + token * a.q_ts + h * a.q_hs
                            : static_cast<const T*>(a.k) + token * a.k_ts + (h - a.nh) * a.k_hs;
          const G* g = !key
                           ? static_cast<const G*>(ga.d_q) + token * ga.dq_ts + h * ga.dq_hs
                           : static_cast<const G*>(ga.d_k) + token * ga.dk_ts +
                                 (h - a.nh) * ga.dk_hs;
          xlo[b].load(x + 8 * at.chunk);
          xhi[b].load(x + half + 8 * at.chunk);
          glo[b].load(g + 8 * at.chunk);
          ghi[b].load(g + half + 8 * at.chunk);
        } else {
          xlo[b].zero();
          xhi[b].zero();
          glo[b].zero();
          ghi[b].zero();
        }
      }
      if (first == slice * per_slice) turning.at(a, token, cos, sin);
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        if (first + b >= last) break;
        const int h = (first + b) * at.per_pass + at.slot;
        const bool key = h >= a.nh;
        const bool norm = (key ? a.gain_k : a.gain_q) != nullptr;
        float x[8], y[8], d0[8], d1[8];
        xlo[b].get(x);
        xhi[b].get(y);
        glo[b].get(d0);
        ghi[b].get(d1);
        float sq = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) sq = fmaf(x[i], x[i], fmaf(y[i], y[i], sq));
        sq = head_sum(sq, a.lanes);
        const float r = norm ? rsqrtf(sq / a.d + a.eps) : 1.f;
        const float* g = gain[key] + 8 * at.chunk;
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float p = d0[i] * cos[i] + d1[i] * sin[i];
          const float q = d1[i] * cos[i] - d0[i] * sin[i];
          x[i] *= r;
          y[i] *= r;
          if (at.has && h < heads) {  // a slot without a head may have r = inf (eps 0)
            if (key) {
              acc[1][i] += p * x[i];
              acc[1][8 + i] += q * y[i];
            } else {
              acc[0][i] += p * x[i];
              acc[0][8 + i] += q * y[i];
            }
            d0[i] = p * g[i];
            d1[i] = q * g[half + i];
          } else {
            d0[i] = d1[i] = 0.f;
          }
          dot = fmaf(d0[i], x[i], fmaf(d1[i], y[i], dot));
        }
        dot = head_sum(dot, a.lanes);
        const float mean = norm ? dot / a.d : 0.f;
        if (!at.has || h >= heads) continue;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          d0[i] = r * (d0[i] - x[i] * mean);
          d1[i] = r * (d1[i] - y[i] * mean);
        }
        void* out = key ? a.k_out : a.q_out;
        const int64_t o = key ? token * a.ko_ts + (h - a.nh) * a.ko_hs
                              : token * a.qo_ts + h * a.qo_hs;
        store_eight(out, a.out_dtype, o + 8 * at.chunk, d0);
        store_eight(out, a.out_dtype, o + half + 8 * at.chunk, d1);
      }
    }
  }
  if (!ga.partial) return;
  // lanes of one chunk, then the CTA's warps, each in a fixed order
  for (int which = 0; which < 2; ++which) {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      for (int o = a.lanes; o < 32; o <<= 1)
        acc[which][i] += __shfl_xor_sync(0xffffffffu, acc[which][i], o);
    if (at.slot == 0 && at.has) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        sums[threadIdx.x >> 5][8 * at.chunk + i] = acc[which][i];
        sums[threadIdx.x >> 5][half + 8 * at.chunk + i] = acc[which][8 + i];
      }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < a.d; c += kThreads) {
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) sum += sums[w][c];
      ga.partial[(static_cast<int64_t>(blockIdx.x) * 2 + which) * a.d + c] = sum;
    }
    __syncthreads();
  }
}

// d_gain[c] (= or +=) the sum of column c of partial [rows][2][d]: a CTA has 32
// columns, its warps a share of the rows each, joined in order.
__global__ void __launch_bounds__(1024) gain_sum_kernel(const float* partial, int rows, int d,
                                                        float* dg_q, float* dg_k,
                                                        int accumulate) {
  __shared__ float sums[32][33];
  after_previous_kernel();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float sum = 0.f;
  if (c < 2 * d)
    for (int r = warp; r < rows; r += 32) sum += partial[static_cast<int64_t>(r) * 2 * d + c];
  sums[warp][lane] = sum;
  __syncthreads();
  if (warp) return;
  sum = 0.f;
#pragma unroll
  for (int w = 0; w < 32; ++w) sum += sums[w][lane];
  float* out = c < d ? dg_q : dg_k;
  if (c < 2 * d && out) {
    out += c < d ? c : c - d;
    *out = accumulate ? *out + sum : sum;
  }
}

constexpr int kCtasPerSm = 4;

// Fills in the split of the work; returns the number of CTAs.
int64_t split_work(NormArgs* a, int ctas_per_sm) {
  int lanes = 1, log2 = 0;
  while (lanes * 16 < a->d) {
    lanes *= 2;
    ++log2;
  }
  a->lanes = lanes;
  a->lanes_log2 = log2;
  const int per_pass = 32 / lanes;
  a->passes = (a->nh + a->nkv + per_pass - 1) / per_pass;
  // few tokens: their heads are spread over more warps, which each take the
  // token's sines again
  const int64_t warps = static_cast<int64_t>(num_sms()) * ctas_per_sm * kWarps;
  const int64_t want = (warps + a->tokens - 1) / a->tokens;
  a->slices = static_cast<int>(std::min<int64_t>(want, a->passes));
  const int per_slice = (a->passes + a->slices - 1) / a->slices;
  a->slices = (a->passes + per_slice - 1) / per_slice;
  const int64_t units = static_cast<int64_t>(a->tokens) * a->slices;
  return std::min<int64_t>((units + kWarps - 1) / kWarps,
                           static_cast<int64_t>(num_sms()) * ctas_per_sm);
}

const char* shape_problem(int tokens, int nh, int nkv, int d) {
  if (tokens < 0) return "tokens must be >= 0";
  if (nh < 0 || nkv < 0 || nh + static_cast<int64_t>(nkv) < 1 || nh > 4096 || nkv > 4096)
    return "n_heads and n_kv_heads must be in [0, 4096] and not both 0";
  if (d < 16 || d > 2 * kMaxHalf || d % 16) return "head_dim must be a multiple of 16 in [16, 256]";
  return nullptr;
}

// Checks what both calls have in common and fills in the arguments.
const char* common_problem(int tokens, int nh, int nkv, int d, const rdt_heads* q,
                           const rdt_heads* k, int dtype, const float* gain_q, const float* gain_k,
                           float eps, const int32_t* positions, int axes, const int32_t* sections,
                           float theta, const rdt_heads* q_out, const rdt_heads* k_out,
                           int out_dtype, NormArgs* a, Rates* rates) {
  if (!dtype_ok(dtype) || !dtype_ok(out_dtype))
    return "dtypes must be RDT_F32, RDT_BF16 or RDT_F16";
  const rdt_heads none = {};
  const rdt_heads *ins[2] = {q, k}, *outs[2] = {q_out, k_out};
  const int heads[2] = {nh, nkv};
  for (int i = 0; i < 2; ++i) {
    if (heads[i] == 0) continue;
    if (const char* why = heads_problem(ins[i], tokens, heads[i], d, dtype_bytes(dtype), false))
      return why;
    if (const char* why =
            heads_problem(outs[i], tokens, heads[i], d, dtype_bytes(out_dtype), true))
      return why;
    if (ins[i]->data == outs[i]->data &&
        (dtype != out_dtype || (tokens > 1 && ins[i]->token_stride != outs[i]->token_stride) ||
         (heads[i] > 1 && ins[i]->head_stride != outs[i]->head_stride)))
      return "an output at its input's place needs the input's type and strides";
  }
  if (nh == 0) q = q_out = &none;
  if (nkv == 0) k = k_out = &none;
  if (!aligned4(gain_q) || !aligned4(gain_k) || !aligned4(positions))
    return "gains and positions must be 4-byte aligned";
  if (!(eps >= 0.f) || std::isinf(eps)) return "eps must be finite and >= 0";
  *rates = Rates{};
  if (positions) {
    if (axes < 1 || axes > 4) return "axes must be in [1, 4]";
    if (!(theta > 0.f) || std::isinf(theta)) return "theta must be finite and > 0";
    if (axes > 1 && !sections) return "sections are needed with more than one axis";
    int sum = 0;
    for (int i = 0; i < 3; ++i) rates->end[i] = INT32_MAX;
    if (sections) {
      for (int i = 0; i < axes; ++i) {
        if (sections[i] < 0 || sections[i] > d) return "a section must be in [0, head_dim / 2]";
        sum += sections[i];
        if (i + 1 < axes) rates->end[i] = sum;
      }
      if (sum != d / 2) return "sections must add up to head_dim / 2";
    }
    for (int i = 0; i < d / 2; ++i) {
      const double turns = std::pow(static_cast<double>(theta), -2.0 * i / d) / 6.283185307179586477;
      // whole turns of a position change nothing; 2^64 itself would not fit
      rates->turn[i] = static_cast<uint64_t>(std::ldexp(turns - std::floor(turns), 63)) * 2;
    }
  }
  *a = NormArgs{q->data,         k->data,         q->token_stride, q->head_stride, k->token_stride,
                k->head_stride,  gain_q,          gain_k,          eps,            positions,
                axes,            q_out->data,     k_out->data,     q_out->token_stride,
                q_out->head_stride, k_out->token_stride, k_out->head_stride, out_dtype,
                tokens,          nh,              nkv,             d,              0, 0, 0, 0};
  return nullptr;
}

template <typename T, int kBatch>
cudaError_t launch_norm(NormArgs a, const Rates& r, cudaStream_t s) {
  const int64_t grid = split_work(&a, kCtasPerSm);
  return launch_overlapping(norm_rope_kernel<T, kBatch>, grid, kThreads, 0, s, a, r);
}

constexpr int kGradCtasPerSm = 2;

template <typename G>
cudaError_t launch_grad(const GradArgs& a, int dtype, int64_t grid, const Rates& r,
                        cudaStream_t s) {
  if (dtype == RDT_F32)
    return launch_overlapping(norm_rope_grad_kernel<G, float, 1>, grid, kThreads, 0, s, a, r);
  if (dtype == RDT_BF16)
    return launch_overlapping(norm_rope_grad_kernel<G, bf16, 2>, grid, kThreads, 0, s, a, r);
  return launch_overlapping(norm_rope_grad_kernel<G, __half, 2>, grid, kThreads, 0, s, a, r);
}

}  // namespace

}  // namespace rdt

using namespace rdt;

extern "C" {

rdt_status rdt_qk_norm_rope(int32_t tokens, int32_t n_heads, int32_t n_kv_heads, int32_t head_dim,
                            const rdt_heads* q, const rdt_heads* k, int32_t dtype,
                            const float* gain_q, const float* gain_k, float eps,
                            const int32_t* positions, int32_t axes, const int32_t* sections,
                            float theta, const rdt_heads* q_out, const rdt_heads* k_out,
                            int32_t out_dtype, void* stream) {
  if (const char* why = shape_problem(tokens, n_heads, n_kv_heads, head_dim)) return refuse(why);
  if (tokens == 0) return RDT_OK;
  NormArgs a;
  Rates r;
  if (const char* why = common_problem(tokens, n_heads, n_kv_heads, head_dim, q, k, dtype, gain_q,
                                       gain_k, eps, positions, axes, sections, theta, q_out, k_out,
                                       out_dtype, &a, &r))
    return refuse(why);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return launched(dtype == RDT_F32    ? launch_norm<float, 2>(a, r, s)
                  : dtype == RDT_BF16 ? launch_norm<bf16, 4>(a, r, s)
                                      : launch_norm<__half, 4>(a, r, s));
}

size_t rdt_qk_norm_rope_backward_workspace_bytes(int32_t tokens, int32_t n_heads,
                                                 int32_t n_kv_heads, int32_t head_dim) {
  if (shape_problem(tokens, n_heads, n_kv_heads, head_dim) || tokens == 0) return 0;
  NormArgs a = {};
  a.tokens = tokens;
  a.nh = n_heads;
  a.nkv = n_kv_heads;
  a.d = head_dim;
  return static_cast<size_t>(split_work(&a, kGradCtasPerSm)) * 2 * head_dim * sizeof(float);
}

rdt_status rdt_qk_norm_rope_backward(int32_t tokens, int32_t n_heads, int32_t n_kv_heads,
                                     int32_t head_dim, const rdt_heads* q, const rdt_heads* k,
                                     int32_t dtype, const float* gain_q, const float* gain_k,
                                     float eps, const int32_t* positions, int32_t axes,
                                     const int32_t* sections, float theta,
                                     const rdt_heads* d_q_out, const rdt_heads* d_k_out,
                                     int32_t d_dtype, const rdt_heads* dq, const rdt_heads* dk,
                                     int32_t out_dtype, float* d_gain_q, float* d_gain_k,
                                     int32_t accumulate, void* ws, size_t ws_bytes, void* stream) {
  if (const char* why = shape_problem(tokens, n_heads, n_kv_heads, head_dim)) return refuse(why);
  if (!aligned4(d_gain_q) || !aligned4(d_gain_k))
    return refuse("gain gradients must be 4-byte aligned");
  if ((d_gain_q && !gain_q) || (d_gain_k && !gain_k))
    return refuse("the gradient of a gain needs the gain");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (tokens == 0) {  // sums over nothing
    cudaError_t e = cudaSuccess;
    for (float* g : {d_gain_q, d_gain_k})
      if (e == cudaSuccess && g && !accumulate)
        e = cudaMemsetAsync(g, 0, sizeof(float) * head_dim, s);
    return launched(e);
  }
  if (!dtype_ok(d_dtype)) return refuse("d_dtype must be RDT_F32, RDT_BF16 or RDT_F16");
  GradArgs a = {};
  Rates r;
  if (const char* why = common_problem(tokens, n_heads, n_kv_heads, head_dim, q, k, dtype, gain_q,
                                       gain_k, eps, positions, axes, sections, theta, dq, dk,
                                       out_dtype, &a.n, &r))
    return refuse(why);
  const rdt_heads none = {};
  for (int i = 0; i < 2; ++i) {
    const rdt_heads *g = i ? d_k_out : d_q_out, *o = i ? dk : dq;
    const int heads = i ? n_kv_heads : n_heads;
    if (heads == 0) continue;
    if (const char* why =
            heads_problem(g, tokens, heads, head_dim, dtype_bytes(d_dtype), false))
      return refuse(why);
    if (g->data == o->data &&
        (d_dtype != out_dtype || (tokens > 1 && g->token_stride != o->token_stride) ||
         (heads > 1 && g->head_stride != o->head_stride)))
      return refuse("an output at its input's place needs the input's type and strides");
  }
  if (n_heads == 0) d_q_out = &none;
  if (n_kv_heads == 0) d_k_out = &none;
  a.d_q = d_q_out->data;
  a.d_k = d_k_out->data;
  a.dq_ts = d_q_out->token_stride;
  a.dq_hs = d_q_out->head_stride;
  a.dk_ts = d_k_out->token_stride;
  a.dk_hs = d_k_out->head_stride;
  const int64_t grid = split_work(&a.n, kGradCtasPerSm);
  const bool sums = d_gain_q || d_gain_k;
  if (sums) {
    if (!ws) return refuse("null pointer");
    if (reinterpret_cast<uintptr_t>(ws) & 255) return refuse("ws must be 256-byte aligned");
    if (ws_bytes < static_cast<size_t>(grid) * 2 * head_dim * sizeof(float))
      return refuse("workspace too small");
    a.partial = static_cast<float*>(ws);
  }
  cudaError_t e = d_dtype == RDT_F32    ? launch_grad<float>(a, dtype, grid, r, s)
                  : d_dtype == RDT_BF16 ? launch_grad<bf16>(a, dtype, grid, r, s)
                                        : launch_grad<__half>(a, dtype, grid, r, s);
  if (e == cudaSuccess && sums)
    e = launch_overlapping(gain_sum_kernel, (2 * head_dim + 31) / 32, 1024, 0, s, a.partial,
                           static_cast<int>(grid), head_dim, d_gain_q, d_gain_k,
                           accumulate ? 1 : 0);
  return launched(e);
}

}  // extern "C"
