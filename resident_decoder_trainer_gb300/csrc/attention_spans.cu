// Attention in which each query sees one span of keys, and its backward pass
// (rdt_attention, rdt_attention_backward).
//
//   s_j = scale q . k_j, capped: s_j = cap tanh(s_j / cap);  p = softmax over lo <= j < hi
//   o = sum_j p_j v_j,  lse = ln sum_j exp(s_j)
// backward: D = d_o . o - d_lse;  ds_j = p_j (d_o . v_j - D) (1 - tanh^2)
//   dq = scale sum_j ds_j k_j,  dk_j = scale sum_t ds_j q,  dv_j = sum_t p_j d_o,
// the sums over t over all query heads of the key's group.
#include <algorithm>
#include <cmath>

#include "heads.cuh"

namespace rdt {

namespace {

struct View {
  bf16* p;
  int64_t ts, hs;
  __device__ __forceinline__ bf16* at(int64_t t, int h) const { return p + t * ts + h * hs; }
};

struct SpanArgs {
  int queries, keys, nh, nkv, rep, d;
  View q, k, v, o, d_o, dq, dk, dv;
  const int *lo, *hi;  // null: 0, keys
  const float* d_lse;  // null: 0
  float* lse;
  float scale, cap;  // cap 0: none
  __device__ __forceinline__ void span(int t, int& first, int& end) const {
    first = lo ? max(lo[t], 0) : 0;
    end = hi ? min(hi[t], keys) : keys;
  }
};

constexpr int kRowWarps = 8, kRowThreads = 32 * kRowWarps;
constexpr int kMaxDim = 128;

// ------------------------------------------------- one warp per row of an output
// Lanes take 32 keys (or queries) at a time for the scores, and four columns
// each for the sums. All in fp32.

// Copies a head's values to shared memory as fp32; whole warp.
__device__ __forceinline__ void stage_row(float* dst, const bf16* src, int d) {
  for (int c = 2 * (threadIdx.x & 31); c < d; c += 64) {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(src + c);
    dst[c] = bf16lo(w);
    dst[c + 1] = bf16hi(w);
  }
}

__device__ __forceinline__ float dot_row(const float* a, const bf16* b, int d) {
  float s0 = 0.f, s1 = 0.f;
  for (int c = 0; c < d; c += 8) {
    Eight<bf16> e;
    float x[8];
    e.load(b + c);
    e.get(x);
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      s0 = fmaf(a[c + i], x[i], s0);
      s1 = fmaf(a[c + i + 1], x[i + 1], s1);
    }
  }
  return s0 + s1;
}

__device__ __forceinline__ float dot_rows(const bf16* a, const bf16* b, int d) {
  float s = 0.f;
  for (int c = 0; c < d; c += 8) {
    Eight<bf16> e, f;
    float x[8], y[8];
    e.load(a + c);
    f.load(b + c);
    e.get(x);
    f.get(y);
#pragma unroll
    for (int i = 0; i < 8; ++i) s = fmaf(x[i], y[i], s);
  }
  return s;
}

// Score of a product q . k, and what its cap's derivative is.
__device__ __forceinline__ float score_of(const SpanArgs& a, float dot, float& slope) {
  const float s = dot * a.scale;
  slope = 1.f;
  if (a.cap == 0.f) return s;
  const float th = tanhf(s / a.cap);
  slope = 1.f - th * th;
  return a.cap * th;
}

// acc[i] += w src[column i], columns 2 lane, 2 lane + 1, and those 64 further.
__device__ __forceinline__ void add_row(float (&acc)[4], float w, const bf16* src, int d) {
  const int c = 2 * (threadIdx.x & 31);
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    if (c + 64 * x >= d) break;
    const uint32_t two = *reinterpret_cast<const uint32_t*>(src + c + 64 * x);
    acc[2 * x] = fmaf(w, bf16lo(two), acc[2 * x]);
    acc[2 * x + 1] = fmaf(w, bf16hi(two), acc[2 * x + 1]);
  }
}
__device__ __forceinline__ void put_row(bf16* dst, const float (&acc)[4], float w, int d) {
  const int c = 2 * (threadIdx.x & 31);
#pragma unroll
  for (int x = 0; x < 2; ++x)
    if (c + 64 * x < d)
      *reinterpret_cast<uint32_t*>(dst + c + 64 * x) =
          pack_bf16x2(acc[2 * x] * w, acc[2 * x + 1] * w);
}

// o and lse of query t, head h. `mem` is kMaxDim floats of the warp's own.
__device__ void row_forward(const SpanArgs& a, float* mem, int t, int h) {
  const int lane = threadIdx.x & 31, g = h / a.rep;
  int first, end;
  a.span(t, first, end);
  __syncwarp();
  stage_row(mem, a.q.at(t, h), a.d);
  __syncwarp();
  float m = -INFINITY, l = 0.f, acc[4] = {};
  for (int64_t base = first; base < end; base += 32) {
    const int64_t j = base + lane;
    float s = -INFINITY, slope;
    if (j < end) s = score_of(a, dot_row(mem, a.k.at(j, g), a.d), slope);
    // fmaxf passes over a NaN; exp(s - m) below does not
    const float top = fmaxf(m, warp_max(s));
    const float alpha = m == top ? 1.f : expf(m - top);
    const float p = j < end ? expf(s - top) : 0.f;
    m = top;
    l = l * alpha + warp_sum(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] *= alpha;
    const int n = static_cast<int>(min(static_cast<int64_t>(32), end - base));
    for (int i = 0; i < n; ++i)
      add_row(acc, __shfl_sync(0xffffffffu, p, i), a.v.at(base + i, g), a.d);
  }
  const bool any = first < end;
  put_row(a.o.at(t, h), acc, any ? 1.f / l : 0.f, a.d);
  if (a.lse && lane == 0)
    a.lse[static_cast<int64_t>(t) * a.nh + h] = any ? m + logf(l) : -INFINITY;
}

// dq of query t, head h. `mem` is 2 kMaxDim floats of the warp's own.
__device__ void row_dq(const SpanArgs& a, float* mem, int t, int h) {
  const int lane = threadIdx.x & 31, g = h / a.rep;
  int first, end;
  a.span(t, first, end);
  float acc[4] = {};
  if (first < end) {
    __syncwarp();
    stage_row(mem, a.q.at(t, h), a.d);
    stage_row(mem + kMaxDim, a.d_o.at(t, h), a.d);
    __syncwarp();
    const int64_t th = static_cast<int64_t>(t) * a.nh + h;
    const float lse = a.lse[th];
    const float own = dot_row(mem + kMaxDim, a.o.at(t, h), a.d) - (a.d_lse ? a.d_lse[th] : 0.f);
    for (int64_t base = first; base < end; base += 32) {
      const int64_t j = base + lane;
      float ds = 0.f;
      if (j < end) {
        float slope;
        const float p = expf(score_of(a, dot_row(mem, a.k.at(j, g), a.d), slope) - lse);
        ds = p * (dot_row(mem + kMaxDim, a.v.at(j, g), a.d) - own) * slope;
      }
      const int n = static_cast<int>(min(static_cast<int64_t>(32), end - base));
      for (int i = 0; i < n; ++i)
        add_row(acc, __shfl_sync(0xffffffffu, ds, i), a.k.at(base + i, g), a.d);
    }
  }
  put_row(a.dq.at(t, h), acc, a.scale, a.d);
}

// dk and dv of key j, kv head g, from queries [t0, t1). `mem` as for row_dq.
__device__ void row_dkdv(const SpanArgs& a, float* mem, int j, int g, int t0, int t1) {
  const int lane = threadIdx.x & 31;
  __syncwarp();
  stage_row(mem, a.k.at(j, g), a.d);
  stage_row(mem + kMaxDim, a.v.at(j, g), a.d);
  __syncwarp();
  float ak[4] = {}, av[4] = {};
  for (int64_t base = t0; base < t1; base += 32) {
    const int64_t t = base + lane;
    bool sees = false;
    if (t < t1) {
      int first, end;
      a.span(static_cast<int>(t), first, end);
      sees = first <= j && j < end;
    }
    const unsigned who = __ballot_sync(0xffffffffu, sees);
    if (!who) continue;
    for (int r = 0; r < a.rep; ++r) {
      const int h = g * a.rep + r;
      float p = 0.f, ds = 0.f;
      if (sees) {
        const int64_t th = t * a.nh + h;
        float slope;
        p = expf(score_of(a, dot_row(mem, a.q.at(t, h), a.d), slope) - a.lse[th]);
        const float own =
            dot_rows(a.d_o.at(t, h), a.o.at(t, h), a.d) - (a.d_lse ? a.d_lse[th] : 0.f);
        ds = p * (dot_row(mem + kMaxDim, a.d_o.at(t, h), a.d) - own) * slope;
      }
      for (unsigned left = who; left; left &= left - 1) {
        const int i = __ffs(left) - 1;
        add_row(ak, __shfl_sync(0xffffffffu, ds, i), a.q.at(base + i, h), a.d);
        add_row(av, __shfl_sync(0xffffffffu, p, i), a.d_o.at(base + i, h), a.d);
      }
    }
  }
  put_row(a.dk.at(j, g), ak, a.scale, a.d);
  put_row(a.dv.at(j, g), av, 1.f, a.d);
}

__global__ void __launch_bounds__(kRowThreads) rows_forward_kernel(const SpanArgs a) {
  __shared__ float mem[kRowWarps][kMaxDim];
  after_previous_kernel();
  const int warp = threadIdx.x >> 5;
  const int64_t rows = static_cast<int64_t>(a.queries) * a.nh;
  for (int64_t r = static_cast<int64_t>(blockIdx.x) * kRowWarps + warp; r < rows;
       r += static_cast<int64_t>(gridDim.x) * kRowWarps)
    row_forward(a, mem[warp], static_cast<int>(r / a.nh), static_cast<int>(r % a.nh));
}

// The rows of dq, then those of dk and dv, in one grid.
__global__ void __launch_bounds__(kRowThreads) rows_backward_kernel(const SpanArgs a) {
  __shared__ float mem[kRowWarps][2 * kMaxDim];
  after_previous_kernel();
  const int warp = threadIdx.x >> 5;
  const int64_t dq_rows = static_cast<int64_t>(a.queries) * a.nh;
  const int64_t rows = dq_rows + static_cast<int64_t>(a.keys) * a.nkv;
  for (int64_t r = static_cast<int64_t>(blockIdx.x) * kRowWarps + warp; r < rows;
       r += static_cast<int64_t>(gridDim.x) * kRowWarps) {
    if (r < dq_rows) {
      row_dq(a, mem[warp], static_cast<int>(r / a.nh), static_cast<int>(r % a.nh));
    } else {
      const int64_t x = r - dq_rows;
      row_dkdv(a, mem[warp], static_cast<int>(x / a.nkv), static_cast<int>(x % a.nkv), 0,
               a.queries);
    }
  }
}

// ------------------------------------------------------------------- host
int64_t row_grid(int64_t rows) {
  return std::min<int64_t>((rows + kRowWarps - 1) / kRowWarps, int64_t{num_sms()} * 8);
}

const char* shape_problem(int queries, int keys, int nh, int nkv, int d) {
  if (queries < 0 || keys < 0 || queries > 1 << 30 || keys > 1 << 30)
    return "queries and keys must be in [0, 2^30]";
  if (nkv < 1 || nh < nkv || nh % nkv || nh > 4096)
    return "n_heads must be a positive multiple of n_kv_heads, at most 4096";
  if (nh / nkv > 128) return "at most 128 query heads may share a key head";
  if (d < 16 || d > kMaxDim || d % 16) return "head_dim must be a multiple of 16 in [16, 128]";
  return nullptr;
}

// An output at the address of an input or of another output.
template <size_t N>
bool shares(const rdt_heads* out, const rdt_heads* const (&others)[N]) {
  for (const rdt_heads* x : others)
    if (out && x && out->data == x->data) return true;
  return false;
}
constexpr char kShared[] = "an output is at an input's place or another output's";

View view_of(const rdt_heads* x) {
  return x ? View{static_cast<bf16*>(x->data), x->token_stride, x->head_stride} : View{};
}

// What both calls have in common.
const char* common_problem(const SpanArgs& a, const void* ws, size_t ws_bytes, size_t need) {
  if (!aligned4(a.lo) || !aligned4(a.hi) || !aligned4(a.lse) || !aligned4(a.d_lse))
    return "lo, hi and lse must be 4-byte aligned";
  if (!(a.scale > 0.f) || std::isinf(a.scale)) return "scale must be finite and > 0";
  if (!(a.cap >= 0.f) || std::isinf(a.cap)) return "softcap must be finite and >= 0";
  if (need) {
    if (!ws) return "null pointer";
    if (reinterpret_cast<uintptr_t>(ws) & 255) return "ws must be 256-byte aligned";
    if (ws_bytes < need) return "workspace too small";
  }
  return nullptr;
}

}  // namespace

}  // namespace rdt

using namespace rdt;

extern "C" {

size_t rdt_attention_workspace_bytes(int32_t queries, int32_t keys, int32_t n_heads,
                                     int32_t n_kv_heads, int32_t head_dim, int32_t backward) {
  if (shape_problem(queries, keys, n_heads, n_kv_heads, head_dim)) return 0;
  return 0;
}

rdt_status rdt_attention(int32_t queries, int32_t keys, int32_t n_heads, int32_t n_kv_heads,
                         int32_t head_dim, const rdt_heads* q, const rdt_heads* k,
                         const rdt_heads* v, const int32_t* lo, const int32_t* hi, float scale,
                         float softcap, const rdt_heads* o, float* lse, void* ws, size_t ws_bytes,
                         void* stream) {
  if (const char* why = shape_problem(queries, keys, n_heads, n_kv_heads, head_dim))
    return refuse(why);
  SpanArgs a = {queries, keys, n_heads, n_kv_heads, n_heads / n_kv_heads, head_dim};
  a.lo = lo;
  a.hi = hi;
  a.lse = lse;
  a.scale = scale;
  a.cap = softcap;
  const size_t need =
      rdt_attention_workspace_bytes(queries, keys, n_heads, n_kv_heads, head_dim, 0);
  if (const char* why = common_problem(a, ws, ws_bytes, need)) return refuse(why);
  if (queries == 0) return RDT_OK;
  for (const rdt_heads* x : {q, o})
    if (const char* why = heads_problem(x, queries, n_heads, head_dim, 2, x == o))
      return refuse(why);
  for (const rdt_heads* x : {k, v})
    if (keys > 0)
      if (const char* why = heads_problem(x, keys, n_kv_heads, head_dim, 2, false))
        return refuse(why);
  if (shares(o, {q, keys ? k : nullptr, keys ? v : nullptr})) return refuse(kShared);
  a.q = view_of(q);
  a.k = view_of(k);
  a.v = view_of(v);
  a.o = view_of(o);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return launched(launch_overlapping(rows_forward_kernel, row_grid(int64_t{queries} * n_heads),
                                     kRowThreads, 0, s, a));
}

rdt_status rdt_attention_backward(int32_t queries, int32_t keys, int32_t n_heads,
                                  int32_t n_kv_heads, int32_t head_dim, const rdt_heads* q,
                                  const rdt_heads* k, const rdt_heads* v, const rdt_heads* o,
                                  const float* lse, const rdt_heads* d_o, const float* d_lse,
                                  const int32_t* lo, const int32_t* hi, float scale, float softcap,
                                  const rdt_heads* dq, const rdt_heads* dk, const rdt_heads* dv,
                                  void* ws, size_t ws_bytes, void* stream) {
  if (const char* why = shape_problem(queries, keys, n_heads, n_kv_heads, head_dim))
    return refuse(why);
  SpanArgs a = {queries, keys, n_heads, n_kv_heads, n_heads / n_kv_heads, head_dim};
  a.lo = lo;
  a.hi = hi;
  a.lse = const_cast<float*>(lse);
  a.d_lse = d_lse;
  a.scale = scale;
  a.cap = softcap;
  const size_t need =
      rdt_attention_workspace_bytes(queries, keys, n_heads, n_kv_heads, head_dim, 1);
  if (const char* why = common_problem(a, ws, ws_bytes, need)) return refuse(why);
  if (queries == 0 && keys == 0) return RDT_OK;
  if (queries > 0) {
    if (!lse) return refuse("null pointer");
    for (const rdt_heads* x : {q, o, d_o, dq})
      if (const char* why = heads_problem(x, queries, n_heads, head_dim, 2, x == dq))
        return refuse(why);
  }
  if (keys > 0)
    for (const rdt_heads* x : {k, v, dk, dv})
      if (const char* why =
              heads_problem(x, keys, n_kv_heads, head_dim, 2, x == dk || x == dv))
        return refuse(why);
  if (queries > 0 && shares(dq, {q, o, d_o})) return refuse(kShared);
  if (keys > 0 && (shares(dk, {k, v, dv}) || shares(dv, {k, v}))) return refuse(kShared);
  if (queries > 0 && keys > 0 &&
      (shares(dq, {k, v, dk, dv}) || shares(dk, {q, o, d_o}) || shares(dv, {q, o, d_o})))
    return refuse(kShared);
  a.q = view_of(q);
  a.k = view_of(k);
  a.v = view_of(v);
  a.o = view_of(o);
  a.d_o = view_of(d_o);
  a.dq = view_of(dq);
  a.dk = view_of(dk);
  a.dv = view_of(dv);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int64_t rows = int64_t{queries} * n_heads + int64_t{keys} * n_kv_heads;
  return launched(
      launch_overlapping(rows_backward_kernel, row_grid(rows), kRowThreads, 0, s, a));
}

}  // extern "C"
