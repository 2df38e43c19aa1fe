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

#include "spans.cuh"

namespace rdt {

namespace {

constexpr int kRowWarps = 8, kRowThreads = 32 * kRowWarps;

__global__ void __launch_bounds__(kRowThreads) rows_forward_kernel(const SpanArgs a) {
  after_previous_kernel();
  const int warp = threadIdx.x >> 5;
  const int64_t rows = static_cast<int64_t>(a.queries) * a.nh;
  for (int64_t r = static_cast<int64_t>(blockIdx.x) * kRowWarps + warp; r < rows;
       r += static_cast<int64_t>(gridDim.x) * kRowWarps)
    row_forward(a, static_cast<int>(r / a.nh), static_cast<int>(r % a.nh), 0, a.d, true);
}

// The rows of dq, then those of dk and dv, in one grid.
__global__ void __launch_bounds__(kRowThreads) rows_backward_kernel(const SpanArgs a) {
  after_previous_kernel();
  const int warp = threadIdx.x >> 5;
  const int64_t dq_rows = static_cast<int64_t>(a.queries) * a.nh;
  const int64_t rows = dq_rows + static_cast<int64_t>(a.keys) * a.nkv;
  for (int64_t r = static_cast<int64_t>(blockIdx.x) * kRowWarps + warp; r < rows;
       r += static_cast<int64_t>(gridDim.x) * kRowWarps) {
    if (r < dq_rows) {
      row_dq(a, static_cast<int>(r / a.nh), static_cast<int>(r % a.nh), 0, a.d);
    } else {
      const int64_t x = r - dq_rows;
      row_dkdv(a, static_cast<int>(x / a.nkv), static_cast<int>(x % a.nkv), 0, a.d);
    }
  }
}

// ------------------------------------------------------------------- host
int64_t row_grid(int64_t rows) {
  return std::min<int64_t>((rows + kRowWarps - 1) / kRowWarps, int64_t{num_sms()} * 8);
}

// A problem without keys has no tensors to load tiles from.
bool in_tiles(int queries, int keys) { return queries > 0 && keys > 0; }

const char* shape_problem(int queries, int keys, int nh, int nkv, int d) {
  if (queries < 0 || keys < 0 || queries > 1 << 30 || keys > 1 << 30)
    return "queries and keys must be in [0, 2^30]";
  if (nkv < 1 || nh < nkv || nh % nkv || nh > 4096)
    return "n_heads must be a positive multiple of n_kv_heads, at most 4096";
  if (nh / nkv > 128) return "at most 128 query heads may share a key head";
  if (d < 16 || d > kMaxDim || d % 16) return "head_dim must be a multiple of 16 in [16, 128]";
  // tiles are counted in 32 bits
  if (int64_t{Tiling::of(queries, nh / nkv).tiles} * nkv > 1 << 29 ||
      (int64_t{keys} + 127) / 128 * nkv > 1 << 29)
    return "queries or keys times heads are too many";
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
  if (!(a.scale >= 1e-6f && a.scale <= 1e6f)) return "scale must be in [1e-6, 1e6]";
  // the seventh power of the quotient, in the cap's polynomial, is a normal number
  if (a.cap != 0.f && !(a.cap >= 1e-5f * a.scale && a.cap <= 1e5f * a.scale))
    return "softcap must be 0 or scale times [1e-5, 1e5]";
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
  if (!in_tiles(queries, keys)) return 0;
  const size_t n = backward
                       ? backward_workspace(queries, keys, n_heads, n_kv_heads, head_dim)
                       : forward_workspace(queries, keys, n_heads, n_kv_heads, head_dim);
  return (n + 255) / 256 * 256;
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
  if (in_tiles(queries, keys)) return launched(forward_tiles(a, ws, s));
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
  if (in_tiles(queries, keys)) return launched(backward_tiles(a, ws, s));
  const int64_t rows = int64_t{queries} * n_heads + int64_t{keys} * n_kv_heads;
  return launched(
      launch_overlapping(rows_backward_kernel, row_grid(rows), kRowThreads, 0, s, a));
}

}  // extern "C"
