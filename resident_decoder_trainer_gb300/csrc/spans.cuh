// Attention over spans of keys: what its files share. The arguments of a call,
// and the computation of one output row by one warp, in fp32: what fills rows
// where there are no queries or no keys, and what repairs rows of the tensor-core
// kernels that are not finite.
#pragma once

#include "heads.cuh"

namespace rdt {

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
  // from 0 on both: differences with a key's index stay within 32 bits
  __device__ __forceinline__ void span(int t, int& first, int& end) const {
    first = lo ? max(lo[t], 0) : 0;
    end = hi ? max(min(hi[t], keys), 0) : keys;
  }
};

constexpr int kMaxDim = 128;  // of a head

// ------------------------------------------------------------------- waits
// A tensor-core kernel's warp computes its rows that came out not finite again,
// one after the other, while its CTA's others wait for it; and the warps of a row
// tile that sees few keys or none wait while their item's other tile walks
// through its own. Both take the longer the more there is to see. So a wait
// gives up after kWaitLimitNs and eight times what 32 rows have been seen to take:
// 16 us a key that a query sees, 30 us a query that sees a key (heads of 128).
constexpr uint64_t kNsOfKey = 8 * 16000, kNsOfQuery = 8 * 30000;
struct Patience {
  int* err;
  uint64_t limit_ns;
};
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, const Patience& p) {
  return mbar_wait(bar, parity, p.err, p.limit_ns);
}
__device__ __noinline__ static bool wait_longer(uint32_t bar, uint32_t parity, Patience p) {
  return mbar_wait(bar, parity, p);
}
__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity, const Patience& p) {
  return mbar_try_wait(bar, parity) || wait_longer(bar, parity, p);
}
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, const Patience& p) {
  return warp_wait(bar, parity, p.err, p.limit_ns);
}

// ------------------------------------------------- one warp per row of an output
// Lanes take 32 keys (or queries) at a time for the scores, and four columns
// each for the sums. All in fp32. Columns [c0, c1) are written.

// Eight consecutive values, as loaded.
struct Eight {
  uint4 a;
  __device__ __forceinline__ void load(const bf16* p) { a = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = bf16lo(w[i]);
      x[2 * i + 1] = bf16hi(w[i]);
    }
  }
};

__device__ __forceinline__ float dot_rows(const bf16* a, const bf16* b, int d) {
  float s0 = 0.f, s1 = 0.f;
#pragma unroll 4
  for (int c = 0; c < d; c += 8) {
    Eight e, f;
    float x[8], y[8];
    e.load(a + c);
    f.load(b + c);
    e.get(x);
    f.get(y);
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      s0 = fmaf(x[i], y[i], s0);
      s1 = fmaf(x[i + 1], y[i + 1], s1);
    }
  }
  return s0 + s1;
}

// Score of a product q . k, and what its cap's derivative is.
__device__ __forceinline__ float score_of(const SpanArgs& a, float dot, float& slope) {
  const float s = dot * a.scale;
  slope = 1.f;
  if (a.cap == 0.f) return s;
  const float x = s / a.cap, e = expf(-2.f * fabsf(x));
  slope = 4.f * e / ((1.f + e) * (1.f + e));  // 1 - tanh^2, which cancels
  return a.cap * tanhf(x);
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
__device__ __forceinline__ void put_row(bf16* dst, const float (&acc)[4], float w, int c0, int c1) {
  const int c = 2 * (threadIdx.x & 31);
#pragma unroll
  for (int x = 0; x < 2; ++x)
    if (c + 64 * x >= c0 && c + 64 * x < c1)
      *reinterpret_cast<uint32_t*>(dst + c + 64 * x) =
          pack_bf16x2(acc[2 * x] * w, acc[2 * x + 1] * w);
}

// o of query t, head h, and its lse where `with_lse`.
__device__ __noinline__ static void row_forward(const SpanArgs& a, int t, int h, int c0, int c1,
                                              bool with_lse) {
  const int lane = threadIdx.x & 31, g = h / a.rep;
  int first, end;
  a.span(t, first, end);
  float m = -INFINITY, l = 0.f, acc[4] = {};
  for (int64_t base = first; base < end; base += 32) {
    const int64_t j = base + lane;
    float s = -INFINITY, slope;
    if (j < end) s = score_of(a, dot_rows(a.q.at(t, h), a.k.at(j, g), a.d), slope);
    // fmaxf passes over a NaN; exp(s - m) below does not
    const float top = fmaxf(m, warp_max(s));
    const float base_of = top == -INFINITY ? 0.f : top;
    const float alpha = m == -INFINITY ? 1.f : expf(m - base_of);
    const float p = j < end ? expf(s - base_of) : 0.f;
    m = top;
    l = l * alpha + warp_sum(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] *= alpha;
    const int n = static_cast<int>(min(static_cast<int64_t>(32), end - base));
    for (int i = 0; i < n; ++i)
      add_row(acc, __shfl_sync(0xffffffffu, p, i), a.v.at(base + i, g), a.d);
  }
  put_row(a.o.at(t, h), acc, l != 0.f ? 1.f / l : 0.f, c0, c1);
  if (with_lse && a.lse && lane == 0)
    a.lse[static_cast<int64_t>(t) * a.nh + h] = l != 0.f ? m + logf(l) : -INFINITY;
}

// dq of query t, head h.
__device__ __noinline__ static void row_dq(const SpanArgs& a, int t, int h, int c0, int c1) {
  const int lane = threadIdx.x & 31, g = h / a.rep;
  int first, end;
  a.span(t, first, end);
  float acc[4] = {};
  if (first < end) {
    const int64_t th = static_cast<int64_t>(t) * a.nh + h;
    const float lse = a.lse[th];
    const float own =
        dot_rows(a.d_o.at(t, h), a.o.at(t, h), a.d) - (a.d_lse ? a.d_lse[th] : 0.f);
    for (int64_t base = first; base < end; base += 32) {
      const int64_t j = base + lane;
      float ds = 0.f;
      if (j < end) {
        float slope;
        const float p =
            expf(score_of(a, dot_rows(a.q.at(t, h), a.k.at(j, g), a.d), slope) - lse);
        ds = p * (dot_rows(a.d_o.at(t, h), a.v.at(j, g), a.d) - own) * slope;
      }
      const int n = static_cast<int>(min(static_cast<int64_t>(32), end - base));
      for (int i = 0; i < n; ++i)
        add_row(acc, __shfl_sync(0xffffffffu, ds, i), a.k.at(base + i, g), a.d);
    }
  }
  put_row(a.dq.at(t, h), acc, a.scale, c0, c1);
}

// dk and dv of key j, kv head g.
__device__ __noinline__ static void row_dkdv(const SpanArgs& a, int j, int g, int c0, int c1) {
  const int lane = threadIdx.x & 31;
  float ak[4] = {}, av[4] = {};
  for (int64_t base = 0; base < a.queries; base += 32) {
    const int64_t t = base + lane;
    bool sees = false;
    if (t < a.queries) {
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
        p = expf(score_of(a, dot_rows(a.q.at(t, h), a.k.at(j, g), a.d), slope) - a.lse[th]);
        const float own =
            dot_rows(a.d_o.at(t, h), a.o.at(t, h), a.d) - (a.d_lse ? a.d_lse[th] : 0.f);
        ds = p * (dot_rows(a.d_o.at(t, h), a.v.at(j, g), a.d) - own) * slope;
      }
      for (unsigned left = who; left; left &= left - 1) {
        const int i = __ffs(left) - 1;
        add_row(ak, __shfl_sync(0xffffffffu, ds, i), a.q.at(base + i, h), a.d);
        add_row(av, __shfl_sync(0xffffffffu, p, i), a.d_o.at(base + i, h), a.d);
      }
    }
  }
  put_row(a.dk.at(j, g), ak, a.scale, c0, c1);
  put_row(a.dv.at(j, g), av, 1.f, c0, c1);
}

// Whether one of the two bf16 values is not finite.
__device__ __forceinline__ bool bad_pair(uint32_t two) {
  return (two & 0x7f80u) == 0x7f80u || (two & 0x7f800000u) == 0x7f800000u;
}

// A lane has the columns [c0, c1) of a row of sums over keys (null: none) as stored,
// and which keys it sees: the lanes (bits) in whose row some column is not finite
// though no seen key is in that column of x, key head g: what is not finite by
// right is not computed again. Whole warp. Reads the seen keys until every such
// column has found one.
__device__ __noinline__ static unsigned bad_rows(const SpanArgs& a, const View& x, int g,
                                                const bf16* row, int c0, int c1, int first,
                                                int end) {
  const int lane = threadIdx.x & 31;
  uint32_t bad[kMaxDim / 32] = {};
  if (row) {
#pragma unroll
    for (int w = 0; w < kMaxDim / 32; ++w)
#pragma unroll 1
      for (int c = max(c0, 32 * w); c < min(c1, 32 * w + 32); ++c)
        if ((*reinterpret_cast<const uint16_t*>(row + c) & 0x7f80u) == 0x7f80u)
          bad[w] |= 1u << (c - 32 * w);
  }
  auto any = [&] { return (bad[0] | bad[1] | bad[2] | bad[3]) != 0u; };
  const int from = __reduce_min_sync(0xffffffffu, any() ? first : INT32_MAX);
  const int to = __reduce_max_sync(0xffffffffu, any() ? end : 0);
  // a lane takes eight columns of one of `at_once` keys
  const int pieces = a.d / 8, at_once = 32 / pieces, key = lane / pieces;
  const bf16* const piece = x.p + g * x.hs + 8 * (lane % pieces);
  for (int64_t j0 = from; j0 < to && __any_sync(0xffffffffu, any()); j0 += 4 * at_once) {
    Eight e[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int64_t j = j0 + u * at_once + key;
      e[u].a = make_uint4(0u, 0u, 0u, 0u);
      if (key < at_once && j < to) e[u].load(piece + j * x.ts);
    }
    bool some = false;
#pragma unroll
    for (int u = 0; u < 4; ++u)
      some |= bad_pair(e[u].a.x) || bad_pair(e[u].a.y) || bad_pair(e[u].a.z) || bad_pair(e[u].a.w);
    if (!__any_sync(0xffffffffu, some)) continue;
    const int64_t j1 = min(j0 + 4 * at_once, static_cast<int64_t>(to));
    for (int64_t j = j0; j < j1; ++j)
#pragma unroll
      for (int w = 0; w < kMaxDim / 32; ++w) {
        const int c = 32 * w + lane;
        const uint32_t v = c < a.d ? *reinterpret_cast<const uint16_t*>(x.at(j, g) + c) : 0u;
        const uint32_t which = __ballot_sync(0xffffffffu, (v & 0x7f80u) == 0x7f80u);
        if (first <= j && j < end) bad[w] &= ~which;
      }
  }
  return __ballot_sync(0xffffffffu, any());
}

// The rows of o that a warp has found not finite (query t and head h of each lane,
// t = -1: none), all of key head g, computed again unless they are so by right.
__device__ __noinline__ static void forward_again(const SpanArgs& a, int g, int t, int h) {
  __syncwarp();  // other lanes stored parts of these rows
  int first = 0, end = 0;
  if (t >= 0) a.span(t, first, end);
  for (unsigned again = bad_rows(a, a.v, g, t >= 0 ? a.o.at(t, h) : nullptr, 0, a.d, first, end);
       again; again &= again - 1) {
    const int from = __ffs(again) - 1;
    row_forward(a, __shfl_sync(0xffffffffu, t, from), __shfl_sync(0xffffffffu, h, from), 0, a.d,
                false);
  }
}

// ------------------------------------------------- tiles of the tensor-core kernels
// A tile of 128 rows is 128 / rep neighbouring queries times the rep query
// heads that share a key head, query by query (rep = 3: 126 rows are used).
// So a key head's tile serves all its query heads, few queries fill a tile
// better, and a tile's queries are fewer, which keeps the union of their spans
// short.
struct Tiling {
  int per;    // queries of a tile
  int tiles;  // tiles of all queries
  __host__ __device__ static Tiling of(int queries, int rep) {
    Tiling t;
    t.per = 128 / rep;
    t.tiles = (queries + t.per - 1) / t.per;
    return t;
  }
};

// Least first key and largest end over each of two tiles' queries, the first
// at t0; 0, 0 where they see nothing. Whole warp.
__device__ __forceinline__ void spans_of_tiles(const SpanArgs& a, const Tiling& tl, int t0,
                                               int (&first)[2], int (&end)[2]) {
  int lo[2] = {INT32_MAX, INT32_MAX}, hi[2] = {0, 0};
  const int n = min(2 * tl.per, a.queries - t0);
#pragma unroll 4
  for (int i = threadIdx.x & 31; i < n; i += 32) {
    int x, y;
    a.span(t0 + i, x, y);
    if (x >= y) continue;
    if (i < tl.per) {
      lo[0] = min(lo[0], x);
      hi[0] = max(hi[0], y);
    } else {
      lo[1] = min(lo[1], x);
      hi[1] = max(hi[1], y);
    }
  }
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    lo[x] = __reduce_min_sync(0xffffffffu, lo[x]);
    hi[x] = __reduce_max_sync(0xffffffffu, hi[x]);
    first[x] = lo[x] < hi[x] ? lo[x] : 0;
    end[x] = lo[x] < hi[x] ? hi[x] : 0;
  }
}

// The cap cap tanh(s scale / cap), in base 2 where scores are exponentiated.
// Arguments of tanh within 0.35 (scores below 0.35 of the cap, nearly all in use)
// go through an odd polynomial (least squares on [0, 0.35], reweighted towards
// the least greatest error: 2^-27.3; with one term less, 2^-22 of a cap of 50
// showed in the log-sum-exp), whose coefficients take up the scale; others
// through the library's tanh.
struct Cap {
  float limit;    // scores beyond it: not the polynomial
  float w;        // scale / cap
  float t[4];     // tanh(w s) = s (t0 + t1 s^2 + ..)
  float z[4];     // cap log2 e tanh(w s), alike
};
inline Cap cap_of(float scale, float cap) {
  constexpr double c[4] = {0.999999848, -0.33331657, 0.132833236, -0.0483769203};
  Cap x = {};
  if (!(cap > 0.f)) return x;
  const double w = static_cast<double>(scale) / cap;
  x.w = static_cast<float>(w);
  x.limit = static_cast<float>(0.35 / w);
  double p = w;
  for (int i = 0; i < 4; ++i, p *= w * w) {
    x.t[i] = static_cast<float>(c[i] * p);
    x.z[i] = static_cast<float>(cap * 1.4426950408889634 * c[i] * p);
  }
  return x;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
// How far a row's scores reach.
struct Reach {
  float hi[2] = {-INFINITY, -INFINITY}, lo[2] = {INFINITY, INFINITY};
  template <bool DOWN>
  __device__ __forceinline__ void take(float2 s, int e) {
    hi[e] = max3(hi[e], s.x, s.y);
    if (DOWN) lo[e] = min3(lo[e], s.x, s.y);
  }
  __device__ __forceinline__ float top() const { return fmaxf(hi[0], hi[1]); }
  // Whether some lane of the warp has a score beyond the polynomial's range.
  __device__ __forceinline__ bool beyond(float limit) const {
    return __any_sync(0xffffffffu, fmaxf(top(), -fminf(lo[0], lo[1])) > limit);
  }
};
// t0 + t1 s^2 + .. of two scores.
__device__ __forceinline__ float2 odd_factor(float2 s, const float (&t)[4]) {
  const float2 y = mul2(s, s);
  float2 p = fma2(y, both(t[3]), both(t[2]));
  p = fma2(p, y, both(t[1]));
  return fma2(p, y, both(t[0]));
}

// Bits c of a word with lo <= c < hi.
__device__ __forceinline__ uint32_t bits_between(int lo, int hi) {
  const uint32_t below_hi = hi >= 32 ? ~0u : hi <= 0 ? 0u : (1u << hi) - 1u;
  const uint32_t below_lo = lo >= 32 ? ~0u : lo <= 0 ? 0u : (1u << lo) - 1u;
  return below_hi & ~below_lo;
}

// ------------------------------------------------- what nobody sees
// What lies beside the keys that are seen (the end of a cache, the rows behind a
// batch's last token) may be memory that nobody wrote. Where it is NaN or infinite,
// 0 times it reaches sums over keys. So a CTA goes through its items in rounds of at
// most kRound: where some came out not finite, the round after takes those once more
// (`kSecond` in their number), with the keys that none of an item's rows sees cleared
// in shared memory, and only what is not finite then is computed again row by row.
// Others pay for one look at a word of shared memory.
constexpr int kRound = 64, kSecond = 1 << 30;
struct Rounds {
  unsigned long long redo;  // the round's items that are to be taken once more, a bit each
  int left;                 // there are items behind the round's
  int lost;                 // a wait has given up: no more rounds
  uint32_t start;           // items before the round
};
// Says so of item `it`, counted over all rounds. One lane of a warp.
__device__ __forceinline__ void take_again(Rounds* r, uint32_t it) {
  atomicOr(&r->redo, 1ull << (it - *reinterpret_cast<volatile uint32_t*>(&r->start)));
}
// A round's end: whether there is another, and the items it takes once more, if any.
// All threads of the CTA, in whole warps, of which thread 0 belongs to the one that hands
// out the items; waits for all of them. Not behind a __syncwarp() of the warps of rows,
// whose loops leave as whole warps: with it heads of 64 took 194 us in place of 179 (8192
// causal tokens, 16 heads).
template <bool MORE>
__device__ __forceinline__ bool next_round(Rounds* r, int threads, unsigned long long& redo) {
  named_bar_sync(1, threads);
  if (!MORE) return false;
  volatile Rounds* v = r;
  redo = v->redo;
  if ((redo == 0ull && v->left == 0) || v->lost) return false;
  named_bar_sync(1, threads);
  if (threadIdx.x == 0) v->redo = 0ull;
  return true;
}

// Clears the rows 32 w + i of a tile of 128 rows (chunks of 64 columns, 128 bytes a row,
// one behind the other) that have a bit i in `which`. Whole warp.
__device__ __forceinline__ void clear_rows(uint8_t* tile, int d, int w, uint32_t which) {
  const int lane = threadIdx.x & 31;
  uint8_t* const at = tile + (lane >> 3) * (128 * 128) + 16 * (lane & 7) + 32 * w * 128;
  const bool has = 64 * (lane >> 3) < d;
#pragma unroll 1
  for (; which; which &= which - 1)
    if (has)
      *reinterpret_cast<uint4*>(at + (__ffs(which) - 1) * 128) = make_uint4(0u, 0u, 0u, 0u);
}
// What a warp has cleared, where the tensor cores see it once `bar` has been arrived on.
__device__ __forceinline__ void hand_over(uint32_t bar) {
  fence_proxy_async_smem();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}
// Waits for a tile of 128 keys from `base` on and clears the rows that none of the `n`
// queries from t0 on sees; then arrives on `full`. Whole warp.
__device__ __forceinline__ bool clear_unseen(const SpanArgs& a, int t0, int n, int base,
                                             uint8_t* tile, uint32_t raw, uint32_t parity,
                                             uint32_t full, const Patience& err) {
  if (!warp_wait(raw, parity, err)) return false;
#pragma unroll 1
  for (int w = 0; w < 4; ++w) {
    uint32_t seen = 0u;
#pragma unroll 1
    for (int i = threadIdx.x & 31; i < n; i += 32) {
      int x, y;
      a.span(t0 + i, x, y);
      if (x < y) seen |= bits_between(x - base - 32 * w, y - base - 32 * w);
    }
    clear_rows(tile, a.d, w, ~__reduce_or_sync(0xffffffffu, seen));
  }
  hand_over(full);
  return true;
}

// Splits of the keys of one (pair of tiles, key head), and the forward pass'
// workspace. Few queries: their keys are spread over the SMs, each part gives
// a partial result, and a second kernel joins them.
int forward_splits(int queries, int keys, int nkv, int rep);
size_t forward_workspace(int queries, int keys, int nh, int nkv, int d);
cudaError_t forward_tiles(const SpanArgs& a, void* ws, cudaStream_t s);

size_t backward_workspace(int queries, int keys, int nh, int nkv, int d);
cudaError_t backward_tiles(const SpanArgs& a, void* ws, cudaStream_t s);

}  // namespace rdt
