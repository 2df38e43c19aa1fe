// Backward pass of the attention over spans of keys on the 5th-generation
// tensor cores, in three kernels without atomic sums, so that results do not
// depend on scheduling:
//  * prepare: D = d_o . o - d_lse and the base-2 log-sum-exp of every row, tile
//    by tile (spans.cuh), both negated; the spans of tiles and of groups of 32
//    tiles, by which the others find what meets what;
//  * dK/dV: a CTA takes (128 keys, key head) items and walks the row tiles that
//    see any of the keys. S^T = K Q^T, P^T, dV += P^T dO; dP^T = V dO^T,
//    dS^T = P^T o (dP^T - D) slope, dK += dS^T Q. P^T and dS^T are written over
//    their scores in TMEM as bf16 and read from there; dK and dV stay in TMEM;
//  * dQ: a CTA takes (row tile, key head) items; S and dP once more,
//    dQ += dS K.
// In both, warp 0 loads by TMA, warp 1 issues the MMAs, and warps 4-19 do the
// elementwise work: TMEM lanes 32 (w mod 4) on, columns 32 (w / 4 - 1) on.
//
// A NaN or infinity where a query does not see a key, times 0, would reach sums. Rows of
// queries that see nothing may be memory that nobody wrote: before and behind a batch
// dK/dV clears them in shared memory (warp 2); dQ takes items once more that came out
// not finite, with the keys cleared that none of their rows sees (spans.cuh). 4096
// packed tokens of which the unused end is NaN: 171 us, without 143. Other rows of dq,
// dk and dv that are not finite are computed again one by one (row_dq, row_dkdv). Not
// where they see a query (dq: in the columns of a key) that is not finite itself: what
// they hold is so by right, and a batch that has diverged throughout costs no more than
// another.
//
// Seven products are formed where five would do: dQ summed beside dK and dV needs
// atomics, whose order changes bits, or key tiles in a fixed order. Bound by the
// products where many tiles are seen whole: 8192 tokens of 32 / 8 heads of 128, a
// quarter of them a prefix, 1189 us (651 dK/dV, 510 dQ), 0.96 and 0.92 of 1890
// TFLOP/s for the four and the three products they form; back to back 1261, by the
// power limit. 4096 tokens in documents up to 1024: 124 us, of them 17 prepare (67
// MB), 58 dK/dV, 50 dQ; bound by the starts and ends of short items.
#include <algorithm>

#include "spans.cuh"

namespace rdt {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kThreads = 640, kEltThreads = 512;
constexpr int kGroup = 32;  // row tiles of a group
constexpr float kNoRow = -1e30f;  // negated lse of a row that sees nothing: p = 0; with D = 0

// Spans of a row tile: keys any of its rows sees, keys all of them see. Rows
// that see nothing (or are none) are left out of both: their p is 0 unmasked.
struct TileSpan {
  int first, end;          // any
  // all; ~all_first where the first or the last query sees nothing, as before and behind a
  // batch: then Q and dO are cleared of such rows before they are multiplied. Queries
  // that see nothing in between are not looked for: that way 8192 tokens of which every
  // 17th sees nothing take 1429 us and not 1157.
  int all_first, all_end;
};

struct Args {
  SpanArgs a;
  Tiling tl;
  int groups;
  Cap cap;
  float scale_log2;
  float *neg_lse, *neg_d;  // [nkv][tiles][128]
  int *lo, *len;           // [tiles][128]
  TileSpan* tiles;
  int2* group;  // first, end
  int64_t key_tiles;  // of all key heads
  int parts;          // items of a key tile
  float4* part;       // parts = 2: sums of each half
  int* arrived;       // and how many of a key tile's are there
  Patience err_rows, err_keys;  // where row tiles are walked through, where key tiles are
  bool wide_dq, wide_dk, wide_dv;  // rows at multiples of 32 bytes
};

// ---------------------------------------------------------------- prepare
constexpr int kPrepThreads = 256;

// Blocks [0, groups) find the groups' spans, the others the tiles' and the rows'
// D and lse.
__global__ void __launch_bounds__(kPrepThreads, 4) prepare_kernel(const __grid_constant__ Args ar) {
  const SpanArgs& a = ar.a;
  __shared__ TileSpan found[kPrepThreads / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  after_previous_kernel();
  // the warps' spans together: whole block
  auto joined = [&](TileSpan s) {
    s.first = __reduce_min_sync(0xffffffffu, s.first);
    s.end = __reduce_max_sync(0xffffffffu, s.end);
    s.all_first = __reduce_max_sync(0xffffffffu, s.all_first);
    s.all_end = __reduce_min_sync(0xffffffffu, s.all_end);
    if (lane == 0) found[warp] = s;
    __syncthreads();
    for (int w = 0; w < kPrepThreads / 32; ++w) {
      s.first = min(s.first, found[w].first);
      s.end = max(s.end, found[w].end);
      s.all_first = max(s.all_first, found[w].all_first);
      s.all_end = min(s.all_end, found[w].all_end);
    }
    __syncthreads();
    if (s.first >= s.end) s.first = s.end = 0;
    return s;
  };
  auto take = [](TileSpan& s, int x, int y) {
    s.first = min(s.first, x);
    s.end = max(s.end, y);
    s.all_first = max(s.all_first, x);
    s.all_end = min(s.all_end, y);
  };
  const TileSpan none = {INT32_MAX, 0, 0, INT32_MAX};
  if (static_cast<int>(blockIdx.x) < ar.groups) {
    if (ar.parts > 1)
      for (int i = blockIdx.x * kPrepThreads + threadIdx.x; i < ar.key_tiles;
           i += ar.groups * kPrepThreads)
        ar.arrived[i] = 0;
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kGroup * ar.tl.per;
    const int64_t t1 = min(t0 + kGroup * ar.tl.per, static_cast<int64_t>(a.queries));
    TileSpan s = none;
#pragma unroll 4
    for (int64_t t = t0 + threadIdx.x; t < t1; t += kPrepThreads) {
      int x, y;
      a.span(static_cast<int>(t), x, y);
      if (x < y) take(s, x, y);
    }
    s = joined(s);
    if (threadIdx.x == 0) ar.group[blockIdx.x] = make_int2(s.first, s.end);
    return;
  }
  // a row is `lanes` lanes of eight columns; a CTA takes a key head's row tile at
  // a time, its warps 16 rows each
  int log2 = 1;
  while ((8 << log2) < a.d) ++log2;
  const int lanes = 1 << log2, per_warp = 32 >> log2, c = 8 * (lane & (lanes - 1));
  const uint32_t inv_rep = (65536u + a.rep - 1) / a.rep;  // row / rep of rows below 128
  const int units = a.nkv * ar.tl.tiles, ctas = gridDim.x - ar.groups;
  for (int unit = blockIdx.x - ar.groups; unit < units; unit += ctas) {
    const int g = unit / ar.tl.tiles, tile = unit - g * ar.tl.tiles;
    if (g == 0) {
      const int row = threadIdx.x;
      TileSpan s = none;
      bool blind = false;
      if (row < 128) {
        const int in = static_cast<int>(row * inv_rep >> 16), t = tile * ar.tl.per + in;
        int x = 0, y = 0;
        if (in < ar.tl.per && t < a.queries) {
          a.span(t, x, y);
          blind = x >= y && (in == 0 || in == ar.tl.per - 1 || t == a.queries - 1);
        }
        if (x < y)
          take(s, x, y);
        else
          x = y = 0;
        ar.lo[tile * int64_t{128} + row] = x;
        ar.len[tile * int64_t{128} + row] = y - x;
      }
      s = joined(s);
      if (__syncthreads_or(blind)) s.all_first = ~s.all_first;
      if (row == 0) ar.tiles[tile] = s;
    }
    // the row that this lane finishes
    const int done = 16 * warp + (lane & 15);
    const int done_in = static_cast<int>(done * inv_rep >> 16), done_t = tile * ar.tl.per + done_in;
    float lse = 0.f, d_lse = 0.f;
    bool sees = false;
    if (done_in < ar.tl.per && done_t < a.queries) {
      const int64_t th = static_cast<int64_t>(done_t) * a.nh + g * a.rep + done - done_in * a.rep;
      int x, y;
      a.span(done_t, x, y);
      sees = x < y;
      lse = a.lse[th];
      if (a.d_lse) d_lse = a.d_lse[th];
    }
    // this lane's part of each of the warp's rows, the loads of four rows at a time
    float part[8] = {};
#pragma unroll
    for (int b0 = 0; b0 < 8; b0 += 4) {
      if (b0 * per_warp >= 16) break;
      Eight x[4], y[4];
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const int row = 16 * warp + (b0 + b) * per_warp + (lane >> log2);
        const int in = static_cast<int>(row * inv_rep >> 16), t = tile * ar.tl.per + in;
        const int h = g * a.rep + row - in * a.rep;
        x[b].a = y[b].a = make_uint4(0u, 0u, 0u, 0u);
        if ((b0 + b) * per_warp < 16 && in < ar.tl.per && t < a.queries && c < a.d) {
          x[b].load(a.d_o.at(t, h) + c);
          y[b].load(a.o.at(t, h) + c);
        }
      }
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        float u[8], v[8];
        x[b].get(u);
        y[b].get(v);
#pragma unroll
        for (int i = 0; i < 8; ++i) part[b0 + b] = fmaf(u[i], v[i], part[b0 + b]);
      }
    }
    // the rows' sums, each to the lane that finishes its row
    float own = 0.f;
#pragma unroll
    for (int b = 0; b < 8; ++b) {
      if (b * per_warp >= 16) break;
      float sum = part[b];
      for (int o = lanes >> 1; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      sum = __shfl_sync(0xffffffffu, sum, (lane & (per_warp - 1)) << log2);
      if (lane / per_warp == b) own = sum;
    }
    if (lane < 16) {
      const int64_t at = (static_cast<int64_t>(g) * ar.tl.tiles + tile) * 128 + done;
      ar.neg_lse[at] = sees ? -lse * kLog2e : kNoRow;
      ar.neg_d[at] = sees ? d_lse - own : 0.f;
    }
  }
}

// ------------------------------------------------------------ elementwise
// Scores sv of 32 columns to p = 2^(score + neg_lse(c)) times the slope of their cap,
// c a multiple of two; put(c, p) takes what p of c and c + 1 were. tanh and its slope
// 1 - tanh^2 by the cap's polynomial; past it, u = 2 / (1 + e^2x), tanh = 1 - u and the
// slope u (2 - u), which loses nothing where tanh is close to 1 (1 - tanh^2 is off by half
// of itself at x = 8).
template <bool CAP, typename N, typename P>
__device__ __forceinline__ void weights(uint32_t (&sv)[32], const Args& ar, N neg_lse, P put) {
  auto of = [&](int c) {
    return make_float2(__uint_as_float(sv[c]), __uint_as_float(sv[c + 1]));
  };
  auto leave = [&](int c, float2 s, float2 slope) {
    float2 p = fma2(s, make_float2(ar.scale_log2, ar.scale_log2), neg_lse(c));
    p.x = ex2_approx(p.x);
    p.y = ex2_approx(p.y);
    put(c, p);
    if constexpr (CAP) p = mul2(p, slope);
    sv[c] = __float_as_uint(p.x);
    sv[c + 1] = __float_as_uint(p.y);
  };
  auto slope_of = [](float2 t) {
    return fma2(make_float2(-t.x, -t.y), t, make_float2(1.f, 1.f));
  };
  if constexpr (CAP) {
    const Cap& cap = ar.cap;
    Reach reach;
#pragma unroll
    for (int c = 0; c < 32; c += 2) reach.take<true>(of(c), (c >> 1) & 1);
    if (reach.beyond(cap.limit)) {
#pragma unroll
      for (int c = 0; c < 32; c += 2) {  // a score by itself decides, not what its warp holds
        const float2 s = of(c);
        float2 t = mul2(s, odd_factor(s, cap.t)), slope = slope_of(t);
        auto far = [&](float x, float& tanh, float& its) {  // without a branch
          const float u = __fdividef(2.f, 1.f + ex2_approx(2.f * kLog2e * cap.w * fabsf(x)));
          const bool past = fabsf(x) > cap.limit;
          tanh = past ? copysignf(1.f - u, x) : tanh;
          its = past ? fmaf(-u, u, 2.f * u) : its;
        };
        far(s.x, t.x, slope.x);
        far(s.y, t.y, slope.y);
        leave(c, t, slope);
      }
      return;
    }
#pragma unroll
    for (int c = 0; c < 32; c += 2) {
      const float2 s = of(c), t = mul2(s, odd_factor(s, cap.t));
      leave(c, t, slope_of(t));
    }
  } else {
#pragma unroll
    for (int c = 0; c < 32; c += 2) leave(c, of(c), both(1.f));
  }
}

// 32 bf16 values of which those with a bit in `seen` stay, whatever the others hold.
__device__ __forceinline__ void clear_unseen(uint32_t (&pk)[16], uint32_t seen) {
#pragma unroll
  for (int c = 0; c < 32; c += 2)
    pk[c / 2] &= (seen & (1u << c) ? 0xffffu : 0u) | (seen & (2u << c) ? 0xffff0000u : 0u);
}

// 32 columns of a row, bf16, of which `left` (a multiple of 16) exist; in pieces
// of 32 bytes where the tensor's rows allow it.
__device__ __forceinline__ void put_columns(bf16* dst, const uint32_t (&r)[32], float w, int left,
                                            bool wide) {
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    if (16 * e >= left) break;
    uint32_t v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      v[i] = pack_bf16x2(__uint_as_float(r[16 * e + 2 * i]) * w,
                         __uint_as_float(r[16 * e + 2 * i + 1]) * w);
    if (wide) {
      store32(dst + 16 * e, v);
    } else {
      reinterpret_cast<uint4*>(dst)[2 * e] = make_uint4(v[0], v[1], v[2], v[3]);
      reinterpret_cast<uint4*>(dst)[2 * e + 1] = make_uint4(v[4], v[5], v[6], v[7]);
    }
  }
}
__device__ __forceinline__ bool all_finite(const uint32_t (&r)[32], int left) {
  float bad = 0.f;
#pragma unroll
  for (int e = 0; e < 32; ++e)
    if (e < left) bad = fmaf(__uint_as_float(r[e]), 0.f, bad);
  return bad == 0.f;
}

__device__ __forceinline__ bool finite_row(float neg_lse, float neg_d) {
  return fabsf(neg_lse) < INFINITY && fabsf(neg_d) < INFINITY;
}

// Whether some query that sees key j has a row (of key head g's) that is not finite. Whole warp.
__device__ __noinline__ bool sees_nonfinite(const Args& ar, int j, int g) {
  const SpanArgs& a = ar.a;
  for (int64_t base = 0; base < a.queries; base += 32) {
    const int64_t t = base + (threadIdx.x & 31);
    bool bad = false;
    if (t < a.queries) {
      int first, end;
      a.span(static_cast<int>(t), first, end);
      if (first <= j && j < end) {
        const int tile = static_cast<int>(t / ar.tl.per), in = static_cast<int>(t % ar.tl.per);
        const int64_t at = (static_cast<int64_t>(g) * ar.tl.tiles + tile) * 128 + in * a.rep;
        for (int r = 0; r < a.rep; ++r) bad |= !finite_row(ar.neg_lse[at + r], ar.neg_d[at + r]);
      }
    }
    if (__any_sync(0xffffffffu, bad)) return true;
  }
  return false;
}

__device__ __forceinline__ void settle(int* err) {
  if (err && *reinterpret_cast<volatile int*>(err) != 0) {
    // after a timed-out wait, copies issued just before may still be landing
    // in this CTA's shared memory: let them finish before it exits
    const uint64_t w0 = global_timer_ns();
    while (global_timer_ns() - w0 < 200000ull) {
    }
  }
}

// ------------------------------------------------------------------ dK, dV
// What the loading warp says of a step: a row tile, or the end of an item.
struct Meta {
  int tile;  // row tile; kEnd: the item's tiles are through; kStop: all items are
  int full;  // bits kFull: every row that sees anything sees all of the item's keys; kBlind: rows
             // that see nothing are to be cleared; with kEnd, how to end
  int n0, g; // the item's first key and key head
};
constexpr int kEnd = -1, kStop = -2, kFull = 1, kBlind = 2;
constexpr int kNothing = 0, kAlone = 1, kShared = 2;  // ways to end; the second half: kShared + 1

template <int D>
struct KvCfg {
  static constexpr uint32_t CHUNK = 128 * 128, TILE = 128 * D * 2;
  // Stages: Q is read by S and, an elementwise pass later, by dK; its copies take
  // longer than that pass, so it has one stage more than dO where memory is short:
  // with two, dK waited for Q for 540 cycles of each row tile; with three one takes
  // 2900, of them 2790 its products.
  static constexpr int QST = D == 128 ? 3 : 4, OST = D == 128 ? 2 : 4, IST = 2;
  static constexpr uint32_t OFF_K = 0, OFF_V = TILE, OFF_Q = 2 * TILE, OFF_DO = OFF_Q + QST * TILE,
                            OFF_ROW = OFF_DO + OST * TILE,  // [IST][neg_lse, neg_d][128]
      OFF_META = OFF_ROW + IST * 1024, OFF_NEXT = OFF_META + IST * sizeof(Meta),
                            OFF_BAR = OFF_NEXT + 16;
  static constexpr size_t SMEM = OFF_BAR + 336;  // at a multiple of 1024, which is checked
  static constexpr uint32_t T_DK = 0, T_DV = 128, T_S = 256, T_DP = 384, TMEM_COLS = 512;
  static_assert(SMEM <= 232448 && OFF_NEXT % 16 == 0, "");
};

// TMEM column, relative to a block of 128, of the packed bf16 A operand for K
// step kk (16 rows): 32 columns' pairs lie in the first 16 of their place.
__device__ __forceinline__ uint32_t packed_col(int kk) { return (kk >> 1) * 32 + (kk & 1) * 8; }

// An item is a key tile of a key head, or (parts = 2) one of two halves of it.
// Where a key tile is seen by fewer than kShareFrom row tiles (45 us of work) its
// first half takes them all; else each takes every second, leaves its sums in
// the workspace, and the one that is done last adds the two (in either order
// the same). 4096 packed tokens, 32 / 8 heads of 128: 133 us in all from 32 row
// tiles on, 141 from 24, 145 from 8, 151 without halves. One CTA of the grid an
// item, taken as CTAs get free, as in the forward pass.
constexpr int kShareFrom = 32;

template <int D, bool CAP>
__global__ void __launch_bounds__(kThreads, 1)
    spans_dkdv_kernel(const __grid_constant__ CUtensorMap tq,
                      const __grid_constant__ CUtensorMap tdo,
                      const __grid_constant__ CUtensorMap tk,
                      const __grid_constant__ CUtensorMap tv, const __grid_constant__ Args ar) {
  using C = KvCfg<D>;
  constexpr uint32_t QST = C::QST, OST = C::OST, IST = C::IST;
  const SpanArgs& a = ar.a;
  const Patience& err = ar.err_rows;
  extern __shared__ __align__(1024) uint8_t smem_tiles[];
  uint8_t* smem = smem_tiles;
  const uint32_t sbase = smem_u32(smem);
  if (sbase & 1023u) {  // the swizzled tiles' layout counts on it
    record_error(err.err, kErrTimeout);
    return;
  }
  const uint32_t bar0 = sbase + C::OFF_BAR;
  const uint32_t kv_full = bar0, kv_empty = bar0 + 8, q_full = bar0 + 16,
                 q_empty = q_full + 8 * QST, o_full = q_empty + 8 * QST, o_empty = o_full + 8 * OST,
                 i_full = o_empty + 8 * OST, i_empty = i_full + 8 * IST, s_full = i_empty + 8 * IST,
                 dp_full = s_full + 8, p_ready = dp_full + 8, ds_ready = p_ready + 8,
                 fin = ds_ready + 8, acc_free = fin + 8, next = acc_free + 8, left_it = next + 8,
                 decided = left_it + 8, drain = decided + 8,
                 // come, but with rows to be cleared; by their order
      q_raw = drain + 8, o_raw = q_raw + 8 * QST;
  static_assert(8 * (3 * (QST + OST) + 2 * IST + 12) <= 328, "");
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_BAR + 328);
  volatile int* decision = reinterpret_cast<volatile int*>(smem + C::OFF_BAR + 332);
  Meta* meta = reinterpret_cast<Meta*>(smem + C::OFF_META);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int chunks = (a.d + 63) / 64, used = ar.tl.per * a.rep;

  if (threadIdx.x == 0) {
    mbar_init(kv_full, 1);
    mbar_init(kv_empty, 1);
    for (uint32_t x = 0; x < QST; ++x) {
      mbar_init(q_full + 8 * x, 1);
      mbar_init(q_empty + 8 * x, 1);
      mbar_init(q_raw + 8 * x, 1);
    }
    for (uint32_t x = 0; x < OST; ++x) {
      mbar_init(o_full + 8 * x, 1);
      mbar_init(o_empty + 8 * x, 1);
      mbar_init(o_raw + 8 * x, 1);
    }
    for (uint32_t x = 0; x < IST; ++x) {
      mbar_init(i_full + 8 * x, 1);
      // the MMA thread, the clearing warp, the elementwise warps
      mbar_init(i_empty + 8 * x, 2 + kEltThreads / 32);
    }
    mbar_init(s_full, 1);
    mbar_init(dp_full, 1);
    mbar_init(p_ready, kEltThreads);
    mbar_init(ds_ready, kEltThreads);
    mbar_init(fin, 1);
    mbar_init(acc_free, kEltThreads);
    mbar_init(next, 1);
    mbar_init(left_it, kEltThreads);
    mbar_init(decided, 1);
    mbar_init(drain, 1);
    fence_mbar_init();
    tma_prefetch_desc(&tq);
    tma_prefetch_desc(&tdo);
    tma_prefetch_desc(&tk);
    tma_prefetch_desc(&tv);
  }
  if (used < 128) {
    // rows past a tile's last are never loaded, and p = 0 does not clear a NaN
    const int words = (128 - used) * 32;
    for (int i = threadIdx.x; i < static_cast<int>(QST + OST) * chunks * words; i += kThreads) {
      const int w = i % words, block = i / words;
      const uint32_t base = C::OFF_Q + (block / chunks) * C::TILE + (block % chunks) * C::CHUNK;
      *reinterpret_cast<uint32_t*>(smem + base + used * 128 + 4 * w) = 0u;
    }
    fence_proxy_async_smem();
  }
  if (warp == 1) tmem_alloc(smem_u32(tmem_slot), C::TMEM_COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  after_previous_kernel();

  if (warp < 4) regs_dec<56>();
  if (warp == 0) {
    // --------------------------------------------------------- producer
    bool ok = true;
    uint32_t r = 0, tiles = 0, loaded = 0;  // steps, row tiles, items with any so far
    uint32_t raws = 0;                      // row tiles with rows to be cleared
    int item = blockIdx.x;
    for (uint32_t it = 0; ok && item >= 0; ++it) {
      const int half = item % ar.parts, x = item / ar.parts;
      const int g = x % a.nkv, n0 = x / a.nkv * 128, n1 = min(n0 + 128, a.keys);
      // calls f(tile, bits) for the row tiles that see any of the keys, until it is false
      auto each = [&](auto f) {
        bool on = true;
        for (int g0 = 0; g0 < ar.groups && on; g0 += 32) {
          const int2 span = g0 + lane < ar.groups ? ar.group[g0 + lane] : make_int2(0, 0);
          unsigned some = __ballot_sync(0xffffffffu, span.x < n1 && span.y > n0);
          for (; some && on; some &= some - 1) {
            const int first = (g0 + __ffs(some) - 1) * kGroup, tile = first + lane;
            TileSpan s = {0, 0, 0, 0};
            if (tile < ar.tl.tiles) s = ar.tiles[tile];
            unsigned meets = __ballot_sync(0xffffffffu, s.first < n1 && s.end > n0);
            const unsigned blind = __ballot_sync(0xffffffffu, s.all_first < 0);
            const unsigned full = __ballot_sync(
                0xffffffffu, (s.all_first ^ (s.all_first >> 31)) <= n0 && s.all_end >= n1);
            for (; meets && on; meets &= meets - 1) {
              const int i = __ffs(meets) - 1;
              on = f(first + i, (full >> i & 1 ? kFull : 0) | (blind >> i & 1 ? kBlind : 0));
            }
          }
        }
      };
      bool shared = false;
      if (ar.parts > 1) {
        int count = 0;
        each([&](int, int) { return ++count < kShareFrom; });
        shared = count >= kShareFrom;
      }
      const bool mine = shared || half == 0;
      bool some = false;  // K and V are under way
      int met = 0;
      auto send = [&](int tile, int full) {
        const bool blind = tile >= 0 && (full & kBlind);
        if (lane == 0) {
          if (tile >= 0) {
            // QST blind tiles later this one's stage is free again: it is cleared by then
            const uint32_t sq = tiles % QST, q = sbase + C::OFF_Q + sq * C::TILE,
                           bar = blind ? q_raw + 8 * (raws % QST) : q_full + 8 * sq;
            ok = wait_for(q_empty + 8 * sq, ((tiles / QST) & 1) ^ 1, err);
            if (ok) {
              mbar_arrive_expect_tx(bar, chunks * used * 128);
              for (int c = 0; c < chunks; ++c)
                tma_load_3d(q + c * C::CHUNK, &tq, bar, c * 64, g * a.rep, tile * ar.tl.per);
            }
            if (ok && !some) ok = wait_for(kv_empty, (loaded & 1) ^ 1, err);
            if (ok && !some) {
              mbar_arrive_expect_tx(kv_full, 2 * chunks * C::CHUNK);
              for (int c = 0; c < chunks; ++c) {
                tma_load_3d(sbase + C::OFF_K + c * C::CHUNK, &tk, kv_full, c * 64, g, n0);
                tma_load_3d(sbase + C::OFF_V + c * C::CHUNK, &tv, kv_full, c * 64, g, n0);
              }
            }
          }
          const uint32_t si = r % IST, row = sbase + C::OFF_ROW + si * 1024;
          ok = ok && wait_for(i_empty + 8 * si, ((r / IST) & 1) ^ 1, err);
          if (ok) {
            meta[si] = Meta{tile, full, n0, g};
            if (tile < 0) {
              mbar_arrive(i_full + 8 * si);
            } else {
              const int64_t at = (static_cast<int64_t>(g) * ar.tl.tiles + tile) * 128;
              mbar_arrive_expect_tx(i_full + 8 * si, 1024);
              bulk_load_1d(row, ar.neg_lse + at, 512, i_full + 8 * si);
              bulk_load_1d(row + 512, ar.neg_d + at, 512, i_full + 8 * si);
              const uint32_t so = tiles % OST, o = sbase + C::OFF_DO + so * C::TILE,
                             bar = blind ? o_raw + 8 * (raws % OST) : o_full + 8 * so;
              ok = wait_for(o_empty + 8 * so, ((tiles / OST) & 1) ^ 1, err);
              if (ok) {
                mbar_arrive_expect_tx(bar, chunks * used * 128);
                for (int c = 0; c < chunks; ++c)
                  tma_load_3d(o + c * C::CHUNK, &tdo, bar, c * 64, g * a.rep, tile * ar.tl.per);
              }
            }
          }
        }
        ok = __shfl_sync(0xffffffffu, static_cast<int>(ok), 0);
        raws += blind;
        ++r;
        if (tile >= 0) {
          ++tiles;
          some = true;
        }
      };
      if (mine)
        each([&](int tile, int full) {
          if (!shared || (met++ & 1) == half) send(tile, full);
          return ok;
        });
      if (some) ++loaded;
      // asked for now, not before: an item that waits here could have been another SM's
      if (lane == 0) next_cta_request(sbase + C::OFF_NEXT, next);
      if (ok) send(kEnd, shared ? kShared + half : mine ? kAlone : kNothing);
      // waited for on the way out too: the answer is written to this CTA's memory
      const bool answered = warp_wait(next, it & 1, err);
      ok = ok && answered;
      if (ok) item = next_cta_answer(sbase + C::OFF_NEXT);
      if (ok && item < 0) send(kStop, 0);
    }
  } else if (warp == 1) {
    if (elect_one()) {
      // -------------------------------------------------------------- MMA
      constexpr uint32_t id_s = idesc_bf16_f32(128, 128, 0, 0);
      const uint32_t id_kv = idesc_bf16_f32(128, a.d, 0, 1);
      const int ksteps = a.d / 16;
      const uint32_t k_desc = desc_low(sbase + C::OFF_K, 16);
      const uint32_t v_desc = desc_low(sbase + C::OFF_V, 16);
      auto scores = [&](uint32_t to, uint32_t kv, uint32_t rows) {
        const uint32_t row = not_hoisted(desc_low(rows, 16));
        kv = not_hoisted(kv);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          if (k >= ksteps) break;
          const uint32_t off = ((k >> 2) * C::CHUNK + (k & 3) * 32) >> 4;
          tc_mma_low(tmem + to, kv + off, row + off, id_s, k > 0);
        }
      };
      auto add = [&](uint32_t to, uint32_t from, uint32_t rows, bool first) {
        const uint32_t row = not_hoisted(desc_low(rows, C::CHUNK));
#pragma unroll
        for (int k = 0; k < 8; ++k)
          tc_mma_ts_low(tmem + to, tmem + from + packed_col(k), row + k * 128, id_kv,
                        !first || k > 0);
      };
      auto wait = [&](uint32_t bar, uint32_t phase) -> bool {
        if (!wait_for(bar, phase & 1, err)) return false;
        tc_fence_after();
        return true;
      };
      auto q_of = [&](uint32_t at) { return sbase + C::OFF_Q + (at % QST) * C::TILE; };
      auto o_of = [&](uint32_t at) { return sbase + C::OFF_DO + (at % OST) * C::TILE; };
      uint32_t r = 0, it = 0, u = 0;  // steps, row tiles, items with any
      // the row tile of step r, or what else it is
      auto step = [&](int& tile) -> bool {
        if (!wait_for(i_full + 8 * (r % IST), (r / IST) & 1, err)) return false;
        tile = meta[r % IST].tile;
        mbar_arrive(i_empty + 8 * (r % IST));
        ++r;
        return true;
      };
      while (true) {
        int tile;
        if (!step(tile) || tile == kStop) break;
        if (tile < 0) continue;
        if (!wait(kv_full, u) || !wait(q_full + 8 * (it % QST), it / QST)) break;
        scores(C::T_S, k_desc, q_of(it));
        tc_commit(s_full);
        if (!wait(o_full + 8 * (it % OST), it / OST)) break;
        scores(C::T_DP, v_desc, o_of(it));
        tc_commit(dp_full);
        bool first = true, ok = true;
        while (tile >= 0) {
          if (!(ok = wait(p_ready, it))) break;
          // dK and dV of the item before have been read out
          if (first && !(ok = wait(acc_free, u ^ 1))) break;
          add(C::T_DV, C::T_S, o_of(it), first);
          tc_commit(o_empty + 8 * (it % OST));
          if (!(ok = step(tile))) break;
          if (tile >= 0) {  // after dV of this tile, which reads P from the same columns
            if (!(ok = wait(q_full + 8 * ((it + 1) % QST), (it + 1) / QST))) break;
            scores(C::T_S, k_desc, q_of(it + 1));
            tc_commit(s_full);
          }
          if (!(ok = wait(ds_ready, it))) break;
          add(C::T_DK, C::T_DP, q_of(it), first);
          tc_commit(q_empty + 8 * (it % QST));
          ++it;
          first = false;
          if (tile >= 0) {
            if (!(ok = wait(o_full + 8 * (it % OST), it / OST))) break;
            scores(C::T_DP, v_desc, o_of(it));
            tc_commit(dp_full);
          }
        }
        if (!ok) break;
        tc_commit(fin);
        tc_commit(kv_empty);
        ++u;
      }
      tc_commit(drain);
      mbar_wait(drain, 0, nullptr);
    }
  } else if (warp == 2) {
    // ------------- clears Q and dO of queries that see nothing: they may be anything
    uint32_t tiles = 0, raws = 0;
    for (uint32_t r = 0;; ++r) {
      const uint32_t si = r % IST;
      if (!warp_wait(i_full + 8 * si, (r / IST) & 1, err)) break;
      const Meta m = meta[si];
      uint32_t none[4];
      if (m.tile >= 0 && (m.full & kBlind)) {
        const float* rows = reinterpret_cast<const float*>(smem + C::OFF_ROW + si * 1024) + lane;
#pragma unroll
        for (int w = 0; w < 4; ++w)
          none[w] =
              __ballot_sync(0xffffffffu, rows[32 * w] == kNoRow && rows[128 + 32 * w] == 0.f);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(i_empty + 8 * si);
      if (m.tile == kStop) break;
      if (m.tile < 0) continue;
      if (m.full & kBlind) {
        const uint32_t sq = tiles % QST, so = tiles % OST;
        bool ok = true;
#pragma unroll 1
        for (int x = 0; x < 2 && ok; ++x) {
          ok = x ? warp_wait(o_raw + 8 * (raws % OST), (raws / OST) & 1, err)
                 : warp_wait(q_raw + 8 * (raws % QST), (raws / QST) & 1, err);
          if (!ok) break;
          uint8_t* const rows = smem + (x ? C::OFF_DO + so * C::TILE : C::OFF_Q + sq * C::TILE);
#pragma unroll
          for (int w = 0; w < 4; ++w) clear_rows(rows, a.d, w, none[w]);
          hand_over(x ? o_full + 8 * so : q_full + 8 * sq);
        }
        if (!ok) break;
        ++raws;
      }
      ++tiles;
    }
  } else if (warp >= 4) {
    regs_inc<104>();
    // ------------------------ P^T and dS^T: one key, 32 of a tile's 128 rows
    const int quarter = warp & 3, block = (warp - 4) >> 2;
    const int row = quarter * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t ts = tmem + lane_base + C::T_S + block * 32;
    const uint32_t tdp = tmem + lane_base + C::T_DP + block * 32;
    uint32_t it = 0, u = 0, shares = 0;
    bool had = false;  // a row tile of this item
    for (uint32_t r = 0;; ++r) {
      const uint32_t si = r % IST;
      if (!warp_wait(i_full + 8 * si, (r / IST) & 1, err)) break;
      const Meta m = meta[si];
      if (m.tile == kStop) break;
      const int key = m.n0 + row;
      if (m.tile >= 0) {
        had = true;
        const uint8_t* rows = smem + C::OFF_ROW + si * 1024 + block * 128;
        const float4* lse4 = reinterpret_cast<const float4*>(rows);
        const float4* d4 = reinterpret_cast<const float4*>(rows + 512);
        uint32_t seen = 0xffffffffu;
        bool full = m.full & kFull;
        if (!full) {
          const int64_t at = m.tile * int64_t{128} + block * 32;
          const int4* lo4 = reinterpret_cast<const int4*>(ar.lo + at);
          const int4* len4 = reinterpret_cast<const int4*>(ar.len + at);
          seen = 0u;
          auto sees = [&](int lo, int len) {
            return static_cast<uint32_t>(key - lo) < static_cast<uint32_t>(len);
          };
          if (a.rep % 4 == 0) {  // four columns are rows of one query
#pragma unroll
            for (int c = 0; c < 8; ++c) seen |= sees(lo4[c].x, len4[c].x) ? 15u << (4 * c) : 0u;
          } else {
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              const int4 lo = lo4[c], len = len4[c];
              seen |= sees(lo.x, len.x) ? 1u << (4 * c) : 0u;
              seen |= sees(lo.y, len.y) ? 2u << (4 * c) : 0u;
              seen |= sees(lo.z, len.z) ? 4u << (4 * c) : 0u;
              seen |= sees(lo.w, len.w) ? 8u << (4 * c) : 0u;
            }
          }
          full = __all_sync(0xffffffffu, seen == ~0u);
        }
        if (!warp_wait(s_full, it & 1, err)) break;
        tc_fence_after();
        uint32_t sv[32], pk[16];
        tmem_ld32(ts, sv);
        tmem_ld_wait();
        weights<CAP>(
            sv, ar,
            [&](int c) {
              const float4 nl = lse4[c / 4];
              return c & 2 ? make_float2(nl.z, nl.w) : make_float2(nl.x, nl.y);
            },
            [&](int c, float2 p) { pk[c / 2] = pack_bf16x2(p.x, p.y); });
        if (!full) clear_unseen(pk, seen);
        tmem_st16(ts, pk);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(p_ready);
        if (!warp_wait(dp_full, it & 1, err)) break;
        tc_fence_after();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t dp[16];
          tmem_ld16(tdp + 16 * h, dp);
          tmem_ld_wait();
#pragma unroll
          for (int c = 0; c < 16; c += 4) {
            const float4 nd = d4[4 * h + c / 4];
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
              float2 ds =
                  add2(make_float2(__uint_as_float(dp[c + e]), __uint_as_float(dp[c + e + 1])),
                       e ? make_float2(nd.z, nd.w) : make_float2(nd.x, nd.y));
              ds = mul2(ds, make_float2(__uint_as_float(sv[16 * h + c + e]),
                                        __uint_as_float(sv[16 * h + c + e + 1])));
              pk[8 * h + (c + e) / 2] = pack_bf16x2(ds.x, ds.y);
            }
          }
        }
        if (!full) clear_unseen(pk, seen);
        tmem_st16(tdp, pk);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(ds_ready);
        __syncwarp();
        if (lane == 0) mbar_arrive(i_empty + 8 * si);
        ++it;
        continue;
      }
      // ------------------------------------------------ the item's end
      __syncwarp();
      if (lane == 0) mbar_arrive(i_empty + 8 * si);
      if (had && !warp_wait(fin, u & 1, err)) break;
      tc_fence_after();
      const int c0 = block * 32, left = a.d - c0;
      // this thread's 32 columns of dK or dV, 0 if the item had no row tile
      auto fetch = [&](uint32_t from, uint32_t (&x)[32]) {
        if (had) {
          tmem_ld32(tmem + lane_base + from + c0, x);
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) x[e] = 0u;
        }
      };
      bool finish = m.full == kAlone;
      // the two halves' sums: four columns of a row at [half][dK, dV][column / 4][row]
      float4* part = nullptr;
      if (m.full >= kShared) {
        const int64_t pair = static_cast<int64_t>(m.n0 >> 7) * a.nkv + m.g;
        const int half = m.full - kShared, quads = a.d / 4;
        float4* const mine = ar.part + (pair * 2 + half) * 2 * quads * 128;
        part = ar.part + (pair * 2 + (half ^ 1)) * 2 * quads * 128;
        if (left > 0) {
#pragma unroll
          for (int which = 0; which < 2; ++which) {
            uint32_t x[32];
            fetch(which ? C::T_DV : C::T_DK, x);
            float4* to = mine + (which * quads + c0 / 4) * 128 + row;
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (4 * e < left)
                __stcg(to + e * 128,
                       make_float4(__uint_as_float(x[4 * e]), __uint_as_float(x[4 * e + 1]),
                                   __uint_as_float(x[4 * e + 2]), __uint_as_float(x[4 * e + 3])));
          }
        }
        __threadfence();
        mbar_arrive(left_it);
        if (warp == 4 && lane == 0) {
          if (mbar_wait(left_it, shares & 1, err)) {
            __threadfence();
            *decision = atomicAdd(ar.arrived + pair, 1);
            __threadfence();
            mbar_arrive(decided);
          }
        }
        __syncwarp();
        if (!warp_wait(decided, shares & 1, err)) break;
        ++shares;
        finish = *decision == 1;  // the other half has been left
      }
      bool fine = true;
      if (finish && left > 0) {
#pragma unroll
        for (int which = 0; which < 2; ++which) {
          uint32_t x[32];
          fetch(which ? C::T_DV : C::T_DK, x);
          if (part) {
            const float4* from = part + (which * (a.d / 4) + c0 / 4) * 128 + row;
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (4 * e < left) {
                const float4 v = __ldcg(from + e * 128);
                x[4 * e] = __float_as_uint(__uint_as_float(x[4 * e]) + v.x);
                x[4 * e + 1] = __float_as_uint(__uint_as_float(x[4 * e + 1]) + v.y);
                x[4 * e + 2] = __float_as_uint(__uint_as_float(x[4 * e + 2]) + v.z);
                x[4 * e + 3] = __float_as_uint(__uint_as_float(x[4 * e + 3]) + v.w);
              }
          }
          fine = fine && all_finite(x, left);
          if (key < a.keys)
            put_columns((which ? a.dv : a.dk).at(key, m.g) + c0, x, which ? 1.f : a.scale, left,
                        which ? ar.wide_dv : ar.wide_dk);
        }
      }
      if (had) {  // dK and dV are free for the next item
        tc_fence_before();
        mbar_arrive(acc_free);
        ++u;
        had = false;
      }
      unsigned again = __ballot_sync(0xffffffffu, !fine && key < a.keys);
      if (again) __syncwarp();  // other lanes store what a row's own lane stored
      for (; again; again &= again - 1) {
        const int j = m.n0 + quarter * 32 + __ffs(again) - 1;
        if (!sees_nonfinite(ar, j, m.g)) row_dkdv(a, j, m.g, c0, min(c0 + 32, a.d));
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  settle(err.err);
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

// ---------------------------------------------------------------------- dQ
// The columns [c0, c1) of rows of dq that a warp has found not finite (query t and head
// h of each lane, t = -1: none), all of key head g, computed again unless they are so
// by right.
__device__ __noinline__ void dq_again(const SpanArgs& a, int g, int t, int h, int c0, int c1) {
  __syncwarp();  // other lanes store what a row's own lane stored
  int first = 0, end = 0;
  if (t >= 0) a.span(t, first, end);
  for (unsigned again = bad_rows(a, a.k, g, t >= 0 ? a.dq.at(t, h) : nullptr, c0, c1, first, end);
       again; again &= again - 1) {
    const int from = __ffs(again) - 1;
    row_dq(a, __shfl_sync(0xffffffffu, t, from), __shfl_sync(0xffffffffu, h, from), c0, c1);
  }
}

constexpr int kItemRing = 4;
struct Item {
  int index;     // row tile and key head, with kSecond or not; -1: no more in this round
  int first, n;  // first key, key tiles
};

template <int D>
struct QCfg {
  static constexpr uint32_t CHUNK = 128 * 128, TILE = 128 * D * 2;
  // K is read by S, and a whole elementwise pass later by dQ; V by dP only
  static constexpr int KST = D == 128 ? 3 : 4, VST = D == 128 ? 2 : 4;
  static constexpr uint32_t OFF_Q = 0, OFF_DO = TILE, OFF_K = 2 * TILE, OFF_V = OFF_K + KST * TILE,
                            OFF_ROW = OFF_V + VST * TILE,  // [neg_lse, neg_d, lo, len][128]
      OFF_ITEM = OFF_ROW + 2048, OFF_RAN = OFF_ITEM + kItemRing * sizeof(Item),
                            OFF_BAR = OFF_RAN + kRound * sizeof(int);
  static constexpr uint32_t OFF_NEXT = OFF_BAR + 352;
  static constexpr size_t SMEM = OFF_NEXT + 16;  // at a multiple of 1024, which is checked
  static constexpr uint32_t T_S = 0, T_DP = 128, T_DQ = 256, T_DS = 384, TMEM_COLS = 512;
  static_assert(SMEM <= 232448 && OFF_NEXT % 16 == 0, "");
};

template <int D, bool CAP>
__global__ void __launch_bounds__(kThreads, 1)
    spans_dq_kernel(const __grid_constant__ CUtensorMap tq,
                    const __grid_constant__ CUtensorMap tdo,
                    const __grid_constant__ CUtensorMap tk,
                    const __grid_constant__ CUtensorMap tv, const __grid_constant__ Args ar) {
  using C = QCfg<D>;
  constexpr int KST = C::KST, VST = C::VST;
  const SpanArgs& a = ar.a;
  const Patience& err = ar.err_keys;
  extern __shared__ __align__(1024) uint8_t smem_tiles[];
  uint8_t* smem = smem_tiles;
  const uint32_t sbase = smem_u32(smem);
  if (sbase & 1023u) {  // the swizzled tiles' layout counts on it
    record_error(err.err, kErrTimeout);
    return;
  }
  const uint32_t bar0 = sbase + C::OFF_BAR;
  const uint32_t q_full = bar0, q_empty = bar0 + 8, k_full = bar0 + 16, k_empty = k_full + 8 * KST,
                 v_full = k_empty + 8 * KST, v_empty = v_full + 8 * VST, s_full = v_empty + 8 * VST,
                 s_free = s_full + 8, ds_ready = s_free + 8, ds_free = ds_ready + 16, dq_done = ds_free + 16,
                 dq_free = dq_done + 8, drain = dq_free + 8, item_full = drain + 8,
                 item_empty = item_full + 8 * kItemRing, next = item_empty + 8 * kItemRing,
                 k_raw = next + 8;  // K has come that is to be cleared
  static_assert(8 * (2 + 2 * KST + 2 * VST + 11 + 2 * kItemRing) <= 312, "");
  Rounds* rounds = reinterpret_cast<Rounds*>(smem + C::OFF_BAR + 312);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_BAR + 344);
  static_assert(312 + sizeof(Rounds) <= 344 && C::OFF_BAR % 8 == 0, "");
  int* ran = reinterpret_cast<int*>(smem + C::OFF_RAN);  // the items of the round
  Item* ring = reinterpret_cast<Item*>(smem + C::OFF_ITEM);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int chunks = (a.d + 63) / 64, used = ar.tl.per * a.rep;
  // item -> row tile (the last first), key head
  auto place = [&](int item, int& tile, int& g) {
    tile = ar.tl.tiles - 1 - item / a.nkv;
    g = item % a.nkv;
  };

  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1 + kEltThreads / 32);  // the MMAs; the warps that read the rows' values
    for (int x = 0; x < kItemRing; ++x) {
      mbar_init(item_full + 8 * x, 1);
      mbar_init(item_empty + 8 * x, 1 + kEltThreads / 32);
    }
    for (int x = 0; x < KST; ++x) {
      mbar_init(k_full + 8 * x, 1);
      mbar_init(k_empty + 8 * x, 1);
    }
    for (int x = 0; x < VST; ++x) {
      mbar_init(v_full + 8 * x, 1);
      mbar_init(v_empty + 8 * x, 1);
    }
    mbar_init(s_full, 1);
    mbar_init(s_free, kEltThreads);
    // one for each buffer: a warp may be done with the next key tile before another is with
    // this one
    mbar_init(ds_ready, kEltThreads);
    mbar_init(ds_ready + 8, kEltThreads);
    mbar_init(ds_free, 1);
    mbar_init(ds_free + 8, 1);
    mbar_init(dq_done, 1);
    mbar_init(dq_free, kEltThreads);
    mbar_init(drain, 1);
    mbar_init(next, 1);
    mbar_init(k_raw, 1);
    *rounds = Rounds{};
    fence_mbar_init();
    tma_prefetch_desc(&tq);
    tma_prefetch_desc(&tdo);
    tma_prefetch_desc(&tk);
    tma_prefetch_desc(&tv);
  }
  if (warp == 1) tmem_alloc(smem_u32(tmem_slot), C::TMEM_COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  after_previous_kernel();

  unsigned long long redo = 0ull;
  if (warp < 4) regs_dec<56>();
  if (warp == 0) {
    // ----------------------------------------------------------- producer
    bool ok = true;
    uint32_t jg = 0, it = 0, asked = 0, raws = 0;
    int loaded = 0;
    int item = blockIdx.x;
    // an item's place in the ring; what it needs of its row tile
    auto publish = [&](int index, int first, int n) {
      ring[it % kItemRing] = Item{index, first, n};
      mbar_arrive(item_full + 8 * (it % kItemRing));
    };
    auto free_slot = [&]() {
      return wait_for(item_empty + 8 * (it % kItemRing), ((it / kItemRing) & 1) ^ 1, err);
    };
    do {
      if (lane == 0) rounds->start = it;
      const bool second = redo != 0ull;
      // a step of an item's loads: tile j of K or V
      auto load = [&](int j, int first, int g, uint32_t bar, uint32_t empty, int stages,
                      uint32_t off, const CUtensorMap* map) -> bool {
        const uint32_t jj = jg + j, st = jj % stages;
        if (!wait_for(empty + 8 * st, ((jj / stages) & 1) ^ 1, err)) return false;
        if (!bar) bar = empty - 8 * stages + 8 * st;  // the stage's own, which lie before
        mbar_arrive_expect_tx(bar, chunks * C::CHUNK);
        for (int c = 0; c < chunks; ++c)
          tma_load_3d(sbase + off + st * C::TILE + c * C::CHUNK, map, bar, c * 64, g,
                      first + j * 128);
        return true;
      };
      auto load_rows = [&](int tile, int g) -> bool {
        if (!wait_for(q_empty, (loaded & 1) ^ 1, err)) return false;
        const int64_t at = (static_cast<int64_t>(g) * ar.tl.tiles + tile) * 128;
        mbar_arrive_expect_tx(q_full, 2 * chunks * used * 128 + 2048);
        for (int c = 0; c < chunks; ++c) {
          tma_load_3d(sbase + C::OFF_Q + c * C::CHUNK, &tq, q_full, c * 64, g * a.rep,
                      tile * ar.tl.per);
          tma_load_3d(sbase + C::OFF_DO + c * C::CHUNK, &tdo, q_full, c * 64, g * a.rep,
                      tile * ar.tl.per);
        }
        bulk_load_1d(sbase + C::OFF_ROW, ar.neg_lse + at, 512, q_full);
        bulk_load_1d(sbase + C::OFF_ROW + 512, ar.neg_d + at, 512, q_full);
        bulk_load_1d(sbase + C::OFF_ROW + 1024, ar.lo + tile * int64_t{128}, 512, q_full);
        bulk_load_1d(sbase + C::OFF_ROW + 1536, ar.len + tile * int64_t{128}, 512, q_full);
        return true;
      };
      if (second) {
        // items once more, K by way of k_raw, its rows that nobody sees cleared; whole warp
        for (; redo && ok; redo &= redo - 1, ++it) {
          const int again = ran[__ffsll(redo) - 1];
          int tile, g;
          place(again, tile, g);
          const int first = ar.tiles[tile].first, n = (ar.tiles[tile].end - first + 127) / 128;
          if (lane == 0) {
            ok = free_slot();
            if (ok) publish(again | kSecond, first, n);
          }
          ok = __shfl_sync(0xffffffffu, static_cast<int>(ok), 0);
          for (int j = 0; j < n && ok; ++j, ++raws) {
            if (lane == 0)
              ok = load(j, first, g, k_raw, k_empty, KST, C::OFF_K, &tk) &&
                   (j > 0 || load_rows(tile, g)) &&
                   load(j, first, g, 0u, v_empty, VST, C::OFF_V, &tv);
            ok = __shfl_sync(0xffffffffu, static_cast<int>(ok), 0);
            const uint32_t st = (jg + j) % KST;
            const int t0 = tile * ar.tl.per;
            ok = ok && clear_unseen(a, t0, min(ar.tl.per, a.queries - t0), first + j * 128,
                                    smem + C::OFF_K + st * C::TILE, k_raw, raws & 1,
                                    k_full + 8 * st, err);
          }
          if (n > 0) {
            jg += n;
            ++loaded;
          }
        }
      }
      if (lane == 0) {
        for (int of = 0; ok; ++of, ++it) {
          ok = free_slot();
          if (!ok) break;
          if (item < 0 || second || of == kRound) {
            rounds->left = item >= 0;
            publish(-1, 0, 0);
            ++it;
            break;
          }
          int tile, g;
          place(item, tile, g);
          const int first = ar.tiles[tile].first, n = (ar.tiles[tile].end - first + 127) / 128;
          publish(item, first, n);
          ran[of] = item;
          if (n > 0) {
            // K's first tile does not wait for the item before to be done with its Q
            ok = load(0, first, g, 0u, k_empty, KST, C::OFF_K, &tk) && load_rows(tile, g);
            for (int j = 0; j < n && ok; ++j) {
              ok = (j == 0 || load(j, first, g, 0u, k_empty, KST, C::OFF_K, &tk)) &&
                   load(j, first, g, 0u, v_empty, VST, C::OFF_V, &tv);
            }
            jg += n;
            ++loaded;
          }
          // asked for now, not before: an item that waits here could have been another SM's;
          // waited for on the way out too: the answer is written to this CTA's memory
          next_cta_request(sbase + C::OFF_NEXT, next);
          const bool answered = wait_for(next, asked++ & 1, err);
          ok = ok && answered;
          if (ok) item = next_cta_answer(sbase + C::OFF_NEXT);
        }
        if (!ok) rounds->lost = 1;
      }
      // the whole warp goes on from what its first lane has counted
      ok = __shfl_sync(0xffffffffu, static_cast<int>(ok), 0);
      it = __shfl_sync(0xffffffffu, it, 0);
      jg = __shfl_sync(0xffffffffu, jg, 0);
      loaded = __shfl_sync(0xffffffffu, loaded, 0);
    } while (next_round<true>(rounds, kThreads, redo));
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA
    constexpr uint32_t id_s = idesc_bf16_f32(128, 128, 0, 0);
    const uint32_t id_q = idesc_bf16_f32(128, a.d, 0, 1);
    const int ksteps = a.d / 16;
    const uint32_t q_desc = desc_low(sbase + C::OFF_Q, 16);
    const uint32_t o_desc = desc_low(sbase + C::OFF_DO, 16);
    auto scores = [&](uint32_t to, uint32_t rows, uint32_t keys) {
      const uint32_t k2 = not_hoisted(desc_low(keys, 16));
      rows = not_hoisted(rows);
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        if (k >= ksteps) break;
        const uint32_t off = ((k >> 2) * C::CHUNK + (k & 3) * 32) >> 4;
        tc_mma_low(tmem + to, rows + off, k2 + off, id_s, k > 0);
      }
    };
    bool ok = true;
    uint32_t jg = 0;
    int loaded = 0, it = 0;
    uint32_t drains = 0;
    do {
      if (elect_one()) {
        bool stop = false;
        for (; ok; ++it) {
          const int slot = it % kItemRing;
          if (!wait_for(item_full + 8 * slot, (it / kItemRing) & 1, err)) break;
          const int index = ring[slot].index, n = ring[slot].n;
          mbar_arrive(item_empty + 8 * slot);
          if (index < 0) {
            ++it;
            stop = true;
            break;
          }
          if (n == 0) continue;
          // S and dP of key tile j, once those of the one before are in registers
          auto issue = [&](int j) -> bool {
            const uint32_t jj = jg + j, ks = jj % KST, vs = jj % VST;
            if (!wait_for(k_full + 8 * ks, (jj / KST) & 1, err) ||
                !wait_for(v_full + 8 * vs, (jj / VST) & 1, err) ||
                !wait_for(s_free, (jj & 1) ^ 1, err))
              return false;
            tc_fence_after();
            scores(C::T_S, q_desc, sbase + C::OFF_K + ks * C::TILE);
            scores(C::T_DP, o_desc, sbase + C::OFF_V + vs * C::TILE);
            tc_commit(s_full);
            tc_commit(v_empty + 8 * vs);
            if (j + 1 == n) tc_commit(q_empty);  // the item's last read of Q and dO
            return true;
          };
          ok = wait_for(q_full, loaded & 1, err) && issue(0);
          for (int j = 0; j < n && ok; ++j) {
            const uint32_t jj = jg + j;
            const int ks = jj % KST;
            if (j + 1 < n) ok = issue(j + 1);
            // dQ of the item before has been read out of TMEM
            if (ok && j == 0) ok = wait_for(dq_free, (loaded & 1) ^ 1, err);
            if (ok) ok = wait_for(ds_ready + 8 * (jj & 1), (jj >> 1) & 1, err);
            if (!ok) break;
            tc_fence_after();
            const uint32_t k_desc =
                not_hoisted(desc_low(sbase + C::OFF_K + ks * C::TILE, C::CHUNK));
            const uint32_t ds = tmem + C::T_DS + (jj & 1) * 64;
#pragma unroll
            for (int k = 0; k < 8; ++k)
              tc_mma_ts_low(tmem + C::T_DQ, ds + 8 * k, k_desc + k * 128, id_q, (j | k) != 0);
            tc_commit(ds_free + 8 * (jj & 1));
            tc_commit(k_empty + 8 * ks);
          }
          if (ok) tc_commit(dq_done);
          jg += n;
          ++loaded;
        }
        if (!stop) rounds->lost = 1;
        tc_commit(drain);
        mbar_wait(drain, drains++ & 1, nullptr);
      }
      __syncwarp();
    } while (next_round<true>(rounds, kThreads, redo));
  } else if (warp < 4) {
    while (next_round<true>(rounds, kThreads, redo)) {
    }
  } else {
    regs_inc<104>();
    // --------------------------- dS: one row, 32 of a key tile's 128 columns
    const int quarter = warp & 3, block = (warp - 4) >> 2;
    const int row = quarter * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    const int row_t = row / a.rep, row_h = row % a.rep;
    bool ok = true;
    uint32_t jg = 0;
    int loaded = 0, it = 0;
    do {
      bool stop = false;
      for (; ok; ++it) {
        const int slot = it % kItemRing;
        if (!warp_wait(item_full + 8 * slot, (it / kItemRing) & 1, err)) break;
        const int item = ring[slot].index, first = ring[slot].first, n = ring[slot].n;
        __syncwarp();
        if (lane == 0) mbar_arrive(item_empty + 8 * slot);
        if (item < 0) {
          ++it;
          stop = true;
          break;
        }
        float nl = 0.f, nd = 0.f;
        int lo = 0, len = 0;
        if (n > 0) {
          if (!warp_wait(q_full, loaded & 1, err)) break;
          const float* rows = reinterpret_cast<const float*>(smem + C::OFF_ROW);
          nl = rows[row];
          nd = rows[128 + row];
          lo = __float_as_int(rows[256 + row]);
          len = __float_as_int(rows[384 + row]);
          __syncwarp();
          if (lane == 0) mbar_arrive(q_empty);
        }
        const float2 nl2 = make_float2(nl, nl), nd2 = make_float2(nd, nd);
        const bool finite = finite_row(nl, nd);
        for (int j = 0; j < n; ++j) {
          const uint32_t jj = jg + j;
          const int buf = jj & 1;
          ok = warp_wait(s_full, jj & 1, err);
          if (!ok) break;
          tc_fence_after();
          uint32_t sv[32], dp[32];
          tmem_ld32(tmem + lane_base + C::T_S + block * 32, sv);
          tmem_ld32(tmem + lane_base + C::T_DP + block * 32, dp);
          tmem_ld_wait();
          tc_fence_before();
          mbar_arrive(s_free);
          // columns l <= c < l + len are seen; a row that sees nothing has p = 0 as it is
          const int l = lo - (first + j * 128 + block * 32);
          const bool full = __all_sync(0xffffffffu, len == 0 || (l <= 0 && l + len >= 32));
          const uint32_t seen = full ? ~0u : bits_between(l, l + len);
          weights<CAP>(sv, ar, [&](int) { return nl2; }, [](int, float2) {});
#pragma unroll
          for (int c = 0; c < 32; c += 2) {
            float2 ds = add2(make_float2(__uint_as_float(dp[c]), __uint_as_float(dp[c + 1])), nd2);
            ds = mul2(ds, make_float2(__uint_as_float(sv[c]), __uint_as_float(sv[c + 1])));
            sv[c / 2] = pack_bf16x2(ds.x, ds.y);  // over what has been used
          }
          uint32_t(&pk)[16] = *reinterpret_cast<uint32_t(*)[16]>(&sv[0]);
          if (!full) clear_unseen(pk, seen);
          // this buffer was last read by dQ += dS K two key tiles ago
          ok = warp_wait(ds_free + 8 * buf, ((jj >> 1) & 1) ^ 1, err);
          if (!ok) break;
          tc_fence_after();
          tmem_st16(tmem + lane_base + C::T_DS + buf * 64 + block * 16, pk);
          tmem_st_wait();
          tc_fence_before();
          mbar_arrive(ds_ready + 8 * buf);
        }
        if (!ok) break;
        uint32_t r[32];
        const int c0 = block * 32, left = a.d - c0;
        if (n > 0) {
          if (!warp_wait(dq_done, loaded & 1, err)) break;
          tc_fence_after();
          if (left > 0) {
            tmem_ld32(tmem + lane_base + C::T_DQ + c0, r);
            tmem_ld_wait();
          }
          tc_fence_before();
          mbar_arrive(dq_free);
          ++loaded;
          jg += n;
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) r[e] = 0u;
        }
        if (left > 0) {
          const int again_of = not_hoisted(item);  // not held meanwhile: registers are short
          int tile, g;
          place(again_of & (kSecond - 1), tile, g);
          const int t = tile * ar.tl.per + row_t, h = g * a.rep + row_h;
          const bool real = row_t < ar.tl.per && t < a.queries;
          if (real) put_columns(a.dq.at(t, h) + c0, r, a.scale, left, ar.wide_dq);
          const bool mine = real && finite && !all_finite(r, left);
          if (__any_sync(0xffffffffu, mine)) {
            if (again_of & kSecond)
              dq_again(a, g, mine ? t : -1, h, c0, min(c0 + 32, a.d));
            else if (lane == 0)
              take_again(rounds, it);
          }
        }
      }
      if (!stop && lane == 0) rounds->lost = 1;
      tc_fence_before();
    } while (next_round<true>(rounds, kThreads, redo));
  }

  // the last round's end has been waited for by all
  settle(err.err);
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

// -------------------------------------------------------------------- host
template <int D, bool CAP>
cudaError_t launch(const Args& ar, cudaStream_t s) {
  const SpanArgs& a = ar.a;
  CUtensorMap tq, tdo, tk, tv;
  if (!make_tma_heads(&tq, a.q.p, a.queries, a.nh, a.d, a.q.ts, a.q.hs, a.rep, ar.tl.per) ||
      !make_tma_heads(&tdo, a.d_o.p, a.queries, a.nh, a.d, a.d_o.ts, a.d_o.hs, a.rep, ar.tl.per) ||
      !make_tma_heads(&tk, a.k.p, a.keys, a.nkv, a.d, a.k.ts, a.k.hs, 1, 128) ||
      !make_tma_heads(&tv, a.v.p, a.keys, a.nkv, a.d, a.v.ts, a.v.hs, 1, 128))
    return cudaErrorInvalidValue;
  cudaError_t e = allow_smem<spans_dkdv_kernel<D, CAP>>(KvCfg<D>::SMEM);
  if (e == cudaSuccess) e = allow_smem<spans_dq_kernel<D, CAP>>(QCfg<D>::SMEM);
  if (e != cudaSuccess) return e;
  const int64_t units = static_cast<int64_t>(a.nkv) * ar.tl.tiles;
  const int64_t prep = ar.groups + std::min<int64_t>(units, int64_t{num_sms()} * 8);
  e = launch_overlapping(prepare_kernel, prep, kPrepThreads, 0, s, ar);
  if (e != cudaSuccess) return e;
  e = launch_overlapping(spans_dkdv_kernel<D, CAP>, ar.key_tiles * ar.parts, kThreads,
                         KvCfg<D>::SMEM, s, tq, tdo, tk, tv, ar);
  if (e != cudaSuccess) return e;
  return launch_overlapping(spans_dq_kernel<D, CAP>, static_cast<int64_t>(ar.tl.tiles) * a.nkv,
                            kThreads, QCfg<D>::SMEM, s, tq, tdo, tk, tv, ar);
}

// Key tiles are halved where there are fewer than this times the SMs: with halves /
// without, documents up to 1024 in 4096 tokens 128 / 145 us, one of 4096 349 / 340;
// from 512 key tiles on nothing is won (8192 tokens in one 1189 / 1158, in eight 297
// / 284).
constexpr int kHalvedBelow = 3;

// The workspace: rows' values, spans of rows, of tiles, of groups; halves' sums.
size_t lay_out(Args* ar, int queries, int keys, int rep, int nkv, int d, void* ws) {
  ar->tl = Tiling::of(queries, rep);
  ar->key_tiles = static_cast<int64_t>((keys + 127) / 128) * nkv;
  // a second half needs row tiles enough to share
  ar->parts = ar->tl.tiles >= kShareFrom && ar->key_tiles < kHalvedBelow * int64_t{num_sms()} ? 2 : 1;
  ar->groups = (ar->tl.tiles + kGroup - 1) / kGroup;
  const size_t rows = static_cast<size_t>(ar->tl.tiles) * 128;
  uint8_t* p = static_cast<uint8_t*>(ws);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    uint8_t* here = p + at;
    at += (bytes + 255) / 256 * 256;
    return here;
  };
  ar->neg_lse = reinterpret_cast<float*>(take(rows * nkv * sizeof(float)));
  ar->neg_d = reinterpret_cast<float*>(take(rows * nkv * sizeof(float)));
  ar->lo = reinterpret_cast<int*>(take(rows * sizeof(int)));
  ar->len = reinterpret_cast<int*>(take(rows * sizeof(int)));
  ar->tiles = reinterpret_cast<TileSpan*>(take(ar->tl.tiles * sizeof(TileSpan)));
  ar->group = reinterpret_cast<int2*>(take(ar->groups * sizeof(int2)));
  if (ar->parts > 1) {
    ar->part = reinterpret_cast<float4*>(take(ar->key_tiles * 4 * 128 * d * sizeof(float)));
    ar->arrived = reinterpret_cast<int*>(take(ar->key_tiles * sizeof(int)));
  }
  return at;
}

}  // namespace

size_t backward_workspace(int queries, int keys, int nh, int nkv, int d) {
  Args ar = {};
  return lay_out(&ar, queries, keys, nh / nkv, nkv, d, nullptr);
}

cudaError_t backward_tiles(const SpanArgs& a, void* ws, cudaStream_t s) {
  Args ar = {};
  ar.a = a;
  lay_out(&ar, a.queries, a.keys, a.rep, a.nkv, a.d, ws);
  ar.cap = cap_of(a.scale, a.cap);
  ar.scale_log2 = (a.cap > 0.f ? a.cap : a.scale) * kLog2e;
  int* const err = device_error_ptr();
  ar.err_rows = {err, kWaitLimitNs + kNsOfQuery * a.queries * a.rep};
  ar.err_keys = {err, kWaitLimitNs + kNsOfKey * a.keys};
  auto wide = [](const View& x, int64_t tokens, int64_t heads) {
    return (reinterpret_cast<uintptr_t>(x.p) | (tokens > 1 ? x.ts * 2 : 0) |
            (heads > 1 ? x.hs * 2 : 0)) % 32 == 0;
  };
  ar.wide_dq = wide(a.dq, a.queries, a.nh);
  ar.wide_dk = wide(a.dk, a.keys, a.nkv);
  ar.wide_dv = wide(a.dv, a.keys, a.nkv);
  if (a.d <= 64) return a.cap > 0.f ? launch<64, true>(ar, s) : launch<64, false>(ar, s);
  return a.cap > 0.f ? launch<128, true>(ar, s) : launch<128, false>(ar, s);
}

}  // namespace rdt
