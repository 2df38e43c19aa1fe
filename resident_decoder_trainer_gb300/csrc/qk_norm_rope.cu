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
// 128 is eight lanes and a warp takes four heads at a time; all heads of a
// token share the lane's eight cosines and sines. The next heads' loads are under
// way while some are computed, in pairs of fp32 (fma.f32x2). q and k have
// CTAs of their own, so that a warp sums one gain's gradient.
// Heads 32 / 8 of 128: 32,768 tokens bf16 112.5 us, 5.96 TB/s (a copy: 6.78); 4096
// tokens fp32 to bf16 25.0 us, 5.0 TB/s, of them 5 us start and end; gradient of 16,384 bf16
// 97 us, 5.2 TB/s, of them 4 us the sums of the gains' gradients; of 16,384 fp32 135 us,
// 6.2 TB/s (its kernels with fp32 q and k spill 8 to 32 bytes).
//
// Angles: a full turn is 2^64. A pair's rate is kept as a 64-bit fraction of a
// turn, the product with the position is taken modulo 2^64, and its upper 32
// bits are the angle, exact to 2^-32 turns beside the rate's own roundings
// (2^-51), however far the position.
#include <algorithm>
#include <cmath>

#include "heads.cuh"

namespace rdt {

namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kCtasPerSm = 2;  // what their registers leave
constexpr int kMaxHalf = 128;  // pairs of a head of 256

// Turns of a pair for each position, in 2^-64, and the pair's axis.
struct Rates {
  uint64_t turn[kMaxHalf];
  uint8_t axis[kMaxHalf];
};

// q or k. A warp takes `per_pass` of its heads at a time, in `passes` over a
// token; the warps of `blocks` CTAs share the passes over all tokens evenly.
struct Side {
  const void *x, *dy;
  void* out;
  const float* gain;  // null: no norm
  int64_t x_ts, x_hs, dy_ts, dy_hs, out_ts, out_hs;
  int heads, passes, blocks;
};

struct NormArgs {
  Side side[2];
  float eps;
  const int32_t* positions;  // null: no rotation
  int axes;
  int tokens, d;
  int lanes, lanes_log2;  // lanes of a head, a power of two; those past d / 16 have nothing
  int f16_in, f16_dy, f16_out;  // of 16-bit types: fp16 rather than bf16
  float* partial;               // CTA's sums of gain gradients, [blocks of q, then of k][d]
};

// A lane's eight pairs of a head as loaded, B bytes a value.
template <int B>
struct Pairs {
  uint4 v[B];  // the lower half's eight values, then the upper's
  __device__ __forceinline__ void load(const char* p, int half) {
#pragma unroll
    for (int i = 0; i < B / 2; ++i) {
      v[i] = reinterpret_cast<const uint4*>(p)[i];
      v[B / 2 + i] = reinterpret_cast<const uint4*>(p + half * B)[i];
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < B; ++i) v[i] = make_uint4(0u, 0u, 0u, 0u);
  }
  // x: [0, 4) the lower half in twos, [4, 8) the upper
  __device__ __forceinline__ void get(float2 (&x)[8], bool f16) const {
#pragma unroll
    for (int i = 0; i < B; ++i) {
      const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
      if constexpr (B == 4) {
        x[2 * i] = make_float2(__uint_as_float(w[0]), __uint_as_float(w[1]));
        x[2 * i + 1] = make_float2(__uint_as_float(w[2]), __uint_as_float(w[3]));
      } else if (f16) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          x[4 * i + e] = __half22float2(*reinterpret_cast<const __half2*>(&w[e]));
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) x[4 * i + e] = make_float2(bf16lo(w[e]), bf16hi(w[e]));
      }
    }
  }
};

template <int B>
__device__ __forceinline__ void put_pairs(char* p, int half, const float2 (&x)[8], bool f16) {
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    uint4* to = reinterpret_cast<uint4*>(p + side * half * B);
    const float2* y = x + 4 * side;
    if constexpr (B == 4) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        to[i] = make_uint4(__float_as_uint(y[2 * i].x), __float_as_uint(y[2 * i].y),
                           __float_as_uint(y[2 * i + 1].x), __float_as_uint(y[2 * i + 1].y));
    } else {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (f16) {
          const __half2 h = __floats2half2_rn(y[i].x, y[i].y);
          w[i] = *reinterpret_cast<const uint32_t*>(&h);
        } else {
          w[i] = pack_bf16x2(y[i].x, y[i].y);
        }
      }
      to[0] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

// Cosine and sine of two angles in 2^-31 of a half turn: the nearest quarter
// turn is taken off, exactly, and least-squares polynomials on the eighth turn
// left (with these coefficients off by 2^-29.1 and 2^-28.7) do the rest.
__device__ __forceinline__ void turn_two(int32_t a, int32_t b, float2& cos, float2& sin) {
  auto quarter = [](int32_t v) {  // the sum passes the type's end, so not in its own
    return static_cast<int32_t>(static_cast<uint32_t>(v) + 0x20000000u) >> 30;
  };
  const int32_t qa = quarter(a), qb = quarter(b);
  const float unit = 1.4629180792671596e-9f;  // pi 2^-31
  const float2 x = make_float2(static_cast<float>(static_cast<int32_t>(
                                   static_cast<uint32_t>(a) - (static_cast<uint32_t>(qa) << 30))) *
                                   unit,
                               static_cast<float>(static_cast<int32_t>(
                                   static_cast<uint32_t>(b) - (static_cast<uint32_t>(qb) << 30))) *
                                   unit);
  auto both = [](float v) { return make_float2(v, v); };
  const float2 y = mul2(x, x);
  float2 s = fma2(y, both(-0.000194956359f), both(0.00833197869f));
  s = fma2(s, y, both(-0.166666508f));
  s = fma2(mul2(s, y), x, x);
  float2 c = fma2(y, both(2.43904506e-5f), both(-0.00138867635f));
  c = fma2(c, y, both(0.0416666232f));
  c = fma2(c, y, both(-0.5f));
  c = fma2(c, y, both(1.f));
  auto place = [](int32_t q, float s1, float c1, float& sn, float& cs) {
    sn = q & 1 ? c1 : s1;
    cs = q & 1 ? s1 : c1;
    if (q & 2) sn = -sn;
    if ((q + 1) & 2) cs = -cs;
  };
  place(qa, s.x, c.x, sin.x, cos.x);
  place(qb, s.y, c.y, sin.y, cos.y);
}

__device__ __forceinline__ float head_sum(float v, int lanes) {
  for (int o = lanes >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Where a lane stands, and the passes its warp goes through, one run of them
// token by token: the loads of a step under way while the one before is
// computed.
struct Walk {
  const NormArgs& a;
  const Side& s;
  int slot, chunk, per_pass;
  bool has;
  int64_t left;  // passes
  int token, pass, last;
  __device__ __forceinline__ Walk(const NormArgs& args, const Side& side, int block)
      : a(args), s(side) {
    const int lane = threadIdx.x & 31;
    slot = lane >> a.lanes_log2;
    chunk = lane & (a.lanes - 1);
    per_pass = 32 >> a.lanes_log2;
    has = 16 * chunk < a.d;
    const int64_t all = static_cast<int64_t>(a.tokens) * s.passes, warps = s.blocks * kWarps;
    const int64_t me = static_cast<int64_t>(block) * kWarps + (threadIdx.x >> 5);
    // the first `all % warps` warps have one more
    const int64_t each = all / warps, more_of = all % warps;
    const int64_t first = me * each + min(me, more_of);
    left = each + (me < more_of);
    token = static_cast<int>(first / s.passes);
    pass = static_cast<int>(first % s.passes);
    last = static_cast<int>(min(static_cast<int64_t>(s.passes), pass + left));
  }
  __device__ __forceinline__ bool more() const { return left > 0; }
  // The next `n` passes; whether they are of another token.
  __device__ __forceinline__ bool advance(int n) {
    left -= min(n, last - pass);
    pass += n;
    if (pass < last) return false;
    ++token;
    pass = 0;
    last = static_cast<int>(min(static_cast<int64_t>(s.passes), left));
    return true;
  }
  __device__ __forceinline__ bool mine(int pass_of) const {
    return has && pass_of < last && pass_of * per_pass + slot < s.heads;
  }
  // This lane's place in a tensor at the pass, in elements.
  __device__ __forceinline__ int64_t at(int64_t ts, int64_t hs) const {
    return token * ts + static_cast<int64_t>(pass * per_pass + slot) * hs + 8 * chunk;
  }
};

// Cosines and sines of a lane's eight pairs at a token's positions. The lanes
// that hold the same pairs of other heads compute a part each (two pairs, four
// where only two heads fit a warp) and pass them on.
__device__ __forceinline__ void turns(const NormArgs& a, const Rates& rates, const Walk& w,
                                      const int (&pos)[4], float2 (&cos)[4], float2 (&sin)[4]) {
  const bool two = w.per_pass == 2;
  float2 c[2], s[2];
#pragma unroll
  for (int part = 0; part < 2; ++part) {
    if (part && !two) break;
    const int i = two ? w.slot + 2 * part : w.slot & 3;
    int32_t angle[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int pair = (8 * w.chunk + 2 * i + e) & (kMaxHalf - 1);
      int p = pos[0];
      if (a.axes > 1) {
        const int which = rates.axis[pair];
        p = which == 0 ? pos[0] : which == 1 ? pos[1] : which == 2 ? pos[2] : pos[3];
      }
      angle[e] = static_cast<int32_t>(
          (static_cast<uint64_t>(static_cast<int64_t>(p)) * rates.turn[pair]) >> 32);
    }
    turn_two(angle[0], angle[1], c[part], s[part]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int from = ((two ? i & 1 : i) << a.lanes_log2) + w.chunk;
    const int part = two && i >= 2;
    cos[i].x = __shfl_sync(0xffffffffu, part ? c[1].x : c[0].x, from);
    cos[i].y = __shfl_sync(0xffffffffu, part ? c[1].y : c[0].y, from);
    sin[i].x = __shfl_sync(0xffffffffu, part ? s[1].x : s[0].x, from);
    sin[i].y = __shfl_sync(0xffffffffu, part ? s[1].y : s[0].y, from);
  }
}

__device__ __forceinline__ void positions_of(const NormArgs& a, int token, int (&pos)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    pos[i] = i < a.axes ? a.positions[static_cast<int64_t>(i) * a.tokens + token] : 0;
}

// A lane's gains: those of its lower eight pairs' values, then of the upper.
__device__ __forceinline__ void gains_of(const float* gain, const Walk& w, int half,
                                         float2 (&g)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 v = *reinterpret_cast<const float4*>(gain + (w.has ? 8 * w.chunk : 0) +
                                                      (i >> 1) * half + 4 * (i & 1));
    g[2 * i] = make_float2(v.x, v.y);
    g[2 * i + 1] = make_float2(v.z, v.w);
  }
}

// Rates and a side's gains (ones without any) to shared memory.
__device__ __forceinline__ void stage_tables(const NormArgs& a, const Side& s, const Rates& from,
                                             Rates& rates, float (&gain)[2 * kMaxHalf]) {
  for (int i = threadIdx.x; i < a.d; i += kThreads) gain[i] = s.gain ? s.gain[i] : 1.f;
  for (int i = threadIdx.x; i < kMaxHalf; i += kThreads) {
    rates.turn[i] = from.turn[i];
    rates.axis[i] = from.axis[i];
  }
  __syncthreads();
}

// IN, OUT: bytes of a value; BATCH passes at a time.
template <int IN, int OUT, int BATCH>
__global__ void __launch_bounds__(kThreads, 2)
    norm_rope_kernel(const __grid_constant__ NormArgs a, const __grid_constant__ Rates given) {
  __shared__ Rates rates;
  __shared__ __align__(16) float gain[2 * kMaxHalf];
  after_previous_kernel();
  const bool second = static_cast<int>(blockIdx.x) >= a.side[0].blocks;
  const Side& s = a.side[second];
  stage_tables(a, s, given, rates, gain);
  Walk w(a, s, second ? blockIdx.x - a.side[0].blocks : blockIdx.x);
  if (!w.more()) return;
  const int half = a.d >> 1;
  const float inv_d = 1.f / static_cast<float>(a.d);
  const int64_t x_pass = w.per_pass * s.x_hs * IN, out_pass = w.per_pass * s.out_hs * OUT;
  float2 g[8];
  gains_of(gain, w, half, g);
  const char* from = static_cast<const char*>(s.x) + w.at(s.x_ts, s.x_hs) * IN;
  char* to = static_cast<char*>(s.out) + w.at(s.out_ts, s.out_hs) * OUT;
  Pairs<IN> next[BATCH];
  auto fetch = [&] {
#pragma unroll
    for (int b = 0; b < BATCH; ++b) {
      if (w.mine(w.pass + b))
        next[b].load(from + b * x_pass, half);
      else
        next[b].zero();
    }
  };
  fetch();
  int pos[4] = {};
  if (a.axes) positions_of(a, w.token, pos);
  bool fresh = true;
  float2 cos[4], sin[4], minus[4];
  while (w.more()) {
    Pairs<IN> now[BATCH];
    bool mine[BATCH];
#pragma unroll
    for (int b = 0; b < BATCH; ++b) {
      now[b] = next[b];
      mine[b] = w.mine(w.pass + b);
    }
    char* const to_now = to;
    if (fresh && a.axes) {
      turns(a, rates, w, pos, cos, sin);
#pragma unroll
      for (int i = 0; i < 4; ++i) minus[i] = make_float2(-sin[i].x, -sin[i].y);
    }
    fresh = w.advance(BATCH);
    if (fresh) {
      if (w.more()) {
        from = static_cast<const char*>(s.x) + w.at(s.x_ts, s.x_hs) * IN;
        to = static_cast<char*>(s.out) + w.at(s.out_ts, s.out_hs) * OUT;
        if (a.axes) positions_of(a, w.token, pos);
      }
    } else {
      from += BATCH * x_pass;
      to += BATCH * out_pass;
    }
    if (w.more()) fetch();
#pragma unroll
    for (int b = 0; b < BATCH; ++b) {
      float2 x[8];
      now[b].get(x, a.f16_in);
      if (s.gain) {
        float2 sq = mul2(x[0], x[0]);
#pragma unroll
        for (int i = 1; i < 8; ++i) sq = fma2(x[i], x[i], sq);
        const float r = rsqrtf(head_sum(sq.x + sq.y, a.lanes) * inv_d + a.eps);
        const float2 r2 = make_float2(r, r);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = mul2(mul2(x[i], r2), g[i]);
      }
      if (a.axes) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 p = x[i], q = x[4 + i];
          x[i] = fma2(q, minus[i], mul2(p, cos[i]));
          x[4 + i] = fma2(p, sin[i], mul2(q, cos[i]));
        }
      }
      if (mine[b]) put_pairs<OUT>(to_now + b * out_pass, half, x, a.f16_out);
    }
  }
}

// G, IN, OUT: bytes of a value of the incoming gradient, of q and k, of the result.
template <int G, int IN, int OUT>
__global__ void __launch_bounds__(kThreads, 2)
    norm_rope_grad_kernel(const __grid_constant__ NormArgs a,
                          const __grid_constant__ Rates given) {
  __shared__ Rates rates;
  __shared__ __align__(16) float gain[2 * kMaxHalf];
  __shared__ float sums[kWarps][2 * kMaxHalf];
  after_previous_kernel();
  const bool second = static_cast<int>(blockIdx.x) >= a.side[0].blocks;
  const Side& s = a.side[second];
  stage_tables(a, s, given, rates, gain);
  Walk w(a, s, second ? blockIdx.x - a.side[0].blocks : blockIdx.x);
  const int half = a.d >> 1;
  const float inv_d = 1.f / static_cast<float>(a.d);
  const int64_t x_pass = w.per_pass * s.x_hs * IN, dy_pass = w.per_pass * s.dy_hs * G,
                out_pass = w.per_pass * s.out_hs * OUT;
  const char *from = nullptr, *from_dy = nullptr;
  char* to = nullptr;
  auto enter = [&] {
    from = static_cast<const char*>(s.x) + w.at(s.x_ts, s.x_hs) * IN;
    from_dy = static_cast<const char*>(s.dy) + w.at(s.dy_ts, s.dy_hs) * G;
    to = static_cast<char*>(s.out) + w.at(s.out_ts, s.out_hs) * OUT;
  };
  Pairs<IN> next_x;
  Pairs<G> next_g;
  auto fetch = [&] {
    if (w.mine(w.pass)) {
      next_x.load(from, half);
      next_g.load(from_dy, half);
    } else {
      next_x.zero();
      next_g.zero();
    }
  };
  int pos[4] = {};
  if (w.more()) {
    enter();
    fetch();
    if (a.axes) positions_of(a, w.token, pos);
  }
  bool fresh = true;
  float2 cos[4], sin[4], acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = make_float2(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    cos[i] = make_float2(1.f, 1.f);
    sin[i] = make_float2(0.f, 0.f);
  }
  while (w.more()) {
    float2 x[8], d[8];
    next_x.get(x, a.f16_in);
    next_g.get(d, a.f16_dy);
    const bool mine = w.mine(w.pass);
    char* const to_now = to;
    if (fresh && a.axes) turns(a, rates, w, pos, cos, sin);
    fresh = w.advance(1);
    if (fresh) {
      if (w.more()) {
        enter();
        if (a.axes) positions_of(a, w.token, pos);
      }
    } else {
      from += x_pass;
      from_dy += dy_pass;
      to += out_pass;
    }
    if (w.more()) fetch();
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // the gradient turned back
      const float2 p = d[i], q = d[4 + i];
      const float2 minus = make_float2(-sin[i].x, -sin[i].y);
      d[i] = fma2(q, sin[i], mul2(p, cos[i]));
      d[4 + i] = fma2(p, minus, mul2(q, cos[i]));
    }
    if (s.gain) {
      float2 sq = mul2(x[0], x[0]);
#pragma unroll
      for (int i = 1; i < 8; ++i) sq = fma2(x[i], x[i], sq);
      const float r = rsqrtf(head_sum(sq.x + sq.y, a.lanes) * inv_d + a.eps);
      const float2 r2 = make_float2(r, r);
      float2 g[8];
      gains_of(gain, w, half, g);
      float2 dot = make_float2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[i] = mul2(x[i], r2);
        if (mine) acc[i] = fma2(d[i], x[i], acc[i]);  // a lane without a head may have r = inf
        d[i] = mul2(d[i], g[i]);
        dot = fma2(d[i], x[i], dot);
      }
      // lanes of no head, and those past the head's end, hold zeros (or, of no head, are not kept)
      const float mean = head_sum(dot.x + dot.y, a.lanes) * inv_d;
      const float2 minus = make_float2(-mean, -mean);
#pragma unroll
      for (int i = 0; i < 8; ++i) d[i] = mul2(fma2(x[i], minus, d[i]), r2);
    }
    if (mine) put_pairs<OUT>(to_now, half, d, a.f16_out);
  }
  if (!a.partial) return;
  // lanes of one chunk, then the CTA's warps, each in a fixed order
#pragma unroll
  for (int i = 0; i < 8; ++i)
    for (int o = a.lanes; o < 32; o <<= 1) {
      acc[i].x += __shfl_xor_sync(0xffffffffu, acc[i].x, o);
      acc[i].y += __shfl_xor_sync(0xffffffffu, acc[i].y, o);
    }
  if (w.slot == 0 && w.has) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      *reinterpret_cast<float2*>(
          &sums[threadIdx.x >> 5][(i < 4 ? 0 : half) + 8 * w.chunk + 2 * (i & 3)]) = acc[i];
  }
  __syncthreads();
  for (int c = threadIdx.x; c < a.d; c += kThreads) {
    float sum = 0.f;
#pragma unroll
    for (int v = 0; v < kWarps; ++v) sum += sums[v][c];
    a.partial[static_cast<int64_t>(blockIdx.x) * a.d + c] = sum;
  }
}

// d_gain[c] (= or +=) the sum of column c of partial [blocks of q, then of k][d]:
// a CTA has 32 columns of one of them, its warps a share of the rows each,
// joined in order.
__global__ void __launch_bounds__(1024) gain_sum_kernel(const float* partial, int q_rows,
                                                        int k_rows, int d, float* dg_q,
                                                        float* dg_k, int accumulate) {
  __shared__ float sums[32][33];
  after_previous_kernel();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per_side = (d + 31) / 32;
  const bool second = static_cast<int>(blockIdx.x) >= per_side;
  const int c = (blockIdx.x - (second ? per_side : 0)) * 32 + lane;
  const int rows = second ? k_rows : q_rows;
  const float* from = partial + (second ? static_cast<int64_t>(q_rows) * d : 0);
  float sum = 0.f;
  if (c < d) {
#pragma unroll 4
    for (int r = warp; r < rows; r += 32) sum += from[static_cast<int64_t>(r) * d + c];
  }
  sums[warp][lane] = sum;
  __syncthreads();
  if (warp) return;
  sum = 0.f;
#pragma unroll
  for (int w = 0; w < 32; ++w) sum += sums[w][lane];
  float* out = second ? dg_k : dg_q;
  if (c < d && out) out[c] = accumulate ? out[c] + sum : sum;
}

// Splits the work: lanes of a head, and the CTAs of q and k, dealt out by passes,
// a token's sines counting as one. Returns the number of CTAs.
int64_t split_work(NormArgs* a) {
  int lanes = 1, log2 = 0;
  while (lanes * 16 < a->d) {
    lanes *= 2;
    ++log2;
  }
  a->lanes = lanes;
  a->lanes_log2 = log2;
  const int per_pass = 32 / lanes;
  int64_t work[2];
  for (int i = 0; i < 2; ++i) {
    a->side[i].passes = (a->side[i].heads + per_pass - 1) / per_pass;
    work[i] = a->side[i].heads ? a->side[i].passes + 1 : 0;
  }
  const int64_t all = static_cast<int64_t>(num_sms()) * kCtasPerSm;
  int64_t total = 0;
  for (int i = 0; i < 2; ++i) {
    Side& s = a->side[i];
    const int64_t share = std::max<int64_t>(1, all * work[i] / (work[0] + work[1]));
    const int64_t steps = static_cast<int64_t>(a->tokens) * s.passes;
    s.blocks = static_cast<int>(std::min<int64_t>((steps + kWarps - 1) / kWarps, share));
    total += s.blocks;
  }
  return total;
}

const char* shape_problem(int tokens, int nh, int nkv, int d) {
  if (tokens < 0) return "tokens must be >= 0";
  if (nh < 0 || nkv < 0 || nh + static_cast<int64_t>(nkv) < 1 || nh > 4096 || nkv > 4096)
    return "n_heads and n_kv_heads must be in [0, 4096] and not both 0";
  if (d < 16 || d > 2 * kMaxHalf || d % 16) return "head_dim must be a multiple of 16 in [16, 256]";
  return nullptr;
}

constexpr char kShared[] = "an output is at the other tensor's place";

// Checks what both calls have in common and fills in the arguments.
const char* common_problem(int tokens, int nh, int nkv, int d, const rdt_heads* q,
                           const rdt_heads* k, int dtype, const float* gain_q, const float* gain_k,
                           float eps, const int32_t* positions, int axes, const int32_t* sections,
                           float theta, const rdt_heads* q_out, const rdt_heads* k_out,
                           int out_dtype, NormArgs* a, Rates* rates) {
  if (!dtype_ok(dtype) || !dtype_ok(out_dtype))
    return "dtypes must be RDT_F32, RDT_BF16 or RDT_F16";
  *a = NormArgs{};
  const rdt_heads *ins[2] = {q, k}, *outs[2] = {q_out, k_out};
  const float* gains[2] = {gain_q, gain_k};
  for (int i = 0; i < 2; ++i) {
    Side& s = a->side[i];
    s.heads = i ? nkv : nh;
    if (s.heads == 0) continue;
    if (const char* why = heads_problem(ins[i], tokens, s.heads, d, dtype_bytes(dtype), false))
      return why;
    if (const char* why = heads_problem(outs[i], tokens, s.heads, d, dtype_bytes(out_dtype), true))
      return why;
    if (ins[i]->data == outs[i]->data &&
        (dtype != out_dtype || (tokens > 1 && ins[i]->token_stride != outs[i]->token_stride) ||
         (s.heads > 1 && ins[i]->head_stride != outs[i]->head_stride)))
      return "an output at its input's place needs the input's type and strides";
    s.x = ins[i]->data;
    s.x_ts = ins[i]->token_stride;
    s.x_hs = ins[i]->head_stride;
    s.out = outs[i]->data;
    s.out_ts = outs[i]->token_stride;
    s.out_hs = outs[i]->head_stride;
    s.gain = gains[i];
  }
  if (nh && nkv &&
      (q_out->data == k_out->data || q_out->data == k->data || k_out->data == q->data))
    return kShared;
  if (!aligned4(gain_q) || !aligned4(gain_k) || !aligned4(positions))
    return "gains and positions must be 4-byte aligned";
  if (!(eps >= 0.f) || std::isinf(eps)) return "eps must be finite and >= 0";
  *rates = Rates{};
  if (positions) {
    if (axes < 1 || axes > 4) return "axes must be in [1, 4]";
    if (!(theta > 0.f) || std::isinf(theta)) return "theta must be finite and > 0";
    if (axes > 1 && !sections) return "sections are needed with more than one axis";
    if (sections) {
      int sum = 0;
      for (int i = 0; i < axes; ++i) {
        if (sections[i] < 0 || sections[i] > d) return "a section must be in [0, head_dim / 2]";
        for (int pair = sum; pair < sum + sections[i] && pair < d / 2; ++pair)
          rates->axis[pair] = static_cast<uint8_t>(i);
        sum += sections[i];
      }
      if (sum != d / 2) return "sections must add up to head_dim / 2";
    }
    // theta^(-2i/d) as a product of two powers: 16 of them, not 64, for a head of 128
    double coarse[kMaxHalf / 8], fine[8];
    for (int i = 0; i < 8; ++i)
      fine[i] = std::pow(static_cast<double>(theta), -2.0 * i / d) / 6.283185307179586477;
    for (int i = 0; i < d / 16; ++i)
      coarse[i] = std::pow(static_cast<double>(theta), -16.0 * i / d);
    for (int i = 0; i < d / 2; ++i) {
      const double turns = coarse[i / 8] * fine[i % 8];
      // whole turns of a position change nothing; 2^64 itself would not fit
      rates->turn[i] = static_cast<uint64_t>(std::ldexp(turns - std::floor(turns), 63)) * 2;
    }
  }
  a->eps = eps;
  a->positions = positions;
  a->axes = positions ? axes : 0;
  a->tokens = tokens;
  a->d = d;
  a->f16_in = dtype == RDT_F16;
  a->f16_out = out_dtype == RDT_F16;
  return nullptr;
}

template <int IN>
cudaError_t launch_norm(NormArgs a, int out_dtype, const Rates& r, cudaStream_t s) {
  const int64_t grid = split_work(&a);
  return out_dtype == RDT_F32
             ? launch_overlapping(norm_rope_kernel<IN, 4, 4 / IN>, grid, kThreads, 0, s, a, r)
             : launch_overlapping(norm_rope_kernel<IN, 2, 4 / IN>, grid, kThreads, 0, s, a, r);
}

template <int G, int IN>
cudaError_t launch_grad(const NormArgs& a, int out_dtype, int64_t grid, const Rates& r,
                        cudaStream_t s) {
  return out_dtype == RDT_F32
             ? launch_overlapping(norm_rope_grad_kernel<G, IN, 4>, grid, kThreads, 0, s, a, r)
             : launch_overlapping(norm_rope_grad_kernel<G, IN, 2>, grid, kThreads, 0, s, a, r);
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
  return launched(dtype == RDT_F32 ? launch_norm<4>(a, out_dtype, r, s)
                                   : launch_norm<2>(a, out_dtype, r, s));
}

size_t rdt_qk_norm_rope_backward_workspace_bytes(int32_t tokens, int32_t n_heads,
                                                 int32_t n_kv_heads, int32_t head_dim) {
  if (shape_problem(tokens, n_heads, n_kv_heads, head_dim) || tokens == 0) return 0;
  NormArgs a = {};
  a.tokens = tokens;
  a.side[0].heads = n_heads;
  a.side[1].heads = n_kv_heads;
  a.d = head_dim;
  return static_cast<size_t>(split_work(&a)) * head_dim * sizeof(float);
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
  NormArgs a;
  Rates r;
  if (const char* why = common_problem(tokens, n_heads, n_kv_heads, head_dim, q, k, dtype, gain_q,
                                       gain_k, eps, positions, axes, sections, theta, dq, dk,
                                       out_dtype, &a, &r))
    return refuse(why);
  for (int i = 0; i < 2; ++i) {
    const rdt_heads *g = i ? d_k_out : d_q_out, *o = i ? dk : dq;
    Side& side = a.side[i];
    if (side.heads == 0) continue;
    if (const char* why =
            heads_problem(g, tokens, side.heads, head_dim, dtype_bytes(d_dtype), false))
      return refuse(why);
    if (g->data == o->data &&
        (d_dtype != out_dtype || (tokens > 1 && g->token_stride != o->token_stride) ||
         (side.heads > 1 && g->head_stride != o->head_stride)))
      return refuse("an output at its input's place needs the input's type and strides");
    side.dy = g->data;
    side.dy_ts = g->token_stride;
    side.dy_hs = g->head_stride;
  }
  if (n_heads && n_kv_heads && (dq->data == d_k_out->data || dk->data == d_q_out->data))
    return refuse(kShared);
  a.f16_dy = d_dtype == RDT_F16;
  const int64_t grid = split_work(&a);
  const bool sums = d_gain_q || d_gain_k;
  if (sums) {
    if (!ws) return refuse("null pointer");
    if (reinterpret_cast<uintptr_t>(ws) & 255) return refuse("ws must be 256-byte aligned");
    if (ws_bytes < static_cast<size_t>(grid) * head_dim * sizeof(float))
      return refuse("workspace too small");
    a.partial = static_cast<float*>(ws);
  }
  const bool wide_g = d_dtype == RDT_F32, wide_x = dtype == RDT_F32;
  cudaError_t e = wide_g ? (wide_x ? launch_grad<4, 4>(a, out_dtype, grid, r, s)
                                   : launch_grad<4, 2>(a, out_dtype, grid, r, s))
                         : (wide_x ? launch_grad<2, 4>(a, out_dtype, grid, r, s)
                                   : launch_grad<2, 2>(a, out_dtype, grid, r, s));
  if (e == cudaSuccess && sums)
    e = launch_overlapping(gain_sum_kernel, 2 * ((head_dim + 31) / 32), 1024, 0, s, a.partial,
                           a.side[0].blocks, a.side[1].blocks, head_dim, d_gain_q, d_gain_k,
                           accumulate ? 1 : 0);
  return launched(e);
}

}  // extern "C"
