// Forward pass of the attention over spans of keys on the 5th-generation
// tensor cores: S = Q K^T and O += P V by tcgen05.mma with accumulators in
// TMEM, operands by TMA, softmax in registers.
//
// One CTA of the grid for each work item; a CTA that runs takes the items of
// those that have not started, one after the other, so that short and long
// spans even out over the SMs. An item is two tiles (A, B) of 128 rows of one
// key head (spans.cuh) that share their K and V tiles of 128 keys. The key
// tiles start at the least key that a row of the item sees, wherever that is.
// Warps: 0 loads (and finds each item's spans, a few items ahead of the
// others), 1 issues the MMAs, 4-7 and 8-11 are the softmax of tile A and B,
// one thread a row. The MMA warp interleaves
//   S_A(0) S_B(0) | PV_A(0) S_A(1) | PV_B(0) S_B(1) | PV_A(1) ...
// so that one tile's products run while the other's softmax does. P (bf16) is
// written over its S in TMEM (next to it, for heads up to 64) and read from
// there; its first 64 keys are handed over while the exponentials of the others
// are formed. O is rescaled only
// when a row's maximum grows by more than 2^8.
//
// A row whose O is not finite, though its sum is, may owe that to a NaN or infinity in
// a value that it does not see, times p = 0. Its item is taken once more with the
// values cleared that none of its rows sees (spans.cuh); a row that is not finite then,
// though all it sees is, is computed key by key (row_forward, 16 us for 32 keys). 4096
// packed tokens of which the unused end is NaN: 54 us, without 42. Parts of keys leave
// that to the join: 1 token against 32,700 keys, NaN behind them, 130 us, without 36.
//
// Bound by the softmax: over all 1850 cycles for 128 x 128 scores, whose two products
// take 1400; 2700 where rows begin or end in the key tile. 8192 tokens of 32 / 8 heads
// of 128, a quarter of them a prefix: 405 us (0.76 of 1890 TFLOP/s); 4096 in documents
// up to 1024: 42 us, bound by masked tiles and by the starts and ends of short items (2 us
// each); 8191 of 16 / 8 heads of 64, capped, a window of 1024: 97 us, the elementwise
// work of the cap; one token against 32,768 keys: 32 us, 4.2 TB/s, with the join.
#include <algorithm>

#include "spans.cuh"

namespace rdt {

namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kThreads = 384;
constexpr float kRescaleLog2 = 8.f;
constexpr int kItemRing = 4;
constexpr int kItemReaders = 1 + 8;  // MMA thread, softmax warps

// What the loading warp found out about an item.
struct Item {
  int index;     // of the item, with kSecond or not; -1: no more in this round
  int first;     // first key of key tile 0
  int n;         // key tiles, of both row tiles together
  int begin[2];  // key tiles [begin, end) of each row tile; begin == end: none
  int end[2];
};

struct Args {
  SpanArgs a;
  Tiling tl;
  int pairs, splits;
  Cap cap;
  float scale_log2;  // of what is exponentiated: scale log2 e, or cap log2 e
  float* part_o;     // splits > 1: fp32 [splits][queries][nh][d] and lse (base 2)
  float* part_lse;
  Patience err;
};

// The key tile where part `split` of `all` tiles begins.
__device__ __forceinline__ int first_tile(int all, int split, int splits) {
  return static_cast<int>(static_cast<int64_t>(all) * split / splits);
}

template <int D>
struct Cfg {
  static constexpr int BM = 128, BN = 128;
  static constexpr uint32_t CHUNK = 128 * 128;  // 64 columns x 128 rows of bf16
  static constexpr uint32_t TILE = 128 * D * 2;
  static constexpr int KS = D == 128 ? 2 : 4, VS = KS;
  static constexpr uint32_t OFF_Q = 0, OFF_K = OFF_Q + 2 * TILE, OFF_V = OFF_K + KS * TILE,
                            OFF_STAGE = OFF_V + VS * TILE,  // 4 KB of each softmax warp
      OFF_NEXT = OFF_STAGE + 8 * 4096, OFF_ITEM = OFF_NEXT + 16,
                            OFF_BAR = OFF_ITEM + kItemRing * sizeof(Item);
  static constexpr size_t SMEM = OFF_BAR + 512 + 1024;
  // Heads up to 64 leave columns for P apart from S: the next scores are formed
  // as soon as these are in registers.
  static constexpr bool APART = D == 64;
  static constexpr uint32_t TMEM_S = 0, TMEM_O = 256, TMEM_P = APART ? 384 : 0,
                            P_STEP = APART ? 64 : 128, TMEM_COLS = 512;
  static_assert(TMEM_O + 2 * D <= (APART ? TMEM_P : TMEM_COLS), "");
  static_assert(SMEM <= 232448 && OFF_BAR % 8 == 0, "");
};

// SPLIT: an item has a part of its keys, the sums of which it leaves in the workspace;
// else it has them all, and o is written.
template <int D, bool CAP, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
    spans_forward_kernel(const __grid_constant__ CUtensorMap tq,
                         const __grid_constant__ CUtensorMap tk,
                         const __grid_constant__ CUtensorMap tv, const __grid_constant__ Args ar) {
  using C = Cfg<D>;
  constexpr int BM = C::BM, BN = C::BN, KS = C::KS, VS = C::VS;
  const SpanArgs& a = ar.a;
  const Patience& err = ar.err;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = sbase + C::OFF_BAR;
  const uint32_t q_full = bar0, q_empty = bar0 + 16, k_full = bar0 + 32, k_empty = k_full + 8 * KS,
                 v_full = k_empty + 8 * KS, v_empty = v_full + 8 * VS, s_full = v_empty + 8 * VS,
                 p_full = s_full + 16,  // [tile][half]
      o_done = p_full + 32, o_free = o_done + 16, item_full = o_free + 16,
                 item_empty = item_full + 8 * kItemRing, drain = item_empty + 8 * kItemRing,
                 next = drain + 8, s_free = next + 8, pv_done = s_free + 16,
                 v_raw = pv_done + 16;  // V has come that is to be cleared
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_BAR + 448);
  static_assert(8 * (4 + 2 * KS + 2 * VS + 2 + 4 + 2 + 2 + 2 * kItemRing + 2 + 4 + 1) <= 448, "");
  Rounds* rounds_of = reinterpret_cast<Rounds*>(smem + C::OFF_BAR + 456);
  static_assert(456 + sizeof(Rounds) <= 512 && (C::OFF_BAR + 456) % 8 == 0, "");
  Item* ring = reinterpret_cast<Item*>(smem + C::OFF_ITEM);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int chunks = (a.d + 63) / 64;
  // item -> pair (the last queries, whose spans are often the longest, first), key head, split
  auto place = [&](int item, int& t0, int& g, int& split) {
    split = SPLIT ? item % ar.splits : 0;
    const int x = SPLIT ? item / ar.splits : item;
    g = x % a.nkv;
    t0 = (ar.pairs - 1 - x / a.nkv) * 2 * ar.tl.per;
  };

  if (threadIdx.x == 0) {
    for (int x = 0; x < KS; ++x) {
      mbar_init(k_full + 8 * x, 1);
      mbar_init(k_empty + 8 * x, 1);
      mbar_init(v_full + 8 * x, 1);
      mbar_init(v_empty + 8 * x, 1);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(q_full + 8 * x, 1);
      mbar_init(q_empty + 8 * x, 1);
      mbar_init(s_full + 8 * x, 1);
      mbar_init(p_full + 16 * x, 128);
      mbar_init(p_full + 16 * x + 8, 128);
      mbar_init(o_done + 8 * x, 1);
      mbar_init(s_free + 8 * x, 128);
      mbar_init(pv_done + 8 * x, 1);
      mbar_init(o_free + 8 * x, 128);
    }
    for (int x = 0; x < kItemRing; ++x) {
      mbar_init(item_full + 8 * x, 1);
      mbar_init(item_empty + 8 * x, kItemReaders);
    }
    mbar_init(drain, 1);
    mbar_init(next, 1);
    mbar_init(v_raw, 1);
    *rounds_of = Rounds{};
    fence_mbar_init();
    tma_prefetch_desc(&tq);
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
  if (warp < 4) {
    regs_dec<72>();
    if (warp == 0) {
      // ------------------------------------------------------- producer
      bool ok = true;
      int jg = 0, loaded = 0;  // key tiles and items with any so far
      int item = blockIdx.x;
      int ran0 = -1, ran1 = -1;  // of lane x: items x and 32 + x of the round
      uint32_t it = 0, asked = 0, raws = 0;
      do {
        const bool second = !SPLIT && redo != 0ull;
        if (lane == 0) rounds_of->start = it;
        for (int of = 0; ok; ++of, ++it) {
          const int slot = it % kItemRing;
          ok = warp_wait(item_empty + 8 * slot, ((it / kItemRing) & 1) ^ 1, err);
          if (!ok) break;
          int work = SPLIT || of < kRound ? item : -1;
          if (second) {
            const int bit = __ffsll(redo) - 1;
            work = bit < 0 ? -1
                           : __shfl_sync(0xffffffffu, bit < 32 ? ran0 : ran1, bit & 31) | kSecond;
            redo &= redo - 1;
          }
          if (work < 0) {
            if (lane == 0) {
              rounds_of->left = !SPLIT && item >= 0;
              ring[slot].index = -1;
              mbar_arrive(item_full + 8 * slot);
            }
            ++it;
            break;
          }
          int t0, g, split;
          place(work & (kSecond - 1), t0, g, split);
          int lo[2], hi[2];
          spans_of_tiles(a, ar.tl, t0, lo, hi);
          Item d;
          d.index = work;
          d.first = lo[0] >= hi[0] ? lo[1] : lo[1] >= hi[1] ? lo[0] : min(lo[0], lo[1]);
          const int all = (max(hi[0], hi[1]) - d.first + BN - 1) / BN;
          d.n = all;
          if constexpr (SPLIT) {
            const int from = first_tile(all, split, ar.splits);
            d.n = first_tile(all, split + 1, ar.splits) - from;
            d.first += from * BN;
          }
          for (int x = 0; x < 2; ++x) {
            d.begin[x] = max(0, (lo[x] - d.first) / BN);
            d.end[x] = min(d.n, (hi[x] - d.first + BN - 1) / BN);
            if (lo[x] >= hi[x] || hi[x] <= d.first || d.begin[x] >= d.end[x])
              d.begin[x] = d.end[x] = 0;
          }
          if (d.end[0] == 0 && d.end[1] == 0) d.n = 0;
          if (lane == 0) {
            ring[slot] = d;
            mbar_arrive(item_full + 8 * slot);
          }
          auto load = [&](int j, uint32_t bar, uint32_t empty, int stages, uint32_t off,
                          const CUtensorMap* map) -> bool {
            const int jj = jg + j, st = jj % stages;
            if (!mbar_wait(empty + 8 * st, ((jj / stages) & 1) ^ 1, err)) return false;
            if (!bar) bar = empty - 8 * stages + 8 * st;  // the stage's own, which lie before
            mbar_arrive_expect_tx(bar, chunks * C::CHUNK);
            for (int c = 0; c < chunks; ++c)
              tma_load_3d(sbase + off + st * C::TILE + c * C::CHUNK, map, bar, c * 64, g,
                          d.first + j * BN);
            return true;
          };
          auto load_q = [&]() -> bool {
            for (int x = 0; x < 2; ++x) {
              if (!mbar_wait(q_empty + 8 * x, (loaded & 1) ^ 1, err)) return false;
              mbar_arrive_expect_tx(q_full + 8 * x, chunks * (ar.tl.per * a.rep * 128));
              for (int c = 0; c < chunks; ++c)
                tma_load_3d(sbase + C::OFF_Q + x * C::TILE + c * C::CHUNK, &tq, q_full + 8 * x,
                            c * 64, g * a.rep, t0 + x * ar.tl.per);
            }
            return true;
          };
          if (second) {
            for (int j = 0; j < d.n && ok; ++j, ++raws) {
              if (lane == 0)
                ok = load(j, 0u, k_empty, KS, C::OFF_K, &tk) && (j > 0 || load_q()) &&
                     load(j, v_raw, v_empty, VS, C::OFF_V, &tv);
              ok = __shfl_sync(0xffffffffu, static_cast<int>(ok), 0);
              const int st = (jg + j) % VS;
              ok = ok && clear_unseen(a, t0, min(2 * ar.tl.per, a.queries - t0), d.first + j * BN,
                                      smem + C::OFF_V + st * C::TILE, v_raw, raws & 1,
                                      v_full + 8 * st, err);
            }
          } else if (d.n > 0 && lane == 0) {
            // K's first tile does not wait for the item before to be done with its Q
            ok = load(0, 0u, k_empty, KS, C::OFF_K, &tk) && load_q();
            for (int j = 1; j < KS - 1 && j < d.n && ok; ++j)
              ok = load(j, 0u, k_empty, KS, C::OFF_K, &tk);
            for (int j = 0; j < d.n && ok; ++j) {
              if (j + KS - 1 < d.n) ok = load(j + KS - 1, 0u, k_empty, KS, C::OFF_K, &tk);
              if (ok) ok = load(j, 0u, v_empty, VS, C::OFF_V, &tv);
            }
          }
          ok = __shfl_sync(0xffffffffu, static_cast<int>(ok), 0);
          if (d.n > 0) {
            jg += d.n;
            ++loaded;
          }
          if (second) continue;
          if (!SPLIT && lane == (of & 31)) (of < 32 ? ran0 : ran1) = work;
          // asked for now, not before: an item that waits here could have been another SM's
          if (lane == 0) next_cta_request(sbase + C::OFF_NEXT, next);
          // waited for on the way out too: the answer is written to this CTA's memory
          const bool answered = warp_wait(next, asked++ & 1, err);
          ok = ok && answered;
          if (ok) item = next_cta_answer(sbase + C::OFF_NEXT);
        }
        if (!ok && lane == 0) rounds_of->lost = 1;
        __syncwarp();
      } while (next_round<!SPLIT>(rounds_of, kThreads, redo));
    } else if (warp == 1) {
      // ------------------------------------------------------------ MMA
      constexpr uint32_t idesc_s = idesc_bf16_f32(BM, BN, 0, 0);
      const uint32_t idesc_o = idesc_bf16_f32(BM, a.d, 0, 1);
      const int ksteps = a.d / 16;
      bool ok = true;
      uint32_t jg = 0, loaded = 0, it = 0, drains = 0;
      uint32_t pv0 = 0, pv1 = 0, rounds0 = 0, rounds1 = 0;  // P V issued; items with any
      uint32_t s0 = 0, s1 = 0;                               // S issued
      do {
        if (elect_one()) {
          bool stop = false;
          for (; ok; ++it) {
            const int slot = it % kItemRing;
            if (!wait_for(item_full + 8 * slot, (it / kItemRing) & 1, err)) break;
            const int index = ring[slot].index, n = ring[slot].n;
            const int begin0 = ring[slot].begin[0], begin1 = ring[slot].begin[1],
                      end0 = ring[slot].end[0], end1 = ring[slot].end[1];
            mbar_arrive(item_empty + 8 * slot);
            if (index < 0) {
              ++it;
              stop = true;
              break;
            }
            if (n == 0) continue;
            // S_x = Q_x K^T of key tile j, where row tile x has any of it
            auto issue_s = [&](auto which, int j) -> bool {
              constexpr int x = decltype(which)::value;
              const int end = x ? end1 : end0;
              if (j < (x ? begin1 : begin0) || j >= end) return true;
              // else P V of the scores before, in order, comes after them
              if constexpr (C::APART) {
                uint32_t& issued = x ? s1 : s0;
                if (issued && !wait_for(s_free + 8 * x, (issued - 1) & 1, err)) return false;
                ++issued;
                tc_fence_after();
              }
              const uint32_t kd = desc_low(sbase + C::OFF_K + ((jg + j) % KS) * C::TILE, 16);
              const uint32_t qd = desc_low(sbase + C::OFF_Q + x * C::TILE, 16);
#pragma unroll
              for (int k = 0; k < D / 16; ++k) {
                if (k >= ksteps) break;
                const uint32_t off = ((k >> 2) * C::CHUNK + (k & 3) * 32) >> 4;
                tc_mma_low(tmem + C::TMEM_S + x * BN, not_hoisted(qd) + off, kd + off, idesc_s,
                           k > 0);
              }
              tc_commit(s_full + 8 * x);
              if (j + 1 == end) tc_commit(q_empty + 8 * x);  // the item's last read of its Q
              return true;
            };
            // O_x += P_x V
            auto issue_pv = [&](auto which, int j) -> bool {
              constexpr int x = decltype(which)::value;
              const int begin = x ? begin1 : begin0, end = x ? end1 : end0;
              if (j < begin || j >= end) return true;
              uint32_t& pv = x ? pv1 : pv0;
              uint32_t& rounds = x ? rounds1 : rounds0;
              if (j == begin && !wait_for(o_free + 8 * x, (rounds & 1) ^ 1, err)) return false;
              const uint32_t vd = desc_low(sbase + C::OFF_V + ((jg + j) % VS) * C::TILE, C::CHUNK);
#pragma unroll
              for (int half = 0; half < 2; ++half) {
                if (!wait_for(p_full + 16 * x + 8 * half, pv & 1, err)) return false;
                tc_fence_after();
#pragma unroll
                for (int k = 4 * half; k < 4 * half + 4; ++k)
                  tc_mma_ts_low(tmem + C::TMEM_O + x * D, tmem + C::TMEM_P + x * C::P_STEP + k * 8,
                                vd + k * 128, idesc_o, j > begin || k > 0);
              }
              ++pv;
              if constexpr (C::APART) tc_commit(pv_done + 8 * x);
              if (j + 1 == end) {
                tc_commit(o_done + 8 * x);
                ++rounds;
              }
              return true;
            };
            constexpr std::integral_constant<int, 0> A{};
            constexpr std::integral_constant<int, 1> B{};
            auto wait_k = [&](int j) {
              return wait_for(k_full + 8 * ((jg + j) % KS), ((jg + j) / KS) & 1, err);
            };
            // what is loaded is waited for even where no row tile reads it: its place is free
            // only once it is there
            ok = wait_k(0) && wait_for(q_full, loaded & 1, err);
            if (!ok) break;
            tc_fence_after();
            ok = issue_s(A, 0);
            if (end0 == 0) mbar_arrive(q_empty);
            ok = ok && wait_for(q_full + 8, loaded & 1, err);
            if (!ok) break;
            tc_fence_after();
            ok = issue_s(B, 0);
            if (end1 == 0) mbar_arrive(q_empty + 8);
            tc_commit(k_empty + 8 * (jg % KS));
            for (int j = 0; j < n && ok; ++j) {
              if constexpr (C::APART) {
                if (j + 1 < n) {
                  ok = wait_k(j + 1);
                  if (!ok) break;
                  tc_fence_after();
                  ok = issue_s(A, j + 1) && issue_s(B, j + 1);
                  if (!ok) break;
                  tc_commit(k_empty + 8 * ((jg + j + 1) % KS));
                }
                ok = wait_for(v_full + 8 * ((jg + j) % VS), ((jg + j) / VS) & 1, err) &&
                     issue_pv(A, j) && issue_pv(B, j);
                if (!ok) break;
                tc_commit(v_empty + 8 * ((jg + j) % VS));
              } else {
                ok = wait_for(v_full + 8 * ((jg + j) % VS), ((jg + j) / VS) & 1, err) &&
                     issue_pv(A, j) && (j + 1 >= n || wait_k(j + 1));
                if (!ok) break;
                tc_fence_after();
                if (j + 1 < n) issue_s(A, j + 1);
                ok = issue_pv(B, j);
                if (!ok) break;
                tc_commit(v_empty + 8 * ((jg + j) % VS));
                if (j + 1 < n) {
                  issue_s(B, j + 1);
                  tc_commit(k_empty + 8 * ((jg + j + 1) % KS));
                }
              }
            }
            jg += n;
            ++loaded;
          }
          if (!stop) rounds_of->lost = 1;
          tc_commit(drain);
          mbar_wait(drain, drains++ & 1, nullptr);
        }
        __syncwarp();
      } while (next_round<!SPLIT>(rounds_of, kThreads, redo));
    } else {
      while (next_round<!SPLIT>(rounds_of, kThreads, redo)) {
      }
    }
  } else {
    regs_inc<216>();
    // --------------------------------- softmax: one row a thread
    const int x = (warp - 4) >> 2;
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lane_base + C::TMEM_S + x * BN;
    const uint32_t tp = tmem + lane_base + C::TMEM_P + x * C::P_STEP;
    const uint32_t t_o = tmem + lane_base + C::TMEM_O + x * D;
    const int row_t = row / a.rep, row_h = row % a.rep;
    const float2 sc2 = make_float2(ar.scale_log2, ar.scale_log2);
    bool ok = true;
    int jx = 0, rounds = 0, it = 0;
    do {
      bool stop = false;
      for (; ok; ++it) {
        const int slot = it % kItemRing;
        if (!warp_wait(item_full + 8 * slot, (it / kItemRing) & 1, err)) break;
        const int item = ring[slot].index, first = ring[slot].first, begin = ring[slot].begin[x],
                  end = ring[slot].end[x];
        __syncwarp();
        if (lane == 0) mbar_arrive(item_empty + 8 * slot);
        if (item < 0) {
          ++it;
          stop = true;
          break;
        }
        // this thread's query and head; whether they exist
        auto whose = [&](int of, int& t, int& h, int& split) {
          int t0, g;
          place(of & (kSecond - 1), t0, g, split);
          t = t0 + x * ar.tl.per + row_t;
          h = g * a.rep + row_h;
          return row_t < ar.tl.per && t < a.queries;
        };
        int lo = 0, hi = INT32_MAX;  // a row that is none needs no mask
        {
          int t, h, split;
          if (whose(item, t, h, split)) a.span(t, lo, hi);
        }
        float m_run = -INFINITY, l_run = 0.f;
        for (int j = begin; j < end; ++j, ++jx) {
          if (!warp_wait(s_full + 8 * x, jx & 1, err)) {
            ok = false;
            break;
          }
          tc_fence_after();
          // columns l <= c < r are seen by this row
          const int base = first + j * BN;
          const int l = lo - base, r = hi - base;
          const bool masked = __any_sync(0xffffffffu, l > 0 || r < BN);
          // -inf where the row does not see 32 columns from q on
          auto mask = [&](uint32_t (&s)[32], int q) {
            const uint32_t seen = bits_between(l - 32 * q, r - 32 * q);
            if (__all_sync(0xffffffffu, seen == ~0u)) return;
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (!(seen & (1u << c))) s[c] = __float_as_uint(-INFINITY);
          };
          // The scores are read twice, for their maximum and for the exponentials, the
          // second time in a loop over halves. Held in registers and unrolled, they spill
          // 80 bytes and masks and all take 16 KB of instructions: 4096 packed tokens took
          // 44.5 us and not 42.7 (8192 tokens of a seen prompt, few masked tiles, 386 and
          // not 404).
          bool far = false;  // a score beyond the cap's polynomial
          float mx;
          if (!masked) {
            uint32_t sv[128];
#pragma unroll
            for (int c = 0; c < 4; ++c)
              tmem_ld32(ts + c * 32, *reinterpret_cast<uint32_t(*)[32]>(&sv[32 * c]));
            tmem_ld_wait();
            Reach reach;
#pragma unroll
            for (int c = 0; c < 128; c += 2)
              reach.take<CAP>(
                  make_float2(__uint_as_float(sv[c]), __uint_as_float(sv[c + 1])), (c >> 1) & 1);
            mx = reach.top();
            if constexpr (CAP) far = reach.beyond(ar.cap.limit);
          } else {
            Reach all, own;
#pragma unroll 1
            for (int q = 0; q < 4; ++q) {
              uint32_t sv[32];
              tmem_ld32(ts + 32 * q, sv);
              tmem_ld_wait();
              if constexpr (CAP) {
#pragma unroll
                for (int c = 0; c < 32; c += 2)
                  all.take<true>(make_float2(__uint_as_float(sv[c]), __uint_as_float(sv[c + 1])),
                                 (c >> 1) & 1);
              }
              mask(sv, q);
#pragma unroll
              for (int c = 0; c < 32; c += 2)
                own.take<false>(make_float2(__uint_as_float(sv[c]), __uint_as_float(sv[c + 1])),
                                (c >> 1) & 1);
            }
            mx = own.top();
            if constexpr (CAP) far = all.beyond(ar.cap.limit);
          }
          uint32_t near[2][32];
          auto fetch = [&](int half) {
            tmem_ld32(ts + 64 * half, near[0]);
            tmem_ld32(ts + 64 * half + 32, near[1]);
          };
          fetch(0);
          // what is exponentiated, in base 2, rises with the score
          if (!CAP)
            mx *= ar.scale_log2;
          else if (mx != -INFINITY)
            mx = far && fabsf(mx) > ar.cap.limit ? ar.scale_log2 * tanhf(ar.cap.w * mx)
                                                 : mx * odd_factor(both(mx), ar.cap.z).x;
          float alpha = 1.f;
          if (mx > m_run + kRescaleLog2) {
            alpha = m_run == -INFINITY ? 1.f : ex2_approx(m_run - mx);  // nothing summed: as it is
            m_run = mx;
          }
          if constexpr (C::APART) {  // P of the tile before has been read, and added to O
            if (jx > 0 && !warp_wait(pv_done + 8 * x, (jx - 1) & 1, err)) {
              ok = false;
              break;
            }
            tc_fence_after();
          }
          if (__any_sync(0xffffffffu, alpha != 1.f)) {
            // the products so far have completed: else the scores were issued after them
#pragma unroll 1
            for (int c = 0; c < a.d; c += 16) {
              uint32_t ov[16];
              tmem_ld16(t_o + c, ov);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 16; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
              tmem_st16(t_o + c, ov);
            }
          }
          const float nm = m_run == -INFINITY ? 0.f : -m_run;
          const float2 nm2 = make_float2(nm, nm);
          float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll 1
          for (int half = 0; half < 2; ++half) {
            uint32_t pk[32];  // 64 keys as bf16 pairs
            tmem_ld_wait();
            if (C::APART && half) {
              tc_fence_before();
              mbar_arrive(s_free + 8 * x);
            }
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              uint32_t(&s)[32] = near[q];
              auto exps = [&](auto ready) {
#pragma unroll
                for (int c = 0; c < 32; c += 2) {
                  float2 p = make_float2(__uint_as_float(s[c]), __uint_as_float(s[c + 1]));
                  if constexpr (!decltype(ready)::value)
                    p = fma2(p, CAP ? odd_factor(p, ar.cap.z) : sc2, nm2);
                  p.x = ex2_approx(p.x);
                  p.y = ex2_approx(p.y);
                  sum[(c >> 1) & 1] = add2(sum[(c >> 1) & 1], p);
                  pk[16 * q + c / 2] = pack_bf16x2(p.x, p.y);
                }
              };
              if (!masked && !far) {
                exps(std::false_type{});
                continue;
              }
              // to base 2, less the maximum, and masked first
              if (CAP && far) {
#pragma unroll
                // a score by itself decides, not what its warp holds
                for (int c = 0; c < 32; ++c) {
                  const float u = __uint_as_float(s[c]);
                  const float z = fabsf(u) > ar.cap.limit
                                      ? fmaf(ar.scale_log2, tanhf(ar.cap.w * u), nm)
                                      : fmaf(u, odd_factor(both(u), ar.cap.z).x, nm);
                  s[c] = __float_as_uint(z);
                }
              } else {
#pragma unroll
                for (int c = 0; c < 32; c += 2) {
                  const float2 u = make_float2(__uint_as_float(s[c]), __uint_as_float(s[c + 1]));
                  const float2 z = fma2(u, CAP ? odd_factor(u, ar.cap.z) : sc2, nm2);
                  s[c] = __float_as_uint(z.x);
                  s[c + 1] = __float_as_uint(z.y);
                }
              }
              mask(s, 2 * half + q);
              exps(std::true_type{});
            }
            if (half == 0) fetch(1);
            tmem_st32(tp + 32 * half, pk);
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive(p_full + 16 * x + 8 * half);
          }
          const float2 two = add2(sum[0], sum[1]);
          l_run = l_run * alpha + (two.x + two.y);
        }
        if (!ok) break;
        if (begin < end) {
          if (!warp_wait(o_done + 8 * x, rounds & 1, err)) break;
          tc_fence_after();
          ++rounds;
        }
        int t, h, split;  // found again: registers are short between
        const bool real = whose(not_hoisted(item), t, h, split);
        const int64_t th = static_cast<int64_t>(t) * a.nh + h;
        const float inv = l_run != 0.f ? 1.f / l_run : 0.f;
        const bool some = l_run != 0.f;  // else p was 0 throughout: 0 times what was not seen
        float bad = 0.f;
        // A thread's row goes through shared memory, so that a store takes whole
        // 128-byte pieces of rows; 64 columns a round.
        bf16* const own = real ? a.o.at(t, h) : nullptr;
        uint8_t* stage = smem + C::OFF_STAGE + (warp - 4) * 4096;
        const bool any = __any_sync(0xffffffffu, real);
#pragma unroll 1
        for (int c0 = 0; any && c0 < a.d; c0 += 64) {
          uint32_t ov[64];
          if (begin < end) {
            tmem_ld32(t_o + c0, *reinterpret_cast<uint32_t(*)[32]>(&ov[0]));
            tmem_ld32(t_o + c0 + 32, *reinterpret_cast<uint32_t(*)[32]>(&ov[32]));
            tmem_ld_wait();
          }
          const int left = a.d - c0;
          float2 worst[2] = {both(0.f), both(0.f)};
#pragma unroll
          for (int e = 0; e < 64; e += 2) {
            float2 v = mul2(make_float2(__uint_as_float(ov[e]), __uint_as_float(ov[e + 1])),
                            both(inv));
            if (!some) v = both(0.f);
            if (e < left) worst[(e >> 1) & 1] = fma2(v, both(0.f), worst[(e >> 1) & 1]);
            ov[e] = __float_as_uint(v.x);
            ov[e + 1] = __float_as_uint(v.y);
          }
          bad += (worst[0].x + worst[0].y) + (worst[1].x + worst[1].y);
          if constexpr (SPLIT) {
            float* out =
                ar.part_o + (static_cast<int64_t>(split) * a.queries * a.nh + th) * a.d + c0;
#pragma unroll
            for (int e = 0; e < 64; e += 4)
              if (real && e < left)
                *reinterpret_cast<uint4*>(out + e) =
                    make_uint4(ov[e], ov[e + 1], ov[e + 2], ov[e + 3]);
            continue;
          }
          __syncwarp();
#pragma unroll
          for (int e = 0; e < 8; ++e) {  // 16-byte piece e of the row, where it spreads banks
            uint32_t two[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              two[i] = pack_bf16x2(__uint_as_float(ov[8 * e + 2 * i]),
                                   __uint_as_float(ov[8 * e + 2 * i + 1]));
            *reinterpret_cast<uint4*>(stage + lane * 128 + ((e ^ (lane & 7)) << 4)) =
                make_uint4(two[0], two[1], two[2], two[3]);
          }
          __syncwarp();
          const int piece = lane & 7;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int from = 4 * i + (lane >> 3);
            bf16* const row_at = reinterpret_cast<bf16*>(
                __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(own), from));
            const uint4 w =
                *reinterpret_cast<const uint4*>(stage + from * 128 + ((piece ^ (from & 7)) << 4));
            if (row_at && 8 * piece < left) *reinterpret_cast<uint4*>(row_at + c0 + 8 * piece) = w;
          }
        }
        if (begin < end) {  // this O is free for the next item
          tc_fence_before();
          mbar_arrive(o_free + 8 * x);
        }
        const float lse2 = l_run != 0.f ? m_run + log2f(l_run) : -INFINITY;
        if (real) {
          if (SPLIT)
            ar.part_lse[static_cast<int64_t>(split) * a.queries * a.nh + th] = lse2;
          else if (a.lse)
            a.lse[th] = lse2 * kLn2;
        }
        const bool mine = !SPLIT && real && bad != 0.f && l_run == l_run;
        if (__any_sync(0xffffffffu, mine)) {
          if (!(item & kSecond)) {
            if (lane == 0) take_again(rounds_of, it);
          } else {
            forward_again(a, (not_hoisted(item) & (kSecond - 1)) % a.nkv, mine ? t : -1, h);
          }
        }
      }
      if (!stop && lane == 0) rounds_of->lost = 1;
      tc_fence_before();
    } while (next_round<!SPLIT>(rounds_of, kThreads, redo));
  }

  // the last round's end has been waited for by all
  if (err.err && *reinterpret_cast<volatile int*>(err.err) != 0) {
    // after a timed-out wait, copies issued just before may still be landing
    // in this CTA's shared memory: let them finish before it exits
    const uint64_t w0 = global_timer_ns();
    while (global_timer_ns() - w0 < 200000ull) {
    }
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

// Joins the splits of a row: o = sum_s w_s o_s, w_s = 2^(lse_s - lse). One CTA a
// row, its warps share the splits, a lane has four columns; fixed order. Bound by
// the latency of its start and of two loads, one behind the other where the first
// parts waited for their weights (1 query, 1024 keys: 9.4 us in all and not 8.9).
// A part whose o is not finite though its lse is may owe that to values that the row
// does not see: its sum is formed again from the keys that the row sees of it, by all
// warps, groups of 2 to 16 lanes a key and four keys of a group under way at a time.
constexpr int kJoinWarps = 4, kJoinAhead = 5, kJoinKeys = 4;
__global__ void __launch_bounds__(32 * kJoinWarps) join_kernel(const __grid_constant__ Args ar) {
  __shared__ float sums[kJoinWarps][kMaxDim];
  __shared__ float weight[1024];
  __shared__ int bad;  // a warp's share of the sum is not finite
  const SpanArgs& a = ar.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t rows = static_cast<int64_t>(a.queries) * a.nh, th = blockIdx.x;
  after_previous_kernel();
  auto part = [&](int s) {
    return *reinterpret_cast<const float4*>(ar.part_o + (s * rows + th) * a.d + 4 * lane);
  };
  float4 ahead[kJoinAhead];  // these loads do not wait for the weights
#pragma unroll
  for (int i = 0; i < kJoinAhead; ++i)
    if (warp + i * kJoinWarps < ar.splits && 4 * lane < a.d) ahead[i] = part(warp + i * kJoinWarps);
  float top = -INFINITY;
  for (int s = lane; s < ar.splits; s += 32) top = fmaxf(top, ar.part_lse[s * rows + th]);
  top = warp_max(top);
  float total = 0.f;
  for (int s = lane; s < ar.splits; s += 32) {
    const float lse = ar.part_lse[s * rows + th];
    const float w = lse == -INFINITY ? 0.f : ex2_approx(lse - top);
    if (warp == 0) weight[s] = w;
    total += w;
  }
  total = warp_sum(total);
  if (threadIdx.x == 0) bad = 0;
  __syncthreads();
  float acc[4] = {};
  auto add = [&](int s, float4 o) {
    const float w = weight[s];
    if (w == 0.f) return;
    acc[0] = fmaf(w, o.x, acc[0]);
    acc[1] = fmaf(w, o.y, acc[1]);
    acc[2] = fmaf(w, o.z, acc[2]);
    acc[3] = fmaf(w, o.w, acc[3]);
  };
  if (4 * lane < a.d) {
#pragma unroll
    for (int i = 0; i < kJoinAhead; ++i)
      if (warp + i * kJoinWarps < ar.splits) add(warp + i * kJoinWarps, ahead[i]);
    for (int s = warp + kJoinAhead * kJoinWarps; s < ar.splits; s += kJoinWarps) add(s, part(s));
    float worst = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      sums[warp][4 * lane + i] = acc[i];
      worst = fmaf(acc[i], 0.f, worst);
    }
    if (worst != 0.f) bad = 1;
  }
  __syncthreads();
  const int t = static_cast<int>(th / a.nh), h = static_cast<int>(th % a.nh);
  auto finish = [&]() {
    if (warp || 4 * lane >= a.d) return;
    float o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o[i] = sums[0][4 * lane + i];
#pragma unroll
      for (int w = 1; w < kJoinWarps; ++w) o[i] += sums[w][4 * lane + i];
      o[i] = total != 0.f ? o[i] / total : 0.f;
    }
    *reinterpret_cast<uint2*>(a.o.at(t, h) + 4 * lane) =
        make_uint2(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]));
  };
  finish();
  if (threadIdx.x == 0 && a.lse)
    a.lse[th] = total != 0.f ? (top + log2f(total)) * kLn2 : -INFINITY;
  if (!bad || total != total) return;  // the same in each warp
  __syncthreads();  // the sums have been read
  auto finite = [](float4 o) {
    return fabsf(o.x) < INFINITY && fabsf(o.y) < INFINITY && fabsf(o.z) < INFINITY &&
           fabsf(o.w) < INFINITY;
  };
  // the other parts as they are
#pragma unroll
  for (int i = 0; i < 4; ++i) acc[i] = 0.f;
  for (int s = warp; s < ar.splits; s += kJoinWarps) {
    const float4 o = 4 * lane < a.d ? part(s) : make_float4(0.f, 0.f, 0.f, 0.f);
    if (__all_sync(0xffffffffu, finite(o))) add(s, o);
  }
  if (4 * lane < a.d)
#pragma unroll
    for (int i = 0; i < 4; ++i) sums[warp][4 * lane + i] = acc[i];
  // the parts' keys, as their items found them
  const int t0 = t / (2 * ar.tl.per) * (2 * ar.tl.per), g = h / a.rep;
  int lo[2], hi[2], row_first, row_end;
  spans_of_tiles(a, ar.tl, t0, lo, hi);
  a.span(t, row_first, row_end);
  const int first = lo[0] >= hi[0] ? lo[1] : lo[1] >= hi[1] ? lo[0] : min(lo[0], lo[1]);
  const int all = (max(hi[0], hi[1]) - first + 127) / 128;
  const int lanes = a.d <= 16 ? 2 : a.d <= 32 ? 4 : a.d <= 64 ? 8 : 16, groups = 32 / lanes;
  const int column = 8 * (lane & (lanes - 1)), group = lane / lanes;
  const bool has = column < a.d;
  auto eight = [&](const bf16* row, bool there) {
    Eight e;
    e.a = make_uint4(0u, 0u, 0u, 0u);
    if (has && there) e.load(row + column);
    return e;
  };
  float q[8], sum[8] = {};
  eight(a.q.at(t, h), true).get(q);
  for (int s = 0; s < ar.splits; ++s) {
    const float4 o = 4 * lane < a.d ? part(s) : make_float4(0.f, 0.f, 0.f, 0.f);
    if (weight[s] == 0.f || __all_sync(0xffffffffu, finite(o))) continue;
    const int from = max(row_first, first + first_tile(all, s, ar.splits) * 128),
              to = min(row_end, first + first_tile(all, s + 1, ar.splits) * 128);
    const int step = kJoinKeys * groups;
    for (int64_t base = from + warp * step; base < to; base += kJoinWarps * step) {
      Eight k[kJoinKeys], v[kJoinKeys];
#pragma unroll
      for (int u = 0; u < kJoinKeys; ++u) {
        const int64_t j = base + u * groups + group;
        k[u] = eight(a.k.at(j, g), j < to);
        v[u] = eight(a.v.at(j, g), j < to);
      }
#pragma unroll
      for (int u = 0; u < kJoinKeys; ++u) {
        float x[8], dot = 0.f, slope;
        k[u].get(x);
#pragma unroll
        for (int i = 0; i < 8; ++i) dot = fmaf(q[i], x[i], dot);
        for (int i = lanes >> 1; i > 0; i >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, i);
        const bool there = base + u * groups + group < to;
        const float p = there ? exp2f(score_of(a, dot, slope) * kLog2e - top) : 0.f;
        v[u].get(x);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[i] = fmaf(p, x[i], sum[i]);
      }
    }
  }
  __syncwarp();  // this warp's sums so far
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    for (int x = lanes; x < 32; x <<= 1) sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], x);
    if (group == 0 && has) sums[warp][column + i] += sum[i];
  }
  __syncthreads();
  finish();
}

// Keys are split where items leave SMs idle, unless joining the rows takes longer
// than the key tiles that are saved: the join as long as two tiles, and one more for
// every 640 rows. Heads 32 / 8 of 128, split into single tiles / not: 1 query and 2
// tiles 8.7 / 8.0 us, 4 tiles 8.5 / 10.8, 8 tiles 8.9 / 16.4; 64 queries and 4 tiles 15.9 /
// 12.4, 8 tiles 16.6 / 18.8; 128 queries and 8 tiles 20.1 / 19.0, 16 tiles 22.0 / 30.9.
// As few parts as keep the longest as short (1 query, 8192 keys: 16 parts of four
// tiles 13.9 us, 19 of three or four 15.5).
constexpr int kRowsOfTile = 640;

template <int D, bool CAP, bool SPLIT>
cudaError_t launch(const Args& ar, cudaStream_t s) {
  const SpanArgs& a = ar.a;
  CUtensorMap tq, tk, tv;
  if (!make_tma_heads(&tq, a.q.p, a.queries, a.nh, a.d, a.q.ts, a.q.hs, a.rep, ar.tl.per) ||
      !make_tma_heads(&tk, a.k.p, a.keys, a.nkv, a.d, a.k.ts, a.k.hs, 1, 128) ||
      !make_tma_heads(&tv, a.v.p, a.keys, a.nkv, a.d, a.v.ts, a.v.hs, 1, 128))
    return cudaErrorInvalidValue;
  constexpr auto kernel = spans_forward_kernel<D, CAP, SPLIT>;
  const cudaError_t e = allow_smem<kernel>(Cfg<D>::SMEM);
  if (e != cudaSuccess) return e;
  return launch_overlapping(kernel, static_cast<int64_t>(ar.pairs) * a.nkv * ar.splits, kThreads,
                            Cfg<D>::SMEM, s, tq, tk, tv, ar);
}
template <int D, bool CAP>
cudaError_t launch(const Args& ar, cudaStream_t s) {
  return ar.splits > 1 ? launch<D, CAP, true>(ar, s) : launch<D, CAP, false>(ar, s);
}

}  // namespace

int forward_splits(int queries, int keys, int nkv, int rep) {
  const Tiling tl = Tiling::of(queries, rep);
  const int64_t items = static_cast<int64_t>((tl.tiles + 1) / 2) * nkv;
  if (items < 1) return 1;
  const int64_t tiles = (keys + 127) / 128, most = num_sms() / items;
  const int64_t rows = static_cast<int64_t>(queries) * nkv * rep;
  if (most < 2 || (tiles - 2) * kRowsOfTile < rows) return 1;
  const int64_t each = (tiles + most - 1) / most;
  return static_cast<int>((tiles + each - 1) / each);
}

size_t forward_workspace(int queries, int keys, int nh, int nkv, int d) {
  const int splits = forward_splits(queries, keys, nkv, nh / nkv);
  return splits == 1 ? 0 : static_cast<size_t>(splits) * queries * nh * (d + 1) * sizeof(float);
}

cudaError_t forward_tiles(const SpanArgs& a, void* ws, cudaStream_t s) {
  Args ar = {};
  ar.a = a;
  ar.tl = Tiling::of(a.queries, a.rep);
  ar.pairs = (ar.tl.tiles + 1) / 2;
  ar.splits = forward_splits(a.queries, a.keys, a.nkv, a.rep);
  ar.cap = cap_of(a.scale, a.cap);
  ar.scale_log2 = (a.cap > 0.f ? a.cap : a.scale) * kLog2e;
  const int64_t rows = static_cast<int64_t>(a.queries) * a.nh;
  ar.part_o = static_cast<float*>(ws);
  ar.part_lse = ar.part_o + ar.splits * rows * a.d;
  ar.err = {device_error_ptr(), kWaitLimitNs + kNsOfKey * a.keys};
  cudaError_t e;
  if (a.d <= 64)
    e = a.cap > 0.f ? launch<64, true>(ar, s) : launch<64, false>(ar, s);
  else
    e = a.cap > 0.f ? launch<128, true>(ar, s) : launch<128, false>(ar, s);
  if (e != cudaSuccess || ar.splits == 1) return e;
  return launch_overlapping(join_kernel, rows, 32 * kJoinWarps, 0, s, ar);
}

}  // namespace rdt
