// Cross attention over a paged cache: every new token of a request attends to
// all of the request's stored keys (an encoder's states: another length, no
// causal mask),
//     out[t][h] = softmax_j(scale * q[t][h] . K[j]) . V[j],   0 <= j < kv_len.
//
// Work.  A query row is (token, head of the KV head's group); an item is (request,
// KV head, up to 256 of its rows), its keys in tiles of 128.  An item of more than
// 128 rows is wide: two row tiles share every key tile, one per softmax group.  An
// item of at most 128 rows (a decoding step, a few beams) is narrow: one row tile,
// and the two groups take the key tiles in turn, so that one's softmax runs beside
// the other's products; their results are joined at the item's end.  All items' key
// tiles, in order, are cut into equal ranges, one per CTA of a persistent grid:
// whatever the batch looks like, every SM streams the same share.  An item that a
// boundary cuts leaves partial results (running max, sum, O), and the CTAs that
// share it join them, each its part of the rows, after their last tile.  They
// wait for each other there, so the launch is cooperative.
//
// Tensor memory (512 columns): S_A|P_A [0,128), S_B|P_B [128,256), O_A, O_B.  P
// (bf16) is written over its own S and is the A operand of O += P V.
//
// A batch whose items have few rows (at most 32: a decoding step, a few beams) takes another
// form of the softmax, in which four warps share each row's keys: softmax_few.
//
// Warps 0-3, 4-7: softmax of group A, B (thread = row); warp 8: TMA loads of Q, K
// and V; warps 9, 10: MMA issue for A, B; one more completes the third warpgroup, which
// gives most of its registers to the other two: a row's 128 scores stay in registers.
// Scores, running max (base 2, scale folded in), sums and O are fp32; the weights are
// rounded to bf16 for the tensor cores (within 2^-8 of each, as the output is of itself)
// and summed before that rounding.  Every wait is bounded; the four warps that meet at a named
// barrier agree there on whether one of them has given up.
//
// Measured (a recorded graph, 6788 GB/s copy rate, 1899 TFLOP/s of a library's product),
// head dimension 128: 48 tokens over 256-8192 keys, 32/8 heads, 142 to 144 us = 0.94 of the
// copy rate; 64 x 4 beams over 512-4096 keys, 32/32 heads, 376 to 382 us = 0.99: HBM bounds both.
// Prompts of 1999, 1203, 515 tokens over 9001, 2500, 777 keys, 32/8 heads, 266 us = 1.32
// PFLOP/s: the chain scores - weights - product of each group bounds them.  Head dimension
// 64, 100 single tokens over 100-3000 keys: 32/32 heads 189 to 192 us = 0.91 to 0.92,
// 32/8 heads 59.5 us = 0.73, of which the launch's start and the joins at its end are 8.
#include <algorithm>
#include <cstddef>

#include "../../include/cbattn.h"
#include "cb_common.cuh"

namespace cb {

namespace {

constexpr int kThreads = 384;
constexpr int kRows = 256;             // of a wide item
constexpr float kNoKey = -__builtin_huge_valf();
constexpr float kMostSum = 1024.f;     // of a tile's weights: none of them is over 2^10
// A weight's exponent is s sl2 - m with one rounding, and m the rounded s sl2 of the largest score: there the
// exponent is what that rounding took, at most 8 for m below this.  Farther out it could be any power of two, and
// every weight or none would pass fp32; see centre.
constexpr float kFar = 268435456.f;    // 2^28

// Cost of a key tile of a narrow and of a wide item, and of an item's start and end (its
// query tile's load, its output), which take as long as one and a half tiles of a wide
// item.  Four prompts of 5 to 1999 tokens: 307 us with a start counted as half a tile of
// a wide item, 295 as one, 265 as one and a half, 270 as two; 64 x 4 beams: 374, 375, 376,
// 379; 100 tokens over 100 to 3000 keys of dimension 64, 32 heads: 198, 186, 189, 194.
constexpr int kNarrow = 2, kWide = 4, kLead = 6;
constexpr int kLeast = 8;              // of a CTA's share

// K and V tiles share one ring of buffers, in the order of their use: a wide item's
// K(0) V(0) K(1) V(1) .., a narrow one's K(0) K(1) V(0) K(2) V(1) .. V(n - 1), since
// its two groups begin with a key tile each.
// F: a launch whose items have at most kFewRows rows; see softmax_few.
constexpr int kFewRows = 32;
template <int A, bool F>
struct Tiles {
  static constexpr int kHalves = A / 64;
  static constexpr int kHalfBytes = 128 * 128;
  static constexpr int kBytes = kHalves * kHalfBytes;     // of 128 rows
  static constexpr int kRing = A == 128 ? 5 : 10;
  // With few rows of dimension 128 there is room for one query tile beside the ring.  Four buffers
  // and two query tiles: 48 tokens over 256-8192 keys 146.8 us, 143.7 so, and 64 x 4 beams 391
  // and 382.
  static constexpr int kQ = A == 128 && F ? 1 : 2;
  static constexpr int kFewHalf = kFewRows * 128, kFewGroup = 2 * kFewHalf;
  uint8_t q[kQ][kHalves][128][128];
  uint8_t weights[F ? 2 : 0][2][kFewRows][128];           // the products read 128 rows, that is, into kv
  float2 top[F ? 2 : 0][4][kFewRows];  // per group, warp and row: the maximum, and whether m must move up
  float sum[F ? 2 : 0][4][kFewRows];   // of a row's weights
  uint8_t kv[kRing][kHalves][128][128];
};

// A request's tokens and stored keys; q_len 0: nothing to do.
struct Request {
  int q0, q_len, kv;
};

// A CTA's part of an item: key tiles [ta, tb) of [0, tiles).
struct Part {
  Request q;
  int r, g, tok_lo, tokens, tiles, ta, tb;
  int at, step;                        // unit of tile 0, units per tile
  bool two_row_tiles;
  __device__ __forceinline__ bool whole() const { return ta == 0 && tb == tiles; }
};

// Whether a launch can have wide items (W) is known to the compiler.  Where it cannot, the
// softmax's code is shorter (100 requests of one token and up to 3000 keys of dimension 64:
// 83 us without that, 78.5 with it); and partial results have another order: see join_rows.
template <bool W>
struct Piece : Part {
  __device__ __forceinline__ bool wide() const { return W && two_row_tiles; }
};

template <int NS>
struct alignas(16) Ctl {
  uint64_t q_full[2], q_empty[2];
  uint64_t full[NS], empty[NS];
  uint64_t s_full[2], p_full[2], o_done[2], o_free[2];        // per group
  uint64_t ml_full;                    // ml is written
  uint64_t turn[2];                    // a wide item's products, group by group
  uint64_t drain[2];
  uint32_t tmem_base;
  volatile int abort;
  int any_empty;                       // a request has tokens and no keys
  int share, total;                    // units of a CTA's range, of all
  int start_r, start_u;                // the request that the CTA's range begins in, its first unit
  int go;
  Part cut[2];                         // pieces of cut items: begun before the CTA, by it; tiles 0: none
  long long scan[kThreads / 32];
  float2 ml[128];                      // (max, sum) of a narrow item's second group
};

// ---------------------------------------------------------------- plan
__device__ __forceinline__ Request load_request(const CrossParams& P, int r, bool report) {
  const int q0 = __ldg(P.cu_q_lens + r), q1 = __ldg(P.cu_q_lens + r + 1), kv = __ldg(P.kv_lens + r);
  const bool bad = q0 < 0 || q1 < q0 || q1 > P.n_tokens || q1 - q0 > P.max_q_len || kv < 0 || kv > P.max_kv_len ||
                   (kv + kBlockSize - 1) / kBlockSize > P.max_blocks_per_seq;
  if (bad) {
    if (report) set_error(P.err, CB_DEVERR_BADLEN);
    return {0, 0, 0};
  }
  return {q0, q1 - q0, kv};
}

// A request's items: per KV head, groups of 256 rows, the last one narrow if it
// has at most 128.
struct Shape {
  int groups, tiles, last;             // last: cost of the last group
  int full;                            // of the others
  __device__ __forceinline__ int head() const { return (groups - 1) * full + last; }
};
__device__ __forceinline__ Shape shape_of(const CrossParams& P, const Request& q) {
  const int tok = kRows >> P.group_log2;
  Shape s;
  s.groups = (q.q_len + tok - 1) / tok;
  s.tiles = (q.kv + kTileN - 1) / kTileN;
  s.full = kLead + s.tiles * kWide;
  s.last = q.q_len - (s.groups - 1) * tok > tok / 2 ? s.full : kLead + s.tiles * kNarrow;
  return s;
}

// Where this CTA's range of the units begins.  All threads; ends with a barrier.
template <class C>
__device__ void make_plan(const CrossParams& P, C& c) {
  const int n = P.n_reqs, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int seg = (n + kThreads - 1) / kThreads, lo = min(n, tid * seg), hi = min(n, lo + seg);
  long long mine = 0;
  for (int r = lo; r < hi; ++r) {
    const Request q = load_request(P, r, blockIdx.x == 0);
    if (q.q_len && q.kv) mine += (long long)shape_of(P, q).head() * P.n_kv_heads;
    if (q.q_len && !q.kv) c.any_empty = 1;
  }
  long long x = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  if (lane == 31) c.scan[warp] = x;
  __syncthreads();
  long long before = x - mine, all = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += c.scan[w];
    all += c.scan[w];
  }
  if (all >= 1LL << 30) {              // not for lengths that the host's bounds allow
    if (blockIdx.x == 0 && tid == 0) set_error(P.err, CB_DEVERR_BADLEN);
    all = 0;
  }
  const int share = max(kLeast, ((int)all + (int)gridDim.x - 1) / (int)gridDim.x);
  const long long u0 = (long long)blockIdx.x * share;
  if (tid == 0) {
    c.total = (int)all;
    c.share = share;
  }
  if (u0 < all && before <= u0 && u0 < before + mine) {
    for (int r = lo; r < hi; ++r) {
      const Request q = load_request(P, r, false);
      if (!q.q_len || !q.kv) continue;
      const int units = shape_of(P, q).head() * P.n_kv_heads;
      if (u0 < before + units) {
        c.start_r = r;
        c.start_u = (int)before;
        break;
      }
      before += units;
    }
  }
  __syncthreads();
}

// Walks a CTA's pieces in order; every role has its own.
template <bool W>
struct Pieces {
  int u0, u1, n;
  int r, g, grp, u;                    // the next item and its first unit
  Request q;
  Shape s;
  template <class C>
  __device__ Pieces(const CrossParams& P, const C& c) : n(P.n_reqs) {
    u0 = (int)min((long long)c.total, (long long)blockIdx.x * c.share);
    u1 = (int)min((long long)c.total, (long long)u0 + c.share);
    u = u1;
    if (u0 >= u1) return;
    r = c.start_r;
    open(P);
    int off = u0 - c.start_u;
    g = off / s.head();
    off -= g * s.head();
    grp = min(off / s.full, s.groups - 1);
    u = c.start_u + g * s.head() + grp * s.full;
  }
  __device__ __forceinline__ void open(const CrossParams& P) {
    q = load_request(P, r, false);
    if (q.q_len && q.kv) s = shape_of(P, q);
  }
  __device__ bool next(const CrossParams& P, Piece<W>& p) {
    while (u < u1) {
      const int tok = kRows >> P.group_log2;
      const bool last = grp == s.groups - 1;
      p.q = q;
      p.r = r;
      p.g = g;
      p.tok_lo = grp * tok;
      p.tokens = min(tok, q.q_len - p.tok_lo);
      p.two_row_tiles = p.tokens > tok / 2;
      p.tiles = s.tiles;
      p.step = p.wide() ? kWide : kNarrow;
      p.at = u + kLead;
      p.ta = min(s.tiles, max(0, u0 - p.at + p.step - 1) / p.step);
      p.tb = min(s.tiles, max(0, u1 - p.at + p.step - 1) / p.step);
      u += last ? s.last : s.full;
      if (!last) {
        ++grp;
      } else {
        grp = 0;
        if (++g == P.n_kv_heads) {
          g = 0;
          do {
            if (++r == n) break;
            open(P);
          } while (!q.q_len || !q.kv);
        }
      }
      if (p.ta < p.tb) return true;
    }
    return false;
  }
};

// ---------------------------------------------------------------- waits
__device__ __forceinline__ bool warp_wait(const CrossParams& P, uint64_t* bar, uint32_t parity) {
  const bool ok = mbar_wait(bar, parity);
  if (!ok) set_error(P.err, CB_DEVERR_TIMEOUT);
  return __all_sync(0xffffffffu, ok);
}

// True in one lane of a converged warp, the same one every time.
__device__ __forceinline__ bool elect_lane() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}

// ---------------------------------------------------------------- loads (warp 8)
// A key tile is eight blocks of 16 rows, in boxes of 64 columns: 16 boxes of 2 KB.  One
// elected lane asks for all of them, from coordinates that are the same in the whole
// warp: a box per lane took 62 cycles each (1000 a tile, as long as its share of the
// memory's time), the loads of one lane after the other.
template <int A, bool W, bool F, class C>
__device__ void loader(const CrossParams& P, const CUtensorMap* kmap, const CUtensorMap* vmap, const CUtensorMap* qmap,
                       Tiles<A, F>& T, C& c) {
  using TT = Tiles<A, F>;
  constexpr int H = TT::kHalves, NS = TT::kRing;
  const unsigned FULL = 0xffffffffu;
  const int lane = threadIdx.x & 31;
  const int none = P.num_blocks * P.n_kv_heads * kBlockSize;      // past the map's rows: zeros
  const int tok_tile = kTileM >> P.group_log2, group = 1 << P.group_log2;
  uint32_t at = 0, qs = 0;                                        // place in the ring's order, query tiles
  Pieces<W> pieces(P, c);
  Piece<W> p;
  // y: rows of the tile's blocks, in lanes [in4 * 8, in4 * 8 + 8)
  auto load = [&](const CUtensorMap* map, int y, int in4) -> bool {
    const uint32_t st = __shfl_sync(FULL, at % NS, 0);
    if (!warp_wait(P, &c.empty[st], ((at / NS) & 1) ^ 1)) return false;
    ++at;
    int rows[8];
#pragma unroll
    for (int b = 0; b < 8; ++b) rows[b] = __shfl_sync(FULL, y, in4 * 8 + b);
    if (elect_lane()) {
      mbar_arrive_expect_tx(&c.full[st], TT::kBytes);
#pragma unroll
      for (int b = 0; b < 8; ++b)
#pragma unroll
        for (int h = 0; h < H; ++h) tma_load_2d(&T.kv[st][h][b * kBlockSize][0], map, h * 64, rows[b], &c.full[st]);
    }
    __syncwarp();
    return true;
  };
  bool ok = true;
  while (ok && !__any_sync(FULL, c.abort) && pieces.next(P, p)) {
    const int n_blocks = (p.q.kv + kBlockSize - 1) / kBlockSize;
    const int32_t* table = P.block_tables + (size_t)p.r * P.max_blocks_per_seq;
    // a lane's entry of the four tiles from j on
    auto entry = [&](int j) { return j * 8 + lane < n_blocks ? __ldg(table + j * 8 + lane) : -1; };
    auto row_of = [&](int j, int e) {
      if (j * 8 + lane >= n_blocks) return none;
      if (e >= 0 && e < P.num_blocks) return (e * P.n_kv_heads + p.g) * kBlockSize;
      set_error(P.err, CB_DEVERR_BADBLOCK);
      return none;
    };
    int e = entry(p.ta), y = none, before = none;
    auto load_q = [&]() {
      for (int side = 0; ok && side < (p.wide() ? 2 : 1); ++side, ++qs) {
        const uint32_t st = qs % TT::kQ;
        ok = warp_wait(P, &c.q_empty[st], ((qs / TT::kQ) & 1) ^ 1);
        if (ok && elect_lane()) {
          mbar_arrive_expect_tx(&c.q_full[st], P.q_bytes * (F ? 4 : 1));
#pragma unroll
          for (int h = 0; h < H; ++h)
#pragma unroll
            for (int w = 0; w < (F ? 4 : 1); ++w)
              tma_load_3d(&T.q[st][h][w * 32][0], qmap, h * 64, p.g * group, p.q.q0 + p.tok_lo + side * tok_tile, &c.q_full[st]);
        }
        __syncwarp();
      }
    };
    if (TT::kQ == 2) load_q();
    for (int j = p.ta; ok && j < p.tb; ++j) {
      const int in4 = (j - p.ta) & 3;
      if (in4 == 0) {                  // the entries asked for four tiles ago; the next ones
        before = y;
        y = row_of(j, e);
        e = j + 4 < p.tb ? entry(j + 4) : -1;
      }
      ok = load(kmap, y, in4);
      // one query tile waits for the last item's scores: the first keys go ahead of it
      if (TT::kQ == 1 && j == p.ta) load_q();
      if (p.wide())
        ok = ok && load(vmap, y, in4);
      else if (j > p.ta)
        ok = ok && load(vmap, in4 ? y : before, (in4 + 3) & 3);
    }
    if (ok && !p.wide()) ok = load(vmap, y, (p.tb - 1 - p.ta) & 3);
  }
  if (!ok) c.abort = 1;
  if (c.abort && lane == 0) {          // copies in flight land before shared memory is given back
    for (int par = 0; par < 2; ++par) {
      for (int s = 0; s < NS; ++s) mbar_wait(&c.full[s], par, 20000000ull);
      mbar_wait(&c.q_full[0], par, 20000000ull);
      if (TT::kQ == 2) mbar_wait(&c.q_full[1], par, 20000000ull);
    }
  }
}

// ---------------------------------------------------------------- MMA issue (warps 9, 10)
// Group s's tiles run as a chain S(0) PV(0) S(1) PV(1) ...; S(i + 1) goes out right
// behind PV(i), which reads P from the columns that S(i + 1) overwrites: operations of
// one thread run in order.  A warp issues each group's chain: while one is at its
// barriers (a few hundred cycles a tile), the tensor core has the other's products.
//
// The whole warp waits and computes; one elected lane issues.  Operands of an MMA
// are read from uniform registers, which the compiler uses for values of a converged
// warp: issued from a branch of one lane, each MMA moved its descriptors there first
// and took about 110 cycles instead of the 64 that it runs.
template <int A, bool W, bool F, class C>
__device__ void issuer(const CrossParams& P, Tiles<A, F>& T, C& c, uint32_t tmem, int side) {
  using TT = Tiles<A, F>;
  constexpr int NS = TT::kRing;
  constexpr uint32_t kIdescS = idesc_bf16_f32(128, 128, 0), kIdescPV = idesc_bf16_f32(128, A, 1);
  const unsigned FULL = 0xffffffffu;
  tmem = __shfl_sync(FULL, tmem, 0);
  side = __shfl_sync(FULL, side, 0);
  const uint32_t base = __shfl_sync(FULL, smem_u32(&T), 0);
  const uint64_t q0 = smem_desc_sw128(base, 16, 1024);
  const uint64_t k0 = smem_desc_sw128(base + (uint32_t)offsetof(TT, kv), 16, 1024);
  const uint64_t v0 = smem_desc_sw128(base + (uint32_t)offsetof(TT, kv), TT::kHalfBytes, 1024);
  const uint64_t p0 = smem_desc_sw128(base + (uint32_t)offsetof(TT, weights) + side * TT::kFewGroup, 16, 1024);
  uint32_t qs = 0, np = 0, items = 0, turns = 0;   // P tiles consumed, items begun, turns taken
  uint32_t st = 0, ph = 0;                         // the ring's next buffer
  int second = side;                               // see softmax
  Pieces<W> pieces(P, c);
  Piece<W> p{};
  bool ok = true;
  // Both warps see every buffer, in the loads' order, and give it back: the one that reads it
  // once its products are done, the other at once.  A wait tells a phase from the one before it
  // only, so neither may run a ring ahead of a load that the other waits for.
  auto step = [&]() {
    if (++st == NS) {
      st = 0;
      ph ^= 1;
    }
  };
  auto give_back = [&](uint64_t* full, uint64_t* empty, uint32_t parity) -> bool {
    if (!warp_wait(P, full, parity)) return false;
    if (elect_lane()) mbar_arrive(empty);
    __syncwarp();
    return true;
  };
  auto other = [&]() -> bool {                     // the other group's tile
    const bool fine = give_back(&c.full[st], &c.empty[st], ph);
    step();
    return fine;
  };
  auto issue_s = [&](uint32_t slot, uint32_t kst, bool last) {
    const uint64_t q = q0 + slot * (TT::kBytes >> 4), k = k0 + kst * (TT::kBytes >> 4);
#pragma unroll
    for (int ks = 0; ks < A / 16; ++ks) {
      const uint64_t off = ((ks >> 2) * TT::kHalfBytes + (ks & 3) * 32) >> 4;
      tc_mma_f16(tmem + side * 128, q + off, k + off, kIdescS, ks > 0);
    }
    tc_commit(&c.s_full[side]);
    tc_commit(&c.empty[kst]);
    if (last) tc_commit(&c.q_empty[slot]);
  };
  auto scores = [&](uint32_t slot, bool last) -> bool {       // S of the next buffer
    if (!warp_wait(P, &c.full[st], ph)) return false;
    tc_fence_after();
    const uint32_t kst = __shfl_sync(FULL, st, 0);
    if (elect_lane()) issue_s(slot, kst, last);
    __syncwarp();
    step();
    return true;
  };
  // PV of the next buffer and, if there is one, S of the group's next tile, in the buffer behind
  // it: 16 products without a pause.
  auto values = [&](bool first, uint32_t slot, bool more, bool last) -> bool {
    const uint32_t vst = __shfl_sync(FULL, st, 0), vph = ph;
    step();
    const uint32_t kst = __shfl_sync(FULL, st, 0);
    if (!warp_wait(P, &c.full[vst], vph)) return false;
    if (more) {
      if (!warp_wait(P, &c.full[kst], ph)) return false;
      step();
    }
    if (first && !warp_wait(P, &c.o_free[side], (items++ & 1) ^ 1)) return false;
    if (p.wide() && !warp_wait(P, &c.turn[side], (turns++ & 1) ^ !side)) return false;
    if (!warp_wait(P, &c.p_full[side], np++ & 1)) return false;
    tc_fence_after();
    const uint64_t v = v0 + vst * (TT::kBytes >> 4);
    if (elect_lane()) {
#pragma unroll
      for (int ks = 0; ks < kTileN / 16; ++ks)
        if constexpr (F)
          tc_mma_f16(tmem + 256 + side * A, p0 + (((ks >> 2) * TT::kFewHalf + (ks & 3) * 32) >> 4),
                     v + ((ks * 16 * 128) >> 4), kIdescPV, (!first || ks > 0) ? 1u : 0u);
        else
          tc_mma_f16_ts(tmem + 256 + side * A, tmem + side * 128 + ks * 8, v + ((ks * 16 * 128) >> 4), kIdescPV,
                        (!first || ks > 0) ? 1u : 0u);
      tc_commit(&c.o_done[side]);
      tc_commit(&c.empty[vst]);
      if (more) issue_s(slot, kst, last);
      if (p.wide()) mbar_arrive(&c.turn[side ^ 1]);
    }
    __syncwarp();
    return true;
  };
  while (ok && !__any_sync(FULL, c.abort) && pieces.next(P, p)) {
    const int n = p.tb - p.ta;
    const uint32_t x = qs + (p.wide() && side), slot = __shfl_sync(FULL, x % TT::kQ, 0);
    const bool mine = p.wide() || n > second;        // this group has a tile
    if (p.wide()) {
      const uint32_t y = qs + !side;               // the other group's query tile
      if (side) ok = give_back(&c.q_full[y & 1], &c.q_empty[y & 1], (y >> 1) & 1);
      ok = ok && warp_wait(P, &c.q_full[slot], (x >> 1) & 1);
      if (!side) ok = ok && give_back(&c.q_full[y & 1], &c.q_empty[y & 1], (y >> 1) & 1);
      ok = ok && scores(slot, n == 1);
      for (int j = 0; ok && j < n; ++j) ok = values(j == 0, slot, j + 1 < n, j + 2 == n);
    } else {
      const uint32_t qp = (x / TT::kQ) & 1;
      ok = mine ? warp_wait(P, &c.q_full[slot], qp) : give_back(&c.q_full[slot], &c.q_empty[slot], qp);
      // K(0) K(1) V(0) K(2) V(1) .. V(n - 1): up to V(second)
      if (second) ok = ok && other();
      if (mine) ok = ok && scores(slot, second + 2 >= n);
      if (n > 1 && !second) ok = ok && other();
      if (second) ok = ok && other();
      if (n > 2 && second) ok = ok && other();
      for (int j = second; ok && j < n; j += 2) {
        ok = values(j == second, slot, j + 2 < n, j + 4 >= n);
        if (j + 1 < n) ok = ok && other();         // V(j + 1)
        if (j + 3 < n) ok = ok && other();         // K(j + 3)
      }
    }
    if (!W) second ^= 1;
    qs += p.wide() ? 2 : 1;
  }
  if (!ok) c.abort = 1;
  if (elect_lane()) tc_commit(&c.drain[side]);     // what was issued completes before the TMEM is freed
  __syncwarp();
  mbar_wait(&c.drain[side], 0, 20000000ull);
}

// ---------------------------------------------------------------- softmax (warps 0-7)
// The scores of a row whose m lies far out become what is left of them beside it: s sl2 is rounded as m was, so
// that the largest is 0, and divided by sl2 (back: 1 / sl2), by which the weights multiply.  The warp's other rows
// keep theirs.  Rarely done, and a loop over the scores' own columns: the softmax goes round a short block for it.
// (Every exponent with two roundings: prompts of up to 2000 tokens 276 to 281 us; this in registers 267; this 265.5;
// without it 262.5.)
__device__ __forceinline__ void centre(float (&s)[128], uint32_t s_at, bool far, float sl2, float back, float m) {
  const float by = far ? sl2 : 1.f, top = far && m != kNoKey ? m : 0.f, per = far ? back : 1.f;
#pragma unroll
  for (int h = 0; h < 4; ++h) tmem_st32(s_at + h * 32, *reinterpret_cast<float(*)[32]>(s + h * 32));
  tmem_wait_st();
#pragma unroll 1
  for (int c = 0; c < 128; c += 8) {
    float x[8];
    tmem_ld8(s_at + c, x);
    tmem_wait_ld();
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = (__fmul_rn(x[k], by) - top) * per;
    tmem_st8(s_at + c, x);
  }
  tmem_wait_st();
  tmem_ld64(s_at, *reinterpret_cast<float(*)[64]>(s));
  tmem_ld64(s_at + 64, *reinterpret_cast<float(*)[64]>(s + 64));
  tmem_wait_ld();
}

// Scale a row's O by alpha.
template <int A>
__device__ __forceinline__ void rescale(uint32_t o, float alpha) {
#pragma unroll 1
  for (int c = 0; c < A / 32; ++c) {
    float x[32];
    tmem_ld32(o + c * 32, x);
    tmem_wait_ld();
#pragma unroll
    for (int k = 0; k < 32; ++k) x[k] *= alpha;
    tmem_st32(o + c * 32, x);
  }
}

// A row's result: its output if the piece is its whole item, else its part of the join.  O and
// the other group's O (two) are scaled by alpha and beta.  (Where they lie is worked out by the
// caller: prompts of up to 2000 tokens took 265 us with that in here, 262 without.)
template <int A, bool W>
__device__ __forceinline__ void write_rows(int part_rows, int irow, bool whole, bool valid, bool two, uint32_t o_at,
                                           uint32_t other_o, float alpha, float beta, float m, float l, uint16_t* dst,
                                           float* part) {
#pragma unroll 1
  for (int ch = 0; ch < A / 32; ++ch) {
    float o[32];
    tmem_ld32(o_at + ch * 32, o);
    if (two) {
      float b[32];
      tmem_ld32(other_o + ch * 32, b);
      tmem_wait_ld();
#pragma unroll
      for (int k = 0; k < 32; ++k) o[k] = o[k] * alpha + b[k] * beta;
    } else {
      tmem_wait_ld();
#pragma unroll
      for (int k = 0; k < 32; ++k) o[k] *= alpha;
    }
    if (valid && whole) {
#pragma unroll
      for (int k = 0; k < 32; k += 8)
        *reinterpret_cast<uint4*>(dst + ch * 32 + k) = make_uint4(pack_bf16(o[k], o[k + 1]), pack_bf16(o[k + 2], o[k + 3]),
                                                                  pack_bf16(o[k + 4], o[k + 5]), pack_bf16(o[k + 6], o[k + 7]));
    } else if (valid) {
#pragma unroll
      for (int k = 0; k < 32; k += 4)
        reinterpret_cast<float4*>(part)[W ? (size_t)(ch * 8 + k / 4) * part_rows + irow : (size_t)irow * (A / 4) + ch * 8 + k / 4] =
            make_float4(o[k], o[k + 1], o[k + 2], o[k + 3]);
    }
  }
  if (valid && !whole) *reinterpret_cast<float2*>(part + (size_t)part_rows * A + irow * 2) = make_float2(m, l);
}

template <int A, bool W, class C>
__device__ void softmax(const CrossParams& P, Tiles<A, false>& T, C& c, uint32_t tmem, int side) {
  using TT = Tiles<A, false>;
  constexpr int H = TT::kHalves, NS = TT::kRing;
  const unsigned FULL = 0xffffffffu;
  const int row = threadIdx.x & 127, warp = (threadIdx.x >> 5) & 3;
  const uint32_t lanes = (uint32_t)(warp * 32) << 16;
  const uint32_t s_at = tmem + lanes + side * 128;
  const uint32_t o_at = tmem + lanes + 256 + side * A, other_o = tmem + lanes + 256 + (side ^ 1) * A;
  const int tok_tile = kTileM >> P.group_log2;
  const float sl2 = P.scale_log2;
  // key tiles before this piece; this group's; the other group's; pieces that both share
  uint32_t kt = 0, sc = 0, oc = 0, shared = 0;
  // Of a narrow piece, the group that has key tiles 1, 3, ..: the groups in turn, so that pieces of
  // one tile run beside each other and those of an odd number fill both groups (32 heads of
  // dimension 64, 100 tokens over 128 keys: 43.5 us, 68.5 with B always; 1408 keys: 203 and 218).
  // Where some items are wide, that cost these more than it gave (prompts 267 us, 263 without).
  int second = W ? side : side ^ 1;
  Pieces<W> pieces(P, c);
  Piece<W> p;
  while (!__any_sync(FULL, c.abort) && pieces.next(P, p)) {
    const int n = p.tb - p.ta;
    if (!W) second ^= 1;
    const int mine = p.wide() ? n : (n + !second) / 2;
    const int tok = (p.wide() && side ? tok_tile : 0) + (row >> P.group_log2);      // of the item
    const bool valid = tok < p.tokens;
    const bool busy = __any_sync(FULL, valid);                                    // this warp has rows
    float m = kNoKey, l = 0.f;         // running max times scale * log2 e; sum
    bool ok = true;
    for (int i = 0; i < mine; ++i, ++sc) {
      const int j = p.wide() ? i : 2 * i + second, key0 = (p.ta + j) * kTileN;
      ok = warp_wait(P, &c.s_full[side], sc & 1);
      if (!ok) break;
      tc_fence_after();
      if (busy) {
        float s[128];
        tmem_ld64(s_at, *reinterpret_cast<float(*)[64]>(s));
        tmem_ld64(s_at + 64, *reinterpret_cast<float(*)[64]>(s + 64));
        tmem_wait_ld();
        if (key0 + kTileN > p.q.kv) {
#pragma unroll
          for (int k = 0; k < 128; ++k) s[k] = key0 + k < p.q.kv ? s[k] : kNoKey;
        }
        // The weights refer to the running max m of an item's first tile, and O and their sum with
        // them: that is exact whatever m is.  A tile's own max is looked for only if its weights' sum
        // says that one may be large (or NaN), or if m lies far out (or has had no key but -inf yet): then m
        // moves up, O is scaled and the weights are made again.
        const uint64_t sl2x2 = f2(sl2, sl2);
        float alpha = 1.f, add;
        bool known = i > 0, bad = i == 0;
#pragma unroll 1
        while (true) {
          if (!known) {
            float a[4] = {kNoKey, kNoKey, kNoKey, kNoKey};
#pragma unroll
            for (int k = 0; k < 128; k += 2) a[(k >> 1) & 3] = max3(a[(k >> 1) & 3], s[k], s[k + 1]);
            const float mn = fmaxf(m, max3(a[0], a[1], fmaxf(a[2], a[3])) * sl2);
            if (bad && mn > m) {           // rows without need keep theirs: no row's result depends on another
              alpha = ex2(m - mn);
              m = mn;
            }
            if (i > 0) {
              ok = warp_wait(P, &c.o_done[side], (sc - 1) & 1);
              if (!ok) break;
              tc_fence_after();
              rescale<A>(o_at, alpha);
              tmem_wait_st();            // with the weights that are made again
            }
            const bool far = valid && fabsf(m) >= kFar;
            if (__any_sync(FULL, far)) centre(s, s_at, far, sl2, P.per_scale_log2, m);
          }
          const float ms = fabsf(m) >= kFar ? 0.f : m;             // no key so far but -inf: weights 0
          const uint64_t nm2 = f2(-ms, -ms);
          uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            uint32_t pk[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              float x0, x1;
              f2split(ffma2(f2(s[h * 32 + 2 * k], s[h * 32 + 2 * k + 1]), sl2x2, nm2), x0, x1);
              const float p0 = ex2(x0), p1 = ex2(x1);
              sum[k & 1] = fadd2(sum[k & 1], f2(p0, p1));
              pk[k] = pack_bf16(p0, p1);
            }
            tmem_st16u(s_at + h * 16, pk);
          }
          float t[4];
          f2split(sum[0], t[0], t[1]);
          f2split(sum[1], t[2], t[3]);
          add = (t[0] + t[1]) + (t[2] + t[3]);
          if (!known) break;
          bad = valid && !(add <= kMostSum && fabsf(m) < kFar);
          if (!__any_sync(FULL, bad)) break;
          known = false;
        }
        if (!ok) break;
        l = l * alpha + add;
      }
      // values behind the last key in its block: whatever the cache holds there, and 0 * inf must
      // not reach O.  In a wide item both groups write the same zeros.
      if (key0 + kTileN > p.q.kv && (p.q.kv & (kBlockSize - 1))) {
        const uint32_t t = 2 * (kt + n) - 1, st = t % NS;           // the piece's last buffer
        ok = warp_wait(P, &c.full[st], (t / NS) & 1);
        if (!ok) break;
        const int r0 = p.q.kv - key0, r1 = ((p.q.kv + kBlockSize - 1) & ~(kBlockSize - 1)) - key0;
        for (int x = row; x < (r1 - r0) * H * 8; x += 128)
          *reinterpret_cast<uint4*>(&T.kv[st][(x >> 3) % H][r0 + x / (H * 8)][(x & 7) << 4]) = make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&c.p_full[side]);
    }
    kt += n;
    const bool two = !p.wide() && n > 1; // both groups hold parts of the same rows
    oc += p.wide() ? n : n - mine;
    shared += two;
    if (ok && mine) ok = warp_wait(P, &c.o_done[side], (sc - 1) & 1);
    if (!ok) {
      c.abort = 1;
      break;
    }
    tc_fence_after();
    float alpha = 1.f, beta = 0.f;     // of this group's O and of the other's
    if (two) {
      if (second) {
        c.ml[row] = make_float2(m, l);
        mbar_arrive(&c.ml_full);
        continue;                      // the first group takes it from here, and frees both O
      }
      if (!warp_wait(P, &c.ml_full, (shared - 1) & 1) || !warp_wait(P, &c.o_done[side ^ 1], (oc - 1) & 1)) {
        c.abort = 1;
        break;
      }
      tc_fence_after();
      const float2 b = c.ml[row];
      const float mn = fmaxf(m, b.x), ms = mn == kNoKey ? 0.f : mn;
      alpha = ex2(m - ms);
      beta = ex2(b.x - ms);
      l = l * alpha + b.y * beta;
      m = mn;
    } else if (!mine) {
      continue;                        // a narrow piece of one tile has nothing for the second group
    }
    const bool whole = p.whole();
    if (!whole && row == 0 && !(p.wide() && side)) c.cut[p.ta == 0] = p;
    const float inv = whole ? 1.f / l : 1.f;
    alpha *= inv;
    beta *= inv;
    const int group = 1 << P.group_log2, irow = (p.wide() && side ? 128 : 0) + row;
    float* part = P.part + (size_t)(2 * (int)blockIdx.x + (p.ta == 0 ? 1 : 0)) * P.part_rows * (A + 2);
    uint16_t* dst = P.out + ((size_t)(p.q.q0 + p.tok_lo + tok) * P.n_q_heads + (size_t)p.g * group + (row & (group - 1))) * A;
    if (busy) write_rows<A, W>(P.part_rows, irow, whole, valid, two, o_at, other_o, alpha, beta, m, l, dst, part);
    tc_fence_before();
    mbar_arrive(&c.o_free[side]);
    if (two) mbar_arrive(&c.o_free[side ^ 1]);
  }
}

// Items of at most 32 rows: thread = row leaves three of a group's warps idle, while one takes
// 1750 cycles for a row's 128 weights.  Here the query tile has its rows four times, one copy
// for each warp's lanes, and so have the scores: warp w makes the weights of keys
// 32 w .. 32 w + 31.  They go to shared memory, one row for all four; O is in warp 0's
// lanes.  m is the same in the four warps, which tell each other their maxima when it may move;
// sums stay apart until the item's end.  Every exit is taken by the four warps together:
// they meet at named barriers.  100 tokens, 32 heads: dimension 64 over 100 to 3000 keys 192 us
// (thread = row: 257), over 128 keys 35.6 (43.4); dimension 128 over 257 keys 108 (162); 8
// tokens each over 257 keys, 32/8 heads of 128, 41 (55.8).
template <int A, class C>
__device__ void softmax_few(const CrossParams& P, Tiles<A, true>& T, C& c, uint32_t tmem, int side) {
  using TT = Tiles<A, true>;
  constexpr int H = TT::kHalves, NS = TT::kRing;
  const int thread = threadIdx.x & 127, warp = thread >> 5, row = thread & 31, bar = 1 + side;
  const uint32_t s_at = tmem + ((uint32_t)(warp * 32) << 16) + side * 128 + warp * 32;
  const uint32_t o_at = tmem + 256 + side * A, other_o = tmem + 256 + (side ^ 1) * A;     // warp 0
  const float sl2 = P.scale_log2;
  uint8_t* const weights = T.weights[side][warp >> 1][row];
  uint32_t kt = 0, sc = 0, oc = 0, shared = 0;          // as in softmax
  int second = side ^ 1;
  bool ok = true;
  Pieces<false> pieces(P, c);
  Piece<false> p;
  while (pieces.next(P, p)) {
    if (named_bar_or(bar, 128, !ok || c.abort)) break;
    const int n = p.tb - p.ta;
    second ^= 1;
    const int mine = (n + !second) / 2;
    const int tok = row >> P.group_log2;
    const bool valid = tok < p.tokens;
    float m = kNoKey, l = 0.f;
    for (int i = 0; i < mine; ++i, ++sc) {
      const int key0 = (p.ta + 2 * i + second) * kTileN, key = key0 + warp * 32;
      ok = ok && warp_wait(P, &c.s_full[side], sc & 1);
      tc_fence_after();
      float s[32];
      tmem_ld32(s_at, s);
      tmem_wait_ld();
      if (key + 32 > p.q.kv) {
#pragma unroll
        for (int k = 0; k < 32; ++k) s[k] = key + k < p.q.kv ? s[k] : kNoKey;
      }
      // scaled and rounded before m, a maximum of such products, is taken off: the largest has exponent 0 however
      // far from 0 it lies (see kFar; in here the product costs next to nothing: 100 tokens over 77 keys 18.2 and
      // 18.9 us, over 257 keys 104.8 and 108)
#pragma unroll
      for (int k = 0; k < 32; ++k) s[k] = __fmul_rn(s[k], sl2);      // never fused with the sum, as packed products can be
      float alpha = 1.f, add;
      uint32_t pk[16];
      bool known = i > 0, bad = i == 0, met = true;
#pragma unroll 1
      while (true) {
        if (!known) {
          float a[2] = {kNoKey, kNoKey};
#pragma unroll
          for (int k = 0; k < 32; k += 2) a[(k >> 1) & 1] = max3(a[(k >> 1) & 1], s[k], s[k + 1]);
          T.top[side][warp][row] = make_float2(fmaxf(a[0], a[1]), bad ? 1.f : 0.f);
          if (named_bar_or(bar, 128, !ok)) {
            met = false;
            break;
          }
          float mn = m, need = 0.f;
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const float2 x = T.top[side][w][row];
            mn = fmaxf(mn, x.x);
            need += x.y;
          }
          if (need > 0.f && mn > m) {
            alpha = ex2(m - mn);
            m = mn;
          }
          if (i > 0 && warp == 0) {
            ok = warp_wait(P, &c.o_done[side], (sc - 1) & 1);
            if (ok) {
              tc_fence_after();
              rescale<A>(o_at, alpha);
              tmem_wait_st();
            }
          }
        }
        const float ms = m == kNoKey ? 0.f : m;
        const uint64_t nm2 = f2(-ms, -ms);
        uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          float x0, x1;
          f2split(fadd2(f2(s[2 * k], s[2 * k + 1]), nm2), x0, x1);
          const float p0 = ex2(x0), p1 = ex2(x1);
          sum[k & 1] = fadd2(sum[k & 1], f2(p0, p1));
          pk[k] = pack_bf16(p0, p1);
        }
        float t[4];
        f2split(sum[0], t[0], t[1]);
        f2split(sum[1], t[2], t[3]);
        add = (t[0] + t[1]) + (t[2] + t[3]);
        if (!known) break;
        bad = valid && !(add <= kMostSum && m > kNoKey);
        if (!named_bar_or(bar, 128, bad || !ok)) break;
        known = false;
      }
      if (!met) {
        ok = false;
        break;
      }
      l = l * alpha + add;
#pragma unroll
      for (int u = 0; u < 4; ++u)
        *reinterpret_cast<uint4*>(weights + ((((warp & 1) * 4 + u) ^ (row & 7)) << 4)) =
            make_uint4(pk[4 * u], pk[4 * u + 1], pk[4 * u + 2], pk[4 * u + 3]);
      if (key0 + kTileN > p.q.kv && (p.q.kv & (kBlockSize - 1))) {       // as in softmax
        const uint32_t t = 2 * (kt + n) - 1, st = t % NS;
        ok = ok && warp_wait(P, &c.full[st], (t / NS) & 1);
        const int r0 = p.q.kv - key0, r1 = ((p.q.kv + kBlockSize - 1) & ~(kBlockSize - 1)) - key0;
        if (ok)
          for (int x = thread; x < (r1 - r0) * H * 8; x += 128)
            *reinterpret_cast<uint4*>(&T.kv[st][(x >> 3) % H][r0 + x / (H * 8)][(x & 7) << 4]) = make_uint4(0, 0, 0, 0);
      }
      fence_proxy_async_smem();
      tc_fence_before();
      if (ok) mbar_arrive(&c.p_full[side]);
    }
    kt += n;
    const bool two = n > 1;
    oc += n - mine;
    shared += two;
    if (!mine) continue;
    ok = ok && warp_wait(P, &c.o_done[side], (sc - 1) & 1);
    tc_fence_after();
    T.sum[side][warp][row] = l;
    if (two && second) {
      if (warp == 0) c.ml[row].x = m;
      if (ok) mbar_arrive(&c.ml_full);
      continue;
    }
    if (named_bar_or(bar, 128, !ok)) {
      ok = false;
      break;
    }
    if (warp > 0) continue;            // their sums are read before any of them comes here again
    auto total = [&](int g) {
      return (T.sum[g][0][row] + T.sum[g][1][row]) + (T.sum[g][2][row] + T.sum[g][3][row]);
    };
    l = total(side);
    float alpha = 1.f, beta = 0.f;
    if (two) {
      ok = warp_wait(P, &c.ml_full, (shared - 1) & 1) && warp_wait(P, &c.o_done[side ^ 1], (oc - 1) & 1);
      if (!ok) continue;
      tc_fence_after();
      const float bm = c.ml[row].x, bl = total(side ^ 1);
      const float mn = fmaxf(m, bm), ms = mn == kNoKey ? 0.f : mn;
      alpha = ex2(m - ms);
      beta = ex2(bm - ms);
      l = l * alpha + bl * beta;
      m = mn;
    }
    const bool whole = p.whole();
    if (!whole && row == 0) c.cut[p.ta == 0] = p;
    const float inv = whole ? 1.f / l : 1.f;
    alpha *= inv;
    beta *= inv;
    const int group = 1 << P.group_log2, irow = row;
    float* part = P.part + (size_t)(2 * (int)blockIdx.x + (p.ta == 0 ? 1 : 0)) * P.part_rows * (A + 2);
    uint16_t* dst = P.out + ((size_t)(p.q.q0 + p.tok_lo + tok) * P.n_q_heads + (size_t)p.g * group + (row & (group - 1))) * A;
    write_rows<A, false>(P.part_rows, irow, whole, valid, two, o_at, other_o, alpha, beta, m, l, dst, part);
    tc_fence_before();
    mbar_arrive(&c.o_free[side]);
    if (two) mbar_arrive(&c.o_free[side ^ 1]);
  }
  if (!ok) c.abort = 1;
}

// ---------------------------------------------------------------- joining
// The pieces of an item that CTA boundaries cut are in the CTAs first .. last: the
// first's slot 2 first + 1, then slot 2 c.  Each of those CTAs joins its part of
// the rows:
//     M = max m_i,  out = sum 2^(m_i - M) O_i / sum 2^(m_i - M) l_i.
// Counter `first` of the stream counts the arrivals of n CTAs, then as many
// departures; the last sets it back to 0.
// LANES lanes take a row's four columns, at most kHold pieces each, which are read at once.
// Where items are wide, four columns of all rows lie together, so that a warp of the softmax
// (thread = row) writes whole lines, and a warp here takes 32 rows: prompts of up to 2000
// tokens 267 us with rows together, 262.5 so.  The few rows of narrow items are better
// kept whole (one token a request, dimension 64: 83.2 and 84.8 us).
constexpr int kHold = 5;
template <int A, bool W, int LANES>
__device__ void join_rows(const CrossParams& P, const Part& p, int first, int n, int lo, int hi) {
  const int sub = threadIdx.x % LANES, group = 1 << P.group_log2, rows = p.tokens << P.group_log2;
  const size_t slot_floats = (size_t)P.part_rows * (A + 2);
  // every lane of a warp goes through the same number of rounds: the shuffles need them all
  for (int base = lo; base < hi; base += kThreads / LANES) {
    const int task = base + threadIdx.x / LANES;
    const bool on = task < hi;
    const int row = !on ? 0 : W ? task % rows : task / (A / 4), col = !on ? 0 : W ? task / rows : task % (A / 4);
    float2 ml[kHold];
    float4 o[kHold];
#pragma unroll
    for (int k = 0; k < kHold; ++k) {
      const int i = sub + k * LANES;
      ml[k] = make_float2(kNoKey, 0.f);
      o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (!on || i >= n) continue;
      const float* piece = P.part + (size_t)(2 * (first + i) + (i == 0 ? 1 : 0)) * slot_floats;
      ml[k] = __ldcg(reinterpret_cast<const float2*>(piece + (size_t)P.part_rows * A) + row);
      o[k] = __ldcg(reinterpret_cast<const float4*>(piece) + (W ? (size_t)col * P.part_rows + row : (size_t)row * (A / 4) + col));
    }
    float M = kNoKey;
#pragma unroll
    for (int k = 0; k < kHold; ++k) M = fmaxf(M, ml[k].x);
#pragma unroll
    for (int d = LANES / 2; d > 0; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
    float L = 0.f;
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < kHold; ++k) {
      if (sub + k * LANES >= n) continue;
      const float w = ex2(ml[k].x - M);
      L += w * ml[k].y;
      y.x += w * o[k].x, y.y += w * o[k].y, y.z += w * o[k].z, y.w += w * o[k].w;
    }
#pragma unroll
    for (int d = LANES / 2; d > 0; d >>= 1) {
      L += __shfl_xor_sync(0xffffffffu, L, d);
      y.x += __shfl_xor_sync(0xffffffffu, y.x, d);
      y.y += __shfl_xor_sync(0xffffffffu, y.y, d);
      y.z += __shfl_xor_sync(0xffffffffu, y.z, d);
      y.w += __shfl_xor_sync(0xffffffffu, y.w, d);
    }
    if (on && sub == 0) {
      const float inv = 1.f / L;
      uint16_t* dst = P.out + ((size_t)(p.q.q0 + p.tok_lo + (row >> P.group_log2)) * P.n_q_heads + (size_t)p.g * group +
                               (row & (group - 1))) * A + col * 4;
      *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16(y.x * inv, y.y * inv), pack_bf16(y.z * inv, y.w * inv));
    }
  }
}
static_assert(kHold * 32 >= kMaxDecodeGrid, "an item's pieces fit a warp");

__device__ __forceinline__ unsigned ld_acquire(const unsigned* p) {
  unsigned v;
  asm volatile("ld.acquire.gpu.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}

// All threads, after the pipeline.
template <int A, bool W, class C>
__device__ void join(const CrossParams& P, C& c) {
  if (c.abort) {                       // the others still wait for this CTA's arrivals
    __syncthreads();
    if (threadIdx.x == 0) {
      Pieces<W> pieces(P, c);
      Piece<W> p;
      while (pieces.next(P, p))
        if (!p.whole()) c.cut[p.ta == 0] = p;
    }
    __syncthreads();
  }
  auto first_of = [&](const Part& p) { return p.at / c.share; };
  if (threadIdx.x == 0) {              // arrive for both before waiting for either
    __threadfence();                   // with the barrier before join(): every thread's partial results
    for (int k = 0; k < 2; ++k)
      if (c.cut[k].tiles) atomicAdd(P.joins + first_of(c.cut[k]), 1u);
  }
  for (int k = 0; k < 2; ++k) {
    const Part& p = c.cut[k];
    if (!p.tiles) continue;
    const int first = first_of(p), n = (p.at + (p.tiles - 1) * p.step) / c.share - first + 1;
    unsigned* count = P.joins + first;
    if (threadIdx.x == 0) {
      int ok = 1;
      const uint64_t t0 = globaltimer_ns();
      while (ld_acquire(count) < (unsigned)n) {
        if (globaltimer_ns() - t0 > kWaitLimitNs) {
          set_error(P.err, CB_DEVERR_TIMEOUT);
          ok = 0;
          break;
        }
      }
      c.go = ok;
    }
    __syncthreads();
    if (c.go && !c.abort) {
      const int rows = p.tokens << P.group_log2, tasks = rows * (A / 4), i = (int)blockIdx.x - first;
      const int lo = (int)((long long)tasks * i / n), hi = (int)((long long)tasks * (i + 1) / n);
      if (n <= kHold) join_rows<A, W, 1>(P, p, first, n, lo, hi);
      else if (n <= 4 * kHold) join_rows<A, W, 4>(P, p, first, n, lo, hi);
      else if (n <= 16 * kHold) join_rows<A, W, 16>(P, p, first, n, lo, hi);
      else join_rows<A, W, 32>(P, p, first, n, lo, hi);
    }
    __syncthreads();
    if (threadIdx.x == 0 && atomicAdd(count, 1u) == 2u * n - 1) *count = 0u;
  }
}

// Rows of requests without keys: zeros.  All threads of the grid.
template <int A>
__device__ void zero_rows(const CrossParams& P) {
  const int lane = threadIdx.x & 31, vecs = P.n_q_heads * (A / 8);
  for (int r = 0; r < P.n_reqs; ++r) {
    const Request q = load_request(P, r, false);
    if (!q.q_len || q.kv) continue;
    for (int t = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); t < q.q_len; t += gridDim.x * (kThreads / 32)) {
      uint4* dst = reinterpret_cast<uint4*>(P.out + (size_t)(q.q0 + t) * P.n_q_heads * A);
      for (int i = lane; i < vecs; i += 32) dst[i] = make_uint4(0, 0, 0, 0);
    }
  }
}

template <int A, bool W, bool F>
__global__ void __launch_bounds__(kThreads, 1)
    cross_kernel(const CrossParams P, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                 const __grid_constant__ CUtensorMap qmap) {
  using TT = Tiles<A, F>;
  constexpr int NS = TT::kRing;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  TT& T = *reinterpret_cast<TT*>(base);
  Ctl<NS>& c = *reinterpret_cast<Ctl<NS>*>(base + sizeof(TT));
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(&c.q_full[s], 1);
      mbar_init(&c.q_empty[s], 2);
      mbar_init(&c.drain[s], 1);
      mbar_init(&c.turn[s], 1);
      mbar_init(&c.s_full[s], 1);
      mbar_init(&c.p_full[s], 128);
      mbar_init(&c.o_done[s], 1);
      mbar_init(&c.o_free[s], F ? 32 : 128);
    }
    for (int s = 0; s < NS; ++s) {
      mbar_init(&c.full[s], 1);
      mbar_init(&c.empty[s], 2);
    }
    mbar_init(&c.ml_full, 128);
    c.abort = 0;
    c.any_empty = 0;
    c.cut[0].tiles = c.cut[1].tiles = 0;
    fence_mbar_init();
    prefetch_tmap(&kmap);
    prefetch_tmap(&vmap);
    prefetch_tmap(&qmap);
  }
  if (warp == 9) {
    tmem_alloc(&c.tmem_base, 512);
    tmem_relinquish();
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  make_plan(P, c);
  const uint32_t tmem = c.tmem_base;
  // three warpgroups of 168 registers a thread at launch: 2 * 208 + 88 = 3 * 168
  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp == 8) {
      loader<A, W, F>(P, &kmap, &vmap, &qmap, T, c);
    } else if (warp < 11) {
      issuer<A, W, F>(P, T, c, tmem, warp - 9);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    if constexpr (F)
      softmax_few<A>(P, T, c, tmem, warp >> 2);
    else
      softmax<A, W>(P, T, c, tmem, warp >> 2);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (c.any_empty) zero_rows<A>(P);
  join<A, W>(P, c);
}

template <int A, bool F>
constexpr int kSmem = 1024 + (int)sizeof(Tiles<A, F>) + (int)sizeof(Ctl<Tiles<A, F>::kRing>);
template <int A, bool F>
constexpr bool fits() {
  using TT = Tiles<A, F>;
  return kSmem<A, F> <= 232448 && sizeof(TT) % 16 == 0 && offsetof(TT, weights) % 1024 == 0 && offsetof(TT, kv) % 1024 == 0;
}
static_assert(fits<128, false>() && fits<128, true>() && fits<64, false>() && fits<64, true>(), "shared memory");

template <int A, bool W, bool F>
cudaError_t launch_cross_t(const CrossParams& p, const CUtensorMap* maps, int grid, cudaStream_t stream) {
  const void* kernel = reinterpret_cast<const void*>(cross_kernel<A, W, F>);
  const cudaError_t e = opt_in_smem(kernel, kSmem<A, F>);
  if (e != cudaSuccess) return e;
  CrossParams pc = p;
  void* args[] = {&pc, const_cast<CUtensorMap*>(&maps[0]), const_cast<CUtensorMap*>(&maps[1]),
                  const_cast<CUtensorMap*>(&maps[2])};
  return cudaLaunchCooperativeKernel(kernel, dim3(grid), dim3(kThreads), args, kSmem<A, F>, stream);
}

}  // namespace

long long cross_units_bound(int n_reqs, int n_tokens, int max_kv_len, int n_kv_heads, int group) {
  constexpr long long kMost = 1LL << 30;                      // what the caller refuses
  const long long groups = (long long)n_tokens / (kRows / group) + n_reqs;
  const long long tiles = ((long long)max_kv_len + kTileN - 1) / kTileN;
  const long long items = groups * n_kv_heads;                // at most 2^59
  return items >= kMost ? kMost : items * (kLead + kWide * tiles);
}
int cross_grid(long long units, int sms) {
  return (int)std::max(1LL, std::min<long long>(std::min(sms, kMaxDecodeGrid), (units + kLeast - 1) / kLeast));
}
int cross_part_rows(int max_q_len, int group) {
  return (int)((std::min<long long>(kRows, (long long)max_q_len * group) + 3) / 4 * 4);
}

cudaError_t launch_cross(const CrossParams& p, const CUtensorMap* maps, int head_dim, int grid, cudaStream_t stream) {
  const long long rows = (long long)p.max_q_len << p.group_log2;      // that an item can have
  const bool wide = rows > kRows / 2;
  const bool few = rows <= kFewRows;
  const auto launch = head_dim == 128 ? (wide  ? launch_cross_t<128, true, false>
                                         : few ? launch_cross_t<128, false, true>
                                               : launch_cross_t<128, false, false>)
                                      : (wide  ? launch_cross_t<64, true, false>
                                         : few ? launch_cross_t<64, false, true>
                                               : launch_cross_t<64, false, false>);
  return launch(p, maps, grid, stream);
}

}  // namespace cb
