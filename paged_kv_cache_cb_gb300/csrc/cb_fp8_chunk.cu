// Attention of several new tokens per request over the 8-bit KV cache (format:
// cb_fp8.cuh) on the tensor cores.
//
// Mathematics.  For a row (token at position p, query head h) with visible keys
// j <= p (and j > p - W under a window), keys k_j 2^ek_j and values v_j 2^ev_j:
//     x_j = scale log2(e) 2^eq 2^ek_j (q . k_j),  p_j = 2^(x_j - m),  out = sum p_j V_j / sum p_j
// with m a running maximum that moves only when a score passes it by 8.
//   S = q k^T takes e4m3 K from the cache as it is; q 2^-eq is two e4m3 terms
//   whose products add up (4 significant bits each: bf16's 8; values down to
//   2^-9 of the row's largest exactly, smaller ones within 2^-17 of it).
//   S is up to 2^24 and ek up to 120, so S 2^ek alone may pass fp32's range where
//   x does not.  What a tile's largest ek has beyond 100 is its E (0 almost always):
//   S is multiplied by 2^(ek - E), the row's factor by 2^E.  No key falls out at the
//   other end: ek - E is -146 at least, a subnormal.  (With an E for every 32 keys
//   the softmax has four factors to hold: 2048 tokens after 30720 keys took 942 us
//   instead of 905.)
//   O = p V takes V as bf16, converted exactly (the rows' scales are powers of
//   two), and p rounded to bf16 (2^-8 relative, the type of the 16-bit cache);
//   the sum of p is taken before that rounding.
// The two S terms cost as much tensor time as one bf16 product and leave K
// unconverted; p in 8-bit terms would cost three, and the softmax's time for
// making them.
//
// Tiles.  An item is (request, KV head, 2 TOK tokens), TOK = 128 / G: two query
// tiles of 128 rows (row i = token i / G, head i % G) that share the keys, in
// tiles of 128.  Tensor memory: S_A | P_A, S_B | P_B (P over the first half of its
// own S), O_A, O_B.  The tensor pipe alternates PV_A(j-1) S_A(j), PV_B(j-1)
// S_B(j): one query tile's softmax runs under the other's products.  P is handed
// over in two halves of 64 keys, so the products start while the second half is
// computed.  An item of at most TOK tokens has one query tile.
//
// Work.  All items' key tiles, each item's behind a few empty places for its start and
// end, laid end to end, are cut into one equal range per CTA (one CTA per SM); an item
// cut at a range's end leaves (m, l, o) per piece and a second kernel
// (cb_fp8_join.cu) joins them.  Where whole items, dealt to the CTAs in turn, end
// sooner than the cut ranges and their joining, they stay whole.
//
// Warps: 0-3 and 4-7 softmax of tiles A and B (thread = row; the row's 128
// scores stay in registers, one read of tensor memory; also the query's terms and
// the output), 8-11 convert V from a staged copy, in short loops (the warps'
// code shares one instruction cache), 12 issues the products, 13 loads K, 15 V and
// the exponents, 14 walks the work and publishes it.  Every wait is bounded.
//
// Bound by a tile's chain, not by a unit: 2048 new tokens after 30720 keys (32 heads
// on 8) take 915 us, 1.16 PFLOP/s, 0.61 of cuBLAS's bf16 rate, with the tensor pipe
// active half of the time; S of a query tile overwrites the columns of its P, so its
// softmax, PV and S follow one another and only the other query tile's hide them.  An
// item's start and end cost about 8 us.  Single tokens (below): 256 requests of 32
// heads on 1 KV head (1024 to 16384 keys, 539 MB) take 159 us, 3.4 TB/s, 0.50 of a
// copy's rate: a tile's conversion, whose shared-memory accesses compete with the
// products' operands, is the longest part of its chain.
#include <algorithm>

#include "cb_decode_item.cuh"
#include "cb_fp8.cuh"

namespace cb {

namespace {

constexpr int kThreads = 512;
constexpr int kRows = kChunkRows;      // rows of an item (two query tiles)
// The cut (see Work above), in key tiles' time (2 us; single tokens 1.4).  An item's
// start and end (its queries, first scores and output) are kLead empty places: cut by
// tiles alone, a range of short items takes as many starts and ends.  With 0, 2, 4 and
// 6 of them 2048 tokens without stored keys, cut, took 180, 99, 89 and 88 us, 8192 of
// them 1037, 730, 604 and 579 (592 whole), 512 after 4096 keys 76, 73, 71 and 72; 256
// single tokens of 32 heads on 1 with 0, 2 and 4 of them 164, 161 and 162.
// kJoinTiles is how much sooner the cut ranges must end than whole items: 512 tokens
// after 2048 keys (10 tiles sooner) take 67 us whole and 56 cut, 2048 after 2048 (12)
// 147 and 142, but 2048 without stored keys of 64 heads on 8 (9) 127 and 143, next to
// 48 single tokens 235 and 257.  At 5 to 8 either may be shorter: next to 48 single
// tokens 512 after 1024 and 2048, 64 heads on 8 (6) 205 and 225, 256 after 1000 (7) 128
// and 121.
template <bool ONE>
constexpr int kLead = ONE ? 2 : kChunkLead;
constexpr int kJoinTiles = 9;
constexpr int kSmemLimit = 232448;

// An item, and the piece [a, b) of its key tiles [first, end); b = a: no more items.
struct Item {
  int r, g, pair, q0, q_len, ctx, tok_lo, tok_hi, first, end, a, b, sides, pad[3];
};
constexpr int kItems = 4;              // published ahead
constexpr int kReaders = 15;           // warps that read them

template <int A>
struct alignas(1024) Smem {
  static constexpr int H = A / 64;     // 64-dimension halves of 128-byte rows
  uint8_t q[2][2][128 * A];            // [query tile][term]: e4m3 rows of A bytes
  uint8_t k[2][128 * A];               // e4m3 as in the cache
  uint8_t vr[2][128 * A];              // V as in the cache, no swizzle
  uint8_t v[2][H][128][128];           // V in bf16
  float fk[4][128];                    // 2^(ek - E) of the tile's keys
  float fe[4][4];                      // 2^E, by the warp that wrote them (single tokens: of its 32 keys)
  float fq[4][32];                     // single tokens: the rows' factors, of four items
  uint32_t v_nan[4][4];                // keys whose V stands for NaNs (stored as zeros)
  uint8_t ex[2][2][128];               // the tile's exponent bytes, K and V
  uint64_t q_full[2], k_full[2], k_empty[2], vr_full[2], vr_empty[2], fk_full[4], v_full[2], v_empty[2];
  uint64_t s_full[2], p_full[2][2], o_full[2], o_free[2], q_free, x_bar, drain, item_full[kItems], item_empty[kItems];
  Item item[kItems];
  int scan[16], iscan[16], tiles, u0, u1, items, longest, high, whole, eff;
  uint32_t tmem;
  volatile int abort;
};

// ---------------------------------------------------------------- work
// Key tiles [first, end) of the `pair`-th 2 TOK tokens of a request.
__device__ __forceinline__ int pair_first(int ctx, int pair, int tok2, int window) {
  return window > 0 ? max(0, ctx + pair * tok2 - window + 1) / kTileN : 0;
}
__device__ __forceinline__ int pair_end(int ctx, int q_len, int pair, int tok2) {
  return (int)(((long long)ctx + min((long long)q_len, (pair + 1LL) * tok2) + kTileN - 1) / kTileN);
}

// (q0, q_len, ctx) of request r if it is one of this kernel's (ONE: with one new
// token, else with several); q_len 0 otherwise.
template <bool ONE>
__device__ __forceinline__ int3 request(const Fp8Step& P, int r, bool report) {
  const int q0 = __ldg(P.cu_q_lens + r), q1 = __ldg(P.cu_q_lens + r + 1), ctx = __ldg(P.ctx_lens + r);
  const long long n = (long long)q1 - q0, kv = (long long)ctx + n;
  if (q0 >= 0 && q1 <= P.n_tokens && n >= 0 && (ONE ? n == 0 || (n > 1 && P.max_q_len > 1) : n < 2)) return make_int3(0, 0, 0);
  if (n < 0 || ctx < 0 || q0 < 0 || q1 > P.n_tokens || n > P.max_q_len || kv > P.max_kv_len ||
      (kv + kBlockSize - 1) / kBlockSize > P.max_blocks_per_seq) {
    if (report) set_error(P.err, CB_DEVERR_BADLEN);
    return make_int3(0, 0, 0);
  }
  return make_int3(q0, (int)n, ctx);
}

// The CTA's pieces in order.  Items of a request: pairs from the last (most
// keys) down, KV heads inside.
template <int TOK, bool ONE>
struct ItemIter {
  static constexpr int LEAD = kLead<ONE>;
  const Fp8Step& P;
  const int* tpre;                     // places before request r
  const int* ipre;                     // items before request r
  int whole, step, index, n_items;   // whole items: index, index + step, ...
  int u, u1;                           // cut ranges
  int3 rq;
  int r, pair, g, j0;                  // the next item, the place within it where the range goes on (cut ranges)
  bool fresh = true;
  template <class S>
  __device__ ItemIter(const Fp8Step& p, const S& s, const int* tp, const int* ip)
      : P(p), tpre(tp), ipre(ip), whole(s.whole), step(s.eff), index(blockIdx.x), n_items(s.items), u(s.u0), u1(s.u1) {}
  __device__ int find(const int* pre, int x) const {
    int lo = 0, hi = P.n_reqs - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (pre[mid] <= x)
        lo = mid;
      else
        hi = mid - 1;
    }
    return lo;
  }
  __device__ void fill(Item& I) const {
    I.r = r;
    I.g = g;
    I.pair = pair;
    I.q0 = rq.x;
    I.q_len = rq.y;
    I.ctx = rq.z;
    I.tok_lo = pair * 2 * TOK;
    I.tok_hi = min(rq.y, I.tok_lo + 2 * TOK);
    I.sides = I.tok_hi - I.tok_lo > TOK ? 2 : 1;
    I.first = pair_first(rq.z, pair, 2 * TOK, P.window);
    I.end = pair_end(rq.z, rq.y, pair, 2 * TOK);
  }
  __device__ bool next(Item& I) {
    const int Hkv = P.cache.n_kv_heads;
    if (whole) {
      if (index >= n_items) return false;
      r = find(ipre, index);
      rq = request<ONE>(P, r, false);
      const int rem = index - ipre[r], pairs = (rq.y + 2 * TOK - 1) / (2 * TOK);
      pair = pairs - 1 - rem / Hkv;
      g = rem % Hkv;
      fill(I);
      I.a = I.first;
      I.b = I.end;
      index += step;
      return true;
    }
    while (u < u1) {
      if (fresh) locate();
      fresh = false;
      fill(I);
      const int last = min(places(), j0 + (u1 - u));           // its places j0 .. last - 1 are in the range
      I.a = I.first + max(j0, LEAD) - LEAD;
      I.b = I.first + last - LEAD;
      u += last - j0;
      j0 = 0;
      if (++g == Hkv) {
        g = 0;
        if (--pair < 0 && u < u1) {
          do {
            ++r;
          } while (tpre[r + 1] <= u);
          rq = request<ONE>(P, r, false);
          pair = (rq.y + 2 * TOK - 1) / (2 * TOK) - 1;
        }
      }
      if (I.b > I.a) return true;                              // not only empty places
    }
    return false;
  }
  // Places of an item of the pair.
  __device__ int places() const { return LEAD + pair_end(rq.z, rq.y, pair, 2 * TOK) - pair_first(rq.z, pair, 2 * TOK, P.window); }
  // The item of place u.
  __device__ void locate() {
    r = find(tpre, u);
    rq = request<ONE>(P, r, false);
    int off = u - tpre[r];
    for (pair = (rq.y + 2 * TOK - 1) / (2 * TOK) - 1; pair > 0; --pair) {
      const int t = places() * P.cache.n_kv_heads;
      if (off < t) break;
      off -= t;
    }
    g = off / places();
    j0 = off % places();
  }
};

// All threads; ends with __syncthreads().
template <int A, int TOK, bool ONE>
__device__ void make_plan(const Fp8Step& P, const Fp8Partials& W, Smem<A>& S, int* tpre, int* ipre) {
  const int n = P.n_reqs, tid = threadIdx.x, lane = tid & 31, wid = tid >> 5, Hkv = P.cache.n_kv_heads;
  if constexpr (!ONE)
    if (tid == kThreads - 1) await_ready(P);           // in front of the barriers below, and those of the loads
  if (tid == 0) S.longest = S.high = 0;
  for (int r = tid; r < n; r += kThreads) {
    const int3 q = request<ONE>(P, r, blockIdx.x == 0);
    ipre[r] = q.y;
    tpre[r] = q.z;
  }
  __syncthreads();
  for (int r = wid; r < n; r += kThreads / 32) {       // a warp per request with pairs
    const int q_len = ipre[r], ctx = tpre[r], pairs = (q_len + 2 * TOK - 1) / (2 * TOK);
    if (pairs == 0) continue;                          // both are 0
    int t = 0, mx = 0;
    for (int p = lane; p < pairs; p += 32) {
      const int x = pair_end(ctx, q_len, p, 2 * TOK) - pair_first(ctx, p, 2 * TOK, P.window);
      t += x;
      mx = max(mx, x);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) t += __shfl_xor_sync(0xffffffffu, t, off);
    mx = __reduce_max_sync(0xffffffffu, mx);
    __syncwarp();
    if (lane == 0) {
      t = (t + pairs * kLead<ONE>) * Hkv;
      tpre[r] = t;
      ipre[r] = pairs * Hkv;
      atomicMax(&S.longest, mx);
      atomicAdd(&S.high, t >> 12);
    }
  }
  __syncthreads();
  // exclusive prefix sums of both
  const int seg = (n + kThreads - 1) / kThreads, lo = min(n, tid * seg), hi = min(n, lo + seg);
  unsigned t_own = 0;
  int i_own = 0;
  for (int r = lo; r < hi; ++r) {
    t_own += tpre[r];
    i_own += ipre[r];
  }
  unsigned t_incl = t_own;
  int i_incl = i_own;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const unsigned x = __shfl_up_sync(0xffffffffu, t_incl, off);
    const int y = __shfl_up_sync(0xffffffffu, i_incl, off);
    if (lane >= off) {
      t_incl += x;
      i_incl += y;
    }
  }
  if (lane == 31) {
    S.scan[wid] = t_incl;
    S.iscan[wid] = i_incl;
  }
  __syncthreads();
  unsigned all = 0, t_run = t_incl - t_own;
  int items = 0, i_run = i_incl - i_own;
  for (int w = 0; w < kThreads / 32; ++w) {
    all += S.scan[w];
    items += S.iscan[w];
    if (w < wid) {
      t_run += S.scan[w];
      i_run += S.iscan[w];
    }
  }
  for (int r = lo; r < hi; ++r) {
    const int t = tpre[r], i = ipre[r];
    tpre[r] = (int)t_run;
    ipre[r] = i_run;
    t_run += t;
    i_run += i;
  }
  if (tid == 0) {
    // Query lengths that increase count every token once, and the host has seen to it that their places fit 32 bits.
    // Others may count a token in many requests.  `high` sums each request's places without their lowest 12 bits,
    // which come to 2^23 at most: below 2^19 of it the sum of all is under 2^31 + 2^23, and shows by its top bit.
    int total = (int)all;
    if (S.high >= 1 << 19 || total < 0) {
      set_error(P.err, CB_DEVERR_BADLEN);
      total = items = 0;                               // no work
    }
    tpre[n] = total;
    ipre[n] = items;
    const int grid = gridDim.x, b = blockIdx.x, eff = max(1, min(grid, total));
    S.tiles = total;
    S.items = items;
    // whole items, dealt in turn: the first CTA's, the longest and mean ones; cut ones: an even share, joined
    const long long more = (items + grid - 1) / grid - 1;
    S.whole = items == 0 || S.longest + more * (total / items) <= (total + grid - 1) / grid + kJoinTiles;
    S.eff = S.whole ? grid : eff;
    S.u0 = b < eff ? (int)((long long)total * b / eff) : total;
    S.u1 = b < eff ? (int)((long long)total * (b + 1) / eff) : total;
  }
  if constexpr (ONE) {
    asm volatile("griddepcontrol.wait;" ::: "memory");   // so far only the requests' lengths were read (launch_after)
    if (tid == 0 && blockIdx.x == 0) signal_ready(P);
  }
  __syncthreads();
  if (tid == 0) {                      // the item that starts in this range and goes on after it
    Fp8Rec rec = {0, 0, 0, 0};
    if (!S.whole && S.u1 > S.u0 && S.u1 < S.tiles) {
      ItemIter<TOK, ONE> it(P, S, tpre, ipre);
      it.u = S.u1 - 1;
      it.locate();
      const int start = it.u - it.j0, first = start + kLead<ONE>, end = start + it.places();
      if (first >= S.u0 && first < S.u1 && end > S.u1)
        rec = {it.r, it.g, cta_of(end - 1, S.tiles, S.eff) - (int)blockIdx.x + 1, it.pair};
    }
    W.rec[blockIdx.x] = rec;
  }
}

// ---------------------------------------------------------------- items (warp 14)
// One warp walks the CTA's pieces and publishes them: the others need no
// registers for the walk.
template <int A, int TOK, bool ONE>
__device__ void publish(const Fp8Step& P, Smem<A>& S, const int* tpre, const int* ipre) {
  ItemIter<TOK, ONE> it(P, S, tpre, ipre);
  Item I;
  for (uint32_t i = 0;; ++i) {
    const bool more = it.next(I);
    if (!wwait(P, S, &S.item_empty[i % kItems], ((i / kItems) & 1) ^ 1)) break;
    if ((threadIdx.x & 31) == 0) {
      if (!more) I.a = I.b = 0;
      S.item[i % kItems] = I;
      mbar_arrive(&S.item_full[i % kItems]);
    }
    __syncwarp();
    if (!more) break;
  }
}
// A warp's walk over the published items.
template <class SM>
struct Items {
  uint32_t i = 0;
  __device__ const Item* next(const Fp8Step& P, SM& S) {
    if (!wwait(P, S, &S.item_full[i % kItems], (i / kItems) & 1)) return nullptr;
    const Item* I = &S.item[i % kItems];
    return I->b > I->a ? I : nullptr;
  }
  __device__ void done(SM& S, int v) { // the whole warp has read what it needs of it: v, from all of that
    arrive_after(&S.item_empty[i % kItems], (uint32_t)v);
    ++i;
  }
};

// ---------------------------------------------------------------- loads (warps 13 and 15)
// One warp brings K into the swizzled operand layout, the other (load_v) V and
// the exponent bytes as they are: neither waits for the other's buffers.
template <int A>
__device__ void load_tiles(const Fp8Step& P, const CUtensorMap* kmap, Smem<A>& S, bool load_v) {
  const unsigned FULL = 0xffffffffu;
  const int lane = threadIdx.x & 31, Hkv = P.cache.n_kv_heads, rows_total = P.cache.num_blocks * Hkv * kBlockSize;
  fence_proxy_async_global();           // the rows were appended by ordinary stores
  Items<Smem<A>> items;
  uint32_t n = 0;
  bool ok = true;
  while (ok) {
    const Item* item = items.next(P, S);
    if (!item) break;
    const int r = item->r, g = item->g, a = item->a, b = item->b, kv_hi = item->ctx + item->tok_hi;
    const int key_lo = P.window > 0 ? max(0, item->ctx + item->tok_lo - P.window + 1) : 0;
    items.done(S, r ^ g ^ a ^ b ^ kv_hi ^ key_lo);
    const int nblk = (kv_hi + kBlockSize - 1) / kBlockSize, blk_lo = key_lo / kBlockSize;
    // lane 8 t + i: entry of block i of tile base + t; 4 tiles at a time, the next 4 on their way.  Blocks
    // that no row of the item sees are not read: they may have been released.
    auto entry = [&](int base) {
      const int blk = base * 8 + lane;
      if (blk < blk_lo || blk >= nblk || base + (lane >> 3) >= b) return -2;
      const int e = __ldg(P.block_tables + (size_t)r * P.max_blocks_per_seq + blk);
      return e < 0 || e >= P.cache.num_blocks ? -1 : e;
    };
    int cur = -2, nxt = entry(a);
    for (int j = a; j < b && ok; ++j, ++n) {
      const int t = (j - a) & 3;
      if (t == 0) {
        cur = nxt;
        nxt = entry(j + 4);
        if (cur == -1 && !load_v) set_error(P.err, CB_DEVERR_BADBLOCK);   // its rows count as zeros
      }
      const int e = __shfl_sync(FULL, cur, t * 8 + (lane & 7));
      const bool have = lane < 8 && e >= 0;
      const int row = e >= 0 ? (e * Hkv + g) * kBlockSize : rows_total;    // past the extent: zeros
      const unsigned blocks = __popc(__ballot_sync(FULL, have));
      const uint32_t st = n & 1, ph = ((n >> 1) & 1) ^ 1;
      ok = wwait(P, S, load_v ? &S.vr_empty[st] : &S.k_empty[st], ph);
      if (!ok) break;
      if (!load_v) {
        if (lane == 0) mbar_arrive_expect_tx(&S.k_full[st], 128 * A);
        __syncwarp();
        if (lane < 8) tma_load_2d(&S.k[st][lane * kBlockSize * A], kmap, 0, row, &S.k_full[st]);
        continue;
      }
      if (lane == 0) mbar_arrive_expect_tx(&S.vr_full[st], blocks * kBlockSize * A);
      __syncwarp();
      if (have) bulk_load(&S.vr[st][lane * kBlockSize * A], P.cache.v + (size_t)row * A, kBlockSize * A, &S.vr_full[st]);
      // the exponents: lanes 0 .. 7 K's, 8 .. 15 V's; zeros, which no stored row has, where there is no block
      if (lane < 16)
        cp_async16(&S.ex[st][lane >> 3][(lane & 7) * kBlockSize], (lane < 8 ? P.cache.k_exps : P.cache.v_exps) + (e >= 0 ? row : 0), e >= 0);
      cp_async_arrive(&S.vr_full[st]);
    }
  }
  cp_async_wait_all();
  if (!ok)                             // copies already issued land before the CTA exits
    for (uint32_t i = n > 2u ? n - 2 : 0; i < n; ++i) mbar_wait(load_v ? &S.vr_full[i & 1] : &S.k_full[i & 1], (i >> 1) & 1, 20000000ull);
}

// ---------------------------------------------------------------- conversion of V (warps 8-11)
// This thread's query row as two e4m3 terms; returns its factor scale log2(e)
// 2^eq: finite and not 0 (keys out of sight are -inf times it), but NaN for a row that
// is not finite, whose terms are zeros.
// ready(): called between the loads and the first store; false: nothing is stored.
template <int A, class F>
__device__ float make_query(const Fp8Step& P, Smem<A>& S, int side, int row, int tok, int head, bool valid, F ready) {
  const uint4* src = reinterpret_cast<const uint4*>(P.q + ((size_t)tok * P.n_q_heads + head) * A);
  uint4 x[A / 8];
#pragma unroll
  for (int i = 0; i < A / 8; ++i) x[i] = valid ? __ldg(src + i) : make_uint4(0, 0, 0, 0);
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < A / 8; ++i)
    m = __vmaxu2(m, __vmaxu2(__vmaxu2(x[i].x & 0x7FFF7FFFu, x[i].y & 0x7FFF7FFFu), __vmaxu2(x[i].z & 0x7FFF7FFFu, x[i].w & 0x7FFF7FFFu)));
  m = max(m & 0xFFFFu, m >> 16);
  const bool bad = m >= 0x7F80u;
  const uint32_t eb = query_exp(m);
  const float factor = bad ? __uint_as_float(0x7FC00000u) : finite(fmaxf(P.scale_log2 * __uint_as_float(eb << 23), 1.4e-45f));
  if (!ready()) return factor;
  const float f = exp_inverse(bad ? 1u : eb);
#pragma unroll
  for (int c = 0; c < A / 16; ++c) {
    const uint32_t w[8] = {x[2 * c].x, x[2 * c].y, x[2 * c].z, x[2 * c].w, x[2 * c + 1].x, x[2 * c + 1].y, x[2 * c + 1].z, x[2 * c + 1].w};
    uint32_t t0[4], t1[4];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float y0 = bad ? 0.f : bf16lo(w[i]) * f, y1 = bad ? 0.f : bf16hi(w[i]) * f;
      uint32_t hi, lo;
      query_terms(y0, y1, hi, lo);
      t0[i / 2] = (i & 1) ? t0[i / 2] | (hi << 16) : hi;
      t1[i / 2] = (i & 1) ? t1[i / 2] | (lo << 16) : lo;
    }
    const uint32_t at = smem_u32(S.q[side]) + row * A + ((A == 128 ? c ^ (row & 7) : c ^ ((row >> 1) & 3)) << 4);
    sts128(at, make_uint4(t0[0], t0[1], t0[2], t0[3]));
    sts128(at + 128 * A, make_uint4(t1[0], t1[1], t1[2], t1[3]));
  }
  fence_proxy_async_smem();
  mbar_arrive(&S.q_full[side]);
  return factor;
}

// ONE: also the query rows of each single-token item, while the softmax is still
// at the item before.
template <int A, int G, bool ONE>
__device__ void convert(const Fp8Step& P, Smem<A>& S) {
  constexpr int LR = A / 16, RP = 32 / LR, N = 32 / RP;   // lanes per row, rows per step, steps
  const unsigned FULL = 0xffffffffu;
  const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) & 3;
  const int col = lane % LR, rsub = lane / LR, key_l = 32 * warp + lane;
  // 16 dimensions: two 16-byte chunks of the half's 128-byte row; lanes of the second half store them in
  // the other order (the halves share banks)
  const int c = (col & 3) * 2, sw = A == 128 ? col >> 2 : 0;
  Items<Smem<A>> items;
  uint32_t n = 0;
  bool ok = true;
  while (ok) {
    const Item* item = items.next(P, S);
    if (!item) break;
    const int a = item->a, b = item->b, kv_hi = item->ctx + item->tok_hi, tok = item->q0, head = item->g * G + lane;
    const int key_lo = P.window > 0 ? max(0, item->ctx + item->tok_lo - P.window + 1) : 0;
    const uint32_t it = items.i;
    items.done(S, a ^ b ^ kv_hi ^ key_lo ^ tok ^ head);
    if constexpr (ONE) {
      // (every tile of the item before is converted: nothing that its S waits for waits for this warp)
      const float fq = make_query<A>(P, S, 0, 32 * warp + lane, tok, head, lane < G,
                                     [&] { return ok = it == 0 || wwait(P, S, &S.q_free, (it - 1) & 1); });
      if (!ok) break;
      if (warp == 0) sts32(smem_u32(&S.fq[it & 3][lane]), __float_as_uint(fq));
    }
    for (int j = a; j < b; ++j, ++n) {
      const uint32_t st = n & 1, ph = (n >> 1) & 1;
      ok = wwait(P, S, &S.vr_full[st], ph);
      if (!ok) break;
      // this lane's key: its factors.  Values that no row of the item sees, and rows of NaNs, become zeros
      // (0 * NaN must not reach O); the latter are told to the softmax, for the rows that see them.  So do those
      // of a bad block id (exponent byte 0), whose rows were not copied.
      const uint32_t kb = lds8(smem_u32(&S.ex[st][0][key_l])), vb = lds8(smem_u32(&S.ex[st][1][key_l]));
      const int key = j * kTileN + key_l;
      const bool seen = key >= key_lo && key < kv_hi, nan = vb == kExpNan;
      uint32_t ke = 1;                                         // the largest exponent byte of the keys that are seen
      if constexpr (ONE) {
        if (seen && kb != kExpNan) ke = kb;
      } else {                                                 // each warp for itself: lane l takes keys 4 l .. 4 l + 3 of the tile
        const uint32_t kb4 = lds32(smem_u32(&S.ex[st][0][4 * lane]));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t b = (kb4 >> (8 * i)) & 255u;
          const int k = j * kTileN + 4 * lane + i;
          if (k >= key_lo && k < kv_hi && b != kExpNan) ke = max(ke, b);
        }
      }
      ke = max(__reduce_max_sync(FULL, ke), 227u) - 100u;
      const int d = (int)(kb + 127u) - (int)ke;                // ek - E + 127
      sts32(smem_u32(&S.fk[n & 3][key_l]), kb == kExpNan ? 0x7FC00000u : d > 0 ? (uint32_t)d << 23 : 0x400000u >> min(-d, 31));
      const unsigned bad = __ballot_sync(FULL, nan && seen);
      if (lane == 0) {
        sts32(smem_u32(&S.v_nan[n & 3][warp]), bad);
        sts32(smem_u32(&S.fe[n & 3][warp]), ke << 23);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.fk_full[n & 3]);
      const uint32_t f1 = seen && !nan && vb != 0u ? factor1(vb) : 0u;
      const bool large = __any_sync(FULL, seen && !nan && vb > 134u);
      const uint32_t src = smem_u32(&S.vr[st][32 * warp * A + lane * 16]), dst = smem_u32(&S.v[st][sw][32 * warp + rsub][0]);
      auto put = [&](int p, const uint4& x) {
        const int row = p * RP + rsub;
        uint32_t o[8];
        const uint32_t f = __shfl_sync(FULL, f1, row);
        widen8(x.x, x.y, f, o);
        widen8(x.z, x.w, f, o + 4);
        if (large) {
          const uint32_t f2 = factor2(__shfl_sync(FULL, vb, row));
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] = mul_bf16x2(o[i], f2);
        }
        const uint4 x0 = make_uint4(o[0], o[1], o[2], o[3]), x1 = make_uint4(o[4], o[5], o[6], o[7]);
        sts128(dst + p * RP * 128 + (((c + sw) ^ (row & 7)) << 4), sw ? x1 : x0);
        sts128(dst + p * RP * 128 + (((c + 1 - sw) ^ (row & 7)) << 4), sw ? x0 : x1);
      };
      if constexpr (ONE) {
        // The conversion is the longest part of a tile's chain here and registers are free: the staged tile is
        // read at once and its buffer given back before the stores (165 -> 156 us for 256 MQA decodes).
        uint4 x[N];
#pragma unroll
        for (int p = 0; p < N; ++p) x[p] = lds128(src + p * 512);
        uint32_t all = 0;
#pragma unroll
        for (int p = 0; p < N; ++p) all ^= x[p].x ^ x[p].y ^ x[p].z ^ x[p].w;
        arrive_after(&S.vr_empty[st], all ^ kb ^ vb);
        ok = wwait(P, S, &S.v_empty[st], ph ^ 1);
        if (!ok) break;
#pragma unroll
        for (int p = 0; p < N; ++p) put(p, x[p]);
      } else {
        ok = wwait(P, S, &S.v_empty[st], ph ^ 1);
        if (!ok) break;
#pragma unroll 2
        for (int p = 0; p < N; ++p) put(p, lds128(src + p * 512));
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&S.v_full[st]);
        if constexpr (!ONE) mbar_arrive(&S.vr_empty[st]);
      }
    }
  }
}

// ---------------------------------------------------------------- products (warp 12)
template <int A>
__device__ void issue(const Fp8Step& P, Smem<A>& S) {
  constexpr uint32_t kIdescS = idesc_f8(128, 128, 0, 0, 0, 0), kIdescO = idesc_bf16_f32(128, A, 1);
  constexpr uint32_t kHalf = 128 * 128, kTile = (A / 64) * kHalf;
  constexpr int kLayout = A == 128 ? 2 : 4;
  const uint64_t qd = smem_desc(smem_u32(S.q), 16, 8 * A, kLayout), kd = smem_desc(smem_u32(S.k), 16, 8 * A, kLayout);
  const uint64_t vd = smem_desc_sw128(smem_u32(S.v), kHalf, 1024);
  Items<Smem<A>> items;
  uint32_t n = 0, np[2] = {0, 0};      // key tiles before this item; products with P issued per side
  uint32_t ni[2] = {0, 0};             // items per side
  bool ok = true;
  while (ok) {
    const Item* item = items.next(P, S);
    if (!item) break;
    const int len = item->b - item->a, sides = item->sides;
    items.done(S, len ^ sides);
    for (int j = 0; j <= len && ok; ++j) {
#pragma unroll
      for (int side = 0; side < 2; ++side) {
        if (side >= sides || !ok) break;
        const uint32_t s_t = S.tmem + side * 128, o_t = S.tmem + 256 + side * A;
        if (j > 0) {                   // O += P V of the tile before
          const uint32_t t = n + j - 1, st = t & 1;
          ok = wwait(P, S, &S.v_full[st], (t >> 1) & 1);
          if (ok && j == 1) ok = wwait(P, S, &S.o_free[side], (ni[side] & 1) ^ 1);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            ok = ok && wwait(P, S, &S.p_full[side][h], np[side] & 1);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
              for (int ks = 4 * h; ks < 4 * h + 4; ++ks)
                tc_mma_f16_ts(o_t, s_t + ks * 8, vd + (uint32_t)((st * kTile + ks * 16 * 128) >> 4), kIdescO, (j > 1 || ks > 0) ? 1u : 0u);
              if (h == 1) {
                if (side == sides - 1) tc_commit(&S.v_empty[st]);
                if (j == len) tc_commit(&S.o_full[side]);
              }
            }
            __syncwarp();
          }
          if (!ok) break;
          ++np[side];
        }
        if (j < len) {                 // S of this one
          const uint32_t t = n + j, st = t & 1;
          if (j == 0) ok = wwait(P, S, &S.q_full[side], ni[side] & 1);
          ok = ok && wwait(P, S, &S.k_full[st], (t >> 1) & 1);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int term = 0; term < 2; ++term)
#pragma unroll
              for (int d = 0; d < A / 32; ++d)
                mma_f8(s_t, qd + (uint32_t)((((side * 2 + term) * 128 * A) >> 4) + 2 * d), kd + (uint32_t)(((st * 128 * A) >> 4) + 2 * d),
                       kIdescS, term > 0 || d > 0);
            tc_commit(&S.s_full[side]);
            if (side == sides - 1) tc_commit(&S.k_empty[st]);
          }
          __syncwarp();
        }
      }
    }
    n += len;
    ++ni[0];
    if (sides == 2) ++ni[1];
  }
  if (!ok) S.abort = 1;
  if (elect_one()) tc_commit(&S.drain);
  __syncwarp();
  mbar_wait(&S.drain, 0, 20000000ull);
}

// ---------------------------------------------------------------- softmax (warps 0-3, 4-7)
// One key tile (number n; this query tile's S in s_t, its O in o_t) of this
// thread's row: its weights into tensor memory, m and l brought up to date.
// fr: the row's factor; it sees the keys lo .. pos.  fresh: O holds nothing yet.
template <int A>
__device__ __forceinline__ void softmax_tile(Smem<A>& S, uint32_t s_t, uint32_t o_t, int side, uint32_t n, int key0, bool fresh, float fr,
                                             int lo, int pos, float& m, float& l) {
  const unsigned FULL = 0xffffffffu;
  const int lane = threadIdx.x & 31;
  const unsigned span = (unsigned)(pos - lo);                // key k is visible iff (unsigned)(k - lo) <= span
  float s[128];
#pragma unroll
  for (int c = 0; c < 4; ++c) tmem_ld32(s_t + 32 * c, reinterpret_cast<float (&)[32]>(s[32 * c]));
  tmem_wait_ld();
  const float4* fk = reinterpret_cast<const float4*>(S.fk[n & 3]);
#pragma unroll
  for (int k = 0; k < 32; ++k) {
    const float4 f = fk[k];
    f2split(fmul2(f2(s[4 * k], s[4 * k + 1]), f2(f.x, f.y)), s[4 * k], s[4 * k + 1]);
    f2split(fmul2(f2(s[4 * k + 2], s[4 * k + 3]), f2(f.z, f.w)), s[4 * k + 2], s[4 * k + 3]);
  }
  const uint4 vn = *reinterpret_cast<const uint4*>(S.v_nan[n & 3]);
  if (__any_sync(FULL, key0 + kTileN - 1 > pos || key0 < lo || (vn.x | vn.y | vn.z | vn.w) != 0)) {
    // keys out of sight; visible ones whose value row is NaNs
#pragma unroll
    for (int k = 0; k < 128; ++k) {
      const uint32_t w = k < 32 ? vn.x : k < 64 ? vn.y : k < 96 ? vn.z : vn.w;
      if ((w >> (k & 31)) & 1) s[k] = __uint_as_float(0x7FC00000u);
      if ((unsigned)(key0 + k - lo) > span) s[k] = kNegInf;
    }
  }
  float a[4] = {kNegInf, kNegInf, kNegInf, kNegInf};
#pragma unroll
  for (int k = 0; k < 128; k += 2) a[(k >> 1) & 3] = max3(a[(k >> 1) & 3], s[k], s[k + 1]);
  const float fq = finite(fr * S.fe[n & 3][0]);
  const float mt = max3(a[0], a[1], fmaxf(a[2], a[3])) * fq;
  const bool need = mt > m + 8.f;
  float alpha = 1.f;
  if (need) {
    alpha = ex2(m - mt);
    m = mt;
  }
  if (!fresh && __any_sync(FULL, need)) {
#pragma unroll 1
    for (int c = 0; c < A / 8; ++c) {
      float o[8];
      tmem_ld8(o_t + c * 8, o);
      tmem_wait_ld();
#pragma unroll
      for (int k = 0; k < 8; ++k) o[k] *= alpha;
      tmem_st8(o_t + c * 8, o);
    }
  }
  l *= alpha;
  const float mr = m == kNegInf ? 0.f : m;               // a row that has seen no key yet: every p is 0
  const uint64_t fq2 = f2(fq, fq), nm2 = f2(-mr, -mr);
  uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t pk[32];
#pragma unroll
    for (int k = 0; k < 32; ++k) {
      float t0, t1;
      f2split(ffma2(f2(s[64 * h + 2 * k], s[64 * h + 2 * k + 1]), fq2, nm2), t0, t1);
      t0 = ex2(t0);
      t1 = ex2(t1);
      sum[k & 1] = fadd2(sum[k & 1], f2(t0, t1));
      pk[k] = pack_bf16(t0, t1);
    }
    tmem_st32u(s_t + 32 * h, pk);
    tmem_wait_st();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&S.p_full[side][h]);
  }
  float r0, r1, r2, r3;
  f2split(sum[0], r0, r1);
  f2split(sum[1], r2, r3);
  l += (r0 + r1) + (r2 + r3);
}

template <int A, int G>
__device__ void softmax(const Fp8Step& P, const Fp8Partials& W, Smem<A>& S, int side) {
  constexpr int TOK = kTileM / G;
  const int row = threadIdx.x & 127, lane = threadIdx.x & 31;
  const uint32_t lane_base = (uint32_t)(row & ~31) << 16;
  const uint32_t s_t = S.tmem + lane_base + side * 128, o_t = S.tmem + lane_base + 256 + side * A;
  Items<Smem<A>> items;
  uint32_t n = 0, ns = 0, ni = 0;      // key tiles of all items, of this side's items; this side's items
  const Item* item = nullptr;
  // the next item that has this side, its query rows made ready
  auto next_item = [&](float& fr) {
    while ((item = items.next(P, S)) != nullptr) {
      if (side < item->sides) {
        const int ti = item->tok_lo + side * TOK + row / G;
        fr = make_query<A>(P, S, side, row, item->q0 + ti, item->g * G + row % G, ti < item->tok_hi, [] { return true; });
        return;
      }
      n += item->b - item->a;
      items.done(S, n);
    }
  };
  float fr = 0.f;
  next_item(fr);
  while (item) {
    const int ti = item->tok_lo + side * TOK + row / G, tok_hi = item->tok_hi, a0 = item->a, b0 = item->b;
    const int pos = item->ctx + min(ti, tok_hi - 1);         // the last key this row sees
    const int lo = P.window > 0 ? max(0, pos - P.window + 1) : 0;
    const bool began = a0 > item->first, cut = began || b0 < item->end;
    uint16_t* dst = P.out + ((size_t)(item->q0 + ti) * P.n_q_heads + (size_t)item->g * G + row % G) * A;
    items.done(S, tok_hi ^ a0 ^ b0 ^ pos ^ lo ^ ti ^ (int)cut ^ (int)(uintptr_t)dst);
    float m = kNegInf, l = 0.f;
    bool ok = true;
    for (int j = a0; j < b0; ++j, ++n, ++ns) {
      // The factors' barrier comes first: it is usually complete by now.  For a piece's first tile it may be
      // several phases behind until S is done (the V of the tile before is then converted).
      ok = j > a0 || wwait(P, S, &S.s_full[side], ns & 1);
      ok = ok && wwait(P, S, &S.fk_full[n & 3], (n >> 2) & 1) && wwait(P, S, &S.s_full[side], ns & 1);   // O holds all products before
      if (!ok) break;
      tc_fence_after();
      softmax_tile<A>(S, s_t, o_t, side, n, j * kTileN, j == a0, fr, lo, pos, m, l);
    }
    if (!ok) {
      S.abort = 1;
      break;
    }
    // the next item's query first: its first scores are computed during this one's output
    next_item(fr);
    if (!wwait(P, S, &S.o_full[side], ni & 1)) break;
    tc_fence_after();
    const float inv = l != 0.f ? 1.f / l : 0.f;              // 0: a piece in which the row saw no key
    // a range's first piece that began before it is 2b, any other one that is cut 2b + 1
    const size_t piece = (size_t)2 * blockIdx.x + (began ? 0 : 1);
    const int prow = side * kTileM + row;
    if (cut) *reinterpret_cast<float2*>(W.ml + (piece * kRows + prow) * 2) = make_float2(m, l);
#pragma unroll 1
    for (int c = 0; c < A / 32; ++c) {
      float o[32];
      tmem_ld32(o_t + 32 * c, o);
      tmem_wait_ld();
      if (cut) {
        // 4 dimensions of all rows together: a warp's store is 512 bytes in a row
        float4* d = reinterpret_cast<float4*>(W.acc) + (piece * (A / 4) + 8 * c) * kRows + prow;
#pragma unroll
        for (int k = 0; k < 8; ++k) d[k * kRows] = make_float4(o[4 * k] * inv, o[4 * k + 1] * inv, o[4 * k + 2] * inv, o[4 * k + 3] * inv);
      } else if (ti < tok_hi) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          *reinterpret_cast<uint4*>(dst + 32 * c + 8 * k) =
              make_uint4(pack_bf16(o[8 * k] * inv, o[8 * k + 1] * inv), pack_bf16(o[8 * k + 2] * inv, o[8 * k + 3] * inv),
                         pack_bf16(o[8 * k + 4] * inv, o[8 * k + 5] * inv), pack_bf16(o[8 * k + 6] * inv, o[8 * k + 7] * inv));
      }
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&S.o_free[side]);
    ++ni;
  }
}

// ---------------------------------------------------------------- single tokens (groups of 16 and 32 heads)
// A step's requests with one new token: an item is (request, KV head) with G rows.
// A query tile holds them four times, at rows 0, 32, 64 and 96, and warp w's copy
// takes the tile's keys 32 w .. 32 w + 31 only (its weights of the others are zeros),
// so that the four warps of a tile share its softmax (one warp per tile: 220 us
// instead of 199 for 256 requests).  Both tiles of tensor memory take the same rows,
// A the even key tiles and B the odd ones, and one's softmax runs under the other's
// products.  At the end of an item the eight copies' (m, l, O) are joined through
// shared memory (Q's second tile, not used here).  The warps that convert V write
// the next item's query rows as soon as this one's last S is done (199 -> 179 us).
template <int A>
__device__ void issue_one(const Fp8Step& P, Smem<A>& S) {
  constexpr uint32_t kIdescS = idesc_f8(128, 128, 0, 0, 0, 0), kIdescO = idesc_bf16_f32(128, A, 1);
  constexpr uint32_t kHalf = 128 * 128, kTile = (A / 64) * kHalf;
  constexpr int kLayout = A == 128 ? 2 : 4;
  const uint64_t qd = smem_desc(smem_u32(S.q), 16, 8 * A, kLayout), kd = smem_desc(smem_u32(S.k), 16, 8 * A, kLayout);
  const uint64_t vd = smem_desc_sw128(smem_u32(S.v), kHalf, 1024);
  Items<Smem<A>> items;
  uint32_t n = 0, i = 0;               // key tiles and items before this one
  uint32_t np[2] = {0, 0}, nb = 0;     // products with P issued per side; items in which B has tiles
  bool ok = true;
  while (ok) {
    const Item* item = items.next(P, S);
    if (!item) break;
    const int len = item->b - item->a;
    items.done(S, len);
    for (int t0 = 0; t0 < len + 2 && ok; t0 += 2) {
#pragma unroll
      for (int side = 0; side < 2; ++side) {
        const int t = t0 + side;
        const uint32_t s_t = S.tmem + side * 128, o_t = S.tmem + 256 + side * A;
        const uint32_t st = (n + t) & 1;                     // the stage of tile t and of tile t - 2
        if (t >= 2 && t - 2 < len) {   // O += P V of this side's tile before
          ok = ok && wwait(P, S, &S.v_full[st], ((n + t - 2) >> 1) & 1);
          if (t < 4) ok = ok && wwait(P, S, &S.o_free[side], ((side ? nb : i) & 1) ^ 1);
          ok = ok && wwait(P, S, &S.p_full[side][0], np[side] & 1);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)
              tc_mma_f16_ts(o_t, s_t + ks * 8, vd + (uint32_t)((st * kTile + ks * 16 * 128) >> 4), kIdescO, (t >= 4 || ks > 0) ? 1u : 0u);
            tc_commit(&S.v_empty[st]);
            if (t >= len) tc_commit(&S.o_full[side]);
          }
          __syncwarp();
          ++np[side];
        }
        if (t < len) {
          if (t == 0) ok = ok && wwait(P, S, &S.q_full[0], i & 1);
          ok = ok && wwait(P, S, &S.k_full[st], ((n + t) >> 1) & 1);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int term = 0; term < 2; ++term)
#pragma unroll
              for (int d = 0; d < A / 32; ++d)
                mma_f8(s_t, qd + (uint32_t)(((term * 128 * A) >> 4) + 2 * d), kd + (uint32_t)(((st * 128 * A) >> 4) + 2 * d), kIdescS,
                       term > 0 || d > 0);
            tc_commit(&S.s_full[side]);
            tc_commit(&S.k_empty[st]);
            if (t == len - 1) tc_commit(&S.q_free);
          }
          __syncwarp();
        }
        if (!ok) break;
      }
    }
    n += len;
    ++i;
    if (len > 1) ++nb;
  }
  if (!ok) S.abort = 1;
  if (elect_one()) tc_commit(&S.drain);
  __syncwarp();
  mbar_wait(&S.drain, 0, 20000000ull);
}

// Bounded meeting of the eight softmax warps (phase: counted by the caller; v: of
// the values loaded from what is overwritten after it).
template <class SM>
__device__ __forceinline__ bool meet(const Fp8Step& P, SM& S, uint32_t& phase, float v = 0.f) {
  __syncwarp();
  arrive_after(&S.x_bar, __float_as_uint(v));
  return wwait(P, S, &S.x_bar, phase++ & 1);
}

template <int A, int G>
__device__ void softmax_one(const Fp8Step& P, const Fp8Partials& W, Smem<A>& S, int side) {
  static_assert(G <= 32 && 8 * 32 * 32 * 4 <= (int)sizeof(S.q[1]), "32 dimensions of each side's copies fit in Q's second tile");
  const unsigned FULL = 0xffffffffu;
  const int lane = threadIdx.x & 31, w = (threadIdx.x >> 5) & 3, copy = 4 * side + w;
  const uint32_t lanes = (uint32_t)(32 * w) << 16;
  const uint32_t s_t = S.tmem + lanes + side * 128, o_t = S.tmem + lanes + 256 + side * A, xs = smem_u32(S.q[1]);
  Items<Smem<A>> items;
  uint32_t n = 0, ns = 0, nb = 0, phase = 0;   // key tiles of all items; this side's; items in which B has tiles
  for (uint32_t i = 0;; ++i) {
    const Item* item = items.next(P, S);
    if (!item) break;
    const int a0 = item->a, b0 = item->b, pos = item->ctx, g = item->g;
    const int lo = P.window > 0 ? max(0, pos - P.window + 1) : 0;
    const unsigned span = (unsigned)(pos - lo);                // key k is visible iff (unsigned)(k - lo) <= span
    const bool began = a0 > item->first, cut = began || b0 < item->end;
    const int tok = item->q0;
    bool ok = true;
    float fr = 0.f;
    items.done(S, a0 ^ b0 ^ pos ^ g ^ tok ^ (int)cut);
    float m = kNegInf, l = 0.f;
    for (int j = a0 + side; j < b0; j += 2, ++ns) {
      const uint32_t nj = n + (j - a0);
      // (the factors' barrier: see softmax())
      ok = j > a0 + side || wwait(P, S, &S.s_full[side], ns & 1);
      ok = ok && wwait(P, S, &S.fk_full[nj & 3], (nj >> 2) & 1) && wwait(P, S, &S.s_full[side], ns & 1);
      if (!ok) break;
      tc_fence_after();
      float s[32];
      tmem_ld32(s_t + 32 * w, s);
      const uint32_t fk = smem_u32(&S.fk[nj & 3][32 * w]);
      const uint32_t vn = lds32(smem_u32(&S.v_nan[nj & 3][w]));
      const float fe = lds32f(smem_u32(&S.fe[nj & 3][w]));
      if (j == a0 + side) fr = lds32f(smem_u32(&S.fq[i & 3][lane]));   // written before the first tile's factors
      const float fq = finite(fr * fe);
      const int key = j * kTileN + 32 * w;
      tmem_wait_ld();
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint4 f = lds128(fk + 16 * k);
        f2split(fmul2(f2(s[4 * k], s[4 * k + 1]), f2(__uint_as_float(f.x), __uint_as_float(f.y))), s[4 * k], s[4 * k + 1]);
        f2split(fmul2(f2(s[4 * k + 2], s[4 * k + 3]), f2(__uint_as_float(f.z), __uint_as_float(f.w))), s[4 * k + 2], s[4 * k + 3]);
      }
      if (key + 31 > pos || key < lo || vn != 0) {             // the same in every lane
#pragma unroll
        for (int k = 0; k < 32; ++k) {
          if ((vn >> k) & 1) s[k] = __uint_as_float(0x7FC00000u);
          if ((unsigned)(key + k - lo) > span) s[k] = kNegInf;
        }
      }
      float a[2] = {kNegInf, kNegInf};
#pragma unroll
      for (int k = 0; k < 32; k += 2) a[(k >> 1) & 1] = max3(a[(k >> 1) & 1], s[k], s[k + 1]);
      const float mt = fmaxf(a[0], a[1]) * fq;
      const bool need = mt > m + 8.f;
      float alpha = 1.f;
      if (need) {
        alpha = ex2(m - mt);
        m = mt;
      }
      if (j > a0 + side && __any_sync(FULL, need)) {
#pragma unroll 1
        for (int c = 0; c < A / 8; ++c) {
          float o[8];
          tmem_ld8(o_t + c * 8, o);
          tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < 8; ++k) o[k] *= alpha;
          tmem_st8(o_t + c * 8, o);
        }
      }
      const float mr = m == kNegInf ? 0.f : m;                 // no key seen yet: every weight is 0
      const uint64_t fq2 = f2(fq, fq), nm2 = f2(-mr, -mr);
      uint64_t sum[2] = {0ull, 0ull};
      uint32_t pk[16], zero[16];
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        float t0, t1;
        f2split(ffma2(f2(s[2 * k], s[2 * k + 1]), fq2, nm2), t0, t1);
        t0 = ex2(t0);
        t1 = ex2(t1);
        sum[k & 1] = fadd2(sum[k & 1], f2(t0, t1));
        pk[k] = pack_bf16(t0, t1);
        zero[k] = 0u;
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (q == w)
          tmem_st16u(s_t + 16 * q, pk);
        else
          tmem_st16u(s_t + 16 * q, zero);
      }
      float r0, r1, r2, r3;
      f2split(sum[0], r0, r1);
      f2split(sum[1], r2, r3);
      l = l * alpha + ((r0 + r1) + (r2 + r3));
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.p_full[side][0]);
    }
    const bool both = a0 + 1 < b0;                             // B has tiles
    ok = ok && wwait(P, S, &S.o_full[0], i & 1) && (!both || wwait(P, S, &S.o_full[1], nb & 1));
    if (!ok) {
      S.abort = 1;
      break;
    }
    tc_fence_after();
    // the copies' maxima and sums; then O, half of the dimensions per side, 32 of them at a time: a warp adds both
    // tiles' rows, then four warps' copies are added through shared memory
    sts32(xs + (copy * 32 + lane) * 8, __float_as_uint(m));
    sts32(xs + (copy * 32 + lane) * 8 + 4, __float_as_uint(l));
    if (!meet(P, S, phase)) break;
    float mm = kNegInf, ls = 0.f, f[2];
    for (int c = 0; c < 8; ++c) mm = fmaxf(mm, lds32f(xs + (c * 32 + lane) * 8));
    // -inf: no key seen, or NaNs only (then the sum is one)
    auto weight = [&](int c, float& lc) {
      const float mc = lds32f(xs + (c * 32 + lane) * 8);
      lc = lds32f(xs + (c * 32 + lane) * 8 + 4);
      return mc == kNegInf ? (lc != 0.f ? 1.f : 0.f) : ex2(mc - mm);
    };
    for (int c = 0; c < 8; ++c) {
      float lc;
      const float wc = weight(c, lc);
      ls += wc * lc;
      if ((c & 3) == w) f[c >> 2] = wc;
    }
    f[0] /= ls;
    f[1] /= ls;
    float read = f[0] + f[1];
    const size_t pr = ((size_t)2 * blockIdx.x + (began ? 0 : 1)) * kSingleRows;
    if (cut && copy == 0 && lane < G) *reinterpret_cast<float2*>(W.ml + (pr + lane) * 2) = make_float2(mm, ls);
    const uint32_t o_a = S.tmem + lanes + 256, xh = xs + side * (128 * 128);
#pragma unroll 1
    for (int c = 0; c < A / 64 && ok; ++c) {
      const int d0 = (A / 2) * side + 32 * c;                  // this side's dimensions
      float o[32], ob[32];
      tmem_ld32(o_a + d0, o);
      if (both) tmem_ld32(o_a + A + d0, ob);
      tmem_wait_ld();
#pragma unroll
      for (int k = 0; k < 32; ++k) o[k] = both ? o[k] * f[0] + ob[k] * f[1] : o[k] * f[0];
      ok = meet(P, S, phase, read);                            // what was there has been read
      // row `lane` of this copy: 32 values, their 16-byte chunks in an order that spreads the banks
#pragma unroll
      for (int k = 0; k < 8; ++k)
        sts128(xh + (w * 32 + lane) * 128 + ((k ^ (lane & 7)) << 4),
               make_uint4(__float_as_uint(o[4 * k]), __float_as_uint(o[4 * k + 1]), __float_as_uint(o[4 * k + 2]), __float_as_uint(o[4 * k + 3])));
      ok = ok && meet(P, S, phase);
      // this side's 128 threads: rows r and r + 16, dimensions 4 k .. 4 k + 3
      const int k = threadIdx.x & 7;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = 16 * h + ((threadIdx.x & 127) >> 3);
        float y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint4 x = lds128(xh + (q * 32 + r) * 128 + ((k ^ (r & 7)) << 4));
          y[0] += __uint_as_float(x.x);
          y[1] += __uint_as_float(x.y);
          y[2] += __uint_as_float(x.z);
          y[3] += __uint_as_float(x.w);
        }
        read = h == 0 ? y[0] + y[1] + y[2] + y[3] : read + (y[0] + y[1] + y[2] + y[3]);
        if (ok && r < G) {
          if (cut)
            *reinterpret_cast<float4*>(W.acc + (pr + r) * A + d0 + 4 * k) = make_float4(y[0], y[1], y[2], y[3]);
          else
            *reinterpret_cast<uint2*>(P.out + ((size_t)tok * P.n_q_heads + (size_t)g * G + r) * A + d0 + 4 * k) =
                make_uint2(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]));
        }
      }
    }
    if (!ok) break;
    tc_fence_before();
    if (!meet(P, S, phase, read)) break;                       // the exchange is free for the next item
    if (lane == 0) {
      mbar_arrive(&S.o_free[0]);
      if (both) mbar_arrive(&S.o_free[1]);
    }
    nb += both;
    n += b0 - a0;
  }
}

template <int A, int G, bool ONE>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_fp8_kernel(const Fp8Step P, const Fp8Partials W, const __grid_constant__ CUtensorMap kmap) {
  constexpr int TOK = kTileM / G;
  extern __shared__ uint8_t smem_raw[];
  Smem<A>& S = *reinterpret_cast<Smem<A>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  int* tpre = reinterpret_cast<int*>(&S + 1);
  int* ipre = tpre + P.n_reqs + 1;
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&S.q_full[i], 128);
      mbar_init(&S.k_full[i], 1);
      mbar_init(&S.k_empty[i], 1);
      mbar_init(&S.vr_full[i], 1 + 32);   // the values' copies; each lane's of the exponents
      mbar_init(&S.vr_empty[i], 4);
      mbar_init(&S.v_full[i], 4);
      mbar_init(&S.v_empty[i], 1);
      mbar_init(&S.s_full[i], 1);
      mbar_init(&S.p_full[i][0], 4);
      mbar_init(&S.p_full[i][1], 4);
      mbar_init(&S.o_full[i], 1);
      mbar_init(&S.o_free[i], ONE ? 8 : 4);
    }
    mbar_init(&S.q_free, 1);
    mbar_init(&S.x_bar, 8);
    for (int i = 0; i < 4; ++i) mbar_init(&S.fk_full[i], 4);
    for (int i = 0; i < kItems; ++i) {
      mbar_init(&S.item_full[i], 1);
      mbar_init(&S.item_empty[i], kReaders);
    }
    mbar_init(&S.drain, 1);
    S.abort = 0;
    fence_mbar_init();
    prefetch_tmap(&kmap);
  }
  if (warp == 12) {
    tmem_alloc(&S.tmem, 512);
    tmem_relinquish();
    tc_fence_before();
  }
  make_plan<A, TOK, ONE>(P, W, S, tpre, ipre);
  __syncthreads();
  tc_fence_after();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // registers of the four warpgroups: 2 x 176 + 72 + 88 = 4 x 128, what the launch holds (single tokens: 128 each)
  if (warp < 8) {
    if constexpr (!ONE) asm volatile("setmaxnreg.inc.sync.aligned.u32 176;");
    if constexpr (ONE)
      softmax_one<A, G>(P, W, S, warp >> 2);
    else
      softmax<A, G>(P, W, S, warp >> 2);
  } else if (warp < 12) {
    if constexpr (!ONE) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    convert<A, G, ONE>(P, S);
  } else {
    if constexpr (!ONE) asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp == 12) {
      if constexpr (ONE)
        issue_one<A>(P, S);
      else
        issue<A>(P, S);
    }
    if (warp == 13 || warp == 15) load_tiles<A>(P, &kmap, S, warp == 15);
    if (warp == 14) publish<A, TOK, ONE>(P, S, tpre, ipre);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    tmem_dealloc(S.tmem, 512);
  }
  // This grid ends after the single tokens' does, so that the joining kernel has both.
  if constexpr (!ONE) asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <int A>
size_t smem_bytes(int n_reqs) {
  return 1024 + sizeof(Smem<A>) + (size_t)(n_reqs + 1) * 8;
}
static_assert(sizeof(Smem<128>) + 1024 + (kMaxReqs + 1) * 8 <= kSmemLimit, "shared memory");

template <int A, int G, bool ONE>
cudaError_t launch_t(const Fp8Step& s, const Fp8Partials& w, int grid, bool chained, cudaStream_t stream) {
  CUtensorMap km;
  const long long rows = (long long)s.cache.num_blocks * s.cache.n_kv_heads * kBlockSize;
  if (!encode_byte_rows(&km, s.cache.k, rows, A, kBlockSize)) return cudaErrorInvalidValue;
  cudaError_t e = opt_in_smem(reinterpret_cast<const void*>(chunk_fp8_kernel<A, G, ONE>), kSmemLimit);
  if (e != cudaSuccess) return e;
  return launch_after(chained, chunk_fp8_kernel<A, G, ONE>, grid, kThreads, smem_bytes<A>(s.n_reqs), stream, s, w, km);
}

}  // namespace

cudaError_t launch_chunk_fp8(const Fp8Step& s, const Fp8Partials& w, bool single, int grid, bool chained, cudaStream_t stream) {
  const int a = s.cache.head_dim, g = s.n_q_heads / s.cache.n_kv_heads;
#define CB_CASE(A_, G_, ONE_) \
  if (a == A_ && g == G_ && single == ONE_) return launch_t<A_, G_, ONE_>(s, w, grid, chained, stream);
  CB_CASE(128, 1, false)
  CB_CASE(128, 2, false)
  CB_CASE(128, 4, false)
  CB_CASE(128, 8, false)
  CB_CASE(128, 16, false)
  CB_CASE(128, 16, true)
  CB_CASE(128, 32, false)
  CB_CASE(128, 32, true)
  CB_CASE(64, 1, false)
  CB_CASE(64, 2, false)
  CB_CASE(64, 4, false)
  CB_CASE(64, 8, false)
#undef CB_CASE
  return cudaErrorInvalidValue;
}

}  // namespace cb
