// Single-token attention over the 8-bit KV cache (format: cb_fp8.cuh) on the
// tensor cores, without converting the cache.
//
// Mathematics.  For a request's query head h with keys j (values k_j 2^ek_j,
// v_j 2^ev_j, k_j and v_j e4m3):
//     x_j = scale log2(e) 2^(eq + ek_j) (q . k_j)          p_j = 2^(x_j - m)
//     o   = sum_j 2^(x_j + ev_j - M) v_j                   l   = sum_j p_j
//     out = o 2^(M - m) / l
// with the running maxima m of x_j and M of x_j + ev_j.  The rows' powers of two
// never touch the matrices: 2^ek_j is a factor of row j's scores, 2^ev_j goes
// into row j's weight.  Two maxima, because the weights' dynamic range is what
// the 8-bit operand has to hold, whatever the value rows' sizes; p is kept in
// fp32 for l alone.
// Both matrix products take e4m3 K and V straight from the cache
// (tcgen05.mma kind::f8f6f4, fp32 accumulation).  Their other operands are split
// into 8-bit terms whose products add up:
//   q    two e4m3 terms (each 4 significant bits, so 8: exactly bf16's) of
//        q 2^-eq, the row's largest value in [128, 256): values down to 2^-9 of
//        the largest are exact, smaller ones are off by 2^-17 of it at most (half
//        of e4m3's least step, 2^-9, beside 128);
//   w    three e5m2 terms of the weight 2^12 w, w in (0, 2^3]: the weight is
//        rounded to 11 bits (half), the first two terms are its top 3 bits and
//        the next 3, the third rounds the rest to 3 bits: within 2^-9 + 2^-11 of w
//        (bf16 rounds within 2^-8) and 2^-29 of the largest.
// Using the 8-bit products instead of converting K and V to bf16 halves what
// passes through shared memory, the second limit after HBM (at the copy rate each
// SM takes 23 bytes of cache a cycle; converted tiles would add a read and twice
// that in writes and operand reads, over its 128 bytes a cycle).
//
// Tiles.  In the cache layout [block][KV head][16 tokens][A], HG heads of one
// block are 16 HG contiguous rows.  A tile is 128 rows: 8 / HG blocks of HG
// heads (HG = 8, 4, 2 or 1, the largest that divides the KV heads), so 8 slots
// of 16 rows, slot j = (block j / HG, head j % HG).
//     S[row, (term, slot, g)] = K_tile . q^T      one MMA per 32 dimensions, N = 16 G
//     O^T[dim, (slot, term, g)] += V^T . w^T      one MMA per 2 slots (32 rows)
// A row needs only its own slot's columns of S.  Each slot keeps its own maxima
// and its own columns of O, so softmax never crosses a half-warp; the slots of a
// head are joined at the end of a sequence.  Head dimension 64: V^T has 64 rows,
// its descriptor repeats them (leading offset 0) to M = 128.
//
// Work.  A sequence is a (request, group of HG heads).  All sequences' tiles, each
// sequence's behind kLead empty places, laid end to end, are cut into one equal
// range per CTA (one CTA per SM).  The empty places stand for what a sequence's end
// costs its CTA (4.5 us; without them and with: 2 sequences 26.0 and 23.3 us, 48 90.7
// and 87.1, 200 of 50-1000 keys 74 and 62.6; 100 of 50-600 keys on 32 KV heads 66 and
// 58.4, with one place 63.4.  With 0, 3, 6 and 9: groups of 2, 48 sequences 81.0, 81.0,
// 79.4 and 79.9, 100 short ones 31.1, 28.8, 28.0 and 28.8; groups of 8, 125, 120, 117.4
// and 118, and 52.2, 46.9, 47.7 and 48.1; 8 heads on 1 KV head 36.7, 34.3, 35.9 and
// 36.5, and 24.2, 23.9, 23.8 and 23.3).  A sequence cut at a range's end leaves
// (m, l, o) per piece, and a second small kernel (cb_fp8_join.cu) joins the pieces by
// log-sum-exp: no counters, no grid barrier, and the same bits every time.
//
// Warps: 0-3 and 4-7 softmax groups, which share a range's parts of sequences
// (segments) tile by tile: every second tile each, with its own maxima, sums and O
// in tensor memory, joined at the segment's end.  A tile's chain (scores, maxima,
// weights, one barrier of the group for a move of O) is mostly waiting, so two
// tiles at a time take little more than one: with a segment per group in turn, 48
// decodes took 104 us instead of 90 (both without the empty places).  8 K loads, 9 V
// loads (TMA through the block table; the exponents by per-thread copies: a TMA copy
// of 16 bytes takes the unit as long as one of 2 KB), 10 issues S, 11 issues O, 12-15
// make the next segments' query terms ready.  Thread = tile row, then output
// dimension.  Every wait is bounded.
//
// Bound by HBM where a KV head has one query head: 64 decodes of 32 heads (512 to
// 4096 keys, 1.30 GB) in 199 us, 6.5 TB/s, 0.96 of a copy's rate.  With four, a
// tile's softmax is four times the work: 48 decodes (256 to 8192 keys, 461 MB) in 86
// us, 5.4 TB/s, 0.79; a segment's end adds 4.5 us to its CTA.  Two sequences of 4900
// keys: 23 us, of which 12 in this kernel, 4 tiles per CTA.
#include <algorithm>

#include "cb_decode_item.cuh"
#include "cb_fp8.cuh"

namespace cb {

namespace {

constexpr int kThreads = 512;
constexpr float kWeightBits = 12.f; // weights are stored times 2^12 (e5m2: up to 2^15.8, down to 2^-16)
constexpr float kLazyP = 8.f;       // the running maxima follow only beyond these (base 2)
constexpr float kLazyW = 3.f;
constexpr int kMaxHeads = kSingleRows;   // query heads of a tile

template <int A, int G>
struct Cfg {
  static constexpr int C = 8 * G;                            // columns: slot x group member
  static constexpr int NS = 2 * C;                           // S columns (two query terms)
  static constexpr int SS = G <= 2 ? 8 : (G == 4 ? 16 : 24); // w rows per slot (three terms x G, padded)
  static constexpr int NO = 8 * SS;                          // O columns
  static constexpr int SB = G == 8 ? 1 : 4, NB = SB == 1 ? 2 : SB;   // S buffers, and their barriers (see issue_s)
  static constexpr int KS = A == 128 ? 4 : 6, VS = KS;       // K and V stages
  static constexpr int PB = 4;                               // w buffers
  static constexpr int ES = 8;                               // exponent stages
  static constexpr int kTile = 128 * A;                      // bytes
  static constexpr int kLead = G >= 2 ? 6 : 3;               // what a segment's end costs, in tiles (see Work above)
  static constexpr int kCols = SB * NS + 2 * NO;
  static constexpr int kTmem = kCols <= 128 ? 128 : (kCols <= 256 ? 256 : 512);
  static_assert(kCols <= 512, "tensor memory");
};

template <int A, int G>
struct alignas(1024) Smem {
  using X = Cfg<A, G>;
  uint8_t k[X::KS][X::kTile];
  uint8_t v[X::VS][X::kTile];
  uint8_t q[2][16 * G * A];          // of two segments: rows (term, slot, g) of A bytes, swizzled like K
  uint8_t p[X::PB][256 * X::SS];     // w: [2 slots][2 SS rows][32 bytes], 8-row x 16-byte core matrices
  uint8_t ex[X::ES][2][128];         // exponent bytes of the tile's K and V rows
  alignas(16) float cf[2][X::C];                 // of two segments: scale log2(e) 2^eq per column
  float alpha[2][2][X::C];           // per group: factors of O when M moves
  float sl[2][X::C], sm[2][X::C], sw[2][X::C];   // per group: a segment's l, m, M
  float of[2][X::C];                 // per group: the slots' factors of O
  float hl[2][X::C], hm[2][X::C], hi[2][X::C];   // l, m, 1 / l per head (each group its own copy)
  uint64_t k_full[X::KS], k_empty[X::KS], v_full[X::VS], v_empty[X::VS];
  uint64_t e_full[X::ES], e_empty[X::ES], s_full[X::NB], s_empty[X::NB], p_full[X::PB], pv_done[X::PB];
  uint64_t q_full[2], q_free[2], o_full, o_free, drain[2];
  int scan[16];
  uint32_t tmem;
  volatile int abort;
  int u0, u1, total, eff;            // this CTA's range of tiles; all tiles; CTAs with a range
};

// Plan arrays after Smem: pre[n + 1] places before request r (one head group), kv[n] keys, tok[n] query row.
struct Plan {
  const int *pre, *kv, *tok;
};

// N consecutive floats of shared memory.
template <int N>
__device__ __forceinline__ void lds_n(uint32_t a, float* v) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const uint4 x = lds128(a + 4 * i);
      v[i] = __uint_as_float(x.x), v[i + 1] = __uint_as_float(x.y), v[i + 2] = __uint_as_float(x.z), v[i + 3] = __uint_as_float(x.w);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = lds32f(a + 4 * i);
  }
}
// N (2, 4, 8, 16) consecutive fp32 columns of this thread's TMEM lane (no wait).
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, float* v) {
  uint32_t r[N];
  if constexpr (N == 2)
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x2.b32 {%0,%1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(taddr));
  if constexpr (N == 4)
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(taddr));
  if constexpr (N == 8)
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
  if constexpr (N == 16)
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = __uint_as_float(r[i]);
}

// ---------------------------------------------------------------- work
// A segment: tiles [t0, t0 + nt) of the `tiles` tiles of sequence (r, hg).
struct Seg {
  int r, hg, t0, nt, tiles, kv, tok, fb;   // fb: the first block its window reaches
};
struct SegIter {
  Plan plan;
  int u, u1, nhg, r, window, lead;
  __device__ SegIter(const Plan& pl, int u0, int u1_, int nhg_, int n, int window_, int lead_)
      : plan(pl), u(u0), u1(u1_), nhg(nhg_), window(window_), lead(lead_) {
    int lo = 0, hi = n - 1;            // the last request whose tiles start at or before u0
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (plan.pre[mid] * nhg <= u0)
        lo = mid;
      else
        hi = mid - 1;
    }
    r = lo;
  }
  // The sequence of place u: its first place and its size.
  __device__ void locate(int& start, int& size, int& hg) {
    while (plan.pre[r + 1] * nhg <= u) ++r;
    size = plan.pre[r + 1] - plan.pre[r];
    const int off = u - plan.pre[r] * nhg;
    hg = off / size;
    start = u - (off - hg * size);
  }
  __device__ bool next(Seg& s) {
    while (u < u1) {
      int start, size;
      locate(start, size, s.hg);
      const int first = start + lead, end = min(start + size, u1), from = max(u, first);
      u = end;
      if (end <= from) continue;       // nothing but the lead
      s.r = r;
      s.tiles = size - lead;
      s.t0 = from - first;
      s.nt = end - from;
      s.kv = plan.kv[r];
      s.tok = plan.tok[r];
      s.fb = window_first_block(s.kv, window);
      return true;
    }
    return false;
  }
};

// Tiles of one head group of request r if it has one new token; 0 otherwise.
__device__ __forceinline__ int request_tiles(const Fp8Step& P, int r, int bpt, int* kv, int* tok) {
  const int q0 = __ldg(P.cu_q_lens + r), q1 = __ldg(P.cu_q_lens + r + 1), ctx = __ldg(P.ctx_lens + r);
  *kv = 0;
  *tok = 0;
  const long long n = (long long)q1 - q0;
  if (q0 >= 0 && q1 <= P.n_tokens && (n == 0 || (n > 1 && P.max_q_len > 1))) return 0;
  const long long keys = (long long)ctx + 1, nblk = (keys + kBlockSize - 1) / kBlockSize;
  if (n != 1 || ctx < 0 || q0 < 0 || q1 > P.n_tokens || keys > P.max_kv_len || nblk > P.max_blocks_per_seq) {
    set_error(P.err, CB_DEVERR_BADLEN);
    return 0;
  }
  *kv = (int)keys;
  *tok = q0;
  return ((int)nblk - window_first_block(keys, P.window) + bpt - 1) / bpt;
}

// All threads; ends with __syncthreads().
template <int A, int G>
__device__ void make_plan(const Fp8Step& P, const Fp8Partials& W, Smem<A, G>& S, int* pre, int* kv, int* tok, int hg_heads) {
  const int n = P.n_reqs, tid = threadIdx.x, lane = tid & 31, wid = tid >> 5, nw = kThreads / 32;
  const int bpt = 8 / hg_heads, nhg = P.cache.n_kv_heads / hg_heads;
  const int seg = (n + kThreads - 1) / kThreads, lo = min(n, tid * seg), hi = min(n, lo + seg);
  int own = 0;
  for (int r = lo; r < hi; ++r) {
    int t = request_tiles(P, r, bpt, kv + r, tok + r);
    if (t > 0) t += Cfg<A, G>::kLead;
    pre[r] = t;
    own += t;
  }
  int incl = own;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += x;
  }
  if (lane == 31) S.scan[wid] = incl;
  __syncthreads();
  int total = 0, run = incl - own;
  for (int w = 0; w < nw; ++w) {
    total += S.scan[w];
    run += w < wid ? S.scan[w] : 0;
  }
  for (int r = lo; r < hi; ++r) {
    const int t = pre[r];
    pre[r] = run;
    run += t;
  }
  if (tid == 0) {
    pre[n] = total;
    total *= nhg;
    const int eff = max(1, min((int)gridDim.x, total));   // a tile per CTA at least: 4 x 250 keys 18 us, with two tiles 21
    const int b = blockIdx.x;
    S.total = total;
    S.eff = eff;
    S.u0 = b < eff ? (int)((long long)total * b / eff) : total;
    S.u1 = b < eff ? (int)((long long)total * (b + 1) / eff) : total;
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");   // so far only the requests' lengths were read (launch_after)
  if (tid == 0 && blockIdx.x == 0) signal_ready(P);
  __syncthreads();
  if (tid == 0) {                     // the sequence that starts in this range and goes on after it
    Fp8Rec rec = {0, 0, 0, 0};
    if (S.u1 > S.u0) {
      SegIter last({pre, kv, tok}, S.u1 - 1, S.u1, nhg, n, P.window, Cfg<A, G>::kLead);
      int start, size, hg;
      last.locate(start, size, hg);
      const int first = start + Cfg<A, G>::kLead, end = start + size;
      if (first >= S.u0 && first < S.u1 && end > S.u1) rec = {last.r, hg, cta_of(end - 1, S.total, S.eff) - (int)blockIdx.x + 1, 0};
    }
    W.rec[blockIdx.x] = rec;
  }
}

// ---------------------------------------------------------------- loads (warps 8, 9)
// A segment's block-table entries, 32 at a time (a lane each), the next 32 (or
// the next segment's first) on their way while these are used.
__device__ __forceinline__ int table_entry(const Fp8Step& P, const Seg& s, int bpt, int chunk) {
  const int b = s.fb + s.t0 * bpt + chunk * 32 + (int)(threadIdx.x & 31);
  const int end = (s.kv + kBlockSize - 1) / kBlockSize;
  // entries past the segment belong to another CTA or to nobody: not read
  if (b >= end || b >= s.fb + (s.t0 + s.nt) * bpt) return -2;
  const int e = __ldg(P.block_tables + (size_t)s.r * P.max_blocks_per_seq + b);
  return e < 0 || e >= P.cache.num_blocks ? -1 : e;
}

// K: also the tiles' exponents.  V: values only.
template <int A, int G, bool IS_K>
__device__ void load_tiles(const Fp8Step& P, const CUtensorMap* map, Smem<A, G>& S, const Plan& plan, int hg_heads) {
  using X = Cfg<A, G>;
  constexpr int NST = IS_K ? X::KS : X::VS;
  const unsigned FULL = 0xffffffffu;
  const int lane = threadIdx.x & 31, Hkv = P.cache.n_kv_heads, bpt = 8 / hg_heads, nhg = Hkv / hg_heads;
  const int rows_total = P.cache.num_blocks * Hkv * kBlockSize, box = hg_heads * kBlockSize;
  uint64_t* full = IS_K ? S.k_full : S.v_full;
  uint64_t* empty = IS_K ? S.k_empty : S.v_empty;
  fence_proxy_async_global();           // the rows were appended by ordinary stores
  SegIter it(plan, S.u0, S.u1, nhg, P.n_reqs, P.window, X::kLead);
  Seg s, nx;
  uint32_t n = 0;
  bool ok = true;
  bool more = it.next(s);
  int nxt = more ? table_entry(P, s, bpt, 0) : -2;
  while (more && ok) {
    const bool again = it.next(nx);
    const int per = 32 / bpt;                        // tiles per 32 entries
    int cur = -2;
    for (int j = 0; j < s.nt && ok; ++j, ++n) {
      if (j % per == 0) {
        cur = nxt;
        if (IS_K && cur == -1) set_error(P.err, CB_DEVERR_BADBLOCK);   // its rows load as zeros
        nxt = j + per < s.nt ? table_entry(P, s, bpt, j / per + 1) : (again ? table_entry(P, nx, bpt, 0) : -2);
      }
      const int e = __shfl_sync(FULL, cur, (j % per) * bpt + (lane & (bpt - 1)));
      const int row = e >= 0 ? (e * Hkv + s.hg * hg_heads) * kBlockSize : rows_total;   // past the extent: zeros
      const int st = n % NST;
      ok = wwait(P, S, &empty[st], ((n / NST) & 1) ^ 1);
      if (!ok) break;
      if (lane == 0) mbar_arrive_expect_tx(&full[st], X::kTile);
      __syncwarp();
      if (lane < bpt) tma_load_2d((IS_K ? S.k[st] : S.v[st]) + lane * box * A, map, 0, row, &full[st]);
      if constexpr (IS_K) {
        const int es = n % X::ES;
        ok = wwait(P, S, &S.e_empty[es], ((n / X::ES) & 1) ^ 1);
        if (!ok) {
          ++n;
          break;
        }
        // exponents, 16 pieces of 16 bytes: lanes 0 .. 7 K's, 8 .. 15 V's, in the tile's order of rows (zeros
        // where there is no block: what the stage held before must not reach the scores)
        const int piece = lane & 7, pe = __shfl_sync(FULL, e, piece / hg_heads);
        if (lane < 16)
          cp_async16(&S.ex[es][lane >> 3][piece * kBlockSize],
                     (lane < 8 ? P.cache.k_exps : P.cache.v_exps) +
                         ((size_t)max(pe, 0) * Hkv + s.hg * hg_heads + piece % hg_heads) * kBlockSize, pe >= 0);
        cp_async_arrive(&S.e_full[es]);
      }
    }
    s = nx;
    more = again;
  }
  if constexpr (IS_K) cp_async_wait_all();
  if (!ok) {
    // let the copies already issued land before the CTA exits
    for (uint32_t i = n > (uint32_t)NST ? n - NST : 0; i < n; ++i) mbar_wait(&full[i % NST], (i / NST) & 1, 20000000ull);
  }
}

// ---------------------------------------------------------------- MMA issue (warps 10, 11)
template <int A, int G>
__device__ void issue_s(const Fp8Step& P, Smem<A, G>& S, const Plan& plan, int nhg) {
  using X = Cfg<A, G>;
  constexpr uint32_t kIdesc = idesc_f8(128, X::NS, 0, 0, 0, 0);
  constexpr int kLayout = A == 128 ? 2 : 4;
  const uint64_t kd = smem_desc(smem_u32(S.k[0]), 16, 8 * A, kLayout), qd = smem_desc(smem_u32(S.q[0]), 16, 8 * A, kLayout);
  SegIter it(plan, S.u0, S.u1, nhg, P.n_reqs, P.window, X::kLead);
  Seg s;
  uint32_t n = 0;
  bool ok = true;
  for (int i = 0; ok && it.next(s); ++i) {
    ok = wwait(P, S, &S.q_full[i & 1], (i >> 1) & 1);
    for (int j = 0; j < s.nt && ok; ++j, ++n) {
      // a single buffer has two barriers all the same: a group looks at every second tile, and a parity cannot
      // tell phases two apart
      const int st = n % X::KS, sb = n % X::SB;
      const uint32_t was = n - X::SB;                          // the tile before in this buffer
      ok = (n < (uint32_t)X::SB || wwait(P, S, &S.s_empty[was % X::NB], (was / X::NB) & 1)) &&
           wwait(P, S, &S.k_full[st], (n / X::KS) & 1);
      if (!ok) break;
      tc_fence_after();
      const uint64_t a = kd + (uint32_t)(st * (X::kTile >> 4)), b = qd + (uint32_t)((i & 1) * ((16 * G * A) >> 4));
      if (elect_one()) {
#pragma unroll
        for (int d = 0; d < A / 32; ++d) mma_f8(S.tmem + sb * X::NS, a + d * 2, b + d * 2, kIdesc, d > 0);
        tc_commit(&S.k_empty[st]);
        tc_commit(&S.s_full[n % X::NB]);
        if (j == s.nt - 1) tc_commit(&S.q_free[i & 1]);
      }
      __syncwarp();
    }
  }
  if (!ok) S.abort = 1;
  if (elect_one()) tc_commit(&S.drain[0]);
  __syncwarp();
  mbar_wait(&S.drain[0], 0, 20000000ull);
}

template <int A, int G>
__device__ void issue_pv(const Fp8Step& P, Smem<A, G>& S, const Plan& plan, int nhg) {
  using X = Cfg<A, G>;
  constexpr uint32_t kIdesc = idesc_f8(128, 2 * X::SS, 0, 1, 1, 0);   // V^T: e4m3, MN-major; w: e5m2, K-major
  constexpr int kLayout = A == 128 ? 2 : 4;
  const uint64_t vd = smem_desc(smem_u32(S.v[0]), 0, 8 * A, kLayout), pd = smem_desc(smem_u32(S.p[0]), 128, 256, 0);
  SegIter it(plan, S.u0, S.u1, nhg, P.n_reqs, P.window, X::kLead);
  Seg s;
  uint32_t n = 0;
  bool ok = true;
  for (int i = 0; ok && it.next(s); ++i) {
    ok = wwait(P, S, &S.o_free, (i & 1) ^ 1);
    for (int j = 0; j < s.nt && ok; ++j, ++n) {
      const int st = n % X::VS, pb = n % X::PB;
      ok = wwait(P, S, &S.v_full[st], (n / X::VS) & 1) && wwait(P, S, &S.p_full[pb], (n / X::PB) & 1);
      if (!ok) break;
      tc_fence_after();
      const uint64_t a = vd + (uint32_t)(st * (X::kTile >> 4)), b = pd + (uint32_t)(pb * ((256 * X::SS) >> 4));
      const uint32_t d = S.tmem + X::SB * X::NS + (n & 1) * X::NO;
      if (elect_one()) {
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          mma_f8(d + ks * 2 * X::SS, a + ((ks * 32 * A) >> 4), b + ((ks * 64 * X::SS) >> 4), kIdesc, j > 1);
        tc_commit(&S.v_empty[st]);
        tc_commit(&S.pv_done[pb]);
        if (j == s.nt - 1) tc_commit(&S.o_full);
      }
      __syncwarp();
    }
  }
  if (!ok) S.abort = 1;
  if (elect_one()) tc_commit(&S.drain[1]);
  __syncwarp();
  mbar_wait(&S.drain[1], 0, 20000000ull);
}

// ---------------------------------------------------------------- queries (warps 12-15)
// Query terms of the segment's heads into q[buf], and the columns' factors.
template <int A, int G>
__device__ void load_query(const Fp8Step& P, Smem<A, G>& S, const Seg& s, int buf, int hg_heads) {
  constexpr int D = A / 32;                  // values per lane
  constexpr int B = 8;                       // heads in flight
  const int warp = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31;
  const int heads = hg_heads * G, bpt = 8 / hg_heads;
  const uint32_t q_at = smem_u32(S.q[buf]);
  const uint16_t* src = P.q + ((size_t)s.tok * P.n_q_heads + (size_t)s.hg * heads) * A + lane * D;
  for (int h0 = warp; h0 < heads; h0 += 4 * B) {
    uint32_t w[B][D / 2];
#pragma unroll
    for (int u = 0; u < B; ++u) {
      const int h = h0 + 4 * u;
#pragma unroll
      for (int d = 0; d < D / 2; ++d)
        w[u][d] = h < heads ? *reinterpret_cast<const uint32_t*>(src + (size_t)h * A + 2 * d) : 0u;
    }
#pragma unroll
    for (int u = 0; u < B; ++u) {
      const int h = h0 + 4 * u;
      if (h >= heads) break;                 // the same in every lane
      uint32_t m = w[u][0] & 0x7FFF7FFFu;
#pragma unroll
      for (int d = 1; d < D / 2; ++d) m = __vmaxu2(m, w[u][d] & 0x7FFF7FFFu);
      m = max(m & 0xFFFFu, m >> 16);
      m = __reduce_max_sync(0xffffffffu, m);
      // not finite: zeros and a NaN factor
      const bool bad = m >= 0x7F80u;
      const uint32_t eb = query_exp(m);
      const float f = bad ? 0.f : exp_inverse(eb);
      uint32_t c0 = 0, c1 = 0;
#pragma unroll
      for (int d = 0; d < D / 2; ++d) {
        const float y0 = bad ? 0.f : bf16lo(w[u][d]) * f, y1 = bad ? 0.f : bf16hi(w[u][d]) * f;
        uint32_t hi, lo;
        query_terms(y0, y1, hi, lo);
        c0 |= hi << (16 * d);
        c1 |= lo << (16 * d);
      }
      const int hh = h / G, g = h - hh * G;
      for (int bi = 0; bi < bpt; ++bi) {
        const int col = (bi * hg_heads + hh) * G + g;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int row = t * Cfg<A, G>::C + col;
          if constexpr (A == 128) {
            sts32(q_at + row * 128 + (((lane >> 2) ^ (row & 7)) << 4) + (lane & 3) * 4, t ? c1 : c0);
          } else {
            sts16(q_at + row * 64 + (((lane >> 3) ^ ((row >> 1) & 3)) << 4) + (lane & 7) * 2, t ? c1 : c0);
          }
        }
        if (lane == 0) S.cf[buf][col] = bad ? __uint_as_float(0x7FC00000u) : P.scale_log2 * __uint_as_float(eb << 23);
      }
    }
  }
}

// The queries of the segments, two ahead of the softmax at most.
template <int A, int G>
__device__ void queries(const Fp8Step& P, Smem<A, G>& S, const Plan& plan, int hg_heads) {
  SegIter it(plan, S.u0, S.u1, P.cache.n_kv_heads / hg_heads, P.n_reqs, P.window, Cfg<A, G>::kLead);
  Seg s;
  for (int i = 0; it.next(s); ++i) {
    if (!wwait(P, S, &S.q_free[i & 1], ((i >> 1) & 1) ^ 1)) break;
    load_query<A, G>(P, S, s, i & 1, hg_heads);
    fence_proxy_async_smem();
    mbar_arrive(&S.q_full[i & 1]);
  }
}

// ---------------------------------------------------------------- softmax groups (warps 0-3, 4-7)
// Output dimension d of this group's heads of the segment (every second): the
// slots of a head joined over both groups' O, o 2^(M - m) / l, written as the output
// or as this piece's part of it with m and l.  2^(M - m) comes as two factors: for
// the smallest and the largest exponents of value rows it is outside fp32's normal
// range.  obs: bit b: O buffer b holds products.
template <int A, int G>
__device__ void write_out(const Fp8Step& P, const Fp8Partials& W, Smem<A, G>& S, const Seg& s, int grp, uint32_t obs,
                          int hg_heads, bool whole, int slot_out) {
  using X = Cfg<A, G>;
  const int t = threadIdx.x & 127, warp = t >> 5, bpt = 8 / hg_heads, heads = hg_heads * G;
  if (A == 64 && warp >= 2) return;          // rows 64 .. 127 repeat 0 .. 63
  const uint32_t base = S.tmem + X::SB * X::NS + ((uint32_t)(warp * 32) << 16);
  for (int hh = grp; hh < hg_heads; hh += 2) {
    float acc[G], inv[G];
#pragma unroll
    for (int g = 0; g < G; ++g) acc[g] = 0.f;
    lds_n<G>(smem_u32(&S.hi[grp][hh * G]), inv);
    for (int bi = 0; bi < bpt; ++bi) {
      const int slot = bi * hg_heads + hh;
      float o[2][X::SS], f[2][G];
#pragma unroll
      for (int ob = 0; ob < 2; ++ob) {
        const uint32_t at = base + ob * X::NO + slot * X::SS;
        if constexpr (X::SS == 24) {
          tmem_ld<16>(at, o[ob]);
          tmem_ld<8>(at + 16, o[ob] + 16);
        } else {
          tmem_ld<X::SS>(at, o[ob]);
        }
        lds_n<G>(smem_u32(&S.of[ob][slot * G]), f[ob]);
      }
      tmem_wait_ld();
#pragma unroll
      for (int ob = 0; ob < 2; ++ob) {
        if (!((obs >> ob) & 1)) continue;      // whatever the buffer holds
#pragma unroll
        for (int g = 0; g < G; ++g) acc[g] += ((o[ob][g] + o[ob][G + g] + o[ob][2 * G + g]) * f[ob][g]) * (f[ob][g] * inv[g]);
      }
    }
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const int h = hh * G + g;
      if (whole) {
        P.out[((size_t)s.tok * P.n_q_heads + (size_t)s.hg * heads + h) * A + t] =
            __bfloat16_as_ushort(__float2bfloat16_rn(acc[g]));
      } else {
        const size_t at = (size_t)slot_out * kMaxHeads + h;
        W.acc[at * A + t] = acc[g];
        if (t == 0) *reinterpret_cast<float2*>(W.ml + at * 2) = make_float2(S.hm[grp][h], S.hl[grp][h]);
      }
    }
  }
}

template <int A, int G>
__device__ void softmax_group(const Fp8Step& P, const Fp8Partials& W, Smem<A, G>& S, const Plan& plan, int grp, int hg_heads) {
  using X = Cfg<A, G>;
  const unsigned FULL = 0xffffffffu;
  const int tid = threadIdx.x & 127, warp = tid >> 5, lane = tid & 31, bar_id = 1 + grp;
  const int slot = tid >> 4, tok = tid & 15, bpt = 8 / hg_heads, nhg = P.cache.n_kv_heads / hg_heads;
  const int bi = slot / hg_heads;
  const bool upper = lane & 16;
  const uint32_t lane_base = (uint32_t)(warp * 32) << 16;
  SegIter it(plan, S.u0, S.u1, nhg, P.n_reqs, P.window, X::kLead);
  Seg s;
  uint32_t n0 = 0;                           // tiles before this segment
  const uint32_t o_tmem = S.tmem + X::SB * X::NS + grp * X::NO;
  for (int i = 0; it.next(s); ++i, n0 += s.nt) {
    bool fail = !wwait(P, S, &S.q_full[i & 1], (i >> 1) & 1);
    float f[G], m[G], M[G], l[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
      f[g] = S.cf[i & 1][slot * G + g];
      m[g] = M[g] = kNegInf;
      l[g] = 0.f;
    }
    uint32_t read = 0;
#pragma unroll
    for (int g = 0; g < G; ++g) read ^= __float_as_uint(f[g]);
    arrive_after(&S.q_free[i & 1], read);
    const int first_key = P.window > 0 ? max(0, s.kv - P.window) : 0;
    const int j0 = (n0 ^ grp) & 1;           // this group's first tile of the segment
    for (int j = j0; j < s.nt; j += 2) {
      const uint32_t n = n0 + j;
      const int sb = n % X::SB, es = n % X::ES, pb = n % X::PB;
      const int pos = (s.fb + (s.t0 + j) * bpt + bi) * kBlockSize + tok;
      const bool valid = pos < s.kv && pos >= first_key;
      fail |= !wwait(P, S, &S.e_full[es], (n / X::ES) & 1);
      const uint32_t kb = lds8(smem_u32(&S.ex[es][0][tid])), vb = lds8(smem_u32(&S.ex[es][1][tid]));
      fail |= !wwait(P, S, &S.s_full[n % X::NB], (n / X::NB) & 1);
      tc_fence_after();
      float s0[2 * G], s1[2 * G];
      const uint32_t at = S.tmem + lane_base + sb * X::NS + 2 * warp * G;
      tmem_ld<2 * G>(at, s0);
      tmem_ld<2 * G>(at + X::C, s1);
      tmem_wait_ld();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&S.s_empty[n % X::NB]);
      }
      const float fk = exp_scale(kb), ev = vb == kExpNan ? __uint_as_float(0x7FC00000u) : (float)((int)vb - 127);
      float x[G];
      bool grow = false;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        x[g] = valid ? (upper ? s0[G + g] + s1[G + g] : s0[g] + s1[g]) * finite(f[g] * fk) : kNegInf;
        grow |= x[g] > m[g] + kLazyP || x[g] + ev > M[g] + kLazyW;
      }
      bool need = false;
      if (__any_sync(FULL, grow)) {
        // the slot's exact maxima; the references move where they would be exceeded
#pragma unroll
        for (int g = 0; g < G; ++g) {
          float mx = x[g], tx = x[g] + ev;
#pragma unroll
          for (int off = 8; off > 0; off >>= 1) {
            mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, off));
            tx = fmaxf(tx, __shfl_xor_sync(FULL, tx, off));
          }
          if (mx > m[g] + kLazyP) {
            l[g] *= ex2(m[g] - mx);
            m[g] = mx;
          }
          float a = 1.f;
          if (tx > M[g] + kLazyW) {
            a = ex2(M[g] - tx);
            M[g] = tx;
            need = true;
          }
          if (tok == 0) sts32(smem_u32(&S.alpha[grp][(n >> 1) & 1][slot * G + g]), __float_as_uint(a));
        }
      } else if (tok < G) {
        sts32(smem_u32(&S.alpha[grp][(n >> 1) & 1][slot * G + tok]), __float_as_uint(1.f));
      }
      if (named_bar_or(bar_id, 128, (need && j > 1) || fail || S.abort)) {
        if (named_bar_or(bar_id, 128, fail || S.abort)) {
          fail = true;
          break;
        }
        // O times the factors, once the products of this group's tile before have landed
        fail |= !wwait(P, S, &S.pv_done[(n - 2) % X::PB], ((n - 2) / X::PB) & 1);
        tc_fence_after();
        if (!fail) {
#pragma unroll 1
          for (int sl = 0; sl < 8; ++sl) {
            const uint32_t oc = o_tmem + lane_base + sl * X::SS;
#pragma unroll
            for (int c = 0; c < X::SS / 8; ++c) {
              float o[8];
              tmem_ld8(oc + 8 * c, o);
              tmem_wait_ld();
#pragma unroll
              for (int u = 0; u < 8; ++u) o[u] *= S.alpha[grp][(n >> 1) & 1][sl * G + (8 * c + u) % G];
              tmem_st8(oc + 8 * c, o);
            }
          }
          tmem_wait_st();
        }
      }
      // weights: three e5m2 terms; p for the sum
      uint32_t b0[(G + 1) / 2], b1[(G + 1) / 2], b2[(G + 1) / 2];
#pragma unroll
      for (int g = 0; g < G; g += 2) {
        float w[2] = {0.f, 0.f};
#pragma unroll
        for (int u = 0; u < 2 && g + u < G; ++u) {
          if (valid) {
            l[g + u] += ex2(x[g + u] - m[g + u]);
            w[u] = ex2(x[g + u] + ev - M[g + u] + kWeightBits);
          }
        }
        uint32_t h, r1, r2;
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(w[1]), "f"(w[0]));
        b0[g / 2] = h & 0xFF00FF00u;                // e5m2 is the top byte of a half: its first 3 bits
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r1) : "r"(h), "r"(b0[g / 2]));
        b1[g / 2] = r1 & 0xFF00FF00u;
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r2) : "r"(r1), "r"(b1[g / 2]));
        uint16_t c;
        asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(c) : "r"(r2));
        b2[g / 2] = c;
      }
      // the buffer is free once the products of tile n - PB have landed
      fail |= !wwait(P, S, &S.pv_done[pb], ((n / X::PB) & 1) ^ 1);
      const uint32_t pp = smem_u32(S.p[pb]) + (slot >> 1) * (64 * X::SS) + (slot & 1) * 128 + tok;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const int sh = (g & 1) ? 24 : 8, sh2 = (g & 1) ? 8 : 0;
#pragma unroll
        for (int t = 0; t < 3; ++t) {
          const int row = (slot & 1) * X::SS + t * G + g;
          sts8(pp + (row >> 3) * 256 + (row & 7) * 16, t == 0 ? b0[g / 2] >> sh : t == 1 ? b1[g / 2] >> sh : b2[g / 2] >> sh2);
        }
      }
      // rows that the request does not have hold whatever the cache had: 0 * NaN must not reach O
      if (!valid) {
        const int st = n % X::VS;
        if (mbar_wait(&S.v_full[st], (n / X::VS) & 1)) {
#pragma unroll
          for (int c = 0; c < A / 16; ++c) sts128(smem_u32(&S.v[st][tid * A + c * 16]), make_uint4(0, 0, 0, 0));
        } else {
          set_error(P.err, CB_DEVERR_TIMEOUT);
          S.abort = 1;
        }
      }
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&S.p_full[pb]);
        mbar_arrive(&S.e_empty[es]);         // its exponents are in the weights
      }
    }
    // the segment's sums; then the heads' and the slots' factors, over both groups.  A group that gave up comes
    // here too: the other one waits for it.
#pragma unroll
    for (int g = 0; g < G; ++g) {
#pragma unroll
      for (int off = 8; off > 0; off >>= 1) l[g] += __shfl_xor_sync(FULL, l[g], off);
      if (tok == 0) {
        S.sl[grp][slot * G + g] = l[g];
        S.sm[grp][slot * G + g] = m[g];
        S.sw[grp][slot * G + g] = M[g];
      }
    }
    if (!fail) fail = !wwait(P, S, &S.o_full, i & 1);
    if (named_bar_or(3, 256, fail || S.abort)) break;
    tc_fence_after();
    if (tid < X::C) {
      const int head = (tid / G) % hg_heads, g = tid % G;
      float hm = kNegInf, hl = 0.f;
      for (int b = 0; b < 2 * bpt; ++b) hm = fmaxf(hm, S.sm[b & 1][((b >> 1) * hg_heads + head) * G + g]);
      for (int b = 0; b < 2 * bpt; ++b) {
        const float sl = S.sl[b & 1][((b >> 1) * hg_heads + head) * G + g], sm = S.sm[b & 1][((b >> 1) * hg_heads + head) * G + g];
        // a slot without keys adds nothing; one whose sum is NaN passes it on
        if (sm != kNegInf)
          hl += sl * ex2(sm - hm);
        else if (sl != 0.f)
          hl += sl;
      }
      S.of[grp][tid] = S.sw[grp][tid] == kNegInf ? (S.sl[grp][tid] != 0.f ? 1.f : 0.f) : ex2(0.5f * (S.sw[grp][tid] - kWeightBits - hm));
      if (tid < hg_heads * G) {
        S.hl[grp][tid] = hl;
        S.hi[grp][tid] = 1.f / hl;
        S.hm[grp][tid] = hm;
      }
    }
    named_bar(3, 256);
    // a range's first segment that began before it is piece 2b, any other one that is cut piece 2b + 1
    write_out<A, G>(P, W, S, s, grp, s.nt > 1 ? 3u : 1u << (n0 & 1), hg_heads, s.nt == s.tiles, 2 * (int)blockIdx.x + (s.t0 > 0 ? 0 : 1));
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&S.o_free);
  }
}

template <int A, int G>
__global__ void __launch_bounds__(kThreads, 1)
    decode_fp8_kernel(const Fp8Step P, const Fp8Partials W, const int hg_heads, const __grid_constant__ CUtensorMap kmap,
                      const __grid_constant__ CUtensorMap vmap) {
  using X = Cfg<A, G>;
  extern __shared__ uint8_t smem_raw[];
  Smem<A, G>& S = *reinterpret_cast<Smem<A, G>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  int* pre = reinterpret_cast<int*>(&S + 1);
  int *kv = pre + P.n_reqs + 1, *tok = kv + P.n_reqs;
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int i = 0; i < X::KS; ++i) {
      mbar_init(&S.k_full[i], 1);
      mbar_init(&S.k_empty[i], 1);
      mbar_init(&S.v_full[i], 1);
      mbar_init(&S.v_empty[i], 1);
    }
    for (int i = 0; i < X::ES; ++i) {
      mbar_init(&S.e_full[i], 32);
      mbar_init(&S.e_empty[i], 4);
    }
    for (int i = 0; i < X::NB; ++i) {
      mbar_init(&S.s_full[i], 1);
      mbar_init(&S.s_empty[i], 4);
    }
    for (int i = 0; i < X::PB; ++i) {
      mbar_init(&S.p_full[i], 4);
      mbar_init(&S.pv_done[i], 1);
    }
    mbar_init(&S.o_full, 1);
    mbar_init(&S.o_free, 8);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&S.q_full[i], 128);
      mbar_init(&S.q_free[i], 1 + 8);   // its products are done; the softmax warps have its factors
      mbar_init(&S.drain[i], 1);
    }
    S.abort = 0;
    fence_mbar_init();
    prefetch_tmap(&kmap);
    prefetch_tmap(&vmap);
  }
  if (warp == 10) {
    tmem_alloc(&S.tmem, X::kTmem);
    tmem_relinquish();
    tc_fence_before();
  }
  for (int i = threadIdx.x; i < (int)sizeof(S.p) / 16; i += kThreads)
    reinterpret_cast<uint4*>(S.p)[i] = make_uint4(0, 0, 0, 0);       // the other slot's rows and the padding stay zero
  fence_proxy_async_smem();
  make_plan<A, G>(P, W, S, pre, kv, tok, hg_heads);
  __syncthreads();
  tc_fence_after();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const Plan plan{pre, kv, tok};
  const int nhg = P.cache.n_kv_heads / hg_heads;
  if (warp < 8)
    softmax_group<A, G>(P, W, S, plan, warp >> 2, hg_heads);
  else if (warp == 8)
    load_tiles<A, G, true>(P, &kmap, S, plan, hg_heads);
  else if (warp == 9)
    load_tiles<A, G, false>(P, &vmap, S, plan, hg_heads);
  else if (warp == 10)
    issue_s<A, G>(P, S, plan, nhg);
  else if (warp >= 12)
    queries<A, G>(P, S, plan, hg_heads);
  else
    issue_pv<A, G>(P, S, plan, nhg);
  tc_fence_before();
  __syncthreads();
  if (warp == 10) {
    tc_fence_after();
    tmem_dealloc(S.tmem, X::kTmem);
  }
}

template <int A, int G>
size_t smem_bytes(int n_reqs) {
  return 1024 + sizeof(Smem<A, G>) + (size_t)(3 * n_reqs + 1) * 4;
}
constexpr int kSmemLimit = 232448;
static_assert(sizeof(Smem<128, 8>) + 1024 + (3 * kMaxReqs + 1) * 4 <= kSmemLimit, "shared memory");
static_assert(sizeof(Smem<128, 4>) + 1024 + (3 * kMaxReqs + 1) * 4 <= kSmemLimit, "shared memory");

template <int A, int G>
cudaError_t launch_t(const Fp8Step& s, const Fp8Partials& w, int grid, bool chained, cudaStream_t stream) {
  const int hg = fp8_head_group(s.cache.n_kv_heads);
  CUtensorMap km, vm;
  const long long rows = (long long)s.cache.num_blocks * s.cache.n_kv_heads * kBlockSize;
  if (!encode_byte_rows(&km, s.cache.k, rows, A, hg * kBlockSize) || !encode_byte_rows(&vm, s.cache.v, rows, A, hg * kBlockSize))
    return cudaErrorInvalidValue;
  cudaError_t e = opt_in_smem(reinterpret_cast<const void*>(decode_fp8_kernel<A, G>), kSmemLimit);
  if (e != cudaSuccess) return e;
  return launch_after(chained, decode_fp8_kernel<A, G>, grid, kThreads, smem_bytes<A, G>(s.n_reqs), stream, s, w, hg, km, vm);
}

}  // namespace

bool fp8_decode_shape(int head_dim, int group) { return (head_dim == 64 || head_dim == 128) && group <= 8; }

int fp8_head_group(int n_kv_heads) {
  int hg = 8;
  while (n_kv_heads % hg) hg >>= 1;
  return hg;
}

cudaError_t launch_decode_fp8(const Fp8Step& s, const Fp8Partials& w, int grid, bool chained, cudaStream_t stream) {
  const int a = s.cache.head_dim, g = s.n_q_heads / s.cache.n_kv_heads;
#define CB_CASE(A_, G_) \
  if (a == A_ && g == G_) return launch_t<A_, G_>(s, w, grid, chained, stream);
  CB_CASE(128, 1)
  CB_CASE(128, 2)
  CB_CASE(128, 4)
  CB_CASE(128, 8)
  CB_CASE(64, 1)
  CB_CASE(64, 2)
  CB_CASE(64, 4)
  CB_CASE(64, 8)
#undef CB_CASE
  return cudaErrorInvalidValue;
}

}  // namespace cb
