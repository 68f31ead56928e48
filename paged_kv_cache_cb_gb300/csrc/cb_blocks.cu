// The block pool on the device: forking, growing and compacting the rows of
// block tables, and whole-block copies in every layer's caches.
//
// State (the caller's): tables [n_rows][width], lens [n_rows] (tokens stored),
// refs [num_blocks] (holders of each block; 0: free).  Row r holds the first
// ceil(lens[r] / 16) entries of its table row.
//
// Fork, grow and compact are one kernel each, of one CTA (sync_all is then a block's
// barrier) or of one cluster of 8 or 16.  They touch a few ints per row and block, so
// what they cost is the chain of dependent reads -- lengths, entries, counts, ranks --
// of 0.3 to 0.7 us each.  A cluster's hardware barrier orders the phases without a
// grid-wide wait; what is a few ints per row every CTA reads and works out for all
// rows, instead of waiting for another's.  Two kernels are ordinary grids without
// barriers between their CTAs: slots_kernel, which a growth by many tokens puts
// behind its own, and the copies.  Blocks are always taken from the lowest free id on,
// in row order: ranks come from prefix sums, never from the order in which atomics
// arrive, so a call's result is the same every time.  The atomics on refs are integer
// sums.
#include <algorithm>

#include "../../include/cbattn.h"
#include "cb_common.cuh"

namespace cb {

namespace {

constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kCluster = 16;           // most CTAs of a call

struct Pool {
  int32_t* tables;
  int32_t* lens;
  int32_t* refs;
  int n_rows, width, num_blocks;
  unsigned int* err;
};

// ---------------------------------------------------------------- the cluster
// Orders every global and shared access of the cluster's threads before it
// against those after it.
__device__ __forceinline__ void sync_all() {
  if (gridDim.x == 1) {
    __syncthreads();
    return;
  }
  __threadfence();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ int blocks_of(int tokens) { return (tokens + kBlockSize - 1) / kBlockSize; }

// Exclusive prefix of v over the CTA's threads; *total: their sum.  red: kWarps
// + 1 ints.  Two barriers.
__device__ __forceinline__ int cta_scan(int v, int* red, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  __syncthreads();                     // red may still be read
  if (lane == 31) red[warp] = x;
  __syncthreads();
  const int w = red[lane];             // kWarps == 32
  int before = lane < warp ? w : 0, all = w;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    before += __shfl_xor_sync(0xffffffffu, before, d);
    all += __shfl_xor_sync(0xffffffffu, all, d);
  }
  *total = all;
  return before + x - v;
}

// This CTA's share of the pool's blocks.
struct Slice {
  int lo, hi;
};
__device__ __forceinline__ int slice_size(int num_blocks) { return (num_blocks + (int)gridDim.x - 1) / (int)gridDim.x; }
__device__ __forceinline__ Slice my_slice(int num_blocks) {
  const int s = slice_size(num_blocks);
  const long long lo = (long long)s * blockIdx.x;
  return {(int)min((long long)num_blocks, lo), (int)min((long long)num_blocks, lo + s)};
}

constexpr int kPer = 4;                // blocks per thread and round of a pass over the pool

// Number of blocks of [lo, hi) with pred(refs); a single CTA stops once it has `enough`.
// (What the first pass has read the second finds in L1: nothing else writes there in between.)
template <class F>
__device__ int count_blocks(const int32_t* refs, int lo, int hi, int enough, int* red, F pred) {
  int n = 0;
  for (long long at = lo; at < hi; at += (long long)kThreads * kPer) {
    int mine = 0, all;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const long long i = at + k * kThreads + threadIdx.x;
      if (i < hi) mine += pred(refs[i]) ? 1 : 0;
    }
    cta_scan(mine, red, &all);
    n += all;
    if (n >= enough) break;
  }
  return n;
}

// f(block, refs, blocks of the pool before it with pred) for the blocks of [lo, hi), in
// rounds from lo on, until `until` blocks with pred lie behind; before: those ahead of lo.
template <class P, class F>
__device__ void visit_blocks(const int32_t* refs, int lo, int hi, int before, int until, int* red, P pred, F f) {
  for (long long at = lo; at < hi && before < until; at += (long long)kThreads * kPer) {
    int v[kPer], mine = 0, all;
    const long long first = at + (long long)threadIdx.x * kPer;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      v[k] = first + k < hi ? refs[first + k] : 0;
      mine += first + k < hi && pred(v[k]) ? 1 : 0;
    }
    int rank = before + cta_scan(mine, red, &all);
#pragma unroll
    for (int k = 0; k < kPer; ++k)
      if (first + k < hi) {
        f((int)(first + k), v[k], rank);
        rank += pred(v[k]) ? 1 : 0;
      }
    before += all;
  }
}

// Sum of the CTAs' counts and of those before this one.
__device__ __forceinline__ void sum_counts(const int* counts, int* before, int* all) {
  int c[kCluster];
#pragma unroll
  for (int b = 0; b < kCluster; ++b) c[b] = b < (int)gridDim.x ? __ldcg(counts + b) : 0;
  *before = *all = 0;
#pragma unroll
  for (int b = 0; b < kCluster; ++b) {
    *before += b < (int)blockIdx.x ? c[b] : 0;
    *all += c[b];
  }
}

struct IsFree {
  __device__ bool operator()(int r) const { return r == 0; }
};
struct IsLive {
  __device__ bool operator()(int r) const { return r > 0; }
};
constexpr int kNoLimit = 0x7fffffff;

// A row's length as far as its table row goes.
__device__ __forceinline__ int fit_len(const Pool& P, int n, bool report) {
  const long long most = (long long)P.width * kBlockSize;
  if (n >= 0 && n <= most) return n;
  if (report) set_error(P.err, CB_DEVERR_BADLEN);
  return n < 0 ? 0 : (int)most;
}

// A table entry that names a block; -1 entries (blocks let go of) name none.
__device__ __forceinline__ bool names_block(const Pool& P, int e) {
  if (e >= P.num_blocks) set_error(P.err, CB_DEVERR_BADBLOCK);
  return e >= 0 && e < P.num_blocks;
}

constexpr int kUnroll = 4;             // reads of a lane in flight in a row's passes

// ---------------------------------------------------------------- fork
// Row j becomes the first keep[j] tokens of row parents[j] as it was before the
// call.  Every CTA knows all rows' parents, lengths and partial last blocks, and
// has the latter in a hash table: how many rows end in each, and the lowest.
//   A  (warp per row) counts of the blocks that the row lets go of and takes;
//      equal entries of both rows cancel.  A row that changes is saved if others
//      come from it.
//   B  rows whose partial last block is held elsewhere too need a copy, but for
//      the lowest of its holders if all of them end in it.
//   C  the k-th row in need gets the k-th lowest free block; tables are written.
//   D  the copies' entries and counts, pairs and lengths.
// A barrier after A, after C's counting of free blocks and after C; the last two
// only if a row is in need.
// 4 beams of up to 400 tokens: 8.3 us with their copies; 128 beams of 1000 to 1700 tokens: 15
// (cold) before the copies.  Five dependent reads bound it.
struct ForkArgs {
  Pool P;
  const int32_t* parents;
  const int32_t* keep;                 // nullptr: all
  int32_t* pairs;                      // [n_rows][2]
  int hash;                            // entries of the hash table, a power of two > n_rows
  // workspace
  int32_t* old_rows;                   // [n_rows][width]
  int32_t* fresh;                      // [n_rows] lowest free blocks
  int32_t* counts;                     // [kCluster]
};
constexpr int kForkInts = 6;           // shared ints per row, and kHashInts per entry of the table
constexpr int kHashInts = 3;

struct ForkRow {
  int parent, had, has;                // parent -1: none; tokens before and after
};

__global__ void __launch_bounds__(kThreads) fork_kernel(const ForkArgs A) {
  __shared__ int red[kWarps];
  extern __shared__ int shared_ints[];
  const Pool& P = A.P;
  const int n = P.n_rows;
  int* parent = shared_ints;
  int* had = parent + n;
  int* has = had + n;
  int* last = has + n;                 // partial last block, -1: none
  int* rank = last + n;                // among the rows in need, -1: none
  int* source = rank + n;              // some other row comes from this one
  int* key = source + n;               // block, -1: empty
  int* ends = key + A.hash;            // rows that end in it
  int* lowest = ends + A.hash;
  const int lane = threadIdx.x & 31;
  const int w0 = blockIdx.x * kWarps + (threadIdx.x >> 5), nw = gridDim.x * kWarps;
  for (int j = threadIdx.x; j < n; j += kThreads) {
    const int p = __ldg(A.parents + j), l = __ldcg(P.lens + j);
    const int k = A.keep ? __ldg(A.keep + j) : -1;
    if (p >= n && blockIdx.x == 0) set_error(P.err, CB_DEVERR_BADLEN);
    parent[j] = p >= n ? -1 : p;
    had[j] = fit_len(P, l, blockIdx.x == 0);
    has[j] = k;
    source[j] = 0;
  }
  for (int h = threadIdx.x; h < A.hash; h += kThreads) {
    key[h] = -1;
    ends[h] = 0;
    lowest[h] = n;
  }
  __syncthreads();
  auto row = [&](int j) { return ForkRow{parent[j], had[j], has[j]}; };
  auto changes = [&](const ForkRow& f, int j) { return f.parent != j || blocks_of(f.has) < blocks_of(f.had); };
  auto place = [&](int e) {            // of block e in the hash table, or of the empty entry for it
    unsigned h = (unsigned)e * 2654435761u >> 16 & (A.hash - 1);
    while (key[h] != e && key[h] != -1) h = (h + 1) & (A.hash - 1);
    return h;
  };
  for (int j = threadIdx.x; j < n; j += kThreads) {
    const int p = parent[j], k = has[j];
    int m = p < 0 ? 0 : had[p];
    if (k >= 0) m = min(m, k);
    has[j] = m;
    if (p >= 0 && p != j) source[p] = 1;
    int e = -1;
    if (m % kBlockSize) {
      e = __ldcg(P.tables + (size_t)p * P.width + m / kBlockSize);
      if (!names_block(P, e)) e = -1;
    }
    last[j] = e;
    if (e >= 0) {
      unsigned h = place(e);
      for (int got; (got = atomicCAS(key + h, -1, e)) != -1 && got != e;) h = (h + 1) & (A.hash - 1);
      atomicAdd(ends + h, 1);
      atomicMin(lowest + h, j);
    }
  }
  __syncthreads();
  // A
  for (int j = w0; j < n; j += nw) {
    const ForkRow f = row(j);
    const int ob = blocks_of(f.had), nb = blocks_of(f.has);
    if (!changes(f, j)) continue;
    const int32_t* mine = P.tables + (size_t)j * P.width;
    const int32_t* theirs = P.tables + (size_t)max(f.parent, 0) * P.width;
    int32_t* save = A.old_rows + (size_t)j * P.width;
    const bool saves = source[j];
    for (int c0 = lane; c0 < max(ob, nb); c0 += 32 * kUnroll) {
      int a[kUnroll], b[kUnroll];
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) {
        const int c = c0 + 32 * k;
        a[k] = c < ob ? __ldcg(mine + c) : -1;
        b[k] = c >= nb ? -1 : f.parent == j ? a[k] : __ldcg(theirs + c);
      }
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) {
        const int c = c0 + 32 * k;
        if (saves && c < ob) save[c] = a[k];
        if (a[k] == b[k]) continue;
        if (names_block(P, a[k])) atomicAdd(P.refs + a[k], -1);
        if (names_block(P, b[k])) atomicAdd(P.refs + b[k], 1);
      }
    }
  }
  sync_all();
  // B
  int wanted = 0;
  for (int at = 0; at < n; at += kThreads) {
    const int j = at + threadIdx.x, e = j < n ? last[j] : -1;
    int need = 0, all;
    if (e >= 0) {
      const int held = __ldcg(P.refs + e);
      const unsigned h = place(e);
      need = held != 1 && !(ends[h] == held && lowest[h] == j);
    }
    const int k = wanted + cta_scan(need, red, &all);
    if (j < n) rank[j] = need ? k : -1;
    wanted += all;                     // the same in every CTA
  }
  // C
  const Slice s = my_slice(P.num_blocks);
  int before = 0, found = 0;
  if (wanted) {
    found = count_blocks(P.refs, s.lo, s.hi, gridDim.x > 1 ? kNoLimit : wanted, red, IsFree());
    if (gridDim.x > 1) {
      if (threadIdx.x == 0) A.counts[blockIdx.x] = found;
      sync_all();
      sum_counts(A.counts, &before, &found);
    }
    visit_blocks(P.refs, s.lo, s.hi, before, wanted, red, IsFree(), [&](int b, int r, int k) {
      if (r == 0 && k < wanted) A.fresh[k] = b;
    });
  }
  for (int j = w0; j < n; j += nw) {
    const ForkRow f = row(j);
    const int ob = blocks_of(f.had), nb = blocks_of(f.has);
    int32_t* mine = P.tables + (size_t)j * P.width;
    if (f.parent >= 0 && f.parent != j) {
      // the parent's row as it was: saved if it changes too, else untouched so far
      const bool saved = changes(row(f.parent), f.parent);
      const int32_t* theirs = (saved ? A.old_rows : P.tables) + (size_t)f.parent * P.width;
      for (int c0 = lane; c0 < nb; c0 += 32 * kUnroll) {
        int b[kUnroll];
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) b[k] = c0 + 32 * k < nb ? __ldcg(theirs + c0 + 32 * k) : 0;
#pragma unroll
        for (int k = 0; k < kUnroll; ++k)
          if (c0 + 32 * k < nb) mine[c0 + 32 * k] = b[k];
      }
    }
    for (int c = nb + lane; c < ob; c += 32) mine[c] = -1;
  }
  if (wanted) sync_all();
  // D
  for (int j = blockIdx.x * kThreads + threadIdx.x; j < n; j += gridDim.x * kThreads) {
    int m = has[j], src = -1, dst = -1;
    if (rank[j] >= 0) {
      const int e = last[j], b = rank[j] < found ? __ldcg(A.fresh + rank[j]) : -1;
      P.tables[(size_t)j * P.width + m / kBlockSize] = b;
      atomicAdd(P.refs + e, -1);
      if (b >= 0) {
        P.refs[b] = 1;
        src = e;
        dst = b;
      } else {
        set_error(P.err, CB_DEVERR_NOBLOCK);
        m = m / kBlockSize * kBlockSize;
      }
    }
    P.lens[j] = m;
    A.pairs[2 * j] = src;
    A.pairs[2 * j + 1] = dst;
  }
}

// ---------------------------------------------------------------- grow
// Row i gets room for its cu[i + 1] - cu[i] new tokens.  Every CTA knows what
// each row needs (a prefix sum over the rows); the CTA that finds the k-th
// lowest free block in its slice hands it to the row that k falls to.  48 rows by up to 8 tokens:
// 8.4 us with the caller's reset of the pool; 512 rows by up to 2000 tokens: 24 (cold: 19.6 and
// 11.1 for the slots).  A pass over the pool's counts, twice, and the barriers bound it.
struct GrowArgs {
  Pool P;
  const int32_t* cu;                   // [n_rows + 1]
  int32_t* ctx;                        // [n_rows]
  int64_t* slots;                      // [n_tokens]
  int n_tokens;
  int many;                            // slots_kernel follows
  int32_t* counts;                     // workspace: [kCluster]
};

// Slot of position pos of row i (pos < 0, or past the table row: none).
__device__ __forceinline__ int64_t slot_of(const Pool& P, int i, int pos) {
  if (pos < 0 || pos / kBlockSize >= P.width) return -1;
  const int e = __ldcg(P.tables + (size_t)i * P.width + pos / kBlockSize);
  if (e >= 0 && e < P.num_blocks) return (int64_t)e * kBlockSize + pos % kBlockSize;
  set_error(P.err, CB_DEVERR_BADBLOCK);
  return -1;
}

// The last i of [0, n) with a[i] <= x (a[0] <= x).
__device__ __forceinline__ int last_at_most(const int* a, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kThreads) grow_kernel(const GrowArgs A) {
  __shared__ int red[kWarps];
  __shared__ int ends[kMaxReqs];       // needs of the rows up to and with this one
  __shared__ int cu[kMaxReqs + 1], len[kMaxReqs];
  __shared__ uint8_t bad[kMaxReqs];
  const Pool& P = A.P;
  const int n = P.n_rows;
  int wanted = 0;
  for (int at = 0; at < n; at += kThreads) {
    const int i = at + threadIdx.x;
    int need = 0, all;
    if (i < n) {
      const int q0 = __ldg(A.cu + i), q1 = __ldg(A.cu + i + 1), raw = __ldcg(P.lens + i);
      const int l = fit_len(P, raw, blockIdx.x == 0);
      const bool no = l != raw || q0 < 0 || q1 < q0 || q1 > A.n_tokens ||
                      (long long)l + (q1 - q0) > (long long)P.width * kBlockSize;
      if (no && blockIdx.x == 0) set_error(P.err, CB_DEVERR_BADLEN);
      if (!no) need = blocks_of(l + (q1 - q0)) - blocks_of(l);
      cu[i] = q0;
      if (i == n - 1) cu[n] = q1;
      len[i] = l;
      bad[i] = no;
    }
    const int rank = wanted + cta_scan(need, red, &all);
    if (i < n) ends[i] = rank + need;
    wanted += all;
  }
  __syncthreads();
  const Slice s = my_slice(P.num_blocks);
  int before = 0, found = 0;
  if (wanted) {                        // the same in every CTA
    found = count_blocks(P.refs, s.lo, s.hi, gridDim.x > 1 ? kNoLimit : wanted, red, IsFree());
    if (gridDim.x > 1 && threadIdx.x == 0) A.counts[blockIdx.x] = found;
  }
  sync_all();                          // every CTA has read lens; counts
  if (wanted) {
    if (gridDim.x > 1) sum_counts(A.counts, &before, &found);
    int i = n;                         // a thread's free blocks go to rows in order
    visit_blocks(P.refs, s.lo, s.hi, before, wanted, red, IsFree(), [&](int b, int r, int rank) {
      if (r != 0 || rank >= wanted) return;
      // the row whose needs reach past rank: the first with ends > rank
      if (i == n || ends[i] <= rank) {
        if (i + 1 < n && ends[i + 1] > rank) {
          ++i;
        } else {
          int lo = 0, hi = n - 1;
          while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (ends[mid] > rank) hi = mid;
            else lo = mid + 1;
          }
          i = lo;
        }
      }
      if (ends[i] > found) return;     // not enough for the whole row: it gets none
      const int first = i ? ends[i - 1] : 0;
      P.tables[(size_t)i * P.width + blocks_of(len[i]) + rank - first] = b;
      P.refs[b] = 1;
    });
    sync_all();
  }
  auto granted = [&](int i) {
    return !bad[i] && (ends[i] <= found || ends[i] == (i ? ends[i - 1] : 0));
  };
  for (int i = blockIdx.x * kThreads + threadIdx.x; i < n; i += gridDim.x * kThreads) {
    const bool ok = granted(i);
    if (!ok && !bad[i]) set_error(P.err, CB_DEVERR_NOBLOCK);
    A.ctx[i] = len[i];
    if (ok) P.lens[i] = len[i] + cu[i + 1] - cu[i];
  }
  if (A.many) return;                  // slots_kernel
  for (int t = blockIdx.x * kThreads + threadIdx.x; t < A.n_tokens; t += gridDim.x * kThreads) {
    const int i = last_at_most(cu, n, t);
    int pos = -1;
    if (t >= cu[i] && t < cu[i + 1] && granted(i)) pos = len[i] + t - cu[i];
    A.slots[t] = slot_of(P, i, pos);
  }
}

// The slots of many tokens, on the whole device: rows that have grown say so by
// their lengths.  A warp takes 32 * kRun tokens, whose entries are read together.
constexpr int kRun = 8, kSlotThreads = 256;
__global__ void __launch_bounds__(kSlotThreads) slots_kernel(const GrowArgs A) {
  __shared__ int cu[kMaxReqs + 1], len[kMaxReqs];
  const Pool& P = A.P;
  const int n = P.n_rows, lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  for (int i = threadIdx.x; i <= n; i += kSlotThreads) {
    cu[i] = __ldg(A.cu + i);
    if (i == n) break;
    const int was = __ldcg(A.ctx + i), now = __ldcg(P.lens + i);
    len[i] = (long long)was + __ldg(A.cu + i + 1) - cu[i] == now ? was : -1;
  }
  __syncthreads();
  const int w0 = blockIdx.x * (kSlotThreads / 32) + (threadIdx.x >> 5), nw = gridDim.x * (kSlotThreads / 32);
  for (long long t0 = (long long)w0 * 32 * kRun; t0 < A.n_tokens; t0 += (long long)nw * 32 * kRun) {
    int i = last_at_most(cu, n, (int)t0);
    int64_t slot[kRun];
#pragma unroll
    for (int k = 0; k < kRun; ++k) {
      const long long t = t0 + k * 32 + lane;
      slot[k] = -1;
      if (t >= A.n_tokens) continue;
      if (t >= cu[i + 1]) i = i + 1 < n && t < cu[i + 2] ? i + 1 : last_at_most(cu, n, (int)t);
      const bool in = t >= cu[i] && t < cu[i + 1] && len[i] >= 0;
      slot[k] = slot_of(P, i, in ? len[i] + (int)t - cu[i] : -1);
    }
#pragma unroll
    for (int k = 0; k < kRun; ++k)
      if (t0 + k * 32 + lane < A.n_tokens) A.slots[t0 + k * 32 + lane] = slot[k];
  }
}

// ---------------------------------------------------------------- compact
// With L live blocks, the k-th lowest live block of id >= L moves to the k-th
// lowest free id < L (there are as many of the one as of the other).  8 rows and 333 blocks:
// 10.5 us with the moves' copies; 256 rows and 28,610 blocks: 17 before the copies.  Seven
// dependent reads and the cluster's barriers bound it.
struct CompactArgs {
  Pool P;
  int32_t* map;                        // [num_blocks]
  int32_t* pairs;                      // [max_pairs][2]
  int max_pairs;
  int32_t* result;                     // [2] live blocks, pairs written
  // workspace
  int2* movers;                        // [num_blocks / 2 + 1] (block, holders)
  int32_t* holes;                      // [num_blocks / 2 + 1]
  int32_t* counts;                     // [kCluster]
};

__global__ void __launch_bounds__(kThreads) compact_kernel(const CompactArgs A) {
  __shared__ int red[kWarps];
  const Pool& P = A.P;
  const int lane = threadIdx.x & 31, nb = P.num_blocks;
  const Slice s = my_slice(nb);
  int before = 0, live = count_blocks(P.refs, s.lo, s.hi, kNoLimit, red, IsLive());
  int under = 0;                       // live blocks under the line: whole slices, then the one that it cuts
  if (gridDim.x > 1) {
    if (threadIdx.x == 0) A.counts[blockIdx.x] = live;
    sync_all();
    sum_counts(A.counts, &before, &live);
    const int size = slice_size(nb), cut = live / size;
#pragma unroll
    for (int b = 0; b < kCluster; ++b) under += b < cut ? __ldcg(A.counts + b) : 0;
    under += count_blocks(P.refs, cut * size, live, kNoLimit, red, IsLive());
  } else {
    under = count_blocks(P.refs, 0, live, kNoLimit, red, IsLive());
  }
  const int moves = live - under, done = min(moves, A.max_pairs);
  visit_blocks(P.refs, s.lo, s.hi, before, kNoLimit, red, IsLive(), [&](int b, int r, int rank) {
    const bool is = r > 0;
    if (b < live) {
      if (!is) A.holes[b - rank] = b;
      A.map[b] = is ? b : -1;
    } else {
      if (is) A.movers[rank - under] = make_int2(b, r);
      if (!is || rank - under >= done) A.map[b] = is ? b : -1;
    }
  });
  if (moves) sync_all();
  for (int k = blockIdx.x * kThreads + threadIdx.x; k < A.max_pairs; k += gridDim.x * kThreads) {
    int src = -1, dst = -1;
    if (k < done) {
      const int2 m = __ldcg(A.movers + k);
      src = m.x;
      dst = __ldcg(A.holes + k);
      A.map[src] = dst;
      P.refs[dst] = m.y;
      P.refs[src] = 0;
    }
    A.pairs[2 * k] = src;
    A.pairs[2 * k + 1] = dst;
  }
  if (blockIdx.x == 0 && threadIdx.x < 2) A.result[threadIdx.x] = threadIdx.x ? done : live;
  if (!done) return;                   // the same in every CTA
  sync_all();
  const int w0 = blockIdx.x * kWarps + (threadIdx.x >> 5), nw = gridDim.x * kWarps;
  for (int j = w0; j < P.n_rows; j += nw) {
    int32_t* row = P.tables + (size_t)j * P.width;
    const int n = blocks_of(fit_len(P, __ldcg(P.lens + j), lane == 0));
    for (int c0 = lane; c0 < n; c0 += 32 * kUnroll) {
      int e[kUnroll], to[kUnroll];
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) e[k] = c0 + 32 * k < n ? __ldcg(row + c0 + 32 * k) : -1;
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) to[k] = names_block(P, e[k]) ? __ldcg(A.map + e[k]) : -1;
#pragma unroll
      for (int k = 0; k < kUnroll; ++k)
        if (to[k] >= 0 && to[k] != e[k]) row[c0 + 32 * k] = to[k];
    }
  }
}

// ---------------------------------------------------------------- copies in every layer
// Block dst becomes block src in every layer of every buffer.  Memory-bound: a
// warp copies 4 KB at a time, eight 16-byte loads in flight per lane.  Pairs are
// taken kTile at a time; each CTA packs the tile's valid ones in shared memory,
// and the 4 KB pieces of all of them are dealt over all warps of the grid.  1024 blocks of 32
// layers, 4.3 GB read and written: 660 to 676 us, 0.94 to 0.96 of a plain copy's rate.
struct CopyArgs {
  const int32_t* pairs;
  int n_pairs, n_layers, num_blocks, n_buffers;
  uint8_t* base[CB_MAX_CACHE_BUFFERS];
  unsigned bytes[CB_MAX_CACHE_BUFFERS];   // of a block
  unsigned ends[CB_MAX_CACHE_BUFFERS];    // pieces of a block of the buffers up to and with this one
  unsigned int* err;
};
constexpr int kCopyThreads = 512, kCopyWarps = kCopyThreads / 32, kTile = 2048, kPiece = 4096;

__global__ void __launch_bounds__(kCopyThreads) copy_layers_kernel(const CopyArgs A) {
  __shared__ int2 valid[kTile];
  __shared__ int warp_n[kCopyWarps + 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const unsigned per_layer = A.ends[A.n_buffers - 1];
  const long long nw = (long long)gridDim.x * kCopyWarps;
  long long turn = (long long)warp * gridDim.x + blockIdx.x;      // this warp's place, over all tiles
  for (int at = 0; at < A.n_pairs; at += kTile) {
    const int n_tile = min(kTile, A.n_pairs - at);
    // pack: warp w takes the pairs [w, w + 1) * kTile / kCopyWarps
    constexpr int kMine = kTile / kCopyWarps / 32;
    int2 p[kMine];
    int kept = 0;
    unsigned ok = 0;
#pragma unroll
    for (int k = 0; k < kMine; ++k) {
      const int i = warp * (kTile / kCopyWarps) + k * 32 + lane;
      p[k] = i < n_tile ? make_int2(__ldg(A.pairs + 2 * (at + i)), __ldg(A.pairs + 2 * (at + i) + 1)) : make_int2(-1, -1);
      bool good = p[k].x >= 0;
      if (good && (p[k].x >= A.num_blocks || p[k].y < 0 || p[k].y >= A.num_blocks)) {
        if (blockIdx.x == 0) set_error(A.err, CB_DEVERR_BADBLOCK);
        good = false;
      }
      ok |= (unsigned)good << k;
      kept += __popc(__ballot_sync(0xffffffffu, good));
    }
    __syncthreads();                   // the last tile's pairs are done with
    if (lane == 0) warp_n[warp] = kept;
    __syncthreads();
    int first = 0, n = 0;
    for (int w = 0; w < kCopyWarps; ++w) {
      first += w < warp ? warp_n[w] : 0;
      n += warp_n[w];
    }
#pragma unroll
    for (int k = 0; k < kMine; ++k) {
      const unsigned m = __ballot_sync(0xffffffffu, ok >> k & 1);
      if (ok >> k & 1) valid[first + __popc(m & ((1u << lane) - 1))] = p[k];
      first += __popc(m);
    }
    __syncthreads();
    const long long per_pair = (long long)per_layer * A.n_layers, total = per_pair * n;
    long long u = turn;
    for (; u < total; u += nw) {
      const int i = (int)(u / per_pair);
      const unsigned rest = (unsigned)(u - i * per_pair);
      const unsigned layer = rest / per_layer;
      unsigned piece = rest - layer * per_layer;
      int b = 0;
      while (piece >= A.ends[b]) ++b;
      if (b) piece -= A.ends[b - 1];
      const size_t bytes = A.bytes[b];
      const size_t off = (size_t)piece * kPiece;
      const size_t at_layer = (size_t)layer * A.num_blocks;
      const int vecs = (int)(min(bytes - off, (size_t)kPiece) / 16);
      const uint4* src = reinterpret_cast<const uint4*>(A.base[b] + (at_layer + valid[i].x) * bytes + off);
      uint4* dst = reinterpret_cast<uint4*>(A.base[b] + (at_layer + valid[i].y) * bytes + off);
      uint4 v[kPiece / 512];
#pragma unroll
      for (int k = 0; k < kPiece / 512; ++k)
        if (k * 32 + lane < vecs) v[k] = __ldcs(src + k * 32 + lane);
#pragma unroll
      for (int k = 0; k < kPiece / 512; ++k)
        if (k * 32 + lane < vecs) __stcs(dst + k * 32 + lane, v[k]);
    }
    turn = u - total;
  }
}

// ---------------------------------------------------------------- launches
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }

// One cluster of `ctas` CTAs (1, 8 or 16).
template <class Args>
cudaError_t launch_pool(void (*kernel)(const Args), const Args& a, int ctas, size_t smem, cudaStream_t stream) {
  if (ctas == 1) {
    kernel<<<1, kThreads, smem, stream>>>(a);
    return cudaGetLastError();
  }
  if (ctas > 8) {                      // past the portable size
    const cudaError_t e = allow_large_clusters(reinterpret_cast<const void*>(kernel));
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

// A kernel that is placed while the one before it on the stream ends, and waits for it itself.
template <class Args>
cudaError_t launch_behind(void (*kernel)(const Args), const Args& a, int ctas, int threads, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

// Slots that one cluster writes itself.  GPU time (us) so and with slots_kernel, a pool of 100,000 blocks: 8000
// tokens 10.5 and 15.0, 16,000 11.1 and 15.0, 64,000 16.7 to 22.8 and 15.9 to 20.8, 512,000 81 and 21: up to some
// 50,000 tokens the second kernel costs 4, past that it gives all but itself.
constexpr int kManyTokens = 8192;
// What a single CTA goes over alone.  GPU time of the call (us) with 1, 8 and 16 CTAs:
//  growth of 48 rows by up to 8 tokens, in pools of 2000 to 65,536 blocks whose first free ones lie low (one CTA
//    stops at the last block that it needs): 6.1-8.0, 8.4-11.1, 10.4-11.5; where the first 95 % are taken: 8000
//    blocks 8.3, 8.8, 10.6; 14,000 11.5, 8.9, 11.2; 32,768 18.6, 9.4, 11.3; 65,536 33.8, 10.9, 10.8.  How full a
//    pool is the host does not know: kSmallGrowth is a size at which neither loses more than 3.
//  growth of 512 rows that take 32,000 of 100,000 blocks, with their slots: 55.8, 31.3, 24.0
//  compaction of 32 rows: 2000 blocks 5.8, 9.5, 11.1; 4000 7.8, 11.1, 13.0; 8192 14.0, 12.7, 15.8; 16,384 23.8,
//    16.0, 18.8; of 64 rows and 1920 blocks 6.6, 9.5, 13.1; of 256 and 7680 16.0, 10.3, 14.0
//  fork without copies, in pools of any size: 8 rows 4.3-4.6, 4.7-5.1, 4.7-5.1; 64 7.6, 6.2, 6.2; 128 10.7, 6.2, 6.3
constexpr int kSmallPool = 8192, kSmallRows = 64, kSmallGrowth = 16384;

constexpr int kMostPairs = 1 << 30;    // their ints are counted in 32 bits
constexpr int kMostBlocks = 1 << 30;   // a CTA's share is rounded up in 32 bits

// The pool arguments that the calls share; false: CB_EINVAL.
bool pool_of(Pool* P, int32_t* tables, int width, int n_rows, int32_t* lens, int32_t* refs, int num_blocks, int block_size) {
  if (n_rows < 0 || n_rows > CB_MAX_REQS || width < 1 || num_blocks < 1 || num_blocks > kMostBlocks ||
      block_size != kBlockSize)
    return false;
  if ((long long)n_rows * width >= 1LL << 31 || (long long)width * kBlockSize >= 1LL << 31) return false;
  if (n_rows == 0) return true;
  if (!tables || !lens || !refs || !aligned4(tables) || !aligned4(lens) || !aligned4(refs)) return false;
  *P = Pool{tables, lens, refs, n_rows, width, num_blocks, nullptr};
  return true;
}

// No C++ exception (an allocation or a lock of the library's host state) leaves an entry point.
template <class F>
int guarded(F call) {
  try {
    return call();
  } catch (...) {
    return CB_ECUDA;
  }
}

// Ints of workspace: the fork's and the compaction's.
size_t fork_ints(int n_rows, int width) { return (size_t)n_rows * width + (size_t)n_rows + kCluster; }
size_t compact_ints(int num_blocks) { return 3 * ((size_t)num_blocks / 2 + 1) + kCluster; }

}  // namespace
}  // namespace cb

using namespace cb;

extern "C" {

size_t cb_block_ops_workspace_size(int n_rows, int max_blocks_per_seq, int num_blocks, int block_size) {
  Pool P;
  int32_t any = 0;
  if (!pool_of(&P, &any, max_blocks_per_seq, n_rows, &any, &any, num_blocks, block_size)) return 0;
  return (std::max(fork_ints(n_rows, max_blocks_per_seq), compact_ints(num_blocks)) * 4 + 255) / 256 * 256;
}

int cb_fork_blocks(const int32_t* parents, const int32_t* keep_lens, int32_t* block_tables, int max_blocks_per_seq,
                   int n_rows, int32_t* lens, int32_t* refs, int num_blocks, int block_size, int32_t* pairs,
                   void* workspace, size_t workspace_bytes, void* stream) {
  return guarded([&]() -> int {
    ForkArgs a{};
    if (!pool_of(&a.P, block_tables, max_blocks_per_seq, n_rows, lens, refs, num_blocks, block_size)) return CB_EINVAL;
    if (n_rows == 0) {
      set_last_launches(0);
      return CB_OK;
    }
    if (!parents || !pairs || !workspace || !aligned4(parents) || !aligned4(keep_lens) || !aligned4(pairs) ||
        !aligned16(workspace))
      return CB_EINVAL;
    if (workspace_bytes < fork_ints(n_rows, max_blocks_per_seq) * 4) return CB_EWORKSPACE;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    int rc = CB_OK;
    a.P.err = stream_error_word(st, &rc);
    if (!a.P.err) return rc;
    a.parents = parents;
    a.keep = keep_lens;
    a.pairs = pairs;
    int32_t* w = static_cast<int32_t*>(workspace);
    a.old_rows = w;
    a.fresh = w + (size_t)n_rows * max_blocks_per_seq;
    a.counts = a.fresh + n_rows;
    a.hash = 64;
    while (a.hash <= n_rows) a.hash *= 2;
    const size_t smem = ((size_t)kForkInts * n_rows + (size_t)kHashInts * a.hash) * 4;
    constexpr int kMostSmem = (kForkInts * CB_MAX_REQS + kHashInts * 2 * CB_MAX_REQS) * 4;
    if (smem > 48 * 1024 - 256 && opt_in_smem(reinterpret_cast<const void*>(fork_kernel), kMostSmem) != cudaSuccess)
      return CB_ECUDA;
    if (launch_pool(fork_kernel, a, n_rows > kSmallRows || num_blocks > kSmallPool ? 8 : 1, smem, st) != cudaSuccess) return CB_ECUDA;
    set_last_launches(1);
    return CB_OK;
  });
}

int cb_grow_blocks(const int32_t* cu_q_lens, int32_t* block_tables, int max_blocks_per_seq, int n_rows, int32_t* lens,
                   int32_t* refs, int num_blocks, int block_size, int32_t* ctx_lens, int64_t* slot_mapping,
                   int n_tokens, void* workspace, size_t workspace_bytes, void* stream) {
  return guarded([&]() -> int {
    GrowArgs a{};
    if (!pool_of(&a.P, block_tables, max_blocks_per_seq, n_rows, lens, refs, num_blocks, block_size) || n_tokens < 0)
      return CB_EINVAL;
    if (n_rows == 0) {
      set_last_launches(0);
      return CB_OK;
    }
    if (!cu_q_lens || !ctx_lens || !workspace || !aligned4(cu_q_lens) || !aligned4(ctx_lens) || !aligned16(workspace) ||
        (n_tokens && (!slot_mapping || reinterpret_cast<uintptr_t>(slot_mapping) & 7)))
      return CB_EINVAL;
    if (workspace_bytes < kCluster * 4) return CB_EWORKSPACE;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    int rc = CB_OK;
    a.P.err = stream_error_word(st, &rc);
    if (!a.P.err) return rc;
    a.cu = cu_q_lens;
    a.ctx = ctx_lens;
    a.slots = slot_mapping;
    a.n_tokens = n_tokens;
    a.counts = static_cast<int32_t*>(workspace);
    a.many = n_tokens > kManyTokens;
    if (launch_pool(grow_kernel, a, a.many ? 16 : num_blocks > kSmallGrowth ? 8 : 1, 0, st) != cudaSuccess) return CB_ECUDA;
    if (a.many) {
      int sms = 0;
      if (!device_sms(&sms)) return CB_ECUDA;
      const int ctas = std::min(2 * sms, (n_tokens - 1) / (kSlotThreads * kRun) + 1);
      if (launch_behind(slots_kernel, a, ctas, kSlotThreads, st) != cudaSuccess) return CB_ECUDA;
    }
    set_last_launches(a.many ? 2 : 1);
    return CB_OK;
  });
}

int cb_compact_blocks(int32_t* block_tables, int max_blocks_per_seq, int n_rows, int32_t* lens, int32_t* refs,
                      int num_blocks, int block_size, int32_t* block_map, int32_t* pairs, int max_pairs, int32_t* counts,
                      void* workspace, size_t workspace_bytes, void* stream) {
  return guarded([&]() -> int {
    CompactArgs a{};
    int32_t any = 0;                   // without rows there is still a pool
    if (!pool_of(&a.P, n_rows ? block_tables : &any, max_blocks_per_seq, n_rows, n_rows ? lens : &any, refs, num_blocks,
                 block_size) || max_pairs < 0 || max_pairs > kMostPairs)
      return CB_EINVAL;
    if (!refs || !aligned4(refs) || !block_map || !counts || !workspace || !aligned4(block_map) || !aligned4(counts) ||
        !aligned16(workspace) || (max_pairs && (!pairs || !aligned4(pairs))))
      return CB_EINVAL;
    if (workspace_bytes < compact_ints(num_blocks) * 4) return CB_EWORKSPACE;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    int rc = CB_OK;
    a.P = Pool{block_tables, lens, refs, n_rows, max_blocks_per_seq, num_blocks, stream_error_word(st, &rc)};
    if (!a.P.err) return rc;
    a.map = block_map;
    a.pairs = pairs;
    a.max_pairs = max_pairs;
    a.result = counts;
    a.movers = static_cast<int2*>(workspace);
    a.holes = reinterpret_cast<int32_t*>(a.movers + num_blocks / 2 + 1);
    a.counts = a.holes + num_blocks / 2 + 1;
    if (launch_pool(compact_kernel, a, num_blocks > kSmallPool || n_rows > kSmallRows ? 8 : 1, 0, st) != cudaSuccess) return CB_ECUDA;
    set_last_launches(1);
    return CB_OK;
  });
}

int cb_copy_blocks_layers(const int32_t* pairs, int n_pairs, void* const* caches, const size_t* block_bytes, int n_caches,
                          int n_layers, int num_blocks, void* stream) {
  return guarded([&]() -> int {
    if (n_pairs < 0 || n_pairs > kMostPairs || n_caches < 1 || n_caches > CB_MAX_CACHE_BUFFERS || n_layers < 1 ||
        num_blocks < 1 || !caches || !block_bytes)
      return CB_EINVAL;
    CopyArgs a{};
    long long pieces = 0;
    for (int i = 0; i < n_caches; ++i) {
      if (!caches[i] || !aligned16(caches[i]) || block_bytes[i] == 0 || block_bytes[i] % 16 || block_bytes[i] >= 1u << 30)
        return CB_EINVAL;
      pieces += ((long long)block_bytes[i] + kPiece - 1) / kPiece;
      a.base[i] = static_cast<uint8_t*>(caches[i]);
      a.bytes[i] = (unsigned)block_bytes[i];
      a.ends[i] = (unsigned)pieces;
    }
    if (pieces * n_layers >= 1LL << 31) return CB_EINVAL;
    if (n_pairs == 0) {
      set_last_launches(0);
      return CB_OK;
    }
    if (!pairs || !aligned4(pairs)) return CB_EINVAL;
    int sms = 0;
    if (!device_sms(&sms)) return CB_ECUDA;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    int rc = CB_OK;
    a.err = stream_error_word(st, &rc);
    if (!a.err) return rc;
    a.pairs = pairs;
    a.n_pairs = n_pairs;
    a.n_layers = n_layers;
    a.num_blocks = num_blocks;
    a.n_buffers = n_caches;
    const long long ctas = (pieces * n_layers * n_pairs + kCopyWarps - 1) / kCopyWarps;
    copy_layers_kernel<<<(unsigned)std::min<long long>(ctas, 2LL * sms), kCopyThreads, 0, st>>>(a);
    if (cudaGetLastError() != cudaSuccess) return CB_ECUDA;
    set_last_launches(1);
    return CB_OK;
  });
}

}  // extern "C"
