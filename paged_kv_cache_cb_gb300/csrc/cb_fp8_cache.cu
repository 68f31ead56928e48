// The 8-bit KV cache's data movement: append with quantisation, read-back and
// block copies (format: cb_fp8.cuh).
//
// One pass each, bound by HBM: 65,536 new tokens (8 KV heads of 128, 404 MB) in 68.5
// us, 5.9 TB/s, 0.87 of a copy's rate; 32,768 rows read back (202 MB) in 34.8 us, 5.8
// TB/s, 0.86; 16,384 blocks of 8 heads copied (1.08 GB) in 171 us, 0.93, 4096 of 32
// heads in 160, 1.00.  A step's few tokens take the launch, 3.5 us of GPU time.
#include <algorithm>

#include "cb_fp8.cuh"

namespace cb {

namespace {

constexpr int kThreads = 256;
constexpr int kPieces = 2;             // per thread, in flight (append, read-back: 1 73, 40 us; 2 70, 36; 4 69, 38)

// 8 bf16 (16 bytes) of a row, its largest |bits| over LANES consecutive lanes.
template <int LANES>
__device__ __forceinline__ uint32_t row_amax(const uint4& x) {
  uint32_t m = __vmaxu2(__vmaxu2(x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu), __vmaxu2(x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu));
#pragma unroll
  for (int o = LANES / 2; o >= 1; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
  return max(m & 0xFFFFu, m >> 16);
}

// 8 bf16 -> 8 e4m3 under the row's exponent byte.
__device__ __forceinline__ uint2 quantise8(const uint4& x, uint32_t b) {
  if (b == kExpNan) return make_uint2(0u, 0u);
  const float f = exp_inverse(b);
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = pack_e4m3(bf16lo(w[i]) * f, bf16hi(w[i]) * f);
  return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}

// 8 e4m3 -> 8 bf16 under the row's exponent byte; exact.
__device__ __forceinline__ uint4 restore8(const uint2& x, uint32_t b) {
  uint32_t o[4];
  widen8(x.x, x.y, factor1(b), o);
  if (b > 134u) {
    const uint32_t f2 = factor2(b), nan = b == kExpNan ? 0x7FC07FC0u : 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = nan ? nan : mul_bf16x2(o[i], f2);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// Where a token's row of a KV head stands in the cache.
__device__ __forceinline__ int64_t cache_row(int64_t slot, uint32_t head, uint32_t n_kv_heads) {
  const uint64_t s = (uint64_t)slot;
  return (int64_t)((s / kBlockSize * n_kv_heads + head) * kBlockSize + s % kBlockSize);
}

// Token t's rows of K and V: LANES = A / 8 lanes hold one row of each, 8 values
// per lane, so a row's largest magnitude is a shuffle reduction and a warp's
// loads and stores are whole 256-byte and 128-byte rows.  A thread has kPieces
// pieces on their way at once.  Rows are counted in 32 bits (2^32 of the smallest
// are 512 GiB of bf16).
template <int LANES>
__global__ void __launch_bounds__(kThreads) append_fp8_kernel(const uint4* __restrict__ k_new, const uint4* __restrict__ v_new,
                                                              const int64_t* __restrict__ slots, int64_t pieces,
                                                              uint2* __restrict__ k_cache, uint2* __restrict__ v_cache,
                                                              uint8_t* __restrict__ k_exps, uint8_t* __restrict__ v_exps,
                                                              int64_t n_slots, uint32_t n_kv_heads, unsigned int* err) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // of a step's attention: it waits for this grid's end
  // rows are whole groups of lanes and pieces % LANES == 0: a group is in or out as one
  for (int64_t i0 = (int64_t)blockIdx.x * kThreads * kPieces; i0 < pieces; i0 += (int64_t)gridDim.x * kThreads * kPieces) {
    uint4 k[kPieces], v[kPieces];
    int64_t slot[kPieces];
    uint32_t head[kPieces];
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
      const int64_t i = i0 + u * kThreads + threadIdx.x;
      const bool in = i < pieces;
      const uint32_t row = (uint32_t)(i / LANES), t = row / n_kv_heads;
      head[u] = row - t * n_kv_heads;
      k[u] = in ? __ldg(k_new + i) : make_uint4(0u, 0u, 0u, 0u);
      v[u] = in ? __ldg(v_new + i) : make_uint4(0u, 0u, 0u, 0u);
      slot[u] = in ? __ldg(slots + t) : -1;
    }
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
      const uint32_t kb = row_exp(row_amax<LANES>(k[u])), vb = row_exp(row_amax<LANES>(v[u]));
      if (slot[u] >= n_slots) {
        set_error(err, CB_DEVERR_BADSLOT);
        slot[u] = -1;
      }
      if (slot[u] < 0) continue;
      const int64_t dst = cache_row(slot[u], head[u], n_kv_heads);
      const int c = threadIdx.x % LANES;
      k_cache[dst * LANES + c] = quantise8(k[u], kb);
      v_cache[dst * LANES + c] = quantise8(v[u], vb);
      if (c == 0) {
        k_exps[dst] = (uint8_t)kb;
        v_exps[dst] = (uint8_t)vb;
      }
    }
  }
}

template <int LANES>
__global__ void __launch_bounds__(kThreads) gather_fp8_kernel(const int64_t* __restrict__ slots, int64_t pieces,
                                                              const uint2* __restrict__ k_cache,
                                                              const uint2* __restrict__ v_cache,
                                                              const uint8_t* __restrict__ k_exps,
                                                              const uint8_t* __restrict__ v_exps, uint4* __restrict__ k_out,
                                                              uint4* __restrict__ v_out, int64_t n_slots, uint32_t n_kv_heads,
                                                              unsigned int* err) {
  for (int64_t i0 = (int64_t)blockIdx.x * kThreads * kPieces; i0 < pieces; i0 += (int64_t)gridDim.x * kThreads * kPieces) {
    int64_t src[kPieces];
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
      const int64_t i = i0 + u * kThreads + threadIdx.x;
      const uint32_t row = (uint32_t)(i / LANES), t = row / n_kv_heads;
      const int64_t slot = i < pieces ? __ldg(slots + t) : -1;
      if (slot >= n_slots) set_error(err, CB_DEVERR_BADSLOT);
      src[u] = slot < 0 || slot >= n_slots ? -1 : cache_row(slot, row - t * n_kv_heads, n_kv_heads);
    }
    uint2 k[kPieces], v[kPieces];
    uint32_t kb[kPieces], vb[kPieces];
    const int c = threadIdx.x % LANES;
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
      const int64_t at = max(src[u], (int64_t)0);            // a row that exists, where there is nothing to read
      k[u] = __ldg(k_cache + at * LANES + c);
      v[u] = __ldg(v_cache + at * LANES + c);
      kb[u] = __ldg(k_exps + at);
      vb[u] = __ldg(v_exps + at);
    }
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
      if (src[u] < 0) continue;
      const int64_t i = i0 + u * kThreads + threadIdx.x;
      k_out[i] = restore8(k[u], kb[u]);
      v_out[i] = restore8(v[u], vb[u]);
    }
  }
}

// Block dst of both caches and of their exponents becomes block src; grid.y =
// pair.  A block is `pieces` 16-byte pieces of values and n_kv_heads of
// exponents.
__global__ void __launch_bounds__(kThreads) copy_blocks_fp8_kernel(const int32_t* __restrict__ pairs, uint4* k_cache, uint4* v_cache,
                                                                   uint4* k_exps, uint4* v_exps, int num_blocks,
                                                                   int64_t pieces, int n_kv_heads, unsigned int* err) {
  const int src = __ldg(pairs + 2 * blockIdx.y), dst = __ldg(pairs + 2 * blockIdx.y + 1);
  if (src < 0 || src >= num_blocks || dst < 0 || dst >= num_blocks) {
    if (blockIdx.x == 0 && threadIdx.x == 0) set_error(err, CB_DEVERR_BADBLOCK);
    return;
  }
  for (int64_t i = blockIdx.x * (int64_t)kThreads + threadIdx.x; i < pieces + n_kv_heads;
       i += (int64_t)gridDim.x * kThreads) {
    const bool e = i >= pieces;
    const int64_t n = e ? n_kv_heads : pieces, at = e ? i - pieces : i;
    uint4* kc = e ? k_exps : k_cache;
    uint4* vc = e ? v_exps : v_cache;
    const uint4 k = kc[src * n + at], v = vc[src * n + at];
    kc[dst * n + at] = k;
    vc[dst * n + at] = v;
  }
}

unsigned grid_for(int64_t pieces) { return (unsigned)std::min<int64_t>((pieces + kThreads - 1) / kThreads, 1 << 20); }

}  // namespace

cudaError_t launch_append_fp8(const void* k_new, const void* v_new, const int64_t* slots, int n_tokens, const Fp8Cache& c,
                              unsigned int* err, cudaStream_t stream) {
  const int lanes = c.head_dim / 8;
  const int64_t pieces = (int64_t)n_tokens * c.n_kv_heads * lanes;
  if (pieces == 0) return cudaSuccess;
#define CB_APPEND(L_)                                                                                                  \
  append_fp8_kernel<L_><<<grid_for((pieces + kPieces - 1) / kPieces), kThreads, 0, stream>>>(                        \
      static_cast<const uint4*>(k_new), static_cast<const uint4*>(v_new), slots, pieces,                               \
      reinterpret_cast<uint2*>(c.k), reinterpret_cast<uint2*>(c.v), c.k_exps, c.v_exps, (int64_t)c.num_blocks * kBlockSize, \
      c.n_kv_heads, err)
  if (lanes == 16)
    CB_APPEND(16);
  else
    CB_APPEND(8);
#undef CB_APPEND
  return cudaGetLastError();
}

cudaError_t launch_gather_fp8(const int64_t* slots, int n_rows, const Fp8Cache& c, void* k_out, void* v_out,
                              unsigned int* err, cudaStream_t stream) {
  const int lanes = c.head_dim / 8;
  const int64_t pieces = (int64_t)n_rows * c.n_kv_heads * lanes;
  if (pieces == 0) return cudaSuccess;
#define CB_GATHER(L_)                                                                                              \
  gather_fp8_kernel<L_><<<grid_for((pieces + kPieces - 1) / kPieces), kThreads, 0, stream>>>(                    \
      slots, pieces, reinterpret_cast<const uint2*>(c.k), reinterpret_cast<const uint2*>(c.v), c.k_exps, c.v_exps, \
      static_cast<uint4*>(k_out), static_cast<uint4*>(v_out), (int64_t)c.num_blocks * kBlockSize, c.n_kv_heads, err)
  if (lanes == 16)
    CB_GATHER(16);
  else
    CB_GATHER(8);
#undef CB_GATHER
  return cudaGetLastError();
}

cudaError_t launch_copy_blocks_fp8(const int32_t* pairs, int n_pairs, const Fp8Cache& c, unsigned int* err,
                                   cudaStream_t stream) {
  if (n_pairs == 0) return cudaSuccess;
  const int64_t pieces = (int64_t)c.n_kv_heads * c.head_dim;        // 16 tokens x head_dim bytes per head
  const int ctas = (int)std::min<int64_t>(8, (pieces + c.n_kv_heads + kThreads - 1) / kThreads);
  copy_blocks_fp8_kernel<<<dim3(ctas, n_pairs), kThreads, 0, stream>>>(
      pairs, reinterpret_cast<uint4*>(c.k), reinterpret_cast<uint4*>(c.v), reinterpret_cast<uint4*>(c.k_exps),
      reinterpret_cast<uint4*>(c.v_exps), c.num_blocks, pieces, c.n_kv_heads, err);
  return cudaGetLastError();
}

}  // namespace cb
