// Joining the pieces that attention over the 8-bit cache has cut sequences into:
//     M = max m_i,  out = sum 2^(m_i - M) l_i o_i / sum 2^(m_i - M) l_i
// over the pieces' (m_i, l_i, o_i), o_i divided by l_i already.  One kernel for the
// single tokens' pieces and the chunks': its first CTAs take the former.  Its CTAs
// are placed while the last pieces are written.
#include "cb_fp8.cuh"

namespace cb {

namespace {

constexpr int kJoinThreads = 256, kWarps = kJoinThreads / 32;

template <int A>
__device__ __forceinline__ void store_row(uint16_t* dst, const float (&o)[A / 32]) {
#pragma unroll
  for (int d = 0; d < A / 32; d += 2) *reinterpret_cast<uint32_t*>(dst + d) = pack_bf16(o[d], o[d + 1]);
}

// n_singles: the CTAs of the single tokens; the others take the chunks.
template <int A>
__global__ void __launch_bounds__(kJoinThreads)
    join_fp8_kernel(const Fp8Step P, const Fp8Partials singles, const Fp8Partials chunks, int ctas, int n_singles, int heads) {
  constexpr int D = A / 32;
  __shared__ int owner[kMaxDecodeGrid];
  __shared__ Fp8Rec recs[kMaxDecodeGrid];
  __shared__ int n_owner;
  __shared__ float red[kWarps][A];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool single = (int)blockIdx.x < n_singles;
  const Fp8Partials& W = single ? singles : chunks;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (P.ready && blockIdx.x == 0 && threadIdx.x == 0) *P.ready = 0ull;   // the call is over (signal_ready)
  if (warp == 0) {
    const int n = join_owners(W, ctas, owner, recs);
    if (lane == 0) n_owner = n;
  }
  __syncthreads();
  float o[D];
  if (single) {
    // A warp takes a (sequence, head); where there are fewer of those than CTAs, a CTA does, its warps taking
    // the pieces in turn.
    const int tasks = n_owner * heads;
    const bool by_cta = tasks <= n_singles;
    for (int task = by_cta ? blockIdx.x : blockIdx.x * kWarps + warp; task < tasks; task += by_cta ? n_singles : n_singles * kWarps) {
      const int b = owner[task / heads], h = task % heads;
      const Fp8Rec rec = recs[task / heads];
      const int t = __ldg(P.cu_q_lens + rec.r);
      join_row<A>(W, kSingleRows, b, rec.n, h, by_cta ? warp : 0, by_cta ? kWarps : 1, o);
      if (by_cta) {
#pragma unroll
        for (int d = 0; d < D; ++d) red[warp][lane * D + d] = o[d];
        __syncthreads();
        if (warp == 0) {
#pragma unroll
          for (int d = 0; d < D; ++d) {
            o[d] = 0.f;
            for (int w = 0; w < kWarps; ++w) o[d] += red[w][lane * D + d];
          }
        }
      }
      if (!by_cta || warp == 0) store_row<A>(P.out + ((size_t)t * P.n_q_heads + (size_t)rec.hg * heads + h) * A + lane * D, o);
      if (by_cta) __syncthreads();
    }
    return;
  }
  // 32 rows of a chunk's item at a time: a lane per row, A / 8 dimensions per warp
  constexpr int V = A / 32;                  // float4 columns per warp
  const int group = P.n_q_heads / P.cache.n_kv_heads, tok = kTileM / group;
  for (int task = blockIdx.x - n_singles; task < n_owner * (kChunkRows / 32); task += gridDim.x - n_singles) {
    const int b = owner[task / (kChunkRows / 32)];
    const Fp8Rec rec = recs[task / (kChunkRows / 32)];
    const int row = (task % (kChunkRows / 32)) * 32 + lane, n = rec.n;
    auto piece = [&](int i) { return (size_t)(i == 0 ? 2 * b + 1 : 2 * (b + i)); };
    auto ml = [&](int i) { return *reinterpret_cast<const float2*>(W.ml + (piece(i) * kChunkRows + row) * 2); };
    float M = -__int_as_float(0x7f800000), L = 0.f;
#pragma unroll 4
    for (int i = 0; i < n; ++i) M = fmaxf(M, ml(i).x);
    float4 y[V];
#pragma unroll
    for (int v = 0; v < V; ++v) y[v] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
      const float2 x = ml(i);
      const float f = x.x == -__int_as_float(0x7f800000) ? x.y : x.y * ex2(x.x - M);
      L += f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float4 a = reinterpret_cast<const float4*>(W.acc)[(piece(i) * (A / 4) + warp * V + v) * kChunkRows + row];
        y[v].x += f * a.x, y[v].y += f * a.y, y[v].z += f * a.z, y[v].w += f * a.w;
      }
    }
    const int q0 = __ldg(P.cu_q_lens + rec.r), q_len = __ldg(P.cu_q_lens + rec.r + 1) - q0;
    const int ti = rec.pad * 2 * tok + row / group;            // rows of tile B follow tile A's: its tokens do too
    if (ti >= q_len) continue;
    uint16_t* dst = P.out + ((size_t)(q0 + ti) * P.n_q_heads + (size_t)rec.hg * group + row % group) * A + warp * (A / 8);
#pragma unroll
    for (int v = 0; v < V; v += 2)
      *reinterpret_cast<uint4*>(dst + 4 * v) = make_uint4(pack_bf16(y[v].x / L, y[v].y / L), pack_bf16(y[v].z / L, y[v].w / L),
                                                          pack_bf16(y[v + 1].x / L, y[v + 1].y / L), pack_bf16(y[v + 1].z / L, y[v + 1].w / L));
  }
}

}  // namespace

cudaError_t launch_join_fp8(const Fp8Step& s, const Fp8Partials& singles, int heads, const Fp8Partials* chunks, int grid, cudaStream_t stream) {
  const int n = 4 * grid, ctas = chunks ? 2 * n : n;
  return s.cache.head_dim == 128
             ? launch_after(true, join_fp8_kernel<128>, ctas, kJoinThreads, 0, stream, s, singles, chunks ? *chunks : singles, grid, n, heads)
             : launch_after(true, join_fp8_kernel<64>, ctas, kJoinThreads, 0, stream, s, singles, chunks ? *chunks : singles, grid, n, heads);
}

}  // namespace cb
