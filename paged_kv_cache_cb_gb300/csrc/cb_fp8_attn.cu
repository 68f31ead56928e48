// Attention over the 8-bit KV cache: one CTA per (token, KV head).
#include "cb_fp8.cuh"

namespace cb {

namespace {

constexpr float kNegInf = -__builtin_inff();
constexpr int kWarps = 4;

// CTA (token t, KV head g, heads h0 .. h0+GS-1 of its group): warps take the
// visible keys in turn, lane = A / 32 dimensions, running max and sum per head
// in base 2; the four warps' (m, l, o) are joined in shared memory.
template <int A, int GS>
__global__ void __launch_bounds__(32 * kWarps) attention_fp8_simple(const Fp8Step P, int group, bool singles) {
  constexpr int D = A / 32;
  __shared__ float sm[kWarps][GS], sl[kWarps][GS], so[kWarps][GS][A];
  const int t = blockIdx.x, g = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int Hq = P.n_q_heads, Hkv = P.cache.n_kv_heads;
  if (t >= __ldg(P.cu_q_lens + P.n_reqs)) return;
  int lo = 0, hi = P.n_reqs - 1;                 // the last request that starts at or before t
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(P.cu_q_lens + mid) <= t)
      lo = mid;
    else
      hi = mid - 1;
  }
  const int r = lo, q0 = __ldg(P.cu_q_lens + r), q_len = __ldg(P.cu_q_lens + r + 1) - q0, ctx = __ldg(P.ctx_lens + r);
  if (q_len == 1 && !singles) return;
  if (ctx < 0 || q0 < 0 || t - q0 >= q_len || q_len > P.max_q_len || (long long)ctx + q_len > P.max_kv_len ||
      ((long long)ctx + q_len + kBlockSize - 1) / kBlockSize > P.max_blocks_per_seq) {
    if (threadIdx.x == 0) set_error(P.err, CB_DEVERR_BADLEN);
    return;
  }
  const int pos = ctx + t - q0, first = P.window > 0 ? max(0, pos - P.window + 1) : 0;
  const int h0 = g * group + blockIdx.z * GS;
  float q[GS][D], o[GS][D], m[GS], l[GS];
#pragma unroll
  for (int i = 0; i < GS; ++i) {
    m[i] = kNegInf;
    l[i] = 0.f;
#pragma unroll
    for (int d = 0; d < D; ++d) {
      q[i][d] = __uint_as_float((uint32_t)P.q[((size_t)t * Hq + h0 + i) * A + lane * D + d] << 16);
      o[i][d] = 0.f;
    }
  }
  for (int key = first + warp; key <= pos; key += kWarps) {
    const int blk = __ldg(P.block_tables + (size_t)r * P.max_blocks_per_seq + key / kBlockSize);
    if (blk < 0 || blk >= P.cache.num_blocks) {
      set_error(P.err, CB_DEVERR_BADBLOCK);
      continue;
    }
    const size_t row = ((size_t)blk * Hkv + g) * kBlockSize + key % kBlockSize;
    const float ks = exp_scale(P.cache.k_exps[row]), vs = exp_scale(P.cache.v_exps[row]);
    float k[D], v[D];
#pragma unroll
    for (int d = 0; d < D; d += 2) {
      e4m3_to_f32(*reinterpret_cast<const uint16_t*>(P.cache.k + row * A + lane * D + d), k[d], k[d + 1]);
      e4m3_to_f32(*reinterpret_cast<const uint16_t*>(P.cache.v + row * A + lane * D + d), v[d], v[d + 1]);
    }
#pragma unroll
    for (int i = 0; i < GS; ++i) {
      float s = 0.f;
#pragma unroll
      for (int d = 0; d < D; ++d) s += q[i][d] * k[d];
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
      s *= ks * P.scale_log2;
      const float mn = fmaxf(m[i], s), a = m[i] == mn ? 1.f : ex2(m[i] - mn), p = ex2(s - mn);
      m[i] = mn;
      l[i] = l[i] * a + p;
#pragma unroll
      for (int d = 0; d < D; ++d) o[i][d] = o[i][d] * a + p * (v[d] * vs);
    }
  }
#pragma unroll
  for (int i = 0; i < GS; ++i) {
    if (lane == 0) {
      sm[warp][i] = m[i];
      sl[warp][i] = l[i];
    }
#pragma unroll
    for (int d = 0; d < D; ++d) so[warp][i][lane * D + d] = o[i][d];
  }
  __syncthreads();
  for (int x = threadIdx.x; x < GS * A; x += 32 * kWarps) {
    const int i = x / A, d = x % A;
    float M = kNegInf, L = 0.f, O = 0.f;
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm[w][i]);
    for (int w = 0; w < kWarps; ++w) {
      if (sl[w][i] == 0.f) continue;             // a warp that saw no key
      const float f = ex2(sm[w][i] - M);
      L += f * sl[w][i];
      O += f * so[w][i][d];
    }
    P.out[((size_t)t * Hq + h0 + i) * A + d] = __bfloat16_as_ushort(__float2bfloat16_rn(O / L));
  }
}

}  // namespace

cudaError_t launch_attention_fp8_simple(const Fp8Step& s, bool singles, cudaStream_t stream) {
  const int group = s.n_q_heads / s.cache.n_kv_heads;
#define CB_SIMPLE(A_, GS_)                                                                                       \
  if (s.cache.head_dim == A_ && (group == GS_ || (GS_ == 8 && group > 8))) {                                     \
    attention_fp8_simple<A_, GS_>                                                                                \
        <<<dim3(s.n_tokens, s.cache.n_kv_heads, group / GS_), 32 * kWarps, 0, stream>>>(s, group, singles);      \
    return cudaGetLastError();                                                                                   \
  }
  CB_SIMPLE(128, 1)
  CB_SIMPLE(128, 2)
  CB_SIMPLE(128, 4)
  CB_SIMPLE(128, 8)
  CB_SIMPLE(64, 1)
  CB_SIMPLE(64, 2)
  CB_SIMPLE(64, 4)
  CB_SIMPLE(64, 8)
#undef CB_SIMPLE
  return cudaErrorInvalidValue;
}

}  // namespace cb
