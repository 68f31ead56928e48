// The 8-bit KV cache format and its conversions.
//
// A row x (one token, one KV head, A values) is stored as A e4m3 values and one
// exponent byte b = e + 127:
//     e = the least integer >= -126 with max|x| <= 448 * 2^e     (448: e4m3's largest)
//     stored value = round_e4m3(x * 2^-e)  (nearest, ties to even; never saturates)
// and stands for value * 2^e.  A row with a NaN or an infinity is stored as
// zeros with b = 255 and stands for NaNs, so no stored value is ever a NaN
// pattern and a bad row poisons only what its own (token, KV head) reaches.
// The scale is a power of two so that reading back is exact: an e4m3 value has 4
// significant bits, and times 2^e it is a bf16 number (8 bits, the exponents of
// fp32).  A free scale would cost a second rounding there, and it gains nothing:
// e4m3's relative step does not depend on where in its range a value falls.
#pragma once
#include "cb_common.cuh"

namespace cb {

constexpr uint32_t kExpNan = 255;      // exponent byte of a row that is not finite

// Exponent byte of a row whose largest magnitude has the bf16 bits `amax` (sign
// cleared): with amax = (1 + m / 128) 2^(E - 127), 448 = 1.75 * 2^8 gives
// e = E - 127 - 8 + (m > 96).
__device__ __forceinline__ uint32_t row_exp(uint32_t amax) {
  if (amax >= 0x7F80u) return kExpNan;
  return (uint32_t)max(1, (int)(amax >> 7) - 8 + ((amax & 127u) > 96u));
}
// 2^e of an exponent byte (NaN for 255); 2^-e of a finite one (1 .. 253).
__device__ __forceinline__ float exp_scale(uint32_t b) {
  return __uint_as_float(b == kExpNan ? 0x7FC00000u : b << 23);
}
__device__ __forceinline__ float exp_inverse(uint32_t b) { return __uint_as_float((254u - b) << 23); }

// The largest finite number for an infinity, a NaN for a NaN: the factors' product may
// pass fp32's range where the score they multiply is 0.
__device__ __forceinline__ float finite(float f) {
  float r;
  asm("min.NaN.f32 %0, %1, 0f7F7FFFFF;" : "=f"(r) : "f"(f));
  return r;
}

// Two floats -> two e4m3 in the low 16 bits (first one lowest), rounded to nearest even.
__device__ __forceinline__ uint32_t pack_e4m3(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two e4m3 (low 16 bits of w) -> two halves packed in a word; exact.
__device__ __forceinline__ uint32_t e4m3_to_f16x2(uint32_t w) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)w));
  return r;
}
// What two floats have left after the e4m3 in w's low 16 bits, as two e4m3.  The
// subtraction takes the halves as they are: conversions run at a fraction of the
// arithmetic's rate.
__device__ __forceinline__ uint32_t pack_rest(uint32_t w, float lo, float hi) {
  asm("{\n\t.reg .f16 a, b, n;\n\tmov.b32 {a, b}, %2;\n\tmov.b16 n, 0xBC00;\n\tfma.rn.f32.f16 %0, a, n, %0;\n\tfma.rn.f32.f16 %1, b, n, %1;\n\t}"
      : "+f"(lo), "+f"(hi)
      : "r"(e4m3_to_f16x2(w)));
  return pack_e4m3(lo, hi);
}

// A query row of largest |bits| amax as two e4m3 terms of q 2^-e: the exponent byte e +
// 127 that brings its largest value into [128, 256), and the terms of two values (lo: of
// what hi leaves of them).  Rows that are not finite are the caller's.
__device__ __forceinline__ uint32_t query_exp(uint32_t amax) { return (uint32_t)max(1, (int)(amax >> 7) - 7); }
__device__ __forceinline__ void query_terms(float y0, float y1, uint32_t& hi, uint32_t& lo) {
  hi = pack_e4m3(y0, y1);
  lo = pack_rest(hi, y0, y1);
}

// e4m3 -> bf16 times 2^e.  Each byte is sign-extended to 16 bits and moved
// up by 4: sign, zeros, the 4 exponent and 3 fraction bits in bf16's places, a
// bf16 2^-120 times too small (also for e4m3's subnormals, which become bf16's);
// one multiplication by 2^(120 + e) is exact.  Bytes b > 134 (e > 7) need a second.
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
template <int SEL>
__device__ __forceinline__ uint32_t permute(uint32_t x) {
  uint32_t r;
  asm("prmt.b32 %0, %1, 0, %2;" : "=r"(r) : "r"(x), "n"(SEL));
  return r;
}
__device__ __forceinline__ void widen8(uint32_t lo, uint32_t hi, uint32_t f, uint32_t* o) {
  // bytes 0, 1 (then 2, 3) as two sign-extended halves: selector bit 3 repeats a byte's sign
  o[0] = mul_bf16x2((permute<0x9180>(lo) << 4) & 0x87F087F0u, f);
  o[1] = mul_bf16x2((permute<0xB3A2>(lo) << 4) & 0x87F087F0u, f);
  o[2] = mul_bf16x2((permute<0x9180>(hi) << 4) & 0x87F087F0u, f);
  o[3] = mul_bf16x2((permute<0xB3A2>(hi) << 4) & 0x87F087F0u, f);
}
// The factor of exponent byte b as a pair of bf16 (up to 2^7 of it: see above), and what is left of it.
__device__ __forceinline__ uint32_t factor1(uint32_t b) { return ((min(b, 134u) + 120u) << 7) * 0x10001u; }
__device__ __forceinline__ uint32_t factor2(uint32_t b) { return ((max(b, 134u) - 134u + 127u) << 7) * 0x10001u; }

// ---------------------------------------------------------------- shared memory
// Shared-memory accesses by address: through a generic pointer whose space the
// compiler cannot see they cost more.
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ float lds32f(uint32_t a) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=h"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void sts128(uint32_t a, const uint4& v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ void sts32(uint32_t a, uint32_t v) { asm volatile("st.shared.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory"); }
__device__ __forceinline__ void sts16(uint32_t a, uint32_t v) {
  asm volatile("st.shared.u16 [%0], %1;" ::"r"(a), "h"((uint16_t)v) : "memory");
}
__device__ __forceinline__ void sts8(uint32_t a, uint32_t v) {
  asm volatile("st.shared.u8 [%0], %1;" ::"r"(a), "h"((uint16_t)v) : "memory");
}

// ---------------------------------------------------------------- 8-bit matrix products
// One lane of the warp (the same each time).
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r;
}
// D(tmem) (+)= A(smem) B(smem), 8-bit floating point operands, fp32 accumulation.
__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Instruction descriptor, kind::f8f6f4: formats 0 = e4m3, 1 = e5m2; fp32 D.
__host__ __device__ constexpr uint32_t idesc_f8(int M, int N, int a_fmt, int b_fmt, int a_mn, int b_mn) {
  return (1u << 4) | ((uint32_t)a_fmt << 7) | ((uint32_t)b_fmt << 10) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// Shared-memory matrix descriptor; layout 0: no swizzle, 2: 128-byte, 4: 64-byte swizzle.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lbo, uint32_t sbo, int layout) {
  return (uint64_t)((addr >> 4) & 0x3FFF) | (uint64_t)((lbo >> 4) & 0x3FFF) << 16 |
         (uint64_t)((sbo >> 4) & 0x3FFF) << 32 | (uint64_t)1 << 46 | (uint64_t)layout << 61;
}
// Untiled bulk copy (16-byte aligned on both sides, a multiple of 16 bytes).
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(static_cast<uint64_t>(__cvta_generic_to_global(src))), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}
// 16-byte asynchronous copy by this thread, outside the bulk-copy unit (which takes
// about as long for 16 bytes as for 2 KB), and the arrival on `bar` once this
// thread's copies have landed (counted among the barrier's expected arrivals).
// !have: zeros; src is not read then.
__device__ __forceinline__ void cp_async16(void* dst, const void* src, bool have) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)),
               "l"(static_cast<uint64_t>(__cvta_generic_to_global(src))), "r"(have ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// ---------------------------------------------------------------- what both attention kernels use
// Bounded wait with the same outcome in all 32 lanes.
template <class S>
__device__ __forceinline__ bool wwait(const Fp8Step& P, S& sm, uint64_t* bar, uint32_t parity) {
  const bool ok = __all_sync(0xffffffffu, mbar_wait(bar, parity));
  if (!ok) {
    set_error(P.err, CB_DEVERR_TIMEOUT);
    sm.abort = 1;
  }
  return ok;
}
// The CTA whose range holds tile u (ranges [total b / eff, total (b + 1) / eff)).
__device__ __forceinline__ int cta_of(int u, int total, int eff) {
  return (int)((((long long)u + 1) * eff - 1) / total);
}

// ---------------------------------------------------------------- joining pieces
// A sequence cut between CTAs leaves per piece and row the maximum m and sum l of
// its weights and its output o (already over l); the joined row is
//     sum_i W_i o_i / sum_i W_i,   W_i = 2^(m_i - M) l_i,  M = max m_i,
// in the pieces' order.  m = -inf: no key seen (l = 0), or NaNs only (l is one).
constexpr int kJoinLoads = (kMaxDecodeGrid + 31) / 32;   // pieces per lane
// The CTAs whose records start such a sequence and those records, into owner[] and
// rec[]; their number.  One warp.
__device__ __forceinline__ int join_owners(const Fp8Partials& W, int ctas, int* owner, Fp8Rec* rec) {
  const int lane = threadIdx.x & 31;
  int4 x[kJoinLoads];
  int found = 0;
#pragma unroll
  for (int k = 0; k < kJoinLoads; ++k)
    x[k] = lane + 32 * k < ctas ? reinterpret_cast<const int4*>(W.rec)[lane + 32 * k] : make_int4(0, 0, 0, 0);
#pragma unroll
  for (int k = 0; k < kJoinLoads; ++k) {
    const unsigned mask = __ballot_sync(0xffffffffu, x[k].z > 1);
    if (x[k].z > 1) {
      const int at = found + __popc(mask & ((1u << lane) - 1));
      owner[at] = lane + 32 * k;
      rec[at] = {x[k].x, x[k].y, x[k].z, x[k].w};
    }
    found += __popc(mask);
  }
  return found;
}
// This warp's share (pieces first, first + step, ...) of the joined row `row` of
// the n pieces that start in CTA b; `rows` rows per partial result.  Lane = A / 32
// dimensions; eight pieces' loads in flight.
template <int A>
__device__ __forceinline__ void join_row(const Fp8Partials& W, int rows, int b, int n, int row, int first, int step, float (&o)[A / 32]) {
  constexpr int D = A / 32;
  const unsigned FULL = 0xffffffffu;
  const int lane = threadIdx.x & 31;
  auto piece = [&](int i) { return (size_t)(i == 0 ? 2 * b + 1 : 2 * (b + i)) * rows + row; };
  float m[kJoinLoads], w[kJoinLoads], M = -__int_as_float(0x7f800000), L = 0.f;
#pragma unroll
  for (int k = 0; k < kJoinLoads; ++k) {
    const int i = lane + 32 * k;
    const float2 ml = i < n ? *reinterpret_cast<const float2*>(W.ml + piece(i) * 2) : make_float2(-__int_as_float(0x7f800000), 0.f);
    m[k] = ml.x;
    w[k] = ml.y;
    M = fmaxf(M, ml.x);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(FULL, M, off));
#pragma unroll
  for (int k = 0; k < kJoinLoads; ++k) {
    if (m[k] != -__int_as_float(0x7f800000)) w[k] *= ex2(m[k] - M);
    L += w[k];
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) L += __shfl_xor_sync(FULL, L, off);
#pragma unroll
  for (int d = 0; d < D; ++d) o[d] = 0.f;
  for (int i0 = first; i0 < n; i0 += 8 * step) {
    float y[8][D];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int i = i0 + u * step;
      const float* src = W.acc + piece(i) * A + lane * D;
#pragma unroll
      for (int d = 0; d < D; ++d) y[u][d] = 0.f;
      if (i < n) {
        if constexpr (D == 4) {
          const float4 v = *reinterpret_cast<const float4*>(src);
          y[u][0] = v.x, y[u][1] = v.y, y[u][2] = v.z, y[u][3] = v.w;
        } else {
          const float2 v = *reinterpret_cast<const float2*>(src);
          y[u][0] = v.x, y[u][1] = v.y;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int i = i0 + u * step;                       // the same in every lane
      if (i >= n) break;
      float f = w[0];
#pragma unroll
      for (int k = 1; k < kJoinLoads; ++k) f = (i >> 5) == k ? w[k] : f;
      f = __shfl_sync(FULL, f, i & 31);
#pragma unroll
      for (int d = 0; d < D; ++d) o[d] += f * y[u][d];
    }
  }
#pragma unroll
  for (int d = 0; d < D; ++d) o[d] /= L;
}

// The warp's arrival that gives back a buffer of shared memory whose values it has
// loaded.  v: of all of the lane's loaded values.  Which lane arrives depends on
// them: an arrival that merely followed the loads was seen to let the next copy
// overwrite the buffer before they had read it.
__device__ __forceinline__ void arrive_after(uint64_t* bar, uint32_t v) {
  if ((threadIdx.x & 31) == (__ballot_sync(0xffffffffu, v != 0u) & 1u)) mbar_arrive(bar);
}

// ---------------------------------------------------------------- the kernels of a call
// Chunks run next to the single tokens' kernel, so they cannot wait for its end, and
// the rows they read were appended by the kernel before it.  That kernel, once its own
// griddepcontrol.wait has made those rows visible to it, releases the call's ticket;
// a chunk CTA that acquires the ticket has them too.  One that does not find it there
// waits for the end of the kernel before, which has them as well: nothing spins, and
// nothing rests on when the kernels start.  The joining kernel clears the word, so that
// a recorded call finds its own ticket only after its own release.  One thread each,
// before the CTA's barrier in front of its first loads; the loading warps then fence,
// because the rows were stored through another proxy than they load them by.
__device__ __forceinline__ void signal_ready(const Fp8Step& P) {
  if (P.ready) asm volatile("st.release.gpu.global.u64 [%0], %1;" ::"l"(P.ready), "l"(P.ticket) : "memory");
}
__device__ __forceinline__ void await_ready(const Fp8Step& P) {
  unsigned long long t;
  asm volatile("ld.acquire.gpu.global.u64 %0, [%1];" : "=l"(t) : "l"(P.ready) : "memory");
  if (t != P.ticket) asm volatile("griddepcontrol.wait;" ::: "memory");
}

// A kernel launch.  chained: the kernel may be placed while the kernel before it on
// the stream, one of the same call, still runs.  Until its griddepcontrol.wait (the
// chunks': await_ready) it reads only what no kernel of the call writes, the requests'
// lengths, and writes nothing to global memory but error flags.  The chunks' kernel
// then writes its rows of out and its part of the workspace, which the single tokens'
// kernel does not touch.  The first kernel of a call is not chained: what stands before
// it on the stream may write those lengths.
template <class... T, class... U>
cudaError_t launch_after(bool chained, void (*kernel)(T...), int grid, int threads, size_t smem, cudaStream_t stream, const U&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = chained ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace cb
