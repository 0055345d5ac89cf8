// lq_rows.cu -- lq_quant_i8 and lq_norm_residual: one pass over the rows of an activation.
//
// A row of the residual stream, its norms, its whitening T and its int8 codes need three or more
// reductions over the same K entries (sum of squares, mean, largest magnitude). One CTA takes one
// row and keeps it in registers as fp32 between them, so each input is read once and each output
// written once; the reductions are warp shuffles and one shared-memory exchange each. A thread
// holds NV vectors of eight consecutive entries, vector j of thread i at column
// 8 * (j * threads + i): a warp's 32 vectors are 256 consecutive entries, so a Hadamard block of
// up to 256 inputs runs in one warp's registers and shuffles.
//
// What bounds it: HBM for many rows (bytes per entry: h + r + r_out + n or the codes), the latency
// of load -> reductions -> store for a few.
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "lq_device.cuh"

namespace lq {
namespace rows {

struct NormArgs {
  int kind;        // 0: none, else an lq_norm_kind
  float eps;
  const void* w;   // [K] or nullptr
  const void* b;   // [K] or nullptr
  int dt;
};

struct RowArgs {
  const void* h;
  const void* r;          // or nullptr
  void* r_out;            // or nullptr
  void* n_out;            // or nullptr
  int8_t* q;              // or nullptr
  float* q_scale;
  void* values;           // or nullptr
  const void* gate;       // or nullptr
  int64_t ldh, ldr, ldro, ldq;
  int hdt, rdt, ndt, vdt, gdt;
  int K, gate_cols, gate_tokens;
  float branch, resid;
  NormArgs post, pre;
  Whiten T;
};

struct F32 { static constexpr int dt = LQ_F32; };
struct F16 { static constexpr int dt = LQ_F16; };
struct BF16 { static constexpr int dt = LQ_BF16; };

// 16 bytes that are read once: not kept in L1, where the norms' weights live
__device__ __forceinline__ uint4 ld_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

__device__ __forceinline__ void unpack2(uint32_t w, int dt, float& lo, float& hi) {
  if (dt == LQ_BF16) {
    lo = __uint_as_float(w << 16);
    hi = __uint_as_float(w & 0xffff0000u);
  } else {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
    lo = f.x;
    hi = f.y;
  }
}

__device__ __forceinline__ void unpack8(const uint4& a, const uint4& b, int dt, float (&v)[8]) {
  if (dt == LQ_F32) {
    v[0] = __uint_as_float(a.x); v[1] = __uint_as_float(a.y);
    v[2] = __uint_as_float(a.z); v[3] = __uint_as_float(a.w);
    v[4] = __uint_as_float(b.x); v[5] = __uint_as_float(b.y);
    v[6] = __uint_as_float(b.z); v[7] = __uint_as_float(b.w);
  } else {
    unpack2(a.x, dt, v[0], v[1]);
    unpack2(a.y, dt, v[2], v[3]);
    unpack2(a.z, dt, v[4], v[5]);
    unpack2(a.w, dt, v[6], v[7]);
  }
}

// entries [c, c + 8) of a vector that every row reads (a norm's weight, a gate), as fp32
template <bool VEC>
__device__ __forceinline__ void load_shared8(const void* p, int dt, int64_t c, int n,
                                             float (&v)[8]) {
  if (VEC) {
    const uint4* s = reinterpret_cast<const uint4*>(static_cast<const char*>(p) +
                                                    c * (dt == LQ_F32 ? 4 : 2));
    const uint4 a = __ldg(s);
    const uint4 b = dt == LQ_F32 ? __ldg(s + 1) : a;
    unpack8(a, b, dt, v);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = e < n ? load_as_f32(p, dt, c + e) : 0.f;
  }
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi, int dt) {
  if (dt == LQ_BF16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// entries [i, i + n) of an output, each rounded once
template <bool VEC>
__device__ __forceinline__ void store8(void* p, int dt, int64_t i, int n, const float (&v)[8]) {
  if (VEC) {
    uint4* d = reinterpret_cast<uint4*>(static_cast<char*>(p) + i * (dt == LQ_F32 ? 4 : 2));
    if (dt == LQ_F32) {
      d[0] = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                        __float_as_uint(v[3]));
      d[1] = make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]),
                        __float_as_uint(v[7]));
    } else {
      d[0] = make_uint4(pack2(v[0], v[1], dt), pack2(v[2], v[3], dt), pack2(v[4], v[5], dt),
                        pack2(v[6], v[7], dt));
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < n) {
        if (dt == LQ_F32) static_cast<float*>(p)[i + e] = v[e];
        else if (dt == LQ_F16) static_cast<__half*>(p)[i + e] = __float2half_rn(v[e]);
        else static_cast<__nv_bfloat16*>(p)[i + e] = __float2bfloat16_rn(v[e]);
      }
  }
}

// Sum over the CTA; `red` holds 32 words and is not the one of the reduction before.
__device__ __forceinline__ float cta_sum(float x, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  if (blockDim.x == 32) return x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) red[warp] = x;
  __syncthreads();
  x = lane < (int)(blockDim.x >> 5) ? red[lane] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

__device__ __forceinline__ uint32_t cta_max(uint32_t x, float* red) {
  x = __reduce_max_sync(0xffffffffu, x);
  if (blockDim.x == 32) return x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) red[warp] = __uint_as_float(x);
  __syncthreads();
  x = lane < (int)(blockDim.x >> 5) ? __float_as_uint(red[lane]) : 0u;
  return __reduce_max_sync(0xffffffffu, x);
}

// v = norm(v), in place. Entries past K are zero before and after.
template <int NV, bool VEC>
__device__ __forceinline__ void apply_norm(float (&v)[NV][8], const NormArgs& p, int K,
                                           float* red0, float* red1) {
  const float inv_k = 1.f / (float)K;
  if (p.kind == LQ_NORM_LAYER) {
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e) s += v[j][e];
    const float mean = cta_sum(s, red1) * inv_k;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int n = K - 8 * (int)(j * blockDim.x + threadIdx.x);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < n) v[j][e] -= mean;
    }
  }
  float ss = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(v[j][e], v[j][e], ss);
  const float rs = 1.f / sqrtf(fmaf(cta_sum(ss, red0), inv_k, p.eps));
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = 8 * (j * blockDim.x + threadIdx.x);
    if (c >= K) continue;
    float w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[j][e] *= rs;
    if (p.w) {
      load_shared8<VEC>(p.w, p.dt, c, K - c, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[j][e] *= w[e];
    }
    if (p.b) {
      load_shared8<VEC>(p.b, p.dt, c, K - c, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[j][e] += w[e];
    }
  }
}

// v = T(v): sign and channel scale, then butterflies over distance 1, 2, 4 in a thread's vector,
// 8 .. 128 across the warp's lanes, 256 and up through shared memory (ex: 8 * threads floats).
template <int NV, bool VEC>
__device__ __forceinline__ void apply_whiten(float (&v)[NV][8], const Whiten& T, int K, float* ex) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = 8 * (j * blockDim.x + threadIdx.x);
    const int n = K - c;
    if (n > 0) {
      if (T.chan_scale) {
        float cs[8];
        load_shared8<VEC>(T.chan_scale, LQ_F32, c, n, cs);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[j][e] *= cs[e];
      }
      if (T.sign) {
        uint32_t lo, hi;
        if (VEC) {
          const uint2 s = __ldg(reinterpret_cast<const uint2*>(T.sign + c));
          lo = s.x;
          hi = s.y;
        } else {
          lo = hi = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (e < n) lo |= (uint32_t)(uint8_t)T.sign[c + e] << (8 * e);
            if (e + 4 < n) hi |= (uint32_t)(uint8_t)T.sign[c + e + 4] << (8 * e);
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          // the sign bit of byte e
          v[j][e] = __uint_as_float(__float_as_uint(v[j][e]) ^ ((lo << (24 - 8 * e)) & 0x80000000u));
          v[j][e + 4] =
              __uint_as_float(__float_as_uint(v[j][e + 4]) ^ ((hi << (24 - 8 * e)) & 0x80000000u));
        }
      }
    }
#pragma unroll
    for (int h = 1; h < 8; h <<= 1)
      if (h < T.block)
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if ((e & h) == 0) {
            const float a = v[j][e], b = v[j][e + h];
            v[j][e] = a + b;
            v[j][e + h] = a - b;
          }
    for (int m = 1; m < 32 && 8 * m < T.block; m <<= 1) {
      const bool upper = (lane & m) != 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float o = __shfl_xor_sync(0xffffffffu, v[j][e], m);
        v[j][e] = upper ? o - v[j][e] : v[j][e] + o;
      }
    }
    // the vectors j of the CTA's threads are 8 * threads consecutive entries, a whole number of
    // blocks
    for (int m = 32; 8 * m < T.block; m <<= 1) {
      __syncthreads();
#pragma unroll
      for (int e = 0; e < 8; ++e) ex[e * blockDim.x + threadIdx.x] = v[j][e];
      __syncthreads();
      const bool upper = (threadIdx.x & m) != 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float o = ex[e * blockDim.x + (threadIdx.x ^ m)];
        v[j][e] = upper ? o - v[j][e] : v[j][e] + o;
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) v[j][e] *= T.inv_sqrt;
  }
}

// Exact rounding of 127 u / a for u >= 0 next to a border m + 1/2 (m = floor): the sign of
// 2 * 127 u - (2m + 1) a, which the two fmas give without a rounding (the first product's error
// is kept; the difference is a small multiple of half an ulp of a).
__device__ __forceinline__ float border_code(float u, float a, float m) {
  const float hi = 127.f * u, lo = fmaf(127.f, u, -hi);
  const float d = fmaf(-(2.f * m + 1.f), a, 2.f * hi) + 2.f * lo;
  const bool odd = ((int)m & 1) != 0;
  return d > 0.f || (d == 0.f && odd) ? m + 1.f : m;
}

// Codes of eight entries: bytes lo (entries 0..3) and hi (4..7). t = v * (127 / a) is off by at
// most 127 * 2^-23 from the quotient, so rounding it is right unless it lies within 1e-4 of a
// border; there border_code decides.
__device__ __forceinline__ void codes8(const float (&v)[8], float inv, float a, uint32_t& lo,
                                       uint32_t& hi) {
  constexpr float kRound = 12582912.f;   // 1.5 * 2^23: adding it rounds half to even
  uint32_t b[8];
  float worst = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float t = v[e] * inv;
    const float m = t + kRound;
    b[e] = __float_as_uint(m);           // low byte: the code
    worst = fmaxf(worst, fabsf(t - (m - kRound)));
  }
  if (worst > 0.4999f) {
#pragma unroll 1
    for (int e = 0; e < 8; ++e) {
      float ve = v[0];
#pragma unroll
      for (int i = 1; i < 8; ++i) ve = e == i ? v[i] : ve;
      const float t = fabsf(ve * inv), m = floorf(t);
      if (fabsf(t - m - 0.5f) < 1.1e-4f) {
        const float c = copysignf(border_code(fabsf(ve), a, m), ve);
#pragma unroll
        for (int i = 0; i < 8; ++i) b[i] = e == i ? (uint32_t)(int)c : b[i];
      }
    }
  }
  lo = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
  hi = __byte_perm(__byte_perm(b[4], b[5], 0x0040), __byte_perm(b[6], b[7], 0x0040), 0x5410);
}

template <class HT, class RT, int NV, bool VEC, int kMaxThreads>
__global__ void __launch_bounds__(kMaxThreads, 1) row_kernel(const __grid_constant__ RowArgs a) {
  extern __shared__ __align__(16) float ex[];   // whitening blocks over 256
  __shared__ float red[4][32];
  const int K = a.K, tid = threadIdx.x, T = blockDim.x;
  const int64_t row = blockIdx.x;
  const int hdt = VEC ? HT::dt : a.hdt, rdt = VEC ? RT::dt : a.rdt;
  float v[NV][8];

  if (VEC) {
    uint4 hr[NV][HT::dt == LQ_F32 ? 2 : 1];
    const char* hp = static_cast<const char*>(a.h) + row * a.ldh * (HT::dt == LQ_F32 ? 4 : 2);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = 8 * (j * T + tid);
      if (c < K) {
        hr[j][0] = ld_stream(hp + (int64_t)c * (HT::dt == LQ_F32 ? 4 : 2));
        if (HT::dt == LQ_F32) hr[j][HT::dt == LQ_F32 ? 1 : 0] = ld_stream(hp + (int64_t)c * 4 + 16);
      } else {
        hr[j][0] = make_uint4(0u, 0u, 0u, 0u);
        if (HT::dt == LQ_F32) hr[j][HT::dt == LQ_F32 ? 1 : 0] = make_uint4(0u, 0u, 0u, 0u);
      }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) unpack8(hr[j][0], hr[j][HT::dt == LQ_F32 ? 1 : 0], HT::dt, v[j]);
  } else {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = 8 * (j * T + tid);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        v[j][e] = c + e < K ? load_as_f32(a.h, hdt, row * a.ldh + c + e) : 0.f;
    }
  }

  if (a.post.kind) apply_norm<NV, VEC>(v, a.post, K, red[0], red[1]);

  if (a.gate) {
    const int64_t g = (row / a.gate_tokens) * a.gate_cols;
    if (a.gate_cols == K && K > 1) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = 8 * (j * T + tid);
        if (c >= K) continue;
        float w[8];
        load_shared8<VEC>(a.gate, a.gdt, g + c, K - c, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[j][e] *= w[e];
      }
    } else {
      const float w = load_as_f32(a.gate, a.gdt, g);
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) v[j][e] *= w;
    }
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = 8 * (j * T + tid);
    if (c >= K) continue;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[j][e] *= a.branch;
    if (a.r) {
      float w[8];
      if (VEC) {
        const char* rp = static_cast<const char*>(a.r) +
                         (row * a.ldr + c) * (RT::dt == LQ_F32 ? 4 : 2);
        const uint4 r0 = ld_stream(rp);
        unpack8(r0, RT::dt == LQ_F32 ? ld_stream(rp + 16) : r0, RT::dt, w);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          w[e] = c + e < K ? load_as_f32(a.r, rdt, row * a.ldr + c + e) : 0.f;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) v[j][e] = fmaf(a.resid, w[e], v[j][e]);
    }
    if (a.r_out) store8<VEC>(a.r_out, rdt, row * a.ldro + c, K - c, v[j]);
  }

  if (a.pre.kind) apply_norm<NV, VEC>(v, a.pre, K, red[2], red[3]);
  if (a.n_out) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = 8 * (j * T + tid);
      if (c < K) store8<VEC>(a.n_out, a.ndt, row * K + c, K - c, v[j]);
    }
  }
  if (!a.q) return;

  if (a.T.block) apply_whiten<NV, VEC>(v, a.T, K, ex);
  // largest magnitude as bits: they order like the values, with infinity and the NaNs on top
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(v[j][e]) & 0x7fffffffu);
  top = cta_max(top, red[1]);
  const bool finite = top < 0x7f800000u;
  const float amax = __uint_as_float(top);
  if (tid == 0) a.q_scale[row] = finite ? amax / 127.f : __uint_as_float(0x7fffffffu);
  // 127 v and 127 / a must neither overflow nor lose bits: rows of extreme magnitude are moved
  // by a power of two (exact for every entry that can differ from code 0)
  float shift = 1.f;
  const int ex_bits = (int)(top >> 23);
  if (ex_bits < 16 || ex_bits > 240)
    shift = __uint_as_float((uint32_t)max(1, min(253, 254 - ex_bits)) << 23);
  const float as = amax * shift;
  const float inv = finite && amax > 0.f ? 127.f / as : 0.f;
  int8_t* qrow = a.q + row * a.ldq;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = 8 * (j * T + tid);
    if (c >= (int)a.ldq) continue;
    uint32_t lo = 0, hi = 0;
    if (inv != 0.f) {
      if (shift != 1.f)
#pragma unroll
        for (int e = 0; e < 8; ++e) v[j][e] *= shift;
      codes8(v[j], inv, as, lo, hi);
    }
    *reinterpret_cast<uint2*>(qrow + c) = make_uint2(lo, hi);
    if (a.values && c < K) {
      const float s = finite ? amax / 127.f : __uint_as_float(0x7fffffffu);
      float o[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        o[e] = s * (float)(int8_t)(lo >> (8 * e));
        o[e + 4] = s * (float)(int8_t)(hi >> (8 * e));
      }
      store8<VEC>(a.values, a.vdt, row * K + c, K - c, o);
    }
  }
}

template <class HT, class RT, bool VEC>
cudaError_t launch_typed(const RowArgs& a, int rows, int threads, int nv, size_t smem,
                         cudaStream_t st) {
  if (nv == 1) row_kernel<HT, RT, 1, VEC, 1024><<<rows, threads, smem, st>>>(a);
  else if (nv == 4) row_kernel<HT, RT, 4, VEC, 512><<<rows, threads, smem, st>>>(a);
  else if (threads <= 512) row_kernel<HT, RT, 8, VEC, 512><<<rows, threads, smem, st>>>(a);
  else row_kernel<HT, RT, 8, VEC, 1024><<<rows, threads, smem, st>>>(a);
  return cudaGetLastError();
}

template <class HT>
cudaError_t launch_h(const RowArgs& a, int rows, int threads, int nv, size_t smem,
                     cudaStream_t st) {
  const int rdt = a.r || a.r_out ? a.rdt : HT::dt;
  if (rdt == LQ_F32) return launch_typed<HT, F32, true>(a, rows, threads, nv, smem, st);
  if (rdt == LQ_F16) return launch_typed<HT, F16, true>(a, rows, threads, nv, smem, st);
  return launch_typed<HT, BF16, true>(a, rows, threads, nv, smem, st);
}

bool al(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
size_t width(int dt) { return dt == LQ_F32 ? 4 : 2; }
bool known(int dt) { return dt == LQ_F32 || dt == LQ_F16 || dt == LQ_BF16; }

// 16-byte loads and stores everywhere: K a multiple of 8 and every pointer and stride aligned
bool vectors_ok(const RowArgs& a) {
  if (a.K % 8 != 0 || !al(a.h, 16) || a.ldh * width(a.hdt) % 16 != 0) return false;
  if (a.r && (!al(a.r, 16) || a.ldr * width(a.rdt) % 16 != 0)) return false;
  if (a.r_out && (!al(a.r_out, 16) || a.ldro * width(a.rdt) % 16 != 0)) return false;
  if (!al(a.n_out, 16) || !al(a.values, 16) || !al(a.gate, 16)) return false;
  for (const NormArgs* p : {&a.post, &a.pre})
    if (p->kind && (!al(p->w, 16) || !al(p->b, 16))) return false;
  return !a.q || !a.T.block || (al(a.T.sign, 8) && al(a.T.chan_scale, 16));
}

cudaError_t launch_rows(const RowArgs& a, int rows, cudaStream_t st) {
  const int vecs = (a.K + 7) / 8;
  // One vector per thread while the rows do not fill the GPU (a few CTAs per SM): the latency of
  // a row is what counts. Else four per thread, so that a CTA is small and several rows are in
  // flight per SM.
  int nv = rows <= 2 * 148 && vecs <= 1024 ? 1 : vecs <= 4 * 512 ? 4 : 8;
  int threads = std::max(32, ((vecs + nv - 1) / nv + 31) / 32 * 32);
  size_t smem = 0;
  if (a.q && a.T.block > 256) {   // a slab of 8 * threads entries holds whole blocks
    const int unit = a.T.block / 8;
    threads = (threads + unit - 1) / unit * unit;
    smem = (size_t)threads * 8 * sizeof(float);
  }
  if (!vectors_ok(a)) return launch_typed<F32, F32, false>(a, rows, threads, nv, smem, st);
  if (a.hdt == LQ_F32) return launch_h<F32>(a, rows, threads, nv, smem, st);
  if (a.hdt == LQ_F16) return launch_h<F16>(a, rows, threads, nv, smem, st);
  return launch_h<BF16>(a, rows, threads, nv, smem, st);
}

thread_local char g_err[512];

lq_status reject(lq_status st, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_err, sizeof(g_err), fmt, ap);
  va_end(ap);
  set_last_error("%s", g_err);
  return st;
}

lq_status check_norm(const lq_norm_desc* d, const char* which, NormArgs* out) {
  out->kind = 0;
  out->eps = 0.f;
  out->w = out->b = nullptr;
  out->dt = LQ_F32;
  if (!d) return LQ_OK;
  if (d->kind != LQ_NORM_RMS && d->kind != LQ_NORM_LAYER)
    return reject(LQ_EINVAL, "%s: unknown norm kind %d", which, (int)d->kind);
  if (!(d->eps >= 0.f) || !std::isfinite(d->eps))
    return reject(LQ_EINVAL, "%s: eps is negative or not finite", which);
  if ((d->weight || d->bias) && !known(d->dtype))
    return reject(LQ_EINVAL, "%s: unknown dtype %d", which, (int)d->dtype);
  out->kind = d->kind;
  out->eps = d->eps;
  out->w = d->weight;
  out->b = d->bias;
  out->dt = known(d->dtype) ? d->dtype : LQ_F32;
  if (!al(out->w, width(out->dt)) || !al(out->b, width(out->dt)))
    return reject(LQ_EINVAL, "%s: misaligned weight or bias", which);
  return LQ_OK;
}

lq_status check_row(int32_t rows, int32_t K, const char* where) {
  if (rows < 0) return reject(LQ_EINVAL, "%s: rows = %d < 0", where, rows);
  if (K < 1) return reject(LQ_EINVAL, "%s: K = %d < 1", where, K);
  if (K > LQ_MAX_ROW)
    return reject(LQ_EUNSUPPORTED, "%s: K = %d exceeds LQ_MAX_ROW (%d)", where, K, LQ_MAX_ROW);
  return LQ_OK;
}

}  // namespace rows
}  // namespace lq

extern "C" {

int64_t lq_i8_row_bytes(int32_t K) { return K < 1 ? -1 : ((int64_t)K + 15) / 16 * 16; }

lq_status lq_quant_i8(const void* x, lq_dtype xdt, int32_t rows, int32_t K, int64_t ldx,
                      const lq_whiten_desc* T, int8_t* q, float* scale, void* values,
                      lq_stream stream) {
  using namespace lq::rows;
  lq::set_last_error("%s", "");
  lq_status st = check_row(rows, K, "lq_quant_i8");
  if (st != LQ_OK) return st;
  if (!known(xdt)) return reject(LQ_EINVAL, "lq_quant_i8: unknown x dtype %d", (int)xdt);
  if (rows == 0) return LQ_OK;
  if (!x || !q || !scale) return reject(LQ_EINVAL, "lq_quant_i8: null pointer");
  if (ldx < K) return reject(LQ_EINVAL, "lq_quant_i8: ldx = %lld < K = %d", (long long)ldx, K);
  if (!al(x, width(xdt)) || !al(q, 16) || !al(scale, 4) || (values && !al(values, width(xdt))))
    return reject(LQ_EINVAL, "lq_quant_i8: misaligned x, q, scale or values");
  RowArgs a{};
  st = lq::whiten_from_desc(T, K, &a.T);
  if (st != LQ_OK) return st;
  a.h = x;
  a.hdt = a.vdt = xdt;
  a.ldh = ldx;
  a.K = K;
  a.branch = 1.f;
  a.q = q;
  a.q_scale = scale;
  a.values = values;
  a.ldq = lq_i8_row_bytes(K);
  const cudaError_t e = launch_rows(a, rows, (cudaStream_t)stream);
  return e == cudaSuccess ? LQ_OK : reject(LQ_ECUDA, "lq_quant_i8: %s", cudaGetErrorString(e));
}

lq_status lq_norm_residual(const void* h, lq_dtype hdt, int64_t ldh, const void* r, lq_dtype rdt,
                           int64_t ldr, int32_t rows, int32_t K, const lq_norm_desc* post,
                           const lq_gate_desc* gate, float branch_scale, float residual_scale,
                           void* r_out, const lq_norm_desc* pre, void* n_out, lq_dtype ndt,
                           const lq_whiten_desc* T, int8_t* q, float* q_scale, lq_stream stream) {
  using namespace lq::rows;
  const char* me = "lq_norm_residual";
  lq::set_last_error("%s", "");
  lq_status st = check_row(rows, K, me);
  if (st != LQ_OK) return st;
  if (!known(hdt)) return reject(LQ_EINVAL, "%s: unknown h dtype %d", me, (int)hdt);
  if ((r || r_out) && !known(rdt)) return reject(LQ_EINVAL, "%s: unknown r dtype %d", me, (int)rdt);
  if (n_out && !known(ndt)) return reject(LQ_EINVAL, "%s: unknown n dtype %d", me, (int)ndt);
  RowArgs a{};
  if ((st = check_norm(post, "lq_norm_residual: post", &a.post)) != LQ_OK) return st;
  if ((st = check_norm(pre, "lq_norm_residual: pre", &a.pre)) != LQ_OK) return st;
  if ((q == nullptr) != (q_scale == nullptr))
    return reject(LQ_EINVAL, "%s: q and q_scale go together", me);
  if (q && (st = lq::whiten_from_desc(T, K, &a.T)) != LQ_OK) return st;
  if (gate) {
    if (!known(gate->dtype)) return reject(LQ_EINVAL, "%s: unknown gate dtype %d", me, (int)gate->dtype);
    if (gate->cols != 1 && gate->cols != K)
      return reject(LQ_EINVAL, "%s: gate cols = %d, neither 1 nor K = %d", me, gate->cols, K);
    if (gate->tokens < 1) return reject(LQ_EINVAL, "%s: gate tokens = %d < 1", me, gate->tokens);
  }
  if (rows == 0) return LQ_OK;
  if (!r_out && !n_out && !q) return reject(LQ_EINVAL, "%s: no output", me);
  if (!h || (gate && !gate->gate)) return reject(LQ_EINVAL, "%s: null pointer", me);
  if (ldh < K || (r && ldr < K)) return reject(LQ_EINVAL, "%s: row stride < K = %d", me, K);
  if (!al(h, width(hdt)) || ((r || r_out) && (!al(r, width(rdt)) || !al(r_out, width(rdt)))) ||
      (n_out && !al(n_out, width(ndt))) || !al(q, 16) || !al(q_scale, 4) ||
      (gate && !al(gate->gate, width(gate->dtype))))
    return reject(LQ_EINVAL, "%s: misaligned pointer", me);
  a.h = h;
  a.hdt = hdt;
  a.ldh = ldh;
  a.r = r;
  a.rdt = (r || r_out) ? rdt : LQ_F32;
  a.ldr = ldr;
  a.r_out = r_out;
  a.ldro = r_out && r_out == r ? ldr : K;
  a.K = K;
  if (gate) {
    a.gate = gate->gate;
    a.gdt = gate->dtype;
    a.gate_cols = gate->cols;
    a.gate_tokens = gate->tokens;
  }
  a.branch = branch_scale;
  a.resid = residual_scale;
  a.n_out = n_out;
  a.ndt = ndt;
  a.q = q;
  a.q_scale = q_scale;
  a.ldq = lq_i8_row_bytes(K);
  const cudaError_t e = launch_rows(a, rows, (cudaStream_t)stream);
  return e == cudaSuccess ? LQ_OK : reject(LQ_ECUDA, "%s: %s", me, cudaGetErrorString(e));
}

}  // extern "C"
