// lq_rows.cu -- lq_quant_i8 and lq_norm_residual: one pass over the rows of an activation.
//
// A row of the residual stream, its norms, its whitening T and its int8 codes need up to five
// reductions over the same K entries (sums, sums of squares, largest magnitude). A row stays in
// registers as fp32 between them, so each input is read once and each output written once. One CTA
// takes a row of up to 8192 entries, a cluster of up to eight CTAs a longer one; a reduction is
// warp shuffles and one exchange through the (cluster's) shared memory.
//
// A thread holds NV vectors of eight consecutive entries; vectors j of a warp's threads are 256
// consecutive entries, its NV runs follow each other. So a Hadamard block of up to 256 NV inputs
// runs in one warp's registers and shuffles.
//
// What bounds it: HBM for many rows (bytes per entry: h + r + r_out + n or the codes) until the
// instructions per entry (about 25 for two norms and a gate, 25 for whitened codes with their
// values) do; the latency of load -> reductions -> store for a few. Measured (device, us and share
// of the 6551 GB/s copy rate): codes of 8192 x 8192 fp32 91 (1.01), of 2048 x 28672 bf16 whitened
// in blocks of 256 with values 70.4 (0.64; 59 % of the issue slots, a warp's reduction and the
// shuffles of T in the rest), of 4 x 8192 2.6 and whitened 3.0; two norms, gate and residual on
// 2048 x 8192 30.8 (0.83), on one row of 8192 3.9.
#include <cmath>
#include <type_traits>

#include "lq_device.cuh"
#include "lq_sm100.cuh"

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
  int rows, ahead;        // the row whose inputs a CTA asks for while it works on its own
  int few;                // the call's CTAs are all resident at once
  int plain;              // lq_quant_i8: codes of T(h) and nothing else
  float branch, resid;
  NormArgs post, pre;
  Whiten T;
};

struct F32 {
  static constexpr int dt = LQ_F32, size = 4;
  typedef float type;
};
struct F16 {
  static constexpr int dt = LQ_F16, size = 2;
  typedef __half type;
};
struct BF16 {
  static constexpr int dt = LQ_BF16, size = 2;
  typedef __nv_bfloat16 type;
};
// In the place of a residual's type: a norm without a residual; lq_quant_i8, where nothing stands
// between the input and T; and lq_quant_i8 of 16-bit inputs whose first butterflies the tensor
// cores take.
struct None { static constexpr int dt = -1, size = 2; };
struct Plain : None {};
struct PlainMma : None {};
template <class RT> constexpr bool has_r() { return RT::dt >= 0; }
template <class RT> constexpr bool is_plain() { return std::is_base_of<None, RT>::value && !std::is_same<RT, None>::value; }

// f with the type that dt names. Loops over a thread's entries go inside f: as a branch around a
// whole loop the choice costs nothing, inside it the compiler evaluates every type and selects.
template <class F>
__device__ __forceinline__ void with_type(int dt, F f) {
  if (dt == LQ_BF16) f(BF16{});
  else if (dt == LQ_F16) f(F16{});
  else f(F32{});
}

// Two fp32 operations in one instruction, on entries 2i and 2i + 1 of a vector.
__device__ __forceinline__ float2 fma2(float2 x, float2 y, float2 z) {
  float2 r;
  asm("{\n .reg .b64 a, b, c;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n"
      " mov.b64 c, {%6, %7};\n fma.rn.f32x2 a, a, b, c;\n mov.b64 {%0, %1}, a;\n}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y), "f"(z.x), "f"(z.y));
  return r;
}

__device__ __forceinline__ float2 mul2(float2 x, float2 y) {
  float2 r;
  asm("{\n .reg .b64 a, b;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n"
      " mul.rn.f32x2 a, a, b;\n mov.b64 {%0, %1}, a;\n}"
      : "=f"(r.x), "=f"(r.y) : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y));
  return r;
}

__device__ __forceinline__ float2 add2(float2 x, float2 y) {
  float2 r;
  asm("{\n .reg .b64 a, b;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n"
      " add.rn.f32x2 a, a, b;\n mov.b64 {%0, %1}, a;\n}"
      : "=f"(r.x), "=f"(r.y) : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y));
  return r;
}

__device__ __forceinline__ float2 pair(const float (&v)[8], int i) {
  return make_float2(v[2 * i], v[2 * i + 1]);
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ void put(float (&v)[8], int i, float2 x) {
  v[2 * i] = x.x;
  v[2 * i + 1] = x.y;
}

// 16 bytes that are read once: not kept in L1, where the norms' weights live
__device__ __forceinline__ uint4 ld_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

// 16 and 8 bytes that every row reads; not read-only (.nc) loads, which may be moved ahead of a wait
// for the kernel before
__device__ __forceinline__ uint4 ld_kept(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ uint2 ld_kept(const uint2* p) {
  uint2 v;
  asm volatile("ld.global.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}

template <class DT>
__device__ __forceinline__ void unpack2(uint32_t w, float& lo, float& hi) {
  if constexpr (DT::dt == LQ_BF16) {
    lo = __uint_as_float(w << 16);
    hi = __uint_as_float(w & 0xffff0000u);
  } else {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
    lo = f.x;
    hi = f.y;
  }
}

template <class DT>
__device__ __forceinline__ void unpack8(const uint4& a, const uint4& b, float (&v)[8]) {
  if constexpr (DT::dt == LQ_F32) {
    v[0] = __uint_as_float(a.x); v[1] = __uint_as_float(a.y);
    v[2] = __uint_as_float(a.z); v[3] = __uint_as_float(a.w);
    v[4] = __uint_as_float(b.x); v[5] = __uint_as_float(b.y);
    v[6] = __uint_as_float(b.z); v[7] = __uint_as_float(b.w);
  } else {
    unpack2<DT>(a.x, v[0], v[1]);
    unpack2<DT>(a.y, v[2], v[3]);
    unpack2<DT>(a.z, v[4], v[5]);
    unpack2<DT>(a.w, v[6], v[7]);
  }
}

template <class DT>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (DT::dt == LQ_BF16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f32(float v, float& x) { x = v; }
__device__ __forceinline__ void from_f32(float v, __half& x) { x = __float2half_rn(v); }
__device__ __forceinline__ void from_f32(float v, __nv_bfloat16& x) { x = __float2bfloat16_rn(v); }

// How the entries of a row map to threads and how they move.
//   kVec     16-byte accesses: K a multiple of 8, everything aligned
//   kStrided any K and alignment, no whitening: a warp's 256 entries are dealt out one by one, so
//            that its 2- and 4-byte accesses fall on consecutive addresses
//   kScalar  any K and alignment with whitening, whose butterflies want eight consecutive entries
//            per thread
//   kFull    kVec without a ragged end: the CTAs of a row cover exactly K entries
enum Mode { kVec, kStrided, kScalar, kFull };
__host__ __device__ constexpr bool is_vec(Mode m) { return m == kVec || m == kFull; }

// whether column c of a part of n columns is there
template <Mode M>
__device__ __forceinline__ bool in_row(int c, int n) { return M == kFull || c < n; }

// column of entry e of vector j of this thread, within the CTA's part of the row: a warp's vectors
// are NV runs of 256 entries, one behind the other
template <int NV, Mode M>
__device__ __forceinline__ int col_of(int j, int e) {
  const int base = 8 * (int)(threadIdx.x & ~31u) * NV + 256 * j, lane = threadIdx.x & 31;
  return M == kStrided ? base + 32 * e + lane : base + 8 * lane + e;
}

// whether all entries of vector j of this warp's threads lie in a part of n columns
template <int NV>
__device__ __forceinline__ bool whole_run(int j, int n) {
  return 8 * (int)(threadIdx.x & ~31u) * NV + 256 * (j + 1) <= n;
}

// f(j, entries of vector j) for the row part at element `off` of p, zero from column n on. One branch
// for all vectors, so that their loads are under way together (2048 x 4097, bf16, one norm and a residual:
// 23.5 against 34.6 us with a branch for each, the residual's prefetch included).
template <class DT, int NV, Mode M, class F>
__device__ __forceinline__ void each_scalar(const void* p, int64_t off, int n, F f) {
  const typename DT::type* q = static_cast<const typename DT::type*>(p) + off + col_of<NV, M>(0, 0);
  constexpr int step = M == kStrided ? 32 : 1;
  if (whole_run<NV>(NV - 1, n)) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = to_f32(q[256 * j + e * step]);
      f(j, v);
    }
  } else {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e)
        v[e] = col_of<NV, M>(j, e) < n ? to_f32(q[256 * j + e * step]) : 0.f;
      f(j, v);
    }
  }
}

// vector j of what every row reads (a norm's weight, a gate); L1 keeps it
template <class DT, int NV, Mode M>
__device__ __forceinline__ void load_shared8(const void* p, int64_t off, int j, float (&v)[8]) {
  const uint4* s = reinterpret_cast<const uint4*>(static_cast<const typename DT::type*>(p) + off +
                                                  col_of<NV, M>(j, 0));
  const uint4 a = ld_kept(s);
  unpack8<DT>(a, DT::size == 4 ? ld_kept(s + 1) : a, v);
}

// entries of vector j of an output row part at element `off` of p, each rounded once
template <class DT, int NV, Mode M>
__device__ __forceinline__ void store8(void* p, int64_t off, int j, int n, const float (&v)[8]) {
  typename DT::type* q = static_cast<typename DT::type*>(p) + off;
  if constexpr (is_vec(M)) {
    uint4* d = reinterpret_cast<uint4*>(q + col_of<NV, M>(j, 0));
    if constexpr (DT::size == 4) {
      d[0] = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                        __float_as_uint(v[3]));
      d[1] = make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]),
                        __float_as_uint(v[7]));
    } else {
      d[0] = make_uint4(pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3]), pack2<DT>(v[4], v[5]),
                        pack2<DT>(v[6], v[7]));
    }
  } else {
    q += col_of<NV, M>(j, 0);
    constexpr int step = M == kStrided ? 32 : 1;
    if (whole_run<NV>(j, n)) {
#pragma unroll
      for (int e = 0; e < 8; ++e) from_f32(v[e], q[e * step]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (col_of<NV, M>(j, e) < n) from_f32(v[e], q[e * step]);
    }
  }
}

// v = op(v, entries of the shared vector p), two entries at a time
template <int NV, Mode M, class Op>
__device__ __forceinline__ void combine(float (&v)[NV][8], const void* p, int dt, int64_t off, int n,
                                        Op op) {
  with_type(dt, [&](auto t) {
    if constexpr (is_vec(M)) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (!in_row<M>(col_of<NV, M>(j, 0), n)) continue;
        float w[8];
        load_shared8<decltype(t), NV, M>(p, off, j, w);
#pragma unroll
        for (int i = 0; i < 4; ++i) put(v[j], i, op(pair(v[j], i), pair(w, i)));
      }
    } else {
      each_scalar<decltype(t), NV, M>(p, off, n, [&](int j, const float (&w)[8]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) put(v[j], i, op(pair(v[j], i), pair(w, i)));
      });
    }
  });
}

template <int NV, Mode M>
__device__ __forceinline__ void store_all(const float (&v)[NV][8], void* p, int dt, int64_t off,
                                          int n) {
  with_type(dt, [&](auto t) {
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (in_row<M>(col_of<NV, M>(j, 0), n)) store8<decltype(t), NV, M>(p, off, j, n, v[j]);
  });
}

// the largest magnitude, NaN if there is one
__device__ __forceinline__ float max_abs(float a, float b, float c) {
  float m;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(a), "f"(b), "f"(c));
  return m;
}

// Reductions over a row: every warp leaves its partial in the shared memory of all the row's CTAs,
// then all threads read all partials. Each reduction has its own slots, so none waits for the one
// before to be read. An entry of a sum passes through at most 32 additions in its thread (8 with one
// vector), 5 between lanes, 2 within a read of four partials and one per read: 8 CTAs x 2 reads with
// four vectors, 8 x 8 with one. So at most 79 roundings of fp32, in either form.
struct Reducer {
  uint32_t* slots;   // [kReductions][8 CTAs][32 warps]
  int ctas, rank;

  __device__ __forceinline__ void put(int which, uint32_t x) const {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    uint32_t* mine = slots + which * 256 + rank * 32 + warp;
    // zeros behind the last warp, up to the four slots of one read
    const int pad = warp == warps - 1 ? -warps & 3 : 0;
    if (ctas == 1) {
      if (lane <= pad) mine[lane] = lane == 0 ? x : 0u;
      __syncthreads();
      return;
    }
    for (int p = 0; p <= pad; ++p) {
      if (lane < ctas) {
        uint32_t addr;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                     : "=r"(addr) : "r"((uint32_t)__cvta_generic_to_shared(mine + p)), "r"(lane));
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(p == 0 ? x : 0u)
                     : "memory");
      }
    }
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;"
                 ::: "memory");
  }

  template <class F>
  __device__ __forceinline__ void each(int which, F f) const {
    const int quads = ((blockDim.x >> 5) + 3) >> 2;
    for (int c = 0; c < ctas; ++c)
      for (int i = 0; i < quads; ++i)
        f(*reinterpret_cast<const uint4*>(slots + which * 256 + c * 32 + 4 * i));
  }

  __device__ __forceinline__ float sum(int which, float x) const {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    if (blockDim.x == 32 && ctas == 1) return x;
    put(which, __float_as_uint(x));
    x = 0.f;
    each(which, [&](uint4 p) {
      x += (__uint_as_float(p.x) + __uint_as_float(p.y)) +
           (__uint_as_float(p.z) + __uint_as_float(p.w));
    });
    return x;
  }

  __device__ __forceinline__ uint32_t max(int which, uint32_t x) const {
    x = __reduce_max_sync(0xffffffffu, x);
    if (blockDim.x == 32 && ctas == 1) return x;
    put(which, x);
    x = 0u;
    each(which, [&](uint4 p) { x = ::max(::max(x, ::max(p.x, p.y)), ::max(p.z, p.w)); });
    return x;
  }
};

template <int NV>
__device__ __forceinline__ void scale_all(float (&v)[NV][8], float f) {
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) put(v[j], i, mul2(pair(v[j], i), both(f)));
}

// v = norm(v), in place. Entries from column n of this CTA's part on are zero before and after.
// first: this norm's two reductions are `first` and `first + 1`.
template <int NV, Mode M>
__device__ __forceinline__ void apply_norm(float (&v)[NV][8], const NormArgs& p, int K, int n,
                                           int64_t off, const Reducer& red, int first) {
  const float inv_k = 1.f / (float)K;
  if (p.kind == LQ_NORM_LAYER) {
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e) s += v[j][e];
    const float mean = red.sum(first + 1, s) * inv_k;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (in_row<M>(col_of<NV, M>(j, e), n)) v[j][e] -= mean;
  }
  float2 ss = both(0.f);
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) ss = fma2(pair(v[j], i), pair(v[j], i), ss);
  const float rs = rsqrtf(fmaf(red.sum(first, ss.x + ss.y), inv_k, p.eps));
  if (p.w) {
    combine<NV, M>(v, p.w, p.dt, off, n,
                   [&](float2 x, float2 w) { return mul2(mul2(x, both(rs)), w); });
  } else {
    scale_all<NV>(v, rs);
  }
  if (p.b) combine<NV, M>(v, p.b, p.dt, off, n, [](float2 x, float2 w) { return add2(x, w); });
}

// The butterflies from distance 8 * kFirst on.
template <int NV, int kFirst>
__device__ __forceinline__ void finish_whiten(float (&v)[NV][8], const Whiten& T, float* ex) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int m = kFirst; m < 32; m <<= 1) {
    if (8 * m >= T.block) break;
    const float2 s = both((lane & m) != 0 ? -1.f : 1.f);
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 o = make_float2(__shfl_xor_sync(0xffffffffu, v[j][2 * i], m),
                                     __shfl_xor_sync(0xffffffffu, v[j][2 * i + 1], m));
        put(v[j], i, fma2(pair(v[j], i), s, o));
      }
  }
  // distance 256 and 512 between a thread's own vectors
#pragma unroll
  for (int h = 1; h < NV; h <<= 1)
    if (256 * h < T.block) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if ((j & h) == 0)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 x = pair(v[j], i), y = pair(v[j + h], i);
            put(v[j], i, add2(x, y));
            put(v[j + h], i, fma2(y, both(-1.f), x));
          }
    }
  // the rest between warps; a CTA's part is a whole number of blocks
  for (int m = 32; 8 * NV * m < T.block; m <<= 1) {
    const float s = (threadIdx.x & m) != 0 ? -1.f : 1.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      __syncthreads();
#pragma unroll
      for (int e = 0; e < 8; ++e) ex[e * blockDim.x + threadIdx.x] = v[j][e];
      __syncthreads();
#pragma unroll
      for (int e = 0; e < 8; ++e)
        v[j][e] = fmaf(v[j][e], s, ex[e * blockDim.x + (threadIdx.x ^ m)]);
    }
  }
}

// v = sqrt(block) T(v): sign and channel scale, then butterflies over distance 1, 2, 4 in a
// thread's vector, 8 .. 128 across the warp's lanes, 256 and up between a thread's vectors and
// through shared memory (ex: 8 * threads floats). The codes do not see a common factor and the scale takes it later.
template <int NV, Mode M>
__device__ __forceinline__ void apply_whiten(float (&v)[NV][8], const Whiten& T, int n, int64_t off,
                                             float* ex) {
  if constexpr (!is_vec(M))
    if (T.chan_scale)
      combine<NV, M>(v, T.chan_scale, LQ_F32, off, n, [](float2 x, float2 w) { return mul2(x, w); });
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = col_of<NV, M>(j, 0);
    if (in_row<M>(c, n)) {
      if constexpr (is_vec(M)) {
        if (T.chan_scale) {
          float cs[8];
          load_shared8<F32, NV, M>(T.chan_scale, off, j, cs);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[j][e] *= cs[e];
        }
      }
      if (T.sign) {
        uint32_t lo, hi;
        if (is_vec(M)) {
          const uint2 s = ld_kept(reinterpret_cast<const uint2*>(T.sign + off + c));
          lo = s.x;
          hi = s.y;
        } else {
          lo = hi = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (c + e < n) lo |= (uint32_t)(uint8_t)T.sign[off + c + e] << (8 * e);
            if (c + e + 4 < n) hi |= (uint32_t)(uint8_t)T.sign[off + c + e + 4] << (8 * e);
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
    const float2 minus = both(-1.f);
    if (T.block > 1) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        put(v[j], i, make_float2(v[j][2 * i] + v[j][2 * i + 1], v[j][2 * i] - v[j][2 * i + 1]));
    }
#pragma unroll
    for (int h = 1; h < 4; h <<= 1)
      if (2 * h < T.block)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if ((i & h) == 0) {
            const float2 x = pair(v[j], i), y = pair(v[j], i + h);
            put(v[j], i, add2(x, y));
            put(v[j], i + h, fma2(y, minus, x));
          }
  }
  finish_whiten<NV, 1>(v, T, ex);
}

// T's signs and its butterflies over distance 1, 2, 8 and 16 of 16-bit inputs, as a product: with
// the eight entries of lane (g, t) as rows g (entries 0 .. 3) and g + 8 (4 .. 7) of a 16 x 16
// matrix, columns t and the entry's low two bits, each row times the Hadamard matrix of order 16.
// Its columns are ordered so that every sum lands where its entry came from. The products are exact;
// the tensor core adds the sixteen of a sum in its own way, not as a chain of fp32 additions rounded to
// nearest. Tests hold all of T to log2(block) + 3 steps of fp32 (2^-23) of the block's sum of
// magnitudes over sqrt(block).
template <class HT, int NV, Mode M>
__device__ __forceinline__ void whiten_mma(float (&v)[NV][8], const uint4 (&raw)[NV][1],
                                           const Whiten& T, int n, int64_t off, float* ex) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  constexpr uint32_t kOne = HT::dt == LQ_BF16 ? 0x3f803f80u : 0x3c003c00u;
  uint32_t h[2][2];   // [output bit 1][input bit 1]: entries of input bit 0 = 0, 1
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const uint32_t base = (uint32_t)(__popc(t & (g >> 1)) + (j & q)) & 1u;
      h[j][q] = kOne ^ (base << 15) ^ ((base ^ (uint32_t)(g & 1)) << 31);
    }
  const float2 minus = both(-1.f);
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = col_of<NV, M>(j, 0);
    uint32_t w[4] = {raw[j][0].x, raw[j][0].y, raw[j][0].z, raw[j][0].w};
    if (T.sign && in_row<M>(c, n)) {
      const uint2 s = ld_kept(reinterpret_cast<const uint2*>(T.sign + off + c));
      // the sign bits of bytes 0, 1 and of 2, 3 over those of a pair of entries
      w[0] ^= __byte_perm(s.x, 0u, 0x1404) & 0x80008000u;
      w[1] ^= __byte_perm(s.x, 0u, 0x3424) & 0x80008000u;
      w[2] ^= __byte_perm(s.y, 0u, 0x1404) & 0x80008000u;
      w[3] ^= __byte_perm(s.y, 0u, 0x3424) & 0x80008000u;
    }
    float o[2][4];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if constexpr (HT::dt == LQ_BF16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%10,%10,%10,%10};"
            : "=f"(o[k][0]), "=f"(o[k][1]), "=f"(o[k][2]), "=f"(o[k][3])
            : "r"(w[0]), "r"(w[2]), "r"(w[1]), "r"(w[3]), "r"(h[k][0]), "r"(h[k][1]), "f"(0.f));
      else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%10,%10,%10,%10};"
            : "=f"(o[k][0]), "=f"(o[k][1]), "=f"(o[k][2]), "=f"(o[k][3])
            : "r"(w[0]), "r"(w[2]), "r"(w[1]), "r"(w[3]), "r"(h[k][0]), "r"(h[k][1]), "f"(0.f));
    }
    // distance 4: entries 0 .. 3 against 4 .. 7
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float2 x = make_float2(o[k][0], o[k][1]), y = make_float2(o[k][2], o[k][3]);
      put(v[j], k, add2(x, y));
      put(v[j], k + 2, fma2(y, minus, x));
    }
  }
  finish_whiten<NV, 4>(v, T, ex);
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

constexpr float kRound = 12582912.f;   // 1.5 * 2^23: adding it rounds half to even

// Codes of eight entries as b[e] = bits of kRound + code (the low byte is the code). fma(v, 127 / a,
// kRound) rounds a quotient that is off by at most 127 * 2^-24, so the code is right unless the
// quotient lies within 2e-5 of a border; there border_code decides. Whitened entries (`exact` false)
// carry the roundings of T, larger than that, and are left at the first answer.
__device__ __forceinline__ void codes8(const float (&v)[8], float inv, float a, bool exact,
                                       uint32_t (&b)[8]) {
  const float2 f = both(inv), one = both(kRound), minus = both(-1.f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 m = fma2(pair(v, i), f, one);
    b[2 * i] = __float_as_uint(m.x);
    b[2 * i + 1] = __float_as_uint(m.y);
  }
  if (!exact) return;
  float worst = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 m = make_float2(__uint_as_float(b[2 * i]), __uint_as_float(b[2 * i + 1]));
    const float2 d = fma2(pair(v, i), f, fma2(m, minus, one));
    worst = max_abs(worst, d.x, d.y);
  }
  if (worst > 0.49998f) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float m = __uint_as_float(b[e]);
      if (fabsf(fmaf(v[e], inv, kRound - m)) > 0.49998f) {
        const float below = floorf(fabsf(v[e] * inv));
        b[e] = __float_as_uint(kRound + copysignf(border_code(fabsf(v[e]), a, below), v[e]));
      }
    }
  }
}

__device__ __forceinline__ uint32_t low_bytes(uint32_t b0, uint32_t b1, uint32_t b2, uint32_t b3) {
  return __byte_perm(__byte_perm(b0, b1, 0x0040), __byte_perm(b2, b3, 0x0040), 0x5410);
}

// The most threads of a CTA and the CTAs an SM should hold. The wide form (NV = 1) is for calls
// whose CTAs are all resident at once, where the latency of a row counts; the other keeps a CTA
// small, so that several rows are in flight per SM: 64 registers a thread without a residual, 80
// with one (64 spill: 2048 x 8192 took 37.2 against 34.4 us).
template <int NV, bool kHasR>
struct Form {
  static constexpr int kThreads = NV == 1 ? 1024 : 256;
  static constexpr int kBlocks = NV == 1 ? 1 : kHasR ? 3 : 4;
};
constexpr int kReductions = 5;

template <class DT, int NV, Mode M>
__device__ __forceinline__ void load_raw(uint4 (&raw)[NV][DT::size / 2], const void* p,
                                         int64_t first, int n) {
  const char* src = static_cast<const char*>(p) + first * DT::size;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = col_of<NV, kVec>(j, 0);
#pragma unroll
    for (int i = 0; i < DT::size / 2; ++i)
      raw[j][i] = in_row<M>(c, n) ? ld_stream(src + c * DT::size + 16 * i) : make_uint4(0u, 0u, 0u, 0u);
  }
}

constexpr uint32_t kInfinity = 0x7f800000u;
// T adds up to 4096 entries before its 1/sqrt(block), so a row of large finite ones can overflow on
// the way. Such a row is moved by 2^-64 first, its scale by 2^64 afterwards; next to its largest
// entry, what that takes from the small ones is nothing.
constexpr float kDown = 0x1p-64f, kUp = 0x1p64f;

// The largest magnitude of the row in v as the bits of an fp32: they order like the magnitudes, with
// infinity and the NaNs on top.
template <int NV>
__device__ __forceinline__ uint32_t row_top(const Reducer& red, int which, const float (&v)[NV][8]) {
  float big = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) big = max_abs(big, v[j][2 * i], v[j][2 * i + 1]);
  return red.max(which, __float_as_uint(big));
}

// The scale of the whitened row in v, its codes, and the values they stand for. top: row_top(v);
// down: v was moved by kDown.
template <class HT, int NV, Mode M>
__device__ __forceinline__ void write_codes(const RowArgs& a, const Reducer& red, int64_t row,
                                            int64_t off, int n, float (&v)[NV][8], uint32_t top,
                                            bool down) {
  const float amax = __uint_as_float(top);
  const float moved = (a.T.block ? amax * a.T.inv_sqrt : amax) / 127.f;
  const bool finite = top < kInfinity && !(down && moved * kUp > 0x1.fffffep127f);
  const float scale = finite ? down ? moved * kUp : moved : __uint_as_float(0x7fffffffu);
  if (threadIdx.x == 0 && red.rank == 0) a.q_scale[row] = scale;
  // 127 v and 127 / a must neither overflow nor lose bits: rows of extreme magnitude are moved
  // by a power of two (exact for every entry that can differ from code 0)
  float shift = 1.f;
  const int exponent = (int)(top >> 23);
  if (exponent < 16 || exponent > 240)
    shift = __uint_as_float((uint32_t)max(1, min(253, 254 - exponent)) << 23);
  const float as = amax * shift;
  const float inv = finite && amax > 0.f ? 127.f / as : 0.f;
  int8_t* qrow = a.q + row * a.ldq + off;
  const int qn = (int)(a.ldq - off);     // columns of the stored row from here on
  const bool exact = a.T.block == 0;
  auto write = [&](auto t) {
    typedef decltype(t) VT;              // the type of `values`, None without
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = col_of<NV, M>(j, 0);
      if (M != kStrided && M != kFull && c >= qn) continue;
      uint32_t b[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) b[e] = __float_as_uint(kRound);
      if (inv != 0.f) {
        if (shift != 1.f)
#pragma unroll
          for (int e = 0; e < 8; ++e) v[j][e] *= shift;
        codes8(v[j], inv, as, exact, b);
      }
      if constexpr (M == kStrided) {
        if (whole_run<NV>(j, qn)) {
#pragma unroll
          for (int e = 0; e < 8; ++e) qrow[c + 32 * e] = (int8_t)b[e];
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (c + 32 * e < qn) qrow[c + 32 * e] = (int8_t)b[e];
        }
      } else {
        *reinterpret_cast<uint2*>(qrow + c) =
            make_uint2(low_bytes(b[0], b[1], b[2], b[3]), low_bytes(b[4], b[5], b[6], b[7]));
      }
      if constexpr (VT::dt >= 0) {
        if (!in_row<M>(c, n)) continue;
        float o[8];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          put(o, i, mul2(add2(make_float2(__uint_as_float(b[2 * i]), __uint_as_float(b[2 * i + 1])),
                              both(-kRound)), both(scale)));
        store8<VT, NV, M>(a.values, row * a.K + off, j, n, o);
      }
    }
  };
  if (!a.values) write(None{});
  else if constexpr (is_vec(M)) write(HT{});   // values have x's type
  else with_type(a.vdt, write);
}

// The codes of a row of lq_quant_i8 whose T overflowed, from its inputs moved by kDown. Out of line:
// few rows ever come here, and the others' registers are not to be shared with it.
template <class HT, int NV, Mode M>
__device__ __noinline__ void again_from_below(const RowArgs& a, Reducer red, int row, int off, int n,
                                              float* ex) {
  uint4 hr[NV][HT::size / 2];
  float v[NV][8];
  load_raw<HT, NV, M>(hr, a.h, (int64_t)row * a.ldh + off, n);
#pragma unroll
  for (int j = 0; j < NV; ++j) unpack8<HT>(hr[j][0], hr[j][HT::size / 2 - 1], v[j]);
  scale_all<NV>(v, kDown);
  apply_whiten<NV, M>(v, a.T, n, off, ex);
  write_codes<HT, NV, M>(a, red, row, off, n, v, row_top<NV>(red, 3, v), true);
}

// n entries of `size` bytes of an input into L2
__device__ __forceinline__ void prefetch_row(const void* p, int64_t first, int n, int size) {
  const char* src = static_cast<const char*>(p) + first * size;
  for (int b = threadIdx.x * 128; b < n * size; b += blockDim.x * 128)
    asm volatile("prefetch.global.L2 [%0];" ::"l"(src + b));
}

// The row in v through the call's steps. add_r(f): v[j] = f(residual's vector j, v[j]) for all j.
template <class HT, class RT, int NV, Mode M, class AddR>
__device__ __forceinline__ void work_row(const RowArgs& a, const Reducer& red, int64_t row,
                                         int64_t off, int n, float (&v)[NV][8], AddR add_r,
                                         float* ex) {
  constexpr bool kHasR = has_r<RT>();
  if (a.post.kind) apply_norm<NV, M>(v, a.post, a.K, n, off, red, 0);

  if (a.gate) {
    const int64_t g = (int64_t)((int)row / a.gate_tokens) * a.gate_cols;
    if (a.gate_cols > 1) {
      combine<NV, M>(v, a.gate, a.gdt, g + off, n,
                     [](float2 x, float2 w) { return mul2(x, w); });
    } else {
      scale_all<NV>(v, load_as_f32(a.gate, a.gdt, g));
    }
  }
  if (a.branch != 1.f) scale_all<NV>(v, a.branch);
  if constexpr (kHasR) {
    add_r([&](float (&x)[8], const float (&w)[8]) {
#pragma unroll
      for (int i = 0; i < 4; ++i) put(x, i, fma2(pair(w, i), both(a.resid), pair(x, i)));
    });
  }
  if (a.r_out) store_all<NV, M>(v, a.r_out, a.rdt, row * a.ldro + off, n);

  if (a.pre.kind) apply_norm<NV, M>(v, a.pre, a.K, n, off, red, 2);
  if (a.n_out) store_all<NV, M>(v, a.n_out, a.ndt, row * a.K + off, n);
  if (!a.q) return;

  bool down = false;
  if constexpr (M != kStrided)
    if (a.T.block) {
      // behind a norm only a weight of 1e30 would make entries that large
      if (!a.pre.kind && row_top<NV>(red, 3, v) >= __float_as_uint(kUp)) {
        down = true;
        scale_all<NV>(v, kDown);
      }
      apply_whiten<NV, M>(v, a.T, n, off, ex);
    }
  write_codes<HT, NV, M>(a, red, row, off, n, v, row_top<NV>(red, 4, v), down);
}

// RT: the residual's type, None without one (then r_out, if any, has type a.rdt)
template <class HT, class RT, int NV, Mode M>
__global__ void __launch_bounds__(Form<NV, has_r<RT>()>::kThreads, Form<NV, has_r<RT>()>::kBlocks)
    row_kernel(const __grid_constant__ RowArgs a, int ctas) {
  extern __shared__ __align__(16) float ex[];   // whitening blocks over 256
  __shared__ __align__(16) uint32_t slots[kReductions * 256];
  constexpr bool kHasR = has_r<RT>();
  const int T = blockDim.x;
  int row, rank;   // a row is a cluster's (of one CTA, too)
  asm("mov.u32 %0, %clusterid.x;" : "=r"(row));
  asm("mov.u32 %0, %cluster_ctarank;" : "=r"(rank));
  const Reducer red{slots, ctas, rank};
  // this CTA's part of the row: n columns from column off
  const int off = red.rank * (8 * NV) * T;
  const int n = min(a.K - off, (8 * NV) * T);
  // all CTAs of the cluster run before one writes to another's shared memory
  if (ctas > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  // a few rows overlap their start with the kernel before and after (4 x 8192 codes 3.1 -> 2.6 us,
  // whitened 3.5 -> 3.0, one row through two norms 4.4 -> 3.9);
  // many would give SMs away early (65536 x 256 and two norms 37.4 -> 68.4 us)
  if (NV == 1 && a.few) {
    sm100::grid_release();
    sm100::grid_wait();
  }
  float v[NV][8];
  if constexpr (is_vec(M)) {
    uint4 hr[NV][HT::size / 2], rr[NV][RT::size / 2];
    load_raw<HT, NV, M>(hr, a.h, row * a.ldh + off, n);
    // in flight during the first norm's reductions
    if constexpr (kHasR) load_raw<RT, NV, M>(rr, a.r, row * a.ldr + off, n);
    if (NV > 1 && a.ahead < a.rows - row) {
      prefetch_row(a.h, (row + a.ahead) * a.ldh + off, n, HT::size);
      if constexpr (kHasR) prefetch_row(a.r, (row + a.ahead) * a.ldr + off, n, RT::size);
    }
    if (ctas > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    if constexpr (std::is_same<RT, PlainMma>::value) {
      whiten_mma<HT, NV, M>(v, hr, a.T, n, off, ex);
    } else {
#pragma unroll
      for (int j = 0; j < NV; ++j) unpack8<HT>(hr[j][0], hr[j][HT::size / 2 - 1], v[j]);
      if constexpr (is_plain<RT>())
        if (a.T.block) apply_whiten<NV, M>(v, a.T, n, off, ex);
    }
    if constexpr (is_plain<RT>()) {
      const uint32_t top = row_top<NV>(red, 4, v);
      // an infinity or a NaN, or sums of T that overflowed (65504 times 4096 does not)
      if constexpr (!(std::is_same<RT, PlainMma>::value && HT::dt == LQ_F16))
        if (a.T.block && top >= kInfinity) {
          again_from_below<HT, NV, M>(a, red, row, off, n, ex);
          return;
        }
      write_codes<HT, NV, M>(a, red, row, off, n, v, top, false);
    } else work_row<HT, RT, NV, M>(a, red, row, off, n, v, [&](auto add) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        float w[8];
        unpack8<RT>(rr[j][0], rr[j][RT::size / 2 - 1], w);
        add(v[j], w);
      }
    }, ex);
  } else {
    if (NV > 1) {
      // the residual's row while this one is on its way and normed; then rows to come
      const int hb = a.hdt == LQ_F32 ? 4 : 2, rb = a.rdt == LQ_F32 ? 4 : 2;
      if (kHasR) prefetch_row(a.r, row * a.ldr + off, n, rb);
      if (a.ahead < a.rows - row) {
        prefetch_row(a.h, (row + a.ahead) * a.ldh + off, n, hb);
        if (kHasR) prefetch_row(a.r, (row + a.ahead) * a.ldr + off, n, rb);
      }
    }
    with_type(a.hdt, [&](auto t) {
      each_scalar<decltype(t), NV, M>(a.h, row * a.ldh + off, n, [&](int j, const float (&x)[8]) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[j][e] = x[e];
      });
    });
    if (ctas > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    work_row<HT, RT, NV, M>(a, red, row, off, n, v, [&](auto add) {
      with_type(a.rdt, [&](auto t) {
        each_scalar<decltype(t), NV, M>(a.r, row * a.ldr + off, n,
                                        [&](int j, const float (&w)[8]) { add(v[j], w); });
      });
    }, ex);
  }
}

struct Shape {
  int nv, ctas, threads;
  size_t smem;
};

// CTAs of one row and their threads, with nv vectors per thread
Shape shape_of(int K, int block, int nv) {
  Shape s;
  const int vecs = (K + 7) / 8, most = nv == 1 ? 1024 : 256 * nv;
  s.nv = nv;
  s.ctas = (vecs + most - 1) / most;
  // a few CTAs more where they divide the row evenly (kFull; 20480 entries: four CTAs 48.9 us,
  // three with a ragged end 54.7)
  for (int c = s.ctas; nv > 1 && s.ctas > 1 && c <= std::min(8, s.ctas + 2); ++c)
    if (vecs % (32 * nv * c) == 0) {
      s.ctas = c;
      break;
    }
  const int part = (vecs + s.ctas - 1) / s.ctas;
  s.threads = (std::max(1, (part + nv - 1) / nv) + 31) / 32 * 32;
  s.smem = 0;
  if (block > 256) {   // a CTA's part holds whole blocks
    const int unit = std::max(32, block / (8 * nv));
    s.threads = (s.threads + unit - 1) / unit * unit;
    if (block > 256 * nv) s.smem = (size_t)s.threads * 8 * sizeof(float);
  }
  s.ctas = (vecs + s.threads * nv - 1) / (s.threads * nv);
  return s;
}

template <class HT, class RT, int NV, Mode M>
cudaError_t launch_one(const RowArgs& a, int rows, const Shape& s, cudaStream_t st) {
  if ((int64_t)rows * s.ctas > INT32_MAX) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)rows * s.ctas);
  cfg.blockDim = dim3(s.threads);
  cfg.dynamicSmemBytes = s.smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  if (s.ctas > 1) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    attr[cfg.numAttrs].val.clusterDim.x = s.ctas;
    attr[cfg.numAttrs].val.clusterDim.y = attr[cfg.numAttrs].val.clusterDim.z = 1;
    ++cfg.numAttrs;
  }
  if (NV == 1 && a.few) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[cfg.numAttrs].val.programmaticStreamSerializationAllowed = 1;
    ++cfg.numAttrs;
  }
  cfg.attrs = attr;
  return cudaLaunchKernelEx(&cfg, row_kernel<HT, RT, NV, M>, a, s.ctas);
}

template <class HT, class RT, Mode M>
cudaError_t launch_nv(const RowArgs& a, int rows, const Shape& s, cudaStream_t st) {
  if (s.nv == 1) return launch_one<HT, RT, 1, M>(a, rows, s, st);
  if constexpr (M == kVec)
    if (a.K == s.ctas * s.threads * s.nv * 8) return launch_one<HT, RT, 4, kFull>(a, rows, s, st);
  return launch_one<HT, RT, 4, M>(a, rows, s, st);
}

template <class HT>
cudaError_t launch_h(const RowArgs& a, int rows, const Shape& s, cudaStream_t st) {
  if constexpr (HT::size == 2)
    if (a.plain && a.T.block >= 32 && !a.T.chan_scale)
      return launch_nv<HT, PlainMma, kVec>(a, rows, s, st);
  if (a.plain) return launch_nv<HT, Plain, kVec>(a, rows, s, st);
  if (!a.r) return launch_nv<HT, None, kVec>(a, rows, s, st);
  if (a.rdt == LQ_F32) return launch_nv<HT, F32, kVec>(a, rows, s, st);
  if (a.rdt == LQ_F16) return launch_nv<HT, F16, kVec>(a, rows, s, st);
  return launch_nv<HT, BF16, kVec>(a, rows, s, st);
}

size_t width(int dt) { return dt == LQ_F32 ? 4 : 2; }
bool known(int dt) { return dt == LQ_F32 || dt == LQ_F16 || dt == LQ_BF16; }

// 16-byte loads and stores everywhere: K a multiple of 8 and every pointer and stride aligned
bool vectors_ok(const RowArgs& a) {
  if (a.K % 8 != 0 || !aligned(a.h, 16) || a.ldh * width(a.hdt) % 16 != 0) return false;
  if (a.r && (!aligned(a.r, 16) || a.ldr * width(a.rdt) % 16 != 0)) return false;
  if (a.r_out && (!aligned(a.r_out, 16) || a.ldro * width(a.rdt) % 16 != 0)) return false;
  if (!aligned(a.n_out, 16) || !aligned(a.values, 16) || !aligned(a.gate, 16)) return false;
  for (const NormArgs* p : {&a.post, &a.pre})
    if (p->kind && (!aligned(p->w, 16) || !aligned(p->b, 16))) return false;
  return !a.q || !a.T.block || (aligned(a.T.sign, 8) && aligned(a.T.chan_scale, 16));
}

cudaError_t launch_rows(RowArgs a, int rows, cudaStream_t st) {
  const int block = a.q ? a.T.block : 0;
  const int sms = tc_sm_count();
  if (sms <= 0) return cudaErrorInvalidDevice;
  // the wide form while about all its threads are resident at once, and for rows too short to give
  // a thread of the small form four vectors
  Shape s = shape_of(a.K, block, 1);
  // Half as many rows ahead as are in flight (2048 x 28672 codes 86 -> 78 us, 2048 x 8192 boundary
  // 36.9 -> 34.7; a whole wave or two ahead were slower). Not for fp32 codes without whitening,
  // which HBM bounds as it is (8192 x 8192: 100 us, with prefetches 107).
  a.ahead = a.plain && block == 0 && a.hdt == LQ_F32
                ? rows
                : std::max(1, sms * (a.r ? 3 : 4) * 256 / 2 / std::max(1, (a.K + 31) / 32));
  // (160 rows of 8192 with two norms: 7.7 us in the wide form, 5.2 in the other)
  a.few = (int64_t)rows * s.ctas * s.threads <= sms * 1024;
  if (!a.few && a.K >= 1024) s = shape_of(a.K, block, 4);
  if (!vectors_ok(a)) {
    if (block)
      return a.r ? launch_nv<F32, F32, kScalar>(a, rows, s, st)
                 : launch_nv<F32, None, kScalar>(a, rows, s, st);
    return a.r ? launch_nv<F32, F32, kStrided>(a, rows, s, st)
               : launch_nv<F32, None, kStrided>(a, rows, s, st);
  }
  if (a.hdt == LQ_F32) return launch_h<F32>(a, rows, s, st);
  if (a.hdt == LQ_F16) return launch_h<F16>(a, rows, s, st);
  return launch_h<BF16>(a, rows, s, st);
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
  if (!aligned(out->w, width(out->dt)) || !aligned(out->b, width(out->dt)))
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
  using namespace lq;
  using namespace lq::rows;
  lq::set_last_error("%s", "");
  lq_status st = check_row(rows, K, "lq_quant_i8");
  if (st != LQ_OK) return st;
  if (!known(xdt)) return reject(LQ_EINVAL, "lq_quant_i8: unknown x dtype %d", (int)xdt);
  if (rows == 0) return LQ_OK;
  if (!x || !q || !scale) return reject(LQ_EINVAL, "lq_quant_i8: null pointer");
  if (ldx < K) return reject(LQ_EINVAL, "lq_quant_i8: ldx = %lld < K = %d", (long long)ldx, K);
  if (!aligned(x, width(xdt)) || !aligned(q, 16) || !aligned(scale, 4) ||
      (values && !aligned(values, width(xdt))))
    return reject(LQ_EINVAL, "lq_quant_i8: misaligned x, q, scale or values");
  RowArgs a{};
  st = lq::whiten_from_desc(T, K, &a.T);
  if (st != LQ_OK) return st;
  a.rows = rows;
  a.h = x;
  a.hdt = a.vdt = xdt;
  a.ldh = ldx;
  a.K = K;
  a.branch = 1.f;
  a.plain = 1;
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
  using namespace lq;
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
  if (!aligned(h, width(hdt)) ||
      ((r || r_out) && (!aligned(r, width(rdt)) || !aligned(r_out, width(rdt)))) ||
      (n_out && !aligned(n_out, width(ndt))) || !aligned(q, 16) || !aligned(q_scale, 4) ||
      (gate && !aligned(gate->gate, width(gate->dtype))))
    return reject(LQ_EINVAL, "%s: misaligned pointer", me);
  a.rows = rows;
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
