// lq_gemm_i8.cu -- the 8-bit matrix product with a scale per token and per output channel:
//   y[t][n] = (sum_k xq[t][k] wq[n][k]) * (xs[t] * ws[n]) + bias[n]
// The sum is an exact int32 (K <= LQ_MAX_I8_K), so neither its order nor its split over warps
// changes a bit of y.
//
// A weight byte is used once per token. Up to some 250 tokens the weights' stream from HBM bounds
// the product, beyond that the int8 tensor rate. Two kernels:
//
//  * gemv_w8_kernel (few tokens): weights as the A operand of mma.sync m16n8k32 (sixteen rows),
//    tokens as B (eight columns per tile). The order of k inside a sum is free, so a lane loads
//    16 consecutive bytes of its row and of its token and feeds them as the operand words of two
//    MMAs: no shuffles and no shared memory on the way in. One CTA takes sixteen rows, its warps
//    interleaved over K; their int32 partials meet in shared memory.
//  * gemm_w8_kernel (any batch): persistent tcgen05.mma kind::i8 over 128-row x BT-token tiles with
//    two int32 accumulators in tensor memory. The weights are the 128 lanes of the accumulator, so
//    the token tile fits the batch and a warp stores 32 consecutive outputs of a token.
// Every wait on an mbarrier is bounded in time: on expiry the kernel records LQ_ETIMEOUT in the
// workspace status word, the roles leave their loops, in-flight copies and MMAs are waited for
// (again bounded) and tensor memory is released before the CTA exits.
#include <cuda.h>

#include <cstdarg>
#include <cstdio>

#include "lq_device.cuh"
#include "lq_sm100.cuh"

namespace lq {
namespace w8 {

using namespace lq::sm100;

struct Args {
  const int8_t* xq;
  const int8_t* wq;
  const float* xs;
  const float* ws;
  const float* bias;   // or nullptr
  void* y;
  uint32_t* status;
  int64_t ld;          // bytes per row of xq and wq
  int batch, N, K, ydt;
  int nks, tiles_t, tiles;
};

__device__ __forceinline__ void store_y(const Args& a, int64_t i, float v) {
  if (a.ydt == LQ_BF16) static_cast<__nv_bfloat16*>(a.y)[i] = __float2bfloat16_rn(v);
  else if (a.ydt == LQ_F16) static_cast<__half*>(a.y)[i] = __float2half_rn(v);
  else static_cast<float*>(a.y)[i] = v;
}

// ------------------------------------------------------------------ few tokens

constexpr int kGemvWarps = 8;
constexpr int kGemvRows = 16;

__device__ __forceinline__ uint4 ld_weights(const int8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.L2::128B.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

__device__ __forceinline__ void mma_16832(int (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 16 bytes of a token at k; bytes from K on read as zero, whatever the padding holds
__device__ __forceinline__ uint4 ld_token(const int8_t* row, int k, int K) {
  uint4 v = __ldg(reinterpret_cast<const uint4*>(row + k));
  if (k + 16 > K) {
    uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int left = K - (k + 4 * i);
      if (left <= 0) w[i] = 0u;
      else if (left < 4) w[i] &= (1u << (8 * left)) - 1u;
    }
  }
  return v;
}

template <int NT, int U>
__global__ void __launch_bounds__(kGemvWarps * 32)
    gemv_w8_kernel(const __grid_constant__ Args a) {
  __shared__ int part[kGemvWarps][NT][4][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int n0 = blockIdx.x * kGemvRows;
  // rows past N and tokens past the batch repeat the last one; their results are not stored
  const int8_t* w0 = a.wq + (int64_t)min(n0 + g, a.N - 1) * a.ld;
  const int8_t* w1 = a.wq + (int64_t)min(n0 + g + 8, a.N - 1) * a.ld;
  const int8_t* x[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) x[i] = a.xq + (int64_t)min(8 * i + g, a.batch - 1) * a.ld;
  int c[NT][4] = {};
  const int ld = (int)a.ld;
  // a warp's step is U pieces of 64 bytes of each row; the warps take steps in turn
  for (int k0 = warp * 64 * U; k0 < ld; k0 += kGemvWarps * 64 * U) {
    uint4 u0[U], u1[U];
#pragma unroll
    for (int s = 0; s < U; ++s) {
      const int k = k0 + 64 * s + 16 * t;
      u0[s] = u1[s] = make_uint4(0u, 0u, 0u, 0u);
      if (k < ld) {
        u0[s] = ld_weights(w0 + k);
        u1[s] = ld_weights(w1 + k);
      }
    }
#pragma unroll
    for (int s = 0; s < U; ++s) {
      const int k = k0 + 64 * s + 16 * t;
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (k < ld) v = ld_token(x[i], k, a.K);
        mma_16832(c[i], u0[s].x, u1[s].x, u0[s].y, u1[s].y, v.x, v.y);
        mma_16832(c[i], u0[s].z, u1[s].z, u0[s].w, u1[s].w, v.z, v.w);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) part[warp][i][e][lane] = c[i][e];
  __syncthreads();
  // c0, c1: row g, tokens 2t, 2t + 1; c2, c3: row g + 8
  for (int o = threadIdx.x; o < 16 * 8 * NT; o += kGemvWarps * 32) {
    const int r = o & 15, tok = o >> 4;
    const int i = tok >> 3, src = (r & 7) * 4 + ((tok & 7) >> 1), e = (r >> 3) * 2 + (tok & 1);
    int acc = 0;
#pragma unroll
    for (int w = 0; w < kGemvWarps; ++w) acc += part[w][i][e][src];
    const int n = n0 + r;
    if (n < a.N && tok < a.batch) {
      const float v = (float)acc * (a.xs[tok] * a.ws[n]) + (a.bias ? a.bias[n] : 0.f);
      store_y(a, (int64_t)tok * a.N + n, v);
    }
  }
}

// ------------------------------------------------------------------ tensor-core tiles

constexpr int BM = 128;                     // weight rows per tile
constexpr int BK = 128;                     // inputs per stage: one 128-byte row
constexpr int UK = 32;                      // K of one kind::i8 MMA
constexpr int kMaxStages = 8;
constexpr int A_BYTES = BM * BK;
constexpr int kEpiWarps = 4;
constexpr int kTmaWarp = 4;
constexpr int kMmaWarp = 5;
constexpr int kThreads = 6 * 32;
constexpr uint64_t kWaitNs = 2000000000ull;

template <int BT>
struct Tile {
  static constexpr int kStageBytes = A_BYTES + BT * BK;
  static constexpr int kStages = BT == 256 ? 4 : (BT == 128 ? 6 : kMaxStages);
  static constexpr int kTmemCols = 2 * BT;   // a power of two >= 32
};

struct Ctl {
  uint64_t full[kMaxStages];
  uint64_t empty[kMaxStages];
  uint64_t tmem_full[2];
  uint64_t tmem_empty[2];
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
};

template <int BT>
constexpr size_t smem_bytes() {
  return 1024 + (size_t)Tile<BT>::kStages * Tile<BT>::kStageBytes + sizeof(Ctl);
}

__device__ __forceinline__ uint64_t globaltimer() {
  uint64_t t;
  asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
  return t;
}

__device__ __noinline__ bool wait_phase(uint64_t* bar, uint32_t parity, volatile int* abort,
                                        bool honor_abort) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer();
  for (;;) {
#pragma unroll 1
    for (int i = 0; i < 32; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    if (honor_abort && *abort) return false;
    if (globaltimer() - t0 > kWaitNs) return false;
  }
}

__device__ __forceinline__ void give_up(Ctl* ctl, uint32_t* status) {
  *reinterpret_cast<volatile int*>(&ctl->abort) = 1;
  atomicCAS(status, 0u, (uint32_t)LQ_ETIMEOUT);
}

template <int BT>
__global__ void __launch_bounds__(kThreads, 1)
    gemm_w8_kernel(const __grid_constant__ CUtensorMap tmap_w,
                   const __grid_constant__ CUtensorMap tmap_x, const __grid_constant__ Args a) {
  constexpr int NSTAGE = Tile<BT>::kStages, STAGE = Tile<BT>::kStageBytes;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  Ctl* ctl = reinterpret_cast<Ctl*>(smem + (size_t)NSTAGE * STAGE);
  volatile int* abort = &ctl->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < NSTAGE; ++s) {
      mbar_init(&ctl->full[s], 1);
      mbar_init(&ctl->empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&ctl->tmem_full[b], 1);
      mbar_init(&ctl->tmem_empty[b], kEpiWarps * 32);
    }
    mbar_init(&ctl->drain, 1);
    ctl->abort = 0;
    mbar_fence_init();
  }
  if (warp == kMmaWarp) tmem_alloc(&ctl->tmem_base, Tile<BT>::kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;

  if (warp < kEpiWarps) {
    // ---------------------------------------------------------------- epilogue
    int lt = 0;
    for (int tile = blockIdx.x; tile < a.tiles; tile += gridDim.x, ++lt) {
      const int tt = tile % a.tiles_t, tn = tile / a.tiles_t;
      const int b = lt & 1;
      if (!__all_sync(0xffffffffu, wait_phase(&ctl->tmem_full[b], (lt >> 1) & 1, abort, true))) {
        give_up(ctl, a.status);
        break;
      }
      tc_fence_after();
      const int n = tn * BM + warp * 32 + lane;
      const bool ok = n < a.N;
      const float sw = ok ? a.ws[n] : 0.f;
      const float bias = ok && a.bias ? a.bias[n] : 0.f;
#pragma unroll 1
      for (int c = 0; c < BT / 32; ++c) {
        uint32_t r[32];
        tmem_ld_32x32b_x32(tmem + ((uint32_t)(warp * 32) << 16) + (uint32_t)(b * BT + c * 32), r);
        const int t0 = tt * BT + c * 32;
        const float sx = t0 + lane < a.batch ? a.xs[t0 + lane] : 0.f;
        tmem_ld_wait();
        if (c == BT / 32 - 1) {
          tc_fence_before();
          mbar_arrive(&ctl->tmem_empty[b]);
        }
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          const float s = __shfl_sync(0xffffffffu, sx, j) * sw;
          if (ok && t0 + j < a.batch)
            store_y(a, (int64_t)(t0 + j) * a.N + n, (float)(int)r[j] * s + bias);
        }
      }
    }
  } else if (warp == kTmaWarp) {
    // ---------------------------------------------------------------- both operands by TMA
    if (lane == 0) {
      prefetch_tmap(&tmap_w);
      prefetch_tmap(&tmap_x);
      uint32_t ctr = 0;
      bool ok = true;
      for (int tile = blockIdx.x; ok && tile < a.tiles; tile += gridDim.x) {
        const int tt = tile % a.tiles_t, tn = tile / a.tiles_t;
        for (int k = 0; k < a.nks; ++k, ++ctr) {
          const int slot = ctr % NSTAGE;
          if (!wait_phase(&ctl->empty[slot], ((ctr / NSTAGE) & 1) ^ 1, abort, true)) {
            give_up(ctl, a.status);
            ok = false;
            break;
          }
          uint8_t* sa = smem + (size_t)slot * STAGE;
          mbar_arrive_expect_tx(&ctl->full[slot], STAGE);
          tma_load_2d(sa, &tmap_w, &ctl->full[slot], k * BK, tn * BM);
          tma_load_2d(sa + A_BYTES, &tmap_x, &ctl->full[slot], k * BK, tt * BT);
        }
      }
      const uint32_t outstanding = ctr < NSTAGE ? ctr : NSTAGE;
      for (uint32_t i = 0; i < outstanding; ++i) {
        const uint32_t c = ctr - 1 - i;
        if (!wait_phase(&ctl->full[c % NSTAGE], (c / NSTAGE) & 1, abort, false))
          give_up(ctl, a.status);
      }
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    // ---------------------------------------------------------------- MMA issue
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_i8_s32(BM, BT);
      uint32_t ctr = 0;
      bool ok = true;
      int lt = 0;
      for (int tile = blockIdx.x; ok && tile < a.tiles; tile += gridDim.x, ++lt) {
        const int b = lt & 1;
        if (!wait_phase(&ctl->tmem_empty[b], ((lt >> 1) & 1) ^ 1, abort, true)) {
          give_up(ctl, a.status);
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem + (uint32_t)(b * BT);
        for (int k = 0; k < a.nks; ++k, ++ctr) {
          const int slot = ctr % NSTAGE;
          if (!wait_phase(&ctl->full[slot], (ctr / NSTAGE) & 1, abort, true)) {
            give_up(ctl, a.status);
            ok = false;
            break;
          }
          tc_fence_after();
          uint8_t* sa = smem + (size_t)slot * STAGE;
          const uint64_t ad = smem_desc_k_sw128(sa);
          const uint64_t bd = smem_desc_k_sw128(sa + A_BYTES);
#pragma unroll
          for (int kk = 0; kk < BK / UK; ++kk)
            tc_mma_i8(d, ad + 2 * kk, bd + 2 * kk, idesc, (k | kk) != 0);
          tc_commit(&ctl->empty[slot]);
        }
        if (ok) tc_commit(&ctl->tmem_full[b]);
      }
      tc_commit(&ctl->drain);
      if (!wait_phase(&ctl->drain, 0, abort, false)) give_up(ctl, a.status);
    }
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, Tile<BT>::kTmemCols);
}

// ------------------------------------------------------------------ host side

// int8 rows at stride ld as a 2-D map of 128-byte x box_rows tiles; bytes from K on read as zero
bool encode_rows(CUtensorMap* m, const int8_t* p, int64_t K, int64_t rows, int64_t ld,
                 uint32_t box_rows) {
  TensorMapEncodeFn enc = tensor_map_encode_fn();
  if (enc == nullptr) return false;
  const cuuint64_t gdim[2] = {(cuuint64_t)K, (cuuint64_t)rows};
  const cuuint64_t gstride[1] = {(cuuint64_t)ld};
  const cuuint32_t box[2] = {BK, box_rows};
  const cuuint32_t estride[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<int8_t*>(p), gdim, gstride, box,
             estride, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int BT>
cudaError_t launch_tc(Args a, int sms, cudaStream_t st) {
  static int smem_set[64];
  cudaError_t e = ensure_smem((const void*)gemm_w8_kernel<BT>, smem_bytes<BT>(), smem_set);
  if (e != cudaSuccess) return e;
  CUtensorMap tw, tx;
  if (!encode_rows(&tw, a.wq, a.K, a.N, a.ld, BM) || !encode_rows(&tx, a.xq, a.K, a.batch, a.ld, BT))
    return cudaErrorInvalidValue;
  a.nks = (a.K + BK - 1) / BK;
  a.tiles_t = (a.batch + BT - 1) / BT;
  const int64_t tiles = (int64_t)a.tiles_t * ((a.N + BM - 1) / BM);
  if (tiles > (1 << 30)) return cudaErrorInvalidValue;
  a.tiles = (int)tiles;
  gemm_w8_kernel<BT><<<std::min(a.tiles, sms), kThreads, smem_bytes<BT>(), st>>>(tw, tx, a);
  return cudaGetLastError();
}

cudaError_t launch(const Args& a, int route, cudaStream_t st) {
  if (route == LQ_I8_ROUTE_GEMV) {
    const int grid = (a.N + kGemvRows - 1) / kGemvRows;
    if (a.batch <= 8) gemv_w8_kernel<1, 4><<<grid, kGemvWarps * 32, 0, st>>>(a);
    else if (a.batch <= 16) gemv_w8_kernel<2, 4><<<grid, kGemvWarps * 32, 0, st>>>(a);
    else gemv_w8_kernel<4, 2><<<grid, kGemvWarps * 32, 0, st>>>(a);
    return cudaGetLastError();
  }
  const int sms = tc_sm_count();
  if (sms <= 0) return cudaErrorInvalidDevice;
  if (a.batch <= 32) return launch_tc<32>(a, sms, st);
  if (a.batch <= 64) return launch_tc<64>(a, sms, st);
  if (a.batch <= 128) return launch_tc<128>(a, sms, st);
  return launch_tc<256>(a, sms, st);
}

int choose(int32_t batch) {
  return batch <= LQ_I8_GEMV_MAX_BATCH ? LQ_I8_ROUTE_GEMV : LQ_I8_ROUTE_TC;
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

bool al(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

}  // namespace w8
}  // namespace lq

extern "C" {

int32_t lq_gemm_i8_route(int32_t batch, int32_t K, int32_t N) {
  if (batch < 1 || N < 1 || K < 1 || K > LQ_MAX_I8_K) return -1;
  return lq::w8::choose(batch);
}

lq_status lq_gemm_i8(const int8_t* xq, const float* xs, int32_t batch, const int8_t* wq,
                     const float* ws, const float* bias, int32_t K, int32_t N, void* y,
                     lq_dtype ydt, void* workspace, size_t workspace_bytes, int32_t route,
                     lq_stream stream) {
  using namespace lq::w8;
  lq::set_last_error("%s", "");
  if (batch < 0) return reject(LQ_EINVAL, "lq_gemm_i8: batch = %d < 0", batch);
  if (N < 0) return reject(LQ_EINVAL, "lq_gemm_i8: N = %d < 0", N);
  if (K < 1) return reject(LQ_EINVAL, "lq_gemm_i8: K = %d < 1", K);
  if (K > LQ_MAX_I8_K)
    return reject(LQ_EUNSUPPORTED, "lq_gemm_i8: K = %d exceeds LQ_MAX_I8_K (%d)", K, LQ_MAX_I8_K);
  if (ydt != LQ_F32 && ydt != LQ_F16 && ydt != LQ_BF16)
    return reject(LQ_EINVAL, "lq_gemm_i8: unknown y dtype %d", (int)ydt);
  if (route < -1 || route > LQ_I8_ROUTE_TC)
    return reject(LQ_EINVAL, "lq_gemm_i8: unknown route %d", route);
  if (route == LQ_I8_ROUTE_GEMV && batch > LQ_I8_GEMV_MAX_BATCH)
    return reject(LQ_EUNSUPPORTED, "lq_gemm_i8: %d tokens on the GEMV route (at most %d)", batch,
                  LQ_I8_GEMV_MAX_BATCH);
  if (batch == 0 || N == 0) return LQ_OK;
  if (!xq || !xs || !wq || !ws || !y || !workspace)
    return reject(LQ_EINVAL, "lq_gemm_i8: null pointer");
  if (!al(xq, 16) || !al(wq, 16)) return reject(LQ_EINVAL, "lq_gemm_i8: xq or wq not 16-byte aligned");
  if (!al(xs, 4) || !al(ws, 4) || !al(bias, 4) || !al(y, ydt == LQ_F32 ? 4 : 2))
    return reject(LQ_EINVAL, "lq_gemm_i8: misaligned xs, ws, bias or y");
  if (!al(workspace, 256)) return reject(LQ_EINVAL, "lq_gemm_i8: workspace not 256-byte aligned");
  if (workspace_bytes < LQ_GEMM_I8_WORKSPACE_BYTES)
    return reject(LQ_EINVAL, "lq_gemm_i8: workspace of %zu bytes, %d needed", workspace_bytes,
                  LQ_GEMM_I8_WORKSPACE_BYTES);
  Args a{};
  a.xq = xq;
  a.wq = wq;
  a.xs = xs;
  a.ws = ws;
  a.bias = bias;
  a.y = y;
  a.status = &static_cast<lq::WsHeader*>(workspace)->status;
  a.ld = ((int64_t)K + 15) / 16 * 16;
  a.batch = batch;
  a.N = N;
  a.K = K;
  a.ydt = ydt;
  const cudaError_t e = launch(a, route < 0 ? choose(batch) : route, (cudaStream_t)stream);
  return e == cudaSuccess ? LQ_OK : reject(LQ_ECUDA, "lq_gemm_i8: %s", cudaGetErrorString(e));
}

}  // extern "C"
