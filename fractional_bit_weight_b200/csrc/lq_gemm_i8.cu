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
//    take turns over K; their int32 partials meet in shared memory. Measured (device): one token
//    28672 -> 8192 36.4 us, 6.45 TB/s, 0.98 of the copy rate; 4096 -> 4096 3.6 us.
//  * gemm_w8_kernel (any batch): persistent tcgen05.mma kind::i8 over tiles of up to 128 rows x 256
//    tokens (256 x 256 by a pair of CTAs) with two int32 accumulators in tensor memory, operands
//    brought by TMA. The weights are the lanes of the accumulator, so the token tile fits the batch
//    and a warp stores 32 consecutive outputs of a token. Copies and MMAs are issued by an elected
//    lane each (64 tokens x 8192 x 8192: 17.1 us, 21.2 with a lane chosen by its number; 128 x 4096 x
//    4096 8.2 and 10.9).
//    Measured (device): 2048 tokens 8192 -> 28672 292 us, 3.29 Pop/s, tensor pipe 86 % busy at the
//    1.56 GHz that the power limit leaves (341 us in a loop of calls); 16 tokens 28672 -> 8192
//    38.8 us, 6.08 TB/s (0.93 of the copy rate). A layer of few tiles is split along K over the
//    CTAs of a cluster, which add their sums up through distributed shared memory: 32 tokens 8192
//    -> 1024 5.9 us (9.6 unsplit), 20 tokens 28672 -> 1024 9.2 us (26.1).
// Every wait on an mbarrier is bounded in time: on expiry the kernel records LQ_ETIMEOUT in the
// workspace status word, the roles leave their loops, in-flight copies and MMAs are waited for
// (again bounded) and tensor memory is released before the CTA exits. tcgen05.alloc has no limit of
// its own; the shared memory of clusters (kAloneSmem) keeps it from waiting for ever.
#include <cuda.h>

#include <mutex>

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
};

__device__ __forceinline__ void store_y(const Args& a, int64_t i, float v) {
  if (a.ydt == LQ_BF16) static_cast<__nv_bfloat16*>(a.y)[i] = __float2bfloat16_rn(v);
  else if (a.ydt == LQ_F16) static_cast<__half*>(a.y)[i] = __float2half_rn(v);
  else static_cast<float*>(a.y)[i] = v;
}

constexpr int kMaxSplit = 8;   // CTAs of a cluster along K

// What the plans go by: the SMs of the current device and how many clusters of 2, 4 and 8 CTAs are
// resident on them at once (that depends on how the SMs are grouped). Looked up once per device;
// without a device, a B200 with 148 SMs.
struct Machine {
  int sms = 148;
  int clusters[kMaxSplit + 1] = {0, 148, 74, 0, 33, 0, 0, 0, 15};
};

void look_up(int dev, Machine* m);
const Machine& machine() {
  static Machine of[64];
  static std::once_flag seen[64];
  static const Machine none;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
    cudaGetLastError();   // not the error of a later call
    return none;
  }
  std::call_once(seen[dev], look_up, dev, &of[dev]);
  return of[dev];
}

// ------------------------------------------------------------------ few tokens

// Loads that stay behind grid_wait: a read-only (.nc) load may be moved ahead of it.
__device__ __forceinline__ uint4 ld_weights(const int8_t* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.L2::128B.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

__device__ __forceinline__ uint4 ld_token(const int8_t* p) {
  uint4 v;
  asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];"
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
__device__ __forceinline__ uint4 ld_token_end(const int8_t* row, int k, int K) {
  uint4 v = make_uint4(0u, 0u, 0u, 0u);
  if (k >= K) return v;
  v = ld_token(row + k);
  uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int left = K - (k + 4 * i);
    if (left <= 0) w[i] = 0u;
    else if (left < 4) w[i] &= (1u << (8 * left)) - 1u;
  }
  return v;
}

// One CTA: 16 weight rows x 8 NT tokens. Its warps take steps of 64 U inputs in turn, so that the
// CTA reads a few KB of each row at a time.
template <int NT, int U>
__global__ void __launch_bounds__(512) gemv_w8_kernel(const __grid_constant__ Args a) {
  extern __shared__ int part[];   // [warps][NT][4][32]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int n0 = blockIdx.x * 16;
  // rows past N and tokens past the batch repeat the last one; their results are not stored
  const int8_t* w[2];
  const int8_t* x[NT];
#pragma unroll
  for (int h = 0; h < 2; ++h)
    w[h] = a.wq + (int64_t)min(n0 + 8 * h + g, a.N - 1) * a.ld + 16 * t;
#pragma unroll
  for (int i = 0; i < NT; ++i) x[i] = a.xq + (int64_t)min(8 * i + g, a.batch - 1) * a.ld + 16 * t;
  int c[NT][4] = {};
  grid_release();
  grid_wait();
  const int stride = warps * (64 * U);
  int k = warp * (64 * U);
  for (; k + 64 * U <= a.K; k += stride) {
    uint4 u[U][2];
#pragma unroll
    for (int s = 0; s < U; ++s)
#pragma unroll
      for (int h = 0; h < 2; ++h) u[s][h] = ld_weights(w[h] + k + 64 * s);
#pragma unroll
    for (int s = 0; s < U; ++s)
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const uint4 v = ld_token(x[i] + k + 64 * s);
        mma_16832(c[i], u[s][0].x, u[s][1].x, u[s][0].y, u[s][1].y, v.x, v.y);
        mma_16832(c[i], u[s][0].z, u[s][1].z, u[s][0].w, u[s][1].w, v.z, v.w);
      }
  }
  // the warp that holds the ragged last step
#pragma unroll 1
  for (const int end = min(k + 64 * U, (int)a.ld); k < end; k += 64) {
    const bool there = k + 16 * t < (int)a.ld;
    uint4 u[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) u[h] = there ? ld_weights(w[h] + k) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const uint4 v = ld_token_end(x[i] - 16 * t, k + 16 * t, a.K);
      mma_16832(c[i], u[0].x, u[1].x, u[0].y, u[1].y, v.x, v.y);
      mma_16832(c[i], u[0].z, u[1].z, u[0].w, u[1].w, v.z, v.w);
    }
  }
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) part[((warp * NT + i) * 4 + e) * 32 + lane] = c[i][e];
  __syncthreads();
  // c0, c1: row g, tokens 2t, 2t + 1; c2, c3: row g + 8
  for (int o = threadIdx.x; o < 16 * 8 * NT; o += blockDim.x) {
    const int r = o % 16, tok = o / 16, n = n0 + r;
    if (n >= a.N || tok >= a.batch) continue;
    const int slot =
        ((tok >> 3) * 4 + (r >> 3) * 2 + (tok & 1)) * 32 + (r & 7) * 4 + ((tok & 7) >> 1);
    int acc = 0;
    for (int v = 0; v < warps; ++v) acc += part[v * (NT * 128) + slot];
    store_y(a, (int64_t)tok * a.N + n,
            (float)acc * (a.xs[tok] * a.ws[n]) + (a.bias ? a.bias[n] : 0.f));
  }
}

template <int NT, int U>
cudaError_t launch_gemv(const Args& a, cudaStream_t st) {
  const int ctas = (a.N + 15) / 16;
  // Up to 31 warps per SM, which registers let be resident at once, but four to a CTA at least, and
  // some steps for each. One token x 8192 x 10240: 18.0 us with four warps (17 per SM), 19.2 with
  // eight (35); 8192 x 28672: 41.0 with four (48), 42.4 with two (24).
  const int most = 31 * machine().sms;
  int warps = 16;
  while ((warps > 4 && (int64_t)ctas * warps > most) || (warps > 1 && (warps / 2) * 64 * U >= a.K))
    warps /= 2;
  const size_t smem = (size_t)warps * NT * 128 * sizeof(int);
  static int smem_set[64];
  const cudaError_t e = ensure_smem((const void*)gemv_w8_kernel<NT, U>, smem, smem_set);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(warps * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, gemv_w8_kernel<NT, U>, a);
}

// ------------------------------------------------------------------ tensor-core tiles

constexpr int kMmaM = 128;                  // rows of one MMA (lanes of tensor memory)
constexpr int kMaxTokens = 256;             // columns of one MMA
constexpr int BK = 128;                     // inputs per chunk: one 128-byte swizzle row
constexpr int UK = 32;                      // K of one kind::i8 MMA
constexpr int kMaxStages = 16;
constexpr int kMaxChunks = 8;               // chunks per stage
constexpr int kEpiWarps = 4;
constexpr int kWeightWarp = 4;              // fetches weights
constexpr int kTokenWarp = 5;               // fetches tokens
constexpr int kMmaWarp = 6;
constexpr int kThreads = 7 * 32;
constexpr int kTmemCols = 2 * kMaxTokens;
constexpr uint64_t kWaitNs = 2000000000ull;

// kOne: one CTA per tile. kPair: two CTAs on one tile of twice the rows. kSplit: a cluster of CTAs
// on one tile, each over a part of K.
enum Kind { kOne, kPair, kSplit };   // LQ_I8_ROUTE_TC and the routes behind it

// One call's tiles over all of K, in stages of `chunks` 128-byte chunks. A tile is `tokens` tokens
// x `rows` weight rows per CTA (a pair of CTAs takes twice the rows, and each fetches half of the
// tokens). A stage in shared memory: [chunks][rows][128 B], then [chunks][fetched tokens][128 B].
struct Plan {
  int kind;                  // kOne, kPair, kSplit
  int split, cols;           // kSplit: CTAs along K, tokens that each of them finishes (of 4)
  int rows, tokens;          // at most 128 and 256; multiples of 8 and of 16 (pairs: 32)
  int tiles_n, tiles_t, tiles;
  int chunks, nks, stages;   // chunks per stage, stages per tile, ring slots
  int wide;                  // K a multiple of 128: one copy brings a stage's chunks of an operand
  int a_bytes, stage_bytes;  // the weights of a stage; all of it
  size_t smem;
};

struct alignas(16) Ctl {
  uint64_t full[kMaxStages];
  uint64_t empty[kMaxStages];
  uint64_t tmem_full[2];
  uint64_t tmem_empty[2];
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
  float scale[kEpiWarps][kMaxTokens];   // each epilogue warp's copy of its tile's token scales
};

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

// A place in the ring of stages and the parity of its barriers there.
struct Slot {
  int at = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void next(int stages) {
    if (++at == stages) {
      at = 0;
      parity ^= 1;
    }
  }
};

// One output element's conversion: values of lanes l and l ^ 1 (neighbouring channels) of two
// tokens become one 4-byte store per lane.
template <class YT>
__device__ __forceinline__ uint32_t pack_y(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack_y<__half>(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t pack_y<__nv_bfloat16>(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ void put_y(float* p, float v) { *p = v; }
__device__ __forceinline__ void put_y(__half* p, float v) { *p = __float2half_rn(v); }
__device__ __forceinline__ void put_y(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// 32 tokens of one warp's 32 rows: lane = output channel, r = the tokens' sums, nt of them there.
// A token's 32 channels are neighbours in y, so the lanes of a store fall on consecutive
// addresses; 16-bit outputs go out two channels per lane, two tokens per store (pairs).
template <class YT>
__device__ __forceinline__ void write_32(const uint32_t (&r)[32], YT* y, int64_t N, bool ok, int nt,
                                         const float* sx, float sw, float bias, bool pairs) {
  const bool odd = threadIdx.x & 1;
  float v[32];
#pragma unroll
  for (int j = 0; j < 32; j += 4) {
    const float4 s = *reinterpret_cast<const float4*>(sx + j);
    v[j] = fmaf((float)(int)r[j], s.x * sw, bias);
    v[j + 1] = fmaf((float)(int)r[j + 1], s.y * sw, bias);
    v[j + 2] = fmaf((float)(int)r[j + 2], s.z * sw, bias);
    v[j + 3] = fmaf((float)(int)r[j + 3], s.w * sw, bias);
  }
  if constexpr (sizeof(YT) == 2) {
    if (pairs && nt >= 32) {
      uint32_t* y2 = reinterpret_cast<uint32_t*>(y + (odd ? N - 1 : 0));
#pragma unroll
      for (int j = 0; j < 32; j += 2) {
        const float other = __shfl_xor_sync(0xffffffffu, odd ? v[j] : v[j + 1], 1);
        if (ok) *y2 = odd ? pack_y<YT>(other, v[j + 1]) : pack_y<YT>(v[j], other);
        y2 += N;   // two rows of y, in pairs of channels
      }
      return;
    }
  }
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    if (ok && j < nt) put_y(y, v[j]);
    y += N;
  }
}

// One warp's 32 rows of a finished tile: columns = tokens t0 .. t0 + nt. The next 32 columns leave
// tensor memory while the last ones are written.
template <class YT>
__device__ __forceinline__ void write_tile(const Args& a, uint32_t taddr, int n, bool ok, int t0,
                                           int nt, const float* sx, float sw, float bias) {
  const bool pairs = sizeof(YT) == 2 && a.N % 2 == 0 && reinterpret_cast<uintptr_t>(a.y) % 4 == 0;
  YT* y = static_cast<YT*>(a.y) + (int64_t)t0 * a.N + n;
  uint32_t r0[32], r1[32];
  tmem_ld_32x32b_x32(taddr, r0);
#pragma unroll 1
  for (int c = 0; c < nt; c += 64) {
    tmem_ld_wait();
    if (c + 32 < nt) tmem_ld_32x32b_x32(taddr + (uint32_t)(c + 32), r1);
    write_32<YT>(r0, y + (int64_t)c * a.N, a.N, ok, nt - c, sx + c, sw, bias, pairs);
    if (c + 32 >= nt) break;
    tmem_ld_wait();
    if (c + 64 < nt) tmem_ld_32x32b_x32(taddr + (uint32_t)(c + 64), r0);
    write_32<YT>(r1, y + (int64_t)(c + 32) * a.N, a.N, ok, nt - c - 32, sx + c + 32, sw, bias, pairs);
  }
}

// The token scales of token tile tt into a warp's copy, zero behind the batch.
__device__ __forceinline__ void load_scales(const Args& a, const Plan& p, int tt, float* sx) {
  const int t0 = tt * p.tokens;
  for (int i = threadIdx.x & 31; i < p.tokens; i += 32)
    sx[i] = t0 + i < a.batch ? a.xs[t0 + i] : 0.f;
  __syncwarp();
}

// kSplit: this warp's 32 rows of the CTA's partial sums, four tokens at a time to the CTA of the
// cluster that finishes them: part there is [CTA they come from][its tokens / 4][128 rows][4].
__device__ __forceinline__ void send_partials(uint32_t taddr, int* part, const Plan& p, int krank,
                                              int row, int nt) {
  int to = 0, col = 0;
#pragma unroll 1
  for (int c = 0; c < nt; c += 32) {
    uint32_t r[32];
    tmem_ld_32x32b_x32(taddr + (uint32_t)c, r);
    tmem_ld_wait();
#pragma unroll
    for (int j = 0; j < 32; j += 4) {
      if (c + j < nt) {
        const uint32_t at = cluster_addr(part + (krank * p.cols + col) * kMmaM + row * 4, to);
        asm volatile("st.shared::cluster.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(r[j]),
                     "r"(r[j + 1]), "r"(r[j + 2]), "r"(r[j + 3])
                     : "memory");
      }
      col += 4;
      if (col == p.cols) {
        col = 0;
        ++to;
      }
    }
  }
}

template <class YT>
__device__ __forceinline__ void finish_split(const Args& a, const Plan& p, const int* part,
                                             int krank, int row, int n, int t0, int nt,
                                             const float* sx, float sw, float bias) {
  const int first = krank * p.cols, end = min(p.cols, nt - first);
  YT* y = static_cast<YT*>(a.y) + (int64_t)(t0 + first) * a.N + n;
  for (int c = 0; c < end; c += 4) {
    int4 sum = make_int4(0, 0, 0, 0);
    for (int s = 0; s < p.split; ++s) {
      const int4 v = *reinterpret_cast<const int4*>(part + (s * p.cols + c) * kMmaM + row * 4);
      sum.x += v.x;
      sum.y += v.y;
      sum.z += v.z;
      sum.w += v.w;
    }
    const int total[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (c + j < end)
        put_y(y + (int64_t)(c + j) * a.N, fmaf((float)total[j], sx[first + c + j] * sw, bias));
  }
}

// An MMA always takes 128 rows of A from a CTA's shared memory. A tile of fewer rows leaves the
// rest to whatever lies behind it there (the ring ends 16 KB before the allocation does): those
// lanes of the accumulator are never read.
//
// kPair: two CTAs work on one tile of twice the rows (cta_group::2). The even CTA's barriers count
// the copies of both, its MMA thread issues for both, and commits arrive in both. Each SM then
// reads and fills 16 KB less shared memory per 128 inputs of a 256-token tile: one CTA alone moves
// 24 KB per MMA through it, 192 clocks against the MMA's 128.
//
// kSplit: each CTA of a cluster sums its part of K of the same tile, then they hand the int32
// partials out over distributed shared memory, every CTA finishing a range of the tokens. For
// layers too small to fill the SMs with tiles, whose time would be one SM's way through all of K.
template <int KIND>
__global__ void __launch_bounds__(kThreads, 1)
    gemm_w8_kernel(const __grid_constant__ CUtensorMap tmap_w,
                   const __grid_constant__ CUtensorMap tmap_x, const __grid_constant__ Args a,
                   const __grid_constant__ Plan p) {
  constexpr bool PAIR = KIND == kPair, SPLIT = KIND == kSplit;
  extern __shared__ uint8_t smem_raw[];
  Ctl* ctl = reinterpret_cast<Ctl*>(smem_raw);
  uint8_t* ring = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw + sizeof(Ctl)) + 1023) & ~static_cast<uintptr_t>(1023));
  volatile int* abort = &ctl->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kCtas = PAIR ? 2 : 1;
  const int rank = PAIR ? (int)(blockIdx.x & 1) : 0;    // clusters are consecutive pairs
  const int group = PAIR ? 2 : SPLIT ? p.split : 1;     // CTAs of a tile
  const int krank = SPLIT ? (int)blockIdx.x % group : 0;
  const int first = (int)blockIdx.x / group, step = (int)gridDim.x / group;

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&ctl->full[s], 2);   // the two fetching lanes
      mbar_init(&ctl->empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&ctl->tmem_full[b], 1);
      mbar_init(&ctl->tmem_empty[b], kCtas * kEpiWarps);
    }
    mbar_init(&ctl->drain, 1);
    ctl->abort = 0;
    mbar_fence_init();
  }
  if (warp == kMmaWarp) {
    if constexpr (PAIR) tmem_alloc_pair(&ctl->tmem_base, kTmemCols);
    else tmem_alloc(&ctl->tmem_base, kTmemCols);
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync();   // both CTAs' barriers are set up
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;
  grid_release();
  grid_wait();

  if (warp < kEpiWarps) {
    // ---------------------------------------------------------------- epilogue
    int lt = 0;
    if constexpr (SPLIT) {
      load_scales(a, p, first % p.tiles_t, ctl->scale[warp]);
      if (!__all_sync(0xffffffffu, wait_phase(&ctl->tmem_full[0], 0, abort, true)))
        give_up(ctl, a.status);
    }
    for (int tile = first; !SPLIT && tile < p.tiles; tile += step, ++lt) {
      const int tn = tile / p.tiles_t, tt = tile - tn * p.tiles_t;
      const int b = lt & 1;
      const int row = warp * 32 + lane, n = (tn * kCtas + rank) * p.rows + row;
      const bool ok = row < p.rows && n < a.N;
      const int t0 = tt * p.tokens, nt = min(p.tokens, a.batch - t0);
      // the scales are on their way while the tile is summed
      const float sw = ok ? a.ws[n] : 0.f;
      const float bias = ok && a.bias ? a.bias[n] : 0.f;
      float* sx = ctl->scale[warp];
      __syncwarp();
      load_scales(a, p, tt, sx);
      if (!__all_sync(0xffffffffu, wait_phase(&ctl->tmem_full[b], (lt >> 1) & 1, abort, true))) {
        give_up(ctl, a.status);
        break;
      }
      tc_fence_after();
      if (warp * 32 < p.rows) {
        const uint32_t taddr = tmem + ((uint32_t)(warp * 32) << 16) + (uint32_t)(b * kMaxTokens);
        if (a.ydt == LQ_BF16) write_tile<__nv_bfloat16>(a, taddr, n, ok, t0, nt, sx, sw, bias);
        else if (a.ydt == LQ_F16) write_tile<__half>(a, taddr, n, ok, t0, nt, sx, sw, bias);
        else write_tile<float>(a, taddr, n, ok, t0, nt, sx, sw, bias);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (PAIR) mbar_arrive_cluster(cluster_addr(&ctl->tmem_empty[b], 0));
        else mbar_arrive(&ctl->tmem_empty[b]);
      }
    }
  } else if (warp == kWeightWarp || warp == kTokenWarp) {
    // ---------------------------------------------------------------- operands by TMA
    if (elect_one()) {
      const bool weights = warp == kWeightWarp;
      const CUtensorMap* tmap = weights ? &tmap_w : &tmap_x;
      prefetch_tmap(tmap);
      const int rows = weights ? p.rows : p.tokens / kCtas;
      uint8_t* base = ring + (weights ? 0 : p.a_bytes);
      const uint32_t bytes = kCtas * p.chunks * rows * BK;
      Slot slot;
      uint32_t issued = 0;
      bool ok = true;
      for (int tile = first; ok && tile < p.tiles; tile += step) {
        const int tn = tile / p.tiles_t, tt = tile - tn * p.tiles_t;
        const int row = ((weights ? tn : tt) * kCtas + rank) * rows;
        for (int k = 0; k < p.nks; ++k, slot.next(p.stages), ++issued) {
          if (!wait_phase(&ctl->empty[slot.at], slot.parity ^ 1, abort, true)) {
            give_up(ctl, a.status);
            ok = false;
            break;
          }
          uint8_t* at = base + slot.at * p.stage_bytes;
          const int ks = krank * p.nks + k;   // past the end of K a copy brings zeros
          if (rank == 0) mbar_arrive_expect_tx(&ctl->full[slot.at], bytes);
          const uint32_t full = PAIR ? cluster_addr(&ctl->full[slot.at], 0) : 0u;
          for (int c = 0; c < (p.wide ? 1 : p.chunks); ++c) {
            const int x = p.wide ? 0 : (ks * p.chunks + c) * BK, z = p.wide ? ks * p.chunks : 0;
            if constexpr (PAIR) tma_load_3d_pair(at + c * rows * BK, tmap, full, x, row, z);
            else tma_load_3d(at + c * rows * BK, tmap, &ctl->full[slot.at], x, row, z);
          }
        }
      }
      // What still arrives at this CTA's barriers does so before it leaves: another CTA may have live
      // barriers in the same place by then. Commits free the last stages in both CTAs of a pair, and
      // a freed stage's copies have landed. After an abort nothing frees them: then the copies in
      // flight are waited for (a stage of which only one operand was asked for never completes: a
      // bounded wait).
      const uint32_t last = min(issued, (uint32_t)p.stages);
      bool freed = ok && weights;
      for (uint32_t i = last; freed && i > 0; --i) {
        const uint32_t c = issued - i;
        freed = wait_phase(&ctl->empty[c % p.stages], (c / p.stages) & 1, abort, true);
        if (!freed) give_up(ctl, a.status);
      }
      if (rank == 0 && !freed) {
        for (uint32_t i = last; i > 0; --i) {
          const uint32_t c = issued - i;
          if (!wait_phase(&ctl->full[c % p.stages], (c / p.stages) & 1, abort, false))
            give_up(ctl, a.status);
        }
      }
      // the even CTA's last commit, which arrives here too
      if (rank == 1 && weights && !wait_phase(&ctl->drain, 0, abort, false)) give_up(ctl, a.status);
    }
    __syncwarp();
  } else if (warp == kMmaWarp && rank == 0) {
    // ---------------------------------------------------------------- MMA issue
    if (elect_one()) {
      const uint32_t idesc = idesc_i8_s32(kCtas * kMmaM, p.tokens);
      auto commit = [](uint64_t* bar) {
        if constexpr (PAIR) tc_commit_pair(bar);
        else tc_commit(bar);
      };
      Slot slot;
      bool ok = true;
      int lt = 0;
      const uint64_t desc = smem_desc_k_sw128(ring);
      const uint32_t desc_stage = p.stage_bytes >> 4;
      const uint32_t chunk_a = p.rows * BK >> 4, chunk_b = p.tokens / kCtas * BK >> 4;
      for (int tile = first; ok && tile < p.tiles; tile += step, ++lt) {
        const int b = lt & 1;
        if (!wait_phase(&ctl->tmem_empty[b], ((lt >> 1) & 1) ^ 1, abort, true)) {
          give_up(ctl, a.status);
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem + (uint32_t)(b * kMaxTokens);
        uint32_t more = 0;   // the tile's first MMA overwrites the accumulator
        for (int k = 0; k < p.nks; ++k, slot.next(p.stages)) {
          if (!wait_phase(&ctl->full[slot.at], slot.parity, abort, true)) {
            give_up(ctl, a.status);
            ok = false;
            break;
          }
          tc_fence_after();
          uint64_t ad = desc + (uint32_t)slot.at * desc_stage, bd = ad + (p.a_bytes >> 4);
          for (int c = 0; c < p.chunks; ++c, ad += chunk_a, bd += chunk_b) {
#pragma unroll
            for (int kk = 0; kk < BK / UK; ++kk) {
              if constexpr (PAIR) tc_mma_i8_pair(d, ad + 2 * kk, bd + 2 * kk, idesc, more);
              else tc_mma_i8(d, ad + 2 * kk, bd + 2 * kk, idesc, more);
              more = 1;
            }
          }
          commit(&ctl->empty[slot.at]);
        }
        if (ok) commit(&ctl->tmem_full[b]);
      }
      commit(&ctl->drain);
      if (!wait_phase(&ctl->drain, 0, abort, false)) give_up(ctl, a.status);
    }
    __syncwarp();
  }

  if constexpr (SPLIT) {
    tc_fence_before();
    __syncthreads();
    cluster_sync();   // all MMAs of the cluster are done: the rings hold partials from here on
    tc_fence_after();
    int* part = reinterpret_cast<int*>(ring);
    const int tn = first / p.tiles_t, t0 = (first - tn * p.tiles_t) * p.tokens;
    const int nt = min(p.tokens, a.batch - t0), row = warp * 32 + lane, n = tn * p.rows + row;
    const bool ok = warp < kEpiWarps && row < p.rows && n < a.N;
    const float sw = ok ? a.ws[n] : 0.f, bias = ok && a.bias ? a.bias[n] : 0.f;
    if (warp < kEpiWarps && warp * 32 < p.rows)
      send_partials(tmem + ((uint32_t)(warp * 32) << 16), part, p, krank, row, nt);
    cluster_sync();
    if (ok) {
      const float* sx = ctl->scale[warp];
      if (a.ydt == LQ_BF16)
        finish_split<__nv_bfloat16>(a, p, part, krank, row, n, t0, nt, sx, sw, bias);
      else if (a.ydt == LQ_F16)
        finish_split<__half>(a, p, part, krank, row, n, t0, nt, sx, sw, bias);
      else
        finish_split<float>(a, p, part, krank, row, n, t0, nt, sx, sw, bias);
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync();   // neither CTA's memory is in use by the other any more
  tc_fence_after();
  if (warp == kMmaWarp) {
    if constexpr (PAIR) tmem_dealloc_pair(tmem, kTmemCols);
    else tmem_dealloc(tmem, kTmemCols);
  }
}

// ------------------------------------------------------------------ host side

constexpr size_t kMaxSmem = 227 * 1024;
// More than half of what an SM has (228 KB, 1 KB of it taken by each CTA): two CTAs of this size
// never share one. A CTA of a cluster keeps its tensor memory until its peers have allocated theirs.
// If CTAs of clusters X and Y shared two SMs, X's could hold one and wait for the other while Y's did
// the reverse, and tcgen05.alloc waits without a limit. So every cluster asks for this much. A CTA
// without a cluster may share an SM with any: with its tensor memory held it waits only (in grid_wait)
// for kernels ahead of it on its stream, and those let it start when all their CTAs had theirs.
constexpr size_t kAloneSmem = kMaxSmem / 2 + 1024;
constexpr int kSplitTokens = 128;           // tokens of a kSplit tile: its partials fit the ring
constexpr int32_t kMost = 1 << 30;          // tokens, rows: tile coordinates stay in 32 bits

// The tile of a call. Rows of a tile are chosen so that its tiles fill whole waves of the SMs: few
// rows cost nothing while the weights' stream bounds the call. Token tiles, rows, CTA pairs and
// clusters along K are compared by an estimate in clocks: per 128 inputs 1.22 for each 128-byte row
// that an SM fetches into shared memory or reads out of it for the MMAs (those take 2 per token, less
// than that); per wave 5050; for the last epilogue 39 per token; for a pair's start 2600. It is
// fitted to sweeps of all tiles over 13 layers of 1024 x 1024 to 8192 x 28672 with 17 batches of 20
// to 4096 tokens: the tile it picks is within 1.0 % of the fastest on average, 4 % in nine of ten,
// 15 % at worst. Pairs against single CTAs: 2048 x 8192 x 28672 293 against 344 us, 256 x 5120 x 5120
// 13.2 against 14.5; and 128 x 4096 x 4096 10.2 against 8.2, 32 x 8192 x 8192 15.4 against 15.0.
//
// Clusters along K are taken while they are all resident at once: the sixteenth cluster of 8 waits
// for the first (15 of them 8.2 us, 16 14.6), as the 34th of 4 does (33 10.9, 34 19.1). Split
// against whole: 32 x 8192 x 1024 5.9 against 9.6 us, 20 x 28672 x 1024 9.2 against 26.1, 64 x 14336
// x 4096 14.9 against 18.5; and 24 x 1024 x 1024 4.3 against 3.5, 64 x 8192 x 8192 16.5 against 15.8.
Plan make_plan(int batch, int K, int N, int force = -1) {
  const Machine& m = machine();
  const int sms = m.sms;
  Plan best{};
  double best_cost = 0;
  const int chunks_k = (K + BK - 1) / BK;
  auto consider = [&](int kind, int split, int rows, int tokens, int64_t tn, int tt, int64_t waves) {
    const int shared = kind == kPair ? 2 : 1;          // CTAs that share a tile's tokens
    const int fetched = rows + tokens / shared;
    const double step = 1.22 * (kMmaM + tokens / shared + fetched);
    double cost;
    if (kind == kSplit)
      cost = (double)waves * (1.4 * ((chunks_k + split - 1) / split) * step + 55.0 * tokens +
                              27.0 * tokens / split + 7000);
    else
      cost = (double)waves * (chunks_k * step + 5050) + 39.0 * tokens + (kind == kPair ? 2600.0 : 0.0);
    if (best.tokens != 0 && cost >= best_cost) return;
    best_cost = cost;
    best.kind = kind;
    best.split = split;
    best.rows = rows;
    best.tokens = tokens;
    best.tiles_n = (int)tn;
    best.tiles_t = tt;
  };
  for (int kind : {kOne, kPair}) {
    if (force >= 0 && kind != force) continue;
    const int ctas = kind == kPair ? 2 : 1, units = sms / ctas, unit = 16 * ctas;
    // Small layers like small tiles: with ten against four counts of token tiles 1024 x 1024 x 1024
    // takes 5.9 against 8.5 us, 400 x 17792 x 1364 20.1 against 26.6.
    int last = 0;
    for (int tiles_t = (batch + kMaxTokens - 1) / kMaxTokens, tries = 0; tries < 10; ++tiles_t, ++tries) {
      const int tokens = ((batch + tiles_t - 1) / tiles_t + unit - 1) / unit * unit;
      if (tokens == last) continue;
      last = tokens;
      const int tt = (batch + tokens - 1) / tokens;
      // the fewest waves whose tiles have at most 128 rows per CTA
      const int64_t full = (int64_t)tt * ((N + ctas * kMmaM - 1) / (ctas * kMmaM));
      int64_t waves = (full + units - 1) / units;
      int64_t tn = std::max<int64_t>(1, waves * units / tt);
      int rows = (int)((N + ctas * tn - 1) / (ctas * tn) + 7) / 8 * 8;
      // nearly full tiles are faster full (512 x 4096 x 4096: 13.9 against 15.4 us at 112 rows)
      if (rows * 8 >= kMmaM * 7) rows = kMmaM;
      tn = (N + ctas * rows - 1) / (ctas * rows);
      waves = (tn * tt + units - 1) / units;
      consider(kind, 1, rows, tokens, tn, tt, waves);
    }
  }
  // clusters along K: the fewest tokens with which all of them are resident at once
  for (int split = 2; split <= kMaxSplit && (force < 0 || force == kSplit); split *= 2) {
    const int64_t full = (N + kMmaM - 1) / kMmaM, fit = std::max(1, m.clusters[split]);
    const int64_t most = std::max<int64_t>(1, fit / full);       // token tiles
    const int tokens = (int)std::min<int64_t>(kSplitTokens, ((batch + most - 1) / most + 15) / 16 * 16);
    const int tt = (batch + tokens - 1) / tokens;
    // tiles of 128 rows, or of fewer on all SMs
    for (int64_t tn : {full, fit / tt}) {
      if (tn < full) continue;
      const int rows = (int)((N + tn - 1) / tn + 7) / 8 * 8;
      tn = (N + rows - 1) / rows;
      const int64_t waves = (tn * tt + fit - 1) / fit;
      if (force >= 0 || waves == 1) consider(kSplit, split, rows, tokens, tn, tt, waves);
    }
  }
  const int fetched = best.tokens / (best.kind == kPair ? 2 : 1);
  best.tiles = best.tiles_n * best.tiles_t;
  best.cols = ((best.tokens + best.split - 1) / best.split + 3) / 4 * 4;
  // stages of up to 48 KB, four of them at least
  best.chunks = std::max(1, std::min({kMaxChunks, (chunks_k + best.split - 1) / best.split,
                                      48 * 1024 / ((best.rows + fetched) * BK)}));
  best.wide = K % BK == 0;
  best.a_bytes = best.chunks * best.rows * BK;
  best.stage_bytes = best.a_bytes + best.chunks * fetched * BK;
  best.nks = ((chunks_k + best.chunks - 1) / best.chunks + best.split - 1) / best.split;
  const size_t fixed = sizeof(Ctl) + 1024 + (size_t)kMmaM * BK;
  best.stages = (int)std::min<size_t>(kMaxStages, (kMaxSmem - fixed) / best.stage_bytes);
  size_t ring = (size_t)best.stages * best.stage_bytes;
  if (best.kind == kSplit)   // the partials take the ring's place
    ring = std::max(ring, (size_t)best.split * best.cols * kMmaM * sizeof(int));
  best.smem = fixed + ring;
  if (best.kind != kOne) best.smem = std::max(best.smem, kAloneSmem);
  return best;
}

// int8 rows at stride ld as a 3-D map of boxes of box_rows x `chunks` 128-byte chunks. With K a
// multiple of 128 the third axis counts the chunks of a row; else it has one entry, a box one
// chunk, and the bytes from K on read as zero.
bool encode_rows(CUtensorMap* m, const int8_t* p, int64_t K, int64_t rows, int64_t ld, int box_rows,
                 int chunks) {
  TensorMapEncodeFn enc = tensor_map_encode_fn();
  if (enc == nullptr) return false;
  const bool wide = K % BK == 0;
  const cuuint64_t gdim[3] = {(cuuint64_t)(wide ? BK : K), (cuuint64_t)rows,
                              (cuuint64_t)(wide ? K / BK : 1)};
  const cuuint64_t gstride[2] = {(cuuint64_t)ld, (cuuint64_t)(wide ? BK : ld)};
  const cuuint32_t box[3] = {BK, (cuuint32_t)box_rows, (cuuint32_t)(wide ? chunks : 1)};
  const cuuint32_t estride[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<int8_t*>(p), gdim, gstride, box,
             estride, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

const void* const kKernels[3] = {(const void*)gemm_w8_kernel<kOne>,
                                 (const void*)gemm_w8_kernel<kPair>,
                                 (const void*)gemm_w8_kernel<kSplit>};

// The tile kernels' limits of shared memory: one size, whatever the plan.
cudaError_t allow_smem(int kind) {
  static int smem_set[3][64];
  return ensure_smem(kKernels[kind], kMaxSmem, smem_set[kind]);
}

void look_up(int dev, Machine* m) {
  int n = 0;
  cudaError_t e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess && n > 0) m->sms = n;
  if (e == cudaSuccess) e = allow_smem(kSplit);
  for (int split = 2; split <= kMaxSplit && e == cudaSuccess; split *= 2) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(split * m->sms);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kMaxSmem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = split;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(&n, kKernels[kSplit], &cfg);
    if (e == cudaSuccess && n > 0) m->clusters[split] = n;
  }
  if (e != cudaSuccess) cudaGetLastError();   // the launch that follows reports its own
}

cudaError_t launch_tc(const Args& a, int force, cudaStream_t st) {
  if ((int64_t)((a.N + 127) / 128) * ((a.batch + 15) / 16) > (1 << 30)) return cudaErrorInvalidValue;
  const Plan p = make_plan(a.batch, a.K, a.N, force);
  const cudaError_t e = allow_smem(p.kind);
  if (e != cudaSuccess) return e;
  const int shared = p.kind == kPair ? 2 : 1;              // CTAs that share a tile's tokens
  const int group = p.kind == kPair ? 2 : p.split;         // CTAs of a cluster
  if ((int64_t)p.tiles * group > INT32_MAX) return cudaErrorInvalidValue;
  CUtensorMap tw, tx;
  if (!encode_rows(&tw, a.wq, a.K, a.N, a.ld, p.rows, p.chunks) ||
      !encode_rows(&tx, a.xq, a.K, a.batch, a.ld, p.tokens / shared, p.chunks))
    return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg{};
  // persistent, except that a cluster along K takes one tile
  cfg.gridDim = dim3(group * (p.kind == kSplit ? p.tiles : std::min(p.tiles, machine().sms / group)));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = p.smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = group;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = group > 1 ? 2 : 1;
  return p.kind == kPair    ? cudaLaunchKernelEx(&cfg, gemm_w8_kernel<kPair>, tw, tx, a, p)
         : p.kind == kSplit ? cudaLaunchKernelEx(&cfg, gemm_w8_kernel<kSplit>, tw, tx, a, p)
                            : cudaLaunchKernelEx(&cfg, gemm_w8_kernel<kOne>, tw, tx, a, p);
}

// Few tokens go to the GEMV, whose start is shorter: at 8 tokens 2.9 against 4.7 us on 4096 x 1024,
// 37.9 against 38.6 us on 28672 x 8192. Its loads of the tokens grow with the batch: at 16 tokens
// 4.9 against 6.5 us on 4096 x 4096, 11.8 against 12.2 on 12288 x 4096, but 14.1 against 13.9 on
// 14336 x 4096, 15.0 against 14.3 on 8192 x 8192 and 43.3 against 38.7 us on 28672 x 8192. With a
// CTA per 16 rows it leaves half the SMs idle on a layer of up to 1184 rows, where clusters along K
// win on long ones: at one token 3.8 against 5.1 us on 8192 x 1024, 6.1 against 6.1 us on 14336 x
// 1024, 12.5 against 8.6 us on 28672 x 1024. Eight of its CTAs are resident per SM. On layers that give
// it more, the second wave is short of CTAs, and the persistent tiles lose nothing between theirs: at
// one token 24.7 against 25.6 us on 8192 x 18432 (1152 CTAs), but 33.8 against 28.9 on 8192 x 20480
// (1280), 37.6 against 33.9 on 8192 x 24576, 40.2 against 39.1 on 8192 x 28672, 40.6 against 34.0 on
// 10240 x 20480; at eight tokens 25.4 against 26.1 on 8192 x 18432, 33.4 against 29.2 on 8192 x 20480.
// Not with short rows, whose waves are short: 29.9 against 28.7 us on 6144 x 28672, 33.9 against 34.1
// on 6144 x 34816, 32.1 against 33.4 on 4096 x 50432.
bool few_tokens(int32_t batch, int32_t K, int32_t N) {
  const int64_t weights = (int64_t)N * K;
  if (batch > LQ_I8_GEMV_MAX_BATCH || (N <= 16 * (machine().sms / 2) && K > 14336)) return false;
  if (N > 16 * 8 * machine().sms && K >= 8192) return false;
  return batch <= 8 || weights <= 54 * 1000 * 1000;
}

cudaError_t launch(const Args& a, int route, cudaStream_t st) {
  if (route < 0 ? few_tokens(a.batch, a.K, a.N) : route == LQ_I8_ROUTE_GEMV) {
    if (a.batch <= 8) return launch_gemv<1, 2>(a, st);
    return launch_gemv<2, 4>(a, st);
  }
  return launch_tc(a, route < 0 ? -1 : route - LQ_I8_ROUTE_TC, st);   // the kinds in route order
}

}  // namespace w8
}  // namespace lq

extern "C" {

int32_t lq_gemm_i8_route(int32_t batch, int32_t K, int32_t N) {
  using namespace lq;
  using namespace lq::w8;
  if (batch < 1 || N < 1 || K < 1 || K > LQ_MAX_I8_K || batch > kMost || N > kMost) return -1;
  if (few_tokens(batch, K, N)) return LQ_I8_ROUTE_GEMV;
  return LQ_I8_ROUTE_TC + make_plan(batch, K, N).kind;
}

lq_status lq_gemm_i8_plan(int32_t batch, int32_t K, int32_t N, int32_t route, int64_t* out) {
  using namespace lq;
  using namespace lq::w8;
  lq::set_last_error("%s", "");
  if (!out) return reject(LQ_EINVAL, "lq_gemm_i8_plan: null out");
  if (lq_gemm_i8_route(batch, K, N) < 0)
    return reject(LQ_EINVAL, "lq_gemm_i8_plan: invalid sizes batch=%d K=%d N=%d", batch, K, N);
  if (route != -1 && (route < LQ_I8_ROUTE_TC || route > LQ_I8_ROUTE_SPLIT))
    return reject(LQ_EINVAL, "lq_gemm_i8_plan: route %d has no tiles", route);
  const Plan p = make_plan(batch, K, N, route < 0 ? -1 : route - LQ_I8_ROUTE_TC);
  const int64_t v[LQ_I8_PLAN_FIELDS] = {LQ_I8_ROUTE_TC + p.kind, p.kind == kPair ? 2 : p.split,
                                        (int64_t)p.tiles_n * p.tiles_t, p.rows, p.tokens, p.chunks,
                                        p.stages, (int64_t)p.smem};
  for (int i = 0; i < LQ_I8_PLAN_FIELDS; ++i) out[i] = v[i];
  return LQ_OK;
}

lq_status lq_gemm_i8(const int8_t* xq, const float* xs, int32_t batch, const int8_t* wq,
                     const float* ws, const float* bias, int32_t K, int32_t N, void* y,
                     lq_dtype ydt, void* workspace, size_t workspace_bytes, int32_t route,
                     lq_stream stream) {
  using namespace lq;
  using namespace lq::w8;
  lq::set_last_error("%s", "");
  if (batch < 0) return reject(LQ_EINVAL, "lq_gemm_i8: batch = %d < 0", batch);
  if (N < 0) return reject(LQ_EINVAL, "lq_gemm_i8: N = %d < 0", N);
  if (K < 1) return reject(LQ_EINVAL, "lq_gemm_i8: K = %d < 1", K);
  if (K > LQ_MAX_I8_K)
    return reject(LQ_EUNSUPPORTED, "lq_gemm_i8: K = %d exceeds LQ_MAX_I8_K (%d)", K, LQ_MAX_I8_K);
  if (batch > kMost || N > kMost)
    return reject(LQ_EUNSUPPORTED, "lq_gemm_i8: batch = %d or N = %d exceeds %d", batch, N, kMost);
  if (ydt != LQ_F32 && ydt != LQ_F16 && ydt != LQ_BF16)
    return reject(LQ_EINVAL, "lq_gemm_i8: unknown y dtype %d", (int)ydt);
  if (route < -1 || route > LQ_I8_ROUTE_SPLIT)
    return reject(LQ_EINVAL, "lq_gemm_i8: unknown route %d", route);
  if (route == LQ_I8_ROUTE_GEMV && batch > LQ_I8_GEMV_MAX_BATCH)
    return reject(LQ_EUNSUPPORTED, "lq_gemm_i8: %d tokens on the GEMV route (at most %d)", batch,
                  LQ_I8_GEMV_MAX_BATCH);
  if (batch == 0 || N == 0) return LQ_OK;
  if (!xq || !xs || !wq || !ws || !y || !workspace)
    return reject(LQ_EINVAL, "lq_gemm_i8: null pointer");
  if (!aligned(xq, 16) || !aligned(wq, 16))
    return reject(LQ_EINVAL, "lq_gemm_i8: xq or wq not 16-byte aligned");
  if (!aligned(xs, 4) || !aligned(ws, 4) || !aligned(bias, 4) || !aligned(y, ydt == LQ_F32 ? 4 : 2))
    return reject(LQ_EINVAL, "lq_gemm_i8: misaligned xs, ws, bias or y");
  if (!aligned(workspace, 256))
    return reject(LQ_EINVAL, "lq_gemm_i8: workspace not 256-byte aligned");
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
  const cudaError_t e = launch(a, route, (cudaStream_t)stream);
  return e == cudaSuccess ? LQ_OK : reject(LQ_ECUDA, "lq_gemm_i8: %s", cudaGetErrorString(e));
}

}  // extern "C"
