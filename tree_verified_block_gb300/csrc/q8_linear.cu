// Products of 8-bit rows with 8-bit weights, the epilogue fused:
//
//   v[m][n]   = x_scale[m] w_scale[n] sum_k x[m][k] w[n][k] + bias[n]
//   out[m][n] = act(v[m][n]) + residual[m][n], or gated
//   out[m][j] = act(v[m][j]) * v[m][N + j]     (w: N gate rows, then N up rows)
//
// Codes are e4m3, K-major on both sides; the tensor core multiplies them exactly
// and sums in fp32 (kind::f8f6f4, K = 32 a step); the scales are per row and per
// output channel, so they leave the sum and act once, in the epilogue.
//
// Two kernels:
//
// * Few rows (q8_linear_few_kernel): bound by reading the weights. The weights
//   are the tensor core's 128-row operand and the rows its narrow one (16 to 128
//   wide), so a step multiplies no padding but in the rows. N / 128 tiles are
//   too few to keep the memory busy, so a cluster of CTAs splits K and joins the
//   fp32 partials through distributed shared memory, every CTA finishing its
//   share of the rows. The first weight stages are on their way before the
//   kernel waits for the one before it.
// * Many rows (q8_linear_wide_kernel): bound by the products. A pair of SMs
//   works on 256 x 256 outputs (each holds half of both operands; 256 x 128 where
//   these would not fill half of the pairs), persistent over the tiles, with two
//   accumulators so that one tile's epilogue runs under the next one's products.
//
// Measured: one row x 4096 x 6144 9.5 us (25 MB; a CTA's start 0.8, its loads 3.7,
// the cluster's two barriers, sums and stores 2.2), 64 rows x 4096 x 4096 9.0,
// gated 64 x 4096 x 2 * 12288 22 us (101 MB, 70 % of the copy rate with start and
// end), logits of 64 rows x 4096 x 151936 in fp32 107.7 us (91 %); gated 8191 x
// 4096 x 2 * 12288 471 us in bursts (3.5 PFLOP/s), 547 under the power limit.
// Where they meet (4096 x 2 * 12288, gated): 192 rows 47 us by the first, 35 by
// the second; 4096 x 4096: 256 rows 15.3 and 22.9, 512 rows 38.9 and 18.5.
#include <mutex>

#include "q8_internal.cuh"

GLANCE_DEFINE_STATUS_WORD(status_q8_linear)

using namespace glance_dev;

namespace {

constexpr int kBK = 128;       // codes of a row in a stage: one 128-byte swizzle row
constexpr int kTile = 128;     // weight rows of an operand tile
constexpr uint32_t kTileBytes = kTile * kBK;  // 16 KB

struct Params {
  int M, N, K;       // N: output columns
  int n_kb;          // stages of K
  int gated, act;    // act: glance_act
  int out_f32;       // out and residual are fp32, else bf16
  const float* x_scale;
  const float* w_scale;
  const float* bias;      // null: none
  const char* residual;   // null: none
  char* out;
  long long r_stride, o_stride;  // bytes
  int tiles_n, tiles_m;  // wide
  int64_t tiles;
};

// ------------------------------------------------------------------- epilogue

__device__ __forceinline__ float sigmoid(float x) { return __fdividef(1.f, 1.f + __expf(-x)); }

template <int kCount>
__device__ __forceinline__ void activate(float (&v)[kCount], int act) {
  if (act == GLANCE_ACT_SILU) {
#pragma unroll
    for (int i = 0; i < kCount; ++i) v[i] *= sigmoid(v[i]);
  } else if (act == GLANCE_ACT_GELU) {
#pragma unroll
    for (int i = 0; i < kCount; ++i) v[i] = 0.5f * v[i] * (1.f + erff(v[i] * 0.70710678118654752f));
  } else if (act == GLANCE_ACT_GELU_TANH) {
    // (1 + tanh z) / 2 = sigmoid(2 z), z = sqrt(2 / pi) (x + 0.044715 x^3)
#pragma unroll
    for (int i = 0; i < kCount; ++i) v[i] *= sigmoid(1.5957691216057308f * fmaf(0.044715f * v[i], v[i] * v[i], v[i]));
  }
}

// Eight consecutive outputs of a row, from column n on: the residual's addition
// and the store. v: after the activation.
__device__ __forceinline__ void store8(const Params& p, int64_t row, int n, float (&v)[8]) {
  if (p.out_f32) {
    if (p.residual) {
      const float4* r = reinterpret_cast<const float4*>(p.residual + row * p.r_stride + 4ll * n);
      const float4 a = r[0], b = r[1];
      v[0] += a.x, v[1] += a.y, v[2] += a.z, v[3] += a.w, v[4] += b.x, v[5] += b.y, v[6] += b.z, v[7] += b.w;
    }
    float4* o = reinterpret_cast<float4*>(p.out + row * p.o_stride + 4ll * n);
    o[0] = make_float4(v[0], v[1], v[2], v[3]);
    o[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    if (p.residual) {
      const uint4 r = *reinterpret_cast<const uint4*>(p.residual + row * p.r_stride + 2ll * n);
      const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] += __uint_as_float(w[i] << 16);
        v[2 * i + 1] += __uint_as_float(w[i] & 0xFFFF0000u);
      }
    }
    *reinterpret_cast<uint4*>(p.out + row * p.o_stride + 2ll * n) =
        make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  }
}

// The residual of 32 outputs of this thread's row from column n on (those that
// are there: N is a multiple of eight). A sector's second half comes from L1.
__device__ __forceinline__ void add_residual(const Params& p, int64_t row, int n, float (&v)[32]) {
#pragma unroll
  for (int j = 0; j < 32; j += 8) {
    if (n + j >= p.N) continue;
    if (p.out_f32) {
      const float4* r = reinterpret_cast<const float4*>(p.residual + row * p.r_stride + 4ll * (n + j));
      const float4 a = r[0], b = r[1];
      v[j] += a.x, v[j + 1] += a.y, v[j + 2] += a.z, v[j + 3] += a.w, v[j + 4] += b.x, v[j + 5] += b.y, v[j + 6] += b.z, v[j + 7] += b.w;
    } else {
      const uint4 r = *reinterpret_cast<const uint4*>(p.residual + row * p.r_stride + 2ll * (n + j));
      const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[j + 2 * i] += __uint_as_float(w[i] << 16);
        v[j + 2 * i + 1] += __uint_as_float(w[i] & 0xFFFF0000u);
      }
    }
  }
}

// A warp's 32 rows of 64 bytes, a row a thread, to out rows row0 .. from byte
// `at` of a row on: through shared memory (16-byte pieces exchanged so that neither
// side meets a bank twice), so that four threads write a row's two sectors whole.
__device__ __forceinline__ void store_rows(const Params& p, unsigned char* buf, const uint32_t (&word)[16], int64_t row0, int64_t at) {
  const int lane = threadIdx.x & 31;
  __syncwarp();
#pragma unroll
  for (int c = 0; c < 4; ++c)
    *reinterpret_cast<uint4*>(buf + lane * 64 + (c ^ ((lane >> 1) & 3)) * 16) =
        make_uint4(word[4 * c], word[4 * c + 1], word[4 * c + 2], word[4 * c + 3]);
  __syncwarp();
  const int piece = lane & 3;
  const bool in = at + 16 * piece < static_cast<int64_t>(p.N) * (p.out_f32 ? 4 : 2);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 8 * i + (lane >> 2);
    const uint4 v = *reinterpret_cast<const uint4*>(buf + r * 64 + (piece ^ ((r >> 1) & 3)) * 16);
    if (in && row0 + r < p.M && GLANCE_IN_BOUNDS(row0 + r, p.M))
      *reinterpret_cast<uint4*>(p.out + (row0 + r) * p.o_stride + at + 16 * piece) = v;
  }
}

// One output.
__device__ __forceinline__ void store1(const Params& p, int64_t row, int n, float v) {
  if (p.out_f32) {
    if (p.residual) v += *reinterpret_cast<const float*>(p.residual + row * p.r_stride + 4ll * n);
    *reinterpret_cast<float*>(p.out + row * p.o_stride + 4ll * n) = v;
  } else {
    if (p.residual) v += __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(p.residual + row * p.r_stride + 2ll * n));
    *reinterpret_cast<__nv_bfloat16*>(p.out + row * p.o_stride + 2ll * n) = __float2bfloat16_rn(v);
  }
}

// ---------------------------------------------------------------------- waits

__device__ __forceinline__ bool aborted(const int* flag) { return *reinterpret_cast<const volatile int*>(flag) != 0; }
// A wait that ends after 2 s or when another role of this CTA has given up.
__device__ __forceinline__ bool wait_or_abort(uint64_t* bar, uint32_t parity, const int* flag) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 63u) == 0 && (aborted(flag) || globaltimer_ns() - t0 > 2000000000ull)) return false;
  }
}
// Gives up: the other roles of this CTA stop too.
__device__ __forceinline__ void give_up(int* flag) {
  report(GLANCE_DEV_PIPELINE_TIMEOUT);
  atomicExch(flag, 1);
}
// After a failure: long enough for every copy and product in flight to land.
__device__ __forceinline__ void settle() {
  const uint64_t t0 = globaltimer_ns();
  while (globaltimer_ns() - t0 < 50000000ull) __nanosleep(1000);
}

// ------------------------------------------------------------------- few rows

constexpr int kFewThreads = 256;
constexpr int kMaxSplit = 8;
constexpr int kMaxRows = 128;  // of a block
constexpr uint32_t kFewMisc = 2048;

template <int kRows>
struct Few {
  static constexpr uint32_t kXBytes = kRows * kBK;
  static constexpr uint32_t kStage = kTileBytes + kXBytes;
  // two CTAs to an SM
  static constexpr int kStages = kRows <= 16 ? 6 : kRows <= 32 ? 5 : kRows <= 64 ? 4 : 3;
  static constexpr uint32_t kArea = kStages * kStage;
  static constexpr uint32_t kSmem = 1024 + kArea + kFewMisc;
  static constexpr uint32_t kCols = kRows < 32 ? 32 : kRows;  // of tensor memory
  static_assert((kRows + kMaxSplit) * kTile * 4 <= kArea, "received partials take the stages' place");
  static_assert(2 * (kSmem + 1024) <= 228 * 1024, "two CTAs per SM");
};

struct FewBars {
  uint64_t full[6], empty[6];
  uint64_t done;
  uint32_t tmem;
  int abort;
  int failed;  // read by the cluster's other CTAs
  float scale[kTile], bias[kTile];  // of the tile's weight rows
  float x_scale[kMaxRows];
};
static_assert(sizeof(FewBars) <= kFewMisc, "barriers and scales");

__device__ __forceinline__ int dsmem_ld_s32(uint32_t addr) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void dsmem_st_f32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// Grid: x = tile * S + rank, clusters of S; y = blocks of kRows rows. A tile is
// 128 weight rows: outputs 128 t .., or, gated, gate rows 64 t .. in the upper
// half and their up rows in the lower.
template <int kRows>
__global__ void __launch_bounds__(kFewThreads, 2)
    q8_linear_few_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x, const Params p,
                         const int S) {
  typedef Few<kRows> C;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  FewBars* bars = reinterpret_cast<FewBars*>(smem + C::kArea);
  float* s_recv = reinterpret_cast<float*>(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = S > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int tile = static_cast<int>(blockIdx.x) / S;
  const int kb0 = static_cast<int>(static_cast<long long>(p.n_kb) * rank / S);
  const int n_it = static_cast<int>(static_cast<long long>(p.n_kb) * (rank + 1) / S) - kb0;  // >= 1: S <= n_kb
  const int m0 = static_cast<int>(blockIdx.y) * kRows;
  // weight rows of the tile's halves
  const int w0 = p.gated ? tile * 64 : tile * kTile, w1 = p.gated ? p.N + tile * 64 : w0 + 64;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&bars->full[s], 1);
      mbar_init(&bars->empty[s], 1);
    }
    mbar_init(&bars->done, 1);
    bars->abort = bars->failed = 0;
    fence_barrier_init();
    const uint64_t pol_w = policy_evict_first();
    for (int it = 0; it < C::kStages && it < n_it; ++it) {
      unsigned char* st = smem + it * C::kStage;
      mbar_arrive_expect_tx(&bars->full[it], C::kStage);
      tma_load_2d(st, &map_w, &bars->full[it], (kb0 + it) * kBK, w0, pol_w);
      tma_load_2d(st + kTileBytes / 2, &map_w, &bars->full[it], (kb0 + it) * kBK, w1, pol_w);
    }
  }
  if (warp == 2) {
    tmem_alloc(&bars->tmem, C::kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem;
  pdl_wait_prior();
  pdl_launch_dependents();
  bool ok = true;
  if (warp == 0) {
    if (lane == 0) {
      const uint64_t pol_w = policy_evict_first(), pol_x = policy_evict_last();
      for (int it = 0; it < n_it; ++it) {
        const int st = it % C::kStages, k = (kb0 + it) * kBK;
        unsigned char* at = smem + st * C::kStage;
        if (it >= C::kStages) {
          if (!wait_or_abort(&bars->empty[st], (it / C::kStages - 1) & 1, &bars->abort)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&bars->full[st], C::kStage);
          tma_load_2d(at, &map_w, &bars->full[st], k, w0, pol_w);
          tma_load_2d(at + kTileBytes / 2, &map_w, &bars->full[st], k, w1, pol_w);
        }
        tma_load_2d(at + kTileBytes, &map_x, &bars->full[st], k, m0, pol_x);
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_e4m3_f32(kTile, kRows);
      const uint32_t a0 = smem_u32(smem);
      for (int it = 0; it < n_it; ++it) {
        const int st = it % C::kStages;
        if (!wait_or_abort(&bars->full[st], (it / C::kStages) & 1, &bars->abort)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t a = a0 + st * C::kStage, b = a + kTileBytes;
#pragma unroll
        for (int k = 0; k < kBK / 32; ++k)
          mma_f8_ss(tmem, sdesc_sw128(a + k * 32, 16, 1024), sdesc_sw128(b + k * 32, 16, 1024), idesc, (it | k) ? 1u : 0u);
        if (it + C::kStages < n_it) mma_commit(&bars->empty[st]);
      }
      if (ok) mma_commit(&bars->done);
    }
  }
  const int M = min(kRows, p.M - m0);  // rows of this block
  if (warp >= 2) {  // what the epilogue needs, while the products run
    const int i = static_cast<int>(threadIdx.x) - 64;
    if (i < kTile) {
      const int n = p.gated ? tile * 64 + (i & 63) : tile * kTile + i, w = i < 64 ? w0 + i : w1 + i - 64;
      bars->scale[i] = n < p.N ? __ldg(p.w_scale + w) : 0.f;
      bars->bias[i] = n < p.N && p.bias ? __ldg(p.bias + w) : 0.f;
    }
    for (int m = i; m < M; m += kFewThreads - 64) bars->x_scale[m] = __ldg(p.x_scale + m0 + m);
  }
  __syncwarp();
  if (ok) ok = wait_or_abort(&bars->done, 0, &bars->abort);
  if (!ok) give_up(&bars->abort);
  // with `done`, every copy of this CTA has landed and been read
  bool bad = __syncthreads_or(!ok) != 0;
  if (bad) settle();
  if (S > 1) {
    if (threadIdx.x == 0) bars->failed = bad;
    __syncthreads();
    cluster_sync_all();  // the whole cluster is done with its stages
    bool peer = false;
    if (threadIdx.x < S) peer = dsmem_ld_s32(dsmem_addr(&bars->failed, threadIdx.x)) != 0;
    bad = __syncthreads_or(peer) != 0;
  }
  const int per = (M + S - 1) / S;  // rows that a CTA finishes
  const bool direct = S == 1 && !p.gated;  // a thread has all of its outputs' sums
  if (!bad) {
    // D: lane = weight row of the tile, column = row. Row m's partial goes to
    // the CTA that finishes it, [source][row][128].
    tc_fence_after();
    const int ch = (warp & 3) * 32 + lane;
    constexpr int kHalf = kRows / 2;  // a warp takes half of the columns
    constexpr int kChunk = kHalf < 32 ? kHalf : 32;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
#pragma unroll 1
    for (int c = 0; c < kHalf; c += kChunk) {
      const int m = (warp >> 2) * kHalf + c;
      uint32_t r[kChunk];
      if constexpr (kChunk == 32)
        tmem_ld32(tmem + lanes + m, r);
      else if constexpr (kChunk == 16)
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
            : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
              "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
            : "r"(tmem + lanes + m));
      else
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                     : "r"(tmem + lanes + m));
      tmem_ld_wait();
      if (direct) {
        const int n = tile * kTile + ch;
        if (n < p.N) {
          const float ws = bars->scale[ch], b = bars->bias[ch];
          float v[kChunk];
#pragma unroll
          for (int j = 0; j < kChunk; ++j) v[j] = fmaf(__uint_as_float(r[j]) * bars->x_scale[m + j], ws, b);
          activate(v, p.act);
          // a warp's 32 outputs of a row lie next to each other
#pragma unroll
          for (int j = 0; j < kChunk; ++j)
            if (m + j < M && GLANCE_IN_BOUNDS(m0 + m + j, p.M)) store1(p, m0 + m + j, n, v[j]);
        }
        continue;
      }
      int owner = m / per, local = m - owner * per;
#pragma unroll
      for (int j = 0; j < kChunk; ++j) {
        if (m + j < M) {
          float* at = s_recv + (rank * per + local) * kTile + ch;
          if (S > 1)
            dsmem_st_f32(dsmem_addr(at, owner), r[j]);
          else
            *at = __uint_as_float(r[j]);
        }
        if (++local == per) local = 0, ++owner;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kCols);
  }
  if (S > 1) cluster_sync_all();  // every partial has reached its owner
  if (bad || direct) return;
  const int first = rank * per, mine = min(per, M - first);
  const int cols = p.gated ? 64 : kTile, groups = cols / 8;
  for (int i = threadIdx.x; i < mine * groups; i += kFewThreads) {
    const int local = i / groups, c = i % groups * 8, n = tile * cols + c;
    if (n >= p.N) continue;
    const int64_t row = m0 + first + local;
    const float xs = bars->x_scale[first + local];
    float v[2][8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (h && !p.gated) break;
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
      for (int s = 0; s < S; ++s) {
        const float* src = s_recv + (s * per + local) * kTile + c + 64 * h;
        const float4 a1 = *reinterpret_cast<const float4*>(src), b1 = *reinterpret_cast<const float4*>(src + 4);
        a.x += a1.x, a.y += a1.y, a.z += a1.z, a.w += a1.w;
        b.x += b1.x, b.y += b1.y, b.z += b1.z, b.w += b1.w;
      }
      const float sum[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
      for (int j = 0; j < 8; ++j) v[h][j] = fmaf(sum[j] * xs, bars->scale[c + 64 * h + j], bars->bias[c + 64 * h + j]);
    }
    activate(v[0], p.act);
    if (p.gated) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[0][j] *= v[1][j];
    }
    if (GLANCE_IN_BOUNDS(row, p.M)) store8(p, row, n, v[0]);
  }
}

// ------------------------------------------------------------------ many rows

constexpr int kWideThreads = 384;  // a warp each for copies, products, tensor memory; one idle; eight for the epilogue
constexpr int kWideStages = 6;
// kN: weight rows of a tile. A stage is a CTA's 128 rows and half of the weight rows.
__host__ __device__ constexpr uint32_t wide_stage(int kN) { return kTileBytes + kN / 2 * kBK; }
constexpr uint32_t kWideArea = kWideStages * wide_stage(256);
constexpr uint32_t kWideVec = 2 * 2 * 256 * 4;  // two tiles' weight scales and biases
constexpr int kEpilogueWarps = 8;
constexpr uint32_t kWideOut = kEpilogueWarps * 32 * 64;  // a warp's 32 rows of 64 bytes on their way out
constexpr uint32_t kWideSmem = 1024 + kWideArea + kWideOut + kWideVec + 1024;
constexpr int kGroupM = 8;  // tiles of the row axis that are taken together, for L2

struct WideBars {
  uint64_t full[kWideStages], empty[kWideStages];
  uint64_t acc_full[2], acc_empty[2];
  uint32_t tmem;
  int abort;
};
static_assert(sizeof(WideBars) <= 1024, "barriers");
static_assert(kWideSmem <= 227 * 1024, "shared memory");

// Tile i: groups of kGroupM row tiles go through all column tiles.
__device__ __forceinline__ void wide_tile(const Params& p, int64_t i, int& tm, int& tn) {
  const int64_t per_group = static_cast<int64_t>(kGroupM) * p.tiles_n;
  const int g = static_cast<int>(i / per_group), in = static_cast<int>(i - g * per_group);
  const int rows = min(kGroupM, p.tiles_m - g * kGroupM);
  tm = g * kGroupM + in % rows;
  tn = in / rows;
}

template <int kN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kWideThreads, 1)
    q8_linear_wide_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x, const Params p) {
  constexpr uint32_t kStage = wide_stage(kN);
  constexpr int kHalf = kN / 2;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  unsigned char* s_out = smem + kWideArea;
  float* s_vec = reinterpret_cast<float*>(smem + kWideArea + kWideOut);  // [2 tiles][scale, bias][256]
  WideBars* bars = reinterpret_cast<WideBars*>(smem + kWideArea + kWideOut + kWideVec);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const int pair = static_cast<int>(blockIdx.x) / 2, pairs = static_cast<int>(gridDim.x) / 2;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kWideStages; ++s) {
      mbar_init(&bars->full[s], 1);
      mbar_init(&bars->empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&bars->acc_full[a], 1);
      mbar_init(&bars->acc_empty[a], 2 * kEpilogueWarps);
    }
    bars->abort = 0;
    fence_barrier_init();
  }
  if (warp == 2) {
    tmem_alloc_pair(&bars->tmem, 2 * kN);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // the other CTA's barriers are ready
  tc_fence_after();
  const uint32_t tmem = bars->tmem;
  pdl_wait_prior();
  pdl_launch_dependents();
  bool ok = true;
  if (warp == 0) {
    if (lane == 0) {
      const uint64_t pol = policy_evict_last();
      const int w_of = p.gated ? kHalf : kN;  // outputs of a tile
      int it = 0;
      for (int64_t i = pair; i < p.tiles && ok; i += pairs) {
        int tm, tn;
        wide_tile(p, i, tm, tn);
        const int x0 = tm * 256 + rank * 128;
        // the pair's second CTA holds the tile's second half: the later columns, or the up rows
        const int w0 = tn * w_of + (rank ? (p.gated ? p.N : kHalf) : 0);
        for (int kb = 0; kb < p.n_kb; ++kb, ++it) {
          const int st = it % kWideStages;
          if (it >= kWideStages && !wait_or_abort(&bars->empty[st], (it / kWideStages - 1) & 1, &bars->abort)) {
            ok = false;
            break;
          }
          unsigned char* at = smem + st * kStage;
          const uint32_t full = dsmem_addr(&bars->full[st], 0);
          if (rank == 0) mbar_arrive_expect_tx(&bars->full[st], 2 * kStage);
          tma_load_2d_pair(at, &map_x, full, kb * kBK, x0, pol);
          tma_load_2d_pair(at + kTileBytes, &map_w, full, kb * kBK, w0, pol);
        }
      }
    }
  } else if (warp == 1) {
    if (rank == 0 && lane == 0) {
      constexpr uint32_t idesc = idesc_e4m3_f32(256, kN);
      const uint32_t a0 = smem_u32(smem);
      int it = 0, n = 0;
      for (int64_t i = pair; i < p.tiles && ok; i += pairs, ++n) {
        const int acc = n & 1;
        if (n >= 2 && !wait_or_abort(&bars->acc_empty[acc], (n / 2 - 1) & 1, &bars->abort)) {
          ok = false;
          break;
        }
        tc_fence_after();
        for (int kb = 0; kb < p.n_kb; ++kb, ++it) {
          const int st = it % kWideStages;
          if (!wait_or_abort(&bars->full[st], (it / kWideStages) & 1, &bars->abort)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a = a0 + st * kStage, b = a + kTileBytes;
#pragma unroll
          for (int k = 0; k < kBK / 32; ++k)
            mma_f8_ss_pair(tmem + acc * kN, sdesc_sw128(a + k * 32, 16, 1024), sdesc_sw128(b + k * 32, 16, 1024), idesc,
                           (kb | k) ? 1u : 0u);
          mma_commit_pair(&bars->empty[st]);
        }
        if (ok) mma_commit_pair(&bars->acc_full[acc]);
      }
    }
  } else if (warp >= 4) {
    const int e = warp - 4, quarter = warp & 3, half = e >> 2;
    const int te = static_cast<int>(threadIdx.x) - 128;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    int n = 0;
    for (int64_t i = pair; i < p.tiles && ok; i += pairs, ++n) {
      const int acc = n & 1;
      int tm, tn;
      wide_tile(p, i, tm, tn);
      const int out0 = tn * (p.gated ? kHalf : kN);
      // this tile's weight scales and biases; the other buffer may still be read
      float* vec = s_vec + (n & 1) * 512;
      if (te < kN) {
        const int w = p.gated ? (te < kHalf ? out0 + te : p.N + out0 + te - kHalf) : out0 + te;
        const bool in = p.gated ? out0 + te % kHalf < p.N : w < p.N;
        vec[te] = in ? __ldg(p.w_scale + w) : 0.f;
        vec[256 + te] = in && p.bias ? __ldg(p.bias + w) : 0.f;
      }
      const int64_t row = static_cast<int64_t>(tm) * 256 + rank * 128 + quarter * 32 + lane;
      const float xs = row < p.M ? __ldg(p.x_scale + row) : 0.f;
      // the eight warps go on together or not at all: none is left at a barrier
      ok = !named_bar_or(1, 32 * kEpilogueWarps, !wait_or_abort(&bars->acc_full[acc], (n / 2) & 1, &bars->abort));
      if (!ok) break;
      tc_fence_after();
      const uint32_t d = tmem + lanes + acc * kN;
      const int width = p.gated ? kHalf / 2 : kHalf;  // this warp's outputs
#pragma unroll 1
      for (int c = half * width; c < (half + 1) * width; c += 32) {
        uint32_t r[32];
        tmem_ld32(d + c, r);
        float v[32];
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
          const float4 s = *reinterpret_cast<const float4*>(vec + c + j), b = *reinterpret_cast<const float4*>(vec + 256 + c + j);
          v[j] = fmaf(__uint_as_float(r[j]) * xs, s.x, b.x);
          v[j + 1] = fmaf(__uint_as_float(r[j + 1]) * xs, s.y, b.y);
          v[j + 2] = fmaf(__uint_as_float(r[j + 2]) * xs, s.z, b.z);
          v[j + 3] = fmaf(__uint_as_float(r[j + 3]) * xs, s.w, b.w);
        }
        activate(v, p.act);
        if (p.gated) {
          tmem_ld32(d + kHalf + c, r);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            const float4 s = *reinterpret_cast<const float4*>(vec + kHalf + c + j),
                         b = *reinterpret_cast<const float4*>(vec + 256 + kHalf + c + j);
            v[j] *= fmaf(__uint_as_float(r[j]) * xs, s.x, b.x);
            v[j + 1] *= fmaf(__uint_as_float(r[j + 1]) * xs, s.y, b.y);
            v[j + 2] *= fmaf(__uint_as_float(r[j + 2]) * xs, s.z, b.z);
            v[j + 3] *= fmaf(__uint_as_float(r[j + 3]) * xs, s.w, b.w);
          }
        }
        if (c + 32 == (half + 1) * width) {  // the accumulator has been read
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(dsmem_addr(&bars->acc_empty[acc], 0));
        }
        if (p.residual && row < p.M) add_residual(p, row, out0 + c, v);
        if (p.out_f32) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t word[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) word[j] = __float_as_uint(v[16 * h + j]);
            store_rows(p, s_out + e * 2048, word, row - lane, (out0 + c + 16 * h) * 4);
          }
        } else {
          uint32_t word[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) word[j] = pack_bf16x2(v[2 * j], v[2 * j + 1]);
          store_rows(p, s_out + e * 2048, word, row - lane, (out0 + c) * 2);
        }
      }
    }
  }
  __syncwarp();
  if (!ok) give_up(&bars->abort);
  if (__syncthreads_or(!ok)) settle();
  tc_fence_before();
  cluster_sync_all();  // the pair is done with both CTAs' memory
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 2 * kN);
  }
}

// ----------------------------------------------------------------------- host

// Shared-memory limits of the kernels, once per device.
template <typename F>
cudaError_t raise(F* f, int bytes) {
  return glance::ensure_smem(reinterpret_cast<const void*>(f), bytes);
}

// Clusters of `size` CTAs of the few-rows kernel that the device holds at once
// (asked once per device, form and size).
template <int kRows>
int max_clusters(int size) {
  static int known[64][kMaxSplit + 1] = {};
  static std::mutex mu;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  std::lock_guard<std::mutex> lock(mu);
  int& n = known[dev][size];
  if (n == 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(size * glance::num_sms()));
    cfg.blockDim = dim3(kFewThreads);
    cfg.dynamicSmemBytes = Few<kRows>::kSmem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = size;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, q8_linear_few_kernel<kRows>, &cfg) != cudaSuccess || n < 1) {
      (void)cudaGetLastError();
      n = -1;
    }
  }
  return n;
}

// How many CTAs split K: as many as the device holds at once (a cluster that has
// to wait for another's end doubles the time), each with two stages at least.
template <int kRows>
int choose_split(int tiles, int blocks_m, int n_kb) {
  int best = 1;
  for (int s = 2; s <= kMaxSplit && n_kb / s >= 2; ++s)
    if (max_clusters<kRows>(s) >= static_cast<int64_t>(tiles) * blocks_m) best = s;
  return best;
}

template <int kRows>
cudaError_t launch_few(const CUtensorMap& mw, const CUtensorMap& mx, const Params& p, cudaStream_t s) {
  typedef Few<kRows> C;
  cudaError_t e = raise(q8_linear_few_kernel<kRows>, C::kSmem);
  if (e != cudaSuccess) return e;
  const int per = p.gated ? 64 : kTile, tiles = (p.N + per - 1) / per, blocks_m = (p.M + kRows - 1) / kRows;
  const int S = choose_split<kRows>(tiles, blocks_m, p.n_kb);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles * S), static_cast<unsigned>(blocks_m));
  cfg.blockDim = dim3(kFewThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = S;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, q8_linear_few_kernel<kRows>, mw, mx, p, S);
}

template <int kN>
cudaError_t launch_wide(const CUtensorMap& mw, const CUtensorMap& mx, Params p, cudaStream_t s) {
  cudaError_t e = raise(q8_linear_wide_kernel<kN>, kWideSmem);
  if (e != cudaSuccess) return e;
  const int per = p.gated ? kN / 2 : kN;
  p.tiles_n = (p.N + per - 1) / per;
  p.tiles_m = (p.M + 255) / 256;
  p.tiles = static_cast<int64_t>(p.tiles_n) * p.tiles_m;
  const int64_t pairs = glance::num_sms() / 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2u * static_cast<unsigned>(p.tiles < pairs ? p.tiles : pairs));
  cfg.blockDim = dim3(kWideThreads);
  cfg.dynamicSmemBytes = kWideSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, q8_linear_wide_kernel<kN>, mw, mx, p);
}

// 256 x 256 tiles of the many-rows kernel.
int64_t wide_tiles(const Params& p) {
  const int64_t per = p.gated ? 128 : 256;
  return (p.N + per - 1) / per * ((p.M + 255) / 256);
}
// The few-rows kernel: up to a block of rows, and up to two while the other's
// tiles would leave half of the SM pairs without work.
bool takes_few(const Params& p) { return p.M <= kMaxRows || (p.M <= 2 * kMaxRows && 4 * wide_tiles(p) <= glance::num_sms()); }
// Many rows: tiles half as wide while the wide ones leave half of the pairs
// without work (512 rows x 4096 x 4096: 23.0 us in wide tiles, 18.5 in these).
bool takes_narrow(const Params& p) { return 4 * wide_tiles(p) <= glance::num_sms(); }

}  // namespace

extern "C" glance_status glance_q8_linear(const void* x, int64_t x_stride, const float* x_scale, int M, const void* w,
                                          int64_t w_stride, const float* w_scale, int N, int K, int gated, glance_act act,
                                          const float* bias, const void* residual, int64_t residual_stride, void* out,
                                          int64_t out_stride, glance_dtype out_dtype, void* stream) {
  using glance::fail;
  using glance::overlap;
  const char* who = "glance_q8_linear";
  if (!x || !x_scale || !w || !w_scale || !out) return fail(GLANCE_ERR_INVALID_ARG, "%s: null pointer argument", who);
  if (out_dtype != GLANCE_BF16 && out_dtype != GLANCE_F32)
    return fail(GLANCE_ERR_INVALID_ARG, "%s: out_dtype must be F32 or BF16", who);
  if (act != GLANCE_ACT_NONE && act != GLANCE_ACT_SILU && act != GLANCE_ACT_GELU && act != GLANCE_ACT_GELU_TANH)
    return fail(GLANCE_ERR_INVALID_ARG, "%s: unknown activation", who);
  if (M < 1 || M > glance::kQ8MaxRows) return fail(GLANCE_ERR_INVALID_ARG, "%s: need 1 <= M <= 2^24", who);
  if (N < 8 || N > (1 << 22) || N % 8 || K < 16 || K > (1 << 20) || K % 16)
    return fail(GLANCE_ERR_UNSUPPORTED, "%s: N must be a multiple of 8 up to 2^22, K a multiple of 16 up to 2^20", who);
  const int esize = out_dtype == GLANCE_BF16 ? 2 : 4;
  if (x_stride < K || w_stride < K || x_stride > glance::kQ8MaxStride || w_stride > glance::kQ8MaxStride || x_stride % 16 ||
      w_stride % 16)
    return fail(GLANCE_ERR_INVALID_ARG, "%s: x_stride and w_stride must cover K and be multiples of 16", who);
  if (out_stride < N || out_stride > glance::kQ8MaxStride || out_stride * esize % 16 ||
      (residual && (residual_stride < N || residual_stride > glance::kQ8MaxStride || residual_stride * esize % 16)))
    return fail(GLANCE_ERR_INVALID_ARG, "%s: out and residual strides must cover N and be multiples of 16 bytes", who);
  if (!glance::aligned16(x) || !glance::aligned16(w) || !glance::aligned16(out) || !glance::aligned16(residual) ||
      ((reinterpret_cast<uintptr_t>(x_scale) | reinterpret_cast<uintptr_t>(w_scale) | reinterpret_cast<uintptr_t>(bias)) & 3))
    return fail(GLANCE_ERR_INVALID_ARG, "%s: x, w, out and residual must be 16-byte aligned, scales and bias 4-byte", who);
  const int64_t rows_w = static_cast<int64_t>(N) * (gated ? 2 : 1), os = out_stride * esize, rs = residual_stride * esize;
  const int64_t no = (M - 1) * os + static_cast<int64_t>(N) * esize, nr = (M - 1) * rs + static_cast<int64_t>(N) * esize;
  if (overlap(out, no, x, (M - 1) * x_stride + K) || overlap(out, no, w, (rows_w - 1) * w_stride + K) ||
      overlap(out, no, x_scale, 4ll * M) || overlap(out, no, w_scale, 4 * rows_w) || (bias && overlap(out, no, bias, 4 * rows_w)) ||
      (residual && overlap(out, no, residual, nr) && !(out == residual && os == rs)))
    return fail(GLANCE_ERR_INVALID_ARG, "%s: out must not overlap an input (it may be the residual itself)", who);
  Params p = {};
  p.M = M;
  p.N = N;
  p.K = K;
  p.n_kb = (K + kBK - 1) / kBK;
  p.gated = gated ? 1 : 0;
  p.act = act;
  p.out_f32 = out_dtype == GLANCE_F32;
  p.x_scale = x_scale;
  p.w_scale = w_scale;
  p.bias = bias;
  p.residual = static_cast<const char*>(residual);
  p.out = static_cast<char*>(out);
  p.r_stride = rs;
  p.o_stride = os;
  const bool few = takes_few(p);
  const bool narrow = !few && takes_narrow(p);
  const int rows = M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 128;
  CUtensorMap mw, mx;
  glance_status st = glance::make_map_u8(&mw, w, K, rows_w, w_stride, few || narrow ? kTile / 2 : kTile, who);
  if (st == GLANCE_OK) st = glance::make_map_u8(&mx, x, K, M, x_stride, few ? rows : kTile, who);
  if (st != GLANCE_OK) return st;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = narrow       ? launch_wide<128>(mw, mx, p, s)
                        : !few       ? launch_wide<256>(mw, mx, p, s)
                        : rows == 16 ? launch_few<16>(mw, mx, p, s)
                        : rows == 32 ? launch_few<32>(mw, mx, p, s)
                        : rows == 64 ? launch_few<64>(mw, mx, p, s)
                                     : launch_few<128>(mw, mx, p, s);
  if (e != cudaSuccess) return glance::cuda_fail(e, who);
  return GLANCE_OK;
}
