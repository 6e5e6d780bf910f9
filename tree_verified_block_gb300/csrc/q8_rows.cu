// Rows in 8 bits: the residual's addition, the RMS norm and the quantisation
// of a row in one pass; rows quantised as they are; their values read back.
//
//   s = round(x + residual),  y = (s w) / sqrt(mean s^2 + eps),
//   e the least integer with max|y| <= 448 * 2^e,  code = e4m3(y 2^-e).
//
// A row stays in the registers of its threads between its one read and its one
// write. The row's sum of squares and the maximum of |s w| come from one block
// reduction: rounding is monotonic, so max|y| is round(max|s w| * r) for the
// row factor r, and a second reduction is not needed. The scale is a power of
// two: e4m3 is a floating type, so that a finer scale would gain nothing but up
// to one of its 15 binades, and the codes' values stay exact in bf16.
//
// Bound by the memory's rate: 2 e bytes read and e + 1 written per element of e
// bytes (with a residual). 16383 bf16 rows of 4096 take 104.0 us with their
// reading back (671 MB, 95 % of the copy rate), one row 3.0 us for both launches.
// The weights are read twice from the cache: kept, they cost the registers that
// hold more of the row.
#include <cuda_fp16.h>

#include "q8_internal.cuh"

GLANCE_DEFINE_STATUS_WORD(status_q8_rows)

using namespace glance_dev;

namespace {

struct RowParams {
  const char* x;
  const char* residual;  // null: none
  char* total;           // null: not written
  const float* weight;   // null: ones
  unsigned char* codes;
  float* scales;
  long long x_stride, r_stride, t_stride, c_stride;  // bytes between rows
  int M, vecs;  // vectors of 16 bytes of x in a row
  float inv_d, inv_d_low, eps;  // 1 / d as two floats
};

template <typename T>
struct Vec;
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int kN = 8;
  static __device__ __forceinline__ void unpack(const uint4& v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
  }
};
template <>
struct Vec<float> {
  static constexpr int kN = 4;
  static __device__ __forceinline__ void unpack(const uint4& v, float (&f)[4]) {
    f[0] = __uint_as_float(v.x), f[1] = __uint_as_float(v.y), f[2] = __uint_as_float(v.z), f[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
};

// What a row's threads reduce: the sum of squares, and the largest magnitude of
// s w (NaN if one is).
struct Stats {
  float ss, ss_low, top;  // the sum is ss + ss_low
};
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// kExact: the last steps, whose roundings all of the row would share, keep what
// the sum loses (a sum of two floats as two floats, after Knuth).
template <bool kNorm, bool kExact>
__device__ __forceinline__ Stats warp_stats(Stats v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    if (kNorm) {
      const float b = __shfl_xor_sync(0xffffffffu, v.ss, o);
      if (kExact) {
        const float a = v.ss, low = __shfl_xor_sync(0xffffffffu, v.ss_low, o);
        v.ss = a + b;
        const float t = v.ss - a;
        v.ss_low = (v.ss_low + low) + ((a - (v.ss - t)) + (b - t));
      } else {
        v.ss += b;
      }
    }
    v.top = max_nan(v.top, __shfl_xor_sync(0xffffffffu, v.top, o));
  }
  return v;
}

// Three roundings may carry a value across the middle of two codes: one of 2^20
// does so, and is off by a step of its code. The bits of a value below a code's say
// how near it is to a middle (from 2^-6 on, where codes keep three fraction
// bits). Of fp32 rows, what is within kReach units is done again with the roundings'
// remainders: a tenth is left (of 115 million values 7 instead of 78), for 167 us
// instead of 159 at 16383 x 4096 with their reading back, 3.4 instead of 3.3 for one
// row. bf16 rows hold 2^-9 themselves and are not: there it took 117 instead of 104.
constexpr uint32_t kBelow = 0xFFFFFu, kMiddle = 0x80000u, kReach = 3;
// s w (f + f_low), rounded so that it is on its side of a middle.
__device__ __forceinline__ float exactly(float s, float w, float f, float f_low) {
  const float t = __fmul_rn(s, w), y = __fmul_rn(t, f);
  const float rest = fmaf(t, f, -y) + fmaf(fmaf(s, w, -t), f, __fmul_rn(t, f_low));
  const float z = __fadd_rn(y, rest), left = __fadd_rn(__fsub_rn(y, z), rest);
  const uint32_t bits = __float_as_uint(z);
  if ((bits & kBelow) != kMiddle || left == 0.f) return z;
  return __uint_as_float((left > 0.f) == (z > 0.f) ? bits + 1 : bits - 1);
}

constexpr int kWarpRows = 4;  // rows of a block whose rows have a warp each
constexpr int kMaxThreads = 512;
constexpr int kMaxWarps = kMaxThreads / 32;
constexpr int kMaxVecs = 4096;  // a row has 64 KB at most

// kVecs: vectors per thread. kNorm: the RMS norm. kWarp: a row per warp, else a row per block.
template <typename T, int kVecs, bool kNorm, bool kWarp>
__global__ void __launch_bounds__(kWarp ? 32 * kWarpRows : kMaxThreads) q8_rows_kernel(const RowParams p) {
  constexpr int kN = Vec<T>::kN;
  constexpr bool kExact = kNorm && sizeof(T) == 4;
  __shared__ Stats s_stats[2][kMaxWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = kWarp ? blockIdx.x * kWarpRows + warp : blockIdx.x;
  const int t = kWarp ? lane : threadIdx.x, nt = kWarp ? 32 : blockDim.x;
  pdl_wait_prior();
  // no dependent starts early: it might read these codes before its wait (as weights)
  if (kWarp && row >= p.M) return;
  const int64_t r = row;
  float s[kVecs][kN];
  {
    uint4 xv[kVecs], rv[kVecs];
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      xv[v] = rv[v] = make_uint4(0, 0, 0, 0);
      const int at = t + v * nt;
      if (at < p.vecs) {
        xv[v] = __ldcs(reinterpret_cast<const uint4*>(p.x + r * p.x_stride) + at);
        if (p.residual) rv[v] = __ldcs(reinterpret_cast<const uint4*>(p.residual + r * p.r_stride) + at);
      }
    }
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      Vec<T>::unpack(xv[v], s[v]);
      if (p.residual) {
        float f[kN];
        Vec<T>::unpack(rv[v], f);
#pragma unroll
        for (int i = 0; i < kN; ++i) s[v][i] += f[i];
        // the stream holds the rounded sum, and the norm is of what it holds
        xv[v] = Vec<T>::pack(s[v]);
        Vec<T>::unpack(xv[v], s[v]);
      }
      const int at = t + v * nt;
      if (p.total && at < p.vecs) __stcs(reinterpret_cast<uint4*>(p.total + r * p.t_stride) + at, xv[v]);
    }
  }
  // the weights are read again where they are used again: from the cache, and
  // the registers go to rows instead
  const auto weights = [&](int at, float (&w)[kN]) {
#pragma unroll
    for (int i = 0; i < kN; ++i) w[i] = 1.f;
    if (p.weight && at < p.vecs) {
#pragma unroll
      for (int i = 0; i < kN; i += 4) {
        const float4 f = __ldg(reinterpret_cast<const float4*>(p.weight + at * kN + i));
        w[i] = f.x, w[i + 1] = f.y, w[i + 2] = f.z, w[i + 3] = f.w;
      }
    }
  };
  const auto stats = [&] {
    Stats st = {0.f, 0.f, 0.f};
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      float w[kN];
      if (kNorm) weights(t + v * nt, w);
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        if (kNorm) st.ss = fmaf(s[v][i], s[v][i], st.ss);
        st.top = max_nan(st.top, fabsf(kNorm ? s[v][i] * w[i] : s[v][i]));
      }
    }
    return st;
  };
  int phase = 0;
  const auto reduce = [&](Stats v) {
    v = warp_stats<kNorm, kExact && kWarp>(v);
    if (kWarp) return v;
    if (lane == 0) s_stats[phase][warp] = v;
    __syncthreads();
    v = {0.f, 0.f, 0.f};
    if (lane < nt / 32) v = s_stats[phase][lane];
    phase ^= 1;
    return warp_stats<kNorm, kExact>(v);
  };
  Stats st = reduce(stats());
  float factor = 1.f, factor_low = 0.f;  // y = s w (factor + factor_low)
  if (kNorm) {
    float eps = p.eps;
    // squares beyond fp32's range, or lost below it where eps does not outweigh
    // them: once more with the row's largest magnitude brought to [1, 2), or up by
    // 2^100 (eps then stays in range)
    if (!(st.ss <= 1e37f && (st.ss >= 1e-18f || eps >= 1e-30f))) {
      float top = 0.f;
#pragma unroll
      for (int v = 0; v < kVecs; ++v)
#pragma unroll
        for (int i = 0; i < kN; ++i) top = max_nan(top, fabsf(s[v][i]));
      top = reduce(Stats{0.f, 0.f, top}).top;
      if (top >= 1.17549435e-38f && top < INFINITY) {
        const int e = static_cast<int>(__float_as_uint(top) >> 23) - 127;
        const float pre = __uint_as_float(static_cast<uint32_t>(min(100, max(-126, -e)) + 127) << 23);
#pragma unroll
        for (int v = 0; v < kVecs; ++v)
#pragma unroll
          for (int i = 0; i < kN; ++i) s[v][i] *= pre;
        eps = eps * pre * pre;
        st = reduce(stats());
      }
    }
    if (kExact) {
      const float mean = __fmul_rn(st.ss, p.inv_d), q = mean + eps, u = q - mean;
      const float q_low = fmaf(st.ss, p.inv_d, -mean) + fmaf(st.ss, p.inv_d_low, st.ss_low * p.inv_d) + ((mean - (q - u)) + (eps - u));
      factor = 1.f / sqrtf(q);
      // what 1 / sqrt(q + q_low) has beyond it: a Newton step
      const float f2 = __fmul_rn(factor, factor);
      if (f2 > 1e-30f && f2 < 1e30f)
        factor_low = 0.5f * factor * (fmaf(-q, f2, 1.f) - fmaf(q, fmaf(factor, factor, -f2), q_low * f2));
    } else {
      factor = 1.f / sqrtf(fmaf(st.ss, p.inv_d, eps));
    }
  }
  // e from the bits of the largest magnitude: 448 = 1.75 * 2^8
  const float most = st.top * factor;
  const uint32_t top = __float_as_uint(most);
  int e = static_cast<int>(top >> 23) - 135 + ((top & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  e = top == 0u ? 0 : max(e, -126);
  const bool valid = most < INFINITY;  // (not NaN)
  if (t == 0 && GLANCE_IN_BOUNDS(row, p.M)) p.scales[row] = valid ? __uint_as_float(static_cast<uint32_t>(e + 127) << 23) : NAN;
  const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
  const float scaled = factor * down, scaled_low = factor_low * down;  // a power of two: s w scaled rounds where s w factor does
#pragma unroll
  for (int v = 0; v < kVecs; ++v) {
    const int at = t + v * nt;
    uint32_t c[kN / 4];
    float w[kN];
    if (kNorm) weights(at, w);
    float y[kN];
    uint32_t near = ~0u;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      y[i] = kNorm ? __fmul_rn(__fmul_rn(s[v][i], w[i]), scaled) : s[v][i] * down;
      if (kExact) near = min(near, (__float_as_uint(y[i]) - (kMiddle - kReach)) & kBelow);
    }
    if (kExact && near <= 2 * kReach) {
#pragma unroll
      for (int i = 0; i < kN; ++i) y[i] = exactly(s[v][i], w[i], scaled, scaled_low);
    }
#pragma unroll
    for (int i = 0; i < kN; i += 4) c[i / 4] = valid ? pack_e4m3x4(y[i], y[i + 1], y[i + 2], y[i + 3]) : 0u;
    if (at >= p.vecs || !GLANCE_IN_BOUNDS(row, p.M)) continue;
    unsigned char* dst = p.codes + r * p.c_stride + static_cast<int64_t>(at) * kN;
    if (kN == 8)
      *reinterpret_cast<uint2*>(dst) = make_uint2(c[0], c[kN / 4 - 1]);
    else
      *reinterpret_cast<uint32_t*>(dst) = c[0];
  }
}

struct ReadParams {
  const unsigned char* codes;
  const float* scales;
  char* out;
  long long c_stride, o_stride;  // bytes
  int M, chunks;  // chunks of 16 codes in a row
};

// A thread per 16 codes; T the type of out.
template <typename T>
__global__ void __launch_bounds__(256) q8_read_rows_kernel(const ReadParams p) {
  pdl_wait_prior();
  const int row = blockIdx.x;
  const float scale = p.scales[row];
  for (int c = threadIdx.x; c < p.chunks; c += blockDim.x) {
    const uint4 v = __ldcs(reinterpret_cast<const uint4*>(p.codes + static_cast<int64_t>(row) * p.c_stride) + c);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    float f[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t h = e4m3x2_to_f16x2(static_cast<uint16_t>(w[i / 2] >> (16 * (i & 1))));
      const float2 g = __half22float2(*reinterpret_cast<const __half2*>(&h));
      f[2 * i] = g.x * scale;
      f[2 * i + 1] = g.y * scale;
    }
    if (!GLANCE_IN_BOUNDS(row, p.M)) continue;
    uint4* dst = reinterpret_cast<uint4*>(p.out + static_cast<int64_t>(row) * p.o_stride) + c * static_cast<int>(sizeof(T));
    constexpr int kN = Vec<T>::kN;
#pragma unroll
    for (int i = 0; i < 16 / kN; ++i) {
      float part[kN];
#pragma unroll
      for (int j = 0; j < kN; ++j) part[j] = f[i * kN + j];
      __stcs(dst + i, Vec<T>::pack(part));
    }
  }
}

typedef void (*RowKernel)(const RowParams);

template <typename T, int kVecs, bool kWarp>
RowKernel pick_norm(bool norm) {
  return norm ? q8_rows_kernel<T, kVecs, true, kWarp> : q8_rows_kernel<T, kVecs, false, kWarp>;
}
// Threads of a row and vectors of a thread: a warp per row where a warp
// suffices, else as few vectors each as the largest block allows.
template <typename T>
RowKernel pick(int vecs, bool norm, int& threads) {
  if (vecs <= 64) {
    threads = 32;
    return pick_norm<T, 2, true>(norm);
  }
  const int n = vecs <= 2 * kMaxThreads ? 2 : vecs <= 4 * kMaxThreads ? 4 : 8;
  threads = ((vecs + n - 1) / n + 31) / 32 * 32;
  return n == 2 ? pick_norm<T, 2, false>(norm) : n == 4 ? pick_norm<T, 4, false>(norm) : pick_norm<T, 8, false>(norm);
}

glance_status launch(const char* who, const void* kernel_args, const void* kernel, unsigned blocks, int threads, void* stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  void* args[1] = {const_cast<void*>(kernel_args)};
  const cudaError_t e = cudaLaunchKernelExC(&cfg, kernel, args);
  if (e != cudaSuccess) return glance::cuda_fail(e, who);
  return GLANCE_OK;
}

// Bytes from the first to behind the last element of rows.
int64_t span(int M, int64_t stride_bytes, int64_t row_bytes) { return (M - 1) * stride_bytes + row_bytes; }

glance_status check_shape(const char* who, glance_dtype dtype, int M, int d, int most, int64_t code_stride) {
  using glance::fail;
  if (dtype != GLANCE_BF16 && dtype != GLANCE_F32) return fail(GLANCE_ERR_INVALID_ARG, "%s: dtype must be F32 or BF16", who);
  if (M < 1 || M > glance::kQ8MaxRows) return fail(GLANCE_ERR_INVALID_ARG, "%s: need 1 <= M <= 2^24", who);
  if (d < 16 || d > most || d % 16) return fail(GLANCE_ERR_UNSUPPORTED, "%s: d must be a multiple of 16, at most %d", who, most);
  if (code_stride < d || code_stride > glance::kQ8MaxStride || code_stride % 16)
    return fail(GLANCE_ERR_INVALID_ARG, "%s: code_stride must cover a row and be a multiple of 16", who);
  return GLANCE_OK;
}

bool bad_stride(int64_t stride, int d, int esize) {
  return stride < d || stride > glance::kQ8MaxStride || stride * esize % 16;
}

glance_status run_rows(const char* who, const void* x, int64_t x_stride, const void* residual, int64_t r_stride,
                       glance_dtype dtype, int M, int d, const float* weight, bool norm, float eps, void* total,
                       int64_t t_stride, void* codes, int64_t code_stride, float* scales, void* stream) {
  using glance::fail;
  using glance::overlap;
  if (!x || !codes || !scales) return fail(GLANCE_ERR_INVALID_ARG, "%s: null pointer argument", who);
  const int esize = dtype == GLANCE_BF16 ? 2 : 4;
  const glance_status st = check_shape(who, dtype, M, d, kMaxVecs * 16 / esize, code_stride);
  if (st != GLANCE_OK) return st;
  if (bad_stride(x_stride, d, esize) || (residual && bad_stride(r_stride, d, esize)) || (total && bad_stride(t_stride, d, esize)))
    return fail(GLANCE_ERR_INVALID_ARG, "%s: row strides must cover a row and be multiples of 16 bytes", who);
  if (norm && (!(eps >= 0.f) || !isfinite(eps))) return fail(GLANCE_ERR_INVALID_ARG, "%s: eps must be finite and >= 0", who);
  if (!glance::aligned16(x) || !glance::aligned16(residual) || !glance::aligned16(total) || !glance::aligned16(weight) ||
      !glance::aligned16(codes) || (reinterpret_cast<uintptr_t>(scales) & 3))
    return fail(GLANCE_ERR_INVALID_ARG, "%s: arrays must be 16-byte aligned", who);
  const int64_t row = static_cast<int64_t>(d) * esize, xs = x_stride * esize, rs = r_stride * esize, ts = t_stride * esize;
  const int64_t nx = span(M, xs, row), nr = residual ? span(M, rs, row) : 0, nt = total ? span(M, ts, row) : 0;
  const int64_t nc = span(M, code_stride, d), ns = 4ll * M;
  const bool clash = overlap(codes, nc, x, nx) || (residual && overlap(codes, nc, residual, nr)) ||
                     (total && overlap(codes, nc, total, nt)) || overlap(scales, ns, codes, nc) || overlap(scales, ns, x, nx) ||
                     (residual && overlap(scales, ns, residual, nr)) || (total && overlap(scales, ns, total, nt)) ||
                     (weight && (overlap(weight, 4ll * d, codes, nc) || overlap(weight, 4ll * d, scales, ns) ||
                                 (total && overlap(weight, 4ll * d, total, nt))));
  // the sum may take the place of x or of the residual, row for row
  const bool bad_total = total && ((overlap(total, nt, x, nx) && !(total == x && ts == xs)) ||
                                   (residual && overlap(total, nt, residual, nr) && !(total == residual && ts == rs)));
  if (clash || bad_total)
    return fail(GLANCE_ERR_INVALID_ARG, "%s: outputs must not overlap inputs (total may be x or residual itself)", who);
  RowParams p;
  p.x = static_cast<const char*>(x);
  p.residual = static_cast<const char*>(residual);
  p.total = static_cast<char*>(total);
  p.weight = weight;
  p.codes = static_cast<unsigned char*>(codes);
  p.scales = scales;
  p.x_stride = xs;
  p.r_stride = rs;
  p.t_stride = ts;
  p.c_stride = code_stride;
  p.M = M;
  p.vecs = static_cast<int>(row / 16);
  p.inv_d = static_cast<float>(1.0 / d);
  p.inv_d_low = static_cast<float>(1.0 / d - p.inv_d);
  p.eps = eps;
  int threads;
  const RowKernel k = dtype == GLANCE_BF16 ? pick<__nv_bfloat16>(p.vecs, norm, threads) : pick<float>(p.vecs, norm, threads);
  if (threads == 32) return launch(who, &p, reinterpret_cast<const void*>(k), (M + kWarpRows - 1) / kWarpRows, 32 * kWarpRows, stream);
  return launch(who, &p, reinterpret_cast<const void*>(k), M, threads, stream);
}

}  // namespace

extern "C" {

glance_status glance_q8_norm_rows(const void* x, int64_t x_stride, const void* residual, int64_t residual_stride,
                                  glance_dtype dtype, int M, int d, const float* weight, float eps, void* total,
                                  int64_t total_stride, void* codes, int64_t code_stride, float* scales, void* stream) {
  return run_rows("glance_q8_norm_rows", x, x_stride, residual, residual_stride, dtype, M, d, weight, true, eps, total,
                  total_stride, codes, code_stride, scales, stream);
}

glance_status glance_q8_rows(const void* x, int64_t x_stride, glance_dtype dtype, int M, int d, void* codes,
                             int64_t code_stride, float* scales, void* stream) {
  return run_rows("glance_q8_rows", x, x_stride, nullptr, 0, dtype, M, d, nullptr, false, 0.f, nullptr, 0, codes, code_stride,
                  scales, stream);
}

glance_status glance_q8_read_rows(const void* codes, int64_t code_stride, const float* scales, glance_dtype dtype, int M, int d,
                                  void* out, int64_t out_stride, void* stream) {
  using glance::fail;
  const char* who = "glance_q8_read_rows";
  if (!codes || !scales || !out) return fail(GLANCE_ERR_INVALID_ARG, "%s: null pointer argument", who);
  const glance_status st = check_shape(who, dtype, M, d, kMaxVecs * 8, code_stride);
  if (st != GLANCE_OK) return st;
  const int esize = dtype == GLANCE_BF16 ? 2 : 4;
  if (bad_stride(out_stride, d, esize))
    return fail(GLANCE_ERR_INVALID_ARG, "%s: row strides must cover a row and be multiples of 16 bytes", who);
  if (!glance::aligned16(codes) || !glance::aligned16(out) || (reinterpret_cast<uintptr_t>(scales) & 3))
    return fail(GLANCE_ERR_INVALID_ARG, "%s: arrays must be 16-byte aligned", who);
  const int64_t no = span(M, out_stride * esize, static_cast<int64_t>(d) * esize);
  if (glance::overlap(out, no, codes, span(M, code_stride, d)) || glance::overlap(out, no, scales, 4ll * M))
    return fail(GLANCE_ERR_INVALID_ARG, "%s: out must not overlap codes or scales", who);
  ReadParams p = {static_cast<const unsigned char*>(codes), scales, static_cast<char*>(out), code_stride, out_stride * esize, M, d / 16};
  const void* k = dtype == GLANCE_BF16 ? reinterpret_cast<const void*>(q8_read_rows_kernel<__nv_bfloat16>)
                                       : reinterpret_cast<const void*>(q8_read_rows_kernel<float>);
  return launch(who, &p, k, M, p.chunks < 256 ? (p.chunks + 31) / 32 * 32 : 256, stream);
}

}  // extern "C"
