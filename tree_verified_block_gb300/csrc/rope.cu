// Per-head RMS norm of q and k with the rotary position in the same pass, k
// and v into the cache.
//
// A target's attention (arXiv 2609.00355, Definition 1, runs it over the
// packed rows; Sections 3.1 and 4.2 over a prompt of text and image tokens)
// takes q and k rows that are RMS-normalised per head and rotated by their
// position: y = x / sqrt(mean x^2 + eps) * w, then for j < D / 2
//   (y_j, y_{j + D/2}) -> (y_j c - y_{j + D/2} s, y_{j + D/2} c + y_j s),
// c, s = cos, sin of pos[axis(j)] * theta^(-2j/D). An image token has three
// positions (time, height, width) and each frequency belongs to one of them.
//
// Angles: a frequency is held as the fraction of a turn per position times
// 2^64, so that position * frequency in 64-bit wrapping integer arithmetic is
// the angle modulo one turn, exact but for the frequency's own rounding
// (2^-53 relative): no position is too far. The top 32 bits go to fp32, whose 24
// bits leave the angle off by up to 2^-26 + 2^-32 of a turn (measured over 10^7
// angles: 1.016 * 2^-26).
#include <math.h>

#include "kv4_internal.cuh"

GLANCE_DEFINE_STATUS_WORD(status_rope)

using namespace glance_dev;

namespace {

constexpr int kMaxB = 16;
constexpr int kThreads = 128;
constexpr int kMaxRows = 2;  // rows of one block

struct Cache {
  char* k;
  char* v;
  const int32_t* t_len;
  long long head_stride, row_stride;  // bytes
  int t_cap;
};

struct RopeParams {
  const char* qkv;
  char* q_out;
  const float* q_norm;
  const float* k_norm;
  const int32_t* pos;   // [n_axes][B M]
  long long row_stride;  // bytes
  int B, M, Hq, Hkv, block_rows, blocks_per_req;
  float eps;
  Cache kv[kMaxB];
  unsigned long long turn[64];
  uint8_t axis[64];
};

template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int n = 4;
  static __device__ __forceinline__ void unpack(const uint4& v, float (&f)[4]) {
    f[0] = __uint_as_float(v.x);
    f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z);
    f[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int n = 8;
  static __device__ __forceinline__ void unpack(const uint4& v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
  }
};

// A head is held by kLanes threads, thread i with dims kV i .. kV i + kV - 1
// and the same dims of the other half, so a rotation pair is in one thread.
// Block: up to kMaxRows rows of one request; their cosines and sines go to
// shared memory first (each is used by every q and k head of the row). Bound by
// memory: each element is read and written once, so a thread has the loads of
// kAhead heads (96 bytes) in flight, the first ones before the cosines. 16383
// rows of 32 / 8 heads x 128 (403 MB): 63.7 us, 93 % of the measured copy rate
// (one head in flight: 80.6); 64 rows 3.3 us, a launch and two trips to memory.
constexpr int kAhead = 3;

template <typename T, int kHeadDim>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int kV = Vec<T>::n;
  constexpr int kHalf = kHeadDim / 2;
  constexpr int kLanes = kHalf / kV;
  constexpr int kSlots = kThreads / kLanes;  // heads at a time
  constexpr int kHeadBytes = kHeadDim * sizeof(T), kHalfBytes = kHeadBytes / 2;
  __shared__ float2 s_cs[kMaxRows][kHalf];
  pdl_wait_prior();  // and no early start for the kernel behind: rows of a prompt may be its prefix
  const int req = blockIdx.x / p.blocks_per_req;
  const int row0 = (blockIdx.x - req * p.blocks_per_req) * p.block_rows;
  const int n_rows = min(p.block_rows, p.M - row0);
  const int i = threadIdx.x % kLanes, slot = threadIdx.x / kLanes;
  const int n_heads = p.Hq + 2 * p.Hkv;
  const char* src = p.qkv + (static_cast<long long>(req) * p.M + row0) * p.row_stride + i * 16;
  uint4 lo[kAhead], hi[kAhead];
  const auto load = [&](int h0) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int h = h0 + u * kSlots + slot;
      lo[u] = hi[u] = make_uint4(0, 0, 0, 0);
      if (h < n_heads) {
        lo[u] = __ldcs(reinterpret_cast<const uint4*>(src + static_cast<long long>(h) * kHeadBytes));
        hi[u] = __ldcs(reinterpret_cast<const uint4*>(src + static_cast<long long>(h) * kHeadBytes + kHalfBytes));
      }
    }
  };
  load(0);
  const Cache& kv = p.kv[req];
  const int T0 = *kv.t_len;
  const bool room = T0 >= 0 && T0 <= kv.t_cap - p.M;
  if (!room && row0 == 0 && threadIdx.x == 0) report(GLANCE_DEV_TREE_CAPACITY);
  for (int e = threadIdx.x; e < n_rows * kHalf; e += kThreads) {
    const int r = e / kHalf, j = e % kHalf;
    const long long at = static_cast<long long>(p.axis[j]) * p.B * p.M + static_cast<long long>(req) * p.M + row0 + r;
    const unsigned long long a = static_cast<unsigned long long>(static_cast<long long>(p.pos[at])) * p.turn[j];
    // [-1, 1) half turns
    const float x = static_cast<float>(static_cast<int32_t>(a >> 32)) * 4.656612873077393e-10f;
    float s, c;
    sincospif(x, &s, &c);
    s_cs[r][j % kV * kLanes + j / kV] = make_float2(c, s);  // a head's threads read next to each other
  }
  __syncthreads();
  for (int r = 0; r < n_rows; ++r) {
    const long long row = static_cast<long long>(req) * p.M + row0 + r;
    const int at = T0 + row0 + r;  // cache slot
    for (int h0 = 0; h0 < n_heads; h0 += kAhead * kSlots) {
      if (h0) load(h0);
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {  // all threads of a warp take part in the sum's shuffles
        const int h = h0 + u * kSlots + slot;
        const bool live = h < n_heads, is_q = h < p.Hq, is_v = h >= p.Hq + p.Hkv;
        float a[kV], b[kV];
        Vec<T>::unpack(lo[u], a);
        Vec<T>::unpack(hi[u], b);
        const float* w = is_q ? p.q_norm : p.k_norm;
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < kV; ++e) ss = fmaf(a[e], a[e], fmaf(b[e], b[e], ss));
#pragma unroll
        for (int o = kLanes / 2; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (!live) continue;
        if (!is_v) {
          if (w) {
            const float inv = rsqrtf(ss * (1.f / kHeadDim) + p.eps);
#pragma unroll
            for (int e = 0; e < kV; ++e) {
              a[e] *= inv * __ldg(w + i * kV + e);
              b[e] *= inv * __ldg(w + i * kV + kHalf + e);
            }
          }
#pragma unroll
          for (int e = 0; e < kV; ++e) {
            const float2 cs = s_cs[r][e * kLanes + i];
            const float x = a[e], y = b[e];
            a[e] = x * cs.x - y * cs.y;
            b[e] = y * cs.x + x * cs.y;
          }
          lo[u] = Vec<T>::pack(a);
          hi[u] = Vec<T>::pack(b);
        }
        char* dst;
        if (is_q) {
          dst = p.q_out + (row * p.Hq + h) * kHeadBytes;
        } else {
          if (!room || !GLANCE_IN_BOUNDS(at, kv.t_cap)) continue;
          const int g = is_v ? h - p.Hq - p.Hkv : h - p.Hq;
          dst = (is_v ? kv.v : kv.k) + g * kv.head_stride + at * kv.row_stride;
        }
        *reinterpret_cast<uint4*>(dst + i * 16) = lo[u];
        *reinterpret_cast<uint4*>(dst + i * 16 + kHalfBytes) = hi[u];
      }
    }
    src += p.row_stride;
    if (r + 1 < n_rows) load(0);
  }
}

typedef void (*RopeKernel)(const RopeParams);

RopeKernel pick(glance_dtype dtype, int head_dim) {
  if (dtype == GLANCE_BF16)
    return head_dim == 128 ? qk_norm_rope_kernel<__nv_bfloat16, 128>
           : head_dim == 64 ? qk_norm_rope_kernel<__nv_bfloat16, 64>
                            : qk_norm_rope_kernel<__nv_bfloat16, 32>;
  return head_dim == 128 ? qk_norm_rope_kernel<float, 128>
         : head_dim == 64 ? qk_norm_rope_kernel<float, 64>
                          : qk_norm_rope_kernel<float, 32>;
}

}  // namespace

extern "C" glance_status glance_rope_init(glance_rope* rope, int head_dim, double theta, int n_axes,
                                          const int32_t* sections, int interleaved) {
  using glance::fail;
  const char* who = "glance_rope_init";
  if (!rope) return fail(GLANCE_ERR_INVALID_ARG, "%s: null rope", who);
  if (head_dim != 32 && head_dim != 64 && head_dim != 128)
    return fail(GLANCE_ERR_UNSUPPORTED, "%s: head_dim must be 32, 64 or 128", who);
  if (!(theta > 0.0) || !isfinite(theta)) return fail(GLANCE_ERR_INVALID_ARG, "%s: theta must be finite and > 0", who);
  if (n_axes < 1 || n_axes > 4 || (n_axes > 1 && !sections))
    return fail(GLANCE_ERR_INVALID_ARG, "%s: need 1 <= n_axes <= 4, and sections with more than one axis", who);
  const int half = head_dim / 2;
  int sec[4] = {half, 0, 0, 0};
  if (sections) {
    int sum = 0;
    for (int a = 0; a < n_axes; ++a) {
      sec[a] = sections[a];
      if (sec[a] < 1 || sec[a] > half) return fail(GLANCE_ERR_INVALID_ARG, "%s: every section must be in 1 .. head_dim / 2", who);
      if (interleaved && a > 0 && sec[a] > (half - a + n_axes - 1) / n_axes)
        return fail(GLANCE_ERR_INVALID_ARG, "%s: section %d has no room in turn", who, a);
      sum += sec[a];
    }
    if (sum != half) return fail(GLANCE_ERR_INVALID_ARG, "%s: the sections must add up to head_dim / 2 = %d", who, half);
  }
  glance_rope r = {};
  r.head_dim = head_dim;
  r.n_axes = n_axes;
  int run = 0, left = sec[0];  // runs: the current axis and what it has left
  for (int j = 0; j < half; ++j) {
    const double turns = pow(theta, -2.0 * j / head_dim) / 6.283185307179586476925;
    if (!isfinite(turns)) return fail(GLANCE_ERR_INVALID_ARG, "%s: theta is too small", who);
    const double frac = turns - floor(turns);
    const double scaled = frac * 18446744073709551616.0;
    r.turn[j] = scaled >= 18446744073709549568.0 ? 0ull : static_cast<uint64_t>(scaled + 0.5);
    if (interleaved) {
      const int a = j % n_axes;
      r.axis[j] = static_cast<uint8_t>(a && j / n_axes < sec[a] ? a : 0);
    } else {
      while (left == 0) left = sec[++run];
      r.axis[j] = static_cast<uint8_t>(run);
      --left;
    }
  }
  *rope = r;
  return GLANCE_OK;
}

extern "C" glance_status glance_qk_norm_rope(const void* qkv, glance_dtype dtype, int B, int M, int64_t row_stride,
                                             int n_q_heads, const float* q_norm, const float* k_norm, float eps,
                                             const int32_t* pos, const glance_rope* rope, void* q_out,
                                             const glance_kv* kv, void* stream) {
  using glance::fail;
  const char* who = "glance_qk_norm_rope";
  if (!qkv || !pos || !rope || !q_out || !kv) return fail(GLANCE_ERR_INVALID_ARG, "%s: null pointer argument", who);
  if (dtype != GLANCE_BF16 && dtype != GLANCE_F32) return fail(GLANCE_ERR_INVALID_ARG, "%s: dtype must be F32 or BF16", who);
  if (B < 1 || B > kMaxB || M < 1 || M > (1 << 30) / B)
    return fail(GLANCE_ERR_INVALID_ARG, "%s: need 1 <= B <= %d, M >= 1 and B * M <= 2^30", who, kMaxB);
  const int D = rope->head_dim, Hkv = kv[0].n_kv_heads;
  if ((D != 32 && D != 64 && D != 128) || rope->n_axes < 1 || rope->n_axes > 4)
    return fail(GLANCE_ERR_INVALID_ARG, "%s: rope is not filled (glance_rope_init)", who);
  for (int j = 0; j < D / 2; ++j)
    if (rope->axis[j] >= rope->n_axes) return fail(GLANCE_ERR_INVALID_ARG, "%s: rope has a bad axis", who);
  if (n_q_heads < 1 || n_q_heads > 4096 || Hkv < 1 || Hkv > 4096)
    return fail(GLANCE_ERR_INVALID_ARG, "%s: need 1 to 4096 heads of each kind", who);
  if (!(eps >= 0.f) || !isfinite(eps)) return fail(GLANCE_ERR_INVALID_ARG, "%s: eps must be finite and >= 0", who);
  const int esize = dtype == GLANCE_BF16 ? 2 : 4;
  const int64_t width = static_cast<int64_t>(n_q_heads + 2 * Hkv) * D;
  if (row_stride < width || row_stride > (1ll << 40) || (row_stride * esize) % 16)
    return fail(GLANCE_ERR_INVALID_ARG, "%s: row_stride must cover the heads and be a multiple of 16 bytes", who);
  if (!glance::aligned16(qkv) || !glance::aligned16(q_out))
    return fail(GLANCE_ERR_INVALID_ARG, "%s: qkv and q_out must be 16-byte aligned", who);
  {
    const char* a0 = static_cast<const char*>(qkv);
    const char* a1 = a0 + ((static_cast<int64_t>(B) * M - 1) * row_stride + width) * esize;
    const char* b0 = static_cast<const char*>(q_out);
    const char* b1 = b0 + static_cast<int64_t>(B) * M * n_q_heads * D * esize;
    if (a0 < b1 && b0 < a1) return fail(GLANCE_ERR_INVALID_ARG, "%s: q_out overlaps qkv", who);
  }
  RopeParams p;
  for (int r = 0; r < B; ++r) {
    const glance_kv& x = kv[r];
    if (!x.k || !x.v || !x.t_len) return fail(GLANCE_ERR_INVALID_ARG, "%s: null kv array (request %d)", who, r);
    if (x.dtype != dtype || x.head_dim != D || x.n_kv_heads != Hkv)
      return fail(GLANCE_ERR_INVALID_ARG, "%s: kv must have the call's dtype, rope's head_dim and one n_kv_heads (request %d)",
                  who, r);
    if (x.t_cap < M || x.row_stride < D || x.head_stride < static_cast<int64_t>(x.t_cap) * x.row_stride)
      return fail(GLANCE_ERR_INVALID_ARG, "%s: bad kv geometry (request %d)", who, r);
    if (!glance::aligned16(x.k) || !glance::aligned16(x.v) || (x.row_stride * esize) % 16 || (x.head_stride * esize) % 16)
      return fail(GLANCE_ERR_INVALID_ARG, "%s: k/v must be 16-byte aligned with 16-byte strides (request %d)", who, r);
    for (int q = 0; q < r; ++q)
      if (kv[q].k == x.k || kv[q].v == x.v)
        return fail(GLANCE_ERR_INVALID_ARG, "%s: requests %d and %d share a cache", who, q, r);
    p.kv[r] = {static_cast<char*>(x.k), static_cast<char*>(x.v), x.t_len, x.head_stride * esize, x.row_stride * esize, x.t_cap};
  }
  p.qkv = static_cast<const char*>(qkv);
  p.q_out = static_cast<char*>(q_out);
  p.q_norm = q_norm;
  p.k_norm = k_norm;
  p.pos = pos;
  p.row_stride = row_stride * esize;
  p.B = B;
  p.M = M;
  p.Hq = n_q_heads;
  p.Hkv = Hkv;
  p.eps = eps;
  // one row a block until the rows fill the GPU several times over
  p.block_rows = static_cast<int64_t>(B) * M >= 16ll * glance::num_sms() ? kMaxRows : 1;
  p.blocks_per_req = (M + p.block_rows - 1) / p.block_rows;
  for (int j = 0; j < 64; ++j) {
    p.turn[j] = rope->turn[j];
    p.axis[j] = rope->axis[j];
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(B) * p.blocks_per_req);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, pick(dtype, D), p);
  if (e != cudaSuccess) return glance::cuda_fail(e, who);
  return GLANCE_OK;
}
