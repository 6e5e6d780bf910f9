// Rows into and out of 4-bit K/V caches, and the walk + commit on them.
//
// The verify pass writes the packed tree rows' K/V to slots T..T+N of every
// layer's cache before tree attention reads them (arXiv 2609.00355, Definition
// 1), and a prompt's rows go in the same way. Each row is quantised by itself,
// so the cache after a commit is the cache that one-by-one decoding would have
// written: the path's rows move as they are.
//
// The row kernels read or write 256 bytes of bf16 and 72 of the cache per row
// and are bound by that: 12 layers x 2 x 8 heads x 8191 rows (516 MB) take 78.6
// us to write (97 % of the measured copy rate) and 76.9 to read (99 %). A
// thread has a group of 16 elements of four rows in flight; writing, the
// arithmetic would bind first (87.8 us with one element per operation) and is
// done two elements at a time. 64 rows of 36 layers take 3.9 and 2.9 us, a
// launch and one trip to memory.
#include "kv4_internal.cuh"

GLANCE_DEFINE_STATUS_WORD(status_kv4)

using namespace glance_dev;

namespace {

constexpr int kMaxLayers = 128;
constexpr int kSmallLayers = 48;  // parameter block of the common calls
constexpr int kRowThreads = 256;  // 32 rows at a time, 8 threads (one group of 16 elements each) a row
constexpr int kRowsPerPass = kRowThreads / 8;
constexpr int kPasses = 4;        // rows per thread of one block

struct Arrays {
  unsigned char* codes;
  unsigned char* scales;
};

template <int kLayers>
struct RowsParams {
  unsigned char* rows16;         // [n_layers][2][n_kv_heads][rows][128] bf16 (read or written)
  Arrays cache[2 * kLayers];     // per (layer, K or V)
  const int32_t* t_len;          // first slot = *t_len, or `first` where null
  int first;
  long long head_stride;         // slots
  int n_kv_heads, rows, t_cap;
  float global[2], inv_global[2];  // K, V; 1 / global rounded
};

// 32 bytes in one load / store.
__device__ __forceinline__ void ld32(const void* p, uint32_t (&r)[8]) {
  asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "l"(p));
}
__device__ __forceinline__ void st32(void* p, const uint32_t (&r)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// x / s rounded to nearest for a scale s of 4 significant bits, from inv =
// 1 / s rounded: the product is off by at most two units in the last place, and
// one step with the exact remainder (a fused multiply-add) leaves an error of
// 2^-46 of the quotient before the final rounding. That rounding is the
// quotient's: with s = m 2^e, m <= 15, the quotient is a multiple of 1 / m of a
// unit, so no midpoint of two fp32 numbers is nearer than 1 / 30 of one. A tie
// between two codes is exact this way and goes to the even one. Two at a time,
// with -s: the call is bound by instruction issue as much as by memory.
__device__ __forceinline__ unsigned long long quotient2(unsigned long long x, unsigned long long neg_s, unsigned long long inv) {
  const unsigned long long q = mul_f2(x, inv);
  return fma_f2(fma_f2(q, neg_s, x), inv, q);
}

// One group of 16 bf16 values (8 words) to 16 codes (2 words) and a scale.
__device__ __forceinline__ void quantise16(const uint32_t (&x)[8], float inv_g, uint32_t (&codes)[2],
                                           uint32_t& scale) {
  // the largest magnitude from the bit patterns, two at a time: their order is
  // that of the absolute values, infinities and NaN on top; rounding keeps the
  // order, so its product is the largest product
  uint32_t top = x[0] & 0x7FFF7FFFu;
#pragma unroll
  for (int i = 1; i < 8; ++i) top = __vmaxu2(top, x[i] & 0x7FFF7FFFu);
  const float amax = __uint_as_float(max(top & 0xFFFF0000u, top << 16)) * inv_g;
  const bool finite = amax < INFINITY;
  scale = finite ? scale1(__fdiv_rn(amax, 6.f)) & 0xFFu : 0x7Fu;
  const float s = f16x2_to_f32(scales2_to_f16(scale)).x;
  const bool any = finite && s > 0.f;
  const float inv_s = any ? __frcp_rn(s) : 0.f;
  const unsigned long long inv_g2 = pair_f2(inv_g, inv_g), inv_s2 = pair_f2(inv_s, inv_s), neg_s2 = pair_f2(-s, -s);
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t y = x[4 * w + i];
      split_f2(quotient2(mul_f2(pair_f2(__uint_as_float(y << 16), __uint_as_float(y & 0xFFFF0000u)), inv_g2), neg_s2, inv_s2),
               v[2 * i], v[2 * i + 1]);
    }
    codes[w] = codes8(v);
  }
  if (!any) codes[0] = codes[1] = 0u;
}

// Block (x, y): rows x * 128 .. of slice y = (layer * 2 + K or V) * heads + head.
template <int kLayers>
__global__ void __launch_bounds__(kRowThreads) kv4_write_rows_kernel(const __grid_constant__ RowsParams<kLayers> p) {
  pdl_wait_prior();
  pdl_launch_dependents();
  const int T = *p.t_len;
  if (T < 0 || T > p.t_cap - p.rows) {
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) report(GLANCE_DEV_TREE_CAPACITY);
    return;
  }
  const int lkv = blockIdx.y / p.n_kv_heads, head = blockIdx.y - lkv * p.n_kv_heads;
  const int is_v = lkv & 1;
  const int grp = threadIdx.x & 7;
  const int row0 = blockIdx.x * (kRowsPerPass * kPasses) + (threadIdx.x >> 3);
  const unsigned char* src = p.rows16 + static_cast<size_t>(blockIdx.y) * p.rows * 256 + grp * 32;
  const long long slot0 = head * p.head_stride + T;
  uint32_t x[kPasses][8];
#pragma unroll
  for (int u = 0; u < kPasses; ++u)  // behind the last row: that row again, not stored
    ld32(src + static_cast<size_t>(min(row0 + u * kRowsPerPass, p.rows - 1)) * 256, x[u]);
#pragma unroll
  for (int u = 0; u < kPasses; ++u) {
    const int row = row0 + u * kRowsPerPass;
    if (__all_sync(0xffffffffu, row >= p.rows)) break;
    uint32_t codes[2], scale;
    quantise16(x[u], p.inv_global[is_v], codes, scale);
    // the row's eight scales to its first thread: one store
    scale <<= 8 * (grp & 3);
    scale |= __shfl_xor_sync(0xffffffffu, scale, 1);
    scale |= __shfl_xor_sync(0xffffffffu, scale, 2);
    const uint32_t upper = __shfl_xor_sync(0xffffffffu, scale, 4);
    if (row >= p.rows || !GLANCE_IN_BOUNDS(T + row, p.t_cap)) continue;
    const long long slot = slot0 + row;
    *reinterpret_cast<uint2*>(p.cache[lkv].codes + slot * glance::kKv4CodeBytes + grp * 8) = make_uint2(codes[0], codes[1]);
    if (grp == 0) *reinterpret_cast<uint2*>(p.cache[lkv].scales + slot * glance::kKv4ScaleBytes) = make_uint2(scale, upper);
  }
}

template <int kLayers>
__global__ void __launch_bounds__(kRowThreads) kv4_read_rows_kernel(const __grid_constant__ RowsParams<kLayers> p) {
  pdl_wait_prior();  // and no early start for the kernel behind: the rows may be the prefix of its 16-bit cache
  const int lkv = blockIdx.y / p.n_kv_heads, head = blockIdx.y - lkv * p.n_kv_heads;
  const float g = p.global[lkv & 1];
  const int grp = threadIdx.x & 7;
  const int row0 = blockIdx.x * (kRowsPerPass * kPasses) + (threadIdx.x >> 3);
  unsigned char* dst = p.rows16 + static_cast<size_t>(blockIdx.y) * p.rows * 256 + grp * 32;
  const long long slot0 = head * p.head_stride + p.first;
  uint2 codes[kPasses];
  uint32_t scale[kPasses];
#pragma unroll
  for (int u = 0; u < kPasses; ++u) {
    const int row = row0 + u * kRowsPerPass;
    if (row < p.rows && GLANCE_IN_BOUNDS(p.first + row, p.t_cap)) {
      codes[u] = *reinterpret_cast<const uint2*>(p.cache[lkv].codes + (slot0 + row) * glance::kKv4CodeBytes + grp * 8);
      scale[u] = p.cache[lkv].scales[(slot0 + row) * glance::kKv4ScaleBytes + grp];
    }
  }
#pragma unroll
  for (int u = 0; u < kPasses; ++u) {
    const int row = row0 + u * kRowsPerPass;
    if (row >= p.rows || !GLANCE_IN_BOUNDS(p.first + row, p.t_cap)) continue;
    const float s = f16x2_to_f32(scales2_to_f16(scale[u])).x * g;  // 4 bits by 24: rounded once
    uint32_t r[8];
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      uint32_t h[4];
      codes8_to_f16(w ? codes[u].y : codes[u].x, h);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 c = f16x2_to_f32(h[i]);
        r[4 * w + i] = pack_bf16x2(c.x * s, c.y * s);
      }
    }
    st32(dst + static_cast<size_t>(row) * 256, r);
  }
}

template <int kLayers>
glance_status launch_rows(const char* who, bool write, void* rows16, const glance_kv4* layers, int n_layers, int rows,
                          int first, cudaStream_t s) {
  const glance_kv4& l0 = layers[0];
  RowsParams<kLayers> p;
  p.rows16 = static_cast<unsigned char*>(rows16);
  p.t_len = l0.t_len;
  p.first = first;
  p.head_stride = l0.head_stride;
  p.n_kv_heads = l0.n_kv_heads;
  p.rows = rows;
  p.t_cap = l0.t_cap;
  const float gl[2] = {l0.k_global, l0.v_global};
  for (int i = 0; i < 2; ++i) {
    p.global[i] = gl[i];
    p.inv_global[i] = 1.f / gl[i];
  }
  for (int l = 0; l < n_layers; ++l) {
    p.cache[2 * l] = {static_cast<unsigned char*>(layers[l].k), static_cast<unsigned char*>(layers[l].k_scale)};
    p.cache[2 * l + 1] = {static_cast<unsigned char*>(layers[l].v), static_cast<unsigned char*>(layers[l].v_scale)};
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((rows + kRowsPerPass * kPasses - 1) / (kRowsPerPass * kPasses), n_layers * 2 * l0.n_kv_heads);
  cfg.blockDim = dim3(kRowThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = write ? cudaLaunchKernelEx(&cfg, kv4_write_rows_kernel<kLayers>, p)
                              : cudaLaunchKernelEx(&cfg, kv4_read_rows_kernel<kLayers>, p);
  if (e != cudaSuccess) return glance::cuda_fail(e, who);
  return GLANCE_OK;
}

glance_status rows_call(const char* who, bool write, void* rows16, const glance_kv4* layers, int n_layers, int rows,
                        int first, void* stream) {
  using glance::fail;
  if (!rows16 || !layers) return fail(GLANCE_ERR_INVALID_ARG, "%s: null pointer argument", who);
  if (n_layers < 1 || n_layers > kMaxLayers || rows < 1 || first < 0)
    return fail(GLANCE_ERR_INVALID_ARG, "%s: need 1 <= n_layers <= %d, rows >= 1 and first >= 0", who, kMaxLayers);
  if (reinterpret_cast<uintptr_t>(rows16) & 31)
    return fail(GLANCE_ERR_INVALID_ARG, "%s: the bf16 rows must be 32-byte aligned", who);
  const glance_kv4& l0 = layers[0];
  for (int l = 0; l < n_layers; ++l) {
    const glance_kv4& x = layers[l];
    const glance_status st = glance::check_kv4(who, x, rows, l);
    if (st != GLANCE_OK) return st;
    if (x.t_len != l0.t_len || x.n_kv_heads != l0.n_kv_heads || x.t_cap != l0.t_cap ||
        x.head_stride != l0.head_stride || x.k_global != l0.k_global || x.v_global != l0.v_global)
      return fail(GLANCE_ERR_INVALID_ARG, "%s: every layer needs the same t_len, geometry and globals (layer %d)", who, l);
  }
  if (!write && first > l0.t_cap - rows)
    return fail(GLANCE_ERR_INVALID_ARG, "%s: slots %d .. %lld end behind t_cap = %d", who, first,
                static_cast<long long>(first) + rows - 1, l0.t_cap);
  if (n_layers * 2ll * l0.n_kv_heads > 65535)
    return fail(GLANCE_ERR_UNSUPPORTED, "%s: need n_layers * n_kv_heads <= 32767", who);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (n_layers <= kSmallLayers) return launch_rows<kSmallLayers>(who, write, rows16, layers, n_layers, rows, first, s);
  return launch_rows<kMaxLayers>(who, write, rows16, layers, n_layers, rows, first, s);
}

}  // namespace

extern "C" glance_status glance_kv4_write_rows(const void* src, const glance_kv4* layers, int n_layers, int rows,
                                               void* stream) {
  return rows_call("glance_kv4_write_rows", true, const_cast<void*>(src), layers, n_layers, rows, 0, stream);
}

extern "C" glance_status glance_kv4_read_rows(const glance_kv4* layers, int n_layers, int first, int rows, void* dst,
                                              void* stream) {
  return rows_call("glance_kv4_read_rows", false, dst, layers, n_layers, rows, first, stream);
}

// ------------------------------------------------------------- walk and commit
//
// The walk of Definition 1 (A(S): descend while the row's argmax is a child)
// and the move of the path's rows, as accept_commit_kernel does them for 16-
// and 32-bit caches. A 4-bit row is 72 bytes, so a slice (layer, K or V, kv
// head) moves at most 17 rows = 1.2 KB: one warp holds it in registers (three
// 16-byte code pieces and one scale row per lane), which makes "read every
// source before any slot is written" a warp barrier, and eight slices share a
// block's walk.

namespace {

constexpr int kCommitThreads = 256;
constexpr int kCommitWarps = kCommitThreads / 32;
constexpr int kMaxB = 16;
constexpr int kMaxEntries = 960;  // requests x layers: the pointers fill the 32 KB of launch parameters
constexpr int kSmallEntries = 64;
constexpr int kMaxPath = 17;

struct CommitReq {
  const int32_t* token;
  const int32_t* parent;
  const int32_t* depth;
  int32_t* t_len;
  long long head_stride;
  int t_cap;
};

template <int kEntries>
struct CommitParams {
  const int32_t* argmax;  // [B][rows]
  const float* gap;       // [B][rows] or null (no gate)
  float gate;
  int32_t* gated;         // [B] or null
  int rows, L, B, n_layers, n_kv_heads, blocks_per_req;
  int32_t* n_accepted;
  int32_t* accepted_tok;
  int32_t* new_root;
  uint32_t* ticket;       // [B]
  CommitReq req[kMaxB];
  Arrays cache[2 * kEntries];  // [B][n_layers][2]
};

template <int kEntries>
__global__ void __launch_bounds__(kCommitThreads)
    kv4_accept_commit_kernel(const __grid_constant__ CommitParams<kEntries> p) {
  __shared__ int s_tok[256], s_par[256], s_dep[256], s_arg[256];
  __shared__ float s_gap[256];
  __shared__ int s_path[kMaxPath];
  __shared__ int s_a, s_root, s_gated, s_T, s_last;
  pdl_wait_prior();  // nothing is read before the previous kernel's writes are visible
  const int req = blockIdx.x / p.blocks_per_req;
  const int block = blockIdx.x - req * p.blocks_per_req;
  const CommitReq& rq = p.req[req];
  const int i = threadIdx.x;
  if (i < p.rows) {
    s_tok[i] = rq.token[i];
    s_par[i] = rq.parent[i];
    s_dep[i] = rq.depth[i];
    s_arg[i] = p.argmax[req * p.rows + i];
    s_gap[i] = p.gap ? p.gap[req * p.rows + i] : INFINITY;
  }
  if (i == 0) s_T = *rq.t_len;
  __syncthreads();
  const int warp = i >> 5, lane = i & 31;
  if (warp == 0) {
    int u = 0, a = 0;
    bool gated = false;
    if (lane == 0) s_path[0] = 0;
    for (int step = 0; step <= p.L; ++step) {
      if (s_gap[u] < p.gate) {  // a near-tie on the path: the caller decides this row
        gated = true;
        break;
      }
      if (s_dep[u] >= p.L || a >= p.L) break;
      const int want = s_arg[u];
      int found = -1;
      for (int base = 0; base < p.rows && found < 0; base += 32) {
        const int c = base + lane;
        const unsigned hit = __ballot_sync(0xffffffffu, c > 0 && c < p.rows && s_par[c] == u && s_tok[c] == want);
        if (hit) found = base + __ffs(hit) - 1;
      }
      if (found < 0) break;
      u = found;
      ++a;
      if (lane == 0) s_path[a] = u;
    }
    if (lane == 0) {
      s_a = a;
      s_root = s_arg[u];
      s_gated = gated ? 1 : 0;
    }
  }
  __syncthreads();
  const int a = s_a, T = s_T;
  const bool room = T >= 0 && T <= rq.t_cap - p.rows;
  if (!room && block == 0 && i == 0) report(GLANCE_DEV_TREE_CAPACITY);
  const int slice = block * kCommitWarps + warp;  // (layer * 2 + K or V) * heads + head
  if (room && a > 0 && slice < p.n_layers * 2 * p.n_kv_heads) {
    const int lkv = slice / p.n_kv_heads, head = slice - lkv * p.n_kv_heads;
    const Arrays& c = p.cache[req * p.n_layers * 2 + lkv];
    const long long slot0 = head * rq.head_stride + T;
    uint4* codes = reinterpret_cast<uint4*>(c.codes + slot0 * glance::kKv4CodeBytes);
    uint2* scales = reinterpret_cast<uint2*>(c.scales + slot0 * glance::kKv4ScaleBytes);
    const int n = 4 * (a + 1);  // 16-byte pieces, <= 68
    uint4 x[3];
    uint2 sc;
#pragma unroll
    for (int u = 0; u < 3; ++u) {
      const int e = lane + 32 * u;
      if (e < n && GLANCE_IN_BOUNDS(T + s_path[e >> 2], rq.t_cap)) x[u] = codes[s_path[e >> 2] * 4 + (e & 3)];
    }
    if (lane <= a && GLANCE_IN_BOUNDS(T + s_path[lane], rq.t_cap)) sc = scales[s_path[lane]];
    __syncwarp();  // every source is in registers
#pragma unroll
    for (int u = 0; u < 3; ++u) {
      const int e = lane + 32 * u;
      if (e < n && GLANCE_IN_BOUNDS(T + (e >> 2), rq.t_cap)) codes[e] = x[u];
    }
    if (lane <= a && GLANCE_IN_BOUNDS(T + lane, rq.t_cap)) scales[lane] = sc;
  }
  // the last block of a request writes its results (all have read T by then)
  __threadfence();
  __syncthreads();
  if (i == 0) s_last = atomicAdd(p.ticket + req, 1u) == static_cast<uint32_t>(p.blocks_per_req - 1);
  __syncthreads();
  if (!s_last) return;
  if (i == 0) {
    p.ticket[req] = 0;
    p.n_accepted[req] = a;
    p.new_root[req] = s_root;
    if (p.gated) p.gated[req] = s_gated;
    if (room) *rq.t_len = T + a + 1;
  }
  if (i >= 1 && i <= a && GLANCE_IN_BOUNDS(s_path[i], p.rows)) p.accepted_tok[req * p.L + i - 1] = s_tok[s_path[i]];
}

template <int kEntries>
glance_status launch_commit(const char* who, const glance_tree* trees, int B, const int32_t* argmax, const float* gap,
                            float gate, const glance_kv4* layers, int n_layers, int32_t* n_accepted,
                            int32_t* accepted_tok, int32_t* new_root, int32_t* gated, void* workspace,
                            cudaStream_t s) {
  using glance::fail;
  CommitParams<kEntries> p;
  const int n = trees[0].n, L = trees[0].L, heads = layers[0].n_kv_heads;
  for (int r = 0; r < B; ++r) {
    const glance_tree& t = trees[r];
    if (t.n != n || t.L != L || n < 1 || n > 255 || L < 1 || L > 16 || !t.token || !t.parent || !t.depth)
      return fail(GLANCE_ERR_INVALID_ARG, "%s: bad tree struct (request %d)", who, r);
    const glance_kv4& f = layers[r * n_layers];
    for (int l = 0; l < n_layers; ++l) {
      const glance_kv4& x = layers[r * n_layers + l];
      const glance_status st = glance::check_kv4(who, x, n + 1, r * n_layers + l);
      if (st != GLANCE_OK) return st;
      if (x.n_kv_heads != heads || x.t_cap != f.t_cap || x.head_stride != f.head_stride || x.t_len != f.t_len)
        return fail(GLANCE_ERR_INVALID_ARG,
                    "%s: every layer of a request must share geometry and t_len (request %d, layer %d)", who, r, l);
      Arrays* c = p.cache + 2 * (r * n_layers + l);
      c[0] = {static_cast<unsigned char*>(x.k), static_cast<unsigned char*>(x.k_scale)};
      c[1] = {static_cast<unsigned char*>(x.v), static_cast<unsigned char*>(x.v_scale)};
    }
    for (int q = 0; q < r; ++q)
      if (layers[q * n_layers].t_len == f.t_len)
        return fail(GLANCE_ERR_INVALID_ARG, "%s: requests %d and %d share t_len", who, q, r);
    p.req[r] = {t.token, t.parent, t.depth, f.t_len, f.head_stride, f.t_cap};
  }
  p.argmax = argmax;
  p.gap = gap;
  p.gate = gate;
  p.gated = gated;
  p.rows = n + 1;
  p.L = L;
  p.B = B;
  p.n_layers = n_layers;
  p.n_kv_heads = heads;
  p.blocks_per_req = (n_layers * 2 * heads + kCommitWarps - 1) / kCommitWarps;
  p.n_accepted = n_accepted;
  p.accepted_tok = accepted_tok;
  p.new_root = new_root;
  p.ticket = static_cast<uint32_t*>(workspace);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(B * p.blocks_per_req);
  cfg.blockDim = dim3(kCommitThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];  // no early start for the kernel behind it: this one writes T and the prefix
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kv4_accept_commit_kernel<kEntries>, p);
  if (e != cudaSuccess) return glance::cuda_fail(e, who);
  return GLANCE_OK;
}

bool commit_sizes_ok(int B, int n_layers) {
  return B >= 1 && B <= kMaxB && n_layers >= 1 && n_layers <= kMaxLayers && B * n_layers <= kMaxEntries;
}

}  // namespace

extern "C" size_t glance_kv4_accept_commit_workspace_bytes(int B, int n_layers) {
  return commit_sizes_ok(B, n_layers) ? 256 : 0;
}

extern "C" glance_status glance_kv4_accept_commit(const glance_tree* trees, int B, const int32_t* argmax,
                                                  const float* gap, float gate_threshold, const glance_kv4* layers,
                                                  int n_layers, int32_t* n_accepted, int32_t* accepted_tok,
                                                  int32_t* new_root, int32_t* gated, void* workspace,
                                                  size_t workspace_bytes, void* stream) {
  using glance::fail;
  const char* who = "glance_kv4_accept_commit";
  if (!trees || !argmax || !layers || !n_accepted || !accepted_tok || !new_root || !workspace)
    return fail(GLANCE_ERR_INVALID_ARG, "%s: null pointer argument", who);
  if ((gap == nullptr) != (gated == nullptr))
    return fail(GLANCE_ERR_INVALID_ARG, "%s: give both gap and gated, or neither", who);
  if (!commit_sizes_ok(B, n_layers))
    return fail(GLANCE_ERR_INVALID_ARG, "%s: need 1 <= B <= %d, 1 <= n_layers <= %d and B * n_layers <= %d", who, kMaxB,
                kMaxLayers, kMaxEntries);
  if (workspace_bytes < 256) return fail(GLANCE_ERR_CAPACITY, "%s: workspace must be >= 256 bytes", who);
  if (reinterpret_cast<uintptr_t>(workspace) & 3)
    return fail(GLANCE_ERR_INVALID_ARG, "%s: workspace must be 4-byte aligned", who);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const float gate = gap ? gate_threshold : 0.f;
  if (B * n_layers <= kSmallEntries)
    return launch_commit<kSmallEntries>(who, trees, B, argmax, gap, gate, layers, n_layers, n_accepted, accepted_tok,
                                        new_root, gated, workspace, s);
  return launch_commit<kMaxEntries>(who, trees, B, argmax, gap, gate, layers, n_layers, n_accepted, accepted_tok,
                                    new_root, gated, workspace, s);
}
