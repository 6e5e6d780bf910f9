// Ancestor-masked tree attention over 4-bit K/V caches (one layer, B requests).
//
// arXiv 2609.00355, Definition 1: packed row i sees the prefix slots 0..T-1
// and the tree slots of its own ancestors; N = 0 is one row, plain decoding.
#include "kv4_internal.cuh"

GLANCE_DEFINE_STATUS_WORD(status_kv4_attention)

using namespace glance_dev;

namespace {

constexpr int kD = glance::kKv4D;
constexpr int kMaxB = 16;
constexpr float kLog2e = 1.4426950408889634f;

struct Request {
  const unsigned char* k;
  const unsigned char* k_scale;
  const unsigned char* v;
  const unsigned char* v_scale;
  const uint64_t* anc;      // null: every row sees itself only (N = 0)
  const int32_t* t_len;
  long long head_stride;
  float k_global, v_global;
  int t_cap;
};

struct Params {
  Request req[kMaxB];
  const __nv_bfloat16* q;
  __nv_bfloat16* out;
  int rows, Hq, G, W;
  float scale_log2;
};

// One block per (request, row, head), one thread per output dim; keys one
// block of 128 at a time.
__global__ void __launch_bounds__(kD) kv4_attention_plain_kernel(const __grid_constant__ Params p) {
  __shared__ float s_q[kD], s_p[kD], s_red[4];
  pdl_wait_prior();
  const int h = blockIdx.x % p.Hq, i = blockIdx.x / p.Hq % p.rows, r = blockIdx.x / p.Hq / p.rows;
  const Request& rq = p.req[r];
  const int t = threadIdx.x, T = *rq.t_len;
  if (T < 0 || T > rq.t_cap - p.rows) {
    if (i == 0 && h == 0 && t == 0) report(GLANCE_DEV_TREE_CAPACITY);
    return;
  }
  const size_t qi = ((static_cast<size_t>(r) * p.rows + i) * p.Hq + h) * kD + t;
  s_q[t] = __bfloat162float(p.q[qi]) * rq.k_global;
  __syncthreads();
  const long long head0 = static_cast<long long>(h / p.G) * rq.head_stride;
  float m = -INFINITY, l = 0.f, acc = 0.f;
  for (int c0 = 0; c0 < T + p.rows; c0 += kD) {
    const int slot = c0 + t;
    const int kr = slot - T;  // tree row
    bool see = slot < T;
    if (!see && kr < p.rows) see = rq.anc ? (rq.anc[i * p.W + (kr >> 6)] >> (kr & 63)) & 1 : kr == i;
    float s = -INFINITY;
    if (see && GLANCE_IN_BOUNDS(slot, rq.t_cap)) {
      const unsigned char* kc = rq.k + (head0 + slot) * 64;
      const unsigned char* ks = rq.k_scale + (head0 + slot) * 8;
      float dot = 0.f;
      for (int g = 0; g < 8; ++g) {
        const float sc = f16x2_to_f32(scales2_to_f16(ks[g])).x;
        float d = 0.f;
        for (int w = 0; w < 2; ++w) {
          uint32_t f[4];
          codes8_to_f16(reinterpret_cast<const uint32_t*>(kc)[2 * g + w], f);
          for (int e = 0; e < 4; ++e) {
            const float2 x = f16x2_to_f32(f[e]);
            d = fmaf(s_q[16 * g + 8 * w + 2 * e], x.x, d);
            d = fmaf(s_q[16 * g + 8 * w + 2 * e + 1], x.y, d);
          }
        }
        dot = fmaf(d, sc, dot);
      }
      s = dot * p.scale_log2;
    }
    float cm = s;
    for (int o = 16; o; o >>= 1) cm = fmaxf(cm, __shfl_xor_sync(0xffffffffu, cm, o));
    if ((t & 31) == 0) s_red[t >> 5] = cm;
    __syncthreads();
    cm = fmaxf(fmaxf(s_red[0], s_red[1]), fmaxf(s_red[2], s_red[3]));
    const float mn = fmaxf(m, cm);
    const float mu = mn == -INFINITY ? 0.f : mn;
    s_p[t] = see ? exp2f(s - mu) : 0.f;
    const float alpha = m == -INFINITY ? 0.f : exp2f(m - mu);
    m = mn;
    l *= alpha;
    acc *= alpha;
    __syncthreads();
    const int n = min(kD, T + p.rows - c0);
    for (int j = 0; j < n; ++j) {
      const float w = s_p[j];
      if (w == 0.f) continue;
      l += w;
      const long long at = head0 + c0 + j;
      const uint32_t b = rq.v[at * 64 + (t >> 1)] >> (4 * (t & 1)) & 15u;
      uint32_t f[4];
      codes8_to_f16(b, f);
      acc = fmaf(w, f16x2_to_f32(f[0]).x * f16x2_to_f32(scales2_to_f16(rq.v_scale[at * 8 + (t >> 4)])).x, acc);
    }
    __syncthreads();
  }
  p.out[qi] = __float2bfloat16(l == 0.f ? 0.f : acc * rq.v_global / l);
}

size_t workspace_bytes_of(int B, int rows, int Hq, const glance_kv4* kv) { return 256; }

}  // namespace

extern "C" size_t glance_kv4_tree_attention_workspace_bytes(int B, int n_rows, int n_q_heads, const glance_kv4* kv) {
  if (!kv || B < 1 || B > kMaxB || n_rows < 1 || n_rows > 256 || n_q_heads < 1) return 0;
  for (int r = 0; r < B; ++r)
    if (kv[r].n_kv_heads != kv[0].n_kv_heads || kv[r].n_kv_heads < 1 || n_q_heads % kv[r].n_kv_heads ||
        kv[r].t_cap < n_rows || kv[r].t_cap > glance::kKv4MaxCap)
      return 0;
  return workspace_bytes_of(B, n_rows, n_q_heads, kv);
}

extern "C" glance_status glance_kv4_tree_attention(const void* q, int n_q_heads, const glance_kv4* kv,
                                                   const glance_tree* trees, int B, float scale, void* out,
                                                   void* workspace, size_t workspace_bytes, void* stream) {
  using glance::fail;
  const char* who = "glance_kv4_tree_attention";
  if (!q || !kv || !trees || !out) return fail(GLANCE_ERR_INVALID_ARG, "%s: null pointer argument", who);
  if (B < 1 || B > kMaxB) return fail(GLANCE_ERR_INVALID_ARG, "%s: need 1 <= B <= %d", who, kMaxB);
  const int rows = trees[0].n + 1;
  Params p;
  for (int r = 0; r < B; ++r) {
    const glance_tree& t = trees[r];
    if (t.n < 0 || t.n > 255 || t.n + 1 != rows || t.mask_words != (rows + 63) / 64 || (!t.anc && t.n > 0))
      return fail(GLANCE_ERR_INVALID_ARG,
                  "%s: every tree needs the same N, 0 <= N <= 255, mask_words = ceil((N+1)/64) and, but for N = 0, anc "
                  "(request %d)", who, r);
    const glance_status st = glance::check_kv4(who, kv[r], rows, r);
    if (st != GLANCE_OK) return st;
    if (kv[r].n_kv_heads != kv[0].n_kv_heads)
      return fail(GLANCE_ERR_INVALID_ARG, "%s: every request needs the same n_kv_heads (request %d)", who, r);
    const glance_kv4& x = kv[r];
    p.req[r] = {static_cast<const unsigned char*>(x.k), static_cast<const unsigned char*>(x.k_scale),
                static_cast<const unsigned char*>(x.v), static_cast<const unsigned char*>(x.v_scale),
                t.anc, x.t_len, x.head_stride, x.k_global, x.v_global, x.t_cap};
  }
  const int Hkv = kv[0].n_kv_heads;
  if (n_q_heads < 1 || n_q_heads % Hkv)
    return fail(GLANCE_ERR_INVALID_ARG, "%s: n_q_heads must be a positive multiple of n_kv_heads", who);
  const int G = n_q_heads / Hkv;
  if (G != 1 && G != 2 && G != 4 && G != 8)
    return fail(GLANCE_ERR_UNSUPPORTED, "%s: need n_q_heads / n_kv_heads in {1, 2, 4, 8}", who);
  if (!(scale > 0.f) || !isfinite(scale)) return fail(GLANCE_ERR_INVALID_ARG, "%s: scale must be finite and > 0", who);
  if (!glance::aligned16(q) || !glance::aligned16(out))
    return fail(GLANCE_ERR_INVALID_ARG, "%s: q and out must be 16-byte aligned", who);
  const size_t n_out = static_cast<size_t>(B) * rows * n_q_heads * kD * 2;
  const char *q0 = static_cast<const char*>(q), *o0 = static_cast<const char*>(out);
  if (q0 < o0 + n_out && o0 < q0 + n_out) return fail(GLANCE_ERR_INVALID_ARG, "%s: out overlaps q", who);
  const size_t need = workspace_bytes_of(B, rows, n_q_heads, kv);
  if (!workspace || workspace_bytes < need)
    return fail(GLANCE_ERR_CAPACITY, "%s: workspace %zu bytes < %zu needed", who, workspace_bytes, need);
  if (reinterpret_cast<uintptr_t>(workspace) & 255)
    return fail(GLANCE_ERR_INVALID_ARG, "%s: workspace must be 256-byte aligned", who);
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.out = static_cast<__nv_bfloat16*>(out);
  p.rows = rows;
  p.Hq = n_q_heads;
  p.G = G;
  p.W = (rows + 63) / 64;
  p.scale_log2 = scale * kLog2e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(B * rows * n_q_heads);
  cfg.blockDim = dim3(kD);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kv4_attention_plain_kernel, p);
  if (e != cudaSuccess) return glance::cuda_fail(e, who);
  return GLANCE_OK;
}
