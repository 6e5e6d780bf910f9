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
  float4* part_o;   // unnormalised partial O of a block
  float2* part_ml;  // its rows' (maximum in log2, sum of weights)
  uint32_t* count;  // [B][Hkv] blocks of a head that are done
  int B, rows, Hq, Hkv, G, W;
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


// ------------------------------------------------- few query rows per kv head
//
// At most 16 query rows share a kv head (decoding, small trees): the call is
// bound by reading the cache, 144 bytes per slot and kv head, so everything
// else is kept off that path.
//
// * A warp takes 32 slots at a time and has three such pieces (4.6 KB each) in
//   flight: bulk copies into its own ring, no other warp to wait for. Codes and
//   scales of a head are contiguous, so a piece is four copies.
// * Both products are m16n8k16 with the query rows as M. The codes become f16
//   in registers, straight in fragment order, by choosing which element each
//   fragment position stands for: a sum over dims (or slots) may take them in
//   any order as long as both operands agree. For S a lane holds 32
//   consecutive dims of one slot (one 16-byte load); for O a lane holds the 16
//   dims of one scale group of four slots (four 8-byte loads), paired by slot.
// * Softmax weights never leave registers: S's accumulator layout is P's
//   operand layout.
// The warps of a block are merged through shared memory, the blocks of a head
// through the workspace by the block that finishes last.

constexpr int kFewWarps = 8;
constexpr int kFewThreads = kFewWarps * 32;
constexpr int kFewRows = 16;
constexpr int kUnit = 32;    // slots of one piece
constexpr int kFewStages = 3;
constexpr uint32_t kUnitCodes = kUnit * glance::kKv4CodeBytes;    // 2048
constexpr uint32_t kUnitScales = kUnit * glance::kKv4ScaleBytes;  // 256
constexpr uint32_t kUnitBytes = 2 * (kUnitCodes + kUnitScales);
constexpr uint32_t kFewRing = kFewWarps * kFewStages * kUnitBytes;  // 110,592
constexpr uint32_t kFewQ = 8 * 32 * 16;                             // Q in fragment order
constexpr uint32_t kFewMisc = 512;
constexpr uint32_t kFewSmem = kFewRing + kFewQ + kFewMisc;
constexpr uint32_t kWarpRing = kFewStages * kUnitBytes;
constexpr uint32_t kWarpO = kFewRows * kD * 4;  // a finished warp's O, then its rows' maxima and sums, in its own ring
static_assert(kWarpO + 2 * kFewRows * 4 <= kWarpRing, "a warp's result fits its ring");
static_assert(2 * (kFewSmem + 1024) <= 228 * 1024, "two blocks per SM");

struct FewMisc {
  uint64_t full[kFewWarps][kFewStages];
  float row_scale[kFewRows];           // score factor of a row, in log2
  int req, head, split, n_split, tau, first_block, last;
};
static_assert(sizeof(FewMisc) <= kFewMisc, "misc block");

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) { return __byte_perm(a, b, sel); }

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// The factor that brings a query row whose largest magnitude is `amax` to
// [2^14, 2^15), so that f16 holds every element down to 2^-31 of it exactly
// (a bf16 has 8 bits): a power of two, at most 2^100. Its inverse goes into
// the row's score factor; a row that is not finite gets NaN there.
__device__ __forceinline__ float query_factor(float amax) {
  int e = 141 - static_cast<int>(__float_as_uint(amax) >> 23);
  e = e > 100 ? 100 : e;
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}
__device__ __forceinline__ float score_factor(float amax, float factor, float scale_log2, float k_global) {
  // at least the least normal number: a score of -infinity stays one
  return amax < INFINITY ? fmaxf(scale_log2 * k_global * (1.f / factor), 1.17549435e-38f) : __uint_as_float(0x7FC00000u);
}

// Which part of which request's slots this block has: head `head` of request
// `req`, units [split * tau, (split + 1) * tau). tau is the smallest number of
// units per block (at least one per warp) at which every head's blocks fit the
// grid; it comes from the prefix lengths themselves, which only the device
// knows. Warp 0 computes it, lane r for request r.
__device__ __forceinline__ void few_plan(const Params& p, FewMisc* ms, int lane) {
  int units = 0;
  if (lane < p.B) {
    const int T = *p.req[lane].t_len;
    const bool room = T >= 0 && T <= p.req[lane].t_cap - p.rows;
    if (!room && blockIdx.x == 0) report(GLANCE_DEV_TREE_CAPACITY);
    units = room ? (T + p.rows + kUnit - 1) / kUnit : 0;
  }
  const int per_head = static_cast<int>(gridDim.x) / p.Hkv;  // blocks for one head of every request
  int lo = kFewWarps, hi = max(kFewWarps, __reduce_max_sync(0xffffffffu, units));
  while (lo < hi) {  // at hi every request has one block, and per_head >= B
    const int mid = (lo + hi) >> 1;
    if (static_cast<int>(__reduce_add_sync(0xffffffffu, (units + mid - 1) / mid)) <= per_head)
      hi = mid;
    else
      lo = mid + 1;
  }
  const int n = (units + lo - 1) / lo;
  int end = n * p.Hkv;  // inclusive scan of the requests' blocks
#pragma unroll
  for (int o = 1; o < kMaxB; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, end, o);
    if (lane >= o) end += v;
  }
  const int at = blockIdx.x;
  const unsigned past = __ballot_sync(0xffffffffu, lane < p.B && at >= end);
  const int r = __popc(past);
  const int start = __shfl_sync(0xffffffffu, end - n * p.Hkv, r & 31);
  const int nr = __shfl_sync(0xffffffffu, n, r & 31);
  if (lane == 0) {
    const bool any = r < p.B && nr > 0;
    ms->req = any ? r : -1;
    ms->head = any ? (at - start) / nr : 0;
    ms->split = any ? (at - start) % nr : 0;
    ms->n_split = nr;
    ms->tau = lo;
    ms->first_block = any ? at - (at - start) % nr : 0;
  }
}

__device__ __forceinline__ void few_copy(const Request& rq, long long head0, int unit, int n_keys, unsigned char* st,
                                         uint64_t* bar) {
  const int key0 = unit * kUnit;
  const int n = min(kUnit, (n_keys - key0 + 1) & ~1);  // an even number: 16 bytes of scales
  if (!GLANCE_IN_BOUNDS(key0 + n - 1, rq.head_stride)) {
    mbar_arrive(bar);
    return;
  }
  mbar_arrive_expect_tx(bar, n * 2 * (glance::kKv4CodeBytes + glance::kKv4ScaleBytes));
  const long long at = head0 + key0;
  bulk_copy_g2s(st, rq.k + at * 64, n * 64, bar);
  bulk_copy_g2s(st + kUnitCodes, rq.v + at * 64, n * 64, bar);
  bulk_copy_g2s(st + 2 * kUnitCodes, rq.k_scale + at * 8, n * 8, bar);
  bulk_copy_g2s(st + 2 * kUnitCodes + kUnitScales, rq.v_scale + at * 8, n * 8, bar);
}

__global__ void __launch_bounds__(kFewThreads, 2) kv4_attention_few_kernel(const __grid_constant__ Params p) {
  extern __shared__ __align__(128) unsigned char smem[];
  unsigned char* ring = smem;
  uint4* sq = reinterpret_cast<uint4*>(smem + kFewRing);
  FewMisc* ms = reinterpret_cast<FewMisc*>(smem + kFewRing + kFewQ);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) {
    for (int s = 0; s < kFewStages; ++s) mbar_init(&ms->full[warp][s], 1);
    fence_barrier_init();
  }
  pdl_wait_prior();
  pdl_launch_dependents();
  if (warp == 0) few_plan(p, ms, lane);
  __syncthreads();
  if (ms->req < 0) return;
  const Request& rq = p.req[ms->req];
  const int head = ms->head, n_split = ms->n_split;
  const int T = *rq.t_len, n_keys = T + p.rows;
  const int n_units = (n_keys + kUnit - 1) / kUnit;
  const int u0 = ms->split * ms->tau, u1 = min(u0 + ms->tau, n_units);
  const long long head0 = static_cast<long long>(head) * rq.head_stride;
  unsigned char* my_ring = ring + warp * kWarpRing;
  if (lane == 0)
    for (int s = 0; s < kFewStages; ++s)
      if (u0 + warp + s * kFewWarps < u1)
        few_copy(rq, head0, u0 + warp + s * kFewWarps, n_keys, my_ring + s * kUnitBytes, &ms->full[warp][s]);
  const int R = p.G * p.rows;
  const size_t q_base = static_cast<size_t>(ms->req) * p.rows * p.Hq + head * p.G;
  {
    // Q into fragment order: thread (row, e) has dims 8e .. 8e + 7
    const int row = threadIdx.x >> 4, e = threadIdx.x & 15;
    uint4 x = make_uint4(0, 0, 0, 0);
    if (row < R)
      x = *reinterpret_cast<const uint4*>(p.q + (q_base + static_cast<size_t>(row % p.rows) * p.Hq + row / p.rows) * kD + e * 8);
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    float f[8], amax = 0.f;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      amax = fmaxf(amax, fmaxf(fabsf(f[2 * i]), fabsf(f[2 * i + 1])));
      bad = bad || !(fabsf(f[2 * i]) < INFINITY) || !(fabsf(f[2 * i + 1]) < INFINITY);
    }
    if (bad) amax = INFINITY;
#pragma unroll
    for (int o = 8; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const float qf = query_factor(amax);
    if (e == 0) ms->row_scale[row] = score_factor(amax, qf, p.scale_log2, rq.k_global);
    uint32_t* s32 = reinterpret_cast<uint32_t*>(sq);
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // dims 8e + 2i, + 1: c = e / 4, step, half of the step
      const int step = (e & 3) * 2 + (i >> 1);
      s32[(step * 32 + (row & 7) * 4 + (e >> 2)) * 4 + (row >> 3) + 2 * (i & 1)] = pack_f16x2(f[2 * i] * qf, f[2 * i + 1] * qf);
    }
  }
  __syncthreads();
  const int r0 = lane >> 2, c = lane & 3;
  const float sc[2] = {ms->row_scale[r0], ms->row_scale[r0 + 8]};
  // visible tree rows (at most 16) of this lane's two query rows
  uint32_t seen[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int qr = r0 + 8 * h, i = qr % p.rows;
    seen[h] = qr >= R ? 0u : rq.anc ? static_cast<uint32_t>(rq.anc[i * p.W]) : 1u << i;
    if (p.rows < 32) seen[h] &= (1u << p.rows) - 1u;
  }
  float o[16][4];
#pragma unroll
  for (int t = 0; t < 16; ++t) o[t][0] = o[t][1] = o[t][2] = o[t][3] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  int stage = 0;
  uint32_t parity = 0;
  for (int u = u0 + warp; u < u1; u += kFewWarps) {
    unsigned char* st = my_ring + stage * kUnitBytes;
    if (!__all_sync(0xffffffffu, mbar_wait(&ms->full[warp][stage], parity))) {
      if (lane == 0) report(GLANCE_DEV_PIPELINE_TIMEOUT);
      for (int s = 1; s < kFewStages; ++s)  // the copies in flight land before the block leaves
        if (u + s * kFewWarps < u1)
          (void)mbar_wait(&ms->full[warp][(stage + s) % kFewStages], parity ^ (stage + s >= kFewStages), 50000000ull);
      break;
    }
    const int key0 = u * kUnit;
    float s[4][4];
#pragma unroll
    for (int b = 0; b < 4; ++b) s[b][0] = s[b][1] = s[b][2] = s[b][3] = 0.f;
    {
      // S: lane (n = r0, c) has slot 8b + 4 (n & 1) + (n >> 1), dims 32c ..
      const int slot = 4 * (r0 & 1) + (r0 >> 1);
      uint4 kw[4];
      uint32_t ks[4][2];
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        kw[b] = *reinterpret_cast<const uint4*>(st + (8 * b + slot) * 64 + c * 16);
        const uint32_t x = scales2_to_f16(*reinterpret_cast<const uint16_t*>(st + 2 * kUnitCodes + (8 * b + slot) * 8 + 2 * c));
        ks[b][0] = prmt(x, x, 0x1010);
        ks[b][1] = prmt(x, x, 0x3232);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint4 a = sq[(2 * j) * 32 + lane], a2 = sq[(2 * j + 1) * 32 + lane];
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          uint32_t h[4];
          codes8_to_f16(j == 0 ? kw[b].x : j == 1 ? kw[b].y : j == 2 ? kw[b].z : kw[b].w, h);
#pragma unroll
          for (int i = 0; i < 4; ++i) h[i] = mul_f16x2(h[i], ks[b][j >> 1]);
          mma16816(s[b], a.x, a.y, a.z, a.w, h[0], h[1]);
          mma16816(s[b], a2.x, a2.y, a2.z, a2.w, h[2], h[3]);
        }
      }
    }
    // slot of s[b][e]: 8b + 4 (e & 1) + c, row r0 + 8 (e >> 1)
    uint32_t zero_v = 0u;  // slots whose V must not be multiplied
    if (key0 + kUnit > T) {
      // tree slots: a row sees its ancestors. What the other rows hold must not
      // reach it even as 0 * NaN: a V row with a scale that is not a number is
      // left out of the product and makes the scores of the rows that see it NaN.
      const uint2 vs = *reinterpret_cast<const uint2*>(st + 2 * kUnitCodes + kUnitScales + lane * 8);
      const uint32_t nan_bytes = __vcmpeq4(vs.x & 0x7F7F7F7Fu, 0x7F7F7F7Fu) | __vcmpeq4(vs.y & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
      const int left = n_keys - key0;
      const uint32_t past = left >= 32 ? 0u : ~((1u << left) - 1u);
      const uint32_t bad = __ballot_sync(0xffffffffu, nan_bytes != 0u) & ~past;
      zero_v = bad | past;
      const int pre = T - key0;  // prefix slots of the piece
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t vis = pre >= 32 ? 0xFFFFFFFFu
                             : pre >= 0 ? ((1u << pre) - 1u) | (seen[h] << pre)
                                        : (-pre < 32 ? seen[h] >> -pre : 0u);
#pragma unroll
        for (int b = 0; b < 4; ++b)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int k = 8 * b + 4 * e + c;
            float& x = s[b][2 * h + e];
            x = !((vis & ~past) >> k & 1u) ? -INFINITY : (bad >> k & 1u) ? __uint_as_float(0x7FC00000u) : x;
          }
      }
    }
    uint32_t pa[2][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float mx = fmaxf(fmaxf(fmaxf(s[0][2 * h], s[0][2 * h + 1]), fmaxf(s[1][2 * h], s[1][2 * h + 1])),
                       fmaxf(fmaxf(s[2][2 * h], s[2][2 * h + 1]), fmaxf(s[3][2 * h], s[3][2 * h + 1])));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2)) * sc[h];  // sc > 0, or NaN (then mx is of no account)
      // the running maximum moves only when it has grown by 8 (in log2): until
      // then the weights stay below 2^8 and nothing is rescaled
      const bool grow = mx > m[h] + 8.f;
      if (__any_sync(0xffffffffu, grow)) {
        const float mn = grow ? mx : m[h];
        const float alpha = m[h] == -INFINITY ? 0.f : ex2_approx(m[h] - mn);
        m[h] = mn;
        l[h] *= alpha;
#pragma unroll
        for (int t = 0; t < 16; ++t) {
          o[t][2 * h] *= alpha;
          o[t][2 * h + 1] *= alpha;
        }
      }
      const float off = m[h] == -INFINITY ? 0.f : m[h];
      float w[4][2];
#pragma unroll
      for (int b = 0; b < 4; ++b)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          w[b][e] = ex2_approx(fmaf(s[b][2 * h + e], sc[h], -off));
          l[h] += w[b][e];
        }
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        pa[kb][h] = pack_f16x2(w[2 * kb][0], w[2 * kb][1]);
        pa[kb][2 + h] = pack_f16x2(w[2 * kb + 1][0], w[2 * kb + 1][1]);
      }
    }
    // O: lane (n = r0, c) has slots 16 kb + 4i + c, dims 16n .. 16n + 15; the
    // product's column n of tile t is dim 16n + t
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      uint2 vw[4];
      uint32_t sb[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int slot = 16 * kb + 4 * i + c;
        vw[i] = *reinterpret_cast<const uint2*>(st + kUnitCodes + slot * 64 + r0 * 8);
        sb[i] = st[2 * kUnitCodes + kUnitScales + slot * 8 + r0];
      }
      uint32_t vs[2] = {scales2_to_f16(sb[0] | sb[1] << 8), scales2_to_f16(sb[2] | sb[3] << 8)};
      if (zero_v) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (zero_v >> (16 * kb + 4 * i + c) & 1u) {
            vw[i] = make_uint2(0u, 0u);
            vs[i >> 1] &= (i & 1) ? 0x0000FFFFu : 0xFFFF0000u;
          }
      }
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        uint32_t h[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) codes8_to_f16(w ? vw[i].y : vw[i].x, h[i]);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            const uint32_t sel = z ? 0x7632 : 0x5410;
            mma16816(o[8 * w + 2 * i + z], pa[kb][0], pa[kb][1], pa[kb][2], pa[kb][3],
                     mul_f16x2(prmt(h[0][i], h[1][i], sel), vs[0]), mul_f16x2(prmt(h[2][i], h[3][i], sel), vs[1]));
          }
      }
    }
    __syncwarp();  // every lane has read the piece
    if (lane == 0 && u + kFewStages * kFewWarps < u1)
      few_copy(rq, head0, u + kFewStages * kFewWarps, n_keys, st, &ms->full[warp][stage]);
    if (++stage == kFewStages) {
      stage = 0;
      parity ^= 1;
    }
  }
  const auto warp_o = [&](int w) { return reinterpret_cast<float4*>(ring + w * kWarpRing); };
  const auto warp_m = [&](int w) { return reinterpret_cast<float*>(ring + w * kWarpRing + kWarpO); };
  // the block's rows: maxima first, then every warp's O relative to them
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
    if (l[h] != l[h]) m[h] = 0.f;  // a NaN row stays one in every merge
    if (c == 0) {
      warp_m(warp)[r0 + 8 * h] = m[h];
      warp_m(warp)[kFewRows + r0 + 8 * h] = l[h];
    }
  }
  __syncthreads();
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int row = r0 + 8 * h;
    if (row < R) {
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < kFewWarps; ++w) M = fmaxf(M, warp_m(w)[row]);
      const float f = m[h] == -INFINITY ? 0.f : ex2_approx(m[h] - M);
      float4* dst = warp_o(warp) + row * 32;  // 4-dim pieces rotated by the row, against bank conflicts
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int t = 0; t < 4; ++t)
          dst[(8 * c + 4 * e + t + row) & 31] = make_float4(o[4 * t][2 * h + e] * f, o[4 * t + 1][2 * h + e] * f,
                                                            o[4 * t + 2][2 * h + e] * f, o[4 * t + 3][2 * h + e] * f);
    }
  }
  __syncthreads();
  float4* out_part = p.part_o + static_cast<size_t>(blockIdx.x) * kFewRows * 32;
  for (int i = threadIdx.x; i < R * 32; i += kFewThreads) {
    const int row = i >> 5, x = i & 31;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    float M = -INFINITY, L = 0.f;
#pragma unroll
    for (int w = 0; w < kFewWarps; ++w) M = fmaxf(M, warp_m(w)[row]);
#pragma unroll
    for (int w = 0; w < kFewWarps; ++w) {
      const float mw = warp_m(w)[row];
      L += mw == -INFINITY ? 0.f : ex2_approx(mw - M) * warp_m(w)[kFewRows + row];
      const float4 v = warp_o(w)[row * 32 + ((x + row) & 31)];
      a.x += v.x;
      a.y += v.y;
      a.z += v.z;
      a.w += v.w;
    }
    if (n_split == 1) {
      const float inv = L == 0.f ? 0.f : rq.v_global / L;
      const size_t at = (q_base + static_cast<size_t>(row % p.rows) * p.Hq + row / p.rows) * kD + x * 4;
      *reinterpret_cast<uint2*>(p.out + at) = make_uint2(pack_bf16x2(a.x * inv, a.y * inv), pack_bf16x2(a.z * inv, a.w * inv));
    } else {
      out_part[i] = a;
      if (x == 0) p.part_ml[blockIdx.x * kFewRows + row] = make_float2(M, L);
    }
  }
  if (n_split == 1) return;
  // the last block of the head merges: its add acquires the others' partials
  __syncthreads();
  if (threadIdx.x == 0) {
    uint32_t* count = p.count + ms->req * p.Hkv + head;
    const bool last = atom_add_acq_rel_gpu(count, 1u) == static_cast<uint32_t>(n_split - 1);
    if (last) *count = 0u;
    ms->last = last;
  }
  __syncthreads();
  if (!ms->last) return;
  const int b0 = ms->first_block;
  for (int i = threadIdx.x; i < R * 32; i += kFewThreads) {
    const int row = i >> 5, x = i & 31;
    float M = -INFINITY, L = 0.f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s0 = 0; s0 < n_split; s0 += 8) {
      float4 v[8];
      float2 ml[8];
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        const bool in = s0 + s < n_split;
        ml[s] = in ? __ldcg(p.part_ml + (b0 + s0 + s) * kFewRows + row) : make_float2(-INFINITY, 0.f);
        v[s] = in ? __ldcg(p.part_o + (static_cast<size_t>(b0 + s0 + s) * kFewRows + row) * 32 + x) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      float mx = M;
#pragma unroll
      for (int s = 0; s < 8; ++s) mx = fmaxf(mx, ml[s].x);
      const float keep = M == -INFINITY ? 0.f : ex2_approx(M - mx);
      M = mx;
      L *= keep;
      a.x *= keep;
      a.y *= keep;
      a.z *= keep;
      a.w *= keep;
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        const float f = ml[s].x == -INFINITY ? 0.f : ex2_approx(ml[s].x - mx);
        L = fmaf(f, ml[s].y, L);
        a.x = fmaf(f, v[s].x, a.x);
        a.y = fmaf(f, v[s].y, a.y);
        a.z = fmaf(f, v[s].z, a.z);
        a.w = fmaf(f, v[s].w, a.w);
      }
    }
    const float inv = L == 0.f ? 0.f : rq.v_global / L;
    const size_t at = (q_base + static_cast<size_t>(row % p.rows) * p.Hq + row / p.rows) * kD + x * 4;
    *reinterpret_cast<uint2*>(p.out + at) = make_uint2(pack_bf16x2(a.x * inv, a.y * inv), pack_bf16x2(a.z * inv, a.w * inv));
  }
}

// Blocks of the few-rows kernel: two per SM, or one per kv head of every
// request where that is more.
int few_grid(int B, int Hkv) {
  const int n = 2 * glance::num_sms();
  return n < B * Hkv ? B * Hkv : n / Hkv * Hkv;
}
size_t few_counter_bytes(int B, int Hkv) { return (static_cast<size_t>(B) * Hkv * 4 + 255) / 256 * 256; }

bool few_rows(int rows, int G) { return rows * G <= kFewRows; }

size_t workspace_bytes_of(int B, int rows, int Hq, const glance_kv4* kv) {
  const int Hkv = kv[0].n_kv_heads;
  if (few_rows(rows, Hq / Hkv))
    return few_counter_bytes(B, Hkv) + static_cast<size_t>(few_grid(B, Hkv)) * kFewRows * (kD * 4 + sizeof(float2));
  return 256;
}

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
  p.B = B;
  p.rows = rows;
  p.Hq = n_q_heads;
  p.Hkv = Hkv;
  p.G = G;
  p.W = (rows + 63) / 64;
  p.scale_log2 = scale * kLog2e;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e;
  if (few_rows(rows, G)) {
    const int grid = few_grid(B, Hkv);
    char* ws = static_cast<char*>(workspace);
    p.count = reinterpret_cast<uint32_t*>(ws);
    p.part_o = reinterpret_cast<float4*>(ws + few_counter_bytes(B, Hkv));
    p.part_ml = reinterpret_cast<float2*>(p.part_o + static_cast<size_t>(grid) * kFewRows * 32);
    e = glance::ensure_smem(reinterpret_cast<const void*>(kv4_attention_few_kernel), kFewSmem);
    if (e != cudaSuccess) return glance::cuda_fail(e, who);
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kFewThreads);
    cfg.dynamicSmemBytes = kFewSmem;
    e = cudaLaunchKernelEx(&cfg, kv4_attention_few_kernel, p);
  } else {
    cfg.gridDim = dim3(B * rows * n_q_heads);
    cfg.blockDim = dim3(kD);
    e = cudaLaunchKernelEx(&cfg, kv4_attention_plain_kernel, p);
  }
  if (e != cudaSuccess) return glance::cuda_fail(e, who);
  return GLANCE_OK;
}
