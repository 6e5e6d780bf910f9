// Ancestor-masked tree attention over 4-bit K/V caches (one layer, B requests).
//
// arXiv 2609.00355, Definition 1: packed row i sees the prefix slots 0..T-1
// and the tree slots of its own ancestors; N = 0 is one row, plain decoding.
//
//   o = sum_s w_s v_s / sum_s w_s,  w_s = 2^(q . k_s * scale * log2 e - m),
// over the visible slots s in one pass: m + 7 is a running maximum that may lag
// the true one by 8, and what was summed before is rescaled when it moves. k_s
// and v_s are code * scale; the globals go into the score factor and the output.
// Sums, maxima and O are fp32; the weights enter the second product as f16,
// because V's 6 significant bits are exact in f16 and a product takes one 16-bit
// type. Half a step is 2^-11 of a weight, an eighth of the output's own rounding
// to bf16, down to 2^-21 of the largest weight, and 2^-32 of the largest weight
// below: the 7 puts the largest at 2^7 to 2^15, the top of f16's range, so that
// the small ones of a long prefix beside a few large ones are not lost (with the
// largest at 1 to 2^8, 20000 weights of 2^-25.5 came out as nothing). It cancels
// between O and the sum and costs no instruction.
//
// Two kernels, by the query rows that share a kv head (G heads x N + 1 rows):
// up to 16, the call is bound by the cache's bytes (kv4_attention_few_kernel);
// beyond, by the products (kv4_attention_wide_kernel, with the tensor core's
// 128-row tiles). At 16 rows, 32 / 8 heads, the first and the second take 56.7
// and 111 us on 131072 slots, 27.6 and 35.9 on 32768, 21.5 and 31.4 for 8
// requests of 512 to 8192, but 14.9 and 13.0 on 4096; the host that picks the
// kernel does not know T.
#include <type_traits>

#include "kv4_internal.cuh"

GLANCE_DEFINE_STATUS_WORD(status_kv4_attention)

using namespace glance_dev;

namespace {

constexpr int kD = glance::kKv4D;
constexpr int kMaxB = 16;
constexpr float kLog2e = 1.4426950408889634f;
// The m of a row is kept this much (log2) under its running maximum, and moves
// when the maximum has grown by 8: weights are at most 2^15.
constexpr float kUnder = 7.f, kGrow = kUnder + 8.f;
// A weight's exponent is one fused multiply-add, score * factor - m, and m comes
// from rounded products: apart by up to half a step of a product, and a weight
// could be 2^(that) larger. Where m is set below kFused the products that count
// are below 2^24, the half step is 1/2 at most, and 2^15.5 is still an f16. From
// kFused on the product is rounded first, in loops of their own (with the choice
// inside, the usual ones take 2 to 4 % longer).
constexpr float kFused = 0x1p23f;

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
  float4* part_o;   // unnormalised partial O of a block (few rows)
  float2* part_ml;  // a part's rows' (maximum in log2, sum of weights)
  uint32_t* count;  // [B][Hkv] blocks of a head that are done; zero between calls
  int B, rows, Hq, Hkv, G, W;
  int n_qt, n_qp;   // query tiles of 128 rows per kv head, and pairs of them
  uint4* part;      // parts of 128 rows: O / l as f16, [16 octets][128 rows]
  int2* group;      // [B][Hkv][n_qp] the first part's block segment and the number of parts
  float scale_log2;
};

// --------------------------------------------------------- work for a block
//
// The slots of every group (request, kv head, query tile pair) are counted in
// units of 32. Where each group can be cut into equal parts that fill the grid,
// a block has one part; else the list of all groups is cut into equal runs and
// a block's run may cross groups (a "segment" is its part in one group). In that
// list a group counts kLead units more than it has, what starting and ending a
// segment takes. The lengths are read on the device: only it knows them.

constexpr int kUnit = 32;

struct Plan {
  int T[kMaxB];
  int units[kMaxB];       // of one group of request r; 0: no room, no output
  long long base[kMaxB];  // length of the list before request r's groups
  long long total;        // of the whole list
  int runs;               // blocks that the list is cut for: none gets less than a tile and its lead
  int tau;                // > 0: every group is cut into parts of tau units
  int blocks0[kMaxB];     // tau > 0: blocks before request r's
};

// A block's part in one group: units [a, a + n) of group g of request r.
struct Segment {
  int r, g, a, n;
  int left;   // length of the run after this segment
  int index;  // of the block's segments
};

// a / b for a run's arithmetic: 64-bit division only where it is needed.
__device__ __forceinline__ long long div_small(long long a, int b) {
  return a <= 0xFFFFFFFFll ? static_cast<long long>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b)) : a / b;
}

// The plan, by one warp; every block comes to the same one.
template <int kMinUnits, int kLead>
__device__ __forceinline__ void make_plan(const Params& p, Plan* pl, int lane, int blocks) {
  int units = 0, T = 0;
  if (lane < p.B) {
    T = *p.req[lane].t_len;
    if (T >= 0 && T <= p.req[lane].t_cap - p.rows) units = (T + p.rows + kUnit - 1) / kUnit;
  }
  const int gpr = p.Hkv * p.n_qp;
  const int sum = __reduce_add_sync(0xffffffffu, units);
  const int length = units > 0 ? units + kLead : 0;
  const long long total = static_cast<long long>(__reduce_add_sync(0xffffffffu, length)) * gpr;
  const int active = __popc(__ballot_sync(0xffffffffu, units > 0));
  const int per_group = blocks / gpr;
  const int runs = static_cast<int>(min(static_cast<long long>(blocks), max(1ll, div_small(total, kMinUnits + kLead))));
  int tau = 0;
  if (per_group >= active && active > 0) {
    // the least tau at which the groups' parts fit the grid, if that is no more
    // than a run of the list: not under the mean, and of use up to `limit` only
    const int limit = static_cast<int>(min(div_small(total, runs), 1ll << 30));
    int lo = max(kMinUnits, (sum + per_group - 1) / per_group), hi = limit + 1, mid = lo;
    while (lo < hi) {
      if (static_cast<int>(__reduce_add_sync(0xffffffffu, (units + mid - 1) / mid)) <= per_group)
        hi = mid;
      else
        lo = mid + 1;
      mid = (lo + hi) >> 1;
    }
    if (lo <= limit) tau = lo;
  }
  const int n = tau ? (units + tau - 1) / tau * gpr : 0;
  int before = length, nb = n;  // inclusive scans over the requests
#pragma unroll 1
  for (int o = 1; o < kMaxB; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, before, o), v = __shfl_up_sync(0xffffffffu, nb, o);
    if (lane >= o) {
      before += u;
      nb += v;
    }
  }
  if (lane < kMaxB) {
    pl->T[lane] = T;
    pl->units[lane] = units;
    pl->base[lane] = static_cast<long long>(before - length) * gpr;
    pl->blocks0[lane] = nb - n;
  }
  if (lane == 0) {
    pl->total = total;
    pl->runs = runs;
    pl->tau = tau;
  }
}

// First unit of block b's run (runs that may cross groups).
__device__ __forceinline__ long long run_start(long long total, int b, int blocks) {
  const long long q = div_small(total, blocks);
  return q * b + div_small((total - q * blocks) * b, blocks);
}

__device__ __forceinline__ void step_group(const Params& p, const Plan& pl, Segment& s) {
  if (++s.g == p.Hkv * p.n_qp) {
    s.g = 0;
    do ++s.r;
    while (pl.units[s.r] == 0);
  }
}
// The run's part from place `at` of the current group's stretch on, or of the
// next group that it has units of.
template <int kLead>
__device__ __forceinline__ bool take_segment(const Params& p, const Plan& pl, Segment& s, int at) {
  for (;;) {
    const int take = min(s.left, pl.units[s.r] + kLead - at), end = at + take - kLead;
    s.left -= take;
    s.a = max(at - kLead, 0);
    s.n = end - s.a;
    if (s.n > 0) {
      ++s.index;
      return true;
    }
    if (s.left == 0) return false;
    step_group(p, pl, s);
    at = 0;
  }
}
// Block b's first segment, by one warp (lane = request, or end of the run).
template <int kLead>
__device__ __forceinline__ bool first_segment(const Params& p, const Plan& pl, int b, int lane, Segment& s) {
  const int gpr = p.Hkv * p.n_qp, r = min(lane, kMaxB - 1);
  s.index = 0;
  if (pl.tau) {
    int n = (pl.units[r] + pl.tau - 1) / pl.tau, at = b - pl.blocks0[r];
    const unsigned mine = __ballot_sync(0xffffffffu, lane < p.B && at >= 0 && at < n * gpr);
    if (!mine) return false;
    s.r = __ffs(mine) - 1;
    n = __shfl_sync(0xffffffffu, n, s.r);
    at = __shfl_sync(0xffffffffu, at, s.r);
    s.g = at / n;
    s.a = at % n * pl.tau;
    s.n = min(pl.tau, pl.units[s.r] - s.a);
    s.left = 0;
    return true;
  }
  if (b >= pl.runs || pl.total == 0) return false;
  const long long end = run_start(pl.total, b + (lane & 1), pl.runs), x = __shfl_sync(0xffffffffu, end, 0);
  // requests without units share their base with the next
  s.r = 31 - __clz(__ballot_sync(0xffffffffu, lane < p.B && x >= pl.base[r]));
  const long long in = x - pl.base[s.r];
  const int length = pl.units[s.r] + kLead;
  s.g = static_cast<int>(div_small(in, length));
  s.index = -1;
  s.left = static_cast<int>(__shfl_sync(0xffffffffu, end, 1) - x);
  return take_segment<kLead>(p, pl, s, static_cast<int>(in - static_cast<long long>(s.g) * length));
}
template <int kLead>
__device__ __forceinline__ bool next_segment(const Params& p, const Plan& pl, Segment& s) {
  if (s.left == 0) return false;
  step_group(p, pl, s);
  return take_segment<kLead>(p, pl, s, 0);
}

// ------------------------------------------------- few query rows per kv head
//
// At most 16 query rows share a kv head (decoding, small trees): the call is
// bound by reading the cache, 144 bytes per slot and kv head, so everything
// else is kept off that path.
//
// * A warp takes 32 slots at a time and has two such pieces (4.6 KB each) in
//   flight: bulk copies into its own ring, no other warp to wait for. Codes and
//   scales of a head are contiguous, so a piece is four copies.
// * Both products are m16n8k16 with the query rows as N, eight or sixteen of
//   them: S^T = K Q^T and O^T = V^T P^T. The codes become f16 in registers,
//   straight in fragment order, by choosing which element each fragment position
//   stands for: a sum over dims (or slots) may take them in any order as long as
//   both operands agree. For S a lane holds 32 consecutive dims of a slot (one
//   16-byte load) and of a query row; for O the 16 dims of one scale group of
//   four slots (four 8-byte loads), paired by slot.
// * Softmax weights never leave registers: an 8 x 8 transpose turns S^T's
//   accumulator layout into P^T's operand layout.
// The warps of a block are merged through shared memory, the blocks of a head
// through the workspace by the block that finishes last.
//
// Measured (32 / 8 heads): one row on 131072 slots 36.7 us (61 % of the copy
// rate), one row x 16 requests of 512 to 32768 slots 40.4 us (57 %). There nothing
// is full (issue slots 52 %, ALU 49 %, memory 45 %): it is latency, a piece being
// one dependent chain of 660 instructions per warp (conversion, S, softmax,
// conversion, O) with four warps per scheduler, which wait for one another's
// blocks at the ends of the runs too. Three blocks per SM (85 registers a thread)
// spill and are slower. Sixteen rows on 131072 slots take 56.7 us (issue slots
// 53 %, memory 34 %): their O and weights do not fit 128 registers a thread, which
// spills (280 bytes of stores and of loads in the code of both loops), and every piece reads Q from shared
// memory. One row on 1000 slots takes 8.4 us: 1.2 until the block knows its work, 1.3 until
// q and the first piece are there, 1.2 for that piece, 0.9 to join the block's
// warps, 1.1 for the ticket and 1.5 to join the parts; much of each step is its
// instructions' first way to the SM.

constexpr int kFewWarps = 8;
constexpr int kFewThreads = kFewWarps * 32;
constexpr int kFewRows = 16;
constexpr int kFewStages = 2;
constexpr uint32_t kUnitCodes = kUnit * glance::kKv4CodeBytes;    // 2048
constexpr uint32_t kUnitScales = kUnit * glance::kKv4ScaleBytes;  // 256
constexpr uint32_t kUnitBytes = 2 * (kUnitCodes + kUnitScales);
constexpr uint32_t kFewRing = kFewWarps * kFewStages * kUnitBytes;  // 73,728
constexpr uint32_t kFewMisc = 1024;
constexpr uint32_t kFewQ = 2 * 4 * 32 * 16;  // sixteen rows' Q fragments
constexpr uint32_t kFewSmem = kFewRing + kFewMisc + kFewQ;
constexpr uint32_t kWarpRing = kFewStages * kUnitBytes;
constexpr uint32_t kWarpO = kFewRows * kD * 4;  // a finished warp's O, then its rows' maxima and sums, in its own ring
static_assert(kWarpO + 2 * kFewRows * 4 <= kWarpRing, "a warp's result fits its ring");
static_assert(2 * (kFewSmem + 1024) <= 228 * 1024, "two blocks per SM");

// A part has a piece for every warp or more. (One part of 32 pieces instead of
// four of 8 takes 11.5 instead of 8.7 us for one row on 1000 slots: a piece takes
// a warp 1.3 us, the merge of the parts 2.) Starting and ending a group costs the
// block about two pieces per warp (8, 12, 16, 20 units measured: 34.3, 30.0, 29.2,
// 28.9 us for 4 rows x 16 requests of 100 to 10000 slots, 41.4, 40.8, 40.5, 40.5
// us for one row x 16 of 512 to 32768).
constexpr int kFewMin = kFewWarps, kFewLead = 16;

struct FewMisc {
  uint64_t full[kFewWarps][kFewStages];
  Segment seg;
  Plan plan;
  float factor[kFewRows];  // of the query rows' scores
  int any;
  int first_part, n_parts;  // of the segment's group: 2 * block + (the block's first or last segment)
  int last;
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
// the row's score factor. A row that is not finite gets NaN, which makes all of
// its scores NaN, and with them every output that sees a slot; the scores of
// slots that it does not see are masked as any row's.
__device__ __forceinline__ float query_factor(float amax) {
  int e = 141 - static_cast<int>(__float_as_uint(amax) >> 23);
  e = e > 100 ? 100 : e;
  return amax < INFINITY ? __uint_as_float(static_cast<uint32_t>(e + 127) << 23) : __uint_as_float(0x7FC00000u);
}
__device__ __forceinline__ float score_factor(float factor, float scale_log2, float k_global) {
  // at least the least normal number, for a factor of NaN as well: a score of -infinity stays one
  return fmaxf(scale_log2 * k_global * (1.f / factor), 1.17549435e-38f);
}

// Which parts the group of a segment (not a whole group) has: their number and
// the first one's place; by one warp.
__device__ __forceinline__ void few_parts(const Plan& pl, const Segment& s, int lane, int& first_part, int& n) {
  const int b = blockIdx.x;
  if (pl.tau) {
    n = (pl.units[s.r] + pl.tau - 1) / pl.tau;
    first_part = 2 * (b - s.a / pl.tau);
    return;
  }
  const int stretch = pl.units[s.r] + kFewLead;
  const long long start = pl.base[s.r] + static_cast<long long>(s.g) * stretch;
  int first = b;
  bool late = s.index > 0;
  if (s.a) {  // back to the block that has the group's first unit
    for (;;) {
      const unsigned before = __ballot_sync(0xffffffffu, run_start(pl.total, max(first - 1 - lane, 0), pl.runs) <= start + kFewLead);
      first = max(first - (before ? __ffs(before) : 32), 0);
      if (before || first == 0) break;
    }
    late = run_start(pl.total, first, pl.runs) < start;
  }
  for (n = b + 1 - first;; n += 32) {  // on to the block whose run ends behind the group
    const unsigned past = __ballot_sync(0xffffffffu, run_start(pl.total, min(first + n + lane, pl.runs), pl.runs) >= start + stretch);
    if (past) {
      n += __ffs(past) - 1;
      break;
    }
  }
  first_part = 2 * first + (late ? 1 : 0);
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

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(x));
  return d;
}

// kN: groups of eight query rows.
template <int kN>
__global__ void __launch_bounds__(kFewThreads, 2) kv4_attention_few_kernel(const __grid_constant__ Params p) {
  extern __shared__ __align__(128) unsigned char smem[];
  unsigned char* ring = smem;
  FewMisc* ms = reinterpret_cast<FewMisc*>(smem + kFewRing);
  uint4* sq = reinterpret_cast<uint4*>(smem + kFewRing + kFewMisc);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) {
    for (int s = 0; s < kFewStages; ++s) mbar_init(&ms->full[warp][s], 1);
    fence_barrier_init();
  }
  pdl_wait_prior();
  pdl_launch_dependents();
  if (warp == 0) {
    make_plan<kFewMin, kFewLead>(p, &ms->plan, lane, gridDim.x);
    __syncwarp();
    Segment s;
    const bool any = first_segment<kFewLead>(p, ms->plan, blockIdx.x, lane, s);
    if (lane == 0) {
      ms->any = any;
      ms->seg = s;
    }
  }
  __syncthreads();
  const Plan& pl = ms->plan;
  if (blockIdx.x == 0 && threadIdx.x < p.B && pl.units[threadIdx.x] == 0) report(GLANCE_DEV_TREE_CAPACITY);
  if (!ms->any) return;
  Segment sg = ms->seg;
  unsigned char* my_ring = ring + warp * kWarpRing;
  int stage = 0;
  uint32_t parity = 0;
  bool dead = false;  // a wait of this warp ran out: its barriers' phases are unknown, and it copies no more
  do {
  const Request& rq = p.req[sg.r];
  const int head = sg.g, T = pl.T[sg.r], n_keys = T + p.rows;
  const int u0 = sg.a, u1 = sg.a + sg.n;
  const bool whole = sg.n == pl.units[sg.r];
  const long long head0 = static_cast<long long>(head) * rq.head_stride;
  const int R = p.G * p.rows;
  const size_t q_base = static_cast<size_t>(sg.r) * p.rows * p.Hq + head * p.G;
  // Fragments: lane = 4 r + c. K: slots r (and r + 8) of sixteen, in the order
  // below, dims 32c ..; Q: row r, dims 32c ..; a lane's scores and O are of
  // query rows 2c and 2c + 1 (of each eight).
  const int r = lane >> 2, c = lane & 3;
  uint32_t seen[kN][2];  // visible tree rows (at most 16)
#pragma unroll
  for (int n = 0; n < kN; ++n)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int qr = 8 * n + 2 * c + h, i = qr % p.rows;
      seen[n][h] = qr >= R ? 0u : rq.anc ? static_cast<uint32_t>(__ldg(reinterpret_cast<const unsigned long long*>(rq.anc) + i * p.W)) : 1u << i;
    }
  // a warp has kN of the query rows, a lane 8 dims of one of them
  const int q_row = kN * warp + (lane >> 4), piece = lane & 15;
  const bool has_q = kN == 2 || lane < 16;
  uint4 v = make_uint4(0, 0, 0, 0);
  if (has_q && q_row < R)
    v = __ldg(reinterpret_cast<const uint4*>(p.q + (q_base + static_cast<size_t>(q_row % p.rows) * p.Hq + q_row / p.rows) * kD) + piece);
  // the first copies go out behind these loads and before their use
  if (lane == 0 && !dead)
    for (int s = 0; s < kFewStages; ++s)
      if (u0 + warp + s * kFewWarps < u1)
        few_copy(rq, head0, u0 + warp + s * kFewWarps, n_keys, my_ring + (stage + s) % kFewStages * kUnitBytes,
                 &ms->full[warp][(stage + s) % kFewStages]);
  {
    // the largest magnitude's bits: in the order of the absolute values
    uint32_t top = max(max(v.x & 0x7FFFu, v.y & 0x7FFFu), max(v.z & 0x7FFFu, v.w & 0x7FFFu));
    top = max(top, max(max(v.x & 0x7FFF0000u, v.y & 0x7FFF0000u), max(v.z & 0x7FFF0000u, v.w & 0x7FFF0000u)) >> 16);
#pragma unroll
    for (int x = 1; x < 16; x <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, x));
    const float amax = top >= 0x7F80u ? INFINITY : __uint_as_float(top << 16);
    const float qf = query_factor(amax);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = pack_f16x2(__uint_as_float(w[i] << 16) * qf, __uint_as_float(w[i] & 0xFFFF0000u) * qf);
    if (has_q) {
      sq[(4 * (q_row >> 3) + (piece & 3)) * 32 + 4 * (q_row & 7) + (piece >> 2)] = make_uint4(h[0], h[1], h[2], h[3]);
      if (piece == 0) ms->factor[q_row] = score_factor(qf, p.scale_log2, rq.k_global);
    }
  }
  __syncthreads();
  uint32_t q[16];  // of eight rows; of sixteen in shared memory, for want of registers
  float sc[kN][2];
#pragma unroll
  for (int n = 0; n < kN; ++n)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      sc[n][h] = ms->factor[8 * n + 2 * c + h];
      seen[n][h] &= (1u << p.rows) - 1u;  // rows <= 16
    }
  if (kN == 1) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint4 f = sq[e * 32 + lane];
      q[4 * e] = f.x;
      q[4 * e + 1] = f.y;
      q[4 * e + 2] = f.z;
      q[4 * e + 3] = f.w;
    }
  }
  float o[8][kN][4];
#pragma unroll
  for (int t = 0; t < 8; ++t)
#pragma unroll
    for (int n = 0; n < kN; ++n) o[t][n][0] = o[t][n][1] = o[t][n][2] = o[t][n][3] = 0.f;
  float m[kN][2], l[kN][2];
#pragma unroll
  for (int n = 0; n < kN; ++n) {
    m[n][0] = m[n][1] = -INFINITY;
    l[n][0] = l[n][1] = 0.f;
  }
  // position j of sixteen slots is slot 4 (j & 1) + (j >> 1 & 3) + (j & 8): the
  // four slots of a lane's V fragment are then 4 apart and the four lanes' next
  // to each other, which loads without bank conflicts
  const int k_slot = 4 * (r & 1) + (r >> 1);
  const auto take_pieces = [&](auto rounded) {
  constexpr bool kRounded = decltype(rounded)::value;
  for (int u = u0 + warp; u < u1 && !dead; u += kFewWarps) {
    unsigned char* st = my_ring + stage * kUnitBytes;
    if (!__all_sync(0xffffffffu, mbar_wait(&ms->full[warp][stage], parity))) {
      if (lane == 0) report(GLANCE_DEV_PIPELINE_TIMEOUT);
      for (int s = 1; s < kFewStages; ++s)  // the copies in flight land before the block leaves
        if (u + s * kFewWarps < u1)
          (void)mbar_wait(&ms->full[warp][(stage + s) % kFewStages], parity ^ (stage + s >= kFewStages), 50000000ull);
      dead = true;
      break;
    }
    const int key0 = u * kUnit;
    float s[2][kN][4];
    {
      uint4 kw[2][2];
      uint32_t ks[2][2];
#pragma unroll
      for (int kt = 0; kt < 2; ++kt) {
#pragma unroll
        for (int n = 0; n < kN; ++n) s[kt][n][0] = s[kt][n][1] = s[kt][n][2] = s[kt][n][3] = 0.f;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const int slot = 16 * kt + 8 * b + k_slot;
          kw[kt][b] = *reinterpret_cast<const uint4*>(st + slot * 64 + c * 16);
          ks[kt][b] = scales2_to_f16(*reinterpret_cast<const uint16_t*>(st + 2 * kUnitCodes + slot * 8 + 2 * c));
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int kt = 0; kt < 2; ++kt) {  // two chains of products side by side
          uint32_t h[2][4];
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            codes8_to_f16(j == 0 ? kw[kt][b].x : j == 1 ? kw[kt][b].y : j == 2 ? kw[kt][b].z : kw[kt][b].w, h[b]);
            const uint32_t f = prmt(ks[kt][b], ks[kt][b], j < 2 ? 0x1010 : 0x3232);
#pragma unroll
            for (int i = 0; i < 4; ++i) h[b][i] = mul_f16x2(h[b][i], f);
          }
#pragma unroll
          for (int n = 0; n < kN; ++n) {
            const uint4 qf = kN > 1 ? sq[(4 * n + j) * 32 + lane] : make_uint4(q[4 * j], q[4 * j + 1], q[4 * j + 2], q[4 * j + 3]);
            mma16816(s[kt][n], h[0][0], h[1][0], h[0][1], h[1][1], qf.x, qf.y);
            mma16816(s[kt][n], h[0][2], h[1][2], h[0][3], h[1][3], qf.z, qf.w);
          }
        }
    }
    // s[kt][n][e]: slot 16 kt + 8 (e >> 1) + k_slot, query row 8n + 2c + (e & 1)
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
      for (int n = 0; n < kN; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t vis = ~past & (pre >= 32 ? 0xFFFFFFFFu
                                        : pre >= 0 ? ((1u << pre) - 1u) | (seen[n][h] << pre)
                                                   : (-pre < 32 ? seen[n][h] >> -pre : 0u));
#pragma unroll
          for (int kt = 0; kt < 2; ++kt)
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              const int k = 16 * kt + 8 * b + k_slot;
              float& x = s[kt][n][2 * b + h];
              x = !(vis >> k & 1u) ? -INFINITY : (bad >> k & 1u) ? __uint_as_float(0x7FC00000u) : x;
            }
        }
    }
    uint32_t pb[2][kN][2];
#pragma unroll
    for (int n = 0; n < kN; ++n) {
      float w[2][2][2];  // [query row][kt][half]
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float mx = fmaxf(fmaxf(s[0][n][h], s[0][n][2 + h]), fmaxf(s[1][n][h], s[1][n][2 + h]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
        mx = __fmul_rn(mx, sc[n][h]);  // sc > 0; not fused with what follows: the rounded products' own maximum
        // m moves only when the maximum has grown by 8 (in log2): until then the
        // weights stay below 2^15 and nothing is rescaled
        const bool grow = mx > __fadd_rd(m[n][h], kGrow);
        if (__any_sync(0xffffffffu, grow)) {
          const float mn = grow ? mx - kUnder : m[n][h];
          const float alpha = m[n][h] == -INFINITY ? 0.f : ex2_approx(m[n][h] - mn);
          m[n][h] = mn;
          l[n][h] *= alpha;
#pragma unroll
          for (int t = 0; t < 8; ++t) {
            o[t][n][h] *= alpha;
            o[t][n][2 + h] *= alpha;
          }
        }
        const float off = m[n][h] == -INFINITY ? 0.f : m[n][h];
#pragma unroll
        for (int kt = 0; kt < 2; ++kt)
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            const float x = s[kt][n][2 * b + h];
            w[h][kt][b] = ex2_approx(kRounded ? __fadd_rn(__fmul_rn(x, sc[n][h]), -off) : fmaf(x, sc[n][h], -off));
            l[n][h] += w[h][kt][b];
          }
      }
#pragma unroll
      for (int kt = 0; kt < 2; ++kt)
#pragma unroll
        for (int b = 0; b < 2; ++b) pb[kt][n][b] = transpose8x8(pack_f16x2(w[0][kt][b], w[1][kt][b]));
    }
    // O^T: lane (r, c) has slots 16 kt + 4i + c, dims 16r .. 16r + 15; rows r and
    // r + 8 of tile t are dims 16r + 2t and 16r + 2t + 1
#pragma unroll
    for (int kt = 0; kt < 2; ++kt) {
      uint2 vw[4];
      uint32_t sb[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int slot = 16 * kt + 4 * i + c;
        vw[i] = *reinterpret_cast<const uint2*>(st + kUnitCodes + slot * 64 + r * 8);
        sb[i] = st[2 * kUnitCodes + kUnitScales + slot * 8 + r];
      }
      uint32_t vs[2] = {scales2_to_f16(sb[0] | sb[1] << 8), scales2_to_f16(sb[2] | sb[3] << 8)};
      if (zero_v) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (zero_v >> (16 * kt + 4 * i + c) & 1u) {
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
        for (int i = 0; i < 4; ++i) {
          const uint32_t a0 = mul_f16x2(prmt(h[0][i], h[1][i], 0x5410), vs[0]), a1 = mul_f16x2(prmt(h[0][i], h[1][i], 0x7632), vs[0]);
          const uint32_t a2 = mul_f16x2(prmt(h[2][i], h[3][i], 0x5410), vs[1]), a3 = mul_f16x2(prmt(h[2][i], h[3][i], 0x7632), vs[1]);
#pragma unroll
          for (int n = 0; n < kN; ++n) mma16816(o[4 * w + i][n], a0, a1, a2, a3, pb[kt][n][0], pb[kt][n][1]);
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
  };
  // scores are at most 128 * 2^15 * 2688 < 2^33.4 times the row's factor: below 2^24
  bool below = true;
#pragma unroll
  for (int n = 0; n < kN; ++n) below = below && fmaxf(sc[n][0], sc[n][1]) < kFused * 0x1p-33f;
  if (__all_sync(0xffffffffu, below))
    take_pieces(std::false_type());
  else
    take_pieces(std::true_type());
  const auto warp_o = [&](int w) { return reinterpret_cast<float4*>(ring + w * kWarpRing); };
  const auto warp_m = [&](int w) { return reinterpret_cast<float*>(ring + w * kWarpRing + kWarpO); };
  // the block's rows: maxima first, then every warp's O relative to them
#pragma unroll
  for (int n = 0; n < kN; ++n)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) l[n][h] += __shfl_xor_sync(0xffffffffu, l[n][h], x);
      if (l[n][h] != l[n][h]) m[n][h] = 0.f;  // a NaN row stays one in every merge
      if (r == 0) {
        warp_m(warp)[8 * n + 2 * c + h] = m[n][h];
        warp_m(warp)[kFewRows + 8 * n + 2 * c + h] = l[n][h];
      }
    }
  __syncthreads();
#pragma unroll
  for (int n = 0; n < kN; ++n)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int row = 8 * n + 2 * c + h;
      if (row < R) {
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kFewWarps; ++w) M = fmaxf(M, warp_m(w)[row]);
        const float f = m[n][h] == -INFINITY ? 0.f : ex2_approx(m[n][h] - M);
        float4* dst = warp_o(warp) + row * 32;  // 4-dim pieces rotated by the row, against bank conflicts
#pragma unroll
        for (int t = 0; t < 4; ++t)
          dst[(4 * r + t + row) & 31] = make_float4(o[2 * t][n][h] * f, o[2 * t][n][2 + h] * f, o[2 * t + 1][n][h] * f,
                                                    o[2 * t + 1][n][2 + h] * f);
      }
    }
  __syncthreads();
  const int part = 2 * blockIdx.x + (sg.index ? 1 : 0);  // two per block: its first segment's and its last one's
  float4* out_part = p.part_o + static_cast<size_t>(part) * kFewRows * 32;
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
    if (whole) {
      const float inv = L == 0.f ? 0.f : rq.v_global / L;
      const size_t at = (q_base + static_cast<size_t>(row % p.rows) * p.Hq + row / p.rows) * kD + x * 4;
      *reinterpret_cast<uint2*>(p.out + at) = make_uint2(pack_bf16x2(a.x * inv, a.y * inv), pack_bf16x2(a.z * inv, a.w * inv));
    } else {
      out_part[i] = a;
      if (x == 0) p.part_ml[part * kFewRows + row] = make_float2(M, L);
    }
  }
  if (!whole && warp == 0) {
    int first_part, n_parts;
    few_parts(pl, sg, lane, first_part, n_parts);
    if (lane == 0) {
      ms->first_part = first_part;
      ms->n_parts = n_parts;
    }
  }
  // the last block of the group merges: its add acquires the others' partials
  __syncthreads();
  if (!whole) {
  if (threadIdx.x == 0) {
    uint32_t* count = p.count + sg.r * p.Hkv + head;
    const bool last = atom_add_acq_rel_gpu(count, 1u) == static_cast<uint32_t>(ms->n_parts - 1);
    if (last) *count = 0u;
    ms->last = last;
  }
  __syncthreads();
  if (ms->last) {
  // thread = (slice of the parts, row, dim quad): few rows leave threads for
  // several slices, which meet in the ring
  const int n_split = ms->n_parts, part0 = ms->first_part, items = R * 32, slices = max(1, kFewThreads / items);
  float4* s_o = reinterpret_cast<float4*>(ring);
  float2* s_ml = reinterpret_cast<float2*>(ring + kFewThreads * 16);
  for (int i0 = 0; i0 < items; i0 += kFewThreads) {
    const int slice = threadIdx.x / items, i = i0 + threadIdx.x - slice * items, row = i >> 5, x = i & 31;
    float M = -INFINITY, L = 0.f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    if (slice < slices && i < items) {
      constexpr int kAhead = 10;
#pragma unroll 1
      for (int s0 = slice; s0 < n_split; s0 += kAhead * slices) {
        float4 v[kAhead];
        float2 ml[kAhead];
#pragma unroll
        for (int e = 0; e < kAhead; ++e) {
          const int b = s0 + e * slices;
          const bool in = b < n_split;
          const int part_b = b ? (part0 & ~1) + 2 * b : part0;
          ml[e] = in ? __ldcg(p.part_ml + part_b * kFewRows + row) : make_float2(-INFINITY, 0.f);
          v[e] = in ? __ldcg(p.part_o + (static_cast<size_t>(part_b) * kFewRows + row) * 32 + x) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        float mx = M;
#pragma unroll
        for (int e = 0; e < kAhead; ++e) mx = fmaxf(mx, ml[e].x);
        const float keep = M == -INFINITY ? 0.f : ex2_approx(M - mx);
        M = mx;
        L *= keep;
        a = make_float4(a.x * keep, a.y * keep, a.z * keep, a.w * keep);
#pragma unroll
        for (int e = 0; e < kAhead; ++e) {
          const float f = ml[e].x == -INFINITY ? 0.f : ex2_approx(ml[e].x - mx);
          L = fmaf(f, ml[e].y, L);
          a = make_float4(fmaf(f, v[e].x, a.x), fmaf(f, v[e].y, a.y), fmaf(f, v[e].z, a.z), fmaf(f, v[e].w, a.w));
        }
      }
    }
    if (slices > 1) {  // then the rows fit the block at once
      s_o[threadIdx.x] = a;
      s_ml[threadIdx.x] = make_float2(M, L);
      __syncthreads();
      for (int y = 1; y < slices && !slice; ++y) {
        const float4 b = s_o[y * items + i];
        const float2 ml = s_ml[y * items + i];
        const float mx = fmaxf(M, ml.x);
        const float f0 = M == -INFINITY ? 0.f : ex2_approx(M - mx), f1 = ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - mx);
        M = mx;
        L = f0 * L + f1 * ml.y;
        a = make_float4(f0 * a.x + f1 * b.x, f0 * a.y + f1 * b.y, f0 * a.z + f1 * b.z, f0 * a.w + f1 * b.w);
      }
    }
    if (slice || i >= items) continue;
    const float inv = L == 0.f ? 0.f : rq.v_global / L;
    const size_t at = (q_base + static_cast<size_t>(row % p.rows) * p.Hq + row / p.rows) * kD + x * 4;
    *reinterpret_cast<uint2*>(p.out + at) = make_uint2(pack_bf16x2(a.x * inv, a.y * inv), pack_bf16x2(a.z * inv, a.w * inv));
  }
  }
  }
  // the ring is the copies' again
  fence_proxy_async_smem();
  __syncthreads();
  } while (next_segment<kFewLead>(p, pl, sg));
}

int few_grid() { return 2 * glance::num_sms(); }  // as many blocks as fit
// The counters come first in a workspace of any call, those of the largest one,
// so that calls of different shapes may take turns on one workspace.
constexpr size_t kCounterBytes = static_cast<size_t>(kMaxB) * glance::kKv4MaxHeads * sizeof(uint32_t);

// ------------------------------------------------ many query rows per kv head
//
// More than 16 query rows share a kv head: the products are worth the tensor
// core's 128-row tiles. A block has two softmax slots, each with its own S and
// O in tensor memory, that take turns on the tensor core: while one slot's
// warps turn S into weights, the other slot's products run.
//
//   warp 2        bulk copies of codes and scales (half tiles, three in flight)
//   warps 12..15  codes -> K (bf16, q's type) and V (f16) tiles in shared
//                 memory, in the 128-byte-swizzled layout of the tensor core, two
//                 stages
//   warp 0        S = Q K^T (both from shared memory) and O += P V (P from
//                 tensor memory, over the columns of its S)
//   warps 4..7, 8..11  softmax of slot 0 and 1, one thread per query row: mask,
//                 running maximum, weights as f16 pairs; Q at a segment's start;
//                 output at its end
//
// Tiles are 128 query rows (head, packed row) x 128 slots. Two neighbouring
// query tiles of a kv head go to the two slots and share every K and V tile
// (codes are widened once for both). A last tile without a neighbour has both
// slots: they take its slot tiles in turn and join at the end.
//
// A group that one block has whole is written out there; the others' parts are
// merged by a second kernel.
//
// Measured (32 / 8 heads, 64 rows): 131072 slots 116.3 us, whose useful operations
// are 62 % of the measured rate of a large bf16 product (the tensor core is active
// in 51 % of the kernel's clocks); 4096 slots 15.0 us; 8 requests of 512 to 8192
// slots 39.3 us. In the steady loop a pair of tiles takes 3500 clocks, of which
// the tensor core is active in 2048: a slot's chain is S and O's products (1380
// with the other slot's in between) and the softmax (2080), together 3460, the
// conversion warps need about as long for the pair's K and V, and tensor memory
// (two S, two O of 128 columns) has no room for a second S per slot that would let
// them overlap.
// S in two halves of 64 slots, which has, takes 170 us (twice the products, Q
// read from shared memory twice as often), weights handed over by halves 136: a
// hand-over costs more than what it lets overlap. Short calls are start-up: 1.4 us until the block knows its work, 3
// until the first S, 3.1 for two tiles, 0.85 for the output, 1 between the
// kernels, 3 for the merge (joining inside this kernel takes 17.9 us instead of
// 16.0 at 4096, blocks that wait for one another).

constexpr int kWideThreads = 512;
// Registers per thread: 128 at launch (65,536 for the block), then shared out
// between products + copies, softmax and conversion (64, 168, 104: 117.6 instead of
// 115.3 us at 131072 slots).
constexpr int kRegsFew = 56, kRegsSoftmax = 176, kRegsConvert = 104;
static_assert(128 * kRegsFew + 256 * kRegsSoftmax + 128 * kRegsConvert <= kWideThreads * 128, "register shares");
constexpr int kBM = 128, kBN = 128;
constexpr int kStages = 2, kRawStages = 3;
constexpr uint32_t kHalfBytes = kBN * 128;       // 64 dims x 128 rows, f16
constexpr uint32_t kTileBytes = 2 * kHalfBytes;  // a Q, K or V tile
constexpr uint32_t kRawCodes = kBN * glance::kKv4CodeBytes, kRawScales = kBN * glance::kKv4ScaleBytes;
constexpr uint32_t kRawBytes = kRawCodes + kRawScales;  // 9,216: codes and scales of a K or V tile
constexpr uint32_t kOffK = 2 * kTileBytes, kOffV = kOffK + kStages * kTileBytes, kOffRaw = kOffV + kStages * kTileBytes;
constexpr uint32_t kOffMisc = kOffRaw + kRawStages * kRawBytes;
constexpr uint32_t kWideMisc = 6144;
constexpr uint32_t kWideSmem = 1024 + kOffMisc + kWideMisc;
static_assert(kWideSmem <= 227 * 1024, "shared memory");
// A part has a tile or more. Starting and ending a group costs about 2.5 tiles
// (8, 10, 12 units measured: 44.6, 42.7, 44.8 us for 64 rows x 8 requests of 512
// to 8192 slots; 74.2, 70.5, 67.8 us for 256 rows x 5 of 100 to 5000).
constexpr int kWideMin = 4, kWideLead = 10;
constexpr unsigned long long kWaitNs = 2000000000ull;

struct WideMisc {
  uint64_t raw_full[kRawStages], raw_empty[kRawStages];
  uint64_t k_full[kStages], v_full[kStages], k_empty[kStages], v_empty[kStages];
  uint64_t q_ready[2], s_full[2], p_ready[2], o_done[2], drain;  // [slot]
  uint32_t tmem;
  int abort_flag, any;
  Segment seg;
  Plan plan;
  float2 ml[2][2][kBM];  // [segment parity][slot][row], slots that share a query tile
};
static_assert(sizeof(WideMisc) <= kWideMisc, "misc block");

// Slots of a segment: [k0, k1); its tiles start at k0, k0 + 128, ...
struct Run {
  int k0, k1, tiles;
  __device__ __forceinline__ Run(const Segment& s, int n_keys) {
    k0 = s.a * kUnit;
    k1 = min(k0 + s.n * kUnit, n_keys);
    tiles = (k1 - k0 + kBN - 1) / kBN;
  }
  __device__ __forceinline__ int key0(int j) const { return k0 + j * kBN; }
  // columns of tile j that its products compute, a multiple of 32
  __device__ __forceinline__ int cols(int j) const { return min(kBN, (k1 - key0(j) + 31) & ~31); }
  // whether tile j's products reach behind the prefix: the one rule by which V
  // rows without a number are left out of them and the softmax looks at the masks
  __device__ __forceinline__ bool tree(int j, int T) const { return key0(j) + cols(j) > T; }
};

__device__ __forceinline__ void wide_fail(WideMisc* ms) {
  report(GLANCE_DEV_PIPELINE_TIMEOUT);
  atomicExch(&ms->abort_flag, 1);
}
// Bounded wait of a converged warp; gives up once another role has.
__device__ __forceinline__ bool wide_wait(uint64_t* bar, uint32_t parity, WideMisc* ms) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t i = 1;; ++i) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    if ((i & 63u) == 0 &&
        __any_sync(0xffffffffu, *reinterpret_cast<volatile int*>(&ms->abort_flag) != 0 || globaltimer_ns() - t0 > kWaitNs))
      return false;
  }
}

__device__ __forceinline__ float max3f(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// kind::f16 with f16 A and B, fp32 accumulator, 128 rows, N columns, B MN-major
// (the V tile).
__host__ __device__ constexpr uint32_t idesc_f16(int N) {
  return (1u << 4) | (1u << 16) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(kBM >> 4) << 24);
}

__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(e));
  return e != 0;
}

// `steps` products of 16 along the inner dimension, issued by one lane of a
// converged warp so that descriptors stay in uniform registers.
__device__ __forceinline__ void issue_qk(uint32_t d, uint64_t q, uint64_t k, uint32_t idesc) {
#pragma unroll
  for (int kk = 0; kk < 8; ++kk) {
    const uint64_t off = ((kk >> 2) * kHalfBytes + (kk & 3) * 32) >> 4;
    mma_bf16_ss(d, q + off, k + off, idesc, kk > 0);
  }
}
__device__ __forceinline__ void issue_pv(uint32_t d, uint32_t p, uint64_t v, uint32_t idesc, int steps, bool fresh) {
#pragma unroll
  for (int kk = 0; kk < 8; ++kk)
    if (kk < steps) mma_bf16_ts(d, p + kk * 8, v + ((kk * 2048) >> 4), idesc, kk > 0 || !fresh);
}

// The 32 slots from tree index (slot - T) 32 i on that a row sees: slots of the
// prefix, then the row's mask up to the last packed row.
__device__ __forceinline__ uint32_t visible32(const uint64_t* anc, int rows, int i) {
  if (i < 0) return 0xFFFFFFFFu;
  const int left = rows - 32 * i;
  if (left <= 0) return 0u;
  const uint32_t seen = __ldg(reinterpret_cast<const uint32_t*>(anc) + i);
  return left < 32 ? seen & ((1u << left) - 1u) : seen;
}

// A thread's share of a tile: rows row + 8i (i = 0..3) of the 128, dims 32q ..
// 32q + 31 (16 bytes of codes, two scales). A warp has 32 rows; lane = 4 (row
// mod 8) + q, so that eight lanes read 128 consecutive bytes of codes.
struct Raw {
  uint4 codes[4];
  uint32_t scales[4];
};
__device__ __forceinline__ void load_raw(Raw& x, const unsigned char* codes, const unsigned char* scales, int row, int q,
                                         int left) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x.codes[i] = *reinterpret_cast<const uint4*>(codes + (row + 8 * i) * 64 + q * 16);
    x.scales[i] = *reinterpret_cast<const uint16_t*>(scales + (row + 8 * i) * 8 + q * 2);
    if (left < kBN && row + 8 * i >= left) {  // behind the run: zero, whatever is there
      x.codes[i] = make_uint4(0, 0, 0, 0);
      x.scales[i] = 0;
    }
  }
}

// ... as 16-bit values into the tile (K as bf16, the type of q; V as f16, the
// type of the weights: a product has one type, and code * scale is exact in
// both): row r's 16-byte chunk c of a half (64 dims) is at
// r * 128 + 16 (c ^ (r & 7)). Lanes of the upper half take their four chunks
// in the order 2, 3, 0, 1: eight lanes (two rows, four q) then write eight
// different 16-byte columns of the 128-byte rows, and no bank twice.
template <bool kIsV>
__device__ __forceinline__ void store_tile(const Raw& x, unsigned char* tile, int row, int q) {
  unsigned char* base = tile + (q >> 1) * kHalfBytes + row * 128;
  const bool up = q >= 2;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t s = scales2_to_f16(x.scales[i]);
    uint32_t s0 = prmt(s, s, up ? 0x3232 : 0x1010), s1 = prmt(s, s, up ? 0x1010 : 0x3232);
    if (!kIsV) {  // times 2^112, as bf16
      const float2 f = f16x2_to_f32(prmt(s0, s1, 0x5410));
      s0 = pack_bf16x2(f.x * 0x1p112f, f.x * 0x1p112f);
      s1 = pack_bf16x2(f.y * 0x1p112f, f.y * 0x1p112f);
    }
    const uint32_t w[4] = {up ? x.codes[i].z : x.codes[i].x, up ? x.codes[i].w : x.codes[i].y,
                           up ? x.codes[i].x : x.codes[i].z, up ? x.codes[i].y : x.codes[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t h[4];
      codes8_to_f16(w[j], h);
      const uint32_t sj = j < 2 ? s0 : s1;
      const int chunk = ((q & 1) * 4 + (j ^ (q & 2))) ^ (row & 7);
      *reinterpret_cast<uint4*>(base + i * 8 * 128 + chunk * 16) =
          kIsV ? make_uint4(mul_f16x2(h[0], sj), mul_f16x2(h[1], sj), mul_f16x2(h[2], sj), mul_f16x2(h[3], sj))
               : make_uint4(mul_bf16x2(f16_codes_to_bf16(h[0]), sj), mul_bf16x2(f16_codes_to_bf16(h[1]), sj),
                            mul_bf16x2(f16_codes_to_bf16(h[2]), sj), mul_bf16x2(f16_codes_to_bf16(h[3]), sj));
    }
  }
}

// Eight values of a row times f, as f16 and as bf16.
__device__ __forceinline__ uint4 eight_f16(const uint32_t* r, float f) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = pack_f16x2(__uint_as_float(r[2 * i]) * f, __uint_as_float(r[2 * i + 1]) * f);
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint4 eight_bf16(const uint32_t* r, float f) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = pack_bf16x2(__uint_as_float(r[2 * i]) * f, __uint_as_float(r[2 * i + 1]) * f);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__global__ void __launch_bounds__(kWideThreads, 1) kv4_attention_wide_kernel(const __grid_constant__ Params p) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                         ~static_cast<uintptr_t>(1023));
  WideMisc* ms = reinterpret_cast<WideMisc*>(smem + kOffMisc);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int blocks = gridDim.x;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kRawStages; ++s) {
      mbar_init(&ms->raw_full[s], 1);
      mbar_init(&ms->raw_empty[s], 4);
    }
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&ms->k_full[s], 4);
      mbar_init(&ms->v_full[s], 4);
      mbar_init(&ms->k_empty[s], 1);
      mbar_init(&ms->v_empty[s], 1);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&ms->q_ready[x], 128);
      mbar_init(&ms->s_full[x], 1);
      mbar_init(&ms->p_ready[x], 4);
      mbar_init(&ms->o_done[x], 1);
    }
    mbar_init(&ms->drain, 1);
    ms->abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(&ms->tmem, 512);
    tmem_relinquish();
  }
  pdl_wait_prior();
  pdl_launch_dependents();
  if (warp == 3) {
    make_plan<kWideMin, kWideLead>(p, &ms->plan, lane, blocks);
    __syncwarp();
    Segment s;
    const bool any = first_segment<kWideLead>(p, ms->plan, blockIdx.x, lane, s);
    if (lane == 0) {
      ms->any = any;
      ms->seg = s;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ms->tmem;
  const Plan& pl = ms->plan;
  const bool any = ms->any != 0;

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsFew));
    if (warp == 0 && any) {
      // ------------------------------------------------------------- products
      const uint64_t q_desc = sdesc_sw128(smem_u32(smem), 16, 1024);
      const uint64_t k_desc = sdesc_sw128(smem_u32(smem + kOffK), 16, 1024);
      const uint64_t v_desc = sdesc_sw128(smem_u32(smem + kOffV), kHalfBytes, 1024);
      constexpr uint64_t kTileStep = kTileBytes >> 4;
      Segment s = ms->seg;
      int t0 = 0;                // slot tiles of the block before this segment
      uint32_t n_q[2] = {0, 0};  // phases of q_ready and p_ready so far
      uint32_t n_p[2] = {0, 0};
      bool good = true;
      do {
        const Run run(s, pl.T[s.r] + p.rows);
        const bool pair = 2 * (s.g % p.n_qp) + 1 < p.n_qt;
        const int items = pair ? 2 * run.tiles : run.tiles;
        // Item k: slot k & 1, tile k / 2 of a pair or tile k. A K or V tile is
        // waited for by its first item and let go by its last one. Tiles are
        // waited for before the weights, which come last.
        const auto tile_of = [&](int k) { return pair ? k >> 1 : k; };
        const auto wait_tile = [&](uint64_t* full, int k) {
          const int t = t0 + tile_of(k);
          return (pair && (k & 1)) || wide_wait(&full[t & 1], (t >> 1) & 1, ms);
        };
        const auto issue_s = [&](int k) {
          const int x = k & 1, j = tile_of(k), st = (t0 + j) & 1;
          if (elect_one()) {
            issue_qk(tmem + x * 128, q_desc + (pair ? x * kTileStep : 0), k_desc + st * kTileStep, idesc_bf16_f32(kBM, run.cols(j), false, false));
            mma_commit(&ms->s_full[x]);
            if (!pair || x) mma_commit(&ms->k_empty[st]);
          }
          __syncwarp();
        };
        for (int x = 0; x < (pair ? 2 : 1) && good; ++x) good = wide_wait(&ms->q_ready[x], n_q[x]++ & 1, ms);
        for (int k = 0; k < 2 && k < items && good; ++k) {
          good = wait_tile(ms->k_full, k);
          tc_fence_after();
          if (good) issue_s(k);
        }
        for (int k = 0; good && k < items; ++k) {
          const int x = k & 1, j = tile_of(k), st = (t0 + j) & 1;
          good = wait_tile(ms->v_full, k) && (k + 2 >= items || wait_tile(ms->k_full, k + 2)) &&
                 wide_wait(&ms->p_ready[x], n_p[x]++ & 1, ms);
          if (!good) break;
          tc_fence_after();
          if (elect_one()) {
            issue_pv(tmem + 256 + x * 128, tmem + x * 128, v_desc + st * kTileStep, idesc_f16(kD), run.cols(j) / 16, k < 2);
            if (!pair || x) mma_commit(&ms->v_empty[st]);
            if (k + 2 >= items) mma_commit(&ms->o_done[x]);
          }
          __syncwarp();
          // the slot's next S takes the columns of these weights: products run in the order of their issue
          if (k + 2 < items) issue_s(k + 2);
        }
        t0 += run.tiles;
      } while (good && next_segment<kWideLead>(p, pl, s));
      if (!good) wide_fail(ms);
    } else if (warp == 2 && any) {
      // ---------------------------------------------------------- bulk copies
      Segment s = ms->seg;
      int h = 0;  // half tiles so far: K, V, K, V, ...
      bool good = true;
      do {
        const Request& rq = p.req[s.r];
        const Run run(s, pl.T[s.r] + p.rows);
        const long long head0 = static_cast<long long>(s.g / p.n_qp) * rq.head_stride;
        for (int e = 0; e < 2 * run.tiles && good; ++e, ++h) {
          const int st = h % kRawStages, key0 = run.key0(e >> 1);
          if (h >= kRawStages) good = wide_wait(&ms->raw_empty[st], (h / kRawStages - 1) & 1, ms);
          if (!good) break;
          if (lane == 0) {
            unsigned char* dst = smem + kOffRaw + st * kRawBytes;
            const int n = min(kBN, (run.k1 - key0 + 1) & ~1);  // an even number: 16 bytes of scales
            if (GLANCE_IN_BOUNDS(key0 + n - 1, rq.head_stride)) {
              const long long at = head0 + key0;
              mbar_arrive_expect_tx(&ms->raw_full[st], n * (glance::kKv4CodeBytes + glance::kKv4ScaleBytes));
              bulk_copy_g2s(dst, (e & 1 ? rq.v : rq.k) + at * 64, n * 64, &ms->raw_full[st]);
              bulk_copy_g2s(dst + kRawCodes, (e & 1 ? rq.v_scale : rq.k_scale) + at * 8, n * 8, &ms->raw_full[st]);
            } else {
              mbar_arrive(&ms->raw_full[st]);
            }
          }
          __syncwarp();
        }
      } while (good && next_segment<kWideLead>(p, pl, s));
      if (!good) {
        wide_fail(ms);
        for (int u = max(0, h - kRawStages); u < h; ++u)  // the copies in flight land before the block leaves
          (void)mbar_wait(&ms->raw_full[u % kRawStages], (u / kRawStages) & 1, 50000000ull);
      }
    } else if (warp == 3) {
      // ------------------------------------------ which blocks have a group
      // for the merge: by the block that has the group's first unit; requests
      // without room have none
      if (any) {
        Segment s = ms->seg;
        do {
          if (s.a) continue;
          int n = 1;
          if (pl.tau) {
            n = (pl.units[s.r] + pl.tau - 1) / pl.tau;
          } else {
            const long long end = pl.base[s.r] + (s.g + 1ll) * (pl.units[s.r] + kWideLead);
            for (;; n += 32) {
              const unsigned past = __ballot_sync(0xffffffffu, run_start(pl.total, blockIdx.x + n + lane, pl.runs) >= end);
              if (past) {
                n += __ffs(past) - 1;
                break;
              }
            }
          }
          if (lane == 0) p.group[s.r * p.Hkv * p.n_qp + s.g] = make_int2(2 * blockIdx.x + (s.index ? 1 : 0), n);
        } while (next_segment<kWideLead>(p, pl, s));
      }
      if (blockIdx.x == 0)
        for (int r = 0; r < p.B; ++r)
          if (pl.units[r] == 0) {
            if (lane == 0) report(GLANCE_DEV_TREE_CAPACITY);
            for (int g = lane; g < p.Hkv * p.n_qp; g += 32) p.group[r * p.Hkv * p.n_qp + g] = make_int2(0, 0);
          }
    }
  } else if (warp >= 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsConvert));
    if (any) {
      // --------------------------------------------------- codes to f16 tiles
      const int row = (warp - 12) * 32 + (lane >> 2), q = lane & 3;
      Segment s = ms->seg;
      int h = 0;
      bool good = true;
      do {
        const int T = pl.T[s.r];
        const Run run(s, T + p.rows);
        for (int e = 0; e < 2 * run.tiles; ++e, ++h) {
          const int rs = h % kRawStages, t = h >> 1, st = t & 1, is_v = h & 1, key0 = run.key0(e >> 1);
          good = wide_wait(&ms->raw_full[rs], (h / kRawStages) & 1, ms);
          if (!good) break;
          const unsigned char* src = smem + kOffRaw + rs * kRawBytes;
          Raw x;
          load_raw(x, src, src + kRawCodes, row, q, run.k1 - key0);
          __syncwarp();
          if (lane == 0) mbar_arrive(&ms->raw_empty[rs]);
          if (is_v && run.tree(e >> 1, T)) {
            // a V row with a scale that is not a number is left out: 0 * NaN
            // would reach the rows that do not see it (the softmax marks the
            // scores of those that do). In a tile of prefix slots alone it stays:
            // every row sees it
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const bool nan = (x.scales[i] & 0x7Fu) == 0x7Fu || (x.scales[i] & 0x7F00u) == 0x7F00u;
              if (__ballot_sync(0xffffffffu, nan) >> (lane & 28) & 15u) {
                x.codes[i] = make_uint4(0, 0, 0, 0);
                x.scales[i] = 0;
              }
            }
          }
          if (t >= kStages) good = wide_wait(is_v ? &ms->v_empty[st] : &ms->k_empty[st], ((t >> 1) - 1) & 1, ms);
          if (!good) break;
          if (is_v)
            store_tile<true>(x, smem + kOffV + st * kTileBytes, row, q);
          else
            store_tile<false>(x, smem + kOffK + st * kTileBytes, row, q);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(is_v ? &ms->v_full[st] : &ms->k_full[st]);
        }
      } while (good && next_segment<kWideLead>(p, pl, s));
      if (!good) wide_fail(ms);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    if (any) {
      // ------------------------------------------------------------- softmax
      const int x = warp >= 8, lrow = (warp & 3) * 32 + lane;
      const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
      const uint32_t tS = tmem + lanes + x * 128, tO = tmem + lanes + 256 + x * 128;
      const int R = p.G * p.rows;
      uint32_t n_s = 0, n_o = 0;  // phases of this slot's s_full and o_done so far
      bool ok = true;
      bool ahead = false;  // the segment's Q is in its tile already
      // A segment's Q into the slot's tile, 16 bytes at a time (thread = chunk, 16
      // to a row); rows behind the last are zero. The products that read the tile
      // before are done.
      const auto copy_q = [&](const Segment& s) {
        const int R = p.G * p.rows, head = s.g / p.n_qp, qt0 = 2 * (s.g % p.n_qp), xq = qt0 + 1 < p.n_qt ? x : 0;
        const int th = (warp & 3) * 32 + lane, c = th & 15;
        unsigned char* dst = smem + xq * kTileBytes + (c >> 3) * kHalfBytes;
        int i = th >> 4, qr = (qt0 + xq) * kBM + i;
        int h = qr / p.rows, pr = qr - h * p.rows;  // query head of the group, packed row
        const __nv_bfloat16* src = p.q + (static_cast<size_t>(s.r) * p.rows * p.Hq + head * p.G) * kD + c * 8;
        int at = (pr * p.Hq + h) * kD;  // of the row's head in q
        const int step = 8 * p.Hq * kD, wrap = kD - p.rows * p.Hq * kD;  // 8 packed rows on; the next head's first
        dst += i * 128 + (((c & 7) ^ (i & 7)) << 4);  // i steps by 8: the swizzle stays
#pragma unroll 4
        for (; i < kBM; i += 8) {
          if (qr < R)
            copy16_async(dst, src + at);
          else
            *reinterpret_cast<uint4*>(dst) = make_uint4(0, 0, 0, 0);
          dst += 8 * 128;
          qr += 8;
          pr += 8;
          at += step;
          while (pr >= p.rows) {
            pr -= p.rows;
            at += wrap;
          }
        }
      };
      const auto q_copied = [&] {
        copy_async_wait();
        fence_proxy_async_smem();
        mbar_arrive(&ms->q_ready[x]);
      };
      Segment s = ms->seg;
      do {
        const Request& rq = p.req[s.r];
        const int T = pl.T[s.r];
        const Run run(s, T + p.rows);
        const int head = s.g / p.n_qp, qt0 = 2 * (s.g % p.n_qp);
        const bool pair = qt0 + 1 < p.n_qt;
        // The thread's query row, worked out anew wherever it is needed: kept,
        // it would cost registers while a row of S is in them.
        const auto query = [&](bool& valid, int& prow) -> size_t {
          int qrow = (pair ? qt0 + x : qt0) * kBM + lrow;
          asm volatile("" : "+r"(qrow));
          valid = qrow < R;
          prow = valid ? qrow % p.rows : 0;
          return ((static_cast<size_t>(s.r) * p.rows + prow) * p.Hq + head * p.G + (valid ? qrow / p.rows : 0)) * kD;
        };
        // score factor, in log2; at least the least normal number: a score of -infinity stays one
        const float sc = fmaxf(p.scale_log2 * rq.k_global, 1.17549435e-38f);
        if (!ahead && (pair || !x)) {
          copy_q(s);
          q_copied();
        }
        ahead = false;
        float m = -INFINITY, l = 0.f;
        const int step = pair ? 1 : 2, j0 = pair ? 0 : x;
        // The segment's tiles from j on, the first one from its half `from` on where
        // that is not -1. Without rounded products: returns at the half whose maximum
        // is the first beyond kFused; else -1.
        const auto softmax_tiles = [&](auto rounded, int& j, int from) -> int {
        constexpr bool kRounded = decltype(rounded)::value;
        for (; j < run.tiles; j += step) {
          const int key0 = run.key0(j);
          const int nc = run.cols(j) / 32;
          const bool tree = run.tree(j, T);
          uint32_t bad[4] = {0u, 0u, 0u, 0u};  // slots with a V scale that is not a number
          uint32_t vis[4];                     // slots that the row sees
          if (tree) {
            bool valid;
            int prow;
            (void)query(valid, prow);
            const uint64_t* anc = rq.anc + static_cast<size_t>(prow) * p.W;
            const int kb = key0 - T;
            uint32_t w[5];
#pragma unroll
            for (int i = 0; i < 5; ++i) w[i] = valid ? visible32(anc, p.rows, (kb >> 5) + i) : 0u;
#pragma unroll
            for (int i = 0; i < 4; ++i) vis[i] = __funnelshift_r(w[i], w[i + 1], kb & 31);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int slot = key0 + 32 * i + lane;
              uint2 vs = make_uint2(0, 0);
              if (slot < run.k1 && GLANCE_IN_BOUNDS(slot, rq.t_cap))
                vs = __ldg(reinterpret_cast<const uint2*>(rq.v_scale) + static_cast<long long>(head) * rq.head_stride + slot);
              const uint32_t nan = __vcmpeq4(vs.x & 0x7F7F7F7Fu, 0x7F7F7F7Fu) | __vcmpeq4(vs.y & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
              bad[i] = __ballot_sync(0xffffffffu, nan != 0u);
            }
          }
          if (!kRounded || from < 0) {
          ok = wide_wait(&ms->s_full[x], n_s++ & 1, ms);
          if (!ok) return -1;
          tc_fence_after();
          if (tree) {
            // masked in place, so that the rest is the same for every tile
#pragma unroll 1
            for (int c = 0; c < nc; ++c) {
              const uint32_t seen = c == 0 ? vis[0] : c == 1 ? vis[1] : c == 2 ? vis[2] : vis[3];
              uint32_t r[32], y[16], z[16];
              tmem_ld32(tS + 32 * c, r);
              tmem_wait32(r);
              const uint32_t b = c == 0 ? bad[0] : c == 1 ? bad[1] : c == 2 ? bad[2] : bad[3];
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                y[e] = !(seen >> e & 1u) ? 0xFF800000u : (b >> e & 1u) ? 0x7FC00000u : r[e];
                z[e] = !(seen >> (16 + e) & 1u) ? 0xFF800000u : (b >> (16 + e) & 1u) ? 0x7FC00000u : r[16 + e];
              }
              tmem_st16(tS + 32 * c, y);
              tmem_st16(tS + 32 * c + 16, z);
            }
            tmem_st_wait();
          }
          }
          // 64 slots at a time: a whole row would not fit the registers
#pragma unroll 1
          for (int h = kRounded ? max(from, 0) : 0; 2 * h < nc; ++h) {
            uint32_t sr[64];
            tmem_row64(tS + 64 * h, sr);
            const bool both = 2 * h + 1 < nc;  // the product has the second 32 slots
            float mx[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) mx[i] = max3f(__uint_as_float(sr[i]), __uint_as_float(sr[8 + i]), __uint_as_float(sr[16 + i]));
#pragma unroll
            for (int i = 0; i < 8; ++i) mx[i] = fmaxf(mx[i], __uint_as_float(sr[24 + i]));
            if (both) {
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                mx[i] = max3f(mx[i], __uint_as_float(sr[32 + i]), __uint_as_float(sr[40 + i]));
                mx[i] = max3f(mx[i], __uint_as_float(sr[48 + i]), __uint_as_float(sr[56 + i]));
              }
            }
            const float top = fmaxf(max3f(mx[0], mx[1], mx[2]), max3f(max3f(mx[3], mx[4], mx[5]), mx[6], mx[7]));
            const float mt = __fmul_rn(top, sc);  // not fused with what follows: the rounded products' own maximum
            // m moves when some row of the warp grew by 8 (log2): a stale one keeps
            // the weights below 2^15 and cancels between O and l
            if (__any_sync(0xffffffffu, mt > __fadd_rd(m, kGrow))) {
              if (!kRounded && __any_sync(0xffffffffu, fabsf(mt) >= kFused && mt > -INFINITY)) return h;
              const float mn = fmaxf(m, mt - kUnder);
              const float alpha = m == -INFINITY ? 0.f : ex2_approx(m - mn);
              m = mn;
              l *= alpha;
              // O is complete (S of this tile came after the product of the last)
              // but for the weights of the row's first half
              if (j > j0)
#pragma unroll 1
                for (int c = 0; c < 8; ++c) {
                  uint32_t r[16];
                  tmem_ld16(tO + 16 * c, r);
#pragma unroll
                  for (int e = 0; e < 16; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * alpha);
                  tmem_st16(tO + 16 * c, r);
                }
              if (h) {
                tmem_st_wait();
#pragma unroll 1
                for (int c = 0; c < 2; ++c) {
                  uint32_t r[16];
                  tmem_ld16(tS + 16 * c, r);
#pragma unroll
                  for (int e = 0; e < 16; ++e) {
                    const float2 f = f16x2_to_f32(r[e]);
                    r[e] = pack_f16x2(f.x * alpha, f.y * alpha);
                  }
                  tmem_st16(tS + 16 * c, r);
                }
              }
            }
            const float off = m == -INFINITY ? 0.f : m;
            const unsigned long long sc2 = pair_f2(sc, sc), no2 = pair_f2(-off, -off);
            unsigned long long l2 = pair_f2(0.f, 0.f), l3 = l2;
#pragma unroll
            for (int c = 0; c < 2; ++c)
              if (c == 0 || both) {
                uint32_t pk[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                  float u0, u1;
                  const float s0 = __uint_as_float(sr[32 * c + 2 * e]), s1 = __uint_as_float(sr[32 * c + 2 * e + 1]);
                  split_f2(kRounded ? add_f2(pair_f2(__fmul_rn(s0, sc), __fmul_rn(s1, sc)), no2) : fma_f2(pair_f2(s0, s1), sc2, no2),
                           u0, u1);
                  const float p0 = ex2_approx(u0), p1 = ex2_approx(u1);
                  if (e & 1)
                    l3 = add_f2(l3, pair_f2(p0, p1));
                  else
                    l2 = add_f2(l2, pair_f2(p0, p1));
                  pk[e] = pack_f16x2(p0, p1);
                }
                tmem_st16(tS + 32 * h + 16 * c, pk);
              }
            float l0, l1;
            split_f2(add_f2(l2, l3), l0, l1);
            l += l0 + l1;
          }
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&ms->p_ready[x]);
          if (kRounded) from = -1;
        }
        return -1;
        };
        int j = j0;
        const int from = softmax_tiles(std::false_type(), j, -1);
        if (from >= 0) (void)softmax_tiles(std::true_type(), j, from);
        if (!ok && pair) break;
        // a row that sees a prefix slot has a weight of 2^7 or more unless all its
        // scores are -infinity: then it is no number
        if (l == 0.f && j0 < run.tiles && run.key0(j0) < T) l = __uint_as_float(0x7FC00000u);
        // ------------------------------------------------ the segment's output
        const bool whole = s.n == pl.units[s.r];
        bool valid;
        int prow;
        const size_t q_at = query(valid, prow);
        // two parts per block: its first segment's and its last one's, each of
        // two query tiles, O / l rounded to f16: off by at most 2^-11 of an
        // element, an eighth of the output's own rounding, and half the bytes
        const size_t part = 2 * (2 * static_cast<size_t>(blockIdx.x) + (s.index ? 1 : 0)) + (pair ? x : 0);
        uint4* po = p.part + part * 16 * kBM + lrow;
        if (l != l) m = 0.f;  // a NaN row stays one in every merge
        if (pair) {
          // the slot's last S is done with the Q tile: the next segment's Q comes
          // during its last product, and the next S during the output
          Segment next = s;
          ahead = next_segment<kWideLead>(p, pl, next) && (!x || 2 * (next.g % p.n_qp) + 1 < p.n_qt);
          if (ahead) copy_q(next);
          ok = wide_wait(&ms->o_done[x], n_o++ & 1, ms);
          if (!ok) break;
          tc_fence_after();
          if (ahead) q_copied();
          const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t r[32];
            tmem_ld32(tO + 32 * c, r);
            tmem_wait32(r);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if (!whole)
                po[(4 * c + e) * kBM] = eight_f16(r + 8 * e, inv);
              else if (valid)
                *reinterpret_cast<uint4*>(p.out + q_at + 32 * c + 8 * e) = eight_bf16(r + 8 * e, inv * rq.v_global);
            }
          }
          if (!whole) p.part_ml[part * kBM + lrow] = make_float2(m, l);
        } else {
          // both slots have this query tile: slot x writes dims 64x .. 64x + 63
          float2(*ml)[kBM] = ms->ml[s.index & 1];
          ml[x][lrow] = make_float2(m, l);
          // each waits for its own products (one tile: slot 1 has none), the barrier for the other's
          if (ok && x < run.tiles) ok = wide_wait(&ms->o_done[x], n_o++ & 1, ms);
          tc_fence_before();
          ok = !named_bar_or(1, 256, !ok);  // both go on, or both leave
          if (!ok) {
            s.left = 0;
            break;
          }
          tc_fence_after();
          const float2 a = ml[0][lrow], b = ml[1][lrow];
          const float M = fmaxf(a.x, b.x);
          const float fa = a.x == -INFINITY ? 0.f : ex2_approx(a.x - M), fb = b.x == -INFINITY ? 0.f : ex2_approx(b.x - M);
          const float L = fa * a.y + fb * b.y, inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll 1
          for (int c = 2 * x; c < 2 * x + 2; ++c) {
            uint32_t r[32], r1[32];
            tmem_ld32(tmem + lanes + 256 + 32 * c, r);
            tmem_wait32(r);
            if (run.tiles > 1) {
              tmem_ld32(tmem + lanes + 384 + 32 * c, r1);
              tmem_wait32(r1);
            }
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const float o1 = run.tiles > 1 ? fb * __uint_as_float(r1[e]) : 0.f;
              r[e] = __float_as_uint(fmaf(fa, __uint_as_float(r[e]), o1));
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if (!whole)
                po[(4 * c + e) * kBM] = eight_f16(r + 8 * e, inv);
              else if (valid)
                *reinterpret_cast<uint4*>(p.out + q_at + 32 * c + 8 * e) = eight_bf16(r + 8 * e, inv * rq.v_global);
            }
          }
          if (!whole && !x) p.part_ml[part * kBM + lrow] = make_float2(M, L);
          tc_fence_before();
          named_bar(1, 256);  // both have read both O before either slot's next product
        }
        tc_fence_before();
      } while (next_segment<kWideLead>(p, pl, s));
      if (!ok) {
        // after a failed wait the other slot gives up as well, but may first come
        // to the barrier of a query tile that both slots have
        wide_fail(ms);
        copy_async_wait();
        while (next_segment<kWideLead>(p, pl, s))
          if (2 * (s.g % p.n_qp) + 1 >= p.n_qt) {
            (void)named_bar_or(1, 256, true);
            break;
          }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (*reinterpret_cast<volatile int*>(&ms->abort_flag) && any) {
    // after a failed wait products may still be running
    if (warp == 0 && lane == 0) {
      mma_commit(&ms->drain);
      (void)mbar_wait(&ms->drain, 0, 50000000ull);
    }
    tc_fence_before();
    __syncthreads();
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// The parts of the groups that several blocks had. Block (query tile, 8 rows):
// thread = (slice of the parts, octet of dims, row); five parts at a time. The
// more blocks a group can have, the more slices share them.
constexpr int kMergeRows = 8;

template <int kSlices>
__global__ void __launch_bounds__(128 * kSlices) kv4_attention_merge_kernel(const __grid_constant__ Params p) {
  __shared__ float s_o[kSlices][8][128];
  __shared__ float2 s_ml[kSlices][128];
  const int tile = blockIdx.x / (kBM / kMergeRows), rows0 = blockIdx.x % (kBM / kMergeRows) * kMergeRows;
  const int qt = tile % p.n_qt, rh = tile / p.n_qt;  // request * Hkv + head
  const int t = threadIdx.x & 127, row = t & 7, octet = t >> 3, slice = threadIdx.x >> 7;
  const int lrow = rows0 + row, qrow = qt * kBM + lrow;
  const int r = rh / p.Hkv, head = rh % p.Hkv;
  size_t at = ((static_cast<size_t>(r) * p.rows + qrow % p.rows) * p.Hq + head * p.G + qrow / p.rows) * kD + octet * 8;
  asm volatile("" : "+l"(at));  // worked out here, while the kernel before this one ends
  pdl_wait_prior();  // in every block: this kernel ends after the one before it
  pdl_launch_dependents();
  if (qt * kBM + rows0 >= p.G * p.rows) return;
  const int2 gi = __ldcg(p.group + rh * p.n_qp + qt / 2);
  const int n = gi.y;
  if (n < 2) return;  // written whole, or no output
  // the first block's part is gi.x (its first or last segment), the others' their first segments
  const auto part_of = [&](int b) { return 2 * static_cast<size_t>(b ? (gi.x & ~1) + 2 * b : gi.x) + (qt & 1); };
  const int per = (n + kSlices - 1) / kSlices, b0 = slice * per, b1 = min(n, b0 + per);
  float M = -INFINITY, L = 0.f, a[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  constexpr int kAhead = 5;
#pragma unroll 1
  for (int s0 = b0; s0 < b1; s0 += kAhead) {
    uint4 v[kAhead];
    float2 ml[kAhead];
#pragma unroll
    for (int e = 0; e < kAhead; ++e) {
      const bool in = s0 + e < b1;
      const size_t part = part_of(in ? s0 + e : b0);
      ml[e] = in ? __ldcg(p.part_ml + part * kBM + lrow) : make_float2(-INFINITY, 0.f);
      v[e] = in ? __ldcg(p.part + (part * 16 + octet) * kBM + lrow) : make_uint4(0, 0, 0, 0);
    }
    float mx = M;
#pragma unroll
    for (int e = 0; e < kAhead; ++e) mx = fmaxf(mx, ml[e].x);
    const float keep = M == -INFINITY ? 0.f : ex2_approx(M - mx);
    M = mx;
    L *= keep;
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] *= keep;
#pragma unroll
    for (int e = 0; e < kAhead; ++e) {
      const float w = ml[e].x == -INFINITY ? 0.f : ex2_approx(ml[e].x - mx) * ml[e].y;
      const uint32_t h[4] = {v[e].x, v[e].y, v[e].z, v[e].w};
      L += w;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = f16x2_to_f32(h[i]);
        a[2 * i] = fmaf(w, f.x, a[2 * i]);
        a[2 * i + 1] = fmaf(w, f.y, a[2 * i + 1]);
      }
    }
  }
  if (kSlices > 1) {
    if (slice) {
#pragma unroll
      for (int i = 0; i < 8; ++i) s_o[slice][i][t] = a[i];
      s_ml[slice][t] = make_float2(M, L);
    }
    __syncthreads();
    if (slice) return;
    float mx = M;
#pragma unroll
    for (int y = 1; y < kSlices; ++y) mx = fmaxf(mx, s_ml[y][t].x);
    const float f0 = M == -INFINITY ? 0.f : ex2_approx(M - mx);
    L *= f0;
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] *= f0;
#pragma unroll
    for (int y = 1; y < kSlices; ++y) {
      const float2 ml = s_ml[y][t];
      const float f = ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - mx);
      L = fmaf(f, ml.y, L);
#pragma unroll
      for (int i = 0; i < 8; ++i) a[i] = fmaf(f, s_o[y][i][t], a[i]);
    }
  }
  if (qrow >= p.G * p.rows) return;
  const float inv = L == 0.f ? 0.f : p.req[r].v_global / L;
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = pack_bf16x2(a[2 * i] * inv, a[2 * i + 1] * inv);
  *reinterpret_cast<uint4*>(p.out + at) = make_uint4(w[0], w[1], w[2], w[3]);
}

size_t wide_group_bytes(int B, int Hkv, int n_qp) { return (static_cast<size_t>(B) * Hkv * n_qp * sizeof(int2) + 255) / 256 * 256; }
size_t wide_parts() { return 4 * static_cast<size_t>(glance::num_sms()); }  // 128 rows each

bool few_rows(int rows, int G) { return rows * G <= kFewRows; }

size_t workspace_bytes_of(int B, int rows, int Hq, const glance_kv4* kv) {
  const int Hkv = kv[0].n_kv_heads;
  if (few_rows(rows, Hq / Hkv))
    return kCounterBytes + 2 * static_cast<size_t>(few_grid()) * kFewRows * (kD * 4 + sizeof(float2));
  const int n_qp = (rows * (Hq / Hkv) + 2 * kBM - 1) / (2 * kBM);
  return kCounterBytes + wide_group_bytes(B, Hkv, n_qp) + wide_parts() * kBM * (kD * 2 + sizeof(float2));
}

}  // namespace

extern "C" size_t glance_kv4_tree_attention_workspace_bytes(int B, int n_rows, int n_q_heads, const glance_kv4* kv) {
  if (!kv || B < 1 || B > kMaxB || n_rows < 1 || n_rows > 256 || n_q_heads < 1) return 0;
  for (int r = 0; r < B; ++r)
    if (kv[r].n_kv_heads != kv[0].n_kv_heads || kv[r].n_kv_heads < 1 || kv[r].n_kv_heads > glance::kKv4MaxHeads ||
        n_q_heads % kv[r].n_kv_heads ||
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
  for (int r = 0; r < B; ++r)  // the kernels' score factor: with infinity a score of 0 would be NaN
    if (!isfinite(scale * kLog2e * kv[r].k_global))
      return fail(GLANCE_ERR_INVALID_ARG, "%s: scale * k_global * log2 e must be finite (request %d)", who, r);
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
  p.n_qt = (G * rows + kBM - 1) / kBM;
  p.n_qp = (p.n_qt + 1) / 2;
  p.part_o = nullptr;
  p.part = nullptr;
  p.group = nullptr;
  p.count = nullptr;
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
    const int grid = few_grid();
    const auto kernel = rows * G <= 8 ? kv4_attention_few_kernel<1> : kv4_attention_few_kernel<2>;
    char* ws = static_cast<char*>(workspace);
    p.count = reinterpret_cast<uint32_t*>(ws);
    p.part_o = reinterpret_cast<float4*>(ws + kCounterBytes);
    p.part_ml = reinterpret_cast<float2*>(p.part_o + 2 * static_cast<size_t>(grid) * kFewRows * 32);
    e = glance::ensure_smem(reinterpret_cast<const void*>(kernel), kFewSmem);
    if (e != cudaSuccess) return glance::cuda_fail(e, who);
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kFewThreads);
    cfg.dynamicSmemBytes = kFewSmem;
    e = cudaLaunchKernelEx(&cfg, kernel, p);
  } else {
    const int grid = glance::num_sms();
    char* ws = static_cast<char*>(workspace) + kCounterBytes;
    p.group = reinterpret_cast<int2*>(ws);
    p.part = reinterpret_cast<uint4*>(ws + wide_group_bytes(B, Hkv, p.n_qp));
    p.part_ml = reinterpret_cast<float2*>(p.part + wide_parts() * kBM * 16);
    e = glance::ensure_smem(reinterpret_cast<const void*>(kv4_attention_wide_kernel), kWideSmem);
    if (e != cudaSuccess) return glance::cuda_fail(e, who);
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kWideThreads);
    cfg.dynamicSmemBytes = kWideSmem;
    e = cudaLaunchKernelEx(&cfg, kv4_attention_wide_kernel, p);
    if (e != cudaSuccess) return glance::cuda_fail(e, who);
    cfg.gridDim = dim3(static_cast<unsigned>(B) * Hkv * p.n_qt * (kBM / kMergeRows));
    cfg.dynamicSmemBytes = 0;
    // blocks per group, where every group has as many
    const int parts = grid / (B * Hkv * p.n_qp);
    const int slices = parts > 10 ? 4 : parts > 5 ? 2 : 1;
    cfg.blockDim = dim3(128 * slices);
    e = cudaLaunchKernelEx(&cfg, slices == 4   ? kv4_attention_merge_kernel<4>
                                 : slices == 2 ? kv4_attention_merge_kernel<2>
                                               : kv4_attention_merge_kernel<1>, p);
  }
  if (e != cudaSuccess) return glance::cuda_fail(e, who);
  return GLANCE_OK;
}
