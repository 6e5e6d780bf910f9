// A token from each row of logits: temperature, top-k, min-p, top-p, and noise
// keyed by the predicted position (arXiv 2609.00355, Section 5.4: under sampling
// the committed token is a draw from the target's own verified row).
//
// With r = 1 / T and w_v = exp((l_v - max l) r), tokens in the order (logit
// descending, id ascending): those with w_v >= min_p among the first k, then the
// shortest prefix of these whose weights reach top_p of their sum. Every rule
// keeps a prefix of that order, so what is kept is given by its last token, as
// one 50-bit number: (order-preserving key of the logit, 2^18 - 1 - id), larger
// = earlier. The token is argmax l_v r + g_v over the kept ones, g_v the noise of
// the LM head's sampling mode: a draw from their renormalised softmax.
//
// Nothing is sorted. One pass finds the row's maximum, and the maxima of 2048
// disjoint parts of it. Then, whichever comes first:
// * k up to 1536: at least k tokens are no smaller than the k-th largest of the
//   parts' maxima, and seldom many more. They are gathered by one CTA, which keeps
//   them in registers, finds the last one that is kept and draws.
// * Else a histogram of (max - l) r in steps of 1/64 holds each bin's count, or
//   its count and weight. Where at most kList tokens lie in the bins up to the
//   border's, these are gathered as above. Where not, the tokens of the border's
//   bin are (divided by further histograms, over ranges of the 50-bit numbers,
//   until they fit the list, and) gathered, which gives the last token, and every
//   CTA draws from its part of the row.
// Within a bin weights are W (1 + y), |y| < 1/127, W a constant of the bin: the
// sum of the y is kept as an integer in 2^-21 units, so that it does not depend
// on the order of the additions and is good to 2^-22 of each weight. For top-p
// alone, tokens whose weights are so small that all of them together could not
// reach (1 - p) / 2 are summed without a bin. Weights below e^-31.9 of the largest
// are outside the histogram: 2^18 of them hold 4e-9 of the sum, under what an
// fp32 top_p can name.
//
// The draw's values are fp32 and compared in fp32 but for the foremost two and what
// comes near the second: these are evaluated again as sums of two floats, so that
// rounding decides next to nothing, and the gap, which may be small, is good to 1e-9.
// Most tokens need no logarithm: g >= t only if 1 - u <= e^-t, and once there are
// two values the noise's own bits decide.
//
// A row has one CTA, or a cluster of 4 or 16, by how many rows there are to fill
// the GPU; a second pass over it reads from L2. Every decision that a cluster's
// CTAs take by themselves is taken from values that all of them hold alike.
//
// Measured (V = 151936): one row, k 20, p 0.8, 7.8 us; 64 bf16 rows at p 0.95, most
// of which keep 10^4 to 10^5 tokens, 66 us (issue slots 58 %: a token has a bin, a
// comparison and a noise word); 512 fp32 rows with parameters of their own 139 to
// 146 us (2.1 to 2.2 TB/s; a cluster's steps one after the other, at two CTAs per
// SM). Clusters of 16, 4, 1 (timed by eager calls): one row 10.3, 12.7, 16.2 us; 64 rows
// 146, 68, 122; 512 rows 355, 149, 200. 4096 rows of 8191 bf16 at p 0.95: 251 us.
#include <cstring>
#include <mutex>

#include "noise.cuh"
#include "q8_internal.cuh"

GLANCE_DEFINE_STATUS_WORD(status_sample)

using namespace glance_dev;

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048, kCoarse = 64, kFine = kBins / kCoarse;
constexpr int kList = 2048;
constexpr int kPer = kList / kThreads;
constexpr int kGroups = 2048;             // parts of a row whose maxima are known
constexpr int kGroupK = kGroups * 3 / 4;  // so many of them are below the k-th, and the list will do
constexpr int kIdBits = 18;
constexpr int kMaxV = 1 << kIdBits;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kBinsPerNat = 64.f, kRange = 31.9f;  // of the histogram
constexpr int kUnitBits = 21;
// What a token adds to its bin: (1 + y) 2^21 less this, which is e^(-1/128) 2^21
// and a little less: at most 2^15 + 200 units, which 2^16 tokens leave within 32 bits.
constexpr uint32_t kUnitOff = 2080639u;

struct Params {
  const char* logits;
  long long stride;  // bytes
  const float* temperature;  // null: 1
  const int32_t* top_k;      // null, or <= 0: off
  const float* top_p;        // null, or >= 1: off
  const float* min_p;        // null, or <= 0: off
  const int32_t* position;
  const int32_t* seq;  // null: 0
  int32_t* tokens;
  float* gap;  // null: not written
  uint32_t k0, k1;
  int M, V, slice;  // slice: ids of a CTA, a multiple of 64
};

// Weights are added up as integers in units of 2^-40 (a row's largest weight is
// 1, its sum at most 2^18): exact, so that the order does not matter, and without
// the fp64 units, of which an SM has two.
typedef unsigned long long Mass;
constexpr int kMassBits = 40;

// e^-i/2 and e^-i/64 in units of 2^-63: a bin's W is the product of two.
struct Exps {
  Mass half[64], part[32];
};
constexpr double series_exp(double x) {  // |x| <= 1/2
  double term = 1, sum = 1;
  for (int i = 1; i < 20; ++i) {
    term *= x / i;
    sum += term;
  }
  return sum;
}
constexpr Exps make_exps() {
  Exps e = {};
  double h = 1;
  for (int i = 0; i < 64; ++i, h *= series_exp(-0.5)) e.half[i] = static_cast<Mass>(h * 9223372036854775808.0);
  for (int i = 0; i < 32; ++i) e.part[i] = static_cast<Mass>(series_exp(-i / 64.0) * 9223372036854775808.0);
  return e;
}
__constant__ Exps c_exps = make_exps();
// W of a bin in units of 2^-62.
__device__ __forceinline__ Mass weight_of_bin(int bin) { return __umul64hi(c_exps.half[bin >> 5], c_exps.part[bin & 31]); }
// W times a sum in units of 2^-21 (at most 2^40).
__device__ __forceinline__ Mass mass_of(Mass w, Mass sum) { return __umul64hi(w, sum << (64 + kMassBits - 62 - kUnitBits)); }
static_assert(kUnitBits + kIdBits + (64 + kMassBits - 62 - kUnitBits) < 64, "units");
// A share (in units of 2^-64) of a weight, at least one unit.
__device__ __forceinline__ Mass part_of(Mass all, Mass share) {
  const Mass m = __umul64hi(all, share);
  return m ? m : 1;
}

struct Border {  // the bin in which a prefix ends
  int bin;       // -1: the prefix has all
  uint32_t count_before, count_in;
  Mass mass_before, mass_all;
};
struct Entry {  // a token, its logit and its value in the draw
  float z, l;
  int id;
};
struct Cut {
  uint64_t number;  // the last token that is kept
  Mass mass;        // the weight up to it (of a search by weight)
};

template <int kCtas>
struct Shared {
  union {
    struct {
      uint32_t count[kBins], sum[kBins];  // (of 2^16 tokens at most: a CTA has no more)
    };
    struct {  // of a search in the list's tokens: a bin's weight in two parts
      uint32_t bin_count[kThreads], bin_low[kThreads], bin_high[kThreads];
    };
  };
  uint64_t mine[kCtas > 1 ? kList : 1];  // numbers of tokens on their way to the first CTA's list
  // written by the cluster's other CTAs
  uint64_t list[kList];
  float group[kGroups];
  Mass coarse_mass[kCtas][kCoarse + 1];  // [kCoarse]: of tokens without a bin
  uint32_t coarse_count[kCtas][kCoarse];
  Entry peer_best[2 * kCtas];
  uint64_t peer_lo[kCtas], peer_hi[kCtas];
  Cut cut;
  int found;
  uint32_t list_n[3];
  // this CTA's own
  uint32_t part_n, mine_n, mine_at;
  uint32_t second;  // key of a value that two of the draw's are no less than
  int part[kThreads];  // the threads whose tokens are looked at again
  Border border;
  Mass fine_mass[kCtas][kFine];
  uint32_t fine_count[kCtas][kFine];
  Mass warp_mass[kWarps];
  uint32_t warp_count[kWarps];
  float warp_f[kWarps], warp_second[kWarps];
  uint64_t warp_lo[kWarps], warp_hi[kWarps];
  Entry warp_best[2 * kWarps];
  float min_l;
};

// ------------------------------------------------- the cluster, if it is one

template <int kCtas>
__device__ __forceinline__ void sync_row() {
  __syncwarp();  // the cluster's barrier wants whole warps
  if (kCtas > 1)
    cluster_sync_all();
  else
    __syncthreads();
}
// To the same place in CTA `rank`.
template <int kCtas, typename X>
__device__ __forceinline__ void to_peer(X* local, int rank, const X& v) {
  if (kCtas == 1) {
    *local = v;
    return;
  }
  static_assert(sizeof(X) % 4 == 0, "words");
  const uint32_t at = dsmem_addr(local, rank);
  uint32_t w[sizeof(X) / 4];
  memcpy(w, &v, sizeof(X));
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(X) / 4); ++i)
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at + 4 * i), "r"(w[i]) : "memory");
}
template <int kCtas>
__device__ __forceinline__ uint32_t peer_u32(const uint32_t* local, int rank) {
  if (kCtas == 1) return *reinterpret_cast<const volatile uint32_t*>(local);
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(dsmem_addr(local, rank)) : "memory");
  return v;
}
template <int kCtas>
__device__ __forceinline__ uint32_t add_first(uint32_t* local, uint32_t v) {  // to the first CTA's counter
  if (kCtas == 1) return atomicAdd(local, v);
  uint32_t old;
  asm volatile("atom.relaxed.cluster.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(old) : "r"(dsmem_addr(local, 0)), "r"(v) : "memory");
  return old;
}

// -------------------------------------------------------------------- the row

__device__ __forceinline__ float of_key(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k); }
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// The row as this CTA sees it.
struct Row {
  const unsigned char* at;  // its part
  bool vec;                 // four logits from a multiple of four on are aligned
  float own;                // the largest logit of this thread's tokens
  float top, r;             // the row's largest; 1 / T
  float min_l;              // tokens below are not kept
  int rank, first, n;       // ids first .. first + n - 1
};

// A bf16 logit's key is its upper half: the lower says only the sign, and a search
// by numbers would go through its bits as well (64 rows of the nucleus case: 67.5
// us with the whole key, 66.0 without).
template <typename T>
constexpr int kShortBy = sizeof(T) == 4 ? 0 : 16;
template <typename T>
__device__ __forceinline__ uint64_t number_of(float l, int id) {
  return static_cast<uint64_t>(ord_key(l) >> kShortBy<T>) << kIdBits | static_cast<uint32_t>(kMaxV - 1 - id);
}
__device__ __forceinline__ int id_of(uint64_t number) { return kMaxV - 1 - static_cast<int>(number & (kMaxV - 1)); }
template <typename T>
__device__ __forceinline__ float logit_of(uint64_t number) {
  const uint32_t k = static_cast<uint32_t>(number >> kIdBits) << kShortBy<T>;
  return of_key(k & 0x80000000u ? k : k | ((1u << kShortBy<T>) - 1u));
}

// Four logits as they are stored.
template <typename T>
struct Four;
template <>
struct Four<float> {
  typedef float4 Raw;
  static __device__ __forceinline__ void unpack(const Raw& v, float (&l)[4]) { l[0] = v.x, l[1] = v.y, l[2] = v.z, l[3] = v.w; }
  static __device__ __forceinline__ Raw pack(const float (&l)[4]) { return make_float4(l[0], l[1], l[2], l[3]); }
};
template <>
struct Four<__nv_bfloat16> {
  typedef uint2 Raw;
  static __device__ __forceinline__ void unpack(const Raw& v, float (&l)[4]) {
    l[0] = __uint_as_float(v.x << 16), l[1] = __uint_as_float(v.x & 0xFFFF0000u);
    l[2] = __uint_as_float(v.y << 16), l[3] = __uint_as_float(v.y & 0xFFFF0000u);
  }
  static __device__ __forceinline__ Raw pack(const float (&l)[4]) { return make_uint2(pack_bf16x2(l[0], l[1]), pack_bf16x2(l[2], l[3])); }
};
// From place i (a multiple of four) of this CTA's tokens on; -infinity behind them.
template <typename T>
__device__ __forceinline__ typename Four<T>::Raw load4(const Row& w, int i) {
  const unsigned char* p = w.at + static_cast<size_t>(i) * sizeof(T);
  if (w.vec && i + 4 <= w.n) return *reinterpret_cast<const typename Four<T>::Raw*>(p);
  float l[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) l[j] = i + j < w.n ? static_cast<float>(reinterpret_cast<const T*>(p)[j]) : -INFINITY;
  return Four<T>::pack(l);
}
// Calls f(four logits, the first one's id) for this CTA's tokens, from a
// multiple of four on, with after() behind it for the warp's lanes together;
// kAhead loads of a thread are in flight. The loop is not unrolled: a thread goes
// through it ten to a hundred times, and the instructions of larger bodies took
// longer to arrive than to run. A thread with its largest logit below `least` is
// passed over.
template <typename T, typename F, typename G>
__device__ __forceinline__ void each4(const Row& w, float least, F f, G after) {
  typedef typename Four<T>::Raw Raw;
  constexpr int kAhead = 4;
  const bool mine = w.own >= least;
  if (!__any_sync(0xffffffffu, mine)) return;
  const int t = threadIdx.x, warp0 = 4 * (t & ~31);
  const float none[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
  Raw ahead[kAhead];
#pragma unroll
  for (int d = 0; d < kAhead; ++d) {
    ahead[d] = Four<T>::pack(none);
    if (mine && 4 * (t + d * kThreads) < w.n) ahead[d] = load4<T>(w, 4 * (t + d * kThreads));
  }
#pragma unroll 1
  for (int base = 0; base + warp0 < w.n; base += 4 * kThreads) {
    float l[4];
    Four<T>::unpack(ahead[0], l);
#pragma unroll
    for (int d = 0; d + 1 < kAhead; ++d) ahead[d] = ahead[d + 1];
    const int next = base + 4 * (t + kAhead * kThreads);
    ahead[kAhead - 1] = Four<T>::pack(none);
    if (mine && next < w.n) ahead[kAhead - 1] = load4<T>(w, next);
    f(l, w.first + base + 4 * t);
    __syncwarp();
    after();
  }
}
template <typename T, typename F>
__device__ __forceinline__ void each(const Row& w, float least, F f) {
  each4<T>(
      w, least,
      [&](const float(&l)[4], int id) {
#pragma unroll
        for (int j = 0; j < 4; ++j) f(l[j], id + j);
      },
      [] {});
}
// The same, for the few threads that have a token with l >= least (others may
// come too): a thread's tokens come from L2, so few threads' are shared out to all.
template <typename T, int kCtas, typename F>
__device__ __forceinline__ void each_of_few(Shared<kCtas>* s, const Row& w, float least, F f) {
  if (threadIdx.x == 0) s->part_n = 0;
  __syncthreads();
  if (w.own >= least) s->part[atomicAdd(&s->part_n, 1u)] = threadIdx.x;
  __syncthreads();
  const int parts = s->part_n, per = (w.n + 4 * kThreads - 1) / (4 * kThreads);  // groups of four of a thread
  if (parts > kThreads / 4) {
    each<T>(w, least, f);
    return;
  }
#pragma unroll 2
  for (int i = threadIdx.x; i < parts * per; i += kThreads) {
    const int at = 4 * (s->part[i / per] + kThreads * (i % per));
    if (at >= w.n) continue;
    float l[4];
    Four<T>::unpack(load4<T>(w, at), l);
#pragma unroll
    for (int j = 0; j < 4; ++j) f(l[j], w.first + at + j);
  }
}

// ------------------------------------------------------------- bins and sums

// A token's bin, the nearest multiple of 1/64 to (max - l) r, and e^(bin / 64 -
// (max - l) r) - 1. False: not kept, or too small for the histogram. The bin does
// not decrease as l falls.
__device__ __forceinline__ bool place(const Row& w, float l, int& bin, float& y) {
  const float x = __fmul_rn(w.top - l, w.r);
  if (!(x < kRange) || l < w.min_l) return false;
  const float n = fmaf(x, kBinsPerNat, 8388608.f);  // 2^23: rounds to a whole number in the low bits
  bin = static_cast<int>(__float_as_uint(n) & 0x7FFFFFu);
  const float d = fmaf(n - 8388608.f, 1.f / kBinsPerNat, -x);  // |d| <= 1/128
  y = d * fmaf(d, fmaf(d, fmaf(d, 1.f / 24, 1.f / 6), 0.5f), 1.f);  // to d^5 / 120 < 3e-13
  return true;
}
// Logits that no token of the bins up to `bin` is below, and none of the bins from
// it on above.
__device__ __forceinline__ float least_of_bin(const Row& w, int bin) {
  const float x = (static_cast<float>(bin) + 0.51f) / kBinsPerNat / w.r;
  return w.top - x - 1e-6f * (fabsf(w.top) + x);
}

__device__ __forceinline__ float most_of_bin(const Row& w, int bin) {
  const float x = (static_cast<float>(bin) - 0.51f) / kBinsPerNat / w.r;
  const float most = w.top - x + 1e-6f * (fabsf(w.top) + fabsf(x));
  return most == most ? most : INFINITY;  // (x beyond fp32's range: no bound)
}

template <int kCtas>
__device__ __forceinline__ void clear_hist(Shared<kCtas>* s) {
  uint4* h = reinterpret_cast<uint4*>(s->count);
  for (int i = threadIdx.x; i < 2 * kBins / 4; i += kThreads) h[i] = make_uint4(0, 0, 0, 0);
  __syncthreads();
}
template <int kCtas>
__device__ __forceinline__ void add_hist(Shared<kCtas>* s, int bin, float y, bool weigh) {
  atomicAdd(&s->count[bin], 1u);
  if (!weigh) return;
  // (1 + y) 2^21 rounded, from the low bits of a float, less the base
  const uint32_t f = (__float_as_uint(fmaf(y, 2097152.f, 2097152.f + 8388608.f)) & 0x7FFFFFu) - kUnitOff;
  atomicAdd(&s->sum[bin], f);
}

template <typename X>
__device__ __forceinline__ X scan_add(X v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const X u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}
// What the warps before this one have, of each warp's amount (weights: below 2^54).
__device__ __forceinline__ uint32_t sum_before(const uint32_t* of_warp, int lane, int warp) {
  return __reduce_add_sync(0xffffffffu, lane < warp ? of_warp[lane] : 0u);
}
__device__ __forceinline__ Mass sum_before(const Mass* of_warp, int lane, int warp) {
  const Mass v = lane < warp ? of_warp[lane] : 0ull;
  return (static_cast<Mass>(__reduce_add_sync(0xffffffffu, static_cast<uint32_t>(v >> 26))) << 26) +
         __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(v) & 0x3FFFFFFu);
}
__device__ __forceinline__ Mass sum_of(uint32_t count, uint32_t sum) { return static_cast<Mass>(count) * kUnitOff + sum; }

// The bin of the row's histogram in which the prefix of `want` tokens (want > 0)
// or else of `share` of the weight (of mass_all if given, else of what there is)
// ends; loose: the weight of this thread's tokens without a bin. fixed_bin >= 0:
// every bin's W is that bin's. count0, mass0: what lies before the histogram.
// Every CTA joins 64 sums of 32 bins of all of them, and looks at one of the 64
// more closely: the same in all of them.
template <int kCtas>
__device__ Border find_border(Shared<kCtas>* s, const Row& w, uint32_t want, Mass share, Mass mass_all, float loose, int fixed_bin,
                              uint32_t count0, Mass mass0) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, t = threadIdx.x;
  constexpr int kEach = kBins / kThreads, kJoin = kFine / kEach;  // bins of a thread, threads of a coarse bin
  __syncthreads();
  uint32_t count = 0;
  Mass mass = 0;
#pragma unroll
  for (int j = 0; j < kEach; ++j) {
    const int bin = t * kEach + j;
    const uint32_t c = s->count[bin];
    if (c) {
      count += c;
      mass += mass_of(weight_of_bin(fixed_bin >= 0 ? fixed_bin : bin), sum_of(c, s->sum[bin]));
    }
  }
#pragma unroll
  for (int o = 1; o < kJoin; o <<= 1) {
    count += __shfl_xor_sync(0xffffffffu, count, o);
    mass += __shfl_xor_sync(0xffffffffu, mass, o);
  }
  Mass extra = __float2ull_rn(loose * 1099511627776.f);
#pragma unroll
  for (int o = 16; o; o >>= 1) extra += __shfl_xor_sync(0xffffffffu, extra, o);
  if (lane == 0) s->warp_mass[warp] = extra;
  for (int q = t % kJoin; q < kCtas; q += kJoin) {
    to_peer<kCtas>(&s->coarse_count[w.rank][t / kJoin], q, count);
    to_peer<kCtas>(&s->coarse_mass[w.rank][t / kJoin], q, mass);
  }
  __syncthreads();
  if (t < kCtas) {
    Mass all = 0;
    for (int i = 0; i < kWarps; ++i) all += s->warp_mass[i];
    to_peer<kCtas>(&s->coarse_mass[w.rank][kCoarse], t, all);
  }
  if (t == 0) s->border.bin = -1;
  sync_row<kCtas>();
  uint32_t count_to = 0;
  Mass mass_to = 0;
  count = 0;
  mass = 0;
  if (t < kCoarse) {
#pragma unroll
    for (int q = 0; q < kCtas; ++q) {
      count += s->coarse_count[q][t];
      mass += s->coarse_mass[q][t];
    }
    count_to = scan_add(count, lane);
    mass_to = scan_add(mass, lane);
    if (lane == 31) {
      s->warp_count[warp] = count_to;
      s->warp_mass[warp] = mass_to;
    }
  }
  __syncthreads();
  Mass all = mass0 + s->warp_mass[0] + s->warp_mass[1];
  for (int q = 0; q < kCtas; ++q) all += s->coarse_mass[q][kCoarse];
  if (mass_all == 0) mass_all = all;
  const Mass target = part_of(mass_all, share);
  if (t < kCoarse) {
    const uint32_t before = count0 + (warp ? s->warp_count[0] : 0u) + count_to - count;
    const Mass before_mass = mass0 + (warp ? s->warp_mass[0] : 0ull) + mass_to - mass;
    if (count && (want ? before < want && before + count >= want : before_mass < target && before_mass + mass >= target)) {
      s->border.bin = t;
      s->border.count_before = before;
      s->border.mass_before = before_mass;
    }
  }
  __syncthreads();
  Border b = s->border;
  b.mass_all = mass_all;
  if (b.bin < 0) return b;
  for (int q = warp; q < kCtas; q += kWarps) {
    const int bin = b.bin * kFine + lane;
    const uint32_t c = peer_u32<kCtas>(&s->count[bin], q), sum = peer_u32<kCtas>(&s->sum[bin], q);
    s->fine_count[q][lane] = c;
    s->fine_mass[q][lane] = c ? mass_of(weight_of_bin(fixed_bin >= 0 ? fixed_bin : bin), sum_of(c, sum)) : 0;
  }
  __syncthreads();
  if (warp == 0) {
    count = 0;
    mass = 0;
    for (int q = 0; q < kCtas; ++q) {
      count += s->fine_count[q][lane];
      mass += s->fine_mass[q][lane];
    }
    const uint32_t before = b.count_before + scan_add(count, lane) - count;
    const Mass before_mass = b.mass_before + scan_add(mass, lane) - mass;
    // the bins were rounded one by one in either place: the sums agree
    const unsigned here = __ballot_sync(0xffffffffu, count && (want ? before < want && before + count >= want
                                                                    : before_mass < target && before_mass + mass >= target));
    if (here && lane == __ffs(here) - 1) s->border = Border{b.bin * kFine + lane, before, count, before_mass, mass_all};
  }
  __syncthreads();
  b = s->border;
  b.mass_all = mass_all;
  return b;
}

// A warp's numbers in descending order.
__device__ __forceinline__ uint64_t sort_warp(uint64_t v, int lane) {
#pragma unroll
  for (int k = 2; k <= 32; k <<= 1)
#pragma unroll
    for (int j = k >> 1; j; j >>= 1) {
      const uint64_t u = __shfl_xor_sync(0xffffffffu, v, j);
      v = (v > u) == (((lane & j) == 0) == ((lane & k) == 0)) ? v : u;
    }
  return v;
}

// A token's weight, to 2^-42 of its bin's.
__device__ __forceinline__ Mass weight_of(const Row& w, float l) {
  int bin;
  float y;
  return place(w, l, bin, y) ? __umul64hi(weight_of_bin(bin), (1ull << 42) + __float2ll_rn(y * 4398046511104.f)) : 0ull;
}
// The list's tokens, kPer to a thread; 0: none.
struct Held {
  uint64_t number[kPer];
  Mass mass[kPer];
};
template <typename T, int kCtas>
__device__ __forceinline__ Held hold_list(Shared<kCtas>* s, const Row& w, int n, bool weigh) {
  Held h;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int e = static_cast<int>(threadIdx.x) + j * kThreads;
    h.number[j] = e < n ? s->list[e] : 0ull;
    h.mass[j] = weigh && e < n ? weight_of(w, logit_of<T>(h.number[j])) : 0ull;
  }
  return h;
}

// The token of those held at which a prefix of `want` of them (want > 0), or of
// the weight `target`, ends, where `mass0` lies before them: by one CTA, 512 bins
// of the numbers' range at a time. The last one if there is none.
template <int kCtas>
__device__ Cut select_held(Shared<kCtas>* s, const Held& h, uint32_t want, Mass target, Mass mass0) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, t = threadIdx.x;
  uint64_t lo = ~0ull, hi = 0;
#pragma unroll
  for (int j = 0; j < kPer; ++j)
    if (h.number[j]) {
      lo = h.number[j] < lo ? h.number[j] : lo;
      hi = h.number[j] > hi ? h.number[j] : hi;
    }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const uint64_t a = __shfl_xor_sync(0xffffffffu, lo, o), c = __shfl_xor_sync(0xffffffffu, hi, o);
    lo = a < lo ? a : lo;
    hi = c > hi ? c : hi;
  }
  if (lane == 0) {
    s->warp_lo[warp] = lo;
    s->warp_hi[warp] = hi;
  }
  __syncthreads();
  for (int i = 0; i < kWarps; ++i) {
    lo = s->warp_lo[i] < lo ? s->warp_lo[i] : lo;
    hi = s->warp_hi[i] > hi ? s->warp_hi[i] : hi;
  }
  const uint64_t least = lo;
  uint32_t count0 = 0;
  int shift = max(0, 64 - __clzll(hi - lo) - 9);
  for (int level = 0; level < 8; ++level) {
    s->bin_count[t] = s->bin_low[t] = s->bin_high[t] = 0;
    if (t == 0) s->found = -1;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      if (h.number[j] >= lo && h.number[j] <= hi) {
        const int bin = static_cast<int>((hi - h.number[j]) >> shift);
        atomicAdd(&s->bin_count[bin], 1u);
        if (!want) {  // (a token's weight is 2^40 at most, and there are 2^11)
          atomicAdd(&s->bin_low[bin], static_cast<uint32_t>(h.mass[j]) & 0xFFFFFu);
          atomicAdd(&s->bin_high[bin], static_cast<uint32_t>(h.mass[j] >> 20));
        }
      }
    __syncthreads();
    const uint32_t count = s->bin_count[t];
    const Mass mass = (static_cast<Mass>(s->bin_high[t]) << 20) + s->bin_low[t];
    const uint32_t count_to = scan_add(count, lane);
    const Mass mass_to = scan_add(mass, lane);
    if (lane == 31) {
      s->warp_count[warp] = count_to;
      s->warp_mass[warp] = mass_to;
    }
    __syncthreads();
    const uint32_t before = count0 + count_to - count + sum_before(s->warp_count, lane, warp);
    const Mass before_mass = mass0 + mass_to - mass + (want ? 0 : sum_before(s->warp_mass, lane, warp));
    if (count && (want ? before < want && before + count >= want : before_mass < target && before_mass + mass >= target)) {
      s->found = t;
      s->border.count_before = before;
      s->border.count_in = count;
      s->border.mass_before = before_mass;
    }
    __syncthreads();
    const int bin = s->found;
    if (bin < 0) return Cut{least, target};
    count0 = s->border.count_before;
    mass0 = s->border.mass_before;
    hi -= static_cast<uint64_t>(bin) << shift;
    const uint64_t last = hi - ((1ull << shift) - 1);
    lo = last > lo ? last : lo;
    if (s->border.count_in == 1) break;  // numbers differ: at shift 0 at the latest
    shift = max(0, shift - 9);
    __syncthreads();
  }
#pragma unroll
  for (int j = 0; j < kPer; ++j)
    if (h.number[j] >= lo && h.number[j] <= hi) s->cut = Cut{h.number[j], mass0 + h.mass[j]};
  __syncthreads();
  return s->cut;
}

// Gathers the numbers of the tokens with least <= l <= most that pass f in the
// first CTA's list and returns how many there were (kList fit). Every CTA collects
// its own first: one trip to the other CTA for all.
template <typename T, int kCtas, typename F>
__device__ uint32_t gather(Shared<kCtas>* s, const Row& w, int turn, float least, float most, F f) {
  const int t = threadIdx.x;
  if (t == 0) s->mine_n = 0;
  uint32_t* n = kCtas == 1 ? &s->list_n[turn] : &s->mine_n;
  uint64_t* to = kCtas == 1 ? s->list : s->mine;
  each_of_few<T, kCtas>(s, w, least, [&](float l, int id) {
    if (l >= least && l <= most) {
      if (f(l, id)) {
        const uint32_t at = atomicAdd(n, 1u);
        if (at < kList) to[at] = number_of<T>(l, id);
      }
    }
  });
  if (kCtas > 1) {
    __syncthreads();
    const uint32_t mine = s->mine_n;
    if (t == 0 && mine) s->mine_at = add_first<kCtas>(&s->list_n[turn], mine);
    __syncthreads();
    const uint32_t at = s->mine_at;
    for (uint32_t i = t; i < mine && i < kList && at + i < kList; i += kThreads) to_peer<kCtas>(&s->list[at + i], 0, s->mine[i]);
  }
  sync_row<kCtas>();
  return peer_u32<kCtas>(&s->list_n[turn], 0);
}

// ------------------------------------------------------------------- the draw

__device__ __forceinline__ bool ahead(float z, int id, float z0, int id0) { return z > z0 || (z == z0 && id < id0); }
constexpr int kNoId = 0x7FFFFFFF;
__device__ __forceinline__ Entry no_entry() { return Entry{-INFINITY, 0.f, kNoId}; }
// The foremost of a warp's entries, and whose it is.
__device__ __forceinline__ Entry warp_first(const Entry& e, int& lane) {
  const uint32_t key = ord_key(e.z), most = __reduce_max_sync(0xffffffffu, key);
  const uint32_t id = __reduce_min_sync(0xffffffffu, key == most ? static_cast<uint32_t>(e.id) : ~0u);
  lane = __ffs(__ballot_sync(0xffffffffu, key == most && static_cast<uint32_t>(e.id) == id)) - 1;
  return Entry{__shfl_sync(0xffffffffu, e.z, lane), __shfl_sync(0xffffffffu, e.l, lane), static_cast<int>(id)};
}

// The two best values that a thread has seen, with their tokens.
struct Two {
  Entry e[2];
};
__device__ __forceinline__ Two no_two() { return Two{{no_entry(), no_entry()}}; }
__device__ __forceinline__ void fold(Two& t, float z, float l, int id) {
  if (ahead(z, id, t.e[0].z, t.e[0].id)) {
    t.e[1] = t.e[0];
    t.e[0] = Entry{z, l, id};
  } else if (ahead(z, id, t.e[1].z, t.e[1].id)) {
    t.e[1] = Entry{z, l, id};
  }
}
// A warp's two best of its threads' two best.
__device__ __forceinline__ Two warp_two(const Two& t) {
  int lane;
  Two b;
  b.e[0] = warp_first(t.e[0], lane);
  b.e[1] = warp_first((threadIdx.x & 31) == static_cast<unsigned>(lane) ? t.e[1] : t.e[0], lane);
  return b;
}
__device__ __forceinline__ uint32_t word_of(const uint4& v, int j) { return j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w; }

struct Key {  // of the row's noise
  uint32_t pos, seq, k0, k1;
};
__device__ __forceinline__ uint4 noise4(const Key& k, int id) {
  return philox4x32_10(make_uint4(static_cast<uint32_t>(id) / 4, k.pos, k.seq, 0u), k.k0, k.k1);
}
// A number as the sum of two floats, the second at most half a step of the first
// (arithmetic on such pairs after Dekker, 1971, and Knuth): 48 bits without the
// fp64 units, whose chains of a few dozen operations took 2.4 us of a call with
// one row.
struct Pair {
  float h, l;
};
__device__ __forceinline__ Pair sum_of_two(float a, float b) {
  const float s = a + b, t = s - a;
  return Pair{s, (a - (s - t)) + (b - t)};
}
// ln a of a normal a > 0 to 1e-10: a = 2^e m, m in [sqrt 1/2, sqrt 2), ln m = 2
// artanh s with s = (m - 1) / (m + 1); s and s^3 / 3 as pairs, the terms from s^5
// on (below 4e-5) in fp32.
__device__ __forceinline__ Pair ln_of(float a) {
  const uint32_t bits = __float_as_uint(a);
  const int e = (static_cast<int>(bits) - 0x3F3504F3) >> 23;
  const float m = __uint_as_float(bits - (static_cast<uint32_t>(e) << 23));
  const float num = m - 1.f, den = m + 1.f, den_low = m - (den - 1.f);  // num and den + den_low are exact
  const float q = __fdiv_rn(num, den), low = __fdividef(fmaf(-q, den_low, fmaf(-q, den, num)), den);
  const float q2 = __fmul_rn(q, q), q2_low = fmaf(q, q, -q2), cube = __fmul_rn(q2, q), cube_low = fmaf(q2_low, q, fmaf(q2, q, -cube));
  constexpr float kThird = 1.f / 3, kThirdLow = -9.934107e-9f;
  const float third = __fmul_rn(cube, kThird), third_low = fmaf(cube_low, kThird, fmaf(cube, kThirdLow, fmaf(cube, kThird, -third)));
  const float tail = cube * q2 * fmaf(q2, fmaf(q2, fmaf(q2, fmaf(q2, 1.f / 13, 1.f / 11), 1.f / 9), 1.f / 7), 0.2f);
  // ln 2 as 0.693145751953125, which e times is exact, and the rest
  const Pair x = sum_of_two(static_cast<float>(e) * 0.693145751953125f, 2.f * q), y = sum_of_two(x.h, 2.f * third);
  const float rest = 2.f * (fmaf(q2, low, low) + (third_low + tail)) + static_cast<float>(e) * 1.42860682e-6f;
  return sum_of_two(y.h, y.l + (x.l + rest));
}
// The draw's value of a token, to 1e-9.
__device__ __noinline__ Pair value_pair(const Row& w, const Key& k, float l, int id) {
  const uint32_t word = word_of(noise4(k, id), id & 3);
  const Pair y = ln_of((static_cast<float>(word >> 9) + 0.5f) * (1.f / 8388608.f)), ln_y = ln_of(-y.h);  // ln u < 0
  const Pair d = sum_of_two(l, -w.top);
  const float x = __fmul_rn(d.h, w.r);
  const Pair z = sum_of_two(x, -ln_y.h);
  return sum_of_two(z.h, z.l + (fmaf(d.l, w.r, fmaf(d.h, w.r, -x)) - (ln_y.l + __fdividef(y.l, y.h))));
}
// Pairs by their bits: larger is larger.
__device__ __forceinline__ uint64_t key_of(const Pair& z) { return static_cast<uint64_t>(ord_key(z.h)) << 32 | ord_key(z.l); }

// The row's token, by a warp that holds the entries that it can be: the two best
// and what comes within the rounding of the second (fp32's and the noise's) are
// evaluated again as pairs, which decides between them and gives the gap.
__device__ void decide(const Params& p, const Row& w, const Key& key, const Entry& e, bool exact, int row) {
  const int lane = threadIdx.x & 31;
  int at, next;
  const Entry a = warp_first(e, at), b = warp_first(lane == at ? no_entry() : e, next);
  int id = a.id;
  float gap = a.z - b.z;
  if (!exact && b.z > -INFINITY) {
    const bool near = e.z >= b.z - (2e-5f + 1e-6f * fabsf(b.z));
    const uint64_t z = near ? key_of(value_pair(w, key, e.l, e.id)) : 0ull;
    __syncwarp();
    uint64_t best = z;
    id = near ? e.id : kNoId;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      const uint64_t u = __shfl_xor_sync(0xffffffffu, best, o);
      const int i = __shfl_xor_sync(0xffffffffu, id, o);
      if (u > best || (u == best && i < id)) best = u, id = i;
    }
    uint64_t second = e.id == id ? 0ull : z;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      const uint64_t u = __shfl_xor_sync(0xffffffffu, second, o);
      second = u > second ? u : second;
    }
    gap = (of_key(static_cast<uint32_t>(best >> 32)) - of_key(static_cast<uint32_t>(second >> 32))) +
          (of_key(static_cast<uint32_t>(best)) - of_key(static_cast<uint32_t>(second)));
  }
  if (lane == 0 && GLANCE_IN_BOUNDS(row, p.M)) {
    p.tokens[row] = id;
    if (p.gap) p.gap[row] = gap;
  }
}

// From the threads' two best values to the row's token. alone: the first CTA's
// threads have all that counts.
template <int kCtas>
__device__ void finish(Shared<kCtas>* s, const Params& p, const Row& w, const Key& key, const Two& t, bool exact, bool alone, int row) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __syncwarp();
  Two b = warp_two(t);
  if (lane < 2) s->warp_best[2 * warp + lane] = lane ? b.e[1] : b.e[0];
  __syncthreads();
  if (kCtas == 1 || alone) {
    if (warp == 0) decide(p, w, key, s->warp_best[lane], exact, row);
    return;
  }
  if (warp == 0) {
    b = warp_two(Two{{s->warp_best[lane], no_entry()}});
    if (lane < 2) to_peer<kCtas>(&s->peer_best[2 * w.rank + lane], 0, lane ? b.e[1] : b.e[0]);
  }
  sync_row<kCtas>();
  if (w.rank == 0 && warp == 0) decide(p, w, key, lane < 2 * kCtas ? s->peer_best[lane] : no_entry(), exact, row);
}
static_assert(2 * kWarps == 32, "a block's entries are a warp's");

// The first CTA draws from its list of n tokens: the first `want` of them (0:
// all), of these `share` of the weight (of mass_all, or of theirs if it is 0).
template <typename T, int kCtas>
__device__ void draw_from_list(Shared<kCtas>* s, const Params& p, const Row& w, const Key& key, int n, uint32_t want, bool all_p, Mass share,
                               Mass mass_all, int row) {
  const int t = threadIdx.x;
  const int kept = want ? min(static_cast<int>(want), n) : n;
  Two two = no_two();
  const auto draw = [&](uint64_t number) {
    const int id = id_of(number);
    const float l = logit_of<T>(number);
    fold(two, (l - w.top) * w.r + gumbel_of(word_of(noise4(key, id), id & 3)), l, id);
  };
  if (n <= 32) {  // one warp's
    if (t >= 32) return;
    const uint64_t number = sort_warp(t < n ? s->list[t] : 0ull, t);
    const Mass m = !all_p && t < kept ? weight_of(w, logit_of<T>(number)) : 0ull;
    const Mass upto = scan_add(m, t), all = mass_all ? mass_all : __shfl_sync(0xffffffffu, upto, 31);
    if (t < kept && (all_p || upto - m < part_of(all, share))) draw(number);
    __syncwarp();
    decide(p, w, key, two.e[0], false, row);
    return;
  }
  Held h = hold_list<T, kCtas>(s, w, n, !all_p);
  uint64_t cut = 1;
  if (kept < n) {
    cut = select_held(s, h, want, 0, 0).number;
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      if (h.number[j] < cut) h.number[j] = 0;
  }
  if (!all_p) {
    if (mass_all == 0) {
      Mass sum = 0;
#pragma unroll
      for (int j = 0; j < kPer; ++j) sum += h.number[j] ? h.mass[j] : 0ull;
#pragma unroll
      for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      __syncthreads();
      if ((t & 31) == 0) s->warp_mass[t >> 5] = sum;
      __syncthreads();
      for (int i = 0; i < kWarps; ++i) mass_all += s->warp_mass[i];
      __syncthreads();
    }
    cut = select_held(s, h, 0u, part_of(mass_all, share), 0).number;
  }
#pragma unroll
  for (int j = 0; j < kPer; ++j)
    if (h.number[j] >= cut) draw(h.number[j]);
  finish(s, p, w, key, two, false, true, row);
}

// The last token that a prefix keeps, and the weight up to it: the tokens of the
// border's bin (from `floor` on) are divided until they fit the list, and that is
// sorted. turn: which of the list's counters.
template <typename T, int kCtas>
__device__ Cut refine(Shared<kCtas>* s, const Row& w, const Border& first, uint64_t floor, uint32_t want, Mass share, int turn) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, t = threadIdx.x;
  Border b = first;
  const int bin = b.bin;
  const Mass all = b.mass_all;
  uint64_t lo = floor, hi = ~0ull;
  const float least = least_of_bin(w, bin), most = most_of_bin(w, bin);
  // the numbers differ and the range shrinks to the tokens' own each time: 50
  // bits are through after five divisions by 2^10 or more
  for (int level = 0; level < 8 && b.count_in > kList; ++level) {
    uint64_t least_n = ~0ull, most_n = 0;
    each<T>(w, least, [&](float l, int id) {
      int at;
      float y;
      if (l >= least && l <= most && place(w, l, at, y) && at == bin) {
        const uint64_t number = number_of<T>(l, id);
        if (number >= lo && number <= hi) {
          least_n = number < least_n ? number : least_n;
          most_n = number > most_n ? number : most_n;
        }
      }
    });
    __syncwarp();
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      const uint64_t a = __shfl_xor_sync(0xffffffffu, least_n, o), c = __shfl_xor_sync(0xffffffffu, most_n, o);
      least_n = a < least_n ? a : least_n;
      most_n = c > most_n ? c : most_n;
    }
    if (lane == 0) {
      s->warp_lo[warp] = least_n;
      s->warp_hi[warp] = most_n;
    }
    __syncthreads();
    for (int i = 0; i < kWarps; ++i) {
      least_n = s->warp_lo[i] < least_n ? s->warp_lo[i] : least_n;
      most_n = s->warp_hi[i] > most_n ? s->warp_hi[i] : most_n;
    }
    if (t < kCtas) {
      to_peer<kCtas>(&s->peer_lo[w.rank], t, least_n);
      to_peer<kCtas>(&s->peer_hi[w.rank], t, most_n);
    }
    sync_row<kCtas>();  // also: the others have read this CTA's histogram
    clear_hist(s);
    lo = s->peer_lo[0];
    hi = s->peer_hi[0];
    for (int q = 1; q < kCtas; ++q) {
      lo = s->peer_lo[q] < lo ? s->peer_lo[q] : lo;
      hi = s->peer_hi[q] > hi ? s->peer_hi[q] : hi;
    }
    const int shift = max(0, 64 - __clzll(hi - lo) - 11);  // the range in 2048 steps at most
    each<T>(w, least, [&](float l, int id) {
      int at;
      float y;
      if (l >= least && l <= most && place(w, l, at, y) && at == bin) {
        const uint64_t number = number_of<T>(l, id);
        if (number >= lo && number <= hi) add_hist(s, static_cast<int>((hi - number) >> shift), y, !want);
      }
    });
    b = find_border(s, w, want, share, all, 0.f, bin, b.count_before, b.mass_before);
    // the sum of the weights came out a rounding short of its share: the range's last token
    if (b.bin < 0) return Cut{lo, all};
    hi -= static_cast<uint64_t>(b.bin) << shift;
    const uint64_t last = hi - ((1ull << shift) - 1);
    lo = last > lo ? last : lo;
  }
  const uint32_t found = gather<T, kCtas>(s, w, turn, least, most, [&](float l, int id) {
    int at;
    float y;
    const uint64_t number = number_of<T>(l, id);
    return number >= lo && number <= hi && place(w, l, at, y) && at == bin;
  });
  if (w.rank == 0) {
    const int n = min(found, static_cast<uint32_t>(kList));
    const Held h = hold_list<T, kCtas>(s, w, n, !want);
    const Cut c = select_held(s, h, want ? want - b.count_before : 0u, part_of(all, share), b.mass_before);
    if (t < kCtas) to_peer<kCtas>(&s->cut, t, c);
  }
  sync_row<kCtas>();
  return s->cut;
}

// ------------------------------------------------------------------ the kernel

// Grid: x = row * kCtas + rank.
template <typename T, int kCtas>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const Params p) {
  extern __shared__ __align__(16) unsigned char smem[];
  Shared<kCtas>* s = reinterpret_cast<Shared<kCtas>*>(smem);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, t = threadIdx.x;
  const int row = static_cast<int>(blockIdx.x) / kCtas;
  Row w;
  w.rank = kCtas > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  w.first = w.rank * p.slice;
  w.n = max(0, min(p.slice, p.V - w.first));
  if (kCtas > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  pdl_wait_prior();
  pdl_launch_dependents();
  const float temperature = p.temperature ? __ldg(p.temperature + row) : 1.f;
  const int k = p.top_k ? __ldg(p.top_k + row) : 0;
  const float top_p = p.top_p ? __ldg(p.top_p + row) : 1.f, min_p = p.min_p ? __ldg(p.min_p + row) : 0.f;
  const Key key = {static_cast<uint32_t>(__ldg(p.position + row)), p.seq ? static_cast<uint32_t>(__ldg(p.seq + row)) : 0u, p.k0, p.k1};
  const bool greedy = temperature == 0.f;
  w.r = greedy ? 1.f : 1.f / temperature;
  if (t < 3) s->list_n[t] = 0;
  const unsigned char* src =
      reinterpret_cast<const unsigned char*>(p.logits) + row * p.stride + static_cast<long long>(w.first) * static_cast<int>(sizeof(T));
  w.vec = reinterpret_cast<uintptr_t>(src) % (4 * sizeof(T)) == 0;
  w.at = src;
  // the maxima of four parts of this thread's tokens; with more CTAs it is
  // kCtas / 4 threads' that are one part
  float group[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
  constexpr int kBatch = sizeof(T) == 4 ? 4 : 8;
  for (int base = 4 * t; base < w.n; base += 4 * kThreads * kBatch) {
    typename Four<T>::Raw raw[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      if (base + u * 4 * kThreads < w.n) raw[u] = load4<T>(w, base + u * 4 * kThreads);
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      if (base + u * 4 * kThreads < w.n) {
        float l[4];
        Four<T>::unpack(raw[u], l);
        group[u & 3] = max_nan(group[u & 3], max_nan(max_nan(l[0], l[1]), max_nan(l[2], l[3])));
      }
  }
  __syncwarp();
  w.own = max_nan(max_nan(group[0], group[1]), max_nan(group[2], group[3]));
  if (kCtas > 1) {
    float part = w.own;
#pragma unroll
    for (int o = 1; o < kCtas / 4; o <<= 1) part = max_nan(part, __shfl_xor_sync(0xffffffffu, part, o));
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // all have begun
    constexpr int kOne = kCtas >= 4 ? kCtas / 4 : 1;  // threads of a part
#pragma unroll
    for (int j = 0; j < 4; ++j) to_peer<kCtas>(&s->group[(w.rank * kThreads + t) / kOne], t % kOne * 4 + j, part);
  }
  sync_row<kCtas>();
  if (kCtas > 1) {
#pragma unroll
    for (int j = 0; j < 4; ++j) group[j] = s->group[t + j * kThreads];
  }
  float top = max_nan(max_nan(group[0], group[1]), max_nan(group[2], group[3]));
#pragma unroll
  for (int o = 16; o; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (lane == 0) s->warp_f[warp] = top;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kWarps; ++i) top = max_nan(top, s->warp_f[i]);
  w.top = top;
  const bool bad_row = !(top > -INFINITY && top < INFINITY);
  const bool bad_param = !(temperature >= 0.f && w.r < INFINITY && w.r > 0.f) || top_p != top_p || min_p != min_p;
  if (bad_row || bad_param) {
    if (t == 0 && w.rank == 0 && GLANCE_IN_BOUNDS(row, p.M)) {
      p.tokens[row] = -1;
      if (p.gap) p.gap[row] = NAN;
      report(bad_row ? GLANCE_DEV_NONFINITE_LOGITS : GLANCE_DEV_BAD_SAMPLING);
    }
    return;
  }
  // the least logit with (l - top) r >= ln min_p: near it in fp32, then by the
  // comparison in fp64
  w.min_l = -INFINITY;
  if (min_p > 0.f && !greedy) {
    if (t == 0) {
      const Pair ln = ln_of(fminf(fmaxf(min_p, 1.17549435e-38f), 1.f));
      const double lg = static_cast<double>(ln.h) + static_cast<double>(ln.l), r = w.r, m = top;
      float x = fminf(fmaf(ln.h, temperature, top), top);
      for (int i = 0; i < 8 && x > -INFINITY && (static_cast<double>(x) - m) * r >= lg; ++i) x = nextafterf(x, -INFINITY);
      for (int i = 0; i < 16 && x < top && (static_cast<double>(x) - m) * r < lg; ++i) x = nextafterf(x, INFINITY);
      s->min_l = x;
    }
    __syncthreads();
    w.min_l = s->min_l;
  }
  const uint32_t want = k > 0 && k < p.V ? k : 0u;
  // top_p in units of 2^-64 (all_p: off)
  const bool all_p = !(top_p < 1.f);
  const Mass share = all_p ? 0 : __float2ull_rz(fmaxf(top_p, 0.f) * 0x1p32f * 0x1p32f);
  uint64_t cut = 0;
  if (!greedy && (want || !all_p)) {
    uint32_t upto = ~0u;
    Border b = {};
    b.bin = -1;
    if (want && want <= kGroupK) {
      // k of the maxima, tokens all, are at or above the upper one of 512 steps of
      // the histogram's range that the k-th is in
      s->part[t] = 0;  // (not the histogram's place: another CTA may write to the list there)
      if (t == 0) s->found = -1;
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float x = __fmul_rn(top - group[j], w.r);
        if (x < kRange) atomicAdd(&s->part[static_cast<int>(x * (kThreads / 32.f))], 1);
      }
      __syncthreads();
      const uint32_t count = s->part[t], count_to = scan_add(count, lane);
      if (lane == 31) s->warp_count[warp] = count_to;
      __syncthreads();
      const uint32_t before = count_to - count + sum_before(s->warp_count, lane, warp);
      if (before < want && before + count >= want) s->found = t;
      __syncthreads();
      const float x = (static_cast<float>(s->found) + 1.01f) * (32.f / kThreads) / w.r;
      const float lo = s->found < 0 ? -INFINITY : top - x - 1e-6f * (fabsf(top) + x);
      const float least = fmaxf(lo, w.min_l);
      upto = gather<T, kCtas>(s, w, 0, least, INFINITY, [&](float l, int) { return __fmul_rn(w.top - l, w.r) < kRange; });
    }
    if (upto > kList) {
      // Tokens with (max - l) r above `skip` need no bin: all of them together
      // weigh less than (1 - p) / 2, and the border is not among them.
      const float skip = want ? kRange : fminf(kRange, logf(2.f * p.V / (1.f - fmaxf(top_p, 0.f))));
      float loose = 0.f;
      clear_hist(s);
      each<T>(w, w.min_l, [&](float l, int) {
        const float x = __fmul_rn(w.top - l, w.r);
        if (x < skip) {
          int bin;
          float y;
          if (place(w, l, bin, y)) add_hist(s, bin, y, !want);
        } else if (!want && l >= w.min_l) {
          loose += ex2_approx(-kLog2e * x);
        }
      });
      b = find_border(s, w, want, share, 0, loose, -1, 0u, 0);
      upto = ~0u;
      if (b.bin >= 0 && b.count_before + b.count_in <= kList) {
        upto = gather<T, kCtas>(s, w, 1, least_of_bin(w, b.bin), INFINITY, [&](float l, int) {
          int bin;
          float y;
          return __fmul_rn(w.top - l, w.r) < skip && place(w, l, bin, y) && bin <= b.bin;
        });
      }
    }
    if (upto <= kList) {
      // all that may be kept is in the first CTA's list
      __syncwarp();
      if (kCtas > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
      if (w.rank == 0) {
        draw_from_list<T, kCtas>(s, p, w, key, static_cast<int>(upto), want, all_p, share, want ? 0 : b.mass_all, row);
        // the others have read its counter
        __syncwarp();
        if (kCtas > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
      }
      return;
    }
    if (b.bin >= 0) {
      cut = refine<T, kCtas>(s, w, b, 0, want, share, 1).number;
      if (want && !all_p) {
        // the first k are known: the share of their weight ends at or before their last
        clear_hist(s);
        each<T>(w, logit_of<T>(cut), [&](float l, int id) {
          int bin;
          float y;
          if (place(w, l, bin, y) && number_of<T>(l, id) >= cut) add_hist(s, bin, y, true);
        });
        b = find_border(s, w, 0u, share, 0, 0.f, -1, 0u, 0);
        if (b.bin >= 0) {
          const Cut c = refine<T, kCtas>(s, w, b, cut, 0u, share, 2);
          if (c.number > cut) cut = c.number;
        }
      }
    } else if (want && !all_p) {
      // fewer than k tokens in reach: the share is of all of them
      sync_row<kCtas>();  // the others have read the sums of the search before
      clear_hist(s);
      each<T>(w, w.min_l, [&](float l, int) {
        int bin;
        float y;
        if (place(w, l, bin, y)) add_hist(s, bin, y, true);
      });
      b = find_border(s, w, 0u, share, 0, 0.f, -1, 0u, 0);
      if (b.bin >= 0) cut = refine<T, kCtas>(s, w, b, 0, 0u, share, 2).number;
    }
  }
  // every CTA looks at its part of the row
  Two two = no_two();
  if (greedy) {
    // two tokens are no smaller than the second largest of the parts' maxima
    float second = -INFINITY;
    int tops = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      tops += group[j] == top;
      if (group[j] != top) second = fmaxf(second, group[j]);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) second = fmaxf(second, __shfl_xor_sync(0xffffffffu, second, o));
    if (lane == 0) s->warp_second[warp] = second;
    if (__syncthreads_count(tops > 0) > 1 || __syncthreads_or(tops > 1)) second = top;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) second = fmaxf(second, s->warp_second[i]);
    each_of_few<T, kCtas>(s, w, second, [&](float l, int id) {
      if (l > -INFINITY) fold(two, l, l, id);
    });
  } else {
    const float cut_l = cut ? logit_of<T>(cut) : -INFINITY;
    const float least = fmaxf(fmaxf(cut_l, w.min_l), -3.4028234e38f);
    const int last = cut ? id_of(cut) : kMaxV;  // of the tokens with the cut's logit
    float second = -INFINITY;  // two of the CTA's values are no less
    if (t == 0) s->second = 0;
    __syncthreads();
    float reach = least;       // tokens below cannot come to it: the noise is below 16.7
    each4<T>(
        w, least,
        [&](const float(&l)[4], int id) {
          const float most = fmaxf(fmaxf(l[0], l[1]), fmaxf(l[2], l[3]));
          if (!(most >= reach)) return;
          const uint4 v = noise4(key, id);
          // x + g >= second asks for 1 - u <= e^(x - second); with the largest x of the
          // four, as a bound of the noise's word, 1 - u = (2^23 - 1/2 - (word >> 9)) 2^-23
          const float rest = ex2_approx(((most - w.top) * w.r - second) * kLog2e) * (4294967296.f * 1.0001f);
          if (!(static_cast<float>(max(max(v.x, v.y), max(v.z, v.w))) >= 4294965248.f - rest)) return;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t word = word_of(v, j);
            if (l[j] >= least && static_cast<float>(word) >= 4294965248.f - rest && (l[j] != cut_l || id + j <= last))
              fold(two, (l[j] - w.top) * w.r + gumbel_of(word), l[j], id + j);
          }
        },
        [&] {
          const uint32_t z0 = ord_key(two.e[0].z), z1 = ord_key(two.e[1].z);
          const uint32_t best = __reduce_max_sync(0xffffffffu, z0);
          const unsigned who = __ballot_sync(0xffffffffu, z0 == best);
          const uint32_t next = __reduce_max_sync(0xffffffffu, lane == __ffs(who) - 1 ? z1 : z0);
          const uint32_t shared = *const_cast<volatile uint32_t*>(&s->second);
          if (lane == 0 && next > shared) atomicMax(&s->second, next);
          second = of_key(max(next, shared));
          reach = fmaxf(least, w.top + (second - 16.8f) / w.r - 1e-5f * fabsf(w.top));
        });
  }
  finish(s, p, w, key, two, greedy, false, row);
}

// CTAs to a row: 16 while all of them are on the device at once (two per SM), 4
// beyond, as long as each has enough of the row.
int cluster_size(int M, int V) {
  if (M * 16 <= 2 * glance::num_sms() && V >= 16 * 2048) return 16;
  return V >= 4 * 2048 ? 4 : 1;
}

// Clusters of 16 are beyond the portable size: allowed once per kernel and device.
cudaError_t allow_large_clusters(const void* f) {
  static std::mutex mu;
  static const void* done[64][2] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lock(mu);
  const bool known = dev >= 0 && dev < 64;
  for (int i = 0; known && i < 2; ++i)
    if (done[dev][i] == f) return cudaSuccess;
  e = cudaFuncSetAttribute(f, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  for (int i = 0; known && e == cudaSuccess && i < 2; ++i)
    if (!done[dev][i]) {
      done[dev][i] = f;
      break;
    }
  return e;
}

template <typename T, int kCtas>
glance_status launch(const char* who, Params p, cudaStream_t stream) {
  const void* f = reinterpret_cast<const void*>(sample_kernel<T, kCtas>);
  p.slice = ((p.V + kCtas - 1) / kCtas + 63) / 64 * 64;
  const int bytes = static_cast<int>(sizeof(Shared<kCtas>));
  cudaError_t e = glance::ensure_smem(f, bytes);
  if (e == cudaSuccess && kCtas > 8) e = allow_large_clusters(f);
  if (e != cudaSuccess) return glance::cuda_fail(e, who);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.M) * kCtas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kCtas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, sample_kernel<T, kCtas>, p);
  if (e != cudaSuccess) return glance::cuda_fail(e, who);
  return GLANCE_OK;
}
template <typename T>
glance_status launch(const char* who, const Params& p, int ctas, cudaStream_t stream) {
  return ctas == 1   ? launch<T, 1>(who, p, stream)
         : ctas == 4 ? launch<T, 4>(who, p, stream)
                     : launch<T, 16>(who, p, stream);
}

}  // namespace

extern "C" glance_status glance_sample(const void* logits, int64_t row_stride, glance_dtype dtype, int M, int V,
                                       const float* temperature, const int32_t* top_k, const float* top_p, const float* min_p,
                                       uint64_t seed, const int32_t* position, const int32_t* seq, int32_t* tokens, float* gap,
                                       void* stream) {
  using glance::fail;
  const char* who = "glance_sample";
  if (!logits || !position || !tokens) return fail(GLANCE_ERR_INVALID_ARG, "%s: null pointer argument", who);
  if (dtype != GLANCE_BF16 && dtype != GLANCE_F32) return fail(GLANCE_ERR_INVALID_ARG, "%s: dtype must be F32 or BF16", who);
  if (M < 1 || M > (1 << 20)) return fail(GLANCE_ERR_INVALID_ARG, "%s: need 1 <= M <= 2^20", who);
  if (V < 2 || V > kMaxV) return fail(GLANCE_ERR_UNSUPPORTED, "%s: need 2 <= V <= %d", who, kMaxV);
  const int esize = dtype == GLANCE_BF16 ? 2 : 4;
  if (row_stride < V || row_stride > glance::kQ8MaxStride) return fail(GLANCE_ERR_INVALID_ARG, "%s: row_stride must cover a row", who);
  if (reinterpret_cast<uintptr_t>(logits) % esize) return fail(GLANCE_ERR_INVALID_ARG, "%s: logits must be aligned to their type", who);
  const uintptr_t words = reinterpret_cast<uintptr_t>(temperature) | reinterpret_cast<uintptr_t>(top_k) | reinterpret_cast<uintptr_t>(top_p) |
                          reinterpret_cast<uintptr_t>(min_p) | reinterpret_cast<uintptr_t>(position) | reinterpret_cast<uintptr_t>(seq) |
                          reinterpret_cast<uintptr_t>(tokens) | reinterpret_cast<uintptr_t>(gap);
  if (words & 3) return fail(GLANCE_ERR_INVALID_ARG, "%s: the rows' parameters and results must be 4-byte aligned", who);
  const int64_t n = ((M - 1) * row_stride + V) * esize;
  if (glance::overlap(tokens, 4ll * M, logits, n) || (gap && (glance::overlap(gap, 4ll * M, logits, n) || glance::overlap(gap, 4ll * M, tokens, 4ll * M))))
    return fail(GLANCE_ERR_INVALID_ARG, "%s: tokens and gap must not overlap logits or one another", who);
  Params p;
  p.logits = static_cast<const char*>(logits);
  p.stride = row_stride * esize;
  p.temperature = temperature;
  p.top_k = top_k;
  p.top_p = top_p;
  p.min_p = min_p;
  p.position = position;
  p.seq = seq;
  p.tokens = tokens;
  p.gap = gap;
  p.k0 = static_cast<uint32_t>(seed);
  p.k1 = static_cast<uint32_t>(seed >> 32);
  p.M = M;
  p.V = V;
  const int ctas = cluster_size(M, V);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  return dtype == GLANCE_BF16 ? launch<__nv_bfloat16>(who, p, ctas, s) : launch<float>(who, p, ctas, s);
}
