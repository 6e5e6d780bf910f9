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
// A row is read once, by a cluster of CTAs that keep it in their shared memory.
// Its border is found without a sort of the row:
// * A histogram of (max - l) r in steps of 1/64 holds each bin's count and its
//   weight. Within a bin weights are W (1 - d), d < 1/64, W a constant of the
//   bin: the sum of the d is kept as an integer (2^-22 units), so that it does not
//   depend on the order of the additions and is good to 2^-23 of each weight.
// * Where at most kList tokens lie in the bins up to the border's, they are
//   gathered by the cluster's first CTA, sorted, summed and drawn from there.
// * Else the border's bin is divided by further histograms, over ranges of the
//   50-bit numbers, until what is left fits the list; then every CTA looks at its
//   part of the row once more for the draw.
// Weights below e^-32 of the largest are outside the histogram: 2^18 of them
// hold 4e-9 of the sum, under what an fp32 top_p can name.
//
// The draw's values are fp32 and compared in fp32 except for those that are near
// the best: these are evaluated again in fp64, so that rounding decides nothing.
#include <cstring>
#include <mutex>

#include "noise.cuh"
#include "q8_internal.cuh"

GLANCE_DEFINE_STATUS_WORD(status_sample)

using namespace glance_dev;

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kList = 2048;
constexpr int kMaxCluster = 16;
constexpr int kIdBits = 18;
constexpr int kMaxV = 1 << kIdBits;
constexpr int kMaxSlice = 32768;  // ids of a CTA: a bin's sum of d (2^16 units each at most) stays within 32 bits
constexpr int kCand = kThreads;
constexpr float kBinsPerNat = 64.f, kRange = 32.f;
constexpr float kUnit = 4194304.f;  // 2^22

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

// e^-i/2 and e^-i/64 to double precision: a bin's W is the product of two.
struct Exps {
  double half[64], part[32];
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
  e.half[0] = 1;
  for (int i = 1; i < 64; ++i) e.half[i] = e.half[i - 1] * series_exp(-0.5);
  for (int i = 0; i < 32; ++i) e.part[i] = series_exp(-i / 64.0);
  return e;
}
__constant__ Exps c_exps = make_exps();

struct Border {  // the bin in which a prefix ends
  int bin;       // -1: the prefix has all
  uint32_t count_before, count_in;
  double mass_before, mass_all;
};
struct Best {
  float z1, z2;
  int id;
};

struct Shared {
  union {
    struct {
      uint32_t count[kBins], d[kBins];
    } hist;
    uint64_t list[kList];
  };
  // written by the cluster's other CTAs
  float peer_max[kMaxCluster];
  uint64_t peer_lo[kMaxCluster], peer_hi[kMaxCluster];
  double peer_mass[kMaxCluster];
  uint32_t peer_count[kMaxCluster];
  Best peer_best[kMaxCluster];
  Border border;
  uint64_t cut;
  double cut_mass;
  uint32_t list_n, cand_n;
  float cand_l[kCand];
  int cand_id[kCand];
  // this CTA's own
  double warp_mass[kWarps];
  uint32_t warp_count[kWarps];
  float warp_f[kWarps];
  uint64_t warp_lo[kWarps], warp_hi[kWarps];
  Best warp_best[kWarps];
  float min_l;
  double log_min_p;
};

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
template <typename X>
__device__ __forceinline__ void to_peer(X* local, int rank, X v) {
  // plain stores of 4-byte words to the same place in CTA `rank`
  static_assert(sizeof(X) % 4 == 0, "words");
  const uint32_t at = dsmem_addr(local, rank);
  uint32_t w[sizeof(X) / 4];
  memcpy(w, &v, sizeof(X));
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(X) / 4); ++i)
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at + 4 * i), "r"(w[i]) : "memory");
}
__device__ __forceinline__ uint32_t peer_u32(const void* local, int rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(dsmem_addr(local, rank)) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t peer_add(uint32_t* local, int rank, uint32_t v) {
  uint32_t old;
  asm volatile("atom.relaxed.cluster.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(old) : "r"(dsmem_addr(local, rank)), "r"(v) : "memory");
  return old;
}

__device__ __forceinline__ uint64_t number_of(float l, int id) {
  return static_cast<uint64_t>(ord_key(l)) << kIdBits | static_cast<uint32_t>(kMaxV - 1 - id);
}
__device__ __forceinline__ int id_of(uint64_t number) { return kMaxV - 1 - static_cast<int>(number & (kMaxV - 1)); }
__device__ __forceinline__ float logit_of(uint64_t number) {
  const uint32_t k = static_cast<uint32_t>(number >> kIdBits);
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

// The row as this thread sees it.
struct Row {
  float top, r;  // the largest logit; 1 / T
  float min_l;   // tokens below are not kept
  int rank, ctas, first, n;  // this CTA's ids: first .. first + n - 1
};

// (max - l) r, its rounding error, and from them the bin and d
__device__ __forceinline__ bool place(const Row& w, float l, int& bin, float& d) {
  const float x = w.top - l, prod = x * w.r;
  if (!(prod < kRange) || l < w.min_l) return false;
  const float err = fmaf(x, w.r, -prod);
  bin = static_cast<int>(prod * kBinsPerNat);
  const float y = fmaxf(fmaf(static_cast<float>(bin), -1.f / kBinsPerNat, prod) + err, 0.f);
  // 1 - e^-y, y < 1/64 (to y^5 / 120 < 1e-11)
  d = y * fmaf(y, fmaf(y, fmaf(y, -1.f / 24, 1.f / 6), -0.5f), 1.f);
  return true;
}
__device__ __forceinline__ double weight_of_bin(int bin) { return c_exps.half[bin >> 5] * c_exps.part[bin & 31]; }

template <typename T>
struct Row4;  // four consecutive logits in shared memory
template <>
struct Row4<float> {
  static __device__ __forceinline__ void load(const unsigned char* s, int i, float (&l)[4]) {
    const float4 v = *reinterpret_cast<const float4*>(s + 4 * i);
    l[0] = v.x, l[1] = v.y, l[2] = v.z, l[3] = v.w;
  }
};
template <>
struct Row4<__nv_bfloat16> {
  static __device__ __forceinline__ void load(const unsigned char* s, int i, float (&l)[4]) {
    const uint2 v = *reinterpret_cast<const uint2*>(s + 2 * i);
    l[0] = __uint_as_float(v.x << 16), l[1] = __uint_as_float(v.x & 0xFFFF0000u);
    l[2] = __uint_as_float(v.y << 16), l[3] = __uint_as_float(v.y & 0xFFFF0000u);
  }
};

// Calls f(logit, id) for this CTA's tokens, four consecutive ids a thread at a
// time (ids behind the row are -infinity).
template <typename T, typename F>
__device__ __forceinline__ void each(const unsigned char* s_row, const Row& w, F f) {
  for (int i = 4 * static_cast<int>(threadIdx.x); i < w.n; i += 4 * kThreads) {
    float l[4];
    Row4<T>::load(s_row, i, l);
#pragma unroll
    for (int j = 0; j < 4; ++j) f(l[j], w.first + i + j);
  }
}

__device__ __forceinline__ void clear_hist(Shared* s) {
  for (int i = threadIdx.x; i < kBins; i += kThreads) s->hist.count[i] = s->hist.d[i] = 0u;
}

__device__ __forceinline__ uint32_t scan_add(uint32_t v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}
__device__ __forceinline__ double scan_add(double v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

// The bin of the cluster's histogram in which the prefix of `want` tokens
// (want > 0) or else of `share` of the weight (of mass_all, if given, else of
// what the histogram has) ends. fixed_bin >= 0: every bin's W is that bin's.
// count0, mass0: what lies before the histogram. All threads of the cluster get
// the same answer.
__device__ Border find_border(Shared* s, const Row& w, uint32_t want, double share, double mass_all, int fixed_bin, uint32_t count0,
                              double mass0) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  cluster_sync_all();  // the histograms are complete
  const int mine = kBins / w.ctas, per = (mine + kThreads - 1) / kThreads;  // bins of this CTA, of a thread: 1, 2 or 4
  uint32_t c[4];
  double m[4], mass = 0;
  uint32_t count = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    c[j] = 0;
    m[j] = 0;
    const int in = static_cast<int>(threadIdx.x) * per + j;
    if (j < per && in < mine) {
      const int bin = w.rank * mine + in;
      uint64_t d = 0;
      for (int q = 0; q < w.ctas; ++q) {
        c[j] += peer_u32(&s->hist.count[bin], q);
        d += peer_u32(&s->hist.d[bin], q);
      }
      if (c[j]) m[j] = weight_of_bin(fixed_bin >= 0 ? fixed_bin : bin) * (c[j] - static_cast<double>(d) * (1.0 / kUnit));
    }
    count += c[j];
    mass += m[j];
  }
  const uint32_t count_to = scan_add(count, lane);
  const double mass_to = scan_add(mass, lane);
  if (lane == 31) {
    s->warp_count[warp] = count_to;
    s->warp_mass[warp] = mass_to;
  }
  __syncthreads();
  uint32_t count_at = 0, count_cta = 0;
  double mass_at = 0, mass_cta = 0;
  for (int i = 0; i < kWarps; ++i) {
    if (i == warp) {
      count_at = count_cta;
      mass_at = mass_cta;
    }
    count_cta += s->warp_count[i];
    mass_cta += s->warp_mass[i];
  }
  if (threadIdx.x < w.ctas) {
    to_peer(&s->peer_count[w.rank], threadIdx.x, count_cta);
    to_peer(&s->peer_mass[w.rank], threadIdx.x, mass_cta);
  }
  if (threadIdx.x == 0) s->border.bin = -1;
  cluster_sync_all();
  uint32_t base_count = count0, count_all = count0;
  double base = mass0, all = mass0;
  for (int q = 0; q < w.ctas; ++q) {
    if (q == w.rank) {
      base_count = count_all;
      base = all;
    }
    count_all += s->peer_count[q];
    all += s->peer_mass[q];
  }
  if (mass_all <= 0) mass_all = all;
  const double target = share * mass_all;
  count_at += base_count + count_to - count;
  mass_at += base + mass_to - mass;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    // the first token at which the prefix is long or heavy enough is in this bin
    const bool here = c[j] && (want ? count_at < want && count_at + c[j] >= want
                                    : mass_at < target && mass_at + m[j] >= target);
    if (here) {
      const Border b = {w.rank * mine + static_cast<int>(threadIdx.x) * per + j, count_at, c[j], mass_at, mass_all};
      for (int q = 0; q < w.ctas; ++q) to_peer(&s->border, q, b);
    }
    count_at += c[j];
    mass_at += m[j];
  }
  cluster_sync_all();
  Border b = s->border;
  b.mass_all = mass_all;
  return b;
}

// Sorts s->list[0 .. n) in descending order (one CTA).
__device__ void sort_list(Shared* s, int n) {
  int size = 32;
  while (size < n) size <<= 1;
  for (int i = n + threadIdx.x; i < size; i += kThreads) s->list[i] = 0;
  __syncthreads();
  for (int k = 2; k <= size; k <<= 1)
    for (int j = k >> 1; j; j >>= 1) {
      for (int i = threadIdx.x; i < size / 2; i += kThreads) {
        const int a = 2 * i - (i & (j - 1)), b = a + j;
        const uint64_t x = s->list[a], y = s->list[b];
        if ((x < y) == ((a & k) == 0)) {
          s->list[a] = y;
          s->list[b] = x;
        }
      }
      __syncthreads();
    }
}

// Weights of the sorted list's tokens before and up to each: this thread's four.
__device__ void list_masses(Shared* s, const Row& w, int n, double mass0, double (&before)[kList / kThreads], double (&upto)[kList / kThreads]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  double sum = 0;
#pragma unroll
  for (int j = 0; j < kList / kThreads; ++j) {
    const int i = threadIdx.x * (kList / kThreads) + j;
    double m = 0;
    int bin;
    float d;
    if (i < n && place(w, logit_of(s->list[i]), bin, d)) m = weight_of_bin(bin) * (1.0 - static_cast<double>(d));
    before[j] = sum;
    sum += m;
    upto[j] = sum;
  }
  const double to = scan_add(sum, lane);
  __syncthreads();
  if (lane == 31) s->warp_mass[warp] = to;
  __syncthreads();
  double at = mass0 + to - sum;
  for (int i = 0; i < warp; ++i) at += s->warp_mass[i];
#pragma unroll
  for (int j = 0; j < kList / kThreads; ++j) {
    before[j] += at;
    upto[j] += at;
  }
}

// Gathers the numbers of the tokens that pass f(logit, id, number) in the first
// CTA's list (there are kList at most); ends with a barrier of the cluster.
template <typename T, typename F>
__device__ void gather(Shared* s, const unsigned char* s_row, const Row& w, F f) {
  each<T>(s_row, w, [&](float l, int id) {
    const uint64_t number = number_of(l, id);
    if (f(l, number)) {
      const uint32_t at = peer_add(&s->list_n, 0, 1u);
      if (at < kList) to_peer(&s->list[at], 0, number);
    }
  });
  cluster_sync_all();
}

__device__ __forceinline__ void merge(Best& a, const Best& b) {
  if (b.z1 > a.z1 || (b.z1 == a.z1 && b.id < a.id)) {
    a.z2 = fmaxf(a.z1, b.z2);
    a.z1 = b.z1;
    a.id = b.id;
  } else {
    a.z2 = fmaxf(a.z2, b.z1);
  }
}
__device__ __forceinline__ Best warp_best(Best v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const Best u = {__shfl_xor_sync(0xffffffffu, v.z1, o), __shfl_xor_sync(0xffffffffu, v.z2, o), __shfl_xor_sync(0xffffffffu, v.id, o)};
    merge(v, u);
  }
  return v;
}
__device__ Best block_best(Shared* s, Best v) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  v = warp_best(v);
  __syncthreads();
  if (lane == 0) s->warp_best[warp] = v;
  __syncthreads();
  return warp_best(lane < kWarps ? s->warp_best[lane] : Best{-INFINITY, -INFINITY, 0x7FFFFFFF});
}

// Two best values that a thread has seen, with their tokens.
struct Two {
  float z[2], l[2];
  int id[2];
};
__device__ __forceinline__ void fold(Two& t, float z, float l, int id) {
  if (z > t.z[0] || (z == t.z[0] && id < t.id[0])) {
    t.z[1] = t.z[0], t.l[1] = t.l[0], t.id[1] = t.id[0];
    t.z[0] = z, t.l[0] = l, t.id[0] = id;
  } else if (z > t.z[1] || (z == t.z[1] && id < t.id[1])) {
    t.z[1] = z, t.l[1] = l, t.id[1] = id;
  }
}

__device__ __forceinline__ uint32_t word_of(const uint4& v, int j) { return j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w; }

// The draw's value of a token in 64 bits.
__device__ double value64(const Params& p, const Row& w, float l, int id, uint32_t pos, uint32_t seq) {
  const uint4 n = philox4x32_10(make_uint4(static_cast<uint32_t>(id) / 4, pos, seq, 0u), p.k0, p.k1);
  const double u = (static_cast<double>(word_of(n, id & 3) >> 9) + 0.5) * (1.0 / 8388608.0);
  return (static_cast<double>(l) - static_cast<double>(w.top)) * static_cast<double>(w.r) - log(-log(u));
}

// From the threads' two best values to the row's token: the first CTA (of the
// cluster, or by itself with `alone`) writes it.
__device__ void finish(Shared* s, const Params& p, const Row& w, const Two& t, bool greedy, bool alone, int row, uint32_t pos,
                       uint32_t seq) {
  Best b = {t.z[0], t.z[1], t.id[0]};
  b = block_best(s, b);
  if (!alone) {
    if (threadIdx.x < w.ctas) to_peer(&s->peer_best[w.rank], threadIdx.x, b);
    cluster_sync_all();
    b = s->peer_best[0];
    for (int q = 1; q < w.ctas; ++q) merge(b, s->peer_best[q]);
  }
  // values within rounding of the best, fp32's and the noise's, are compared in fp64
  const float near = b.z1 - (2e-5f + 1e-6f * fabsf(b.z1));
  if (!greedy) {
#pragma unroll
    for (int j = 0; j < 2; ++j)
      if (t.z[j] >= near) {
        const uint32_t at = alone ? atomicAdd(&s->cand_n, 1u) : peer_add(&s->cand_n, 0, 1u);
        if (at < kCand) {
          if (alone) {
            s->cand_l[at] = t.l[j];
            s->cand_id[at] = t.id[j];
          } else {
            to_peer(&s->cand_l[at], 0, t.l[j]);
            to_peer(&s->cand_id[at], 0, t.id[j]);
          }
        }
      }
    if (alone)
      __syncthreads();
    else
      cluster_sync_all();
  }
  if (w.rank != 0) return;
  float gap = b.z1 - b.z2;
  int id = b.id;
  const int n = greedy ? 1 : static_cast<int>(s->cand_n);
  if (n > 1 && n <= kCand) {
    double z = -INFINITY;
    int mine = 0x7FFFFFFF;
    if (threadIdx.x < n) {
      mine = s->cand_id[threadIdx.x];
      z = value64(p, w, s->cand_l[threadIdx.x], mine, pos, seq);
    }
    // by one thread over the few of them
    double* zs = reinterpret_cast<double*>(s->list);
    __syncthreads();
    if (threadIdx.x < n) zs[threadIdx.x] = z;
    __syncthreads();
    if (threadIdx.x == 0) {
      double z1 = -INFINITY, z2 = -INFINITY;
      id = 0x7FFFFFFF;
      for (int i = 0; i < n; ++i) {
        if (zs[i] > z1 || (zs[i] == z1 && s->cand_id[i] < id)) {
          z2 = z1;
          z1 = zs[i];
          id = s->cand_id[i];
        } else if (zs[i] > z2) {
          z2 = zs[i];
        }
      }
      gap = static_cast<float>(z1 - z2);
    }
  }
  if (threadIdx.x == 0 && GLANCE_IN_BOUNDS(row, p.M)) {
    p.tokens[row] = id;
    if (p.gap) p.gap[row] = gap;
  }
}

// The number of the last token that a prefix keeps, and the weight up to it:
// the bin's tokens (from `floor` on) are divided until they fit the list, and
// that is sorted.
template <typename T>
__device__ void refine(Shared* s, const unsigned char* s_row, const Row& w, const Border& first, uint64_t floor, uint32_t want,
                       double share, uint64_t* cut, double* mass) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Border b = first;
  const int bin = b.bin;
  uint64_t lo = floor, hi = ~0ull;
  const auto inside = [&](float l, uint64_t number) {
    int at;
    float d;
    return number >= lo && number <= hi && place(w, l, at, d) && at == bin;
  };
  // the numbers differ and the range shrinks to the tokens' own each time: 50
  // bits are through after five divisions by 2^10 or more
  for (int level = 0; level < 8 && b.count_in > kList; ++level) {
    uint64_t least = ~0ull, most = 0;
    each<T>(s_row, w, [&](float l, int id) {
      const uint64_t number = number_of(l, id);
      if (inside(l, number)) {
        least = min(least, number);
        most = max(most, number);
      }
    });
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      least = min(least, __shfl_xor_sync(0xffffffffu, least, o));
      most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
    }
    if (lane == 0) {
      s->warp_lo[warp] = least;
      s->warp_hi[warp] = most;
    }
    __syncthreads();
    for (int i = 0; i < kWarps; ++i) {
      least = min(least, s->warp_lo[i]);
      most = max(most, s->warp_hi[i]);
    }
    if (threadIdx.x < w.ctas) {
      to_peer(&s->peer_lo[w.rank], threadIdx.x, least);
      to_peer(&s->peer_hi[w.rank], threadIdx.x, most);
    }
    clear_hist(s);
    cluster_sync_all();
    for (int q = 0; q < w.ctas; ++q) {
      least = min(least, s->peer_lo[q]);
      most = max(most, s->peer_hi[q]);
    }
    lo = least;
    hi = most;
    int shift = 0;
    while ((hi - lo) >> shift >= kBins) ++shift;
    each<T>(s_row, w, [&](float l, int id) {
      const uint64_t number = number_of(l, id);
      int at;
      float d;
      if (number >= lo && number <= hi && place(w, l, at, d) && at == bin) {
        const int sub = static_cast<int>((hi - number) >> shift);
        atomicAdd(&s->hist.count[sub], 1u);
        atomicAdd(&s->hist.d[sub], __float2uint_rn(d * kUnit));
      }
    });
    const double all = b.mass_all;
    b = find_border(s, w, want, share, all, bin, b.count_before, b.mass_before);
    if (b.bin < 0) {  // the sum of the weights came out a rounding short of its share: the range's last token
      *cut = lo;
      *mass = all;
      return;
    }
    hi -= static_cast<uint64_t>(b.bin) << shift;
    const uint64_t least_of_bin = hi - ((1ull << shift) - 1);
    if (least_of_bin > lo) lo = least_of_bin;
  }
  gather<T>(s, s_row, w, [&](float l, uint64_t number) { return inside(l, number); });
  if (w.rank == 0) {
    const int n = min(static_cast<int>(s->list_n), kList);
    __syncthreads();
    if (threadIdx.x == 0) s->list_n = 0;
    sort_list(s, n);
    double before[kList / kThreads], upto[kList / kThreads];
    list_masses(s, w, n, b.mass_before, before, upto);
    const double target = share * b.mass_all;
    if (threadIdx.x == 0) {  // unless a token is found: the last one
      s->cut = s->list[n - 1];
      s->cut_mass = b.mass_all;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kList / kThreads; ++j) {
      const int i = threadIdx.x * (kList / kThreads) + j;
      if (i < n && (want ? b.count_before + i + 1 == want : before[j] < target && upto[j] >= target)) {
        s->cut = s->list[i];
        s->cut_mass = upto[j];
      }
    }
    __syncthreads();
    if (threadIdx.x < w.ctas && threadIdx.x > 0) {
      to_peer(&s->cut, threadIdx.x, s->cut);
      to_peer(&s->cut_mass, threadIdx.x, s->cut_mass);
    }
  }
  cluster_sync_all();
  *cut = s->cut;
  *mass = s->cut_mass;
}

// Grid: x = row * cluster size + rank.
template <typename T>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const Params p, const int ctas) {
  extern __shared__ __align__(16) unsigned char smem[];
  Shared* s = reinterpret_cast<Shared*>(smem);
  unsigned char* s_row = smem + (sizeof(Shared) + 15) / 16 * 16;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = static_cast<int>(blockIdx.x) / ctas;
  Row w;
  w.ctas = ctas;
  w.rank = static_cast<int>(cluster_ctarank());
  w.first = w.rank * p.slice;
  w.n = max(0, min(p.slice, p.V - w.first));
  pdl_wait_prior();
  pdl_launch_dependents();
  const float temperature = p.temperature ? __ldg(p.temperature + row) : 1.f;
  const int k = p.top_k ? __ldg(p.top_k + row) : 0;
  const float top_p = p.top_p ? __ldg(p.top_p + row) : 1.f, min_p = p.min_p ? __ldg(p.min_p + row) : 0.f;
  const uint32_t pos = static_cast<uint32_t>(__ldg(p.position + row)), seq = p.seq ? static_cast<uint32_t>(__ldg(p.seq + row)) : 0u;
  const bool greedy = temperature == 0.f;
  w.r = greedy ? 1.f : 1.f / temperature;
  if (threadIdx.x == 0) {
    s->list_n = s->cand_n = 0;
    s->log_min_p = min_p > 0.f ? log(static_cast<double>(min_p)) : 0.0;
  }
  // the row's part into shared memory, its largest logit on the way
  constexpr int kN = 16 / static_cast<int>(sizeof(T));
  const char* src = p.logits + row * p.stride + static_cast<long long>(w.first) * static_cast<int>(sizeof(T));
  float top = -INFINITY;
  int done = 0;
  if ((reinterpret_cast<uintptr_t>(src) & 15) == 0) {
    const int vecs = w.n / kN;
    done = vecs * kN;
#pragma unroll 4
    for (int i = threadIdx.x; i < vecs; i += kThreads) {
      const uint4 v = __ldcs(reinterpret_cast<const uint4*>(src) + i);
      *reinterpret_cast<uint4*>(s_row + 16 * i) = v;
      const uint32_t q[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (sizeof(T) == 4)
          top = max_nan(top, __uint_as_float(q[j]));
        else
          top = max_nan(top, max_nan(__uint_as_float(q[j] << 16), __uint_as_float(q[j] & 0xFFFF0000u)));
      }
    }
  }
#pragma unroll 4
  for (int i = done + threadIdx.x; i < w.n; i += kThreads) {
    const T v = reinterpret_cast<const T*>(src)[i];
    reinterpret_cast<T*>(s_row)[i] = v;
    top = max_nan(top, static_cast<float>(v));
  }
  if (threadIdx.x < 4) reinterpret_cast<T*>(s_row)[w.n + threadIdx.x] = static_cast<T>(-INFINITY);
#pragma unroll
  for (int o = 16; o; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (lane == 0) s->warp_f[warp] = top;
  __syncthreads();
  for (int i = 0; i < kWarps; ++i) top = max_nan(top, s->warp_f[i]);
  // (the barrier of the cluster that every path has after this one keeps the CTAs together)
  cluster_sync_all();  // the other CTAs have begun: their shared memory may be written
  if (threadIdx.x < ctas) to_peer(&s->peer_max[w.rank], threadIdx.x, top);
  cluster_sync_all();
  for (int q = 0; q < ctas; ++q) top = max_nan(top, s->peer_max[q]);
  w.top = top;
  const bool bad_row = !(top > -INFINITY && top < INFINITY);
  const bool bad_param = !(temperature >= 0.f && w.r < INFINITY && w.r > 0.f) || top_p != top_p || min_p != min_p;
  if (bad_row || bad_param) {
    if (threadIdx.x == 0 && w.rank == 0 && GLANCE_IN_BOUNDS(row, p.M)) {
      p.tokens[row] = -1;
      if (p.gap) p.gap[row] = NAN;
      report(bad_row ? GLANCE_DEV_NONFINITE_LOGITS : GLANCE_DEV_BAD_SAMPLING);
    }
    return;
  }
  // the least logit with (l - top) r >= ln min_p, in fp64
  w.min_l = -INFINITY;
  if (min_p > 0.f && !greedy) {
    if (threadIdx.x == 0) {
      const double lg = fmin(s->log_min_p, 0.0), r = w.r, t = top;
      float x = static_cast<float>(t + lg / r);
      x = fminf(x, top);
      for (int i = 0; i < 4 && x > -INFINITY && (static_cast<double>(x) - t) * r >= lg; ++i) x = nextafterf(x, -INFINITY);
      for (int i = 0; i < 8 && (static_cast<double>(x) - t) * r < lg; ++i) x = nextafterf(x, INFINITY);
      s->min_l = x;
    }
    __syncthreads();
    w.min_l = s->min_l;
  }
  const uint32_t want = k > 0 && k < p.V ? k : 0u;
  const double share = top_p < 1.f ? static_cast<double>(fmaxf(top_p, 0.f)) : 1.0;
  uint64_t cut = 0;  // the last number that is kept
  if (!greedy && (want || share < 1.0)) {
    clear_hist(s);
    __syncthreads();
    each<T>(s_row, w, [&](float l, int) {
      int bin;
      float d;
      if (place(w, l, bin, d)) {
        atomicAdd(&s->hist.count[bin], 1u);
        atomicAdd(&s->hist.d[bin], __float2uint_rn(d * kUnit));
      }
    });
    // share 0: the first token alone, which any positive share has
    const double least = share > 0 ? share : 1e-300;
    Border b = find_border(s, w, want, want ? 1.0 : least, 0, -1, 0u, 0);
    const uint32_t upto = b.bin < 0 ? 0xFFFFFFFFu : b.count_before + b.count_in;
    if (upto <= kList) {
      // all that may be kept fits the list: the first CTA draws from it
      gather<T>(s, s_row, w, [&](float l, uint64_t) {
        int bin;
        float d;
        return place(w, l, bin, d) && bin <= b.bin;
      });
      if (w.rank != 0) return;
      const int n = min(static_cast<int>(s->list_n), kList);
      sort_list(s, n);
      double before[kList / kThreads], upto_mass[kList / kThreads];
      list_masses(s, w, n, 0, before, upto_mass);
      const int kept = want ? min(static_cast<int>(want), n) : n;
      // the weight of the first k, or of all
      if (want && static_cast<int>(threadIdx.x) == (kept - 1) / (kList / kThreads)) {
#pragma unroll
        for (int j = 0; j < kList / kThreads; ++j)
          if ((kept - 1) % (kList / kThreads) == j) s->cut_mass = upto_mass[j];
      }
      __syncthreads();
      const double target = least * (want ? s->cut_mass : b.mass_all);
      Two t = {{-INFINITY, -INFINITY}, {0.f, 0.f}, {0x7FFFFFFF, 0x7FFFFFFF}};
#pragma unroll
      for (int j = 0; j < kList / kThreads; ++j) {
        const int i = threadIdx.x * (kList / kThreads) + j;
        if (i < kept && (share >= 1.0 || before[j] < target)) {
          const uint64_t number = s->list[i];
          const int id = id_of(number);
          const float l = logit_of(number);
          const uint4 v = philox4x32_10(make_uint4(static_cast<uint32_t>(id) / 4, pos, seq, 0u), p.k0, p.k1);
          fold(t, fmaf(l - w.top, w.r, gumbel_of(word_of(v, id & 3))), l, id);
        }
      }
      finish(s, p, w, t, false, true, row, pos, seq);
      return;
    }
    if (b.bin >= 0) {
      double mass = b.mass_all;
      uint64_t last;
      refine<T>(s, s_row, w, b, 0, want, want ? 1.0 : least, &last, &mass);
      cut = last;
      if (want && share < 1.0) {
        // the first k are known: the share of their weight ends at or before their last
        clear_hist(s);
        __syncthreads();
        each<T>(s_row, w, [&](float l, int id) {
          int bin;
          float d;
          if (place(w, l, bin, d) && number_of(l, id) >= cut) {
            atomicAdd(&s->hist.count[bin], 1u);
            atomicAdd(&s->hist.d[bin], __float2uint_rn(d * kUnit));
          }
        });
        b = find_border(s, w, 0u, least, mass, -1, 0u, 0);
        if (b.bin >= 0) {
          refine<T>(s, s_row, w, b, cut, 0u, least, &last, &mass);
          if (last > cut) cut = last;
        }
      }
    } else if (want && share < 1.0) {
      // fewer than k tokens in reach: the share is of all of them
      b = find_border(s, w, 0u, least, 0, -1, 0u, 0);
      if (b.bin >= 0) {
        double mass;
        refine<T>(s, s_row, w, b, 0, 0u, least, &cut, &mass);
      }
    }
  }
  // every CTA looks at its part of the row
  Two t = {{-INFINITY, -INFINITY}, {0.f, 0.f}, {0x7FFFFFFF, 0x7FFFFFFF}};
  if (greedy) {
    each<T>(s_row, w, [&](float l, int id) {
      if (l > -INFINITY) fold(t, l, l, id);
    });
  } else {
    for (int i = 4 * static_cast<int>(threadIdx.x); i < w.n; i += 4 * kThreads) {
      float l[4];
      Row4<T>::load(s_row, i, l);
      const int id = w.first + i;
      bool any[4], some = false;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        // the noise is below 16.7: a token that cannot reach this thread's second best is passed over
        any[j] = l[j] > -INFINITY && l[j] >= w.min_l && fmaf(l[j] - w.top, w.r, 16.7f) >= t.z[1] &&
                 (!cut || number_of(l[j], id + j) >= cut);
        some |= any[j];
      }
      if (!some) continue;
      const uint4 v = philox4x32_10(make_uint4(static_cast<uint32_t>(id) / 4, pos, seq, 0u), p.k0, p.k1);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (any[j]) fold(t, fmaf(l[j] - w.top, w.r, gumbel_of(word_of(v, j))), l[j], id + j);
    }
  }
  finish(s, p, w, t, greedy, false, row, pos, seq);
}

// CTAs to a row: as few as hold it with two of them on an SM, more while the
// rows alone would leave SMs idle and each keeps 4096 tokens.
int cluster_size(int M, int V, int esize) {
  int c = 1;
  while (c < kMaxCluster && ((V + c - 1) / c > kMaxSlice || (V + c - 1) / c * esize > 77 * 1024)) c <<= 1;
  while (c < kMaxCluster && static_cast<int64_t>(M) * c * 2 <= glance::num_sms() && V / (2 * c) >= 4096) c <<= 1;
  return c;
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

template <typename T>
glance_status launch(const char* who, const Params& p, int ctas, cudaStream_t stream) {
  const void* f = reinterpret_cast<const void*>(sample_kernel<T>);
  const int bytes = static_cast<int>((sizeof(Shared) + 15) / 16 * 16 + (static_cast<size_t>(p.slice) + 8) * sizeof(T));
  cudaError_t e = glance::ensure_smem(f, bytes);
  if (e == cudaSuccess && ctas > 8) e = allow_large_clusters(f);
  if (e != cudaSuccess) return glance::cuda_fail(e, who);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.M) * ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, sample_kernel<T>, p, ctas);
  if (e != cudaSuccess) return glance::cuda_fail(e, who);
  return GLANCE_OK;
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
  const int ctas = cluster_size(M, V, esize);
  p.slice = ((V + ctas - 1) / ctas + 63) / 64 * 64;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  return dtype == GLANCE_BF16 ? launch<__nv_bfloat16>(who, p, ctas, s) : launch<float>(who, p, ctas, s);
}
