// bl_sample.cu - one token per row of logits: temperature, top-k, top-p, min-p
// and a draw by a given uniform number.
//
// Weights w = exp((x - max) / T) are whole multiples of 2^-40 (each within one of
// the exact value) and added as 64-bit integers (V <= 2^22 keeps a row's sum below
// 2^62), so every sum of them is exact and no order of adding changes the token.
//
// A cluster of 1 to 16 CTAs owns a row: each CTA reads its stretch once into
// shared memory, and every later pass runs there. The thresholds of top-k and
// top-p come from one histogram of 2048 bins, linear in x, of one 32-bit atomic
// per token: a count and the sum of the tokens' places in the bin. Counts place
// the k-th token in a bin exactly; the places bound every bin's weight to
// about 0.05%, which places the border of top-p within a few bins without an
// exponential. Where a list holds the tokens of those bins (1024; some hundreds at
// p = 0.9 of 128000), they settle the border exactly; where it does not (p near 1 in
// a broad row; more than 16 x 16383 = 262128 tokens, whose words have no room for
// places and bound a bin's weight to about 1.4%), finer bins over their range come
// first. Top-p then needs one exponential per token for the exact sum, a draw
// without filters likewise, top-k none beyond the kept tokens.
//
// Few rows are bound by the chain of barriers (one over a cluster takes about
// 1 us), so a row is spread over up to 16 CTAs and no CTA waits for another's
// verdict. Many rows are bound by latency too, not by the single read of the logits
// and by no unit: in 256 x 128000 with top-p the schedulers issue 54% of the time
// (ALU 39%, shared memory 36%, fp64 8%, DRAM 6%), and of 12 cycles that a warp takes
// per instruction 2.4 are fixed latencies, 2.0 barriers, 1.4 shared memory: two CTAs
// an SM (64 registers, 104 KB) cover one another's phases only in part.
// Measured in a graph, fp32 logits: 1 x 128000, top-k and top-p, 16.5 us, top-p alone
// 21.6; 32 x 32000 without filters 10.3; 256 x 128000 with p = 0.9 248, with p of
// 0.8 to 0.99 by rows 277 to 286 (131 MB: a copy's rate is 20 us); 64 x 262128 187,
// 64 x 262144 290. The 1024-thread bf16 form spills 36 bytes a thread at its 64 registers.
#include "bl_internal.h"
#include "bl_sample_bounds.h"
#include "bl_sample_cut.h"

#include <cstddef>
#include <type_traits>

namespace bl {

namespace {

constexpr int kMaxWarps = 32;
constexpr int kBins = 2048;          // the last one holds what lies past the range
constexpr int kListMax = 1024;       // tokens that a list of candidates holds
constexpr int kDigitBits = 9, kDigits = 1 << kDigitBits;  // of a key, where a border is sought among candidates
constexpr int kWholeMax = 512;       // up to this many the draw itself runs from the list (a sort in registers)
constexpr double kWeightOne = 1099511627776.0;  // 2^40
constexpr double kTail = 29.0;       // exp(-29) * 2^40 rounds to zero

using u64 = unsigned long long;

// Keys order the logits as unsigned integers; 0 stands for a token that is
// out (NaN or -inf). -0 counts as +0.
__device__ __forceinline__ uint32_t sample_key(float x) {
  if (!(x > -INFINITY)) return 0u;
  const uint32_t b = __float_as_uint(x + 0.0f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}

// Shared memory of a CTA; the logits follow it. Every member starts on a 16-byte
// boundary.
struct alignas(16) Smem {
  uint32_t cnt[kBins], off[kBins];  // the row's histogram: counts and sums of places
  alignas(16) u64 list[kListMax];   // the row's candidates: key << 32 | ~index
  union {
    uint32_t hist[kBins];    // this CTA's histogram: counts above sums of places
    u64 local[kListMax];     // this CTA's candidates
    u64 wlist[kListMax];     // weights of the list
    uint32_t part[2 * kMaxWarps * 32];  // weights by the thread that owns the token, likewise
    uint32_t digit[2 * kDigits];  // weights by a digit of the key: low 20 bits, the others
  };
  alignas(16) double tab[256];           // 2^(40 + j / 256)
  alignas(16) u64 red[3][kMaxWarps];
  alignas(16) float redf[2][kMaxWarps];
  alignas(16) u64 xch[2][kMaxCluster][4];  // what the CTAs of the cluster tell one another
  alignas(16) uint32_t slice[2][kBins / 8];  // sums of this CTA's share of the bins
  alignas(16) uint32_t list_n;           // of the first CTA: places given out in the lists
  uint32_t local_n, base;    // this CTA's candidates, and their place in the lists
  int bin_lo, bin_hi;        // bins of the candidates
  uint32_t mode;
  uint32_t lo_key, hi_key;   // their keys: lo_key <= key < hi_key
  alignas(16) u64 need, count;
};
static_assert(sizeof(Smem) % 16 == 0 && offsetof(Smem, xch) % 16 == 0 && offsetof(Smem, need) % 16 == 0, "alignment");

// Shared memory of another CTA of the cluster, by its address there.
__device__ __forceinline__ uint32_t remote_addr(const void* mine, int rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(mine)), "r"(rank));
  return a;
}
__device__ __forceinline__ void remote_store(uint32_t a, u64 v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(a), "l"(v) : "memory");
}
__device__ __forceinline__ void remote_store(uint32_t a, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t remote_add(uint32_t a, uint32_t v) {
  uint32_t old;
  asm volatile("atom.relaxed.cluster.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(old) : "r"(a), "r"(v) : "memory");
  return old;
}
__device__ __forceinline__ uint32_t remote_load(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// Every thread of the cluster; what was written before is seen after.
__device__ __forceinline__ void cluster_sync() {
  cluster_arrive();
  cluster_wait();
}

struct Sums {
  u64 a, b;  // of every thread
  u64 c;     // of every CTA: the same value in its threads
};

// What follows from a histogram.
enum : uint32_t {
  kWhole,   // the candidates are all that can stay: draw from the list
  kBorder,  // the candidates hold the border
  kCrowd,   // more of them than a list holds
  kZeros,   // only tokens of weight zero are in question
};

struct Row {
  double mx;      // largest logit
  double c;       // -256 log2(e) / T
  uint32_t top;   // its key
  float mxf;
};

// 2^(40 + j / 256), by the exponential's series.
struct alignas(16) Exp2Table {
  double v[256];
};
constexpr Exp2Table make_exp2_table() {
  Exp2Table t{};
  for (int j = 0; j < 256; ++j) {
    const double y = j * (0.693147180559945309417 / 256.0);
    double sum = 0.0;
    for (int i = 24; i > 0; --i) sum = (sum + 1.0) * y / i;
    t.v[j] = (sum + 1.0) * kWeightOne;
  }
  return t;
}
__device__ const Exp2Table kExp2Table = make_exp2_table();

// exp((x - max) / T) in units of 2^-40, by a table of 2^(j/256) and a cubic
// (P. T. P. Tang, ACM TOMS 15(2), 1989): within 2^-42 relative before rounding.
// The result is 2^52 + w as a double's bits: kMagicBits less is w, and sums of
// such bits, modulo 2^64, are sums of weights and counts of kMagicBits.
constexpr u64 kMagicBits = 0x4330000000000000ull;  // 2^52
__device__ __forceinline__ u64 weight_bits_at(double t, const double* tab) {  // t: 256ths of an octave, > -2^14
  const double magic = 6755399441055744.0;  // 1.5 * 2^52: adding it rounds to an integer
  const double tm = t + magic;
  const int n = __double2loint(tm);
  const double f = t - (tm - magic);
  constexpr double ln = 0.693147180559945309417 / 256.0;
  const double q = f * fma(f, fma(f, ln * ln * ln / 6.0, ln * ln / 2.0), ln);
  double v = tab[n & 255];
  v = fma(v, q, v);
  v = __hiloint2double(__double2hiint(v) + ((n & ~255) << 12), __double2loint(v));  // times 2^(n >> 8)
  return (u64)__double_as_longlong(v + 4503599627370496.0);
}
__device__ __forceinline__ u64 weight_bits(float x, const Row& r, const double* tab) {
  return weight_bits_at(fmax((r.mx - (double)x) * r.c, -256.0 * 63.0), tab);
}
// As weight_bits for x within 44 T of the largest logit (44 log2(e) < 64 octaves).
__device__ __forceinline__ u64 weight_bits_near(float x, const Row& r, const double* tab) {
  return weight_bits_at((r.mx - (double)x) * r.c, tab);
}
__device__ __forceinline__ u64 weight(float x, const Row& r, const double* tab) {
  if (x == r.mxf) return 1ull << 40;
  if (!(x > -INFINITY) || r.mxf == INFINITY) return 0ull;
  return weight_bits(x, r, tab) - kMagicBits;
}
__device__ __forceinline__ u64 key_weight(uint32_t key, const Row& r, const double* tab) {
  return weight(key_value(key), r, tab);
}

// kBins bins of equal width in x, from `origin` down.
struct Bins {
  float origin, scale;  // bin position = (origin - x) * scale
};
// 64ths of a bin from the origin; monotone in x.
__device__ __forceinline__ uint32_t bin64(float x, const Bins& g) {
  const float pos = fminf((g.origin - x) * g.scale, (float)(kBins - 1));
  const uint32_t v = (uint32_t)__float_as_int(fmaf(pos, 64.0f, 8388608.0f)) & 0x7FFFFFu;  // 2^23: rounds
  return x == g.origin ? 0u : v;  // infinities and a scale beyond fp32 included
}
// The smallest key in (from, to] whose token lies before bin `bin`; `to` does.
// By a warp, 32 probes at a time.
__device__ __forceinline__ uint32_t bin_key(uint32_t bin, const Bins& g, uint32_t from, uint32_t to) {
  const uint32_t lane = threadIdx.x & 31;
  uint32_t lo = from, hi = to;  // `lo` does not, or bounds the search
  while (hi - lo > 1u) {
    const uint32_t step = (hi - lo + 31u) / 32u;
    const uint32_t probe = hi - lo <= step * (lane + 1u) ? hi : lo + step * (lane + 1u);
    const bool before = (bin64(key_value(probe), g) >> 6) < bin;
    const int first = __ffs(__ballot_sync(0xFFFFFFFFu, before)) - 1;  // lane 31 probes hi
    const uint32_t nhi = __shfl_sync(0xFFFFFFFFu, probe, first);
    const uint32_t nlo = __shfl_sync(0xFFFFFFFFu, probe, first > 0 ? first - 1 : 0);
    lo = first > 0 ? nlo : lo;
    hi = nhi;
  }
  return hi;
}
constexpr uint32_t kNoKey = 0x007FFFFFu;  // the keys up to this one are -inf and NaN

template <typename T>
__device__ __forceinline__ T warp_sum(T v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
  return v;
}

// Exclusive prefix over the block; the block's sum in `all`.
template <int kThreads>
__device__ __forceinline__ u64 block_scan(u64 v, Smem& s, u64& all) {
  constexpr int kWarps = kThreads / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  u64 inc = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const u64 o = __shfl_up_sync(0xFFFFFFFFu, inc, d);
    if (lane >= d) inc += o;
  }
  __syncthreads();
  if (lane == 31) s.red[0][warp] = inc;
  __syncthreads();
  u64 w = lane < kWarps ? s.red[0][lane] : 0ull;
#pragma unroll
  for (int d = 1; d < kWarps; d <<= 1) {
    const u64 o = __shfl_up_sync(0xFFFFFFFFu, w, d);
    if (lane >= d) w += o;
  }
  all = __shfl_sync(0xFFFFFFFFu, w, kWarps - 1);
  const u64 before = __shfl_sync(0xFFFFFFFFu, w, warp > 0 ? warp - 1 : 0);
  return (warp > 0 ? before : 0ull) + inc - v;
}

// Sorts n <= kListMax entries of `a` (bitonic, padded to a power of two), largest
// first or smallest first. Up to kThreads entries: one per thread in a register,
// partners less than a warp apart by shuffles, the others through `a`. More: in
// `a`, where a warp's 32 pairs of a stage lie in 64 entries of its own while
// partners are at most 32 apart, so that those stages need no block barrier.
template <int kThreads>
__device__ __forceinline__ void block_sort(u64* a, int n, bool descending) {
  const int tid = threadIdx.x;
  int p = 64;
  while (p < n) p <<= 1;
  __syncthreads();
  if (p <= kThreads) {
    const bool mine = tid < p;  // whole warps
    u64 x = tid < n ? a[tid] : (descending ? 0ull : ~0ull);
    const auto keep = [&](u64 y, int k, int j) {
      const bool small = ((tid & k) == 0) == ((tid & j) == 0);
      x = (x > y) == (small != descending) ? y : x;
    };
    for (int k = 2; k <= p; k <<= 1) {
      int j = k >> 1;
      for (; j >= 32; j >>= 1) {
        __syncthreads();
        if (mine) a[tid] = x;
        __syncthreads();
        if (mine) keep(a[tid ^ j], k, j);
      }
      if (mine) {
        for (; j > 0; j >>= 1) keep(__shfl_xor_sync(0xFFFFFFFFu, x, j), k, j);
      }
    }
    __syncthreads();
    if (mine) a[tid] = x;
    __syncthreads();
    return;
  }
  for (int i = n + tid; i < p; i += kThreads) a[i] = descending ? 0ull : ~0ull;
  __syncthreads();
  for (int k = 2; k <= p; k <<= 1) {
    for (int j = k >> 1; j > 0; j >>= 1) {
      for (int i = tid; i < (p >> 1); i += kThreads) {
        const int lo = 2 * i - (i & (j - 1)), hi = lo + j;
        const u64 x = a[lo], y = a[hi];
        const bool up = ((lo & k) == 0) != descending;
        if ((x > y) == up) {
          a[lo] = y;
          a[hi] = x;
        }
      }
      const int next = j > 1 ? j >> 1 : k;
      if (j > 32 || next > 32) __syncthreads();
      else __syncwarp();
    }
  }
  __syncthreads();
}

struct SampleParams {
  const void* logits;
  SampleHow how;
  const float* u;
  int64_t* tokens;
  float* logprobs;
  int64_t V, ld;
  int per;        // tokens per CTA
  int cluster;    // CTAs per row
};

template <int kThreads, bool kBf16, bool kResident>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) sample_kernel(const SampleParams p) {
  constexpr int kWarps = kThreads / 32;
  extern __shared__ __align__(128) uint8_t raw[];
  Smem& s = *reinterpret_cast<Smem*>(raw);
  const int C = p.cluster, rank = (int)(blockIdx.x % (unsigned)C);  // clusters are runs of C blocks
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int64_t b = blockIdx.x / C;
  const int64_t i0 = (int64_t)rank * p.per;
  const int64_t rest = p.V - i0;
  const int n = rest <= 0 ? 0 : (rest < p.per ? (int)rest : p.per);
  // Another CTA's shared memory may be touched once it has begun: waited for
  // below, before the first exchange.
  cluster_arrive();
  // What later passes start from.
  double2 tab2 = make_double2(0.0, 0.0);
  if (tid < 128) tab2 = __ldg(reinterpret_cast<const double2*>(kExp2Table.v) + tid);
  for (int i = tid; i < kBins; i += kThreads) s.hist[i] = 0u;
  if (tid < kBins / 8) s.slice[0][tid] = s.slice[1][tid] = 0u;
  if (tid == 0) s.list_n = s.local_n = 0u;
  // The launch may begin while the one before it runs; nothing that one may write
  // is read, and nothing is written, before it has ended.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // Only now may the next launch begin: whatever it does before its own wait, the
  // work before this one is behind it.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // ---- settings of the row (used after the row's loads are under way)
  const float T = p.how.temperature != nullptr ? p.how.temperature[b] : p.how.temperature_value;
  const int kset = p.how.top_k != nullptr ? p.how.top_k[b] : p.how.top_k_value;
  const float pset = p.how.top_p != nullptr ? p.how.top_p[b] : p.how.top_p_value;
  const float mset = p.how.min_p != nullptr ? p.how.min_p[b] : p.how.min_p_value;

  // ---- the row, once: logits (NaN as -inf, -0 as 0), their extremes, how many are in
  const char* row = static_cast<const char*>(p.logits) + (b * p.ld + i0) * (kBf16 ? 2 : 4);
  const auto clean = [](float x) { return fmaxf(x, -INFINITY) + 0.0f; };
  const auto load = [&](int i) {
    return clean(kBf16 ? bf16_bits_to_float(reinterpret_cast<const uint16_t*>(row)[i])
                       : reinterpret_cast<const float*>(row)[i]);
  };
  // Element i sits at data[i]: shifted so that 16-byte pieces of the row stay 16-byte pieces.
  constexpr int kVec = kBf16 ? 8 : 4;
  const int shift = (int)((reinterpret_cast<uintptr_t>(row) / (kBf16 ? 2 : 4)) & (kVec - 1));
  float* const base = reinterpret_cast<float*>(raw + sizeof(Smem));
  float* const data = base + shift;
  const auto at = [&](int i) { return kResident ? data[i] : load(i); };
  float fmx = -INFINITY, fmn = INFINITY;
  uint32_t valid = 0u;
  const auto note = [&](float x) {
    fmx = fmaxf(fmx, x);
    if (x > -INFINITY) {
      fmn = fminf(fmn, x);
      ++valid;
    }
  };
  if (kResident) {
    const int pieces = (n + shift + kVec - 1) / kVec;
    constexpr int kLoads = kBf16 ? 4 : 8;
    for (int v0 = tid; v0 < pieces; v0 += kThreads * kLoads) {
      uint4 q[kLoads];
#pragma unroll
      for (int j = 0; j < kLoads; ++j) {
        const int v = v0 + j * kThreads, e = v * kVec - shift;
        if (v < pieces && e >= 0 && e + kVec <= n)
          q[j] = *reinterpret_cast<const uint4*>(row + (int64_t)e * (kBf16 ? 2 : 4));
      }
#pragma unroll
      for (int j = 0; j < kLoads; ++j) {
        const int v = v0 + j * kThreads, e = v * kVec - shift;
        if (v >= pieces) break;
        if (e >= 0 && e + kVec <= n) {
          const uint32_t w[4] = {q[j].x, q[j].y, q[j].z, q[j].w};
          float f[kVec];
#pragma unroll
          for (int i = 0; i < kVec; ++i)
            f[i] = clean(kBf16 ? __uint_as_float((i & 1) ? w[i >> 1] & 0xFFFF0000u : w[i >> 1] << 16)
                               : __uint_as_float(w[i & 3]));
          float least = f[0], most = f[0];
#pragma unroll
          for (int i = 1; i < kVec; ++i) {
            least = fminf(least, f[i]);
            most = fmaxf(most, f[i]);
          }
          if (least > -INFINITY) {  // all are in
            fmn = fminf(fmn, least);
            fmx = fmaxf(fmx, most);
            valid += kVec;
          } else {
#pragma unroll
            for (int i = 0; i < kVec; ++i) note(f[i]);
          }
#pragma unroll
          for (int i = 0; i < kVec; i += 4)
            *reinterpret_cast<float4*>(base + v * kVec + i) = make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]);
        } else {  // the ragged ends
          for (int i = e < 0 ? 0 : e; i < e + kVec && i < n; ++i) {
            const float x = load(i);
            data[i] = x;
            note(x);
          }
        }
      }
    }
  } else {
    for (int i = tid; i < n; i += kThreads) note(load(i));
  }

  const bool greedy = !(T > 0.0f);
  const bool by_p = pset < 1.0f;  // false for NaN
  const double pp = pset > 0.0f ? (double)pset : 0.0;
  const u64 wmin = mset > 0.0f ? (u64)ceil((mset < 1.0f ? (double)mset : 1.0) * kWeightOne) : 0ull;

  if (tid < 128) reinterpret_cast<double2*>(s.tab)[tid] = tab2;

  // Three values of every CTA to all CTAs; one cluster barrier. The two buffers
  // alternate, so a CTA writes a buffer again only after every reader of it
  // has passed the barrier between.
  int par = 0;
  const auto exchange = [&](u64 va, u64 vb, u64 vc) {
    if (tid < C) {
      const uint32_t to = remote_addr(&s.xch[par][rank][0], tid);
      remote_store(to, va);
      remote_store(to + 8, vb);
      remote_store(to + 16, vc);
    }
    cluster_sync();
  };
  u64 before_me = 0;  // the first sum over the CTAs before this one
  const auto gather_sums = [&]() {
    Sums t = {0, 0, 0};
    before_me = 0;
    for (int r = 0; r < C; ++r) {
      if (r == rank) before_me = t.a;
      t.a += s.xch[par][r][0];
      t.b += s.xch[par][r][1];
      t.c += s.xch[par][r][2];
    }
    par ^= 1;
    return t;
  };
  const auto cluster_sum = [&](Sums v) {
    v.a = warp_sum(v.a);
    v.b = warp_sum(v.b);
    __syncthreads();  // v.c: one value per CTA
    if (lane == 0) {
      s.red[0][wid] = v.a;
      s.red[1][wid] = v.b;
    }
    __syncthreads();
    if (wid == 0) {
      v.a = warp_sum(lane < kWarps ? s.red[0][lane] : 0ull);
      v.b = warp_sum(lane < kWarps ? s.red[1][lane] : 0ull);
    }
    exchange(v.a, v.b, v.c);  // threads of warp 0 send
    return gather_sums();
  };
  uint32_t kmax, kmin;
  {
    kmax = sample_key(fmx);
    kmin = fmn < INFINITY ? sample_key(fmn) : (valid != 0u ? sample_key(INFINITY) : 0xFFFFFFFFu);
    kmax = __reduce_max_sync(0xFFFFFFFFu, kmax);
    kmin = __reduce_min_sync(0xFFFFFFFFu, kmin);
    valid = __reduce_add_sync(0xFFFFFFFFu, valid);
    if (lane == 0) {
      s.red[0][wid] = kmax;
      s.red[1][wid] = kmin;
      s.red[2][wid] = valid;
    }
    __syncthreads();
    if (wid == 0) {
      kmax = __reduce_max_sync(0xFFFFFFFFu, lane < kWarps ? (uint32_t)s.red[0][lane] : 0u);
      kmin = __reduce_min_sync(0xFFFFFFFFu, lane < kWarps ? (uint32_t)s.red[1][lane] : 0xFFFFFFFFu);
      valid = __reduce_add_sync(0xFFFFFFFFu, lane < kWarps ? (uint32_t)s.red[2][lane] : 0u);
    }
    cluster_wait();
    exchange(kmax, kmin, valid);
    kmax = 0u;
    kmin = 0xFFFFFFFFu;
    valid = 0u;
    for (int r = 0; r < C; ++r) {
      kmax = max(kmax, (uint32_t)s.xch[par][r][0]);
      kmin = min(kmin, (uint32_t)s.xch[par][r][1]);
      valid += (uint32_t)s.xch[par][r][2];
    }
    par ^= 1;
  }
  if (kmax == 0u) {
    if (rank == 0 && tid == 0) {
      p.tokens[b] = -1;
      if (p.logprobs != nullptr) p.logprobs[b] = -INFINITY;
    }
    return;
  }
  Row r;
  r.top = kmax;
  r.mxf = key_value(kmax);
  r.mx = (double)r.mxf;
  const double inv_t = 1.0 / (double)T;
  r.c = greedy ? 0.0 : -369.329930467574631 * inv_t;  // 256 log2(e)

  const auto finish = [&](int64_t token, float x, u64 total) {
    p.tokens[b] = token;
    if (p.logprobs != nullptr) {
      const double d = x == r.mxf ? 0.0 : ((double)x - r.mx) / (double)T;
      p.logprobs[b] = greedy ? 0.0f : (float)(d - log((double)total / kWeightOne));
    }
  };
  const auto target_of = [&](u64 total) {
    const float ub = p.u[b];
    u64 t = ub > 0.0f ? (ub < 1.0f ? (u64)((double)ub * (double)total) : total - 1) : 0ull;
    return t < total ? t : total - 1;
  };

  if (greedy) {  // the first token with the largest logit
    uint32_t first = 0xFFFFFFFFu;
    for (int i = tid; i < n; i += kThreads)
      if (at(i) == r.mxf) first = min(first, (uint32_t)(i0 + i));
    first = __reduce_min_sync(0xFFFFFFFFu, first);
    __syncthreads();
    if (lane == 0) s.red[0][wid] = first;
    __syncthreads();
    if (wid == 0) first = __reduce_min_sync(0xFFFFFFFFu, lane < kWarps ? (uint32_t)s.red[0][lane] : 0xFFFFFFFFu);
    exchange(first, 0, 0);
    if (rank == 0 && tid == 0) {
      uint32_t f = 0xFFFFFFFFu;
      for (int c = 0; c < C; ++c) f = min(f, (uint32_t)s.xch[par][c][0]);
      finish((int64_t)f, r.mxf, 1ull << 40);
    }
    return;
  }

  const float span = r.mxf < INFINITY ? r.mxf - key_value(kmin) : 0.0f;  // may round to infinity
  const float reach = fminf((float)kTail * T, span);  // the bins' range, in x
  const bool tail_out = reach < span;                 // the last bin's weights are all zero
  const Bins whole{r.mxf, span > 0.0f ? (float)(kBins - 1) / reach : 1.0f};
  // A histogram word: a count above `packed` bits of a sum of 64ths of a bin (13 +
  // 19 bits), of sixteenths where a CTA has more tokens (14 + 18), or a count alone.
  const int packed = p.per <= kPackMax / 2 ? 19 : (p.per <= kPackMax ? 18 : 0);
  const uint32_t drop = packed == 18 ? 2u : 0u;

  // The kept tokens so far: x > cut and the first `ties` with x == cut.
  float cut = -INFINITY;
  u64 ties = 0;
  bool partial = true;  // more tokens than `ties` are at the cut
  bool by_k = kset > 0 && (uint32_t)kset < valid;

  // Histogram of the tokens with lo <= x < hi (no upper end for a NaN), to every
  // CTA. Each adds up its share of the bins over the cluster and sends it to all:
  // an atomic per bin and CTA on one of them took four times as long, and with
  // the row's histogram everywhere no verdict has to be sent around.
  const auto histogram = [&](const Bins& g, float lo, float hi) {
    if (packed != 0 && lo == -INFINITY && !(hi < INFINITY) && valid == (uint32_t)p.V && g.scale < INFINITY &&
        g.origin < INFINITY) {
      // As below, where nothing has to be left out and no place is special.
#pragma unroll 4
      for (int i = tid; i < n; i += kThreads) {
        const float pos = fminf((g.origin - at(i)) * g.scale, (float)(kBins - 1));
        const uint32_t v = (uint32_t)__float_as_int(fmaf(pos, 64.0f, 8388608.0f));
        atomicAdd(&s.hist[(v >> 6) & (kBins - 1)], (1u << packed) + ((v & 63u) >> drop));
      }
    } else {
#pragma unroll 4
      for (int i = tid; i < n; i += kThreads) {
        const float x = at(i);
        if (x >= lo && x > -INFINITY && !(x >= hi)) {
          const uint32_t v = bin64(x, g);
          atomicAdd(&s.hist[v >> 6], packed != 0 ? (1u << packed) + ((v & 63u) >> drop) : 1u);
        }
      }
    }
    cluster_sync();
    const int share = kBins / C;  // bins of this CTA
    const int groups = share <= kBins / 8 ? kThreads / share : 1, sources = C / groups;  // several from 8 CTAs on
    for (int k = tid; k < share * groups; k += kThreads) {
      const int bin = rank * share + k % share, from = k / share * sources;
      uint32_t c = 0u, o = 0u;
      for (int q = 0; q < sources; ++q) {
        const uint32_t h = remote_load(remote_addr(&s.hist[bin], from + q));
        c += packed != 0 ? h >> packed : h;
        o += packed != 0 ? h & ((1u << packed) - 1u) : h;
      }
      if (groups == 1) {
        for (int q = 0; q < C; ++q) {
          remote_store(remote_addr(&s.cnt[bin], q), c);
          remote_store(remote_addr(&s.off[bin], q), o);
        }
      } else if (c != 0u) {
        atomicAdd(&s.slice[0][k % share], c);
        atomicAdd(&s.slice[1][k % share], o);
      }
    }
    if (groups > 1) {
      __syncthreads();
      for (int k = tid; k < share * C; k += kThreads) {
        const int bin = k % share, to = k / share;
        remote_store(remote_addr(&s.cnt[rank * share + bin], to), s.slice[0][bin]);
        remote_store(remote_addr(&s.off[rank * share + bin], to), s.slice[1][bin]);
      }
      __syncthreads();
      if (tid < share) s.slice[0][tid] = s.slice[1][tid] = 0u;
    }
    cluster_sync();
  };
  // Ready for another histogram (its predecessor's readers are past a cluster barrier).
  const auto clear_histogram = [&]() {
    __syncthreads();
    for (int i = tid; i < kBins; i += kThreads) s.hist[i] = 0u;
    if (tid == 0) s.local_n = 0u;
    __syncthreads();
  };
  constexpr int kPerThread = kBins / kThreads;  // neighbouring bins of a thread
  const auto collect = [&](int i, float x) {
    const uint32_t slot = atomicAdd(&s.local_n, 1u);
    if (slot < (uint32_t)kListMax) s.local[slot] = ((u64)sample_key(x) << 32) | (0xFFFFFFFFu - (uint32_t)(i0 + i));
  };
  // This CTA's candidates to the lists of the first `to` CTAs; complete after a
  // cluster barrier. Returns how many.
  const auto flush = [&](int to) {
    __syncthreads();
    const uint32_t m = s.local_n < (uint32_t)kListMax ? s.local_n : (uint32_t)kListMax;
    if (m != 0u) {
      if (tid == 0) s.base = remote_add(remote_addr(&s.list_n, 0), m);
      __syncthreads();
      const uint32_t at0 = s.base;
      for (uint32_t k = tid; k < m * to; k += kThreads) {
        const uint32_t i = k % m, q = k / m;
        if (at0 + i < (uint32_t)kListMax) remote_store(remote_addr(&s.list[at0 + i], (int)q), s.local[i]);
      }
    }
    return (u64)m;
  };
  // From a list of m candidates, which holds every kept token: apply
  // top-k (keep), top-p (of row_total, or of the kept ones' sum) and min-p, and draw.
  const auto draw_from_list = [&](int m, int keep, bool use_p, bool own_total, u64 row_total) {
    block_sort<kThreads>(s.list, m, true);
    keep = keep < m ? keep : m;
    for (int i = tid; i < kListMax; i += kThreads)
      s.wlist[i] = i < keep ? key_weight((uint32_t)(s.list[i] >> 32), r, s.tab) : 0ull;
    __syncthreads();
    constexpr int kE = kListMax / kThreads;
    if (use_p) {
      u64 w[kE], sum = 0, all;
#pragma unroll
      for (int j = 0; j < kE; ++j) sum += w[j] = s.wlist[tid * kE + j];
      u64 run = block_scan<kThreads>(sum, s, all);
      const double want = ceil(pp * (double)(own_total ? all : row_total));
      const u64 need = want > 1.0 ? (u64)want : 1ull;
#pragma unroll
      for (int j = 0; j < kE; ++j) {
        if (run >= need) s.wlist[tid * kE + j] = 0ull;  // the prefix before it reaches the sum
        run += w[j];
      }
      __syncthreads();
    }
    // Index order: sort index << 32 | place, then scan the weights in that order.
    for (int i = tid; i < m; i += kThreads) {
      const u64 w = s.wlist[i];
      const uint32_t idx = 0xFFFFFFFFu - (uint32_t)s.list[i];
      s.list[i] = w == 0ull || w < wmin ? ~0ull : ((u64)idx << 32) | (uint32_t)i;
    }
    block_sort<kThreads>(s.list, m, false);
    u64 w[kE], sum = 0, total;
#pragma unroll
    for (int j = 0; j < kE; ++j) {
      const int i = tid * kE + j;
      const u64 e = i < m ? s.list[i] : ~0ull;
      w[j] = e == ~0ull ? 0ull : s.wlist[(uint32_t)e];
      sum += w[j];
    }
    u64 run = block_scan<kThreads>(sum, s, total);
    const u64 target = target_of(total);
#pragma unroll
    for (int j = 0; j < kE; ++j) {
      if (run <= target && target < run + w[j]) {
        const int64_t idx = (int64_t)(s.list[tid * kE + j] >> 32);
        const char* src = static_cast<const char*>(p.logits) + (b * p.ld + idx) * (kBf16 ? 2 : 4);
        finish(idx,
               clean(kBf16 ? bf16_bits_to_float(*reinterpret_cast<const uint16_t*>(src))
                           : *reinterpret_cast<const float*>(src)),
               total);
      }
      run += w[j];
    }
  };
  // From a list of the m tokens of consecutive bins: the border after the
  // shortest run, largest first, of `need` tokens, or of weight `need`, which the
  // list holds. Every CTA has the list and comes to the same border. Digits of the
  // key from the top, kDigits values each: weights added up per value, the value
  // that holds the border, then its keys alone (two rounds for most rows; a sort of
  // 800 candidates in all CTAs took a quarter of a row's time, 21000 of 85000 cycles).
  // False, and nothing settled, where the list does not hold the border.
  const auto settle = [&](int m, u64 need, bool by_weight) {
    constexpr int kE = kListMax / kThreads;
    uint32_t key[kE];
    u64 w[kE];
    uint32_t hk = 0u, lk = 0xFFFFFFFFu;
#pragma unroll
    for (int j = 0; j < kE; ++j) {
      const int i = tid + j * kThreads;
      key[j] = i < m ? (uint32_t)(s.list[i] >> 32) : 0u;
      w[j] = i < m ? (by_weight ? key_weight(key[j], r, s.tab) : 1ull) : 0ull;
      if (i < m) {
        hk = max(hk, key[j]);
        lk = min(lk, key[j]);
      }
    }
    hk = __reduce_max_sync(0xFFFFFFFFu, hk);
    lk = __reduce_min_sync(0xFFFFFFFFu, lk);
    if (lane == 0) s.red[1][wid] = ((u64)hk << 32) | lk;
    __syncthreads();
    {
      const u64 v = lane < kWarps ? s.red[1][lane] : 0xFFFFFFFFull;
      hk = __reduce_max_sync(0xFFFFFFFFu, (uint32_t)(v >> 32));
      lk = __reduce_min_sync(0xFFFFFFFFu, (uint32_t)v);
    }
    for (int round = 0; round < (32 + kDigitBits - 1) / kDigitBits; ++round) {
      const int width = 32 - __clz(hk - lk);  // bits that differ
      const int sh = width > kDigitBits ? width - kDigitBits : 0;
      for (int i = tid; i < 2 * kDigits; i += kThreads) s.digit[i] = 0u;
      __syncthreads();
#pragma unroll
      for (int j = 0; j < kE; ++j) {
        if (w[j] != 0ull && key[j] >= lk && key[j] <= hk) {
          // 1024 weights of up to 2^40, in two words of 20 bits and the rest.
          const uint32_t d = (hk - key[j]) >> sh;
          if (by_weight) {
            atomicAdd(&s.digit[d], (uint32_t)w[j] & 0xFFFFFu);
            atomicAdd(&s.digit[kDigits + d], (uint32_t)(w[j] >> 20));
          } else {
            atomicAdd(&s.digit[d], 1u);
          }
        }
      }
      __syncthreads();
      const u64 mine = tid < kDigits ? s.digit[tid] + ((u64)s.digit[kDigits + tid] << 20) : 0ull;
      u64 all;
      const u64 run = block_scan<kThreads>(mine, s, all);
      if (need - 1ull >= all) return false;  // none, or more than the list weighs
      if (run < need && run + mine >= need) {
        const uint32_t top = hk - ((uint32_t)tid << sh), span = (1u << sh) - 1u;
        s.hi_key = top;
        s.lo_key = top - lk > span ? top - span : lk;
        s.need = need - run;
        s.count = mine;  // weight of the value's tokens
      }
      __syncthreads();
      hk = s.hi_key;
      lk = s.lo_key;
      need = s.need;
      if (sh == 0) break;
    }
    const u64 each = by_weight ? key_weight(hk, r, s.tab) : 1ull, weight_all = s.count;
    __syncthreads();
    if (tid == 0) s.list_n = s.local_n = 0u;
    cut = key_value(hk);
    ties = (need + each - 1) / each;
    partial = ties * each < weight_all;
    __syncthreads();
    return true;
  };
  // The border without a list (more equal or near tokens than one holds):
  // bisection over the keys, a pass each. All CTAs take part and agree.
  const auto bisect = [&](u64 need, bool by_weight) {
    const float cut0 = cut;
    const u64 ties0 = ties;
    const bool partial0 = partial;
    const uint32_t key0 = cut0 > -INFINITY ? sample_key(cut0) : 1u;
    const auto sums = [&](uint32_t from, u64& reached, u64& equal) {  // kept tokens >= from; those == from
      Sums v = {0, 0, 0};
      for (int i = tid; i < n; i += kThreads) {
        const float x = at(i);
        const uint32_t key = sample_key(x);
        if (key < from || key == 0u || (partial0 && x == cut0)) continue;
        v.a += by_weight ? weight(x, r, s.tab) : 1ull;
        if (key == from) ++v.b;
      }
      v = cluster_sum(v);
      if (partial0 && from <= key0) {
        v.a += ties0 * (by_weight ? weight(cut0, r, s.tab) : 1ull);
        if (from == key0) v.b += ties0;
      }
      reached = v.a;
      equal = v.b;
    };
    uint32_t lo = key0, hi = r.top;  // the largest key from which on the need is reached
    u64 got, eq;
    while (lo < hi) {
      const uint32_t mid = lo + (hi - lo + 1u) / 2u;
      sums(mid, got, eq);
      if (got >= need) lo = mid;
      else hi = mid - 1u;
    }
    sums(lo, got, eq);
    const u64 w = by_weight ? key_weight(lo, r, s.tab) : 1ull;
    const u64 above = got - eq * w;
    u64 want = w > 0 ? (need - above + w - 1) / w : eq;
    want = want < 1 ? 1 : want;
    partial = want < eq || (partial0 && lo == key0);
    cut = key_value(lo);
    ties = want;
  };

  // Keys of the logits in bins s.bin_lo .. s.bin_hi: [lo_key, hi_key), within [from, to).
  const auto bin_range = [&](const Bins& g, uint32_t from, uint32_t to) {
    const uint32_t top = to == 0xFFFFFFFFu ? r.top : to - 1u;  // lies in bin 0
    const uint32_t below = from > kNoKey ? from - 1u : kNoKey;
    if (wid == 0) {
      const uint32_t k = s.bin_lo == 0 ? to : bin_key((uint32_t)s.bin_lo, g, below, top);
      if (lane == 0) s.hi_key = k;
    } else if (wid == 1) {
      const uint32_t k = s.bin_hi == kBins - 1 ? from : bin_key((uint32_t)s.bin_hi + 1u, g, below, top);
      if (lane == 0) s.lo_key = k;
    }
    __syncthreads();
  };
  // The bin of the need-th token of the histogram, and what to do about it.
  const auto place_count = [&](u64 need, bool may_whole) {
    u64 mine[kPerThread], sum = 0, all;
#pragma unroll
    for (int j = 0; j < kPerThread; ++j) sum += mine[j] = s.cnt[tid * kPerThread + j];
    u64 run = block_scan<kThreads>(sum, s, all);
#pragma unroll
    for (int j = 0; j < kPerThread; ++j) {
      if (run < need && run + mine[j] >= need) {
        const int bin = tid * kPerThread + j;
        s.mode = may_whole && run + mine[j] <= (by_p ? 2 : 1) * kWholeMax ? kWhole
                 : mine[j] <= kListMax                                ? kBorder
                 : may_whole && bin == kBins - 1 && tail_out          ? kZeros
                                                                      : kCrowd;
        s.bin_hi = bin;
        s.bin_lo = s.mode == kWhole ? 0 : bin;
        s.need = need - run;  // how many of the bin's tokens stay
        s.count = mine[j];    // of how many
      }
      run += mine[j];
    }
    __syncthreads();
  };
  // The bins in which a running weight meets a target, by bounds of every bin's
  // weight (bin_weight). `first` is the weight at the bins' origin. The target is
  // share * total (target < 0) or a weight. In fp32: the exponent (up to 29) has
  // three roundings and expf two ulp, under 6e-6, a bound's own arithmetic, the
  // additions of a prefix (14 deep) and the comparison under 2e-6; the borders are
  // widened by 2e-5 on either side.
  const auto place_weight = [&](const Bins& g, float first, float target, bool may_whole, bool open_end) {
    // Exponent per bin (no bins to speak of where all tokens are equal or T is infinite).
    const float inv_tf = (float)inv_t;
    const float delta = g.scale < INFINITY && inv_tf > 0.0f ? fminf(inv_tf / g.scale, 1.0f) : 0.0f;
    // T and the span so large that their bins' range is infinite: the first bin and
    // the last hold tokens at any distance, and a bin's weight is between none and all.
    const bool blind = !(g.scale > 0.0f);
    const BinPlaces places = bin_places(packed);
    const float step = expf(-delta);
    float e = first * expf(-delta * (float)(tid * kPerThread));
    float lo[kPerThread], hi[kPerThread], slo = 0.f, shi = 0.f;
    uint32_t mine[kPerThread], cnt = 0;
    const uint32_t cut_bin = cut > -INFINITY && partial ? bin64(cut, g) >> 6 : 0xFFFFFFFFu;
#pragma unroll
    for (int j = 0; j < kPerThread; ++j) {
      const int bin = tid * kPerThread + j;
      cnt += mine[j] = s.cnt[bin];
      const WeightBounds w = bin_weight(e, delta, places, mine[j], s.off[bin]);
      lo[j] = blind ? 0.f : w.lo;
      hi[j] = blind ? first * (float)mine[j] : w.hi;
      if ((open_end && bin == kBins - 1) || (uint32_t)bin == cut_bin) lo[j] = 0.f;
      slo += lo[j];
      shi += hi[j];
      e *= step;
    }
    float plo = slo, phi = shi;  // prefixes of both, and of the counts
    uint32_t run = cnt;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const float x = __shfl_up_sync(0xFFFFFFFFu, plo, d), y = __shfl_up_sync(0xFFFFFFFFu, phi, d);
      const uint32_t z = __shfl_up_sync(0xFFFFFFFFu, run, d);
      if (lane >= d) {
        plo += x;
        phi += y;
        run += z;
      }
    }
    if (lane == 31) {
      s.redf[0][wid] = plo;
      s.redf[1][wid] = phi;
      s.red[0][wid] = run;
    }
    if (tid == 0) s.bin_lo = s.bin_hi = kBins - 1;
    __syncthreads();
    float wlo = lane < kWarps ? s.redf[0][lane] : 0.f, whi = lane < kWarps ? s.redf[1][lane] : 0.f;
    uint32_t wrun = lane < kWarps ? (uint32_t)s.red[0][lane] : 0u;
#pragma unroll
    for (int d = 1; d < kWarps; d <<= 1) {
      const float x = __shfl_up_sync(0xFFFFFFFFu, wlo, d), y = __shfl_up_sync(0xFFFFFFFFu, whi, d);
      const uint32_t z = __shfl_up_sync(0xFFFFFFFFu, wrun, d);
      if (lane >= d) {
        wlo += x;
        whi += y;
        wrun += z;
      }
    }
    const float tlo = __shfl_sync(0xFFFFFFFFu, wlo, kWarps - 1), thi = __shfl_sync(0xFFFFFFFFu, whi, kWarps - 1);
    const int prev = wid > 0 ? wid - 1 : 0;
    const float blo_f = __shfl_sync(0xFFFFFFFFu, wlo, prev), bhi_f = __shfl_sync(0xFFFFFFFFu, whi, prev);
    const uint32_t brun = __shfl_sync(0xFFFFFFFFu, wrun, prev);
    plo += (wid > 0 ? blo_f : 0.f) - slo;
    phi += (wid > 0 ? bhi_f : 0.f) - shi;
    run += (wid > 0 ? brun : 0u) - cnt;
    int first_lo = kBins - 1, first_hi = kBins - 1;
    const float want_lo = target < 0.f ? (float)pp * tlo : target, want_hi = target < 0.f ? (float)pp * thi : target;
#pragma unroll
    for (int j = 0; j < kPerThread; ++j) {
      const int bin = tid * kPerThread + j;
      if ((phi + hi[j]) * (1.0f + 2e-5f) >= want_lo * (1.0f - 2e-5f)) first_lo = min(first_lo, bin);
      if ((plo + lo[j]) * (1.0f - 2e-5f) >= want_hi * (1.0f + 2e-5f)) first_hi = min(first_hi, bin);
      plo += lo[j];
      phi += hi[j];
    }
    first_lo = __reduce_min_sync(0xFFFFFFFFu, first_lo);
    first_hi = __reduce_min_sync(0xFFFFFFFFu, first_hi);
    if (lane == 0 && first_lo < kBins - 1) atomicMin(&s.bin_lo, first_lo);
    if (lane == 0 && first_hi < kBins - 1) atomicMin(&s.bin_hi, first_hi);
    __syncthreads();
    const int blo = s.bin_lo, bhi = s.bin_hi;
#pragma unroll
    for (int j = 0; j < kPerThread; ++j) {
      const int bin = tid * kPerThread + j;
      if (bin == blo) s.red[1][0] = run;            // tokens before the candidates' bins
      if (bin == bhi) s.red[1][1] = run + mine[j];  // and through them
      run += mine[j];
    }
    __syncthreads();
    const uint32_t before = (uint32_t)s.red[1][0], through = (uint32_t)s.red[1][1];
    const uint32_t mode = may_whole && through <= kWholeMax ? kWhole : (through - before <= kListMax ? kBorder : kCrowd);
    if (tid == 0) {
      s.mode = mode;
      s.count = through - before;
      if (mode == kWhole) s.bin_lo = 0;
    }
    __syncthreads();
  };
  // The border among the `count` tokens of keys [lk, hk), more than a list holds:
  // finer bins over that range, until a list holds a bin's tokens or all have one
  // value.
  const auto zoom = [&](u64 need, bool by_weight, uint32_t lk, uint32_t hk, u64 count) {
    for (int level = 0; level < 4; ++level) {
      lk = max(max(lk, kmin), cut > -INFINITY ? sample_key(cut) : 0u);
      if (by_weight) lk = max(lk, sample_key(r.mxf - (float)kTail * T));  // weights below are zero
      const uint32_t last = hk == 0xFFFFFFFFu ? r.top : hk - 1u;
      if (lk >= last) {  // ties
        const u64 w = by_weight ? key_weight(last, r, s.tab) : 1ull;
        if (w == 0ull) break;
        cut = key_value(last);
        ties = (need + w - 1) / w;
        partial = ties < count;
        return true;
      }
      const float lo_v = key_value(lk), hi_v = key_value(last);
      const float width = hi_v - lo_v;
      if (!(width > 0.0f && width < INFINITY)) break;
      const Bins g{hi_v, (float)(kBins - 1) / width};
      const float hi_x = hk == 0xFFFFFFFFu ? __uint_as_float(0x7FC00000u) : key_value(hk);
      clear_histogram();
      histogram(g, lo_v, hi_x);
      if (by_weight)
        place_weight(g, (float)((double)key_weight(last, r, s.tab) / kWeightOne), (float)((double)need / kWeightOne),
                     false, false);
      else
        place_count(need, false);
      bin_range(g, lk, hk);
      const uint32_t mode = s.mode, nlk = s.lo_key, nhk = s.hi_key;
      count = s.count;
      const u64 in_bin = s.need;
      const bool list = mode == kBorder;
      Sums v = {0, 0, 0};
      for (int i = tid; i < n; i += kThreads) {
        const float x = at(i);
        const uint32_t key = sample_key(x);
        if (key < nlk || key >= hk) continue;
        if (key >= nhk) v.b += by_weight ? weight(x, r, s.tab) : 0ull;
        else if (list) collect(i, x);
      }
      if (list) v.c = flush(C);
      v = cluster_sum(v);
      if (by_weight && v.b >= need) return false;
      need = by_weight ? need - v.b : in_bin;
      if (list) return settle((int)v.c, need, by_weight);
      if (nlk == lk && nhk == hk) break;
      lk = nlk;
      hk = nhk;
    }
    return false;
  };

  // ---- top-k
  if (by_k) {
    histogram(whole, -INFINITY, __uint_as_float(0x7FC00000u));
    place_count((u64)kset, true);
    const uint32_t mode = s.mode, b0 = (uint32_t)s.bin_lo, b1 = (uint32_t)s.bin_hi;
    const u64 in_bin = s.need, count = s.count;
    if (mode == kWhole || mode == kBorder) {
#pragma unroll 4
      for (int i = tid; i < n; i += kThreads) {
        const float x = at(i);
        const uint32_t bin = bin64(x, whole) >> 6;
        if (x > -INFINITY && bin >= b0 && bin <= b1) collect(i, x);
      }
      const u64 m = cluster_sum(Sums{0, 0, flush(mode == kWhole ? 1 : C)}).c;
      if (mode == kWhole) {
        if (rank == 0) draw_from_list((int)m, kset, by_p, true, 0ull);
        return;
      }
      settle((int)m, in_bin, false);
    } else if (mode == kCrowd) {
      bin_range(whole, 1u, 0xFFFFFFFFu);
      if (!zoom(in_bin, false, s.lo_key, s.hi_key, count)) bisect((u64)kset, false);
    }
    if (by_p) clear_histogram();  // again, of what is left
  }

  // Thread t owns tokens [t * own, (t + 1) * own) of the CTA's stretch from here
  // on: an odd number of shared-memory words, so that a warp's reads meet no
  // bank twice.
  const int own = ((n + kThreads - 1) / kThreads) | 1;
  const int t0 = own * tid < n ? own * tid : n, t1 = t0 + own < n ? t0 + own : n;
  u64 sure = 0;           // weight of the thread's tokens that are kept whatever the border
  uint32_t sure_to = 0u;  // those at places before this one
  int listed = 0;         // the kept tokens at other places are among this many in the list

  // ---- top-p
  if (by_p) {
    histogram(whole, cut, __uint_as_float(0x7FC00000u));
    place_weight(whole, 1.0f, -1.0f, true, true);
    const uint32_t mode = s.mode;
    const u64 count = s.count;
    sure_to = (uint32_t)s.bin_lo << 6;  // kept whatever the border: places before it
    const uint32_t to = ((uint32_t)s.bin_hi + 1u) << 6;  // candidates: places from there to here
    // One pass with an exponential per token: the sum of all kept tokens, of
    // those above the candidates, and the candidates. A sum of weight bits holds
    // kMagicBits once per token, taken off at the end; the largest logit
    // and those beside an infinite one take no exponential.
    Sums v = {0, 0, 0};
    const bool list = mode != kCrowd;
    const float floor_x = r.mxf - 44.0f * T;  // weights from here down are zero
    if (wmin == 0 && r.mxf < INFINITY && floor_x > -0x1p126f && r.mxf - floor_x >= 30.0f * T) {
      // The usual settings (44 T is above the rounding of the largest logit): what is not kept weighs what floor_x does, nothing.
      // Sums of weight bits hold kMagicBits once per token, taken off at the end.
      const float first = cut > -INFINITY ? (partial ? nextafterf(cut, INFINITY) : cut) : floor_x;
      const int above_to = (int)(0x4B000000u + sure_to);  // a place as bits of 2^23 + place
      const int list_to = list ? (int)(0x4B000000u + to) : 0;
      u64 all_bits = 0, above_bits = 0;
      uint32_t above_n = 0;
#pragma unroll 4
      for (int i = t0; i < t1; ++i) {
        const float x = at(i);
        const float y = fmaxf(x >= first ? x : floor_x, floor_x);
        const u64 w = weight_bits_near(y, r, s.tab);
        all_bits += w;
        const float pos = fminf((whole.origin - x) * whole.scale, (float)(kBins - 1));
        const int place = x == whole.origin ? 0x4B000000 : __float_as_int(fmaf(pos, 64.0f, 8388608.0f));
        if (place < above_to) {
          above_bits += w;
          ++above_n;
        } else if (place < list_to && x >= cut && x > -INFINITY) {
          collect(i, x);
        }
      }
      v.a = all_bits - (u64)(t1 - t0) * kMagicBits;
      sure = v.b = above_bits - (u64)above_n * kMagicBits;
    } else {
      const bool inf = r.mxf == INFINITY;
      for (int i = t0; i < t1; ++i) {
        const float x = at(i);
        u64 w = weight_bits(x, r, s.tab) - kMagicBits;  // of -inf: zero
        w = inf ? 0ull : w;
        w = x == r.mxf ? 1ull << 40 : w;
        w = x >= cut ? w : 0ull;
        const uint32_t place = bin64(x, whole);
        const bool above = place < sure_to;
        v.a += partial && x == cut ? 0ull : w;  // a tie of top-k's border is counted by its rank
        v.b += above ? w : 0ull;
        sure += above && w >= wmin ? w : 0ull;
        if (list && !above && place < to && x >= cut && x > -INFINITY) collect(i, x);
      }
    }
    if (list) v.c = flush(mode == kWhole ? 1 : C);
    v = cluster_sum(v);  // its barrier also completes the list
    const u64 total = v.a + (partial && ties > 0 ? ties * weight(cut, r, s.tab) : 0ull);
    const double want = ceil(pp * (double)total);
    const u64 need = want > 1.0 ? (u64)want : 1ull;
    if (mode == kWhole) {
      // All that can stay is in the list; top-k's border cuts it at kset tokens.
      if (rank == 0) draw_from_list((int)v.c, by_k ? kset : kListMax, true, false, total);
      return;
    }
    bool settled = v.b < need;
    if (settled && mode == kBorder) {
      settled = settle((int)v.c, need - v.b, true);
      if (settled && !partial) listed = (int)v.c;
    } else if (settled) {
      bin_range(whole, 1u, 0xFFFFFFFFu);
      settled = zoom(need - v.b, true, s.lo_key, s.hi_key, count);
    }
    if (!settled) {
      bisect(need, true);
      sure = 0;
      sure_to = 0u;
    }
  }

  // ---- the draw, in index order
  u64 tie = 0;  // rank of the thread's first token at the cut
  const bool ranked = partial && ties > 0;
  if (ranked) {
    u64 mine = 0, all;
    for (int i = t0; i < t1; ++i) mine += at(i) == cut ? 1 : 0;
    tie = block_scan<kThreads>(mine, s, all);
    exchange(all, 0, 0);
    gather_sums();
    tie += before_me;
  }
  const auto kept_weight = [&](float x, u64 rank_of_tie) {
    if (!(x >= cut) || !(x > -INFINITY) || (partial && x == cut && rank_of_tie >= ties)) return 0ull;
    const u64 w = weight(x, r, s.tab);
    return w >= wmin ? w : 0ull;
  };
  u64 sum = sure, tr = tie;
  if (listed != 0) {
    // To the threads that own them, in two words as above; a pass over all tokens
    // took a tenth of a row's time.
    for (int i = tid; i < 2 * kThreads; i += kThreads) s.part[i] = 0u;
    __syncthreads();
    const uint32_t cut_key = sample_key(cut);
    for (int i = tid; i < listed; i += kThreads) {
      const u64 e = s.list[i];
      const int at_i = (int)((int64_t)(0xFFFFFFFFu - (uint32_t)e) - i0);
      if ((uint32_t)(e >> 32) < cut_key || at_i < 0 || at_i >= n) continue;
      const u64 w = key_weight((uint32_t)(e >> 32), r, s.tab);
      if (w < wmin) continue;
      atomicAdd(&s.part[at_i / own], (uint32_t)w & 0xFFFFFu);
      atomicAdd(&s.part[kThreads + at_i / own], (uint32_t)(w >> 20));
    }
    __syncthreads();
    sum += s.part[tid] + ((u64)s.part[kThreads + tid] << 20);
  } else {
#pragma unroll 4
    for (int i = t0; i < t1; ++i) {
      const float x = at(i);
      if (x >= cut && bin64(x, whole) >= sure_to) {
        sum += kept_weight(x, tr);
        if (x == cut) ++tr;
      }
    }
  }
  u64 mine_all;
  u64 run = block_scan<kThreads>(sum, s, mine_all);
  exchange(mine_all, 0, 0);
  const u64 total = gather_sums().a, target = target_of(total);
  run += before_me;
  // The warp whose lane's stretch holds the target walks that stretch together.
  const uint32_t hit = __ballot_sync(0xFFFFFFFFu, run <= target && target < run + sum);
  if (hit != 0u) {
    const int from = __ffs(hit) - 1;
    const int a0 = __shfl_sync(0xFFFFFFFFu, t0, from), a1 = __shfl_sync(0xFFFFFFFFu, t1, from);
    u64 pos = __shfl_sync(0xFFFFFFFFu, run, from), rk = __shfl_sync(0xFFFFFFFFu, tie, from);
    for (int i = a0; i < a1; i += 32) {
      const float x = i + lane < a1 ? at(i + lane) : -INFINITY;
      const uint32_t eq = __ballot_sync(0xFFFFFFFFu, x == cut && i + lane < a1);
      const u64 w = kept_weight(x, rk + __popc(eq & ((1u << lane) - 1u)));
      u64 inc = w;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const u64 o = __shfl_up_sync(0xFFFFFFFFu, inc, d);
        if (lane >= d) inc += o;
      }
      const u64 end = pos + inc;
      if (end - w <= target && target < end) finish(i0 + i + lane, x, total);
      pos = __shfl_sync(0xFFFFFFFFu, end, 31);
      rk += __popc(eq);
    }
  }
}

// A launch of B rows, C CTAs each.
struct Launch {
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = {};  // points at attr
  Launch(const Launch&) = delete;
  Launch(int64_t B, int C, int threads, size_t smem, cudaStream_t stream) {
    cfg.gridDim = dim3((unsigned)(B * C));
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = C;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
  }
};

template <int kThreads, bool kBf16, bool kResident>
cudaError_t allow_sample() {
  static std::atomic<uint64_t> allowed{0};
  return allow_smem(sample_kernel<kThreads, kBf16, kResident>, kSampleSmemMax, allowed, true);
}

template <int kThreads, bool kBf16, bool kResident>
cudaError_t launch_sample_t(const SampleParams& p, int64_t B, int C, size_t smem, cudaStream_t stream) {
  const cudaError_t e = allow_sample<kThreads, kBf16, kResident>();
  if (e != cudaSuccess) return e;
  const Launch l(B, C, kThreads, smem, stream);
  return cudaLaunchKernelEx(&l.cfg, sample_kernel<kThreads, kBf16, kResident>, p);
}

// How many clusters of C CTAs of this form device dev (the current one) runs at a time;
// 0 where it cannot say. Asked once per device, C, and CTAs that shared memory lets on
// an SM.
template <int kThreads, bool kBf16, bool kResident>
int clusters_at_once(int dev, int C, size_t smem) {
  static std::atomic<int> known[64][5][2];  // the answer + 1
  constexpr size_t kTwo = 228 * 1024 / 2 - 1024;  // shared memory of a CTA that leaves room for a second one
  const bool two = kThreads == 512 && smem <= kTwo;
  int size = 0;
  while ((1 << size) < C) ++size;
  std::atomic<int>& mine = known[dev & 63][size][two];
  int n = mine.load(std::memory_order_relaxed) - 1;
  if (n < 0) {
    n = 0;
    const Launch l(1, C, kThreads, two ? kTwo : kSampleSmemMax, nullptr);
    if (allow_sample<kThreads, kBf16, kResident>() != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, sample_kernel<kThreads, kBf16, kResident>, &l.cfg) != cudaSuccess) {
      cudaGetLastError();  // an answer, not an error of the call
      n = 0;
    }
    mine.store(n + 1, std::memory_order_relaxed);
  }
  return n;
}

// One of the six kernel forms: f(threads, bf16, resident) with each as a constant.
template <bool kBf16, typename F>
auto with_form(const SampleCut& c, F f) {
  using std::integral_constant;
  using Bf16 = integral_constant<bool, kBf16>;
  if (!c.resident) return f(integral_constant<int, 512>(), Bf16(), std::false_type());
  if (c.wide) return f(integral_constant<int, 1024>(), Bf16(), std::true_type());
  return f(integral_constant<int, 512>(), Bf16(), std::true_type());
}

template <bool kBf16>
cudaError_t launch_sample_x(const void* logits, int64_t B, int64_t V, int64_t ld, const SampleHow& how, const float* u,
                            int64_t* tokens, float* logprobs, cudaStream_t stream, int num_sms) {
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const SampleCut c = sample_cut(B, V, num_sms, sizeof(Smem), [&](const SampleCut& s) {
    return with_form<kBf16>(s, [&](auto threads, auto bf16, auto resident) {
      return clusters_at_once<decltype(threads)::value, decltype(bf16)::value, decltype(resident)::value>(
          dev, s.cluster, s.smem);
    });
  });
  SampleParams p;
  p.logits = logits;
  p.how = how;
  p.u = u;
  p.tokens = tokens;
  p.logprobs = logprobs;
  p.V = V;
  p.ld = ld;
  p.per = c.per;
  p.cluster = c.cluster;
  // A launch takes fewer than 2^31 CTAs: long batches go in parts.
  const int64_t rows = 0x7FFFFFFF / c.cluster;
  for (int64_t b = 0; b < B; b += rows) {
    SampleParams q = p;
    const int64_t part = B - b < rows ? B - b : rows;
    q.logits = static_cast<const char*>(logits) + b * ld * (kBf16 ? 2 : 4);
    if (how.temperature != nullptr) q.how.temperature += b;
    if (how.top_k != nullptr) q.how.top_k += b;
    if (how.top_p != nullptr) q.how.top_p += b;
    if (how.min_p != nullptr) q.how.min_p += b;
    q.u += b;
    q.tokens += b;
    if (logprobs != nullptr) q.logprobs += b;
    const cudaError_t e = with_form<kBf16>(c, [&](auto threads, auto bf16, auto resident) {
      return launch_sample_t<decltype(threads)::value, decltype(bf16)::value, decltype(resident)::value>(
          q, part, c.cluster, c.smem, stream);
    });
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_sample(const void* logits, bool bf16, int64_t B, int64_t V, int64_t ld, const SampleHow& how,
                          const float* u, int64_t* tokens, float* logprobs, cudaStream_t stream, int num_sms) {
  return bf16 ? launch_sample_x<true>(logits, B, V, ld, how, u, tokens, logprobs, stream, num_sms)
              : launch_sample_x<false>(logits, B, V, ld, how, u, tokens, logprobs, stream, num_sms);
}

}  // namespace bl
