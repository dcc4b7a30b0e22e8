// bl_sample.cu - one token per row of logits: temperature, top-k, top-p, min-p
// and a draw by a given uniform number.
//
// Weights w = exp((x - max) / T) are rounded to multiples of 2^-40 and added as
// 64-bit integers (V <= 2^22 keeps a row's sum below 2^62), so every sum is
// exact and no order of adding changes the token.
//
// A cluster of 1 to 8 CTAs owns a row: each CTA reads its stretch once into
// shared memory as ordered 32-bit keys, and every later pass runs there. The
// thresholds of top-k and top-p come from one histogram of 2048 bins, linear in
// x, of one 32-bit atomic per token: a count and the sum of the tokens' sixteenths
// of a bin. Counts place the k-th token in a bin exactly; the sixteenths bound
// every bin's weight to about 0.1%, which places the border of top-p within a
// bin or two without an exponential. The tokens of those bins (some hundreds)
// are sorted and settle the border exactly. Top-p then needs one exponential
// per token for the exact sum, a draw without filters likewise, top-k none
// beyond the kept tokens. What bounds it: the exponentials' 64-bit arithmetic
// (ten instructions a token) for large batches, the cluster barriers (five to
// seven of about a microsecond) for a single row.
#include "bl_internal.h"

#include <cstddef>

namespace bl {

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;          // the last one holds what lies past the range
constexpr int kListMax = 2048;       // tokens that a list of candidates holds
constexpr int kMaxCluster = 8;
constexpr int kPackMax = 16383;      // tokens per CTA whose count and sixteenths fit 14 + 18 bits
constexpr size_t kSampleSmemMax = 225 * 1024;
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

// Shared memory of a CTA; the keys follow it. Every member starts on a 16-byte
// boundary. Two regions serve twice: the
// leader's totals hold the candidates once a border's bins are known, its
// histogram their weights.
struct alignas(16) Smem {
  union {
    struct {
      uint32_t cnt[kBins];
      uint32_t off[kBins];
    } total;                 // leader: counts and sixteenths of the row
    u64 list[kListMax];      // leader: key << 32 | ~index
  };
  union {
    uint32_t hist[kBins];    // this CTA: count << 18 | sixteenths, or counts
    u64 wlist[kListMax];
  };
  alignas(16) double tab[256];           // 2^(40 + j / 256)
  alignas(16) u64 red[kWarps];
  alignas(16) double redd[2][kWarps];
  alignas(16) u64 xch[2][kMaxCluster][4];  // what the CTAs of the cluster tell one another
  alignas(16) int list_n;                // leader
  // Broadcast by the leader.
  int g_lo, g_hi;            // bins to collect
  uint32_t cut;              // kept: key > cut, and the first `ties` with key == cut
  u64 ties;
  int cut_partial;           // more tokens than `ties` have that key
};
static_assert(sizeof(Smem) % 16 == 0 && offsetof(Smem, xch) % 16 == 0, "alignment");

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
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// Every thread of the cluster; what was written before is seen after.
__device__ __forceinline__ void cluster_sync() {
  cluster_arrive();
  cluster_wait();
}
struct Sums {
  u64 a, b, c;
};

struct Row {
  double mx;      // largest logit
  double c;       // -256 log2(e) / T
  uint32_t top;   // its key
  float mxf, scale;  // bin position = (mxf - x) * scale
};

// exp((x - max) / T) in units of 2^-40, by a table of 2^(j/256) and a cubic
// (P. T. P. Tang, ACM TOMS 15(2), 1989): within 2^-42 relative before rounding.
__device__ __forceinline__ u64 key_weight(uint32_t key, const Row& r, const double* tab) {
  if (key == r.top) return 1ull << 40;
  if (key == 0u || r.mxf == INFINITY) return 0ull;
  double t = (r.mx - (double)key_value(key)) * r.c;
  t = fmax(t, -256.0 * 64.0);
  const double magic = 6755399441055744.0;  // 1.5 * 2^52: adding it rounds to an integer
  const double tm = t + magic;
  const int n = __double2loint(tm);
  const double rho = (t - (tm - magic)) * (0.693147180559945309417 / 256.0);
  const double q = rho * fma(rho, fma(rho, 1.0 / 6.0, 0.5), 1.0);
  double v = tab[n & 255];
  v = fma(v, q, v);
  v = __hiloint2double(__double2hiint(v) + (n >> 8) * (1 << 20), __double2loint(v));  // times 2^(n >> 8)
  const double vm = v + 4503599627370496.0;  // 2^52: the integer nearest to v in the low bits
  return ((u64)(uint32_t)(__double2hiint(vm) & 0x000FFFFF) << 32) | (uint32_t)__double2loint(vm);
}

// Sixteenths of a bin from the largest logit; monotone in x.
__device__ __forceinline__ uint32_t bin16(uint32_t key, const Row& r) {
  if (key == r.top) return 0u;
  const float pos = fminf((r.mxf - key_value(key)) * r.scale, (float)(kBins - 1));
  return (uint32_t)__float_as_int(fmaf(pos, 16.0f, 8388608.0f)) & 0x7FFFFFu;  // 2^23: rounds to an integer
}

template <typename T>
__device__ __forceinline__ T warp_sum(T v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
  return v;
}

// Exclusive prefix over the block; the block's sum in `all`.
__device__ __forceinline__ u64 block_scan(u64 v, Smem& s, u64& all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  u64 inc = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const u64 o = __shfl_up_sync(0xFFFFFFFFu, inc, d);
    if (lane >= d) inc += o;
  }
  __syncthreads();
  if (lane == 31) s.red[warp] = inc;
  __syncthreads();
  u64 before = 0, t = 0;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    const u64 x = s.red[i];
    if (i < warp) before += x;
    t += x;
  }
  all = t;
  return before + inc - v;
}

// Sorts the first 2^k >= n entries of `a` (zeros or ones past n, whichever
// belongs last), largest first or smallest first.
__device__ __forceinline__ void block_sort(u64* a, int n, bool descending) {
  int p = 2;
  while (p < n) p <<= 1;
  for (int i = n + threadIdx.x; i < p; i += kThreads) a[i] = descending ? 0ull : ~0ull;
  __syncthreads();
  for (int k = 2; k <= p; k <<= 1) {
    for (int j = k >> 1; j > 0; j >>= 1) {
      for (int i = threadIdx.x; i < (p >> 1); i += kThreads) {
        const int lo = 2 * i - (i & (j - 1)), hi = lo + j;
        const u64 x = a[lo], y = a[hi];
        const bool up = ((lo & k) == 0) != descending;
        if ((x > y) == up) {
          a[lo] = y;
          a[hi] = x;
        }
      }
      __syncthreads();
    }
  }
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

template <bool kBf16, bool kResident>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleParams p) {
  extern __shared__ __align__(128) uint8_t raw[];
  Smem& s = *reinterpret_cast<Smem*>(raw);
  uint32_t* skey = reinterpret_cast<uint32_t*>(raw + sizeof(Smem));
  const int C = p.cluster, rank = (int)(blockIdx.x % (unsigned)C);  // clusters are runs of C blocks
  const int tid = threadIdx.x, lane = tid & 31;
  const int64_t b = blockIdx.x / C;
  const int64_t i0 = (int64_t)rank * p.per;
  const int64_t rest = p.V - i0;
  const int n = rest <= 0 ? 0 : (rest < p.per ? (int)rest : p.per);
  const uint32_t lead_cnt = remote_addr(s.total.cnt, 0), lead_off = remote_addr(s.total.off, 0);
  const uint32_t lead_list = remote_addr(s.list, 0), lead_n = remote_addr(&s.list_n, 0);
  // Another CTA's shared memory may be touched once it has begun: waited for
  // below, before the first exchange.
  cluster_arrive();

  // ---- settings of the row
  const float T = p.how.temperature != nullptr ? p.how.temperature[b] : p.how.temperature_value;
  const int kset = p.how.top_k != nullptr ? p.how.top_k[b] : p.how.top_k_value;
  const float pset = p.how.top_p != nullptr ? p.how.top_p[b] : p.how.top_p_value;
  const float mset = p.how.min_p != nullptr ? p.how.min_p[b] : p.how.min_p_value;
  const bool greedy = !(T > 0.0f);
  const bool by_p = pset < 1.0f;  // false for NaN
  const double pp = pset > 0.0f ? (double)pset : 0.0;
  const u64 wmin = mset > 0.0f ? (u64)ceil((mset < 1.0f ? (double)mset : 1.0) * kWeightOne) : 0ull;

  // ---- the row, once: keys, their largest and smallest, how many are in
  const char* row = static_cast<const char*>(p.logits) + (b * p.ld + i0) * (kBf16 ? 2 : 4);
  const auto load = [&](int i) {
    return sample_key(kBf16 ? bf16_bits_to_float(reinterpret_cast<const uint16_t*>(row)[i])
                            : reinterpret_cast<const float*>(row)[i]);
  };
  const auto key_at = [&](int i) { return kResident ? skey[i] : load(i); };
  uint32_t kmax = 0u, kmin = 0xFFFFFFFFu, valid32 = 0u;
  constexpr int kLoads = 8;
  for (int base = tid; base < n; base += kThreads * kLoads) {
    uint32_t k8[kLoads];
#pragma unroll
    for (int j = 0; j < kLoads; ++j) k8[j] = base + j * kThreads < n ? load(base + j * kThreads) : 0u;
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      if (kResident && base + j * kThreads < n) skey[base + j * kThreads] = k8[j];
      kmax = max(kmax, k8[j]);
      if (k8[j] != 0u) {
        kmin = min(kmin, k8[j]);
        ++valid32;
      }
    }
  }
  for (int i = tid; i < kBins; i += kThreads) s.hist[i] = 0u;
  if (rank == 0) {
    for (int i = tid; i < kBins; i += kThreads) s.total.cnt[i] = s.total.off[i] = 0u;
    if (tid == 0) s.list_n = 0;
  }
  if (tid < 256) s.tab[tid] = exp2(40.0 + tid * (1.0 / 256.0));

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
  const auto block_total = [&](u64 v) {
    v = warp_sum(v);
    __syncthreads();
    if (lane == 0) s.red[tid >> 5] = v;
    __syncthreads();
    u64 t = 0;
    for (int i = 0; i < kWarps; ++i) t += s.red[i];
    return t;
  };
  // Sums over the cluster's threads, and of its first value over the CTAs before this one.
  u64 before_me = 0;
  const auto cluster_sum = [&](const Sums& v) {
    const u64 va = block_total(v.a), vb = block_total(v.b), vc = block_total(v.c);
    exchange(va, vb, vc);
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
  {
    kmax = __reduce_max_sync(0xFFFFFFFFu, kmax);
    kmin = __reduce_min_sync(0xFFFFFFFFu, kmin);
    valid32 = __reduce_add_sync(0xFFFFFFFFu, valid32);
    if (lane == 0) {
      s.red[tid >> 5] = ((u64)kmax << 32) | kmin;
      s.redd[0][tid >> 5] = (double)valid32;
    }
    __syncthreads();
    cluster_wait();
    u64 vmax = 0, vmin = 0xFFFFFFFFull, vn = 0;
    for (int i = 0; i < kWarps; ++i) {
      vmax = max(vmax, s.red[i] >> 32);
      vmin = min(vmin, s.red[i] & 0xFFFFFFFFull);
      vn += (u64)s.redd[0][i];
    }
    exchange(vmax, vmin, vn);
    kmax = 0u;
    kmin = 0xFFFFFFFFu;
    valid32 = 0u;
    for (int r = 0; r < C; ++r) {
      kmax = max(kmax, (uint32_t)s.xch[par][r][0]);
      kmin = min(kmin, (uint32_t)s.xch[par][r][1]);
      valid32 += (uint32_t)s.xch[par][r][2];
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
  r.c = greedy ? 0.0 : -369.329930467574631 / (double)T;  // 256 log2(e)

  const auto finish = [&](int64_t token, uint32_t key, u64 total) {
    p.tokens[b] = token;
    if (p.logprobs != nullptr) {
      const double d = key == r.top ? 0.0 : ((double)key_value(key) - r.mx) / (double)T;
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
      if (key_at(i) == r.top) first = min(first, (uint32_t)(i0 + i));
    first = __reduce_min_sync(0xFFFFFFFFu, first);
    __syncthreads();
    if (lane == 0) s.red[tid >> 5] = first;
    __syncthreads();
    u64 mine = 0xFFFFFFFFull;
    for (int i = 0; i < kWarps; ++i) mine = min(mine, s.red[i]);
    exchange(mine, 0, 0);
    if (rank == 0 && tid == 0) {
      u64 f = 0xFFFFFFFFull;
      for (int c = 0; c < C; ++c) f = min(f, s.xch[par][c][0]);
      finish((int64_t)f, r.top, 1ull << 40);
    }
    return;
  }

  const double span = key_value(kmax) == INFINITY ? 0.0 : r.mx - (double)key_value(kmin);
  const double reach = fmin(kTail * (double)T, span);  // the bins' range, in x
  const bool tail_out = reach < span;                  // the last bin's weights are all zero
  r.scale = span > 0.0 ? (float)((kBins - 1) / reach) : 1.0f;
  const double delta = span > 0.0 ? reach / (double)T / (kBins - 1) : 0.0;  // exponent per bin
  const int packed = p.per <= kPackMax ? 18 : 0;

  // The kept tokens so far: key > cut and the first `ties` with key == cut.
  uint32_t cut = 1u;
  u64 ties = ~0ull;
  bool cut_partial = false;
  bool by_k = kset > 0 && (uint32_t)kset < valid32;

  // Histogram of the tokens with key >= cut into the leader's totals.
  const auto histogram = [&]() {
    for (int i = tid; i < n; i += kThreads) {
      const uint32_t key = key_at(i);
      if (key >= cut && key != 0u) {
        const uint32_t v = bin16(key, r);
        atomicAdd(&s.hist[v >> 4], packed != 0 ? (1u << 18) + (v & 15u) : 1u);
      }
    }
    __syncthreads();
    for (int i = tid; i < kBins; i += kThreads) {
      const uint32_t h = s.hist[i];
      if (h != 0u) {
        const uint32_t c = packed != 0 ? h >> 18 : h, o = packed != 0 ? h & 0x3FFFFu : 8u * h;
        remote_add(lead_cnt + 4 * i, c);
        if (o != 0u) remote_add(lead_off + 4 * i, o);
      }
    }
    cluster_sync();
  };
  // The leader's verdict to every CTA.
  const auto broadcast = [&]() {
    __syncthreads();
    if (rank == 0 && tid > 0 && tid < C) {
      remote_store(remote_addr(&s.g_lo, tid), (uint32_t)s.g_lo);
      remote_store(remote_addr(&s.g_hi, tid), (uint32_t)s.g_hi);
      remote_store(remote_addr(&s.cut, tid), s.cut);
      remote_store(remote_addr(&s.ties, tid), s.ties);
      remote_store(remote_addr(&s.cut_partial, tid), (uint32_t)s.cut_partial);
    }
    cluster_sync();
  };
  // Tokens of a CTA counted from the leader's bins: 4 per thread, in order.
  constexpr int kPerThread = kBins / kThreads;
  const auto collect = [&](int i, uint32_t key) {
    const uint32_t at = remote_add(lead_n, 1u);
    if (at < (uint32_t)kListMax) remote_store(lead_list + 8 * at, ((u64)key << 32) | (0xFFFFFFFFu - (uint32_t)(i0 + i)));
  };

  // From the leader's sorted list of `m` candidates that holds every kept token:
  // apply top-k (keep), top-p (need: the sum to reach, 0: off) and min-p, and draw.
  const auto draw_from_list = [&](int m, int keep, bool use_p, bool own_total, u64 row_total) {
    block_sort(s.list, m, true);
    keep = keep < m ? keep : m;
    for (int i = tid; i < kListMax; i += kThreads)
      s.wlist[i] = i < keep ? key_weight((uint32_t)(s.list[i] >> 32), r, s.tab) : 0ull;
    __syncthreads();
    constexpr int kE = kListMax / kThreads;
    if (use_p) {
      u64 w[kE], sum = 0, all;
#pragma unroll
      for (int j = 0; j < kE; ++j) sum += w[j] = s.wlist[tid * kE + j];
      u64 run = block_scan(sum, s, all);
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
      u64 w = s.wlist[i];
      const uint32_t idx = 0xFFFFFFFFu - (uint32_t)s.list[i];
      if (w < wmin) w = s.wlist[i] = 0ull;
      s.list[i] = w == 0ull ? ~0ull : ((u64)idx << 32) | (uint32_t)i;
    }
    __syncthreads();
    // Keys of the drawn token come back from its index.
    block_sort(s.list, m, false);
    u64 w[kE], sum = 0, total;
#pragma unroll
    for (int j = 0; j < kE; ++j) {
      const int i = tid * kE + j;
      const u64 e = i < m ? s.list[i] : ~0ull;
      w[j] = e == ~0ull ? 0ull : s.wlist[(uint32_t)e];
      sum += w[j];
    }
    u64 run = block_scan(sum, s, total);
    const u64 target = target_of(total);
#pragma unroll
    for (int j = 0; j < kE; ++j) {
      if (run <= target && target < run + w[j]) {
        const int64_t idx = (int64_t)(s.list[tid * kE + j] >> 32);
        const char* at = static_cast<const char*>(p.logits) + (b * p.ld + idx) * (kBf16 ? 2 : 4);
        finish(idx,
               sample_key(kBf16 ? bf16_bits_to_float(*reinterpret_cast<const uint16_t*>(at))
                                : *reinterpret_cast<const float*>(at)),
               total);
      }
      run += w[j];
    }
  };
  // From the leader's list of `m` tokens of consecutive bins: the border after
  // the shortest run, largest first, of `need` tokens, or of weight `need`.
  const auto settle = [&](int m, u64 need, bool by_weight) {
    block_sort(s.list, m, true);
    constexpr int kE = kListMax / kThreads;
    u64 w[kE], sum = 0, all;
#pragma unroll
    for (int j = 0; j < kE; ++j) {
      const int i = tid * kE + j;
      w[j] = i < m ? (by_weight ? key_weight((uint32_t)(s.list[i] >> 32), r, s.tab) : 1ull) : 0ull;
      sum += w[j];
    }
    u64 run = block_scan(sum, s, all);
#pragma unroll
    for (int j = 0; j < kE; ++j) {
      const int i = tid * kE + j;
      if (i < m && run < need && run + w[j] >= need) {
        const uint32_t key = (uint32_t)(s.list[i] >> 32);
        int lo = 0, hi = i;  // the first token of this key
        while (lo < hi) {
          const int mid = (lo + hi) / 2;
          if ((uint32_t)(s.list[mid] >> 32) > key) lo = mid + 1;
          else hi = mid;
        }
        s.cut = key;
        s.ties = (u64)(i - lo + 1);
        s.cut_partial = i + 1 < m && (uint32_t)(s.list[i + 1] >> 32) == key;
      }
      run += w[j];
    }
    __syncthreads();
  };
  // The border without a list (more equal or near tokens than one holds):
  // bisection over the keys, a pass each. All CTAs take part and agree.
  const auto bisect = [&](u64 need, bool by_weight) {
    const uint32_t cut0 = cut;
    const u64 ties0 = ties;
    const bool partial0 = cut_partial;
    const auto sums = [&](uint32_t from, u64& reached, u64& equal) {  // kept tokens >= from; those == from
      Sums v = {0, 0, 0};
      for (int i = tid; i < n; i += kThreads) {
        const uint32_t key = key_at(i);
        if (key < from || key == 0u || (partial0 && key == cut0)) continue;
        v.a += by_weight ? key_weight(key, r, s.tab) : 1ull;
        if (key == from) ++v.b;
      }
      v = cluster_sum(v);
      if (partial0 && from <= cut0) {
        v.a += ties0 * (by_weight ? key_weight(cut0, r, s.tab) : 1ull);
        if (from == cut0) v.b += ties0;
      }
      reached = v.a;
      equal = v.b;
    };
    uint32_t lo = cut0, hi = r.top;  // the largest key from which on the need is reached
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
    cut = lo;
    ties = want;
    cut_partial = want < eq || (partial0 && lo == cut0);
  };

  // ---- top-k
  if (by_k) {
    histogram();
    if (rank == 0) {
      u64 mine[kPerThread], sum = 0, all;
#pragma unroll
      for (int j = 0; j < kPerThread; ++j) sum += mine[j] = s.total.cnt[tid * kPerThread + j];
      u64 run = block_scan(sum, s, all);
#pragma unroll
      for (int j = 0; j < kPerThread; ++j) {
        if (run < (u64)kset && run + mine[j] >= (u64)kset) {
          const int bin = tid * kPerThread + j;
          // Everything down to this bin, or the bin alone, or (-1) neither fits a list.
          s.g_hi = bin;
          s.g_lo = run + mine[j] <= kListMax ? 0 : (mine[j] <= kListMax ? bin : -1);
          if (s.g_lo < 0 && bin == kBins - 1 && tail_out) s.g_lo = -2;  // only zero weights are in question
          s.ties = (u64)kset - run;  // how many of the bin's tokens stay
        }
        run += mine[j];
      }
    }
    broadcast();
    const int g_lo = s.g_lo, g_hi = s.g_hi;
    const u64 in_bin = s.ties;
    if (g_lo >= 0) {
      for (int i = tid; i < n; i += kThreads) {
        const uint32_t key = key_at(i);
        if (key == 0u) continue;
        const int bin = (int)(bin16(key, r) >> 4);
        if (bin >= g_lo && bin <= g_hi) collect(i, key);
      }
      cluster_sync();
      // A list of one bin only settles top-k unless that bin is the first.
      if (g_lo == 0) {
        if (rank == 0) draw_from_list(s.list_n, kset, by_p, true, 0ull);
        return;
      }
      if (rank == 0) {
        settle(s.list_n, in_bin, false);
        if (tid == 0) s.list_n = 0;
      }
      broadcast();
      cut = s.cut;
      ties = s.ties;
      cut_partial = s.cut_partial != 0;
    } else if (g_lo == -1) {
      bisect((u64)kset, false);
    }
    if (by_p) {  // the histogram again, of what is left
      __syncthreads();
      for (int i = tid; i < kBins; i += kThreads) s.hist[i] = 0u;
      if (rank == 0)
        for (int i = tid; i < kBins; i += kThreads) s.total.cnt[i] = s.total.off[i] = 0u;
      cluster_sync();
    }
  }

  // Thread t owns tokens [t * own, (t + 1) * own) of the CTA's stretch from here
  // on: an odd number of shared-memory words, so that a warp's reads meet no
  // bank twice.
  const int own = ((n + kThreads - 1) / kThreads) | 1;
  const int t0 = own * tid < n ? own * tid : n, t1 = t0 + own < n ? t0 + own : n;
  u64 sure = 0;    // weight of the thread's tokens that are kept whatever the border
  int g_lo = 0;    // first bin that `sure` does not cover

  // ---- top-p
  if (by_p) {
    histogram();
    if (rank == 0) {
      // Bounds of every bin's weight: a token f bins past the bin's start
      // weighs e^(-delta f), between 1 - delta f and the chord; f is known to half
      // a sixteenth (and the rounding of the bin position, below 0.01 bins), or
      // not at all without the sixteenths.
      double lo[kPerThread], hi[kPerThread], slo = 0.0, shi = 0.0;
      const double fe = packed != 0 ? 1.0 / 32.0 + 0.01 : 0.51;
      const double shrink = 1.0 - exp(-delta);
#pragma unroll
      for (int j = 0; j < kPerThread; ++j) {
        const int bin = tid * kPerThread + j;
        const double c = s.total.cnt[bin], f = s.total.off[bin] * (1.0 / 16.0);
        const double e = exp(-delta * bin);
        lo[j] = c > 0.0 ? fmax(e * (c - delta * (f + c * fe)) - c / kWeightOne, 0.0) : 0.0;
        hi[j] = c > 0.0 ? e * (c - shrink * (f - c * fe)) * (1.0 + delta * delta) + c / kWeightOne : 0.0;
        if (bin == kBins - 1 || (cut_partial && bin == (int)(bin16(cut, r) >> 4))) lo[j] = 0.0;
        if (bin == kBins - 1) hi[j] = c * e * (1.0 + delta) + c / kWeightOne;
        slo += lo[j];
        shi += hi[j];
      }
      // Prefixes of both.
      const int warp = tid >> 5;
      double plo = slo, phi = shi;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const double a = __shfl_up_sync(0xFFFFFFFFu, plo, d), c = __shfl_up_sync(0xFFFFFFFFu, phi, d);
        if (lane >= d) {
          plo += a;
          phi += c;
        }
      }
      if (lane == 31) {
        s.redd[0][warp] = plo;
        s.redd[1][warp] = phi;
      }
      if (tid == 0) {
        s.g_lo = kBins - 1;
        s.g_hi = kBins - 1;
      }
      __syncthreads();
      double tlo = 0.0, thi = 0.0;
      plo -= slo;
      phi -= shi;
      for (int i = 0; i < kWarps; ++i) {
        if (i < warp) {
          plo += s.redd[0][i];
          phi += s.redd[1][i];
        }
        tlo += s.redd[0][i];
        thi += s.redd[1][i];
      }
      const double want_lo = pp * tlo * (1.0 - 1e-9), want_hi = pp * thi * (1.0 + 1e-9);
#pragma unroll
      for (int j = 0; j < kPerThread; ++j) {
        const int bin = tid * kPerThread + j;
        if (phi + hi[j] >= want_lo) atomicMin(&s.g_lo, bin);
        if (plo + lo[j] >= want_hi) atomicMin(&s.g_hi, bin);
        plo += lo[j];
        phi += hi[j];
      }
      __syncthreads();
      u64 mine[kPerThread], sum = 0, all;
#pragma unroll
      for (int j = 0; j < kPerThread; ++j) sum += mine[j] = s.total.cnt[tid * kPerThread + j];
      u64 run = block_scan(sum, s, all);
      const int blo = s.g_lo, bhi = s.g_hi;
      u64 upto = 0, inside = 0;  // tokens in bins 0..bhi and blo..bhi
#pragma unroll
      for (int j = 0; j < kPerThread; ++j) {
        const int bin = tid * kPerThread + j;
        if (bin <= bhi) upto += mine[j];
        if (bin >= blo && bin <= bhi) inside += mine[j];
      }
      (void)run;
      u64 dummy;
      block_scan(upto, s, dummy);
      upto = dummy;
      block_scan(inside, s, dummy);
      inside = dummy;
      __syncthreads();
      if (tid == 0) {
        if (upto <= kListMax) s.g_lo = 0;
        else if (inside > kListMax) s.g_lo = -1;
        s.cut = cut;
        s.ties = ties;
        s.cut_partial = cut_partial ? 1 : 0;
      }
    }
    broadcast();
    g_lo = s.g_lo;
    const int g_hi = s.g_hi;
    // One pass with an exponential per token: the sum of all kept tokens, of
    // those before bin g_lo, and the candidates between.
    Sums v = {0, 0, 0};
    for (int i = t0; i < t1; ++i) {
      const uint32_t key = key_at(i);
      if (key < cut || key == 0u || (cut_partial && key == cut)) {
        if (key == cut && key != 0u && g_lo >= 0) {  // a tie of top-k's border: counted by its rank, below
          const int bin = (int)(bin16(key, r) >> 4);
          if (bin >= g_lo && bin <= g_hi) collect(i, key);
        }
        continue;
      }
      const u64 w = key_weight(key, r, s.tab);
      v.a += w;
      if (g_lo < 0) continue;
      const int bin = (int)(bin16(key, r) >> 4);
      if (bin < g_lo) {
        v.b += w;
        if (w >= wmin) sure += w;
      } else if (bin <= g_hi) {
        collect(i, key);
      }
    }
    v = cluster_sum(v);  // its barrier also completes the list
    const u64 total = v.a + (cut_partial ? ties * key_weight(cut, r, s.tab) : 0ull);
    const double want = ceil(pp * (double)total);
    const u64 need = want > 1.0 ? (u64)want : 1ull;
    if (g_lo == 0) {
      // All that can stay is in the list; top-k's border cuts it at kset tokens.
      if (rank == 0) draw_from_list(s.list_n, by_k ? kset : kListMax, true, false, total);
      return;
    }
    if (g_lo > 0) {
      if (rank == 0) settle(s.list_n, need - v.b, true);
      broadcast();
      cut = s.cut;
      ties = s.ties;
      cut_partial = s.cut_partial != 0;
    } else {
      bisect(need, true);
      sure = 0;
      g_lo = 0;
    }
  }

  // ---- the draw, in index order
  u64 tie = 0;  // rank of the thread's first token with key == cut
  if (cut_partial) {
    u64 mine = 0, all;
    for (int i = t0; i < t1; ++i) mine += key_at(i) == cut ? 1 : 0;
    tie = block_scan(mine, s, all);
    cluster_sum(Sums{mine, 0, 0});
    tie += before_me;
  }
  const auto kept_weight = [&](uint32_t key, u64 rank_of_tie) {
    if (key < cut || key == 0u || (cut_partial && key == cut && rank_of_tie >= ties)) return 0ull;
    const u64 w = key_weight(key, r, s.tab);
    return w >= wmin ? w : 0ull;
  };
  u64 sum = sure, tr = tie;
  for (int i = t0; i < t1; ++i) {
    const uint32_t key = key_at(i);
    if (key < cut) continue;
    if (g_lo > 0 && (int)(bin16(key, r) >> 4) < g_lo) continue;  // in `sure`
    sum += kept_weight(key, tr);
    if (key == cut) ++tr;
  }
  u64 mine_all;
  u64 run = block_scan(sum, s, mine_all);
  const u64 total = cluster_sum(Sums{sum, 0, 0}).a, target = target_of(total);
  run += before_me;
  // The warp whose lane's stretch holds the target walks that stretch together.
  const uint32_t hit = __ballot_sync(0xFFFFFFFFu, run <= target && target < run + sum);
  if (hit != 0u) {
    const int from = __ffs(hit) - 1;
    const int a0 = __shfl_sync(0xFFFFFFFFu, t0, from), a1 = __shfl_sync(0xFFFFFFFFu, t1, from);
    u64 at = __shfl_sync(0xFFFFFFFFu, run, from), rk = __shfl_sync(0xFFFFFFFFu, tie, from);
    for (int i = a0; i < a1; i += 32) {
      const uint32_t key = i + lane < a1 ? key_at(i + lane) : 0u;
      const uint32_t eq = __ballot_sync(0xFFFFFFFFu, key == cut && key != 0u);
      const u64 w = kept_weight(key, rk + __popc(eq & ((1u << lane) - 1u)));
      u64 inc = w;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const u64 o = __shfl_up_sync(0xFFFFFFFFu, inc, d);
        if (lane >= d) inc += o;
      }
      const u64 end = at + inc;
      if (end - w <= target && target < end) finish(i0 + i + lane, key, total);
      at = __shfl_sync(0xFFFFFFFFu, end, 31);
      rk += __popc(eq);
    }
  }
}

template <bool kBf16, bool kResident>
cudaError_t launch_sample_t(const SampleParams& p, int64_t B, int C, size_t smem, cudaStream_t stream) {
  static std::atomic<uint64_t> allowed{0};
  auto kern = sample_kernel<kBf16, kResident>;
  const cudaError_t e = allow_smem(kern, kSampleSmemMax, allowed);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(B * C));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace

cudaError_t launch_sample(const void* logits, bool bf16, int64_t B, int64_t V, int64_t ld, const SampleHow& how,
                          const float* u, int64_t* tokens, float* logprobs, cudaStream_t stream, int num_sms) {
  // CTAs per row: so many that a stretch packs its histogram and two CTAs fit
  // an SM, then more while rows alone leave SMs idle and stretches stay long.
  int C = 1;
  while (C < kMaxCluster && ((V + C - 1) / C > kPackMax || (B * C * 2 <= 2 * num_sms && V / (2 * C) >= 2048))) C *= 2;
  SampleParams p;
  p.logits = logits;
  p.how = how;
  p.u = u;
  p.tokens = tokens;
  p.logprobs = logprobs;
  p.V = V;
  p.ld = ld;
  p.per = (int)((V + C - 1) / C);
  p.cluster = C;
  const size_t need = sizeof(Smem) + 4 * (size_t)p.per;
  const bool resident = need <= kSampleSmemMax;
  const size_t smem = resident ? need : sizeof(Smem);
  // A launch takes fewer than 2^31 CTAs: long batches go in parts.
  const int64_t rows = 0x7FFFFFFF / C;
  for (int64_t b = 0; b < B; b += rows) {
    SampleParams q = p;
    const int64_t part = B - b < rows ? B - b : rows;
    q.logits = static_cast<const char*>(logits) + b * ld * (bf16 ? 2 : 4);
    if (how.temperature != nullptr) q.how.temperature += b;
    if (how.top_k != nullptr) q.how.top_k += b;
    if (how.top_p != nullptr) q.how.top_p += b;
    if (how.min_p != nullptr) q.how.min_p += b;
    q.u += b;
    q.tokens += b;
    if (logprobs != nullptr) q.logprobs += b;
    const cudaError_t e = bf16 ? (resident ? launch_sample_t<true, true>(q, part, C, smem, stream)
                                           : launch_sample_t<true, false>(q, part, C, smem, stream))
                               : (resident ? launch_sample_t<false, true>(q, part, C, smem, stream)
                                           : launch_sample_t<false, false>(q, part, C, smem, stream));
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace bl
