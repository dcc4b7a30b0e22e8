// bl_sample.cu - one token per row of logits: temperature, top-k, top-p, min-p
// and a draw by a given uniform number.
//
// Weights w = exp((x - max) / T) are rounded to multiples of 2^-40 and added as
// 64-bit integers (V <= 2^22 keeps a row's sum below 2^62), so every sum is
// exact and no order of adding changes the token.
#include "bl_internal.h"

namespace bl {

namespace {

constexpr int kSampleThreads = 512;
constexpr double kWeightOne = 1099511627776.0;  // 2^40

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

struct RowHow {
  double c;       // -1 / T
  bool greedy;
  int k;          // 0: off
  double p;       // 1: off
  double m;       // min-p threshold in weight units, 0: off
};

__device__ __forceinline__ RowHow row_how(const SampleHow& h, int64_t b) {
  RowHow r;
  const float T = h.temperature != nullptr ? h.temperature[b] : h.temperature_value;
  const int k = h.top_k != nullptr ? h.top_k[b] : h.top_k_value;
  const float p = h.top_p != nullptr ? h.top_p[b] : h.top_p_value;
  const float m = h.min_p != nullptr ? h.min_p[b] : h.min_p_value;
  r.greedy = !(T > 0.0f);
  r.c = r.greedy ? 0.0 : -1.0 / (double)T;
  r.k = k > 0 ? k : 0;
  r.p = p < 1.0f ? (p > 0.0f ? (double)p : 0.0) : 1.0;
  r.m = m > 0.0f ? (m < 1.0f ? (double)m : 1.0) * kWeightOne : 0.0;
  return r;
}

// The weight of a key in units of 2^-40.
__device__ __forceinline__ unsigned long long key_weight(uint32_t key, uint32_t top, double max, double c) {
  if (key == top) return 1ull << 40;
  if (key == 0u || max == INFINITY) return 0ull;
  return (unsigned long long)__double2ll_rn(exp((max - (double)key_value(key)) * c) * kWeightOne);
}

template <typename T>
__device__ T block_sum(T v, T* sh) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
  __syncthreads();
  T t = 0;
  for (int i = 0; i < kSampleThreads / 32; ++i) t += sh[i];
  return t;
}

// One CTA per row. Thresholds by bisection over keys, a pass over the row each.
template <bool kBf16>
__global__ void __launch_bounds__(kSampleThreads)
    sample_kernel(const void* __restrict__ logits, int64_t V, int64_t ld, const SampleHow how,
                  const float* __restrict__ u, int64_t* __restrict__ tokens, float* __restrict__ logprobs) {
  __shared__ unsigned long long sh[kSampleThreads / 32];
  __shared__ uint32_t sh_key[kSampleThreads / 32];
  const int64_t b = blockIdx.x;
  const int tid = threadIdx.x;
  const RowHow h = row_how(how, b);
  const float* rowf = static_cast<const float*>(logits) + b * ld;
  const uint16_t* rowh = static_cast<const uint16_t*>(logits) + b * ld;
  const auto key_at = [&](int64_t i) {
    return sample_key(kBf16 ? bf16_bits_to_float(rowh[i]) : rowf[i]);
  };
  uint32_t top = 0u;
  for (int64_t i = tid; i < V; i += kSampleThreads) top = max(top, key_at(i));
  top = __reduce_max_sync(0xFFFFFFFFu, top);
  if ((tid & 31) == 0) sh_key[tid >> 5] = top;
  __syncthreads();
  for (int i = 0; i < kSampleThreads / 32; ++i) top = max(top, sh_key[i]);
  if (top == 0u) {
    if (tid == 0) {
      tokens[b] = -1;
      if (logprobs != nullptr) logprobs[b] = -INFINITY;
    }
    return;
  }
  const double mx = (double)key_value(top);
  // Kept: key > cut, and the first `ties` of those with key == cut.
  uint32_t cut = h.greedy ? top : 1u;
  int64_t ties = h.greedy ? 1 : V;
  const auto count_from = [&](uint32_t from) {
    unsigned long long n = 0;
    for (int64_t i = tid; i < V; i += kSampleThreads) n += key_at(i) >= from ? 1 : 0;
    return block_sum(n, sh);
  };
  if (!h.greedy && h.k > 0 && count_from(1u) > (unsigned long long)h.k) {
    uint32_t lo = 1u, hi = top;  // the largest key with at least k tokens from it on
    while (lo < hi) {
      const uint32_t mid = lo + (hi - lo + 1u) / 2u;
      if (count_from(mid) >= (unsigned long long)h.k) lo = mid;
      else hi = mid - 1u;
    }
    cut = lo;
    ties = (int64_t)h.k - (lo == 0xFFFFFFFFu ? 0 : (int64_t)count_from(lo + 1u));
  }
  // Sum of the weights of the kept keys >= from (from >= cut).
  const auto sum_from = [&](uint32_t from) {
    unsigned long long s = 0;
    for (int64_t i = tid; i < V; i += kSampleThreads) {
      const uint32_t key = key_at(i);
      if (key >= from && key > cut) s += key_weight(key, top, mx, h.c);
    }
    unsigned long long t = block_sum(s, sh);
    if (from <= cut) {
      unsigned long long n = 0;
      for (int64_t i = tid; i < V; i += kSampleThreads) n += key_at(i) == cut ? 1 : 0;
      n = block_sum(n, sh);
      n = n < (unsigned long long)ties ? n : (unsigned long long)ties;
      t += n * key_weight(cut, top, mx, h.c);
    }
    return t;
  };
  if (!h.greedy && h.p < 1.0) {
    const double need = h.p * (double)sum_from(cut);
    uint32_t lo = cut, hi = top;  // the largest key whose sum reaches `need`
    while (lo < hi) {
      const uint32_t mid = lo + (hi - lo + 1u) / 2u;
      if ((double)sum_from(mid) >= need) lo = mid;
      else hi = mid - 1u;
    }
    const unsigned long long above = lo == 0xFFFFFFFFu ? 0ull : sum_from(lo + 1u);
    const unsigned long long w = key_weight(lo, top, mx, h.c);
    // The shortest run of ties that reaches it: above + r * w >= need.
    int64_t r = w > 0ull ? (int64_t)ceil((need - (double)above) / (double)w) : V;
    if (r < 1) r = 1;
    if (lo > cut || r < ties) ties = r;
    cut = lo;
  }
  // Final pass: index order, thread t owns one stretch of the row.
  const int64_t per = (V + kSampleThreads - 1) / kSampleThreads;
  const int64_t i0 = per * tid, i1 = i0 + per < V ? i0 + per : V;
  __shared__ unsigned long long pre[kSampleThreads + 1];
  unsigned long long n = 0;
  for (int64_t i = i0; i < i1; ++i) n += key_at(i) == cut ? 1 : 0;
  __syncthreads();
  pre[tid + 1] = n;
  __syncthreads();
  if (tid == 0) {
    pre[0] = 0;
    for (int i = 0; i < kSampleThreads; ++i) pre[i + 1] += pre[i];
  }
  __syncthreads();
  const unsigned long long tie0 = pre[tid];
  __syncthreads();
  const auto kept_weight = [&](int64_t i, unsigned long long& tie) {
    const uint32_t key = key_at(i);
    if (key < cut || key == 0u) return 0ull;
    if (key == cut && tie++ >= (unsigned long long)ties) return 0ull;
    const unsigned long long w = key_weight(key, top, mx, h.c);
    return (double)w >= h.m ? w : 0ull;
  };
  unsigned long long s = 0, tie = tie0;
  for (int64_t i = i0; i < i1; ++i) s += kept_weight(i, tie);
  pre[tid + 1] = s;
  __syncthreads();
  if (tid == 0) {
    for (int i = 0; i < kSampleThreads; ++i) pre[i + 1] += pre[i];
  }
  __syncthreads();
  const unsigned long long total = pre[kSampleThreads];
  const float ub = u[b];
  unsigned long long target = ub > 0.0f ? (ub < 1.0f ? (unsigned long long)((double)ub * (double)total) : total - 1) : 0;
  if (target >= total) target = total - 1;
  unsigned long long run = pre[tid];
  if (run <= target && pre[tid + 1] > target) {
    tie = tie0;
    for (int64_t i = i0; i < i1; ++i) {
      run += kept_weight(i, tie);
      if (run > target) {
        tokens[b] = i;
        if (logprobs != nullptr) {
          const uint32_t key = key_at(i);
          const double d = key == top ? 0.0 : (mx - (double)key_value(key)) * h.c;
          logprobs[b] = h.greedy ? 0.0f : (float)(d - log((double)total / kWeightOne));
        }
        break;
      }
    }
  }
}

}  // namespace

cudaError_t launch_sample(const void* logits, bool bf16, int64_t B, int64_t V, int64_t ld, const SampleHow& how,
                          const float* u, int64_t* tokens, float* logprobs, cudaStream_t stream, int num_sms) {
  (void)num_sms;
  if (bf16)
    sample_kernel<true><<<(unsigned)B, kSampleThreads, 0, stream>>>(logits, V, ld, how, u, tokens, logprobs);
  else
    sample_kernel<false><<<(unsigned)B, kSampleThreads, 0, stream>>>(logits, V, ld, how, u, tokens, logprobs);
  return cudaGetLastError();
}

}  // namespace bl
