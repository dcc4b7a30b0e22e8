// bl_w4.cu - linear layers with 4-bit weights and group scales: packing, layout
// conversion and the product
//   y[m,n] = sum_G S[n,G] * (sum over k in G of c[n,k] * x[m,k]).
// bl_internal.h describes the packed layout.
#include "bl_internal.h"

namespace bl {

namespace {

__device__ __forceinline__ float w4_scale_load(const uint8_t* p, int i, int scale_bytes) {
  return scale_bytes == 4 ? reinterpret_cast<const float*>(p)[i]
                          : bf16_bits_to_float(reinterpret_cast<const uint16_t*>(p)[i]);
}

// bf16 nearest to a finite v (half to even), as bits.
__device__ __forceinline__ uint32_t bf16_rn_bits(float v) {
  const uint32_t b = __float_as_uint(v);
  return (b + 0x7FFFu + ((b >> 16) & 1u)) >> 16;
}

// Eight codes c + 8 (one to a byte of lo, hi; columns 0..3 and 4..7) to a packed word.
__device__ __forceinline__ uint32_t w4_word(const uint32_t (&c)[8]) {
  uint32_t w = 0u;
#pragma unroll
  for (int p = 0; p < 4; ++p) w |= (c[2 * p] << (4 * p)) | (c[2 * p + 1] << (4 * p + 16));
  return w;
}

__device__ __forceinline__ int64_t w4_block_off(const W4Shape& sh, int64_t tile, int64_t block) {
  return (tile * sh.blocks() + block) * sh.block_bytes();
}

// One warp per row of a block: lane l owns the block's columns 4l .. 4l+3, so
// 8, 16 or 32 neighbouring lanes hold a group. Bandwidth-bound (W is read once).
template <bool kBf16>
__global__ void __launch_bounds__(256) w4_pack_kernel(const void* __restrict__ W, const W4Shape sh,
                                                      uint8_t* __restrict__ packed, uint32_t* status) {
  const int lane = threadIdx.x & 31;
  const int64_t nwarps = (int64_t)gridDim.x * 8;
  const int64_t blocks = sh.blocks();
  const int64_t jobs = sh.tiles() * kW4Rows * blocks;
  const int glanes = sh.group / 4;
  for (int64_t job = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); job < jobs; job += nwarps) {
    const int64_t n = job / blocks, kb = job - n * blocks;
    const int64_t k = kb * kW4Cols + 4 * lane;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (n < sh.N && k < sh.K) v = load4<kBf16>(W, (n * sh.K + k) >> 2);  // K % 16 == 0: all four or none
    float a = fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w)));
    // fmaxf drops NaN: a non-finite weight is found on its own.
    bool bad = !(isfinite(v.x) && isfinite(v.y) && isfinite(v.z) && isfinite(v.w));
    for (int d = 1; d < glanes; d <<= 1) {
      a = fmaxf(a, __shfl_xor_sync(0xFFFFFFFFu, a, d));
      bad = __shfl_xor_sync(0xFFFFFFFFu, (int)bad, d) != 0 || bad;
    }
    float s = bad ? 0.0f : __fdiv_rn(a, 7.0f);
    if (sh.scale_bytes == 2) s = bf16_bits_to_float(bf16_rn_bits(s));
    if (bad && (lane % glanes) == 0) atomicOr(status, 1u);
    const float w4v[4] = {v.x, v.y, v.z, v.w};
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      int q = 0;
      if (s > 0.0f) {
        q = __float2int_rn(__fdiv_rn(w4v[i], s));
        q = q < -8 ? -8 : (q > 7 ? 7 : q);
      }
      c[i] = (uint32_t)(q + 8);
    }
    // Lanes 2i and 2i + 1 share a word (columns 8i .. 8i + 7).
    uint32_t half = c[0] | (c[1] << 16) | (c[2] << 4) | (c[3] << 20);
    half = (lane & 1) ? half << 8 : half;
    const uint32_t word = half | __shfl_xor_sync(0xFFFFFFFFu, half, 1);
    const int r = (int)(n % kW4Rows);
    uint8_t* blk = packed + w4_block_off(sh, n / kW4Rows, kb);
    const int wi = lane >> 1;  // word of columns 8*wi: j = wi / 4, t = wi % 4
    if ((lane & 1) == 0) reinterpret_cast<uint32_t*>(blk)[r * 16 + 4 * (wi & 3) + (wi >> 2)] = word;
    if ((lane % glanes) == 0) {
      uint8_t* sp = blk + kW4CodeBytes;
      const int si = (lane / glanes) * kW4Rows + r;
      if (sh.scale_bytes == 4)
        reinterpret_cast<float*>(sp)[si] = s;
      else
        reinterpret_cast<uint16_t*>(sp)[si] = (uint16_t)(__float_as_uint(s) >> 16);
    }
  }
}

// Natural nibbles [N, K/2] and scales [N, G] to the packed layout: one thread
// per word of eight columns; the first word of a group also moves its scale.
__global__ void __launch_bounds__(256) w4_import_kernel(const uint8_t* __restrict__ codes, const void* __restrict__ S,
                                                        const W4Shape sh, uint8_t* __restrict__ packed) {
  const int64_t words = sh.blocks() * 16;
  const int64_t jobs = sh.tiles() * kW4Rows * words;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < jobs; i += (int64_t)gridDim.x * 256) {
    const int64_t n = i / words, wi = i - n * words;
    const int64_t kb = wi >> 4;
    const int w = (int)(wi & 15);
    const int64_t k = wi * 8;
    uint32_t word = 0x88888888u;  // code 0
    const bool in = n < sh.N && k < sh.K;
    if (in) {
      const uint32_t nat = reinterpret_cast<const uint32_t*>(codes)[(n * sh.K + k) >> 3];
      uint32_t c[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) c[j] = (nat >> (4 * j)) & 15u;
      word = w4_word(c);
    }
    const int r = (int)(n % kW4Rows);
    uint8_t* blk = packed + w4_block_off(sh, n / kW4Rows, kb);
    reinterpret_cast<uint32_t*>(blk)[r * 16 + 4 * (w & 3) + (w >> 2)] = word;
    if ((8 * w) % sh.group == 0) {
      const int si = (8 * w / sh.group) * kW4Rows + r;
      const int64_t src = n * sh.groups() + k / sh.group;
      uint8_t* sp = blk + kW4CodeBytes;
      if (sh.scale_bytes == 4)
        reinterpret_cast<float*>(sp)[si] = in ? static_cast<const float*>(S)[src] : 0.0f;
      else
        reinterpret_cast<uint16_t*>(sp)[si] = in ? static_cast<const uint16_t*>(S)[src] : (uint16_t)0;
    }
  }
}

__global__ void __launch_bounds__(256) w4_export_kernel(const uint8_t* __restrict__ packed, const W4Shape sh,
                                                        int8_t* __restrict__ codes, void* __restrict__ S) {
  const int64_t words = sh.K / 8;
  const int64_t jobs = sh.N * words;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < jobs; i += (int64_t)gridDim.x * 256) {
    const int64_t n = i / words, wi = i - n * words;
    const int64_t kb = wi >> 4;
    const int w = (int)(wi & 15);
    const int r = (int)(n % kW4Rows);
    const uint8_t* blk = packed + w4_block_off(sh, n / kW4Rows, kb);
    const uint32_t word = reinterpret_cast<const uint32_t*>(blk)[r * 16 + 4 * (w & 3) + (w >> 2)];
    uint32_t out[2] = {0u, 0u};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = (int)((word >> (4 * (j >> 1) + 16 * (j & 1))) & 15u) - 8;
      out[j >> 2] |= ((uint32_t)c & 0xFFu) << (8 * (j & 3));
    }
    *reinterpret_cast<uint2*>(codes + n * sh.K + wi * 8) = make_uint2(out[0], out[1]);
    if ((8 * w) % sh.group == 0) {
      const int si = (8 * w / sh.group) * kW4Rows + r;
      const int64_t dst = n * sh.groups() + wi * 8 / sh.group;
      const uint8_t* sp = blk + kW4CodeBytes;
      if (sh.scale_bytes == 4)
        static_cast<float*>(S)[dst] = reinterpret_cast<const float*>(sp)[si];
      else
        static_cast<uint16_t*>(S)[dst] = reinterpret_cast<const uint16_t*>(sp)[si];
    }
  }
}

// One warp per output row and up to four tokens: lanes stride over the row's
// words; a lane's word lies in one group, whose scale multiplies the word's sum.
template <bool kBf16>
__global__ void __launch_bounds__(256) w4_plain_kernel(const void* __restrict__ x, int64_t M, const W4Shape sh,
                                                       const uint8_t* __restrict__ packed, float* __restrict__ y) {
  const int lane = threadIdx.x & 31;
  const int64_t words = sh.K / 8;
  const int64_t mtiles = (M + 3) / 4;
  const int64_t jobs = sh.N * mtiles;
  for (int64_t job = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); job < jobs; job += (int64_t)gridDim.x * 8) {
    const int64_t n = job / mtiles, m0 = (job - n * mtiles) * 4;
    const int r = (int)(n % kW4Rows);
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    for (int64_t wi = lane; wi < words; wi += 32) {
      const int w = (int)(wi & 15);
      const uint8_t* blk = packed + w4_block_off(sh, n / kW4Rows, wi >> 4);
      const uint32_t word = reinterpret_cast<const uint32_t*>(blk)[r * 16 + 4 * (w & 3) + (w >> 2)];
      const float s = w4_scale_load(blk + kW4CodeBytes, (8 * w / sh.group) * kW4Rows + r, sh.scale_bytes);
      float c[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) c[j] = (float)((int)((word >> (4 * (j >> 1) + 16 * (j & 1))) & 15u) - 8);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (m0 + i >= M) break;
        const float4 a = load4<kBf16>(x, ((m0 + i) * sh.K + wi * 8) >> 2);
        const float4 b = load4<kBf16>(x, (((m0 + i) * sh.K + wi * 8) >> 2) + 1);
        float t = c[0] * a.x;
        t = fmaf(c[1], a.y, t);
        t = fmaf(c[2], a.z, t);
        t = fmaf(c[3], a.w, t);
        t = fmaf(c[4], b.x, t);
        t = fmaf(c[5], b.y, t);
        t = fmaf(c[6], b.z, t);
        t = fmaf(c[7], b.w, t);
        acc[i] = fmaf(s, t, acc[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float v = acc[i];
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
      if (lane == 0 && m0 + i < M) y[(m0 + i) * sh.N + n] = v;
    }
  }
}

int64_t grid_for(int64_t jobs, int64_t per_cta, int num_sms) {
  const int64_t want = (jobs + per_cta - 1) / per_cta, most = (int64_t)num_sms * 16;
  return want < most ? want : most;
}

}  // namespace

cudaError_t launch_w4_pack(const void* W, bool bf16, const W4Shape& sh, void* packed, uint32_t* status,
                           cudaStream_t stream, int num_sms) {
  const int grid = (int)grid_for(sh.tiles() * kW4Rows * sh.blocks(), 8, num_sms);
  uint8_t* out = static_cast<uint8_t*>(packed);
  if (bf16)
    w4_pack_kernel<true><<<grid, 256, 0, stream>>>(W, sh, out, status);
  else
    w4_pack_kernel<false><<<grid, 256, 0, stream>>>(W, sh, out, status);
  return cudaGetLastError();
}

cudaError_t launch_w4_import(const uint8_t* codes, const void* S, const W4Shape& sh, void* packed,
                             cudaStream_t stream, int num_sms) {
  const int grid = (int)grid_for(sh.tiles() * kW4Rows * sh.blocks() * 16, 256, num_sms);
  w4_import_kernel<<<grid, 256, 0, stream>>>(codes, S, sh, static_cast<uint8_t*>(packed));
  return cudaGetLastError();
}

cudaError_t launch_w4_export(const void* packed, const W4Shape& sh, int8_t* codes, void* S, cudaStream_t stream,
                             int num_sms) {
  const int grid = (int)grid_for(sh.N * (sh.K / 8), 256, num_sms);
  w4_export_kernel<<<grid, 256, 0, stream>>>(static_cast<const uint8_t*>(packed), sh, codes, S);
  return cudaGetLastError();
}

cudaError_t launch_forward_w4(const void* x, bool bf16, int64_t M, const W4Shape& sh, const void* packed, float* y,
                              void* ws, cudaStream_t stream, int num_sms) {
  const cudaError_t e = cudaMemsetAsync(ws, 0, 4, stream);  // the error word
  if (e != cudaSuccess) return e;
  const int grid = (int)grid_for(sh.N * ((M + 3) / 4), 8, num_sms);
  const uint8_t* p = static_cast<const uint8_t*>(packed);
  if (bf16)
    w4_plain_kernel<true><<<grid, 256, 0, stream>>>(x, M, sh, p, y);
  else
    w4_plain_kernel<false><<<grid, 256, 0, stream>>>(x, M, sh, p, y);
  return cudaGetLastError();
}

}  // namespace bl
