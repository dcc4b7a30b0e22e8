// bl_w4.cu - linear layers with 4-bit weights and group scales: packing, layout
// conversion and the product
//   y[m,n] = sum_G S[n,G] * (sum over k in G of c[n,k] * x[m,k]).
// bl_internal.h describes the packed layout.
#include "bl_internal.h"

namespace bl {

namespace {

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
// 8, 16 or 32 neighbouring lanes hold a group. W is read once, but a warp has one
// load of 512 bytes in flight and divides 64-bit indexes for each: 128000 x 2560
// fp32 929 us with the read of the status word, where its bytes take 229.
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
      const int si = sh.scale_index(r, lane / glanes);
      if (sh.scale_bytes == 4)
        reinterpret_cast<float*>(sp)[si] = s;
      else
        reinterpret_cast<uint16_t*>(sp)[si] = (uint16_t)(__float_as_uint(s) >> 16);
    }
  }
}

// Natural nibbles [N, K/2] and scales [N, G] to the packed layout: one thread
// per word of eight columns; the first word of a group also moves its scale.
// Offline: 128000 x 2560 354 us (its bytes take 52), the export 342 (78); a 64-bit
// division and four scattered bytes per thread.
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
      const int si = sh.scale_index(r, 8 * w / sh.group);
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
      const int si = sh.scale_index(r, 8 * w / sh.group);
      const int64_t dst = n * sh.groups() + wi * 8 / sh.group;
      const uint8_t* sp = blk + kW4CodeBytes;
      if (sh.scale_bytes == 4)
        static_cast<float*>(S)[dst] = reinterpret_cast<const float*>(sp)[si];
      else
        static_cast<uint16_t*>(S)[dst] = reinterpret_cast<const uint16_t*>(sp)[si];
    }
  }
}

// ------------------------------------------------- few tokens: one stream --
// The weights are the traffic: 1 KiB of codes and 32..256 bytes of scales per
// block of 16 rows x 128 columns, read once. A CTA owns a run of whole row
// tiles, and its warps equal runs of that run's blocks, wherever tiles begin or
// end in it (an even split of whole tiles left a fifth of the machine idle). A
// warp keeps kDepth blocks in registers, loaded 512 consecutive bytes at a
// time and refilled as soon as they have been used. Codes become bf16
// pairs (w4_unpack) and are multiplied with mma.sync m16n8k16: the weights are
// the 16-row operand, up to 8 columns of x the other. bf16 codes and their
// products are exact; a group's sum stays in fp32 and is multiplied by its
// scale once. A tile that several warps share is added up through shared
// memory in warp order after one barrier at the end. At full stream rate an SM has
// 47 cycles a block, and its integer pipe takes 2 cycles per warp instruction:
// what is not unpacking is kept off it (columns past the last token read a row
// of zeros instead of being masked, products start from a zero register).
// The ring takes all 80 registers of three CTAs an SM, and most forms with fp32 x or
// fp32 scales pass them: 4 to 36 bytes a thread are spilled (groups of 32, fp32 scales).
// Measured in a graph, weights taken in turn from more than L2 holds: one bf16 token,
// 128000 x 2560 33.2 us (169 MB, 5.1 TB/s, 79% of a copy's rate), 13824 x 2560 6.8 us,
// groups of 32 7.0 us (20 MB); 16 bf16 tokens, 2560 x 2560 5.9, 13824 x 2560 9.8,
// 128000 x 2560 48.1 us.
constexpr int kStreamWarps = 8;
constexpr int kStreamPadBytes = 64;  // column stride = 64 mod 128: no bank conflicts between columns
constexpr size_t kStreamSmemMax = 225 * 1024;

struct StreamParams {
  const void* x;
  const uint8_t* packed;
  float* y;
  uint32_t* err;
  int M, K;
  int64_t N;
  int cols;     // columns of x: M, or 3 M for fp32
  int blocks;   // 128-column blocks per row
  int64_t tiles;
};

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint4 ldg_stream128(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
// 16 bytes to shared memory, or zeros (then src is not read).
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ uint2 ldg_stream64(const void* p) {
  uint2 v;
  asm volatile("ld.global.nc.L1::no_allocate.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}
__device__ __forceinline__ uint32_t ldg_stream32(const void* p) {
  uint32_t v;
  asm volatile("ld.global.nc.L1::no_allocate.b32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}
// d = a * b (+ d)
__device__ __forceinline__ void mma_bf16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// One block of a lane: its 16 code bytes of rows g and g + 8, and the scales of
// both rows for the block's groups.
template <int GPB, bool kBf16S>
struct LaneBlock {
  static constexpr int kScaleWords = kBf16S ? GPB : 2 * GPB;
  uint4 w0, w1;
  uint32_t s[kScaleWords];
  // src: the block's first byte plus 16 * lane; scales: the lane's scales.
  __device__ __forceinline__ void load(const uint8_t* src, const uint8_t* scales) {
    w0 = ldg_stream128(src);
    w1 = ldg_stream128(src + 512);
    if (kScaleWords == 1) {
      s[0] = ldg_stream32(scales);
    } else if (kScaleWords == 2) {
      const uint2 v = ldg_stream64(scales);
      s[0] = v.x;
      s[1] = v.y;
    } else {
#pragma unroll
      for (int i = 0; i < kScaleWords; i += 4) {
        const uint4 v = ldg_stream128(scales + 4 * i);
        s[i] = v.x;
        s[i + 1] = v.y;
        s[i + 2] = v.z;
        s[i + 3] = v.w;
      }
    }
  }
  __device__ __forceinline__ float scale(int gi, int half) const {
    if (kBf16S) return __uint_as_float(half == 0 ? s[gi] << 16 : s[gi] & 0xFFFF0000u);
    return __uint_as_float(s[2 * gi + half]);
  }
};

// tot += scales * (codes * x) over one block; xb[nt] + xk: the lane's x.
template <int NT, int GPB, bool kBf16S>
__device__ __forceinline__ void stream_block(const LaneBlock<GPB, kBf16S>& blk, const uint32_t (&xb)[NT], uint32_t xk,
                                             float (&tot)[NT][4]) {
  const uint32_t w0[4] = {blk.w0.x, blk.w0.y, blk.w0.z, blk.w0.w};
  const uint32_t w1[4] = {blk.w1.x, blk.w1.y, blk.w1.z, blk.w1.w};
#pragma unroll
  for (int gi = 0; gi < GPB; ++gi) {
    float acc[NT][4];
#pragma unroll
    for (int jj = 0; jj < 4 / GPB; ++jj) {
      const int j = gi * (4 / GPB) + jj;
      uint32_t a[4], b[4];
      w4_unpack(w0[j], a);
      w4_unpack(w1[j], b);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const uint4 xv = lds128(xb[nt] + xk + 64 * j);
        if (jj == 0)
          mma_bf16_first(acc[nt], a[0], b[0], a[1], b[1], xv.x, xv.y);
        else
          mma_bf16(acc[nt], a[0], b[0], a[1], b[1], xv.x, xv.y);
        mma_bf16(acc[nt], a[2], b[2], a[3], b[3], xv.z, xv.w);
      }
    }
    const float s0 = blk.scale(gi, 0), s1 = blk.scale(gi, 1);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      tot[nt][0] = fmaf(s0, acc[nt][0], tot[nt][0]);
      tot[nt][1] = fmaf(s0, acc[nt][1], tot[nt][1]);
      tot[nt][2] = fmaf(s1, acc[nt][2], tot[nt][2]);
      tot[nt][3] = fmaf(s1, acc[nt][3], tot[nt][3]);
    }
  }
}

// CTAs per SM: as many as the registers of a kDepth-block ring allow.
template <int NT>
constexpr int stream_ctas() { return NT == 1 ? 3 : 2; }

template <int NT, bool kBf16X, int GPB, bool kBf16S>
__global__ void __launch_bounds__(kStreamWarps * 32, stream_ctas<NT>()) w4_stream_kernel(const StreamParams p) {
  constexpr int kScaleBytes = kW4Rows * GPB * (kBf16S ? 2 : 4);
  constexpr int kBlockBytes = kW4CodeBytes + kScaleBytes;
  constexpr int kCols = 8 * NT;
  constexpr int kDepth = kScaleBytes > 64 ? 2 : 3;
  constexpr int kPartStride = kCols + 2;  // of a row: 16 rows on different banks
  constexpr int kPart = kW4Rows * kPartStride;  // one warp's sums of a tile
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int xstride = p.blocks * kW4Cols * 2 + kStreamPadBytes;
  // [warp][slot][row][col]: slot 0 a tile that an earlier warp began, 1 a whole
  // tile or, at the end, one that a later warp ends.
  float* part = reinterpret_cast<float*>(smem);
  uint8_t* xs = smem + 2 * kStreamWarps * kPart * 4;

  const int64_t tile0 = p.tiles * blockIdx.x / gridDim.x, tile1 = p.tiles * (blockIdx.x + 1) / gridDim.x;
  const int64_t run = (tile1 - tile0) * p.blocks;
  const auto warp_begin = [&](int w) { return run * w / kStreamWarps; };
  const int64_t b0 = warp_begin(warp), b1 = warp_begin(warp + 1);
  const uint8_t* src = p.packed + (tile0 * p.blocks + b0) * kBlockBytes + 16 * lane;
  const int soff = kW4CodeBytes - 16 * lane + g * (kScaleBytes / 8);
  int64_t left = b1 - b0;
  // The launch may begin while the one before it still runs. Until that has
  // ended nothing it may write is read: the first blocks are only asked into L2.
  if (lane == 0 && left > 0) {
    const int n = (int)(left < kDepth ? left : kDepth);
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "r"(n * kBlockBytes) : "memory");
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // Only now may the next launch begin: whatever it does before its own wait, the
  // work before this one is behind it.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  LaneBlock<GPB, kBf16S> ring[kDepth];
#pragma unroll
  for (int i = 0; i < kDepth; ++i)
    if (i < left) ring[i].load(src + i * kBlockBytes, src + i * kBlockBytes + soff);

  if (blockIdx.x == 0 && threadIdx.x == 0) *p.err = 0u;
  // x to bf16 columns (column piece * M + m), zeros past K; then one column of zeros.
  // All loads of a thread are in flight together (fp32: four, for registers): one
  // after another, 8 tokens of 6912 columns took 1.9 us longer.
  const int kpad = p.blocks * kW4Cols;
  if (kBf16X) {
    const int per = kpad / 8;
    for (int i = threadIdx.x; i < p.M * per; i += kStreamWarps * 32) {
      const int m = i / per, k = (i - m * per) * 8;
      const bool in = k < p.K;
      cp_async16_or_zero(smem_u32(xs + (size_t)m * xstride + k * 2),
                         static_cast<const uint16_t*>(p.x) + (in ? (int64_t)m * p.K + k : 0), in);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else {
    const int per = kpad / 4, all = p.M * per;
    const size_t plane = (size_t)p.M * xstride;
    constexpr int kAtOnce = 4;
    for (int i0 = threadIdx.x; i0 < all; i0 += kAtOnce * kStreamWarps * 32) {
      float4 v[kAtOnce];
#pragma unroll
      for (int q = 0; q < kAtOnce; ++q) {
        const int i = i0 + q * kStreamWarps * 32;
        const int m = i / per, k = (i - m * per) * 4;
        v[q] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i < all && k < p.K)
          v[q] = *reinterpret_cast<const float4*>(static_cast<const float*>(p.x) + (int64_t)m * p.K + k);
      }
#pragma unroll
      for (int q = 0; q < kAtOnce; ++q) {
        const int i = i0 + q * kStreamWarps * 32;
        if (i >= all) break;
        const int m = i / per, k = (i - m * per) * 4;
        const float f[4] = {v[q].x, v[q].y, v[q].z, v[q].w};
        uint32_t h[4], mi[4], l[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) split_bf16x3(f[j], h[j], mi[j], l[j]);
        uint8_t* d = xs + (size_t)m * xstride + k * 2;
        *reinterpret_cast<uint2*>(d) = make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
        *reinterpret_cast<uint2*>(d + plane) = make_uint2(mi[0] | (mi[1] << 16), mi[2] | (mi[3] << 16));
        *reinterpret_cast<uint2*>(d + 2 * plane) = make_uint2(l[0] | (l[1] << 16), l[2] | (l[3] << 16));
      }
    }
  }
  for (int i = threadIdx.x; i < kpad / 8; i += kStreamWarps * 32)
    *reinterpret_cast<uint4*>(xs + (size_t)p.cols * xstride + i * 16) = make_uint4(0u, 0u, 0u, 0u);
  __syncthreads();

  uint32_t xb[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
    xb[nt] = smem_u32(xs) + (8 * nt + g < p.cols ? 8 * nt + g : p.cols) * xstride + 16 * t;
  float tot[NT][4];
  const auto clear = [&]() {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) tot[nt][i] = 0.f;
  };
  const auto store_part = [&](int slot) {
    float* mine = part + (warp * 2 + slot) * kPart;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      *reinterpret_cast<float2*>(mine + g * kPartStride + 8 * nt + 2 * t) = make_float2(tot[nt][0], tot[nt][1]);
      *reinterpret_cast<float2*>(mine + (g + 8) * kPartStride + 8 * nt + 2 * t) = make_float2(tot[nt][2], tot[nt][3]);
    }
  };
  // y of a tile: this warp's sums in `slot`, and where `end` is not 0 slot 0 of
  // the warps after it whose run begins before block `end` of the CTA's run
  // (an empty run, of a CTA with fewer blocks than warps, holds nothing). Row
  // fastest, so 16 neighbouring y are written together. A lane's sums are added
  // side by side, warp after warp: one after the other, 16 tokens through 2560 x
  // 2560 took 10.9 us instead of 6.5 (two CTAs an SM).
  const auto write_tile = [&](int64_t tile, int slot, int64_t end) {
    constexpr int kMine = kW4Rows * kCols / 32;  // columns of a lane, every second one
    const int row = lane & (kW4Rows - 1), col0 = lane / kW4Rows;
    float* mine = part + (warp * 2 + slot) * kPart + row * kPartStride;
    float v[kMine];
#pragma unroll
    for (int i = 0; i < kMine; ++i)
      if (2 * i < p.cols) v[i] = mine[col0 + 2 * i];
    for (int w = warp + 1; w < kStreamWarps && warp_begin(w) < end; ++w) {
      if (warp_begin(w) == warp_begin(w + 1)) continue;
      const float* q = part + w * 2 * kPart + row * kPartStride + col0;
#pragma unroll
      for (int i = 0; i < kMine; ++i)
        if (2 * i < p.cols) v[i] += q[2 * i];
    }
    const int64_t n = tile * kW4Rows + row;
    if (kBf16X) {
#pragma unroll
      for (int i = 0; i < kMine; ++i)
        if (col0 + 2 * i < p.M && n < p.N) p.y[(int64_t)(col0 + 2 * i) * p.N + n] = v[i] * kW4Unit;
    } else {  // the columns of a token's pieces meet in this warp's slot
#pragma unroll
      for (int i = 0; i < kMine; ++i)
        if (2 * i < p.cols) mine[col0 + 2 * i] = v[i];
      __syncwarp();
      for (int m = col0; m < p.M; m += 2)
        if (n < p.N) p.y[(int64_t)m * p.N + n] = (mine[m] + (mine[m + p.M] + mine[m + 2 * p.M])) * kW4Unit;
    }
  };
  clear();
  int64_t tile = tile0 + b0 / p.blocks;
  int kb = (int)(b0 % p.blocks);  // block of the tile
  bool head = kb != 0;            // the tile was begun by an earlier warp
  const uint32_t xend = p.blocks * (kW4Cols * 2);
  uint32_t xk = kb * (kW4Cols * 2);
  while (left > 0) {
    src += kDepth * kBlockBytes;
    const uint8_t* ssrc = src + soff;
#pragma unroll
    for (int i = 0; i < kDepth; ++i) {
      if (i < left) {
        stream_block<NT, GPB, kBf16S>(ring[i], xb, xk, tot);
        xk += kW4Cols * 2;
        if (xk == xend) {
          store_part(head ? 0 : 1);
          if (!head) {
            __syncwarp();
            write_tile(tile, 1, 0);
            __syncwarp();
          }
          clear();
          head = false;
          xk = 0;
          ++tile;
        }
      }
      if (i + kDepth < left) ring[i].load(src + i * kBlockBytes, ssrc + i * kBlockBytes);
    }
    left -= kDepth;
  }
  if (xk != 0 && b1 > b0) store_part(head ? 0 : 1);
  __syncthreads();
  // The warp in which a shared tile begins adds it up.
  if (xk != 0 && b1 > b0 && !head) write_tile(tile, 1, (tile + 1 - tile0) * p.blocks);
}

size_t w4_stream_smem(int NT, int64_t cols, const W4Shape& sh) {
  return (size_t)2 * kStreamWarps * kW4Rows * (8 * NT + 2) * 4 +
         (size_t)(cols + 1) * ((size_t)sh.blocks() * kW4Cols * 2 + kStreamPadBytes);
}

template <int NT, bool kBf16X, int GPB, bool kBf16S>
cudaError_t launch_w4_stream_t(const StreamParams& p, int grid, size_t smem, cudaStream_t stream) {
  static std::atomic<uint64_t> allowed{0};
  auto kern = w4_stream_kernel<NT, kBf16X, GPB, kBf16S>;
  const cudaError_t e = allow_smem(kern, kStreamSmemMax, allowed);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kStreamWarps * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

template <int NT, bool kBf16X>
cudaError_t launch_w4_stream_n(const StreamParams& p, const W4Shape& sh, int grid, size_t smem, cudaStream_t stream) {
  const bool s16 = sh.scale_bytes == 2;
  switch (sh.group) {
    case 32: return s16 ? launch_w4_stream_t<NT, kBf16X, 4, true>(p, grid, smem, stream)
                        : launch_w4_stream_t<NT, kBf16X, 4, false>(p, grid, smem, stream);
    case 64: return s16 ? launch_w4_stream_t<NT, kBf16X, 2, true>(p, grid, smem, stream)
                        : launch_w4_stream_t<NT, kBf16X, 2, false>(p, grid, smem, stream);
    default: return s16 ? launch_w4_stream_t<NT, kBf16X, 1, true>(p, grid, smem, stream)
                        : launch_w4_stream_t<NT, kBf16X, 1, false>(p, grid, smem, stream);
  }
}

cudaError_t launch_w4_stream(const void* x, bool bf16, int64_t M, const W4Shape& sh, const uint8_t* packed, float* y,
                             uint32_t* err, cudaStream_t stream, int num_sms) {
  StreamParams p;
  p.x = x;
  p.packed = packed;
  p.y = y;
  p.err = err;
  p.M = (int)M;
  p.K = (int)sh.K;
  p.N = sh.N;
  p.cols = (int)(bf16 ? M : 3 * M);
  p.blocks = (int)sh.blocks();
  p.tiles = sh.tiles();
  const int NT = p.cols <= 8 ? 1 : 2;
  const size_t smem = w4_stream_smem(NT, p.cols, sh);
  int64_t per_sm = (227 * 1024) / (int64_t)(smem + 1024);
  // 9 to 16 columns: a second CTA on an SM stages x a second time, which pays only
  // where the SM has more than four tiles to stream (16 bf16 tokens through 2560
  // columns, one CTA against two: 160 tiles 5.6 / 6.5 us, 600 9.0 / 9.5, 864 10.1 /
  // 9.6, 8000 65 / 47; three weights in turn in a graph).
  const int most = NT == 1 ? stream_ctas<1>() : (p.tiles > 4 * (int64_t)num_sms ? stream_ctas<2>() : 1);
  per_sm = per_sm < 1 ? 1 : (per_sm > most ? most : per_sm);
  const int64_t slots = num_sms * per_sm;
  const int grid = (int)(p.tiles < slots ? p.tiles : slots);
  if (bf16)
    return NT == 1 ? launch_w4_stream_n<1, true>(p, sh, grid, smem, stream)
                   : launch_w4_stream_n<2, true>(p, sh, grid, smem, stream);
  return NT == 1 ? launch_w4_stream_n<1, false>(p, sh, grid, smem, stream)
                 : launch_w4_stream_n<2, false>(p, sh, grid, smem, stream);
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

bool w4_stream_fits(int64_t M, bool bf16, const W4Shape& sh) {
  const int64_t cols = bf16 ? M : 3 * M;
  return cols <= kW4StreamCols && w4_stream_smem(cols <= 8 ? 1 : 2, cols, sh) <= kStreamSmemMax;
}

cudaError_t launch_forward_w4(const void* x, bool bf16, int64_t M, const W4Shape& sh, const void* packed, float* y,
                              void* ws, cudaStream_t stream, int num_sms) {
  if (w4_stream_fits(M, bf16, sh))
    return launch_w4_stream(x, bf16, M, sh, static_cast<const uint8_t*>(packed), y, static_cast<uint32_t*>(ws), stream,
                            num_sms);
  return launch_w4_gemm(x, bf16, M, sh, static_cast<const uint8_t*>(packed), y, ws, stream, num_sms);
}

}  // namespace bl
