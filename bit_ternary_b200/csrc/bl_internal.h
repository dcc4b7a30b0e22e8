// bl_internal.h - declarations shared by the libbitlinear translation units.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "bl_device.cuh"

#include <cudaTypedefs.h>

#include <atomic>

namespace bl {

// Pack workspace: header (the sticky status word at 0, this call's status at
// 4, a count of finished CTAs at 8, mean_c and s at 16/20) + bins:
// kPackBins sums of significands by weight (bin b weighs 2^(max(b,1)-1) units
// of 2^-149) and, at kPackNonFiniteBin, a count of non-finite weights.
constexpr int kPackBins = 320;
constexpr int kPackNonFiniteBin = kPackBins - 1;
// After the bins: one fp64 partial sum of |W| per CTA of the first pass.
constexpr int kPackSumBlocks = 1024;
constexpr size_t kPackWsBytes = kHeaderBytes + kPackBins * sizeof(unsigned long long) + kPackSumBlocks * sizeof(double);

// Decode path (bl_decode.cu): at most 16 tokens per BitLinear, up to 8
// BitLinears per launch; their activation codes and a ring of at least two
// 16-row weight tiles must fit in shared memory.
constexpr int64_t kDecodeMaxM = 16;
constexpr int kDecodeMaxGroup = 8;                     // BitLinears per grouped launch
constexpr int kDecodeSlots = 16;                       // weight tiles tracked per CTA
constexpr int64_t kDecodeSmemShared = 110 * 1024;   // two CTAs per SM (room for the next launch)
constexpr int64_t kDecodeSmemMax = 225 * 1024;      // one CTA per SM

// I2_S conversion (bl_i2s.cu): to_i2s packs `in` (BitLinear words, D_in)
// into I2_S words at `out`; otherwise unpacks I2_S words at `in` into packed
// words at `out` and D_out. err (a device word, not cleared here) gets bit 0
// OR-ed in for a field holding 3 and bit 1 for a scale that is not finite and
// positive (or rows of D_in that differ).
cudaError_t launch_i2s(bool to_i2s, bool quarters, const void* in, void* out, const float* D_in, float* D_out,
                       int64_t N, int64_t K, uint32_t* err, cudaStream_t stream, int sms);

// One decode BitLinear. x: fp32 [M,K], bf16 bit patterns, or (prepared
// input) int8 codes in the forward workspace's private order with s_x (sx)
// and row sums (rs). y fp32 [M,N], or acc int32 [M,N] when acc is non-null.
struct DecCall {
  const void* x;
  const float* sx;
  const int32_t* rs;
  const uint32_t* packed;
  const float* D;
  float* y;
  int32_t* acc;
  int64_t M, N, K;
};

enum DecInput : int { kDecF32 = 0, kDecBf16 = 1, kDecPrepared = 2, kDecRms = 3 };

// Whether one call of M tokens and K columns (rms: with the RMSNorm input
// mode) fits the decode kernel, and whether a group of calls fits one launch.
bool decode_fits(int64_t M, int64_t K, bool rms);
bool decode_group_fits(const DecCall* calls, int n);
// One launch over n calls (all y or all acc). input: a DecInput; prepared and
// RMSNorm inputs take one call (g: norm weight [K], eps). pdl: launch with
// programmatic stream serialization (the packed weights and D may be read
// before the previous kernel in the stream has finished; activations are read
// after it). err: the workspace error word, cleared by the launch.
cudaError_t launch_decode(const DecCall* calls, int n, int input, const float* g, float eps, uint32_t* err, bool pdl,
                          cudaStream_t stream, int num_sms);

// The driver's cuTensorMapEncodeTiled (looked up once), or nullptr.
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

// W is fp32, or bf16 bit patterns when bf16 (widened exactly).
// clear_sticky: also zero the workspace's first word, where every call ORs in
// its failure (asynchronous packs leave it for bitlinear_pack_status).
cudaError_t launch_pack(const void* W, bool bf16, int64_t N, int64_t K, uint32_t* packed, float* D, void* ws,
                        bool clear_sticky, cudaStream_t stream, int num_sms);
// err_reset (nullable): the workspace error word, cleared by the kernel.
// x is fp32, or bf16 bit patterns when bf16 (widened exactly).
cudaError_t launch_act_quant(const void* x, bool bf16, int64_t M, int64_t K, int8_t* q, float* s_x, int32_t* rowsum,
                             bool permuted, cudaStream_t stream, uint32_t* err_reset);
// RMSNorm (weight g [K], eps) then ActQuant, per token; K <= kRmsMaxK.
constexpr int64_t kRmsMaxK = 16384;
cudaError_t launch_rms_act_quant(const float* x, const float* g, float eps, int64_t M, int64_t K, int8_t* q,
                                 float* s_x, int32_t* rowsum, bool permuted, cudaStream_t stream,
                                 uint32_t* err_reset);
// Natural-order int8 codes and scales (bitlinear_quant_act's output) into the
// forward workspace layout (private order, row sums); err_reset as above.
cudaError_t launch_q_prepare(const int8_t* q, const float* s_x, int64_t M, int64_t K, int8_t* wq, float* wsx,
                             int32_t* wrs, cudaStream_t stream, uint32_t* err_reset);
// Expects the permuted activations, s_x and row sums already in the forward
// workspace (launch_act_quant with permuted = true).
cudaError_t launch_gemm(int64_t M, int64_t N, int64_t K, const uint32_t* packed, const float* D, float* y,
                        int32_t* acc_out, void* ws, cudaStream_t stream, int num_sms);
// The same tensor-core kernel over the K range [k0, k0 + K) of rows that are
// kfull columns long (k0 % 16 == 0): the weights' words and the workspace's
// activation codes of that range, the row sums of the codes over it (rowsum,
// or the workspace's when null), D[n * dstride], and with accumulate the
// rescaled tile is added to y (one fp32 rounding per element) instead of
// stored.
struct GemmSlice {
  int64_t k0;
  int64_t kfull;
  int dstride;
  bool accumulate;
  const int32_t* rowsum;
};
cudaError_t launch_gemm_slice(int64_t M, int64_t N, int64_t K, const GemmSlice& sl, const uint32_t* packed,
                              const float* D, float* y, int32_t* acc_out, void* ws, cudaStream_t stream,
                              int num_sms);

// Per-256-block scale variant (bl_block.cu): blocks of 256 consecutive
// columns within a row, D fp32 [N, scale_blocks(K)].
constexpr int kScaleBlock = 256;
inline int64_t scale_blocks(int64_t K) { return (K + kScaleBlock - 1) / kScaleBlock; }
constexpr size_t kBlockFwdSmemMax = 200 * 1024;
// status: a device word that gets bit 0 OR-ed in for a block holding a
// non-finite weight (that block's words and scale are left unwritten).
// W is fp32, or bf16 bit patterns when bf16 (widened exactly).
cudaError_t launch_pack_blocks(const void* W, bool bf16, int64_t N, int64_t K, uint32_t* packed, float* D,
                               uint32_t* status, cudaStream_t stream, int num_sms);
// Tokens per CTA tile of the block forward (its activation codes fit in
// kBlockFwdSmemMax of shared memory); always >= 1 for K <= kMaxK.
int block_forward_tile(int64_t M, int64_t K);
// One token with K % 256 == 0 and K <= kBlockDecMaxK: a single launch that
// quantises x in every CTA. Otherwise ActQuant into the forward workspace ws
// (private order), then the contraction as its programmatic dependent.
constexpr int kBlockDecMaxK = 32 * kScaleBlock;
// From this many tokens on, the block forward runs one tensor-core GEMM per
// block; its workspace then also holds the per-block row sums of the codes.
constexpr int64_t kBlockGemmMinM = 128;
inline size_t ws_blocks_bytes(int64_t M, int64_t K) {
  return ws_forward_bytes(M, K) + align256(4 * (size_t)M * (size_t)scale_blocks(K));
}
// x is fp32, or bf16 bit patterns when bf16 (widened exactly).
cudaError_t launch_forward_blocks(const void* x, bool bf16, int64_t M, int64_t N, int64_t K, const uint32_t* packed,
                                  const float* D, float* y, void* ws, cudaStream_t stream, int num_sms);

// 4-bit weights with group scales (bl_w4.cu). The packed buffer is a run of
// 16-row tiles, each a run of ceil(K / 128) blocks. A block is 16 rows x 64
// bytes of codes, then its 128 / group scales of each row, [row % 8][group]
// [row / 8] (a lane's two rows and all their groups side by side). Row r
// of a block holds 16 words, word 4*t + j the columns 32*j + 8*t .. + 7: the
// 16 bytes that lane (r % 8, t) of a 16x8x16 matrix instruction takes from the
// row, so a warp's load of eight rows is 512 consecutive bytes, and a thread
// that owns a whole row reads 64. Nibble p of a word (p < 4) is column 2p of
// its eight, nibble 4 + p column 2p + 1: (word >> 4p) & 0x000F000F is a pair
// of neighbouring columns in the halves of a register. Stored as c + 8.
constexpr int kW4Rows = 16;
constexpr int kW4Cols = 128;
constexpr int kW4CodeBytes = kW4Rows * kW4Cols / 2;
struct W4Shape {
  int64_t N, K;
  int group;       // 32, 64 or 128
  int scale_bytes; // 4 (fp32) or 2 (bf16)
  __host__ __device__ int64_t tiles() const { return (N + kW4Rows - 1) / kW4Rows; }
  __host__ __device__ int64_t blocks() const { return (K + kW4Cols - 1) / kW4Cols; }
  __host__ __device__ int scale_index(int row, int gi) const {  // row of 16, group of the block
    return ((row & 7) * (kW4Cols / group) + gi) * 2 + (row >> 3);
  }
  __host__ __device__ int64_t groups() const { return (K + group - 1) / group; }
  __host__ __device__ int block_bytes() const { return kW4CodeBytes + kW4Rows * (kW4Cols / group) * scale_bytes; }
  __host__ __device__ size_t bytes() const { return (size_t)tiles() * (size_t)blocks() * (size_t)block_bytes(); }
};
// status: a device word that gets bit 0 OR-ed in for a group holding a
// non-finite weight (that group is packed as zeros).
cudaError_t launch_w4_pack(const void* W, bool bf16, const W4Shape& sh, void* packed, uint32_t* status,
                           cudaStream_t stream, int num_sms);
cudaError_t launch_w4_import(const uint8_t* codes, const void* S, const W4Shape& sh, void* packed,
                             cudaStream_t stream, int num_sms);
cudaError_t launch_w4_export(const void* packed, const W4Shape& sh, int8_t* codes, void* S, cudaStream_t stream,
                             int num_sms);
// The three bf16 pieces of an fp32 x: its significand cut into 8 + 8 + 8 bits,
// so h + m + l == x exactly (bits under 2^-133, which only |x| < 2^-110 can
// have, are dropped). A non-finite x is h alone.
__device__ __forceinline__ void split_bf16x3(float x, uint32_t& h, uint32_t& m, uint32_t& l) {
  const uint32_t b = __float_as_uint(x);
  if ((b & 0x7F800000u) == 0x7F800000u) {
    h = (b >> 16) | ((b & 0x007FFFFFu) != 0u ? 0x0040u : 0u);  // a NaN stays one
    m = 0u;
    l = 0u;
    return;
  }
  h = b >> 16;
  const float r = x - __uint_as_float(b & 0xFFFF0000u);
  const uint32_t rb = __float_as_uint(r);
  m = rb >> 16;
  l = __float_as_uint(r - __uint_as_float(rb & 0xFFFF0000u)) >> 16;
}
// Eight codes of a packed word to four bf16 pairs of c * 2^-6. A bf16 whose
// bits are an integer v below 256 is v * 2^-133 (subnormals and the first
// binade are one line), so a nibble masked out where it stands, at bit 0 or at
// bit 4 of a half, is u * 2^-133 or u * 2^-129 without a shift or an offset.
// One fused multiply-add, exact, brings both to (u - 8) * 2^-6 = c * 2^-6:
// nine instructions a word, five of them on the integer pipe.
constexpr float kW4Unit = 64.0f;  // 2^6, what a sum of products is multiplied by
__device__ __forceinline__ void w4_unpack(uint32_t w, uint32_t (&pair)[4]) {
  const uint32_t v = w >> 8;
  const uint32_t off = 0xBE00BE00u;                          // -8 * 2^-6
  const uint32_t up0 = 0x7F007F00u, up1 = 0x7D007D00u;       // 2^127, 2^123
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(pair[0]) : "r"(w & 0x000F000Fu), "r"(up0), "r"(off));
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(pair[1]) : "r"(w & 0x00F000F0u), "r"(up1), "r"(off));
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(pair[2]) : "r"(v & 0x000F000Fu), "r"(up0), "r"(off));
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(pair[3]) : "r"(v & 0x00F000F0u), "r"(up1), "r"(off));
}
// The one-launch kernel for few tokens (bl_w4.cu) holds x in shared memory as
// bf16 columns: a token of bf16 x is one, a token of fp32 x three. Up to 16, two
// matrix instructions a step: 16 bf16 tokens take 5.6 us through 2560 x 2560 and
// 9.1 through 13824 x 2560 (weights in L2), where the tensor-core kernel takes 7.9 and 11.8.
constexpr int kW4StreamCols = 16;
bool w4_stream_fits(int64_t M, bool bf16, const W4Shape& sh);
// Most parts of K whose partial sums the workspace holds: none where tiles of 128
// x 128 fill a B200's 148 SMs by themselves, or where a part's sums would not
// start on a 16-byte boundary.
constexpr int kW4MaxParts = 8;
inline int w4_parts(int64_t M, int64_t N) {
  const int64_t tiles = ((M + 127) / 128) * ((N + 127) / 128);
  return tiles < 148 && (M * N) % 4 == 0 ? kW4MaxParts : 1;
}
// [header | x as three bf16 planes | partial sums]
inline size_t ws_w4_bytes(int64_t M, int64_t N, int64_t K) {
  const int parts = w4_parts(M, N);
  return kHeaderBytes + align256(6 * (size_t)M * (size_t)K) +
         (parts > 1 ? align256(4 * (size_t)parts * (size_t)M * (size_t)N) : 0);
}
// The tensor-core kernel for many tokens (bl_w4_gemm.cu).
cudaError_t launch_w4_gemm(const void* x, bool bf16, int64_t M, const W4Shape& sh, const uint8_t* packed, float* y,
                           void* ws, cudaStream_t stream, int num_sms);
// x is fp32, or bf16 bit patterns when bf16.
cudaError_t launch_forward_w4(const void* x, bool bf16, int64_t M, const W4Shape& sh, const void* packed, float* y,
                              void* ws, cudaStream_t stream, int num_sms);

// Sampling (bl_sample.cu). Settings as in bl_sampling.
constexpr int64_t kSampleMaxV = 4194304;
struct SampleHow {
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  float temperature_value;
  int32_t top_k_value;
  float top_p_value;
  float min_p_value;
};
cudaError_t launch_sample(const void* logits, bool bf16, int64_t B, int64_t V, int64_t ld, const SampleHow& how,
                          const float* u, int64_t* tokens, float* logprobs, cudaStream_t stream, int num_sms);

// Shared memory beyond 48 KB, and clusters of more than 8 CTAs, have to be
// allowed once per kernel and device.
template <typename Kernel>
cudaError_t allow_smem(Kernel kern, size_t bytes, std::atomic<uint64_t>& done, bool large_clusters = false) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if ((done.load(std::memory_order_relaxed) & bit) != 0) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess && large_clusters) e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

cudaError_t launch_selftest_wait(uint32_t* err, uint64_t limit_ns, cudaStream_t stream);

}  // namespace bl
