// bl_w4_gemm.cu - the 4-bit group-scale product of many tokens on the 5th-generation
// tensor cores (tcgen05.mma kind::f16, fp32 accumulators in tensor memory).
//
//   y[m,n] = sum_G S[n,G] * (sum over k in G of c[n,k] * x[m,k])
//
// Tile: H x 128 weight rows (MMA M) x BN tokens (MMA N); a stage is 128 columns
// of K, one block of the packed weights for each of 8 H row tiles. With H = 1
// every byte of x that TMA writes to shared memory is read by one MMA, and both
// together take all of its bandwidth (an MMA every ~100 cycles instead of 64 for
// 128 tokens); H = 2 uses a stage of x for two halves of the rows. Where the
// tiles leave SMs idle, K is cut into parts: partial sums go to the workspace
// and a second launch adds them in order.
//   A = the codes as bf16 (c * 2^-6, exact), unpacked by four warps from
//       registers into TMEM (tcgen05.st), a ring of stages.
//   B = x as bf16, loaded by TMA with 128-byte swizzle: the caller's own bf16 x,
//       or the three pieces of an fp32 x, which take three MMAs over one A
//       stage into one accumulator.
//   D = one group's sum: a scale multiplies sums over its 32, 64 or 128 columns
//       only, so each group has an accumulator of its own (a ring in TMEM), which
//       eight drain warps read, multiply by the row's scale and add to the
//       tile's sums in registers. Scaling the weights instead would round them
//       to bf16.
// Warp roles: 0 TMA producer (TMEM owner), 1 MMA issuer, 4..7 unpack, 8..15
// drain (a warp owns 32 rows x BN / 2 tokens, or 32 rows of its half x BN). The
// scheduler slots they share bound it: beside twelve busy warps an instruction of
// the MMA issuer takes about 8 cycles, so its loop holds little but MMAs, and a
// group of 32 columns (two MMAs, then a drain) costs twice one of 128.
// Measured back to back, bf16 x, 13824 x 2560: 4096 tokens 248 us at full clock (1170
// TFLOP/s, 69% of cuBLAS's bf16 rate; 270 to 290 where the power cap holds the clock),
// with groups of 32 564 us; 1024 tokens, groups of 64, 89 us. fp32 x, 2560 x 6912,
// 512 tokens: 48 us (1130 TFLOP/s of bf16 MMAs).
// Every barrier wait is bounded in time; a timeout sets a shared abort flag and
// the workspace's error word, and all roles run out and exit.
#include "bl_internal.h"

#include <atomic>
#include <cstring>

namespace bl {

namespace {

constexpr int kBM = 128;
constexpr int kStageK = kW4Cols;
constexpr int kACols = kStageK / 2;  // TMEM columns of an A stage (two bf16 each)
constexpr uint32_t kTmemCols = 512;
constexpr int kUnpackWarp0 = 4;
constexpr int kDrainWarp0 = 8;
constexpr int kDrainWarps = 8;
constexpr int kThreads = 32 * (kDrainWarp0 + kDrainWarps);
constexpr size_t kSmemMax = 227 * 1024;

template <int BN, int H, int PLANES>
struct Shape {
  // Group accumulators in flight: with H = 2 one per half, drained while the other half's fills.
  static constexpr int kDBufs = H == 2 || BN == 128 ? 2 : 4;
  static constexpr int kAStages = H == 2 ? 2 : 4;
  static constexpr int kACol = kDBufs * BN;
  static constexpr int kAStageCols = H * kACols;
  static constexpr uint32_t kBoxBytes = BN * 128;   // BN tokens x 64 columns
  static constexpr uint32_t kBStageBytes = PLANES * 2 * kBoxBytes;
  static constexpr int kBStages = (int)((200 * 1024) / kBStageBytes) < 6 ? (int)((200 * 1024) / kBStageBytes) : 6;
  static constexpr int kWarpTokens = H == 2 ? BN : BN / 2;
  static constexpr int kDrainers = kDrainWarps / H;  // warps that read an accumulator
  static_assert(kACol + kAStages * kAStageCols <= (int)kTmemCols, "TMEM budget");
  static_assert(kBStages >= 2 && kBoxBytes % 1024 == 0, "shared memory ring");
};

template <int BN, int H, int PLANES>
struct Sync {
  using Sh = Shape<BN, H, PLANES>;
  // Each empty_x right after its full_x (the MMA issuer counts on it).
  uint64_t full_b[Sh::kBStages];
  uint64_t empty_b[Sh::kBStages];
  uint64_t full_a[Sh::kAStages];
  uint64_t empty_a[Sh::kAStages];
  uint64_t acc_full[Sh::kDBufs];
  uint64_t acc_empty[Sh::kDBufs];
  uint64_t drain;
  uint32_t tmem_base;
  int abort_flag;
};

struct Params {
  const uint8_t* packed;
  float* y;           // or the partial sums [parts][M][N]
  uint32_t* err;
  int M;
  int64_t N;
  int64_t row_tiles;  // 16-row tiles of the packed weight
  int blocks;         // 128-column blocks per row: stages per tile
  int tiles_n;
  int parts;          // of K
  int units;          // tiles x parts
};

// One CTA's share: a part of a tile, stages kb .. kb_end.
struct Unit {
  int tile, part, kb, kb_end;
  __device__ __forceinline__ Unit(const Params& p, int local) {
    const int u = blockIdx.x + local * gridDim.x;
    tile = u / p.parts;
    part = u - tile * p.parts;
    kb = (int)((int64_t)p.blocks * part / p.parts);
    kb_end = (int)((int64_t)p.blocks * (part + 1) / p.parts);
  }
};

template <int BN, int H, int PLANES>
constexpr size_t smem_bytes() {
  return 1024 + (size_t)Shape<BN, H, PLANES>::kBStages * Shape<BN, H, PLANES>::kBStageBytes +
         ((sizeof(Sync<BN, H, PLANES>) + 127) & ~size_t(127));
}

__device__ __forceinline__ void tma_load_3d(void* smem_dst, const void* tmap, int32_t c0, int32_t c1, int32_t c2,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar))
      : "memory");
}

// D[tmem] (+)= A[tmem] * B[smem]^T, bf16 operands, fp32 accumulate.
__device__ __forceinline__ void umma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// fp32 accumulator, bf16 A and B, both K-major.
constexpr uint32_t umma_idesc_bf16(int M, int N) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (uint32_t(N >> 3) << 17) | (uint32_t(M >> 4) << 24);
}

// acc.xy += v.xy * s.xx (two fp32 multiply-adds)
__device__ __forceinline__ void fma2(float& a0, float& a1, uint32_t v0, uint32_t v1, uint64_t ss) {
  asm("{\n\t.reg .b64 a, v;\n\t"
      "mov.b64 a, {%0, %1};\n\t"
      "mov.b64 v, {%2, %3};\n\t"
      "fma.rn.f32x2 a, v, %4, a;\n\t"
      "mov.b64 {%0, %1}, a;\n\t}"
      : "+f"(a0), "+f"(a1)
      : "r"(v0), "r"(v1), "l"(ss));
}

// 16, 32 or 64 consecutive TMEM columns of the warp's 32 lanes.
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
        "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t (&v)[32]) { tmem_ld_32x32b_x32(taddr, v); }
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t (&v)[64]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, "
      "%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, "
      "%48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%64];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
        "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]),
        "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]),
        "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31]),
        "=r"(v[32]), "=r"(v[33]), "=r"(v[34]), "=r"(v[35]), "=r"(v[36]), "=r"(v[37]), "=r"(v[38]), "=r"(v[39]),
        "=r"(v[40]), "=r"(v[41]), "=r"(v[42]), "=r"(v[43]), "=r"(v[44]), "=r"(v[45]), "=r"(v[46]), "=r"(v[47]),
        "=r"(v[48]), "=r"(v[49]), "=r"(v[50]), "=r"(v[51]), "=r"(v[52]), "=r"(v[53]), "=r"(v[54]), "=r"(v[55]),
        "=r"(v[56]), "=r"(v[57]), "=r"(v[58]), "=r"(v[59]), "=r"(v[60]), "=r"(v[61]), "=r"(v[62]), "=r"(v[63])
      : "r"(taddr)
      : "memory");
}

// The whole warp waits; the outcome is warp-uniform.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, uint32_t* err,
                                          uint32_t code) {
  if (__all_sync(0xFFFFFFFFu, mbar_try_wait(bar, parity))) return true;
  int ok = 0;
  if ((threadIdx.x & 31) == 0) ok = mbar_wait(bar, parity, abort_flag, err, code) ? 1 : 0;
  ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
  return ok != 0;
}

template <int kRegs>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

__device__ __forceinline__ bool mbar_try_wait_at(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ void tc_commit_at(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xFFFFFFFF;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

template <int N>
__device__ __forceinline__ void ring_next(int& s, uint32_t& ph) {
  if (++s == N) {
    s = 0;
    ph ^= 1;
  }
}

template <int BN, int H, int PLANES, int GPB, bool kBf16S>
__global__ void __launch_bounds__(kThreads, 1)
    w4_gemm_kernel(const __grid_constant__ CUtensorMap tmap_x, const Params p) {
  using Sh = Shape<BN, H, PLANES>;
  constexpr int kBStages = Sh::kBStages, kAStages = Sh::kAStages, kDBufs = Sh::kDBufs, kACol = Sh::kACol;
  constexpr int kBlockBytes = kW4CodeBytes + kW4Rows * GPB * (kBf16S ? 2 : 4);
  constexpr int kSteps = kStageK / GPB / 16;  // MMAs of one group and piece
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sB = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Sync<BN, H, PLANES>& S = *reinterpret_cast<Sync<BN, H, PLANES>*>(sB + (size_t)kBStages * Sh::kBStageBytes);

  // Warp-uniform by construction, so that what follows from it stays in uniform registers.
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int my_units = p.units > (int)blockIdx.x ? (p.units - 1 - (int)blockIdx.x) / (int)gridDim.x + 1 : 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kBStages; ++s) {
      mbar_init(&S.full_b[s], 1);
      mbar_init(&S.empty_b[s], 1);
    }
    for (int s = 0; s < kAStages; ++s) {
      mbar_init(&S.full_a[s], 4);
      mbar_init(&S.empty_a[s], 1);
    }
    for (int b = 0; b < kDBufs; ++b) {
      mbar_init(&S.acc_full[b], 1);
      mbar_init(&S.acc_empty[b], Sh::kDrainers);
    }
    mbar_init(&S.drain, 1);
    S.abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tmap_x);
  }
  if (warp == 0) {
    tmem_alloc(&S.tmem_base, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, S.tmem_base, 0);
  volatile int* abort_flag = &S.abort_flag;
  // The launch may begin while the one before it runs; nothing that one may
  // write is read before it has ended.
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // 128 registers a thread at launch, shared out anew among the four groups of
  // four warps: 40 + 120 + 176 + 176 = 512.
  if (warp < kUnpackWarp0) {
    regs_down<40>();
    if (warp == 0) {
      // ------------------------------------------------ TMA producer (x)
      if (lane == 0) {
        int s = 0;
        uint32_t ph = 0;
        int issued = 0;
        for (int lt = 0; lt < my_units; ++lt) {
          const Unit u(p, lt);
          const int m0 = (u.tile / p.tiles_n) * BN;
          for (int kb = u.kb; kb < u.kb_end; ++kb) {
            if (!mbar_wait(&S.empty_b[s], ph ^ 1, abort_flag, p.err, kDevTimeoutProducer)) {
              lt = my_units;
              break;
            }
            // Columns past K and tokens past M arrive as zeros.
            mbar_arrive_expect_tx(&S.full_b[s], Sh::kBStageBytes);
#pragma unroll
            for (int pl = 0; pl < PLANES; ++pl)
#pragma unroll
              for (int h = 0; h < 2; ++h)
                tma_load_3d(sB + (size_t)s * Sh::kBStageBytes + (pl * 2 + h) * Sh::kBoxBytes, &tmap_x,
                            kb * kStageK + 64 * h, m0, pl, &S.full_b[s]);
            ++issued;
            ring_next<kBStages>(s, ph);
          }
        }
        // Let every issued copy land before the CTA can exit.
        const int first = issued > kBStages ? issued - kBStages : 0;
        for (int j = first; j < issued; ++j)
          mbar_wait(&S.full_b[j % kBStages], (j / kBStages) & 1, nullptr, p.err, kDevTimeoutDrain, 100000000ull);
      }
    } else if (warp == 1) {
      // ------------------------------------------------ MMA issuer
      // The whole warp walks the groups and one lane issues, so that descriptors
      // and addresses stay in uniform registers, as the instruction wants them
      // (a lane of its own, in a divergent branch, needed 135 cycles an MMA for
      // the moves, where 128 tokens take the tensor pipe 64). The pipe's queue
      // covers a few MMAs, and beside busy warps every instruction between two
      // groups costs this warp some eight cycles: barriers are 32-bit addresses
      // counted up, all of a group's are tried at once, and stages are counted in
      // 32 bits.
      const uint32_t idesc = umma_idesc_bf16(kBM, BN);
      const uint64_t bdesc0 = umma_sdesc_sw128(sB);
      const uint32_t bhi = (uint32_t)(bdesc0 >> 32), blo0 = (uint32_t)bdesc0;
      const uint32_t a0 = smem_u32(&S.full_a[0]), b0 = smem_u32(&S.full_b[0]), d0 = smem_u32(&S.acc_full[0]);
      constexpr uint32_t kAEmpty = kAStages * 8, kBEmpty = kBStages * 8, kDEmpty = kDBufs * 8;  // empty_x follows full_x
      uint32_t sb = 0, sa = 0, d = 0;
      uint32_t phb = 0, pha = 0, phd = 1;
      bool ok = true;
      uint32_t stages = 0;
      for (int lt = 0; lt < my_units; ++lt) {
        const Unit u(p, lt);
        stages += u.kb_end - u.kb;
      }
      constexpr int kGroups = GPB * H;  // accumulators of a stage: group by group, half by half
      for (uint32_t j = 0; j < stages && ok; ++j) {
        const uint32_t blo = blo0 + sb * (Sh::kBStageBytes >> 4);
        const uint32_t a_tmem = tmem + kACol + Sh::kAStageCols * sa;
#pragma unroll
        for (int gh = 0; gh < kGroups; ++gh) {
          const int gi = gh / H, h = gh % H;
          bool there = mbar_try_wait_at(d0 + kDEmpty + 8 * d, phd);
          if (gh == 0) there = there & mbar_try_wait_at(a0 + 8 * sa, pha) & mbar_try_wait_at(b0 + 8 * sb, phb);
          if (!__all_sync(0xFFFFFFFFu, there)) {
            ok = (gh != 0 || (warp_wait(&S.full_a[sa], pha, abort_flag, p.err, kDevTimeoutMma) &&
                              warp_wait(&S.full_b[sb], phb, abort_flag, p.err, kDevTimeoutMma))) &&
                 warp_wait(&S.acc_empty[d], phd, abort_flag, p.err, kDevTimeoutMma);
            if (!ok) break;
          }
          tc_fence_after();
          if (elect_one()) {
            const uint32_t d_tmem = tmem + d * BN;
#pragma unroll
            for (int q = 0; q < PLANES; ++q) {
              const int pl = PLANES - 1 - q;  // the smallest piece first
#pragma unroll
              for (int k = 0; k < kSteps; ++k) {
                const int ks = gi * kSteps + k;  // 16-column step of the stage
                const uint32_t lo = blo + (pl * 2 + (ks >> 2)) * (Sh::kBoxBytes >> 4) + 2 * (ks & 3);
                umma_bf16_ts(d_tmem, a_tmem + kACols * h + 8 * ks, ((uint64_t)bhi << 32) | lo, idesc,
                             (q | k) != 0 ? 1u : 0u);
              }
            }
            tc_commit_at(d0 + 8 * d);
            if (gh == kGroups - 1) {
              tc_commit_at(a0 + kAEmpty + 8 * sa);
              tc_commit_at(b0 + kBEmpty + 8 * sb);
            }
          }
          __syncwarp();
          d = d + 1 == kDBufs ? 0 : d + 1;
          phd ^= d == 0 ? 1u : 0u;
        }
        sa = sa + 1 == kAStages ? 0 : sa + 1;
        pha ^= sa == 0 ? 1u : 0u;
        sb = sb + 1 == kBStages ? 0 : sb + 1;
        phb ^= sb == 0 ? 1u : 0u;
      }
      // All issued MMAs complete before TMEM is released.
      if (elect_one()) {
        tc_commit(&S.drain);
        mbar_wait(&S.drain, 0, nullptr, p.err, kDevTimeoutDrain, 100000000ull);
      }
      __syncwarp();
    }
  } else if (warp < kDrainWarp0) {
    // ------------------------------------------------ unpack: one weight row of each half per thread
    regs_down<120>();
    if (warp == kUnpackWarp0 && lane == 0 && blockIdx.x == 0) *p.err = 0u;
    const int quarter = warp & 3;  // TMEM lane quarter (hardware rule: warp id % 4)
    const int row = quarter * 32 + lane;
    const uint32_t lane_base = tmem + ((uint32_t)(quarter * 32) << 16);
    constexpr int kAhead = H == 2 ? 2 : 3;  // stages of codes in flight
    uint4 buf[kAhead][H][4];
    int lt = 0, kb = 0, kb_end = 0;  // the next stage to load
    const uint8_t* src[H];
    const auto load = [&](uint4(&w)[H][4]) {  // false past the last stage
      if (kb == kb_end) {
        if (lt == my_units) return false;
        const Unit u(p, lt++);
        kb = u.kb;
        kb_end = u.kb_end;
#pragma unroll
        for (int h = 0; h < H; ++h) {
          int64_t rt = ((int64_t)(u.tile % p.tiles_n) * H + h) * (kBM / kW4Rows) + (row / kW4Rows);
          rt = rt < p.row_tiles ? rt : p.row_tiles - 1;  // rows past the last tile: anything in bounds
          src[h] = p.packed + (rt * p.blocks + kb) * kBlockBytes + (row % kW4Rows) * (kStageK / 2);
        }
      }
#pragma unroll
      for (int h = 0; h < H; ++h) {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[h][i] = *(reinterpret_cast<const uint4*>(src[h]) + i);
        src[h] += kBlockBytes;
      }
      ++kb;
      return true;
    };
    bool have[kAhead];
#pragma unroll
    for (int q = 0; q < kAhead; ++q) have[q] = load(buf[q]);
    int s = 0;
    uint32_t ph = 0;
    for (bool ok = true; ok && have[0];) {
#pragma unroll
      for (int q = 0; q < kAhead; ++q) {
        if (!have[q] || !ok) break;
        if (!warp_wait(&S.empty_a[s], ph ^ 1, abort_flag, p.err, kDevTimeoutUnpack)) {
          ok = false;
          break;
        }
        tc_fence_after();
        // Word (t, j) of a row holds columns 32 j + 8 t ..: pairs 16 j + 4 t .. of the stage.
#pragma unroll
        for (int h = 0; h < H; ++h) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t v[32];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
              const uint32_t w0 = c == 0 ? buf[q][h][t].x : buf[q][h][t].z;
              const uint32_t w1 = c == 0 ? buf[q][h][t].y : buf[q][h][t].w;
              uint32_t pr[4];
              w4_unpack(w0, pr);
#pragma unroll
              for (int i = 0; i < 4; ++i) v[4 * t + i] = pr[i];
              w4_unpack(w1, pr);
#pragma unroll
              for (int i = 0; i < 4; ++i) v[16 + 4 * t + i] = pr[i];
            }
            tmem_st_32x32b_x32(lane_base + kACol + Sh::kAStageCols * s + kACols * h + 32 * c, v);
          }
        }
        have[q] = load(buf[q]);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.full_a[s]);
        ring_next<kAStages>(s, ph);
      }
    }
  } else {
    // ------------------------------------------------ drain: 32 rows x kWarpTokens tokens per warp
    regs_up<176>();
    constexpr int kTok = Sh::kWarpTokens;
    constexpr int kChunk = kTok == 128 ? 32 : kTok;
    const int quarter = warp & 3, half = (warp - kDrainWarp0) >> 2;  // of the tokens, or (H = 2) of the rows
    const int row = quarter * 32 + lane;
    const uint32_t lane_base = tmem + ((uint32_t)(quarter * 32) << 16) + (H == 2 ? 0 : half * kTok);
    const int soff = kW4CodeBytes + ((row & 7) * GPB * 2 + ((row >> 3) & 1)) * (kBf16S ? 2 : 4);
    int d = H == 2 ? half : 0;
    uint32_t ph = 0;
    bool ok = true;
    for (int lt = 0; lt < my_units && ok; ++lt) {
      const Unit u(p, lt);
      const int m0 = (u.tile / p.tiles_n) * BN + (H == 2 ? 0 : half * kTok);
      const int64_t n = ((int64_t)(u.tile % p.tiles_n) * H + (H == 2 ? half : 0)) * kBM + row;
      int64_t rt = n / kW4Rows;
      rt = rt < p.row_tiles ? rt : p.row_tiles - 1;
      const uint8_t* sp = p.packed + (rt * p.blocks + u.kb) * kBlockBytes + soff;
      // Bits as loaded: a conversion here would wait for the load (500 cycles a
      // stage), where it is only used a stage later.
      const auto scale_bits = [&](int gi) -> uint32_t {
        if (kBf16S) return *(reinterpret_cast<const uint16_t*>(sp) + 2 * gi);
        return *(reinterpret_cast<const uint32_t*>(sp) + 2 * gi);
      };
      float acc[kTok];
#pragma unroll
      for (int i = 0; i < kTok; ++i) acc[i] = 0.f;
      uint32_t sc[GPB];
#pragma unroll
      for (int gi = 0; gi < GPB; ++gi) sc[gi] = scale_bits(gi);
      for (int kb = u.kb; kb < u.kb_end && ok; ++kb) {
        uint32_t nsc[GPB] = {};
        sp += kBlockBytes;
        if (kb + 1 < u.kb_end) {
#pragma unroll
          for (int gi = 0; gi < GPB; ++gi) nsc[gi] = scale_bits(gi);
        }
#pragma unroll
        for (int gi = 0; gi < GPB; ++gi) {
          if (ok && !warp_wait(&S.acc_full[d], ph, abort_flag, p.err, kDevTimeoutEpilogue)) ok = false;
          if (ok) {
            tc_fence_after();
            uint64_t ss;
            asm("mov.b64 %0, {%1, %1};" : "=l"(ss) : "r"(kBf16S ? sc[gi] << 16 : sc[gi]));
#pragma unroll
            for (int c = 0; c < kTok; c += kChunk) {
              uint32_t v[kChunk];
              tmem_ld_cols(lane_base + d * BN + c, v);
              tmem_wait_ld();
              if (c + kChunk == kTok) {  // all of it is in registers
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&S.acc_empty[d]);
              }
#pragma unroll
              for (int i = 0; i < kChunk; i += 2) fma2(acc[c + i], acc[c + i + 1], v[i], v[i + 1], ss);
            }
            if (H == 2) ph ^= 1;
            else ring_next<kDBufs>(d, ph);
          }
        }
#pragma unroll
        for (int gi = 0; gi < GPB; ++gi) sc[gi] = nsc[gi];
      }
      if (ok && n < p.N) {
        float* out = p.y + ((int64_t)u.part * p.M + m0) * p.N + n;
#pragma unroll
        for (int i = 0; i < kTok; ++i) {
          if (m0 + i < p.M) __stcs(out, acc[i] * kW4Unit);
          out += p.N;
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// The three bf16 pieces of an fp32 x [M, K], planes [3][M][K].
__global__ void __launch_bounds__(256) w4_split_kernel(const float4* x, int64_t n4, uint2* planes) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n4; i += (int64_t)gridDim.x * 256) {
    const float4 v = x[i];
    const float f[4] = {v.x, v.y, v.z, v.w};
    uint32_t h[4], m[4], l[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) split_bf16x3(f[j], h[j], m[j], l[j]);
    planes[i] = make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
    planes[n4 + i] = make_uint2(m[0] | (m[1] << 16), m[2] | (m[3] << 16));
    planes[2 * n4 + i] = make_uint2(l[0] | (l[1] << 16), l[2] | (l[3] << 16));
  }
}

// y = part[0] + part[1] + ..., in this order.
__global__ void __launch_bounds__(256) w4_add_parts_kernel(const float4* part, int parts, int64_t total, float* y) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t n4 = total / 4;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n4; i += (int64_t)gridDim.x * 256) {
    float4 a = part[i];
    for (int q = 1; q < parts; ++q) {
      // total % 4 == 0 keeps every part 16-byte aligned (the launch sees to it).
      const float4 v = part[q * n4 + i];
      a.x += v.x;
      a.y += v.y;
      a.z += v.z;
      a.w += v.w;
    }
    reinterpret_cast<float4*>(y)[i] = a;
  }
}

template <typename Kernel, typename... Args>
cudaError_t launch_dependent(Kernel kern, int grid, int threads, size_t smem, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <int BN, int H, int PLANES, int GPB, bool kBf16S>
cudaError_t launch_t(const CUtensorMap& tx, const Params& p, int grid, cudaStream_t stream) {
  static std::atomic<uint64_t> allowed{0};
  auto kern = w4_gemm_kernel<BN, H, PLANES, GPB, kBf16S>;
  constexpr size_t smem = smem_bytes<BN, H, PLANES>();
  static_assert(smem <= kSmemMax, "shared memory");
  const cudaError_t e = allow_smem(kern, smem, allowed);
  if (e != cudaSuccess) return e;
  return launch_dependent(kern, grid, kThreads, smem, stream, tx, p);
}

template <int BN, int H, int PLANES>
cudaError_t launch_n(const CUtensorMap& tx, const Params& p, const W4Shape& sh, int grid, cudaStream_t stream) {
  const bool s16 = sh.scale_bytes == 2;
  switch (sh.group) {
    case 32: return s16 ? launch_t<BN, H, PLANES, 4, true>(tx, p, grid, stream)
                        : launch_t<BN, H, PLANES, 4, false>(tx, p, grid, stream);
    case 64: return s16 ? launch_t<BN, H, PLANES, 2, true>(tx, p, grid, stream)
                        : launch_t<BN, H, PLANES, 2, false>(tx, p, grid, stream);
    default: return s16 ? launch_t<BN, H, PLANES, 1, true>(tx, p, grid, stream)
                        : launch_t<BN, H, PLANES, 1, false>(tx, p, grid, stream);
  }
}

template <int PLANES>
cudaError_t launch_p(int BN, int H, const CUtensorMap& tx, const Params& p, const W4Shape& sh, int grid,
                     cudaStream_t stream) {
  if (BN == 32) return launch_n<32, 1, PLANES>(tx, p, sh, grid, stream);
  if (BN == 64) return launch_n<64, 1, PLANES>(tx, p, sh, grid, stream);
  return H == 2 ? launch_n<128, 2, PLANES>(tx, p, sh, grid, stream) : launch_n<128, 1, PLANES>(tx, p, sh, grid, stream);
}

// How a product is cut: tokens per tile, 128-row halves, parts of K.
struct Cut {
  int BN, H, parts;
};

// Estimated cycles of a launch: the longest CTA's units, each stage of them as
// long as its MMAs, its unpacking or its drains, whichever takes longest
// (cycles per stage measured on 4096, 1024 and 512 tokens), and for parts the
// second launch and its traffic.
int64_t estimate(const Cut& c, int planes, int gpb, int64_t M, int64_t N, int64_t blocks, int sms) {
  const int64_t tiles = (M + c.BN - 1) / c.BN * ((N + kBM * c.H - 1) / (kBM * c.H));
  const int64_t waves = (tiles * c.parts + sms - 1) / sms;
  const int64_t per_mma = c.BN == 128 ? (c.H == 2 ? 75 : 100) : (c.BN == 64 ? 55 : 50);
  const int64_t mma = (int64_t)planes * 8 * c.H * per_mma;
  const int64_t drain = (int64_t)gpb * (c.H == 2 ? 2 * 300 : (c.BN == 128 ? 400 : 300));
  const int64_t unpack = 300 * c.H;
  int64_t stage = mma > drain ? mma : drain;
  stage = stage > unpack ? stage : unpack;
  const int64_t add = c.parts > 1 ? 5000 + M * N * c.parts / sms / 8 : 0;
  return waves * ((blocks + c.parts - 1) / c.parts * stage + 2000 * c.H) + add;
}

Cut choose_cut(int planes, int gpb, int64_t M, int64_t N, int64_t blocks, int sms) {
  Cut best{32, 1, 1};
  int64_t cost = estimate(best, planes, gpb, M, N, blocks, sms);
  const int most = w4_parts(M, N);
  for (const Cut shape : {Cut{32, 1, 1}, Cut{64, 1, 1}, Cut{128, 1, 1}, Cut{128, 2, 1}}) {
    for (int parts = 1; parts <= most && parts <= blocks; ++parts) {
      const Cut c{shape.BN, shape.H, parts};
      const int64_t e = estimate(c, planes, gpb, M, N, blocks, sms);
      if (e < cost) {
        cost = e;
        best = c;
      }
    }
  }
  return best;
}

}  // namespace

cudaError_t launch_w4_gemm(const void* x, bool bf16, int64_t M, const W4Shape& sh, const uint8_t* packed, float* y,
                           void* ws, cudaStream_t stream, int num_sms) {
  PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
  if (encode == nullptr) return cudaErrorNotSupported;
  const int planes = bf16 ? 1 : 3;
  uint8_t* base = static_cast<uint8_t*>(ws);
  void* xb = const_cast<void*>(x);
  if (!bf16) {
    xb = base + kHeaderBytes;
    const int64_t n4 = M * sh.K / 4;
    const int64_t want = (n4 + 255) / 256, most = (int64_t)num_sms * 8;
    const cudaError_t e =
        launch_dependent(w4_split_kernel, (int)(want < most ? want : most), 256, 0, stream,
                         static_cast<const float4*>(x), n4, static_cast<uint2*>(xb));
    if (e != cudaSuccess) return e;
  }
  Params p;
  p.packed = packed;
  p.y = y;
  p.err = reinterpret_cast<uint32_t*>(base);
  p.M = (int)M;
  p.N = sh.N;
  p.row_tiles = sh.tiles();
  p.blocks = (int)sh.blocks();
  const Cut c = choose_cut(planes, kW4Cols / sh.group, M, sh.N, p.blocks, num_sms);
  const int BN = c.BN;
  const int64_t tiles_n = (sh.N + kBM * c.H - 1) / (kBM * c.H);
  p.tiles_n = (int)tiles_n;
  p.parts = c.parts;
  const int64_t nt = (M + BN - 1) / BN * tiles_n * c.parts;
  if (nt > 0x7FFFFFFF) return cudaErrorInvalidValue;
  p.units = (int)nt;
  float* parts = reinterpret_cast<float*>(base + kHeaderBytes + align256(6 * (size_t)M * (size_t)sh.K));
  if (c.parts > 1) p.y = parts;
  CUtensorMap tx;
  const cuuint64_t gdim[3] = {(cuuint64_t)sh.K, (cuuint64_t)M, (cuuint64_t)planes};
  const cuuint64_t gstride[2] = {(cuuint64_t)sh.K * 2, (cuuint64_t)sh.K * 2 * (cuuint64_t)M};
  const cuuint32_t box[3] = {64u, (cuuint32_t)BN, 1u};
  const cuuint32_t estride[3] = {1, 1, 1};
  if (encode(&tx, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, xb, gdim, gstride, box, estride, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  const int grid = (int)(nt < num_sms ? nt : num_sms);
  const cudaError_t e = planes == 1 ? launch_p<1>(BN, c.H, tx, p, sh, grid, stream)
                                    : launch_p<3>(BN, c.H, tx, p, sh, grid, stream);
  if (e != cudaSuccess || c.parts == 1) return e;
  const int64_t total = M * sh.N, want = (total / 4 + 255) / 256, most = (int64_t)num_sms * 8;
  return launch_dependent(w4_add_parts_kernel, (int)(want < most ? want : most), 256, 0, stream,
                          static_cast<const float4*>(static_cast<const void*>(parts)), c.parts, total, y);
}

}  // namespace bl
