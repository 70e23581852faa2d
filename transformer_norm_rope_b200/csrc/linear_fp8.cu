// linear_fp8.cu - matrix product of two 8-bit (e4m3) operands with block scales, on the tcgen05
// tensor cores:
//   y[m, n] = act( sum_b sa[m, b] sb[n', b] sum_{k in block b} A[m, k] B[n, k]  + d[n] ),
// b over the blocks of 128 of the contraction, n' = n / 128 (a weight's 128 x 128 blocks) or n.
//
// The scales change with b, so the tensor cores may only sum within a block: every block's product is
// a fresh accumulator in tensor memory, which warps read back and add, scaled, to the running total
// in their registers (fp32 throughout; a product of two e4m3 values is exact). Two accumulators
// alternate, so the tensor cores form block b + 1 while block b is added. For a 128 x 256 share per SM a
// block takes the tensor cores 128 * 256 * 128 / 8192 = 512 cycles, 0.26 us; the adding takes 8 warps 256 cycles
// of tensor-memory reads and 128 of packed FMAs on each scheduler, and its waits and hand-overs are not hidden by
// them: a block takes 0.51 us (0.84 with a scale per row of B), the tensor pipe is busy 45 % of the time
// (8192 x 5120 x 5120), and without the adding the kernel reached 2193 TFLOP/s where it reaches 1700.
//
// Two kernels, by shape (see fp8_run):
//   * linear_fp8_pair_kernel: pairs of SMs on 256 x 256 tiles (tcgen05.mma.cta_group::2, M = 256,
//     N = 256, K = 32), persistent over the tiles: the work that bounds it is the tensor cores'.
//   * linear_fp8_split_kernel: the operands' roles exchanged (B's rows on the 128 lanes, 16 to 128 rows
//     of A as columns) and the contraction split over the CTAs of a cluster, whose partial totals meet
//     in distributed shared memory in a fixed order: for few rows, where reading B bounds it and every SM
//     has to read, and for outputs of few tiles.
// Every mbarrier wait is bounded; a timeout records the error bit, and the CTA leaves its loops, waits
// for its own tensor-core work and copies, frees its tensor memory and exits.
#include "act_pairs.cuh"
#include "gn_common.cuh"
#include "gn_host.h"
#include "tcgen05.cuh"

namespace gn {
namespace {

constexpr int kBlk = 128;                // values that share a scale; also the tile depth
constexpr uint32_t kTileBytes = 128 * kBlk;  // 128 rows of one block: 16 KiB
constexpr int64_t kMaxRows = 65535ll * 128;

struct Fp8Args {
  const float* sa;
  const float* sb;
  const float* d;  // [N] or null
  void* y;         // split kernel (the pair kernel writes through its tensor map)
  int M, N, K, nkb;
  int64_t ldsa, ldsb, ldy;
  int accumulate;
  int b_shift;     // 7: sb has a row per 128 rows of B; 0: one per row
  unsigned* err;
};

// instruction descriptor of tcgen05.mma kind::f8f6f4: D fp32 (bits 4-5 = 1), A and B e4m3 (0), both
// K-major, N >> 3 at bit 17, M >> 4 at bit 24
constexpr uint32_t idesc_f8(int m, int n) { return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24); }

// K-major tile of 128-byte rows, 128-byte swizzle (the layout TMA writes): see norm_linear.cu. One
// instruction's 32 values of the contraction are 32 bytes, two descriptor units.
__device__ __forceinline__ uint64_t f8_desc(const void* tile) {
  return (uint64_t)((smem_addr(tile) & 0x3FFFFu) >> 4) | (1ull << 16) | ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) |
         (2ull << 61);
}

template <int CG, int M, int N>
__device__ __forceinline__ void umma_f8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t accumulate) {
  if constexpr (CG == 2)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc_f8(M, N)), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc_f8(M, N)), "r"(accumulate)
        : "memory");
}

// 16 consecutive columns of this warp's 32 lanes
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float2 (&v)[8]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = make_float2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
}

// the same for 32 columns, in two steps: the load is issued, and its registers may be used after the wait
__device__ __forceinline__ void tmem_ld32_issue(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
// (the registers pass through the wait so that no use of them can be scheduled before it)
__device__ __forceinline__ void tmem_ld_wait(uint32_t (&r)[32], uint32_t (&t)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                 "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                 "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
                 "+r"(r[29]), "+r"(r[30]), "+r"(r[31]), "+r"(t[0]), "+r"(t[1]), "+r"(t[2]), "+r"(t[3]), "+r"(t[4]),
                 "+r"(t[5]), "+r"(t[6]), "+r"(t[7]), "+r"(t[8]), "+r"(t[9]), "+r"(t[10]), "+r"(t[11]), "+r"(t[12]),
                 "+r"(t[13]), "+r"(t[14]), "+r"(t[15]), "+r"(t[16]), "+r"(t[17]), "+r"(t[18]), "+r"(t[19]),
                 "+r"(t[20]), "+r"(t[21]), "+r"(t[22]), "+r"(t[23]), "+r"(t[24]), "+r"(t[25]), "+r"(t[26]),
                 "+r"(t[27]), "+r"(t[28]), "+r"(t[29]), "+r"(t[30]), "+r"(t[31])
               :
               : "memory");
}

// 32 columns of 16 lanes as fragments: r[4 j + 2 h + e] = (lane of the address) + lane / 4 + 8 h, column
// 8 j + 2 (lane % 4) + e
__device__ __forceinline__ void tmem_ld16x32_issue(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld_wait(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}

// arrive on the barrier at this shared::cluster address (either CTA's). What it orders are tensor-memory
// reads, by the tcgen05 fences around it; a fence or an arrival that releases ordinary memory to the whole
// cluster cost more than a block's product (measured at 32768 x 5120 x 5120: 1.69 ms with, 1.07 without).
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar_cluster) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar_cluster) : "memory");
}

// ---------------------------------------------------------------- pairs of SMs
// Warp 0 loads (each CTA its 128 rows of A and its half of B's 256 rows per stage), warp 1 of the leader
// issues the instructions, warps 4-11 of each CTA own 128 rows x 256 columns of totals: warp w the rows
// 32 (w % 4).. (the tensor-memory lanes it may read) and the column half w / 4 - 1, one row and 128
// columns a thread. The 128 totals a thread do not fit the 168 registers of an even split: the first four
// warps give theirs up (3 x 168 = 40 + 2 x 232 a thread and scheduler).
constexpr int kPairThreads = 384;
constexpr uint32_t kPairStage = 2 * kTileBytes;
constexpr uint32_t kBoxBytes = 32 * 128;  // one output box of a warp: 32 rows x 128 bytes
// Scales travel in groups of four blocks: warp 3 of each CTA copies, asynchronously and up to kSlots groups
// ahead, the 128 rows' [row][4] of sa and the tile's [2][4] (or, BROW, [256][4]) of sb. Read row by row where
// they lie, a block at a time, they cost a quarter more L2 traffic (a 32-byte sector per row and block) and
// their latency (5120 x 5120 x 4096 with row scales: 270 us a block at a time, 189 in groups).
constexpr int kPairStages = 5, kSlots = 4;
template <bool BROW>
struct Pair {
  static constexpr int SbRows = BROW ? 256 : 2;
  static constexpr uint32_t Slot = (128 + SbRows) * 16;
  static constexpr size_t Smem = 1024 + (size_t)kPairStages * kPairStage + 8 * kBoxBytes + 256 + kSlots * Slot;
};

// one row's scales of blocks b .. b + 3 into 16 bytes of shared memory; blocks at and past nkb, and rows that
// are not `in`, are zero
__device__ __forceinline__ void copy_scales(float* dst, const float* row, int b, int nkb, bool in, bool vec) {
  const int n = !in ? 0 : nkb - b < 4 ? nkb - b : 4;
  if (vec) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)), "l"(row + b), "r"(4 * n) : "memory");
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_addr(dst + i)), "l"(row + (i < n ? b + i : b)),
                   "r"(i < n ? 4 : 0)
                   : "memory");
  }
}

template <int EPI, bool F32, bool BROW>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    linear_fp8_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                           const __grid_constant__ CUtensorMap tmY, const Fp8Args a) {
  constexpr int kStages = kPairStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* boxes = smem + kStages * kPairStage;
  uint64_t* full = reinterpret_cast<uint64_t*>(boxes + 8 * kBoxBytes);  // leader: both CTAs' tiles landed
  uint64_t* empty = full + kStages;   // the pair's instructions are done with the stage
  uint64_t* accf = empty + kStages;   // [2] accumulator formed
  uint64_t* acce = accf + 2;          // [2] leader: accumulator read by all 16 warps
  uint64_t* scf = acce + 2;           // [kSlots] a group of scales has landed
  uint64_t* sce = scf + kSlots;       // [kSlots] it has been read by this CTA's 8 warps
  uint32_t* tslot = reinterpret_cast<uint32_t*>(sce + kSlots);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tslot + 1);
  float* scales = reinterpret_cast<float*>(boxes + 8 * kBoxBytes + 256);
  constexpr int kSlotFloats = Pair<BROW>::Slot / 4;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const bool leader = rank == 0;
  const int nt = (a.N + 255) / 256, mt = (a.M + 255) / 256;
  const int64_t tiles = (int64_t)nt * mt;
  const int64_t step = gridDim.x >> 1;
  auto A = [&](int s) { return smem + s * kPairStage; };
  auto B = [&](int s) { return smem + s * kPairStage + kTileBytes; };

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&accf[i], 1);
      mbar_init(&acce[i], 16);
    }
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&scf[i], 32);
      mbar_init(&sce[i], 8);
    }
    *abort_flag = 0;
    mbar_fence_init();
  }
  if (warp == 1) tmem_alloc_pair(tslot, 512);
  tc_fence_before();
  cluster_sync_all();  // both CTAs' barriers exist before any load counts on them
  tc_fence_after();
  const uint32_t tmem = *tslot;
  if (warp < 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer (both CTAs)
    if (lane == 0) {
      uint32_t lastph = 0, used = 0, ph = 0;
      int s = 0;
      bool go = true, wrapped = false;
      for (int64_t t = blockIdx.x >> 1; go && t < tiles; t += step) {
        const int m0 = (int)(t / nt) * 256 + 128 * (int)rank, n0 = (int)(t % nt) * 256 + 128 * (int)rank;
        for (int kb = 0; kb < a.nkb; ++kb) {
          if ((wrapped && !mbar_wait(&empty[s], ph ^ 1u, a.err)) || *abort_flag) {
            *abort_flag = 1;
            go = false;
            break;
          }
          const uint32_t bar = cluster_addr(&full[s], 0);
          if (leader) mbar_expect_tx(&full[s], 2 * kPairStage);  // both CTAs' bytes
          tma_load_2d_pair(A(s), &tmA, kb * kBlk, m0, bar);
          tma_load_2d_pair(B(s), &tmB, kb * kBlk, n0, bar);
          used |= 1u << s;
          lastph = (lastph & ~(1u << s)) | (ph << s);
          if (++s == kStages) s = 0, ph ^= 1u, wrapped = true;
        }
      }
      // the leader's barriers count both CTAs' copies: every copy issued has landed once they
      // complete (bounded waits)
      if (leader)
        for (int i = 0; i < kStages; ++i)
          if (used & (1u << i)) (void)mbar_wait(&full[i], (lastph >> i) & 1u, a.err);
    }
  } else if (warp <= 2) {
    // ------------------------------------------------------------ MMA issuers (leader)
    // Two warps, each with one of the two accumulators and every other block: the waits of one pass
    // while the other's instructions run. (A wait on a barrier that is ready costs the issuer about
    // 180 cycles next to the operand traffic in shared memory; one issuer's two waits a block left
    // the tensor cores idle that long.)
    if (leader && lane == 0) {
      const int buf = warp - 1;
      const int64_t mine = blockIdx.x >> 1 < tiles ? (tiles - 1 - (blockIdx.x >> 1)) / step + 1 : 0;
      const int64_t blocks = mine * a.nkb;
      uint32_t full_ph = 0, acc_ph = 1;
      int s = buf;
      bool go = true;
      for (int64_t i = buf; i < blocks; i += 2) {
        if ((i >= 2 && !mbar_wait(&acce[buf], acc_ph, a.err)) || !mbar_wait(&full[s], full_ph, a.err)) {
          go = false;
          break;
        }
        tc_fence_after();
        const uint64_t ad = f8_desc(A(s)), bd = f8_desc(B(s));
#pragma unroll
        for (int k = 0; k < kBlk / 32; ++k) umma_f8<2, 256, 256>(tmem + 256u * buf, ad + 2 * k, bd + 2 * k, k != 0);
        umma_commit_pair(&accf[buf]);
        umma_commit_pair(&empty[s]);
        acc_ph ^= 1u;
        s += 2;
        if (s >= kStages) s -= kStages, full_ph ^= 1u;
      }
      if (!go) {  // both CTAs' other warps wait for the work in flight
        *abort_flag = 1;
        umma_commit_pair(&accf[buf]);
      }
    }
    __syncwarp();
  } else if (warp == 3) {
    // ------------------------------------------------------------ scales (both CTAs)
    const bool va = (a.ldsa & 3) == 0 && (reinterpret_cast<uintptr_t>(a.sa) & 15) == 0;
    const bool vb = (a.ldsb & 3) == 0 && (reinterpret_cast<uintptr_t>(a.sb) & 15) == 0;
    int slot = 0;
    uint32_t ph = 1;
    bool go = true, wrapped = false;
    for (int64_t t = blockIdx.x >> 1; go && t < tiles; t += step) {
      const int m0 = (int)(t / nt) * 256 + 128 * (int)rank, n0 = (int)(t % nt) * 256;
      for (int b = 0; b < a.nkb; b += 4) {
        if (wrapped && !__all_sync(0xffffffffu, mbar_wait(&sce[slot], ph, a.err))) {
          go = false;
          break;
        }
        float* dst = scales + slot * kSlotFloats;
#pragma unroll 1
        for (int i = 0; i < 4; ++i) {
          const int r = 32 * i + lane, m = m0 + r;
          copy_scales(dst + 4 * r, a.sa + (int64_t)(m < a.M ? m : 0) * a.ldsa, b, a.nkb, m < a.M, va);
        }
        if constexpr (BROW) {
#pragma unroll 1
          for (int i = 0; i < 8; ++i) {
            const int r = 32 * i + lane, n = n0 + r;
            copy_scales(dst + 512 + 4 * r, a.sb + (int64_t)(n < a.N ? n : 0) * a.ldsb, b, a.nkb, n < a.N, vb);
          }
        } else if (lane < 2) {
          const int n = n0 + 128 * lane;
          copy_scales(dst + 512 + 4 * lane, a.sb + (int64_t)(n < a.N ? n >> 7 : 0) * a.ldsb, b, a.nkb, n < a.N, vb);
        }
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(&scf[slot])) : "memory");
        if (++slot == kSlots) slot = 0, ph ^= 1u, wrapped = true;
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");  // this warp's copies have landed
  } else if (warp >= 4) {
    // ------------------------------------------------------------ totals and epilogue
    asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
    const int q = warp & 3;                // tensor-memory lane quadrant
    const int half = (warp >> 2) - 1;      // column half
    const uint32_t lanes = (uint32_t)(32 * q) << 16;
    const uint32_t empty_bar[2] = {cluster_addr(&acce[0], 0), cluster_addr(&acce[1], 0)};
    uint8_t* box = boxes + (size_t)(warp - 4) * kBoxBytes;
    uint32_t ph = 0, sph = 0;
    int buf = 0, slot = 0;
    bool ok = true, box_used = false;
    for (int64_t t = blockIdx.x >> 1; ok && t < tiles; t += step) {
      const int m0 = (int)(t / nt) * 256 + 128 * (int)rank, n0 = (int)(t % nt) * 256;
      const int nh = n0 + 128 * half;      // first column of this thread
      constexpr int kSa = BROW ? 4 : 1;    // rows of a thread
      const int row0 = 32 * q + (BROW ? lane >> 2 : lane);
      float2 acc[64];
#pragma unroll
      for (int i = 0; i < 64; ++i) acc[i] = make_float2(0.0f, 0.0f);
      for (int kb = 0; kb < a.nkb; ++kb) {
        const int k4 = kb & 3;
        if (k4 == 0) ok = __all_sync(0xffffffffu, mbar_wait(&scf[slot], sph, a.err));
        const float* sc = scales + slot * kSlotFloats + k4;
        float sav[kSa];
#pragma unroll
        for (int i = 0; i < kSa; ++i) sav[i] = sc[4 * (row0 + 8 * i)];
        sc += 512;
        ok = ok && __all_sync(0xffffffffu, mbar_wait(&accf[buf], ph, a.err));
        if (!ok) break;
        tc_fence_after();
        const uint32_t src = tmem + lanes + 256u * buf + 128u * half;
        uint32_t p[2][BROW ? 16 : 32];
        auto release = [&] {  // the accumulator is read: its next block may start
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(empty_bar[buf]);
        };
        if constexpr (BROW) {
          // fragments: a thread has four rows and 32 columns, so that it reads 32 of B's scales and not
          // 128 (one row and 128 columns a thread: 512 bytes to a warp and value, 1024 cycles a block for the
          // reads alone)
          const float* sr = sc + 4 * (128 * half + 2 * (lane & 3));
          auto at = [&](int c) { return src + ((uint32_t)(c & 1) << 20) + 32u * (c >> 1); };  // chunk c: 16 rows x 32 columns
          tmem_ld16x32_issue(at(0), p[0]);
#pragma unroll
          for (int c = 0; c < 8; ++c) {  // chunk c + 1 is on its way while chunk c is added
            const uint32_t(&v)[16] = p[c & 1];
            tmem_ld_wait(p[c & 1]);
            if (c < 7) tmem_ld16x32_issue(at(c + 1), p[(c + 1) & 1]);
            else release();
#pragma unroll
            for (int jj = 0; jj < 4; ++jj) {
              const int o = 4 * (32 * (c >> 1) + 8 * jj);
              const float2 s2 = make_float2(sr[o], sr[o + 4]);
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                float2* t = acc + 32 * (c & 1) + 8 * (c >> 1) + 2 * jj + h;
                *t = fma2(make_float2(__uint_as_float(v[4 * jj + 2 * h]), __uint_as_float(v[4 * jj + 2 * h + 1])),
                          mul2(s2, dup2(sav[2 * (c & 1) + h])), *t);
              }
            }
          }
        } else {
          const float2 f = dup2(sav[0] * sc[4 * half]);
          auto add = [&](const uint32_t (&v)[32], int c) {  // the totals of columns 32 c.. of the half
#pragma unroll
            for (int i = 0; i < 16; ++i)
              acc[16 * c + i] = fma2(make_float2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), f, acc[16 * c + i]);
          };
          tmem_ld32_issue(src, p[0]);
          tmem_ld32_issue(src + 32, p[1]);
          tmem_ld_wait(p[0], p[1]);
          add(p[0], 0);
          tmem_ld32_issue(src + 64, p[0]);
          add(p[1], 1);
          tmem_ld32_issue(src + 96, p[1]);
          tmem_ld_wait(p[0], p[1]);
          release();
          add(p[0], 2);
          add(p[1], 3);
        }
        if (++buf == 2) buf = 0, ph ^= 1u;
        if (k4 == 3 || kb == a.nkb - 1) {  // the group of scales has been read
          __syncwarp();
          if (lane == 0) mbar_arrive1(&sce[slot]);
          if (++slot == kSlots) slot = 0, sph ^= 1u;
        }
      }
      if (!ok) break;
      // Bias and activation. (By act_pair: 1 + tanh(u) from the hardware tanh, which is off by 2^-11, left GeLU
      // values near z = -3 off by a fifth. 32768 x 5120 x 5120: 995 us with the tanh, 1013 with these; a tile's
      // work outside its blocks 5.8 us and 6.3, without an activation 3.5.) Then the way out: boxes of 128 bytes x
      // 32 rows in shared memory (128-byte swizzle: 16-byte chunk c of row r at position c ^ (r % 8)), written by
      // TMA with the rows and columns past M and N clipped
      constexpr int kCols = F32 ? 32 : 64;  // columns of a box
#pragma unroll
      for (int b = 0; b < 128 / kCols; ++b) {
        const int col0 = nh + b * kCols;
        if (col0 < a.N) {  // uniform over the warp
          // (the values first, so that the wait for the box passes meanwhile)
          auto box_free = [&] {  // the box's previous store has finished reading it
            if (box_used) {
              if (lane == 0) bulk_wait_read<0>();
              __syncwarp();
            }
          };
          auto bias = [&](int n) { return a.d && n < a.N ? __ldg(a.d + n) : 0.0f; };
          auto bias4 = [&](int n) {
            if (a.d && n + 4 <= a.N) return __ldg(reinterpret_cast<const float4*>(a.d + n));
            return make_float4(bias(n), bias(n + 1), bias(n + 2), bias(n + 3));
          };
          if constexpr (BROW) {
            float2 o[kCols / 8][4];
#pragma unroll
            for (int jj = 0; jj < kCols / 8; ++jj) {
              const int c = col0 + 8 * jj + 2 * (lane & 3);
              const float2 d = make_float2(bias(c), bias(c + 1));
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int cb = b * kCols + 8 * jj;  // column of the half
                o[jj][i] = act_pair<EPI, true>(add2(acc[32 * (i >> 1) + 16 * (cb >> 6) + 2 * ((cb & 63) >> 3) + (i & 1)], d));
              }
            }
            box_free();
#pragma unroll
            for (int jj = 0; jj < kCols / 8; ++jj) {
              const int c = 8 * jj + 2 * (lane & 3);  // column of the box
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int r = (lane >> 2) + 8 * i;
                constexpr int kEs = F32 ? 4 : 2;
                uint8_t* at = box + r * 128 + ((((c * kEs) >> 4) ^ (r & 7)) << 4) + ((c * kEs) & 15);
                if constexpr (F32) *reinterpret_cast<float2*>(at) = o[jj][i];
                else *reinterpret_cast<uint32_t*>(at) = Vec<__nv_bfloat16>::join(o[jj][i].x, o[jj][i].y);
              }
            }
          } else {
            uint8_t* row = box + lane * 128;
            uint4 w[8];
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              constexpr int kE = kCols / 8;  // elements of a 16-byte chunk
              float o[kE];
#pragma unroll
              for (int e = 0; e < kE; e += 4) {
                const float4 d = bias4(col0 + c * kE + e);
                const float2 u = act_pair<EPI, true>(add2(acc[(b * kCols + c * kE + e) / 2], make_float2(d.x, d.y)));
                const float2 v = act_pair<EPI, true>(add2(acc[(b * kCols + c * kE + e) / 2 + 1], make_float2(d.z, d.w)));
                o[e] = u.x, o[e + 1] = u.y, o[e + 2] = v.x, o[e + 3] = v.y;
              }
              if constexpr (F32) w[c] = Vec<float>::pack(o);
              else w[c] = Vec<__nv_bfloat16>::pack(o);
            }
            box_free();
#pragma unroll
            for (int c = 0; c < 8; ++c) *reinterpret_cast<uint4*>(row + ((c ^ (lane & 7)) << 4)) = w[c];
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) {
            if (F32 && a.accumulate) tma_reduce_add_2d(&tmY, box, col0, m0 + 32 * q);
            else tma_store_2d(&tmY, box, col0, m0 + 32 * q);
          }
          box_used = true;
        }
      }
    }
    if (lane == 0) bulk_wait_read<0>();  // the boxes are read before the CTA may leave
    __syncwarp();
  }

  // teardown: neither CTA leaves while the pair's instructions may still touch its shared or tensor
  // memory; then both free the pair's tensor memory
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

// ---------------------------------------------------------------- few rows: roles exchanged, split contraction
// A cluster of CS CTAs shares one output tile of 128 columns n x MT rows m; its CTA r sums the blocks
// [r nkb / CS, (r + 1) nkb / CS) with B's 128 rows on the tensor-memory lanes (one n a thread) and MT
// columns m. The totals go to shared memory, [m][n] fp32; after a cluster barrier CTA r adds the CS
// copies of its share of the rows m in rank order and writes it.
constexpr int kSplitThreads = 192;
constexpr int kTotLd = 132;  // floats between the rows of the totals: conflict-free for both who write and who read them
template <int MT>
struct Split {
  static constexpr uint32_t Stage = kTileBytes + MT * kBlk;
  static constexpr int Stages = MT == 16 ? 6 : MT == 32 ? 5 : MT == 64 ? 4 : 6;
  static constexpr int PerSm = MT == 128 ? 1 : 2;  // CTAs: 128 totals a thread leave room for one
  static constexpr uint32_t TmemCols = 2 * MT;
  static constexpr size_t Smem = 1024 + (size_t)Stages * Stage + 256 + 2 * MT * 4;
  static_assert((size_t)Stages * Stage >= (size_t)MT * kTotLd * 4, "the totals reuse the stages");
};

__device__ __forceinline__ float4 ld_cluster(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}

// Rows i0 .. i1 of the output tile: a warp adds the cs copies of its rows in rank order, four columns a lane. U rows
// at a time, all their copies under way together (a read from another SM takes hundreds of cycles).
template <int CS, int U, int EPI, bool F32>
__device__ __forceinline__ void add_totals(const Fp8Args& a, const float* total, int cs, int n0, int m0, int i0, int i1,
                                           int warp, int lane) {
  const int n = n0 + 4 * lane;
  uint32_t peer[CS];
#pragma unroll
  for (int j = 0; j < CS; ++j) peer[j] = cluster_addr(total, j < cs ? (uint32_t)j : 0u) + 16u * (uint32_t)lane;
  float d[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) d[e] = a.d && n + e < a.N ? __ldg(a.d + n + e) : 0.0f;
  if (i1 > a.M - m0) i1 = a.M - m0;
  for (int i = i0 + warp; i < i1; i += 4 * U) {
    float4 v[U][CS];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < CS; ++j)
        if (j < cs && i + 4 * u < i1) v[u][j] = ld_cluster(peer[j] + (uint32_t)(i + 4 * u) * (4u * kTotLd));
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i + 4 * u >= i1) break;
      float z[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int j = 0; j < CS; ++j)
        if (j < cs) z[0] += v[u][j].x, z[1] += v[u][j].y, z[2] += v[u][j].z, z[3] += v[u][j].w;
#pragma unroll
      for (int e = 0; e < 4; e += 2) {
        const float2 o = act_pair<EPI, true>(make_float2(z[e] + d[e], z[e + 1] + d[e + 1]));
        z[e] = o.x, z[e + 1] = o.y;
      }
      const int64_t at = (int64_t)(m0 + i + 4 * u) * a.ldy + n;
      if constexpr (F32) {
        float* p = static_cast<float*>(a.y) + at;
        if (n + 4 <= a.N) {
          float4 o = make_float4(z[0], z[1], z[2], z[3]);
          if (a.accumulate) {
            const float4 c = *reinterpret_cast<const float4*>(p);
            o.x += c.x, o.y += c.y, o.z += c.z, o.w += c.w;
          }
          *reinterpret_cast<float4*>(p) = o;
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (n + e < a.N) p[e] = a.accumulate ? p[e] + z[e] : z[e];
        }
      } else {
        __nv_bfloat16* p = static_cast<__nv_bfloat16*>(a.y) + at;
        if (n + 4 <= a.N) {
          *reinterpret_cast<uint2*>(p) = make_uint2(Vec<__nv_bfloat16>::join(z[0], z[1]), Vec<__nv_bfloat16>::join(z[2], z[3]));
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (n + e < a.N) p[e] = __float2bfloat16_rn(z[e]);
        }
      }
    }
  }
}

template <int MT, int EPI, bool F32>
__global__ void __launch_bounds__(kSplitThreads, Split<MT>::PerSm)
    linear_fp8_split_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                            const Fp8Args a, int cs) {
  using SP = Split<MT>;
  constexpr int kStages = SP::Stages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kStages * SP::Stage);
  uint64_t* empty = full + kStages;
  uint64_t* accf = empty + kStages;  // [2]
  uint64_t* acce = accf + 2;         // [2]
  uint32_t* tslot = reinterpret_cast<uint32_t*>(acce + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tslot + 1);
  float* sa_col = reinterpret_cast<float*>(smem + kStages * SP::Stage + 256);  // [2][MT]
  float* total = reinterpret_cast<float*>(smem);                              // [MT][kTotLd]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_rank();
  const int n0 = (int)(blockIdx.x / cs) * 128, m0 = (int)blockIdx.y * MT;
  const int kb0 = (int)((int64_t)rank * a.nkb / cs), kb1 = (int)((int64_t)(rank + 1) * a.nkb / cs);
  auto W = [&](int s) { return smem + s * SP::Stage; };
  auto X = [&](int s) { return smem + s * SP::Stage + kTileBytes; };

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&accf[i], 1);
      mbar_init(&acce[i], 4);
    }
    *abort_flag = 0;
    mbar_fence_init();
  }
  if (warp == 1) tmem_alloc(tslot, SP::TmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  bool ok = true;
  constexpr bool FRAG = MT >= 32;
  float2 acc[MT / 2];

  if (warp == 0) {
    if (lane == 0) {
      uint32_t lastph = 0, used = 0, ph = 0;
      int s = 0;
      for (int kb = kb0; kb < kb1; ++kb) {
        if ((kb - kb0 >= kStages && !mbar_wait(&empty[s], ph ^ 1u, a.err)) || *abort_flag) {
          *abort_flag = 1;
          break;
        }
        mbar_expect_tx(&full[s], SP::Stage);
        tma_load_2d(W(s), &tmB, kb * kBlk, n0, &full[s]);
        tma_load_2d(X(s), &tmA, kb * kBlk, m0, &full[s]);
        used |= 1u << s;
        lastph = (lastph & ~(1u << s)) | (ph << s);
        if (++s == kStages) s = 0, ph ^= 1u;
      }
      for (int i = 0; i < kStages; ++i)
        if (used & (1u << i)) (void)mbar_wait(&full[i], (lastph >> i) & 1u, a.err);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      uint32_t ph = 0;
      int s = 0;
      for (int kb = kb0; kb < kb1; ++kb) {
        const int i = kb - kb0, buf = i & 1;
        if ((i >= 2 && !mbar_wait(&acce[buf], (uint32_t)((i >> 1) - 1) & 1u, a.err)) || !mbar_wait(&full[s], ph, a.err) ||
            *abort_flag) {
          *abort_flag = 1;
          umma_commit(&accf[0]);
          umma_commit(&accf[1]);
          break;
        }
        tc_fence_after();
        const uint64_t wd = f8_desc(W(s)), xd = f8_desc(X(s));
#pragma unroll
        for (int k = 0; k < kBlk / 32; ++k) umma_f8<1, 128, MT>(tmem + (uint32_t)(MT * buf), wd + 2 * k, xd + 2 * k, k != 0);
        umma_commit(&empty[s]);
        umma_commit(&accf[buf]);
        if (++s == kStages) s = 0, ph ^= 1u;
      }
    }
    __syncwarp();
  } else {
    const int q = warp & 3;
    const int ct = threadIdx.x - 64;   // 0..127
    const int n = n0 + 32 * q + lane;  // this thread's column of y
    // FRAG: four columns of y (lane / 4 + 8 i of the warp's 32) and MT / 4 rows a thread, so that it reads as
    // many of A's scales; with one column and MT rows a thread those reads alone, 512 bytes to a warp and
    // value, took the shared memory 512 cycles a block at MT = 128
    constexpr int kCols = FRAG ? 4 : 1;
    const int nq = n0 + 32 * q;
    const float* sb[kCols];
    float sb_next[kCols];
#pragma unroll
    for (int i = 0; i < kCols; ++i) {
      const int c = FRAG ? nq + (lane >> 2) + 8 * i : n;
      sb[i] = a.sb + (int64_t)((c < a.N ? c : a.N - 1) >> a.b_shift) * a.ldsb;
      sb_next[i] = kb0 < kb1 ? __ldg(sb[i] + kb0) : 0.0f;
    }
    const float* sa = a.sa + (int64_t)(m0 + ct < a.M ? m0 + ct : a.M - 1) * a.ldsa;
#pragma unroll
    for (int i = 0; i < MT / 2; ++i) acc[i] = make_float2(0.0f, 0.0f);
    float sa_next = kb0 < kb1 && ct < MT ? __ldg(sa + kb0) : 0.0f;
    for (int kb = kb0; kb < kb1; ++kb) {
      const int i = kb - kb0, buf = i & 1;
      float sbv[kCols];
#pragma unroll
      for (int c = 0; c < kCols; ++c) sbv[c] = sb_next[c];
      if (ct < MT) sa_col[buf * MT + ct] = sa_next;  // last read before the barrier of the block before
      asm volatile("bar.sync 1, 128;" ::: "memory");
      if (kb + 1 < kb1) {
#pragma unroll
        for (int c = 0; c < kCols; ++c) sb_next[c] = __ldg(sb[c] + kb + 1);
        if (ct < MT) sa_next = __ldg(sa + kb + 1);
      }
      ok = ok && __all_sync(0xffffffffu, mbar_wait(&accf[buf], (uint32_t)(i >> 1) & 1u, a.err));
      tc_fence_after();
      const uint32_t src = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(MT * buf);
      if (ok) {
        if constexpr (FRAG) {
          const float* sr = sa_col + buf * MT + 2 * (lane & 3);
          // chunk c: 16 lanes x 32 columns; up to four are read together, as a read's latency is several times
          // what the chunk's FMAs take
          constexpr int kChunks = MT / 16, kTogether = kChunks < 4 ? kChunks : 4;
          auto at = [&](int c) { return src + ((uint32_t)(c & 1) << 20) + 32u * (c >> 1); };
#pragma unroll
          for (int c0 = 0; c0 < kChunks; c0 += kTogether) {
            uint32_t p[kTogether][16];
#pragma unroll
            for (int k = 0; k < kTogether; ++k) tmem_ld16x32_issue(at(c0 + k), p[k]);
#pragma unroll
            for (int k = 0; k < kTogether; ++k) tmem_ld_wait(p[k]);
#pragma unroll
            for (int k = 0; k < kTogether; ++k) {
              const int c = c0 + k;
#pragma unroll
              for (int jj = 0; jj < 4; ++jj) {
                const float2 s2 = *reinterpret_cast<const float2*>(sr + 32 * (c >> 1) + 8 * jj);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  float2* t = acc + MT / 4 * (c & 1) + 8 * (c >> 1) + 2 * jj + h;
                  const uint32_t* v = p[k] + 4 * jj + 2 * h;
                  *t = fma2(make_float2(__uint_as_float(v[0]), __uint_as_float(v[1])), mul2(s2, dup2(sbv[2 * (c & 1) + h])), *t);
                }
              }
            }
          }
        } else {
          float2 p[8];
          tmem_ld16(src, p);
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            const float4 s4 = *reinterpret_cast<const float4*>(sa_col + buf * MT + 2 * e);
            acc[e] = fma2(p[e], mul2(make_float2(s4.x, s4.y), dup2(sbv[0])), acc[e]);
            acc[e + 1] = fma2(p[e + 1], mul2(make_float2(s4.z, s4.w), dup2(sbv[0])), acc[e + 1]);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive1(&acce[buf]);
    }
  }
  // the stages are free once the last accumulator is formed (its blocks' tiles have been read); every
  // warp meets here, then the totals take their place
  __syncthreads();
  if (warp >= 2) {
    const int nl = 32 * (warp & 3);
    if constexpr (FRAG) {
#pragma unroll
      for (int jj = 0; jj < MT / 8; ++jj) {
        const int m = 8 * jj + 2 * (lane & 3);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 v = acc[MT / 4 * (i >> 1) + 2 * jj + (i & 1)];
          float* t = total + m * kTotLd + nl + (lane >> 2) + 8 * i;
          t[0] = v.x;
          t[kTotLd] = v.y;
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < MT / 2; ++i) {
        total[2 * i * kTotLd + nl + lane] = acc[i].x;
        total[(2 * i + 1) * kTotLd + nl + lane] = acc[i].y;
      }
    }
  }
  if (cs > 1) cluster_sync_all();
  else __syncthreads();
  if (!*abort_flag && warp >= 2) {
    const int i0 = MT * rank / cs, i1 = MT * (rank + 1) / cs;
    if (cs <= 2) add_totals<2, 8, EPI, F32>(a, total, cs, n0, m0, i0, i1, warp - 2, lane);
    else add_totals<8, 2, EPI, F32>(a, total, cs, n0, m0, i0, i1, warp - 2, lane);
  }
  // no CTA leaves while another may read its totals
  if (cs > 1) cluster_sync_all();
  else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, SP::TmemCols);
  }
}

// ---------------------------------------------------------------- host side

// codes [rows, K] with row stride ld, boxes of box_rows x 128 values, 128-byte swizzle; outside: zeros
bool make_code_map(CUtensorMap* map, const void* base, int64_t rows, int64_t K, int64_t ld, uint32_t box_rows) {
  EncodeTiled enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)ld};
  const cuuint32_t box[2] = {kBlk, box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// y [rows, cols]: boxes of 32 rows x 128 bytes
bool make_y_map(CUtensorMap* map, void* base, int64_t rows, int64_t cols, int64_t ld, bool f32) {
  EncodeTiled enc = encode_fn();
  if (!enc) return false;
  const size_t es = f32 ? 4 : 2;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)(ld * es)};
  const cuuint32_t box[2] = {(cuuint32_t)(128 / es), 32u};
  const cuuint32_t estr[2] = {1, 1};
  return enc(map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, dims, strides,
             box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool BROW>
void* pick_pair(int epi, bool f32) {
  return f32                       ? (void*)linear_fp8_pair_kernel<EPI_NONE, true, BROW>
         : epi == GN_EPI_GELU_TANH ? (void*)linear_fp8_pair_kernel<EPI_GELU_TANH, false, BROW>
         : epi == GN_EPI_SILU      ? (void*)linear_fp8_pair_kernel<EPI_SILU, false, BROW>
                                   : (void*)linear_fp8_pair_kernel<EPI_NONE, false, BROW>;
}

template <int MT>
void* pick_split(int epi, bool f32) {
  return f32                       ? (void*)linear_fp8_split_kernel<MT, EPI_NONE, true>
         : epi == GN_EPI_GELU_TANH ? (void*)linear_fp8_split_kernel<MT, EPI_GELU_TANH, false>
         : epi == GN_EPI_SILU      ? (void*)linear_fp8_split_kernel<MT, EPI_SILU, false>
                                   : (void*)linear_fp8_split_kernel<MT, EPI_NONE, false>;
}

gn_status fp8_run(const void* A, int64_t lda, const void* B, int64_t ldb, Fp8Args a, int epi, bool f32,
                  cudaStream_t stream) {
  const int sms = sm_count();
  if (sms <= 0) return GN_ERR_CUDA;
  const int64_t pairs = (int64_t)((a.M + 255) / 256) * ((a.N + 255) / 256);
  CUtensorMap ta, tb, ty;
  // The split kernel's cluster: as many CTAs as fit at once, with room for the clusters not to divide a GPC's
  // SMs evenly. Measured at 5120 columns and one row: 12.4 us with clusters of 2 (80 CTAs), 8.1 with 6 (240),
  // 11.9 with 8 (320: a second wave).
  auto split = [&](int MT, int64_t* tiles) {
    *tiles = (int64_t)((a.N + 127) / 128) * ((a.M + MT - 1) / MT);
    const int64_t slots = (int64_t)((MT == 128 ? 0.9f : 1.7f) * (float)sms), cs = slots / *tiles;
    return (int)(cs < 1 ? 1 : cs > 8 ? (a.nkb < 8 ? a.nkb : 8) : cs < a.nkb ? cs : a.nkb);
  };
  bool pair = a.M > 128 && a.N > 128;
  if (pair) {
    // a block of the contraction takes a pair 0.62 us and a split CTA of 128 rows 0.78: the shorter of the
    // two by waves x blocks (5120 x 5120 weight: 128 rows 15.8 us split, 26 as a pair tile half empty; 200
    // rows 32 split, 26 in pairs; 333 x 1288 x 5120: 13.1 split by four, 25.4 in pairs)
    int64_t tiles;
    const int cs = split(128, &tiles);
    const int64_t slots = (int64_t)(0.9f * (float)sms);
    const int64_t pair_cost = 4 * ((pairs + sms / 2 - 1) / (sms / 2)) * a.nkb;
    const int64_t split_cost = 5 * ((tiles * cs + slots - 1) / slots) * ((a.nkb + cs - 1) / cs);
    pair = pair_cost <= split_cost;
  }
  if (pair) {
    if (!make_code_map(&ta, A, a.M, a.K, lda, 128) || !make_code_map(&tb, B, a.N, a.K, ldb, 128) ||
        !make_y_map(&ty, a.y, a.M, a.N, a.ldy, f32))
      return GN_ERR_CUDA;
    const bool brow = a.b_shift == 0;
    void* kern = brow ? pick_pair<true>(epi, f32) : pick_pair<false>(epi, f32);
    const size_t smem = brow ? Pair<true>::Smem : Pair<false>::Smem;
    if (!kernel_attrs(kern, smem)) return GN_ERR_CUDA;
    const int64_t clusters = pairs < sms / 2 ? pairs : sms / 2;
    void* args[] = {&ta, &tb, &ty, &a};
    if (cudaLaunchKernel(kern, dim3((unsigned)(2 * clusters)), dim3(kPairThreads), args, smem, stream) != cudaSuccess)
      return GN_ERR_CUDA;
    count_launches(1);
    return launch_status();
  }
  const int MT = a.M <= 16 ? 16 : a.M <= 32 ? 32 : a.M <= 64 ? 64 : 128;
  int64_t tiles;
  int cs = split(MT, &tiles);
  if (!make_code_map(&ta, A, a.M, a.K, lda, (uint32_t)MT) || !make_code_map(&tb, B, a.N, a.K, ldb, 128)) return GN_ERR_CUDA;
  void* kern = MT == 16   ? pick_split<16>(epi, f32)
               : MT == 32 ? pick_split<32>(epi, f32)
               : MT == 64 ? pick_split<64>(epi, f32)
                          : pick_split<128>(epi, f32);
  const size_t smem = MT == 16 ? Split<16>::Smem : MT == 32 ? Split<32>::Smem : MT == 64 ? Split<64>::Smem : Split<128>::Smem;
  if (!kernel_attrs(kern, smem)) return GN_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(cs * ((a.N + 127) / 128)), (unsigned)((a.M + MT - 1) / MT));
  cfg.blockDim = dim3(kSplitThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)cs;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  void* args[] = {&ta, &tb, &a, &cs};
  if (cudaLaunchKernelExC(&cfg, kern, args) != cudaSuccess) return GN_ERR_CUDA;
  count_launches(1);
  return launch_status();
}

}  // namespace
}  // namespace gn

using namespace gn;

extern "C" gn_status gn_linear_fp8(const void* A, const float* sa, const void* B, const float* sb, const float* d,
                                   void* y, int64_t M, int64_t N, int64_t K, int64_t ld_a, int64_t ld_sa, int64_t ld_b,
                                   int64_t ld_sb, int64_t ld_y, int64_t b_rows, int accumulate, gn_epilogue epi,
                                   gn_dtype out, void* stream) {
  if (!dt_ok(out) || !epi_ok(epi)) return GN_ERR_DTYPE;
  if (M < 0 || N < 0 || K <= 0 || M > kMaxRows || N > kMaxRows || K > INT32_MAX - kBlk || (b_rows != 1 && b_rows != kBlk))
    return GN_ERR_SHAPE;
  const int64_t kb = (K + kBlk - 1) / kBlk;
  if (ld_a < K || ld_b < K || ld_sa < kb || ld_sb < kb || ld_y < N) return GN_ERR_SHAPE;
  if (out == GN_F32 ? epi != GN_EPI_NONE : accumulate != 0) return GN_ERR_UNSUPPORTED;
  if (M == 0 || N == 0) return GN_OK;
  if (!A || !sa || !B || !sb || !y) return GN_ERR_NULL;
  if (!aligned16(A) || !aligned16(B) || !aligned16(y) || ld_a % 16 || ld_b % 16 || ld_y * dt_size(out) % 16 ||
      (d && !aligned16(d)) || (reinterpret_cast<uintptr_t>(sa) & 3) || (reinterpret_cast<uintptr_t>(sb) & 3))
    return GN_ERR_ALIGN;
  Fp8Args a{};
  a.sa = sa, a.sb = sb, a.d = d, a.y = y;
  a.M = (int)M, a.N = (int)N, a.K = (int)K, a.nkb = (int)kb;
  a.ldsa = ld_sa, a.ldsb = ld_sb, a.ldy = ld_y;
  a.accumulate = accumulate != 0;
  a.b_shift = b_rows == kBlk ? 7 : 0;
  a.err = device_err_word();
  if (!a.err) return GN_ERR_CUDA;
  return fp8_run(A, ld_a, B, ld_b, a, epi, out == GN_F32, (cudaStream_t)stream);
}
