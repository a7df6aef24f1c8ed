// grouped_mx4.cu -- the experts' matrix product in microscaled 4-bit floating point (the format: mx4_cast.cu).
//
//   out[r, n] = bf16( sum_k x[r, k] w[e, n, k] )  for the rows r of expert e (offsets[e] .. offsets[e] + counts[e] - 1)
// or, with the gate,
//   out[r, n] = bf16( silu(a) b ), a = sum_k x[r, k] w[e, n, k], b = sum_k x[r, k] w[e, N/2 + n, k], n < N/2,
// silu(a) = a / (1 + exp(-a)), sums and gate in fp32, one rounding.
//
// A tile is features of one expert (operand A = weights, the 128 TMEM lanes of a CTA) by up to kTileT of its rows
// (operand B, the accumulator's columns).  Features, not rows, take the fixed side: an expert has any number of rows,
// one at decode, and the column side of tcgen05.mma goes in steps of 16 or 32.  With the gate a warp's 32 lanes are 16
// gate and the 16 matching up features, so that one thread holds both.  The rows of an expert are split evenly over as
// few tiles as hold them.
//
// Two forms (Shape): for few rows an expert, one CTA a tile, 128 features by up to 64 rows, a deep ring of
// stages; for many, a pair of CTAs a tile (cta_group::2), 256 features by up to 224 rows, each CTA loading its own
// 128 features and half of the rows, which halves what comes through L2 per product.
//
// The CTAs (one per SM) walk the tiles.  Warp 0: TMA loads into a ring of 256-element stages.  Warps 2 and 3: the
// scale words of the stage's two 128-element chunks, by four-byte copies into the order that tcgen05.cp wants.
// Warp 1: copies the scales to TMEM and issues the products (kind::mxf4, block-scaled, 64 elements each; in a pair the
// second CTA's warp 1 only tells the first that its stage is there).  Warps 4..11: the accumulator of the previous tile
// out of TMEM, each warp its 32 lanes by every other 32 columns, transposed by stmatrix into rows of out.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"

namespace {

constexpr int kThreads = 384;
constexpr int kEpiWarps = 8;
constexpr int kTileF = 128;             // features a CTA and tile
constexpr int kStageK = 256;            // elements of K a stage: 128 bytes, one swizzle atom
constexpr int kBoxRows = 16;            // rows of the smallest TMA box of x; gate features before the up ones
constexpr int kBytesA = kTileF * kStageK / 2;
constexpr int kAtom = 512;              // scales of 128 rows by 128 elements
constexpr int kEpiT = 32;               // columns an epilogue warp takes at a time
constexpr int kMaxExperts = 1024;
constexpr uint32_t kTmemCols = 512;

template <int CG, bool kGate>  // CTAs a tile; whether silu(gate) * up follows
struct Shape {
  static constexpr int kTileT = CG == 1 ? 64 : 224;  // rows a tile, at most
  static constexpr int kStepT = CG == 1 ? 16 : 32;   // columns of a product: a multiple of this
  static constexpr int kStages = CG == 1 ? 7 : kGate ? 6 : 5;  // (as shared memory allows)
  static constexpr int kEpiBytes = kEpiT * (kGate ? 32 : 64);  // an epilogue warp's transposed block
  static constexpr int kRowsB = kTileT / CG;         // rows of x a CTA loads
  static constexpr int kBytesB = kRowsB * kStageK / 2;
  static constexpr int kStageBytes = kBytesA + kBytesB;
  static constexpr int kAtomsB = (kTileT + 127) / 128;
  static constexpr int kBytesSf = 2 * kAtom * (1 + kAtomsB);
  // TMEM columns: two accumulators, then two sets of a stage's scales (four columns an atom)
  static constexpr uint32_t kSfCols = 8 + 8 * kAtomsB;
  static constexpr uint32_t kTmemSf = 2 * kTileT;
  static_assert(kTmemSf + 2 * kSfCols <= kTmemCols, "TMEM columns");
  static_assert(kStageBytes % 1024 == 0 && kRowsB % kBoxRows == 0 && kRowsB < 128, "swizzle atoms, boxes");

  struct __align__(1024) Smem {
    uint8_t ab[kStages][kStageBytes];  // A then B, 128-byte swizzled
    uint8_t sf[kStages][kBytesSf];     // A's two atoms, then B's, chunk by chunk
    uint8_t epi[kEpiWarps][2][kEpiBytes];
    int32_t first_tile[kMaxExperts + 1];  // row tiles before expert e
    int32_t warp_sums[kThreads / 32];
    float warp_rows[kThreads / 32];
    int tiles;
    uint64_t full[kStages], empty[kStages], acc_full[2], acc_empty[2], drained;
    uint32_t tmem;
    int abort;
  };
  static_assert(sizeof(Smem) + 1024 <= 232448, "shared memory");
};

struct ProductArgs {
  const uint32_t* x_sf;  // [chunks, capacity] scale words
  const uint32_t* w_sf;  // [chunks, E*N]
  const int32_t* counts;
  const int32_t* offsets;
  int E, N, K;
  int kstages;    // ceil(K / 256)
  int ftiles;     // feature tiles (of a CTA, or of a pair)
  int gate_box;   // 1: map_w has the gate's boxes (N a multiple of 32), 0: boxes of 16 rows
  int64_t capacity;
  __nv_bfloat16* out;
  int64_t ld_out;  // N or N / 2
  int32_t* status;
};

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// x, 0, 0, group, expert: with the gate, four groups of 16 gate and the 16 matching up features
__device__ __forceinline__ void tma_load_gate(void* dst, const CUtensorMap* map, int x, int group, int e, uint64_t* bar) {
  asm volatile("cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %3, %4, %5}], [%6];" ::"r"(
                   moe::smem_addr(dst)),
               "l"(map), "r"(x), "r"(0), "r"(group), "r"(e), "r"(moe::smem_addr(bar))
               : "memory");
}

__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
  asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
                   moe::smem_addr(dst)),
               "l"(map), "r"(x), "r"(y), "r"(moe::smem_addr(bar))
               : "memory");
}

// Shared-memory operand descriptors: start, stride between 8-row groups, fixed field 1 at bit 46, swizzle at bit 61.
__device__ __forceinline__ uint64_t desc_sw128(uint32_t addr) {
  return static_cast<uint64_t>((addr & 0x3ffffu) >> 4) | (uint64_t{1} << 16) | (uint64_t{1024 >> 4} << 32) |
         (uint64_t{1} << 46) | (uint64_t{2} << 61);
}
__device__ __forceinline__ uint64_t desc_plain(uint32_t addr) {
  return static_cast<uint64_t>((addr & 0x3ffffu) >> 4) | (uint64_t{1} << 16) | (uint64_t{128 >> 4} << 32) |
         (uint64_t{1} << 46);
}

__device__ __forceinline__ void copy_word(uint8_t* dst, const uint32_t* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(moe::smem_addr(dst)), "l"(src) : "memory");
}

// 512 bytes of scales to four TMEM columns; in a pair, each CTA's own shared memory to its own TMEM.
template <int CG>
__device__ __forceinline__ void sf_to_tmem(uint32_t taddr, uint64_t smem_desc) {
  if constexpr (CG == 1)
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(smem_desc) : "memory");
  else
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(smem_desc) : "memory");
}

template <int CG>
__device__ __forceinline__ void mma_mx4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                        bool accumulate) {
  if constexpr (CG == 1)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate ? 1u : 0u)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate ? 1u : 0u)
        : "memory");
}

// Arrive at the barrier (in a pair: at both CTAs') once the tensor operations issued so far are done.
template <int CG>
__device__ __forceinline__ void commit(uint64_t* bar) {
  if constexpr (CG == 1)
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                     moe::smem_addr(bar))
                 : "memory");
  else
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            moe::smem_addr(bar)),
        "h"(static_cast<uint16_t>(3))
        : "memory");
}

// Arrive at this CTA's own barrier once the tensor operations issued so far are done, in a pair those of both CTAs.
template <int CG>
__device__ __forceinline__ void commit_own(uint64_t* bar) {
  if constexpr (CG == 1)
    commit<1>(bar);
  else
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                     moe::smem_addr(bar))
                 : "memory");
}

// Arrive at CTA 0's barrier of the pair.  What it announces is in shared memory or TMEM, which have one copy, and was
// complete before (the stage's own barrier, tcgen05.wait), so the release need not reach beyond the CTA: with
// .release.cluster an arrival also waits for the CTA's global stores, about 1300 cycles, and bounded the whole kernel.
__device__ __forceinline__ void arrive_first(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .b32 r;\n\tmapa.shared::cluster.u32 r, %0, 0;\n\t"
      "mbarrier.arrive.shared::cluster.b64 _, [r];\n\t}" ::"r"(moe::smem_addr(bar))
      : "memory");
}

// Non-blocking test of a phase.
__device__ __forceinline__ bool phase_done(uint64_t* bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(moe::smem_addr(bar)), "r"(parity)
      : "memory");
  return done != 0u;
}
__device__ __forceinline__ bool phases_done(uint64_t* bar, uint32_t parity, uint64_t* bar2, uint32_t parity2) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 q, [%3], %4;\n\t"
      "and.pred p, p, q;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(moe::smem_addr(bar)), "r"(parity), "r"(moe::smem_addr(bar2)), "r"(parity2)
      : "memory");
  return done != 0u;
}
__device__ __forceinline__ void tmem_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 16 lanes by 32 columns: thread t gets, for columns 8i + 2 (t % 4) + {0, 1}, v[4i + {0, 1}] of lane t / 4 and
// v[4i + {2, 3}] of lane t / 4 + 8.
__device__ __forceinline__ void tmem_ld16x32(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// Four 8x8 blocks of bf16, transposed: lane 8m + j gives the address of row j of block m.
__device__ __forceinline__ void stmatrix_trans(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b),
               "r"(c), "r"(d)
               : "memory");
}

// silu(g) u, with the exponential taken of -|g|: the divisor stays between 1 and 2 (__fdividef gives 0 beyond 2^126).
__device__ __forceinline__ float silu_times(uint32_t gate, uint32_t up) {
  const float g = __uint_as_float(gate), t = __expf(-fabsf(g));
  return __fdividef(g >= 0.f ? g : g * t, 1.f + t) * __uint_as_float(up);
}

// A bounded wait of a warp; it also gives up when another role of the CTA has.  The first test is inline and its vote
// uniform, so that the loops around it stay convergent: the issuing warps must not run as a lone lane, whose operands
// go one by one through vector registers (1675 cycles to issue a stage that takes 450 to compute).
__device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, volatile int* abort, int32_t* status) {
  uint64_t t0 = 0;
  for (;;) {
#pragma unroll 1
    for (int i = 0; i < 256; ++i)
      if (phase_done(bar, parity)) return true;
    if (*abort != 0) return false;
    const uint64_t t = moe::global_ns();
    if (t0 == 0) t0 = t;
    if (t - t0 > moe::kWaitLimitNs) {
      moe::record_status(status, MOE_ERR_TIMEOUT);
      *abort = 1;
      return false;
    }
  }
}
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort, int32_t* status) {
  if (__all_sync(0xffffffffu, phase_done(bar, parity))) return true;
  return __all_sync(0xffffffffu, wait_slow(bar, parity, abort, status));
}

// One lane of a converged warp, always the same.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0u;
}

// Tile t: its first row, and 10 bits of expert, 8 of rows, 13 of feature tile.  (By value, not a method: a struct whose
// address is taken lives in local memory.)
template <int kTileStep>
__device__ __noinline__ int2 tile_of(int t, const int32_t* first, const int32_t* counts, const int32_t* offsets, int E,
                                     int ftiles) {
  const int rt = t / ftiles, ft = t - rt * ftiles;
  int lo = 0, hi = E - 1;  // the last expert with first[] <= rt: one that has rows
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (first[mid] <= rt) lo = mid;
    else hi = mid - 1;
  }
  const int cnt = counts[lo], n = first[lo + 1] - first[lo], i = rt - first[lo];
  const int per = ((cnt + n - 1) / n + kTileStep - 1) / kTileStep * kTileStep;  // at most kTileT
  return make_int2(offsets[lo] + i * per, (lo << 21) | ((cnt - i * per < per ? cnt - i * per : per) << 13) | ft);
}

// The tiles of this CTA (or pair), in order: expert by expert, then row tiles, features fastest.  The lanes of a warp
// work out 32 tiles at a time (a search, a division and two loads each, over 1000 cycles), which next() passes round.
template <int CG, bool kGate>
struct Tiles {
  static constexpr int kStep = Shape<CG, kGate>::kStepT;
  const ProductArgs& a;
  const int32_t* first;  // row tiles before expert e
  int e, f, row0, rows;  // expert, this CTA's feature tile, the tile's first row, its rows
  int at, total;         // the next tile, and all
  int turn = 32;         // lane that holds the next tile
  int2 mine;             // this lane's tile

  __device__ __forceinline__ Tiles(const ProductArgs& args, const int32_t* first_tile, int tiles)
      : a(args), first(first_tile), at(blockIdx.x / CG), total(tiles) {}
  __device__ __forceinline__ bool next() {
    if (at >= total) return false;
    if (turn == 32) {
      const int t = at + static_cast<int>(threadIdx.x & 31) * static_cast<int>(gridDim.x / CG);
      mine = make_int2(0, 0);
      if (t < total) mine = tile_of<kStep>(t, first, a.counts, a.offsets, a.E, a.ftiles);
      __syncwarp();
      turn = 0;
    }
    row0 = __shfl_sync(0xffffffffu, mine.x, turn);
    const int v = __shfl_sync(0xffffffffu, mine.y, turn);
    e = v >> 21;
    rows = (v >> 13) & 255;
    f = (v & 8191) * CG + (CG == 1 ? 0 : blockIdx.x % CG);
    ++turn;
    at += gridDim.x / CG;
    return true;
  }
  // the product's columns
  __device__ __forceinline__ int cols() const { return (rows + kStep - 1) / kStep * kStep; }
  // the first weight row of the tile (with the gate: of its gate features)
  __device__ __forceinline__ int64_t weight_row0() const {
    return static_cast<int64_t>(e) * a.N + static_cast<int64_t>(f) * (kGate ? kTileF / 2 : kTileF);
  }
  // row of the weights that lane m of the tile holds (clamped: lanes past the expert's features are not stored)
  __device__ __forceinline__ int64_t weight_row(int m) const {
    const int64_t r = weight_row0() + (!kGate ? m : (m & 16 ? a.N / 2 : 0) + (m >> 5) * 16 + (m & 15));
    const int64_t last = static_cast<int64_t>(a.E) * a.N - 1;
    return r < last ? r : last;
  }
};

template <int CG, bool kGate>
__global__ void __launch_bounds__(kThreads, 1)
grouped_mx4_kernel(const __grid_constant__ CUtensorMap map_x16, const __grid_constant__ CUtensorMap map_x32,
                   const __grid_constant__ CUtensorMap map_x64, const __grid_constant__ CUtensorMap map_x,
                   const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_out,
                   const ProductArgs a) {
  using S = Shape<CG, kGate>;
  constexpr int kStages = S::kStages;
  extern __shared__ uint8_t smem_raw[];
  typename S::Smem& s =
      *reinterpret_cast<typename S::Smem*>(smem_raw + ((1024u - (moe::smem_addr(smem_raw) & 1023u)) & 1023u));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = CG == 1 ? 0 : blockIdx.x % CG;  // in the pair
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      // the TMA warp and the lanes of the two scale warps; in a pair, at the first CTA, the second's stage too
      moe::mbar_init(&s.full[i], CG == 2 && rank == 0 ? 66 : 65);
      moe::mbar_init(&s.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      moe::mbar_init(&s.acc_full[i], 1);
      moe::mbar_init(&s.acc_empty[i], CG * kEpiWarps);
    }
    moe::mbar_init(&s.drained, 1);
    s.abort = 0;
    moe::fence_barrier_init();
  }
  if (warp == 1) {
    if constexpr (CG == 1) {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(moe::smem_addr(&s.tmem)),
                   "r"(kTmemCols)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    } else {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(moe::smem_addr(&s.tmem)),
                   "r"(kTmemCols)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
  }
  if (warp == 0 && elect_one()) {
    prefetch_map(&map_w);
    prefetch_map(&map_x16);
    prefetch_map(&map_x32);
    prefetch_map(&map_x64);
    prefetch_map(&map_x);
    prefetch_map(&map_out);
  }
  moe::pdl_launch_dependents();
  moe::pdl_wait();  // rows, scales, counts and offsets may come from the previous kernel

  // row tiles before each expert: a scan, a thread per expert
  float all_rows = 0.f;
  int before = 0;
  for (int e0 = 0; e0 < a.E; e0 += kThreads) {
    const int ex = e0 + tid;
    int n = 0;
    float rows = 0.f;
    if (ex < a.E) {
      const int64_t cnt = a.counts[ex], off = a.offsets[ex];
      if (cnt < 0 || off < 0 || off + cnt > a.capacity) {
        moe::record_status(a.status, MOE_ERR_BAD_ROW);  // skipped
      } else {
        n = static_cast<int>((cnt + S::kTileT - 1) / S::kTileT);
        rows = static_cast<float>(cnt);
      }
    }
    int incl = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += o;
      rows += __shfl_xor_sync(0xffffffffu, rows, d);
    }
    if (lane == 31) {
      s.warp_sums[warp] = incl;
      s.warp_rows[warp] = rows;
    }
    __syncthreads();
    int all = 0, mine = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w == warp) mine = all;
      all += s.warp_sums[w];
      all_rows += s.warp_rows[w];
    }
    if (ex < a.E) s.first_tile[ex + 1] = before + mine + incl;
    before += all;
    if (e0 + kThreads < a.E) __syncthreads();  // before the sums are written again
  }
  if (tid == 0) {
    s.first_tile[0] = 0;
    s.tiles = before * a.ftiles;
    // ranges that overlap so much that the tiles might not fit an int: nothing is done (the sum's rounding is far less)
    if (all_rows > 1.001f * static_cast<float>(a.capacity) + 1.f) {
      moe::record_status(a.status, MOE_ERR_BAD_ROW);
      s.tiles = 0;
    }
  }
  tmem_fence_before();
  __syncthreads();
  if constexpr (CG == 2) {  // the other CTA's barriers are initialised
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  }
  tmem_fence_after();
  const uint32_t tmem = s.tmem;
  volatile int* abort = &s.abort;

  if (warp == 0) {
    Tiles<CG, kGate> tl(a, s.first_tile, s.tiles);
    int st = 0;
    uint32_t round = 0;
    int64_t issued = 0;
    bool ok = true;
    while (ok && tl.next()) {
      const int half = tl.cols() / CG;  // columns whose rows this CTA loads
      // ... in one box, which may be a little higher: a box costs the issuing warp about 100 cycles, rows little
      const int box = half <= 16 ? 16 : half <= 32 ? 32 : half <= 64 ? 64 : S::kRowsB;
      const CUtensorMap* map = half <= 16 ? &map_x16 : half <= 32 ? &map_x32 : half <= 64 ? &map_x64 : &map_x;
      const int wr = static_cast<int>(tl.weight_row0()), up = a.N / 2;
      const int xr = tl.row0 + rank * half;
      for (int kb = 0; kb < a.kstages; ++kb) {
        if (!wait_warp(&s.empty[st], (round & 1u) ^ 1u, abort, a.status)) {
          ok = false;
          break;
        }
        if (elect_one()) {
          moe::mbar_arrive_expect_tx(&s.full[st], kBytesA + box * 128);
          const int x = kb * 128;
          uint8_t* dst = s.ab[st];
          if (!kGate) {
            tma_load_2d(dst, &map_w, x, wr, &s.full[st]);
          } else if (a.gate_box) {
            tma_load_gate(dst, &map_w, x, tl.f * (kTileF / 2 / kBoxRows), tl.e, &s.full[st]);
          } else {
#pragma unroll
            for (int b = 0; b < kTileF / (2 * kBoxRows); ++b) {
              tma_load_2d(dst + (2 * b) * kBoxRows * 128, &map_w, x, wr + b * kBoxRows, &s.full[st]);
              tma_load_2d(dst + (2 * b + 1) * kBoxRows * 128, &map_w, x, wr + up + b * kBoxRows, &s.full[st]);
            }
          }
          tma_load_2d(dst + kBytesA, map, x, xr, &s.full[st]);
        }
        __syncwarp();
        ++issued;
        if (++st == kStages) { st = 0; ++round; }
      }
    }
    // Never leave with an arrival on its way to this CTA's barriers.  The last stages' releases (in a pair they come from
    // the other CTA's commits) are waited for by nobody else; how they stand to the accumulator's arrival, which the
    // epilogue waits for, is not promised.
    const int64_t last = issued > kStages ? issued - kStages : 0;
    for (int64_t q = last; ok && q < issued; ++q)
      ok = wait_warp(&s.empty[q % kStages], static_cast<uint32_t>(q / kStages) & 1u, abort, a.status);
    if (*abort != 0) {  // nor with loads in flight into this CTA's shared memory
      for (int64_t q = last; q < issued; ++q)
        moe::mbar_wait(&s.full[q % kStages], static_cast<uint32_t>(q / kStages) & 1u, 200000000ull);
    }
  } else if (warp == 1 && rank == 0) {
    // instruction descriptor: A and B e2m1, scales e8m0, 128 lanes a CTA; columns and scale ids below
    constexpr uint32_t kDesc = (1u << 7) | (1u << 10) | (1u << 23) | ((CG * 128u >> 4) << 24);
    Tiles<CG, kGate> tl(a, s.first_tile, s.tiles);
    const uint64_t da0 = desc_sw128(moe::smem_addr(s.ab[0])), sf0 = desc_plain(moe::smem_addr(s.sf[0]));
    int st = 0, st2 = 0;  // the stage, and the one two before it
    uint32_t round = 0, round2 = 0, buf = 0, buf_round = 0, set = 0;
    int before = 0;      // stages before this one, up to 2
    bool ok = true;
    while (ok && tl.next()) {
      if (!wait_warp(&s.acc_empty[buf], (buf_round & 1u) ^ 1u, abort, a.status)) break;
      tmem_fence_after();
      const uint32_t idesc = kDesc | ((static_cast<uint32_t>(tl.cols()) >> 3) << 17);
      const uint32_t d = tmem + buf * S::kTileT;
      for (int kb = 0; kb < a.kstages; ++kb) {
        // the stage is there, and the products that read this set of TMEM scales, two stages ago, are done
        // (one test of both: a test takes about 100 cycles to answer)
        const bool older = before == 2;
        if (!__all_sync(0xffffffffu, phases_done(&s.full[st], round & 1u, older ? &s.empty[st2] : &s.full[st],
                                                 (older ? round2 : round) & 1u))) {
          ok = wait_warp(&s.full[st], round & 1u, abort, a.status) &&
               (!older || wait_warp(&s.empty[st2], round2 & 1u, abort, a.status));
          if (!ok) break;
        }
        if (older) {
          if (++st2 == kStages) { st2 = 0; ++round2; }
        } else {
          ++before;
        }
        const int now = st;
        if (++st == kStages) { st = 0; ++round; }
        moe::fence_proxy_async_smem();  // the scales were written by ordinary copies
        tmem_fence_after();
        if (elect_one()) {
          const uint32_t sf = tmem + S::kTmemSf + set * S::kSfCols;
          const uint64_t sfd = sf0 + static_cast<uint32_t>(now * (S::kBytesSf >> 4));
#pragma unroll
          for (int i = 0; i < S::kBytesSf / kAtom; ++i) sf_to_tmem<CG>(sf + 4 * i, sfd + i * (kAtom >> 4));
          const uint64_t da = da0 + static_cast<uint32_t>(now * (S::kStageBytes >> 4)), db = da + (kBytesA >> 4);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {  // 64 elements: 32 bytes further in the swizzle atom
            const uint32_t id = (kk & 1) * 2;  // which two of the chunk's four scales
            mma_mx4<CG>(d, da + kk * 2, db + kk * 2, idesc | (id << 4) | (id << 29), sf + 4 * (kk >> 1),
                        sf + 8 + 4 * S::kAtomsB * (kk >> 1), kb > 0 || kk > 0);
          }
          commit<CG>(&s.empty[now]);
          if (kb == a.kstages - 1) commit<CG>(&s.acc_full[buf]);
        }
        __syncwarp();
        set ^= 1u;
      }
      if (++buf == 2) { buf = 0; ++buf_round; }
    }
    if (before != 0) {  // products in flight still read shared memory and write TMEM
      if (elect_one()) commit_own<CG>(&s.drained);
      __syncwarp();
      moe::mbar_wait(&s.drained, 0, 200000000ull);
      // after a wait that ran out, the other CTA may no longer wait for the arrivals of the commits above: they get a
      // millisecond, where they take well under a microsecond
      if (CG == 2 && *abort != 0) __nanosleep(1000000);
    }
  } else if (warp == 1) {  // the pair's second CTA: tell the first that a stage is there
    Tiles<CG, kGate> tl(a, s.first_tile, s.tiles);
    int st = 0;
    uint32_t round = 0;
    bool ok = true;
    while (ok && tl.next()) {
      for (int kb = 0; kb < a.kstages; ++kb) {
        if (!wait_warp(&s.full[st], round & 1u, abort, a.status)) {
          ok = false;
          break;
        }
        moe::fence_proxy_async_smem();  // the scales were written by ordinary copies
        if (elect_one()) arrive_first(&s.full[st]);
        __syncwarp();
        if (++st == kStages) { st = 0; ++round; }
      }
    }
  } else if (warp < 4) {
    // Scales: chunk 2 kb + (warp - 2) of each stage.  Lane l copies the words of rows l, 32 + l, 64 + l, 96 + l (of the
    // weights' tile, then of each 128 of x's) side by side; the copies (cp.async) complete on the stage's barrier.
    Tiles<CG, kGate> tl(a, s.first_tile, s.tiles);
    const int which = warp - 2;
    const int64_t w_rows = static_cast<int64_t>(a.E) * a.N;
    int st = 0;
    uint32_t round = 0;
    bool ok = true;
    while (ok && tl.next()) {
      const int groups = (tl.cols() + 31) / 32;
      int wr[4], xr[4 * S::kAtomsB];
#pragma unroll
      for (int c = 0; c < 4; ++c) wr[c] = static_cast<int>(tl.weight_row(32 * c + lane));
#pragma unroll
      for (int c = 0; c < 4 * S::kAtomsB; ++c) {  // (columns past the rows repeat the last one: not stored)
        const int n = 32 * c + lane;
        xr[c] = tl.row0 + (n < tl.rows ? n : tl.rows - 1);
      }
      const uint32_t* w = a.w_sf + which * w_rows;
      const uint32_t* x = a.x_sf + which * a.capacity;
      for (int kb = 0; kb < a.kstages; ++kb, w += 2 * w_rows, x += 2 * a.capacity) {
        if (!wait_warp(&s.empty[st], (round & 1u) ^ 1u, abort, a.status)) {
          ok = false;
          break;
        }
        uint8_t* sfa = s.sf[st] + which * kAtom + lane * 16;
        uint8_t* sfb = s.sf[st] + (2 + which * S::kAtomsB) * kAtom + lane * 16;
        if ((kb + 1) * kStageK <= a.K) {
#pragma unroll
          for (int c = 0; c < 4; ++c) copy_word(sfa + 4 * c, w + wr[c]);
#pragma unroll
          for (int c = 0; c < 4 * S::kAtomsB; ++c)
            if (c < groups) copy_word(sfb + (c >> 2) * kAtom + 4 * (c & 3), x + xr[c]);
          asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(moe::smem_addr(&s.full[st]))
                       : "memory");
        } else {  // the last stage of a K that is no multiple of 256
          // bytes of blocks past K: 1, whatever is there (their codes are zeros, but NaN times zero is NaN)
          const int c0 = 2 * kb + which, past = (c0 + 1) * 4 - a.K / 32;
          const uint32_t keep = past <= 0 ? 0xffffffffu : past >= 4 ? 0u : 0xffffffffu >> (8 * past);
          auto put = [&](uint8_t* dst, const uint32_t* src) {
            *reinterpret_cast<uint32_t*>(dst) = ((keep != 0u ? __ldg(src) : 0u) & keep) | (0x7f7f7f7fu & ~keep);
          };
#pragma unroll
          for (int c = 0; c < 4; ++c) put(sfa + 4 * c, w + wr[c]);
#pragma unroll
          for (int c = 0; c < 4 * S::kAtomsB; ++c)
            if (c < groups) put(sfb + (c >> 2) * kAtom + 4 * (c & 3), x + xr[c]);
          moe::fence_proxy_async_smem();
          moe::mbar_arrive(&s.full[st]);
        }
        if (++st == kStages) { st = 0; ++round; }
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else {
    Tiles<CG, kGate> tl(a, s.first_tile, s.tiles);
    const int quad = warp & 3, turn = (warp - 4) >> 2;  // lanes 32 quad .. +31, column blocks turn, turn + 2, ...
    uint32_t buf = 0, buf_round = 0, half = 0;
    // a lane's place in a block: stmatrix writes 16 bytes of row j at chunk m, both swizzled as the store's map says
    const int sj = lane & 7, sm = lane >> 3;
    while (tl.next()) {
      if (!wait_warp(&s.acc_full[buf], buf_round & 1u, abort, a.status)) break;
      tmem_fence_after();
      const int cols = tl.cols();
      const int col0 = kGate ? tl.f * (kTileF / 2) + quad * 16 : tl.f * kTileF + quad * 32;
      for (int c0 = turn * kEpiT; c0 < cols; c0 += 2 * kEpiT) {
        uint32_t lo[16], hi[16];  // lanes 0..15 and 16..31: with the gate, gate and up
        const uint32_t taddr = tmem + (static_cast<uint32_t>(quad * 32) << 16) + buf * S::kTileT + c0;
        tmem_ld16x32(taddr, lo);
        tmem_ld16x32(taddr + (16u << 16), hi);
        uint8_t* epi = s.epi[warp - 4][half];
        const uint32_t epi_addr = moe::smem_addr(epi);
        half ^= 1u;
        if (elect_one()) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");  // this half has been read
        __syncwarp();
        tmem_wait_ld();
        if (kGate) {  // 16 features, rows of 32 bytes: chunk ^= row / 4
#pragma unroll
          for (int i = 0; i < 4; i += 2) {
            uint32_t p[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int v = 4 * i + 2 * q;
              p[q] = moe::pack_bf16x2(silu_times(lo[v], hi[v]), silu_times(lo[v + 1], hi[v + 1]));
            }
            // blocks: columns 8i, features 0..7 and 8..15; columns 8i + 8, the same
            stmatrix_trans(epi_addr + (8 * (i + (sm >> 1)) + sj) * 32 + (((sm & 1) ^ (sj >> 2)) << 4), p[0], p[1], p[2],
                           p[3]);
          }
        } else {  // 32 features, rows of 64 bytes: chunk ^= row / 2
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int v = 4 * i;
            stmatrix_trans(epi_addr + (8 * i + sj) * 64 + ((sm ^ (sj >> 1)) << 4),
                           moe::pack_bf16x2(__uint_as_float(lo[v]), __uint_as_float(lo[v + 1])),
                           moe::pack_bf16x2(__uint_as_float(lo[v + 2]), __uint_as_float(lo[v + 3])),
                           moe::pack_bf16x2(__uint_as_float(hi[v]), __uint_as_float(hi[v + 1])),
                           moe::pack_bf16x2(__uint_as_float(hi[v + 2]), __uint_as_float(hi[v + 3])));
          }
        }
        const int left = tl.rows - c0;
        if (left >= kEpiT) {  // whole: one copy (features past the last are clipped)
          moe::fence_proxy_async_smem();
          __syncwarp();
          if (elect_one()) {
            if (col0 < a.ld_out)
              asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                               &map_out),
                           "r"(col0), "r"(tl.row0 + c0), "r"(epi_addr)
                           : "memory");
            moe::bulk_commit();
          }
        } else {  // the last rows of an expert: what follows is not this expert's to write
          __syncwarp();
          __nv_bfloat16* out = a.out + static_cast<int64_t>(tl.row0 + c0) * a.ld_out + col0;
          constexpr int shift = kGate ? 1 : 2;  // log2 of a row's 16-byte chunks
          for (int i = lane; i < left << shift; i += 32) {
            const int j = i >> shift, g = i & ((1 << shift) - 1);
            if (col0 + g * 8 >= a.ld_out) continue;
            const int at = kGate ? j * 32 + ((g ^ ((j >> 2) & 1)) << 4) : j * 64 + ((g ^ ((j >> 1) & 3)) << 4);
            moe::st_plain(reinterpret_cast<uint4*>(out + j * a.ld_out + g * 8), moe::lds128(epi + at));
          }
          if (elect_one()) moe::bulk_commit();  // (empty: a group a block)
        }
      }
      tmem_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (CG == 1 || rank == 0)
          moe::mbar_arrive(&s.acc_empty[buf]);
        else
          arrive_first(&s.acc_empty[buf]);
      }
      if (++buf == 2) { buf = 0; ++buf_round; }
    }
    __syncwarp();
    if (elect_one()) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }
  tmem_fence_before();
  __syncthreads();
  if constexpr (CG == 2) {  // the pair's products read both CTAs' memory, and its barriers are reached from both
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  }
  if (warp == 1) {
    tmem_fence_after();
    if constexpr (CG == 1)
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
    else
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
  }
}

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
  static const EncodeTiled fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeTiled>(p);
  }();
  return fn;
}

// codes [rows, K/2] in boxes of `box` rows by 128 bytes, 128-byte swizzle, zeros outside
bool codes_map(CUtensorMap* m, const void* codes, int64_t rows, int32_t K, uint32_t box) {
  const EncodeTiled enc = encode_tiled();
  if (enc == nullptr) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(K / 2), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(K / 2)};
  const cuuint32_t boxes[2] = {kStageK / 2, box};
  const cuuint32_t ones[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(codes), dims, strides, boxes, ones,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// codes [E, 2, N/2, K/2] with the N/2 features in groups of 16: a box is four groups' gate and up features by 128
// bytes, group by group
bool gate_map(CUtensorMap* m, const void* codes, int32_t E, int32_t N, int32_t K) {
  const EncodeTiled enc = encode_tiled();
  if (enc == nullptr) return false;
  const cuuint64_t row = static_cast<cuuint64_t>(K / 2);
  const cuuint64_t dims[5] = {row, kBoxRows, 2, static_cast<cuuint64_t>(N / 2 / kBoxRows), static_cast<cuuint64_t>(E)};
  const cuuint64_t strides[4] = {row, row * (N / 2), row * kBoxRows, row * N};
  const cuuint32_t boxes[5] = {kStageK / 2, kBoxRows, 2, kTileF / 2 / kBoxRows, 1};
  const cuuint32_t ones[5] = {1, 1, 1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 5, const_cast<void*>(codes), dims, strides, boxes, ones,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// out [capacity, cols] bf16: a box is 32 rows of an epilogue warp's 32 features, 16 with the gate
bool out_map(CUtensorMap* m, void* out, int64_t rows, int64_t cols, bool gate) {
  const EncodeTiled enc = encode_tiled();
  if (enc == nullptr) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(cols) * 2};
  const cuuint32_t boxes[2] = {gate ? 16u : 32u, kEpiT};
  const cuuint32_t ones[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, out, dims, strides, boxes, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
             gate ? CU_TENSOR_MAP_SWIZZLE_32B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Rows of capacity an expert from which on pairs of CTAs take a tile.  Both forms with 128 experts and blocks of 16,
// us, single | pair: 4096 -> 2816 gated, 8 rows an expert 127 | 132, 48 rows 132 | 138, 64 rows 161 | 139, 128 rows
// 266 | 151; 768 -> 2048, 8 rows 22.6 | 23.9, 48 rows 25.4 | 26.3, 64 rows 31.9 | 27.4, 128 rows 50.8 | 32.1; one token of
// six experts 4.7 | 5.7.  (A single CTA's tile ends at 64 rows.  The host knows the capacity only: all T k slots, other
// ranks' among them, and padding.  A rank with an eighth of the experts takes pairs from 8 rows an expert on, which by
// the sweep costs it 3.5 to 6 % below 64; where padding makes the most of it, 2 rows in blocks of 128, 0 to 5 %.)
constexpr int kPairRows = 64;

template <int CG, bool kGate>
moe_status_t launch_product(ProductArgs a, const CUtensorMap (&mx)[4], const CUtensorMap& mw,
                            const CUtensorMap& mo, cudaStream_t st) {
  const int per = CG * (kGate ? kTileF / 2 : kTileF);
  a.ftiles = static_cast<int>((a.ld_out + per - 1) / per);
  const int sms = moe_host::sm_count();
  if (sms <= 0) return MOE_ERR_CUDA;
  // no more CTAs than tiles there can be: a row tile per expert and per kTileT rows
  const int64_t most = ((a.E < a.capacity ? a.E : a.capacity) + a.capacity / Shape<CG, kGate>::kTileT) * a.ftiles;
  const int64_t grid = (most < sms / CG ? most : sms / CG) * CG;
  const size_t smem = sizeof(typename Shape<CG, kGate>::Smem) + 1024;
  const void* kernel = reinterpret_cast<const void*>(&grouped_mx4_kernel<CG, kGate>);
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) !=
          cudaSuccess ||
      moe_host::prefer_max_shared(kernel) != cudaSuccess)
    return MOE_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CG;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = CG == 1 ? 1 : 2;
  return cudaLaunchKernelEx(&cfg, grouped_mx4_kernel<CG, kGate>, mx[0], mx[1], mx[2], mx[3], mw, mo, a) == cudaSuccess
             ? MOE_OK
             : MOE_ERR_CUDA;
}

}  // namespace

extern "C" moe_status_t moe_grouped_gemm_mx4(const void* x_codes, const void* x_scales, const void* w_codes,
                                             const void* w_scales, const int32_t* counts, const int32_t* offsets,
                                             int32_t E_local, int64_t capacity, int32_t N, int32_t K, uint32_t flags,
                                             void* out, int32_t* device_status, void* stream) {
  if (E_local < 1 || capacity < 0 || N < 8 || (N % 8) != 0 || K < 32 || (K % 32) != 0) return MOE_ERR_INVALID_ARG;
  if ((flags & ~MOE_MX4_SWIGLU) != 0u) return MOE_ERR_INVALID_ARG;
  const bool gate = (flags & MOE_MX4_SWIGLU) != 0u;
  if (gate && (N % 16) != 0) return MOE_ERR_INVALID_ARG;
  if (capacity >= (int64_t{1} << 31) - 256 || K > (1 << 20) || N > (1 << 20)) return MOE_ERR_INVALID_ARG;
  if (E_local > kMaxExperts) return MOE_ERR_UNSUPPORTED;  // (E_local * N is at most 2^30: row indices are int32)
  if (capacity == 0) return MOE_OK;
  if (x_codes == nullptr || x_scales == nullptr || w_codes == nullptr || w_scales == nullptr || counts == nullptr ||
      offsets == nullptr || out == nullptr)
    return MOE_ERR_INVALID_ARG;
  if (!moe_host::aligned16(x_codes) || !moe_host::aligned16(x_scales) || !moe_host::aligned16(w_codes) ||
      !moe_host::aligned16(w_scales) || !moe_host::aligned16(out))
    return MOE_ERR_INVALID_ARG;
  ProductArgs a{};
  a.x_sf = static_cast<const uint32_t*>(x_scales);
  a.w_sf = static_cast<const uint32_t*>(w_scales);
  a.counts = counts;
  a.offsets = offsets;
  a.E = E_local;
  a.N = N;
  a.K = K;
  a.kstages = (K + kStageK - 1) / kStageK;
  a.ld_out = gate ? N / 2 : N;
  a.capacity = capacity;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.status = device_status;
  a.gate_box = gate && (N % 32) == 0 ? 1 : 0;
  const bool pair = capacity >= int64_t{E_local} * kPairRows;  // many rows an expert
  CUtensorMap mx[4], mw, mo;
  if (!out_map(&mo, out, capacity, a.ld_out, gate)) return MOE_ERR_CUDA;
  for (int i = 0; i < 4; ++i) {
    const uint32_t box = i < 3 ? kBoxRows << i : pair ? Shape<2, false>::kRowsB : Shape<1, false>::kRowsB;
    if (!codes_map(&mx[i], x_codes, capacity, K, box)) return MOE_ERR_CUDA;
  }
  if (!(a.gate_box ? gate_map(&mw, w_codes, E_local, N, K)
                   : codes_map(&mw, w_codes, static_cast<int64_t>(E_local) * N, K, gate ? kBoxRows : kTileF)))
    return MOE_ERR_CUDA;
  const auto launch = pair ? (gate ? launch_product<2, true> : launch_product<2, false>)
                           : (gate ? launch_product<1, true> : launch_product<1, false>);
  return launch(a, mx, mw, mo, static_cast<cudaStream_t>(stream));
}
