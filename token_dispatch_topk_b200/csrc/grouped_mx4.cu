// grouped_mx4.cu -- the experts' matrix product in microscaled 4-bit floating point (the format: mx4_cast.cu).
//
//   out[r, n] = bf16( sum_k x[r, k] w[e, n, k] )  for the rows r of expert e (offsets[e] .. offsets[e] + counts[e] - 1)
// or, with the gate,
//   out[r, n] = bf16( silu(a) b ), a = sum_k x[r, k] w[e, n, k], b = sum_k x[r, k] w[e, N/2 + n, k], n < N/2,
// silu(a) = a / (1 + exp(-a)), sums and gate in fp32, one rounding.
//
// A tile is 128 features of one expert (the 128 TMEM lanes, operand A = weights) by up to kTileT of its rows
// (operand B, the accumulator's columns).  Features, not rows, take the fixed side of 128: an expert has any number
// of rows, one at decode, and the column side of tcgen05.mma goes in steps of 16.  With the gate a tile's lanes are
// 64 gate and the 64 matching up features.  The rows of an expert are split evenly over as few tiles as hold them.
//
// One CTA per SM walks the tiles.  Warp 0: TMA loads into a ring of 256-element stages.  Warps 2 and 3: the scale
// words of the stage's two 128-element chunks into the order tcgen05.cp wants, read ahead into registers.
// Warp 1: copies the scales to TMEM and issues the products (kind::mxf4, block-scaled, 64 elements each).  Warps
// 4..7: the accumulator of the previous tile out of TMEM, through shared memory, to rows of out.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"

namespace {

constexpr int kThreads = 256;
constexpr int kTileF = 128;             // features a tile
constexpr int kTileT = 128;             // rows a tile, at most
constexpr int kStageK = 256;            // elements of K a stage: 128 bytes, one swizzle atom
constexpr int kStages = 6;
constexpr int kBoxT = 32;               // rows of x a TMA box
constexpr int kBoxF = 64;               // features a TMA box (the gate and up halves of a tile)
constexpr int kBytesA = kTileF * kStageK / 2;
constexpr int kBytesB = kTileT * kStageK / 2;
constexpr int kAtom = 512;              // scales of 128 rows by 128 elements
constexpr int kBytesSf = 2 * kAtom + 2 * kAtom * (kTileT / 128);
constexpr int kStageBytes = kBytesA + kBytesB;
constexpr int kEpiT = 32;               // rows of a tile that go through shared memory at a time
constexpr int kEpiStride = kTileF + 4;  // fp32 words a row there
constexpr int kMaxExperts = 1024;
constexpr int kSfAhead = 4;             // stages whose scales are in registers
// TMEM columns: two accumulators, then each stage's scales (four columns an atom)
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemSf = 2 * kTileT;
constexpr uint32_t kTmemSfStage = 8 + 8 * (kTileT / 128);
static_assert(kTmemSf + kStages * kTmemSfStage <= kTmemCols, "TMEM columns");

struct __align__(1024) Smem {
  uint8_t ab[kStages][kStageBytes];  // A then B, 128-byte swizzled
  uint8_t sf[kStages][kBytesSf];     // A's two atoms, then B's
  float epi[kEpiT * kEpiStride];
  int32_t first_tile[kMaxExperts + 1];  // row tiles before expert e
  int32_t warp_sums[8];
  uint64_t full[kStages], empty[kStages], acc_full[2], acc_empty[2], drained;
  uint32_t tmem;
  int abort;
  int epi_go;
};
static_assert(sizeof(Smem) + 1024 <= 232448, "shared memory");

struct ProductArgs {
  const uint32_t* x_sf;  // [chunks, capacity] scale words
  const uint32_t* w_sf;  // [chunks, E*N]
  const int32_t* counts;
  const int32_t* offsets;
  int E, N, K;
  int chunks;     // ceil(K / 128)
  int kstages;    // ceil(K / 256)
  int ftiles;     // feature tiles
  int gate;       // 1: silu(gate) * up
  int64_t capacity;
  __nv_bfloat16* out;
  int64_t ld_out;  // N or N / 2
  int32_t* status;
};

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

__device__ __forceinline__ void sf_to_tmem(uint32_t taddr, uint32_t smem) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc_plain(smem)) : "memory");
}

__device__ __forceinline__ void mma_mx4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                        bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate ? 1u : 0u)
      : "memory");
}

__device__ __forceinline__ void commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(moe::smem_addr(bar))
               : "memory");
}
__device__ __forceinline__ void tmem_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
        "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
        "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// A bounded wait that polls without sleeping (the wait itself suspends in hardware); it also gives up when another
// role of the CTA has.
__device__ __forceinline__ bool wait_stage(uint64_t* bar, uint32_t parity, volatile int* abort, int32_t* status) {
  if (moe::mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = moe::global_ns();
  for (;;) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (moe::mbar_try_wait(bar, parity)) return true;
    if (*abort != 0) return false;
    if (moe::global_ns() - t0 > moe::kWaitLimitNs) {
      moe::record_status(status, MOE_ERR_TIMEOUT);
      *abort = 1;
      return false;
    }
  }
}

// The tiles of this CTA, in order: expert by expert, then row tiles, features fastest.
struct Tiles {
  const ProductArgs& a;
  const int32_t* first;  // row tiles before expert e
  int64_t t, end;
  int e = 0;
  int f, row0, rows;  // feature tile, first row, rows

  __device__ Tiles(const ProductArgs& args, const int32_t* first_tile)
      : a(args), first(first_tile), t(static_cast<int64_t>(blockIdx.x) - gridDim.x),
        end(static_cast<int64_t>(first_tile[args.E]) * args.ftiles) {}
  __device__ bool next() {
    t += gridDim.x;
    if (t >= end) return false;
    const int rt = static_cast<int>(t / a.ftiles);
    f = static_cast<int>(t - static_cast<int64_t>(rt) * a.ftiles);
    while (first[e + 1] <= rt) ++e;
    const int cnt = a.counts[e], n = first[e + 1] - first[e];
    const int per = ((cnt + n - 1) / n + 15) & ~15;  // at most kTileT
    const int i = rt - first[e];
    row0 = a.offsets[e] + i * per;
    rows = cnt - i * per < per ? cnt - i * per : per;
    return true;
  }
  __device__ int cols() const { return (rows + 15) & ~15; }  // the product's columns
  // row of the weights that lane m of the tile holds (clamped: lanes past the expert's features are not stored)
  __device__ int weight_row(int m) const {
    const int64_t base = static_cast<int64_t>(e) * a.N;
    const int64_t r = !a.gate ? base + f * kTileF + m
                              : base + f * kBoxF + (m < kBoxF ? m : a.N / 2 + m - kBoxF);
    const int64_t last = static_cast<int64_t>(a.E) * a.N - 1;
    return static_cast<int>(r < last ? r : last);
  }
};

__global__ void __launch_bounds__(kThreads, 1)
grouped_mx4_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                   const ProductArgs a) {
  extern __shared__ uint8_t smem_raw[];
  Smem& s = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      moe::mbar_init(&s.full[i], 3);  // the TMA warp and the two scale warps
      moe::mbar_init(&s.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      moe::mbar_init(&s.acc_full[i], 1);
      moe::mbar_init(&s.acc_empty[i], 4);
    }
    moe::mbar_init(&s.drained, 1);
    s.abort = 0;
    moe::fence_barrier_init();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(moe::smem_addr(&s.tmem)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  moe::pdl_launch_dependents();
  moe::pdl_wait();  // rows, scales, counts and offsets may come from the previous kernel

  // row tiles before each expert: four experts a thread
  {
    int n[4], sum = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = tid * 4 + i;
      n[i] = 0;
      if (e < a.E) {
        const int64_t cnt = a.counts[e], off = a.offsets[e];
        if (cnt < 0 || off < 0 || off + cnt > a.capacity)
          moe::record_status(a.status, MOE_ERR_BAD_ROW);  // skipped
        else
          n[i] = static_cast<int>((cnt + kTileT - 1) / kTileT);
      }
      sum += n[i];
    }
    int incl = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += o;
    }
    if (lane == 31) s.warp_sums[warp] = incl;
    __syncthreads();
    int before = incl - sum;
    for (int w = 0; w < warp; ++w) before += s.warp_sums[w];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = tid * 4 + i;
      if (e <= a.E) s.first_tile[e] = before;
      before += n[i];
    }
    if (tid == kThreads - 1 && a.E == kMaxExperts) s.first_tile[kMaxExperts] = before;
  }
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = s.tmem;
  volatile int* abort = &s.abort;

  if (warp == 0) {
    if (lane == 0) {
      Tiles tl(a, s.first_tile);
      int st = 0;
      uint32_t round = 0;
      int64_t issued = 0;
      bool ok = true;
      while (ok && tl.next()) {
        const int boxes = (tl.cols() + kBoxT - 1) / kBoxT;
        const int64_t wr = static_cast<int64_t>(tl.e) * a.N + static_cast<int64_t>(tl.f) * (a.gate ? kBoxF : kTileF);
        const int w0 = static_cast<int>(wr), w1 = w0 + (a.gate ? a.N / 2 : kBoxF);
        for (int kb = 0; kb < a.kstages; ++kb) {
          if (!wait_stage(&s.empty[st], (round & 1u) ^ 1u, abort, a.status)) {
            ok = false;
            break;
          }
          moe::mbar_arrive_expect_tx(&s.full[st], kBytesA + boxes * (kBoxT * 128));
          const int x = kb * 128;
          tma_load_2d(s.ab[st], &map_w, x, w0, &s.full[st]);
          tma_load_2d(s.ab[st] + kBytesA / 2, &map_w, x, w1, &s.full[st]);
          for (int b = 0; b < boxes; ++b)
            tma_load_2d(s.ab[st] + kBytesA + b * (kBoxT * 128), &map_x, x, tl.row0 + b * kBoxT, &s.full[st]);
          ++issued;
          if (++st == kStages) { st = 0; ++round; }
        }
      }
      if (*abort != 0) {  // never leave with loads in flight into this CTA's shared memory
        for (int64_t q = issued > kStages ? issued - kStages : 0; q < issued; ++q)
          moe::mbar_wait(&s.full[q % kStages], static_cast<uint32_t>(q / kStages) & 1u, 200000000ull);
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      // instruction descriptor: A and B e2m1, scales e8m0, 128 lanes; columns and scale ids below
      constexpr uint32_t kDesc = (1u << 7) | (1u << 10) | (1u << 23) | ((128u >> 4) << 24);
      Tiles tl(a, s.first_tile);
      int st = 0;
      uint32_t round = 0, buf = 0, buf_round = 0;
      bool ok = true;
      while (ok && tl.next()) {
        if (!wait_stage(&s.acc_empty[buf], (buf_round & 1u) ^ 1u, abort, a.status)) break;
        tmem_fence_after();
        const uint32_t cols = static_cast<uint32_t>(tl.cols());
        const uint32_t idesc = kDesc | ((cols >> 3) << 17);
        const uint32_t d = tmem + buf * kTileT;
        for (int kb = 0; kb < a.kstages; ++kb) {
          if (!wait_stage(&s.full[st], round & 1u, abort, a.status)) {
            ok = false;
            break;
          }
          tmem_fence_after();
          const uint32_t sf = tmem + kTmemSf + static_cast<uint32_t>(st) * kTmemSfStage;
          const uint32_t sf_smem = moe::smem_addr(s.sf[st]);
#pragma unroll
          for (int i = 0; i < kBytesSf / kAtom; ++i) sf_to_tmem(sf + 4 * i, sf_smem + i * kAtom);
          const uint64_t da = desc_sw128(moe::smem_addr(s.ab[st]));
          const uint64_t db = desc_sw128(moe::smem_addr(s.ab[st] + kBytesA));
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {  // 64 elements: 32 bytes further in the swizzle atom
            const uint32_t id = (kk & 1) * 2;  // which two of the chunk's four scales
            mma_mx4(d, da + kk * 2, db + kk * 2, idesc | (id << 4) | (id << 29), sf + 4 * (kk >> 1),
                    sf + 8 + 4 * (kTileT / 128) * (kk >> 1), kb > 0 || kk > 0);
          }
          commit(&s.empty[st]);
          if (++st == kStages) { st = 0; ++round; }
        }
        if (!ok) break;
        commit(&s.acc_full[buf]);
        if (++buf == 2) { buf = 0; ++buf_round; }
      }
      if (*abort != 0) {  // products in flight still read shared memory and write TMEM
        commit(&s.drained);
        moe::mbar_wait(&s.drained, 0, 200000000ull);
      }
    }
  } else if (warp < 4) {
    // scales: chunk 2 kb + (warp - 2) of each stage, for lane l the words of rows l, 32 + l, 64 + l, 96 + l
    Tiles tl(a, s.first_tile);
    const int which = warp - 2;
    int kb = 0;
    bool more = tl.next();
    uint4 va[kSfAhead], vb[kSfAhead][kTileT / 128];
    bool have[kSfAhead];
    const int64_t w_rows = static_cast<int64_t>(a.E) * a.N;
    auto load = [&](int i) {
      have[i] = more;
      if (!more) return;
      const int c = kb * 2 + which;
      constexpr uint32_t kOne = 0x7f7f7f7fu;
      va[i] = make_uint4(kOne, kOne, kOne, kOne);
#pragma unroll
      for (int h = 0; h < kTileT / 128; ++h) vb[i][h] = va[i];
      if (c < a.chunks) {
        // bytes of blocks past K: 1, whatever is there (the codes are zeros, but NaN times zero is NaN)
        const int past = (c + 1) * 4 - a.K / 32;
        const uint32_t keep = past > 0 ? 0xffffffffu >> (8 * past) : 0xffffffffu;
        auto ours = [&](uint32_t v) -> uint32_t { return (v & keep) | (kOne & ~keep); };
        const uint32_t* w = a.w_sf + c * w_rows;
        va[i] = make_uint4(ours(__ldg(w + tl.weight_row(lane))), ours(__ldg(w + tl.weight_row(lane + 32))),
                           ours(__ldg(w + tl.weight_row(lane + 64))), ours(__ldg(w + tl.weight_row(lane + 96))));
        const uint32_t* x = a.x_sf + c * a.capacity;
        auto word = [&](int n) -> uint32_t { return n < tl.rows ? ours(__ldg(x + tl.row0 + n)) : kOne; };
#pragma unroll
        for (int h = 0; h < kTileT / 128; ++h)
          vb[i][h] = make_uint4(word(h * 128 + lane), word(h * 128 + 32 + lane), word(h * 128 + 64 + lane),
                                word(h * 128 + 96 + lane));
      }
      if (++kb == a.kstages) {
        kb = 0;
        more = tl.next();
      }
    };
#pragma unroll
    for (int i = 0; i < kSfAhead; ++i) load(i);
    int st = 0;
    uint32_t round = 0;
    bool ok = true;
    while (ok) {
#pragma unroll
      for (int i = 0; i < kSfAhead; ++i) {
        if (!ok || !have[i]) {
          ok = false;
          continue;
        }
        if (!__all_sync(0xffffffffu, wait_stage(&s.empty[st], (round & 1u) ^ 1u, abort, a.status))) {
          ok = false;
          continue;
        }
        uint8_t* sf = s.sf[st];
        *reinterpret_cast<uint4*>(sf + which * kAtom + lane * 16) = va[i];
#pragma unroll
        for (int h = 0; h < kTileT / 128; ++h)
          *reinterpret_cast<uint4*>(sf + 2 * kAtom + (which * (kTileT / 128) + h) * kAtom + lane * 16) = vb[i][h];
        moe::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) moe::mbar_arrive(&s.full[st]);
        if (++st == kStages) { st = 0; ++round; }
        load(i);
      }
    }
  } else {
    Tiles tl(a, s.first_tile);
    const int et = tid - 128, quad = warp - 4;
    uint32_t buf = 0, buf_round = 0;
    while (tl.next()) {
      // one thread waits, so that the four warps agree whether the accumulator came
      if (et == 0) s.epi_go = wait_stage(&s.acc_full[buf], buf_round & 1u, abort, a.status) ? 1 : 0;
      moe::named_barrier(1, 128);
      if (s.epi_go == 0) break;
      while (!moe::mbar_try_wait(&s.acc_full[buf], buf_round & 1u)) {
      }  // completed already: each thread's own acquire
      tmem_fence_after();
      const int cols = tl.cols();
      for (int c0 = 0; c0 < cols; c0 += kEpiT) {
        uint32_t v[32];
        tmem_ld32(tmem + (static_cast<uint32_t>(quad * 32) << 16) + buf * kTileT + c0, v);
        if (c0 + kEpiT >= cols) {
          tmem_fence_before();
          __syncwarp();
          if (lane == 0) moe::mbar_arrive(&s.acc_empty[buf]);
        }
        moe::named_barrier(1, 128);  // the previous rows have been read
#pragma unroll
        for (int j = 0; j < 32; ++j) s.epi[j * kEpiStride + quad * 32 + lane] = __uint_as_float(v[j]);
        moe::named_barrier(1, 128);
        const int left = tl.rows - c0 < kEpiT ? tl.rows - c0 : kEpiT;
        __nv_bfloat16* out = a.out + static_cast<int64_t>(tl.row0 + c0) * a.ld_out;
        if (a.gate) {
          for (int i = et; i < left * 8; i += 128) {
            const int j = i >> 3, g = (i & 7) * 8;
            const int64_t col = static_cast<int64_t>(tl.f) * kBoxF + g;
            if (col >= a.ld_out) continue;
            const float* p = s.epi + j * kEpiStride + g;
            uint32_t o[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const float g0 = p[2 * q], g1 = p[2 * q + 1];
              o[q] = moe::pack_bf16x2(__fdividef(g0, 1.f + __expf(-g0)) * p[kBoxF + 2 * q],
                                      __fdividef(g1, 1.f + __expf(-g1)) * p[kBoxF + 2 * q + 1]);
            }
            moe::st_plain(reinterpret_cast<uint4*>(out + j * a.ld_out + col), make_uint4(o[0], o[1], o[2], o[3]));
          }
        } else {
          for (int i = et; i < left * 16; i += 128) {
            const int j = i >> 4, g = (i & 15) * 8;
            const int64_t col = static_cast<int64_t>(tl.f) * kTileF + g;
            if (col >= a.ld_out) continue;
            const float4 p = *reinterpret_cast<const float4*>(s.epi + j * kEpiStride + g);
            const float4 q = *reinterpret_cast<const float4*>(s.epi + j * kEpiStride + g + 4);
            moe::st_plain(reinterpret_cast<uint4*>(out + j * a.ld_out + col),
                          make_uint4(moe::pack_bf16x2(p.x, p.y), moe::pack_bf16x2(p.z, p.w),
                                     moe::pack_bf16x2(q.x, q.y), moe::pack_bf16x2(q.z, q.w)));
          }
        }
      }
      if (++buf == 2) { buf = 0; ++buf_round; }
    }
  }
  tmem_fence_before();
  __syncthreads();
  if (warp == 1) {
    tmem_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
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
  a.chunks = (K + 127) / 128;
  a.kstages = (K + kStageK - 1) / kStageK;
  a.gate = gate ? 1 : 0;
  a.ld_out = gate ? N / 2 : N;
  const int per = gate ? kBoxF : kTileF;
  a.ftiles = static_cast<int>((a.ld_out + per - 1) / per);
  a.capacity = capacity;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.status = device_status;
  CUtensorMap mx, mw;
  if (!codes_map(&mx, x_codes, capacity, K, kBoxT) ||
      !codes_map(&mw, w_codes, static_cast<int64_t>(E_local) * N, K, kBoxF))
    return MOE_ERR_CUDA;
  const int sms = moe_host::sm_count();
  if (sms <= 0) return MOE_ERR_CUDA;
  // no more CTAs than tiles there can be: a row tile per expert and per kTileT rows
  const int64_t most = (E_local < capacity ? E_local : capacity) + capacity / kTileT;
  const int64_t grid = most * a.ftiles < sms ? most * a.ftiles : sms;
  const size_t smem = sizeof(Smem) + 1024;
  if (cudaFuncSetAttribute(grouped_mx4_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) !=
      cudaSuccess)
    return MOE_ERR_CUDA;
  return moe_host::launch_pdl_max_shared(grouped_mx4_kernel, dim3(static_cast<unsigned>(grid)), dim3(kThreads), smem,
                                         static_cast<cudaStream_t>(stream), mx, mw, a);
}
