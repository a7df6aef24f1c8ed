// route_grads.cu -- gradients of the routing layer: of the weighted combine, the permute-gather and the gating.
//
// Combine, out[t] = sum_j w[t,j] y[r(t,j)], with grad_out = dL/dout:
//   dL/dy[r(t,j)] = w[t,j] grad_out[t]        one rounding to bf16
//   dL/dw[t,j]    = sum_h grad_out[t,h] y[r(t,j),h]   fp32
// Permute-gather, permuted[r(t,j)] = hidden[t]:
//   dL/dhidden[t] = sum_j dL/dpermuted[r(t,j)]   fp32, one rounding to bf16
// Gating, over the selected experts i_1..i_k with incoming g_j = dL/dw_j and G = sum_j g_j w_j:
//   softmax over all E       dL/dx_e   = p_e (g_e - G), p = softmax(x), g_e = 0 where e is not selected
//   softmax, renormalised    dL/dx_i_j = w_j (g_j - G), 0 elsewhere (the logits are not read)
//   logistic                 dL/dx_i_j = g_j w_j (1 - s_j)
//   logistic, renormalised   dL/dx_i_j = w_j (1 - s_j) (g_j - G)
// with 1 - s = 1 / (1 + exp(x)) taken from the logit, not by subtracting from 1.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"

namespace {

constexpr int kWarps = 8;
constexpr int kUnroll = 4;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}

struct CombineGradArgs {
  const uint4* gout;        // [T, H] bf16, NV vectors a row
  const uint4* y;           // [capacity, H] bf16
  const float* w;           // [T*k]
  const int32_t* inv_perm;  // [T*k]
  int64_t slots;            // T*k
  int k;
  int nv;                   // H / 8
  int64_t capacity;
  uint4* gy;                // [capacity, H] bf16 or null
  float* gw;                // [T*k] or null
  const int32_t* sorted_ids;  // pads: null unless the pad rows are to be zeroed
  const int32_t* n_pad;
  int64_t slot_blocks;      // CTAs below this index take slots, the others pad rows
  int pad_rows;             // rows that a warp of those looks at
  int32_t* status;
};


// One warp per slot; the k slots of a token sit in neighbouring warps, so its gradient row comes from DRAM once and from
// L1 / L2 after that.  Bandwidth-bound: a row of y in, a row of gy out, 16 bytes a lane and kUnroll vectors in flight
// (four; two measured 1 % slower, one 15 %, fewer registers for more warps 6 %).  The pad rows follow at the end of the
// grid, one or two a warp: they are up to a tenth of a large batch's rows and most of a small one's, and with 32 rows a
// warp a few SMs wrote them alone at the end.  16384 x 8 x 7168, 4.23 GB: 650 us (6.5 TB/s, the copy rate), 726 with 32
// rows a warp, 668 with 8; 8 tokens of 64 experts in blocks of 64: 6.3 us, 34 with 32.
__global__ void __launch_bounds__(kWarps * 32) combine_grad_kernel(CombineGradArgs a) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  moe::pdl_launch_dependents();
  moe::pdl_wait();  // every input may come from the previous kernel
  if (blockIdx.x >= a.slot_blocks) {  // +0 into the pad rows below N_pad (their sorted id is T*k)
    const int64_t p0 = ((static_cast<int64_t>(blockIdx.x) - a.slot_blocks) * kWarps + warp) * a.pad_rows;
    int64_t end = a.n_pad[0];
    if (end > a.capacity) end = a.capacity;
    // a lane looks at a row, the warp then writes its pad rows one by one
    const bool pad = lane < a.pad_rows && p0 + lane < end && a.sorted_ids[p0 + lane] == static_cast<int32_t>(a.slots);
    for (unsigned pads = __ballot_sync(0xffffffffu, pad); pads != 0u; pads &= pads - 1u) {
      uint4* row = a.gy + (p0 + __ffs(pads) - 1) * a.nv;
      for (int v = lane; v < a.nv; v += 32) moe::st_plain(row + v, make_uint4(0u, 0u, 0u, 0u));
    }
    return;
  }
  const int64_t s = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  if (s >= a.slots) return;
  const int32_t r = a.inv_perm[s];
  if (r < 0 || r >= a.capacity) {  // remote slot (-1): no row, no gradient of its weight
    if (lane == 0) {
      if (r != -1) moe::record_status(a.status, MOE_ERR_BAD_ROW);
      if (a.gw != nullptr) a.gw[s] = 0.f;
    }
    return;
  }
  const float w = a.w[s];
  const uint4* g = a.gout + (s / a.k) * a.nv;
  const uint4* y = a.y + static_cast<int64_t>(r) * a.nv;
  uint4* gy = a.gy == nullptr ? nullptr : a.gy + static_cast<int64_t>(r) * a.nv;
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int vb = 0; vb < a.nv; vb += 32 * kUnroll) {
    uint4 gv[kUnroll], yv[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int v = vb + u * 32 + lane;
      gv[u] = yv[u] = make_uint4(0u, 0u, 0u, 0u);
      if (v < a.nv) {
        gv[u] = moe::ld_plain(g + v);
        if (a.gw != nullptr) yv[u] = moe::ld_stream(y + v);
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int v = vb + u * 32 + lane;
      const uint32_t gx[4] = {gv[u].x, gv[u].y, gv[u].z, gv[u].w}, yx[4] = {yv[u].x, yv[u].y, yv[u].z, yv[u].w};
      uint32_t o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float lo = moe::bf16_lo(gx[i]), hi = moe::bf16_hi(gx[i]);
        acc[2 * i] = fmaf(lo, moe::bf16_lo(yx[i]), acc[2 * i]);
        acc[2 * i + 1] = fmaf(hi, moe::bf16_hi(yx[i]), acc[2 * i + 1]);
        o[i] = moe::pack_bf16x2(w * lo, w * hi);
      }
      if (gy != nullptr && v < a.nv) moe::st_plain(gy + v, make_uint4(o[0], o[1], o[2], o[3]));
    }
  }
  if (a.gw != nullptr) {
    const float d = warp_sum(((acc[0] + acc[1]) + (acc[2] + acc[3])) + ((acc[4] + acc[5]) + (acc[6] + acc[7])));
    if (lane == 0) a.gw[s] = d;
  }
}

// ---------------------------------------------------------------------------------------------- gather --
// grad_hidden[t] = the sum of the token's local rows.  A warp takes kSumVecs vectors a lane of `per` tokens, whose slots
// its lanes read at once, and adds a token's rows kSumRows at a time, their loads in flight together.  Rows that are
// not there (other ranks' experts) cost nothing, which the combine's ring of fixed k-row stages cannot offer (one of
// four ranks, 16384 x 6 x 4096: 113 us by that kernel, 56 by this one; 4096 x 8 x 2048, all rows there: 26 and 21).
// Several tokens a warp, two rows at a time, are for sparse rows (one of eight ranks, 65536 x 8 x 2048: 89 us against
// 117 with one token and four rows) and cost full ones 4 % (16384 x 8 x 7168: 321 against 308, 323 at the copy rate).
constexpr int kSumVecs = 2;

template <int kSumRows, bool kOne>  // kOne: one token a warp
__global__ void __launch_bounds__(kWarps * 32)
gather_grad_kernel(const uint4* __restrict__ gp, const int32_t* __restrict__ inv_perm, int64_t T, int k, int per,
                   int nv, int segs, int64_t capacity, uint4* __restrict__ gx, int32_t* status) {
  moe::pdl_launch_dependents();
  moe::pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t wid = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int64_t group = wid / segs, t0 = kOne ? group : group * per;
  if (t0 >= T) return;
  const int n = kOne ? 1 : T - t0 < per ? static_cast<int>(T - t0) : per;
  int r = -1;
  if (lane < n * k) {
    r = inv_perm[t0 * k + lane];
    if (r < -1 || static_cast<int64_t>(r) >= capacity) {
      moe::record_status(status, MOE_ERR_BAD_ROW);
      r = -1;
    }
  }
  const unsigned local = __ballot_sync(0xffffffffu, r >= 0);
  const int v0 = static_cast<int>(wid - group * segs) * (32 * kSumVecs) + lane;
  for (int i = 0; i < n; ++i) {
    float acc[kSumVecs][8];
#pragma unroll
    for (int u = 0; u < kSumVecs; ++u)
#pragma unroll
      for (int q = 0; q < 8; ++q) acc[u][q] = 0.f;
    unsigned left = kOne || k == 32 ? local : local & (((1u << k) - 1u) << (i * k));
    while (left != 0u) {
      uint4 in[kSumRows][kSumVecs];
#pragma unroll
      for (int q = 0; q < kSumRows; ++q) {
#pragma unroll
        for (int u = 0; u < kSumVecs; ++u) in[q][u] = make_uint4(0u, 0u, 0u, 0u);
        if (left != 0u) {  // uniform; ascending slot order
          const int64_t row = __shfl_sync(0xffffffffu, r, __ffs(left) - 1);
          left &= left - 1u;
#pragma unroll
          for (int u = 0; u < kSumVecs; ++u)
            if (v0 + 32 * u < nv) in[q][u] = moe::ld_stream(gp + row * nv + v0 + 32 * u);
        }
      }
#pragma unroll
      for (int q = 0; q < kSumRows; ++q)  // (a row that is not there adds +0, which changes no sum)
#pragma unroll
        for (int u = 0; u < kSumVecs; ++u) {
          const uint32_t x[4] = {in[q][u].x, in[q][u].y, in[q][u].z, in[q][u].w};
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            acc[u][2 * w] += moe::bf16_lo(x[w]);
            acc[u][2 * w + 1] += moe::bf16_hi(x[w]);
          }
        }
    }
#pragma unroll
    for (int u = 0; u < kSumVecs; ++u)
      if (v0 + 32 * u < nv)
        moe::st_plain(gx + (t0 + i) * nv + v0 + 32 * u,
                      make_uint4(moe::pack_bf16x2(acc[u][0], acc[u][1]), moe::pack_bf16x2(acc[u][2], acc[u][3]),
                                 moe::pack_bf16x2(acc[u][4], acc[u][5]), moe::pack_bf16x2(acc[u][6], acc[u][7])));
  }
}

// ---------------------------------------------------------------------------------------------- gating --
constexpr int kGateWarps = 8;

struct GateGradArgs {
  const float* gw;      // [T, k] incoming
  const void* x;        // [T, E]
  const float* w;       // [T, k]
  const int32_t* ids;   // [T, k]
  int64_t T;
  int E, k;
  int renorm, sigmoid;
  int kp_log2;          // log2 of the lanes a row's slots take (k rounded up to a power of two)
  int g_log2;           // log2 of the lanes a row's logits take (dense)
  int iters;            // groups of 32 / G rows a warp takes (dense)
  int sums;             // floats of shared memory a warp's rows take (dense; a multiple of 4)
  void* gx;             // [T, E] out
  int32_t* status;
};

template <typename TX, int VEC>
struct RowVec;
template <>
struct RowVec<float, 4> {
  static __device__ __forceinline__ void load(const float* p, float (&v)[4]) {
    const float4 u = __ldcs(reinterpret_cast<const float4*>(p));
    v[0] = u.x; v[1] = u.y; v[2] = u.z; v[3] = u.w;
  }
  static __device__ __forceinline__ void store(float* p, const float (&v)[4]) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  }
};
template <>
struct RowVec<float, 1> {
  static __device__ __forceinline__ void load(const float* p, float (&v)[1]) { v[0] = __ldcs(p); }
  static __device__ __forceinline__ void store(float* p, const float (&v)[1]) { *p = v[0]; }
};
template <>
struct RowVec<__nv_bfloat16, 8> {
  static __device__ __forceinline__ void load(const __nv_bfloat16* p, float (&v)[8]) {
    const uint4 u = moe::ld_stream(reinterpret_cast<const uint4*>(p));
    v[0] = moe::bf16_lo(u.x); v[1] = moe::bf16_hi(u.x); v[2] = moe::bf16_lo(u.y); v[3] = moe::bf16_hi(u.y);
    v[4] = moe::bf16_lo(u.z); v[5] = moe::bf16_hi(u.z); v[6] = moe::bf16_lo(u.w); v[7] = moe::bf16_hi(u.w);
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float (&v)[8]) {
    moe::st_plain(reinterpret_cast<uint4*>(p),
                  make_uint4(moe::pack_bf16x2(v[0], v[1]), moe::pack_bf16x2(v[2], v[3]), moe::pack_bf16x2(v[4], v[5]),
                             moe::pack_bf16x2(v[6], v[7])));
  }
};
template <>
struct RowVec<__nv_bfloat16, 1> {
  static __device__ __forceinline__ void load(const __nv_bfloat16* p, float (&v)[1]) { v[0] = __bfloat162float(*p); }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float (&v)[1]) { *p = __float2bfloat16_rn(v[0]); }
};

template <typename TX>
__device__ __forceinline__ float one_logit(const TX* p) {
  float v[1];
  RowVec<TX, 1>::load(p, v);
  return v[0];
}

// The slots of a few rows, kp lanes a row (k rounded up to a power of two): lane j of a row's lanes has selected expert
// j.  value: what the expert's logit gets, complete in the lane that leads its expert (an expert named twice in a row
// adds up, in slot order); G = sum_j g_j w_j of the row.
struct Slots {
  int id;       // -1: none
  bool lead;
  float value, G;
};
template <typename TX, bool kDense>
__device__ __forceinline__ Slots take_slots(const GateGradArgs& a, int64_t t0, int r, int n, const TX* x, int lane) {
  const int kp = 1 << a.kp_log2, j = lane & (kp - 1), base = lane & ~(kp - 1);
  Slots s;
  s.id = -1;
  float g = 0.f, w = 0.f;
  if (r < n && j < a.k) {
    const int64_t at = (t0 + r) * a.k + j;
    s.id = a.ids[at];
    g = a.gw[at];
    w = a.w[at];
    if (s.id < 0 || s.id >= a.E) {
      moe::record_status(a.status, MOE_ERR_BAD_EXPERT_ID);
      s.id = -1;
      g = w = 0.f;
    }
  }
  float xs = 0.f;
  if (!kDense && a.sigmoid && s.id >= 0) xs = one_logit(x + static_cast<int64_t>(r) * a.E + s.id);
  s.G = g * w;
  for (int d = kp >> 1; d > 0; d >>= 1) s.G += __shfl_xor_sync(0xffffffffu, s.G, d);
  s.value = kDense ? g : a.renorm ? w * (g - s.G) : w * g;
  const unsigned same = __match_any_sync(0xffffffffu, s.id >= 0 ? (r << 10) | s.id : -1 - lane);
  s.lead = s.id >= 0 && __ffs(same) - 1 == lane;
  if (!kDense && a.sigmoid) {
    // all of a row's scores underflowed to 0: its weights are the constant 1/k
    const unsigned some = __ballot_sync(0xffffffffu, s.id >= 0 && expf(-xs) < INFINITY);
    const unsigned group = (kp == 32 ? 0xffffffffu : (1u << kp) - 1u) << base;
    s.value = (some & group) != 0u ? s.value / (1.f + expf(xs)) : 0.f;
  }
  if (__any_sync(0xffffffffu, __popc(same) > 1)) {
    const float mine = s.value;
    for (int m = 1; m < kp; ++m) {
      const float o = __shfl_sync(0xffffffffu, mine, base | ((j + m) & (kp - 1)));
      if (j + m < kp && ((same >> (lane + m)) & 1u)) s.value += o;
    }
  }
  return s;
}

// Only the selected experts' logits have a gradient: a warp takes as many rows as its lanes have room for their slots,
// sends zeros to the rows at once, while the slots (and, for the logistic, the scattered logits) are on their way, and
// then writes the selected elements over them.  Bound by the T E elements written and, for the logistic, by the
// 128-byte lines that hold the selected logits (eight of 256 bf16 logits lie in 3.6 of a row's four lines).  65536 x
// 256 bf16, k = 8: 13.6 us; 16.7 us with the rows put together in shared memory first.
template <typename TX, int VEC>
__global__ void __launch_bounds__(kGateWarps * 32) gate_grad_sparse_kernel(GateGradArgs a) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, E = a.E;
  const int rows = 32 >> a.kp_log2;
  const int64_t t0 = (static_cast<int64_t>(blockIdx.x) * kGateWarps + warp) * rows;
  const int n = a.T - t0 < rows ? static_cast<int>(a.T - t0) : rows;
  moe::pdl_launch_dependents();
  moe::pdl_wait();
  if (n <= 0) return;  // uniform per warp
  const TX* x = static_cast<const TX*>(a.x) + t0 * E;
  TX* gx = static_cast<TX*>(a.gx) + t0 * E;
  const bool in_place = a.sigmoid && a.x == a.gx;  // the logits are read before they are written
  const float zeros[VEC] = {};
  if (!in_place)
    for (int i = lane * VEC; i < n * E; i += 32 * VEC) RowVec<TX, VEC>::store(gx + i, zeros);
  const int r = lane >> a.kp_log2;
  const Slots s = take_slots<TX, false>(a, t0, r, n, x, lane);
  __syncwarp();
  if (in_place) {
    for (int i = lane * VEC; i < n * E; i += 32 * VEC) RowVec<TX, VEC>::store(gx + i, zeros);
    __syncwarp();
  }
  if (s.lead) {
    const float v[1] = {s.value};
    RowVec<TX, 1>::store(gx + r * E + s.id, v);
  }
}

// The softmax over all experts: every logit has a gradient.  A row takes G lanes, CPL vectors each; a warp takes
// a.iters (at most R, and R CPL VEC <= 32 registers) times 32 / G rows, all read first of all; the selected experts' g_j
// go into the rows' fp32 sums in shared memory meanwhile; the probabilities are recomputed.  Small batches wait for two
// dependent loads (16384 x 60 fp32: 4.7 us, 5.9 with one group of rows a warp), large ones for the chain of shuffles and
// exponentials of a row (65536 x 256 bf16: 37 us, 48 with one group, against 11 at the copy rate).  At most 64 registers:
// 37 us against 40.
constexpr int kDenseRows = 64;  // of a warp, at most
template <typename TX, int VEC, int CPL, int R>
__global__ void __launch_bounds__(kGateWarps * 32, 4) gate_grad_dense_kernel(GateGradArgs a) {
  extern __shared__ __align__(16) float s_rows[];  // as much as the rows need: more would cost resident warps
  __shared__ float s_sum[kGateWarps][kDenseRows];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, E = a.E;
  float* sums = s_rows + warp * a.sums;
  const int G = 1 << a.g_log2, side = 32 >> a.g_log2, rows = side * a.iters;
  const int l = lane & (G - 1), r1 = lane >> a.g_log2, chunks = E / VEC;
  const int64_t t0 = (static_cast<int64_t>(blockIdx.x) * kGateWarps + warp) * rows;
  const int n = a.T - t0 < rows ? static_cast<int>(a.T - t0) : rows;
  for (int i = lane * 4; i < n * E; i += 128) *reinterpret_cast<float4*>(sums + i) = make_float4(0.f, 0.f, 0.f, 0.f);
  moe::pdl_launch_dependents();
  moe::pdl_wait();
  if (n <= 0) return;  // uniform per warp
  const TX* x = static_cast<const TX*>(a.x) + t0 * E;
  TX* gx = static_cast<TX*>(a.gx) + t0 * E;
  float v[R][CPL][VEC];
#pragma unroll
  for (int o = 0; o < R; ++o) {
    const int r = o * side + r1;
#pragma unroll
    for (int i = 0; i < CPL; ++i) {
      const int c = l + i * G;
#pragma unroll
      for (int q = 0; q < VEC; ++q) v[o][i][q] = -INFINITY;
      if (r < n && c < chunks) RowVec<TX, VEC>::load(x + r * E + c * VEC, v[o][i]);
    }
  }
  __syncwarp();
  for (int r0 = 0; r0 < n; r0 += 32 >> a.kp_log2) {
    const int rs = r0 + (lane >> a.kp_log2);
    const Slots s = take_slots<TX, true>(a, t0, rs, n, x, lane);
    if (s.lead) sums[rs * E + s.id] = s.value;
    if ((lane & ((1 << a.kp_log2) - 1)) == 0 && rs < n) s_sum[warp][rs] = s.G;
  }
  __syncwarp();
#pragma unroll
  for (int o = 0; o < R; ++o) {
    if (o >= a.iters) break;  // uniform
    const int r = o * side + r1;
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < CPL; ++i)
#pragma unroll
      for (int q = 0; q < VEC; ++q) m = fmaxf(m, v[o][i][q]);
    for (int d = G >> 1; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    float z = 0.f;
#pragma unroll
    for (int i = 0; i < CPL; ++i)
#pragma unroll
      for (int q = 0; q < VEC; ++q) {
        v[o][i][q] = expf(v[o][i][q] - m);
        if (r < n && l + i * G < chunks) z += v[o][i][q];
      }
    for (int d = G >> 1; d > 0; d >>= 1) z += __shfl_xor_sync(0xffffffffu, z, d);
    z = 1.f / z;
    if (r < n) {
      const float mean = s_sum[warp][r];
#pragma unroll
      for (int i = 0; i < CPL; ++i) {
        const int c = l + i * G;
        if (c < chunks) {
#pragma unroll
          for (int q = 0; q < VEC; ++q) v[o][i][q] = v[o][i][q] * z * (sums[r * E + c * VEC + q] - mean);
          RowVec<TX, VEC>::store(gx + r * E + c * VEC, v[o][i]);
        }
      }
    }
  }
}

using GateKernel = void (*)(GateGradArgs);

// Vectors a lane for the dense gradient: the next of {1, 2, 4} (16-byte vectors of bf16), {1, 2, 8} (of fp32) or
// {2, 8, 32} (single elements) that holds E experts; and the row groups a warp holds in 32 registers a lane, at most 4.
struct DenseKernel {
  GateKernel kernel;
  int most;
};
template <typename TX, int VEC, int CPL>
DenseKernel dense_kernel() {
  constexpr int R = VEC * CPL >= 32 ? 1 : VEC * CPL >= 16 ? 2 : 4;
  return {gate_grad_dense_kernel<TX, VEC, CPL, R>, R};
}
template <typename TX, int VEC>
DenseKernel dense_kernel_for(int cpl) {
  if constexpr (VEC == 8)
    return cpl <= 1 ? dense_kernel<TX, 8, 1>() : cpl <= 2 ? dense_kernel<TX, 8, 2>() : dense_kernel<TX, 8, 4>();
  else if constexpr (VEC == 4)
    return cpl <= 1 ? dense_kernel<TX, 4, 1>() : cpl <= 2 ? dense_kernel<TX, 4, 2>() : dense_kernel<TX, 4, 8>();
  else
    return cpl <= 2 ? dense_kernel<TX, 1, 2>() : cpl <= 8 ? dense_kernel<TX, 1, 8>() : dense_kernel<TX, 1, 32>();
}

template <typename TX>
moe_status_t launch_gate_grad(GateGradArgs a, cudaStream_t st) {
  constexpr int kWide = 16 / sizeof(TX);
  const bool dense = !a.renorm && !a.sigmoid;
  const bool wide = a.E % kWide == 0 && moe_host::aligned16(a.gx) && (!dense || moe_host::aligned16(a.x));
  const int chunks = wide ? a.E / kWide : a.E;
  a.kp_log2 = 0;
  while ((1 << a.kp_log2) < a.k) ++a.kp_log2;
  a.g_log2 = 0;
  while ((1 << a.g_log2) < chunks && a.g_log2 < 5) ++a.g_log2;
  const int cpl = (chunks + 31) / 32;
  int rows = 32 >> (dense ? a.g_log2 : a.kp_log2);
  GateKernel kernel;
  if (dense) {
    const DenseKernel d = wide ? dense_kernel_for<TX, kWide>(cpl) : dense_kernel_for<TX, 1>(cpl);
    kernel = d.kernel;
    // row groups a warp: as many as its registers hold, where that leaves every SM 16 warps and the rows' slots fill
    // the lanes at most twice
    const int sms = moe_host::sm_count();
    if (sms <= 0) return MOE_ERR_CUDA;
    a.iters = 1;
    while (a.iters < d.most && 2 * a.iters * rows <= (kDenseRows >> a.kp_log2) &&
           a.T >= int64_t{2} * a.iters * rows * sms * 16)
      a.iters *= 2;
    rows *= a.iters;
  } else {
    kernel = wide ? gate_grad_sparse_kernel<TX, kWide> : gate_grad_sparse_kernel<TX, 1>;
  }
  a.sums = (rows * a.E + 3) & ~3;  // where dense at most 1024: rows E <= 32 CPL VEC iters
  const size_t smem = dense ? kGateWarps * a.sums * sizeof(float) : 0;
  const int64_t batches = (a.T + rows - 1) / rows;
  return moe_host::launch_pdl(kernel, dim3(static_cast<unsigned>((batches + kGateWarps - 1) / kGateWarps)),
                              dim3(kGateWarps * 32), smem, st, a);
}

}  // namespace

extern "C" moe_status_t moe_combine_backward(const void* grad_out, const void* expert_out, const float* topk_weights,
                                             const int32_t* inv_perm, const int32_t* sorted_token_ids,
                                             const int32_t* num_tokens_post_pad, int64_t T, int32_t k, int32_t H,
                                             int64_t capacity, uint32_t flags, void* grad_expert_out,
                                             float* grad_topk_weights, int32_t* device_status, void* stream) {
  if (T < 0 || H < 1 || k < 1 || capacity < 0) return MOE_ERR_INVALID_ARG;
  if (k > 32) return MOE_ERR_UNSUPPORTED;
  if ((H % 8) != 0) return MOE_ERR_INVALID_ARG;
  if ((flags & ~MOE_GATHER_ZERO_PAD) != 0u) return MOE_ERR_INVALID_ARG;
  if (T > (int64_t{1} << 40) || T * k >= (int64_t{1} << 30) || capacity >= (int64_t{1} << 31))
    return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;  // no slots, and with them no blocks to pad
  if (grad_expert_out == nullptr && grad_topk_weights == nullptr) return MOE_ERR_INVALID_ARG;
  const bool zero_pad = (flags & MOE_GATHER_ZERO_PAD) != 0u;
  if (zero_pad && (sorted_token_ids == nullptr || num_tokens_post_pad == nullptr || grad_expert_out == nullptr))
    return MOE_ERR_INVALID_ARG;
  if (grad_out == nullptr || topk_weights == nullptr || inv_perm == nullptr) return MOE_ERR_INVALID_ARG;
  if (capacity > 0 && grad_topk_weights != nullptr && expert_out == nullptr) return MOE_ERR_INVALID_ARG;
  if (!moe_host::aligned16(grad_out) || !moe_host::aligned16(expert_out) || !moe_host::aligned16(grad_expert_out))
    return MOE_ERR_INVALID_ARG;
  CombineGradArgs a{};
  a.gout = static_cast<const uint4*>(grad_out);
  a.y = static_cast<const uint4*>(expert_out);
  a.w = topk_weights;
  a.inv_perm = inv_perm;
  a.slots = T * k;
  a.k = k;
  a.nv = H / 8;
  a.capacity = capacity;
  a.gy = static_cast<uint4*>(grad_expert_out);
  a.gw = grad_topk_weights;
  a.sorted_ids = zero_pad ? sorted_token_ids : nullptr;
  a.n_pad = num_tokens_post_pad;
  a.slot_blocks = (a.slots + kWarps - 1) / kWarps;
  a.status = device_status;
  int64_t grid = a.slot_blocks;
  if (zero_pad) {
    const int sms = moe_host::sm_count();
    if (sms <= 0) return MOE_ERR_CUDA;
    a.pad_rows = capacity < int64_t{64} * sms ? 1 : 2;
    grid += (capacity + kWarps * a.pad_rows - 1) / (kWarps * a.pad_rows);
  }
  return moe_host::launch_pdl(combine_grad_kernel, dim3(static_cast<unsigned>(grid)), dim3(kWarps * 32), 0,
                              static_cast<cudaStream_t>(stream), a);
}

extern "C" moe_status_t moe_topk_softmax_backward(const float* grad_topk_weights, const void* logits,
                                                  moe_dtype_t dtype, const float* topk_weights,
                                                  const int32_t* topk_ids, int64_t T, int32_t E, int32_t k,
                                                  uint32_t flags, void* grad_logits, int32_t* device_status,
                                                  void* stream) {
  if (T < 0 || E < 1 || k < 1 || k > E) return MOE_ERR_INVALID_ARG;
  if (dtype != MOE_DTYPE_F32 && dtype != MOE_DTYPE_BF16) return MOE_ERR_INVALID_ARG;
  if ((flags & ~(MOE_RENORMALIZE | MOE_SCORING_SIGMOID)) != 0u) return MOE_ERR_INVALID_ARG;
  if (E > 1024 || k > 32) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (T > (int64_t{1} << 30)) return MOE_ERR_INVALID_ARG;
  GateGradArgs a{};
  a.renorm = (flags & MOE_RENORMALIZE) != 0u;
  a.sigmoid = (flags & MOE_SCORING_SIGMOID) != 0u;
  if (grad_topk_weights == nullptr || topk_weights == nullptr || topk_ids == nullptr || grad_logits == nullptr)
    return MOE_ERR_INVALID_ARG;
  if (logits == nullptr && !(a.renorm && !a.sigmoid)) return MOE_ERR_INVALID_ARG;
  const uintptr_t elem = dtype == MOE_DTYPE_BF16 ? 2 : 4;
  if (reinterpret_cast<uintptr_t>(logits) % elem != 0 || reinterpret_cast<uintptr_t>(grad_logits) % elem != 0)
    return MOE_ERR_INVALID_ARG;
  a.gw = grad_topk_weights;
  a.x = logits;
  a.w = topk_weights;
  a.ids = topk_ids;
  a.T = T;
  a.E = E;
  a.k = k;
  a.gx = grad_logits;
  a.status = device_status;
  return dtype == MOE_DTYPE_BF16 ? launch_gate_grad<__nv_bfloat16>(a, static_cast<cudaStream_t>(stream))
                                 : launch_gate_grad<float>(a, static_cast<cudaStream_t>(stream));
}

extern "C" moe_status_t moe_gather_backward(const void* grad_permuted, const int32_t* inv_perm, int64_t T, int32_t k,
                                            int32_t H, int64_t capacity, void* grad_hidden, int32_t* device_status,
                                            void* stream) {
  if (T < 0 || H < 1 || k < 1 || capacity < 0) return MOE_ERR_INVALID_ARG;
  if (k > 32) return MOE_ERR_UNSUPPORTED;
  if ((H % 8) != 0) return MOE_ERR_INVALID_ARG;
  if (T > (int64_t{1} << 40) || T * k >= (int64_t{1} << 30) || capacity >= (int64_t{1} << 31))
    return MOE_ERR_INVALID_ARG;
  if (T * H > (int64_t{1} << 40)) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (inv_perm == nullptr || grad_hidden == nullptr || (capacity > 0 && grad_permuted == nullptr))
    return MOE_ERR_INVALID_ARG;
  if (!moe_host::aligned16(grad_permuted) || !moe_host::aligned16(grad_hidden)) return MOE_ERR_INVALID_ARG;
  const int nv = H / 8, segs = (nv + 32 * kSumVecs - 1) / (32 * kSumVecs);
  // tokens a warp: up to four, as far as that leaves every SM 64 warps
  const int sms = moe_host::sm_count();
  if (sms <= 0) return MOE_ERR_CUDA;
  int per = 1;
  while (per < 4 && 2 * per * k <= 32 && T * segs >= int64_t{2} * per * sms * 64) per *= 2;
  const int64_t grid = ((T + per - 1) / per * segs + kWarps - 1) / kWarps;  // (T segs <= T H / 512 + T: below 2^29)
  const auto kernel = per == 1 ? gather_grad_kernel<4, true> : gather_grad_kernel<2, false>;
  return moe_host::launch_pdl(kernel, dim3(static_cast<unsigned>(grid)), dim3(kWarps * 32), 0,
                              static_cast<cudaStream_t>(stream), static_cast<const uint4*>(grad_permuted), inv_perm, T,
                              static_cast<int>(k), per, nv, segs, capacity, static_cast<uint4*>(grad_hidden),
                              device_status);
}
