// route_grads.cu -- gradients of the routing layer: of the weighted combine and of the gating.
// (The gradient of the permute-gather is the combine with unit weights: gather_combine.cu.)
//
// Combine, out[t] = sum_j w[t,j] y[r(t,j)], with grad_out = dL/dout:
//   dL/dy[r(t,j)] = w[t,j] grad_out[t]        one rounding to bf16
//   dL/dw[t,j]    = sum_h grad_out[t,h] y[r(t,j),h]   fp32
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

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
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
  int32_t* status;
};

constexpr int kPadRowsPerCta = 256;

// One warp per slot; the k slots of a token sit in neighbouring warps, so its gradient row comes from DRAM once
// and from L1 / L2 after that.  Bandwidth-bound: a row of y in, a row of gy out, 16 bytes a lane and kUnroll
// vectors in flight.
__global__ void __launch_bounds__(kWarps * 32) combine_grad_kernel(CombineGradArgs a) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  moe::pdl_launch_dependents();
  moe::pdl_wait();  // every input may come from the previous kernel
  if (blockIdx.x >= a.slot_blocks) {  // +0 into the pad rows below N_pad (their sorted id is T*k)
    const int64_t p0 = (static_cast<int64_t>(blockIdx.x) - a.slot_blocks) * kPadRowsPerCta;
    int64_t end = a.n_pad[0];
    if (end > a.capacity) end = a.capacity;
    for (int64_t p = p0 + warp; p < p0 + kPadRowsPerCta && p < end; p += kWarps) {
      if (a.sorted_ids[p] != static_cast<int32_t>(a.slots)) continue;
      for (int v = lane; v < a.nv; v += 32) moe::st_plain(a.gy + p * a.nv + v, make_uint4(0u, 0u, 0u, 0u));
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

// ---------------------------------------------------------------------------------------------- gating --
constexpr int kGateWarps = 8;

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

struct GateGradArgs {
  const float* gw;      // [T, k] incoming
  const void* x;        // [T, E]
  const float* w;       // [T, k]
  const int32_t* ids;   // [T, k]
  int64_t T;
  int E, k;
  int renorm, sigmoid;
  void* gx;             // [T, E] out
  int32_t* status;
};

// One warp per row.  Lane j < k holds selected expert j; its value goes into the row's E fp32 sums in shared
// memory, which the warp then reads in order (for the dense softmax gradient with the recomputed probabilities).
template <typename TX>
__global__ void __launch_bounds__(kGateWarps * 32) gate_grad_kernel(GateGradArgs a) {
  extern __shared__ float s_rows[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float* row = s_rows + static_cast<size_t>(warp) * a.E;
  moe::pdl_launch_dependents();
  moe::pdl_wait();
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kGateWarps + warp;
  if (t >= a.T) return;
  const TX* x = static_cast<const TX*>(a.x) + t * a.E;
  TX* gx = static_cast<TX*>(a.gx) + t * a.E;
  for (int e = lane; e < a.E; e += 32) row[e] = 0.f;
  int id = -1;
  float g = 0.f, w = 0.f;
  if (lane < a.k) {
    id = a.ids[t * a.k + lane];
    g = a.gw[t * a.k + lane];
    w = a.w[t * a.k + lane];
    if (id < 0 || id >= a.E) {
      moe::record_status(a.status, MOE_ERR_BAD_EXPERT_ID);
      id = -1;
      g = w = 0.f;
    }
  }
  const float G = warp_sum(g * w);
  const bool dense = !a.renorm && !a.sigmoid;
  float v = dense ? g : a.renorm ? w * (g - G) : w * g;
  if (a.sigmoid) {
    const float xs = id >= 0 ? to_f32<TX>(x[id]) : 0.f;
    // all scores underflowed to 0: the weights are the constant 1/k
    const bool any = __any_sync(0xffffffffu, id >= 0 && expf(-xs) < INFINITY);
    v = any ? v / (1.f + expf(xs)) : 0.f;
  }
  __syncwarp();
  const unsigned same = __match_any_sync(0xffffffffu, id >= 0 ? id : -1 - lane);
  if (__any_sync(0xffffffffu, __popc(same) > 1)) {  // an expert named twice: add in slot order
    for (int j = 0; j < a.k; ++j) {
      const int ij = __shfl_sync(0xffffffffu, id, j);
      const float vj = __shfl_sync(0xffffffffu, v, j);
      if (lane == 0 && ij >= 0) row[ij] += vj;
    }
  } else if (id >= 0) {
    row[id] = v;
  }
  __syncwarp();
  if (dense) {
    float m = -INFINITY;
    for (int e = lane; e < a.E; e += 32) m = fmaxf(m, to_f32<TX>(x[e]));
    m = warp_max(m);
    float z = 0.f;
    for (int e = lane; e < a.E; e += 32) z += expf(to_f32<TX>(x[e]) - m);
    z = 1.f / warp_sum(z);
    for (int e = lane; e < a.E; e += 32) gx[e] = from_f32<TX>(expf(to_f32<TX>(x[e]) - m) * z * (row[e] - G));
  } else {
    for (int e = lane; e < a.E; e += 32) gx[e] = from_f32<TX>(row[e]);
  }
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
  if (grad_expert_out == nullptr && grad_topk_weights == nullptr) return MOE_ERR_INVALID_ARG;
  const bool zero_pad = (flags & MOE_GATHER_ZERO_PAD) != 0u;
  if (zero_pad && (sorted_token_ids == nullptr || num_tokens_post_pad == nullptr || grad_expert_out == nullptr))
    return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;  // no slots, and with them no blocks to pad
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
  const int64_t grid = a.slot_blocks + (zero_pad ? (capacity + kPadRowsPerCta - 1) / kPadRowsPerCta : 0);
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
  const int64_t grid = (T + kGateWarps - 1) / kGateWarps;
  const size_t smem = static_cast<size_t>(kGateWarps) * E * sizeof(float);  // <= 32 KB
  return moe_host::launch_pdl(dtype == MOE_DTYPE_BF16 ? gate_grad_kernel<__nv_bfloat16> : gate_grad_kernel<float>,
                              dim3(static_cast<unsigned>(grid)), dim3(kGateWarps * 32), smem,
                              static_cast<cudaStream_t>(stream), a);
}
