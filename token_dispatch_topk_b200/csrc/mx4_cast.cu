// mx4_cast.cu -- rows to microscaled 4-bit floating point and back, and the permute-gather in that format.
//
// Format (the OCP Microscaling Formats specification v1.0, MXFP4): 32 consecutive elements of a row share one
// power-of-two scale 2^s, kept as the byte s + 127 (E8M0); an element is an E2M1 code c (sign, two exponent bits,
// one mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6) and stands for c 2^s.
//   s = clamp(floor(log2(max |x|)) - 2, -127, 127), c = x 2^-s to nearest, ties to the even code, beyond 6 to 6.
// 2^-s is exact and x 2^-s is exact in fp32 (or below the smallest code's half), so each element is rounded once.
// A block that holds an infinity or a NaN gets the scale byte 255, which stands for NaN, and zero codes: the block
// reads back as NaN.  A block of zeros gets scale byte 0.
//
// Layout: codes [rows, K/2], the even element in the low half of the byte; scales [ceil(K/128), rows, 4]: the bytes
// of the four blocks of a 128-element chunk side by side, rows next to each other, which is how the product's tiles
// read them (32 lanes, 128 bytes).  Blocks past K in the last chunk hold 127 (a scale of 1).
//
// All three kernels are bandwidth-bound: 2 K bytes a row on the wide side, 17/32 K on the narrow one.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"

namespace {

constexpr int kCastThreads = 256;

// Eight bf16 of a lane (four lanes hold a block): the block's scale byte and the lane's eight codes.
__device__ __forceinline__ uint32_t quantize8(const uint4& v, uint32_t& scale_byte) {
  const uint32_t a0 = v.x & 0x7fff7fffu, a1 = v.y & 0x7fff7fffu, a2 = v.z & 0x7fff7fffu, a3 = v.w & 0x7fff7fffu;
  uint32_t m = __vmaxu2(__vmaxu2(a0, a1), __vmaxu2(a2, a3));  // magnitudes order as integers, NaN above infinity
  m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 2));
  const uint32_t top = max(m & 0xffffu, m >> 16);
  const uint32_t field = top >> 7;  // biased exponent: floor(log2) + 127 where normal; s + 127 = field - 2, at least 0
  if (field == 255u) {
    scale_byte = 255u;
    return 0u;
  }
  scale_byte = field > 2u ? field - 2u : 0u;
  const float f = __uint_as_float((254u - scale_byte) << 23);  // 2^-s, normal: the byte is at most 252
  // pairs of fp32 (low half, high half of a word), scaled two at a time
  const uint64_t ff = moe::f32x2(f, f);
  uint32_t codes;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t.reg .b64 p0, p1, p2, p3;\n\t.reg .f32 l0, h0, l1, h1, l2, h2, l3, h3;\n\t"
      "mul.rn.f32x2 p0, %1, %5;\n\tmul.rn.f32x2 p1, %2, %5;\n\tmul.rn.f32x2 p2, %3, %5;\n\tmul.rn.f32x2 p3, %4, %5;\n\t"
      "mov.b64 {l0, h0}, p0;\n\tmov.b64 {l1, h1}, p1;\n\tmov.b64 {l2, h2}, p2;\n\tmov.b64 {l3, h3}, p3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, h0, l0;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, h1, l1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, h2, l2;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, h3, l3;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(codes)
      : "l"(moe::f32x2(moe::bf16_lo(v.x), moe::bf16_hi(v.x))), "l"(moe::f32x2(moe::bf16_lo(v.y), moe::bf16_hi(v.y))),
        "l"(moe::f32x2(moe::bf16_lo(v.z), moe::bf16_hi(v.z))), "l"(moe::f32x2(moe::bf16_lo(v.w), moe::bf16_hi(v.w))),
        "l"(ff));
  return codes;
}

// Four chunks' scale bytes to words.  Half a warp holds a chunk, four lanes a block: byte u of `bytes` is the lane's
// block's scale in chunk u.  The result, in the lanes of block b: the word (its four blocks' bytes) of chunk b.  A
// transpose of four by four bytes, two shuffles.
__device__ __forceinline__ uint32_t chunk_words(uint32_t bytes) {
  const int b = (threadIdx.x >> 2) & 3;
  uint32_t o = __shfl_xor_sync(0xffffffffu, bytes, 4);
  bytes = (b & 1) ? __byte_perm(bytes, o, 0x3715) : __byte_perm(bytes, o, 0x6240);
  o = __shfl_xor_sync(0xffffffffu, bytes, 8);
  return (b & 2) ? __byte_perm(bytes, o, 0x3276) : __byte_perm(bytes, o, 0x5410);
}

// A warp takes one 128-element chunk of kRowsPerWarp consecutive rows, half a warp a row at a time: every load of the
// eight rows is in flight before the first is used, and the rows' scale words leave as one 32-byte sector.
constexpr int kRowsPerWarp = 8;

__device__ __forceinline__ bool warp_chunk(int64_t rows, int chunks, int64_t& row0, int& chunk) {
  const int64_t wid = (static_cast<int64_t>(blockIdx.x) * kCastThreads + threadIdx.x) >> 5;
  const int64_t group = wid / chunks;
  chunk = static_cast<int>(wid - group * chunks);
  row0 = group * kRowsPerWarp;
  return row0 < rows;
}

// (full occupancy: 32 registers a thread, 178 us against 194 at 39; then 152 with fewer instructions an element)
__global__ void __launch_bounds__(kCastThreads, 8)
quantize_kernel(const uint4* __restrict__ x, int64_t rows, const int32_t* __restrict__ num_rows, int nv, int chunks,
                uint32_t* __restrict__ codes, uint32_t* __restrict__ scales) {
  moe::pdl_launch_dependents();
  moe::pdl_wait();
  const int lane = threadIdx.x & 31;
  int64_t row0;
  int c;
  const int64_t end = num_rows == nullptr || num_rows[0] > rows ? rows : num_rows[0];
  if (!warp_chunk(rows, chunks, row0, c) || row0 >= end) return;
  const int v = c * 16 + (lane & 15);
  const int64_t row = row0 + (lane >> 4);
  const int left = v >= nv ? 0 : end - row < kRowsPerWarp ? static_cast<int>(end - row) : kRowsPerWarp;
  const uint4* src = x + row * nv + v;
  uint32_t* dst = codes + row * nv + v;
  uint4 in[kRowsPerWarp / 2];
#pragma unroll
  for (int u = 0; u < kRowsPerWarp / 2; ++u) {
    in[u] = make_uint4(0u, 0u, 0u, 0u);
    if (2 * u < left) in[u] = moe::ld_stream(src);
    src += 2 * nv;
  }
  uint32_t bytes = 0u;
#pragma unroll
  for (int u = 0; u < kRowsPerWarp / 2; ++u) {
    uint32_t sb;
    const uint32_t q = quantize8(in[u], sb);
    if (2 * u < left) *dst = q;
    dst += 2 * nv;
    bytes |= sb << (8 * u);
  }
  if (v >= nv) bytes = 0x7f7f7f7fu;  // blocks past K
  const uint32_t word = chunk_words(bytes);
  const int64_t to = row + 2 * ((lane >> 2) & 3);  // the row whose word this lane holds
  if ((lane & 3) == 0 && to < end) scales[static_cast<int64_t>(c) * rows + to] = word;
}

// The permute-gather: a token's row is read and quantised once and written to each of its local rows.
// A warp takes kPieces pieces of 256 elements, all in flight together.
constexpr int kPieces = 4;  // (chunk_words takes four)
__global__ void __launch_bounds__(kCastThreads, 6)
gather_mx4_kernel(const uint4* __restrict__ x, int64_t T, int nv, int segs, int k,
                  const int32_t* __restrict__ inv_perm, int64_t capacity, uint32_t* __restrict__ codes,
                  uint32_t* __restrict__ scales, int32_t* status) {
  moe::pdl_launch_dependents();
  moe::pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t wid = (static_cast<int64_t>(blockIdx.x) * kCastThreads + threadIdx.x) >> 5;
  const int64_t t = wid / segs;
  if (t >= T) return;
  int r = -1;
  if (lane < k) {
    r = inv_perm[t * k + lane];
    if (r < -1 || static_cast<int64_t>(r) >= capacity) {
      moe::record_status(status, MOE_ERR_BAD_ROW);
      r = -1;
    }
  }
  const unsigned local = __ballot_sync(0xffffffffu, r >= 0);
  if (local == 0u) return;  // no local slot: the row is not read
  const int v0 = static_cast<int>(wid - t * segs) * (32 * kPieces) + lane;
  uint4 in[kPieces];
#pragma unroll
  for (int u = 0; u < kPieces; ++u) {
    in[u] = make_uint4(0u, 0u, 0u, 0u);
    if (v0 + 32 * u < nv) in[u] = moe::ld_stream(x + t * nv + v0 + 32 * u);
  }
  uint32_t q[kPieces], bytes = 0u;
#pragma unroll
  for (int u = 0; u < kPieces; ++u) {
    uint32_t sb;
    q[u] = quantize8(in[u], sb);
    bytes |= (v0 + 32 * u < nv ? sb : 127u) << (8 * u);
  }
  const uint32_t word = chunk_words(bytes);
  const int chunk = (v0 - lane) / 16 + 2 * ((lane >> 2) & 3) + (lane >> 4);  // the chunk whose word this lane holds
  const bool has_word = (lane & 3) == 0 && chunk * 16 < nv;
  for (unsigned left = local; left != 0u; left &= left - 1u) {
    const int64_t dst = __shfl_sync(0xffffffffu, r, __ffs(left) - 1);
    uint32_t* to = codes + dst * nv + v0;
#pragma unroll
    for (int u = 0; u < kPieces; ++u)
      if (v0 + 32 * u < nv) to[32 * u] = q[u];
    if (has_word) scales[static_cast<int64_t>(chunk) * capacity + dst] = word;
  }
}

// Eight codes and their block's scale byte -> eight bf16 (exact where the value is representable).
__device__ __forceinline__ uint4 dequantize8(uint32_t c, uint32_t byte) {
  // 2^(byte - 127): below a byte of 1 a subnormal, 255 NaN
  const float f = byte == 255u ? __uint_as_float(0x7fc00000u)
                               : byte == 0u ? __uint_as_float(0x00400000u) : __uint_as_float(byte << 23);
  uint32_t h[4];
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(c));
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo, hi;
    asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, u;\n\t}"
        : "=f"(lo), "=f"(hi)
        : "r"(h[i]));
    o[i] = moe::pack_bf16x2(lo * f, hi * f);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

__global__ void __launch_bounds__(kCastThreads)
dequantize_kernel(const uint32_t* __restrict__ codes, const uint8_t* __restrict__ scales, int64_t rows, int nv,
                  int chunks, uint4* __restrict__ out) {
  moe::pdl_launch_dependents();
  moe::pdl_wait();
  const int lane = threadIdx.x & 31;
  int64_t row0;
  int c;
  if (!warp_chunk(rows, chunks, row0, c)) return;
  const int v = c * 16 + (lane & 15);
  const int64_t row = row0 + (lane >> 4);
  uint32_t q[kRowsPerWarp / 2], byte[kRowsPerWarp / 2];
#pragma unroll
  for (int u = 0; u < kRowsPerWarp / 2; ++u) {
    q[u] = byte[u] = 0u;
    if (v < nv && row + 2 * u < rows) {
      q[u] = __ldcs(codes + (row + 2 * u) * nv + v);
      byte[u] = scales[(static_cast<int64_t>(c) * rows + row + 2 * u) * 4 + ((v >> 2) & 3)];
    }
  }
#pragma unroll
  for (int u = 0; u < kRowsPerWarp / 2; ++u)
    if (v < nv && row + 2 * u < rows) moe::st_stream(out + (row + 2 * u) * nv + v, dequantize8(q[u], byte[u]));
}

// Sizes of a matrix in the format: K in blocks of 32.  Beyond kMaxElements a call is refused as unsupported.
constexpr int64_t kMaxElements = int64_t{1} << 41;
bool mx4_sizes_ok(int64_t rows, int32_t K) {
  return rows >= 0 && rows < (int64_t{1} << 31) && K >= 32 && (K % 32) == 0 && K <= (1 << 20);
}

// CTAs for as many warps: below 2^30, as a warp takes 1024 elements or the rest of a row, and rows stay below 2^31
unsigned cast_grid(int64_t warps) {
  return static_cast<unsigned>((warps + kCastThreads / 32 - 1) / (kCastThreads / 32));
}

}  // namespace

extern "C" moe_status_t moe_quantize_mx4(const void* x, int64_t rows, int32_t K, const int32_t* num_rows,
                                         void* codes, void* scales, void* stream) {
  if (!mx4_sizes_ok(rows, K)) return MOE_ERR_INVALID_ARG;
  if (rows * K > kMaxElements) return MOE_ERR_UNSUPPORTED;
  if (rows == 0) return MOE_OK;
  if (x == nullptr || codes == nullptr || scales == nullptr) return MOE_ERR_INVALID_ARG;
  if (!moe_host::aligned16(x) || !moe_host::aligned16(codes) || !moe_host::aligned16(scales))
    return MOE_ERR_INVALID_ARG;
  const int nv = K / 8, chunks = (K + 127) / 128;
  const unsigned grid = cast_grid((rows + kRowsPerWarp - 1) / kRowsPerWarp * chunks);
  return moe_host::launch_pdl(quantize_kernel, dim3(grid), dim3(kCastThreads), 0, static_cast<cudaStream_t>(stream),
                              static_cast<const uint4*>(x), rows, num_rows, nv, chunks, static_cast<uint32_t*>(codes),
                              static_cast<uint32_t*>(scales));
}

extern "C" moe_status_t moe_dequantize_mx4(const void* codes, const void* scales, int64_t rows, int32_t K, void* out,
                                           void* stream) {
  if (!mx4_sizes_ok(rows, K)) return MOE_ERR_INVALID_ARG;
  if (rows * K > kMaxElements) return MOE_ERR_UNSUPPORTED;
  if (rows == 0) return MOE_OK;
  if (out == nullptr || codes == nullptr || scales == nullptr) return MOE_ERR_INVALID_ARG;
  if (!moe_host::aligned16(out) || !moe_host::aligned16(codes) || !moe_host::aligned16(scales))
    return MOE_ERR_INVALID_ARG;
  const int nv = K / 8, chunks = (K + 127) / 128;
  const unsigned grid = cast_grid((rows + kRowsPerWarp - 1) / kRowsPerWarp * chunks);
  return moe_host::launch_pdl(dequantize_kernel, dim3(grid), dim3(kCastThreads), 0,
                              static_cast<cudaStream_t>(stream), static_cast<const uint32_t*>(codes),
                              static_cast<const uint8_t*>(scales), rows, nv, chunks, static_cast<uint4*>(out));
}

extern "C" moe_status_t moe_gather_mx4(const void* hidden, int64_t T, int32_t H, int32_t k, const int32_t* inv_perm,
                                       int64_t capacity, void* codes, void* scales, int32_t* device_status,
                                       void* stream) {
  if (T < 0 || k < 1 || !mx4_sizes_ok(capacity, H)) return MOE_ERR_INVALID_ARG;
  if (k > 32) return MOE_ERR_UNSUPPORTED;
  if (T > (int64_t{1} << 40) || T * k >= (int64_t{1} << 30)) return MOE_ERR_INVALID_ARG;
  if (T * H > kMaxElements || capacity * H > kMaxElements) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (hidden == nullptr || inv_perm == nullptr) return MOE_ERR_INVALID_ARG;
  if (capacity > 0 && (codes == nullptr || scales == nullptr)) return MOE_ERR_INVALID_ARG;
  if (!moe_host::aligned16(hidden) || !moe_host::aligned16(codes) || !moe_host::aligned16(scales))
    return MOE_ERR_INVALID_ARG;
  const int nv = H / 8, segs = (nv + 32 * kPieces - 1) / (32 * kPieces);
  const unsigned grid = cast_grid(T * segs);
  return moe_host::launch_pdl(gather_mx4_kernel, dim3(grid), dim3(kCastThreads), 0, static_cast<cudaStream_t>(stream),
                              static_cast<const uint4*>(hidden), T, nv, segs, static_cast<int>(k), inv_perm, capacity,
                              static_cast<uint32_t*>(codes), static_cast<uint32_t*>(scales), device_status);
}
