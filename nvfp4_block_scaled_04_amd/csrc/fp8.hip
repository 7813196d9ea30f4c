// BF16 -> FP8 block quantisers (gfx950).
//
// FP8 here is OCP E4M3 with one fp32 scale per 128 columns of a row
// (activations) or per 128 x 128 block (weights).  With b = max(amax of the
// block, 2^-100), every step in fp32 rounded to nearest even:
//   scale = b / 448,  r = 448 / b,  code = E4M3(x * r).
// |x * r| <= 448 * (1 + 2^-23), which rounds to at most 448, so no clamp is
// needed; the 2^-100 floor keeps r finite and gives an all-zero block codes 0
// and a positive scale.  v_cvt_pk_fp8_f32 rounds to nearest, ties to even.  fmaxf
// passes over a NaN, so one bad value keeps its NaN code to itself; an infinity
// gives an infinite scale and r = 0.
//
// All three are bound by HBM: rows read 2 and write 1 + 4/128 bytes per
// element, SwiGLU reads 4, weights read 2 and write 1.  Sixteen lanes hold
// one 128-column block, 16 bytes (8 BF16) each, so its maximum is four lane
// exchanges and nothing is read twice.  Measured: 8192 rows of 7168 29 us
// (178 MB: 6.1 TB/s); SwiGLU of 65536 x 2048 122 to 126 us (5.4 TB/s), of
// 2048 x 2048 6.2 to 6.6 us (latency); weights 32 x 4096 x 7168 520 us (2.8 GB:
// 5.4 TB/s).
#include "internal.hpp"
#include "device.hpp"

namespace nvfp4 {

namespace {

constexpr float kFp8Max = 448.0f;
constexpr float kFp8Floor = 7.888609052210118e-31f;   // 2^-100
constexpr int kQThreads = 256;
constexpr int kQGroups = kQThreads / 16;              // blocks of 128 per pass of a workgroup

__device__ __forceinline__ float amax8(const float (&x)[8]) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(x[i]));
  return m;
}

// largest over the 16 lanes that hold one 128-column block
__device__ __forceinline__ float max16(float m) {
#pragma unroll
  for (int o = 8; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
  return m;
}

__device__ __forceinline__ uint2 encode8(const float (&x)[8], float r) {
#pragma clang fp contract(off)
  int lo = 0, hi = 0;
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[0] * r, x[1] * r, lo, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[2] * r, x[3] * r, lo, true);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(x[4] * r, x[5] * r, hi, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(x[6] * r, x[7] * r, hi, true);
  return make_uint2((uint32_t)lo, (uint32_t)hi);
}

// silu(g) * u = (g / 4) / ((1 + exp(-g)) / 4) * u within 2^-21 of itself, far
// below the codes' 2^-4.  exp(-g) is 2^t times 1 + lo ln 2 with t + lo = -g log2 e
// (lo: what t's rounding and the constant's leave); the quarter keeps the
// reciprocal a normal number up to the largest finite exp(-g).  g beyond +-100
// gives g or 0, -inf and NaN give NaN, as the formula does.  The hardware's exp2
// and reciprocal (2^-23 each) without the library's exp and a full division,
// half the instructions, which bound large calls (65536 x 2048: 148 us with them, 129 without).
__device__ __forceinline__ float swiglu(float g, float u) {
#pragma clang fp contract(off)
  constexpr float kLog2e = 1.44269502e+00f, kLog2eLo = 1.92596299e-08f, kLn2 = 0.693147181f;
  const float c = __builtin_amdgcn_fmed3f(g, -100.0f, 100.0f);
  const float t = c * -kLog2e;
  const float lo = fmaf(c, -kLog2eLo, fmaf(c, -kLog2e, -t));
  const float d = fmaf(__builtin_amdgcn_exp2f(t), fmaf(lo, 0.25f * kLn2, 0.25f), 0.25f);
  return 0.25f * g * __builtin_amdgcn_rcpf(d) * u;
}
__device__ __forceinline__ void swiglu8(const uint4& gv, const uint4& uv, float (&h)[8]) {
  float g[8], u[8];
  unpack8(gv, g);
  unpack8(uv, u);
#pragma unroll
  for (int i = 0; i < 8; ++i) h[i] = swiglu(g[i], u[i]);
}

// One lane group per (ROWS rows, 128-column block).  SWIGLU: x rows hold
// [gate | up], each cols wide.
template <bool SWIGLU, int ROWS>
__global__ __launch_bounds__(kQThreads) void fp8_rows_kernel(
    const uint16_t* __restrict__ x, int64_t rows, int cols, int64_t ld_x, int kblocks,
    const int32_t* __restrict__ n_rows, uint8_t* __restrict__ q, float* __restrict__ sf) {
  if (n_rows) {
    const int64_t n = n_rows[0];
    rows = n < rows ? n : rows;
  }
  const uint32_t unit = row_workgroup() * kQGroups + (threadIdx.x >> 4);
  const uint32_t chunk = unit / (uint32_t)kblocks;
  const int kb = (int)(unit - chunk * (uint32_t)kblocks);
  const int64_t row0 = (int64_t)chunk * ROWS;
  const int l = threadIdx.x & 15;
  const int col = kb * 128 + l * 8;
  const bool in = col < cols;
  uint4 a[ROWS], b[ROWS];
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    a[i] = make_uint4(0, 0, 0, 0);
    b[i] = make_uint4(0, 0, 0, 0);
    if (in && row0 + i < rows) {
      const uint16_t* src = x + (row0 + i) * ld_x + col;
      a[i] = *reinterpret_cast<const uint4*>(src);
      if constexpr (SWIGLU) b[i] = *reinterpret_cast<const uint4*>(src + cols);
    }
  }
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    float v[8];
    if constexpr (SWIGLU) swiglu8(a[i], b[i], v);
    else unpack8(a[i], v);
    const float m = fmaxf(max16(amax8(v)), kFp8Floor);
    if (row0 + i < rows) {
      if (in) *reinterpret_cast<uint2*>(q + (row0 + i) * cols + col) = encode8(v, kFp8Max / m);
      if (l == 0) sf[(row0 + i) * kblocks + kb] = m / kFp8Max;
    }
  }
}

// One workgroup per 128 x 128 block: 16 rows per pass, eight passes in registers.
__global__ __launch_bounds__(kQThreads) void fp8_weight_kernel(
    const uint16_t* __restrict__ w, int64_t rows, int64_t cols, int nblocks, int kblocks, uint32_t units,
    uint8_t* __restrict__ q, float* __restrict__ sf) {
  const uint32_t unit = row_workgroup();
  if (unit >= units) return;
  const uint32_t t = unit / (uint32_t)kblocks;
  const int kb = (int)(unit - t * (uint32_t)kblocks);
  const uint32_t g = t / (uint32_t)nblocks;
  const int nb = (int)(t - g * (uint32_t)nblocks);
  const int l = threadIdx.x & 15, rr = threadIdx.x >> 4;
  const int64_t col = kb * 128 + l * 8;
  const int64_t r0 = (int64_t)nb * 128 + rr;
  const int64_t base = (int64_t)g * rows * cols;
  uint4 a[8];
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t row = r0 + 16 * i;
    a[i] = make_uint4(0, 0, 0, 0);
    if (col < cols && row < rows) a[i] = *reinterpret_cast<const uint4*>(w + base + row * cols + col);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float v[8];
    unpack8(a[i], v);
    m = fmaxf(m, amax8(v));
  }
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
  __shared__ float part[kQThreads / 64];
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = m;
  __syncthreads();
  m = fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3]));
  m = fmaxf(m, kFp8Floor);
  const float r = kFp8Max / m;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t row = r0 + 16 * i;
    float v[8];
    unpack8(a[i], v);
    if (col < cols && row < rows) *reinterpret_cast<uint2*>(q + base + row * cols + col) = encode8(v, r);
  }
  if (threadIdx.x == 0) sf[unit] = m / kFp8Max;
}

}  // namespace

template <bool SWIGLU, int ROWS>
static void rows_launch(const void* x, int64_t rows, int64_t cols, int64_t ld_x, int kblocks,
                        const int32_t* n_rows, uint8_t* q, float* sf, hipStream_t stream) {
  const int64_t units = (rows + ROWS - 1) / ROWS * kblocks;
  fp8_rows_kernel<SWIGLU, ROWS><<<grid_rows((units + kQGroups - 1) / kQGroups), kQThreads, 0, stream>>>(
      static_cast<const uint16_t*>(x), rows, (int)cols, ld_x, kblocks, n_rows, q, sf);
}

hipError_t launch_fp8_rows(bool swiglu, const void* x, int64_t rows, int64_t cols, int64_t ld_x,
                           const int32_t* n_rows, uint8_t* q, float* sf, hipStream_t stream) {
  if (rows == 0) return hipSuccess;
  const int kblocks = (int)((cols + 127) / 128);
  // rows: four a lane group where that still gives every CU several workgroups
  // (8192 x 7168: 29.7 us, one row 32.7; 1024 x 7168: 6.8, one row 6.3).  SwiGLU
  // loads twice as much a row: one (65536 x 2048: 126 us, four rows 129; 2048 x
  // 2048: 6.2, four rows 7.7).
  if (swiglu) rows_launch<true, 1>(x, rows, cols, ld_x, kblocks, n_rows, q, sf, stream);
  else if (rows * kblocks < (1 << 16)) rows_launch<false, 1>(x, rows, cols, ld_x, kblocks, n_rows, q, sf, stream);
  else rows_launch<false, 4>(x, rows, cols, ld_x, kblocks, n_rows, q, sf, stream);
  return hipGetLastError();
}

hipError_t launch_fp8_weight(const void* w, int64_t groups, int64_t rows, int64_t cols, uint8_t* q,
                             float* sf, hipStream_t stream) {
  if (groups == 0 || rows == 0) return hipSuccess;
  const int nblocks = (int)((rows + 127) / 128), kblocks = (int)((cols + 127) / 128);
  const int64_t units = groups * nblocks * kblocks;
  fp8_weight_kernel<<<grid_rows(units), kQThreads, 0, stream>>>(static_cast<const uint16_t*>(w), rows, cols, nblocks,
                                                                kblocks, (uint32_t)units, q, sf);
  return hipGetLastError();
}

}  // namespace nvfp4
