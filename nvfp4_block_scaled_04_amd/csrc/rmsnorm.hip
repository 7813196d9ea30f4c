// RMS norm with the residual's addition and outputs in BF16 and FP8, and its
// gradient (gfx950).
//
//   h = bf16(x + residual),  rstd = 1/sqrt(mean h^2 + eps),  v = h * rstd * w,
//   y = bf16(v);  FP8 codes and scales of v as fp8_quantize's (one scale per
//   128 columns).
// The norm is of the stored sum h, so that it can be made again from h.
//   g = dy * w, n = h * rstd:  dx = dh + rstd * (g - n * mean(g * n)),
//   dw = sum over rows of dy * n.
// Sums in fp32: a lane's own elements in order, then lane exchanges, then the
// workgroup's waves in order; equal inputs give equal bits.
#include "internal.hpp"
#include "device.hpp"

namespace nvfp4 {

namespace {


// Sum of v over the LANES lanes of a row; every lane gets it.  red: LDS of
// threads / 64 floats, free for the next sum only after a barrier.
template <int LANES>
__device__ __forceinline__ float row_sum(float v, float* red) {
#pragma unroll
  for (int o = (LANES < 64 ? LANES : 64) / 2; o >= 1; o >>= 1) v += __shfl_xor(v, o);
  if constexpr (LANES > 64) {
    constexpr int W = LANES / 64;
    const int wave = threadIdx.x >> 6, first = wave / W * W;
    if ((threadIdx.x & 63) == 0) red[wave] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < W; ++i) v += red[first + i];
  }
  return v;
}

__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                    pack_bf16x2(v[6], v[7]));
}

template <bool WIDE>
__device__ __forceinline__ void load_w(const void* w, int vec, float (&v)[8]) {
  if constexpr (WIDE) {
    const float4 a = static_cast<const float4*>(w)[2 * vec], b = static_cast<const float4*>(w)[2 * vec + 1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
    unpack8(static_cast<const uint4*>(w)[vec], v);
  }
}

// Squares are summed times 2^-16 (at most 2^15 columns), so that the sum stays
// finite wherever the mean does.
constexpr float kSquareScale = 1.52587890625e-05f;

// LANES lanes a row, NV vectors of eight columns each (vector i * LANES + lane).
template <int LANES, int NV, bool WIDE>
__global__ __launch_bounds__(LANES < 256 ? 256 : LANES) void rmsnorm_kernel(RmsnormArgs p) {
  constexpr int kThreads = LANES < 256 ? 256 : LANES;
  __shared__ float red[kThreads / 64];
  const int lane = threadIdx.x % LANES;
  const int64_t row = (int64_t)row_workgroup() * (kThreads / LANES) + threadIdx.x / LANES;
  const int vecs = p.cols / 8;
  const bool on = row < p.rows;
  const uint4* x = reinterpret_cast<const uint4*>(p.x + row * p.ld_x);
  const uint4* r = reinterpret_cast<const uint4*>(p.residual + row * p.ld_r);
  uint4 h[NV];
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int vec = i * LANES + lane;
    h[i] = make_uint4(0, 0, 0, 0);
    if (on && vec < vecs) h[i] = x[vec];
  }
  if (p.residual) {
    uint4 a[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int vec = i * LANES + lane;
      a[i] = make_uint4(0, 0, 0, 0);
      if (on && vec < vecs) a[i] = r[vec];
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float u[8], v[8];
      unpack8(h[i], u);
      unpack8(a[i], v);
#pragma unroll
      for (int j = 0; j < 8; ++j) u[j] += v[j];
      h[i] = pack8(u);
      const int vec = i * LANES + lane;
      if (on && vec < vecs) reinterpret_cast<uint4*>(p.h + row * p.cols)[vec] = h[i];
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float u[8];
    unpack8(h[i], u);
#pragma unroll
    for (int j = 0; j < 8; ++j) sum = fmaf(u[j] * kSquareScale, u[j], sum);
  }
  sum = row_sum<LANES>(sum, red);
  const float rstd = 1.0f / sqrtf(sum / ((float)p.cols * kSquareScale) + p.eps);
  if (p.rstd && lane == 0 && on) p.rstd[row] = rstd;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int vec = i * LANES + lane;
    const bool in = on && vec < vecs;
    float v[8], w[8];
    unpack8(h[i], v);
    if (vec < vecs) load_w<WIDE>(p.w, vec, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = vec < vecs ? v[j] * rstd * w[j] : 0.0f;
    if (p.y && in) reinterpret_cast<uint4*>(p.y + row * p.cols)[vec] = pack8(v);
    if (p.q) {
      float m = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(v[j]));
#pragma unroll
      for (int o = 8; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
      m = fmaxf(m, kFp8Floor);
      if (in) {
        *reinterpret_cast<uint2*>(p.q + row * p.cols + 8 * vec) = fp8_encode8(v, kE4m3Max / m);
        if ((lane & 15) == 0) p.sf[row * ((p.cols + 127) / 128) + vec / 16] = m / kE4m3Max;
      }
    }
  }
}

// dx of the rows this workgroup takes (every gridDim-th group of them) and its
// sum of dy * n, into part[workgroup][cols].
template <int LANES, int NV, bool WIDE>
__global__ __launch_bounds__(LANES < 256 ? 256 : LANES) void rmsnorm_bwd_kernel(RmsnormBwdArgs p, int groups) {
  constexpr int kThreads = LANES < 256 ? 256 : LANES, kRows = kThreads / LANES;
  __shared__ float red[2][kThreads / 64];
  extern __shared__ __align__(16) float dw_red[];       // [kRows][cols], several rows a workgroup
  const int lane = threadIdx.x % LANES, sub = threadIdx.x / LANES;
  const int vecs = p.cols / 8;
  float acc[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[i][j] = 0.0f;
  int flip = 0;
  for (int64_t row0 = (int64_t)blockIdx.x * kRows; row0 < p.rows; row0 += (int64_t)groups * kRows) {
    const int64_t row = row0 + sub;
    const bool on = row < p.rows;
    uint4 hv[NV], dv[NV], av[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int vec = i * LANES + lane;
      const bool in = on && vec < vecs;
      hv[i] = dv[i] = av[i] = make_uint4(0, 0, 0, 0);
      if (in) {
        hv[i] = reinterpret_cast<const uint4*>(p.h + row * p.cols)[vec];
        dv[i] = reinterpret_cast<const uint4*>(p.dy + row * p.cols)[vec];
        if (p.dh) av[i] = reinterpret_cast<const uint4*>(p.dh + row * p.cols)[vec];
      }
    }
    const float rstd = on ? p.rstd[row] : 0.0f;
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int vec = i * LANES + lane;
      if (vec >= vecs) continue;
      float n[8], d[8], w[8];
      unpack8(hv[i], n);
      unpack8(dv[i], d);
      load_w<WIDE>(p.w, vec, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        n[j] *= rstd;
        acc[i][j] = fmaf(d[j], n[j], acc[i][j]);
        sum = fmaf(d[j] * w[j], n[j], sum);
      }
    }
    sum = row_sum<LANES>(sum, red[flip]) / (float)p.cols;   // two buffers: one barrier a row
    flip ^= 1;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int vec = i * LANES + lane;
      if (!on || vec >= vecs) continue;
      float n[8], d[8], w[8], a[8];
      unpack8(hv[i], n);
      unpack8(dv[i], d);
      unpack8(av[i], a);
      load_w<WIDE>(p.w, vec, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) a[j] = fmaf(rstd, fmaf(-(n[j] * rstd), sum, d[j] * w[j]), a[j]);
      reinterpret_cast<uint4*>(p.dx + row * p.cols)[vec] = pack8(a);
    }
  }
  if (!p.part) return;
  float* part = p.part + (int64_t)blockIdx.x * p.cols;
  if constexpr (kRows == 1) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int vec = i * LANES + lane;
      if (vec >= vecs) continue;
      reinterpret_cast<float4*>(part)[2 * vec] = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
      reinterpret_cast<float4*>(part)[2 * vec + 1] = make_float4(acc[i][4], acc[i][5], acc[i][6], acc[i][7]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int vec = i * LANES + lane;
      if (vec >= vecs) continue;
      float4* dst = reinterpret_cast<float4*>(dw_red + sub * p.cols);
      dst[2 * vec] = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
      dst[2 * vec + 1] = make_float4(acc[i][4], acc[i][5], acc[i][6], acc[i][7]);
    }
    __syncthreads();
    for (int c = threadIdx.x; c < p.cols; c += kThreads) {
      float s = 0.0f;
#pragma unroll
      for (int k = 0; k < kRows; ++k) s += dw_red[k * p.cols + c];
      part[c] = s;
    }
  }
}

// dw = the workgroups' sums, added in order: 16 columns a workgroup, 16 threads
// a column over every 16th sum each.
__global__ __launch_bounds__(256) void rmsnorm_dw_kernel(const float* __restrict__ part, int groups, int cols,
                                                         float* __restrict__ dw) {
  __shared__ float red[16][17];
  const int c = threadIdx.x & 15, k = threadIdx.x >> 4;
  const int col = blockIdx.x * 16 + c;
  float s = 0.0f;
  if (col < cols)
    for (int g = k; g < groups; g += 16) s += part[(int64_t)g * cols + col];
  red[k][c] = s;
  __syncthreads();
  if (k == 0 && col < cols) {
#pragma unroll
    for (int i = 1; i < 16; ++i) s += red[i][c];
    dw[col] = s;
  }
}

template <int LANES, int NV>
hipError_t fwd(const RmsnormArgs& a, hipStream_t stream) {
  constexpr int kThreads = LANES < 256 ? 256 : LANES, kRows = kThreads / LANES;
  const dim3 grid = grid_rows((a.rows + kRows - 1) / kRows);
  if (a.wide) rmsnorm_kernel<LANES, NV, true><<<grid, kThreads, 0, stream>>>(a);
  else rmsnorm_kernel<LANES, NV, false><<<grid, kThreads, 0, stream>>>(a);
  return hipGetLastError();
}

template <int LANES, int NV>
hipError_t bwd(const RmsnormBwdArgs& a, int groups, hipStream_t stream) {
  constexpr int kThreads = LANES < 256 ? 256 : LANES, kRows = kThreads / LANES;
  const size_t lds = kRows > 1 ? sizeof(float) * kRows * a.cols : 0;
  if (a.wide) rmsnorm_bwd_kernel<LANES, NV, true><<<groups, kThreads, lds, stream>>>(a, groups);
  else rmsnorm_bwd_kernel<LANES, NV, false><<<groups, kThreads, lds, stream>>>(a, groups);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rmsnorm(const RmsnormArgs& a, hipStream_t stream) {
  const int vecs = a.cols / 8;
  if (vecs <= 16) return fwd<16, 1>(a, stream);
  if (vecs <= 64) return fwd<64, 1>(a, stream);
  if (vecs <= 128) return fwd<64, 2>(a, stream);
  if (vecs <= 256) return fwd<256, 1>(a, stream);
  if (vecs <= 512) return fwd<256, 2>(a, stream);
  if (vecs <= 1024) return fwd<256, 4>(a, stream);
  return fwd<1024, 4>(a, stream);
}

int rmsnorm_bwd_groups(int64_t rows, int64_t cols) {
  const int64_t per = cols <= 128 ? 16 : cols <= 1024 ? 4 : 1, n = (rows + per - 1) / per;
  return (int)(n < 1 ? 1 : n < 512 ? n : 512);
}

hipError_t launch_rmsnorm_bwd(const RmsnormBwdArgs& a, hipStream_t stream) {
  const int vecs = a.cols / 8, groups = rmsnorm_bwd_groups(a.rows, a.cols);
  hipError_t err;
  if (vecs <= 16) err = bwd<16, 1>(a, groups, stream);
  else if (vecs <= 64) err = bwd<64, 1>(a, groups, stream);
  else if (vecs <= 128) err = bwd<64, 2>(a, groups, stream);
  else if (vecs <= 256) err = bwd<256, 1>(a, groups, stream);
  else if (vecs <= 512) err = bwd<256, 2>(a, groups, stream);
  else if (vecs <= 1024) err = bwd<256, 4>(a, groups, stream);
  else err = bwd<1024, 4>(a, groups, stream);
  if (err != hipSuccess || !a.dw) return err;
  rmsnorm_dw_kernel<<<(a.cols + 15) / 16, 256, 0, stream>>>(a.part, groups, a.cols, a.dw);
  return hipGetLastError();
}

}  // namespace nvfp4
