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

typedef uint32_t uint4v __attribute__((ext_vector_type(4)));
typedef uint32_t uint2v __attribute__((ext_vector_type(2)));

// Rows past the caches where a call moves more than these hold (STREAM)
template <bool STREAM>
__device__ __forceinline__ uint4 load16(const uint16_t* p) {
  if constexpr (STREAM) {
    const uint4v v = __builtin_nontemporal_load(reinterpret_cast<const uint4v*>(p));
    return make_uint4(v.x, v.y, v.z, v.w);
  } else {
    return *reinterpret_cast<const uint4*>(p);
  }
}
template <bool STREAM>
__device__ __forceinline__ void store16(uint16_t* p, const uint4& v) {
  if constexpr (STREAM) __builtin_nontemporal_store(uint4v{v.x, v.y, v.z, v.w}, reinterpret_cast<uint4v*>(p));
  else *reinterpret_cast<uint4*>(p) = v;
}
template <bool STREAM>
__device__ __forceinline__ void store8(uint8_t* p, const uint2& v) {
  if constexpr (STREAM) __builtin_nontemporal_store(uint2v{v.x, v.y}, reinterpret_cast<uint2v*>(p));
  else *reinterpret_cast<uint2*>(p) = v;
}

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
    lds_barrier();
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

// Eight weights as they are stored
template <bool WIDE>
struct W8 {
  uint4 v[WIDE ? 2 : 1];
  __device__ __forceinline__ void load(const void* w, int vec) {
#pragma unroll
    for (int i = 0; i < (WIDE ? 2 : 1); ++i) v[i] = static_cast<const uint4*>(w)[(WIDE ? 2 : 1) * vec + i];
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    if constexpr (WIDE) {
      const uint32_t u[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = __uint_as_float(u[j]);
    } else {
      unpack8(v[0], f);
    }
  }
};

// Squares are summed times 2^-16 (at most 2^15 columns), so that the sum stays
// finite wherever the mean does.  Sums that this makes subnormal (a mean below 2^-113
// in rows of 128, where the smallest eps allowed, 1e-30, is 2^-99.7) need fp32's
// subnormal numbers, which this build keeps: their roundings of 2^-150 are 2^-134
// each in the mean, 2^-34 of that eps; flushed to zero they would cost 2^-14 of 1/rms.
constexpr float kSquareScale = 1.52587890625e-05f;

// LANES lanes a row, NV vectors of eight columns each (vector i * LANES + lane): the
// row stays in registers from its one read to the outputs, its weights are on their
// way with it.  Bound by HBM from some thousand rows on, below by the launch and two
// round trips to memory.  Measured with residual, BF16 and FP8 outputs: 8192 x 7168
// 88 to 92 us (531 MB, 5.8 to 6.0 TB/s; 256 lanes a row 98), 2048 x 7168 21 us (6.2
// TB/s), 512 x 7168 7.6; one row of 7168 3.5 us, an empty launch 2.6; 65536 rows of
// 128 in BF16 alone 7.7 us.
template <int LANES, int NV, bool WIDE, bool STREAM>
__global__ __launch_bounds__(LANES < 256 ? 256 : LANES) void rmsnorm_kernel(RmsnormArgs p) {
  constexpr int kThreads = LANES < 256 ? 256 : LANES;
  __shared__ float red[kThreads / 64];
  const int lane = threadIdx.x % LANES;
  const int64_t row = (int64_t)row_workgroup() * (kThreads / LANES) + threadIdx.x / LANES;
  const int vecs = p.cols / 8;
  const bool on = row < p.rows;
  const uint16_t* x = p.x + row * p.ld_x;
  const uint16_t* r = p.residual + row * p.ld_r;
  uint4 h[NV];
  W8<WIDE> wv[NV];
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int vec = i * LANES + lane;
    wv[i].load(p.w, vec < vecs ? vec : 0);
    h[i] = make_uint4(0, 0, 0, 0);
    if (on && vec < vecs) h[i] = load16<STREAM>(x + 8 * vec);
  }
  if (p.residual) {
    uint4 a[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int vec = i * LANES + lane;
      a[i] = make_uint4(0, 0, 0, 0);
      if (on && vec < vecs) a[i] = load16<STREAM>(r + 8 * vec);
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
      if (on && vec < vecs) store16<STREAM>(p.h + row * p.cols + 8 * vec, h[i]);
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
    wv[i].get(w);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = vec < vecs ? v[j] * rstd * w[j] : 0.0f;
    if (p.y && in) store16<STREAM>(p.y + row * p.cols + 8 * vec, pack8(v));
    if (p.q) {
      float m = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(v[j]));
#pragma unroll
      for (int o = 8; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
      m = fmaxf(m, kFp8Floor);
      if (in) {
        store8<STREAM>(p.q + row * p.cols + 8 * vec, fp8_encode8(v, kE4m3Max / m));
        if ((lane & 15) == 0) p.sf[row * ((p.cols + 127) / 128) + vec / 16] = m / kE4m3Max;
      }
    }
  }
}

// Bound by HBM: 8192 x 7168 with dh 84 to 87 us (470 MB, 5.4 to 5.6 TB/s) and 5 for dw
// below; 77 x 1000 3.8 us and 2.4, of which an empty launch is 2.6.
// dx of the rows this workgroup takes (every groups-th of them) and its sum of
// dy * n, into part[workgroup][cols].  With one vector a lane a row's loads go out
// before the row in front is summed, whose sum is a barrier for all (16384 x 2048:
// 53 us, without 60); with more the registers cost more than that gives (8192 x
// 7168: 103 us, without 89), and with four the weights stay out of them too.
template <int LANES, int NV, bool WIDE, bool STREAM>
__global__ __launch_bounds__(LANES < 256 ? 256 : LANES, 4) void rmsnorm_bwd_kernel(RmsnormBwdArgs p, int groups) {
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
  struct Row {
    uint4 h[NV], dy[NV], dh[NV];
    float rstd;
  };
  auto load = [&](int64_t row, Row& x) {
    const bool on = row < p.rows;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int vec = i * LANES + lane;
      x.h[i] = x.dy[i] = x.dh[i] = make_uint4(0, 0, 0, 0);
      if (on && vec < vecs) {
        x.h[i] = load16<STREAM>(p.h + row * p.ld_h + 8 * vec);
        x.dy[i] = load16<STREAM>(p.dy + row * p.cols + 8 * vec);
        if (p.dh) x.dh[i] = load16<STREAM>(p.dh + row * p.cols + 8 * vec);
      }
    }
    x.rstd = on ? p.rstd[row] : 0.0f;
  };
  W8<WIDE> wv[NV];
  auto weights = [&](int i) {
    const int vec = i * LANES + lane;
    wv[i].load(p.w, vec < vecs ? vec : 0);
  };
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if constexpr (NV <= 2) weights(i);
  int flip = 0;
  const int64_t step = (int64_t)groups * kRows;
  constexpr bool kAhead = NV == 1, kHeld = NV <= 2;
  Row x, next;
  if constexpr (kAhead) load((int64_t)blockIdx.x * kRows + sub, x);
  for (int64_t row0 = (int64_t)blockIdx.x * kRows; row0 < p.rows; row0 += step) {
    const int64_t row = row0 + sub;
    if constexpr (kAhead) load(row + step, next);
    else load(row, x);
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int vec = i * LANES + lane;
      if (vec >= vecs) continue;
      float n[8], d[8], w[8];
      unpack8(x.h[i], n);
      unpack8(x.dy[i], d);
      if constexpr (!kHeld) weights(i);
      wv[i].get(w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        n[j] *= x.rstd;
        acc[i][j] = fmaf(d[j], n[j], acc[i][j]);
        sum = fmaf(d[j] * w[j], n[j], sum);
      }
    }
    sum = row_sum<LANES>(sum, red[flip]) / (float)p.cols;   // two buffers: one barrier a row
    flip ^= 1;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int vec = i * LANES + lane;
      if (row >= p.rows || vec >= vecs) continue;
      float n[8], d[8], w[8], a[8];
      unpack8(x.h[i], n);
      unpack8(x.dy[i], d);
      unpack8(x.dh[i], a);
      if constexpr (!kHeld) weights(i);
      wv[i].get(w);
#pragma unroll
      for (int j = 0; j < 8; ++j) a[j] = fmaf(x.rstd, fmaf(-(n[j] * x.rstd), sum, d[j] * w[j]), a[j]);
      store16<STREAM>(p.dx + row * p.cols + 8 * vec, pack8(a));
    }
    if constexpr (kAhead) x = next;
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

// dw = the workgroups' sums: 32 columns a workgroup, 32 threads for four of them,
// each adding every 32nd sum in order, then the threads' sums in order.
__global__ __launch_bounds__(256) void rmsnorm_dw_kernel(const float* __restrict__ part, int groups, int cols,
                                                         float* __restrict__ dw) {
  __shared__ float4 red[32][8];
  const int c = threadIdx.x & 7, k = threadIdx.x >> 3;
  const int col = blockIdx.x * 32 + 4 * c;
  float4 s = make_float4(0, 0, 0, 0);
  if (col < cols) {
#pragma unroll 8
    for (int g = k; g < groups; g += 32) {
      const float4 v = *reinterpret_cast<const float4*>(part + (int64_t)g * cols + col);
      s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
    }
  }
  red[k][c] = s;
  __syncthreads();
  const int at = blockIdx.x * 32 + threadIdx.x;
  if (threadIdx.x < 32 && at < cols) {
    float v = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) v += reinterpret_cast<const float*>(red[i])[threadIdx.x];
    dw[at] = v;
  }
}

// Rows go past the caches where a tensor holds more than 64 MiB (norm with residual,
// BF16 and FP8; gradient): 8192 x 7168 92 and 87 us, through them 98 and 96; 8192 x
// 4096 53 and 50, through them 53 and 45; 2048 x 7168 26 and 30, through them 21 and 26.
bool streams(int64_t rows, int64_t cols) { return rows * cols > (int64_t(1) << 25); }

template <int LANES, int NV>
hipError_t fwd(const RmsnormArgs& a, hipStream_t stream) {
  constexpr int kThreads = LANES < 256 ? 256 : LANES, kRows = kThreads / LANES;
  const dim3 grid = grid_rows((a.rows + kRows - 1) / kRows);
  auto run = [&](auto kernel) { kernel<<<grid, kThreads, 0, stream>>>(a); };
  if (streams(a.rows, a.cols)) run(a.wide ? rmsnorm_kernel<LANES, NV, true, true> : rmsnorm_kernel<LANES, NV, false, true>);
  else run(a.wide ? rmsnorm_kernel<LANES, NV, true, false> : rmsnorm_kernel<LANES, NV, false, false>);
  return hipGetLastError();
}

template <int LANES, int NV>
hipError_t bwd(const RmsnormBwdArgs& a, int groups, hipStream_t stream) {
  constexpr int kThreads = LANES < 256 ? 256 : LANES, kRows = kThreads / LANES;
  const size_t lds = kRows > 1 ? sizeof(float) * kRows * a.cols : 0;
  auto run = [&](auto kernel) { kernel<<<groups, kThreads, lds, stream>>>(a, groups); };
  if (streams(a.rows, a.cols)) run(a.wide ? rmsnorm_bwd_kernel<LANES, NV, true, true> : rmsnorm_bwd_kernel<LANES, NV, false, true>);
  else run(a.wide ? rmsnorm_bwd_kernel<LANES, NV, true, false> : rmsnorm_bwd_kernel<LANES, NV, false, false>);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rmsnorm(const RmsnormArgs& a, hipStream_t stream) {
  const int vecs = a.cols / 8;
  if (vecs <= 16) return fwd<16, 1>(a, stream);
  if (vecs <= 64) return fwd<64, 1>(a, stream);
  if (vecs <= 128) return fwd<64, 2>(a, stream);
  if (vecs <= 256) return fwd<256, 1>(a, stream);
  if (vecs <= 512) return fwd<512, 1>(a, stream);
  if (vecs <= 1024) return fwd<512, 2>(a, stream);
  if (vecs <= 2048) return fwd<1024, 2>(a, stream);
  return fwd<1024, 4>(a, stream);
}

// Workgroups of the gradient: one a CU, which keeps the sums of dw few (1024 x 7168:
// 17 us, with 512 21), and two from 16 rows each on (8192 x 4096: 50 us, with 256 62).
int rmsnorm_bwd_groups(int64_t rows, int64_t cols) {
  const int64_t per = cols <= 128 ? 16 : cols <= 1024 ? 4 : 1, n = (rows + per - 1) / per;
  const int most = n >= 16 * 512 && cols <= 16384 ? 512 : 256;
  return (int)(n < 1 ? 1 : n < most ? n : most);
}

hipError_t launch_rmsnorm_bwd(const RmsnormBwdArgs& a, hipStream_t stream) {
  const int vecs = a.cols / 8, groups = rmsnorm_bwd_groups(a.rows, a.cols);
  hipError_t err;
  if (vecs <= 16) err = bwd<16, 1>(a, groups, stream);
  else if (vecs <= 64) err = bwd<64, 1>(a, groups, stream);
  else if (vecs <= 128) err = bwd<64, 2>(a, groups, stream);
  else if (vecs <= 256) err = bwd<256, 1>(a, groups, stream);
  else if (vecs <= 512) err = bwd<512, 1>(a, groups, stream);
  else if (vecs <= 1024) err = bwd<512, 2>(a, groups, stream);
  else if (vecs <= 2048) err = bwd<1024, 2>(a, groups, stream);
  else err = bwd<1024, 4>(a, groups, stream);
  if (err != hipSuccess || !a.dw) return err;
  rmsnorm_dw_kernel<<<(a.cols + 31) / 32, 256, 0, stream>>>(a.part, groups, a.cols, a.dw);
  return hipGetLastError();
}

}  // namespace nvfp4
