// Expert dispatch (bf16 rows in expert order) and the gradients of dispatch
// and combine (gfx950).
//
// With inv = inv_perm of nvfp4_moe_route and n = expert_offsets[E]:
//   dispatch            rows[inv[t*k+j]] = x[t] if inv < n, else 0
//   its gradient        dx[t] = bf16(sum over j with inv < n of drows[inv[t*k+j]])
//   combine's gradient  dy[inv[t*k+j]] = bf16(w[t][j] * dout[t]) if inv < n, else 0
//                       dw[t][j] = <dout[t], y[inv[t*k+j]]>      if inv < n, else 0
// inv_perm is a permutation of the T*k rows, so one group of threads per
// token touches every row exactly once: no atomics, a fixed summation order,
// and each token row is read once for its k expert rows.  All are bound by
// HBM (16-byte vectors, kBatch rows in flight per thread).  Measured with 8192
// tokens x 8 rows of 7168: dispatch 185 us in a graph's replays, 221 traced call
// by call, its gradient 181 to 187 us (1.06 GB: 5.8, 4.8 and 5.7 TB/s),
// combine's gradient 335 to 408 us, by the machine (2.0 GB: 4.9 to 6.0 TB/s); a
// large copy reaches 4.9 TB/s.  256 tokens: dispatch 6.5 to 6.8 us.
#include "internal.hpp"
#include "device.hpp"

namespace nvfp4 {

namespace {

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
constexpr int kBatch = 8;

__device__ __forceinline__ u32x4 load_nt(const u32x4* p) { return __builtin_nontemporal_load(p); }
__device__ __forceinline__ void store_nt(const u32x4& v, u32x4* p) { __builtin_nontemporal_store(v, p); }

__device__ __forceinline__ u32x4 pack8(const float (&x)[8]) {
  return u32x4{pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
               pack_bf16x2(x[6], x[7])};
}

// Token of this thread group (whole waves, so it is made uniform) and the
// thread's index in it.  A group is TPT threads; short rows put several
// tokens in one workgroup of kGroupThreads.
constexpr int kGroupThreads = 256;
template <int TPT>
__device__ __forceinline__ int64_t my_token(int& tid) {
  constexpr int per = TPT >= kGroupThreads ? 1 : kGroupThreads / TPT;
  tid = threadIdx.x % TPT;
  return (int64_t)row_workgroup() * per + __builtin_amdgcn_readfirstlane(threadIdx.x / TPT);
}

// Reads of a token's slots through the constant address space: scalar loads,
// all in flight together, so that which rows are routed is known in scalar
// registers before the first row is touched.
template <typename T>
__device__ __forceinline__ T uniform_load(const T* p, int64_t i) {
  return ((const __attribute__((address_space(4))) T*)p)[i];
}

// Rows of slots j0 .. j0 + kBatch - 1: -1 behind slot k - 1 and outside [0, M)
__device__ __forceinline__ void slot_rows(const int32_t* inv, int64_t t, int k, int j0, int64_t M,
                                          int32_t (&d)[kBatch]) {
#pragma unroll
  for (int b = 0; b < kBatch; ++b) d[b] = uniform_load(inv, t * k + (j0 + b < k ? j0 + b : k - 1));
#pragma unroll
  for (int b = 0; b < kBatch; ++b)
    if (j0 + b >= k || d[b] < 0 || d[b] >= M) d[b] = -1;
}

template <int TPT>
__global__ __launch_bounds__(TPT >= kGroupThreads ? TPT : kGroupThreads) void dispatch_kernel(
    const u32x4* __restrict__ x, const int32_t* __restrict__ inv, const int32_t* __restrict__ n_valid,
    int64_t T, int k, int hv, u32x4* __restrict__ rows) {
  int tid;
  const int64_t t = my_token<TPT>(tid);
  if (t >= T) return;
  const int32_t n = uniform_load(n_valid, 0);
  const int64_t M = T * k;
  for (int v = tid; v < hv; v += TPT) {
    const u32x4 a = x[t * hv + v];
    for (int j0 = 0; j0 < k; j0 += kBatch) {
      int32_t d[kBatch];
      slot_rows(inv, t, k, j0, M, d);
#pragma unroll
      for (int b = 0; b < kBatch; ++b)
        if (d[b] >= 0) store_nt(d[b] < n ? a : u32x4{0, 0, 0, 0}, rows + (int64_t)d[b] * hv + v);
    }
  }
}

template <int TPT>
__global__ __launch_bounds__(TPT >= kGroupThreads ? TPT : kGroupThreads) void dispatch_bwd_kernel(
    const u32x4* __restrict__ drows, const int32_t* __restrict__ inv,
    const int32_t* __restrict__ n_valid, int64_t T, int k, int hv, u32x4* __restrict__ dx) {
  int tid;
  const int64_t t = my_token<TPT>(tid);
  if (t >= T) return;
  const int64_t M = T * k;
  const int32_t n = uniform_load(n_valid, 0);
  for (int v = tid; v < hv; v += TPT) {
    float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    for (int j0 = 0; j0 < k; j0 += kBatch) {
      int32_t d[kBatch];
      slot_rows(inv, t, k, j0, M, d);
      u32x4 r[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        r[b] = u32x4{0, 0, 0, 0};
        if (d[b] >= 0 && d[b] < n) r[b] = load_nt(drows + (int64_t)d[b] * hv + v);
      }
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        float f[8];
        unpack8(r[b], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] += f[i];
      }
    }
    store_nt(pack8(acc), dx + t * hv + v);
  }
}

// dw may be null: then y is not read.
template <int TPT>
__global__ __launch_bounds__(TPT >= kGroupThreads ? TPT : kGroupThreads) void combine_bwd_kernel(
    const u32x4* __restrict__ dout, const u32x4* __restrict__ y, const int32_t* __restrict__ inv,
    const float* __restrict__ w, const int32_t* __restrict__ n_valid, int64_t T, int k, int hv,
    u32x4* __restrict__ dy, float* __restrict__ dw) {
  constexpr int kThreads = TPT >= kGroupThreads ? TPT : kGroupThreads;
  __shared__ float part[kThreads / 64][kBatch];
  int tid;
  const int64_t t = my_token<TPT>(tid);
  const bool live = t < T;                      // the whole group
  const int64_t M = T * k;
  const int32_t n = uniform_load(n_valid, 0);
  for (int j0 = 0; j0 < k; j0 += kBatch) {
    float dot[kBatch] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (live) {
      int32_t d[kBatch];
      float wj[kBatch];
      slot_rows(inv, t, k, j0, M, d);
#pragma unroll
      for (int b = 0; b < kBatch; ++b) wj[b] = uniform_load(w, t * k + (j0 + b < k ? j0 + b : k - 1));
      for (int v = tid; v < hv; v += TPT) {
        u32x4 r[kBatch];
        const u32x4 gv = dout[t * hv + v];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
          r[b] = u32x4{0, 0, 0, 0};
          if (dw && d[b] >= 0 && d[b] < n) r[b] = load_nt(y + (int64_t)d[b] * hv + v);
        }
        float g[8];
        unpack8(gv, g);
        // the stores first: they need no row of y
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
          if (d[b] < 0) continue;
          float o[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] = wj[b] * g[i];
          store_nt(d[b] < n ? pack8(o) : u32x4{0, 0, 0, 0}, dy + (int64_t)d[b] * hv + v);
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
          float f[8], s = 0.0f;
          unpack8(r[b], f);
#pragma unroll
          for (int i = 0; i < 8; ++i) s = fmaf(g[i], f[i], s);
          dot[b] += s;
        }
      }
      // no row: 0 also where dout is not finite
#pragma unroll
      for (int b = 0; b < kBatch; ++b)
        if (d[b] < 0 || d[b] >= n) dot[b] = 0.0f;
    }
    if (!dw) continue;
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
#pragma unroll
      for (int o = 32; o >= 1; o >>= 1) dot[b] += __shfl_xor(dot[b], o);
    }
    if constexpr (TPT == 64) {
      float mine = dot[0];
#pragma unroll
      for (int b = 1; b < kBatch; ++b)
        if (tid == b) mine = dot[b];
      if (live && tid < kBatch && j0 + tid < k) dw[t * k + j0 + tid] = mine;
    } else {
      if ((threadIdx.x & 63) == 0) {
#pragma unroll
        for (int b = 0; b < kBatch; ++b) part[threadIdx.x >> 6][b] = dot[b];
      }
      __syncthreads();
      if (live && tid < kBatch && j0 + tid < k) {
        const int w0 = (threadIdx.x - tid) >> 6;
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < TPT / 64; ++i) s += part[w0 + i][tid];
        dw[t * k + j0 + tid] = s;
      }
      __syncthreads();
    }
  }
}

// threads per token: the fewest waves (1, 2, 4, 8 or 14) that give each
// thread at most one vector, or 14
template <template <int> class F, typename... A>
void by_width(int hv, A&&... a) {
  if (hv <= 64) F<64>::go(a...);
  else if (hv <= 128) F<128>::go(a...);
  else if (hv <= 256) F<256>::go(a...);
  else if (hv <= 512) F<512>::go(a...);
  else F<896>::go(a...);
}

template <int TPT>
dim3 grid_of(int64_t T) {
  constexpr int64_t per = TPT >= kGroupThreads ? 1 : kGroupThreads / TPT;
  return grid_rows((T + per - 1) / per);
}
template <int TPT>
constexpr int threads_of() { return TPT >= kGroupThreads ? TPT : kGroupThreads; }

template <int TPT>
struct Dispatch {
  static void go(const void* x, const int32_t* inv, const int32_t* n, int64_t T, int k, int hv,
                 void* rows, hipStream_t s) {
    dispatch_kernel<TPT><<<grid_of<TPT>(T), threads_of<TPT>(), 0, s>>>(
        static_cast<const u32x4*>(x), inv, n, T, k, hv, static_cast<u32x4*>(rows));
  }
};
template <int TPT>
struct DispatchBwd {
  static void go(const void* drows, const int32_t* inv, const int32_t* n, int64_t T, int k, int hv,
                 void* dx, hipStream_t s) {
    dispatch_bwd_kernel<TPT><<<grid_of<TPT>(T), threads_of<TPT>(), 0, s>>>(
        static_cast<const u32x4*>(drows), inv, n, T, k, hv, static_cast<u32x4*>(dx));
  }
};
template <int TPT>
struct CombineBwd {
  static void go(const void* dout, const void* y, const int32_t* inv, const float* w,
                 const int32_t* n, int64_t T, int k, int hv, void* dy, float* dw, hipStream_t s) {
    combine_bwd_kernel<TPT><<<grid_of<TPT>(T), threads_of<TPT>(), 0, s>>>(
        static_cast<const u32x4*>(dout), static_cast<const u32x4*>(y), inv, w, n, T, k, hv,
        static_cast<u32x4*>(dy), dw);
  }
};

}  // namespace

hipError_t launch_dispatch(const void* x, const int32_t* inv_perm, const int32_t* offsets, int64_t T,
                           int k, int E, int64_t H, void* rows, hipStream_t stream) {
  if (T == 0) return hipSuccess;
  by_width<Dispatch>((int)(H / 8), x, inv_perm, offsets + E, T, k, (int)(H / 8), rows, stream);
  return hipGetLastError();
}

hipError_t launch_dispatch_bwd(const void* drows, const int32_t* inv_perm, const int32_t* offsets,
                               int64_t T, int k, int E, int64_t H, void* dx, hipStream_t stream) {
  if (T == 0) return hipSuccess;
  by_width<DispatchBwd>((int)(H / 8), drows, inv_perm, offsets + E, T, k, (int)(H / 8), dx, stream);
  return hipGetLastError();
}

hipError_t launch_combine_bwd(const void* dout, const void* y, const int32_t* inv_perm,
                              const float* topk_w, const int32_t* offsets, int64_t T, int k, int E,
                              int64_t H, void* dy, float* dw, hipStream_t stream) {
  if (T == 0) return hipSuccess;
  by_width<CombineBwd>((int)(H / 8), dout, y, inv_perm, topk_w, offsets + E, T, k, (int)(H / 8), dy,
                       dw, stream);
  return hipGetLastError();
}

}  // namespace nvfp4
