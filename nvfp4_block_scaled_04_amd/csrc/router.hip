// Router: top-k of the expert logits and a softmax over the k chosen.
//
// The pages take routing ids and weights as inputs to the MoE runner (its
// last step scatters "with routing weights"); the tiny workload fixes the
// router as top-k of the logits followed by a softmax over those k.  The
// choice: the k largest logits in decreasing order, equal logits in
// increasing expert id, w_j = exp(l_j - l_max) / sum_i exp(l_i - l_max) in
// fp32.
//
// One wave per token.  Lane l holds logits l, l + 64, ... (up to 16 per
// lane, E <= 1024); each of the k rounds takes the wave-wide largest
// remaining value (lowest id among equals) with a butterfly reduction and
// retires it; lane j keeps round j's winner for the softmax and the store.
#include "internal.hpp"
#include "device.hpp"

namespace nvfp4 {

namespace {

constexpr int kRouterMaxPerLane = 16;    // E <= 1024

// (value, id) of the better of two candidates: larger value, then lower id
__device__ __forceinline__ void better(float& v, int& id, float v2, int id2) {
  if (v2 > v || (v2 == v && id2 < id)) {
    v = v2;
    id = id2;
  }
}

__global__ __launch_bounds__(256) void router_topk_kernel(const float* __restrict__ logits,
                                                          int64_t T, int E, int k,
                                                          int32_t* __restrict__ topk_ids,
                                                          float* __restrict__ topk_w) {
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t >= T) return;                          // the whole wave
  const float* row = logits + t * E;
  float v[kRouterMaxPerLane];
#pragma unroll
  for (int i = 0; i < kRouterMaxPerLane; ++i) {
    const int e = lane + 64 * i;
    v[i] = e < E ? row[e] : -INFINITY;         // logits are finite: padding never wins
  }
  float my_v = 0.0f;
  int my_id = 0;
  for (int j = 0; j < k; ++j) {
    // this lane's best remaining candidate
    float bv = v[0];
    int bid = lane;
#pragma unroll
    for (int i = 1; i < kRouterMaxPerLane; ++i) better(bv, bid, v[i], lane + 64 * i);
    // wave-wide best
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) {
      const float ov = __shfl_xor(bv, off);
      const int oid = __shfl_xor(bid, off);
      better(bv, bid, ov, oid);
    }
    // retire it (its owner lane), keep it in lane j
#pragma unroll
    for (int i = 0; i < kRouterMaxPerLane; ++i)
      if (lane + 64 * i == bid) v[i] = -INFINITY;
    if (lane == j) {
      my_v = bv;
      my_id = bid;
    }
  }
  // softmax over the chosen logits; round 0's winner is the maximum
  const float vmax = __shfl(my_v, 0);
  const float ex = lane < k ? __expf(my_v - vmax) : 0.0f;
  float sum = ex;
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) sum += __shfl_xor(sum, off);
  if (lane < k) {
    topk_ids[t * k + lane] = my_id;
    topk_w[t * k + lane] = ex / sum;
  }
}

// Gradient of the weights with respect to the logits: with w the softmax over
// the k chosen logits, dlogits[t][ids[t][j]] += w_j (dw_j - sum_i w_i dw_i),
// 0 for every other expert.  One wave per token: lane j forms term j, lane l
// then builds dlogits for four experts of each 256 in registers (4 l .. + 3
// with 16-byte stores, else l, l + 64, ...), taking the terms in slot order
// (ids repeated in a row add up in that order; ids outside [0, E) match no
// expert).  VEC: E % 4 == 0, 16-byte stores.  Bound by the 4 E bytes written
// per token when large, by latency below that: 8192 x 256 with k 8 takes
// 5.4 us (9.2 MB, 1.7 TB/s), 33 x 70 with k 3 2.6 us.
template <bool VEC>
__global__ __launch_bounds__(256) void router_topk_bwd_kernel(const int32_t* __restrict__ topk_ids,
                                                              const float* __restrict__ topk_w,
                                                              const float* __restrict__ dw,
                                                              int64_t T, int E, int k,
                                                              float* __restrict__ dlogits) {
#pragma clang fp contract(off)   // else w * g would round differently lane by lane in the exchanges
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)row_workgroup() * 4 + (threadIdx.x >> 6);
  if (t >= T) return;                          // the whole wave
  float w = 0.0f, g = 0.0f;
  int id = -1;
  if (lane < k) {
    w = topk_w[t * k + lane];
    g = dw[t * k + lane];
    id = topk_ids[t * k + lane];
  }
  float mean = w * g;
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) mean += __shfl_xor(mean, off);
  const float term = w * (g - mean);
  // every lane takes every pass: the terms are read from lanes that may hold
  // no expert of this pass
  for (int base = 0; base < E; base += 256) {
    constexpr int kStep = VEC ? 1 : 64;        // between a lane's experts
    const int e0 = base + (VEC ? 4 * lane : lane);
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int j = 0; j < k; ++j) {
      const int e = __builtin_amdgcn_readlane(id, j);
      const float d = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(term), j));
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] += e == e0 + kStep * i ? d : 0.0f;
    }
    if constexpr (VEC) {
      if (e0 < E) *reinterpret_cast<float4*>(dlogits + t * E + e0) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (e0 + kStep * i < E) dlogits[t * E + e0 + kStep * i] = v[i];
    }
  }
}

}  // namespace

hipError_t launch_router_topk_bwd(const int32_t* topk_ids, const float* topk_w, const float* dw,
                                  int64_t T, int E, int k, float* dlogits, hipStream_t stream) {
  if (T == 0) return hipSuccess;
  const dim3 blocks = grid_rows((T + 3) / 4);
  // 16-byte stores where every row starts on a 16-byte boundary
  if (E % 4 == 0 && reinterpret_cast<uintptr_t>(dlogits) % 16 == 0)
    router_topk_bwd_kernel<true><<<blocks, 256, 0, stream>>>(topk_ids, topk_w, dw, T, E, k, dlogits);
  else
    router_topk_bwd_kernel<false><<<blocks, 256, 0, stream>>>(topk_ids, topk_w, dw, T, E, k, dlogits);
  return hipGetLastError();
}

hipError_t launch_router_topk(const float* logits, int64_t T, int E, int k, int32_t* topk_ids,
                              float* topk_w, hipStream_t stream) {
  if (T == 0) return hipSuccess;
  // in pieces, since a launch of 2^32 threads or more would wrap without an error
  constexpr int64_t kPiece = int64_t(1) << 24;
  for (int64_t t = 0; t < T; t += kPiece) {
    const int64_t n = T - t < kPiece ? T - t : kPiece;
    router_topk_kernel<<<(unsigned)((n + 3) / 4), 256, 0, stream>>>(logits + t * E, n, E, k, topk_ids + t * k,
                                                                    topk_w + t * k);
  }
  return hipGetLastError();
}

}  // namespace nvfp4
