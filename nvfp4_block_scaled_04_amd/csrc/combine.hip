// Routing-weighted combine of expert outputs back to tokens (gfx950).
//
// README "NVFP4 MegaMoE Kernel", "What We Have", MoE runner step 6: scatter
// with routing weights.  Written as a gather so no atomics are needed and the
// result is deterministic:
//   out[t][n] = bf16( sum_{j<k} w[t][j] * y[inv_perm[t*k+j]][n] ),
// fp32 accumulation in slot order; rows d >= offsets[E] (invalid expert ids)
// contribute nothing.  One block per token; each thread moves 16 bytes
// (8 BF16) per row of up to two column vectors kThreads apart at a time, so
// every wave reads 1 KiB contiguous spans and a thread keeps kBatch (or
// 2 * kBatch) row loads in flight.  896 threads cover a 7168-wide row in one
// pass with one vector per thread: 10% faster at T=8192, H=7168, k=8 than
// 128 threads with two vectors each over 3.5 passes (224 and 448 threads
// fell between).  y is read
// once and out written once: both go through non-temporal accesses, which
// keep them from displacing other lines in the caches (6% faster at
// T=8192, H=7168, k=8 than plain accesses).
#include "internal.hpp"
#include "device.hpp"

namespace nvfp4 {

namespace {

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
constexpr int kThreads = 896;
constexpr int kBatch = 8;                   // rows whose loads are in flight together

__global__ __launch_bounds__(kThreads) void combine_kernel(
    const uint4* __restrict__ y, const int32_t* __restrict__ inv_perm,
    const float* __restrict__ topk_w, const int32_t* __restrict__ offsets, int k, int E,
    int64_t H, uint4* __restrict__ out) {
  const int64_t t = blockIdx.x;
  const int64_t hv = H / 8;                 // 16-byte vectors per row
  const int32_t n_valid = offsets[E];
  // two vectors per thread per pass (kBatch rows each): 2 * kBatch loads in flight
  for (int64_t v0 = threadIdx.x; v0 < hv; v0 += 2 * kThreads) {
    const int64_t v1 = v0 + kThreads;
    const bool has1 = v1 < hv;
    float acc0[8] = {0, 0, 0, 0, 0, 0, 0, 0}, acc1[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    for (int j0 = 0; j0 < k; j0 += kBatch) {
      uint4 r0[kBatch], r1[kBatch];
      float w[kBatch];
      bool ok[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int j = j0 + b;
        const int32_t d = j < k ? inv_perm[t * k + j] : n_valid;
        ok[b] = d < n_valid;
        w[b] = ok[b] ? topk_w[t * k + j] : 0.0f;
        r0[b] = make_uint4(0, 0, 0, 0);
        r1[b] = make_uint4(0, 0, 0, 0);
        if (ok[b]) {
          const u32x4 q = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(y + (int64_t)d * hv + v0));
          r0[b] = make_uint4(q[0], q[1], q[2], q[3]);
          if (has1) {
            const u32x4 q1 = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(y + (int64_t)d * hv + v1));
            r1[b] = make_uint4(q1[0], q1[1], q1[2], q1[3]);
          }
        }
      }
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        if (!ok[b]) continue;
        const uint32_t p0[4] = {r0[b].x, r0[b].y, r0[b].z, r0[b].w};
        const uint32_t p1[4] = {r1[b].x, r1[b].y, r1[b].z, r1[b].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          acc0[2 * i] = fmaf(w[b], bf16_to_f32(p0[i] & 0xFFFFu), acc0[2 * i]);
          acc0[2 * i + 1] = fmaf(w[b], bf16_to_f32(p0[i] >> 16), acc0[2 * i + 1]);
          acc1[2 * i] = fmaf(w[b], bf16_to_f32(p1[i] & 0xFFFFu), acc1[2 * i]);
          acc1[2 * i + 1] = fmaf(w[b], bf16_to_f32(p1[i] >> 16), acc1[2 * i + 1]);
        }
      }
    }
    const u32x4 o0 = {pack_bf16x2(acc0[0], acc0[1]), pack_bf16x2(acc0[2], acc0[3]),
                      pack_bf16x2(acc0[4], acc0[5]), pack_bf16x2(acc0[6], acc0[7])};
    __builtin_nontemporal_store(o0, reinterpret_cast<u32x4*>(out + t * hv + v0));
    if (has1) {
      const u32x4 o1 = {pack_bf16x2(acc1[0], acc1[1]), pack_bf16x2(acc1[2], acc1[3]),
                        pack_bf16x2(acc1[4], acc1[5]), pack_bf16x2(acc1[6], acc1[7])};
      __builtin_nontemporal_store(o1, reinterpret_cast<u32x4*>(out + t * hv + v1));
    }
  }
}

}  // namespace

hipError_t launch_combine(const void* y, const int32_t* inv_perm, const float* topk_w,
                          const int32_t* offsets, int64_t T, int k, int E, int64_t H, void* out,
                          hipStream_t stream) {
  if (T == 0) return hipSuccess;
  // In pieces of 2^22 tokens, since a launch of 2^32 threads or more would wrap
  // without an error.  (A bound check in the kernel, for a grid in two
  // dimensions, takes 10% of a small call: 1000 x 6 x 512, 4.3 -> 4.8 us.)
  constexpr int64_t kPiece = int64_t(1) << 22;
  for (int64_t t = 0; t < T; t += kPiece) {
    combine_kernel<<<(unsigned)(T - t < kPiece ? T - t : kPiece), kThreads, 0, stream>>>(
        static_cast<const uint4*>(y), inv_perm + t * k, topk_w + t * k, offsets, k, E, H,
        static_cast<uint4*>(out) + t * (H / 8));
  }
  return hipGetLastError();
}

}  // namespace nvfp4
