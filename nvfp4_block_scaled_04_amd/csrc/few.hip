// The expert layer for a few tokens in two kernels (gfx950).
//
//   up:    a = W1[e] x_t,  h = c_te * silu(gate) * up   for every expert e with a
//          token and its tokens t;  c_te = sum of w[t][j] over ids[t][j] == e
//   down:  out[t][n] = bf16( sum over experts e of W2[e][n] . h_te )
// Weights FP8 (one scale per 128 x 128) or packed NVFP4 (E4M3 per 16, a global
// scale an expert, taken into c).  Activations are not quantised: x enters the
// matrix unit as BF16, h as two BF16 (its rounding and what that leaves, 16 bits
// in all), the weight codes as BF16, which holds them exactly.  Sums in fp32.
//
// Each live expert's weights are read once; their bytes are the bound.  Tokens
// are the matrix unit's 16 columns, so up to 16 tokens cost what one costs, and
// the second product adds its experts up in the accumulators: a column whose
// token did not choose the expert is fed zeros.
//
// A workgroup's eight waves split the K blocks of 128 of its tile and join
// through LDS in wave order (equal inputs give equal bits).  A wave's loads go on
// across tile ends, kDepth blocks ahead.
#include <atomic>

#include "internal.hpp"
#include "device.hpp"

namespace nvfp4 {

namespace {

typedef int int4v __attribute__((ext_vector_type(4)));
typedef float float4v __attribute__((ext_vector_type(4)));
typedef float float2v __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kWaves = 8, kThreads = kWaves * 64;
constexpr int kPairs = kFewTokens * 64;               // (token, slot) pairs at most
constexpr int kMaxExperts = 4096;

// A byte offset with this bit set lies behind every resource below (they all
// hold less than 2^31 bytes): the load returns zeros and touches no memory.
constexpr uint32_t kNowhere = 0x80000000u;

__device__ const float kNoScale = 0.0f;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc_of(const void* base, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, 0x00020000);
}

__device__ __forceinline__ float uniform_load(const float* p) {
  return *(const __attribute__((address_space(4))) float*)p;
}

// The experts that have a token, in order of their first pair: expert, its
// tokens as a bit mask, and the row of its first token in h (rows follow the
// experts and, inside one, the tokens).
struct Live {
  int n;
  int e[kPairs], mask[kPairs], row[kPairs];
  int id[kPairs];               // the pairs' experts, -1 for those without one
  float w[kPairs];              // and weights
};

struct LiveScratch {
  int first[kMaxExperts];       // first pair of an expert, then its place in the list
  int count[kPairs / 64];
};

__device__ void build_live(const FewArgs& p, Live& L, LiveScratch& S) {
  const int pairs = p.T * p.k, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  constexpr int kPer = kPairs / kThreads;
  int e[kPer];
  for (int i = threadIdx.x; i < p.E; i += kThreads) S.first[i] = 0x7FFFFFFF;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int f = i * kThreads + threadIdx.x;
    e[i] = f < pairs ? p.ids[f] : -1;
    if (e[i] < 0 || e[i] >= p.E) e[i] = -1;
    else atomicMin(&S.first[e[i]], f);
    L.id[f] = e[i];
    L.w[f] = f < pairs ? p.topk_w[f] : 0.0f;
  }
  __syncthreads();
  uint64_t firsts[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    firsts[i] = __ballot(e[i] >= 0 && S.first[e[i] < 0 ? 0 : e[i]] == i * kThreads + (int)threadIdx.x);
    if (lane == 0) S.count[i * kWaves + wave] = __popcll(firsts[i]);
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    int at = 0;
    for (int c = 0; c < i * kWaves + wave; ++c) at += S.count[c];
    if (firsts[i] >> lane & 1) {
      at += __popcll(firsts[i] & ((uint64_t(1) << lane) - 1));
      L.e[at] = e[i];
      L.mask[at] = 0;
      S.first[e[i]] = at;
    }
  }
  if (threadIdx.x == 0) {
    int n = 0;
    for (int c = 0; c < kPer * kWaves; ++c) n += S.count[c];
    L.n = n;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (e[i] >= 0) atomicOr(&L.mask[S.first[e[i]]], 1 << ((i * kThreads + (int)threadIdx.x) / p.k));
  __syncthreads();
  if (wave == 0) {
    int run = 0;
    for (int u0 = 0; u0 < L.n; u0 += 64) {
      const int u = u0 + lane, own = u < L.n ? __popc(L.mask[u]) : 0;
      int incl = own;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const int v = __shfl_up(incl, o);
        incl += lane >= o ? v : 0;
      }
      if (u < L.n) L.row[u] = run + incl - own;
      run += __shfl(incl, 63);
    }
  }
  __syncthreads();
}

// One operand of a product: the weights of all experts, N rows of K.
template <bool FP8>
struct Weights {
  const uint8_t* q;
  const uint8_t* sf;            // FP8: float scales
  int64_t N;
  int K, KB;                    // KB: K blocks of 128
  int64_t q_bytes, sf_bytes;    // of one expert
  int NB;                       // FP8: scale blocks along N
};

template <bool FP8>
__device__ __forceinline__ Weights<FP8> weights_of(const uint8_t* q, const void* sf, int64_t N, int64_t K) {
  Weights<FP8> w;
  w.q = q;
  w.sf = static_cast<const uint8_t*>(sf);
  w.N = N;
  w.K = (int)K;
  w.KB = (int)((K + 127) / 128);
  w.NB = (int)((N + 127) / 128);
  const int64_t Np = (N + NVFP4_PACK_ROWS - 1) / NVFP4_PACK_ROWS * NVFP4_PACK_ROWS;
  w.q_bytes = FP8 ? N * K : Np * (K / 2);
  w.sf_bytes = FP8 ? (int64_t)w.NB * w.KB * 4 : Np * (K / 16);
  return w;
}

// A wave's share of one K block: RF fragments of 16 weight rows and the tokens.
// Lane (r = lane & 15, g = lane >> 4) holds row or token r and the columns
//   FP8    16g .. 16g + 15 and 64 + 16g .. 64 + 16g + 15 of the block,
//   NVFP4  32g .. 32g + 31,
// eight of them a matrix instruction.
template <bool FP8, int RF, int HT>
struct Step {
  int4v w[RF][FP8 ? 2 : 1];
  uint32_t s[FP8 ? 1 : RF];     // NVFP4: the lane's two scale bytes
  float sb[FP8 ? RF : 1];       // FP8: the block's scale, uniform
  int4v t[HT][4];               // tokens: HT terms (x: 1, h: 2) of 32 columns
  bool mine;                    // the lane's token has the expert
};

__device__ __forceinline__ bf16x8 as_bf16(const int4v& v) { return __builtin_bit_cast(bf16x8, v); }

// Eight weights of the lane's 32 as BF16: number m.
template <bool FP8>
__device__ __forceinline__ bf16x8 decode8(const int4v* w, uint32_t scales, int m) {
  uint32_t o[4];
  if constexpr (FP8) {
    const int lo = w[m >> 1][2 * (m & 1)], hi = w[m >> 1][2 * (m & 1) + 1];
    o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false));
    o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true));
    o[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false));
    o[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true));
  } else {
    const float s = m < 2 ? __builtin_amdgcn_cvt_f32_fp8(scales, 0) : __builtin_amdgcn_cvt_f32_fp8(scales, 1);
    const uint32_t c = w[0][m];
    const float2v a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 1);
    const float2v d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 2), f = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 3);
    o[0] = pack_bf16x2(a[0] * s, a[1] * s);      // exact: 2 + 4 bits of significand
    o[1] = pack_bf16x2(b[0] * s, b[1] * s);
    o[2] = pack_bf16x2(d[0] * s, d[1] * s);
    o[3] = pack_bf16x2(f[0] * s, f[1] * s);
  }
  return __builtin_bit_cast(bf16x8, int4v{(int)o[0], (int)o[1], (int)o[2], (int)o[3]});
}

// A token without the expert gets nothing of it, whatever its weights hold
// (zeros times a NaN or an infinity would be no zeros).
template <bool FP8, int RF, int HT>
__device__ __forceinline__ void add_step(float4v (&acc)[RF], const Step<FP8, RF, HT>& x) {
#pragma unroll
  for (int f = 0; f < RF; ++f) {
    float4v d = float4v{0, 0, 0, 0};
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const bf16x8 w = decode8<FP8>(x.w[f], x.s[FP8 ? 0 : f], m);
#pragma unroll
      for (int t = 0; t < HT; ++t) d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, as_bf16(x.t[t][m]), d, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float v = FP8 ? fmaf(d[i], x.sb[f], acc[f][i]) : acc[f][i] + d[i];
      acc[f][i] = x.mine ? v : acc[f][i];
    }
  }
}

// Loads of weight rows row[f] .. row[f] + 15 of expert e, K block b; none if !on.
template <bool FP8, int RF, int HT>
__device__ __forceinline__ void load_weights(const Weights<FP8>& W, int e, const int (&row)[RF], int b, bool on,
                                             int lane, Step<FP8, RF, HT>& x) {
  const int r = lane & 15, g = lane >> 4;
  const auto rq = rsrc_of(W.q + e * W.q_bytes, W.q_bytes);
  const uint32_t off = on ? 0 : kNowhere;
  if constexpr (FP8) {
    const int left = W.K - b * 128;
    const uint32_t lo = 16 * g < left ? off : kNowhere, hi = 64 + 16 * g < left ? off : kNowhere;
    const uint32_t at = (uint32_t)r * (uint32_t)W.K + 16 * g;
#pragma unroll
    for (int f = 0; f < RF; ++f) {
      const int so = on ? row[f] * W.K + b * 128 : 0;
      x.w[f][0] = __builtin_amdgcn_raw_buffer_load_b128(rq, at | lo, so, 2);
      x.w[f][1] = __builtin_amdgcn_raw_buffer_load_b128(rq, (at + 64) | hi, so, 2);
      const float* s = reinterpret_cast<const float*>(W.sf + e * W.sf_bytes) + (row[f] / 128) * W.KB + b;
      x.sb[f] = uniform_load(on ? s : &kNoScale);
    }
  } else {
    const auto rs = rsrc_of(W.sf + e * W.sf_bytes, W.sf_bytes);
#pragma unroll
    for (int f = 0; f < RF; ++f) {
      const int at = on ? ((row[f] / NVFP4_PACK_ROWS) * W.KB + b) * NVFP4_PACK_ROWS + row[f] % NVFP4_PACK_ROWS : 0;
      x.w[f][0] = __builtin_amdgcn_raw_buffer_load_b128(rq, (uint32_t)(64 * r + 16 * g) | off, at * 64, 2);
      x.s[f] = __builtin_amdgcn_raw_buffer_load_b16(rs, (uint32_t)(8 * r + 2 * g) | off, at * 8, 2);
    }
  }
}

// Loads of 32 columns of a token's row that starts at byte `row` of the resource.
template <bool FP8>
__device__ __forceinline__ void load_tokens(__amdgpu_buffer_rsrc_t rt, uint32_t row, int K, int b, bool on, int lane,
                                            int4v (&t)[4]) {
  const int g = lane >> 4;
#pragma unroll
  for (int m = 0; m < 4; ++m) {
    const int col = FP8 ? 16 * g + 8 * (m & 1) + 64 * (m >> 1) : 32 * g + 8 * m;
    const bool in = on && b * 128 + col < K;
    t[m] = __builtin_amdgcn_raw_buffer_load_b128(rt, in ? row + 2 * (b * 128 + col) : kNowhere, 0, 0);
  }
}

// barrier without a fence: the loads in flight stay there
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// UP: tile i is 16 columns of h of one live expert (their gate and up rows);
// !UP: 16 columns of out, over all live experts.
template <bool FP8, bool UP>
__global__ __launch_bounds__(kThreads, 2) void few_kernel(FewArgs p) {
  constexpr int RF = UP ? 2 : 1, HT = UP ? 1 : 2, kDepth = 4, kStride = 16 * RF + 4;
  __shared__ Live L;
  __shared__ union {
    LiveScratch build;
    float red[2][kWaves][16][kStride];
  } S;
  build_live(p, L, S.build);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int n = __builtin_amdgcn_readfirstlane(L.n), stride = gridDim.x;
  const auto W = UP ? weights_of<FP8>(p.w1_q, p.w1_sf, 2 * p.I, p.H) : weights_of<FP8>(p.w2_q, p.w2_sf, p.H, p.I);
  const int per = (int)(p.I / 16);                       // UP: tiles of an expert
  const int tiles = UP ? n * per : (int)(p.H / 16);
  if ((int)blockIdx.x >= tiles) return;
  const int blocks = UP ? W.KB : n * W.KB;
  const int steps = blocks > kWaves ? (blocks + kWaves - 1) / kWaves : 1;
  const int total = ((tiles - 1 - (int)blockIdx.x) / stride + 1) * steps;
  const int64_t h_bytes = (int64_t)p.T * p.k * p.I * 2;
  const auto rx = rsrc_of(UP ? p.x : p.h_hi, UP ? (int64_t)p.T * p.H * 2 : h_bytes);
  const auto rl = rsrc_of(UP ? nullptr : p.h_lo, UP ? 0 : h_bytes);

  // where the loads are: step s of tile i, K block b of the list's expert u
  struct {
    int i, s, u, b, e, mask, first;
    int row[RF];
  } at;
  auto set_expert = [&]() {
    const int u = at.u < n ? at.u : 0;
    at.e = __builtin_amdgcn_readfirstlane(L.e[u]);
    at.mask = __builtin_amdgcn_readfirstlane(L.mask[u]);
    at.first = __builtin_amdgcn_readfirstlane(L.row[u]);
  };
  auto set_tile = [&]() {
    at.s = 0;
    if constexpr (UP) {
      at.u = at.i / per;
      at.b = wave;
      const int c = 16 * (at.i - at.u * per);
      at.row[0] = FP8 ? c : 2 * c;
      at.row[1] = FP8 ? (int)p.I + c : 2 * c + 16;
    } else {
      at.u = wave / W.KB;
      at.b = wave - at.u * W.KB;
      at.row[0] = 16 * at.i;
    }
    set_expert();
  };
  auto issue = [&](Step<FP8, RF, HT>& x) {
    const bool on = at.i < tiles && (UP ? at.b < W.KB : at.u < n);
    load_weights<FP8, RF, HT>(W, at.e, at.row, at.b, on, lane, x);
    const bool mine = x.mine = on && (at.mask >> r & 1);
    const int row = UP ? r : at.first + __popc(at.mask & ((1 << r) - 1));
    const uint32_t byte = (uint32_t)row * (uint32_t)W.K * 2;
    load_tokens<FP8>(rx, byte, W.K, at.b, mine, lane, x.t[0]);
    if constexpr (!UP) load_tokens<FP8>(rl, byte, W.K, at.b, mine, lane, x.t[HT - 1]);
    asm volatile("" ::: "memory");                       // issued here, not where they are used
    if (++at.s == steps) {
      at.i += stride;
      set_tile();
    } else {
      at.b += kWaves;
      if constexpr (!UP) {
        if (at.b >= W.KB) {
          do { at.b -= W.KB; ++at.u; } while (at.b >= W.KB);
          set_expert();
        }
      }
    }
  };

  float4v acc[RF];
#pragma unroll
  for (int f = 0; f < RF; ++f) acc[f] = float4v{0, 0, 0, 0};
  int flip = 0;
  auto finish = [&](int i) {
    auto& red = S.red[flip];
    flip ^= 1;
#pragma unroll
    for (int f = 0; f < RF; ++f) {
      *reinterpret_cast<float4v*>(&red[wave][r][16 * f + 4 * g]) = acc[f];
      acc[f] = float4v{0, 0, 0, 0};
    }
    lds_barrier();
    const int tok = threadIdx.x >> 4, c = threadIdx.x & 15;
    if constexpr (UP) {
      const int u = i / per, mask = L.mask[u];
      if (threadIdx.x < 256 && (mask >> tok & 1)) {
        const int e = L.e[u], gate = FP8 ? c : 16 * (c >> 3) + (c & 7), up = gate + (FP8 ? 16 : 8);
        float a = 0.0f, b = 0.0f, coef = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
          a += red[w][tok][gate];
          b += red[w][tok][up];
        }
        for (int j = 0; j < p.k; ++j) coef += L.id[tok * p.k + j] == e ? L.w[tok * p.k + j] : 0.0f;
        if constexpr (!FP8) {
          const float g1 = p.gs_w1[e];
          a /= g1;
          b /= g1;
          coef /= p.gs_w2[e];
        }
        const float h = a / (1.0f + expf(-a)) * b * coef;
        const uint32_t hi = pack_bf16x2(h, 0.0f);
        const float rest = h - bf16_to_f32(hi & 0xFFFFu);
        const int64_t at_h = (int64_t)(L.row[u] + __popc(mask & ((1 << tok) - 1))) * p.I + 16 * (i - u * per) + c;
        p.h_hi[at_h] = (uint16_t)hi;
        p.h_lo[at_h] = (uint16_t)pack_bf16x2(rest - rest == 0.0f ? rest : 0.0f, 0.0f);
      }
    } else {
      if (tok < p.T) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) v += red[w][tok][c];
        p.out[(int64_t)tok * p.H + 16 * i + c] = (uint16_t)pack_bf16x2(v, 0.0f);
      }
    }
  };

  at.i = blockIdx.x;
  set_tile();
  lds_barrier();                                         // the list's scratch becomes the sums' place
  Step<FP8, RF, HT> x[kDepth];
#pragma unroll
  for (int d = 0; d < kDepth; ++d) issue(x[d]);
  int i = blockIdx.x, s = 0;
  for (int q = 0; q < total; q += kDepth) {
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      add_step<FP8, RF, HT>(acc, x[d]);
      issue(x[d]);
      if (++s == steps && i < tiles) {
        finish(i);
        i += stride;
        s = 0;
      }
    }
  }
}

template <bool FP8>
hipError_t launch(const FewArgs& a, int cus, hipStream_t stream) {
  const int64_t pairs = (int64_t)a.T * a.k, live = pairs < a.E ? pairs : a.E, up = live * (a.I / 16), down = a.H / 16;
  few_kernel<FP8, true><<<(unsigned)(up < cus ? up : cus), kThreads, 0, stream>>>(a);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  few_kernel<FP8, false><<<(unsigned)(down < 2 * cus ? down : 2 * cus), kThreads, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_few(const FewArgs& a, hipStream_t stream) {
  int cus = 0;
  const hipError_t err = device_cus(cus);
  if (err != hipSuccess) return err;
  return a.fp8 ? launch<true>(a, cus, stream) : launch<false>(a, cus, stream);
}

}  // namespace nvfp4
