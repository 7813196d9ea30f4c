// Expert-grouped (or dense) product of FP8 operands with a scale for each
// block of 128 (gfx950).
//
// For row d of expert e, with A row s = a_row_src[d] / a_row_div (or d):
//   c[d][n] = bf16( sum_b a_sf[s][b] * b_sf[e][n/128][b]
//                       * sum_{k in block b} a[s][k] * w[e][n][k] ),
// codes OCP E4M3.  One v_mfma_f32_16x16x128_f8f6f4 is exactly one 128-wide
// scale block of 16 weight rows and 16 tokens: it runs from a zero C operand
// and its four results per lane are scaled and added to fp32 accumulators
// (weight rows are the MFMA's rows, tokens its columns, so the token's scale
// is one value per lane and the weight block's scale is uniform).
#include <atomic>

#include "internal.hpp"
#include "device.hpp"

namespace nvfp4 {

namespace {

typedef int int8v __attribute__((ext_vector_type(8)));
typedef int int4v __attribute__((ext_vector_type(4)));
typedef float float4v __attribute__((ext_vector_type(4)));

struct Fp8Params {
  const uint8_t* a_q;
  const float* a_sf;
  int64_t rows_a;
  const int32_t* a_row_src;   // nullptr: row d
  int a_row_div;
  const int32_t* offsets;     // nullptr: one expert, rows 0..M-1
  int E;
  int64_t M, N;
  int K, KB, NB;              // KB, NB: scale blocks along K and N
  const uint8_t* b_q;
  const float* b_sf;
  uint16_t* c;
  int n_groups;
};

// A byte offset with this bit set lies behind every resource below (they all
// hold less than 2^31 bytes): the load returns zeros and touches no memory.
constexpr uint32_t kNowhere = 0x80000000u;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc_of(const void* base, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, 0x00020000);
}

// Wave-uniform read through the constant address space (a scalar load); only
// for arrays the kernel does not write.
__device__ __forceinline__ float uniform_load(const float* p, int i) {
  return ((const __attribute__((address_space(4))) float*)p)[i];
}

// Rows of one m tile: expert e, rows row0 .. row0 + nrows - 1 of the grouped
// operand (nrows <= BM).
struct RowTile {
  int e, nrows;
  int64_t row0;
};

// The mt-th tile of BM rows in expert order; false if there are fewer.  Lane
// l scans expert e0 + l, 64 experts at a time.
template <int BM>
__device__ __forceinline__ bool row_tile(const Fp8Params& p, int mt, RowTile& t) {
  if (!p.offsets) {
    t.e = 0;
    t.row0 = (int64_t)mt * BM;
    const int64_t left = p.M - t.row0;
    t.nrows = (int)(left < BM ? left : BM);
    return left > 0;
  }
  const int lane = threadIdx.x & 63;
  int before = 0;
  for (int e0 = 0; e0 < p.E; e0 += 64) {
    const int e = e0 + lane;
    const int lo = p.offsets[e < p.E ? e : p.E], hi = p.offsets[e < p.E ? e + 1 : p.E];
    const int tiles = hi > lo ? (hi - lo + BM - 1) / BM : 0;
    int incl = tiles;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int v = __shfl_up(incl, o);
      incl += lane >= o ? v : 0;
    }
    const int total = __builtin_amdgcn_readlane(incl, 63);
    if (mt < before + total) {
      const int src = __ffsll((unsigned long long)__ballot(before + incl > mt)) - 1;
      const int first = __builtin_amdgcn_readlane(lo, src) +
                        (mt - before - (__builtin_amdgcn_readlane(incl, src) -
                                        __builtin_amdgcn_readlane(tiles, src))) * BM;
      int left = __builtin_amdgcn_readlane(hi, src) - first;
      if ((int64_t)first + left > p.M) left = (int)(p.M - first);
      t.e = e0 + src;
      t.row0 = first;
      t.nrows = left < BM ? left : BM;
      return t.nrows > 0;
    }
    before += total;
  }
  return false;
}

// A row of tile row i, or -1 (behind the tile, or an index outside A)
__device__ __forceinline__ int64_t a_row(const Fp8Params& p, const RowTile& t, int i) {
  if (i >= t.nrows) return -1;
  int64_t r = t.row0 + i;
  if (p.a_row_src) r = p.a_row_src[r] / p.a_row_div;
  return r >= 0 && r < p.rows_a ? r : -1;
}

__device__ __forceinline__ float4v mfma_block(const int8v& w, const int8v& t) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, t, float4v{0, 0, 0, 0}, 0, 0, 0, 0, 0, 0);
}

// ------------------------------------------------------------ few rows
//
// 64 weight rows x up to 16*JT tokens per workgroup.  Weights are read once
// and by one wave only, so they go straight to registers; the eight waves
// split the K blocks (block b to wave b % 8, so the workgroup reads 1 KiB
// runs of each weight row) and join through LDS in wave order.

constexpr int kSkWaves = 8;
constexpr int kSkRows = 64;
constexpr int kSkStride = kSkRows + 4;      // LDS floats per token

template <int JT>
struct SkFrag {
  int8v w[4], t[JT];
  float s[JT], sb;
};

__device__ __forceinline__ int8v join(const int4v& lo, const int4v& hi) {
  return int8v{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
}

template <int JT>
__global__ __launch_bounds__(kSkWaves * 64) void fp8_skinny_kernel(Fp8Params p) {
  __shared__ float red[kSkWaves][16][kSkStride];
  const int mt = blockIdx.x / p.n_groups, ng = blockIdx.x - mt * p.n_groups;
  RowTile t;
  if (!row_tile<16 * JT>(p, mt, t)) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int64_t n0 = (int64_t)ng * kSkRows;
  const int64_t K = p.K;

  // without a gather the resource starts at the tile's first row, so offsets
  // stay small whatever M is; with one A holds less than 2 GiB
  const int64_t a_base = p.a_row_src ? 0 : t.row0;
  const int64_t a_rows = p.a_row_src ? p.rows_a : t.nrows;
  const auto ra = rsrc_of(p.a_q + a_base * K, a_rows * K);
  const auto rs = rsrc_of(p.a_sf + a_base * p.KB, a_rows * p.KB * 4);
  const auto rb = rsrc_of(p.b_q + (int64_t)t.e * p.N * K, p.N * K);
  const float* bsf = p.b_sf + ((int64_t)t.e * p.NB + n0 / 128) * p.KB;

  uint32_t wo[4], to[JT], so[JT];
#pragma unroll
  for (int f = 0; f < 4; ++f) {
    const int64_t n = n0 + 16 * f + r;
    wo[f] = n < p.N ? (uint32_t)(n * K) + 16 * g : kNowhere;
  }
#pragma unroll
  for (int j = 0; j < JT; ++j) {
    const int64_t row = a_row(p, t, 16 * j + r);
    to[j] = row >= 0 ? (uint32_t)((row - a_base) * K) + 16 * g : kNowhere;
    so[j] = row >= 0 ? (uint32_t)((row - a_base) * p.KB * 4) : kNowhere;
  }
  // columns behind K in the last block: 16-byte chunk g and chunk 4 + g
  const int tail = p.K - (p.KB - 1) * 128;
  const uint32_t cut_lo = 16 * g < tail ? 0 : kNowhere, cut_hi = 64 + 16 * g < tail ? 0 : kNowhere;

  float4v acc[4][JT];
#pragma unroll
  for (int f = 0; f < 4; ++f)
#pragma unroll
    for (int j = 0; j < JT; ++j) acc[f][j] = float4v{0, 0, 0, 0};

  auto load = [&](int b, SkFrag<JT>& x) {
    const bool none = b >= p.KB, last = b == p.KB - 1;
    const uint32_t lo = none ? kNowhere : last ? cut_lo : 0, hi = none ? kNowhere : last ? cut_hi : 0;
    const int at = none ? 0 : b * 128;
#pragma unroll
    for (int f = 0; f < 4; ++f)
      x.w[f] = join(__builtin_amdgcn_raw_buffer_load_b128(rb, wo[f] | lo, at, 2),
                    __builtin_amdgcn_raw_buffer_load_b128(rb, (wo[f] + 64) | hi, at, 2));
#pragma unroll
    for (int j = 0; j < JT; ++j) {
      x.t[j] = join(__builtin_amdgcn_raw_buffer_load_b128(ra, to[j] | lo, at, 0),
                    __builtin_amdgcn_raw_buffer_load_b128(ra, (to[j] + 64) | hi, at, 0));
      x.s[j] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rs, so[j] | (none ? kNowhere : 0), none ? 0 : b * 4, 0));
    }
    x.sb = bsf[none ? 0 : b];
  };
  auto add = [&](const SkFrag<JT>& x) {
#pragma unroll
    for (int j = 0; j < JT; ++j) {
      const float s = x.s[j] * x.sb;
#pragma unroll
      for (int f = 0; f < 4; ++f) {
        const float4v d = mfma_block(x.w[f], x.t[j]);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[f][j][i] = fmaf(d[i], s, acc[f][j][i]);
      }
    }
  };
  SkFrag<JT> x0, x1;
  load(wave, x0);
  for (int b = wave; b < p.KB; b += 2 * kSkWaves) {
    load(b + kSkWaves, x1);
    add(x0);
    load(b + 2 * kSkWaves, x0);
    add(x1);
  }

  const int tok = threadIdx.x >> 5, n2 = (threadIdx.x & 31) * 2;
#pragma unroll
  for (int j = 0; j < JT; ++j) {
    if (16 * j >= t.nrows) break;
    if (j) __syncthreads();
#pragma unroll
    for (int f = 0; f < 4; ++f)
      *reinterpret_cast<float4v*>(&red[wave][r][16 * f + 4 * g]) = acc[f][j];
    __syncthreads();
    float v0 = 0.0f, v1 = 0.0f;
#pragma unroll
    for (int w = 0; w < kSkWaves; ++w) {
      const float2 v = *reinterpret_cast<const float2*>(&red[w][tok][n2]);
      v0 += v.x;
      v1 += v.y;
    }
    if (16 * j + tok < t.nrows && n0 + n2 < p.N) {
      uint16_t* dst = p.c + (t.row0 + 16 * j + tok) * p.N + n0 + n2;
      const uint32_t o = pack_bf16x2(v0, v1);
      if (p.N % 2 == 0) {
        *reinterpret_cast<uint32_t*>(dst) = o;
      } else {
        dst[0] = (uint16_t)o;
        if (n0 + n2 + 1 < p.N) dst[1] = (uint16_t)(o >> 16);
      }
    }
  }
}

// ------------------------------------------------------------ many rows
//
// 256 weight rows x up to 256 tokens per workgroup of eight waves (4 along N,
// 2 along the tokens); a wave holds 64 weight rows x 16*JV tokens, JV the
// 32-token blocks that the tile's rows fill.  Stages of one K block go from
// HBM straight to LDS, double-buffered; 16-byte chunk q of a row lies at place
// q ^ ((row >> 1) & 7), so the sixteen rows of a fragment read spread over all
// banks.

constexpr int kTlWaves = 8;
constexpr int kTlN = 256, kTlM = 256;
constexpr int kTlTok = kTlN * 128;                    // LDS offsets in a stage: tokens,
constexpr int kTlSf = kTlTok + kTlM * 128;            // token scales
constexpr int kTlStage = kTlSf + kTlWaves * 64 * 4;   // (the upper four waves' scales are zeros)
constexpr int kTlEpiStride = 64 * 2 + 16;             // LDS bytes per staged token row

typedef __attribute__((address_space(3))) void* lds_ptr_t;
__device__ __forceinline__ lds_ptr_t lds_addr(const uint8_t* p) {
  return (lds_ptr_t)(uint32_t)(uintptr_t)p;
}

// barrier without a fence: every wait it needs is written out
__device__ __forceinline__ void bare_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

struct TlLoads {
  __amdgpu_buffer_rsrc_t ra, rs, rb;
  uint32_t wo[4], to[4], so;      // byte offsets of this lane's chunks and scale
  uint32_t cut;                   // kNowhere if the lane's chunk lies behind K in the last block
};

// Direct loads of K block b into `dst`; zeros for a block behind the last.  No
// branch: code would move across it and out of the order the stage is written in.
template <int JV>
__device__ __forceinline__ void tl_issue(const TlLoads& L, int b, int KB, int wave, uint8_t* __restrict__ dst) {
  const uint32_t cut = b < KB - 1 ? 0 : b == KB - 1 ? L.cut : kNowhere;
  const int at = b < KB ? b * 128 : 0;
#pragma unroll
  for (int c = 0; c < 4; ++c)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(L.rb, lds_addr(dst + (wave + 8 * c) * 1024), 16, L.wo[c] | cut, at, 0, 0);
#pragma unroll
  for (int c = 0; c < (JV + 1) / 2; ++c)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(L.ra, lds_addr(dst + kTlTok + (wave + 8 * c) * 1024), 16, L.to[c] | cut, at, 0, 0);
  __builtin_amdgcn_raw_ptr_buffer_load_lds(L.rs, lds_addr(dst + kTlSf + wave * 256), 4, L.so | (b < KB ? 0 : kNowhere), b < KB ? b * 4 : 0, 0, 0);
}

__device__ __forceinline__ int8v tl_frag(const uint8_t* row, int at0, int at1) {
  return join(*reinterpret_cast<const int4v*>(row + at0), *reinterpret_cast<const int4v*>(row + at1));
}

// One stage: the loads of block b + 1 into nxt, the products of block b from cur.
template <int JV>
__device__ __forceinline__ void tl_stage(float4v (&acc)[4][JV], const TlLoads& L, int b, int KB, int wave,
                                         int lane, float sb, const uint8_t* __restrict__ cur,
                                         uint8_t* __restrict__ nxt) {
  const int r = lane & 15, g = lane >> 4, wn = wave >> 1, wt = wave & 1;
  tl_issue<JV>(L, b + 1, KB, wave, nxt);
  const int at0 = (g ^ ((r >> 1) & 7)) * 16, at1 = ((4 + g) ^ ((r >> 1) & 7)) * 16;
  int8v w[4];
#pragma unroll
  for (int f = 0; f < 4; ++f) w[f] = tl_frag(cur + (wn * 64 + 16 * f + r) * 128, at0, at1);
  const uint8_t* tok = cur + kTlTok + (wt * 16 + r) * 128;
  const uint8_t* sfs = cur + kTlSf + (wt * 16 + r) * 4;
  int8v t = tl_frag(tok, at0, at1);
  float s = *reinterpret_cast<const float*>(sfs) * sb;
  float4v dp[4];                       // products of the block before, not yet added
  float sp = 0.0f;
  // Per token block: its four products, the next block's operands, and the
  // scaling of the block before, which needs no wait on the matrix unit.
#pragma unroll
  for (int j = 0; j < JV; ++j) {
    int8v tn = t;
    float sn = 0.0f;
    if (j + 1 < JV) {
      tn = tl_frag(tok + (j + 1) * 4096, at0, at1);
      sn = *reinterpret_cast<const float*>(sfs + (j + 1) * 128) * sb;
    }
    float4v d[4];
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      d[f] = mfma_block(w[f], t);
      if (j > 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[f][j - 1][i] = fmaf(dp[f][i], sp, acc[f][j - 1][i]);
      }
    }
#pragma unroll
    for (int f = 0; f < 4; ++f) dp[f] = d[f];
    t = tn;
    sp = s;
    s = sn;
    __builtin_amdgcn_sched_barrier(0);
  }
#pragma unroll
  for (int f = 0; f < 4; ++f)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[f][JV - 1][i] = fmaf(dp[f][i], sp, acc[f][JV - 1][i]);
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  bare_barrier();
}

template <int JV>
__device__ __forceinline__ void tl_run(const Fp8Params& p, const RowTile& t, int64_t n0, const TlLoads& L,
                                       int wave, int lane, uint8_t* __restrict__ buf0, uint8_t* __restrict__ buf1) {
  const int r = lane & 15, g = lane >> 4, wn = wave >> 1, wt = wave & 1;
  float4v acc[4][JV];
#pragma unroll
  for (int f = 0; f < 4; ++f)
#pragma unroll
    for (int j = 0; j < JV; ++j) acc[f][j] = float4v{0, 0, 0, 0};
  int nb = (int)((n0 + wn * 64) / 128);
  if (nb >= p.NB) nb = p.NB - 1;
  const float* bsf = p.b_sf + ((int64_t)t.e * p.NB + nb) * p.KB;
  tl_issue<JV>(L, 0, p.KB, wave, buf0);
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  bare_barrier();
  // an odd number of blocks runs one more of zeros
  for (int b = 0; b < p.KB; b += 2) {
    tl_stage<JV>(acc, L, b, p.KB, wave, lane, uniform_load(bsf, b), buf0, buf1);
    tl_stage<JV>(acc, L, b + 1, p.KB, wave, lane, uniform_load(bsf, b + 1 < p.KB ? b + 1 : b), buf1, buf0);
  }
  // BF16 through LDS (a region per wave): a lane holds four consecutive
  // columns of one token, the stores want sixteen bytes of a token's row
  uint8_t* ep = buf0 + wave * (16 * kTlEpiStride);
  const bool vec = p.N % 8 == 0 && (reinterpret_cast<uintptr_t>(p.c) & 15) == 0;
  const int64_t nw = n0 + wn * 64;
#pragma unroll
  for (int j = 0; j < JV; ++j) {
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      uint2 o;
      o.x = pack_bf16x2(acc[f][j][0], acc[f][j][1]);
      o.y = pack_bf16x2(acc[f][j][2], acc[f][j][3]);
      *reinterpret_cast<uint2*>(ep + r * kTlEpiStride + 2 * (16 * f + 4 * g)) = o;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int tok = 8 * h + (lane >> 3), ch = lane & 7;
      const uint4 v = *reinterpret_cast<const uint4*>(ep + tok * kTlEpiStride + 16 * ch);
      const int row = (2 * j + wt) * 16 + tok;
      const int64_t n = nw + 8 * ch;
      if (row < t.nrows && n < p.N) {
        uint16_t* dst = p.c + (t.row0 + row) * p.N + n;
        if (vec) {
          *reinterpret_cast<uint4*>(dst) = v;
        } else {
          const uint32_t q[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (n + i < p.N) dst[i] = (uint16_t)(q[i >> 1] >> (16 * (i & 1)));
        }
      }
    }
  }
}

__global__ __launch_bounds__(kTlWaves * 64, 2) void fp8_tile_kernel(Fp8Params p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const int mt = blockIdx.x / p.n_groups, ng = blockIdx.x - mt * p.n_groups;
  RowTile t;
  if (!row_tile<kTlM>(p, mt, t)) return;
  t.e = __builtin_amdgcn_readfirstlane(t.e);
  t.nrows = __builtin_amdgcn_readfirstlane(t.nrows);
  t.row0 = __builtin_amdgcn_readfirstlane((int)t.row0);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t n0 = (int64_t)ng * kTlN, K = p.K;
  const int64_t a_base = p.a_row_src ? 0 : t.row0;
  const int64_t a_rows = p.a_row_src ? p.rows_a : t.nrows;
  TlLoads L;
  L.ra = rsrc_of(p.a_q + a_base * K, a_rows * K);
  L.rs = rsrc_of(p.a_sf + a_base * p.KB, a_rows * p.KB * 4);
  L.rb = rsrc_of(p.b_q + (int64_t)t.e * p.N * K, p.N * K);
  const int q = (lane & 7) ^ ((4 * wave + (lane >> 4)) & 7);
  const int tail = p.K - (p.KB - 1) * 128;
  L.cut = 16 * q < tail ? 0 : kNowhere;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const int row = (wave + 8 * c) * 8 + (lane >> 3);
    const int64_t n = n0 + row;
    L.wo[c] = n < p.N ? (uint32_t)(n * K) + 16 * q : kNowhere;
    const int64_t ar = a_row(p, t, row);
    L.to[c] = ar >= 0 ? (uint32_t)((ar - a_base) * K) + 16 * q : kNowhere;
  }
  {
    const int64_t ar = wave < 4 ? a_row(p, t, wave * 64 + lane) : -1;
    L.so = ar >= 0 ? (uint32_t)((ar - a_base) * p.KB * 4) : kNowhere;
  }
  uint8_t *b0 = smem, *b1 = smem + kTlStage;
  switch ((t.nrows + 31) / 32) {
    case 1: tl_run<1>(p, t, n0, L, wave, lane, b0, b1); break;
    case 2: tl_run<2>(p, t, n0, L, wave, lane, b0, b1); break;
    case 3: tl_run<3>(p, t, n0, L, wave, lane, b0, b1); break;
    case 4: tl_run<4>(p, t, n0, L, wave, lane, b0, b1); break;
    case 5: tl_run<5>(p, t, n0, L, wave, lane, b0, b1); break;
    case 6: tl_run<6>(p, t, n0, L, wave, lane, b0, b1); break;
    case 7: tl_run<7>(p, t, n0, L, wave, lane, b0, b1); break;
    default: tl_run<8>(p, t, n0, L, wave, lane, b0, b1); break;
  }
}

// m tiles of at most bm rows that E experts with M rows in all can need
int64_t tile_bound(const Fp8GemmArgs& a, int bm) {
  if (!a.offsets) return (a.M + bm - 1) / bm;
  const int64_t b = (a.M + (int64_t)a.E * (bm - 1)) / bm;
  return b < a.M ? b : a.M;
}

template <int JT>
hipError_t launch_skinny(const Fp8GemmArgs& a, Fp8Params p, hipStream_t stream) {
  p.n_groups = (int)((a.N + kSkRows - 1) / kSkRows);
  const int64_t grid = tile_bound(a, 16 * JT) * p.n_groups;
  if (grid >= (int64_t(1) << 31)) return hipErrorInvalidConfiguration;
  fp8_skinny_kernel<JT><<<(unsigned)grid, kSkWaves * 64, 0, stream>>>(p);
  return hipGetLastError();
}

constexpr int kMaxDevices = 64;

hipError_t launch_tile(const Fp8GemmArgs& a, Fp8Params p, hipStream_t stream) {
  p.n_groups = (int)((a.N + kTlN - 1) / kTlN);
  const int64_t grid = tile_bound(a, kTlM) * p.n_groups;
  if (grid >= (int64_t(1) << 31)) return hipErrorInvalidConfiguration;
  int dev = 0;
  hipError_t err = hipGetDevice(&dev);
  if (err != hipSuccess) return err;
  if (dev < 0 || dev >= kMaxDevices) return hipErrorInvalidDevice;
  static std::atomic<bool> attr_set[kMaxDevices];
  if (!attr_set[dev].load(std::memory_order_relaxed)) {
    err = hipFuncSetAttribute(reinterpret_cast<const void*>(fp8_tile_kernel),
                              hipFuncAttributeMaxDynamicSharedMemorySize, 2 * kTlStage);
    if (err != hipSuccess) return err;
    attr_set[dev].store(true, std::memory_order_relaxed);
  }
  fp8_tile_kernel<<<(unsigned)grid, kTlWaves * 64, 2 * kTlStage, stream>>>(p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_fp8_gemm(const Fp8GemmArgs& a, hipStream_t stream) {
  Fp8Params p;
  p.a_q = a.a_q; p.a_sf = a.a_sf; p.rows_a = a.rows_a; p.a_row_src = a.a_row_src;
  p.a_row_div = a.a_row_div; p.offsets = a.offsets; p.E = a.E; p.M = a.M; p.N = a.N;
  p.K = (int)a.K; p.KB = (int)((a.K + 127) / 128); p.NB = (int)((a.N + 127) / 128);
  p.b_q = a.b_q; p.b_sf = a.b_sf; p.c = static_cast<uint16_t*>(a.c);
  p.n_groups = 0;
  if (a.M <= 16 * (int64_t)a.E) return launch_skinny<1>(a, p, stream);
  if (a.M <= 32 * (int64_t)a.E) return launch_skinny<2>(a, p, stream);
  if (a.M <= 64 * (int64_t)a.E) return launch_skinny<4>(a, p, stream);
  return launch_tile(a, p, stream);
}

}  // namespace nvfp4
