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
//
// Rounding inside the instruction: the products of eight consecutive k are
// added in fixed point aligned to the largest of them, with 13 bits below it
// kept; the eights' sums, and everything after them, are fp32.  A product so
// loses less than 2^-13 of the largest of its eight.  On data of one size this
// stays an order of magnitude below the BF16 rounding of c, and the codes
// themselves are off by up to 2^-4, so no slower instruction is taken for it.
#include <atomic>
#include <cmath>

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
  int n_groups;               // n tiles
  int bm;                     // rows of an m tile at most (tile kernel)
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

__device__ const float kNoScale = 0.0f;

// Rows of one m tile: expert e, rows row0 .. row0 + nrows - 1 of the grouped
// operand (nrows <= BM).
struct RowTile {
  int e, nrows;
  int64_t row0;
};

// Tile i of the tiles of at most bm rows that `rows` (> 0) rows from `first` on
// are cut into.  Up to 2^31 - 1 rows, so sizes are rounded up without a sum that
// passes them.  The tiles take even shares of the 32-row blocks: 300 rows are
// 160 and 140, not 288 and 12, whose second tile would stream the whole
// weight tile for a twelfth of the work.
__host__ __device__ __forceinline__ bool cut_tile(const Fp8Params& p, int bm, int first, int rows, int i, RowTile& t) {
  const int unit = bm % 32 ? bm : 32;
  const int n = (rows - 1) / bm + 1;
  const int units = (rows - 1) / unit + 1, per = units / n, more = units - per * n;
  const int at = (per * i + (i < more ? i : more)) * unit, size = (per + (i < more ? 1 : 0)) * unit;
  int left = rows - at < size ? rows - at : size;
  t.row0 = (int64_t)first + at;
  if (t.row0 + left > p.M) left = (int)(p.M - t.row0);
  t.nrows = left;
  return left > 0 && t.row0 >= 0;
}

// Wave-wide sum of v over the lanes up to this one.
__device__ __forceinline__ int scan64(int v) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int u = __shfl_up(v, o);
    v += lane >= o ? u : 0;
  }
  return v;
}

// The m tiles of at most bm rows, in expert order: first count() their number,
// then find() the mt-th.  Lane l counts the tiles of the S = ceil(E / 64)
// experts from l * S on (independent loads, one scan); find() then scans the
// S experts of the lane that holds the tile.
struct TileList {
  int S, incl, own;

  __host__ __device__ __forceinline__ static int tiles(int lo, int hi, int bm) {
    return hi > lo ? (hi - lo - 1) / bm + 1 : 0;
  }
  __device__ __forceinline__ int count(const Fp8Params& p, int bm) {
    if (!p.offsets) return (int)((p.M + bm - 1) / bm);
    S = (p.E + 63) >> 6;
    own = 0;
    const int e0 = (threadIdx.x & 63) * S;
#pragma unroll 4
    for (int i = 0; i < S; ++i) {
      const int e = e0 + i < p.E ? e0 + i : p.E, e1 = e < p.E ? e + 1 : p.E;
      own += tiles(p.offsets[e], p.offsets[e1], bm);
    }
    incl = scan64(own);
    return __builtin_amdgcn_readlane(incl, 63);
  }
  __device__ __forceinline__ bool find(const Fp8Params& p, int bm, int mt, RowTile& t) const {
    if (!p.offsets) {
      t.e = 0;
      if (mt >= (p.M + bm - 1) / bm) return false;
      return cut_tile(p, bm, 0, (int)p.M, mt, t);
    }
    if (mt >= __builtin_amdgcn_readlane(incl, 63)) return false;
    const int at = __ffsll((unsigned long long)__ballot(incl > mt)) - 1;
    int rest = mt - (__builtin_amdgcn_readlane(incl, at) - __builtin_amdgcn_readlane(own, at));
    const int lane = threadIdx.x & 63;
    int e = at * S + lane;
    if (lane >= S || e >= p.E) e = p.E;
    const int lo = p.offsets[e], hi = p.offsets[e < p.E ? e + 1 : p.E], n = tiles(lo, hi, bm);
    const int sum = scan64(n);
    const int src = __ffsll((unsigned long long)__ballot(sum > rest)) - 1;
    rest -= __builtin_amdgcn_readlane(sum, src) - __builtin_amdgcn_readlane(n, src);
    const int first = __builtin_amdgcn_readlane(lo, src);
    t.e = at * S + src;
    return cut_tile(p, bm, first, __builtin_amdgcn_readlane(hi, src) - first, rest, t);
  }
};

__device__ __forceinline__ bool row_tile(const Fp8Params& p, int bm, int mt, RowTile& t) {
  TileList list;
  list.count(p, bm);
  return list.find(p, bm, mt, t);
}

// A row of tile row i, or -1 (behind the tile, or an index outside A)
__device__ __forceinline__ int64_t a_row(const Fp8Params& p, const RowTile& t, int i) {
  if (i >= t.nrows) return -1;
  int64_t r = t.row0 + i;
  if (p.a_row_src) {
    const int s = p.a_row_src[r];
    r = s < 0 ? -1 : s / p.a_row_div;
  }
  return r >= 0 && r < p.rows_a ? r : -1;
}

__device__ __forceinline__ float4v mfma_block(const int8v& w, const int8v& t) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, t, float4v{0, 0, 0, 0}, 0, 0, 0, 0, 0, 0);
}

// ------------------------------------------------------------ few rows
//
// 16*RF weight rows x up to 16*JT tokens per workgroup, for products whose
// tiles would leave most CUs idle.  Weights go straight to registers; the
// eight waves split the K blocks (block b to wave b % 8, so the workgroup reads
// 1 KiB runs of each weight row), D blocks in flight per wave, and join
// through LDS in wave order.  Bound by latency: the fewer rows, the more
// workgroups pull at once.  Measured at K 7168, N 2048: one token 7.1 to 7.4 us
// (14.7 MB: 2.0 TB/s, of which 2.6 us are an empty launch; N 2048 makes 128
// workgroups, half as many as CUs), 512 tokens 36 us.

constexpr int kSkWaves = 8;

template <int RF, int JT>
struct SkFrag {
  int8v w[RF], t[JT];
  float s[JT], sb;
};

__device__ __forceinline__ int8v join(const int4v& lo, const int4v& hi) {
  return int8v{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
}

template <int RF, int JT, int D>
__global__ __launch_bounds__(kSkWaves * 64) void fp8_skinny_kernel(Fp8Params p) {
  constexpr int kRows = 16 * RF, kStride = kRows + 4;
  __shared__ float red[kSkWaves][16][kStride];
  const uint32_t wg = row_workgroup();
  const int mt = wg / p.n_groups, ng = wg - mt * p.n_groups;
  RowTile t;
  if (!row_tile(p, 16 * JT, mt, t)) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int64_t n0 = (int64_t)ng * kRows;
  const int64_t K = p.K;

  // without a gather the resource starts at the tile's first row, so offsets
  // stay small whatever M is; with one A holds less than 2 GiB
  const int64_t a_base = p.a_row_src ? 0 : t.row0;
  const int64_t a_rows = p.a_row_src ? p.rows_a : t.nrows;
  const auto ra = rsrc_of(p.a_q + a_base * K, a_rows * K);
  const auto rs = rsrc_of(p.a_sf + a_base * p.KB, a_rows * p.KB * 4);
  const auto rb = rsrc_of(p.b_q + (int64_t)t.e * p.N * K, p.N * K);
  const float* bsf = p.b_sf + ((int64_t)t.e * p.NB + n0 / 128) * p.KB;

  uint32_t wo[RF], to[JT], so[JT];
#pragma unroll
  for (int f = 0; f < RF; ++f) {
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

  float4v acc[RF][JT];
#pragma unroll
  for (int f = 0; f < RF; ++f)
#pragma unroll
    for (int j = 0; j < JT; ++j) acc[f][j] = float4v{0, 0, 0, 0};

  auto load = [&](int b, SkFrag<RF, JT>& x) {
    const bool last = b == p.KB - 1;
    const uint32_t lo = last ? cut_lo : 0, hi = last ? cut_hi : 0;
#pragma unroll
    for (int f = 0; f < RF; ++f)
      x.w[f] = join(__builtin_amdgcn_raw_buffer_load_b128(rb, wo[f] | lo, b * 128, 0),
                    __builtin_amdgcn_raw_buffer_load_b128(rb, (wo[f] + 64) | hi, b * 128, 0));
#pragma unroll
    for (int j = 0; j < JT; ++j) {
      x.t[j] = join(__builtin_amdgcn_raw_buffer_load_b128(ra, to[j] | lo, b * 128, 0),
                    __builtin_amdgcn_raw_buffer_load_b128(ra, (to[j] + 64) | hi, b * 128, 0));
      x.s[j] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rs, so[j], b * 4, 0));
    }
    x.sb = uniform_load(bsf, b);
    asm volatile("" ::: "memory");      // issued here, not where they are used
  };
  auto add = [&](const SkFrag<RF, JT>& x) {
#pragma unroll
    for (int j = 0; j < JT; ++j) {
      const float s = x.s[j] * x.sb;
#pragma unroll
      for (int f = 0; f < RF; ++f) {
        const float4v d = mfma_block(x.w[f], x.t[j]);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[f][j][i] = fmaf(d[i], s, acc[f][j][i]);
      }
    }
  };
  SkFrag<RF, JT> x[D];
#pragma unroll
  for (int d = 0; d < D; ++d)
    if (wave + kSkWaves * d < p.KB) load(wave + kSkWaves * d, x[d]);
  for (int b = wave; b < p.KB; b += D * kSkWaves) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      if (b + kSkWaves * d < p.KB) add(x[d]);
      if (b + kSkWaves * (d + D) < p.KB) load(b + kSkWaves * (d + D), x[d]);
    }
  }

#pragma unroll
  for (int j = 0; j < JT; ++j) {
    if (16 * j >= t.nrows) break;
    if (j) __syncthreads();
#pragma unroll
    for (int f = 0; f < RF; ++f)
      *reinterpret_cast<float4v*>(&red[wave][r][16 * f + 4 * g]) = acc[f][j];
    __syncthreads();
    for (int o = threadIdx.x; o < 16 * kRows / 2; o += kSkWaves * 64) {
      const int tok = o / (kRows / 2), n2 = o % (kRows / 2) * 2;
      float v0 = 0.0f, v1 = 0.0f;
#pragma unroll
      for (int w = 0; w < kSkWaves; ++w) {
        const float2 v = *reinterpret_cast<const float2*>(&red[w][tok][n2]);
        v0 += v.x;
        v1 += v.y;
      }
      if (16 * j + tok < t.nrows && n0 + n2 < p.N) {
        uint16_t* dst = p.c + (t.row0 + 16 * j + tok) * p.N + n0 + n2;
        const uint32_t q = pack_bf16x2(v0, v1);
        if (p.N % 2 == 0 && (reinterpret_cast<uintptr_t>(p.c) & 3) == 0) {
          *reinterpret_cast<uint32_t*>(dst) = q;
        } else {
          dst[0] = (uint16_t)q;
          if (n0 + n2 + 1 < p.N) dst[1] = (uint16_t)(q >> 16);
        }
      }
    }
  }
}

typedef __attribute__((address_space(3))) void* lds_ptr_t;
__device__ __forceinline__ lds_ptr_t lds_addr(const uint8_t* p) {
  return (lds_ptr_t)(uintptr_t)(uint32_t)(uintptr_t)p;
}

// ------------------------------------------------------------ few rows, many experts
//
// 128 weight rows x up to 16 tokens per workgroup of four waves.  A wave
// streams its own 32 weight rows through a ring of four LDS stages (4 KB of one
// K block each), three stages ahead and past the caches (each weight is read
// once), so no wave waits for another.  The tokens, the same for all waves and
// n tiles, come from L1/L2 straight to registers two stages ahead.
// HBM-bound: what the ring keeps in flight (96 KB a CU at two workgroups) is
// what counts.  Measured: 2048 rows over 256 experts, N 4096, K 7168 in
// 1.12 ms, 6.7 TB/s of weights (such a read alone reaches 7.1).  Chunk q of a row
// lies at place q ^ ((row >> 1) & 7): no bank conflicts in the fragment reads.

constexpr int kStWaves = 4, kStN = 128, kStRing = 4;
constexpr int kStStage = 32 * 128;                    // LDS bytes of a wave's stage

struct StTok {
  int8v t;
  float s;
};

struct StLoads {
  __amdgpu_buffer_rsrc_t ra, rs, rb;
  uint32_t wo[4], to, so;               // byte offsets of this lane's chunks and scales
  uint32_t w_cut[2], t_cut_lo, t_cut_hi;   // kNowhere for chunks behind K in the last block (w: even, odd loads)
  int KB, at0, at1;                     // at0, at1: this lane's fragment chunks in a stage
};

// weights of K block b into dst; zeros behind the last block
template <int POL>
__device__ __forceinline__ void st_load_w(const StLoads& st, int b, uint8_t* dst) {
  const uint32_t c0 = b < st.KB - 1 ? 0 : b == st.KB - 1 ? st.w_cut[0] : kNowhere;
  const uint32_t c1 = b < st.KB - 1 ? 0 : b == st.KB - 1 ? st.w_cut[1] : kNowhere;
#pragma unroll
  for (int c = 0; c < 4; ++c)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(st.rb, lds_addr(dst + c * 1024), 16, st.wo[c] | (c & 1 ? c1 : c0), b < st.KB ? b * 128 : 0, 0, POL);
}

__device__ __forceinline__ void st_load_t(const StLoads& st, int b, StTok& x) {
  const bool none = b >= st.KB, last = b == st.KB - 1;
  const uint32_t lo = none ? kNowhere : last ? st.t_cut_lo : 0, hi = none ? kNowhere : last ? st.t_cut_hi : 0;
  const int at = none ? 0 : b * 128;
  x.t = join(__builtin_amdgcn_raw_buffer_load_b128(st.ra, st.to | lo, at, 0),
             __builtin_amdgcn_raw_buffer_load_b128(st.ra, (st.to + 64) | hi, at, 0));
  x.s = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(st.rs, st.so | (none ? kNowhere : 0), none ? 0 : b * 4, 0));
}

// Stage b: loads of the weights of b + 3 and the tokens of b + 2, products of
// b.  cur and nxt are __restrict__: the fragment reads get no wait on the
// direct loads in flight beyond the one written here.
template <int POL>
__device__ __forceinline__ void st_stage(float4v (&acc)[2], const StLoads& st, int b, float sb, const StTok& x, StTok& ahead, const uint8_t* __restrict__ cur,
                                         uint8_t* __restrict__ nxt) {
  st_load_t(st, b + 2, ahead);
  asm volatile("" ::: "memory");       // the count below relies on this order
  st_load_w<POL>(st, b + 3, nxt);
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"((kStRing - 1) * (4 + 3)) : "memory");
  int8v w[2];
#pragma unroll
  for (int f = 0; f < 2; ++f)
    w[f] = join(*reinterpret_cast<const int4v*>(cur + f * 2048 + st.at0), *reinterpret_cast<const int4v*>(cur + f * 2048 + st.at1));
  const float s = x.s * sb;
#pragma unroll
  for (int f = 0; f < 2; ++f) {
    const float4v d = mfma_block(w[f], x.t);
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[f][i] = fmaf(d[i], s, acc[f][i]);
  }
  // the reads of cur are done before the next stage's loads reuse it
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
}

template <int POL>
__global__ __launch_bounds__(kStWaves * 64, 2) void fp8_stream_kernel(Fp8Params p) {
  __shared__ __align__(1024) uint8_t smem[kStWaves * kStRing * kStStage];
  const uint32_t wg = row_workgroup();
  const int mt = wg / p.n_groups, ng = wg - mt * p.n_groups;
  RowTile t;
  if (!row_tile(p, 16, mt, t)) return;
  t.e = __builtin_amdgcn_readfirstlane(t.e);
  t.nrows = __builtin_amdgcn_readfirstlane(t.nrows);
  t.row0 = __builtin_amdgcn_readfirstlane((int)t.row0);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int64_t n0 = (int64_t)ng * kStN, nw = n0 + wave * 32, K = p.K;
  const int64_t a_base = p.a_row_src ? 0 : t.row0;
  const int64_t a_rows = p.a_row_src ? p.rows_a : t.nrows;
  const float* bsf = p.b_sf + ((int64_t)t.e * p.NB + ng) * p.KB;
  StLoads st;
  float4v acc[2];
  st.ra = rsrc_of(p.a_q + a_base * K, a_rows * K);
  st.rs = rsrc_of(p.a_sf + a_base * p.KB, a_rows * p.KB * 4);
  st.rb = rsrc_of(p.b_q + (int64_t)t.e * p.N * K, p.N * K);
  st.KB = p.KB;
  acc[0] = acc[1] = float4v{0, 0, 0, 0};
  const int tail = p.K - (p.KB - 1) * 128;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const int row = 8 * c + (lane >> 3), q = (lane & 7) ^ ((row >> 1) & 7);
    st.wo[c] = nw + row < p.N ? (uint32_t)((nw + row) * K) + 16 * q : kNowhere;
    if (c < 2) st.w_cut[c] = 16 * q < tail ? 0 : kNowhere;   // rows 16 apart have one chunk order
  }
  const int64_t row = a_row(p, t, r);
  st.to = row >= 0 ? (uint32_t)((row - a_base) * K) + 16 * g : kNowhere;
  st.so = row >= 0 ? (uint32_t)((row - a_base) * p.KB * 4) : kNowhere;
  st.t_cut_lo = 16 * g < tail ? 0 : kNowhere;
  st.t_cut_hi = 64 + 16 * g < tail ? 0 : kNowhere;
  st.at0 = r * 128 + (g ^ ((r >> 1) & 7)) * 16;
  st.at1 = r * 128 + ((4 + g) ^ ((r >> 1) & 7)) * 16;
  uint8_t* ring = smem + wave * (kStRing * kStStage);
  uint8_t *s0 = ring, *s1 = ring + kStStage, *s2 = ring + 2 * kStStage, *s3 = ring + 3 * kStStage;

  StTok x0, x1, x2, x3;
  st_load_w<POL>(st, 0, s0);
  asm volatile("" ::: "memory");
  st_load_t(st, 0, x0);
  asm volatile("" ::: "memory");
  st_load_w<POL>(st, 1, s1);
  asm volatile("" ::: "memory");
  st_load_t(st, 1, x1);
  asm volatile("" ::: "memory");
  st_load_w<POL>(st, 2, s2);
  asm volatile("" ::: "memory");
  // four stages a pass, those behind the last on zeros with scale 0: a block's
  // own may be infinite, and 0 times that no number.  The address is chosen, not
  // the value, which would be waited for here (decode 0.6% slower).
  auto sb = [&](int b) { return uniform_load(b < p.KB ? bsf + b : &kNoScale, 0); };
  for (int b = 0; b < p.KB; b += 4) {
    const float f0 = sb(b), f1 = sb(b + 1), f2 = sb(b + 2), f3 = sb(b + 3);
    st_stage<POL>(acc, st, b, f0, x0, x2, s0, s3);
    st_stage<POL>(acc, st, b + 1, f1, x1, x3, s1, s0);
    st_stage<POL>(acc, st, b + 2, f2, x2, x0, s2, s1);
    st_stage<POL>(acc, st, b + 3, f3, x3, x1, s3, s2);
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  const bool vec = p.N % 4 == 0 && (reinterpret_cast<uintptr_t>(p.c) & 7) == 0;
  if (r >= t.nrows) return;
#pragma unroll
  for (int f = 0; f < 2; ++f) {
    const int64_t n = nw + 16 * f + 4 * g;
    if (n >= p.N) continue;
    uint16_t* dst = p.c + (t.row0 + r) * p.N + n;
    uint2 o;
    o.x = pack_bf16x2(acc[f][0], acc[f][1]);
    o.y = pack_bf16x2(acc[f][2], acc[f][3]);
    if (vec) {
      *reinterpret_cast<uint2*>(dst) = o;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (n + i < p.N) dst[i] = (uint16_t)((i < 2 ? o.x : o.y) >> (16 * (i & 1)));
    }
  }
}

// ------------------------------------------------------------ many rows
//
// 256 weight rows x up to 288 tokens per workgroup of eight waves (4 along N,
// 2 along the tokens); a wave holds 64 weight rows x 16*JV tokens, JV the
// 32-token blocks that the tile's rows fill.  Operands go from HBM straight to
// LDS, where 16-byte chunk q of a row lies at place q ^ ((row >> 1) & 7), so
// the sixteen rows of a fragment read spread over all banks.
//
// A stage is one K block, in JV steps of one token block each.  Its weight
// fragments are in registers before it starts, so its weight buffer is free
// early, and its token buffer in two parts (T1: blocks 0..JH-1, T2: the rest)
// as the steps pass them.  Two barriers a stage hand the parts over:
//   steps 0 .. JH-2      loads of T2 of stage b + 1
//   barrier B            T2 of this stage has landed; weights and T1 are read
//   steps JH-1 .. JV-2   loads of the weights and T1 of stage b + 2
//   barrier S            weights and T1 of stage b + 1 have landed; T2 is read
//   step JV-1            the next stage's fragments replace this one's
// so that two buffers keep a whole stage's loads (72 KB) in flight at every
// wait, and the loads are spread over the stage instead of queueing at its
// start.
//
// Measured: 65536 rows over 256 experts, N 4096, K 7168 in 2.07 to 2.17 ms, 1.8
// PFLOP/s (all of a stage's loads at its start, one barrier, 256-token tiles:
// 2.82); the same rows as 256 in each expert 2.03; dense 2.3 PFLOP/s on random
// codes, 3.1 on zeros.  Bound by power: the
// clock falls to 1.7 GHz on random codes.  The tile's height is what the
// accumulators leave room for: 64 x 144 a wave is 144 of its 256 registers, and
// 288 tokens cover an expert that gets a few rows more than 256 in one tile.

constexpr int kTlWaves = 8;
constexpr int kTlN = 256, kTlM = 288, kTlMin = 96;
constexpr int kTlTokLoads = 5;                        // 64-row token loads of a stage (kTlM rounded up)
constexpr int kTlWBytes = kTlN * 128, kTlTBytes = kTlTokLoads * 64 * 128;
constexpr int kTlSfWaves = 6;                         // five waves' token scales, one place for the others' zeros
constexpr int kTlSfBytes = kTlSfWaves * 1024;         // four K blocks of scales for 64 tokens per wave
constexpr int kTlLds = 2 * (kTlWBytes + kTlTBytes + kTlSfBytes);
constexpr int kTlEpiStride = 64 * 2 + 16;             // LDS bytes per staged token row

// barrier without a fence: every wait it needs is written out
__device__ __forceinline__ void bare_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

struct TlLoads {
  __amdgpu_buffer_rsrc_t ra, rs, rb;
  uint32_t wo[4], to[kTlTokLoads], so;   // byte offsets of this lane's chunks and scales
  uint32_t cut;                   // kNowhere if the lane's chunk lies behind K in the last block
  int KB, wave;
};

// Direct loads of K block b, zeros for a block behind the last: 64 weight
// rows c, 64 token rows c, the token scales of blocks b .. b + 3.  No branch:
// code would move across it and out of the order the stages are written in.
// POL: the weights' cache policy, 2 (non-temporal) where they are read once.
__device__ __forceinline__ uint32_t tl_cut(const TlLoads& L, int b) {
  return b < L.KB - 1 ? 0 : b == L.KB - 1 ? L.cut : kNowhere;
}
template <int POL>
__device__ __forceinline__ void tl_load_w(const TlLoads& L, int b, int c, uint8_t* dst) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(L.rb, lds_addr(dst + (L.wave + 8 * c) * 1024), 16, L.wo[c] | tl_cut(L, b), b < L.KB ? b * 128 : 0, 0, POL);
}
__device__ __forceinline__ void tl_load_t(const TlLoads& L, int b, int c, uint8_t* dst) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(L.ra, lds_addr(dst + (L.wave + 8 * c) * 1024), 16, L.to[c] | tl_cut(L, b), b < L.KB ? b * 128 : 0, 0, 0);
}
__device__ __forceinline__ void tl_load_s(const TlLoads& L, int b, uint8_t* dst) {
  const int w = L.wave < kTlSfWaves ? L.wave : kTlSfWaves - 1;
  __builtin_amdgcn_raw_ptr_buffer_load_lds(L.rs, lds_addr(dst + w * 1024), 16, L.so | (b < L.KB ? 0 : kNowhere), b < L.KB ? b * 4 : 0, 0, 0);
}

template <int JV>
struct TlState {
  // 64-row loads: NT of the tokens, N1 of them in T1; JH = token blocks of T1
  static constexpr int NT = (JV + 1) / 2, N1 = NT > 1 ? NT / 2 : 1, JH = 2 * N1;
  static constexpr int kLoads = 4 + NT;
  float4v acc[4][JV];
  int8v w[4], t;                  // fragments of the next step
  float s;                        // its scale
  float4v dp[4];                  // products of the step before, not yet added
  float sp;
  int tok_at0, tok_at1, w_at0, w_at1, sf_at;   // this lane's LDS offsets
};

__device__ __forceinline__ int8v tl_frag(const uint8_t* base, int at0, int at1, int off) {
  return join(*reinterpret_cast<const int4v*>(base + at0 + off), *reinterpret_cast<const int4v*>(base + at1 + off));
}

#define NVFP4_TL_WAIT(n) asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(n) : "memory")

// The four products of the step's token block, and the scaling of the step
// before, which needs no wait on the matrix unit.  J: its block; after the
// last one's products the next stage's weight fragments are read from wn.
template <int JV, int J>
__device__ __forceinline__ void tl_products(TlState<JV>& st, const int8v& tn, float sn, const uint8_t* wn) {
  constexpr int P = J > 0 ? J - 1 : JV - 1;
  float4v d[4];
#pragma unroll
  for (int f = 0; f < 4; ++f) {
    d[f] = mfma_block(st.w[f], st.t);
    if constexpr (J == JV - 1) st.w[f] = tl_frag(wn, st.w_at0, st.w_at1, f * 2048);
#pragma unroll
    for (int i = 0; i < 4; ++i) st.acc[f][P][i] = fmaf(st.dp[f][i], st.sp, st.acc[f][P][i]);
    asm volatile("" : "+v"(st.acc[f][P]));   // summed here: not sunk to a later block
  }
#pragma unroll
  for (int f = 0; f < 4; ++f) st.dp[f] = d[f];
  st.t = tn;
  st.sp = st.s;
  st.s = sn;
  __builtin_amdgcn_sched_group_barrier(2, 4, 0);
  __builtin_amdgcn_sched_group_barrier(8, 1, 0);
  __builtin_amdgcn_sched_group_barrier(2, 4, 0);
  __builtin_amdgcn_sched_group_barrier(8, 1, 0);
  __builtin_amdgcn_sched_group_barrier(256, 3, 0);
  __builtin_amdgcn_sched_group_barrier(2, 4, 0);
  __builtin_amdgcn_sched_group_barrier(8, 1, 0);
  __builtin_amdgcn_sched_group_barrier(2, 4, 0);
  __builtin_amdgcn_sched_group_barrier(8, 1, 0);
  __builtin_amdgcn_sched_group_barrier(32, 1, 0);
  __builtin_amdgcn_sched_barrier(0);
}

// Steps 0 .. JH-2: fragments from T1 (t1), loads of T2 of block b + 1 into
// nt2 and, every fourth stage, of the next four blocks' scales into ns.  The
// pointers are __restrict__, and apart within one function: a fragment read
// is then known not to alias the loads in flight, and gets no wait on them.
template <int JV, int J>
__device__ __forceinline__ void tl_first(TlState<JV>& st, const TlLoads& L, int b, float sb, bool on,
                                         const uint8_t* __restrict__ t1, const uint8_t* __restrict__ sf,
                                         uint8_t* __restrict__ nt) {
  using S = TlState<JV>;
  if constexpr (J < S::JH - 1) {
    const int8v tn = tl_frag(t1, st.tok_at0, st.tok_at1, (J + 1) * 4096);
    const float v = *reinterpret_cast<const float*>(sf + st.sf_at + (J + 1) * 512) * sb;
    const float sn = on ? v : 0.0f;
    constexpr int steps = S::JH - 1, n2 = S::NT - S::N1;
#pragma unroll
    for (int c = 0; c < n2; ++c)
      if (c * steps / n2 == J) tl_load_t(L, b + 1, S::N1 + c, nt);
    tl_products<JV, J>(st, tn, sn, nullptr);
    tl_first<JV, J + 1>(st, L, b, sb, on, t1, sf, nt);
  }
}

// Steps JH-1 .. JV-2: fragments from T2 (t2), loads of the weights and T1 of
// block b + 2 into this stage's buffers.
template <int JV, int J, int POL>
__device__ __forceinline__ void tl_second(TlState<JV>& st, const TlLoads& L, int b, float sb, bool on,
                                          const uint8_t* __restrict__ t2, const uint8_t* __restrict__ sf,
                                          uint8_t* __restrict__ w, uint8_t* __restrict__ t1) {
  using S = TlState<JV>;
  if constexpr (J < JV - 1) {
    const int8v tn = tl_frag(t2, st.tok_at0, st.tok_at1, (J + 1) * 4096);
    const float v = *reinterpret_cast<const float*>(sf + st.sf_at + (J + 1) * 512) * sb;
    const float sn = on ? v : 0.0f;
    constexpr int steps = JV - S::JH, n = 4 + S::N1, at = J - (S::JH - 1);
#pragma unroll
    for (int c = 0; c < n; ++c)
      if (c * steps / n == at) {
        if (c < 4) tl_load_w<POL>(L, b + 2, c, w);
        else tl_load_t(L, b + 2, c - 4, t1);
      }
    tl_products<JV, J>(st, tn, sn, nullptr);
    tl_second<JV, J + 1, POL>(st, L, b, sb, on, t2, sf, w, t1);
  }
}

// Step JV-1: the next stage's first fragments.
template <int JV>
__device__ __forceinline__ void tl_last(TlState<JV>& st, float sb_next, bool on, const uint8_t* __restrict__ wn,
                                        const uint8_t* __restrict__ t1n, const uint8_t* __restrict__ sfn) {
  const int8v tn = tl_frag(t1n, st.tok_at0, st.tok_at1, 0);
  const float v = *reinterpret_cast<const float*>(sfn + st.sf_at) * sb_next;
  const float sn = on ? v : 0.0f;
  tl_products<JV, JV - 1>(st, tn, sn, wn);
}

template <int JV, int POL>
__device__ __forceinline__ void tl_run(const Fp8Params& p, const RowTile& t, int64_t n0, const TlLoads& L,
                                       int lane, uint8_t* smem) {
  using S = TlState<JV>;
  const int wave = L.wave, KB = L.KB;
  const int r = lane & 15, g = lane >> 4, wn = wave >> 1, wt = wave & 1;
  S st;
#pragma unroll
  for (int f = 0; f < 4; ++f) {
    st.dp[f] = float4v{0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < JV; ++j) st.acc[f][j] = float4v{0, 0, 0, 0};
  }
  st.sp = 0.0f;
  const int at0 = (g ^ ((r >> 1) & 7)) * 16, at1 = ((4 + g) ^ ((r >> 1) & 7)) * 16;
  st.w_at0 = (wn * 64 + r) * 128 + at0;
  st.w_at1 = (wn * 64 + r) * 128 + at1;
  st.tok_at0 = (wt * 16 + r) * 128 + at0;
  st.tok_at1 = (wt * 16 + r) * 128 + at1;
  st.sf_at = (wt * 16 + r) * 16;
  int nb = (int)((n0 + wn * 64) / 128);
  if (nb >= p.NB) nb = p.NB - 1;
  const float* bsf = p.b_sf + ((int64_t)t.e * p.NB + nb) * p.KB;
  uint8_t *w0 = smem, *w1 = smem + kTlWBytes, *t0 = smem + 2 * kTlWBytes, *t1 = t0 + kTlTBytes, *sf = t1 + kTlTBytes;
  auto sf_of = [&](int b) { return sf + ((b >> 2) & 1) * kTlSfBytes + (b & 3) * 4; };
  auto sb_of = [&](int b) { return uniform_load(bsf, b < KB ? b : 0); };

#pragma unroll
  for (int c = 0; c < 4; ++c) tl_load_w<POL>(L, 0, c, w0);
  tl_load_s(L, 0, sf);
#pragma unroll
  for (int c = 0; c < S::N1; ++c) tl_load_t(L, 0, c, t0);
  asm volatile("" ::: "memory");   // these first: the wait below counts the later ones
#pragma unroll
  for (int c = S::N1; c < S::NT; ++c) tl_load_t(L, 0, c, t0);
  asm volatile("" ::: "memory");   // and T2 before the next stage's, as barrier B counts
#pragma unroll
  for (int c = 0; c < 4; ++c) tl_load_w<POL>(L, 1, c, w1);
#pragma unroll
  for (int c = 0; c < S::N1; ++c) tl_load_t(L, 1, c, t1);
  NVFP4_TL_WAIT(S::kLoads);
  bare_barrier();
#pragma unroll
  for (int f = 0; f < 4; ++f) st.w[f] = tl_frag(w0, st.w_at0, st.w_at1, f * 2048);
  st.t = tl_frag(t0, st.tok_at0, st.tok_at1, 0);
  st.s = *reinterpret_cast<const float*>(sf + st.sf_at) * sb_of(0);

  auto stage = [&](int b, uint8_t* wc, uint8_t* tc, uint8_t* wx, uint8_t* tx) {
    // behind an odd number of blocks one of zeros is run: what its scales'
    // place holds (another row's, maybe no number) must not count
    const float sb = sb_of(b), sb_next = sb_of(b + 1);
    const bool on = b < KB, on_next = b + 1 < KB;
    if ((b & 3) == 0) tl_load_s(L, b + 4, sf + (((b >> 2) + 1) & 1) * kTlSfBytes);
    tl_first<JV, 0>(st, L, b, sb, on, tc, sf_of(b), tx);
    NVFP4_TL_WAIT(S::kLoads);
    bare_barrier();
    tl_second<JV, S::JH - 1, POL>(st, L, b, sb, on, tc, sf_of(b), wc, tc);
    NVFP4_TL_WAIT(S::kLoads);
    bare_barrier();
    tl_last<JV>(st, sb_next, on_next, wx, tx, sf_of(b + 1));
  };
  for (int b = 0; b < KB; b += 2) {
    stage(b, w0, t0, w1, t1);
    stage(b + 1, w1, t1, w0, t0);
  }
#pragma unroll
  for (int f = 0; f < 4; ++f)
#pragma unroll
    for (int i = 0; i < 4; ++i) st.acc[f][JV - 1][i] = fmaf(st.dp[f][i], st.sp, st.acc[f][JV - 1][i]);
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
  bare_barrier();
  // BF16 through LDS (a region per wave): a lane holds four consecutive
  // columns of one token, the stores want sixteen bytes of a token's row
  uint8_t* ep = smem + wave * (16 * kTlEpiStride);
  const bool vec = p.N % 8 == 0 && (reinterpret_cast<uintptr_t>(p.c) & 15) == 0;
  const bool even = p.N % 2 == 0 && (reinterpret_cast<uintptr_t>(p.c) & 3) == 0;
  const int64_t nw = n0 + wn * 64;
#pragma unroll
  for (int j = 0; j < JV; ++j) {
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      uint2 o;
      o.x = pack_bf16x2(st.acc[f][j][0], st.acc[f][j][1]);
      o.y = pack_bf16x2(st.acc[f][j][2], st.acc[f][j][3]);
      *reinterpret_cast<uint2*>(ep + r * kTlEpiStride + 2 * (16 * f + 4 * g)) = o;
    }
    if (vec) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int tok = 8 * h + (lane >> 3), ch = lane & 7;
        const uint4 v = *reinterpret_cast<const uint4*>(ep + tok * kTlEpiStride + 16 * ch);
        const int row = (2 * j + wt) * 16 + tok;
        const int64_t n = nw + 8 * ch;
        if (row < t.nrows && n < p.N) *reinterpret_cast<uint4*>(p.c + (t.row0 + row) * p.N + n) = v;
      }
    } else if (even) {
      // rows at multiples of four bytes: two tokens' columns in pairs per store
      // (4096 x 4094 x 256: 17 us, one column per lane 20 us)
      const int left = t.nrows - (2 * j + wt) * 16, n2 = 2 * (lane & 31);
#pragma unroll
      for (int h = 0; h < 8; ++h) {
        const int tok = 2 * h + (lane >> 5);
        if (tok < left && nw + n2 < p.N)
          *reinterpret_cast<uint32_t*>(p.c + (t.row0 + (2 * j + wt) * 16 + tok) * p.N + nw + n2) =
              *reinterpret_cast<const uint32_t*>(ep + tok * kTlEpiStride + 2 * n2);
      }
    } else {
      // rows at odd places: a token's 64 columns per store
      const int left = t.nrows - (2 * j + wt) * 16;
#pragma unroll 4
      for (int tok = 0; tok < 16; ++tok)
        if (tok < left && nw + lane < p.N)
          p.c[(t.row0 + (2 * j + wt) * 16 + tok) * p.N + nw + lane] =
              *reinterpret_cast<const uint16_t*>(ep + tok * kTlEpiStride + 2 * lane);
    }
  }
}

template <int POL>
__global__ __launch_bounds__(kTlWaves * 64, 2) void fp8_tile_kernel(Fp8Params p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  // Blocks go round the eight XCDs; each XCD takes a contiguous eighth of the
  // tiles in m tile order, so that the n tiles of an m tile share its tokens,
  // and an expert's m tiles its weights, in one L2.
  TileList list;
  const int64_t all = (int64_t)list.count(p, p.bm) * p.n_groups, chunk = (all + 7) >> 3;
  const uint32_t wg = row_workgroup();             // rows of workgroups are whole rounds of the XCDs
  const int64_t at = (int64_t)(wg & 7) * chunk + (wg >> 3);
  if ((wg >> 3) >= chunk || at >= all) return;
  const int mt = (int)(at / p.n_groups), ng = (int)(at - (int64_t)mt * p.n_groups);
  RowTile t;
  if (!list.find(p, p.bm, mt, t)) return;
  t.e = __builtin_amdgcn_readfirstlane(t.e);
  t.nrows = __builtin_amdgcn_readfirstlane(t.nrows);
  t.row0 = __builtin_amdgcn_readfirstlane((int)t.row0);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t n0 = (int64_t)ng * kTlN, K = p.K;
  const int64_t a_base = p.a_row_src ? 0 : t.row0;
  const int64_t a_rows = p.a_row_src ? p.rows_a : t.nrows;
  TlLoads L;
  L.KB = p.KB;
  L.wave = wave;
  L.ra = rsrc_of(p.a_q + a_base * K, a_rows * K);
  L.rs = rsrc_of(p.a_sf + a_base * p.KB, a_rows * p.KB * 4);
  L.rb = rsrc_of(p.b_q + (int64_t)t.e * p.N * K, p.N * K);
  const int q = (lane & 7) ^ ((4 * wave + (lane >> 4)) & 7);
  const int tail = p.K - (p.KB - 1) * 128;
  L.cut = 16 * q < tail ? 0 : kNowhere;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const int64_t n = n0 + (wave + 8 * c) * 8 + (lane >> 3);
    L.wo[c] = n < p.N ? (uint32_t)(n * K) + 16 * q : kNowhere;
  }
#pragma unroll
  for (int c = 0; c < kTlTokLoads; ++c) {
    const int64_t ar = a_row(p, t, (wave + 8 * c) * 8 + (lane >> 3));
    L.to[c] = ar >= 0 ? (uint32_t)((ar - a_base) * K) + 16 * q : kNowhere;
  }
  {
    const int64_t ar = wave < kTlTokLoads ? a_row(p, t, wave * 64 + lane) : -1;
    L.so = ar >= 0 ? (uint32_t)((ar - a_base) * p.KB * 4) : kNowhere;
  }
  switch ((t.nrows + 31) / 32) {
    case 1:
    case 2:
    case 3: tl_run<3, POL>(p, t, n0, L, lane, smem); break;
    case 4: tl_run<4, POL>(p, t, n0, L, lane, smem); break;
    case 5: tl_run<5, POL>(p, t, n0, L, lane, smem); break;
    case 6: tl_run<6, POL>(p, t, n0, L, lane, smem); break;
    case 7: tl_run<7, POL>(p, t, n0, L, lane, smem); break;
    case 8: tl_run<8, POL>(p, t, n0, L, lane, smem); break;
    default: tl_run<9, POL>(p, t, n0, L, lane, smem); break;
  }
}

// m tiles of at most bm rows that E experts with M rows in all can need
int64_t tile_bound(const Fp8GemmArgs& a, int bm) {
  if (!a.offsets) return (a.M + bm - 1) / bm;
  const int64_t b = (a.M + (int64_t)a.E * (bm - 1)) / bm;
  return b < a.M ? b : a.M;
}

template <int POL>
hipError_t launch_stream(const Fp8GemmArgs& a, Fp8Params p, hipStream_t stream) {
  p.n_groups = (int)((a.N + kStN - 1) / kStN);
  const int64_t grid = tile_bound(a, 16) * p.n_groups;
  if (grid >= (int64_t(1) << 31)) return hipErrorInvalidConfiguration;
  fp8_stream_kernel<POL><<<grid_rows(grid), kStWaves * 64, 0, stream>>>(p);
  return hipGetLastError();
}

template <int RF, int JT, int D>
hipError_t launch_skinny(const Fp8GemmArgs& a, Fp8Params p, hipStream_t stream) {
  p.n_groups = (int)((a.N + 16 * RF - 1) / (16 * RF));
  const int64_t grid = tile_bound(a, 16 * JT) * p.n_groups;
  if (grid >= (int64_t(1) << 31)) return hipErrorInvalidConfiguration;
  fp8_skinny_kernel<RF, JT, D><<<grid_rows(grid), kSkWaves * 64, 0, stream>>>(p);
  return hipGetLastError();
}

constexpr int kMaxDevices = 64;

template <int POL>
hipError_t launch_tile(const Fp8GemmArgs& a, Fp8Params p, hipStream_t stream) {
  p.n_groups = (int)((a.N + kTlN - 1) / kTlN);
  const int64_t grid = (tile_bound(a, p.bm) * p.n_groups + 7) / 8 * 8;
  if (grid >= (int64_t(1) << 31)) return hipErrorInvalidConfiguration;
  int dev = 0;
  hipError_t err = hipGetDevice(&dev);
  if (err != hipSuccess) return err;
  if (dev < 0 || dev >= kMaxDevices) return hipErrorInvalidDevice;
  static std::atomic<bool> attr_set[kMaxDevices];
  if (!attr_set[dev].load(std::memory_order_relaxed)) {
    err = hipFuncSetAttribute(reinterpret_cast<const void*>(fp8_tile_kernel<POL>),
                              hipFuncAttributeMaxDynamicSharedMemorySize, kTlLds);
    if (err != hipSuccess) return err;
    attr_set[dev].store(true, std::memory_order_relaxed);
  }
  fp8_tile_kernel<POL><<<grid_rows(grid), kTlWaves * 64, kTlLds, stream>>>(p);
  return hipGetLastError();
}

// Which kernel, and how it is cut.  The row counts of the experts are on the
// device, so the choice goes by the average over the experts that can have
// rows.  The cost of each kernel in units of 0.67 ns times K, as measured on 256
// CUs at K = 7168 (a unit is 4.8 us there):
//   few rows   (RF + JT) a round of workgroups, one per CU (N 2048: 1 row 7.3 us
//              with 16 x 16, 21 us with 64 x 64; 256 rows 25 us with 64 x 32,
//              38 us with 64 x 16)
//   tiles      (6 + JV) a round (N 2048: 2048 rows 50 us with 96-row tiles in one
//              round, 74 us with 288; 4096 rows 92 us with 96-row tiles in
//              two rounds, 65 us with 128), and 12 at least where the weights
//              are one tile's alone and each stage waits for HBM (8 experts of
//              14 rows, N 4096: 63 us, streaming 42 us)
//   streaming  3.2 + B/60 for B workgroups (1 row, N 32768: 36 us; the others
//              43 us and more), 1.3 of that for experts of several tiles
//              (2 experts of 33 rows, N 3473, K 3328: 21 us, 64 x 32 14 us)
// and none is faster than its experts' weights come from HBM: N * live / 4100
// units (256 experts, N 4096, 8 rows each: streaming 1.11 ms, tiles 1.15 ms; 16
// rows each: 1.27 ms, 1.20 ms).  Over 122 shapes the choice takes 1.04 times as
// long as the best of all kernels and cuts (geometric mean; worst 1.38).
struct Fp8Plan {
  int kind;    // 0 stream, 1 few rows, 2 tiles
  int rf, jt, bm;
};

Fp8Plan plan_of(const Fp8GemmArgs& a, int cus) {
  const int64_t live = a.E < a.M ? a.E : a.M;
  const double avg = (double)a.M / live;
  auto up = [](int64_t x, int64_t y) { return (x + y - 1) / y; };
  // m tiles of bm rows: an expert's last one is half full on average; rows that
  // spread by the root of their average and still fit one tile are one (25
  // experts of about 53 rows, N 529, K 5984: 64 x 64 a workgroup 35 us, tiles 58 us)
  auto m_tiles = [&](int bm) {
    if (!a.offsets) return (double)up(a.M, bm);
    return live * (avg + std::sqrt(avg) <= bm ? 1.0 : std::fmax(avg / bm + 0.5, 1.0));
  };
  auto rounds = [&](double tiles, int64_t n_tiles) { return (double)(int64_t)((tiles * n_tiles + cus - 1) / cus); };
  const double hbm = (double)live * a.N / 4100.0 * (256.0 / cus);
  auto over_hbm = [&](double c) { return std::fmax(c, hbm * 1.02 + 0.01 * c); };
  const double blocks = m_tiles(16) * up(a.N, kStN) * (256.0 / cus);
  const double first = 3.2 + blocks / 60, flow = m_tiles(16) * a.N / 4400.0 * (256.0 / cus);
  double cost = (first > flow ? first : flow) * (avg > 16 ? 1.3 : 1.0);
  Fp8Plan best{0, 0, 1, 0};
  for (int bm = kTlMin; bm <= kTlM; bm += 32) {
    const double tiles = m_tiles(bm), wgs = tiles * up(a.N, kTlN), r = rounds(tiles, up(a.N, kTlN));
    const double jv = (double)up((int64_t)(a.M / tiles + 0.999), 32);
    const double stages = std::fmax(6.0 + std::fmax(jv, 3.0), tiles < 2 * live ? 12.0 : 0.0);
    // Experts above the average: in a round that is nearly full their further
    // tiles start another one, so high tiles (16 experts of about 116 rows, N 4096,
    // K 2048: 31 us with 288, 48 us with 128); else they fill idle CUs, so low ones.
    const bool full = a.offsets && wgs > (r - 0.25) * cus;
    const double c = over_hbm(r * stages * (full && r < 4 ? 1.1 : 1.0)) + (full ? kTlM - bm : bm) * 1e-5;
    if (c < cost) { cost = c; best = Fp8Plan{2, 0, 0, bm}; }
  }
  static const int kShape[6][2] = {{1, 1}, {2, 1}, {4, 1}, {2, 2}, {4, 2}, {4, 4}};
  for (const auto& s : kShape) {
    const double c = over_hbm(rounds(m_tiles(16 * s[1]), up(a.N, 16 * s[0])) * (s[0] + s[1]));
    if (c < cost) { cost = c; best = Fp8Plan{1, s[0], s[1], 0}; }
  }
  return best;
}

}  // namespace

// The device's cut of expert rows [lo, hi), on the host for the tests: the
// number of tiles of at most bm rows, and tile i (0 rows if there is none).
extern "C" int nvfp4_internal_fp8_cut(int64_t M, int lo, int hi, int bm, int i, int64_t* row0, int* nrows) {
  Fp8Params p{};
  p.M = M;
  RowTile t{};
  *nrows = cut_tile(p, bm, lo, hi - lo, i, t) ? t.nrows : 0;
  *row0 = t.row0;
  return TileList::tiles(lo, hi, bm);
}

// The choice of kernel on `cus` CUs, for the tests that each kernel is run by
// sizes meant for it: plan = {kind, RF, JT, tile height}.
extern "C" void nvfp4_internal_fp8_plan(int E, int grouped, int64_t M, int64_t N, int64_t K, int cus, int* plan) {
  static const int32_t some = 0;
  Fp8GemmArgs a{};
  a.offsets = grouped ? &some : nullptr;
  a.E = E; a.M = M; a.N = N; a.K = K;
  const Fp8Plan p = plan_of(a, cus);
  plan[0] = p.kind; plan[1] = p.rf; plan[2] = p.jt; plan[3] = p.bm;
}

hipError_t launch_fp8_gemm(const Fp8GemmArgs& a, hipStream_t stream) {
  Fp8Params p;
  p.a_q = a.a_q; p.a_sf = a.a_sf; p.rows_a = a.rows_a; p.a_row_src = a.a_row_src;
  p.a_row_div = a.a_row_div; p.offsets = a.offsets; p.E = a.E; p.M = a.M; p.N = a.N;
  p.K = (int)a.K; p.KB = (int)((a.K + 127) / 128); p.NB = (int)((a.N + 127) / 128);
  p.b_q = a.b_q; p.b_sf = a.b_sf; p.c = static_cast<uint16_t*>(a.c);
  p.n_groups = 0;
  int cus = 0;
  const hipError_t err = device_cus(cus);
  if (err != hipSuccess) return err;
  const Fp8Plan plan = plan_of(a, cus);
  p.bm = plan.bm;
  // Weights read once go past the caches, unless rows are no multiple of 128
  // bytes: two K blocks then share a line, which would be fetched twice (40
  // experts of 115 rows, N 1001, K 1040: 23 us, 32 us past the caches).
  const bool aligned = a.K % 128 == 0;
  if (plan.kind == 0) return aligned ? launch_stream<2>(a, p, stream) : launch_stream<0>(a, p, stream);
  if (plan.kind == 2)   // once: where an expert is one tile on average
    return aligned && a.M <= plan.bm * (int64_t)a.E ? launch_tile<2>(a, p, stream) : launch_tile<0>(a, p, stream);
  switch (plan.rf * 8 + plan.jt) {
    case 9: return launch_skinny<1, 1, 3>(a, p, stream);
    case 17: return launch_skinny<2, 1, 3>(a, p, stream);
    case 33: return launch_skinny<4, 1, 2>(a, p, stream);
    case 18: return launch_skinny<2, 2, 2>(a, p, stream);
    case 34: return launch_skinny<4, 2, 2>(a, p, stream);
    default: return launch_skinny<4, 4, 1>(a, p, stream);
  }
}

}  // namespace nvfp4
