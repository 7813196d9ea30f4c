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
  return launch_skinny<4>(a, p, stream);
}

}  // namespace nvfp4
