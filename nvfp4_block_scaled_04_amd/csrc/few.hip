// The expert layer for a few tokens in two kernels (gfx950).
//
//   up:    a = W1[e] x_t,  h = c_te * silu(gate) * up   for every expert e with a
//          token and its tokens t;  c_te = sum of w[t][j] over ids[t][j] == e
//   down:  out[t][n] = bf16( sum over experts e of W2[e][n] . h_te )
// Weights FP8 (one scale per 128 x 128) or packed NVFP4 (E4M3 per 16, a global
// scale an expert).  Activations are not quantised: the bytes of each live
// expert's weights are the bound.  They are read once for every four of its
// tokens, or every eight (launch_few): once in all where routing is even.
//
// FP8 weights enter the matrix unit as BF16 (exact), with x as it is and h as two
// BF16, its rounding and what that leaves (16 bits in all).  A block's scale
// multiplies the sums of 64 codes (448 at most) times these, which are finite where
// they are below 2^112.  NVFP4 weights enter as FP16, in which a scale is one packed product for two weights (exact; in BF16
// it would be three times the instructions, and decoding them bounds the kernels):
// x with its exponents moved so that a token's largest just fits (exact down to
// 2^-29 of that, below off by 2^-30 of it), h rounded to FP16 (11 bits, an eighth
// of what the rounding of out to BF16 takes) with a power of two for each 16
// columns.  Sums in fp32.
//
// An expert has few tokens, so the matrix unit's 16 rows are 4 weight rows x 4
// quarters of a K step, and its 16 columns 4 tokens x the same quarters: of the
// 16 x 16 results those of equal quarters count (64 of 256; the unit has the
// room).  Weights so come in runs of 256 bytes a row, and a step's tokens are
// loaded in the unit's own layout with no lane to spare.  A K step is 256 columns
// (FP8) or 512 (NVFP4: four stages of the packed layout), 16 bytes of weights a
// lane and row group.
//
// Equal inputs give equal bits: waves and quarters are joined in a fixed order.
#include <climits>
#include <cstddef>
#include <type_traits>

#include "internal.hpp"
#include "device.hpp"

namespace nvfp4 {

namespace {

typedef int int4v __attribute__((ext_vector_type(4)));
typedef float float4v __attribute__((ext_vector_type(4)));
typedef uint32_t uint4v __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef _Float16 half8v __attribute__((ext_vector_type(8)));

constexpr int kWaves = 8, kThreads = kWaves * 64;
constexpr int kPairs = kFewTokens * 64;               // (token, slot) pairs at most
constexpr int kMaxExperts = 4096;

// A byte offset with this bit set lies behind every resource below (they all
// hold less than 2^31 bytes): the load returns zeros and touches no memory, if its
// scalar offset lies inside the resource.
constexpr uint32_t kNowhere = 0x80000000u;

__device__ const float kNoScale = 0.0f;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc_of(const void* base, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, 0x00020000);
}

__device__ __forceinline__ float uniform_load(const float* p) {
  return *(const __attribute__((address_space(4))) float*)p;
}

// Between LDS writes of the wave's lanes and reads of theirs by others, or the
// other way round.  The hardware keeps a wave's LDS accesses in order; this keeps the
// compiler from moving them past each other, and costs no instruction.
__device__ __forceinline__ void wave_order() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// ------------------------------------------------------------ the work
//
// The live experts in order of their first pair, each cut into entries of at
// most `cap` tokens.  A row of h is one (expert, token); rows follow the entries.
struct alignas(16) Entry {      // the second product reads one as a uint4
  uint16_t e, row;              // expert, first row
  uint32_t count;               // rows
  uint8_t tok[8];               // their tokens
};

struct Live {
  Entry entry[kPairs];
  float coef[kPairs];           // a row's weight
  int n;                        // entries
};
static_assert(sizeof(Entry) == 16 && alignof(Entry) >= alignof(uint4) && offsetof(Live, entry) % 16 == 0,
              "an entry is read as a uint4");

struct LiveScratch {
  int first[kMaxExperts];       // first pair of an expert, then its place among the experts
  int count[kPairs / 64];
  int id[kPairs];               // the pairs' experts, -1 for those without one
  float w[kPairs];              // and weights
  int mask[kPairs], row[kPairs];   // an expert's tokens and first row
};

// inclusive sum over the wave's lanes
__device__ __forceinline__ int scan64(int v) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int u = __shfl_up(v, o);
    v += lane >= o ? u : 0;
  }
  return v;
}

// An expert's entries: `rows` rows from `row` on, first entry `at`; their tokens
// and weights come from the pairs.
__device__ __forceinline__ void put_entries(Live& L, int e, int rows, int row, int at, int cap) {
  for (; rows > 0; rows -= cap, row += cap, ++at) {
    L.entry[at].e = (uint16_t)e;
    L.entry[at].row = (uint16_t)row;
    L.entry[at].count = (uint32_t)(rows < cap ? rows : cap);
  }
}

// At most 64 pairs: one wave, a lane a pair, the last wave, which has no token's
// largest to find where there are fewer than eight (NVFP4, one token: the first
// product 29.6 -> 28.7 us, of the small layer 9.8 -> 9.1).  Pairs of one expert find each other
// by writing their lane to the expert's place: whichever stays there collects for
// all of them.
__device__ __forceinline__ void build_small(const FewArgs& p, int cap, Live& L, LiveScratch& S) {
  if (threadIdx.x >= kThreads - 64) {
    const int pairs = p.T * p.k, lane = threadIdx.x & 63;
    const int e = lane < pairs ? p.ids[lane] : -1;
    const float w = lane < pairs ? p.topk_w[lane] : 0.0f;
    const int t = (int)(((float)lane + 0.5f) * __builtin_amdgcn_rcpf((float)p.k));   // lane / k: never within 2^-7 of a whole number
    const bool on = e >= 0 && e < p.E;
    int *mask_of = S.mask, *first_of = S.row, *count_of = S.id;
    mask_of[lane] = 0;
    first_of[lane] = 64;
    count_of[lane] = 0;
    if (on) S.first[e] = lane;
    wave_order();
    int mask = 0, first = 64, count = 0, by = 0;
    if (on) {
      by = S.first[e];
      atomicOr(&mask_of[by], 1 << t);
      atomicMin(&first_of[by], lane);
      atomicAdd(&count_of[by], 1);
      wave_order();
      mask = mask_of[by];
      first = first_of[by];
      count = count_of[by];
    }
    const int tokens = __popc(mask), rows = first == lane ? tokens : 0, entries = (rows + cap - 1) / cap;
    const int row_end = scan64(rows), entry_end = scan64(entries);
    const int row = __shfl(row_end - rows, first & 63), entry = __shfl(entry_end - entries, first & 63);
    bool head = on;                                      // the token's first pair with the expert
    float coef = w;                                      // and all its pairs' weights
    if (__ballot(count != tokens) != 0) {                // an expert twice in a token's row
      coef = 0.0f;
      for (int j = 0; j < p.k; ++j) {
        const int f = t * p.k + j;
        const bool hit = __shfl(e, f & 63) == e && f < pairs;
        const float wj = __shfl(w, f & 63);
        coef += hit ? wj : 0.0f;
        head = head && !(hit && f < lane);
      }
    }
    put_entries(L, e, rows, row, entry, cap);
    if (head) {
      const int at = __popc(mask & ((1 << t) - 1));
      L.entry[entry + at / cap].tok[at % cap] = (uint8_t)t;
      L.coef[row + at] = coef;
    }
    if (lane == 63) L.n = entry_end;
  }
  __syncthreads();
}

__device__ void build_large(const FewArgs& p, int cap, Live& L, LiveScratch& S) {
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
    S.id[f] = e[i];
    S.w[f] = f < pairs ? p.topk_w[f] : 0.0f;
  }
  __syncthreads();
  uint64_t firsts[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    firsts[i] = __ballot(e[i] >= 0 && S.first[e[i] < 0 ? 0 : e[i]] == i * kThreads + (int)threadIdx.x);
    if (lane == 0) S.count[i * kWaves + wave] = __popcll(firsts[i]);
  }
  __syncthreads();
  int n = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    int at = 0;
    for (int c = 0; c < i * kWaves + wave; ++c) at += S.count[c];
    if (firsts[i] >> lane & 1) {
      at += __popcll(firsts[i] & ((uint64_t(1) << lane) - 1));
      S.mask[at] = 0;
      S.first[e[i]] = at;
    }
  }
  for (int c = 0; c < kPer * kWaves; ++c) n += S.count[c];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (e[i] >= 0) atomicOr(&S.mask[S.first[e[i]]], 1 << ((i * kThreads + (int)threadIdx.x) / p.k));
  __syncthreads();
  if (wave == 0) {
    int row = 0, entry = 0;
    for (int u0 = 0; u0 < n; u0 += 64) {
      const int u = u0 + lane, rows = u < n ? __popc(S.mask[u]) : 0, entries = (rows + cap - 1) / cap;
      const int row_end = scan64(rows), entry_end = scan64(entries);
      if (u < n) {
        const int first_row = row + row_end - rows, first_entry = entry + entry_end - entries;
        put_entries(L, 0, rows, first_row, first_entry, cap);   // the expert is put in below
        S.row[u] = first_row;
        S.mask[u] |= first_entry << 16;
      }
      row += __shfl(row_end, 63);
      entry += __shfl(entry_end, 63);
    }
    if (lane == 0) L.n = entry;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (e[i] < 0) continue;
    const int f = i * kThreads + threadIdx.x, t = f / p.k, u = S.first[e[i]];
    const int mask = S.mask[u] & 0xFFFF, entry = S.mask[u] >> 16;
    bool head = true;
    float sum = 0.0f;
    for (int j = t * p.k; j < (t + 1) * p.k; ++j) {
      if (S.id[j] != e[i]) continue;
      head = head && j >= f;
      sum += S.w[j];
    }
    if (head) {
      const int at = __popc(mask & ((1 << t) - 1));
      L.entry[entry + at / cap].tok[at % cap] = (uint8_t)t;
      L.coef[S.row[u] + at] = sum;
      if (at % cap == 0) L.entry[entry + at / cap].e = (uint16_t)e[i];
    }
  }
  __syncthreads();
}

// One operand of a product: the weights of all experts, N rows of K.  Sizes and
// counts come from the host: a kernel that runs for some microseconds has no time
// for divisions.
struct Weights {
  const uint8_t* q;
  const uint8_t* sf;            // FP8: float scales
  int N, K, KB, KS;             // KB: scale blocks or stages of 128; KS: K steps
  int64_t q_bytes, sf_bytes;    // of one expert
};

template <bool FP8>
struct Format {
  static constexpr int kCols = FP8 ? 256 : 512;          // a K step
  static constexpr int kM = FP8 ? 2 : 4;                 // its matrix instructions a row group
};

struct FewParams {
  FewArgs a;
  Weights w;                    // w1 (up) or w2 (down)
  int tiles;                    // up: of one entry; down: all
  float inv_tiles, inv_grid;    // up: 1 / tiles, 1 / workgroups
  int64_t t_bytes;              // of x or of one plane of h
};

// A lane holds, of weight row group f (4 rows), row r & 3 and of quarter r >> 2
// the 16 bytes g (r = lane & 15, g = lane >> 4); of token group j, token r & 3 and
// the same columns.
template <bool FP8, int RF>
struct StepW {
  int4v w[RF];
  int4v s;                      // NVFP4: the scales of two rows of stage q (16 bytes)
  float sc[2][2];               // FP8, uniform: scales of two row blocks, two K blocks
};

// Where row group f of a tile begins in one expert's weights, in bytes, K step 0.
template <bool FP8>
__device__ __forceinline__ int group_at(const Weights& W, int row) {
  return FP8 ? row * W.K : ((row / NVFP4_PACK_ROWS) * W.KB * NVFP4_PACK_ROWS + row % NVFP4_PACK_ROWS) * 64;
}

// Loads of K step b of the row groups at `at` of expert e; none if !on.  Past the
// caches: each is read once an entry.  block (FP8): the two 128-row blocks that the groups
// lie in; scale_at (NVFP4): this lane's place in the scales of step 0.  TURN: the
// groups are eight in a row, 256 bytes each, and load f takes group f ^ q of
// quarter q: stages are 32 KiB apart, so one group's quarters would all come from
// one memory channel (sixteen tokens, first product: 327 us, turned 308).
template <bool FP8, int RF, bool TURN>
__device__ __forceinline__ void load_weights(const Weights& W, int e, const int (&at)[RF], const int (&block)[2],
                                             uint32_t scale_at, int b, bool on, int lane, StepW<FP8, RF>& x) {
  const int r = lane & 15, g = lane >> 4, q = r >> 2;
  const auto rq = rsrc_of(W.q + e * W.q_bytes, W.q_bytes);
  const int step = on ? b : 0;
  uint32_t to;
  if constexpr (FP8) {
    const int col = 64 * q + 16 * g;
    to = ((uint32_t)(r & 3) * (uint32_t)W.K + col) | (on && col < W.K - b * 256 ? 0 : kNowhere);
    const float* s = reinterpret_cast<const float*>(W.sf + e * W.sf_bytes) + 2 * b;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float* si = s + block[i] * W.KB;
      x.sc[i][0] = uniform_load(on ? si : &kNoScale);
      x.sc[i][1] = uniform_load(on && 2 * b + 1 < W.KB ? si + 1 : &kNoScale);
    }
  } else {
    const auto rs = rsrc_of(W.sf + e * W.sf_bytes, W.sf_bytes);
    x.s = __builtin_amdgcn_raw_buffer_load_b128(rs, scale_at | (on && 4 * b + g < W.KB ? 0 : kNowhere), step * (4 * NVFP4_PACK_ROWS * 8), 2);
    to = (uint32_t)((q * NVFP4_PACK_ROWS + (r & 3)) * 64 + 16 * g) | (on && 4 * b + q < W.KB ? 0 : kNowhere);
  }
#pragma unroll
  for (int f = 0; f < RF; ++f) {
    const int so = at[TURN ? 0 : f] + step * (FP8 ? 256 : 4 * NVFP4_PACK_ROWS * 64);
    x.w[f] = __builtin_amdgcn_raw_buffer_load_b128(rq, TURN ? to + 256 * (f ^ q) : to, so, 2);
  }
}

// The lane's place of load_weights' scales: rows row0 + 2r and the next of the
// groups' 4 * RF rows, stage g.
template <int RF>
__device__ __forceinline__ uint32_t scale_place(int row0, int end, int KB, int lane) {
  const int r = lane & 15, g = lane >> 4, row = row0 + 2 * r;
  return r < 2 * RF && row < end ? (uint32_t)(((row / NVFP4_PACK_ROWS) * KB + g) * NVFP4_PACK_ROWS + row % NVFP4_PACK_ROWS) * 8 : kNowhere;
}

// NVFP4 scales of a step on their way through the wave's LDS, from the lanes that
// loaded them to those that hold the weights.
struct Scales {
  uint16_t v[4][32][4];         // stage, row, two scales each
};

// Eight weights of the lane's 16 (FP8: as BF16) or 32 (NVFP4: as FP16): number m.
template <bool FP8>
__device__ __forceinline__ int4v decode8(const int4v& w, half2v s, int m) {
  int4v o;
  if constexpr (FP8) {
    const int lo = w[2 * m], hi = w[2 * m + 1];
    o[0] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false));
    o[1] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true));
    o[2] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false));
    o[3] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true));
  } else {
    const half2v t = m < 2 ? half2v{s.x, s.x} : half2v{s.y, s.y};
    const uint32_t c = w[m];
    o[0] = __builtin_bit_cast(int, (half2v)__builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, 1.0f, 0) * t);
    o[1] = __builtin_bit_cast(int, (half2v)__builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, 1.0f, 1) * t);
    o[2] = __builtin_bit_cast(int, (half2v)__builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, 1.0f, 2) * t);
    o[3] = __builtin_bit_cast(int, (half2v)__builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, 1.0f, 3) * t);
  }
  return o;
}

template <bool FP8>
__device__ __forceinline__ float4v mfma(const int4v& w, const int4v& t, const float4v& c) {
  if constexpr (FP8) return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w), __builtin_bit_cast(bf16x8, t), c, 0, 0, 0);
  else return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8v, w), __builtin_bit_cast(half8v, t), c, 0, 0, 0);
}

// largest over the 16 lanes of a row of them
__device__ __forceinline__ float max16(float m) {
  m = fmaxf(m, __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(m), 0x128, 0xF, 0xF, true)));
  m = fmaxf(m, __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(m), 0x124, 0xF, 0xF, true)));
  m = fmaxf(m, __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(m), 0x122, 0xF, 0xF, true)));
  return fmaxf(m, __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(m), 0x121, 0xF, 0xF, true)));
}

// Two BF16 -> two FP16 with `less` (both halves) taken off their exponents; what
// falls below FP16's smallest exponent is as good as zero.
__device__ __forceinline__ uint32_t move_exponents(uint32_t v, uint32_t less) {
  typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
  const u16x2 mag = __builtin_elementwise_sub_sat(__builtin_bit_cast(u16x2, v & 0x7FFF7FFFu), __builtin_bit_cast(u16x2, less));
  return (v & 0x80008000u) | (__builtin_bit_cast(uint32_t, mag) << 3);
}

// ------------------------------------------------------------ up
//
// A tile is 16 columns of h of one entry: their 16 gate and 16 up rows.  `split`
// waves of a workgroup take its K steps in turn and join through LDS; the
// workgroup works on 8 / split tiles at a time, and a wave's loads run on across
// tile ends: a step's go out before the one in front of it is added, so that two are
// in flight.  Alone with its tile a wave needs no barrier.
//
// Measured, one MI355X, H 7168, I 2048, 8 of 256 experts a token: one token FP8 38
// to 40 us (235 MB), NVFP4 28 to 30 us (132 MB), of which 2.6 us are an empty
// launch, 1 the list, 3 the way to the first weights and 2 the end; sixteen tokens
// (102 experts) FP8 442 to 464 us (6.5 to 6.8 TB/s), NVFP4 305 us (5.5).
// Bound by HBM, for small layers (H 2048, I 768: 10 us a token) by the ends.  Three
// steps in flight: 1 to 2 us slower for one token, no faster for sixteen.  Every copy
// of a step's code comes cold at each launch: with two steps' loads in front of the
// loop in place of one the small layer's kernels took 1 us more each (FP8, 4 tokens:
// 24.8 and 15.8 us, now 23.8 and 14.4).

template <bool FP8, int NG>
__global__ __launch_bounds__(kThreads, 2) void few_up_kernel(FewParams P) {
  constexpr int RF = 8, kCols = Format<FP8>::kCols, kM = Format<FP8>::kM, kTok = 4 * NG;
  const FewArgs& p = P.a;
  const Weights& W = P.w;
  __shared__ Live L;
  __shared__ union {
    LiveScratch build;
    float sums[kWaves][4][kTok][4 * RF + 4];
  } S;
  __shared__ Scales scales[FP8 ? 1 : kWaves];
  __shared__ uint32_t largest[kFewTokens];               // NVFP4: of a token's |x|, BF16 bits
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  if constexpr (!FP8) {
    for (int t = wave; t < p.T; t += kWaves) {
      const uint4* x = reinterpret_cast<const uint4*>(p.x + (int64_t)t * p.H);
      uint32_t m = 0;
      for (int i = lane; i < p.H / 8; i += 64) {
        const uint4 v = x[i];
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) m = max(m, max(w[j] & 0x7FFFu, w[j] >> 16 & 0x7FFFu));
      }
#pragma unroll
      for (int o = 32; o >= 1; o >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, o));
      if (lane == 0) largest[t] = m;
    }
  }
  if (p.T * p.k <= 64) build_small(p, kTok, L, S.build);
  else build_large(p, kTok, L, S.build);

  const int I = W.N / 2, per = P.tiles, tiles = __builtin_amdgcn_readfirstlane(L.n) * per;
  // Waves a tile (their log2, sp): the fewest rounds of K steps, where the join of
  // several costs two fifths of a step a round.  1, 2, 4, 8 waves, us: FP8 one token
  // 57, 38, 38, 41, small layer of four tokens 24, 25, 22, 25; NVFP4 small 13, 11, 8,
  // 8, its four tokens 16, 18, 18, 26, sixteen tokens 323, 303, 310, 314.
  int sp = 0, best = INT_MAX;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = ((tiles << i) + kWaves - 1) / kWaves;
    const int rounds = __builtin_amdgcn_readfirstlane((int)((float)(n - 1) * P.inv_grid)) + 1;
    const int cost = rounds * (5 * ((W.KS + (1 << i) - 1) >> i) + (i > 0 ? 2 : 0));
    if (cost < best) {
      best = cost;
      sp = i;
    }
  }
  const int split = 1 << sp, subs = kWaves >> sp, sub = wave >> sp, part = wave & (split - 1);
  const int units = (tiles + subs - 1) >> (3 - sp), stride = gridDim.x, steps = (W.KS + split - 1) >> sp;
  if ((int)blockIdx.x >= units) return;
  const auto rx = rsrc_of(p.x, P.t_bytes);
  const int lane_col = kCols / 4 * (r >> 2) + kCols / 16 * g;   // of this lane's tokens in a K step
  // the entry of a tile: its quotient by `per` to one, then put right
  auto entry_of = [&](int tile) {
    int u = __builtin_amdgcn_readfirstlane((int)((float)tile * P.inv_tiles));
    const int left = tile - u * per;
    return u + (left >= per ? 1 : 0) - (left < 0 ? 1 : 0);
  };

  struct Step {
    StepW<FP8, RF> w;
    int4v t[NG][kM];
  };
  struct {
    int i, s, b, e;
    int w[RF], block[2];        // the row groups' bytes, and (FP8) their 128-row blocks
    bool on;
    uint32_t t[NG], sc;         // this lane's tokens' bytes, and place in the scales
  } at;
  auto set_tile = [&]() {
    // behind the last tile the first one's places: a load's range is checked with
    // its scalar offset taken off the resource's size, so that stays inside it always
    const int next = at.i * subs + sub, tile = next < tiles ? next : 0, u = entry_of(tile);
    at.on = next < tiles;
    at.s = 0;
    at.b = part;
    const int c0 = 16 * (tile - u * per);
    const Entry& y = L.entry[u];
    at.e = __builtin_amdgcn_readfirstlane(y.e);
    at.sc = scale_place<RF>(2 * c0, 2 * I, W.KB, lane);
    // FP8: four groups of gate rows, then of up rows; NVFP4: 32 rows, eight of each in turn
#pragma unroll
    for (int f = 0; f < RF; ++f) at.w[f] = group_at<FP8>(W, FP8 ? c0 + 4 * (f & 3) + (f < 4 ? 0 : I) : 2 * c0 + 4 * f);
    at.block[0] = c0 / 128;
    at.block[1] = (I + c0) / 128;
#pragma unroll
    for (int j = 0; j < NG; ++j) {
      const int c = 4 * j + (r & 3);
      at.t[j] = c < (int)y.count ? (uint32_t)y.tok[c] * (uint32_t)W.K * 2 + 2 * lane_col : kNowhere;
    }
  };
  auto issue = [&](Step& x) {
    const bool on = at.on && at.b < W.KS;
    const uint32_t off = on && lane_col < W.K - at.b * kCols ? 0 : kNowhere;
    const int so = on ? at.b * kCols * 2 : 0;
#pragma unroll
    for (int j = 0; j < NG; ++j)
#pragma unroll
      for (int m = 0; m < kM; ++m) x.t[j][m] = __builtin_amdgcn_raw_buffer_load_b128(rx, (at.t[j] + 16 * m) | off, so, 0);
    load_weights<FP8, RF, !FP8>(W, at.e, at.w, at.block, at.sc, at.b, on, lane, x.w);
    asm volatile("" ::: "memory");                       // issued here, not where they are used
    at.b += split;
    if (++at.s == steps) {
      at.i += stride;
      set_tile();
    }
  };

  float4v acc[NG][RF];
#pragma unroll
  for (int j = 0; j < NG; ++j)
#pragma unroll
    for (int f = 0; f < RF; ++f) acc[j][f] = float4v{0, 0, 0, 0};
  uint32_t less[NG];            // NVFP4: taken off the exponents of this lane's tokens
  auto scale_of = [&](int t) {  // the same for token t, as an exponent
    const int e = (int)(largest[t] >> 7) - 30;
    return e > 0 ? e : 0;
  };
  float r1 = 1.0f, r2 = 1.0f;   // NVFP4: 1 / the global scales of the tile that this wave finishes
  auto start = [&](int unit) {
    if constexpr (!FP8) {
      const int mine = unit * subs + wave, e = __builtin_amdgcn_readfirstlane(L.entry[wave < subs && mine < tiles ? entry_of(mine) : 0].e);
      r1 = 1.0f / uniform_load(p.gs_w1 + e);
      r2 = 1.0f / uniform_load(p.gs_w2 + e);
    }
    const int tile = unit * subs + sub;
    const Entry& y = L.entry[tile < tiles ? entry_of(tile) : 0];
#pragma unroll
    for (int j = 0; j < NG; ++j) {
      const int c = 4 * j + (r & 3);
      if constexpr (!FP8) less[j] = (uint32_t)scale_of(c < (int)y.count ? y.tok[c] : 0) * 0x00800080u;
    }
  };
  auto add = [&](Step& x) {
    float s0, s1;
    if constexpr (FP8) {
      s0 = g < 2 ? x.w.sc[0][0] : x.w.sc[0][1];
      s1 = g < 2 ? x.w.sc[1][0] : x.w.sc[1][1];
    } else {
      wave_order();                                      // the last step's scales are read
      *reinterpret_cast<int4v*>(&scales[wave].v[g][2 * r][0]) = x.w.s;
      wave_order();
#pragma unroll
      for (int j = 0; j < NG; ++j)
#pragma unroll
        for (int m = 0; m < kM; ++m)
#pragma unroll
          for (int i = 0; i < 4; ++i) x.t[j][m][i] = (int)move_exponents((uint32_t)x.t[j][m][i], less[j]);
    }
#pragma unroll
    for (int f = 0; f < RF; ++f) {
      float4v d[NG];
#pragma unroll
      for (int j = 0; j < NG; ++j) d[j] = FP8 ? float4v{0, 0, 0, 0} : acc[j][f];
      half2v s{0, 0};
      if constexpr (!FP8)
        s = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(scales[wave].v[r >> 2][4 * (f ^ (r >> 2)) + (r & 3)][g], 1.0f, false);
#pragma unroll
      for (int m = 0; m < kM; ++m) {
        const int4v w = decode8<FP8>(x.w.w[f], s, m);
#pragma unroll
        for (int j = 0; j < NG; ++j) d[j] = mfma<FP8>(w, x.t[j][m], d[j]);
      }
#pragma unroll
      for (int j = 0; j < NG; ++j) {
        if constexpr (FP8) {
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[j][f][i] = fmaf(d[j][i], f < 4 ? s0 : s1, acc[j][f][i]);
        } else {
          acc[j][f] = d[j];
        }
      }
    }
  };
  // the unit's sums over its waves and quarters, SwiGLU, and h in its 16 bits
  auto finish = [&](int unit) {
    if (split > 1) lds_barrier();                        // the last unit's sums are read
    else wave_order();
    if ((r >> 2) == g) {
#pragma unroll
      for (int j = 0; j < NG; ++j)
#pragma unroll
        for (int f = 0; f < RF; ++f) *reinterpret_cast<float4v*>(&S.sums[wave][g][4 * j + (r & 3)][FP8 ? 4 * f : 4 * (f ^ g)]) = acc[j][f];
    }
#pragma unroll
    for (int j = 0; j < NG; ++j)
#pragma unroll
      for (int f = 0; f < RF; ++f) acc[j][f] = float4v{0, 0, 0, 0};
    if (split > 1) lds_barrier();
    else wave_order();
    // a thread an output: 16 columns of four tokens a wave, as many waves as tiles
    if (wave >= subs) return;
    const int c = lane & 15, t = lane >> 4, tile = unit * subs + wave;
    const int gate = FP8 ? c : 16 * (c >> 3) + (c & 7), up = gate + (FP8 ? 16 : 8);
    if (tile >= tiles) return;
    const int u = entry_of(tile), row = L.entry[u].row, count = (int)L.entry[u].count;
#pragma unroll
    for (int j = 0; j < NG; ++j) {
      const int k = 4 * j + t;
      float a = 0.0f, b = 0.0f;
#pragma unroll 2
      for (int w = wave * split; w < (wave + 1) * split; ++w) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          a += S.sums[w][q][k][gate];
          b += S.sums[w][q][k][up];
        }
      }
      if (4 * j >= count) continue;                      // uniform
      const bool in = k < count;
      const int at_row = row + (in ? k : 0);
      const int64_t to = (int64_t)at_row * I + 16 * (tile - u * per) + c;
      if constexpr (FP8) {
        const float h = a / (1.0f + expf(-a)) * b * L.coef[at_row];
        const uint32_t hi = pack_bf16x2(h, 0.0f);
        const float rest = h - bf16_to_f32(hi & 0xFFFFu);
        if (in) {
          p.h_hi[to] = (uint16_t)hi;
          p.h_lo[to] = (uint16_t)pack_bf16x2(rest - rest == 0.0f ? rest : 0.0f, 0.0f);   // none of an infinity
        }
      } else {
        // back to x's own exponents; a token that is not finite gives NaN
        const int tok = L.entry[u].tok[in ? k : 0];
        const float back = largest[tok] >= 0x7F80u ? __uint_as_float(0x7FC00000u) : ldexpf(1.0f, scale_of(tok) - 112);
        a = a * r1 * back;
        b = b * r1 * back;
        const float h = a / (1.0f + expf(-a)) * b * L.coef[at_row] * r2;
        const int ex = __float_as_uint(max16(fabsf(h))) >> 23;
        const _Float16 v = (_Float16)ldexpf(h, 141 - ex);   // the 16 columns' largest: 2^14 .. 2^15
        if (in) {
          p.h_hi[to] = __builtin_bit_cast(uint16_t, v);
          if (c == 0) reinterpret_cast<uint8_t*>(p.h_lo)[to >> 4] = (uint8_t)ex;
        }
      }
    }
  };

  at.i = blockIdx.x;
  set_tile();
  Step x[2];
  issue(x[0]);
  int unit = blockIdx.x, s = 0;
  for (;;) {
#pragma unroll
    for (int d = 0; d < 2; ++d) {
      issue(x[d ^ 1]);
      if (s == 0) start(unit);
      add(x[d]);
      if (++s == steps) {
        finish(unit);
        unit += stride;
        if (unit >= units) return;
        s = 0;
      }
    }
  }
}

// ------------------------------------------------------------ down
//
// A tile is 4 * RF columns of out, over all entries: a workgroup's waves take the
// K steps of all entries in turn.  What a step gives its tokens is added to the
// wave's own sums in LDS, [token][quarter][column], so a token gets nothing from
// experts it did not choose, whatever these hold.
//
// Measured as above: one token FP8 21 us (117 MB), NVFP4 18 us (66 MB); sixteen FP8 223
// to 240 us (6.2 to 6.7 TB/s), NVFP4 164 to 175 us (4.8 to 5.1).  Bound by HBM; H 2048,
// I 768, one token and four NVFP4 experts, 5 us: by the ends.

template <bool FP8, int RF, int NG>
__global__ __launch_bounds__(kThreads, 2) void few_down_kernel(FewParams P) {
  constexpr int kCols = Format<FP8>::kCols, kM = Format<FP8>::kM, kTok = 4 * NG, kStride = 4 * RF + 4;
  const FewArgs& p = P.a;
  const Weights& W = P.w;
  __shared__ Live L;
  __shared__ union {
    LiveScratch build;
    float sums[kWaves][kFewTokens][4][kStride];
  } S;
  __shared__ Scales scales[FP8 ? 1 : kWaves];
  if (p.T * p.k <= 64) build_small(p, kTok, L, S.build);
  else build_large(p, kTok, L, S.build);

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int n = __builtin_amdgcn_readfirstlane(L.n), stride = gridDim.x, T = p.T;
  const int H = W.N, tiles = P.tiles;
  const int steps = (n * W.KS + kWaves - 1) / kWaves;
  const auto rh = rsrc_of(p.h_hi, P.t_bytes), rl = rsrc_of(p.h_lo, FP8 ? P.t_bytes : P.t_bytes / 32);
  const int lane_col = kCols / 4 * (r >> 2) + kCols / 16 * g;   // of this lane's tokens in a K step

  struct Step {
    StepW<FP8, RF> w;
    int4v t[NG][FP8 ? 2 : 1][kM];
    uint64_t ex[FP8 ? 1 : NG];  // NVFP4: the exponents of the lane's quarter's 8 x 16 columns
    int tok[NG];                // the token of this lane's results, or -1
    int cut;                    // FP8: row groups in the tile's first row block
  };
  struct {
    int i, s, u, b;
    int w[RF], block[2], cut;
    uint32_t sc;
    uint4 y;                    // the entry, read one step before it is used
  } at;
  auto set_entry = [&]() { at.y = *reinterpret_cast<const uint4*>(&L.entry[at.u < n ? at.u : 0]); };
  auto set_tile = [&]() {
    at.s = 0;
    at.u = 0;
    for (at.b = wave; at.b >= W.KS; at.b -= W.KS) ++at.u;
    const int row0 = 4 * RF * at.i;
    at.sc = scale_place<RF>(row0, H, W.KB, lane);
#pragma unroll
    for (int f = 0; f < RF; ++f) at.w[f] = group_at<FP8>(W, row0 + 4 * f < H ? row0 + 4 * f : H - 4);   // none behind the last row
    at.block[0] = (row0 < H ? row0 : H - 4) / 128;
    at.block[1] = (row0 + 4 * RF < H ? row0 + 4 * RF - 4 : H - 4) / 128;
    at.cut = (at.block[0] + 1) * 32 - row0 / 4;
    set_entry();
  };
  auto issue = [&](Step& x) {
    const bool on = at.i < tiles && at.u < n;
    const int so = on ? at.b * kCols * 2 : 0;
    const int e = __builtin_amdgcn_readfirstlane(at.y.x & 0xFFFF), row = at.y.x >> 16;
    const int count = on && lane_col < W.K - at.b * kCols ? (int)at.y.y : 0;
#pragma unroll
    for (int j = 0; j < NG; ++j) {
      const int c = 4 * j + (r & 3);
      const bool in = c < count;
      const uint32_t t = in ? (uint32_t)(row + c) * (uint32_t)W.K * 2 + 2 * lane_col : kNowhere;
#pragma unroll
      for (int m = 0; m < kM; ++m) {
        x.t[j][0][m] = __builtin_amdgcn_raw_buffer_load_b128(rh, t + 16 * m, so, 0);
        if constexpr (FP8) x.t[j][FP8 ? 1 : 0][m] = __builtin_amdgcn_raw_buffer_load_b128(rl, t + 16 * m, so, 0);
      }
      if constexpr (!FP8)
        x.ex[j] = __builtin_bit_cast(uint64_t, __builtin_amdgcn_raw_buffer_load_b64(rl, in ? (uint32_t)(row + c) * (uint32_t)(W.K / 16) + 8 * (r >> 2) : kNowhere, on ? at.b * 32 : 0, 0));
      // a lane of equal quarters has its token's results, in or behind K
      x.tok[j] = on && c < (int)at.y.y && (r >> 2) == g ? (int)((j ? at.y.w : at.y.z) >> (8 * (r & 3)) & 255) : -1;
    }
    load_weights<FP8, RF, false>(W, e, at.w, at.block, at.sc, at.b, on, lane, x.w);
    x.cut = at.cut;
    asm volatile("" ::: "memory");                       // issued here, not where they are used
    if (++at.s == steps) {
      at.i += stride;
      set_tile();
    } else {
      at.b += kWaves;
      if (at.b >= W.KS) {
        do { at.b -= W.KS; ++at.u; } while (at.b >= W.KS);
        set_entry();
      }
    }
  };
  auto add = [&](Step& x) {
    float s0, s1, back[NG];
    wave_order();                                        // the last step's sums are written, by other lanes of a token, and its scales read
    if constexpr (FP8) {
      s0 = g < 2 ? x.w.sc[0][0] : x.w.sc[0][1];
      s1 = g < 2 ? x.w.sc[1][0] : x.w.sc[1][1];
    } else {
      *reinterpret_cast<int4v*>(&scales[wave].v[g][2 * r][0]) = x.w.s;
      wave_order();
#pragma unroll
      for (int j = 0; j < NG; ++j) {
        // this quarter's columns to one power of two: its largest
        const uint32_t lo = (uint32_t)x.ex[j], hi = (uint32_t)(x.ex[j] >> 32), own = (g < 2 ? lo : hi) >> (16 * (g & 1));
        int top = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) top = max(top, max((int)(lo >> (8 * i) & 255), (int)(hi >> (8 * i) & 255)));
        auto shift = [&](int d0, int d1) {
          const _Float16 p0 = __builtin_ldexpf16((_Float16)1.0f, d0), p1 = __builtin_ldexpf16((_Float16)1.0f, d1);
          const half2v f0{p0, p0}, f1{p1, p1};
#pragma unroll
          for (int m = 0; m < kM; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int two = x.t[j][0][m][i];
              x.t[j][0][m][i] = __builtin_bit_cast(int, __builtin_bit_cast(half2v, two) * (m < 2 ? f0 : f1));
            }
        };
        // FP16's least power of two is 2^-24: what lies further below takes two factors
        const int d0 = (int)(own & 255) - top, d1 = (int)(own >> 8 & 255) - top;
        shift(max(d0, -24), max(d1, -24));
        if (__any(min(d0, d1) < -24)) shift(min(d0 + 24, 0), min(d1 + 24, 0));
        back[j] = ldexpf(1.0f, top - 141);
      }
    }
#pragma unroll
    for (int f = 0; f < RF; ++f) {
      float4v d[NG];
#pragma unroll
      for (int j = 0; j < NG; ++j) d[j] = float4v{0, 0, 0, 0};
      half2v s{0, 0};
      if constexpr (!FP8) s = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(scales[wave].v[r >> 2][4 * f + (r & 3)][g], 1.0f, false);
#pragma unroll
      for (int m = 0; m < kM; ++m) {
        const int4v w = decode8<FP8>(x.w.w[f], s, m);
#pragma unroll
        for (int j = 0; j < NG; ++j) {
          d[j] = mfma<FP8>(w, x.t[j][0][m], d[j]);
          if constexpr (FP8) d[j] = mfma<FP8>(w, x.t[j][FP8 ? 1 : 0][m], d[j]);
        }
      }
#pragma unroll
      for (int j = 0; j < NG; ++j) {
        if (x.tok[j] < 0) continue;
        const float sc = !FP8 ? back[j] : f < x.cut ? s0 : s1;
        float4v* to = reinterpret_cast<float4v*>(&S.sums[wave][x.tok[j]][g][4 * f]);
        float4v v = *to;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = fmaf(d[j][i], sc, v[i]);
        *to = v;
      }
    }
  };
  auto clear = [&]() {
    float4v* own = reinterpret_cast<float4v*>(&S.sums[wave][0][0][0]);
    for (int i = lane; i < T * kStride; i += 64) own[i] = float4v{0, 0, 0, 0};
  };
  // the tile's sums over waves and quarters, and out
  auto finish = [&](int i) {
    lds_barrier();
    const int q = threadIdx.x & 3;
    for (int o = threadIdx.x >> 2; o < T * 4 * RF; o += kWaves * 16) {
      const int t = o / (4 * RF), c = o - t * (4 * RF);
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) v += S.sums[w][t][q][c];
      v += __shfl_xor(v, 1);
      v += __shfl_xor(v, 2);
      if (q == 0 && 4 * RF * i + c < H) p.out[(int64_t)t * H + 4 * RF * i + c] = (uint16_t)pack_bf16x2(v, 0.0f);
    }
    lds_barrier();
    clear();
  };

  at.i = blockIdx.x;
  set_tile();
  Step x[2];
  issue(x[0]);
  clear();
  if (steps == 0) {                                      // no token has an expert
    for (int i = blockIdx.x; i < tiles; i += stride) finish(i);
    return;
  }
  int i = blockIdx.x, s = 0;
  for (;;) {
#pragma unroll
    for (int d = 0; d < 2; ++d) {
      issue(x[d ^ 1]);
      add(x[d]);
      if (++s == steps) {
        finish(i);
        i += stride;
        if (i >= tiles) return;
        s = 0;
      }
    }
  }
}

template <bool FP8>
Weights weights_of(const uint8_t* q, const void* sf, int64_t N, int64_t K) {
  Weights w;
  w.q = q;
  w.sf = static_cast<const uint8_t*>(sf);
  w.N = (int)N;
  w.K = (int)K;
  w.KB = (int)((K + 127) / 128);
  w.KS = (int)((K + Format<FP8>::kCols - 1) / Format<FP8>::kCols);
  w.q_bytes = FP8 ? N * K : packed_rows(N) * (K / 2);
  w.sf_bytes = FP8 ? (N + 127) / 128 * w.KB * 4 : packed_rows(N) * (K / 16);
  return w;
}

template <bool FP8, int NG>
hipError_t launch(const FewArgs& a, int cus, hipStream_t stream) {
  auto up = [](int64_t x, int64_t y) { return (x + y - 1) / y; };
  const int64_t pairs = (int64_t)a.T * a.k, live = pairs < a.E ? pairs : a.E;
  FewParams p;
  p.a = a;
  p.w = weights_of<FP8>(a.w1_q, a.w1_sf, 2 * a.I, a.H);
  p.tiles = (int)(a.I / 16);
  p.inv_tiles = 1.0f / (float)p.tiles;
  p.t_bytes = (int64_t)a.T * a.H * 2;
  const int64_t tiles = (live + pairs / (4 * NG)) * p.tiles;   // at most: entries are full but for one an expert
  const int grid = (int)(tiles < cus ? tiles : cus);
  p.inv_grid = 1.0f / (float)grid;
  few_up_kernel<FP8, NG><<<grid, kThreads, 0, stream>>>(p);
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  p.w = weights_of<FP8>(a.w2_q, a.w2_sf, a.H, a.I);
  p.t_bytes = pairs * a.I * 2;
  auto down = [&](auto rf) {
    constexpr int RF = decltype(rf)::value;
    p.tiles = (int)up(a.H, 4 * RF);
    few_down_kernel<FP8, RF, NG><<<p.tiles < cus ? p.tiles : cus, kThreads, 0, stream>>>(p);
  };
  // Columns a tile: those that make about one tile a CU (7168: 28 columns, one token
  // FP8 22 us, 32 columns 26, 16 columns in two rounds 28; 2048: 8 columns, four tokens,
  // 14.5 us, 16 columns 17.9), eight at least.
  if (a.H <= 8 * cus) down(std::integral_constant<int, 2>{});
  else if (a.H <= 16 * cus) down(std::integral_constant<int, 4>{});
  else if (a.H <= 28 * cus) down(std::integral_constant<int, 7>{});
  else down(std::integral_constant<int, 8>{});
  return hipGetLastError();
}

}  // namespace

hipError_t launch_few(const FewArgs& a, hipStream_t stream) {
  int cus = 0;
  const hipError_t err = device_cus(cus);
  if (err != hipSuccess) return err;
  // Entries of eight tokens, two groups an instruction's weights, from more than two
  // tokens an expert on average (7168, 2048, 32 experts, both products: four tokens each
  // FP8 257 us and NVFP4 184, in entries of four 311 and 212; three each FP8 244, in fours
  // 261; two each 215 and 150, in fours 211 and 144).  All of that was routed evenly: an
  // expert of many tokens among few pairs is read once for every four of them (one
  // expert of sixteen tokens alone: FP8 38.6 us, 176 MB; 44 MB would be its weights once).
  const bool busy = a.T > 4 && (int64_t)a.T * a.k > 2 * (int64_t)a.E;
  if (a.fp8) return busy ? launch<true, 2>(a, cus, stream) : launch<true, 1>(a, cus, stream);
  return busy ? launch<false, 2>(a, cus, stream) : launch<false, 1>(a, cus, stream);
}

}  // namespace nvfp4
