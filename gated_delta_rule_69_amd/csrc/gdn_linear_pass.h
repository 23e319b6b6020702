// The chunked pass of linear attention with one decay a head.
//
// A pass runs over the positions 0 .. n-1 of every (sequence, head) and computes, for rows
// a, b of DA channels and c of DC channels and with l = e^g,
//     X_p = l X_{p-1} + b_p c_p^T,     out_p = X_p^T a_p         (X_{-1} given)
// The forward pass is (a, b, c) = (q, k, v). The gradients are passes too: with do the
// upstream gradient, dq is (do, v, k) from the transposed state; and from the last token to
// the first, dv is (k, q, do) and dk is (v, do, q), whose state G meets its first row
// undecayed (`shift` = 1: the state before a position is already l times the one after).
//
// In a chunk of C positions with start state X,
//     out = (mask(a b^T)) c + Diag(l^{i+1}) a X,   X' = l^n X + b^T Diag(l^{n-1-j}) c
// with mask_ij = l^{i-j} for j <= i. All four products run on bf16 MFMA 16x16x32. Factors
// that are not bf16 values enter as sums of bf16 parts x = x0 + x1 (+ x2), each the rounding
// of what is left (8 bits a part, float32's range). The weighted c of the state update is three
// parts (2^-24), so that the state is a float32 sum on either type. Of bf16 inputs the masked
// scores and the state as it enters a X are two (2^-16 at most, under the output's 2^-8): three of
// the state take 382 us for 359 at the long prompt below and 145 for 133 for the 4K gradients,
// three of the scores the LDS of a second workgroup, and the outputs are as far from float64
// either way, 1.7e-3. Float32 inputs are three parts themselves, and of the nine products of
// parts the six above 2^-24 are formed: results 2 to 3e-7 from float64. By the instructions'
// rates six bf16 products are 2.7 times as fast as the float32 MFMA.
//
// One workgroup runs one segment of a head. Its waves share the chunk's tiles in LDS and
// split the DC columns of the state, sixteen a wave, which it keeps in accumulators: an
// accumulator tile is, register for register, the operand of the next chunk's a X, with
// its rows spread so that eight consecutive channels of `a` are one 16-byte LDS read.
// Operands with positions as the summed index are read transposed (ds_read_b64_tr_b16).
// Outputs are formed transposed, so that a lane holds consecutive channels of one row.
#pragma once

#include <type_traits>

#include "gdn_layer.h"
#include "gdn_layer_device.h"

namespace gdn {

struct LinearPass {
  const void *a, *b, *c;
  void* out;
  int64_t lda, ldb, ldc;       // elements from token to token
  int group_a, group_b, group_c;  // value heads a head of a, b, c serves
  int H;
  int64_t T;
  const float* log_decay;
  const int32_t* seq_lens;
  const float* x0;             // state before position 0: (i, j) at x0[i * x0_sa + j * x0_sc]; NULL: zero
  float* x1;                   // state after the last position, the same way; NULL: not wanted
  int64_t x0_sa, x0_sc;
  float* states;               // state before segment s of every (b, h), DA * DC floats each (nseg > 1; slot 0 only with x0)
  int64_t st_sa, st_sc;
  int64_t seg;                 // positions a segment, a multiple of the chunk
  int nseg;
  int shift;
  int zero_tail;               // write zeros to rows behind the sequence
  int back;                    // from the last token to the first
};

// Passes of one launch, all of the same dimensions: blockIdx.y tells which.
constexpr int kMostPasses = 3;
struct LinearPasses {
  LinearPass pass[kMostPasses];
};

// log of a head's decay; everything below e^-128 is taken as 0, -Inf included.
__device__ __forceinline__ float head_log_decay(const float* g, int h) {
  const float x = g[h];
  return x < -128.0f ? -128.0f : x;
}

// e^g as hi + lo. Rounded to hi alone a token's decay is off by up to 2^-25, the same way at
// every token, and a state that keeps some 1 / |g| tokens adds that up to 2^-25 / |g|: 1.3e-4 of
// the state at g = -1e-4 in 20,000 tokens, where the state's own roundings come to 2e-6. A
// chunk's or a segment's decay is applied less often and adds up to 4.5e-5 at g = -3e-6 in
// 131,072 tokens. From a factor of e^-1/2 on it is gone before it adds up.
__device__ __forceinline__ void two_floats(float g, float* hi, float* lo) {
  const float less = expm1f(g);
  const bool slow = fabsf(g) < 0.5f;
  *hi = slow ? 1.0f + less : expf(g);
  *lo = slow ? less - (*hi - 1.0f) : 0.0f;
}

// Tokens of sequence b.
__device__ __forceinline__ int64_t length_of(const int32_t* lens, int64_t b, int64_t T) {
  if (lens == nullptr) return T;
  const int64_t n = lens[b];
  return n < 0 ? 0 : n > T ? T : n;
}

template <typename E> struct PassShape {
  static constexpr bool kHalf = sizeof(E) == 2;
  static constexpr int kParts = kHalf ? 1 : 3;      // parts of an input
  static constexpr int kScoreParts = kHalf ? 2 : 3; // parts of the scores and of the state
  static constexpr int kChunk = kHalf ? 64 : 32;
};
constexpr int pass_waves(int DC) { return DC / 16; }  // sixteen columns of the state a wave
// Bytes of LDS of a workgroup of the outputs' kernel (asserted there): tiles of a, b and c,
// scores, weights, decays and what the last leaves out, and an int a column.
constexpr int outputs_lds(bool half, int DA, int DC) {
  const int C = half ? 64 : 32, parts = half ? 1 : 3;
  const int tiles = 2 * parts * C * ((half ? 3 : 2) * DA + DC), scores = half ? 4 * 32 * (32 + 64) : 6 * (32 * 32 + 64);
  return (tiles + scores + 4 * (2 * C + C + 2 + DC) + 15) / 16 * 16;
}

// x[0..N) as sums of PARTS bf16 values part[p][i], two at a time: one packed conversion,
// and what is left by subtracting its halves, which are floats but for their position.
template <int PARTS, int N>
__device__ __forceinline__ void split_parts(const float* x, vec<__bf16, N>* part) {
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    float2v rest = {x[i], x[i + 1]};
#pragma unroll
    for (int p = 0; p < PARTS; ++p) {
      const bhalf2 r = __builtin_convertvector(rest, bhalf2);
      part[p][i] = r[0], part[p][i + 1] = r[1];
      if (p + 1 < PARTS) {
        const uint32_t u = __builtin_bit_cast(uint32_t, r);
        rest[0] -= __uint_as_float(u << 16);
        rest[1] -= __uint_as_float(u & 0xffff0000u);
      }
    }
  }
}

__device__ __forceinline__ float4v mma(bhalf8 a, bhalf8 b, float4v acc) { return mma_pair_bf16(a, b, acc); }

// acc[t] += the products of the parts of a[t] and b[t], the smallest first; those of order
// above MOST are left out. Each product goes round the N tiles, so that neighbouring
// instructions do not wait for one another.
template <int N, int PA, int PB, int MOST, typename A, typename B>
__device__ __forceinline__ void mma_parts(A a, B b, float4v* acc) {
#pragma unroll
  for (int order = MOST; order >= 0; --order)
#pragma unroll
    for (int p = 0; p < PA; ++p)
      if (order - p >= 0 && order - p < PB) {
#pragma unroll
        for (int t = 0; t < N; ++t) acc[t] = mma(a(t, p), b(t, order - p), acc[t]);
      }
}

typedef __attribute__((address_space(3))) bhalf4 lds_bhalf4;
__device__ __forceinline__ bhalf4 read_tr(const __bf16* p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bhalf4*)(p));
}
__device__ __forceinline__ bhalf8 join(bhalf4 lo, bhalf4 hi) { return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7); }

// A tile of C rows of D channels, PARTS planes of 16-byte slots. Slot c of a row lies at
// c ^ turn(row), so that the lanes served together by a 16-byte read of rows (measured: rows
// 0-3 and 12-15 of one k-group with 4-11 of the next) and those of a transposed read (four
// rows, four slots) fall into different banks: 4.3 cycles a wave's 16-byte read and 4.3 or
// 2.6 a transposed one, against 8.1 and 4.3 to 8.1 for simpler turns and 32 and 16 for none.
template <int C, int D, int PARTS> struct Tile {
  static constexpr int kSlots = D / 8;
  static constexpr int kPlane = C * D;
  __align__(16) __bf16 x[PARTS * kPlane];

  // Bits 2 and 3 of the row turn the low two bits of the slot (2 and 3: their sum is 1),
  // bits 0 and 1 the high ones where a row fills or half fills the banks.
  __device__ static __forceinline__ int turn(int row) {
    if constexpr (kSlots == 2) return row >> 3 & 1;
    const int low = (row >> 1 & 2) ^ (row >> 3 & 1) * 3;
    if constexpr (kSlots == 16) return (row & 3) << 2 | low;
    if constexpr (kSlots == 8) return (row & 2) << 1 | low;
    return low;
  }
  // place of channels col .. col+3 (or a whole slot) of a row
  __device__ static __forceinline__ int place(int row, int col) {
    return row * D + ((col / 8) ^ turn(row)) * 8 + (col & 4);
  }
  // A lane's place for row(): row i, its eight channels of a k-block (four of sixteen).
  __device__ static __forceinline__ int row_place(int i, int g) { return place(i, D == 16 ? 4 * g : 8 * g); }
  // rows 16 r + i, channels of k-block kb: the order of the state's accumulator tiles
  __device__ __forceinline__ bhalf8 row(int p, int r, int kb, int at) const {
    const __bf16* from = x + p * kPlane + 16 * r * D + (at ^ 32 * kb);
    if constexpr (D == 16) return join(*reinterpret_cast<const bhalf4*>(from), bhalf4{});
    else return *reinterpret_cast<const bhalf8*>(from);
  }
  // A lane's place for columns(): of the positions 8 g + e of a k-block, it reads the four
  // channels at `column` + (i % 4) step of position i / 4 (and of i / 4 + 4).
  __device__ static __forceinline__ int column_place(int column, int step, int i, int g) {
    return place(8 * g + i / 4, column + (i % 4) * step);
  }
  // positions 32 kb + 8 g + e of channel column + (i / 4) step + i % 4, read transposed;
  // `block` moves the column by 32 channels, `half` by four
  __device__ __forceinline__ bhalf8 columns(int p, int kb, int at, int block, int half) const {
    const __bf16* from = x + p * kPlane + 32 * kb * D + 4 * half;
    const int near = at ^ 32 * block, far = kSlots == 2 ? near : near ^ 16;  // four rows on, turn() differs by 2
    return join(read_tr(from + near), read_tr(from + 4 * D + far));
  }
  __device__ __forceinline__ void put4(int p, int row, int col, bhalf4 v) {
    *reinterpret_cast<bhalf4*>(x + p * kPlane + place(row, col)) = v;
  }
};

// The masked scores of a chunk: of 64 positions, the first half's rows hold 32 columns.
template <int C, int PARTS> struct Scores {
  Tile<32, 32, PARTS> first;
  Tile<C == 64 ? 32 : 1, 64, PARTS> second;
  __device__ __forceinline__ void put4(int p, int row, int col, bhalf4 v) {
    if (C == 64 && row >= 32) second.put4(p, row - 32, col, v);
    else first.put4(p, row, col, v);
  }
  __device__ __forceinline__ bhalf8 row(int p, int r, int kb, int at_first, int at_second) const {
    return r < 2 ? first.row(p, r, kb, at_first) : second.row(p, r - 2, kb, at_second);
  }
};

// A tile's way from memory to LDS. Rows 0 .. rows-1 come from `base` on, `step` bytes apart
// (the last first, going backwards); the others are zero: their offsets lie outside the
// range. Token strides are at most 2^24 elements, so a tile's offsets fit in 31 bits.
//
// bf16 rows go straight to LDS (buffer_load_dwordx4 ... lds: lane l's 16 bytes land at the
// wave's base + 16 l, so the tile's slots are chosen by where a lane loads from). The
// loads are written as assembly, which has no registers to guard and leaves the waiting to
// wait_loads(); the compiler's own counts only ever wait for more.
template <int C, int D, int NT> struct Direct {
  static constexpr int kSlots = D / 8, kAll = C * kSlots;
  static constexpr int kRows = NT / kSlots;        // rows a step of the workgroup covers
  static constexpr bool kSame = kRows % 16 == 0;   // so that turn() is the same in each
  bool back;
  uint32_t step;    // bytes from row to row
  uint32_t offset;  // of the thread's slot of its first row
  __device__ __forceinline__ uint32_t offset_of(uint32_t at) const {
    const uint32_t row = at / kSlots, to = (at % kSlots ^ Tile<C, D, 1>::turn(row)) * 16;
    return back ? to - row * step : to + row * step;
  }
  __device__ __forceinline__ Direct(int64_t ld, bool back_) : back(back_), step(uint32_t(ld * 2)), offset(offset_of(threadIdx.x)) {}
  __device__ __forceinline__ void load(Tile<C, D, 1>& t, const __bf16* base, int rows) const {
    typedef uint32_t uint4v __attribute__((ext_vector_type(4)));
    auto uniform = [](uint32_t x) { return uint32_t(__builtin_amdgcn_readfirstlane(int(x))); };
    const uint64_t from = reinterpret_cast<uintptr_t>(base);
    const uint32_t top = uint32_t(rows - 1) * step, from_end = back ? top : 0;
    const uint4v range = {uniform(uint32_t(from)), uniform(uint32_t(from >> 32) & 0xffffu), uniform(top + 2 * D), 0x00020000u};
    const uint32_t lds = uint32_t(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) __bf16*)(t.x)));
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
#pragma unroll
    for (int n = 0; n < (kAll + NT - 1) / NT; ++n) {
      const int first = n * NT + 64 * wave;
      if (kAll % NT != 0 && first >= kAll) break;
      const uint32_t here = kSame ? offset + (back ? 0u - uint32_t(n * kRows) * step : uint32_t(n * kRows) * step) + from_end
                                  : offset_of(n * NT + threadIdx.x) + from_end;
      asm volatile("s_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                   :: "{m0}"(uniform(lds + 16 * first)), "v"(here), "s"(range) : "memory");
    }
  }
};
__device__ __forceinline__ void wait_loads() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// float32 rows pass through registers, where they become three bf16 planes.
template <int C, int D, int NT> struct Staged {
  static constexpr int kPerRow = D / 4;
  static constexpr int kCount = (C * kPerRow + NT - 1) / NT;
  uint4 v[kCount];
  bool back;
  uint32_t step;
  __device__ __forceinline__ Staged(int64_t ld, bool back_) : back(back_), step(uint32_t(ld * 4)) {}
  __device__ __forceinline__ void load(const float* base, int rows) {
    const auto range = __builtin_amdgcn_make_buffer_rsrc(const_cast<float*>(base), 0, uint32_t(rows - 1) * step + 4 * D, 0x00020000);
#pragma unroll
    for (int n = 0; n < kCount; ++n) {
      const uint32_t at = threadIdx.x + n * NT, row = at / kPerRow, col = at % kPerRow;
      v[n] = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(range, (back ? uint32_t(rows - 1) - row : row) * step + col * 16, 0, 0));
    }
  }
  template <int PARTS>
  __device__ __forceinline__ void store(Tile<C, D, PARTS>& t) const {
#pragma unroll
    for (int n = 0; n < kCount; ++n) {
      const int at = threadIdx.x + n * NT, row = at / kPerRow, col = at % kPerRow;
      if (C * kPerRow % NT != 0 && row >= C) break;
      const float f[4] = {__uint_as_float(v[n].x), __uint_as_float(v[n].y), __uint_as_float(v[n].z), __uint_as_float(v[n].w)};
      bhalf4 part[PARTS];
      split_parts<PARTS, 4>(f, part);
#pragma unroll
      for (int p = 0; p < PARTS; ++p) t.put4(p, row, 4 * col, part[p]);
    }
  }
};

// Whether one of eight bf16 values is a NaN or Inf.
__device__ __forceinline__ bool any_bad(bhalf8 x) {
  typedef uint32_t uint4v __attribute__((ext_vector_type(4)));
  const uint4v w = (__builtin_bit_cast(uint4v, x) & 0x7f807f80u) + 0x00800080u;
  return ((w[0] | w[1] | w[2] | w[3]) & 0x80008000u) != 0;
}
__device__ __forceinline__ bool is_bad(__bf16 x) { return (__builtin_bit_cast(uint16_t, x) & 0x7f80u) == 0x7f80u; }

// What both kernels of a pass know of their workgroup's segment, and the state of a wave's
// sixteen columns in accumulators.
template <typename E, int DA, int DC> struct Segment {
  static constexpr int C = PassShape<E>::kChunk, NT = 64 * pass_waves(DC), KT = DA / 16;
  const LinearPass& s;
  int wave, i, g, h, seg;
  int n, begin, last, end;  // end: the segment's last real position + 1; last: of any
  int64_t b, bh;
  float lg;                            // log2 of the decay

  // Workgroups go over heads, segments and sequences, the heads first or last: last for the
  // states, whose work goes by the head's decay, so that a CU gets heads of different ones
  // (98 -> 90 us at the long prompt); first for the outputs, whose work goes by the sequence's
  // length (a padded float32 batch 126 against 160 us a call).
  __device__ __forceinline__ Segment(const LinearPass& s_, int segs, bool heads_last) : s(s_) {
    wave = threadIdx.x / 64;
    const int lane = threadIdx.x % 64;
    i = lane % 16, g = lane / 16;
    const unsigned per = heads_last ? gridDim.x / unsigned(s.H) : unsigned(s.H);
    unsigned bs = blockIdx.x / per;
    h = int(blockIdx.x - bs * per);
    if (heads_last) {
      const unsigned rest = unsigned(h);
      h = int(bs), bs = rest;
    }
    const unsigned bq = bs / unsigned(segs);
    seg = int(bs - bq * unsigned(segs));
    b = bq;
    bh = b * s.H + h;
    n = __builtin_amdgcn_readfirstlane(int(length_of(s.seq_lens, b, s.T)));
    lg = head_log_decay(s.log_decay, h) * 1.44269504088896341f;
    begin = int(seg * s.seg);
    last = int(begin + s.seg < s.T ? begin + s.seg : s.T);
    end = last < n ? last : n;
  }
  __device__ __forceinline__ float power(int m) const { return __builtin_amdgcn_exp2f(lg * float(m)); }
  __device__ __forceinline__ int size(int p) const { return end - p < C ? end - p : C; }  // positions of the chunk at p
  // first token in memory of positions p .. p + m - 1: token p, or n - m - p backwards
  __device__ __forceinline__ const E* rows(const void* x, int64_t ld, int group, int d, int p) const {
    return static_cast<const E*>(x) + (b * s.T + int64_t(s.back ? n - size(p) - p : p)) * ld + int64_t(h / group) * d;
  }
  // a lane's first channel in state tile kt (four rows), and its column
  __device__ __forceinline__ int row_channel(int kt) const { return KT == 1 ? 4 * g : 32 * (kt / 2) + 8 * g + 4 * (kt % 2); }
  __device__ __forceinline__ int column() const { return 16 * wave + i; }

  __device__ __forceinline__ void load_state(float4v (&X)[KT], const float* from, int64_t sa, int64_t sc) const {
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) {
      if (from == nullptr) {
        X[kt] = float4v{0.0f, 0.0f, 0.0f, 0.0f};
      } else if (sa == 1) {
        X[kt] = *reinterpret_cast<const float4v*>(from + row_channel(kt) + column() * sc);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) X[kt][e] = from[(row_channel(kt) + e) * sa + column() * sc];
      }
    }
  }
  __device__ __forceinline__ void store_state(const float4v (&X)[KT], float* to, int64_t sa, int64_t sc) const {
    if (to == nullptr) return;
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) {
      if (sa == 1) {
        *reinterpret_cast<float4v*>(to + row_channel(kt) + column() * sc) = X[kt];
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) to[(row_channel(kt) + e) * sa + column() * sc] = X[kt][e];
      }
    }
  }
};

// c of a k-block of positions for the wave's columns, and c times its positions' weights.
template <typename E, int DC, typename T>
__device__ __forceinline__ void weighted(const T& tile, const float* weight, int kb, int at, int g, bhalf8* cv, float* x) {
  constexpr int P = PassShape<E>::kParts;
#pragma unroll
  for (int q = 0; q < P; ++q) {
    cv[q] = tile.columns(q, kb, at, 0, 0);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = q == 0 ? float(cv[q][e]) : x[e] + float(cv[q][e]);
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] *= weight[32 * kb + 8 * g + e];
}

// X += b^T (weighted c) of a k-block of positions, three parts of c: a float32 sum.
template <typename E, int DA, typename T>
__device__ __forceinline__ void add_outer(float4v* X, const T& tile, int kb, int at, const float* x) {
  constexpr int P = PassShape<E>::kParts, W = 3, KT = DA / 16, N = KT < 2 ? KT : 2;
  bhalf8 wv[W];
  split_parts<W, 8>(x, wv);
#pragma unroll
  for (int kt = 0; kt < KT; kt += N) {
    bhalf8 bv[N][P];
#pragma unroll
    for (int t = 0; t < N; ++t)
#pragma unroll
      for (int q = 0; q < P; ++q) bv[t][q] = tile.columns(q, kb, at, (kt + t) / 2, (kt + t) % 2);
    mma_parts<N, P, W, W - 1>([&](int t, int p) { return bv[t][p]; }, [&](int, int p) { return wv[p]; }, X + kt);
  }
}

// The states after segments 0 .. nseg-2, each from zero (the first from x0): the sum of
// l^{end-1-p} b_p c_p^T, for scan_states to join. A segment is walked from its end, so that
// nothing is scaled on the way, the positions whose weight is under 2^-127 (0 in float32)
// are never read, and what the outputs' kernel reads first was read here last.
//
// Barriers and instructions bound it: at B2 T32768 H16 d128 bf16 90 us, 80 with its loads left
// out and 116 with its arithmetic left out before it passed over what counts nothing (332 of
// 503 MB are read). Float32 B8 T2047 H32 d64, padded: 39 us.
template <typename E, int DA, int DC>
__global__ __launch_bounds__(64 * pass_waves(DC), PassShape<E>::kHalf ? 4 : 2) void linear_states_kernel(LinearPasses all) {
  const LinearPass s = all.pass[blockIdx.y];
  using S = PassShape<E>;
  constexpr int C = S::kChunk, NT = 64 * pass_waves(DC), P = S::kParts;
  constexpr bool kDirect = S::kHalf;
  struct Shared {
    Tile<C, DA, P> b[kDirect ? 2 : 1];
    Tile<C, DC, P> c[kDirect ? 2 : 1];
    float weight[2][C];
  };
  __shared__ Shared sh;
  const Segment<E, DA, DC> me(s, s.nseg - 1, true);
  float4v X[DA / 16];
  float* slots = s.states + me.bh * s.nseg * (DA * DC);
  const int begin = me.begin, end = me.end;
  const bool first = me.seg == 0 && s.x0 != nullptr;
  me.load_state(X, first ? s.x0 + me.bh * (DA * DC) : nullptr, s.x0_sa, s.x0_sc);
  // x0 may be overwritten by the last segment's state while the first segment's outputs are
  // still to come: they read this copy
  if (first) me.store_state(X, slots, s.st_sa, s.st_sc);
  const float whole = me.power(end > begin ? end - begin : 0);
#pragma unroll
  for (int kt = 0; kt < DA / 16; ++kt) X[kt] *= whole;

  std::conditional_t<kDirect, Direct<C, DA, NT>, Staged<C, DA, NT>> rb(s.ldb, s.back);
  std::conditional_t<kDirect, Direct<C, DC, NT>, Staged<C, DC, NT>> rc(s.ldc, s.back);
  auto fetch = [&](int p, int buf) {
    const E *fb = me.rows(s.b, s.ldb, s.group_b, DA, p), *fc = me.rows(s.c, s.ldc, s.group_c, DC, p);
    if constexpr (kDirect) rb.load(sh.b[buf], fb, me.size(p)), rc.load(sh.c[buf], fc, me.size(p));
    else rb.load(fb, me.size(p)), rc.load(fc, me.size(p));
  };
  const int at_b = Tile<C, DA, P>::column_place(0, DA == 16 ? 4 : 8, me.i, me.g);
  const int at_c = Tile<C, DC, P>::column_place(16 * me.wave, 4, me.i, me.g);
  int p = end > begin ? begin + (end - 1 - begin) / C * C : begin - C;
  if (p >= begin) fetch(p, 0);
  for (int buf = 0; p >= begin; p -= C, buf ^= 1) {
    const bool more = p - C >= begin && me.lg * float(end - p + s.shift) > -127.0f;
    if constexpr (kDirect) wait_loads();
    else rb.store(sh.b[0]), rc.store(sh.c[0]);
    if (threadIdx.x < C) {
      const int left = end - 1 - p - int(threadIdx.x);
      sh.weight[buf][threadIdx.x] = left >= 0 ? me.power(left + s.shift) : 0.0f;
    }
    __syncthreads();
    if (more) fetch(p - C, buf ^ 1);
    const int at = kDirect ? buf : 0;
#pragma unroll
    for (int kb = 0; kb < C / 32; ++kb) {
      bhalf8 cv[P];
      float x[8];
      weighted<E, DC>(sh.c[at], sh.weight[buf], kb, at_c, me.g, cv, x);
      add_outer<E, DA>(X, sh.b[at], kb, at_b, x);
    }
    if (!more) break;
    if constexpr (!kDirect) __syncthreads();
  }
  me.store_state(X, slots + (me.seg + 1) * (DA * DC), s.st_sa, s.st_sc);
}

// The outputs of a segment, chunk by chunk from the state before it; the last segment's
// workgroup also has the pass's last state.
//
// At B2 T32768 H16 d128 bf16 it takes 234 us at best for 1.07 GB (4.6 TB/s), 279 on average
// under load; its loads and stores alone take 220: vector instructions (addresses, splits into
// parts, scores) take 68 % of the issue slots, the MFMAs are busy 43 %. Sixteen columns a wave
// and eight waves equal thirty-two and four there and are a tenth faster at T4096, where a
// chunk's latency counts. Float32 B8 T2047 H32 d64, padded: 82 us.
template <typename E, typename O, int DA, int DC>
__global__ __launch_bounds__(64 * pass_waves(DC), PassShape<E>::kHalf ? 4 : 2) void linear_outputs_kernel(LinearPasses all) {
  const LinearPass s = all.pass[blockIdx.y];
  using S = PassShape<E>;
  constexpr int C = S::kChunk, NW = pass_waves(DC), NT = 64 * NW;
  constexpr int P = S::kParts, PS = S::kScoreParts;
  constexpr int RT = C / 16;          // row tiles of a chunk
  constexpr int KT = DA / 16;         // state tiles of a wave
  constexpr int KB = (DA + 31) / 32;  // k-blocks along DA
  constexpr int PB = C / 32;          // k-blocks of positions
  constexpr bool kDirect = S::kHalf;
  struct Shared {
    Tile<C, DA, P> a, b[kDirect ? 2 : 1];
    Tile<C, DC, P> c;
    Scores<C, PS> scores;
    float weight[2][C];  // l^{n-1-j+shift}
    float decay[C + 1];  // powers of l
    float decay_lo;      // of l^C: what decay[C] leaves out
    int bad_from[DC];    // first position of the chunk whose c is not finite, a channel
  };
  static_assert(sizeof(Shared) == outputs_lds(S::kHalf, DA, DC), "choose_segments goes by outputs_lds");
  __shared__ Shared sh;
  Segment<E, DA, DC> me(s, s.nseg, false);
  const int wave = me.wave;
  const int begin = me.begin, end = me.end;
  float4v X[KT];
  if (s.nseg == 1)
    me.load_state(X, s.x0 == nullptr ? nullptr : s.x0 + me.bh * (DA * DC), s.x0_sa, s.x0_sc);
  else
    me.load_state(X, me.seg == 0 && s.x0 == nullptr ? nullptr : s.states + (me.bh * s.nseg + me.seg) * (DA * DC), s.st_sa, s.st_sc);

  std::conditional_t<kDirect, Direct<C, DA, NT>, Staged<C, DA, NT>> ra(s.lda, s.back), rb(s.ldb, s.back);
  std::conditional_t<kDirect, Direct<C, DC, NT>, Staged<C, DC, NT>> rc(s.ldc, s.back);
  auto fetch_a = [&](int p) {
    const E* from = me.rows(s.a, s.lda, s.group_a, DA, p);
    if constexpr (kDirect) ra.load(sh.a, from, me.size(p));
    else ra.load(from, me.size(p));
  };
  auto fetch_b = [&](int p, int buf) {
    const E* from = me.rows(s.b, s.ldb, s.group_b, DA, p);
    if constexpr (kDirect) rb.load(sh.b[buf], from, me.size(p));
    else rb.load(from, me.size(p));
  };
  auto fetch_c = [&](int p) {
    const E* from = me.rows(s.c, s.ldc, s.group_c, DC, p);
    if constexpr (kDirect) rc.load(sh.c, from, me.size(p));
    else rc.load(from, me.size(p));
  };
  // A lane's places in the tiles, and the offset of its part of an output row. Opaque in
  // every chunk, as what is formed from them would be held in registers otherwise.
  int at_row = Tile<C, DA, P>::row_place(me.i, me.g);
  int at_b = Tile<C, DA, P>::column_place(0, DA == 16 ? 4 : 8, me.i, me.g);
  int at_c = Tile<C, DC, P>::column_place(16 * wave, 4, me.i, me.g);
  int at_first = Tile<32, 32, PS>::row_place(me.i, me.g), at_second = Tile<32, 64, PS>::row_place(me.i, me.g);
  const uint32_t out_step = uint32_t(s.H) * DC * uint32_t(sizeof(O));  // at most 2^25: a chunk's offsets fit in 31 bits
  uint32_t at_out = (16 * wave + 4 * me.g) * uint32_t(sizeof(O)) + (s.back ? 0u - me.i * out_step : me.i * out_step);
  // Order of a chunk's loads and barriers. bf16: `a` and `b` are there at the start of a
  // chunk; `c` arrives while scores and a X are formed, the next `a` (its tile is read no
  // more) and `b` (the other buffer) while the chunk's own rows are summed: two workgroups
  // fit a CU. float32: the next chunk's rows wait in registers.
  if (begin < end) {
    fetch_a(begin);
    fetch_b(begin, 0);
    if constexpr (kDirect) wait_loads();
    else fetch_c(begin);
  }

  for (int at = threadIdx.x; at < C; at += NT) sh.decay[at] = me.power(at);
  if (threadIdx.x == 0) two_floats(head_log_decay(s.log_decay, me.h) * float(C), &sh.decay[C], &sh.decay_lo);
  float left = 0.0f;  // of the chunks' decays, not in the state yet: into it as soon as it is half a step of the next
  __syncthreads();
  int buf = 0;
  for (int p = begin; p < end; p += C, buf ^= 1) {
    const int m = me.size(p);
    const bool more = p + C < end;
    asm volatile("" : "+v"(me.lg), "+v"(me.i), "+v"(me.g), "+v"(at_row), "+v"(at_b), "+v"(at_c), "+v"(at_first), "+v"(at_second), "+v"(at_out));
    const int i = me.i, g = me.g;
    if constexpr (kDirect) {
      fetch_c(p);
    } else {
      ra.store(sh.a);
      rb.store(sh.b[0]);
      rc.store(sh.c);
    }
    if (threadIdx.x < C) {
      const int left = m - 1 - int(threadIdx.x);
      sh.weight[buf][threadIdx.x] = left >= 0 ? me.power(left + s.shift) : 0.0f;
    }
    if constexpr (!kDirect) {
      __syncthreads();
      if (more) fetch_a(p + C), fetch_b(p + C, 0), fetch_c(p + C);
    }
    Tile<C, DA, P>& tb = sh.b[kDirect ? buf : 0];

    // Scores, transposed: column i of tile (r, jt) is position 16 r + i, its rows are
    // positions 16 jt + 4 g + e. The tiles at and under the diagonal go round the waves,
    // then those right of it that a k-block of 32 positions reads as zeros.
    constexpr int kLower = RT * (RT + 1) / 2;
    for (int t = wave; t < kLower + RT / 2; t += NW) {
      int r = 0, jt = t;
      float x[4] = {};
      if (t < kLower) {
        while (jt > r) jt -= ++r;
        float4v d{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
          bhalf8 av[P], bv[P];
#pragma unroll
          for (int q = 0; q < P; ++q) av[q] = sh.a.row(q, r, kb, at_row), bv[q] = tb.row(q, jt, kb, at_row);
          mma_parts<1, P, P, P - 1>([&](int, int p) { return bv[p]; }, [&](int, int p) { return av[p]; }, &d);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int ahead = 16 * r + i - (16 * jt + 4 * g + e);
          x[e] = ahead >= 0 ? d[e] * sh.decay[ahead] : 0.0f;
        }
      } else {
        r = 2 * (t - kLower), jt = r + 1;
      }
      bhalf4 part[PS];
      split_parts<PS, 4>(x, part);
#pragma unroll
      for (int q = 0; q < PS; ++q) sh.scores.put4(q, 16 * r + i, 16 * jt + 4 * g, part[q]);
    }
    // What the state before the chunk gives. Wave priorities rise through a chunk, so that
    // the CU's two workgroups drift into different phases of theirs: 380 -> 366 us at B2
    // T32768 H16 d128 bf16, 138 -> 133 us for its gradients at T4096.
    __builtin_amdgcn_s_setprio(1);
    float4v acc[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) acc[r] = float4v{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      float x[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[e] = X[2 * kb][e];
        x[4 + e] = KT > 1 ? X[KT > 1 ? 2 * kb + 1 : 0][e] : 0.0f;
      }
      bhalf8 xv[PS];
      split_parts<PS, 8>(x, xv);
      bhalf8 av[RT][P];
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int q = 0; q < P; ++q) av[r][q] = sh.a.row(q, r, kb, at_row);
      mma_parts<RT, PS, P, PS - 1>([&](int, int p) { return xv[p]; }, [&](int t, int p) { return av[t][p]; }, acc);
    }
#pragma unroll
    for (int r = 0; r < RT; ++r) acc[r] *= sh.decay[16 * r + i + 1 - s.shift];
    if constexpr (kDirect) wait_loads();
    __syncthreads();
    if constexpr (kDirect) {
      if (more) fetch_a(p + C), fetch_b(p + C, buf ^ 1);
    }

    // what the chunk's own rows give, and the state after it
    __builtin_amdgcn_s_setprio(2);
    bool bad = false;
    left += sh.decay_lo;
    const float once = m == C ? sh.decay[C] : me.power(m), whole = once + left;
    left = __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(left - (whole - once))));
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) X[kt] *= whole;
#pragma unroll
    for (int kb = 0; kb < PB; ++kb) {
      bhalf8 cv[P];
      float x[8];
      weighted<E, DC>(sh.c, sh.weight[buf], kb, at_c, g, cv, x);
      // A masked score is 0, but 0 times Inf is not: such values leave the product, and the
      // rows from theirs on become NaN.
      if (__builtin_expect(__any(any_bad(cv[0])), 0)) {
        const int column = 16 * wave + i;
        if (!bad && g == 0) sh.bad_from[column] = C;
        bad = true;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (!is_bad(cv[0][e])) continue;
          atomicMin(&sh.bad_from[column], 32 * kb + 8 * g + e);
#pragma unroll
          for (int q = 0; q < P; ++q) cv[q][e] = __bf16(0.0f);
        }
      }
      // rows before the block see none of it
      auto own_rows = [&](auto from) {
        constexpr int R = decltype(from)::value;
        bhalf8 sv[RT - R][PS];
#pragma unroll
        for (int r = R; r < RT; ++r)
#pragma unroll
          for (int q = 0; q < PS; ++q) sv[r - R][q] = sh.scores.row(q, r, kb, at_first, at_second);
        mma_parts<RT - R, P, PS, PS - 1>([&](int, int p) { return cv[p]; }, [&](int t, int p) { return sv[t][p]; }, acc + R);
      };
      if (kb == 0) own_rows(std::integral_constant<int, 0>{});
      else own_rows(std::integral_constant<int, PB == 2 ? 2 : 0>{});
      add_outer<E, DA>(X, tb, kb, at_b, x);
    }

    if constexpr (kDirect) wait_loads();
    __builtin_amdgcn_s_setprio(0);
    // rows 16 r + i; stores behind the chunk's end fall out of the range
    const uint32_t top = uint32_t(m - 1) * out_step;
    O* to = static_cast<O*>(s.out) + ((me.b * s.T + int64_t(s.back ? me.n - p - m : p)) * s.H + me.h) * DC;
    const auto range = __builtin_amdgcn_make_buffer_rsrc(to, 0, top + DC * uint32_t(sizeof(O)), 0x00020000);
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      float x4[4] = {acc[r][0], acc[r][1], acc[r][2], acc[r][3]};
      if (__builtin_expect(bad, 0)) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (16 * r + i >= sh.bad_from[16 * wave + 4 * g + e]) x4[e] = __builtin_nanf("");
      }
      vec<O, 4> o;
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = O(x4[e]);
      const uint32_t at = at_out + (s.back ? top - 16u * r * out_step : 16u * r * out_step);
      if constexpr (sizeof(O) == 2) __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(vec<uint32_t, 2>, o), range, at, 0, 0);
      else __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(vec<uint32_t, 4>, o), range, at, 0, 0);
    }
    __syncthreads();
  }

  if (s.zero_tail) {
    const int first = begin > me.n ? begin : me.n;
    constexpr int V = DC / 4;
    for (int64_t at = threadIdx.x; at < int64_t(me.last - first) * V; at += NT) {
      const float zero[4] = {};
      store4(static_cast<O*>(s.out) + ((me.b * s.T + first + at / V) * s.H + me.h) * DC + at % V * 4, zero);
    }
  }
  if (me.seg == s.nseg - 1)
    me.store_state(X, s.x1 == nullptr ? nullptr : s.x1 + me.bh * (DA * DC), s.x0_sa, s.x0_sc);
}

// Launches of `count` passes of B sequences of either type, in their own translation units:
// the segments' states, or the outputs (float32 where wide_out).
int launch_pass_bf16(const LinearPasses& s, int count, int64_t B, int da, int dc, bool out, bool wide_out, void* stream);
int launch_pass_f32(const LinearPasses& s, int count, int64_t B, int da, int dc, bool out, void* stream);

template <typename E, typename O, int DA, int DC>
int launch_pass_dims(const LinearPasses& s, int count, int64_t B, bool out, hipStream_t stream) {
  constexpr int kThreads = 64 * pass_waves(DC);
  const LinearPass& p = s.pass[0];
  const dim3 grid(unsigned(B * p.H * (out ? p.nseg : p.nseg - 1)), unsigned(count));
  if (out) linear_outputs_kernel<E, O, DA, DC><<<grid, kThreads, 0, stream>>>(s);
  else linear_states_kernel<E, DA, DC><<<grid, kThreads, 0, stream>>>(s);
  return int(hipGetLastError());
}

template <typename E, typename O>
int launch_pass_any(const LinearPasses& s, int count, int64_t B, int da, int dc, bool out, hipStream_t stream) {
  switch (da * 1000 + dc) {
#define GDN_PASS(DA, DC) case DA * 1000 + DC: return launch_pass_dims<E, O, DA, DC>(s, count, B, out, stream);
    GDN_PASS(16, 16) GDN_PASS(16, 32) GDN_PASS(16, 64) GDN_PASS(16, 128)
    GDN_PASS(32, 16) GDN_PASS(32, 32) GDN_PASS(32, 64) GDN_PASS(32, 128)
    GDN_PASS(64, 16) GDN_PASS(64, 32) GDN_PASS(64, 64) GDN_PASS(64, 128)
    GDN_PASS(128, 16) GDN_PASS(128, 32) GDN_PASS(128, 64) GDN_PASS(128, 128)
#undef GDN_PASS
    default: return int(hipErrorInvalidValue);
  }
}

}  // namespace gdn
