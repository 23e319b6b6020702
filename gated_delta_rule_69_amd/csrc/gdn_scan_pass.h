// The gated recurrence a channel, h_t = a_t h_{t-1} + b_t, over long sequences: kernels and
// their launches for one element type.
//
// Eight or 32 lanes of a wave lie across the channels of a slice, four bytes a lane and row, and groups
// of such lanes hold a run of eight consecutive tokens each. A lane joins the tokens of its run, the
// groups join theirs by DPP, the waves of a workgroup theirs through LDS, in a row of sixteen lanes
// for each channel, and the workgroup walks the tiles of its segment with the state it carries.
// Joining two runs of tokens is (A, h) (A', h') -> (A A', A' h + h'): no division, so a decay may be
// 0.
//
// SIGMOID and POWER, whose a is at most 1: what a run leaves of the state before it is held
// twice, as the product A and as 1 - A, summed from the 1 - a of its tokens. Where less than half
// goes, the state loses (1 - A) h instead of being multiplied by a rounded A near 1, whose error a
// channel that keeps many tokens would add up at every step; and the state a workgroup carries
// is a sum of two floats, for the same reason.
//
// LOG, whose a may exceed 1: 1 - A of a run that grew is a large number, in which what a later run
// takes away is lost to rounding, and A itself may leave float32's range where the state does not
// (a thousand tokens that grow an empty state). So what a run leaves is held as log2 A, from the sum of
// its f, in two floats, and 1 - A is formed from that where a state is passed on.
//
// Where slices and sequences do not fill the CUs, segments of a sequence run side by side: a first
// launch finds what each makes of the state before it, walking it from its end until nothing before
// can be left in float32 (a thousand tokens and more under forget gates of logits around 3; twice as
// many under LOG, where the tokens before may have grown the state), and the second joins those before
// its own.
//
// Memory bounds it, as long as a CU's loads under way are long ones: the launch that writes h of B2 T32768
// C2048 (bf16, sigmoid; 805 MB) takes 314 us with rows of 32 bytes a slice (and no segments), 202 with 64
// and 173 with 128. Both launches 206 us (3.9 TB/s; 177 with C 2112, whose rows do not start at the same 4
// KiB). What the first launch may leave out goes by the gates: of those 28 us under sigmoid gates of
// logits around 3, 46 under the same decays by LOG, 140 under power gates whose channels keep thousands of
// tokens (300 in all, 389 with an input gate). One launch does for B8 T1024 C8192 with power and input gate
// (143 us, 537 MB); B1 T4096 C2048 takes 25 to 36 us, two short launches. The gradients of B2 T4096 C2048 with
// power and input gate 77 us (235 MB, 3.0 TB/s): 250 registers, two waves a SIMD, whose eighty vector
// instructions a channel and token take 45 % of the issue slots.
#pragma once

#include <algorithm>

#include "gdn_block.h"
#include "gdn_block_device.h"

namespace gdn {
namespace scan {

constexpr int kSpan = GDN_SCAN_SPAN;   // tokens between checkpoints
constexpr int kRun = 8;                // tokens a lane joins by itself
constexpr int kWaves = 16;             // waves a workgroup, each with tokens of its own: a tile
constexpr int kBackWaves = 8;          // the same in the gradients, which take twice the registers

// How a wave lies over rows and channels: LANES lanes across a slice, four bytes each, and groups of
// lanes with a run of consecutive tokens each.
template <int LANES> struct Geo {
  static constexpr int kRuns = 64 / LANES;
  static constexpr int kTokens = kRuns * kRun;   // of a wave
  static constexpr int kRow = 4 * LANES;         // bytes of a slice's row
  static constexpr int kApart = 16 / kRuns;      // lanes from group to group
  template <typename E> static constexpr int kChannels = kRow / int(sizeof(E));
};
// The forward pass reads whole lines of 128 bytes, where a CU's loads under way hold the most; the
// gradients' waves have a checkpoint's span, whose states before each token they form alone.
constexpr int kLanes = 32, kBackLanes = 8;
constexpr int kTile = kWaves * Geo<kLanes>::kTokens, kBackTile = kBackWaves * Geo<kBackLanes>::kTokens;
static_assert(Geo<kBackLanes>::kTokens == kSpan, "a checkpoint is the state before a wave's tokens");

// 1 - e^y for |y| < 1/4: the series' next term, y^8 / 9!, is 2^-34 of the first.
__device__ __forceinline__ float less_exp(float y) {
  const float p = 1.0f / 24 + y * (1.0f / 120 + y * (1.0f / 720 + y * (1.0f / 5040 + y * (1.0f / 40320))));
  return -y * (1.0f + y * (0.5f + y * (1.0f / 6 + y * p)));
}

// e^y and 1 - e^y for y <= 0 (and what they are above), the second to a few steps of its own: a series
// where the difference would cancel. For bf16 y comes times log2 e, which takes one instruction for 2^y;
// for float32 as it is.
template <typename E>
__device__ __forceinline__ void exp_both(float y, float* a, float* c) {
  float p;
  bool near;
  if constexpr (sizeof(E) == 2) {   // z = y ln 2, |z| < 1/4: z^5 / 720 is 2^-19 of z
    constexpr float L = 0.69314718056f;
    *a = __builtin_amdgcn_exp2f(y);
    p = -L + y * (-L * L / 2 + y * (-L * L * L / 6 + y * (-L * L * L * L / 24 + y * (-L * L * L * L * L / 120))));
    p *= y;
    near = fabsf(y) < 0.36f;
  } else {
    *a = expf(y);
    p = less_exp(y);
    near = fabsf(y) < 0.25f;
  }
  // both sides in every lane: a branch for the series costs more than it
  asm volatile("" : "+v"(p));
  *c = near ? p : 1.0f - *a;
}

// A token's factors: h = a h + m g x with c = 1 - a (LOG, but for STEP: c = ln a, finite). s and rest
// (sigmoid(f) and its complement) are the gradients'.
struct Gate {
  float a, c, m, s, rest;
};
// What gate_of takes for a channel's decay.
template <typename E>
__device__ __forceinline__ float scaled_decay(float decay) {
  return sizeof(E) == 2 ? -1.44269504089f * decay : -decay;
}
template <typename E, int KIND, bool STEP = false>
__device__ __forceinline__ Gate gate_of(float f, float decay) {
  Gate g;
  if constexpr (KIND == GDN_SCAN_LOG) {
    if constexpr (STEP) {
      exp_both<E>(sizeof(E) == 2 ? 1.44269504089f * f : f, &g.a, &g.c);
    } else {
      g.a = exp_of<E>(f);
      // sums of two floats know no infinity; 1e28 a token is one to any state, and 2^31 of them add up
      g.c = __builtin_amdgcn_fmed3f(f, -1e28f, 1e28f);
    }
    g.m = 1.0f;
    g.s = g.rest = 0.0f;
  } else {
    sigmoids<E>(f, &g.s, &g.rest);
    if constexpr (KIND == GDN_SCAN_SIGMOID) {
      g.a = g.s;
      g.c = g.m = g.rest;
    } else {
      exp_both<E>(decay * g.s, &g.a, &g.c);
      // 1 - a^2 = c (1 + a)
      const float m2 = fmaf(g.c, g.a, g.c);
      g.m = sizeof(E) == 2 ? __builtin_amdgcn_sqrtf(m2) : sqrtf(m2);
    }
  }
  return g;
}

// A run of tokens: what is left of the state before it (A, and C = 1 - A; LOG: the two floats whose
// sum is log2 A), and what it adds.
struct Run {
  float A, C, H;
};

// x 2^(hi + lo): 2 to the whole part by the exponent, rounded up so that the rest of it makes no x
// larger: nothing on the way leaves float32's range unless the result does. Beyond 2^1000 that is 0 or
// infinite for every x.
__device__ __forceinline__ float times_exp2(float x, float hi, float lo) {
  const float n = ceilf(__builtin_amdgcn_fmed3f(hi, -1000.0f, 1000.0f));
  const float r = __builtin_amdgcn_fmed3f((hi - n) + lo, -2.0f, 2.0f);
  return ldexpf(x * __builtin_amdgcn_exp2f(r), int(n));
}

template <bool LOG> struct Runs;

template <> struct Runs<false> {
  static __device__ __forceinline__ Run empty() { return {1.0f, 0.0f, 0.0f}; }
  static __device__ __forceinline__ Run join(const Run& first, const Run& then) {
    return {first.A * then.A, fmaf(then.C, first.A, first.C), fmaf(then.A, first.H, then.H)};
  }
  template <typename E>
  static __device__ __forceinline__ Run token(const Run& first, float a, float c, float add) { return join(first, {a, c, add}); }
  static __device__ __forceinline__ Run close(const Run& r) { return r; }
  // The product of rounded A's is off by a step for each of them, 1 - C by one: where a run leaves more
  // than half, that is its A.
  static __device__ __forceinline__ Run settle(const Run& r) { return {r.C < 0.5f ? 1.0f - r.C : r.A, r.C, r.H}; }
  static __device__ __forceinline__ Run join_settled(const Run& first, const Run& then) { return settle(join(first, then)); }
  // The state x behind the run.
  static __device__ __forceinline__ float after(const Run& r, float x) { return fmaf(r.A, x, r.H); }
  // Nothing of what lies before can be left.
  static __device__ __forceinline__ bool gone(const Run& r) { return r.A == 0.0f; }
};

template <> struct Runs<true> {
  static __device__ __forceinline__ Run empty() { return {0.0f, 0.0f, 0.0f}; }
  // The logarithms' sum, its rounding's rest with the lower parts.
  static __device__ __forceinline__ Run add(const Run& first, float hi, float lo, float H) {
    const float sum = first.A + hi, back = sum - first.A;
    return {sum, first.C + lo + ((first.A - (sum - back)) + (hi - back)), H};
  }
  static __device__ __forceinline__ Run join(const Run& first, const Run& then) {
    return add(first, then.A, then.C, times_exp2(first.H, then.A, then.C) + then.H);
  }
  // A lane's own tokens, one by one: A is the sum of f. Eight numbers of eight bits add up without a
  // rounding as long as they are within 2^13 of each other.
  template <typename E>
  static __device__ __forceinline__ Run token(const Run& first, float a, float f, float more) {
    const float H = fmaf(a, first.H, more);
    if constexpr (sizeof(E) == 2) return {first.A + f, 0.0f, H};
    return add(first, f, 0.0f, H);
  }
  // From the sum of f to log2 A.
  static __device__ __forceinline__ Run close(const Run& r) {
    constexpr float K = 1.44269504089f, REST = 1.92596299e-8f;   // log2 e, and what K is off by
    const float hi = K * r.A;
    return {hi, fmaf(K, r.C, fmaf(REST, r.A, fmaf(K, r.A, -hi))), r.H};
  }
  static __device__ __forceinline__ Run settle(const Run& r) { return r; }
  static __device__ __forceinline__ Run join_settled(const Run& first, const Run& then) { return join(first, then); }
  static __device__ __forceinline__ float after(const Run& r, float x) { return times_exp2(x, r.A, r.C) + r.H; }
  // The tokens before may have grown the state to the largest float, 2^128: of that less than half of
  // the smallest, 2^-149, is left. (B2 T32768 C2048 bf16, f around -0.05: 46 us for the first launch, 29 if
  // it stopped at a product of 2^-149, which states that had grown before would miss.)
  static __device__ __forceinline__ bool gone(const Run& r) { return r.A <= -279.0f; }
};

// A state held as hi + lo.
template <bool LOG> struct State {
  float hi, lo;
  __device__ __forceinline__ void pass(const Run& r) {
    bool slow;
    float base, add, low;
    if constexpr (LOG) {
      const float y = 0.69314718056f * r.A, c = fabsf(y) < 0.25f ? less_exp(y) : 1.0f - __builtin_amdgcn_exp2f(r.A);
      slow = fabsf(c) < 0.5f;
      base = slow ? hi : times_exp2(hi, r.A, r.C);
      add = slow ? fmaf(-c, hi, r.H) : r.H;
      low = times_exp2(lo, r.A, r.C);
    } else {
      slow = r.C < 0.5f;
      base = slow ? hi : r.A * hi;
      add = slow ? fmaf(-r.C, hi, r.H) : r.H;
      low = lo * r.A;
    }
    const float sum = base + add, back = sum - base;
    lo = low + ((base - (sum - back)) + (add - back));
    hi = sum;
  }
  // hi + lo where lo is a rounding's rest, hi where that is none (infinities)
  __device__ __forceinline__ float value() const {
    const float v = hi + lo;
    return v == v ? v : hi;
  }
};

struct Pass {
  const void *x, *f, *i;
  const float* decay;
  const int32_t* lens;
  const float* h0;
  float *h_final, *marks;
  void* h;
  int64_t ldx, ldf, ldi, T, C;
  int64_t seg;          // tokens a segment, a multiple of a tile
  unsigned slices, segs, blocks;
  float* start;         // [B][C]: h0, where segments run side by side
  Run* totals;          // [B][segs - 1][C]
  // gradients
  const void* d_h;
  const float* d_final;
  void *dx, *df, *di;
  float *dh0, *ddecay;  // ddecay: [B * segs][C] partial sums
};

typedef uint32_t uint4v __attribute__((ext_vector_type(4)));

// A buffer of `rows` rows (at most `most`, up to 64) of `width` bytes from `base` on, `ld` bytes
// apart; none for rows <= 0. Loads behind its last row give zero, stores are dropped. Strides are at
// most 2^26 bytes, so that offsets fit in 32 bits.
__device__ __forceinline__ uint4v rows_from(const char* base, int64_t ld, int64_t rows, int most, uint32_t width) {
  auto uniform = [](uint32_t x) { return uint32_t(__builtin_amdgcn_readfirstlane(int(x))); };
  const uint64_t from = reinterpret_cast<uintptr_t>(base);
  const uint32_t bytes = rows > 0 ? uint32_t(rows < most ? rows - 1 : most - 1) * uint32_t(ld) + width : 0u;
  return {uniform(uint32_t(from)), uniform(uint32_t(from >> 32) & 0xffffu), uniform(bytes), 0x00020000u};
}

// Rows on their way from memory to LDS, ahead of their use: a wave's own, so that nothing but its own
// count of loads says when they are there. Lane l of a load brings sixteen bytes to the wave's place
// 16 l: the rows r of the runs lie side by side there, at 256 r + kRow run, so that a wave reads 256 bytes
// in a row (what the LDS counters show of bank conflicts is the exchange between waves). The
// loads are written as assembly, which has no registers to guard; the compiler's own counts only ever
// wait for more.
template <int LANES> struct Feed {
  static constexpr int kRuns = Geo<LANES>::kRuns;
  uint32_t off[4], ld[4];
  const char* base[4];
  // a lane's place in a span for sixteen bytes, and in its row
  static __device__ __forceinline__ uint32_t column(int lane) { return lane % (LANES / 4) * 16; }
  static __device__ __forceinline__ uint32_t place(int lane, int64_t ld) {
    const int p = lane / (LANES / 4);
    return uint32_t((p % kRuns) * kRun + p / kRuns) * uint32_t(ld) + column(lane);
  }
  __device__ __forceinline__ void open(int k, const void* p, int64_t ld_, int64_t first, int lane) {
    base[k] = static_cast<const char*>(p) + first, ld[k] = uint32_t(ld_), off[k] = place(lane, ld_);
  }
  __device__ __forceinline__ void load(int k, char* to, int64_t t0, int64_t left, uint32_t width) const {
    const uint4v range = rows_from(base[k] + t0 * int64_t(ld[k]), ld[k], left, Geo<LANES>::kTokens, width);
    const uint32_t lds = __builtin_amdgcn_readfirstlane(uint32_t(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) char*)(to))));
    asm volatile("s_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"{m0}"(lds), "v"(off[k]), "s"(range) : "memory");
    asm volatile("s_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"{m0}"(lds + 1024), "v"(off[k] + 4 * uint32_t(ld[k])), "s"(range) : "memory");
  }
};
// Four bytes a lane, one load.
__device__ __forceinline__ void load_words(char* to, const char* from, uint32_t bytes, int lane) {
  const uint4v range = rows_from(from, 0, bytes > 0 ? 1 : 0, 1, bytes);
  const uint32_t lds = __builtin_amdgcn_readfirstlane(uint32_t(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) char*)(to))));
  asm volatile("s_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds" ::"{m0}"(lds), "v"(lane * 4), "s"(range) : "memory");
}
// Waits until no more than N of the wave's loads and stores are under way, the latest ones.
template <int N>
__device__ __forceinline__ void wait_memory() {
  static_assert(N < 64, "the counter has six bits");
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

template <typename E>
__device__ __forceinline__ float part_of(uint32_t raw, int v) {
  if constexpr (sizeof(E) == 4) return __uint_as_float(raw);
  return v == 0 ? __uint_as_float(raw << 16) : __uint_as_float(raw & 0xffff0000u);
}

template <typename E>
__device__ __forceinline__ uint32_t packed(const float* x) {
  if constexpr (sizeof(E) == 4) {
    return __float_as_uint(x[0]);
  } else {
    const bhalf2 r = {E(x[0]), E(x[1])};
    return __builtin_bit_cast(uint32_t, r);
  }
}

// A lane's place among the rows r of a span in LDS, and its channels.
template <int LANES> struct Lane {
  static constexpr int kApart = Geo<LANES>::kApart;
  int run, slot;
  __device__ __forceinline__ Lane(int lane) : run(lane / kApart % Geo<LANES>::kRuns), slot(lane / 16 * kApart + lane % kApart) {}
  __device__ __forceinline__ uint32_t at(int r) const { return 256 * r + Geo<LANES>::kRow * run + 4 * slot; }
};

// A wave's rows by way of LDS, laid as they came, in two stores: channels behind the last and rows
// that are not there lie behind the buffer.
template <int LANES>
__device__ __forceinline__ void store_span(char* by, char* base, int64_t ld, int64_t left, uint32_t width, const Lane<LANES>& l, int lane,
                                           const uint32_t* x) {
#pragma unroll
  for (int r = 0; r < kRun; ++r) *reinterpret_cast<uint32_t*>(by + l.at(r)) = x[r];
  const auto to = __builtin_amdgcn_make_buffer_rsrc(base, 0, int(rows_from(base, ld, left, Geo<LANES>::kTokens, width)[2]), 0x00020000);
  const uint32_t at = Feed<LANES>::column(lane) < width ? Feed<LANES>::place(lane, ld) : 0x80000000u;
#pragma unroll
  for (int j = 0; j < 2; ++j)
    __builtin_amdgcn_raw_buffer_store_b128(*reinterpret_cast<const uint4v*>(by + 1024 * j + 16 * lane), to, at + j * 4 * uint32_t(ld), 0, 0);
}

// Where a workgroup stands: blocks that follow each other on one XCD (their index modulo 8) are
// neighbouring slices of one segment, which share lines where a slice has less than one (the gradients).
struct Place {
  int64_t b;
  unsigned seg, slice;
  __device__ Place(const Pass& p, unsigned segs) {
    const unsigned xcd = blockIdx.x % 8, k = blockIdx.x / 8, each = p.blocks / 8, rest = p.blocks % 8;
    const unsigned id = xcd * each + (xcd < rest ? xcd : rest) + k;
    slice = id % p.slices;
    const unsigned q = id / p.slices;
    seg = q % segs;
    b = q / segs;
  }
};

// Lanes n before (BACK: behind) in a row of sixteen; `none` where there is no such lane.
template <int N, bool BACK>
__device__ __forceinline__ float beside(float x, float none) {
  return __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(none), __float_as_int(x), (BACK ? 0x100 : 0x110) + N, 0xf, 0xf, false));
}
template <int N, bool BACK, bool LOG>
__device__ __forceinline__ Run beside(const Run& r) {
  return {beside<N, BACK>(r.A, Runs<LOG>::empty().A), beside<N, BACK>(r.C, 0.0f), beside<N, BACK>(r.H, 0.0f)};
}

// Joins over the lane groups: own becomes the runs up to and with the lane's (BACK: from the last one
// down to it), before those without it. Without C (AH; not LOG) A is the product.
template <int V, int LANES, bool BACK, bool AH, bool LOG>
__device__ __forceinline__ void join_lanes(Run* own, Run* before) {
#pragma unroll
  for (int v = 0; v < V; ++v) {
    auto take = [&](const Run& o) { own[v] = AH ? Runs<LOG>::join(o, own[v]) : Runs<LOG>::join_settled(o, own[v]); };
    if constexpr (Geo<LANES>::kRuns >= 8) take(beside<2, BACK, LOG>(own[v]));
    if constexpr (Geo<LANES>::kRuns >= 4) take(beside<4, BACK, LOG>(own[v]));
    take(beside<8, BACK, LOG>(own[v]));
    before[v] = beside<Geo<LANES>::kApart, BACK, LOG>(own[v]);
  }
}

// What the waves of a workgroup exchange: their spans' runs, a channel's side by side, and the state
// before each.
template <int N, int NW> struct Exchange {
  float4 runs[N][NW + 1];
  float before[NW][N];
};

// The channels that a wave carries the state of, N / NW of them: one a row of sixteen lanes, whose
// lanes are the waves (BACK: from the last).
template <int N, int NW, bool BACK, bool LOG> struct Keeper {
  static constexpr int kOwn = N < NW ? 1 : N / NW;
  static_assert(kOwn <= 4, "a wave has four rows");
  int ch, from;   // the row's channel in the slice, and the wave whose run the lane takes
  bool on, there, first;
  State<LOG> carry = {0.0f, 0.0f};
  __device__ __forceinline__ Keeper(int wave, int lane, int channels) {
    ch = wave * kOwn + lane / 16;
    from = BACK ? NW - 1 - lane % 16 : lane % 16;
    on = lane / 16 < kOwn && ch < N;
    there = on && ch < channels;
    first = there && lane % 16 == 0;
  }
  // Joins the runs of a row's lanes: up to and with the lane's, and of all.
  static __device__ __forceinline__ Run join_row(Run r, int lane, Run* whole) {
    r = Runs<LOG>::join_settled(beside<1, false, LOG>(r), r);
    r = Runs<LOG>::join_settled(beside<2, false, LOG>(r), r);
    r = Runs<LOG>::join_settled(beside<4, false, LOG>(r), r);
    r = Runs<LOG>::join_settled(beside<8, false, LOG>(r), r);
    const int end = lane | 15;
    *whole = {__shfl(r.A, end), __shfl(r.C, end), __shfl(r.H, end)};
    return r;
  }
  // The runs of a tile's waves.
  __device__ __forceinline__ Run tile(const Exchange<N, NW>& x, int lane, Run* whole) const {
    Run r = Runs<LOG>::empty();
    if (lane % 16 < NW) {
      const float4 q = x.runs[ch][from];
      r = {q.x, q.y, q.z};
    }
    return join_row(r, lane, whole);
  }
  // Passes the carried state over `count` segments, of(k) the k-th to be passed: sixteen of them at a
  // time, a lane each, for one after the other each would wait for its load.
  template <typename F>
  __device__ __forceinline__ void over(int64_t count, int lane, F of) {
    if (!on) return;
    for (int64_t k = 0; k < count; k += 16) {
      Run r = Runs<LOG>::empty(), whole;
      if (k + lane % 16 < count && there) r = of(k + lane % 16);
      join_row(r, lane, &whole);
      carry.pass(whole);
    }
  }
  // Passes the carried state over a tile; gives each wave its own.
  __device__ __forceinline__ void pass(Exchange<N, NW>& x, int lane) {
    if (!on) return;
    Run whole;
    const Run r = tile(x, lane, &whole);
    State<LOG> s = carry;
    s.pass(beside<1, false, LOG>(r));
    if (lane % 16 < NW) x.before[from][ch] = s.value();
    carry.pass(whole);
  }
  // Joins a tile before those of `total`; whether nothing of what lies before can be left.
  __device__ __forceinline__ bool extend(const Exchange<N, NW>& x, int lane, Run* total) const {
    if (!on) return true;
    Run whole;
    tile(x, lane, &whole);
    *total = Runs<LOG>::join_settled(whole, *total);
    return Runs<LOG>::gone(*total) || !there;
  }
};

// Forward. TOTALS: only what each segment but the last makes of the state before it, from its end
// backwards, as far as rows have a weight that float32 holds.
template <typename E, int KIND, bool IG, bool TOTALS>
__global__ __launch_bounds__(64 * kWaves) void scan_kernel(Pass p) {
  constexpr int V = 4 / int(sizeof(E)), N = Geo<kLanes>::kChannels<E>, NT = IG ? 3 : 2, kTokens = Geo<kLanes>::kTokens;
  constexpr bool LOG = KIND == GDN_SCAN_LOG;
  __shared__ __attribute__((aligned(16))) char raw[kWaves][NT][64 * 4 * kRun];
  __shared__ __attribute__((aligned(16))) char out[kWaves][TOTALS ? 16 : 64 * 4 * kRun];
  __shared__ Exchange<N, kWaves> exchange;
  const Place at(p, TOTALS ? p.segs - 1 : p.segs);
  const int lane = threadIdx.x % 64;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const Lane<kLanes> l(lane);
  const int64_t c0 = int64_t(at.slice) * N, cb = at.b * p.C + c0;
  const uint32_t channels = p.C - c0 < N ? uint32_t(p.C - c0) : N, width = channels * sizeof(E);   // a slice may end behind C
  Keeper<N, kWaves, false, LOG> keeper(wave, lane, channels);
  const int64_t n = tokens_of(p.lens, at.b, p.T);
  const int64_t begin = at.seg * p.seg;
  if (begin >= n && at.seg > 0) return;
  const bool last = n - begin <= p.seg;
  if (TOTALS && at.seg == 0 && keeper.first) p.start[cb + keeper.ch] = p.h0 != nullptr ? p.h0[cb + keeper.ch] : 0.0f;
  if (TOTALS && last) return;
  const int64_t end = last ? n : begin + p.seg;
  Feed<kLanes> feed;
  feed.open(0, p.x, p.ldx, at.b * p.T * p.ldx + c0 * int64_t(sizeof(E)), lane);
  feed.open(1, p.f, p.ldf, at.b * p.T * p.ldf + c0 * int64_t(sizeof(E)), lane);
  if constexpr (IG) feed.open(2, p.i, p.ldi, at.b * p.T * p.ldi + c0 * int64_t(sizeof(E)), lane);
  auto fetch = [&](int64_t t0) {
    const int64_t left = t0 < begin ? 0 : end - t0;
#pragma unroll
    for (int k = 0; k < NT; ++k) feed.load(k, raw[wave][k], t0, left, width);
  };
  const int64_t tiles = (end - begin + kTile - 1) / kTile, step = TOTALS ? -kTile : kTile;
  const int64_t first = begin + wave * kTokens + (TOTALS ? (tiles - 1) * kTile : 0);
  fetch(first);
  const int64_t ldh = p.C * sizeof(E);
  char* h = static_cast<char*>(p.h) + at.b * p.T * ldh + c0 * int64_t(sizeof(E));
  Run total = Runs<LOG>::empty();
  if constexpr (!TOTALS) {
    const float* from = p.segs > 1 ? p.start : p.h0;
    if (from != nullptr && keeper.there) keeper.carry.hi = from[cb + keeper.ch];
    keeper.over(at.seg, lane, [&](int64_t k) { return p.totals[(at.b * (p.segs - 1) + k) * p.C + c0 + keeper.ch]; });
  }
  float decay[V];
#pragma unroll
  for (int v = 0; v < V; ++v)
    decay[v] = KIND == GDN_SCAN_POWER && uint32_t(l.slot * V) < channels ? scaled_decay<E>(p.decay[c0 + l.slot * V + v]) : 0.0f;
  // a tile whose rows are all there, or the last
  auto walk = [&](auto full, int64_t k) {
    constexpr bool FULL = decltype(full)::value;
    const int64_t t0 = first + k * step, left = end - t0;
    if (!TOTALS && p.h != nullptr && k > 0) wait_memory<2>();   // the stores behind its loads
    else wait_memory<0>();
    uint32_t in[NT][kRun];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int r = 0; r < kRun; ++r) in[t][r] = *reinterpret_cast<const uint32_t*>(raw[wave][t] + l.at(r));
    }
    wait_lds();
    fetch(t0 + step);
    float a[kRun][V], b[kRun][V];
    Run own[V], before[V];
#pragma unroll
    for (int v = 0; v < V; ++v) own[v] = Runs<LOG>::empty();
#pragma unroll
    for (int r = 0; r < kRun; ++r) {
      const bool here = FULL || l.run * kRun + r < left;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const Gate t = gate_of<E, KIND>(part_of<E>(in[1][r], v), decay[v]);
        a[r][v] = here ? t.a : 1.0f;
        b[r][v] = KIND == GDN_SCAN_LOG ? part_of<E>(in[0][r], v) : t.m * part_of<E>(in[0][r], v);
        if constexpr (IG) b[r][v] *= sigmoid_of<E>(part_of<E>(in[2][r], v));
        if (!here) b[r][v] = 0.0f;
        own[v] = Runs<LOG>::template token<E>(own[v], a[r][v], here ? t.c : 0.0f, b[r][v]);
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) own[v] = Runs<LOG>::settle(Runs<LOG>::close(own[v]));
    join_lanes<V, kLanes, false, false, LOG>(own, before);
    if (l.run == Geo<kLanes>::kRuns - 1) {
#pragma unroll
      for (int v = 0; v < V; ++v) exchange.runs[l.slot * V + v][wave] = make_float4(own[v].A, own[v].C, own[v].H, 0.0f);
    }
    __syncthreads();
    if constexpr (TOTALS) {
      return __syncthreads_and(keeper.extend(exchange, lane, &total)) != 0;
    } else {
      keeper.pass(exchange, lane);
      __syncthreads();
      float y[V];
#pragma unroll
      for (int v = 0; v < V; ++v) y[v] = Runs<LOG>::after(before[v], exchange.before[wave][l.slot * V + v]);
      if (p.marks != nullptr && l.run == 0 && uint32_t(l.slot * V) < channels && left > 0 && t0 % kSpan == 0) {
        float* m = p.marks + (at.b * ((p.T + kSpan - 1) / kSpan) + t0 / kSpan) * p.C + c0 + l.slot * V;
#pragma unroll
        for (int v = 0; v < V; ++v) m[v] = y[v];
      }
      if (p.h != nullptr) {
        uint32_t rows[kRun];
#pragma unroll
        for (int r = 0; r < kRun; ++r) {
#pragma unroll
          for (int v = 0; v < V; ++v) y[v] = fmaf(a[r][v], y[v], b[r][v]);
          rows[r] = packed<E>(y);
        }
        store_span(out[wave], h + t0 * ldh, ldh, left, width, l, lane, rows);
      }
      return false;
    }
  };
  int64_t k = 0;
  for (; (k + 1) * kTile <= end - begin; ++k)
    if (walk(std::true_type{}, k)) break;
  if (!TOTALS && k < tiles) walk(std::false_type{}, k);
  wait_memory<0>();   // of LDS that the next workgroup may get
  if (!keeper.first) return;
  if constexpr (TOTALS)
    p.totals[(at.b * (p.segs - 1) + at.seg) * p.C + c0 + keeper.ch] = total;
  else if (last && p.h_final != nullptr)
    p.h_final[cb + keeper.ch] = keeper.carry.value();
}

// Gradients, from a sequence's end: with G_t = a_t (d_h_t + G_{t+1}) the same recurrence, whose
// value behind token t is l_t = d_h_t + G_{t+1}. h comes from the state before the span. TOTALS:
// only what each segment but the first makes of the gradient behind it, from its start on.
template <typename E, int KIND, bool IG, bool TOTALS>
__global__ __launch_bounds__(64 * kBackWaves) void scan_bwd_kernel(Pass p) {
  constexpr int V = 4 / int(sizeof(E)), N = Geo<kBackLanes>::kChannels<E>, R = kRun, kRuns = Geo<kBackLanes>::kRuns;
  constexpr int NT = TOTALS ? 2 : IG ? 4 : 3, kLoads = 2 * NT + (TOTALS ? 0 : 1), kStores = TOTALS ? 0 : IG ? 6 : 4;
  constexpr bool LOG = KIND == GDN_SCAN_LOG;
  __shared__ __attribute__((aligned(16))) char raw[2][kBackWaves][NT][64 * 4 * kRun];
  __shared__ __attribute__((aligned(16))) char raw_marks[2][kBackWaves][TOTALS ? 16 : 256];
  __shared__ __attribute__((aligned(16))) char out[kBackWaves][TOTALS ? 16 : 64 * 4 * kRun];
  __shared__ Exchange<N, kBackWaves> exchange;
  Place at(p, TOTALS ? p.segs - 1 : p.segs);
  if (TOTALS) ++at.seg;
  const int lane = threadIdx.x % 64;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const Lane<kBackLanes> l(lane);
  const int64_t c0 = int64_t(at.slice) * N, cb = at.b * p.C + c0;
  const uint32_t channels = p.C - c0 < N ? uint32_t(p.C - c0) : N, width = channels * sizeof(E);
  const bool own_lane = uint32_t(l.slot * V) < channels;
  Keeper<N, kBackWaves, true, LOG> keeper(wave, lane, channels);
  const int64_t n = tokens_of(p.lens, at.b, p.T);
  const int64_t begin = at.seg * p.seg;
  const int64_t stop = std::min(begin + p.seg, p.T), end = std::min(stop, n);
  const int64_t ldh = p.C * sizeof(E), row0 = at.b * p.T * ldh + c0 * int64_t(sizeof(E));
  char* dx = static_cast<char*>(p.dx) + row0;
  char* df = static_cast<char*>(p.df) + row0;
  char* di = static_cast<char*>(p.di) + row0;
  if constexpr (!TOTALS) {
    // rows behind the length: zero
    for (int64_t t = std::max(begin, n) + wave * kRuns + l.run; own_lane && t < stop; t += kBackWaves * kRuns) {
      const int64_t to = t * ldh + 4 * l.slot;
      *reinterpret_cast<uint32_t*>(dx + to) = 0, *reinterpret_cast<uint32_t*>(df + to) = 0;
      if constexpr (IG) *reinterpret_cast<uint32_t*>(di + to) = 0;
    }
  }
  if (TOTALS && begin >= n) return;
  Feed<kBackLanes> feed;
  feed.open(0, p.f, p.ldf, at.b * p.T * p.ldf + c0 * int64_t(sizeof(E)), lane);
  feed.open(1, p.d_h, ldh, row0, lane);
  if constexpr (!TOTALS) feed.open(2, p.x, p.ldx, at.b * p.T * p.ldx + c0 * int64_t(sizeof(E)), lane);
  if constexpr (!TOTALS && IG) feed.open(3, p.i, p.ldi, at.b * p.T * p.ldi + c0 * int64_t(sizeof(E)), lane);
  const int64_t spans = (p.T + kSpan - 1) / kSpan;
  auto fetch = [&](int stage, int64_t t0) {
    const int64_t left = t0 < begin ? 0 : end - t0;
#pragma unroll
    for (int k = 0; k < NT; ++k) feed.load(k, raw[stage][wave][k], t0, left, width);
    if constexpr (!TOTALS) {
      const float* m = p.marks + (at.b * spans + t0 / kSpan) * p.C + c0;
      load_words(raw_marks[stage][wave], reinterpret_cast<const char*>(m), left > 0 ? 4 * channels : 0, lane);
    }
  };
  const int64_t tiles = end > begin ? (end - begin + kBackTile - 1) / kBackTile : 0;
  const int64_t step = TOTALS ? kBackTile : -kBackTile;
  const int64_t first = begin + wave * kSpan + (TOTALS ? 0 : (tiles - 1) * kBackTile);
  if (tiles > 0) {
    fetch(0, first);
    fetch(1, first + step);
  }
  float raw_decay[V], decay[V], sum[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    raw_decay[v] = KIND == GDN_SCAN_POWER && own_lane ? p.decay[c0 + l.slot * V + v] : 0.0f;
    decay[v] = scaled_decay<E>(raw_decay[v]), sum[v] = 0.0f;
  }
  Run total = Runs<LOG>::empty();
  if constexpr (!TOTALS) {
    if (p.d_final != nullptr && keeper.there) keeper.carry.hi = p.d_final[cb + keeper.ch];
    const int64_t last = (n + p.seg - 1) / p.seg - 1;   // the last segment with tokens
    keeper.over(last - at.seg, lane, [&](int64_t k) { return p.totals[(at.b * (p.segs - 1) + last - k - 1) * p.C + c0 + keeper.ch]; });
  }
  auto walk = [&](auto full, int64_t k) {
    constexpr bool FULL = decltype(full)::value;
    const int stage = k & 1;
    const int64_t t0 = first + k * step, left = end - t0;
    // Behind the tile's loads came those of the next one and the stores of the two before it. What may be
    // out of range in part (the next tile's loads at an end, the first tile's stores) is not counted on.
    const int64_t next = t0 + step;
    const bool ahead = next >= begin && end - next >= kSpan;
    if (!ahead) wait_memory<0>();
    else if (TOTALS || k <= 1) wait_memory<kLoads>();
    else if (k == 2) wait_memory<kLoads + kStores>();
    else wait_memory<kLoads + 2 * kStores>();
    uint32_t in[NT][R];
    float mark[V];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int r = 0; r < R; ++r) in[t][r] = *reinterpret_cast<const uint32_t*>(raw[stage][wave][t] + l.at(r));
    }
    if constexpr (!TOTALS) {
#pragma unroll
      for (int v = 0; v < V; ++v) mark[v] = reinterpret_cast<const float*>(raw_marks[stage][wave])[l.slot * V + v];
    }
    wait_lds();
    fetch(stage, t0 + 2 * step);
    Gate gate[R][V];
    float si[R][V], resti[R][V], before[R][V];
    Run own[V], lanes[V];
#pragma unroll
    for (int v = 0; v < V; ++v) own[v] = Runs<LOG>::empty();
    // G of the run, from its last token
#pragma unroll
    for (int r = R - 1; r >= 0; --r) {
      const bool here = FULL || l.run * R + r < left;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        Gate& t = gate[r][v];
        t = gate_of<E, KIND>(part_of<E>(in[0][r], v), decay[v]);
        if (!here) t.a = 1.0f;
        const float up = part_of<E>(in[1][r], v);
        own[v] = Runs<LOG>::template token<E>(own[v], t.a, here ? t.c : 0.0f, here ? t.a * up : 0.0f);
        if constexpr (!TOTALS) {
          before[r][v] = KIND == GDN_SCAN_LOG ? part_of<E>(in[2][r], v) : t.m * part_of<E>(in[2][r], v);
          if constexpr (IG) {
            sigmoids<E>(part_of<E>(in[3][r], v), &si[r][v], &resti[r][v]);
            before[r][v] *= si[r][v];
          }
          if (!here) before[r][v] = 0.0f;
        }
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) own[v] = Runs<LOG>::close(own[v]);
    if constexpr (!TOTALS) {
      // h before each token: from what each adds
      Run fwd[V], earlier[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        fwd[v] = {own[v].A, LOG ? own[v].C : 0.0f, 0.0f};
#pragma unroll
        for (int r = 0; r < R; ++r) fwd[v].H = fmaf(gate[r][v].a, fwd[v].H, before[r][v]);
      }
      join_lanes<V, kBackLanes, false, true, LOG>(fwd, earlier);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float y = Runs<LOG>::after(earlier[v], mark[v]);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float add = before[r][v];
          before[r][v] = y;
          y = fmaf(gate[r][v].a, y, add);
        }
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) own[v] = Runs<LOG>::settle(own[v]);
    join_lanes<V, kBackLanes, true, false, LOG>(own, lanes);
    if (l.run == 0) {
#pragma unroll
      for (int v = 0; v < V; ++v) exchange.runs[l.slot * V + v][wave] = make_float4(own[v].A, own[v].C, own[v].H, 0.0f);
    }
    __syncthreads();
    if constexpr (TOTALS) {
      return __syncthreads_and(keeper.extend(exchange, lane, &total)) != 0;
    } else {
      keeper.pass(exchange, lane);
      __syncthreads();
      float G[V];
#pragma unroll
      for (int v = 0; v < V; ++v) G[v] = Runs<LOG>::after(lanes[v], exchange.before[wave][l.slot * V + v]);
#pragma unroll
      for (int r = R - 1; r >= 0; --r) {
        const bool here = FULL || l.run * R + r < left;
        float ox[V], of[V], oi[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const Gate& t = gate[r][v];
          const float xv = part_of<E>(in[2][r], v), g = part_of<E>(in[1][r], v) + G[v];
          const float gm = KIND == GDN_SCAN_LOG ? g : g * t.m;
          ox[v] = IG ? gm * si[r][v] : gm;
          if constexpr (IG) oi[v] = ox[v] * xv * resti[r][v];
          const float gx = IG ? si[r][v] * xv : xv;
          if constexpr (KIND == GDN_SCAN_LOG) {
            of[v] = g * before[r][v] * t.a;
          } else if constexpr (KIND == GDN_SCAN_SIGMOID) {
            of[v] = g * (before[r][v] - gx) * (t.a * t.c);
          } else {
            // d m / d a = -a / m
            const float slope = t.m > 0.0f ? t.a * gx * __builtin_amdgcn_rcpf(t.m) : 0.0f;
            const float dlog = g * t.a * (before[r][v] - slope) * t.s;
            of[v] = -raw_decay[v] * t.rest * dlog;
            sum[v] -= here ? dlog : 0.0f;
          }
          G[v] = here ? t.a * g : G[v];
        }
        in[2][r] = packed<E>(ox), in[0][r] = packed<E>(of);
        if constexpr (IG) in[3][r] = packed<E>(oi);
      }
      store_span(out[wave], dx + t0 * ldh, ldh, left, width, l, lane, in[2]);
      store_span(out[wave], df + t0 * ldh, ldh, left, width, l, lane, in[0]);
      if constexpr (IG) store_span(out[wave], di + t0 * ldh, ldh, left, width, l, lane, in[3]);
      return false;
    }
  };
  // the tile that may be in part behind the end is the last one of the segment
  const bool part = tiles > 0 && tiles * kBackTile > end - begin;
  int64_t k = 0;
  if (!TOTALS && part) walk(std::false_type{}, k++);
  bool gone = false;
  for (; k < tiles - (TOTALS && part) && !gone; ++k) gone = walk(std::true_type{}, k);
  if (TOTALS && part && !gone) walk(std::false_type{}, k);
  wait_memory<0>();
  if constexpr (TOTALS) {
    if (keeper.first) p.totals[(at.b * (p.segs - 1) + at.seg - 1) * p.C + c0 + keeper.ch] = total;
  } else {
    if (at.seg == 0 && p.dh0 != nullptr && keeper.first) p.dh0[cb + keeper.ch] = keeper.carry.value();
    if (KIND == GDN_SCAN_POWER && p.ddecay != nullptr) {
      // over the lane groups, then the waves
#pragma unroll
      for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int m = Geo<kBackLanes>::kApart; m < 16; m *= 2) sum[v] += __shfl_xor(sum[v], m);
      }
      __syncthreads();
      if (l.run == 0) {
#pragma unroll
        for (int v = 0; v < V; ++v) exchange.before[wave][l.slot * V + v] = sum[v];
      }
      __syncthreads();
      if (threadIdx.x < channels) {
        float t = 0.0f;
        for (int w = 0; w < kBackWaves; ++w) t += exchange.before[w][threadIdx.x];
        p.ddecay[(at.b * p.segs + at.seg) * p.C + c0 + threadIdx.x] = t;
      }
    }
  }
}

// Token by token, four channels a thread, for few tokens: each sequence's state is read and written
// once, and the rows of AT tokens are loaded together. Where less than half of a state goes, (1 - a) h
// is taken from it.
constexpr int kStepThreads = 256;
template <typename E, int KIND, bool IG, int AT>
__global__ __launch_bounds__(kStepThreads) void scan_step_kernel(Pass p) {
  typedef vec<E, 4> Row;
  const unsigned per = unsigned(p.C / 4);
  const unsigned id = blockIdx.x * kStepThreads + threadIdx.x;
  if (id >= p.blocks) return;   // (sequence, channels): B * C / 4 of them
  const int64_t b = id / per, c = int64_t(id % per) * 4;
  const int64_t n = tokens_of(p.lens, b, p.T);
  float h[4] = {}, decay[4] = {};
  if (p.h0 != nullptr) load4(p.h0 + b * p.C + c, h);
  if constexpr (KIND == GDN_SCAN_POWER) {
    load4(p.decay + c, decay);
#pragma unroll
    for (int v = 0; v < 4; ++v) decay[v] = scaled_decay<E>(decay[v]);
  }
  const char* x = static_cast<const char*>(p.x) + b * p.T * p.ldx + c * sizeof(E);
  const char* f = static_cast<const char*>(p.f) + b * p.T * p.ldf + c * sizeof(E);
  const char* g = static_cast<const char*>(p.i) + b * p.T * p.ldi + c * sizeof(E);
  E* out = static_cast<E*>(p.h) + b * p.T * p.C + c;
  for (int64_t t0 = 0; t0 < n; t0 += AT) {
    Row rx[AT], rf[AT], ri[AT];
#pragma unroll
    for (int k = 0; k < AT; ++k) {
      const int64_t t = t0 + k < n ? t0 + k : n - 1;
      rx[k] = *reinterpret_cast<const Row*>(x + t * p.ldx);
      rf[k] = *reinterpret_cast<const Row*>(f + t * p.ldf);
      if constexpr (IG) ri[k] = *reinterpret_cast<const Row*>(g + t * p.ldi);
    }
#pragma unroll
    for (int k = 0; k < AT; ++k) {
      const int64_t t = t0 + k;
      if (t >= n) break;
      if (p.marks != nullptr && t % kSpan == 0) store4(p.marks + (b * ((p.T + kSpan - 1) / kSpan) + t / kSpan) * p.C + c, h);
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const Gate q = gate_of<E, KIND, true>(float(rf[k][v]), decay[v]);
        float add = q.m * float(rx[k][v]);
        if constexpr (IG) add *= sigmoid_of<E>(float(ri[k][v]));
        h[v] = q.c < 0.5f ? h[v] + fmaf(-q.c, h[v], add) : fmaf(q.a, h[v], add);
      }
      if (p.h != nullptr) store4(out + t * p.C, h);
    }
  }
  if (p.h_final != nullptr && (n > 0 || p.h_final != p.h0)) store4(p.h_final + b * p.C + c, h);
}

template <typename F>
int by_gate(const gdn_scan_args& a, F f) {
  auto with = [&](auto kind) {
    return a.i != nullptr ? f(kind, std::true_type{}) : f(kind, std::false_type{});
  };
  switch (a.gate) {
    case GDN_SCAN_LOG: return with(std::integral_constant<int, GDN_SCAN_LOG>{});
    case GDN_SCAN_SIGMOID: return with(std::integral_constant<int, GDN_SCAN_SIGMOID>{});
    default: return with(std::integral_constant<int, GDN_SCAN_POWER>{});
  }
}

template <typename E>
int launch_step(const ScanProblem& q, const Pass& p, hipStream_t s) {
  return by_gate(q.a, [&](auto kind, auto gated) {
    constexpr int K = decltype(kind)::value;
    constexpr bool G = decltype(gated)::value;
    const unsigned blocks = (p.blocks + kStepThreads - 1) / kStepThreads;
    if (p.T == 1)
      scan_step_kernel<E, K, G, 1><<<blocks, kStepThreads, 0, s>>>(p);
    else
      scan_step_kernel<E, K, G, 4><<<blocks, kStepThreads, 0, s>>>(p);
    return int(hipGetLastError());
  });
}

// BACK: the gradients. Segments side by side take a first launch for their totals.
template <typename E, bool BACK>
int launch_pass(const ScanProblem& q, Pass p, hipStream_t s) {
  constexpr int N = Geo<BACK ? kBackLanes : kLanes>::template kChannels<E>;
  const int64_t slices = (q.a.C + N - 1) / N;
  p.slices = unsigned(slices);
  return by_gate(q.a, [&](auto kind, auto gated) {
    constexpr int K = decltype(kind)::value;
    constexpr bool G = decltype(gated)::value;
    if (p.segs > 1) {
      p.blocks = unsigned(q.a.B * slices * (p.segs - 1));
      if constexpr (BACK)
        scan_bwd_kernel<E, K, G, true><<<p.blocks, 64 * kBackWaves, 0, s>>>(p);
      else
        scan_kernel<E, K, G, true><<<p.blocks, 64 * kWaves, 0, s>>>(p);
      const int rc = int(hipGetLastError());
      if (rc != 0) return rc;
    }
    p.blocks = unsigned(q.a.B * slices * p.segs);
    if constexpr (BACK)
      scan_bwd_kernel<E, K, G, false><<<p.blocks, 64 * kBackWaves, 0, s>>>(p);
    else
      scan_kernel<E, K, G, false><<<p.blocks, 64 * kWaves, 0, s>>>(p);
    return int(hipGetLastError());
  });
}

// The instances, one element type a translation unit.
int step_bf16(const ScanProblem& q, const Pass& p, hipStream_t s);
int step_f32(const ScanProblem& q, const Pass& p, hipStream_t s);
int fwd_bf16(const ScanProblem& q, const Pass& p, hipStream_t s);
int fwd_f32(const ScanProblem& q, const Pass& p, hipStream_t s);
int bwd_bf16(const ScanProblem& q, const Pass& p, hipStream_t s);
int bwd_f32(const ScanProblem& q, const Pass& p, hipStream_t s);

}  // namespace scan
}  // namespace gdn
