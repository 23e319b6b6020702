// The gated recurrence a channel, h_t = a_t h_{t-1} + b_t, over long sequences: kernels and
// their launches for one element type.
//
// Eight lanes of a wave lie across the channels of a slice, four bytes a lane and row, and eight
// groups of lanes hold a run of consecutive tokens each. A lane joins the tokens of its run, the groups join theirs by shuffles, the waves of a workgroup theirs
// through LDS, and the workgroup walks the tiles of its segment with the state it carries.
// Joining two runs of tokens is (A, h) (A', h') -> (A A', A' h + h'): no division, so a decay
// may be 0, and nothing exceeds what the recurrence itself does.
//
// What a run leaves of the state before it is held twice: as the product A and as 1 - A,
// summed from the 1 - a of its tokens. Where less than half goes, the state loses (1 - A) h
// instead of being multiplied by a rounded A near 1, whose error a channel that keeps many
// tokens would add up at every step; and the state a workgroup carries is a sum of two
// floats, for the same reason.
#pragma once

#include <algorithm>

#include "gdn_block.h"
#include "gdn_block_device.h"

namespace gdn {
namespace scan {

constexpr int kSpan = GDN_SCAN_SPAN;   // tokens between checkpoints
constexpr int kLanes = 8;              // lanes across a slice's channels
constexpr int kRuns = 64 / kLanes;     // lane groups, a run of tokens each
constexpr int kWaves = 8;              // waves a workgroup
constexpr int kRun = kSpan / kRuns;    // tokens a run: a wave has a span
constexpr int kTile = kWaves * kSpan;

template <typename E> struct Shape {
  static constexpr int V = 4 / sizeof(E);   // channels a lane
  static constexpr int N = kLanes * V;      // channels a slice
};

// 1 - e^y for y <= 0 (and what it is above), to a few steps of its own: a series where the
// difference would cancel.
template <typename E>
__device__ __forceinline__ float one_minus_exp(float y, float ey) {
  float p;
  if constexpr (sizeof(E) == 2) {   // |y| < 1/4: y^5/720 is 2^-19 of y
    p = 1.0f + y * (0.5f + y * (1.0f / 6 + y * (1.0f / 24 + y * (1.0f / 120))));
  } else {                          // y^8/9! is 2^-34
    p = 1.0f / 24 + y * (1.0f / 120 + y * (1.0f / 720 + y * (1.0f / 5040 + y * (1.0f / 40320))));
    p = 1.0f + y * (0.5f + y * (1.0f / 6 + y * p));
  }
  return fabsf(y) < 0.25f ? -y * p : 1.0f - ey;
}

// A token's factors: h = a h + m g x with c = 1 - a. s and rest (sigmoid(f) and its
// complement) are the gradients'.
struct Gate {
  float a, c, m, s, rest;
};
template <typename E, int KIND>
__device__ __forceinline__ Gate gate_of(float f, float decay) {
  Gate g;
  if constexpr (KIND == GDN_SCAN_LOG) {
    g.a = exp_of<E>(f);
    g.c = one_minus_exp<E>(f, g.a);
    g.m = 1.0f;
    g.s = g.rest = 0.0f;
  } else {
    sigmoids<E>(f, &g.s, &g.rest);
    if constexpr (KIND == GDN_SCAN_SIGMOID) {
      g.a = g.s;
      g.c = g.m = g.rest;
    } else {
      const float y = -decay * g.s;
      g.a = exp_of<E>(y);
      g.c = one_minus_exp<E>(y, g.a);
      // 1 - a^2 = c (1 + a)
      g.m = sizeof(E) == 2 ? __builtin_amdgcn_sqrtf(g.c * (1.0f + g.a)) : sqrtf(g.c * (1.0f + g.a));
    }
  }
  return g;
}

// A run of tokens: what is left of the state before it (A, and C = 1 - A), and what it adds.
struct Run {
  float A, C, H;
};
__device__ __forceinline__ Run empty_run() { return {1.0f, 0.0f, 0.0f}; }
__device__ __forceinline__ Run join(const Run& first, const Run& then) {
  return {first.A * then.A, fmaf(then.C, first.A, first.C), fmaf(then.A, first.H, then.H)};
}

// The product of a run's rounded a's is off by a step for each of them, 1 - C by one: where a run
// leaves more than half, that is its A.
__device__ __forceinline__ void settle(Run& r) { r.A = r.C < 0.5f ? 1.0f - r.C : r.A; }

// A state held as hi + lo.
struct State {
  float hi, lo;
  __device__ __forceinline__ void pass(const Run& r) {
    const bool slow = r.C < 0.5f;
    const float base = slow ? hi : r.A * hi;
    const float add = slow ? fmaf(-r.C, hi, r.H) : r.H;
    const float sum = base + add, back = sum - base;
    lo = lo * r.A + ((base - (sum - back)) + (add - back));
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

// A buffer of `rows` rows of `width` bytes from `base` on, `ld` bytes apart; none for rows <= 0.
// Loads behind its last row give zero, stores are dropped. Strides are at most 2^26 bytes, so
// a span's offsets fit in 32 bits.
__device__ __forceinline__ uint4v rows_from(const char* base, int64_t ld, int64_t rows, uint32_t width) {
  auto uniform = [](uint32_t x) { return uint32_t(__builtin_amdgcn_readfirstlane(int(x))); };
  const uint64_t from = reinterpret_cast<uintptr_t>(base);
  const uint32_t bytes = rows > 0 ? uint32_t(rows < kSpan ? rows - 1 : kSpan - 1) * uint32_t(ld) + width : 0u;
  return {uniform(uint32_t(from)), uniform(uint32_t(from >> 32) & 0xffffu), uniform(bytes), 0x00020000u};
}

// Rows on their way from memory to LDS, two tiles ahead of their use: 32 bytes a row of a slice,
// a wave's own span, so that nothing but its own count of loads says when they are there. Lane l
// of a load brings sixteen bytes to the wave's place 16 l: row (l / 2 % 8) * 8 + l / 16 (and four
// on), so that the eight runs' rows r lie side by side and a lane reads its own at 256 r + 4 l,
// free of bank conflicts. The loads are written as assembly, which has no registers to guard;
// the compiler's own counts only ever wait for more.
struct Feed {
  uint32_t off[4];
  int64_t ld[4];
  const char* base[4];
  __device__ __forceinline__ void open(int k, const void* p, int64_t ld_, int64_t first, int lane) {
    base[k] = static_cast<const char*>(p) + first, ld[k] = ld_;
    off[k] = uint32_t((lane / 2 % 8) * 8 + lane / 16) * uint32_t(ld_) + lane % 2 * 16;
  }
  __device__ __forceinline__ void load(int k, char* to, int64_t t0, int64_t left, uint32_t width) const {
    const uint4v range = rows_from(base[k] + t0 * ld[k], ld[k], left, width);
    const uint32_t lds = __builtin_amdgcn_readfirstlane(uint32_t(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) char*)(to))));
    asm volatile("s_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"{m0}"(lds), "v"(off[k]), "s"(range) : "memory");
    asm volatile("s_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"{m0}"(lds + 1024), "v"(off[k] + 4 * uint32_t(ld[k])), "s"(range) : "memory");
  }
};
// Four bytes a lane, one load.
__device__ __forceinline__ void load_words(char* to, const char* from, uint32_t bytes, int lane) {
  const uint4v range = rows_from(from, 0, bytes > 0 ? 1 : 0, bytes);
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
// Before tile k: behind its LOADS loads came those of the tile after it and, from each of the two
// tiles before, STORES stores (others only add to what is waited for).
template <int LOADS, int STORES>
__device__ __forceinline__ void wait_tile(int64_t k) {
  if (STORES == 0 || k == 0) wait_memory<LOADS>();
  else if (k == 1) wait_memory<LOADS + STORES>();
  else wait_memory<LOADS + 2 * STORES>();
}
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
// A run's rows, one store each: `at` is the lane's place in the span's first row, behind the
// buffer where it has no channels.
__device__ __forceinline__ void store_run(char* base, int64_t ld, int64_t left, uint32_t width, int run, uint32_t at, const uint32_t* x) {
  const auto to = __builtin_amdgcn_make_buffer_rsrc(base, 0, int(rows_from(base, ld, left, width)[2]), 0x00020000);
#pragma unroll
  for (int r = 0; r < kRun; ++r)
    __builtin_amdgcn_raw_buffer_store_b32(x[r], to, at + uint32_t(run * kRun + r) * uint32_t(ld), 0, 0);
}

// Where a workgroup stands: blocks that follow each other on one XCD (their index modulo 8)
// are neighbouring slices of one segment, which share lines.
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

// The runs of a tile's waves through LDS, in order: `all` of them joined, and `mine`, those
// before this wave's.
template <int V, bool BACK>
__device__ __forceinline__ void join_waves(float4 (*part)[kLanes * V], int wave, int lane, const Run* own, Run* mine, Run* all) {
  if (lane / kLanes == (BACK ? 0 : kRuns - 1)) {
#pragma unroll
    for (int v = 0; v < V; ++v) part[wave][(lane % kLanes) * V + v] = make_float4(own[v].A, own[v].C, own[v].H, 0.0f);
  }
  __syncthreads();
#pragma unroll
  for (int v = 0; v < V; ++v) mine[v] = all[v] = empty_run();
#pragma unroll 2   // all at once would hold every wave's runs in registers
  for (int j = 0; j < kWaves; ++j) {
    const int w = BACK ? kWaves - 1 - j : j;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (w == wave) mine[v] = all[v];
      const float4 t = part[w][(lane % kLanes) * V + v];
      all[v] = join(all[v], {t.x, t.y, t.z});
    }
  }
}

// Joins over the lane groups: own becomes the runs up to and with the lane's (BACK: from the
// last one down to it); before those without it.
template <int V, bool BACK>
__device__ __forceinline__ void join_lanes(Run* own, Run* before, int lane) {
#pragma unroll
  for (int v = 0; v < V; ++v) {
#pragma unroll
    for (int d = kLanes; d < 64; d *= 2) {
      const Run o = BACK ? Run{__shfl_down(own[v].A, d), __shfl_down(own[v].C, d), __shfl_down(own[v].H, d)}
                         : Run{__shfl_up(own[v].A, d), __shfl_up(own[v].C, d), __shfl_up(own[v].H, d)};
      const Run j = join(o, own[v]);
      const bool there = BACK ? lane + d < 64 : lane >= d;
      own[v].A = there ? j.A : own[v].A, own[v].C = there ? j.C : own[v].C, own[v].H = there ? j.H : own[v].H;
    }
    const Run e = empty_run();
    before[v] = BACK ? Run{__shfl_down(own[v].A, kLanes), 0.0f, __shfl_down(own[v].H, kLanes)}
                     : Run{__shfl_up(own[v].A, kLanes), 0.0f, __shfl_up(own[v].H, kLanes)};
    if (BACK ? lane >= 64 - kLanes : lane < kLanes) before[v] = e;
  }
}

// Forward. TOTALS: only what each segment but the last makes of the state before it.
template <typename E, int KIND, bool IG, bool TOTALS>
__global__ __launch_bounds__(64 * kWaves) void scan_kernel(Pass p) {
  constexpr int V = Shape<E>::V, N = Shape<E>::N, NT = IG ? 3 : 2, kLoads = 2 * NT;
  __shared__ __attribute__((aligned(16))) char raw[2][kWaves][NT][32 * kSpan];
  __shared__ float4 part[2][kWaves][N];
  const Place at(p, TOTALS ? p.segs - 1 : p.segs);
  const int lane = threadIdx.x % 64, run = lane / kLanes;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int64_t c0 = int64_t(at.slice) * N;
  const bool own = c0 + (lane % kLanes) * V < p.C;                          // a slice may end behind C
  const uint32_t ch = own ? (lane % kLanes) * V : 0, width = (p.C - c0 < N ? uint32_t(p.C - c0) : N) * sizeof(E);
  const int64_t c = at.b * p.C + c0 + ch;
  const int64_t n = tokens_of(p.lens, at.b, p.T);
  const int64_t begin = at.seg * p.seg;
  if (begin >= n && at.seg > 0) return;
  const bool last = n - begin <= p.seg;
  if (TOTALS && at.seg == 0 && wave == 0 && run == 0 && own) {
#pragma unroll
    for (int v = 0; v < V; ++v) p.start[c + v] = p.h0 != nullptr ? p.h0[c + v] : 0.0f;
  }
  if (TOTALS && last) return;
  const int64_t end = last ? n : begin + p.seg;
  const int64_t ldh = p.C * sizeof(E);
  char* h = static_cast<char*>(p.h) + at.b * p.T * ldh + c0 * sizeof(E);
  const uint32_t to = own ? ch * uint32_t(sizeof(E)) : 0x80000000u;
  float decay[V];
  State carry[V];
  Run total[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    decay[v] = KIND == GDN_SCAN_POWER ? p.decay[c0 + ch + v] : 0.0f;
    const float* from = p.segs > 1 ? p.start : p.h0;
    carry[v] = {TOTALS || from == nullptr ? 0.0f : from[c + v], 0.0f};
    if constexpr (!TOTALS) {
      for (unsigned s = 0; s < at.seg; ++s) carry[v].pass(p.totals[(at.b * (p.segs - 1) + s) * p.C + c0 + ch + v]);
    }
    total[v] = empty_run();
  }
  Feed feed;
  feed.open(0, p.x, p.ldx, at.b * p.T * p.ldx + c0 * int64_t(sizeof(E)), lane);
  feed.open(1, p.f, p.ldf, at.b * p.T * p.ldf + c0 * int64_t(sizeof(E)), lane);
  if constexpr (IG) feed.open(2, p.i, p.ldi, at.b * p.T * p.ldi + c0 * int64_t(sizeof(E)), lane);
  auto fetch = [&](int stage, int64_t t0) {
#pragma unroll
    for (int k = 0; k < NT; ++k) feed.load(k, raw[stage][wave][k], t0, end - t0, width);
  };
  const int64_t first = begin + wave * kSpan, tiles = (end - begin + kTile - 1) / kTile;
  fetch(0, first);
  fetch(1, first + kTile);
  // a tile whose rows are all there, or the last
  auto walk = [&](auto full, int64_t k) {
    constexpr bool FULL = decltype(full)::value;
    const int stage = k & 1;
    const int64_t t0 = first + k * kTile, left = end - t0;
    if (!TOTALS && p.h != nullptr) wait_tile<kLoads, kRun>(k);
    else wait_tile<kLoads, 0>(k);
    uint32_t in[NT][kRun];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int r = 0; r < kRun; ++r) in[t][r] = *reinterpret_cast<const uint32_t*>(raw[stage][wave][t] + 256 * r + 4 * lane);
    }
    wait_lds();
    fetch(stage, t0 + 2 * kTile);
    float a[kRun][V], b[kRun][V];
    Run own_run[V], before[V], mine[V], all[V];
#pragma unroll
    for (int v = 0; v < V; ++v) own_run[v] = empty_run();
#pragma unroll
    for (int r = 0; r < kRun; ++r) {
      const bool here = FULL || run * kRun + r < left;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const Gate t = gate_of<E, KIND>(part_of<E>(in[1][r], v), decay[v]);
        a[r][v] = here ? t.a : 1.0f;
        b[r][v] = KIND == GDN_SCAN_LOG ? part_of<E>(in[0][r], v) : t.m * part_of<E>(in[0][r], v);
        if constexpr (IG) b[r][v] *= sigmoid_of<E>(part_of<E>(in[2][r], v));
        if (!here) b[r][v] = 0.0f;
        own_run[v] = join(own_run[v], Run{a[r][v], here ? t.c : 0.0f, b[r][v]});
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) settle(own_run[v]);
    join_lanes<V, false>(own_run, before, lane);
    join_waves<V, false>(part[stage], wave, lane, own_run, mine, all);
    if constexpr (TOTALS) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        carry[v].pass(all[v]);
        total[v] = join(total[v], all[v]);
      }
    } else {
      float y[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        State s = carry[v];
        s.pass(mine[v]);
        y[v] = fmaf(before[v].A, s.value(), before[v].H);
        carry[v].pass(all[v]);
      }
      if (p.marks != nullptr && run == 0 && own && left > 0) {
        float* m = p.marks + (at.b * ((p.T + kSpan - 1) / kSpan) + t0 / kSpan) * p.C + c0 + ch;
#pragma unroll
        for (int v = 0; v < V; ++v) m[v] = y[v];
      }
      if (p.h != nullptr) {
        uint32_t out[kRun];
#pragma unroll
        for (int r = 0; r < kRun; ++r) {
#pragma unroll
          for (int v = 0; v < V; ++v) y[v] = fmaf(a[r][v], y[v], b[r][v]);
          out[r] = packed<E>(y);
        }
        store_run(h + t0 * ldh, ldh, left, width, run, to, out);
      }
    }
  };
  int64_t k = 0;
  for (; (k + 1) * kTile <= end - begin; ++k) walk(std::true_type{}, k);
  if (k < tiles) walk(std::false_type{}, k);
  wait_memory<0>();   // of LDS that the next workgroup may get
  if (wave != 0 || run != 0 || !own) return;
  if constexpr (TOTALS) {
#pragma unroll
    for (int v = 0; v < V; ++v)
      p.totals[(at.b * (p.segs - 1) + at.seg) * p.C + c0 + ch + v] = {total[v].A, total[v].C, carry[v].value()};
  } else if (last && p.h_final != nullptr) {
#pragma unroll
    for (int v = 0; v < V; ++v) p.h_final[c + v] = carry[v].value();
  }
}

// Gradients, from a sequence's end: with G_t = a_t (d_h_t + G_{t+1}) the same recurrence, whose
// value behind token t is l_t = d_h_t + G_{t+1}. h comes from the state before the span. TOTALS:
// only what each segment but the first makes of the gradient behind it.
template <typename E, int KIND, bool IG, bool TOTALS>
__global__ __launch_bounds__(64 * kWaves) void scan_bwd_kernel(Pass p) {
  constexpr int V = Shape<E>::V, N = Shape<E>::N, R = kRun;
  constexpr int NT = TOTALS ? 2 : IG ? 4 : 3, kLoads = 2 * NT + (TOTALS ? 0 : 1), kStores = TOTALS ? 0 : R * (IG ? 3 : 2);
  __shared__ __attribute__((aligned(16))) char raw[2][kWaves][NT][32 * kSpan];
  __shared__ __attribute__((aligned(16))) char raw_marks[2][kWaves][TOTALS ? 16 : 256];
  __shared__ float4 part[2][kWaves][N];
  Place at(p, TOTALS ? p.segs - 1 : p.segs);
  if (TOTALS) ++at.seg;
  const int lane = threadIdx.x % 64, run = lane / kLanes;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int64_t c0 = int64_t(at.slice) * N;
  const bool own = c0 + (lane % kLanes) * V < p.C;
  const uint32_t ch = own ? (lane % kLanes) * V : 0, channels = p.C - c0 < N ? uint32_t(p.C - c0) : N;
  const uint32_t width = channels * sizeof(E);
  const int64_t c = at.b * p.C + c0 + ch;
  const int64_t n = tokens_of(p.lens, at.b, p.T);
  const int64_t begin = at.seg * p.seg;
  const int64_t stop = std::min(begin + p.seg, p.T), end = std::min(stop, n);
  const int64_t ldh = p.C * sizeof(E), row0 = at.b * p.T * ldh + c0 * int64_t(sizeof(E));
  char* dx = static_cast<char*>(p.dx) + row0;
  char* df = static_cast<char*>(p.df) + row0;
  char* di = static_cast<char*>(p.di) + row0;
  const uint32_t to = own ? ch * uint32_t(sizeof(E)) : 0x80000000u;
  if constexpr (!TOTALS) {
    // rows behind the length: zero
    for (int64_t t = std::max(begin, n) + wave * kRuns + run; own && t < stop; t += kWaves * kRuns) {
      *reinterpret_cast<uint32_t*>(dx + t * ldh + to) = 0, *reinterpret_cast<uint32_t*>(df + t * ldh + to) = 0;
      if constexpr (IG) *reinterpret_cast<uint32_t*>(di + t * ldh + to) = 0;
    }
  }
  if (TOTALS && begin >= n) return;
  float decay[V], sum[V];
  State carry[V];
  Run total[V];
  const int64_t segs_used = (n + p.seg - 1) / p.seg;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    decay[v] = KIND == GDN_SCAN_POWER ? p.decay[c0 + ch + v] : 0.0f;
    carry[v] = {TOTALS || p.d_final == nullptr ? 0.0f : p.d_final[c + v], 0.0f};
    if constexpr (!TOTALS) {
      for (int64_t s = segs_used - 1; s > int64_t(at.seg); --s)
        carry[v].pass(p.totals[(at.b * (p.segs - 1) + s - 1) * p.C + c0 + ch + v]);
    }
    total[v] = empty_run(), sum[v] = 0.0f;
  }
  Feed feed;
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
  const int64_t tiles = end > begin ? (end - begin + kTile - 1) / kTile : 0;
  const int64_t first = begin + (tiles - 1) * kTile + wave * kSpan;   // the last tile comes first
  if (tiles > 0) {
    fetch(0, first);
    fetch(1, first - kTile);
  }
  auto walk = [&](auto full, int64_t k) {
    constexpr bool FULL = decltype(full)::value;
    const int stage = k & 1;
    const int64_t t0 = first - k * kTile, left = end - t0;
    wait_tile<kLoads, kStores>(k);
    uint32_t in[NT][R];
    float mark[V];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int r = 0; r < R; ++r) in[t][r] = *reinterpret_cast<const uint32_t*>(raw[stage][wave][t] + 256 * r + 4 * lane);
    }
    if constexpr (!TOTALS) {
#pragma unroll
      for (int v = 0; v < V; ++v) mark[v] = reinterpret_cast<const float*>(raw_marks[stage][wave])[(lane % kLanes) * V + v];
    }
    wait_lds();
    fetch(stage, t0 - 2 * kTile);
    Gate gate[R][V];
    float si[R][V], resti[R][V], before[R][V];
    Run own_run[V], lanes[V], mine[V], all[V];
#pragma unroll
    for (int v = 0; v < V; ++v) own_run[v] = empty_run();
    // G of the run, from its last token
#pragma unroll
    for (int r = R - 1; r >= 0; --r) {
      const bool here = FULL || run * R + r < left;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        Gate& t = gate[r][v];
        t = gate_of<E, KIND>(part_of<E>(in[0][r], v), decay[v]);
        if (!here) t.a = 1.0f;
        const float up = part_of<E>(in[1][r], v);
        own_run[v] = join(own_run[v], Run{t.a, here ? t.c : 0.0f, here ? t.a * up : 0.0f});
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
    if constexpr (!TOTALS) {
      // h before each token: from what each adds
      Run fwd[V], ahead[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        fwd[v] = {own_run[v].A, 0.0f, 0.0f};
#pragma unroll
        for (int r = 0; r < R; ++r) fwd[v].H = fmaf(gate[r][v].a, fwd[v].H, before[r][v]);
      }
      join_lanes<V, false>(fwd, ahead, lane);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float y = fmaf(ahead[v].A, mark[v], ahead[v].H);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float add = before[r][v];
          before[r][v] = y;
          y = fmaf(gate[r][v].a, y, add);
        }
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) settle(own_run[v]);
    join_lanes<V, true>(own_run, lanes, lane);
    join_waves<V, true>(part[stage], wave, lane, own_run, mine, all);
    if constexpr (TOTALS) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        carry[v].pass(all[v]);
        total[v] = join(total[v], all[v]);
      }
    } else {
      float G[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        State s = carry[v];
        s.pass(mine[v]);
        G[v] = fmaf(lanes[v].A, s.value(), lanes[v].H);
        carry[v].pass(all[v]);
      }
#pragma unroll
      for (int r = R - 1; r >= 0; --r) {
        const bool here = FULL || run * R + r < left;
        float ox[V], of[V], oi[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const Gate& t = gate[r][v];
          const float xv = part_of<E>(in[2][r], v), l = part_of<E>(in[1][r], v) + G[v];
          const float lm = KIND == GDN_SCAN_LOG ? l : l * t.m;
          ox[v] = IG ? lm * si[r][v] : lm;
          if constexpr (IG) oi[v] = ox[v] * xv * resti[r][v];
          const float gx = IG ? si[r][v] * xv : xv;
          if constexpr (KIND == GDN_SCAN_LOG) {
            of[v] = l * before[r][v] * t.a;
          } else if constexpr (KIND == GDN_SCAN_SIGMOID) {
            of[v] = l * (before[r][v] - gx) * (t.a * t.c);
          } else {
            // d m / d a = -a / m
            const float slope = t.m > 0.0f ? t.a * gx * __builtin_amdgcn_rcpf(t.m) : 0.0f;
            const float dlog = l * t.a * (before[r][v] - slope) * t.s;
            of[v] = -decay[v] * t.rest * dlog;
            sum[v] -= here ? dlog : 0.0f;
          }
          G[v] = here ? t.a * l : G[v];
        }
        in[2][r] = packed<E>(ox), in[0][r] = packed<E>(of);
        if constexpr (IG) in[3][r] = packed<E>(oi);
      }
      store_run(dx + t0 * ldh, ldh, left, width, run, to, in[2]);
      store_run(df + t0 * ldh, ldh, left, width, run, to, in[0]);
      if constexpr (IG) store_run(di + t0 * ldh, ldh, left, width, run, to, in[3]);
    }
  };
  int64_t k = 0;
  if (tiles * kTile > end - begin && tiles > 0) walk(std::false_type{}, k++);
  for (; k < tiles; ++k) walk(std::true_type{}, k);
  wait_memory<0>();
  if constexpr (TOTALS) {
    if (wave == 0 && run == 0 && own) {
#pragma unroll
      for (int v = 0; v < V; ++v)
        p.totals[(at.b * (p.segs - 1) + at.seg - 1) * p.C + c0 + ch + v] = {total[v].A, total[v].C, carry[v].value()};
    }
  } else {
    if (at.seg == 0 && p.dh0 != nullptr && wave == 0 && run == 0 && own) {
#pragma unroll
      for (int v = 0; v < V; ++v) p.dh0[c + v] = carry[v].value();
    }
    if (KIND == GDN_SCAN_POWER && p.ddecay != nullptr) {
      // over the lane groups, then the waves
      float* sums = reinterpret_cast<float*>(part);
      __syncthreads();
#pragma unroll
      for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int m = kLanes; m < 64; m *= 2) sum[v] += __shfl_xor(sum[v], m);
        if (run == 0) sums[wave * N + (lane % kLanes) * V + v] = sum[v];
      }
      __syncthreads();
      if (wave == 0 && run == 0 && own) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
          float t = 0.0f;
          for (int w = 0; w < kWaves; ++w) t += sums[w * N + (lane % kLanes) * V + v];
          p.ddecay[(at.b * p.segs + at.seg) * p.C + c0 + ch + v] = t;
        }
      }
    }
  }
}

// Token by token, four channels a thread: single tokens, where each sequence's state is read
// and written once. Where less than half of a state goes, (1 - a) h is taken from it.
constexpr int kStepThreads = 256;
template <typename E, int KIND, bool IG>
__global__ __launch_bounds__(kStepThreads) void scan_step_kernel(Pass p) {
  const unsigned per = unsigned(p.C / 4);
  const unsigned id = blockIdx.x * kStepThreads + threadIdx.x;
  if (id >= p.blocks) return;   // (sequence, channels): B * C / 4 of them
  const int64_t b = id / per, c = int64_t(id % per) * 4;
  const int64_t n = tokens_of(p.lens, b, p.T);
  float h[4] = {}, decay[4] = {};
  if (p.h0 != nullptr) load4(p.h0 + b * p.C + c, h);
  if constexpr (KIND == GDN_SCAN_POWER) load4(p.decay + c, decay);
  const int64_t ldh = p.C * int64_t(sizeof(E));
  for (int64_t t = 0; t < n; ++t) {
    const int64_t row = b * p.T + t;
    float x[4], f[4], i[4], out[4];
    load4(reinterpret_cast<const E*>(static_cast<const char*>(p.x) + row * p.ldx) + c, x);
    load4(reinterpret_cast<const E*>(static_cast<const char*>(p.f) + row * p.ldf) + c, f);
    if constexpr (IG) load4(reinterpret_cast<const E*>(static_cast<const char*>(p.i) + row * p.ldi) + c, i);
    if (p.marks != nullptr && t % kSpan == 0) store4(p.marks + (b * ((p.T + kSpan - 1) / kSpan) + t / kSpan) * p.C + c, h);
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const Gate g = gate_of<E, KIND>(f[v], decay[v]);
      float add = g.m * x[v];
      if constexpr (IG) add *= sigmoid_of<E>(i[v]);
      out[v] = h[v] = g.c < 0.5f ? h[v] + fmaf(-g.c, h[v], add) : fmaf(g.a, h[v], add);
    }
    store4(reinterpret_cast<E*>(static_cast<char*>(p.h) + row * ldh) + c, out);
  }
  if (p.h_final != nullptr) store4(p.h_final + b * p.C + c, h);
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
    scan_step_kernel<E, decltype(kind)::value, decltype(gated)::value>
        <<<(p.blocks + kStepThreads - 1) / kStepThreads, kStepThreads, 0, s>>>(p);
    return int(hipGetLastError());
  });
}

// BACK: the gradients. Segments side by side take a first launch for their totals.
template <typename E, bool BACK>
int launch_pass(const ScanProblem& q, Pass p, hipStream_t s) {
  const int64_t slices = (q.a.C + Shape<E>::N - 1) / Shape<E>::N;
  p.slices = unsigned(slices);
  return by_gate(q.a, [&](auto kind, auto gated) {
    constexpr int K = decltype(kind)::value;
    constexpr bool G = decltype(gated)::value;
    if (p.segs > 1) {
      p.blocks = unsigned(q.a.B * slices * (p.segs - 1));
      if constexpr (BACK)
        scan_bwd_kernel<E, K, G, true><<<p.blocks, 64 * kWaves, 0, s>>>(p);
      else
        scan_kernel<E, K, G, true><<<p.blocks, 64 * kWaves, 0, s>>>(p);
      const int rc = int(hipGetLastError());
      if (rc != 0) return rc;
    }
    p.blocks = unsigned(q.a.B * slices * p.segs);
    if constexpr (BACK)
      scan_bwd_kernel<E, K, G, false><<<p.blocks, 64 * kWaves, 0, s>>>(p);
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
