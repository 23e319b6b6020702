// The gated recurrence a channel, h_t = a_t h_{t-1} + b_t, over long sequences: kernels and
// their launches for one element type.
//
// A span of 64 tokens is a wave's: eight lanes lie across the channels of a slice, four bytes
// a lane and row, and eight groups of lanes hold eight consecutive tokens each. A lane joins
// its eight tokens, the groups join theirs by shuffles, the waves of a workgroup theirs
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

constexpr int kSpan = GDN_SCAN_SPAN;
constexpr int kLanes = 8;              // lanes across a slice's channels
constexpr int kRuns = 64 / kLanes;     // lane groups, a run of tokens each
constexpr int kRun = kSpan / kRuns;    // tokens a run
constexpr int kWaves = 16;             // waves a workgroup of the forward pass: spans a tile
constexpr int kBackWaves = 8;          // and of the gradients

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

// Rows of a run of tokens, four bytes a lane: `base` is a span's first row at a slice's first
// channel, `at` the lane's channel in bytes. `left` (>= 1) tokens of the span are present; those
// behind them repeat the last.
__device__ __forceinline__ void load_run(uint32_t* out, const char* base, int64_t ld, int run, uint32_t at, int64_t left) {
  if (left >= kSpan) {
    const uint32_t off = uint32_t(run * kRun) * uint32_t(ld) + at;
#pragma unroll
    for (int r = 0; r < kRun; ++r) out[r] = *reinterpret_cast<const uint32_t*>(base + r * ld + off);
  } else {
#pragma unroll
    for (int r = 0; r < kRun; ++r) {
      const int row = run * kRun + r;
      out[r] = *reinterpret_cast<const uint32_t*>(base + (row < left ? row : left - 1) * ld + at);
    }
  }
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
// Row r of a run goes to `base` (a span's first row) where it is present and the lane has channels.
__device__ __forceinline__ void store_row(char* base, int64_t ld, int run, int r, uint32_t at, int64_t left, bool own, uint32_t x) {
  const uint32_t off = uint32_t(run * kRun) * uint32_t(ld) + at;
  if (own && run * kRun + r < left) *reinterpret_cast<uint32_t*>(base + r * ld + off) = x;
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
template <int V, int NW, bool BACK>
__device__ __forceinline__ void join_waves(float4 (*part)[kLanes * V], int wave, int lane, const Run* own, Run* mine, Run* all) {
  if (lane / kLanes == (BACK ? 0 : kRuns - 1)) {
#pragma unroll
    for (int v = 0; v < V; ++v) part[wave][(lane % kLanes) * V + v] = make_float4(own[v].A, own[v].C, own[v].H, 0.0f);
  }
  __syncthreads();
#pragma unroll
  for (int v = 0; v < V; ++v) mine[v] = all[v] = empty_run();
#pragma unroll 2   // all at once would hold every wave's runs in registers
  for (int j = 0; j < NW; ++j) {
    const int w = BACK ? NW - 1 - j : j;
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

// Forward. TOTALS: only what each segment but the last makes of the state before it. A tile's
// rows are loaded while the one before it is joined and written.
template <typename E, int KIND, bool IG, bool TOTALS>
__global__ __launch_bounds__(64 * kWaves) void scan_kernel(Pass p) {
  constexpr int V = Shape<E>::V, N = Shape<E>::N, kTile = kWaves * kSpan;
  __shared__ float4 part[2][kWaves][N];
  const Place at(p, TOTALS ? p.segs - 1 : p.segs);
  const int lane = threadIdx.x % 64, run = lane / kLanes;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int64_t c0 = int64_t(at.slice) * N;
  const bool own = c0 + (lane % kLanes) * V < p.C;
  const uint32_t ch = own ? (lane % kLanes) * V : uint32_t(p.C - V - c0);   // of a slice that ends behind C
  const uint32_t off = ch * sizeof(E);
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
  const char* x = static_cast<const char*>(p.x) + at.b * p.T * p.ldx + c0 * sizeof(E);
  const char* f = static_cast<const char*>(p.f) + at.b * p.T * p.ldf + c0 * sizeof(E);
  const char* g = static_cast<const char*>(p.i) + at.b * p.T * p.ldi + c0 * sizeof(E);
  char* h = static_cast<char*>(p.h) + at.b * p.T * ldh + c0 * sizeof(E);
  uint32_t rx[kRun], rf[kRun], ri[kRun];
  auto fetch = [&](int64_t t0) {
    const int64_t left = end - t0;
    if (left <= 0) return;
    load_run(rx, x + t0 * p.ldx, p.ldx, run, off, left);
    load_run(rf, f + t0 * p.ldf, p.ldf, run, off, left);
    if constexpr (IG) load_run(ri, g + t0 * p.ldi, p.ldi, run, off, left);
  };
  fetch(begin + wave * kSpan);
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
  int buf = 0;
  for (int64_t tile = begin; tile < end; tile += kTile, buf ^= 1) {
    const int64_t t0 = tile + wave * kSpan, left = end - t0;
    float a[kRun][V], b[kRun][V];
    Run own_run[V], before[V], mine[V], all[V];
#pragma unroll
    for (int v = 0; v < V; ++v) own_run[v] = empty_run();
    if (left > 0) {
#pragma unroll
      for (int r = 0; r < kRun; ++r) {
        const bool here = run * kRun + r < left;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const Gate t = gate_of<E, KIND>(part_of<E>(rf[r], v), decay[v]);
          float add = t.m * part_of<E>(rx[r], v);
          if constexpr (IG) add *= sigmoid_of<E>(part_of<E>(ri[r], v));
          a[r][v] = here ? t.a : 1.0f;
          b[r][v] = here ? add : 0.0f;
          own_run[v] = join(own_run[v], Run{a[r][v], here ? t.c : 0.0f, b[r][v]});
        }
      }
    }
    fetch(t0 + kTile);
    join_lanes<V, false>(own_run, before, lane);
    join_waves<V, kWaves, false>(part[buf], wave, lane, own_run, mine, all);
    if constexpr (TOTALS) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        carry[v].pass(all[v]);
        total[v] = join(total[v], all[v]);
      }
    } else {
      float in[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        State s = carry[v];
        s.pass(mine[v]);
        in[v] = s.value();
        carry[v].pass(all[v]);
      }
      if (left > 0) {
        if (p.marks != nullptr && run == 0 && own) {
          float* m = p.marks + (at.b * ((p.T + kSpan - 1) / kSpan) + t0 / kSpan) * p.C + c0 + ch;
#pragma unroll
          for (int v = 0; v < V; ++v) m[v] = in[v];
        }
        if (p.h != nullptr) {
          float y[V];
#pragma unroll
          for (int v = 0; v < V; ++v) y[v] = fmaf(before[v].A, in[v], before[v].H);
#pragma unroll
          for (int r = 0; r < kRun; ++r) {
#pragma unroll
            for (int v = 0; v < V; ++v) y[v] = fmaf(a[r][v], y[v], b[r][v]);
            store_row(h + t0 * ldh, ldh, run, r, off, left, own, packed<E>(y));
          }
        }
      }
    }
  }
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
__global__ __launch_bounds__(64 * kBackWaves) void scan_bwd_kernel(Pass p) {
  constexpr int V = Shape<E>::V, N = Shape<E>::N, kTile = kBackWaves * kSpan;
  __shared__ float4 part[2][kBackWaves][N];
  Place at(p, TOTALS ? p.segs - 1 : p.segs);
  if (TOTALS) ++at.seg;
  const int lane = threadIdx.x % 64, run = lane / kLanes;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int64_t c0 = int64_t(at.slice) * N;
  const bool own = c0 + (lane % kLanes) * V < p.C;
  const uint32_t ch = own ? (lane % kLanes) * V : uint32_t(p.C - V - c0);
  const uint32_t off = ch * sizeof(E);
  const int64_t c = at.b * p.C + c0 + ch;
  const int64_t n = tokens_of(p.lens, at.b, p.T);
  const int64_t begin = at.seg * p.seg;
  const int64_t stop = std::min(begin + p.seg, p.T), end = std::min(stop, n);
  const int64_t ldh = p.C * sizeof(E);
  char* dx = static_cast<char*>(p.dx) + at.b * p.T * ldh + c0 * sizeof(E);
  char* df = static_cast<char*>(p.df) + at.b * p.T * ldh + c0 * sizeof(E);
  char* di = static_cast<char*>(p.di) + at.b * p.T * ldh + c0 * sizeof(E);
  if constexpr (!TOTALS) {
    // rows behind the length: zero
    for (int64_t t = std::max(begin, n) + wave * kRuns + run; t < stop; t += kBackWaves * kRuns) {
      if (!own) break;
      *reinterpret_cast<uint32_t*>(dx + t * ldh + off) = 0, *reinterpret_cast<uint32_t*>(df + t * ldh + off) = 0;
      if constexpr (IG) *reinterpret_cast<uint32_t*>(di + t * ldh + off) = 0;
    }
  }
  if (TOTALS && begin >= n) return;
  const char* x = static_cast<const char*>(p.x) + at.b * p.T * p.ldx + c0 * sizeof(E);
  const char* f = static_cast<const char*>(p.f) + at.b * p.T * p.ldf + c0 * sizeof(E);
  const char* g = static_cast<const char*>(p.i) + at.b * p.T * p.ldi + c0 * sizeof(E);
  const char* d = static_cast<const char*>(p.d_h) + at.b * p.T * ldh + c0 * sizeof(E);
  struct Rows {
    uint32_t x[kRun], f[kRun], i[kRun], d[kRun];
  } next;
  auto fetch = [&](int64_t t0) {
    const int64_t left = end - t0;
    if (left <= 0) return;
    load_run(next.f, f + t0 * p.ldf, p.ldf, run, off, left);
    load_run(next.d, d + t0 * ldh, ldh, run, off, left);
    if constexpr (!TOTALS) {
      load_run(next.x, x + t0 * p.ldx, p.ldx, run, off, left);
      if constexpr (IG) load_run(next.i, g + t0 * p.ldi, p.ldi, run, off, left);
    }
  };
  const int64_t tiles = end > begin ? (end - begin + kTile - 1) / kTile : 0;
  int64_t tile = begin + (tiles - 1) * kTile;
  if (tiles > 0) fetch(tile + wave * kSpan);
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
  int buf = 0;
  for (int64_t k = 0; k < tiles; ++k, tile -= kTile, buf ^= 1) {
    const int64_t t0 = tile + wave * kSpan, left = end - t0;
    const Rows now = next;
    Gate gate[kRun][V];
    float si[kRun][V], resti[kRun][V], before[kRun][V];
    Run own_run[V], lanes[V], mine[V], all[V];
#pragma unroll
    for (int v = 0; v < V; ++v) own_run[v] = empty_run();
    if (left > 0) {
      // G of the run, from its last token
#pragma unroll
      for (int r = kRun - 1; r >= 0; --r) {
        const bool here = run * kRun + r < left;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          Gate& t = gate[r][v];
          t = gate_of<E, KIND>(part_of<E>(now.f[r], v), decay[v]);
          t.a = here ? t.a : 1.0f;
          const float up = here ? part_of<E>(now.d[r], v) : 0.0f;
          own_run[v] = join(own_run[v], Run{t.a, here ? t.c : 0.0f, t.a * up});
          if constexpr (!TOTALS) {
            float add = t.m * part_of<E>(now.x[r], v);
            if constexpr (IG) {
              sigmoids<E>(part_of<E>(now.i[r], v), &si[r][v], &resti[r][v]);
              add *= si[r][v];
            }
            before[r][v] = here ? add : 0.0f;
          }
        }
      }
    }
    if (k + 1 < tiles) fetch(t0 - kTile);
    if constexpr (!TOTALS) {
      // h before each token: from what each adds
      Run fwd[V], ahead[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        fwd[v] = empty_run();
        if (left > 0) {
#pragma unroll
          for (int r = 0; r < kRun; ++r) fwd[v] = join(fwd[v], Run{gate[r][v].a, 0.0f, before[r][v]});
        }
      }
      join_lanes<V, false>(fwd, ahead, lane);
      if (left > 0) {
        const float* m = p.marks + (at.b * ((p.T + kSpan - 1) / kSpan) + t0 / kSpan) * p.C + c0 + ch;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          float y = fmaf(ahead[v].A, m[v], ahead[v].H);
#pragma unroll
          for (int r = 0; r < kRun; ++r) {
            const float add = before[r][v];
            before[r][v] = y;
            y = fmaf(gate[r][v].a, y, add);
          }
        }
      }
    }
    join_lanes<V, true>(own_run, lanes, lane);
    join_waves<V, kBackWaves, true>(part[buf], wave, lane, own_run, mine, all);
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
      if (left > 0) {
#pragma unroll
        for (int r = kRun - 1; r >= 0; --r) {
          float ox[V], of[V], oi[V];
          const bool here = run * kRun + r < left;
#pragma unroll
          for (int v = 0; v < V; ++v) {
            const Gate& t = gate[r][v];
            const float xv = part_of<E>(now.x[r], v), l = part_of<E>(now.d[r], v) + G[v];
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
          store_row(dx + t0 * ldh, ldh, run, r, off, left, own, packed<E>(ox));
          store_row(df + t0 * ldh, ldh, run, r, off, left, own, packed<E>(of));
          if constexpr (IG) store_row(di + t0 * ldh, ldh, run, r, off, left, own, packed<E>(oi));
        }
      }
    }
  }
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
          for (int w = 0; w < kBackWaves; ++w) t += sums[w * N + (lane % kLanes) * V + v];
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
