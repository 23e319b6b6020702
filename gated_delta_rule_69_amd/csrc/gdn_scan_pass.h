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
constexpr int kWaves = 4;              // waves a workgroup: spans a tile
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
  int64_t seg;          // tokens a segment, a multiple of kTile
  unsigned slices, segs, blocks;
  float* start;         // [B][C]: h0, where segments run side by side
  Run* totals;          // [B][segs - 1][C]
  // gradients
  const void* d_h;
  const float* d_final;
  void *dx, *df, *di;
  float *dh0, *ddecay;  // ddecay: [B * segs][C] partial sums
};

// Rows base + r ld of a run of tokens, four bytes a lane: from a span's first row at a lane's
// channel, `left` (>= 1) tokens of it present; those behind them repeat the last.
__device__ __forceinline__ void load_run(uint32_t* out, const char* base, int64_t ld, int run, int64_t left) {
  if (left >= kSpan) {
    const uint32_t off = uint32_t(run * kRun) * uint32_t(ld);
#pragma unroll
    for (int r = 0; r < kRun; ++r) out[r] = *reinterpret_cast<const uint32_t*>(base + r * ld + off);
  } else {
#pragma unroll
    for (int r = 0; r < kRun; ++r) {
      const int row = run * kRun + r;
      out[r] = *reinterpret_cast<const uint32_t*>(base + (row < left ? row : left - 1) * ld);
    }
  }
}
template <typename E>
__device__ __forceinline__ float part_of(uint32_t raw, int v) {
  if constexpr (sizeof(E) == 4) return __uint_as_float(raw);
  return v == 0 ? __uint_as_float(raw << 16) : __uint_as_float(raw & 0xffff0000u);
}
template <typename E>
__device__ __forceinline__ void store_parts(char* at, const float* x) {
  if constexpr (sizeof(E) == 4) {
    *reinterpret_cast<float*>(at) = x[0];
  } else {
    bhalf2 r = {E(x[0]), E(x[1])};
    *reinterpret_cast<bhalf2*>(at) = r;
  }
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

// The runs of a tile's waves through LDS: joined up to this wave, and in all.
template <int V, bool BACK>
__device__ __forceinline__ void pass_waves(float4 (*part)[kLanes * V], int wave, int lane, const Run* own, State* carry,
                                           float* in) {
  if (lane / kLanes == (BACK ? 0 : kRuns - 1)) {
#pragma unroll
    for (int v = 0; v < V; ++v) part[wave][(lane % kLanes) * V + v] = make_float4(own[v].A, own[v].C, own[v].H, 0.0f);
  }
  __syncthreads();
#pragma unroll
  for (int v = 0; v < V; ++v) {
#pragma unroll
    for (int j = 0; j < kWaves; ++j) {
      const int w = BACK ? kWaves - 1 - j : j;
      if (w == wave) in[v] = carry[v].value();
      const float4 t = part[w][(lane % kLanes) * V + v];
      carry[v].pass({t.x, t.y, t.z});
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
  constexpr int V = Shape<E>::V, N = Shape<E>::N;
  __shared__ float4 part[2][kWaves][N];
  const Place at(p, TOTALS ? p.segs - 1 : p.segs);
  const int lane = threadIdx.x % 64, run = lane / kLanes;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int64_t c_all = int64_t(at.slice) * N + (lane % kLanes) * V;
  const bool own = c_all < p.C;
  const int64_t c = own ? c_all : p.C - V;   // of a slice that ends behind C
  const int64_t n = tokens_of(p.lens, at.b, p.T);
  const int64_t begin = at.seg * p.seg;
  if (begin >= n && at.seg > 0) return;
  const bool last = n - begin <= p.seg;
  if (TOTALS && at.seg == 0 && wave == 0 && run == 0 && own) {
#pragma unroll
    for (int v = 0; v < V; ++v) p.start[at.b * p.C + c + v] = p.h0 != nullptr ? p.h0[at.b * p.C + c + v] : 0.0f;
  }
  if (TOTALS && last) return;
  const int64_t end = last ? n : begin + p.seg;
  float decay[V];
  State carry[V];
  float A_all[V], C_all[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    decay[v] = KIND == GDN_SCAN_POWER ? p.decay[c + v] : 0.0f;
    const float* from = p.segs > 1 ? p.start : p.h0;
    carry[v] = {TOTALS || from == nullptr ? 0.0f : from[at.b * p.C + c + v], 0.0f};
    if constexpr (!TOTALS) {
      for (unsigned s = 0; s < at.seg; ++s) carry[v].pass(p.totals[(at.b * (p.segs - 1) + s) * p.C + c + v]);
    }
    A_all[v] = 1.0f, C_all[v] = 0.0f;
  }
  const char* x = static_cast<const char*>(p.x) + at.b * p.T * p.ldx + c * sizeof(E);
  const char* f = static_cast<const char*>(p.f) + at.b * p.T * p.ldf + c * sizeof(E);
  const char* g = static_cast<const char*>(p.i) + at.b * p.T * p.ldi + c * sizeof(E);
  const int64_t ldh = p.C * sizeof(E);
  char* h = static_cast<char*>(p.h) + at.b * p.T * ldh + c * sizeof(E);
  int buf = 0;
  for (int64_t tile = begin; tile < end; tile += kTile, buf ^= 1) {
    const int64_t t0 = tile + wave * kSpan, left = end - t0;
    float a[kRun][V], b[kRun][V];
    Run own_run[V], before[V];
#pragma unroll
    for (int v = 0; v < V; ++v) own_run[v] = empty_run();
    if (left > 0) {
      uint32_t rx[kRun], rf[kRun], ri[kRun];
      load_run(rx, x + t0 * p.ldx, p.ldx, run, left);
      load_run(rf, f + t0 * p.ldf, p.ldf, run, left);
      if constexpr (IG) load_run(ri, g + t0 * p.ldi, p.ldi, run, left);
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
    join_lanes<V, false>(own_run, before, lane);
    float in[V];
    if constexpr (TOTALS) {
      // the whole segment's A and C: joined like a state's, from the same parts
      if (run == kRuns - 1) {
#pragma unroll
        for (int v = 0; v < V; ++v)
          part[buf][wave][(lane % kLanes) * V + v] = make_float4(own_run[v].A, own_run[v].C, own_run[v].H, 0.0f);
      }
      __syncthreads();
#pragma unroll
      for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
          const float4 t = part[buf][w][(lane % kLanes) * V + v];
          carry[v].pass({t.x, t.y, t.z});
          C_all[v] = fmaf(t.y, A_all[v], C_all[v]);
          A_all[v] *= t.x;
        }
      }
    } else {
      pass_waves<V, false>(part[buf], wave, lane, own_run, carry, in);
      if (left > 0) {
        if (p.marks != nullptr && run == 0 && own) {
          float* m = p.marks + (at.b * ((p.T + kSpan - 1) / kSpan) + t0 / kSpan) * p.C + c;
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
            const int row = run * kRun + r;
            if (own && row < left) store_parts<E>(h + (t0 + row) * ldh, y);
          }
        }
      }
    }
  }
  if constexpr (TOTALS) {
    if (wave == 0 && run == 0 && own) {
#pragma unroll
      for (int v = 0; v < V; ++v)
        p.totals[(at.b * (p.segs - 1) + at.seg) * p.C + c + v] = {A_all[v], C_all[v], carry[v].value()};
    }
  } else if (last && p.h_final != nullptr && wave == 0 && run == 0 && own) {
#pragma unroll
    for (int v = 0; v < V; ++v) p.h_final[at.b * p.C + c + v] = carry[v].value();
  }
}

// Gradients, from a sequence's end: with G_t = a_t (d_h_t + G_{t+1}) the same recurrence, whose
// value behind token t is l_t = d_h_t + G_{t+1}. h comes from the state before the span. TOTALS:
// only what each segment but the first makes of the gradient behind it.
template <typename E, int KIND, bool IG, bool TOTALS>
__global__ __launch_bounds__(64 * kWaves) void scan_bwd_kernel(Pass p) {
  constexpr int V = Shape<E>::V, N = Shape<E>::N;
  __shared__ float4 part[2][kWaves][N];
  Place at(p, TOTALS ? p.segs - 1 : p.segs);
  if (TOTALS) ++at.seg;
  const int lane = threadIdx.x % 64, run = lane / kLanes;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int64_t c_all = int64_t(at.slice) * N + (lane % kLanes) * V;
  const bool own = c_all < p.C;
  const int64_t c = own ? c_all : p.C - V;
  const int64_t n = tokens_of(p.lens, at.b, p.T);
  const int64_t begin = at.seg * p.seg;
  const int64_t stop = std::min(begin + p.seg, p.T), end = std::min(stop, n);
  const int64_t ldh = p.C * sizeof(E);
  char* dx = static_cast<char*>(p.dx) + at.b * p.T * ldh + c * sizeof(E);
  char* df = static_cast<char*>(p.df) + at.b * p.T * ldh + c * sizeof(E);
  char* di = static_cast<char*>(p.di) + at.b * p.T * ldh + c * sizeof(E);
  if constexpr (!TOTALS) {
    // rows behind the length: zero
    const float zero[V] = {};
    for (int64_t t = std::max(begin, n) + wave * kRuns + run; t < stop; t += kWaves * kRuns) {
      if (!own) break;
      store_parts<E>(dx + t * ldh, zero), store_parts<E>(df + t * ldh, zero);
      if constexpr (IG) store_parts<E>(di + t * ldh, zero);
    }
  }
  if (TOTALS && begin >= n) return;
  float decay[V], sum[V];
  State carry[V];
  float A_all[V], C_all[V];
  const int64_t segs_used = (n + p.seg - 1) / p.seg;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    decay[v] = KIND == GDN_SCAN_POWER ? p.decay[c + v] : 0.0f;
    carry[v] = {TOTALS || p.d_final == nullptr ? 0.0f : p.d_final[at.b * p.C + c + v], 0.0f};
    if constexpr (!TOTALS) {
      for (int64_t s = segs_used - 1; s > int64_t(at.seg); --s) carry[v].pass(p.totals[(at.b * (p.segs - 1) + s - 1) * p.C + c + v]);
    }
    A_all[v] = 1.0f, C_all[v] = 0.0f, sum[v] = 0.0f;
  }
  const char* x = static_cast<const char*>(p.x) + at.b * p.T * p.ldx + c * sizeof(E);
  const char* f = static_cast<const char*>(p.f) + at.b * p.T * p.ldf + c * sizeof(E);
  const char* g = static_cast<const char*>(p.i) + at.b * p.T * p.ldi + c * sizeof(E);
  const char* d = static_cast<const char*>(p.d_h) + at.b * p.T * ldh + c * sizeof(E);
  int buf = 0;
  const int64_t tiles = end > begin ? (end - begin + kTile - 1) / kTile : 0;
  for (int64_t tile = begin + (tiles - 1) * kTile; tile >= begin && tiles > 0; tile -= kTile, buf ^= 1) {
    const int64_t t0 = tile + wave * kSpan, left = end - t0;
    uint32_t rx[kRun], rf[kRun], ri[kRun], rd[kRun];
    float a[kRun][V], before[kRun][V];
    Run own_run[V], lanes[V];
#pragma unroll
    for (int v = 0; v < V; ++v) own_run[v] = empty_run();
    if (left > 0) {
      load_run(rf, f + t0 * p.ldf, p.ldf, run, left);
      load_run(rd, d + t0 * ldh, ldh, run, left);
      if constexpr (!TOTALS) {
        load_run(rx, x + t0 * p.ldx, p.ldx, run, left);
        if constexpr (IG) load_run(ri, g + t0 * p.ldi, p.ldi, run, left);
      }
      // G of the run, from its last token
#pragma unroll
      for (int r = kRun - 1; r >= 0; --r) {
        const bool here = run * kRun + r < left;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const Gate t = gate_of<E, KIND>(part_of<E>(rf[r], v), decay[v]);
          a[r][v] = here ? t.a : 1.0f;
          const float up = here ? part_of<E>(rd[r], v) : 0.0f;
          own_run[v] = join(own_run[v], Run{a[r][v], here ? t.c : 0.0f, a[r][v] * up});
          if constexpr (!TOTALS) {
            float add = t.m * part_of<E>(rx[r], v);
            if constexpr (IG) add *= sigmoid_of<E>(part_of<E>(ri[r], v));
            before[r][v] = here ? add : 0.0f;
          }
        }
      }
    }
    if constexpr (!TOTALS) {
      // h before each token: from what each adds
      Run fwd[V], ahead[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        fwd[v] = empty_run();
        if (left > 0) {
#pragma unroll
          for (int r = 0; r < kRun; ++r) fwd[v] = join(fwd[v], Run{a[r][v], 0.0f, before[r][v]});
        }
      }
      join_lanes<V, false>(fwd, ahead, lane);
      if (left > 0) {
        const float* m = p.marks + (at.b * ((p.T + kSpan - 1) / kSpan) + t0 / kSpan) * p.C + c;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          float y = fmaf(ahead[v].A, m[v], ahead[v].H);
#pragma unroll
          for (int r = 0; r < kRun; ++r) {
            const float add = before[r][v];
            before[r][v] = y;
            y = fmaf(a[r][v], y, add);
          }
        }
      }
    }
    join_lanes<V, true>(own_run, lanes, lane);
    float in[V];
    if constexpr (TOTALS) {
      if (run == 0) {
#pragma unroll
        for (int v = 0; v < V; ++v)
          part[buf][wave][(lane % kLanes) * V + v] = make_float4(own_run[v].A, own_run[v].C, own_run[v].H, 0.0f);
      }
      __syncthreads();
#pragma unroll
      for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int w = kWaves - 1; w >= 0; --w) {
          const float4 t = part[buf][w][(lane % kLanes) * V + v];
          carry[v].pass({t.x, t.y, t.z});
          C_all[v] = fmaf(t.y, A_all[v], C_all[v]);
          A_all[v] *= t.x;
        }
      }
    } else {
      pass_waves<V, true>(part[buf], wave, lane, own_run, carry, in);
      if (left > 0) {
        float G[V];
#pragma unroll
        for (int v = 0; v < V; ++v) G[v] = fmaf(lanes[v].A, in[v], lanes[v].H);
#pragma unroll
        for (int r = kRun - 1; r >= 0; --r) {
          float ox[V], of[V], oi[V];
          const int row = run * kRun + r;
          const bool here = row < left;
#pragma unroll
          for (int v = 0; v < V; ++v) {
            const Gate t = gate_of<E, KIND>(part_of<E>(rf[r], v), decay[v]);
            const float xv = part_of<E>(rx[r], v), l = part_of<E>(rd[r], v) + G[v];
            float s = 1.0f, rest = 0.0f;
            if constexpr (IG) sigmoids<E>(part_of<E>(ri[r], v), &s, &rest);
            const float lm = l * t.m;
            ox[v] = IG ? lm * s : lm;
            if constexpr (IG) oi[v] = ox[v] * xv * rest;
            const float gx = IG ? s * xv : xv;
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
          if (own && here) {
            store_parts<E>(dx + (t0 + row) * ldh, ox);
            store_parts<E>(df + (t0 + row) * ldh, of);
            if constexpr (IG) store_parts<E>(di + (t0 + row) * ldh, oi);
          }
        }
      }
    }
  }
  if constexpr (TOTALS) {
    if (wave == 0 && run == 0 && own) {
#pragma unroll
      for (int v = 0; v < V; ++v)
        p.totals[(at.b * (p.segs - 1) + at.seg - 1) * p.C + c + v] = {A_all[v], C_all[v], carry[v].value()};
    }
  } else {
    if (at.seg == 0 && p.dh0 != nullptr && wave == 0 && run == 0 && own) {
#pragma unroll
      for (int v = 0; v < V; ++v) p.dh0[at.b * p.C + c + v] = carry[v].value();
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
          p.ddecay[(at.b * p.segs + at.seg) * p.C + c + v] = t;
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
