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
// of what is left (8 bits a part, float32's range): bf16 inputs take the masked scores and
// the state in two parts (2^-16, under the output's rounding) and the weighted c of the state
// update in three (2^-24: the state is a float32 result); float32 inputs are three parts
// themselves, and of the nine products of parts the six above 2^-24 are formed. Six bf16
// products are 2.7 times as fast as the float32 MFMA here.
//
// One workgroup runs one segment of a head. Its waves share the chunk's tiles in LDS and
// split the DC columns of the state, whose slice a wave keeps in accumulators: an
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
};

// log of a head's decay; everything below e^-128 is taken as 0, -Inf included.
__device__ __forceinline__ float head_log_decay(const float* g, int h) {
  const float x = g[h];
  return x < -128.0f ? -128.0f : x;
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
constexpr int pass_waves(int DC) { return DC >= 64 ? 4 : DC / 16; }

// x[0..N) as PARTS sums of bf16: part[p][i].
template <int PARTS, int N>
__device__ __forceinline__ void split_parts(const float* x, vec<__bf16, N>* part) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float rest = x[i];
#pragma unroll
    for (int p = 0; p < PARTS; ++p) {
      part[p][i] = __bf16(rest);
      if (p + 1 < PARTS) rest -= float(part[p][i]);
    }
  }
}

__device__ __forceinline__ float4v mma(bhalf8 a, bhalf8 b, float4v acc) { return mma_pair_bf16(a, b, acc); }

// Sum of the products of parts, the smallest first; those of order above MOST are left out.
template <int PA, int PB, int MOST>
__device__ __forceinline__ float4v mma_parts(const bhalf8* a, const bhalf8* b, float4v acc) {
#pragma unroll
  for (int order = MOST; order >= 0; --order)
#pragma unroll
    for (int p = 0; p < PA; ++p)
      if (order - p >= 0 && order - p < PB) acc = mma(a[p], b[order - p], acc);
  return acc;
}

typedef __attribute__((address_space(3))) bhalf4 lds_bhalf4;
__device__ __forceinline__ bhalf4 read_tr(const __bf16* p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bhalf4*)(p));
}
__device__ __forceinline__ bhalf8 join(bhalf4 lo, bhalf4 hi) { return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7); }

// A tile of C rows of D channels: PARTS planes of rows padded by 16 bytes, so that sixteen
// rows start in sixteen different groups of banks.
template <int C, int D, int PARTS> struct Tile {
  static constexpr int kLd = D + 8;
  static constexpr int kPlane = C * kLd;
  __bf16 x[PARTS * kPlane];

  // rows 16 r + i, channels of k-block kb: the order of the state's accumulator tiles
  __device__ __forceinline__ bhalf8 row(int p, int r, int kb, int i, int g) const {
    const __bf16* at = x + p * kPlane + (16 * r + i) * kLd;
    if constexpr (D == 16) {
      const bhalf4 lo = *reinterpret_cast<const bhalf4*>(at + 4 * g);
      return join(lo, bhalf4{});
    } else {
      return *reinterpret_cast<const bhalf8*>(at + 32 * kb + 8 * g);
    }
  }
  // positions 32 kb + 8 g + e of channel `column` + (i % 4) + step (i / 4), read transposed
  __device__ __forceinline__ bhalf8 columns(int p, int kb, int column, int step, int i, int g) const {
    const __bf16* at = x + p * kPlane + (32 * kb + 8 * g + i / 4) * kLd + column + (i % 4) * step;
    return join(read_tr(at), read_tr(at + 4 * kLd));
  }
};

template <typename E, int DA, int DC, bool OUT> struct PassShared {
  using S = PassShape<E>;
  static constexpr int C = S::kChunk;
  Tile<C, DA, S::kParts> b;
  Tile<C, DC, S::kParts> c;
  Tile<OUT ? C : 1, DA, S::kParts> a;
  Tile<OUT ? C : 1, C, S::kScoreParts> scores;
  float end_weight[C];   // l^{n-1-j+shift}
  int bad_from[DC];      // first position of the chunk whose c is not finite, a channel
  int bad;
};

// Vectors of 16 bytes of a tile, held between their load and their store to LDS.
template <typename E, int C, int D, int NT> struct Staged {
  static constexpr int kPerRow = D * int(sizeof(E)) / 16;
  static constexpr int kCount = (C * kPerRow + NT - 1) / NT;
  uint4 v[kCount];
  __device__ __forceinline__ void load(const E* base, int64_t step, int rows) {
#pragma unroll
    for (int n = 0; n < kCount; ++n) {
      const int at = threadIdx.x + n * NT, row = at / kPerRow, col = at % kPerRow;
      v[n] = row < rows ? *reinterpret_cast<const uint4*>(base + row * step + col * (16 / sizeof(E))) : uint4{0, 0, 0, 0};
    }
  }
  template <int PARTS>
  __device__ __forceinline__ void store(Tile<C, D, PARTS>& t) const {
#pragma unroll
    for (int n = 0; n < kCount; ++n) {
      const int at = threadIdx.x + n * NT, row = at / kPerRow, col = at % kPerRow;
      if (C * kPerRow % NT != 0 && row >= C) break;
      if constexpr (sizeof(E) == 2) {
        *reinterpret_cast<uint4*>(t.x + row * t.kLd + col * 8) = v[n];
      } else {
        const float f[4] = {__uint_as_float(v[n].x), __uint_as_float(v[n].y), __uint_as_float(v[n].z), __uint_as_float(v[n].w)};
        bhalf4 part[PARTS];
        split_parts<PARTS, 4>(f, part);
#pragma unroll
        for (int p = 0; p < PARTS; ++p) *reinterpret_cast<bhalf4*>(t.x + p * t.kPlane + row * t.kLd + col * 4) = part[p];
      }
    }
  }
  // Marks channels with a NaN or Inf: a masked score is 0, but 0 times Inf is not.
  __device__ __forceinline__ void mark_bad(int* bad, int* bad_from) const {
    constexpr uint32_t kExp = sizeof(E) == 2 ? 0x7f807f80u : 0x7f800000u, kOne = sizeof(E) == 2 ? 0x00800080u : 0x00800000u,
                       kTop = sizeof(E) == 2 ? 0x80008000u : 0x80000000u;
#pragma unroll
    for (int n = 0; n < kCount; ++n) {
      const uint32_t w[4] = {v[n].x, v[n].y, v[n].z, v[n].w};
      const uint32_t any = (((w[0] & kExp) + kOne) | ((w[1] & kExp) + kOne) | ((w[2] & kExp) + kOne) | ((w[3] & kExp) + kOne)) & kTop;
      if (any == 0) continue;
      const int at = threadIdx.x + n * NT, row = at / kPerRow, col = at % kPerRow;
      *bad = 1;
      for (int e = 0; e < int(16 / sizeof(E)); ++e) {
        const uint32_t x = sizeof(E) == 2 ? w[e / 2] >> (16 * (e % 2)) & 0x7f80u : w[e] >> 16 & 0x7f80u;
        if (x == 0x7f80u) atomicMin(&bad_from[col * int(16 / sizeof(E)) + e], row);
      }
    }
  }
};

// OUT: outputs, from the state before the segment. Otherwise the states after the segments
// 0 .. nseg-2, each from zero (the first from x0), for scan_states to join.
template <typename E, typename O, int DA, int DC, bool REV, bool OUT>
__global__ __launch_bounds__(64 * pass_waves(DC)) void linear_pass_kernel(LinearPass s) {
  using S = PassShape<E>;
  constexpr int C = S::kChunk, NW = pass_waves(DC), NT = 64 * NW;
  constexpr int P = S::kParts, PS = S::kScoreParts;
  constexpr int RT = C / 16;          // row tiles of a chunk
  constexpr int KT = DA / 16;         // state tiles along DA
  constexpr int KB = (DA + 31) / 32;  // k-blocks along DA
  constexpr int CT = DC / 16 / NW;    // state tiles of a wave along DC
  constexpr int PB = C / 32;          // k-blocks of positions
  constexpr int kColStep = CT == 2 ? 8 : 4;  // channels between a wave's runs of four columns
  __shared__ PassShared<E, DA, DC, OUT> sh;

  const int wave = threadIdx.x / 64, lane = threadIdx.x % 64, i = lane % 16, g = lane / 16;
  const int h = int(blockIdx.x) % s.H;
  const int64_t bs = int64_t(blockIdx.x) / s.H;
  const int segs = OUT ? s.nseg : s.nseg - 1;
  const int seg = int(bs % segs);
  const int64_t b = bs / segs;
  const int64_t bh = b * s.H + h;
  const int64_t n = length_of(s.seq_lens, b, s.T);
  const float lg = head_log_decay(s.log_decay, h) * 1.44269504088896341f;  // log2
  auto power = [&](int m) { return __builtin_amdgcn_exp2f(lg * float(m)); };

  const int64_t begin = seg * s.seg;
  const int64_t last = begin + s.seg < s.T ? begin + s.seg : s.T;   // positions of the segment, real or not
  const int64_t end = last < n ? last : n;
  constexpr int kDir = REV ? -1 : 1;
  // rows of position p: token p, or n - 1 - p backwards
  auto rows = [&](const void* x, int64_t ld, int group, int d, int64_t p) {
    return static_cast<const E*>(x) + (b * s.T + (REV ? n - 1 - p : p)) * ld + int64_t(h / group) * d;
  };
  // channel of the state's row e of tile kt, and of its column of tile ct
  auto row_channel = [&](int kt) { return KT == 1 ? 4 * g : 32 * (kt / 2) + 8 * g + 4 * (kt % 2); };
  auto col_channel = [&](int ct) { return 16 * CT * wave + kColStep * (i / 4) + 4 * ct + i % 4; };

  // the state of the wave's columns
  float4v X[KT][CT];
  // The outputs' pass takes x0 from slot 0 where there are several segments: x1 may be x0
  // itself, and the last segment's workgroup may end before the first one's begins.
  float* slots = s.states + bh * s.nseg * (DA * DC);
  const bool given = seg > 0 ? OUT : s.x0 != nullptr;
  const bool direct = seg == 0 && (!OUT || s.nseg == 1);
  const float* from = !given ? nullptr : direct ? s.x0 + bh * (DA * DC) : slots + seg * (DA * DC);
  const int64_t sa = direct ? s.x0_sa : s.st_sa, sc = direct ? s.x0_sc : s.st_sc;
#pragma unroll
  for (int kt = 0; kt < KT; ++kt)
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
      if (from == nullptr) {
        X[kt][ct] = float4v{0.0f, 0.0f, 0.0f, 0.0f};
      } else if (sa == 1) {
        X[kt][ct] = *reinterpret_cast<const float4v*>(from + row_channel(kt) + col_channel(ct) * sc);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) X[kt][ct][e] = from[(row_channel(kt) + e) * sa + col_channel(ct) * sc];
      }
    }

  auto store_state = [&](float* to, int64_t ta, int64_t tc) {
    if (to == nullptr) return;
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) {
        if (ta == 1) {
          *reinterpret_cast<float4v*>(to + row_channel(kt) + col_channel(ct) * tc) = X[kt][ct];
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) to[(row_channel(kt) + e) * ta + col_channel(ct) * tc] = X[kt][ct][e];
        }
      }
  };
  if (!OUT && seg == 0 && given) store_state(slots, s.st_sa, s.st_sc);

  Staged<E, C, DA, NT> ra, rb;
  Staged<E, C, DC, NT> rc;
  auto fetch = [&](int64_t p) {
    const int m = int(end - p < C ? end - p : C);
    if constexpr (OUT) ra.load(rows(s.a, s.lda, s.group_a, DA, p), kDir * s.lda, m);
    rb.load(rows(s.b, s.ldb, s.group_b, DA, p), kDir * s.ldb, m);
    rc.load(rows(s.c, s.ldc, s.group_c, DC, p), kDir * s.ldc, m);
  };
  if (begin < end) fetch(begin);
  if constexpr (OUT) {
    for (int at = threadIdx.x; at < DC; at += NT) sh.bad_from[at] = C;
    if (threadIdx.x == 0) sh.bad = 0;
    __syncthreads();
  }

  for (int64_t p = begin; p < end; p += C) {
    const int m = int(end - p < C ? end - p : C);  // positions of the chunk
    if constexpr (OUT) {
      ra.store(sh.a);
      rc.mark_bad(&sh.bad, sh.bad_from);
    }
    rb.store(sh.b);
    rc.store(sh.c);
    if (threadIdx.x < C) {
      const int left = m - 1 - int(threadIdx.x);
      sh.end_weight[threadIdx.x] = left >= 0 ? power(left + s.shift) : 0.0f;
    }
    __syncthreads();
    if (p + C < end) fetch(p + C);

    float4v acc[OUT ? RT : 1][CT];
    if constexpr (OUT) {
      // scores, transposed: column i of a tile is position 16 r + i, its rows positions 16 jt + 4 g + e
      for (int r = wave; r < RT; r += NW) {
        bhalf8 av[KB][P];
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
          for (int q = 0; q < P; ++q) av[kb][q] = sh.a.row(q, r, kb, i, g);
#pragma unroll
        for (int jt = 0; jt < RT; ++jt) {
          if (jt > (r | 1)) continue;
          float x[4] = {};
          if (jt <= r) {
            float4v t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) {
              bhalf8 bv[P];
#pragma unroll
              for (int q = 0; q < P; ++q) bv[q] = sh.b.row(q, jt, kb, i, g);
              t = mma_parts<P, P, P - 1>(bv, av[kb], t);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int ahead = 16 * r + i - (16 * jt + 4 * g + e);
              x[e] = ahead >= 0 ? t[e] * power(ahead) : 0.0f;
            }
          }
          bhalf4 part[PS];
          split_parts<PS, 4>(x, part);
#pragma unroll
          for (int q = 0; q < PS; ++q)
            *reinterpret_cast<bhalf4*>(sh.scores.x + q * sh.scores.kPlane + (16 * r + i) * sh.scores.kLd + 16 * jt + 4 * g) = part[q];
        }
      }
      // what the state before the chunk gives
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) acc[r][ct] = float4v{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
        bhalf8 xv[CT][PS];
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
          float x[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            x[e] = X[2 * kb][ct][e];
            x[4 + e] = KT > 1 ? X[KT > 1 ? 2 * kb + 1 : 0][ct][e] : 0.0f;
          }
          split_parts<PS, 8>(x, xv[ct]);
        }
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          bhalf8 av[P];
#pragma unroll
          for (int q = 0; q < P; ++q) av[q] = sh.a.row(q, r, kb, i, g);
#pragma unroll
          for (int ct = 0; ct < CT; ++ct) acc[r][ct] = mma_parts<PS, P, PS - 1>(xv[ct], av, acc[r][ct]);
        }
      }
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const float w = power(16 * r + i + 1 - s.shift);
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) acc[r][ct] *= w;
      }
      __syncthreads();
    }

    // what the chunk's own rows give, and the state after it
    const int bad = OUT ? sh.bad : 0;
    const float whole = power(m);
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) X[kt][ct] *= whole;
#pragma unroll
    for (int kb = 0; kb < PB; ++kb) {
      bhalf8 wv[CT][3];
      float w[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = sh.end_weight[32 * kb + 8 * g + e];
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) {
        bhalf8 cv[P];
        float x[8] = {};
#pragma unroll
        for (int q = 0; q < P; ++q) {
          cv[q] = sh.c.columns(q, kb, 16 * CT * wave + 4 * ct, kColStep, i, g);
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] += float(cv[q][e]);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= w[e];
        split_parts<3, 8>(x, wv[ct]);
        if constexpr (OUT) {
          if (bad) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if ((__builtin_bit_cast(uint16_t, (__bf16)cv[0][e]) & 0x7f80u) == 0x7f80u)
#pragma unroll
                for (int q = 0; q < P; ++q) cv[q][e] = __bf16(0.0f);
          }
#pragma unroll
          for (int r = 2 * kb; r < RT; ++r) {
            bhalf8 sv[PS];
#pragma unroll
            for (int q = 0; q < PS; ++q) sv[q] = sh.scores.row(q, r, kb, i, g);
            acc[r][ct] = mma_parts<P, PS, PS - 1>(cv, sv, acc[r][ct]);
          }
        }
      }
#pragma unroll
      for (int kt = 0; kt < KT; ++kt) {
        bhalf8 bv[P];
#pragma unroll
        for (int q = 0; q < P; ++q)
          bv[q] = sh.b.columns(q, kb, KT == 1 ? 0 : 32 * (kt / 2) + 4 * (kt % 2), KT == 1 ? 4 : 8, i, g);
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) X[kt][ct] = mma_parts<P, 3, 2>(bv, wv[ct], X[kt][ct]);
      }
    }

    if constexpr (OUT) {
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const int at = 16 * r + i;
        if (at < m) {
          const int64_t token = b * s.T + (REV ? n - 1 - p - at : p + at);
          const int ch = 16 * CT * wave + 4 * CT * g;
          float x[4 * CT];
#pragma unroll
          for (int ct = 0; ct < CT; ++ct)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              x[4 * ct + e] = acc[r][ct][e];
              if (bad && at >= sh.bad_from[ch + 4 * ct + e]) x[4 * ct + e] = __builtin_nanf("");
            }
          vec<O, 4 * CT> out;
#pragma unroll
          for (int e = 0; e < 4 * CT; ++e) out[e] = O(x[e]);
          *reinterpret_cast<vec<O, 4 * CT>*>(static_cast<O*>(s.out) + (token * s.H + h) * DC + ch) = out;
        }
      }
    }
    __syncthreads();
    if constexpr (OUT) {
      if (bad) {
        for (int at = threadIdx.x; at < DC; at += NT) sh.bad_from[at] = C;
        if (threadIdx.x == 0) sh.bad = 0;
        __syncthreads();
      }
    }
  }

  if constexpr (OUT) {
    if (s.zero_tail) {
      const int64_t first = begin > n ? begin : n;
      constexpr int V = DC / 4;
      for (int64_t at = threadIdx.x; at < (last - first) * V; at += NT) {
        const float zero[4] = {};
        store4(static_cast<O*>(s.out) + ((b * s.T + first + at / V) * s.H + h) * DC + at % V * 4, zero);
      }
    }
  }

  if (OUT && seg < s.nseg - 1) return;
  store_state(OUT ? (s.x1 == nullptr ? nullptr : s.x1 + bh * (DA * DC)) : slots + (seg + 1) * (DA * DC),
              OUT ? s.x0_sa : s.st_sa, OUT ? s.x0_sc : s.st_sc);
}

// Launches of one direction and type, in the translation units of each element type.
int launch_pass_bf16(const LinearPass& s, int64_t B, int da, int dc, bool rev, bool out, bool wide_out, void* stream);
int launch_pass_f32(const LinearPass& s, int64_t B, int da, int dc, bool rev, bool out, void* stream);

template <typename E, typename O, int DA, int DC>
int launch_pass_dims(const LinearPass& s, int64_t B, bool rev, bool out, hipStream_t stream) {
  constexpr int kThreads = 64 * pass_waves(DC);
  const unsigned grid = unsigned(B * s.H * (out ? s.nseg : s.nseg - 1));
  if (rev) {
    if (out) linear_pass_kernel<E, O, DA, DC, true, true><<<grid, kThreads, 0, stream>>>(s);
    else linear_pass_kernel<E, E, DA, DC, true, false><<<grid, kThreads, 0, stream>>>(s);
  } else {
    if (out) linear_pass_kernel<E, O, DA, DC, false, true><<<grid, kThreads, 0, stream>>>(s);
    else linear_pass_kernel<E, E, DA, DC, false, false><<<grid, kThreads, 0, stream>>>(s);
  }
  return int(hipGetLastError());
}

template <typename E, typename O>
int launch_pass_any(const LinearPass& s, int64_t B, int da, int dc, bool rev, bool out, hipStream_t stream) {
  switch (da * 1000 + dc) {
#define GDN_PASS(DA, DC) case DA * 1000 + DC: return launch_pass_dims<E, O, DA, DC>(s, B, rev, out, stream);
    GDN_PASS(16, 16) GDN_PASS(16, 32) GDN_PASS(16, 64) GDN_PASS(16, 128)
    GDN_PASS(32, 16) GDN_PASS(32, 32) GDN_PASS(32, 64) GDN_PASS(32, 128)
    GDN_PASS(64, 16) GDN_PASS(64, 32) GDN_PASS(64, 64) GDN_PASS(64, 128)
    GDN_PASS(128, 16) GDN_PASS(128, 32) GDN_PASS(128, 64) GDN_PASS(128, 128)
#undef GDN_PASS
    default: return int(hipErrorInvalidValue);
  }
}

}  // namespace gdn
