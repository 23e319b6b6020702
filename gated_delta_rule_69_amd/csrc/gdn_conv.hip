// Short causal convolution a channel, forward and backward:
//     z_t = bias + sum_j w_j x_{t - W + 1 + j},   y = silu(z) or z
//
// A thread has neighbouring channels (sixteen bytes; four channels in the gradients) and a run of
// tokens, and keeps the last W - 1 rows in registers: every row is read once, but for the W - 1 before
// a run. A workgroup is 32 such threads across the channels and eight runs. Memory bounds it.
//
// bf16, four taps: 32,768 tokens of 6,144 channels 165 us (805 MB, 4.9 TB/s; a copy of 512 MiB reaches
// 5.25), float32 8,192 x 2,048 26 us; one token of 512 sequences 11 us (50 MB); the
// gradients of 8,192 x 6,144 71 us, 4 of them the weights' sums in a second kernel (4.1 TB/s: 160 registers,
// three waves a SIMD, whose vector instructions take two thirds of the issue slots).
#include <algorithm>

#include "gdn_block.h"
#include "gdn_block_device.h"

namespace gdn {
namespace {

constexpr int kAcross = 32, kDown = 8, kThreads = kAcross * kDown;
constexpr int kStep = 4;   // rows whose loads are under way together
constexpr int kBackChannels = 4;   // channels a thread in the gradients: eight would take 210 registers, two waves a SIMD

struct Conv {
  const void* x;
  const float *w, *bias;
  const int32_t* lens;
  const void* s0;
  void *s_final, *y;
  int64_t T, C, ldx;      // ldx in elements
  int64_t run;            // tokens a run
  unsigned columns, runs, blocks;   // workgroups across the channels, and down a sequence
  // gradients
  const void *d_y, *d_s;
  void *dx, *ds0;
  float* partial;         // [B * runs][C * W + C]
};

template <typename E, int N>
__device__ __forceinline__ void unpack(const vec<E, N>& r, float* x) {
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = float(r[i]);
}
template <typename E, int N>
__device__ __forceinline__ void store_row(E* p, const float* x) {
  vec<E, N> r;
#pragma unroll
  for (int i = 0; i < N; ++i) r[i] = E(x[i]);
  *reinterpret_cast<vec<E, N>*>(p) = r;
}

// Row t of what the convolution reads: x, or the state's rows before token 0 (or zero).
template <typename E, int W, int N>
__device__ __forceinline__ vec<E, N> input_row(const Conv& a, int64_t b, int64_t t, int64_t c) {
  vec<E, N> r = {};
  if (t >= 0) return *reinterpret_cast<const vec<E, N>*>(static_cast<const E*>(a.x) + (b * a.T + t) * a.ldx + c);
  if (a.s0 != nullptr) r = *reinterpret_cast<const vec<E, N>*>(static_cast<const E*>(a.s0) + (b * (W - 1) + t + W - 1) * a.C + c);
  return r;
}

template <int W, int N>
__device__ __forceinline__ void load_weights(const Conv& a, int64_t c, float (*w)[N], float* bias) {
  float flat[N * W];
#pragma unroll
  for (int i = 0; i < N * W; i += 4) load4(a.w + c * W + i, flat + i);
#pragma unroll
  for (int i = 0; i < N; ++i) {
#pragma unroll
    for (int j = 0; j < W; ++j) w[j][i] = flat[i * W + j];
    bias[i] = 0.0f;
  }
  if (a.bias != nullptr) {
#pragma unroll
    for (int i = 0; i < N; i += 4) load4(a.bias + c + i, bias + i);
  }
}

template <typename E, int W, bool SILU>
__global__ __launch_bounds__(kThreads) void conv_kernel(Conv a) {
  constexpr int N = 16 / sizeof(E);
  typedef vec<E, N> Row;
  const unsigned col = blockIdx.x % a.columns, q = blockIdx.x / a.columns;
  const unsigned down = q % a.runs;
  const int64_t b = q / a.runs;
  const int64_t c = (int64_t(col) * kAcross + threadIdx.x % kAcross) * N;
  if (c >= a.C) return;
  const int64_t n = tokens_of(a.lens, b, a.T);
  const int64_t r = int64_t(down) * kDown + threadIdx.x / kAcross;
  const int64_t begin = r * a.run, end = std::min(begin + a.run, n);
  if (begin >= end && r > 0) return;
  float w[W][N], bias[N], past[W - 1][N];
  load_weights<W, N>(a, c, w, bias);
  Row before[W - 1];
#pragma unroll
  for (int j = 0; j < W - 1; ++j) {
    before[j] = input_row<E, W, N>(a, b, begin - (W - 1) + j, c);
    unpack<E, N>(before[j], past[j]);
  }
  if (r == 0 && a.s_final != nullptr) {
    // the last W - 1 inputs; s_final may be s0, whose rows are here already
    Row left[W - 1];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      const int64_t t = n - (W - 1) + j;
      if (t >= 0) {
        left[j] = input_row<E, W, N>(a, b, t, c);
      } else {
#pragma unroll
        for (int k = 0; k < W - 1; ++k)
          if (k == t + W - 1) left[j] = before[k];
      }
    }
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
      *reinterpret_cast<Row*>(static_cast<E*>(a.s_final) + (b * (W - 1) + j) * a.C + c) = left[j];
  }
  const E* x = static_cast<const E*>(a.x) + b * a.T * a.ldx + c;
  E* y = static_cast<E*>(a.y) + b * a.T * a.C + c;
  for (int64_t t = begin; t < end; t += kStep) {
    Row rows[kStep];
#pragma unroll
    for (int k = 0; k < kStep; ++k) rows[k] = *reinterpret_cast<const Row*>(x + std::min(t + k, end - 1) * a.ldx);
#pragma unroll
    for (int k = 0; k < kStep; ++k) {
      float now[N], out[N];
      unpack<E, N>(rows[k], now);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        float z = bias[i];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) z = fmaf(w[j][i], past[j][i], z);
        z = fmaf(w[W - 1][i], now[i], z);
        out[i] = SILU ? z * sigmoid_of<E>(z) : z;
#pragma unroll
        for (int j = 0; j + 1 < W - 1; ++j) past[j][i] = past[j + 1][i];
        past[W - 2][i] = now[i];
      }
      if (t + k < end) store_row<E, N>(y + (t + k) * a.C, out);
    }
  }
}

// A few tokens a sequence: G sequences a thread, so that the weights (16 bytes a channel of four
// taps, as much as a token's rows) are read once for them, and their rows are under way together.
template <typename E, int W, bool SILU, int G>
__global__ __launch_bounds__(kThreads) void conv_step_kernel(Conv a, int64_t B) {
  constexpr int N = 16 / sizeof(E);
  typedef vec<E, N> Row;
  const unsigned col = blockIdx.x % a.columns, q = blockIdx.x / a.columns;
  const int64_t c = (int64_t(col) * kAcross + threadIdx.x % kAcross) * N;
  if (c >= a.C) return;
  const int64_t first = (int64_t(q) * kDown + threadIdx.x / kAcross) * G;
  float w[W][N], bias[N];
  load_weights<W, N>(a, c, w, bias);
  Row past[G][W - 1], now[G];
  int64_t n[G];
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int64_t b = first + g;
    n[g] = b < B ? tokens_of(a.lens, b, a.T) : 0;
    now[g] = Row{};
#pragma unroll
    for (int j = 0; j < W - 1; ++j) past[g][j] = Row{};
    if (b >= B) continue;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) past[g][j] = input_row<E, W, N>(a, b, j - (W - 1), c);
    if (n[g] > 0) now[g] = input_row<E, W, N>(a, b, 0, c);
  }
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int64_t b = first + g;
    for (int64_t t = 0; t < n[g]; ++t) {
      if (t > 0) now[g] = input_row<E, W, N>(a, b, t, c);
      float out[N];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        float z = bias[i];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) z = fmaf(w[j][i], float(past[g][j][i]), z);
        z = fmaf(w[W - 1][i], float(now[g][i]), z);
        out[i] = SILU ? z * sigmoid_of<E>(z) : z;
      }
      store_row<E, N>(static_cast<E*>(a.y) + (b * a.T + t) * a.C + c, out);
#pragma unroll
      for (int j = 0; j + 1 < W - 1; ++j) past[g][j] = past[g][j + 1];
      past[g][W - 2] = now[g];
    }
    if (b < B && a.s_final != nullptr && (n[g] > 0 || a.s_final != a.s0)) {
#pragma unroll
      for (int j = 0; j < W - 1; ++j)
        *reinterpret_cast<Row*>(static_cast<E*>(a.s_final) + (b * (W - 1) + j) * a.C + c) = past[g][j];
    }
  }
}

// Gradients: dz_t = d_y_t act'(z_t), dx_t = sum_j w_j dz_{t + W - 1 - j}, dw_j = sum_t dz_t
// x_{t - W + 1 + j}. A run forms the dz of its own tokens and of the W - 1 behind it; those of
// its own go into the workgroup's sums for the weights.
template <typename E, int W, bool SILU>
__global__ __launch_bounds__(kThreads) void conv_bwd_kernel(Conv a) {
  constexpr int N = kBackChannels;
  typedef vec<E, N> Row;
  const unsigned col = blockIdx.x % a.columns, q = blockIdx.x / a.columns;
  const unsigned down = q % a.runs;
  const int64_t b = q / a.runs;
  const int64_t c = (int64_t(col) * kAcross + threadIdx.x % kAcross) * N;
  const bool own = c < a.C;
  const int64_t n = tokens_of(a.lens, b, a.T);
  const int64_t r = int64_t(down) * kDown + threadIdx.x / kAcross;
  const int64_t begin = r * a.run, stop = std::min(begin + a.run, a.T);
  float sums[W + 1][N] = {};
  if (own && (begin < stop || r == 0)) {
    float w[W][N], bias[N], past[W - 1][N], dz[W - 1][N] = {};
    load_weights<W, N>(a, c, w, bias);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      Row row = {};
      if (begin - (W - 1) + j < n) row = input_row<E, W, N>(a, b, begin - (W - 1) + j, c);
      unpack<E, N>(row, past[j]);
    }
    const E* x = static_cast<const E*>(a.x) + b * a.T * a.ldx + c;
    const E* dy = static_cast<const E*>(a.d_y) + b * a.T * a.C + c;
    E* dx = static_cast<E*>(a.dx) + b * a.T * a.C + c;
    const int64_t mine = std::min(stop, n);   // tokens from here on are another run's, or none
    // INSIDE: kStep tokens of the run's own whose rows' gradients are the run's too
    auto step = [&](auto inside, int64_t t) {
      constexpr bool INSIDE = decltype(inside)::value;
      Row rx[kStep], rd[kStep];
#pragma unroll
      for (int k = 0; k < kStep; ++k) {
        rx[k] = rd[k] = Row{};
        if (INSIDE || n > 0) {
          const int64_t at = INSIDE ? t + k : std::min(t + k, n - 1);
          rx[k] = *reinterpret_cast<const Row*>(x + at * a.ldx);
          rd[k] = *reinterpret_cast<const Row*>(dy + at * a.C);
        }
      }
#pragma unroll
      for (int k = 0; k < kStep; ++k) {
        const int64_t here = t + k, to = here - (W - 1);   // token, and the row whose gradient ends with it
        float now[N], g[N], out[N];
        unpack<E, N>(rx[k], now);
        unpack<E, N>(rd[k], g);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          if constexpr (SILU) {
            float z = bias[i], s, rest;
#pragma unroll
            for (int j = 0; j < W - 1; ++j) z = fmaf(w[j][i], past[j][i], z);
            z = fmaf(w[W - 1][i], now[i], z);
            sigmoids<E>(z, &s, &rest);
            g[i] *= s * (1.0f + z * rest);
          }
          if (!INSIDE) g[i] = here < n ? g[i] : 0.0f;
          if (INSIDE || here < mine) {
#pragma unroll
            for (int j = 0; j < W - 1; ++j) sums[j][i] = fmaf(g[i], past[j][i], sums[j][i]);
            sums[W - 1][i] = fmaf(g[i], now[i], sums[W - 1][i]);
            sums[W][i] += g[i];
          }
          // row `to` is read by tokens to .. to + W - 1 through w[W - 1] .. w[0]
          float d = w[0][i] * g[i];
#pragma unroll
          for (int j = 0; j < W - 1; ++j) d = fmaf(w[W - 1 - j][i], dz[j][i], d);
          out[i] = d;
#pragma unroll
          for (int j = 0; j + 1 < W - 1; ++j) past[j][i] = past[j + 1][i], dz[j][i] = dz[j + 1][i];
          past[W - 2][i] = now[i], dz[W - 2][i] = g[i];
        }
        if constexpr (INSIDE) {
          store_row<E, N>(dx + to * a.C, out);
        } else {
          if (to >= stop || (to < begin && r > 0)) continue;
          // the final state's rows are inputs n - W + 1 .. n - 1
          const int64_t j = to - (n - (W - 1));
          if (a.d_s != nullptr && j >= 0 && j < W - 1) {
            float up[N];
            unpack<E, N>(*reinterpret_cast<const Row*>(static_cast<const E*>(a.d_s) + (b * (W - 1) + j) * a.C + c), up);
#pragma unroll
            for (int i = 0; i < N; ++i) out[i] += up[i];
          }
          if (to >= n) {
#pragma unroll
            for (int i = 0; i < N; ++i) out[i] = 0.0f;
          }
          if (to >= 0)
            store_row<E, N>(dx + to * a.C, out);
          else if (a.ds0 != nullptr && to >= -(W - 1))
            store_row<E, N>(static_cast<E*>(a.ds0) + (b * (W - 1) + to + W - 1) * a.C + c, out);
        }
      }
    };
    // the final state's gradient meets rows from n - W + 1 on, with tokens n and behind
    int64_t t = begin;
    step(std::false_type{}, t);
    for (t += kStep; t + kStep <= mine; t += kStep) step(std::true_type{}, t);
    for (; t < stop + W - 1; t += kStep) step(std::false_type{}, t);
  }
  if (a.partial == nullptr) return;
  // over the workgroup's runs, in order
  __shared__ float part[kDown][kAcross][N];
  float* to = a.partial + (b * a.runs + down) * (a.C * (W + 1));
#pragma unroll
  for (int j = 0; j <= W; ++j) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) part[threadIdx.x / kAcross][threadIdx.x % kAcross][i] = sums[j][i];
    __syncthreads();
    for (int e = threadIdx.x; e < kAcross * N; e += kThreads) {
      const int64_t channel = int64_t(col) * kAcross * N + e;
      float s = 0.0f;
      for (int d = 0; d < kDown; ++d) s += part[d][e / N][e % N];
      if (channel < a.C) to[j < W ? channel * W + j : a.C * W + channel] = s;
    }
  }
}

int64_t columns_of(const gdn_conv_args& a, bool back) {
  const int64_t channels = kAcross * (back || a.dtype == GDN_DTYPE_F32 ? 4 : 8);
  return (a.C + channels - 1) / channels;
}
int64_t runs_of(const gdn_conv_args& a, int64_t run) { return std::max<int64_t>(1, (a.T + run * kDown - 1) / (run * kDown)); }
// Tokens a run: long ones read fewer rows twice (the gradients of B2 T4096 C6144 73 us at 64, 74 at 32, 73
// at 128), short ones give every CU its threads. A launch has fewer than 2^32 threads (B * C <= 2^24 keeps
// the workgroups of one run each under 2^22).
int64_t run_of(const gdn_conv_args& a, bool back) {
  int64_t run = back ? 64 : 32;
  while (run > 8 && a.B * columns_of(a, back) * runs_of(a, run) < (back ? 768 : 1024)) run /= 2;
  while (a.B * columns_of(a, back) * runs_of(a, run) > 1 << 22 && runs_of(a, run) > 1) run *= 2;
  return run;
}

// Few tokens go one by one, more of them where the sequences alone fill the CUs (C 6144, bf16, against
// runs: one sequence of 8 tokens 6.1 and 5.9 us, of 16 8.9 and 5.4; 64 sequences of 32 20.1 and 20.6, of 64
// 36 and 23; 512 sequences of 32 97 and 120).
int64_t few_tokens(const gdn_conv_args& a) { return a.B * columns_of(a, false) >= 1024 ? 32 : kConvInPlace; }

Conv conv_of(const gdn_conv_args& a, bool back) {
  Conv k{};
  k.x = a.x, k.w = a.w, k.bias = a.bias, k.lens = a.seq_lens, k.y = a.y;
  k.T = a.T, k.C = a.C, k.ldx = a.x_stride;
  k.run = run_of(a, back);
  k.columns = unsigned(columns_of(a, back));
  k.runs = unsigned(runs_of(a, k.run));
  k.blocks = unsigned(a.B * k.columns * k.runs);
  return k;
}

template <typename F>
int by_width(const gdn_conv_args& a, F f) {
  auto with = [&](auto type) {
    auto silu = [&](auto width) {
      return a.activation == GDN_ACT_SILU ? f(type, width, std::true_type{}) : f(type, width, std::false_type{});
    };
    switch (a.W) {
      case 2: return silu(std::integral_constant<int, 2>{});
      case 3: return silu(std::integral_constant<int, 3>{});
      default: return silu(std::integral_constant<int, 4>{});
    }
  };
  return a.dtype == GDN_DTYPE_BF16 ? with(__bf16{}) : with(float{});
}

}  // namespace

int launch_conv_fwd(const ConvProblem& p, const void* s0, void* s_final, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  Conv k = conv_of(p.a, false);
  k.s0 = s0, k.s_final = s_final;
  if (p.a.T <= few_tokens(p.a)) {
    const int64_t B = p.a.B;
    return by_width(p.a, [&](auto type, auto width, auto silu) {
      typedef decltype(type) E;
      constexpr int W = decltype(width)::value;
      constexpr bool S = decltype(silu)::value;
      // two sequences a thread where that leaves every CU two workgroups (C 6144, bf16: 512 sequences 11.1
      // us against 13.4 with one, 8 sequences 4.4 against 3.7; four take 11.8 and 5.9)
      const int64_t two = (B + 2 * kDown - 1) / (2 * kDown) * k.columns;
      if (two >= 512)
        conv_step_kernel<E, W, S, 2><<<unsigned(two), kThreads, 0, s>>>(k, B);
      else
        conv_step_kernel<E, W, S, 1><<<unsigned((B + kDown - 1) / kDown * k.columns), kThreads, 0, s>>>(k, B);
      return int(hipGetLastError());
    });
  }
  return by_width(p.a, [&](auto type, auto width, auto silu) {
    conv_kernel<decltype(type), decltype(width)::value, decltype(silu)::value><<<k.blocks, kThreads, 0, s>>>(k);
    return int(hipGetLastError());
  });
}

size_t conv_bwd_workspace(const ConvProblem& p) {
  return std::max<size_t>(256, size_t(p.a.B) * runs_of(p.a, run_of(p.a, true)) * p.a.C * (p.a.W + 1) * sizeof(float));
}

int launch_conv_bwd(const ConvProblem& p, const void* d_y, const void* d_s_final, const gdn_conv_grads& g, void* ws,
                    void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  Conv k = conv_of(p.a, true);
  k.s0 = p.a.s0, k.d_y = d_y, k.d_s = d_s_final, k.dx = g.dx, k.ds0 = g.ds0;
  const bool sums = g.dw != nullptr || g.dbias != nullptr;
  k.partial = sums ? static_cast<float*>(ws) : nullptr;
  const int rc = by_width(p.a, [&](auto type, auto width, auto silu) {
    conv_bwd_kernel<decltype(type), decltype(width)::value, decltype(silu)::value><<<k.blocks, kThreads, 0, s>>>(k);
    return int(hipGetLastError());
  });
  if (rc != 0 || !sums) return rc;
  return launch_column_sum({k.partial, int(p.a.B * k.runs), p.a.C * (p.a.W + 1), p.a.C * p.a.W, 0, g.dw, nullptr, g.dbias}, s);
}

}  // namespace gdn
