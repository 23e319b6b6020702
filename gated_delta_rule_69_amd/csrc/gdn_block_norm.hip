// Norms around a block with its gate and residual scale, forward and backward:
//     u = y rms(y) post_weight (or y),  r' = rho r + scale act(gate) u,  n = r' rms(r') weight
//
// A row is a workgroup's: eight channels a lane, a wave for every 512 channels (two vectors a
// lane above 8,192, in the gradients above 4,096), so that each tensor is read and written once and
// a row's sums are a few DPP adds and one exchange through LDS. Memory bounds it.
//
// bf16, gate, norm after and before, C 2,048: 65,536 tokens 252 us (1.34 GB, 5.3 TB/s: a copy's rate); the
// gradients of 8,192 tokens 61 us (268 MB, 4.4 TB/s), 5 of them the weights' sums in a second kernel.
#include <algorithm>

#include "gdn_block.h"
#include "gdn_block_device.h"

namespace gdn {
namespace {

constexpr int kMaxWaves = 16;

struct Norm {
  const void *r, *y, *gate;
  const float *scale, *post_w, *w;
  void *r_out, *out;
  int64_t rows, C, ldr, ldy, ldg;
  float eps, rho, mean;   // mean = 1 / C
  bool post;
  // gradients
  const void *d_r, *d_out;
  void *dr, *dy, *dgate;
  float* partial;         // [blocks][3][C]: dweight, dpost_weight, dscale
};

__device__ __forceinline__ float wave_sum(float x) {
  x = row_sum<16>(x);
  x += __shfl_xor(x, 16);
  return x + __shfl_xor(x, 32);
}
// K sums over the workgroup, in every thread; `part` is another one from call to call.
template <int K>
__device__ __forceinline__ void block_sum(float* s, float (*part)[K], int waves) {
#pragma unroll
  for (int k = 0; k < K; ++k) s[k] = wave_sum(s[k]);
  if (waves == 1) return;
  if (threadIdx.x % 64 == 0) {
#pragma unroll
    for (int k = 0; k < K; ++k) part[threadIdx.x / 64][k] = s[k];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < K; ++k) s[k] = 0.0f;
  for (int w = 0; w < waves; ++w) {
#pragma unroll
    for (int k = 0; k < K; ++k) s[k] += part[w][k];
  }
}

// Eight channels; rows start at any multiple of sixteen bytes, also of float32.
template <typename E> using Eight = E __attribute__((ext_vector_type(8), aligned(16)));

template <typename E>
__device__ __forceinline__ void load8(const void* p, int64_t at, float* x) {
  const Eight<E> r = *reinterpret_cast<const Eight<E>*>(static_cast<const E*>(p) + at);
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = float(r[i]);
}
template <typename E>
__device__ __forceinline__ void store8(void* p, int64_t at, const float* x) {
  Eight<E> r;
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = E(x[i]);
  *reinterpret_cast<Eight<E>*>(static_cast<E*>(p) + at) = r;
}
__device__ __forceinline__ void ones_or(const float* w, int64_t c, float* out) {
#pragma unroll
  for (int i = 0; i < 8; ++i) out[i] = 1.0f;
  if (w != nullptr) load4(w + c, out), load4(w + c + 4, out + 4);
}

// NV: vectors of eight channels a lane. The row's vector k of a thread is at 8 (k threads + thread).
template <typename E, typename R, int NV, bool SILU>
__global__ __launch_bounds__(1024) void block_norm_kernel(Norm a) {
  __shared__ float part[2][2][kMaxWaves][1];
  const int waves = blockDim.x / 64;
  int buf = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, buf ^= 1) {
    float r[NV][8] = {}, u[NV][8] = {};
    int64_t c[NV];
    bool own[NV];
    float sum = 0.0f;
  #pragma unroll
    for (int k = 0; k < NV; ++k) {
      c[k] = 8 * (int64_t(k) * blockDim.x + threadIdx.x);
      own[k] = c[k] < a.C;
      if (!own[k]) continue;
      load8<R>(a.r, row * a.ldr + c[k], r[k]);
      if (a.y != nullptr) load8<E>(a.y, row * a.ldy + c[k], u[k]);
  #pragma unroll
      for (int i = 0; i < 8; ++i) sum += u[k][i] * u[k][i];
    }
    float post = 1.0f;
    if (a.post) {
      block_sum<1>(&sum, part[buf][0], waves);
      post = 1.0f / sqrtf(sum * a.mean + a.eps);
    }
    sum = 0.0f;
  #pragma unroll
    for (int k = 0; k < NV; ++k) {
      if (!own[k]) continue;
      float pw[8], sc[8], z[8];
      if (a.y != nullptr) {
        ones_or(a.post_w, c[k], pw);
        ones_or(a.scale, c[k], sc);
        if (a.gate != nullptr) load8<E>(a.gate, row * a.ldg + c[k], z);
  #pragma unroll
        for (int i = 0; i < 8; ++i) {
          float act = 1.0f;
          if (a.gate != nullptr) {
            act = sigmoid_of<E>(z[i]);
            if (SILU) act *= z[i];
          }
          u[k][i] *= post * pw[i] * sc[i] * act;
        }
      }
  #pragma unroll
      for (int i = 0; i < 8; ++i) {
        r[k][i] = fmaf(a.rho, r[k][i], u[k][i]);
        sum += r[k][i] * r[k][i];
      }
      if (a.r_out != nullptr) store8<R>(a.r_out, row * a.C + c[k], r[k]);
    }
    if (a.out == nullptr) continue;
    block_sum<1>(&sum, part[buf][1], waves);
    const float rms = 1.0f / sqrtf(sum * a.mean + a.eps);
  #pragma unroll
    for (int k = 0; k < NV; ++k) {
      if (!own[k]) continue;
      float w[8];
      ones_or(a.w, c[k], w);
  #pragma unroll
      for (int i = 0; i < 8; ++i) r[k][i] *= rms * w[i];
      store8<E>(a.out, row * a.C + c[k], r[k]);
    }
  }
}

// Gradients, r' from the inputs once more. A workgroup walks every gridDim-th row and keeps its
// sums for the weights in registers. MOST threads a workgroup. One vector a lane (rows of up to
// 4,096 channels) leaves registers for the weights too and for a row's loads one ahead of its use.
template <typename E, typename R, int NV, bool SILU, int MOST>
__global__ __launch_bounds__(MOST) void block_norm_bwd_kernel(Norm a) {
  constexpr bool KEEP = NV == 1;
  __shared__ float part[2][3][kMaxWaves][2];
  const int waves = blockDim.x / 64;
  float s_w[NV][8] = {}, s_p[NV][8] = {}, s_s[NV][8] = {};
  float kept[KEEP ? 3 : 1][NV][8];
  int64_t c[NV];
  bool own[NV];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    c[k] = 8 * (int64_t(k) * blockDim.x + threadIdx.x);
    own[k] = c[k] < a.C;
    if (!own[k]) c[k] = 0;
    if constexpr (KEEP) ones_or(a.w, c[k], kept[0][k]), ones_or(a.post_w, c[k], kept[1][k]), ones_or(a.scale, c[k], kept[2][k]);
  }
  struct Loaded {
    Eight<R> r, up;
    Eight<E> y, z, dn;
  };
  // rows of absent inputs are zero; so are a lane's channels behind the last
  auto fetch = [&](Loaded* f, int64_t row) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      f[k] = Loaded{};
      if (!own[k]) continue;
      f[k].r = *reinterpret_cast<const Eight<R>*>(static_cast<const R*>(a.r) + row * a.ldr + c[k]);
      if (a.y != nullptr) f[k].y = *reinterpret_cast<const Eight<E>*>(static_cast<const E*>(a.y) + row * a.ldy + c[k]);
      if (a.gate != nullptr) f[k].z = *reinterpret_cast<const Eight<E>*>(static_cast<const E*>(a.gate) + row * a.ldg + c[k]);
      if (a.d_out != nullptr) f[k].dn = *reinterpret_cast<const Eight<E>*>(static_cast<const E*>(a.d_out) + row * a.C + c[k]);
      if (a.d_r != nullptr) f[k].up = *reinterpret_cast<const Eight<R>*>(static_cast<const R*>(a.d_r) + row * a.C + c[k]);
    }
  };
  Loaded next[NV];
  int buf = 0;
  int64_t row = blockIdx.x;
  if (KEEP && row < a.rows) fetch(next, row);
  for (; row < a.rows; row += gridDim.x, buf ^= 1) {
    if constexpr (!KEEP) fetch(next, row);
    float r[NV][8], y[NV][8], dn[NV][8], up[NV][8], act[NV][8], slope[NV][8];
    float sum[2] = {0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < NV; ++k) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        r[k][i] = float(next[k].r[i]), y[k][i] = float(next[k].y[i]), dn[k][i] = float(next[k].dn[i]), up[k][i] = float(next[k].up[i]);
        act[k][i] = 1.0f, slope[k][i] = 0.0f;
        if (a.gate != nullptr) {
          const float z = float(next[k].z[i]);
          float s, rest;
          sigmoids<E>(z, &s, &rest);
          act[k][i] = SILU ? z * s : s;
          slope[k][i] = SILU ? s * (1.0f + z * rest) : s * rest;
        }
        sum[0] += y[k][i] * y[k][i];
      }
    }
    if (KEEP && row + gridDim.x < a.rows) fetch(next, row + gridDim.x);
    float post = 1.0f;
    if (a.post) {
      block_sum<1>(sum, reinterpret_cast<float(*)[1]>(part[buf][0]), waves);
      post = 1.0f / sqrtf(sum[0] * a.mean + a.eps);
    }
    // y becomes y rms(y) (or stays), r becomes r'
    auto weights = [&](int k, float* w, float* pw, float* sc) {
      if constexpr (KEEP) {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = kept[0][k][i], pw[i] = kept[1][k][i], sc[i] = kept[2][k][i];
      } else {
        ones_or(a.w, c[k], w), ones_or(a.post_w, c[k], pw), ones_or(a.scale, c[k], sc);
      }
    };
    sum[0] = sum[1] = 0.0f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      float w[8], pw[8], sc[8];
      weights(k, w, pw, sc);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        y[k][i] *= post;
        r[k][i] = fmaf(a.rho, r[k][i], y[k][i] * pw[i] * sc[i] * act[k][i]);
        sum[0] += r[k][i] * r[k][i];
        sum[1] += dn[k][i] * w[i] * r[k][i];
      }
    }
    block_sum<2>(sum, part[buf][1], waves);
    const float rms = 1.0f / sqrtf(sum[0] * a.mean + a.eps);
    const float dot = sum[1] * rms * a.mean;
    sum[0] = 0.0f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      float w[8], pw[8], sc[8], out[8];
      weights(k, w, pw, sc);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float n = r[k][i] * rms;
        s_w[k][i] += dn[k][i] * n;
        const float d = up[k][i] + rms * (dn[k][i] * w[i] - n * dot);   // of r'
        out[i] = a.rho * d;
        const float u = y[k][i] * pw[i], du = d * act[k][i];
        s_s[k][i] += du * u;
        slope[k][i] *= d * sc[i] * u;    // of the gate
        dn[k][i] = du * sc[i];           // of u
        s_p[k][i] += dn[k][i] * y[k][i];
        dn[k][i] *= pw[i];               // of y rms(y)
        sum[0] += dn[k][i] * y[k][i];
      }
      if (a.dr != nullptr && own[k]) store8<R>(a.dr, row * a.C + c[k], out);
      if (a.dgate != nullptr && own[k]) store8<E>(a.dgate, row * a.C + c[k], slope[k]);
    }
    if (a.dy == nullptr) continue;
    float back = 0.0f;
    if (a.post) {
      block_sum<1>(sum, reinterpret_cast<float(*)[1]>(part[buf][2]), waves);
      back = sum[0] * a.mean;
    }
#pragma unroll
    for (int k = 0; k < NV; ++k) {
#pragma unroll
      for (int i = 0; i < 8; ++i) dn[k][i] = post * (dn[k][i] - y[k][i] * back);
      if (own[k]) store8<E>(a.dy, row * a.C + c[k], dn[k]);
    }
  }
  if (a.partial == nullptr) return;
  float* to = a.partial + int64_t(blockIdx.x) * 3 * a.C;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    if (!own[k]) continue;
    store8<float>(to, c[k], s_w[k]);
    store8<float>(to + a.C, c[k], s_p[k]);
    store8<float>(to + 2 * a.C, c[k], s_s[k]);
  }
}

// Threads of a gradient launch: two vectors a lane from 4,096 channels on, whose sums and rows take
// 256 registers, so 512 threads.
unsigned bwd_threads(int64_t C) {
  const int64_t lanes = C <= 4096 ? 512 : 1024;   // channels a wave
  return unsigned((C + lanes - 1) / lanes * 64);
}
// Blocks of a gradient launch, eight waves a CU: partial sums of so many rows.
int64_t bwd_blocks(int64_t rows, int64_t C) {
  return std::max<int64_t>(1, std::min<int64_t>(rows, std::max<int64_t>(256, 2048 * 64 / bwd_threads(C))));
}

Norm norm_of(const BlockNormProblem& p) {
  const gdn_block_norm_args& a = p.a;
  Norm n{};
  n.r = a.r, n.y = a.y, n.gate = a.gate, n.scale = a.scale, n.post_w = a.post_weight, n.w = a.weight;
  n.r_out = a.residual_out, n.out = a.out;
  n.rows = p.tokens, n.C = a.C, n.ldr = a.r_stride, n.ldy = a.y_stride, n.ldg = a.gate_stride;
  n.eps = a.eps, n.rho = a.residual_scale, n.mean = 1.0f / float(a.C), n.post = a.post_norm != 0;
  return n;
}

template <typename F>
int by_types(const gdn_block_norm_args& a, F f) {
  auto width = [&](auto e, auto r) {
    auto act = [&](auto nv) {
      return a.activation == GDN_ACT_SILU ? f(e, r, nv, std::true_type{}) : f(e, r, nv, std::false_type{});
    };
    return a.C <= 8192 ? act(std::integral_constant<int, 1>{}) : act(std::integral_constant<int, 2>{});
  };
  if (a.dtype == GDN_DTYPE_F32) return width(float{}, float{});
  return a.residual_dtype == GDN_DTYPE_F32 ? width(__bf16{}, float{}) : width(__bf16{}, __bf16{});
}

unsigned threads_of(int64_t C) { return C <= 8192 ? unsigned((C + 511) / 512 * 64) : 1024; }

}  // namespace

int launch_block_norm_fwd(const BlockNormProblem& p, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  const Norm n = norm_of(p);
  return by_types(p.a, [&](auto e, auto r, auto nv, auto silu) {
    block_norm_kernel<decltype(e), decltype(r), decltype(nv)::value, decltype(silu)::value>
        <<<unsigned(std::min<int64_t>(n.rows, 1 << 20)), threads_of(n.C), 0, s>>>(n);
    return int(hipGetLastError());
  });
}

size_t block_norm_bwd_workspace(const BlockNormProblem& p) {
  return size_t(bwd_blocks(p.tokens, p.a.C)) * 3 * p.a.C * sizeof(float);
}

int launch_block_norm_bwd(const BlockNormProblem& p, const gdn_block_norm_grads& g, void* ws, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  Norm n = norm_of(p);
  n.d_r = g.d_residual_out, n.d_out = g.d_out, n.dr = g.dr, n.dy = g.dy, n.dgate = g.dgate;
  const bool sums = g.dweight != nullptr || g.dpost_weight != nullptr || g.dscale != nullptr;
  n.partial = sums ? static_cast<float*>(ws) : nullptr;
  const int64_t blocks = bwd_blocks(n.rows, n.C);
  const int rc = by_types(p.a, [&](auto e, auto r, auto, auto silu) {
    typedef decltype(e) E;
    typedef decltype(r) R;
    constexpr bool SILU = decltype(silu)::value;
    const unsigned threads = bwd_threads(n.C);
    if (n.C <= 2048)
      block_norm_bwd_kernel<E, R, 1, SILU, 256><<<unsigned(blocks), threads, 0, s>>>(n);
    else if (n.C <= 4096)
      block_norm_bwd_kernel<E, R, 1, SILU, 512><<<unsigned(blocks), threads, 0, s>>>(n);
    else if (n.C <= 8192)
      block_norm_bwd_kernel<E, R, 2, SILU, 512><<<unsigned(blocks), threads, 0, s>>>(n);
    else
      block_norm_bwd_kernel<E, R, 2, SILU, 1024><<<unsigned(blocks), threads, 0, s>>>(n);
    return int(hipGetLastError());
  });
  if (rc != 0 || !sums) return rc;
  return launch_column_sum({n.partial, int(blocks), 3 * n.C, n.C, n.C, g.dweight, g.dpost_weight, g.dscale}, s);
}

}  // namespace gdn
