// Norms around a block with its gate and residual scale, forward and backward:
//     u = y rms(y) post_weight (or y),  r' = rho r + scale act(gate) u,  n = r' rms(r') weight
//
// A row is a workgroup's: eight channels a lane, a wave for every 512 channels (two vectors a
// lane above 8,192; in the gradients two above 4,096 and four above 8,192), so that each tensor is read
// and written once and a row's sums are a few DPP adds and one exchange through LDS. Memory bounds it.
//
// bf16, gate, norm after and before, C 2,048: 65,536 tokens 252 us (1.34 GB, 5.3 TB/s: a copy's rate); the
// gradients of 8,192 tokens 60 us (268 MB, 4.5 TB/s), 4 of them the weights' sums in a second kernel; of
// 2,048 tokens with C 8,192 77 us and of 1,024 with C 16,384 93 us (268 MB, 3.5 and 2.9 TB/s).
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
  float* partial;         // [blocks][2][C]: dweight; dpost_weight / scale = dscale / post_weight
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

// Eight channels; rows start at any multiple of sixteen bytes, also of float32. A row's start is the
// same for all lanes and a lane's place in it 32 bits, so that no address takes a lane's registers.
template <typename E> using Eight = E __attribute__((ext_vector_type(8), aligned(16)));

template <typename E>
__device__ __forceinline__ Eight<E> eight(const void* p, int64_t row, uint32_t c) {
  return *reinterpret_cast<const Eight<E>*>(static_cast<const E*>(p) + row + c);
}
template <typename E>
__device__ __forceinline__ void load8(const void* p, int64_t row, uint32_t c, float* x) {
  const Eight<E> r = eight<E>(p, row, c);
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = float(r[i]);
}
template <typename E>
__device__ __forceinline__ void store8(void* p, int64_t row, uint32_t c, const float* x) {
  Eight<E> r;
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = E(x[i]);
  *reinterpret_cast<Eight<E>*>(static_cast<E*>(p) + row + c) = r;
}
__device__ __forceinline__ void ones_or(const float* w, uint32_t c, float* out) {
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
    uint32_t c[NV];
    bool own[NV];
    float sum = 0.0f;
  #pragma unroll
    for (int k = 0; k < NV; ++k) {
      c[k] = 8 * (k * blockDim.x + threadIdx.x);
      own[k] = c[k] < a.C;
      if (!own[k]) continue;
      load8<R>(a.r, row * a.ldr, c[k], r[k]);
      if (a.y != nullptr) load8<E>(a.y, row * a.ldy, c[k], u[k]);
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
        if (a.gate != nullptr) load8<E>(a.gate, row * a.ldg, c[k], z);
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
      if (a.r_out != nullptr) store8<R>(a.r_out, row * a.C, c[k], r[k]);
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
      store8<E>(a.out, row * a.C, c[k], r[k]);
    }
  }
}

// What follows takes x from its registers anew: nothing formed from it before is kept.
template <typename V> __device__ __forceinline__ void forget(V& x) {
  typedef uint32_t Words __attribute__((ext_vector_type(4)));
  Words w[sizeof(V) / 16];
  __builtin_memcpy(w, &x, sizeof(V));
#pragma unroll
  for (int i = 0; i < int(sizeof(V) / 16); ++i) asm volatile("" : "+v"(w[i])::"memory");
  __builtin_memcpy(&x, w, sizeof(V));
  __builtin_amdgcn_sched_barrier(0);
}

// A thread's eight sums of vector k in LDS, four side by side a thread: x added to them (or in their place).
template <int THREADS>
__device__ __forceinline__ void add8(float* sums, int k, float* x, bool add) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float4* at = reinterpret_cast<float4*>(sums) + threadIdx.x + (2 * k + h) * THREADS;
    float4 v = make_float4(x[4 * h], x[4 * h + 1], x[4 * h + 2], x[4 * h + 3]);
    if (add) {
      const float4 o = *at;
      v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
    }
    *at = v;
    x[4 * h] = v.x, x[4 * h + 1] = v.y, x[4 * h + 2] = v.z, x[4 * h + 3] = v.w;
  }
}

// Gradients, r' from the inputs once more. A workgroup walks every gridDim-th row and keeps its
// sums for the weights in registers; post_weight's and scale's are one, of d_r' act(gate) y rms(y),
// which is multiplied by the other weight at the end. MOST threads a workgroup.
// KEEP: one vector a lane leaves registers for the weights too. AHEAD: a row's loads come one row ahead
// of their use; two vectors a lane of bf16 leave registers for that (C 6,144 118 us against 127), of
// float32 they do not. WIDE: four vectors a lane leave none for the sums, which go to LDS, nor for what
// the loaded rows give, which is formed anew in each phase (C 16,384 93 us; with sums and gates in
// registers, two vectors a lane and 1,024 threads 317, all of it spilled).
template <typename E, typename R, int NV, bool SILU, int MOST>
__global__ __launch_bounds__(MOST) void block_norm_bwd_kernel(Norm a) {
  constexpr bool KEEP = NV == 1, AHEAD = KEEP || (NV == 2 && sizeof(E) == 2), WIDE = NV == 4;
  __shared__ float part[2][3][kMaxWaves][2];
  const int waves = blockDim.x / 64;
  __shared__ __attribute__((aligned(16))) float wide[WIDE ? 2 : 1][WIDE ? NV * 8 * MOST : 4];
  float s_w[WIDE ? 1 : NV][8] = {}, s_u[WIDE ? 1 : NV][8] = {};
  float kept[KEEP ? 3 : 1][NV][8];
  uint32_t c[NV];
  bool own[NV];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    c[k] = 8 * (k * blockDim.x + threadIdx.x);
    own[k] = c[k] < a.C;
    if (!own[k]) c[k] = 0;
    if constexpr (WIDE) add8<MOST>(wide[0], k, s_w[0], false), add8<MOST>(wide[1], k, s_u[0], false);
    if constexpr (KEEP) ones_or(a.w, c[k], kept[0][k]), ones_or(a.post_w, c[k], kept[1][k]), ones_or(a.scale, c[k], kept[2][k]);
  }
  // A lane's place, taken anew at each use: else a lane's addresses in every tensor are formed ahead of
  // the loop, two registers each.
  auto at = [&](int k) {
    uint32_t x = c[k];
    asm volatile("" : "+v"(x));
    return x;
  };
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
      f[k].r = eight<R>(a.r, row * a.ldr, at(k));
      if (a.y != nullptr) f[k].y = eight<E>(a.y, row * a.ldy, at(k));
      if (a.gate != nullptr) f[k].z = eight<E>(a.gate, row * a.ldg, at(k));
      if (a.d_out != nullptr) f[k].dn = eight<E>(a.d_out, row * a.C, at(k));
      if (a.d_r != nullptr) f[k].up = eight<R>(a.d_r, row * a.C, at(k));
    }
  };
  Loaded next[NV];
  int buf = 0;
  int64_t row = blockIdx.x;
  if (AHEAD && row < a.rows) fetch(next, row);
  for (; row < a.rows; row += gridDim.x, buf ^= 1) {
    if constexpr (!AHEAD) fetch(next, row);
    float r[NV][8], y[NV][8];
    float dn_kept[WIDE ? 1 : NV][8], up_kept[WIDE ? 1 : NV][8], act_kept[WIDE ? 1 : NV][8], slope_kept[WIDE ? 1 : NV][8];
    auto gate_of = [&](int k, int i, float* act, float* slope) {
      *act = 1.0f, *slope = 0.0f;
      if (a.gate == nullptr) return;
      const float z = float(next[k].z[i]);
      float s, rest;
      sigmoids<E>(z, &s, &rest);
      *act = SILU ? z * s : s;
      *slope = SILU ? s * (1.0f + z * rest) : s * rest;
    };
    float sum[2] = {0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < NV; ++k) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        r[k][i] = float(next[k].r[i]), y[k][i] = float(next[k].y[i]);
        if constexpr (!WIDE) {
          dn_kept[k][i] = float(next[k].dn[i]), up_kept[k][i] = float(next[k].up[i]);
          gate_of(k, i, &act_kept[k][i], &slope_kept[k][i]);
        }
        sum[0] += y[k][i] * y[k][i];
      }
    }
    if (AHEAD && row + gridDim.x < a.rows) fetch(next, row + gridDim.x);
    float post = 1.0f;
    if (a.post) {
      block_sum<1>(sum, reinterpret_cast<float(*)[1]>(part[buf][0]), waves);
      post = 1.0f / sqrtf(sum[0] * a.mean + a.eps);
    }
    auto dn_of = [&](int k, int i) {
      if constexpr (WIDE) return float(next[k].dn[i]); else return dn_kept[k][i];
    };
    // y becomes y rms(y) (or stays), r becomes r'
    auto weights = [&](int k, float* w, float* pw, float* sc) {
      if constexpr (KEEP) {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = kept[0][k][i], pw[i] = kept[1][k][i], sc[i] = kept[2][k][i];
      } else {
        ones_or(a.w, at(k), w), ones_or(a.post_w, at(k), pw), ones_or(a.scale, at(k), sc);
      }
    };
    sum[0] = sum[1] = 0.0f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      if constexpr (WIDE) forget(next[k].z), forget(next[k].dn);
      float w[8], pw[8], sc[8];
      weights(k, w, pw, sc);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        y[k][i] *= post;
        float act, slope;
        if constexpr (WIDE) gate_of(k, i, &act, &slope); else act = act_kept[k][i];
        r[k][i] = fmaf(a.rho, r[k][i], y[k][i] * pw[i] * sc[i] * act);
        sum[0] += r[k][i] * r[k][i];
        sum[1] += dn_of(k, i) * w[i] * r[k][i];
      }
    }
    block_sum<2>(sum, part[buf][1], waves);
    const float rms = 1.0f / sqrtf(sum[0] * a.mean + a.eps);
    const float dot = sum[1] * rms * a.mean;
    sum[0] = 0.0f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      if constexpr (WIDE) forget(next[k].z), forget(next[k].dn), forget(next[k].up);
      float w[8], pw[8], sc[8], out[8], dgate[8], add_w[8], add_u[8];
      weights(k, w, pw, sc);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float act, slope, up;
        if constexpr (WIDE)
          gate_of(k, i, &act, &slope), up = float(next[k].up[i]);
        else
          act = act_kept[k][i], slope = slope_kept[k][i], up = up_kept[k][i];
        const float n = r[k][i] * rms, dn = dn_of(k, i);
        add_w[i] = dn * n;
        const float d = up + rms * (dn * w[i] - n * dot);   // of r'
        out[i] = a.rho * d;
        const float du = d * act;
        add_u[i] = du * y[k][i];
        dgate[i] = slope * (d * sc[i] * (y[k][i] * pw[i]));
        r[k][i] = du * sc[i] * pw[i];   // of y rms(y)
        sum[0] += r[k][i] * y[k][i];
      }
      if constexpr (WIDE) {
        add8<MOST>(wide[0], k, add_w, true), add8<MOST>(wide[1], k, add_u, true);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) s_w[k][i] += add_w[i], s_u[k][i] += add_u[i];
      }
      if (a.dr != nullptr && own[k]) store8<R>(a.dr, row * a.C, at(k), out);
      if (a.dgate != nullptr && own[k]) store8<E>(a.dgate, row * a.C, at(k), dgate);
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
      for (int i = 0; i < 8; ++i) r[k][i] = post * (r[k][i] - y[k][i] * back);
      if (own[k]) store8<E>(a.dy, row * a.C, at(k), r[k]);
    }
  }
  if (a.partial == nullptr) return;
  float* to = a.partial + int64_t(blockIdx.x) * 2 * a.C;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    if (!own[k]) continue;
    if constexpr (WIDE) {
#pragma unroll
      for (int i = 0; i < 8; ++i) s_w[0][i] = s_u[0][i] = 0.0f;
      add8<MOST>(wide[0], k, s_w[0], true), add8<MOST>(wide[1], k, s_u[0], true);
    }
    store8<float>(to, 0, c[k], s_w[WIDE ? 0 : k]);
    store8<float>(to, a.C, c[k], s_u[WIDE ? 0 : k]);
  }
}

// Channels a lane in the gradients.
int bwd_vectors(int64_t C) { return C <= 4096 ? 1 : C <= 8192 ? 2 : 4; }
unsigned bwd_threads(int64_t C) {
  const int64_t lanes = 512 * bwd_vectors(C);   // channels a wave
  return unsigned((C + lanes - 1) / lanes * 64);
}
// Workgroups of a gradient launch, and rows of partial sums: those that stand on the CUs together at
// eight waves a CU, since each walks as many rows as the others (C 6,144, six waves: 256 workgroups
// 126 us, 341 take 175; at twelve waves a CU bf16 rows gain 0 to 2 %, float32 ones lose 3 to 13).
int64_t bwd_blocks(int64_t rows, int64_t C) {
  return std::max<int64_t>(1, std::min<int64_t>(rows, 256 * std::max<int64_t>(1, 8 * 64 / bwd_threads(C))));
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
  return size_t(bwd_blocks(p.tokens, p.a.C)) * 2 * p.a.C * sizeof(float);
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
      block_norm_bwd_kernel<E, R, 4, SILU, 512><<<unsigned(blocks), threads, 0, s>>>(n);
    return int(hipGetLastError());
  });
  if (rc != 0 || !sums) return rc;
  return launch_column_sum({n.partial, int(blocks), 2 * n.C, n.C, n.C, g.dweight, g.dpost_weight, nullptr, g.dscale, n.scale, n.post_w}, s);
}

}  // namespace gdn
