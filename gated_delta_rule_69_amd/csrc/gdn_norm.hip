// Norms of queries and keys a head with the position rotation, and the gated norm of a
// layer's outputs; forward and backward.
//
// Both are streams: each row of d channels is read once and written once, so memory
// bounds them. A row lies in d / 8 neighbouring lanes, eight channels a lane, and its sum
// of squares is a few DPP adds; nothing goes through LDS. A block walks the rows of a
// range of its own and keeps (token, head) of its next row by addition, so there is no
// division in the loop, and a row's loads run one step ahead of its use.
//
// bf16, d 128: queries and keys of 65,536 tokens, 16 heads each, 215 to 228 us (1.11 GB, 4.9
// to 5.1 TB/s; a copy of 512 MiB reaches 5.39), float32 382 us (5.7); the gated norm of 65,536
// tokens x 16 heads 142 to 145 us (805 MB, 5.6 TB/s), float32 277 us (5.8). Backward at 8,192
// tokens: 34 to 35 us (153 MB) and 29 to 30 us (168 MB), and 4 us for the weights' sums in a
// second kernel, whose order is fixed. Those sums are float32: at d 128 rows / 16,384 terms a
// lane, then 16 of a block, 16 blocks and a tree of six, 6e-6 at worst for a million rows.
#include <algorithm>

#include "gdn_layer.h"
#include "gdn_layer_device.h"

namespace gdn {
namespace {

constexpr int kThreads = 256;

// Row `hh` of `heads` of token `token`, advanced by `step` rows at a time. PLACE: also the
// token's place `pos` in its sequence of T (1 to 2^31).
template <bool PLACE>
struct RowWalk {
  int64_t token;
  unsigned hh, heads, step_tokens, step_heads, pos = 0, step_pos = 0, T = 1;
  __device__ RowWalk(int64_t row, unsigned heads_, unsigned step, int64_t T_) : heads(heads_) {
    token = row / heads_;
    hh = unsigned(row - token * heads_);
    step_tokens = step / heads_;
    step_heads = step % heads_;
    if constexpr (PLACE) {
      T = unsigned(T_);
      pos = unsigned(token % T_);
      step_pos = step_tokens % T;
    }
  }
  __device__ void next() {
    const unsigned carry = hh + step_heads >= heads;
    token += step_tokens + carry;
    hh += step_heads - (carry ? heads : 0);
    if constexpr (PLACE) {
      pos += step_pos + carry;  // at most 2 T - 1
      if (pos >= T) pos -= T;
    }
  }
};

// The channels of lane `l` of a row, two runs of four: for half-split pairs the runs are
// channels i and i + rot/2 of four pairs, so that a pair never leaves its lane.
struct Channels {
  int c0, c1, pair;
  bool turned;
  __device__ Channels(int l, int rot, bool interleaved) {
    turned = 8 * l < rot;
    pair = 4 * l;
    const bool split = turned && !interleaved;
    c0 = split ? 4 * l : 8 * l;
    c1 = split ? rot / 2 + 4 * l : 8 * l + 4;
  }
};

// Rotates the four pairs of a lane by (cos, sign * sin); x[0..3] and x[4..7] are its runs.
__device__ __forceinline__ void turn(float* x, const float* cs, const float* sn, float sign, bool interleaved) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float s = sign * sn[i];
    float& a = interleaved ? x[2 * i] : x[i];
    float& b = interleaved ? x[2 * i + 1] : x[4 + i];
    const float t = a * cs[i] - b * s;
    b = b * cs[i] + a * s;
    a = t;
  }
}

struct QkNorm {
  const void *q, *k;
  void *q_out, *k_out;
  const float *wq, *wk, *cos, *sin;
  const int32_t* positions;
  int64_t rows, rows_per_block, ldq, ldk, T, n_pos;
  unsigned hq, hk;
  int rot;
  float mean;  // 1 / d (RMS) or 1 (L2): of a row's sums
  float eps, q_scale;
  bool interleaved;
  // backward
  const void *dq_out, *dk_out;
  void *dq, *dk;
  float* partial;  // [blocks][2][d]
};

__device__ __forceinline__ void ones_or(const float* w, int c, float* out) {
  if (w != nullptr) {
    load4(w + c, out);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) out[i] = 1.0f;
  }
}

// cos and sin of a lane's pairs, if it has any, at its token's position; false, in every
// lane of the row, for a position outside the table (the row becomes NaN).
template <bool GIVEN, typename Walk>
__device__ __forceinline__ bool angles(const QkNorm& a, const Walk& at_row, const Channels& ch, float* cs, float* sn) {
  const int64_t pos = GIVEN ? int64_t(a.positions[at_row.token]) : int64_t(at_row.pos);
  const bool in = pos >= 0 && pos < a.n_pos;
  const int64_t at = (in ? pos : 0) * (a.rot / 2) + ch.pair;
  if (ch.turned) {
    load4(a.cos + at, cs);
    load4(a.sin + at, sn);
  }
  return in;
}

// BWD: gradients of the inputs from those of the outputs (of type G) and the block's sums
// for the weights; otherwise the forward pass. GIVEN: positions are read (or nothing is
// rotated); without them a token's place is walked along: at bf16, 32 x d 128, 65,536 tokens 203
// us and 8,192 tokens' gradients (32 heads) 36 against 205 and 39 with a division a row, and
// with given positions 217 against 228 in one kernel for both.
template <typename E, typename G, int D, bool GIVEN, bool BWD>
__global__ __launch_bounds__(kThreads) void qk_norm_kernel(QkNorm a) {
  constexpr int L = D / 8;               // lanes a row
  constexpr int R = kThreads / L;        // rows a step
  const int l = threadIdx.x % L;
  const Channels ch(l, a.rot, a.interleaved);
  float wq[8], wk[8], sum_q[8] = {}, sum_k[8] = {};
  ones_or(a.wq, ch.c0, wq), ones_or(a.wq, ch.c1, wq + 4);
  ones_or(a.wk, ch.c0, wk), ones_or(a.wk, ch.c1, wk + 4);
  const int64_t begin = int64_t(blockIdx.x) * a.rows_per_block;
  const int64_t end = begin + a.rows_per_block < a.rows ? begin + a.rows_per_block : a.rows;
  int64_t row = begin + threadIdx.x / L;
  RowWalk<!GIVEN> at(row, a.hq + a.hk, R, a.T);
  // A row's loads run one step ahead of its use.
  struct Loaded {
    vec<E, 4> x[2];
    vec<G, 4> dy[2];
    float cs[4], sn[4];
    bool in;
  };
  auto fetch = [&](Loaded& f) {
    const bool key = at.hh >= a.hq;
    const unsigned h = key ? at.hh - a.hq : at.hh;
    const E* x = static_cast<const E*>(key ? a.k : a.q) + at.token * (key ? a.ldk : a.ldq) + int64_t(h) * D;
    f.x[0] = *reinterpret_cast<const vec<E, 4>*>(x + ch.c0);
    f.x[1] = *reinterpret_cast<const vec<E, 4>*>(x + ch.c1);
    if constexpr (BWD) {
      const G* dy = static_cast<const G*>(key ? a.dk_out : a.dq_out) + (at.token * (key ? a.hk : a.hq) + h) * D;
      f.dy[0] = *reinterpret_cast<const vec<G, 4>*>(dy + ch.c0);
      f.dy[1] = *reinterpret_cast<const vec<G, 4>*>(dy + ch.c1);
    }
    f.in = a.rot == 0 || angles<GIVEN>(a, at, ch, f.cs, f.sn);
  };
  Loaded next;
  if (row < end) fetch(next);
  while (row < end) {
    const Loaded now = next;
    const bool key = at.hh >= a.hq;
    const unsigned h = key ? at.hh - a.hq : at.hh;
    const int64_t out_row = (at.token * (key ? a.hk : a.hq) + h) * D;
    row += R;
    at.next();
    if (row < end) fetch(next);
    float x[8], y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[i] = float(now.x[i / 4][i % 4]);
      if constexpr (BWD) y[i] = float(now.dy[i / 4][i % 4]);
    }
    const float *cs = now.cs, *sn = now.sn;
    const bool in = now.in;
    const float scale = key ? 1.0f : a.q_scale;
    float sq = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) sq += x[i] * x[i];
    sq = row_sum<L>(sq);
    const float r = 1.0f / sqrtf(sq * a.mean + a.eps);
    if constexpr (!BWD) {
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = x[i] * r * (key ? wk[i] : wq[i]);
      if (ch.turned) turn(y, cs, sn, 1.0f, a.interleaved);
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = in ? y[i] * scale : __builtin_nanf("");
      E* out = static_cast<E*>(key ? a.k_out : a.q_out) + out_row;
      store4(out + ch.c0, y);
      store4(out + ch.c1, y + 4);
    } else {
      // with n = x r: dn = w (the rotation backwards of dy), dx = r (dn - n mean(dn n))
      if (ch.turned) turn(y, cs, sn, -1.0f, a.interleaved);
      float dot = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[i] *= r;
        y[i] = in ? y[i] * scale : __builtin_nanf("");
        const float dw = y[i] * x[i];
        sum_q[i] += key ? 0.0f : dw;
        sum_k[i] += key ? dw : 0.0f;
        y[i] *= key ? wk[i] : wq[i];
        dot += y[i] * x[i];
      }
      dot = row_sum<L>(dot) * a.mean;
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = r * (y[i] - x[i] * dot);
      E* out = static_cast<E*>(key ? a.dk : a.dq) + out_row;
      store4(out + ch.c0, y);
      store4(out + ch.c1, y + 4);
    }
  }
  if constexpr (BWD) {
    // the block's sums a channel, over its R rows' lanes in a fixed order
    __shared__ float part[kThreads][8];
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 8; ++i) part[threadIdx.x][i] = w ? sum_k[i] : sum_q[i];
      __syncthreads();
      if (threadIdx.x < D) {
        // channel c belongs to lane ll, place i (as Channels lays them out)
        const int ll = threadIdx.x / 8, i = threadIdx.x % 8;
        const Channels own(ll, a.rot, a.interleaved);
        float s = 0.0f;
        for (int g = 0; g < R; ++g) s += part[g * L + ll][i];
        a.partial[(int64_t(blockIdx.x) * 2 + w) * D + (i < 4 ? own.c0 + i : own.c1 + i - 4)] = s;
      }
    }
  }
}

struct GatedNorm {
  const void *x, *gate;
  const float* w;
  void* y;
  int64_t rows, rows_per_block, ldx, ldg;
  unsigned heads;
  float eps;
  // backward
  const void* dy;
  void *dx, *dgate;
  float* partial;  // [blocks][d]
};

// 1 / (1 + e^-z), the reciprocal (of at least 1) within 1 ulp. __expf rounds z log2 e first,
// which puts it off by |z| 2^-24: nothing for a gate of bf16, 30 steps for a float32 one at
// -60, which takes expf.
template <typename E>
__device__ __forceinline__ float sigmoid(float z) {
  return __builtin_amdgcn_rcpf(1.0f + (sizeof(E) == 2 ? __expf(-z) : expf(-z)));
}

// The sigmoid s and 1 - s, both from e = e^-|z|: 1 / (1 + e) and e / (1 + e) are within a few
// steps wherever they lie, where the difference 1 - s would hold nothing of a gate far open
// (e^-z is under a step of 1 from z = 17 on, and 1 % of it is lost at 12).
template <typename E>
__device__ __forceinline__ void sigmoid_both(float z, float* s, float* rest) {
  const float e = sizeof(E) == 2 ? __expf(-fabsf(z)) : expf(-fabsf(z));
  const float big = __builtin_amdgcn_rcpf(1.0f + e), small = e * big;
  *s = z < 0.0f ? small : big;
  *rest = z < 0.0f ? big : small;
}

template <typename E, int D, bool SILU, bool BWD>
__global__ __launch_bounds__(kThreads) void gated_norm_kernel(GatedNorm a) {
  constexpr int L = D / 8;
  constexpr int R = kThreads / L;
  const int l = threadIdx.x % L;
  const int c = 8 * l;
  float w[8], sum[8] = {};
  ones_or(a.w, c, w), ones_or(a.w, c + 4, w + 4);
  const int64_t begin = int64_t(blockIdx.x) * a.rows_per_block;
  const int64_t end = begin + a.rows_per_block < a.rows ? begin + a.rows_per_block : a.rows;
  int64_t row = begin + threadIdx.x / L;
  RowWalk<false> at(row, a.heads, R, 1);
  struct Loaded {  // one step ahead of its use
    vec<E, 8> x, z, dy;
  };
  auto fetch = [&](Loaded& f) {
    f.x = *reinterpret_cast<const vec<E, 8>*>(static_cast<const E*>(a.x) + at.token * a.ldx + int64_t(at.hh) * D + c);
    f.z = *reinterpret_cast<const vec<E, 8>*>(static_cast<const E*>(a.gate) + at.token * a.ldg + int64_t(at.hh) * D + c);
    if constexpr (BWD) f.dy = *reinterpret_cast<const vec<E, 8>*>(static_cast<const E*>(a.dy) + row * D + c);
  };
  Loaded next;
  if (row < end) fetch(next);
  while (row < end) {
    const Loaded now = next;
    const int64_t here = row;
    row += R;
    at.next();
    if (row < end) fetch(next);
    float x[8], z[8], dy[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[i] = float(now.x[i]), z[i] = float(now.z[i]);
      if constexpr (BWD) dy[i] = float(now.dy[i]);
    }
    float sq = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) sq += x[i] * x[i];
    sq = row_sum<L>(sq);
    const float r = 1.0f / sqrtf(sq * (1.0f / D) + a.eps);
    if constexpr (!BWD) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float s = sigmoid<E>(z[i]);
        x[i] = x[i] * r * w[i] * (SILU ? z[i] * s : s);
      }
      E* out = static_cast<E*>(a.y) + here * D + c;
      store4(out, x), store4(out + 4, x + 4);
    } else {
      float dot = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float s, rest;
        sigmoid_both<E>(z[i], &s, &rest);
        const float act = SILU ? z[i] * s : s;
        const float slope = SILU ? s * (1.0f + z[i] * rest) : s * rest;
        x[i] *= r;
        const float dn = dy[i] * x[i];   // gradient of w act, but for its factors
        z[i] = dn * w[i] * slope;
        sum[i] += dn * act;
        dy[i] *= act * w[i];
        dot += dy[i] * x[i];
      }
      dot = row_sum<L>(dot) * (1.0f / D);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = r * (dy[i] - x[i] * dot);
      E* dx = static_cast<E*>(a.dx) + here * D + c;
      E* dg = static_cast<E*>(a.dgate) + here * D + c;
      store4(dx, x), store4(dx + 4, x + 4);
      store4(dg, z), store4(dg + 4, z + 4);
    }
  }
  if constexpr (BWD) {
    __shared__ float part[kThreads][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) part[threadIdx.x][i] = sum[i];
    __syncthreads();
    if (threadIdx.x < D) {
      float s = 0.0f;
      for (int g = 0; g < R; ++g) s += part[g * L + threadIdx.x / 8][threadIdx.x % 8];
      a.partial[int64_t(blockIdx.x) * D + threadIdx.x] = s;
    }
  }
}

// out[i][c] = sum over blocks of partial[block][i][c], a block for 16 channels of one i:
// 64 threads a channel add up every 64th row, then a tree of fixed order.
__global__ __launch_bounds__(1024) void partial_sum_kernel(const float* __restrict__ partial, int blocks, int rows, int d,
                                                           float* out0, float* out1) {
  const int c = int(blockIdx.x) * 16 % d + threadIdx.x % 16, row = int(blockIdx.x) * 16 / d;
  const int n = threadIdx.x / 16;
  float s = 0.0f;
#pragma unroll 8
  for (int b = n; b < blocks; b += 64) s += partial[(int64_t(b) * rows + row) * d + c];
  __shared__ float part[1024];
  part[threadIdx.x] = s;
#pragma unroll
  for (int step = 512; step >= 16; step /= 2) {
    __syncthreads();
    if (threadIdx.x < step) part[threadIdx.x] += part[threadIdx.x + step];
  }
  float* out = row == 0 ? out0 : out1;
  if (threadIdx.x < 16 && out != nullptr) out[c] = part[threadIdx.x];
}

// Blocks of a launch over `rows` rows, `per_step` at a time, and the rows each takes.
int64_t split_rows(int64_t rows, int64_t per_step, int64_t most, int64_t* per_block) {
  const int64_t steps = (rows + per_step - 1) / per_step;
  const int64_t each = std::max<int64_t>(1, (steps + most - 1) / most);
  *per_block = each * per_step;
  return (steps + each - 1) / each;
}

// Blocks of a forward launch: each takes at least four steps where there are enough, and a
// launch has fewer than 2^32 threads.
int64_t forward_blocks(int64_t rows, int64_t per_step) {
  const int64_t steps = (rows + per_step - 1) / per_step;
  return steps < 4096 ? std::max<int64_t>(steps, 1) : std::min<int64_t>((steps + 3) / 4, int64_t(1) << 23);
}

template <typename F>
int by_dim(int64_t d, F f) {
  switch (d) {
    case 16: return f(std::integral_constant<int, 16>{});
    case 32: return f(std::integral_constant<int, 32>{});
    case 64: return f(std::integral_constant<int, 64>{});
    case 128: return f(std::integral_constant<int, 128>{});
    default: return int(hipErrorInvalidValue);
  }
}

QkNorm qk_params(const QkNormProblem& p) {
  const gdn_qk_norm_args& a = p.a;
  QkNorm n{};
  n.q = a.q, n.k = a.k, n.q_out = a.q_out, n.k_out = a.k_out, n.wq = a.wq, n.wk = a.wk;
  n.cos = a.cos, n.sin = a.sin, n.positions = a.positions;
  n.rows = p.tokens * (a.Hq + a.Hk);
  n.ldq = a.q_stride, n.ldk = a.k_stride, n.T = a.T, n.n_pos = a.n_pos;
  n.mean = a.norm == GDN_NORM_L2 ? 1.0f : 1.0f / float(a.d);
  n.hq = unsigned(a.Hq), n.hk = unsigned(a.Hk), n.rot = int(a.rot);
  n.eps = a.eps, n.q_scale = a.q_scale, n.interleaved = a.interleaved != 0;
  return n;
}

template <typename E, typename G, bool BWD>
int launch_qk(QkNorm n, const QkNormProblem& p, int64_t most, int64_t* blocks, hipStream_t s) {
  return by_dim(p.a.d, [&](auto dim) {
    constexpr int D = decltype(dim)::value;
    constexpr int64_t R = kThreads / (D / 8);
    *blocks = split_rows(n.rows, R, most ? most : forward_blocks(n.rows, R), &n.rows_per_block);
    if (*blocks == 0) return 0;
    if (n.positions != nullptr || n.rot == 0)
      qk_norm_kernel<E, G, D, true, BWD><<<unsigned(*blocks), kThreads, 0, s>>>(n);
    else
      qk_norm_kernel<E, G, D, false, BWD><<<unsigned(*blocks), kThreads, 0, s>>>(n);
    return int(hipGetLastError());
  });
}

GatedNorm gated_params(const GatedNormProblem& p) {
  const gdn_gated_norm_args& a = p.a;
  GatedNorm n{};
  n.x = a.x, n.gate = a.gate, n.w = a.weight, n.y = a.y;
  n.rows = p.tokens * a.H;
  n.ldx = a.x_stride, n.ldg = a.gate_stride;
  n.heads = unsigned(a.H), n.eps = a.eps;
  return n;
}

template <typename E, bool BWD>
int launch_gated(GatedNorm n, const GatedNormProblem& p, int64_t most, int64_t* blocks, hipStream_t s) {
  return by_dim(p.a.d, [&](auto dim) {
    constexpr int D = decltype(dim)::value;
    constexpr int64_t R = kThreads / (D / 8);
    *blocks = split_rows(n.rows, R, most ? most : forward_blocks(n.rows, R), &n.rows_per_block);
    if (*blocks == 0) return 0;
    if (p.a.activation == GDN_ACT_SILU)
      gated_norm_kernel<E, D, true, BWD><<<unsigned(*blocks), kThreads, 0, s>>>(n);
    else
      gated_norm_kernel<E, D, false, BWD><<<unsigned(*blocks), kThreads, 0, s>>>(n);
    return int(hipGetLastError());
  });
}

int launch_partial_sum(const float* partial, int64_t blocks, int rows, int64_t d, float* out0, float* out1, hipStream_t s) {
  partial_sum_kernel<<<unsigned(rows * d / 16), 1024, 0, s>>>(partial, int(blocks), rows, int(d), out0, out1);
  return int(hipGetLastError());
}

}  // namespace

int launch_qk_norm_fwd(const QkNormProblem& p, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  int64_t blocks;
  const QkNorm n = qk_params(p);
  return p.a.dtype == GDN_DTYPE_BF16 ? launch_qk<__bf16, __bf16, false>(n, p, 0, &blocks, s)
                                     : launch_qk<float, float, false>(n, p, 0, &blocks, s);
}

int launch_qk_norm_bwd(const QkNormProblem& p, const gdn_qk_norm_grads& g, void* ws, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  QkNorm n = qk_params(p);
  n.dq_out = g.dq_out, n.dk_out = g.dk_out, n.dq = g.dq, n.dk = g.dk;
  n.partial = static_cast<float*>(ws);
  int64_t blocks = 0;
  int rc;
  if (p.a.dtype == GDN_DTYPE_F32)
    rc = launch_qk<float, float, true>(n, p, kNormPartials, &blocks, s);
  else if (g.grad_dtype == GDN_DTYPE_F32)
    rc = launch_qk<__bf16, float, true>(n, p, kNormPartials, &blocks, s);
  else
    rc = launch_qk<__bf16, __bf16, true>(n, p, kNormPartials, &blocks, s);
  if (rc != 0 || (g.dwq == nullptr && g.dwk == nullptr)) return rc;
  return launch_partial_sum(n.partial, blocks, 2, p.a.d, g.dwq, g.dwk, s);
}

int launch_gated_norm_fwd(const GatedNormProblem& p, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  int64_t blocks;
  const GatedNorm n = gated_params(p);
  return p.a.dtype == GDN_DTYPE_BF16 ? launch_gated<__bf16, false>(n, p, 0, &blocks, s)
                                     : launch_gated<float, false>(n, p, 0, &blocks, s);
}

int launch_gated_norm_bwd(const GatedNormProblem& p, const gdn_gated_norm_grads& g, void* ws, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  GatedNorm n = gated_params(p);
  n.dy = g.dy, n.dx = g.dx, n.dgate = g.dgate;
  n.partial = static_cast<float*>(ws);
  int64_t blocks = 0;
  const int rc = p.a.dtype == GDN_DTYPE_BF16 ? launch_gated<__bf16, true>(n, p, kNormPartials, &blocks, s)
                                             : launch_gated<float, true>(n, p, kNormPartials, &blocks, s);
  if (rc != 0 || g.dweight == nullptr) return rc;
  return launch_partial_sum(n.partial, blocks, 1, p.a.d, g.dweight, nullptr, s);
}

}  // namespace gdn
