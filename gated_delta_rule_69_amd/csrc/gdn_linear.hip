// Linear attention with one decay a head, token by token:
//     S <- e^g S + k_t v_t^T,   o_t = S^T q_t
//
// One wave owns a slice of W = min(dv, 32) value columns of one (sequence, head) state, in
// registers for all of its tokens: W/4 lanes cover a state row of the slice with 16-byte
// vectors, and the wave's 256/W lane groups hold dk W / 256 rows each. A group's rows are
// contiguous, so a lane reads its part of q and k as vectors. The sum of o over key rows
// is a partial sum a lane and the exchanges across lane groups.
//
// One token moves the state once each way, 8 dk dv bytes a head against 4 dk dv flops:
// memory bounds it, and the state's rows of a slice are whole 128-byte lines.
#include "gdn_layer.h"
#include "gdn_layer_device.h"

namespace gdn {
namespace {

struct LinearSeq {
  const void *q, *k, *v;
  const float* log_decay;
  const int32_t* seq_lens;
  const float* s0;
  float* s1;
  void* o;
  int64_t T, ldq, ldk, ldv;
  int H, group, dv;
};

// Decay of a head: e^g, with everything below e^-128 taken as 0 (so that -Inf works).
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

template <typename E, int DK, int W>
__global__ __launch_bounds__(64) void linear_seq_kernel(LinearSeq a) {
  constexpr int LC = W / 4;          // lanes across the slice's columns
  constexpr int G = 64 / LC;         // lane groups
  constexpr int NR = DK / G;         // rows a lane holds
  const int j = threadIdx.x % LC, g = threadIdx.x / LC;
  const int slices = a.dv / W;
  const int64_t bh = blockIdx.x / slices;
  const int col = int(blockIdx.x % slices) * W + 4 * j;
  const int64_t b = bh / a.H;
  const int h = int(bh - b * a.H);
  const int64_t n = length_of(a.seq_lens, b, a.T);
  const float decay = expf(head_log_decay(a.log_decay, h));
  const int64_t at = (bh * DK + g * NR) * a.dv + col;

  float S[NR][4];
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    if (a.s0 != nullptr) {
      load4(a.s0 + at + int64_t(r) * a.dv, S[r]);
    } else {
      S[r][0] = S[r][1] = S[r][2] = S[r][3] = 0.0f;
    }
  }
  const E* q = static_cast<const E*>(a.q) + b * a.T * a.ldq + (h / a.group) * DK + g * NR;
  const E* k = static_cast<const E*>(a.k) + b * a.T * a.ldk + (h / a.group) * DK + g * NR;
  const E* v = static_cast<const E*>(a.v) + b * a.T * a.ldv + int64_t(h) * a.dv + col;
  E* o = static_cast<E*>(a.o) + (b * a.T * a.H + h) * a.dv + col;
  for (int64_t t = 0; t < n; ++t) {
    float qv[NR], kv[NR], vv[4], ov[4] = {};
    if constexpr (NR % 4 == 0) {
#pragma unroll
      for (int r = 0; r < NR; r += 4) load4(q + r, qv + r), load4(k + r, kv + r);
    } else {
#pragma unroll
      for (int r = 0; r < NR; ++r) qv[r] = float(q[r]), kv[r] = float(k[r]);
    }
    load4(v, vv);
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        S[r][c] = S[r][c] * decay + kv[r] * vv[c];
        ov[c] += qv[r] * S[r][c];
      }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if constexpr (LC <= 4) ov[c] += dpp<0x124>(ov[c]);  // row_ror:4, then the sum over 8: lanes l ^ 4 m
      if constexpr (LC <= 8) ov[c] += dpp<0x128>(ov[c]);  // row_ror:8
      ov[c] = sum_over_groups(ov[c]);
    }
    if (g == 0) store4(o, ov);
    q += a.ldq, k += a.ldk, v += a.ldv, o += int64_t(a.H) * a.dv;
  }
  if (a.s1 != nullptr && !(n == 0 && a.s1 == a.s0)) {
#pragma unroll
    for (int r = 0; r < NR; ++r) store4(a.s1 + at + int64_t(r) * a.dv, S[r]);
  }
}

template <typename E, int W>
int launch_seq(const LinearProblem& p, const LinearSeq& a, hipStream_t s) {
  const unsigned grid = unsigned(p.B * p.H * (p.dv / W));
  switch (p.dk) {
    case 16: linear_seq_kernel<E, 16, W><<<grid, 64, 0, s>>>(a); break;
    case 32: linear_seq_kernel<E, 32, W><<<grid, 64, 0, s>>>(a); break;
    case 64: linear_seq_kernel<E, 64, W><<<grid, 64, 0, s>>>(a); break;
    case 128: linear_seq_kernel<E, 128, W><<<grid, 64, 0, s>>>(a); break;
    default: return int(hipErrorInvalidValue);
  }
  return int(hipGetLastError());
}

int launch_seq(const LinearProblem& p, const float* s0, float* s1, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  const LinearSeq a{p.q, p.k, p.v, p.log_decay, p.seq_lens, s0, s1, p.o, p.T,
                    p.ldq, p.ldk, p.ldv, int(p.H), int(p.group), int(p.dv)};
  if (p.dtype == GDN_DTYPE_BF16)
    return p.dv == 16 ? launch_seq<__bf16, 16>(p, a, s) : launch_seq<__bf16, 32>(p, a, s);
  return p.dv == 16 ? launch_seq<float, 16>(p, a, s) : launch_seq<float, 32>(p, a, s);
}

}  // namespace

int launch_linear_step(const LinearProblem& p, float* state, void* stream) {
  return launch_seq(p, state, state, stream);
}

int launch_linear_fwd(const LinearProblem& p, void* ws, void* stream) {
  return launch_seq(p, p.s0, p.s_final, stream);
}
size_t linear_fwd_workspace(const LinearProblem& p) { return 256; }

}  // namespace gdn
