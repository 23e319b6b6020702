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
#include <algorithm>

#include "gdn_linear_pass.h"

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

namespace {

// slot[s] += l^{positions of segment s - 1} slot[s - 1] along the segments of a (b, h): the
// workgroup's slice of 1024 floats of its state, in the order the passes left it.
__global__ __launch_bounds__(256) void scan_states_kernel(LinearPass s, int per_state) {
  const int parts = (per_state + 1023) / 1024;
  const int64_t bh = blockIdx.x / parts;
  const int at = int(blockIdx.x % parts) * 1024 + 4 * threadIdx.x;
  if (at >= per_state) return;
  const int64_t n = length_of(s.seq_lens, bh / s.H, s.T);
  const float lg = head_log_decay(s.log_decay, int(bh % s.H));
  float* slot = s.states + bh * s.nseg * per_state + at;
  float x[4];
  load4(slot + per_state, x);
  // eight segments' loads at a time: the chain itself is one multiplication and addition each
  for (int seg = 2; seg < s.nseg; seg += 8) {
    float y[8][4];
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (seg + k < s.nseg) load4(slot + int64_t(seg + k) * per_state, y[k]);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (seg + k >= s.nseg) break;
      const int64_t left = n - (seg + k - 1) * s.seg;
      const float w = expf(lg * float(left < 0 ? 0 : left > s.seg ? s.seg : left));
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = y[k][e] + w * x[e];
      store4(slot + int64_t(seg + k) * per_state, x);
    }
  }
}

int launch_scan(const LinearPass& s, int64_t B, int per_state, hipStream_t stream) {
  if (s.nseg <= 2) return 0;
  scan_states_kernel<<<unsigned(B * s.H * ((per_state + 1023) / 1024)), 256, 0, stream>>>(s, per_state);
  return int(hipGetLastError());
}

// Segments: enough workgroups for two on each of the 256 CUs, of at least four chunks.
void choose_segments(const LinearProblem& p, int64_t* seg, int64_t* nseg) {
  const int64_t C = p.dtype == GDN_DTYPE_BF16 ? 64 : 32;
  const int64_t chunks = (p.T + C - 1) / C;
  const int64_t want = std::max<int64_t>(1, 512 / (p.B * p.H));
  const int64_t each = std::max<int64_t>(4, (chunks + want - 1) / want);
  *seg = each * C;
  *nseg = std::max<int64_t>(1, (chunks + each - 1) / each);
}

// A pass from its start states to its outputs: the segments' own states, their joining, and
// the outputs (one launch where there is one segment).
int run_pass(const LinearPass& s, const LinearProblem& p, int da, int dc, bool rev, bool wide_out, void* stream) {
  auto launch = [&](bool out) {
    return p.dtype == GDN_DTYPE_BF16 ? launch_pass_bf16(s, p.B, da, dc, rev, out, wide_out, stream)
                                     : launch_pass_f32(s, p.B, da, dc, rev, out, stream);
  };
  int rc = 0;
  if (s.nseg > 1) {
    if ((rc = launch(false)) != 0) return rc;
    if ((rc = launch_scan(s, p.B, da * dc, static_cast<hipStream_t>(stream))) != 0) return rc;
  }
  return launch(true);
}

LinearPass base_pass(const LinearProblem& p) {
  LinearPass s{};
  s.H = int(p.H), s.T = p.T;
  s.log_decay = p.log_decay, s.seq_lens = p.seq_lens;
  int64_t nseg;
  choose_segments(p, &s.seg, &nseg);
  s.nseg = int(nseg);
  return s;
}

size_t states_bytes(const LinearProblem& p) {
  int64_t seg, nseg;
  choose_segments(p, &seg, &nseg);
  return nseg > 1 ? size_t(p.B) * size_t(p.H) * size_t(nseg) * size_t(p.dk) * size_t(p.dv) * sizeof(float) : 256;
}

}  // namespace

size_t linear_fwd_workspace(const LinearProblem& p) { return states_bytes(p); }

int launch_linear_fwd(const LinearProblem& p, void* ws, void* stream) {
  LinearPass s = base_pass(p);
  s.a = p.q, s.b = p.k, s.c = p.v, s.out = p.o;
  s.lda = p.ldq, s.ldb = p.ldk, s.ldc = p.ldv;
  s.group_a = s.group_b = int(p.group), s.group_c = 1;
  s.x0 = p.s0, s.x1 = p.s_final, s.x0_sa = p.dv, s.x0_sc = 1;
  s.states = static_cast<float*>(ws), s.st_sa = 1, s.st_sc = p.dk;
  return run_pass(s, p, int(p.dk), int(p.dv), false, false, stream);
}

namespace {

// out[row] = the sum of `group` rows of in, for rows of d channels, rounded once.
template <typename E>
__global__ __launch_bounds__(256) void group_sum_kernel(const float* in, E* out, int64_t n, int d, int group) {
  const int64_t at = (int64_t(blockIdx.x) * 256 + threadIdx.x) * 4;
  if (at >= n) return;
  const int64_t row = at / d;
  const float* from = in + row * group * d + (at - row * d);
  float x[4], y[4];
  load4(from, x);
  for (int k = 1; k < group; ++k) {
    load4(from + int64_t(k) * d, y);
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] += y[e];
  }
  store4(out + at, x);
}

size_t per_head_bytes(const LinearProblem& p) {
  return p.group > 1 ? size_t(p.B) * size_t(p.T) * size_t(p.H) * size_t(p.dk) * sizeof(float) : 0;
}
size_t round256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

size_t linear_bwd_workspace(const LinearProblem& p) { return round256(states_bytes(p)) + per_head_bytes(p); }

int launch_linear_bwd(const LinearProblem& p, const LinearGrads& g, void* ws, void* stream) {
  hipStream_t hs = static_cast<hipStream_t>(stream);
  const int dk = int(p.dk), dv = int(p.dv), group = int(p.group);
  const bool shared = group > 1;
  float* per_head = reinterpret_cast<float*>(static_cast<char*>(ws) + round256(states_bytes(p)));
  const int64_t ldo = p.H * p.dv;
  auto sum_groups = [&](void* out) {
    const int64_t n = p.B * p.T * p.Hk * p.dk;
    if (!shared || n == 0) return 0;
    const unsigned grid = unsigned((n + 1023) / 1024);
    if (p.dtype == GDN_DTYPE_BF16)
      group_sum_kernel<<<grid, 256, 0, hs>>>(per_head, static_cast<__bf16*>(out), n, dk, group);
    else
      group_sum_kernel<<<grid, 256, 0, hs>>>(per_head, static_cast<float*>(out), n, dk, group);
    return int(hipGetLastError());
  };
  LinearPass s = base_pass(p);
  s.states = static_cast<float*>(ws);
  s.zero_tail = p.seq_lens != nullptr;
  int rc;
  // dq = S do: rows (do, v, k) with the transposed state
  s.a = g.d_o, s.b = p.v, s.c = p.k, s.out = shared ? per_head : g.dq;
  s.lda = ldo, s.ldb = p.ldv, s.ldc = p.ldk;
  s.group_a = s.group_b = 1, s.group_c = group;
  s.x0 = p.s0, s.x0_sa = 1, s.x0_sc = p.dv;
  s.st_sa = 1, s.st_sc = p.dv;
  if ((rc = run_pass(s, p, dv, dk, false, shared, stream)) != 0) return rc;
  if ((rc = sum_groups(g.dq)) != 0) return rc;
  // dk = G v backwards: rows (v, do, q), G transposed
  s.shift = 1;
  s.a = p.v, s.b = g.d_o, s.c = p.q, s.out = shared ? per_head : g.dk;
  s.lda = p.ldv, s.ldb = ldo, s.ldc = p.ldq;
  s.x0 = g.d_s_final;
  if ((rc = run_pass(s, p, dv, dk, true, shared, stream)) != 0) return rc;
  if ((rc = sum_groups(g.dk)) != 0) return rc;
  // dv = G^T k backwards: rows (k, q, do); its last state is ds0
  s.a = p.k, s.b = p.q, s.c = g.d_o, s.out = g.dv;
  s.lda = p.ldk, s.ldb = p.ldq, s.ldc = ldo;
  s.group_a = s.group_b = group, s.group_c = 1;
  s.x1 = g.ds0, s.x0_sa = p.dv, s.x0_sc = 1;
  s.st_sa = 1, s.st_sc = p.dk;
  return run_pass(s, p, dk, dv, true, false, stream);
}

}  // namespace gdn
