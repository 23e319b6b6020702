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
// memory bounds it, and the state's rows of a slice are whole 128-byte lines. The slices of
// a state lie in one workgroup, so that its rows are read whole by one CU (512 sequences of
// 16 heads, d 128: 205 us against 212 with two slices a workgroup and 217 with one). Now 202
// us, 5.36 TB/s (a copy of 512 MiB: 5.39).
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
  unsigned waves;  // slices of all states
};
constexpr int kSeqWaves = 4;

// ONE: a call of one token, whose state takes hi and lo. In longer ones a token's factor is hi
// and what those before left out, as soon as that is half a step, and the state takes the rest
// in the end (hi and lo at every token: 33 us against 27 for 8 tokens of 1024 heads of 128).
template <typename E, int DK, int W, bool ONE>
__global__ __launch_bounds__(64 * kSeqWaves) void linear_seq_kernel(LinearSeq a) {
  constexpr int LC = W / 4;          // lanes across the slice's columns
  constexpr int G = 64 / LC;         // lane groups
  constexpr int NR = DK / G;         // rows a lane holds
  const unsigned wave = __builtin_amdgcn_readfirstlane(blockIdx.x * kSeqWaves + threadIdx.x / 64);
  if (wave >= a.waves) return;
  const int lane = threadIdx.x % 64, j = lane % LC, g = lane / LC;
  const unsigned slices = unsigned(a.dv) / W;
  const int64_t bh = wave / slices;
  const int col = int(wave % slices) * W + 4 * j;
  const int64_t b = bh / a.H;
  const int h = int(bh - b * a.H);
  const int64_t n = length_of(a.seq_lens, b, a.T);
  float decay, decay_lo;
  two_floats(head_log_decay(a.log_decay, h), &decay, &decay_lo);
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
  float left = 0.0f;  // of the decay, not in the state yet
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
    left += decay_lo;
    float by = decay;
    if constexpr (!ONE) {
      by += left;
      left -= by - decay;
    }
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float add = kv[r] * vv[c];
        S[r][c] = S[r][c] * by + (ONE ? S[r][c] * left + add : add);
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
  if (!ONE && left != 0.0f) {
    left /= decay;
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
      for (int c = 0; c < 4; ++c) S[r][c] += S[r][c] * left;
  }
  if (a.s1 != nullptr && !(n == 0 && a.s1 == a.s0)) {
#pragma unroll
    for (int r = 0; r < NR; ++r) store4(a.s1 + at + int64_t(r) * a.dv, S[r]);
  }
}

template <typename E, int W, bool ONE>
int launch_seq(const LinearProblem& p, const LinearSeq& a, hipStream_t s) {
  const unsigned grid = (a.waves + kSeqWaves - 1) / kSeqWaves;
  switch (p.dk) {
    case 16: linear_seq_kernel<E, 16, W, ONE><<<grid, 64 * kSeqWaves, 0, s>>>(a); break;
    case 32: linear_seq_kernel<E, 32, W, ONE><<<grid, 64 * kSeqWaves, 0, s>>>(a); break;
    case 64: linear_seq_kernel<E, 64, W, ONE><<<grid, 64 * kSeqWaves, 0, s>>>(a); break;
    case 128: linear_seq_kernel<E, 128, W, ONE><<<grid, 64 * kSeqWaves, 0, s>>>(a); break;
    default: return int(hipErrorInvalidValue);
  }
  return int(hipGetLastError());
}

template <typename E>
int launch_seq(const LinearProblem& p, const LinearSeq& a, hipStream_t s) {
  if (p.T == 1) return p.dv == 16 ? launch_seq<E, 16, true>(p, a, s) : launch_seq<E, 32, true>(p, a, s);
  return p.dv == 16 ? launch_seq<E, 16, false>(p, a, s) : launch_seq<E, 32, false>(p, a, s);
}

int launch_seq(const LinearProblem& p, const float* s0, float* s1, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  const LinearSeq a{p.q, p.k, p.v, p.log_decay, p.seq_lens, s0, s1, p.o, p.T,
                    p.ldq, p.ldk, p.ldv, int(p.H), int(p.group), int(p.dv), unsigned(p.B * p.H * (p.dv == 16 ? 1 : p.dv / 32))};
  return p.dtype == GDN_DTYPE_BF16 ? launch_seq<__bf16>(p, a, s) : launch_seq<float>(p, a, s);
}

}  // namespace

int launch_linear_step(const LinearProblem& p, float* state, void* stream) {
  return launch_seq(p, state, state, stream);
}

namespace {

// slot[s] += l^{positions of segment s - 1} slot[s - 1] along the segments of a (b, h): the
// workgroup's slice of 1024 floats of its state, in the order the passes left it.
__global__ __launch_bounds__(256) void scan_states_kernel(LinearPasses all, int per_state) {
  const LinearPass s = all.pass[blockIdx.y];
  const int parts = (per_state + 1023) / 1024;
  const int64_t bh = blockIdx.x / parts;
  const int at = int(blockIdx.x % parts) * 1024 + 4 * threadIdx.x;
  if (at >= per_state) return;
  const int64_t n = length_of(s.seq_lens, bh / s.H, s.T);
  const float lg = head_log_decay(s.log_decay, int(bh % s.H));
  // a segment that leaves nothing of the one before: every state is its segment's own already
  float whole, whole_lo;
  two_floats(lg * float(s.seg), &whole, &whole_lo);
  if (n > (s.nseg - 1) * s.seg && whole == 0.0f) return;
  float* slot = s.states + bh * s.nseg * per_state + at;
  float x[4];
  load4(slot + per_state, x);
  // sixteen segments' loads at a time: the chain itself is one multiplication and addition each
  constexpr int N = 16;
  for (int seg = 2; seg < s.nseg; seg += N) {
    float y[N][4];
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (seg + k < s.nseg) load4(slot + int64_t(seg + k) * per_state, y[k]);
#pragma unroll
    for (int k = 0; k < N; ++k) {
      if (seg + k >= s.nseg) break;
      const int64_t left = n - (seg + k - 1) * s.seg;
      float w = whole, w_lo = whole_lo;
      if (left < s.seg) two_floats(lg * float(left < 0 ? 0 : left), &w, &w_lo);
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = w * x[e] + (w_lo * x[e] + y[k][e]);
      store4(slot + int64_t(seg + k) * per_state, x);
    }
  }
}

// Segments of `passes` passes that share a launch: as many workgroups as the 256 CUs hold at
// once (by LDS, and by registers 16 waves a CU in bf16 and 12 in float32), a third more of a
// padded batch, where some find nothing to do; each at least four chunks (three of float32).
// Measured at bf16 d 128: B2 T32768 H16 forward with 256 / 512 / 768 / 1024 workgroups 417 /
// 378 / 435 / 408 us; B2 T4096 gradients with 170 / 256 / 512 a pass 135 / 152 / 170 us; B1
// T4096 forward with 2 / 4 / 8 chunks at least 54 / 47 / 63 us. Padded float32 B8 T2047 H32
// d64 with 768 / 1024 / 1536: 145 / 130 / 141 us.
struct Segments {
  int64_t tokens, count;
};
Segments choose_segments(const LinearProblem& p, int da, int dc, int passes) {
  const bool half = p.dtype == GDN_DTYPE_BF16;
  const int64_t C = half ? 64 : 32;
  const int64_t resident = std::max<int64_t>(1, std::min<int64_t>((160 << 10) / outputs_lds(half, da, dc), (half ? 16 : 12) / pass_waves(dc)));
  const int64_t wanted = 256 * resident * (p.seq_lens != nullptr ? 4 : 3) / 3;
  const int64_t chunks = (p.T + C - 1) / C;
  const int64_t want = std::max<int64_t>(1, wanted / (p.B * p.H * passes));
  const int64_t each = std::max<int64_t>(half ? 4 : 3, (chunks + want - 1) / want);
  return {each * C, std::max<int64_t>(1, (chunks + each - 1) / each)};
}
Segments forward_segments(const LinearProblem& p) { return choose_segments(p, int(p.dk), int(p.dv), 1); }
// dq, dk and dv in one launch where they can be, else dq and dk
Segments backward_segments(const LinearProblem& p) {
  return choose_segments(p, int(p.dv), int(p.dk), p.dk == p.dv && p.group == 1 ? 3 : 2);
}

int launch_pass(const LinearPasses& s, int count, const LinearProblem& p, int da, int dc, bool out, bool wide_out, void* stream) {
  return p.dtype == GDN_DTYPE_BF16 ? launch_pass_bf16(s, count, p.B, da, dc, out, wide_out, stream)
                                   : launch_pass_f32(s, count, p.B, da, dc, out, stream);
}

// The states before every segment of `count` passes (nothing to do for one segment): the
// segments' own, then their joining.
int launch_states(const LinearPasses& s, int count, const LinearProblem& p, int da, int dc, void* stream) {
  const LinearPass& first = s.pass[0];
  if (first.nseg == 1) return 0;
  const int rc = launch_pass(s, count, p, da, dc, false, false, stream);
  if (rc != 0 || first.nseg == 2) return rc;
  const dim3 grid(unsigned(p.B * p.H * ((da * dc + 1023) / 1024)), unsigned(count));
  scan_states_kernel<<<grid, 256, 0, static_cast<hipStream_t>(stream)>>>(s, da * dc);
  return int(hipGetLastError());
}

LinearPass base_pass(const LinearProblem& p, const Segments& segments) {
  LinearPass s{};
  s.H = int(p.H), s.T = p.T;
  s.log_decay = p.log_decay, s.seq_lens = p.seq_lens;
  s.seg = segments.tokens, s.nseg = int(segments.count);
  return s;
}

// Bytes of a pass's states, a multiple of 256.
size_t states_bytes(const LinearProblem& p, const Segments& segments) {
  if (segments.count == 1) return 256;
  return size_t(p.B) * size_t(p.H) * size_t(segments.count) * size_t(p.dk) * size_t(p.dv) * sizeof(float);
}

}  // namespace

size_t linear_fwd_workspace(const LinearProblem& p) { return states_bytes(p, forward_segments(p)); }

int launch_linear_fwd(const LinearProblem& p, void* ws, void* stream) {
  // Up to eight tokens go one by one: 4 to 8 us against a chunk's 7 to 10 for 16 heads of 128
  // or 32 of 64 (both take 10 to 12 tokens for the same), 27 against 32 us for 1024 heads.
  if (p.T <= 8) return launch_seq(p, p.s0, p.s_final, stream);
  LinearPasses all{};
  LinearPass& s = all.pass[0];
  s = base_pass(p, forward_segments(p));
  s.a = p.q, s.b = p.k, s.c = p.v, s.out = p.o;
  s.lda = p.ldq, s.ldb = p.ldk, s.ldc = p.ldv;
  s.group_a = s.group_b = int(p.group), s.group_c = 1;
  s.x0 = p.s0, s.x1 = p.s_final, s.x0_sa = p.dv, s.x0_sc = 1;
  s.states = static_cast<float*>(ws), s.st_sa = 1, s.st_sc = p.dk;
  const int rc = launch_states(all, 1, p, int(p.dk), int(p.dv), stream);
  return rc != 0 ? rc : launch_pass(all, 1, p, int(p.dk), int(p.dv), true, false, stream);
}

namespace {

// out[row] = the sum of `group` rows of in, for rows of d channels, rounded once.
template <typename E>
__global__ __launch_bounds__(256) void group_sum_kernel(const float* in0, const float* in1, E* out0, E* out1, int64_t n, int d, int group) {
  const float* in = blockIdx.y == 0 ? in0 : in1;
  E* out = blockIdx.y == 0 ? out0 : out1;
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

// Where key heads are shared, dq and dk of every value head come first, in float32.
size_t per_head_bytes(const LinearProblem& p) {
  return p.group > 1 ? size_t(p.B) * size_t(p.T) * size_t(p.H) * size_t(p.dk) * sizeof(float) : 0;
}

}  // namespace

size_t linear_bwd_workspace(const LinearProblem& p) {
  return 2 * (states_bytes(p, backward_segments(p)) + per_head_bytes(p));
}

// Gradients: the states S before every segment and, backwards, G behind it, both transposed
// ([dv] rows, as dq and dk take them); then the outputs of dq, dk and dv, in one launch
// where their dimensions and types are the same.
int launch_linear_bwd(const LinearProblem& p, const LinearGrads& g, void* ws, void* stream) {
  hipStream_t hs = static_cast<hipStream_t>(stream);
  const int dk = int(p.dk), dv = int(p.dv), group = int(p.group);
  const bool shared = group > 1;
  char* mem = static_cast<char*>(ws);
  const Segments segments = backward_segments(p);
  const size_t states = states_bytes(p, segments);
  float* per_head[2] = {reinterpret_cast<float*>(mem + 2 * states),
                        reinterpret_cast<float*>(mem + 2 * states + per_head_bytes(p))};
  const int64_t ldo = p.H * p.dv;
  LinearPasses all{};
  LinearPass &q = all.pass[0], &k = all.pass[1], &v = all.pass[2];
  q = base_pass(p, segments);
  q.zero_tail = p.seq_lens != nullptr;
  k = v = q;
  k.back = v.back = k.shift = v.shift = 1;
  // dq = S do: rows (do, v, k)
  q.a = g.d_o, q.b = p.v, q.c = p.k, q.out = shared ? per_head[0] : g.dq;
  q.lda = ldo, q.ldb = p.ldv, q.ldc = p.ldk;
  q.group_a = q.group_b = 1, q.group_c = group;
  q.x0 = p.s0, q.states = reinterpret_cast<float*>(mem);
  // dk = G v: rows (v, do, q)
  k.a = p.v, k.b = g.d_o, k.c = p.q, k.out = shared ? per_head[1] : g.dk;
  k.lda = p.ldv, k.ldb = ldo, k.ldc = p.ldq;
  k.group_a = k.group_b = 1, k.group_c = group;
  k.x0 = g.d_s_final, k.states = reinterpret_cast<float*>(mem + states);
  q.x0_sa = k.x0_sa = 1, q.x0_sc = k.x0_sc = p.dv;
  q.st_sa = k.st_sa = 1, q.st_sc = k.st_sc = p.dv;
  // dv = G^T k: rows (k, q, do), G as dk's states have it; its last state is ds0
  v.a = p.k, v.b = p.q, v.c = g.d_o, v.out = g.dv;
  v.lda = p.ldk, v.ldb = p.ldq, v.ldc = ldo;
  v.group_a = v.group_b = group, v.group_c = 1;
  v.x0 = g.d_s_final, v.x1 = g.ds0, v.x0_sa = p.dv, v.x0_sc = 1;
  v.states = k.states, v.st_sa = p.dv, v.st_sc = 1;

  int rc = launch_states(all, 2, p, dv, dk, stream);
  if (rc != 0) return rc;
  const bool one = dk == dv && !shared;
  if ((rc = launch_pass(all, one ? 3 : 2, p, dv, dk, true, shared, stream)) != 0) return rc;
  if (!one) {
    LinearPasses last{};
    last.pass[0] = v;
    if ((rc = launch_pass(last, 1, p, dk, dv, true, false, stream)) != 0) return rc;
  }
  const int64_t n = p.B * p.T * p.Hk * p.dk;
  if (!shared || n == 0) return 0;
  const dim3 grid(unsigned((n + 1023) / 1024), 2);
  if (p.dtype == GDN_DTYPE_BF16)
    group_sum_kernel<<<grid, 256, 0, hs>>>(per_head[0], per_head[1], static_cast<__bf16*>(g.dq), static_cast<__bf16*>(g.dk), n, dk, group);
  else
    group_sum_kernel<<<grid, 256, 0, hs>>>(per_head[0], per_head[1], static_cast<float*>(g.dq), static_cast<float*>(g.dk), n, dk, group);
  return int(hipGetLastError());
}

}  // namespace gdn
