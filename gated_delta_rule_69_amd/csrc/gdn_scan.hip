// The gated recurrence a channel: how a sequence is cut into segments, the workspaces, and
// the launches' order.
#include "gdn_scan_pass.h"

namespace gdn {
namespace {

using scan::Pass;
using scan::Run;

int64_t slices_of(const gdn_scan_args& a, bool back) {
  const int64_t row = back ? scan::Geo<scan::kBackLanes>::kRow : scan::Geo<scan::kLanes>::kRow;
  return (a.C * (a.dtype == GDN_DTYPE_BF16 ? 2 : 4) + row - 1) / row;
}
constexpr int64_t kGroups = 256;   // workgroups that fill the CUs
int64_t spans_of(int64_t T) { return (T + scan::kSpan - 1) / scan::kSpan; }

// Segments of a sequence and the tokens of each. A workgroup walks its segment; where slices and
// sequences alone leave CUs idle, segments of two tiles and more run side by side, at the price of a
// first pass over the inputs for what each makes of the state (B2 T32768 C2048 bf16: 512 and 1,024
// workgroups 223 and 268 us against 205 with 256; 300 tokens in one walk 13.1 against 16.4).
void cut(const gdn_scan_args& a, bool back, unsigned* segs, int64_t* seg) {
  const int64_t tile = back ? scan::kBackTile : scan::kTile;
  const int64_t tiles = std::max<int64_t>(1, (a.T + tile - 1) / tile);
  const int64_t walks = a.B * slices_of(a, back);
  const int64_t want = std::min<int64_t>((tiles + 1) / 2, std::max<int64_t>(1, kGroups / walks));
  const int64_t each = (tiles + want - 1) / want;
  *segs = unsigned((tiles + each - 1) / each);
  *seg = each * tile;
}

Pass pass_of(const gdn_scan_args& a, bool back) {
  const int64_t es = a.dtype == GDN_DTYPE_BF16 ? 2 : 4;
  Pass p{};
  p.x = a.x, p.f = a.f, p.i = a.i, p.decay = a.decay, p.lens = a.seq_lens;
  p.h0 = a.h0, p.h_final = a.h_final, p.marks = a.checkpoints, p.h = a.h;
  p.ldx = a.x_stride * es, p.ldf = a.f_stride * es, p.ldi = a.i_stride * es;
  p.T = a.T, p.C = a.C;
  cut(a, back, &p.segs, &p.seg);
  return p;
}

size_t rounded(size_t bytes) { return (bytes + 255) / 256 * 256; }
size_t totals_bytes(const gdn_scan_args& a, bool back) {
  unsigned segs;
  int64_t seg;
  cut(a, back, &segs, &seg);
  return rounded(size_t(a.B) * (segs - 1) * a.C * sizeof(Run));
}
size_t start_bytes(const gdn_scan_args& a) { return rounded(size_t(a.B) * a.C * sizeof(float)); }
size_t marks_bytes(const gdn_scan_args& a) {
  return a.checkpoints != nullptr ? 0 : rounded(size_t(a.B) * spans_of(a.T) * a.C * sizeof(float));
}
size_t sums_bytes(const gdn_scan_args& a) {
  unsigned segs;
  int64_t seg;
  cut(a, true, &segs, &seg);
  return a.gate == GDN_SCAN_POWER ? rounded(size_t(a.B) * segs * a.C * sizeof(float)) : 0;
}

int token_by_token(const ScanProblem& q, Pass p, hipStream_t s) {
  p.blocks = unsigned(q.a.B * q.a.C / 4);
  return q.a.dtype == GDN_DTYPE_BF16 ? scan::step_bf16(q, p, s) : scan::step_f32(q, p, s);
}

// Few tokens go one by one: 0.35 us each, where a tile takes 8 us for every 256 workgroups (C 2048, bf16
// with an input gate, one by one against tiles: one sequence of 8 tokens 5.2 against 7.9 us and of 24 10.6
// against 7.9; 64 sequences of 64 tokens 30 against 55 and of 96 44 against 56).
bool few(const gdn_scan_args& a) {
  const int64_t rounds = (a.B * slices_of(a, false) + kGroups - 1) / kGroups;
  return a.T <= 16 * std::min<int64_t>(rounds, 8);
}

int forward(const ScanProblem& q, Pass p, char* ws, hipStream_t s) {
  if (few(q.a)) return token_by_token(q, p, s);
  p.start = reinterpret_cast<float*>(ws);
  p.totals = reinterpret_cast<Run*>(ws + start_bytes(q.a));
  return q.a.dtype == GDN_DTYPE_BF16 ? scan::fwd_bf16(q, p, s) : scan::fwd_f32(q, p, s);
}

}  // namespace

size_t scan_fwd_workspace(const ScanProblem& q) { return start_bytes(q.a) + totals_bytes(q.a, false); }

int launch_scan_fwd(const ScanProblem& q, void* ws, void* stream) {
  return forward(q, pass_of(q.a, false), static_cast<char*>(ws), static_cast<hipStream_t>(stream));
}

int launch_scan_step(const ScanProblem& q, const float* before, float* after, void* stream) {
  Pass p = pass_of(q.a, false);
  p.h0 = before, p.h_final = after, p.marks = nullptr;
  return token_by_token(q, p, static_cast<hipStream_t>(stream));
}

// Gradients' workspace: the forward pass's or the totals from the end, the states before the
// spans where they are not given, and the segments' sums for ddecay.
size_t scan_bwd_workspace(const ScanProblem& q) {
  return std::max(scan_fwd_workspace(q), totals_bytes(q.a, true)) + marks_bytes(q.a) + sums_bytes(q.a);
}

int launch_scan_bwd(const ScanProblem& q, const void* d_h, const float* d_h_final, const gdn_scan_grads& g, void* ws,
                    void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  char* at = static_cast<char*>(ws);
  float* marks = reinterpret_cast<float*>(at + std::max(scan_fwd_workspace(q), totals_bytes(q.a, true)));
  float* sums = marks + marks_bytes(q.a) / sizeof(float);
  Pass p = pass_of(q.a, true);
  if (p.marks == nullptr) {
    p.marks = marks;
    if (q.a.T > 0) {
      Pass first = pass_of(q.a, false);
      first.h = nullptr, first.h_final = nullptr, first.marks = marks;
      const int rc = forward(q, first, at, s);
      if (rc != 0) return rc;
    }
  }
  p.totals = reinterpret_cast<Run*>(at);
  p.d_h = d_h, p.d_final = d_h_final;
  p.dx = g.dx, p.df = g.df, p.di = g.di, p.dh0 = g.dh0;
  p.ddecay = g.ddecay == nullptr ? nullptr : sums;
  const int rc = q.a.dtype == GDN_DTYPE_BF16 ? scan::bwd_bf16(q, p, s) : scan::bwd_f32(q, p, s);
  if (rc != 0 || g.ddecay == nullptr) return rc;
  return launch_column_sum({sums, int(q.a.B * p.segs), q.a.C, q.a.C, 0, g.ddecay, nullptr, nullptr}, s);
}

}  // namespace gdn
