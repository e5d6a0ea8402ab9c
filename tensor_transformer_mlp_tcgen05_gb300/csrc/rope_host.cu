// Host side of the query/key operators (tp_rope.h): frequencies, validation
// of the views, the choice of the kind of rows and of the tasks.
#include <algorithm>

#include "host_common.cuh"
#include "qk_rows.cuh"
#include "tp_rope.h"

using namespace tpmlp;
using namespace tpmlp::host;

struct tp_rope_handle {
  int d = 0, r = 0, interleaved = 0;
  double amplitude = 1.0;
  double inv_freq[qk::MAX_PAIRS];
  unsigned long long turns[qk::MAX_PAIRS];  // turns per position, 2^-64
};

namespace {

constexpr int MAX_TOKENS = 1 << 28;
constexpr int MAX_HEADS = 65535;

int bad(int code, const char* msg) {
  set_detail_msg(msg);
  return code;
}

// t modulo one in 64-bit fixed point, rounded to the nearest 2^-64.
unsigned long long fixed_fraction(double t) {
  t -= std::nearbyint(t);                   // exact, [-1/2, 1/2]
  const unsigned long long u = static_cast<unsigned long long>(
      std::nearbyint(std::ldexp(std::fabs(t), 64)));
  return t < 0 ? 0ull - u : u;
}

// frac(f / 2 pi) in 64-bit fixed point, within 2^-64 for |f| <= 2^40.  Positions
// are integers, so whole turns drop out.  The error is multiplied by the
// position, so the quotient is made to twice a double's bits: f times 1 / 2 pi
// as a sum of two doubles (off by 2^-110).
unsigned long long fixed_turns(double f) {
  constexpr double HI = 0x1.45f306dc9c883p-3, LO = -0x1.6b01ec5417056p-57;
  // (volatile: the product is rounded here, not fused into what uses it)
  const volatile double product = f * HI;
  const double hi = product;
  const double lo = std::fma(f, LO, std::fma(f, HI, -hi));
  return fixed_fraction(hi) + fixed_fraction(lo);
}

bool positive(double x) { return x > 0 && std::isfinite(x); }

// Dimensions of a view that have more than one step, as (stride, count).
struct Steps {
  long long stride[3];
  long long count[3];
  int n = 0;
  void add(long long s, long long c) {
    if (c > 1) {
      stride[n] = s;
      count[n++] = c;
    }
  }
};

Steps steps_of(const tp_heads& v, int tokens) {
  Steps s;
  s.add(v.token_stride, tokens);
  s.add(v.group_stride, v.heads / v.group);
  s.add(v.head_stride, std::min(v.group, v.heads));
  return s;
}

// One past the last element of the view (elements from data).
long long extent(const tp_heads& v, int tokens, int d) {
  const Steps s = steps_of(v, tokens);
  long long e = d;
  for (int i = 0; i < s.n; ++i) e += s.stride[i] * (s.count[i] - 1);
  return e;
}

// Every (token, head) row of an output has its own elements: the dimensions
// nest, each step at least as long as all that lies inside it.
bool rows_apart(const tp_heads& v, int tokens, int d) {
  Steps s = steps_of(v, tokens);
  for (int i = 0; i < s.n; ++i)
    for (int j = i + 1; j < s.n; ++j)
      if (s.stride[j] < s.stride[i]) {
        std::swap(s.stride[i], s.stride[j]);
        std::swap(s.count[i], s.count[j]);
      }
  long long inside = d;
  for (int i = 0; i < s.n; ++i) {
    if (s.stride[i] < inside) return false;
    inside += s.stride[i] * (s.count[i] - 1);
  }
  return true;
}

// Start of head j inside its token.
long long head_at(const tp_heads& v, int j) {
  return (j / v.group) * v.group_stride + (j % v.group) * v.head_stride;
}

bool same_view(const tp_heads& a, const tp_heads& b, int tokens) {
  if (a.data != b.data || a.heads != b.heads) return false;
  if (tokens > 1 && a.token_stride != b.token_stride) return false;
  if (a.group == b.group)
    return (a.heads == a.group || a.group_stride == b.group_stride) &&
           (a.group == 1 || a.head_stride == b.head_stride);
  for (int j = 0; j < a.heads; ++j)
    if (head_at(a, j) != head_at(b, j)) return false;
  return true;
}

// Two views with the same strides whose dimensions nest: whether an element of
// one, at sum of i_n stride_n, is one of the other, `delta` further and at sum of
// j_n stride_n.  What is left of delta after the outer dimensions has to come from
// the inner ones, which reach less than one outer step: j_n - i_n is one of the
// two quotients around it.  Dimensions in falling order of their strides.
bool lattice_meets(long long delta, const Steps& a, const Steps& b, int n,
                   int d) {
  if (n == a.n) return delta > -d && delta < d;
  const long long s = a.stride[n];
  long long q = -(delta / s);   // delta + q s is the remainder
  for (long long k = q - 1; k <= q + 1; ++k)
    if (k > -a.count[n] && k < b.count[n] && std::llabs(delta + k * s) < s + d &&
        lattice_meets(delta + k * s, a, b, n + 1, d))
      return true;
  return false;
}

void sort_falling(Steps* s) {
  for (int i = 0; i < s->n; ++i)
    for (int j = i + 1; j < s->n; ++j)
      if (s->stride[j] > s->stride[i]) {
        std::swap(s->stride[i], s->stride[j]);
        std::swap(s->count[i], s->count[j]);
      }
}

// Whether two views may share an element (false only if they share none): exact
// for views with the same strides, as those of one buffer have; views with the
// same token stride are compared head by head modulo that stride where every
// head is inside it and the heads lie in rising order; others of one stretch of
// memory are taken to overlap.
bool may_overlap(const tp_heads& a, const tp_heads& b, int tokens, int d,
                 int size) {
  const char* pa = static_cast<const char*>(a.data);
  const char* pb = static_cast<const char*>(b.data);
  if (pa + extent(a, tokens, d) * size <= pb ||
      pb + extent(b, tokens, d) * size <= pa)
    return false;
  if ((pb - pa) % size != 0) return true;
  long long delta = (pb - pa) / size;
  if (rows_apart(a, tokens, d) && rows_apart(b, tokens, d)) {
    Steps sa = steps_of(a, tokens), sb = steps_of(b, tokens);
    sort_falling(&sa);
    sort_falling(&sb);
    bool same = sa.n == sb.n;
    for (int i = 0; same && i < sa.n; ++i) same = sa.stride[i] == sb.stride[i];
    // (nested for the larger of the two counts, too)
    long long inside = d;
    for (int i = sa.n - 1; same && i >= 0; --i) {
      same = sa.stride[i] >= inside;
      inside += sa.stride[i] * (std::max(sa.count[i], sb.count[i]) - 1);
    }
    if (same) return lattice_meets(delta, sa, sb, 0, d);
  }
  const long long ts = tokens > 1 ? a.token_stride : 0;
  if (tokens > 1 && a.token_stride != b.token_stride) return true;
  auto rising = [&](const tp_heads& v) {
    for (int j = 1; j < v.heads; ++j)
      if (head_at(v, j) < head_at(v, j - 1)) return false;
    return ts == 0 || head_at(v, v.heads - 1) + d <= ts;
  };
  if (!rising(a) || !rising(b)) return true;
  if (ts > 0) delta = ((delta % ts) + ts) % ts;
  // b's heads lie delta (and, wrapped into the token before, delta - ts) after
  // a's
  for (int wrap = 0; wrap < (ts > 0 ? 2 : 1); ++wrap) {
    const long long shift = delta - wrap * ts;
    int i = 0, j = 0;
    while (i < a.heads && j < b.heads) {
      const long long x = head_at(a, i), y = head_at(b, j) + shift;
      if (x + d <= y) ++i;
      else if (y + d <= x) ++j;
      else return true;
    }
  }
  return false;
}

bool present(const tp_heads* v) { return v != nullptr && v->heads > 0; }

int check_view(const tp_heads& v, int tokens, int d, int size) {
  if (v.group <= 0 || v.heads > MAX_HEADS || v.heads % v.group != 0)
    return bad(TPMLP_ERR_SHAPE, "heads: 1 <= group, a divisor of at most "
                                "65535 heads");
  if (v.token_stride < 0 || v.group_stride < 0 || v.head_stride < 0)
    return bad(TPMLP_ERR_SHAPE, "heads: negative stride");
  const Steps st = steps_of(v, tokens);
  for (int i = 0; i < st.n; ++i)
    if (st.stride[i] > ((1LL << 32) - 1) / size)   // 4 GB
      return bad(TPMLP_ERR_SHAPE, "heads: stride too large");
  if (v.data == nullptr && tokens > 0)
    return bad(TPMLP_ERR_ARG, "heads: null data");
  if (reinterpret_cast<uintptr_t>(v.data) % size != 0)
    return bad(TPMLP_ERR_ALIGN, "heads: data is not aligned to its element");
  return TPMLP_OK;
}

// The views of one call: per side the inputs and the output.
struct Call {
  const tp_heads* in[2][2] = {{nullptr, nullptr}, {nullptr, nullptr}};
  const tp_heads* out[2] = {nullptr, nullptr};
  int inputs = 1;
};

int check_call(const Call& c, int tokens, int d, int size) {
  for (int s = 0; s < 2; ++s) {
    const bool on = present(c.out[s]);
    for (int i = 0; i < c.inputs; ++i)
      if (present(c.in[s][i]) != on ||
          (on && c.in[s][i]->heads != c.out[s]->heads))
        return bad(TPMLP_ERR_SHAPE,
                   "heads: inputs and outputs differ in their head counts");
    if (!on) {
      if (s == 0) return bad(TPMLP_ERR_ARG, "heads: q is missing");
      continue;
    }
    for (int i = 0; i < c.inputs; ++i)
      TRY(check_view(*c.in[s][i], tokens, d, size));
    TRY(check_view(*c.out[s], tokens, d, size));
  }
  if (tokens == 0) return TPMLP_OK;
  for (int s = 0; s < 2; ++s) {
    if (!present(c.out[s])) continue;
    if (!rows_apart(*c.out[s], tokens, d))
      return bad(TPMLP_ERR_ARG, "heads: an output's rows overlap one another");
    for (int s2 = 0; s2 < 2; ++s2) {
      if (!present(c.out[s2])) continue;
      if (s2 > s && may_overlap(*c.out[s], *c.out[s2], tokens, d, size))
        return bad(TPMLP_ERR_ARG, "heads: the outputs overlap");
      for (int i = 0; i < c.inputs; ++i) {
        if (s == s2 && same_view(*c.out[s], *c.in[s2][i], tokens)) continue;
        if (may_overlap(*c.out[s], *c.in[s2][i], tokens, d, size))
          return bad(TPMLP_ERR_ARG, "heads: an output overlaps an input that "
                                    "is not the same view");
      }
    }
  }
  return TPMLP_OK;
}

// Largest power of two up to `bytes` that divides every distance of the view.
int fit_bytes(int bytes, const tp_heads& v, int tokens, int size) {
  const Steps s = steps_of(v, tokens);
  while (bytes > size) {
    bool ok = reinterpret_cast<uintptr_t>(v.data) % bytes == 0;
    for (int i = 0; i < s.n; ++i) ok = ok && s.stride[i] * size % bytes == 0;
    if (ok) break;
    bytes /= 2;
  }
  return bytes;
}

qk::View kernel_view(const tp_heads& v, int size) {
  const bool single = v.group == 1;   // heads lie group_stride apart
  qk::View k;
  k.p = static_cast<char*>(v.data);
  k.ts = v.token_stride * size;
  k.gs = static_cast<unsigned>(v.group_stride * size);
  k.hs = static_cast<unsigned>((single ? v.group_stride : v.head_stride) * size);
  k.group = static_cast<unsigned>(single ? v.heads : v.group);
  k.magic = k.group == 1 ? 0u   // a single head: group 0
                         : static_cast<unsigned>(((1ull << 32) + k.group - 1) /
                                                 k.group);
  return k;
}

// The kernel's arguments, without norm and parameter pointers.  with_rest: the
// elements past r are read and written too (else a row is its first r).  Returns
// the kernels' `bits`: rows move in 16-byte vectors where r / 2, the elements past
// r and every distance are whole ones, else in bits of as many elements as divide
// r / 2 (interleaved: r), the elements past r and a row.
int plan(const tp_rope_handle& H, const Call& c, int tokens, int size,
         int inverse, bool with_rest, const tp_positions* pos, qk::Args* a) {
  std::memset(a, 0, sizeof(*a));
  int bytes = 16;
  for (int s = 0; s < 2; ++s) {
    if (!present(c.out[s])) continue;
    for (int i = 0; i < c.inputs; ++i)
      bytes = fit_bytes(bytes, *c.in[s][i], tokens, size);
    bytes = fit_bytes(bytes, *c.out[s], tokens, size);
  }
  const int d = with_rest ? H.d : H.r;   // elements of a row that count
  const int vec = 16 / size;
  int bits = 0;
  if (bytes < 16 || H.r / 2 % vec != 0 || (d - H.r) % (2 * vec) != 0) {
    const int part = H.interleaved ? H.r : H.r / 2;
    bits = 4;
    while (bits > 1 && (part % bits != 0 || (d - H.r) % bits != 0 ||
                        d % bits != 0))
      bits /= 2;
  }
  const int per = bits ? 8 : vec;        // pairs of a unit
  a->tokens = tokens;
  a->d = d;
  a->rot = H.r;
  a->rot_units = (H.r / 2 + per - 1) / per;
  a->units = a->rot_units + (d - H.r + 2 * per - 1) / (2 * per);
  a->rows = 32 / a->units;
  while (d * size % bytes != 0) bytes /= 2;   // whole pieces in a row
  a->piece = bytes;
  a->row_pieces = d * size / bytes;
  a->row_pieces_magic =
      a->row_pieces == 1 ? 0u
                         : static_cast<unsigned>(
                               ((1ull << 32) + a->row_pieces - 1) / a->row_pieces);
  for (int s = 0; s < 2; ++s) {
    qk::Side& sd = a->side[s];
    if (!present(c.out[s])) continue;
    sd.in = kernel_view(*c.in[s][0], size);
    if (c.inputs > 1) sd.x = kernel_view(*c.in[s][1], size);
    sd.out = kernel_view(*c.out[s], size);
    sd.heads = c.out[s]->heads;
    sd.steps = (sd.heads + a->rows - 1) / a->rows;
  }
  if (pos != nullptr) {
    a->pos = pos->data;
    a->pos64 = pos->is_int64;
    a->offset = pos->offset;
    a->seq_len = pos->seq_len > 0x7fffffffLL
                     ? 0u : static_cast<unsigned>(pos->seq_len);
  }
  a->amp = static_cast<float>(H.amplitude);
  a->sign = inverse ? -1.f : 1.f;
  a->inv_d = 1.0f / static_cast<float>(H.d);
  for (int i = 0; i < H.r / 2; ++i) a->freq[i] = H.turns[i];
  return bits;
}

int check_common(const tp_rope_handle* H, int tokens, int dtype,
                 const tp_positions* pos) {
  if (H == nullptr) return bad(TPMLP_ERR_ARG, "null handle");
  if (dtype != TPMLP_BF16 && dtype != TPMLP_FP32)
    return bad(TPMLP_ERR_ARG, "dtype must be TPMLP_BF16 or TPMLP_FP32");
  if (tokens < 0 || tokens > MAX_TOKENS)
    return bad(TPMLP_ERR_SHAPE, "tokens must be 0 .. 2^28");
  if (pos != nullptr) {
    if (pos->is_int64 != 0 && pos->is_int64 != 1)
      return bad(TPMLP_ERR_ARG, "positions: is_int64 must be 0 or 1");
    if (pos->seq_len < 0)
      return bad(TPMLP_ERR_SHAPE, "positions: seq_len must be >= 0");
    if (reinterpret_cast<uintptr_t>(pos->data) % (pos->is_int64 ? 8 : 4) != 0)
      return bad(TPMLP_ERR_ALIGN, "positions: data is not aligned");
  }
  return TPMLP_OK;
}

int check_norm(const tp_qk_norm* n) {
  if (n == nullptr) return bad(TPMLP_ERR_ARG, "norm: null");
  if (n->norm != TPQK_RMSNORM && n->norm != TPQK_LAYERNORM)
    return bad(TPMLP_ERR_ARG, "norm must be TPQK_RMSNORM or TPQK_LAYERNORM");
  if (!(n->eps >= 0.f) || !std::isfinite(n->eps))
    return bad(TPMLP_ERR_ARG, "norm: eps must be finite and >= 0");
  if (n->norm == TPQK_RMSNORM && (n->q_beta || n->k_beta))
    return bad(TPMLP_ERR_ARG, "norm: the RMS norm has no beta");
  for (const float* p : {n->q_gamma, n->q_beta, n->k_gamma, n->k_beta})
    if (reinterpret_cast<uintptr_t>(p) % 4 != 0)
      return bad(TPMLP_ERR_ALIGN, "norm: a parameter is not aligned");
  return TPMLP_OK;
}

int params_aligned(const tp_qk_norm& n) {
  return aligned16(n.q_gamma) && aligned16(n.q_beta) && aligned16(n.k_gamma) &&
         aligned16(n.k_beta);
}

int cuda_rc(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return TPMLP_OK;
  set_detail(what, e);
  return TPMLP_ERR_CUDA;
}

// Steps of a task when a token's `steps` are split so that there are at least
// `want` tasks, as far as there are steps, and at most `most` steps in each.
int steps_per_task(int steps, int tokens, long long want, int most) {
  const long long segs = std::min<long long>(
      steps, std::max<long long>((steps + most - 1) / most,
                                 (want + tokens - 1) / tokens));
  return static_cast<int>((steps + segs - 1) / segs);
}

// A task's start (angles, coefficients, first loads) costs about as much as two
// steps.  Forward: tokens are split until 12 warps a SM (of a GB300's 152) have
// work (2047 tokens of 14 steps: 16.6 us whole, 17.5 in halves, 20.2 in fifths),
// and into tasks of at most 16 steps (4096 tokens of 56 steps: 82.6 us whole, 73.2
// in halves, 71.9 in thirds; 8192 of 20: 54.8 whole, 52.2 in halves).
constexpr long long FORWARD_TASKS = 152 * 12;
constexpr int FORWARD_STEPS = 16;
// Backward: until the resident blocks have a task for every warp, and into tasks
// of at most 8 steps (8192 tokens of 10 steps: 82.8 us whole, 79.5 in halves, 81.2
// in quarters).
constexpr long long BACKWARD_TASKS = 1LL * qk::BWD_BLOCKS * qk::WARPS;
constexpr int BACKWARD_STEPS = 8;

int run_forward(tp_rope_handle* H, int tokens, int dtype, int inverse,
                const tp_qk_norm* norm, const tp_heads* q_in,
                const tp_heads* q_out, const tp_heads* k_in,
                const tp_heads* k_out, const tp_positions* pos, void* stream) {
  TRY(check_common(H, tokens, dtype, pos));
  if (norm != nullptr) TRY(check_norm(norm));
  const int size = dtype == TPMLP_BF16 ? 2 : 4;
  Call c;
  c.in[0][0] = q_in;
  c.out[0] = q_out;
  c.in[1][0] = k_in;
  c.out[1] = k_out;
  TRY(check_call(c, tokens, H->d, size));
  int sms = 0;
  TRY(check_device(&sms));
  if (tokens == 0) return TPMLP_OK;
  bool tail = true;
  if (norm == nullptr) {
    // in place, the elements past r stay as they are
    tail = !same_view(*q_in, *q_out, tokens) ||
           (present(k_out) && !same_view(*k_in, *k_out, tokens));
    if (!tail && H->r == 0) return TPMLP_OK;
  }
  qk::Args a;
  const int bits = plan(*H, c, tokens, size, inverse, tail, pos, &a);
  const int steps = a.side[0].steps + a.side[1].steps;
  a.per = steps_per_task(steps, tokens, FORWARD_TASKS, FORWARD_STEPS);
  a.segs = (steps + a.per - 1) / a.per;
  if (norm != nullptr) {
    a.eps = norm->eps;
    a.side[0].gamma = norm->q_gamma;
    a.side[0].beta = norm->q_beta;
    a.side[1].gamma = norm->k_gamma;
    a.side[1].beta = norm->k_beta;
    a.param16 = params_aligned(*norm);
  }
  return cuda_rc(qk::launch_forward(a, dtype == TPMLP_BF16, bits,
                                    norm ? norm->norm : 0, H->interleaved != 0,
                                    static_cast<cudaStream_t>(stream)),
                 norm ? "qk_norm_forward" : "rope_apply");
}

}  // namespace

extern "C" {

int tp_rope_create(const tp_rope_config* cfg, tp_rope_handle** out) {
  if (cfg == nullptr || out == nullptr)
    return bad(TPMLP_ERR_ARG, "rope: null argument");
  const int d = cfg->head_dim, r = cfg->rot_dim;
  if (d < 1 || d > TPROPE_MAX_HEAD_DIM)
    return bad(TPMLP_ERR_SHAPE, "rope: head_dim must be 1 .. 256");
  if (r < 0 || r > d || r % 2 != 0)
    return bad(TPMLP_ERR_SHAPE, "rope: rot_dim must be even, 0 .. head_dim");
  if (cfg->interleaved != 0 && cfg->interleaved != 1)
    return bad(TPMLP_ERR_ARG, "rope: interleaved must be 0 or 1");
  const int sc = cfg->scaling;
  if (sc < TPROPE_SCALE_NONE || sc > TPROPE_SCALE_CUSTOM)
    return bad(TPMLP_ERR_ARG, "rope: unknown scaling");
  if (sc != TPROPE_SCALE_CUSTOM && !positive(cfg->base))
    return bad(TPMLP_ERR_ARG, "rope: base must be positive and finite");
  if ((sc == TPROPE_SCALE_LINEAR || sc == TPROPE_SCALE_NTK ||
       sc == TPROPE_SCALE_YARN) && !positive(cfg->factor))
    return bad(TPMLP_ERR_ARG, "rope: factor must be positive and finite");
  if (sc == TPROPE_SCALE_YARN &&
      (!positive(cfg->original_length) || !std::isfinite(cfg->slow_turns) ||
       !std::isfinite(cfg->fast_turns) || cfg->fast_turns <= cfg->slow_turns))
    return bad(TPMLP_ERR_ARG, "rope: YARN needs original_length > 0 and "
                              "fast_turns > slow_turns");
  if (!(std::fabs(cfg->amplitude) <= 3.4e38))   // (the kernels' is an fp32)
    return bad(TPMLP_ERR_ARG, "rope: amplitude must be at most 3.4e38");
  if (sc == TPROPE_SCALE_CUSTOM && r > 0 && cfg->inv_freq == nullptr)
    return bad(TPMLP_ERR_ARG, "rope: CUSTOM needs inv_freq");
  tp_rope_handle h;
  h.d = d;
  h.r = r;
  h.interleaved = cfg->interleaved;
  h.amplitude = cfg->amplitude != 0.0 ? cfg->amplitude
                : sc == TPROPE_SCALE_YARN ? 0.1 * std::log(cfg->factor) + 1.0
                                          : 1.0;
  double base = cfg->base;
  if (sc == TPROPE_SCALE_NTK && r > 2)
    base *= std::pow(cfg->factor, static_cast<double>(r) / (r - 2));
  for (int i = 0; i < r / 2; ++i) {
    double f = sc == TPROPE_SCALE_CUSTOM ? cfg->inv_freq[i]
                                         : std::pow(base, -2.0 * i / r);
    if (sc == TPROPE_SCALE_LINEAR) f /= cfg->factor;
    if (sc == TPROPE_SCALE_YARN) {
      const double n =
          cfg->original_length * f / 6.283185307179586476925286766559;
      const double k = std::min(1.0, std::max(0.0, (n - cfg->slow_turns) /
                                   (cfg->fast_turns - cfg->slow_turns)));
      f = k * f + (1.0 - k) * f / cfg->factor;
    }
    if (!std::isfinite(f))
      return bad(TPMLP_ERR_ARG, "rope: a frequency is not finite");
    h.inv_freq[i] = f;
    h.turns[i] = fixed_turns(f);
  }
  tp_rope_handle* p = new (std::nothrow) tp_rope_handle(h);
  if (p == nullptr) return bad(TPMLP_ERR_ARG, "rope: out of host memory");
  *out = p;
  return TPMLP_OK;
}

int tp_rope_destroy(tp_rope_handle* handle) {
  delete handle;
  return TPMLP_OK;
}

int tp_rope_frequencies(const tp_rope_handle* H, double* inv_freq,
                        double* amplitude) {
  if (H == nullptr) return bad(TPMLP_ERR_ARG, "null handle");
  if (inv_freq != nullptr)
    std::memcpy(inv_freq, H->inv_freq, sizeof(double) * (H->r / 2));
  if (amplitude != nullptr) *amplitude = H->amplitude;
  return TPMLP_OK;
}

int tp_rope_apply(tp_rope_handle* H, int tokens, int dtype, int inverse,
                  const tp_heads* q_in, const tp_heads* q_out,
                  const tp_heads* k_in, const tp_heads* k_out,
                  const tp_positions* positions, void* stream) {
  if (inverse != 0 && inverse != 1)
    return bad(TPMLP_ERR_ARG, "inverse must be 0 or 1");
  return run_forward(H, tokens, dtype, inverse, nullptr, q_in, q_out, k_in,
                     k_out, positions, stream);
}

int tp_qk_norm_forward(tp_rope_handle* H, int tokens, int dtype,
                       const tp_qk_norm* norm, const tp_heads* q_in,
                       const tp_heads* q_out, const tp_heads* k_in,
                       const tp_heads* k_out, const tp_positions* positions,
                       void* stream) {
  if (norm == nullptr) return bad(TPMLP_ERR_ARG, "norm: null");
  return run_forward(H, tokens, dtype, 0, norm, q_in, q_out, k_in, k_out,
                     positions, stream);
}

size_t tp_qk_norm_workspace_bytes(const tp_rope_handle* H) {
  if (H == nullptr) return 0;
  return sizeof(float) * 2 * qk::BWD_BLOCKS * static_cast<size_t>(H->d);
}

int tp_qk_norm_backward(tp_rope_handle* H, int tokens, int dtype,
                        const tp_qk_norm* norm, const tp_heads* dq,
                        const tp_heads* q_in, const tp_heads* dq_out,
                        const tp_heads* dk, const tp_heads* k_in,
                        const tp_heads* dk_out, const tp_positions* positions,
                        const tp_qk_norm_grads* grads, void* workspace,
                        size_t workspace_bytes, void* stream) {
  TRY(check_common(H, tokens, dtype, positions));
  TRY(check_norm(norm));
  const int size = dtype == TPMLP_BF16 ? 2 : 4;
  Call c;
  c.inputs = 2;
  c.in[0][0] = dq;
  c.in[0][1] = q_in;
  c.out[0] = dq_out;
  c.in[1][0] = dk;
  c.in[1][1] = k_in;
  c.out[1] = dk_out;
  TRY(check_call(c, tokens, H->d, size));
  float* out[4] = {nullptr, nullptr, nullptr, nullptr};
  if (grads != nullptr) {
    out[0] = grads->q_gamma;
    out[1] = grads->q_beta;
    out[2] = grads->k_gamma;
    out[3] = grads->k_beta;
  }
  const bool has_k = present(dk_out);
  if (norm->norm == TPQK_RMSNORM && (out[1] || out[3]))
    return bad(TPMLP_ERR_ARG, "norm: the RMS norm has no beta");
  if (!has_k && (out[2] || out[3]))
    return bad(TPMLP_ERR_ARG, "norm: gradients of k without k");
  bool params = false;
  for (int i = 0; i < 4; ++i) {
    if (reinterpret_cast<uintptr_t>(out[i]) % 4 != 0)
      return bad(TPMLP_ERR_ALIGN, "norm: a gradient is not aligned");
    params = params || out[i] != nullptr;
    for (int j = 0; j < i; ++j)
      if (out[i] != nullptr && out[j] != nullptr &&
          std::llabs(out[i] - out[j]) < H->d)
        return bad(TPMLP_ERR_ARG, "norm: two gradients share memory");
  }
  if (params && tokens > 0) {
    if (workspace == nullptr) return bad(TPMLP_ERR_ARG, "null workspace");
    if (!aligned16(workspace))
      return bad(TPMLP_ERR_ALIGN, "workspace is not 16-byte aligned");
    if (workspace_bytes < tp_qk_norm_workspace_bytes(H))
      return bad(TPMLP_ERR_WORKSPACE, "workspace too small");
  }
  int sms = 0;
  TRY(check_device(&sms));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (tokens == 0) {
    for (float* p : out)
      if (p != nullptr)
        TRY(cuda_rc(cudaMemsetAsync(p, 0, sizeof(float) * H->d, s),
                    "cudaMemsetAsync(zero gradients)"));
    return TPMLP_OK;
  }
  qk::Args a;
  const int bits = plan(*H, c, tokens, size, 1, true, positions, &a);
  a.eps = norm->eps;
  a.side[0].gamma = norm->q_gamma;
  a.side[1].gamma = norm->k_gamma;
  a.param16 = params_aligned(*norm);
  a.part = params ? static_cast<float*>(workspace) : nullptr;
  // blocks in proportion to the steps, no more than there are tasks
  const long long all = a.side[0].steps + a.side[1].steps;
  long long bq = has_k ? std::min<long long>(
                             qk::BWD_BLOCKS - 1,
                             std::max(1LL, qk::BWD_BLOCKS * a.side[0].steps / all))
                       : qk::BWD_BLOCKS;
  long long side_blocks[2] = {bq, qk::BWD_BLOCKS - bq};
  for (int i = 0; i < (has_k ? 2 : 1); ++i) {
    const int steps = a.side[i].steps;
    a.per_side[i] =
        steps_per_task(steps, tokens, BACKWARD_TASKS * steps / all,
                       BACKWARD_STEPS);
    a.segs_side[i] = (steps + a.per_side[i] - 1) / a.per_side[i];
    const long long tasks = static_cast<long long>(tokens) * a.segs_side[i];
    side_blocks[i] = std::min(side_blocks[i], (tasks + qk::WARPS - 1) / qk::WARPS);
  }
  bq = side_blocks[0];
  const long long bk = side_blocks[1];
  a.q_blocks = static_cast<int>(bq);
  const int blocks = static_cast<int>(bq + bk);
  TRY(cuda_rc(qk::launch_backward(a, dtype == TPMLP_BF16, bits, norm->norm,
                                  H->interleaved != 0, blocks, s),
              "qk_norm_backward"));
  if (!params) return TPMLP_OK;
  return cuda_rc(qk::launch_param_sums(a.part, H->d, a.q_blocks, blocks, out, s),
                 "qk_param_sums");
}

}  // extern "C"
