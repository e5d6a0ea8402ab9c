// Host side of the head-parallel self-attention block: validation,
// workspace layout, tensor maps and launch sequencing.
//
// Forward (Megatron-LM explainer, "Attention: a design that parallelises
// naturally"; Megatron-LM notes, "Self-attention block split"):
//   [LayerNorm] -> QKV = Xn W_qkv + b_qkv (pair GEMM, one column group per
//   shard) -> [norm and rotation of Q's and K's heads, tp_rope.h] ->
//   attention core per (sequence, head, query block) -> Z =
//   sum_i Ctx_i W_o,i + b_o (pair GEMM, fixed-order shard sum = g) [+ X].
// Backward: db_o, dW_o = Ctx^T dZ, dCtx = dZ W_o^T -> dQ and delta =
//   rowsum(dCtx * Ctx) per head (one CTA per query block) -> dK, dV (one CTA
//   per key block) -> db_qkv, dW_qkv = Xn^T dQKV, dXn = sum_i dQKV_i W_qkv,i^T
//   (fixed-order shard sum = f's backward) -> [LayerNorm backward] [+ dZ].
#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>

#include "host_common.cuh"
#include "tp_attn.h"

using namespace tpmlp;
using namespace tpmlp::host;

namespace {

struct AttnLayout {
  size_t status = 0, xn = 0, mean = 0, rstd = 0, qkv = 0, ctx = 0, lse = 0,
         dctx = 0, delta = 0, dqkv = 0, dxn = 0, part = 0, tailp = 0,
         total = 0, lnp = 0, qkr = 0, qkpart = 0;
  size_t lnsync_words = 0;   // the LayerNorm prologue's counters
  int chunks = 0;   // 256-row column-sum chunks
  int groups = 0;   // 32-row groups of the core kernels' fused db_qkv partials
};

size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

}  // namespace

struct tp_attn_handle {
  HandleCore core;
  tp_attn_config cfg;
  bool ln_prologue = true;   // tp_attn_set_ln_prologue
  tp_rope_handle* rope = nullptr;   // tp_attn_set_rope
  tp_rope_handle* plain = nullptr;  // no rotation: the norm alone
  int qk_norm = 0;                  // tp_attn_set_qk_norm
  float qk_eps = 0.f;

  ~tp_attn_handle() {
    tp_rope_destroy(rope);
    tp_rope_destroy(plain);
  }
  // The handle the norm and the rotation run with (null: neither is set).
  tp_rope_handle* qk() const {
    return rope != nullptr ? rope : qk_norm != 0 ? plain : nullptr;
  }
};

namespace {

AttnLayout attn_layout(const tp_attn_handle* handle, int tokens,
                       int training) {
  const tp_attn_config& c = handle->cfg;
  AttnLayout L;
  const size_t T = static_cast<size_t>(tokens);
  const size_t h = static_cast<size_t>(c.hidden);
  const size_t H = static_cast<size_t>(c.heads);
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = align_up(off + bytes, 256);
    return o;
  };
  if (c.use_layernorm) {
    // the status word, then the LayerNorm prologue's row counters
    // (GemmArgs::ln_sync: 1 + ceil(T / 128) words)
    L.lnsync_words = 1 + (T + 127) / 128;
    L.status = take(16 + 4 * L.lnsync_words);
  } else {
    L.status = take(256);
  }
  if (c.use_layernorm) {
    L.xn = take(T * h * 2);
    L.mean = take(T * 4);
    L.rstd = take(T * 4);
  }
  L.qkv = take(T * 3 * h * 2);
  L.ctx = take(T * h * 2);
  L.lse = take(H * T * 4);
  L.tailp = take(static_cast<size_t>(TAIL_PART_BYTES));  // GEMM tail split
  if (training) {
    L.dctx = take(T * h * 2);
    L.delta = take(2 * H * T * 4);   // -lse2 and -delta' (AttnArgs::delta)
    L.dqkv = take(T * 3 * h * 2);
    if (c.use_layernorm) L.dxn = take(T * h * 4);
    L.chunks = colsum_chunks(tokens);
    L.groups = (tokens + 31) / 32;
    // db_o (chunks x h), db_qkv (max(groups, chunks) x 3h), dgamma and
    // dbeta (lnp x h each)
    const size_t rows3 = static_cast<size_t>(L.groups > L.chunks ? L.groups : L.chunks);
    L.lnp = static_cast<size_t>(L.chunks);
    L.part = take((static_cast<size_t>(L.chunks) * h + rows3 * 3 * h +
                   2 * L.lnp * h) * 4);
  }
  // Q and K as the core reads them: in place, but for a training forward with
  // the norm, whose gradient needs them as projected too
  L.qkr = L.qkv;
  if (training && handle->qk_norm != 0) {
    L.qkr = take(T * 3 * h * 2);
    L.qkpart = take(tp_qk_norm_workspace_bytes(handle->qk()));
  }
  L.total = off;
  return L;
}

GemmArgs gemm_args(const tp_attn_handle* H, char* ws, const AttnLayout& L) {
  GemmArgs a;
  std::memset(&a, 0, sizeof(a));
  a.group_m = 16;
  a.status = reinterpret_cast<int*>(ws + L.status);
  a.budget_ns = H->core.budget_ns;
  a.num_seg = 1;
  a.part = reinterpret_cast<float*>(ws + L.tailp);
  a.part_bytes = TAIL_PART_BYTES;
  return a;
}

AttnArgs core_args(const tp_attn_handle* H, char* ws, const AttnLayout& L,
                   int tokens) {
  const tp_attn_config& c = H->cfg;
  AttnArgs a;
  std::memset(&a, 0, sizeof(a));
  a.heads = c.heads;
  a.heads_per_shard = c.heads / c.shards;
  a.head_dim = c.hidden / c.heads;
  a.shard_width = c.hidden / c.shards;
  a.seq_len = c.seq_len;
  a.nq = c.seq_len / 128;
  a.causal = c.causal;
  a.scale_log2 = static_cast<float>(1.4426950408889634 /
                                    std::sqrt(static_cast<double>(a.head_dim)));
  a.ctx = reinterpret_cast<__nv_bfloat16*>(ws + L.ctx);
  a.ld_ctx = c.hidden;
  a.lse = reinterpret_cast<float*>(ws + L.lse);
  a.ld_stat = tokens;
  a.ld_qkv = 3LL * c.hidden;
  a.status = reinterpret_cast<int*>(ws + L.status);
  a.budget_ns = H->core.budget_ns;
  return a;
}

// The heads of Q (which = 0) or K (1) in a buffer laid out as QKV.
tp_heads qk_heads(const tp_attn_handle* H, void* qkv, int which) {
  const tp_attn_config& c = H->cfg;
  const int ht = c.hidden / c.shards;
  tp_heads v;
  v.data = static_cast<char*>(qkv) + 2LL * which * ht;
  v.token_stride = 3LL * c.hidden;
  v.group_stride = 3LL * ht;
  v.head_stride = c.hidden / c.heads;
  v.heads = c.heads;
  v.group = c.heads / c.shards;
  return v;
}

// Everything about qk and qk_grads that can be refused, before any launch.
int check_qk(const tp_attn_handle* H, const tp_attn_qk* qk,
             const tp_qk_norm_grads* g) {
  const void* params[4] = {nullptr, nullptr, nullptr, nullptr};
  const void* grads[4] = {nullptr, nullptr, nullptr, nullptr};
  if (qk != nullptr) {
    if (qk->positions_int64 != 0 && qk->positions_int64 != 1) return TPMLP_ERR_ARG;
    if (qk->positions != nullptr && H->rope == nullptr) {
      set_detail_msg("positions without tp_attn_set_rope");
      return TPMLP_ERR_ARG;
    }
    if (reinterpret_cast<uintptr_t>(qk->positions) %
            (qk->positions_int64 ? 8 : 4) != 0)
      return TPMLP_ERR_ALIGN;
    params[0] = qk->q_gamma;
    params[1] = qk->q_beta;
    params[2] = qk->k_gamma;
    params[3] = qk->k_beta;
  }
  if (g != nullptr) {
    grads[0] = g->q_gamma;
    grads[1] = g->q_beta;
    grads[2] = g->k_gamma;
    grads[3] = g->k_beta;
  }
  for (int i = 0; i < 4; ++i) {
    if (params[i] == nullptr && grads[i] == nullptr) continue;
    if (H->qk_norm == 0) {
      set_detail_msg("norm parameters without tp_attn_set_qk_norm");
      return TPMLP_ERR_ARG;
    }
    if (H->qk_norm == TPQK_RMSNORM && i % 2 == 1) {
      set_detail_msg("the RMS norm has no beta");
      return TPMLP_ERR_ARG;
    }
    if (reinterpret_cast<uintptr_t>(params[i]) % 4 != 0 ||
        reinterpret_cast<uintptr_t>(grads[i]) % 4 != 0)
      return TPMLP_ERR_ALIGN;
    for (int j = 0; j < i; ++j)
      if (grads[i] != nullptr && grads[j] != nullptr &&
          std::abs(static_cast<const float*>(grads[i]) -
                   static_cast<const float*>(grads[j])) <
              H->cfg.hidden / H->cfg.heads) {
        set_detail_msg("two gradients of the norm share memory");
        return TPMLP_ERR_ARG;
      }
  }
  return TPMLP_OK;
}

tp_positions qk_positions(const tp_attn_handle* H, const tp_attn_qk* qk) {
  tp_positions p;
  p.data = qk != nullptr ? qk->positions : nullptr;
  p.is_int64 = qk != nullptr ? qk->positions_int64 : 0;
  p.offset = 0;
  p.seq_len = H->cfg.seq_len;
  return p;
}

tp_qk_norm qk_norm_args(const tp_attn_handle* H, const tp_attn_qk* qk,
                        bool beta) {
  tp_qk_norm n;
  std::memset(&n, 0, sizeof(n));
  n.norm = H->qk_norm;
  n.eps = H->qk_eps;
  if (qk != nullptr) {
    n.q_gamma = qk->q_gamma;
    n.k_gamma = qk->k_gamma;
    n.q_beta = beta ? qk->q_beta : nullptr;
    n.k_beta = beta ? qk->k_beta : nullptr;
  }
  return n;
}

// A call of tp_rope.h as one of the handle's launches.
template <class F>
int run_qk(HandleCore* core, const char* name, cudaStream_t s, F&& call) {
  int rc = TPMLP_OK;
  TRY(run(core, name, s, [&] {
    rc = call();
    return cudaSuccess;
  }));
  return rc;
}

// Norm and rotation of Q and K, from `from` to `to` (both laid out as QKV).
int qk_forward(tp_attn_handle* H, int tokens, void* from, void* to,
               const tp_attn_qk* qk, cudaStream_t s) {
  const tp_heads q = qk_heads(H, from, 0), k = qk_heads(H, from, 1);
  const tp_heads q2 = qk_heads(H, to, 0), k2 = qk_heads(H, to, 1);
  const tp_positions pos = qk_positions(H, qk);
  if (H->qk_norm == 0)
    return run_qk(&H->core, "rope", s, [&] {
      return tp_rope_apply(H->rope, tokens, TPMLP_BF16, 0, &q, &q2, &k, &k2,
                           &pos, s);
    });
  const tp_qk_norm n = qk_norm_args(H, qk, true);
  return run_qk(&H->core, "qk_norm_rope", s, [&] {
    return tp_qk_norm_forward(H->qk(), tokens, TPMLP_BF16, &n, &q, &q2, &k, &k2,
                              &pos, s);
  });
}

// Their gradient, in place in dqkv.
int qk_backward(tp_attn_handle* H, int tokens, void* dqkv, void* qkv,
                const tp_attn_qk* qk, const tp_qk_norm_grads* grads,
                void* part, cudaStream_t s) {
  const tp_heads dq = qk_heads(H, dqkv, 0), dk = qk_heads(H, dqkv, 1);
  const tp_positions pos = qk_positions(H, qk);
  if (H->qk_norm == 0)
    return run_qk(&H->core, "rope_bwd", s, [&] {
      return tp_rope_apply(H->rope, tokens, TPMLP_BF16, 1, &dq, &dq, &dk, &dk,
                           &pos, s);
    });
  const tp_heads q = qk_heads(H, qkv, 0), k = qk_heads(H, qkv, 1);
  const tp_qk_norm n = qk_norm_args(H, qk, false);
  if (grads != nullptr && (grads->q_gamma || grads->q_beta || grads->k_gamma ||
                           grads->k_beta))
    H->core.launches++;   // the parameter gradients' sums
  return run_qk(&H->core, "qk_norm_rope_bwd", s, [&] {
    return tp_qk_norm_backward(H->qk(), tokens, TPMLP_BF16, &n, &dq, &q, &dq,
                               &dk, &k, &dk, &pos, grads, part,
                               tp_qk_norm_workspace_bytes(H->qk()), s);
  });
}

int check_ptrs(std::initializer_list<const void*> ptrs) {
  for (const void* p : ptrs)
    if (p && !aligned16(p)) return TPMLP_ERR_ALIGN;
  return TPMLP_OK;
}

}  // namespace

extern "C" {

int tp_attn_create(const tp_attn_config* cfg, tp_attn_handle** out) {
  if (cfg == nullptr || out == nullptr) return TPMLP_ERR_ARG;
  if ((cfg->causal != 0 && cfg->causal != 1) ||
      (cfg->use_layernorm != 0 && cfg->use_layernorm != 1) ||
      (cfg->use_residual != 0 && cfg->use_residual != 1))
    return TPMLP_ERR_ARG;
  if (cfg->use_layernorm && !(cfg->ln_eps >= 0.f && std::isfinite(cfg->ln_eps)))
    return TPMLP_ERR_ARG;
  if (cfg->hidden <= 0 || cfg->heads <= 0 || cfg->shards <= 0 ||
      cfg->seq_len <= 0 || cfg->max_tokens < 0)
    return TPMLP_ERR_SHAPE;
  if (cfg->hidden % cfg->heads != 0 || cfg->heads % cfg->shards != 0)
    return TPMLP_ERR_SHAPE;
  const int d = cfg->hidden / cfg->heads;
  if (d != 64 && d != 96 && d != 128) return TPMLP_ERR_SHAPE;
  if ((cfg->hidden / cfg->shards) % 64 != 0) return TPMLP_ERR_SHAPE;
  if (cfg->seq_len % 128 != 0) return TPMLP_ERR_SHAPE;
  if (static_cast<long long>(cfg->max_tokens) > (1LL << 28) ||
      cfg->hidden > (1 << 20))
    return TPMLP_ERR_SHAPE;
  tp_attn_handle* h = new (std::nothrow) tp_attn_handle();
  if (h == nullptr) return TPMLP_ERR_ARG;
  h->cfg = *cfg;
  *out = h;
  return TPMLP_OK;
}

int tp_attn_destroy(tp_attn_handle* handle) {
  delete handle;
  return TPMLP_OK;
}

size_t tp_attn_workspace_bytes(const tp_attn_handle* handle, int tokens,
                               int training) {
  if (handle == nullptr || tokens < 0) return 0;
  return attn_layout(handle, tokens, training ? 1 : 0).total;
}

long long tp_attn_workspace_offset(const tp_attn_handle* handle, int tokens,
                                   int training, int which) {
  if (handle == nullptr || tokens < 0) return -1;
  const AttnLayout L = attn_layout(handle, tokens, training ? 1 : 0);
  switch (which) {
    case TPATTN_WS_QKV: return static_cast<long long>(L.qkv);
    case TPATTN_WS_CTX: return static_cast<long long>(L.ctx);
    case TPATTN_WS_LSE: return static_cast<long long>(L.lse);
    case TPATTN_WS_DQKV:
      return training ? static_cast<long long>(L.dqkv) : -1;
    case TPATTN_WS_QKR: return static_cast<long long>(L.qkr);
    default: return -1;
  }
}

int tp_attn_forward(tp_attn_handle* H, int tokens, const void* X,
                    const void* Wqkv, const void* Wo, const float* bqkv,
                    const float* bo, const float* ln_gamma,
                    const float* ln_beta, void* Z, void* workspace,
                    size_t workspace_bytes, int training, void* stream) {
  return tp_attn_forward_qk(H, tokens, X, Wqkv, Wo, bqkv, bo, ln_gamma, ln_beta,
                            Z, workspace, workspace_bytes, training, nullptr,
                            stream);
}

int tp_attn_forward_qk(tp_attn_handle* H, int tokens, const void* X,
                       const void* Wqkv, const void* Wo, const float* bqkv,
                       const float* bo, const float* ln_gamma,
                       const float* ln_beta, void* Z, void* workspace,
                       size_t workspace_bytes, int training,
                       const tp_attn_qk* qk, void* stream) {
  if (H == nullptr) return TPMLP_ERR_ARG;
  const tp_attn_config& c = H->cfg;
  if (tokens < 0 || tokens > c.max_tokens || tokens % c.seq_len != 0)
    return TPMLP_ERR_SHAPE;
  if (!Wqkv || !Wo || !workspace || (tokens > 0 && (!X || !Z)))
    return TPMLP_ERR_ARG;
  if (c.use_layernorm && (!ln_gamma || !ln_beta)) return TPMLP_ERR_ARG;
  TRY(check_ptrs({X, Wqkv, Wo, bqkv, bo, ln_gamma, ln_beta, Z, workspace}));
  TRY(check_qk(H, qk, nullptr));
  const AttnLayout L = attn_layout(H, tokens, training ? 1 : 0);
  if (workspace_bytes < L.total) return TPMLP_ERR_WORKSPACE;
  int sms = 0;
  TRY(check_device(&sms));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  // LayerNorm inside the QKV projection's launch (GemmArgs::ln_x)
  const bool ln_fused = c.use_layernorm && H->ln_prologue &&
                        c.hidden % 256 == 0 && c.hidden / 256 <= LN_VMAX;
  // the status word, and with the fused LayerNorm its counters, cleared
  const size_t clear = ln_fused ? 16 + 4 * L.lnsync_words : 16;
  cudaError_t e = cudaMemsetAsync(ws + L.status, 0, clear, s);
  if (e != cudaSuccess) {
    set_detail("cudaMemsetAsync(status)", e);
    return TPMLP_ERR_CUDA;
  }
  if (tokens == 0) return TPMLP_OK;

  const int T = tokens, h = c.hidden, ht = h / c.shards;
  const void* Xop = X;
  if (ln_fused) {
    Xop = ws + L.xn;
  } else if (c.use_layernorm) {
    void* Xn = ws + L.xn;
    TRY(run(&H->core, "layernorm_fwd", s, [&] {
      return launch_ln_fwd(true, X, ln_gamma, ln_beta, Xn,
                           reinterpret_cast<float*>(ws + L.mean),
                           reinterpret_cast<float*>(ws + L.rstd), T, h,
                           c.ln_eps, s);
    }));
    Xop = Xn;
  }
  CUtensorMap ta, tb;
  // QKV = Xn W_qkv + b_qkv
  GemmArgs gq = gemm_args(H, ws, L);
  gq.M = T; gq.N = 3 * h; gq.K = h; gq.kb_per_seg = h / TC_BK;
  gq.out = ws + L.qkv; gq.ldo = 3LL * h; gq.bias = bqkv;
  if (ln_fused) {
    gq.ln_x = static_cast<const __nv_bfloat16*>(X);
    gq.ln_gamma = ln_gamma;
    gq.ln_beta = ln_beta;
    gq.ln_xn = reinterpret_cast<__nv_bfloat16*>(ws + L.xn);
    gq.ln_mean = reinterpret_cast<float*>(ws + L.mean);
    gq.ln_rstd = reinterpret_cast<float*>(ws + L.rstd);
    gq.ln_eps = c.ln_eps;
    gq.ln_sync = reinterpret_cast<unsigned int*>(ws + L.status + 16);
  }
  TRY(kmajor_map(&ta, Xop, T, h, TC_BM));
  TRY(mnmajor_map(&tb, Wqkv, h, 3 * h));
  TRY(tc_gemm(&H->core, ln_fused ? "gemm_ln_qkv" : "gemm_qkv", s, sms,
              EPI_BIAS_BF16, false, true, ta, tb, gq));
  if (H->qk() != nullptr)
    TRY(qk_forward(H, T, ws + L.qkv, ws + L.qkr, qk, s));
  // attention core
  AttnArgs aa = core_args(H, ws, L, T);
  CUtensorMap tqk, tv;
  TRY(encode_map(&tqk, ws + L.qkr, 3ULL * h, T, 3ULL * h, 128));
  TRY(encode_map(&tv, ws + L.qkv, 3ULL * h, T, 3ULL * h, 64));
  // persistent forward: two CTAs per SM walk the items, one group of
  // (sequence, head) pairs per round
  const int items = (T / c.seq_len) * c.heads * aa.nq;
  const int grid = std::min(items, 2 * sms);
  aa.hs_group = std::max(1, grid / aa.nq);
  TRY(run(&H->core, "attn_fwd", s,
          [&] { return launch_attn_fwd(tqk, tv, aa, grid, s); }));
  // Z = sum_i Ctx_i W_o,i + b_o [+ X]
  GemmArgs go = gemm_args(H, ws, L);
  go.M = T; go.N = h; go.K = h; go.num_seg = c.shards;
  go.kb_per_seg = ht / TC_BK;
  go.out = Z; go.ldo = h; go.bias = bo;
  if (c.use_residual) {
    go.aux = X;
    go.ldaux = h;
  }
  TRY(kmajor_map(&ta, ws + L.ctx, T, h, TC_BM));
  TRY(mnmajor_map(&tb, Wo, h, h));
  return tc_gemm(&H->core, "gemm_out_shardsum", s, sms, EPI_SHARDSUM, false,
                 true, ta, tb, go);
}

int tp_attn_backward(tp_attn_handle* H, int tokens, const void* dZ,
                     const void* X, const void* Wqkv, const void* Wo,
                     const float* ln_gamma, void* workspace,
                     size_t workspace_bytes, void* dX, float* dWqkv,
                     float* dWo, float* dbqkv, float* dbo, float* dgamma,
                     float* dbeta, void* stream) {
  return tp_attn_backward_qk(H, tokens, dZ, X, Wqkv, Wo, ln_gamma, workspace,
                             workspace_bytes, dX, dWqkv, dWo, dbqkv, dbo, dgamma,
                             dbeta, nullptr, nullptr, stream);
}

int tp_attn_backward_qk(tp_attn_handle* H, int tokens, const void* dZ,
                        const void* X, const void* Wqkv, const void* Wo,
                        const float* ln_gamma, void* workspace,
                        size_t workspace_bytes, void* dX, float* dWqkv,
                        float* dWo, float* dbqkv, float* dbo, float* dgamma,
                        float* dbeta, const tp_attn_qk* qk,
                        const tp_qk_norm_grads* qk_grads, void* stream) {
  if (H == nullptr) return TPMLP_ERR_ARG;
  const tp_attn_config& c = H->cfg;
  if (tokens < 0 || tokens > c.max_tokens || tokens % c.seq_len != 0)
    return TPMLP_ERR_SHAPE;
  if (!Wqkv || !Wo || !workspace || !dWqkv || !dWo ||
      (tokens > 0 && (!dZ || !X || !dX)))
    return TPMLP_ERR_ARG;
  if (c.use_layernorm && !ln_gamma) return TPMLP_ERR_ARG;
  TRY(check_ptrs({dZ, X, Wqkv, Wo, ln_gamma, workspace, dX, dWqkv, dWo, dbqkv,
                  dbo, dgamma, dbeta}));
  TRY(check_qk(H, qk, qk_grads));
  const AttnLayout L = attn_layout(H, tokens, 1);
  if (workspace_bytes < L.total) return TPMLP_ERR_WORKSPACE;
  int sms = 0;
  TRY(check_device(&sms));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  const int T = tokens, h = c.hidden, ht = h / c.shards;
  const bool ln = c.use_layernorm != 0;

  if (T == 0) {
    const tp_qk_norm_grads none = {nullptr, nullptr, nullptr, nullptr};
    const tp_qk_norm_grads& qg = qk_grads != nullptr ? *qk_grads : none;
    const size_t d4 = size_t(h / c.heads) * 4;
    struct Zero {
      void* p;
      size_t n;
    } zs[] = {{qg.q_gamma, d4}, {qg.q_beta, d4}, {qg.k_gamma, d4}, {qg.k_beta, d4},
              {dWqkv, size_t(h) * 3 * h * 4}, {dWo, size_t(h) * h * 4},
              {dbqkv, size_t(3) * h * 4},      {dbo, size_t(h) * 4},
              {ln ? dgamma : nullptr, size_t(h) * 4},
              {ln ? dbeta : nullptr, size_t(h) * 4}};
    for (auto& z : zs) {
      if (!z.p) continue;
      const cudaError_t e = cudaMemsetAsync(z.p, 0, z.n, s);
      if (e != cudaSuccess) {
        set_detail("cudaMemsetAsync(zero gradients)", e);
        return TPMLP_ERR_CUDA;
      }
    }
    return TPMLP_OK;
  }

  float* part = reinterpret_cast<float*>(ws + L.part);
  const void* Xop = ln ? static_cast<const void*>(ws + L.xn) : X;
  void* ctx = ws + L.ctx;
  void* dctx = ws + L.dctx;
  void* dqkv = ws + L.dqkv;
  CUtensorMap ta, tb;
  const int kbT = (T + TC_BK - 1) / TC_BK;

  if (dbo) TRY(colsum(&H->core, "colsum_dbo", s, true, dZ, part, dbo, T, h));
  // dW_o = Ctx^T dZ
  GemmArgs gw = gemm_args(H, ws, L);
  gw.M = h; gw.N = h; gw.K = T; gw.kb_per_seg = kbT;
  gw.out = dWo; gw.ldo = h;
  TRY(mnmajor_map(&ta, ctx, T, h));
  TRY(mnmajor_map(&tb, dZ, T, h));
  TRY(tc_gemm(&H->core, "gemm_wgrad_dWo", s, sms, EPI_STORE_F32, true, true, ta,
              tb, gw));
  // dCtx = dZ W_o^T
  GemmArgs gc = gemm_args(H, ws, L);
  gc.M = T; gc.N = h; gc.K = h; gc.kb_per_seg = h / TC_BK;
  gc.out = dctx; gc.ldo = h;
  TRY(kmajor_map(&ta, dZ, T, h, TC_BM));
  TRY(kmajor_map(&tb, Wo, h, h, TC2_BN_HALF));
  TRY(tc_gemm(&H->core, "gemm_dctx", s, sms, EPI_BIAS_BF16, false, false, ta,
              tb, gc));
  // attention core backward
  AttnArgs aa = core_args(H, ws, L, T);
  aa.dctx = static_cast<const __nv_bfloat16*>(dctx);
  aa.delta = reinterpret_cast<float*>(ws + L.delta);
  aa.dqkv = static_cast<__nv_bfloat16*>(dqkv);
  CUtensorMap tqk128, tqk64, tv128, tv64, tdo128, tdo64, tctx128, tdqkv_out;
  TRY(encode_map(&tqk128, ws + L.qkr, 3ULL * h, T, 3ULL * h, 128));
  TRY(encode_map(&tqk64, ws + L.qkr, 3ULL * h, T, 3ULL * h, 64));
  TRY(encode_map(&tv128, ws + L.qkv, 3ULL * h, T, 3ULL * h, 128));
  TRY(encode_map(&tv64, ws + L.qkv, 3ULL * h, T, 3ULL * h, 64));
  TRY(encode_map(&tdo128, dctx, h, T, h, 128));
  TRY(encode_map(&tdo64, dctx, h, T, h, 64));
  TRY(encode_map(&tctx128, ctx, h, T, h, 128));
  TRY(out_map(&tdqkv_out, dqkv, false, T, 3 * h, 3LL * h));
  const int grid = (T / c.seq_len) * c.heads * aa.nq;
  aa.hs_group = std::max(1, sms / aa.nq);   // one backward CTA per SM
  // db_qkv = sum_T dQKV: both kernels write 32-row partials of what they
  // store (the chunks they stage for their TMA stores, and at d = 96 the
  // 32-column tails); one fixed-order pass sums them.  (With a norm or a
  // rotation the projection's dQ and dK exist only after their gradient: then
  // a pass over dQKV makes the sums.)
  float* part3 = part + size_t(L.chunks) * h;
  const bool fused_dbqkv = dbqkv != nullptr && H->qk() == nullptr;
  if (fused_dbqkv) {
    aa.colsum = part3;
    aa.ld_colsum = 3LL * h;
  }
  // the query kernel also writes delta = rowsum(dCtx * Ctx), which the
  // key/value kernel reads
  TRY(run(&H->core, "attn_bwd_dq", s, [&] {
    return launch_attn_dq(tqk128, tqk64, tv64, tdo128, tctx128, tdqkv_out, aa,
                          grid, s);
  }));
  TRY(run(&H->core, "attn_bwd_dkdv", s, [&] {
    return launch_attn_dkdv(tqk128, tv128, tqk64, tdo64, tdqkv_out, aa, grid, s);
  }));
  if (H->qk() != nullptr) {
    TRY(qk_backward(H, T, dqkv, ws + L.qkv, qk, qk_grads, ws + L.qkpart, s));
    if (dbqkv != nullptr)
      TRY(colsum(&H->core, "colsum_dbqkv", s, true, dqkv, part3, dbqkv, T,
                 3 * h));
  }
  if (fused_dbqkv) {
    TRY(run(&H->core, "colsum_finalize", s, [&] {
      return launch_colsum_finalize(part3, dbqkv, L.groups, 3 * h, s);
    }));
  }
  // dW_qkv = Xn^T dQKV
  GemmArgs gwq = gemm_args(H, ws, L);
  gwq.M = h; gwq.N = 3 * h; gwq.K = T; gwq.kb_per_seg = kbT;
  gwq.out = dWqkv; gwq.ldo = 3LL * h;
  TRY(mnmajor_map(&ta, Xop, T, h));
  TRY(mnmajor_map(&tb, dqkv, T, 3 * h));
  TRY(tc_gemm(&H->core, "gemm_wgrad_dWqkv", s, sms, EPI_STORE_F32, true, true,
              ta, tb, gwq));
  // dXn = sum_i dQKV_i W_qkv,i^T (segment i = shard i's 3 h_t columns)
  GemmArgs gx = gemm_args(H, ws, L);
  gx.M = T; gx.N = h; gx.K = 3 * h; gx.num_seg = c.shards;
  gx.kb_per_seg = 3 * ht / TC_BK;
  gx.out = ln ? static_cast<void*>(ws + L.dxn) : dX;
  gx.ldo = h;
  gx.out_f32 = ln ? 1 : 0;
  if (c.use_residual && !ln) {
    gx.aux = dZ;
    gx.ldaux = h;
  }
  TRY(kmajor_map(&ta, dqkv, T, 3 * h, TC_BM));
  TRY(kmajor_map(&tb, Wqkv, h, 3 * h, TC2_BN_HALF));
  TRY(tc_gemm(&H->core, "gemm_dx_shardsum", s, sms, EPI_SHARDSUM, false, false,
              ta, tb, gx));
  if (ln) {
    const float* dXn = reinterpret_cast<const float*>(ws + L.dxn);
    const float* mean = reinterpret_cast<const float*>(ws + L.mean);
    const float* rstd = reinterpret_cast<const float*>(ws + L.rstd);
    const void* dres = c.use_residual ? dZ : nullptr;
    float* pg = part3 + size_t(L.groups > L.chunks ? L.groups : L.chunks) * 3 * h;
    float* pb = pg + L.lnp * h;
    TRY(ln_backward(&H->core, s, true, dXn, X, mean, rstd, ln_gamma, dres, dX,
                    pg, pb, dgamma, dbeta, T, h));
  }
  return TPMLP_OK;
}

int tp_attn_check(tp_attn_handle* H, void* workspace, void* stream) {
  if (H == nullptr || workspace == nullptr) return TPMLP_ERR_ARG;
  return check_status(workspace, static_cast<cudaStream_t>(stream));
}

long long tp_attn_launch_count(const tp_attn_handle* handle) {
  return handle ? handle->core.launches : -1;
}

int tp_attn_set_timing(tp_attn_handle* handle, int enable) {
  if (handle == nullptr) return TPMLP_ERR_ARG;
  handle->core.timing = enable != 0;
  return TPMLP_OK;
}

int tp_attn_timing_get(tp_attn_handle* H, int index, const char** name,
                       long long* launches, double* total_ms) {
  if (H == nullptr) return TPMLP_ERR_ARG;
  return timing_get(&H->core, index, name, launches, total_ms);
}

int tp_attn_timing_reset(tp_attn_handle* H) {
  if (H == nullptr) return TPMLP_ERR_ARG;
  timing_get(&H->core, -1, nullptr, nullptr, nullptr);
  H->core.stats.clear();
  return TPMLP_OK;
}

int tp_attn_set_nvtx(tp_attn_handle* handle, int enable) {
  if (handle == nullptr || (enable != 0 && enable != 1)) return TPMLP_ERR_ARG;
  handle->core.nvtx = enable != 0;
  return TPMLP_OK;
}

int tp_attn_set_ln_prologue(tp_attn_handle* handle, int enable) {
  if (handle == nullptr || (enable != 0 && enable != 1)) return TPMLP_ERR_ARG;
  handle->ln_prologue = enable != 0;
  return TPMLP_OK;
}

int tp_attn_set_rope(tp_attn_handle* handle, const tp_rope_config* config) {
  if (handle == nullptr) return TPMLP_ERR_ARG;
  tp_rope_handle* r = nullptr;
  if (config != nullptr) {
    if (config->head_dim != handle->cfg.hidden / handle->cfg.heads) {
      set_detail_msg("rope: head_dim is not hidden / heads");
      return TPMLP_ERR_SHAPE;
    }
    TRY(tp_rope_create(config, &r));
  }
  tp_rope_destroy(handle->rope);
  handle->rope = r;
  return TPMLP_OK;
}

int tp_attn_set_qk_norm(tp_attn_handle* handle, int norm, float eps) {
  if (handle == nullptr ||
      (norm != 0 && norm != TPQK_RMSNORM && norm != TPQK_LAYERNORM))
    return TPMLP_ERR_ARG;
  if (norm != 0 && (!(eps >= 0.f) || !std::isfinite(eps))) return TPMLP_ERR_ARG;
  if (norm != 0 && handle->plain == nullptr) {
    tp_rope_config c;
    std::memset(&c, 0, sizeof(c));
    c.head_dim = handle->cfg.hidden / handle->cfg.heads;
    c.base = 1.0;
    TRY(tp_rope_create(&c, &handle->plain));
  }
  handle->qk_norm = norm;
  handle->qk_eps = eps;
  return TPMLP_OK;
}

int tp_attn_set_wait_budget(tp_attn_handle* handle, unsigned long long ns) {
  if (handle == nullptr) return TPMLP_ERR_ARG;
  handle->core.budget_ns = ns;
  return TPMLP_OK;
}

}  // extern "C"
