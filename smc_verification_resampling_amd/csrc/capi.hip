// capi.hip - extern "C" entry points of libsmcsd.so: argument validation, dtype
// dispatch and launch.  Declarations and the full contract are in include/smcsd.h.
#include <cmath>
#include <mutex>

#include "../../include/smcsd.h"
#include "internal.hpp"
#include "kv_layout.hpp"

using namespace smcsd;

namespace {

inline hipStream_t as_stream(void *s) { return reinterpret_cast<hipStream_t>(s); }

inline int hip_rc(hipError_t e) { return e == hipSuccess ? SMCSD_OK : SMCSD_EHIP; }

inline bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

}  // namespace

extern "C" {

int smcsd_version(void) { return SMCSD_VERSION; }

const char *smcsd_status_string(int code) {
  switch (code) {
    case SMCSD_OK: return "ok";
    case SMCSD_EINVAL: return "invalid argument";
    case SMCSD_EDTYPE: return "unsupported dtype";
    case SMCSD_EHIP: return "HIP launch error";
    case SMCSD_EWORKSPACE: return "workspace too small or missing";
    case SMCSD_ESCRATCH: return "call needs more scratch than the static array holds";
    case SMCSD_ST_NAN_INPUT: return "NaN or +inf logit";
    case SMCSD_ST_EMPTY_ROW: return "row with no finite logit";
    case SMCSD_ST_NOSPACE: return "block pool exhausted";
    case SMCSD_ST_DEGENERATE_WEIGHTS: return "all particle weights zero or NaN";
    case SMCSD_ST_BAD_INPUT: return "token, ancestor or block id out of range";
    case SMCSD_ST_KV_INCONSISTENT: return "block tables, refcounts and free stack disagree";
    default: return "unknown code";
  }
}

size_t smcsd_workspace_bytes(int op, int B, int N, int K, int V, int64_t P) {
  if (B < 0 || N < 0) return 0;
  const int64_t S = (int64_t)B * N;
  if (op == SMCSD_OP_VERIFY_SMC || op == SMCSD_OP_VERIFY_SPS) {
    if (K < 0 || K > kMaxK || V < 1 || V > kMaxV) return 0;
    return verify_ws_layout(S, K, V, op == SMCSD_OP_VERIFY_SPS ? 1 : 0).total;
  }
  if (op == SMCSD_OP_DRAFT) {
    if (V < 1 || V > kMaxV) return 0;
    return verify_ws_layout(S, 0, V, 0).total;
  }
  if (op == SMCSD_OP_KV) {
    if (P < 1) return 0;
    return kv_ws_layout(S, P).total;
  }
  if (op == SMCSD_OP_KV_CHECK) {
    if (P < 1 || P > INT32_MAX) return 0;
    return kv_check_ws_bytes(P);
  }
  if (op == SMCSD_OP_TREE_ATTN) {
    if (K < 1 || K > kMaxNodes || V < 1 || P < 1 || V % P || S > INT32_MAX || S * K > INT32_MAX ||
        S * K > INT64_MAX / 64 / V)
      return 0;
    return tree_attn_ws_bytes(B, N, K, V, P);
  }
  if (op == SMCSD_OP_LOGPROBS) {
    if (V < 1 || V > kMaxV || K < 0 || K > kMaxTop || K > V || S > INT32_MAX) return 0;
    return logprobs_ws_bytes(S, K, V);
  }
  if (op == SMCSD_OP_KV_FREE || op == SMCSD_OP_KV_COMPACT) {
    if (P < 1 || P > SMCSD_POOL_OPS_MAX_BLOCKS) return 0;
    return op == SMCSD_OP_KV_FREE ? kv_free_ws_bytes(P) : kv_compact_ws_bytes(P);
  }
  return 0;
}

}  // extern "C"

namespace {

// The verify's scratch for callers that cannot allocate: a file-scope device array, one copy
// per GPU, held until the process ends.  Host code never uses the array's name as an
// address: each device's copy is found once with hipGetSymbolAddress and kept.
constexpr size_t kStaticScratchBytes = SMCSD_STATIC_SCRATCH_BYTES;
static __device__ __align__(256) unsigned char scratch[kStaticScratchBytes];

constexpr int kMaxDevices = 64;
std::mutex g_scratch_mu;
void *g_scratch_ptr[kMaxDevices];

// The current device's copy of the array (looked up on its first use on that device).
int static_scratch(void **out) {
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return SMCSD_EHIP;
  std::lock_guard<std::mutex> lock(g_scratch_mu);
  if (!g_scratch_ptr[dev]) {
    void *p = nullptr;
    if (hipGetSymbolAddress(&p, HIP_SYMBOL(scratch)) != hipSuccess || !p) return SMCSD_EHIP;
    g_scratch_ptr[dev] = p;
  }
  *out = g_scratch_ptr[dev];
  return SMCSD_OK;
}

// smcsd_verify with the workspace either given (static_ws = false) or the library's array.
int verify_impl(const void *target_logits, const void *draft_logits, int dtype,
                int64_t row_stride, int seq_step, const int32_t *draft_tokens, int B, int N, int K,
                int V, float temperature, float alpha, int mode, uint64_t seed, uint64_t step,
                const float *lse_in, const float *logq_in, float *log_weights,
                int32_t *out_tokens, int32_t *out_num_tokens, float *out_logp, float *out_logq,
                float *out_lse, int32_t *status, void *workspace, size_t workspace_bytes,
                bool static_ws, void *stream) {
  if (dtype != SMCSD_DTYPE_F32 && dtype != SMCSD_DTYPE_BF16) return SMCSD_EDTYPE;
  if (mode != SMCSD_MODE_SMC && mode != SMCSD_MODE_SPS && mode != SMCSD_MODE_SMC_RACE)
    return SMCSD_EINVAL;
  const bool smc = mode != SMCSD_MODE_SPS;
  if (B < 0 || N < 0 || K < 0 || K > kMaxK || V < 1 || V > kMaxV || seq_step < 1)
    return SMCSD_EINVAL;
  if (row_stride < V) return SMCSD_EINVAL;
  if (!(temperature > 0.0f) || !std::isfinite(temperature) || !std::isfinite(alpha))
    return SMCSD_EINVAL;
  const int64_t S = (int64_t)B * N;
  if (S == 0) return SMCSD_OK;
  if (S > INT32_MAX / 2) return SMCSD_EINVAL;
  const size_t esz = dtype == SMCSD_DTYPE_BF16 ? 2 : 4;
  if (!target_logits || !aligned(target_logits, esz)) return SMCSD_EINVAL;
  if (logq_in && !smc) return SMCSD_EINVAL;
  if (K > 0 && (!draft_tokens || (!logq_in && (!draft_logits || !aligned(draft_logits, esz)))))
    return SMCSD_EINVAL;
  if (!out_tokens || !status) return SMCSD_EINVAL;
  if (smc && (!log_weights || lse_in)) return SMCSD_EINVAL;
  const size_t need = verify_ws_layout(S, K, V, mode == SMCSD_MODE_SPS ? 1 : 0).total;
  if (static_ws) {
    if (need > kStaticScratchBytes) return SMCSD_ESCRATCH;
    const int rc = static_scratch(&workspace);
    if (rc != SMCSD_OK) return rc;
    workspace_bytes = kStaticScratchBytes;
  }
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < need) return SMCSD_EWORKSPACE;

  VerifyArgs a{};
  a.tgt = target_logits;
  a.drf = draft_logits;
  a.dtype = dtype;
  a.row_stride = row_stride;
  a.seq_step = seq_step;
  a.draft_tokens = draft_tokens;
  a.nseq = (int)S;
  a.K = K;
  a.V = V;
  a.c = (float)(1.4426950408889634073599246810018921 / (double)temperature);
  a.alpha = alpha;
  a.mode = mode;
  a.seed = seed;
  a.step = step;
  a.lse_in = lse_in;
  a.logq_in = logq_in;
  a.bonus_tag = 1u;
  a.log_weights = log_weights;
  a.out_tokens = out_tokens;
  a.out_num_tokens = out_num_tokens;
  a.out_logp = out_logp;
  a.out_logq = out_logq;
  a.out_lse = out_lse;
  a.status = status;
  a.ws = static_cast<char *>(workspace);
  a.stream = as_stream(stream);
  return hip_rc(launch_verify(a));
}

}  // namespace

extern "C" {

int smcsd_verify(const void *target_logits, const void *draft_logits, int dtype,
                 int64_t row_stride, int seq_step, const int32_t *draft_tokens, int B, int N,
                 int K, int V, float temperature, float alpha, int mode, uint64_t seed,
                 uint64_t step, const float *lse_in, const float *logq_in, float *log_weights,
                 int32_t *out_tokens, int32_t *out_num_tokens, float *out_logp, float *out_logq,
                 float *out_lse, int32_t *status, void *workspace, size_t workspace_bytes,
                 void *stream) {
  return verify_impl(target_logits, draft_logits, dtype, row_stride, seq_step, draft_tokens, B,
                     N, K, V, temperature, alpha, mode, seed, step, lse_in, logq_in, log_weights,
                     out_tokens, out_num_tokens, out_logp, out_logq, out_lse, status, workspace,
                     workspace_bytes, false, stream);
}

int smcsd_verify_static(const void *target_logits, const void *draft_logits, int dtype,
                        int64_t row_stride, int seq_step, const int32_t *draft_tokens, int B,
                        int N, int K, int V, float temperature, float alpha, int mode,
                        uint64_t seed, uint64_t step, const float *lse_in, const float *logq_in,
                        float *log_weights, int32_t *out_tokens, int32_t *out_num_tokens,
                        float *out_logp, float *out_logq, float *out_lse, int32_t *status,
                        void *stream) {
  return verify_impl(target_logits, draft_logits, dtype, row_stride, seq_step, draft_tokens, B,
                     N, K, V, temperature, alpha, mode, seed, step, lse_in, logq_in, log_weights,
                     out_tokens, out_num_tokens, out_logp, out_logq, out_lse, status, nullptr, 0,
                     true, stream);
}

int smcsd_draft_sample(const void *draft_logits, int dtype, int64_t row_stride, int n, int V,
                       float temperature, uint64_t seed, uint64_t step, int pos,
                       int32_t *out_tokens, float *out_logq, int32_t *status, void *workspace,
                       size_t workspace_bytes, void *stream) {
  if (dtype != SMCSD_DTYPE_F32 && dtype != SMCSD_DTYPE_BF16) return SMCSD_EDTYPE;
  if (n < 0 || V < 1 || V > kMaxV || row_stride < V || pos < 0 || pos >= (1 << 24))
    return SMCSD_EINVAL;
  if (!(temperature > 0.0f) || !std::isfinite(temperature)) return SMCSD_EINVAL;
  if (n == 0) return SMCSD_OK;
  const size_t esz = dtype == SMCSD_DTYPE_BF16 ? 2 : 4;
  if (!draft_logits || !aligned(draft_logits, esz) || !out_tokens || !status) return SMCSD_EINVAL;
  const size_t need = verify_ws_layout(n, 0, V, 0).total;
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < need) return SMCSD_EWORKSPACE;
  // the row-K draw of a verify with K = 0 over the draft rows, with the draft's RNG tag
  VerifyArgs a{};
  a.tgt = draft_logits;
  a.drf = nullptr;
  a.dtype = dtype;
  a.row_stride = row_stride;
  a.seq_step = 1;
  a.draft_tokens = nullptr;
  a.nseq = n;
  a.K = 0;
  a.V = V;
  a.c = (float)(1.4426950408889634073599246810018921 / (double)temperature);
  a.alpha = 1.0f;
  a.mode = SMCSD_MODE_SMC;
  a.seed = seed;
  a.step = step;
  a.log_weights = nullptr;
  a.out_tokens = out_tokens;
  a.out_logp = out_logq;
  a.status = status;
  a.ws = static_cast<char *>(workspace);
  a.stream = as_stream(stream);
  a.bonus_tag = 5u | ((uint32_t)pos << 8);
  return hip_rc(launch_verify(a));
}

int smcsd_resample(float *log_weights, int B, int N, float tau, uint64_t seed, uint64_t step,
                   int32_t *ancestors, float *ess, int32_t *resampled, int32_t *status,
                   void *stream) {
  if (B < 0 || N < 1 || N > kMaxN || !std::isfinite(tau)) return SMCSD_EINVAL;
  if (B == 0) return SMCSD_OK;
  if (!log_weights || !ancestors || !ess || !resampled || !status) return SMCSD_EINVAL;
  return hip_rc(launch_resample(log_weights, B, N, tau, seed, step, ancestors, ess, resampled,
                                status, as_stream(stream)));
}

// Host checks of a KV reassign call (SMCSD_OK to go ahead, 1 for an empty batch).
static int kv_check(int B, int N, const int32_t *block_tables, int M_cap, int block_size,
                    int64_t seq_len, int reserve_tokens, const int32_t *refcounts,
                    const int32_t *free_list, const int32_t *free_top, int64_t P, const int32_t *cow,
                    const int32_t *cow_count, const int32_t *status, const void *workspace,
                    size_t workspace_bytes) {
  if (B < 0 || N < 1 || N > kMaxN || M_cap < 1 || block_size < 1 || seq_len < 0 ||
      reserve_tokens < 0 || P < 1 || P > INT32_MAX)
    return SMCSD_EINVAL;
  if (ceil_div(seq_len + reserve_tokens, block_size) > M_cap) return SMCSD_EINVAL;
  if (B == 0) return 1;
  if ((int64_t)B * N * M_cap >= INT32_MAX) return SMCSD_EINVAL;  // 32-bit table indexing
  // one exchange workgroup per prompt part: the dispatch must stay under 2^32 threads
  const KvSplit ks = kv_split(N, (int)ceil_div(seq_len, block_size), (int)(seq_len % block_size));
  if ((int64_t)B * ks.parts * kKvThreads > (int64_t)0xFFFFFFFF) return SMCSD_EINVAL;
  if (!block_tables || !refcounts || !free_list || !free_top || !cow || !cow_count || !status)
    return SMCSD_EINVAL;
  const size_t need = kv_ws_layout((int64_t)B * N, P).total;
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < need) return SMCSD_EWORKSPACE;
  return SMCSD_OK;
}

int smcsd_kv_reassign(const int32_t *ancestors, const int32_t *resampled, int B, int N,
                      int32_t *block_tables, int M_cap, int block_size, int64_t seq_len,
                      int reserve_tokens, int32_t *refcounts, int32_t *free_list,
                      int32_t *free_top, int64_t P, int32_t *cow, int32_t *cow_count,
                      int32_t *status, void *workspace, size_t workspace_bytes, void *stream) {
  const int chk = kv_check(B, N, block_tables, M_cap, block_size, seq_len, reserve_tokens,
                           refcounts, free_list, free_top, P, cow, cow_count, status, workspace,
                           workspace_bytes);
  if (chk == 1) return SMCSD_OK;
  if (chk != SMCSD_OK) return chk;
  if (!ancestors || !resampled) return SMCSD_EINVAL;
  const FusedResample none{};
  return hip_rc(launch_kv(ancestors, resampled, none, B, N, block_tables, M_cap, block_size,
                          seq_len, reserve_tokens, refcounts, free_list, free_top, P, cow,
                          cow_count, status, static_cast<char *>(workspace), as_stream(stream)));
}

int smcsd_resample_kv_reassign(float *log_weights, int B, int N, float tau, uint64_t seed,
                               uint64_t step, int32_t *ancestors, float *ess, int32_t *resampled,
                               int32_t *block_tables, int M_cap, int block_size, int64_t seq_len,
                               int reserve_tokens, int32_t *refcounts, int32_t *free_list,
                               int32_t *free_top, int64_t P, int32_t *cow, int32_t *cow_count,
                               int32_t *status, void *workspace, size_t workspace_bytes,
                               void *stream) {
  if (!std::isfinite(tau)) return SMCSD_EINVAL;
  const int chk = kv_check(B, N, block_tables, M_cap, block_size, seq_len, reserve_tokens,
                           refcounts, free_list, free_top, P, cow, cow_count, status, workspace,
                           workspace_bytes);
  if (chk == 1) return SMCSD_OK;
  if (chk != SMCSD_OK) return chk;
  if (!log_weights || !ancestors || !ess || !resampled) return SMCSD_EINVAL;
  const FusedResample fr{log_weights, tau, seed, step, ancestors, ess, resampled};
  return hip_rc(launch_kv(nullptr, nullptr, fr, B, N, block_tables, M_cap, block_size, seq_len,
                          reserve_tokens, refcounts, free_list, free_top, P, cow, cow_count,
                          status, static_cast<char *>(workspace), as_stream(stream)));
}

int smcsd_step(const void *target_logits, const void *draft_logits, int dtype, int64_t row_stride,
               const int32_t *draft_tokens, int B, int N, int K, int V, float temperature,
               float alpha, int mode, float tau, uint64_t seed, uint64_t step,
               const float *logq_in, float *log_weights, int32_t *out_tokens,
               int32_t *out_num_tokens, float *out_logp, float *out_logq, float *out_lse,
               int32_t *ancestors, float *ess, int32_t *resampled, int32_t *block_tables,
               int M_cap, int block_size, int64_t seq_len, int reserve_tokens, int32_t *refcounts,
               int32_t *free_list, int32_t *free_top, int64_t P, int32_t *cow, int32_t *cow_count,
               int32_t *status, void *verify_workspace, size_t verify_workspace_bytes,
               void *kv_workspace, size_t kv_workspace_bytes, void *stream) {
  // the checks of smcsd_verify (SMC modes) and of smcsd_resample_kv_reassign
  if (dtype != SMCSD_DTYPE_F32 && dtype != SMCSD_DTYPE_BF16) return SMCSD_EDTYPE;
  if (mode != SMCSD_MODE_SMC && mode != SMCSD_MODE_SMC_RACE) return SMCSD_EINVAL;
  if (B < 0 || N < 1 || N > kMaxN || K < 0 || K > kMaxK || V < 1 || V > kMaxV) return SMCSD_EINVAL;
  if (row_stride < V) return SMCSD_EINVAL;
  if (!(temperature > 0.0f) || !std::isfinite(temperature) || !std::isfinite(alpha) ||
      !std::isfinite(tau))
    return SMCSD_EINVAL;
  const int chk = kv_check(B, N, block_tables, M_cap, block_size, seq_len, reserve_tokens,
                           refcounts, free_list, free_top, P, cow, cow_count, status, kv_workspace,
                           kv_workspace_bytes);
  if (chk == 1) return SMCSD_OK;
  if (chk != SMCSD_OK) return chk;
  const int64_t S = (int64_t)B * N;
  if (S > INT32_MAX / 2) return SMCSD_EINVAL;
  const size_t esz = dtype == SMCSD_DTYPE_BF16 ? 2 : 4;
  if (!target_logits || !aligned(target_logits, esz)) return SMCSD_EINVAL;
  if (K > 0 && (!draft_tokens || (!logq_in && (!draft_logits || !aligned(draft_logits, esz)))))
    return SMCSD_EINVAL;
  if (!out_tokens || !log_weights || !ancestors || !ess || !resampled) return SMCSD_EINVAL;
  const size_t need = verify_ws_layout(S, K, V, 0).total;
  if (!verify_workspace || !aligned(verify_workspace, 256) || verify_workspace_bytes < need)
    return SMCSD_EWORKSPACE;

  VerifyArgs a{};
  a.tgt = target_logits;
  a.drf = draft_logits;
  a.dtype = dtype;
  a.row_stride = row_stride;
  a.seq_step = 1;
  a.draft_tokens = draft_tokens;
  a.nseq = (int)S;
  a.K = K;
  a.V = V;
  a.c = (float)(1.4426950408889634073599246810018921 / (double)temperature);
  a.alpha = alpha;
  a.mode = mode;
  a.seed = seed;
  a.step = step;
  a.logq_in = logq_in;
  a.bonus_tag = 1u;
  a.log_weights = log_weights;
  a.out_tokens = out_tokens;
  a.out_num_tokens = out_num_tokens;
  a.out_logp = out_logp;
  a.out_logq = out_logq;
  a.out_lse = out_lse;
  a.status = status;
  a.ws = static_cast<char *>(verify_workspace);
  a.stream = as_stream(stream);
  // The verify's kernels, then the resample + exchange kernels on the same stream: the
  // latter read the log-weights the verify wrote.
  const hipError_t e = launch_verify(a);
  if (e != hipSuccess) return hip_rc(e);
  const FusedResample fr{log_weights, tau, seed, step, ancestors, ess, resampled};
  return hip_rc(launch_kv(nullptr, nullptr, fr, B, N, block_tables, M_cap, block_size, seq_len,
                          reserve_tokens, refcounts, free_list, free_top, P, cow, cow_count, status,
                          static_cast<char *>(kv_workspace), as_stream(stream)));
}

int smcsd_kv_check(const int32_t *block_tables, int64_t S, int M_cap, int slots,
                   const int32_t *refcounts, const int32_t *free_list, const int32_t *free_top,
                   int64_t P, int32_t *violations, int32_t *status, void *workspace,
                   size_t workspace_bytes, void *stream) {
  if (S < 0 || M_cap < 1 || slots < 0 || slots > M_cap || P < 1 || P > INT32_MAX)
    return SMCSD_EINVAL;
  if ((S > 0 && !block_tables) || !refcounts || !free_list || !free_top || !violations || !status)
    return SMCSD_EINVAL;
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < kv_check_ws_bytes(P))
    return SMCSD_EWORKSPACE;
  return hip_rc(launch_kv_check(block_tables, S, M_cap, slots, refcounts, free_list, free_top, P,
                                violations, status, static_cast<char *>(workspace),
                                as_stream(stream)));
}

int smcsd_kv_fork(const int32_t *forked, int B, int N, int32_t *block_tables, int M_cap,
                  int32_t *refcounts, int64_t P, int32_t *status, void *stream) {
  if (B < 0 || N < 1 || N > kMaxN || M_cap < 1 || P < 1 || P > INT32_MAX) return SMCSD_EINVAL;
  if (B == 0) return SMCSD_OK;
  if ((int64_t)B * N >= INT32_MAX || (int64_t)B * N * M_cap >= INT32_MAX) return SMCSD_EINVAL;
  if (!forked || !block_tables || !refcounts || !status) return SMCSD_EINVAL;
  return hip_rc(launch_kv_fork(forked, B, N, block_tables, M_cap, refcounts, P, status,
                               as_stream(stream)));
}

int smcsd_kv_free(const int32_t *freed, int64_t S, int32_t *block_tables, int M_cap,
                  int32_t *refcounts, int32_t *free_list, int32_t *free_top, int64_t P,
                  int32_t *status, void *workspace, size_t workspace_bytes, void *stream) {
  if (S < 0 || M_cap < 1 || P < 1 || P > SMCSD_POOL_OPS_MAX_BLOCKS || S >= INT32_MAX ||
      S * M_cap >= INT32_MAX)
    return SMCSD_EINVAL;
  if (S == 0) return SMCSD_OK;
  if (!freed || !block_tables || !refcounts || !free_list || !free_top || !status)
    return SMCSD_EINVAL;
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < kv_free_ws_bytes(P))
    return SMCSD_EWORKSPACE;
  return hip_rc(launch_kv_free(freed, S, block_tables, M_cap, refcounts, free_list, free_top, P,
                               status, static_cast<char *>(workspace), as_stream(stream)));
}

int smcsd_kv_compact(int32_t *block_tables, int64_t S, int M_cap, int block_size,
                     int32_t *refcounts, int32_t *free_list, int32_t *free_top, int64_t P,
                     int32_t *moves, int32_t *move_count, int32_t *status, void *workspace,
                     size_t workspace_bytes, void *stream) {
  if (S < 0 || M_cap < 1 || block_size < 1 || P < 1 || P > SMCSD_POOL_OPS_MAX_BLOCKS ||
      S >= INT32_MAX || S * M_cap >= INT32_MAX)
    return SMCSD_EINVAL;
  if ((S > 0 && !block_tables) || !refcounts || !free_list || !free_top || (P > 1 && !moves) ||
      !move_count || !status)
    return SMCSD_EINVAL;
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < kv_compact_ws_bytes(P))
    return SMCSD_EWORKSPACE;
  return hip_rc(launch_kv_compact(block_tables, S, M_cap, block_size, refcounts, free_list,
                                  free_top, P, moves, move_count, status,
                                  static_cast<char *>(workspace), as_stream(stream)));
}

int smcsd_kv_copy(void *const *caches, int n_caches, int64_t block_stride, int segments,
                  int64_t segment_stride, int64_t token_bytes, int block_size,
                  const int32_t *list, const int32_t *count, int64_t capacity, int64_t P,
                  int32_t *status, void *stream) {
  if (n_caches < 0 || n_caches > SMCSD_KV_COPY_MAX_CACHES || segments < 1 || token_bytes < 1 ||
      block_size < 1 || token_bytes > INT32_MAX || block_size * token_bytes > INT32_MAX ||
      block_stride < 0 || segment_stride < 0 || P < 1 || P > INT32_MAX || capacity < 0 ||
      capacity > INT32_MAX)
    return SMCSD_EINVAL;
  if (n_caches == 0 || capacity == 0) return SMCSD_OK;
  if (!caches || !list || !count || !status) return SMCSD_EINVAL;
  for (int i = 0; i < n_caches; ++i)
    if (!caches[i]) return SMCSD_EINVAL;
  return hip_rc(launch_kv_copy(caches, n_caches, block_stride, segments, segment_stride,
                               token_bytes, block_size, list, count, capacity, P, status,
                               as_stream(stream)));
}

// Host checks of a paged cache of 16-bit elements.
static bool paged_ok(const void *k, const void *v, int64_t page, int64_t token, int64_t head,
                     const int32_t *tables, int M_cap, int block_size, int64_t P, int D) {
  return k && v && aligned(k, 16) && aligned(v, 16) && page >= D && token >= D && head >= D &&
         page % 8 == 0 && token % 8 == 0 && head % 8 == 0 && tables && M_cap >= 1 &&
         block_size >= 1 && (int64_t)M_cap * block_size < INT32_MAX - 4096 && P >= 1 && P <= INT32_MAX;
}

int smcsd_qk_norm_rope(const void *q, const void *k, const void *v, int dtype, int64_t q_stride,
                       int64_t k_stride, int64_t v_stride, int S, int R, int Hq, int Hkv, int D,
                       const void *q_weight, const void *k_weight, float eps,
                       const float *cos_sin, int64_t max_pos, int rot_dim, int interleaved,
                       const int32_t *positions, const int32_t *ctx_lens,
                       const int32_t *num_nodes, const int32_t *block_tables, int M_cap,
                       int block_size, int64_t P, void *k_cache, void *v_cache,
                       int64_t page_stride, int64_t token_stride, int64_t head_stride,
                       void *q_out, int32_t *status, void *stream) {
  if (dtype != SMCSD_DTYPE_BF16 && dtype != SMCSD_DTYPE_F16) return SMCSD_EDTYPE;
  if (S < 0 || R < 1 || Hq < 1 || Hkv < 1 || Hq > INT32_MAX / 4 || Hkv > INT32_MAX / 8 || D < 8 ||
      D > kMaxHeadDim || D % 8 || rot_dim < 0 || rot_dim > D || rot_dim % 16 || max_pos < 0 ||
      !(eps >= 0.0f) || !std::isfinite(eps))
    return SMCSD_EINVAL;
  if (S == 0) return SMCSD_OK;
  if ((int64_t)Hq * D >= INT32_MAX || (int64_t)Hkv * D >= INT32_MAX || (int64_t)S * R >= INT32_MAX ||
      (int64_t)S * R * (Hq + 2 * Hkv) >= INT32_MAX ||
      (int64_t)S * M_cap >= INT32_MAX)
    return SMCSD_EINVAL;
  if (q_stride < (int64_t)Hq * D || k_stride < (int64_t)Hkv * D || v_stride < (int64_t)Hkv * D ||
      q_stride % 8 || k_stride % 8 || v_stride % 8)
    return SMCSD_EINVAL;
  if (!q || !k || !v || !q_out || !aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) ||
      !aligned(q_out, 16) || !aligned(q_weight, 16) || !aligned(k_weight, 16) ||
      !aligned(cos_sin, 16) || (rot_dim > 0 && !cos_sin) || !ctx_lens || !status)
    return SMCSD_EINVAL;
  if (!paged_ok(k_cache, v_cache, page_stride, token_stride, head_stride, block_tables, M_cap,
                block_size, P, D))
    return SMCSD_EINVAL;
  QkNormRopeArgs a{};
  a.q = static_cast<const uint16_t *>(q);
  a.k = static_cast<const uint16_t *>(k);
  a.v = static_cast<const uint16_t *>(v);
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.S = S;
  a.R = R;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.D = D;
  a.q_weight = static_cast<const uint16_t *>(q_weight);
  a.k_weight = static_cast<const uint16_t *>(k_weight);
  a.eps = eps;
  a.cos_sin = cos_sin;
  a.max_pos = max_pos;
  a.rot_dim = rot_dim;
  a.interleaved = interleaved;
  a.positions = positions;
  a.ctx_lens = ctx_lens;
  a.num_nodes = num_nodes;
  a.cache = PagedCache{page_stride, token_stride, head_stride, block_tables, M_cap, block_size, P};
  a.k_cache = static_cast<uint16_t *>(k_cache);
  a.v_cache = static_cast<uint16_t *>(v_cache);
  a.q_out = static_cast<uint16_t *>(q_out);
  a.status = status;
  return hip_rc(launch_qk_norm_rope(a, dtype, as_stream(stream)));
}

int smcsd_tree_attention(const void *q, int dtype, int64_t q_stride, const void *k_cache,
                         const void *v_cache, int64_t page_stride, int64_t token_stride,
                         int64_t head_stride, const int32_t *block_tables, int M_cap,
                         int block_size, int64_t P, const int32_t *ctx_lens,
                         const int32_t *num_nodes, const uint64_t *tree_mask, int B, int N, int R,
                         int Hq, int Hkv, int D, float scale, int64_t max_len, void *out,
                         float *lse, int32_t *status, void *workspace, size_t workspace_bytes,
                         void *stream) {
  if (dtype != SMCSD_DTYPE_BF16 && dtype != SMCSD_DTYPE_F16) return SMCSD_EDTYPE;
  if (B < 0 || N < 0 || R < 1 || R > kMaxNodes || Hq < 1 || Hkv < 1 || Hq % Hkv || D < 8 ||
      D > kMaxHeadDim || D % 8 || !(std::fabs(scale) <= 0x1p127f) || max_len < 0)
    return SMCSD_EINVAL;  // (times log2(e), a scale past 2^127 could be infinite)
  const int64_t S = (int64_t)B * N;
  if (S == 0) return SMCSD_OK;
  if (S >= INT32_MAX || S * R >= INT32_MAX || S * R * Hq > kMaxAttnRows || (int64_t)Hq * D >= INT32_MAX ||
      S * M_cap >= INT32_MAX)
    return SMCSD_EINVAL;
  if (q_stride < (int64_t)Hq * D || q_stride % 8 || !q || !aligned(q, 16) || !out ||
      !aligned(out, 16) || !ctx_lens || !status || !aligned(tree_mask, 8))
    return SMCSD_EINVAL;
  if (!paged_ok(k_cache, v_cache, page_stride, token_stride, head_stride, block_tables, M_cap,
                block_size, P, D))
    return SMCSD_EINVAL;
  if (!workspace || !aligned(workspace, 256) ||
      workspace_bytes < tree_attn_ws_bytes(B, N, R, (int64_t)Hq * D, Hkv))
    return SMCSD_EWORKSPACE;
  TreeAttnArgs a{};
  a.q = static_cast<const uint16_t *>(q);
  a.k_cache = static_cast<const uint16_t *>(k_cache);
  a.v_cache = static_cast<const uint16_t *>(v_cache);
  a.q_stride = q_stride;
  a.cache = PagedCache{page_stride, token_stride, head_stride, block_tables, M_cap, block_size, P};
  a.ctx_lens = ctx_lens;
  a.num_nodes = num_nodes;
  a.tree_mask = tree_mask;
  a.B = B;
  a.N = N;
  a.R = R;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.D = D;
  a.scale = scale;
  a.max_len = max_len;
  a.out = static_cast<uint16_t *>(out);
  a.lse = lse;
  a.status = status;
  a.ws = static_cast<char *>(workspace);
  return hip_rc(launch_tree_attn(a, dtype, as_stream(stream)));
}

int smcsd_token_logprobs(const void *logits, int dtype, int64_t row_stride, int n, int V,
                         float temperature, const int32_t *tokens, int C, int k,
                         float *out_logp, float *out_entropy, float *out_lse, int32_t *top_ids,
                         float *top_logp, int32_t *status, void *workspace,
                         size_t workspace_bytes, void *stream) {
  if (dtype != SMCSD_DTYPE_F32 && dtype != SMCSD_DTYPE_BF16) return SMCSD_EDTYPE;
  if (n < 0 || V < 1 || V > kMaxV || row_stride < V || C < 0 || C > kMaxGiven || k < 0 ||
      k > kMaxTop || k > V)
    return SMCSD_EINVAL;
  if (!(temperature > 0.0f) || !std::isfinite(temperature)) return SMCSD_EINVAL;
  const float c = (float)(1.4426950408889634073599246810018921 / (double)temperature);
  if (!std::isfinite(c)) return SMCSD_EINVAL;  // differences of logits are multiplied by it
  if (n == 0) return SMCSD_OK;
  const size_t esz = dtype == SMCSD_DTYPE_BF16 ? 2 : 4;
  if (!logits || !aligned(logits, esz) || !status || (C > 0 && out_logp && !tokens))
    return SMCSD_EINVAL;
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < logprobs_ws_bytes(n, k, V))
    return SMCSD_EWORKSPACE;
  LogprobsArgs a{};
  a.logits = static_cast<const char *>(logits);
  a.row_bytes = row_stride * (int64_t)esz;
  a.n = n;
  a.V = V;
  a.c = c;
  a.inv_T = 1.0 / (double)temperature;
  a.tokens = tokens;
  a.C = C;
  a.k = k;
  a.logp = out_logp;
  a.entropy = out_entropy;
  a.lse = out_lse;
  a.top_ids = top_ids;
  a.top_logp = top_logp;
  a.status = status;
  a.ws = static_cast<char *>(workspace);
  return hip_rc(launch_logprobs(a, dtype, as_stream(stream)));
}

int smcsd_stream_read(const void *p, int64_t bytes, uint32_t *tile_xor, void *stream) {
  if (bytes < 0 || bytes > SMCSD_STREAM_READ_MAX_BYTES || (bytes & 15)) return SMCSD_EINVAL;
  if (bytes == 0) return SMCSD_OK;
  if (!p || !aligned(p, 16) || !tile_xor) return SMCSD_EINVAL;
  return hip_rc(launch_stream_read(p, bytes, tile_xor, as_stream(stream)));
}

int smcsd_philox4x32_10(const uint32_t *counters, const uint32_t *keys, int n, uint32_t *out,
                        void *stream) {
  if (n < 0) return SMCSD_EINVAL;
  if (n == 0) return SMCSD_OK;
  if (!counters || !keys || !out) return SMCSD_EINVAL;
  return hip_rc(launch_philox(counters, keys, n, out, as_stream(stream)));
}

}  // extern "C"
