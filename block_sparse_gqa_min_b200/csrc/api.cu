// extern "C" entry points of libsba.so: argument validation on the host, then
// the kernel launches of the other files.  Nothing here allocates, keeps state
// or synchronises.
#include <stdint.h>

#include <initializer_list>

#include "common.cuh"
#include "kv4.cuh"
#include "launch.cuh"

using namespace sba;

namespace sba {
namespace {
thread_local cudaError_t g_last = cudaSuccess;
}
void note_cuda_error(cudaError_t e) { g_last = e; }
cudaError_t last_cuda_error() { return g_last; }
}  // namespace sba

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace

namespace sba {
// Checks shared by every call that takes a cache.
int check_cache(const sba_cache* c) {
    if (!c || !c->k || !c->v || !c->seq_lens) return SBA_ERR_INVALID_ARG;
    if (!aligned16(c->k) || !aligned16(c->v)) return SBA_ERR_INVALID_ARG;
    if (c->B < 1 || c->H_kv < 1 || c->H_q < 1 || c->H_q % c->H_kv != 0) return SBA_ERR_INVALID_ARG;
    if (c->max_blocks < 1 || c->num_pages < 1 || c->max_len < 0) return SBA_ERR_INVALID_ARG;
    if (c->d != kHeadDim) return SBA_ERR_UNSUPPORTED;
    if (c->b != 64 && c->b != 128) return SBA_ERR_UNSUPPORTED;
    if (c->H_q / c->H_kv > kMaxGroup) return SBA_ERR_UNSUPPORTED;
    if (c->max_blocks > kMaxBlocksPerSeq) return SBA_ERR_UNSUPPORTED;
    if ((int64_t)c->max_len > (int64_t)c->max_blocks * c->b) return SBA_ERR_INVALID_ARG;
    if (!c->block_table && (int64_t)c->num_pages < (int64_t)c->B * c->max_blocks) return SBA_ERR_INVALID_ARG;
    // TMA row coordinates are signed 32-bit
    if ((int64_t)c->num_pages * c->H_kv * c->b >= (int64_t)1 << 31) return SBA_ERR_UNSUPPORTED;
    if (c->desc && !aligned16(c->desc)) return SBA_ERR_INVALID_ARG;
    if (c->kg && !aligned16(c->kg)) return SBA_ERR_INVALID_ARG;
    return SBA_OK;
}
}  // namespace sba

namespace {

int check_params(const sba_select_params* p) {
    if (!p) return SBA_ERR_INVALID_ARG;
    if (p->n_budget < 0 || p->n_local < 0 || p->n_min < 0) return SBA_ERR_INVALID_ARG;
    if (p->keep_den < 0 || p->keep_num < 0 || (p->keep_den > 0 && p->keep_num > p->keep_den))
        return SBA_ERR_INVALID_ARG;
    if (p->scorer != SBA_SCORER_QUEST && p->scorer != SBA_SCORER_GATE) return SBA_ERR_INVALID_ARG;
    if (p->log_gate < SBA_LOG_GATE_OFF || p->log_gate > SBA_LOG_GATE_OUTER) return SBA_ERR_INVALID_ARG;
    if (p->gate_act < SBA_GATE_SOFTMAX || p->gate_act > SBA_GATE_RAW) return SBA_ERR_INVALID_ARG;
    if (p->scorer == SBA_SCORER_QUEST && (p->log_gate != 0 || p->gate_act != 0)) return SBA_ERR_INVALID_ARG;
    return SBA_OK;
}

}  // namespace

namespace sba {
// Every host-side check of sba_score_select except the workspace (also used by the
// allocation-free variant, which must reject a call before it enqueues anything).
int check_score_select(const sba_cache* c, const void* q, const sba_select_params* p, const int32_t* sel_idx,
                       const int32_t* sel_cnt, int32_t n_max) {
    int rc = check_cache(c);
    if (rc != SBA_OK) return rc;
    rc = check_params(p);
    if (rc != SBA_OK) return rc;
    if (!q || !sel_idx || !sel_cnt || n_max < 1 || !aligned16(q)) return SBA_ERR_INVALID_ARG;
    if (p->scorer == SBA_SCORER_QUEST && !c->desc) return SBA_ERR_INVALID_ARG;
    if (p->scorer == SBA_SCORER_GATE && !c->kg) return SBA_ERR_INVALID_ARG;
    const int n_need = num_selected((c->max_len + c->b - 1) / c->b, *p);
    if (n_max < n_need) return SBA_ERR_INVALID_ARG;
    return SBA_OK;
}
}  // namespace sba

namespace {

int after_launch(int rc) {
    if (rc != SBA_OK) return rc;
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) return SBA_OK;
    note_cuda_error(e);
    return SBA_ERR_CUDA;
}

}  // namespace

extern "C" {

const char* sba_status_string(int status) {
    switch (status) {
        case SBA_OK: return "ok";
        case SBA_ERR_INVALID_ARG: return "invalid argument (null, misaligned or inconsistent sizes)";
        case SBA_ERR_UNSUPPORTED: return "unsupported shape (d must be 128, b 64 or 128, G <= 16)";
        case SBA_ERR_WORKSPACE: return "workspace missing or too small";
        case SBA_ERR_CUDA: return "CUDA launch or runtime error";
        default: return "unknown status";
    }
}

const char* sba_last_cuda_error(void) {
    const cudaError_t e = last_cuda_error();
    return e == cudaSuccess ? "no error" : cudaGetErrorString(e);
}

int sba_selftest_wait_timeout(int32_t* status, uint64_t limit_ns, void* stream) {
    if (!status || limit_ns == 0 || limit_ns > 10000000000ull) return SBA_ERR_INVALID_ARG;
    return after_launch(launch_wait_timeout_selftest(status, limit_ns, static_cast<cudaStream_t>(stream)));
}

int sba_selftest_wait_vote(int32_t* status, int32_t* verdicts, uint64_t limit_ns, void* stream) {
    if (!status || !verdicts || limit_ns == 0 || limit_ns > 1000000000ull) return SBA_ERR_INVALID_ARG;
    return after_launch(
        launch_wait_vote_selftest(status, verdicts, limit_ns, static_cast<cudaStream_t>(stream)));
}

int32_t sba_num_selected(int32_t N, const sba_select_params* p) {
    if (!p) return -1;
    return num_selected(N, *p);
}

int32_t sba_budget_from_sparsity(int32_t N, int32_t keep_num, int32_t keep_den) {
    if (keep_den <= 0 || N <= 0 || keep_num < 0) return 0;
    return (int32_t)(((int64_t)N * keep_num + keep_den - 1) / keep_den);
}

int32_t sba_default_num_splits(const sba_cache* c, int32_t n_max, int32_t num_sms) {
    if (!c || c->B < 1 || c->H_kv < 1 || n_max < 1) return 1;
    if (num_sms < 1) num_sms = 148;
    const int64_t units = (int64_t)c->B * c->H_kv;
    int64_t s = num_sms / units;  // one wave of one-CTA-per-SM decode CTAs
    if (s < 1) s = 1;
    if (s > n_max) s = n_max;
    return (int32_t)s;
}

size_t sba_workspace_size(const sba_cache* c, const sba_select_params* p) {
    if (check_cache(c) != SBA_OK || check_params(p) != SBA_OK) return 0;
    return score_workspace_bytes(*c, *p);
}

int sba_append_kv(const sba_cache* c, const void* k_new, const void* v_new, const int32_t* pos_start, int32_t n_new,
                  void* stream) {
    int rc = check_cache(c);
    if (rc != SBA_OK) return rc;
    if (!k_new || !v_new || !pos_start || n_new < 0) return SBA_ERR_INVALID_ARG;
    if (!aligned16(k_new) || !aligned16(v_new)) return SBA_ERR_INVALID_ARG;
    if (n_new == 0) return SBA_OK;
    return after_launch(launch_append_kv(*c, k_new, v_new, pos_start, n_new, static_cast<cudaStream_t>(stream)));
}

int sba_update_descriptors(const sba_cache* c, const int32_t* pos_start, int32_t n_new, const sba_gate* gate,
                           void* stream) {
    int rc = check_cache(c);
    if (rc != SBA_OK) return rc;
    if (!pos_start || n_new < 0) return SBA_ERR_INVALID_ARG;
    if (gate && (!gate->Wq || !gate->Wk || gate->dg < 1 || gate->dg > 256 || !c->kg)) return SBA_ERR_INVALID_ARG;
    if (!c->desc && !gate) return SBA_ERR_INVALID_ARG;
    if (n_new == 0) return SBA_OK;
    return after_launch(launch_update_descriptors(*c, pos_start, n_new, gate, static_cast<cudaStream_t>(stream)));
}

int sba_score_select(const sba_cache* c, const void* q, const sba_select_params* p, int32_t* sel_idx,
                     int32_t* sel_cnt, float* gate_bias, int32_t n_max, void* ws, size_t ws_bytes, void* stream) {
    const int rc = check_score_select(c, q, p, sel_idx, sel_cnt, n_max);
    if (rc != SBA_OK) return rc;
    if (!ws || !aligned16(ws) || ws_bytes < score_workspace_bytes(*c, *p)) return SBA_ERR_WORKSPACE;
    return after_launch(launch_score_select(*c, q, 1, *p, sel_idx, sel_cnt, p->scorer == SBA_SCORER_GATE ? gate_bias : nullptr,
                                            n_max, ws, static_cast<cudaStream_t>(stream)));
}

// a softmax scale is positive and finite
static bool good_scale(float s) { return s > 0.f && s <= 3.4028234e38f; }

static int sparse_decode_any(const sba_cache* c, const void* q, const int32_t* sel_idx, const int32_t* sel_cnt,
                             const float* gate_bias, int32_t n_max, float softmax_scale, int32_t num_splits,
                             float* o_part, float* lse_part, bool outer, void* stream) {
    int rc = check_cache(c);
    if (rc != SBA_OK) return rc;
    if (!q || !sel_idx || !sel_cnt || !o_part || !lse_part || n_max < 1) return SBA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(o_part)) return SBA_ERR_INVALID_ARG;
    if (num_splits < 1 || num_splits > 65535) return SBA_ERR_INVALID_ARG;
    if (!good_scale(softmax_scale)) return SBA_ERR_INVALID_ARG;
    if (outer && !gate_bias) return SBA_ERR_INVALID_ARG;
    return after_launch(launch_sparse_decode(*c, q, sel_idx, sel_cnt, gate_bias, n_max, softmax_scale, num_splits,
                                             o_part, lse_part, outer, static_cast<cudaStream_t>(stream)));
}

int sba_sparse_decode(const sba_cache* c, const void* q, const int32_t* sel_idx, const int32_t* sel_cnt,
                      const float* gate_bias, int32_t n_max, float softmax_scale, int32_t num_splits, float* o_part,
                      float* lse_part, void* stream) {
    return sparse_decode_any(c, q, sel_idx, sel_cnt, gate_bias, n_max, softmax_scale, num_splits, o_part, lse_part,
                             false, stream);
}

int sba_sparse_decode_outer(const sba_cache* c, const void* q, const int32_t* sel_idx, const int32_t* sel_cnt,
                            const float* gate_bias, int32_t n_max, float softmax_scale, int32_t num_splits,
                            float* o_part, float* lse_part, void* stream) {
    return sparse_decode_any(c, q, sel_idx, sel_cnt, gate_bias, n_max, softmax_scale, num_splits, o_part, lse_part,
                             true, stream);
}

int sba_score_select_multi(const sba_cache* c, const void* q, int32_t M, const sba_select_params* p,
                           int32_t* sel_idx, int32_t* sel_cnt, int32_t n_max, void* ws, size_t ws_bytes,
                           void* stream) {
    const int rc = check_score_select(c, q, p, sel_idx, sel_cnt, n_max);
    if (rc != SBA_OK) return rc;
    if (M < 1 || M > kMaxQueryTokens) return SBA_ERR_INVALID_ARG;
    if (p->scorer != SBA_SCORER_QUEST) return SBA_ERR_UNSUPPORTED;
    if (!ws || !aligned16(ws) || ws_bytes < score_workspace_bytes(*c, *p)) return SBA_ERR_WORKSPACE;
    return after_launch(launch_score_select(*c, q, M, *p, sel_idx, sel_cnt, nullptr, n_max, ws,
                                            static_cast<cudaStream_t>(stream)));
}

static int check_multi(const sba_cache* c, const void* q, int32_t M, float softmax_scale, int32_t num_splits,
                       const float* o_part, const float* lse_part) {
    const int rc = check_cache(c);
    if (rc != SBA_OK) return rc;
    if (!q || !o_part || !lse_part || !aligned16(q)) return SBA_ERR_INVALID_ARG;
    if (M < 1 || M > kMaxQueryTokens) return SBA_ERR_INVALID_ARG;
    if (num_splits < 1 || num_splits > 65535) return SBA_ERR_INVALID_ARG;
    if (!good_scale(softmax_scale)) return SBA_ERR_INVALID_ARG;
    if ((int64_t)c->H_kv * mq_row_groups(*c, M) > 65535 || c->B > 65535) return SBA_ERR_UNSUPPORTED;
    return SBA_OK;
}

int32_t sba_multi_row_groups(const sba_cache* c, int32_t M) {
    if (check_cache(c) != SBA_OK || M < 1) return 0;
    return mq_row_groups(*c, M);
}

int sba_sparse_decode_multi(const sba_cache* c, const void* q, int32_t M, const int32_t* sel_idx,
                            const int32_t* sel_cnt, int32_t n_max, float softmax_scale, int32_t num_splits,
                            float* o_part, float* lse_part, void* stream) {
    const int rc = check_multi(c, q, M, softmax_scale, num_splits, o_part, lse_part);
    if (rc != SBA_OK) return rc;
    if (!sel_idx || !sel_cnt || n_max < 1) return SBA_ERR_INVALID_ARG;
    return after_launch(launch_multi_query(*c, q, M, sel_idx, sel_cnt, n_max, softmax_scale, num_splits, o_part, lse_part,
                                           static_cast<cudaStream_t>(stream)));
}

int sba_rectify(const sba_cache* c, const void* q, const void* k_new, const void* v_new, int32_t f,
                float softmax_scale, int32_t num_splits, float* o_part, float* lse_part, void* stream) {
    const int rc = check_multi(c, q, f, softmax_scale, num_splits, o_part, lse_part);
    if (rc != SBA_OK) return rc;
    if (f > kMaxRectifyTokens) return SBA_ERR_UNSUPPORTED;
    if (!k_new || !v_new || !aligned16(k_new) || !aligned16(v_new)) return SBA_ERR_INVALID_ARG;
    return after_launch(launch_rectify_tc(*c, q, f, k_new, v_new, softmax_scale, num_splits, o_part, lse_part,
                                          static_cast<cudaStream_t>(stream)));
}

int sba_combine(const float* o_part, const float* lse_part, int32_t B, int32_t H_q, int32_t num_splits, int32_t d,
                void* out, int32_t out_dtype, float* lse_out, void* stream) {
    if (!o_part || !lse_part || !out || B < 1 || H_q < 1 || num_splits < 1) return SBA_ERR_INVALID_ARG;
    if (d != kHeadDim) return SBA_ERR_UNSUPPORTED;
    if (out_dtype != SBA_OUT_F32 && out_dtype != SBA_OUT_BF16) return SBA_ERR_INVALID_ARG;
    if (B > 65535) return SBA_ERR_UNSUPPORTED;
    return after_launch(launch_combine(o_part, lse_part, B, H_q, num_splits, out, out_dtype, lse_out,
                                       static_cast<cudaStream_t>(stream)));
}

int sba_fold_gate(const sba_gate* g, float* A, void* stream) {
    if (!g || !g->Wq || !g->Wk || !A || g->dg < 1 || g->dg > 256) return SBA_ERR_INVALID_ARG;
    return after_launch(launch_fold_gate(g->Wq, g->Wk, g->dg, A, static_cast<cudaStream_t>(stream)));
}

int32_t sba_decode_step_cluster(const sba_cache* c, const sba_select_params* p) {
    if (check_cache(c) != SBA_OK || check_params(p) != SBA_OK) return 0;
    int dev = 0, sms = 148;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    return step_cluster_size(*c, *p, sms);
}

int sba_decode_step(const sba_cache* c, const void* q, const void* k_new, const void* v_new, const int32_t* pos_start,
                    int32_t n_new, const float* gate_A, const sba_select_params* p, float softmax_scale, void* out,
                    int32_t out_dtype, float* lse_out, int32_t* sel_idx, int32_t* sel_cnt, float* gate_bias,
                    int32_t n_max, void* stream) {
    int rc = check_cache(c);
    if (rc != SBA_OK) return rc;
    rc = check_params(p);
    if (rc != SBA_OK) return rc;
    if (!q || !out || !aligned16(q) || n_new < 0) return SBA_ERR_INVALID_ARG;
    if (out_dtype != SBA_OUT_F32 && out_dtype != SBA_OUT_BF16) return SBA_ERR_INVALID_ARG;
    if (!good_scale(softmax_scale)) return SBA_ERR_INVALID_ARG;
    if (n_new > 0 && (!k_new || !v_new || !pos_start || !aligned16(k_new) || !aligned16(v_new)))
        return SBA_ERR_INVALID_ARG;
    if (p->scorer == SBA_SCORER_QUEST && !c->desc) return SBA_ERR_INVALID_ARG;
    if (p->scorer == SBA_SCORER_GATE && (!c->kg || !gate_A)) return SBA_ERR_INVALID_ARG;
    const int n_need = num_selected((c->max_len + c->b - 1) / c->b, *p);
    if ((sel_idx || gate_bias) && n_max < n_need) return SBA_ERR_INVALID_ARG;
    if (c->B > 65535 || c->H_kv > 65535) return SBA_ERR_UNSUPPORTED;
    const int C = sba_decode_step_cluster(c, p);
    if (C < 1) return SBA_ERR_UNSUPPORTED;
    return after_launch(launch_decode_step(*c, q, k_new, v_new, pos_start, n_new, gate_A, *p, softmax_scale, out,
                                           out_dtype, lse_out, sel_idx, sel_cnt,
                                           p->scorer == SBA_SCORER_GATE ? gate_bias : nullptr, n_max, C,
                                           static_cast<cudaStream_t>(stream)));
}

// ---------------------------------------------------------------------------
// Four-bit caches, attention weights, eviction
// ---------------------------------------------------------------------------

namespace {

bool aligned32(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }
// 32-bit words (NULL, an argument that is not there, passes).
bool aligned4(std::initializer_list<const void*> words) {
    for (const void* p : words)
        if (reinterpret_cast<uintptr_t>(p) & 3u) return false;
    return true;
}

// A four-bit cache seen as a bf16 one: the same checks, and the view that scoring (which reads the
// descriptors only) takes.
sba_cache view_of(const sba_cache4& c) {
    sba_cache v{};
    v.k = c.kv;
    v.v = c.kv;
    v.block_table = c.block_table;
    v.seq_lens = c.seq_lens;
    v.B = c.B;
    v.H_q = c.H_q;
    v.H_kv = c.H_kv;
    v.d = c.d;
    v.b = c.b;
    v.max_blocks = c.max_blocks;
    v.num_pages = c.num_pages;
    v.max_len = c.max_len;
    v.desc = c.desc;
    v.status = c.status;
    return v;
}

int check_cache4(const sba_cache4* c) {
    if (!c) return SBA_ERR_INVALID_ARG;
    const sba_cache v = view_of(*c);
    const int rc = check_cache(&v);
    if (rc != SBA_OK) return rc;
    if (c->B > 65535 || c->H_kv > 65535) return SBA_ERR_UNSUPPORTED;
    return aligned4({c->block_table, c->seq_lens, c->status}) ? SBA_OK : SBA_ERR_INVALID_ARG;
}

// Arguments of the calls that attend with M query tokens over a selection or (sel_idx NULL) all blocks.
int check_attend(int B, int H_q, int H_kv, const void* q, int32_t M, const int32_t* sel_idx, const int32_t* sel_cnt,
                 int32_t n_max, float softmax_scale) {
    if (!q || !aligned16(q) || M < 1 || M > kMaxQueryTokens || !good_scale(softmax_scale)) return SBA_ERR_INVALID_ARG;
    if (sel_idx ? (!sel_cnt || n_max < 1) : (sel_cnt != nullptr || n_max != 0)) return SBA_ERR_INVALID_ARG;
    if (!aligned4({sel_idx, sel_cnt})) return SBA_ERR_INVALID_ARG;
    const int64_t groups = (int64_t)H_kv * (((int64_t)M * (H_q / H_kv) + 7) / 8);
    if (groups > 65535 || groups * B >= (int64_t)1 << 31) return SBA_ERR_UNSUPPORTED;
    return SBA_OK;
}

size_t cells(int num_pages, int H_kv, int b) { return (size_t)num_pages * H_kv * b; }
bool overlap(const float* x, size_t nx, const float* y, size_t ny) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(x), b = reinterpret_cast<uintptr_t>(y);
    return x && y && a < b + ny * 4 && b < a + nx * 4;
}

// A token's sum is read and written by one thread: in place is fine, one array shifted over the other is not.
int check_weights(const float* lse, const float* acc_in, const float* acc_out, size_t n) {
    if (!lse || !acc_in || !acc_out || !aligned4({lse, acc_in, acc_out})) return SBA_ERR_INVALID_ARG;
    if (acc_in != acc_out && overlap(acc_in, n, acc_out, n)) return SBA_ERR_INVALID_ARG;
    return SBA_OK;
}

// Arguments of an eviction; src and dst seen as bf16 caches (checked each by itself before), page_bytes those of
// one of k's pages.
int check_evict(const sba_cache& src, int64_t page_bytes, const float* acc, const sba_evict_params* p,
                const sba_cache& dst, const float* acc_dst, const int32_t* new_lens, const int32_t* kept) {
    if (!acc || !aligned16(acc) || !p || !new_lens || !kept || !aligned4({acc_dst, new_lens, kept}))
        return SBA_ERR_INVALID_ARG;
    if (!aligned4({src.block_table, src.seq_lens, src.status, dst.block_table, dst.status})) return SBA_ERR_INVALID_ARG;
    if (p->n_keep < 1 || p->n_sink < 0 || p->n_recent < 0 || (int64_t)p->n_sink + p->n_recent > p->n_keep)
        return SBA_ERR_INVALID_ARG;
    if (dst.B != src.B || dst.H_kv != src.H_kv || dst.b != src.b) return SBA_ERR_INVALID_ARG;
    if ((int64_t)p->n_keep > (int64_t)dst.max_blocks * dst.b) return SBA_ERR_INVALID_ARG;
    // the lengths are read while the new ones are written
    const intptr_t apart = reinterpret_cast<intptr_t>(new_lens) - reinterpret_cast<intptr_t>(src.seq_lens);
    const intptr_t size = (intptr_t)src.B * 4;
    if (apart > -size && apart < size) return SBA_ERR_INVALID_ARG;
    // One pool: the caches' pages are apart only where a block table says so, for without one either begins at
    // page 0.
    const bool one_pool = dst.k == src.k && dst.v == src.v;
    if (!src.block_table && !dst.block_table && (dst.k == src.k || dst.v == src.v)) return SBA_ERR_INVALID_ARG;
    if (dst.desc && dst.desc == src.desc && !dst.block_table && !(one_pool && src.block_table)) return SBA_ERR_INVALID_ARG;
    // Its weights are one array too: dst's begin at the page at which dst's rows do.  Weights that overlap in any
    // other way are read where others are written.
    if (overlap(acc, cells(src.num_pages, src.H_kv, src.b), acc_dst, cells(dst.num_pages, dst.H_kv, dst.b))) {
        const intptr_t at = static_cast<const char*>(dst.k) - static_cast<const char*>(src.k);
        const intptr_t at_v = static_cast<const char*>(dst.v) - static_cast<const char*>(src.v);
        const intptr_t page = page_bytes, page_acc = (intptr_t)src.H_kv * src.b * 4;
        if (at != at_v || at % page != 0 || (intptr_t)(acc_dst - acc) * 4 != at / page * page_acc) return SBA_ERR_INVALID_ARG;
    }
    if (src.B > 65535 || src.H_kv > 65535) return SBA_ERR_UNSUPPORTED;
    return SBA_OK;
}

}  // namespace

int sba_append_kv4(const sba_cache4* c, const void* k_new, const void* v_new, const int32_t* pos_start, int32_t n_new,
                   void* stream) {
    const int rc = check_cache4(c);
    if (rc != SBA_OK) return rc;
    if (!k_new || !v_new || !pos_start || n_new < 0) return SBA_ERR_INVALID_ARG;
    if (!aligned32(k_new) || !aligned32(v_new) || !aligned4({pos_start})) return SBA_ERR_INVALID_ARG;
    if (n_new == 0) return SBA_OK;
    return after_launch(launch_append_kv4(*c, k_new, v_new, pos_start, n_new, static_cast<cudaStream_t>(stream)));
}

int sba_read_kv4(const sba_cache4* c, const int32_t* pos_start, int32_t n, void* k_out, void* v_out, void* stream) {
    const int rc = check_cache4(c);
    if (rc != SBA_OK) return rc;
    if (!k_out || !v_out || !pos_start || n < 0) return SBA_ERR_INVALID_ARG;
    if (!aligned32(k_out) || !aligned32(v_out) || !aligned4({pos_start})) return SBA_ERR_INVALID_ARG;
    if (n == 0) return SBA_OK;
    return after_launch(launch_read_kv4(*c, pos_start, n, k_out, v_out, static_cast<cudaStream_t>(stream)));
}

size_t sba_score_select_kv4_workspace_size(const sba_cache4* c, const sba_select_params* p) {
    if (check_cache4(c) != SBA_OK || check_params(p) != SBA_OK) return 0;
    return score_workspace_bytes(view_of(*c), *p);
}

int sba_score_select_kv4(const sba_cache4* c, const void* q, int32_t M, const sba_select_params* p, int32_t* sel_idx,
                         int32_t* sel_cnt, int32_t n_max, void* ws, size_t ws_bytes, void* stream) {
    const int rc = check_cache4(c);
    if (rc != SBA_OK) return rc;
    const sba_cache v = view_of(*c);
    if (p && p->scorer == SBA_SCORER_GATE) return SBA_ERR_UNSUPPORTED;
    return sba_score_select_multi(&v, q, M, p, sel_idx, sel_cnt, n_max, ws, ws_bytes, stream);
}

size_t sba_decode_kv4_workspace_size(const sba_cache4* c, int32_t M, int32_t n_max) {
    if (check_cache4(c) != SBA_OK || M < 1 || M > kMaxQueryTokens || n_max < 0) return 0;
    return decode_kv4_workspace_bytes(*c, M, n_max);
}

int sba_decode_kv4(const sba_cache4* c, const void* q, int32_t M, const int32_t* sel_idx, const int32_t* sel_cnt,
                   int32_t n_max, float softmax_scale, void* out, int32_t out_dtype, float* lse_out, void* ws,
                   size_t ws_bytes, void* stream) {
    int rc = check_cache4(c);
    if (rc != SBA_OK) return rc;
    rc = check_attend(c->B, c->H_q, c->H_kv, q, M, sel_idx, sel_cnt, n_max, softmax_scale);
    if (rc != SBA_OK) return rc;
    if (!out || !aligned16(out) || (out_dtype != SBA_OUT_F32 && out_dtype != SBA_OUT_BF16)) return SBA_ERR_INVALID_ARG;
    if (!aligned4({lse_out})) return SBA_ERR_INVALID_ARG;
    if (!ws || !aligned16(ws) || ws_bytes < decode_kv4_workspace_bytes(*c, M, n_max)) return SBA_ERR_WORKSPACE;
    return after_launch(launch_decode_kv4(*c, q, M, sel_idx, sel_cnt, n_max, softmax_scale, out, out_dtype, lse_out, ws,
                                          static_cast<cudaStream_t>(stream)));
}

int sba_accumulate_weights(const sba_cache* c, const void* q, int32_t M, const int32_t* sel_idx,
                           const int32_t* sel_cnt, const float* gate_bias, int32_t n_max, float softmax_scale,
                           const float* lse, const float* acc_in, float* acc_out, void* stream) {
    int rc = check_cache(c);
    if (rc != SBA_OK) return rc;
    rc = check_attend(c->B, c->H_q, c->H_kv, q, M, sel_idx, sel_cnt, n_max, softmax_scale);
    if (rc != SBA_OK) return rc;
    if (gate_bias && (!sel_idx || M != 1 || !aligned4({gate_bias}))) return SBA_ERR_INVALID_ARG;
    if (!aligned4({c->block_table, c->seq_lens, c->status})) return SBA_ERR_INVALID_ARG;
    rc = check_weights(lse, acc_in, acc_out, cells(c->num_pages, c->H_kv, c->b));
    if (rc != SBA_OK) return rc;
    if (c->B > 65535 || c->H_kv > 65535) return SBA_ERR_UNSUPPORTED;
    return after_launch(launch_accumulate_weights(*c, q, M, sel_idx, sel_cnt, gate_bias, n_max, softmax_scale, lse,
                                                  acc_in, acc_out, static_cast<cudaStream_t>(stream)));
}

int sba_accumulate_weights_kv4(const sba_cache4* c, const void* q, int32_t M, const int32_t* sel_idx,
                               const int32_t* sel_cnt, int32_t n_max, float softmax_scale, const float* lse,
                               const float* acc_in, float* acc_out, void* stream) {
    int rc = check_cache4(c);
    if (rc != SBA_OK) return rc;
    rc = check_attend(c->B, c->H_q, c->H_kv, q, M, sel_idx, sel_cnt, n_max, softmax_scale);
    if (rc != SBA_OK) return rc;
    rc = check_weights(lse, acc_in, acc_out, cells(c->num_pages, c->H_kv, c->b));
    if (rc != SBA_OK) return rc;
    return after_launch(launch_accumulate_weights_kv4(*c, q, M, sel_idx, sel_cnt, n_max, softmax_scale, lse, acc_in,
                                                      acc_out, static_cast<cudaStream_t>(stream)));
}

int sba_evict(const sba_cache* src, const float* acc, const sba_evict_params* p, const sba_cache* dst, float* acc_dst,
              int32_t* new_lens, int32_t* kept, void* stream) {
    int rc = check_cache(src);
    if (rc == SBA_OK) rc = check_cache(dst);
    if (rc == SBA_OK)
        rc = check_evict(*src, (int64_t)src->H_kv * src->b * kHeadDim * 2, acc, p, *dst, acc_dst, new_lens, kept);
    if (rc != SBA_OK) return rc;
    return after_launch(launch_evict(*src, acc, *p, *dst, acc_dst, new_lens, kept, static_cast<cudaStream_t>(stream)));
}

int sba_evict_kv4(const sba_cache4* src, const float* acc, const sba_evict_params* p, const sba_cache4* dst,
                  float* acc_dst, int32_t* new_lens, int32_t* kept, void* stream) {
    int rc = check_cache4(src);
    if (rc == SBA_OK) rc = check_cache4(dst);
    if (rc == SBA_OK)
        rc = check_evict(view_of(*src), (int64_t)src->H_kv * (src->b / kStripTokens) * kStripBytes, acc, p, view_of(*dst),
                         acc_dst, new_lens, kept);
    if (rc != SBA_OK) return rc;
    return after_launch(
        launch_evict_kv4(*src, acc, *p, *dst, acc_dst, new_lens, kept, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
