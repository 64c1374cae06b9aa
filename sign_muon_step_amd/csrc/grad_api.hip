// grad_api.hip -- host side of the gradient operators declared in
// include/signmuon.h: argument checks, workspace layout and launches.
#include <cmath>

#include "signmuon.h"
#include "grad_internal.h"

namespace {

constexpr int64_t kMaxDim = (int64_t)1 << 20;      // vocab and cols, as a matrix's rows and cols
constexpr int64_t kMaxN = ((int64_t)1 << 31) - 1;  // entries of one weight, as in the step
constexpr int32_t kMaxWorkers = 255;
constexpr int64_t kMaxTokens = (int64_t)1 << 25;   // over all workers: a launch's threads stay below 2^32
constexpr size_t kSectionAlign = 256;

inline size_t align_up(size_t x) { return (x + kSectionAlign - 1) / kSectionAlign * kSectionAlign; }
inline bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }
inline bool dtype_ok(int d) { return d == SIGNMUON_F32 || d == SIGNMUON_BF16; }

template <typename... P>
bool all_aligned(const P *...p) { return (aligned16(p) && ...); }

int check_workspace(const void *ws, size_t have, size_t need) {
    if (need == 0) return SIGNMUON_OK;
    if (!ws || have < need) return SIGNMUON_EWORKSPACE;
    return aligned16(ws) ? SIGNMUON_OK : SIGNMUON_EALIGN;
}

// ---------------------------------------------------------------------------
// Embedding
// ---------------------------------------------------------------------------
int check_embedding(int64_t workers, int64_t tokens, int64_t vocab, int64_t cols) {
    if (workers < 1 || tokens < 1 || vocab < 1 || cols < 1) return SIGNMUON_EINVAL;
    if (workers > kMaxWorkers || tokens > kMaxTokens / workers) return SIGNMUON_ERANGE;
    if (vocab > kMaxDim || cols > kMaxDim || vocab * cols > kMaxN) return SIGNMUON_ERANGE;
    return SIGNMUON_OK;
}

struct EmbedPlan {
    int32_t seg, segments;
    size_t keys[2], partial, total;
};

EmbedPlan embedding_plan(int64_t workers, int64_t tokens, int64_t cols) {
    EmbedPlan p;
    p.seg = sm::embed_segment((int32_t)workers, tokens, cols);
    p.segments = (int32_t)((tokens + p.seg - 1) / p.seg);
    const size_t keys = align_up((size_t)(workers * tokens) * sizeof(uint64_t));
    p.keys[0] = 0;
    p.keys[1] = keys;
    p.partial = sm::embed_merge_passes(tokens) > 0 ? 2 * keys : keys;
    // one segment shares no row with another
    p.total = p.partial + (p.segments > 1 ? (size_t)(workers * p.segments * 2 * cols) * sizeof(float) : 0);
    return p;
}

// ---------------------------------------------------------------------------
// Layer norm
// ---------------------------------------------------------------------------
int check_norm(int64_t workers, int64_t rows, int64_t cols) {
    if (workers < 1 || rows < 1 || cols < 1) return SIGNMUON_EINVAL;
    if (workers > kMaxWorkers || rows > kMaxTokens / workers || cols > kMaxDim) return SIGNMUON_ERANGE;
    return SIGNMUON_OK;
}

size_t norm_workspace(int32_t workers, int64_t rows, int64_t cols) {
    const int32_t parts = sm::norm_parts(workers, rows, cols);
    return parts > 1 ? (size_t)((int64_t)workers * parts * 2 * cols) * sizeof(float) : 0;
}

}  // namespace

extern "C" {

int signmuon_embedding(const void *ids, signmuon_itype id_type, const void *table,
                       signmuon_dtype table_dtype, int64_t tokens, int64_t vocab, int64_t cols,
                       float scale, void *y, signmuon_dtype y_dtype, signmuon_stream stream) {
    if (!ids || !table || !y) return SIGNMUON_EINVAL;
    if (int rc = check_embedding(1, tokens, vocab, cols)) return rc;
    if (!std::isfinite(scale)) return SIGNMUON_EINVAL;
    if ((id_type != SIGNMUON_I32 && id_type != SIGNMUON_I64) || !dtype_ok(table_dtype) || !dtype_ok(y_dtype))
        return SIGNMUON_EDTYPE;
    if (!all_aligned(ids, table, y)) return SIGNMUON_EALIGN;
    sm::Embed e{};
    e.ids = ids;
    e.table = table;
    e.y = y;
    e.tokens = tokens;
    e.vocab = vocab;
    e.cols = cols;
    e.scale = scale;
    e.id64 = id_type == SIGNMUON_I64;
    e.table_bf16 = table_dtype == SIGNMUON_BF16;
    e.y_bf16 = y_dtype == SIGNMUON_BF16;
    sm::launch_embedding(e, static_cast<hipStream_t>(stream));
    return sm::launch_status();
}

size_t signmuon_embedding_workspace_bytes(int32_t workers, int64_t tokens, int64_t vocab, int64_t cols) {
    if (check_embedding(workers, tokens, vocab, cols) != SIGNMUON_OK) return 0;
    return embedding_plan(workers, tokens, cols).total;
}

int signmuon_embedding_backward(const void *ids, signmuon_itype id_type, const void *dy,
                                signmuon_dtype dy_dtype, int32_t workers, int64_t tokens,
                                int64_t vocab, int64_t cols, float scale, void *grad,
                                signmuon_dtype grad_dtype, int32_t accumulate, void *workspace,
                                size_t workspace_bytes, signmuon_stream stream) {
    if (!ids || !dy || !grad) return SIGNMUON_EINVAL;
    if (int rc = check_embedding(workers, tokens, vocab, cols)) return rc;
    if (!std::isfinite(scale) || (accumulate != 0 && accumulate != 1)) return SIGNMUON_EINVAL;
    if ((id_type != SIGNMUON_I32 && id_type != SIGNMUON_I64) || !dtype_ok(dy_dtype) || !dtype_ok(grad_dtype))
        return SIGNMUON_EDTYPE;
    if (!all_aligned(ids, dy, grad)) return SIGNMUON_EALIGN;
    const EmbedPlan p = embedding_plan(workers, tokens, cols);
    if (int rc = check_workspace(workspace, workspace_bytes, p.total)) return rc;
    char *ws = static_cast<char *>(workspace);
    const hipStream_t st = static_cast<hipStream_t>(stream);
    sm::EmbedGrad e{};
    e.ids = ids;
    e.dy = dy;
    e.grad = grad;
    e.keys[0] = reinterpret_cast<uint64_t *>(ws + p.keys[0]);
    e.keys[1] = reinterpret_cast<uint64_t *>(ws + p.keys[1]);
    e.partial = reinterpret_cast<float *>(ws + p.partial);
    e.tokens = tokens;
    e.vocab = vocab;
    e.cols = cols;
    e.workers = workers;
    e.seg = p.seg;
    e.segments = p.segments;
    e.scale = scale;
    e.id64 = id_type == SIGNMUON_I64;
    e.dy_bf16 = dy_dtype == SIGNMUON_BF16;
    e.grad_bf16 = grad_dtype == SIGNMUON_BF16;
    e.accumulate = accumulate != 0;
    sm::launch_embedding_sort(e, st);
    if (int rc = sm::launch_status()) return rc;
    for (int pass = 0; pass < sm::embed_merge_passes(tokens); ++pass) {
        sm::launch_embedding_merge(e, pass, st);
        if (int rc = sm::launch_status()) return rc;
    }
    sm::launch_embedding_sums(e, st);
    if (int rc = sm::launch_status()) return rc;
    if (e.segments == 1) return SIGNMUON_OK;
    sm::launch_embedding_join(e, st);
    return sm::launch_status();
}

int signmuon_layer_norm(const void *x, signmuon_dtype x_dtype, int64_t rows, int64_t cols,
                        const float *gamma, const float *beta, float eps, void *y, float *mean,
                        float *rstd, signmuon_stream stream) {
    if (!x || !gamma || !y) return SIGNMUON_EINVAL;
    if (int rc = check_norm(1, rows, cols)) return rc;
    if (!std::isfinite(eps) || eps <= 0.0f) return SIGNMUON_EINVAL;
    if (!dtype_ok(x_dtype)) return SIGNMUON_EDTYPE;
    if (!all_aligned(x, gamma, beta, y, mean, rstd)) return SIGNMUON_EALIGN;
    sm::Norm n{};
    n.x = x;
    n.gamma = gamma;
    n.beta = beta;
    n.y = y;
    n.mean = mean;
    n.rstd = rstd;
    n.rows = rows;
    n.cols = cols;
    n.eps = eps;
    n.bf16 = x_dtype == SIGNMUON_BF16;
    sm::launch_layer_norm(n, static_cast<hipStream_t>(stream));
    return sm::launch_status();
}

size_t signmuon_layer_norm_workspace_bytes(int32_t workers, int64_t rows, int64_t cols) {
    if (check_norm(workers, rows, cols) != SIGNMUON_OK) return 0;
    return norm_workspace(workers, rows, cols);
}

int signmuon_layer_norm_backward(const void *dy, const void *x, signmuon_dtype x_dtype,
                                 int32_t workers, int64_t rows, int64_t cols, const float *gamma,
                                 const float *mean, const float *rstd, void *dx, void *dgamma,
                                 void *dbeta, signmuon_dtype grad_dtype, void *workspace,
                                 size_t workspace_bytes, signmuon_stream stream) {
    if (!dy || !x || !gamma || !mean || !rstd || (!dx && !dgamma && !dbeta)) return SIGNMUON_EINVAL;
    if (int rc = check_norm(workers, rows, cols)) return rc;
    if (!dtype_ok(x_dtype) || !dtype_ok(grad_dtype)) return SIGNMUON_EDTYPE;
    if (!all_aligned(dy, x, gamma, mean, rstd, dx, dgamma, dbeta)) return SIGNMUON_EALIGN;
    if (int rc = check_workspace(workspace, workspace_bytes, norm_workspace(workers, rows, cols))) return rc;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    sm::NormGrad n{};
    n.dy = dy;
    n.x = x;
    n.gamma = gamma;
    n.mean = mean;
    n.rstd = rstd;
    n.dx = dx;
    n.dgamma = dgamma;
    n.dbeta = dbeta;
    n.partial = static_cast<float *>(workspace);
    n.rows = rows;
    n.cols = cols;
    n.workers = workers;
    n.parts = sm::norm_parts(workers, rows, cols);
    n.bf16 = x_dtype == SIGNMUON_BF16;
    n.grad_bf16 = grad_dtype == SIGNMUON_BF16;
    sm::launch_layer_norm_backward(n, st);
    if (int rc = sm::launch_status()) return rc;
    if (n.parts == 1 || (!dgamma && !dbeta)) return SIGNMUON_OK;
    sm::launch_layer_norm_sums(n, st);
    return sm::launch_status();
}

}  // extern "C"
