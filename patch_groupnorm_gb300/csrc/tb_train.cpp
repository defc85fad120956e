// tb_train.cpp -- C ABI of the training calls: layer norm forward and
// backward, the gradient norm and clip, PatchGroupNorm's backward pass.
// Argument validation and launch configuration only.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "tb_internal.h"
#include "tileblend.h"

#define TB_API extern "C" __attribute__((visibility("default")))

namespace {

tb_status launched(cudaError_t e) {
    if (e == cudaSuccess) return TB_OK;
    tb::record_cuda_error(e);
    return TB_ERR_CUDA;
}

bool known(tb_dtype d) { return d == TB_F32 || d == TB_F16 || d == TB_BF16; }
int elem_bytes(tb_dtype d) { return d == TB_F32 ? 4 : 2; }
bool aligned(const void* p, int bytes) { return ((uintptr_t)p & (uintptr_t)(bytes - 1)) == 0; }

// ---------------------------------------------------------------------------
// layer norm
// ---------------------------------------------------------------------------

tb_status ln_shape(tb_dtype dtype, tb_dtype wdtype, int64_t rows, int64_t cols) {
    if (!known(dtype) || !known(wdtype)) return TB_ERR_DTYPE;
    if (wdtype != dtype && wdtype != TB_F32) return TB_ERR_DTYPE;
    if (rows < 0 || cols < 1) return TB_ERR_SHAPE;
    if (cols > (int64_t)1 << 30) return TB_ERR_UNSUPPORTED;
    return TB_OK;
}

// One row tensor: its stride and alignment.  Clears *vector when its rows
// cannot be read in 16-byte chunks.
tb_status ln_rows(const void* p, int64_t ld, tb_dtype dtype, int64_t rows, int64_t cols, bool* vector) {
    if (p == nullptr) return TB_ERR_NULL;
    if (rows > 1 && ld < cols) return TB_ERR_SHAPE;
    if (rows > 1 && (double)rows * (double)ld > 2.0e18) return TB_ERR_SHAPE;
    if (!aligned(p, elem_bytes(dtype))) return TB_ERR_UNSUPPORTED;
    if (!aligned(p, 16) || (rows > 1 && ld % (16 / elem_bytes(dtype)) != 0)) *vector = false;
    return TB_OK;
}

tb_status ln_weight(const void* p, tb_dtype wdtype, bool* vector) {
    if (p == nullptr) return TB_OK;
    if (!aligned(p, elem_bytes(wdtype))) return TB_ERR_UNSUPPORTED;
    if (!aligned(p, 16)) *vector = false;
    return TB_OK;
}

#define TB_TRY(call)                          \
    do {                                      \
        const tb_status try_status = (call);  \
        if (try_status != TB_OK) return try_status; \
    } while (0)

// ---------------------------------------------------------------------------
// gradients
// ---------------------------------------------------------------------------

tb_status grad_validate(const void* const* grads, const int64_t* numel, const tb_dtype* dtypes, int32_t T) {
    if (T < 0) return TB_ERR_SHAPE;
    if (T == 0) return TB_OK;
    if (T > TB_MAX_GRADS) return TB_ERR_UNSUPPORTED;
    if (grads == nullptr || numel == nullptr || dtypes == nullptr) return TB_ERR_NULL;
    for (int t = 0; t < T; ++t) {
        if (!known(dtypes[t])) return TB_ERR_DTYPE;
        if (numel[t] < 0) return TB_ERR_SHAPE;
        if (numel[t] > 0 && grads[t] == nullptr) return TB_ERR_NULL;
        if (numel[t] > 0 && !aligned(grads[t], elem_bytes(dtypes[t]))) return TB_ERR_UNSUPPORTED;
        // pieces of one launch are counted in 31 bits
        if (numel[t] > (int64_t)1 << 42) return TB_ERR_UNSUPPORTED;
    }
    return TB_OK;
}

// Tensors [t0, t0 + count) as the parameters of one launch.
template <typename P>
tb_status grad_table(P& prm, const void* const* grads, void* const* outs, const int64_t* numel, const tb_dtype* dtypes,
                     int32_t t0, int32_t count) {
    int64_t pieces = 0;
    for (int k = 0; k < count; ++k) {
        const int t = t0 + k, es = elem_bytes(dtypes[t]);
        const int64_t to_boundary = (int64_t)((16 - ((uintptr_t)grads[t] & 15u)) & 15u) / es;
        const int64_t head = std::min<int64_t>(numel[t], to_boundary);
        const int64_t chunk_bytes = (numel[t] - head) / (16 / es) * 16;
        prm.in[k] = grads[t];
        prm.out[k] = outs ? outs[t] : nullptr;
        prm.numel[k] = numel[t];
        prm.dtype[k] = (uint8_t)dtypes[t];
        prm.head[k] = (uint8_t)head;
        prm.start[k] = (int32_t)pieces;
        if (numel[t] > 0)
            pieces += std::max<int64_t>(1, (chunk_bytes + tb::GRAD_PIECE_BYTES - 1) / tb::GRAD_PIECE_BYTES);
        if (pieces > 2147483647LL) return TB_ERR_UNSUPPORTED;
    }
    prm.start[count] = (int32_t)pieces;
    prm.T = count;
    prm.status = tb::checked_build_status();
    return TB_OK;
}

// Calls go(params, index of the launch) for every launch's table.
template <typename F>
tb_status each_table(const void* const* grads, void* const* outs, const int64_t* numel, const tb_dtype* dtypes,
                     int32_t T, F&& go) {
    if (T <= tb::GRAD_SMALL_MAXT) {
        tb::GradParamsSmall prm;
        TB_TRY(grad_table(prm, grads, outs, numel, dtypes, 0, T));
        return go(prm, 0);
    }
    tb::GradParamsLarge prm;
    for (int t0 = 0, k = 0; t0 < T; t0 += tb::GRAD_MAXT, ++k) {
        TB_TRY(grad_table(prm, grads, outs, numel, dtypes, t0, std::min(T - t0, tb::GRAD_MAXT)));
        TB_TRY(go(prm, k));
    }
    return TB_OK;
}

// ---------------------------------------------------------------------------
// PatchGroupNorm backward
// ---------------------------------------------------------------------------

// Validates a call and fills everything but the work.  `outs` NULL: a
// statistics call.  *ring: every tensor of a patch has the same offset from
// 16-byte boundaries.
tb_status gn_grad_params(tb::GnGradParams& prm, bool* ring, const void* const* patches, const void* const* grads,
                         void* const* outs, int32_t P, tb_dtype dtype, int64_t N, int64_t C, const int64_t* spatial,
                         int32_t G, const tb_gn_partial* partials, int32_t R, const void* gamma, const void* beta,
                         float eps, int32_t silu, const void* grad_partials, void* dgamma, void* dbeta) {
    if (!known(dtype)) return TB_ERR_DTYPE;
    if (P < 1 || N < 0 || C < 0 || G < 1 || R < 1) return TB_ERR_SHAPE;
    if (C % G != 0) return TB_ERR_SHAPE;
    if (!(eps >= 0.0f) || std::isinf(eps)) return TB_ERR_SHAPE;
    if (P > tb::GN_MAXP || R > 65536) return TB_ERR_UNSUPPORTED;
    if (spatial == nullptr || patches == nullptr || grads == nullptr) return TB_ERR_NULL;
    if ((double)std::max(P, R) * (double)N * (double)C * TB_GN_PARTS > 2.0e9) return TB_ERR_UNSUPPORTED;
    std::memset(&prm, 0, sizeof(prm));
    const int es = elem_bytes(dtype);
    *ring = true;
    for (int p = 0; p < P; ++p) {
        if (spatial[p] < 0) return TB_ERR_SHAPE;
        prm.patches[p] = patches[p];
        prm.grads[p] = grads[p];
        prm.outs[p] = outs ? outs[p] : nullptr;
        prm.spatial[p] = spatial[p];
        if (N == 0 || C == 0 || spatial[p] == 0) continue;
        if (patches[p] == nullptr || grads[p] == nullptr || (outs && outs[p] == nullptr)) return TB_ERR_NULL;
        if ((double)N * (double)C * (double)spatial[p] > 2.0e18) return TB_ERR_SHAPE;
        if (!aligned(patches[p], es) || !aligned(grads[p], es) || !aligned(prm.outs[p], es)) return TB_ERR_UNSUPPORTED;
        const uintptr_t off = (uintptr_t)patches[p] & 15u;
        if (((uintptr_t)grads[p] & 15u) != off || (outs && ((uintptr_t)outs[p] & 15u) != off)) *ring = false;
    }
    if (N > 0 && C > 0 && (partials == nullptr || grad_partials == nullptr)) return TB_ERR_NULL;
    if (!aligned(gamma, es) || !aligned(beta, es) || !aligned(dgamma, es) || !aligned(dbeta, es))
        return TB_ERR_UNSUPPORTED;
    if (!aligned(partials, 16) || !aligned(grad_partials, 16)) return TB_ERR_UNSUPPORTED;
    prm.partials = reinterpret_cast<const tb::GnPartial*>(partials);
    prm.grad_partials = reinterpret_cast<float2*>(const_cast<void*>(grad_partials));
    prm.gamma = gamma;
    prm.beta = beta;
    prm.dgamma = dgamma;
    prm.dbeta = dbeta;
    prm.N = N;
    prm.C = C;
    prm.P = P;
    prm.G = G;
    prm.R = R;
    prm.eps = eps;
    prm.silu = silu ? 1 : 0;
    prm.wtasks = dgamma != nullptr || dbeta != nullptr ? (int32_t)((C + tb::GRAD_CHANNELS - 1) / tb::GRAD_CHANNELS) : 0;
    prm.status = tb::device_status_word();
    return TB_OK;
}

// Cuts the work of `mode` into tasks: whole rows, as many as one ring stage
// holds, or parts of a row of a stage each; smaller ones where that gives less
// than two tasks per SM.
tb_status gn_grad_tasks(tb::GnGradParams& prm, int mode, tb_dtype dtype, int sms) {
    const int es = elem_bytes(dtype), vec = 16 / es;
    const int64_t K = prm.C / prm.G, units = prm.N * prm.G;
    prm.mode = mode;
    for (int p = 0; p < prm.P; ++p) {
        const int64_t row = prm.spatial[p] * es;
        prm.rows[p] = prm.parts[p] = 0;
        if (row == 0 && mode != tb::GRAD_STATS) continue;  // no elements; a statistics call still writes its records
        const int64_t fit = row > 0 ? tb::GRAD_STAGE_BYTES / row : tb::GRAD_MAX_ROWS;
        prm.rows[p] = (int32_t)std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(fit, tb::GRAD_MAX_ROWS), K));
        const int64_t want = (row + tb::GRAD_STAGE_BYTES - 1) / tb::GRAD_STAGE_BYTES;
        prm.parts[p] = (int32_t)std::max<int64_t>(1, std::min<int64_t>(want, (int64_t)TB_GN_PARTS));
    }
    auto tasks_of = [&](int p) {
        if (prm.rows[p] == 0) return (int64_t)0;
        return prm.parts[p] > 1 ? K * prm.parts[p] : (K + prm.rows[p] - 1) / prm.rows[p];
    };
    for (bool smaller = true; smaller;) {
        int64_t total = 0;
        for (int p = 0; p < prm.P; ++p) total += units * tasks_of(p);
        if (total >= 2 * (int64_t)sms) break;
        smaller = false;
        for (int p = 0; p < prm.P; ++p) {
            if (prm.rows[p] > 1) {
                prm.rows[p] = (prm.rows[p] + 1) / 2;
                smaller = true;
            } else if (prm.rows[p] == 1 && prm.parts[p] < TB_GN_PARTS &&
                       prm.spatial[p] / vec / (prm.parts[p] + 1) >= 256) {
                ++prm.parts[p];
                smaller = true;
            }
        }
    }
    int64_t at = 0;
    for (int p = 0; p < prm.P; ++p) {
        // whole words, evenly; the last part takes what is left
        if (prm.parts[p] > 1) prm.part_elems[p] = prm.spatial[p] / vec / prm.parts[p] * vec;
        prm.task_start[p] = (int32_t)at;
        at += tasks_of(p);
        if (at > 1000000000LL) return TB_ERR_UNSUPPORTED;
    }
    prm.task_start[prm.P] = (int32_t)at;
    prm.unit_tasks = (int32_t)at;
    if ((double)units * (double)at > 2.0e9) return TB_ERR_UNSUPPORTED;
    return TB_OK;
}

}  // namespace

TB_API tb_status tb_layer_norm(const void* x, int64_t x_ld, const void* residual, int64_t residual_ld, tb_dtype dtype,
                               int64_t rows, int64_t cols, const void* gamma, const void* beta, tb_dtype wdtype,
                               float eps, void* total, int64_t total_ld, void* y, int64_t y_ld, float* mean,
                               float* rstd, void* stream) {
    TB_TRY(ln_shape(dtype, wdtype, rows, cols));
    if (!(eps >= 0.0f) || std::isinf(eps)) return TB_ERR_SHAPE;
    if (rows == 0) return TB_OK;
    bool vector = cols % (16 / elem_bytes(dtype)) == 0;
    TB_TRY(ln_rows(x, x_ld, dtype, rows, cols, &vector));
    TB_TRY(ln_rows(y, y_ld, dtype, rows, cols, &vector));
    if (residual != nullptr) {
        TB_TRY(ln_rows(residual, residual_ld, dtype, rows, cols, &vector));
        TB_TRY(ln_rows(total, total_ld, dtype, rows, cols, &vector));
    }
    TB_TRY(ln_weight(gamma, wdtype, &vector));
    TB_TRY(ln_weight(beta, wdtype, &vector));
    if (!aligned(mean, 4) || !aligned(rstd, 4)) return TB_ERR_UNSUPPORTED;
    int sms = 0;
    TB_TRY(tb::sm_count(&sms));
    tb::LnFwdParams p;
    p.x = x;
    p.residual = residual;
    p.gamma = gamma;
    p.beta = beta;
    p.total = total;
    p.y = y;
    p.mean = mean;
    p.rstd = rstd;
    p.rows = rows;
    p.cols = cols;
    p.x_ld = x_ld;
    p.r_ld = residual_ld;
    p.t_ld = total_ld;
    p.y_ld = y_ld;
    p.status = tb::checked_build_status();
    p.wdtype = (int32_t)wdtype;
    p.eps = eps;
    return launched(tb::launch_ln_fwd(p, (int)dtype, vector, sms, reinterpret_cast<cudaStream_t>(stream)));
}

TB_API int64_t tb_layer_norm_workspace(int64_t rows, int64_t cols) {
    if (rows < 0 || cols < 1 || cols > (int64_t)1 << 30) return -1;
    return std::min<int64_t>(rows, TB_LN_PARTS) * cols * 8;
}

TB_API tb_status tb_layer_norm_backward(const void* dy, int64_t dy_ld, const void* x, int64_t x_ld, tb_dtype dtype,
                                        int64_t rows, int64_t cols, const float* mean, const float* rstd,
                                        const void* gamma, tb_dtype wdtype, const void* dtotal, int64_t dtotal_ld,
                                        void* dx, int64_t dx_ld, void* dgamma, void* dbeta, void* workspace,
                                        int64_t workspace_bytes, void* stream) {
    TB_TRY(ln_shape(dtype, wdtype, rows, cols));
    bool vector = cols % (16 / elem_bytes(dtype)) == 0;
    const bool weights = dgamma != nullptr || dbeta != nullptr;
    TB_TRY(ln_weight(gamma, wdtype, &vector));
    if (!aligned(dgamma, elem_bytes(wdtype)) || !aligned(dbeta, elem_bytes(wdtype))) return TB_ERR_UNSUPPORTED;
    if (rows > 0) {
        TB_TRY(ln_rows(dy, dy_ld, dtype, rows, cols, &vector));
        TB_TRY(ln_rows(x, x_ld, dtype, rows, cols, &vector));
        if (mean == nullptr || rstd == nullptr) return TB_ERR_NULL;
        if (!aligned(mean, 4) || !aligned(rstd, 4)) return TB_ERR_UNSUPPORTED;
        if (dx != nullptr) TB_TRY(ln_rows(dx, dx_ld, dtype, rows, cols, &vector));
        if (dtotal != nullptr) TB_TRY(ln_rows(dtotal, dtotal_ld, dtype, rows, cols, &vector));
        if (weights) {
            if (workspace == nullptr) return TB_ERR_NULL;
            if (!aligned(workspace, 16)) return TB_ERR_UNSUPPORTED;
            if (workspace_bytes < tb_layer_norm_workspace(rows, cols)) return TB_ERR_SHAPE;
        }
    }
    int parts = 0;
    if (rows > 0 && (weights || dx != nullptr)) {
        int sms = 0;
        TB_TRY(tb::sm_count(&sms));
        tb::LnBwdParams p;
        p.dy = dy;
        p.x = x;
        p.mean = mean;
        p.rstd = rstd;
        p.gamma = gamma;
        p.dtotal = dtotal;
        p.dx = dx;
        p.workspace = weights ? reinterpret_cast<float*>(workspace) : nullptr;
        p.rows = rows;
        p.cols = cols;
        p.dy_ld = dy_ld;
        p.x_ld = x_ld;
        p.dt_ld = dtotal_ld;
        p.dx_ld = dx_ld;
        p.status = tb::device_status_word();
        p.wdtype = (int32_t)wdtype;
        TB_TRY(launched(tb::launch_ln_bwd(p, (int)dtype, vector, sms, &parts, reinterpret_cast<cudaStream_t>(stream))));
    }
    if (!weights) return TB_OK;
    tb::LnWgradParams w;
    w.workspace = reinterpret_cast<const float*>(workspace);
    w.dgamma = dgamma;
    w.dbeta = dbeta;
    w.cols = cols;
    w.parts = parts;
    w.wdtype = (int32_t)wdtype;
    return launched(tb::launch_ln_wgrad(w, reinterpret_cast<cudaStream_t>(stream)));
}

TB_API int64_t tb_grad_records(int32_t T) {
    if (T < 0 || T > TB_MAX_GRADS) return -1;
    return (int64_t)TB_GRAD_PARTS * std::max(1, (T + TB_GRAD_TABLE - 1) / TB_GRAD_TABLE);
}

TB_API tb_status tb_grad_stats(const void* const* grads, const int64_t* numel, const tb_dtype* dtypes, int32_t T,
                               double* records, void* stream) {
    TB_TRY(grad_validate(grads, numel, dtypes, T));
    if (records == nullptr) return TB_ERR_NULL;
    if (!aligned(records, 8)) return TB_ERR_UNSUPPORTED;
    int sms = 0;
    TB_TRY(tb::sm_count(&sms));
    return each_table(grads, nullptr, numel, dtypes, T, [&](auto& prm, int k) {
        prm.records = records + (int64_t)k * TB_GRAD_PARTS;
        prm.n_records = 0;
        prm.norm = nullptr;
        prm.max_norm = 0.f;
        prm.first = 0;
        return launched(tb::launch_grad_stats(prm, sms, reinterpret_cast<cudaStream_t>(stream)));
    });
}

TB_API tb_status tb_grad_norm(const double* records, int64_t n_records, float* norm, void* stream) {
    if (n_records < 0) return TB_ERR_SHAPE;
    if (norm == nullptr || (records == nullptr && n_records > 0)) return TB_ERR_NULL;
    if (!aligned(records, 8) || !aligned(norm, 4)) return TB_ERR_UNSUPPORTED;
    return launched(tb::launch_grad_norm(records, n_records, norm, reinterpret_cast<cudaStream_t>(stream)));
}

TB_API tb_status tb_grad_clip(const void* const* grads, void* const* outs, const int64_t* numel,
                              const tb_dtype* dtypes, int32_t T, const double* records, int64_t n_records,
                              float max_norm, float* norm, void* stream) {
    TB_TRY(grad_validate(grads, numel, dtypes, T));
    if (!(max_norm >= 0.0f) || n_records < 0) return TB_ERR_SHAPE;
    if (records == nullptr && n_records > 0) return TB_ERR_NULL;
    if (!aligned(records, 8) || !aligned(norm, 4)) return TB_ERR_UNSUPPORTED;
    if (T > 0 && outs == nullptr) return TB_ERR_NULL;
    for (int t = 0; t < T; ++t) {
        if (numel[t] > 0 && outs[t] == nullptr) return TB_ERR_NULL;
        if (numel[t] > 0 && !aligned(outs[t], elem_bytes(dtypes[t]))) return TB_ERR_UNSUPPORTED;
    }
    int sms = 0;
    TB_TRY(tb::sm_count(&sms));
    return each_table(grads, outs, numel, dtypes, T, [&](auto& prm, int k) {
        prm.records = const_cast<double*>(records);
        prm.n_records = n_records;
        prm.norm = norm;
        prm.max_norm = max_norm;
        prm.first = k == 0 ? 1 : 0;
        return launched(tb::launch_grad_clip(prm, sms, reinterpret_cast<cudaStream_t>(stream)));
    });
}

TB_API tb_status tb_patch_gn_grad_stats(const void* const* patches, const void* const* grads, int32_t P,
                                        tb_dtype dtype, int64_t N, int64_t C, const int64_t* spatial, int32_t G,
                                        const tb_gn_partial* partials, int32_t R, const void* gamma, const void* beta,
                                        float eps, int32_t silu, tb_gn_grad_partial* grad_partials, void* stream) {
    tb::GnGradParams prm;
    bool ring = false;
    TB_TRY(gn_grad_params(prm, &ring, patches, grads, nullptr, P, dtype, N, C, spatial, G, partials, R, gamma, beta,
                          eps, silu, grad_partials, nullptr, nullptr));
    if (N == 0 || C == 0) return TB_OK;
    int sms = 0;
    TB_TRY(tb::sm_count(&sms));
    TB_TRY(gn_grad_tasks(prm, tb::GRAD_STATS, dtype, sms));
    return launched(tb::launch_gn_grad(prm, (int)dtype, ring, sms, reinterpret_cast<cudaStream_t>(stream)));
}

TB_API tb_status tb_patch_gn_grad_apply(const void* const* patches, const void* const* grads, void* const* outs,
                                        int32_t P, tb_dtype dtype, int64_t N, int64_t C, const int64_t* spatial,
                                        int32_t G, const tb_gn_partial* partials,
                                        const tb_gn_grad_partial* grad_partials, int32_t R, const void* gamma,
                                        const void* beta, float eps, int32_t silu, void* dgamma, void* dbeta,
                                        void* stream) {
    tb::GnGradParams prm;
    bool ring = false;
    if (outs == nullptr) return TB_ERR_NULL;
    TB_TRY(gn_grad_params(prm, &ring, patches, grads, outs, P, dtype, N, C, spatial, G, partials, R, gamma, beta, eps,
                          silu, grad_partials, dgamma, dbeta));
    if (C == 0 || (N == 0 && prm.wtasks == 0)) return TB_OK;
    int sms = 0;
    TB_TRY(tb::sm_count(&sms));
    TB_TRY(gn_grad_tasks(prm, tb::GRAD_APPLY, dtype, sms));
    return launched(tb::launch_gn_grad(prm, (int)dtype, ring, sms, reinterpret_cast<cudaStream_t>(stream)));
}
