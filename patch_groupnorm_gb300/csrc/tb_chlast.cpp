// tb_chlast.cpp -- C ABI of the channels-last calls: PatchGroupNorm forward and
// backward, and dropout.  Argument validation and launch configuration only.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <numeric>

#include "tb_args.h"

namespace {

using tb::aligned;
using tb::elem_bytes;
using tb::known;
using tb::launched;

// What a call gives; outs, grads and the rest are NULL where it has none.
struct ClCall {
    const void* const* patches;
    const void* const* grads;
    void* const* outs;
    int32_t P;
    tb_dtype dtype;
    int64_t N, C;
    const int64_t* spatial;
    int32_t G;
    const tb_gn_partial* partials;
    int32_t R;
    const void* gamma;
    const void* beta;
    float eps;
    int32_t silu;
};

tb_status cl_params(tb::GnClParams& prm, const ClCall& c, bool grads, bool outs) {
    if (!known(c.dtype)) return TB_ERR_DTYPE;
    if (c.P < 1 || c.N < 0 || c.C < 0 || c.G < 1 || c.R < 1) return TB_ERR_SHAPE;
    if (c.C % c.G != 0) return TB_ERR_SHAPE;
    if (!(c.eps >= 0.0f) || std::isinf(c.eps)) return TB_ERR_SHAPE;
    if (c.P > tb::GN_MAXP || c.R > 65536 || c.C > tb::CL_MAXC) return TB_ERR_UNSUPPORTED;
    if (c.spatial == nullptr || c.patches == nullptr || (grads && c.grads == nullptr) || (outs && c.outs == nullptr))
        return TB_ERR_NULL;
    if ((double)std::max(c.P, c.R) * (double)c.N * (double)std::max<int64_t>(c.C, c.G) * TB_GN_PARTS > 2.0e9)
        return TB_ERR_UNSUPPORTED;
    std::memset(&prm, 0, sizeof(prm));
    const int es = elem_bytes(c.dtype);
    for (int p = 0; p < c.P; ++p) {
        if (c.spatial[p] < 0) return TB_ERR_SHAPE;
        prm.spatial[p] = c.spatial[p];
        if (c.N == 0 || c.C == 0 || c.spatial[p] == 0) continue;
        if ((double)c.N * (double)c.C * (double)c.spatial[p] > 1.0e13) return TB_ERR_UNSUPPORTED;
        prm.patches[p] = c.patches[p];
        if (grads) prm.grads[p] = c.grads[p];
        if (outs) prm.outs[p] = c.outs[p];
        if (prm.patches[p] == nullptr || (grads && prm.grads[p] == nullptr) || (outs && prm.outs[p] == nullptr))
            return TB_ERR_NULL;
        if (!aligned(prm.patches[p], es) || !aligned(prm.grads[p], es) || !aligned(prm.outs[p], es))
            return TB_ERR_UNSUPPORTED;
    }
    if (c.N > 0 && c.C > 0 && c.partials == nullptr) return TB_ERR_NULL;
    if (!aligned(c.gamma, es) || !aligned(c.beta, es) || !aligned(c.partials, 16)) return TB_ERR_UNSUPPORTED;
    prm.partials = reinterpret_cast<tb::GnPartial*>(const_cast<tb_gn_partial*>(c.partials));
    prm.gamma = c.gamma;
    prm.beta = c.beta;
    prm.N = c.N;
    prm.C = c.C;
    prm.P = c.P;
    prm.G = c.G;
    prm.K = (int32_t)(c.C / c.G);
    prm.R = c.R;
    prm.eps = c.eps;
    prm.silu = c.silu ? 1 : 0;
    prm.status = tb::checked_build_status();
    return TB_OK;
}

// Chunks of 16 bytes, if the call's tensors of every patch share their offset
// from 16-byte boundaries; then the period, and the columns a CTA takes at a time.
bool cl_chunks(tb::GnClParams& prm, tb_dtype dtype, bool grads, bool outs) {
    const int vec = 16 / elem_bytes(dtype);
    bool vector = true;
    for (int p = 0; p < prm.P; ++p) {
        const uintptr_t off = (uintptr_t)prm.patches[p] & 15u;
        if (grads && ((uintptr_t)prm.grads[p] & 15u) != off) vector = false;
        if (outs && ((uintptr_t)prm.outs[p] & 15u) != off) vector = false;
    }
    prm.period = (int32_t)(vector ? prm.C / std::gcd<int64_t>(prm.C, vec) : prm.C);
    const int turns = (prm.period + tb::CL_BLOCK - 1) / tb::CL_BLOCK;
    prm.columns = (prm.period + turns - 1) / turns;
    return vector;
}

int64_t cl_rows(const tb::GnClParams& prm, int p, int vec) {
    const int64_t chunks = prm.spatial[p] * prm.C / vec;
    return (chunks + prm.period - 1) / prm.period;
}

// The share of the SMs' places that clusters of this size find: theirs have to be in
// one group of SMs.  Of 304 places (two on each SM) clusters of 1 and 2 take all, of 3
// to 5 290 to 296, of 6 to 8 266 to 288; of 152, 138 to 144 and 105 to 138 (the
// runtime's own count).
double cl_places(int cluster, int per_sm) {
    if (cluster <= 2) return 1.0;
    if (cluster <= 5) return per_sm > 1 ? 0.95 : 0.9;
    return per_sm > 1 ? 0.87 : 0.69;
}

int cl_slabs(int width) {
    const int turns = (width + tb::CL_BLOCK - 1) / tb::CL_BLOCK;
    return turns <= tb::CL_MAX_CLUSTER ? turns : 1;
}

// Statistics: every (patch, sample) is a unit, cut into up to TB_GN_PARTS records
// of a cluster each; the channels may be split too, into runs of whole groups of at
// least 256 bytes a position.  Of the ways to cut, the one that comes nearest to the
// CTAs wanted (those resident at once), and of equals the one with the fewest splits,
// then the smallest clusters.
tb_status cl_plan_stats(tb::GnClParams& prm, tb_dtype dtype, bool vector, int ctas_wanted, int64_t* ctas) {
    const int es = elem_bytes(dtype), vec = vector ? 16 / es : 1;
    bool whole = prm.C % vec == 0;
    for (int p = 0; p < prm.P; ++p) whole = whole && (vec == 1 || aligned(prm.patches[p], 16));
    int64_t rows[tb::GN_MAXP], most = 1;
    for (int p = 0; p < prm.P; ++p) {
        rows[p] = cl_rows(prm, p, vec);
        most = std::max(most, rows[p]);
    }
    int64_t best = 0;
    int32_t splits = 1, cluster = cl_slabs(prm.period), parts = 1;
    for (int s = 1; s <= 16; s *= 2) {
        if (s > 1 && !(whole && prm.G % s == 0 && (prm.C / s) % vec == 0 && prm.C / s * es >= 256)) break;
        const int64_t columns = std::min<int64_t>(prm.period / s, tb::CL_BLOCK);
        // columns that do not fit a CTA's threads go to CTAs of a cluster, up to eight
        const int slabs = cl_slabs(prm.period / s);
        // at least four turns of a CTA's threads each
        const int64_t useful = std::max<int64_t>(1, most / (tb::CL_BLOCK / columns * 4)) * slabs;
        for (int c = slabs; c <= tb::CL_MAX_CLUSTER; c += slabs) {
            const double places = cl_places(c, 2) * ctas_wanted;
            for (int k = 1; k <= TB_GN_PARTS; ++k) {
                if (c * k > useful && c * k > slabs) continue;
                int64_t total = 0;
                for (int p = 0; p < prm.P; ++p) total += std::max<int64_t>(1, (rows[p] * k + most / 2) / most);
                total *= prm.N * c * s;
                if (total <= best || ((double)total > places && best > 0)) continue;
                best = total;
                splits = s;
                cluster = c;
                parts = k;
            }
        }
    }
    prm.splits = splits;
    prm.cluster = cluster;
    const int width = prm.period / splits, turns = (width + tb::CL_BLOCK - 1) / tb::CL_BLOCK;
    prm.columns = (width + turns - 1) / turns;
    prm.slabs = cl_slabs(width);
    int64_t at = 0;
    for (int p = 0; p < prm.P; ++p) {
        prm.parts[p] = (int32_t)std::max<int64_t>(1, (rows[p] * parts + most / 2) / most);
        prm.start[p] = (int32_t)at;
        at += prm.N * prm.parts[p];
        const int64_t pieces = (int64_t)prm.parts[p] * (cluster / prm.slabs);
        const int64_t side = tb::CL_BLOCK / prm.columns, blocks = (rows[p] + side - 1) / side;
        if (blocks / pieces > 2000000000LL) return TB_ERR_UNSUPPORTED;  // past any memory
        prm.rows[p] = rows[p];
        prm.share[p] = (int32_t)(blocks / pieces);
        prm.extra[p] = (int32_t)(blocks % pieces);
    }
    prm.start[prm.P] = (int32_t)at;
    *ctas = at * cluster;
    return TB_OK;
}

// Whether a call fits into shared memory in one launch, and how it is cut (see
// tb_gncl_fused.cu): of the ways for which all clusters have room at once, the fastest
// by an account fitted to measurements (us): 5.5 (backward 6.4) for the launch and the
// joining of sums, 0.43 (0.62) for each chunk that a thread takes after the other, half
// as much again with twice the threads on an SM, and forward 0.25 for every further sum
// that a chunk leaves.  The general path takes 9.8 and 0.36 a MB (12 and 0.26):
// where that is less, it is taken.  Both, by graph: 2 patches of 15 x 16 x 64 bf16 5.5
// and 7.9 us (6.6 and 10.7), 64 x 64 x 512 8.9 and 11.3 (11.4 and 14.1), 80 x 80 x 512
// 11.3 and 12.1, 96 x 96 x 512 13.8 and 13.5; where the groups cannot be split among
// clusters, 2 x 25 x 60 x 200 in 4 groups, 15.9 and 10.6 (13.2 and 13.3).
bool cl_plan_fused(tb::GnClParams& prm, tb_dtype dtype, bool grad, int sms, int* block) {
    const int es = elem_bytes(dtype), vec = 16 / es, tensors = grad ? 2 : 1;
    double bytes = 0;
    for (int p = 0; p < prm.P; ++p) {
        if (!aligned(prm.patches[p], 16) || !aligned(prm.outs[p], 16) || !aligned(prm.grads[p], 16)) return false;
        if (prm.spatial[p] * prm.C % vec != 0) return false;  // no single elements
        bytes += (double)prm.N * (double)prm.spatial[p] * (double)prm.C * es * tensors;
    }
    if (bytes > (double)sms * tb::CL_MAX_SMEM || prm.N > 65535) return false;
    prm.period = (int32_t)(prm.C / std::gcd<int64_t>(prm.C, vec));
    uint32_t rows[tb::GN_MAXP];  // below 2^31: they fit into shared memory
    for (int p = 0; p < prm.P; ++p)
        rows[p] = (uint32_t)((prm.spatial[p] * prm.C / vec + prm.period - 1) / prm.period);
    const int unit = std::min(vec, prm.K & -prm.K), sums = prm.K >= vec && unit * 2 < vec ? 2 : vec / unit;
    double best = (grad ? 12.0 : 9.8) + (grad ? 0.26e-6 : 0.36e-6) * bytes;
    int32_t splits = 0, slabs = 0, columns = 0, cluster = 0, most = 0;
    for (int s = 1; s <= prm.G && (s == 1 || prm.C / s * es >= 64); s *= 2) {
        if (s > 1 && (prm.G % s != 0 || prm.C % vec != 0 || (prm.C / s) % vec != 0)) break;
        prm.splits = s;
        const int width = prm.period / s;
        for (int b = 256; b <= 512; b *= 2) {
            const int turns = (width + b - 1) / b, wide = (width + turns - 1) / turns;
            for (int c = turns; c <= tb::CL_MAX_CLUSTER; c *= 2) {
                const uint32_t side = (uint32_t)(b / wide) * (uint32_t)(c / turns);
                uint32_t held = 0;
                for (int p = 0; p < prm.P; ++p) held += (rows[p] + side - 1) / side;
                if ((double)held * b * 16 > tb::CL_MAX_SMEM) continue;
                const size_t smem = tb::gncl_fused_smem(prm, (int)dtype, grad, b, (int)held);
                if (smem > (size_t)tb::CL_MAX_SMEM) continue;
                const int per_sm = (int)std::min<size_t>((size_t)(227 * 1024) / (smem + 1024), (size_t)(512 / b));
                const int64_t ctas = prm.N * s * c;
                if ((double)ctas > cl_places(c, per_sm) * per_sm * sms) continue;
                const int64_t threads = std::min<int64_t>(per_sm, (ctas + sms - 1) / sms) * b;
                const double us = grad ? 6.4 + held * (0.24 + threads / 670.0)
                                       : 5.5 + held * (0.2 + threads / 1100.0) + 0.25 * (sums - 1);
                if (us >= best) continue;
                best = us;
                splits = s;
                slabs = turns;
                columns = wide;
                cluster = c;
                most = (int32_t)held;
                *block = b;
            }
        }
    }
    prm.splits = splits;
    prm.slabs = slabs;
    prm.columns = columns;
    prm.cluster = cluster;
    prm.held = most;
    if (splits == 0) return false;
    prm.parts[0] = prm.G / splits;
    prm.parts[1] = prm.period / splits;
    prm.share[0] = cluster / slabs;
    for (int p = 0; p < prm.P; ++p) prm.start[p] = (int32_t)(prm.spatial[p] * prm.C / vec);
    return true;
}

// Element-wise passes: runs of rows of about the same length, as many as are
// resident at once.
void cl_plan_rows(tb::GnClParams& prm, tb_dtype dtype, bool vector, int ctas_wanted, int64_t* ctas) {
    const int vec = vector ? 16 / elem_bytes(dtype) : 1;
    const int64_t slabs = (prm.period + prm.columns - 1) / prm.columns;
    const int64_t wanted = std::max<int64_t>(1, ctas_wanted / slabs);
    const int64_t side = std::max(1, tb::CL_BLOCK / prm.columns);
    int64_t rows[tb::GN_MAXP], total = 0;
    for (int p = 0; p < prm.P; ++p) {
        rows[p] = cl_rows(prm, p, vec);
        total += prm.N * rows[p];
    }
    int64_t run = std::max<int64_t>(side, (total + wanted - 1) / wanted);
    for (;;) {
        int64_t at = 0;
        bool single = true;
        for (int p = 0; p < prm.P; ++p) {
            prm.parts[p] = (int32_t)std::max<int64_t>(1, (rows[p] + run - 1) / run);
            single = single && prm.parts[p] == 1;
            prm.start[p] = (int32_t)at;
            at += prm.N * prm.parts[p];
        }
        prm.start[prm.P] = (int32_t)at;
        *ctas = at;
        if (at <= wanted || single) return;
        run += std::max<int64_t>(1, run / 64);
    }
}

tb_status cl_stats(tb::GnClParams& prm, tb_dtype dtype, int sms, cudaStream_t s) {
    const bool vector = cl_chunks(prm, dtype, false, false);
    int64_t ctas = 0;
    TB_TRY(cl_plan_stats(prm, dtype, vector, 2 * sms, &ctas));
    return launched(tb::launch_gncl_stats(prm, (int)dtype, vector, ctas, s));
}

tb_status cl_apply(tb::GnClParams& prm, tb_dtype dtype, int sms, cudaStream_t s) {
    const bool vector = cl_chunks(prm, dtype, false, true);
    int64_t ctas = 0;
    cl_plan_rows(prm, dtype, vector, 2 * sms, &ctas);
    return launched(tb::launch_gncl_apply(prm, (int)dtype, vector, ctas, s));
}

tb_status cl_grad_stats(tb::GnClParams& prm, tb_dtype dtype, int sms, cudaStream_t s) {
    const bool vector = cl_chunks(prm, dtype, true, false);
    int64_t ctas = 0;
    TB_TRY(cl_plan_stats(prm, dtype, vector, 2 * sms, &ctas));
    return launched(tb::launch_gncl_grad_stats(prm, (int)dtype, vector, ctas, s));
}

tb_status cl_grad_apply(tb::GnClParams& prm, tb_dtype dtype, int sms, cudaStream_t s) {
    TB_TRY(launched(tb::launch_gncl_coefs(prm, (int)dtype, false, s)));
    if (prm.N == 0) return TB_OK;
    const bool vector = cl_chunks(prm, dtype, true, true);
    int64_t ctas = 0;
    cl_plan_rows(prm, dtype, vector, 2 * sms, &ctas);
    return launched(tb::launch_gncl_grad_apply(prm, (int)dtype, vector, ctas, s));
}

tb_status cl_records(tb::GnClParams& prm, const tb_gn_grad_partial* grad_partials) {
    if (grad_partials == nullptr && prm.N > 0 && prm.C > 0) return TB_ERR_NULL;
    if (!aligned(grad_partials, 16)) return TB_ERR_UNSUPPORTED;
    prm.grad_partials = reinterpret_cast<float2*>(const_cast<tb_gn_grad_partial*>(grad_partials));
    return TB_OK;
}

tb_status cl_weights(tb::GnClParams& prm, tb_dtype dtype, void* dgamma, void* dbeta, void* workspace,
                     int64_t workspace_bytes) {
    const int es = elem_bytes(dtype);
    if (!aligned(dgamma, es) || !aligned(dbeta, es) || !aligned(workspace, 16)) return TB_ERR_UNSUPPORTED;
    if (prm.N > 0 && prm.C > 0) {
        if (workspace == nullptr) return TB_ERR_NULL;
        if (workspace_bytes < tb_patch_gn_workspace_cl(prm.N, prm.G)) return TB_ERR_SHAPE;
    }
    prm.dgamma = dgamma;
    prm.dbeta = dbeta;
    prm.coefs = reinterpret_cast<float4*>(workspace);
    return TB_OK;
}

cudaStream_t as_stream(void* stream) { return reinterpret_cast<cudaStream_t>(stream); }

}  // namespace

TB_API tb_status tb_patch_gn_stats_cl(const void* const* patches, int32_t P, tb_dtype dtype, int64_t N, int64_t C,
                                      const int64_t* spatial, int32_t G, tb_gn_partial* partials, void* stream) {
    tb::GnClParams prm;
    TB_TRY(cl_params(prm, {patches, nullptr, nullptr, P, dtype, N, C, spatial, G, partials, 1, nullptr, nullptr, 0.f, 0},
                     false, false));
    if (N == 0 || C == 0) return TB_OK;
    int sms = 0;
    TB_TRY(tb::sm_count(&sms));
    return cl_stats(prm, dtype, sms, as_stream(stream));
}

TB_API tb_status tb_patch_gn_apply_cl(const void* const* patches, void* const* outs, int32_t P, tb_dtype dtype,
                                      int64_t N, int64_t C, const int64_t* spatial, int32_t G,
                                      const tb_gn_partial* partials, int32_t R, const void* gamma, const void* beta,
                                      float eps, int32_t silu, void* stream) {
    tb::GnClParams prm;
    TB_TRY(cl_params(prm, {patches, nullptr, outs, P, dtype, N, C, spatial, G, partials, R, gamma, beta, eps, silu},
                     false, true));
    if (N == 0 || C == 0) return TB_OK;
    int sms = 0;
    TB_TRY(tb::sm_count(&sms));
    return cl_apply(prm, dtype, sms, as_stream(stream));
}

TB_API tb_status tb_patch_group_norm_cl(const void* const* patches, void* const* outs, int32_t P, tb_dtype dtype,
                                        int64_t N, int64_t C, const int64_t* spatial, int32_t G,
                                        tb_gn_partial* partials, const void* gamma, const void* beta, float eps,
                                        int32_t silu, void* stream) {
    tb::GnClParams prm;
    TB_TRY(cl_params(prm, {patches, nullptr, outs, P, dtype, N, C, spatial, G, partials, P, gamma, beta, eps, silu},
                     false, true));
    if (N == 0 || C == 0) return TB_OK;
    int sms = 0;
    TB_TRY(tb::sm_count(&sms));
    int block = 0;
    if (cl_plan_fused(prm, dtype, false, sms, &block))
        return launched(tb::launch_gncl_fused(prm, (int)dtype, false, block, as_stream(stream)));
    TB_TRY(cl_stats(prm, dtype, sms, as_stream(stream)));
    return cl_apply(prm, dtype, sms, as_stream(stream));
}

TB_API int64_t tb_patch_gn_workspace_cl(int64_t N, int32_t G) {
    if (N < 0 || G < 1 || G > tb::CL_MAXC || N > (int64_t)1 << 31) return -1;
    return 16 * N * G;
}

TB_API tb_status tb_patch_gn_grad_stats_cl(const void* const* patches, const void* const* grads, int32_t P,
                                           tb_dtype dtype, int64_t N, int64_t C, const int64_t* spatial, int32_t G,
                                           const tb_gn_partial* partials, int32_t R, const void* gamma,
                                           const void* beta, float eps, int32_t silu,
                                           tb_gn_grad_partial* grad_partials, void* stream) {
    tb::GnClParams prm;
    TB_TRY(cl_params(prm, {patches, grads, nullptr, P, dtype, N, C, spatial, G, partials, R, gamma, beta, eps, silu},
                     true, false));
    TB_TRY(cl_records(prm, grad_partials));
    if (N == 0 || C == 0) return TB_OK;
    int sms = 0;
    TB_TRY(tb::sm_count(&sms));
    return cl_grad_stats(prm, dtype, sms, as_stream(stream));
}

TB_API tb_status tb_patch_gn_grad_apply_cl(const void* const* patches, const void* const* grads, void* const* outs,
                                           int32_t P, tb_dtype dtype, int64_t N, int64_t C, const int64_t* spatial,
                                           int32_t G, const tb_gn_partial* partials,
                                           const tb_gn_grad_partial* grad_partials, int32_t R, const void* gamma,
                                           const void* beta, float eps, int32_t silu, void* dgamma, void* dbeta,
                                           void* workspace, int64_t workspace_bytes, void* stream) {
    tb::GnClParams prm;
    TB_TRY(cl_params(prm, {patches, grads, outs, P, dtype, N, C, spatial, G, partials, R, gamma, beta, eps, silu}, true,
                     true));
    TB_TRY(cl_records(prm, grad_partials));
    TB_TRY(cl_weights(prm, dtype, dgamma, dbeta, workspace, workspace_bytes));
    if (C == 0 || (N == 0 && dgamma == nullptr && dbeta == nullptr)) return TB_OK;
    int sms = 0;
    TB_TRY(tb::sm_count(&sms));
    return cl_grad_apply(prm, dtype, sms, as_stream(stream));
}

TB_API tb_status tb_patch_group_norm_backward_cl(const void* const* patches, const void* const* grads,
                                                 void* const* outs, int32_t P, tb_dtype dtype, int64_t N, int64_t C,
                                                 const int64_t* spatial, int32_t G, const tb_gn_partial* partials,
                                                 tb_gn_grad_partial* grad_partials, const void* gamma,
                                                 const void* beta, float eps, int32_t silu, void* dgamma, void* dbeta,
                                                 void* workspace, int64_t workspace_bytes, void* stream) {
    tb::GnClParams prm;
    TB_TRY(cl_params(prm, {patches, grads, outs, P, dtype, N, C, spatial, G, partials, P, gamma, beta, eps, silu}, true,
                     true));
    TB_TRY(cl_records(prm, grad_partials));
    TB_TRY(cl_weights(prm, dtype, dgamma, dbeta, workspace, workspace_bytes));
    if (C == 0 || (N == 0 && dgamma == nullptr && dbeta == nullptr)) return TB_OK;
    int sms = 0;
    TB_TRY(tb::sm_count(&sms));
    int block = 0;
    if (N > 0 && cl_plan_fused(prm, dtype, true, sms, &block)) {
        TB_TRY(launched(tb::launch_gncl_fused(prm, (int)dtype, true, block, as_stream(stream))));
        if (N == 1 || (dgamma == nullptr && dbeta == nullptr)) return TB_OK;
        prm.coefs = nullptr;
        return launched(tb::launch_gncl_coefs(prm, (int)dtype, true, as_stream(stream)));
    }
    if (N > 0) TB_TRY(cl_grad_stats(prm, dtype, sms, as_stream(stream)));
    return cl_grad_apply(prm, dtype, sms, as_stream(stream));
}

TB_API tb_status tb_dropout(const void* x, int64_t x_ld, const void* residual, int64_t residual_ld, tb_dtype dtype,
                            int64_t rows, int64_t cols, double p, uint64_t seed, uint64_t offset,
                            const uint64_t* state, void* y, int64_t y_ld, void* stream) {
    if (!known(dtype)) return TB_ERR_DTYPE;
    if (rows < 0 || cols < 0 || !(p >= 0.0 && p <= 1.0)) return TB_ERR_SHAPE;
    if (rows == 0 || cols == 0) return TB_OK;
    if ((double)rows * (double)cols > 1099511627776.0) return TB_ERR_UNSUPPORTED;
    const int es = elem_bytes(dtype);
    bool vector = true, dense = true;
    const struct {
        const void* at;
        int64_t ld;
        bool needed;
    } tensors[3] = {{x, x_ld, true}, {y, y_ld, true}, {residual, residual_ld, residual != nullptr}};
    for (const auto& t : tensors) {
        if (!t.needed) continue;
        if (t.at == nullptr) return TB_ERR_NULL;
        if (rows > 1 && (t.ld < cols || (double)rows * (double)t.ld > 2.0e18)) return TB_ERR_SHAPE;
        if (!aligned(t.at, es)) return TB_ERR_UNSUPPORTED;
        if (!aligned(t.at, 16) || (rows > 1 && t.ld % (16 / es) != 0)) vector = false;
        if (rows > 1 && t.ld != cols) dense = false;
    }
    if (!aligned(state, 8)) return TB_ERR_UNSUPPORTED;
    tb::DropoutParams prm;
    prm.x = x;
    prm.residual = residual;
    prm.y = y;
    prm.state = state;
    prm.rows = dense ? 1 : rows;
    prm.cols = dense ? rows * cols : cols;
    prm.x_ld = x_ld;
    prm.r_ld = residual_ld;
    prm.y_ld = y_ld;
    if (prm.rows == 1) prm.x_ld = prm.r_ld = prm.y_ld = prm.cols;
    prm.seed = seed;
    prm.offset = offset;
    prm.status = tb::checked_build_status();
    prm.threshold = (uint32_t)std::floor(p * 65536.0 + 0.5);
    prm.scale = prm.threshold < 65536u ? (float)(65536.0 / (65536 - prm.threshold)) : 0.f;
    // dense rows of any width are one row: its base decides
    if (dense) vector = aligned(x, 16) && aligned(y, 16) && aligned(residual, 16);
    else vector = vector && cols % 8 == 0;
    return launched(tb::launch_dropout(prm, (int)dtype, vector, as_stream(stream)));
}
