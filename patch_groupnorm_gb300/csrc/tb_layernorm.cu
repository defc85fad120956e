// tb_layernorm.cu -- layer norm over the last axis, forward and backward.
//
// Forward, row by row (n = cols):
//     h = residual ? rnd(x + residual) : x
//     mean = sum(h) / n,  var = sum((h - mean)^2) / n,  rstd = 1 / sqrt(var + eps)
//     y = rnd((h - mean) * rstd * gamma + beta)
// Backward, with xhat = (h - mean) * rstd and g = dy * gamma:
//     dx = rnd(rstd * (g - sum(g) / n - xhat * sum(g * xhat) / n) + dtotal)
//     dgamma = sum over rows of dy * xhat,  dbeta = sum over rows of dy
// All sums and statistics are fp32; every output is rounded once.
//
// A row is held by TPR threads, CPT chunks each, in registers: one read of
// the row serves the mean, the squares about it (a second pass over
// registers, so an outlier or a large offset costs no precision) and the
// output.  Both kernels are bound by memory bandwidth; the next row's chunks
// are requested before the current row is reduced.
#include "tb_elem.cuh"

namespace tb {
namespace {

// Threads per CTA: a row's threads, at least four warps.
__host__ __device__ constexpr int ln_block(int tpr) { return tpr < 128 ? 128 : tpr; }
// CTAs per SM the forward kernel is compiled for.
__host__ __device__ constexpr int ln_fwd_ctas(int tpr) { return tpr <= 128 ? 8 : tpr <= 256 ? 4 : tpr <= 512 ? 2 : 1; }

// Sum over the TPR threads of a row; every thread gets the result.  `slot`
// (one float per warp) must not be reused before another barrier.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* slot) {
    v = warp_sum(v);
    if constexpr (TPR > 32) {
        if ((threadIdx.x & 31) == 0) slot[threadIdx.x >> 5] = v;
        __syncthreads();
        v = 0.f;
#pragma unroll
        for (int w = 0; w < TPR / 32; ++w) v += slot[w];
    }
    return v;
}

template <int DT, int VEC, int TPR, int CPT, bool RES>
__global__ void __launch_bounds__(ln_block(TPR), ln_fwd_ctas(TPR)) ln_fwd_kernel(const __grid_constant__ LnFwdParams p) {
    using W = typename Word<VEC * elem_size(DT)>::T;
    constexpr int RPC = ln_block(TPR) / TPR;  // rows per CTA
    constexpr bool KEEP = CPT * VEC <= 16;    // weights stay in registers
    __shared__ float s_a[32], s_b[32];
    const int t = threadIdx.x % TPR;
    const int64_t step = (int64_t)gridDim.x * RPC;
    int64_t row = (int64_t)blockIdx.x * RPC + threadIdx.x / TPR;
    const int nchunk = (int)(p.cols / VEC);
    const float n = (float)p.cols;
    const int64_t row_bytes = p.cols * elem_size(DT);
    grid_wait();

    float g[KEEP ? CPT * VEC : 1], b[KEEP ? CPT * VEC : 1];
    if constexpr (KEEP) {
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
            const int c = t + k * TPR;
            if (c < nchunk) {
                float gv[VEC], bv[VEC];
                weights_at<VEC, true>(p.gamma, p.wdtype, (int64_t)c * VEC, 1.f, gv);
                weights_at<VEC, true>(p.beta, p.wdtype, (int64_t)c * VEC, 0.f, bv);
#pragma unroll
                for (int q = 0; q < VEC; ++q) {
                    g[k * VEC + q] = gv[q];
                    b[k * VEC + q] = bv[q];
                }
            }
        }
    }
    auto row_at = [&](const void* base, int64_t r, int64_t ld) {
        return reinterpret_cast<const char*>(base) + r * ld * elem_size(DT);
    };
    auto fetch = [&](const void* base, int64_t r, int64_t ld, W (&v)[CPT]) {
        const char* const at = row_at(base, r, ld);
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
            const int c = t + k * TPR;
            const W* const src = reinterpret_cast<const W*>(at) + c;
            if (c < nchunk && in_bounds(src, sizeof(W), at, row_bytes, p.status)) v[k] = __ldcs(src);
        }
    };
    W nx[CPT], nr[RES ? CPT : 1];
    if (row < p.rows) {
        fetch(p.x, row, p.x_ld, nx);
        if constexpr (RES) fetch(p.residual, row, p.r_ld, nr);
    }
    for (; row < p.rows; row += step) {
        float h[CPT * VEC];
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
            const int c = t + k * TPR;
            if (c < nchunk) {
                float f[VEC];
                unpack<DT, VEC>(nx[k], f);
                if constexpr (RES) {
                    float r[VEC];
                    unpack<DT, VEC>(nr[k], r);
#pragma unroll
                    for (int q = 0; q < VEC; ++q) f[q] += r[q];
                    const W w = pack<DT, VEC>(f);  // the sum as stored is what is normalised
                    unpack<DT, VEC>(w, f);
                    char* const at = reinterpret_cast<char*>(p.total) + row * p.t_ld * elem_size(DT);
                    W* const dst = reinterpret_cast<W*>(at) + c;
                    if (in_bounds(dst, sizeof(W), at, row_bytes, p.status)) *dst = w;
                }
#pragma unroll
                for (int q = 0; q < VEC; ++q) {
                    h[k * VEC + q] = f[q];
                    sum += f[q];
                }
            }
        }
        if (row + step < p.rows) {
            fetch(p.x, row + step, p.x_ld, nx);
            if constexpr (RES) fetch(p.residual, row + step, p.r_ld, nr);
        }
        const float mean = row_sum<TPR>(sum, s_a) / n;
        float m2 = 0.f;
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
            if (t + k * TPR < nchunk) {
#pragma unroll
                for (int q = 0; q < VEC; ++q) {
                    h[k * VEC + q] -= mean;
                    m2 = fmaf(h[k * VEC + q], h[k * VEC + q], m2);
                }
            }
        }
        const float rstd = 1.0f / sqrtf(row_sum<TPR>(m2, s_b) / n + p.eps);
        if (t == 0) {
            if (p.mean) p.mean[row] = mean;
            if (p.rstd) p.rstd[row] = rstd;
        }
        char* const at = reinterpret_cast<char*>(p.y) + row * p.y_ld * elem_size(DT);
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
            const int c = t + k * TPR;
            if (c < nchunk) {
                float f[VEC];
                if constexpr (KEEP) {
#pragma unroll
                    for (int q = 0; q < VEC; ++q) f[q] = fmaf(h[k * VEC + q] * rstd, g[k * VEC + q], b[k * VEC + q]);
                } else {
                    float gv[VEC], bv[VEC];
                    weights_at<VEC, true>(p.gamma, p.wdtype, (int64_t)c * VEC, 1.f, gv);
                    weights_at<VEC, true>(p.beta, p.wdtype, (int64_t)c * VEC, 0.f, bv);
#pragma unroll
                    for (int q = 0; q < VEC; ++q) f[q] = fmaf(h[k * VEC + q] * rstd, gv[q], bv[q]);
                }
                W* const dst = reinterpret_cast<W*>(at) + c;
                if (in_bounds(dst, sizeof(W), at, row_bytes, p.status)) *dst = pack<DT, VEC>(f);
            }
        }
    }
}

// Rows too long for registers: one CTA per row, which it reads three times
// (sum, squares about the mean, output; the second and third time mostly
// from L2).  Each thread reads back only what it wrote itself.
constexpr int LONG_BLOCK = 1024;

template <int DT, int VEC, bool RES>
__global__ void __launch_bounds__(LONG_BLOCK) ln_fwd_long_kernel(const __grid_constant__ LnFwdParams p) {
    using W = typename Word<VEC * elem_size(DT)>::T;
    __shared__ float s_a[32], s_b[32];
    const int64_t nchunk = p.cols / VEC;
    const float n = (float)p.cols;
    grid_wait();
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const W* const x = reinterpret_cast<const W*>(reinterpret_cast<const char*>(p.x) + row * p.x_ld * elem_size(DT));
        const W* r = nullptr;
        const W* h = x;
        W* tot = nullptr;
        if constexpr (RES) {
            r = reinterpret_cast<const W*>(reinterpret_cast<const char*>(p.residual) + row * p.r_ld * elem_size(DT));
            tot = reinterpret_cast<W*>(reinterpret_cast<char*>(p.total) + row * p.t_ld * elem_size(DT));
            h = tot;
        }
        float sum = 0.f;
        for (int64_t c = threadIdx.x; c < nchunk; c += LONG_BLOCK) {
            float f[VEC];
            unpack<DT, VEC>(x[c], f);
            if constexpr (RES) {
                float rf[VEC];
                unpack<DT, VEC>(r[c], rf);
#pragma unroll
                for (int q = 0; q < VEC; ++q) f[q] += rf[q];
                const W w = pack<DT, VEC>(f);
                unpack<DT, VEC>(w, f);
                tot[c] = w;
            }
#pragma unroll
            for (int q = 0; q < VEC; ++q) sum += f[q];
        }
        const float mean = row_sum<LONG_BLOCK>(sum, s_a) / n;
        float m2 = 0.f;
        for (int64_t c = threadIdx.x; c < nchunk; c += LONG_BLOCK) {
            float f[VEC];
            unpack<DT, VEC>(h[c], f);
#pragma unroll
            for (int q = 0; q < VEC; ++q) m2 = fmaf(f[q] - mean, f[q] - mean, m2);
        }
        const float rstd = 1.0f / sqrtf(row_sum<LONG_BLOCK>(m2, s_b) / n + p.eps);
        if (threadIdx.x == 0) {
            if (p.mean) p.mean[row] = mean;
            if (p.rstd) p.rstd[row] = rstd;
        }
        W* const y = reinterpret_cast<W*>(reinterpret_cast<char*>(p.y) + row * p.y_ld * elem_size(DT));
        for (int64_t c = threadIdx.x; c < nchunk; c += LONG_BLOCK) {
            float f[VEC], gv[VEC], bv[VEC];
            unpack<DT, VEC>(h[c], f);
            weights_at<VEC, true>(p.gamma, p.wdtype, c * VEC, 1.f, gv);
            weights_at<VEC, true>(p.beta, p.wdtype, c * VEC, 0.f, bv);
#pragma unroll
            for (int q = 0; q < VEC; ++q) f[q] = fmaf((f[q] - mean) * rstd, gv[q], bv[q]);
            y[c] = pack<DT, VEC>(f);
        }
    }
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------

// CTAs per SM the backward kernel is compiled for, and so the number of
// partial weight gradients (one per CTA).
__host__ __device__ constexpr int ln_bwd_ctas(int tpr) { return tpr <= 128 ? 3 : tpr <= 256 ? 2 : 1; }
__host__ __device__ constexpr int ln_bwd_block(int tpr) { return tpr < 256 ? 256 : tpr; }

// Each thread keeps the weight gradients of its own columns over all rows
// its CTA takes; the CTA's sums go to workspace[part][2][cols] (dgamma, then
// dbeta), which ln_wgrad_kernel adds up in part order: no atomics, the same
// bits every time.
template <int DT, int VEC, int TPR, int CPT, bool TOT>
__global__ void __launch_bounds__(ln_bwd_block(TPR), ln_bwd_ctas(TPR)) ln_bwd_kernel(const __grid_constant__ LnBwdParams p) {
    using W = typename Word<VEC * elem_size(DT)>::T;
    constexpr int N = CPT * VEC;
    constexpr int RPC = ln_bwd_block(TPR) / TPR;
    constexpr int WPR = TPR / 32;
    __shared__ float2 s_sum[2][ln_bwd_block(TPR) / 32];
    extern __shared__ float s_acc[];  // RPC > 1: [2][cols]
    const int t = threadIdx.x % TPR, rl = threadIdx.x / TPR;
    const int64_t step = (int64_t)gridDim.x * RPC;
    const int nchunk = (int)(p.cols / VEC);
    const float inv_n = 1.0f / (float)p.cols;
    const int64_t row_bytes = p.cols * elem_size(DT);
    grid_wait();

    float g[N], dg[N], db[N];
#pragma unroll
    for (int k = 0; k < CPT; ++k) {
        const int c = t + k * TPR;
        float gv[VEC];
#pragma unroll
        for (int q = 0; q < VEC; ++q) gv[q] = 0.f;
        if (c < nchunk) weights_at<VEC, true>(p.gamma, p.wdtype, (int64_t)c * VEC, 1.f, gv);
#pragma unroll
        for (int q = 0; q < VEC; ++q) {
            g[k * VEC + q] = gv[q];
            dg[k * VEC + q] = 0.f;
            db[k * VEC + q] = 0.f;
        }
    }
    auto fetch = [&](const void* base, int64_t r, int64_t ld, W (&v)[CPT]) {
        const char* const at = reinterpret_cast<const char*>(base) + r * ld * elem_size(DT);
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
            const int c = t + k * TPR;
            const W* const src = reinterpret_cast<const W*>(at) + c;
            if (c < nchunk && in_bounds(src, sizeof(W), at, row_bytes, p.status)) v[k] = __ldcs(src);
        }
    };
    W nd[CPT], nx[CPT], nt[TOT ? CPT : 1];
    float nmean = 0.f, nrstd = 0.f;
    int64_t row = (int64_t)blockIdx.x * RPC + rl;
    if (row < p.rows) {
        fetch(p.dy, row, p.dy_ld, nd);
        fetch(p.x, row, p.x_ld, nx);
        if constexpr (TOT) fetch(p.dtotal, row, p.dt_ld, nt);
        nmean = p.mean[row];
        nrstd = p.rstd[row];
    }
    int phase = 0;
    for (; row < p.rows; row += step) {
        const float mean = nmean, rstd = nrstd;
        W cd[CPT], cx[CPT], ct[TOT ? CPT : 1];
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
            cd[k] = nd[k];
            cx[k] = nx[k];
            if constexpr (TOT) ct[k] = nt[k];
        }
        if (row + step < p.rows) {
            fetch(p.dy, row + step, p.dy_ld, nd);
            fetch(p.x, row + step, p.x_ld, nx);
            if constexpr (TOT) fetch(p.dtotal, row + step, p.dt_ld, nt);
            nmean = p.mean[row + step];
            nrstd = p.rstd[row + step];
        }
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
            if (t + k * TPR < nchunk) {
                float d[VEC], x[VEC];
                unpack<DT, VEC>(cd[k], d);
                unpack<DT, VEC>(cx[k], x);
#pragma unroll
                for (int q = 0; q < VEC; ++q) {
                    const float xh = (x[q] - mean) * rstd;
                    const float gd = d[q] * g[k * VEC + q];
                    s1 += gd;
                    s2 = fmaf(gd, xh, s2);
                    dg[k * VEC + q] = fmaf(d[q], xh, dg[k * VEC + q]);
                    db[k * VEC + q] += d[q];
                }
            }
        }
        s1 = warp_sum(s1);
        s2 = warp_sum(s2);
        if constexpr (TPR > 32) {
            // the slots alternate, so one barrier per row suffices
            if ((threadIdx.x & 31) == 0) s_sum[phase][threadIdx.x >> 5] = make_float2(s1, s2);
            if constexpr (RPC == 1) {
                __syncthreads();
            } else {  // the row's own threads only: rows of a CTA run apart
                asm volatile("bar.sync %0, %1;" ::"r"(rl + 1), "n"(TPR) : "memory");
            }
            s1 = 0.f;
            s2 = 0.f;
#pragma unroll
            for (int w = 0; w < WPR; ++w) {
                const float2 v = s_sum[phase][rl * WPR + w];
                s1 += v.x;
                s2 += v.y;
            }
            phase ^= 1;
        }
        const float c1 = s1 * inv_n, c2 = s2 * inv_n;
        if (p.dx != nullptr) {
            char* const at = reinterpret_cast<char*>(p.dx) + row * p.dx_ld * elem_size(DT);
#pragma unroll
            for (int k = 0; k < CPT; ++k) {
                const int c = t + k * TPR;
                if (c < nchunk) {
                    float d[VEC], x[VEC], o[VEC];
                    unpack<DT, VEC>(cd[k], d);
                    unpack<DT, VEC>(cx[k], x);
#pragma unroll
                    for (int q = 0; q < VEC; ++q) {
                        const float xh = (x[q] - mean) * rstd;
                        o[q] = rstd * (fmaf(d[q], g[k * VEC + q], -c1) - xh * c2);
                    }
                    if constexpr (TOT) {
                        float tt[VEC];
                        unpack<DT, VEC>(ct[k], tt);
#pragma unroll
                        for (int q = 0; q < VEC; ++q) o[q] += tt[q];
                    }
                    W* const dst = reinterpret_cast<W*>(at) + c;
                    if (in_bounds(dst, sizeof(W), at, row_bytes, p.status)) *dst = pack<DT, VEC>(o);
                }
            }
        }
    }

    if (p.workspace == nullptr) return;
    if constexpr (RPC > 1) {
        // the CTA's row groups add their sums in turn (a fixed order)
        for (int w = 0; w < RPC; ++w) {
            if (rl == w) {
#pragma unroll
                for (int k = 0; k < CPT; ++k) {
                    const int c = t + k * TPR;
                    if (c < nchunk) {
#pragma unroll
                        for (int q = 0; q < VEC; ++q) {
                            float* const a = s_acc + c * VEC + q;
                            const float vg = dg[k * VEC + q] + (w ? a[0] : 0.f);
                            const float vb = db[k * VEC + q] + (w ? a[p.cols] : 0.f);
                            a[0] = vg;
                            a[p.cols] = vb;
                        }
                    }
                }
            }
            __syncthreads();
        }
        float* const out = p.workspace + (int64_t)blockIdx.x * 2 * p.cols;
        for (int64_t i = threadIdx.x; i < 2 * p.cols; i += ln_bwd_block(TPR)) out[i] = s_acc[i];
    } else {
        float* const out = p.workspace + (int64_t)blockIdx.x * 2 * p.cols;
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
            const int c = t + k * TPR;
            if (c < nchunk) {
#pragma unroll
                for (int q = 0; q < VEC; ++q) {
                    out[c * VEC + q] = dg[k * VEC + q];
                    out[p.cols + c * VEC + q] = db[k * VEC + q];
                }
            }
        }
    }
}

// Rows too long for registers: one CTA per row, the row's columns read twice
// (sums, then outputs), and the weight gradients accumulated in the CTA's
// own workspace slice, each column by one thread.
template <int DT, int VEC, bool TOT>
__global__ void __launch_bounds__(LONG_BLOCK) ln_bwd_long_kernel(const __grid_constant__ LnBwdParams p) {
    using W = typename Word<VEC * elem_size(DT)>::T;
    __shared__ float s_a[32], s_b[32];
    const int64_t nchunk = p.cols / VEC;
    const float inv_n = 1.0f / (float)p.cols;
    float* const acc = p.workspace == nullptr ? nullptr : p.workspace + (int64_t)blockIdx.x * 2 * p.cols;
    grid_wait();
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const W* const dy = reinterpret_cast<const W*>(reinterpret_cast<const char*>(p.dy) + row * p.dy_ld * elem_size(DT));
        const W* const x = reinterpret_cast<const W*>(reinterpret_cast<const char*>(p.x) + row * p.x_ld * elem_size(DT));
        const float mean = p.mean[row], rstd = p.rstd[row];
        float s1 = 0.f, s2 = 0.f;
        const bool first = row == blockIdx.x;
        for (int64_t c = threadIdx.x; c < nchunk; c += LONG_BLOCK) {
            float d[VEC], xv[VEC], gv[VEC];
            unpack<DT, VEC>(dy[c], d);
            unpack<DT, VEC>(x[c], xv);
            weights_at<VEC, true>(p.gamma, p.wdtype, c * VEC, 1.f, gv);
#pragma unroll
            for (int q = 0; q < VEC; ++q) {
                const float xh = (xv[q] - mean) * rstd, gd = d[q] * gv[q];
                s1 += gd;
                s2 = fmaf(gd, xh, s2);
                if (acc != nullptr) {
                    float* const a = acc + c * VEC + q;
                    a[0] = fmaf(d[q], xh, first ? 0.f : a[0]);
                    a[p.cols] = d[q] + (first ? 0.f : a[p.cols]);
                }
            }
        }
        const float c1 = row_sum<LONG_BLOCK>(s1, s_a) * inv_n, c2 = row_sum<LONG_BLOCK>(s2, s_b) * inv_n;
        if (p.dx == nullptr) continue;
        W* const dx = reinterpret_cast<W*>(reinterpret_cast<char*>(p.dx) + row * p.dx_ld * elem_size(DT));
        for (int64_t c = threadIdx.x; c < nchunk; c += LONG_BLOCK) {
            float d[VEC], xv[VEC], gv[VEC], o[VEC];
            unpack<DT, VEC>(dy[c], d);
            unpack<DT, VEC>(x[c], xv);
            weights_at<VEC, true>(p.gamma, p.wdtype, c * VEC, 1.f, gv);
#pragma unroll
            for (int q = 0; q < VEC; ++q) {
                const float xh = (xv[q] - mean) * rstd;
                o[q] = rstd * (fmaf(d[q], gv[q], -c1) - xh * c2);
            }
            if constexpr (TOT) {
                float tt[VEC];
                unpack<DT, VEC>(reinterpret_cast<const W*>(reinterpret_cast<const char*>(p.dtotal) +
                                                           row * p.dt_ld * elem_size(DT))[c], tt);
#pragma unroll
                for (int q = 0; q < VEC; ++q) o[q] += tt[q];
            }
            dx[c] = pack<DT, VEC>(o);
        }
    }
}

// dgamma[c] and dbeta[c]: the sum of the parts' columns.  A CTA takes 32
// columns of one of the two; its 16 warps sum every 16th part, and warp 0
// adds the 16 in order.
constexpr int WG_SLICES = 16;

__global__ void __launch_bounds__(32 * WG_SLICES) ln_wgrad_kernel(const __grid_constant__ LnWgradParams p) {
    __shared__ float s[WG_SLICES][32];
    const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane;
    const int which = blockIdx.y;
    void* const out = which ? p.dbeta : p.dgamma;
    grid_wait();
    if (out == nullptr) return;
    float v = 0.f;
    if (c < p.cols) {
        const float* const at = p.workspace + which * p.cols + c;
        for (int k = slice; k < p.parts; k += WG_SLICES) v += at[(int64_t)k * 2 * p.cols];
    }
    s[slice][lane] = v;
    __syncthreads();
    if (slice == 0 && c < p.cols) {
        v = s[0][lane];
#pragma unroll
        for (int k = 1; k < WG_SLICES; ++k) v += s[k][lane];
        store_weight(out, p.wdtype, c, v);
    }
}

// ---------------------------------------------------------------------------
// dispatch: a row's chunk count picks the threads and chunks per thread
// ---------------------------------------------------------------------------

template <int DT, int VEC, int TPR, int CPT>
cudaError_t fwd_launch(const LnFwdParams& p, int sms, cudaStream_t s) {
    constexpr int rpc = ln_block(TPR) / TPR;
    const int64_t want = (p.rows + rpc - 1) / rpc;
    const unsigned grid = (unsigned)(want < (int64_t)sms * ln_fwd_ctas(TPR) ? want : (int64_t)sms * ln_fwd_ctas(TPR));
    return launch_pdl(p.residual ? ln_fwd_kernel<DT, VEC, TPR, CPT, true> : ln_fwd_kernel<DT, VEC, TPR, CPT, false>, p,
                      dim3(grid), ln_block(TPR), 0, s);
}

template <int DT, int VEC>
cudaError_t fwd_long(const LnFwdParams& p, int sms, cudaStream_t s) {
    const unsigned grid = (unsigned)(p.rows < 2 * sms ? p.rows : 2 * sms);
    return launch_pdl(p.residual ? ln_fwd_long_kernel<DT, VEC, true> : ln_fwd_long_kernel<DT, VEC, false>, p,
                      dim3(grid), LONG_BLOCK, 0, s);
}

template <int DT>
cudaError_t fwd_dt(const LnFwdParams& p, bool vector, int sms, cudaStream_t s) {
    if (vector) {
        constexpr int V = 16 / elem_size(DT);
        const int64_t n = p.cols / V;
        if (n <= 32) return fwd_launch<DT, V, 32, 1>(p, sms, s);
        if (n <= 64) return fwd_launch<DT, V, 32, 2>(p, sms, s);
        if (n <= 128) return fwd_launch<DT, V, 32, 4>(p, sms, s);
        if (n <= 256) return fwd_launch<DT, V, 128, 2>(p, sms, s);
        if (n <= 512) return fwd_launch<DT, V, 256, 2>(p, sms, s);
        if (n <= 1024) return fwd_launch<DT, V, 512, 2>(p, sms, s);
        if (n <= 2048) return fwd_launch<DT, V, 1024, 2>(p, sms, s);
        if (n <= 4096) return fwd_launch<DT, V, 1024, 4>(p, sms, s);
        return fwd_long<DT, V>(p, sms, s);
    }
    if (p.cols <= 256) return fwd_launch<DT, 1, 32, 8>(p, sms, s);
    if (p.cols <= 1024) return fwd_launch<DT, 1, 128, 8>(p, sms, s);
    if (p.cols <= 2048) return fwd_launch<DT, 1, 256, 8>(p, sms, s);
    if (p.cols <= 4096) return fwd_launch<DT, 1, 512, 8>(p, sms, s);
    if (p.cols <= 16384) return fwd_launch<DT, 1, 1024, 16>(p, sms, s);
    return fwd_long<DT, 1>(p, sms, s);
}

template <int DT, int VEC, int TPR, int CPT>
cudaError_t bwd_launch(const LnBwdParams& p, int sms, int* parts, cudaStream_t s) {
    constexpr int rpc = ln_bwd_block(TPR) / TPR;
    const int64_t want = (p.rows + rpc - 1) / rpc;
    int64_t grid = (int64_t)sms * ln_bwd_ctas(TPR);
    if (grid > TB_LN_PARTS) grid = TB_LN_PARTS;
    if (grid > want) grid = want;
    *parts = (int)grid;
    const size_t smem = rpc > 1 && p.workspace != nullptr ? (size_t)p.cols * 8 : 0;
    return launch_pdl(p.dtotal ? ln_bwd_kernel<DT, VEC, TPR, CPT, true> : ln_bwd_kernel<DT, VEC, TPR, CPT, false>, p,
                      dim3((unsigned)grid), ln_bwd_block(TPR), smem, s);
}

template <int DT, int VEC>
cudaError_t bwd_long(const LnBwdParams& p, int sms, int* parts, cudaStream_t s) {
    int64_t grid = p.rows < sms ? p.rows : sms;
    if (grid > TB_LN_PARTS) grid = TB_LN_PARTS;
    *parts = (int)grid;
    return launch_pdl(p.dtotal ? ln_bwd_long_kernel<DT, VEC, true> : ln_bwd_long_kernel<DT, VEC, false>, p,
                      dim3((unsigned)grid), LONG_BLOCK, 0, s);
}

template <int DT>
cudaError_t bwd_dt(const LnBwdParams& p, bool vector, int sms, int* parts, cudaStream_t s) {
    if (vector) {
        constexpr int V = 16 / elem_size(DT);
        const int64_t n = p.cols / V;
        if (n <= 32) return bwd_launch<DT, V, 32, 1>(p, sms, parts, s);
        if (n <= 64) return bwd_launch<DT, V, 32, 2>(p, sms, parts, s);
        if (n <= 128) return bwd_launch<DT, V, 64, 2>(p, sms, parts, s);
        if (n <= 256) return bwd_launch<DT, V, 128, 2>(p, sms, parts, s);
        if (n <= 512) return bwd_launch<DT, V, 256, 2>(p, sms, parts, s);
        if (n <= 1024) return bwd_launch<DT, V, 512, 2>(p, sms, parts, s);
        if (n <= 2048) return bwd_launch<DT, V, 1024, 2>(p, sms, parts, s);
        return bwd_long<DT, V>(p, sms, parts, s);
    }
    if (p.cols <= 256) return bwd_launch<DT, 1, 32, 8>(p, sms, parts, s);
    if (p.cols <= 512) return bwd_launch<DT, 1, 64, 8>(p, sms, parts, s);
    if (p.cols <= 1024) return bwd_launch<DT, 1, 128, 8>(p, sms, parts, s);
    if (p.cols <= 2048) return bwd_launch<DT, 1, 256, 8>(p, sms, parts, s);
    if (p.cols <= 4096) return bwd_launch<DT, 1, 512, 8>(p, sms, parts, s);
    if (p.cols <= 8192) return bwd_launch<DT, 1, 1024, 8>(p, sms, parts, s);
    return bwd_long<DT, 1>(p, sms, parts, s);
}

}  // namespace

cudaError_t launch_ln_fwd(const LnFwdParams& p, int dtype, bool vector, int sms, cudaStream_t s) {
    switch (dtype) {
        case F32: return fwd_dt<F32>(p, vector, sms, s);
        case F16: return fwd_dt<F16>(p, vector, sms, s);
        default: return fwd_dt<BF16>(p, vector, sms, s);
    }
}

cudaError_t launch_ln_bwd(const LnBwdParams& p, int dtype, bool vector, int sms, int* parts, cudaStream_t s) {
    switch (dtype) {
        case F32: return bwd_dt<F32>(p, vector, sms, parts, s);
        case F16: return bwd_dt<F16>(p, vector, sms, parts, s);
        default: return bwd_dt<BF16>(p, vector, sms, parts, s);
    }
}

cudaError_t launch_ln_wgrad(const LnWgradParams& p, cudaStream_t s) {
    return launch_pdl(ln_wgrad_kernel, p, dim3((unsigned)((p.cols + 31) / 32), 2), 32 * WG_SLICES, 0, s);
}

}  // namespace tb
