// tb_layernorm_bwd.cu -- the gradients of the layer norm.
//
// With xhat = (h - mean) * rstd and g = dy * gamma, row by row (n = cols):
//     dx = rnd(rstd * (g - sum(g) / n - xhat * sum(g * xhat) / n) + dtotal)
//     dgamma = sum over rows of dy * xhat,  dbeta = sum over rows of dy
// All sums are fp32; every output is rounded once.
#include "tb_layernorm.cuh"

namespace tb {
namespace {

// CTAs per SM the backward kernel is compiled for, and so the number of
// partial weight gradients (one per CTA): 512 threads of 128 registers.
#ifndef TB_LN_BWD_THREADS
#define TB_LN_BWD_THREADS 512
#endif
__host__ __device__ constexpr int ln_bwd_ctas(int tpr) { return tpr >= 512 ? 1 : TB_LN_BWD_THREADS / ln_block(tpr); }

// Each thread keeps the weight gradients of its own columns over all rows
// its CTA takes; the CTA's sums go to workspace[part][2][cols] (dgamma, then
// dbeta), which ln_wgrad_kernel adds up in part order: no atomics, the same
// bits every time.
template <int DT, int VEC, int TPR, int CPT, bool TOT, bool WIDE>
__global__ void __launch_bounds__(ln_block(TPR), ln_bwd_ctas(TPR)) ln_bwd_kernel(const __grid_constant__ LnBwdParams p) {
    using W = typename Word<VEC * elem_size(DT)>::T;
    using L = Lanes<VEC>;
    using T = typename L::T;
    constexpr int BLOCK = ln_block(TPR);
    constexpr int RPC = BLOCK / TPR;
    constexpr int WPR = TPR / 32;
    __shared__ float2 s_sum[2][BLOCK / 32];
    extern __shared__ float s_acc[];  // RPC > 1: [2][cols]
    const int t = threadIdx.x % TPR, rl = threadIdx.x / TPR;
    const int64_t step = (int64_t)gridDim.x * RPC;
    const int nchunk = (int)(p.cols / VEC);
    const float n = (float)p.cols;
    const int64_t row_bytes = p.cols * elem_size(DT);
    grid_wait();

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
    Weights<DT, VEC, WIDE> g[CPT];
    T dg[CPT][L::N], db[CPT][L::N];
#pragma unroll
    for (int k = 0; k < CPT; ++k) {
        const int c = t + k * TPR;
        if (c < nchunk) g[k].load(p.gamma, p.wdtype, (int64_t)c * VEC, 1.f);
#pragma unroll
        for (int q = 0; q < L::N; ++q) dg[k][q] = db[k][q] = L::splat(0.f);
    }
    int phase = 0;
    for (; row < p.rows; row += step) {
        const T mean = L::splat(nmean), rstd = L::splat(nrstd);
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
        T a1 = L::splat(0.f), a2 = L::splat(0.f);
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
            if (t + k * TPR < nchunk) {
                T d[L::N], x[L::N], gv[L::N];
                to_lanes<DT, VEC>(cd[k], d);
                to_lanes<DT, VEC>(cx[k], x);
                g[k].get(gv);
#pragma unroll
                for (int q = 0; q < L::N; ++q) {
                    const T xh = vmul(vsub(x[q], mean), rstd);
                    const T gd = vmul(d[q], gv[q]);
                    a1 = vadd(a1, gd);
                    a2 = vfma(gd, xh, a2);
                    dg[k][q] = vfma(d[q], xh, dg[k][q]);
                    db[k][q] = vadd(db[k][q], d[q]);
                }
            }
        }
        float s1 = warp_sum(vsum(a1)), s2 = warp_sum(vsum(a2));
        if constexpr (TPR > 32) {
            // the slots alternate, so one barrier per row suffices
            if ((threadIdx.x & 31) == 0) s_sum[phase][threadIdx.x >> 5] = make_float2(s1, s2);
            row_barrier<TPR, BLOCK>(rl);
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
        if (p.dx != nullptr) {
            const T c1 = L::splat(s1 / n), c2 = L::splat(-s2 / n);
            char* const at = reinterpret_cast<char*>(p.dx) + row * p.dx_ld * elem_size(DT);
#pragma unroll
            for (int k = 0; k < CPT; ++k) {
                const int c = t + k * TPR;
                if (c < nchunk) {
                    T d[L::N], x[L::N], gv[L::N];
                    to_lanes<DT, VEC>(cd[k], d);
                    to_lanes<DT, VEC>(cx[k], x);
                    g[k].get(gv);
#pragma unroll
                    for (int q = 0; q < L::N; ++q) {
                        const T xh = vmul(vsub(x[q], mean), rstd);
                        d[q] = vmul(rstd, vfma(xh, c2, vsub(vmul(d[q], gv[q]), c1)));
                    }
                    if constexpr (TOT) {
                        T tt[L::N];
                        to_lanes<DT, VEC>(ct[k], tt);
#pragma unroll
                        for (int q = 0; q < L::N; ++q) d[q] = vadd(d[q], tt[q]);
                    }
                    W* const dst = reinterpret_cast<W*>(at) + c;
                    if (in_bounds(dst, sizeof(W), at, row_bytes, p.status)) *dst = from_lanes<DT, VEC>(d);
                }
            }
        }
    }

    float fg[CPT][VEC], fb[CPT][VEC];
#pragma unroll
    for (int k = 0; k < CPT; ++k) {
        if constexpr (VEC == 1) {
            fg[k][0] = dg[k][0];
            fb[k][0] = db[k][0];
        } else {
#pragma unroll
            for (int q = 0; q < VEC / 2; ++q) {
                halves(dg[k][q], fg[k][2 * q], fg[k][2 * q + 1]);
                halves(db[k][q], fb[k][2 * q], fb[k][2 * q + 1]);
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
                            const float vg = fg[k][q] + (w ? a[0] : 0.f);
                            const float vb = fb[k][q] + (w ? a[p.cols] : 0.f);
                            a[0] = vg;
                            a[p.cols] = vb;
                        }
                    }
                }
            }
            __syncthreads();
        }
        float* const out = p.workspace + (int64_t)blockIdx.x * 2 * p.cols;
        for (int64_t i = threadIdx.x; i < 2 * p.cols; i += ln_block(TPR)) out[i] = s_acc[i];
    } else {
        float* const out = p.workspace + (int64_t)blockIdx.x * 2 * p.cols;
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
            const int c = t + k * TPR;
            if (c < nchunk) {
#pragma unroll
                for (int q = 0; q < VEC; ++q) {
                    out[c * VEC + q] = fg[k][q];
                    out[p.cols + c * VEC + q] = fb[k][q];
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
    const float n = (float)p.cols;
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
        const float c1 = row_sum<LONG_BLOCK, LONG_BLOCK>(s1, s_a, 0) / n, c2 = row_sum<LONG_BLOCK, LONG_BLOCK>(s2, s_b, 0) / n;
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
// columns of one of the two; its 32 warps sum every 32nd part, and warp 0
// adds the 32 in order.
constexpr int WG_SLICES = 32;

__global__ void __launch_bounds__(32 * WG_SLICES) ln_wgrad_kernel(const __grid_constant__ LnWgradParams p) {
    __shared__ float s[WG_SLICES][33];
    const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane;
    const int which = blockIdx.y;
    void* const out = which ? p.dbeta : p.dgamma;
    grid_wait();
    if (out == nullptr) return;
    float v = 0.f;
    if (c < p.cols) {
        const float* const at = p.workspace + which * p.cols + c;
        constexpr int PER = TB_LN_PARTS / WG_SLICES;  // every load is issued before the first is used
        float part[PER];
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const int i = slice + k * WG_SLICES;
            part[k] = i < p.parts ? at[(int64_t)i * 2 * p.cols] : 0.f;
        }
#pragma unroll
        for (int k = 0; k < PER; ++k) v += part[k];
    }
    s[slice][lane] = v;
    __syncthreads();
    // a warp per column: the 32 slices, pairwise
    v = warp_sum(s[lane][slice]);
    const int64_t col = (int64_t)blockIdx.x * 32 + slice;
    if (lane == 0 && col < p.cols) store_weight(out, p.wdtype, col, v);
}

template <int DT, int VEC, int TPR, int CPT, bool TOT>
void (*bwd_fn(bool wide))(const LnBwdParams) {
    if constexpr (DT != F32 && VEC > 1) {
        if (!wide) return ln_bwd_kernel<DT, VEC, TPR, CPT, TOT, false>;
    }
    return ln_bwd_kernel<DT, VEC, TPR, CPT, TOT, true>;
}

template <int DT, int VEC, int TPR, int CPT>
cudaError_t bwd_launch(const LnBwdParams& p, int sms, int* parts, cudaStream_t s) {
    constexpr int rpc = ln_block(TPR) / TPR;
    const int64_t want = (p.rows + rpc - 1) / rpc;
    int64_t grid = (int64_t)sms * ln_bwd_ctas(TPR);
    if (grid > TB_LN_PARTS) grid = TB_LN_PARTS;
    if (grid > want) grid = want;
    *parts = (int)grid;
    const size_t smem = rpc > 1 && p.workspace != nullptr ? (size_t)p.cols * 8 : 0;
    const bool wide = p.wdtype == F32;
    return launch_pdl(p.dtotal ? bwd_fn<DT, VEC, TPR, CPT, true>(wide) : bwd_fn<DT, VEC, TPR, CPT, false>(wide), p,
                      dim3((unsigned)grid), ln_block(TPR), smem, s);
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
