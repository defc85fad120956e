// tb_layernorm.cu -- layer norm over the last axis, forward.
//
// Row by row (n = cols):
//     h = residual ? rnd(x + residual) : x
//     mean = sum(h) / n,  var = sum((h - mean)^2) / n,  rstd = 1 / sqrt(var + eps)
//     y = rnd((h - mean) * rstd * gamma + beta)
// Sums and statistics are fp32; every output is rounded once.
//
// A row is held by TPR threads (fewer than a warp where rows are short), CPT
// chunks each, in registers and in its
// storage type: one read of the row serves the mean, the squares about it (a
// second pass over registers, so an outlier or a large offset costs no
// precision) and the output.  The next row's chunks are requested before the
// current row is reduced.
//
// Bound by memory: 16384 x 4096 bf16 with residual moves 537 MB in 82.5 us (6.5
// TB/s, 97 % of the measured copy rate), 65536 x 512 bf16 134 MB in 25.5 us (79
// %, where ten shuffles a row per warp count), 262144 x 64 bf16 67 MB in 14.3 us
// (73 %).  One row of 4096 takes 9 us, all of it the call.
// Rows of single elements (no 16-byte words) are bound by this kernel, which
// moves an element a lane and instruction, not by memory: 65536 x 515 bf16 takes
// 71 us, 29 %, 13419 x 5001 107 us, 37 %, in f32 122 us, 66 %.
// Registers run out, and spill, with 16 single elements a thread (256 threads
// 112 to 936 bytes, 1024 threads 308 to 1068), with the 1024-thread forms of 16-bit
// rows (40 to 256 bytes) and of f32 rows past 8192 columns (296, with residual
// 656), and a little (16 to 72 bytes) with residual in 16-bit rows of up to 2048
// columns: 4096 x 16384 f32 takes 105 us, 76 %, with residual 241, 67 %.
#include "tb_layernorm.cuh"

namespace tb {
namespace {

// CTAs per SM the forward kernel is compiled for: 768 threads of 85 registers.
// (16384 x 4096 bf16 with residual, f32 weights: 1024 / 768 / 512 threads take
// 93.7 / 82.4 / 89.2 us; the first spill, the last have too few loads in flight.)
__host__ __device__ constexpr int ln_fwd_ctas(int tpr) { return tpr >= 1024 ? 1 : 768 / ln_block(tpr); }

template <int DT, int VEC, int TPR, int CPT, bool RES>
__global__ void __launch_bounds__(ln_block(TPR), ln_fwd_ctas(TPR)) ln_fwd_kernel(const __grid_constant__ LnFwdParams p) {
    using W = typename Word<VEC * elem_size(DT)>::T;
    using L = Lanes<VEC>;
    using T = typename L::T;
    constexpr int BLOCK = ln_block(TPR);
    constexpr int RPC = BLOCK / TPR;        // rows per CTA
    constexpr bool KEEP = CPT * VEC <= 16;  // the weights stay in registers
    __shared__ float s_a[BLOCK / 32], s_b[BLOCK / 32];
    const int t = threadIdx.x % TPR, rl = threadIdx.x / TPR;
    const int64_t step = (int64_t)gridDim.x * RPC;
    int64_t row = (int64_t)blockIdx.x * RPC + rl;
    // the rows of one warp stay together: its first row ends the loop for all
    int64_t lead = TPR < 32 ? row - rl % (TPR < 32 ? 32 / TPR : 1) : row;
    const int chunks = (int)(p.cols / VEC);
    const float n = (float)p.cols;
    const int64_t row_bytes = p.cols * elem_size(DT);
    grid_wait();

    auto fetch = [&](const void* base, int64_t r, int64_t ld, W (&v)[CPT]) {
        const char* const at = reinterpret_cast<const char*>(base) + r * ld * elem_size(DT);
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
            const int c = t + k * TPR;
            const W* const src = reinterpret_cast<const W*>(at) + c;
            if (c < chunks && in_bounds(src, sizeof(W), at, row_bytes, p.status)) v[k] = __ldcs(src);
        }
    };
    W nx[CPT], nr[RES ? CPT : 1];
    if (row < p.rows) {
        fetch(p.x, row, p.x_ld, nx);
        if constexpr (RES) fetch(p.residual, row, p.r_ld, nr);
    }
    T g[KEEP ? CPT : 1][L::N], b[KEEP ? CPT : 1][L::N];
    if constexpr (KEEP) {
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
            const int c = t + k * TPR;
            if (c < chunks) {
                weight_lanes<VEC>(p.gamma, p.wdtype, (int64_t)c * VEC, 1.f, g[k]);
                weight_lanes<VEC>(p.beta, p.wdtype, (int64_t)c * VEC, 0.f, b[k]);
            }
        }
    }
    for (; lead < p.rows; lead += step, row += step) {
        const bool here = TPR >= 32 || row < p.rows;
        const int nchunk = here ? chunks : 0;
        W h[CPT];  // the row as stored
        T sum = L::splat(0.f);
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
            const int c = t + k * TPR;
            if (c < nchunk) {
                T f[L::N];
                h[k] = nx[k];
                to_lanes<DT, VEC>(h[k], f);
                if constexpr (RES) {
                    T r[L::N];
                    to_lanes<DT, VEC>(nr[k], r);
#pragma unroll
                    for (int q = 0; q < L::N; ++q) f[q] = vadd(f[q], r[q]);
                    h[k] = from_lanes<DT, VEC>(f);  // the sum as stored is what is normalised
                    to_lanes<DT, VEC>(h[k], f);
                    char* const at = reinterpret_cast<char*>(p.total) + row * p.t_ld * elem_size(DT);
                    W* const dst = reinterpret_cast<W*>(at) + c;
                    if (in_bounds(dst, sizeof(W), at, row_bytes, p.status)) *dst = h[k];
                }
#pragma unroll
                for (int q = 0; q < L::N; ++q) sum = vadd(sum, f[q]);
            }
        }
        if (row + step < p.rows) {
            fetch(p.x, row + step, p.x_ld, nx);
            if constexpr (RES) fetch(p.residual, row + step, p.r_ld, nr);
        }
        const float mean = row_sum<TPR, BLOCK>(vsum(sum), s_a, rl) / n;
        const T mean2 = L::splat(mean);
        T m2 = L::splat(0.f);
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
            if (t + k * TPR < nchunk) {
                T f[L::N];
                to_lanes<DT, VEC>(h[k], f);
#pragma unroll
                for (int q = 0; q < L::N; ++q) {
                    const T d = vsub(f[q], mean2);
                    m2 = vfma(d, d, m2);
                }
            }
        }
        const float rstd = 1.0f / sqrtf(row_sum<TPR, BLOCK>(vsum(m2), s_b, rl) / n + p.eps);
        if (t == 0 && here) {
            if (p.mean) p.mean[row] = mean;
            if (p.rstd) p.rstd[row] = rstd;
        }
        const T rstd2 = L::splat(rstd);
        char* const at = reinterpret_cast<char*>(p.y) + row * p.y_ld * elem_size(DT);
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
            const int c = t + k * TPR;
            if (c < nchunk) {
                T f[L::N];
                to_lanes<DT, VEC>(h[k], f);
                if constexpr (KEEP) {
#pragma unroll
                    for (int q = 0; q < L::N; ++q) f[q] = vfma(vsub(f[q], mean2), vmul(rstd2, g[k][q]), b[k][q]);
                } else {
                    T gv[L::N], bv[L::N];
                    weight_lanes<VEC>(p.gamma, p.wdtype, (int64_t)c * VEC, 1.f, gv);
                    weight_lanes<VEC>(p.beta, p.wdtype, (int64_t)c * VEC, 0.f, bv);
#pragma unroll
                    for (int q = 0; q < L::N; ++q) f[q] = vfma(vsub(f[q], mean2), vmul(rstd2, gv[q]), bv[q]);
                }
                W* const dst = reinterpret_cast<W*>(at) + c;
                if (in_bounds(dst, sizeof(W), at, row_bytes, p.status)) *dst = from_lanes<DT, VEC>(f);
            }
        }
    }
}

// Rows too long for registers: one CTA per row, which it reads three times
// (sum, squares about the mean, output; the second and third time mostly
// from L2).  Each thread reads back only what it wrote itself.
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
        const float mean = row_sum<LONG_BLOCK, LONG_BLOCK>(sum, s_a, 0) / n;
        float m2 = 0.f;
        for (int64_t c = threadIdx.x; c < nchunk; c += LONG_BLOCK) {
            float f[VEC];
            unpack<DT, VEC>(h[c], f);
#pragma unroll
            for (int q = 0; q < VEC; ++q) m2 = fmaf(f[q] - mean, f[q] - mean, m2);
        }
        const float rstd = 1.0f / sqrtf(row_sum<LONG_BLOCK, LONG_BLOCK>(m2, s_b, 0) / n + p.eps);
        if (threadIdx.x == 0) {
            if (p.mean) p.mean[row] = mean;
            if (p.rstd) p.rstd[row] = rstd;
        }
        W* const y = reinterpret_cast<W*>(reinterpret_cast<char*>(p.y) + row * p.y_ld * elem_size(DT));
        for (int64_t c = threadIdx.x; c < nchunk; c += LONG_BLOCK) {
            float f[VEC], gv[VEC], bv[VEC];
            unpack<DT, VEC>(h[c], f);
            weights_at<VEC>(p.gamma, p.wdtype, c * VEC, 1.f, gv);
            weights_at<VEC>(p.beta, p.wdtype, c * VEC, 0.f, bv);
#pragma unroll
            for (int q = 0; q < VEC; ++q) f[q] = fmaf((f[q] - mean) * rstd, gv[q], bv[q]);
            y[c] = pack<DT, VEC>(f);
        }
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
        // (a warp takes several short rows, two words a thread: 262144 x 64 / 128 bf16
        // 14.3 / 25.7 us, with a word a thread 15.5 / 29.3, a warp to a row 52.8 / 53.3;
        // 131072 x 256 25.6 against 28.2)
        if (n <= 4) return fwd_launch<DT, V, 4, 1>(p, sms, s);
        if (n <= 8) return fwd_launch<DT, V, 4, 2>(p, sms, s);
        if (n <= 16) return fwd_launch<DT, V, 8, 2>(p, sms, s);
        if (n <= 32) return fwd_launch<DT, V, 16, 2>(p, sms, s);
        if (n <= 64) return fwd_launch<DT, V, 32, 2>(p, sms, s);
        if (n <= 128) return fwd_launch<DT, V, 64, 2>(p, sms, s);
        if (n <= 256) return fwd_launch<DT, V, 128, 2>(p, sms, s);
        if (n <= 512) return fwd_launch<DT, V, 256, 2>(p, sms, s);
        if (n <= 1024) return fwd_launch<DT, V, 512, 2>(p, sms, s);
        if (n <= 2048) return fwd_launch<DT, V, 1024, 2>(p, sms, s);
        if (n <= 4096) return fwd_launch<DT, V, 1024, 4>(p, sms, s);
        return fwd_long<DT, V>(p, sms, s);
    }
    // (16 columns a thread from 2049 on: with 8, bf16 rows of 4095 / 5001 / 8191
    // took 105 / 158 / 103 us instead of 76 / 108 / 78, and with 16 below, rows of
    // 515 / 2047 took 77 / 79 us instead of 72 / 77; 67 M elements, at most 65536 rows)
    // (short rows: several to a warp; one to a warp took 64.6 us where 262144 x 63 bf16 takes 24.0)
    if (p.cols <= 64) return fwd_launch<DT, 1, 8, 8>(p, sms, s);
    if (p.cols <= 128) return fwd_launch<DT, 1, 16, 8>(p, sms, s);
    if (p.cols <= 256) return fwd_launch<DT, 1, 32, 8>(p, sms, s);
    if (p.cols <= 512) return fwd_launch<DT, 1, 64, 8>(p, sms, s);
    if (p.cols <= 1024) return fwd_launch<DT, 1, 128, 8>(p, sms, s);
    if (p.cols <= 2048) return fwd_launch<DT, 1, 256, 8>(p, sms, s);
    if (p.cols <= 4096) return fwd_launch<DT, 1, 256, 16>(p, sms, s);
    if (p.cols <= 8192) return fwd_launch<DT, 1, 512, 16>(p, sms, s);
    if (p.cols <= 16384) return fwd_launch<DT, 1, 1024, 16>(p, sms, s);
    return fwd_long<DT, 1>(p, sms, s);
}

}  // namespace

cudaError_t launch_ln_fwd(const LnFwdParams& p, int dtype, bool vector, int sms, cudaStream_t s) {
    switch (dtype) {
        case F32: return fwd_dt<F32>(p, vector, sms, s);
        case F16: return fwd_dt<F16>(p, vector, sms, s);
        default: return fwd_dt<BF16>(p, vector, sms, s);
    }
}

}  // namespace tb
