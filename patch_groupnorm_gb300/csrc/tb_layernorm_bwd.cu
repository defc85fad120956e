// tb_layernorm_bwd.cu -- the gradients of the layer norm.
//
// With xhat = (h - mean) * rstd and g = dy * gamma, row by row (n = cols):
//     dx = rnd(rstd * (g - sum(g) / n - xhat * sum(g * xhat) / n) + dtotal)
//     dgamma = sum over rows of dy * xhat,  dbeta = sum over rows of dy
// All sums are fp32; every output is rounded once.
#include "tb_layernorm.cuh"

namespace tb {
namespace {

// Ring stages per row group at most.
constexpr int LN_BWD_MAX_STAGES = 8;
// Shared memory of an SM that the rings of its CTA share.  A warp's own row
// (TPR 32) is refilled as soon as it is done with it; wider rows only past the
// next row's barrier, so they want a stage more.  Measured (bf16, us): 65536 x
// 512 rows with 64 / 80 / 96 / 144 / 216 KB 36.7 / 36.7 / 35.6 / 35.4 / 37.4;
// 16384 x 4096 with dtotal and 112 / 216 KB 111 / 92 (two CTAs per SM).
constexpr int64_t ln_bwd_room(int tpr) { return (tpr == 32 ? 144 : 216) * 1024; }

// Threads per CTA: a row's threads, at least 16 warps.  One CTA per SM: 512
// threads of 128 registers, and one partial weight gradient each.
#ifndef TB_LN_BWD_BLOCK
#define TB_LN_BWD_BLOCK 512
#endif
__host__ __device__ constexpr int bwd_block(int tpr) { return tpr < TB_LN_BWD_BLOCK ? TB_LN_BWD_BLOCK : tpr; }
__host__ __device__ constexpr int bwd_ctas(int tpr) { return 512 / bwd_block(tpr) > 1 ? 512 / bwd_block(tpr) : 1; }

// Each thread keeps the weight gradients of its own columns over all rows
// its CTA takes; the CTA's sums go to workspace[part][2][cols] (dgamma, then
// dbeta), which ln_wgrad_kernel adds up in part order: no atomics, the same
// bits every time.
//
// 16-byte chunks (RING): every row group has p.stages buffers in shared
// memory, each one row of dy, x and dtotal.  The group's first thread copies
// whole rows into them (bulk copies that complete on the stage's mbarrier),
// up to p.stages rows ahead; the threads read the row twice from shared
// memory, once for the sums and once for dx, which leaves the registers to
// the weight gradients.  Single elements: the next row waits in registers.
template <int DT, int VEC, int TPR, int CPT, bool TOT>
__global__ void __launch_bounds__(bwd_block(TPR), bwd_ctas(TPR))
    ln_bwd_kernel(const __grid_constant__ LnBwdParams p) {
    using W = typename Word<VEC * elem_size(DT)>::T;
    using L = Lanes<VEC>;
    using T = typename L::T;
    constexpr int BLOCK = bwd_block(TPR);
    constexpr int RPC = BLOCK / TPR;
    constexpr int WPR = TPR / 32;
    constexpr bool RING = VEC > 1;
    constexpr int NT = TOT ? 3 : 2;
    constexpr int REGS = RING ? 1 : CPT;  // chunks of the next row in registers
    __shared__ float2 s_sum[2][BLOCK / 32];
    __shared__ __align__(8) unsigned long long s_bar[RING ? RPC * LN_BWD_MAX_STAGES : 1];
    extern __shared__ __align__(16) unsigned char s_rows[];  // RING: [RPC][stages][NT][row]; then [2][cols] fp32
    const int t = threadIdx.x % TPR, rl = threadIdx.x / TPR;
    const int64_t step = (int64_t)gridDim.x * RPC;
    const int nchunk = (int)(p.cols / VEC);
    const float inv_n = 1.0f / (float)p.cols;
    const uint32_t row_bytes = (uint32_t)p.cols * elem_size(DT);
    const int stages = p.stages;
    const uint32_t ring = RING ? smem_addr(s_rows) + (uint32_t)(rl * stages * NT) * row_bytes : 0u;
    const uint32_t bars = smem_addr(s_bar) + (uint32_t)(rl * LN_BWD_MAX_STAGES) * 8u;
    if constexpr (RING) {
        if (t == 0) {
            for (int k = 0; k < stages; ++k) bar_init(bars + k * 8u, 1);
            bar_init_fence();
        }
        __syncthreads();
    }
    grid_wait();

    auto row_at = [&](const void* base, int64_t r, int64_t ld) {
        return reinterpret_cast<const char*>(base) + r * ld * elem_size(DT);
    };
    auto fetch = [&](const void* base, int64_t r, int64_t ld, W (&v)[REGS]) {
        const char* const at = row_at(base, r, ld);
#pragma unroll
        for (int k = 0; k < REGS; ++k) {
            const int c = t + k * TPR;
            const W* const src = reinterpret_cast<const W*>(at) + c;
            if (c < nchunk && in_bounds(src, sizeof(W), at, row_bytes, p.status)) v[k] = __ldcs(src);
        }
    };
    // copies the row group's next row into stage `st` (one thread of the group)
    int64_t ahead = (int64_t)blockIdx.x * RPC + rl;  // that row
    auto issue = [&](int st) {
        const uint32_t dst = ring + (uint32_t)(st * NT) * row_bytes, bar = bars + st * 8u;
        bar_expect(bar, NT * row_bytes);
        bulk_load(dst, row_at(p.dy, ahead, p.dy_ld), row_bytes, bar);
        bulk_load(dst + row_bytes, row_at(p.x, ahead, p.x_ld), row_bytes, bar);
        if constexpr (TOT) bulk_load(dst + 2 * row_bytes, row_at(p.dtotal, ahead, p.dt_ld), row_bytes, bar);
        ahead += step;
    };
    W nd[REGS], nx[REGS], nt[REGS];
    // the statistics of the row group's next 32 rows, one row per lane, and of
    // the 32 after them
    const int lane = threadIdx.x & 31;
    float mean_now, rstd_now, mean_next, rstd_next;
    auto stats = [&](int64_t r, float& m, float& rs) {
        r += lane * step;
        m = rs = 0.f;
        if (r < p.rows) {
            m = p.mean[r];
            rs = p.rstd[r];
        }
    };
    int64_t row = (int64_t)blockIdx.x * RPC + rl;
    if (row < p.rows) {
        if constexpr (RING) {
            if (t == 0)
                for (int k = 0; k < stages && ahead < p.rows; ++k) issue(k);
        } else {
            fetch(p.dy, row, p.dy_ld, nd);
            fetch(p.x, row, p.x_ld, nx);
            if constexpr (TOT) fetch(p.dtotal, row, p.dt_ld, nt);
        }
    }
    stats(row, mean_now, rstd_now);
    stats(row + 32 * step, mean_next, rstd_next);
    T g[CPT][L::N], dg[CPT][L::N], db[CPT][L::N];
#pragma unroll
    for (int k = 0; k < CPT; ++k) {
        const int c = t + k * TPR;
        if (c < nchunk) weight_lanes<VEC>(p.gamma, p.wdtype, (int64_t)c * VEC, 1.f, g[k]);
#pragma unroll
        for (int q = 0; q < L::N; ++q) dg[k][q] = db[k][q] = L::splat(0.f);
    }
    int phase = 0, st = 0, turn = 0;
    uint32_t parity = 0;
    bool late = false;  // a copy did not arrive: nothing more is written
    for (; row < p.rows; row += step) {
        if (turn == 32) {
            turn = 0;
            mean_now = mean_next;
            rstd_now = rstd_next;
            stats(row + 32 * step, mean_next, rstd_next);
        }
        const float mean = __shfl_sync(0xffffffffu, mean_now, turn), rstd = __shfl_sync(0xffffffffu, rstd_now, turn);
        ++turn;
        const T mean2 = L::splat(mean), rstd2 = L::splat(rstd);
        W cd[REGS], cx[REGS], ct[REGS];
        if constexpr (!RING) {
#pragma unroll
            for (int k = 0; k < REGS; ++k) {
                cd[k] = nd[k];
                cx[k] = nx[k];
                if constexpr (TOT) ct[k] = nt[k];
            }
        }
        if (!RING && row + step < p.rows) {
            fetch(p.dy, row + step, p.dy_ld, nd);
            fetch(p.x, row + step, p.x_ld, nx);
            if constexpr (TOT) fetch(p.dtotal, row + step, p.dt_ld, nt);
        }
        const uint32_t at = ring + (uint32_t)(st * NT) * row_bytes + t * 16u;
        if constexpr (RING) {
            if (!late && !bar_wait(bars + st * 8u, parity, p.status)) {
                late = true;
                // no new copies from here on; those in flight must land (or
                // run out their own wait) before the CTA's memory is given up
                if (t == 0)
                    for (int64_t r = row, s = st; r < ahead; r += step) {
                        bar_wait(bars + (uint32_t)s * 8u, s >= st ? parity : parity ^ 1u, p.status);
                        if (++s == stages) s = 0;
                    }
            }
        }
        // chunk k of the row of tensor `which`
        auto chunk = [&](int which, const W (&regs)[REGS], int k, T (&f)[L::N]) {
            if constexpr (RING) {
                to_lanes<DT, VEC>(smem_load<W>(at + (uint32_t)which * row_bytes + (uint32_t)(k * TPR) * 16u), f);
            } else {
                to_lanes<DT, VEC>(regs[k], f);
            }
        };
        T d[CPT][L::N], x[CPT][L::N];
        T a1 = L::splat(0.f), a2 = L::splat(0.f);
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
            if (t + k * TPR < nchunk) {
                chunk(0, cd, k, d[k]);
                chunk(1, cx, k, x[k]);
#pragma unroll
                for (int q = 0; q < L::N; ++q) {
                    db[k][q] = vadd(db[k][q], d[k][q]);
                    x[k][q] = vsub(x[k][q], mean2);
                    d[k][q] = vmul(d[k][q], rstd2);
                    const T gd = vmul(d[k][q], g[k][q]);
                    a1 = vadd(a1, gd);
                    a2 = vfma(gd, x[k][q], a2);
                    dg[k][q] = vfma(d[k][q], x[k][q], dg[k][q]);
                }
            }
        }
        float s1 = warp_sum(vsum(a1)), s2 = warp_sum(vsum(a2));
        if constexpr (TPR > 32) {
            // the slots alternate, so one barrier per row suffices
            if ((threadIdx.x & 31) == 0) s_sum[phase][threadIdx.x >> 5] = make_float2(s1, s2);
            row_barrier<TPR, BLOCK>(rl);
            if constexpr (RING) {
                // past the barrier nobody reads the stage before this one
                if (t == 0 && !late && ahead < p.rows && ahead < row + (int64_t)stages * step)
                    issue(st == 0 ? stages - 1 : st - 1);
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
        if (p.dx != nullptr) {
            // s1 = rstd * sum(g), s2 = sum(g * xhat): with u = x - mean and
            // v = dy * rstd, dx = v * gamma - u * rstd^2 * s2 / n - s1 / n
            const T ca = L::splat(-rstd * rstd * (s2 * inv_n)), cb = L::splat(-(s1 * inv_n));
            char* const out = reinterpret_cast<char*>(p.dx) + row * p.dx_ld * elem_size(DT);
#pragma unroll
            for (int k = 0; k < CPT; ++k) {
                const int c = t + k * TPR;
                if (c < nchunk) {
                    T o[L::N];
                    if constexpr (TOT) {
                        chunk(2, ct, k, o);
#pragma unroll
                        for (int q = 0; q < L::N; ++q) o[q] = vadd(o[q], cb);
                    } else {
#pragma unroll
                        for (int q = 0; q < L::N; ++q) o[q] = cb;
                    }
#pragma unroll
                    for (int q = 0; q < L::N; ++q)
                        o[q] = vfma(d[k][q], g[k][q], vfma(x[k][q], ca, o[q]));
                    W* const dst = reinterpret_cast<W*>(out) + c;
                    if (!late && in_bounds(dst, sizeof(W), out, row_bytes, p.status)) *dst = from_lanes<DT, VEC>(o);
                }
            }
        }
        if constexpr (RING) {
            if constexpr (TPR == 32) {
                __syncwarp();
                if (t == 0 && !late && ahead < p.rows) issue(st);
            }
            if (++st == stages) {
                st = 0;
                parity ^= 1u;
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
    if (p.workspace == nullptr || late) return;
    float* const out = p.workspace + (int64_t)blockIdx.x * 2 * p.cols;
    if constexpr (RPC > 1) {
        // the CTA's row groups' sums meet in the ring's memory, each thread's
        // column k * VEC + q at [group][which][k * VEC + q][t], the rows four
        // words longer than TPR so that neighbouring columns are in different
        // banks; then every column is added up over the groups in order
        constexpr int PITCH = TPR + 4, N = CPT * VEC;
        float* const s_acc = reinterpret_cast<float*>(s_rows);
        __syncthreads();
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
#pragma unroll
            for (int q = 0; q < VEC; ++q) {
                s_acc[((rl * 2 + 0) * N + k * VEC + q) * PITCH + t] = fg[k][q];
                s_acc[((rl * 2 + 1) * N + k * VEC + q) * PITCH + t] = fb[k][q];
            }
        }
        __syncthreads();
        for (int i = threadIdx.x; i < 2 * (int)p.cols; i += BLOCK) {
            const int which = i >= (int)p.cols ? 1 : 0;
            const int col = i - which * (int)p.cols, c = col / VEC;
            const float* const at = s_acc + (which * N + c / TPR * VEC + col % VEC) * PITCH + c % TPR;
            float v = at[0];
#pragma unroll
            for (int w = 1; w < RPC; ++w) v += at[w * 2 * N * PITCH];
            out[i] = v;
        }
    } else {
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

template <int DT, int VEC, int TPR, int CPT>
cudaError_t bwd_launch(const LnBwdParams& p, int sms, int* parts, cudaStream_t s) {
    constexpr int rpc = bwd_block(TPR) / TPR;
    const int64_t want = (p.rows + rpc - 1) / rpc;
    int64_t grid = (int64_t)sms * bwd_ctas(TPR);
    if (grid > TB_LN_PARTS) grid = TB_LN_PARTS;
    if (grid > want) grid = want;
    *parts = (int)grid;
    LnBwdParams q = p;
    int64_t smem = rpc > 1 ? (int64_t)rpc * 2 * CPT * VEC * (TPR + 4) * 4 : 0;
    q.stages = 0;
    if (VEC > 1) {
        const int64_t stage = (int64_t)rpc * (p.dtotal ? 3 : 2) * p.cols * elem_size(DT);
        const int64_t room = ln_bwd_room(TPR) / bwd_ctas(TPR);
        const int64_t fit = room / stage;
        q.stages = (int)(fit < 2 ? 2 : fit > LN_BWD_MAX_STAGES ? LN_BWD_MAX_STAGES : fit);
        if (smem < q.stages * stage) smem = q.stages * stage;
    }
    void (*fn)(const LnBwdParams) =
        p.dtotal ? ln_bwd_kernel<DT, VEC, TPR, CPT, true> : ln_bwd_kernel<DT, VEC, TPR, CPT, false>;
    if (smem > 40 * 1024) {  // with the static shared memory, past the 48 KB default
        const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    return launch_pdl(fn, q, dim3((unsigned)grid), bwd_block(TPR), (size_t)smem, s);
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
