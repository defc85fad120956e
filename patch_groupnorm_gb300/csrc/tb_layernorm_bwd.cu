// tb_layernorm_bwd.cu -- the gradients of the layer norm.
//
// With xhat = (h - mean) * rstd and g = dy * gamma, row by row (n = cols):
//     dx = rnd(rstd * (g - sum(g) / n - xhat * sum(g * xhat) / n) + dtotal)
//     dgamma = sum over rows of dy * xhat,  dbeta = sum over rows of dy
// All sums are fp32; every output is rounded once.
//
// Bound by memory where rows are wide: 16384 x 4096 bf16 with dtotal moves 537 MB
// (and 10 MB of partial weight gradients) in 86.7 us, 93 % of the measured copy
// rate; 65536 x 512 bf16 201 MB in 34.9 us (86 %, half of all issue slots busy).
// One launch more adds up the CTAs' partial weight gradients.
// Farther from it: rows of 1025 to 2048 words (4096 x 16384 bf16 131 us, 46 %: one
// row a CTA at a time, read twice from shared memory, and 80 MB of partial
// weight gradients), single elements (65536 x 515 bf16 87 us, 35 %: an element
// a lane and instruction), and rows past 2048 words (4096 x 16384 f32 416 us, 29 %;
// 2048 x 40000 bf16 778 us, 9 %: the weight gradients are read and written in
// memory once a row, and nothing is copied ahead).
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
constexpr int64_t ln_bwd_room(int tpr) { return (tpr <= 32 ? 144 : 216) * 1024; }

// Threads per CTA, one CTA per SM: 128 registers a thread, and one partial
// weight gradient each.  Rows past 1024 words take four words a thread; 1024
// threads of 64 registers with two words each took 138 us where they take 133
// (4096 x 16384 bf16; 161 / 145 with dtotal, 185 / 131 at 12001 columns).
constexpr int BWD_BLOCK = 512;

// Each thread keeps the weight gradients of its own columns over all rows
// its CTA takes; the CTA's sums go to workspace[part][2][cols] (dgamma, then
// dbeta), which ln_wgrad_kernel adds up in part order: no atomics, the same
// bits every time.
//
// Every row group (TPR threads) has p.stages buffers in shared memory, each
// one row of dy, x and dtotal.  The group's first thread copies whole rows into
// them (bulk copies that complete on the stage's mbarrier), up to p.stages rows
// ahead, which leaves the registers to the weight gradients.
//
// WHOLE: rows start on 16-byte boundaries and are whole 16-byte words; thread t
// takes words t + k * TPR.  Otherwise the copies keep each row's offset from
// its boundary, the elements before the first and after the last boundary are
// copied one by one, and thread t takes the columns t + j * TPR, whose
// neighbours lie in neighbouring lanes.
template <int DT, int TPR, int CPT, bool TOT, bool WHOLE>
__global__ void __launch_bounds__(BWD_BLOCK, 1)
    ln_bwd_kernel(const __grid_constant__ LnBwdParams p) {
    constexpr int ES = elem_size(DT), VEC = 16 / ES;
    using E = typename Word<ES>::T;
    using L = Lanes<VEC>;
    using T = typename L::T;
    constexpr int BLOCK = BWD_BLOCK;
    constexpr int RPC = BLOCK / TPR;
    constexpr int WPR = TPR / 32;
    constexpr int HOLD = TPR < 32 ? TPR : 32;  // lanes of a warp in one row group
    constexpr int NT = TOT ? 3 : 2;
    constexpr bool LEAN = CPT > 2;  // no registers left for anything but the weight gradients
    __shared__ float2 s_sum[2][BLOCK / 32];
    __shared__ __align__(8) unsigned long long s_bar[RPC * LN_BWD_MAX_STAGES];
    extern __shared__ __align__(16) unsigned char s_rows[];  // [RPC][stages][NT][pitch]; then the CTA's sums
    const int t = threadIdx.x % TPR, rl = threadIdx.x / TPR, lane = threadIdx.x & 31;
    const int64_t step = (int64_t)gridDim.x * RPC;
    const int cols = (int)p.cols;
    const float inv_n = 1.0f / (float)p.cols;
    const uint32_t row_bytes = (uint32_t)cols * ES;
    const uint32_t pitch = WHOLE ? row_bytes : (row_bytes + 31u) & ~15u;
    const int stages = p.stages;
    const uint32_t ring = smem_addr(s_rows) + (uint32_t)(rl * stages * NT) * pitch;
    const uint32_t bars = smem_addr(s_bar) + (uint32_t)(rl * LN_BWD_MAX_STAGES) * 8u;
    if (t == 0) {
        for (int k = 0; k < stages; ++k) bar_init(bars + k * 8u, WHOLE ? 1 : 2);
        bar_init_fence();
    }
    __syncthreads();
    grid_wait();

    // column of lane element q of group k, and whether the thread has it
    auto column = [&](int k, int q) { return WHOLE ? (t + k * TPR) * VEC + q : (k * VEC + q) * TPR + t; };
    auto has = [&](int k) { return WHOLE ? t + k * TPR < cols / VEC : k * VEC * TPR + t < cols; };
    auto row_at = [&](const void* base, int64_t r, int64_t ld) {
        return reinterpret_cast<const char*>(base) + r * ld * ES;
    };
    // a row's offset from its 16-byte boundary
    auto shift_of = [&](const void* base, int64_t r, int64_t ld) {
        return WHOLE ? 0u : ((uint32_t)reinterpret_cast<uintptr_t>(base) + (uint32_t)r * (uint32_t)ld * ES) & 15u;
    };
    // copies the row group's next row into stage `st`: by the group's first
    // thread, or with single elements by its first warp
    int64_t ahead = (int64_t)blockIdx.x * RPC + rl;  // that row
    const bool issuer = WHOLE ? t == 0 : t < 32;
    auto issue = [&](int st) {
        const uint32_t dst = ring + (uint32_t)(st * NT) * pitch, bar = bars + st * 8u;
        if constexpr (WHOLE) {
            bar_expect(bar, NT * row_bytes);
            bulk_load(dst, row_at(p.dy, ahead, p.dy_ld), row_bytes, bar);
            bulk_load(dst + pitch, row_at(p.x, ahead, p.x_ld), row_bytes, bar);
            if constexpr (TOT) bulk_load(dst + 2 * pitch, row_at(p.dtotal, ahead, p.dt_ld), row_bytes, bar);
        } else {
            const char* from[3] = {row_at(p.dy, ahead, p.dy_ld), row_at(p.x, ahead, p.x_ld),
                                   TOT ? row_at(p.dtotal, ahead, p.dt_ld) : nullptr};
            uint32_t head[3], bulk[3], total = 0;
#pragma unroll
            for (int w = 0; w < NT; ++w) {
                const uint32_t shift = (uint32_t)reinterpret_cast<uintptr_t>(from[w]) & 15u;
                head[w] = min((16u - shift) & 15u, row_bytes);
                bulk[w] = (row_bytes - head[w]) & ~15u;
                total += bulk[w];
            }
            if (lane == 0) bar_expect(bar, total);
            __syncwarp();
#pragma unroll
            for (int w = 0; w < NT; ++w) {
                const uint32_t to = dst + (uint32_t)w * pitch + ((uint32_t)reinterpret_cast<uintptr_t>(from[w]) & 15u);
                if (lane == 0 && bulk[w] > 0) bulk_load(to + head[w], from[w] + head[w], bulk[w], bar);
                // lane k < 8: element k before the bulk copy; lane 8 + k: element k after it
                const uint32_t k = (lane & 7) * ES, tail = head[w] + bulk[w] + k;
                const uint32_t at = lane < 8 ? k : tail;
                if (lane < 8 ? k < head[w] : lane < 16 && tail < row_bytes) copy_element<ES>(to + at, from[w] + at);
            }
            __syncwarp();
            if (lane == 0) bar_arrive(bar);  // the elements copied one by one
        }
        ahead += step;
    };
    // the statistics of the row group's next HOLD rows, one row per lane, and
    // of the HOLD after them
    float mean_now, rstd_now, mean_next, rstd_next;
    auto stats = [&](int64_t r, float& m, float& rs) {
        r += (lane & (HOLD - 1)) * step;
        m = rs = 0.f;
        if (r < p.rows) {
            m = p.mean[r];
            rs = p.rstd[r];
        }
    };
    int64_t row = ahead;
    if (issuer)
        for (int k = 0; k < stages && ahead < p.rows; ++k) issue(k);
    stats(row, mean_now, rstd_now);
    stats(row + HOLD * step, mean_next, rstd_next);
    // gamma of the lanes of group k (zero past the row's end)
    auto gamma = [&](int k, T (&f)[L::N]) {
        if constexpr (WHOLE) {
            if (has(k)) weight_lanes<VEC>(p.gamma, p.wdtype, column(k, 0), 1.f, f);
        } else {
            float e[VEC];
#pragma unroll
            for (int q = 0; q < VEC; ++q) e[q] = column(k, q) < cols ? weight_at(p.gamma, p.wdtype, column(k, q), 1.f) : 0.f;
#pragma unroll
            for (int q = 0; q < L::N; ++q) f[q] = pair(e[2 * q], e[2 * q + 1]);
        }
    };
    T g[LEAN ? 1 : CPT][L::N], dg[CPT][L::N], db[CPT][L::N];
#pragma unroll
    for (int k = 0; k < CPT; ++k) {
        if constexpr (!LEAN) gamma(k, g[k]);
#pragma unroll
        for (int q = 0; q < L::N; ++q) dg[k][q] = db[k][q] = L::splat(0.f);
    }
    int phase = 0, st = 0, turn = 0;
    uint32_t parity = 0;
    bool late = false;  // a copy did not arrive: nothing more is written
    // (the row groups of one warp go round together, those without a row idle)
    const int64_t warp_row = TPR < 32 ? (int64_t)blockIdx.x * RPC + rl / (32 / HOLD) * (32 / HOLD) : row;
    for (int64_t any = warp_row; any < p.rows; any += step, row += step) {
        const bool here = TPR >= 32 || row < p.rows;
        if (turn == HOLD) {
            turn = 0;
            mean_now = mean_next;
            rstd_now = rstd_next;
            stats(row + HOLD * step, mean_next, rstd_next);
        }
        const float mean = __shfl_sync(0xffffffffu, mean_now, (lane & ~(HOLD - 1)) + turn);
        const float rstd = __shfl_sync(0xffffffffu, rstd_now, (lane & ~(HOLD - 1)) + turn);
        ++turn;
        const T mean2 = L::splat(mean), rstd2 = L::splat(rstd);
        const uint32_t at = ring + (uint32_t)(st * NT) * pitch;
        // (no new copies from there on)
        if (here && !late && !bar_wait(bars + st * 8u, parity, p.status)) late = true;
        if constexpr (!WHOLE) {
            late = __any_sync(0xffffffffu, late);  // a row group's first warp copies together
            // (by the last warp, since the first has the next row to copy: 13419 x 5001
            // bf16 198.3 us, by the copying lane 203.2, without a fence 197.3)
            if (t >= TPR - 32) bulk_fence();
        }
        // the lanes of group k of one tensor's row (zero past the row's end)
        auto lanes_of = [&](uint32_t from, int k, T (&f)[L::N]) {
            if constexpr (WHOLE) {
                to_lanes<DT, VEC>(smem_load<uint4>(from + (uint32_t)(t + k * TPR) * 16u), f);
            } else {
                float e[VEC];
#pragma unroll
                for (int q = 0; q < VEC; ++q) {
                    uint32_t bits = 0u;
                    if (column(k, q) < cols) bits = smem_element<ES>(from + (uint32_t)column(k, q) * ES);
                    e[q] = elem_to_f<DT>(bits);
                }
#pragma unroll
                for (int q = 0; q < L::N; ++q) f[q] = pair(e[2 * q], e[2 * q + 1]);
            }
        };
        const uint32_t at_dy = at + (here ? shift_of(p.dy, row, p.dy_ld) : 0u);
        const uint32_t at_x = at + pitch + (here ? shift_of(p.x, row, p.x_ld) : 0u);
        T d[LEAN ? 1 : CPT][L::N], x[LEAN ? 1 : CPT][L::N];
        T a1 = L::splat(0.f), a2 = L::splat(0.f);
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
            if (here && has(k)) {
                constexpr int ONE = LEAN ? 0 : 1;
                T gk[L::N];
                lanes_of(at_dy, k, d[k * ONE]);
                lanes_of(at_x, k, x[k * ONE]);
                if constexpr (LEAN) gamma(k, gk);
#pragma unroll
                for (int q = 0; q < L::N; ++q) {
                    T &dq = d[k * ONE][q], &xq = x[k * ONE][q];
                    db[k][q] = vadd(db[k][q], dq);
                    xq = vsub(xq, mean2);
                    dq = vmul(dq, rstd2);
                    T gd;
                    if constexpr (LEAN) gd = vmul(dq, gk[q]);
                    else gd = vmul(dq, g[k][q]);
                    a1 = vadd(a1, gd);
                    a2 = vfma(gd, xq, a2);
                    dg[k][q] = vfma(dq, xq, dg[k][q]);
                }
            }
        }
        float s1 = vsum(a1), s2 = vsum(a2);
#pragma unroll
        for (int o = HOLD / 2; o >= 1; o >>= 1) {
            s1 += __shfl_xor_sync(0xffffffffu, s1, o);
            s2 += __shfl_xor_sync(0xffffffffu, s2, o);
        }
        if constexpr (TPR > 32) {
            // the slots alternate, so one barrier per row suffices
            if (lane == 0) s_sum[phase][threadIdx.x >> 5] = make_float2(s1, s2);
            row_barrier<TPR, BLOCK>(rl);
            // past the barrier nobody reads the stage before this one
            if (issuer && !late && ahead < p.rows && ahead < row + (int64_t)stages * step)
                issue(st == 0 ? stages - 1 : st - 1);
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
        if (p.dx != nullptr && here) {
            // s1 = rstd * sum(g), s2 = sum(g * xhat): with u = x - mean and
            // v = dy * rstd, dx = v * gamma - u * rstd^2 * s2 / n - s1 / n
            const T ca = L::splat(-rstd * rstd * (s2 * inv_n)), cb = L::splat(-(s1 * inv_n));
            char* const out = reinterpret_cast<char*>(p.dx) + row * p.dx_ld * ES;
            const uint32_t at_t = TOT ? at + 2 * pitch + shift_of(p.dtotal, row, p.dt_ld) : 0u;
#pragma unroll
            for (int k = 0; k < CPT; ++k) {
                if (has(k)) {
                    constexpr int ONE = LEAN ? 0 : 1;
                    T o[L::N], gk[L::N];
                    if constexpr (TOT) {
                        lanes_of(at_t, k, o);
#pragma unroll
                        for (int q = 0; q < L::N; ++q) o[q] = vadd(o[q], cb);
                    } else {
#pragma unroll
                        for (int q = 0; q < L::N; ++q) o[q] = cb;
                    }
                    if constexpr (LEAN) {
                        lanes_of(at_dy, k, d[0]);
                        lanes_of(at_x, k, x[0]);
                        gamma(k, gk);
#pragma unroll
                        for (int q = 0; q < L::N; ++q) {
                            x[0][q] = vsub(x[0][q], mean2);
                            d[0][q] = vmul(d[0][q], rstd2);
                        }
                    }
#pragma unroll
                    for (int q = 0; q < L::N; ++q) {
                        if constexpr (LEAN) o[q] = vfma(d[0][q], gk[q], vfma(x[0][q], ca, o[q]));
                        else o[q] = vfma(d[k * ONE][q], g[k][q], vfma(x[k * ONE][q], ca, o[q]));
                    }
                    const uint4 w = from_lanes<DT, VEC>(o);
                    if constexpr (WHOLE) {
                        uint4* const dst = reinterpret_cast<uint4*>(out) + t + k * TPR;
                        if (!late && in_bounds(dst, 16, out, row_bytes, p.status)) *dst = w;
                    } else {
                        const uint32_t bits[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                        for (int q = 0; q < VEC; ++q) {
                            E* const dst = reinterpret_cast<E*>(out) + column(k, q);
                            if (column(k, q) < cols && !late && in_bounds(dst, ES, out, row_bytes, p.status)) {
                                if constexpr (ES == 4) *dst = bits[q];
                                else *dst = (E)(bits[q >> 1] >> (16 * (q & 1)));
                            }
                        }
                    }
                }
            }
        }
        if constexpr (TPR <= 32) {
            __syncwarp();
            if (issuer && !late && ahead < p.rows) issue(st);
        }
        if (++st == stages) {
            st = 0;
            parity ^= 1u;
        }
    }

    if (late && t == 0) {
        // copies in flight must land (or run out their own wait) before the
        // CTA's memory is given up: every stage's last one
        const int copied = (int)((ahead - ((int64_t)blockIdx.x * RPC + rl)) / step);
        for (int s = 0; s < stages && s < copied; ++s)
            bar_wait(bars + s * 8u, (uint32_t)((copied - 1 - s) / stages) & 1u, p.status);
    }
    if (p.workspace == nullptr || late) return;
    float* const out = p.workspace + (int64_t)blockIdx.x * 2 * p.cols;
    if constexpr (RPC > 1) {
        static_assert(WHOLE, "wide odd rows have a CTA each");
        // the CTA's row groups' sums meet in the ring's memory, a thread's
        // value k * VEC + q at [group][which][k * VEC + q][t], the rows four
        // words longer than TPR so that neighbouring columns are in different
        // banks; then every column is added up over the groups in order
        constexpr int PITCH = TPR + 4, N = CPT * VEC;
        float* const s_acc = reinterpret_cast<float*>(s_rows);
        __syncthreads();
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
#pragma unroll
            for (int q = 0; q < L::N; ++q) {
                float* const to = s_acc + (rl * 2 * N + k * VEC + 2 * q) * PITCH + t;
                halves(dg[k][q], to[0], to[PITCH]);
                halves(db[k][q], to[N * PITCH], to[(N + 1) * PITCH]);
            }
        }
        __syncthreads();
        for (int i = threadIdx.x; i < 2 * cols; i += BLOCK) {
            const int which = i >= cols ? 1 : 0;
            const int col = i - which * cols, c = col / VEC;
            const float* const at = s_acc + (which * N + c / TPR * VEC + col % VEC) * PITCH + c % TPR;
            float v = at[0];
#pragma unroll 8
            for (int w = 1; w < RPC; ++w) v += at[w * 2 * N * PITCH];
            out[i] = v;
        }
    } else {
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
#pragma unroll
            for (int q = 0; q < L::N; ++q) {
                float a, b, c, e;
                halves(dg[k][q], a, b);
                halves(db[k][q], c, e);
                const int c0 = column(k, 2 * q), c1 = column(k, 2 * q + 1);
                if (c0 < cols) {
                    out[c0] = a;
                    out[p.cols + c0] = c;
                }
                if (c1 < cols) {
                    out[c1] = b;
                    out[p.cols + c1] = e;
                }
            }
        }
    }
}

// Rows that cannot be copied in 16-byte words, up to ELEM_COLS columns: thread
// t takes the columns t + k * TPR, and the next row waits in registers.
// (Measured against the ring with single elements, us: bf16 65536 x 515 86 and
// 126, 32784 x 2047 108 and 138, 13419 x 5001 493 and 196.)
constexpr int64_t ELEM_COLS = 4096;

template <int DT, int TPR, int CPT, bool TOT>
__global__ void __launch_bounds__(BWD_BLOCK, 1)
    ln_bwd_elem_kernel(const __grid_constant__ LnBwdParams p) {
    using W = typename Word<elem_size(DT)>::T;
    constexpr int BLOCK = BWD_BLOCK;
    constexpr int RPC = BLOCK / TPR;
    constexpr int WPR = TPR / 32;
    constexpr int HOLD = TPR < 32 ? TPR : 32;  // lanes of a warp in one row group
    __shared__ float2 s_sum[2][BLOCK / 32];
    extern __shared__ __align__(16) unsigned char s_rows[];  // RPC > 1: the CTA's sums
    const int t = threadIdx.x % TPR, rl = threadIdx.x / TPR;
    const int64_t step = (int64_t)gridDim.x * RPC;
    const int cols = (int)p.cols;
    const float inv_n = 1.0f / (float)p.cols;
    const uint32_t row_bytes = (uint32_t)p.cols * elem_size(DT);
    grid_wait();

    auto row_at = [&](const void* base, int64_t r, int64_t ld) {
        return reinterpret_cast<const char*>(base) + r * ld * elem_size(DT);
    };
    auto fetch = [&](const void* base, int64_t r, int64_t ld, W (&v)[CPT]) {
        const char* const at = row_at(base, r, ld);
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
            const int c = t + k * TPR;
            const W* const src = reinterpret_cast<const W*>(at) + c;
            if (c < cols && in_bounds(src, sizeof(W), at, row_bytes, p.status)) v[k] = __ldcs(src);
        }
    };
    W nd[CPT], nx[CPT], nt[CPT];
    // the statistics of the row group's next HOLD rows, one row per lane, and of
    // the HOLD after them
    const int lane = threadIdx.x & 31;
    float mean_now, rstd_now, mean_next, rstd_next;
    auto stats = [&](int64_t r, float& m, float& rs) {
        r += lane % HOLD * step;
        m = rs = 0.f;
        if (r < p.rows) {
            m = p.mean[r];
            rs = p.rstd[r];
        }
    };
    int64_t row = (int64_t)blockIdx.x * RPC + rl;
    if (row < p.rows) {
        fetch(p.dy, row, p.dy_ld, nd);
        fetch(p.x, row, p.x_ld, nx);
        if constexpr (TOT) fetch(p.dtotal, row, p.dt_ld, nt);
    }
    stats(row, mean_now, rstd_now);
    stats(row + HOLD * step, mean_next, rstd_next);
    float g[CPT], dg[CPT], db[CPT];
#pragma unroll
    for (int k = 0; k < CPT; ++k) {
        const int c = t + k * TPR;
        if (c < cols) g[k] = weight_at(p.gamma, p.wdtype, c, 1.f);
        dg[k] = db[k] = 0.f;
    }
    int phase = 0, turn = 0;
    // (the row groups of one warp go round together, those without a row idle)
    const int64_t warp_row = TPR < 32 ? (int64_t)blockIdx.x * RPC + rl / (32 / HOLD) * (32 / HOLD) : row;
    for (int64_t any = warp_row; any < p.rows; any += step, row += step) {
        const int mine = TPR >= 32 || row < p.rows ? cols : 0;
        if (turn == HOLD) {
            turn = 0;
            mean_now = mean_next;
            rstd_now = rstd_next;
            stats(row + HOLD * step, mean_next, rstd_next);
        }
        const float mean = __shfl_sync(0xffffffffu, mean_now, (lane & ~(HOLD - 1)) + turn);
        const float rstd = __shfl_sync(0xffffffffu, rstd_now, (lane & ~(HOLD - 1)) + turn);
        ++turn;
        W cd[CPT], cx[CPT], ct[CPT];
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
        }
        float d[CPT], x[CPT], s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
            if (t + k * TPR < mine) {
                d[k] = elem_to_f<DT>(cd[k]);
                x[k] = elem_to_f<DT>(cx[k]) - mean;
                db[k] += d[k];
                d[k] *= rstd;
                const float gd = d[k] * g[k];
                s1 += gd;
                s2 = fmaf(gd, x[k], s2);
                dg[k] = fmaf(d[k], x[k], dg[k]);
            }
        }
#pragma unroll
        for (int o = HOLD / 2; o >= 1; o >>= 1) {
            s1 += __shfl_xor_sync(0xffffffffu, s1, o);
            s2 += __shfl_xor_sync(0xffffffffu, s2, o);
        }
        if constexpr (TPR > 32) {
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
            // s1 = rstd * sum(g), s2 = sum(g * xhat): with u = x - mean and
            // v = dy * rstd, dx = v * gamma - u * rstd^2 * s2 / n - s1 / n
            const float ca = -rstd * rstd * (s2 * inv_n), cb = -(s1 * inv_n);
            char* const out = reinterpret_cast<char*>(p.dx) + row * p.dx_ld * elem_size(DT);
#pragma unroll
            for (int k = 0; k < CPT; ++k) {
                const int c = t + k * TPR;
                if (c < mine) {
                    const float t0 = TOT ? elem_to_f<DT>(ct[k]) + cb : cb;
                    const float o[1] = {fmaf(d[k], g[k], fmaf(x[k], ca, t0))};
                    W* const dst = reinterpret_cast<W*>(out) + c;
                    if (in_bounds(dst, sizeof(W), out, row_bytes, p.status)) *dst = pack<DT, 1>(o);
                }
            }
        }
    }

    if (p.workspace == nullptr) return;
    float* const out = p.workspace + (int64_t)blockIdx.x * 2 * p.cols;
    if constexpr (RPC > 1) {
        // the CTA's row groups' sums meet in shared memory, a thread's column k at
        // [group][which][k][t], the rows four words longer than TPR so that
        // neighbouring columns are in different banks; then every column is
        // added up over the groups in order
        constexpr int PITCH = TPR + 4;
        float* const s_acc = reinterpret_cast<float*>(s_rows);
        __syncthreads();
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
            s_acc[((rl * 2 + 0) * CPT + k) * PITCH + t] = dg[k];
            s_acc[((rl * 2 + 1) * CPT + k) * PITCH + t] = db[k];
        }
        __syncthreads();
        for (int i = threadIdx.x; i < 2 * cols; i += BLOCK) {
            const int which = i >= cols ? 1 : 0;
            const int col = i - which * cols;
            const float* const at = s_acc + (which * CPT + col / TPR) * PITCH + col % TPR;
            float v = at[0];
#pragma unroll
            for (int w = 1; w < RPC; ++w) v += at[w * 2 * CPT * PITCH];
            out[i] = v;
        }
    } else {
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
            const int c = t + k * TPR;
            if (c < cols) {
                out[c] = dg[k];
                out[p.cols + c] = db[k];
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
            weights_at<VEC>(p.gamma, p.wdtype, c * VEC, 1.f, gv);
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
            weights_at<VEC>(p.gamma, p.wdtype, c * VEC, 1.f, gv);
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

template <int DT, int TPR, int CPT, bool WHOLE>
cudaError_t bwd_launch(const LnBwdParams& p, int sms, int* parts, cudaStream_t s) {
    constexpr int VEC = 16 / elem_size(DT), rpc = BWD_BLOCK / TPR;
    const int64_t want = (p.rows + rpc - 1) / rpc;
    int64_t grid = sms < TB_LN_PARTS ? sms : TB_LN_PARTS;
    if (grid > want) grid = want;
    *parts = (int)grid;
    LnBwdParams q = p;
    const int64_t bytes = p.cols * elem_size(DT), pitch = WHOLE ? bytes : (bytes + 31) / 16 * 16;
    const int64_t stage = (int64_t)rpc * (p.dtotal ? 3 : 2) * pitch;
    constexpr int64_t room = ln_bwd_room(TPR), sums = rpc > 1 ? (int64_t)rpc * 2 * CPT * VEC * (TPR + 4) * 4 : 0;
    static_assert(2 * rpc * 3 * (TPR * CPT * 16 + (WHOLE ? 0 : 16)) <= room && sums <= room,
                  "two stages of the widest rows, or the row groups' sums, do not fit");
    const int64_t fit = room / stage;
    q.stages = (int)(fit > LN_BWD_MAX_STAGES ? LN_BWD_MAX_STAGES : fit);
    const int64_t smem = q.stages * stage > sums ? q.stages * stage : sums;
    void (*fn)(const LnBwdParams) =
        p.dtotal ? ln_bwd_kernel<DT, TPR, CPT, true, WHOLE> : ln_bwd_kernel<DT, TPR, CPT, false, WHOLE>;
    if (smem > 40 * 1024) {  // with the static shared memory, past the 48 KB default
        // the limit belongs to the function, not to the launch: one value for
        // rows of every width, since several host threads may be launching it
        const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)room);
        if (e != cudaSuccess) return e;
    }
    return launch_pdl(fn, q, dim3((unsigned)grid), BWD_BLOCK, (size_t)smem, s);
}

template <int DT, int VEC>
cudaError_t bwd_long(const LnBwdParams& p, int sms, int* parts, cudaStream_t s) {
    int64_t grid = p.rows < sms ? p.rows : sms;
    if (grid > TB_LN_PARTS) grid = TB_LN_PARTS;
    *parts = (int)grid;
    return launch_pdl(p.dtotal ? ln_bwd_long_kernel<DT, VEC, true> : ln_bwd_long_kernel<DT, VEC, false>, p,
                      dim3((unsigned)grid), LONG_BLOCK, 0, s);
}

template <int DT, int TPR, int CPT>
cudaError_t bwd_elem(const LnBwdParams& p, int sms, int* parts, cudaStream_t s) {
    constexpr int rpc = BWD_BLOCK / TPR;
    const int64_t want = (p.rows + rpc - 1) / rpc;
    int64_t grid = sms < TB_LN_PARTS ? sms : TB_LN_PARTS;
    if (grid > want) grid = want;
    *parts = (int)grid;
    const size_t smem = rpc > 1 ? (size_t)rpc * 2 * CPT * (TPR + 4) * 4 : 0;  // at most 40 KB
    return launch_pdl(p.dtotal ? ln_bwd_elem_kernel<DT, TPR, CPT, true> : ln_bwd_elem_kernel<DT, TPR, CPT, false>, p,
                      dim3((unsigned)grid), BWD_BLOCK, smem, s);
}

// A row's 16-byte words, or columns, pick its threads.
template <int DT>
cudaError_t bwd_dt(const LnBwdParams& p, bool vector, int sms, int* parts, cudaStream_t s) {
    constexpr int V = 16 / elem_size(DT);
    const int64_t n = (p.cols + V - 1) / V;
    if (vector) {
        if (n <= 8) return bwd_launch<DT, 8, 1, true>(p, sms, parts, s);
        if (n <= 16) return bwd_launch<DT, 16, 1, true>(p, sms, parts, s);
        if (n <= 32) return bwd_launch<DT, 32, 1, true>(p, sms, parts, s);
        if (n <= 64) return bwd_launch<DT, 32, 2, true>(p, sms, parts, s);
        if (n <= 128) return bwd_launch<DT, 64, 2, true>(p, sms, parts, s);
        if (n <= 256) return bwd_launch<DT, 128, 2, true>(p, sms, parts, s);
        if (n <= 512) return bwd_launch<DT, 256, 2, true>(p, sms, parts, s);
        if (n <= 1024) return bwd_launch<DT, 512, 2, true>(p, sms, parts, s);
        if (n <= 2048) return bwd_launch<DT, 512, 4, true>(p, sms, parts, s);
        return bwd_long<DT, V>(p, sms, parts, s);
    }
    // (short rows two to a warp: 262144 x 63 bf16 42.1 us, 131072 x 127 28.8; one to a warp 72.7 and 42.9)
    if (p.cols <= 64) return bwd_elem<DT, 16, 4>(p, sms, parts, s);
    if (p.cols <= 128) return bwd_elem<DT, 16, 8>(p, sms, parts, s);
    if (p.cols <= 256) return bwd_elem<DT, 32, 8>(p, sms, parts, s);
    if (p.cols <= 512) return bwd_elem<DT, 64, 8>(p, sms, parts, s);
    if (p.cols <= 1024) return bwd_elem<DT, 128, 8>(p, sms, parts, s);
    if (p.cols <= 2048) return bwd_elem<DT, 256, 8>(p, sms, parts, s);
    if (p.cols <= ELEM_COLS) return bwd_elem<DT, 512, 8>(p, sms, parts, s);
    if (n <= 1024) return bwd_launch<DT, 512, 2, false>(p, sms, parts, s);
    if (n <= 2048) return bwd_launch<DT, 512, 4, false>(p, sms, parts, s);
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
