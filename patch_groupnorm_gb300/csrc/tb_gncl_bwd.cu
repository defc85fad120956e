// tb_gncl_bwd.cu -- the backward pass of channels-last PatchGroupNorm (+ SiLU).
//
// With d = x - mean, xhat = d * rstd, z = xhat * gamma + beta, s = 1 / (1 + e^-z):
//     dz = silu ? dy * s * (1 + z * (1 - s)) : dy
//     B(n, c) = sum dz,  A(n, c) = sum dz * xhat     (over the channel's elements)
//     dgamma(c) = sum_n A,  dbeta(c) = sum_n B
//     c1 = sum over the group's channels of gamma * B / count,  c2 the same of A
//     dx = rnd(rstd * (gamma * dz - c1 - xhat * c2)) = rnd(a * dz + u * d + v),
//          a = rstd * gamma, u = -rstd^2 c2, v = -rstd c1
//
// Three launches: the records (B, A) of every channel; (mean, rstd, u, v) of every
// group and the weight gradients from the records; dx.  A CTA of the last would
// otherwise read every channel's records (131 KB for 512 channels in 32 parts).  The
// second triggers the third, which fetches its first chunks meanwhile.
//
// x and dy are read twice.  1 x 256 x 256 x 512 bf16 in four patches takes 60.5 us
// (the records 26.4, the constants and dx 34.7), where 335 MB are 49 us at the copy
// rate; 13 x 120 x 208 x 384: 199 us, of 184.  The records are bound by memory and by
// issue slots (43 % busy over the launch, 55 % while CTAs are resident): per pair of
// chunks an exponential and a reciprocal an element, and 128 registers, so two CTAs
// of 256 threads per SM.
#include "tb_gncl.cuh"

namespace tb {
namespace {

// --- the records ------------------------------------------------------------------

constexpr int FOLD = 60;  // chunks between two foldings of a thread's sums: whole turns of DEPTH
constexpr int DEPTH = 6;  // chunks of x and of dy of a thread on their way or in work

template <int DT, int VEC, bool SILU>
__global__ void __launch_bounds__(CL_BLOCK, 2) gncl_grad_stats_kernel(const __grid_constant__ GnClParams p) {
    using L = Lanes<VEC>;
    using W = ClWord<DT, VEC>;
    constexpr int ES = elem_size(DT), NL = L::N;
    extern __shared__ uint4 shared4[];
    const int C = (int)p.C, K = p.K;
    const int cs = C / p.splits, c0 = (int)blockIdx.y * cs;  // this CTA's channels
    using Stream = ClStream<DT, VEC, 2, DEPTH>;
    float2* const stage = reinterpret_cast<float2*>(shared4 + Stream::SMEM / 16);  // [CL_BLOCK * VEC]: (sum dz, sum dz * d)
    float2* const table = stage + CL_BLOCK * VEC;              // [cs]: (sum dz, sum dz * xhat)
    float2* const stats = table + cs;                          // groups of those channels: (mean, rstd)
    const int g0 = c0 / K, g1 = (c0 + cs + K - 1) / K;
    for (int c = threadIdx.x; c < cs; c += CL_BLOCK) table[c] = make_float2(0.f, 0.f);
    const ClUnit u = cl_unit(p);
    const int parts = p.parts[u.p], piece = u.piece, pieces = u.pieces, last = cl_last_piece(p, u.p, pieces);
    const ClRun run = cl_run<ES, VEC>(p.patches[u.p], p.spatial[u.p], p.C, u.n);
    const char* const patch = static_cast<const char*>(p.patches[u.p]);
    const char* const grad = static_cast<const char*>(p.grads[u.p]);
    const int64_t bytes = p.N * run.elems * ES, from = (run.first + run.head) * ES;
    const int split_width = p.period / p.splits, split0 = (int)blockIdx.y * split_width;
    Stream in;
    in.base[0] = patch;
    in.base[1] = grad;
    in.bytes = bytes;
    in.status = p.status;
    auto begin = [&](const ClWalk& w) {
        const int64_t at = from + w.at * (int64_t)sizeof(W);
        in.at[0] = patch + at;
        in.at[1] = grad + at;
        in.stride = w.stride * (int64_t)sizeof(W);
        in.start(w.count, shared4);
    };
    grid_wait();
    // the first columns' chunks are on their way while the groups' statistics are found
    const int mine = split0 + u.slab * p.columns;
    begin(cl_walk_share(p, cl_place(p, mine, min(mine + p.columns, split0 + split_width)), u.p, piece, pieces, run.chunks));
    cl_group_stats(p, u.n, g0, g1, stats);
    __syncthreads();

    for (int j0 = mine; j0 < split0 + split_width; j0 += p.slabs * p.columns) {
        const int j1 = min(j0 + p.columns, split0 + split_width);
        const ClPlace q = cl_place(p, j0, j1);
        const ClWalk w = cl_walk_share(p, q, u.p, piece, pieces, run.chunks);
        typename L::T mean[NL], ga[NL], be[NL], sb[NL], sa[NL], tb_[NL], ta[NL];
        float f0[VEC], f1[VEC], f2[VEC];
        if constexpr (SILU) cl_weights<DT, VEC>(p, run.head, q.col * VEC, f1, f2);
        ClChannel ch(run.head, q.col * VEC, C, K);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            // threads without a place may point past this CTA's groups
            const float2 s = q.row >= 0 ? stats[ch.g - g0] : make_float2(0.f, 0.f);
            f0[i] = s.x;
            f1[i] = SILU ? s.y * f1[i] : 0.f;
            f2[i] = SILU ? f2[i] : 0.f;
            ch.next();
        }
        cl_lanes<VEC>(f0, mean);
        cl_lanes<VEC>(f1, ga);
        cl_lanes<VEC>(f2, be);
#pragma unroll
        for (int i = 0; i < NL; ++i) tb_[i] = ta[i] = L::splat(0.f);
        if (j0 != mine) begin(w);
        for (int done = 0; done < w.count; done += FOLD) {
            const int now = min(FOLD, w.count - done);
#pragma unroll
            for (int i = 0; i < NL; ++i) sb[i] = sa[i] = L::splat(0.f);
            cl_each(in, now, [&](const W (&v)[2], int) {
                typename L::T f[NL], dy[NL];
                to_lanes<DT, VEC>(v[0], f);
                to_lanes<DT, VEC>(v[1], dy);
#pragma unroll
                for (int i = 0; i < NL; ++i) {
                    const typename L::T d = vsub(f[i], mean[i]);
                    const typename L::T dz = dz_of<SILU>(dy[i], vfma(d, ga[i], be[i]));
                    sb[i] = vadd(sb[i], dz);
                    sa[i] = vfma(dz, d, sa[i]);
                }
            });
#pragma unroll
            for (int i = 0; i < NL; ++i) {
                tb_[i] = vadd(tb_[i], sb[i]);
                ta[i] = vadd(ta[i], sa[i]);
            }
        }
        cl_values<VEC>(tb_, f0);
        cl_values<VEC>(ta, f1);
        __syncthreads();  // the columns before these are merged
#pragma unroll
        for (int i = 0; i < VEC; ++i) stage[threadIdx.x * VEC + i] = make_float2(f0[i], f1[i]);
        __syncthreads();
        const int lo = run.head + j0 * VEC, hi = run.head + j1 * VEC, pitch = q.width * VEC;
        for (int i = threadIdx.x; i < cs; i += CL_BLOCK) {
            const int c = c0 + i;
            float2 t = table[i];
            const float rstd = stats[c / K - g0].y;
            for (int at = c + (lo > c ? (lo - c + C - 1) / C * C : 0); at < hi; at += C) {
                for (int r = 0; r < q.rows; ++r) {
                    const float2 v = stage[r * pitch + at - lo];
                    t.x += v.x;
                    t.y = fmaf(v.y, rstd, t.y);
                }
            }
            table[i] = t;
        }
    }
    // elements outside the whole chunks: the first piece's before, the last one's after; a lane each
    __syncthreads();
    if (VEC > 1 && threadIdx.x < 32) {
        const int lane = threadIdx.x;
        const int h = piece == 0 && u.slab == 0 ? run.head : 0, t = piece == last && u.slab == 0 ? run.tail : 0;
        float dz = 0.f, xhat = 0.f;
        int c = -1;
        if (lane < h + t) {
            const int64_t e = lane < h ? lane : run.elems - run.tail + (lane - h);
            c = (int)(e % C);
            if (c >= c0 && c < c0 + cs) {
                const float2 s = stats[c / K - g0];
                xhat = (cl_elem<DT>(patch, run.first + e, bytes, p.status) - s.x) * s.y;
                dz = dz_of<SILU>(cl_elem<DT>(grad, run.first + e, bytes, p.status),
                                 fmaf(xhat, cl_weight<DT>(p, p.gamma, c, 1.f), cl_weight<DT>(p, p.beta, c, 0.f)));
            } else {
                c = -1;
            }
        }
        for (unsigned left = __ballot_sync(0xffffffffu, c >= 0); left; left &= left - 1) {
            const int k = __ffs(left) - 1;
            const int ck = __shfl_sync(0xffffffffu, c, k);
            const float zk = __shfl_sync(0xffffffffu, dz, k), hk = __shfl_sync(0xffffffffu, xhat, k);
            if (lane == 0) {
                table[ck - c0].x += zk;
                table[ck - c0].y = fmaf(zk, hk, table[ck - c0].y);
            }
        }
        __syncwarp();
    }
    if (p.cluster > 1) cluster_sync();
    else __syncthreads();
    float2* const out = p.grad_partials + ((int64_t)u.p * p.N + u.n) * C * TB_GN_PARTS;
    for (int i = u.rank * CL_BLOCK + (int)threadIdx.x; i < cs; i += p.cluster * CL_BLOCK) {
        float2 t = table[i];
        if (p.cluster > 1) {
            t = make_float2(0.f, 0.f);
            uint2 v[CL_MAX_CLUSTER];
#pragma unroll
            for (int r = 0; r < CL_MAX_CLUSTER; ++r)  // all on their way before the first sum
                v[r] = r < p.cluster ? cluster_load8(smem_addr(table + i), (uint32_t)r) : make_uint2(0u, 0u);
#pragma unroll
            for (int r = 0; r < CL_MAX_CLUSTER; ++r) {
                t.x += __uint_as_float(v[r].x);
                t.y += __uint_as_float(v[r].y);
            }
        }
        float2* const at = out + (int64_t)(c0 + i) * TB_GN_PARTS;
        if (!in_bounds(at, TB_GN_PARTS * sizeof(float2), p.grad_partials,
                       (int64_t)p.P * p.N * C * TB_GN_PARTS * (int64_t)sizeof(float2), p.status))
            continue;
        at[u.part] = t;
        if (u.part == 0)
            for (int r = parts; r < TB_GN_PARTS; ++r) at[r] = make_float2(0.f, 0.f);
    }
    if (p.cluster > 1) cluster_sync();  // nobody leaves while its table may be read
}

static_assert(FOLD % DEPTH == 0, "a fold ends a turn");

template <int DT, int VEC>
size_t grad_stats_smem(int64_t C, int G, int splits) {
    const int64_t cs = C / splits, K = C / G;
    return ClStream<DT, VEC, 2, DEPTH>::SMEM + (size_t)(CL_BLOCK * VEC + cs + (cs + K - 1) / K + 1) * sizeof(float2);
}

// --- the groups' constants and the weight gradients -----------------------------------

// CTAs 0 .. N * G - 1: one group of one sample; the rest: COEF_CHANNELS channels'
// weight gradients each.
constexpr int COEF_CHANNELS = CL_BLOCK / TB_GN_PARTS;

template <int DT>
__global__ void __launch_bounds__(CL_BLOCK) gncl_coefs_kernel(const __grid_constant__ GnClParams p) {
    __shared__ float2 sums[CL_BLOCK / 32];
    __shared__ float2 stats[1];
    const int C = (int)p.C, K = p.K;
    const int64_t units = p.coefs != nullptr ? p.N * p.G : 0, set = p.N * C * TB_GN_PARTS;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t size = (int64_t)p.R * set * (int64_t)sizeof(float2);
    grid_wait();
    // what came before is done, so dx's launch may fetch its first chunks of x and dy
    // while this one works; it waits before it reads a constant or writes a chunk
    if (units > 0) pdl_trigger_dependents();
    if ((int64_t)blockIdx.x < units) {
        const int64_t n = blockIdx.x / p.G;
        const int g = (int)(blockIdx.x - n * p.G);
        const int per_set = K * TB_GN_PARTS;
        float B = 0.f, A = 0.f;
        for (int r = 0; r < p.R; ++r) {
            const float2* const first = p.grad_partials + r * set + (n * C + (int64_t)g * K) * TB_GN_PARTS;
#pragma unroll 4
            for (int i = threadIdx.x; i < per_set; i += CL_BLOCK) {
                if (!in_bounds(first + i, sizeof(float2), p.grad_partials, size, p.status)) continue;
                const float2 v = first[i];
                const float w = cl_weight<DT>(p, p.gamma, g * K + i / TB_GN_PARTS, 1.f);
                B = fmaf(w, v.x, B);
                A = fmaf(w, v.y, A);
            }
        }
        B = warp_sum(B);
        A = warp_sum(A);
        if (lane == 0) sums[warp] = make_float2(B, A);
        // the count: of the forward pass's records
        long long count = 0;
        if (warp == 0) {
            for (int q = lane; q < p.R * TB_GN_PARTS; q += 32) {
                const GnPartial* const at =
                    p.partials + (((int64_t)(q / TB_GN_PARTS) * p.N + n) * p.G + g) * TB_GN_PARTS + q % TB_GN_PARTS;
                if (in_bounds(at, sizeof(GnPartial), p.partials,
                              p.R * p.N * p.G * TB_GN_PARTS * (int64_t)sizeof(GnPartial), p.status))
                    count += at->n;
            }
#pragma unroll
            for (int d = 16; d >= 1; d >>= 1) count += __shfl_xor_sync(0xffffffffu, count, d);
        }
        cl_group_stats(p, n, g, g + 1, stats);
        __syncthreads();
        if (threadIdx.x == 0) {
            B = A = 0.f;
            for (int k = 0; k < CL_BLOCK / 32; ++k) {
                B += sums[k].x;
                A += sums[k].y;
            }
            const float inv = count > 0 ? 1.f / (float)count : 0.f, rstd = stats[0].y;
            if (index_ok(blockIdx.x < p.N * p.G, p.status))
                p.coefs[blockIdx.x] = make_float4(stats[0].x, rstd, -(rstd * rstd) * (A * inv), -rstd * (B * inv));
        }
        return;
    }
    // a channel per eight lanes, a lane per part
    const int64_t c = ((int64_t)blockIdx.x - units) * COEF_CHANNELS + threadIdx.x / TB_GN_PARTS;
    float B = 0.f, A = 0.f;
    if (c < C) {
        for (int64_t r = 0; r < p.R * p.N; ++r) {
            const float2* const at = p.grad_partials + (r * C + c) * TB_GN_PARTS + threadIdx.x % TB_GN_PARTS;
            if (!in_bounds(at, sizeof(float2), p.grad_partials, size, p.status)) continue;
            const float2 v = *at;
            B += v.x;
            A += v.y;
        }
    }
#pragma unroll
    for (int d = TB_GN_PARTS / 2; d >= 1; d >>= 1) {
        B += __shfl_xor_sync(0xffffffffu, B, d);
        A += __shfl_xor_sync(0xffffffffu, A, d);
    }
    if (c < C && threadIdx.x % TB_GN_PARTS == 0) {
        cl_store_weight<DT>(p, p.dgamma, c, A);
        cl_store_weight<DT>(p, p.dbeta, c, B);
    }
}

// --- dx -----------------------------------------------------------------------------

// As DEPTH, pairs of chunks (two CTAs per SM: 114 us alone for 13 x 120 x 208 x 384 bf16,
// 122 with 5).  Single elements: with 4, 6, 8, 10 and 12 the whole call takes 138, 120, 122,
// 118 and 113 us for 65536 x 512 bf16, 318, 288, 275, 281 and 273 for 3 x 24568 x 515 f32.
template <int VEC>
constexpr int APPLY_DEPTH = VEC > 1 ? 4 : 12;

template <int DT, int VEC, bool SILU>
__global__ void __launch_bounds__(CL_BLOCK, 2) gncl_grad_apply_kernel(const __grid_constant__ GnClParams p) {
    using L = Lanes<VEC>;
    using W = ClWord<DT, VEC>;
    constexpr int ES = elem_size(DT), NL = L::N;
    const int C = (int)p.C, K = p.K;
    int pt = 0;
    while (pt + 1 < p.P && (int)blockIdx.x >= p.start[pt + 1]) ++pt;
    const int local = (int)blockIdx.x - p.start[pt], n = local / p.parts[pt], piece = local - n * p.parts[pt];
    const ClRun run = cl_run<ES, VEC>(p.patches[pt], p.spatial[pt], p.C, n);
    const char* const patch = static_cast<const char*>(p.patches[pt]);
    const char* const grad = static_cast<const char*>(p.grads[pt]);
    char* const out = static_cast<char*>(p.outs[pt]);
    const int64_t bytes = p.N * run.elems * ES, from = (run.first + run.head) * ES;
    const int j0 = (int)blockIdx.y * p.columns, j1 = min(j0 + p.columns, p.period);
    const ClPlace q = cl_place(p, j0, j1);
    const ClWalk w = cl_walk_dealt(q, piece, p.parts[pt], p.period, run.chunks);
    const float4* const coefs = p.coefs + (int64_t)n * p.G;
    // from the end: the records' pass left that in L2
    const int64_t last = from + (w.at + (w.count - 1) * w.stride) * (int64_t)sizeof(W);
    extern __shared__ uint4 shared4[];
    ClStream<DT, VEC, 2, APPLY_DEPTH<VEC>> in;
    in.base[0] = patch;
    in.base[1] = grad;
    in.at[0] = patch + last;
    in.at[1] = grad + last;
    in.stride = -w.stride * (int64_t)sizeof(W);
    in.bytes = bytes;
    in.status = p.status;
    // the launch before this one is always the constants', which starts it once
    // everything before that is done: x and dy are in place, the constants are not
    in.start(w.count, shared4);
    grid_wait();
    typename L::T mean[NL], ga[NL], be[NL], cu[NL], cv[NL];
    {
        float f0[VEC], f1[VEC], f2[VEC], f3[VEC], f4[VEC];
        cl_weights<DT, VEC>(p, run.head, q.col * VEC, f1, f2);
        ClChannel ch(run.head, q.col * VEC, C, K);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const float4 k = index_ok(ch.g >= 0 && ch.g < p.G, p.status) ? coefs[ch.g] : make_float4(0.f, 0.f, 0.f, 0.f);
            f0[i] = k.x;
            f1[i] *= k.y;
            f3[i] = k.z;
            f4[i] = k.w;
            ch.next();
        }
        cl_lanes<VEC>(f0, mean);
        cl_lanes<VEC>(f1, ga);
        cl_lanes<VEC>(f2, be);
        cl_lanes<VEC>(f3, cu);
        cl_lanes<VEC>(f4, cv);
    }
    char* to = out + last;
    cl_each(in, w.count, [&](const W (&v)[2], int) {
        typename L::T f[NL], dy[NL];
        to_lanes<DT, VEC>(v[0], f);
        to_lanes<DT, VEC>(v[1], dy);
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            const typename L::T d = vsub(f[i], mean[i]);
            const typename L::T dz = dz_of<SILU>(dy[i], vfma(d, ga[i], be[i]));
            f[i] = vfma(dz, ga[i], vfma(d, cu[i], cv[i]));
        }
        if (in_bounds(to, sizeof(W), out, bytes, p.status)) __stcs(reinterpret_cast<W*>(to), from_lanes<DT, VEC>(f));
        to += in.stride;
    });
    if (VEC > 1 && blockIdx.y == 0) {
        const int h = piece == 0 ? run.head : 0, t = piece == p.parts[pt] - 1 ? run.tail : 0;
        if ((int)threadIdx.x < h + t) {
            const int64_t e = (int)threadIdx.x < h ? threadIdx.x : run.elems - run.tail + (threadIdx.x - h);
            const int c = (int)(e % C);
            const float4 k = index_ok(c / K < p.G, p.status) ? coefs[c / K] : make_float4(0.f, 0.f, 0.f, 0.f);
            const float gam = k.y * cl_weight<DT>(p, p.gamma, c, 1.f);
            const float d = cl_elem<DT>(patch, run.first + e, bytes, p.status) - k.x;
            const float dz = dz_of<SILU>(cl_elem<DT>(grad, run.first + e, bytes, p.status),
                                         fmaf(d, gam, cl_weight<DT>(p, p.beta, c, 0.f)));
            cl_store_elem<DT>(out, run.first + e, fmaf(dz, gam, fmaf(d, k.z, k.w)), bytes, p.status);
        }
    }
}

template <int DT>
cudaError_t stats_launch(const GnClParams& p, bool vector, int64_t ctas, cudaStream_t s) {
    constexpr int V = 16 / elem_size(DT);
    void (*const fn)(const GnClParams) =
        vector ? (p.silu ? gncl_grad_stats_kernel<DT, V, true> : gncl_grad_stats_kernel<DT, V, false>)
               : (p.silu ? gncl_grad_stats_kernel<DT, 1, true> : gncl_grad_stats_kernel<DT, 1, false>);
    const size_t smem = vector ? grad_stats_smem<DT, V>(p.C, p.G, p.splits) : grad_stats_smem<DT, 1>(p.C, p.G, p.splits);
    return launch_cluster(fn, p, dim3((unsigned)ctas, (unsigned)p.splits, 1), p.cluster, smem, s);
}

template <int DT>
cudaError_t apply_launch(const GnClParams& p, bool vector, int64_t ctas, cudaStream_t s) {
    constexpr int V = 16 / elem_size(DT);
    void (*const fn)(const GnClParams) =
        vector ? (p.silu ? gncl_grad_apply_kernel<DT, V, true> : gncl_grad_apply_kernel<DT, V, false>)
               : (p.silu ? gncl_grad_apply_kernel<DT, 1, true> : gncl_grad_apply_kernel<DT, 1, false>);
    const unsigned slabs = (unsigned)((p.period + p.columns - 1) / p.columns);
    return launch_cluster(fn, p, dim3((unsigned)ctas, slabs, 1), 1, vector ? ClStream<DT, V, 2, APPLY_DEPTH<V>>::SMEM : 0, s);
}

}  // namespace

cudaError_t launch_gncl_grad_stats(const GnClParams& p, int dtype, bool vector, int64_t ctas, cudaStream_t s) {
    if (dtype == F32) return stats_launch<F32>(p, vector, ctas, s);
    if (dtype == F16) return stats_launch<F16>(p, vector, ctas, s);
    return stats_launch<BF16>(p, vector, ctas, s);
}

cudaError_t launch_gncl_coefs(const GnClParams& p, int dtype, bool weights_only, cudaStream_t s) {
    const int64_t weights = p.dgamma != nullptr || p.dbeta != nullptr ? (p.C + COEF_CHANNELS - 1) / COEF_CHANNELS : 0;
    const dim3 grid((unsigned)((weights_only ? 0 : p.N * p.G) + weights), 1, 1);
    void (*const fn)(const GnClParams) = dtype == F32 ? gncl_coefs_kernel<F32>
                                         : dtype == F16 ? gncl_coefs_kernel<F16>
                                                        : gncl_coefs_kernel<BF16>;
    return launch_cluster(fn, p, grid, 1, 0, s);
}

cudaError_t launch_gncl_grad_apply(const GnClParams& p, int dtype, bool vector, int64_t ctas, cudaStream_t s) {
    if (dtype == F32) return apply_launch<F32>(p, vector, ctas, s);
    if (dtype == F16) return apply_launch<F16>(p, vector, ctas, s);
    return apply_launch<BF16>(p, vector, ctas, s);
}

}  // namespace tb
