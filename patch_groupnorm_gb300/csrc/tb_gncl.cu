// tb_gncl.cu -- PatchGroupNorm (+ SiLU) of channels-last patches: statistics
// records, and the normalisation.
//
// y = silu(d * a + beta), d = x - mean, a = rstd * gamma, with mean and rstd of
// the group pooled over the patches.  Subtracting the mean first keeps what a
// single x * a + b would lose where the mean is far from zero.
//
// Statistics need all of a group before the first output, so x is read twice, by
// two launches; what is bound by memory is bound there.
#include "tb_gncl.cuh"

namespace tb {
namespace {

// --- statistics -------------------------------------------------------------------

// Groups of one CTA: count, mean and sum of squared deviations of what it read.
struct ClTable {
    int2* moments;   // (mean, M2) as bits
    long long* n;
};

__device__ __forceinline__ void chan(long long& n, float& mean, float& m2, long long bn, float bmean, float bm2) {
    if (bn == 0) return;
    if (n == 0) {
        n = bn;
        mean = bmean;
        m2 = bm2;
        return;
    }
    const float na = (float)n, nb = (float)bn, total = (float)(n + bn);
    const float d = bmean - mean, f = nb / total;
    mean = fmaf(d, f, mean);
    m2 += fmaf(d * d, na * f, bm2);
    n += bn;
}

constexpr int FOLD = 64;  // chunks between two foldings of a thread's sums
constexpr int SU = 4;     // chunks a thread loads together

// Each thread sums x - K and (x - K)^2 of its VEC channels on packed pairs, K its
// own first value, then its mean so far; after SU, SU, 2 SU, 4 SU, ... and then every
// FOLD chunks the sums are merged into (mean, M2) (Chan), so that neither a far mean
// nor a long run loses digits, nor a first value far from all others: n chunks
// about a mean that it has moved by 1 / n of its distance add 1 / n of its square.
// A CTA's threads meet in shared memory, group by group, and the CTAs of a
// cluster read each other's tables, in a fixed order: one record per cluster.
template <int DT, int VEC>
__global__ void __launch_bounds__(CL_BLOCK, 3) gncl_stats_kernel(const __grid_constant__ GnClParams p) {
    using L = Lanes<VEC>;
    using W = ClWord<DT, VEC>;
    constexpr int ES = elem_size(DT), NL = L::N;
    extern __shared__ uint4 shared4[];
    float* const stage_mean = reinterpret_cast<float*>(shared4);      // [CL_BLOCK * VEC]
    float* const stage_m2 = stage_mean + CL_BLOCK * VEC;              // [CL_BLOCK * VEC]
    int* const stage_n = reinterpret_cast<int*>(stage_m2 + CL_BLOCK * VEC);  // [CL_BLOCK]
    const int C = (int)p.C, G = p.G, K = C / G;
    const int gs = G / p.splits, g0 = (int)blockIdx.y * gs, g1 = g0 + gs;  // this CTA's groups
    ClTable table;
    table.n = reinterpret_cast<long long*>(stage_n + CL_BLOCK);       // [gs]
    table.moments = reinterpret_cast<int2*>(table.n + gs);            // [gs]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int g = threadIdx.x; g < gs; g += CL_BLOCK) {
        table.n[g] = 0;
        table.moments[g] = make_int2(0, 0);
    }
    const ClUnit u = cl_unit(p);
    const int parts = p.parts[u.p], piece = u.part * p.cluster + u.rank, pieces = parts * p.cluster;
    const ClRun run = cl_run<ES, VEC>(p.patches[u.p], p.spatial[u.p], p.C, u.n);
    const char* const patch = static_cast<const char*>(p.patches[u.p]);
    const int64_t bytes = p.N * run.elems * ES;
    const W* const base = reinterpret_cast<const W*>(patch + (run.first + run.head) * ES);
    grid_wait();

    // elements outside the whole chunks: the first piece's before, the last one's after; a lane each
    float edge = 0.f;
    int edge_group = -1;
    if (VEC > 1 && warp == 0) {
        const int h = piece == 0 ? run.head : 0, t = piece == pieces - 1 ? run.tail : 0;
        if (lane < h + t) {
            const int64_t e = lane < h ? lane : run.elems - run.tail + (lane - h);
            if (in_bounds(patch + (run.first + e) * ES, ES, patch, bytes, p.status))
                edge = cl_elem<DT>(patch, run.first + e);
            edge_group = (int)(e % C) / K;
        }
    }

    const int64_t total_rows = (run.chunks + p.period - 1) / p.period;
    int64_t a, b;
    cl_piece(total_rows, piece, pieces, a, b);
    const int split_width = p.period / p.splits, split0 = (int)blockIdx.y * split_width;
    for (int j0 = split0; j0 < split0 + split_width; j0 += p.columns) {
        const int j1 = min(j0 + p.columns, split0 + split_width);
        const ClPlace q = cl_place(j0, j1);
        const ClWalk w = cl_walk(q, a, b, p.period, run.chunks);
        typename L::T k[NL], s1[NL], s2[NL], mean[NL], m2[NL];
#pragma unroll
        for (int i = 0; i < NL; ++i) k[i] = mean[i] = m2[i] = L::splat(0.f);
        const W* at = base + w.at;
        for (int done = 0, now; done < w.count; done += now) {
            now = min(min(FOLD, max(SU, done)), w.count - done);
#pragma unroll
            for (int i = 0; i < NL; ++i) s1[i] = s2[i] = L::splat(0.f);
            for (int s = 0; s < now; s += SU) {
                W v[SU];
#pragma unroll
                for (int r = 0; r < SU; ++r)
                    if (s + r < now && in_bounds(at + r * w.stride, sizeof(W), patch, bytes, p.status))
                        v[r] = __ldg(at + r * w.stride);
                at += SU * w.stride;
                if (done == 0 && s == 0) to_lanes<DT, VEC>(v[0], k);
#pragma unroll
                for (int r = 0; r < SU; ++r) {
                    if (s + r < now) {
                        typename L::T f[NL];
                        to_lanes<DT, VEC>(v[r], f);
#pragma unroll
                        for (int i = 0; i < NL; ++i) {
                            const typename L::T d = vsub(f[i], k[i]);
                            s1[i] = vadd(s1[i], d);
                            s2[i] = vfma(d, d, s2[i]);
                        }
                    }
                }
            }
            // the sums of `now` chunks about k join those of `done` before
            const float nb = (float)now, total = (float)(done + now);
            const auto inv = L::splat(1.f / nb), f = L::splat(nb / total), g = L::splat((float)done * (nb / total));
#pragma unroll
            for (int i = 0; i < NL; ++i) {
                const typename L::T d1 = vmul(s1[i], inv);                       // mean - k
                const typename L::T bm2 = vsub(s2[i], vmul(s1[i], d1));
                const typename L::T bmean = vadd(k[i], d1), d = vsub(bmean, mean[i]);
                mean[i] = vfma(d, f, mean[i]);
                m2[i] = vadd(m2[i], vfma(vmul(d, d), g, bm2));
                k[i] = mean[i];
            }
        }
        // rounding may leave a tiny negative sum of squares: it is a zero one
        float fm[VEC], f2[VEC];
        cl_values<VEC>(mean, fm);
        cl_values<VEC>(m2, f2);
        __syncthreads();  // the table is set, or the columns before these are merged
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            stage_mean[threadIdx.x * VEC + i] = fm[i];
            stage_m2[threadIdx.x * VEC + i] = f2[i] < 0.f ? 0.f : f2[i];
        }
        stage_n[threadIdx.x] = w.count;
        __syncthreads();
        // phases [head + j0 * VEC, head + j1 * VEC) hold this group's channels in runs of at most K
        const int lo = run.head + j0 * VEC, hi = run.head + j1 * VEC, pitch = q.width * VEC;
        for (int g = g0 + warp; g < g1; g += CL_BLOCK / 32) {
            const int c0 = g * K;
            const int m_first = lo >= c0 + K ? (lo - c0 - K) / C + 1 : 0;  // the first run that ends past lo
            long long n = 0;
            float gm = 0.f, k0 = 0.f, s = 0.f;
            for (int pass = 0; pass < 2; ++pass) {
                long long sn = 0;
                s = 0.f;
                for (int m = m_first; c0 + m * C < hi; ++m) {
                    const int from = max(c0 + m * C, lo) - lo, len = min(c0 + m * C + K, hi) - lo - from;
                    if (pass == 0 && m == m_first) k0 = stage_mean[from];
                    for (int e = lane; e < q.rows * len; e += 32) {
                        const int row = e / len, idx = row * pitch + from + (e - row * len);
                        const int ni = stage_n[idx / VEC];
                        if (ni == 0) continue;
                        if (pass == 0) {
                            sn += ni;
                            s = fmaf((float)ni, stage_mean[idx] - k0, s);
                        } else {
                            const float d = stage_mean[idx] - gm;
                            s += fmaf((float)ni * d, d, stage_m2[idx]);
                        }
                    }
                }
                s = warp_sum(s);
                if (pass == 0) {
#pragma unroll
                    for (int d = 16; d >= 1; d >>= 1) sn += __shfl_xor_sync(0xffffffffu, sn, d);
                    n = sn;
                    gm = n > 0 ? k0 + s / (float)n : 0.f;
                }
            }
            if (lane == 0 && n > 0) {
                const int i = g - g0;
                long long tn = table.n[i];
                float tm = __int_as_float(table.moments[i].x), t2 = __int_as_float(table.moments[i].y);
                chan(tn, tm, t2, n, gm, s);
                table.n[i] = tn;
                table.moments[i] = make_int2(__float_as_int(tm), __float_as_int(t2));
            }
        }
    }
    __syncthreads();
    if (VEC > 1 && warp == 0) {
        for (unsigned left = __ballot_sync(0xffffffffu, edge_group >= g0 && edge_group < g1); left; left &= left - 1) {
            const int from = __ffs(left) - 1, i = __shfl_sync(0xffffffffu, edge_group, from) - g0;
            const float v = __shfl_sync(0xffffffffu, edge, from);
            if (lane == 0) {
                long long tn = table.n[i];
                float tm = __int_as_float(table.moments[i].x), t2 = __int_as_float(table.moments[i].y);
                chan(tn, tm, t2, 1, v, 0.f);
                table.n[i] = tn;
                table.moments[i] = make_int2(__float_as_int(tm), __float_as_int(t2));
            }
        }
        __syncwarp();
    }
    if (p.cluster > 1) cluster_sync();
    else __syncthreads();
    GnPartial* const out = p.partials + ((int64_t)u.p * p.N + u.n) * G * TB_GN_PARTS;
    for (int i = u.rank * CL_BLOCK + (int)threadIdx.x; i < gs; i += p.cluster * CL_BLOCK) {
        long long n = 0;
        float mean = 0.f, m2 = 0.f;
        for (int r = 0; r < p.cluster; ++r) {
            long long bn;
            int2 bm;
            if (r == u.rank) {
                bn = table.n[i];
                bm = table.moments[i];
            } else {
                const uint2 c = cluster_load8(smem_addr(table.n + i), (uint32_t)r);
                const uint2 m = cluster_load8(smem_addr(table.moments + i), (uint32_t)r);
                bn = (long long)(((unsigned long long)c.y << 32) | c.x);
                bm = make_int2((int)m.x, (int)m.y);
            }
            chan(n, mean, m2, bn, __int_as_float(bm.x), __int_as_float(bm.y));
        }
        GnPartial* const at = out + (int64_t)(g0 + i) * TB_GN_PARTS;
        if (!in_bounds(at, TB_GN_PARTS * sizeof(GnPartial), p.partials,
                       (int64_t)p.P * p.N * G * TB_GN_PARTS * (int64_t)sizeof(GnPartial), p.status))
            continue;
        at[u.part] = GnPartial{n, mean, m2};
        if (u.part == 0)
            for (int r = parts; r < TB_GN_PARTS; ++r) at[r] = GnPartial{0, 0.f, 0.f};
    }
    if (p.cluster > 1) cluster_sync();  // nobody leaves while its table may be read
}

size_t stats_smem(int vec, int groups) { return (size_t)CL_BLOCK * vec * 8 + CL_BLOCK * 4 + (size_t)groups * 16; }

// --- normalisation ------------------------------------------------------------------

constexpr int AU = 4;  // chunks a thread loads together

template <bool SILU>
__device__ __forceinline__ f32x2 act(f32x2 z) {
    if constexpr (SILU) {
        float zl, zh, tl, th;
        halves(z, zl, zh);
        halves(vmul(z, pair(-1.4426950408889634f, -1.4426950408889634f)), tl, th);
        float al, ah;
        halves(vadd(pair(ex2_ftz(tl), ex2_ftz(th)), pair(1.f, 1.f)), al, ah);
        return vmul(z, pair(rcp_ftz(al), rcp_ftz(ah)));
    } else {
        return z;
    }
}
template <bool SILU>
__device__ __forceinline__ float act(float z) {
    return SILU ? z * rcp_ftz(1.f + ex2_ftz(z * -1.4426950408889634f)) : z;
}

template <int DT, int VEC, bool SILU>
__global__ void __launch_bounds__(CL_BLOCK, 3) gncl_apply_kernel(const __grid_constant__ GnClParams p) {
    using L = Lanes<VEC>;
    using W = ClWord<DT, VEC>;
    constexpr int ES = elem_size(DT), NL = L::N;
    extern __shared__ uint4 shared4[];
    float2* const stats = reinterpret_cast<float2*>(shared4);  // [G]
    const int C = (int)p.C, K = C / p.G;
    int pt = 0;
    while (pt + 1 < p.P && (int)blockIdx.x >= p.start[pt + 1]) ++pt;
    const int local = (int)blockIdx.x - p.start[pt], n = local / p.parts[pt], piece = local - n * p.parts[pt];
    const ClRun run = cl_run<ES, VEC>(p.patches[pt], p.spatial[pt], p.C, n);
    const char* const patch = static_cast<const char*>(p.patches[pt]);
    char* const out = static_cast<char*>(p.outs[pt]);
    const int64_t bytes = p.N * run.elems * ES, from = (run.first + run.head) * ES;
    const int j0 = (int)blockIdx.y * p.columns, j1 = min(j0 + p.columns, p.period);
    const ClPlace q = cl_place(j0, j1);
    int64_t a, b;
    cl_piece((run.chunks + p.period - 1) / p.period, piece, p.parts[pt], a, b);
    const ClWalk w = cl_walk(q, a, b, p.period, run.chunks);
    grid_wait();
    // this thread's channels
    float fm[VEC], fa[VEC], fb[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        const int c = cl_channel(run.head, q.col * VEC + i, C);
        fa[i] = weight_at(p.gamma, DT, c, 1.f);
        fb[i] = weight_at(p.beta, DT, c, 0.f);
    }
    cl_group_stats(p, n, 0, p.G, stats);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        const float2 s = stats[cl_channel(run.head, q.col * VEC + i, C) / K];
        fm[i] = s.x;
        fa[i] *= s.y;
    }
    typename L::T mean[NL], ga[NL], be[NL];
    cl_lanes<VEC>(fm, mean);
    cl_lanes<VEC>(fa, ga);
    cl_lanes<VEC>(fb, be);
    // from the end of the run: the statistics left that in L2
    const W* const base = reinterpret_cast<const W*>(patch + from) + w.at;
    W* const to = reinterpret_cast<W*>(out + from) + w.at;
    for (int s = w.count - 1; s >= 0; s -= AU) {
        W v[AU];
#pragma unroll
        for (int r = 0; r < AU; ++r)
            if (s - r >= 0 && in_bounds(base + (s - r) * w.stride, sizeof(W), patch, bytes, p.status))
                v[r] = __ldcs(base + (s - r) * w.stride);
#pragma unroll
        for (int r = 0; r < AU; ++r) {
            if (s - r >= 0) {
                typename L::T f[NL];
                to_lanes<DT, VEC>(v[r], f);
#pragma unroll
                for (int i = 0; i < NL; ++i) f[i] = act<SILU>(vfma(vsub(f[i], mean[i]), ga[i], be[i]));
                if (in_bounds(to + (s - r) * w.stride, sizeof(W), out, bytes, p.status))
                    __stcs(to + (s - r) * w.stride, from_lanes<DT, VEC>(f));
            }
        }
    }
    if (VEC > 1 && blockIdx.y == 0) {
        const int h = piece == 0 ? run.head : 0, t = piece == p.parts[pt] - 1 ? run.tail : 0;
        if ((int)threadIdx.x < h + t) {
            const int64_t e = (int)threadIdx.x < h ? threadIdx.x : run.elems - run.tail + (threadIdx.x - h);
            const int c = (int)(e % C);
            const float2 s = stats[c / K];
            if (in_bounds(patch + (run.first + e) * ES, ES, patch, bytes, p.status)) {
                const float d = cl_elem<DT>(patch, run.first + e) - s.x;
                const float z = fmaf(d, s.y * weight_at(p.gamma, DT, c, 1.f), weight_at(p.beta, DT, c, 0.f));
                cl_store_elem<DT>(out, run.first + e, act<SILU>(z));
            }
        }
    }
}

template <int DT>
cudaError_t stats_launch(const GnClParams& p, bool vector, int64_t ctas, cudaStream_t s) {
    constexpr int V = 16 / elem_size(DT);
    void (*const fn)(const GnClParams) = vector ? gncl_stats_kernel<DT, V> : gncl_stats_kernel<DT, 1>;
    return launch_cluster(fn, p, dim3((unsigned)ctas, (unsigned)p.splits, 1), p.cluster,
                          stats_smem(vector ? V : 1, p.G / p.splits), s);
}

template <int DT>
cudaError_t apply_launch(const GnClParams& p, bool vector, int64_t ctas, cudaStream_t s) {
    constexpr int V = 16 / elem_size(DT);
    void (*const fn)(const GnClParams) =
        vector ? (p.silu ? gncl_apply_kernel<DT, V, true> : gncl_apply_kernel<DT, V, false>)
               : (p.silu ? gncl_apply_kernel<DT, 1, true> : gncl_apply_kernel<DT, 1, false>);
    const unsigned slabs = (unsigned)((p.period + p.columns - 1) / p.columns);
    return launch_cluster(fn, p, dim3((unsigned)ctas, slabs, 1), 1, (size_t)p.G * sizeof(float2), s);
}

}  // namespace

cudaError_t launch_gncl_stats(const GnClParams& p, int dtype, bool vector, int64_t ctas, cudaStream_t s) {
    if (dtype == F32) return stats_launch<F32>(p, vector, ctas, s);
    if (dtype == F16) return stats_launch<F16>(p, vector, ctas, s);
    return stats_launch<BF16>(p, vector, ctas, s);
}

cudaError_t launch_gncl_apply(const GnClParams& p, int dtype, bool vector, int64_t ctas, cudaStream_t s) {
    if (dtype == F32) return apply_launch<F32>(p, vector, ctas, s);
    if (dtype == F16) return apply_launch<F16>(p, vector, ctas, s);
    return apply_launch<BF16>(p, vector, ctas, s);
}

}  // namespace tb
