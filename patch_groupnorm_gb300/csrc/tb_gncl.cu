// tb_gncl.cu -- PatchGroupNorm (+ SiLU) of channels-last patches: statistics
// records, and the normalisation.
//
// y = silu(d * a + beta), d = x - mean, a = rstd * gamma, with mean and rstd of
// the group pooled over the patches.  Subtracting the mean first keeps what a
// single x * a + b would lose where the mean is far from zero.
//
// Statistics need all of a group before the first output, so x is read twice, by
// two launches (where it fits into shared memory, once: tb_gncl_fused.cu).  1 x 256 x
// 256 x 512 bf16 in four patches takes 37.7 us, 16.3 of them the statistics; 67 MB
// read twice and written once are 29.7 us at the copy rate.  What is left is the start
// and the end of each launch: sums joined over rows, groups and clusters, a latency
// after the other (3 us), and the groups' pooled statistics before the first output
// (2 us).  13 x 120 x 208 x 384: 126 us, of 110 at that rate; the channels-first kernels
// take 114 for the same bytes, so a tenth is these kernels' own.
//
// Statistics grids: 288 CTAs in clusters of 3 for four patches on 152 SMs; 256 in
// clusters of 8 took 18.8 us for the first and 50.8 for the second (16.3, 43), 304
// that find no room at once 23 and 65.  Splits of the channels down to 64 bytes a
// position cost nothing (16.1 us), of 32 bytes 20.4.
#include "tb_gncl.cuh"

namespace tb {
namespace {

// --- statistics -------------------------------------------------------------------

constexpr int FOLD = 64;  // chunks between two foldings of a thread's sums
constexpr int DEPTH = 8;  // chunks of a thread on their way or in work

// Each thread sums x - K and (x - K)^2 of its VEC channels on packed pairs, K its
// own first value, then its mean so far; after DEPTH, DEPTH, 2 DEPTH, 4 DEPTH, ... and
// then every FOLD chunks the sums are merged into (mean, M2) (Chan), so that neither a far mean
// nor a long run loses digits, nor a first value far from all others: n chunks
// about a mean that it has moved by 1 / n of its distance add 1 / n of its square.
// A CTA's threads meet in shared memory, group by group, and the CTAs of a
// cluster read each other's tables, in a fixed order: one record per cluster.
template <int DT, int VEC>
__global__ void __launch_bounds__(CL_BLOCK, 3) gncl_stats_kernel(const __grid_constant__ GnClParams p) {
    using W = ClWord<DT, VEC>;
    constexpr int ES = elem_size(DT);
    extern __shared__ uint4 shared4[];
    using Stream = ClStream<DT, VEC, 1, DEPTH>;
    float* const stage_mean = reinterpret_cast<float*>(shared4 + Stream::SMEM / 16);  // [CL_BLOCK * VEC]
    float* const stage_m2 = stage_mean + CL_BLOCK * VEC;
    int* const stage_n = reinterpret_cast<int*>(stage_m2 + CL_BLOCK * VEC);  // [CL_BLOCK]
    const int C = (int)p.C, G = p.G, K = p.K;
    const int gs = G / p.splits, g0 = (int)blockIdx.y * gs, g1 = g0 + gs;  // this CTA's groups
    float2* const warps = reinterpret_cast<float2*>(stage_n + CL_BLOCK);     // [CL_BLOCK / 32]
    float4* const table = reinterpret_cast<float4*>(warps + CL_BLOCK / 32);  // [gs]: (count, mean, M2)
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int i = threadIdx.x; i < gs; i += CL_BLOCK) table[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    const ClUnit u = cl_unit(p);
    const int parts = p.parts[u.p], piece = u.piece, pieces = u.pieces, last = cl_last_piece(p, u.p, pieces);
    const ClRun run = cl_run<ES, VEC>(p.patches[u.p], p.spatial[u.p], p.C, u.n);
    const char* const patch = static_cast<const char*>(p.patches[u.p]);
    const int64_t bytes = p.N * run.elems * ES;
    grid_wait();

    // elements outside the whole chunks: the first piece's before, the last one's after; a lane each
    float edge = 0.f;
    int edge_group = -1;
    if (VEC > 1 && warp == 0) {
        const int h = piece == 0 && u.slab == 0 ? run.head : 0, t = piece == last && u.slab == 0 ? run.tail : 0;
        if (lane < h + t) {
            const int64_t e = lane < h ? lane : run.elems - run.tail + (lane - h);
            edge = cl_elem<DT>(patch, run.first + e, bytes, p.status);
            edge_group = (int)(e % C) / K;
        }
    }

    const int split_width = p.period / p.splits, split0 = (int)blockIdx.y * split_width;
    for (int j0 = split0 + u.slab * p.columns; j0 < split0 + split_width; j0 += p.slabs * p.columns) {
        const int j1 = min(j0 + p.columns, split0 + split_width);
        const ClPlace q = cl_place(p, j0, j1);
        const ClWalk w = cl_walk_share(p, q, u.p, piece, pieces, run.chunks);
        ClMoments<DT, VEC> sums;
        sums.clear();
        Stream in;
        in.base[0] = patch;
        in.at[0] = patch + (run.first + run.head) * ES + w.at * (int64_t)sizeof(W);
        in.stride = w.stride * (int64_t)sizeof(W);
        in.bytes = bytes;
        in.status = p.status;
        in.start(w.count, shared4);
        for (int done = 0, now; done < w.count; done += now) {
            now = min(min(FOLD, max(DEPTH, done)), w.count - done);
            cl_each(in, now, [&](const W (&v)[1], int j) { sums.add(v[0], done + j == 0); });
            sums.fold(done, now);
        }
        __syncthreads();  // the table is set, or the columns before these are merged
        cl_join(sums, w.count, q, run.head, j0, j1, C, K, g0, gs, stage_mean, stage_m2, stage_n, warps, table);
    }
    __syncthreads();
    if (VEC > 1 && warp == 0) {
        for (unsigned left = __ballot_sync(0xffffffffu, edge_group >= g0 && edge_group < g1); left; left &= left - 1) {
            const int from = __ffs(left) - 1, i = __shfl_sync(0xffffffffu, edge_group, from) - g0;
            const float v = __shfl_sync(0xffffffffu, edge, from);
            if (lane == 0) {
                float4 t = table[i];
                chan(t.x, t.y, t.z, 1.f, v, 0.f);
                table[i] = t;
            }
        }
        __syncwarp();
    }
    if (p.cluster > 1) cluster_sync();
    else __syncthreads();
    // the cluster's tables: eight threads to a group, one for each CTA
    static_assert(TB_GN_PARTS == 8, "the eight threads of a group write its parts");
    // whole rows have reps * K elements of every group; whoever has the last row has
    // whatever the others leave, and the first piece the head's too
    const int reps = (int)((unsigned)(p.period * VEC) / (unsigned)C), slices = p.cluster / p.slabs;
    const int first_piece = u.part * slices, side = CL_BLOCK / p.columns;
    const bool ends = p.rows[u.p] > 0 && last >= first_piece && last < first_piece + slices;
    int64_t whole = ((int64_t)p.share[u.p] * slices + min(max(p.extra[u.p] - first_piece, 0), slices)) * side;
    if (ends) {  // its last block may be short; its last row is counted apart
        const int64_t blocks = (int64_t)p.share[u.p] * pieces + p.extra[u.p];
        whole -= blocks * side - p.rows[u.p] + 1;
    }
    GnPartial* const out = p.partials + ((int64_t)u.p * p.N + u.n) * G * TB_GN_PARTS;
    for (int first = 0; first < gs; first += p.cluster * (CL_BLOCK / 8)) {
        const int i = first + u.rank * (CL_BLOCK / 8) + (int)threadIdx.x / 8, r = threadIdx.x & 7;
        const float4 t = cl_join_cluster(table, i, gs, p.cluster);
        if (i >= gs) continue;
        GnPartial* const at = out + (int64_t)(g0 + i) * TB_GN_PARTS;
        if (!in_bounds(at, TB_GN_PARTS * sizeof(GnPartial), p.partials,
                       (int64_t)p.P * p.N * G * TB_GN_PARTS * (int64_t)sizeof(GnPartial), p.status))
            continue;
        const int c0 = (g0 + i) * K;
        const int64_t ahead = min(max((run.head % C) - c0, 0), K) + (int64_t)(run.head / C) * K;
        int64_t count = whole * reps * K + (u.part == 0 ? ahead : 0);
        if (ends) count += p.spatial[u.p] * K - ahead - (p.rows[u.p] - 1) * reps * K;
        // a sample of less than a chunk has no rows
        if (p.rows[u.p] == 0) count = u.part == 0 ? p.spatial[u.p] * K : 0;
        if (r == 0) at[u.part] = GnPartial{count, t.y, t.z};
        if (u.part == 0 && r >= parts) at[r] = GnPartial{0, 0.f, 0.f};
    }
    if (p.cluster > 1) cluster_sync();  // nobody leaves while its table may be read
}

template <int DT, int VEC>
size_t stats_smem(int groups) {
    return ClStream<DT, VEC, 1, DEPTH>::SMEM + CL_BLOCK * VEC * 8 + CL_BLOCK * 4 + CL_BLOCK / 4 + (size_t)groups * 16;
}

// --- normalisation ------------------------------------------------------------------

// As DEPTH.  Two CTAs per SM; 8 chunks and two, or 6 and three, take 88 us for 13 x 120 x
// 208 x 384 bf16 alone, 6 and two 79: reads and writes together want fewer on their way.
// Single elements are small, and no load moves ahead of the stores between them: with 6,
// 8, 10, 12 and 16 the whole call takes 62.5, 56.3, 54.0, 54.2 and 50.3 us for 65536 x 512
// bf16 at offsets of 0, 1 and 2 elements, 137, 125, 118, 112 and 114 for 3 x 24568 x 515 f32.
template <int VEC>
constexpr int APPLY_DEPTH = VEC > 1 ? 6 : 16;

template <int DT, int VEC, bool SILU>
__global__ void __launch_bounds__(CL_BLOCK, 3) gncl_apply_kernel(const __grid_constant__ GnClParams p) {
    using L = Lanes<VEC>;
    using W = ClWord<DT, VEC>;
    constexpr int ES = elem_size(DT), NL = L::N;
    extern __shared__ uint4 shared4[];
    using Stream = ClStream<DT, VEC, 1, APPLY_DEPTH<VEC>>;
    float2* const stats = reinterpret_cast<float2*>(shared4 + Stream::SMEM / 16);  // [G]
    const int C = (int)p.C, K = p.K;
    int pt = 0;
    while (pt + 1 < p.P && (int)blockIdx.x >= p.start[pt + 1]) ++pt;
    const int local = (int)blockIdx.x - p.start[pt], n = local / p.parts[pt], piece = local - n * p.parts[pt];
    const ClRun run = cl_run<ES, VEC>(p.patches[pt], p.spatial[pt], p.C, n);
    const char* const patch = static_cast<const char*>(p.patches[pt]);
    char* const out = static_cast<char*>(p.outs[pt]);
    const int64_t bytes = p.N * run.elems * ES, from = (run.first + run.head) * ES;
    const int j0 = (int)blockIdx.y * p.columns, j1 = min(j0 + p.columns, p.period);
    const ClPlace q = cl_place(p, j0, j1);
    const ClWalk w = cl_walk_dealt(q, piece, p.parts[pt], p.period, run.chunks);
    // from the end: the statistics left that in L2
    const int64_t last = from + (w.at + (w.count - 1) * w.stride) * (int64_t)sizeof(W);
    Stream in;
    in.base[0] = patch;
    in.at[0] = patch + last;
    in.stride = -w.stride * (int64_t)sizeof(W);
    in.bytes = bytes;
    in.status = p.status;
    grid_wait();
    in.start(w.count, shared4);
    // this thread's channels
    float fm[VEC], fa[VEC], fb[VEC];
    cl_weights<DT, VEC>(p, run.head, q.col * VEC, fa, fb);
    cl_group_stats(p, n, 0, p.G, stats);
    __syncthreads();
    ClChannel ch(run.head, q.col * VEC, C, K);
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        const float2 s = stats[ch.g];
        fm[i] = s.x;
        fa[i] *= s.y;
        ch.next();
    }
    typename L::T mean[NL], ga[NL], be[NL];
    cl_lanes<VEC>(fm, mean);
    cl_lanes<VEC>(fa, ga);
    cl_lanes<VEC>(fb, be);
    char* to = out + last;
    cl_each(in, w.count, [&](const W (&v)[1], int) {
        typename L::T f[NL];
        to_lanes<DT, VEC>(v[0], f);
#pragma unroll
        for (int i = 0; i < NL; ++i) f[i] = act<SILU>(vfma(vsub(f[i], mean[i]), ga[i], be[i]));
        if (in_bounds(to, sizeof(W), out, bytes, p.status)) __stcs(reinterpret_cast<W*>(to), from_lanes<DT, VEC>(f));
        to += in.stride;
    });
    if (VEC > 1 && blockIdx.y == 0) {
        const int h = piece == 0 ? run.head : 0, t = piece == p.parts[pt] - 1 ? run.tail : 0;
        if ((int)threadIdx.x < h + t) {
            const int64_t e = (int)threadIdx.x < h ? threadIdx.x : run.elems - run.tail + (threadIdx.x - h);
            const int c = (int)(e % C);
            const float2 s = stats[c / K];
            const float d = cl_elem<DT>(patch, run.first + e, bytes, p.status) - s.x;
            const float z = fmaf(d, s.y * cl_weight<DT>(p, p.gamma, c, 1.f), cl_weight<DT>(p, p.beta, c, 0.f));
            cl_store_elem<DT>(out, run.first + e, act<SILU>(z), bytes, p.status);
        }
    }
}

template <int DT>
cudaError_t stats_launch(const GnClParams& p, bool vector, int64_t ctas, cudaStream_t s) {
    constexpr int V = 16 / elem_size(DT);
    void (*const fn)(const GnClParams) = vector ? gncl_stats_kernel<DT, V> : gncl_stats_kernel<DT, 1>;
    return launch_cluster(fn, p, dim3((unsigned)ctas, (unsigned)p.splits, 1), p.cluster,
                          vector ? stats_smem<DT, V>(p.G / p.splits) : stats_smem<DT, 1>(p.G / p.splits), s);
}

template <int DT>
cudaError_t apply_launch(const GnClParams& p, bool vector, int64_t ctas, cudaStream_t s) {
    constexpr int V = 16 / elem_size(DT);
    void (*const fn)(const GnClParams) =
        vector ? (p.silu ? gncl_apply_kernel<DT, V, true> : gncl_apply_kernel<DT, V, false>)
               : (p.silu ? gncl_apply_kernel<DT, 1, true> : gncl_apply_kernel<DT, 1, false>);
    const unsigned slabs = (unsigned)((p.period + p.columns - 1) / p.columns);
    const size_t ring = vector ? ClStream<DT, V, 1, APPLY_DEPTH<V>>::SMEM : 0;
    return launch_cluster(fn, p, dim3((unsigned)ctas, slabs, 1), 1, ring + (size_t)p.G * sizeof(float2), s);
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
