// tb_gncl_fused.cu -- channels-last PatchGroupNorm in one launch, forward and
// backward, where the tensors fit into shared memory.
//
// A cluster of up to eight CTAs takes one sample's groups, or as many of them as
// whole chunks allow (a split), of all patches.  Its CTAs copy their chunks of x (and
// of dy) into shared memory once, sum them as they arrive, read each other's sums
// (one barrier of the cluster), and go over the same chunks again from shared
// memory: every tensor is read once, and what two or three launches of the general
// path spend on starting and on waiting for each other is spent once.  Chunks are a
// thread's own from its copy to its result, so the copies need no barrier.
//
// What bounds it is latency: 2 patches of 15 x 16 x 64 bf16 take 5.5 us (backward 6.5; in
// several launches 7.7 and 10.3), 64 x 64 x 512 8.9 (11.4): starting, the
// first chunks' way, and the joining of sums, some 2000 instructions a warp of which
// few overlap.
//
// Taken where every patch starts on 16 bytes, samples and splits are whole chunks, and
// all clusters find room at once (cl_plan_fused).
#include "tb_gncl.cuh"

namespace tb {
namespace {

template <int N>
struct Count {
    static constexpr int value = N;
};

// A thread's chunks of all patches, in the order in which they are copied: chunk k of
// NS tensors in slots k * NS .. of its column of the ring.
template <int NS>
struct ClHeld {
    const GnClParams& p;
    ClPlace q;
    int slice;               // this CTA's blocks of rows: slice, slice + slices, ...
    int stride;              // chunks from one of them to the next
    uint32_t slot;
    int count;               // chunks
    int sure;                // of these, known to have arrived

    // Calls body(patch, chunk of the sample, k, count) for every chunk, or pair of
    // chunks `stride` apart: count is a constant of 1 or 2.
    template <typename Body>
    __device__ __forceinline__ void each(Body&& body) {
        const int first = (slice * q.rows + q.row) * p.period + q.col;
        int k = 0;
        if (q.row >= 0) {
            for (int pt = 0; pt < p.P; ++pt) {
                const int chunks = p.start[pt];
                int at = first;
                for (; at + stride < chunks; at += 2 * stride, k += 2) body(pt, at, k, Count<2>());
                if (at < chunks) body(pt, at, k++, Count<1>());
            }
        }
        count = k;
    }
    // Chunk k has arrived: waits in steps, as the number of copies that may still be
    // on their way is part of the instruction.
    __device__ __forceinline__ void arrived(int k) {
        if (k < sure) return;
        const int after = count - k - 1;
        if (after >= 16) {
            asm volatile("cp.async.wait_group 16;" ::: "memory");
            sure = count - 16;
        } else if (after >= 8) {
            asm volatile("cp.async.wait_group 8;" ::: "memory");
            sure = count - 8;
        } else if (after >= 4) {
            asm volatile("cp.async.wait_group 4;" ::: "memory");
            sure = count - 4;
        } else {
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            sure = count;
        }
    }
    __device__ __forceinline__ uint32_t at(int k, int tensor) const {
        return slot + (uint32_t)((k * NS + tensor) * (int)blockDim.x * 16);
    }
};

__device__ __forceinline__ void copy16(uint32_t to, const char* from, const char* base, int64_t bytes, uint32_t* status) {
    if (in_bounds(from, 16, base, bytes, status))
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }

// Where a CTA stands: grid.x is the rank in the cluster (the slabs of the split's
// columns, then the slices of the rows), grid.y the split, grid.z the sample.
struct ClSeat {
    int64_t n;
    int split, rank, g0, gs, j0, j1;
    template <int NS>
    __device__ __forceinline__ static ClSeat take(const GnClParams& p, void* ring, ClHeld<NS>& held) {
        ClSeat s;
        s.rank = (int)blockIdx.x;
        s.n = blockIdx.z;
        s.split = (int)blockIdx.y;
        s.gs = p.parts[0];
        s.g0 = s.split * s.gs;
        const int width = p.parts[1], first = s.split * width;
        const int slice = p.slabs == 1 ? s.rank : s.rank / p.slabs;
        s.j0 = first + (s.rank - slice * p.slabs) * p.columns;
        s.j1 = min(s.j0 + p.columns, first + width);
        held.q = cl_place(p, s.j0, s.j1);
        held.slice = slice;
        held.stride = p.share[0] * held.q.rows * p.period;
        held.slot = smem_addr(ring) + threadIdx.x * 16;
        held.sure = 0;
        return s;
    }
};

// --- forward ------------------------------------------------------------------------

template <int DT, bool SILU, int BLOCK>
__global__ void __launch_bounds__(BLOCK, 512 / BLOCK) gncl_fused_kernel(const __grid_constant__ GnClParams p) {
    constexpr int ES = elem_size(DT), VEC = 16 / ES;
    using L = Lanes<VEC>;
    using W = ClWord<DT, VEC>;
    constexpr int NL = L::N;
    extern __shared__ uint4 shared4[];
    float* const stage_mean = reinterpret_cast<float*>(shared4 + p.held * BLOCK);  // [BLOCK * VEC]
    float* const stage_m2 = stage_mean + BLOCK * VEC;                              // [BLOCK * VEC]
    int* const stage_n = reinterpret_cast<int*>(stage_m2 + BLOCK * VEC);           // [BLOCK]
    float2* const warps = reinterpret_cast<float2*>(stage_n + BLOCK);              // [BLOCK / 32]
    float4* const table = reinterpret_cast<float4*>(warps + BLOCK / 32);           // [gs]: (count, mean, M2)
    const int C = (int)p.C, K = p.K;
    ClHeld<1> held{p};
    const ClSeat seat = ClSeat::take(p, shared4, held);
    float4* const stats = table + seat.gs;                                         // [gs]: (mean, rstd, M2)
    for (int i = threadIdx.x; i < seat.gs; i += BLOCK) table[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    grid_wait();
    held.each([&](int pt, int at, int k, auto count) {
        const char* const patch = static_cast<const char*>(p.patches[pt]);
        const int64_t bytes = p.spatial[pt] * C * ES;
        const char* const from = patch + seat.n * bytes + (int64_t)at * 16;
#pragma unroll
        for (int j = 0; j < decltype(count)::value; ++j) {
            copy16(held.at(k + j, 0), from + (int64_t)j * held.stride * 16, patch, p.N * bytes, p.status);
            copies_end();
        }
    });
    float fm[VEC], fa[VEC], fb[VEC];
    cl_weights<DT, VEC>(p, 0, held.q.col * VEC, fa, fb);
    ClMoments<DT, VEC> sums;
    sums.clear();
    for (int done = 0, now; done < held.count; done += now) {
        now = min(max(8, done), held.count - done);
        for (int k = done; k < done + now; ++k) {
            held.arrived(k);
            sums.add(smem_load<W>(held.at(k, 0)), k == 0);
        }
        sums.fold(done, now);
    }
    cl_join(sums, held.count, held.q, 0, seat.j0, seat.j1, C, K, seat.g0, seat.gs, stage_mean, stage_m2, stage_n, warps,
            table);
    if (p.cluster > 1) cluster_sync();
    else __syncthreads();
    // every CTA joins all of its split's groups for itself
    for (int first = 0; first < seat.gs; first += BLOCK / 8) {
        const int i = first + (int)threadIdx.x / 8;
        const float4 t = cl_join_cluster(table, i, seat.gs, p.cluster);
        if (i < seat.gs && (threadIdx.x & 7) == 0) {
            const float var = t.x > 0.f ? t.z / t.x : 0.f;  // biased: divided by the count
            stats[i] = make_float4(t.y, rsqrtf(var + p.eps), t.z, 0.f);
        }
    }
    if (p.cluster > 1) cluster_arrive();  // this CTA has read the others' tables
    __syncthreads();
    ClChannel ch(0, held.q.col * VEC, C, K);
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        const float4 s = held.q.row >= 0 ? stats[ch.g - seat.g0] : make_float4(0.f, 0.f, 0.f, 0.f);
        fm[i] = s.x;
        fa[i] *= s.y;
        ch.next();
    }
    typename L::T mean[NL], ga[NL], be[NL];
    cl_lanes<VEC>(fm, mean);
    cl_lanes<VEC>(fa, ga);
    cl_lanes<VEC>(fb, be);
    held.each([&](int pt, int at, int k, auto count) {
        constexpr int N = decltype(count)::value;
        typename L::T f[N][NL];
#pragma unroll
        for (int j = 0; j < N; ++j) to_lanes<DT, VEC>(smem_load<W>(held.at(k + j, 0)), f[j]);
#pragma unroll
        for (int j = 0; j < N; ++j) {
#pragma unroll
            for (int i = 0; i < NL; ++i) f[j][i] = act<SILU>(vfma(vsub(f[j][i], mean[i]), ga[i], be[i]));
        }
        char* const out = static_cast<char*>(p.outs[pt]);
        const int64_t bytes = p.spatial[pt] * C * ES;
        char* const to = out + seat.n * bytes + (int64_t)at * 16;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            char* const here = to + (int64_t)j * held.stride * 16;
            if (in_bounds(here, 16, out, p.N * bytes, p.status)) *reinterpret_cast<W*>(here) = from_lanes<DT, VEC>(f[j]);
        }
    });
    if (seat.rank == 0) {  // the records of all patches together are one, the others are empty
        int64_t count = 0;
        for (int pt = 0; pt < p.P; ++pt) count += p.spatial[pt] * K;
        for (int j = threadIdx.x; j < seat.gs * TB_GN_PARTS; j += BLOCK) {
            const float4 t = stats[j / TB_GN_PARTS];
            for (int pt = 0; pt < p.P; ++pt) {
                GnPartial* const at = p.partials + (((int64_t)pt * p.N + seat.n) * p.G + seat.g0) * TB_GN_PARTS + j;
                if (in_bounds(at, sizeof(GnPartial), p.partials,
                              (int64_t)p.P * p.N * p.G * TB_GN_PARTS * (int64_t)sizeof(GnPartial), p.status))
                    *at = pt == 0 && j % TB_GN_PARTS == 0 ? GnPartial{count, t.x, t.z} : GnPartial{0, 0.f, 0.f};
            }
        }
    }
    if (p.cluster > 1) cluster_wait();  // nobody leaves while its table may be read
}

// --- backward -----------------------------------------------------------------------

template <int DT, bool SILU, int BLOCK>
__global__ void __launch_bounds__(BLOCK, 512 / BLOCK) gncl_fused_grad_kernel(const __grid_constant__ GnClParams p) {
    constexpr int ES = elem_size(DT), VEC = 16 / ES;
    using L = Lanes<VEC>;
    using W = ClWord<DT, VEC>;
    constexpr int NL = L::N;
    extern __shared__ uint4 shared4[];
    float2* const stage = reinterpret_cast<float2*>(shared4 + p.held * 2 * BLOCK);  // [BLOCK * VEC]: (sum dz, sum dz * d)
    float2* const table = stage + BLOCK * VEC;                                      // [cs]: (sum dz, sum dz * xhat)
    const int C = (int)p.C, K = p.K;
    ClHeld<2> held{p};
    const ClSeat seat = ClSeat::take(p, shared4, held);
    const int cs = seat.gs * K, c0 = seat.g0 * K;                // the split's channels
    float2* const whole = table + cs;                            // [cs]: the cluster's sums
    float4* const coefs = reinterpret_cast<float4*>(whole + cs); // [gs]: (mean, rstd, u, v)
    float2* const stats = reinterpret_cast<float2*>(coefs + seat.gs);  // [gs]: (mean, rstd)
    for (int i = threadIdx.x; i < cs; i += BLOCK) table[i] = make_float2(0.f, 0.f);
    grid_wait();
    held.each([&](int pt, int at, int k, auto count) {
        const char* const patch = static_cast<const char*>(p.patches[pt]);
        const char* const grad = static_cast<const char*>(p.grads[pt]);
        const int64_t bytes = p.spatial[pt] * C * ES;
#pragma unroll
        for (int j = 0; j < decltype(count)::value; ++j) {
            const int64_t from = seat.n * bytes + (at + (int64_t)j * held.stride) * 16;
            copy16(held.at(k + j, 0), patch + from, patch, p.N * bytes, p.status);
            copy16(held.at(k + j, 1), grad + from, grad, p.N * bytes, p.status);
            copies_end();
        }
    });
    float f0[VEC], f1[VEC], f2[VEC];
    cl_weights<DT, VEC>(p, 0, held.q.col * VEC, f1, f2);
    cl_group_stats(p, seat.n, seat.g0, seat.g0 + seat.gs, stats);
    __syncthreads();
    {
        ClChannel ch(0, held.q.col * VEC, C, K);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const float2 s = held.q.row >= 0 ? stats[ch.g - seat.g0] : make_float2(0.f, 0.f);
            f0[i] = s.x;
            f1[i] *= s.y;
            ch.next();
        }
    }
    typename L::T mean[NL], ga[NL], be[NL], sb[NL], sa[NL];
    cl_lanes<VEC>(f0, mean);
    cl_lanes<VEC>(f1, ga);
    cl_lanes<VEC>(f2, be);
#pragma unroll
    for (int i = 0; i < NL; ++i) sb[i] = sa[i] = L::splat(0.f);
    for (int k = 0; k < held.count; ++k) {
        held.arrived(k);
        typename L::T f[NL], dy[NL];
        to_lanes<DT, VEC>(smem_load<W>(held.at(k, 0)), f);
        to_lanes<DT, VEC>(smem_load<W>(held.at(k, 1)), dy);
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            const typename L::T d = vsub(f[i], mean[i]);
            const typename L::T dz = dz_of<SILU>(dy[i], vfma(d, ga[i], be[i]));
            sb[i] = vadd(sb[i], dz);
            sa[i] = vfma(dz, d, sa[i]);
        }
    }
    {
        float b[VEC], a[VEC];
        cl_values<VEC>(sb, b);
        cl_values<VEC>(sa, a);
#pragma unroll
        for (int i = 0; i < VEC; ++i) stage[threadIdx.x * VEC + i] = make_float2(b[i], a[i]);
    }
    __syncthreads();
    const int lo = seat.j0 * VEC, hi = seat.j1 * VEC, pitch = held.q.width * VEC;
    for (int i = threadIdx.x; i < cs; i += BLOCK) {
        const int c = c0 + i;
        float2 t = make_float2(0.f, 0.f);
        for (int at = c + (lo > c ? (lo - c + C - 1) / C * C : 0); at < hi; at += C) {
            for (int r = 0; r < held.q.rows; ++r) {
                const float2 v = stage[r * pitch + at - lo];
                t.x += v.x;
                t.y += v.y;
            }
        }
        t.y *= stats[i / K].y;
        table[i] = t;
    }
    if (p.cluster > 1) cluster_sync();
    else __syncthreads();
    // every CTA joins all of its split's channels for itself
    for (int i = threadIdx.x; i < cs; i += BLOCK) {
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
        whole[i] = t;
    }
    if (p.cluster > 1) cluster_arrive();  // this CTA has read the others' tables
    __syncthreads();
    // (mean, rstd, u, v) of the groups: eight threads to a group
    int64_t count = 0;
    for (int pt = 0; pt < p.P; ++pt) count += p.spatial[pt] * K;
    const float inv = count > 0 ? 1.f / (float)count : 0.f;
    for (int first = 0; first < seat.gs; first += BLOCK / 8) {
        const int i = first + (int)threadIdx.x / 8;
        float B = 0.f, A = 0.f;
        if (i < seat.gs) {
            for (int j = threadIdx.x & 7; j < K; j += 8) {
                const float w = cl_weight<DT>(p, p.gamma, c0 + i * K + j, 1.f);
                const float2 t = whole[i * K + j];
                B = fmaf(w, t.x, B);
                A = fmaf(w, t.y, A);
            }
        }
#pragma unroll
        for (int d = 4; d >= 1; d >>= 1) {
            B += __shfl_xor_sync(0xffffffffu, B, d);
            A += __shfl_xor_sync(0xffffffffu, A, d);
        }
        if (i < seat.gs && (threadIdx.x & 7) == 0) {
            const float2 s = stats[i];
            coefs[i] = make_float4(s.x, s.y, -(s.y * s.y) * (A * inv), -s.y * (B * inv));
        }
    }
    __syncthreads();
    typename L::T cu[NL], cv[NL];
    {
        float u[VEC], v[VEC];
        ClChannel ch(0, held.q.col * VEC, C, K);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const float4 k = held.q.row >= 0 ? coefs[ch.g - seat.g0] : make_float4(0.f, 0.f, 0.f, 0.f);
            u[i] = k.z;
            v[i] = k.w;
            ch.next();
        }
        cl_lanes<VEC>(u, cu);
        cl_lanes<VEC>(v, cv);
    }
    held.each([&](int pt, int at, int k, auto count) {
        constexpr int N = decltype(count)::value;
        typename L::T f[N][NL], dy[N][NL];
#pragma unroll
        for (int j = 0; j < N; ++j) {
            to_lanes<DT, VEC>(smem_load<W>(held.at(k + j, 0)), f[j]);
            to_lanes<DT, VEC>(smem_load<W>(held.at(k + j, 1)), dy[j]);
        }
#pragma unroll
        for (int j = 0; j < N; ++j) {
#pragma unroll
            for (int i = 0; i < NL; ++i) {
                const typename L::T d = vsub(f[j][i], mean[i]);
                const typename L::T dz = dz_of<SILU>(dy[j][i], vfma(d, ga[i], be[i]));
                f[j][i] = vfma(dz, ga[i], vfma(d, cu[i], cv[i]));
            }
        }
        char* const out = static_cast<char*>(p.outs[pt]);
        const int64_t bytes = p.spatial[pt] * C * ES;
        char* const to = out + seat.n * bytes + (int64_t)at * 16;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            char* const here = to + (int64_t)j * held.stride * 16;
            if (in_bounds(here, 16, out, p.N * bytes, p.status)) *reinterpret_cast<W*>(here) = from_lanes<DT, VEC>(f[j]);
        }
    });
    if (seat.rank == 0 && (p.dgamma != nullptr || p.dbeta != nullptr)) {
        for (int i = threadIdx.x; i < cs; i += BLOCK) {
            const float2 t = whole[i];
            if (p.N == 1) {
                cl_store_weight<DT>(p, p.dgamma, c0 + i, t.y);
                cl_store_weight<DT>(p, p.dbeta, c0 + i, t.x);
                continue;
            }
            // one record a sample, for the launch that adds the samples up
            for (int pt = 0; pt < p.P; ++pt) {
                float2* const at = p.grad_partials + (((int64_t)pt * p.N + seat.n) * C + c0 + i) * TB_GN_PARTS;
                if (!in_bounds(at, TB_GN_PARTS * sizeof(float2), p.grad_partials,
                               (int64_t)p.P * p.N * C * TB_GN_PARTS * (int64_t)sizeof(float2), p.status))
                    continue;
#pragma unroll
                for (int r = 0; r < TB_GN_PARTS; ++r) at[r] = pt == 0 && r == 0 ? t : make_float2(0.f, 0.f);
            }
        }
    }
    if (p.cluster > 1) cluster_wait();  // nobody leaves while its table may be read
}

template <int DT, int BLOCK>
cudaError_t fused_launch(const GnClParams& p, bool grad, cudaStream_t s) {
    const dim3 grid((unsigned)p.cluster, (unsigned)p.splits, (unsigned)p.N);
    void (*const fn)(const GnClParams) =
        grad ? (p.silu ? gncl_fused_grad_kernel<DT, true, BLOCK> : gncl_fused_grad_kernel<DT, false, BLOCK>)
             : (p.silu ? gncl_fused_kernel<DT, true, BLOCK> : gncl_fused_kernel<DT, false, BLOCK>);
    return launch_cluster(fn, p, grid, p.cluster, gncl_fused_smem(p, DT, grad, BLOCK, p.held), s, BLOCK);
}

template <int DT>
cudaError_t fused_launch(const GnClParams& p, bool grad, int block, cudaStream_t s) {
    return block == 512 ? fused_launch<DT, 512>(p, grad, s) : fused_launch<DT, 256>(p, grad, s);
}

}  // namespace

size_t gncl_fused_smem(const GnClParams& p, int dtype, bool grad, int block, int held) {
    const int vec = 16 / elem_size(dtype);
    const size_t gs = (size_t)(p.G / p.splits), cs = (size_t)(p.C / p.splits);
    const size_t stage = (size_t)block * vec * 8;
    return grad ? (size_t)held * 2 * block * 16 + stage + cs * 16 + gs * 24
                : (size_t)held * block * 16 + stage + (size_t)block * 4 + (size_t)block / 4 + gs * 32;
}

cudaError_t launch_gncl_fused(const GnClParams& p, int dtype, bool grad, int block, cudaStream_t s) {
    if (dtype == F32) return fused_launch<F32>(p, grad, block, s);
    if (dtype == F16) return fused_launch<F16>(p, grad, block, s);
    return fused_launch<BF16>(p, grad, block, s);
}

}  // namespace tb
