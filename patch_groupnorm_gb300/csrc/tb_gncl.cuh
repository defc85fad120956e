// tb_gncl.cuh -- what the forward and backward kernels of channels-last
// PatchGroupNorm share: how a sample's elements are cut into chunks, columns
// and rows, and the tables that the CTAs of a cluster merge.
//
// A sample of a patch is one dense run of spatial * C elements.  From its first
// 16-byte boundary on it is read in whole 16-byte chunks (VEC elements); the
// elements before that boundary and after the last whole chunk (`head` and
// `tail`, fewer than VEC each) are taken one by one.  Chunk q holds the elements
// head + q * VEC ..., so its channels repeat with period C / gcd(C, VEC) chunks,
// whatever C is: a thread that keeps to one column of that period keeps its
// VEC channels, and their constants and sums stay in its registers.  A row is
// one period of chunks (a whole position, where VEC divides C); a CTA reads
// rows side by side, so its accesses are contiguous.  VEC is 1 where the
// tensors of a call lie at different offsets from 16-byte boundaries.
#pragma once

#include "tb_elem.cuh"
#include "tb_groupnorm.cuh"

namespace tb {

// A chunk as it is loaded.
template <int DT, int VEC>
using ClWord = typename Word<VEC * elem_size(DT)>::T;

// One sample of one patch.
struct ClRun {
    int64_t first;   // its first element, counted in the patch
    int64_t elems;   // spatial * C
    int64_t chunks;  // whole chunks
    int32_t head, tail;
};

template <int ES, int VEC>
__device__ __forceinline__ ClRun cl_run(const void* patch, int64_t spatial, int64_t C, int64_t n) {
    ClRun r;
    r.elems = spatial * C;
    r.first = n * r.elems;
    if constexpr (VEC == 1) {
        r.head = r.tail = 0;
        r.chunks = r.elems;
    } else {
        const uintptr_t at = reinterpret_cast<uintptr_t>(patch) + (uintptr_t)r.first * ES;
        const int64_t head = (int64_t)((16u - (unsigned)(at & 15u)) & 15u) / ES;
        r.head = (int32_t)(head < r.elems ? head : r.elems);
        r.chunks = (r.elems - r.head) / VEC;
        r.tail = (int32_t)(r.elems - r.head - r.chunks * VEC);
    }
    return r;
}

// A thread's place among the columns [j0, j1) of the period.
struct ClPlace {
    int32_t width, rows;  // columns, and rows side by side
    int32_t row, col;     // this thread's (row < 0: none)
};

__device__ __forceinline__ ClPlace cl_place(int j0, int j1) {
    ClPlace q;
    q.width = j1 - j0;
    q.rows = CL_BLOCK / q.width;
    q.row = (int)threadIdx.x / q.width;
    q.col = j0 + (int)threadIdx.x - q.row * q.width;
    if (q.row >= q.rows) q.row = -1;
    return q;
}

// The chunks of this thread in rows [a, b): `count` of them, `stride` chunks
// apart, the first at chunk `at`.
struct ClWalk {
    int64_t at, stride;
    int32_t count;
};

__device__ __forceinline__ ClWalk cl_walk(const ClPlace& q, int64_t a, int64_t b, int period, int64_t chunks) {
    ClWalk w;
    w.at = (a + q.row) * period + q.col;
    w.stride = (int64_t)q.rows * period;
    w.count = 0;
    if (q.row >= 0 && a + q.row < b) {
        w.count = (int32_t)((b - a - q.row + q.rows - 1) / q.rows);
        // only the sample's last row may be cut short
        if (w.at + (w.count - 1) * w.stride >= chunks) --w.count;
    }
    return w;
}

// Rows [a, b) of piece i of `pieces` (rows < 2^47, pieces < 2^16).
__device__ __forceinline__ void cl_piece(int64_t rows, int i, int pieces, int64_t& a, int64_t& b) {
    a = rows * i / pieces;
    b = rows * (i + 1) / pieces;
}

__device__ __forceinline__ int cl_channel(int head, int phase, int C) { return (head + phase) % C; }

// --- a thread's chunks, in flight ahead of their use --------------------------------

// NS tensors' chunks of one walk: DEPTH - 1 of each are on their way while one is in
// work.  16-byte chunks go through the thread's own slots in shared memory
// (cp.async: no registers are held, no barrier is needed), single elements through
// registers.  A slot is filled again only one step after its chunk was read, when
// that chunk's values are in use.  step() is called with r = the step modulo DEPTH,
// a constant once the caller's loop is unrolled.
template <int DT, int VEC, int NS, int DEPTH>
struct ClStream {
    using W = ClWord<DT, VEC>;
    static constexpr size_t SMEM = VEC > 1 ? (size_t)DEPTH * NS * CL_BLOCK * 16 : 0;
    const char* at[NS];
    const char* base[NS];
    int64_t stride, bytes;  // from chunk to chunk; of a tensor (bounds-checked build)
    int32_t left;           // chunks still to fetch
    uint32_t slot;          // shared address of this thread's first slot
    uint32_t* status;
    W reg[VEC > 1 ? 1 : DEPTH][NS];

    __device__ __forceinline__ void fetch(int r) {
        if (left > 0) {
#pragma unroll
            for (int k = 0; k < NS; ++k) {
                if (in_bounds(at[k], sizeof(W), base[k], bytes, status)) {
                    if constexpr (VEC > 1) {
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                                         slot + (uint32_t)((r * NS + k) * CL_BLOCK * 16)),
                                     "l"(at[k])
                                     : "memory");
                    } else {
                        reg[r][k] = __ldg(reinterpret_cast<const W*>(at[k]));
                    }
                }
                at[k] += stride;
            }
        }
        --left;
        if constexpr (VEC > 1) asm volatile("cp.async.commit_group;" ::: "memory");
    }
    __device__ __forceinline__ void start(int count, void* ring) {
        left = count;
        slot = smem_addr(ring) + threadIdx.x * 16;
#pragma unroll
        for (int r = 0; r < DEPTH - 1; ++r) fetch(r);
    }
    __device__ __forceinline__ void step(int r, W (&v)[NS]) {
        if constexpr (VEC > 1) {
            asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH - 2) : "memory");
            fetch((r + DEPTH - 1) % DEPTH);
#pragma unroll
            for (int k = 0; k < NS; ++k) v[k] = smem_load<W>(slot + (uint32_t)((r * NS + k) * CL_BLOCK * 16));
        } else {
#pragma unroll
            for (int k = 0; k < NS; ++k) v[k] = reg[r][k];
            fetch((r + DEPTH - 1) % DEPTH);
        }
    }
};

// --- thread-block clusters ------------------------------------------------------

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// 8 bytes of shared memory of CTA `rank` of this cluster, at this CTA's address `at`.
__device__ __forceinline__ uint2 cluster_load8(uint32_t at, uint32_t rank) {
    uint32_t far;
    uint2 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(far) : "r"(at), "r"(rank));
    asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(far) : "memory");
    return v;
}

// The (patch, sample, part) and place of a statistics CTA.  Clusters are
// numbered patch by patch, then sample, then part.
struct ClUnit {
    int p, part, rank;
    int64_t n;
};

__device__ __forceinline__ ClUnit cl_unit(const GnClParams& prm) {
    const int cluster = (int)blockIdx.x / prm.cluster;
    ClUnit u;
    u.rank = (int)blockIdx.x - cluster * prm.cluster;
    u.p = 0;
    while (u.p + 1 < prm.P && cluster >= prm.start[u.p + 1]) ++u.p;
    const int local = cluster - prm.start[u.p];
    u.n = local / prm.parts[u.p];
    u.part = local - (int)u.n * prm.parts[u.p];
    return u;
}

// (mean, rstd) of groups [g0, g1) of sample n into out[0 .. g1 - g0), a group per
// warp at a time: each record (count c, mean m, M2) adds c, c * (m - K) and
// M2 + c * (m - K)^2 to sums about K, the mean of the first record with elements,
// as the channels-first kernels pool them; unlike there, a NaN stays one.  Four
// groups' records (32 of them: a load per lane) are on their way together, since a
// wait for one group after the other would hold the CTA up for microseconds.
__device__ __forceinline__ void cl_group_stats(const GnClParams& p, int64_t n, int g0, int g1, float2* out) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = (int)blockDim.x >> 5;
    const int total = p.R * TB_GN_PARTS;
    constexpr int B = 4;
    auto record = [&](int g, int q, long long& c, float& m, float& m2) {
        c = 0;
        m = m2 = 0.f;
        if (g >= g1 || q >= total) return;
        const GnPartial* const at = p.partials + (((int64_t)(q / TB_GN_PARTS) * p.N + n) * p.G + g) * TB_GN_PARTS +
                                    q % TB_GN_PARTS;
        if (!in_bounds(at, sizeof(GnPartial), p.partials,
                       (int64_t)p.R * p.N * p.G * TB_GN_PARTS * (int64_t)sizeof(GnPartial), p.status))
            return;
        const longlong2 raw = __ldg(reinterpret_cast<const longlong2*>(at));
        c = raw.x;
        m = __int_as_float((int)(raw.y & 0xffffffffLL));
        m2 = __int_as_float((int)(raw.y >> 32));
    };
    for (int first = g0 + warp; first < g1; first += warps * B) {
        long long c[B];
        float m[B], m2[B];
#pragma unroll
        for (int k = 0; k < B; ++k) record(first + k * warps, lane, c[k], m[k], m2[k]);
#pragma unroll
        for (int k = 0; k < B; ++k) {
            const int g = first + k * warps;
            if (g >= g1) break;
            unsigned has = __ballot_sync(0xffffffffu, c[k] > 0);
            float K = has ? __shfl_sync(0xffffffffu, m[k], __ffs(has) - 1) : 0.f;
            for (int base = 32; has == 0u && base < total; base += 32) {
                long long oc;
                float om, o2;
                record(g, base + lane, oc, om, o2);
                has = __ballot_sync(0xffffffffu, oc > 0);
                if (has) K = __shfl_sync(0xffffffffu, om, __ffs(has) - 1);
            }
            long long sn = 0;
            float s1 = 0.f, s2 = 0.f;
            auto add = [&](long long rc, float rm, float r2) {
                if (rc > 0) {
                    const float cf = (float)rc, d = rm - K;
                    sn += rc;
                    s1 = fmaf(cf, d, s1);
                    s2 += fmaf(cf * d, d, r2);
                }
            };
            add(c[k], m[k], m2[k]);
            for (int q = 32 + lane; q < total; q += 32) {
                long long oc;
                float om, o2;
                record(g, q, oc, om, o2);
                add(oc, om, o2);
            }
#pragma unroll
            for (int delta = 16; delta >= 1; delta >>= 1) {  // fixed order: deterministic
                sn += __shfl_down_sync(0xffffffffu, sn, delta);
                s1 += __shfl_down_sync(0xffffffffu, s1, delta);
                s2 += __shfl_down_sync(0xffffffffu, s2, delta);
            }
            if (lane == 0) {
                const float nf = (float)sn;
                const float q1 = sn > 0 ? s1 / nf : 0.f;
                float var = sn > 0 ? fmaf(-s1, q1, s2) / nf : 0.f;  // biased: divided by the count
                if (var < 0.f) var = 0.f;
                out[g - g0] = make_float2(K + q1, 1.0f / sqrtf(var + p.eps));
            }
        }
    }
}

// VEC values of a thread's channels as lanes.
template <int VEC>
__device__ __forceinline__ void cl_lanes(const float (&f)[VEC], typename Lanes<VEC>::T (&l)[Lanes<VEC>::N]) {
    if constexpr (VEC == 1) {
        l[0] = f[0];
    } else {
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) l[i] = pair(f[2 * i], f[2 * i + 1]);
    }
}
template <int VEC>
__device__ __forceinline__ void cl_values(const typename Lanes<VEC>::T (&l)[Lanes<VEC>::N], float (&f)[VEC]) {
    if constexpr (VEC == 1) {
        f[0] = l[0];
    } else {
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) halves(l[i], f[2 * i], f[2 * i + 1]);
    }
}

// One element, as the elements of head and tail are read and written.
template <int DT>
__device__ __forceinline__ float cl_elem(const void* base, int64_t i) {
    if constexpr (DT == F32) return reinterpret_cast<const float*>(base)[i];
    else return elem_to_f<DT>(reinterpret_cast<const unsigned short*>(base)[i]);
}
template <int DT>
__device__ __forceinline__ void cl_store_elem(void* base, int64_t i, float v) {
    float f[1] = {v};
    reinterpret_cast<ClWord<DT, 1>*>(base)[i] = pack<DT, 1>(f);
}

// Shared memory of the largest call (CL_MAXC channels in as many groups).  A kernel
// that needs more than the default is given this limit whatever the call's size:
// calls of other threads may set it between this one's two steps.
constexpr int CL_MAX_SMEM = 216 * 1024;

// Launches `fn` with programmatic stream serialisation in clusters of `cluster` CTAs.
inline cudaError_t launch_cluster(void (*fn)(const GnClParams), const GnClParams& p, dim3 grid, int cluster, size_t smem,
                                  cudaStream_t s) {
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, CL_MAX_SMEM);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(CL_BLOCK, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, fn, p);
}

}  // namespace tb
