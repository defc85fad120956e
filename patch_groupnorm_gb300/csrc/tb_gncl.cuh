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

__device__ __forceinline__ ClPlace cl_place(const GnClParams& p, int j0, int j1) {
    ClPlace q;
    q.width = j1 - j0;
    q.rows = (int)blockDim.x / p.columns;  // of every slab, the last and narrower one too
    q.row = (int)threadIdx.x / q.width;
    q.col = j0 + (int)threadIdx.x - q.row * q.width;
    if (q.row >= q.rows) q.row = -1;
    return q;
}

// The chunks of this thread: `count` of them, `stride` chunks apart, the first at
// chunk `at`.
struct ClWalk {
    int64_t at, stride;
    int32_t count;
};

// Rows dealt out in turn: piece i of `pieces` takes `rows` of them, then the pieces
// after it, so that neighbouring CTAs read neighbouring addresses.
__device__ __forceinline__ ClWalk cl_walk_dealt(const ClPlace& q, int i, int pieces, int period, int64_t chunks) {
    ClWalk w;
    w.at = ((int64_t)i * q.rows + q.row) * period + q.col;
    w.stride = (int64_t)pieces * q.rows * period;
    w.count = 0;
    if (q.row >= 0 && w.at < chunks) {
        const uint64_t left = (uint64_t)(chunks - w.at - 1);
        // a 64-bit division is a hundred instructions
        w.count = (int32_t)(left >> 32 || w.stride >> 32 ? left / (uint64_t)w.stride
                                                         : (uint32_t)left / (uint32_t)w.stride) + 1;
    }
    return w;
}

// The same for piece i of `pieces` of a statistics pass, whose share of blocks (rows
// side by side) the host has counted from a sample that starts on a boundary; another
// may have a chunk less, in its last row.
__device__ __forceinline__ ClWalk cl_walk_share(const GnClParams& prm, const ClPlace& q, int p, int i, int pieces,
                                                int64_t chunks) {
    ClWalk w;
    w.at = ((int64_t)i * q.rows + q.row) * prm.period + q.col;
    w.stride = (int64_t)pieces * q.rows * prm.period;
    w.count = q.row >= 0 ? prm.share[p] + (i < prm.extra[p] ? 1 : 0) : 0;
    if (w.count > 0 && w.at + (w.count - 1) * w.stride >= chunks) --w.count;
    return w;
}

// The piece that has the sample's last block, and with it its tail.
__device__ __forceinline__ int cl_last_piece(const GnClParams& prm, int p, int pieces) {
    return (prm.extra[p] > 0 ? prm.extra[p] : pieces) - 1;
}

// --- a thread's chunks, in flight ahead of their use --------------------------------

// NS tensors' chunks of one walk: DEPTH - 1 of each are on their way while one is in
// work.  16-byte chunks go through the thread's own slots in shared memory
// (cp.async: no registers are held, no barrier is needed; with 4 or 8 chunks loaded
// into registers at a time the forward pass of 256 x 256 x 512 bf16 took 49 us, not
// 38), single elements through registers.  A slot is filled again only one step after
// its chunk was read, when that chunk's values are in use.  step() is called with r =
// the step modulo DEPTH, a constant once the caller's loop is unrolled.
template <int DT, int VEC, int NS, int DEPTH>
struct ClStream {
    using W = ClWord<DT, VEC>;
    static constexpr int D = DEPTH, N = NS;
    static constexpr size_t SMEM = VEC > 1 ? (size_t)DEPTH * NS * CL_BLOCK * 16 : 0;
    const char* at[NS];
    const char* base[NS];
    int64_t stride, bytes;  // from chunk to chunk; of a tensor (bounds-checked build)
    int32_t left;           // chunks still to fetch
    uint32_t slot;          // shared address of this thread's first slot
    uint32_t* status;
    W reg[VEC > 1 ? 1 : DEPTH][NS];

    // SURE: the caller knows that there is one more
    template <bool SURE = false>
    __device__ __forceinline__ void fetch(int r) {
        if (SURE || left > 0) {
#pragma unroll
            for (int k = 0; k < NS; ++k) {
                if (in_bounds(at[k], sizeof(W), base[k], bytes, status)) {
                    if constexpr (VEC > 1) {
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                                         slot + (uint32_t)((r * NS + k) * CL_BLOCK * 16)),
                                     "l"(at[k])
                                     : "memory");
                    } else {
                        reg[r][k] = *reinterpret_cast<const W*>(at[k]);
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
    // whether the next DEPTH steps each fetch another chunk
    __device__ __forceinline__ bool full() const { return left >= DEPTH; }
    template <bool SURE = false>
    __device__ __forceinline__ void step(int r, W (&v)[NS]) {
        if constexpr (VEC > 1) {
            asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH - 2) : "memory");
            fetch<SURE>((r + DEPTH - 1) % DEPTH);
#pragma unroll
            for (int k = 0; k < NS; ++k) v[k] = smem_load<W>(slot + (uint32_t)((r * NS + k) * CL_BLOCK * 16));
        } else {
#pragma unroll
            for (int k = 0; k < NS; ++k) v[k] = reg[r][k];
            fetch<SURE>((r + DEPTH - 1) % DEPTH);
        }
    }
};

// The next `count` chunks (at most the whole turns of DEPTH that precede another
// call, or the rest): body(v, k) for chunk k of them.
template <typename Stream, typename Body>
__device__ __forceinline__ void cl_each(Stream& in, int count, Body&& body) {
    constexpr int D = Stream::D, NS = Stream::N;
    typename Stream::W v[NS];
    int k = 0;
    for (; k + D <= count && in.full(); k += D) {
#pragma unroll
        for (int r = 0; r < D; ++r) {
            in.template step<true>(r, v);
            body(v, k + r);
        }
    }
    for (; k < count; k += D) {
#pragma unroll
        for (int r = 0; r < D; ++r) {
            if (k + r < count) {
                in.step(r, v);
                body(v, k + r);
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

// (n, mean, M2) joined with (bn, bmean, bm2), Chan's way.  Counts are floats, exact up
// to 2^24 elements: they weigh means and squares here; a record's own count comes
// from the sizes.
__device__ __forceinline__ void chan(float& n, float& mean, float& m2, float bn, float bmean, float bm2) {
    const float total = n + bn;
    const float f = bn > 0.f ? __fdividef(bn, total) : 0.f;  // 1, exactly, where n is 0
    const float d = n > 0.f && bn > 0.f ? bmean - mean : 0.f;
    mean = n > 0.f ? fmaf(d, f, mean) : bmean;
    m2 += fmaf(d * d, n * f, bn > 0.f ? bm2 : 0.f);
    n = total;
}

// --- a thread's statistics --------------------------------------------------------

// (mean, M2) of each of a thread's VEC channels, with the sums of what came since:
// x - k and (x - k)^2, k the channel's first value, then its mean so far.
template <int DT, int VEC>
struct ClMoments {
    using L = Lanes<VEC>;
    using T = typename L::T;
    static constexpr int NL = L::N;
    T k[NL], s1[NL], s2[NL], mean[NL], m2[NL];

    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < NL; ++i) k[i] = mean[i] = m2[i] = s1[i] = s2[i] = L::splat(0.f);
    }
    __device__ __forceinline__ void add(const ClWord<DT, VEC>& v, bool first) {
        T f[NL];
        to_lanes<DT, VEC>(v, f);
        if (first) {
#pragma unroll
            for (int i = 0; i < NL; ++i) k[i] = mean[i] = f[i];
        }
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            const T d = vsub(f[i], k[i]);
            s1[i] = vadd(s1[i], d);
            s2[i] = vfma(d, d, s2[i]);
        }
    }
    // The sums of the last `now` chunks join those of `done` before (Chan).
    __device__ __forceinline__ void fold(int done, int now) {
        const float nb = (float)now, total = (float)(done + now);
        const T inv = L::splat(1.f / nb), f = L::splat(nb / total), g = L::splat((float)done * (nb / total));
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            const T d1 = vmul(s1[i], inv);  // mean - k
            const T bm2 = vsub(s2[i], vmul(s1[i], d1));
            const T bmean = vadd(k[i], d1), d = vsub(bmean, mean[i]);
            mean[i] = vfma(d, f, mean[i]);
            m2[i] = vadd(m2[i], vfma(vmul(d, d), g, bm2));
            k[i] = mean[i];
            s1[i] = s2[i] = L::splat(0.f);
        }
    }
    // Into shared memory: `unit` neighbouring channels, which are one group's, as one.
    __device__ __forceinline__ void store_units(int count, int unit, float* stage_mean, float* stage_m2) const {
        float fm[VEC], f2[VEC];
        cl_values<VEC>(mean, fm);
        cl_values<VEC>(m2, f2);
        // rounding may leave a tiny negative sum of squares: it is a zero one
#pragma unroll
        for (int i = 0; i < VEC; ++i) f2[i] = f2[i] < 0.f ? 0.f : f2[i];
#pragma unroll
        for (int d = 1; d < VEC; d *= 2) {
            if (d < unit) {  // their counts are equal
                const float half = 0.5f * (float)(count * d);
#pragma unroll
                for (int i = 0; i < VEC; i += 2 * d) {
                    const float away = fm[i + d] - fm[i];
                    fm[i] = fmaf(0.5f, away, fm[i]);
                    f2[i] = f2[i] + f2[i + d] + half * away * away;
                }
            }
        }
        const int each = VEC / unit;
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            if (i % unit == 0) {
                stage_mean[threadIdx.x * each + i / unit] = fm[i];
                stage_m2[threadIdx.x * each + i / unit] = f2[i];
            }
        }
    }
    // Into shared memory, two sums: of the first `in_first` lanes, which are one group's, and
    // of the others, which are the next one's (their counts are equal).
    __device__ __forceinline__ void store_pairs(int count, int in_first, float* stage_mean, float* stage_m2) const {
        float fm[VEC], f2[VEC];
        cl_values<VEC>(mean, fm);
        cl_values<VEC>(m2, f2);
        float s0 = 0.f, s1_ = 0.f, q0 = 0.f, q1 = 0.f;
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            s0 += i < in_first ? fm[i] - fm[0] : 0.f;
            s1_ += i < in_first ? 0.f : fm[i] - fm[VEC - 1];
        }
        const float m0 = fm[0] + __fdividef(s0, (float)in_first);
        const float m1 = in_first < VEC ? fm[VEC - 1] + __fdividef(s1_, (float)(VEC - in_first)) : 0.f;
        const float n = (float)count;
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            // rounding may have left a tiny negative sum of squares: it is a zero one
            const float d = fm[i] - (i < in_first ? m0 : m1), q = fmaf(n * d, d, f2[i] < 0.f ? 0.f : f2[i]);
            q0 += i < in_first ? q : 0.f;
            q1 += i < in_first ? 0.f : q;
        }
        stage_mean[threadIdx.x * 2] = m0;
        stage_mean[threadIdx.x * 2 + 1] = m1;
        stage_m2[threadIdx.x * 2] = q0;
        stage_m2[threadIdx.x * 2 + 1] = q1;
    }
};

// What a thread leaves of a chunk: one sum for every `unit` lanes, the largest power of
// two that divides a group's channels and the elements before the first chunk; where
// that is less than half a chunk and a group has at least a chunk's channels, two sums,
// of the lanes of either group (each lane's alone took 2.3 us to join, 1.2 with two).
__device__ __forceinline__ int cl_unit_channels(int VEC, int K, int head) { return min(VEC, (K | head) & -(K | head)); }
__device__ __forceinline__ bool cl_in_pairs(int VEC, int K, int unit) { return VEC > 2 && unit * 2 < VEC && K >= VEC; }

// Lanes of a chunk at column `col` that belong to its first channel's group.
__device__ __forceinline__ int cl_in_first(int VEC, int head, int col, int C, int K) {
    int c = head + col * VEC;
    if (c >= C) c %= C;
    return min(VEC, K - c % K);
}

// Sums of a pair over `team` neighbouring threads (a power of two, the same for all
// threads of the CTA), for every one of them; teams of several warps meet in `warps`
// [blockDim / 32].
__device__ __forceinline__ float2 cl_team_sum(float a, float b, int team, float2* warps) {
    for (int d = min(team, 32) / 2; d >= 1; d >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, d);
        b += __shfl_xor_sync(0xffffffffu, b, d);
    }
    if (team > 32) {
        __syncthreads();  // whoever read them before is done
        if ((threadIdx.x & 31) == 0) warps[threadIdx.x >> 5] = make_float2(a, b);
        __syncthreads();
        const int first = (int)(threadIdx.x & ~(unsigned)(team - 1)) >> 5;
        a = b = 0.f;
        for (int w = 0; w < team >> 5; ++w) {
            a += warps[first + w].x;
            b += warps[first + w].y;
        }
    }
    return make_float2(a, b);
}

// The staged sums of groups g0 .. g0 + gs - 1 join those groups' entries of `table`
// (count, mean, M2).  The lanes of a row that are one group's lie in phases [head + j0 *
// VEC, head + j1 * VEC), in runs of at most K.  A team of threads joins a group: the
// mean about one of its means, then squares about that mean, corrected by what it was
// off (it may come from a value far from all others).  PAIRS: two sums a chunk.
template <int VEC, bool PAIRS>
__device__ __forceinline__ void cl_join_groups(const ClPlace& q, int head, int j0, int j1, int unit, int C, int K, int g0,
                                               int gs, const float* stage_mean, const float* stage_m2,
                                               const int* stage_n, float2* warps, float4* table) {
    // in units of lanes (PAIRS: in lanes)
    const int log2_unit = PAIRS ? 0 : 31 - __clz(unit), log2_each = (VEC == 8 ? 3 : VEC == 4 ? 2 : 0) - log2_unit;
    const int lo = (head + j0 * VEC) >> log2_unit, hi = (head + j1 * VEC) >> log2_unit, pitch = q.width << log2_each;
    const int Ku = K >> log2_unit, Cu = C >> log2_unit;
    // a warp to a group; more where that leaves threads idle and has much to add up
    int team = 32;
    while (team > 1 && gs * team > (int)blockDim.x) team >>= 1;
    while (gs * team * 2 <= (int)blockDim.x && q.rows * (PAIRS ? q.width : pitch) > gs * team * 8) team <<= 1;
    const int lane = threadIdx.x & (team - 1);
    for (int first = 0; first < gs; first += (int)blockDim.x / team) {
        const int i = first + (int)threadIdx.x / team, c0 = (g0 + i) * Ku;
        const int m_first = lo >= c0 + Ku ? (lo - c0 - Ku) / Cu + 1 : 0;
        // body(entry, its elements), for each of this thread's
        auto each = [&](auto&& body) {
            if (i >= gs) return;
            for (int m = m_first; c0 + m * Cu < hi; ++m) {
                const int start = c0 + m * Cu - lo, from = max(start, 0), to = min(start + Ku, hi - lo);
                // PAIRS: the run's chunks; its first one begins with another group's lanes if the
                // run starts inside it
                const int at0 = PAIRS ? from / VEC : from, len = (PAIRS ? (to + VEC - 1) / VEC : to) - at0;
                const float per = __fdividef(1.f, (float)len);
                for (int e = lane; e < q.rows * len; e += team) {
                    // e / len: both below 2^13, so half a step keeps the product from the borders
                    const int row = (int)(((float)e + 0.5f) * per), at = at0 + e - row * len;
                    if constexpr (PAIRS) {
                        const int t = row * q.width + at, lanes = min(to, at * VEC + VEC) - max(from, at * VEC);
                        body(t * 2 + (start > at * VEC ? 1 : 0), (float)(stage_n[t] * lanes));
                    } else {
                        body(row * pitch + at, (float)stage_n[(row * pitch + at) >> log2_each]);
                    }
                }
            }
        };
        float k0 = 0.f;
        if (i < gs && c0 + m_first * Cu < hi) {
            const int start = c0 + m_first * Cu - lo, from = max(start, 0);
            k0 = stage_mean[PAIRS ? from / VEC * 2 + (start > from / VEC * VEC ? 1 : 0) : from];
        }
        float n = 0.f, s = 0.f;
        each([&](int at, float ni) {
            n += ni;
            s = fmaf(ni, stage_mean[at] - k0, s);
        });
        const float2 ns = cl_team_sum(n, s, team, warps);
        const float inv = ns.x > 0.f ? 1.f / ns.x : 0.f, mean = fmaf(ns.y, inv, k0);
        float off = 0.f, m2 = 0.f;
        each([&](int at, float ni) {
            const float d = stage_mean[at] - mean;
            off = fmaf(ni, d, off);
            m2 += fmaf(ni * d, d, ni > 0.f ? stage_m2[at] : 0.f);
        });
        const float2 om = cl_team_sum(off, m2, team, warps);
        if (i < gs && lane == 0 && ns.x > 0.f) {
            const float by = om.x * inv, left = fmaf(-om.x, by, om.y);
            float4 t = table[i];
            chan(t.x, t.y, t.z, ns.x, mean + by, left < 0.f ? 0.f : left);
            table[i] = t;
        }
    }
}

// A thread's sums into shared memory, and from there into the table.
template <int DT, int VEC>
__device__ __forceinline__ void cl_join(const ClMoments<DT, VEC>& sums, int count, const ClPlace& q, int head, int j0,
                                        int j1, int C, int K, int g0, int gs, float* stage_mean, float* stage_m2,
                                        int* stage_n, float2* warps, float4* table) {
    const int unit = cl_unit_channels(VEC, K, head);
    if (cl_in_pairs(VEC, K, unit)) {
        sums.store_pairs(count, cl_in_first(VEC, head, q.col, C, K), stage_mean, stage_m2);
        stage_n[threadIdx.x] = count;
        __syncthreads();
        cl_join_groups<VEC, true>(q, head, j0, j1, unit, C, K, g0, gs, stage_mean, stage_m2, stage_n, warps, table);
    } else {
        sums.store_units(count, unit, stage_mean, stage_m2);
        stage_n[threadIdx.x] = count * unit;
        __syncthreads();
        cl_join_groups<VEC, false>(q, head, j0, j1, unit, C, K, g0, gs, stage_mean, stage_m2, stage_n, warps, table);
    }
}

// --- thread-block clusters ------------------------------------------------------

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync() {
    cluster_arrive();
    cluster_wait();
}
// 8 bytes of shared memory of CTA `rank` of this cluster, at this CTA's address `at`.
__device__ __forceinline__ uint2 cluster_load8(uint32_t at, uint32_t rank) {
    uint32_t far;
    uint2 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(far) : "r"(at), "r"(rank));
    asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(far) : "memory");
    return v;
}

// 16 bytes.
__device__ __forceinline__ float4 cluster_load16(uint32_t at, uint32_t rank) {
    uint32_t far;
    float4 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(far) : "r"(at), "r"(rank));
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(far)
                 : "memory");
    return v;
}

// (count, mean, M2) of entry `i` of the cluster's tables, for each of its team of eight
// threads, one for each CTA.
__device__ __forceinline__ float4 cl_join_cluster(const float4* table, int i, int gs, int cluster) {
    static_assert(CL_MAX_CLUSTER == 8, "eight threads read the CTAs' sums");
    const int r = threadIdx.x & 7;
    float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
    if (i < gs && r < cluster) t = cluster > 1 ? cluster_load16(smem_addr(table + i), (uint32_t)r) : table[i];
    const float k0 = __shfl_sync(0xffffffffu, t.y, threadIdx.x & 24);
    float n = t.x, s = t.x > 0.f ? t.x * (t.y - k0) : 0.f;
#pragma unroll
    for (int d = 4; d >= 1; d >>= 1) {
        n += __shfl_xor_sync(0xffffffffu, n, d);
        s += __shfl_xor_sync(0xffffffffu, s, d);
    }
    const float inv = n > 0.f ? 1.f / n : 0.f, mean = fmaf(s, inv, k0), d = t.y - mean;
    float off = t.x > 0.f ? t.x * d : 0.f, m2 = t.x > 0.f ? fmaf(t.x * d, d, t.z) : 0.f;
#pragma unroll
    for (int k = 4; k >= 1; k >>= 1) {
        off += __shfl_xor_sync(0xffffffffu, off, k);
        m2 += __shfl_xor_sync(0xffffffffu, m2, k);
    }
    const float by = off * inv, left = fmaf(-off, by, m2);
    return make_float4(n, mean + by, left < 0.f ? 0.f : left, 0.f);
}

// The (patch, sample, part) of a statistics CTA, its rank in the part's cluster, its
// piece of the sample's rows, and its slab of the columns.  Clusters are numbered
// patch by patch, then sample, then part; in a cluster the slabs run fastest.
struct ClUnit {
    int p, part, rank;
    int piece, pieces;  // of the sample's rows
    int slab;
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
    const int each = prm.cluster / prm.slabs;
    u.piece = u.part * each + u.rank / prm.slabs;
    u.pieces = prm.parts[u.p] * each;
    u.slab = u.rank % prm.slabs;
    return u;
}

// (mean, rstd) of groups [g0, g1) of sample n into out[0 .. g1 - g0): eight
// threads to a group, four of whose record sets are on their way at once (a wait for
// one after the other would hold the CTA up for microseconds).  A NaN stays one.
__device__ __forceinline__ void cl_group_stats(const GnClParams& p, int64_t n, int g0, int g1, float2* out) {
    static_assert(TB_GN_PARTS == 8, "a thread takes one part of every set");
    constexpr int B = 4;
    const int part = threadIdx.x & 7, teams = (int)blockDim.x >> 3;
    const int64_t set = p.N * p.G * TB_GN_PARTS;
    for (int first = g0; first < g1; first += teams) {
        const int g = first + ((int)threadIdx.x >> 3);
        const GnPartial* const unit = p.partials + (n * p.G + g) * TB_GN_PARTS + part;
        float c = 0.f, m = 0.f, m2 = 0.f;
        for (int r0 = 0; r0 < p.R; r0 += B) {
            longlong2 raw[B];
#pragma unroll
            for (int k = 0; k < B; ++k) {
                const GnPartial* const at = unit + (r0 + k) * set;
                raw[k] = make_longlong2(0, 0);
                if (g < g1 && r0 + k < p.R &&
                    in_bounds(at, sizeof(GnPartial), p.partials, p.R * set * (int64_t)sizeof(GnPartial), p.status))
                    raw[k] = *reinterpret_cast<const longlong2*>(at);
            }
#pragma unroll
            for (int k = 0; k < B; ++k)
                chan(c, m, m2, (float)raw[k].x, __int_as_float((int)(raw[k].y & 0xffffffffLL)),
                     __int_as_float((int)(raw[k].y >> 32)));
        }
#pragma unroll
        for (int d = 4; d >= 1; d >>= 1) {
            const float bc = __shfl_down_sync(0xffffffffu, c, d), bm = __shfl_down_sync(0xffffffffu, m, d);
            chan(c, m, m2, bc, bm, __shfl_down_sync(0xffffffffu, m2, d));
        }
        if (g < g1 && part == 0) {
            const float var = c > 0.f ? m2 / c : 0.f;  // biased: divided by the count
            out[g - g0] = make_float2(m, 1.0f / sqrtf(var + p.eps));
        }
    }
}

// A thread's channels, one after the other: the channel and its group.
struct ClChannel {
    int c, g, k;  // channel, group, place in the group
    int C, K;
    __device__ __forceinline__ ClChannel(int head, int phase, int C_, int K_) : C(C_), K(K_) {
        c = head + phase;
        if (c >= C) c %= C;
        g = c / K;
        k = c - g * K;
    }
    __device__ __forceinline__ void next() {
        ++c;
        if (++k == K) {
            k = 0;
            ++g;
        }
        if (c == C) c = g = 0;
    }
};

// gamma's or beta's value for channel c, and a weight's gradient; w is null where the call
// has none.
template <int DT>
__device__ __forceinline__ float cl_weight(const GnClParams& p, const void* w, int64_t c, float dflt) {
    return index_ok(c >= 0 && c < p.C, p.status) ? weight_at(w, DT, c, dflt) : dflt;
}
template <int DT>
__device__ __forceinline__ void cl_store_weight(const GnClParams& p, void* w, int64_t c, float v) {
    if (w != nullptr && index_ok(c >= 0 && c < p.C, p.status)) store_weight(w, DT, c, v);
}

// gamma and beta of a thread's VEC channels: one load each where they lie together.
template <int DT, int VEC>
__device__ __forceinline__ void cl_weights(const GnClParams& p, int head, int phase, float (&ga)[VEC], float (&be)[VEC]) {
    int c0 = head + phase;
    if (c0 >= p.C) c0 %= (int)p.C;
    if (VEC > 1 && c0 % VEC == 0 && c0 + VEC <= p.C &&
        ((reinterpret_cast<uintptr_t>(p.gamma) | reinterpret_cast<uintptr_t>(p.beta)) & 15u) == 0) {
        weights_at<VEC>(p.gamma, DT, c0, 1.f, ga);
        weights_at<VEC>(p.beta, DT, c0, 0.f, be);
    } else {
        ClChannel ch(head, phase, (int)p.C, 1);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            ga[i] = cl_weight<DT>(p, p.gamma, ch.c, 1.f);
            be[i] = cl_weight<DT>(p, p.beta, ch.c, 0.f);
            ch.next();
        }
    }
}

// --- the activation -------------------------------------------------------------------

// silu(z), or z.
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

// dz = dy * silu'(z), or dy.  e^-z and the reciprocal are approximate (2^-22 each);
// e^-z overflows for z < -88, where s = 0 and dz = 0.
template <bool SILU>
__device__ __forceinline__ f32x2 dz_of(f32x2 dy, f32x2 z) {
    if constexpr (SILU) {
        const f32x2 one = pair(1.f, 1.f);
        float tl, th, al, ah;
        halves(vmul(z, pair(-1.4426950408889634f, -1.4426950408889634f)), tl, th);
        halves(vadd(pair(ex2_ftz(tl), ex2_ftz(th)), one), al, ah);
        const f32x2 s = pair(rcp_ftz(al), rcp_ftz(ah));
        return vmul(dy, vmul(s, vfma(z, vsub(one, s), one)));
    } else {
        return dy;
    }
}
template <bool SILU>
__device__ __forceinline__ float dz_of(float dy, float z) {
    if constexpr (SILU) {
        const float s = rcp_ftz(1.f + ex2_ftz(z * -1.4426950408889634f));
        return dy * (s * fmaf(z, 1.f - s, 1.f));
    } else {
        return dy;
    }
}

// One element, as the elements of head and tail are read and written; `bytes` of a
// tensor (bounds-checked build).
template <int DT>
__device__ __forceinline__ float cl_elem(const void* base, int64_t i, int64_t bytes, uint32_t* status) {
    const ClWord<DT, 1>* const at = reinterpret_cast<const ClWord<DT, 1>*>(base) + i;
    return in_bounds(at, sizeof(*at), base, bytes, status) ? elem_to_f<DT>(*at) : 0.f;
}
template <int DT>
__device__ __forceinline__ void cl_store_elem(void* base, int64_t i, float v, int64_t bytes, uint32_t* status) {
    ClWord<DT, 1>* const at = reinterpret_cast<ClWord<DT, 1>*>(base) + i;
    float f[1] = {v};
    if (in_bounds(at, sizeof(*at), base, bytes, status)) *at = pack<DT, 1>(f);
}

// Launches `fn` with programmatic stream serialisation in clusters of `cluster` CTAs.
// A kernel that needs more shared memory than the default is given the limit of the
// largest call: calls of other threads may set it between this one's two steps.
inline cudaError_t launch_cluster(void (*fn)(const GnClParams), const GnClParams& p, dim3 grid, int cluster, size_t smem,
                                  cudaStream_t s, int block = CL_BLOCK) {
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, CL_MAX_SMEM);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)block, 1, 1);
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
