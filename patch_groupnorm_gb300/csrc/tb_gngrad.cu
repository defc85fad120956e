// tb_gngrad.cu -- the backward pass of PatchGroupNorm (+ SiLU).
//
// With the pooled mean and rstd of the forward pass's records,
// xhat = (x - mean) * rstd, z = xhat * gamma + beta and s = 1 / (1 + e^-z):
//     dz = silu ? dy * s * (1 + z * (1 - s)) : dy
//     B(n, c) = sum dz,  A(n, c) = sum dz * xhat     (over the channel's elements)
//     dgamma(c) = sum_n A,  dbeta(c) = sum_n B
//     c1 = sum over the group's channels of gamma * B / count,  c2 the same of A
//     dx = rnd(rstd * (gamma * dz - c1 - xhat * c2))
// Sums are fp32, in an order fixed by the sizes and the GPU.
//
// dx needs sums over the whole group, so x and dy are read twice, once by each
// of two launches of gn_grad_kernel: GRAD_STATS leaves the records (B, A) of
// every channel, GRAD_APPLY writes dx.  A CTA takes the same contiguous run of
// tasks (some rows of a group, or a part of one) in both, the second time from
// its end, where the first has left its rows in L2 (about 100 MB of them).
// 4D (1 x 512 x 256 x 256 bf16) takes 62.8 us, 5D (1 x 384 x 13 x 120 x 208) 200.
// One launch with both passes interleaved, a group's dx following its records
// by 15 to 60 MB, was built and measured: it reads memory once, but its waits
// cost most of what that saves (61.8 and 184 us).  What bounds 4D is latency,
// neither memory (55 % busy in both passes) nor the issue slots (53 and 45 %): a
// warp has one word of x and dy in work at a time, and a chain of an exponential
// and a reciprocal for each pair of elements.  Without SiLU 4D takes 56.4 us.
// In f32 both passes are near the copy rate (4D 105 us, read twice 100).
// Tensors at different offsets from 16-byte boundaries take the element kernels
// (4D with dy one element off: 253 us).
//
// One CTA per SM: 16 warps compute, a 17th copies the tasks' rows into a ring
// of three stages in shared memory (64 KB each: x and dy), and each stage has a
// warp that finds the unit's and the rows' constants and writes the records
// (chains of dependent loads of about three times a stage's computing time:
// with one warp for everything 4D took 126 us).  Stages of 16 KB a tensor, six
// of them, took 92 us: a stage costs its copying warp 1.2 us whatever its size.
// Bulk copies move whole 16-byte words; the elements before the first and after
// the last boundary are copied one by one, so rows of any length and offset
// take this path.
#include "tb_elem.cuh"
#include "tb_groupnorm.cuh"

namespace tb {
namespace {

constexpr int GG_LOG2 = 4, GG_WARPS = 1 << GG_LOG2;  // computing warps
constexpr int GG_THREADS = GG_WARPS * 32;
constexpr int GG_STAGES = 3;
constexpr int GG_BLOCK = GG_THREADS + 32 * (1 + GG_STAGES);  // + the copying warp, and a warp of constants per stage
// Bytes of x (and of dy) at the end of each CTA's run that L2 is to keep for the
// second launch, 97 MB over 152 CTAs of this GPU's 129; GRAD_STATS reads what
// comes before them evict-first.  (4D / 5D with 192, 256, 320, 384 KB and all
// alike: 63.7 / 200, 62.9 / 199, 62.5 / 199, 62.8 / 200, 63.2 / 206 us: what counts
// is that some are marked, the size within these does not.)
constexpr int64_t GG_KEEP = 320 * 1024;
constexpr int GG_TENSOR = GRAD_STAGE_BYTES + 128;  // room for a first, partial word
constexpr int GG_SMEM = GG_STAGES * 2 * GG_TENSOR;
constexpr int GG_SLOTS = GG_THREADS;               // a lane's sums each, or a warp's of every row
static_assert(GG_SMEM + GG_STAGES * (GG_SLOTS + 64) * 8 <= 224 * 1024, "ring too large");

enum TaskKind : int32_t { TASK_STATS = 0, TASK_APPLY = 1, TASK_WEIGHTS = 2, TASK_END = 3 };

// What the computing warps need of the stage's rows.
struct Stage {
    int32_t kind;
    int32_t rows;        // channel rows in the stage
    int32_t row_elems;   // elements of each (of the part of one) in the stage
    int32_t shift;       // elements before the first in the first word
    int32_t last;        // TASK_STATS: the part ends with this stage
    int32_t slot;        // TASK_STATS: the part's record slot
    int64_t record;      // TASK_STATS: row index p * N * C + n * C + c of the first row; TASK_WEIGHTS: channel
    int32_t n, g;        // sample and group
    int64_t channel;     // of the first row
    char* out;           // TASK_APPLY: address of the first element
    float mean;
    float u, v;          // TASK_APPLY: dx = dz * rstd * gamma + (x - mean) * u + v
    float2 row[GRAD_MAX_ROWS + 1];  // (rstd * gamma, beta) of each row
};

// dz of one pair of elements (see the top of this file).  e^-z and the
// reciprocal are approximate (2^-22 each); e^-z overflows for z < -88, where
// s = 0 and dz = 0 (its true size is below 1e-36 of dy).
template <bool SILU>
__device__ __forceinline__ f32x2 dz_pair(f32x2 u, f32x2 dy, f32x2 za, f32x2 zb) {
    if constexpr (SILU) {
        const f32x2 one = pair(1.f, 1.f);
        const f32x2 z = vfma(u, za, zb);
        float tl, th, al, ah;
        halves(vmul(z, pair(-1.4426950408889634f, -1.4426950408889634f)), tl, th);
        halves(vadd(pair(ex2_ftz(tl), ex2_ftz(th)), one), al, ah);
        const f32x2 s = pair(rcp_ftz(al), rcp_ftz(ah));
        return vmul(dy, vmul(s, vfma(z, vsub(one, s), one)));
    } else {
        return dy;
    }
}

// --- the ring -------------------------------------------------------------------

// The computing warps work in 2^row_groups_log2 groups on a stage's rows, a row
// per group.
__device__ __forceinline__ int row_groups_log2(int rows) { return min(GG_LOG2, 31 - __clz(rows)); }

struct Ring {
    Stage* stage;
    float2* slots;  // [stage][GG_SLOTS]: sums of dz and dz * (x - mean), see compute_loop
    // shared addresses: mbarriers (a stage's task is set; its rows and
    // constants are there; the computing warps are done with it; their sums of
    // one part are there) and the first stage's rows.  All are per stage: a
    // warp may be two stages ahead of another
    uint32_t task, full, empty, sums, data;
    volatile int* dead;          // a wait ran out: everyone leaves
    int s = 0;
    uint32_t parity = 0;
    __device__ __forceinline__ void next() {
        if (++s == GG_STAGES) {
            s = 0;
            parity ^= 1u;
        }
    }
};

// (u, v) of a unit from its records, by one warp: c1 and c2 are its channels'
// sums weighted with gamma, over the count.
__device__ __forceinline__ float2 unit_sums(const GnGradParams& p, int dtype, int64_t n, int64_t g, float rstd,
                                            float count) {
    const uint32_t K = (uint32_t)(p.C / p.G);
    const uint32_t total = (uint32_t)p.R * K * TB_GN_PARTS;
    const float2* const first = p.grad_partials + (n * p.C + g * K) * TB_GN_PARTS;
    const int64_t set = p.N * p.C * TB_GN_PARTS;
    float B = 0.f, A = 0.f;
    for (uint32_t q0 = threadIdx.x & 31; q0 < total; q0 += 4 * 32) {
        float2 v[4];
        float w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {  // all loads before the first sum
            const uint32_t q = q0 + k * 32;
            const uint32_t row = q / TB_GN_PARTS, r = row / K, c = row - r * K;
            v[k] = make_float2(0.f, 0.f);
            w[k] = 0.f;
            if (q < total) {
                v[k] = first[r * set + c * TB_GN_PARTS + q % TB_GN_PARTS];
                w[k] = weight_at(p.gamma, dtype, g * K + c, 1.f);
            }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            B = fmaf(v[k].x, w[k], B);
            A = fmaf(v[k].y, w[k], A);
        }
    }
    return make_float2(-warp_sum(A) / count * rstd * rstd, -warp_sum(B) / count * rstd);
}

// The warp of stage `s`: for every task that comes through the stage, the
// unit's and the rows' constants and, once the computing warps have left their
// sums of a part, its records.
__device__ __forceinline__ void constants_loop(const GnGradParams& p, int dtype, Ring ring, int s) {
    const int lane = threadIdx.x & 31;
    Stage& d = ring.stage[s];
    const uint32_t full = ring.full + s * 8u;
    uint32_t sums_parity = 0;
    // the unit that the constants at hand are of: a CTA's tasks follow each
    // other, so it seldom changes
    int unit_n = -1, unit_g = -1;
    float mean = 0.f, rstd = 0.f;
    float2 uv = make_float2(0.f, 0.f);
    for (uint32_t parity = 0;; parity ^= 1u) {
        bool ok = bar_wait(ring.task + s * 8u, parity, p.status);
        if (__any_sync(0xffffffffu, !ok) || *ring.dead) {
            if (lane == 0) *ring.dead = 1;
            return;
        }
        const int kind = d.kind;
        // (the stage is refilled while the records are written)
        const int rows = d.rows, slot = d.slot;
        const bool last = d.last;
        const int64_t record = d.record;
        if (kind == TASK_END) {
            if (lane == 0) bar_arrive(full);
            return;
        }
        if (kind != TASK_WEIGHTS) {
            const int64_t ch = d.channel + lane;
            const float gamma = lane < rows ? weight_at(p.gamma, dtype, ch, 1.f) : 0.f;
            const float beta = lane < rows ? weight_at(p.beta, dtype, ch, 0.f) : 0.f;
            if (d.n != unit_n || d.g != unit_g) {
                unit_n = d.n;
                unit_g = d.g;
                float count;
                pooled_stats(p, unit_n, unit_g, mean, rstd, count);
                mean = __shfl_sync(0xffffffffu, mean, 0);
                rstd = __shfl_sync(0xffffffffu, rstd, 0);
                count = __shfl_sync(0xffffffffu, count, 0);
                if (kind == TASK_APPLY) uv = unit_sums(p, dtype, unit_n, unit_g, rstd, count);
            }
            if (lane < rows) d.row[lane] = make_float2(rstd * gamma, beta);
            if (lane == 0) {
                d.mean = mean;
                d.u = uv.x;
                d.v = uv.y;
            }
        }
        __syncwarp();
        if (lane == 0) bar_arrive(full);
        if (kind == TASK_STATS && last) {
            ok = bar_wait(ring.sums + s * 8u, sums_parity, p.status);
            sums_parity ^= 1u;
            if (__any_sync(0xffffffffu, !ok)) {
                if (lane == 0) *ring.dead = 1;
                return;
            }
            const float2* const sums = ring.slots + s * GG_SLOTS;
            float2 t = make_float2(0.f, 0.f);
            if (rows == 1) {
#pragma unroll
                for (int w = 0; w < GG_WARPS; ++w) {
                    t.x += sums[w * 32 + lane].x;
                    t.y += sums[w * 32 + lane].y;
                }
                t = make_float2(warp_sum(t.x), warp_sum(t.y));
            } else if (lane < rows) {
                const int wpr = GG_WARPS >> row_groups_log2(rows);
                for (int w = 0; w < wpr; ++w) {
                    t.x += sums[lane * wpr + w].x;
                    t.y += sums[lane * wpr + w].y;
                }
            }
            t.y *= rstd;
            if (lane < rows) {
                float2* const rec = p.grad_partials + (record + lane) * TB_GN_PARTS;
                rec[slot] = t;
                if (slot == 0) {
                    // the slots of parts that do not exist
                    const int parts = p.parts[record / (p.N * p.C)];
                    for (int q = parts; q < TB_GN_PARTS; ++q) rec[q] = make_float2(0.f, 0.f);
                }
            }
        }
    }
}

template <int DT>
__device__ __forceinline__ void copy_loop(const GnGradParams& p, Ring ring) {
    constexpr int ES = elem_size(DT);
    const int lane = threadIdx.x & 31;
    // (the host keeps the tasks below 2^31: 32-bit divisions throughout, the
    // 64-bit ones took longer than a task's copies)
    const uint32_t G = (uint32_t)p.G, K = (uint32_t)(p.C / p.G);
    const uint32_t T = (uint32_t)p.unit_tasks;
    const int64_t body = p.N * p.G * (int64_t)T;
    const uint32_t begin = (uint32_t)(body * blockIdx.x / gridDim.x);
    const uint32_t end = (uint32_t)(body * (blockIdx.x + 1) / gridDim.x);
    const int kind = p.mode == GRAD_STATS ? TASK_STATS : TASK_APPLY;
    bool ok = true;
    auto claim = [&]() -> bool {  // the ring's next stage, once the computing warps are done with it
        ok = ok && bar_wait(ring.empty + ring.s * 8u, ring.parity ^ 1u, p.status);
        if (__any_sync(0xffffffffu, !ok) || *ring.dead) ok = false;
        return ok;
    };
    for (uint32_t w = blockIdx.x; w < (uint32_t)p.wtasks && claim(); w += gridDim.x) {
        if (lane == 0) {
            Stage& d = ring.stage[ring.s];
            d.kind = TASK_WEIGHTS;
            d.channel = (int64_t)w * GRAD_CHANNELS;
            bar_arrive(ring.full + ring.s * 8u);  // (no copies)
            bar_arrive(ring.full + ring.s * 8u);
            bar_arrive(ring.task + ring.s * 8u);
        }
        ring.next();
    }
    for (uint32_t k = begin; k < end && ok; ++k) {
        // the dx from the end of the run: what was read last is in L2
        const uint32_t task = kind == TASK_APPLY ? end - 1 - (k - begin) : k;
        const uint32_t unit = task / T;
        uint32_t item = task - unit * T;
        int pp = 0;
        while ((uint32_t)p.task_start[pp + 1] <= item) ++pp;
        item -= (uint32_t)p.task_start[pp];
        const int64_t n = unit / G, g = unit - (uint32_t)n * G;
        const int64_t S = p.spatial[pp];
        const uint32_t parts = (uint32_t)p.parts[pp];
        int rows, part = 0, c_first;  // c_first: first row, within the group
        int64_t e0, e1;               // element range within the row
        if (parts > 1) {
            c_first = (int)(item / parts);
            part = (int)(item - (uint32_t)c_first * parts);
            rows = 1;
            const int64_t each = p.part_elems[pp];
            e0 = part * each;
            e1 = part + 1 == (int)parts ? S : e0 + each;
        } else {
            c_first = (int)item * p.rows[pp];
            rows = min(p.rows[pp], (int)K - c_first);
            e0 = 0;
            e1 = S;
        }
        const int64_t row = n * p.C + g * K + c_first;
        const char* const xbase = reinterpret_cast<const char*>(p.patches[pp]);
        const char* const dbase = reinterpret_cast<const char*>(p.grads[pp]);
        constexpr int64_t MOST = GRAD_STAGE_BYTES / ES;
        const bool once = kind == TASK_APPLY || (int64_t)(end - k) * rows * (e1 - e0) * ES > GG_KEEP;
        // (one stage for whole rows; the stages of a part in turn)
        // (an empty patch's rows still get their records)
        for (int64_t at = e0; (at < e1 || at == e0) && ok; at += MOST) {
            const int64_t len = min(MOST, e1 - at);
            if (!claim()) break;
            Stage& d = ring.stage[ring.s];
            const uint32_t bar = ring.full + ring.s * 8u;
            const int64_t first = row * S + at;
            // x on the lower lanes, dy on the upper ones: `head` bytes before the
            // first 16-byte boundary, the bulk copy's, and the rest
            const char* const from = (lane < 16 ? xbase : dbase) + first * ES;
            const uint32_t bytes = (uint32_t)(rows * (int)len) * ES;
            const uint32_t shift = (uint32_t)reinterpret_cast<uintptr_t>(from) & 15u;
            const uint32_t head = min((16u - shift) & 15u, bytes), bulk = (bytes - head) & ~15u;
            const uint32_t to = ring.data + (ring.s * 2 + (lane < 16 ? 0 : 1)) * GG_TENSOR + shift;
            if (lane == 0) {
                bar_expect(bar, 2 * bulk);
                d.kind = kind;
                d.rows = rows;
                d.row_elems = (int32_t)len;
                d.shift = (int32_t)shift / ES;
                d.last = at + len >= e1;
                d.slot = part;
                d.record = pp * p.N * p.C + row;
                d.n = (int32_t)n;
                d.g = (int32_t)g;
                d.channel = g * K + c_first;
                d.out = reinterpret_cast<char*>(p.outs[pp]) + first * ES;
                bar_arrive(ring.task + ring.s * 8u);
            }
            __syncwarp();
            if ((lane & 15) == 0 && bulk > 0) {
                if (once) bulk_load_once(to + head, from + head, bulk, bar);
                else bulk_load(to + head, from + head, bulk, bar);
            }
            if (bytes != bulk) {
                // lane k < 8 of either half: element k before the bulk copy, and k after it
                const uint32_t k = (lane & 7) * ES, tail = head + bulk + k;
                if ((lane & 8) == 0) {
                    if (k < head) copy_element<ES>(to + k, from + k);
                } else if (tail < bytes) {
                    copy_element<ES>(to + tail, from + tail);
                }
                bulk_fence();
                __syncwarp();
            }
            if (lane == 0) bar_arrive(bar);  // the elements copied one by one
            ring.next();
        }
    }
    for (int k = 0; k < GG_STAGES && ok && claim(); ++k) {  // each stage's warp must see it
        if (lane == 0) {
            ring.stage[ring.s].kind = TASK_END;
            bar_arrive(ring.full + ring.s * 8u);
            bar_arrive(ring.full + ring.s * 8u);
            bar_arrive(ring.task + ring.s * 8u);
        }
        ring.next();
    }
    if (!ok) {
        // a wait ran out, of this warp or of another: everyone leaves, once the
        // copies in flight have landed (or their own waits have run out)
        if (lane == 0) *ring.dead = 1;
        for (int k = 0; k < GG_STAGES; ++k)
            bar_wait(ring.full + k * 8u, k < ring.s ? ring.parity : ring.parity ^ 1u, p.status);
    }
}

// --- the computing warps ----------------------------------------------------------

template <int DT, bool SILU>
__device__ __forceinline__ void compute_loop(const GnGradParams& p, Ring ring) {
    constexpr int ES = elem_size(DT);
    constexpr int VEC = 16 / ES;
    constexpr int NP = VEC / 2;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    f32x2 B = 0ull, A = 0ull;  // 0ull: a pair of zeros
    while (true) {
        const bool here = bar_wait(ring.full + ring.s * 8u, ring.parity, p.status);
        if (!here && lane == 0) *ring.dead = 1;
        if (__any_sync(0xffffffffu, !here) || *ring.dead) return;
        const Stage& d = ring.stage[ring.s];
        const int kind = d.kind;
        const uint32_t empty = ring.empty + ring.s * 8u;
        if (kind == TASK_END) return;
        if (kind == TASK_WEIGHTS) {
            // a warp per channel adds up its records of all samples and sets
            const int64_t c = d.channel + warp;
            if (c < p.C) {
                float b = 0.f, a = 0.f;
                for (int64_t q = lane; q < (int64_t)p.R * p.N * TB_GN_PARTS; q += 32) {
                    const float2 v = p.grad_partials[(q / TB_GN_PARTS * p.C + c) * TB_GN_PARTS + q % TB_GN_PARTS];
                    b += v.x;
                    a += v.y;
                }
                b = warp_sum(b);
                a = warp_sum(a);
                if (lane == 0) {
                    if (p.dgamma != nullptr) store_weight(p.dgamma, DT, c, a);
                    if (p.dbeta != nullptr) store_weight(p.dbeta, DT, c, b);
                }
            }
            __syncwarp();
            if (lane == 0) bar_arrive(empty);
            ring.next();
            continue;
        }
        const int rows = d.rows, len = d.row_elems, shift = d.shift;
        // 2^lg row groups of `wpr` warps each (GG_WARPS is a power of two)
        const int lg = row_groups_log2(rows), wpr = GG_WARPS >> lg, groups = 1 << lg;
        const int wg = warp >> (GG_LOG2 - lg), wi = warp & (wpr - 1);
        const uint32_t xs = ring.data + ring.s * 2 * GG_TENSOR;
        const float mean = d.mean;
        const f32x2 mean2 = pair(mean, mean);
        const f32x2 u2 = pair(d.u, d.u), v2 = pair(d.v, d.v);
        for (int r = wg; r < rows; r += groups) {
            const float2 k = d.row[r];
            const f32x2 za = pair(k.x, k.x), zb = pair(k.y, k.y);
            const int lo = shift + r * len, hi = lo + len;            // the row's elements in the buffer
            const int w0 = (lo + VEC - 1) / VEC, w1 = hi / VEC;       // its whole words
            const int first = w0 + wi * 32 + lane, step = wpr * 32;
            // the words at its ends: x and dy as lanes, (mean, 0) outside [lo, hi)
            const int edge = lane == 0 ? lo / VEC : hi / VEC;
            const bool at_edge = wi == 0 && ((lane == 0 && lo < w0 * VEC) || (lane == 1 && hi > w1 * VEC && w1 >= w0));
            auto edge_word = [&](f32x2 (&x)[NP], f32x2 (&dy)[NP]) {
                to_lanes<DT, VEC>(smem_load<uint4>(xs + edge * 16u), x);
                to_lanes<DT, VEC>(smem_load<uint4>(xs + GG_TENSOR + edge * 16u), dy);
#pragma unroll
                for (int q = 0; q < NP; ++q) {
                    float a, b, c, e;
                    halves(x[q], a, b);
                    halves(dy[q], c, e);
                    const int i = edge * VEC + 2 * q;
                    if (i < lo || i >= hi) a = mean, c = 0.f;
                    if (i + 1 < lo || i + 1 >= hi) b = mean, e = 0.f;
                    x[q] = pair(a, b);
                    dy[q] = pair(c, e);
                }
            };
            if (kind == TASK_STATS) {
                auto add = [&](const f32x2 (&x)[NP], const f32x2 (&dy)[NP]) {
#pragma unroll
                    for (int q = 0; q < NP; ++q) {
                        const f32x2 u = vsub(x[q], mean2);
                        const f32x2 dz = dz_pair<SILU>(u, dy[q], za, zb);
                        B = vadd(B, dz);
                        A = vfma(dz, u, A);
                    }
                };
                uint32_t at = xs + first * 16u;
                for (int w = first; w < w1; w += step, at += step * 16u) {
                    f32x2 x[NP], dy[NP];
                    to_lanes<DT, VEC>(smem_load<uint4>(at), x);
                    to_lanes<DT, VEC>(smem_load<uint4>(at + GG_TENSOR), dy);
                    add(x, dy);
                }
                if (at_edge) {
                    f32x2 x[NP], dy[NP];
                    edge_word(x, dy);
                    add(x, dy);
                }
                if (d.last) {
                    float2* const slot = ring.slots + ring.s * GG_SLOTS;
                    if (rows == 1) {
                        // every lane leaves its own sums: ten dependent shuffles
                        // less at the end of a task
                        slot[threadIdx.x] = make_float2(vsum(B), vsum(A));
                    } else {
                        __syncwarp();
                        const float b = warp_sum(vsum(B)), a = warp_sum(vsum(A));
                        if (lane == 0) slot[r * wpr + wi] = make_float2(b, a);
                    }
                    B = A = 0ull;
                }
            } else {
                auto grad = [&](f32x2 (&x)[NP], const f32x2 (&dy)[NP]) {
#pragma unroll
                    for (int q = 0; q < NP; ++q) {
                        const f32x2 u = vsub(x[q], mean2);
                        x[q] = vfma(dz_pair<SILU>(u, dy[q], za, zb), za, vfma(u, u2, v2));
                    }
                };
                uint32_t at = xs + first * 16u;
                uint4* out = reinterpret_cast<uint4*>(d.out - shift * ES) + first;
                for (int w = first; w < w1; w += step, at += step * 16u, out += step) {
                    f32x2 x[NP], dy[NP];
                    to_lanes<DT, VEC>(smem_load<uint4>(at), x);
                    to_lanes<DT, VEC>(smem_load<uint4>(at + GG_TENSOR), dy);
                    grad(x, dy);
                    __stcs(out, from_lanes<DT, VEC>(x));
                }
                if (at_edge) {
                    f32x2 x[NP], dy[NP];
                    edge_word(x, dy);
                    grad(x, dy);
                    using E = typename Word<ES>::T;
                    const uint4 o = from_lanes<DT, VEC>(x);
                    const uint32_t bits[4] = {o.x, o.y, o.z, o.w};
                    E* const to = reinterpret_cast<E*>(d.out) + (edge * VEC - shift);
#pragma unroll
                    for (int q = 0; q < VEC; ++q) {
                        const int i = edge * VEC + q;
                        if (i < lo || i >= hi) continue;
                        if constexpr (ES == 4) to[q] = bits[q];
                        else to[q] = (E)(bits[q >> 1] >> (16 * (q & 1)));
                    }
                }
            }
        }
        if (kind == TASK_STATS && d.last) {
            // the stage's warp of constants takes the sums from here
            __syncwarp();
            if (lane == 0) bar_arrive(ring.sums + ring.s * 8u);
        }
        __syncwarp();
        if (lane == 0) bar_arrive(empty);
        ring.next();
    }
}

template <int DT, bool SILU>
__global__ void __launch_bounds__(GG_BLOCK, 1) gn_grad_kernel(const __grid_constant__ GnGradParams p) {
    extern __shared__ __align__(128) unsigned char s_data[];
    __shared__ Stage s_stage[GG_STAGES];
    __shared__ float2 s_slots[GG_STAGES][GG_SLOTS];
    __shared__ __align__(8) unsigned long long s_bar[4 * GG_STAGES];
    __shared__ int s_dead;
    Ring ring;
    ring.stage = s_stage;
    ring.slots = &s_slots[0][0];
    ring.full = smem_addr(s_bar);
    ring.empty = ring.full + GG_STAGES * 8u;
    ring.task = ring.empty + GG_STAGES * 8u;
    ring.sums = ring.task + GG_STAGES * 8u;
    ring.data = smem_addr(s_data);
    ring.dead = &s_dead;
    if (threadIdx.x == 0) {
        s_dead = 0;
        for (int k = 0; k < GG_STAGES; ++k) {
            bar_init(ring.task + k * 8u, 1);
            bar_init(ring.full + k * 8u, 3);  // the copies' bytes, the single elements, the constants
            bar_init(ring.empty + k * 8u, GG_WARPS);
            bar_init(ring.sums + k * 8u, GG_WARPS);
        }
        bar_init_fence();
    }
    __syncthreads();
    // the second pass may be placed as the first one's CTAs leave: a CTA fills
    // its SM, so none of them takes a place that this grid still needs
    if (p.mode == GRAD_STATS) pdl_trigger_dependents();
    grid_wait();
    if (threadIdx.x < GG_THREADS) compute_loop<DT, SILU>(p, ring);
    else if (threadIdx.x < GG_THREADS + 32) copy_loop<DT>(p, ring);
    else constants_loop(p, DT, ring, (int)(threadIdx.x - GG_THREADS) / 32 - 1);
    __syncthreads();  // (no warp's memory goes before the copies have landed)
}

// --- element kernels: patches, gradients and outputs at different offsets from
// 16-byte boundaries -------------------------------------------------------------

constexpr int EL_BLOCK = 256;
constexpr int EL_SEG = 4096;  // elements per CTA of the second pass

template <int DT>
__device__ __forceinline__ float elem_at(const void* base, int64_t i) {
    return elem_to_f<DT>(reinterpret_cast<const typename Word<elem_size(DT)>::T*>(base)[i]);
}

template <bool SILU>
__device__ __forceinline__ float dz_one(float u, float dy, float2 k) {
    float lo, hi;
    halves(dz_pair<SILU>(pair(u, u), pair(dy, dy), pair(k.x, k.x), pair(k.y, k.y)), lo, hi);
    return lo;
}

// One CTA per (patch, sample, channel) row: record 0, the others zero.
template <int DT, bool SILU>
__global__ void __launch_bounds__(EL_BLOCK) gn_grad_stats_elem_kernel(const __grid_constant__ GnGradParams p) {
    __shared__ float2 s_warp[EL_BLOCK / 32];
    const int64_t row = blockIdx.x, NC = p.N * p.C;
    const int pp = (int)(row / NC);
    const int64_t nc = row - pp * NC, n = nc / p.C, c = nc - n * p.C, g = c / (p.C / p.G);
    grid_wait();
    float mean, rstd, count;
    pooled_stats(p, n, g, mean, rstd, count);
    mean = __shfl_sync(0xffffffffu, mean, 0);
    rstd = __shfl_sync(0xffffffffu, rstd, 0);
    const float2 k = make_float2(rstd * weight_at(p.gamma, DT, c, 1.f), weight_at(p.beta, DT, c, 0.f));
    const int64_t S = p.spatial[pp], base = nc * S;
    float B = 0.f, A = 0.f;
    for (int64_t i = threadIdx.x; i < S; i += EL_BLOCK) {
        const float u = elem_at<DT>(p.patches[pp], base + i) - mean;
        const float dz = dz_one<SILU>(u, elem_at<DT>(p.grads[pp], base + i), k);
        B += dz;
        A = fmaf(dz, u, A);
    }
    B = warp_sum(B);
    A = warp_sum(A) * rstd;
    if ((threadIdx.x & 31) == 0) s_warp[threadIdx.x >> 5] = make_float2(B, A);
    __syncthreads();
    if (threadIdx.x < TB_GN_PARTS) {
        float2 t = make_float2(0.f, 0.f);
        if (threadIdx.x == 0) {
            for (int w = 0; w < EL_BLOCK / 32; ++w) {
                t.x += s_warp[w].x;
                t.y += s_warp[w].y;
            }
        }
        p.grad_partials[row * TB_GN_PARTS + threadIdx.x] = t;
    }
}

// grid (row segments of the longest patch, rows + weight-gradient CTAs).
template <int DT, bool SILU>
__global__ void __launch_bounds__(EL_BLOCK) gn_grad_apply_elem_kernel(const __grid_constant__ GnGradParams p) {
    const int64_t NC = p.N * p.C, rows = (int64_t)p.P * NC;
    grid_wait();
    for (int64_t row = blockIdx.x; row < rows + p.wtasks; row += gridDim.x) {
        if (row >= rows) {
            const int64_t c0 = (row - rows) * GRAD_CHANNELS;
            for (int64_t c = c0 + (threadIdx.x >> 5); c < min(p.C, c0 + GRAD_CHANNELS); c += EL_BLOCK / 32) {
                if (blockIdx.y > 0) break;
                float b = 0.f, a = 0.f;
                for (int64_t q = threadIdx.x & 31; q < (int64_t)p.R * p.N * TB_GN_PARTS; q += 32) {
                    const float2 v = p.grad_partials[(q / TB_GN_PARTS * p.C + c) * TB_GN_PARTS + q % TB_GN_PARTS];
                    b += v.x;
                    a += v.y;
                }
                b = warp_sum(b);
                a = warp_sum(a);
                if ((threadIdx.x & 31) == 0) {
                    if (p.dgamma != nullptr) store_weight(p.dgamma, DT, c, a);
                    if (p.dbeta != nullptr) store_weight(p.dbeta, DT, c, b);
                }
            }
            continue;
        }
        const int pp = (int)(row / NC);
        const int64_t nc = row - pp * NC, n = nc / p.C, c = nc - n * p.C, g = c / (p.C / p.G);
        const int64_t S = p.spatial[pp];
        if ((int64_t)blockIdx.y * EL_SEG >= S) continue;
        float mean, rstd, count;
        pooled_stats(p, n, g, mean, rstd, count);
        mean = __shfl_sync(0xffffffffu, mean, 0);
        rstd = __shfl_sync(0xffffffffu, rstd, 0);
        count = __shfl_sync(0xffffffffu, count, 0);
        const float2 k = make_float2(rstd * weight_at(p.gamma, DT, c, 1.f), weight_at(p.beta, DT, c, 0.f));
        const float2 uv = unit_sums(p, DT, n, g, rstd, count);
        using E = typename Word<elem_size(DT)>::T;
        for (int64_t e0 = (int64_t)blockIdx.y * EL_SEG; e0 < S; e0 += (int64_t)gridDim.y * EL_SEG) {
            for (int64_t i = e0 + threadIdx.x; i < min(S, e0 + EL_SEG); i += EL_BLOCK) {
                const float u = elem_at<DT>(p.patches[pp], nc * S + i) - mean;
                const float dz = dz_one<SILU>(u, elem_at<DT>(p.grads[pp], nc * S + i), k);
                const float o[1] = {fmaf(dz, k.x, fmaf(u, uv.x, uv.y))};
                reinterpret_cast<E*>(p.outs[pp])[nc * S + i] = pack<DT, 1>(o);
            }
        }
    }
}

template <int DT, bool SILU>
cudaError_t grad_launch(const GnGradParams& p, bool ring, int sms, cudaStream_t s) {
    if (ring) {
        const int64_t body = p.N * p.G * (int64_t)p.unit_tasks, tasks = body > p.wtasks ? body : p.wtasks;
        if (tasks == 0) return cudaSuccess;
        cudaError_t e = cudaFuncSetAttribute(gn_grad_kernel<DT, SILU>, cudaFuncAttributeMaxDynamicSharedMemorySize, GG_SMEM);
        if (e != cudaSuccess) return e;
        return launch_pdl(gn_grad_kernel<DT, SILU>, p, dim3((unsigned)(tasks < sms ? tasks : sms)), GG_BLOCK, GG_SMEM, s);
    }
    const int64_t rows = (int64_t)p.P * p.N * p.C;
    if (p.mode == GRAD_STATS) return launch_pdl(gn_grad_stats_elem_kernel<DT, SILU>, p, dim3((unsigned)rows), EL_BLOCK, 0, s);
    int64_t longest = 0;
    for (int q = 0; q < p.P; ++q) longest = longest < p.spatial[q] ? p.spatial[q] : longest;
    int64_t segs = (longest + EL_SEG - 1) / EL_SEG;
    segs = segs < 1 ? 1 : segs > 65535 ? 65535 : segs;
    return launch_pdl(gn_grad_apply_elem_kernel<DT, SILU>, p, dim3((unsigned)(rows + p.wtasks), (unsigned)segs), EL_BLOCK, 0,
                      s);
}

template <int DT>
cudaError_t grad_dt(const GnGradParams& p, bool ring, int sms, cudaStream_t s) {
    return p.silu ? grad_launch<DT, true>(p, ring, sms, s) : grad_launch<DT, false>(p, ring, sms, s);
}

}  // namespace

cudaError_t launch_gn_grad(const GnGradParams& p, int dtype, bool ring, int sms, cudaStream_t s) {
    switch (dtype) {
        case F32: return grad_dt<F32>(p, ring, sms, s);
        case F16: return grad_dt<F16>(p, ring, sms, s);
        default: return grad_dt<BF16>(p, ring, sms, s);
    }
}

}  // namespace tb
