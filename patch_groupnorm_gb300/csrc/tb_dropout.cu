// tb_dropout.cu -- dropout from a counter-based generator: the mask is computed
// where it is needed, forward and backward, and never stored.
//
// Element i (counted over the rows' elements, whatever their strides) belongs to
// block b = i / 8 of Philox 4x32 with ten rounds (Salmon, Moraes, Dror, Shaw:
// "Parallel random numbers: as easy as 1, 2, 3", 2011): key = seed, counter =
// (b, offset), each as two 32-bit words, the low one first.  A round is two
// 32 x 32 -> 64 bit products, four exclusive-ors and the key's step.  The block's
// four words give eight 16-bit numbers, each word's low half first; an element is
// dropped where its number is below `threshold`, and what is kept is multiplied by
// 65536 / (65536 - threshold), the inverse of the share that is kept exactly.
//
// 16 bits an element, not 32: the generator's products and sums are what bounds
// the kernel otherwise.  16384 x 4096 bf16: 53.4 us with a word an element, 43.1
// with half a word; a copy of that size takes 42.4.
#include "tb_elem.cuh"

namespace tb {
namespace {

constexpr int DROP_BLOCK = 256;
constexpr int RB = 8;  // elements of one block of random numbers
constexpr int DU = 2;  // blocks a thread loads together

struct Keys {
    uint32_t k0[10], k1[10];
};

__device__ __forceinline__ void key_schedule(uint64_t seed, Keys& k) {
#pragma unroll
    for (uint32_t r = 0; r < 10; ++r) {
        k.k0[r] = (uint32_t)seed + r * 0x9E3779B9u;
        k.k1[r] = (uint32_t)(seed >> 32) + r * 0xBB67AE85u;
    }
}

__device__ __forceinline__ void philox(uint64_t block, uint64_t offset, const Keys& k, uint32_t (&c)[4]) {
    c[0] = (uint32_t)block;
    c[1] = (uint32_t)(block >> 32);
    c[2] = (uint32_t)offset;
    c[3] = (uint32_t)(offset >> 32);
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t p0 = (uint64_t)0xD2511F53u * c[0], p1 = (uint64_t)0xCD9E8D57u * c[2];
        c[0] = (uint32_t)(p1 >> 32) ^ c[1] ^ k.k0[r];
        c[1] = (uint32_t)p1;
        c[2] = (uint32_t)(p0 >> 32) ^ c[3] ^ k.k1[r];
        c[3] = (uint32_t)p0;
    }
}

// The mask of a block, element e in bit e.  RANDOM false: all kept or all dropped.
template <bool RANDOM>
__device__ __forceinline__ void kept(uint64_t block, uint64_t offset, const Keys& k, uint32_t threshold, bool (&keep)[RB]) {
    if constexpr (RANDOM) {
        uint32_t c[4];
        philox(block, offset, k, c);
        const uint32_t t = threshold << 16;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            keep[2 * w] = (c[w] << 16) >= t;
            keep[2 * w + 1] = c[w] >= t;  // the low half cannot change it
        }
    } else {
#pragma unroll
        for (int e = 0; e < RB; ++e) keep[e] = threshold == 0u;
    }
}

// (seed, offset) of this call.
template <bool STATE>
__device__ __forceinline__ void generator(const DropoutParams& p, uint64_t& offset, Keys& keys) {
    uint64_t seed = p.seed;
    offset = p.offset;
    if constexpr (STATE) {
        seed += __ldg(p.state);
        offset += __ldg(p.state + 1);
    }
    key_schedule(seed, keys);
}

// Whole chunks: a block's elements per thread and turn, DU turns side by side.
// Rows of whole blocks; one row may end inside a block (its last thread takes the
// rest one by one).
template <int DT, bool RES, bool RANDOM, bool STATE>
__global__ void __launch_bounds__(DROP_BLOCK) dropout_kernel(const __grid_constant__ DropoutParams p) {
    constexpr int ES = elem_size(DT), VEC = 16 / ES, NW = RB / VEC;
    const int64_t per_row = p.cols / RB, blocks = per_row * p.rows;
    const int64_t first = (int64_t)blockIdx.x * (DROP_BLOCK * DU) + threadIdx.x;
    const char* const x = static_cast<const char*>(p.x);
    const char* const res = static_cast<const char*>(p.residual);
    char* const y = static_cast<char*>(p.y);
    // row and block of the row, stepped from turn to turn
    int64_t row = 0, col = first;
    if (p.rows > 1) {
        row = first / per_row;
        col = first - row * per_row;
    }
    grid_wait();
    Keys keys;
    uint64_t offset;
    generator<STATE>(p, offset, keys);
    uint4 vx[DU][NW], vr[DU][NW];
    int64_t at_y[DU];
#pragma unroll
    for (int u = 0; u < DU; ++u) {
        at_y[u] = -1;
        if (first + u * DROP_BLOCK < blocks) {
            at_y[u] = (row * p.y_ld + col * RB) * ES;
            const char* const ax = x + (row * p.x_ld + col * RB) * ES;
            const char* const ar = RES ? res + (row * p.r_ld + col * RB) * ES : nullptr;
            if (!in_bounds(ax, RB * ES, x, ((p.rows - 1) * p.x_ld + p.cols) * ES, p.status) ||
                (RES && !in_bounds(ar, RB * ES, res, ((p.rows - 1) * p.r_ld + p.cols) * ES, p.status)) ||
                !in_bounds(y + at_y[u], RB * ES, y, ((p.rows - 1) * p.y_ld + p.cols) * ES, p.status)) {
                at_y[u] = -1;
            } else {
#pragma unroll
                for (int w = 0; w < NW; ++w) {
                    vx[u][w] = reinterpret_cast<const uint4*>(ax)[w];
                    if (RES) vr[u][w] = reinterpret_cast<const uint4*>(ar)[w];
                }
            }
        }
        if (p.rows > 1) {
            col += DROP_BLOCK;
            while (col >= per_row) {
                col -= per_row;
                ++row;
            }
        } else {
            col += DROP_BLOCK;
        }
    }
#pragma unroll
    for (int u = 0; u < DU; ++u) {
        if (at_y[u] < 0) continue;
        bool keep[RB];
        kept<RANDOM>((uint64_t)(first + u * DROP_BLOCK), offset, keys, p.threshold, keep);
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            float f[VEC], r[VEC];
            unpack<DT, VEC>(vx[u][w], f);
            if (RES) unpack<DT, VEC>(vr[u][w], r);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                // chosen, not multiplied: a dropped infinity or NaN is gone
                const bool k = keep[w * VEC + e];
                f[e] = RES ? (k ? fmaf(f[e], p.scale, r[e]) : r[e]) : (k ? f[e] * p.scale : 0.f);
            }
            *reinterpret_cast<uint4*>(y + at_y[u] + w * 16) = pack<DT, VEC>(f);
        }
    }
    const int rest = (int)(p.cols - per_row * RB);  // one row only
    if (rest > 0 && blockIdx.x == gridDim.x - 1 && threadIdx.x == 0) {
        bool keep[RB];
        kept<RANDOM>((uint64_t)per_row, offset, keys, p.threshold, keep);
        using W = typename Word<ES>::T;
#pragma unroll
        for (int e = 0; e < RB; ++e) {
            if (e < rest) {
                const int64_t i = per_row * RB + e;
                if (!in_bounds(x + i * ES, ES, x, p.cols * ES, p.status)) continue;
                float f[1], r[1] = {0.f};
                unpack<DT, 1>(reinterpret_cast<const W*>(x)[i], f);
                if (RES) unpack<DT, 1>(reinterpret_cast<const W*>(res)[i], r);
                f[0] = RES ? (keep[e] ? fmaf(f[0], p.scale, r[0]) : r[0]) : (keep[e] ? f[0] * p.scale : 0.f);
                reinterpret_cast<W*>(y)[i] = pack<DT, 1>(f);
            }
        }
    }
}

// Any strides and addresses: a warp takes 32 blocks (256 neighbouring elements),
// each lane a block's mask, and the elements in turns of 32, whose bits come from
// the lane that has their block.
template <int DT, bool RES, bool RANDOM, bool STATE>
__global__ void __launch_bounds__(DROP_BLOCK) dropout_elem_kernel(const __grid_constant__ DropoutParams p) {
    constexpr int ES = elem_size(DT), SPAN = 32 * RB;
    using W = typename Word<ES>::T;
    const int lane = threadIdx.x & 31;
    const int64_t warp = ((int64_t)blockIdx.x * DROP_BLOCK + threadIdx.x) >> 5, total = p.rows * p.cols;
    const int64_t first = warp * SPAN;
    if (first >= total) return;
    const W* const x = static_cast<const W*>(p.x);
    const W* const res = static_cast<const W*>(p.residual);
    W* const y = static_cast<W*>(p.y);
    const int64_t row0 = first / p.cols, col0 = first - row0 * p.cols;
    grid_wait();
    Keys keys;
    uint64_t offset;
    generator<STATE>(p, offset, keys);
    W vx[RB], vr[RB];
    int64_t at_y[RB];
#pragma unroll
    for (int j = 0; j < RB; ++j) {
        int64_t row = row0, col = col0 + j * 32 + lane;
        at_y[j] = -1;
        if (first + j * 32 + lane < total) {
            if (p.cols >= SPAN) {
                if (col >= p.cols) {
                    col -= p.cols;
                    ++row;
                }
            } else {
                const uint32_t k = (uint32_t)col / (uint32_t)p.cols;
                row += k;
                col -= (int64_t)k * p.cols;
            }
            at_y[j] = row * p.y_ld + col;
            const int64_t ax = row * p.x_ld + col, ar = row * p.r_ld + col;
            if (!in_bounds(x + ax, ES, x, ((p.rows - 1) * p.x_ld + p.cols) * ES, p.status) ||
                (RES && !in_bounds(res + ar, ES, res, ((p.rows - 1) * p.r_ld + p.cols) * ES, p.status)) ||
                !in_bounds(y + at_y[j], ES, y, ((p.rows - 1) * p.y_ld + p.cols) * ES, p.status)) {
                at_y[j] = -1;
            } else {
                vx[j] = x[ax];
                if (RES) vr[j] = res[ar];
            }
        }
    }
    bool keep[RB];
    kept<RANDOM>((uint64_t)(warp * 32 + lane), offset, keys, p.threshold, keep);
    uint32_t mask = 0;
#pragma unroll
    for (int e = 0; e < RB; ++e) mask |= (uint32_t)keep[e] << e;
#pragma unroll
    for (int j = 0; j < RB; ++j) {
        const uint32_t m = __shfl_sync(0xffffffffu, mask, j * 4 + (lane >> 3));
        if (at_y[j] < 0) continue;
        const bool k = (m >> (lane & 7)) & 1u;
        float f[1], r[1] = {0.f};
        unpack<DT, 1>(vx[j], f);
        if (RES) unpack<DT, 1>(vr[j], r);
        f[0] = RES ? (k ? fmaf(f[0], p.scale, r[0]) : r[0]) : (k ? f[0] * p.scale : 0.f);
        y[at_y[j]] = pack<DT, 1>(f);
    }
}

template <int DT, bool RES, bool RANDOM>
cudaError_t drop_launch(const DropoutParams& p, bool vector, cudaStream_t s) {
    const int64_t span = (int64_t)DROP_BLOCK * RB * (vector ? DU : 1), total = p.rows * p.cols;
    const int64_t ctas = (total + span - 1) / span;
    if (ctas > 2147483647LL) return cudaErrorInvalidValue;
    void (*const fn)(const DropoutParams) =
        vector ? (RANDOM && p.state ? dropout_kernel<DT, RES, RANDOM, RANDOM> : dropout_kernel<DT, RES, RANDOM, false>)
               : (RANDOM && p.state ? dropout_elem_kernel<DT, RES, RANDOM, RANDOM>
                                    : dropout_elem_kernel<DT, RES, RANDOM, false>);
    return launch_pdl(fn, p, dim3((unsigned)ctas, 1, 1), DROP_BLOCK, 0, s);
}

template <int DT>
cudaError_t drop_launch(const DropoutParams& p, bool vector, cudaStream_t s) {
    const bool random = p.threshold > 0u && p.threshold < 65536u;
    if (p.residual != nullptr)
        return random ? drop_launch<DT, true, true>(p, vector, s) : drop_launch<DT, true, false>(p, vector, s);
    return random ? drop_launch<DT, false, true>(p, vector, s) : drop_launch<DT, false, false>(p, vector, s);
}

}  // namespace

cudaError_t launch_dropout(const DropoutParams& p, int dtype, bool vector, cudaStream_t s) {
    if (dtype == F32) return drop_launch<F32>(p, vector, s);
    if (dtype == F16) return drop_launch<F16>(p, vector, s);
    return drop_launch<BF16>(p, vector, s);
}

}  // namespace tb
