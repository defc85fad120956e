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
// the kernel otherwise (a trial of 16384 x 4096 bf16: 53.4 us with a word an element,
// 43.1 with half a word, 42.4 for a copy).  That size takes 40.2 us, 6680 GB/s; 65536 x 512
// onto a residual 29.1 in a graph, 6910 GB/s (two reads to a write; a copy, with one, gives
// 6790), and 30.2 from call to call.
#include "tb_elem.cuh"

namespace tb {
namespace {

constexpr int DROP_BLOCK = 256;
constexpr int RB = 8;  // elements of one block of random numbers

// Blocks a thread loads together.  16384 x 4096 bf16 with 1, 2, 4, 6 and 8: 48.9, 41.9,
// 42.1, 40.1 and 41.0 us; 16384 x 2048 out of wider rows 31.1, 27.9, 25.2, 28.4 (6); f32 and
// with a residual, where a block is two 16-byte words or more, 65536 x 512 bf16 onto a
// residual 29.2, 29.4 (2), 29.9 (4).
template <int DT, bool RES, bool ROWS>
constexpr int DROP_TURNS = DT == F32 || RES ? 1 : ROWS ? 4 : 6;

// Rows of 16-bit elements that are not whole vectors, from WORD_COLS on: turns of a warp, and
// threads of a CTA (16387 x 2047 bf16 out of wider rows with 2, 3, 4, 6 and 8 turns 39.8,
// 34.0, 36.0, 37.1 and 51.5 us; 4099 x 1111 f16 onto a residual 8.7, 8.5, 11.1, 9.8 and 14.4,
// 7.9 with CTAs half as large).  Element by element: rows of 257, 23.3 and 20.6 us onto a
// residual, of 300 20.0 and 19.6, of 511 15.1 and 17.7; f32 gains nothing (1111, 17.9 and 17.5).
constexpr int WORD_TURNS = 3, WORD_BLOCK = 128, WORD_COLS = 320;

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
        seed += p.state[0];
        offset += p.state[1];
    }
    key_schedule(seed, keys);
}

// Whole chunks: a block's elements per thread and turn, DROP_TURNS turns side by side.
// Nothing is read twice: loads and stores are marked so (44.6 us against 47.2).
// ROWS: rows of whole blocks, with strides.  Else one row, which may end inside a block
// (its last thread takes the rest one by one): an instance for both took 44.6 us for
// 16384 x 4096 bf16, this one 42.1.
template <int DT, bool RES, bool RANDOM, bool STATE, bool ROWS>
__global__ void __launch_bounds__(DROP_BLOCK) dropout_kernel(const __grid_constant__ DropoutParams p) {
    constexpr int ES = elem_size(DT), VEC = 16 / ES, NW = RB / VEC, DU = DROP_TURNS<DT, RES, ROWS>;
    const int64_t per_row = p.cols / RB, blocks = per_row * p.rows;
    const int64_t first = (int64_t)blockIdx.x * (DROP_BLOCK * DU) + threadIdx.x;
    const char* const x = static_cast<const char*>(p.x);
    const char* const res = static_cast<const char*>(p.residual);
    char* const y = static_cast<char*>(p.y);
    // row and block of the row, stepped from turn to turn (a 64-bit division is a hundred
    // instructions; 2 000 000 x 8 bf16 out of wider rows takes 15.3 us, 116 row by row)
    int64_t row = 0, col = first;
    [[maybe_unused]] int row_step = 0, col_step = DROP_BLOCK;
    if constexpr (ROWS) {
        row = blocks >> 32 ? first / per_row : (uint32_t)first / (uint32_t)per_row;
        col = first - row * per_row;
        row_step = per_row > DROP_BLOCK ? 0 : DROP_BLOCK / (int)per_row;
        col_step -= row_step * (int)per_row;
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
                    vx[u][w] = __ldcs(reinterpret_cast<const uint4*>(ax) + w);
                    if (RES) vr[u][w] = __ldcs(reinterpret_cast<const uint4*>(ar) + w);
                }
            }
        }
        if constexpr (ROWS) {
            row += row_step;
            col += col_step;
            if (col >= per_row) {
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
            __stcs(reinterpret_cast<uint4*>(y + at_y[u] + w * 16), pack<DT, VEC>(f));
        }
    }
    const int rest = ROWS ? 0 : (int)(p.cols - per_row * RB);  // one row only
    if (rest > 0 && blockIdx.x == gridDim.x - 1 && threadIdx.x == 0) {
        bool keep[RB];
        kept<RANDOM>((uint64_t)per_row, offset, keys, p.threshold, keep);
        using W = typename Word<ES>::T;
#pragma unroll
        for (int e = 0; e < RB; ++e) {
            if (e < rest) {
                const int64_t i = per_row * RB + e;
                if (!in_bounds(x + i * ES, ES, x, p.cols * ES, p.status) ||
                    (RES && !in_bounds(res + i * ES, ES, res, p.cols * ES, p.status)) ||
                    !in_bounds(y + i * ES, ES, y, p.cols * ES, p.status))
                    continue;
                float f[1], r[1] = {0.f};
                unpack<DT, 1>(reinterpret_cast<const W*>(x)[i], f);
                if (RES) unpack<DT, 1>(reinterpret_cast<const W*>(res)[i], r);
                f[0] = RES ? (keep[e] ? fmaf(f[0], p.scale, r[0]) : r[0]) : (keep[e] ? f[0] * p.scale : 0.f);
                reinterpret_cast<W*>(y)[i] = pack<DT, 1>(f);
            }
        }
    }
}

// One element.
template <int DT, bool RES>
__device__ __forceinline__ typename Word<elem_size(DT)>::T drop_one(typename Word<elem_size(DT)>::T x,
                                                                    typename Word<elem_size(DT)>::T res, bool keep,
                                                                    float scale) {
    float f[1], r[1] = {0.f};
    unpack<DT, 1>(x, f);
    if (RES) unpack<DT, 1>(res, r);
    f[0] = RES ? (keep ? fmaf(f[0], scale, r[0]) : r[0]) : (keep ? f[0] * scale : 0.f);
    return pack<DT, 1>(f);
}

// Single elements, any strides and addresses: a warp takes 32 blocks (256 neighbouring elements),
// each lane a block's mask, and the elements in turns of 32, whose bits come from
// the lane that has their block.  Where a row has at least as many elements (not
// NARROW) they lie in one row or two, and an element's address is one of two bases
// and a constant; in narrower rows the row and the column are stepped from turn to
// turn.  (16387 x 2047 bf16 out of wider rows: 78 us with an index for every element.)
template <int DT, bool RES, bool RANDOM, bool STATE, bool NARROW>
__global__ void __launch_bounds__(DROP_BLOCK) dropout_elem_kernel(const __grid_constant__ DropoutParams p) {
    constexpr int ES = elem_size(DT), SPAN = 32 * RB;
    using W = typename Word<ES>::T;
    const int lane = threadIdx.x & 31;
    const int64_t warp = ((int64_t)blockIdx.x * DROP_BLOCK + threadIdx.x) >> 5, total = p.rows * p.cols;
    const int64_t first = warp * SPAN;
    if (first >= total) return;
    // a 64-bit division is a hundred instructions
    const int64_t row0 = total >> 32 ? first / p.cols : (uint32_t)first / (uint32_t)p.cols, col0 = first - row0 * p.cols;
    const int left = (int)min((int64_t)SPAN, total - first);           // elements of this warp
    const int cut = (int)min((int64_t)SPAN, p.cols - col0);            // of these, in the first row
    const int cols = NARROW ? (int)p.cols : 0, row_step = NARROW ? 32 / cols : 0, col_step = 32 - row_step * cols;
    const int64_t last = p.rows - 1;
    const W* const x = static_cast<const W*>(p.x) + row0 * p.x_ld + col0;
    const W* const res = RES ? static_cast<const W*>(p.residual) + row0 * p.r_ld + col0 : nullptr;
    W* const y = static_cast<W*>(p.y) + row0 * p.y_ld + col0;
    // Calls body(turn, element of x, of the residual, of y) for each of the lane's eight
    // elements; those past the end are the last one again, so that all loads are on
    // their way before the first is waited for (with a branch each: 68 us).
    auto each = [&](auto&& body) {
        [[maybe_unused]] int row = 0, at = (int)col0 + lane;
        if constexpr (NARROW) {
            row = at / cols;
            at -= row * cols;
        }
        [[maybe_unused]] const int end = (int)col0 + left - 1, end_row = NARROW ? end / cols : 0;
        [[maybe_unused]] const int end_at = end - end_row * cols;
#pragma unroll
        for (int j = 0; j < RB; ++j) {
            if constexpr (NARROW) {
                const bool past = j * 32 + lane >= left;
                const int r = past ? end_row : row, c = (past ? end_at : at) - (int)col0;
                body(j, x + r * p.x_ld + c, RES ? res + r * p.r_ld + c : nullptr, y + r * p.y_ld + c);
                row += row_step;
                at += col_step;
                if (at >= cols) {
                    at -= cols;
                    ++row;
                }
            } else {
                const int e = min(j * 32 + lane, left - 1);
                const bool second = e >= cut;  // the next row's first element is number `cut`
                body(j, x + (second ? p.x_ld - p.cols : 0) + e, RES ? res + (second ? p.r_ld - p.cols : 0) + e : nullptr,
                     y + (second ? p.y_ld - p.cols : 0) + e);
            }
        }
    };
    // The lane's elements, masked and scaled.
    auto drop = [&](const W (&vx)[RB], const W (&vr)[RB], W (&out)[RB], const Keys& keys, uint64_t offset) {
        bool keep[RB];
        kept<RANDOM>((uint64_t)(warp * 32 + lane), offset, keys, p.threshold, keep);
        uint32_t mask = 0;
#pragma unroll
        for (int e = 0; e < RB; ++e) mask |= (uint32_t)keep[e] << e;
#pragma unroll
        for (int j = 0; j < RB; ++j) {
            const uint32_t m = __shfl_sync(0xffffffffu, mask, j * 4 + (lane >> 3));
            out[j] = drop_one<DT, RES>(vx[j], vr[j], (m >> (lane & 7)) & 1u, p.scale);
        }
    };
    grid_wait();
    Keys keys;
    uint64_t offset;
    generator<STATE>(p, offset, keys);
    W vx[RB], vr[RB], out[RB];
    if (!NARROW && cut == SPAN) {  // one row
#pragma unroll
        for (int j = 0; j < RB; ++j) {
            vx[j] = vr[j] = W{};
            if (in_bounds(x + j * 32 + lane, ES, p.x, (last * p.x_ld + p.cols) * ES, p.status)) vx[j] = x[j * 32 + lane];
            if (RES && in_bounds(res + j * 32 + lane, ES, p.residual, (last * p.r_ld + p.cols) * ES, p.status))
                vr[j] = res[j * 32 + lane];
        }
        drop(vx, vr, out, keys, offset);
#pragma unroll
        for (int j = 0; j < RB; ++j)
            if (in_bounds(y + j * 32 + lane, ES, p.y, (last * p.y_ld + p.cols) * ES, p.status)) y[j * 32 + lane] = out[j];
        return;
    }
    each([&](int j, const W* ax, const W* ar, W*) {
        vx[j] = vr[j] = W{};
        if (in_bounds(ax, ES, p.x, (last * p.x_ld + p.cols) * ES, p.status)) vx[j] = *ax;
        if (RES && in_bounds(ar, ES, p.residual, (last * p.r_ld + p.cols) * ES, p.status)) vr[j] = *ar;
    });
    drop(vx, vr, out, keys, offset);
    each([&](int j, const W*, const W*, W* ay) {
        if (j * 32 + lane < left && in_bounds(ay, ES, p.y, (last * p.y_ld + p.cols) * ES, p.status)) *ay = out[j];
    });
}

template <int N>
struct Words {
    static constexpr int value = N;
};

// The words that hold a unit's elements, the first at `at`, `off` bytes past a 16-byte
// boundary.  WHOLE: 16 bytes from that boundary on, and 16 more if off > 0, lie in the
// tensor; else elements [lo, hi) one by one, from the first word's start.  The tensor:
// `size` bytes at `base` (bounds-checked build).
template <bool WHOLE>
__device__ __forceinline__ void load_unit(const char* at, int off, int lo, int hi, uint4 (&w)[2], const char* base,
                                          int64_t size, uint32_t* status) {
    w[0] = w[1] = make_uint4(0u, 0u, 0u, 0u);
    if constexpr (WHOLE) {
        const uint4* const from = reinterpret_cast<const uint4*>(at - off);
        if (in_bounds(from, 16, base, size, status)) w[0] = from[0];
        if (off > 0 && in_bounds(from + 1, 16, base, size, status)) w[1] = from[1];
    } else {
        const unsigned short* const from = reinterpret_cast<const unsigned short*>(at);
        uint32_t u[4] = {};
#pragma unroll
        for (int e = 0; e < RB; ++e)
            if (e >= lo && e < hi && in_bounds(from + e, 2, base, size, status))
                u[e / 2] |= (uint32_t)from[e] << (e % 2 * 16);
        w[0] = make_uint4(u[0], u[1], u[2], u[3]);
    }
}

// The 16 bytes that start `off` bytes into w.  A branch on the whole words of the offset,
// which is the warp's: choosing them is ten operations more on the busiest pipe.
__device__ __forceinline__ void shift_unit(const uint4 (&w)[2], int off, uint32_t (&u)[4]) {
    const uint32_t v[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
    const int by = (off & 2) * 8;
    auto from = [&](auto first) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            constexpr int F = decltype(first)::value;
            u[k] = __funnelshift_r(v[k + F], v[k + F + 1], by);
        }
    };
    if (off < 8) {
        if (off < 4) from(Words<0>());
        else from(Words<1>());
    } else {
        if (off < 12) from(Words<2>());
        else from(Words<3>());
    }
}

// A word's two elements: all ones where bit 2 * word, and the one after, of m are set.
__device__ __forceinline__ uint32_t spread(uint32_t m, int word) {
    uint32_t r;  // a byte's sign, twice, and another's
    asm("prmt.b32 %0, %1, %2, 0xCC88;" : "=r"(r) : "r"(m << (7 - 2 * word)), "r"(m << (6 - 2 * word)));
    return r;
}

// A block's mask, element e in bit e.  The bits are summed as powers of two in a float's
// last places: that pipe is the least busy.
template <bool RANDOM>
__device__ __forceinline__ uint32_t mask_bits(uint64_t block, uint64_t offset, const Keys& k, uint32_t threshold) {
    if constexpr (RANDOM) {
        uint32_t c[4];
        philox(block, offset, k, c);
        const uint32_t t = threshold << 16;
        float lo = 8388608.f, hi = 8388608.f;  // 2^23
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            asm("{\n\t.reg .pred p;\n\tsetp.ge.u32 p, %1, %2;\n\t@p add.f32 %0, %0, %3;\n\t}"
                : "+f"(lo)
                : "r"(c[w] << 16), "r"(t), "f"((float)(1 << (2 * w))));
            asm("{\n\t.reg .pred p;\n\tsetp.ge.u32 p, %1, %2;\n\t@p add.f32 %0, %0, %3;\n\t}"
                : "+f"(hi)
                : "r"(c[w]), "r"(t), "f"((float)(2 << (2 * w))));
        }
        return (__float_as_uint(lo) | __float_as_uint(hi)) & 0xffu;
    } else {
        return threshold == 0u ? 0xffu : 0u;
    }
}

// Rows of 16-bit elements of any width from WORD_COLS on, any strides and addresses.  A
// unit is 16 bytes, eight elements, of a row of y from a 16-byte boundary on (the first of a
// row may begin before it, the last end behind it: those are stored one by one).  A warp
// takes 32 * T units of one row, so that everything about the row is its own, not a
// lane's.  What a unit needs of x and of the residual is loaded in aligned words and
// shifted into place; its elements lie in two blocks of random numbers, of which a lane
// computes the first and has the second from the next lane, except at the end of a row and
// of the warp's units.  Words that reach into what lies between two rows are read
// whole; where they would reach out of the tensor, the warp's elements are read one by one.
//
// What bounds it is issue slots (72 % of all cycles) and the pipe of integer and logic
// operations.  16387 x 2047 bf16 out of wider rows: 33.6 us, element by element 44.1.
template <int DT, bool RES, bool RANDOM, bool STATE>
__global__ void __launch_bounds__(WORD_BLOCK) dropout_word_kernel(const __grid_constant__ DropoutParams p) {
    static_assert(elem_size(DT) == 2, "a unit is 16 bytes");
    constexpr int T = WORD_TURNS, SPAN = 32 * T * RB;
    const int lane = threadIdx.x & 31;
    const int64_t runs = (p.cols + RB - 1 + SPAN - 1) / SPAN, total = runs * p.rows;
    const int64_t warp = (int64_t)blockIdx.x * (WORD_BLOCK / 32) + __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0);
    if (warp >= total) return;
    const int64_t row = total >> 32 ? warp / runs : (uint32_t)warp / (uint32_t)runs;
    const char* const x = static_cast<const char*>(p.x);
    const char* const res = static_cast<const char*>(p.residual);
    // the warp's first element; a row's first `before` belong to the row before, or to nobody
    char* const y_row = static_cast<char*>(p.y) + row * p.y_ld * 2;
    const int before = (int)(reinterpret_cast<uintptr_t>(y_row) & 15u) / 2;
    const int64_t col = (warp - row * runs) * SPAN - before, left = p.cols - col;
    if (left <= 0) return;
    const int64_t at = row * p.cols + col;
    char* const to = y_row + col * 2;
    const char* const from_x = x + (row * p.x_ld + col) * 2;
    const char* const from_r = RES ? res + (row * p.r_ld + col) * 2 : nullptr;
    const int off_x = (int)(reinterpret_cast<uintptr_t>(from_x) & 15u);
    const int off_r = RES ? (int)(reinterpret_cast<uintptr_t>(from_r) & 15u) : 0;
    const int first = col < 0 ? before : 0, end = (int)min(left, (int64_t)SPAN), units = (end + RB - 1) / RB;
    auto bytes = [&](int64_t ld) { return ((p.rows - 1) * ld + p.cols) * 2; };
    // all units' words lie in the tensor
    auto inside = [&](const char* from, int off, const char* base, int64_t ld) {
        return from - off >= base && from - off + (units + (off > 0)) * 16 <= base + bytes(ld);
    };
    const bool whole = inside(from_x, off_x, x, p.x_ld) && (!RES || inside(from_r, off_r, res, p.r_ld));
    uint4 vx[T][2], vr[T][2];
    grid_wait();
    Keys keys;
    uint64_t offset;
    generator<STATE>(p, offset, keys);
    if (whole) {
#pragma unroll
        for (int t = 0; t < T; ++t) {
            const int u = t * 32 + lane;
            if (u < units) {
                load_unit<true>(from_x + u * 16, off_x, 0, RB, vx[t], x, bytes(p.x_ld), p.status);
                if (RES) load_unit<true>(from_r + u * 16, off_r, 0, RB, vr[t], res, bytes(p.r_ld), p.status);
            }
        }
    } else {
#pragma unroll
        for (int t = 0; t < T; ++t) {
            const int u = t * 32 + lane, lo = max(first - u * RB, 0), hi = end - u * RB;
            load_unit<false>(from_x + u * 16, 0, lo, hi, vx[t], x, bytes(p.x_ld), p.status);
            if (RES) load_unit<false>(from_r + u * 16, 0, lo, hi, vr[t], res, bytes(p.r_ld), p.status);
        }
    }
    const int by_x = whole ? off_x : 0, by_r = whole ? off_r : 0;
    [[maybe_unused]] const int into = (int)(at & 7);
    auto bits = [&](int u) { return mask_bits<RANDOM>((uint64_t)((at >> 3) + u), offset, keys, p.threshold); };
    const int64_t size = bytes(p.y_ld);
    uint32_t mask = bits(lane);
#pragma unroll
    for (int t = 0; t < T; ++t) {
        if (t * 32 >= units) break;
        const int u = t * 32 + lane;
        uint32_t m = mask;  // where nothing is random every block's is the same
        if constexpr (RANDOM) {
            const uint32_t later = t + 1 < T && t * 32 + 32 < units ? bits(u + 32) : 0u;
            const uint32_t turn = __shfl_sync(0xffffffffu, later, 0);
            uint32_t next = __shfl_down_sync(0xffffffffu, mask, 1);
            if (lane == 31) next = turn;
            // the last unit, if it reaches into the next block
            if (u + 1 == units && RB - into < end - u * RB) next = bits(u + 1);
            m = (mask | next << RB) >> into;
            mask = later;
        }
        uint32_t word[4], r_word[4];
        shift_unit(vx[t], by_x, word);
        if (RES) shift_unit(vr[t], by_r, r_word);
        float f[RB], r[RB];
        unpack<DT, RB>(make_uint4(word[0], word[1], word[2], word[3]), f);
        if (RES) unpack<DT, RB>(make_uint4(r_word[0], r_word[1], r_word[2], r_word[3]), r);
#pragma unroll
        for (int e = 0; e < RB; ++e) f[e] = RES ? fmaf(f[e], p.scale, r[e]) : f[e] * p.scale;
        const uint4 out = pack<DT, RB>(f);
        const uint32_t kept_word[4] = {out.x, out.y, out.z, out.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            // chosen, not multiplied: a dropped infinity or NaN is gone
            const uint32_t on = spread(m, k);
            word[k] = RES ? (kept_word[k] & on) | (r_word[k] & ~on) : kept_word[k] & on;
        }
        char* const here = to + u * 16;
        const int lo = max(first - u * RB, 0), hi = end - u * RB;
        if (lo == 0 && hi >= RB) {
            if (in_bounds(here, 16, p.y, size, p.status))
                *reinterpret_cast<uint4*>(here) = make_uint4(word[0], word[1], word[2], word[3]);
        } else if (hi > 0) {
#pragma unroll
            for (int e = 0; e < RB; ++e) {
                if (e >= lo && e < hi && in_bounds(here + e * 2, 2, p.y, size, p.status))
                    *(reinterpret_cast<unsigned short*>(here) + e) = (unsigned short)(word[e / 2] >> (e % 2 * 16));
            }
        }
    }
}

template <int DT, bool RES, bool RANDOM>
cudaError_t drop_launch(const DropoutParams& p, bool vector, cudaStream_t s) {
    constexpr bool R = RANDOM, HALVES = elem_size(DT) == 2;
    constexpr int H = HALVES ? DT : F16;
    int64_t work = (p.rows * p.cols + RB - 1) / RB;  // blocks, or warps
    int per_cta = DROP_BLOCK, block = DROP_BLOCK;
    void (*fn)(const DropoutParams);
    if (vector && p.rows > 1) {
        per_cta = DROP_BLOCK * DROP_TURNS<DT, RES, true>;
        fn = R && p.state ? dropout_kernel<DT, RES, R, R, true> : dropout_kernel<DT, RES, R, false, true>;
    } else if (vector) {
        per_cta = DROP_BLOCK * DROP_TURNS<DT, RES, false>;
        fn = R && p.state ? dropout_kernel<DT, RES, R, R, false> : dropout_kernel<DT, RES, R, false, false>;
    } else if (HALVES && p.cols >= WORD_COLS) {
        constexpr int span = 32 * WORD_TURNS * RB;
        work = p.rows * ((p.cols + RB - 1 + span - 1) / span);
        per_cta = WORD_BLOCK / 32;
        block = WORD_BLOCK;
        fn = R && p.state ? dropout_word_kernel<H, RES, R, R> : dropout_word_kernel<H, RES, R, false>;
    } else if (p.cols < 32 * RB) {
        fn = R && p.state ? dropout_elem_kernel<DT, RES, R, R, true> : dropout_elem_kernel<DT, RES, R, false, true>;
    } else {
        fn = R && p.state ? dropout_elem_kernel<DT, RES, R, R, false> : dropout_elem_kernel<DT, RES, R, false, false>;
    }
    const int64_t ctas = (work + per_cta - 1) / per_cta;
    if (ctas > 2147483647LL) return cudaErrorInvalidValue;
    return launch_pdl(fn, p, dim3((unsigned)ctas, 1, 1), block, 0, s);
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
