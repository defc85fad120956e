// tb_gradclip.cu -- the global norm of many gradient tensors, and the clip.
//
//     norm = sqrt(sum over all elements of g^2)
//     out  = rnd(g * min(1, max_norm / (norm + 1e-6)))
//
// Two launches over the same pieces of work (GRAD_PIECE_BYTES of one tensor
// each; a CTA takes a contiguous run of them).  grad_stats_kernel leaves one
// fp64 record per CTA, the sum of its squares; grad_clip_kernel's CTAs each
// add up all records in one fixed order (so all see the same norm, and the
// same bits every time) and scale their pieces, walking them from the last
// to the first: the pieces the first kernel read last are still in L2.
//
// Bound by memory: 368 M elements (1024-wide blocks, bf16) take 344 us, the read
// by the first kernel (736 MB; 124 us timed alone) and the read and write by the
// second (229 us alone, 6.4 TB/s).  3.5 M fp32 elements take 10 us, the time of
// the two launches.
//
// Within a piece a thread adds the squares of its elements in fp32, and it
// carries the pieces' sums with their rounding errors.  A thread whose fp32
// sum could have overflowed or lost squares to underflow takes them again
// scaled by a power of two, so any finite gradients give their norm wherever
// fp32 can hold it.
#include "tb_elem.cuh"

namespace tb {
namespace {

constexpr int GC_BLOCK = 256;
constexpr int GC_CTAS = 5;                                    // per SM (344 us; 6 take 347, 4 346: no difference that counts)
// The last pieces of each CTA's run are the ones that grad_clip_kernel takes first; those before them are
// read evict-first, so that these stay in L2: 8 x 16 KB x 760 CTAs, 100 MB of this GPU's 129 (344 us; all read
// alike 354).
constexpr int GC_KEEP = 8;
constexpr int GC_CPT = GRAD_PIECE_BYTES / (GC_BLOCK * 16);    // chunks per thread and piece

// The tensor that piece `piece` belongs to.
template <int MAXT>
__device__ __forceinline__ int tensor_of(const GradParams<MAXT>& p, int piece) {
    int lo = 0, hi = p.T - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.start[mid] <= piece) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// One piece of a tensor: its chunks c0 .. c0 + n - 1 at `body`, and up to two
// runs of single elements (the head, the rest).
struct Piece {
    int64_t first;       // element index of chunk 0 of the piece
    int n;               // chunks
    int head;            // elements 0 .. head - 1 belong to this piece
    int64_t rest;        // elements rest .. numel - 1 belong to this piece
};

template <int MAXT>
__device__ __forceinline__ Piece piece_of(const GradParams<MAXT>& p, int t, int piece) {
    const int vec = p.dtype[t] == F32 ? 4 : 8;
    const int64_t numel = p.numel[t];
    const int head = p.head[t];
    const int64_t chunks = (numel - head) / vec;
    const int64_t c0 = (int64_t)(piece - p.start[t]) * (GRAD_PIECE_BYTES / 16);
    const int64_t left = chunks - c0;
    Piece r;
    r.first = head + c0 * vec;
    r.n = (int)(left < GRAD_PIECE_BYTES / 16 ? left : GRAD_PIECE_BYTES / 16);
    r.head = c0 == 0 ? head : 0;
    r.rest = piece + 1 == p.start[t + 1] ? head + chunks * vec : numel;
    return r;
}

template <int DT>
__device__ __forceinline__ float squares(const uint4& v, float scale) {
    constexpr int VEC = 16 / elem_size(DT);
    float f[VEC];
    unpack<DT, VEC>(v, f);
    float a = 0.f;
#pragma unroll
    for (int q = 0; q < VEC; ++q) a = fmaf(f[q] * scale, f[q] * scale, a);
    return a;
}

// fp32 sums of squares inside (LOW, HIGH) have lost nothing: a sum below LOW
// may miss squares that underflowed, one above HIGH may soon overflow.  Such
// sums are taken again of the elements times or over 2^96, and kept apart.
constexpr float SQ_LOW = 0x1p-90f, SQ_HIGH = 0x1p100f;
constexpr float SQ_SCALE = 0x1p96f;

// A thread's sums: the ordinary ones with their rounding errors (Knuth's
// two-sum), those of squares times 2^192 and over 2^192.
struct Squares {
    float sum = 0.f, err = 0.f, small = 0.f, large = 0.f;
};

template <int DT>
__device__ __forceinline__ void piece_squares(Squares& acc, const void* base, int64_t numel, const Piece& c,
                                              uint32_t* status, bool keep) {
    constexpr int VEC = 16 / elem_size(DT);
    const char* const b = reinterpret_cast<const char*>(base);
    const int64_t bytes = numel * elem_size(DT);
    const uint4* const src = reinterpret_cast<const uint4*>(b + c.first * elem_size(DT));
    uint4 v[GC_CPT];
#pragma unroll
    for (int k = 0; k < GC_CPT; ++k) {
        const int i = threadIdx.x + k * GC_BLOCK;
        v[k] = make_uint4(0u, 0u, 0u, 0u);
        if (i < c.n && in_bounds(src + i, 16, b, bytes, status)) v[k] = keep ? src[i] : __ldcs(src + i);
    }
    // the head and the rest are fewer than VEC elements each
    uint32_t one = 0u;
    const int64_t single = threadIdx.x < VEC ? threadIdx.x : c.rest + (threadIdx.x - VEC);
    const bool has = threadIdx.x < VEC ? threadIdx.x < c.head : threadIdx.x < 2 * VEC && single < numel;
    if (has && in_bounds(b + single * elem_size(DT), elem_size(DT), b, bytes, status)) {
        if constexpr (DT == F32) one = reinterpret_cast<const uint32_t*>(b)[single];
        else one = reinterpret_cast<const unsigned short*>(b)[single];
    }
    auto total = [&](float scale) {
        float a = elem_to_f<DT>(one) * scale;
        a *= a;
#pragma unroll
        for (int k = 0; k < GC_CPT; ++k) a += squares<DT>(v[k], scale);
        return a;
    };
    const float v2 = total(1.f);
    if (v2 > SQ_LOW && v2 < SQ_HIGH) {
        const float t = acc.sum + v2, b2 = t - acc.sum;
        acc.err += (acc.sum - (t - b2)) + (v2 - b2);
        acc.sum = t;
    } else if (v2 < 1.f) {
        acc.small += total(SQ_SCALE);
    } else {
        acc.large += total(1.f / SQ_SCALE);
    }
}

// Sum over the CTA; every thread gets it.  `slots` must not be reused before
// another barrier.
__device__ __forceinline__ float block_sum(float v, float* slots) {
    v = warp_sum(v);
    if ((threadIdx.x & 31) == 0) slots[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int w = 0; w < GC_BLOCK / 32; ++w) v += slots[w];
    return v;
}

template <int MAXT>
__global__ void __launch_bounds__(GC_BLOCK, GC_CTAS) grad_stats_kernel(const __grid_constant__ GradParams<MAXT> p) {
    __shared__ float s_part[3][GC_BLOCK / 32];
    const int64_t total = p.start[p.T];
    const int begin = (int)(total * blockIdx.x / gridDim.x), end = (int)(total * (blockIdx.x + 1) / gridDim.x);
    int t = begin < end ? tensor_of(p, begin) : 0;
    grid_wait();
    Squares acc;
    for (int piece = begin; piece < end; ++piece) {
        while (p.start[t + 1] <= piece) ++t;
        const Piece c = piece_of(p, t, piece);
        const int dt = p.dtype[t];
        const bool keep = end - piece <= GC_KEEP;
        if (dt == F32) piece_squares<F32>(acc, p.in[t], p.numel[t], c, p.status, keep);
        else if (dt == F16) piece_squares<F16>(acc, p.in[t], p.numel[t], c, p.status, keep);
        else piece_squares<BF16>(acc, p.in[t], p.numel[t], c, p.status, keep);
    }
    const float sum = block_sum(acc.sum + acc.err, s_part[0]);
    const bool scaled = __syncthreads_or(acc.small != 0.f || acc.large != 0.f);
    float small = 0.f, large = 0.f;
    if (scaled) {
        small = block_sum(acc.small, s_part[1]);
        large = block_sum(acc.large, s_part[2]);
    }
    if (threadIdx.x == 0) {
        double r = (double)sum;
        if (scaled) r += (double)small * 0x1p-192 + (double)large * 0x1p192;
        p.records[blockIdx.x] = r;
        for (int k = blockIdx.x + gridDim.x; k < TB_GRAD_PARTS; k += gridDim.x) p.records[k] = 0.0;
    }
}

// The norm from all records, the same in every CTA: the records' fp64 values
// are added in 64-bit fixed point relative to the largest one's exponent (exact
// sums, in any order, on the integer units: fp64 additions took longer than
// the rest of a small clip, 10 of 18 us for 3.5 M elements).  An infinite
// record makes the norm infinite, a NaN one NaN.
__device__ __forceinline__ float norm_of(const double* records, int64_t n) {
    __shared__ uint32_t s_max[GC_BLOCK / 32];
    __shared__ unsigned long long s_sum[GC_BLOCK / 32];
    constexpr int KEEP = TB_GRAD_PARTS / GC_BLOCK;  // one record set stays in registers
    const unsigned long long* const bits = reinterpret_cast<const unsigned long long*>(records);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    unsigned long long r[KEEP];
    uint32_t top = 0u;
#pragma unroll
    for (int k = 0; k < KEEP; ++k) {
        const int64_t i = threadIdx.x + k * GC_BLOCK;
        r[k] = i < n ? bits[i] : 0ull;
        top = max(top, (uint32_t)(r[k] >> 32));
    }
    for (int64_t i = threadIdx.x + KEEP * GC_BLOCK; i < n; i += GC_BLOCK) top = max(top, (uint32_t)(bits[i] >> 32));
    top = __reduce_max_sync(0xffffffffu, top);
    if (lane == 0) s_max[warp] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < GC_BLOCK / 32; ++w) top = max(top, s_max[w]);
    if (top >= 0x7ff00000u) return top == 0x7ff00000u ? INFINITY : NAN;
    // 53-bit mantissas: 1024 of them fit 63 bits, more are shifted down
    const int head = n <= 1024 ? 0 : 64 - __clzll(n - 1) - 10;
    const int e_top = (int)(top >> 20);
    unsigned long long sum = 0ull;
    auto add = [&](unsigned long long v) {
        const int e = (int)(v >> 52);
        const int shift = e_top - e + head;
        if (e > 0 && shift < 64) sum += ((v & 0xfffffffffffffull) | 0x10000000000000ull) >> shift;
    };
#pragma unroll
    for (int k = 0; k < KEEP; ++k) add(r[k]);
    for (int64_t i = threadIdx.x + KEEP * GC_BLOCK; i < n; i += GC_BLOCK) add(bits[i]);
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if (lane == 0) s_sum[warp] = sum;
    __syncthreads();
    sum = 0ull;
#pragma unroll
    for (int w = 0; w < GC_BLOCK / 32; ++w) sum += s_sum[w];
    // sqrt(sum * 2^e): fp32 roundings of the sum, the root and the result
    const int e = e_top - 1075 + head;
    const float odd = (e & 1) ? 2.f : 1.f;
    return ldexpf(sqrtf((float)sum * odd), (e - (e & 1)) / 2);
}

template <int DT>
__device__ __forceinline__ void piece_scale(const void* in, void* out, int64_t numel, const Piece& c, float coef,
                                            uint32_t* status) {
    constexpr int VEC = 16 / elem_size(DT);
    using E = typename Word<elem_size(DT)>::T;
    const char* const b = reinterpret_cast<const char*>(in);
    char* const o = reinterpret_cast<char*>(out);
    const int64_t bytes = numel * elem_size(DT);
    const uint4* const src = reinterpret_cast<const uint4*>(b + c.first * elem_size(DT));
    char* const dst = o + c.first * elem_size(DT);
    const bool same = ((reinterpret_cast<uintptr_t>(dst)) & 15u) == 0;  // out shares the input's alignment
    uint4 v[GC_CPT];
#pragma unroll
    for (int k = 0; k < GC_CPT; ++k) {
        const int i = threadIdx.x + k * GC_BLOCK;
        v[k] = make_uint4(0u, 0u, 0u, 0u);
        if (i < c.n && in_bounds(src + i, 16, b, bytes, status)) v[k] = src[i];
    }
    const int64_t single = threadIdx.x < VEC ? threadIdx.x : c.rest + (threadIdx.x - VEC);
    const bool has = threadIdx.x < VEC ? threadIdx.x < c.head : threadIdx.x < 2 * VEC && single < numel;
    if (has && in_bounds(b + single * elem_size(DT), elem_size(DT), b, bytes, status)) {
        float f[1];
        unpack<DT, 1>(reinterpret_cast<const E*>(b)[single], f);
        f[0] *= coef;
        reinterpret_cast<E*>(o)[single] = pack<DT, 1>(f);
    }
#pragma unroll
    for (int k = 0; k < GC_CPT; ++k) {
        const int i = threadIdx.x + k * GC_BLOCK;
        if (i >= c.n) continue;
        float f[VEC];
        unpack<DT, VEC>(v[k], f);
#pragma unroll
        for (int q = 0; q < VEC; ++q) f[q] *= coef;
        const uint4 w = pack<DT, VEC>(f);
        if (!in_bounds(dst + (int64_t)i * 16, 16, o, bytes, status)) continue;
        if (same) {
            __stcs(reinterpret_cast<uint4*>(dst) + i, w);
        } else {
#pragma unroll
            for (int q = 0; q < VEC; ++q) {
                const float g[1] = {f[q]};
                reinterpret_cast<E*>(dst)[i * VEC + q] = pack<DT, 1>(g);
            }
        }
    }
}

template <int MAXT>
__global__ void __launch_bounds__(GC_BLOCK, GC_CTAS) grad_clip_kernel(const __grid_constant__ GradParams<MAXT> p) {
    const int64_t total = p.start[p.T];
    const int begin = (int)(total * blockIdx.x / gridDim.x), end = (int)(total * (blockIdx.x + 1) / gridDim.x);
    int t = begin < end ? tensor_of(p, end - 1) : 0;
    grid_wait();
    const float norm = norm_of(p.records, p.n_records);
    if (p.first && p.norm != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *p.norm = norm;
    const float q = p.max_norm / (norm + 1e-6f);
    const float coef = q >= 1.f ? 1.f : q;  // a NaN stays one
    for (int piece = end - 1; piece >= begin; --piece) {
        while (p.start[t] > piece) --t;
        if (coef == 1.f && p.in[t] == p.out[t]) continue;  // in place, nothing to change
        const Piece c = piece_of(p, t, piece);
        const int dt = p.dtype[t];
        if (dt == F32) piece_scale<F32>(p.in[t], p.out[t], p.numel[t], c, coef, p.status);
        else if (dt == F16) piece_scale<F16>(p.in[t], p.out[t], p.numel[t], c, coef, p.status);
        else piece_scale<BF16>(p.in[t], p.out[t], p.numel[t], c, coef, p.status);
    }
}

struct GradNormParams {
    const double* records;
    int64_t n;
    float* norm;
};

__global__ void __launch_bounds__(GC_BLOCK) grad_norm_kernel(const __grid_constant__ GradNormParams p) {
    grid_wait();
    const float norm = norm_of(p.records, p.n);
    if (threadIdx.x == 0) *p.norm = norm;
}

template <int MAXT>
unsigned grad_grid(const GradParams<MAXT>& p, int sms) {
    int64_t g = (int64_t)sms * GC_CTAS;
    if (g > TB_GRAD_PARTS) g = TB_GRAD_PARTS;
    if (g > p.start[p.T]) g = p.start[p.T];
    return (unsigned)(g < 1 ? 1 : g);
}

}  // namespace

cudaError_t launch_grad_stats(const GradParamsSmall& p, int sms, cudaStream_t s) {
    return launch_pdl(grad_stats_kernel<GRAD_SMALL_MAXT>, p, dim3(grad_grid(p, sms)), GC_BLOCK, 0, s);
}
cudaError_t launch_grad_stats(const GradParamsLarge& p, int sms, cudaStream_t s) {
    return launch_pdl(grad_stats_kernel<GRAD_MAXT>, p, dim3(grad_grid(p, sms)), GC_BLOCK, 0, s);
}
cudaError_t launch_grad_clip(const GradParamsSmall& p, int sms, cudaStream_t s) {
    return launch_pdl(grad_clip_kernel<GRAD_SMALL_MAXT>, p, dim3(grad_grid(p, sms)), GC_BLOCK, 0, s);
}
cudaError_t launch_grad_clip(const GradParamsLarge& p, int sms, cudaStream_t s) {
    return launch_pdl(grad_clip_kernel<GRAD_MAXT>, p, dim3(grad_grid(p, sms)), GC_BLOCK, 0, s);
}
cudaError_t launch_grad_norm(const double* records, int64_t n, float* norm, cudaStream_t s) {
    GradNormParams p = {records, n, norm};
    return launch_pdl(grad_norm_kernel, p, dim3(1), GC_BLOCK, 0, s);
}

}  // namespace tb
