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
// Within a piece a thread adds the squares of its elements in fp32 and
// carries the pieces' sums in fp64.  A thread whose fp32 sum could have
// overflowed or lost squares to underflow takes them again scaled by a power
// of two, so any finite gradients give their norm wherever fp32 can hold it.
#include "tb_elem.cuh"

namespace tb {
namespace {

constexpr int GC_BLOCK = 256;
constexpr int GC_CTAS = 6;                                    // per SM
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
// may miss squares that underflowed, one above HIGH may be about to overflow.
constexpr float SQ_LOW = 0x1p-90f, SQ_HIGH = 0x1p120f;
constexpr float SQ_SCALE = 0x1p96f;

template <int DT>
__device__ __forceinline__ double piece_squares(const void* base, int64_t numel, const Piece& c, uint32_t* status) {
    constexpr int VEC = 16 / elem_size(DT);
    const char* const b = reinterpret_cast<const char*>(base);
    const int64_t bytes = numel * elem_size(DT);
    const uint4* const src = reinterpret_cast<const uint4*>(b + c.first * elem_size(DT));
    uint4 v[GC_CPT];
#pragma unroll
    for (int k = 0; k < GC_CPT; ++k) {
        const int i = threadIdx.x + k * GC_BLOCK;
        v[k] = make_uint4(0u, 0u, 0u, 0u);
        if (i < c.n && in_bounds(src + i, 16, b, bytes, status)) v[k] = src[i];
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
    const float s = total(1.f);
    if (s > SQ_LOW && s < SQ_HIGH) return (double)s;
    if (s < 1.f) return (double)total(SQ_SCALE) * 0x1p-192;
    return (double)total(1.f / SQ_SCALE) * 0x1p192;
}

__device__ __forceinline__ double block_sum(double v, double* slots) {
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    if ((threadIdx.x & 31) == 0) slots[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.0;
#pragma unroll
    for (int w = 0; w < GC_BLOCK / 32; ++w) v += slots[w];
    return v;
}

template <int MAXT>
__global__ void __launch_bounds__(GC_BLOCK, GC_CTAS) grad_stats_kernel(const __grid_constant__ GradParams<MAXT> p) {
    __shared__ double s_part[GC_BLOCK / 32];
    const int64_t total = p.start[p.T];
    const int begin = (int)(total * blockIdx.x / gridDim.x), end = (int)(total * (blockIdx.x + 1) / gridDim.x);
    int t = begin < end ? tensor_of(p, begin) : 0;
    grid_wait();
    double acc = 0.0;
    for (int piece = begin; piece < end; ++piece) {
        while (p.start[t + 1] <= piece) ++t;
        const Piece c = piece_of(p, t, piece);
        const int dt = p.dtype[t];
        if (dt == F32) acc += piece_squares<F32>(p.in[t], p.numel[t], c, p.status);
        else if (dt == F16) acc += piece_squares<F16>(p.in[t], p.numel[t], c, p.status);
        else acc += piece_squares<BF16>(p.in[t], p.numel[t], c, p.status);
    }
    acc = block_sum(acc, s_part);
    if (threadIdx.x == 0) {
        p.records[blockIdx.x] = acc;
        for (int k = blockIdx.x + gridDim.x; k < TB_GRAD_PARTS; k += gridDim.x) p.records[k] = 0.0;
    }
}

// The norm from all records, the same in every CTA.
__device__ __forceinline__ float norm_of(const double* records, int64_t n, double* slots) {
    double v = 0.0;
    for (int64_t k = threadIdx.x; k < n; k += GC_BLOCK) v += records[k];
    return (float)sqrt(block_sum(v, slots));
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
    __shared__ double s_part[GC_BLOCK / 32];
    const int64_t total = p.start[p.T];
    const int begin = (int)(total * blockIdx.x / gridDim.x), end = (int)(total * (blockIdx.x + 1) / gridDim.x);
    int t = begin < end ? tensor_of(p, end - 1) : 0;
    grid_wait();
    const float norm = norm_of(p.records, p.n_records, s_part);
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
    __shared__ double s_part[GC_BLOCK / 32];
    grid_wait();
    const float norm = norm_of(p.records, p.n, s_part);
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
