// tb_elem.cuh -- element and chunk helpers of the training kernels (layer
// norm, gradient clipping, PatchGroupNorm's backward pass).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "tb_internal.h"

namespace tb {

__host__ __device__ constexpr int elem_size(int dt) { return dt == F32 ? 4 : 2; }

// A chunk: VEC neighbouring elements, loaded and stored as one word of
// VEC * elem_size(DT) bytes (2, 4, 8 or 16).
template <int BYTES>
struct Word;
template <>
struct Word<16> {
    using T = uint4;
};
template <>
struct Word<8> {
    using T = uint2;
};
template <>
struct Word<4> {
    using T = uint32_t;
};
template <>
struct Word<2> {
    using T = unsigned short;
};

template <int DT>
__device__ __forceinline__ float elem_to_f(uint32_t bits) {
    if constexpr (DT == F32) {
        return __uint_as_float(bits);
    } else if constexpr (DT == F16) {
        return __half2float(__ushort_as_half((unsigned short)bits));
    } else {
        return __uint_as_float(bits << 16);
    }
}

// Two 16-bit elements of a 32-bit word, low half first.
template <int DT>
__device__ __forceinline__ void pair_to_f(uint32_t v, float& lo, float& hi) {
    if constexpr (DT == F16) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&v));
        lo = f.x;
        hi = f.y;
    } else {
        lo = __uint_as_float(v << 16);
        hi = __uint_as_float(v & 0xffff0000u);
    }
}

// Round to nearest even, once, into the storage type.
template <int DT>
__device__ __forceinline__ uint32_t f_to_pair(float lo, float hi) {
    if constexpr (DT == F16) {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
}

template <int DT, int VEC>
__device__ __forceinline__ void unpack(const typename Word<VEC * elem_size(DT)>::T& w, float (&f)[VEC]) {
    if constexpr (VEC == 1) {
        f[0] = elem_to_f<DT>((uint32_t)w);
    } else {
        uint32_t u[VEC * elem_size(DT) / 4];
        *reinterpret_cast<typename Word<VEC * elem_size(DT)>::T*>(u) = w;
#pragma unroll
        for (int q = 0; q < VEC * elem_size(DT) / 4; ++q) {
            if constexpr (DT == F32) {
                f[q] = __uint_as_float(u[q]);
            } else {
                pair_to_f<DT>(u[q], f[2 * q], f[2 * q + 1]);
            }
        }
    }
}

template <int DT, int VEC>
__device__ __forceinline__ typename Word<VEC * elem_size(DT)>::T pack(const float (&f)[VEC]) {
    if constexpr (VEC == 1) {
        if constexpr (DT == F32) {
            return __float_as_uint(f[0]);
        } else {
            return (unsigned short)(f_to_pair<DT>(f[0], 0.f) & 0xffffu);
        }
    } else {
        uint32_t u[VEC * elem_size(DT) / 4];
#pragma unroll
        for (int q = 0; q < VEC * elem_size(DT) / 4; ++q) {
            if constexpr (DT == F32) {
                u[q] = __float_as_uint(f[q]);
            } else {
                u[q] = f_to_pair<DT>(f[2 * q], f[2 * q + 1]);
            }
        }
        return *reinterpret_cast<const typename Word<VEC * elem_size(DT)>::T*>(u);
    }
}

// fp32 arithmetic on pairs of lanes (one instruction for two elements, each
// lane rounded as the scalar instruction rounds) and on single elements.
using f32x2 = unsigned long long;

__device__ __forceinline__ f32x2 pair(float lo, float hi) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void halves(f32x2 v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ f32x2 vadd(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 vsub(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 vmul(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 vfma(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ float vsum(f32x2 v) {
    float lo, hi;
    halves(v, lo, hi);
    return lo + hi;
}
__device__ __forceinline__ float vadd(float a, float b) { return a + b; }
__device__ __forceinline__ float vsub(float a, float b) { return a - b; }
__device__ __forceinline__ float vmul(float a, float b) { return a * b; }
__device__ __forceinline__ float vfma(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ float vsum(float v) { return v; }

// The lanes of a chunk: VEC / 2 pairs, or one single element.
template <int VEC>
struct Lanes {
    using T = f32x2;
    static constexpr int N = VEC / 2;
    __device__ __forceinline__ static T splat(float v) { return pair(v, v); }
};
template <>
struct Lanes<1> {
    using T = float;
    static constexpr int N = 1;
    __device__ __forceinline__ static T splat(float v) { return v; }
};

template <int DT, int VEC>
__device__ __forceinline__ void to_lanes(const typename Word<VEC * elem_size(DT)>::T& w,
                                         typename Lanes<VEC>::T (&f)[Lanes<VEC>::N]) {
    float e[VEC];
    unpack<DT, VEC>(w, e);
    if constexpr (VEC == 1) {
        f[0] = e[0];
    } else {
#pragma unroll
        for (int q = 0; q < VEC / 2; ++q) f[q] = pair(e[2 * q], e[2 * q + 1]);
    }
}

template <int DT, int VEC>
__device__ __forceinline__ typename Word<VEC * elem_size(DT)>::T from_lanes(
    const typename Lanes<VEC>::T (&f)[Lanes<VEC>::N]) {
    float e[VEC];
    if constexpr (VEC == 1) {
        e[0] = f[0];
    } else {
#pragma unroll
        for (int q = 0; q < VEC / 2; ++q) halves(f[q], e[2 * q], e[2 * q + 1]);
    }
    return pack<DT, VEC>(e);
}

// Element i of a weight vector whose type is the rows' or f32, as f32.
__device__ __forceinline__ float weight_at(const void* w, int dtype, int64_t i, float dflt) {
    if (w == nullptr) return dflt;
    if (dtype == F32) return reinterpret_cast<const float*>(w)[i];
    const uint32_t v = reinterpret_cast<const unsigned short*>(w)[i];
    return dtype == F16 ? elem_to_f<F16>(v) : elem_to_f<BF16>(v);
}

// VEC neighbouring weights starting at element i (16-byte aligned where VEC > 1).
template <int VEC>
__device__ __forceinline__ void weights_at(const void* w, int dtype, int64_t i, float dflt, float (&f)[VEC]) {
    if (w == nullptr) {
#pragma unroll
        for (int q = 0; q < VEC; ++q) f[q] = dflt;
    } else if constexpr (VEC == 1) {
        f[0] = weight_at(w, dtype, i, dflt);
    } else if (dtype == F32) {
#pragma unroll
        for (int q = 0; q < VEC; q += 4) {
            const float4 v = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(w) + i + q);
            f[q] = v.x;
            f[q + 1] = v.y;
            f[q + 2] = v.z;
            f[q + 3] = v.w;
        }
    } else {
        if constexpr (VEC == 8) {
            const uint4 v = *reinterpret_cast<const uint4*>(reinterpret_cast<const unsigned short*>(w) + i);
            if (dtype == F16) unpack<F16, 8>(v, f);
            else unpack<BF16, 8>(v, f);
        }
    }
}

// One chunk's weights as fp32 lanes (16-byte aligned where VEC > 1).
template <int VEC>
__device__ __forceinline__ void weight_lanes(const void* w, int dtype, int64_t i, float dflt,
                                             typename Lanes<VEC>::T (&f)[Lanes<VEC>::N]) {
    float e[VEC];
    weights_at<VEC>(w, dtype, i, dflt, e);
    if constexpr (VEC == 1) {
        f[0] = e[0];
    } else {
#pragma unroll
        for (int q = 0; q < VEC / 2; ++q) f[q] = pair(e[2 * q], e[2 * q + 1]);
    }
}

__device__ __forceinline__ void store_weight(void* w, int dtype, int64_t i, float v) {
    if (dtype == F32) {
        reinterpret_cast<float*>(w)[i] = v;
    } else {
        reinterpret_cast<unsigned short*>(w)[i] =
            (unsigned short)((dtype == F16 ? f_to_pair<F16>(v, 0.f) : f_to_pair<BF16>(v, 0.f)) & 0xffffu);
    }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}

// --- copies of whole rows into shared memory, completing on an mbarrier -------

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_init_fence() { asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory"); }
__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t phase) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(phase)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ uint64_t timer_ns() {
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}
// A wait for copies gives up after this long (nanoseconds).
constexpr uint64_t BAR_WAIT_NS = 1000000000ull;
// Waits for the phase of `bar`; false, with DEV_WAIT_TIMEOUT recorded, if it
// does not complete in time.
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t phase, uint32_t* status) {
    if (bar_try(bar, phase)) return true;
    const uint64_t t0 = timer_ns();
    while (!bar_try(bar, phase)) {
        if (timer_ns() - t0 > BAR_WAIT_NS) {
            if (status != nullptr) atomicCAS(status, (uint32_t)DEV_OK, (uint32_t)DEV_WAIT_TIMEOUT);
            return false;
        }
    }
    return true;
}
// `bytes` (a multiple of 16) from global memory, both addresses 16-byte
// aligned; counts towards the phase of `bar`.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}
// The same for bytes that nobody reads again soon: L2 may drop them first.
__device__ __forceinline__ void bulk_load_once(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    uint64_t policy;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(
            dst),
        "l"(src), "r"(bytes), "r"(bar), "l"(policy)
        : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// For the bulk copies that come after this fence (and a barrier in between):
// elements that were copied one by one, by this thread or before a barrier that it
// has passed, are in place, and a bulk copy may overwrite them.
__device__ __forceinline__ void bulk_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
// One of the elements on either side of a bulk copy, into shared memory.
template <int ES>
__device__ __forceinline__ void copy_element(uint32_t to, const char* from) {
    if constexpr (ES == 4) {
        asm volatile("st.shared.u32 [%0], %1;" ::"r"(to), "r"(*reinterpret_cast<const uint32_t*>(from)) : "memory");
    } else {
        asm volatile("st.shared.u16 [%0], %1;" ::"r"(to), "h"(*reinterpret_cast<const unsigned short*>(from))
                     : "memory");
    }
}
template <int ES>
__device__ __forceinline__ uint32_t smem_element(uint32_t at) {
    if constexpr (ES == 4) {
        uint32_t v;
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(at));
        return v;
    } else {
        unsigned short v;
        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(at));
        return v;
    }
}
template <typename W>
__device__ __forceinline__ W smem_load(uint32_t at) {
    static_assert(sizeof(W) == 16, "16-byte words");
    W v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
    return v;
}

// Waits until the grids before this one on the stream have completed and
// their writes are visible (launches use programmatic stream serialisation).
// What they may have written is read behind the wait with coherent loads: the read-only
// path (__ldg) is for what nothing writes while a kernel is resident, and its loads need
// not stay behind the wait.
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Launches `fn` with programmatic stream serialisation, as every kernel of
// the library is launched.
template <typename P>
inline cudaError_t launch_pdl(void (*fn)(const P), const P& p, dim3 grid, int block, size_t smem, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)block, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fn, p);
}

}  // namespace tb
