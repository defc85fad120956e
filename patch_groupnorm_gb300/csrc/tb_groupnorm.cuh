// tb_groupnorm.cuh -- what PatchGroupNorm's forward and backward kernels share.
#pragma once

#include "tb_internal.h"

namespace tb {

// Pooled (mean, rstd) of group g of sample n from the part records, computed
// by one warp.  `partials` holds R record sets of [N][G][TB_GN_PARTS] (the
// sets of one or more statistics calls, e.g. gathered from every rank), and
// every record describes itself: records with count 0 hold no elements and
// are skipped, whichever call wrote them and however it split its units.
// Each record (count c, mean m, M2) adds c, c * (m - K) and
// M2 + c * (m - K)^2 to three sums taken about K, the mean of the first
// record with elements (so the sums do not cancel); then
//     mean = K + S1 / n,   M2 = S2 - S1^2 / n   (Chan's combination, summed),
// and the variance is M2 / n, biased.  Counts are summed exactly in 64 bits
// and converted to fp32 once.  Lane 0 holds the result.
// P: the parameters of the apply or of the backward pass.
template <typename P>
__device__ __forceinline__ void pooled_stats(const P& p, int64_t n, int64_t g, float& mean, float& rstd, float& count) {
    const int lane = threadIdx.x & 31;
    const int total = p.R * TB_GN_PARTS;
    const int64_t set_stride = p.N * p.G * TB_GN_PARTS;  // records between consecutive sets
    const GnPartial* const unit0 = p.partials + (n * p.G + g) * TB_GN_PARTS;
    auto record = [&](int q, long long& c, float& m, float& m2) {
        const int r = q / TB_GN_PARTS, k = q - r * TB_GN_PARTS;
        const GnPartial* const at = unit0 + r * set_stride + k;
        if (!in_bounds(at, sizeof(GnPartial), p.partials, (int64_t)p.R * set_stride * (int64_t)sizeof(GnPartial),
                       p.status)) {
            c = 0;
            m = m2 = 0.f;
            return;
        }
        const longlong2 raw = __ldg(reinterpret_cast<const longlong2*>(at));
        c = raw.x;
        m = __int_as_float((int)(raw.y & 0xffffffffLL));
        m2 = __int_as_float((int)(raw.y >> 32));
    };
    // the first 32 records stay in registers (all of them when R <= 4)
    long long c0 = 0;
    float m0 = 0.f, v0 = 0.f;
    if (lane < total) record(lane, c0, m0, v0);
    float K = 0.f;
    unsigned has = __ballot_sync(0xffffffffu, c0 > 0);
    if (has != 0u) {
        K = __shfl_sync(0xffffffffu, m0, __ffs(has) - 1);
    } else {
        for (int base = 32; base < total; base += 32) {
            long long c = 0;
            float m = 0.f, m2 = 0.f;
            if (base + lane < total) record(base + lane, c, m, m2);
            has = __ballot_sync(0xffffffffu, c > 0);
            if (has != 0u) {
                K = __shfl_sync(0xffffffffu, m, __ffs(has) - 1);
                break;
            }
        }
    }
    long long sn = 0;
    float s1 = 0.f, s2 = 0.f;
    auto add = [&](long long c, float m, float m2) {
        if (c > 0) {
            const float cf = (float)c;
            const float d = m - K;
            sn += c;
            s1 = fmaf(cf, d, s1);
            s2 += fmaf(cf * d, d, m2);
        }
    };
    add(c0, m0, v0);
    for (int q = lane + 32; q < total; q += 32) {
        long long c;
        float m, m2;
        record(q, c, m, m2);
        add(c, m, m2);
    }
#pragma unroll
    for (int delta = 16; delta >= 1; delta >>= 1) {  // fixed order: deterministic
        sn += __shfl_down_sync(0xffffffffu, sn, delta);
        s1 += __shfl_down_sync(0xffffffffu, s1, delta);
        s2 += __shfl_down_sync(0xffffffffu, s2, delta);
    }
    const float nf = (float)sn;
    const float q1 = sn > 0 ? s1 / nf : 0.f;
    const float var = sn > 0 ? fmaxf(0.f, fmaf(-s1, q1, s2) / nf) : 0.f;  // biased: divide by the count
    mean = K + q1;
    rstd = 1.0f / sqrtf(var + p.eps);
    count = nf;
}

// silu(z) = z / (1 + e^-z), with e^-z = 2^(-z log2 e) and the reciprocal
// from the approximate special-function unit (relative errors ~2^-22, far
// inside the output tolerances).  Flushing subnormals there is harmless:
// e^-z is subnormal only for z > 87, where 1 + e^-z rounds to 1, and the
// reciprocal only for z < -87, where silu(z) lies below 1e-35.
__device__ __forceinline__ float ex2_ftz(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp_ftz(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

}  // namespace tb
