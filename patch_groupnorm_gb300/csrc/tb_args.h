// tb_args.h -- what the host files check arguments with.
#pragma once

#include <cstdint>

#include "tb_internal.h"
#include "tileblend.h"

#define TB_API extern "C" __attribute__((visibility("default")))

#define TB_TRY(call)                          \
    do {                                      \
        const tb_status try_status = (call);  \
        if (try_status != TB_OK) return try_status; \
    } while (0)

namespace tb {

inline tb_status launched(cudaError_t e) {
    if (e == cudaSuccess) return TB_OK;
    record_cuda_error(e);
    return TB_ERR_CUDA;
}

inline bool known(tb_dtype d) { return d == TB_F32 || d == TB_F16 || d == TB_BF16; }
inline int elem_bytes(tb_dtype d) { return d == TB_F32 ? 4 : 2; }
inline bool aligned(const void* p, int bytes) { return ((uintptr_t)p & (uintptr_t)(bytes - 1)) == 0; }

}  // namespace tb
