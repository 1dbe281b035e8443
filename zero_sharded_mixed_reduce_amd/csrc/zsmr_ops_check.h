// The checks of arguments that the host files of the operators share.  Internal,
// not part of the public ABI.
#pragma once
#include <cstdint>

#include "zsmr_ctx.h"
#include "zsmr_ops.h"

namespace zsmr {

inline int32_t done(hipError_t e) { return e == hipSuccess ? ZSMR_OK : hip_fail(e); }

// rows x width elements of 16 bits, stride apart
inline int32_t check_rows(const void* p, int64_t rows, int64_t width, int64_t stride) {
    if (!p && rows > 0) return ZSMR_ERR_ARG;
    if (stride < width || stride > ZSMR_MAX_WIDTH) return ZSMR_ERR_ARG;
    return al(p, 2) ? ZSMR_OK : ZSMR_ERR_ALIGN;
}

inline int32_t check_sizes(int64_t tokens, int64_t vocab, int64_t width) {
    if (tokens < 0 || tokens > ZSMR_MAX_TOKENS || vocab < 1 || vocab > ZSMR_MAX_VOCAB ||
        width < 1 || width > ZSMR_MAX_WIDTH)
        return ZSMR_ERR_ARG;
    return ZSMR_OK;
}

inline int32_t check_ids(const void* ids, int32_t id_bytes, int64_t tokens) {
    if ((id_bytes != 4 && id_bytes != 8) || (!ids && tokens > 0)) return ZSMR_ERR_ARG;
    return al(ids, id_bytes) ? ZSMR_OK : ZSMR_ERR_ALIGN;
}

inline int32_t check_space(const void* ws, int64_t ws_bytes, int64_t need) {
    if (need > 0 && (!ws || ws_bytes < need)) return ZSMR_ERR_ARG;
    return al(ws, 16) ? ZSMR_OK : ZSMR_ERR_ALIGN;
}

}  // namespace zsmr
