// MXFP4 x MXFP4 products: which kernel serves which sizes.
#include "launch.hpp"
#include "mxfp4_epilogue.hpp"

namespace mxfp4 {

hipError_t launch_gemm_tiled(const uint8_t *xq, const uint8_t *xs, const uint8_t *wq,
                             const uint8_t *ws, const Groups &g, int N, int K, int epilogue,
                             const Output &o, hipStream_t stream);
hipError_t launch_gemm_decode(const uint8_t *xq, const uint8_t *xs, const uint8_t *wq,
                              const uint8_t *ws, const Groups &g, int N, int K, int epilogue,
                              const Output &o, int row_tiles, hipStream_t stream);

// Few rows stream the weights (mxfp4_decode.hip), many take LDS tiles
// (mxfp4_tiled.hip). Measured, us, streaming with 16, 32, 64 rows against 64 x 64
// (64 x 128) tiles: dense N = K = 4096, M = 16 4.3, 4.7, 6.0 against 7.4; M = 32
// 5.4, 4.8, 5.9 / 7.5; M = 64 8.0, 7.9, 6.6 / 8.1; M = 96 11.8, 11.4, 9.0 / 8.0;
// 257 x 1040 x 1312 5.5, 6.2, 4.4 / 5.1. 32 experts' down products [4096, 2048],
// 8 rows each on average 24.9, 26.8, 36.1 / 32.1, 32 rows 47.9, 39.4, 45.3 / 36.2.
hipError_t launch_gemm(const uint8_t *xq, const uint8_t *xs, const uint8_t *wq, const uint8_t *ws,
                       const Groups &g, int N, int K, int epilogue, const Output &o,
                       hipStream_t stream) {
    int row_tiles = 0;  // 16-row tiles that stream the weights together
    if (g.offsets) {
        // the groups' sizes are on the device: their average decides
        if ((int64_t)g.S <= 12ll * g.E) row_tiles = 1;
        else if ((int64_t)g.S <= 24ll * g.E) row_tiles = 2;
    } else {
        const int64_t tiles = (int64_t)((g.S + 63) / 64) * ((N + 63) / 64);
        if (g.S <= 16) row_tiles = 1;
        else if (g.S <= 32) row_tiles = 2;
        else if (2 * tiles < w8a8::device_cu_count()) row_tiles = 4;  // half the CUs idle with tiles
    }
    if (row_tiles > 0)
        return launch_gemm_decode(xq, xs, wq, ws, g, N, K, epilogue, o, row_tiles, stream);
    return launch_gemm_tiled(xq, xs, wq, ws, g, N, K, epilogue, o, stream);
}

}  // namespace mxfp4
