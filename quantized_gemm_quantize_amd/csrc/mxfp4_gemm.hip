// MXFP4 x MXFP4 products: which kernel serves which sizes.
#include "launch.hpp"
#include "mxfp4_epilogue.hpp"
#include "mxfp4_form.hpp"

namespace mxfp4 {

hipError_t launch_gemm_tiled(const uint8_t *xq, const uint8_t *xs, const uint8_t *wq,
                             const uint8_t *ws, const Groups &g, int N, int K, int epilogue,
                             const Output &o, const Form &f, hipStream_t stream);
hipError_t launch_gemm_decode(const uint8_t *xq, const uint8_t *xs, const uint8_t *wq,
                              const uint8_t *ws, const Groups &g, int N, int K, int epilogue,
                              const Output &o, const Form &f, hipStream_t stream);

namespace {

// Channels and wavefronts of a workgroup that streams. Grouped rows: 64 channels by 2
// wavefronts (40 KB of LDS: four workgroups of a CU hide each other's start and
// end; 32 experts' down products of 8 rows, 25.5 us against 28.5 with 4
// wavefronts), unless there are too few workgroups for that: 4 wavefronts
// (1 token, 4 experts: gate and up 9.6 against 10.2 us, down 5.6 against 6.1).
// Dense: 16 channels by 8 wavefronts, as a single weight has few channels.
Form streaming_form(int row_tiles, const Rows &r, int N, int epilogue, int64_t cus) {
    const int rows = 16 * row_tiles;
    if (!r.grouped) return Form{true, rows, 16, row_tiles < 4 ? 8 : 4};
    if (most_tiles(r.S, r.E, rows, true) * ((N + 63) / 64) > 2 * cus) return Form{true, rows, 64, 2};
    return Form{true, rows, epilogue == kSwiglu ? 64 : 32, 4};
}

// The smallest tile whose tiles all run at once (one workgroup per CU),
// else 256 x 256, whose operands' bytes per product are the fewest. Measured
// at N = K = 4096 (us; 64x64, 64x128, 128x128, 256x128, 256x256): M = 256
// 8.6, 10.0, 11.3, 14.3, 25.3; M = 384 10.9, 10.4, 11.5, 14.4, 25.2; M = 768
// 16.4, 14.6, 12.4, 15.3, 26.5; M = 1536 28.1, 23.4, 24.1, 17.5, 27.6; M = 4096
// 68.5, 54.4, 49.5, 47.5, 36.1.
// Short K: two workgroups of 256 x 128 per CU with 128-element stages, whose
// starts and stores overlap each other's products (8192 x 8192, against 256 x
// 256: K = 512 43.3 -> 39.2 us, K = 1024 56.0 -> 56.3, K = 2048 81.4 -> 89.6; 32
// experts' gate and up [2944, 960] with 285 rows each 41.3 -> 35.4).
// Small groups: 64 rows, as a taller tile is mostly empty (32 experts with 64
// rows each: gate and up [4096, 4096] 82.1 -> 77.5, down [4096, 2048] 45.1 -> 38.9;
// with 256 rows 111 -> 152 and 63 -> 82).
Form tiled_form(const Rows &r, int N, int K, int epilogue, int64_t cus) {
    auto tiles = [&](int bm, int bn) {
        return most_tiles(r.S, r.E, bm, r.grouped) * ((N + bn - 1) / bn);
    };
    if (tiles(64, 64) <= cus && epilogue != kSwiglu) return Form{false, 64, 64, 4};
    if (tiles(64, 128) <= cus) return Form{false, 64, 128, 4};
    if (r.grouped && r.S < 96ll * r.E) return Form{false, 64, 128, 4};
    if (tiles(128, 128) <= cus) return Form{false, 128, 128, 8};
    if (tiles(256, 128) <= cus) return Form{false, 256, 128, 8};
    if (K <= 1024) return Form{false, 256, 128, 4};
    return Form{false, 256, 256, 8};
}

}  // namespace

// Few rows stream the weights (mxfp4_decode.hip), many take LDS tiles
// (mxfp4_tiled.hip). Measured, us, streaming with 16, 32, 64 rows against 64 x 64
// (64 x 128) tiles: dense N = K = 4096, M = 16 4.3, 4.7, 6.0 against 7.4; M = 32
// 5.4, 4.8, 5.9 / 7.5; M = 64 8.0, 7.9, 6.6 / 8.1; M = 96 11.8, 11.4, 9.0 / 8.0;
// 257 x 1040 x 1312 5.5, 6.2, 4.4 / 5.1. 32 experts' down products [4096, 2048],
// 8 rows each on average 24.9, 26.8, 36.1 / 32.1, 32 rows 47.9, 39.4, 45.3 / 36.2.
// More than 32 dense rows stream, 64 at a time by 16 channels, while tiles would
// leave half the CUs idle and the streaming workgroups, each of which reads its rows and
// its channels itself, run at once, or K is short and the starts count (streaming
// against tiles, us: 64 x 1040 x 4096 5.8 / 7.2, 1000 x 256 x 8192 9.6 / 12.3, 8000 x
// 16 x 4096 7.6 / 7.9; past the CUs 257 x 1040 3.7 / 4.6 for K = 1024, 9.6 / 8.0 for
// 4096, 1500 x 304 x 2048 7.7 / 5.6, 8000 x 64 x 8192 27.4 / 12.9).
Form product_form(const Rows &r, int N, int K, int epilogue, int64_t cus) {
    int row_tiles = 0;  // 16-row tiles that stream the weights together
    if (r.grouped) {
        // the groups' sizes are on the device: their average decides
        if (r.S <= 12ll * r.E) row_tiles = 1;
        else if (r.S <= 24ll * r.E) row_tiles = 2;
    } else {
        const int64_t tiles = (r.S + 63) / 64 * ((N + 63) / 64);
        if (r.S <= 16) row_tiles = 1;
        else if (r.S <= 32) row_tiles = 2;
        else if (2 * tiles < cus && ((r.S + 63) / 64 * ((N + 15) / 16) <= cus || (K <= 1536 && r.S <= 1024)))
            row_tiles = 4;
    }
    return row_tiles > 0 ? streaming_form(row_tiles, r, N, epilogue, cus) : tiled_form(r, N, K, epilogue, cus);
}

// SwiGLU's tiles of the tiled kernel are taken by as many workgroups as run at once.
bool product_fits(const Rows &r, int N, int K, int epilogue) {
    const Form f = product_form(r, N, K, epilogue, w8a8::device_cu_count());
    if (!f.stream && epilogue == kSwiglu) return true;
    const int64_t tiles = most_tiles(r.S, r.E, f.rows, r.grouped) * ((N + f.channels - 1) / f.channels);
    return w8a8::grid_fits(tiles, f.waves * kWave);
}

hipError_t launch_gemm(const uint8_t *xq, const uint8_t *xs, const uint8_t *wq, const uint8_t *ws,
                       const Groups &g, int N, int K, int epilogue, const Output &o,
                       hipStream_t stream) {
    const Form f = product_form(Rows{g.S, g.E, g.offsets != nullptr}, N, K, epilogue, w8a8::device_cu_count());
    if (f.stream) return launch_gemm_decode(xq, xs, wq, ws, g, N, K, epilogue, o, f, stream);
    return launch_gemm_tiled(xq, xs, wq, ws, g, N, K, epilogue, o, f, stream);
}

}  // namespace mxfp4
