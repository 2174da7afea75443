// Kernel launchers (defined in the .hip files, called by the C ABI layer).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <initializer_list>

#include "swz_common.h"

namespace swz {

struct ConvertJob {
    const void* src;
    void* dst;
    int64_t batch, rows, cols;
    LdsLayout layout;
    bool aligned;  // 16-byte vector path allowed (pointers and pitches)
    bool direct;   // direct HBM -> LDS fill (needs aligned and an unpadded layout)
    int order;     // tile order, enum swz_tile_order
};

struct StageJob {
    const void* src;
    void* frag;
    int64_t mn, k;
    LdsLayout layout;
    bool direct;  // direct HBM -> LDS fill
    // A second operand staged by the same launch (src2 == nullptr: none):
    // src2 [mn2][k] into frag2, same k, layout and fill.
    const void* src2 = nullptr;
    void* frag2 = nullptr;
    int64_t mn2 = 0;
};

hipError_t launch_convert(int kind, const ConvertJob& job, hipStream_t stream);
// SWZ_READ_ROWS: whole rows of any width up to 128 columns (kernels_rows.hip).
// A tile is as many whole rows as fit in rows_tile_bytes of LDS, in groups
// of 64 lane-words (a lane-word: 4 bytes of consecutive rows of one column,
// so a group is 256 / E rows): 16 KiB and 256 threads up to 64 columns,
// 32 KiB and 512 threads up to 128.  Its run in each output row may be
// shifted to start on a kRowsLine-byte line of the output; it then also
// loads up to kRowsLine / E rows past its own (at most a quarter of the
// tile's bytes), so the LDS holds rows_lds_bytes.
hipError_t launch_rows(int esz, const ConvertJob& job, hipStream_t stream);
constexpr int kRowsLine = 64;
inline int rows_tile_bytes(int64_t cols) { return cols <= 64 ? 16384 : 32768; }
inline int rows_threads(int64_t cols) { return cols <= 64 ? 256 : 512; }
inline int rows_lds_bytes(int64_t cols) { return rows_tile_bytes(cols) + rows_tile_bytes(cols) / 4; }
inline int64_t rows_halo_rows(int esz) { return kRowsLine / esz; }
inline int64_t rows_tile_rows(int64_t cols, int esz) {
    const int64_t group = 64 * (4 / esz);
    return cols <= 0 || cols > 128 ? 0 : rows_tile_bytes(cols) / (cols * esz) / group * group;
}
hipError_t launch_stage(const StageJob& job, hipStream_t stream);
hipError_t launch_gemm_frag(const void* fa, const void* fb, float* c, int64_t m, int64_t n, int64_t k,
                            hipStream_t stream);
hipError_t launch_gemm_tiles(const void* a, const void* bt, void* c, int64_t m, int64_t n, int64_t k,
                             const LdsLayout& layout, bool bf16c, hipStream_t stream);

// swz_quant_f8: x to 8-bit values with power-of-two scales, and its transpose.
struct QuantJob {
    const void* x;
    int32_t x_type;  // enum swz_x_type
    int64_t rows, cols, ldx;
    bool e5m2, square, f32_scale;
    void* q;
    void* scale;
    int64_t ldq;
    void* qt;
    void* scale_t;
    int64_t ldqt;
};
hipError_t launch_quant(const QuantJob& job, hipStream_t stream);

// Row pitches of the products' operands stay below this many bytes, so that
// the 256 rows of a tile lie within 31-bit offsets from its first (mma_core.h).
constexpr int64_t kMaxPitch = int64_t(1) << 23;

// swz_gemm_f8: C [m][n] = A B^T of 8-bit operands with scales.
struct GemmF8Job {
    const void *a, *scale_a, *b, *scale_b;
    void* c;
    int64_t m, n, k, lda, ldb;
    bool a_e5m2, b_e5m2, a_square, b_square, e8m0, bf16c;
};
hipError_t launch_gemm_f8(const GemmF8Job& job, hipStream_t stream);
hipError_t launch_gemm_f8_few(const GemmF8Job& job, hipStream_t stream);  // m <= kFewRows
constexpr int64_t kFewRows = 16;
// Tile of swz_gemm_f8 by the number of workgroups it leaves, 256 being one a compute unit.
// A stage costs a workgroup at least its barrier, loads and fragment reads,
// some 0.3 us for 64 x 64 and 0.8 us for 128 x 128, however few workgroups
// run; so small tiles where all of them run at once (m x 4096 x 4096: m = 128,
// 64 x 64 tiles 12 us, 64 x 128 16, 128 x 128 23, 256 x 256 45; m = 512: 16,
// 17, 24, 48; 256 x 8192 x 8192: 43, 35, 46, 114), and 256 x 256, which reads
// the least per product, where there is work for all units anyway (m = 2048:
// 62, 61, 47, 49).  In the small grids the workgroups of an XCD take
// neighbouring tiles, which share B's rows in its cache (512 x 8192 x 8192,
// 128 x 128 tiles: 73 -> 47 us); 256 x 256 tiles lose by it (8192 x 8192 x
// 4096: 237 -> 267 us).
enum class GemmF8Tile { k64x64, k64x128, k128x128, k256x256 };
inline GemmF8Tile gemm_f8_tile(int64_t m, int64_t n) {
    auto tiles = [&](int64_t rows, int64_t cols) { return ((m + rows - 1) / rows) * ((n + cols - 1) / cols); };
    if (tiles(64, 64) <= 256) return GemmF8Tile::k64x64;
    if (tiles(64, 128) <= 256) return GemmF8Tile::k64x128;
    if (tiles(128, 128) <= 256) return GemmF8Tile::k128x128;
    return GemmF8Tile::k256x256;
}

// swz_linear_ce, swz_linear_distill and their gradients.  teacher ==
// nullptr: cross entropy (top 1, tau 1).
constexpr int kMaxTop = 256;
struct LossJob {
    const void *h, *w;  // bf16 or fp16 [n][k], [v][k]
    bool bf16;
    int64_t n, v, k;
    const int64_t* index;  // [n][top]
    const float* teacher;  // [n][top]
    int top;
    float tau;
    float *loss, *lse, *zt;  // the gradient reads lse and zt
    const float* upstream;   // [n]
    void *dh, *dw;           // either may be nullptr
    void* ws;
};
// Workspace of the gradient: byte offsets, words of a piece of the
// vocabulary, the parts that dH's sum over a piece is split into, and the rows
// of its tiles.
struct LossPlan {
    int64_t slots, g, weight, dz, dzt, ht, wt, sums, bytes;
    int64_t piece, parts, h_rows;
};
// Rows of the losses' product tiles (columns: 256), for col_tiles tiles of
// columns: the smallest of 64, 128 and 256 that covers the rows or leaves no
// more than 256 workgroups, one a compute unit, so that all run at once.
// Forward and gradient calls, us: 250 x 32000 x 2048 in tiles of 64 rows 55 and
// 298, 128 (250 tiles) 44 and 268, 256 57 and 287; 1000 x 8192 x 1024: 35 and
// 172, 27 and 156 (256 tiles), 35 and 180; 306 x 1264 x 656: 19 and 74 (25
// tiles), 20 and 82, 27 and 98; but 509 x 32000 x 2048: 98 and 426, 77 and 370,
// 65 and 352.
inline int64_t loss_tile_rows(int64_t n, int64_t col_tiles) {
    for (const int64_t t : {int64_t(64), int64_t(128)})
        if (n <= t || (n + t - 1) / t * col_tiles <= 256) return t;
    return 256;
}
hipError_t launch_loss(const LossJob& job, hipStream_t stream);
hipError_t launch_loss_grad(const LossJob& job, const LossPlan& plan, hipStream_t stream);
hipError_t launch_map(const int32_t* in, int32_t* out, int64_t n, swz_params p, hipStream_t stream);

// Up to kMapBatch triples of one batched-map launch, passed by value.
constexpr int kMapBatch = 128;
struct MapParamPack {
    uint8_t B[kMapBatch], M[kMapBatch];
    int8_t S[kMapBatch];
};
hipError_t launch_map_batch(const int32_t* in, int32_t* out, int64_t n, const MapParamPack& pk, int count,
                            hipStream_t stream);
hipError_t launch_copy(const void* src, void* dst, int64_t bytes, hipStream_t stream);
hipError_t launch_lds_probe(const uint32_t* addrs, const uint64_t* masks, int n_patterns, int width, bool write,
                            int iters, int waves, uint64_t* cycles, hipStream_t stream);

}  // namespace swz
