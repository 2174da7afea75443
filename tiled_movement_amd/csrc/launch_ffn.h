// Launchers of the feed-forward calls: the gated block, 4-bit weights, and the
// gradients' norm.  Weak, so that the host code also links without kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "launch.h"
#include "swz.h"

namespace swz {

#define SWZ_LAUNCHER __attribute__((weak)) hipError_t

// swz_gated and its gradients.
struct GatedJob {
    const void *x, *wg, *wu;  // bf16 or fp16 [n][k], [f][k]
    bool bf16;
    int act;  // enum swz_act
    int64_t n, f, k;
    void* y;
    float* pre;  // [2][n][f] or nullptr; the gradient reads it
    const void* dy;
    void *dx, *dwg, *dwu;  // each may be nullptr
    void* ws;
};
// Whether a forward call goes to the kernel that streams the weights without LDS:
// up to 16 rows, and up to 32 of small weights (20 x 520 to 600: 4.0 us, 6.5 in
// tiles; but 24 x 4096 to 8192 37 and 32).
inline bool gated_few(int64_t n, int64_t f, int64_t k) { return n <= 16 || (n <= 32 && f <= (int64_t(1) << 22) / k); }
// Rows x features of a tile of the forward product: the smallest that covers the
// rows, and up to 128 x 128 the smallest that leaves no more than 256
// workgroups, one a compute unit.  us, tiles in the order below: 64 x 4096 to 8192
// 32, 37, 53, 59, 91; 128 x 4096 to 8192 44, 39, 54, 62, 97; 77 x 2056 to 5000 29,
// 24, 40, 47, 64; 256 x 4096 to 8192 80, 73, 53, 65, 103; 512 x 4096 to 8192 139,
// 136, 96, 73, 103; 1000 x 4096 to 8192 256, 271, 183, 138, 114; 128 x 1024 to 1024
// 8.7, 10.9, 12.5, 17, 25.
enum class GatedTile { k64x32, k128x32, k64x128, k128x128, k256x128 };
inline GatedTile gated_tile(int64_t n, int64_t f) {
    auto fits = [&](int64_t rows, int64_t cols) { return ((n + rows - 1) / rows) * ((f + cols - 1) / cols) <= 256; };
    if (n <= 64 || fits(64, 32)) return GatedTile::k64x32;
    if (n <= 128 || fits(128, 32)) return GatedTile::k128x32;
    if (fits(64, 128)) return GatedTile::k64x128;
    if (fits(128, 128)) return GatedTile::k128x128;
    return GatedTile::k256x128;
}
// Rows x columns of a tile of the gradients' products.
enum class ProductTile { k64x64, k64x256, k128x128, k128x256, k256x256 };
// Whether dg and du are held as two values of x's type each, what they round to
// and the rest, and the gradients' products go over both.  Rounded once they add
// an error as large as the results' own rounding, 1.41 times that together, and
// up to 1.76 times where few values leave the roundings' sizes to chance (1 x 864
// to 272; below 1.48 from n f k = 2^23).  The gradients of 128 x 256 to 256
// in bf16 take 20.5 us with it, 17.5 without; of 2 x 1000 to 2777 31 and 23.
inline bool gated_two_terms(int64_t n, int64_t f, int64_t k) { return n * f <= (int64_t(1) << 23) / k; }
// Workspace of the gradient: byte offsets, the pitch of dg and du in elements,
// and for the products their tiles and the parts that their sums are split into.
// `rest` is from dg to its rest, and from du to its; 0: none are held.  slots: an
// fp16 call's magnitudes of dg and du, joined (256 bytes), then by workgroups.
constexpr int kGatedSlots = 2048;
struct GatedPlan {
    int64_t dg, du, rest, slots, sums, bytes;
    int64_t ldz, dx_parts, dw_parts;
    ProductTile dx_tile, dw_tile;
};
SWZ_LAUNCHER launch_gated(const GatedJob& job, hipStream_t stream);
SWZ_LAUNCHER launch_gated_grad(const GatedJob& job, const GatedPlan& plan, hipStream_t stream);

// swz_quant_w4 and swz_dequant_w4.
struct QuantW4Job {
    const void* w;
    int32_t w_type;  // enum swz_x_type
    bool bf16;       // of the scales (and the result of the way back)
    int64_t n, k;
    int group;
    void *q, *scale;
    uint8_t* zero;  // or nullptr
};
SWZ_LAUNCHER launch_quant_w4(const QuantW4Job& job, hipStream_t stream);

struct WeightsW4 {
    const uint8_t* q;     // [n][k / 2]
    const void* scale;    // x's type [n][ceil(k / group)]
    const uint8_t* zero;  // the same, or nullptr: 8
};
SWZ_LAUNCHER launch_dequant_w4(const WeightsW4& w, bool bf16, int64_t n, int64_t k, int group, void* out, hipStream_t stream);

// swz_gemm_w4 (act < 0) and swz_gated_w4 (both weights).
struct GemmW4Job {
    const void* x;  // [m][k]
    bool bf16;
    int64_t m, n, k;
    int group, act;
    WeightsW4 w[2];
    void* c;  // [m][n]
};
SWZ_LAUNCHER launch_gemm_w4(const GemmW4Job& job, hipStream_t stream);

// swz_grad_norm (out == nullptr) and swz_clip_grads: tensors by the list.
struct NormJob {
    const void* const* data;
    void* const* out;
    const int64_t* numel;
    const int32_t* type;  // enum swz_x_type
    int32_t count;
    bool clip;
    float max_norm;
    float* norm;  // [1], or [2] with the factor
    double* ws;
};
// A launch takes up to kNormTensors tensors and runs at most kNormBlocks
// workgroups, each of which leaves a partial sum; work goes by chunks of
// kNormPieces pieces of 16 bytes, from the boundary at or before a tensor's
// start.
constexpr int kNormTensors = 64;
constexpr int64_t kNormPieces = 2048, kNormBlocks = 2048;
inline int64_t norm_chunks(const void* p, int64_t numel, int32_t type) {
    const int64_t es = type == SWZ_X_F32 ? 4 : 2, per = 16 / es;
    const int64_t skew = static_cast<int64_t>(reinterpret_cast<uintptr_t>(p) % 16) / es;
    return ((skew + numel + per - 1) / per + kNormPieces - 1) / kNormPieces;
}
SWZ_LAUNCHER launch_norm(const NormJob& job, hipStream_t stream);

}  // namespace swz
