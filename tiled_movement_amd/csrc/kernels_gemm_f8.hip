// C = A B^T of 8-bit floating-point operands with a scale per block of 128
// along k, K-contiguous on both sides:
//   C[i][j] = sum_b sA[i][b] sB[j][b] sum_{k in block b} A[i][k] B[j][k].
// A stage of the core (mma_core.h) is one block of 128, so the scales change
// exactly from stage to stage.
#include "launch.h"
#include "mma_core.h"

namespace swz {
namespace {

using namespace mma;

// Workgroups go to the eight XCDs in turn; this numbering gives each XCD a run
// of consecutive tiles.
__device__ __forceinline__ uint32_t xcd_tile(uint32_t id, uint32_t total) {
    const uint32_t x = id % 8, each = total / 8, more = total % 8;
    return x * each + (x < more ? x : more) + id / 8;
}

template <class C, class CT>
__global__ __launch_bounds__(C::NT) void k_gemm_f8(Operand A, Operand B, CT* __restrict__ c, int64_t ldc, int64_t k,
                                                   TileMap map, int vec, int by_xcd) {
    __shared__ i32x4 lds_v[C::kLds / 16];
    lds_u8* lds = (lds_u8*)(reinterpret_cast<uint8_t*>(lds_v));
    int64_t tm, tn;
    if (by_xcd) {
        const uint32_t tile = xcd_tile(blockIdx.x, gridDim.x);
        tm = tile % map.f, tn = tile / map.f;
    } else if (!map.at(blockIdx.x, &tm, &tn)) {
        return;
    }
    const int64_t i0 = tm * C::TL, j0 = tn * C::TR;
    f32x4 acc[C::BL][C::BR];
    tile_product<C>(acc, A, B, i0, j0, k, lds);
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    lds_f32* slice = (lds_f32*)(lds + wave * C::kSlice);
    const int64_t wi = i0 + wave / C::WR * C::BL * 16, wj = j0 + wave % C::WR * C::BR * 16;
    store_tile<C>(acc, slice, c, ldc, wi, wj, A.rows, B.rows, vec, lane, [](float v) { return v; });
}

// A launch's threads stay below 2^32 along x, so more than 2^22 tiles (the
// entry point's bound is in tiles of 256 x 256) go by ranges of rows.
template <class C, class CT>
hipError_t launch_tiles(const GemmF8Job& j, bool by_xcd, hipStream_t stream) {
    constexpr int ES = C::SC == kE8M0 ? 1 : 4;
    const int64_t tn = (j.n + C::TR - 1) / C::TR, kb = (j.k + 127) / 128, most = (int64_t(1) << 22) / tn * C::TL;
    const int vec = j.n * static_cast<int64_t>(sizeof(CT)) % 16 == 0 && reinterpret_cast<uintptr_t>(j.c) % 16 == 0;
    const Operand B{static_cast<const uint8_t*>(j.b), j.ldb, j.n, j.scale_b, kb, j.b_square ? 7 : 0};
    static_assert(C::TL % 128 == 0 || C::TL == 64, "ranges of rows are whole squares (64 rows: a single range)");
    for (int64_t i0 = 0; i0 < j.m; i0 += most) {
        const int64_t rows = j.m - i0 < most ? j.m - i0 : most, tm = (rows + C::TL - 1) / C::TL;
        const int64_t scale0 = (j.a_square ? i0 / 128 : i0) * kb * ES;
        const Operand A{static_cast<const uint8_t*>(j.a) + i0 * j.lda, j.lda, rows,
                        static_cast<const uint8_t*>(j.scale_a) + scale0, kb, j.a_square ? 7 : 0};
        const TileMap map = TileMap::make(tm, tn);
        hipLaunchKernelGGL((k_gemm_f8<C, CT>), dim3(by_xcd ? static_cast<unsigned>(tm * tn) : map.grid), dim3(C::NT), 0, stream, A,
                           B, static_cast<CT*>(j.c) + i0 * j.n, j.n, j.k, map, vec, by_xcd ? 1 : 0);
    }
    return hipGetLastError();
}

// fp32 scales of both operands' rows on widened operands need more registers
// than a 64 x 128 wave tile leaves (145 spilled): half the rows.
template <int ELEM, int LT, int RT, int SC, class CT>
hipError_t launch_sized(const GemmF8Job& j, hipStream_t stream) {
    switch (gemm_f8_tile(j.m, j.n)) {
        case GemmF8Tile::k64x64: return launch_tiles<Config<ELEM, LT, RT, SC, 2, 2, 2, 2>, CT>(j, true, stream);
        case GemmF8Tile::k64x128: return launch_tiles<Config<ELEM, LT, RT, SC, 2, 4, 2, 2>, CT>(j, true, stream);
        case GemmF8Tile::k128x128: return launch_tiles<Config<ELEM, LT, RT, SC, 2, 4, 4, 2>, CT>(j, true, stream);
        default: return launch_tiles<Config<ELEM, LT, RT, SC, 4, 2, ELEM == kF8Wide && SC == kF32Rows ? 2 : 4, 8>, CT>(j, false, stream);
    }
}

// A bf16 result takes the one-byte instruction, whose dropped bits are a
// hundredth of the rounding to bf16; an fp32 result is asked for its bits and
// takes the bf16 instruction on widened operands.
template <int LT, int RT, int SC>
hipError_t launch_typed(const GemmF8Job& j, hipStream_t stream) {
    return j.bf16c ? launch_sized<kF8, LT, RT, SC, __bf16>(j, stream) : launch_sized<kF8Wide, LT, RT, SC, float>(j, stream);
}

template <int SC>
hipError_t launch_scaled(const GemmF8Job& j, hipStream_t stream) {
    if (j.a_e5m2) return j.b_e5m2 ? launch_typed<1, 1, SC>(j, stream) : launch_typed<1, 0, SC>(j, stream);
    return j.b_e5m2 ? launch_typed<0, 1, SC>(j, stream) : launch_typed<0, 0, SC>(j, stream);
}

}  // namespace

hipError_t launch_gemm_f8(const GemmF8Job& j, hipStream_t stream) {
    if (j.m == 0 || j.n == 0) return hipSuccess;
    if (j.m <= kFewRows) return launch_gemm_f8_few(j, stream);
    if (j.e8m0) return launch_scaled<kE8M0>(j, stream);
    return j.b_square ? launch_scaled<kF32Square>(j, stream) : launch_scaled<kF32Rows>(j, stream);
}

}  // namespace swz
