// C = A B^T of 8-bit operands with scales where A has few rows (up to 128):
// decoding, where the time is B's bytes.
//
// A workgroup owns 16 or 32 rows of B and all (up to 16 MB) rows of A; its
// waves split k, wave w taking the blocks of 128 w, w + NW, ..., so together
// they read runs of 128 NW bytes of every row, and their partial sums are
// joined through LDS in wave order.  B goes from HBM straight into matrix
// fragments, with no LDS in between: with so few rows of A a wave uses every
// byte of B once.  A's fragments come from the caches.  Products are made as
// for an fp32 result (mma_core.h, kF8Wide): the widening costs nothing next to
// the loads.
#include "launch.h"
#include "mma_core.h"

namespace swz {
namespace {

using namespace mma;

// Chunk g + 4 j of block b of a row (row: its first byte).  rem: bytes of k
// from the block on; chunks behind them are read from the block's first.
template <bool TAIL>
__device__ __forceinline__ i32x4 load_piece(const uint8_t* row, int64_t b, int j, int g, int rem) {
    int at = 16 * g + 64 * j;
    if constexpr (TAIL) {
        const int valid = rem - at;
        if (valid <= 0) at = 0;
        return keep_bytes(*reinterpret_cast<const i32x4*>(row + b * 128 + at), valid);
    }
    return *reinterpret_cast<const i32x4*>(row + b * 128 + at);
}

template <int LT, int RT, bool E8M0, class CT, int MB, int RB, int NW>
__global__ __launch_bounds__(64 * NW) void k_gemm_f8_few(Operand A, Operand B, CT* __restrict__ c, int64_t ldc, int64_t k) {
    __shared__ f32x4 red[NW][MB * RB * 64];
    const int t = threadIdx.x, lane = t % 64, g = lane / 16, l16 = lane % 16;
    const int wave = __builtin_amdgcn_readfirstlane(t / 64);
    const int64_t n0 = static_cast<int64_t>(blockIdx.x) * 16 * RB;
    const int64_t blocks = (k + 127) / 128, full = k / 128;
    const uint8_t *pa[MB], *pb[RB];
    const uint8_t *sa[MB], *sb[RB];  // scales of the rows this lane's fragments hold
    constexpr int ES = E8M0 ? 1 : 4;
#pragma unroll
    for (int x = 0; x < MB; ++x) {
        int64_t r = 16 * x + l16;
        r = r < A.rows ? r : A.rows - 1;
        pa[x] = A.data + r * A.ld;
        sa[x] = static_cast<const uint8_t*>(A.scale) + (r >> A.scale_shift) * A.scale_ld * ES;
    }
#pragma unroll
    for (int y = 0; y < RB; ++y) {
        int64_t r = n0 + 16 * y + l16;
        r = r < B.rows ? r : B.rows - 1;
        pb[y] = B.data + r * B.ld;
        sb[y] = static_cast<const uint8_t*>(B.scale) + (r >> B.scale_shift) * B.scale_ld * ES;
    }
    f32x4 acc[MB][RB];
#pragma unroll
    for (int x = 0; x < MB; ++x)
#pragma unroll
        for (int y = 0; y < RB; ++y) acc[x][y] = f32x4{0.f, 0.f, 0.f, 0.f};

    // U blocks of this wave from b on, loads before products
    auto step = [&](int64_t b, auto un, auto tail) {
        constexpr int U = decltype(un)::value;
        constexpr bool TAIL = decltype(tail)::value;
        const int rem = static_cast<int>(k - b * 128 < 128 ? k - b * 128 : 128);
        i32x4 vb[U][RB][2], va[U][MB][2];
        float fa[U][MB], fb[U][RB];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t q = b + u * NW;
#pragma unroll
            for (int y = 0; y < RB; ++y) {
#pragma unroll
                for (int j = 0; j < 2; ++j) vb[u][y][j] = load_piece<TAIL>(pb[y], q, j, g, rem);
                fb[u][y] = E8M0 ? e8m0_value(sb[y][q]) : reinterpret_cast<const float*>(sb[y])[q];
            }
#pragma unroll
            for (int x = 0; x < MB; ++x) {
#pragma unroll
                for (int j = 0; j < 2; ++j) va[u][x][j] = load_piece<TAIL>(pa[x], q, j, g, rem);
                fa[u][x] = E8M0 ? e8m0_value(sa[x][q]) : reinterpret_cast<const float*>(sa[x])[q];
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int y = 0; y < RB; ++y) {
                i32x8 r[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) r[j] = widen<RT == 1>(vb[u][y][j], E8M0 ? fb[u][y] : 1.f);
                f32x4 rs;  // fp32: scales of the four rows of B in this lane's registers
                if constexpr (!E8M0) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) rs[i] = __shfl(fb[u][y], 4 * g + i);
                }
#pragma unroll
                for (int x = 0; x < MB; ++x) {
                    f32x4 p = E8M0 ? acc[x][y] : f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        p = mfma_bf16_pair(r[j], widen<LT == 1>(va[u][x][j], E8M0 ? fa[u][x] : 1.f), p);
                    if constexpr (E8M0) {
                        acc[x][y] = p;
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[x][y][i] = __builtin_fmaf(p[i], rs[i] * fa[u][x], acc[x][y][i]);
                    }
                }
            }
        }
    };
    constexpr int U = MB * RB <= 1 ? 4 : MB <= 4 ? 2 : 1;
    int64_t b = wave;
    for (; b + (U - 1) * NW < full; b += U * NW) step(b, std::integral_constant<int, U>{}, std::false_type{});
    for (; b < full; b += NW) step(b, std::integral_constant<int, 1>{}, std::false_type{});
    if (full < blocks && full % NW == wave) step(full, std::integral_constant<int, 1>{}, std::true_type{});

    // lane (g, l16) of block (x, y): row l16 of A, columns 4g .. 4g+3 of C
#pragma unroll
    for (int x = 0; x < MB; ++x)
#pragma unroll
        for (int y = 0; y < RB; ++y) red[wave][(x * RB + y) * 64 + l16 * 4 + g] = acc[x][y];
    __syncthreads();
    const float* rf = reinterpret_cast<const float*>(red);
    for (int e = t; e < MB * RB * 256; e += 64 * NW) {
        const int blk = e / 256, row = 16 * (blk / RB) + e % 256 / 16;
        const int64_t col = n0 + 16 * (blk % RB) + e % 16;
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) s += rf[w * MB * RB * 256 + e];
        if (row < A.rows && col < B.rows) c[row * ldc + col] = static_cast<CT>(s);
    }
}

template <int LT, int RT, bool E8M0, class CT, int MB, int RB, int NW>
hipError_t launch_few(const GemmF8Job& j, hipStream_t stream) {
    const Operand A{static_cast<const uint8_t*>(j.a), j.lda, j.m, j.scale_a, (j.k + 127) / 128, j.a_square ? 7 : 0};
    const Operand B{static_cast<const uint8_t*>(j.b), j.ldb, j.n, j.scale_b, (j.k + 127) / 128, j.b_square ? 7 : 0};
    const int64_t grid = (j.n + 16 * RB - 1) / (16 * RB);
    if (grid > (int64_t(1) << 31) / (64 * NW) - 1) return hipErrorInvalidValue;
    hipLaunchKernelGGL((k_gemm_f8_few<LT, RT, E8M0, CT, MB, RB, NW>), dim3(static_cast<unsigned>(grid)), dim3(64 * NW), 0, stream,
                       A, B, static_cast<CT*>(j.c), j.n, j.k);
    return hipGetLastError();
}

template <int LT, int RT, bool E8M0, class CT>
hipError_t launch_rows_of(const GemmF8Job& j, hipStream_t stream) {
    return launch_few<LT, RT, E8M0, CT, 1, 1, 8>(j, stream);
}

template <int LT, int RT>
hipError_t launch_typed(const GemmF8Job& j, hipStream_t stream) {
    if (j.e8m0)
        return j.bf16c ? launch_rows_of<LT, RT, true, __bf16>(j, stream) : launch_rows_of<LT, RT, true, float>(j, stream);
    return j.bf16c ? launch_rows_of<LT, RT, false, __bf16>(j, stream) : launch_rows_of<LT, RT, false, float>(j, stream);
}

}  // namespace

hipError_t launch_gemm_f8_few(const GemmF8Job& j, hipStream_t stream) {
    if (j.a_e5m2) return j.b_e5m2 ? launch_typed<1, 1>(j, stream) : launch_typed<1, 0>(j, stream);
    return j.b_e5m2 ? launch_typed<0, 1>(j, stream) : launch_typed<0, 0>(j, stream);
}

}  // namespace swz
