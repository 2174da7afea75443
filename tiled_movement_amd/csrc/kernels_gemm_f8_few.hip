// C = A B^T of 8-bit operands with scales where A has at most 16 rows:
// decoding, where the time is B's bytes.
//
// A workgroup owns 16 rows of B and all rows of A; its eight waves split k, wave w taking the blocks of 128 w, w + NW, ..., so together
// they read runs of 128 NW bytes of every row, and their partial sums are
// joined through LDS in wave order.  B goes from HBM straight into matrix
// fragments, with no LDS in between: with so few rows of A a wave uses every
// byte of B once.  A's fragments come from the caches.  Products are made as
// for an fp32 result (mma_core.h, kF8Wide): the widening costs nothing next to
// the loads.  1 x 8192 x 4096: 8.8 us, 3.8 TB/s; 1 x 8192 x 8192: 15 us, 4.4
// TB/s.  Blocks of 32, 64 and 128 rows of A in this form took 12, 19 and 30 us
// at n = k = 4096, where the tiles of the general kernel take 12.
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

constexpr int kWaves = 8;

template <int LT, int RT, bool E8M0, class CT>
__global__ __launch_bounds__(64 * kWaves) void k_gemm_f8_few(Operand A, Operand B, CT* __restrict__ c, int64_t ldc,
                                                             int64_t k) {
    __shared__ f32x4 red[kWaves][64];
    const int t = threadIdx.x, lane = t % 64, g = lane / 16, l16 = lane % 16;
    const int wave = __builtin_amdgcn_readfirstlane(t / 64);
    const int64_t n0 = static_cast<int64_t>(blockIdx.x) * 16;
    const int64_t blocks = (k + 127) / 128, full = k / 128;
    // this lane's rows (the last one stands in for rows behind it; their
    // results are not stored) and where their scales begin
    const int64_t ra = l16 < A.rows ? l16 : A.rows - 1, rb = n0 + l16 < B.rows ? n0 + l16 : B.rows - 1;
    const uint8_t *pa = A.data + ra * A.ld, *pb = B.data + rb * B.ld;
    constexpr int ES = E8M0 ? 1 : 4;
    const uint8_t* sa = static_cast<const uint8_t*>(A.scale) + (ra >> A.scale_shift) * A.scale_ld * ES;
    const uint8_t* sb = static_cast<const uint8_t*>(B.scale) + (rb >> B.scale_shift) * B.scale_ld * ES;
    auto scale = [](const uint8_t* s, int64_t b) { return E8M0 ? e8m0_value(s[b]) : reinterpret_cast<const float*>(s)[b]; };
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
    // U blocks of this wave from b on, all loads before the products
    auto step = [&](int64_t b, auto un, auto tail) {
        constexpr int U = decltype(un)::value;
        constexpr bool TAIL = decltype(tail)::value;
        const int rem = static_cast<int>(k - b * 128 < 128 ? k - b * 128 : 128);
        i32x4 vb[U][2], va[U][2];
        float fa[U], fb[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t q = b + u * kWaves;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                vb[u][j] = load_piece<TAIL>(pb, q, j, g, rem);
                va[u][j] = load_piece<TAIL>(pa, q, j, g, rem);
            }
            fb[u] = scale(sb, q);
            fa[u] = scale(sa, q);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            f32x4 p = E8M0 ? acc : f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < 2; ++j)
                p = mfma_pair<kBf16>(widen<RT == 1>(vb[u][j], E8M0 ? fb[u] : 1.f), widen<LT == 1>(va[u][j], E8M0 ? fa[u] : 1.f), p);
            if constexpr (E8M0) {
                acc = p;
            } else {  // the scales of the four rows of B in this lane's registers are other lanes'
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[i] = __builtin_fmaf(p[i], __shfl(fb[u], 4 * g + i) * fa[u], acc[i]);
            }
        }
    };
    constexpr int U = 4;
    int64_t b = wave;
    for (; b + (U - 1) * kWaves < full; b += U * kWaves) step(b, std::integral_constant<int, U>{}, std::false_type{});
    for (; b < full; b += kWaves) step(b, std::integral_constant<int, 1>{}, std::false_type{});
    if (full < blocks && full % kWaves == wave) step(full, std::integral_constant<int, 1>{}, std::true_type{});

    // lane (g, l16): row l16 of A, columns 4g .. 4g+3 of C
    red[wave][l16 * 4 + g] = acc;
    __syncthreads();
    if (t >= 256) return;
    const float* rf = reinterpret_cast<const float*>(red);
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) s += rf[w * 256 + t];
    if (t / 16 < A.rows && n0 + t % 16 < B.rows) c[t / 16 * ldc + n0 + t % 16] = static_cast<CT>(s);
}

template <int LT, int RT, bool E8M0, class CT>
hipError_t launch_few(const GemmF8Job& j, hipStream_t stream) {
    const Operand A{static_cast<const uint8_t*>(j.a), j.lda, j.m, j.scale_a, (j.k + 127) / 128, j.a_square ? 7 : 0};
    const Operand B{static_cast<const uint8_t*>(j.b), j.ldb, j.n, j.scale_b, (j.k + 127) / 128, j.b_square ? 7 : 0};
    const int64_t grid = (j.n + 15) / 16;
    if (grid > (int64_t(1) << 31) / (64 * kWaves) - 1) return hipErrorInvalidValue;
    hipLaunchKernelGGL((k_gemm_f8_few<LT, RT, E8M0, CT>), dim3(static_cast<unsigned>(grid)), dim3(64 * kWaves), 0, stream, A, B,
                       static_cast<CT*>(j.c), j.n, j.k);
    return hipGetLastError();
}

template <int LT, int RT>
hipError_t launch_typed(const GemmF8Job& j, hipStream_t stream) {
    if (j.e8m0)
        return j.bf16c ? launch_few<LT, RT, true, __bf16>(j, stream) : launch_few<LT, RT, true, float>(j, stream);
    return j.bf16c ? launch_few<LT, RT, false, __bf16>(j, stream) : launch_few<LT, RT, false, float>(j, stream);
}

}  // namespace

hipError_t launch_gemm_f8_few(const GemmF8Job& j, hipStream_t stream) {
    if (j.a_e5m2) return j.b_e5m2 ? launch_typed<1, 1>(j, stream) : launch_typed<1, 0>(j, stream);
    return j.b_e5m2 ? launch_typed<0, 1>(j, stream) : launch_typed<0, 0>(j, stream);
}

}  // namespace swz
