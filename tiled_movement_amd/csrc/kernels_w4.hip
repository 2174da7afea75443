// Weights of 4 bits with a scale, and on request a zero point, per group of 32,
// 64 or 128 along k: w = (code - zero) scale.  To that form, back from it,
// and the product of a few rows with such weights.
#include "activation.h"
#include "launch_ffn.h"
#include "mma_core.h"

namespace swz {
namespace {

using namespace mma;

typedef uint16_t u16x8 __attribute__((ext_vector_type(8)));

template <bool BF16>
using Value = std::conditional_t<BF16, __bf16, _Float16>;

unsigned blocks_of(int64_t n, int64_t per) { return static_cast<unsigned>((n + per - 1) / per); }

// ------------------------------------------------------------- quantizer
// A lane has 8 consecutive values of a row, GROUP / 8 lanes a group.  Bound by
// its bytes but for the divisions, which have to be exact: a 16-bit value is
// often halfway between two codes.
template <class WT, class ST, int GROUP, bool ZERO>
__global__ __launch_bounds__(256) void k_quant_w4(const WT* __restrict__ w, int64_t n, int64_t k, int64_t groups,
                                                  uint32_t* __restrict__ q, ST* __restrict__ scale, uint8_t* __restrict__ zero) {
    constexpr int LANES = GROUP / 8;
    typedef WT wt8 __attribute__((ext_vector_type(8), aligned(16)));
    // the block's first group, then this thread's by 32 bits
    const int64_t first = static_cast<int64_t>(blockIdx.x) * (256 / LANES), row0 = first / groups;
    const uint64_t at = static_cast<uint64_t>(first - row0 * groups) + threadIdx.x / LANES;
    const int64_t skip = static_cast<int64_t>(at / static_cast<uint64_t>(groups));
    const int64_t row = row0 + skip, grp = static_cast<int64_t>(at) - skip * groups;
    const int64_t col = grp * GROUP + threadIdx.x % LANES * 8;
    const bool in = row < n && col < k;
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (in) {
        const wt8 x = *reinterpret_cast<const wt8*>(w + row * k + col);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = static_cast<float>(x[i]);
    }
    // the largest magnitude by its bits, where infinities and NaN come out on top
    uint32_t big = 0;
    float lo = 0.f, hi = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        big = max(big, __float_as_uint(v[i]) & 0x7fffffffu);
        if constexpr (ZERO) lo = fminf(lo, v[i]), hi = fmaxf(hi, v[i]);
    }
#pragma unroll
    for (int d = 1; d < LANES; d *= 2) {
        big = max(big, static_cast<uint32_t>(__shfl_xor(static_cast<int>(big), d)));
        if constexpr (ZERO) lo = fminf(lo, __shfl_xor(lo, d)), hi = fmaxf(hi, __shfl_xor(hi, d));
    }
    float unrounded = ZERO ? (hi - lo) * (1.f / 15.f) : __uint_as_float(big) * (1.f / 7.f);
    asm("" : "+v"(unrounded));  // rounded to fp32 first, not to fp16 at once by a mixed-precision multiply
    ST st = static_cast<ST>(unrounded);
    float s = static_cast<float>(st);
    if (big >= 0x7f800000u || !(s < __builtin_inff())) {
        s = __builtin_nanf("");
        st = static_cast<ST>(s);
    }
    const bool some = s > 0.f;
    const float z = ZERO ? (some ? fminf(fmaxf(rintf(-lo / s), 0.f), 15.f) : 0.f) : 8.f;
    uint32_t word = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float c = some ? fminf(fmaxf(rintf(v[i] / s) + z, 0.f), 15.f) : z;
        word |= static_cast<uint32_t>(c) << (4 * i);
    }
    if (!in) return;
    q[(row * k + col) / 8] = word;
    if (threadIdx.x % LANES == 0) {
        scale[row * groups + grp] = st;
        if constexpr (ZERO) zero[row * groups + grp] = static_cast<uint8_t>(z);
    }
}

// ------------------------------------------------------------ and back
template <bool BF16>
__global__ __launch_bounds__(256) void k_dequant_w4(WeightsW4 w, int64_t k8, int64_t pieces, int group8, int64_t groups,
                                                    Value<BF16>* __restrict__ out) {
    typedef Value<BF16> v8 __attribute__((ext_vector_type(8)));
    const int64_t step = static_cast<int64_t>(gridDim.x) * 256;
    for (int64_t u = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; u < pieces; u += step) {
        const int64_t row = u / k8, at = row * groups + (u - row * k8) / group8;
        const uint32_t word = reinterpret_cast<const uint32_t*>(w.q)[u];
        const float s = static_cast<float>(static_cast<const Value<BF16>*>(w.scale)[at]);
        const float z = w.zero ? static_cast<float>(w.zero[at]) : 8.f;
        v8 o;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            o[i] = static_cast<Value<BF16>>((static_cast<float>((word >> (4 * i)) & 15u) - z) * s);
        reinterpret_cast<v8*>(out)[u] = o;
    }
}

// --------------------------------------------------------------- product
// C = X W^T.  A workgroup owns 16 rows of W (of both matrices of a gated
// block) and up to 16 rows of X; its waves split k into runs of whole blocks of
// 128, and their sums are joined through LDS in their order.
//
// Codes become matrix operands without arithmetic: 16 + code has the code as
// the upper bits of its mantissa in bf16 and fp16 alike, so a shift and a
// masked or make two of them.  Products and sums of x (16 + code) are taken by
// the matrix instruction, which starts from -(16 + zero) sum x instead of zero
// (sum x from the same instruction, against ones), and the group's scale
// multiplies its sum once.  The sum's terms are up to six times as large as
// with code - zero and so is the rounding of their sum, 2^-24 each.
//
// A word has codes k .. k + 7 in order; shifts make pairs (0, 4), (1, 5), (2,
// 6), (3, 7) of it, and x's pieces are put into that order.
//
// A lane loads 16 bytes of its row, codes 32 g .. 32 g + 31 of a block (g =
// lane / 16), so the row's 64 bytes are one run.  With groups of 128 word s of
// all lanes is one product's operand; shorter groups first exchange words
// between the lanes of a row, so that a product is of one group.
template <bool BF16>
__device__ __forceinline__ i32x4 operand_of(uint32_t word) {
    constexpr uint32_t kMask = BF16 ? 0x00780078u : 0x03c003c0u, kOne = BF16 ? 0x41804180u : 0x4c004c00u;
    constexpr int kUp = BF16 ? 3 : 6;  // where the code's lowest bit belongs
    i32x4 v;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t m = 4 * j <= kUp ? word << (kUp - 4 * j) : word >> (4 * j - kUp);
        v[j] = static_cast<int>((m & kMask) | kOne);
    }
    return v;
}

__device__ __forceinline__ i32x4 paired(i32x4 x) {
    i32x4 v;
    v[0] = static_cast<int>(__builtin_amdgcn_perm(x[2], x[0], 0x05040100u));
    v[1] = static_cast<int>(__builtin_amdgcn_perm(x[2], x[0], 0x07060302u));
    v[2] = static_cast<int>(__builtin_amdgcn_perm(x[3], x[1], 0x05040100u));
    v[3] = static_cast<int>(__builtin_amdgcn_perm(x[3], x[1], 0x07060302u));
    return v;
}

template <bool BF16>
__device__ __forceinline__ f32x4 mfma16(i32x4 a, i32x4 b, f32x4 c) {
    if constexpr (BF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// The words of lanes g and g ^ 2 (g ^ 1) exchanged so that `a` has both
// lanes' first and `b` both lanes' second.
__device__ __forceinline__ void swap32(int& a, int& b) {
    const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
    a = static_cast<int>(r[0]), b = static_cast<int>(r[1]);
}
__device__ __forceinline__ void swap16(int& a, int& b) {
    const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
    a = static_cast<int>(r[0]), b = static_cast<int>(r[1]);
}

// Which 8 values of k (of 16 in a block of 128) lane g has in product s.
template <int GROUP>
__device__ __forceinline__ int unit_of(int s, int g) {
    if constexpr (GROUP == 128) return 4 * g + s;
    // words s and s + 2 exchanged between lanes g and g ^ 2: lanes 0, 1 keep the
    // first group's, lanes 2, 3 take theirs
    if constexpr (GROUP == 64) return 8 * (s / 2) + 4 * (g & 1) + 2 * (g / 2) + s % 2;
    // and words s and s + 1 between lanes g and g ^ 1
    return 4 * s + 2 * (g / 2) + (g & 1);
}

constexpr int kW4Waves = 8;

template <bool BF16, int GROUP, bool ZERO, int MATS, int ACT>
__global__ __launch_bounds__(64 * kW4Waves) void k_gemm_w4(const uint8_t* __restrict__ x, WeightsW4 w0, WeightsW4 w1, int64_t m,
                                                           int64_t n, int64_t k, Value<BF16>* __restrict__ c) {
    constexpr int PER = 128 / GROUP;  // groups of a block
    __shared__ float red[MATS][kW4Waves][256];
    const int t = threadIdx.x, lane = t % 64, g = lane / 16, l16 = lane % 16;
    const int wave = __builtin_amdgcn_readfirstlane(t / 64);
    const int64_t n0 = static_cast<int64_t>(blockIdx.x) * 16, m0 = static_cast<int64_t>(blockIdx.y) * 16;
    // this lane's rows; the last stands in for rows behind it, whose results are not stored
    const int64_t rx = m0 + l16 < m ? m0 + l16 : m - 1, rw = n0 + l16 < n ? n0 + l16 : n - 1;
    const int64_t groups = (k + GROUP - 1) / GROUP, blocks = (k + 127) / 128;
    const uint8_t* px = x + 2 * rx * k;
    const WeightsW4 w[2] = {w0, w1};
    const uint8_t* pq[MATS];
    const Value<BF16>* ps[MATS];
    const uint8_t* pz[MATS];
#pragma unroll
    for (int o = 0; o < MATS; ++o) {
        pq[o] = w[o].q + rw * (k / 2) + 16 * g;
        ps[o] = static_cast<const Value<BF16>*>(w[o].scale) + rw * groups;
        pz[o] = ZERO ? w[o].zero + rw * groups : nullptr;
    }
    f32x4 total[MATS];
#pragma unroll
    for (int o = 0; o < MATS; ++o) total[o] = f32x4{0.f, 0.f, 0.f, 0.f};
    const i32x4 ones = BF16 ? i32x4{0x3f803f80, 0x3f803f80, 0x3f803f80, 0x3f803f80}
                            : i32x4{0x3c003c00, 0x3c003c00, 0x3c003c00, 0x3c003c00};
    const i32x4 none = {0, 0, 0, 0};

    // U blocks from b on, all loads before the products.  LAST: k ends in this block.
    auto step = [&](int64_t b, auto un, auto last) {
        constexpr int U = decltype(un)::value;
        constexpr bool LAST = decltype(last)::value;
        const int units = LAST ? static_cast<int>((k - b * 128) / 8) : 16;  // of 8 values
        i32x4 vq[U][MATS], vx[U][4];
        float sc[U][MATS][PER], zp[U][MATS][PER];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t at = b + u;
#pragma unroll
            for (int o = 0; o < MATS; ++o) {
                vq[u][o] = !LAST || 4 * g < units ? *reinterpret_cast<const i32x4*>(pq[o] + at * 64) : none;
#pragma unroll
                for (int p = 0; p < PER; ++p) {
                    const int64_t grp = at * PER + p;
                    const bool here = !LAST || grp < groups;
                    sc[u][o][p] = here ? static_cast<float>(ps[o][grp]) : 0.f;
                    zp[u][o][p] = ZERO && here ? static_cast<float>(pz[o][grp]) : 8.f;
                }
            }
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const int unit = unit_of<GROUP>(s, g);
                vx[u][s] = !LAST || unit < units ? *reinterpret_cast<const i32x4*>(px + at * 256 + 16 * unit) : none;
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            f32x4 sx[PER];
#pragma unroll
            for (int p = 0; p < PER; ++p) sx[p] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                vx[u][s] = paired(vx[u][s]);
                sx[s * PER / 4] = mfma16<BF16>(vx[u][s], ones, sx[s * PER / 4]);
            }
#pragma unroll
            for (int o = 0; o < MATS; ++o) {
                int a[4] = {vq[u][o][0], vq[u][o][1], vq[u][o][2], vq[u][o][3]};
                if constexpr (GROUP < 128) {
                    swap32(a[0], a[2]);
                    swap32(a[1], a[3]);
                }
                if constexpr (GROUP < 64) {
                    swap16(a[0], a[1]);
                    swap16(a[2], a[3]);
                }
                f32x4 acc[PER];
#pragma unroll
                for (int p = 0; p < PER; ++p) acc[p] = sx[p] * -(16.f + zp[u][o][p]);
#pragma unroll
                for (int s = 0; s < 4; ++s)
                    acc[s * PER / 4] = mfma16<BF16>(vx[u][s], operand_of<BF16>(static_cast<uint32_t>(a[s])), acc[s * PER / 4]);
#pragma unroll
                for (int p = 0; p < PER; ++p)
#pragma unroll
                    for (int i = 0; i < 4; ++i) total[o][i] = __builtin_fmaf(acc[p][i], sc[u][o][p], total[o][i]);
            }
        }
    };
    constexpr int U = 2;
    const int64_t full = k / 128, end = blocks * (wave + 1) / kW4Waves;
    int64_t b = blocks * wave / kW4Waves;
    for (; b + U <= end && b + U <= full; b += U) step(b, std::integral_constant<int, U>{}, std::false_type{});
    for (; b < end && b < full; ++b) step(b, std::integral_constant<int, 1>{}, std::false_type{});
    if (b < end) step(b, std::integral_constant<int, 1>{}, std::true_type{});

    // lane (g, l16): rows 4g .. 4g+3 of X, row l16 of W
#pragma unroll
    for (int o = 0; o < MATS; ++o)
#pragma unroll
        for (int i = 0; i < 4; ++i) red[o][wave][(4 * g + i) * 16 + l16] = total[o][i];
    __syncthreads();
    if (t >= 256) return;
    float z[MATS];
#pragma unroll
    for (int o = 0; o < MATS; ++o) {
        z[o] = 0.f;
#pragma unroll
        for (int v = 0; v < kW4Waves; ++v) z[o] += red[o][v][t];
    }
    const int64_t i = m0 + t / 16, j = n0 + t % 16;
    if (i >= m || j >= n) return;
    float r = z[0];
    if constexpr (MATS == 2) r = act::both<ACT, false>(z[0]).x * z[1];
    c[i * n + j] = static_cast<Value<BF16>>(r);
}

template <bool BF16, int GROUP, bool ZERO>
hipError_t gemm_of(const GemmW4Job& j, hipStream_t stream) {
    const auto run = [&](auto kernel) {
        // rows of X by the grid's second axis, as many a launch as it takes
        constexpr int64_t kMost = 32768;
        for (int64_t r0 = 0; r0 < j.m; r0 += 16 * kMost) {
            const int64_t rows = j.m - r0 < 16 * kMost ? j.m - r0 : 16 * kMost;
            hipLaunchKernelGGL(kernel, dim3(blocks_of(j.n, 16), blocks_of(rows, 16)), dim3(64 * kW4Waves), 0, stream,
                               static_cast<const uint8_t*>(j.x) + 2 * r0 * j.k, j.w[0], j.w[1], rows, j.n, j.k,
                               static_cast<Value<BF16>*>(j.c) + r0 * j.n);
        }
        return hipGetLastError();
    };
    if (j.act < 0) return run(k_gemm_w4<BF16, GROUP, ZERO, 1, 0>);
    if (j.act == SWZ_ACT_GELU) return run(k_gemm_w4<BF16, GROUP, ZERO, 2, SWZ_ACT_GELU>);
    if (j.act == SWZ_ACT_GELU_TANH) return run(k_gemm_w4<BF16, GROUP, ZERO, 2, SWZ_ACT_GELU_TANH>);
    return run(k_gemm_w4<BF16, GROUP, ZERO, 2, SWZ_ACT_SILU>);
}

template <bool BF16, int GROUP>
hipError_t gemm_by_zero(const GemmW4Job& j, hipStream_t stream) {
    return j.w[0].zero ? gemm_of<BF16, GROUP, true>(j, stream) : gemm_of<BF16, GROUP, false>(j, stream);
}
template <bool BF16>
hipError_t gemm_by_group(const GemmW4Job& j, hipStream_t stream) {
    return j.group == 32 ? gemm_by_zero<BF16, 32>(j, stream)
                         : j.group == 64 ? gemm_by_zero<BF16, 64>(j, stream) : gemm_by_zero<BF16, 128>(j, stream);
}

template <class WT, class ST, int GROUP>
hipError_t quant_of(const QuantW4Job& j, hipStream_t stream) {
    const int64_t groups = (j.k + GROUP - 1) / GROUP, per = 256 / (GROUP / 8);
    const auto kernel = j.zero ? k_quant_w4<WT, ST, GROUP, true> : k_quant_w4<WT, ST, GROUP, false>;
    hipLaunchKernelGGL(kernel, dim3(blocks_of(j.n * groups, per)), dim3(256), 0, stream, static_cast<const WT*>(j.w), j.n, j.k,
                       groups, static_cast<uint32_t*>(j.q), static_cast<ST*>(j.scale), j.zero);
    return hipGetLastError();
}
template <class WT, class ST>
hipError_t quant_by_group(const QuantW4Job& j, hipStream_t stream) {
    return j.group == 32 ? quant_of<WT, ST, 32>(j, stream)
                         : j.group == 64 ? quant_of<WT, ST, 64>(j, stream) : quant_of<WT, ST, 128>(j, stream);
}
template <class WT>
hipError_t quant_by_scale(const QuantW4Job& j, hipStream_t stream) {
    return j.bf16 ? quant_by_group<WT, __bf16>(j, stream) : quant_by_group<WT, _Float16>(j, stream);
}

}  // namespace

hipError_t launch_quant_w4(const QuantW4Job& j, hipStream_t stream) {
    if (j.w_type == SWZ_X_F32) return quant_by_scale<float>(j, stream);
    return j.w_type == SWZ_X_BF16 ? quant_by_scale<__bf16>(j, stream) : quant_by_scale<_Float16>(j, stream);
}

hipError_t launch_dequant_w4(const WeightsW4& w, bool bf16, int64_t n, int64_t k, int group, void* out, hipStream_t stream) {
    const int64_t pieces = n * (k / 8), groups = (k + group - 1) / group;
    const dim3 grid(pieces > 65536 * 256 ? 65536u : blocks_of(pieces, 256));
    if (bf16)
        hipLaunchKernelGGL(k_dequant_w4<true>, grid, dim3(256), 0, stream, w, k / 8, pieces, group / 8, groups, static_cast<__bf16*>(out));
    else
        hipLaunchKernelGGL(k_dequant_w4<false>, grid, dim3(256), 0, stream, w, k / 8, pieces, group / 8, groups,
                           static_cast<_Float16*>(out));
    return hipGetLastError();
}

hipError_t launch_gemm_w4(const GemmW4Job& j, hipStream_t stream) {
    return j.bf16 ? gemm_by_group<true>(j, stream) : gemm_by_group<false>(j, stream);
}

}  // namespace swz
