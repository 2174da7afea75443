// Weights of 4 bits with a scale, and on request a zero point, per group of 32,
// 64 or 128 along k: w = (code - zero) scale.  To that form, and back from it.
#include "launch_ffn.h"

namespace swz {
namespace {

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

}  // namespace swz
