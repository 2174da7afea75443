// Weights of 4 bits with a scale, and on request a zero point, per group of 32,
// 64 or 128 along k: w = (code - zero) scale.  To that form, and back from it.
#include "launch_ffn.h"

namespace swz {
namespace {

template <bool BF16>
using Value = std::conditional_t<BF16, __bf16, _Float16>;

unsigned blocks_of(int64_t n, int64_t per) { return static_cast<unsigned>((n + per - 1) / per); }

// ------------------------------------------------------------- quantizer
// v / s rounded to a whole number, ties to even, as the correctly rounded
// quotient gives it, where |v / s| stays below 32; as the bits of kWhole + it (a
// sum that holds no digits behind the point rounds so by itself).
// 16-bit values are often halfway between two whole numbers (exactly: then one
// step of Newton's iteration ends on the halfway point itself) and never within
// 2^-12 of such a point without being on it, far more than the step's error.  fp32
// values within 2^-17 of one, where a product by 1 / s could be on the other
// side, are divided.  A division for each value would take longer than the bytes
// (8192 x 4096 bf16: 28 us, 18 so).
constexpr float kWhole = 12582912.f;  // 1.5 2^23
template <bool HALF>
struct Rounded {
    float s, r, up;
    __device__ __forceinline__ explicit Rounded(float scale) : s(scale), up(1.f) {
        if (s < 0x1p-100f) up = 0x1p100f;  // 1 / s has to be a number; both are multiplied exactly
        s *= up;
        r = __builtin_amdgcn_rcpf(s);
    }
    __device__ __forceinline__ float quotient(float v) const {
        v *= up;
        const float q = v * r;
        return HALF ? __builtin_fmaf(__builtin_fmaf(-q, s, v), r, q) : q;
    }
    // Whether a quotient may be on the wrong side.
    __device__ __forceinline__ bool unsure(float q) const { return !HALF && !(fabsf(q - (q + kWhole - kWhole)) <= 0.5f - 0x1p-17f); }
    __device__ __forceinline__ float divided(float v) const { return v * up / s; }
};
// A quotient cut to lo .. hi, whole numbers.
__device__ __forceinline__ int whole_bits(float q, float lo, float hi) {
    return __float_as_int(__builtin_amdgcn_fmed3f(q, lo, hi) + kWhole);
}

// A maximum (f) over aligned runs of LANES lanes, 16 at most: exchanges within
// four lanes, and mirrored halves, which hold the same once the fours agree.
template <int LANES, class T, class F>
__device__ __forceinline__ T over_lanes(T v, F f) {
    auto with = [&](auto ctrl) {
        v = f(v, __builtin_bit_cast(T, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), decltype(ctrl)::value, 0xf, 0xf, true)));
    };
    with(std::integral_constant<int, 0xb1>{});                         // quad_perm 1 0 3 2
    with(std::integral_constant<int, 0x4e>{});                         // quad_perm 2 3 0 1
    if constexpr (LANES > 4) with(std::integral_constant<int, 0x141>{});  // row_half_mirror
    if constexpr (LANES > 8) with(std::integral_constant<int, 0x140>{});  // row_mirror
    return v;
}

// The largest magnitude of 8 values as the bits of an fp32 number, where
// infinities and NaN come out on top.
template <class WT, class V>
__device__ __forceinline__ uint32_t largest_bits(V x) {
    if constexpr (sizeof(WT) == 2) {
        typedef uint16_t u16x8 __attribute__((ext_vector_type(8)));
        const u16x8 m = __builtin_bit_cast(u16x8, x) & uint16_t(0x7fff);
        uint16_t big = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) big = m[i] > big ? m[i] : big;
        return __float_as_uint(static_cast<float>(__builtin_bit_cast(WT, big)));
    } else {
        uint32_t big = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) big = max(big, __float_as_uint(x[i]) & 0x7fffffffu);
        return big;
    }
}

// A thread has 8 consecutive values of a row, GROUP / 8 of them a group; 2^log_tx
// threads along the row, the others in rows below.
template <class WT, class ST, int GROUP, bool ZERO>
__global__ __launch_bounds__(256) void k_quant_w4(const WT* __restrict__ w, int64_t n, int64_t k, int64_t groups, int log_tx,
                                                  uint32_t* __restrict__ q, ST* __restrict__ scale, uint8_t* __restrict__ zero) {
    constexpr int LANES = GROUP / 8;
    typedef WT wt8 __attribute__((ext_vector_type(8), aligned(16)));
    const int tx = threadIdx.x & ((1 << log_tx) - 1), ty = threadIdx.x >> log_tx, down = 256 >> log_tx;
    const int64_t piece = (static_cast<int64_t>(blockIdx.x) << log_tx) + tx, col = piece * 8;
    for (int64_t row = static_cast<int64_t>(blockIdx.y) * down + ty; row - ty < n; row += static_cast<int64_t>(gridDim.y) * down) {
        const bool in = row < n && col < k;
        wt8 x = 0;
        if (in) x = *reinterpret_cast<const wt8*>(w + row * k + col);
        uint32_t big = largest_bits<WT>(x);
        float lo = 0.f, hi = 0.f;
        if constexpr (ZERO) {
#pragma unroll
            for (int i = 0; i < 8; ++i) lo = fminf(lo, static_cast<float>(x[i])), hi = fmaxf(hi, static_cast<float>(x[i]));
        }
        big = over_lanes<LANES>(big, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
        if constexpr (ZERO) {
            lo = over_lanes<LANES>(lo, [](float a, float b) { return fminf(a, b); });
            hi = over_lanes<LANES>(hi, [](float a, float b) { return fmaxf(a, b); });
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
        const Rounded<sizeof(WT) == 2> over(some ? s : 1.f);
        const int whole = __float_as_int(kWhole);
        const int z = ZERO ? (some ? whole_bits(over.divided(-lo), 0.f, 15.f) - whole : 0) : 8;
        const float least = static_cast<float>(-z), most = static_cast<float>(15 - z);
        // codes are whole numbers plus z - whole, all taken off at once (modulo 2^32)
        uint32_t word = static_cast<uint32_t>(z - whole) * 0x11111111u;
        bool unsure = false;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float v = over.quotient(static_cast<float>(x[i]));
            unsure |= over.unsure(v);
            word += static_cast<uint32_t>(whole_bits(v, least, most)) << (4 * i);
        }
        if (unsure) {
            word = static_cast<uint32_t>(z - whole) * 0x11111111u;
#pragma unroll 1
            for (int i = 0; i < 8; ++i)
                word += static_cast<uint32_t>(whole_bits(over.divided(static_cast<float>(w[row * k + col + i])), least, most)) << (4 * i);
        }
        if (!some) word = static_cast<uint32_t>(z) * 0x11111111u;
        if (!in) continue;
        q[(row * k + col) / 8] = word;
        if (tx % LANES == 0) {
            scale[row * groups + piece / LANES] = st;
            if constexpr (ZERO) zero[row * groups + piece / LANES] = static_cast<uint8_t>(z);
        }
    }
}

// ------------------------------------------------------------ and back
template <bool BF16>
__global__ __launch_bounds__(256) void k_dequant_w4(WeightsW4 w, int64_t n, int64_t k8, int log_group8, int64_t groups, int log_tx,
                                                    Value<BF16>* __restrict__ out) {
    typedef Value<BF16> v8 __attribute__((ext_vector_type(8)));
    const int tx = threadIdx.x & ((1 << log_tx) - 1), ty = threadIdx.x >> log_tx, down = 256 >> log_tx;
    const int64_t piece = (static_cast<int64_t>(blockIdx.x) << log_tx) + tx;
    if (piece >= k8) return;
    for (int64_t row = static_cast<int64_t>(blockIdx.y) * down + ty; row < n; row += static_cast<int64_t>(gridDim.y) * down) {
        const int64_t at = row * groups + (piece >> log_group8);
        const uint32_t word = reinterpret_cast<const uint32_t*>(w.q)[row * k8 + piece];
        const float s = static_cast<float>(static_cast<const Value<BF16>*>(w.scale)[at]);
        const float z = w.zero ? static_cast<float>(w.zero[at]) : 8.f;
        v8 o;
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = static_cast<Value<BF16>>((static_cast<float>((word >> (4 * i)) & 15u) - z) * s);
        __builtin_nontemporal_store(o, reinterpret_cast<v8*>(out) + row * k8 + piece);
    }
}

// A grid of 256 threads over rows of `pieces` pieces: 2^log_tx threads along a
// row (16 at least: a group stays in a wave), the others in rows below.
struct RowGrid {
    int log_tx = 4;
    dim3 grid;
    RowGrid(int64_t n, int64_t pieces) {
        while (log_tx < 8 && (int64_t(1) << log_tx) < pieces) ++log_tx;
        const int64_t down = (n + (256 >> log_tx) - 1) / (256 >> log_tx);
        grid = dim3(blocks_of(pieces, 1 << log_tx), static_cast<unsigned>(down < 32768 ? down : 32768));
    }
};

template <class WT, class ST, int GROUP>
hipError_t quant_of(const QuantW4Job& j, hipStream_t stream) {
    const int64_t groups = (j.k + GROUP - 1) / GROUP;
    const RowGrid g(j.n, groups * (GROUP / 8));
    const auto kernel = j.zero ? k_quant_w4<WT, ST, GROUP, true> : k_quant_w4<WT, ST, GROUP, false>;
    hipLaunchKernelGGL(kernel, g.grid, dim3(256), 0, stream, static_cast<const WT*>(j.w), j.n, j.k, groups, g.log_tx,
                       static_cast<uint32_t*>(j.q), static_cast<ST*>(j.scale), j.zero);
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
    const RowGrid g(n, k / 8);
    const int log_group8 = group == 32 ? 2 : group == 64 ? 3 : 4;
    const int64_t groups = (k + group - 1) / group;
    if (bf16)
        hipLaunchKernelGGL(k_dequant_w4<true>, g.grid, dim3(256), 0, stream, w, n, k / 8, log_group8, groups, g.log_tx,
                           static_cast<__bf16*>(out));
    else
        hipLaunchKernelGGL(k_dequant_w4<false>, g.grid, dim3(256), 0, stream, w, n, k / 8, log_group8, groups, g.log_tx,
                           static_cast<_Float16*>(out));
    return hipGetLastError();
}

}  // namespace swz
