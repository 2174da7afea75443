// A matrix to 8-bit floating point with a power-of-two scale per block of
// 128 along its rows, or per 128 x 128 square, and on request the same of its
// transpose, in one pass over the input.
//
// With a the largest finite magnitude of a block and F = 1.75 * 2^p the
// largest 8-bit value (448 = 1.75 * 2^8, 57344 = 1.75 * 2^15), the scale is
// 2^e, e the smallest integer with a <= F 2^e, and the stored values are x
// 2^-e rounded to nearest even.  Both multiplications by a power of two are
// exact, so the one rounding is that to 8 bits, the transpose's blocks hold
// exactly rounded values of their own, and the matrix instruction applies the
// scale as an exponent.  A floating-point format keeps its relative precision
// wherever in its range the block's largest value lies, so less than one of the
// 17 (e4m3) or 31 (e5m2) binades is all that the power of two gives up against
// a scale of a / F.  Infinities and NaN stay out of a and are stored as NaN
// (e5m2 keeps infinities): one bad element does not spoil its block.
//
// The kernels are bound by HBM: 2 or 4 bytes read, 1 or 2 written per element.
// 8192 x 4096 bf16 with the transpose 29 us, 4.6 TB/s (35 us when every element
// was unpacked, multiplied and tested for NaN by itself); 5001 x 6008 fp32 in
// squares with the transpose 36 us, 5.0 TB/s.
#include "launch.h"

namespace swz {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) uint8_t lds_u8;

typedef uint16_t u16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x8 __attribute__((ext_vector_type(8)));
typedef short s16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

// e + 127 for a block's largest finite magnitude (bits).  Subnormal blocks (a
// below 2^-126) need e < -127 and take -127.
template <bool E5M2>
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax) {
    if (amax == 0) return 127u;
    constexpr int p = E5M2 ? 15 : 8;
    const int ex = static_cast<int>(amax >> 23);  // biased exponent
    const int e = ex - p + ((amax & 0x7fffffu) > 0x600000u ? 1 : 0);
    return e > 0 ? static_cast<uint32_t>(e) : 0u;
}
__device__ __forceinline__ float pow2_biased(uint32_t b) {  // 2^(b - 127), b < 255
    return __uint_as_float(b ? b << 23 : 0x400000u);
}

// What the kernels do with eight elements of an input type, held as their bit
// patterns.  Largest finite magnitudes are compared as integers (for
// non-negative floating-point numbers the orders agree), two at a time for
// the 2-byte types.
template <class X, class B8>
struct Bits {
    typedef X Elem;
    typedef B8 Vec;
};
// 2-byte types go through the conversion with a scale: one instruction for two
// elements, which divides by the scale.
struct Bf16 : Bits<uint16_t, u16x8> {
    static constexpr uint32_t kInf = 0x7f80;
    static __device__ __forceinline__ uint32_t f32_bits(uint32_t m) { return m << 16; }
    template <bool E5M2>
    static __device__ __forceinline__ uint32_t pack4(const uint16_t* v, uint32_t sb) {
        const float s = pow2_biased(sb);
        const bf16x2 lo = __builtin_bit_cast(bf16x2, v[0] | static_cast<uint32_t>(v[1]) << 16);
        const bf16x2 hi = __builtin_bit_cast(bf16x2, v[2] | static_cast<uint32_t>(v[3]) << 16);
        s16x2 w = {0, 0};
        if constexpr (E5M2) {
            w = __builtin_amdgcn_cvt_scalef32_pk_bf8_bf16(w, lo, s, false);
            w = __builtin_amdgcn_cvt_scalef32_pk_bf8_bf16(w, hi, s, true);
        } else {
            w = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(w, lo, s, false);
            w = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(w, hi, s, true);
        }
        return __builtin_bit_cast(uint32_t, w);
    }
};
struct F16 : Bits<uint16_t, u16x8> {
    static constexpr uint32_t kInf = 0x7c00;
    static __device__ __forceinline__ uint32_t f32_bits(uint32_t m) {
        return __float_as_uint(static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(m))));
    }
    template <bool E5M2>
    static __device__ __forceinline__ uint32_t pack4(const uint16_t* v, uint32_t sb) {
        const float s = pow2_biased(sb);
        const f16x2 lo = __builtin_bit_cast(f16x2, v[0] | static_cast<uint32_t>(v[1]) << 16);
        const f16x2 hi = __builtin_bit_cast(f16x2, v[2] | static_cast<uint32_t>(v[3]) << 16);
        s16x2 w = {0, 0};
        if constexpr (E5M2) {
            w = __builtin_amdgcn_cvt_scalef32_pk_bf8_f16(w, lo, s, false);
            w = __builtin_amdgcn_cvt_scalef32_pk_bf8_f16(w, hi, s, true);
        } else {
            w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f16(w, lo, s, false);
            w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f16(w, hi, s, true);
        }
        return __builtin_bit_cast(uint32_t, w);
    }
};
struct F32 : Bits<uint32_t, u32x8> {
    static constexpr uint32_t kInf = 0x7f800000u;
    static __device__ __forceinline__ uint32_t f32_bits(uint32_t m) { return m; }
    template <bool E5M2>
    static __device__ __forceinline__ uint32_t pack4(const uint32_t* v, uint32_t sb) {
        const float inv = pow2_biased(254 - sb);
        float s[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            s[i] = __uint_as_float(v[i]) * inv;
            if (!E5M2) s[i] = (v[i] & 0x7f800000u) == 0x7f800000u ? __uint_as_float(0x7fc00000u) : s[i];
        }
        int w = 0;
        if constexpr (E5M2) {
            w = __builtin_amdgcn_cvt_pk_bf8_f32(s[0], s[1], w, false);
            w = __builtin_amdgcn_cvt_pk_bf8_f32(s[2], s[3], w, true);
        } else {
            w = __builtin_amdgcn_cvt_pk_fp8_f32(s[0], s[1], w, false);
            w = __builtin_amdgcn_cvt_pk_fp8_f32(s[2], s[3], w, true);
        }
        return static_cast<uint32_t>(w);
    }
};

template <class X>
__device__ __forceinline__ typename X::Vec magnitudes(typename X::Vec v) {
    typedef typename X::Elem E;
    typedef typename X::Vec V;
    v &= static_cast<E>(sizeof(E) == 2 ? 0x7fff : 0x7fffffff);
    return v < static_cast<E>(X::kInf) ? v : V(0);
}
template <class V>
__device__ __forceinline__ V larger(V a, V b) {
    return a > b ? a : b;
}
template <class V>
__device__ __forceinline__ uint32_t largest(V m) {
    uint32_t a = m[0];
#pragma unroll
    for (int e = 1; e < 8; ++e) a = max(a, static_cast<uint32_t>(m[e]));
    return a;
}
__device__ __forceinline__ uint32_t lane_max(uint32_t a, int lanes) {
#pragma unroll
    for (int d = 1; d < lanes; d *= 2) a = max(a, static_cast<uint32_t>(__shfl_xor(static_cast<int>(a), d)));
    return a;
}
template <class X, bool E5M2>
__device__ __forceinline__ u32x2 pack8(typename X::Vec v, uint32_t sb) {
    typename X::Elem e[8];
    __builtin_memcpy(e, &v, sizeof(v));
    return u32x2{X::template pack4<E5M2>(e, sb), X::template pack4<E5M2>(e + 4, sb)};
}

// Eight consecutive elements of a row of `cols` (VEC: the row's pieces are
// 16-byte aligned and cols is a multiple of 8, so a piece is inside or outside
// as a whole); zeros outside.
template <class X, bool VEC>
__device__ __forceinline__ typename X::Vec load8(const typename X::Elem* __restrict__ row, int64_t c, int64_t cols, bool in) {
    typename X::Vec v = 0;
    if constexpr (VEC) {
        if (in && c < cols) {
            u32x4 raw[sizeof(v) / 16];
#pragma unroll
            for (unsigned i = 0; i < sizeof(v) / 16; ++i) raw[i] = reinterpret_cast<const u32x4*>(row + c)[i];
            __builtin_memcpy(&v, raw, sizeof(v));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = in && c + i < cols ? row[c + i] : 0;
    }
    return v;
}

// Eight bytes to a row of q whose pitch is a multiple of 16.
__device__ __forceinline__ void store8(uint8_t* __restrict__ row, int64_t c, int64_t cols, u32x2 w) {
    if (c + 8 <= cols) {
        *reinterpret_cast<u32x2*>(row + c) = w;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c + i < cols) row[c + i] = static_cast<uint8_t>(w[i / 4] >> (8 * (i % 4)));
    }
}

__device__ __forceinline__ void put_scale(void* s, int64_t at, uint32_t byte, bool f32) {
    if (f32)
        static_cast<float*>(s)[at] = pow2_biased(byte);
    else
        static_cast<uint8_t*>(s)[at] = static_cast<uint8_t>(byte);
}

// Row blocks alone.  16 lanes hold a block of 128, 8 elements each.
template <class X, bool E5M2, bool VEC>
__global__ __launch_bounds__(256) void k_quant_rows(const typename X::Elem* __restrict__ x, int64_t ldx, int64_t rows,
                                                    int64_t cols, uint8_t* __restrict__ q, int64_t ldq,
                                                    void* __restrict__ scale, int f32, int64_t kb, int64_t block0) {
    const int64_t blk = block0 + static_cast<int64_t>(blockIdx.x) * 16 + threadIdx.x / 16;
    const int64_t r = blk / kb, b = blk - r * kb, c = b * 128 + 8 * (threadIdx.x % 16);
    const bool in = r < rows;
    const typename X::Vec v = load8<X, VEC>(x + (in ? r : 0) * ldx, c, cols, in);
    const uint32_t a = lane_max(largest(magnitudes<X>(v)), 16);
    if (!in) return;
    const uint32_t sb = scale_byte<E5M2>(X::f32_bits(a));
    if (threadIdx.x % 16 == 0) put_scale(scale, r * kb + b, sb, f32);
    if (c < cols) store8(q + r * ldq, c, cols, pack8<X, E5M2>(v, sb));
}

// A 128 x 128 tile: row blocks or the square, with or without the transpose.
// Thread (i, h) = (t % 16, t / 16) holds rows 8h .. 8h+7 of columns 8i ..
// 8i+7, so its part of a transposed row is 8 consecutive bytes.  The
// transposed tile goes through LDS in rows of 128 bytes; 8-byte slot h of row
// c sits at slot h ^ (c / 8) (Swizzle<4,0,7> on slots): the 16 lanes i that
// write the same h of rows 8 apart then use all 64 banks, and the 16-byte
// reads along a row keep their pieces whole (halves exchanged for odd c / 8).
template <class X, bool E5M2, bool VEC, bool SQUARE>
__global__ __launch_bounds__(256) void k_quant_tile(const typename X::Elem* __restrict__ x, int64_t ldx, int64_t rows, int64_t cols,
                                                    uint8_t* __restrict__ q, int64_t ldq, void* __restrict__ scale,
                                                    uint8_t* __restrict__ qt, int64_t ldqt, void* __restrict__ scale_t,
                                                    int f32, int64_t tiles_c) {
    __shared__ u32x4 tile_v[128 * 128 / 16];
    __shared__ uint32_t part[16][128];
    lds_u8* tile = (lds_u8*)(reinterpret_cast<uint8_t*>(tile_v));
    const int t = threadIdx.x, i = t % 16, h = t / 16;
    const int64_t tr = blockIdx.x / tiles_c, tc = blockIdx.x - tr * tiles_c;
    const int64_t r0 = tr * 128, c0 = tc * 128, kb = (cols + 127) / 128, kbt = (rows + 127) / 128;
    const int64_t c = c0 + 8 * i;
    typedef typename X::Vec V;
    V v[8];
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        const int64_t r = r0 + 8 * h + p;
        v[p] = load8<X, VEC>(x + (r < rows ? r : 0) * ldx, c, cols, r < rows);
    }
    uint32_t sq = 0;
    if constexpr (SQUARE) {
        V m = magnitudes<X>(v[0]);
#pragma unroll
        for (int p = 1; p < 8; ++p) m = larger(m, magnitudes<X>(v[p]));
        const uint32_t a = lane_max(largest(m), 64);
        if (t % 64 == 0) part[0][t / 64] = a;
        __syncthreads();
        sq = scale_byte<E5M2>(X::f32_bits(max(max(part[0][0], part[0][1]), max(part[0][2], part[0][3]))));
        if (t == 0) {
            if (q) put_scale(scale, tr * kb + tc, sq, f32);
            if (qt) put_scale(scale_t, tc * kbt + tr, sq, f32);
        }
    }
    if (q) {
#pragma unroll
        for (int p = 0; p < 8; ++p) {
            const int64_t r = r0 + 8 * h + p;
            uint32_t sb = sq;
            if constexpr (!SQUARE) {
                sb = scale_byte<E5M2>(X::f32_bits(lane_max(largest(magnitudes<X>(v[p])), 16)));
                if (i == 0 && r < rows) put_scale(scale, r * kb + tc, sb, f32);
            }
            if (r < rows && c < cols) store8(q + r * ldq, c, cols, pack8<X, E5M2>(v[p], sb));
        }
    }
    if (!qt) return;
    uint32_t sb[8];
    if constexpr (SQUARE) {
#pragma unroll
        for (int e = 0; e < 8; ++e) sb[e] = sq;
    } else {
        // columns' largest values: this thread's 8 rows, then the 16 row groups
        V m = magnitudes<X>(v[0]);
#pragma unroll
        for (int p = 1; p < 8; ++p) m = larger(m, magnitudes<X>(v[p]));
#pragma unroll
        for (int e = 0; e < 8; ++e) part[h][8 * i + e] = m[e];
        __syncthreads();
        if (t < 128) {
            uint32_t a = 0;
#pragma unroll
            for (int g = 0; g < 16; ++g) a = max(a, part[g][t]);
            const uint32_t s = scale_byte<E5M2>(X::f32_bits(a));
            part[0][t] = s;
            if (c0 + t < cols) put_scale(scale_t, (c0 + t) * kbt + tr, s, f32);
        }
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 8; ++e) sb[e] = part[0][8 * i + e];
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        V w;
#pragma unroll
        for (int p = 0; p < 8; ++p) w[p] = v[p][e];
        *reinterpret_cast<__attribute__((address_space(3))) u32x2*>(tile + (8 * i + e) * 128 + 8 * (h ^ i)) =
            pack8<X, E5M2>(w, sb[e]);
    }
    __syncthreads();
#pragma unroll
    for (int u = t; u < 128 * 8; u += 256) {
        const int cc = u / 8, s = u % 8, key = cc / 8;
        u32x4 w = *reinterpret_cast<__attribute__((address_space(3))) u32x4*>(tile + cc * 128 + 16 * (s ^ (key >> 1)));
        if (key & 1) w = __builtin_shufflevector(w, w, 2, 3, 0, 1);
        const int64_t r = r0 + 16 * s;
        if (c0 + cc >= cols || r >= rows) continue;
        uint8_t* dst = qt + (c0 + cc) * ldqt + r;
        if (r + 16 <= rows) {
            *reinterpret_cast<u32x4*>(dst) = w;
        } else {
            for (int b = 0; b < 16 && r + b < rows; ++b) dst[b] = static_cast<uint8_t>(w[b / 4] >> (8 * (b % 4)));
        }
    }
}

template <class X, bool E5M2, bool VEC>
hipError_t launch_typed(const QuantJob& j, hipStream_t stream) {
    const auto* x = static_cast<const typename X::Elem*>(j.x);
    auto* q = static_cast<uint8_t*>(j.q);
    auto* qt = static_cast<uint8_t*>(j.qt);
    const int64_t tr = (j.rows + 127) / 128, tc = (j.cols + 127) / 128;
    if (!j.qt && !j.square) {
        const int64_t blocks = j.rows * tc;
        constexpr int64_t kStep = int64_t(1) << 24;  // blocks of 128 per launch: whole workgroups, within the grid limit
        for (int64_t b0 = 0; b0 < blocks; b0 += kStep) {
            const int64_t n = blocks - b0 < kStep ? blocks - b0 : kStep;
            hipLaunchKernelGGL((k_quant_rows<X, E5M2, VEC>), dim3(static_cast<unsigned>((n + 15) / 16)), dim3(256), 0, stream,
                               x, j.ldx, j.rows, j.cols, q, j.ldq, j.scale, j.f32_scale ? 1 : 0, tc, b0);
        }
        return hipGetLastError();
    }
    if (tr > (int64_t(1) << 23) / tc) return hipErrorInvalidValue;
    const dim3 grid(static_cast<unsigned>(tr * tc));
    if (j.square)
        hipLaunchKernelGGL((k_quant_tile<X, E5M2, VEC, true>), grid, dim3(256), 0, stream, x, j.ldx, j.rows, j.cols, q, j.ldq,
                           j.scale, qt, j.ldqt, j.scale_t, j.f32_scale ? 1 : 0, tc);
    else
        hipLaunchKernelGGL((k_quant_tile<X, E5M2, VEC, false>), grid, dim3(256), 0, stream, x, j.ldx, j.rows, j.cols, q, j.ldq,
                           j.scale, qt, j.ldqt, j.scale_t, j.f32_scale ? 1 : 0, tc);
    return hipGetLastError();
}

template <class X>
hipError_t launch_x(const QuantJob& j, hipStream_t stream) {
    const bool vec = reinterpret_cast<uintptr_t>(j.x) % 16 == 0 && j.ldx * static_cast<int64_t>(sizeof(typename X::Elem)) % 16 == 0 &&
                     j.cols % 8 == 0;
    if (j.e5m2) return vec ? launch_typed<X, true, true>(j, stream) : launch_typed<X, true, false>(j, stream);
    return vec ? launch_typed<X, false, true>(j, stream) : launch_typed<X, false, false>(j, stream);
}

}  // namespace

hipError_t launch_quant(const QuantJob& j, hipStream_t stream) {
    if (j.rows == 0 || j.cols == 0) return hipSuccess;
    switch (j.x_type) {
        case SWZ_X_BF16: return launch_x<Bf16>(j, stream);
        case SWZ_X_F16: return launch_x<F16>(j, stream);
        default: return launch_x<F32>(j, stream);
    }
}

}  // namespace swz
