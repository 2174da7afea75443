// Losses of an output layer whose logits z = H W^T are never kept: softmax
// cross entropy against one word a row, and distillation from a teacher's top
// logits, with their gradients.
//
//   lse_i  = log sum_v exp(z_iv / tau)
//   loss_i = tau^2 sum_j p_ij (log p_ij - (z_{i,t_ij} / tau - lse_i))
//   dz_iv  = g_i tau (exp(z_iv / tau - lse_i) - sum_{j: t_ij = v} p_ij)
//   dH = dz W,  dW = dz^T H
//
// with p_i the softmax of the row's teacher logits over tau; cross entropy is
// one entry with p = 1 and tau = 1.
//
// Forward: the logits of a 256 x 256 tile stay in accumulators, and a tile
// leaves only each row's maximum and sum of exponentials (8 bytes per row and
// 256 words); a second kernel joins them.  Bound by the bf16 / fp16 matrix rate.
// A logit is one number wherever it enters: a tile writes cross entropy's at
// the target, and distillation's at listed words are made by the same
// instructions in the same order; and lse is the largest logit over tau plus a
// logarithm of at least one, with the same product by 1/tau (over_tau) wherever
// a logit meets lse.  So lse is never below a listed logit, cross
// entropy's loss and the target's p - 1 have their signs, and a row that is
// certain of its target has no loss and no gradient (with a sum of its own for
// the target's logit: losses of +-2e-5 at logits of 90).
//
// Backward, a piece of the vocabulary at a time: the piece's logits again, dz
// from them and the saved lse, then both gradient products.  Their operands
// have to be contiguous along the summed axis, so dz, W's piece and H are
// transposed through LDS on the way (5% of the time at 4096 x 65536 x 4096).
//
// Rounding: dz is held in fp16 (2^-11), not bf16 (2^-8), because the result
// is rounded to its own type once more and a bf16 dz would add an error of
// the same size.  A row's g_i tau is split into f_i 2^s_i max_j |g_j tau| with
// 1/2 < |f_i| <= 1: f_i enters dz (1 where all rows weigh the same, so a mean's
// 1/n leaves no rounding), 2^s_i is exact and enters behind it, in dH at the
// end and in dW with H's row.  So every row of dz has all of fp16's range,
// however little the row weighs, and a factor of 2^14 puts probabilities down
// to 2^-27 in its normal part.  H (its rows times 2^s_i) and bf16 W are widened
// to fp16 by a power of two that puts their largest value into [2^14, 2^15):
// exact for all values down to 2^-28 of the largest, and off by at most 2^-39
// of it below that.
#include "launch.h"
#include "mma_core.h"

namespace swz {
namespace {

using namespace mma;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kDzScale = 16384.f;
constexpr int kSlots = 3;  // maxima, as bits: 0 |H|, 1 |W|, 2 |g tau|

typedef uint16_t u16x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ float half_bits_to_f32(uint16_t b, bool bf16) {
    return bf16 ? __uint_as_float(static_cast<uint32_t>(b) << 16)
                : static_cast<float>(__builtin_bit_cast(_Float16, b));
}

// z / tau as one product by inv = 1 / tau, rounded by itself (a fused
// multiply-add with what it meets would round elsewhere): rounding keeps the
// order, so no logit comes out above its row's largest, however far over tau.
__device__ __forceinline__ float over_tau(float z, float inv) {
#pragma clang fp contract(off)
    return z * inv;
}
// exp(z / tau - lse): at most one.
__device__ __forceinline__ float probability(float z, float inv, float lse) {
#pragma clang fp contract(off)
    return __builtin_amdgcn_exp2f((over_tau(z, inv) - lse) * kLog2e);
}

// ------------------------------------------------------------------ forward
// Rows [i0, i0 + TL) against words [j0, j0 + TR): part[tile][row] = (largest
// logit m, sum of 2^((z - m) c2)), c2 = log2(e) / tau.  Cross entropy (index
// given): zt of the rows whose target is in the tile.
template <class C>
__global__ __launch_bounds__(C::NT) void k_logit_stats(Operand H, Operand W, int64_t kbytes, float c2,
                                                       float2* __restrict__ part, const int64_t* __restrict__ index,
                                                       float* __restrict__ zt, TileMap map) {
    __shared__ i32x4 lds_v[C::kLds / 16];
    lds_u8* lds = (lds_u8*)(reinterpret_cast<uint8_t*>(lds_v));
    int64_t tm, tn;
    if (!map.at(blockIdx.x, &tm, &tn)) return;
    const int64_t i0 = tm * C::TL, j0 = tn * C::TR;
    f32x4 acc[C::BL][C::BR];
    tile_product<C>(acc, H, W, i0, j0, kbytes, lds);
    const int t = threadIdx.x, lane = t % 64, g = lane / 16, l16 = lane % 16;
    const int wave = __builtin_amdgcn_readfirstlane(t / 64), wl = wave / C::WR, wr = wave % C::WR;
    lds_f32* red = (lds_f32*)lds;  // [2][WR][TL]
    const bool whole = j0 + C::TR <= W.rows;
    const int64_t jw = j0 + wr * C::BR * 16 + 4 * g;
#pragma unroll
    for (int x = 0; x < C::BL; ++x) {
        if (index) {
            const int64_t row = i0 + (wl * C::BL + x) * 16 + l16, word = row < H.rows ? index[row] : -1, at = word - jw;
            const bool here = word < W.rows && at >= 0 && at < 16 * C::BR && at % 16 < 4;
            if (__any(here)) {
#pragma unroll
                for (int y = 0; y < C::BR; ++y)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (here && at == 16 * y + i) zt[row] = acc[x][y][i];
            }
        }
        float m = -__builtin_inff();
#pragma unroll
        for (int y = 0; y < C::BR; ++y)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (!whole && jw + 16 * y + i >= W.rows) acc[x][y][i] = -__builtin_inff();
                m = fmaxf(m, acc[x][y][i]);
            }
        m = fmaxf(m, __shfl_xor(m, 16));
        m = fmaxf(m, __shfl_xor(m, 32));
        const float mm = m == -__builtin_inff() ? 0.f : m;  // no words here: a sum of zeros
        float s = 0.f;
#pragma unroll
        for (int y = 0; y < C::BR; ++y)
#pragma unroll
            for (int i = 0; i < 4; ++i) s += __builtin_amdgcn_exp2f((acc[x][y][i] - mm) * c2);
        s += __shfl_xor(s, 16);
        s += __shfl_xor(s, 32);
        if (g == 0) {
            red[wr * C::TL + (wl * C::BL + x) * 16 + l16] = m;
            red[(C::WR + wr) * C::TL + (wl * C::BL + x) * 16 + l16] = s;
        }
    }
    __syncthreads();
    for (int r = t; r < C::TL; r += C::NT) {
        if (i0 + r >= H.rows) continue;
        float m = red[r];
#pragma unroll
        for (int w = 1; w < C::WR; ++w) m = fmaxf(m, red[w * C::TL + r]);
        const float mm = m == -__builtin_inff() ? 0.f : m;
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < C::WR; ++w)
            s += red[(C::WR + w) * C::TL + r] * __builtin_amdgcn_exp2f((red[w * C::TL + r] - mm) * c2);
        part[tn * H.rows + i0 + r] = make_float2(m, s);
    }
}

// lse from the pieces: 32 rows a workgroup, eight threads a row; and cross
// entropy's loss (index given), with zt of the rows that do not count.
__global__ __launch_bounds__(256) void k_join_stats(const float2* __restrict__ part, int64_t tiles, int64_t n, float c2,
                                                    float inv, float* __restrict__ lse, const int64_t* __restrict__ index,
                                                    int64_t v, float* __restrict__ zt, float* __restrict__ loss) {
    __shared__ float2 red[8][32];
    const int r = threadIdx.x % 32, sub = threadIdx.x / 32;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * 32 + r;
    float m = -__builtin_inff(), s = 0.f;
    if (row < n) {
#pragma unroll 4
        for (int64_t i = sub; i < tiles; i += 8) {
            const float2 p = part[i * n + row];
            const float big = fmaxf(m, p.x);
            const float b = big == -__builtin_inff() ? 0.f : big;
            s = s * __builtin_amdgcn_exp2f((m - b) * c2) + p.y * __builtin_amdgcn_exp2f((p.x - b) * c2);
            m = big;
        }
    }
    red[sub][r] = make_float2(m, s);
    __syncthreads();
    if (sub == 0 && row < n) {
        for (int i = 1; i < 8; ++i) m = fmaxf(m, red[i][r].x);
        const float b = m == -__builtin_inff() ? 0.f : m;
        float total = 0.f;
        for (int i = 0; i < 8; ++i) total += red[i][r].y * __builtin_amdgcn_exp2f((red[i][r].x - b) * c2);
        const float l = over_tau(m, inv) + logf(total);
        lse[row] = l;
        if (index) {
            const bool counts = index[row] >= 0 && index[row] < v;
            if (!counts) zt[row] = 0.f;
            loss[row] = counts ? l - zt[row] : 0.f;
        }
    }
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int d = 1; d < 64; d *= 2) v += __shfl_xor(v, d);
    return v;
}
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
    for (int d = 1; d < 64; d *= 2) v = fmaxf(v, __shfl_xor(v, d));
    return v;
}

// Whether entry j of a row counts: its word exists and its teacher logit is
// not the lowest.
__device__ __forceinline__ bool entry_counts(int64_t word, float teacher, int64_t v) {
    return word >= 0 && word < v && teacher != -__builtin_inff();
}

// Distillation, one workgroup a row: the logits at its listed words, then its
// loss.  A wave makes 16 logits with the instructions and the order of k of
// tile_product, so they are its numbers: the words' rows feed the
// instruction's rows, H's row all of its columns.  k is a multiple of 8, so
// 16-byte chunks are inside or outside as a whole.
template <bool BF16>
__global__ __launch_bounds__(256) void k_listed_loss(const uint16_t* __restrict__ h, const uint16_t* __restrict__ w,
                                                     const int64_t* __restrict__ index,
                                                     const float* __restrict__ teacher, int64_t v, int64_t k, int top,
                                                     float tau, float inv, const float* __restrict__ lse,
                                                     float* __restrict__ zt, float* __restrict__ loss) {
    __shared__ float z[kMaxTop];
    const int64_t row = blockIdx.x;
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64, waves = blockDim.x / 64, g = lane / 16, l16 = lane % 16;
    const uint8_t* hr = reinterpret_cast<const uint8_t*>(h + row * k);
    for (int j0 = 16 * wave; j0 < top; j0 += 16 * waves) {
        // absent entries take word 0, and their result is dropped
        const int mine = j0 + l16;
        const int64_t word = mine < top ? index[row * top + mine] : -1;
        const bool counts = mine < top && entry_counts(word, teacher[row * top + mine], v);
        const uint8_t* wr = reinterpret_cast<const uint8_t*>(w + (counts ? word : 0) * k);
        f32x4 acc = {0.f, 0.f, 0.f, 0.f};
        // U stages from byte `at` of the rows, all loads before the products
        const int64_t kbytes = 2 * k, full = kbytes / 128 * 128;
        auto stages = [&](int64_t at, auto un, bool lo_in, bool hi_in) {
            constexpr int U = decltype(un)::value;
            const i32x4 none = {0, 0, 0, 0};
            i32x4 r[U][2], c[U][2];
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int64_t b = at + 128 * u + 64 * j + 16 * g;
                    const bool in = j ? hi_in : lo_in;
                    r[u][j] = in ? *reinterpret_cast<const i32x4*>(wr + b) : none;
                    c[u][j] = in ? *reinterpret_cast<const i32x4*>(hr + b) : none;
                }
#pragma unroll
            for (int u = 0; u < U; ++u)
                acc = mfma_pair<BF16 ? kBf16 : kF16>(__builtin_shufflevector(r[u][0], r[u][1], 0, 1, 2, 3, 4, 5, 6, 7),
                                                     __builtin_shufflevector(c[u][0], c[u][1], 0, 1, 2, 3, 4, 5, 6, 7), acc);
        };
        constexpr int U = 8;
        int64_t at = 0;
        for (; at + 128 * U <= full; at += 128 * U) stages(at, std::integral_constant<int, U>{}, true, true);
        for (; at < full; at += 128) stages(at, std::integral_constant<int, 1>{}, true, true);
        if (full < kbytes) stages(full, std::integral_constant<int, 1>{}, full + 16 * g < kbytes, full + 16 * g + 64 < kbytes);
        // lane 16 g holds words 4 g .. 4 g + 3 (all columns are the same)
        const unsigned long long here = __ballot(counts);
        if (l16 == 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int j = j0 + 4 * g + i;
                if (j >= top) continue;
                z[j] = (here >> (4 * g + i)) & 1 ? acc[i] : 0.f;
                zt[row * top + j] = z[j];
            }
        }
    }
    __syncthreads();
    if (wave != 0) return;
    const float l = lse[row];
    float out = 0.f, m = -__builtin_inff();
    bool any = false;
    for (int j = lane; j < top; j += 64) {
        const float t = teacher[row * top + j];
        if (entry_counts(index[row * top + j], t, v)) m = fmaxf(m, t), any = true;
    }
    // (t - m) / tau, not t / tau - m / tau: the lowest float over a tau below
    // one would overflow
    if (__any(any)) {
        m = wave_max(m);
        float s = 0.f;
        for (int j = lane; j < top; j += 64) {
            const float t = teacher[row * top + j];
            if (entry_counts(index[row * top + j], t, v)) s += expf((t - m) / tau);
        }
        const float ls = logf(wave_sum(s));
        for (int j = lane; j < top; j += 64) {
            const float t = teacher[row * top + j];
            if (!entry_counts(index[row * top + j], t, v)) continue;
            const float lp = (t - m) / tau - ls, p = expf(lp);
            out += p > 0.f || p != p ? p * (lp - (over_tau(z[j], inv) - l)) : 0.f;
        }
        out = tau * (tau * wave_sum(out));  // tau^2 alone may leave fp32's range
    }
    if (lane == 0) loss[row] = out;
}

// ----------------------------------------------------------------- backward
__global__ void k_clear_slots(uint32_t* slots) {
    if (threadIdx.x < kSlots) slots[threadIdx.x] = 0;
}

// g_i tau as f 2^s times the largest of them (its bits), 1/2 < |f| <= 1 and
// s <= 0.  0, and what is not finite, is its own f.
struct RowScale {
    float f;
    int s;
    __device__ __forceinline__ RowScale(float g, uint32_t gmax) : f(g), s(0) {
        if (g == 0.f || magnitude_bits(g) >= 0x7f800000u) return;
        int eg, em;
        float mg = frexpf(g, &eg);
        const float mm = frexpf(__uint_as_float(gmax), &em);
        s = eg - em;
        if (fabsf(mg) > mm) mg *= 0.5f, ++s;
        f = mg / mm;
    }
};

// Largest finite magnitudes, as fp32 bits (the order of atomic maxima does not
// matter): of H's rows times their 2^s_i, and of a bf16 W.  At most one atomic
// a workgroup, and none where the slot already holds as much: with one a wave
// the atomics took four fifths of the time (200 MB: 190 us).
// Grid row 0 takes H, row 1 W; a side that no gradient needs has no pieces.
// H's rows of factor g = 0 stay out (row_pieces: 16-byte pieces a row): they
// may hold anything, and their largest value would push the others' digits
// out of the widened range.
template <bool BF16>
__global__ __launch_bounds__(256) void k_absmax(const uint16_t* __restrict__ h, int64_t h_pieces, uint32_t row_pieces,
                                                const float* __restrict__ g, const uint16_t* __restrict__ w,
                                                int64_t w_pieces, uint32_t* slots) {
    __shared__ uint32_t part[4];
    const uint16_t* x = blockIdx.y ? w : h;
    const int64_t pieces = blockIdx.y ? w_pieces : h_pieces;
    uint32_t* slot = slots + blockIdx.y;
    if (static_cast<int64_t>(blockIdx.x) * 256 >= pieces) return;
    const uint32_t step = gridDim.x * 256, first = blockIdx.x * 256 + threadIdx.x;
    auto magnitudes = [&](int64_t i) {
        const u16x8 a = reinterpret_cast<const u16x8*>(x)[i] & uint16_t(0x7fff);
        return a < uint16_t(BF16 ? 0x7f80 : 0x7c00) ? a : u16x8(0);
    };
    auto largest = [](u16x8 m) {
        uint32_t best = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) best = max(best, static_cast<uint32_t>(m[e]));
        return half_bits_to_f32(static_cast<uint16_t>(best), BF16);
    };
    uint32_t best = 0;
    if (blockIdx.y) {
        u16x8 m = 0;
#pragma unroll 4
        for (int64_t i = first; i < pieces; i += step) {
            const u16x8 a = magnitudes(i);
            m = a > m ? a : m;
        }
        best = __float_as_uint(largest(m));
    } else {
        // the row of a piece by steps: a division a piece would cost more than its load
        const uint32_t rows = step / row_pieces, rest = step % row_pieces, gmax = slots[2];
        uint32_t row = first / row_pieces, at = first % row_pieces;
#pragma unroll 4
        for (int64_t i = first; i < pieces; i += step) {
            const float gr = g[row];
            if (gr != 0.f) best = max(best, __float_as_uint(ldexpf(largest(magnitudes(i)), RowScale(gr, gmax).s)));
            row += rows;
            at += rest;
            if (at >= row_pieces) at -= row_pieces, ++row;
        }
    }
#pragma unroll
    for (int d = 1; d < 64; d *= 2) best = max(best, static_cast<uint32_t>(__shfl_xor(static_cast<int>(best), d)));
    if (threadIdx.x % 64 == 0) part[threadIdx.x / 64] = best;
    __syncthreads();
    if (threadIdx.x == 0) raise_slot(slot, max(max(part[0], part[1]), max(part[2], part[3])));
}

// The power of two that takes a largest magnitude (bits) just below 2^15, as
// its exponent; 0 where nothing was measured.
__device__ __forceinline__ int widen_exponent(uint32_t bits) {
    if (bits == 0) return 0;
    const int e = 14 - (static_cast<int>(bits >> 23) - 127);  // subnormals: bits >> 23 == 0
    return e < -113 ? -113 : e > 126 ? 126 : e;
}

// Cross entropy, a thread a row: the target's weight and g, 0 for rows that do
// not count.
__global__ __launch_bounds__(256) void k_ce_prep(const int64_t* __restrict__ index, const float* __restrict__ upstream,
                                                 int64_t n, int64_t v, float* __restrict__ weight, float* __restrict__ g,
                                                 uint32_t* slot) {
    const int64_t row = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    uint32_t b = 0;
    if (row < n) {
        const bool counts = index[row] >= 0 && index[row] < v;
        const float gt = counts ? upstream[row] : 0.f;
        weight[row] = counts ? 1.f : 0.f;
        g[row] = gt;
        b = magnitude_bits(gt);
        b = b < 0x7f800000u ? b : 0u;
    }
#pragma unroll
    for (int d = 1; d < 64; d *= 2) b = max(b, static_cast<uint32_t>(__shfl_xor(static_cast<int>(b), d)));
    if (threadIdx.x % 64 == 0) raise_slot(slot, b);
}

// Distillation, a wave a row: the entries' weights with equal words joined
// (each holds the sum, so writing it twice writes the same), and g tau.
__global__ __launch_bounds__(64) void k_distill_prep(const int64_t* __restrict__ index, const float* __restrict__ teacher,
                                                     const float* __restrict__ upstream, int64_t v, int top, float tau,
                                                     float* __restrict__ weight, float* __restrict__ g, uint32_t* slot) {
    __shared__ float p[kMaxTop];
    __shared__ int64_t words[kMaxTop];
    const int64_t row = blockIdx.x;
    const int lane = threadIdx.x;
    float m = -__builtin_inff();
    bool any = false;
    for (int j = lane; j < top; j += 64) {
        const float t = teacher[row * top + j];
        if (entry_counts(index[row * top + j], t, v)) m = fmaxf(m, t), any = true;
    }
    any = __any(any);
    m = wave_max(m);
    float s = 0.f;
    for (int j = lane; j < top; j += 64) {
        const float t = teacher[row * top + j];
        const bool here = entry_counts(index[row * top + j], t, v);
        const float e = here ? expf((t - m) / tau) : 0.f;
        words[j] = here ? index[row * top + j] : -1;
        p[j] = e;
        s += e;
    }
    s = wave_sum(s);
    __syncthreads();
    for (int j = lane; j < top; j += 64) {
        float sum = 0.f;
        for (int i = 0; i < top; ++i) sum += words[i] == words[j] ? p[i] : 0.f;
        weight[row * top + j] = any ? sum / s : 0.f;
    }
    if (lane == 0) {
        const float gt = any ? upstream[row] * tau : 0.f;
        g[row] = gt;
        raise_slot(slot, magnitude_bits(gt));
    }
}

// What a gradient's sum is multiplied by at the end: the largest upstream,
// 2^-14, the power of two of its widened operand, and of dH's row (s).
// Exponents are added before they are applied, so nothing on the way leaves
// the range that the result is in.
struct Unscale {
    float m;
    int e;
    __device__ __forceinline__ Unscale(uint32_t gmax, uint32_t operand_max, int s = 0) {
        int ge;
        m = frexpf(__uint_as_float(gmax), &ge);
        e = ge - 14 - widen_exponent(operand_max) + s;
    }
    __device__ __forceinline__ float operator()(float v) const { return ldexpf(v * m, e); }
};

// A 128 x 128 tile of 2-byte values transposed through LDS: in [rows][ldin]
// to fp16 [cols][ldout], WIDEN: times the power of two of `slot` and, where g is
// given, 2^s of the row; else as they are.  Thread (i, h) takes the 8 x 8 block of columns 8i and rows
// 8h, so each of its columns is one 16-byte piece of an output row; piece h
// of output row c sits at slot h ^ (c / 8) of the row's 16 (Swizzle<4,0,7> on
// slots), which spreads the 16 rows that 16 lanes write over all 64 banks.
// Rows whose factor g is 0 become zeros: they may hold anything, and their
// zeros in dz would not cancel a NaN.  ldin, ldout: elements, multiples of 8; pieces behind `rows` are written into
// the output's padding (at most 7 elements, inside ldout).
template <bool BF16, bool WIDEN>
__global__ __launch_bounds__(256) void k_transpose16(const uint16_t* __restrict__ in, int64_t ldin, int64_t rows,
                                                     int64_t cols, uint16_t* __restrict__ out, int64_t ldout,
                                                     int64_t tiles_c, const uint32_t* __restrict__ slot,
                                                     const float* __restrict__ g, const uint32_t* __restrict__ gmax) {
    __shared__ u16x8 tile[128 * 16];
    const int t = threadIdx.x, i = t % 16, h = t / 16;
    const int64_t tr = blockIdx.x / tiles_c, tc = blockIdx.x - tr * tiles_c;
    const int64_t r0 = tr * 128, c0 = tc * 128;
    u16x8 v[8];
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        const int64_t r = r0 + 8 * h + p, c = c0 + 8 * i;
        v[p] = r < rows && c < cols && (!g || g[r] != 0.f) ? *reinterpret_cast<const u16x8*>(in + r * ldin + c)
                                                           : u16x8{0, 0, 0, 0, 0, 0, 0, 0};
    }
    if constexpr (WIDEN) {
        const int widen = widen_exponent(*slot);
#pragma unroll
        for (int p = 0; p < 8; ++p) {
            const int64_t r = r0 + 8 * h + p;
            const int x = widen + (g && r < rows ? RowScale(g[r], *gmax).s : 0);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[p][e] = __builtin_bit_cast(uint16_t, static_cast<_Float16>(ldexpf(half_bits_to_f32(v[p][e], BF16), x)));
        }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        u16x8 o;
#pragma unroll
        for (int p = 0; p < 8; ++p) o[p] = v[p][e];
        tile[(8 * i + e) * 16 + (h ^ i)] = o;
    }
    __syncthreads();
#pragma unroll
    for (int u = t; u < 128 * 16; u += 256) {
        const int c = u / 16, s = u % 16;
        const int64_t r = r0 + 8 * s;
        if (c0 + c < cols && r < rows)
            *reinterpret_cast<u16x8*>(out + (c0 + c) * ldout + r) = tile[c * 16 + (s ^ (c / 8))];
    }
}

// dz of words [j0, ...) of a piece (W starts at the piece): fp16 [rows][ldz].
template <class C>
__global__ __launch_bounds__(C::NT) void k_dz(Operand H, Operand W, int64_t kbytes, float inv,
                                              const float* __restrict__ lse, const float* __restrict__ g,
                                              const uint32_t* __restrict__ slots, _Float16* __restrict__ dz, int64_t ldz,
                                              TileMap map) {
    __shared__ i32x4 lds_v[C::kLds / 16];
    lds_u8* lds = (lds_u8*)(reinterpret_cast<uint8_t*>(lds_v));
    int64_t tm, tn;
    if (!map.at(blockIdx.x, &tm, &tn)) return;
    const int64_t i0 = tm * C::TL, j0 = tn * C::TR;
    f32x4 acc[C::BL][C::BR];
    tile_product<C>(acc, H, W, i0, j0, kbytes, lds);
    const int t = threadIdx.x, lane = t % 64, l16 = lane % 16;
    const int wave = __builtin_amdgcn_readfirstlane(t / 64), wl = wave / C::WR, wr = wave % C::WR;
    const uint32_t gmax = slots[2];
#pragma unroll
    for (int x = 0; x < C::BL; ++x) {
        int64_t row = i0 + (wl * C::BL + x) * 16 + l16;
        row = row < H.rows ? row : H.rows - 1;
        const float f = RowScale(g[row], gmax).f * kDzScale, l = lse[row];
#pragma unroll
        for (int y = 0; y < C::BR; ++y)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float p = probability(acc[x][y][i], inv, l);
                acc[x][y][i] = f == 0.f ? 0.f : p * f;
            }
    }
    // whole 16-byte pieces: ldz is a multiple of 8, and what a last piece
    // writes behind the piece's words is not read
    const int64_t cols = (W.rows + 7) / 8 * 8;
    store_tile<C>(acc, (lds_f32*)(lds + wave * C::kSlice), dz, ldz, i0 + wl * C::BL * 16, j0 + wr * C::BR * 16, H.rows,
                  cols, true, lane, [](float v) { return v; });
}

// dz at the listed words of a piece: the one place where the target's weight
// enters, so its difference from the softmax is rounded once.
__global__ __launch_bounds__(256) void k_dz_targets(const int64_t* __restrict__ index, const float* __restrict__ weight,
                                                    const float* __restrict__ zt, const float* __restrict__ lse,
                                                    const float* __restrict__ g, const uint32_t* __restrict__ slots,
                                                    int64_t n, int top, float inv, int64_t v0, int64_t vc, int64_t v,
                                                    const float* __restrict__ teacher, _Float16* __restrict__ dz,
                                                    int64_t ldz) {
    const int64_t u = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (u >= n * top) return;
    const int64_t row = u / top, word = index[u];
    if (!entry_counts(word, teacher ? teacher[u] : 0.f, v) || word < v0 || word >= v0 + vc) return;
    const float f = RowScale(g[row], slots[2]).f * kDzScale;
    const float p = probability(zt[u], inv, lse[row]);
    dz[row * ldz + word - v0] = static_cast<_Float16>(f == 0.f ? 0.f : (p - weight[u]) * f);
}

// dW of a piece: rows are words (L = dz^T), columns k (R = H^T).
template <class C, class CT>
__global__ __launch_bounds__(C::NT) void k_grad_w(Operand Z, Operand H, int64_t kbytes, CT* __restrict__ dw, int64_t k,
                                                  const uint32_t* __restrict__ slots, TileMap map) {
    __shared__ i32x4 lds_v[C::kLds / 16];
    lds_u8* lds = (lds_u8*)(reinterpret_cast<uint8_t*>(lds_v));
    int64_t tm, tn;
    if (!map.at(blockIdx.x, &tn, &tm)) return;
    const int64_t i0 = tm * C::TL, j0 = tn * C::TR;
    f32x4 acc[C::BL][C::BR];
    tile_product<C>(acc, Z, H, i0, j0, kbytes, lds);
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const Unscale unscale(slots[2], slots[0]);
    store_tile<C>(acc, (lds_f32*)(lds + wave * C::kSlice), dw, k, i0 + wave / C::WR * C::BL * 16,
                  j0 + wave % C::WR * C::BR * 16, Z.rows, H.rows, true, lane,
                  unscale);
}

// dH's sum over a part of a piece's words into its own fp32 buffer (blockIdx.y).
template <class C>
__global__ __launch_bounds__(C::NT) void k_grad_h(Operand Z, Operand W, int64_t kbytes, int64_t part_bytes,
                                                  float* __restrict__ sums, int add, TileMap map) {
    __shared__ i32x4 lds_v[C::kLds / 16];
    lds_u8* lds = (lds_u8*)(reinterpret_cast<uint8_t*>(lds_v));
    int64_t tm, tn;
    if (!map.at(blockIdx.x, &tm, &tn)) return;
    const int64_t i0 = tm * C::TL, j0 = tn * C::TR;
    const int64_t k0 = static_cast<int64_t>(blockIdx.y) * part_bytes;
    int64_t kb = kbytes - k0 < part_bytes ? kbytes - k0 : part_bytes;
    if (kb < 0) kb = 0;
    Z.data += kb ? k0 : 0;
    W.data += kb ? k0 : 0;
    f32x4 acc[C::BL][C::BR];
    tile_product<C>(acc, Z, W, i0, j0, kb, lds);
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int64_t k = W.rows, n = Z.rows, wi = i0 + wave / C::WR * C::BL * 16, wj = j0 + wave % C::WR * C::BR * 16;
    float* out = sums + static_cast<int64_t>(blockIdx.y) * n * k;
    // k is a multiple of 8, so a lane's four columns are inside or outside together
    const int g = lane / 16, l16 = lane % 16;
#pragma unroll
    for (int x = 0; x < C::BL; ++x)
#pragma unroll
        for (int y = 0; y < C::BR; ++y) {
            const int64_t r = wi + 16 * x + l16, c = wj + 16 * y + 4 * g;
            if (r >= n || c >= k) continue;
            f32x4* p = reinterpret_cast<f32x4*>(out + r * k + c);
            *p = add ? *p + acc[x][y] : acc[x][y];
        }
}

// dH from its parts.  A workgroup has 256 / quads rows of `quads` pieces of four
// (at least one), or 256 pieces of one (blockIdx.y).
template <class CT>
__global__ __launch_bounds__(256) void k_finish_h(const float* __restrict__ sums, int parts, int64_t n, uint32_t quads,
                                                  const float* __restrict__ g, const uint32_t* __restrict__ slots,
                                                  CT* __restrict__ dh) {
    typedef CT ct4 __attribute__((ext_vector_type(4)));
    const uint32_t t = threadIdx.x, rows = quads < 256 ? 256 / quads : 1, r = rows > 1 ? t / quads : 0;
    const uint32_t q = rows > 1 ? t - r * quads : blockIdx.y * 256 + t;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * rows + r, u = row * quads + q;
    if (r >= rows || q >= quads || row >= n) return;
    f32x4 s = reinterpret_cast<const f32x4*>(sums)[u];
    for (int p = 1; p < parts; ++p) s += reinterpret_cast<const f32x4*>(sums)[p * n * quads + u];
    const Unscale unscale(slots[2], slots[1], RowScale(g[row], slots[2]).s);
    ct4 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = static_cast<CT>(unscale(s[i]));
    reinterpret_cast<ct4*>(dh)[u] = o;
}

__global__ __launch_bounds__(256) void k_zero16(i32x4* __restrict__ p, int64_t pieces) {
    const int64_t step = static_cast<int64_t>(gridDim.x) * 256;
    for (int64_t u = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; u < pieces; u += step) p[u] = i32x4{0, 0, 0, 0};
}

unsigned blocks_of(int64_t n, int64_t per) { return static_cast<unsigned>((n + per - 1) / per); }

// Tiles of 256, 128 and 64 rows by 256 columns.
template <int ELEM> using Big = Config<ELEM, 0, 0, kNoScale, 4, 2, 4, 8>;
template <int ELEM> using Mid = Config<ELEM, 0, 0, kNoScale, 2, 4, 4, 4>;
template <int ELEM> using Low = Config<ELEM, 0, 0, kNoScale, 1, 8, 4, 2>;

template <int ELEM, class F>
hipError_t by_rows_of(int64_t tile_rows, F f) {
    if (tile_rows == 64) return f(Low<ELEM>{});
    if (tile_rows == 128) return f(Mid<ELEM>{});
    return f(Big<ELEM>{});
}
template <class F>
hipError_t by_rows(int64_t tile_rows, bool bf16, F f) {
    return bf16 ? by_rows_of<kBf16>(tile_rows, f) : by_rows_of<kF16>(tile_rows, f);
}

// slot: widened; g and gmax: rows times their 2^s.
hipError_t transpose16(const void* in, int64_t ldin, int64_t rows, int64_t cols, uint16_t* out, int64_t ldout, bool bf16,
                       const uint32_t* slot, const float* g, const uint32_t* gmax, hipStream_t stream) {
    const int64_t tc = (cols + 127) / 128, tr = (rows + 127) / 128;
    const auto kernel = bf16 ? k_transpose16<true, true> : slot ? k_transpose16<false, true> : k_transpose16<false, false>;
    hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(tc * tr)), dim3(256), 0, stream, static_cast<const uint16_t*>(in), ldin,
                       rows, cols, out, ldout, tc, slot, g, gmax);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_loss(const LossJob& j, hipStream_t stream) {
    const auto* h = static_cast<const uint8_t*>(j.h);
    const auto* w = static_cast<const uint8_t*>(j.w);
    auto* part = reinterpret_cast<float2*>(static_cast<uint8_t*>(j.ws));
    const Operand H{h, 2 * j.k, j.n, nullptr, 0, 0}, W{w, 2 * j.k, j.v, nullptr, 0, 0};
    const float c2 = kLog2e / j.tau, inv = 1.f / j.tau;
    int64_t tiles = 0;
    const hipError_t e = by_rows(loss_tile_rows(j.n, (j.v + 255) / 256), j.bf16, [&](auto cfg) {
        using C = decltype(cfg);
        const int64_t tm = (j.n + C::TL - 1) / C::TL;
        tiles = (j.v + C::TR - 1) / C::TR;
        const TileMap map = TileMap::make(tm, tiles);
        hipLaunchKernelGGL(k_logit_stats<C>, dim3(map.grid), dim3(C::NT), 0, stream, H, W, 2 * j.k, c2, part,
                           j.teacher ? nullptr : j.index, j.zt, map);
        return hipGetLastError();
    });
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(k_join_stats, dim3(blocks_of(j.n, 32)), dim3(256), 0, stream, part, tiles, j.n, c2, inv, j.lse,
                       j.teacher ? nullptr : j.index, j.v, j.zt, j.loss);
    if (j.teacher) {
        const int waves = (j.top + 15) / 16;
        hipLaunchKernelGGL(j.bf16 ? k_listed_loss<true> : k_listed_loss<false>, dim3(static_cast<unsigned>(j.n)),
                           dim3(64 * (waves < 4 ? waves : 4)), 0, stream, static_cast<const uint16_t*>(j.h),
                           static_cast<const uint16_t*>(j.w), j.index, j.teacher, j.v, j.k, j.top, j.tau, inv, j.lse,
                           j.zt, j.loss);
    }
    return hipGetLastError();
}

hipError_t launch_loss_grad(const LossJob& j, const LossPlan& p, hipStream_t stream) {
    auto* ws = static_cast<uint8_t*>(j.ws);
    if (j.n == 0) {  // no rows: the weights' gradient is zero (v k is a multiple of 8)
        if (j.dw) {
            const int64_t pieces = j.v * j.k / 8;  // may be more than one launch has threads
            const unsigned grid = pieces > 65536 * 256 ? 65536u : blocks_of(pieces, 256);
            hipLaunchKernelGGL(k_zero16, dim3(grid), dim3(256), 0, stream, static_cast<i32x4*>(j.dw), pieces);
        }
        return hipGetLastError();
    }
    auto* slots = reinterpret_cast<uint32_t*>(ws + p.slots);
    auto* g = reinterpret_cast<float*>(ws + p.g);
    auto* weight = reinterpret_cast<float*>(ws + p.weight);
    auto* dz = reinterpret_cast<_Float16*>(ws + p.dz);
    auto* dzt = reinterpret_cast<uint16_t*>(ws + p.dzt);
    auto* ht = reinterpret_cast<uint16_t*>(ws + p.ht);
    auto* wt = reinterpret_cast<uint16_t*>(ws + p.wt);
    auto* sums = reinterpret_cast<float*>(ws + p.sums);
    const float inv = 1.f / j.tau;
    const int64_t ldn = (j.n + 7) / 8 * 8;
    hipLaunchKernelGGL(k_clear_slots, dim3(1), dim3(64), 0, stream, slots);
    if (j.teacher)
        hipLaunchKernelGGL(k_distill_prep, dim3(static_cast<unsigned>(j.n)), dim3(64), 0, stream, j.index, j.teacher, j.upstream,
                           j.v, j.top, j.tau, weight, g, slots + 2);
    else
        hipLaunchKernelGGL(k_ce_prep, dim3(blocks_of(j.n, 256)), dim3(256), 0, stream, j.index, j.upstream, j.n, j.v, weight, g,
                           slots + 2);
    const int64_t hp = j.dw ? j.n * j.k / 8 : 0, wp = j.dh && j.bf16 ? j.v * j.k / 8 : 0, most = hp > wp ? hp : wp;
    if (most) {
        const dim3 grid(most > 1024 * 256 ? 1024u : blocks_of(most, 256), wp ? 2 : 1);
        hipLaunchKernelGGL(j.bf16 ? k_absmax<true> : k_absmax<false>, grid, dim3(256), 0, stream, static_cast<const uint16_t*>(j.h),
                           hp, static_cast<uint32_t>(j.k / 8), g, static_cast<const uint16_t*>(j.w), wp, slots);
    }
    hipError_t e = hipGetLastError();
    if (e == hipSuccess && j.dw) e = transpose16(j.h, j.k, j.n, j.k, ht, ldn, j.bf16, slots, g, slots + 2, stream);
    for (int64_t v0 = 0; v0 < j.v && e == hipSuccess; v0 += p.piece) {
        const int64_t vc = j.v - v0 < p.piece ? j.v - v0 : p.piece, ldz = (vc + 7) / 8 * 8;
        const uint8_t* wp = static_cast<const uint8_t*>(j.w) + v0 * j.k * 2;
        const Operand H{static_cast<const uint8_t*>(j.h), 2 * j.k, j.n, nullptr, 0, 0}, W{wp, 2 * j.k, vc, nullptr, 0, 0};
        e = by_rows(loss_tile_rows(j.n, (vc + 255) / 256), j.bf16, [&](auto cfg) {
            using C = decltype(cfg);
            const int64_t tm = (j.n + C::TL - 1) / C::TL, tn = (vc + C::TR - 1) / C::TR;
            const TileMap map = TileMap::make(tm, tn);
            hipLaunchKernelGGL(k_dz<C>, dim3(map.grid), dim3(C::NT), 0, stream, H, W, 2 * j.k, inv, j.lse, g, slots, dz, ldz, map);
            return hipGetLastError();
        });
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL(k_dz_targets, dim3(blocks_of(j.n * j.top, 256)), dim3(256), 0, stream, j.index, weight, j.zt, j.lse, g,
                           slots, j.n, j.top, inv, v0, vc, j.v, j.teacher, dz, ldz);
        if (j.dw) {
            e = transpose16(dz, ldz, j.n, vc, dzt, ldn, false, nullptr, nullptr, nullptr, stream);
            if (e != hipSuccess) return e;
            const Operand Z{reinterpret_cast<const uint8_t*>(dzt), 2 * ldn, vc, nullptr, 0, 0};
            const Operand HT{reinterpret_cast<const uint8_t*>(ht), 2 * ldn, j.k, nullptr, 0, 0};
            e = by_rows_of<kF16>(loss_tile_rows(vc, (j.k + 255) / 256), [&](auto cfg) {
                using C = decltype(cfg);
                const int64_t tm = (vc + C::TL - 1) / C::TL, tn = (j.k + C::TR - 1) / C::TR;
                const TileMap map = TileMap::make(tn, tm);
                if (j.bf16)
                    hipLaunchKernelGGL((k_grad_w<C, __bf16>), dim3(map.grid), dim3(C::NT), 0, stream, Z, HT, 2 * j.n,
                                       static_cast<__bf16*>(j.dw) + v0 * j.k, j.k, slots, map);
                else
                    hipLaunchKernelGGL((k_grad_w<C, _Float16>), dim3(map.grid), dim3(C::NT), 0, stream, Z, HT, 2 * j.n,
                                       static_cast<_Float16*>(j.dw) + v0 * j.k, j.k, slots, map);
                return hipGetLastError();
            });
        }
        if (j.dh && e == hipSuccess) {
            e = transpose16(wp, j.k, vc, j.k, wt, ldz, j.bf16, j.bf16 ? slots + 1 : nullptr, nullptr, nullptr, stream);
            if (e != hipSuccess) return e;
            const Operand Z{reinterpret_cast<const uint8_t*>(dz), 2 * ldz, j.n, nullptr, 0, 0};
            const Operand WT{reinterpret_cast<const uint8_t*>(wt), 2 * ldz, j.k, nullptr, 0, 0};
            // whole stages of 128 bytes a part
            const int64_t part_bytes = ((2 * vc + 127) / 128 + p.parts - 1) / p.parts * 128;
            e = by_rows_of<kF16>(p.h_rows, [&](auto cfg) {
                using C = decltype(cfg);
                const int64_t tm = (j.n + C::TL - 1) / C::TL, tn = (j.k + C::TR - 1) / C::TR;
                const TileMap map = TileMap::make(tm, tn);
                hipLaunchKernelGGL(k_grad_h<C>, dim3(map.grid, static_cast<unsigned>(p.parts)), dim3(C::NT), 0, stream, Z, WT,
                                   2 * vc, part_bytes, sums, v0 > 0 ? 1 : 0, map);
                return hipGetLastError();
            });
        }
    }
    if (e == hipSuccess && j.dh) {
        const uint32_t quads = static_cast<uint32_t>(j.k / 4), rows = quads < 256 ? 256 / quads : 1;
        const dim3 grid(blocks_of(j.n, rows), (quads + 255) / 256);
        if (j.bf16)
            hipLaunchKernelGGL(k_finish_h<__bf16>, grid, dim3(256), 0, stream, sums, static_cast<int>(p.parts), j.n, quads, g, slots,
                               static_cast<__bf16*>(j.dh));
        else
            hipLaunchKernelGGL(k_finish_h<_Float16>, grid, dim3(256), 0, stream, sums, static_cast<int>(p.parts), j.n, quads, g, slots,
                               static_cast<_Float16*>(j.dh));
        e = hipGetLastError();
    }
    return e;
}

}  // namespace swz
