// C = X W^T of a few rows of X with weights of 4 bits, w = (code - zero) scale per
// group of 32, 64 or 128 along k; and the gated block of two such weights.
//
// A workgroup owns 16 NB rows of W (of both matrices of a gated block) and up to
// 64 rows of X; its waves split k into runs of whole blocks of 128, and their sums are
// joined through LDS in their order.  W comes from HBM once for 64 rows of X; X, read
// again by every workgroup, comes from the caches.
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
#include "activation.h"
#include "launch_ffn.h"
#include "mma_core.h"
#include "w4_layout.h"

namespace swz {
namespace {

using namespace mma;

typedef __attribute__((address_space(3))) uint16_t lds_u16;

template <bool BF16>
using Value = std::conditional_t<BF16, __bf16, _Float16>;

unsigned blocks_of(int64_t n, int64_t per) { return static_cast<unsigned>((n + per - 1) / per); }

template <bool BF16>
__device__ __forceinline__ i32x4 operand_of(uint32_t word) {
    constexpr uint32_t kMask = BF16 ? 0x00780078u : 0x03c003c0u, kOne = BF16 ? 0x41804180u : 0x4c004c00u;
    constexpr int kUp = BF16 ? 3 : 6;  // where the code's lowest bit belongs
    i32x4 v;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t m = 4 * j <= kUp ? word << (kUp - 4 * j) : word >> (4 * j - kUp);
        v[j] = __builtin_amdgcn_bitop3_b32(m, kMask, kOne, 0xea);  // (m & kMask) | kOne
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

// What bounds it beside W's bytes is the way of addresses: an instruction whose
// lanes touch many lines costs by the line.  So X comes in whole 256-byte runs, four
// rows an instruction, and the scales and zero points of 32 groups at a time.  8 x
// 8192 x 8192 gated, us: fragments of X as they lie (64 lines an instruction) and a
// load of scales a block 28, X in runs 25, scales in runs 23, X by 8 rows 21; W's
// loads alone 15.
//
// W and X go straight into LDS, a block a wave, and from there into registers;
// then the next block's loads start, and this one's products run beside them.  No
// other wave reads a wave's block, so the loop has no barrier.  Two to eight blocks in
// flight were slower (19 to 25 us where this takes 18: LDS halves the waves),
// and so was the same by way of registers.  The code is short on purpose: a call
// that runs each instruction a few times waits for the instructions (4 x 2048 x 1024
// gated: 4.7 us, 12 with four blocks in a step).
//
// What a wave holds in LDS, and where: W4Layout.
// MATS: 1, or 2 for a gated block.  XL: X's rows in fours.
template <bool BF16, int GROUP, bool ZERO, int MATS, int NB, int XL, int WAVES>
__device__ __forceinline__ void gemm_w4(const uint8_t* __restrict__ x, const WeightsW4& w0, const WeightsW4& w1, int64_t m, int64_t n,
                                        int64_t k, int act, Value<BF16>* __restrict__ c) {
    using V = Value<BF16>;
    using L = W4Layout<GROUP, ZERO, MATS, NB, XL>;
    constexpr int MB = L::MB, PER = L::PER, COLS = L::COLS, kRun = L::kRun, kScaleRow = L::kScaleRow, kZeroRow = L::kZeroRow;
    constexpr int kZero = L::kZero, kW = L::kW, kX = L::kX, kRed = L::kRed, kOwn = L::kOwn;
    __shared__ i32x4 lds_v[WAVES * (kOwn > kRed ? kOwn : kRed) / 16];
    const int t = threadIdx.x, lane = t % 64, g = lane / 16, l16 = lane % 16;
    const int wave = __builtin_amdgcn_readfirstlane(t / 64);
    lds_u8* own = (lds_u8*)(reinterpret_cast<uint8_t*>(lds_v)) + wave * kOwn;
    const int64_t n0 = static_cast<int64_t>(blockIdx.x) * (16 * NB), m0 = static_cast<int64_t>(blockIdx.y) * (4 * XL);
    const int64_t groups = (k + GROUP - 1) / GROUP, blocks = (k + 127) / 128;
    const WeightsW4 from[2] = {w0, w1};
    // rows behind the last are read as the last; their results are not stored
    auto w_row = [&](int o, int r) {
        const int64_t row = n0 + 16 * (o % NB) + r;
        return row < n ? row : n - 1;
    };
    auto x_row = [&](int r) { return m0 + r < m ? m0 + r : m - 1; };
    // this lane's rows in the loads; its piece of W's is cq, its unit of X's cx(a)
    const uint8_t *pq[COLS], *px[XL];
    const int cq = (lane % 4) ^ g;
    auto cx = [&](int a) { return l16 ^ ((4 * a + g) % 16); };
#pragma unroll
    for (int o = 0; o < COLS; ++o) pq[o] = from[o / NB].q + w_row(o, lane / 4) * (k / 2);
#pragma unroll
    for (int a = 0; a < XL; ++a) px[a] = x + 2 * x_row(4 * a + g) * k;
    f32x4 total[COLS][MB];
#pragma unroll
    for (int o = 0; o < COLS; ++o)
#pragma unroll
        for (int a = 0; a < MB; ++a) total[o][a] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int one = BF16 ? 0x3f803f80 : 0x3c003c00;
    const i32x4 ones = {one, one, one, one};
    const int64_t first = blocks * wave / WAVES, end = blocks * (wave + 1) / WAVES;

    // Scales and zero points of kRun groups from `grp` on, group 4 i + g to lane
    // (g, l16) for its row, i < 8, as far as this wave's blocks reach; 0 behind the
    // row's last.
    uint16_t vs[COLS][kRun / 4];
    uint8_t vz[COLS][kRun / 4];
    const int64_t last_group = end * PER;
    auto fetch_groups = [&](int64_t grp) {
#pragma unroll
        for (int o = 0; o < COLS; ++o) {
            const int64_t at = w_row(o, l16) * groups;
#pragma unroll
            for (int i = 0; i < kRun / 4; ++i) {
                if (grp + 4 * i >= last_group) break;
                const int64_t j = grp + 4 * i + g < groups ? grp + 4 * i + g : groups - 1;
                vs[o][i] = static_cast<const uint16_t*>(from[o / NB].scale)[at + j];
                if constexpr (ZERO) vz[o][i] = from[o / NB].zero[at + j];
            }
        }
    };
    auto put_groups = [&](int64_t grp) {
#pragma unroll
        for (int o = 0; o < COLS; ++o)
#pragma unroll
            for (int i = 0; i < kRun / 4; ++i) {
                if (grp + 4 * i >= last_group) break;
                const bool here = grp + 4 * i + g < groups;
                *reinterpret_cast<lds_u16*>(own + (o * 16 + l16) * kScaleRow + 2 * (4 * i + g)) = here ? vs[o][i] : uint16_t(0);
                if constexpr (ZERO) own[kZero + (o * 16 + l16) * kZeroRow + 4 * i + g] = vz[o][i];
            }
    };
    // Loads of block b.  Where k ends in it, what lies behind is read from the
    // block's start, and X there counts as zero.
    auto units_of = [&](int64_t b) { return k - b * 128 < 128 ? static_cast<int>((k - b * 128) / 8) : 16; };
    auto issue = [&](int64_t b) {
        const int units = units_of(b);
#pragma unroll
        for (int o = 0; o < COLS; ++o)
            __builtin_amdgcn_global_load_lds(pq[o] + b * 64 + (4 * cq < units ? 16 * cq : 0), own + kW + o * 1024, 16, 0, 0);
#pragma unroll
        for (int a = 0; a < XL; ++a)
            __builtin_amdgcn_global_load_lds(px[a] + b * 256 + (cx(a) < units ? 16 * cx(a) : 0), own + kX + a * 1024, 16, 0, 0);
    };
    // What this lane has of a block: pieces of W, scales (two a word) and zero
    // points (four a word) of its row, fragments of X.
    struct Block {
        i32x4 q[COLS], x[MB][4];
        uint32_t s[COLS][2], z[COLS];
    };
    // at: of the run's groups, the block's first
    auto read_groups = [&](Block& v, int at) {
#pragma unroll
        for (int o = 0; o < COLS; ++o) {
            const lds_u8* s = own + (o * 16 + l16) * kScaleRow + 2 * at;
            const lds_u8* z = own + kZero + (o * 16 + l16) * kZeroRow + at;
            if constexpr (PER == 1) {
                v.s[o][0] = *reinterpret_cast<const lds_u16*>(s);
                if constexpr (ZERO) v.z[o] = z[0];
            } else {
#pragma unroll
                for (int p = 0; p < PER / 2; ++p) v.s[o][p] = *reinterpret_cast<const lds_u32*>(s + 4 * p);
                if constexpr (ZERO && PER == 2) v.z[o] = *reinterpret_cast<const lds_u16*>(z);
                if constexpr (ZERO && PER == 4) v.z[o] = *reinterpret_cast<const lds_u32*>(z);
            }
        }
    };
    // Of whose X `units` count.
    auto read = [&](Block& v, int units) {
#pragma unroll
        for (int o = 0; o < COLS; ++o)
            v.q[o] = *reinterpret_cast<const lds_i32x4*>(own + L::w_at(o, l16, g));
#pragma unroll
        for (int a = 0; a < MB; ++a)
#pragma unroll
            for (int s = 0; s < 4; ++s)
                v.x[a][s] = *reinterpret_cast<const lds_i32x4*>(own + L::x_at(a, L::x_row(l16), w4_unit_of<GROUP>(s, g)));
        if (units < 16) {
#pragma unroll
            for (int a = 0; a < MB; ++a)
#pragma unroll
                for (int s = 0; s < 4; ++s)
                    if (w4_unit_of<GROUP>(s, g) >= units) v.x[a][s] = i32x4{0, 0, 0, 0};
        }
    };
    auto scale = [](const uint32_t* s, int p) {
        const uint32_t h = p % 2 ? s[p / 2] >> 16 : s[p / 2] & 0xffffu;
        if constexpr (BF16) return __uint_as_float(h << 16);
        return static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(h)));
    };
    auto products = [&](const Block& v) {
        i32x4 vw[COLS][4];
#pragma unroll
        for (int o = 0; o < COLS; ++o) {
            int q[4] = {v.q[o][0], v.q[o][1], v.q[o][2], v.q[o][3]};
            if constexpr (GROUP < 128) {
                swap32(q[0], q[2]);
                swap32(q[1], q[3]);
            }
            if constexpr (GROUP < 64) {
                swap16(q[0], q[1]);
                swap16(q[2], q[3]);
            }
#pragma unroll
            for (int s = 0; s < 4; ++s) vw[o][s] = operand_of<BF16>(static_cast<uint32_t>(q[s]));
        }
#pragma unroll
        for (int a = 0; a < MB; ++a) {
            f32x4 sx[PER];
#pragma unroll
            for (int p = 0; p < PER; ++p) sx[p] = f32x4{0.f, 0.f, 0.f, 0.f};
            i32x4 f[4];
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                f[s] = paired(v.x[a][s]);
                sx[s * PER / 4] = mfma16<BF16>(f[s], ones, sx[s * PER / 4]);
            }
#pragma unroll
            for (int o = 0; o < COLS; ++o) {
                f32x4 acc[PER];
#pragma unroll
                for (int p = 0; p < PER; ++p)
                    acc[p] = sx[p] * -(16.f + (ZERO ? static_cast<float>((v.z[o] >> (8 * p)) & 255u) : 8.f));
#pragma unroll
                for (int s = 0; s < 4; ++s) acc[s * PER / 4] = mfma16<BF16>(f[s], vw[o][s], acc[s * PER / 4]);
#pragma unroll
                for (int p = 0; p < PER; ++p)
#pragma unroll
                    for (int i = 0; i < 4; ++i) total[o][a][i] = __builtin_fmaf(acc[p][i], scale(v.s[o], p), total[o][a][i]);
            }
        }
    };
    if (first < end) {
        fetch_groups(first * PER);
        issue(first);
        put_groups(first * PER);
        int run = 0;  // of the run's groups, the next block's first
        for (int64_t b = first; b < end; ++b) {
            if (run == kRun) {
                fetch_groups(b * PER);
                put_groups(b * PER);
                run = 0;
            }
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            Block v;
            read_groups(v, run);
            read(v, units_of(b));
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            __builtin_amdgcn_sched_barrier(0);
            if (b + 1 < end) issue(b + 1);
            asm volatile("" ::: "memory");
            products(v);
            run += PER;
        }
    }

    // lane (g, l16): rows 4g .. 4g+3 of X, row l16 of W
    __syncthreads();
    lds_f32* red = (lds_f32*)(reinterpret_cast<float*>(lds_v));
#pragma unroll
    for (int a = 0; a < MB; ++a)
#pragma unroll
        for (int o = 0; o < COLS; ++o)
#pragma unroll
            for (int i = 0; i < 4; ++i) red[((wave * MB + a) * COLS + o) * 256 + (4 * g + i) * 16 + l16] = total[o][a][i];
    __syncthreads();
    for (int e = t; e < MB * NB * 256; e += 64 * WAVES) {
        const int a = e / (NB * 256), o = e / 256 % NB, r = e % 256;
        const int64_t i = m0 + 16 * a + r / 16, j = n0 + 16 * o + r % 16;
        if (16 * a + r / 16 >= 4 * XL || i >= m || j >= n) continue;
        float z[MATS];
#pragma unroll
        for (int v = 0; v < MATS; ++v) {
            z[v] = 0.f;
#pragma unroll
            for (int u = 0; u < WAVES; ++u) z[v] += red[((u * MB + a) * COLS + v * NB + o) * 256 + r];
        }
        if constexpr (MATS == 2) {
            const float h = act == SWZ_ACT_GELU ? act::both<SWZ_ACT_GELU, false>(z[0]).x
                            : act == SWZ_ACT_GELU_TANH ? act::both<SWZ_ACT_GELU_TANH, false>(z[0]).x
                                                       : act::both<SWZ_ACT_SILU, false>(z[0]).x;
            z[0] = h * z[1];
        }
        c[i * n + j] = static_cast<V>(z[0]);
    }
}

template <bool BF16, int GROUP, bool ZERO, int MATS, int NB, int XL, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void k_gemm_w4(const uint8_t* __restrict__ x, WeightsW4 w0, WeightsW4 w1, int64_t m,
                                                        int64_t n, int64_t k, int act, Value<BF16>* __restrict__ c) {
    gemm_w4<BF16, GROUP, ZERO, MATS, NB, XL, WAVES>(x, w0, w1, m, n, k, act, c);
}

template <bool BF16, int GROUP, bool ZERO, int MATS, int NB, int XL, int WAVES>
hipError_t run(const GemmW4Job& j, hipStream_t stream) {
    // rows of X by the grid's second axis, as many a launch as it takes
    constexpr int64_t kRows = 4 * XL, kMost = 32768 * kRows;
    for (int64_t r0 = 0; r0 < j.m; r0 += kMost) {
        const int64_t rows = j.m - r0 < kMost ? j.m - r0 : kMost;
        hipLaunchKernelGGL((k_gemm_w4<BF16, GROUP, ZERO, MATS, NB, XL, WAVES>), dim3(blocks_of(j.n, 16 * NB), blocks_of(rows, kRows)),
                           dim3(64 * WAVES), 0, stream, static_cast<const uint8_t*>(j.x) + 2 * r0 * j.k, j.w[0], j.w[1], rows, j.n,
                           j.k, j.act, static_cast<Value<BF16>*>(j.c) + r0 * j.n);
    }
    return hipGetLastError();
}

// X's rows by the smallest size that holds them, 64 at most; four waves where a
// block of X is 16 KiB (LDS).
template <bool BF16, int GROUP, bool ZERO, int MATS, int NB>
hipError_t by_rows(const GemmW4Job& j, hipStream_t stream) {
    if (j.m <= 4) return run<BF16, GROUP, ZERO, MATS, NB, 1, 8>(j, stream);
    if (j.m <= 8) return run<BF16, GROUP, ZERO, MATS, NB, 2, 8>(j, stream);
    if (j.m <= 16) return run<BF16, GROUP, ZERO, MATS, NB, 4, 8>(j, stream);
    if (j.m <= 32) return run<BF16, GROUP, ZERO, MATS, NB, 8, 8>(j, stream);
    return run<BF16, GROUP, ZERO, MATS, NB, 16, 4>(j, stream);
}

// 32 rows of W a workgroup, so that X is read half as often (64 x 8192 x 4096: 17
// us, 24 with 16), but 16 where all those run at once anyway, one a compute
// unit (1 x 1024 x 4096: 5.0 us, 6.4 with 32).  A gated block has 16 of both.
template <bool BF16, int GROUP, bool ZERO>
hipError_t by_columns(const GemmW4Job& j, hipStream_t stream) {
    if (j.act >= 0) return by_rows<BF16, GROUP, ZERO, 2, 1>(j, stream);
    return j.n <= 16 * 256 ? by_rows<BF16, GROUP, ZERO, 1, 1>(j, stream) : by_rows<BF16, GROUP, ZERO, 1, 2>(j, stream);
}

template <bool BF16, int GROUP>
hipError_t by_zero(const GemmW4Job& j, hipStream_t stream) {
    return j.w[0].zero ? by_columns<BF16, GROUP, true>(j, stream) : by_columns<BF16, GROUP, false>(j, stream);
}
template <bool BF16>
hipError_t by_group(const GemmW4Job& j, hipStream_t stream) {
    return j.group == 32 ? by_zero<BF16, 32>(j, stream) : j.group == 64 ? by_zero<BF16, 64>(j, stream) : by_zero<BF16, 128>(j, stream);
}

}  // namespace

hipError_t launch_gemm_w4(const GemmW4Job& j, hipStream_t stream) { return j.bf16 ? by_group<true>(j, stream) : by_group<false>(j, stream); }

}  // namespace swz
