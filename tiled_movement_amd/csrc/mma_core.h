// Core of the products of K-contiguous operands: C[i][j] = sum_k L[i][k] R[j][k]
// with both operands staged through swizzled LDS tiles of 128-byte rows, 64
// two-byte or 128 one-byte values of k per stage.
//
// A workgroup of WL x WR waves owns a TL x TR tile of C.  Per stage it brings
// TL rows of L and TR rows of R, 128 bytes each, into LDS with direct
// HBM -> LDS loads of 16 bytes per lane.  16-byte slot p = 8 row + chunk of a
// tile holds the tile element of slot swizzle(p), Swizzle<3,0,4> on slots
// (Swizzle<3,3,4> on two-byte elements): the row's bits 1..3 are XORed into
// its chunk, so the 16 rows that one fragment read touches in the same chunk
// fall on 16 different 16-byte groups of the 64 banks (0 predicted and
// measured conflict cycles; plain rows: 96 per 256 x 64 tile read).  Bits 4 and
// up of the row stay out of the swizzle, so a lane's fragment addresses
// differ by constants only and fold into the read instructions' offsets.
//
// Fragments: lane l reads row l%16 of a 16-row block, chunks l/16 and
// l/16 + 4.  For the 16x16x32 two-byte instructions these are the two k steps
// of the stage; for the 16x16x128 one-byte instruction they are the lane's 32
// values of k.  That is not the instruction's own k order, but a sum over k
// only asks that both operands use the same one, and the block of 128 shares
// its scale.
//
// The R operand feeds the instruction's rows and L its columns, so lane l of
// the wave holds four consecutive j (4*(l/16) .. +3 of a block) of one i
// (l%16): results leave in runs along j, sums over j are sums within a lane
// before they are sums over lanes, and an L row's scale is one number a lane.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace swz {
namespace mma {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) uint8_t lds_u8;
typedef __attribute__((address_space(3))) float lds_f32;
typedef __attribute__((address_space(3))) f32x4 lds_f32x4;
typedef __attribute__((address_space(3))) uint32_t lds_u32;
typedef __attribute__((address_space(3))) i32x4 lds_i32x4;

// kF8Wide: one-byte operands widened to bf16 in registers (exact) and
// multiplied by the bf16 instruction, at its rate.  The one-byte instructions
// align the products of each group of eight values of k to the largest and
// keep about 13 bits below it: 1.5e-5 of the result's norm on normal
// operands (16x16x32 and 16x16x128 alike), against 4e-8 for bf16.
enum Elem { kBf16, kF16, kF8, kF8Wide };
// Scales of one-byte operands, one per row (or 128 rows) and stage: none;
// powers of two as exponent bytes, applied by the matrix instruction; fp32,
// applied to the stage's product (kF32Square: R's scale is the same for all
// rows of a wave, so only L's varies within a register block).
enum Scale { kNoScale, kE8M0, kF32Rows, kF32Square };

struct Operand {
    const uint8_t* data;  // [rows][ld] bytes
    int64_t ld;           // row pitch in bytes, a multiple of 16, below kMaxPitch
    int64_t rows;
    const void* scale;    // [rows >> scale_shift][scale_ld]
    int64_t scale_ld;
    int scale_shift;      // 0: a scale per row, 7: per 128 rows
};

template <int ELEM_, int LT_, int RT_, int SC_, int WL_, int WR_, int BL_, int BR_>
struct Config {
    static constexpr int ELEM = ELEM_, LT = LT_, RT = RT_, SC = SC_;
    static constexpr int WL = WL_, WR = WR_, BL = BL_, BR = BR_;  // waves; blocks of 16 rows per wave
    static constexpr int NT = 64 * WL * WR;
    static constexpr int TL = 16 * WL * BL, TR = 16 * WR * BR;
    static constexpr int kBuf = (TL + TR) * 128;
    // The 4 x 2 waves of 4 x 8 blocks run their own main loop (slots); the
    // others keep several stages in flight (deep).
    static constexpr bool kSlots = BL == 4 && BR == 8 && WL == 4 && WR == 2 && ELEM != kF8Wide;
    static constexpr int NS = (TL + TR + NT - 1) / NT;  // scales a thread stages
    // Scales of a stage in LDS: a word a row; slots with E8M0 a byte a row.
    static constexpr bool kScaleBytes = SC == kE8M0 && kSlots;
    static constexpr int kScaleBuf = SC == kNoScale ? 0 : kScaleBytes ? (TL + TR + 63) / 64 * 64 : NS * NT * 4;
    static constexpr int kStage = kBuf + kScaleBuf;
    static constexpr int kFit = 160 * 1024 / kStage;
    static constexpr int NBUF = kSlots ? 2 : kFit < 4 ? kFit : 4;
    static constexpr int kMain = NBUF * kStage;
    // Two stages: scales go through registers, and E8M0 ones of widened
    // operands become fp32 on the way, once a row instead of once a fragment.
    static constexpr bool kPutScales = NBUF == 2;
    // a wave's slice of the epilogue: 16 rows of C, padded by 16 bytes
    static constexpr int kPitch = 16 * BR + 4;
    static constexpr int kSlice = 16 * kPitch * 4;
    static constexpr int kLds = kMain > WL * WR * kSlice ? kMain : WL * WR * kSlice;
    static_assert(NBUF >= 2, "two stages fit in LDS");
    static_assert(TL * 8 % NT == 0 && TR * 8 % NT == 0 && NT % 128 == 0, "the fills split evenly");
    static_assert(kLds <= 160 * 1024, "the stages fit in LDS");
};

__device__ __forceinline__ void wg_barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// Which tile a workgroup takes, in a grid of f x s tiles (f: the direction
// that neighbours step along).  Workgroups go to the eight XCDs in turn, and
// the 32 of an XCD that run at once share its L2: the fewer rows and columns of
// tiles they span, the less is fetched.  The XCDs are laid out 2^log_xf along f
// by 8 / 2^log_xf along s, each taking every such tile, so that an XCD's 32
// cover about 4 x 8 tiles (against tiles dealt out along f: distillation step
// 2000 x 50001 x 2048, 8 tiles of rows, 2.07 -> 1.96 ms; cross entropy step 4096
// x 65536 x 4096, 16 of them, 7.80 -> 7.59 ms; in turn on one box).
struct TileMap {
    uint32_t f, s, log_xf, grid;
    static TileMap make(int64_t f, int64_t s) {
        uint32_t log_xf = 0;
        while (log_xf < 3 && (f >> (log_xf + 1)) >= 4) ++log_xf;
        const int64_t fl = (f + (1 << log_xf) - 1) >> log_xf, xs = 8 >> log_xf, sl = (s + xs - 1) / xs;
        return TileMap{static_cast<uint32_t>(f), static_cast<uint32_t>(s), log_xf, static_cast<uint32_t>(8 * fl * sl)};
    }
    // False for the workgroups that have no tile.
    __device__ __forceinline__ bool at(uint32_t id, int64_t* fi, int64_t* si) const {
        const uint32_t x = id & 7u, slot = id >> 3, fl = (f + (1u << log_xf) - 1) >> log_xf;
        const uint32_t a = ((slot % fl) << log_xf) + (x & ((1u << log_xf) - 1)), b = slot / fl * (8u >> log_xf) + (x >> log_xf);
        *fi = a;
        *si = b;
        return a < f && b < s;
    }
};

// 16-byte slot of a tile that holds tile slot p, and the reverse.
__device__ __forceinline__ uint32_t swz_slot(uint32_t p) { return p ^ ((p >> 4) & 7u); }

// This thread's part of the fills of one operand's tile: slots t + NT q.
// swizzle(t + NT q) = swizzle(t) + NT q (NT is a multiple of 128), so the
// chunk is the same for all q and the row moves by NT / 8.  Rows behind the
// operand's last are read as its last row; their results are not stored.
template <int T, int NT>
struct Fill {
    static constexpr int Q = T * 8 / NT;
    const uint8_t* base;
    uint32_t off[Q];
    uint32_t chunk16;
    __device__ __forceinline__ void init(const Operand& o, int64_t row0, int t) {
        base = o.data + row0 * o.ld;
        const uint32_t e = swz_slot(static_cast<uint32_t>(t));
        chunk16 = 16 * (e % 8);
        const int64_t left = o.rows - row0 - 1;
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const int64_t r = static_cast<int64_t>(e / 8 + NT / 8 * q);
            off[q] = static_cast<uint32_t>((r < left ? r : left) * o.ld) + chunk16;
        }
    }
    // rem: bytes of k from this stage on; chunks behind them are read from
    // the stage's first chunk (masked when used).
    __device__ __forceinline__ void issue(int64_t stage, int64_t rem, lds_u8* dst, int wave) const {
        const uint8_t* b = base + stage * 128;
        const uint32_t back = static_cast<int64_t>(chunk16) < rem ? 0u : chunk16;
#pragma unroll
        for (int q = 0; q < Q; ++q)
            __builtin_amdgcn_global_load_lds(b + (off[q] - back), dst + 16 * (64 * wave + NT * q), 16, 0, 0);
    }
};

// 2^(b - 127) of the low byte of a word; 255 is NaN.
__device__ __forceinline__ float e8m0_value(uint32_t w) {
    const uint32_t b = w & 255u;
    return __uint_as_float(b == 255u ? 0x7fc00000u : b ? b << 23 : 0x400000u);
}

template <class C>
struct Stager {
    Fill<C::TL, C::NT> fl;
    Fill<C::TR, C::NT> fr;
    const uint8_t* sp[C::NS ? C::NS : 1];  // this thread's scales, advanced stage by stage
    uint32_t sv[C::NS ? C::NS : 1];
    int t, wave;
    int64_t kbytes;

    __device__ __forceinline__ void init(const Operand& L, const Operand& R, int64_t l0, int64_t r0, int64_t kb,
                                         int tid) {
        t = tid;
        wave = __builtin_amdgcn_readfirstlane(tid / 64);
        kbytes = kb;
        fl.init(L, l0, tid);
        fr.init(R, r0, tid);
        if constexpr (C::SC != kNoScale) {
            constexpr int ES = C::SC == kE8M0 ? 1 : 4;
#pragma unroll
            for (int i = 0; i < C::NS; ++i) {
                int e = t + C::NT * i;
                if (e >= C::TL + C::TR) e = C::TL + C::TR - 1;
                const bool left = e < C::TL;
                const Operand& o = left ? L : R;
                int64_t row = left ? l0 + e : r0 + (e - C::TL);
                row = row < o.rows ? row : o.rows - 1;
                sp[i] = static_cast<const uint8_t*>(o.scale) + (row >> o.scale_shift) * o.scale_ld * ES;
            }
        }
    }
    __device__ __forceinline__ void issue(int64_t s, lds_u8* buf) {
        issue_l(s, buf);
        issue_r(s, buf);
    }
    __device__ __forceinline__ void issue_l(int64_t s, lds_u8* buf) const { fl.issue(s, kbytes - s * 128, buf, wave); }
    __device__ __forceinline__ void issue_r(int64_t s, lds_u8* buf) {
        fr.issue(s, kbytes - s * 128, buf + C::TL * 128, wave);
        if constexpr (C::SC == kE8M0) {
#pragma unroll
            for (int i = 0; i < C::NS; ++i) sv[i] = sp[i][s];
        } else if constexpr (C::SC != kNoScale) {
#pragma unroll
            for (int i = 0; i < C::NS; ++i) sv[i] = reinterpret_cast<const uint32_t*>(sp[i])[s];
        }
    }
    // The same with the scales straight into LDS, so that a stage is a fixed
    // number of loads into LDS and nothing else: the aligned word that holds
    // an E8M0 scale's byte (in its page, and what else it holds is not used),
    // or the fp32 scale.
    static constexpr int kLoads = Fill<C::TL, C::NT>::Q + Fill<C::TR, C::NT>::Q + (C::SC == kNoScale ? 0 : C::NS);
    __device__ __forceinline__ void issue_deep(int64_t s, lds_u8* buf) const {
        fl.issue(s, kbytes - s * 128, buf, wave);
        fr.issue(s, kbytes - s * 128, buf + C::TL * 128, wave);
        if constexpr (C::SC != kNoScale) {
#pragma unroll
            for (int i = 0; i < C::NS; ++i) {
                const uintptr_t at = reinterpret_cast<uintptr_t>(sp[i] + s * (C::SC == kE8M0 ? 1 : 4)) & ~uintptr_t(3);
                __builtin_amdgcn_global_load_lds(reinterpret_cast<const uint8_t*>(at), buf + C::kBuf + 4 * (64 * wave + C::NT * i),
                                                 4, 0, 0);
            }
        }
    }
    // Scales that issue() fetched into their LDS buffer: fp32 by row; bytes so
    // that the four rows 16 apart of a 64-row group share a word.
    __device__ __forceinline__ void put_scales(lds_u8* sbuf) const {
        if constexpr (C::SC != kNoScale) {
#pragma unroll
            for (int i = 0; i < C::NS; ++i) {
                const int e = t + C::NT * i;
                if (C::NS * C::NT == C::TL + C::TR || e < C::TL + C::TR) {
                    if constexpr (C::SC == kE8M0 && !C::kScaleBytes)
                        reinterpret_cast<lds_f32*>(sbuf)[e] = e8m0_value(sv[i]);
                    else if constexpr (C::kScaleBytes)
                        sbuf[e / 64 * 64 + e % 16 * 4 + e / 16 % 4] = static_cast<uint8_t>(sv[i]);
                    else
                        reinterpret_cast<lds_u32*>(sbuf)[e] = sv[i];
                }
            }
        }
    }
};

// Bytes of k at or behind `valid` cleared in one 16-byte piece.
__device__ __forceinline__ i32x4 keep_bytes(i32x4 v, int valid) {
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        const int n = valid - 4 * d;  // bytes kept of this word
        const uint32_t m = n >= 4 ? 0xffffffffu : n <= 0 ? 0u : (1u << (8 * n)) - 1u;
        v[d] = static_cast<int>(static_cast<uint32_t>(v[d]) & m);
    }
    return v;
}

// One 16-row fragment at byte `at` of the tile (chunk l/16; the other half
// is 64 bytes away by XOR).  rem: bytes of k left, for the last stage.
template <bool TAIL>
__device__ __forceinline__ i32x8 read_frag(const lds_u8* tile, uint32_t at, uint32_t off, int g, int rem) {
    i32x4 lo = *reinterpret_cast<const lds_i32x4*>(tile + at + off);
    i32x4 hi = *reinterpret_cast<const lds_i32x4*>(tile + (at ^ 64u) + off);
    if constexpr (TAIL) {
        lo = keep_bytes(lo, rem - 16 * g);
        hi = keep_bytes(hi, rem - 16 * g - 64);
    }
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}

template <class C, int OL, int OR>
__device__ __forceinline__ f32x4 mfma_e8m0(i32x8 r, i32x8 l, f32x4 c, int sr, int sl) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(r, l, c, C::RT, C::LT, OR, sr, OL, sl);
}

template <class C, int OL>
__device__ __forceinline__ f32x4 mfma_e8m0_r(i32x8 r, i32x8 l, f32x4 c, int sr, int sl, int o) {
    switch (o) {
        case 0: return mfma_e8m0<C, OL, 0>(r, l, c, sr, sl);
        case 1: return mfma_e8m0<C, OL, 1>(r, l, c, sr, sl);
        case 2: return mfma_e8m0<C, OL, 2>(r, l, c, sr, sl);
        default: return mfma_e8m0<C, OL, 3>(r, l, c, sr, sl);
    }
}

// The stage's two 16x16x32 products of two-byte fragments.
template <int ELEM>
__device__ __forceinline__ f32x4 mfma_pair(i32x8 r, i32x8 l, f32x4 acc) {
    const i32x4 r0 = __builtin_shufflevector(r, r, 0, 1, 2, 3), r1 = __builtin_shufflevector(r, r, 4, 5, 6, 7);
    const i32x4 l0 = __builtin_shufflevector(l, l, 0, 1, 2, 3), l1 = __builtin_shufflevector(l, l, 4, 5, 6, 7);
    if constexpr (ELEM == kF16) {
        acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, r0), __builtin_bit_cast(f16x8, l0), acc, 0, 0, 0);
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, r1), __builtin_bit_cast(f16x8, l1), acc, 0, 0, 0);
    } else {
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, r0), __builtin_bit_cast(bf16x8, l0), acc, 0, 0, 0);
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, r1), __builtin_bit_cast(bf16x8, l1), acc, 0, 0, 0);
    }
}

// Adds one stage's product of block fragments: r rows (registers), l columns
// (lanes).  ol, orr: bytes of the scale words (constants after unrolling).
template <class C>
__device__ __forceinline__ void mma_stage(f32x4& acc, i32x8 r, i32x8 l, int sr, int sl, int orr, int ol, f32x4 fr,
                                          float fl) {
    if constexpr (C::ELEM == kF8) {
        if constexpr (C::SC == kE8M0) {
            switch (ol) {
                case 0: acc = mfma_e8m0_r<C, 0>(r, l, acc, sr, sl, orr); break;
                case 1: acc = mfma_e8m0_r<C, 1>(r, l, acc, sr, sl, orr); break;
                case 2: acc = mfma_e8m0_r<C, 2>(r, l, acc, sr, sl, orr); break;
                default: acc = mfma_e8m0_r<C, 3>(r, l, acc, sr, sl, orr); break;
            }
        } else {
            const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
            const f32x4 p = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(r, l, zero, C::RT, C::LT, 0, 0, 0, 0);
            if constexpr (C::SC == kF32Square) {
                const float s = fr[0] * fl;
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[i] = __builtin_fmaf(p[i], s, acc[i]);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[i] = __builtin_fmaf(p[i], fr[i] * fl, acc[i]);
            }
        }
    } else {
        acc = mfma_pair<C::ELEM>(r, l, acc);
    }
}

// This lane's scales of a stage: l(x), r(y) are words whose byte lsel(x),
// rsel(y) is block x's or y's E8M0 scale; lf, rf and rvec are fp32.
template <class C>
struct LaneScales {
    static constexpr bool kWords = C::SC == kE8M0 && !C::kPutScales;
    static constexpr bool kKept = C::ELEM == kF8;  // widened operands read their words when they convert
    int lw[!kKept ? 1 : kWords ? C::BL : (C::BL + 3) / 4], rw[!kKept ? 1 : kWords ? C::BR : (C::BR + 3) / 4];
    float lf[C::BL], rf;
    __device__ __forceinline__ int l(int x) const { return lw[kWords ? x : x / 4]; }
    __device__ __forceinline__ int r(int y) const { return rw[kWords ? y : y / 4]; }
    static __device__ __forceinline__ constexpr int sel(int b) { return kWords ? 0 : b % 4; }
    // skew: kWords: where the scales of this lane's rows begin, modulo 4
    // (ScaleSkew); s: the stage.
    template <class K>
    __device__ __forceinline__ void read(const lds_u8* sbuf, int wl, int wr, int lane, const K& skew, int s) {
        const int l16 = lane % 16;
        const lds_u32* w = reinterpret_cast<const lds_u32*>(sbuf);
        if constexpr (C::kScaleBytes) {
#pragma unroll
            for (int i = 0; i < (C::BL + 3) / 4; ++i) lw[i] = static_cast<int>(w[(wl * C::BL / 4 + i) * 16 + l16]);
#pragma unroll
            for (int i = 0; i < (C::BR + 3) / 4; ++i)
                rw[i] = static_cast<int>(w[(C::TL / 64 + wr * C::BR / 4 + i) * 16 + l16]);
        } else if constexpr (C::SC == kE8M0) {
            if constexpr (kKept) {
#pragma unroll
                for (int x = 0; x < C::BL; ++x) lw[x] = static_cast<int>(skew.word(sbuf, (wl * C::BL + x) * 16 + l16, x, s));
#pragma unroll
                for (int y = 0; y < C::BR; ++y)
                    rw[y] = static_cast<int>(skew.word(sbuf, C::TL + (wr * C::BR + y) * 16 + l16, C::BL + y, s));
            }
        } else if constexpr (C::SC != kNoScale) {
            const lds_f32* f = reinterpret_cast<const lds_f32*>(sbuf);
#pragma unroll
            for (int x = 0; x < C::BL; ++x) lf[x] = f[(wl * C::BL + x) * 16 + l16];
            if constexpr (C::SC == kF32Square) rf = f[C::TL + wr * C::BR * 16];
        }
    }
    __device__ __forceinline__ f32x4 rvec(const lds_u8* sbuf, int wr, int y, int lane) const {
        if constexpr (C::SC == kF32Rows)
            return *reinterpret_cast<const lds_f32x4*>(sbuf + 4 * (C::TL + (wr * C::BR + y) * 16 + 4 * (lane / 16)));
        else if constexpr (C::SC == kF32Square)
            return f32x4{rf, rf, rf, rf};
        else
            return f32x4{0.f, 0.f, 0.f, 0.f};
    }
};

struct NoSkew {
    __device__ __forceinline__ uint32_t word(const lds_u8*, int, int, int) const { return 0; }
};
template <class C>
struct ScaleSkew {
    static_assert(C::BL + C::BR <= 16, "two bits a block");
    uint32_t at = 0;
    // The word of a tile row whose low byte is its E8M0 scale of stage s.
    __device__ __forceinline__ uint32_t word(const lds_u8* sbuf, int row, int block, int s) const {
        return reinterpret_cast<const lds_u32*>(sbuf)[row] >> (8 * (((at >> (2 * block)) + s) & 3u));
    }
    __device__ __forceinline__ void init(const Operand& L, const Operand& R, int64_t l0, int64_t r0, int wl, int wr, int l16) {
        auto begin = [](const Operand& o, int64_t row) {
            row = row < o.rows ? row : o.rows - 1;
            return static_cast<uint32_t>(reinterpret_cast<uintptr_t>(o.scale) + (row >> o.scale_shift) * o.scale_ld) & 3u;
        };
#pragma unroll
        for (int x = 0; x < C::BL; ++x) at |= begin(L, l0 + (wl * C::BL + x) * 16 + l16) << (2 * x);
#pragma unroll
        for (int y = 0; y < C::BR; ++y) at |= begin(R, r0 + (wr * C::BR + y) * 16 + l16) << (2 * (C::BL + y));
    }
};

// 16 one-byte values times a power of two as two bf16 fragments.
template <bool E5M2>
__device__ __forceinline__ i32x8 widen(i32x4 v, float scale) {
    i32x8 o;
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        if constexpr (E5M2) {
            o[2 * d] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(v[d], scale, false));
            o[2 * d + 1] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(v[d], scale, true));
        } else {
            o[2 * d] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[d], scale, false));
            o[2 * d + 1] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[d], scale, true));
        }
    }
    return o;
}

// One stage of widened operands, 64 values of k at a time.  E8M0 scales go
// into the conversions; fp32 scales multiply each half's product.
template <class C, bool TAIL, class K>
__device__ __forceinline__ void stage_products_wide(f32x4 (&acc)[C::BL][C::BR], const lds_u8* buf, const lds_u8* sbuf,
                                                    const LaneScales<C>& sc, uint32_t lat, uint32_t rat, int wl, int wr,
                                                    int lane, int rem, const K& skew, int s) {
    const int g = lane / 16;
    auto scale = [&](int tile_row, int block) {  // E8M0, of this lane's row of a block
        if constexpr (C::SC != kE8M0)
            return 1.f;
        else if constexpr (C::kPutScales)
            return reinterpret_cast<const lds_f32*>(sbuf)[tile_row + lane % 16];
        else
            return e8m0_value(skew.word(sbuf, tile_row + lane % 16, block, s));
    };
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        __builtin_amdgcn_sched_barrier(0);  // both halves' fragments at once would not fit in registers
        auto piece = [&](const lds_u8* tile, uint32_t at, uint32_t off) {
            i32x4 v = *reinterpret_cast<const lds_i32x4*>(tile + (at ^ (64u * j)) + off);
            if constexpr (TAIL) v = keep_bytes(v, rem - 16 * g - 64 * j);
            return v;
        };
        i32x8 lf[C::BL];
#pragma unroll
        for (int x = 0; x < C::BL; ++x)
            lf[x] = widen<C::LT == 1>(piece(buf, lat, 2048 * x), scale((wl * C::BL + x) * 16, x));
#pragma unroll
        for (int y = 0; y < C::BR; ++y) {
            const i32x8 rf = widen<C::RT == 1>(piece(buf + C::TL * 128, rat, 2048 * y),
                                               scale(C::TL + (wr * C::BR + y) * 16, C::BL + y));
            const f32x4 rs = sc.rvec(sbuf, wr, y, lane);
#pragma unroll
            for (int x = 0; x < C::BL; ++x) {
                f32x4 p = C::SC == kE8M0 ? acc[x][y] : f32x4{0.f, 0.f, 0.f, 0.f};
                p = mfma_pair<kBf16>(rf, lf[x], p);
                if constexpr (C::SC == kE8M0) {
                    acc[x][y] = p;
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[x][y][i] = __builtin_fmaf(p[i], rs[i] * sc.lf[x], acc[x][y][i]);
                }
            }
        }
    }
}

template <class C, bool TAIL, class K>
__device__ __forceinline__ void stage_products(f32x4 (&acc)[C::BL][C::BR], const lds_u8* buf, const lds_u8* sbuf,
                                               const LaneScales<C>& sc, uint32_t lat, uint32_t rat, int wl, int wr, int lane,
                                               int rem, const K& skew, int s) {
    if constexpr (C::ELEM == kF8Wide) {
        stage_products_wide<C, TAIL>(acc, buf, sbuf, sc, lat, rat, wl, wr, lane, rem, skew, s);
    } else {
        const int g = lane / 16;
        i32x8 lf[C::BL];
#pragma unroll
        for (int x = 0; x < C::BL; ++x) lf[x] = read_frag<TAIL>(buf, lat, 2048 * x, g, rem);
#pragma unroll
        for (int y = 0; y < C::BR; ++y) {
            const i32x8 rf = read_frag<TAIL>(buf + C::TL * 128, rat, 2048 * y, g, rem);
            const f32x4 rs = sc.rvec(sbuf, wr, y, lane);
#pragma unroll
            for (int x = 0; x < C::BL; ++x)
                mma_stage<C>(acc[x][y], rf, lf[x], sc.r(y), sc.l(x), sc.sel(y), sc.sel(x), rs, sc.lf[x]);
        }
    }
}

// Main loop of the 4 x 2 waves of 4 x 8 blocks: each wave alternates between a
// slot of memory work and a slot of products, all slots ended by a barrier,
// and the second half of the waves (one of each SIMD's two) runs one slot
// behind, so that a SIMD's matrix unit works for one wave while the other
// reads its next fragments.  A stage is four quadrants of 2 x 4 blocks in the
// order (L0 R0) (L1 R0) (L1 R1) (L0 R1), each with one new operand half, which
// the slot before it reads: L0, L1, R1, and R0 of the next stage.
// At 8192 x 8192 x 4096 with one-byte operands 217 us (2.54 PFLOP/s); against
// all waves in step (reads, then products, one barrier a stage) 221 to 236, in
// turn on one box, before the loads were split (below).  No better: the halves in the order L0 R0, L0 R1, L1 R1, L1 R0 (12, 8, 4 and 0
// reads a slot), a pipelined loop with one barrier a stage whose reads run one
// quadrant ahead (267 us, 21 registers spilled), and L's loads two slots before
// R's (269 us).  What bounds it, from builds that leave one thing out (of one
// at 229 us): without the loads into LDS 161 us, with half of them 175, without
// waiting for them 219, without the fragment reads 222, without barriers 209.  So it is the rate
// of the loads into LDS, 64 KiB a stage and workgroup; the matrix units are
// busy 53% of the cycles at 2.1 GHz.
// Slots of stage s, counted from the leading waves' first (8 s; the second half
// is one later):
//   8s + 4: R1 is read, and then no fragment of stage s is missing; each wave
//           waits for its reads and for its loads of stage s + 1;
//   8s + 6: stage s + 1 has landed for all (the last wait is in slot 8s + 5)
//           and its R0 is read; stage s + 2's loads may overwrite stage s.
//           Two-byte operands issue all of them here; one-byte operands R's
//           here and L's in slot 8s + 8 (8192 x 8192 x 4096: 213 us, all at
//           once 220; cross entropy with gradients at 4096 x 65536 x 4096 in
//           bf16 8.22 ms so split, 7.63 at once; both in turn on one box).
template <class C>
__device__ __forceinline__ void pingpong(f32x4 (&acc)[C::BL][C::BR], Stager<C>& st, lds_u8* lds, lds_u8* sbufs, uint32_t lat,
                                         uint32_t rat, int wl, int wr, int lane, int64_t full, int64_t stages) {
    static_assert(C::BL == 4 && C::BR == 8 && C::WL * C::WR == 8, "two waves a SIMD");
    const bool lag = st.wave >= 4;
    auto slot = [] {
        __builtin_amdgcn_sched_barrier(0);
        wg_barrier();
        __builtin_amdgcn_sched_barrier(0);
    };
    const int g = lane / 16;
    i32x8 l[2][2], r[2][4];
    auto read_r = [&](const lds_u8* buf, int h) {
#pragma unroll
        for (int y = 0; y < 4; ++y) r[h][y] = read_frag<false>(buf + C::TL * 128, rat, 2048 * (4 * h + y), g, 128);
    };
    auto read_l = [&](const lds_u8* buf, int h) {
#pragma unroll
        for (int x = 0; x < 2; ++x) l[h][x] = read_frag<false>(buf, lat, 2048 * (2 * h + x), g, 128);
    };
    // stage 0 has landed; stage 1 (or stage 0 again) goes to the other buffer
    constexpr bool kSplit = C::ELEM == kF8;
    if constexpr (!kSplit) st.issue_l(stages > 1 ? 1 : 0, lds + C::kBuf);
    st.issue_r(stages > 1 ? 1 : 0, lds + C::kBuf);
    read_r(lds, 0);
    if (lag) slot();
    // No branch inside: across one the compiler moves products out of their
    // slots.  Loads behind the last stage fetch it again into a buffer that is
    // not read any more.
    for (int64_t s = 0; s < full; ++s) {
        lds_u8* buf = lds + (s & 1) * C::kBuf;
        const lds_u8* sbuf = sbufs + (s & 1) * C::kScaleBuf;
        LaneScales<C> sc;
        auto products = [&](int lh, int rh) {
            __builtin_amdgcn_s_setprio(1);
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const f32x4 rs = sc.rvec(sbuf, wr, 4 * rh + y, lane);
#pragma unroll
                for (int x = 0; x < 2; ++x)
                    mma_stage<C>(acc[2 * lh + x][4 * rh + y], r[rh][y], l[lh][x], sc.r(4 * rh + y), sc.l(0), y, 2 * lh + x, rs,
                                 sc.lf[2 * lh + x]);
            }
            __builtin_amdgcn_s_setprio(0);
        };
        if constexpr (kSplit) st.issue_l(s + 1 < stages ? s + 1 : s, lds + ((s + 1) & 1) * C::kBuf);
        sc.read(sbuf, wl, wr, lane, NoSkew{}, 0);
        read_l(buf, 0);
        slot();
        products(0, 0);
        slot();
        read_l(buf, 1);
        slot();
        products(1, 0);
        slot();
        read_r(buf, 1);
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        st.put_scales(sbufs + ((s + 1) & 1) * C::kScaleBuf);
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        slot();
        products(1, 1);
        slot();
        read_r(lds + ((s + 1) & 1) * C::kBuf, 0);
        if constexpr (!kSplit) st.issue_l(s + 2 < stages ? s + 2 : stages - 1, buf);
        st.issue_r(s + 2 < stages ? s + 2 : stages - 1, buf);
        slot();
        products(0, 1);
        slot();
    }
    if (!lag) slot();
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

// The whole product of one tile: rows l0 .. of L against rows r0 .. of R over
// kbytes bytes of k.  Sums run over k in increasing order.
template <class C>
__device__ __forceinline__ void tile_product(f32x4 (&acc)[C::BL][C::BR], const Operand& L, const Operand& R, int64_t l0,
                                             int64_t r0, int64_t kbytes, lds_u8* lds) {
    const int t = threadIdx.x, lane = t % 64;
    const int wave = __builtin_amdgcn_readfirstlane(t / 64);
    const int wl = wave / C::WR, wr = wave % C::WR;
#pragma unroll
    for (int x = 0; x < C::BL; ++x)
#pragma unroll
        for (int y = 0; y < C::BR; ++y) acc[x][y] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int64_t stages = (kbytes + 127) / 128, full = kbytes / 128;
    if (stages == 0) return;
    Stager<C> st;
    st.init(L, R, l0, r0, kbytes, t);
    const int l16 = lane % 16, rem = static_cast<int>(kbytes - full * 128);
    const uint32_t at = l16 * 128 + 16 * ((lane / 16) ^ ((l16 >> 1) & 7));
    const uint32_t lat = wl * C::BL * 2048 + at, rat = wr * C::BR * 2048 + at;
    LaneScales<C> sc;
    if constexpr (C::kSlots) {
        lds_u8* sbufs = lds + 2 * C::kBuf;
        st.issue(0, lds);
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        st.put_scales(sbufs);
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        wg_barrier();
        if (full > 0) pingpong<C>(acc, st, lds, sbufs, lat, rat, wl, wr, lane, full, stages);
        if (full < stages) {
            const lds_u8* sbuf = sbufs + (full & 1) * C::kScaleBuf;
            sc.read(sbuf, wl, wr, lane, NoSkew{}, 0);
            stage_products<C, true>(acc, lds + (full & 1) * C::kBuf, sbuf, sc, lat, rat, wl, wr, lane, rem, NoSkew{}, 0);
        }
    } else {
        // NBUF - 1 stages in flight: with few workgroups a stage's products are
        // short against the way of its loads.  A wave waits for its own loads
        // of stage s (those of the NBUF - 2 behind it may still be on their
        // way; every stage is kLoads of them, the ones behind the last stage
        // fetch it again), the barrier covers the other waves', and with it all
        // are done with stage s - 1, whose buffer the next loads take.
        constexpr int N = C::NBUF;
        auto issue = [&](int64_t s, lds_u8* buf) {
            if constexpr (C::kPutScales)
                st.issue(s, buf);
            else
                st.issue_deep(s, buf);
        };
        std::conditional_t<LaneScales<C>::kWords, ScaleSkew<C>, NoSkew> skew;
        if constexpr (LaneScales<C>::kWords) skew.init(L, R, l0, r0, wl, wr, l16);
#pragma unroll
        for (int i = 0; i < N - 1; ++i) issue(i < stages ? i : stages - 1, lds + i * C::kStage);
        int at_buf = 0;
        auto begin = [&](int64_t s) {
            asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"((N - 2) * Stager<C>::kLoads) : "memory");
            if constexpr (C::kPutScales) {
                st.put_scales(lds + at_buf * C::kStage + C::kBuf);
                asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            }
            wg_barrier();
            const int prev = at_buf == 0 ? N - 1 : at_buf - 1;
            issue(s + N - 1 < stages ? s + N - 1 : stages - 1, lds + prev * C::kStage);
            const lds_u8* buf = lds + at_buf * C::kStage;
            at_buf = at_buf + 1 == N ? 0 : at_buf + 1;
            sc.read(buf + C::kBuf, wl, wr, lane, skew, static_cast<int>(s));
            return buf;
        };
        for (int64_t s = 0; s < full; ++s) {
            const lds_u8* buf = begin(s);
            stage_products<C, false>(acc, buf, buf + C::kBuf, sc, lat, rat, wl, wr, lane, 128, skew, static_cast<int>(s));
        }
        if (full < stages) {
            const lds_u8* buf = begin(full);
            stage_products<C, true>(acc, buf, buf + C::kBuf, sc, lat, rat, wl, wr, lane, rem, skew, static_cast<int>(full));
        }
    }
    // every wave is done reading, and nothing is on its way into LDS, before
    // the epilogue reuses the buffers
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    wg_barrier();
}

// A wave's accumulators out to C [rows][ldc] of CT, rows i0 .., columns j0 ..
// of the wave, through its LDS slice: 16 rows at a time, so that stores are
// whole runs of C rows.  vec: ldc and the pointer allow 16-byte stores (the
// columns then end on a whole piece too).  f(value) is applied first.
template <class C, class CT, class F>
__device__ __forceinline__ void store_tile(const f32x4 (&acc)[C::BL][C::BR], lds_f32* slice, CT* __restrict__ c,
                                           int64_t ldc, int64_t i0, int64_t j0, int64_t rows, int64_t cols, bool vec,
                                           int lane, F f) {
    constexpr int W = 16 * C::BR, P = C::kPitch, V = 16 / sizeof(CT), PER = W / V;  // V elements a piece
    typedef CT ctv __attribute__((ext_vector_type(V)));
    const int g = lane / 16, l16 = lane % 16;
#pragma unroll
    for (int x = 0; x < C::BL; ++x) {
#pragma unroll
        for (int y = 0; y < C::BR; ++y) *reinterpret_cast<lds_f32x4*>(slice + l16 * P + 16 * y + 4 * g) = acc[x][y];
        const int64_t ib = i0 + 16 * x;
        if (ib >= rows) continue;
        if (vec) {
            static_assert(16 * PER % 64 == 0, "whole pieces per wave");
#pragma unroll
            for (int q = 0; q < 16 * PER / 64; ++q) {
                const int u = 64 * q + lane, r = u / PER, cc = V * (u % PER);
                ctv o;
#pragma unroll
                for (int h = 0; h < V / 4; ++h) {
                    const f32x4 v = *reinterpret_cast<const lds_f32x4*>(slice + r * P + cc + 4 * h);
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[4 * h + i] = static_cast<CT>(f(v[i]));
                }
                if (ib + r < rows && j0 + cc < cols)
                    __builtin_nontemporal_store(o, reinterpret_cast<ctv*>(c + (ib + r) * ldc + j0 + cc));
            }
        } else {
            for (int u = lane; u < 16 * W; u += 64) {
                const int r = u / W, cc = u % W;
                if (ib + r < rows && j0 + cc < cols) c[(ib + r) * ldc + j0 + cc] = static_cast<CT>(f(slice[r * P + cc]));
            }
        }
    }
}

}  // namespace mma
}  // namespace swz
