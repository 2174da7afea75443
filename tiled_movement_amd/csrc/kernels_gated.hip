// A gated feed-forward block's two projections, its activation and the
// product, y = act(g) u with g = x Wg^T and u = x Wu^T, and its gradients
//   dg = dy u act'(g),  du = dy act(g),
//   dx = dg Wg + du Wu,  dWg = dg^T x,  dWu = du^T x.
//
// Forward: a tile of x against rows of both weights in turn (Gated in
// mma_core.h), so that a lane holds g and u of its places; y is their only
// rounding.  On request g and u are kept in fp32 for the backward pass (8 bytes a
// place against 4 k operations to make them again).
//
// Backward: dg and du are made once, in x's type (as two terms for small
// products: gated_two_terms(); in fp16 times a power of two where they leave its
// range: held_times()), by elements from the kept g
// and u or by the forward products over again.  The products that follow sum over
// f (dx) and over the rows of x (dW), where the weights, dg, du and x
// lie across the sum; they are read as they lie, by transposing reads out of
// LDS (Across in mma_core.h), so nothing is transposed through memory.
#include "activation.h"
#include "launch_ffn.h"
#include "mma_core.h"

namespace swz {
namespace {

using namespace mma;

// A configuration's half along R: what the epilogue of a Gated one stores.
template <class C>
struct HalfR {
    static constexpr int BL = C::BL, BR = C::BR / 2, kPitch = 16 * BR + 4;
};

template <int ELEM>
using Value = std::conditional_t<ELEM == kBf16, __bf16, _Float16>;

// The order of a grid's tiles, `times` times over (parts, products): TileMap's,
// which keeps neighbours on one XCD, unless all workgroups could run at once and
// it would give some XCD more than its 32 compute units (700 x 1024 from 4000, 24
// tiles in 10 parts: on four of the eight XCDs, 70 us, 46 in plain order).
struct Order {
    TileMap map;
    bool plain;
    static Order make(int64_t f, int64_t s, int64_t times) {
        const TileMap m = TileMap::make(f, s);
        return Order{m, f * s * times <= 256 && static_cast<int64_t>(m.grid / 8) * times > 32};
    }
    unsigned grid() const { return plain ? map.f * map.s : map.grid; }
    __device__ __forceinline__ bool at(uint32_t id, int64_t* fi, int64_t* si) const {
        if (!plain) return map.at(id, fi, si);
        *fi = id % map.f;
        *si = id / map.f;
        return true;
    }
};

// What a workgroup of a tile kernel works on.
template <class C>
struct Place {
    int lane, g, l16, wave, wl, wr;
    int64_t i0, f0;  // the wave's first row and feature
    __device__ __forceinline__ Place(int64_t tm, int64_t tn) {
        const int t = threadIdx.x;
        lane = t % 64, g = lane / 16, l16 = lane % 16;
        wave = __builtin_amdgcn_readfirstlane(t / 64), wl = wave / C::WR, wr = wave % C::WR;
        i0 = tm * C::TL + wl * C::BL * 16;
        f0 = tn * (C::TR / 2) + wr * C::BR * 8;
    }
};

// store_tile for rows of any length at any element: whole pieces as they lie
// (stores of 16 bytes need no alignment here; those of 333 x 1000 to 2777 by
// elements took 4 us more), a row's last one by elements.  Rows of whole aligned
// pieces, and the 256 x 256 tiles, whose registers are full, go by store_tile.
template <class H, class CT>
__device__ __forceinline__ void store_rows(const f32x4 (&acc)[H::BL][H::BR], lds_f32* slice, CT* __restrict__ c, int64_t i0,
                                           int64_t j0, int64_t rows, int64_t cols, int lane) {
    constexpr int W = 16 * H::BR, P = H::kPitch, V = 16 / sizeof(CT), PER = W / V;
    typedef CT ctv __attribute__((ext_vector_type(V), aligned(sizeof(CT))));
    static_assert(16 * PER % 64 == 0, "whole pieces per wave");
    const int g = lane / 16, l16 = lane % 16;
#pragma unroll
    for (int x = 0; x < H::BL; ++x) {
#pragma unroll
        for (int y = 0; y < H::BR; ++y) *reinterpret_cast<lds_f32x4*>(slice + l16 * P + 16 * y + 4 * g) = acc[x][y];
        const int64_t ib = i0 + 16 * x;
        if (ib >= rows) continue;
#pragma unroll
        for (int q = 0; q < 16 * PER / 64; ++q) {
            const int u = 64 * q + lane, r = u / PER, cc = V * (u % PER);
            ctv o;
#pragma unroll
            for (int h = 0; h < V / 4; ++h) {
                const f32x4 v = *reinterpret_cast<const lds_f32x4*>(slice + r * P + cc + 4 * h);
#pragma unroll
                for (int i = 0; i < 4; ++i) o[4 * h + i] = static_cast<CT>(v[i]);
            }
            if (ib + r >= rows) continue;
            CT* to = c + (ib + r) * cols + j0 + cc;
            if (j0 + cc + V <= cols) {
                __builtin_nontemporal_store(o, reinterpret_cast<ctv*>(to));
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (j0 + cc + i < cols) to[i] = o[i];
            }
        }
    }
}

template <class C, int ACT>
__global__ __launch_bounds__(C::NT) void k_gated(Operand X, PairOperand W, int64_t kbytes, Value<C::ELEM>* __restrict__ y,
                                                 float* __restrict__ pre, int vec, Order order) {
    __shared__ i32x4 lds_v[C::kLds / 16];
    lds_u8* lds = (lds_u8*)(reinterpret_cast<uint8_t*>(lds_v));
    int64_t tm, tn;
    if (!order.at(blockIdx.x, &tm, &tn)) return;
    f32x4 acc[C::BL][C::BR];
    tile_product<C>(acc, X, W, tm * C::TL, tn * (C::TR / 2), kbytes, lds);
    const Place<C> at(tm, tn);
    using H = HalfR<C>;
    lds_f32* slice = (lds_f32*)(lds + at.wave * C::kSlice);
    const int64_t n = X.rows, f = W.rows;
    f32x4 part[H::BL][H::BR];
    auto store = [&](auto* to) {
        if (C::kSlots || vec)
            store_tile<H>(part, slice, to, f, at.i0, at.f0, n, f, vec, at.lane, [](float v) { return v; });
        else
            store_rows<H>(part, slice, to, at.i0, at.f0, n, f, at.lane);
    };
    if (pre) {
#pragma unroll
        for (int p = 0; p < 2; ++p) {
#pragma unroll
            for (int x = 0; x < H::BL; ++x)
#pragma unroll
                for (int b = 0; b < H::BR; ++b) part[x][b] = acc[x][p * H::BR + b];
            store(pre + p * n * f);
        }
    }
#pragma unroll
    for (int x = 0; x < H::BL; ++x)
#pragma unroll
        for (int b = 0; b < H::BR; ++b) {
            __builtin_amdgcn_sched_barrier(0);  // all places' activations at once would not fit in registers
#pragma unroll
            for (int i = 0; i < 4; ++i) part[x][b][i] = act::both<ACT, false>(acc[x][b][i]).x * acc[x][H::BR + b][i];
        }
    store(y);
}

template <bool DERIV>
__device__ __forceinline__ float2 act_of(int act, float z) {
    if (act == SWZ_ACT_GELU) return act::both<SWZ_ACT_GELU, DERIV>(z);
    if (act == SWZ_ACT_GELU_TANH) return act::both<SWZ_ACT_GELU_TANH, DERIV>(z);
    return act::both<SWZ_ACT_SILU, DERIV>(z);
}

// Up to 16 MB rows of x: the time is the weights' bytes.  A workgroup owns 16
// features of both weights and all rows; its waves split k into runs of blocks of
// 64, and operands go from memory straight into matrix fragments (a fragment is 16
// rows of 64 bytes, and the weights are used once): no barrier and no LDS
// between a load and its product, so that all loads of U blocks are in flight
// together.  The waves' sums are joined through LDS in their order.
constexpr int kFewWaves = 8;
template <int ELEM, int MB>
__global__ __launch_bounds__(64 * kFewWaves) void k_gated_few(const uint8_t* __restrict__ x, const uint8_t* __restrict__ wg,
                                                              const uint8_t* __restrict__ wu, int64_t n, int64_t f, int64_t k, int act,
                                                              Value<ELEM>* __restrict__ y, float* __restrict__ pre) {
    __shared__ f32x4 red[2][kFewWaves][64];
    const int t = threadIdx.x, lane = t % 64, g = lane / 16, l16 = lane % 16;
    const int wave = __builtin_amdgcn_readfirstlane(t / 64);
    const int64_t f0 = static_cast<int64_t>(blockIdx.x) * 16;
    // this lane's rows; the last stands in for rows behind it, whose results are not stored
    const int64_t rw = f0 + l16 < f ? f0 + l16 : f - 1;
    const uint8_t* row[2 + MB] = {wg + 2 * rw * k, wu + 2 * rw * k};
#pragma unroll
    for (int a = 0; a < MB; ++a) row[2 + a] = x + 2 * (16 * a + l16 < n ? 16 * a + l16 : n - 1) * k;
    const int64_t kbytes = 2 * k, full = kbytes / 128, blocks = (kbytes + 127) / 128;
    f32x4 acc[2][MB];
#pragma unroll
    for (int o = 0; o < 2; ++o)
#pragma unroll
        for (int a = 0; a < MB; ++a) acc[o][a] = f32x4{0.f, 0.f, 0.f, 0.f};
    // UN blocks from b on, all loads before the products
    auto step = [&](int64_t b, auto un, bool lo_in, bool hi_in) {
        constexpr int UN = decltype(un)::value;
        i32x8 v[UN][2 + MB];
#pragma unroll
        for (int u = 0; u < UN; ++u)
#pragma unroll
            for (int o = 0; o < 2 + MB; ++o) {
                const uint8_t* p = row[o] + (b + u) * 128;
                i32x4 lo = *reinterpret_cast<const i32x4*>(p + (lo_in ? 16 * g : 0));
                i32x4 hi = *reinterpret_cast<const i32x4*>(p + (hi_in ? 16 * g + 64 : 0));
                v[u][o] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
            }
#pragma unroll
        for (int u = 0; u < UN; ++u) {
            if (UN == 1 && !(lo_in && hi_in)) {  // behind k nothing counts
#pragma unroll
                for (int o = 0; o < 2 + MB; ++o)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (!lo_in) v[u][o][i] = 0;
                        if (!hi_in) v[u][o][4 + i] = 0;
                    }
            }
#pragma unroll
            for (int a = 0; a < MB; ++a)
#pragma unroll
                for (int o = 0; o < 2; ++o) acc[o][a] = mfma_pair<ELEM>(v[u][o], v[u][2 + a], acc[o][a]);
        }
    };
    constexpr int U = 2;
    const int64_t end = blocks * (wave + 1) / kFewWaves, whole = end < full ? end : full;
    int64_t b = blocks * wave / kFewWaves;
    for (; b + U <= whole; b += U) step(b, std::integral_constant<int, U>{}, true, true);
    if constexpr (U > 1)
        for (; b < whole; ++b) step(b, std::integral_constant<int, 1>{}, true, true);
    // k is a multiple of 8: 16-byte chunks are inside or outside as a whole
    if (b < end) step(b, std::integral_constant<int, 1>{}, b * 128 + 16 * g < kbytes, b * 128 + 16 * g + 64 < kbytes);

    // lane (g, l16): row l16 of x, features 4g .. 4g+3
#pragma unroll
    for (int a = 0; a < MB; ++a) {
        if (a > 0) __syncthreads();
#pragma unroll
        for (int o = 0; o < 2; ++o) red[o][wave][l16 * 4 + g] = acc[o][a];
        __syncthreads();
        const int64_t i = 16 * a + t / 16, j = f0 + t % 16;
        if (t >= 256 || i >= n || j >= f) continue;
        const float* rf = reinterpret_cast<const float*>(red);
        float z[2] = {0.f, 0.f};
#pragma unroll
        for (int w = 0; w < kFewWaves; ++w) z[0] += rf[w * 256 + t], z[1] += rf[(kFewWaves + w) * 256 + t];
        if (pre) pre[i * f + j] = z[0], pre[(n + i) * f + j] = z[1];
        y[i * f + j] = static_cast<Value<ELEM>>(act_of<false>(act, z[0]).x * z[1]);
    }
}

// What a call holds dg (du) times, from the bits of its largest finite magnitude m.
// 1 in bf16, whose range is fp32's.  In fp16 1 where m is 2^-4 to below 65520:
// it rounds to a number, and what is 2^-10 of it still has all its digits; else
// the power of two that brings m to 2^14 .. 2^15, but 2^64 at most (a sum of 2^22
// products of 2^16 by what lies below 2^-64 rounds to zero in fp16).
template <int ELEM>
__device__ __forceinline__ float held_times(uint32_t bits) {
    if constexpr (ELEM != kF16) return 1.f;
    if (bits == 0 || (bits >= 0x3d800000u && bits < 0x477ff000u)) return 1.f;
    const int e = 141 - static_cast<int>(bits >> 23);
    return __uint_as_float(static_cast<uint32_t>(127 + (e < 64 ? e : 64)) << 23);
}
// 1 / v of a power of two.
__device__ __forceinline__ float inverse(float v) { return __uint_as_float((254u << 23) - __float_as_uint(v)); }
// The larger of a and |v|'s bits, if v is finite.
__device__ __forceinline__ uint32_t larger(uint32_t a, float v) {
    const uint32_t b = magnitude_bits(v);
    return b < 0x7f800000u && b > a ? b : a;
}
__device__ __forceinline__ uint32_t wave_most(uint32_t m) {
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const uint32_t o = __shfl_xor(m, d);
        m = o > m ? o : m;
    }
    return m;
}
// m is known when all of dg is made, so a call makes dg and du at 1 and leaves
// their workgroups' magnitudes in slots, up to kGatedSlots of dg, then of du.  A
// second launch joins them, leaves the result (`most`) for the products, and makes
// both again where 1 is not what they are to be held times.
// Gradients of 333 x 1000 to 2777 41.5 us without this, 46 with it; one slot for all
// workgroups, raised by atomics, 51.  tmp: 2 NT / 64 words of LDS.
template <int NT>
__device__ __forceinline__ uint2 join_slots(const uint32_t* __restrict__ slots, int count, lds_u32* tmp) {
    uint32_t m[2] = {0, 0};
    for (int i = threadIdx.x; i < count; i += NT) {
#pragma unroll
        for (int o = 0; o < 2; ++o) {
            const uint32_t v = slots[o * kGatedSlots + i];
            m[o] = v > m[o] ? v : m[o];
        }
    }
#pragma unroll
    for (int o = 0; o < 2; ++o) {
        m[o] = wave_most(m[o]);
        if (threadIdx.x % 64 == 0) tmp[o * (NT / 64) + threadIdx.x / 64] = m[o];
    }
    __syncthreads();
#pragma unroll
    for (int o = 0; o < 2; ++o)
#pragma unroll
        for (int w = 0; w < NT / 64; ++w) {
            const uint32_t v = tmp[o * (NT / 64) + w];
            m[o] = v > m[o] ? v : m[o];
        }
    __syncthreads();
    return make_uint2(m[0], m[1]);
}
// A workgroup's magnitudes into its slots.  Workgroups beyond kGatedSlots share
// them, zeroed before.
template <int NT>
__device__ __forceinline__ void leave_slots(uint32_t mg, uint32_t mu, uint32_t* slots, uint32_t id, bool shared, lds_u32* tmp) {
    mg = wave_most(mg), mu = wave_most(mu);
    if (threadIdx.x % 64 == 0) tmp[threadIdx.x / 64] = mg, tmp[NT / 64 + threadIdx.x / 64] = mu;
    __syncthreads();
    if (threadIdx.x >= 2) return;
    uint32_t m = 0;
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) {
        const uint32_t v = tmp[threadIdx.x * (NT / 64) + w];
        m = v > m ? v : m;
    }
    uint32_t* slot = slots + threadIdx.x * kGatedSlots + id % kGatedSlots;
    if (shared)
        raise_slot(slot, m);
    else
        *slot = m;
}
__global__ __launch_bounds__(256) void k_clear_slots(uint32_t* slots) { slots[blockIdx.x * 256 + threadIdx.x] = 0; }

// What is left of v when it is rounded to CT; nothing where that has no end.
template <class CT>
__device__ __forceinline__ float rest_of(float v) {
    const float r = static_cast<float>(static_cast<CT>(v));
    return __builtin_isfinite(r) ? v - r : 0.f;
}

// dg and du ([n][ldz], x's type) from the kept g and u, eight places a thread;
// rows by blockIdx.y.  Bound by the bytes.  Rows of an f that is no multiple of 8
// begin at any element: their pieces are loaded as they lie, and the last one by
// elements.  joined: 0 in the first launch, else its workgroups.
template <int ELEM, int ACT>
__global__ __launch_bounds__(256) void k_gated_dz(const float* __restrict__ pre, const Value<ELEM>* __restrict__ dy, int64_t n,
                                                  int64_t f, int64_t ldz, Value<ELEM>* __restrict__ dg,
                                                  Value<ELEM>* __restrict__ du, int64_t rest, uint32_t* __restrict__ slots,
                                                  int joined, uint32_t* __restrict__ most) {
    using CT = Value<ELEM>;
    __shared__ uint32_t tmp[8];
    typedef float f32x8 __attribute__((ext_vector_type(8), aligned(4)));
    typedef CT ct8 __attribute__((ext_vector_type(8)));
    typedef CT ct8_any __attribute__((ext_vector_type(8), aligned(2)));
    const int64_t j = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 8;
    const int here = f - j < 8 ? static_cast<int>(f - j) : 8;
    float tg = 1.f, tu = 1.f;
    if (ELEM == kF16 && joined) {
        const uint2 m = join_slots<256>(slots, joined, (lds_u32*)tmp);
        if (blockIdx.x + blockIdx.y + threadIdx.x == 0) most[0] = m.x, most[1] = m.y;
        tg = held_times<ELEM>(m.x), tu = held_times<ELEM>(m.y);
        if (tg == 1.f && tu == 1.f) return;
    }
    uint32_t mg = 0, mu = 0;
    for (int64_t i = j < f ? blockIdx.y : n; i < n; i += gridDim.y) {
        f32x8 g = 0.f, u = 0.f;
        ct8_any d = 0;
        if (here == 8) {
            g = *reinterpret_cast<const f32x8*>(pre + i * f + j);
            u = *reinterpret_cast<const f32x8*>(pre + (n + i) * f + j);
            d = *reinterpret_cast<const ct8_any*>(dy + i * f + j);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < here) g[e] = pre[i * f + j + e], u[e] = pre[(n + i) * f + j + e], d[e] = dy[i * f + j + e];
        }
        ct8 zg, zu, rg, ru;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float2 a = act::both<ACT, true>(g[e]);
            const float de = static_cast<float>(d[e]);
            float vg = de * u[e] * a.y, vu = de * a.x;
            if constexpr (ELEM == kF16) {
                mg = larger(mg, vg), mu = larger(mu, vu);
                vg *= tg, vu *= tu;
            }
            zg[e] = static_cast<CT>(vg), zu[e] = static_cast<CT>(vu);
            rg[e] = static_cast<CT>(rest_of<CT>(vg)), ru[e] = static_cast<CT>(rest_of<CT>(vu));
        }
        // whole pieces: ldz is a multiple of 8, and what lies behind f is not used
        *reinterpret_cast<ct8*>(dg + i * ldz + j) = zg;
        *reinterpret_cast<ct8*>(du + i * ldz + j) = zu;
        if (rest) {
            *reinterpret_cast<ct8*>(dg + rest + i * ldz + j) = rg;
            *reinterpret_cast<ct8*>(du + rest + i * ldz + j) = ru;
        }
    }
    if constexpr (ELEM == kF16) {
        if (joined) return;
        leave_slots<256>(mg, mu, slots, blockIdx.y * gridDim.x + blockIdx.x, false, (lds_u32*)tmp);
    }
}

// The same with g and u made again.
template <class C, int ACT>
__global__ __launch_bounds__(C::NT) void k_gated_again_dz(Operand X, PairOperand W, int64_t kbytes,
                                                          const Value<C::ELEM>* __restrict__ dy, int64_t ldz,
                                                          Value<C::ELEM>* __restrict__ dg, Value<C::ELEM>* __restrict__ du,
                                                          int64_t rest, uint32_t* __restrict__ slots, int joined,
                                                          uint32_t* __restrict__ most, Order order) {
    __shared__ i32x4 lds_v[C::kLds / 16];
    lds_u8* lds = (lds_u8*)(reinterpret_cast<uint8_t*>(lds_v));
    int64_t tm, tn;
    if (!order.at(blockIdx.x, &tm, &tn)) {
        if (C::ELEM == kF16 && !joined && gridDim.x <= kGatedSlots && threadIdx.x < 2) slots[threadIdx.x * kGatedSlots + blockIdx.x] = 0;
        return;
    }
    float tg = 1.f, tu = 1.f;
    if (C::ELEM == kF16 && joined) {
        const uint2 m = join_slots<C::NT>(slots, joined, (lds_u32*)lds);
        if (tm + tn + threadIdx.x == 0) most[0] = m.x, most[1] = m.y;
        tg = held_times<C::ELEM>(m.x), tu = held_times<C::ELEM>(m.y);
        if (tg == 1.f && tu == 1.f) return;
    }
    f32x4 acc[C::BL][C::BR];
    tile_product<C>(acc, X, W, tm * C::TL, tn * (C::TR / 2), kbytes, lds);
    const Place<C> at(tm, tn);
    using H = HalfR<C>;
    lds_f32* slice = (lds_f32*)(lds + at.wave * C::kSlice);
    const int64_t n = X.rows, f = W.rows;
    f32x4 z[H::BL][H::BR];
    uint32_t mg = 0, mu = 0;
#pragma unroll
    for (int x = 0; x < H::BL; ++x)
#pragma unroll
        for (int b = 0; b < H::BR; ++b) {
            __builtin_amdgcn_sched_barrier(0);  // all places' activations at once would not fit in registers
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t r = at.i0 + 16 * x + at.l16, j = at.f0 + 16 * b + 4 * at.g + i;
                const float d = r < n && j < f ? static_cast<float>(dy[r * f + j]) : 0.f;
                const float2 a = act::both<ACT, true>(acc[x][b][i]);
                float vg = d * acc[x][H::BR + b][i] * a.y, vu = d * a.x;
                if constexpr (C::ELEM == kF16) {
                    if (r < n && j < f) mg = larger(mg, vg), mu = larger(mu, vu);
                    vg *= tg, vu *= tu;
                }
                z[x][b][i] = vg;
                acc[x][b][i] = vu;
            }
        }
    if constexpr (C::ELEM == kF16) {
        constexpr int kSlices = C::WL * C::WR * C::kSlice;  // the words are behind what the waves store from
        static_assert(kSlices + 8 * C::NT / 64 <= C::kLds, "fits");
        if (!joined) leave_slots<C::NT>(mg, mu, slots, blockIdx.x, gridDim.x > kGatedSlots, (lds_u32*)(lds + kSlices));
    }
    // whole pieces: ldz is a multiple of 8, and what lies behind f is not used
    const auto same = [](float v) { return v; };
    const auto left = [](float v) { return rest_of<Value<C::ELEM>>(v); };
    store_tile<H>(z, slice, dg, ldz, at.i0, at.f0, n, ldz, true, at.lane, same);
    if (rest) store_tile<H>(z, slice, dg + rest, ldz, at.i0, at.f0, n, ldz, true, at.lane, left);
#pragma unroll
    for (int x = 0; x < H::BL; ++x)
#pragma unroll
        for (int b = 0; b < H::BR; ++b) z[x][b] = acc[x][b];
    store_tile<H>(z, slice, du, ldz, at.i0, at.f0, n, ldz, true, at.lane, same);
    if (rest) store_tile<H>(z, slice, du + rest, ldz, at.i0, at.f0, n, ldz, true, at.lane, left);
}

// Sums of part `part` of a product in fp32, or its result; in fp16 times `by`.
template <class C, class CT>
__device__ __forceinline__ void store_result(const f32x4 (&acc)[C::BL][C::BR], lds_u8* lds, CT* c, float* sums, int64_t part,
                                             int64_t rows, int64_t cols, int64_t tm, int64_t tn, float by) {
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int64_t i0 = tm * C::TL + wave / C::WR * C::BL * 16, j0 = tn * C::TR + wave % C::WR * C::BR * 16;
    lds_f32* slice = (lds_f32*)(lds + wave * C::kSlice);
    const auto out = [&](float v) { return C::ELEM == kF16 ? v * by : v; };
    if (sums)
        store_tile<C>(acc, slice, sums + part * rows * cols, cols, i0, j0, rows, cols, true, lane, out);
    else
        store_tile<C>(acc, slice, c, cols, i0, j0, rows, cols, true, lane, out);
}

// The columns [k0, k0 + kb) of bytes of the summed axis that part `part` has.
__device__ __forceinline__ int64_t part_of(int64_t kbytes, int64_t part_bytes, int64_t part, int64_t* k0) {
    *k0 = part * part_bytes;
    const int64_t kb = kbytes - *k0 < part_bytes ? kbytes - *k0 : part_bytes;
    if (kb <= 0) *k0 = 0;
    return kb > 0 ? kb : 0;
}

// dx = dg Wg + du Wu, or the part blockIdx.y of its sum over f; TWO: over the
// rests of dg and du too, `rest` bytes on.  (As a loop in the large tiles it
// costs registers: dx of 4096 x 4096 from 8192 484 us, 563.)  In fp16 the sum is
// held times what du is; dg's part is brought there where dg is held otherwise.
template <class C, bool TWO>
__global__ __launch_bounds__(C::NT) void k_gated_dx(Operand Zg, Operand Zu, Operand Wg, Operand Wu, int64_t kbytes,
                                                    int64_t part_bytes, int64_t rest, Value<C::ELEM>* __restrict__ dx,
                                                    float* __restrict__ sums, const uint32_t* __restrict__ most, Order order) {
    __shared__ i32x4 lds_v[C::kLds / 16];
    lds_u8* lds = (lds_u8*)(reinterpret_cast<uint8_t*>(lds_v));
    int64_t tm, tn, k0;
    if (!order.at(blockIdx.x, &tm, &tn)) return;
    const int64_t kb = part_of(kbytes, part_bytes, blockIdx.y, &k0);
    Zg.data += k0, Zu.data += k0, Wg.data += k0 / 2 * Wg.ld, Wu.data += k0 / 2 * Wu.ld;
    f32x4 acc[C::BL][C::BR];
    const auto bring = [&](int from, int to) {
        if constexpr (C::ELEM == kF16) {
            const float tf = held_times<C::ELEM>(most[from]), tt = held_times<C::ELEM>(most[to]);
            if (tf == tt) return;
#pragma unroll
            for (int x = 0; x < C::BL; ++x)
#pragma unroll
                for (int y = 0; y < C::BR; ++y) acc[x][y] *= tt * inverse(tf);
        }
    };
    tile_product<C>(acc, Zg, Wg, tm * C::TL, tn * C::TR, kb, lds);
    bring(0, 1);
    tile_product<C>(acc, Zu, Wu, tm * C::TL, tn * C::TR, kb, lds, true);
    if (TWO) {
        Zg.data += rest, Zu.data += rest;
        bring(1, 0);
        tile_product<C>(acc, Zg, Wg, tm * C::TL, tn * C::TR, kb, lds, true);
        bring(0, 1);
        tile_product<C>(acc, Zu, Wu, tm * C::TL, tn * C::TR, kb, lds, true);
    }
    store_result<C>(acc, lds, dx, sums, blockIdx.y, Zg.rows, Wg.rows, tm, tn, inverse(C::ELEM == kF16 ? held_times<C::ELEM>(most[1]) : 1.f));
}

// dWg = dg^T x (blockIdx.z 0) and dWu = du^T x (1), or the part blockIdx.y of
// their sums over x's rows; TWO: of the rests of dg and du too.
template <class C, bool TWO>
__global__ __launch_bounds__(C::NT) void k_gated_dw(Operand Zg, Operand Zu, Operand X, int64_t kbytes, int64_t part_bytes,
                                                    int64_t rest, Value<C::ELEM>* __restrict__ dwg,
                                                    Value<C::ELEM>* __restrict__ dwu, float* __restrict__ sums,
                                                    const uint32_t* __restrict__ most, Order order) {
    __shared__ i32x4 lds_v[C::kLds / 16];
    lds_u8* lds = (lds_u8*)(reinterpret_cast<uint8_t*>(lds_v));
    int64_t tm, tn, k0;
    if (!order.at(blockIdx.x, &tn, &tm)) return;
    const int64_t kb = part_of(kbytes, part_bytes, blockIdx.y, &k0);
    const bool up = blockIdx.z != 0 || !dwg;
    Operand Z = up ? Zu : Zg;
    Z.data += k0 / 2 * Z.ld, X.data += k0 / 2 * X.ld;
    f32x4 acc[C::BL][C::BR];
    tile_product<C>(acc, Z, X, tm * C::TL, tn * C::TR, kb, lds);
    if (TWO) {
        Z.data += rest;
        tile_product<C>(acc, Z, X, tm * C::TL, tn * C::TR, kb, lds, true);
    }
    store_result<C>(acc, lds, up ? dwu : dwg, sums, blockIdx.z * gridDim.y + blockIdx.y, Z.rows, X.rows, tm, tn,
                    inverse(C::ELEM == kF16 ? held_times<C::ELEM>(most[up ? 1 : 0]) : 1.f));
}

// A result from the fp32 sums of its parts, eight values a thread, the loads of
// kAhead parts in flight together (dx of 333 x 1000 from 2777, 10 parts: 30.6 us
// one at a time, 28.0 by 3, 28.6 by 4, 28.3 by 8; 16 x 1032 from 1000: 14.3, 12.8,
// 13.2, 14.4).
constexpr int kAhead = 3;
template <class CT>
__global__ __launch_bounds__(256) void k_join_parts(const float* __restrict__ sums, int parts, int64_t pieces, CT* __restrict__ out) {
    typedef CT ct8 __attribute__((ext_vector_type(8)));
    const int64_t u = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (u >= pieces) return;
    const f32x4* p = reinterpret_cast<const f32x4*>(sums) + 2 * u;
    f32x4 s0 = p[0], s1 = p[1];
    int i = 1;
    for (; i + kAhead <= parts; i += kAhead) {
        f32x4 v[kAhead][2];
#pragma unroll
        for (int h = 0; h < kAhead; ++h) v[h][0] = p[2 * (i + h) * pieces], v[h][1] = p[2 * (i + h) * pieces + 1];
        asm volatile("" ::: "memory");  // all loads before the first sum
#pragma unroll
        for (int h = 0; h < kAhead; ++h) s0 += v[h][0], s1 += v[h][1];
    }
    for (; i < parts; ++i) s0 += p[2 * i * pieces], s1 += p[2 * i * pieces + 1];
    ct8 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = static_cast<CT>(s0[i]), o[4 + i] = static_cast<CT>(s1[i]);
    reinterpret_cast<ct8*>(out)[u] = o;
}

__global__ __launch_bounds__(256) void k_zero(i32x4* __restrict__ p, int64_t pieces) {
    const int64_t step = static_cast<int64_t>(gridDim.x) * 256;
    for (int64_t u = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; u < pieces; u += step) p[u] = i32x4{0, 0, 0, 0};
}

// Tiles of GatedTile and of ProductTile.
template <int ELEM> using T256x256 = Config<ELEM, 0, 0, kNoScale, 4, 2, 4, 8>;
template <int ELEM> using T128x256 = Config<ELEM, 0, 0, kNoScale, 2, 4, 4, 4>;
template <int ELEM> using T64x256 = Config<ELEM, 0, 0, kNoScale, 2, 4, 2, 4>;
template <int ELEM> using T128x128 = Config<ELEM, 0, 0, kNoScale, 2, 2, 4, 4>;
template <int ELEM> using T64x64 = Config<ELEM, 0, 0, kNoScale, 2, 2, 2, 2>;
template <int ELEM> using T128x64 = Config<ELEM, 0, 0, kNoScale, 4, 1, 2, 4>;
template <int ELEM> using T64x64Slim = Config<ELEM, 0, 0, kNoScale, 4, 1, 1, 4>;  // a wave has both halves of its features

template <int ELEM, class F>
hipError_t by_gated_tile(GatedTile tile, F f) {
    switch (tile) {
        case GatedTile::k64x32: return f(Gated<T64x64Slim<ELEM>>{});
        case GatedTile::k128x32: return f(Gated<T128x64<ELEM>>{});
        case GatedTile::k64x128: return f(Gated<T64x256<ELEM>>{});
        case GatedTile::k128x128: return f(Gated<T128x256<ELEM>>{});
        default: return f(Gated<T256x256<ELEM>>{});
    }
}
// f of a tile and whether the product is over two terms.
template <int ELEM, bool L, bool R, class F>
hipError_t by_product_tile(ProductTile tile, bool two, F f) {
    if (two)
        return tile == ProductTile::k64x64 ? f(Across<T64x64<ELEM>, L, R>{}, std::true_type{})
                                           : f(Across<T128x256<ELEM>, L, R>{}, std::true_type{});
    switch (tile) {
        case ProductTile::k64x64: return f(Across<T64x64<ELEM>, L, R>{}, std::false_type{});
        case ProductTile::k64x256: return f(Across<T64x256<ELEM>, L, R>{}, std::false_type{});
        case ProductTile::k128x128: return f(Across<T128x128<ELEM>, L, R>{}, std::false_type{});
        case ProductTile::k128x256: return f(Across<T128x256<ELEM>, L, R>{}, std::false_type{});
        default: return f(Across<T256x256<ELEM>, L, R>{}, std::false_type{});
    }
}
template <class F>
hipError_t by_act(int act, F f) {
    if (act == SWZ_ACT_GELU) return f(std::integral_constant<int, SWZ_ACT_GELU>{});
    if (act == SWZ_ACT_GELU_TANH) return f(std::integral_constant<int, SWZ_ACT_GELU_TANH>{});
    return f(std::integral_constant<int, SWZ_ACT_SILU>{});
}

unsigned blocks_of(int64_t n, int64_t per) { return static_cast<unsigned>((n + per - 1) / per); }

Operand operand(const void* p, int64_t ld, int64_t rows) {
    return Operand{static_cast<const uint8_t*>(p), 2 * ld, rows, nullptr, 0, 0};
}
PairOperand pair_operand(const GatedJob& j) {
    PairOperand w;
    static_cast<Operand&>(w) = operand(j.wg, j.k, j.f);
    w.second = static_cast<const uint8_t*>(j.wu);
    return w;
}

template <int ELEM>
hipError_t forward(const GatedJob& j, hipStream_t stream) {
    using CT = Value<ELEM>;
    if (gated_few(j.n, j.f, j.k)) {
        const auto few = [&](auto mb) {
            hipLaunchKernelGGL((k_gated_few<ELEM, decltype(mb)::value>), dim3(blocks_of(j.f, 16)), dim3(64 * kFewWaves), 0, stream,
                               static_cast<const uint8_t*>(j.x), static_cast<const uint8_t*>(j.wg), static_cast<const uint8_t*>(j.wu),
                               j.n, j.f, j.k, j.act, static_cast<CT*>(j.y), j.pre);
            return hipGetLastError();
        };
        return j.n <= 16 ? few(std::integral_constant<int, 1>{}) : few(std::integral_constant<int, 2>{});
    }
    return by_act(j.act, [&](auto a) {
        constexpr int ACT = decltype(a)::value;
        return by_gated_tile<ELEM>(gated_tile(j.n, j.f), [&](auto cfg) {
            using C = decltype(cfg);
            const int64_t tm = (j.n + C::TL - 1) / C::TL, tn = (j.f + C::TR / 2 - 1) / (C::TR / 2);
            const Order order = Order::make(tm, tn, 1);
            const bool vec = j.f % 8 == 0 && (reinterpret_cast<uintptr_t>(j.y) | reinterpret_cast<uintptr_t>(j.pre)) % 16 == 0;
            hipLaunchKernelGGL((k_gated<C, ACT>), dim3(order.grid()), dim3(C::NT), 0, stream, operand(j.x, j.k, j.n), pair_operand(j),
                               2 * j.k, static_cast<CT*>(j.y), j.pre, vec, order);
            return hipGetLastError();
        });
    });
}

template <int ELEM>
hipError_t backward(const GatedJob& j, const GatedPlan& p, hipStream_t stream) {
    using CT = Value<ELEM>;
    auto* ws = static_cast<uint8_t*>(j.ws);
    auto* dg = reinterpret_cast<CT*>(ws + p.dg);
    auto* du = reinterpret_cast<CT*>(ws + p.du);
    auto* sums = reinterpret_cast<float*>(ws + p.sums);
    auto* most = reinterpret_cast<uint32_t*>(ws + p.slots);
    auto* slots = most + 64;
    const int64_t ldz = p.ldz;
    // joined: the first launch's slots, which it leaves here
    const auto make_dz = [&](int* joined) {
        return by_act(j.act, [&](auto a) {
            constexpr int ACT = decltype(a)::value;
            if (j.pre) {
                const int64_t across = blocks_of(j.f, 2048), down = ELEM == kF16 ? kGatedSlots / across : 16384;
                const dim3 grid(static_cast<unsigned>(across), static_cast<unsigned>(j.n < down ? j.n : down));
                hipLaunchKernelGGL((k_gated_dz<ELEM, ACT>), grid, dim3(256), 0, stream, j.pre, static_cast<const CT*>(j.dy), j.n, j.f,
                                   ldz, dg, du, p.rest / 2, slots, *joined, most);
                *joined = static_cast<int>(grid.x * grid.y);
                return hipGetLastError();
            }
            return by_gated_tile<ELEM>(gated_tile(j.n, j.f), [&](auto cfg) {
                using C = decltype(cfg);
                const int64_t tm = (j.n + C::TL - 1) / C::TL, tn = (j.f + C::TR / 2 - 1) / (C::TR / 2);
                const Order order = Order::make(tm, tn, 1);
                if (ELEM == kF16 && !*joined && order.grid() > kGatedSlots)
                    hipLaunchKernelGGL(k_clear_slots, dim3(2 * kGatedSlots / 256), dim3(256), 0, stream, slots);
                hipLaunchKernelGGL((k_gated_again_dz<C, ACT>), dim3(order.grid()), dim3(C::NT), 0, stream, operand(j.x, j.k, j.n),
                                   pair_operand(j), 2 * j.k, static_cast<const CT*>(j.dy), ldz, dg, du, p.rest / 2, slots, *joined,
                                   most, order);
                *joined = order.grid() < kGatedSlots ? static_cast<int>(order.grid()) : kGatedSlots;
                return hipGetLastError();
            });
        });
    };
    int joined = 0;
    hipError_t e = make_dz(&joined);
    if (e == hipSuccess && ELEM == kF16) e = make_dz(&joined);
    const auto join = [&](const float* from, int64_t parts, int64_t values, void* out) {
        hipLaunchKernelGGL(k_join_parts<CT>, dim3(blocks_of(values / 8, 256)), dim3(256), 0, stream, from, static_cast<int>(parts),
                           values / 8, static_cast<CT*>(out));
        return hipGetLastError();
    };
    if (e == hipSuccess && j.dx) {
        e = by_product_tile<ELEM, false, true>(p.dx_tile, p.rest != 0, [&](auto cfg, auto two) {
            using C = decltype(cfg);
            const int64_t tm = (j.n + C::TL - 1) / C::TL, tn = (j.k + C::TR - 1) / C::TR;
            const Order order = Order::make(tm, tn, p.dx_parts);
            const int64_t part_bytes = ((2 * j.f + 127) / 128 + p.dx_parts - 1) / p.dx_parts * 128;
            hipLaunchKernelGGL((k_gated_dx<C, decltype(two)::value>), dim3(order.grid(), static_cast<unsigned>(p.dx_parts)), dim3(C::NT), 0, stream,
                               operand(dg, ldz, j.n), operand(du, ldz, j.n), operand(j.wg, j.k, j.k), operand(j.wu, j.k, j.k),
                               2 * j.f, part_bytes, p.rest, static_cast<CT*>(j.dx), p.dx_parts > 1 ? sums : nullptr, most,
                               order);
            return hipGetLastError();
        });
        if (e == hipSuccess && p.dx_parts > 1) e = join(sums, p.dx_parts, j.n * j.k, j.dx);
    }
    if (e == hipSuccess && (j.dwg || j.dwu)) {
        const unsigned both = j.dwg && j.dwu ? 2 : 1;
        e = by_product_tile<ELEM, true, true>(p.dw_tile, p.rest != 0, [&](auto cfg, auto two) {
            using C = decltype(cfg);
            const int64_t tm = (j.f + C::TL - 1) / C::TL, tn = (j.k + C::TR - 1) / C::TR;
            const Order order = Order::make(tn, tm, p.dw_parts * both);
            const int64_t part_bytes = ((2 * j.n + 127) / 128 + p.dw_parts - 1) / p.dw_parts * 128;
            hipLaunchKernelGGL((k_gated_dw<C, decltype(two)::value>), dim3(order.grid(), static_cast<unsigned>(p.dw_parts), both), dim3(C::NT), 0, stream,
                               operand(dg, ldz, j.f), operand(du, ldz, j.f), operand(j.x, j.k, j.k), 2 * j.n, part_bytes,
                               p.rest, static_cast<CT*>(j.dwg), static_cast<CT*>(j.dwu), p.dw_parts > 1 ? sums : nullptr, most,
                               order);
            return hipGetLastError();
        });
        if (p.dw_parts > 1) {
            const int64_t one = p.dw_parts * j.f * j.k;
            if (e == hipSuccess && j.dwg) e = join(sums, p.dw_parts, j.f * j.k, j.dwg);
            if (e == hipSuccess && j.dwu) e = join(sums + (both == 2 ? one : 0), p.dw_parts, j.f * j.k, j.dwu);
        }
    }
    return e;
}

}  // namespace

hipError_t launch_gated(const GatedJob& j, hipStream_t stream) {
    return j.bf16 ? forward<kBf16>(j, stream) : forward<kF16>(j, stream);
}

hipError_t launch_gated_grad(const GatedJob& j, const GatedPlan& p, hipStream_t stream) {
    if (j.n == 0) {  // no rows: the weights' gradients are zero (f k is a multiple of 8)
        for (void* w : {j.dwg, j.dwu}) {
            const int64_t pieces = j.f * j.k / 8;
            if (w)
                hipLaunchKernelGGL(k_zero, dim3(pieces > 65536 * 256 ? 65536u : blocks_of(pieces, 256)), dim3(256), 0, stream,
                                   static_cast<i32x4*>(w), pieces);
        }
        return hipGetLastError();
    }
    return j.bf16 ? backward<kBf16>(j, p, stream) : backward<kF16>(j, p, stream);
}

}  // namespace swz
