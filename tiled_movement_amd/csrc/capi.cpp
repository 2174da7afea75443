// C ABI of libswz.so: argument checks, parameter choice and launches.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstring>
#include <map>
#include <memory>
#include <mutex>
#include <new>
#include <tuple>

#include "chooser.h"
#include "launch.h"
#include "launch_ffn.h"
#include "swz.h"

#define SWZ_API extern "C" __attribute__((visibility("default")))

namespace {

using swz::KindInfo;

bool mul_ok(int64_t a, int64_t b, int64_t* out) {
    if (a < 0 || b < 0) return false;
    if (a != 0 && b > INT64_MAX / a) return false;
    *out = a * b;
    return true;
}

bool overlaps(const void* a, int64_t abytes, const void* b, int64_t bbytes) {
    const auto pa = reinterpret_cast<uintptr_t>(a), pb = reinterpret_cast<uintptr_t>(b);
    return pa < pb + static_cast<uintptr_t>(bbytes) && pb < pa + static_cast<uintptr_t>(abytes);
}

// Whether n elements of esz bytes make a whole number of 16-byte vectors;
// unsigned, so that a huge n wraps instead of overflowing (16 divides 2^64).
bool pitch16(int64_t n, int32_t esz) { return (static_cast<uint64_t>(n) * static_cast<uint64_t>(esz)) % 16 == 0; }

int hip_status(hipError_t e) { return e == hipSuccess ? SWZ_OK : SWZ_EHIP; }

// Elements from the first of [rows][ld] to the last of `cols` used in the last
// row: what lies behind them is not the matrix's (it may be a part of a wider
// one).  False where rows ld leaves 64 bits; ld >= cols >= 0.
bool span_elems(int64_t rows, int64_t cols, int64_t ld, int64_t* elems) {
    if (!mul_ok(rows, ld, elems)) return false;
    *elems = rows && cols ? *elems - ld + cols : 0;
    return true;
}

// Bytes of an 8-bit operand [rows][ld], of which rows use `used` bytes, and of
// its scales.
bool f8_operand_bytes(int64_t rows, int64_t cols, int64_t used, int64_t ld, bool square, int32_t scale_type, int64_t* data,
                      int64_t* scales) {
    int64_t n;
    const int64_t srows = square ? rows / 128 + (rows % 128 != 0) : rows, scols = cols / 128 + (cols % 128 != 0);
    return span_elems(rows, used, ld, data) && mul_ok(srows, scols, &n) &&
           mul_ok(n, scale_type == SWZ_SCALE_F32 ? 4 : 1, scales);
}

// Sizes of an output-layer loss that the kernels' grids and offsets take:
// SWZ_OK, or why not.  Each size is bounded by itself before it enters a
// product.
int check_loss_sizes(int64_t n, int64_t v, int64_t k, int32_t top) {
    if (n < 0 || v < 1 || k < 8 || k % 8 || top < 1) return SWZ_EINVAL;
    if (top > swz::kMaxTop || k >= swz::kMaxPitch / 2 || n >= swz::kMaxPitch / 2 - 8 || v >= int64_t(1) << 31) return SWZ_EUNSUPPORTED;
    if ((n / 256 + 1) * (v / 256 + 1) > int64_t(1) << 22) return SWZ_EUNSUPPORTED;  // tiles of one launch
    return SWZ_OK;
}

int64_t up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

// Words of a piece, at most `most` (a multiple of 256), for row_tiles tiles of
// rows.  A piece's products run in rounds of 256 tiles, one a compute unit, and
// a started round takes as long as a full one: pieces of whole rounds with a
// short last one (of smaller tiles' cost, at least a third of a round a piece)
// against pieces alike in size, whichever has fewer.
int64_t piece_words(int64_t v, int64_t most, int64_t row_tiles) {
    auto cost = [&](int64_t piece) {
        double rounds = 0;
        for (int64_t at = 0; at < v; at += piece) {
            const int64_t words = v - at < piece ? v - at : piece;
            rounds += static_cast<double>(((words + 255) / 256 * row_tiles + 255) / 256) + 0.34;
        }
        return rounds;
    };
    const int64_t pieces = (v + most - 1) / most;
    const int64_t alike = up((v + pieces - 1) / pieces, 256);
    int64_t whole = 256;  // word tiles of whole rounds
    for (int64_t t = row_tiles; whole > 1 && t % 2 == 0; t /= 2) whole /= 2;
    const int64_t aligned = most / (256 * whole) * (256 * whole);
    return aligned > 0 && aligned < alike * pieces && v / aligned < 4096 && cost(aligned) < cost(alike) ? aligned : alike;
}

// The gradient's workspace.  dz of a piece stays within 2^27 values (256 MiB)
// unless that leaves fewer than 8192 words.  Where
// dH has fewer tiles than the 256 compute units, its sum over a piece is split
// into parts (of at least 8 stages) with buffers of their own.
swz::LossPlan plan_loss(int64_t n, int64_t v, int64_t k, int32_t top) {
    swz::LossPlan p{};
    int64_t most = (int64_t(1) << 27) / (n ? n : 1) / 256 * 256;
    most = most < 8192 ? 8192 : most > 32768 ? 32768 : most;
    const int64_t tl = n <= 64 ? 64 : n <= 128 ? 128 : 256;
    p.piece = piece_words(v, most, (n + tl - 1) / tl + (n == 0));
    const int64_t tiles = ((n + tl - 1) / tl) * ((k + 255) / 256), stages = p.piece / 64;
    p.h_rows = tl;  // parts fill the card, so the largest tile that the rows fill
    p.parts = tiles >= 256 || tiles == 0 ? 1 : 256 / tiles;
    if (p.parts > 32) p.parts = 32;
    if (p.parts > stages / 8) p.parts = stages / 8 ? stages / 8 : 1;
    const int64_t ldn = up(n, 8);
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        const int64_t here = at;
        at += up(bytes, 256);
        return here;
    };
    p.slots = take(64);
    p.g = take(4 * n);
    p.weight = take(4 * n * top);
    p.dz = take(2 * n * p.piece);
    p.dzt = take(2 * p.piece * ldn);
    p.ht = take(2 * k * ldn);
    p.wt = take(2 * k * p.piece);
    p.sums = take(4 * p.parts * n * k);
    p.bytes = at;
    return p;
}

int64_t loss_forward_bytes(int64_t n, int64_t v) { return up(8 * n * ((v + 255) / 256), 256); }

struct Span {
    const void* p;
    int64_t bytes;
    uintptr_t align;
    bool written;
};

// NULL, alignment and overlap of a call's buffers: nothing written may
// overlap anything else.
bool spans_ok(const Span* s, int count) {
    for (int i = 0; i < count; ++i) {
        if (s[i].bytes == 0) continue;
        if (!s[i].p || reinterpret_cast<uintptr_t>(s[i].p) % s[i].align) return false;
        for (int j = 0; j < i; ++j)
            if ((s[i].written || s[j].written) && s[j].bytes && overlaps(s[i].p, s[i].bytes, s[j].p, s[j].bytes)) return false;
    }
    return true;
}

// Sizes of a gated block that the kernels' grids and offsets take.
int check_gated_sizes(int64_t n, int64_t f, int64_t k) {
    if (n < 0 || f < 1 || k < 8 || k % 8) return SWZ_EINVAL;
    for (const int64_t v : {n, f, k})
        if (v >= swz::kMaxPitch / 2 - 8) return SWZ_EUNSUPPORTED;
    const int64_t tiles = int64_t(1) << 21;
    if ((n / 256 + 1) * (f / 128 + 1) > tiles || (n / 256 + 1) * (k / 256 + 1) > tiles || (f / 256 + 1) * (k / 256 + 1) > tiles)
        return SWZ_EUNSUPPORTED;
    return SWZ_OK;
}

bool half_type(int32_t x_type) { return x_type == SWZ_X_BF16 || x_type == SWZ_X_F16; }
bool act_known(int32_t act) { return act == SWZ_ACT_SILU || act == SWZ_ACT_GELU || act == SWZ_ACT_GELU_TANH; }

// The tile of a gradient product and the parts that its sum over `stages` (of 64)
// is split into, with fp32 sums of their own: the cheapest by what was measured,
// in us: a workgroup's start and end, a stage, the parts' sums written and read at
// 4.5 TB/s, and a launch.  A compute unit holds one workgroup, two of 64 x 64.
// Gradients of 333 x 1000 to 2777 in 256 x 256 tiles alone 55 us, so 45; of 700 x 1024
// to 4000 102 and 68; from 4096 x 4096 to 8192 on it comes out at 256 x 256.
// pairs: of operands whose sums follow one another, each with a start of its own;
// two: over two terms, twice the pairs and stages, in 64 x 64 and 128 x 256 tiles
// only (dW of 8192 x 1024 from one row in 64 x 64 36 us, 18 so).
void plan_product(int64_t rows, int64_t cols, int64_t products, int64_t pairs, int64_t stages, bool two, swz::ProductTile* tile,
                  int64_t* parts) {
    static const struct {
        swz::ProductTile tile;
        int64_t rows, cols, at_once;
        double fixed, stage;
    } kinds[] = {{swz::ProductTile::k256x256, 256, 256, 256, 7.5, 1.5}, {swz::ProductTile::k128x256, 128, 256, 256, 5.3, 1.6},
                 {swz::ProductTile::k64x256, 64, 256, 256, 3.7, 1.3},   {swz::ProductTile::k128x128, 128, 128, 256, 4.6, 1.1},
                 {swz::ProductTile::k64x64, 64, 64, 512, 5.1, 0.7}};
    static const int64_t tries[] = {1, 2, 3, 4, 5, 6, 8, 10, 12, 16, 20, 24, 32};
    double best = -1;
    if (two) pairs *= 2, stages *= 2;
    for (const auto& k : kinds) {
        if (two && k.tile != swz::ProductTile::k64x64 && k.tile != swz::ProductTile::k128x256) continue;
        const int64_t tiles = (rows + k.rows - 1) / k.rows * ((cols + k.cols - 1) / k.cols) * products;
        for (const int64_t p : tries) {
            if (p > 1 && p > stages / 4) break;
            const double rounds = static_cast<double>((tiles * p + k.at_once - 1) / k.at_once);
            double us = rounds * (k.fixed + 5 * static_cast<double>(pairs - 1) + k.stage * static_cast<double>((stages + p - 1) / p));
            if (p > 1) us += 4 + static_cast<double>(p * rows) * static_cast<double>(cols * products) * 8 / 4.5e6;
            if (best >= 0 && us >= best) continue;
            best = us;
            *tile = k.tile;
            *parts = p;
        }
    }
}

swz::GatedPlan plan_gated(int64_t n, int64_t f, int64_t k) {
    swz::GatedPlan p{};
    p.ldz = up(f, 8);
    const bool two = swz::gated_two_terms(n, f, k);
    plan_product(n, k, 1, 2, 2 * ((f + 63) / 64), two, &p.dx_tile, &p.dx_parts);
    plan_product(f, k, 2, 1, (n + 63) / 64, two, &p.dw_tile, &p.dw_parts);
    const int64_t dx = p.dx_parts > 1 ? 4 * p.dx_parts * n * k : 0, dw = p.dw_parts > 1 ? 8 * p.dw_parts * f * k : 0;
    p.dg = 0;
    p.du = up(2 * n * p.ldz, 256);
    p.rest = two ? 2 * p.du : 0;
    p.slots = 2 * p.du + p.rest;
    p.sums = p.slots + (n > 0 ? 256 + 2 * 4 * swz::kGatedSlots : 0);
    p.bytes = p.sums + up(dx > dw ? dx : dw, 256);
    return p;
}

int check_w4_sizes(int64_t n, int64_t k, int32_t group) {
    if (n < 0 || k < 32 || k % 32 || (group != 32 && group != 64 && group != 128)) return SWZ_EINVAL;
    if (n > 0 && k >= (int64_t(1) << 34) / n) return SWZ_EUNSUPPORTED;
    return SWZ_OK;
}

int gemm_w4(const void* d_x, int32_t x_type, int32_t act, const swz::WeightsW4* w, int mats, int32_t group, void* d_c, int64_t m,
            int64_t n, int64_t k, void* stream) {
    if (!half_type(x_type) || m < 0) return SWZ_EINVAL;
    const int st = check_w4_sizes(n, k, group);
    if (st != SWZ_OK) return st;
    if (m >= int64_t(1) << 22 || k >= int64_t(1) << 22 || n >= int64_t(1) << 26) return SWZ_EUNSUPPORTED;
    if (m == 0 || n == 0) return SWZ_OK;
    const int64_t groups = (k + group - 1) / group;
    Span s[8] = {{d_x, 2 * m * k, 16, false}, {d_c, 2 * m * n, 2, true}};
    int count = 2;
    for (int i = 0; i < mats; ++i) {
        s[count++] = {w[i].q, n * (k / 2), 16, false};
        s[count++] = {w[i].scale, 2 * n * groups, 2, false};
        if (w[i].zero) s[count++] = {w[i].zero, n * groups, 1, false};
    }
    if (!spans_ok(s, count)) return SWZ_EINVAL;
    swz::GemmW4Job j{d_x, x_type == SWZ_X_BF16, m, n, k, group, mats == 2 ? act : -1, {w[0], w[mats - 1]}, d_c};
    return hip_status(swz::launch_gemm_w4(j, static_cast<hipStream_t>(stream)));
}

int norm_workspace(int32_t count, int64_t* bytes) {
    if (count < 0) return SWZ_EINVAL;
    if (count > 1 << 20) return SWZ_EUNSUPPORTED;
    *bytes = 8 * swz::kNormBlocks * ((count + swz::kNormTensors - 1) / swz::kNormTensors);
    return SWZ_OK;
}

// The list of a norm call: SWZ_OK, or why not.
int check_norm_list(const void* const* d_t, const int64_t* numel, const int32_t* type, int32_t count) {
    if (count > 0 && (!d_t || !numel || !type)) return SWZ_EINVAL;
    for (int32_t i = 0; i < count; ++i) {
        if (numel[i] < 0 || (type[i] != SWZ_X_BF16 && type[i] != SWZ_X_F16 && type[i] != SWZ_X_F32)) return SWZ_EINVAL;
        if (numel[i] >= int64_t(1) << 38) return SWZ_EUNSUPPORTED;
        if (numel[i] > 0 && (!d_t[i] || reinterpret_cast<uintptr_t>(d_t[i]) % (type[i] == SWZ_X_F32 ? 4 : 2))) return SWZ_EINVAL;
    }
    return SWZ_OK;
}

// Whether nothing written overlaps anything else, in time linear but for a sort.
bool apart(Span* s, int64_t count) {
    std::sort(s, s + count, [](const Span& a, const Span& b) {
        return reinterpret_cast<uintptr_t>(a.p) < reinterpret_cast<uintptr_t>(b.p);
    });
    uintptr_t read_end = 0, written_end = 0;  // of those before
    for (int64_t i = 0; i < count; ++i) {
        const auto at = reinterpret_cast<uintptr_t>(s[i].p);
        if (at < written_end || (s[i].written && at < read_end)) return false;
        uintptr_t& end = s[i].written ? written_end : read_end;
        end = std::max(end, at + static_cast<uintptr_t>(s[i].bytes));
    }
    return true;
}

int norm_call(const void* const* d_t, void* const* d_out, const int64_t* numel, const int32_t* type, int32_t count, bool clip,
              float max_norm, float* d_norm, void* d_ws, int64_t ws_bytes, void* stream) {
    int64_t need;
    int st = norm_workspace(count, &need);
    if (st == SWZ_OK) st = check_norm_list(d_t, numel, type, count);
    if (st != SWZ_OK) return st;
    if (!d_norm || reinterpret_cast<uintptr_t>(d_norm) % 4) return SWZ_EINVAL;
    if (std::all_of(numel, numel + count, [](int64_t n) { return n == 0; })) need = 0;  // nothing to sum
    if (need > 0 && (!d_ws || reinterpret_cast<uintptr_t>(d_ws) % 8 || ws_bytes < need)) return SWZ_EINVAL;
    const std::unique_ptr<Span[]> s(new (std::nothrow) Span[2 * static_cast<size_t>(count) + 2]);
    if (!s) return SWZ_EUNSUPPORTED;
    int64_t spans = 0;
    for (int32_t i = 0; i < count; ++i) {
        if (numel[i] == 0) continue;
        const int64_t es = type[i] == SWZ_X_F32 ? 4 : 2, bytes = es * numel[i];
        const void* out = clip && d_out ? d_out[i] : d_t[i];
        if (!out || reinterpret_cast<uintptr_t>(out) % static_cast<uintptr_t>(es)) return SWZ_EINVAL;
        s[spans++] = {out, bytes, 1, clip};
        if (out != d_t[i]) s[spans++] = {d_t[i], bytes, 1, false};
    }
    s[spans++] = {d_norm, clip ? 8 : 4, 1, true};
    if (need > 0) s[spans++] = {d_ws, need, 1, true};
    if (!apart(s.get(), spans)) return SWZ_EINVAL;
    const swz::NormJob j{d_t, d_out, numel, type, count, clip, max_norm, d_norm, static_cast<double*>(d_ws)};
    return hip_status(swz::launch_norm(j, static_cast<hipStream_t>(stream)));
}

int loss_forward(const void* d_h, const void* d_w, int32_t x_type, const int64_t* index, const float* teacher, int32_t top,
                 float tau, float* loss, float* lse, float* zt, int64_t n, int64_t v, int64_t k, void* ws, int64_t ws_bytes,
                 void* stream) {
    if (x_type != SWZ_X_BF16 && x_type != SWZ_X_F16) return SWZ_EINVAL;
    if (!(tau >= FLT_MIN && tau <= FLT_MAX)) return SWZ_EINVAL;  // 1 / tau and log2(e) / tau are finite then
    const int st = check_loss_sizes(n, v, k, top);
    if (st != SWZ_OK) return st;
    if (n == 0) return SWZ_OK;
    const int64_t need = loss_forward_bytes(n, v);
    if (ws_bytes < need) return SWZ_EINVAL;
    const bool distill = teacher != nullptr;
    const Span s[8] = {{d_h, 2 * n * k, 16, false},     {d_w, 2 * v * k, 16, false}, {index, 8 * n * top, 8, false},
                       {teacher, distill ? 4 * n * top : 0, 4, false}, {loss, 4 * n, 4, true}, {lse, 4 * n, 4, true},
                       {zt, 4 * n * top, 4, true},      {ws, need, 256, true}};
    if (!spans_ok(s, 8)) return SWZ_EINVAL;
    swz::LossJob j{};
    j.h = d_h, j.w = d_w, j.bf16 = x_type == SWZ_X_BF16, j.n = n, j.v = v, j.k = k, j.index = index, j.teacher = teacher;
    j.top = top, j.tau = tau, j.loss = loss, j.lse = lse, j.zt = zt, j.ws = ws;
    return hip_status(swz::launch_loss(j, static_cast<hipStream_t>(stream)));
}

int loss_backward(const void* d_h, const void* d_w, int32_t x_type, const int64_t* index, const float* teacher, int32_t top,
                  float tau, const float* lse, const float* zt, const float* upstream, void* dh, void* dw, int64_t n,
                  int64_t v, int64_t k, void* ws, int64_t ws_bytes, void* stream) {
    if (x_type != SWZ_X_BF16 && x_type != SWZ_X_F16) return SWZ_EINVAL;
    if (!(tau >= FLT_MIN && tau <= FLT_MAX)) return SWZ_EINVAL;  // 1 / tau and log2(e) / tau are finite then
    const int st = check_loss_sizes(n, v, k, top);
    if (st != SWZ_OK) return st;
    if (!dh && !dw) return SWZ_EINVAL;
    if (n == 0 && !dw) return SWZ_OK;
    const swz::LossPlan plan = plan_loss(n, v, k, top);
    if (n > 0 && ws_bytes < plan.bytes) return SWZ_EINVAL;
    const bool distill = teacher != nullptr;
    const Span s[10] = {{d_h, 2 * n * k, 16, false},
                        {d_w, n ? 2 * v * k : 0, 16, false},
                        {index, 8 * n * top, 8, false},
                        {teacher, distill ? 4 * n * top : 0, 4, false},
                        {lse, 4 * n, 4, false},
                        {zt, 4 * n * top, 4, false},
                        {upstream, 4 * n, 4, false},
                        {dh, dh ? 2 * n * k : 0, 16, true},
                        {dw, dw ? 2 * v * k : 0, 16, true},
                        {ws, n ? plan.bytes : 0, 256, true}};
    if (!spans_ok(s, 10)) return SWZ_EINVAL;
    swz::LossJob j{};
    j.h = d_h, j.w = d_w, j.bf16 = x_type == SWZ_X_BF16, j.n = n, j.v = v, j.k = k, j.index = index, j.teacher = teacher;
    j.top = top, j.tau = tau, j.lse = const_cast<float*>(lse), j.zt = const_cast<float*>(zt), j.upstream = upstream;
    j.dh = dh, j.dw = dw, j.ws = ws;
    return hip_status(swz::launch_loss_grad(j, plan, static_cast<hipStream_t>(stream)));
}

int ilog2(int64_t v) {
    int r = -1;
    while (v > 0) {
        v >>= 1;
        ++r;
    }
    return r;
}

// Parameters and LDS row pitch of a layout for a kind: the caller's swizzle
// or the chooser's for SWIZZLE and SWIZZLE_DIRECT (the direct fill also needs
// S >= B, so that the swizzle is its own inverse), the pad for PAD.
int resolve_layout(int kind, int32_t layout, const swz_params* p, swz_params* q, int* pad) {
    *q = swz_params{0, 0, 0};
    *pad = 0;
    switch (layout) {
        case SWZ_LAYOUT_SWIZZLE:
        case SWZ_LAYOUT_SWIZZLE_DIRECT:
            if (p) {
                if (!swz::params_ok_for_kind(kind, *p)) return SWZ_EINVAL;
                if (layout == SWZ_LAYOUT_SWIZZLE_DIRECT && p->B > 0 && (p->S < 0 ? -p->S : p->S) < p->B)
                    return SWZ_EINVAL;  // only |S| >= B makes the swizzle its own inverse
                *q = *p;
            } else {
                *q = swz::cached_choice(kind);
            }
            return SWZ_OK;
        case SWZ_LAYOUT_PAD: {
            // A row narrower than one 4-byte LDS write cannot get a pad of
            // its own: the write would straddle the gap.
            KindInfo k;
            if (swz::is_narrow(kind) && swz::kind_info(kind, &k) && k.tc * k.esz < 4) return SWZ_EUNSUPPORTED;
            *pad = swz::pad_elems(kind);
            return SWZ_OK;
        }
        case SWZ_LAYOUT_PLAIN: return SWZ_OK;
        default: return SWZ_EINVAL;
    }
}

// Resolve read kind, layout and parameters into a plan; shared by the calls
// and by swz_plan.  aligned_out: pointers and the output row pitch allow
// 16-byte vectors; aligned_in: so does the input row pitch.  Whole-row
// (narrow) tiles are contiguous stretches of the input, so they need only
// the first.
int make_plan(int op, int64_t rows, int64_t cols, int32_t esz, int32_t layout, int32_t read_kind,
              const swz_params* p, bool aligned_out, bool aligned_in, swz_plan_info* out) {
    if (layout < SWZ_LAYOUT_SWIZZLE || layout > SWZ_LAYOUT_SWIZZLE_DIRECT) return SWZ_EINVAL;
    int kind = read_kind;
    if (op == 0) {
        if (esz != 1 && esz != 2 && esz != 4) return SWZ_EINVAL;
        if (kind == SWZ_READ_AUTO) {
            // whole-row tiles: the swizzled kinds for power-of-two widths of
            // 1 to 64 bytes, flat rows for the other widths up to 128 columns
            // (fp32 from 96 columns on only where the last 32 x 32 tile
            // column would hold at most 19 columns: with fuller tiles the
            // tile kind ran faster, x 96 0.79 against 0.72 of a copy, x 120
            // 0.74 against 0.68, x 127 0.69 against 0.58; x 115 0.51
            // against 0.79)
            const bool pow2 = cols >= 1 && (cols & (cols - 1)) == 0;
            const bool narrow = pow2 && cols * esz <= 64;
            const int lc = ilog2(cols);
            const bool flat_rows = !pow2 && cols >= 1 && cols <= swz::kRowsMaxCols &&
                                   (esz != 4 || cols < 96 || (cols % 32 >= 1 && cols % 32 <= 19));
            // Power-of-two widths whose output rows (or pointers) rule out
            // 16-byte vectors: the swizzled narrow kinds then move elements
            // one by one, and flat rows ran faster for every fp32 width,
            // 2-byte widths of 8 to 32 and bytes x 64 (odd row counts, 64
            // MiB, share of a copy: fp32 x 1 0.59 -> 0.90, x 8 0.49 -> 0.75,
            // x 16 0.48 -> 0.74; 2-byte x 16 0.54 -> 0.72; bytes x 64 0.59
            // -> 0.64; narrower 2-byte and byte widths kept their kinds, at
            // 0.73-1.0)
            const bool unaligned_pow2 =
                narrow && !aligned_out && (esz == 4 || (esz == 2 && cols >= 8) || (esz == 1 && cols == 64));
            // (the flat-row kind has no padded or direct layout: those keep
            // the tile kinds)
            const bool rows_layout = layout == SWZ_LAYOUT_SWIZZLE || layout == SWZ_LAYOUT_PLAIN;
            if ((flat_rows || unaligned_pow2) && rows_layout)
                kind = SWZ_READ_ROWS;
            else if (esz == 4)
                kind = narrow ? SWZ_READ_NARROW1 + lc : SWZ_READ_SCALAR_COL;
            else if (esz == 2)
                kind = narrow        ? SWZ_READ_HNARROW1 + lc
                       : cols <= 64  ? SWZ_READ_B64_TR16
                       : cols <= 128 ? SWZ_READ_B128_8X8
                       : cols <= 256 ? SWZ_READ_B64_TR16
                       : rows % 2 == 0 && (!aligned_out || !aligned_in || swz::partial_line_output(rows, esz))
                           ? SWZ_READ_B64_TR16  // see below
                           : SWZ_READ_B64_4X4;
            // (Above 256 columns, for an even number of rows whose pitches
            // or pointers are off 16 bytes or whose output rows are off the
            // 64-byte lines, the transpose read ran faster: 4096 x 4100 0.81
            // -> 0.87 of a copy, 4100 x 4096 0.69 -> 0.73, 67108 x 500 0.63
            // -> 0.66, 111848 x 300 0.53 -> 0.56; with an odd number of rows
            // the 4x4 reads stay ahead: 5801 x 5801 0.67 against 0.56.)
            else
                kind = narrow ? SWZ_READ_BNARROW1 + lc : SWZ_READ_B64_TR8;
        }
        if (kind == SWZ_READ_MFMA_16X16X32) return SWZ_EINVAL;
        if (kind == SWZ_READ_ROWS) {
            // flat whole rows, swizzled on word offsets (M = 0, B <= S <=
            // 11: a bit of the tile's word offset XORs into a lower one;
            // B <= 10, so the XOR stays inside the 20 or 40 KiB of LDS, whole
            // 4 KiB blocks, that tile and halo take), or plain; no padded or
            // direct layout
            if (cols < 1 || cols > swz::kRowsMaxCols) return SWZ_EINVAL;
            if (layout == SWZ_LAYOUT_PAD || layout == SWZ_LAYOUT_SWIZZLE_DIRECT) return SWZ_EUNSUPPORTED;
            if (p && p->B != 0 && (p->B < 0 || p->B > 10 || p->M != 0 || p->S < p->B || p->S > 11))
                return SWZ_EINVAL;
            swz_params q{0, 0, 0};
            if (layout == SWZ_LAYOUT_SWIZZLE) q = p ? (p->B == 0 ? swz_params{0, 0, 0} : *p) : swz::rows_choice(static_cast<int>(cols));
            std::memset(out, 0, sizeof(*out));
            out->params = q;
            out->read_kind = kind;
            out->tile_rows = static_cast<int32_t>(swz::rows_tile_rows(cols, esz));
            out->tile_cols = static_cast<int32_t>(cols);
            out->layout = layout;
            out->lds_bytes = static_cast<int32_t>((out->tile_rows + swz::rows_halo_rows(esz)) * cols * esz);
            out->vec_bytes = 16;
            out->aligned = 1;  // any pitch: unaligned rows take the same accesses
            out->threads = swz::rows_threads(cols);
            out->interior_tiles = 1;
            return SWZ_OK;
        }
    } else {
        if (esz != 2) return SWZ_EINVAL;
        if (kind != SWZ_READ_AUTO && kind != SWZ_READ_MFMA_16X16X32) return SWZ_EINVAL;
        kind = SWZ_READ_MFMA_16X16X32;
    }
    KindInfo k;
    if (!swz::kind_info(kind, &k)) return SWZ_EINVAL;
    if (k.esz != esz) return SWZ_EINVAL;
    if (swz::is_narrow(kind) && cols != k.tc) return SWZ_EINVAL;  // whole rows per tile
    const bool aligned = aligned_out && (aligned_in || swz::is_narrow(kind));

    swz_params q;
    int pad;
    const int st = resolve_layout(kind, layout, p, &q, &pad);
    if (st != SWZ_OK) return st;
    if (layout == SWZ_LAYOUT_SWIZZLE_DIRECT && !aligned) return SWZ_EUNSUPPORTED;
    std::memset(out, 0, sizeof(*out));
    out->read_kind = kind;
    out->tile_rows = k.tr;
    out->tile_cols = k.tc;
    out->layout = layout;
    out->params = q;
    out->pad_elems = pad;
    out->lds_bytes = k.tr * (k.tc + pad) * k.esz;
    out->vec_bytes = layout == SWZ_LAYOUT_SWIZZLE_DIRECT ? (k.esz == 2 ? 16 : 4) : k.vec;
    out->aligned = aligned ? 1 : 0;
    out->threads = k.nt;
    out->interior_tiles = swz::interior_stack(kind) * swz::interior_stack_cols(kind);
    (void)rows;
    return SWZ_OK;
}

swz::LdsLayout layout_of(const swz_plan_info& pl) {
    return swz::LdsLayout{static_cast<uint32_t>(pl.tile_cols + pl.pad_elems), static_cast<uint32_t>(pl.params.B),
                          static_cast<uint32_t>(pl.params.M), pl.params.S};
}

// The order of a shape with none pinned, from sweeps of every order over
// matrices of 32-512 MiB with sides from 1,024 to 16,384 (bench.py
// --order-shapes).  What decides is the source row pitch:
// - not within 1% of a multiple of 4 KiB: slope 1/32.  Workgroups then walk
//   down the block columns nearly in order, so the output rows are written
//   in long runs, while the reads, a pitch apart, still spread over the
//   memory channels.  Over 745 fp32, 723 16-bit and 471 byte such shapes
//   the mean rate rose from 0.85, 0.87 and 0.84 of a copy of the same bytes
//   to 0.95, 0.96 and 0.90; one shape lost more than 1% (a byte matrix, 2.6%).
// - within 1% of a multiple of 4 KiB: reads a pitch apart fall on few
//   channels in that walk and the diagonal is needed; for fp32 matrices
//   with at most 10,240 rows and a side that is not a power of two, slope
//   1/8 did better still (462 shapes: 0.85 -> 0.91; 11 lost 2-6%; beyond
//   10,240 rows it lost up to 8%).
// Where the output rows are not whole 64-byte pieces (at 2,000 rows and
// more), whole tile columns in turn: the grid that serves those shapes has
// workgroups on one XCD take consecutive blocks, and in this order those
// are the neighbours that share the pieces (fp32, 16-bit and byte matrices
// of 2,000-9,000 rows: 0.45-0.60 of a copy before, 0.63-0.75 after; slope
// 1/32 within 1% of it, the diagonal up to 0.17 behind).  The whole-row
// kinds have one tile column, where every order is the same, and keep the
// diagonal.
int default_order(int kind, int64_t rows, int64_t cols) {
    const int esz = kind == SWZ_READ_SCALAR_COL ? 4
                    : kind == SWZ_READ_B64_4X4 || kind == SWZ_READ_B64_TR16 || kind == SWZ_READ_B128_8X8 ? 2
                    : kind == SWZ_READ_B64_TR8                                                          ? 1
                                                                                                        : 0;
    if (esz == 0) return SWZ_ORDER_DIAGONAL;
    // Output rows off the 64-byte pieces (the XCD-grouped grid): neighbours
    // down a block column share those pieces, so they go in turn, unless the
    // matrix is under 16 tiles wide; then the workgroups in flight would
    // crowd a few output rows, and the shallowest slope spreads them (odd row
    // counts, share of a copy, columns against slope 1/32: bytes x 300, 3
    // tiles, 0.30 against 0.42; 2-byte x 500, 8 tiles, 0.50 against 0.63;
    // bytes x 1000, 8 tiles, 0.50 against 0.59; from 16 tiles columns won or
    // tied: fp32 x 500 0.63 against 0.61, 2-byte x 1000 0.60 against 0.58).
    if (swz::partial_line_output(rows, esz)) {
        const int64_t tile_cols = kind == SWZ_READ_SCALAR_COL ? 32 : esz == 2 && kind != SWZ_READ_B128_8X8 ? 64 : 128;
        return (cols + tile_cols - 1) / tile_cols < 16 ? SWZ_ORDER_SLOPE_32 : SWZ_ORDER_COLUMNS;
    }
    const uint64_t pitch = static_cast<uint64_t>(cols) * static_cast<uint64_t>(esz), r = pitch % 4096;
    const uint64_t off = r < 4096 - r ? r : 4096 - r;  // distance to the nearest multiple of 4 KiB
    if (off * 100 > pitch) return SWZ_ORDER_SLOPE_32;
    const bool pow2 = (rows & (rows - 1)) == 0 && (cols & (cols - 1)) == 0;
    return esz == 4 && !pow2 && rows <= 10240 ? SWZ_ORDER_SLOPE_8 : SWZ_ORDER_DIAGONAL;
}

// Tile orders pinned per conversion shape (swz_set_tile_order,
// swz_tune_tile_order); shapes not listed use their default order.
using ShapeKey = std::tuple<int, int64_t, int64_t, int64_t>;  // read kind, batch, rows, cols
std::mutex g_order_mu;
std::map<ShapeKey, int>& order_table() {
    static std::map<ShapeKey, int> t;
    return t;
}
int pinned_order(int kind, int64_t batch, int64_t rows, int64_t cols) {
    std::lock_guard<std::mutex> lock(g_order_mu);
    const auto it = order_table().find(ShapeKey{kind, batch, rows, cols});
    return it == order_table().end() ? default_order(kind, rows, cols) : it->second;
}

}  // namespace

SWZ_API const char* swz_strerror(int status) {
    switch (status) {
        case SWZ_OK: return "ok";
        case SWZ_EINVAL: return "invalid argument";
        case SWZ_EUNSUPPORTED: return "unsupported request";
        case SWZ_EHIP: return "HIP runtime error";
        default: return "unknown status";
    }
}

SWZ_API int swz_map(const int32_t* d_in, int32_t* d_out, int64_t n, swz_params p, void* stream) {
    if (n < 0) return SWZ_EINVAL;
    const int64_t abs_s = p.S < 0 ? -static_cast<int64_t>(p.S) : p.S;
    if (p.B < 0 || p.M < 0 || static_cast<int64_t>(p.B) + p.M + abs_s > 32) return SWZ_EINVAL;
    if (n == 0) return SWZ_OK;
    if (!d_in || !d_out) return SWZ_EINVAL;
    if (reinterpret_cast<uintptr_t>(d_in) % 4 || reinterpret_cast<uintptr_t>(d_out) % 4) return SWZ_EINVAL;
    int64_t bytes;
    if (!mul_ok(n, 4, &bytes)) return SWZ_EINVAL;
    if (d_in != d_out && overlaps(d_in, bytes, d_out, bytes)) return SWZ_EINVAL;
    return hip_status(swz::launch_map(d_in, d_out, n, p, static_cast<hipStream_t>(stream)));
}

SWZ_API int swz_map_batch(const int32_t* d_in, int32_t* d_out, int64_t n, const swz_params* h_params,
                          int32_t n_params, void* stream) {
    if (n < 0 || n_params < 0) return SWZ_EINVAL;
    if (n_params > 0 && !h_params) return SWZ_EINVAL;
    for (int32_t j = 0; j < n_params; ++j) {
        const swz_params& p = h_params[j];
        const int64_t abs_s = p.S < 0 ? -static_cast<int64_t>(p.S) : p.S;
        if (p.B < 0 || p.M < 0 || static_cast<int64_t>(p.B) + p.M + abs_s > 32) return SWZ_EINVAL;
    }
    if (n == 0 || n_params == 0) return SWZ_OK;
    if (!d_in || !d_out) return SWZ_EINVAL;
    if (reinterpret_cast<uintptr_t>(d_in) % 4 || reinterpret_cast<uintptr_t>(d_out) % 4) return SWZ_EINVAL;
    int64_t in_bytes, out_elems, out_bytes;
    if (!mul_ok(n, 4, &in_bytes) || !mul_ok(n, n_params, &out_elems) || !mul_ok(out_elems, 4, &out_bytes))
        return SWZ_EINVAL;
    if (overlaps(d_in, in_bytes, d_out, out_bytes)) return SWZ_EINVAL;
    const auto st = static_cast<hipStream_t>(stream);
    for (int32_t j0 = 0; j0 < n_params; j0 += swz::kMapBatch) {
        const int count = n_params - j0 < swz::kMapBatch ? n_params - j0 : swz::kMapBatch;
        swz::MapParamPack pk{};
        for (int k = 0; k < count; ++k) {
            pk.B[k] = static_cast<uint8_t>(h_params[j0 + k].B);
            pk.M[k] = static_cast<uint8_t>(h_params[j0 + k].M);
            pk.S[k] = static_cast<int8_t>(h_params[j0 + k].S);
        }
        const int rc = hip_status(swz::launch_map_batch(d_in, d_out + static_cast<int64_t>(j0) * n, n, pk, count, st));
        if (rc != SWZ_OK) return rc;
    }
    return SWZ_OK;
}

SWZ_API int swz_plan(int32_t op, int64_t rows, int64_t cols, int32_t elem_bytes, int32_t layout, int32_t read_kind,
                     const swz_params* p_or_null, swz_plan_info* out) {
    if (!out || (op != 0 && op != 1) || rows < 0 || cols < 0) return SWZ_EINVAL;
    if (op == 1 && (rows % 16 || cols % 32)) return SWZ_EINVAL;
    // Pointers are taken as 16-byte aligned; the row pitches decide the rest.
    return make_plan(op, rows, cols, elem_bytes, layout, read_kind, p_or_null,
                     op == 1 || pitch16(rows, elem_bytes), op == 1 || pitch16(cols, elem_bytes), out);
}

SWZ_API int swz_convert_layout(const void* d_src, void* d_dst, int64_t batch, int64_t rows, int64_t cols,
                               int32_t elem_bytes, int32_t layout, int32_t read_kind, const swz_params* p_or_null,
                               void* stream) {
    if (batch < 0 || rows < 0 || cols < 0) return SWZ_EINVAL;
    if (elem_bytes != 1 && elem_bytes != 2 && elem_bytes != 4) return SWZ_EINVAL;
    int64_t n, n2, bytes;
    if (!mul_ok(batch, rows, &n) || !mul_ok(n, cols, &n2) || !mul_ok(n2, elem_bytes, &bytes)) return SWZ_EINVAL;
    const auto ps = reinterpret_cast<uintptr_t>(d_src), pd = reinterpret_cast<uintptr_t>(d_dst);
    swz_plan_info pl;
    const int st = make_plan(0, rows, cols, elem_bytes, layout, read_kind, p_or_null,
                             ps % 16 == 0 && pd % 16 == 0 && pitch16(rows, elem_bytes), pitch16(cols, elem_bytes), &pl);
    if (st != SWZ_OK) return st;
    if (bytes == 0) return SWZ_OK;
    if (!d_src || !d_dst) return SWZ_EINVAL;
    if (ps % elem_bytes || pd % elem_bytes) return SWZ_EINVAL;
    if (overlaps(d_src, bytes, d_dst, bytes)) return SWZ_EINVAL;
    swz::ConvertJob job{d_src, d_dst, batch, rows, cols, layout_of(pl), pl.aligned != 0,
                        layout == SWZ_LAYOUT_SWIZZLE_DIRECT, pinned_order(pl.read_kind, batch, rows, cols)};
    if (pl.read_kind == SWZ_READ_ROWS)
        return hip_status(swz::launch_rows(elem_bytes, job, static_cast<hipStream_t>(stream)));
    return hip_status(swz::launch_convert(pl.read_kind, job, static_cast<hipStream_t>(stream)));
}

SWZ_API int swz_transpose(const void* d_src, void* d_dst, int64_t rows, int64_t cols, int32_t elem_bytes,
                          int32_t layout, int32_t read_kind, const swz_params* p_or_null, void* stream) {
    return swz_convert_layout(d_src, d_dst, 1, rows, cols, elem_bytes, layout, read_kind, p_or_null, stream);
}

SWZ_API int swz_set_tile_order(int64_t batch, int64_t rows, int64_t cols, int32_t elem_bytes, int32_t read_kind,
                               int32_t order) {
    if (batch < 0 || rows < 0 || cols < 0) return SWZ_EINVAL;
    if (order < -1 || order > SWZ_ORDER_SLOPE_32) return SWZ_EINVAL;
    swz_plan_info pl;
    const int st = make_plan(0, rows, cols, elem_bytes, SWZ_LAYOUT_SWIZZLE, read_kind, nullptr,
                             pitch16(rows, elem_bytes), pitch16(cols, elem_bytes), &pl);
    if (st != SWZ_OK) return st;
    std::lock_guard<std::mutex> lock(g_order_mu);
    const ShapeKey key{pl.read_kind, batch, rows, cols};
    if (order < 0)
        order_table().erase(key);
    else
        order_table()[key] = order;
    return SWZ_OK;
}

SWZ_API int swz_get_tile_order(int64_t batch, int64_t rows, int64_t cols, int32_t elem_bytes, int32_t read_kind,
                               int32_t* order) {
    if (!order || batch < 0 || rows < 0 || cols < 0) return SWZ_EINVAL;
    swz_plan_info pl;
    const int st = make_plan(0, rows, cols, elem_bytes, SWZ_LAYOUT_SWIZZLE, read_kind, nullptr,
                             pitch16(rows, elem_bytes), pitch16(cols, elem_bytes), &pl);
    if (st != SWZ_OK) return st;
    *order = pinned_order(pl.read_kind, batch, rows, cols);
    return SWZ_OK;
}

SWZ_API int swz_tune_tile_order(const void* d_src, void* d_dst, int64_t batch, int64_t rows, int64_t cols,
                                int32_t elem_bytes, int32_t layout, int32_t read_kind, const swz_params* p_or_null,
                                int32_t reps, int32_t* chosen, void* stream) {
    if (!chosen || reps < 1 || reps > 1000) return SWZ_EINVAL;
    if (batch < 0 || rows < 0 || cols < 0) return SWZ_EINVAL;
    swz_plan_info pl;
    const auto ps = reinterpret_cast<uintptr_t>(d_src), pd = reinterpret_cast<uintptr_t>(d_dst);
    int st = make_plan(0, rows, cols, elem_bytes, layout, read_kind, p_or_null,
                       ps % 16 == 0 && pd % 16 == 0 && pitch16(rows, elem_bytes), pitch16(cols, elem_bytes), &pl);
    if (st != SWZ_OK) return st;
    int64_t n, n2, bytes;
    if (!mul_ok(batch, rows, &n) || !mul_ok(n, cols, &n2) || !mul_ok(n2, elem_bytes, &bytes)) return SWZ_EINVAL;
    const int dflt = default_order(pl.read_kind, rows, cols);
    if (bytes == 0) {
        *chosen = dflt;
        return SWZ_OK;
    }
    if (!d_src || !d_dst) return SWZ_EINVAL;
    const auto strm = static_cast<hipStream_t>(stream);
    hipEvent_t e0 = nullptr, e1 = nullptr;
    if (hipEventCreate(&e0) != hipSuccess || hipEventCreate(&e1) != hipSuccess) {
        if (e0) (void)hipEventDestroy(e0);
        return SWZ_EHIP;
    }
    // Three rounds over the orders (interleaved, so slow drifts of clock or
    // temperature hit them alike), each one untimed and reps timed calls;
    // an order's time is its best round.
    constexpr int kOrders = SWZ_ORDER_SLOPE_32 + 1, kRounds = 3;
    float t[kOrders];
    for (int o = 0; o < kOrders; ++o) t[o] = -1.0f;
    for (int round = 0; round < kRounds && st == SWZ_OK; ++round) {
        for (int order = 0; order < kOrders && st == SWZ_OK; ++order) {
            st = swz_set_tile_order(batch, rows, cols, elem_bytes, pl.read_kind, order);
            for (int r = 0; r <= reps && st == SWZ_OK; ++r) {
                if (r == 1 && hipEventRecord(e0, strm) != hipSuccess) st = SWZ_EHIP;
                if (st == SWZ_OK)
                    st = swz_convert_layout(d_src, d_dst, batch, rows, cols, elem_bytes, layout, read_kind,
                                            p_or_null, stream);
            }
            float ms = 0.0f;
            if (st == SWZ_OK && (hipEventRecord(e1, strm) != hipSuccess || hipEventSynchronize(e1) != hipSuccess ||
                                 hipEventElapsedTime(&ms, e0, e1) != hipSuccess))
                st = SWZ_EHIP;
            if (st == SWZ_OK && (t[order] < 0.0f || ms < t[order])) t[order] = ms;
        }
    }
    // Another order replaces the default one only when it is at least 3%
    // faster: the timed calls reuse one buffer pair, which the caches hold
    // in part, so small differences need not carry over to other buffers.
    int best = dflt;
    for (int o = 0; o < kOrders; ++o)
        if (o != dflt && t[o] >= 0.0f && t[o] < t[best] && (best != dflt || t[o] < 0.97f * t[best])) best = o;
    (void)hipEventDestroy(e0);
    (void)hipEventDestroy(e1);
    if (st != SWZ_OK) {
        (void)swz_set_tile_order(batch, rows, cols, elem_bytes, pl.read_kind, -1);
        return st;
    }
    // the last call left the result in d_dst; the pinned order gives the same bits
    *chosen = best;
    return swz_set_tile_order(batch, rows, cols, elem_bytes, pl.read_kind, best);
}

SWZ_API int swz_stage_operand(const void* d_src, void* d_frag, int64_t mn, int64_t k, int32_t elem_bytes,
                              int32_t frag_kind, int32_t layout, const swz_params* p_or_null, void* stream) {
    if (mn < 0 || k < 0 || mn % 16 || k % 32) return SWZ_EINVAL;
    if (elem_bytes != 2 || frag_kind != SWZ_FRAG_MFMA_F32_16X16X32_BF16) return SWZ_EINVAL;
    int64_t n, bytes;
    if (!mul_ok(mn, k, &n) || !mul_ok(n, 2, &bytes)) return SWZ_EINVAL;
    swz_plan_info pl;
    const int st = make_plan(1, mn, k, elem_bytes, layout, SWZ_READ_MFMA_16X16X32, p_or_null, true, true, &pl);
    if (st != SWZ_OK) return st;
    if (bytes == 0) return SWZ_OK;
    if (!d_src || !d_frag) return SWZ_EINVAL;
    if (reinterpret_cast<uintptr_t>(d_src) % 16 || reinterpret_cast<uintptr_t>(d_frag) % 16) return SWZ_EINVAL;
    if (overlaps(d_src, bytes, d_frag, bytes)) return SWZ_EINVAL;
    swz::StageJob job{d_src, d_frag, mn, k, layout_of(pl), layout == SWZ_LAYOUT_SWIZZLE_DIRECT};
    return hip_status(swz::launch_stage(job, static_cast<hipStream_t>(stream)));
}

SWZ_API int swz_stage_operands(const void* d_a, void* d_fa, int64_t m, const void* d_bt, void* d_fb, int64_t n,
                               int64_t k, int32_t elem_bytes, int32_t frag_kind, int32_t layout,
                               const swz_params* p_or_null, void* stream) {
    if (m < 0 || n < 0 || k < 0 || m % 16 || n % 16 || k % 32) return SWZ_EINVAL;
    if (elem_bytes != 2 || frag_kind != SWZ_FRAG_MFMA_F32_16X16X32_BF16) return SWZ_EINVAL;
    int64_t ea, eb, a_bytes, b_bytes;
    if (!mul_ok(m, k, &ea) || !mul_ok(ea, 2, &a_bytes) || !mul_ok(n, k, &eb) || !mul_ok(eb, 2, &b_bytes))
        return SWZ_EINVAL;
    swz_plan_info pl;
    const int st = make_plan(1, m > n ? m : n, k, elem_bytes, layout, SWZ_READ_MFMA_16X16X32, p_or_null, true, true, &pl);
    if (st != SWZ_OK) return st;
    if (a_bytes == 0 && b_bytes == 0) return SWZ_OK;
    if ((a_bytes && (!d_a || !d_fa)) || (b_bytes && (!d_bt || !d_fb))) return SWZ_EINVAL;
    for (const void* q : {d_a, static_cast<const void*>(d_fa), d_bt, static_cast<const void*>(d_fb)})
        if (reinterpret_cast<uintptr_t>(q) % 16) return SWZ_EINVAL;
    // each fragment buffer is disjoint from both sources and from the other
    // one (the sources are only read and may share memory)
    if (overlaps(d_fa, a_bytes, d_a, a_bytes) || overlaps(d_fa, a_bytes, d_bt, b_bytes) ||
        overlaps(d_fb, b_bytes, d_a, a_bytes) || overlaps(d_fb, b_bytes, d_bt, b_bytes) ||
        overlaps(d_fa, a_bytes, d_fb, b_bytes))
        return SWZ_EINVAL;
    swz::StageJob job{d_a, d_fa, m, k, layout_of(pl), layout == SWZ_LAYOUT_SWIZZLE_DIRECT};
    if (a_bytes == 0) {  // only B^T
        job.src = d_bt;
        job.frag = d_fb;
        job.mn = n;
    } else if (b_bytes > 0) {
        job.src2 = d_bt;
        job.frag2 = d_fb;
        job.mn2 = n;
    }
    return hip_status(swz::launch_stage(job, static_cast<hipStream_t>(stream)));
}

SWZ_API int swz_gemm_frag(const void* d_fa, const void* d_fb, float* d_c, int64_t m, int64_t n, int64_t k,
                          int32_t frag_kind, void* stream) {
    if (m < 0 || n < 0 || k < 0 || m % 16 || n % 16 || k % 32) return SWZ_EINVAL;
    if (frag_kind != SWZ_FRAG_MFMA_F32_16X16X32_BF16) return SWZ_EINVAL;
    int64_t a_elems, b_elems, c_elems, a_bytes, b_bytes, c_bytes;
    if (!mul_ok(m, k, &a_elems) || !mul_ok(n, k, &b_elems) || !mul_ok(m, n, &c_elems)) return SWZ_EINVAL;
    if (!mul_ok(a_elems, 2, &a_bytes) || !mul_ok(b_elems, 2, &b_bytes) || !mul_ok(c_elems, 4, &c_bytes))
        return SWZ_EINVAL;
    if (m == 0 || n == 0) return SWZ_OK;
    if (!d_c) return SWZ_EINVAL;
    if (k > 0 && (!d_fa || !d_fb)) return SWZ_EINVAL;
    const auto pa = reinterpret_cast<uintptr_t>(d_fa), pb = reinterpret_cast<uintptr_t>(d_fb),
               pc = reinterpret_cast<uintptr_t>(d_c);
    if (pa % 16 || pb % 16 || pc % 16) return SWZ_EINVAL;
    if (k > 0 && (overlaps(d_c, c_bytes, d_fa, a_bytes) || overlaps(d_c, c_bytes, d_fb, b_bytes))) return SWZ_EINVAL;
    return hip_status(swz::launch_gemm_frag(d_fa, d_fb, d_c, m, n, k, static_cast<hipStream_t>(stream)));
}

SWZ_API int swz_gemm_ex(const void* d_a, const void* d_bt, void* d_c, int64_t m, int64_t n, int64_t k,
                        int32_t layout, const swz_params* p_or_null, int32_t c_type, void* stream) {
    if (c_type != SWZ_C_F32 && c_type != SWZ_C_BF16) return SWZ_EINVAL;
    if (m < 0 || n < 0 || k < 0 || m % 16 || n % 16 || k % 32) return SWZ_EINVAL;
    if (layout == SWZ_LAYOUT_PAD) return SWZ_EUNSUPPORTED;  // the direct fill writes whole rows
    swz_plan_info pl;
    const int st = make_plan(1, m, k, 2, layout == SWZ_LAYOUT_SWIZZLE ? SWZ_LAYOUT_SWIZZLE_DIRECT : layout,
                             SWZ_READ_MFMA_16X16X32, p_or_null, true, true, &pl);
    if (st != SWZ_OK) return st;
    int64_t a_elems, b_elems, c_elems, a_bytes, b_bytes, c_bytes;
    if (!mul_ok(m, k, &a_elems) || !mul_ok(n, k, &b_elems) || !mul_ok(m, n, &c_elems)) return SWZ_EINVAL;
    if (!mul_ok(a_elems, 2, &a_bytes) || !mul_ok(b_elems, 2, &b_bytes) ||
        !mul_ok(c_elems, c_type == SWZ_C_BF16 ? 2 : 4, &c_bytes))
        return SWZ_EINVAL;
    if (m == 0 || n == 0) return SWZ_OK;
    if (!d_c) return SWZ_EINVAL;
    if (k > 0 && (!d_a || !d_bt)) return SWZ_EINVAL;
    const auto pa = reinterpret_cast<uintptr_t>(d_a), pb = reinterpret_cast<uintptr_t>(d_bt),
               pc = reinterpret_cast<uintptr_t>(d_c);
    if (pa % 16 || pb % 16 || pc % 16) return SWZ_EINVAL;
    if (k > 0 && (overlaps(d_c, c_bytes, d_a, a_bytes) || overlaps(d_c, c_bytes, d_bt, b_bytes))) return SWZ_EINVAL;
    return hip_status(swz::launch_gemm_tiles(d_a, d_bt, d_c, m, n, k, layout_of(pl), c_type == SWZ_C_BF16,
                                             static_cast<hipStream_t>(stream)));
}

SWZ_API int swz_gemm(const void* d_a, const void* d_bt, float* d_c, int64_t m, int64_t n, int64_t k, int32_t layout,
                     const swz_params* p_or_null, void* stream) {
    return swz_gemm_ex(d_a, d_bt, d_c, m, n, k, layout, p_or_null, SWZ_C_F32, stream);
}

SWZ_API int swz_quant_f8(const void* d_x, int32_t x_type, int64_t rows, int64_t cols, int64_t ld_x, int32_t f8_type,
                         int32_t block, int32_t scale_type, void* d_q, void* d_scale, int64_t ld_q, void* d_qt,
                         void* d_scale_t, int64_t ld_qt, void* stream) {
    if (x_type != SWZ_X_BF16 && x_type != SWZ_X_F16 && x_type != SWZ_X_F32) return SWZ_EINVAL;
    if (f8_type != SWZ_F8_E4M3 && f8_type != SWZ_F8_E5M2) return SWZ_EINVAL;
    if (block != SWZ_BLOCK_1X128 && block != SWZ_BLOCK_128X128) return SWZ_EINVAL;
    if (scale_type != SWZ_SCALE_F32 && scale_type != SWZ_SCALE_E8M0) return SWZ_EINVAL;
    if (rows < 0 || cols < 0 || ld_x < cols) return SWZ_EINVAL;
    if (!d_q && !d_qt) return SWZ_EINVAL;
    const int64_t esz = x_type == SWZ_X_F32 ? 4 : 2;
    const bool square = block == SWZ_BLOCK_128X128;
    int64_t n, x_bytes, q_bytes = 0, s_bytes = 0, qt_bytes = 0, st_bytes = 0;
    if (!span_elems(rows, cols, ld_x, &n) || !mul_ok(n, esz, &x_bytes)) return SWZ_EINVAL;
    if (d_q) {
        if (!d_scale || ld_q < cols || ld_q % 16 || !f8_operand_bytes(rows, cols, cols, ld_q, square, scale_type, &q_bytes, &s_bytes))
            return SWZ_EINVAL;
        if (reinterpret_cast<uintptr_t>(d_q) % 16) return SWZ_EINVAL;
    }
    if (d_qt) {
        if (!d_scale_t || ld_qt < rows || ld_qt % 16 ||
            !f8_operand_bytes(cols, rows, rows, ld_qt, square, scale_type, &qt_bytes, &st_bytes))
            return SWZ_EINVAL;
        if (reinterpret_cast<uintptr_t>(d_qt) % 16) return SWZ_EINVAL;
    }
    if (rows == 0 || cols == 0) return SWZ_OK;
    if (!d_x || reinterpret_cast<uintptr_t>(d_x) % static_cast<uintptr_t>(esz)) return SWZ_EINVAL;
    const uintptr_t sal = scale_type == SWZ_SCALE_F32 ? 4 : 1;
    const void* buf[5] = {d_x, d_q, d_q ? d_scale : nullptr, d_qt, d_qt ? d_scale_t : nullptr};
    const int64_t bytes[5] = {x_bytes, q_bytes, s_bytes, qt_bytes, st_bytes};
    for (int i = 0; i < 5; ++i) {
        if (!buf[i]) continue;
        if ((i == 2 || i == 4) && reinterpret_cast<uintptr_t>(buf[i]) % sal) return SWZ_EINVAL;
        for (int j = 0; j < i; ++j)
            if (buf[j] && overlaps(buf[i], bytes[i], buf[j], bytes[j])) return SWZ_EINVAL;
    }
    const int64_t tr = (rows - 1) / 128 + 1, tc = (cols - 1) / 128 + 1;
    if ((d_qt || square) && tr > (int64_t(1) << 23) / tc) return SWZ_EUNSUPPORTED;
    const swz::QuantJob job{d_x,   x_type,  rows, cols,      ld_x, f8_type == SWZ_F8_E5M2, square, scale_type == SWZ_SCALE_F32,
                            d_q,   d_scale, ld_q, d_qt, d_scale_t, ld_qt};
    return hip_status(swz::launch_quant(job, static_cast<hipStream_t>(stream)));
}

SWZ_API int swz_gemm_f8(const void* d_a, const void* d_scale_a, const void* d_b, const void* d_scale_b, void* d_c,
                        int64_t m, int64_t n, int64_t k, int64_t lda, int64_t ldb, int32_t a_type, int32_t b_type,
                        int32_t a_block, int32_t b_block, int32_t scale_type, int32_t c_type, void* stream) {
    for (const int32_t t : {a_type, b_type})
        if (t != SWZ_F8_E4M3 && t != SWZ_F8_E5M2) return SWZ_EINVAL;
    for (const int32_t b : {a_block, b_block})
        if (b != SWZ_BLOCK_1X128 && b != SWZ_BLOCK_128X128) return SWZ_EINVAL;
    if (scale_type != SWZ_SCALE_F32 && scale_type != SWZ_SCALE_E8M0) return SWZ_EINVAL;
    if (c_type != SWZ_C_F32 && c_type != SWZ_C_BF16) return SWZ_EINVAL;
    if (m < 0 || n < 0 || k < 0 || lda < k || ldb < k || lda % 16 || ldb % 16) return SWZ_EINVAL;
    const bool sqa = a_block == SWZ_BLOCK_128X128, sqb = b_block == SWZ_BLOCK_128X128;
    const int64_t esz = c_type == SWZ_C_BF16 ? 2 : 4;
    int64_t a_bytes, sa_bytes, b_bytes, sb_bytes, c_elems, c_bytes;
    const int64_t k16 = k + (16 - k % 16) % 16;  // rows are read in pieces of 16 bytes; k <= lda, a multiple of 16
    if (!f8_operand_bytes(m, k, k16, lda, sqa, scale_type, &a_bytes, &sa_bytes) ||
        !f8_operand_bytes(n, k, k16, ldb, sqb, scale_type, &b_bytes, &sb_bytes) || !mul_ok(m, n, &c_elems) ||
        !mul_ok(c_elems, esz, &c_bytes))
        return SWZ_EINVAL;
    if (m == 0 || n == 0) return SWZ_OK;
    if (!d_c || reinterpret_cast<uintptr_t>(d_c) % static_cast<uintptr_t>(esz)) return SWZ_EINVAL;
    if (k > 0) {
        if (!d_a || !d_b || !d_scale_a || !d_scale_b) return SWZ_EINVAL;
        if (reinterpret_cast<uintptr_t>(d_a) % 16 || reinterpret_cast<uintptr_t>(d_b) % 16) return SWZ_EINVAL;
        if (scale_type == SWZ_SCALE_F32 &&
            (reinterpret_cast<uintptr_t>(d_scale_a) % 4 || reinterpret_cast<uintptr_t>(d_scale_b) % 4))
            return SWZ_EINVAL;
        if (overlaps(d_c, c_bytes, d_a, a_bytes) || overlaps(d_c, c_bytes, d_b, b_bytes) ||
            overlaps(d_c, c_bytes, d_scale_a, sa_bytes) || overlaps(d_c, c_bytes, d_scale_b, sb_bytes))
            return SWZ_EINVAL;
    }
    if (lda >= swz::kMaxPitch || ldb >= swz::kMaxPitch) return SWZ_EUNSUPPORTED;
    if (n >= int64_t(1) << 26 || (m - 1) / 256 + 1 > ((int64_t(1) << 22) - 1) / ((n - 1) / 256 + 1)) return SWZ_EUNSUPPORTED;
    const swz::GemmF8Job job{d_a, d_scale_a, d_b, d_scale_b, d_c, m, n, k, lda, ldb, a_type == SWZ_F8_E5M2,
                             b_type == SWZ_F8_E5M2, sqa, sqb, scale_type == SWZ_SCALE_E8M0, c_type == SWZ_C_BF16};
    return hip_status(swz::launch_gemm_f8(job, static_cast<hipStream_t>(stream)));
}

SWZ_API int swz_linear_loss_workspace(int64_t n, int64_t v, int64_t k, int32_t top, int32_t grad, int64_t* bytes) {
    if (!bytes || (grad != 0 && grad != 1)) return SWZ_EINVAL;
    const int st = check_loss_sizes(n, v, k, top);
    if (st != SWZ_OK) return st;
    *bytes = loss_forward_bytes(n, v);
    if (grad) {
        const int64_t b = plan_loss(n, v, k, top).bytes;
        if (b > *bytes) *bytes = b;
    }
    return SWZ_OK;
}

SWZ_API int swz_linear_ce(const void* d_h, const void* d_w, int32_t x_type, const int64_t* d_target, float* d_loss,
                          float* d_lse, float* d_zt, int64_t n, int64_t v, int64_t k, void* d_ws, int64_t ws_bytes,
                          void* stream) {
    return loss_forward(d_h, d_w, x_type, d_target, nullptr, 1, 1.f, d_loss, d_lse, d_zt, n, v, k, d_ws, ws_bytes, stream);
}

SWZ_API int swz_linear_ce_grad(const void* d_h, const void* d_w, int32_t x_type, const int64_t* d_target,
                               const float* d_lse, const float* d_zt, const float* d_upstream, void* d_dh, void* d_dw,
                               int64_t n, int64_t v, int64_t k, void* d_ws, int64_t ws_bytes, void* stream) {
    return loss_backward(d_h, d_w, x_type, d_target, nullptr, 1, 1.f, d_lse, d_zt, d_upstream, d_dh, d_dw, n, v, k, d_ws,
                         ws_bytes, stream);
}

SWZ_API int swz_linear_distill(const void* d_h, const void* d_w, int32_t x_type, const int64_t* d_index,
                               const float* d_teacher, int32_t top, float tau, float* d_loss, float* d_lse, float* d_zt,
                               int64_t n, int64_t v, int64_t k, void* d_ws, int64_t ws_bytes, void* stream) {
    if (n > 0 && !d_teacher) return SWZ_EINVAL;
    return loss_forward(d_h, d_w, x_type, d_index, d_teacher, top, tau, d_loss, d_lse, d_zt, n, v, k, d_ws, ws_bytes, stream);
}

SWZ_API int swz_linear_distill_grad(const void* d_h, const void* d_w, int32_t x_type, const int64_t* d_index,
                                    const float* d_teacher, int32_t top, float tau, const float* d_lse, const float* d_zt,
                                    const float* d_upstream, void* d_dh, void* d_dw, int64_t n, int64_t v, int64_t k,
                                    void* d_ws, int64_t ws_bytes, void* stream) {
    if (n > 0 && !d_teacher) return SWZ_EINVAL;
    return loss_backward(d_h, d_w, x_type, d_index, d_teacher, top, tau, d_lse, d_zt, d_upstream, d_dh, d_dw, n, v, k, d_ws,
                         ws_bytes, stream);
}

SWZ_API int swz_gated(const void* d_x, const void* d_wg, const void* d_wu, int32_t x_type, int32_t act, void* d_y, float* d_pre,
                      int64_t n, int64_t f, int64_t k, void* stream) {
    if (!half_type(x_type) || !act_known(act)) return SWZ_EINVAL;
    const int st = check_gated_sizes(n, f, k);
    if (st != SWZ_OK) return st;
    if (n == 0) return SWZ_OK;
    const Span s[] = {{d_x, 2 * n * k, 16, false}, {d_wg, 2 * f * k, 16, false}, {d_wu, 2 * f * k, 16, false},
                      {d_y, 2 * n * f, 2, true}, {d_pre, d_pre ? 8 * n * f : 0, 4, true}};
    if (!spans_ok(s, 5)) return SWZ_EINVAL;
    swz::GatedJob j{};
    j.x = d_x, j.wg = d_wg, j.wu = d_wu, j.bf16 = x_type == SWZ_X_BF16, j.act = act, j.n = n, j.f = f, j.k = k, j.y = d_y;
    j.pre = d_pre;
    return hip_status(swz::launch_gated(j, static_cast<hipStream_t>(stream)));
}

SWZ_API int swz_gated_workspace(int64_t n, int64_t f, int64_t k, int64_t* bytes) {
    if (!bytes) return SWZ_EINVAL;
    const int st = check_gated_sizes(n, f, k);
    if (st != SWZ_OK) return st;
    *bytes = plan_gated(n, f, k).bytes;
    return SWZ_OK;
}

SWZ_API int swz_gated_grad(const void* d_x, const void* d_wg, const void* d_wu, int32_t x_type, int32_t act, const void* d_dy,
                           const float* d_pre, void* d_dx, void* d_dwg, void* d_dwu, int64_t n, int64_t f, int64_t k, void* d_ws,
                           int64_t ws_bytes, void* stream) {
    if (!half_type(x_type) || !act_known(act)) return SWZ_EINVAL;
    const int st = check_gated_sizes(n, f, k);
    if (st != SWZ_OK) return st;
    if (!d_dx && !d_dwg && !d_dwu) return SWZ_EINVAL;
    const swz::GatedPlan p = plan_gated(n, f, k);
    const bool any = n > 0;
    if (ws_bytes < p.bytes) return SWZ_EINVAL;
    const Span s[] = {{d_x, 2 * n * k, 16, false}, {d_wg, any ? 2 * f * k : 0, 16, false}, {d_wu, any ? 2 * f * k : 0, 16, false},
                      {d_dy, 2 * n * f, 2, false}, {d_pre, d_pre ? 8 * n * f : 0, 4, false}, {d_dx, d_dx ? 2 * n * k : 0, 16, true},
                      {d_dwg, d_dwg ? 2 * f * k : 0, 16, true}, {d_dwu, d_dwu ? 2 * f * k : 0, 16, true},
                      {d_ws, p.bytes, 256, true}};
    if (!spans_ok(s, 9)) return SWZ_EINVAL;
    swz::GatedJob j{};
    j.x = d_x, j.wg = d_wg, j.wu = d_wu, j.bf16 = x_type == SWZ_X_BF16, j.act = act, j.n = n, j.f = f, j.k = k, j.dy = d_dy;
    j.pre = const_cast<float*>(d_pre), j.dx = d_dx, j.dwg = d_dwg, j.dwu = d_dwu, j.ws = d_ws;
    return hip_status(swz::launch_gated_grad(j, p, static_cast<hipStream_t>(stream)));
}

SWZ_API int swz_quant_w4(const void* d_w, int32_t w_type, int64_t n, int64_t k, int32_t group, int32_t x_type, void* d_q,
                         void* d_scale, uint8_t* d_zero, void* stream) {
    if ((!half_type(w_type) && w_type != SWZ_X_F32) || !half_type(x_type)) return SWZ_EINVAL;
    const int st = check_w4_sizes(n, k, group);
    if (st != SWZ_OK) return st;
    const int64_t groups = (k + group - 1) / group;
    const Span s[] = {{d_w, n * k * (w_type == SWZ_X_F32 ? 4 : 2), 16, false}, {d_q, n * (k / 2), 16, true},
                      {d_scale, 2 * n * groups, 2, true}, {d_zero, d_zero ? n * groups : 0, 1, true}};
    if (n == 0) return SWZ_OK;
    if (!spans_ok(s, 4)) return SWZ_EINVAL;
    const swz::QuantW4Job j{d_w, w_type, x_type == SWZ_X_BF16, n, k, group, d_q, d_scale, d_zero};
    return hip_status(swz::launch_quant_w4(j, static_cast<hipStream_t>(stream)));
}

SWZ_API int swz_dequant_w4(const void* d_q, const void* d_scale, const uint8_t* d_zero, int64_t n, int64_t k, int32_t group,
                           int32_t x_type, void* d_w, void* stream) {
    if (!half_type(x_type)) return SWZ_EINVAL;
    const int st = check_w4_sizes(n, k, group);
    if (st != SWZ_OK) return st;
    const int64_t groups = (k + group - 1) / group;
    const Span s[] = {{d_q, n * (k / 2), 16, false}, {d_scale, 2 * n * groups, 2, false}, {d_zero, d_zero ? n * groups : 0, 1, false},
                      {d_w, 2 * n * k, 16, true}};
    if (n == 0) return SWZ_OK;
    if (!spans_ok(s, 4)) return SWZ_EINVAL;
    const swz::WeightsW4 w{static_cast<const uint8_t*>(d_q), d_scale, d_zero};
    return hip_status(swz::launch_dequant_w4(w, x_type == SWZ_X_BF16, n, k, group, d_w, static_cast<hipStream_t>(stream)));
}

SWZ_API int swz_gemm_w4(const void* d_x, int32_t x_type, const void* d_q, const void* d_scale, const uint8_t* d_zero, int32_t group,
                        void* d_c, int64_t m, int64_t n, int64_t k, void* stream) {
    const swz::WeightsW4 w{static_cast<const uint8_t*>(d_q), d_scale, d_zero};
    return gemm_w4(d_x, x_type, 0, &w, 1, group, d_c, m, n, k, stream);
}

SWZ_API int swz_gated_w4(const void* d_x, int32_t x_type, int32_t act, const void* d_qg, const void* d_scale_g,
                         const uint8_t* d_zero_g, const void* d_qu, const void* d_scale_u, const uint8_t* d_zero_u, int32_t group,
                         void* d_c, int64_t m, int64_t n, int64_t k, void* stream) {
    if (!act_known(act) || !d_zero_g != !d_zero_u) return SWZ_EINVAL;
    const swz::WeightsW4 w[2] = {{static_cast<const uint8_t*>(d_qg), d_scale_g, d_zero_g},
                                 {static_cast<const uint8_t*>(d_qu), d_scale_u, d_zero_u}};
    return gemm_w4(d_x, x_type, act, w, 2, group, d_c, m, n, k, stream);
}

SWZ_API int swz_grad_norm_workspace(int32_t count, int64_t* bytes) { return bytes ? norm_workspace(count, bytes) : SWZ_EINVAL; }

SWZ_API int swz_grad_norm(const void* const* d_t, const int64_t* numel, const int32_t* type, int32_t count, float* d_norm,
                          void* d_ws, int64_t ws_bytes, void* stream) {
    return norm_call(d_t, nullptr, numel, type, count, false, 0.f, d_norm, d_ws, ws_bytes, stream);
}

SWZ_API int swz_clip_grads(const void* const* d_t, void* const* d_out, const int64_t* numel, const int32_t* type, int32_t count,
                           float max_norm, float* d_norm, void* d_ws, int64_t ws_bytes, void* stream) {
    if (!(max_norm >= 0.f)) return SWZ_EINVAL;
    return norm_call(d_t, d_out, numel, type, count, true, max_norm, d_norm, d_ws, ws_bytes, stream);
}

SWZ_API int swz_fold(const swz_params* p, uint32_t base, uint32_t active, uint32_t* collision,
                     uint32_t* folded_base, int64_t* strides) {
    if (!p || !collision) return SWZ_EINVAL;
    const int64_t abs_s = p->S < 0 ? -static_cast<int64_t>(p->S) : p->S;
    if (p->B < 0 || p->M < 0 || p->B + p->M + abs_s > 32) return SWZ_EINVAL;
    if (base & active) return SWZ_EINVAL;
    const auto B = static_cast<uint32_t>(p->B), M = static_cast<uint32_t>(p->M);
    *collision = active & ~swz::swizzle(active, B, M, p->S);
    if (*collision) return SWZ_EUNSUPPORTED;
    const uint32_t sb = swz::swizzle(base, B, M, p->S);
    if (folded_base) *folded_base = sb;
    if (strides) {
        for (int b = 0; b < 32; ++b) {
            strides[b] = 0;
            if (!((active >> b) & 1u)) continue;
            // Flipping bit b flips the bits of swizzle(1 << b) in swizzle(base):
            // each flip adds its power of two where that bit was clear and
            // subtracts it where it was set.  Without collisions the bits
            // flipped by different active bits never meet, so the moves add.
            const uint32_t v = swz::swizzle(1u << b, B, M, p->S);
            int64_t d = 0;
            for (int t = 0; t < 32; ++t)
                if ((v >> t) & 1u) d += ((sb >> t) & 1u) ? -(int64_t(1) << t) : (int64_t(1) << t);
            strides[b] = d;
        }
    }
    return SWZ_OK;
}

SWZ_API int swz_choose(int32_t elem_bytes, int32_t vec_bytes, int32_t tile_rows, int32_t tile_cols, int32_t read_kind,
                       swz_params* out) {
    if (!out) return SWZ_EINVAL;
    KindInfo k;
    if (!swz::kind_info(read_kind, &k)) return SWZ_EINVAL;
    if (k.esz != elem_bytes || k.vec != vec_bytes || k.tr != tile_rows || k.tc != tile_cols) return SWZ_EUNSUPPORTED;
    *out = swz::cached_choice(read_kind);
    return SWZ_OK;
}

SWZ_API int swz_predict_conflicts(int32_t read_kind, int32_t layout, const swz_params* p_or_null, int64_t* wcyc,
                                  int64_t* rcyc) {
    if (!wcyc || !rcyc) return SWZ_EINVAL;
    KindInfo k;
    if (!swz::kind_info(read_kind, &k)) return SWZ_EINVAL;
    swz_params q;
    int pad;
    const int st = resolve_layout(read_kind, layout, p_or_null, &q, &pad);
    if (st != SWZ_OK) return st;
    swz::predict_tile(read_kind, swz::gfx950_bank_model(), static_cast<uint32_t>(k.tc + pad), q, wcyc, rcyc,
                      layout == SWZ_LAYOUT_SWIZZLE_DIRECT);
    return SWZ_OK;
}

SWZ_API int swz_kernel_accesses(int32_t read_kind, int32_t layout, const swz_params* p_or_null, int32_t is_write,
                                int32_t* addrs, int32_t max_accesses, int32_t* n_accesses, int32_t* width) {
    if (!n_accesses || !width || max_accesses < 0 || (max_accesses > 0 && !addrs)) return SWZ_EINVAL;
    if (is_write != 0 && is_write != 1) return SWZ_EINVAL;
    KindInfo k;
    if (!swz::kind_info(read_kind, &k)) return SWZ_EINVAL;
    swz_params q;
    int pad;
    const int st = resolve_layout(read_kind, layout, p_or_null, &q, &pad);
    if (st != SWZ_OK) return st;
    int w = 0;
    *n_accesses = swz::kernel_accesses(read_kind, static_cast<uint32_t>(k.tc + pad), q,
                                       layout == SWZ_LAYOUT_SWIZZLE_DIRECT, is_write != 0, addrs, max_accesses, &w);
    *width = w;
    return SWZ_OK;
}

SWZ_API int swz_copy(const void* d_src, void* d_dst, int64_t bytes, void* stream) {
    if (bytes < 0 || bytes % 16) return SWZ_EINVAL;
    if (bytes == 0) return SWZ_OK;
    if (!d_src || !d_dst) return SWZ_EINVAL;
    if (reinterpret_cast<uintptr_t>(d_src) % 16 || reinterpret_cast<uintptr_t>(d_dst) % 16) return SWZ_EINVAL;
    if (overlaps(d_src, bytes, d_dst, bytes)) return SWZ_EINVAL;
    return hip_status(swz::launch_copy(d_src, d_dst, bytes, static_cast<hipStream_t>(stream)));
}

SWZ_API int swz_bank_model_get(swz_bank_model* out) {
    if (!out) return SWZ_EINVAL;
    const swz::BankModel& m = swz::gfx950_bank_model();
    for (int d = 0; d < 2; ++d) {
        for (int w = 0; w < 3; ++w) {
            out->n_banks[d][w] = m.n_banks[d][w];
            out->bank_bytes[d][w] = m.bank_bytes[d][w];
        }
    }
    std::memcpy(out->phase, m.phase, sizeof(out->phase));
    return SWZ_OK;
}

SWZ_API int swz_lds_probe(const uint32_t* d_addrs, const uint64_t* d_masks, int32_t n_patterns, int32_t width_bytes,
                          int32_t is_write, int32_t iters, int32_t waves, uint64_t* d_cycles, void* stream) {
    if (n_patterns < 0 || (width_bytes != 1 && width_bytes != 2 && width_bytes != 4 && width_bytes != 8 &&
                           width_bytes != 16))
        return SWZ_EINVAL;
    if (iters < 1 || iters > (1 << 20) || waves < 1 || waves > 16 || (is_write != 0 && is_write != 1))
        return SWZ_EINVAL;
    if (n_patterns == 0) return SWZ_OK;
    if (!d_addrs || !d_masks || !d_cycles) return SWZ_EINVAL;
    return hip_status(swz::launch_lds_probe(d_addrs, d_masks, n_patterns, width_bytes, is_write != 0, iters, waves,
                                            d_cycles, static_cast<hipStream_t>(stream)));
}
