// The norm of many tensors together, sqrt(sum over all of x^2), and the
// tensors scaled so that it is at most a given one.
//
// Bound by the tensors' bytes, read once for the norm and once more, and
// written, where they are scaled.  Squares are summed in fp64, which costs
// nothing beside the loads: no square leaves its range, and the sums' order
// is fixed by the sizes, so the same call gives the same bits.
//
// A launch takes up to kNormTensors tensors, described in its arguments, so the
// host's lists are not read after the call and a captured call holds its own.
// Work is dealt out in chunks of kNormPieces pieces of 16 bytes, counted from
// the 16-byte boundary at or before a tensor's start; a tensor's first and last
// piece may be partly its own and go by elements.
#include "launch_ffn.h"

namespace swz {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

struct Pack {
    const uint8_t* in[kNormTensors];
    uint8_t* out[kNormTensors];
    int64_t numel[kNormTensors];
    uint32_t first[kNormTensors + 1];  // each tensor's first chunk
    uint8_t type[kNormTensors];
    int count;
};
static_assert(sizeof(Pack) <= 4000, "fits a launch's arguments");

template <int TYPE>
struct Kind {
    static constexpr int E = TYPE == SWZ_X_F32 ? 4 : 8;  // elements of a piece
    using T = std::conditional_t<TYPE == SWZ_X_F32, float, std::conditional_t<TYPE == SWZ_X_BF16, __bf16, _Float16>>;
    typedef T vec __attribute__((ext_vector_type(E)));
};

__device__ __forceinline__ int tensor_of(const Pack& p, uint32_t chunk) {
    int lo = 0, hi = p.count;  // first[lo] <= chunk < first[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (p.first[mid] <= chunk)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// A thread's part of a chunk: all(first element of each of its kPer pieces,
// whether it is the tensor's as a whole; another's place where not), and
// edge(first element, elements) for a tensor's first and last piece where they are
// not whole.  No load waits for a branch.
constexpr int kPer = kNormPieces / 256;
template <int TYPE, class A, class S>
__device__ __forceinline__ void pieces_of(const uint8_t* in, int64_t numel, int64_t chunk, A all, S edge) {
    constexpr int E = Kind<TYPE>::E, ES = 16 / E;
    const int64_t skew = static_cast<int64_t>(reinterpret_cast<uintptr_t>(in) % 16) / ES;
    const int64_t p0 = chunk * kNormPieces, whole0 = skew ? 1 : 0, whole1 = (skew + numel) / E;  // whole pieces
    if (whole0 < whole1) {
        int64_t at[kPer];
        bool valid[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int64_t p = p0 + 256 * i + threadIdx.x, q = p < whole0 ? whole0 : p < whole1 ? p : whole1 - 1;
            valid[i] = p == q;
            at[i] = q * E - skew;
        }
        all(at, valid);
    }
    if (threadIdx.x == 0 && chunk == 0 && skew) edge(int64_t(0), static_cast<int>(numel < E - skew ? numel : E - skew));
    if (threadIdx.x == 64 && whole1 >= whole0 && (skew + numel) % E && whole1 >= p0 && whole1 < p0 + kNormPieces)
        edge(whole1 * E - skew, static_cast<int>((skew + numel) % E));
}

template <int TYPE>
__device__ __forceinline__ double squares(const uint8_t* in, int64_t numel, int64_t chunk) {
    using T = typename Kind<TYPE>::T;
    using V = typename Kind<TYPE>::vec;
    constexpr int E = Kind<TYPE>::E;
    const T* x = reinterpret_cast<const T*>(in);
    double s = 0.0;
    auto add = [](double& to, T v) {
        const double d = static_cast<double>(static_cast<float>(v));
        to = __builtin_fma(d, d, to);
    };
    pieces_of<TYPE>(
        in, numel, chunk,
        [&](const int64_t (&at)[kPer], const bool (&valid)[kPer]) {
            V v[kPer];
#pragma unroll
            for (int i = 0; i < kPer; ++i) v[i] = *reinterpret_cast<const V*>(x + at[i]);
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                double part = 0.0;
#pragma unroll
                for (int e = 0; e < E; ++e) add(part, v[i][e]);
                s += valid[i] ? part : 0.0;
            }
        },
        [&](int64_t at, int n) {
            for (int i = 0; i < n; ++i) add(s, x[at + i]);
        });
    return s;
}

// Sum over the workgroup, in thread 0.
template <int NT>
__device__ __forceinline__ double block_sum(double s) {
    __shared__ double part[NT / 64];
#pragma unroll
    for (int d = 1; d < 64; d *= 2) s += __shfl_xor(s, d);
    if (threadIdx.x % 64 == 0) part[threadIdx.x / 64] = s;
    __syncthreads();
    if (threadIdx.x == 0)
        for (int w = 1; w < NT / 64; ++w) s += part[w];
    return s;
}

__global__ __launch_bounds__(256) void k_squares(Pack p, double* __restrict__ partial) {
    double s = 0.0;
    for (uint32_t c = blockIdx.x; c < p.first[p.count]; c += gridDim.x) {
        const int t = tensor_of(p, c);
        const int64_t chunk = c - p.first[t];
        if (p.type[t] == SWZ_X_BF16)
            s += squares<SWZ_X_BF16>(p.in[t], p.numel[t], chunk);
        else if (p.type[t] == SWZ_X_F16)
            s += squares<SWZ_X_F16>(p.in[t], p.numel[t], chunk);
        else
            s += squares<SWZ_X_F32>(p.in[t], p.numel[t], chunk);
    }
    s = block_sum<256>(s);
    if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

__global__ __launch_bounds__(1024) void k_norm(const double* __restrict__ partial, int64_t partials, float max_norm, bool clip,
                                               float* __restrict__ norm) {
    double s = 0.0;
    for (int64_t i = threadIdx.x; i < partials; i += 1024) s += partial[i];
    s = block_sum<1024>(s);
    if (threadIdx.x) return;
    const double r = sqrt(s);
    norm[0] = static_cast<float>(r);
    if (clip) {
        const bool over = r > static_cast<double>(max_norm) && r < static_cast<double>(__builtin_inff());
        norm[1] = over ? static_cast<float>(static_cast<double>(max_norm) / r) : 1.f;
    }
}

// x factor, rounded to fp32 before it is rounded to its type, in whatever form
// the compiler meets it (a mixed-precision multiply would round to fp16 at once,
// and a value's bits would depend on its tensor's alignment).
template <class T>
__device__ __forceinline__ T scaled(T x, float factor) {
    float p = static_cast<float>(x) * factor;
    asm("" : "+v"(p));
    return static_cast<T>(p);
}

template <int TYPE>
__device__ __forceinline__ void scale_chunk(const uint8_t* in, uint8_t* to, int64_t numel, int64_t chunk, float factor) {
    using T = typename Kind<TYPE>::T;
    using V = typename Kind<TYPE>::vec;
    constexpr int E = Kind<TYPE>::E;
    const T* x = reinterpret_cast<const T*>(in);
    T* o = reinterpret_cast<T*>(to);
    const bool alike = (reinterpret_cast<uintptr_t>(in) - reinterpret_cast<uintptr_t>(to)) % 16 == 0;
    auto one = [&](T v) { return factor == 1.f ? v : scaled<T>(v, factor); };
    pieces_of<TYPE>(
        in, numel, chunk,
        [&](const int64_t (&at)[kPer], const bool (&valid)[kPer]) {
            V v[kPer];
#pragma unroll
            for (int i = 0; i < kPer; ++i) v[i] = __builtin_nontemporal_load(reinterpret_cast<const V*>(x + at[i]));
            asm volatile("" ::: "memory");  // in place: nothing is read again behind a store
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
#pragma unroll
                for (int e = 0; e < E; ++e) v[i][e] = one(v[i][e]);
                if (!valid[i]) continue;
                if (alike) {
                    __builtin_nontemporal_store(v[i], reinterpret_cast<V*>(o + at[i]));
                } else {
#pragma unroll
                    for (int e = 0; e < E; ++e) o[at[i] + e] = v[i][e];
                }
            }
        },
        [&](int64_t at, int n) {
            for (int i = 0; i < n; ++i) o[at + i] = one(x[at + i]);
        });
}

// Chunks from the last to the first: what the squares read last is still in the
// 256 MB cache.
__global__ __launch_bounds__(256) void k_scale(Pack p, const float* __restrict__ norm) {
    const float factor = norm[1];
    for (uint32_t i = blockIdx.x; i < p.first[p.count]; i += gridDim.x) {
        const uint32_t c = p.first[p.count] - 1 - i;
        const int t = tensor_of(p, c);
        if (factor == 1.f && p.in[t] == p.out[t]) continue;
        const int64_t chunk = c - p.first[t];
        if (p.type[t] == SWZ_X_BF16)
            scale_chunk<SWZ_X_BF16>(p.in[t], p.out[t], p.numel[t], chunk, factor);
        else if (p.type[t] == SWZ_X_F16)
            scale_chunk<SWZ_X_F16>(p.in[t], p.out[t], p.numel[t], chunk, factor);
        else
            scale_chunk<SWZ_X_F32>(p.in[t], p.out[t], p.numel[t], chunk, factor);
    }
}

// The launches of a list, from its first tensor or from its last: f(pack, blocks).
template <class F>
hipError_t by_packs(const NormJob& j, bool backwards, F f) {
    Pack p;
    p.count = 0;
    uint32_t chunks = 0;
    auto launch = [&] {
        if (p.count == 0) return hipSuccess;
        p.first[p.count] = chunks;
        const hipError_t e = f(p, static_cast<unsigned>(chunks < kNormBlocks ? chunks : kNormBlocks));
        p.count = 0;
        chunks = 0;
        return e;
    };
    for (int32_t i = 0; i < j.count; ++i) {
        const int32_t t = backwards ? j.count - 1 - i : i;
        if (j.numel[t] == 0) continue;
        p.in[p.count] = static_cast<const uint8_t*>(j.data[t]);
        p.out[p.count] = static_cast<uint8_t*>(j.clip ? (j.out ? j.out[t] : const_cast<void*>(j.data[t])) : nullptr);
        p.numel[p.count] = j.numel[t];
        p.type[p.count] = static_cast<uint8_t>(j.type[t]);
        p.first[p.count++] = chunks;
        chunks += static_cast<uint32_t>(norm_chunks(j.data[t], j.numel[t], j.type[t]));
        if (p.count < kNormTensors) continue;
        const hipError_t e = launch();
        if (e != hipSuccess) return e;
    }
    return launch();
}

}  // namespace

hipError_t launch_norm(const NormJob& j, hipStream_t stream) {
    double* partial = j.ws;
    hipError_t e = by_packs(j, false, [&](const Pack& p, unsigned blocks) {
        hipLaunchKernelGGL(k_squares, dim3(blocks), dim3(256), 0, stream, p, partial);
        partial += blocks;
        return hipGetLastError();
    });
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(k_norm, dim3(1), dim3(1024), 0, stream, j.ws, partial - j.ws, j.max_norm, j.clip, j.norm);
    e = hipGetLastError();
    if (e != hipSuccess || !j.clip) return e;
    return by_packs(j, true, [&](const Pack& p, unsigned blocks) {
        hipLaunchKernelGGL(k_scale, dim3(blocks), dim3(256), 0, stream, p, j.norm);
        return hipGetLastError();
    });
}

}  // namespace swz
