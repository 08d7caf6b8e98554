// grads.cu -- the norm of all of a model's gradients taken as one vector, and their
// clipping to a largest norm.
//
//   norm = sqrt(sum over all tensors of g^2),    out = g min(1, max_norm / norm).
//
// Bound by reading the gradients, once for the norm and once for the scaling.  The tensors
// come as kernel parameters (addresses, lengths, first tiles; up to kMany a launch), so that
// a call copies nothing to the device and can be captured.  They are cut into tiles, which
// the blocks share evenly, each block a run of neighbouring ones; the scaling takes a run
// from its end, where what the norm read last may still be in L2.
//
// The sum: a thread adds the squares of its 32 elements of a tile in float32, and the tiles'
// sums, the blocks' and the call's with their rounding errors kept (two float32 numbers), in a
// fixed order; the last by every block of the scaling for itself.  So the norm of N elements
// is within a few float32 roundings, whatever N, and equal calls give equal bits.  Squares
// that leave float32's range, upward or downward, are added again in float64 (always in
// float64, a call of 1.3 M elements took 15.4 us).

#include <float.h>

#include "gdn_internal.h"
#include "rows.cuh"

namespace gdn {
namespace {

using namespace rows;

constexpr int kTile = kThreads * 32;  // elements
// Tensors of a launch: as many as fit 4 KB of parameters, or nearly 32 KB.
constexpr int kFew = 120, kMany = 1000;

// A tensor of a launch.  n: the length, with the types in its top bits.  tile0: the tiles of
// the tensors before.
struct Entry {
    const void* p;
    void* out;
    uint64_t n;
    uint32_t tile0;
};
template <int N>
struct List {
    Entry e[N];
    uint32_t tiles;
    int count;
};
constexpr uint64_t kOutBf16 = 1ull << 63, kInBf16 = 1ull << 62, kLength = kInBf16 - 1;

// A tensor as a block walks it.  Tiles begin at the 16-byte boundary before its first
// element, `lead` elements earlier.
struct Tensor {
    const char* p;
    char* out;
    int64_t n;
    uint32_t first, end;  // tiles
    int lead;
    bool in16, out16;
    template <int N>
    __device__ __forceinline__ void at(const List<N>& l, int i) {
        p = (const char*)l.e[i].p;
        out = (char*)l.e[i].out;
        const uint64_t n_ = l.e[i].n;
        n = (int64_t)(n_ & kLength);
        in16 = n_ & kInBf16;
        out16 = n_ & kOutBf16;
        first = l.e[i].tile0;
        end = i + 1 < l.count ? l.e[i + 1].tile0 : l.tiles;
        lead = (int)((uintptr_t)p & 15) >> (in16 ? 1 : 2);
    }
};

// The tensor that holds a tile: the last one that begins at or before it (empty tensors
// have no tiles).
template <int N>
__device__ __forceinline__ int find(const List<N>& l, uint32_t tile) {
    int lo = 0, hi = l.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (l.e[mid].tile0 <= tile) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

__device__ __forceinline__ float at1(const char* p, int64_t e, bool half) {
    return half ? __bfloat162float(((const __nv_bfloat16*)p)[e]) : ((const float*)p)[e];
}

// 16 bytes from element e on (e a whole number of vectors behind the boundary): elements
// outside the tensor are zeros.
template <int VEC>
__device__ __forceinline__ uint4 vector_at(const Tensor& t, int64_t e) {
    constexpr bool kHalf = VEC == 8;
    if (e >= 0 && e + VEC <= t.n) return *reinterpret_cast<const uint4*>(t.p + e * (16 / VEC));
    uint32_t w[4] = {0, 0, 0, 0};
    if (e >= t.n || e + VEC <= 0) return make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
        if (e + j < 0 || e + j >= t.n) continue;
        if (kHalf) w[j / 2] |= (uint32_t)((const uint16_t*)t.p)[e + j] << (j % 2 * 16);
        else w[j] = ((const uint32_t*)t.p)[e + j];
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// A sum as two float32 numbers, the second what the first's roundings left out; `rest` is what
// float32's range does not take, nearly always 0.
struct Sum {
    float s = 0.f, c = 0.f;
    double rest = 0.;
    __device__ __forceinline__ void add(float x) {
        const float t = s + x, b = t - s;
        c += (s - (t - b)) + (x - b);
        s = t;
    }
};

template <int VEC>
__device__ __forceinline__ void square_vectors(const Tensor& t, int64_t e, Sum& sum) {
    constexpr int M = 32 / VEC;
    uint4 v[M];
#pragma unroll
    for (int j = 0; j < M; ++j) v[j] = vector_at<VEC>(t, e + (int64_t)j * kThreads * VEC);
    uint64_t ss[2] = {twice(0.f), twice(0.f)};
#pragma unroll
    for (int j = 0; j < M; ++j) {
        uint64_t f[VEC / 2];
        get(v[j], f);
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) ss[i & 1] = fma2(f[i], f[i], ss[i & 1]);
    }
    const float s = sum2(add2(ss[0], ss[1]));
    // below 2^-100 a square may have been rounded to a subnormal or to 0; of sums above 2^85
    // the 2^31 tiles' might not fit
    if (s >= 7.888609e-31f && s <= 3.8685626e25f) {
        sum.add(s);
        return;
    }
    uint32_t any = 0;
#pragma unroll
    for (int j = 0; j < M; ++j) any |= v[j].x | v[j].y | v[j].z | v[j].w;
    if ((any & (VEC == 8 ? 0x7fff7fffu : 0x7fffffffu)) == 0) return;  // zeros, or no elements
    double d = 0.;
#pragma unroll
    for (int j = 0; j < M; ++j) {
        uint64_t f[VEC / 2];
        get(v[j], f);
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) {
            float a, b;
            unpair(f[i], a, b);
            if (a != 0.f) d += (double)a * a;
            if (b != 0.f) d += (double)b * b;
        }
    }
    sum.rest += d;
}

// A tile's squares, by kThreads threads.
__device__ __forceinline__ void square_tile(const Tensor& t, uint32_t tile, int thread, Sum& sum) {
    const int64_t e = (int64_t)(tile - t.first) * kTile - t.lead;
    if (t.in16) square_vectors<8>(t, e + thread * 8, sum);
    else square_vectors<4>(t, e + thread * 4, sum);
}

// The sums of a block's T threads added in a fixed order; the same in every thread.  Without
// float64 unless some thread has a rest: its operations run at a small part of float32's rate.
template <int T>
__device__ __forceinline__ Sum block_sum(Sum x) {
    __shared__ float2 part[T / 32];
    __shared__ double rests[T / 32];
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        const float s = __shfl_xor_sync(0xffffffffu, x.s, off), c = __shfl_xor_sync(0xffffffffu, x.c, off);
        x.add(s);
        x.c += c;
    }
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = make_float2(x.s, x.c);
    const bool any = __syncthreads_or(x.rest != 0.);  // true of NaN
    if (any) {
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) x.rest += __shfl_xor_sync(0xffffffffu, x.rest, off);
        if ((threadIdx.x & 31) == 0) rests[threadIdx.x >> 5] = x.rest;
        __syncthreads();
        x.rest = 0.;
        for (int i = 0; i < T / 32; ++i) x.rest += rests[i];
    }
    x.s = x.c = 0.f;
#pragma unroll
    for (int i = 0; i < T / 32; ++i) {
        x.add(part[i].x);
        x.c += part[i].y;
    }
    return x;
}

// Worker b's tiles, of n workers.
__device__ __forceinline__ void run_of(uint32_t tiles, uint32_t b, uint32_t n, uint32_t& from, uint32_t& to) {
    from = (uint32_t)((uint64_t)tiles * b / n);
    to = (uint32_t)((uint64_t)tiles * (b + 1) / n);
}

// Blocks an SM holds (252 M float32 into bf16, a whole call: 3 for the scaling 375 us, 4 391; where
// boundaries are apart, 22 M: 41 and 35).
constexpr int kSumPerSm = 4;
template <bool kApart>
constexpr int kScalePerSm = kApart ? 4 : 3;

template <int N>
__global__ void __launch_bounds__(kThreads, kSumPerSm)
grad_sum_kernel(const __grid_constant__ List<N> l, GradPart* __restrict__ part) {
    uint32_t tile, to;
    run_of(l.tiles, blockIdx.x, gridDim.x, tile, to);
    Sum sum;
    int i = 0;
    Tensor t;
    if (tile < to) t.at(l, i = find(l, tile));
    await_previous();
    for (; tile < to; ++tile) {
        while (tile >= t.end) t.at(l, ++i);
        square_tile(t, tile, threadIdx.x, sum);
    }
    sum = block_sum<kThreads>(sum);
    if (threadIdx.x == 0) part[blockIdx.x] = {sum.s, sum.c, sum.rest};
}

// What the gradients are multiplied by: the product of two numbers.  A factor below 2^-126, of which
// one float32 number would keep few bits or none, is first * 2^-126 with a normal first (below
// 2^-252, which takes a max_norm below 2^-102, no result is more than a subnormal); all others
// are first * 1.  The product by `first` overflows for no finite gradient: it is below 1 where the
// norm is past 2^65, and below 2 elsewhere.
struct Factor {
    float first, then;
    __device__ __forceinline__ bool one() const { return first == 1.f && then == 1.f; }
    __device__ __forceinline__ float of(float x) const { return x * first * then; }
    __device__ __forceinline__ uint64_t of(uint64_t x) const { return mul2(mul2(x, twice(first)), twice(then)); }
};
constexpr float kLeast = 1.17549435e-38f, kMost = 8.507059e37f;  // 2^-126, 2^126

// The norm from the blocks' sums, and the factor that takes it to max_norm; the same in every
// thread.
struct Norm {
    float norm;
    Factor by;
};
template <int T>
__device__ __forceinline__ Norm norm_of(Sum x, float max_norm) {
    __shared__ Norm all;
    x = block_sum<T>(x);
    const float s = x.s + x.c;
    if (x.rest == 0. && s <= FLT_MAX) {
        // the root of s, and half of what its square leaves of the sum over itself
        const float n = sqrtf(s), left = fmaf(-n, n, x.s) + x.c;
        const float norm = s > 0.f ? n + 0.5f * left / n : 0.f;
        if (!(norm > max_norm)) return {norm, {1.f, 1.f}};
        // a quotient near 2^-126 or below (max_norm is below 2^-60 then)
        const bool small = max_norm < norm * (2.f * kLeast);
        return {norm, {(small ? max_norm * kMost : max_norm) / norm, small ? kLeast : 1.f}};
    }
    if (threadIdx.x == 0) {
        const double n = sqrt((double)x.s + (double)x.c + x.rest);
        // where an element is not finite the norm says nothing of how long the gradients are: they
        // stay; finite ones whose norm leaves float32's range are clipped by the float64 norm
        const double by = n > (double)max_norm && n <= DBL_MAX ? (double)max_norm / n : 1.;
        const bool small = by < (double)kLeast;
        all = {(float)n, {(float)(small ? by * (double)kMost : by), small ? kLeast : 1.f}};
    }
    __syncthreads();
    return all;
}
__device__ __forceinline__ Sum parts_of(const GradPart* __restrict__ part, int parts) {
    Sum x;
    for (int i = threadIdx.x; i < parts; i += kThreads) {
        const GradPart p = part[i];
        x.add(p.s);
        x.c += p.c;
        x.rest += p.rest;
    }
    return x;
}

__global__ void __launch_bounds__(kThreads) grad_norm_kernel(const GradPart* __restrict__ part, int parts, float* norm) {
    await_previous();
    const Norm x = norm_of<kThreads>(parts_of(part, parts), __int_as_float(0x7f800000));  // no limit
    if (threadIdx.x == 0) *norm = x.norm;
}

// VEC neighbouring results from element e on, whose address is a whole number of vectors;
// none outside the tensor.
template <int VEC, bool kHalf>
__device__ __forceinline__ void put_vector(const Tensor& t, int64_t e, const uint64_t (&f)[VEC / 2]) {
    if (e >= 0 && e + VEC <= t.n) {
        if constexpr (kHalf && VEC == 8) {
            *reinterpret_cast<uint4*>(t.out + e * 2) = put(f);
        } else if constexpr (kHalf) {
            *reinterpret_cast<uint2*>(t.out + e * 2) = make_uint2(pack2(f[0]), pack2(f[1]));
        } else {
#pragma unroll
            for (int i = 0; i < VEC / 4; ++i) {
                const uint64_t g[2] = {f[2 * i], f[2 * i + 1]};
                *reinterpret_cast<uint4*>(t.out + (e + 4 * i) * 4) = put(g);
            }
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) {
        float a[2];
        unpair(f[i], a[0], a[1]);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int64_t at = e + 2 * i + k;
            if (at < 0 || at >= t.n) continue;
            if (kHalf) ((__nv_bfloat16*)t.out)[at] = __float2bfloat16_rn(a[k]);
            else ((float*)t.out)[at] = a[k];
        }
    }
}

template <int VEC, bool kHalf>
__device__ __forceinline__ void scale_vectors(const Tensor& t, int64_t e, const Factor& by) {
    constexpr int M = 32 / VEC;
    uint4 v[M];
#pragma unroll
    for (int j = 0; j < M; ++j) v[j] = vector_at<VEC>(t, e + (int64_t)j * kThreads * VEC);
#pragma unroll
    for (int j = 0; j < M; ++j) {
        uint64_t f[VEC / 2];
        get(v[j], f);
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) f[i] = by.of(f[i]);
        put_vector<VEC, kHalf>(t, e + (int64_t)j * kThreads * VEC, f);
    }
}

// N bf16 elements from the address p on, in words and not beyond them but for the halves of the
// first and the last word.
template <int N>
struct Halves {
    uint32_t w[N / 2 + 1];
    __device__ __forceinline__ void load(const char* p) {
        const uint32_t* q = reinterpret_cast<const uint32_t*>((uintptr_t)p & ~(uintptr_t)3);
#pragma unroll
        for (int k = 0; k < N / 2; ++k) w[k] = q[k];
        w[N / 2] = (uintptr_t)p & 2 ? q[N / 2] : 0;
    }
    __device__ __forceinline__ void get(bool odd, uint64_t (&f)[N / 2]) const {
#pragma unroll
        for (int k = 0; k < N / 2; ++k) f[k] = bf16_pair(odd ? __funnelshift_r(w[k], w[k + 1], 16) : w[k]);
    }
};

// Where the output's 16-byte boundaries are not the input's, as in a flat buffer: vectors of
// whole 16 bytes of the output, whose elements are read one by one (bf16: by words).  A tile
// takes the vectors that begin in it, but for the last at its end and with the one before its
// begin; the tensor's last tile takes one more.  (Elements one by one on both sides: 22 M bf16
// in odd places of a flat buffer 61 us a call, so 23.)
template <bool kIn16, bool kOut16>
__device__ __forceinline__ void scale_apart(const Tensor& t, uint32_t tile, int thread, const Factor& by) {
    constexpr int VEC = kOut16 ? 8 : 4, M = 32 / VEC;
    const int64_t e0 = (int64_t)(tile - t.first) * kTile - t.lead;
    const int lead = (int)((uintptr_t)t.out & 15) >> (kOut16 ? 1 : 2);
    const int64_t first = e0 - ((e0 + lead) & (VEC - 1)), e = first + thread * VEC;
    if (first >= 1 && first + kTile < t.n) {  // a word more on either side is the tensor's
        uint64_t f[M][VEC / 2];
        if constexpr (kIn16) {
            const bool odd = ((uintptr_t)t.p + 2 * e) & 2;
            Halves<VEC> h[M];
#pragma unroll
            for (int j = 0; j < M; ++j) h[j].load(t.p + 2 * (e + j * kThreads * VEC));
#pragma unroll
            for (int j = 0; j < M; ++j) h[j].get(odd, f[j]);
        } else {
#pragma unroll
            for (int j = 0; j < M; ++j) {
                const float* q = (const float*)t.p + e + j * kThreads * VEC;
#pragma unroll
                for (int k = 0; k < VEC / 2; ++k) f[j][k] = pair(q[2 * k], q[2 * k + 1]);
            }
        }
#pragma unroll
        for (int j = 0; j < M; ++j) {
#pragma unroll
            for (int k = 0; k < VEC / 2; ++k) f[j][k] = by.of(f[j][k]);
            put_vector<VEC, kOut16>(t, e + j * kThreads * VEC, f[j]);
        }
    } else {
        auto one = [&](int64_t at) {
            for (int k = 0; k < VEC; ++k, ++at) {
                if (at < 0 || at >= t.n) continue;
                const float x = by.of(at1(t.p, at, kIn16));
                if (kOut16) ((__nv_bfloat16*)t.out)[at] = __float2bfloat16_rn(x);
                else ((float*)t.out)[at] = x;
            }
        };
        for (int j = 0; j < M; ++j) one(e + j * kThreads * VEC);
    }
    if (tile + 1 == t.end && thread == 0) {
        const int64_t at = first + kTile;
        for (int k = 0; k < VEC; ++k) {
            if (at + k >= t.n) break;
            const float x = by.of(at1(t.p, at + k, kIn16));
            if (kOut16) ((__nv_bfloat16*)t.out)[at + k] = __float2bfloat16_rn(x);
            else ((float*)t.out)[at + k] = x;
        }
    }
}

// Whether a tensor's output has its boundaries where the input has.
__host__ __device__ __forceinline__ bool together(uintptr_t in, uintptr_t out, bool in16, bool out16) {
    const uintptr_t lead = (in & 15) >> (in16 ? 1 : 2);
    return (out - lead * (out16 ? 2 : 4)) % (in16 && out16 ? 16 : out16 ? 8 : 16) == 0;
}

// A tile times `by`, by kThreads threads.  kApart: some tensor's boundaries are apart.
template <bool kApart>
__device__ __forceinline__ void scale_tile(const Tensor& t, uint32_t tile, int thread, const Factor& by) {
    if (by.one() && t.out == t.p) return;
    const int64_t e = (int64_t)(tile - t.first) * kTile - t.lead;
    if (kApart && !together((uintptr_t)t.p, (uintptr_t)t.out, t.in16, t.out16)) {
        if (t.in16 && t.out16) scale_apart<true, true>(t, tile, thread, by);
        else if (t.in16) scale_apart<true, false>(t, tile, thread, by);
        else if (t.out16) scale_apart<false, true>(t, tile, thread, by);
        else scale_apart<false, false>(t, tile, thread, by);
    } else if (t.in16 && t.out16) scale_vectors<8, true>(t, e + thread * 8, by);
    else if (t.in16) scale_vectors<8, false>(t, e + thread * 8, by);
    else if (t.out16) scale_vectors<4, true>(t, e + thread * 4, by);
    else scale_vectors<4, false>(t, e + thread * 4, by);
}

// in_place: every tensor is its own output.
template <int N, bool kApart>
__global__ void __launch_bounds__(kThreads, kScalePerSm<kApart>)
grad_scale_kernel(const __grid_constant__ List<N> l, const GradPart* __restrict__ part, int parts, float max_norm,
                  float* norm, bool in_place) {
    uint32_t from, tile;
    run_of(l.tiles, blockIdx.x, gridDim.x, from, tile);
    int i = 0;
    Tensor t;
    if (from < tile) t.at(l, i = find(l, tile - 1));
    await_previous();
    const Norm x = norm_of<kThreads>(parts_of(part, parts), max_norm);
    if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = x.norm;
    const Factor by = x.by;
    if ((in_place && by.one()) || from >= tile) return;
    while (tile-- > from) {
        while (tile < t.first) t.at(l, --i);
        scale_tile<kApart>(t, tile, threadIdx.x, by);
    }
}

// Both passes of a few tiles in one launch: the blocks of one cluster, kWorkers workers of
// kThreads threads each, hand their sums around through shared memory, and the second pass reads
// what the first left in L2.  Without `clip` the norm alone.
constexpr int kWorkers = 3;
template <int N>
__global__ void __launch_bounds__(kThreads * kWorkers, 1)
grad_clip_kernel(const __grid_constant__ List<N> l, float max_norm, float* norm, bool clip) {
    __shared__ GradPart mine;
    const uint32_t worker = blockIdx.x * kWorkers + threadIdx.x / kThreads;
    const int thread = threadIdx.x % kThreads;
    uint32_t from, to;
    run_of(l.tiles, worker, gridDim.x * kWorkers, from, to);
    Sum sum;
    int i = 0;
    Tensor t;
    if (from < to) t.at(l, i = find(l, from));
    await_previous();
    for (uint32_t tile = from; tile < to; ++tile) {
        while (tile >= t.end) t.at(l, ++i);
        square_tile(t, tile, thread, sum);
    }
    sum = block_sum<kThreads * kWorkers>(sum);
    if (threadIdx.x == 0) mine = {sum.s, sum.c, sum.rest};
    cluster_sync();
    Sum all;
    if (threadIdx.x < gridDim.x) {
        float w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = cluster_word((const float*)&mine + k, threadIdx.x);
        all.s = w[0], all.c = w[1];
        all.rest = __hiloint2double(__float_as_int(w[3]), __float_as_int(w[2]));
    }
    cluster_sync();  // no block leaves before the others have read its sum
    const Norm x = norm_of<kThreads * kWorkers>(all, max_norm);
    if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = x.norm;
    if (!clip) return;
    for (uint32_t tile = to; tile-- > from;) {
        while (tile < t.first) t.at(l, --i);
        scale_tile<true>(t, tile, thread, x.by);
    }
}

// One launch's list from tensors a .. b - 1.
template <int N>
void fill(List<N>& l, const gdn_grad* g, int64_t a, int64_t b) {
    uint64_t tiles = 0;
    l.count = (int)(b - a);
    for (int64_t i = a; i < b; ++i) {
        const bool in16 = g[i].dtype == GDN_BF16;
        const int lead = (int)((uintptr_t)g[i].grad & 15) >> (in16 ? 1 : 2);
        l.e[i - a] = {g[i].grad, g[i].out, (uint64_t)g[i].n | (in16 ? kInBf16 : 0) | (g[i].out_dtype == GDN_BF16 ? kOutBf16 : 0),
                      (uint32_t)tiles};
        if (g[i].n) tiles += ((uint64_t)g[i].n + lead + kTile - 1) / kTile;
    }
    l.tiles = (uint32_t)tiles;
}

int grid_of(uint32_t tiles, int per_sm) {
    const uint32_t cap = (uint32_t)(per_sm * sm_count());
    return (int)(tiles < 1 ? 1 : tiles < cap ? tiles : cap);
}

template <int N>
cudaError_t sum(const gdn_grad* g, int64_t a, int64_t b, GradPart* part, int* parts, cudaStream_t st) {
    List<N> l;
    fill(l, g, a, b);
    const int grid = grid_of(l.tiles, kSumPerSm);
    GradPart* to = part + *parts;
    *parts += grid;
    return launch_dependent(grad_sum_kernel<N>, dim3(grid), kThreads, 0, st, l, to);
}

template <int N>
cudaError_t scale(const gdn_grad* g, int64_t a, int64_t b, const GradPart* part, int parts, float max_norm, float* norm,
                  bool in_place, cudaStream_t st) {
    List<N> l;
    fill(l, g, a, b);
    bool apart = false;
    for (int64_t i = a; i < b; ++i)
        apart = apart || (g[i].n && !together((uintptr_t)g[i].grad, (uintptr_t)g[i].out, g[i].dtype == GDN_BF16, g[i].out_dtype == GDN_BF16));
    const dim3 grid(grid_of(l.tiles, apart ? kScalePerSm<true> : kScalePerSm<false>));
    return apart ? launch_dependent(grad_scale_kernel<N, true>, grid, kThreads, 0, st, l, part, parts, max_norm, norm, in_place)
                 : launch_dependent(grad_scale_kernel<N, false>, grid, kThreads, 0, st, l, part, parts, max_norm, norm, in_place);
}

template <int N>
cudaError_t cluster(const gdn_grad* g, int64_t count, int blocks, float max_norm, float* norm, bool clip, cudaStream_t st) {
    static std::atomic<uint64_t> done{0};
    List<N> l;
    fill(l, g, 0, count);
    return launch_one_cluster(grad_clip_kernel<N>, blocks, kThreads * kWorkers, 0, done, st, l, max_norm, norm, clip);
}

// Tiles that one cluster takes, to clip them or for their norm alone.  Of 4 to 48 tiles calls one
// behind the other take 5.3 to 6.5 us and 4.5 to 5.2, as two launches, bound by the host, 6.6
// and 6.1; the GPU alone needs as long, and of two launches 4.1 to 4.6 and 3.1 to 3.4.  With
// 96 tiles the host's time is even, and the GPU's 6.2 to 6.9 against 3.6 to 4.5.
constexpr int64_t kClusterTiles = 48;

}  // namespace

int64_t grad_tiles(int64_t n) { return n / kTile + 2; }

size_t grad_parts(int64_t count) {
    const int64_t launches = count <= kMany ? 1 : (count + kMany - 1) / kMany;
    return (size_t)launches * kSumPerSm * sm_count();
}

int grad_cluster(const gdn_grad* g, int64_t count) {
    if (count > kFew) return 0;
    int64_t tiles = 0;
    for (int64_t i = 0; i < count; ++i) tiles += g[i].n / kTile + (g[i].n % kTile != 0);
    if (tiles > kClusterTiles) return 0;
    int blocks = 1;
    while (blocks < kMostCluster && blocks * kWorkers < tiles) blocks *= 2;
    return one_cluster(blocks) ? blocks : 0;
}

cudaError_t launch_grad_cluster(const gdn_grad* g, int64_t count, int blocks, float max_norm, float* norm, bool clip,
                                cudaStream_t st) {
    return cluster<kFew>(g, count, blocks, max_norm, norm, clip, st);
}

cudaError_t launch_grad_sums(const gdn_grad* g, int64_t count, GradPart* part, int* parts, cudaStream_t st) {
    *parts = 0;
    cudaError_t e = cudaSuccess;
    for (int64_t a = 0; e == cudaSuccess && (a == 0 || a < count); a += kMany) {
        const int64_t b = count - a < kMany ? count : a + kMany;
        e = b - a <= kFew ? sum<kFew>(g, a, b, part, parts, st) : sum<kMany>(g, a, b, part, parts, st);
    }
    return e;
}

cudaError_t launch_grad_norm(const GradPart* part, int parts, float* norm, cudaStream_t st) {
    return launch_dependent(grad_norm_kernel, dim3(1), kThreads, 0, st, part, parts, norm);
}

cudaError_t launch_grad_scale(const gdn_grad* g, int64_t count, const GradPart* part, int parts, float max_norm,
                              float* norm, cudaStream_t st) {
    cudaError_t e = cudaSuccess;
    for (int64_t a = 0; e == cudaSuccess && (a == 0 || a < count); a += kMany) {
        const int64_t b = count - a < kMany ? count : a + kMany;
        bool in_place = true;
        for (int64_t i = a; i < b; ++i) in_place = in_place && g[i].out == g[i].grad;
        float* to = a == 0 ? norm : nullptr;
        e = b - a <= kFew ? scale<kFew>(g, a, b, part, parts, max_norm, to, in_place, st)
                          : scale<kMany>(g, a, b, part, parts, max_norm, to, in_place, st);
    }
    return e;
}

}  // namespace gdn
