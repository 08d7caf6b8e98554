// add_norm.cu -- the residual's addition with the RMS norm of the sum, its form with an
// 8-bit output, and the gradients: the step in front of a layer's projection.
//
// Row x of D elements, residual s, weight w; h = x + s, r = (mean h^2 + eps)^(-1/2):
//   y = h r w,     y8 = e4m3(y / scale) with scale = max|y| / 448 over a group of columns.
// Backward, from dy and the gradient dh that reaches h by the residual stream, with
// hh = h r and t = dy w:
//   d = r (t - hh mean(t hh)) + dh   (of x and of the residual),    dw = sum over rows of dy hh.
//
// The sum is normalised as it stands in float32; h is what the residual stream keeps, in
// its own type, and what the backward reads.
//
// Bound by reading and writing the rows.  A row is held by L lanes (8 to 512), each with up to
// kPieces pieces of it a stride of L apart, so that a warp's loads and stores fill whole sectors;
// the row is read once, its sum of squares is made of registers.  Persistent blocks with a ring
// of asynchronous copies (rows.cuh) keep the next rows in flight.

#include <float.h>

#include "gdn_internal.h"
#include "rows.cuh"

namespace gdn {
namespace {

using namespace rows;

constexpr int kPieces = 4, kStages = 2;

// A piece: VEC elements, 16 bytes of the wider of a call's two types, 8 of the other.
template <typename T, int VEC>
struct Piece {
    static constexpr int BYTES = VEC * (int)sizeof(T);
    static __device__ __forceinline__ void copy(uint32_t at, const T* src) {
        if constexpr (BYTES == 16)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at), "l"(src) : "memory");
        else
            asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(at), "l"(src) : "memory");
    }
    static __device__ __forceinline__ void unpack(const uint4& x, uint64_t (&f)[VEC / 2]) {
        if constexpr (BYTES == 16) get(x, f);
        else f[0] = bf16_pair(x.x), f[1] = bf16_pair(x.y);
    }
    static __device__ __forceinline__ void load(uint32_t at, uint64_t (&f)[VEC / 2]) {
        uint4 x = make_uint4(0, 0, 0, 0);
        if constexpr (BYTES == 16)
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(at) : "memory");
        else asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(x.x), "=r"(x.y) : "r"(at) : "memory");
        unpack(x, f);
    }
    static __device__ __forceinline__ uint4 ldg(const T* p) {
        if constexpr (BYTES == 16) return ldg16(p);
        const uint2 x = __ldg(reinterpret_cast<const uint2*>(p));
        return make_uint4(x.x, x.y, 0, 0);
    }
    static __device__ __forceinline__ void store(T* p, const uint64_t (&f)[VEC / 2]) {
        if constexpr (BYTES == 16) __stcs(reinterpret_cast<uint4*>(p), put(f));
        else __stcs(reinterpret_cast<uint2*>(p), make_uint2(pack2(f[0]), pack2(f[1])));
    }
};

// NP pieces (16 bytes of room each) of S rows for each of N threads.
template <int NP, int S, int N>
struct Slots {
    static constexpr int BYTES = NP * S * N * 16;
    uint32_t base;
    __device__ __forceinline__ explicit Slots(void* sm)
        : base((uint32_t)__cvta_generic_to_shared(sm) + threadIdx.x * 16) {}
    __device__ __forceinline__ uint32_t at(int slot, int piece) const {
        return base + (uint32_t)((slot * NP + piece) * N * 16);
    }
};
__device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void wait_group() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// max(|pair's two|, m)
__device__ __forceinline__ float abs_max(const uint64_t& p, float m) {
    float a, b, r;
    unpair(p, a, b);
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(m));
    return r;
}

// A thread's place: its row of the block's in each turn, and in the row the columns c0 + p LV of
// its pieces p < n.  Pieces behind the row's end and rows behind the last are not read,
// computed or written; their lanes only take part in exchanges and barriers.
template <int VEC>
struct Place {
    int L, LV, c0, n;
    int warps, first;   // of a row that takes whole warps: how many, and the first
    int64_t row, step;  // this thread's first row, and the rows that all blocks take in a turn
    int turns;          // the same for every thread of a block
    __device__ __forceinline__ Place(int64_t rows, int D, int L_) : L(L_), LV(L_ * VEC), n(0), warps(L_ / 32) {
        const int per = blockDim.x / L_, mine = threadIdx.x / L_;
        c0 = ((int)threadIdx.x - mine * L_) * VEC;
        first = mine * warps;
#pragma unroll
        for (int p = 0; p < kPieces; ++p) n += c0 + p * LV < D;
        const int64_t base = (int64_t)blockIdx.x * per;
        row = base + mine;
        step = (int64_t)gridDim.x * per;
        turns = base < rows ? (int)((rows - base + step - 1) / step) : 0;
    }
};

// Over the L lanes of a row, or those of them that are in this warp.
template <typename F>
__device__ __forceinline__ float over_lanes(float x, int L, F&& both) {
    x = both(x, __shfl_xor_sync(0xffffffffu, x, 1));
    x = both(x, __shfl_xor_sync(0xffffffffu, x, 2));
    if (L > 4) x = both(x, __shfl_xor_sync(0xffffffffu, x, 4));
    if (L > 8) x = both(x, __shfl_xor_sync(0xffffffffu, x, 8));
    if (L > 16) x = both(x, __shfl_xor_sync(0xffffffffu, x, 16));
    return x;
}
struct Plus {
    __device__ __forceinline__ float operator()(float x, float y) const { return x + y; }
};
struct Max {
    __device__ __forceinline__ float operator()(float x, float y) const { return max_nan(x, y); }
};
// Of sizes, which as whole numbers have the order that they have as floats, NaN behind them:
// over a warp in one instruction (float32 in groups of 128 columns, 25 M elements, rows of 1024,
// 2048, 4096 and 8192: 89, 89, 90 and 92% of the copy rate, with five exchanges 88, 88, 90 and
// 93; over the halves of a warp it is slower, bf16 79 to 73).
__device__ __forceinline__ float over_lanes(float x, int L, Max both) {
    if (L >= 32) return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(x)));
    return over_lanes<Max>(x, L, static_cast<Max&&>(both));
}
// The largest of each piece over the groups of `lanes` lanes that hold the columns of a scale.
template <int K>
__device__ __forceinline__ void over_groups(float (&m)[kPieces], int lanes, int D, int LV) {
    auto all = [&](auto&& f) {
#pragma unroll
        for (int p = 0; p < kPieces; ++p) {
            if (K ? p >= K : p * LV >= D) break;
            m[p] = f(m[p]);
        }
    };
    auto with = [](int off) { return [off](float x) { return max_nan(x, __shfl_xor_sync(0xffffffffu, x, off)); }; };
    if (lanes == 32) {
        all([](float x) { return over_lanes(x, 32, Max()); });
        return;
    }
    all(with(1));
    all(with(2));
    if (lanes > 4) all(with(4));
    if (lanes > 8) all(with(8));
}
// Over a row the sum of a, and of b what F makes of it; `part` has two halves, used in turn, so
// that one barrier a turn is enough.
template <int N, typename F, int VEC>
__device__ __forceinline__ void row_both(float& a, float& b, F f, const Place<VEC>& at, float2 (*part)[N / 32], int turn) {
    a = over_lanes(a, at.L, Plus());
    b = over_lanes(b, at.L, f);
    if (at.L <= 32) return;
    float2* p = part[turn & 1];
    if ((threadIdx.x & 31) == 0) p[threadIdx.x >> 5] = make_float2(a, b);
    __syncthreads();
    const float2 s = p[at.first];
    a = s.x, b = s.y;
    for (int i = 1; i < at.warps; ++i) {
        const float2 s = p[at.first + i];
        a += s.x;
        b = f(b, s.y);
    }
}
template <int N, int VEC>
__device__ __forceinline__ float row_sum(float a, const Place<VEC>& at, float2 (*part)[N / 32], int turn) {
    a = over_lanes(a, at.L, Plus());
    if (at.L <= 32) return a;
    float2* p = part[turn & 1];
    if ((threadIdx.x & 31) == 0) p[threadIdx.x >> 5].x = a;
    __syncthreads();
    a = p[at.first].x;
    for (int i = 1; i < at.warps; ++i) a += p[at.first + i].x;
    return a;
}
template <int N, int VEC>
__device__ __forceinline__ float row_max(float m, const Place<VEC>& at, float (*part)[N / 32], int turn) {
    m = over_lanes(m, at.L, max_nan);
    if (at.L <= 32) return m;
    float* p = part[turn & 1];
    if ((threadIdx.x & 31) == 0) p[threadIdx.x >> 5] = m;
    __syncthreads();
    m = p[at.first];
    for (int i = 1; i < at.warps; ++i) m = max_nan(m, p[at.first + i]);
    return m;
}

// Two floats as e4m3 (nearest, ties to even, past 448: 448), the first in the lower byte.
__device__ __forceinline__ uint32_t e4m3x2(uint64_t p) {
    float lo, hi;
    uint16_t r;
    unpair(p, lo, hi);
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

constexpr float kLeast = 1.17549435e-38f;  // 2^-126, the least scale

// The 8-bit form.  With t = h w and m = max|t| over the group, y / scale = 448 t / m: the
// row's r is no part of it.  t (448 / m) in float32 is off by up to 8 of its last bits, which
// matters next to the middle between two e4m3 numbers only, where the 20 mantissa bits that
// e4m3 drops are near 10...0.  There (one element of 60000) 448 t is compared with the middle
// times m, both exactly, so that y8 is the number nearest to the exact quotient.  (Below 2^-6
// e4m3 drops more bits, and an element there may fall on either side of a middle that is
// within float32's error.)  In float64 that comparison made the kernel 1.8 times slower,
// rare as it is.
// How far a quotient's low 20 bits are behind the first that are near (times 2^12, which
// drops the other bits): up to kNear they are.
constexpr uint32_t kNear = 16u << 12;
__device__ __forceinline__ uint32_t behind(float q) { return __float_as_uint(q) * 4096u - (0x7fff8u << 12); }
// (x + res) w as two float32 numbers, the second what the first's roundings left out.
__device__ __forceinline__ float2 product_of(float x, float res, float w) {
    const float h = x + res, b = h - x, left = (x - (h - b)) + (res - b);
    const float t = h * w;
    return make_float2(t, fmaf(left, w, fmaf(h, w, -t)));
}
// q, near a middle, moved to the side of it on which 448 t / m is (m = most + left).
__device__ __forceinline__ float beside_middle(float q, float2 t, float most, float left) {
    const uint32_t at = (__float_as_uint(q) & 0x7ff00000u) | 0x80000u;
    const float middle = __uint_as_float(at), sign = copysignf(1.f, q);
    const float a = 448.f * fabsf(t.x), a1 = fmaf(448.f, fabsf(t.x), -a), b = middle * most, b1 = fmaf(middle, most, -b);
    const float d = (a - b) + ((a1 - b1) + fmaf(448.f, sign * t.y, -(middle * left)));
    return copysignf(__uint_as_float(d > 0.f ? at + 1 : d < 0.f ? at - 1 : at), q);
}

// What is needed rarely is not inlined: it would take the registers of every row.  x and res
// (0: no residual): the row's places in shared memory.
// The piece's 8-bit numbers from its quotients, those next to a middle decided exactly.
struct Quotients {
    uint64_t z[4];
};
template <typename TX, typename TR>
__device__ __noinline__ uint2 exact_piece(uint32_t x, uint32_t res, uint4 w, Quotients q, float most, float left) {
    constexpr int VEC = 16 / (int)sizeof(TR);
    uint64_t f[VEC / 2], g[VEC / 2], k[VEC / 2];
    Piece<TX, VEC>::load(x, f);
    if (res) Piece<TR, VEC>::load(res, g);
    Piece<TX, VEC>::unpack(w, k);
    uint32_t code[4] = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < VEC / 2; ++j) {
        float xv[2], rv[2] = {0.f, 0.f}, wv[2], z[2];
        unpair(f[j], xv[0], xv[1]);
        if (res) unpair(g[j], rv[0], rv[1]);
        unpair(k[j], wv[0], wv[1]);
        unpair(q.z[j], z[0], z[1]);
#pragma unroll
        for (int e = 0; e < 2; ++e)
            if (behind(z[e]) <= kNear) z[e] = beside_middle(z[e], product_of(xv[e], rv[e], wv[e]), most, left);
        code[j] = e4m3x2(pair(z[0], z[1]));
    }
    return make_uint2(code[0] | code[1] << 16, code[2] | code[3] << 16);
}
// What float32's rounding left out of the largest |t|, of the piece's elements that are it.
template <typename TX, typename TR>
__device__ __noinline__ float left_of(uint32_t x, uint32_t res, uint4 w, float most, float left) {
    constexpr int VEC = 16 / (int)sizeof(TR);
    uint64_t f[VEC / 2], g[VEC / 2], k[VEC / 2];
    Piece<TX, VEC>::load(x, f);
    if (res) Piece<TR, VEC>::load(res, g);
    Piece<TX, VEC>::unpack(w, k);
#pragma unroll
    for (int j = 0; j < VEC / 2; ++j) {
        float xv[2], rv[2] = {0.f, 0.f}, wv[2];
        unpair(f[j], xv[0], xv[1]);
        if (res) unpair(g[j], rv[0], rv[1]);
        unpair(k[j], wv[0], wv[1]);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float2 t = product_of(xv[e], rv[e], wv[e]);
            if (fabsf(t.x) == most) left = fmaxf(left, copysignf(1.f, t.x) * t.y);
        }
    }
    return left;
}

struct Scale {
    float scale;
    uint64_t by;  // what takes t, or y where `plain`, to 8 bits
    bool plain;   // m or the scale next to the end of float32's range, or not finite
};
// NaN stays NaN, and a group with an infinite scale is read back as NaN.
__device__ __forceinline__ Scale scale_of(float m, float r) {
    const float s = m * r * (1.f / 448.f);
    Scale c;
    c.scale = s < kLeast ? kLeast : s;
    c.plain = !(m >= 7.888609e-31f && s >= kLeast && s <= 3.402823466e38f);
    const float inverse = inverse_of(c.plain ? c.scale : m);
    c.by = twice(c.plain ? inverse : 448.f * inverse);
    return c;
}

struct NormDims {
    int64_t rows, x_stride, r_stride;
    int D, L;
    int group, shift;  // columns of a scale (D: a row's), and for groups of 32 to 128 their logarithm
    float eps;
};

// Threads an SM holds, and blocks of N of them.
constexpr int kPerSm = 512;
constexpr int per_sm(int N) { return kPerSm / N; }
constexpr int kFwdSlots = 2 * kPieces, kBwdSlots = 3 * kPieces;

// K: every lane holds K pieces of its row (0: as many as it has, some fewer than others).  Without
// branches between pieces they are worked on together; rows behind the last are computed from
// what lies in the ring, but not written.  (25 M elements in 8 bits, groups of 128, of the
// copy rate: 2048 columns of bf16 79 to 84%, 5120 75 to 83; a float32 stream 8192 78 to 88.)
template <typename TX, typename TR, int N, bool kQuant, int K>
__global__ void __launch_bounds__(N, per_sm(N))
add_norm_fwd_kernel(NormDims d, const TX* __restrict__ x, const TR* res, const TX* __restrict__ w, TR* h,
                    void* __restrict__ y, float* __restrict__ scales) {
    constexpr int VEC = 16 / (int)sizeof(TR), S = kStages;
    using PX = Piece<TX, VEC>;
    using PR = Piece<TR, VEC>;
    await_previous();
    extern __shared__ __align__(16) unsigned char sm[];
    __shared__ float2 part[2][N / 32];
    __shared__ float lefts[kQuant && sizeof(TR) == 4 ? 2 : 1][N / 32];
    const Slots<kFwdSlots, S, N> ring(sm);
    const Place<VEC> at(d.rows, d.D, d.L);
    const float inv_d = 1.f / d.D;
    // where the thread's pieces of the row copied and of the row worked on are
    const TX* x_next = x + at.row * d.x_stride + at.c0;
    const TR* r_next = res ? res + at.row * d.r_stride + at.c0 : nullptr;
    const int64_t x_step = at.step * d.x_stride, r_step = at.step * d.r_stride, step = at.step * d.D;
    int64_t now = at.row, next = now, out = now * d.D + at.c0;
    auto issue = [&](int slot) {
        if (next < d.rows) {
#pragma unroll
            for (int p = 0; p < kPieces; ++p) {
                if (K ? p >= K : p >= at.n) break;
                PX::copy(ring.at(slot, p), x_next + p * at.LV);
                if (res) PR::copy(ring.at(slot, kPieces + p), r_next + p * at.LV);
            }
        }
        commit();
        next += at.step, x_next += x_step, r_next += r_step;
    };
    uint4 wv[kPieces];
#pragma unroll
    for (int p = 0; p < kPieces; ++p) wv[p] = (K ? p < K : p < at.n) ? PX::ldg(w + at.c0 + p * at.LV) : make_uint4(0, 0, 0, 0);
    if (at.turns) {
#pragma unroll
        for (int i = 0; i < S - 1; ++i) issue(i);
    }
    for (int turn = 0, slot = 0, fill = S - 1; turn < at.turns; ++turn, now += at.step, out += step) {
        issue(fill);
        fill = fill + 1 == S ? 0 : fill + 1;
        wait_group<S - 1>();
        const bool live = now < d.rows;
        const int n = K ? K : live ? at.n : 0;
        uint64_t a[kPieces][VEC / 2], ss = twice(0.f);
#pragma unroll
        for (int p = 0; p < kPieces; ++p) {
            if (p >= n) break;
            PX::load(ring.at(slot, p), a[p]);
            if (res) {
                uint64_t s[VEC / 2];
                PR::load(ring.at(slot, kPieces + p), s);
#pragma unroll
                for (int j = 0; j < VEC / 2; ++j) a[p][j] = add2(a[p][j], s[j]);
                if (h && (!K || live)) PR::store(h + out + p * at.LV, a[p]);
            }
#pragma unroll
            for (int j = 0; j < VEC / 2; ++j) ss = fma2(a[p][j], a[p][j], ss);
        }
        if constexpr (!kQuant) {
            const float r = rsqrtf(fmaf(row_sum<N>(sum2(ss), at, part, turn), inv_d, d.eps));
#pragma unroll
            for (int p = 0; p < kPieces; ++p) {
                if (p >= n) break;
                uint64_t f[VEC / 2];
                PX::unpack(wv[p], f);
#pragma unroll
                for (int j = 0; j < VEC / 2; ++j) a[p][j] = mul2(mul2(a[p][j], twice(r)), f[j]);
                if (!K || live) PX::store((TX*)y + out + p * at.LV, a[p]);
            }
        } else {
            constexpr bool kWide = sizeof(TR) == 4;
            auto place = [&](int p) { return res ? ring.at(slot, kPieces + p) : 0u; };
            // the piece's t in the place of h, and its largest |t|
            auto weighted = [&](int p) {
                uint64_t f[VEC / 2];
                PX::unpack(wv[p], f);
                float m = 0.f;
#pragma unroll
                for (int j = 0; j < VEC / 2; ++j) {
                    a[p][j] = mul2(a[p][j], f[j]);
                    m = abs_max(a[p][j], m);
                }
                return m;
            };
            // What the float32 t leave out of the group's largest |t|: with a float32 stream it is
            // taken from the elements that are the largest, where a quotient next to a middle
            // asks for it.  Of bf16, whose sums and products mostly need no more bits than
            // float32 has, the largest counts as float32 holds it: where it is rounded, by up to
            // 2^-24, a quotient as close as that to a middle may fall on either side.
            auto left_out = [&](int p, float most, float left) {
                bool is = false;
#pragma unroll
                for (int j = 0; j < VEC / 2; ++j) {
                    float t0, t1;
                    unpair(a[p][j], t0, t1);
                    is = is || fabsf(t0) == most || fabsf(t1) == most;
                }
                return is ? left_of<TX, TR>(ring.at(slot, p), place(p), wv[p], most, left) : left;
            };
            // the piece's numbers, and whether a quotient is next to a middle
            auto coded = [&](int p, const Scale& c, float r, uint2& code, Quotients& z) {
                uint32_t q[4] = {0, 0, 0, 0}, near = kNear + 1;
                if (c.plain) {
#pragma unroll
                    for (int j = 0; j < VEC / 2; ++j) a[p][j] = mul2(a[p][j], twice(r));
                }
#pragma unroll
                for (int j = 0; j < VEC / 2; ++j) {
                    z.z[j] = mul2(a[p][j], c.by);
                    float z0, z1;
                    unpair(z.z[j], z0, z1);
                    near = min(near, min(behind(z0), behind(z1)));
                    q[j] = e4m3x2(z.z[j]);
                }
                code = make_uint2(q[0] | q[1] << 16, q[2] | q[3] << 16);
                return near <= kNear && !c.plain;
            };
            auto exact = [&](int p, float most, float left, const Quotients& z) {
                return exact_piece<TX, TR>(ring.at(slot, p), place(p), wv[p], z, most, left);
            };
            auto store = [&](int p, const uint2& code) {
                if (K && !live) return;
                unsigned char* to = (unsigned char*)y + out + p * at.LV;
                if constexpr (VEC == 8) *reinterpret_cast<uint2*>(to) = code;
                else *reinterpret_cast<uint32_t*>(to) = code.x;
            };
            // Quotients next to a middle are decided behind all pieces: a call between two keeps
            // them from being worked on together (25 M elements of a float32 stream in groups of
            // 128, 2048 columns: 82 to 91% of the copy rate).  Only bf16 in lanes of different
            // numbers of pieces, which branch between them all the same, loses by it (1 to 2%).
            uint32_t near = 0;  // a bit a piece
            auto first = [&](int p, const Scale& c, float r, float most) {
                uint2 code;
                Quotients z;
                const bool is = coded(p, c, r, code, z);
                if constexpr (kWide || K) near |= (uint32_t)is << p;
                else if (is) code = exact(p, most, 0.f, z);
                store(p, code);
            };
            auto again = [&](int p, const Scale& c, float r, float most, float left) {
                uint2 code;
                Quotients z;
                coded(p, c, r, code, z);
                store(p, exact(p, most, left, z));
            };
            if (d.group < d.D) {
                const int lanes = d.group / VEC;  // a group's, neighbours: 4 to 32 of them
                float m[kPieces];
#pragma unroll
                for (int p = 0; p < kPieces; ++p) m[p] = p < n ? weighted(p) : 0.f;
                over_groups<K>(m, lanes, d.D, at.LV);
                const float r = rsqrtf(fmaf(row_sum<N>(sum2(ss), at, part, turn), inv_d, d.eps));
#pragma unroll
                for (int p = 0; p < kPieces; ++p) {
                    if (p >= n) break;
                    const Scale c = scale_of(m[p], r);
                    if ((!K || live) && ((at.c0 + p * at.LV) & (d.group - 1)) == 0) scales[(out + p * at.LV) >> d.shift] = c.scale;
                    first(p, c, r, m[p]);
                }
                if (kWide ? __any_sync(0xffffffffu, near) : near) {
#pragma unroll
                    for (int p = 0; p < kPieces; ++p) {
                        const bool mine = near >> p & 1;
                        float left = 0.f;
                        if constexpr (kWide) {
                            if (!__any_sync(0xffffffffu, mine)) continue;
                            left = over_lanes(p < n ? left_out(p, m[p], -FLT_MAX) : -FLT_MAX, lanes, max_nan);
                        }
                        if (mine) again(p, scale_of(m[p], r), r, m[p], left);
                    }
                }
            } else {
                float m = 0.f;
#pragma unroll
                for (int p = 0; p < kPieces; ++p) {
                    if (p >= n) break;
                    m = max_nan(m, weighted(p));
                }
                // the largest |t| needs nothing of the row's norm: both in one exchange
                float sum = sum2(ss);
                row_both<N>(sum, m, Max(), at, part, turn);
                const float r = rsqrtf(fmaf(sum, inv_d, d.eps));
                const Scale c = scale_of(m, r);
                if (at.c0 == 0 && (K ? live : n > 0)) scales[now] = c.scale;
#pragma unroll
                for (int p = 0; p < kPieces; ++p) {
                    if (p >= n) break;
                    first(p, c, r, m);
                }
                float left = 0.f;
                if constexpr (kWide) {
                    if (at.L > 32 ? __syncthreads_or(near) : __any_sync(0xffffffffu, near)) {
                        left = -FLT_MAX;
#pragma unroll
                        for (int p = 0; p < kPieces; ++p) {
                            if (p >= n) break;
                            left = left_out(p, m, left);
                        }
                        left = row_max<N>(left, at, lefts, turn);
                    }
                }
                if (near) {
#pragma unroll
                    for (int p = 0; p < kPieces; ++p)
                        if (near >> p & 1) again(p, c, r, m, left);
                }
            }
        }
        slot = slot + 1 == S ? 0 : slot + 1;
    }
    wait_group<0>();  // no copy outlives the block
}

// Each block leaves one row of column sums in sums [gridDim.x][D]; the blocks of a cluster
// (kCluster, the whole grid) add theirs up to dw, each some columns.
template <typename TX, typename TR, int N, bool kCluster, int K>
__global__ void __launch_bounds__(N, per_sm(N))
add_norm_bwd_kernel(NormDims d, const TR* __restrict__ h, const TX* __restrict__ w, const TX* __restrict__ dy,
                    const TR* __restrict__ dh, TX* __restrict__ dx, TR* __restrict__ dr, TX* __restrict__ dw, float* __restrict__ sums) {
    constexpr int VEC = 16 / (int)sizeof(TR), S = kStages;
    using PX = Piece<TX, VEC>;
    using PR = Piece<TR, VEC>;
    await_previous();
    extern __shared__ __align__(16) unsigned char sm[];
    __shared__ float2 part[2][N / 32];
    const Slots<kBwdSlots, S, N> ring(sm);
    const Place<VEC> at(d.rows, d.D, d.L);
    const float inv_d = 1.f / d.D;
    const TR* h_next = h + at.row * d.r_stride + at.c0;
    const int64_t h_step = at.step * d.r_stride, step = at.step * d.D;
    int64_t now = at.row, next = now, out = now * d.D + at.c0, in = out;
    auto issue = [&](int slot) {
        if (next < d.rows) {
#pragma unroll
            for (int p = 0; p < kPieces; ++p) {
                if (K ? p >= K : p >= at.n) break;
                PR::copy(ring.at(slot, p), h_next + p * at.LV);
                PX::copy(ring.at(slot, kPieces + p), dy + in + p * at.LV);
                if (dh) PR::copy(ring.at(slot, 2 * kPieces + p), dh + in + p * at.LV);
            }
        }
        commit();
        next += at.step, h_next += h_step, in += step;
    };
    uint4 wv[kPieces];
    uint64_t acc[kPieces][VEC / 2];
#pragma unroll
    for (int p = 0; p < kPieces; ++p) {
        wv[p] = (K ? p < K : p < at.n) ? PX::ldg(w + at.c0 + p * at.LV) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int j = 0; j < VEC / 2; ++j) acc[p][j] = twice(0.f);
    }
    if (at.turns) {
#pragma unroll
        for (int i = 0; i < S - 1; ++i) issue(i);
    }
    for (int turn = 0, slot = 0, fill = S - 1; turn < at.turns; ++turn, now += at.step, out += step) {
        issue(fill);
        fill = fill + 1 == S ? 0 : fill + 1;
        wait_group<S - 1>();
        const bool live = now < d.rows;
        const int n = K ? K : live ? at.n : 0;
        uint64_t ss = twice(0.f), tx = ss;
#pragma unroll
        for (int p = 0; p < kPieces; ++p) {
            if (p >= n) break;
            uint64_t a[VEC / 2], g[VEC / 2], f[VEC / 2];
            PR::load(ring.at(slot, p), a);
            PX::load(ring.at(slot, kPieces + p), g);
            PX::unpack(wv[p], f);
#pragma unroll
            for (int j = 0; j < VEC / 2; ++j) {
                ss = fma2(a[j], a[j], ss);
                tx = fma2(mul2(g[j], f[j]), a[j], tx);
            }
        }
        float sq = sum2(ss), st = sum2(tx);
        row_both<N>(sq, st, Plus(), at, part, turn);
        const float r = rsqrtf(fmaf(sq, inv_d, d.eps));
        // mean(t hh) = r mean(t h), times r of hh
        const uint64_t m = twice(-st * r * r * inv_d), r2 = twice(r);
        // the pieces are read again from shared memory: held in registers over the sum they
        // would leave room for half of the warps
#pragma unroll
        for (int p = 0; p < kPieces; ++p) {
            if (K ? !live || p >= K : p >= n) break;
            uint64_t a[VEC / 2], g[VEC / 2], f[VEC / 2];
            PR::load(ring.at(slot, p), a);
            PX::load(ring.at(slot, kPieces + p), g);
            PX::unpack(wv[p], f);
#pragma unroll
            for (int j = 0; j < VEC / 2; ++j) {
                acc[p][j] = fma2(mul2(g[j], a[j]), r2, acc[p][j]);
                a[j] = mul2(fma2(a[j], m, mul2(g[j], f[j])), r2);
            }
            if (dh) {
                PR::load(ring.at(slot, 2 * kPieces + p), g);
#pragma unroll
                for (int j = 0; j < VEC / 2; ++j) a[j] = add2(a[j], g[j]);
            }
            PX::store(dx + out + p * at.LV, a);
            if constexpr (sizeof(TX) != sizeof(TR)) PR::store(dr + out + p * at.LV, a);
        }
        slot = slot + 1 == S ? 0 : slot + 1;
    }
    wait_group<0>();
    // the sums of a warp's rows; then each warp or row of warps leaves its own, and a thread adds
    // four columns' in a fixed order: the same call gives the same bits
    const bool part_warp = at.L < 32;
    if (part_warp) {
#pragma unroll
        for (int p = 0; p < kPieces; ++p)
#pragma unroll
            for (int j = 0; j < VEC / 2; ++j) {
                float lo, hi;
                unpair(acc[p][j], lo, hi);
                for (int off = at.L; off < 32; off *= 2) {
                    lo += __shfl_xor_sync(0xffffffffu, lo, off);
                    hi += __shfl_xor_sync(0xffffffffu, hi, off);
                }
                acc[p][j] = pair(lo, hi);
            }
    }
    __syncthreads();
    float* col = (float*)sm;
    const int wide = part_warp ? 32 : at.L, parts = N / wide;
    if (!part_warp || (int)(threadIdx.x & 31) < at.L) {
        float* to = col + (int)threadIdx.x / wide * d.D + at.c0;
#pragma unroll
        for (int p = 0; p < kPieces; ++p) {
            if (p >= at.n) break;
#pragma unroll
            for (int j = 0; j < VEC / 4; ++j) {
                const uint64_t four[2] = {acc[p][2 * j], acc[p][2 * j + 1]};
                *reinterpret_cast<uint4*>(to + p * at.LV + 4 * j) = put(four);
            }
        }
    }
    __syncthreads();
    for (int c = 4 * threadIdx.x; c < d.D; c += 4 * N) {
        float4 s = *reinterpret_cast<const float4*>(col + c);
        for (int i = 1; i < parts; ++i) {
            const float4 x = *reinterpret_cast<const float4*>(col + i * d.D + c);
            s.x += x.x, s.y += x.y, s.z += x.z, s.w += x.w;
        }
        *reinterpret_cast<float4*>(kCluster ? col + c : sums + (int64_t)blockIdx.x * d.D + c) = s;
    }
    if constexpr (kCluster) {
        cluster_sync();
        for (int c = blockIdx.x * N + threadIdx.x; c < d.D; c += gridDim.x * N) store1(dw + c, cluster_sum(col + c));
        cluster_sync();  // no block leaves before the others have read its sums
    }
}

// Whether every lane has three pieces, or every lane four (lane: a piece of all).
bool even(int D, int lane) { return D == 3 * lane || D == 4 * lane; }

// Lanes a row of pieces of VEC elements takes, kPieces a lane: a warp at least, or two pieces
// a lane of fewer (35 x 1755 rows of 512 bf16 with 16 lanes 86.3 us forward and backward, with
// 32 83.3).  The 8-bit form, which computes more, takes kPieces from 8 lanes on (29 x 1429 rows
// of 272 with 16 lanes 15.9 us, with 32 23.2), but all of a group of columns with a scale.
// Past a warp: a power of two, but where `most`, the most that let an SM hold as many rows as
// the fewest would: 96 of them hold 288 or 384 pieces in five rows where 128 hold four.  Of 25 M
// elements in the 8-bit form rows of 2304 bf16 so take 81% of the copy rate for 66 in groups of
// 128 and 87 for 80 without, with a float32 stream 83 for 69 and 88 for 73, of float32 91 for 82;
// of 6144 bf16 192 lanes take 79 and 85% and 256, the most of two rows, 82 and 86.  Lanes that share
// the pieces evenly come before more lanes (4608 float32 78 to 86%, 7168 bf16 73 to 78).  Rows
// without a residual, which have less in flight, gain (2304 bf16 85 to 107%, partly from L2);
// those with one lose (89 to 86%), and so does the backward (2304 bf16 with a float32 stream 91
// to 83%).
int lanes_of(int D, int vec, bool quant, int group, bool most) {
    int L = 8;
    if (quant)
        while (L * vec < group) L *= 2;
    else
        while (L < 32 && L * 2 * vec < D) L *= 2;
    while ((L < 32 || !most) && L * kPieces * vec < D) L *= 2;
    if (L * kPieces * vec >= D) return L;
    const int warp = 32 * kPieces * vec, fewest = (D + warp - 1) / warp * 32, rows = kPerSm / fewest;
    const int widest = kPerSm / rows / 32 * 32;
    for (int L = widest; L >= fewest; L -= 32)
        if (even(D, L * vec)) return L;
    return widest;
}

template <typename TX, typename TR, int N, bool kQuant, int K>
cudaError_t fwd_k(const AddNormCall& c, const NormDims& d, cudaStream_t st) {
    auto kern = add_norm_fwd_kernel<TX, TR, N, kQuant, K>;
    constexpr int smem = Slots<kFwdSlots, kStages, N>::BYTES;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(kern, smem, done);
    if (e != cudaSuccess) return e;
    const int per = d.L < N ? N / d.L : 1, threads = per * d.L;
    const int64_t want = (d.rows + per - 1) / per, cap = (int64_t)sm_count() * per_sm(threads);
    return launch_dependent(kern, dim3((unsigned)(want < cap ? want : cap)), threads, smem, st, d, (const TX*)c.x,
                            (const TR*)c.res, (const TX*)c.w, (TR*)c.h, c.y, c.scales);
}

template <typename TX, typename TR, int N, bool kQuant>
cudaError_t fwd(const AddNormCall& c, const NormDims& d, cudaStream_t st) {
    const int lane = 16 / (int)sizeof(TR) * d.L;
    if (!even(d.D, lane)) return fwd_k<TX, TR, N, kQuant, 0>(c, d, st);
    return d.D == 3 * lane ? fwd_k<TX, TR, N, kQuant, 3>(c, d, st) : fwd_k<TX, TR, N, kQuant, 4>(c, d, st);
}

template <typename TX, typename TR, int N>
cudaError_t bwd(const AddNormCall& c, const NormDims& d, cudaStream_t st) {
    constexpr int smem = Slots<kBwdSlots, kStages, N>::BYTES;
    static_assert(smem >= N * kPieces * (16 / (int)sizeof(TR)) * 4, "every thread's column sums fit the ring");
    static std::atomic<uint64_t> done{0}, done1{0};
    const TR *h = (const TR*)c.h_in, *dh = (const TR*)c.dh;
    const TX *w = (const TX*)c.w, *dy = (const TX*)c.dy;
    if (c.grid.cluster)
        return launch_one_cluster(add_norm_bwd_kernel<TX, TR, N, true, 0>, c.grid.blocks, N, smem, done1, st, d, h, w, dy, dh,
                                  (TX*)c.dx, (TR*)c.dr, (TX*)c.dw, c.part);
    auto launch = [&](auto kern, std::atomic<uint64_t>& done) {
        cudaError_t e = allow_smem(kern, smem, done);
        if (e != cudaSuccess) return e;
        return launch_dependent(kern, dim3((unsigned)c.grid.blocks), N, smem, st, d, h, w, dy, dh, (TX*)c.dx, (TR*)c.dr,
                                (TX*)c.dw, c.part);
    };
    static std::atomic<uint64_t> done3{0}, done4{0};
    const int lane = 16 / (int)sizeof(TR) * d.L;
    if (!even(d.D, lane)) return launch(add_norm_bwd_kernel<TX, TR, N, false, 0>, done);
    return d.D == 3 * lane ? launch(add_norm_bwd_kernel<TX, TR, N, false, 3>, done3)
                           : launch(add_norm_bwd_kernel<TX, TR, N, false, 4>, done4);
}

template <typename TX, typename TR, bool kQuant>
cudaError_t fwd_n(const AddNormCall& c, const NormDims& d, cudaStream_t st) {
    static_assert(kAddNormMost <= 256 * kPieces * 8, "rows of bf16 take 256 lanes at most");
    if constexpr (sizeof(TR) == 4)
        if (d.L > 256) return fwd<TX, TR, 512, kQuant>(c, d, st);
    return d.L <= 128 ? fwd<TX, TR, 128, kQuant>(c, d, st) : fwd<TX, TR, 256, kQuant>(c, d, st);
}

template <typename TX, typename TR>
cudaError_t launch_t(const AddNormCall& c, AddNormKind kind, cudaStream_t st) {
    const bool quant = kind == AddNormKind::QUANT, most = quant || (kind == AddNormKind::FWD && !c.res);
    const NormDims d{c.rows, c.x_stride, c.r_stride, c.D, lanes_of(c.D, 16 / (int)sizeof(TR), quant, c.group, most),
                     c.group ? c.group : c.D, c.group == 32 ? 5 : c.group == 64 ? 6 : 7, c.eps};
    switch (kind) {
        case AddNormKind::FWD: return fwd_n<TX, TR, false>(c, d, st);
        case AddNormKind::QUANT: return fwd_n<TX, TR, true>(c, d, st);
        default:
            if constexpr (sizeof(TR) == 4)
                if (d.L > 256) return bwd<TX, TR, 512>(c, d, st);
            return bwd<TX, TR, 256>(c, d, st);
    }
}

}  // namespace

// Where every row has a place in one turn of a cluster, the backward is one cluster and one
// launch: 1 to 16 blocks of rows of 768 to 8192 elements take 3.8 to 5.9 us, as two launches 4.1 to
// 5.8, but 1.2 us less of the host's time, which bounds such calls, and no workspace; of two
// turns (bf16) 5.3 to 7.1, as two launches 4.7 to 5.5.
AddNormGrid add_norm_bwd_grid(int64_t rows, int D, int wide) {
    const int L = lanes_of(D, 16 / wide, false, 0, false), n = L <= 256 ? 256 : 512;
    const int64_t per = n / L, want = (rows + per - 1) / per, cap = (int64_t)sm_count() * per_sm(n);
    if (one_cluster(want)) return {(int)(want < 1 ? 1 : want), true};
    return {(int)(want < cap ? want : cap), false};
}

std::atomic<int> test_cluster_limit{0};

// Asked of the kernel that takes most of an SM (512 threads and 192 KB; as all that run in one
// cluster it has an SM to itself), once for a context.  Where no GPU answers, the largest.  (This
// GPU as a whole: 16; a green context of 8, 16 or 32 of its SMs: 8.)
int cluster_limit() {
    if (const int n = test_cluster_limit.load(std::memory_order_relaxed)) return n;
    static std::atomic<uint64_t> known[4];  // a context's number times 256, and its limit
    const uint64_t context = context_number();
    std::atomic<uint64_t>& mine = known[context & 3];
    const uint64_t was = mine.load(std::memory_order_relaxed);
    if (context && was >> 8 == context) return (int)(was & 255);
    auto kern = add_norm_bwd_kernel<float, float, 512, true, 0>;
    constexpr int smem = Slots<kBwdSlots, kStages, 512>::BYTES;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return kMostCluster;
    }
    int n = kMostCluster;
    for (; n > 1; n /= 2) {
        cudaLaunchConfig_t c = {};
        c.gridDim = dim3((unsigned)n);
        c.blockDim = dim3(512);
        c.dynamicSmemBytes = smem;
        cudaLaunchAttribute a;
        a.id = cudaLaunchAttributeClusterDimension;
        a.val.clusterDim.x = (unsigned)n;
        a.val.clusterDim.y = a.val.clusterDim.z = 1;
        c.attrs = &a;
        c.numAttrs = 1;
        int placed = 0;
        if (cudaOccupancyMaxActiveClusters(&placed, kern, &c) != cudaSuccess) cudaGetLastError();
        else if (placed > 0) break;
    }
    if (context) mine.store(context << 8 | (uint64_t)n, std::memory_order_relaxed);
    return n;
}

cudaError_t launch_add_norm(const AddNormCall& c, InType ty, InType stream_ty, AddNormKind kind, cudaStream_t st) {
    if (ty == InType::F32) return launch_t<float, float>(c, kind, st);
    return stream_ty == InType::BF16 ? launch_t<__nv_bfloat16, __nv_bfloat16>(c, kind, st)
                                     : launch_t<__nv_bfloat16, float>(c, kind, st);
}

}  // namespace gdn
