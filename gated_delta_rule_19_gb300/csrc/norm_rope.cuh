// norm_rope.cuh -- RMS norm of every head's query and key row with the position's
// rotation in the same pass, and its gradients: the step in front of linear
// attention, as prologue.cu is the step in front of the delta rule.
//
// Row x of D elements, weight w, r = (mean x^2 + eps)^(-1/2), n = x r w; with c, s the
// cosine and sine of the token's position for pair p:
//   (y1, y2) = (n1 c - n2 s, n2 c + n1 s)     for the R / 2 pairs, y = n elsewhere,
// pair p being elements (p, p + R/2), or (2p, 2p + 1) when interleaved.  Backward, with
// dn = the rotation of dy by the opposite angle, xh = x r and t = dn w:
//   dw = sum over rows of dn xh,      dx = r (t - xh mean(t xh)).
// A group of lanes holds a row (rows.cuh), each lane with a slot of two 16-byte pieces:
// slot u has pieces (u, u + R/(2 VEC)) of the rotated part, so that in the first order
// both elements of a pair are in one lane, and likewise of the rest.  An item of a group
// is kHeads heads of one token, which share the angles' pieces.
//
// With several axes a token has a position on each of up to four, and every pair takes its
// angle from the tables' row of one of them.  The calls of one position (norm_rope.cu,
// kAxes 0) and of several (norm_rope_axes.cu) are compiled apart, and those in three forms.
// Where every unit of angles that lie together and are copied together belongs to one axis
// (kAxes 1), a lane keeps the positions of its two units' axes.  Else a lane of a few tokens'
// calls keeps those of all axes and copies angle by angle (kAxes 2), and for many tokens a
// kernel in front gathers each token's angles, once for all of its heads (kAxes 3).
#pragma once

#include "gdn_internal.h"
#include "rows.cuh"

namespace gdn {
namespace {

using namespace rows;

// What a group works on: item i of one side (queries or keys) is up to `per` heads of
// token i / blocks, the heads shared evenly among the blocks.
template <typename T>
struct Side {
    const T* x;   // rows, `stride` elements from token to token
    const T* w;   // [D]
    const T* dy;  // backward: [tokens, H, D]
    T* out;       // y or dx, [tokens, H, D]
    T* dw;        // backward in one cluster (kAxes > 0): the weight's gradient; else NULL
    int64_t stride;
    int H, blocks, per;
};

struct RopeDims {
    int64_t tokens;
    int T, D, R, rows;  // rows: of the cosine and sine tables
    float eps;
};

struct Tables {
    const float *cos, *sin;
    const int32_t* pos;  // or NULL: the token's place in its sequence; kAxes > 0: [axes][tokens]
    int axes;            // kAxes > 0: the positions of a token, and the pairs' axes
    AxesMap map;
};

// The table row of a token.
__device__ __forceinline__ int position(const RopeDims& d, const Tables& t, int64_t tok) {
    return t.pos ? t.pos[tok] : (int)(tok % d.T);
}

// The pair of a lane's angle j: its slot's pairs in order, or interleaved those of the first
// piece, then those of the second, a quarter of the row behind.
template <int VEC, bool kInter>
__device__ __forceinline__ int pair_of(const RopeDims& d, int u, int j) {
    if (!kInter) return u * VEC + j;
    return u * (VEC / 2) + (j < VEC / 2 ? j : d.R / 4 + j - VEC / 2);
}

// Angles that are copied together: four, or the two that lie together of interleaved float32.
template <int VEC, bool kInter>
constexpr int kUnit = kInter && VEC == 4 ? 2 : 4;

__device__ __forceinline__ uint32_t axis_of(const AxesMap& m, int pair) {
    const int word = pair >> 5;
    const uint64_t w = word < 2 ? word == 0 ? m.w[0] : m.w[1] : word == 2 ? m.w[2] : m.w[3];
    return (uint32_t)(w >> (2 * (pair & 31))) & 3;
}

// Where a token's angles are.  One position: its row of the tables.
template <int VEC, bool kInter, int kAxes>
struct Where {
    int pos = 0;
    __device__ __forceinline__ Where(const RopeDims&, const Tables&, int, bool) {}
    __device__ __forceinline__ void move(const RopeDims& d, const Tables& t, int64_t tok) { pos = position(d, t, tok); }
};
// Gathered angles: the token's own row.
template <int VEC, bool kInter>
struct Where<VEC, kInter, 3> {
    int pos = 0;
    __device__ __forceinline__ Where(const RopeDims&, const Tables&, int, bool) {}
    __device__ __forceinline__ void move(const RopeDims&, const Tables&, int64_t tok) { pos = (int)tok; }
};
// The rows of the lane's units.
template <int VEC, bool kInter>
struct Where<VEC, kInter, 1> {
    static constexpr int N = VEC / kUnit<VEC, kInter>;
    const int32_t* from[N];  // the axis's positions
    int pos[N];
    __device__ __forceinline__ Where(const RopeDims& d, const Tables& t, int u, bool turns) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            from[i] = t.pos;
            pos[i] = 0;
            if (turns) from[i] += axis_of(t.map, pair_of<VEC, kInter>(d, u, i * kUnit<VEC, kInter>)) * d.tokens;
        }
    }
    __device__ __forceinline__ void move(const RopeDims&, const Tables&, int64_t tok) {
#pragma unroll
        for (int i = 0; i < N; ++i) pos[i] = from[i][tok];
    }
};
// The rows of all axes, and the axes of the lane's VEC pairs, two bits each.
template <int VEC, bool kInter>
struct Where<VEC, kInter, 2> {
    int pos[4] = {0, 0, 0, 0};
    uint32_t axis = 0;
    __device__ __forceinline__ Where(const RopeDims& d, const Tables& t, int u, bool turns) {
        if (!turns) return;
#pragma unroll
        for (int j = 0; j < VEC; ++j) axis |= axis_of(t.map, pair_of<VEC, kInter>(d, u, j)) << (2 * j);
    }
    __device__ __forceinline__ void move(const RopeDims& d, const Tables& t, int64_t tok) {
#pragma unroll
        for (int a = 0; a < 4; ++a)
            if (a < t.axes) pos[a] = t.pos[a * d.tokens + tok];
    }
    // the row of angle j
    __device__ __forceinline__ int row(int j) const {
        const uint32_t a = axis >> (2 * j) & 3;
        return a < 2 ? a == 0 ? pos[0] : pos[1] : a == 2 ? pos[2] : pos[3];
    }
};

// copy_angles (below) for several axes.  A position outside the tables gives its own pairs
// NaN.
template <int VEC, bool kInter, typename R>
__device__ __forceinline__ void copy_angles(const R& ring, int slot, int p0, const RopeDims& d, const Tables& t,
                                            const Where<VEC, kInter, 1>& at, int u, bool turns) {
    if (!turns) return;
    const float nan = __int_as_float(0x7fc00000);
    constexpr int U = kUnit<VEC, kInter>;
#pragma unroll
    for (int i = 0; i < VEC / U; ++i) {
        const int row = at.pos[i], p = p0 + i * U / 4;
        if (row < 0 || row >= d.rows) {
#pragma unroll
            for (int j = 0; j < U; ++j) {
                ring.put4(slot, p, i * U % 4 + j, nan);
                ring.put4(slot, p + VEC / 4, i * U % 4 + j, nan);
            }
            continue;
        }
        const int64_t e = (int64_t)row * (d.R / 2) + pair_of<VEC, kInter>(d, u, i * U);
        if constexpr (U == 4) {
            ring.copy_shared(slot, p, t.cos + e);
            ring.copy_shared(slot, p + VEC / 4, t.sin + e);
        } else {
            ring.copy8(slot, p, i, t.cos + e);
            ring.copy8(slot, p + VEC / 4, i, t.sin + e);
        }
    }
}
// Four angles of one row that lie together in one copy, others by 4 bytes each: the four at
// the border of two axes' pairs, and all where the axes take turns.
template <int VEC, bool kInter, typename R>
__device__ __forceinline__ void copy_angles(const R& ring, int slot, int p0, const RopeDims& d, const Tables& t,
                                            const Where<VEC, kInter, 2>& at, int u, bool turns) {
    if (!turns) return;
    const float nan = __int_as_float(0x7fc00000);
#pragma unroll
    for (int q = 0; q < VEC / 4; ++q) {
        const uint32_t axes = at.axis >> (8 * q) & 255;
        if (!(kInter && VEC == 4) && axes == (axes & 3) * 0x55) {
            const int row = at.row(4 * q);
            const int64_t e = (int64_t)row * (d.R / 2) + pair_of<VEC, kInter>(d, u, 4 * q);
            if (row < 0 || row >= d.rows) {
                ring.put(slot, p0 + q, nan);
                ring.put(slot, p0 + VEC / 4 + q, nan);
            } else {
                ring.copy_shared(slot, p0 + q, t.cos + e);
                ring.copy_shared(slot, p0 + VEC / 4 + q, t.sin + e);
            }
            continue;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int row = at.row(4 * q + j);
            const int64_t e = (int64_t)row * (d.R / 2) + pair_of<VEC, kInter>(d, u, 4 * q + j);
            if (row < 0 || row >= d.rows) {
                ring.put4(slot, p0 + q, j, nan);
                ring.put4(slot, p0 + VEC / 4 + q, j, nan);
            } else {
                ring.copy4(slot, p0 + q, j, t.cos + e);
                ring.copy4(slot, p0 + VEC / 4 + q, j, t.sin + e);
            }
        }
    }
}

// The VEC cosines of a slot's pairs, then the sines, into the ring from piece p0 on; a
// position outside the tables gives NaN, so that the token's rows show it.  In the
// first order pair j is elements j of the two pieces; interleaved, the pairs of the
// first piece come first, then those of the second, a quarter of the row behind.
template <int VEC, bool kInter, typename R, int A>
__device__ __forceinline__ void copy_angles(const R& ring, int slot, int p0, const RopeDims& d, const Tables& t,
                                            const Where<VEC, kInter, A>& at, int u, bool turns) {
    static_assert(A == 0 || A == 3, "one row for all pairs");
    if (!turns) return;
    const int pos = at.pos;
    if (pos < 0 || pos >= d.rows) {
#pragma unroll
        for (int j = 0; j < VEC / 2; ++j) ring.put(slot, p0 + j, __int_as_float(0x7fc00000));
        return;
    }
    const int64_t row = (int64_t)pos * (d.R / 2);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const float* f = (k ? t.sin : t.cos) + row + (kInter ? u * (VEC / 2) : u * VEC);
        const int p = p0 + k * (VEC / 4);
        if (!kInter) {
#pragma unroll
            for (int j = 0; j < VEC / 4; ++j) ring.copy_shared(slot, p + j, f + 4 * j);
        } else if (VEC == 8) {
            ring.copy_shared(slot, p, f);
            ring.copy_shared(slot, p + VEC / 4 - 1, f + d.R / 4);
        } else {
            ring.copy8(slot, p, 0, f);
            ring.copy8(slot, p, 1, f + d.R / 4);
        }
    }
}
// The angles as pairs, the sines times `sign`.
template <int VEC, typename R>
__device__ __forceinline__ void get_angles(const R& ring, int slot, int p0, bool turns, float sign, uint64_t (&c)[VEC / 2],
                                           uint64_t (&s)[VEC / 2]) {
    if (!turns) return;
#pragma unroll
    for (int j = 0; j < VEC / 4; ++j) {
        uint64_t f[2];
        get(ring.get(slot, p0 + j), f);
        c[2 * j] = f[0], c[2 * j + 1] = f[1];
        get(ring.get(slot, p0 + VEC / 4 + j), f);
        s[2 * j] = mul2(f[0], twice(sign)), s[2 * j + 1] = mul2(f[1], twice(sign));
    }
}

// Rotates the slot's pairs by (c, s); the halves' partners are elements of a and b, the
// interleaved order's are neighbours within a, then within b (their angles likewise).
template <int VEC, bool kInter>
__device__ __forceinline__ void turn(uint64_t (&a)[VEC / 2], uint64_t (&b)[VEC / 2], const uint64_t (&c)[VEC / 2],
                                     const uint64_t (&s)[VEC / 2]) {
    if constexpr (kInter) {
        auto one = [](uint64_t x, float cj, float sj) {
            float x1, x2;
            unpair(x, x1, x2);
            return fma2(pair(x2, x1), pair(-sj, sj), mul2(x, twice(cj)));
        };
#pragma unroll
        for (int j = 0; j < VEC / 4; ++j) {
            float c0, c1, s0, s1;
            unpair(c[j], c0, c1);
            unpair(s[j], s0, s1);
            a[2 * j] = one(a[2 * j], c0, s0), a[2 * j + 1] = one(a[2 * j + 1], c1, s1);
            unpair(c[VEC / 4 + j], c0, c1);
            unpair(s[VEC / 4 + j], s0, s1);
            b[2 * j] = one(b[2 * j], c0, s0), b[2 * j + 1] = one(b[2 * j + 1], c1, s1);
        }
    } else {
#pragma unroll
        for (int j = 0; j < VEC / 2; ++j) {
            const uint64_t x1 = a[j], x2 = b[j];
            a[j] = fma2(x2, mul2(s[j], twice(-1.f)), mul2(x1, c[j]));
            b[j] = fma2(x1, s[j], mul2(x2, c[j]));
        }
    }
}

struct Slot {
    int c0, c1;  // first elements of the lane's two pieces
    bool live, turns;
};
template <int VEC>
__device__ __forceinline__ Slot slot_of(const RopeDims& d, int u) {
    Slot s;
    const int turned = d.R / (2 * VEC);  // slots of the rotated part
    s.live = u * 2 * VEC < d.D;
    s.turns = u < turned;
    s.c0 = s.turns ? u * VEC : d.R + (u - turned) * VEC;
    s.c1 = s.c0 + (s.turns ? d.R : d.D - d.R) / 2;
    return s;
}

// Heads of an item, and stages of the ring: what two blocks of an SM hold.  (B8 T4096,
// 6 + 6 heads of 128, bf16: forward 3 heads 37.5 us, 4 39.8, 6 40.8; backward 2 heads
// 56.5, 3 66.6.  The angles come through L1, as the blocks of a token's heads share
// them: 41.6 and 61.3 us past it.)
constexpr int kFwdHeads = 3, kFwdStages = 2, kBwdHeads = 2, kBwdStages = 2;
template <typename T>
using FwdRing = Ring<2 * kFwdHeads + kVec<T> / 2, kFwdStages>;
template <typename T>
using BwdRing = Ring<4 * kBwdHeads + kVec<T> / 2, kBwdStages>;

template <typename T, int G, bool kInter, int kAxes>
__global__ void __launch_bounds__(kThreads, 2)
qk_norm_rope_fwd_kernel(RopeDims d, Side<T> q, Side<T> k, Tables tab) {
    constexpr int VEC = kVec<T>, NH = kFwdHeads, S = kFwdStages;
    await_previous();
    extern __shared__ __align__(16) unsigned char sm[];
    const FwdRing<T> ring(sm);
    const float inv_d = 1.f / d.D;
    const int u = threadIdx.x % G;
    const Slot sl = slot_of<VEC>(d, u);
    const int64_t step = (int64_t)gridDim.x * (kThreads / G);
    const int64_t first = (int64_t)blockIdx.x * (kThreads / G) + threadIdx.x / G;
    const int blocks = q.blocks + k.blocks;
    const int64_t turns = (d.tokens * blocks - (int64_t)blockIdx.x * (kThreads / G) + step - 1) / step;
    Walk now(first, step, blocks), ahead = now;  // the item worked on, the item copied
    Where<VEC, kInter, kAxes> at(d, tab, u, sl.turns);
    if (sl.turns && ahead.hi < d.tokens) at.move(d, tab, ahead.hi);
    auto heads = [&](const Walk& w, bool is_k, int& h0) {
        const int per = is_k ? k.per : q.per;
        h0 = (is_k ? w.lo - q.blocks : w.lo) * per;
        return w.hi < d.tokens && sl.live ? min(per, (is_k ? k.H : q.H) - h0) : 0;
    };
    auto issue = [&](int slot) {
        const bool is_k = ahead.lo >= q.blocks;
        int h0;
        const int n = heads(ahead, is_k, h0);
        const T* x = is_k ? k.x : q.x;
        if (n) x += ahead.hi * (is_k ? k.stride : q.stride) + (int64_t)h0 * d.D;
#pragma unroll
        for (int i = 0; i < NH; ++i) {
            ring.copy(slot, 2 * i, x + i * d.D + sl.c0, i < n);
            ring.copy(slot, 2 * i + 1, x + i * d.D + sl.c1, i < n);
        }
        if (n) copy_angles<VEC, kInter>(ring, slot, 2 * NH, d, tab, at, u, sl.turns);
        ring.commit();
        ahead.move();
        if (sl.turns && ahead.hi < d.tokens) at.move(d, tab, ahead.hi);
    };
#pragma unroll
    for (int i = 0; i < S - 1; ++i) issue(i);
    // every lane of the block takes the same number of turns, so the row sums are whole
    for (int slot = 0, fill = S - 1, left = (int)turns; left > 0; --left, slot = ring.after(slot)) {
        issue(fill);
        fill = ring.after(fill);
        ring.wait();
        const bool is_k = now.lo >= q.blocks;
        int h0;
        const int n = heads(now, is_k, h0);
        const T* w = is_k ? k.w : q.w;
        uint64_t wa[VEC / 2], wb[VEC / 2], c[VEC / 2], s[VEC / 2];
        get(sl.live ? ldg16(w + sl.c0) : make_uint4(0, 0, 0, 0), wa);
        get(sl.live ? ldg16(w + sl.c1) : make_uint4(0, 0, 0, 0), wb);
        get_angles<VEC>(ring, slot, 2 * NH, sl.turns, 1.f, c, s);
        T* y = (is_k ? k.out : q.out) + (now.hi * (is_k ? k.H : q.H) + h0) * d.D;
#pragma unroll
        for (int i = 0; i < NH; ++i) {
            uint64_t a[VEC / 2], b[VEC / 2], ss = twice(0.f);
            get(ring.get(slot, 2 * i), a);
            get(ring.get(slot, 2 * i + 1), b);
#pragma unroll
            for (int j = 0; j < VEC / 2; ++j) ss = fma2(a[j], a[j], fma2(b[j], b[j], ss));
            const uint64_t r = twice(rsqrtf(fmaf(group_sum<G>(sum2(ss)), inv_d, d.eps)));
#pragma unroll
            for (int j = 0; j < VEC / 2; ++j) {
                a[j] = mul2(mul2(a[j], r), wa[j]);
                b[j] = mul2(mul2(b[j], r), wb[j]);
            }
            if (sl.turns) turn<VEC, kInter>(a, b, c, s);
            if (i < n) {
                sts16(y + i * d.D + sl.c0, put(a));
                sts16(y + i * d.D + sl.c1, put(b));
            }
        }
        now.move();
    }
    ring.wait_all();  // no copy outlives the block
}

// Walks the queries' items, then the keys', and leaves one row of column sums per block
// and side in part [2][gridDim.x][D]; the blocks of a cluster add theirs up themselves, in the
// order of the blocks as the sum behind this kernel does.
template <typename T, int G, bool kInter, int kAxes>
__global__ void __launch_bounds__(kThreads, kRopeBwdPerSm)
qk_norm_rope_bwd_kernel(RopeDims d, Side<T> q, Side<T> k, Tables tab, float* __restrict__ part) {
    constexpr int VEC = kVec<T>, NH = kBwdHeads, S = kBwdStages;
    await_previous();
    extern __shared__ __align__(16) unsigned char sm[];
    const BwdRing<T> ring(sm);
    const float inv_d = 1.f / d.D;
    const int u = threadIdx.x % G;
    const Slot sl = slot_of<VEC>(d, u);
    const int64_t step = (int64_t)gridDim.x * (kThreads / G);
#pragma unroll 1
    for (int side = 0; side < 2; ++side) {
        const Side<T> sd = side ? k : q;
        uint64_t wa[VEC / 2], wb[VEC / 2], acc[VEC];
        get(sl.live ? ldg16(sd.w + sl.c0) : make_uint4(0, 0, 0, 0), wa);
        get(sl.live ? ldg16(sd.w + sl.c1) : make_uint4(0, 0, 0, 0), wb);
#pragma unroll
        for (int j = 0; j < VEC; ++j) acc[j] = twice(0.f);
        const int64_t items = d.tokens * sd.blocks, base = (int64_t)blockIdx.x * (kThreads / G);
        const int64_t turns = base < items ? (items - base + step - 1) / step : 0;
        if (turns) {
            Walk now(base + threadIdx.x / G, step, sd.blocks), ahead = now;
            Where<VEC, kInter, kAxes> at(d, tab, u, sl.turns);
            if (sl.turns && ahead.hi < d.tokens) at.move(d, tab, ahead.hi);
            auto issue = [&](int slot) {
                const int h0 = ahead.lo * sd.per, n = ahead.hi < d.tokens && sl.live ? min(sd.per, sd.H - h0) : 0;
                const T *x = sd.x, *dy = sd.dy;
                if (n) x += ahead.hi * sd.stride + (int64_t)h0 * d.D, dy += (ahead.hi * sd.H + h0) * d.D;
#pragma unroll
                for (int i = 0; i < NH; ++i) {
                    const bool on = i < n;
                    ring.copy(slot, 4 * i, x + i * d.D + sl.c0, on);
                    ring.copy(slot, 4 * i + 1, x + i * d.D + sl.c1, on);
                    ring.copy(slot, 4 * i + 2, dy + i * d.D + sl.c0, on);
                    ring.copy(slot, 4 * i + 3, dy + i * d.D + sl.c1, on);
                }
                if (n) copy_angles<VEC, kInter>(ring, slot, 4 * NH, d, tab, at, u, sl.turns);
                ring.commit();
                ahead.move();
                if (sl.turns && ahead.hi < d.tokens) at.move(d, tab, ahead.hi);
            };
#pragma unroll
            for (int i = 0; i < S - 1; ++i) issue(i);
            // every lane of the block takes the same number of turns, so the sums are whole
            for (int slot = 0, fill = S - 1, left = (int)turns; left > 0; --left, slot = ring.after(slot)) {
                issue(fill);
                fill = ring.after(fill);
                ring.wait();
                const int h0 = now.lo * sd.per, n = now.hi < d.tokens && sl.live ? min(sd.per, sd.H - h0) : 0;
                const int64_t row = (now.hi * sd.H + h0) * d.D;
                uint64_t c[VEC / 2], s[VEC / 2];
                get_angles<VEC>(ring, slot, 4 * NH, sl.turns, -1.f, c, s);
#pragma unroll
                for (int i = 0; i < NH; ++i) {
                    uint64_t a[VEC / 2], b[VEC / 2], ta[VEC / 2], tb[VEC / 2], pa[VEC / 2], pb[VEC / 2];
                    uint64_t ss = twice(0.f), tx = ss;
                    get(ring.get(slot, 4 * i), a);
                    get(ring.get(slot, 4 * i + 1), b);
                    get(ring.get(slot, 4 * i + 2), ta);
                    get(ring.get(slot, 4 * i + 3), tb);
                    if (sl.turns && i < n) turn<VEC, kInter>(ta, tb, c, s);
#pragma unroll
                    for (int j = 0; j < VEC / 2; ++j) {
                        ss = fma2(a[j], a[j], fma2(b[j], b[j], ss));
                        pa[j] = mul2(ta[j], a[j]), pb[j] = mul2(tb[j], b[j]);
                        tx = fma2(pa[j], wa[j], fma2(pb[j], wb[j], tx));
                    }
                    const float ms = fmaf(group_sum<G>(sum2(ss)), inv_d, d.eps);
                    // 0 where there is no row: its zeros times 1 / sqrt(eps) are NaN for eps = 0
                    const float r = i < n ? rsqrtf(ms) : 0.f;
                    // mean(t xh) = r mean(t x), times r of xh
                    const uint64_t m = twice(-group_sum<G>(sum2(tx)) * r * r * inv_d), r2 = twice(r);
#pragma unroll
                    for (int j = 0; j < VEC / 2; ++j) {
                        acc[j] = fma2(pa[j], r2, acc[j]);
                        acc[VEC / 2 + j] = fma2(pb[j], r2, acc[VEC / 2 + j]);
                        a[j] = mul2(fma2(a[j], m, mul2(ta[j], wa[j])), r2);
                        b[j] = mul2(fma2(b[j], m, mul2(tb[j], wb[j])), r2);
                    }
                    if (i < n) {
                        sts16(sd.out + row + i * d.D + sl.c0, put(a));
                        sts16(sd.out + row + i * d.D + sl.c1, put(b));
                    }
                }
                now.move();
            }
            ring.wait_all();  // the ring's memory serves the sums next
        }
        float* to = part + ((int64_t)side * gridDim.x + blockIdx.x) * d.D;
        if constexpr (kAxes > 0) {
            __shared__ float mine[256];
            if (sd.dw) to = mine;
            block_columns<G, VEC>(acc, sl.c0, sl.c1, sl.live, d.D, (float*)sm, to);
            if (sd.dw) {
                cluster_sync();
                for (int col = blockIdx.x * kThreads + threadIdx.x; col < d.D; col += gridDim.x * kThreads)
                    store1(sd.dw + col, cluster_sum(mine + col));
                cluster_sync();  // no block takes its sums back, or leaves, before the others have read them
            }
        } else {
            block_columns<G, VEC>(acc, sl.c0, sl.c1, sl.live, d.D, (float*)sm, to);
        }
    }
}

template <typename T, int G, bool kInter, int kAxes>
cudaError_t launch_k(const RopeDims& d, bool bwd, const Side<T>& q, const Side<T>& k, const Tables& tab, float* part,
                     int blocks, cudaStream_t st) {
    if (!bwd) {
        auto kern = qk_norm_rope_fwd_kernel<T, G, kInter, kAxes>;
        constexpr int smem = FwdRing<T>::BYTES;
        static std::atomic<uint64_t> done{0};
        cudaError_t e = allow_smem(kern, smem, done);
        if (e != cudaSuccess) return e;
        return launch_dependent(kern, dim3((unsigned)blocks_for(d.tokens * (q.blocks + k.blocks), G, 2, sm_count())),
                                kThreads, smem, st, d, q, k, tab);
    } else {
        auto kern = qk_norm_rope_bwd_kernel<T, G, kInter, kAxes>;
        constexpr int smem = BwdRing<T>::BYTES;
        static_assert(smem >= (kThreads / 32) * 256 * 4, "the column sums fit the ring");
        static std::atomic<uint64_t> done{0}, done1{0};
        if (kAxes > 0 && q.dw) return launch_one_cluster(kern, blocks, kThreads, smem, done1, st, d, q, k, tab, part);
        cudaError_t e = allow_smem(kern, smem, done);
        if (e != cudaSuccess) return e;
        return launch_dependent(kern, dim3((unsigned)blocks), kThreads, smem, st, d, q, k, tab, part);
    }
}

template <typename T, int G, int kAxes>
cudaError_t launch_g(const RopeDims& d, bool inter, bool bwd, Side<T> q, Side<T> k, const Tables& tab, float* part,
                     int blocks, cudaStream_t st) {
    return inter ? launch_k<T, G, true, kAxes>(d, bwd, q, k, tab, part, blocks, st)
                 : launch_k<T, G, false, kAxes>(d, bwd, q, k, tab, part, blocks, st);
}

template <typename T, int kAxes>
cudaError_t launch_t(const RopeCall& c, bool bwd, cudaStream_t st) {
    RopeDims d{c.tokens, c.T, c.D, c.R, c.rows, c.eps};
    const Tables tab{c.cos, c.sin, c.pos, c.axes, c.map};
    const int nh = bwd ? kBwdHeads : kFwdHeads;
    auto side = [&](const void* x, const void* w, const void* dy, void* out, void* dw, int64_t stride, int H) {
        const int blocks = (H + nh - 1) / nh;
        return Side<T>{(const T*)x, (const T*)w, (const T*)dy, (T*)out, (T*)dw, stride, H, blocks, blocks ? (H + blocks - 1) / blocks : 0};
    };
    const Side<T> q = side(c.q, c.wq, c.dqo, c.qo, c.dwq, c.q_stride, c.Hq), k = side(c.k, c.wk, c.dko, c.ko, c.dwk, c.k_stride, c.Hk);
    switch (lanes_for(c.D, kVec<T>)) {
        case 1: return launch_g<T, 1, kAxes>(d, c.interleaved, bwd, q, k, tab, c.part, c.blocks, st);
        case 2: return launch_g<T, 2, kAxes>(d, c.interleaved, bwd, q, k, tab, c.part, c.blocks, st);
        case 4: return launch_g<T, 4, kAxes>(d, c.interleaved, bwd, q, k, tab, c.part, c.blocks, st);
        case 8: return launch_g<T, 8, kAxes>(d, c.interleaved, bwd, q, k, tab, c.part, c.blocks, st);
        case 16: return launch_g<T, 16, kAxes>(d, c.interleaved, bwd, q, k, tab, c.part, c.blocks, st);
        default:
            if constexpr (kVec<T> == 4)  // 256 32-bit elements take a whole warp
                return launch_g<T, 32, kAxes>(d, c.interleaved, bwd, q, k, tab, c.part, c.blocks, st);
            return cudaErrorInvalidValue;
    }
}

}  // namespace
}  // namespace gdn
