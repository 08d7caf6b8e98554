// norm_rope.cu -- RMS norm of every head's query and key row with the position's
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
// slot u holds pieces (u, u + R/(2 VEC)) of the rotated part, so both elements of a
// pair are in one lane, then neighbouring pieces of the rest; interleaved, neighbouring
// pieces throughout.  Either way the slot's VEC pairs are u VEC .. u VEC + VEC - 1, so
// one piece of the cosine and sine rows serves both orders.  A group takes kHeads
// heads of one token, which share that piece.  Bound by reading and writing the rows.

#include "gdn_internal.h"
#include "rows.cuh"

namespace gdn {
namespace {

using namespace rows;

constexpr int kThreads = 256;
constexpr int kHeads = 4;  // rows of one token that a group takes at a time

// What a group works on: item i of one side (queries or keys) is kHeads heads of token
// i / blocks.
template <typename T>
struct Side {
    const T* x;   // rows, `stride` elements from token to token
    const T* w;   // [D]
    const T* dy;  // backward: [tokens, H, D]
    T* out;       // y or dx, [tokens, H, D]
    int64_t stride;
    int H, blocks;
};

struct RopeDims {
    int64_t tokens;
    int T, D, R, rows;  // rows: of the cosine and sine tables
    float eps;
};

// The angles of a lane's pairs; a position outside the tables gives NaN, so that
// the token's rows show it.
template <int VEC>
__device__ __forceinline__ void angles(const RopeDims& d, const float* cs, const float* sn, const int32_t* pos,
                                       int64_t tok, int slot, bool turns, float (&c)[VEC], float (&s)[VEC]) {
    if (!turns) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) c[j] = 1.f, s[j] = 0.f;
        return;
    }
    const int p = pos ? pos[tok] : (int)(tok % d.T);
    if (p < 0 || p >= d.rows) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) c[j] = s[j] = __int_as_float(0x7fc00000);
        return;
    }
    const int64_t at = (int64_t)p * (d.R / 2) + slot * VEC;
    ldf<VEC>(cs + at, c);
    ldf<VEC>(sn + at, s);
}

// Rotates the slot's pairs by (c, s); the halves' partners are (a[j], b[j]), the
// interleaved order's are neighbours within a, then within b.
template <int VEC, bool kInter>
__device__ __forceinline__ void turn(float (&a)[VEC], float (&b)[VEC], const float (&c)[VEC], const float (&s)[VEC],
                                     float sign) {
    if constexpr (kInter) {
#pragma unroll
        for (int j = 0; j < VEC / 2; ++j) {
            const float a1 = a[2 * j], a2 = a[2 * j + 1], b1 = b[2 * j], b2 = b[2 * j + 1];
            const float ca = c[j], sa = sign * s[j], cb = c[VEC / 2 + j], sb = sign * s[VEC / 2 + j];
            a[2 * j] = a1 * ca - a2 * sa, a[2 * j + 1] = a2 * ca + a1 * sa;
            b[2 * j] = b1 * cb - b2 * sb, b[2 * j + 1] = b2 * cb + b1 * sb;
        }
    } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            const float x1 = a[j], x2 = b[j], sj = sign * s[j];
            a[j] = x1 * c[j] - x2 * sj, b[j] = x2 * c[j] + x1 * sj;
        }
    }
}

struct Slot {
    int c0, c1;  // first elements of the lane's two pieces
    bool live, turns;
};
template <int VEC, bool kInter>
__device__ __forceinline__ Slot slot_of(const RopeDims& d, int u) {
    Slot s;
    s.live = u * 2 * VEC < d.D;
    s.turns = u * 2 * VEC < d.R;
    if (!kInter && s.turns) s.c0 = u * VEC, s.c1 = d.R / 2 + u * VEC;
    else s.c0 = u * 2 * VEC, s.c1 = s.c0 + VEC;
    return s;
}

template <typename T, int G, bool kInter>
__global__ void __launch_bounds__(kThreads)
qk_norm_rope_fwd_kernel(RopeDims d, Side<T> q, Side<T> k, const float* __restrict__ cs, const float* __restrict__ sn,
                        const int32_t* __restrict__ pos) {
    constexpr int VEC = kVec<T>;
    const int u = threadIdx.x % G;
    const int64_t item = (int64_t)blockIdx.x * (kThreads / G) + threadIdx.x / G;
    const int blocks = q.blocks + k.blocks;
    const bool on = item < d.tokens * blocks;
    const int64_t tok = on ? item / blocks : 0;
    const int hb = on ? (int)(item % blocks) : 0;
    const bool is_k = hb >= q.blocks;
    const T* w = is_k ? k.w : q.w;
    const int H = is_k ? k.H : q.H;
    const Slot sl = slot_of<VEC, kInter>(d, u);
    const int h0 = (is_k ? hb - q.blocks : hb) * kHeads;
    const int n = on && sl.live ? min(kHeads, H - h0) : 0;

    const T* x = (is_k ? k.x + tok * k.stride : q.x + tok * q.stride) + (int64_t)h0 * d.D;
    uint4 xa[kHeads], xb[kHeads];
#pragma unroll
    for (int i = 0; i < kHeads; ++i)
        if (i < n) xa[i] = lds16(x + i * d.D + sl.c0), xb[i] = lds16(x + i * d.D + sl.c1);
        else xa[i] = xb[i] = make_uint4(0, 0, 0, 0);
    float wa[VEC], wb[VEC], c[VEC], s[VEC];
    get(sl.live ? ldg16(w + sl.c0) : make_uint4(0, 0, 0, 0), wa);
    get(sl.live ? ldg16(w + sl.c1) : make_uint4(0, 0, 0, 0), wb);
    angles<VEC>(d, cs, sn, pos, tok, u, sl.turns && on, c, s);

    T* y = (is_k ? k.out : q.out) + (tok * H + h0) * d.D;
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
        float a[VEC], b[VEC], ss = 0.f;
        get(xa[i], a);
        get(xb[i], b);
#pragma unroll
        for (int j = 0; j < VEC; ++j) ss = fmaf(a[j], a[j], fmaf(b[j], b[j], ss));
        const float r = rsqrtf(group_sum<G>(ss) / d.D + d.eps);
#pragma unroll
        for (int j = 0; j < VEC; ++j) a[j] = a[j] * r * wa[j], b[j] = b[j] * r * wb[j];
        if (sl.turns) turn<VEC, kInter>(a, b, c, s, 1.f);
        if (i < n) {
            sts16(y + i * d.D + sl.c0, put(a));
            sts16(y + i * d.D + sl.c1, put(b));
        }
    }
}

// Persistent blocks walk the queries' items, then the keys', and leave one row of
// column sums per block and side in part [2][gridDim.x][D].
template <typename T, int G, bool kInter>
__global__ void __launch_bounds__(kThreads)
qk_norm_rope_bwd_kernel(RopeDims d, Side<T> q, Side<T> k, const float* __restrict__ cs, const float* __restrict__ sn,
                        const int32_t* __restrict__ pos, float* __restrict__ part) {
    constexpr int VEC = kVec<T>;
    extern __shared__ float sm[];  // [8 warps][D]
    const int u = threadIdx.x % G;
    const Slot sl = slot_of<VEC, kInter>(d, u);
    const int64_t step = (int64_t)gridDim.x * (kThreads / G);
#pragma unroll 1
    for (int side = 0; side < 2; ++side) {
        const Side<T> sd = side ? k : q;
        float wa[VEC], wb[VEC], acc[2 * VEC];
        get(sl.live ? ldg16(sd.w + sl.c0) : make_uint4(0, 0, 0, 0), wa);
        get(sl.live ? ldg16(sd.w + sl.c1) : make_uint4(0, 0, 0, 0), wb);
#pragma unroll
        for (int j = 0; j < 2 * VEC; ++j) acc[j] = 0.f;
        const int64_t items = d.tokens * sd.blocks;
        // every lane of the block takes the same number of turns, so the sums are whole
        for (int64_t base = (int64_t)blockIdx.x * (kThreads / G); base < items; base += step) {
            const int64_t item = base + threadIdx.x / G;
            const bool on = item < items && sl.live;
            const int64_t tok = on ? item / sd.blocks : 0;
            const int h0 = on ? (int)(item % sd.blocks) * kHeads : 0;
            const int n = on ? min(kHeads, sd.H - h0) : 0;
            float c[VEC], s[VEC];
            angles<VEC>(d, cs, sn, pos, tok, u, sl.turns && on, c, s);
            const T* x = sd.x + tok * sd.stride + (int64_t)h0 * d.D;
            const int64_t row = (tok * sd.H + h0) * d.D;
            uint4 xa[kHeads], xb[kHeads], ya[kHeads], yb[kHeads];
#pragma unroll
            for (int i = 0; i < kHeads; ++i) {
                if (i < n) {
                    xa[i] = lds16(x + i * d.D + sl.c0), xb[i] = lds16(x + i * d.D + sl.c1);
                    ya[i] = lds16(sd.dy + row + i * d.D + sl.c0), yb[i] = lds16(sd.dy + row + i * d.D + sl.c1);
                } else {
                    xa[i] = xb[i] = ya[i] = yb[i] = make_uint4(0, 0, 0, 0);
                }
            }
#pragma unroll
            for (int i = 0; i < kHeads; ++i) {
                float a[VEC], b[VEC], ta[VEC], tb[VEC], ss = 0.f, tx = 0.f;
                get(xa[i], a);
                get(xb[i], b);
                get(ya[i], ta);
                get(yb[i], tb);
                if (sl.turns && i < n) turn<VEC, kInter>(ta, tb, c, s, -1.f);
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    ss = fmaf(a[j], a[j], fmaf(b[j], b[j], ss));
                    tx = fmaf(ta[j] * wa[j], a[j], fmaf(tb[j] * wb[j], b[j], tx));
                }
                ss = group_sum<G>(ss);
                tx = group_sum<G>(tx);
                const float r = rsqrtf(ss / d.D + d.eps);
                const float m = tx * r * r / d.D;  // mean(t xh) = r mean(t x), times r of xh
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    acc[j] = fmaf(ta[j], a[j] * r, acc[j]);
                    acc[VEC + j] = fmaf(tb[j], b[j] * r, acc[VEC + j]);
                    a[j] = r * (ta[j] * wa[j] - a[j] * m);
                    b[j] = r * (tb[j] * wb[j] - b[j] * m);
                }
                if (i < n) {
                    sts16(sd.out + row + i * d.D + sl.c0, put(a));
                    sts16(sd.out + row + i * d.D + sl.c1, put(b));
                }
            }
        }
        block_columns<G, VEC, kThreads / 32>(acc, sl.c0, sl.c1, sl.live, d.D, sm,
                                             part + ((int64_t)side * gridDim.x + blockIdx.x) * d.D);
    }
}

template <typename T, int G>
cudaError_t launch_g(const RopeDims& d, bool inter, bool bwd, Side<T> q, Side<T> k, const float* cs, const float* sn,
                     const int32_t* pos, float* part, int blocks, cudaStream_t st) {
    if (!bwd) {
        const int64_t items = d.tokens * (q.blocks + k.blocks), per = kThreads / G;
        const unsigned grid = (unsigned)((items + per - 1) / per);
        if (inter) qk_norm_rope_fwd_kernel<T, G, true><<<grid, kThreads, 0, st>>>(d, q, k, cs, sn, pos);
        else qk_norm_rope_fwd_kernel<T, G, false><<<grid, kThreads, 0, st>>>(d, q, k, cs, sn, pos);
    } else {
        const size_t smem = (size_t)(kThreads / 32) * d.D * sizeof(float);
        if (inter) qk_norm_rope_bwd_kernel<T, G, true><<<blocks, kThreads, smem, st>>>(d, q, k, cs, sn, pos, part);
        else qk_norm_rope_bwd_kernel<T, G, false><<<blocks, kThreads, smem, st>>>(d, q, k, cs, sn, pos, part);
    }
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_t(const RopeCall& c, bool bwd, cudaStream_t st) {
    RopeDims d{c.tokens, c.T, c.D, c.R, c.rows, c.eps};
    auto blocks = [](int H) { return (H + kHeads - 1) / kHeads; };
    Side<T> q{(const T*)c.q, (const T*)c.wq, (const T*)c.dqo, (T*)c.qo, c.q_stride, c.Hq, blocks(c.Hq)};
    Side<T> k{(const T*)c.k, (const T*)c.wk, (const T*)c.dko, (T*)c.ko, c.k_stride, c.Hk, blocks(c.Hk)};
    switch (lanes_for(c.D, kVec<T>)) {
        case 1: return launch_g<T, 1>(d, c.interleaved, bwd, q, k, c.cos, c.sin, c.pos, c.part, c.blocks, st);
        case 2: return launch_g<T, 2>(d, c.interleaved, bwd, q, k, c.cos, c.sin, c.pos, c.part, c.blocks, st);
        case 4: return launch_g<T, 4>(d, c.interleaved, bwd, q, k, c.cos, c.sin, c.pos, c.part, c.blocks, st);
        case 8: return launch_g<T, 8>(d, c.interleaved, bwd, q, k, c.cos, c.sin, c.pos, c.part, c.blocks, st);
        case 16: return launch_g<T, 16>(d, c.interleaved, bwd, q, k, c.cos, c.sin, c.pos, c.part, c.blocks, st);
        default:
            if constexpr (kVec<T> == 4)  // 256 32-bit elements take a whole warp
                return launch_g<T, 32>(d, c.interleaved, bwd, q, k, c.cos, c.sin, c.pos, c.part, c.blocks, st);
            return cudaErrorInvalidValue;
    }
}

}  // namespace

cudaError_t launch_qk_norm_rope(const RopeCall& c, InType ty, bool bwd, cudaStream_t st) {
    return ty == InType::BF16 ? launch_t<__nv_bfloat16>(c, bwd, st) : launch_t<float>(c, bwd, st);
}

}  // namespace gdn
