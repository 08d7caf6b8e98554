// add_norm.cu -- the residual's addition with the RMS norm of the sum, its form with an
// 8-bit output, and the gradients: the step in front of a layer's projection.
//
// Row x of D elements, residual s, weight w; h = x + s, r = (mean h^2 + eps)^(-1/2):
//   y = h r w,     y8 = e4m3(y / scale) with scale = max(|y|) / 448 over a group of columns.
// Backward, from dy and the gradient dh that reaches h by the residual stream, with
// hh = h r and t = dy w:
//   d = r (t - hh mean(t hh)) + dh   (of x and of the residual),    dw = sum over rows of dy hh.
//
// The sum is normalised as it stands in float32; h is what the residual stream keeps, in
// its own type, and what the backward reads.
//
// Bound by reading and writing the rows.  A row is held by L lanes (a power of two, a warp
// at least), each with kPieces pieces of it a stride of L apart, so that a warp's loads and
// stores fill whole sectors; the row is read once, its sum of squares is made of registers.
// Persistent blocks with a ring of asynchronous copies (rows.cuh) keep the next rows in
// flight.

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
    static __device__ __forceinline__ void copy(uint32_t at, const T* src, bool on) {
        if constexpr (BYTES == 16)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(at), "l"(src), "r"(on ? 16 : 0) : "memory");
        else
            asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(at), "l"(src), "r"(on ? 8 : 0) : "memory");
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
        if constexpr (BYTES == 16) *reinterpret_cast<uint4*>(p) = put(f);
        else *reinterpret_cast<uint2*>(p) = make_uint2(pack2(f[0]), pack2(f[1]));
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

// The larger one; NaN where either is.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float abs_max(const uint64_t& p, float m) {
    float a, b;
    unpair(p, a, b);
    return max_nan(m, max_nan(fabsf(a), fabsf(b)));
}

// A row's place: row `turn * gridDim.x * rows a block + ...`, its lane u of L.
struct Place {
    int L, u, per;       // lanes a row, this lane, rows a block
    int64_t first, step;  // this thread's first row, and the rows that all blocks take in a turn
    int turns;            // the same for every thread of a block: the sums' barriers are whole
    __device__ __forceinline__ Place(int64_t rows, int L_, int n)
        : L(L_), u(threadIdx.x & (L_ - 1)), per(n / L_), first((int64_t)blockIdx.x * per + threadIdx.x / L_),
          step((int64_t)gridDim.x * per) {
        const int64_t base = (int64_t)blockIdx.x * per;
        turns = base < rows ? (int)((rows - base + step - 1) / step) : 0;
    }
};

// Sums of two values over the L lanes of a row; `part` has two halves, used in turn, so that
// one barrier a turn is enough.
template <int N>
__device__ __forceinline__ void row_sums(float& a, float& b, int L, float2 (*part)[N / 32], int turn) {
    a = group_sum<32>(a);
    b = group_sum<32>(b);
    if (L == 32) return;
    float2* p = part[turn & 1];
    const int warp = threadIdx.x >> 5, w = L / 32, first = warp & ~(w - 1);
    if ((threadIdx.x & 31) == 0) p[warp] = make_float2(a, b);
    __syncthreads();
    a = b = 0.f;
    for (int i = 0; i < w; ++i) {
        const float2 s = p[first + i];
        a += s.x;
        b += s.y;
    }
}
template <int N>
__device__ __forceinline__ float row_max(float m, int L, float (*part)[N / 32], int turn) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, off));
    if (L == 32) return m;
    float* p = part[turn & 1];
    const int warp = threadIdx.x >> 5, w = L / 32, first = warp & ~(w - 1);
    if ((threadIdx.x & 31) == 0) p[warp] = m;
    __syncthreads();
    m = p[first];
    for (int i = 1; i < w; ++i) m = max_nan(m, p[first + i]);
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

// The scale of a group whose largest number is m: m / 448, so that e4m3's largest number
// stands for it, but no subnormal one, whose inverse would be infinite.  NaN stays NaN, and
// with an infinite scale the group is read back as NaN.
__device__ __forceinline__ float scale_of(float m) {
    const float s = m / 448.f;
    return s < 1.17549435e-38f ? 1.17549435e-38f : s;
}

struct NormDims {
    int64_t rows, x_stride, r_stride;
    int D, L, group;  // group: columns of a scale
    float eps;
};

constexpr int kFwdSlots = 2 * kPieces, kBwdSlots = 3 * kPieces;

template <typename TX, typename TR, int N, bool kQuant>
__global__ void __launch_bounds__(N, N == 256 ? 3 : 1)
add_norm_fwd_kernel(NormDims d, const TX* __restrict__ x, const TR* res, const TX* __restrict__ w, TR* h,
                    void* __restrict__ y, float* __restrict__ scales) {
    constexpr int VEC = 16 / (int)sizeof(TR), S = kStages;
    using PX = Piece<TX, VEC>;
    using PR = Piece<TR, VEC>;
    await_previous();
    extern __shared__ __align__(16) unsigned char sm[];
    __shared__ float2 part[2][N / 32];
    __shared__ float most[2][N / 32];
    const Slots<kFwdSlots, S, N> ring(sm);
    const Place at(d.rows, d.L, N);
    const float inv_d = 1.f / d.D;
    auto live = [&](int p) { return (at.u + p * at.L) * VEC < d.D; };
    auto column = [&](int p) { return (at.u + p * at.L) * VEC; };
    int64_t now = at.first, next = now;
    auto issue = [&](int slot) {
        const TX* xp = x + next * d.x_stride;
        const TR* rp = res + next * d.r_stride;
#pragma unroll
        for (int p = 0; p < kPieces; ++p) {
            if (p * at.L * VEC >= d.D) break;
            const bool on = next < d.rows && live(p);
            PX::copy(ring.at(slot, p), on ? xp + column(p) : x, on);
            if (res) PR::copy(ring.at(slot, kPieces + p), on ? rp + column(p) : res, on);
        }
        commit();
        next += at.step;
    };
    uint4 wv[kPieces];
#pragma unroll
    for (int p = 0; p < kPieces; ++p) wv[p] = live(p) ? PX::ldg(w + column(p)) : make_uint4(0, 0, 0, 0);
    if (at.turns) issue(0);
    for (int turn = 0, slot = 0; turn < at.turns; ++turn, slot ^= 1, now += at.step) {
        issue(slot ^ 1);
        wait_group<S - 1>();
        uint64_t a[kPieces][VEC / 2], ss = twice(0.f);
#pragma unroll
        for (int p = 0; p < kPieces; ++p) {
            if (p * at.L * VEC >= d.D) break;
            PX::load(ring.at(slot, p), a[p]);
            if (res) {
                uint64_t s[VEC / 2];
                PR::load(ring.at(slot, kPieces + p), s);
#pragma unroll
                for (int j = 0; j < VEC / 2; ++j) a[p][j] = add2(a[p][j], s[j]);
                if (h && now < d.rows && live(p)) PR::store(h + now * d.D + column(p), a[p]);
            }
#pragma unroll
            for (int j = 0; j < VEC / 2; ++j) ss = fma2(a[p][j], a[p][j], ss);
        }
        float sum = sum2(ss), none = 0.f;
        row_sums<N>(sum, none, at.L, part, turn);
        const uint64_t r = twice(rsqrtf(fmaf(sum, inv_d, d.eps)));
        float m = 0.f;
#pragma unroll
        for (int p = 0; p < kPieces; ++p) {
            if (p * at.L * VEC >= d.D) break;
            uint64_t f[VEC / 2];
            PX::unpack(wv[p], f);
#pragma unroll
            for (int j = 0; j < VEC / 2; ++j) {
                a[p][j] = mul2(mul2(a[p][j], r), f[j]);
                if (kQuant) m = abs_max(a[p][j], m);
            }
            if constexpr (!kQuant) {
                if (now < d.rows && live(p)) PX::store((TX*)y + now * d.D + column(p), a[p]);
            } else if (d.group < d.D) {
                // a group's lanes are neighbours: 4 to 32 of them
                for (int off = d.group / VEC / 2; off > 0; off >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, off));
                const float scale = scale_of(m);
                const uint64_t by = twice(1.f / scale);
#pragma unroll
                for (int j = 0; j < VEC / 2; ++j) a[p][j] = mul2(a[p][j], by);
                if (column(p) % d.group == 0 && now < d.rows && live(p))
                    scales[now * (d.D / d.group) + column(p) / d.group] = scale;
                m = 0.f;
            }
        }
        if constexpr (kQuant) {
            uint64_t by = twice(1.f);
            if (d.group >= d.D) {
                const float scale = scale_of(row_max<N>(m, at.L, most, turn));
                by = twice(1.f / scale);
                if (at.u == 0 && now < d.rows) scales[now] = scale;
            }
#pragma unroll
            for (int p = 0; p < kPieces; ++p) {
                if (p * at.L * VEC >= d.D || now >= d.rows || !live(p)) break;
                uint32_t q[VEC / 2];
#pragma unroll
                for (int j = 0; j < VEC / 2; ++j) q[j] = e4m3x2(mul2(a[p][j], by));
                unsigned char* out = (unsigned char*)y + now * d.D + column(p);
                if constexpr (VEC == 8) *reinterpret_cast<uint2*>(out) = make_uint2(q[0] | q[1] << 16, q[2] | q[3] << 16);
                else *reinterpret_cast<uint32_t*>(out) = q[0] | q[1] << 16;
            }
        }
    }
    wait_group<0>();  // no copy outlives the block
}

// Each block leaves one row of column sums in part [gridDim.x][D].
template <typename TX, typename TR, int N>
__global__ void __launch_bounds__(N, N == 256 ? 2 : 1)
add_norm_bwd_kernel(NormDims d, const TR* __restrict__ h, const TX* __restrict__ w, const TX* __restrict__ dy,
                    const TR* __restrict__ dh, TX* __restrict__ dx, TR* __restrict__ dr, float* __restrict__ sums) {
    constexpr int VEC = 16 / (int)sizeof(TR), S = kStages;
    using PX = Piece<TX, VEC>;
    using PR = Piece<TR, VEC>;
    await_previous();
    extern __shared__ __align__(16) unsigned char sm[];
    __shared__ float2 part[2][N / 32];
    const Slots<kBwdSlots, S, N> ring(sm);
    const Place at(d.rows, d.L, N);
    const float inv_d = 1.f / d.D;
    auto live = [&](int p) { return (at.u + p * at.L) * VEC < d.D; };
    auto column = [&](int p) { return (at.u + p * at.L) * VEC; };
    int64_t now = at.first, next = now;
    auto issue = [&](int slot) {
        const TR* hp = h + next * d.r_stride;
#pragma unroll
        for (int p = 0; p < kPieces; ++p) {
            if (p * at.L * VEC >= d.D) break;
            const bool on = next < d.rows && live(p);
            PR::copy(ring.at(slot, p), on ? hp + column(p) : h, on);
            PX::copy(ring.at(slot, kPieces + p), on ? dy + next * d.D + column(p) : dy, on);
            if (dh) PR::copy(ring.at(slot, 2 * kPieces + p), on ? dh + next * d.D + column(p) : dh, on);
        }
        commit();
        next += at.step;
    };
    uint4 wv[kPieces];
    uint64_t acc[kPieces][VEC / 2];
#pragma unroll
    for (int p = 0; p < kPieces; ++p) {
        wv[p] = live(p) ? PX::ldg(w + column(p)) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int j = 0; j < VEC / 2; ++j) acc[p][j] = twice(0.f);
    }
    if (at.turns) issue(0);
    for (int turn = 0, slot = 0; turn < at.turns; ++turn, slot ^= 1, now += at.step) {
        issue(slot ^ 1);
        wait_group<S - 1>();
        uint64_t ss = twice(0.f), tx = ss;
#pragma unroll
        for (int p = 0; p < kPieces; ++p) {
            if (p * at.L * VEC >= d.D) break;
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
        row_sums<N>(sq, st, at.L, part, turn);
        // 0 where there is no row: its zeros times 1 / sqrt(eps) are NaN for eps = 0
        const float r = now < d.rows ? rsqrtf(fmaf(sq, inv_d, d.eps)) : 0.f;
        // mean(t hh) = r mean(t h), times r of hh
        const uint64_t m = twice(-st * r * r * inv_d), r2 = twice(r);
        // the pieces are read again from shared memory: held in registers over the sum they
        // would leave room for half of the warps
#pragma unroll
        for (int p = 0; p < kPieces; ++p) {
            if (p * at.L * VEC >= d.D) break;
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
            if (now < d.rows && live(p)) {
                PX::store(dx + now * d.D + column(p), a);
                if constexpr (sizeof(TX) != sizeof(TR)) PR::store(dr + now * d.D + column(p), a);
            }
        }
    }
    wait_group<0>();
    // the block's rows of sums, one after the other: the same call gives the same bits
    __syncthreads();
    float* col = (float*)sm;
    for (int g = 0; g < at.per; ++g) {
        if ((int)threadIdx.x / at.L == g) {
#pragma unroll
            for (int p = 0; p < kPieces; ++p) {
                if (!live(p)) break;
#pragma unroll
                for (int j = 0; j < VEC / 2; ++j) {
                    float* c = col + column(p) + 2 * j;
                    float lo, hi;
                    unpair(acc[p][j], lo, hi);
                    c[0] = g ? c[0] + lo : lo;
                    c[1] = g ? c[1] + hi : hi;
                }
            }
        }
        __syncthreads();
    }
    for (int c = threadIdx.x; c < d.D; c += N) sums[(int64_t)blockIdx.x * d.D + c] = col[c];
}

// Lanes a row takes: pieces of VEC elements, kPieces a lane, a warp at least.
int lanes_of(int D, int vec) {
    int L = 32;
    while (L * kPieces * vec < D) L *= 2;
    return L;
}

template <typename TX, typename TR, int N, bool kQuant>
cudaError_t fwd(const AddNormCall& c, const NormDims& d, cudaStream_t st) {
    auto kern = add_norm_fwd_kernel<TX, TR, N, kQuant>;
    constexpr int smem = Slots<kFwdSlots, kStages, N>::BYTES;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(kern, smem, done);
    if (e != cudaSuccess) return e;
    const int64_t want = (d.rows + N / d.L - 1) / (N / d.L), cap = (int64_t)sm_count() * (N == 256 ? 3 : 1);
    return launch_dependent(kern, dim3((unsigned)(want < cap ? want : cap)), N, smem, st, d, (const TX*)c.x,
                            (const TR*)c.res, (const TX*)c.w, (TR*)c.h, c.y, c.scales);
}

template <typename TX, typename TR, int N>
cudaError_t bwd(const AddNormCall& c, const NormDims& d, cudaStream_t st) {
    auto kern = add_norm_bwd_kernel<TX, TR, N>;
    constexpr int smem = Slots<kBwdSlots, kStages, N>::BYTES;
    static_assert(smem >= 8192 * 4, "the column sums fit the ring");
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(kern, smem, done);
    if (e != cudaSuccess) return e;
    return launch_dependent(kern, dim3((unsigned)c.blocks), N, smem, st, d, (const TR*)c.h_in, (const TX*)c.w,
                            (const TX*)c.dy, (const TR*)c.dh, (TX*)c.dx, (TR*)c.dr, c.part);
}

template <typename TX, typename TR, int N>
cudaError_t any(const AddNormCall& c, const NormDims& d, AddNormKind kind, cudaStream_t st) {
    switch (kind) {
        case AddNormKind::FWD: return fwd<TX, TR, N, false>(c, d, st);
        case AddNormKind::QUANT: return fwd<TX, TR, N, true>(c, d, st);
        default: return bwd<TX, TR, N>(c, d, st);
    }
}

template <typename TX, typename TR>
cudaError_t launch_t(const AddNormCall& c, AddNormKind kind, cudaStream_t st) {
    const NormDims d{c.rows, c.x_stride, c.r_stride, c.D, lanes_of(c.D, 16 / (int)sizeof(TR)), c.group ? c.group : c.D, c.eps};
    return d.L <= 256 ? any<TX, TR, 256>(c, d, kind, st) : any<TX, TR, 512>(c, d, kind, st);
}

}  // namespace

int add_norm_bwd_blocks(int64_t rows, int D, int wide) {
    const int L = lanes_of(D, 16 / wide), n = L <= 256 ? 256 : 512;
    const int64_t per = n / L, want = (rows + per - 1) / per, cap = (int64_t)sm_count() * (n == 256 ? 2 : 1);
    return (int)(want < 1 ? 1 : want < cap ? want : cap);
}

cudaError_t launch_add_norm(const AddNormCall& c, InType ty, InType stream_ty, AddNormKind kind, cudaStream_t st) {
    if (ty == InType::F32) return launch_t<float, float>(c, kind, st);
    return stream_ty == InType::BF16 ? launch_t<__nv_bfloat16, __nv_bfloat16>(c, kind, st)
                                     : launch_t<__nv_bfloat16, float>(c, kind, st);
}

}  // namespace gdn
