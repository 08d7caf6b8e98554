// gated_norm.cu -- RMS norm of every head's output row times the silu of a gate, and
// its gradients: the step behind the recurrence, before the output projection; and the
// last sum of a weight's gradient, which norm_rope.cu shares.
//
// Row x of D elements, gate z, weight w; r = (mean x^2 + eps)^(-1/2), xh = x r,
// sg = 1 / (1 + e^-z), act = z sg:
//   y = xh w act
//   dw = sum over rows of dy act xh,   dz = dy xh w (sg + act (1 - sg)),
//   dx = r (t - xh mean(t xh)),  t = dy act w.
// A group of lanes holds a row (rows.cuh: lane u has pieces u and u + D/(2 VEC)).

#include "gdn_internal.h"
#include "rows.cuh"

namespace gdn {
namespace {

using namespace rows;

struct GatedDims {
    int64_t rows;
    int H, D;
    int64_t x_stride, z_stride;  // elements from token to token
    float eps;
};

// Stages of the ring, and blocks per SM: the backward's registers leave room for two.
// (At 100 MB of rows: forward 2 stages in 4 blocks 25.8 us, 3 in 3 26.2; backward 2
// stages 51.9, 3 53.8, 4 54.5.)
constexpr int kStages = 2, kFwdPerSm = 4;
using FwdRing = Ring<4, kStages>;
using BwdRing = Ring<6, kStages>;

template <typename T, int G>
__global__ void __launch_bounds__(kThreads, kFwdPerSm)
gated_norm_fwd_kernel(GatedDims d, const T* __restrict__ x, const T* __restrict__ z, const T* __restrict__ w,
                      T* __restrict__ y) {
    constexpr int VEC = kVec<T>, S = kStages;
    await_previous();
    extern __shared__ __align__(16) unsigned char sm[];
    const FwdRing ring(sm);
    const float inv_d = 1.f / d.D;
    const int c0 = (threadIdx.x % G) * VEC, half = d.D / 2;
    const bool live = c0 < half;
    const int64_t per = kThreads / G, step = (int64_t)gridDim.x * per, base = (int64_t)blockIdx.x * per;
    const int64_t turns = (d.rows - base + step - 1) / step;
    int64_t now = base + threadIdx.x / G, next = now;
    Walk ahead(next, step, d.H);  // (token, head) of the row copied
    auto issue = [&](int slot) {
        const bool on = live && next < d.rows;
        const int off = ahead.lo * d.D + c0;
        const T* xp = x + ahead.hi * d.x_stride + off;
        const T* zp = z + ahead.hi * d.z_stride + off;
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            ring.copy(slot, p, xp + p * half, on);
            ring.copy(slot, 2 + p, zp + p * half, on);
        }
        ring.commit();
        ahead.move();
        next += step;
    };
    uint64_t wv[2][VEC / 2];
#pragma unroll
    for (int p = 0; p < 2; ++p) get(live ? ldg16(w + c0 + p * half) : make_uint4(0, 0, 0, 0), wv[p]);
#pragma unroll
    for (int i = 0; i < S - 1; ++i) issue(i);
    // every lane of the block takes the same number of turns, so the row sums are whole
    for (int slot = 0, fill = S - 1, left = (int)turns; left > 0; --left, slot = ring.after(slot), now += step) {
        issue(fill);
        fill = ring.after(fill);
        ring.wait();
        uint64_t xv[2][VEC / 2], ss = twice(0.f);
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            get(ring.get(slot, p), xv[p]);
#pragma unroll
            for (int j = 0; j < VEC / 2; ++j) ss = fma2(xv[p][j], xv[p][j], ss);
        }
        const uint64_t r = twice(rsqrtf(fmaf(group_sum<G>(sum2(ss)), inv_d, d.eps)));
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            uint64_t zv[VEC / 2];
            get(ring.get(slot, 2 + p), zv);
#pragma unroll
            for (int j = 0; j < VEC / 2; ++j)
                xv[p][j] = mul2(mul2(mul2(xv[p][j], r), wv[p][j]), mul2(zv[j], sigmoid2(zv[j])));
            if (live && now < d.rows) sts16(y + now * d.D + c0 + p * half, put(xv[p]));
        }
    }
    ring.wait_all();  // no copy outlives the block
}

// Each block leaves one row of column sums in part [gridDim.x][D].
template <typename T, int G>
__global__ void __launch_bounds__(kThreads, kGatedBwdPerSm)
gated_norm_bwd_kernel(GatedDims d, const T* __restrict__ x, const T* __restrict__ z, const T* __restrict__ w,
                      const T* __restrict__ dy, T* __restrict__ dx, T* __restrict__ dz, float* __restrict__ part) {
    constexpr int VEC = kVec<T>, S = kStages;
    await_previous();
    extern __shared__ __align__(16) unsigned char sm[];
    const BwdRing ring(sm);
    const float inv_d = 1.f / d.D;
    const int c0 = (threadIdx.x % G) * VEC, half = d.D / 2;
    const bool live = c0 < half;
    uint64_t wv[2][VEC / 2], acc[VEC];
#pragma unroll
    for (int p = 0; p < 2; ++p) get(live ? ldg16(w + c0 + p * half) : make_uint4(0, 0, 0, 0), wv[p]);
#pragma unroll
    for (int j = 0; j < VEC; ++j) acc[j] = twice(0.f);
    const int64_t per = kThreads / G, step = (int64_t)gridDim.x * per, base = (int64_t)blockIdx.x * per;
    const int64_t turns = base < d.rows ? (d.rows - base + step - 1) / step : 0;
    int64_t now = base + threadIdx.x / G, next = now;
    Walk ahead(next, step, d.H);
    auto issue = [&](int slot) {
        const bool on = live && next < d.rows;
        const int off = ahead.lo * d.D + c0;
        const T* xp = x + ahead.hi * d.x_stride + off;
        const T* zp = z + ahead.hi * d.z_stride + off;
        const T* yp = dy + next * d.D + c0;
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            ring.copy(slot, p, xp + p * half, on);
            ring.copy(slot, 2 + p, zp + p * half, on);
            ring.copy(slot, 4 + p, yp + p * half, on);
        }
        ring.commit();
        ahead.move();
        next += step;
    };
    if (turns) {
#pragma unroll
        for (int i = 0; i < S - 1; ++i) issue(i);
    }
    for (int slot = 0, fill = S - 1, left = (int)turns; left > 0; --left, slot = ring.after(slot), now += step) {
        issue(fill);
        fill = ring.after(fill);
        ring.wait();
        // with u = dy w, p = dy act x, sl = the slope of silu = sg + act (1 - sg), which is
        // 1 for any large gate (as sg (1 + z - act) the sum 1 + z is wrong from 2^24 on):
        // t = u act, dz = r u x sl, dw += r p, t x = p w
        uint64_t xv[2][VEC / 2], t[2][VEC / 2], gz[2][VEC / 2], pr[2][VEC / 2], ss = twice(0.f), tx = ss;
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            uint64_t zv[VEC / 2], yv[VEC / 2];
            get(ring.get(slot, p), xv[p]);
            get(ring.get(slot, 2 + p), zv);
            get(ring.get(slot, 4 + p), yv);
#pragma unroll
            for (int j = 0; j < VEC / 2; ++j) {
                const uint64_t sg = sigmoid2(zv[j]), act = mul2(zv[j], sg), u = mul2(yv[j], wv[p][j]);
                const uint64_t sl = fma2(act, fma2(sg, twice(-1.f), twice(1.f)), sg);
                gz[p][j] = mul2(mul2(u, xv[p][j]), sl);
                t[p][j] = mul2(u, act);
                pr[p][j] = mul2(mul2(yv[j], act), xv[p][j]);
                ss = fma2(xv[p][j], xv[p][j], ss);
                tx = fma2(pr[p][j], wv[p][j], tx);
            }
        }
        const bool on = live && now < d.rows;
        const float ms = fmaf(group_sum<G>(sum2(ss)), inv_d, d.eps);
        // 0 where there is no row: its zeros times 1 / sqrt(eps) are NaN for eps = 0
        const float r = on ? rsqrtf(ms) : 0.f;
        // mean(t xh) = r mean(t x), times r of xh
        const uint64_t m = twice(-group_sum<G>(sum2(tx)) * r * r * inv_d), r2 = twice(r);
#pragma unroll
        for (int p = 0; p < 2; ++p) {
#pragma unroll
            for (int j = 0; j < VEC / 2; ++j) {
                acc[p * (VEC / 2) + j] = fma2(pr[p][j], r2, acc[p * (VEC / 2) + j]);
                gz[p][j] = mul2(gz[p][j], r2);
                xv[p][j] = mul2(fma2(xv[p][j], m, t[p][j]), r2);
            }
            if (on) {
                sts16(dx + now * d.D + c0 + p * half, put(xv[p]));
                sts16(dz + now * d.D + c0 + p * half, put(gz[p]));
            }
        }
    }
    ring.wait_all();  // the ring's memory serves the sums next
    block_columns<G, VEC>(acc, c0, c0 + half, live, d.D, (float*)sm, part + (int64_t)blockIdx.x * d.D);
}

__device__ __forceinline__ void store1(float* p, float x) { *p = x; }
__device__ __forceinline__ void store1(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// dw[c] = sum over the blocks' rows of part, in a fixed order: a warp takes 32 columns'
// rows w, w + 32, ..., the warps' sums are added in order.  blockIdx.y picks the side
// (part and dw of the queries, then of the keys).  Bound by latency: 32 warps a block, so
// that a thread's few loads are in flight together (8 warps took 9 us for 304 rows).
template <typename T>
__global__ void __launch_bounds__(1024)
weight_sum_kernel(int blocks, int D, const float* __restrict__ part, T* __restrict__ dw0, T* __restrict__ dw1) {
    __shared__ float sm[32][32];
    await_previous();
    const int lane = threadIdx.x & 31, c = blockIdx.x * 32 + lane, w = threadIdx.x >> 5;
    const float* p = part + (int64_t)blockIdx.y * blocks * D;
    float s = 0.f;
    if (c < D)
#pragma unroll 10
        for (int b = w; b < blocks; b += 32) s += p[(int64_t)b * D + c];
    sm[w][lane] = s;
    __syncthreads();
    if (w == 0 && c < D) {
#pragma unroll
        for (int i = 1; i < 32; ++i) s += sm[i][lane];
        store1((blockIdx.y ? dw1 : dw0) + c, s);
    }
}

template <typename T, int G>
cudaError_t launch_g(const GatedCall& c, const GatedDims& d, bool bwd, cudaStream_t st) {
    const T *x = (const T*)c.x, *z = (const T*)c.z, *w = (const T*)c.w;
    if (!bwd) {
        constexpr int smem = FwdRing::BYTES;
        static std::atomic<uint64_t> done{0};
        cudaError_t e = allow_smem(gated_norm_fwd_kernel<T, G>, smem, done);
        if (e != cudaSuccess) return e;
        return launch_dependent(gated_norm_fwd_kernel<T, G>,
                                dim3((unsigned)blocks_for(d.rows, G, kFwdPerSm, sm_count())), kThreads, smem, st, d, x,
                                z, w, (T*)c.y);
    } else {
        constexpr int smem = BwdRing::BYTES;
        static_assert(smem >= (kThreads / 32) * 256 * 4, "the column sums fit the ring");
        static std::atomic<uint64_t> done{0};
        cudaError_t e = allow_smem(gated_norm_bwd_kernel<T, G>, smem, done);
        if (e != cudaSuccess) return e;
        return launch_dependent(gated_norm_bwd_kernel<T, G>, dim3((unsigned)c.blocks), kThreads, smem, st, d, x, z, w,
                                (const T*)c.dy, (T*)c.dx, (T*)c.dz, c.part);
    }
}

template <typename T>
cudaError_t launch_t(const GatedCall& c, bool bwd, cudaStream_t st) {
    const GatedDims d{c.rows, c.H, c.D, c.x_stride, c.z_stride, c.eps};
    switch (lanes_for(c.D, kVec<T>)) {
        case 1: return launch_g<T, 1>(c, d, bwd, st);
        case 2: return launch_g<T, 2>(c, d, bwd, st);
        case 4: return launch_g<T, 4>(c, d, bwd, st);
        case 8: return launch_g<T, 8>(c, d, bwd, st);
        case 16: return launch_g<T, 16>(c, d, bwd, st);
        default:
            if constexpr (kVec<T> == 4) return launch_g<T, 32>(c, d, bwd, st);
            return cudaErrorInvalidValue;
    }
}

}  // namespace

cudaError_t launch_gated_norm(const GatedCall& c, InType ty, bool bwd, cudaStream_t st) {
    return ty == InType::BF16 ? launch_t<__nv_bfloat16>(c, bwd, st) : launch_t<float>(c, bwd, st);
}

cudaError_t launch_weight_sum(int sides, int blocks, int D, InType ty, const float* part, void* dw0, void* dw1,
                              cudaStream_t st) {
    const dim3 grid((D + 31) / 32, sides);
    if (ty == InType::BF16)
        return launch_dependent(weight_sum_kernel<__nv_bfloat16>, grid, 1024, 0, st, blocks, D, part,
                                (__nv_bfloat16*)dw0, (__nv_bfloat16*)dw1);
    return launch_dependent(weight_sum_kernel<float>, grid, 1024, 0, st, blocks, D, part, (float*)dw0, (float*)dw1);
}

// Blocks of the backward kernels: all that fit on the GPU at once, never more than there
// is work for.
int rows_bwd_blocks(int64_t rows, int per_sm) {
    const int64_t cap = per_sm * (int64_t)sm_count(), want = (rows + 15) / 16;
    return (int)(want < 1 ? 1 : want < cap ? want : cap);
}

}  // namespace gdn
