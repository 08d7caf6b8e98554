// gated_norm.cu -- RMS norm of every head's output row times the silu of a gate, and
// its gradients: the step behind the recurrence, before the output projection; and the
// last sum of a weight's gradient, which norm_rope.cu shares.
//
// Row x of D elements, gate z, weight w; r = (mean x^2 + eps)^(-1/2), xh = x r,
// sg = 1 / (1 + e^-z), act = z sg:
//   y = xh w act
//   dw = sum over rows of dy act xh,   dz = dy xh w (sg + act (1 - sg)),
//   dx = r (t - xh mean(t xh)),  t = dy act w.
// A group of lanes holds a row (rows.cuh: two neighbouring 16-byte pieces a lane) and
// takes kRows rows at a time, all their loads in flight together.  Bound by reading
// and writing the rows.

#include "gdn_internal.h"
#include "rows.cuh"

namespace gdn {
namespace {

using namespace rows;

constexpr int kThreads = 256;

struct GatedDims {
    int64_t rows;
    int H, D;
    int64_t x_stride, z_stride;  // elements from token to token
    float eps;
};

template <typename T, int G>
__global__ void __launch_bounds__(kThreads)
gated_norm_fwd_kernel(GatedDims d, const T* __restrict__ x, const T* __restrict__ z, const T* __restrict__ w,
                      T* __restrict__ y) {
    constexpr int VEC = kVec<T>, kRows = 4;
    const int c0 = (threadIdx.x % G) * 2 * VEC;
    const bool live = c0 < d.D;
    const int64_t first = ((int64_t)blockIdx.x * (kThreads / G) + threadIdx.x / G) * kRows;
    uint4 xr[kRows][2], zr[kRows][2];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int64_t row = first + i;
        xr[i][0] = xr[i][1] = zr[i][0] = zr[i][1] = make_uint4(0, 0, 0, 0);
        if (live && row < d.rows) {
            const int64_t tok = row / d.H;
            const int off = (int)(row - tok * d.H) * d.D + c0;
            const T* xp = x + tok * d.x_stride + off;
            const T* zp = z + tok * d.z_stride + off;
            xr[i][0] = lds16(xp), xr[i][1] = lds16(xp + VEC);
            zr[i][0] = lds16(zp), zr[i][1] = lds16(zp + VEC);
        }
    }
    float wv[2][VEC];
#pragma unroll
    for (int p = 0; p < 2; ++p) get(live ? ldg16(w + c0 + p * VEC) : make_uint4(0, 0, 0, 0), wv[p]);
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        float xv[2][VEC], ss = 0.f;
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            get(xr[i][p], xv[p]);
#pragma unroll
            for (int j = 0; j < VEC; ++j) ss = fmaf(xv[p][j], xv[p][j], ss);
        }
        const float r = rsqrtf(group_sum<G>(ss) / d.D + d.eps);
        const int64_t row = first + i;
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            float zv[VEC];
            get(zr[i][p], zv);
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const float act = __fdividef(zv[j], 1.f + expf(-zv[j]));
                xv[p][j] = xv[p][j] * r * wv[p][j] * act;
            }
            if (live && row < d.rows) sts16(y + row * d.D + c0 + p * VEC, put(xv[p]));
        }
    }
}

// Persistent blocks; each leaves one row of column sums in part [gridDim.x][D].
template <typename T, int G>
__global__ void __launch_bounds__(kThreads)
gated_norm_bwd_kernel(GatedDims d, const T* __restrict__ x, const T* __restrict__ z, const T* __restrict__ w,
                      const T* __restrict__ dy, T* __restrict__ dx, T* __restrict__ dz, float* __restrict__ part) {
    constexpr int VEC = kVec<T>, kRows = 2;
    extern __shared__ float sm[];  // [8 warps][D]
    const int c0 = (threadIdx.x % G) * 2 * VEC;
    const bool live = c0 < d.D;
    float wv[2][VEC], acc[2 * VEC];
#pragma unroll
    for (int p = 0; p < 2; ++p) get(live ? ldg16(w + c0 + p * VEC) : make_uint4(0, 0, 0, 0), wv[p]);
#pragma unroll
    for (int j = 0; j < 2 * VEC; ++j) acc[j] = 0.f;
    const int64_t per = (kThreads / G) * kRows, step = (int64_t)gridDim.x * per;
    for (int64_t base = (int64_t)blockIdx.x * per; base < d.rows; base += step) {
        const int64_t first = base + (threadIdx.x / G) * kRows;
        uint4 xr[kRows][2], zr[kRows][2], yr[kRows][2];
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int64_t row = first + i;
#pragma unroll
            for (int p = 0; p < 2; ++p) xr[i][p] = zr[i][p] = yr[i][p] = make_uint4(0, 0, 0, 0);
            if (live && row < d.rows) {
                const int64_t tok = row / d.H;
                const int off = (int)(row - tok * d.H) * d.D + c0;
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    xr[i][p] = lds16(x + tok * d.x_stride + off + p * VEC);
                    zr[i][p] = lds16(z + tok * d.z_stride + off + p * VEC);
                    yr[i][p] = lds16(dy + row * d.D + c0 + p * VEC);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            float xv[2][VEC], t[2][VEC], gz[2][VEC], ss = 0.f, tx = 0.f;
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                float zv[VEC];
                get(xr[i][p], xv[p]);
                get(zr[i][p], zv);
                get(yr[i][p], t[p]);
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    const float sg = __fdividef(1.f, 1.f + expf(-zv[j])), act = zv[j] * sg;
                    gz[p][j] = t[p][j] * wv[p][j] * xv[p][j] * (sg + act * (1.f - sg));
                    t[p][j] *= act;
                    ss = fmaf(xv[p][j], xv[p][j], ss);
                    tx = fmaf(t[p][j] * wv[p][j], xv[p][j], tx);
                }
            }
            ss = group_sum<G>(ss);
            tx = group_sum<G>(tx);
            const float r = rsqrtf(ss / d.D + d.eps);
            const float m = tx * r * r / d.D;  // mean(t xh) = r mean(t x), times r of xh
            const int64_t row = first + i;
#pragma unroll
            for (int p = 0; p < 2; ++p) {
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    acc[p * VEC + j] = fmaf(t[p][j], xv[p][j] * r, acc[p * VEC + j]);
                    gz[p][j] *= r;
                    xv[p][j] = r * (t[p][j] * wv[p][j] - xv[p][j] * m);
                }
                if (live && row < d.rows) {
                    sts16(dx + row * d.D + c0 + p * VEC, put(xv[p]));
                    sts16(dz + row * d.D + c0 + p * VEC, put(gz[p]));
                }
            }
        }
    }
    block_columns<G, VEC, kThreads / 32>(acc, c0, c0 + VEC, live, d.D, sm, part + (int64_t)blockIdx.x * d.D);
}

__device__ __forceinline__ void store1(float* p, float x) { *p = x; }
__device__ __forceinline__ void store1(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// dw[c] = sum over the blocks' rows of part, in a fixed order: a warp takes 32
// columns' rows w, w + 8, ..., the warps' sums are added in order.  blockIdx.y picks
// the side (part and dw of the queries, then of the keys).
template <typename T>
__global__ void __launch_bounds__(256)
weight_sum_kernel(int blocks, int D, const float* __restrict__ part, T* __restrict__ dw0, T* __restrict__ dw1) {
    __shared__ float sm[8][32];
    const int c = blockIdx.x * 32 + (threadIdx.x & 31), w = threadIdx.x >> 5;
    const float* p = part + (int64_t)blockIdx.y * blocks * D;
    float s = 0.f;
    if (c < D)
#pragma unroll 8
        for (int b = w; b < blocks; b += 8) s += p[(int64_t)b * D + c];
    sm[w][threadIdx.x & 31] = s;
    __syncthreads();
    if (w == 0 && c < D) {
        for (int i = 1; i < 8; ++i) s += sm[i][threadIdx.x];
        store1((blockIdx.y ? dw1 : dw0) + c, s);
    }
}

template <typename T, int G>
cudaError_t launch_g(const GatedCall& c, const GatedDims& d, bool bwd, cudaStream_t st) {
    const T *x = (const T*)c.x, *z = (const T*)c.z, *w = (const T*)c.w;
    if (!bwd) {
        const int64_t per = (int64_t)(kThreads / G) * 4;
        gated_norm_fwd_kernel<T, G><<<(unsigned)((d.rows + per - 1) / per), kThreads, 0, st>>>(d, x, z, w, (T*)c.y);
    } else {
        const size_t smem = (size_t)(kThreads / 32) * d.D * sizeof(float);
        gated_norm_bwd_kernel<T, G>
            <<<c.blocks, kThreads, smem, st>>>(d, x, z, w, (const T*)c.dy, (T*)c.dx, (T*)c.dz, c.part);
    }
    return cudaGetLastError();
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
        weight_sum_kernel<<<grid, 256, 0, st>>>(blocks, D, part, (__nv_bfloat16*)dw0, (__nv_bfloat16*)dw1);
    else weight_sum_kernel<<<grid, 256, 0, st>>>(blocks, D, part, (float*)dw0, (float*)dw1);
    return cudaGetLastError();
}

// Blocks of the backward kernels: a few per SM, never more than there is work for.
int rows_bwd_blocks(int64_t rows) {
    const int64_t cap = 4 * (int64_t)sm_count(), want = (rows + 63) / 64;
    return (int)(want < 1 ? 1 : want < cap ? want : cap);
}

}  // namespace gdn
