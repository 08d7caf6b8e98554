// la.cu -- linear attention with a fixed decay per head, on CUDA cores in 32 bits:
//   S_t = gamma S_{t-1} + v_t k_t^T,   o_t = S_t q_t,   gamma = e^g, g <= 0, S [V, K],
// chunked for prompts and training, and the recurrent step for single tokens.
//
// Its output and its three input gradients are one operation, a scan of three streams:
//   out_r = sum over s of gamma^|r-s| (a_r . b_s) c_s,   s up to r, or from r on,
//   M     = the decayed sum of c_s b_s^T over the tokens already passed,
// with (a, b, c, M) = (q, k, v, S) for o and (d_o, v, k, S^T) for dq, both in the order
// of time, and (v, d_o, q, dS^T) for dk and (k, q, d_o, dS) for dv against it, where dS
// is the gradient with respect to the state behind the token.  With rho the index in a
// chunk of n tokens in the order of the scan and rev = 1 against the order of time:
//   out = (A B^T .* D) C + diag(gamma^(rho + 1 - rev)) A M^T,  D_rs = gamma^|r-s| (rho_s <= rho_r)
//   M  <- gamma^n M + sum over rho of gamma^(n - 1 - rho + rev) c b^T.
// Every power of gamma has an exponent >= 0, so nothing overflows for g <= 0.
//
// Streams alone are too few to fill the GPU, so a sequence is cut into segments of L
// tokens: a first pass sums c b^T over each segment (from M = 0), a second links the sums
// to the states that enter the segments, and the third runs every segment from its own.

#include <cuda_bf16.h>

#include "gdn_internal.h"

namespace gdn {
namespace {

__device__ __forceinline__ float4 ld4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ void st1(float* p, float x) { *p = x; }
__device__ __forceinline__ void st1(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// gamma^e for e >= 0: 1 at e = 0 whatever g is (g = -inf forgets everything).
__device__ __forceinline__ float power(float g, float e) { return e > 0.f ? expf(g * e) : 1.f; }

constexpr int kTok = 64;  // tokens of a chunk

// Shared memory of the chunk kernel, in floats: rows of D (or 64) padded by four so
// that the float4 reads of neighbouring rows fall into different banks.
template <int D>
struct Smem {
    static constexpr int CS = D < 64 ? D : 64;  // columns of c that one CTA carries
    static constexpr int RA = D + 4, RC = CS + 4, RP = kTok + 4;
    static constexpr int A = 0, B = A + kTok * RA, C = B + kTok * RA, M = C + kTok * RC, P = M + D * RC,
                         W = P + kTok * RP, SIZE = W + kTok + 8;
};

// One CTA: one (stream, segment), CS columns of c, one role.  256 threads as 16 x 16:
// thread (ty, tx) has rows 4 ty .. 4 ty + 3 and columns 4 (tx) .. of each product, and
// M's rows ty, ty + 16, ... in registers; a copy in shared memory feeds A M^T.
template <int D, bool kOut>
__global__ void __launch_bounds__(256)
la_chunk_kernel(LaDims d, LaRoles roles) {
    using L = Smem<D>;
    constexpr int CT = L::CS / 16, BT = D / 16;  // columns of c, rows of b per thread
    extern __shared__ __align__(16) float sm[];
    float *sA = sm + L::A, *sB = sm + L::B, *sC = sm + L::C, *sM = sm + L::M, *sP = sm + L::P, *sW = sm + L::W;
    const LaRole& ro = roles.r[blockIdx.z];
    const int c0 = blockIdx.y * L::CS;
    if (c0 >= ro.Dc) return;
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const int nseg = kOut ? d.nseg : d.nseg - 1;  // the last segment's own sum feeds nobody
    const int64_t stream = blockIdx.x / nseg;
    const int slot = (int)(blockIdx.x % nseg);
    const int seg = !kOut && ro.rev ? slot + 1 : slot;
    const int b = (int)(stream / d.H), h = (int)(stream % d.H);
    const float g = d.log_decay[h];
    const int t_lo = seg * d.L, t_hi = min(d.T, t_lo + d.L);
    for (int e = tid; e <= kTok; e += 256) sW[e] = power(g, (float)e);

    // The state that enters: M[c][b] of the caller's [V, K] matrices by strides.
    float m[BT][CT];
#pragma unroll
    for (int i = 0; i < BT; ++i)
#pragma unroll
        for (int j = 0; j < CT; ++j) m[i][j] = 0.f;
    if (kOut) {
        const bool first = seg == (ro.rev ? d.nseg - 1 : 0);
        const int64_t VK = (int64_t)ro.Db * ro.Dc;
        const float* src = first ? (ro.m0 ? ro.m0 + stream * VK : nullptr)
                                 : ro.R + (stream * (d.nseg - 1) + (ro.rev ? seg : seg - 1)) * VK;
        if (src) {
#pragma unroll
            for (int i = 0; i < BT; ++i)
#pragma unroll
                for (int j = 0; j < CT; ++j) {
                    const int bb = ty + 16 * i, cc = c0 + tx * CT + j;
                    if (bb < ro.Db && cc < ro.Dc) m[i][j] = src[cc * ro.m_sc + bb * ro.m_sb];
                }
        }
    }

    const float* pa = (const float*)ro.a + (int64_t)b * d.T * ro.sa + (int64_t)h * ro.Db;
    const float* pb = (const float*)ro.b + (int64_t)b * d.T * ro.sb + (int64_t)h * ro.Db;
    const float* pc = (const float*)ro.c + (int64_t)b * d.T * ro.sc + (int64_t)h * ro.Dc + c0;
    float* po = (float*)ro.out + ((int64_t)b * d.T * d.H + h) * ro.Dc + c0;
    const int cw = min(L::CS, ro.Dc - c0);
    const int chunks = (t_hi - t_lo + kTok - 1) / kTok;
    for (int it = 0; it < chunks; ++it) {
        const int t0 = t_lo + (ro.rev ? chunks - 1 - it : it) * kTok, n = min(kTok, t_hi - t0);
        __syncthreads();
        const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int i = tid; i < kTok * (D / 4); i += 256) {
            const int r = i / (D / 4), x = (i % (D / 4)) * 4;
            const bool in = r < n && x < ro.Db;
            if (kOut) *(float4*)(sA + r * L::RA + x) = in ? ld4(pa + (int64_t)(t0 + r) * ro.sa + x) : zero;
            *(float4*)(sB + r * L::RA + x) = in ? ld4(pb + (int64_t)(t0 + r) * ro.sb + x) : zero;
        }
        for (int i = tid; i < kTok * (L::CS / 4); i += 256) {
            const int r = i / (L::CS / 4), x = (i % (L::CS / 4)) * 4;
            *(float4*)(sC + r * L::RC + x) = r < n && x < cw ? ld4(pc + (int64_t)(t0 + r) * ro.sc + x) : zero;
        }
        if (kOut) {
#pragma unroll
            for (int i = 0; i < BT; ++i)
#pragma unroll
                for (int j = 0; j < CT; ++j) sM[(ty + 16 * i) * L::RC + tx * CT + j] = m[i][j];
        }
        __syncthreads();

        float acc[4][CT];
        if (kOut) {
            // scores: rows 4 ty + i, columns tx + 16 j
            float p[4][4] = {};
#pragma unroll 4
            for (int x = 0; x < D; x += 4) {
                float4 av[4], bv[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) av[i] = *(const float4*)(sA + (4 * ty + i) * L::RA + x);
#pragma unroll
                for (int j = 0; j < 4; ++j) bv[j] = *(const float4*)(sB + (tx + 16 * j) * L::RA + x);
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        p[i][j] = fmaf(av[i].x, bv[j].x, p[i][j]);
                        p[i][j] = fmaf(av[i].y, bv[j].y, p[i][j]);
                        p[i][j] = fmaf(av[i].z, bv[j].z, p[i][j]);
                        p[i][j] = fmaf(av[i].w, bv[j].w, p[i][j]);
                    }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int r = 4 * ty + i, s = tx + 16 * j, dist = ro.rev ? s - r : r - s;
                    sP[r * L::RP + s] = dist >= 0 ? p[i][j] * sW[dist] : 0.f;
                }
            // A M^T from the state that entered the chunk
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < CT; ++j) acc[i][j] = 0.f;
#pragma unroll 2
            for (int x = 0; x < D; x += 4) {
                float av[4][4], mv[4][CT];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float4 f = *(const float4*)(sA + (4 * ty + i) * L::RA + x);
                    av[i][0] = f.x, av[i][1] = f.y, av[i][2] = f.z, av[i][3] = f.w;
                }
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                    for (int j = 0; j < CT; ++j) mv[e][j] = sM[(x + e) * L::RC + tx * CT + j];
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
#pragma unroll
                        for (int j = 0; j < CT; ++j) acc[i][j] = fmaf(av[i][e], mv[e][j], acc[i][j]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = 4 * ty + i, e = ro.rev ? n - 1 - r : r + 1;
                const float w = sW[max(e, 0)];
#pragma unroll
                for (int j = 0; j < CT; ++j) acc[i][j] *= w;
            }
            __syncthreads();
#pragma unroll 2
            for (int s = 0; s < kTok; s += 4) {
                float pv[4][4], cv[4][CT];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float4 f = *(const float4*)(sP + (4 * ty + i) * L::RP + s);
                    pv[i][0] = f.x, pv[i][1] = f.y, pv[i][2] = f.z, pv[i][3] = f.w;
                }
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                    for (int j = 0; j < CT; ++j) cv[e][j] = sC[(s + e) * L::RC + tx * CT + j];
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
#pragma unroll
                        for (int j = 0; j < CT; ++j) acc[i][j] = fmaf(pv[i][e], cv[e][j], acc[i][j]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = 4 * ty + i;
#pragma unroll
                for (int j = 0; j < CT; ++j)
                    if (r < n && tx * CT + j < cw)
                        po[(int64_t)(t0 + r) * d.H * ro.Dc + tx * CT + j] = acc[i][j];
            }
        }
        // M <- gamma^n M + sum of gamma^(n-1-rho+rev) b c^T
        const float gn = sW[n];
#pragma unroll
        for (int i = 0; i < BT; ++i)
#pragma unroll
            for (int j = 0; j < CT; ++j) m[i][j] *= gn;
#pragma unroll 2
        for (int s = 0; s < n; ++s) {
            const float w = sW[ro.rev ? s + 1 : n - 1 - s];
            float cv[CT];
#pragma unroll
            for (int j = 0; j < CT; ++j) cv[j] = w * sC[s * L::RC + tx * CT + j];
#pragma unroll
            for (int i = 0; i < BT; ++i) {
                const float bv = sB[s * L::RA + ty + 16 * i];
#pragma unroll
                for (int j = 0; j < CT; ++j) m[i][j] = fmaf(bv, cv[j], m[i][j]);
            }
        }
    }

    // What leaves: a segment's own sum, or the state behind the last one.
    const bool last = kOut && ro.mT && seg == (ro.rev ? 0 : d.nseg - 1);
    if (!kOut || last) {
        const int64_t VK = (int64_t)ro.Db * ro.Dc;
        float* dst = kOut ? ro.mT + stream * VK : const_cast<float*>(ro.R) + (stream * nseg + slot) * VK;
#pragma unroll
        for (int i = 0; i < BT; ++i)
#pragma unroll
            for (int j = 0; j < CT; ++j) {
                const int bb = ty + 16 * i, cc = c0 + tx * CT + j;
                if (bb < ro.Db && cc < ro.Dc) dst[cc * ro.m_sc + bb * ro.m_sb] = m[i][j];
            }
    }
}

template <int D, bool kOut>
cudaError_t launch_chunk(const LaDims& d, const LaRoles& roles, cudaStream_t st) {
    using L = Smem<D>;
    const size_t smem = L::SIZE * sizeof(float);
    cudaError_t e = cudaFuncSetAttribute(la_chunk_kernel<D, kOut>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)smem);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)(d.NS() * (kOut ? d.nseg : d.nseg - 1)), D / L::CS, roles.n);
    la_chunk_kernel<D, kOut><<<grid, 256, smem, st>>>(d, roles);
    return cudaGetLastError();
}

template <bool kOut>
cudaError_t launch_width(const LaDims& d, const LaRoles& roles, cudaStream_t st) {
    switch (d.K > d.V ? d.K : d.V) {
        case 16: return launch_chunk<16, kOut>(d, roles, st);
        case 32: return launch_chunk<32, kOut>(d, roles, st);
        case 64: return launch_chunk<64, kOut>(d, roles, st);
        default: return launch_chunk<128, kOut>(d, roles, st);
    }
}

// The segments' sums R become, in place, the states that enter the segments behind them
// (in the order of the scan): S <- gamma^L S + R from the caller's state on.  A thread
// has four elements of one stream's matrix; its loads do not wait for one another.
__global__ void __launch_bounds__(256)
la_link_kernel(LaDims d, LaRoles roles) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const LaRole& ro = roles.r[blockIdx.y];
    const int64_t VK = (int64_t)ro.Db * ro.Dc, i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    const int64_t stream = i / VK, e = i % VK;
    if (stream >= d.NS()) return;
    const float g = d.log_decay[stream % d.H];
    const int n = d.nseg - 1;
    const float step = power(g, (float)d.L), tail = power(g, (float)(d.T - n * d.L));
    float* R = const_cast<float*>(ro.R) + stream * n * VK + e;
    float4 s = ro.m0 ? *(const float4*)(ro.m0 + stream * VK + e) : make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = 0; k0 < n; k0 += 8) {
        float4 r[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k0 + k < n) r[k] = *(const float4*)(R + (ro.rev ? n - 1 - k0 - k : k0 + k) * VK);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k0 + k < n) {
                const float w = ro.rev && k0 + k == 0 ? tail : step;
                s = make_float4(fmaf(w, s.x, r[k].x), fmaf(w, s.y, r[k].y), fmaf(w, s.z, r[k].z),
                                fmaf(w, s.w, r[k].w));
                *(float4*)(R + (ro.rev ? n - 1 - k0 - k : k0 + k) * VK) = s;
            }
    }
}

// ------------------------------------------------------------ single tokens

// N consecutive values (aligned to N elements) as floats, and N floats back.
template <int N>
__device__ __forceinline__ void ldn(const float* p, float (&f)[N]) {
    if constexpr (N == 4) {
        const float4 x = __ldcs(reinterpret_cast<const float4*>(p));
        f[0] = x.x, f[1] = x.y, f[2] = x.z, f[3] = x.w;
    } else if constexpr (N == 2) {
        const float2 x = __ldcs(reinterpret_cast<const float2*>(p));
        f[0] = x.x, f[1] = x.y;
    } else {
        f[0] = __ldcs(p);
    }
}
template <int N>
__device__ __forceinline__ void ldn(const __nv_bfloat16* p, float (&f)[N]) {
    if constexpr (N == 4) {
        const uint2 x = *reinterpret_cast<const uint2*>(p);
        f[0] = __uint_as_float(x.x << 16), f[1] = __uint_as_float(x.x & 0xffff0000u);
        f[2] = __uint_as_float(x.y << 16), f[3] = __uint_as_float(x.y & 0xffff0000u);
    } else if constexpr (N == 2) {
        const uint32_t x = *reinterpret_cast<const uint32_t*>(p);
        f[0] = __uint_as_float(x << 16), f[1] = __uint_as_float(x & 0xffff0000u);
    } else {
        f[0] = __bfloat162float(*p);
    }
}
template <int N>
__device__ __forceinline__ void stn(float* p, const float (&f)[N]) {
    if constexpr (N == 4) __stcs(reinterpret_cast<float4*>(p), make_float4(f[0], f[1], f[2], f[3]));
    else if constexpr (N == 2) __stcs(reinterpret_cast<float2*>(p), make_float2(f[0], f[1]));
    else __stcs(p, f[0]);
}

constexpr int kRows = 8;  // state rows of a warp

// The sums over the warp of 8 values a lane; lane l receives that of row
// (l / 16) * 4 + (l / 8 % 2) * 2 + l / 4 % 2: at each of the first three steps a lane
// keeps half of its values and hands on the others, 9 exchanges instead of 40.
__device__ __forceinline__ float sum_rows(const float (&v)[kRows], int lane) {
    float a[4], b[2], c;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bool up = lane & 16;
        a[i] = (up ? v[i + 4] : v[i]) + __shfl_xor_sync(0xffffffffu, up ? v[i] : v[i + 4], 16);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const bool up = lane & 8;
        b[i] = (up ? a[i + 2] : a[i]) + __shfl_xor_sync(0xffffffffu, up ? a[i] : a[i + 2], 8);
    }
    const bool up = lane & 4;
    c = (up ? b[1] : b[0]) + __shfl_xor_sync(0xffffffffu, up ? b[0] : b[1], 4);
    c += __shfl_xor_sync(0xffffffffu, c, 2);
    return c + __shfl_xor_sync(0xffffffffu, c, 1);
}

// A warp holds kRows rows of one head's state in registers across the call's tokens,
// lane l the K/32 columns from l K/32 on (K = 16: lanes 0-15, one column each).  Bound
// by reading and writing the state once.
template <typename T, int KPL>
__global__ void __launch_bounds__(256)
la_decode_kernel(LaDims d, const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v, int64_t sq,
                 int64_t sk, int64_t sv, float* __restrict__ state, T* __restrict__ o) {
    const int lane = threadIdx.x & 31, groups = d.V / kRows, c0 = lane * KPL;
    const int64_t unit = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (unit >= d.NS() * groups) return;
    const int64_t stream = unit / groups;
    const int v0 = (int)(unit % groups) * kRows, h = (int)(stream % d.H);
    const int64_t b = stream / d.H;
    const bool live = c0 < d.K;
    float* rows = state + (stream * d.V + v0) * d.K + c0;
    float S[kRows][KPL];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        if (live) ldn<KPL>(rows + r * d.K, S[r]);
        else
#pragma unroll
            for (int i = 0; i < KPL; ++i) S[r][i] = 0.f;
    }
    const float gamma = expf(d.log_decay[h]);
    const int mine = (lane >> 4) * 4 + (lane >> 3 & 1) * 2 + (lane >> 2 & 1);
    for (int t = 0; t < d.T; ++t) {
        const int64_t tok = b * d.T + t;
        float kv[KPL] = {}, qv[KPL] = {}, vv[2][4], red[kRows];
        if (live) {
            ldn<KPL>(k + tok * sk + (int64_t)h * d.K + c0, kv);
            ldn<KPL>(q + tok * sq + (int64_t)h * d.K + c0, qv);
        }
        ldn<4>(v + tok * sv + (int64_t)h * d.V + v0, vv[0]);
        ldn<4>(v + tok * sv + (int64_t)h * d.V + v0 + 4, vv[1]);
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            red[r] = 0.f;
#pragma unroll
            for (int i = 0; i < KPL; ++i) {
                S[r][i] = fmaf(vv[r >> 2][r & 3], kv[i], gamma * S[r][i]);
                red[r] = fmaf(S[r][i], qv[i], red[r]);
            }
        }
        const float sum = sum_rows(red, lane);
        if ((lane & 3) == 0) st1(o + (tok * d.H + h) * d.V + v0 + mine, sum);
    }
    if (live)
#pragma unroll
        for (int r = 0; r < kRows; ++r) stn<KPL>(rows + r * d.K, S[r]);
}

template <typename T>
cudaError_t launch_decode_t(const LaDims& d, const void* q, const void* k, const void* v, int64_t sq, int64_t sk,
                            int64_t sv, float* state, void* o, cudaStream_t st) {
    const unsigned grid = (unsigned)((d.NS() * (d.V / kRows) + 7) / 8);
    const T *qp = (const T*)q, *kp = (const T*)k, *vp = (const T*)v;
    if (d.K <= 32) la_decode_kernel<T, 1><<<grid, 256, 0, st>>>(d, qp, kp, vp, sq, sk, sv, state, (T*)o);
    else if (d.K == 64) la_decode_kernel<T, 2><<<grid, 256, 0, st>>>(d, qp, kp, vp, sq, sk, sv, state, (T*)o);
    else la_decode_kernel<T, 4><<<grid, 256, 0, st>>>(d, qp, kp, vp, sq, sk, sv, state, (T*)o);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_la_states(const LaDims& d, InType ty, const LaRoles& roles, cudaStream_t st) {
    return ty == InType::BF16 ? launch_la_states_tc(d, roles, st) : launch_width<false>(d, roles, st);
}
cudaError_t launch_la_link(const LaDims& d, const LaRoles& roles, cudaStream_t st) {
    const int64_t threads = d.NS() * d.K * d.V / 4;
    return launch_dependent(la_link_kernel, dim3((unsigned)((threads + 255) / 256), roles.n), 256, 0, st, d, roles);
}
cudaError_t launch_la_scan(const LaDims& d, InType ty, const LaRoles& roles, cudaStream_t st) {
    return ty == InType::BF16 ? launch_la_scan_tc(d, roles, st) : launch_width<true>(d, roles, st);
}

cudaError_t launch_la_decode(const LaDims& d, InType ty, const void* q, const void* k, const void* v, int64_t sq,
                             int64_t sk, int64_t sv, float* state, void* o, cudaStream_t st) {
    return ty == InType::BF16 ? launch_decode_t<__nv_bfloat16>(d, q, k, v, sq, sk, sv, state, o, st)
                              : launch_decode_t<float>(d, q, k, v, sq, sk, sv, state, o, st);
}

// How a call cuts its sequences, in whole 128-token tiles: the cut with the least
// estimated time, in units of a tile of the scan.  A CTA takes its tiles one after the
// other behind a fixed part (launch, first loads, the state that enters); the CTAs go in
// waves of one per SM; with several segments the sums (0.6 of a tile each) and the link
// come first.  The backward's three scans want fewer segments than the forward's one;
// but cut like the forward's it can take over the forward's sums (`saved`).
namespace {
constexpr double kScanFixed = 4, kSumFixed = 3, kSumTile = 0.6, kLinkFixed = 1.5;

double cut_cost(int64_t streams, int64_t tiles, int64_t per, int scans, int sums) {
    const int64_t nseg = (tiles + per - 1) / per, sms = sm_count();
    auto waves = [&](int64_t ctas) { return (double)((ctas + sms - 1) / sms); };
    double t = waves(streams * scans * nseg) * (per + kScanFixed);
    if (nseg > 1) t += waves(streams * sums * (nseg - 1)) * (kSumTile * per + kSumFixed) + kLinkFixed;
    return t;
}

// The best number of tiles a segment, and its cost.
int64_t best_cut(int64_t streams, int64_t tiles, int scans, int sums, double* cost) {
    int64_t best = tiles;
    *cost = cut_cost(streams, tiles, tiles, scans, sums);
    const int64_t most = streams * scans < sm_count() ? 2 * sm_count() / (streams * scans) : 1;
    for (int64_t n = 2; n <= most && n <= tiles; ++n) {
        const int64_t per = (tiles + n - 1) / n;
        const double c = cut_cost(streams, tiles, per, scans, sums);
        if (c < *cost) best = per, *cost = c;
    }
    return best;
}
}  // namespace

void la_segments(LaDims* d, bool bwd) {
    const int64_t tiles = (d->T + 127) / 128, streams = d->NS();
    int64_t per = tiles;
    if (streams > 0 && tiles > 1) {
        double cf, cb;
        per = best_cut(streams, tiles, 1, 1, &cf);
        if (bwd) {
            const double shared = cut_cost(streams, tiles, per, 3, 1);
            const int64_t own = best_cut(streams, tiles, 3, 2, &cb);
            if (cb < shared) per = own;
        }
    }
    d->L = (int)(per * 128);
    d->nseg = tiles ? (int)((tiles + per - 1) / per) : 1;
}

}  // namespace gdn
