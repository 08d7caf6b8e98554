// la.cu -- linear attention with a fixed decay per head: float32 inputs, and the step:
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

#include <type_traits>

#include "f32x2.cuh"
#include "gdn_internal.h"

namespace gdn {
namespace {

__device__ __forceinline__ void st1(float* p, float x) { *p = x; }
__device__ __forceinline__ void st1(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// gamma^e for e >= 0: 1 at e = 0 whatever g is (g = -inf forgets everything).
__device__ __forceinline__ float power(float g, float e) { return e > 0.f ? expf(g * e) : 1.f; }

constexpr int kTok = 64;  // tokens of a chunk

// A float32 product on the tensor cores: each factor is split into two tf32 numbers, its
// rounding to 11 bits and the rest (which the product reads 11 bits of), and
// x y = hi hi + (hi lo + lo hi); what is left out, lo lo, is below 2^-22 of a product and
// of either sign.  (Cutting instead of rounding saves 5% of the time, but leaves a lo lo
// of one sign.)  The small products have sums of their own, and no sum on the tensor
// cores runs over more than one chunk: what is carried from chunk to chunk is added in
// float32.  Results are within 5.5e-7 of the value (relative L2, T up to 4096), up to twice
// as far as the same sums in float32.
//
// The rounding takes a number within 2^-12 of the largest one to infinity, and what is left
// of an infinity is a NaN, so no such number comes out finite.  kSafe's hi stops at the
// largest tf32 number, but in every split it takes 14 to 32% more time (B8 T2048 H8 K = V = 64
// forward 127 -> 149 us, B4 T2048 H6 K = V = 128 backward 298 -> 394).  So a CTA looks at its
// results, and does its work again that way if one is not finite (127 -> 129, 298 -> 300).
//
// These warp-level products run at 512 a cycle and SM, which three tf32 products for one
// make 170; float32 arithmetic has 128, of which its operands' reads from shared memory
// left about half (B4 T2048 H6 K = V = 128 forward 197 us, now 147).
struct Sum {
    float hi[4], lo[4];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < 4; ++i) hi[i] = lo[i] = 0.f;
    }
    __device__ __forceinline__ float get(int i) const { return hi[i] + lo[i]; }
};
template <int N, bool kSafe>
struct Split {
    uint32_t hi[N], lo[N];
    __device__ __forceinline__ void set(int i, float x) {
        if constexpr (kSafe)
            asm("cvt.rna.satfinite.tf32.f32 %0, %1;" : "=r"(hi[i]) : "f"(x));
        else
            hi[i] = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;
        lo[i] = __float_as_uint(x - __uint_as_float(hi[i]));
    }
};
__device__ __forceinline__ void mma8(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
    asm volatile(
        "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
// d[j] += a b[j]; the products of one sum are kept apart, each waits for the one before
template <int N, bool kSafe>
__device__ __forceinline__ void mma8(Sum (&d)[N], const Split<4, kSafe>& a, const Split<2, kSafe> (&b)[N]) {
#pragma unroll
    for (int j = 0; j < N; ++j) mma8(d[j].lo, a.lo, b[j].hi);
#pragma unroll
    for (int j = 0; j < N; ++j) mma8(d[j].hi, a.hi, b[j].hi);
#pragma unroll
    for (int j = 0; j < N; ++j) mma8(d[j].lo, a.hi, b[j].lo);
}

// Shared memory of the chunk kernel, in floats.  With rows 4 (mod 32) words apart, the
// fragments read along a row (8 rows, 4 columns) and those read across rows 2 t, 2 t + 1
// (the sum over tokens may take them in any order) fall into 32 banks; P and M's copy
// have rows 8 apart for theirs.  Up to D = 64 two CTAs share an SM and hide each other's
// loads; at 128 one has it alone and two buffers of A, B, C, so that a chunk is loaded
// while the one before it is worked on.
template <int D>
struct Smem {
    static constexpr int CS = D < 64 ? D : 64;  // columns of c that one CTA carries
    static constexpr int RA = D + 4, RC = CS + 4, RM = CS + 8, RP = kTok + 8;
    static constexpr int A = 0, B = A + kTok * RA, C = B + kTok * RA, BUF = C + kTok * RC;
    static constexpr int THREADS = D > 64 ? 512 : 256, COLS = THREADS / 128;  // groups of columns
    static constexpr int NBUF = D > 64 ? 2 : 1, M = NBUF * BUF, P = M + D * RM, W = P + kTok * RP, SIZE = W + kTok + 8;
};
static_assert(Smem<128>::SIZE * 4 <= 232448 && Smem<64>::SIZE * 8 <= 231424, "shared memory");

// One CTA: one (stream, segment), CS columns of c, one role.  Eight warps: for the scores
// and the outputs 4 groups of 16 rows by 2 halves of the columns, for M RG groups of
// rows (b) by CG of columns; a warp's part of M stays in its registers, and a copy in
// shared memory feeds A M^T.  Warps w and w + 4, which share a scheduler, have row groups
// w and 3 - w, so that what the causal mask leaves out is shared evenly.  (At 128 columns
// sixteen warps of half the columns each: 1 to 7% less time.)  Bound by the warps' issue
// and the tensor pipe together: 61 and 54% of their rates where two CTAs share an SM.
template <int D, bool kOut>
__global__ void __launch_bounds__(Smem<D>::THREADS, D > 64 ? 1 : 2)
la_chunk_kernel(LaDims d, LaRoles roles) {
    using L = Smem<D>;
    constexpr int RG = D < 64 ? D / 16 : 4, MT = D / 16 / RG;                  // M: groups of rows, tiles in each
    constexpr int WARPS = L::THREADS / 32, CM = L::CS / 8;
    constexpr int CG = WARPS / RG < CM ? WARPS / RG : CM, NM = CM / CG;        // and of columns
    constexpr int NO = CM / L::COLS, NY = kTok / 8 / L::COLS;                  // column tiles of outputs, scores
    extern __shared__ __align__(16) float sm[];
    float *sM = sm + L::M, *sP = sm + L::P, *sW = sm + L::W;
    await_previous();
    const LaRole& ro = roles.r[blockIdx.z];
    const int c0 = blockIdx.y * L::CS;
    if (c0 >= ro.Dc) return;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gq = lane >> 2, tq = lane & 3;
    const int nseg = kOut ? d.nseg : d.nseg - 1;  // the last segment's own sum feeds nobody
    const int64_t stream = blockIdx.x / nseg;
    const int slot = (int)(blockIdx.x % nseg);
    const int seg = !kOut && ro.rev ? slot + 1 : slot;
    const int b = (int)(stream / d.H), h = (int)(stream % d.H);
    const float g = d.log_decay[h];
    const int t_lo = seg * d.L, t_hi = min(d.T, t_lo + d.L);
    const int chunks = (t_hi - t_lo + kTok - 1) / kTok;
    for (int e = tid; e <= kTok; e += L::THREADS) sW[e] = power(g, (float)e);

    const float* pa = (const float*)ro.a + (int64_t)b * d.T * ro.sa + (int64_t)h * ro.Db;
    const float* pb = (const float*)ro.b + (int64_t)b * d.T * ro.sb + (int64_t)h * ro.Db;
    const float* pc = (const float*)ro.c + (int64_t)b * d.T * ro.sc + (int64_t)h * ro.Dc + c0;
    float* po = (float*)ro.out + ((int64_t)b * d.T * d.H + h) * ro.Dc + c0;
    const int cw = min(L::CS, ro.Dc - c0);
    auto chunk_t0 = [&](int it) { return t_lo + (ro.rev ? chunks - 1 - it : it) * kTok; };
    // rows past the sequence and columns past the tensors' are zeros
    auto load = [&](int it) {
        const int t0 = chunk_t0(it), n = min(kTok, t_hi - t0);
        float* buf = sm + it % L::NBUF * L::BUF;
        auto rows = [&](float* to, int stride, const float* from, int64_t step, int width, int cols) {
            for (int i = tid; i < kTok * (width / 4); i += L::THREADS) {
                const int r = i / (width / 4), x = (i % (width / 4)) * 4;
                const bool in = r < n && x < cols;
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                                 (uint32_t)__cvta_generic_to_shared(to + r * stride + x)),
                             "l"(in ? from + (int64_t)(t0 + r) * step + x : from), "r"(in ? 16 : 0)
                             : "memory");
            }
        };
        if (kOut) rows(buf + L::A, L::RA, pa, ro.sa, D, ro.Db);
        rows(buf + L::B, L::RA, pb, ro.sb, D, ro.Db);
        rows(buf + L::C, L::RC, pc, ro.sc, L::CS, cw);
        asm volatile("cp.async.commit_group;" ::: "memory");
    };

    // M[c][b] of the caller's [V, K] matrices by strides: this warp's tiles of 16 rows (b)
    // by 8 columns (c).  A lane has rows gq and gq + 8, columns 2 tq and 2 tq + 1 of a tile.
    const int mg = warp / CG, mc = warp % CG;
    const bool carries = RG * CG == WARPS || warp < RG * CG;
    float m[MT][NM][4];
    auto row_b = [&](int x) { return (x * RG + mg) * 16 + gq; };
    auto col_c = [&](int j) { return (mc * NM + j) * 8 + 2 * tq; };
    auto each = [&](auto&& f) {  // f(row, column within the CTA's, element)
#pragma unroll
        for (int x = 0; x < MT; ++x)
#pragma unroll
            for (int j = 0; j < NM; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) f(row_b(x) + 8 * (e >> 1), col_c(j) + (e & 1), m[x][j][e]);
    };
    const bool last = kOut && ro.mT && seg == (ro.rev ? 0 : d.nseg - 1);
    const bool leaves = carries && (!kOut || last);  // M does: a segment's own sum, or the last state
    const int part = warp >> 2, r0 = (part & 1 ? 3 - (warp & 3) : warp & 3) * 16;  // group of columns, first row
    const int y0 = part * NY * 8, o0 = part * NO * 8;                             // first columns
    // All chunks.  Returns 0, or a NaN if some result is not finite.
    auto pass = [&](auto safe) {
        using SplitA = Split<4, decltype(safe)::value>;
        using SplitB = Split<2, decltype(safe)::value>;
        float bad = 0.f;
        load(0);
        each([](int, int, float& x) { x = 0.f; });
        if (kOut && carries) {
            const bool first = seg == (ro.rev ? d.nseg - 1 : 0);
            const int64_t VK = (int64_t)ro.Db * ro.Dc;
            const float* src = first ? (ro.m0 ? ro.m0 + stream * VK : nullptr)
                                     : ro.R + (stream * (d.nseg - 1) + (ro.rev ? seg : seg - 1)) * VK;
            if (src)
                each([&](int bb, int cc, float& x) {
                    if (bb < ro.Db && cc < cw) x = src[(c0 + cc) * ro.m_sc + bb * ro.m_sb];
                });
        }

        for (int it = 0; it < chunks; ++it) {
            const int t0 = chunk_t0(it), n = min(kTok, t_hi - t0);
            const float *sA = sm + it % L::NBUF * L::BUF + L::A, *sB = sA + L::B, *sC = sA + L::C;
            if (L::NBUF == 1 && it) {
                __syncthreads();  // the chunk before is done with the buffer
                load(it);
            }
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            if (kOut && carries) {
#pragma unroll
                for (int x = 0; x < MT; ++x)
#pragma unroll
                    for (int j = 0; j < NM; ++j)
#pragma unroll
                        for (int e = 0; e < 4; e += 2)
                            *(float2*)(sM + (row_b(x) + 4 * e) * L::RM + col_c(j)) =
                                make_float2(m[x][j][e], m[x][j][e + 1]);
            }
            __syncthreads();  // this chunk is there, the other buffer and P are free
            if (L::NBUF == 2 && it + 1 < chunks) load(it + 1);

            if (kOut) {
                auto rows_a = [&](int k, SplitA& a) {  // A's fragment: rows r0 .. r0 + 15, columns k .. k + 7
                    const float* at = sA + (r0 + gq) * L::RA + k + tq;
                    a.set(0, at[0]), a.set(1, at[8 * L::RA]), a.set(2, at[4]), a.set(3, at[8 * L::RA + 4]);
                };
                {  // scores, where the mask leaves some of this warp's
                    Sum y[NY];
#pragma unroll
                    for (int j = 0; j < NY; ++j) y[j].zero();
                    if (ro.rev ? y0 + NY * 8 > r0 : y0 <= r0 + 15) {
#pragma unroll 8
                        for (int k = 0; k < D; k += 8) {
                            SplitA a;
                            SplitB f[NY];
                            rows_a(k, a);
#pragma unroll
                            for (int j = 0; j < NY; ++j) {
                                const float* at = sB + (y0 + j * 8 + gq) * L::RA + k + tq;
                                f[j].set(0, at[0]), f[j].set(1, at[4]);
                            }
                            mma8(y, a, f);
                        }
                    }
#pragma unroll
                    for (int j = 0; j < NY; ++j)
#pragma unroll
                        for (int e = 0; e < 4; e += 2) {
                            const int r = r0 + gq + 4 * e, s = y0 + j * 8 + 2 * tq, dist = ro.rev ? s - r : r - s;
                            const int next = ro.rev ? dist + 1 : dist - 1;
                            *(float2*)(sP + r * L::RP + s) =
                                make_float2(dist >= 0 ? y[j].get(e) * sW[dist] : 0.f,
                                            next >= 0 ? y[j].get(e + 1) * sW[next] : 0.f);
                        }
                }
                Sum o[NO];
#pragma unroll
                for (int j = 0; j < NO; ++j) o[j].zero();
                const int cb = o0 + gq;
                // A M^T, the state that entered the chunk
#pragma unroll 8
                for (int k = 0; k < D; k += 8) {
                    SplitA a;
                    SplitB f[NO];
                    rows_a(k, a);
#pragma unroll
                    for (int j = 0; j < NO; ++j) {
                        const float* at = sM + (k + tq) * L::RM + cb + j * 8;
                        f[j].set(0, at[0]), f[j].set(1, at[4 * L::RM]);
                    }
                    mma8(o, a, f);
                }
#pragma unroll
                for (int e = 0; e < 4; e += 2) {
                    const int r = r0 + gq + 4 * e;
                    const float w = sW[max(ro.rev ? n - 1 - r : r + 1, 0)];
#pragma unroll
                    for (int j = 0; j < NO; ++j)
#pragma unroll
                        for (int i = e; i < e + 2; ++i) o[j].hi[i] *= w, o[j].lo[i] *= w;
                }
                __syncthreads();
                const int s_lo = ro.rev ? r0 : 0, s_hi = ro.rev ? kTok : r0 + 16;
#pragma unroll 4
                for (int s = s_lo; s < s_hi; s += 8) {
                    const float2 x = *(const float2*)(sP + (r0 + gq) * L::RP + s + 2 * tq),
                                 z = *(const float2*)(sP + (r0 + gq + 8) * L::RP + s + 2 * tq);
                    SplitA a;
                    SplitB f[NO];
                    a.set(0, x.x), a.set(1, z.x), a.set(2, x.y), a.set(3, z.y);
#pragma unroll
                    for (int j = 0; j < NO; ++j) {
                        const float* at = sC + (s + 2 * tq) * L::RC + cb + j * 8;
                        f[j].set(0, at[0]), f[j].set(1, at[L::RC]);
                    }
                    mma8(o, a, f);
                }
#pragma unroll
                for (int j = 0; j < NO; ++j)
#pragma unroll
                    for (int e = 0; e < 4; e += 2) {
                        const int r = r0 + gq + 4 * e, c = o0 + j * 8 + 2 * tq;
                        const float2 y = make_float2(o[j].get(e), o[j].get(e + 1));
                        bad = fmaf(y.x, 0.f, fmaf(y.y, 0.f, bad));
                        if (r < n && c < cw) *(float2*)(po + (int64_t)(t0 + r) * d.H * ro.Dc + c) = y;
                    }
            }
            // M <- gamma^n M + sum of gamma^(n-1-rho+rev) b c^T
            if (carries) {
                Sum u[MT][NM];
#pragma unroll
                for (int x = 0; x < MT; ++x)
#pragma unroll
                    for (int j = 0; j < NM; ++j) u[x][j].zero();
#pragma unroll 4
                for (int s = 0; s < n; s += 8) {
                    const int s0 = s + 2 * tq;
                    const float w0 = sW[ro.rev ? s0 + 1 : max(n - 1 - s0, 0)],
                                w1 = sW[ro.rev ? s0 + 2 : max(n - 2 - s0, 0)];
                    SplitA a[MT];
#pragma unroll
                    for (int x = 0; x < MT; ++x) {
                        const float* at = sB + s0 * L::RA + row_b(x);
                        a[x].set(0, at[0]), a[x].set(1, at[8]), a[x].set(2, at[L::RA]), a[x].set(3, at[L::RA + 8]);
                    }
                    SplitB f[NM];
#pragma unroll
                    for (int j = 0; j < NM; ++j) {
                        const float* at = sC + s0 * L::RC + (mc * NM + j) * 8 + gq;
                        f[j].set(0, at[0] * w0), f[j].set(1, at[L::RC] * w1);
                    }
#pragma unroll
                    for (int x = 0; x < MT; ++x) mma8(u[x], a[x], f);
                }
                const float gn = sW[n];
#pragma unroll
                for (int x = 0; x < MT; ++x)
#pragma unroll
                    for (int j = 0; j < NM; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) m[x][j][e] = fmaf(m[x][j][e], gn, u[x][j].get(e));
            }
        }

        if (leaves) each([&](int, int, float& x) { bad = fmaf(x, 0.f, bad); });
        return bad;
    };
    if (__syncthreads_or(pass(std::false_type()) != 0.f)) pass(std::true_type());

    if (leaves) {
        const int64_t VK = (int64_t)ro.Db * ro.Dc;
        float* dst = kOut ? ro.mT + stream * VK : const_cast<float*>(ro.R) + (stream * nseg + slot) * VK;
        each([&](int bb, int cc, float& x) {
            if (bb < ro.Db && cc < cw) dst[(c0 + cc) * ro.m_sc + bb * ro.m_sb] = x;
        });
    }
}

template <int D, bool kOut>
cudaError_t launch_chunk(const LaDims& d, const LaRoles& roles, cudaStream_t st) {
    using L = Smem<D>;
    const size_t smem = L::SIZE * sizeof(float);
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(la_chunk_kernel<D, kOut>, (int)smem, done);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)(d.NS() * (kOut ? d.nseg : d.nseg - 1)), D / L::CS, roles.n);
    return launch_dependent(la_chunk_kernel<D, kOut>, grid, L::THREADS, smem, st, d, roles);
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
    await_previous();
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

// Four consecutive values (aligned to four elements) as floats.
__device__ __forceinline__ void ld4(const float* p, float (&f)[4]) {
    const float4 x = *reinterpret_cast<const float4*>(p);
    f[0] = x.x, f[1] = x.y, f[2] = x.z, f[3] = x.w;
}
__device__ __forceinline__ void ld4(const __nv_bfloat16* p, float (&f)[4]) {
    const uint2 x = *reinterpret_cast<const uint2*>(p);
    f[0] = __uint_as_float(x.x << 16), f[1] = __uint_as_float(x.x & 0xffff0000u);
    f[2] = __uint_as_float(x.y << 16), f[3] = __uint_as_float(x.y & 0xffff0000u);
}
__device__ __forceinline__ float ld1(const float* p) { return *p; }
__device__ __forceinline__ float ld1(const __nv_bfloat16* p) { return __bfloat162float(*p); }

// Sums over each group of L lanes of R values a lane.  While a lane has several values
// it keeps half of them at each step and hands on the others (R = 8, L = 32: 9 exchanges
// instead of 40).  Leaves the sums of rows `first` .. `first` + kept - 1 in v[0 .. kept-1],
// in the lanes where `writes`.
template <int R, int L>
struct RowSums {
    static constexpr int kept = R > L ? R / L : 1;
    int first = 0;
    bool writes = true;
    __device__ __forceinline__ RowSums(float (&v)[R], int lane) {
#pragma unroll
        for (int off = L / 2, n = R; off > 0; off >>= 1) {
            const bool up = lane & off;
            if (n > 1) {
                n >>= 1;
#pragma unroll
                for (int i = 0; i < n; ++i)
                    v[i] = (up ? v[i + n] : v[i]) + __shfl_xor_sync(0xffffffffu, up ? v[i] : v[i + n], off);
                first += up ? n : 0;
            } else {
                v[0] += __shfl_xor_sync(0xffffffffu, v[0], off);
                writes = writes && !up;
            }
        }
    }
};

// A warp holds R * 32 / L rows of one head's state in registers across the call's tokens:
// L = K / 4 lanes a row, four columns each, so that a load takes whole 128-byte lines
// for any K.  Bound by reading and writing the state once.
template <typename T, int L, int R>
__global__ void __launch_bounds__(256)
la_decode_kernel(LaDims d, const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v, int64_t sq,
                 int64_t sk, int64_t sv, float* __restrict__ state, T* __restrict__ o) {
    await_previous();
    constexpr int K = 4 * L, W = 32 / L;  // rows of one load
    const int lane = threadIdx.x & 31, groups = d.V / (R * W), c0 = lane % L * 4;
    const int64_t unit = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (unit >= d.NS() * groups) return;
    const int64_t stream = unit / groups;
    const int v0 = (int)(unit % groups) * R * W + lane / L, h = (int)(stream % d.H);  // row of load r: v0 + r W
    const int64_t b = stream / d.H;
    float* rows = state + (stream * d.V + v0) * K + c0;
    float S[R][4];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const float4 x = __ldcs((const float4*)(rows + r * W * K));
        S[r][0] = x.x, S[r][1] = x.y, S[r][2] = x.z, S[r][3] = x.w;
    }
    const float gamma = expf(d.log_decay[h]);
    for (int t = 0; t < d.T; ++t) {
        const int64_t tok = b * d.T + t;
        float kv[4], qv[4], red[R];
        ld4(k + tok * sk + (int64_t)h * K + c0, kv);
        ld4(q + tok * sq + (int64_t)h * K + c0, qv);
        const T* vp = v + tok * sv + (int64_t)h * d.V + v0;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float vr = ld1(vp + r * W);
            red[r] = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                S[r][i] = fmaf(vr, kv[i], gamma * S[r][i]);
                red[r] = fmaf(S[r][i], qv[i], red[r]);
            }
        }
        const RowSums<R, L> sum(red, lane);
        if (sum.writes) {
            T* op = o + (tok * d.H + h) * d.V + v0 + sum.first * W;
#pragma unroll
            for (int i = 0; i < sum.kept; ++i) st1(op + i * W, red[i]);
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
        __stcs((float4*)(rows + r * W * K), make_float4(S[r][0], S[r][1], S[r][2], S[r][3]));
}

template <typename T, int L, int R>
cudaError_t launch_decode_k(const LaDims& d, const void* q, const void* k, const void* v, int64_t sq, int64_t sk,
                            int64_t sv, float* state, void* o, cudaStream_t st) {
    const int64_t units = d.NS() * (d.V / (R * 32 / L));
    return launch_dependent(la_decode_kernel<T, L, R>, dim3((unsigned)((units + 7) / 8)), 256, 0, st, d, (const T*)q,
                            (const T*)k, (const T*)v, sq, sk, sv, state, (T*)o);
}

// Eight loads a lane, or as many as the head's V rows give one warp.
template <typename T>
cudaError_t launch_decode_t(const LaDims& d, const void* q, const void* k, const void* v, int64_t sq, int64_t sk,
                            int64_t sv, float* state, void* o, cudaStream_t st) {
    if (d.K == 128) return launch_decode_k<T, 32, 8>(d, q, k, v, sq, sk, sv, state, o, st);
    if (d.K == 64) return launch_decode_k<T, 16, 8>(d, q, k, v, sq, sk, sv, state, o, st);
    if (d.K == 32 && d.V >= 32) return launch_decode_k<T, 8, 8>(d, q, k, v, sq, sk, sv, state, o, st);
    if (d.K == 32) return launch_decode_k<T, 8, 4>(d, q, k, v, sq, sk, sv, state, o, st);
    if (d.V >= 64) return launch_decode_k<T, 4, 8>(d, q, k, v, sq, sk, sv, state, o, st);
    if (d.V == 32) return launch_decode_k<T, 4, 4>(d, q, k, v, sq, sk, sv, state, o, st);
    return launch_decode_k<T, 4, 2>(d, q, k, v, sq, sk, sv, state, o, st);
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

// How a call cuts its sequences, in whole tiles (128 tokens of bf16, a chunk of 64 of
// float32): the cut with the least estimated time, in units of a tile of the scan.  A CTA
// takes its tiles one after the other behind a fixed part (launch, first loads, the state
// that enters); the CTAs go in waves of as many as the GPU holds; with several segments
// the sums and the link come first.  In bf16 a tile takes 2.4 us alone, the fixed parts 11
// us (scan) and 2 us each (sums, link), a tile of the sums 1.2 us (with 0.9 B6 T1000 H12
// was cut and took 34.9 us, whole it takes 30.0); in float32 a chunk of K = V = 64 takes
// 6 us and the fixed parts about as much together.
// The backward's three scans want fewer segments than the forward's one; but cut like
// the forward's it can take over the forward's sums (`saved`).
namespace {
// in tiles, but for the counts
struct CutModel {
    double scan_fixed, sum_fixed, sum_tile, link;
    int64_t tile;    // tokens
    int64_t slots;   // CTAs that run at once
    int64_t slices;  // CTAs per (stream, segment, role)
};

CutModel cut_model(const LaDims& d, InType ty) {
    if (ty == InType::BF16) return {4.5, 1.0, 0.5, 1.0, 128, sm_count(), 1};
    const int D = d.K > d.V ? d.K : d.V;
    return {0.6, 0.4, 0.4, 0.4, kTok, (int64_t)sm_count() * (D > 64 ? 1 : 2), D > 64 ? 2 : 1};
}

double cut_cost(const CutModel& m, int64_t streams, int64_t tiles, int64_t per, int scans, int sums) {
    const int64_t nseg = (tiles + per - 1) / per;
    auto waves = [&](int64_t ctas) { return (double)((ctas * m.slices + m.slots - 1) / m.slots); };
    double t = waves(streams * scans * nseg) * (per + m.scan_fixed);
    if (nseg > 1) t += waves(streams * sums * (nseg - 1)) * (m.sum_tile * per + m.sum_fixed) + m.link;
    return t;
}

// The best number of tiles a segment, and its cost.
int64_t best_cut(const CutModel& m, int64_t streams, int64_t tiles, int scans, int sums, double* cost) {
    int64_t best = tiles;
    *cost = cut_cost(m, streams, tiles, tiles, scans, sums);
    for (int64_t n = 2; n <= tiles && streams * scans * (n - 1) < 2 * m.slots; ++n) {
        const int64_t per = (tiles + n - 1) / n;
        const double c = cut_cost(m, streams, tiles, per, scans, sums);
        if (c < *cost) best = per, *cost = c;
    }
    return best;
}
}  // namespace

void la_segments(LaDims* d, InType ty, bool bwd) {
    const CutModel m = cut_model(*d, ty);
    const int64_t tiles = (d->T + m.tile - 1) / m.tile, streams = d->NS();
    int64_t per = tiles;
    if (streams > 0 && tiles > 1) {
        // the search takes up to 30 us, so a thread keeps its last results by size
        struct Found {
            int64_t streams, tiles, per;
            int width, ty, bwd;
        };
        static thread_local Found kept[16] = {};
        const int width = d->K > d->V ? d->K : d->V;
        Found& f = kept[(streams * 31 + tiles * 7 + width / 16 + (int)ty * 2 + bwd) % 16];
        if (f.streams != streams || f.tiles != tiles || f.width != width || f.ty != (int)ty || f.bwd != bwd) {
            double cost;
            per = best_cut(m, streams, tiles, 1, 1, &cost);
            if (bwd) {
                const double shared = cut_cost(m, streams, tiles, per, 3, 1);
                const int64_t own = best_cut(m, streams, tiles, 3, 2, &cost);
                if (cost < shared) per = own;
            }
            f = {streams, tiles, per, width, (int)ty, (int)bwd};
        }
        per = f.per;
    }
    d->L = (int)(per * m.tile);
    d->nseg = tiles ? (int)((tiles + per - 1) / per) : 1;
}

}  // namespace gdn
