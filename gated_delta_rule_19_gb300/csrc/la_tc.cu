// la_tc.cu -- linear attention with a decay per head on the tensor cores, for bf16
// inputs: the scan of la.cu (its header has the formulas) in tiles of 128 tokens.
//
// Per tile, with A, B, C [128 tokens, 128] in shared memory and M [c, b] the state
// that enters:
//   scores Y = A B^T,   P = Y .* D (bf16, written over Y in tensor memory)
//   X = A M^T,  X <- diag(gamma^(rho + 1 - rev)) X,  X += P C    -> the tile's outputs
//   U = C'^T B,  M <- gamma^n M + U,   C' = C's rows times gamma^(n - 1 - rho + rev).
// M is kept in float32 in registers; the product A M^T reads it rounded to bf16.  C' is
// split into two bf16 terms (high part, and the rest), two products, so that the state
// keeps 16 bits of every decayed value (2.7e-6 rms of the sum) instead of 8.
//
// One CTA per SM: two warpgroups carry the state (each half of the tokens of C' and
// half of M's columns), one the rows of P and X (thread = token = tensor-memory lane),
// one warp issues TMA, one the MMAs.  The hand-offs are mbarriers; every wait is
// bounded.  Tensor memory: X, Y, U of 128 columns each and C' of 2 x 64.  Shared
// memory: two stages of A, B, C and M; a tile's outputs are staged over its A.
//
// K or V below 128: TMA fills the missing columns with zeros, and the products run over
// the columns that are there (N and K of each MMA follow Db and Dc).

#include <cuda_bf16.h>

#include "gdn_internal.h"
#include "tc.cuh"

namespace gdn {
namespace {

using namespace tc;

constexpr int kTile = 128;
constexpr int kTileBytes = kTile * 128 * 2;
constexpr int kThreads = 448;  // 3 warpgroups, the TMA warp, the MMA warp
constexpr int kTmaWarp = 12, kMmaWarp = 13;

// Error bits of the workspace's first int.
constexpr int kErrTma = 1, kErrMma = 2, kErrRows = 4, kErrState = 8, kErrDrain = 16;

struct LaMaps {
    CUtensorMap a[3], b[3], c[3], out[3];
};

// Tensor memory columns.
constexpr uint32_t T_X = 0, T_Y = 128, T_U = 256, T_HI = 384, T_LO = 448;

struct __align__(8) Bars {
    uint64_t full[2];   // TMA: the stage's tiles have landed
    uint64_t cv;        // C' is in tensor memory (256 arrivals)
    uint64_t u;         // U is complete
    uint64_t s;         // M is in shared memory (256 arrivals)
    uint64_t k;         // the scores are complete
    uint64_t q;         // A M^T is complete (M's shared memory may be rewritten)
    uint64_t p;         // P is in tensor memory and X rescaled (128 arrivals)
    uint64_t o;         // the outputs are complete
    uint64_t x;         // the outputs are read out of X (128 arrivals)
    uint64_t free[2];   // the stage is used up, its outputs staged (128 arrivals; the sums: 1)
    uint64_t drain;
    uint32_t tmem;
};

constexpr int S_M = 2 * 3 * kTileBytes, S_POW = S_M + kTileBytes, S_UPD = S_POW + 132 * 4,
              S_BARS = S_UPD + 4 * kTile * 4, S_SIZE = S_BARS + (int)sizeof(Bars);
static_assert(S_SIZE <= 232448, "shared memory of one CTA");

__device__ __forceinline__ float power(float g, float e) { return e > 0.f ? expf(g * e) : 1.f; }

// A wait whose outcome is the same for the whole warp.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t ph, int* err, int code, uint32_t ns) {
    return __all_sync(0xffffffffu, mbar_wait(bar, ph, err, code, ns));
}

// C' of 64 of the tile's tokens (from s0) for this thread's lane c, as two bf16 terms
// in tensor memory columns s / 2.
__device__ __forceinline__ void put_updates(const unsigned char* sC, const float* upd, uint32_t tm, int c, int s0) {
    const unsigned char* col = sC + (c >> 6) * (kTile * 128) + (c & 7) * 2;
    const uint32_t ch = (c >> 3) & 7;
#pragma unroll
    for (int b = 0; b < 64; b += 32) {
        uint32_t hi[16], lo[16];
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
            const int s = s0 + b + j;
            const float4 w4 = *(const float4*)(upd + s);
            const float w[4] = {w4.x, w4.y, w4.z, w4.w};
            float f[4], r[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint16_t v = *(const uint16_t*)(col + (s + e) * 128 + ((ch ^ ((s + e) & 7)) << 4));
                f[e] = __uint_as_float((uint32_t)v << 16) * w[e];
            }
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
                const uint32_t h = pack_bf16(f[e], f[e + 1]);
                r[e] = f[e] - __uint_as_float(h << 16);
                r[e + 1] = f[e + 1] - __uint_as_float(h & 0xffff0000u);
                hi[(j + e) / 2] = h;
                lo[(j + e) / 2] = pack_bf16(r[e], r[e + 1]);
            }
        }
        tmem_st16(tm + T_HI + (s0 + b) / 2, hi);
        tmem_st16(tm + T_LO + (s0 + b) / 2, lo);
    }
    tmem_wait_st();
}

// One CTA: role blockIdx.y, (stream, segment) blockIdx.x.  kOut: the outputs and, from
// the last segment, the state that leaves; else the segments' sums.
template <bool kOut>
__global__ void __launch_bounds__(kThreads, 1)
la_tile_kernel(LaDims d, LaRoles roles, const __grid_constant__ LaMaps maps) {
    extern __shared__ __align__(1024) unsigned char sm[];
    Bars& bar = *reinterpret_cast<Bars*>(sm + S_BARS);
    float* sPow = reinterpret_cast<float*>(sm + S_POW);
    unsigned char* sM = sm + S_M;
    const int rl = blockIdx.y;
    const LaRole& ro = roles.r[rl];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int nseg = kOut ? d.nseg : d.nseg - 1;
    const int64_t stream = blockIdx.x / nseg;
    const int slot = (int)(blockIdx.x % nseg);
    const int rev = ro.rev, seg = !kOut && rev ? slot + 1 : slot;
    const int b = (int)(stream / d.H), h = (int)(stream % d.H);
    const float g = d.log_decay[h];
    const int t_lo = seg * d.L, t_hi = min(d.T, t_lo + d.L);
    const int tiles = (t_hi - t_lo + kTile - 1) / kTile;
    const int Db = ro.Db, Dc = ro.Dc;
    auto tile_t0 = [&](int it) { return t_lo + (rev ? tiles - 1 - it : it) * kTile; };

    if (warp == kMmaWarp) {
        tmem_alloc(&bar.tmem, 512);
        tmem_relinquish();
    } else if (tid == kTmaWarp * 32) {
        mbar_init(&bar.full[0], 1);
        mbar_init(&bar.full[1], 1);
        mbar_init(&bar.cv, 256);
        mbar_init(&bar.u, 1);
        mbar_init(&bar.s, 256);
        mbar_init(&bar.k, 1);
        mbar_init(&bar.q, 1);
        mbar_init(&bar.p, 128);
        mbar_init(&bar.o, 1);
        mbar_init(&bar.x, 128);
        mbar_init(&bar.free[0], kOut ? 128 : 1);
        mbar_init(&bar.free[1], kOut ? 128 : 1);
        mbar_init(&bar.drain, 1);
        fence_mbar_init();
    }
    for (int e = tid; e <= kTile; e += kThreads) sPow[e] = power(g, (float)e);
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tm = bar.tmem;
    const uint32_t lane_base = (uint32_t)(warp & 3) << 21;  // this warp's quarter of the lanes

    if (warp == kTmaWarp) {
        if (lane == 0) {
            const int nb = Db > 64 ? 2 : 1, nc = Dc > 64 ? 2 : 1;
            const uint32_t bytes = (uint32_t)(((kOut ? 2 : 1) * nb + nc) * (kTileBytes / 2));
            auto load = [&](int it) {
                unsigned char* st = sm + (it & 1) * 3 * kTileBytes;
                uint64_t* f = &bar.full[it & 1];
                const int t0 = tile_t0(it);
                mbar_arrive_expect_tx(f, bytes);
                for (int i = 0; i < nb; ++i) {
                    if (kOut) tma_load_4d(st + i * (kTileBytes / 2), &maps.a[rl], f, 64 * i, h, t0, b);
                    tma_load_4d(st + kTileBytes + i * (kTileBytes / 2), &maps.b[rl], f, 64 * i, h, t0, b);
                }
                for (int i = 0; i < nc; ++i)
                    tma_load_4d(st + 2 * kTileBytes + i * (kTileBytes / 2), &maps.c[rl], f, 64 * i, h, t0, b);
            };
            int issued = 0, it = 0;
            for (; issued < 2 && issued < tiles; ++issued) load(issued);
            for (; it < tiles; ++it) {
                if (!mbar_wait(&bar.free[it & 1], (it >> 1) & 1, d.err, kErrTma, d.wait_ns)) break;
                if (kOut) {
                    const unsigned char* st = sm + (it & 1) * 3 * kTileBytes;
                    for (int i = 0; i < nc; ++i)
                        tma_store_4d(&maps.out[rl], st + i * (kTileBytes / 2), 64 * i, h, tile_t0(it), b);
                    bulk_commit();
                    if (issued < tiles) bulk_wait_read0();
                }
                if (issued < tiles) load(issued++);
            }
            for (int i = max(0, issued - 2); i < issued; ++i)  // no copy outlives the CTA
                mbar_wait(&bar.full[i & 1], (i >> 1) & 1, d.err, kErrDrain);
            bulk_wait0();
        }
    } else if (warp == kMmaWarp) {
        if (lane == 0) {
            const uint32_t i_k = idesc_bf16(128, 128, false, false), i_q = idesc_bf16(128, Dc, false, false),
                           i_p = idesc_bf16(128, Dc, false, true), i_u = idesc_bf16(128, Db, false, true);
            for (int it = 0; it < tiles; ++it) {
                const uint32_t ph = it & 1;
                const uint32_t sA = smem_u32(sm + (it & 1) * 3 * kTileBytes), sB = sA + kTileBytes,
                               sC = sB + kTileBytes, sMm = smem_u32(sM);
                if (!mbar_wait(&bar.full[it & 1], (it >> 1) & 1, d.err, kErrMma, d.wait_ns)) break;
                if (kOut) {
                    for (int s = 0; s < Db / 16; ++s)
                        mma_bf16_ss(tm + T_Y, desc_kmaj(sA, 128, s), desc_kmaj(sB, 128, s), i_k, s > 0);
                    mma_commit(&bar.k);
                    if (!mbar_wait(&bar.s, ph, d.err, kErrMma, d.wait_ns)) break;
                    if (it && !mbar_wait(&bar.x, ph ^ 1, d.err, kErrMma, d.wait_ns)) break;
                    fence_after_sync();
                    for (int s = 0; s < Db / 16; ++s)
                        mma_bf16_ss(tm + T_X, desc_kmaj(sA, 128, s), desc_kmaj(sMm, 128, s), i_q, s > 0);
                    mma_commit(&bar.q);
                }
                if (!mbar_wait(&bar.cv, ph, d.err, kErrMma, d.wait_ns)) break;
                fence_after_sync();
                for (int s = 0; s < kTile / 16; ++s)
                    mma_bf16_ts(tm + T_U, tm + T_HI + 8 * s, desc_mnmaj(sB, 128, s), i_u, s > 0);
                for (int s = 0; s < kTile / 16; ++s)
                    mma_bf16_ts(tm + T_U, tm + T_LO + 8 * s, desc_mnmaj(sB, 128, s), i_u, 1);
                mma_commit(&bar.u);
                if (!kOut) mma_commit(&bar.free[it & 1]);
                if (kOut) {
                    if (!mbar_wait(&bar.p, ph, d.err, kErrMma, d.wait_ns)) break;
                    fence_after_sync();
                    for (int s = 0; s < kTile / 16; ++s)
                        mma_bf16_ts(tm + T_X, tm + T_Y + 8 * s, desc_mnmaj(sC, 128, s), i_p, 1);
                    mma_commit(&bar.o);
                }
            }
            mma_commit(&bar.drain);  // no MMA outlives the CTA
            mbar_wait(&bar.drain, 0, d.err, kErrDrain);
        }
    } else if (warp >= 4) {
        // ------------------------------------------------ the state: lane c, half the columns
        const int c = tid & 127, half = (warp >> 2) - 1, b0 = half * 64;
        const uint32_t tl = tm + lane_base;
        float m[64];
#pragma unroll
        for (int i = 0; i < 64; ++i) m[i] = 0.f;
        const int64_t VK = (int64_t)Db * Dc;
        if (kOut) {
            auto add = [&](const float* src, float w) {
                if (c >= Dc) return;
                src += (int64_t)c * ro.m_sc;
#pragma unroll
                for (int i = 0; i < 64; i += 4) {
                    if (b0 + i >= Db) break;
                    float4 f;
                    if (ro.m_sb == 1) f = *(const float4*)(src + b0 + i);
                    else
                        f = make_float4(src[(b0 + i) * ro.m_sb], src[(b0 + i + 1) * ro.m_sb],
                                        src[(b0 + i + 2) * ro.m_sb], src[(b0 + i + 3) * ro.m_sb]);
                    m[i] = fmaf(w, f.x, m[i]), m[i + 1] = fmaf(w, f.y, m[i + 1]);
                    m[i + 2] = fmaf(w, f.z, m[i + 2]), m[i + 3] = fmaf(w, f.w, m[i + 3]);
                }
            };
            if (ro.m0) add(ro.m0 + stream * VK, power(g, (float)(rev ? d.T - t_hi : t_lo)));
            const float* R = ro.R + stream * (d.nseg - 1) * VK;
            if (!rev)
                for (int i = 0; i < seg; ++i) add(R + i * VK, power(g, (float)(t_lo - (i + 1) * d.L)));
            else
                for (int i = d.nseg - 1; i > seg; --i) add(R + (i - 1) * VK, power(g, (float)(i * d.L - t_hi)));
        }
        auto put_state = [&] {  // M's bf16 copy, for A M^T
#pragma unroll
            for (int i = 0; i < 64; i += 16) {
                if (b0 + i >= Db) break;
                float f[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) f[j] = m[i + j];
                tile_put16(sM, kTile, c, b0 + i, f);
            }
            fence_proxy_async();
            mbar_arrive(&bar.s);
        };
        if (kOut) put_state();
        // this warp's copy of the update weights (the warps of a warpgroup's half share
        // nothing, so that no warp waits for another outside the bounded waits)
        float* upd = reinterpret_cast<float*>(sm + S_UPD) + (warp & 3) * kTile;
        const int s0 = half * 64;
        int n_have = -1;
        bool ok = true;
        for (int it = 0; it < tiles && ok; ++it) {
            const uint32_t ph = it & 1;
            const int n = min(kTile, t_hi - tile_t0(it));
            if (n != n_have) {
                __syncwarp();
                for (int s = s0 + lane; s < s0 + 64; s += 32) upd[s] = sPow[max(rev ? min(s + 1, n) : n - 1 - s, 0)];
                __syncwarp();
                n_have = n;
            }
            if (!(ok = warp_wait(&bar.full[it & 1], (it >> 1) & 1, d.err, kErrState, d.wait_ns))) break;
            put_updates(sm + (it & 1) * 3 * kTileBytes + 2 * kTileBytes, upd, tl, c, s0);
            fence_before_sync();
            mbar_arrive(&bar.cv);
            if (!(ok = warp_wait(&bar.u, ph, d.err, kErrState, d.wait_ns))) break;
            fence_after_sync();
            const float gn = sPow[n];
#pragma unroll
            for (int i = 0; i < 64; i += 32) {
                if (b0 + i >= Db) break;
                uint32_t u[32];
                tmem_ld32(tl + T_U + b0 + i, u);
                tmem_wait_ld(u);
#pragma unroll
                for (int j = 0; j < 32; ++j) m[i + j] = fmaf(gn, m[i + j], __uint_as_float(u[j]));
            }
            fence_before_sync();
            if (kOut && it + 1 < tiles) {
                if (!(ok = warp_wait(&bar.q, ph, d.err, kErrState, d.wait_ns))) break;
                put_state();
            }
        }
        const bool last = kOut && ro.mT && seg == (rev ? 0 : d.nseg - 1);
        if (ok && c < Dc && (!kOut || last)) {
            float* dst = (kOut ? ro.mT + stream * VK : const_cast<float*>(ro.R) + (stream * nseg + slot) * VK) +
                         (int64_t)c * ro.m_sc;
#pragma unroll
            for (int i = 0; i < 64; ++i)
                if (b0 + i < Db) dst[(b0 + i) * ro.m_sb] = m[i];
        }
    } else if (kOut) {
        // ------------------------------------------------ the rows: lane = token
        const uint32_t tl = tm + lane_base;
        const int r = tid;
        float fine[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) fine[j] = sPow[rev ? j : 15 - j];
        for (int it = 0; it < tiles; ++it) {
            const uint32_t ph = it & 1;
            const int n = min(kTile, t_hi - tile_t0(it));
            if (!warp_wait(&bar.k, ph, d.err, kErrRows, d.wait_ns)) break;
            fence_after_sync();
            // P = Y .* D: 32 columns at a time, below, on or above this warp's diagonal
            // block; within a block gamma^|r - s| is a power of the row's distance to its
            // edge times one of the 16 (column) powers, both with exponents >= 0
#pragma unroll 1
            for (int cb = 0; cb < 4; ++cb) {
                uint32_t y[32], p[16];
                if (rev ? cb < warp : cb > warp) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) p[j] = 0;
                } else {
                    tmem_ld32(tl + T_Y + cb * 32, y);
                    tmem_wait_ld(y);
                    if (cb == warp) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            const int dist = rev ? j - lane : lane - j;
                            y[j] = dist >= 0 ? __float_as_uint(__uint_as_float(y[j]) * sPow[max(dist, 0)]) : 0u;
                        }
                    } else {
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf) {
                            const int s = cb * 32 + hf * 16;
                            const float far = sPow[rev ? s - r : r - s - 15];
#pragma unroll
                            for (int j = 0; j < 16; ++j)
                                y[hf * 16 + j] =
                                    __float_as_uint(__uint_as_float(y[hf * 16 + j]) * (far * fine[j]));
                        }
                    }
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        p[j] = pack_bf16(__uint_as_float(y[2 * j]), __uint_as_float(y[2 * j + 1]));
                }
                tmem_st16(tl + T_Y + cb * 16, p);  // over scores already read
            }
            if (!warp_wait(&bar.q, ph, d.err, kErrRows, d.wait_ns)) break;
            fence_after_sync();
            const float w = sPow[max(rev ? n - 1 - r : r + 1, 0)];
#pragma unroll 1
            for (int cb = 0; cb < Dc; cb += 32) {
                uint32_t x[32];
                tmem_ld32(tl + T_X + cb, x);
                tmem_wait_ld(x);
#pragma unroll
                for (int j = 0; j < 32; ++j) x[j] = __float_as_uint(__uint_as_float(x[j]) * w);
                tmem_st32(tl + T_X + cb, x);
            }
            tmem_wait_st();
            fence_before_sync();
            mbar_arrive(&bar.p);
            if (!warp_wait(&bar.o, ph, d.err, kErrRows, d.wait_ns)) break;
            fence_after_sync();
            unsigned char* so = sm + (it & 1) * 3 * kTileBytes;
#pragma unroll 1
            for (int cb = 0; cb < Dc; cb += 32) {
                uint32_t x[32];
                tmem_ld32(tl + T_X + cb, x);
                tmem_wait_ld(x);
#pragma unroll
                for (int i = 0; i < 32; i += 16) {
                    float f[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) f[j] = __uint_as_float(x[i + j]);
                    tile_put16(so, kTile, r, cb + i, f);
                }
            }
            fence_proxy_async();
            fence_before_sync();
            mbar_arrive(&bar.x);
            mbar_arrive(&bar.free[it & 1]);
        }
    }
    __syncwarp();
    fence_before_sync();
    __syncthreads();
    if (warp == kMmaWarp) tmem_dealloc(tm, 512);
}

bool make_maps(const LaDims& d, const LaRoles& roles, bool out, LaMaps* m) {
    for (int i = 0; i < roles.n; ++i) {
        const LaRole& r = roles.r[i];
        if (!tmap_rows_bthd(&m->b[i], r.b, d.B, d.T, d.H, r.Db, r.sb) ||
            !tmap_rows_bthd(&m->c[i], r.c, d.B, d.T, d.H, r.Dc, r.sc))
            return false;
        if (out && (!tmap_rows_bthd(&m->a[i], r.a, d.B, d.T, d.H, r.Db, r.sa) ||
                    !tmap_rows_bthd(&m->out[i], r.out, d.B, d.T, d.H, r.Dc, (int64_t)d.H * r.Dc)))
            return false;
    }
    return true;
}

template <bool kOut>
cudaError_t launch(const LaDims& d, const LaRoles& roles, cudaStream_t st) {
    LaMaps maps;
    if (!make_maps(d, roles, kOut, &maps)) return cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(la_tile_kernel<kOut>, cudaFuncAttributeMaxDynamicSharedMemorySize, S_SIZE);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)(d.NS() * (kOut ? d.nseg : d.nseg - 1)), roles.n);
    la_tile_kernel<kOut><<<grid, kThreads, S_SIZE, st>>>(d, roles, maps);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_la_states_tc(const LaDims& d, const LaRoles& roles, cudaStream_t st) {
    return launch<false>(d, roles, st);
}
cudaError_t launch_la_scan_tc(const LaDims& d, const LaRoles& roles, cudaStream_t st) {
    return launch<true>(d, roles, st);
}

}  // namespace gdn
