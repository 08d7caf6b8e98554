// la_tc.cu -- linear attention with a decay per head on the tensor cores, for bf16
// inputs: the scan of la.cu (its header has the formulas) in tiles of 128 tokens.
//
// Per tile, with A, B, C [128 tokens, 128] in shared memory and M [c, b] the state
// that enters:
//   scores Y = A B^T,   P = Y .* D (bf16, in tensor memory)
//   X = A M^T,  X <- diag(gamma^(rho + 1 - rev)) X,  X += P C    -> the tile's outputs
//   U = C'^T B,  M <- gamma^n M + U,   C' = C's rows times gamma^(n - 1 - rho + rev).
// M is kept in float32 in registers; the products A M^T and P C read M and P rounded to
// bf16, an error of the size of the outputs' own rounding (2.35e-3 relative L2 in all, the
// outputs' rounding alone 1.66e-3): a second term of each would double two of the four
// products, and tensor memory and shared memory have no room for it.  C' is
// split into bf16 terms (the high part, then what is left), one product each: two where
// M only feeds outputs (16 bits of every decayed value, 2.5e-6 rms of the sum; one would
// add as much error to the outputs as M's own rounding), three in the sums and where M is
// returned (24 bits: the state is then as exact as float32 sums are).
//
// One CTA per SM.  la_scan_kernel: two warpgroups carry the state (thread = row of M,
// half of the columns each), two the rows of P and X (thread = token = tensor-memory
// lane, half of the columns each), and each makes C' of 32 tokens; one warp issues TMA,
// one the MMAs.  la_sums_kernel, the segments' sums, is the U part alone.  The hand-offs
// are mbarriers; every wait is bounded.
//
// What bounds a tile is its chain of hand-offs (scores, P, outputs; C', U, M), through a
// shared memory that is busy most of it: of the 6400 cycles that a tile of the backward takes
// (B8 T4096 H6 K = V = 128), operands of MMAs read it for 1880 and the warps use it for 1660,
// and the copies in and out need another 1000; tensor pipe 47%, issue 41%, DRAM 52%, L2 30% of
// their rates.  An operand is read at 128 bytes a cycle, so P and C' are operands in tensor
// memory, and most decay factors are multiplied up in registers rather than read from
// tables.  Outputs stored from registers (32 bytes of a row per lane) kept the load-store
// unit busy and cost more than staging them does.
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
constexpr int kThreads = 576;  // 4 warpgroups, the TMA warp, the MMA warp
constexpr int kTmaWarp = 16, kMmaWarp = 17;

// Up to this many tiles a segment the scan moves its states in whole lines (see
// la_scan_kernel).
constexpr int kLinesMax = 8;

// Error bits of the workspace's first int.
constexpr int kErrTma = 1, kErrMma = 2, kErrRows = 4, kErrState = 8, kErrDrain = 16;

struct LaMaps {
    CUtensorMap a[3], b[3], c[3], out[3];
};

// One CTA's part of the work: a role, a (stream, segment), and its tiles in the order
// of the scan.
struct Part {
    const LaRole& ro;
    int rl, nseg, slot, seg, rev, b, h, t_lo, t_hi, tiles;
    int64_t stream;
    float g;
    __device__ Part(const LaDims& d, const LaRoles& roles, bool sums)
        : ro(roles.r[blockIdx.y]), rl(blockIdx.y), nseg(sums ? d.nseg - 1 : d.nseg) {
        stream = blockIdx.x / nseg;
        slot = (int)(blockIdx.x % nseg);
        rev = ro.rev;
        seg = sums && rev ? slot + 1 : slot;  // the last segment's own sum feeds nobody
        b = (int)(stream / d.H);
        h = (int)(stream % d.H);
        g = d.log_decay[h];
        t_lo = seg * d.L;
        t_hi = min(d.T, t_lo + d.L);
        tiles = (t_hi - t_lo + kTile - 1) / kTile;
    }
    __device__ int t0(int it) const { return t_lo + (rev ? tiles - 1 - it : it) * kTile; }
    __device__ int len(int it) const { return min(kTile, t_hi - t0(it)); }
    __device__ int tail() const { return t_hi - t_lo - (tiles - 1) * kTile; }
};

__device__ __forceinline__ float power(float g, float e) { return e > 0.f ? expf(g * e) : 1.f; }

// mbar_wait for a whole warp, one outcome for all its lanes.  The clock is read once in
// 16 tries.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t ph, int* err, int code, uint32_t ns) {
    bool ok = mbar_try_wait(bar, ph);
    if (!__all_sync(0xffffffffu, ok)) {
        const uint64_t limit = ns ? ns : kWaitLimitNs, t0 = globaltimer();
        do {
            for (int i = 0; i < 16 && !ok; ++i) ok = mbar_try_wait(bar, ph);
        } while (!ok && globaltimer() - t0 <= limit);
        if (!ok) atomicOr(err, code);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) return false;
    }
    return true;
}

// A pair of bf16 values times a pair of weights, rounded to bf16; `left` is what that
// leaves of the products.
__device__ __forceinline__ uint32_t split_off(uint64_t f, uint64_t& left) {
    float x, y;
    unpair(f, x, y);
    const uint32_t h = pack_bf16(x, y);
    left = fma2(bf16_pair(h), twice(-1.f), f);
    return h;
}

// C' of NT of the tile's tokens (from s0) for the 32 columns of C that are this warp's
// lanes (from c0), as `terms` (2 or 3) bf16 terms in tensor memory, 64 columns apart from
// t_c on, token s in column s / 2.  Blocks of 8 tokens x 8 columns are read transposed,
// which is the register layout of the 16x128b store.
template <int NT>
__device__ __forceinline__ void put_updates(uint32_t sC, const float* upd, uint32_t t_c, int c0, int s0, int lane,
                                            int terms) {
    // this lane's row in the four blocks of an ldmatrix: tokens (0-7, 0-7, 8-15, 8-15)
    // of columns (0-7, 8-15, 0-7, 8-15)
    const int row = (lane & 7) + ((lane >> 4) << 3), cb = (lane >> 3) & 1;
    const uint32_t blk = sC + (uint32_t)(c0 >> 6) * (kTile * 128) + (uint32_t)(s0 + row) * 128;
    const uint32_t ch = (uint32_t)((c0 & 63) >> 3) + cb;
    const uint32_t from[2] = {blk + ((ch ^ (lane & 7)) << 4), blk + (((ch + 2) ^ (lane & 7)) << 4)};
    upd += s0 + 2 * (lane & 3);
#pragma unroll
    for (int b = 0; b < NT; b += 16) {
        const uint64_t w0 = *(const uint64_t*)(upd + b), w1 = *(const uint64_t*)(upd + b + 8);
#pragma unroll
        for (int i = 0; i < 2; ++i) {  // 16 lanes at a time
            uint32_t v[4], h[4];
            uint64_t f[4];
            ldmatrix_x4_trans(from[i] + b * 128, v);
            uint32_t to = t_c + ((uint32_t)(16 * i) << 16) + (s0 + b) / 2;
#pragma unroll
            for (int j = 0; j < 4; ++j) h[j] = split_off(mul2(bf16_pair(v[j]), j < 2 ? w0 : w1), f[j]);
            tmem_st_16x128b_x2(to, h);
#pragma unroll
            for (int j = 0; j < 4; ++j) h[j] = split_off(f[j], f[j]);
            tmem_st_16x128b_x2(to + 64, h);
            if (terms == 3) {
#pragma unroll
                for (int j = 0; j < 4; ++j) h[j] = split_off(f[j], f[j]);
                tmem_st_16x128b_x2(to + 128, h);
            }
        }
    }
    tmem_wait_st();
}

// The weights of C' for a whole tile, then for the sequence's last, shorter one.
__device__ __forceinline__ void fill_weights(const Part& w, float* upd) {
    for (int i = threadIdx.x; i < 2 * kTile; i += kThreads) {
        const int s = i & (kTile - 1), n = i < kTile ? kTile : w.tail();
        upd[i] = power(w.g, (float)max(w.rev ? s + 1 : n - 1 - s, 0));
    }
}

// gamma^n M + U for NC columns of this thread's lane.
template <int NC>
__device__ __forceinline__ void add_update(float (&m)[NC], uint32_t t_u, float gn, int cols) {
#pragma unroll
    for (int i = 0; i < NC; i += 16) {
        if (i < cols) {
            uint32_t u[16];
            tmem_ld16(t_u + i, u);
            tmem_wait_ld(u);
#pragma unroll
            for (int j = 0; j < 16; j += 2)
                unpair(fma2(pair(gn, gn), pair(m[i + j], m[i + j + 1]),
                            pair(__uint_as_float(u[j]), __uint_as_float(u[j + 1]))),
                       m[i + j], m[i + j + 1]);
        }
    }
}

// The first `cols` of NC elements of M's row to the caller's matrix: 16 bytes at a time
// where the row lies there as a row (single stores took 8 us for a state), else one by
// one, with the lanes' elements side by side.
template <int NC>
__device__ __forceinline__ void store_state(const float (&m)[NC], float* dst, int step, int cols) {
#pragma unroll
    for (int i = 0; i < NC; i += 4)
        if (i < cols) {
            if (step == 1) {
                *(float4*)(dst + i) = make_float4(m[i], m[i + 1], m[i + 2], m[i + 3]);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) dst[(i + e) * step] = m[i + e];
            }
        }
}

// A warp's 32 rows of a state (lane = row, NC columns each) from and to a matrix with
// rows `ld` apart, of which `rows` rows and `cols` columns are there.  Whole 128-byte lines
// go through 4 KB of the warp's own shared memory `sx`, its 16-byte pieces swizzled by
// the row; lanes that read their own rows took 3.6 us for a state, each way.
template <int NC>
__device__ __forceinline__ void load_rows(float (&m)[NC], const float* src, int ld, int rows, int cols, float* sx,
                                          int lane) {
#pragma unroll
    for (int p = 0; p < NC / 32; ++p) {
        float4 t[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = 4 * i + (lane >> 3), x = 32 * p + (lane & 7) * 4;
            t[i] = r < rows && x < cols ? *(const float4*)(src + (int64_t)r * ld + x) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = 4 * i + (lane >> 3);
            *(float4*)(sx + r * 32 + ((lane ^ r) & 7) * 4) = t[i];
        }
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float4 f = *(const float4*)(sx + lane * 32 + ((j ^ lane) & 7) * 4);
            float* to = m + 32 * p + 4 * j;
            to[0] = f.x, to[1] = f.y, to[2] = f.z, to[3] = f.w;
        }
    }
}
template <int NC>
__device__ __forceinline__ void store_rows(const float (&m)[NC], float* dst, int ld, int rows, int cols, float* sx,
                                           int lane) {
#pragma unroll
    for (int p = 0; p < NC / 32; ++p) {
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float* from = m + 32 * p + 4 * j;
            *(float4*)(sx + lane * 32 + ((j ^ lane) & 7) * 4) = make_float4(from[0], from[1], from[2], from[3]);
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = 4 * i + (lane >> 3), x = 32 * p + (lane & 7) * 4;
            if (r < rows && x < cols)
                *(float4*)(dst + (int64_t)r * ld + x) = *(const float4*)(sx + r * 32 + ((lane ^ r) & 7) * 4);
        }
    }
}

// ------------------------------------------------------------------- the sums

struct __align__(8) SumBars {
    uint64_t full[3], free[3];
    uint64_t cv[2];  // C' is in tensor memory (512 arrivals)
    uint64_t u;      // U is complete
    uint64_t a;      // U is read (512 arrivals)
    uint64_t drain;
    uint32_t tmem;
};
constexpr int SS_STAGES = 3, SS_UPD = SS_STAGES * 2 * kTileBytes, SS_POW = SS_UPD + 2 * kTile * 4,
              SS_BARS = SS_POW + 132 * 4, SS_SIZE = SS_BARS + (int)sizeof(SumBars);

// One CTA: one (stream, segment) of one role; its sum to R.  Four warpgroups make C' of
// 32 tokens each and hold 32 columns of M each; C' is double-buffered in tensor memory,
// so that a tile's is made while the one before it is multiplied.
__global__ void __launch_bounds__(kThreads, 1)
la_sums_kernel(LaDims d, LaRoles roles, const __grid_constant__ LaMaps maps) {
    await_previous();
    extern __shared__ __align__(1024) unsigned char sm[];
    SumBars& bar = *reinterpret_cast<SumBars*>(sm + SS_BARS);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const Part w(d, roles, true);
    const LaRole& ro = w.ro;
    const int Db = ro.Db, Dc = ro.Dc, tiles = w.tiles;
    float *upd = (float*)(sm + SS_UPD), *pw = (float*)(sm + SS_POW);
    const int nb = Db > 64 ? 2 : 1, nc = Dc > 64 ? 2 : 1;
    auto load = [&](int it) {
        unsigned char* st = sm + (it % SS_STAGES) * 2 * kTileBytes;
        uint64_t* f = &bar.full[it % SS_STAGES];
        mbar_arrive_expect_tx(f, (uint32_t)((nb + nc) * (kTileBytes / 2)));
        for (int i = 0; i < nb; ++i)
            tma_load_4d(st + i * (kTileBytes / 2), &maps.b[w.rl], f, 64 * i, w.h, w.t0(it), w.b);
        for (int i = 0; i < nc; ++i)
            tma_load_4d(st + kTileBytes + i * (kTileBytes / 2), &maps.c[w.rl], f, 64 * i, w.h, w.t0(it), w.b);
    };
    if (warp == kMmaWarp) {
        tmem_alloc(&bar.tmem, 512);
        tmem_relinquish();
    } else if (tid == kTmaWarp * 32) {
        for (int i = 0; i < SS_STAGES; ++i) mbar_init(&bar.full[i], 1), mbar_init(&bar.free[i], 1);
        mbar_init(&bar.cv[0], 512);
        mbar_init(&bar.cv[1], 512);
        mbar_init(&bar.u, 1);
        mbar_init(&bar.a, 512);
        mbar_init(&bar.drain, 1);
        fence_mbar_init();
        fence_proxy_async();
        for (int i = 0; i < SS_STAGES && i < tiles; ++i) load(i);
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    for (int e = tid; e <= kTile; e += kThreads) pw[e] = power(w.g, (float)e);
    fill_weights(w, upd);
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tm = bar.tmem;
    constexpr uint32_t t_u = 384;
    auto t_c = [&](int it) { return (uint32_t)(it & 1) * 192; };  // three terms of 64 columns

    if (warp == kTmaWarp) {
        if (lane == 0) {
            int issued = min(SS_STAGES, tiles);
            for (; issued < tiles; ++issued) {
                if (!mbar_wait(&bar.free[issued % SS_STAGES], (issued / SS_STAGES - 1) & 1, d.err, kErrTma, d.wait_ns))
                    break;
                load(issued);
            }
            for (int i = max(0, issued - SS_STAGES); i < issued; ++i)  // no copy outlives the CTA
                mbar_wait(&bar.full[i % SS_STAGES], (i / SS_STAGES) & 1, d.err, kErrDrain);
        }
    } else if (warp == kMmaWarp) {
        const uint32_t i_u = idesc_bf16(128, Db, false, true);
        for (int it = 0; it < tiles; ++it) {
            const uint64_t dB = desc_mnmaj(smem_u32(sm) + (uint32_t)(it % SS_STAGES) * 2 * kTileBytes, 128, 0);
            if (!warp_wait(&bar.cv[it & 1], (it >> 1) & 1, d.err, kErrMma, d.wait_ns)) break;
            if (it && !warp_wait(&bar.a, (it & 1) ^ 1, d.err, kErrMma, d.wait_ns)) break;
            fence_after_sync();
            const uint32_t c = tm + t_c(it);
            if (elect_one()) {
#pragma unroll
                for (int s = 0; s < 24; ++s)
                    mma_bf16_ts(tm + t_u, c + 8 * s, desc_add(dB, (s & 7) * 2048), i_u, s > 0);
                mma_commit(&bar.u);
                mma_commit(&bar.free[it % SS_STAGES]);
            }
            __syncwarp();
        }
        if (elect_one()) mma_commit(&bar.drain);  // no MMA outlives the CTA
        warp_wait(&bar.drain, 0, d.err, kErrDrain, 0);
    } else {
        const int part = warp >> 2, cols = Db - part * 32;
        const uint32_t tl = tm + ((uint32_t)(warp & 3) << 21);
        const bool live = (warp & 3) * 32 < Dc;  // this warp's lanes have columns of C
        float m[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) m[i] = 0.f;
        auto make = [&](int it) {
            if (!warp_wait(&bar.full[it % SS_STAGES], (it / SS_STAGES) & 1, d.err, kErrState, d.wait_ns)) return false;
            if (live)
                put_updates<32>(smem_u32(sm) + (uint32_t)(it % SS_STAGES) * 2 * kTileBytes + kTileBytes,
                            upd + (w.len(it) < kTile ? kTile : 0), tl + t_c(it), (warp & 3) * 32, part * 32, lane, 3);
            fence_before_sync();
            mbar_arrive(&bar.cv[it & 1]);
            return true;
        };
        bool ok = make(0);
        for (int it = 0; it < tiles && ok; ++it) {
            if (it + 1 < tiles && !(ok = make(it + 1))) break;
            if (!(ok = warp_wait(&bar.u, it & 1, d.err, kErrState, d.wait_ns))) break;
            fence_after_sync();
            add_update(m, tl + t_u + part * 32, pw[w.len(it)], live ? cols : 0);
            fence_before_sync();
            mbar_arrive(&bar.a);
        }
        // every product is done with the stages: they serve the rows' way out
        if (ok && live)
            store_rows(m,
                       const_cast<float*>(ro.R) + (w.stream * w.nseg + w.slot) * (int64_t)Db * Dc +
                           (int64_t)(warp & 3) * 32 * Db + part * 32,
                       Db, Dc - (warp & 3) * 32, cols, (float*)(sm + warp * 4096), lane);
    }
    __syncwarp();
    fence_before_sync();
    __syncthreads();
    if (warp == kMmaWarp) tmem_dealloc(tm, 512);
}

// ------------------------------------------------------------------- the scan

// Tensor memory columns: X; the scores, and after they are read U; P; C' (three terms).
constexpr uint32_t T_X = 0, T_Y = 128, T_U = 128, T_P = 256, T_C = 320;

struct __align__(8) Bars {
    uint64_t full[2];   // TMA: the stage's tiles have landed
    uint64_t staged[2]; // the outputs lie over the stage's A (256 arrivals)
    uint64_t cv;        // C' is in tensor memory (512 arrivals)
    uint64_t u;         // U is complete
    uint64_t s;         // M is in shared memory (256 arrivals)
    uint64_t k;         // the scores are complete
    uint64_t q;         // A M^T is complete (M's shared memory may be rewritten)
    uint64_t r;         // the scores are read (256 arrivals)
    uint64_t a;         // U is read (256 arrivals)
    uint64_t p;         // P is in tensor memory and X rescaled (256 arrivals)
    uint64_t o;         // the outputs are complete
    uint64_t x;         // the outputs are read out of X (256 arrivals)
    uint64_t drain;
    uint32_t tmem;
};

// Behind the stages and M: gamma^0 .. gamma^128; a diagonal block's powers by 31 + row -
// column (0 above it); the weights of C'.
constexpr int S_M = 2 * 3 * kTileBytes, S_POW = S_M + kTileBytes, S_DIAG = S_POW + 132 * 4, S_UPD = S_DIAG + 64 * 4,
              S_BARS = S_UPD + 2 * kTile * 4, S_SIZE = S_BARS + (int)sizeof(Bars);
static_assert(S_SIZE <= 232448 && SS_SIZE <= 232448, "shared memory of one CTA");

// P of a 32-column block off the diagonal: gamma^(distance) of the column nearest the
// row is `near`; each pair of columns further on has gamma^2 of the last one's.  Every
// exponent is >= 0.
template <bool kRev>
__device__ __forceinline__ void scale_block(const uint32_t (&y)[32], float near, float g1, uint32_t (&p)[16]) {
    const uint64_t g2 = pair(g1 * g1, g1 * g1);
    uint64_t w = kRev ? pair(near, near * g1) : pair(near * g1, near);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int j = kRev ? i : 15 - i;
        float e, f;
        unpair(mul2(pair(__uint_as_float(y[2 * j]), __uint_as_float(y[2 * j + 1])), w), e, f);
        p[j] = pack_bf16(e, f);
        w = mul2(w, g2);
    }
}

// The state's warps: lane c of M, half of the columns.  M's bf16 copy of a warp's rows
// and columns is 4 KB in one piece, which its whole lines go through before and after.
template <bool kLines, typename Make>
__device__ __forceinline__ void state_warps(const LaDims& d, const Part& w, Bars& bar, unsigned char* sm, uint32_t tl,
                                            Make&& make) {
    const LaRole& ro = w.ro;
    const float* sPow = (const float*)(sm + S_POW);
    const int c = threadIdx.x & 127, half = (threadIdx.x >> 7) - 2, b0 = half * 64;
    const int cols = (c & ~31) < ro.Dc ? ro.Db - b0 : 0;  // none where the warp has no row of M
    const int lane = threadIdx.x & 31;
    float* near = (float*)(sm + S_M) + ((threadIdx.x >> 5) - 8) * 1024;
    float m[64];
#pragma unroll
    for (int i = 0; i < 64; ++i) m[i] = 0.f;
    const int64_t VK = (int64_t)ro.Db * ro.Dc;
    bool ok = make(0);
    await_previous();  // the linked states
    const bool first = w.seg == (w.rev ? d.nseg - 1 : 0);
    const float* src = first ? (ro.m0 ? ro.m0 + w.stream * VK : nullptr)
                             : ro.R + (w.stream * (d.nseg - 1) + (w.rev ? w.seg : w.seg - 1)) * VK;
    if (kLines && src && ro.m_sb == 1) {
        load_rows(m, src + (int64_t)(c - lane) * ro.m_sc + b0, ro.m_sc, ro.Dc - (c - lane), cols, near, lane);
    } else if (src && c < ro.Dc) {
        src += (int64_t)c * ro.m_sc + b0 * ro.m_sb;
#pragma unroll
        for (int i = 0; i < 64; i += 4) {
            if (i < cols) {
                if (ro.m_sb == 1) {
                    const float4 v = *(const float4*)(src + i);
                    m[i] = v.x, m[i + 1] = v.y, m[i + 2] = v.z, m[i + 3] = v.w;
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) m[i + e] = src[(i + e) * ro.m_sb];
                }
            }
        }
    }
    auto put_state = [&] {  // M's bf16 copy, for A M^T
#pragma unroll
        for (int i = 0; i < 64; i += 16) {
            if (i < cols) {
                float f[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) f[j] = m[i + j];
                tile_put16(sm + S_M, kTile, c, b0 + i, f);
            }
        }
        fence_proxy_async();
        mbar_arrive(&bar.s);
    };
    put_state();
    for (int it = 0; it < w.tiles && ok; ++it) {
        const uint32_t ph = it & 1;
        if (!(ok = warp_wait(&bar.u, ph, d.err, kErrState, d.wait_ns))) break;
        fence_after_sync();
        add_update(m, tl + T_U + b0, sPow[w.len(it)], cols);
        fence_before_sync();
        mbar_arrive(&bar.a);
        if (it + 1 < w.tiles) {
            if (!(ok = warp_wait(&bar.q, ph, d.err, kErrState, d.wait_ns))) break;
            put_state();
            ok = make(it + 1);
        }
    }
    if (!ok || !ro.mT || w.seg != (w.rev ? 0 : d.nseg - 1)) return;
    float* dst = ro.mT + w.stream * VK;
    if (kLines && ro.m_sb == 1)
        store_rows(m, dst + (int64_t)(c - lane) * ro.m_sc + b0, ro.m_sc, ro.Dc - (c - lane), cols, near, lane);
    else if (c < ro.Dc)
        store_state(m, dst + (int64_t)c * ro.m_sc + b0 * ro.m_sb, ro.m_sb, cols);
}

// The rows' warps: lane = token, half of the columns.
template <typename Make>
__device__ __forceinline__ void row_warps(const LaDims& d, const Part& w, Bars& bar, unsigned char* sm, uint32_t tl,
                                          Make&& make) {
    const LaRole& ro = w.ro;
    const float *sPow = (const float*)(sm + S_POW), *sDiag = (const float*)(sm + S_DIAG);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, rev = w.rev;
    const int r = threadIdx.x & 127, q = warp & 3, wg = warp >> 2;  // q: the 32-token block of this warp's rows
    const int cw = ro.Dc > 16 ? ro.Dc / 2 : 16, x0 = wg * cw, xn = min(cw, ro.Dc - x0);  // columns of X
    const float g1 = sPow[1];
    if (!make(0)) return;
    for (int it = 0; it < w.tiles; ++it) {
        const uint32_t ph = it & 1;
        const int n = w.len(it);
        if (!warp_wait(&bar.k, ph, d.err, kErrRows, d.wait_ns)) return;
        fence_after_sync();
        // P = Y .* D: blocks of 32 columns below, on or above this warp's diagonal block.
        // One warpgroup has blocks 0 and 3, the other 1 and 2, so that the causal half is
        // shared evenly.
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            uint32_t y[32];
            tmem_ld32(tl + T_Y + (k ? 3 - wg : wg) * 32, y);
            tmem_wait_ld(y);
            if (k) {
                fence_before_sync();
                mbar_arrive(&bar.r);
            }
            const int cb = k ? 3 - wg : wg;
            uint32_t p[16];
            if (cb == q) {
                const float* f = sDiag + 31 + lane;
#pragma unroll
                for (int j = 0; j < 32; j += 2) {
                    float e0, e1;
                    unpair(mul2(pair(__uint_as_float(y[j]), __uint_as_float(y[j + 1])), pair(f[-j], f[-j - 1])), e0, e1);
                    p[j / 2] = pack_bf16(e0, e1);
                }
            } else if (rev ? cb < q : cb > q) {
#pragma unroll
                for (int j = 0; j < 16; ++j) p[j] = 0;
            } else if (rev) {
                scale_block<true>(y, sPow[cb * 32 - r], g1, p);
            } else {
                scale_block<false>(y, sPow[r - cb * 32 - 31], g1, p);
            }
            tmem_st16(tl + T_P + cb * 16, p);  // the P before it is used up: its outputs have been read
        }
        if (!warp_wait(&bar.q, ph, d.err, kErrRows, d.wait_ns)) return;
        fence_after_sync();
        const float f = sPow[max(rev ? n - 1 - r : r + 1, 0)];
        uint32_t x[4][16];  // this warpgroup's columns of X
        auto read_x = [&] {
#pragma unroll
            for (int k = 0; k < 4; ++k) tmem_ld16(tl + T_X + x0 + 16 * k, x[k]);
#pragma unroll
            for (int k = 0; k < 4; ++k) tmem_wait_ld(x[k]);
        };
        read_x();
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (16 * k < xn) {
#pragma unroll
                for (int j = 0; j < 16; ++j) x[k][j] = __float_as_uint(__uint_as_float(x[k][j]) * f);
                tmem_st16(tl + T_X + x0 + 16 * k, x[k]);
            }
        tmem_wait_st();
        fence_before_sync();
        mbar_arrive(&bar.p);
        if (!warp_wait(&bar.o, ph, d.err, kErrRows, d.wait_ns)) return;
        fence_after_sync();
        read_x();
        fence_before_sync();
        mbar_arrive(&bar.x);
        unsigned char* out = sm + (it & 1) * 3 * kTileBytes;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (16 * k < xn) {
                float v[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) v[j] = __uint_as_float(x[k][j]);
                tile_put16(out, kTile, r, x0 + 16 * k, v);
            }
        fence_proxy_async();
        mbar_arrive(&bar.staged[it & 1]);
        // the next tile's C', once U no longer reads this one's: after the outputs, which
        // must not wait for the next tile's load
        if (it + 1 < w.tiles) {
            if (!warp_wait(&bar.u, ph, d.err, kErrRows, d.wait_ns)) return;
            fence_after_sync();
            if (!make(it + 1)) return;
        }
    }
}

// One CTA: one (stream, segment) of one role: its outputs and, from the last segment,
// the state that leaves.  kLines: states that lie there as M does move in whole lines,
// which saves 4.5 us a call (forward at K = V = 128: T128 H16 14.3 -> 9.9 us, B64 T1024
// H2, 8 tiles a segment, 41.6 -> 37.1), but the compiler's loop over many tiles is then up
// to 16% slower (32 tiles a segment: B32 T4096 H6 K = V = 64 forward 156 -> 177 us, B8
// T4096 H6 K = V = 128 backward 104 -> 121), so it is for segments of few tiles.
template <bool kLines>
__global__ void __launch_bounds__(kThreads, 1)
la_scan_kernel(LaDims d, LaRoles roles, const __grid_constant__ LaMaps maps) {
    if (d.nseg == 1) await_previous();  // else the sums did; the linked states are waited for below
    extern __shared__ __align__(1024) unsigned char sm[];
    Bars& bar = *reinterpret_cast<Bars*>(sm + S_BARS);
    float *sPow = reinterpret_cast<float*>(sm + S_POW), *sDiag = (float*)(sm + S_DIAG), *sUpd = (float*)(sm + S_UPD);
    unsigned char* sM = sm + S_M;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const Part w(d, roles, false);
    const LaRole& ro = w.ro;
    const int Db = ro.Db, Dc = ro.Dc, tiles = w.tiles, rev = w.rev;
    const bool last = w.seg == (rev ? 0 : d.nseg - 1);
    const int terms = last && ro.mT ? 3 : 2;
    const int nb = Db > 64 ? 2 : 1, nc = Dc > 64 ? 2 : 1;
    auto stage = [&](int it) { return sm + (it & 1) * 3 * kTileBytes; };
    auto load = [&](int it) {
        uint64_t* full = &bar.full[it & 1];
        mbar_arrive_expect_tx(full, (uint32_t)((2 * nb + nc) * (kTileBytes / 2)));
        auto put = [&](const CUtensorMap* map, int blocks, unsigned char* to) {
            for (int i = 0; i < blocks; ++i)
                tma_load_4d(to + i * (kTileBytes / 2), map, full, 64 * i, w.h, w.t0(it), w.b);
        };
        put(&maps.b[w.rl], nb, stage(it) + kTileBytes);
        put(&maps.c[w.rl], nc, stage(it) + 2 * kTileBytes);
        put(&maps.a[w.rl], nb, stage(it));
    };

    if (warp == kMmaWarp) {
        tmem_alloc(&bar.tmem, 512);
        tmem_relinquish();
    } else if (tid == kTmaWarp * 32) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar.full[i], 1);
            mbar_init(&bar.staged[i], 256);
        }
        mbar_init(&bar.cv, 512);
        mbar_init(&bar.u, 1);
        mbar_init(&bar.s, 256);
        mbar_init(&bar.k, 1);
        mbar_init(&bar.q, 1);
        mbar_init(&bar.r, 256);
        mbar_init(&bar.a, 256);
        mbar_init(&bar.p, 256);
        mbar_init(&bar.o, 1);
        mbar_init(&bar.x, 256);
        mbar_init(&bar.drain, 1);
        fence_mbar_init();
        fence_proxy_async();
        for (int i = 0; i < 2 && i < tiles; ++i) load(i);
    }
    for (int e = tid; e <= kTile; e += kThreads) sPow[e] = power(w.g, (float)e);
    for (int i = tid; i < 63; i += kThreads) {
        const int dist = rev ? 31 - i : i - 31;
        sDiag[i] = dist >= 0 ? power(w.g, (float)dist) : 0.f;
    }
    fill_weights(w, sUpd);
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tm = bar.tmem;
    const uint32_t tl = tm + ((uint32_t)(warp & 3) << 21);  // this warp's quarter of the lanes

    if (warp == kTmaWarp) {
        if (lane == 0) {
            // The next load waits for the outputs and their store's reads: sooner, it took
            // shared memory from the tile under work (B, C after the products, A after the
            // store: backward of B8 T4096 H6 108 instead of 104 us; A after A M^T, 117).
            int issued = min(2, tiles);
            for (int it = 0; it < tiles; ++it) {
                if (!mbar_wait(&bar.staged[it & 1], (it >> 1) & 1, d.err, kErrTma, d.wait_ns)) break;
                for (int i = 0; i < nc; ++i)
                    tma_store_4d(&maps.out[w.rl], stage(it) + i * (kTileBytes / 2), 64 * i, w.h, w.t0(it), w.b);
                bulk_commit();
                if (issued < tiles) {
                    bulk_wait_read0();
                    load(issued++);
                }
            }
            // no copy outlives the CTA
            for (int i = max(0, issued - 2); i < issued; ++i)
                mbar_wait(&bar.full[i & 1], (i >> 1) & 1, d.err, kErrDrain);
            bulk_wait0();
        }
    } else if (warp == kMmaWarp) {
        const uint32_t i_k = idesc_bf16(128, 128, false, false), i_q = idesc_bf16(128, Dc, false, false),
                       i_p = idesc_bf16(128, Dc, false, true), i_u = idesc_bf16(128, Db, false, true);
        const uint64_t dM = desc_kmaj(smem_u32(sM), 128, 0);
        for (int it = 0; it < tiles; ++it) {
            const uint32_t ph = it & 1;
            const uint32_t sA = smem_u32(sm) + (uint32_t)(it & 1) * 3 * kTileBytes;
            const uint64_t dA = desc_kmaj(sA, 128, 0), dB = desc_add(dA, kTileBytes),
                           dBt = desc_mnmaj(sA + kTileBytes, 128, 0), dCt = desc_add(dBt, kTileBytes);
            if (!warp_wait(&bar.full[it & 1], (it >> 1) & 1, d.err, kErrMma, d.wait_ns)) break;
            if (it && !warp_wait(&bar.a, ph ^ 1, d.err, kErrMma, d.wait_ns)) break;
            fence_after_sync();
            if (elect_one()) {
#pragma unroll
                for (int s = 0; s < 8; ++s)
                    if (16 * s < Db) {
                        const uint32_t at = (s >> 2) * (kTileBytes / 2) + (s & 3) * 32;
                        mma_bf16_ss(tm + T_Y, desc_add(dA, at), desc_add(dB, at), i_k, s > 0);
                    }
                mma_commit(&bar.k);
            }
            __syncwarp();
            if (!warp_wait(&bar.s, ph, d.err, kErrMma, d.wait_ns)) break;
            if (it && !warp_wait(&bar.x, ph ^ 1, d.err, kErrMma, d.wait_ns)) break;
            fence_after_sync();
            if (elect_one()) {
#pragma unroll
                for (int s = 0; s < 8; ++s)
                    if (16 * s < Db) {
                        const uint32_t at = (s >> 2) * (kTileBytes / 2) + (s & 3) * 32;
                        mma_bf16_ss(tm + T_X, desc_add(dA, at), desc_add(dM, at), i_q, s > 0);
                    }
                mma_commit(&bar.q);
            }
            __syncwarp();
            if (!warp_wait(&bar.cv, ph, d.err, kErrMma, d.wait_ns)) break;
            if (!warp_wait(&bar.r, ph, d.err, kErrMma, d.wait_ns)) break;
            fence_after_sync();
            if (elect_one()) {
#pragma unroll
                for (int s = 0; s < 24; ++s)
                    if (s < 8 * terms)
                        mma_bf16_ts(tm + T_U, tm + T_C + 8 * s, desc_add(dBt, (s & 7) * 2048), i_u, s > 0);
                mma_commit(&bar.u);
            }
            __syncwarp();
            if (!warp_wait(&bar.p, ph, d.err, kErrMma, d.wait_ns)) break;
            fence_after_sync();
            if (elect_one()) {
#pragma unroll
                for (int s = 0; s < 8; ++s)
                    mma_bf16_ts(tm + T_X, tm + T_P + 8 * s, desc_add(dCt, s * 2048), i_p, 1);
                mma_commit(&bar.o);
            }
            __syncwarp();
        }
        if (elect_one()) mma_commit(&bar.drain);  // no MMA outlives the CTA
        warp_wait(&bar.drain, 0, d.err, kErrDrain, 0);
    } else {
        // C' of this warpgroup's 32 tokens of tile it
        auto make = [&](int it) {
            if (!warp_wait(&bar.full[it & 1], (it >> 1) & 1, d.err, kErrState, d.wait_ns)) return false;
            if ((warp & 3) * 32 < Dc)  // else this warp's lanes have no columns of C
                put_updates<32>(smem_u32(sm) + (uint32_t)(it & 1) * 3 * kTileBytes + 2 * kTileBytes,
                            sUpd + (w.len(it) < kTile ? kTile : 0), tl + T_C, (warp & 3) * 32, (warp >> 2) * 32, lane,
                            terms);
            fence_before_sync();
            mbar_arrive(&bar.cv);
            return true;
        };
        if (warp >= 8) state_warps<kLines>(d, w, bar, sm, tl, make);
        else row_warps(d, w, bar, sm, tl, make);
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

template <bool kLines>
cudaError_t launch_scan(const LaDims& d, const LaRoles& roles, const LaMaps& maps, cudaStream_t st) {
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(la_scan_kernel<kLines>, S_SIZE, done);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)(d.NS() * d.nseg), roles.n);
    return launch_dependent(la_scan_kernel<kLines>, grid, kThreads, S_SIZE, st, d, roles, maps);
}

}  // namespace

cudaError_t launch_la_states_tc(const LaDims& d, const LaRoles& roles, cudaStream_t st) {
    LaMaps maps;
    if (!make_maps(d, roles, false, &maps)) return cudaErrorInvalidValue;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(la_sums_kernel, SS_SIZE, done);
    if (e != cudaSuccess) return e;
    return launch_dependent(la_sums_kernel, dim3((unsigned)(d.NS() * (d.nseg - 1)), roles.n), kThreads, SS_SIZE, st, d,
                            roles, maps);
}
cudaError_t launch_la_scan_tc(const LaDims& d, const LaRoles& roles, cudaStream_t st) {
    LaMaps maps;
    if (!make_maps(d, roles, true, &maps)) return cudaErrorInvalidValue;
    return d.L <= kLinesMax * kTile ? launch_scan<true>(d, roles, maps, st) : launch_scan<false>(d, roles, maps, st);
}

}  // namespace gdn
