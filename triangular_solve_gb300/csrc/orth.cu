// Orthogonalisation by Newton-Schulz products (trsm_orthogonalize):
//
//     S = X X^T,   C = a I + b S + c S^2,   X <- C X
//
// for r x c matrices X with r <= c (a taller matrix is taken transposed).
// Of the three products of a step the first two are symmetric and are
// computed for their lower tiles only, each stored twice.
//
// Precision.  Every product takes f16 factors and sums in f32.  What the
// steps amplify is rounding of X in directions where X is small: a step
// multiplies it by a (3.4 as the defaults stand), 140 times over four steps,
// while the large directions stay at one.  Rounding in S and C only turns
// the left singular vectors by as much and is not amplified.  So X alone is
// held in two halves (head and tail, 22 bits) until what is left to amplify
// is below 16, and C X takes two products then.  Measured on low-rank
// matrices over noise: 2.5e-2 of |O|_F with single f16 factors throughout
// (2e-1 with bfloat16), 2e-3 so.
//
// Scaling.  X is stored times 2^14, S and C times 2^12: in f16's normal range
// for any shape, since the singular values stay near or below one.  G enters
// by an exact power of two; what remains of 1 / (|G|_F + eps), a factor rho in
// [1, 2), is applied to the first step's sums, so 16-bit inputs enter exactly.
#include <math.h>
#include <stdint.h>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "internal.h"
#include "orth.h"
#include "tcgen05.cuh"
#include "trsm_model.h"

namespace trsm {
namespace orth {

constexpr float kScaleX = 16384.f, kScaleS = 4096.f;  // 2^14, 2^12

// ------------------------------------------------------------------ |G|_F and the f16 copy
template <typename T> __device__ __forceinline__ float to_f32(T v);
template <> __device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }
template <> __device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }

// Sum of squares without overflow or underflow (J. L. Blue, "A portable
// Fortran program to find the Euclidean norm of a vector", ACM TOMS 4(1),
// 1978): large and small values are squared scaled, each kind on its own.
struct Squares {
    float big = 0.f, mid = 0.f, small = 0.f;
    __device__ __forceinline__ void add(float x) {
        const float y = fabsf(x);
        if (y > 0x1p48f || y < 0x1p-48f) {
            const float b = x * 0x1p-75f, s = x * 0x1p75f;
            if (y > 1.f) big = fmaf(b, b, big);
            else small = fmaf(s, s, small);
        } else {
            mid = fmaf(x, x, mid);  // NaN too
        }
    }
    __device__ __forceinline__ double total() const {
        return (double)big * 0x1p150 + (double)mid + (double)small * 0x1p-150;
    }
};

constexpr int kNormThreads = 256;
constexpr int kNormBlocks = 64;  // per matrix, at most

// Sum over a block's threads, in a fixed order; valid in thread 0.
__device__ __forceinline__ double block_sum(double v) {
    __shared__ double part[kNormThreads / 32];
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_down_sync(~0u, v, o);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    if (threadIdx.x == 0)
        for (int w = 1; w < kNormThreads / 32; ++w) v += part[w];
    return v;
}

struct Input {
    const void *G;
    int64_t m, n, ld, stride;  // rows, columns as given
    bool vec;                  // rows of 16-byte vectors
};

template <typename T>
__global__ void __launch_bounds__(kNormThreads) norm_kernel(const Input in, double *__restrict__ partial) {
    constexpr int kVec = 16 / sizeof(T);
    const T *G = static_cast<const T *>(in.G) + blockIdx.y * in.stride;
    Squares s;
    // vectors (or elements) of the rows in turn, without a division in the loop
    const int64_t per = in.vec ? in.n / kVec : in.n;
    const int64_t first = (int64_t)blockIdx.x * kNormThreads + threadIdx.x, step = (int64_t)gridDim.x * kNormThreads;
    const int64_t drow = step / per, dcol = step % per;
    int64_t row = first / per, col = first % per;
    while (row < in.m) {
        if (in.vec) {
            const uint4 w = *reinterpret_cast<const uint4 *>(G + row * in.ld + col * kVec);
            const T *v = reinterpret_cast<const T *>(&w);
#pragma unroll
            for (int k = 0; k < kVec; ++k) s.add(to_f32<T>(v[k]));
        } else {
            s.add(to_f32<T>(G[row * in.ld + col]));
        }
        row += drow;
        col += dcol;
        if (col >= per) {
            col -= per;
            ++row;
        }
    }
    const double t = block_sum(s.total());
    if (threadIdx.x == 0) partial[(int64_t)blockIdx.y * gridDim.x + blockIdx.x] = t;
}

// 1 / (|G|_F + eps) as 2^e rho, rho in [1, 2); NaN where it is no positive
// number.  Called by a whole block; every thread gets the same.
struct Scale {
    float up, more, rho;  // 2^e = up * more, neither of which overflows
};
__device__ __forceinline__ Scale scale_of(const double *partial, int count, double eps) {
    __shared__ Scale shared;
    if (threadIdx.x < 32) {
        double sum = 0;
        for (int i = threadIdx.x; i < count; i += 32) sum += partial[i];
#pragma unroll
        for (int o = 16; o; o >>= 1) sum += __shfl_down_sync(~0u, sum, o);
        if (threadIdx.x == 0) {
            const double s = 1.0 / (sqrt(sum) + eps);
            if (s > 0 && s < 1e300) {
                int e = ilogb(s);
                const float rho = (float)scalbn(s, -e);
                e = min(max(e, -160), 240);
                shared = {scalbnf(1.f, e / 2), scalbnf(1.f, e - e / 2), rho};
            } else {
                shared = {1.f, 1.f, __int_as_float(0x7fffffff)};
            }
        }
    }
    __syncthreads();
    return shared;
}

struct Halves {
    __half *hi, *lo;      // lo: null where X is not split
    int64_t r, c, ld, stride;
};

__device__ __forceinline__ void split(float x, __half &hi, __half &lo) {
    hi = __float2half_rn(x);
    lo = __float2half_rn(x - __half2float(hi));
}

// X_0 = 2^14 2^e G in f16 (head and tail), transposed for a tall G, in tiles
// of 64 x 64 through shared memory; rho goes to rho[b].  With out != null
// (no steps): O = 2^e rho G instead.
template <typename T, bool TALL>
__global__ void __launch_bounds__(256) convert_kernel(const Input in, const double *__restrict__ partial, int count,
                                                      double eps, const Halves x, float *__restrict__ rho, void *out,
                                                      int64_t ldo, int64_t strideO, int out_bf16) {
    __shared__ float tile[64][65];
    const int b = blockIdx.z, tid = threadIdx.x;
    const Scale sc = scale_of(partial + (int64_t)b * count, count, eps);
    const T *G = static_cast<const T *>(in.G) + b * in.stride;
    // tile of X: rows i0.., columns j0..; G's element is (i, j), or (j, i) tall
    const int64_t i0 = (int64_t)blockIdx.y * 64, j0 = (int64_t)blockIdx.x * 64;
    if (tid == 0 && blockIdx.x == 0 && blockIdx.y == 0) rho[b] = sc.rho;
    const float s14 = out ? 1.f : kScaleX;
#pragma unroll
    for (int q = 0; q < 16; ++q) {
        const int u = q * 4 + tid / 64, v = tid % 64;  // v along G's rows
        const int64_t i = TALL ? i0 + v : i0 + u, j = TALL ? j0 + u : j0 + v;
        float g = 0.f;
        if (i < x.r && j < x.c) {
            g = to_f32<T>(TALL ? G[j * in.ld + i] : G[i * in.ld + j]);
            g = g * sc.up * sc.more * s14;
        }
        if (TALL) tile[v][u] = g;
        else tile[u][v] = g;
    }
    __syncthreads();
    if (out) {
#pragma unroll
        for (int q = 0; q < 16; ++q) {
            const int u = q * 4 + tid / 64, v = tid % 64;  // v along O's rows
            const int64_t i = TALL ? i0 + v : i0 + u, j = TALL ? j0 + u : j0 + v;
            if (i < x.r && j < x.c) {
                const float o = (TALL ? tile[v][u] : tile[u][v]) * sc.rho;
                const int64_t at = b * strideO + (TALL ? j * ldo + i : i * ldo + j);
                if (out_bf16) static_cast<__nv_bfloat16 *>(out)[at] = __float2bfloat16_rn(o);
                else static_cast<__half *>(out)[at] = __float2half_rn(o);
            }
        }
        return;
    }
    // 8 halves a thread: 64 rows of 8 groups; the row's padding gets zeros
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int u = q * 32 + tid / 8, v = tid % 8 * 8;
        const int64_t i = i0 + u, j = j0 + v;
        if (i < x.r && j < x.ld) {
            alignas(16) __half hi[8], lo[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) split(tile[u][v + k], hi[k], lo[k]);
            const int64_t at = b * x.stride + i * x.ld + j;
            *reinterpret_cast<uint4 *>(x.hi + at) = *reinterpret_cast<const uint4 *>(hi);
            if (x.lo) *reinterpret_cast<uint4 *>(x.lo + at) = *reinterpret_cast<const uint4 *>(lo);
        }
    }
}

// ------------------------------------------------------------------ products
enum Mode { kGram, kPoly, kApply, kFinish };

struct ProductArgs {
    int M, N, K, batch;
    int tiles_m, tiles_n, tiles;  // of one matrix; all
    int symmetric;                // only tiles that reach the diagonal or below
    int halves;                   // B head only (1) or head and tail (2)
    Mode mode;
    float alpha;                  // factor of the sums (kGram, kApply, kFinish: times rho's power)
    float beta, diag;             // kPoly: plus beta S plus diag I
    const float *rho;             // per matrix, or null
    const __half *S;
    __half *out, *out_lo;         // out_lo: tail, or null
    int64_t ld, stride;           // of S, out and out_lo
    void *O;                      // kFinish
    int64_t ldo, strideO;
    int transposed, bf16, vec;    // of O; vec: its rows take 16-byte stores
    int *status;
};

struct Maps {
    CUtensorMap a, b_hi, b_lo;
};

constexpr int kTileM = 256, kBK = 64;
constexpr uint32_t kABytes = 128 * kBK * 2;  // 128 rows of A per CTA
constexpr uint32_t kTmemCols = 512;

template <int BN> struct Ring {
    static constexpr uint32_t kBBytes = BN / 2 * kBK * 2;  // half of B's columns per CTA
    static constexpr uint32_t kStage = kABytes + kBBytes;
    static constexpr int kStages = BN == 256 ? 6 : 8;
    static constexpr uint32_t kBars = 8u * (2 * kStages + 5);
    static constexpr size_t kSmem = 1024 + kStages * kStage + 256;
    static_assert(kBars + 4 <= 256, "barriers and the TMEM address fit their region");
};

__device__ __forceinline__ uint32_t pack_half(float x, float y) {
    const __half2 h = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// A persistent kernel on CTA pairs; each pair takes 256 x BN tiles of the
// output in turn.  Warp 0 loads (TMA, a ring of kStages slabs of K = 64),
// warp 1 of the even CTA issues the MMAs, warps 2..5 empty the accumulators
// (two in TMEM, so a tile's stores run under the next one's MMAs).
//
// B is Y^T for a K-major Y (kGram, kPoly; Y = A's matrix) or a K x N matrix
// with contiguous N (kApply, kFinish; BMN).
template <int BN, bool BMN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(192, 1)
    product_kernel(const __grid_constant__ Maps maps, const __grid_constant__ ProductArgs g) {
    using R = Ring<BN>;
    extern __shared__ unsigned char smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;  // the swizzle's period
    const uint32_t bars = base + R::kStages * R::kStage;
    auto full = [&](int s) { return bars + 8u * s; };
    auto empty = [&](int s) { return bars + 8u * (R::kStages + s); };
    auto acc_full = [&](int a) { return bars + 8u * (2 * R::kStages + a); };
    auto acc_empty = [&](int a) { return bars + 8u * (2 * R::kStages + 2 + a); };
    const uint32_t drain = bars + 8u * (2 * R::kStages + 4);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem_raw + (bars - raw) + R::kBars);
    __shared__ int abort_flag;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster::rank();
    const bool leader = rank == 0;
    const int pair = (int)blockIdx.x >> 1, npairs = (int)gridDim.x >> 1;
    const int nk = (g.K + kBK - 1) / kBK, slabs = nk * g.halves;
    // tile t -> matrix z, row tile tm, column tile tn
    auto tile_of = [&](int t, int &z, int &tm, int &tn) {
        const int per = g.tiles / g.batch;
        z = t / per;
        int u = t % per;
        if (g.symmetric) {
            // row tile tm has the column tiles up to the diagonal's
            constexpr int kPer = kTileM / BN;
            tm = 0;
            int width = min(kPer, g.tiles_n);
            while (u >= width) {
                u -= width;
                ++tm;
                width = min(kPer * (tm + 1), g.tiles_n);
            }
            tn = u;
        } else {
            // groups of 8 row tiles, so that a wave shares its operands in L2
            const int grp = u / (8 * g.tiles_n), rem = u - grp * 8 * g.tiles_n;
            const int size = min(8, g.tiles_m - grp * 8);
            tm = grp * 8 + rem % size;
            tn = rem / size;
        }
    };

    if (threadIdx.x == 0) {
        abort_flag = 0;
        for (int s = 0; s < R::kStages; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(acc_full(a), 1);
            mbar_init(acc_empty(a), 8);  // four warps in each CTA
        }
        mbar_init(drain, 1);
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    }
    if (warp == 1) tc5::alloc_pair(smem_u32(tmem_slot), kTmemCols);
    tc5::fence_before();
    __syncthreads();
    cluster::sync();  // the peer's barriers exist before anything signals them
    tc5::fence_after();
    const uint32_t tmem = *tmem_slot;
    auto aborted = [&]() { return *(volatile int *)&abort_flag != 0; };
    auto fail = [&]() {
        record_timeout(g.status);
        *(volatile int *)&abort_flag = 1;
    };

    if (warp == 0) {
        if (lane == 0) {
            int it = 0;
            for (int t = pair; t < g.tiles && !aborted(); t += npairs) {
                int z, tm, tn;
                tile_of(t, z, tm, tn);
                const int ya = tm * kTileM + 128 * (int)rank, yb = tn * BN + BN / 2 * (int)rank;
                for (int kb = 0; kb < slabs; ++kb, ++it) {
                    const int s = it % R::kStages;
                    if (it >= R::kStages && !mbar_wait(empty(s), ((it / R::kStages) - 1) & 1)) {
                        fail();
                        break;
                    }
                    if (leader) mbar_expect_tx(full(s), 2 * R::kStage);
                    const uint32_t st = base + s * R::kStage, fb = cluster::map(full(s), 0);
                    const int kx = kb % nk * kBK;
                    const CUtensorMap *mb = kb < nk ? &maps.b_hi : &maps.b_lo;
                    tc5::load_pair(st, &maps.a, kx, ya, z, fb);
                    if constexpr (BMN) {
#pragma unroll
                        for (int q = 0; q < BN / 128; ++q)
                            tc5::load_pair(st + kABytes + q * (64 * kBK * 2), mb, yb + 64 * q, kx, z, fb);
                    } else {
                        tc5::load_pair(st + kABytes, mb, kx, yb, z, fb);
                    }
                }
            }
            if (aborted() && leader) {
                // the pair's loads counted on these barriers land before shared memory goes away
                for (int j = (it > R::kStages ? it - R::kStages : 0); j < it; ++j)
                    if (!mbar_wait(full(j % R::kStages), (j / R::kStages) & 1)) record_timeout(g.status);
            }
        }
    } else if (warp == 1) {
        if (lane == 0 && leader) {
            constexpr uint32_t idesc = tc5::idesc_f16(kTileM, BN, BMN);
            int it = 0, i = 0;
            for (int t = pair; t < g.tiles && !aborted(); t += npairs, ++i) {
                const int a = i & 1;
                if (i >= 2 && !mbar_wait(acc_empty(a), ((i >> 1) - 1) & 1)) {
                    fail();
                    break;
                }
                tc5::fence_after();
                const uint32_t d = tmem + (uint32_t)(a * 256);
                bool ok = true;
                for (int kb = 0; kb < slabs; ++kb, ++it) {
                    const int s = it % R::kStages;
                    if (!mbar_wait(full(s), (it / R::kStages) & 1)) {
                        fail();
                        ok = false;
                        break;
                    }
                    tc5::fence_after();
                    const uint32_t st = base + s * R::kStage;
#pragma unroll
                    for (int kk = 0; kk < kBK / 16; ++kk) {
                        const uint64_t da = tc5::desc_k_major(st + kk * 32);
                        const uint64_t db = BMN ? tc5::desc_mn_major(st + kABytes + kk * 2048, 64 * kBK * 2)
                                                : tc5::desc_k_major(st + kABytes + kk * 32);
                        tc5::mma_pair(d, da, db, idesc, kb != 0 || kk != 0);
                    }
                    tc5::commit_both(empty(s));  // both CTAs' slab is free once these have read it
                }
                tc5::commit_both(acc_full(a));
                if (!ok) break;
            }
            tc5::commit_local(drain);
            if (!mbar_wait(drain, 0)) record_timeout(g.status);
        }
    } else {
        const int quarter = warp & 3;  // TMEM lanes 32 * quarter .. + 31
        int i = 0;
        for (int t = pair; t < g.tiles; t += npairs, ++i) {
            const int a = i & 1;
            int z, tm, tn;
            tile_of(t, z, tm, tn);
            const int row = tm * kTileM + 128 * (int)rank + 32 * quarter + lane, col0 = tn * BN;
            const bool row_ok = row < g.M;
            const int64_t at = z * g.stride + (int64_t)row * g.ld;
            float alpha = g.alpha;
            if (g.rho) alpha *= g.mode == kGram ? g.rho[z] * g.rho[z] : g.rho[z];
            if (!mbar_wait(acc_full(a), (i >> 1) & 1)) {
                if (lane == 0) fail();
                break;
            }
            if (aborted()) break;
            tc5::fence_after();
            const uint32_t addr = tmem + ((uint32_t)(32 * quarter) << 16) + (uint32_t)(a * 256);
#pragma unroll 1
            for (int chunk = 0; chunk < BN / 32; ++chunk) {
                const int col = col0 + chunk * 32;
                uint32_t v[32];
                tc5::read_32(v, addr + chunk * 32);
                if (chunk + 1 == BN / 32) {
                    tc5::fence_before();
                    __syncwarp();
                    if (lane == 0) tc5::arrive_cluster(cluster::map(acc_empty(a), 0));
                }
                if (!row_ok || col >= g.N) continue;
                if (g.mode == kFinish) {
                    float o[32];
#pragma unroll
                    for (int j = 0; j < 32; ++j) o[j] = alpha * __uint_as_float(v[j]);
                    const int64_t zo = z * g.strideO;
                    auto put = [&](int64_t p, float x) {
                        if (g.bf16) static_cast<__nv_bfloat16 *>(g.O)[p] = __float2bfloat16_rn(x);
                        else static_cast<__half *>(g.O)[p] = __float2half_rn(x);
                    };
                    if (g.transposed) {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (col + j < g.N) put(zo + (int64_t)(col + j) * g.ldo + row, o[j]);
                    } else if (g.vec && col + 32 <= g.N) {
                        uint32_t w[16];
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            if (g.bf16) {
                                const __nv_bfloat162 h = __floats2bfloat162_rn(o[2 * j], o[2 * j + 1]);
                                w[j] = *reinterpret_cast<const uint32_t *>(&h);
                            } else {
                                w[j] = pack_half(o[2 * j], o[2 * j + 1]);
                            }
                        }
                        uint4 *p = reinterpret_cast<uint4 *>(static_cast<__half *>(g.O) + zo + (int64_t)row * g.ldo + col);
#pragma unroll
                        for (int j = 0; j < 4; ++j) p[j] = make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (col + j < g.N) put(zo + (int64_t)row * g.ldo + col + j, o[j]);
                    }
                    continue;
                }
                if (g.symmetric && col > row) continue;
                float o[32];
                if (g.mode == kPoly) {
                    const __half *s = g.S + at + col;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        uint4 w = make_uint4(0, 0, 0, 0);
                        if (col + 8 * q < g.ld) w = *reinterpret_cast<const uint4 *>(s + 8 * q);
                        const __half *h = reinterpret_cast<const __half *>(&w);
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            o[8 * q + j] = fmaf(g.beta, __half2float(h[j]), alpha * __uint_as_float(v[8 * q + j]));
                            if (col + 8 * q + j == row) o[8 * q + j] += g.diag;
                        }
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j) o[j] = alpha * __uint_as_float(v[j]);
                }
                if (!g.symmetric) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        if (col + 8 * q < g.ld) {  // the row's padding gets the zeros beyond N
                            alignas(16) __half hi[8], lo[8];
#pragma unroll
                            for (int j = 0; j < 8; ++j) split(o[8 * q + j], hi[j], lo[j]);
                            *reinterpret_cast<uint4 *>(g.out + at + col + 8 * q) = *reinterpret_cast<const uint4 *>(hi);
                            if (g.out_lo)
                                *reinterpret_cast<uint4 *>(g.out_lo + at + col + 8 * q) =
                                    *reinterpret_cast<const uint4 *>(lo);
                        }
                    }
                } else {
                    // the part on and below the diagonal, and its mirror image
                    __half *out = g.out + z * g.stride;
                    if (col + 31 <= row) {
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            *reinterpret_cast<uint4 *>(out + (int64_t)row * g.ld + col + 8 * q) = make_uint4(
                                pack_half(o[8 * q], o[8 * q + 1]), pack_half(o[8 * q + 2], o[8 * q + 3]),
                                pack_half(o[8 * q + 4], o[8 * q + 5]), pack_half(o[8 * q + 6], o[8 * q + 7]));
#pragma unroll
                        for (int j = 0; j < 32; ++j) out[(int64_t)(col + j) * g.ld + row] = __float2half_rn(o[j]);
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            if (col + j <= row) {
                                const __half h = __float2half_rn(o[j]);
                                out[(int64_t)row * g.ld + col + j] = h;
                                out[(int64_t)(col + j) * g.ld + row] = h;
                            }
                        }
                    }
                }
            }
        }
    }
    tc5::fence_before();
    __syncthreads();
    cluster::sync();  // the pair's MMAs and loads are done with both CTAs' memory
    if (warp == 1) {
        tc5::fence_after();
        tc5::dealloc_pair(tmem, kTmemCols);
    }
}

// ------------------------------------------------------------------ launch
int64_t up8(int64_t v) { return (v + 7) / 8 * 8; }

// Which X_k (k = 0 .. steps - 1) have a tail: those whose rounding the steps
// from k on can amplify more than kMostAmplified times.  X_0 of a 16-bit
// input is exact.
constexpr double kMostAmplified = 16.0;
bool has_tail(const double *coef, int steps, int k, bool exact_input) {
    if (k == 0 && exact_input) return false;
    double grow = 1;
    for (int j = k; j < steps; ++j) grow *= fabs(coef[3 * j]);
    return grow > kMostAmplified;
}

int norm_blocks(int64_t m, int64_t n) {
    const int64_t want = (m * n + kNormThreads * 32 - 1) / (kNormThreads * 32);
    return (int)(want < 1 ? 1 : want > kNormBlocks ? kNormBlocks : want);
}

// Regions of the workspace, each a multiple of 256 bytes: X twice (a step
// reads one and writes the other), its tails twice, S, C, the partial sums
// and rho.
struct Layout {
    int64_t r, c, ldx, lds;
    size_t x, s, partial, rho;
    Layout(int64_t m, int64_t n, int64_t batch) {
        r = m < n ? m : n;
        c = m < n ? n : m;
        ldx = up8(c);
        lds = up8(r);
        x = (size_t)round256(batch * r * ldx * 2);
        s = (size_t)round256(batch * r * lds * 2);
        partial = (size_t)round256(batch * kNormBlocks * 8);
        rho = (size_t)round256(batch * 4);
    }
    size_t total() const { return 4 * x + 2 * s + partial + rho; }
};

int make_map(CUtensorMap *map, const __half *p, int64_t inner, int64_t rows, int64_t batch, int64_t ld, int64_t stride,
             int box_inner, int box_rows) {
    static const PFN_cuTensorMapEncodeTiled_v12000 encode = [] {
        void *fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) !=
                cudaSuccess || q != cudaDriverEntryPointSuccess)
            fn = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    }();
    if (!encode) return TRSM_ERR_CUDA_BASE + (int)cudaErrorNotSupported;
    const cuuint64_t dims[3] = {(cuuint64_t)inner, (cuuint64_t)rows, (cuuint64_t)batch};
    const cuuint64_t strides[2] = {(cuuint64_t)(ld * 2), (cuuint64_t)(stride * 2)};
    const cuuint32_t box[3] = {(cuuint32_t)box_inner, (cuuint32_t)box_rows, 1}, one[3] = {1, 1, 1};
    const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<__half *>(p), dims, strides, box, one,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? TRSM_SUCCESS : TRSM_ERR_CUDA_BASE + (int)cudaErrorInvalidValue;
}

int sm_count(int *out) {
    static int sms = 0;
    if (!sms) {
        int dev = 0, v = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e == cudaSuccess) e = cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return cuda_status(e);
        sms = v;
    }
    *out = sms;
    return TRSM_SUCCESS;
}

// One operand: an f16 matrix per batch entry, inner x rows, ld and stride in halves.
struct Operand {
    const __half *hi, *lo;
    int64_t inner, rows, ld, stride;
};

template <int BN, bool BMN>
int launch_product(const Operand &A, const Operand &B, ProductArgs g, cudaStream_t st) {
    using R = Ring<BN>;
    Maps maps;
    int rc = make_map(&maps.a, A.hi, A.inner, A.rows, g.batch, A.ld, A.stride, kBK, 128);
    const int bi = BMN ? 64 : kBK, br = BMN ? kBK : BN / 2;
    if (!rc) rc = make_map(&maps.b_hi, B.hi, B.inner, B.rows, g.batch, B.ld, B.stride, bi, br);
    if (!rc) rc = make_map(&maps.b_lo, B.lo ? B.lo : B.hi, B.inner, B.rows, g.batch, B.ld, B.stride, bi, br);
    int sms = 0;
    if (!rc) rc = sm_count(&sms);
    if (!rc) rc = device_status_word(&g.status);
    if (rc) return rc;
    g.halves = B.lo ? 2 : 1;
    g.tiles_m = (g.M + kTileM - 1) / kTileM;
    g.tiles_n = (g.N + BN - 1) / BN;
    int64_t per = (int64_t)g.tiles_m * g.tiles_n;
    if (g.symmetric) {
        per = 0;
        for (int tm = 0; tm < g.tiles_m; ++tm) {
            const int w = kTileM / BN * (tm + 1);
            per += w < g.tiles_n ? w : g.tiles_n;
        }
    }
    if (per * g.batch > 0x7fffffff) return -11;
    g.tiles = (int)(per * g.batch);
    cudaError_t e = cudaFuncSetAttribute(product_kernel<BN, BMN>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)R::kSmem);
    if (e != cudaSuccess) return cuda_status(e);
    const int pairs = g.tiles < sms / 2 ? g.tiles : sms / 2;
    product_kernel<BN, BMN><<<2 * pairs, 192, R::kSmem, st>>>(maps, g);
    return launch_status();
}

template <bool BMN>
int product(const Operand &A, const Operand &B, const ProductArgs &g, int sms, cudaStream_t st) {
    // 256 x 128 tiles while 256 x 256 ones would leave CTA pairs without one
    const int64_t wide = (int64_t)((g.M + 255) / 256) * ((g.N + 255) / 256) * g.batch;
    if (g.N <= 128 || wide < sms / 2) return launch_product<128, BMN>(A, B, g, st);
    return launch_product<256, BMN>(A, B, g, st);
}

template <typename T>
int convert(const OrthArgs &a, const Input &in, const Halves &x, double *partial, float *rho, cudaStream_t st) {
    const int nb = norm_blocks(a.m, a.n);
    norm_kernel<T><<<dim3(nb, (unsigned)a.batch), kNormThreads, 0, st>>>(in, partial);
    int rc = launch_status();
    if (rc) return rc;
    const dim3 grid((unsigned)((x.c + 63) / 64), (unsigned)((x.r + 63) / 64), (unsigned)a.batch);
    void *out = a.steps ? nullptr : a.O;
    if (a.m > a.n)
        convert_kernel<T, true><<<grid, 256, 0, st>>>(in, partial, nb, a.eps, x, rho, out, a.ldo, a.strideO,
                                                      a.out_dtype == TRSM_ELEM_BF16);
    else
        convert_kernel<T, false><<<grid, 256, 0, st>>>(in, partial, nb, a.eps, x, rho, out, a.ldo, a.strideO,
                                                       a.out_dtype == TRSM_ELEM_BF16);
    return launch_status();
}

int run(const OrthArgs &a, cudaStream_t st) {
    const Layout w(a.m, a.n, a.batch);
    char *p = static_cast<char *>(a.ws);
    __half *xh[2], *xl[2];
    for (int k = 0; k < 2; ++k) {
        xh[k] = reinterpret_cast<__half *>(p + k * w.x);
        xl[k] = reinterpret_cast<__half *>(p + (2 + k) * w.x);
    }
    __half *S = reinterpret_cast<__half *>(p + 4 * w.x), *C = reinterpret_cast<__half *>(p + 4 * w.x + w.s);
    double *partial = reinterpret_cast<double *>(p + 4 * w.x + 2 * w.s);
    float *rho = reinterpret_cast<float *>(p + 4 * w.x + 2 * w.s + w.partial);

    const int64_t es = a.in_dtype == TRSM_ELEM_F32 ? 4 : 2;
    Input in = {a.G, a.m, a.n, a.ldg, a.strideG, false};
    uintptr_t bits = (uintptr_t)a.G | (uintptr_t)(a.n * es);
    if (a.m > 1) bits |= (uintptr_t)(a.ldg * es);
    if (a.batch > 1) bits |= (uintptr_t)(a.strideG * es);
    in.vec = bits % 16 == 0;
    const bool exact = a.in_dtype != TRSM_ELEM_F32;
    bool tail = has_tail(a.coef, a.steps, 0, exact);
    const Halves x0 = {xh[0], tail ? xl[0] : nullptr, w.r, w.c, w.ldx, w.r * w.ldx};
    int rc, sms = 0;
    switch (a.in_dtype) {
        case TRSM_ELEM_F32: rc = convert<float>(a, in, x0, partial, rho, st); break;
        case TRSM_ELEM_F16: rc = convert<__half>(a, in, x0, partial, rho, st); break;
        default: rc = convert<__nv_bfloat16>(a, in, x0, partial, rho, st); break;
    }
    if (!rc) rc = sm_count(&sms);
    for (int k = 0; k < a.steps && !rc; ++k) {
        const double ca = a.coef[3 * k], cb = a.coef[3 * k + 1], cc = a.coef[3 * k + 2];
        const int from = k & 1, to = from ^ 1;
        const Operand X = {xh[from], tail ? xl[from] : nullptr, w.c, w.r, w.ldx, w.r * w.ldx};
        const Operand Xhead = {X.hi, nullptr, X.inner, X.rows, X.ld, X.stride};
        const Operand So = {S, nullptr, w.r, w.r, w.lds, w.r * w.lds}, Co = {C, nullptr, w.r, w.r, w.lds, w.r * w.lds};
        ProductArgs g = {};
        g.batch = (int)a.batch;
        g.rho = k == 0 ? rho : nullptr;
        // S = X X^T
        g.M = g.N = (int)w.r;
        g.K = (int)w.c;
        g.symmetric = 1;
        g.mode = kGram;
        g.alpha = kScaleS / (kScaleX * kScaleX);
        g.out = S;
        g.ld = w.lds;
        g.stride = w.r * w.lds;
        rc = product<false>(Xhead, Xhead, g, sms, st);
        if (rc) break;
        // C = a I + b S + c S^2
        g.K = (int)w.r;
        g.mode = kPoly;
        g.rho = nullptr;
        g.alpha = (float)cc / kScaleS;
        g.beta = (float)cb;
        g.diag = (float)ca * kScaleS;
        g.S = S;
        g.out = C;
        rc = product<false>(So, So, g, sms, st);
        if (rc) break;
        // X = C X
        g.rho = k == 0 ? rho : nullptr;
        g.symmetric = 0;
        g.N = (int)w.c;
        g.alpha = 1.f / kScaleS;
        g.ld = w.ldx;
        g.stride = w.r * w.ldx;
        if (k + 1 < a.steps) {
            tail = has_tail(a.coef, a.steps, k + 1, exact);
            g.mode = kApply;
            g.out = xh[to];
            g.out_lo = tail ? xl[to] : nullptr;
        } else {
            g.mode = kFinish;
            g.alpha /= kScaleX;
            g.O = a.O;
            g.ldo = a.ldo;
            g.strideO = a.strideO;
            g.transposed = a.m > a.n;
            g.bf16 = a.out_dtype == TRSM_ELEM_BF16;
            uintptr_t ob = (uintptr_t)a.O | (uintptr_t)(a.ldo * 2);
            if (a.batch > 1) ob |= (uintptr_t)(a.strideO * 2);
            g.vec = ob % 16 == 0;
        }
        rc = product<true>(Co, X, g, sms, st);
    }
    return rc;
}

}  // namespace orth

size_t orth_workspace_bytes(int, int64_t m, int64_t n, int64_t batch, int64_t) {
    return orth::Layout(m, n, batch).total();
}

int orth_run(const OrthArgs &a, cudaStream_t st) { return orth::run(a, st); }

}  // namespace trsm
