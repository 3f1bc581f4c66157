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
constexpr int kNormBlocks = 512;  // per matrix, at most

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

// Eight elements of a row of G from column j on, zero past column n.
template <typename T>
__device__ __forceinline__ void load_8(const T *row, int64_t j, int64_t n, bool vec, float (&g)[8]) {
    if (vec && j + 8 <= n) {
        alignas(16) T v[8];
#pragma unroll
        for (int k = 0; k < (int)sizeof(T) / 2; ++k)
            reinterpret_cast<uint4 *>(v)[k] = reinterpret_cast<const uint4 *>(row + j)[k];
#pragma unroll
        for (int k = 0; k < 8; ++k) g[k] = to_f32<T>(v[k]);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) g[k] = j + k < n ? to_f32<T>(row[j + k]) : 0.f;
    }
}

// X_0 = 2^14 2^e G in f16 (head and tail), transposed for a tall G, in tiles
// of 64 x 64, a few for each block; rho goes to rho[b].  With out != null (no
// steps): O = 2^e rho G instead.
template <typename T, bool TALL>
__global__ void __launch_bounds__(256) convert_kernel(const Input in, const double *__restrict__ partial, int count,
                                                      double eps, const Halves x, float *__restrict__ rho, void *out,
                                                      int64_t ldo, int64_t strideO, int out_bf16) {
    __shared__ float tile[TALL ? 64 : 1][65];
    const int b = blockIdx.y, tid = threadIdx.x, u = tid / 8, v = tid % 8 * 8;
    const Scale sc = scale_of(partial + (int64_t)b * count, count, eps);
    const T *G = static_cast<const T *>(in.G) + b * in.stride;
    if (tid == 0 && blockIdx.x == 0) rho[b] = sc.rho;
    const int64_t across = (in.n + 63) / 64, tiles = across * ((in.m + 63) / 64);
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        const int64_t i0 = t / across * 64, j0 = t % across * 64;  // of G
        if (TALL) __syncthreads();
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int64_t i = i0 + u + 32 * q, j = j0 + v;
            if (i >= in.m) continue;
            float g[8];
            load_8<T>(G + i * in.ld, j, in.n, in.vec, g);
            if (out) {
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    if (j + k >= in.n) break;
                    const float o = g[k] * sc.up * sc.more * sc.rho;
                    const int64_t at = b * strideO + i * ldo + j + k;
                    if (out_bf16) static_cast<__nv_bfloat16 *>(out)[at] = __float2bfloat16_rn(o);
                    else static_cast<__half *>(out)[at] = __float2half_rn(o);
                }
                continue;
            }
            alignas(16) __half hi[8], lo[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                g[k] = g[k] * sc.up * sc.more * kScaleX;
                if (TALL) tile[u + 32 * q][v + k] = g[k];
                else split(g[k], hi[k], lo[k]);
            }
            if (!TALL && j < x.ld) {
                const int64_t at = b * x.stride + i * x.ld + j;
                *reinterpret_cast<uint4 *>(x.hi + at) = *reinterpret_cast<const uint4 *>(hi);
                if (x.lo) *reinterpret_cast<uint4 *>(x.lo + at) = *reinterpret_cast<const uint4 *>(lo);
            }
        }
        if (!TALL || out) continue;
        __syncthreads();
        // X's row is G's column; rows of the tile past m hold leftovers, which
        // only reach the padding of X's rows
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int64_t i = j0 + u + 32 * q, j = i0 + v;  // of X
            if (i >= x.r || j >= x.ld) continue;
            alignas(16) __half hi[8], lo[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) split(tile[v + k][u + 32 * q], hi[k], lo[k]);
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
    int tail;                     // kApply: the result's tail goes out too
    int transposed, bf16;         // kFinish
    void *O;                      // kFinish: stored element by element; null: through the maps
    int64_t ldo, strideO;
    int *status;
};

// out: the output in boxes of 32 rows x 64 columns (128-byte swizzle).
// second: kApply the tail's likewise; symmetric or transposed, the output in
// boxes of 64 rows x 32 columns.  in: kPoly, S as `out`.
struct Maps {
    CUtensorMap a, b_hi, b_lo, out, second, in;
};

constexpr int kTileM = 256, kBK = 64;
constexpr uint32_t kABytes = 128 * kBK * 2;  // 128 rows of A per CTA
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kBox = 32 * 64 * 2;       // bytes of a box of the output

template <int BN> struct Ring {
    static constexpr uint32_t kBBytes = BN / 2 * kBK * 2;  // half of B's columns per CTA
    static constexpr uint32_t kStage = kABytes + kBBytes;
    static constexpr int kStages = BN == 256 ? 5 : 6;
    static constexpr uint32_t kOut = kStages * kStage;     // output boxes: 2 by turns x 2 for each of 4 warps
    static constexpr uint32_t kBars = kOut + 16 * kBox;
    static constexpr uint32_t kTmem = kBars + 8u * (2 * kStages + 5 + 8);
    static constexpr size_t kSmem = 1024 + kBars + 256;
    static_assert(kTmem + 4 <= kBars + 256 && kSmem <= 227 * 1024, "shared memory");
};

__device__ __forceinline__ uint32_t pack_half(float x, float y) {
    const __half2 h = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t pack_out(float x, float y, bool bf16) {
    if (!bf16) return pack_half(x, y);
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// A persistent kernel on CTA pairs; each pair takes 256 x BN tiles of the
// output in turn.  Warp 0 loads (TMA, a ring of slabs of K = 64), warp 1 of
// the even CTA issues the MMAs, warps 2..5 empty the accumulators (two in
// TMEM, so a tile's way out runs under the next one's MMAs): 64 columns at a
// time through shared memory, from where TMA stores them, rows whole, and
// for a symmetric product below the diagonal once more transposed.
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
    unsigned char *const smem = smem_raw + (base - raw);
    const uint32_t bars = base + R::kBars;
    auto full = [&](int s) { return bars + 8u * s; };
    auto empty = [&](int s) { return bars + 8u * (R::kStages + s); };
    auto acc_full = [&](int a) { return bars + 8u * (2 * R::kStages + a); };
    auto acc_empty = [&](int a) { return bars + 8u * (2 * R::kStages + 2 + a); };
    const uint32_t drain = bars + 8u * (2 * R::kStages + 4);
    auto s_full = [&](int w, int k) { return bars + 8u * (2 * R::kStages + 5 + 2 * w + k); };  // kPoly: S has come
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + R::kTmem);
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
        for (int w = 0; w < 4; ++w)
            for (int k = 0; k < 2; ++k) mbar_init(s_full(w, k), 1);
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
        // this warp's boxes, first and second of each turn
        auto box = [&](int turn, int k) { return R::kOut + (uint32_t)(quarter * 4 + turn * 2 + k) * kBox; };
        int i = 0, turns = 0, issued = 0;  // groups done; loads of S (lane 0)
        bool ok = true;
        for (int t = pair; t < g.tiles && ok; t += npairs, ++i) {
            const int a = i & 1;
            int z, tm, tn;
            tile_of(t, z, tm, tn);
            const int row0 = tm * kTileM + 128 * (int)rank + 32 * quarter, row = row0 + lane, col0 = tn * BN;
            // 64-column groups of this warp inside the output
            const int groups = row0 >= g.M ? 0 : min(BN / 64, (g.N - col0 + 63) / 64);
            const bool mirror = g.symmetric && col0 + BN <= tm * kTileM;  // below the diagonal tile
            float alpha = g.alpha;
            if (g.rho) alpha *= g.mode == kGram ? g.rho[z] * g.rho[z] : g.rho[z];
            auto fetch_s = [&](int q, int turn) {  // lane 0: S's box q into the turn's first box
                const uint32_t bar = s_full(quarter, turn & 1);
                mbar_expect_tx(bar, kBox);
                tma_load_3d(base + box(turn & 1, 0), &maps.in, col0 + 64 * q, row0, z, bar);
                ++issued;
            };
            if (g.mode == kPoly && groups && lane == 0) {
                bulk_wait_read<1>();  // the box's last store, two groups ago
                fetch_s(0, turns);
            }
            if (!mbar_wait(acc_full(a), (i >> 1) & 1)) {
                if (lane == 0) fail();
                ok = false;
            }
            ok = __all_sync(~0u, ok && !aborted());
            tc5::fence_after();
            const uint32_t addr = tmem + ((uint32_t)(32 * quarter) << 16) + (uint32_t)(a * 256);
#pragma unroll 1
            for (int q = 0; q < groups && ok; ++q, ++turns) {
                const int k = turns & 1;
                const int col = col0 + 64 * q;
                unsigned char *const first = smem + box(k, 0), *const second = smem + box(k, 1);
                if (g.mode == kPoly) {
                    if (lane == 0 && q + 1 < groups) {
                        bulk_wait_read<0>();  // the other box's last store, the group before
                        fetch_s(q + 1, turns + 1);
                    }
                    ok = __all_sync(~0u, mbar_wait(s_full(quarter, k), (turns >> 1) & 1));
                    if (!ok) {
                        if (lane == 0) fail();
                        break;
                    }
                } else {
                    // the boxes' last stores, two groups ago, have been read
                    if (lane == 0) bulk_wait_read<1>();
                    __syncwarp();
                }
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t v[32];
                    tc5::read_32(v, addr + 64 * q + 32 * half);
                    float o[32];
#pragma unroll
                    for (int j = 0; j < 32; ++j) o[j] = alpha * __uint_as_float(v[j]);
                    // 16-byte piece p of this thread's row, under the swizzle
                    auto piece = [&](unsigned char *b, int p) {
                        return reinterpret_cast<uint4 *>(b + lane * 128 + ((4 * half + p) ^ (lane & 7)) * 16);
                    };
                    if (g.mode == kPoly) {
#pragma unroll
                        for (int p = 0; p < 4; ++p) {
                            const uint4 w = *piece(first, p);
                            const __half *h = reinterpret_cast<const __half *>(&w);
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                o[8 * p + j] = fmaf(g.beta, __half2float(h[j]), o[8 * p + j]);
                                if (col + 32 * half + 8 * p + j == row) o[8 * p + j] += g.diag;
                            }
                        }
                    }
                    if (g.mode == kFinish && g.O) {
                        const int64_t zo = z * g.strideO;
                        auto put = [&](int64_t at, float x) {
                            if (g.bf16) static_cast<__nv_bfloat16 *>(g.O)[at] = __float2bfloat16_rn(x);
                            else static_cast<__half *>(g.O)[at] = __float2half_rn(x);
                        };
                        if (row < g.M) {
#pragma unroll
                            for (int j = 0; j < 32; ++j) {
                                const int64_t c = col + 32 * half + j;
                                if (c < g.N) put(zo + (g.transposed ? c * g.ldo + row : row * g.ldo + c), o[j]);
                            }
                        }
                        continue;
                    }
                    uint32_t w[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) w[j] = pack_out(o[2 * j], o[2 * j + 1], g.mode == kFinish && g.bf16);
                    if (!(g.mode == kFinish && g.transposed)) {
#pragma unroll
                        for (int p = 0; p < 4; ++p)
                            *piece(first, p) = make_uint4(w[4 * p], w[4 * p + 1], w[4 * p + 2], w[4 * p + 3]);
                    }
                    if (mirror || (g.mode == kFinish && g.transposed)) {
                        // column j of the warp's rows as row j of the second box
                        uint16_t *b = reinterpret_cast<uint16_t *>(second) + 32 * half * 32 + lane;
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            b[(2 * j) * 32] = (uint16_t)w[j];
                            b[(2 * j + 1) * 32] = (uint16_t)(w[j] >> 16);
                        }
                    } else if (g.tail) {
#pragma unroll
                        for (int p = 0; p < 4; ++p) {
                            uint32_t lo[4];
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const __half2 hi = *reinterpret_cast<const __half2 *>(&w[4 * p + j]);
                                lo[j] = pack_half(o[8 * p + 2 * j] - __low2float(hi),
                                                  o[8 * p + 2 * j + 1] - __high2float(hi));
                            }
                            *piece(second, p) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                        }
                    }
                }
                if (g.mode == kFinish && g.O) continue;
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    if (!(g.mode == kFinish && g.transposed)) tma_store_3d(&maps.out, col, row0, z, base + box(k, 0));
                    if (mirror || (g.mode == kFinish && g.transposed))
                        tma_store_3d(&maps.second, row0, col, z, base + box(k, 1));
                    else if (g.tail) tma_store_3d(&maps.second, col, row0, z, base + box(k, 1));
                    bulk_commit();
                }
            }
            // every TMEM read of accumulator a is done: hand it back
            tc5::fence_before();
            __syncwarp();
            if (lane == 0) tc5::arrive_cluster(cluster::map(acc_empty(a), 0));
        }
        if (lane == 0) {
            bulk_wait<0>();
            // given up: loads of S in flight land before shared memory goes away
            for (; turns < issued; ++turns)
                if (!mbar_wait(s_full(quarter, turns & 1), (turns >> 1) & 1)) record_timeout(g.status);
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
        partial = (size_t)round256(batch * norm_blocks(m, n) * 8);
        rho = (size_t)round256(batch * 4);
    }
    size_t total() const { return 4 * x + 2 * s + partial + rho; }
};

// An f16 (or 16-bit) matrix per batch entry, inner x rows; ld and stride in elements.
struct Matrix {
    const void *p;
    int64_t inner, rows, ld, stride;
};

int make_map(CUtensorMap *map, const Matrix &x, int64_t batch, int box_inner, int box_rows, bool swizzled = true) {
    static const PFN_cuTensorMapEncodeTiled_v12000 encode = [] {
        void *fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) !=
                cudaSuccess || q != cudaDriverEntryPointSuccess)
            fn = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    }();
    if (!encode) return TRSM_ERR_CUDA_BASE + (int)cudaErrorNotSupported;
    const cuuint64_t dims[3] = {(cuuint64_t)x.inner, (cuuint64_t)x.rows, (cuuint64_t)batch};
    const cuuint64_t strides[2] = {(cuuint64_t)(x.ld * 2), (cuuint64_t)(x.stride * 2)};
    const cuuint32_t box[3] = {(cuuint32_t)box_inner, (cuuint32_t)box_rows, 1}, one[3] = {1, 1, 1};
    const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void *>(x.p), dims, strides, box, one,
                              CU_TENSOR_MAP_INTERLEAVE_NONE,
                              swizzled ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
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

template <int BN, bool BMN>
int launch_product(const Maps &maps, const ProductArgs &g, int sms, cudaStream_t st) {
    using R = Ring<BN>;
    cudaError_t e = cudaFuncSetAttribute(product_kernel<BN, BMN>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)R::kSmem);
    if (e != cudaSuccess) return cuda_status(e);
    const int pairs = g.tiles < sms / 2 ? g.tiles : sms / 2;
    product_kernel<BN, BMN><<<2 * pairs, 192, R::kSmem, st>>>(maps, g);
    return launch_status();
}

// The column tile of a product and its tiles, counted into g.
int plan(ProductArgs &g, int sms, int *bn) {
    // 256 x 128 tiles while 256 x 256 ones would leave CTA pairs without one
    const int64_t wide = (int64_t)((g.M + 255) / 256) * ((g.N + 255) / 256) * g.batch;
    *bn = g.N <= 128 || wide < sms / 2 ? 128 : 256;
    g.tiles_m = (g.M + kTileM - 1) / kTileM;
    g.tiles_n = (g.N + *bn - 1) / *bn;
    int64_t per = (int64_t)g.tiles_m * g.tiles_n;
    if (g.symmetric) {
        per = 0;
        for (int tm = 0; tm < g.tiles_m; ++tm) {
            const int w = kTileM / *bn * (tm + 1);
            per += w < g.tiles_n ? w : g.tiles_n;
        }
    }
    if (per * g.batch > 0x7fffffff) return -11;
    g.tiles = (int)(per * g.batch);
    return TRSM_SUCCESS;
}

template <typename T>
int convert(const OrthArgs &a, const Input &in, const Halves &x, double *partial, float *rho, cudaStream_t st) {
    const int nb = norm_blocks(a.m, a.n);
    norm_kernel<T><<<dim3(nb, (unsigned)a.batch), kNormThreads, 0, st>>>(in, partial);
    int rc = launch_status();
    if (rc) return rc;
    // about 8 blocks for each SM (each computes the scale once)
    const int64_t tiles = ((a.m + 63) / 64) * ((a.n + 63) / 64), most = (8 * 152 + a.batch - 1) / a.batch;
    const dim3 grid((unsigned)(tiles < most ? tiles : most), (unsigned)a.batch);
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
    if (rc || !a.steps) return rc;

    // The two shapes of product, and every tensor map that the steps use: each
    // buffer in each part that it plays, by turns for X.
    ProductArgs sym = {}, app = {};
    sym.M = sym.N = app.M = (int)w.r;
    app.N = (int)w.c;
    app.K = (int)w.r;
    sym.batch = app.batch = (int)a.batch;
    sym.symmetric = 1;
    int bn_sym, bn_app;
    rc = plan(sym, sms, &bn_sym);
    if (!rc) rc = plan(app, sms, &bn_app);
    if (!rc) rc = device_status_word(&sym.status);
    app.status = sym.status;
    const Matrix mS = {S, w.r, w.r, w.lds, w.r * w.lds}, mC = {C, w.r, w.r, w.lds, w.r * w.lds};
    Maps gram[2], poly, apply[2];
    auto map = [&](CUtensorMap *m, const Matrix &x, int inner, int rows, bool swizzled = true) {
        if (!rc) rc = make_map(m, x, a.batch, inner, rows, swizzled);
    };
    for (int k = 0; k < 2; ++k) {
        const Matrix mX = {xh[k], w.c, w.r, w.ldx, w.r * w.ldx}, mL = {xl[k], w.c, w.r, w.ldx, w.r * w.ldx};
        if (k && a.steps == 1) break;
        // S = X X^T
        map(&gram[k].a, mX, kBK, 128);
        map(&gram[k].b_hi, mX, kBK, bn_sym / 2);
        gram[k].b_lo = gram[k].b_hi;
        if (k == 0) {
            map(&gram[0].out, mS, 64, 32);
            map(&gram[0].second, mS, 32, 64, false);
        } else {
            gram[1].out = gram[0].out;
            gram[1].second = gram[0].second;
        }
        gram[k].in = gram[k].out;
        // X = C X, from buffer k to the other
        map(&apply[k].b_hi, mX, 64, kBK);
        map(&apply[k].b_lo, mL, 64, kBK);
        map(&apply[k ^ 1].out, mX, 64, 32);
        map(&apply[k ^ 1].second, mL, 64, 32);
    }
    map(&poly.a, mS, kBK, 128);
    map(&poly.b_hi, mS, kBK, bn_sym / 2);
    poly.b_lo = poly.b_hi;
    map(&poly.out, mC, 64, 32);
    map(&poly.second, mC, 32, 64, false);
    poly.in = gram[0].out;
    map(&apply[0].a, mC, kBK, 128);
    apply[1].a = apply[0].a;
    // the last product writes O, by TMA where its rows start on 16-byte boundaries
    Maps finish = apply[(a.steps - 1) & 1];
    const bool tall = a.m > a.n;
    uintptr_t ob = (uintptr_t)a.O;
    if (a.m > 1) ob |= (uintptr_t)(a.ldo * 2);
    if (a.batch > 1) ob |= (uintptr_t)(a.strideO * 2);
    const bool direct = ob % 16 != 0;
    if (!direct) {
        // strides of a single row or matrix are of no account, but a map needs valid ones
        const int64_t ld = a.m > 1 ? a.ldo : up8(a.n), so = a.batch > 1 ? a.strideO : up8(a.m * ld);
        const Matrix mO = {a.O, a.n, a.m, ld, so};
        map(tall ? &finish.second : &finish.out, mO, tall ? 32 : 64, tall ? 64 : 32, !tall);
        if (tall) finish.out = finish.second;
        else finish.second = finish.out;
    }

    for (int k = 0; k < a.steps && !rc; ++k) {
        const double ca = a.coef[3 * k], cb = a.coef[3 * k + 1], cc = a.coef[3 * k + 2];
        const int from = k & 1;
        const bool last = k + 1 == a.steps;
        ProductArgs g = sym;
        g.mode = kGram;
        g.K = (int)w.c;
        g.halves = 1;
        g.rho = k == 0 ? rho : nullptr;
        g.alpha = kScaleS / (kScaleX * kScaleX);
        rc = bn_sym == 256 ? launch_product<256, false>(gram[from], g, sms, st)
                           : launch_product<128, false>(gram[from], g, sms, st);
        if (rc) break;
        g.mode = kPoly;
        g.K = (int)w.r;
        g.rho = nullptr;
        g.alpha = (float)cc / kScaleS;
        g.beta = (float)cb;
        g.diag = (float)ca * kScaleS;
        rc = bn_sym == 256 ? launch_product<256, false>(poly, g, sms, st)
                           : launch_product<128, false>(poly, g, sms, st);
        if (rc) break;
        g = app;
        g.mode = last ? kFinish : kApply;
        g.halves = tail ? 2 : 1;
        g.rho = k == 0 ? rho : nullptr;
        g.alpha = last ? 1.f / (kScaleS * kScaleX) : 1.f / kScaleS;
        tail = !last && has_tail(a.coef, a.steps, k + 1, exact);
        g.tail = tail;
        if (last) {
            g.transposed = tall;
            g.bf16 = a.out_dtype == TRSM_ELEM_BF16;
            g.O = direct ? a.O : nullptr;
            g.ldo = a.ldo;
            g.strideO = a.strideO;
        }
        const Maps &m = last ? finish : apply[from];
        rc = bn_app == 256 ? launch_product<256, true>(m, g, sms, st) : launch_product<128, true>(m, g, sms, st);
    }
    return rc;
}

}  // namespace orth

size_t orth_workspace_bytes(int, int64_t m, int64_t n, int64_t batch, int64_t) {
    return orth::Layout(m, n, batch).total();
}

int orth_run(const OrthArgs &a, cudaStream_t st) { return orth::run(a, st); }

}  // namespace trsm
