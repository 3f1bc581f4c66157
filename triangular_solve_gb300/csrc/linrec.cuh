// The gated linear recurrence h_t = a_t h_{t-1} + u_t along time, forward and
// backward, and its single-token form.
//
// Mathematics.  A run of tokens acts on the state it starts from as
// h -> A h + H, A the product of its decays and H its result from zero; two
// runs in a row compose to (A2 A1, A2 H1 + H2).  So each thread reduces its
// few tokens to (A, H), the pairs of the runs before it are composed to its
// starting state, and it walks its tokens again from there.  The backward
// pass is the same recurrence over the tokens in reverse: with
// D_t = dh_t + c_{t+1} the full gradient of h_t and c_t = a_t D_t what it
// passes back,
//     c_t = a_t c_{t+1} + a_t dh_t,
// which needs no decay but the token's own.
//
// Bound: memory.  The kernel reads every input and writes every output once
// (forward 3 elements a token and channel, backward 5, or 6 in the sigmoid
// form) and does a few operations on each.
//
// Layout.  A CTA of 256 threads takes `VEC` channels per lane and `LANES`
// lanes side by side (128 bytes of a row with 16-byte vectors), and 256 /
// LANES time slots of ROWS consecutive tokens each.  Every thread copies its
// own tokens into shared memory ahead of time (cp.async, so no registers and
// no block barrier are spent on it) and walks them twice from there; they are
// read from memory once.  A cluster of 1..8 CTAs takes consecutive stretches
// of the same channels and sequence and steps along the sequence; each step
// composes the warps' pairs in shared memory and the CTAs' pairs through
// distributed shared memory.  There is no flag or wait in global memory, and
// the order of every sum is fixed by the shapes, so results do not vary from
// run to run.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "cluster.cuh"
#include "common.cuh"
#include "linrec.h"
#include "trsm_model.h"

namespace trsm {
namespace linrec {

constexpr int kThreads = 256;
constexpr int kMaxCluster = 8;

template <typename T> __device__ __forceinline__ float to_f32(T v);
template <> __device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }
template <> __device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// VEC elements of T as one access (VEC * sizeof(T) is 16, or VEC = 1).
template <typename T, int VEC> struct alignas(VEC * sizeof(T)) Pack {
    T v[VEC];
};
template <typename T, int VEC>
__device__ __forceinline__ Pack<T, VEC> load_pack(const T *p) {
    return *reinterpret_cast<const Pack<T, VEC> *>(p);
}
template <typename T, int VEC>
__device__ __forceinline__ void store_pack(T *p, const Pack<T, VEC> &r) {
    *reinterpret_cast<Pack<T, VEC> *>(p) = r;
}

// 2^x, 2^-22 relative, and 1 / x for x in [1, 2^127), rounded to within a unit
// in the last place: the hardware's approximation after one Newton step.
__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float recip_newton(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return fmaf(r, fmaf(-x, r, 1.f), r);
}
__device__ __forceinline__ float min_nan(float x, float y) {  // NaN if either is
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
    return r;
}

// a and 1 - a of a gate value.  Gates of 16 bits take the hardware's
// exponential, which is far closer than the gate's own rounding.  The
// reciprocal is refined: an error of one sign in every token's decay adds up
// over a long memory (7e-6 of dh0 over 4096 tokens with the bare one).
//
// sigmoid: e = exp(-g) held below 2^126, so that neither 1 + e nor e a
// overflows; a is then 2^-126 where it would be smaller still.
template <typename T, int FORM>
__device__ __forceinline__ void open_gate(T gate, float &a, float &rest) {
    constexpr float kLog2e = 1.44269504f;
    const float g = to_f32<T>(gate);
    constexpr bool kFull = sizeof(T) == 4;
    if constexpr (FORM == TRSM_GATE_DECAY) {
        a = g;
    } else if constexpr (FORM == TRSM_GATE_LOG) {
        a = kFull ? expf(g) : exp2_fast(g * kLog2e);
    } else {
        const float e = kFull ? min_nan(expf(-g), 0x1p126f) : exp2_fast(min_nan(g * -kLog2e, 126.f));
        a = recip_newton(1.f + e);
        rest = e * a;
    }
}

// The state A h + H; a run that starts from zero is H even where the product
// of its decays has overflowed.
__device__ __forceinline__ float apply(float A, float H, float h) { return h == 0.f ? H : fmaf(A, h, H); }

// First row (in the tensors) and length of sequence b; packed sequences have
// their offsets held inside the list.
struct Sequence {
    int64_t b, row0;
    int len;
};
__device__ __forceinline__ Sequence sequence(const LinrecArgs &g, int64_t b) {
    const int T = (int)g.T;
    if (!g.offsets) return {b, 0, T};
    const int lo = min(max(g.offsets[b], 0), T), hi = min(max(g.offsets[b + 1], 0), T);
    return {0, lo, hi > lo ? hi - lo : 0};
}

// A sequence of one tensor as the walk meets it: position p at
// at + p * step (the backward pass walks from the last row up).
template <typename T> struct Walk {
    T *at;
    int64_t step;
};
template <typename T, bool BWD>
__device__ __forceinline__ Walk<T> walk(const LinrecRows &r, const Sequence &s, int64_t d) {
    T *first = static_cast<T *>(const_cast<void *>(r.p)) + s.b * r.sb + s.row0 * r.st + d;
    if constexpr (BWD) return {first + (int64_t)(s.len - 1) * r.st, -r.st};
    return {first, r.st};
}

// Shapes and shared memory of one instantiation.
template <typename T, int FORM, bool BWD, int VEC, int LANES, int ROWS> struct Shape {
    static constexpr int kChannels = LANES * VEC;               // channels of a CTA
    static constexpr int kStretch = kThreads / LANES * ROWS;    // tokens of a CTA in one step
    static __device__ __forceinline__ int channel_at(int i) {   // see slot_A
        constexpr int q = VEC < 4 ? VEC : 4;
        return (i / q) % LANES * VEC + i / (q * LANES) * q + i % q;
    }
    static constexpr bool kSigmoid = FORM == TRSM_GATE_SIGMOID;
    // two buffers each of the gate and x (backward: dh), and in the backward
    // pass one each of h and (sigmoid) x
    static constexpr int kBuffers = 4 + (BWD ? 1 + (kSigmoid ? 1 : 0) : 0);
    static constexpr int kBufferElems = kStretch * kChannels;
    static constexpr size_t kSmem = (size_t)kBuffers * kBufferElems * sizeof(T);
};

template <typename T, int FORM, bool BWD, int VEC, int LANES, int ROWS>
__global__ void __launch_bounds__(kThreads, 2) scan_kernel(const __grid_constant__ LinrecArgs g, const int groups) {
    using S = Shape<T, FORM, BWD, VEC, LANES, ROWS>;
    constexpr int kChannels = S::kChannels, kStretch = S::kStretch;
    constexpr int kSlots = kThreads / LANES, kParts = kThreads / kChannels, kPartSlots = kSlots / kParts;
    constexpr bool kSigmoid = S::kSigmoid;
    // The forward sigmoid keeps a and u of its tokens between the two walks
    // (their exponential and reciprocal cost more than the registers); the
    // others open the gate again.
    constexpr bool kKeep = kSigmoid && !BWD;
    using P = Pack<T, VEC>;

    extern __shared__ __align__(16) unsigned char staged[];
    // Channels in shared memory stand in the order of the threads' 16-byte
    // accesses: place i holds channel channel_at(i) of the CTA.
    __shared__ __align__(16) float slot_A[kSlots][kChannels], slot_H[kSlots][kChannels];  // pair of each slot
    __shared__ float2 part_pair[kParts][kChannels];           // of each part of the slots
    __shared__ float2 cta_pair[2][kMaxCluster][kChannels];    // of each CTA, written by all of them

    const int tid = threadIdx.x, col = tid % LANES, slot = tid / LANES;
    // Between the walks thread (place, part) composes the slots of one part.
    const int place = tid % kChannels, part = tid / kChannels;
    const int csize = (int)cluster::size(), crank = (int)cluster::rank();
    const int64_t unit = (int64_t)(blockIdx.x / csize);
    const int64_t b = unit / groups;
    const int64_t c0 = (unit % groups) * kChannels;
    const int64_t d = c0 + col * VEC;
    const bool live = d < g.D;
    const Sequence seq = sequence(g, b);
    const int len = live ? seq.len : 0;  // tokens this thread may touch

    // each of them carries the state of its channel from step to step
    const int64_t dc = c0 + S::channel_at(place);
    float carry = 0.f;
    if (dc < g.D) {
        if constexpr (BWD) {
            if (g.dh_last) carry = g.dh_last[b * g.D + dc];
        } else {
            if (g.h0) carry = g.h0[b * g.h0_stride + dc];
        }
    }
    if (csize > 1) cluster::sync();  // every CTA has started before any writes into its shared memory

    // this thread's place in staged buffer i, row r: mine(i)[r * kChannels]
    auto mine = [&](int i) {
        return reinterpret_cast<T *>(staged) + i * S::kBufferElems + slot * ROWS * kChannels + col * VEC;
    };
    // Copies positions base .. base + ROWS - 1 (those below `end`) into buffer i.
    auto stage = [&](const Walk<const T> &w, int base, int end, int i) {
        const T *p = w.at + base * w.step;
        T *s = mine(i);
        if constexpr (VEC * sizeof(T) == 16) {
#pragma unroll
            for (int r = 0; r < ROWS; ++r)
                if (base + r < end) cp_async<16>(s + r * kChannels, p + r * w.step);
        } else {
            P v[ROWS];
#pragma unroll
            for (int r = 0; r < ROWS; ++r)
                if (base + r < end) v[r] = load_pack<T, VEC>(p + r * w.step);
#pragma unroll
            for (int r = 0; r < ROWS; ++r)
                if (base + r < end) store_pack<T, VEC>(s + r * kChannels, v[r]);
        }
    };
    const Walk<const T> wg = walk<const T, BWD>(g.gate, seq, d);
    const Walk<const T> wu = walk<const T, BWD>(BWD ? g.dh : g.x, seq, d);

    // T is at most 2^31 - 2^16: positions past the end by two steps fit an int
    const int step = csize * kStretch;
    const int steps = (seq.len + step - 1) / step;
    int base = crank * kStretch + slot * ROWS;  // this thread's first position
    stage(wg, base, len, 0);
    stage(wu, base, len, 1);
    cp_async_commit();
    int parity = 0;
    for (int i = 0; i < steps; ++i, base += step, parity ^= 1) {
        const T *pg = mine(2 * parity), *pu = mine(2 * parity + 1);
        if constexpr (BWD) {
            // for the second walk: the row before each token (the last
            // position is row 0, whose state before is h0), and x
            const Walk<const T> wh = walk<const T, BWD>(g.h, seq, d);
            stage({wh.at + wh.step, wh.step}, base, len - 1, 4);
            if constexpr (kSigmoid) stage(walk<const T, BWD>(g.x, seq, d), base, len, 5);
            cp_async_commit();
        }
        stage(wg, base + step, len, 2 * (parity ^ 1));
        stage(wu, base + step, len, 2 * (parity ^ 1) + 1);
        cp_async_commit();
        cp_async_wait<BWD ? 2 : 1>();  // this step's gate and x (dh)

        // first walk: (A, H) of the slot
        float a[kKeep ? ROWS : 1][VEC], u[kKeep ? ROWS : 1][VEC];
        alignas(16) float A[VEC], H[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            A[v] = 1.f;
            H[v] = 0.f;
        }
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            if (base + r < len) {
                const P q = load_pack<T, VEC>(pg + r * kChannels), e = load_pack<T, VEC>(pu + r * kChannels);
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
                    float at, ut = to_f32<T>(e.v[v]), rest;
                    open_gate<T, FORM>(q.v[v], at, rest);
                    if constexpr (kSigmoid && !BWD) ut *= rest;
                    H[v] = BWD ? at * (H[v] + ut) : fmaf(at, H[v], ut);
                    A[v] *= at;
                    if constexpr (kKeep) {
                        a[r][v] = at;
                        u[r][v] = ut;
                    }
                }
            }
        }

        // (A, H) of the slots -> of the parts -> of the CTA -> of the CTAs
        // before; then back down to the state each slot starts from
        constexpr int kQuad = VEC < 4 ? VEC : 4;
#pragma unroll
        for (int v = 0; v < VEC; v += kQuad) {
            const int at = v * LANES + col * kQuad;
            store_pack<float, kQuad>(&slot_A[slot][at], *reinterpret_cast<const Pack<float, kQuad> *>(&A[v]));
            store_pack<float, kQuad>(&slot_H[slot][at], *reinterpret_cast<const Pack<float, kQuad> *>(&H[v]));
        }
        __syncthreads();
        float sa[kPartSlots], sh[kPartSlots];
        {
            float pa = 1.f, ph = 0.f;
#pragma unroll
            for (int k = 0; k < kPartSlots; ++k) {
                sa[k] = slot_A[part * kPartSlots + k][place];
                sh[k] = slot_H[part * kPartSlots + k][place];
                ph = apply(sa[k], sh[k], ph);
                pa *= sa[k];
            }
            part_pair[part][place] = make_float2(pa, ph);
        }
        __syncthreads();
        if (csize > 1) {
            if (part == 0) {
                float ca = 1.f, ch = 0.f;
#pragma unroll
                for (int k = 0; k < kParts; ++k) {
                    const float2 q = part_pair[k][place];
                    ch = apply(q.x, q.y, ch);
                    ca *= q.x;
                }
                const uint32_t at = smem_u32(&cta_pair[parity][crank][place]);
                for (int k = 0; k < csize; ++k) cluster::store_f32x2(cluster::map(at, k), ca, ch);
            }
            // Two buffers by turns: a CTA writes a buffer again only after the
            // next step's barrier, which all pass after reading it.
            cluster::sync();
        }
        float state = carry;
        if (csize > 1) {
            for (int k = 0; k < csize; ++k) {
                if (k == crank) state = carry;
                const float2 q = cta_pair[parity][k][place];
                carry = apply(q.x, q.y, carry);
            }
        }
#pragma unroll
        for (int k = 0; k < kParts; ++k) {
            const float2 q = part_pair[k][place];
            if (k < part) state = apply(q.x, q.y, state);
            if (csize == 1) carry = apply(q.x, q.y, carry);
        }
#pragma unroll
        for (int k = 0; k < kPartSlots; ++k) {
            slot_H[part * kPartSlots + k][place] = state;
            state = apply(sa[k], sh[k], state);
        }
        if constexpr (BWD) cp_async_wait<1>();  // h and x
        __syncthreads();

        // second walk, from the slot's starting state
        alignas(16) float h[VEC];
#pragma unroll
        for (int v = 0; v < VEC; v += kQuad)
            *reinterpret_cast<Pack<float, kQuad> *>(&h[v]) =
                load_pack<float, kQuad>(&slot_H[slot][v * LANES + col * kQuad]);
        if constexpr (!BWD) {
            const Walk<T> wo = walk<T, BWD>(g.h, seq, d);
            T *out = wo.at + base * wo.step;
#pragma unroll
            for (int r = 0; r < ROWS; ++r) {
                if (base + r < len) {
                    P o, q, e;
                    if constexpr (!kKeep) {
                        q = load_pack<T, VEC>(pg + r * kChannels);
                        e = load_pack<T, VEC>(pu + r * kChannels);
                    }
#pragma unroll
                    for (int v = 0; v < VEC; ++v) {
                        float at, ut, rest;
                        if constexpr (kKeep) {
                            at = a[r][v];
                            ut = u[r][v];
                        } else {
                            open_gate<T, FORM>(q.v[v], at, rest);
                            ut = to_f32<T>(e.v[v]);
                        }
                        h[v] = fmaf(at, h[v], ut);
                        o.v[v] = from_f32<T>(h[v]);
                    }
                    store_pack<T, VEC>(out + r * wo.step, o);
                }
            }
        } else {
            const Walk<T> wo = walk<T, BWD>(g.dgate, seq, d), wx = walk<T, BWD>(g.dx, seq, d);
            T *og = wo.at + base * wo.step, *ox = wx.at + base * wx.step;
            const T *ph = mine(4), *px = mine(S::kBuffers - 1);
#pragma unroll
            for (int r = 0; r < ROWS; ++r) {
                if (base + r < len) {
                    const P q = load_pack<T, VEC>(pg + r * kChannels), e = load_pack<T, VEC>(pu + r * kChannels);
                    P before, in, o0, o1;
                    const bool start = base + r + 1 == len;
                    if (!start) before = load_pack<T, VEC>(ph + r * kChannels);
                    if constexpr (kSigmoid) in = load_pack<T, VEC>(px + r * kChannels);
#pragma unroll
                    for (int v = 0; v < VEC; ++v) {
                        float at, rest;
                        open_gate<T, FORM>(q.v[v], at, rest);
                        const float prev = !start ? to_f32<T>(before.v[v])
                                                  : g.h0 ? g.h0[b * g.h0_stride + d + v] : 0.f;
                        const float full = to_f32<T>(e.v[v]) + h[v];
                        h[v] = at * full;
                        if constexpr (FORM == TRSM_GATE_DECAY) {
                            o0.v[v] = from_f32<T>(full * prev);
                            o1.v[v] = from_f32<T>(full);
                        } else if constexpr (FORM == TRSM_GATE_LOG) {
                            o0.v[v] = from_f32<T>(h[v] * prev);
                            o1.v[v] = from_f32<T>(full);
                        } else {
                            o0.v[v] = from_f32<T>((prev - to_f32<T>(in.v[v])) * (h[v] * rest));
                            o1.v[v] = from_f32<T>(full * rest);
                        }
                    }
                    store_pack<T, VEC>(og + r * wo.step, o0);
                    store_pack<T, VEC>(ox + r * wx.step, o1);
                }
            }
        }
    }
    if (g.last && crank == 0 && part == 0 && dc < g.D) g.last[b * g.D + dc] = carry;
}

// One token per row: y = next[s] = a state[s] + u.
template <typename T, int FORM, int VEC>
__global__ void __launch_bounds__(128) step_kernel(const __grid_constant__ LinrecStepArgs g) {
    using P = Pack<T, VEC>;
    using S = Pack<float, VEC>;
    const int64_t d = ((int64_t)blockIdx.x * 128 + threadIdx.x) * VEC;
    if (d >= g.D) return;
    for (int64_t i = blockIdx.y; i < g.batch; i += gridDim.y) {
        const int64_t s = g.slots ? (int64_t)g.slots[i] : i;
        T *y = static_cast<T *>(g.y) + i * g.y_stride + d;
        P o;
        if (s < 0 || s >= g.nslots) {
#pragma unroll
            for (int v = 0; v < VEC; ++v) o.v[v] = from_f32<T>(0.f);
            store_pack<T, VEC>(y, o);
            continue;
        }
        const P pg = load_pack<T, VEC>(static_cast<const T *>(g.gate) + i * g.gate_stride + d);
        const P px = load_pack<T, VEC>(static_cast<const T *>(g.x) + i * g.x_stride + d);
        // plain accesses: next may be state
        S h = *reinterpret_cast<const S *>(g.state + s * g.state_stride + d);
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            float a, rest, u = to_f32<T>(px.v[v]);
            open_gate<T, FORM>(pg.v[v], a, rest);
            if constexpr (FORM == TRSM_GATE_SIGMOID) u *= rest;
            h.v[v] = fmaf(a, h.v[v], u);
            o.v[v] = from_f32<T>(h.v[v]);
        }
        *reinterpret_cast<S *>(g.next + s * g.next_stride + d) = h;
        store_pack<T, VEC>(y, o);
    }
}

// ------------------------------------------------------------------ launch
inline int sm_count(int *out) {
    static int sms = 0;  // of the first device used; all are alike here
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

// Whether every row of the tensor starts on a 16-byte boundary.
inline bool rows_vec(const LinrecArgs &a, const LinrecRows &r, int64_t elem) {
    uintptr_t bits = (uintptr_t)r.p;
    if (a.batch > 1 && !a.offsets) bits |= (uintptr_t)(r.sb * elem);
    if (a.T > 1) bits |= (uintptr_t)(r.st * elem);
    return bits % 16 == 0;
}

template <typename T, int FORM, bool BWD, int VEC, int LANES, int ROWS>
int launch_scan(const LinrecArgs &a, cudaStream_t st) {
    using S = Shape<T, FORM, BWD, VEC, LANES, ROWS>;
    int sms = 0;
    const int rc = sm_count(&sms);
    if (rc) return rc;
    const int64_t groups = (a.D + LANES * VEC - 1) / (LANES * VEC);
    const int64_t units = a.batch * groups;
    // CTAs along a sequence: until the GPU is full, but no more than it has stretches
    const int64_t len = a.offsets ? (a.T + a.batch - 1) / a.batch : a.T;
    int cs = 1;
    while (cs < kMaxCluster && units * cs < 4 * sms && cs * S::kStretch < len) cs *= 2;
    if (units * cs > 0x7fffffff) return -3;
    auto *kernel = scan_kernel<T, FORM, BWD, VEC, LANES, ROWS>;
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::kSmem);
    if (e != cudaSuccess) return cuda_status(e);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(units * cs));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = S::kSmem;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = cs;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cuda_status(cudaLaunchKernelEx(&cfg, kernel, a, (int)groups));
}

template <typename T, int FORM, bool BWD>
int run(const LinrecArgs &a, cudaStream_t st) {
    constexpr int kVec = 16 / sizeof(T);
    bool vec = a.D % kVec == 0 && rows_vec(a, a.gate, sizeof(T)) && rows_vec(a, a.h, sizeof(T));
    if (!BWD || FORM == TRSM_GATE_SIGMOID) vec = vec && rows_vec(a, a.x, sizeof(T));
    if (BWD) vec = vec && rows_vec(a, a.dh, sizeof(T)) && rows_vec(a, a.dgate, sizeof(T)) && rows_vec(a, a.dx, sizeof(T));
    if (vec) return launch_scan<T, FORM, BWD, kVec, 8, 32 / kVec>(a, st);
    return launch_scan<T, FORM, BWD, 1, 32, 8>(a, st);
}

template <typename T>
int run_form(const LinrecArgs &a, int form, bool backward, cudaStream_t st) {
    switch (form) {
        case TRSM_GATE_DECAY:
            return backward ? run<T, TRSM_GATE_DECAY, true>(a, st) : run<T, TRSM_GATE_DECAY, false>(a, st);
        case TRSM_GATE_LOG:
            return backward ? run<T, TRSM_GATE_LOG, true>(a, st) : run<T, TRSM_GATE_LOG, false>(a, st);
        default:
            return backward ? run<T, TRSM_GATE_SIGMOID, true>(a, st) : run<T, TRSM_GATE_SIGMOID, false>(a, st);
    }
}

template <typename T, int FORM, int VEC>
int launch_step(const LinrecStepArgs &a, cudaStream_t st) {
    const int64_t bx = (a.D + 128 * VEC - 1) / (128 * VEC);
    if (bx > 0x7fffffff) return -4;
    const dim3 grid((unsigned)bx, (unsigned)(a.batch < 65535 ? a.batch : 65535));
    step_kernel<T, FORM, VEC><<<grid, 128, 0, st>>>(a);
    return launch_status();
}

template <typename T, int FORM>
int step_vec(const LinrecStepArgs &a, cudaStream_t st) {
    constexpr int kVec = 16 / sizeof(T);
    const bool vec = a.D % kVec == 0 &&
                     ((uintptr_t)a.gate | (uintptr_t)a.x | (uintptr_t)a.y | (uintptr_t)a.state | (uintptr_t)a.next |
                      (uintptr_t)((a.gate_stride | a.x_stride | a.y_stride) * (int64_t)sizeof(T))) % 16 == 0 &&
                     ((a.state_stride | a.next_stride) * 4) % (4 * kVec) == 0 &&
                     ((uintptr_t)a.state | (uintptr_t)a.next) % (4 * kVec) == 0;
    return vec ? launch_step<T, FORM, kVec>(a, st) : launch_step<T, FORM, 1>(a, st);
}

template <typename T>
int step_form(const LinrecStepArgs &a, int form, cudaStream_t st) {
    switch (form) {
        case TRSM_GATE_DECAY: return step_vec<T, TRSM_GATE_DECAY>(a, st);
        case TRSM_GATE_LOG: return step_vec<T, TRSM_GATE_LOG>(a, st);
        default: return step_vec<T, TRSM_GATE_SIGMOID>(a, st);
    }
}

}  // namespace linrec
}  // namespace trsm
