// The joint between two halves of a block, forward and backward: the first half's
// output is normed (post), gated and added to the residual stream, and the
// stream is normed for the second half.
//
//   u = N(o) pw + pb  (or o)      s = alpha r + gate u      n = N(s) w + b
//   N(v) = (v - mean v) / sqrt(mean (v - mean v)^2 + eps), or without the means (RMS)
//
//   z = N(s), oz = N(o), h = dn w
//   D = ds + rstd (h - [mean h] - z mean(h z))        dr = alpha D
//   q = gate D, p = q pw, do = orstd (p - [mean p] - oz mean(p oz))   (or do = q)
//   dw = sum dn z   db = sum dn   dpw = sum q oz   dpb = sum q
//   dgate = sum D u, over the rows (a gate per channel) or the columns (per token)
// [..]: layer norm only.  A gate per channel leaves the sum over the rows: dpw =
// gate A, dpb = gate C, dgate = pw A + pb C with A = sum D oz, C = sum D, so two
// column sums serve all three.
//
// Statistics, sums and everything between are FP32; s and n are rounded once (n
// comes from the unrounded s, which the backward takes from o and r again).  The
// variance is taken around the mean, never as E[v^2] - m^2.
//
// Bound by DRAM: forward 4, backward 6 rows of H elements.  Persistent blocks of
// groups; a group of threads takes a row, eight columns a thread (the backward's
// column sums stay in tensor memory for the life of the block).  The rows to come
// are copied ahead by cp.async into a ring of shared memory: rows that lie on
// 16-byte boundaries by the thread that will read them, others as the whole
// 16-byte pieces around them (kVec false), read element by element after the
// group's barrier.  A stage is filled again as soon as its row is in registers.
// The parameters stay in shared memory in FP32, as far as they fit beside two
// stages.  Arithmetic is on pairs (fma.f32x2): at 8192 x 7168 the issue slots,
// not DRAM, bound the first form of it.  Rows of more than 7168 columns are read
// again for every pass.  FP32 rows take fewer groups than the threads allow where two
// stages of all would not fit.
//
// Measured, bf16 (the bytes at the copy rate): 8192 x 7168, RMS, post norm, a gate per
// token 81 + 143 us (70 + 106), without post norm and gate 82 + 118 us; layer norms
// with everything 122 + 181 us; 8192 x 4096, RMS with post norm 46 + 77 us (40 + 60);
// 4096 x 2048, RMS 12.4 + 24 us (10 + 15).  What is left in the backward is the
// latency of two sums a row with one row at a time on an SM (without them 26 us less)
// and the column sums (6 us).  Rows off the 16-byte boundaries take two to five times the
// instructions a column: 8192 x 7161 150 + 235 us.  FP32: 8192 x 7168 161 + 345 us (141 +
// 211), backward of 4096 x 1024 25 (15), 1000 x 3584 29-32 (13), 8192 x 128 15-17 (4).
//
// Column sums: one row of partial sums a block, joined in a fixed order by a second
// kernel, or (few rows) by the blocks themselves as one cluster: deterministic, no atomics.
#pragma once

#include <cuda_fp16.h>

#include "moe_internal.h"
#include "ptx.cuh"
#include "smem_limit.h"

namespace moe {

namespace {

constexpr int kRnCols = 8;  // columns of a thread
constexpr int kRnMaxH = 896 * kRnCols;
constexpr int kRnLongThreads = 1024;
// Of a group's sums: two turns of 32 warps' float4, or (many warps) the parts of up to
// kRnSums sums and, behind all of them, the results.
constexpr int kRnSums = 3, kRnResults = kRnSums * 32 * 4;
constexpr int kRnRedBytes = kRnResults * 4 + 16;
constexpr int kRnFewWarps = 8;
constexpr int kRnSmem = 227 * 1024 - 64;  // dynamic, beside a few static bytes

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// ---------------------------------------------------------- pairs of FP32
struct F2 {
    uint64_t v;
};
__device__ __forceinline__ F2 f2(float a, float b) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ F2 f2(float a) { return f2(a, a); }
__device__ __forceinline__ float2 unpack(F2 a) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
    return r;
}
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 operator+(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ float both(F2 a) {
    const float2 f = unpack(a);
    return f.x + f.y;
}
// A thread's E columns.
template <int E>
struct Cols {
    F2 p[E / 2];
};
template <int E>
__device__ __forceinline__ float sum_of(const Cols<E>& c) {
    F2 s = c.p[0], u = c.p[1];
#pragma unroll
    for (int i = 2; i < E / 2; i += 2) s = s + c.p[i], u = u + c.p[i + 1];
    return both(s + u);
}
template <int E>
__device__ __forceinline__ float dot(const Cols<E>& a, const Cols<E>& b) {
    F2 s = a.p[0] * b.p[0], u = a.p[1] * b.p[1];
#pragma unroll
    for (int i = 2; i < E / 2; i += 2) s = fma2(a.p[i], b.p[i], s), u = fma2(a.p[i + 1], b.p[i + 1], u);
    return both(s + u);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int s = 16; s >= 1; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
    return v;
}

// A parameter of type FP32 or T.
template <typename T>
struct Param {
    const void* p;
    int f32;
    __device__ __forceinline__ float at(int c) const {
        return f32 ? __ldg(static_cast<const float*>(p) + c) : to_f(static_cast<const T*>(p)[c]);
    }
};

// A group of a block: nt threads that take one row at a time.
struct Group {
    int id, t, nt, warps, warp;  // warp: within the group
    float4* red;                 // two turns of a value a warp
    int turn;
    __device__ __forceinline__ void sync() const {
        if (warps == 1)
            __syncwarp();
        else
            asm volatile("bar.sync %0, %1;" ::"r"(1 + id), "r"(nt) : "memory");
    }
    // Sums over the group, in the same order in every thread.  Shuffles and shared
    // memory take their turns in one pipe: with many warps, each finishing the sum for
    // itself, that pipe is what a row costs.  Then each warp leaves four parts, one
    // warp adds them, and the others read the result.
    template <int N>
    __device__ __forceinline__ void sum(float (&v)[N]) {
        const int lane = threadIdx.x & 31;
        if (warps <= kRnFewWarps) {
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = warp_sum(v[i]);
            if (warps == 1) return;
            float* r = reinterpret_cast<float*>(red + turn * 32);
            turn ^= 1;
            if (lane == 0) {
#pragma unroll
                for (int i = 0; i < N; ++i) r[4 * warp + i] = v[i];
            }
            sync();
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = lane < warps ? r[4 * lane + i] : 0.0f;
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = warp_sum(v[i]);
            return;
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
#pragma unroll
            for (int k = 16; k >= 4; k >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], k);
        }
        // Parts [N][warps][4].  The results' place is the same for every N: a warp may still
        // read them when another writes the next call's parts, and until that call's
        // first barrier, which both pass, only those are written.
        static_assert(N <= kRnSums, "parts");
        float* r = reinterpret_cast<float*>(red);
        if (lane < 4) {
#pragma unroll
            for (int i = 0; i < N; ++i) r[(i * 32 + warp) * 4 + lane] = v[i];
        }
        sync();
        if (warp < N) {
            const float4 f = lane < warps ? reinterpret_cast<const float4*>(r)[warp * 32 + lane] : make_float4(0, 0, 0, 0);
            const float total = warp_sum((f.x + f.y) + (f.z + f.w));
            if (lane == 0) r[kRnResults + warp] = total;
        }
        sync();
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = r[kRnResults + i];
    }
    __device__ __forceinline__ float sum(float a) {
        float v[1] = {a};
        sum(v);
        return v[0];
    }
};

struct RnShape {
    long long rows;
    int H, rms, gate, w_f32;
    float alpha, eps, inv;  // inv: 1 / H
    int groups, nt, row_bytes, stages, in_smem;  // in_smem: parameters held in shared memory
};

// Where a thread's E columns are: vectors of 16 bytes nt apart, or elements nt
// apart (kVec false).
template <typename T, bool kVec, int E>
struct Place {
    static constexpr int V = kVec ? 16 / (int)sizeof(T) : 1, NV = E / V;
    int H, t, nt;
    __device__ __forceinline__ int col(int j) const { return (t + j * nt) * V; }
    __device__ __forceinline__ bool in(int j) const { return col(j) < H; }
    // A parameter's place in shared memory [E nt]: two-byte vectors take it as two
    // planes of four columns a vector, so that a warp's reads do not collide.
    __device__ __forceinline__ int at(int c) const {
        return V == 8 ? ((c >> 2) & 1) * 4 * nt * NV + (c >> 3) * 4 + (c & 3) : c;
    }
    __device__ __forceinline__ Cols<E> load_smem(const float* s) const {
        Cols<E> r;
        if constexpr (V == 1) {
#pragma unroll
            for (int i = 0; i < E / 2; ++i) r.p[i] = f2(s[t + 2 * i * nt], s[t + (2 * i + 1) * nt]);
        } else {
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int k = 0; k < V / 4; ++k) {
                    const ulonglong2 u = *reinterpret_cast<const ulonglong2*>(s + 4 * (t + j * nt) + k * 4 * nt * NV);
                    r.p[j * V / 2 + 2 * k].v = u.x;
                    r.p[j * V / 2 + 2 * k + 1].v = u.y;
                }
        }
        return r;
    }
    __device__ __forceinline__ static Cols<E> pairs(const float (&f)[E]) {
        Cols<E> r;
#pragma unroll
        for (int i = 0; i < E / 2; ++i) r.p[i] = f2(f[2 * i], f[2 * i + 1]);
        return r;
    }
    __device__ __forceinline__ static void singles(const Cols<E>& v, float (&f)[E]) {
#pragma unroll
        for (int i = 0; i < E / 2; ++i) {
            const float2 u = unpack(v.p[i]);
            f[2 * i] = u.x, f[2 * i + 1] = u.y;
        }
    }
    // From global memory: zeros past the row.
    __device__ __forceinline__ Cols<E> load_global(const Param<T>& w) const {
        float f[E];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = col(j);
            if (c >= H) {
#pragma unroll
                for (int i = 0; i < V; ++i) f[j * V + i] = 0.0f;
            } else if constexpr (V == 1) {
                f[j] = w.at(c);
            } else if (w.f32) {
#pragma unroll
                for (int i = 0; i < V / 4; ++i) {
                    const float4 u = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(w.p) + c) + i);
                    f[j * V + 4 * i] = u.x, f[j * V + 4 * i + 1] = u.y;
                    f[j * V + 4 * i + 2] = u.z, f[j * V + 4 * i + 3] = u.w;
                }
            } else {
                const uint4 u = __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(w.p) + c));
                const T* e = reinterpret_cast<const T*>(&u);
#pragma unroll
                for (int i = 0; i < V; ++i) f[j * V + i] = to_f(e[i]);
            }
        }
        return pairs(f);
    }
    __device__ __forceinline__ void store(T* row, const Cols<E>& v) const {
        float f[E];
        singles(v, f);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = col(j);
            if (c >= H) continue;
            if constexpr (V == 1) {
                row[c] = from_f<T>(f[j]);
            } else {
                uint4 u;
                T* e = reinterpret_cast<T*>(&u);
#pragma unroll
                for (int i = 0; i < V; ++i) e[i] = from_f<T>(f[j * V + i]);
                __stcs(reinterpret_cast<uint4*>(row + c), u);
            }
        }
    }
};

// The parameters of a kernel: all of them in shared memory (kHeld), or the first
// ones and the rest through L1.
template <typename T, bool kVec, int E, bool kHeld>
struct Params {
    const Place<T, kVec, E>& at;
    const float* smem;
    int in_smem, f32;
    __device__ __forceinline__ Cols<E> operator()(int slot, const void* p) const {
        if (kHeld || slot < in_smem) return at.load_smem(smem + slot * E * at.nt);
        return at.load_global(Param<T>{p, f32});
    }
    // Every thread of the block: parameter `slot`, zeros past the row.
    __device__ __forceinline__ void fill(float* s, int slot, const void* p) const {
        if (slot >= in_smem || !p) return;
        const Param<T> w = {p, f32};
        for (int c = threadIdx.x; c < E * at.nt; c += blockDim.x) s[slot * E * at.nt + at.at(c)] = c < at.H ? w.at(c) : 0.0f;
    }
};

// A thread's columns as they were stored, two bytes an element where they are: what
// is kept from one pass over a row to the next.
template <typename T, int E>
struct RawHalves {
    uint32_t w[E / 2];
};
template <typename T, int E>
struct RawOf {
    using type = RawHalves<T, E>;
};
template <int E>
struct RawOf<float, E> {
    using type = Cols<E>;
};
template <typename T, int E>
using Raw = typename RawOf<T, E>::type;
template <int E>
__device__ __forceinline__ Cols<E> widen(const Cols<E>& v) {
    return v;
}
template <typename T, int E>
__device__ __forceinline__ Cols<E> widen(const RawHalves<T, E>& v) {
    Cols<E> r;
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
        if constexpr (__is_same(T, __nv_bfloat16)) {
            r.p[i] = f2(__uint_as_float(v.w[i] << 16), __uint_as_float(v.w[i] & 0xffff0000u));
        } else {
            const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&v.w[i]));
            r.p[i] = f2(h.x, h.y);
        }
    }
    return r;
}

// The ring of one group: stages of kTensors rows.
template <typename T, bool kVec, int E, int kTensors>
struct Ring {
    using P = Place<T, kVec, E>;
    static constexpr int V = P::V, NV = P::NV;
    const P& at;
    uint8_t* base;  // the group's
    int row_bytes;
    __device__ __forceinline__ uint8_t* slot(int stage, int k) const { return base + (stage * kTensors + k) * row_bytes; }
    __device__ __forceinline__ static int shift(const T* row) { return kVec ? 0 : (int)(reinterpret_cast<uintptr_t>(row) & 15); }
    // Vectors past the row are never copied: their slots hold zeros from the start.
    __device__ __forceinline__ void clear(int stages) const {
        if constexpr (kVec) {
#pragma unroll
            for (int j = 0; j < NV; ++j)
                if (!at.in(j))
                    for (int k = 0; k < stages * kTensors; ++k)
                        *reinterpret_cast<uint4*>(slot(0, k) + at.col(j) * (int)sizeof(T)) = make_uint4(0, 0, 0, 0);
        }
    }
    __device__ __forceinline__ void fetch(int stage, int k, const T* row) const {
        const uint32_t dst = smem_addr(slot(stage, k));
        if constexpr (kVec) {
#pragma unroll
            for (int j = 0; j < NV; ++j)
                if (at.in(j)) cp_async_16(dst + at.col(j) * (int)sizeof(T), row + at.col(j), 16);
        } else {
            // the 16-byte pieces that hold the row: what is around it lies in the same
            // pieces as its ends, and nothing behind its last byte is read
            const int s = shift(row), bytes = s + at.H * (int)sizeof(T);
            const uint8_t* src = reinterpret_cast<const uint8_t*>(row) - s;
            for (int c = 16 * at.t; c < bytes; c += 16 * at.nt) cp_async_16(dst + c, src + c, bytes - c < 16 ? bytes - c : 16);
        }
    }
    // Zeros for a tensor that is not there.
    __device__ __forceinline__ Raw<T, E> read(int stage, int k, const T* row, bool there = true) const {
        const uint8_t* s = slot(stage, k);
        Raw<T, E> r;
        if (!there) {
            if constexpr (sizeof(T) == 4) {
#pragma unroll
                for (int i = 0; i < E / 2; ++i) r.p[i].v = 0;
            } else {
#pragma unroll
                for (int i = 0; i < E / 2; ++i) r.w[i] = 0;
            }
            return r;
        }
        if constexpr (sizeof(T) == 4) {
            if constexpr (kVec) {
                r = at.load_smem(reinterpret_cast<const float*>(s));
            } else {
                const float* e = reinterpret_cast<const float*>(s + shift(row));
                float f[E];
#pragma unroll
                for (int j = 0; j < E; ++j) f[j] = at.in(j) ? e[at.col(j)] : 0.0f;
                r = P::pairs(f);
            }
        } else if constexpr (kVec) {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const uint4 u = *reinterpret_cast<const uint4*>(s + 16 * (at.t + j * at.nt));
                r.w[4 * j] = u.x, r.w[4 * j + 1] = u.y, r.w[4 * j + 2] = u.z, r.w[4 * j + 3] = u.w;
            }
        } else {
            const uint16_t* e = reinterpret_cast<const uint16_t*>(s + shift(row));
#pragma unroll
            for (int j = 0; j < E / 2; ++j) {
                const uint32_t lo = at.in(2 * j) ? e[at.col(2 * j)] : 0, hi = at.in(2 * j + 1) ? e[at.col(2 * j + 1)] : 0;
                r.w[j] = lo | hi << 16;
            }
        }
        return r;
    }
};

// A row's number that the compiler does not turn into a running pointer for each
// tensor: sixteen of those in registers spilled what the loop works on.
__device__ __forceinline__ uint32_t plain_row(uint32_t row) {
    asm volatile("" : "+r"(row));
    return row;
}

// Waits until at most n of this thread's groups of copies are in flight (0 to 3).
__device__ __forceinline__ void ring_wait(int n) {
    if (n <= 0)
        cp_async_wait_group<0>();
    else if (n == 1)
        cp_async_wait_group<1>();
    else if (n == 2)
        cp_async_wait_group<2>();
    else
        cp_async_wait_group<3>();
}

struct RnFwd {
    RnShape s;
    const void *o, *r;
    long long os, rs;
    const void *g, *pw, *pb, *w, *b;
    void *stream, *normed;
    float* stats;  // [4][rows]: mean and rstd of o, mean and rstd of s
};
// Parameters in the order in which they get shared memory.
enum { kFwdW, kFwdPw, kFwdGate, kFwdB, kFwdPb };
enum { kBwdW, kBwdPw, kBwdGate, kBwdPb };

// v about the mean, columns past the row 0.
template <typename T, bool kVec, int E>
__device__ __forceinline__ Cols<E> about(const Cols<E>& v, float mean, const Place<T, kVec, E>& at) {
    constexpr int V = Place<T, kVec, E>::V;
    Cols<E> d;
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
        float2 f = unpack(v.p[i] + f2(-mean));
        if (!at.in(2 * i / V)) f.x = 0.0f;
        if (!at.in((2 * i + 1) / V)) f.y = 0.0f;
        d.p[i] = f2(f.x, f.y);
    }
    return d;
}
// Mean (0 for an RMS norm) and rstd of one or two rows, whose sums go together: what
// a row costs is the sums' latency.
template <typename T, bool kVec, bool kRms, int E, int kRows>
__device__ __forceinline__ void row_stats(const Cols<E> (&v)[kRows], float2 (&st)[kRows], const Place<T, kVec, E>& at,
                                          Group& grp, const RnShape& s) {
    float a[kRows];
    if constexpr (kRms) {
#pragma unroll
        for (int k = 0; k < kRows; ++k) st[k].x = 0.0f, a[k] = dot(v[k], v[k]);
    } else {
#pragma unroll
        for (int k = 0; k < kRows; ++k) a[k] = sum_of(v[k]);
        grp.sum(a);
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
            st[k].x = a[k] * s.inv;
            const Cols<E> d = about(v[k], st[k].x, at);
            a[k] = dot(d, d);
        }
    }
    grp.sum(a);
#pragma unroll
    for (int k = 0; k < kRows; ++k) st[k].y = rsqrtf(a[k] * s.inv + s.eps);
}

template <typename T, bool kVec, bool kPost, bool kRms, bool kHeld, int kThreads>
__global__ void __launch_bounds__(kThreads) rn_fwd_kernel(const RnFwd p) {
    constexpr int E = kRnCols, N = E / 2;
    extern __shared__ __align__(16) uint8_t smem[];
    const RnShape& s = p.s;
    const int id = (int)threadIdx.x / s.nt, t = (int)threadIdx.x - id * s.nt;
    const Place<T, kVec, E> at = {s.H, t, s.nt};
    Group grp = {id, t, s.nt, s.nt >> 5, t >> 5, reinterpret_cast<float4*>(smem + id * kRnRedBytes), 0};
    float* held = reinterpret_cast<float*>(smem + s.groups * kRnRedBytes);
    const Params<T, kVec, E, kHeld> param = {at, held, s.in_smem, s.w_f32};
    uint8_t* rings = reinterpret_cast<uint8_t*>(held + s.in_smem * E * s.nt);
    const Ring<T, kVec, E, 2> ring = {at, rings + id * s.stages * 2 * s.row_bytes, s.row_bytes};
    ring.clear(s.stages);
    const T *o = static_cast<const T*>(p.o), *r = static_cast<const T*>(p.r);
    // below 2^31 + 64 x 152 x 32: 32 bits without a sign
    const uint32_t step = gridDim.x * s.groups, row0 = blockIdx.x * s.groups + id, rows = (uint32_t)s.rows;
    auto fetch = [&](int stage, uint32_t row) {
        if (row < rows) ring.fetch(stage, 0, o + row * p.os), ring.fetch(stage, 1, r + row * p.rs);
        cp_async_commit();
    };
    for (int i = 0; i < s.stages; ++i) fetch(i, row0 + i * step);
    param.fill(held, kFwdW, p.w);
    param.fill(held, kFwdPw, p.pw);
    param.fill(held, kFwdGate, s.gate == MOE_GATE_CHANNEL ? p.g : nullptr);
    param.fill(held, kFwdB, p.b);
    param.fill(held, kFwdPb, p.pb);
    // The tokens' gates of this group's next 32 rows, a lane each: a load for each row
    // was waited for every time (8192 x 7168: 81 -> 107 us).
    const bool token = s.gate == MOE_GATE_TOKEN;
    float gates = 1.0f, gates_after = 1.0f;
    auto load_gates = [&](uint32_t row) {
        const uint32_t at = row + (threadIdx.x & 31) * step;
        return at < rows ? Param<T>{p.g, s.w_f32}.at((int)at) : 1.0f;
    };
    if (token) gates_after = load_gates(row0);
    uint32_t turn32 = 0;
    __syncthreads();
    // The post norm's statistics are taken a row ahead, with those of the stream.
    Raw<T, E> raw_o;
    float2 ost = make_float2(0.0f, 1.0f);
    if (kPost && row0 < rows) {
        ring_wait(s.stages - 1);
        if (!kVec) grp.sync();
        raw_o = ring.read(0, 0, o + row0 * p.os);
        const Cols<E> v[1] = {widen(raw_o)};
        float2 st[1];
        row_stats<T, kVec, kRms, E, 1>(v, st, at, grp, s);
        ost = st[0];
    }
    int stage = 0;
    for (uint32_t at_row = row0; at_row < rows; at_row += step) {
        const uint32_t row = plain_row(at_row), after = row + step;
        float gate = 1.0f;
        if (token) {
            if ((turn32 & 31) == 0) {
                gates = gates_after;
                gates_after = load_gates(row + 32 * step);
            }
            gate = __shfl_sync(0xffffffffu, gates, turn32 & 31);
            ++turn32;
        }
        const bool ahead = kPost && after < rows;
        ring_wait(s.stages - (kPost ? 2 : 1));
        if (!kVec) grp.sync();
        if (!kPost) raw_o = ring.read(stage, 0, o + row * p.os);
        Cols<E> v[kPost ? 2 : 1];
        v[0] = widen(raw_o);
        const Raw<T, E> raw_r = ring.read(stage, 1, r + row * p.rs);
        if constexpr (kPost) {
            if (t == 0) p.stats[row] = ost.x, p.stats[s.rows + row] = ost.y;
            const Cols<E> w = param(kFwdPw, p.pw);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                if (!kRms) v[0].p[i] = v[0].p[i] + f2(-ost.x);
                v[0].p[i] = v[0].p[i] * f2(ost.y) * w.p[i];
            }
            if (p.pb) {
                const Cols<E> b = param(kFwdPb, p.pb);
#pragma unroll
                for (int i = 0; i < N; ++i) v[0].p[i] = v[0].p[i] + b.p[i];
            }
        }
        if (s.gate == MOE_GATE_CHANNEL) {
            const Cols<E> g = param(kFwdGate, p.g);
#pragma unroll
            for (int i = 0; i < N; ++i) v[0].p[i] = v[0].p[i] * g.p[i];
        }
        {
            const Cols<E> res = widen(raw_r);
#pragma unroll
            for (int i = 0; i < N; ++i) v[0].p[i] = fma2(f2(s.alpha), res.p[i], v[0].p[i] * f2(gate));
        }
        at.store(static_cast<T*>(p.stream) + (size_t)row * s.H, v[0]);
        float2 st[kPost ? 2 : 1];
        if constexpr (kPost) {
            // (past the last row: this row's own, for nothing)
            raw_o = ring.read(ahead ? (stage + 1 == s.stages ? 0 : stage + 1) : stage, 0, o + (ahead ? after : row) * p.os);
            v[1] = widen(raw_o);
        }
        row_stats<T, kVec, kRms, E, kPost ? 2 : 1>(v, st, at, grp, s);
        if constexpr (kPost) ost = st[1];
        // every thread has read the stage before the sums' barrier
        fetch(stage, row + s.stages * step);
        if (t == 0) p.stats[2 * s.rows + row] = st[0].x, p.stats[3 * s.rows + row] = st[0].y;
        const Cols<E> w = param(kFwdW, p.w);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (!kRms) v[0].p[i] = v[0].p[i] + f2(-st[0].x);
            v[0].p[i] = v[0].p[i] * f2(st[0].y) * w.p[i];
        }
        if (p.b) {
            const Cols<E> b = param(kFwdB, p.b);
#pragma unroll
            for (int i = 0; i < N; ++i) v[0].p[i] = v[0].p[i] + b.p[i];
        }
        at.store(static_cast<T*>(p.normed) + (size_t)row * s.H, v[0]);
        if (++stage == s.stages) stage = 0;
    }
    cp_async_wait_all();
}

// ---------------------------------------------------------------- backward
struct RnJoin {
    const float* part;
    int parts, H, sums, w_f32, channel, post;
    const void *g, *pw, *pb;
    void *dw, *db, *dpw, *dpb, *dgate;  // null: not wanted
};
template <typename T>
__device__ __forceinline__ void put_param(void* p, int f32, int c, float v) {
    if (!p) return;
    if (f32)
        static_cast<float*>(p)[c] = v;
    else
        static_cast<T*>(p)[c] = from_f<T>(v);
}
// One column's gradients of its four sums.
template <typename T>
__device__ __forceinline__ void finish_column(const RnJoin& p, int c, const float (&v)[4]) {
    put_param<T>(p.dw, p.w_f32, c, v[0]);
    put_param<T>(p.db, p.w_f32, c, v[1]);
    const float gate = p.channel ? Param<T>{p.g, p.w_f32}.at(c) : 1.0f;
    put_param<T>(p.dpw, p.w_f32, c, gate * v[2]);
    put_param<T>(p.dpb, p.w_f32, c, gate * v[3]);
    if (p.channel && p.dgate) {
        float d = v[2];
        if (p.post) d = Param<T>{p.pw, p.w_f32}.at(c) * v[2] + (p.pb ? Param<T>{p.pb, p.w_f32}.at(c) * v[3] : 0.0f);
        put_param<T>(p.dgate, p.w_f32, c, d);
    }
}

struct RnBwd {
    RnShape s;
    const void *ds, *dn, *o, *r;  // ds, dn: may be null (zero)
    long long dss, dns, os, rs;
    const void *g, *pw, *pb, *w;
    const float* stats;
    void *dout, *dres;
    float* dgate_rows;  // MOE_GATE_TOKEN: FP32 [rows]; or null
    void* dgate_typed;  // the same in the gate's type, where that is not FP32
    int sums;           // column sums: 0 dn z, 1 dn, 2 (q or D) oz or D o, 3 q or D; a bit each
    float* part;        // [blocks][4][H]
    RnJoin join;        // kDirect
};

// What one row's scalars are: its statistics and its gate.
struct RnRow {
    float om, ors, m, rs, gt;
};

// Column sums in tensor memory: eight columns (of 32 lanes) a warp and sum, warp w in
// the lanes 32 (w % 4) .. that it reaches.  Two sums of a thread's columns are 16
// of its 72 registers, four are 32: in registers they left spills of 4 to 230
// bytes, which go to L2 (the rings leave L1 little): 8192 x 7168 with a post norm,
// 207 to 320 us.
template <int kSums>
struct TmemSums {
    uint32_t base;  // of this warp
    static constexpr int kCols = kRnCols * kSums;
    static __host__ __device__ constexpr int columns(int warps) {  // to allocate: a power of two from 32 on
        int n = 32;
        while (n < (warps + 3) / 4 * kCols) n *= 2;
        return n;
    }
    __device__ __forceinline__ Cols<kRnCols> load(int k) const {
        uint32_t r[8];
        __syncwarp();
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                     : "r"(base + kRnCols * k)
                     : "memory");
        tmem_ld_wait();
        Cols<kRnCols> c;
#pragma unroll
        for (int i = 0; i < 4; ++i) c.p[i] = f2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
        return c;
    }
    __device__ __forceinline__ void store(int k, const Cols<kRnCols>& c) const {
        uint32_t r[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = unpack(c.p[i]);
            r[2 * i] = __float_as_uint(f.x), r[2 * i + 1] = __float_as_uint(f.y);
        }
        asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(base + kRnCols * k),
                     "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                     : "memory");
    }
    // Stores have to have landed before the next load of the same columns.
    __device__ __forceinline__ static void settle() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
};

// A float of block `rank` of the cluster, at this block's address of it.
__device__ __forceinline__ float load_peer(const float* own, uint32_t rank) {
    uint32_t at;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(own)), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
    return v;
}

// kMode: an RMS or a layer norm without biases (column sums 0 and 2), or either
// with all four.
enum { kRms2, kLayer2, kAny4 };
// kDirect: few rows, the blocks are one cluster and add their column sums up themselves.
template <typename T, bool kVec, bool kPost, int kMode, bool kHeld, int kThreads, bool kDirect = false>
__global__ void __launch_bounds__(kThreads) rn_bwd_kernel(const RnBwd p) {
    constexpr int E = kRnCols, N = E / 2;
    constexpr bool kFour = kMode == kAny4, kRms = kMode == kRms2;
    extern __shared__ __align__(16) uint8_t smem[];
    const RnShape& s = p.s;
    const int id = (int)threadIdx.x / s.nt, t = (int)threadIdx.x - id * s.nt;
    const Place<T, kVec, E> at = {s.H, t, s.nt};
    Group grp = {id, t, s.nt, s.nt >> 5, t >> 5, reinterpret_cast<float4*>(smem + id * kRnRedBytes), 0};
    float* held = reinterpret_cast<float*>(smem + s.groups * kRnRedBytes);
    const Params<T, kVec, E, kHeld> param = {at, held, s.in_smem, s.w_f32};
    uint8_t* rings = reinterpret_cast<uint8_t*>(held + s.in_smem * E * s.nt);
    const Ring<T, kVec, E, 4> ring = {at, rings + id * s.stages * 4 * s.row_bytes, s.row_bytes};
    ring.clear(s.stages);
    const T *o = static_cast<const T*>(p.o), *r = static_cast<const T*>(p.r), *ds = static_cast<const T*>(p.ds),
            *dn = static_cast<const T*>(p.dn);
    // below 2^31 + 64 x 152 x 32: 32 bits without a sign
    const uint32_t step = gridDim.x * s.groups, row0 = blockIdx.x * s.groups + id, rows = (uint32_t)s.rows;
    auto fetch = [&](int stage, uint32_t row) {
        if (row < rows) {
            ring.fetch(stage, 0, o + row * p.os);
            ring.fetch(stage, 1, r + row * p.rs);
            if (dn) ring.fetch(stage, 2, dn + row * p.dns);
            if (ds) ring.fetch(stage, 3, ds + row * p.dss);
        }
        cp_async_commit();
    };
    for (int i = 0; i < s.stages; ++i) fetch(i, row0 + i * step);
    param.fill(held, kBwdW, p.w);
    param.fill(held, kBwdPw, p.pw);
    param.fill(held, kBwdGate, s.gate == MOE_GATE_CHANNEL ? p.g : nullptr);
    if (kFour) param.fill(held, kBwdPb, p.pb);
    const bool token = s.gate == MOE_GATE_TOKEN, channel = s.gate == MOE_GATE_CHANNEL;
    // A lane holds one of the group's next 32 rows': a load for each row was waited for
    // every time (see the forward).
    auto scalars = [&](uint32_t row0) {
        const uint32_t row = row0 + (threadIdx.x & 31) * step;
        RnRow c = {0.0f, 1.0f, 0.0f, 0.0f, 1.0f};
        if (row >= rows) return c;
        if (kPost) {
            if (!kRms) c.om = __ldg(p.stats + row);
            c.ors = __ldg(p.stats + s.rows + row);
        }
        if (!kRms) c.m = __ldg(p.stats + 2 * s.rows + row);
        c.rs = __ldg(p.stats + 3 * s.rows + row);
        if (token) c.gt = Param<T>{p.g, s.w_f32}.at((int)row);
        return c;
    };
    auto of_lane = [&](const RnRow& held, int lane) {
        RnRow c = {0.0f, 1.0f, 0.0f, 0.0f, 1.0f};
        if (kPost) {
            if (!kRms) c.om = __shfl_sync(0xffffffffu, held.om, lane);
            c.ors = __shfl_sync(0xffffffffu, held.ors, lane);
        }
        if (!kRms) c.m = __shfl_sync(0xffffffffu, held.m, lane);
        c.rs = __shfl_sync(0xffffffffu, held.rs, lane);
        if (token) c.gt = __shfl_sync(0xffffffffu, held.gt, lane);
        return c;
    };
    constexpr int kSums = kFour ? 4 : 2;  // of two, k is column sum 2 k
    __shared__ uint32_t tmem_slot;
    const int warp = (int)threadIdx.x >> 5, warps = (int)blockDim.x >> 5;
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&tmem_slot)),
                     "r"(TmemSums<kSums>::columns(warps))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    RnRow held_rows = scalars(row0);
    int turn32 = 0;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // not before the columns are this block's: a later kernel's block that took them
    // would wait for this one
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const TmemSums<kSums> acc = {tmem_slot + ((uint32_t)(warp & 3) << 21) + (uint32_t)(warp >> 2) * TmemSums<kSums>::kCols};
    {
        Cols<E> zero;
#pragma unroll
        for (int i = 0; i < N; ++i) zero.p[i].v = 0;
#pragma unroll
        for (int k = 0; k < kSums; ++k) acc.store(k, zero);
        acc.settle();
    }
    int stage = 0;
    for (uint32_t at_row = row0; at_row < rows; at_row += step) {
        const uint32_t row = plain_row(at_row);
        if (turn32 == 32) {
            held_rows = scalars(row);
            turn32 = 0;
        }
        __syncwarp();
        const RnRow c = of_lane(held_rows, turn32++);
        ring_wait(s.stages - 1);
        if (!kVec) grp.sync();
        const Raw<T, E> raw_o = ring.read(stage, 0, o + row * p.os), raw_dn = ring.read(stage, 2, dn + row * p.dns, dn != nullptr);
        auto normed_o = [&]() {  // N(o), or o
            Cols<E> v = widen(raw_o);
            if constexpr (kPost) {
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    if (!kRms) v.p[i] = v.p[i] + f2(-c.om);
                    v.p[i] = v.p[i] * f2(c.ors);
                }
            }
            return v;
        };
        auto dn_w = [&]() {
            Cols<E> v = widen(raw_dn);
            const Cols<E> w = param(kBwdW, p.w);
#pragma unroll
            for (int i = 0; i < N; ++i) v.p[i] = v.p[i] * w.p[i];
            return v;
        };
        Cols<E> z = normed_o();
        if constexpr (kPost) {
            const Cols<E> w = param(kBwdPw, p.pw);
#pragma unroll
            for (int i = 0; i < N; ++i) z.p[i] = z.p[i] * w.p[i];
            if (kFour && p.pb) {
                const Cols<E> b = param(kBwdPb, p.pb);
#pragma unroll
                for (int i = 0; i < N; ++i) z.p[i] = z.p[i] + b.p[i];
            }
        }
        if (channel) {
            const Cols<E> g = param(kBwdGate, p.g);
#pragma unroll
            for (int i = 0; i < N; ++i) z.p[i] = z.p[i] * g.p[i];
        }
        float hs[kRms ? 1 : 2];
        {
            const Cols<E> res = widen(ring.read(stage, 1, r + row * p.rs));
#pragma unroll
            for (int i = 0; i < N; ++i) {
                z.p[i] = fma2(f2(s.alpha), res.p[i], z.p[i] * f2(c.gt));
                if (!kRms) z.p[i] = z.p[i] + f2(-c.m);
                z.p[i] = z.p[i] * f2(c.rs);
            }
            const Cols<E> d = widen(raw_dn);
            acc.settle();
            {
                Cols<E> a = acc.load(0);
#pragma unroll
                for (int i = 0; i < N; ++i) a.p[i] = fma2(d.p[i], z.p[i], a.p[i]);
                acc.store(0, a);
            }
            if constexpr (kFour) {
                Cols<E> a = acc.load(1);
#pragma unroll
                for (int i = 0; i < N; ++i) a.p[i] = a.p[i] + d.p[i];
                acc.store(1, a);
            }
            const Cols<E> h = dn_w();
            hs[0] = dot(h, z);
            if constexpr (!kRms) hs[1] = sum_of(h);
        }
        // (in vectors each thread reads its own copies only, so later is soon enough)
        Raw<T, E> raw_ds;
        if (!kVec) raw_ds = ring.read(stage, 3, ds + row * p.dss, ds != nullptr);
        grp.sum(hs);
        if (kVec) raw_ds = ring.read(stage, 3, ds + row * p.dss, ds != nullptr);
        // every thread has read the stage before the sums' barrier
        fetch(stage, row + s.stages * step);
        const float h2 = hs[0] * s.inv, h1 = kRms || (kFour && s.rms) ? 0.0f : hs[kRms ? 0 : 1] * s.inv;
        Cols<E> D, q;
        {
            const Cols<E> h = dn_w(), d = widen(raw_ds);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                F2 v = fma2(z.p[i], f2(-h2), h.p[i]);
                if (!kRms) v = v + f2(-h1);
                D.p[i] = fma2(v, f2(c.rs), d.p[i]);
                q.p[i] = D.p[i] * f2(s.alpha);
            }
        }
        at.store(static_cast<T*>(p.dres) + (size_t)row * s.H, q);
        const Cols<E> oz = normed_o();
        // q, but for a gate per channel, which the join applies to the column sums
#pragma unroll
        for (int i = 0; i < N; ++i) q.p[i] = D.p[i] * f2(c.gt);
        {
            Cols<E> a = acc.load(kFour ? 2 : 1);
#pragma unroll
            for (int i = 0; i < N; ++i) a.p[i] = fma2(q.p[i], oz.p[i], a.p[i]);
            acc.store(kFour ? 2 : 1, a);
        }
        if constexpr (kFour) {
            Cols<E> a = acc.load(3);
#pragma unroll
            for (int i = 0; i < N; ++i) a.p[i] = a.p[i] + q.p[i];
            acc.store(3, a);
        }
        float pg = 0.0f;  // sum D u
        if constexpr (kPost) {
            // with p = gate D pw: sums of D pw (a gate per channel: D gate pw), the token's gate applied to them
            float ps[kRms ? 1 : kFour ? 3 : 2];
            if constexpr (kFour) {
                ps[2] = 0.0f;
                if (token && p.pb) ps[2] = dot(D, param(kBwdPb, p.pb));
            }
            const Cols<E> w = param(kBwdPw, p.pw);
#pragma unroll
            for (int i = 0; i < N; ++i) D.p[i] = D.p[i] * w.p[i];
            if (channel) {
                const Cols<E> g = param(kBwdGate, p.g);
#pragma unroll
                for (int i = 0; i < N; ++i) D.p[i] = D.p[i] * g.p[i];
            }
            ps[0] = dot(D, oz);
            if constexpr (!kRms) ps[1] = sum_of(D);
            grp.sum(ps);
            const float p2 = ps[0] * s.inv, p1 = kRms || (kFour && s.rms) ? 0.0f : ps[kRms ? 0 : 1] * s.inv, k = c.ors * c.gt;
            pg = ps[0] + (kFour ? ps[kFour ? 2 : 0] : 0.0f);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                F2 v = fma2(oz.p[i], f2(-p2), D.p[i]);
                if (!kRms) v = v + f2(-p1);
                q.p[i] = v * f2(k);
            }
        } else {
            if (token) pg = grp.sum(dot(D, oz));
            if (channel) {
                const Cols<E> g = param(kBwdGate, p.g);
#pragma unroll
                for (int i = 0; i < N; ++i) q.p[i] = q.p[i] * g.p[i];
            }
        }
        at.store(static_cast<T*>(p.dout) + (size_t)row * s.H, q);
        if (token && t == 0) {
            if (p.dgate_rows)
                p.dgate_rows[row] = pg;
            else if (p.dgate_typed)
                static_cast<T*>(p.dgate_typed)[row] = from_f<T>(pg);
        }
        if (++stage == s.stages) stage = 0;
    }
    cp_async_wait_all();
    acc.settle();
    // The groups' column sums in the rings' place, then each column's added in order by the
    // thread that alone reads them (the threads' own writes would be a quarter of a sector
    // each): all together (two stages are as much as four sums), but two sums with a post
    // norm one after the other, with which the compiler leaves the rows' loop faster (8192 x
    // 7168 145.6 -> 142.9 us; without a post norm 118 against 122).
    constexpr int V = Place<T, kVec, E>::V, NV = Place<T, kVec, E>::NV;
    const int sum_floats = s.groups * E * s.nt;
    float* col = reinterpret_cast<float*>(rings);  // [sums][groups][E nt], in the parameters' order
    auto leave = [&](int k, float* own) {
        float f[E];
        at.singles(acc.load(k), f);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if constexpr (V == 1) {
                own[at.col(j)] = f[j];
            } else {
#pragma unroll
                for (int h = 0; h < V / 4; ++h)
                    *reinterpret_cast<float4*>(own + 4 * (t + j * s.nt) + h * 4 * s.nt * NV) =
                        make_float4(f[j * V + 4 * h], f[j * V + 4 * h + 1], f[j * V + 4 * h + 2], f[j * V + 4 * h + 3]);
            }
        }
    };
    if constexpr (kFour || kDirect || !kPost) {
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kSums; ++k) leave(k, col + k * sum_floats + id * E * s.nt);
        __syncthreads();
        for (int c = p.sums ? (int)threadIdx.x : s.H; c < s.H; c += blockDim.x) {
            float v[kSums];
#pragma unroll
            for (int k = 0; k < kSums; ++k) v[k] = 0.0f;
            float* of = col + at.at(c);
            for (int gi = 0; gi < s.groups; ++gi)
#pragma unroll
                for (int k = 0; k < kSums; ++k) v[k] += of[k * sum_floats + gi * E * s.nt];
#pragma unroll
            for (int k = 0; k < kSums; ++k) {
                const int sum = kFour ? k : 2 * k;
                if constexpr (kDirect)
                    of[k * sum_floats] = v[k];
                else if (p.sums >> sum & 1)
                    p.part[((size_t)blockIdx.x * 4 + sum) * s.H + c] = v[k];
            }
        }
    } else {
#pragma unroll
        for (int k = 0; k < kSums; ++k) {
            if (!(p.sums >> 2 * k & 1)) continue;
            __syncthreads();
            leave(k, col + id * E * s.nt);
            __syncthreads();
            float* part = p.part + ((size_t)blockIdx.x * 4 + 2 * k) * s.H;
            for (int c = threadIdx.x; c < s.H; c += blockDim.x) {
                float v = 0.0f;
                for (int gi = 0; gi < s.groups; ++gi) v += col[gi * E * s.nt + at.at(c)];
                part[c] = v;
            }
        }
    }
    if constexpr (kDirect) {
        __syncthreads();
        cluster_sync();
        for (int c = (int)(blockIdx.x * blockDim.x + threadIdx.x); c < s.H; c += (int)(gridDim.x * blockDim.x)) {
            float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            for (uint32_t b = 0; b < gridDim.x; ++b)
#pragma unroll
                for (int k = 0; k < kSums; ++k) v[kFour ? k : 2 * k] += load_peer(col + k * sum_floats + at.at(c), b);
            finish_column<T>(p.join, c, v);
        }
        __syncthreads();
        cluster_sync();  // no block's memory goes while another reads it
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_slot),
                     "r"(TmemSums<kSums>::columns(warps)));
    }
}

// ------------------------------------------------------------- long rows
// Sums over the block (kRnLongThreads threads).
__device__ __forceinline__ float2 block_sum(float a, float b, float2* red) {
    a = warp_sum(a);
    b = warp_sum(b);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    __syncthreads();  // red may still be read
    if (lane == 0) red[warp] = make_float2(a, b);
    __syncthreads();
    const float2 v = red[lane];
    return make_float2(warp_sum(v.x), warp_sum(v.y));
}

template <typename T>
__global__ void __launch_bounds__(kRnLongThreads) rn_fwd_long_kernel(const RnFwd p) {
    __shared__ float2 red[32];
    const RnShape& s = p.s;
    const Param<T> pw = {p.pw, s.w_f32}, pb = {p.pb, s.w_f32}, w = {p.w, s.w_f32}, b = {p.b, s.w_f32}, g = {p.g, s.w_f32};
    for (long long row = blockIdx.x; row < s.rows; row += gridDim.x) {
        const T *o = static_cast<const T*>(p.o) + row * p.os, *r = static_cast<const T*>(p.r) + row * p.rs;
        float om = 0.0f, ors = 1.0f;
        if (p.pw) {
            float a = 0.0f;
            if (!s.rms) {
                for (int c = threadIdx.x; c < s.H; c += kRnLongThreads) a += to_f(o[c]);
                om = block_sum(a, 0.0f, red).x * s.inv;
            }
            a = 0.0f;
            for (int c = threadIdx.x; c < s.H; c += kRnLongThreads) {
                const float d = to_f(o[c]) - om;
                a += d * d;
            }
            ors = rsqrtf(block_sum(a, 0.0f, red).x * s.inv + s.eps);
            if (threadIdx.x == 0) p.stats[row] = om, p.stats[s.rows + row] = ors;
        }
        const float gt = s.gate == MOE_GATE_TOKEN ? g.at((int)row) : 1.0f;
        auto at = [&](int c) {
            float u = to_f(o[c]);
            if (p.pw) u = (u - om) * ors * pw.at(c) + (p.pb ? pb.at(c) : 0.0f);
            if (s.gate == MOE_GATE_CHANNEL) u *= g.at(c);
            return s.alpha * to_f(r[c]) + gt * u;
        };
        float a = 0.0f, m = 0.0f;
        if (!s.rms) {
            for (int c = threadIdx.x; c < s.H; c += kRnLongThreads) a += at(c);
            m = block_sum(a, 0.0f, red).x * s.inv;
        }
        a = 0.0f;
        for (int c = threadIdx.x; c < s.H; c += kRnLongThreads) {
            const float d = at(c) - m;
            a += d * d;
        }
        const float rstd = rsqrtf(block_sum(a, 0.0f, red).x * s.inv + s.eps);
        if (threadIdx.x == 0) p.stats[2 * s.rows + row] = m, p.stats[3 * s.rows + row] = rstd;
        for (int c = threadIdx.x; c < s.H; c += kRnLongThreads) {
            const float v = at(c);
            static_cast<T*>(p.stream)[row * s.H + c] = from_f<T>(v);
            static_cast<T*>(p.normed)[row * s.H + c] = from_f<T>((v - m) * rstd * w.at(c) + (p.b ? b.at(c) : 0.0f));
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(kRnLongThreads) rn_bwd_long_kernel(const RnBwd p) {
    __shared__ float2 red[32];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const RnShape& s = p.s;
    const Param<T> pw = {p.pw, s.w_f32}, pb = {p.pb, s.w_f32}, w = {p.w, s.w_f32}, g = {p.g, s.w_f32};
    float* part = p.part + (size_t)blockIdx.x * 4 * s.H;  // a column is one thread's
    bool first = true;
    for (long long row = blockIdx.x; row < s.rows; row += gridDim.x, first = false) {
        const T *o = static_cast<const T*>(p.o) + row * p.os, *r = static_cast<const T*>(p.r) + row * p.rs;
        const T* dn = p.dn ? static_cast<const T*>(p.dn) + row * p.dns : nullptr;
        const T* ds = p.ds ? static_cast<const T*>(p.ds) + row * p.dss : nullptr;
        const float om = p.pw ? p.stats[row] : 0.0f, ors = p.pw ? p.stats[s.rows + row] : 1.0f;
        const float m = p.stats[2 * s.rows + row], rs = p.stats[3 * s.rows + row];
        const float gt = s.gate == MOE_GATE_TOKEN ? g.at((int)row) : 1.0f;
        auto oz_at = [&](int c) { return p.pw ? (to_f(o[c]) - om) * ors : to_f(o[c]); };
        auto u_at = [&](int c) { return p.pw ? oz_at(c) * pw.at(c) + (p.pb ? pb.at(c) : 0.0f) : to_f(o[c]); };
        auto gate_at = [&](int c) { return s.gate == MOE_GATE_CHANNEL ? g.at(c) : gt; };
        auto z_at = [&](int c) { return (s.alpha * to_f(r[c]) + gate_at(c) * u_at(c) - m) * rs; };
        auto dn_at = [&](int c) { return dn ? to_f(dn[c]) : 0.0f; };
        float h1 = 0.0f, h2 = 0.0f;
        for (int c = threadIdx.x; c < s.H; c += kRnLongThreads) {
            const float h = dn_at(c) * w.at(c);
            h1 += h;
            h2 += h * z_at(c);
        }
        float2 sum = block_sum(h1, h2, red);
        h1 = s.rms ? 0.0f : sum.x * s.inv, h2 = sum.y * s.inv;
        auto D_at = [&](int c) {
            return (ds ? to_f(ds[c]) : 0.0f) + rs * (dn_at(c) * w.at(c) - h1 - z_at(c) * h2);
        };
        float p1 = 0.0f, p2 = 0.0f, pg = 0.0f;
        for (int c = threadIdx.x; c < s.H; c += kRnLongThreads) {
            const float D = D_at(c), oz = oz_at(c), pc = p.pw ? gate_at(c) * D * pw.at(c) : 0.0f;
            p1 += pc;
            p2 += pc * oz;
            pg += D * u_at(c);
        }
        sum = block_sum(p1, p2, red);
        p1 = s.rms ? 0.0f : sum.x * s.inv, p2 = sum.y * s.inv;
        if (s.gate == MOE_GATE_TOKEN && (p.dgate_rows || p.dgate_typed)) {
            pg = block_sum(pg, 0.0f, red).x;
            if (threadIdx.x == 0) {
                if (p.dgate_rows)
                    p.dgate_rows[row] = pg;
                else
                    static_cast<T*>(p.dgate_typed)[row] = from_f<T>(pg);
            }
        }
        for (int c = threadIdx.x; c < s.H; c += kRnLongThreads) {
            const float D = D_at(c), oz = oz_at(c), q = gate_at(c) * D, qs = gt * D, d = dn_at(c);
            static_cast<T*>(p.dres)[row * s.H + c] = from_f<T>(s.alpha * D);
            static_cast<T*>(p.dout)[row * s.H + c] = from_f<T>(p.pw ? ors * (q * pw.at(c) - p1 - oz * p2) : q);
            const float v[4] = {d * z_at(c), d, qs * oz, qs};
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (p.sums >> k & 1) part[(size_t)k * s.H + c] = (first ? 0.0f : part[(size_t)k * s.H + c]) + v[k];
        }
    }
}

// ---------------------------------------------------------------- the join
// 32 columns a block, a warp every 32nd part; all of a thread's loads are in flight
// together (a few at a time they were twenty trips to L2 one after another: the four
// sums of 2048 x 1024 took 14.8 us of its 25.4, 5 of 16.2 now).
constexpr int kJoinWarps = 32, kJoinMost = (152 + kJoinWarps - 1) / kJoinWarps;
template <typename T>
__global__ void __launch_bounds__(32 * kJoinWarps) rn_join_kernel(const RnJoin p) {
    __shared__ float red[4][kJoinWarps][33];
    asm volatile("griddepcontrol.launch_dependents;\n\tgriddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31, c = blockIdx.x * 32 + lane, warp = threadIdx.x >> 5;
    float u[4][kJoinMost];
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int i = 0; i < kJoinMost; ++i) {
            const int part = warp + kJoinWarps * i;
            u[k][i] = (p.sums >> k & 1) && part < p.parts && c < p.H ? p.part[((size_t)part * 4 + k) * p.H + c] : 0.0f;
        }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        float v = 0.0f;
#pragma unroll
        for (int i = 0; i < kJoinMost; ++i) v += u[k][i];
        red[k][warp][lane] = v;
    }
    __syncthreads();
    if (warp < 4) {  // a warp a sum
        float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < kJoinWarps; ++i) v[i & 3] += red[warp][i][lane];
        __syncwarp();
        red[warp][0][lane] = (v[0] + v[1]) + (v[2] + v[3]);
    }
    __syncthreads();
    if (warp || c >= p.H) return;
    const float v[4] = {red[0][0][lane], red[1][0][lane], red[2][0][lane], red[3][0][lane]};
    finish_column<T>(p, c, v);
}

// ----------------------------------------------------------------- launches
bool on16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// Groups, threads, ring and shared parameters (`params` of them at most) of a
// call; false: rows too long for the ring.  As many groups as the threads allow; where
// not even two stages of theirs fit, with no parameter beside them (the backward of
// FP32 rows: 28 groups of 128 columns would take 276 KB), fewer: one fits at every width.
int rn_group_threads(int H) { return ((H + kRnCols - 1) / kRnCols + 31) / 32 * 32; }
// Groups that the rows ask for and the threads allow, spread over so many blocks.
int rn_most_groups(long long rows, int nt, int threads, int spread) {
    int most = threads / nt;
    // sixteen hardware barriers, one of them the block's; a group of one warp needs none
    if (nt > 32 && most > 15) most = 15;
    const long long want = (rows + spread - 1) / spread;
    return (int)(want < most ? want : most);
}
bool rn_plan(RnShape& s, int elt, int tensors, int threads, int params, int* blocks, int* smem, int spread = 152) {
    if (s.H > kRnMaxH) return false;
    s.nt = rn_group_threads(s.H);
    // the threads' columns, or the row and the bytes before an unaligned one
    s.row_bytes = s.nt * kRnCols * elt + 16;
    const int param = s.nt * kRnCols * 4;
    auto fits = [&](int in_smem) {
        s.in_smem = in_smem;
        s.stages = (kRnSmem - s.groups * kRnRedBytes - in_smem * param) / (s.groups * tensors * s.row_bytes);
        return s.stages >= 2;
    };
    s.groups = rn_most_groups(s.rows, s.nt, threads, spread);
    while (s.groups > 1 && !fits(0)) --s.groups;
    int held = params;
    while (held > 0 && !fits(held)) --held;
    if (!fits(held)) return false;
    if (s.stages > 4) s.stages = 4;
    *smem = s.groups * kRnRedBytes + s.in_smem * param + s.stages * s.groups * tensors * s.row_bytes;
    const long long b = (s.rows + s.groups - 1) / s.groups;
    *blocks = (int)(b < spread ? b : spread);
    return true;
}

// Few rows in a backward: at most two for a group of a cluster of eight blocks (with
// any number of parameters, all of them held).  They need no second kernel and no
// partial sums in memory, which saves 5 us of the host's in a call (64 x 128, layer norms with
// everything on: 32 -> 27 us as called, whatever the rows) and, with one row a group, time
// on the GPU as well (64 x 128 8.6 -> 5.5 us, 24 x 2048 RMS 9.8 -> 8.6).  A second row comes after
// the first: 448 x 128 7.6 -> 10.8 us, 112 x 1024 10.5 -> 14.2, still less than what the host
// takes; a third was 16.9 of 8.8 us at 168 x 1024.  Long rows are added up by eight SMs alone (16 x
// 4096 12.1 -> 15.4).  Not where the groups had to be fewer: 300 x 128 f32 8.2 us otherwise, 11.0
// so, 96 x 1024 8.2 and 10.8.
constexpr int kDirectBlocks = 8, kDirectRows = 2, kDirectMaxH = 2048;
bool rn_direct(long long rows, int H, int elt) {
    RnShape s = {};
    s.rows = rows, s.H = H;
    int blocks, smem;
    if (rows < 1 || H > kDirectMaxH || !rn_plan(s, elt, 4, 896, 4, &blocks, &smem, kDirectBlocks)) return false;
    return s.in_smem == 4 && s.groups == rn_most_groups(rows, s.nt, 896, kDirectBlocks) &&
           rows <= (long long)kDirectRows * blocks * s.groups;
}

template <typename K, typename A>
int rn_launch(K kernel, SmemLimit& limit, int blocks, int threads, int smem, const A& a, const char* name, cudaStream_t st,
              int cluster = 1) {
    if (const int e = limit.allow(kernel, kRnSmem)) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 1 : 0;
    trace_pre(st);
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a);
    trace_post(st, name);
    return (int)(e != cudaSuccess ? e : cudaGetLastError());
}

RnShape rn_shape(const moe_residual_norm_shape& s) {
    RnShape r = {};
    r.rows = s.rows;
    r.H = s.H;
    r.rms = s.kind == MOE_NORM_RMS;
    r.gate = s.gate;
    r.w_f32 = s.w_type == MOE_F32;
    r.alpha = s.residual_scale;
    r.eps = s.eps;
    r.inv = 1.0f / (float)s.H;
    return r;
}
int rn_long_blocks(long long rows, int H) {
    long long most = (1 << 24) / H;
    most = most < 8 ? 8 : most > 152 ? 152 : most;
    return (int)(rows < most ? rows : most);
}

template <typename T, bool kPost, bool kRms>
int rn_forward(RnFwd& a, cudaStream_t st) {
    int blocks, smem;
    RnShape& s = a.s;
    const int params = a.pb ? 5 : a.b ? 4 : s.gate == MOE_GATE_CHANNEL ? 3 : kPost ? 2 : 1;
    constexpr int V = 16 / sizeof(T);
    const bool vec = s.H % V == 0 && a.os % V == 0 && a.rs % V == 0 && on16(a.o) && on16(a.r) && on16(a.stream) &&
                     on16(a.normed) && on16(a.pw) && on16(a.pb) && on16(a.w) && on16(a.b) &&
                     (s.gate != MOE_GATE_CHANNEL || on16(a.g));
    // 1024 threads at 64 registers where they hold one more row (8192 x 4096, post
    // norm: 65 -> 49 us)
    const int nt = rn_group_threads(s.H);
    const bool more = vec && 1024 / nt > 896 / nt;
    if (!rn_plan(s, sizeof(T), 2, more ? 1024 : 896, params, &blocks, &smem)) {
        trace_pre(st);
        rn_fwd_long_kernel<T><<<(unsigned)(s.rows < 304 ? s.rows : 304), kRnLongThreads, 0, st>>>(a);
        trace_post(st, "residual_norm_fwd");
        return (int)cudaGetLastError();
    }
    auto run = [&](auto kernel, SmemLimit& l) {
        return rn_launch(kernel, l, blocks, s.groups * s.nt, smem, a, "residual_norm_fwd", st);
    };
    static SmemLimit l[6];
    if (s.in_smem == params) {
        if (!vec) return run(rn_fwd_kernel<T, false, kPost, kRms, true, 896>, l[0]);
        return more ? run(rn_fwd_kernel<T, true, kPost, kRms, true, 1024>, l[1])
                    : run(rn_fwd_kernel<T, true, kPost, kRms, true, 896>, l[2]);
    }
    if (!vec) return run(rn_fwd_kernel<T, false, kPost, kRms, false, 896>, l[3]);
    return more ? run(rn_fwd_kernel<T, true, kPost, kRms, false, 1024>, l[4])
                : run(rn_fwd_kernel<T, true, kPost, kRms, false, 896>, l[5]);
}

template <typename T, bool kPost, int kMode>
int rn_backward(RnBwd& a, RnJoin& j, cudaStream_t st) {
    int blocks, smem, e;
    RnShape& s = a.s;
    const int params = a.pb ? 4 : s.gate == MOE_GATE_CHANNEL ? 3 : kPost ? 2 : 1;
    constexpr int V = 16 / sizeof(T);
    const bool vec = s.H % V == 0 && a.os % V == 0 && a.rs % V == 0 && (!a.dn || a.dns % V == 0) &&
                     (!a.ds || a.dss % V == 0) && on16(a.o) && on16(a.r) && on16(a.dn) && on16(a.ds) && on16(a.dout) &&
                     on16(a.dres) && on16(a.pw) && on16(a.pb) && on16(a.w) && (s.gate != MOE_GATE_CHANNEL || on16(a.g));
    // as in the forward (8192 x 4096, post norm: 104 -> 81 us), but FP32 rows, which
    // stay as wide from pass to pass and would spill (4096 x 2048: 45 -> 207 us)
    const int nt = rn_group_threads(s.H);
    const bool direct = a.sums && rn_direct(s.rows, s.H, sizeof(T));
    a.join = j;
    const bool more = !direct && vec && sizeof(T) == 2 && 1024 / nt > 896 / nt;
    if (!rn_plan(s, sizeof(T), 4, more ? 1024 : 896, params, &blocks, &smem, direct ? kDirectBlocks : 152)) {
        blocks = rn_long_blocks(s.rows, s.H);
        trace_pre(st);
        rn_bwd_long_kernel<T><<<blocks, kRnLongThreads, 0, st>>>(a);
        trace_post(st, "residual_norm_bwd");
        e = (int)cudaGetLastError();
    } else {
        if (direct && blocks > 1) blocks = kDirectBlocks;  // (the last ones may have no row)
        auto run = [&](auto kernel, SmemLimit& l) {
            return rn_launch(kernel, l, blocks, s.groups * s.nt, smem, a, "residual_norm_bwd", st, direct ? blocks : 1);
        };
        static SmemLimit l[8];
        if (direct)
            e = vec ? run(rn_bwd_kernel<T, true, kPost, kMode, true, 896, true>, l[6])
                    : run(rn_bwd_kernel<T, false, kPost, kMode, true, 896, true>, l[7]);
        else if (s.in_smem == params)
            e = !vec  ? run(rn_bwd_kernel<T, false, kPost, kMode, true, 896>, l[0])
                : more ? run(rn_bwd_kernel<T, true, kPost, kMode, true, 1024>, l[1])
                       : run(rn_bwd_kernel<T, true, kPost, kMode, true, 896>, l[2]);
        else
            e = !vec  ? run(rn_bwd_kernel<T, false, kPost, kMode, false, 896>, l[3])
                : more ? run(rn_bwd_kernel<T, true, kPost, kMode, false, 1024>, l[4])
                       : run(rn_bwd_kernel<T, true, kPost, kMode, false, 896>, l[5]);
    }
    if (e || !a.sums || direct) return e;
    j.parts = blocks;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)((s.H + 31) / 32));
    cfg.blockDim = dim3(32 * kJoinWarps);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    trace_pre(st);
    const cudaError_t ce = cudaLaunchKernelEx(&cfg, rn_join_kernel<T>, j);
    trace_post(st, "residual_norm_join");
    return (int)(ce != cudaSuccess ? ce : cudaGetLastError());
}

template <typename T>
int rn_forward_t(RnFwd& a, cudaStream_t st) {
    if (a.s.rms) return a.pw ? rn_forward<T, true, true>(a, st) : rn_forward<T, false, true>(a, st);
    return a.pw ? rn_forward<T, true, false>(a, st) : rn_forward<T, false, false>(a, st);
}
template <typename T>
int rn_backward_t(RnBwd& a, RnJoin& j, cudaStream_t st) {
    // 1 and 3: the biases' sums
    if (a.pb || (a.sums & 10)) return a.pw ? rn_backward<T, true, kAny4>(a, j, st) : rn_backward<T, false, kAny4>(a, j, st);
    if (a.s.rms) return a.pw ? rn_backward<T, true, kRms2>(a, j, st) : rn_backward<T, false, kRms2>(a, j, st);
    return a.pw ? rn_backward<T, true, kLayer2>(a, j, st) : rn_backward<T, false, kLayer2>(a, j, st);
}

// One type's calls: instantiated in a file of its own for each (the kernels take long to compile).
template <typename T>
int residual_norm_fwd(const moe_residual_norm_shape& s, const ResNormPtrs& f, cudaStream_t st) {
    RnFwd a = {rn_shape(s), f.out, f.residual, f.out_stride, f.residual_stride, f.gate, f.post_weight, f.post_bias,
               f.weight, f.bias, f.stream, f.normed, f.stats};
    return rn_forward_t<T>(a, st);
}
template <typename T>
int residual_norm_bwd(const moe_residual_norm_shape& s, const ResNormPtrs& f, cudaStream_t st) {
    const bool channel = s.gate == MOE_GATE_CHANNEL, token = s.gate == MOE_GATE_TOKEN;
    const int f32 = s.w_type == MOE_F32;
    const int sums = (f.dweight ? 1 : 0) | (f.dbias ? 2 : 0) | (f.dpost_weight || (channel && f.dgate) ? 4 : 0) |
                     (f.dpost_bias || (channel && f.dgate && f.post_bias) ? 8 : 0);
    RnBwd a = {rn_shape(s), f.dstream, f.dnormed, f.out, f.residual, f.dstream_stride, f.dnormed_stride, f.out_stride,
               f.residual_stride, f.gate, f.post_weight, f.post_bias, f.weight, f.stats, f.dout, f.dresidual,
               token && f32 ? static_cast<float*>(f.dgate) : nullptr, token && !f32 ? f.dgate : nullptr, sums, f.part, {}};
    RnJoin j = {f.part, 0, s.H, sums, f32, channel, f.post_weight != nullptr, f.gate, f.post_weight, f.post_bias,
                f.dweight, f.dbias, f.dpost_weight, f.dpost_bias, f.dgate};
    return rn_backward_t<T>(a, j, st);
}

}  // namespace

}  // namespace moe
