// Layer norm over the last axis, forward and backward (the norm in front of
// the router and the experts of a block).
//
//   m = mean_h x[r, h]            s = 1 / sqrt(mean_h (x[r, h] - m)^2 + eps)
//   z = (x - m) s                 y = z w + b
//   g = dy w                      dx = s (g - mean_h g - z mean_h (g z))
//   dw[h] = sum_r dy[r, h] z[r, h]                  db[h] = sum_r dy[r, h]
//
// All statistics and sums are FP32; the variance is taken around the mean in
// a second pass over the row's registers (no E[x^2] - m^2 cancellation).
// Bound by DRAM: the forward reads x and writes y, the backward reads x and
// dy and writes dx.
//
// A row stays in registers between the passes: one warp per row up to 128
// vectors, one block per row above, each thread holding NV vectors of V
// elements (16 bytes; V = 1 where the width, a stride or a base address is
// not a multiple of 16 bytes).  Rows too long for that are read again for
// every pass (ln_fwd_long, ln_bwd_long): the second and third time from L2.
//
// The weight's and bias's gradients: every block of the backward sums its own
// rows' dy z and dy per column in registers and leaves one row of partial
// sums; a second kernel adds the partials of each column in a fixed order
// (deterministic, no atomics).
#include "moe_internal.h"

#include <cuda_fp16.h>

namespace moe {

namespace {

constexpr int kLnWarps = 4;         // rows per block of the one-warp-per-row form
constexpr int kLnWarpVecs = 128;    // vectors of a row up to which one warp takes it
constexpr int kLnLongThreads = 1024;

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

// V consecutive elements of p as floats (p aligned to V sizeof(T) bytes).
template <typename T, int V>
__device__ __forceinline__ void load_vec(const T* p, float (&f)[V]) {
    if constexpr (V == 1) {
        f[0] = to_f(__ldg(p));
    } else if constexpr (V * sizeof(T) == 32) {  // eight floats
        const uint4 a = __ldg(reinterpret_cast<const uint4*>(p)), b = __ldg(reinterpret_cast<const uint4*>(p) + 1);
        const float* fa = reinterpret_cast<const float*>(&a);
        const float* fb = reinterpret_cast<const float*>(&b);
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = fa[i], f[4 + i] = fb[i];
    } else {
        static_assert(V * sizeof(T) == 16, "vector width");
        const uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
        const T* t = reinterpret_cast<const T*>(&u);
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = to_f(t[i]);
    }
}
template <typename T, int V>
__device__ __forceinline__ void store_vec(T* p, const float (&f)[V]) {
    if constexpr (V == 1) {
        *p = from_f<T>(f[0]);
    } else {
        static_assert(V * sizeof(T) == 16, "vector width");
        uint4 u;
        T* t = reinterpret_cast<T*>(&u);
#pragma unroll
        for (int i = 0; i < V; ++i) t[i] = from_f<T>(f[i]);
        *reinterpret_cast<uint4*>(p) = u;
    }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int s = 16; s >= 1; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
    return v;
}

// Sum of v over the row's threads (a warp, or the block), the same value and
// order in every thread.  red: 32 floats; two calls in turn use different ones.
template <bool kWarpRow>
__device__ __forceinline__ float row_sum(float v, float* red) {
    v = warp_sum(v);
    if constexpr (!kWarpRow) {
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
        __syncthreads();
        const int nw = (int)blockDim.x >> 5;
        v = warp_sum((int)(threadIdx.x & 31) < nw ? red[threadIdx.x & 31] : 0.0f);
    }
    return v;
}

// ------------------------------------------------------------------ forward
template <typename T, typename W, int V, int NV, bool kWarpRow>
__global__ void __launch_bounds__(1024) ln_fwd(long long rows, int H, const T* __restrict__ x, long long xs,
                                               const W* __restrict__ w, const W* __restrict__ b, float eps,
                                               T* __restrict__ y, float* __restrict__ mean, float* __restrict__ rstd) {
    __shared__ float red[64];
    const long long row = kWarpRow ? (long long)blockIdx.x * kLnWarps + (threadIdx.x >> 5) : (long long)blockIdx.x;
    if (row >= rows) return;  // whole warps of the one-warp-per-row form
    const int t = kWarpRow ? (int)(threadIdx.x & 31) : (int)threadIdx.x;
    const int nt = kWarpRow ? 32 : (int)blockDim.x;
    const int nvec = H / V;
    const T* xr = x + row * xs;
    float v[NV][V];
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = t + i * nt;
        if (c < nvec) {
            load_vec<T, V>(xr + (size_t)c * V, v[i]);
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) v[i][j] = 0.0f;
        }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) s += v[i][j];
    const float m = row_sum<kWarpRow>(s, red) / (float)H;
    float q = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (t + i * nt < nvec) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float d = v[i][j] - m;
                q = fmaf(d, d, q);
            }
        }
    const float r = 1.0f / sqrtf(row_sum<kWarpRow>(q, red + 32) / (float)H + eps);
    if (t == 0) {
        mean[row] = m;
        rstd[row] = r;
    }
    T* yr = y + row * (long long)H;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = t + i * nt;
        if (c < nvec) {
            float wv[V], o[V];
            load_vec<W, V>(w + (size_t)c * V, wv);
#pragma unroll
            for (int j = 0; j < V; ++j) o[j] = (v[i][j] - m) * r * wv[j];
            if (b) {
                load_vec<W, V>(b + (size_t)c * V, wv);
#pragma unroll
                for (int j = 0; j < V; ++j) o[j] += wv[j];
            }
            store_vec<T, V>(yr + (size_t)c * V, o);
        }
    }
}

// Rows of any length: three passes over the row.
template <typename T, typename W, int V>
__global__ void __launch_bounds__(kLnLongThreads)
    ln_fwd_long(long long rows, int H, const T* __restrict__ x, long long xs, const W* __restrict__ w,
                const W* __restrict__ b, float eps, T* __restrict__ y, float* __restrict__ mean,
                float* __restrict__ rstd) {
    __shared__ float red[64];
    const long long row = blockIdx.x;
    const T* xr = x + row * xs;
    const int nvec = H / V;
    float s = 0.0f, f[V];
    for (int c = threadIdx.x; c < nvec; c += kLnLongThreads) {
        load_vec<T, V>(xr + (size_t)c * V, f);
#pragma unroll
        for (int j = 0; j < V; ++j) s += f[j];
    }
    const float m = row_sum<false>(s, red) / (float)H;
    float q = 0.0f;
    for (int c = threadIdx.x; c < nvec; c += kLnLongThreads) {
        load_vec<T, V>(xr + (size_t)c * V, f);
#pragma unroll
        for (int j = 0; j < V; ++j) q = fmaf(f[j] - m, f[j] - m, q);
    }
    const float r = 1.0f / sqrtf(row_sum<false>(q, red + 32) / (float)H + eps);
    if (threadIdx.x == 0) {
        mean[row] = m;
        rstd[row] = r;
    }
    T* yr = y + row * (long long)H;
    for (int c = threadIdx.x; c < nvec; c += kLnLongThreads) {
        float wv[V], o[V];
        load_vec<T, V>(xr + (size_t)c * V, f);
        load_vec<W, V>(w + (size_t)c * V, wv);
#pragma unroll
        for (int j = 0; j < V; ++j) o[j] = (f[j] - m) * r * wv[j];
        if (b) {
            load_vec<W, V>(b + (size_t)c * V, wv);
#pragma unroll
            for (int j = 0; j < V; ++j) o[j] += wv[j];
        }
        store_vec<T, V>(yr + (size_t)c * V, o);
    }
}

// ----------------------------------------------------------------- backward
struct LnBwd {
    long long rows;
    int H;
    const void *dy, *x, *w;
    long long dys, xs;
    const float *mean, *rstd;
    void* dx;
    float* part;  // [blocks][2][H]: sums of dy z, sums of dy
};

// One row's dx in registers plus the block's column sums.  One warp per row:
// the block's warps join their column sums through shared memory at the end.
template <typename T, typename W, int V, int NV, bool kWarpRow>
__global__ void __launch_bounds__(512) ln_bwd(const LnBwd p) {
    __shared__ float red[2][32];
    extern __shared__ float colsum[];  // one-warp-per-row form: [2][H]
    const int t = kWarpRow ? (int)(threadIdx.x & 31) : (int)threadIdx.x;
    const int nt = kWarpRow ? 32 : (int)blockDim.x;
    const int H = p.H, nvec = H / V;
    const T *dy = static_cast<const T*>(p.dy), *x = static_cast<const T*>(p.x);
    const W* w = static_cast<const W*>(p.w);
    T* dx = static_cast<T*>(p.dx);
    float sw[NV][V], sb[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) sw[i][j] = sb[i][j] = 0.0f;
    const long long step = kWarpRow ? (long long)gridDim.x * kLnWarps : (long long)gridDim.x;
    const long long first = kWarpRow ? (long long)blockIdx.x * kLnWarps + (threadIdx.x >> 5) : (long long)blockIdx.x;
    for (long long row = first; row < p.rows; row += step) {
        const float m = __ldg(p.mean + row), r = __ldg(p.rstd + row);
        float z[NV][V], g[NV][V];
        float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = t + i * nt;
            if (c < nvec) {
                load_vec<T, V>(x + row * p.xs + (size_t)c * V, z[i]);
                load_vec<T, V>(dy + row * p.dys + (size_t)c * V, g[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = t + i * nt;
            if (c < nvec) {
                float wv[V];
                load_vec<W, V>(w + (size_t)c * V, wv);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    z[i][j] = (z[i][j] - m) * r;
                    sb[i][j] += g[i][j];
                    sw[i][j] = fmaf(g[i][j], z[i][j], sw[i][j]);
                    g[i][j] *= wv[j];
                    s1 += g[i][j];
                    s2 = fmaf(g[i][j], z[i][j], s2);
                }
            }
        }
        s1 = warp_sum(s1);
        s2 = warp_sum(s2);
        if constexpr (!kWarpRow) {
            const int lane = threadIdx.x & 31;
            if (lane == 0) {
                red[0][threadIdx.x >> 5] = s1;
                red[1][threadIdx.x >> 5] = s2;
            }
            __syncthreads();
            const int nw = (int)blockDim.x >> 5;
            s1 = warp_sum(lane < nw ? red[0][lane] : 0.0f);
            s2 = warp_sum(lane < nw ? red[1][lane] : 0.0f);
            __syncthreads();  // before the next row's partial sums overwrite these
        }
        const float c1 = s1 / (float)H, c2 = s2 / (float)H;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = t + i * nt;
            if (c < nvec) {
                float o[V];
#pragma unroll
                for (int j = 0; j < V; ++j) o[j] = r * (g[i][j] - c1 - z[i][j] * c2);
                store_vec<T, V>(dx + row * (long long)H + (size_t)c * V, o);
            }
        }
    }
    float* out = p.part + (size_t)blockIdx.x * 2 * H;
    if constexpr (kWarpRow) {
        // warp after warp in a fixed order
        for (int wi = 0; wi < kLnWarps; ++wi) {
            if ((int)(threadIdx.x >> 5) == wi) {
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int c = t + i * nt;
                    if (c < nvec) {
#pragma unroll
                        for (int j = 0; j < V; ++j) {
                            const int h = c * V + j;
                            colsum[h] = wi ? colsum[h] + sw[i][j] : sw[i][j];
                            colsum[H + h] = wi ? colsum[H + h] + sb[i][j] : sb[i][j];
                        }
                    }
                }
            }
            __syncthreads();
        }
        for (int h = threadIdx.x; h < 2 * H; h += blockDim.x) out[h] = colsum[h];
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = t + i * nt;
            if (c < nvec) {
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    out[c * V + j] = sw[i][j];
                    out[H + c * V + j] = sb[i][j];
                }
            }
        }
    }
}

// Rows of any length: dx with three passes over the row, and the column sums
// of a band of rows by one thread per column.
template <typename T, typename W, int V>
__global__ void __launch_bounds__(kLnLongThreads) ln_bwd_long(const LnBwd p) {
    __shared__ float red[64];
    const int H = p.H, nvec = H / V;
    const long long row = blockIdx.x;
    const T *dy = static_cast<const T*>(p.dy) + row * p.dys, *x = static_cast<const T*>(p.x) + row * p.xs;
    const W* w = static_cast<const W*>(p.w);
    T* dx = static_cast<T*>(p.dx) + row * (long long)H;
    const float m = __ldg(p.mean + row), r = __ldg(p.rstd + row);
    float s1 = 0.0f, s2 = 0.0f, xv[V], gv[V], wv[V];
    for (int c = threadIdx.x; c < nvec; c += kLnLongThreads) {
        load_vec<T, V>(x + (size_t)c * V, xv);
        load_vec<T, V>(dy + (size_t)c * V, gv);
        load_vec<W, V>(w + (size_t)c * V, wv);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float g = gv[j] * wv[j];
            s1 += g;
            s2 = fmaf(g, (xv[j] - m) * r, s2);
        }
    }
    const float c1 = row_sum<false>(s1, red) / (float)H;
    const float c2 = row_sum<false>(s2, red + 32) / (float)H;
    for (int c = threadIdx.x; c < nvec; c += kLnLongThreads) {
        float o[V];
        load_vec<T, V>(x + (size_t)c * V, xv);
        load_vec<T, V>(dy + (size_t)c * V, gv);
        load_vec<W, V>(w + (size_t)c * V, wv);
#pragma unroll
        for (int j = 0; j < V; ++j) o[j] = r * (gv[j] * wv[j] - c1 - (xv[j] - m) * r * c2);
        store_vec<T, V>(dx + (size_t)c * V, o);
    }
}
template <typename T>
__global__ void __launch_bounds__(256) ln_bwd_long_cols(const LnBwd p, int bands) {
    const int h = blockIdx.x * 256 + threadIdx.x;
    if (h >= p.H) return;
    const T *dy = static_cast<const T*>(p.dy), *x = static_cast<const T*>(p.x);
    const long long per = (p.rows + bands - 1) / bands;
    const long long r0 = (long long)blockIdx.y * per, r1 = r0 + per < p.rows ? r0 + per : p.rows;
    float sw = 0.0f, sb = 0.0f;
    for (long long row = r0; row < r1; ++row) {
        const float g = to_f(__ldg(dy + row * p.dys + h));
        sb += g;
        sw = fmaf(g, (to_f(__ldg(x + row * p.xs + h)) - __ldg(p.mean + row)) * __ldg(p.rstd + row), sw);
    }
    p.part[(size_t)blockIdx.y * 2 * p.H + h] = sw;
    p.part[(size_t)blockIdx.y * 2 * p.H + p.H + h] = sb;
}

// dw[h] (and db[h]) = sum over the nb partial rows, in order.  32 columns per
// block; warp k takes every 8th partial row, then the eight are added.
template <typename W>
__global__ void __launch_bounds__(256) ln_bwd_join(const float* __restrict__ part, int nb, int H, W* __restrict__ dw,
                                                   W* __restrict__ db) {
    __shared__ float s[8][33];
    const int lane = threadIdx.x & 31, k = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + lane;  // of 2 H
    float a = 0.0f;
    if (col < 2 * H)
        for (int i = k; i < nb; i += 8) a += __ldg(part + (size_t)i * 2 * H + col);
    s[k][lane] = a;
    __syncthreads();
    if (k == 0 && col < 2 * H) {
#pragma unroll
        for (int i = 1; i < 8; ++i) a += s[i][lane];
        if (col < H)
            dw[col] = from_f<W>(a);
        else if (db)
            db[col - H] = from_f<W>(a);
    }
}

// Launch shape of a row form: vector width, vectors per thread, threads.
struct LnForm {
    bool vec, warp_row, longrow;
    int nv, threads;
};
LnForm ln_form(int H, int elt, bool vec, int max_threads) {
    LnForm f = {};
    const int V = vec ? 16 / elt : 1;
    const int nvec = H / V;
    f.vec = vec;
    if (nvec <= kLnWarpVecs) {
        f.warp_row = true;
        f.nv = nvec <= 32 ? 1 : nvec <= 64 ? 2 : 4;
        f.threads = 32 * kLnWarps;
        return f;
    }
    for (f.nv = 4; f.nv <= 16 && f.nv * V <= 32; f.nv *= 2) {
        f.threads = ((nvec + f.nv - 1) / f.nv + 31) / 32 * 32;
        if (f.threads <= max_threads) return f;
    }
    f.longrow = true;
    return f;
}

bool mult16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

template <typename T, typename W, int V, int NV>
void run_fwd(const LnForm& f, const LnFwdArgs& a, cudaStream_t st) {
    const T* x = static_cast<const T*>(a.x);
    const W *w = static_cast<const W*>(a.weight), *b = static_cast<const W*>(a.bias);
    T* y = static_cast<T*>(a.y);
    if constexpr (NV <= 4) {
        if (f.warp_row) {
            ln_fwd<T, W, V, NV, true><<<(unsigned)((a.rows + kLnWarps - 1) / kLnWarps), f.threads, 0, st>>>(
                a.rows, a.H, x, a.x_stride, w, b, a.eps, y, a.mean, a.rstd);
            return;
        }
    }
    if constexpr (NV >= 4)
        ln_fwd<T, W, V, NV, false><<<(unsigned)a.rows, f.threads, 0, st>>>(a.rows, a.H, x, a.x_stride, w, b, a.eps, y,
                                                                            a.mean, a.rstd);
}
template <typename T, typename W, int V>
int fwd_v(const LnFwdArgs& a, cudaStream_t st) {
    const LnForm f = ln_form(a.H, sizeof(T), V > 1, 1024);
    if (f.longrow) {
        ln_fwd_long<T, W, V><<<(unsigned)a.rows, kLnLongThreads, 0, st>>>(
            a.rows, a.H, static_cast<const T*>(a.x), a.x_stride, static_cast<const W*>(a.weight),
            static_cast<const W*>(a.bias), a.eps, static_cast<T*>(a.y), a.mean, a.rstd);
    } else {
        switch (f.nv) {
            case 1: run_fwd<T, W, V, 1>(f, a, st); break;
            case 2: run_fwd<T, W, V, 2>(f, a, st); break;
            case 4: run_fwd<T, W, V, 4>(f, a, st); break;
            case 8: if constexpr (8 * V <= 32) run_fwd<T, W, V, 8>(f, a, st); break;
            default: if constexpr (16 * V <= 32) run_fwd<T, W, V, 16>(f, a, st); break;
        }
    }
    return (int)cudaGetLastError();
}
template <typename T, typename W>
int fwd_t(const LnFwdArgs& a, cudaStream_t st) {
    constexpr int V = 16 / sizeof(T);
    const bool vec = a.H % V == 0 && a.x_stride % V == 0 && mult16(a.x) && mult16(a.y) && mult16(a.weight) &&
                     mult16(a.bias);
    return vec ? fwd_v<T, W, V>(a, st) : fwd_v<T, W, 1>(a, st);
}

template <typename T, typename W, int V, int NV>
void run_bwd(const LnForm& f, const LnBwd& p, int blocks, cudaStream_t st) {
    if constexpr (NV <= 4) {
        if (f.warp_row) {
            ln_bwd<T, W, V, NV, true><<<blocks, f.threads, sizeof(float) * 2 * p.H, st>>>(p);
            return;
        }
    }
    if constexpr (NV >= 4) ln_bwd<T, W, V, NV, false><<<blocks, f.threads, 0, st>>>(p);
}
template <typename T, typename W, int V>
int bwd_v(const LnBwdArgs& a, cudaStream_t st) {
    LnBwd p = {a.rows, a.H, a.dy, a.x, a.weight, a.dy_stride, a.x_stride, a.mean, a.rstd, a.dx, a.part};
    const LnForm f = ln_form(a.H, sizeof(T), V > 1, 512);
    int blocks;
    if (f.longrow) {
        blocks = (int)(a.rows < kLnBwdBlocks ? a.rows : kLnBwdBlocks);  // bands of rows
        ln_bwd_long<T, W, V><<<(unsigned)a.rows, kLnLongThreads, 0, st>>>(p);
        ln_bwd_long_cols<T><<<dim3((a.H + 255) / 256, blocks), 256, 0, st>>>(p, blocks);
    } else {
        const long long units = f.warp_row ? (a.rows + kLnWarps - 1) / kLnWarps : a.rows;
        blocks = (int)(units < kLnBwdBlocks ? units : kLnBwdBlocks);
        switch (f.nv) {
            case 1: run_bwd<T, W, V, 1>(f, p, blocks, st); break;
            case 2: run_bwd<T, W, V, 2>(f, p, blocks, st); break;
            case 4: run_bwd<T, W, V, 4>(f, p, blocks, st); break;
            case 8: if constexpr (8 * V <= 32) run_bwd<T, W, V, 8>(f, p, blocks, st); break;
            default: if constexpr (16 * V <= 32) run_bwd<T, W, V, 16>(f, p, blocks, st); break;
        }
    }
    ln_bwd_join<W><<<(2 * a.H + 31) / 32, 256, 0, st>>>(a.part, blocks, a.H, static_cast<W*>(a.dweight),
                                                         static_cast<W*>(a.dbias));
    return (int)cudaGetLastError();
}
template <typename T, typename W>
int bwd_t(const LnBwdArgs& a, cudaStream_t st) {
    constexpr int V = 16 / sizeof(T);
    const bool vec = a.H % V == 0 && a.x_stride % V == 0 && a.dy_stride % V == 0 && mult16(a.x) && mult16(a.dy) &&
                     mult16(a.dx) && mult16(a.weight);
    return vec ? bwd_v<T, W, V>(a, st) : bwd_v<T, W, 1>(a, st);
}

}  // namespace

int launch_layer_norm_fwd(int x_type, int w_type, const LnFwdArgs& a, cudaStream_t st) {
    const bool same = x_type == w_type;
    switch (x_type) {
        case MOE_F32: return fwd_t<float, float>(a, st);
        case MOE_F16: return same ? fwd_t<__half, __half>(a, st) : fwd_t<__half, float>(a, st);
        default: return same ? fwd_t<__nv_bfloat16, __nv_bfloat16>(a, st) : fwd_t<__nv_bfloat16, float>(a, st);
    }
}
int launch_layer_norm_bwd(int x_type, int w_type, const LnBwdArgs& a, cudaStream_t st) {
    const bool same = x_type == w_type;
    switch (x_type) {
        case MOE_F32: return bwd_t<float, float>(a, st);
        case MOE_F16: return same ? bwd_t<__half, __half>(a, st) : bwd_t<__half, float>(a, st);
        default: return same ? bwd_t<__nv_bfloat16, __nv_bfloat16>(a, st) : bwd_t<__nv_bfloat16, float>(a, st);
    }
}

}  // namespace moe
