// Layer norm over the last axis, forward and backward (the norm in front of
// the router and the experts of a block).
//
//   m = mean_h x[r, h]            s = 1 / sqrt(mean_h (x[r, h] - m)^2 + eps)
//   z = (x - m) s                 y = z w + b
//   g = dy w                      dx = s (g - mean_h g - z mean_h (g z))
//   dw[h] = sum_r dy[r, h] z[r, h]                  db[h] = sum_r dy[r, h]
//
// All statistics and sums are FP32; the variance is taken around a mean (the
// row's, or the thread's own and joined exactly), never as E[x^2] - m^2.
// Bound by DRAM: the forward reads x and writes y, the backward reads x and
// dy and writes dx.  Measured at 8192 x 7168: FP32 6.1 (forward) and 6.4 TB/s
// (backward), bf16 5.4 and 5.0 TB/s (43.3 and 70.0 us), of 6.8 TB/s for a plain
// copy.  The two-byte types fill neither the issue slots (54-57 %) nor DRAM
// (51-61 % of its nominal peak): with one block of 15 or 16 warps on an SM and a
// barrier for every row, what is left is latency.
//
// Three forms, by a rule on sizes, alignment and rows (ln_form, ring_pays):
//  * ring: tensors that start on 16-byte boundaries, rows up to 1920 vectors of
//    16 bytes (backward 2048).  Persistent blocks cut into groups; a group takes
//    one row at a time, each of its gt threads NV vectors of it.  Every thread
//    copies its own vectors of the group's next rows ahead with cp.async into
//    its own slots of shared memory (so no barrier guards the copies, and rows
//    stay in flight whatever a row's reduction waits for), and keeps its
//    columns' weight (and the backward's column sums) in registers for the life
//    of the block: read per row, an FP32 weight and bias are four times the
//    bytes of a bf16 row (one block per row with those reads: forward 60 us,
//    backward 190 us).
//    Every warp reducing (two chains of five shuffles per sum) took 22 of a
//    56 us forward.  So a group of several warps has one more warp that only
//    reduces: step n of a group is row n's per-thread partials (one store each),
//    row n - 1's reduction by that warp and row n - 2's output, side by side,
//    then one barrier.  A group of one warp reduces by shuffles.
//    Widths that are no multiple of 16 bytes: rows start anywhere in a vector,
//    but a group's rows are a multiple of 8 apart and so start equally far into
//    one; the columns around the whole vectors go to one warp's lanes (kShift).
//  * register: other addresses and strides, and few rows of such widths, one
//    element at a time; one warp per row up to 128 elements, one block above.
//  * long: rows too long for the others are read again for every pass (the
//    second and third time from L2).
//
// The weight's and bias's gradients: every block of the backward sums its own
// rows' dy z and dy per column in registers and leaves one row of partial
// sums; a second kernel adds the partials of each column in a fixed order
// (deterministic, no atomics).
#include "moe_internal.h"
#include "ptx.cuh"
#include "smem_limit.h"

#include <cuda_fp16.h>

namespace moe {

namespace {

constexpr int kLnWarps = 4;         // rows per block of the one-warp-per-row form
constexpr int kLnLongThreads = 1024;
// ring form: threads per block (128 registers each), rows held or in flight
// per group
constexpr int kLnRingThreads = 512;
constexpr int kLnFwdRing = 6;
__host__ __device__ constexpr int ln_bwd_ring_rows(int nv) { return nv > 2 ? 3 : 6; }
constexpr int kLnMaxGroups = 16, kLnGroupWarps = 16;

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

// ------------------------------------------------------------ register form
template <typename T, typename W, int NV, bool kWarpRow>
__global__ void __launch_bounds__(kWarpRow ? 32 * kLnWarps : 1024)
    ln_fwd(long long rows, int H, const T* __restrict__ x, long long xs, const W* __restrict__ w,
           const W* __restrict__ b, float eps, T* __restrict__ y, float* __restrict__ mean, float* __restrict__ rstd) {
    __shared__ float red[64];
    const long long row = kWarpRow ? (long long)blockIdx.x * kLnWarps + (threadIdx.x >> 5) : (long long)blockIdx.x;
    if (row >= rows) return;  // whole warps of the one-warp-per-row form
    const int t = kWarpRow ? (int)(threadIdx.x & 31) : (int)threadIdx.x;
    const int nt = kWarpRow ? 32 : (int)blockDim.x;
    const T* xr = x + row * xs;
    float v[NV], wv[NV], bv[NV];  // all loads at once: the reductions would hide none of the later ones
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = t + i * nt;
        v[i] = c < H ? to_f(__ldg(xr + c)) : 0.0f;
        wv[i] = c < H ? to_f(__ldg(w + c)) : 0.0f;
        bv[i] = b && c < H ? to_f(__ldg(b + c)) : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) s += v[i];
    const float m = row_sum<kWarpRow>(s, red) / (float)H;
    float q = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (t + i * nt < H) q = fmaf(v[i] - m, v[i] - m, q);
    const float r = 1.0f / sqrtf(row_sum<kWarpRow>(q, red + 32) / (float)H + eps);
    if (t == 0) {
        mean[row] = m;
        rstd[row] = r;
    }
    T* yr = y + row * (long long)H;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = t + i * nt;
        if (c < H) {
            yr[c] = from_f<T>(fmaf((v[i] - m) * r, wv[i], bv[i]));
        }
    }
}

// ---------------------------------------------------------------- ring form
// Named barrier 1 + g over a group's threads (its reducing warp among them).
__device__ __forceinline__ void group_sync(int g, int n) {
    asm volatile("bar.sync %0, %1;" ::"r"(g + 1), "r"(n) : "memory");
}

// Two floats in one 64-bit register pair: add, multiply and fused multiply-add
// take both at once, which halves the instructions of these kernels (at bf16
// the instruction issue, not DRAM, bounded the scalar form).
typedef unsigned long long f2;
__device__ __forceinline__ f2 f2_make(float a, float b) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 f2_get(f2 v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ f2 f2_add(f2 a, f2 b) {
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 f2_mul(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 f2_fma(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ float f2_sum(f2 v) {
    const float2 t = f2_get(v);
    return t.x + t.y;
}

// Two elements packed in a word as floats, and back.
template <typename T>
__device__ __forceinline__ f2 unpack2(uint32_t u);
template <>
__device__ __forceinline__ f2 unpack2<__nv_bfloat16>(uint32_t u) {
    return f2_make(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
template <>
__device__ __forceinline__ f2 unpack2<__half>(uint32_t u) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u));
    return f2_make(f.x, f.y);
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(f2 v);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(f2 v) {
    const float2 f = f2_get(v);
    return pack_bf16x2(f.x, f.y);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(f2 v) {
    const float2 f = f2_get(v);
    const __half2 h = __floats2half2_rn(f.x, f.y);
    return *reinterpret_cast<const uint32_t*>(&h);
}
// A 16-byte vector of T as P = 8 / sizeof(T) pairs, and back.
template <typename T, int P>
__device__ __forceinline__ void unpack_vec(const uint4& u, f2 (&f)[P]) {
    if constexpr (sizeof(T) == 4) {
        f[0] = f2_make(__uint_as_float(u.x), __uint_as_float(u.y));
        f[1] = f2_make(__uint_as_float(u.z), __uint_as_float(u.w));
    } else {
        f[0] = unpack2<T>(u.x);
        f[1] = unpack2<T>(u.y);
        f[2] = unpack2<T>(u.z);
        f[3] = unpack2<T>(u.w);
    }
}
template <typename T, int P>
__device__ __forceinline__ uint4 pack_vec(const f2 (&f)[P]) {
    if constexpr (sizeof(T) == 4) {
        const float2 a = f2_get(f[0]), b = f2_get(f[1]);
        return make_uint4(__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x), __float_as_uint(b.y));
    } else {
        return make_uint4(pack2<T>(f[0]), pack2<T>(f[1]), pack2<T>(f[2]), pack2<T>(f[3]));
    }
}
// 2 P consecutive elements of a weight vector as pairs.
template <typename W, int P>
__device__ __forceinline__ void load_pairs(const W* p, f2 (&f)[P]) {
    float v[2 * P];
    load_vec<W, 2 * P>(p, v);
#pragma unroll
    for (int i = 0; i < P; ++i) f[i] = f2_make(v[2 * i], v[2 * i + 1]);
}

// 2 P weights from anywhere, one by one.
template <typename W, int P>
__device__ __forceinline__ void load_each(const W* p, f2 (&f)[P]) {
#pragma unroll
    for (int j = 0; j < P; ++j) f[j] = f2_make(to_f(__ldg(p + 2 * j)), to_f(__ldg(p + 2 * j + 1)));
}

// Mean and rstd of a row from its threads' sums and their squared distances
// from their own means (n values each): the sums give the mean m, and
// sum (x - m)^2 = sum_t M2_t + sum_t n_t (mean_t - m)^2.  No difference of
// large squares: exact however far the row lies from zero.
struct LnStat {
    float mean, rstd;
};

// gt working threads per group; groups of several warps have a reducing warp
// after them (kReducer).
// kShift: rows that start between 16-byte boundaries.  A group's rows are then a
// multiple of 8 apart, so that they all start equally far past one: the groups'
// threads take the whole vectors between the first boundary and the last, and
// the few columns around them are the reducing (or the only) warp's, one a lane,
// which has time for them (masked vectors at the ends held their warps up, and
// so every row's barrier: 8192 x 7161 bf16 114 us, 48 us with the ends apart, 7168 43 us).
template <typename T, typename W, int NV, bool kBias, bool kReducer, bool kShift>
__global__ void __launch_bounds__(kLnRingThreads, 1)
    ln_fwd_ring(long long rows, int H, int gt, const T* __restrict__ x, long long xs, const W* __restrict__ w,
                const W* __restrict__ b, float eps, T* __restrict__ y, float* __restrict__ mean,
                float* __restrict__ rstd) {
    constexpr int V = 16 / sizeof(T), P = V / 2, kRing = kLnFwdRing, kLag = kReducer ? 2 : 0;
    extern __shared__ uint4 ring[];  // [kRing][NV][blockDim.x]
    __shared__ float2 psum[kReducer ? 2 : 1][kReducer ? kLnRingThreads : 1];  // sum, M2 of a thread
    __shared__ LnStat stat[kReducer ? kLnMaxGroups : 1][2];
    const int gn = kReducer ? gt + 32 : gt;
    const int g = threadIdx.x / gn, t = threadIdx.x - g * gn, ng = blockDim.x / gn;
    const long long step = (long long)gridDim.x * ng;
    const long long first = (long long)blockIdx.x * ng + g;
    // columns before the row's first 16-byte boundary, vectors, columns after the
    // last; every lane of one warp has at most one column outside the vectors
    int head = kShift ? (int)(-(first * H) & (V - 1)) : 0;
    if (kShift && head > H) head = H;
    const int nvec = (H - head) / V, tail = H - head - nvec * V;
    const int el = threadIdx.x & 31;
    const int ec = !kShift ? -1 : el < head ? el : el >= 16 && el - 16 < tail ? H - tail + el - 16 : -1;
    const float ew = kShift && ec >= 0 ? to_f(__ldg(w + ec)) : 0.0f;
    const float eb = kShift && kBias && ec >= 0 ? to_f(__ldg(b + ec)) : 0.0f;
    auto edge = [&](long long i) {  // this lane's column of row i of the group
        return kShift && ec >= 0 && first + i * step < rows ? x[(first + i * step) * xs + ec] : T(0.0f);
    };
    auto store_edge = [&](long long i, float v, float m, float r) {
        if (kShift && ec >= 0) {
            v = (v - m) * r;
            y[(first + i * step) * H + ec] = from_f<T>(kBias ? fmaf(v, ew, eb) : v * ew);
        }
    };
    const float inv_h = 1.0f / (float)H;
    const long long n = first < rows ? (rows - first + step - 1) / step : 0;  // rows of this group
    if (kReducer && t >= gt) {
        // values per partial of this lane
        const int lane = t - gt, nw = gt >> 5;
        float cnt[kLnGroupWarps];
#pragma unroll
        for (int k = 0; k < kLnGroupWarps; ++k) {
            int c = 0;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int v = lane + 32 * k + i * gt;
                if (k < nw && v < nvec) c += V;
            }
            cnt[k] = (float)c;
        }
        T ex = T(0.0f);
        for (long long i = 0; i < n + kLag; ++i) {
            const T next = edge(i);  // its vectors' copies are under way
            if (i >= 1 && i <= n) {
                const float2* ps = psum[(i - 1) & 1] + g * gn;
                float2 v[kLnGroupWarps];
                float sum = 0.0f;
#pragma unroll
                for (int k = 0; k < kLnGroupWarps; ++k)
                    if (k < nw) {
                        v[k] = ps[lane + 32 * k];
                        sum += v[k].x;
                    }
                const float ef = kShift ? to_f(ex) : 0.0f;
                const float m = warp_sum(kShift ? sum + ef : sum) * inv_h;
                float q = kShift && ec >= 0 ? (ef - m) * (ef - m) : 0.0f;
#pragma unroll
                for (int k = 0; k < kLnGroupWarps; ++k)
                    if (k < nw && cnt[k] > 0.0f) {
                        const float d = __fdividef(v[k].x, cnt[k]) - m;
                        q += fmaf(cnt[k] * d, d, v[k].y);
                    }
                const float r = rsqrtf(fmaf(warp_sum(q), inv_h, eps));
                if (lane == 0) {
                    stat[g][(i - 1) & 1] = {m, r};
                    mean[first + (i - 1) * step] = m;
                    rstd[first + (i - 1) * step] = r;
                }
                store_edge(i - 1, ef, m, r);
            }
            ex = next;
            group_sync(g, gn);
        }
        return;
    }
    const uint32_t slot0 = smem_addr(ring) + threadIdx.x * 16u;
    const uint32_t vstride = blockDim.x * 16u;
    bool have[NV];
    int mine = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        have[i] = t + i * gt < nvec;
        mine += have[i] ? V : 0;
    }
    const float inv_mine = mine ? 1.0f / (float)mine : 0.0f;
    // the next row to copy: its number and this thread's first element of it
    long long frow = 0;
    const T* fx = x + first * xs + head + (size_t)t * V;
    auto fetch = [&](int s) {
        if (frow < n) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (have[i])
                    cp_async_16(slot0 + (uint32_t)(s * NV + i) * vstride, fx + (size_t)(i * gt) * V, 16u);
        }
        cp_async_commit();
        ++frow;
        fx += step * xs;
    };
    // rows in flight: the ring less the rows between arrival and output
    constexpr int kAhead = kRing - 1 - kLag;
#pragma unroll
    for (int s = 0; s < kAhead; ++s) fetch(s);
    f2 wv[NV][P], bv[kBias ? NV : 1][P];
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (have[i]) {
            const int c0 = (t + i * gt) * V + head;
            if constexpr (kShift) {
                load_each<W, P>(w + c0, wv[i]);
                if constexpr (kBias) load_each<W, P>(b + c0, bv[i]);
            } else {
                load_pairs<W, P>(w + c0, wv[i]);
                if constexpr (kBias) load_pairs<W, P>(b + c0, bv[i]);
            }
        }
    T* yr = y + first * H + head + (size_t)t * V;
    // (x - m) r w + b of the row in slot s
    auto output = [&](int s, float m, float r) {
        const f2 nm = f2_make(-m, -m), r2 = f2_make(r, r);
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (have[i]) {
                f2 v[P];
                unpack_vec<T, P>(ring[(s * NV + i) * blockDim.x + threadIdx.x], v);
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    v[j] = f2_mul(f2_add(v[j], nm), r2);
                    if constexpr (kBias)
                        v[j] = f2_fma(v[j], wv[i][j], bv[i][j]);
                    else
                        v[j] = f2_mul(v[j], wv[i][j]);
                }
                *reinterpret_cast<uint4*>(yr + (size_t)(i * gt) * V) = pack_vec<T, P>(v);
            }
        yr += step * H;
    };
    constexpr bool kEdge = kShift && !kReducer;
    T ex = kEdge ? edge(0) : T(0.0f);
    int s = 0;  // slot of row i
    for (long long i = 0; i < n + kLag; ++i) {
        cp_async_wait_group<kAhead - 1>();
        float sum = 0.0f, m2 = 0.0f;
        if (i < n) {
            const float ef = kEdge ? to_f(ex) : 0.0f;
            if constexpr (kEdge) ex = edge(i + 1);
            f2 v[NV][P];
            f2 acc[2] = {0ull, 0ull};  // (+0, +0)
#pragma unroll
            for (int k = 0; k < NV; ++k)
                if (have[k]) {
                    unpack_vec<T, P>(ring[(s * NV + k) * blockDim.x + threadIdx.x], v[k]);
#pragma unroll
                    for (int j = 0; j < P; ++j) acc[j & 1] = f2_add(acc[j & 1], v[k][j]);
                }
            sum = f2_sum(f2_add(acc[0], acc[1]));
            if constexpr (kEdge) sum += ef;
            // around the thread's own mean, or (one warp) the row's
            const float c = kReducer ? sum * inv_mine : warp_sum(sum) * inv_h;
            const f2 nc = f2_make(-c, -c);
            acc[0] = acc[1] = 0ull;
#pragma unroll
            for (int k = 0; k < NV; ++k)
                if (have[k]) {
#pragma unroll
                    for (int j = 0; j < P; ++j) v[k][j] = f2_add(v[k][j], nc);
#pragma unroll
                    for (int j = 0; j < P; ++j) acc[j & 1] = f2_fma(v[k][j], v[k][j], acc[j & 1]);
                }
            m2 = f2_sum(f2_add(acc[0], acc[1]));
            if (kEdge && ec >= 0) m2 = fmaf(ef - c, ef - c, m2);
            if constexpr (kReducer) {
                psum[i & 1][threadIdx.x] = make_float2(sum, m2);
            } else {
                const float r = rsqrtf(fmaf(warp_sum(m2), inv_h, eps));
                if (t == 0) {
                    mean[first + i * step] = c;
                    rstd[first + i * step] = r;
                }
                store_edge(i, ef, c, r);
                output(s, c, r);
            }
        }
        if constexpr (kReducer) {
            if (i >= 2) {
                const LnStat st = stat[g][i & 1];  // of row i - 2
                output((s + kRing - 2) % kRing, st.mean, st.rstd);
            }
        }
        fetch((s + kAhead) % kRing);
        if constexpr (kReducer) group_sync(g, gn);
        s = (s + 1) % kRing;
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

// Ring form.  The groups of a block leave their column sums in shared memory
// (the ring's, free by then) and the block adds them in the groups' order.
// kMode: LN_ONE_WARP groups of one warp, LN_REDUCER with a reducing warp, or
// LN_ALL_WARPS, for rows of which shared memory does not hold the two more that
// the reducing warp's lag takes (NV = 4): every warp reduces.
enum { LN_ONE_WARP, LN_REDUCER, LN_ALL_WARPS };
template <typename T, typename W, int NV, int kMode, bool kShift>
__global__ void __launch_bounds__(kLnRingThreads, 1) ln_bwd_ring(const LnBwd p, int gt) {
    constexpr bool kReducer = kMode == LN_REDUCER;
    constexpr int V = 16 / sizeof(T), P = V / 2, kRing = ln_bwd_ring_rows(NV), kLag = kReducer ? 2 : 0;
    constexpr bool kHoldW = NV * V <= 16;  // else the weight is read again from L1: its registers go to the sums
    extern __shared__ uint4 ring[];  // [kRing][2][NV][blockDim.x]: x, dy
    __shared__ float2 psum[kReducer ? 2 : 1][kReducer ? kLnRingThreads : 1];  // sums of g, g z of a thread
    __shared__ float2 tot[kReducer ? kLnMaxGroups : 1][2];                     // their means over the row
    __shared__ float2 red[kMode == LN_ALL_WARPS ? kLnMaxGroups : 1][2][kLnGroupWarps];
    const int gn = kReducer ? gt + 32 : gt;
    const int g = threadIdx.x / gn, t = threadIdx.x - g * gn, ng = blockDim.x / gn;
    const int H = p.H;
    const long long step = (long long)gridDim.x * ng;
    const long long first = (long long)blockIdx.x * ng + g;
    int head = kShift ? (int)(-(first * H) & (V - 1)) : 0;  // as in the forward
    if (kShift && head > H) head = H;
    const int nvec = (H - head) / V, tail = H - head - nvec * V;
    const long long n = first < p.rows ? (p.rows - first + step - 1) / step : 0;  // rows of this group
    const float inv_h = 1.0f / (float)H;
    const bool worker = !kReducer || t < gt;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the join: it waits for this grid's end
    bool have[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) have[i] = worker && t + i * gt < nvec;
    // the reducing (or the group's first) warp's lanes: a column outside the vectors
    const int el = threadIdx.x & 31;
    const int ec = !kShift || (kReducer ? worker : t >= 32)        ? -1
                   : el < head                                       ? el
                   : el >= 16 && el - 16 < tail ? H - tail + el - 16 : -1;
    const float ew = kShift && ec >= 0 ? to_f(__ldg(static_cast<const W*>(p.w) + ec)) : 0.0f;
    float esw = 0.0f, esb = 0.0f;
    auto edge = [&](const void* v, long long stride, long long i) {  // that column of row i of the group
        return kShift && ec >= 0 && i < n ? static_cast<const T*>(v)[(first + i * step) * stride + ec] : T(0.0f);
    };
    auto store_edge = [&](long long i, float z, float d, float r, float c1, float c2) {
        if (kShift && ec >= 0)
            static_cast<T*>(p.dx)[(first + i * step) * H + ec] = from_f<T>(fmaf(z, c2, fmaf(d, ew, c1)) * r);
    };
    f2 sw[NV][P], sb[NV][P];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < P; ++j) sw[i][j] = sb[i][j] = 0ull;  // (+0, +0)
    if (!worker) {
        const int lane = t - gt, nw = gt >> 5;
        T ex = T(0.0f), ed = T(0.0f);
        float em = 0.0f, er = 0.0f;  // of row i - 1
        for (long long i = 0; i < n + kLag; ++i) {
            const T nx = edge(p.x, p.xs, i), nd = edge(p.dy, p.dys, i);  // their vectors' copies are under way
            const bool load = kShift && ec >= 0 && i < n;
            const float nmean = load ? __ldg(p.mean + first + i * step) : 0.0f;
            const float nrstd = load ? __ldg(p.rstd + first + i * step) : 0.0f;
            if (i >= 1 && i <= n) {
                const float2* ps = psum[(i - 1) & 1] + g * gn;
                const float ez = kShift ? (to_f(ex) - em) * er : 0.0f, ef = kShift ? to_f(ed) : 0.0f;
                float a = ef * ew, c = a * ez;
                esb += ef;
                esw = fmaf(ef, ez, esw);
#pragma unroll
                for (int k = 0; k < kLnGroupWarps; ++k)
                    if (k < nw) {
                        const float2 v = ps[lane + 32 * k];
                        a += v.x;
                        c += v.y;
                    }
                a = warp_sum(a);
                c = warp_sum(c);
                if (lane == 0) tot[g][(i - 1) & 1] = make_float2(-a * inv_h, -c * inv_h);
                store_edge(i - 1, ez, ef, er, -a * inv_h, -c * inv_h);
            }
            ex = nx, ed = nd, em = nmean, er = nrstd;
            group_sync(g, gn);
        }
    } else {
        const uint32_t slot0 = smem_addr(ring) + threadIdx.x * 16u;
        const uint32_t vstride = blockDim.x * 16u;
        const W* w = static_cast<const W*>(p.w) + (t * V + head);
        long long frow = 0;
        const T* fx = static_cast<const T*>(p.x) + first * p.xs + head + (size_t)t * V;
        const T* fd = static_cast<const T*>(p.dy) + first * p.dys + head + (size_t)t * V;
        auto fetch = [&](int s) {
            if (frow < n) {
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    if (have[i]) {
                        const uint32_t dst = slot0 + (uint32_t)(s * 2 * NV + i) * vstride;
                        cp_async_16(dst, fx + (size_t)(i * gt) * V, 16u);
                        cp_async_16(dst + NV * vstride, fd + (size_t)(i * gt) * V, 16u);
                    }
            }
            cp_async_commit();
            ++frow;
            fx += step * p.xs;
            fd += step * p.dys;
        };
        constexpr int kAhead = kRing - 1 - kLag;
#pragma unroll
        for (int s = 0; s < kAhead; ++s) fetch(s);
        f2 wv[kHoldW ? NV : 1][P];
        auto load_w = [&](int i, f2 (&v)[P]) {
            if constexpr (kShift)
                load_each<W, P>(w + i * gt * V, v);
            else
                load_pairs<W, P>(w + i * gt * V, v);
        };
        if constexpr (kHoldW) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (have[i]) load_w(i, wv[i]);
        }
        T* out = static_cast<T*>(p.dx) + first * H + head + (size_t)t * V;
        // z and dy of vector i of the row in slot s (and the weight, where it is not held)
        auto vectors = [&](int s, int i, f2 nm, f2 r2, f2 (&z)[P], f2 (&d)[P]) {
            unpack_vec<T, P>(ring[(s * 2 * NV + i) * blockDim.x + threadIdx.x], z);
            unpack_vec<T, P>(ring[(s * 2 * NV + NV + i) * blockDim.x + threadIdx.x], d);
            if constexpr (!kHoldW) load_w(i, wv[0]);
#pragma unroll
            for (int j = 0; j < P; ++j) z[j] = f2_mul(f2_add(z[j], nm), r2);
        };
        // dx of the row in slot s; c1, c2: minus the means of g and of g z
        auto output = [&](int s, float m, float r, float c1, float c2) {
            const f2 nm = f2_make(-m, -m), r2 = f2_make(r, r), d1 = f2_make(c1, c1), d2 = f2_make(c2, c2);
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (have[i]) {
                    f2 z[P], d[P];
                    vectors(s, i, nm, r2, z, d);
#pragma unroll
                    for (int j = 0; j < P; ++j)
                        d[j] = f2_mul(f2_fma(z[j], d2, f2_fma(d[j], wv[kHoldW ? i : 0][j], d1)), r2);
                    *reinterpret_cast<uint4*>(out + (size_t)(i * gt) * V) = pack_vec<T, P>(d);
                }
            out += step * H;
        };
        // mean and rstd of rows i - 2 .. i + 1 (read a step ahead)
        float m0 = 0.0f, r0 = 0.0f, m1 = 0.0f, r1 = 0.0f, m = 0.0f, r = 0.0f, ma = 0.0f, ra = 0.0f;
        if (n > 0) m = __ldg(p.mean + first), r = __ldg(p.rstd + first);
        constexpr bool kEdge = kShift && !kReducer;
        T ex = kEdge ? edge(p.x, p.xs, 0) : T(0.0f), ed = kEdge ? edge(p.dy, p.dys, 0) : T(0.0f);
        int s = 0;  // slot of row i
        for (long long i = 0; i < n + kLag; ++i) {
            if (i + 1 < n) ma = __ldg(p.mean + first + (i + 1) * step), ra = __ldg(p.rstd + first + (i + 1) * step);
            cp_async_wait_group<kAhead - 1>();
            if (i < n) {
                const f2 nm = f2_make(-m, -m), r2 = f2_make(r, r);
                f2 a1 = 0ull, a2 = 0ull;
#pragma unroll
                for (int k = 0; k < NV; ++k)
                    if (have[k]) {
                        f2 z[P], d[P];
                        vectors(s, k, nm, r2, z, d);
#pragma unroll
                        for (int j = 0; j < P; ++j) {
                            sb[k][j] = f2_add(sb[k][j], d[j]);
                            sw[k][j] = f2_fma(d[j], z[j], sw[k][j]);
                            d[j] = f2_mul(d[j], wv[kHoldW ? k : 0][j]);
                            a1 = f2_add(a1, d[j]);
                            a2 = f2_fma(d[j], z[j], a2);
                        }
                    }
                if constexpr (kReducer) {
                    psum[i & 1][threadIdx.x] = make_float2(f2_sum(a1), f2_sum(a2));
                } else {
                    float p1 = f2_sum(a1), p2 = f2_sum(a2), ez = 0.0f, ef = 0.0f;
                    if constexpr (kEdge) {
                        ez = (to_f(ex) - m) * r;
                        ef = to_f(ed);
                        ex = edge(p.x, p.xs, i + 1);
                        ed = edge(p.dy, p.dys, i + 1);
                        if (ec < 0) ez = 0.0f;
                        esb += ef;
                        esw = fmaf(ef, ez, esw);
                        p1 = fmaf(ef, ew, p1);
                        p2 = fmaf(ef * ew, ez, p2);
                    }
                    float c1 = warp_sum(p1), c2 = warp_sum(p2);
                    if constexpr (kMode == LN_ALL_WARPS) {
                        // two buffers in turn: row i + 2 reuses this one, after row i + 1's barrier
                        const int lane = t & 31;
                        if (lane == 0) red[g][i & 1][t >> 5] = make_float2(c1, c2);
                        group_sync(g, gt);
                        const float2 v = lane < (gt >> 5) ? red[g][i & 1][lane] : make_float2(0.0f, 0.0f);
                        c1 = warp_sum(v.x);
                        c2 = warp_sum(v.y);
                    }
                    store_edge(i, ez, ef, r, -c1 * inv_h, -c2 * inv_h);
                    output(s, m, r, -c1 * inv_h, -c2 * inv_h);
                }
            }
            if constexpr (kReducer) {
                if (i >= 2) {
                    const float2 c = tot[g][i & 1];  // of row i - 2
                    output((s + kRing - 2) % kRing, m0, r0, c.x, c.y);
                }
            }
            fetch((s + kAhead) % kRing);
            m0 = m1, r0 = r1, m1 = m, r1 = r, m = ma, r = ra;
            if constexpr (kReducer) group_sync(g, gn);
            s = (s + 1) % kRing;
        }
    }
    float* part = p.part + (size_t)blockIdx.x * 2 * H;
    float* col = reinterpret_cast<float*>(ring) + (size_t)g * 2 * H;  // [groups][2][H]
    static_assert(kRing * 2 * 16 >= 2 * V * 4, "the ring holds the groups' column sums");
    float* to = ng > 1 ? col : part;
    cp_async_wait_all();
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (have[i]) {
#pragma unroll
            for (int j = 0; j < P; ++j) {
                const int h = (t + i * gt) * V + head + 2 * j;
                const float2 a = f2_get(sw[i][j]), b = f2_get(sb[i][j]);
                if constexpr (kShift) {
                    to[h] = a.x, to[H + h] = b.x;
                    to[h + 1] = a.y, to[H + h + 1] = b.y;
                } else {
                    *reinterpret_cast<float2*>(to + h) = a;
                    *reinterpret_cast<float2*>(to + H + h) = b;
                }
            }
        }
    if (kShift && ec >= 0) to[ec] = esw, to[H + ec] = esb;
    if (ng > 1) {
        __syncthreads();
        for (int h = threadIdx.x; h < 2 * H; h += blockDim.x) {
            float a = reinterpret_cast<const float*>(ring)[h];
            for (int gi = 1; gi < ng; ++gi) a += reinterpret_cast<const float*>(ring)[(size_t)gi * 2 * H + h];
            part[h] = a;
        }
    }
}

// Register form.  One warp per row: the block's warps join their column sums
// through shared memory at the end.
template <typename T, typename W, int NV, bool kWarpRow>
__global__ void __launch_bounds__(kWarpRow ? 32 * kLnWarps : 512) ln_bwd(const LnBwd p) {
    __shared__ float red[2][32];
    __shared__ float colsum[kWarpRow ? 2 * 32 * NV : 1];  // one warp per row: [2][H]
    const int t = kWarpRow ? (int)(threadIdx.x & 31) : (int)threadIdx.x;
    const int nt = kWarpRow ? 32 : (int)blockDim.x;
    const int H = p.H;
    const T *dy = static_cast<const T*>(p.dy), *x = static_cast<const T*>(p.x);
    const W* w = static_cast<const W*>(p.w);
    T* dx = static_cast<T*>(p.dx);
    float sw[NV], sb[NV], wv[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        sw[i] = sb[i] = 0.0f;
        wv[i] = t + i * nt < H ? to_f(__ldg(w + t + i * nt)) : 0.0f;
    }
    const long long step = kWarpRow ? (long long)gridDim.x * kLnWarps : (long long)gridDim.x;
    const long long first = kWarpRow ? (long long)blockIdx.x * kLnWarps + (threadIdx.x >> 5) : (long long)blockIdx.x;
    for (long long row = first; row < p.rows; row += step) {
        const float m = __ldg(p.mean + row), r = __ldg(p.rstd + row);
        float z[NV], g[NV];
        float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = t + i * nt;
            z[i] = c < H ? to_f(__ldg(x + row * p.xs + c)) : 0.0f;
            g[i] = c < H ? to_f(__ldg(dy + row * p.dys + c)) : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (t + i * nt < H) {
                z[i] = (z[i] - m) * r;
                sb[i] += g[i];
                sw[i] = fmaf(g[i], z[i], sw[i]);
                g[i] *= wv[i];
                s1 += g[i];
                s2 = fmaf(g[i], z[i], s2);
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
        for (int i = 0; i < NV; ++i)
            if (t + i * nt < H) dx[row * (long long)H + t + i * nt] = from_f<T>(r * (g[i] - c1 - z[i] * c2));
    }
    float* out = p.part + (size_t)blockIdx.x * 2 * H;
    if constexpr (kWarpRow) {
        // warp after warp in a fixed order
        for (int wi = 0; wi < kLnWarps; ++wi) {
            if ((int)(threadIdx.x >> 5) == wi) {
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int h = t + i * 32;
                    if (h < H) {
                        colsum[h] = wi ? colsum[h] + sw[i] : sw[i];
                        colsum[H + h] = wi ? colsum[H + h] + sb[i] : sb[i];
                    }
                }
            }
            __syncthreads();
        }
        for (int h = threadIdx.x; h < 2 * H; h += blockDim.x) out[h] = colsum[h];
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (t + i * nt < H) {
                out[t + i * nt] = sw[i];
                out[H + t + i * nt] = sb[i];
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
__global__ void __launch_bounds__(256) ln_bwd_join(const float* part, int nb, int H, W* __restrict__ dw,
                                                   W* __restrict__ db) {
    __shared__ float s[8][33];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31, k = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + lane;  // of 2 H
    float a = 0.0f;
    if (col < 2 * H) {
        int i = k;
        for (; i + 56 < nb; i += 64) {  // eight loads in flight
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = part[(size_t)(i + 8 * j) * 2 * H + col];
#pragma unroll
            for (int j = 0; j < 8; ++j) a += v[j];
        }
        for (; i < nb; i += 8) a += part[(size_t)i * 2 * H + col];
    }
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

// Launch shape of a call: form, vectors (or elements) per thread, threads of
// a group (ring), of a row's block or of a block of warps (register).
enum { LN_RING, LN_WARP, LN_BLOCK, LN_LONG };
struct LnForm {
    int form, nv, threads;
    bool shift;  // ring: rows start between 16-byte boundaries
};
// Whether the ring form can take rows of width H, its tensors' rows `stride`
// apart and starting at p: rows of all tensors start equally far past a 16-byte
// boundary.
bool ring_rows(const void* p, long long stride, int H, int elt) {
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (stride - H) * elt % 16 == 0;
}
// Blocks of a ring launch: up to one per SM, and a multiple of 8 for shifted
// rows (152 is one).
int ring_blocks(long long need, bool shift) {
    if (need > 152) need = 152;
    return (int)(shift ? (need + 7) / 8 * 8 : need);
}
LnForm ln_form(int H, int elt, bool vec, int max_threads, int wide_nv, int max_ring) {
    LnForm f = {};
    if (vec) {
        const int V = 16 / elt;
        f.shift = H % V != 0;
        const int nvec = H >= V ? H / V : 1;  // whole ones, at most
        f.form = LN_RING;
        f.nv = nvec <= 32 ? 1 : nvec <= 64 ? 2 : nvec <= 2 * (kLnRingThreads - 32) ? wide_nv : 4;
        f.threads = ((nvec + f.nv - 1) / f.nv + 31) / 32 * 32;
        if (f.threads > max_ring) f.form = LN_LONG;
        return f;
    }
    if (H <= 128) {
        f.form = LN_WARP;
        f.nv = H <= 32 ? 1 : H <= 64 ? 2 : 4;
        f.threads = 32 * kLnWarps;
        return f;
    }
    f.form = LN_BLOCK;
    for (f.nv = 4; f.nv <= 16; f.nv *= 2) {
        f.threads = ((H + f.nv - 1) / f.nv + 31) / 32 * 32;
        if (f.threads <= max_threads) return f;
    }
    f.form = LN_LONG;
    return f;
}

bool mult16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Groups of a block and its threads; named barriers 1..15 tell groups of
// several warps apart.
int ln_groups(int gt, bool reducer, int* threads) {
    const int gn = reducer ? gt + 32 : gt;
    int ng = kLnRingThreads / gn;
    if (gt > 32 && ng > 15) ng = 15;
    *threads = ng * gn;
    return ng;
}
// Shifted rows load their weights one by one: a group that takes few rows does
// not earn that back.  us, ring | register form, at rows per group:
//   forward, groups of several warps: 1.0 8.4 | 6.8 (300 x 7161 bf16), 1.6 7.4 |
//   10.0 (500 x 5001 bf16)
//   forward, groups of one warp (2432 of them), by width:
//      333 bf16   1.6  5.4 |  4.9   2.0  5.5 |  5.7   2.8  6.4 |  7.1   3.2  7.4 |  7.9
//      777 bf16   1.6 10.1 |  9.6   2.0 10.7 | 12.1   2.8 13.2 | 16.1   3.2 15.2 | 18.0
//     1001 f16    1.6 11.8 | 10.8   2.0 12.4 | 13.2   2.8 15.0 | 17.4   3.2 17.1 | 19.4
//      251 f32    2.0  4.6 |  4.7   2.8  6.2 |  6.1   3.2  7.0 |  6.8   4.0  7.5 |  7.9
//       33 bf16   2.0  3.2 |  1.9   3.2  4.8 |  2.7   4.0  4.8 |  2.9   6.0  6.1 |  3.8
//   (from 333 columns on two rows would do; at 33 the register form stays ahead)
//   backward: 1.0 9.8 | 7.2 (777 x 1001 f16), 1.6 10.6 | 15.1 (4000 x 333 bf16)
bool ring_pays(const LnForm& f, bool reducer, long long rows, int half_rows) {
    int threads;
    return f.form != LN_RING || !f.shift || 2 * rows >= half_rows * 152ll * ln_groups(f.threads, reducer, &threads);
}
template <typename T, typename W, int NV, bool kBias, bool kReducer, bool kShift>
int run_fwd_ring(const LnForm& f, const LnFwdArgs& a, cudaStream_t st) {
    static SmemLimit limit;
    int threads;
    const int ng = ln_groups(f.threads, kReducer, &threads);
    constexpr int per_thread = kLnFwdRing * NV * 16;
    static_assert(per_thread * kLnRingThreads <= 200 * 1024, "shared memory per block");
    if (const int e = limit.allow(ln_fwd_ring<T, W, NV, kBias, kReducer, kShift>, per_thread * kLnRingThreads)) return e;
    const long long need = (a.rows + ng - 1) / ng;
    trace_pre(st);
    ln_fwd_ring<T, W, NV, kBias, kReducer, kShift><<<ring_blocks(need, kShift), threads, per_thread * threads, st>>>(
        a.rows, a.H, f.threads, static_cast<const T*>(a.x), a.x_stride, static_cast<const W*>(a.weight),
        static_cast<const W*>(a.bias), a.eps, static_cast<T*>(a.y), a.mean, a.rstd);
    trace_post(st, "layer_norm_fwd");
    return (int)cudaGetLastError();
}
template <typename T, typename W, bool kBias, bool kShift>
int fwd_ring(const LnForm& f, const LnFwdArgs& a, cudaStream_t st) {
    if (f.nv == 1) return run_fwd_ring<T, W, 1, kBias, false, kShift>(f, a, st);
    if (f.nv == 2) return run_fwd_ring<T, W, 2, kBias, false, kShift>(f, a, st);
    return f.threads > 32 ? run_fwd_ring<T, W, 4, kBias, true, kShift>(f, a, st)
                          : run_fwd_ring<T, W, 4, kBias, false, kShift>(f, a, st);
}
template <typename T, typename W, int NV, bool kWarpRow>
int run_fwd(const LnForm& f, const LnFwdArgs& a, cudaStream_t st) {
    const long long blocks = kWarpRow ? (a.rows + kLnWarps - 1) / kLnWarps : a.rows;
    trace_pre(st);
    ln_fwd<T, W, NV, kWarpRow><<<(unsigned)blocks, f.threads, 0, st>>>(
        a.rows, a.H, static_cast<const T*>(a.x), a.x_stride, static_cast<const W*>(a.weight),
        static_cast<const W*>(a.bias), a.eps, static_cast<T*>(a.y), a.mean, a.rstd);
    trace_post(st, "layer_norm_fwd");
    return (int)cudaGetLastError();
}
template <typename T, typename W, int V>
int run_fwd_long(const LnFwdArgs& a, cudaStream_t st) {
    trace_pre(st);
    ln_fwd_long<T, W, V><<<(unsigned)a.rows, kLnLongThreads, 0, st>>>(
        a.rows, a.H, static_cast<const T*>(a.x), a.x_stride, static_cast<const W*>(a.weight),
        static_cast<const W*>(a.bias), a.eps, static_cast<T*>(a.y), a.mean, a.rstd);
    trace_post(st, "layer_norm_fwd");
    return (int)cudaGetLastError();
}
template <typename T, typename W>
int fwd_t(const LnFwdArgs& a, cudaStream_t st) {
    constexpr int V = 16 / sizeof(T);
    const bool ring = ring_rows(a.x, a.x_stride, a.H, sizeof(T)) && ring_rows(a.y, a.H, a.H, sizeof(T)) &&
                      (a.H % V || (mult16(a.weight) && mult16(a.bias)));
    const bool vec = ring && a.H % V == 0;
    LnForm f = ln_form(a.H, sizeof(T), ring, 1024, 4, kLnRingThreads - 32);
    if (!ring_pays(f, f.threads > 32, a.rows, f.threads > 32 ? 3 : 6)) f = ln_form(a.H, sizeof(T), false, 1024, 4, 0);
    const bool b = a.bias != nullptr;
    switch (f.form) {
        case LN_RING:
            if (f.shift) return b ? fwd_ring<T, W, true, true>(f, a, st) : fwd_ring<T, W, false, true>(f, a, st);
            return b ? fwd_ring<T, W, true, false>(f, a, st) : fwd_ring<T, W, false, false>(f, a, st);
        case LN_WARP:
            return f.nv == 1   ? run_fwd<T, W, 1, true>(f, a, st)
                   : f.nv == 2 ? run_fwd<T, W, 2, true>(f, a, st)
                               : run_fwd<T, W, 4, true>(f, a, st);
        case LN_BLOCK:
            return f.nv == 4   ? run_fwd<T, W, 4, false>(f, a, st)
                   : f.nv == 8 ? run_fwd<T, W, 8, false>(f, a, st)
                               : run_fwd<T, W, 16, false>(f, a, st);
        default: return vec ? run_fwd_long<T, W, V>(a, st) : run_fwd_long<T, W, 1>(a, st);
    }
}

template <typename T, typename W, int NV, int kMode, bool kShift>
int run_bwd_ring(const LnForm& f, const LnBwd& p, int* blocks, cudaStream_t st) {
    static SmemLimit limit;
    int threads;
    const int ng = ln_groups(f.threads, kMode == LN_REDUCER, &threads);
    constexpr int per_thread = ln_bwd_ring_rows(NV) * 2 * NV * 16;
    static_assert(per_thread * kLnRingThreads <= 200 * 1024, "shared memory per block");
    if (const int e = limit.allow(ln_bwd_ring<T, W, NV, kMode, kShift>, per_thread * kLnRingThreads)) return e;
    const long long need = (p.rows + ng - 1) / ng;
    *blocks = ring_blocks(need, kShift);
    trace_pre(st);
    ln_bwd_ring<T, W, NV, kMode, kShift><<<*blocks, threads, per_thread * threads, st>>>(p, f.threads);
    trace_post(st, "layer_norm_bwd");
    return (int)cudaGetLastError();
}
template <typename T, typename W, bool kShift>
int bwd_ring(const LnForm& f, const LnBwd& p, int* blocks, cudaStream_t st) {
    return f.nv == 1        ? run_bwd_ring<T, W, 1, LN_ONE_WARP, kShift>(f, p, blocks, st)
           : f.nv > 2       ? run_bwd_ring<T, W, 4, LN_ALL_WARPS, kShift>(f, p, blocks, st)
           : f.threads > 32 ? run_bwd_ring<T, W, 2, LN_REDUCER, kShift>(f, p, blocks, st)
                            : run_bwd_ring<T, W, 2, LN_ONE_WARP, kShift>(f, p, blocks, st);
}
template <typename T, typename W, int NV, bool kWarpRow>
int run_bwd(const LnForm& f, const LnBwd& p, int* blocks, cudaStream_t st) {
    const long long need = kWarpRow ? (p.rows + kLnWarps - 1) / kLnWarps : p.rows;
    *blocks = (int)(need < kLnBwdBlocks ? need : kLnBwdBlocks);
    trace_pre(st);
    ln_bwd<T, W, NV, kWarpRow><<<*blocks, f.threads, 0, st>>>(p);
    trace_post(st, "layer_norm_bwd");
    return (int)cudaGetLastError();
}
template <typename T, typename W, int V>
int run_bwd_long(const LnBwd& p, int* blocks, cudaStream_t st) {
    *blocks = (int)(p.rows < kLnBwdBlocks ? p.rows : kLnBwdBlocks);  // bands of rows
    trace_pre(st);
    ln_bwd_long<T, W, V><<<(unsigned)p.rows, kLnLongThreads, 0, st>>>(p);
    trace_post(st, "layer_norm_bwd");
    if (const cudaError_t e = cudaGetLastError()) return (int)e;
    trace_pre(st);
    ln_bwd_long_cols<T><<<dim3((p.H + 255) / 256, *blocks), 256, 0, st>>>(p, *blocks);
    trace_post(st, "layer_norm_bwd_cols");
    return (int)cudaGetLastError();
}
template <typename T, typename W>
int bwd_t(const LnBwdArgs& a, cudaStream_t st) {
    constexpr int V = 16 / sizeof(T);
    const bool ring = ring_rows(a.x, a.x_stride, a.H, sizeof(T)) && ring_rows(a.dy, a.dy_stride, a.H, sizeof(T)) &&
                      ring_rows(a.dx, a.H, a.H, sizeof(T)) && (a.H % V || mult16(a.weight));
    const bool vec = ring && a.H % V == 0;
    const LnBwd p = {a.rows, a.H, a.dy, a.x, a.weight, a.dy_stride, a.x_stride, a.mean, a.rstd, a.dx, a.part};
    LnForm f = ln_form(a.H, sizeof(T), ring, 512, 2, kLnRingThreads);
    if (!ring_pays(f, f.nv == 2 && f.threads > 32, a.rows, 3)) f = ln_form(a.H, sizeof(T), false, 512, 2, 0);
    int e, blocks = 0;
    switch (f.form) {
        case LN_RING:
            e = f.shift ? bwd_ring<T, W, true>(f, p, &blocks, st) : bwd_ring<T, W, false>(f, p, &blocks, st);
            break;
        case LN_WARP:
            e = f.nv == 1   ? run_bwd<T, W, 1, true>(f, p, &blocks, st)
                : f.nv == 2 ? run_bwd<T, W, 2, true>(f, p, &blocks, st)
                            : run_bwd<T, W, 4, true>(f, p, &blocks, st);
            break;
        case LN_BLOCK:
            e = f.nv == 4   ? run_bwd<T, W, 4, false>(f, p, &blocks, st)
                : f.nv == 8 ? run_bwd<T, W, 8, false>(f, p, &blocks, st)
                            : run_bwd<T, W, 16, false>(f, p, &blocks, st);
            break;
        default: e = vec ? run_bwd_long<T, W, V>(p, &blocks, st) : run_bwd_long<T, W, 1>(p, &blocks, st);
    }
    if (e) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((2 * a.H + 31) / 32);
    cfg.blockDim = dim3(256);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    trace_pre(st);
    const cudaError_t ce = cudaLaunchKernelEx(&cfg, ln_bwd_join<W>, (const float*)a.part, blocks, a.H,
                                              static_cast<W*>(a.dweight), static_cast<W*>(a.dbias));
    trace_post(st, "layer_norm_bwd_join");
    return (int)(ce != cudaSuccess ? ce : cudaGetLastError());
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
