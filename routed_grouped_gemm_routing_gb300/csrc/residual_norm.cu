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
// column sums stay in its registers for the life of the block).  The rows to come
// are copied ahead by cp.async into a ring of shared memory: rows that lie on
// 16-byte boundaries by the thread that will read them, others as the whole
// 16-byte pieces around them (kVec false), read element by element after the
// group's barrier.  The parameters come from L1, which the ring's depth leaves
// room for.  Rows of more than 7168 columns are read again for every pass.
//
// Column sums: one row of partial sums a block, joined in a fixed order by a
// second kernel (deterministic, no atomics).
#include <cuda_fp16.h>

#include "moe_internal.h"
#include "ptx.cuh"
#include "smem_limit.h"

namespace moe {

namespace {

constexpr int kRnThreads = 896;  // of a block: 72 registers each
constexpr int kRnCols = 8;       // columns of a thread
constexpr int kRnMaxH = kRnThreads * kRnCols;
constexpr int kRnLongThreads = 1024;

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
    template <int V>
    __device__ __forceinline__ void load(int c, float (&f)[V]) const {
        if constexpr (V == 1) {
            f[0] = at(c);
        } else if (f32) {
#pragma unroll
            for (int i = 0; i < V / 4; ++i) {
                const float4 v = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p) + c) + i);
                f[4 * i] = v.x, f[4 * i + 1] = v.y, f[4 * i + 2] = v.z, f[4 * i + 3] = v.w;
            }
        } else {
            const uint4 u = __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(p) + c));
            const T* t = reinterpret_cast<const T*>(&u);
#pragma unroll
            for (int i = 0; i < V; ++i) f[i] = to_f(t[i]);
        }
    }
};

// A group of a block: nt threads that take one row at a time.
struct Group {
    int id, t, nt, warps, warp;  // warp: within the group
    float2* red;                 // two buffers of warps values
    int turn;
    __device__ __forceinline__ void sync() const {
        if (warps == 1)
            __syncwarp();
        else
            asm volatile("bar.sync %0, %1;" ::"r"(1 + id), "r"(nt) : "memory");
    }
    // Sums of a and b over the group, in the same order in every thread.
    __device__ __forceinline__ float2 sum(float a, float b) {
        a = warp_sum(a);
        b = warp_sum(b);
        if (warps == 1) return make_float2(a, b);
        const int lane = threadIdx.x & 31;
        float2* r = red + turn * 32;
        turn ^= 1;
        if (lane == 0) r[warp] = make_float2(a, b);
        sync();
        const float2 v = lane < warps ? r[lane] : make_float2(0.0f, 0.0f);
        return make_float2(warp_sum(v.x), warp_sum(v.y));
    }
    __device__ __forceinline__ float sum(float a) {
        a = warp_sum(a);
        if (warps == 1) return a;
        const int lane = threadIdx.x & 31;
        float2* r = red + turn * 32;
        turn ^= 1;
        if (lane == 0) r[warp].x = a;
        sync();
        return warp_sum(lane < warps ? r[lane].x : 0.0f);
    }
};

// The ring of one group: stages of kTensors rows.
template <typename T, bool kVec, int kTensors>
struct Ring {
    static constexpr int V = kVec ? 16 / (int)sizeof(T) : 1, NV = kRnCols / V;
    uint8_t* base;  // the group's
    int row_bytes, stages, H, t, nt;
    __device__ __forceinline__ uint8_t* slot(int stage, int k) const { return base + (stage * kTensors + k) * row_bytes; }
    __device__ __forceinline__ static int shift(const T* row) { return kVec ? 0 : (int)(reinterpret_cast<uintptr_t>(row) & 15); }
    __device__ __forceinline__ void fetch(int stage, int k, const T* row) const {
        if (!row) return;
        const uint32_t dst = smem_addr(slot(stage, k));
        if constexpr (kVec) {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = (t + j * nt) * V;
                if (c < H) cp_async_16(dst + c * (int)sizeof(T), row + c, 16);
            }
        } else {
            // the 16-byte pieces that hold the row: those around it lie in the same
            // pieces as its ends, and nothing behind its last byte is read
            const int s = shift(row), bytes = s + H * (int)sizeof(T);
            const uint8_t* src = reinterpret_cast<const uint8_t*>(row) - s;
            for (int c = 16 * t; c < bytes; c += 16 * nt) cp_async_16(dst + c, src + c, bytes - c < 16 ? bytes - c : 16);
        }
    }
    // The thread's columns j * V .. of tensor k; zeros past the row and for a tensor that is not there.
    __device__ __forceinline__ void read(int stage, int k, const T* row, int j, float (&f)[V]) const {
        const int c = (t + j * nt) * V;
        if (!row || c >= H) {
#pragma unroll
            for (int i = 0; i < V; ++i) f[i] = 0.0f;
            return;
        }
        if constexpr (kVec) {
            const uint4 u = *reinterpret_cast<const uint4*>(slot(stage, k) + c * (int)sizeof(T));
            const T* e = reinterpret_cast<const T*>(&u);
#pragma unroll
            for (int i = 0; i < V; ++i) f[i] = to_f(e[i]);
        } else {
            f[0] = to_f(*reinterpret_cast<const T*>(slot(stage, k) + shift(row) + c * (int)sizeof(T)));
        }
    }
    __device__ __forceinline__ void write(T* row, int j, const float (&f)[V]) const {
        const int c = (t + j * nt) * V;
        if (c >= H) return;
        if constexpr (kVec) {
            uint4 u;
            T* e = reinterpret_cast<T*>(&u);
#pragma unroll
            for (int i = 0; i < V; ++i) e[i] = from_f<T>(f[i]);
            *reinterpret_cast<uint4*>(row + c) = u;
        } else {
            row[c] = from_f<T>(f[0]);
        }
    }
    __device__ __forceinline__ bool in(int j) const { return (t + j * nt) * V < H; }
    __device__ __forceinline__ int col(int j) const { return (t + j * nt) * V; }
};

// Waits for the oldest of `stages` - 1 copies in flight.
__device__ __forceinline__ void ring_wait(int stages) {
    if (stages == 2)
        cp_async_wait_group<0>();
    else if (stages == 3)
        cp_async_wait_group<1>();
    else
        cp_async_wait_group<2>();
}

struct RnShape {
    long long rows;
    int H, rms, gate, w_f32;
    float alpha, eps, inv;  // inv: 1 / H
    int groups, nt, row_bytes, stages;
};
struct RnFwd {
    RnShape s;
    const void *o, *r;
    long long os, rs;
    const void *g, *pw, *pb, *w, *b;
    void *stream, *normed;
    float* stats;  // [4][rows]: mean and rstd of o, mean and rstd of s
};

template <typename T, bool kVec, bool kPost>
__global__ void __launch_bounds__(kRnThreads) rn_fwd_kernel(const RnFwd p) {
    using R = Ring<T, kVec, 2>;
    constexpr int V = R::V, NV = R::NV;
    extern __shared__ __align__(16) uint8_t smem[];
    const RnShape& s = p.s;
    const int id = (int)threadIdx.x / s.nt, t = (int)threadIdx.x - id * s.nt;
    Group grp = {id, t, s.nt, s.nt >> 5, t >> 5, reinterpret_cast<float2*>(smem) + id * 64, 0};
    const R ring = {smem + s.groups * 512 + id * s.stages * 2 * s.row_bytes, s.row_bytes, s.stages, s.H, t, s.nt};
    const T *o = static_cast<const T*>(p.o), *r = static_cast<const T*>(p.r);
    const Param<T> pw = {p.pw, s.w_f32}, pb = {p.pb, s.w_f32}, w = {p.w, s.w_f32}, b = {p.b, s.w_f32}, g = {p.g, s.w_f32};
    const long long step = (long long)gridDim.x * s.groups, row0 = (long long)blockIdx.x * s.groups + id;
    for (int i = 0; i < s.stages - 1; ++i) {
        const long long row = row0 + i * step;
        if (row < s.rows) ring.fetch(i, 0, o + row * p.os), ring.fetch(i, 1, r + row * p.rs);
        cp_async_commit();
    }
    int stage = 0;
    for (long long row = row0; row < s.rows; row += step) {
        ring_wait(s.stages);
        if (!kVec) grp.sync();
        {
            const long long next = row + (s.stages - 1) * step;
            const int at = stage == 0 ? s.stages - 1 : stage - 1;
            if (next < s.rows) ring.fetch(at, 0, o + next * p.os), ring.fetch(at, 1, r + next * p.rs);
            cp_async_commit();
        }
        const T *orow = o + row * p.os, *rrow = r + row * p.rs;
        float v[NV][V];
#pragma unroll
        for (int j = 0; j < NV; ++j) ring.read(stage, 0, orow, j, v[j]);
        if constexpr (kPost) {
            float mean = 0.0f, sq = 0.0f;
            if (!s.rms) {
                float a = 0.0f;
#pragma unroll
                for (int j = 0; j < NV; ++j)
#pragma unroll
                    for (int i = 0; i < V; ++i) a += v[j][i];
                mean = grp.sum(a) * s.inv;
            }
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float d = ring.in(j) ? v[j][i] - mean : 0.0f;
                    sq += d * d;
                }
            const float rstd = rsqrtf(grp.sum(sq) * s.inv + s.eps);
            if (t == 0) p.stats[row] = mean, p.stats[s.rows + row] = rstd;
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                if (!ring.in(j)) continue;
                float f[V], c[V] = {};
                pw.template load<V>(ring.col(j), f);
                if (p.pb) pb.template load<V>(ring.col(j), c);
#pragma unroll
                for (int i = 0; i < V; ++i) v[j][i] = (v[j][i] - mean) * rstd * f[i] + c[i];
            }
        }
        const float gt = s.gate == MOE_GATE_TOKEN ? g.at((int)row) : 1.0f;
        float a = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            float f[V];
            ring.read(stage, 1, rrow, j, f);
            if (s.gate == MOE_GATE_CHANNEL) {
                float c[V] = {};
                if (ring.in(j)) g.template load<V>(ring.col(j), c);
#pragma unroll
                for (int i = 0; i < V; ++i) v[j][i] *= c[i];
            }
#pragma unroll
            for (int i = 0; i < V; ++i) {
                v[j][i] = s.alpha * f[i] + gt * v[j][i];
                a += v[j][i];
            }
            ring.write(static_cast<T*>(p.stream) + row * s.H, j, v[j]);
        }
        const float mean = s.rms ? 0.0f : grp.sum(a) * s.inv;
        float sq = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float d = ring.in(j) ? v[j][i] - mean : 0.0f;
                sq += d * d;
            }
        const float rstd = rsqrtf(grp.sum(sq) * s.inv + s.eps);
        if (t == 0) p.stats[2 * s.rows + row] = mean, p.stats[3 * s.rows + row] = rstd;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if (!ring.in(j)) continue;
            float f[V], c[V] = {};
            w.template load<V>(ring.col(j), f);
            if (p.b) b.template load<V>(ring.col(j), c);
#pragma unroll
            for (int i = 0; i < V; ++i) f[i] = (v[j][i] - mean) * rstd * f[i] + c[i];
            ring.write(static_cast<T*>(p.normed) + row * s.H, j, f);
        }
        if (++stage == s.stages) stage = 0;
    }
    cp_async_wait_all();
}

// ---------------------------------------------------------------- backward
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
};

// What one row's scalars are: its statistics and its gate.
struct RnRow {
    float om, ors, m, rs, gt;
};

template <typename T, bool kVec, bool kPost>
__global__ void __launch_bounds__(kRnThreads) rn_bwd_kernel(const RnBwd p) {
    using R = Ring<T, kVec, 4>;
    constexpr int V = R::V, NV = R::NV;
    extern __shared__ __align__(16) uint8_t smem[];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const RnShape& s = p.s;
    const int id = (int)threadIdx.x / s.nt, t = (int)threadIdx.x - id * s.nt;
    Group grp = {id, t, s.nt, s.nt >> 5, t >> 5, reinterpret_cast<float2*>(smem) + id * 64, 0};
    uint8_t* rings = smem + s.groups * 512;
    const R ring = {rings + id * s.stages * 4 * s.row_bytes, s.row_bytes, s.stages, s.H, t, s.nt};
    const T *o = static_cast<const T*>(p.o), *r = static_cast<const T*>(p.r), *ds = static_cast<const T*>(p.ds),
            *dn = static_cast<const T*>(p.dn);
    const Param<T> pw = {p.pw, s.w_f32}, pb = {p.pb, s.w_f32}, w = {p.w, s.w_f32}, g = {p.g, s.w_f32};
    const long long step = (long long)gridDim.x * s.groups, row0 = (long long)blockIdx.x * s.groups + id;
    auto fetch = [&](int at, long long row) {
        if (row < s.rows) {
            ring.fetch(at, 0, o + row * p.os);
            ring.fetch(at, 1, r + row * p.rs);
            ring.fetch(at, 2, dn ? dn + row * p.dns : nullptr);
            ring.fetch(at, 3, ds ? ds + row * p.dss : nullptr);
        }
        cp_async_commit();
    };
    auto scalars = [&](long long row) {
        RnRow c = {0.0f, 1.0f, 0.0f, 0.0f, 1.0f};
        if (row >= s.rows) return c;
        if (kPost) {
            c.om = __ldg(p.stats + row);
            c.ors = __ldg(p.stats + s.rows + row);
        }
        c.m = __ldg(p.stats + 2 * s.rows + row);
        c.rs = __ldg(p.stats + 3 * s.rows + row);
        if (s.gate == MOE_GATE_TOKEN) c.gt = g.at((int)row);
        return c;
    };
    for (int i = 0; i < s.stages - 1; ++i) fetch(i, row0 + i * step);
    float acc[4][NV][V];
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) acc[k][j][i] = 0.0f;
    RnRow next = scalars(row0);
    int stage = 0;
    for (long long row = row0; row < s.rows; row += step) {
        const RnRow c = next;
        ring_wait(s.stages);
        if (!kVec) grp.sync();
        fetch(stage == 0 ? s.stages - 1 : stage - 1, row + (s.stages - 1) * step);
        next = scalars(row + step);
        const T *orow = o + row * p.os, *rrow = r + row * p.rs, *dnrow = dn ? dn + row * p.dns : nullptr,
                *dsrow = ds ? ds + row * p.dss : nullptr;
        float oz[NV][V], D[NV][V];  // oz: N(o), or o; D: z first
        float h1 = 0.0f, h2 = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            float u[V], f[V];
            ring.read(stage, 0, orow, j, oz[j]);
            const bool in = ring.in(j);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if (kPost) oz[j][i] = in ? (oz[j][i] - c.om) * c.ors : 0.0f;
                u[i] = oz[j][i];
            }
            if (kPost && in) {
                pw.template load<V>(ring.col(j), f);
#pragma unroll
                for (int i = 0; i < V; ++i) u[i] *= f[i];
                if (p.pb) {
                    pb.template load<V>(ring.col(j), f);
#pragma unroll
                    for (int i = 0; i < V; ++i) u[i] += f[i];
                }
            }
            if (s.gate == MOE_GATE_CHANNEL && in) {
                g.template load<V>(ring.col(j), f);
#pragma unroll
                for (int i = 0; i < V; ++i) u[i] *= f[i];
            }
            ring.read(stage, 1, rrow, j, f);
#pragma unroll
            for (int i = 0; i < V; ++i) D[j][i] = in ? (s.alpha * f[i] + c.gt * u[i] - c.m) * c.rs : 0.0f;
            ring.read(stage, 2, dnrow, j, u);
            if (in) w.template load<V>(ring.col(j), f);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                acc[0][j][i] += u[i] * D[j][i];
                acc[1][j][i] += u[i];
                const float h = in ? u[i] * f[i] : 0.0f;
                h1 += h;
                h2 += h * D[j][i];
            }
        }
        if (s.rms) {
            h1 = 0.0f;
            h2 = grp.sum(h2) * s.inv;
        } else {
            const float2 m = grp.sum(h1, h2);
            h1 = m.x * s.inv, h2 = m.y * s.inv;
        }
        float p1 = 0.0f, p2 = 0.0f, pg = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            float u[V], f[V];
            const bool in = ring.in(j);
            ring.read(stage, 2, dnrow, j, u);
            if (in) w.template load<V>(ring.col(j), f);
#pragma unroll
            for (int i = 0; i < V; ++i) u[i] = in ? c.rs * (u[i] * f[i] - h1 - D[j][i] * h2) : 0.0f;
            ring.read(stage, 3, dsrow, j, f);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                D[j][i] = f[i] + u[i];
                u[i] = s.alpha * D[j][i];
            }
            ring.write(static_cast<T*>(p.dres) + row * s.H, j, u);
            // q, but for a gate per channel, which the join applies to the column sums
#pragma unroll
            for (int i = 0; i < V; ++i) {
                u[i] = c.gt * D[j][i];
                acc[2][j][i] += u[i] * oz[j][i];
                acc[3][j][i] += u[i];
            }
            if (s.gate == MOE_GATE_CHANNEL && in) {
                g.template load<V>(ring.col(j), f);
#pragma unroll
                for (int i = 0; i < V; ++i) u[i] *= f[i];
            }
            if constexpr (kPost) {
                if (in) pw.template load<V>(ring.col(j), f);
                if (s.gate == MOE_GATE_TOKEN) {
                    float e[V] = {};
                    if (p.pb && in) pb.template load<V>(ring.col(j), e);
#pragma unroll
                    for (int i = 0; i < V; ++i) pg += in ? D[j][i] * (oz[j][i] * f[i] + e[i]) : 0.0f;
                }
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    D[j][i] = in ? u[i] * f[i] : 0.0f;  // p
                    p1 += D[j][i];
                    p2 += D[j][i] * oz[j][i];
                }
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) pg += D[j][i] * oz[j][i];
                ring.write(static_cast<T*>(p.dout) + row * s.H, j, u);
            }
        }
        if constexpr (kPost) {
            if (s.rms) {
                p1 = 0.0f;
                p2 = grp.sum(p2) * s.inv;
            } else {
                const float2 m = grp.sum(p1, p2);
                p1 = m.x * s.inv, p2 = m.y * s.inv;
            }
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                float u[V];
#pragma unroll
                for (int i = 0; i < V; ++i) u[i] = c.ors * (D[j][i] - p1 - oz[j][i] * p2);
                ring.write(static_cast<T*>(p.dout) + row * s.H, j, u);
            }
        }
        if (s.gate == MOE_GATE_TOKEN && (p.dgate_rows || p.dgate_typed)) {
            pg = grp.sum(pg);
            if (t == 0) {
                if (p.dgate_rows)
                    p.dgate_rows[row] = pg;
                else
                    static_cast<T*>(p.dgate_typed)[row] = from_f<T>(pg);
            }
        }
        if (++stage == s.stages) stage = 0;
    }
    cp_async_wait_all();
    if (!p.sums) return;
    // the groups' column sums, added in order through shared memory
    __syncthreads();
    float* col = reinterpret_cast<float*>(rings);  // [H]
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if (!(p.sums >> k & 1)) continue;
        for (int gi = 0; gi < s.groups; ++gi) {
            if (gi == id) {
                const bool last = gi == s.groups - 1;
#pragma unroll
                for (int j = 0; j < NV; ++j) {
                    if (!ring.in(j)) continue;
                    const int c0 = ring.col(j);
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const float v = gi == 0 ? acc[k][j][i] : col[c0 + i] + acc[k][j][i];
                        if (last)
                            p.part[((size_t)blockIdx.x * 4 + k) * s.H + c0 + i] = v;
                        else
                            col[c0 + i] = v;
                    }
                }
            }
            if (s.groups > 1) __syncthreads();
        }
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
// 32 columns a block, eight threads a column and sum.
template <typename T>
__global__ void __launch_bounds__(256) rn_join_kernel(const RnJoin p) {
    __shared__ float red[4][8][33];
    asm volatile("griddepcontrol.launch_dependents;\n\tgriddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31, c = blockIdx.x * 32 + lane, k8 = threadIdx.x >> 5;
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (c < p.H) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (!(p.sums >> k & 1)) continue;
#pragma unroll 4
            for (int i = k8; i < p.parts; i += 8) v[k] += p.part[((size_t)i * 4 + k) * p.H + c];
        }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) red[k][k8][lane] = v[k];
    __syncthreads();
    if (k8 || c >= p.H) return;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        v[k] = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[k] += red[k][i][lane];
    }
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

// ----------------------------------------------------------------- launches
bool on16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// Groups, threads and ring of a call; false: rows too long for the ring.
bool rn_plan(RnShape& s, int elt, int tensors, int* blocks, int* smem) {
    if (s.H > kRnMaxH) return false;
    s.nt = ((s.H + kRnCols - 1) / kRnCols + 31) / 32 * 32;
    int most = kRnThreads / s.nt;
    // sixteen hardware barriers, one of them the block's; a group of one warp needs none
    if (s.nt > 32 && most > 15) most = 15;
    const long long want = (s.rows + 151) / 152;
    s.groups = (int)(want < most ? want : most);
    s.row_bytes = (s.H * elt + 31) / 16 * 16;  // and the bytes before an unaligned row
    const int stage = s.groups * tensors * s.row_bytes;
    // L1 keeps 64 KB or more for the parameters while two stages allow it
    s.stages = 160 * 1024 / stage;
    s.stages = s.stages < 2 ? 2 : s.stages > 4 ? 4 : s.stages;
    *smem = s.groups * 512 + s.stages * stage;
    while (*smem > 227 * 1024) {
        --s.groups;
        *smem = s.groups * (512 + s.stages * tensors * s.row_bytes);
    }
    if (*smem < s.groups * 512 + s.H * 4) *smem = s.groups * 512 + s.H * 4;  // the groups' column sums
    const long long b = (s.rows + s.groups - 1) / s.groups;
    *blocks = (int)(b < 152 ? b : 152);
    return true;
}

template <typename K, typename A>
int rn_launch(K kernel, SmemLimit& limit, int blocks, int threads, int smem, const A& a, const char* name, cudaStream_t st) {
    if (const int e = limit.allow(kernel, 227 * 1024)) return e;
    trace_pre(st);
    kernel<<<blocks, threads, smem, st>>>(a);
    trace_post(st, name);
    return (int)cudaGetLastError();
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

template <typename T, bool kPost>
int rn_forward(RnFwd& a, cudaStream_t st) {
    int blocks, smem;
    RnShape& s = a.s;
    if (!rn_plan(s, sizeof(T), 2, &blocks, &smem)) {
        trace_pre(st);
        rn_fwd_long_kernel<T><<<(unsigned)(s.rows < 304 ? s.rows : 304), kRnLongThreads, 0, st>>>(a);
        trace_post(st, "residual_norm_fwd");
        return (int)cudaGetLastError();
    }
    constexpr int V = 16 / sizeof(T);
    const bool vec = s.H % V == 0 && a.os % V == 0 && a.rs % V == 0 && on16(a.o) && on16(a.r) && on16(a.stream) &&
                     on16(a.normed) && on16(a.pw) && on16(a.pb) && on16(a.w) && on16(a.b) &&
                     (s.gate != MOE_GATE_CHANNEL || on16(a.g));
    static SmemLimit lv, le;
    return vec ? rn_launch(rn_fwd_kernel<T, true, kPost>, lv, blocks, s.groups * s.nt, smem, a, "residual_norm_fwd", st)
               : rn_launch(rn_fwd_kernel<T, false, kPost>, le, blocks, s.groups * s.nt, smem, a, "residual_norm_fwd", st);
}

template <typename T, bool kPost>
int rn_backward(RnBwd& a, RnJoin& j, cudaStream_t st) {
    int blocks, smem, e;
    RnShape& s = a.s;
    if (!rn_plan(s, sizeof(T), 4, &blocks, &smem)) {
        blocks = rn_long_blocks(s.rows, s.H);
        trace_pre(st);
        rn_bwd_long_kernel<T><<<blocks, kRnLongThreads, 0, st>>>(a);
        trace_post(st, "residual_norm_bwd");
        e = (int)cudaGetLastError();
    } else {
        constexpr int V = 16 / sizeof(T);
        const bool vec = s.H % V == 0 && a.os % V == 0 && a.rs % V == 0 && (!a.dn || a.dns % V == 0) &&
                         (!a.ds || a.dss % V == 0) && on16(a.o) && on16(a.r) && on16(a.dn) && on16(a.ds) && on16(a.dout) &&
                         on16(a.dres) && on16(a.pw) && on16(a.pb) && on16(a.w) &&
                         (s.gate != MOE_GATE_CHANNEL || on16(a.g));
        static SmemLimit lv, le;
        e = vec ? rn_launch(rn_bwd_kernel<T, true, kPost>, lv, blocks, s.groups * s.nt, smem, a, "residual_norm_bwd", st)
                : rn_launch(rn_bwd_kernel<T, false, kPost>, le, blocks, s.groups * s.nt, smem, a, "residual_norm_bwd", st);
    }
    if (e || !a.sums) return e;
    j.parts = blocks;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)((s.H + 31) / 32));
    cfg.blockDim = dim3(256);
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
    return a.pw ? rn_forward<T, true>(a, st) : rn_forward<T, false>(a, st);
}
template <typename T>
int rn_backward_t(RnBwd& a, RnJoin& j, cudaStream_t st) {
    return a.pw ? rn_backward<T, true>(a, j, st) : rn_backward<T, false>(a, j, st);
}

}  // namespace

long long residual_norm_part_bytes(const moe_residual_norm_shape& s) {
    const long long blocks = s.H > kRnMaxH ? rn_long_blocks(s.rows, s.H) : s.rows < 152 ? s.rows : 152;
    return blocks * 4 * s.H * 4;
}

int launch_residual_norm_fwd(const moe_residual_norm_shape& s, const ResNormPtrs& f, cudaStream_t st) {
    RnFwd a = {rn_shape(s), f.out, f.residual, f.out_stride, f.residual_stride, f.gate, f.post_weight, f.post_bias,
               f.weight, f.bias, f.stream, f.normed, f.stats};
    return s.x_type == MOE_F32 ? rn_forward_t<float>(a, st)
           : s.x_type == MOE_F16 ? rn_forward_t<__half>(a, st)
                                 : rn_forward_t<__nv_bfloat16>(a, st);
}

int launch_residual_norm_bwd(const moe_residual_norm_shape& s, const ResNormPtrs& f, cudaStream_t st) {
    const bool channel = s.gate == MOE_GATE_CHANNEL, token = s.gate == MOE_GATE_TOKEN;
    const int f32 = s.w_type == MOE_F32;
    const int sums = (f.dweight ? 1 : 0) | (f.dbias ? 2 : 0) | (f.dpost_weight || (channel && f.dgate) ? 4 : 0) |
                     (f.dpost_bias || (channel && f.dgate && f.post_bias) ? 8 : 0);
    RnBwd a = {rn_shape(s), f.dstream, f.dnormed, f.out, f.residual, f.dstream_stride, f.dnormed_stride, f.out_stride,
               f.residual_stride, f.gate, f.post_weight, f.post_bias, f.weight, f.stats, f.dout, f.dresidual,
               token && f32 ? static_cast<float*>(f.dgate) : nullptr, token && !f32 ? f.dgate : nullptr, sums, f.part};
    RnJoin j = {f.part, 0, s.H, sums, f32, channel, f.post_weight != nullptr, f.gate, f.post_weight, f.post_bias,
                f.dweight, f.dbias, f.dpost_weight, f.dpost_bias, f.dgate};
    return s.x_type == MOE_F32 ? rn_backward_t<float>(a, j, st)
           : s.x_type == MOE_F16 ? rn_backward_t<__half>(a, j, st)
                                 : rn_backward_t<__nv_bfloat16>(a, j, st);
}

}  // namespace moe
