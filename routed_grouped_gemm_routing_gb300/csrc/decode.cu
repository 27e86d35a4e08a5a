// The whole expert layer for the few tokens of decoding, in two kernels:
//
//   l = x R,  idx = the k largest (equal ones: the lower id),  w = softmax over them
//   a[t, j] = silu(clamp x W1_g[e]) clamp(x W1_u[e])   e = idx[t, j]
//   y[t] = sum_j w[t, j] a[t, j] W2[e] + a_s[t] S2     (a_s: of the shared expert S1)
//
// Bound by DRAM: every weight of an expert that some token picks is read once, and
// used for the few tokens that picked it.
//
// decode_router_kernel: the logits, 32 experts x eight tokens to a cluster of
// eight blocks that split the width; FP32 sums of at most H / 512 terms a thread, joined in a
// fixed order.  It also clears the counters of the second kernel.
//
// decode_experts_kernel: one block on each SM.  Every block takes the top k of all
// tokens for itself (a few kilobytes of logits) and lists the experts' tokens.
// The work is a list of jobs that all blocks know: first, for each expert in use
// (the shared one first), 64 features of gate and up projection and a range of K;
// then, for each expert, 128 columns of the down projection and a range of K.
// Running blocks draw jobs from a counter.  A warp streams a job's weights by TMA, 128 of
// K x 2 x 64 columns a stage, and goes on to the next job's while this one's end is
// still computed, so that 160 KB are in flight on every SM all the time.
// Two warps gather the tokens' rows (cp.async) and, for the down projection,
// wait until the expert's activations are there: they come from jobs drawn
// earlier, by blocks that are running and that wait for nothing before them (a
// block draws in order, and gate and up jobs come first), so the wait ends whichever
// blocks are resident.  One warp tells the others of what a job has written, so that
// none that multiplies waits for the fence.  Eight warps multiply (mma
// m16n8k16, weights as A straight out of the boxes by transposed ldmatrix): eight
// gate and the same eight up features a warp, so that the activation needs no
// exchange; eight tokens as B, kNt such groups.  tcgen05 would want 128-row tiles
// of tokens or weights out of TMEM: at 8 to 64 tokens the weights' bytes, not the
// products, set the pace.
//
// FP32 partial sums of a K range of gate and up are added by whichever block
// finishes a tile last, in the order of the ranges; those of the down projection
// and a token's slots, in the order of its routing, by the blocks that run out of
// jobs.  Deterministic.
//
// Measured (the used weights' bytes at the copy rate): 16 V3-shaped tokens with a
// shared expert 1245-1342 us (1359: reads alone run above the copy rate), 32 V2-Lite-shaped
// ones 170-173 us (164), one V3-shaped token 117-122 us (106), where the router (6 us), the
// choice (4 us) and the first stages (4 us) come before any stream; 4 tokens of 128 x 64, 8 experts
// 12.3-14.9 us.
#include <math.h>

#include <type_traits>

#include "clamp.cuh"
#include "grouped_gemm_2sm.cuh"
#include "smem_limit.h"

namespace moe {

namespace {

constexpr int kDcConsumers = 8, kDcWarpTma = 8, kDcWarpGather = 9, kDcGathers = 2, kDcWarpSignal = 11;
constexpr int kDcThreads = 384;
// of K in a stage: with 64 the threads that fill the ring took as long for a stage
// as its bytes (64 tokens, 2048 x 1408, top 6 of 64: 205 us, 186 with 128)
constexpr int kDcK = 128;
constexpr int kDcBox = kDcK * 128;  // kDcK of K x 64 columns
constexpr int kDcJobs = 4;      // jobs drawn ahead
constexpr int kDcMaxSplit = 16;
constexpr int kRtCluster = 8, kRtRows = 1024;  // of the router: blocks of a cluster, rows of x held at once

// ----------------------------------------------------------------- router
template <int kTok>
__global__ void __launch_bounds__(256)
    decode_router_kernel(const __nv_bfloat16* __restrict__ x, const __nv_bfloat16* __restrict__ R, int T, int H, int E,
                         float* __restrict__ logits, int* __restrict__ counters, int n_counters) {
    __shared__ __align__(16) float xs[kTok][kTok == 1 ? 4 : kRtRows];
    __shared__ float red[8][kTok][32];
    __shared__ float all[kRtCluster][kTok][32];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");  // waited for before the stores to other blocks
    const int tid = threadIdx.x, cv = tid & 3, rl = tid >> 2, rank = (int)cluster_ctarank();
    {
        const int blocks = gridDim.x * gridDim.y * gridDim.z;
        const int b = blockIdx.x + gridDim.x * (blockIdx.y + gridDim.y * blockIdx.z);
        for (int i = b * 256 + tid; i < n_counters; i += blocks * 256) counters[i] = 0;
    }
    const int e0 = blockIdx.x * 32, t0 = blockIdx.y * kTok, e = e0 + 8 * cv;
    // multiples of 8, as H is
    const int per = (H / 8 + kRtCluster - 1) / kRtCluster * 8, h0 = rank * per, h1 = h0 + per < H ? h0 + per : H;
    const bool whole = E % 8 == 0;  // rows of R on 16-byte boundaries
    float acc[kTok][8];
#pragma unroll
    for (int t = 0; t < kTok; ++t)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[t][j] = 0.0f;
    // rows of R whose loads are in flight together: what the router takes is latency
    constexpr int kAhead = kTok == 1 ? 16 : 4;
    for (int c0 = h0; c0 < h1; c0 += kRtRows) {
        const int rows = h1 - c0 < kRtRows ? h1 - c0 : kRtRows;
        if constexpr (kTok > 1) {
            __syncthreads();
            {  // a warp a token, eight of its values a lane (the ranges are multiples of 8)
                const int t = tid >> 5;
                const __nv_bfloat16* src = x + (size_t)(t0 + t) * H + c0;
                for (int r = 8 * (tid & 31); r < rows; r += 256) {
                    float f[8] = {};
                    if (t0 + t < T) unpack_bf16x8(__ldg(reinterpret_cast<const uint4*>(src + r)), f);
                    *reinterpret_cast<float4*>(&xs[t][r]) = make_float4(f[0], f[1], f[2], f[3]);
                    *reinterpret_cast<float4*>(&xs[t][r + 4]) = make_float4(f[4], f[5], f[6], f[7]);
                }
            }
            __syncthreads();
        }
        if (e < E) {
            for (int r0 = rl; r0 < rows; r0 += 64 * kAhead) {
                uint4 u[kAhead];
                float x1[kAhead];
#pragma unroll
                for (int a = 0; a < kAhead; ++a) {
                    const int r = r0 + 64 * a;
                    u[a] = make_uint4(0, 0, 0, 0);
                    x1[a] = 0.0f;
                    if (r >= rows) continue;
                    const __nv_bfloat16* src = R + (size_t)(c0 + r) * E + e;
                    if (whole) {
                        u[a] = __ldg(reinterpret_cast<const uint4*>(src));
                    } else {
                        uint16_t h[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j) h[j] = e + j < E ? reinterpret_cast<const uint16_t*>(src)[j] : 0;
                        u[a] = make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
                    }
                    if constexpr (kTok == 1) x1[a] = __bfloat162float(x[(size_t)t0 * H + c0 + r]);
                }
#pragma unroll
                for (int a = 0; a < kAhead; ++a) {
                    const int r = r0 + 64 * a;
                    if (r >= rows) continue;
                    float w[8];
                    unpack_bf16x8(u[a], w);
#pragma unroll
                    for (int t = 0; t < kTok; ++t) {
                        const float v = kTok == 1 ? x1[a] : xs[t][r];
#pragma unroll
                        for (int j = 0; j < 8; ++j) acc[t][j] = fmaf(v, w[j], acc[t][j]);
                    }
                }
            }
        }
    }
    // eight rows of lanes, eight warps, eight blocks
#pragma unroll
    for (int t = 0; t < kTok; ++t)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float v = acc[t][j];
            v += __shfl_xor_sync(0xffffffffu, v, 4);
            v += __shfl_xor_sync(0xffffffffu, v, 8);
            v += __shfl_xor_sync(0xffffffffu, v, 16);
            if ((tid & 31) < 4) red[tid >> 5][t][8 * cv + j] = v;
        }
    __syncthreads();
    // No block's memory is written before that block runs: one whose range of the width is
    // empty (H = 8: seven of eight) would be here at once.
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    // a block's sums go to the block that finishes their token (one token: all to the first)
    for (int i = tid; i < kTok * 32; i += 256) {
        const int t = i >> 5, c = i & 31;
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < 8; ++w) v += red[w][t][c];
        const uint32_t dst = cluster_addr_of(smem_addr(&all[rank][t][c]), t);
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(dst), "f"(v) : "memory");
    }
    cluster_sync();
    const int t = rank, c = tid;
    if (t < kTok && t0 + t < T && c < 32 && e0 + c < E) {
        float v = 0.0f;
#pragma unroll
        for (int b = 0; b < kRtCluster; ++b) v += all[b][t][c];
        logits[(size_t)(t0 + t) * E + e0 + c] = v;
    }
}

// ----------------------------------------------------------------- experts
struct DecodeArgs {
    int T, H, I, E, k, Is;
    float clamp;
    int kp1, kp1s, kp2, kp2s;  // K ranges: gate and up, down; of a routed expert and of the shared one
    int stages;
    const __nv_bfloat16* x;
    const float* logits;  // null: the routing is given
    int32_t* topk_idx;    // [T][k], written, or read without logits
    float* topk_w;
    __nv_bfloat16 *act, *act_s;  // [T k][I], [T][Is]; up to 16 tokens [..][2][I]: and the rests
    float *part1, *part1s;       // [T k][kp1][2][I], [T][kp1s][2][Is]
    float *part2, *part2s;       // [T k][kp2][H], [T][kp2s][H]
    int *ticket, *done, *tiles_done, *joined;  // counters: jobs drawn, tiles of a group's activations that are there,
                                               // jobs of a column tile that are done, K ranges of a group's tile
    int32_t* status;
    __nv_bfloat16* y;
};

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* m, int c0, int c1, int c2, int c3, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::
            "r"(dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void dc_ldmatrix_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void dc_ldmatrix_x4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void dc_mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// A barrier of the multiplying warps that ends when one of them gave up.
struct ConsumerBarrier {
    uint32_t bar, phase;
    volatile int* abort;
    __device__ __forceinline__ bool sync() {
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
        const bool ok = warp_wait(bar, phase, abort);
        phase ^= 1u;
        return ok;
    }
};

// Counts a block's finished part (its threads have met at a barrier since they
// wrote it); whether it was the last of n, whose parts it may then read.
__device__ __forceinline__ int draw_last(int* counter, int n) {
    __threadfence();
    const int last = atomicAdd(counter, 1) == n - 1;
    __threadfence();
    return last;
}

// One warp: waits until a counter that other blocks raise is at `want` and sees
// what they wrote before; false when it gave up.
__device__ __forceinline__ bool warp_wait_flag(const int* flag, int want, volatile int* abort) {
    bool ok = true;
    if ((threadIdx.x & 31) == 0) {
        const uint64_t t0 = global_timer_ns();
        for (uint32_t it = 1;; ++it) {
            int v;
            asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(flag) : "memory");
            if (v >= want) break;
            if ((it & 63u) == 0 && (*abort || global_timer_ns() - t0 > kWaitLimitNs)) {
                *abort = 1;
                ok = false;
                break;
            }
        }
    }
    return __all_sync(0xffffffffu, ok);
}

// What every block keeps of the routing, in shared memory behind the ring.
struct Routing {
    float* w;         // [T k]
    int16_t* idx;     // [T k], -1: dropped
    uint16_t* list;   // slots by expert
    uint16_t *ge, *gb, *gn;  // groups: expert, start in list, slots
    int* n;           // groups
};
__host__ __device__ constexpr int dc_table_bytes(int slots) {
    return slots * 4 + (slots * 2 + 15) / 16 * 16 * 2 + (slots + 8) * 2 * 3 + 32;
}
// Up to 16 tokens the activations go into the down projection as two bf16 numbers
// each, the second the rounding's rest: the outputs then err by their own rounding
// alone, and what it costs, a second product on the same weights, is hidden there.
__host__ __device__ constexpr bool dc_two(int nt) { return nt <= 2; }
// eight tokens' rows of a stage: two halves of 64 of K, 128 bytes a row each
constexpr int kDcRows8 = 2048;
__host__ __device__ constexpr int dc_stage_bytes(int nt) { return 2 * kDcBox + nt * kDcRows8 * (dc_two(nt) ? 2 : 1); }
__host__ __device__ constexpr int dc_bar_bytes(int stages) { return 8 * (2 * stages + 3 * kDcJobs) + 8 * kDcJobs + 16; }

// One warp: the k largest of a token's E logits, as the layer's router takes them
// (equal ones by id, a NaN as -infinity, softmax over the chosen ones).
template <int P>
__device__ __forceinline__ void warp_topk(const float (&row)[P], int E, int k, int* idx, float* w) {
    const int lane = threadIdx.x & 31;
    uint32_t v[P];  // order-preserving codes
    uint32_t taken = 0;
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const float f = isnan(row[i]) ? -INFINITY : row[i];
        const uint32_t u = __float_as_uint(f == 0.0f ? 0.0f : f);
        v[i] = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
        if (lane + 32 * i >= E) taken |= 1u << i;
    }
    float m = 0.0f, sum = 0.0f;
    for (int j = 0; j < k; ++j) {
        uint32_t best = 0, at = 0xffffffffu;
#pragma unroll
        for (int i = 0; i < P; ++i)
            if (!(taken >> i & 1u) && (at == 0xffffffffu || v[i] > best)) best = v[i], at = lane + 32 * i;
        const uint32_t top = __reduce_max_sync(0xffffffffu, at == 0xffffffffu ? 0u : best);
        const uint32_t id = __reduce_min_sync(0xffffffffu, best == top ? at : 0xffffffffu);
        if ((id & 31) == lane) taken |= 1u << (id >> 5);
        const float key = __uint_as_float((top & 0x80000000u) ? (top & 0x7fffffffu) : ~top);
        if (j == 0) m = key;
        // limits of the softmax where the largest is infinite: 1 for each equal to it
        const float ex = isinf(m) ? (key == m ? 1.0f : 0.0f) : expf(key - m);
        sum += ex;
        if (lane == 0) idx[j] = (int)id, w[j] = ex;
    }
    __syncwarp();
    for (int j = lane; j < k; j += 32) w[j] = w[j] / sum;
    __syncwarp();
}
// All tokens, a warp each; the next one's logits come while one is chosen from.
template <int P>
__device__ __forceinline__ void block_topk(const float* logits, int T, int E, int k, int* idx, float* w) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int kWarps = kDcThreads / 32;
    float row[P], next[P];
    auto load = [&](int t, float (&r)[P]) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int e = lane + 32 * i;
            r[i] = t < T && e < E ? __ldcg(logits + (size_t)t * E + e) : -INFINITY;
        }
    };
    load(warp, row);
    for (int t = warp; t < T; t += kWarps) {
        if (P <= 8) load(t + kWarps, next);
        warp_topk<P>(row, E, k, idx + t * k, w + t * k);
        if (P > 8) load(t + kWarps, next);
#pragma unroll
        for (int i = 0; i < P; ++i) row[i] = next[i];
    }
}
__device__ __forceinline__ void block_topk_any(const float* logits, int T, int E, int k, int* idx, float* w) {
    const int p = (E + 31) / 32;
    if (p <= 2)
        block_topk<2>(logits, T, E, k, idx, w);
    else if (p <= 8)
        block_topk<8>(logits, T, E, k, idx, w);
    else
        block_topk<32>(logits, T, E, k, idx, w);
}

// The routing and the groups of at most `cap` slots of an expert.  Scratch (the
// ring's place): ids and places [slots], counts, starts and first groups [E + 1].
__device__ void build_routing(const DecodeArgs& p, const Routing& r, int cap, int* scratch) {
    const int slots = p.T * p.k, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int *ids = scratch, *rank = ids + slots, *cnt = rank + slots, *start = cnt + p.E + 1, *first = start + p.E + 1;
    for (int i = tid; i <= p.E; i += kDcThreads) cnt[i] = 0;
    if (p.logits) {
        block_topk_any(p.logits, p.T, p.E, p.k, ids, r.w);
    } else {
        for (int i = tid; i < slots; i += kDcThreads) ids[i] = __ldg(p.topk_idx + i), r.w[i] = __ldg(p.topk_w + i);
    }
    __syncthreads();
    if (warp == 0) {
        // each slot's place among its expert's, 32 slots at a time in order
        for (int i0 = 0; i0 < slots; i0 += 32) {
            const int i = i0 + lane, e = i < slots ? ids[i] : -1;
            const bool ok = e >= 0 && e < p.E;
            const uint32_t same = __match_any_sync(0xffffffffu, ok ? e : -1), before = same & ((1u << lane) - 1u);
            const int base = ok ? cnt[e] : 0;
            __syncwarp();
            if (ok) {
                rank[i] = base + __popc(before);
                if (before == 0) cnt[e] = base + __popc(same);
            }
            __syncwarp();
        }
        // prefix sums of the counts and of the groups: a run of experts a lane
        const int run = (p.E + 31) / 32, e0 = lane * run, e1 = e0 + run < p.E ? e0 + run : p.E;
        int s = 0, g = 0;
        for (int e = e0; e < e1; ++e) s += cnt[e], g += (cnt[e] + cap - 1) / cap;
        const int s0 = s, g0 = g;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int a = __shfl_up_sync(0xffffffffu, s, d), b = __shfl_up_sync(0xffffffffu, g, d);
            if (lane >= d) s += a, g += b;
        }
        const int all = __shfl_sync(0xffffffffu, g, 31);
        s -= s0;
        g -= g0;
        for (int e = e0; e < e1; ++e) {
            start[e] = s, first[e] = g;
            s += cnt[e], g += (cnt[e] + cap - 1) / cap;
        }
        if (lane == 0) *r.n = all;
    } else {
        for (int i = tid - 32; i < slots; i += kDcThreads - 32) {
            const int e = ids[i];
            r.idx[i] = (int16_t)(e >= 0 && e < p.E ? e : -1);
            if (p.logits && blockIdx.x == 0) p.topk_idx[i] = e, p.topk_w[i] = r.w[i];
        }
    }
    __syncthreads();
    for (int i = tid; i < slots; i += kDcThreads) {
        const int e = r.idx[i];
        if (e >= 0) r.list[start[e] + rank[i]] = (uint16_t)i;
    }
    for (int e = tid; e < p.E; e += kDcThreads)
        for (int q = 0; q * cap < cnt[e]; ++q) {
            r.ge[first[e] + q] = (uint16_t)e;
            r.gb[first[e] + q] = (uint16_t)(start[e] + q * cap);
            r.gn[first[e] + q] = (uint16_t)(cnt[e] - q * cap < cap ? cnt[e] - q * cap : cap);
        }
    __syncthreads();
}

// The jobs, in the order in which they are drawn.
struct Jobs {
    int tiles1, tiles1s, tiles2, st1, st2, st2s;  // column tiles; stages of K
    int n1s, n1, n2s, total, per1, per2;          // jobs; of a routed group
    __device__ __forceinline__ Jobs(const DecodeArgs& p, int groups) {
        tiles1 = (p.I + 63) / 64, tiles1s = (p.Is + 63) / 64, tiles2 = (p.H + 127) / 128;
        st1 = (p.H + kDcK - 1) / kDcK, st2 = (p.I + kDcK - 1) / kDcK, st2s = (p.Is + kDcK - 1) / kDcK;
        per1 = tiles1 * p.kp1, per2 = tiles2 * p.kp2;
        n1s = p.Is ? tiles1s * p.kp1s : 0;
        n1 = n1s + groups * per1;
        n2s = p.Is ? tiles2 * p.kp2s : 0;
        total = n1 + n2s + groups * per2;
    }
};
struct Job {
    bool down, shared;
    int group, tile, part, kb0, kb1;  // group: of the routed ones
};
__device__ __forceinline__ Job job_of(const DecodeArgs& p, const Jobs& n, int j) {
    Job q;
    q.down = j >= n.n1;
    if (q.down) j -= n.n1;
    const int ns = q.down ? n.n2s : n.n1s;
    q.shared = j < ns;
    if (!q.shared) j -= ns;
    const int per = q.down ? n.per2 : n.per1;
    const int kp = q.down ? (q.shared ? p.kp2s : p.kp2) : (q.shared ? p.kp1s : p.kp1);
    q.group = q.shared ? 0 : j / per;
    if (!q.shared) j -= q.group * per;
    q.tile = j / kp;
    q.part = j - q.tile * kp;
    const int st = q.down ? (q.shared ? n.st2s : n.st2) : n.st1;
    q.kb0 = st * q.part / kp;
    q.kb1 = st * (q.part + 1) / kp;
    return q;
}

template <int kNt>
__global__ void __launch_bounds__(kDcThreads, 1)
    decode_experts_kernel(const __grid_constant__ CUtensorMap mW1, const __grid_constant__ CUtensorMap mW2,
                          const __grid_constant__ CUtensorMap mS1, const __grid_constant__ CUtensorMap mS2,
                          const DecodeArgs p) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ int abort_word, last_word;
    volatile int* abort = &abort_word;
    const uint32_t raw = smem_addr(smem_raw), ring = (raw + 1023u) & ~1023u;
    constexpr uint32_t kStage = dc_stage_bytes(kNt);
    constexpr bool kTwo = dc_two(kNt);
    uint8_t* tail = smem_raw + (ring - raw) + p.stages * kStage;
    const uint32_t bar0 = smem_addr(tail);
    auto full = [&](int s) { return bar0 + 8u * s; };
    auto empty = [&](int s) { return bar0 + 8u * (p.stages + s); };
    auto jfull = [&](int s) { return bar0 + 8u * (2 * p.stages + s); };
    auto jempty = [&](int s) { return bar0 + 8u * (2 * p.stages + kDcJobs + s); };
    // a job's outputs: an arrival of each multiplying warp
    auto written = [&](int s) { return bar0 + 8u * (2 * p.stages + 2 * kDcJobs + s); };
    volatile int* jobs = reinterpret_cast<volatile int*>(tail + 8 * (2 * p.stages + 3 * kDcJobs));
    volatile int* joins = jobs + kDcJobs;  // of a job: whether its block joined the K ranges
    ConsumerBarrier cbar = {bar0 + 8u * (2 * p.stages + 3 * kDcJobs) + 8u * kDcJobs, 0, abort};
    const int slots = p.T * p.k;
    uint8_t* tab = tail + dc_bar_bytes(p.stages);
    Routing rt;
    rt.n = reinterpret_cast<int*>(tab);
    rt.w = reinterpret_cast<float*>(tab + 16);
    rt.idx = reinterpret_cast<int16_t*>(rt.w + slots);
    rt.list = reinterpret_cast<uint16_t*>(rt.idx + (slots + 7) / 8 * 8);
    rt.ge = rt.list + (slots + 7) / 8 * 8;
    rt.gb = rt.ge + slots + 8;
    rt.gn = rt.gb + slots + 8;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(full(s), 1 + 32 * kDcGathers);  // the TMA thread's arrival and the gathering lanes'
            mbar_init(empty(s), kDcConsumers);
        }
        for (int s = 0; s < kDcJobs; ++s) {
            mbar_init(jfull(s), 1);
            mbar_init(jempty(s), kDcConsumers + kDcGathers + 1);
            mbar_init(written(s), kDcConsumers);
        }
        mbar_init(cbar.bar, kDcConsumers);
        *abort = 0;
        fence_mbar_init();
        tma_prefetch_map(&mW1);
        tma_prefetch_map(&mW2);
        if (p.Is) {
            tma_prefetch_map(&mS1);
            tma_prefetch_map(&mS2);
        }
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    int ticket = 0;  // drawn here: its latency passes under the routing
    if (threadIdx.x == 32 * kDcWarpTma) ticket = atomicAdd(p.ticket, 1);
    build_routing(p, rt, 8 * kNt, reinterpret_cast<int*>(smem_raw + (ring - raw)));
    fence_proxy_async_smem();  // the scratch was the ring's
    __syncthreads();
    const int groups = *rt.n;
    const Jobs n(p, groups);
    const int down_jobs = (p.Is ? p.kp2s : 0) + groups * p.kp2;  // of a column tile

    if (warp == kDcWarpTma) {
        if (lane == 0) {
            int stage = 0, slot = 0;
            uint32_t phase = 0, jphase = 0;
            for (;;) {
                const int j = ticket < n.total ? ticket : -1;
                // drawn ahead: its latency passes under this job's copies
                if (j >= 0) ticket = atomicAdd(p.ticket, 1);
                if (!mbar_wait(jempty(slot), jphase ^ 1u, abort)) break;
                jobs[slot] = j;
                mbar_arrive(jfull(slot));
                if (++slot == kDcJobs) slot = 0, jphase ^= 1u;
                if (j < 0) break;
                const Job q = job_of(p, n, j);
                const int e = q.shared ? 0 : rt.ge[q.group];
                const CUtensorMap* m = q.down ? (q.shared ? &mS2 : &mW2) : (q.shared ? &mS1 : &mW1);
                bool ok = true;
                for (int kb = q.kb0; kb < q.kb1; ++kb) {
                    if (!(ok = mbar_wait(empty(stage), phase ^ 1u, abort))) break;
                    const uint32_t b = full(stage), dst = ring + stage * kStage;
                    mbar_arrive_expect_tx(b, 2 * kDcBox);
                    if (q.down) {
                        tma_load_3d(dst, m, 128 * q.tile, kDcK * kb, e, b);
                        tma_load_3d(dst + kDcBox, m, 128 * q.tile + 64, kDcK * kb, e, b);
                    } else {
                        tma_load_4d(dst, m, 64 * q.tile, 0, kDcK * kb, e, b);
                        tma_load_4d(dst + kDcBox, m, 64 * q.tile, 1, kDcK * kb, e, b);
                    }
                    if (++stage == p.stages) stage = 0, phase ^= 1u;
                }
                if (!ok) break;
            }
        }
    } else if (warp >= kDcWarpGather && warp < kDcWarpGather + kDcGathers) {
        int stage = 0, slot = 0;
        uint32_t phase = 0, jphase = 0;
        for (;;) {
            if (!warp_wait(jfull(slot), jphase, abort)) break;
            const int j = jobs[slot];
            __syncwarp();
            if (lane == 0) mbar_arrive(jempty(slot));
            if (++slot == kDcJobs) slot = 0, jphase ^= 1u;
            if (j < 0) break;
            const Job q = job_of(p, n, j);
            const int rows = q.shared ? p.T : rt.gn[q.group], K = q.down ? (q.shared ? p.Is : p.I) : p.H;
            const __nv_bfloat16* src = q.down ? (q.shared ? p.act_s : p.act) : p.x;
            // this lane's rows: 2 (this warp) + lane / 16, + 4, ..; a piece of 8 of K of each
            const int r0 = 2 * (warp - kDcWarpGather) + (lane >> 4);
            int at[2 * kNt];
#pragma unroll
            for (int i = 0; i < 2 * kNt; ++i) {
                const int r = r0 + 4 * i;
                at[i] = -1;
                if (r < rows) {
                    int s = r;
                    if (!q.shared) {
                        s = rt.list[rt.gb[q.group] + r];
                        if (!q.down) s /= p.k;
                    }
                    at[i] = s * K * (kTwo && q.down ? 2 : 1);
                }
            }
            bool ok = true;
            if (q.down) {  // the activations of this expert
                const int want = q.shared ? n.tiles1s : n.tiles1;
                const int* flag = p.done + (q.shared ? 0 : 1 + q.group);
                ok = warp_wait_flag(flag, want, abort);
            }
            const int live = (rows + 7) / 8 * 2;  // of the lanes' rows
            for (int kb = q.kb0; ok && kb < q.kb1; ++kb) {
                if (!(ok = warp_wait(empty(stage), phase ^ 1u, abort))) break;
                const int piece = lane & 15, k0 = kDcK * kb + 8 * piece;
                const uint32_t dst = ring + stage * kStage + 2 * kDcBox + (piece >> 3) * kNt * 1024;
                const bool in = k0 < K;
#pragma unroll
                for (int i = 0; i < 2 * kNt; ++i) {
                    if (i >= live) break;
                    const int r = r0 + 4 * i;
                    const bool there = at[i] >= 0 && in;
                    const uint32_t to = dst + r * 128 + (((piece ^ r) & 7) << 4);
                    cp_async_16(to, there ? src + at[i] + k0 : src, there ? 16 : 0);
                    if (kTwo && q.down) cp_async_16(to + kNt * kDcRows8, there ? src + at[i] + K + k0 : src, there ? 16 : 0);
                }
                cp_async_arrive_noinc(full(stage));
                if (++stage == p.stages) stage = 0, phase ^= 1u;
            }
            if (!ok) break;
        }
        cp_async_wait_all();
    } else if (warp == kDcWarpSignal) {
        // Tells the other blocks of a job's outputs, so that no multiplying warp waits
        // for the fence.
        int slot = 0;
        uint32_t jphase = 0;
        for (;;) {
            if (!warp_wait(jfull(slot), jphase, abort)) break;
            const int j = jobs[slot];
            const Job q = job_of(p, n, j < 0 ? 0 : j);
            if (j >= 0) {
                if (!warp_wait(written(slot), jphase, abort)) break;
                if (lane == 0 && (q.down || (q.shared ? p.kp1s : p.kp1) == 1 || joins[slot])) {
                    __threadfence();
                    atomicAdd(q.down ? p.tiles_done + q.tile : p.done + (q.shared ? 0 : 1 + q.group), 1);
                }
                __syncwarp();
            }
            if (lane == 0) mbar_arrive(jempty(slot));
            if (++slot == kDcJobs) slot = 0, jphase ^= 1u;
            if (j < 0) break;
        }
    } else {
        int stage = 0, slot = 0;
        uint32_t phase = 0, jphase = 0;
        const int tid = threadIdx.x, fl = lane >> 2, tk = 2 * (lane & 3);
        // weights: K row l % 8 (+ 8 from lane 16 on), first or second box, this warp's eight columns
        const int ak = (lane & 7) + (lane >= 16 ? 8 : 0);
        const uint32_t abase = ((lane >> 3) & 1) * kDcBox + ak * 128 + ((warp ^ (ak & 7)) << 4);
        for (;;) {
            if (!warp_wait(jfull(slot), jphase, abort)) break;
            const int j = jobs[slot], at_slot = slot;
            __syncwarp();
            if (j < 0) {
                if (lane == 0) mbar_arrive(jempty(slot));
                break;
            }
            if (++slot == kDcJobs) slot = 0, jphase ^= 1u;
            const Job q = job_of(p, n, j);
            const int rows = q.shared ? p.T : rt.gn[q.group], tiles = (rows + 7) / 8;
            // chains of dependent products: their latency, not a stage's bytes, is what a
            // single one would wait for
            constexpr int kChains = kNt <= 2 ? 4 : 2;
            float part_acc[kChains][kNt][4];
#pragma unroll
            for (int h = 0; h < kChains; ++h)
#pragma unroll
                for (int i = 0; i < kNt; ++i)
                    part_acc[h][i][0] = part_acc[h][i][1] = part_acc[h][i][2] = part_acc[h][i][3] = 0.0f;
            bool ok = true;
            for (int kb = q.kb0; kb < q.kb1; ++kb) {
                if (!(ok = warp_wait(full(stage), phase, abort))) break;
                const uint32_t a0 = ring + stage * kStage;
                uint32_t a[8][4];
#pragma unroll
                for (int s = 0; s < 8; ++s) dc_ldmatrix_x4_trans(a0 + abase + s * 2048, a[s]);
                const int r = lane & 7, v = lane >> 3;
#pragma unroll
                for (int i = 0; i < kNt; ++i) {
                    if (i >= tiles) break;
                    const uint32_t b0 = a0 + 2 * kDcBox + (8 * i + r) * 128;
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        uint32_t b[4];
                        float(&c0)[4] = part_acc[(2 * h) % kChains][i];
                        float(&c1)[4] = part_acc[(2 * h + 1) % kChains][i];
                        const uint32_t from = b0 + (h >> 1) * kNt * 1024 + (((4 * (h & 1) + v) ^ r) << 4);
                        dc_ldmatrix_x4(from, b);
                        dc_mma(c0, a[2 * h], b[0], b[1]);
                        dc_mma(c1, a[2 * h + 1], b[2], b[3]);
                        if (kTwo && q.down) {
                            dc_ldmatrix_x4(from + kNt * kDcRows8, b);
                            dc_mma(c0, a[2 * h], b[0], b[1]);
                            dc_mma(c1, a[2 * h + 1], b[2], b[3]);
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(empty(stage));
                if (++stage == p.stages) stage = 0, phase ^= 1u;
            }
            float acc[kNt][4];
#pragma unroll
            for (int i = 0; i < kNt; ++i)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    acc[i][c] = part_acc[0][i][c];
#pragma unroll
                    for (int h = 1; h < kChains; ++h) acc[i][c] += part_acc[h][i][c];
                }
            if (!ok) break;
            // ---- the end of a job.  acc: first box's column fl (8 a warp), tokens tk and
            // tk + 1 of each eight; then the second box's
            auto slot_of = [&](int r) { return q.shared ? r : (int)rt.list[rt.gb[q.group] + r]; };
            if (!q.down) {
                const int I = q.shared ? p.Is : p.I, kp = q.shared ? p.kp1s : p.kp1, f = 64 * q.tile + 8 * warp + fl;
                __nv_bfloat16* act = q.shared ? p.act_s : p.act;
                float* part = q.shared ? p.part1s : p.part1;
                const int g = q.shared ? 0 : 1 + q.group;
                bool mine = true;
                if (kp > 1) {
#pragma unroll
                    for (int i = 0; i < kNt; ++i)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const int r = 8 * i + tk + c;
                            if (r >= rows || f >= I) continue;
                            float* d = part + ((size_t)slot_of(r) * kp + q.part) * 2 * I + f;
                            __stcg(d, acc[i][c]);
                            __stcg(d + I, acc[i][2 + c]);
                        }
                    if (!cbar.sync()) break;
                    if (tid == 0) {
                        int* c = p.joined + (size_t)g * (n.tiles1 > n.tiles1s ? n.tiles1 : n.tiles1s) + q.tile;
                        last_word = draw_last(c, kp);
                    }
                    if (!cbar.sync()) break;
                    mine = last_word != 0;
                    if (tid == 0) joins[at_slot] = mine;
                }
                if (mine) {
#pragma unroll
                    for (int i = 0; i < kNt; ++i)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const int r = 8 * i + tk + c;
                            if (r >= rows || f >= I) continue;
                            const int s = slot_of(r);
                            float gate = acc[i][c], up = acc[i][2 + c];
                            if (kp > 1) {
                                gate = up = 0.0f;
                                const float* d = part + (size_t)s * kp * 2 * I + f;
#pragma unroll 4
                                for (int b = 0; b < kp; ++b) {
                                    gate += __ldcg(d + (size_t)b * 2 * I);
                                    up += __ldcg(d + (size_t)b * 2 * I + I);
                                }
                            }
                            gate = clamp_keep_nan(gate, p.clamp);
                            up = clamp_keep_nan(up, p.clamp);
                            const float a = gate / (1.0f + expf(-gate)) * up;
                            __nv_bfloat16 h = __float2bfloat16_rn(a);
                            if constexpr (kTwo) {
                                // (no rest of an infinity or a NaN; what only rounds to one is cut instead)
                                if (isfinite(a) && isinf(__bfloat162float(h))) h = __float2bfloat16_rz(a);
                                const float rest = isfinite(a) ? a - __bfloat162float(h) : 0.0f;
                                act[(size_t)s * 2 * I + I + f] = __float2bfloat16_rn(rest);
                            }
                            act[(size_t)s * (kTwo ? 2 : 1) * I + f] = h;
                        }
                }
            } else {
                const int kp = q.shared ? p.kp2s : p.kp2, c0 = 128 * q.tile + 8 * warp + fl;
                float* part = q.shared ? p.part2s : p.part2;
#pragma unroll
                for (int i = 0; i < kNt; ++i)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const int r = 8 * i + tk + c;
                        if (r >= rows) continue;
                        float* d = part + ((size_t)slot_of(r) * kp + q.part) * p.H;
                        if (c0 < p.H) __stcg(d + c0, acc[i][c]);
                        if (c0 + 64 < p.H) __stcg(d + c0 + 64, acc[i][2 + c]);
                    }
            }
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(written(at_slot));
                mbar_arrive(jempty(at_slot));
            }
        }
        // ---- y, 128 columns of a token a warp, once every part of them is there
        const int items = n.total ? p.T * n.tiles2 : 0;
        for (int i = blockIdx.x * kDcConsumers + warp; i < items; i += gridDim.x * kDcConsumers) {
            const int t = i / n.tiles2, tile = i - t * n.tiles2;
            if (!warp_wait_flag(p.tiles_done + tile, down_jobs, abort)) break;
            const int c = 128 * tile + 4 * lane;
            if (c >= p.H) continue;
            // K ranges of a slot, then slots, in order; eight loads in flight
            float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            auto add = [&](const float* base, int terms, int kp, auto weight) {
                float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                for (int n0 = 0, b = 0, sl = 0; n0 < terms; n0 += 8) {
                    float4 u[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        u[e] = n0 + e < terms ? __ldcg(reinterpret_cast<const float4*>(base + (size_t)(n0 + e) * p.H))
                                              : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        if (n0 + e >= terms) break;
                        v.x += u[e].x, v.y += u[e].y, v.z += u[e].z, v.w += u[e].w;
                        if (++b < kp) continue;
                        b = 0;
                        float w;
                        if (weight(sl++, w)) s.x += w * v.x, s.y += w * v.y, s.z += w * v.z, s.w += w * v.w;
                        v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    }
                }
            };
            // (a dropped slot's parts hold whatever was there: they are not added)
            add(p.part2 + (size_t)t * p.k * p.kp2 * p.H + c, p.k * p.kp2, p.kp2, [&](int sl, float& w) {
                w = rt.w[t * p.k + sl];
                return rt.idx[t * p.k + sl] >= 0;
            });
            if (p.Is)
                add(p.part2s + (size_t)t * p.kp2s * p.H + c, p.kp2s, p.kp2s, [&](int, float& w) {
                    w = 1.0f;
                    return true;
                });
            *reinterpret_cast<uint2*>(p.y + (size_t)t * p.H + c) = make_uint2(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w));
        }
    }
    __syncthreads();
    const bool gave_up = *abort != 0;
    if (gave_up) {  // copies in flight land before the block's shared memory goes
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 2000000ull) {
        }
        if (threadIdx.x == 0) atomicOr(reinterpret_cast<int*>(p.status), 1);
    }
    // no expert at all: zeros; a wait that ran out: NaN
    if (gave_up || n.total == 0) {
        const __nv_bfloat16 v = __float2bfloat16_rn(gave_up ? __int_as_float(0x7fffffff) : 0.0f);
        const int at = gave_up ? 0 : (int)blockIdx.x, step = gave_up ? 1 : (int)gridDim.x;
        for (long long i = (long long)at * kDcThreads + threadIdx.x; i < (long long)p.T * p.H; i += (long long)step * kDcThreads)
            p.y[i] = v;
    }
}

// ----------------------------------------------------------------- launches
int cdiv_i(long long a, int b) { return (int)((a + b - 1) / b); }
size_t up256_d(size_t v) { return (v + 255) / 256 * 256; }

// K ranges of the jobs of a column tile: as few as give most SMs one.  DRAM is kept
// busy by some 60 SMs with 190 KB in flight each, so uneven ends cost little, and a
// range's sums have to be joined.  Two stages (64 KB of weights) at least.  One token, 1024 x
// 512, 16 experts and a shared one: 16.9 us without ranges, 16.0 with; 64 tokens, 2048 x 1408, 4
// experts 42.9 with this rule, 57 with 152 jobs as the aim.  Where the ranges are short they
// cost more than they give: 32 tokens, 1024 x 512, 8 experts 20.9 without, 23.3 with.
int split_of(int stages, double jobs) {
    int s = jobs >= 96 ? 1 : (int)(128 / jobs + 0.5);
    if (s > stages / 2) s = stages / 2;
    if (s > kDcMaxSplit) s = kDcMaxSplit;
    return s < 1 ? 1 : s;
}

struct DecodePlan {
    int kp1, kp1s, kp2, kp2s, counters, joined, nt;
    size_t logits, count, act, act_s, part1, part1s, part2, part2s, bytes;
};
DecodePlan decode_plan(const moe_decode_shape& s) {
    DecodePlan d = {};
    const long long slots = (long long)s.T * s.k;
    // experts in use, as even routing has it
    const double used = s.E * (1.0 - pow(1.0 - (double)s.k / s.E, (double)s.T));
    const int st1 = cdiv_i(s.H, kDcK), st2 = cdiv_i(s.I, kDcK), st2s = cdiv_i(s.Is, kDcK);
    const int tiles1 = cdiv_i(s.I, 64), tiles1s = cdiv_i(s.Is, 64), tiles2 = cdiv_i(s.H, 128);
    d.kp1 = d.kp1s = split_of(st1, used * tiles1 + tiles1s);
    d.kp2 = split_of(st2, (used + (s.Is ? 1 : 0)) * tiles2);
    d.kp2s = s.Is ? split_of(st2s, (used + 1) * tiles2) : 1;
    d.nt = s.T <= 8 ? 1 : s.T <= 16 ? 2 : s.T <= 32 ? 4 : 8;
    const int groups = (int)slots + 1;
    d.joined = 16 + tiles2 + groups;  // ticket and status; column tiles; groups
    d.counters = d.joined + (d.kp1 > 1 || d.kp1s > 1 ? groups * (tiles1 > tiles1s ? tiles1 : tiles1s) : 0);
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t o = at;
        at += up256_d(bytes);
        return o;
    };
    d.count = take((size_t)d.counters * 4);
    d.logits = take((size_t)s.T * s.E * 4);
    const int two = dc_two(d.nt) ? 2 : 1;
    d.act = take((size_t)slots * s.I * 2 * two);
    d.act_s = take((size_t)s.T * s.Is * 2 * two);
    d.part1 = take(d.kp1 > 1 ? (size_t)slots * d.kp1 * 2 * s.I * 4 : 0);
    d.part1s = take(d.kp1s > 1 ? (size_t)s.T * d.kp1s * 2 * s.Is * 4 : 0);
    d.part2 = take((size_t)slots * d.kp2 * s.H * 4);
    d.part2s = take(s.Is ? (size_t)s.T * d.kp2s * s.H * 4 : 0);
    d.bytes = at;
    return d;
}

template <int kNt>
int launch_experts(const DecodeArgs& a0, const CUtensorMap (&m)[4], int sms, bool after_own, cudaStream_t st) {
    static SmemLimit limit;
    DecodeArgs a = a0;
    const int slots = a.T * a.k, most = 227 * 1024 - 64;
    a.stages = (most - 1024 - dc_table_bytes(slots) - dc_bar_bytes(16)) / dc_stage_bytes(kNt);
    if (a.stages > 16) a.stages = 16;
    const int bytes = 1024 + a.stages * dc_stage_bytes(kNt) + dc_bar_bytes(a.stages) + dc_table_bytes(slots);
    if (const int e = limit.allow(decode_experts_kernel<kNt>, most)) return e;
    long long jobs = (long long)(slots < a.E ? slots : a.E) * cdiv_i(a.I, 64) * a.kp1 + (long long)cdiv_i(a.Is, 64) * a.kp1s;
    const long long down = (long long)(slots < a.E ? slots : a.E) * cdiv_i(a.H, 128) * a.kp2;
    if (down > jobs) jobs = down;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)(jobs < sms ? jobs : sms));
    cfg.blockDim = dim3(kDcThreads);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = after_own ? 1 : 0;
    trace_pre(st);
    const cudaError_t e = cudaLaunchKernelEx(&cfg, decode_experts_kernel<kNt>, m[0], m[1], m[2], m[3], a);
    trace_post(st, "decode_experts");
    return (int)(e != cudaSuccess ? e : cudaGetLastError());
}

template <int kTok>
int launch_router(const moe_decode_shape& s, const DecodePtrs& f, const DecodePlan& d, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = kRtCluster;
    cfg.gridDim = dim3((unsigned)cdiv_i(s.E, 32), (unsigned)cdiv_i(s.T, kTok), kRtCluster);
    cfg.blockDim = dim3(256);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    trace_pre(st);
    const cudaError_t e = cudaLaunchKernelEx(
        &cfg, decode_router_kernel<kTok>, static_cast<const __nv_bfloat16*>(f.x), static_cast<const __nv_bfloat16*>(f.router),
        s.T, s.H, s.E, reinterpret_cast<float*>(f.ws + d.logits), reinterpret_cast<int*>(f.ws + d.count), d.counters);
    trace_post(st, "decode_router");
    return (int)(e != cudaSuccess ? e : cudaGetLastError());
}

}  // namespace

size_t decode_workspace_bytes(const moe_decode_shape& s) { return decode_plan(s).bytes; }

int launch_decode(const moe_decode_shape& s, const DecodePtrs& f, int sms, cudaStream_t st) {
    const DecodePlan d = decode_plan(s);
    int* count = reinterpret_cast<int*>(f.ws + d.count);
    DecodeArgs a = {};
    a.T = s.T, a.H = s.H, a.I = s.I, a.E = s.E, a.k = s.k, a.Is = s.Is;
    a.clamp = s.activation_clamp > 0.0f ? s.activation_clamp : INFINITY;
    a.kp1 = d.kp1, a.kp1s = d.kp1s, a.kp2 = d.kp2, a.kp2s = d.kp2s;
    a.x = static_cast<const __nv_bfloat16*>(f.x);
    a.logits = f.router ? reinterpret_cast<const float*>(f.ws + d.logits) : nullptr;
    a.topk_idx = f.topk_idx;
    a.topk_w = f.topk_w;
    a.act = reinterpret_cast<__nv_bfloat16*>(f.ws + d.act);
    a.act_s = reinterpret_cast<__nv_bfloat16*>(f.ws + d.act_s);
    a.part1 = reinterpret_cast<float*>(f.ws + d.part1);
    a.part1s = reinterpret_cast<float*>(f.ws + d.part1s);
    a.part2 = reinterpret_cast<float*>(f.ws + d.part2);
    a.part2s = reinterpret_cast<float*>(f.ws + d.part2s);
    a.ticket = count;
    a.status = count + 1;
    a.tiles_done = count + 16;
    a.done = a.tiles_done + cdiv_i(s.H, 128);
    a.joined = count + d.joined;
    a.y = static_cast<__nv_bfloat16*>(f.y);
    int rc;
    CUtensorMap m[4] = {};
    if ((rc = abi_map_nd(&m[0], f.W1, 2, {s.I, 2, s.H, s.E}, {64, 1, kDcK, 1}, "W1 (gate/up halves)"))) return rc;
    if ((rc = abi_map_nd(&m[1], f.W2, 2, {s.H, s.I, s.E}, {64, kDcK, 1}, "W2"))) return rc;
    if (s.Is) {
        if ((rc = abi_map_nd(&m[2], f.S1, 2, {s.Is, 2, s.H, 1}, {64, 1, kDcK, 1}, "S1 (gate/up halves)"))) return rc;
        if ((rc = abi_map_nd(&m[3], f.S2, 2, {s.H, s.Is, 1}, {64, kDcK, 1}, "S2"))) return rc;
    }
    int e;
    if (f.router) {
        e = s.T == 1 ? launch_router<1>(s, f, d, st) : launch_router<8>(s, f, d, st);
    } else {
        e = (int)cudaMemsetAsync(count, 0, (size_t)d.counters * 4, st);
    }
    if (e) return abi_cuda_fail(e, "router launch");
    const bool own = f.router != nullptr;
    e = d.nt == 1   ? launch_experts<1>(a, m, sms, own, st)
        : d.nt == 2 ? launch_experts<2>(a, m, sms, own, st)
        : d.nt == 4 ? launch_experts<4>(a, m, sms, own, st)
                    : launch_experts<8>(a, m, sms, own, st);
    return e ? abi_cuda_fail(e, "decoding experts launch") : MOE_OK;
}

}  // namespace moe
