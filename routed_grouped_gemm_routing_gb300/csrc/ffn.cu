// The dense gated feed-forward block (a shared expert beside the routed ones),
// forward and backward:
//
//   h = x W1 (gate | up)     a = silu(clamp h_g) clamp h_u     y = a W2
//   da = dY W2^T             dW2 = a^T dY
//   dh_g = da u' sig(g')(1 + g'(1 - sig(g'))) [g passes]
//   dh_u = da silu(g') [u passes]              (g', u': the clamped inputs)
//   dx = dh W1^T             dW1 = x^T dh
//
// Six products of 2 T H I (y, da, dW2) or 4 T H I (h, dx, dW1) operations, all
// bound by the tensor cores from a few hundred tokens on: a step of 8192 x 7168 x
// 2048 takes 1.17 ms in a short burst, 1.85 PFLOP/s, 96 % of the measured bf16
// rate (1.37 ms and 1.58 PFLOP/s, 92 % of the sustained rate, when run for
// seconds under the power limit).  One kernel serves
// them (dense_pair_kernel): D[256 x 256] per pair of SMs, tcgen05 cta_group::2,
// operands by TMA (128-byte swizzle, K blocks of 64) straight from the
// row-major tensors: an operand whose rows run along K is K-major, one whose
// columns are the output's is MN-major, so nothing is ever transposed.  Each
// CTA of the pair loads 128 rows of A and 128 columns of B and holds 128 x 256
// of D in TMEM, twice, so that a tile's epilogue runs under the next one's
// products.  The epilogues do the rest of the block on the accumulators:
//   EPI_GATED  the tile's columns are 128 gate features (the first CTA's B) and
//              the same 128 up features (the second's): both projections, the
//              activation and the product in one kernel.  Leaves a and, for the
//              backward, h.
//   EPI_DGATE  dh from da in TMEM and h by TMA, both halves at once.
//   EPI_PLAIN  bf16 D.
//   EPI_PART   FP32 partial sums of a K range (see below).
//
// Roundings: a and dh are operands of bf16 products and are rounded once each.
// h stays FP32 for the backward: its rounding would come on top of dh's (dx and
// dW1 would err by half as much again), and its bytes, written and read once,
// are a few percent of the block's time.
//
// Few tiles (few tokens): the K range is split over several pairs per tile, each
// leaving FP32 partial sums, and ffn_join adds them in a fixed order and applies
// the epilogue; every SM then streams a part of the weights (dense_shape).
// Deterministic in every form: no atomics.
//
// The kernels of a call follow one another by programmatic launches: each
// starts, sets up its barriers and TMEM where an SM is free, and waits for the
// one before it before it touches any tensor.  dW2, dW1 and dx need nothing of
// each other once dh is there: one launch takes the tiles of all three, the
// deepest products first, so that one last round is ragged instead of three
// (4096 x 2048 x 1408: 164 us a step, 186 in three launches; 777 x 1160 x 712:
// 44 and 56 us).
//
// The forward of few tokens (ffn_few_takes) is ffn_few.cu's.
//
// Roles (10 warps per CTA): 0-7 epilogue (warp w: TMEM lanes 32 (w % 4) .. of
// the CTA's 128 rows, every other group of columns from w / 4 on; with four
// warps the arithmetic of EPI_DGATE took longer than the products of a
// 2048-deep tile: 72 -> 38 us at 4096 x 2048 x 1408), 8 TMA producer, 9 MMA
// issuer (first CTA of the pair).  Every wait is bounded; one that runs out
// sets bit 0 of the status word.
//
// The tile is 256 x 256, or narrower (192, 128 columns) where that wastes less of
// the last round over the pairs (dense_shape).
#include "clamp.cuh"
#include "grouped_gemm_2sm.cuh"

namespace moe {

namespace {

enum DenseMode { KK, KN, NN };  // majorness of A, B: K-major or MN-major (N)
enum DenseEpi { EPI_PLAIN, EPI_GATED, EPI_DGATE, EPI_PART, EPI_PART_GATED };  // EPI_PLAIN: plain_kernel below

constexpr int kDenseEpiWarps = 8;
constexpr int kDenseWarpTma = 8, kDenseWarpMma = 9;
constexpr int kDenseThreads = 320;
constexpr int kDenseClusters = 76;  // pairs of the 152 SMs: what the split of K aims at
constexpr int kDenseStageBytes = 32768;  // A and B blocks of one CTA: 128 x 64 bf16 each

template <int EPI>
__host__ __device__ constexpr int dense_stages() {
    return EPI == EPI_PLAIN || EPI == EPI_PART || EPI == EPI_PART_GATED ? 6 : 5;
}
// staging per epilogue warp: 4 KB boxes (EPI_GATED: h out, EPI_DGATE: h in)
template <int EPI>
__host__ __device__ constexpr int dense_boxes() {
    return EPI == EPI_GATED || EPI == EPI_DGATE ? 2 : 1;
}
constexpr int kDenseTail = 256;
template <int EPI>
__host__ __device__ constexpr int dense_smem() {
    return 1024 + dense_stages<EPI>() * kDenseStageBytes + kDenseEpiWarps * dense_boxes<EPI>() * 4096 + kDenseTail;
}
static_assert(dense_smem<EPI_GATED>() <= 232448 && dense_smem<EPI_PLAIN>() <= 232448, "shared memory per CTA");

struct DenseArgs {
    int M, N;      // rows; columns (EPI_GATED, EPI_DGATE: features of one half)
    int tiles_m, tiles_n;
    int kblocks;   // 64-deep K blocks
    int splits;    // K ranges (EPI_PART*)
    int width;     // columns of a tile (gated forms: both halves')
    float clamp;   // INFINITY: none
    int save_h;    // EPI_GATED: store h
    int32_t* status;
    __nv_bfloat16* out;  // EPI_GATED: a [M][N]; EPI_DGATE: dh [M][2][N]
};
struct DenseMaps {
    CUtensorMap a, b, c0, c1;
};

struct DenseBars {
    uint32_t base;
    int stages;
    __device__ __forceinline__ uint32_t full(int s) const { return base + 8u * s; }
    __device__ __forceinline__ uint32_t empty(int s) const { return base + 8u * (stages + s); }
    __device__ __forceinline__ uint32_t tfull(int a) const { return base + 8u * (2 * stages + a); }
    __device__ __forceinline__ uint32_t tempty(int a) const { return base + 8u * (2 * stages + 2 + a); }
    __device__ __forceinline__ uint32_t drain() const { return base + 8u * (2 * stages + 4); }
    __device__ __forceinline__ uint32_t hin(int w) const { return base + 8u * (2 * stages + 5 + w); }
};
static_assert(8 * (2 * 6 + 5 + kDenseEpiWarps) + 8 <= kDenseTail, "barrier area");

__device__ __forceinline__ void tma_store_3d(const CUtensorMap* m, int c0, int c1, int c2, uint32_t src) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                     reinterpret_cast<uint64_t>(m)),
                 "r"(c0), "r"(c1), "r"(c2), "r"(src)
                 : "memory");
}
__device__ __forceinline__ void tma_store_4d(const CUtensorMap* m, int c0, int c1, int c2, int c3, uint32_t src) {
    asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.bulk_group [%0, {%1, %2, %3, %4}], [%5];" ::"l"(
                     reinterpret_cast<uint64_t>(m)),
                 "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(src)
                 : "memory");
}

// Work items of a cluster: (tile, K range), tiles eight row tiles by all column
// tiles at a time so that the pairs that run together share their operands in L2.
struct DenseItem {
    int m0, n0, kb0, kb1, split;
};
template <int EPI>
struct DenseWalk {
    const DenseArgs& p;
    int w, total;
    __device__ __forceinline__ DenseWalk(const DenseArgs& p_)
        : p(p_), w((int)blockIdx.x >> 1), total(p_.tiles_m * p_.tiles_n * p_.splits) {}
    __device__ __forceinline__ bool valid() const { return w < total; }
    __device__ __forceinline__ void next() { w += (int)gridDim.x >> 1; }
    __device__ __forceinline__ DenseItem item() const {
        DenseItem it;
        const int tile = w / p.splits;
        it.split = w - tile * p.splits;
        const int per = 8 * p.tiles_n, group = tile / per, r = tile - group * per;
        const int rows = p.tiles_m - 8 * group < 8 ? p.tiles_m - 8 * group : 8;
        const int n = r / rows, m = 8 * group + r - n * rows;
        it.m0 = m * 256;
        it.n0 = n * (EPI == EPI_GATED || EPI == EPI_PART_GATED ? p.width / 2 : p.width);
        it.kb0 = (int)((long long)p.kblocks * it.split / p.splits);
        it.kb1 = (int)((long long)p.kblocks * (it.split + 1) / p.splits);
        return it;
    }
};

// ------------------------------------------------------------ TMA producer
template <int MODE, int EPI>
__device__ void dense_producer(const CUtensorMap* mA, const CUtensorMap* mB, const DenseArgs& p, uint32_t ring,
                               DenseBars bars, volatile int* abort, int rank) {
    constexpr bool kAN = MODE == NN, kBN = MODE != KK;
    constexpr bool kGated = EPI == EPI_GATED || EPI == EPI_PART_GATED;
    int stage = 0;
    uint32_t phase = 0;
    const int half = p.width / 2;      // this CTA's columns of B
    const bool two = half > 64;        // MN-major: boxes of 64 columns
    const uint32_t tx = 2u * (kDenseStageBytes / 2 + (kBN ? (two ? 16384u : 8192u) : (uint32_t)half * 128u));
    for (DenseWalk<EPI> w(p); w.valid(); w.next()) {
        const DenseItem it = w.item();
        const int m = it.m0 + 128 * rank, n = it.n0 + (kGated ? 0 : half * rank);
        for (int kb = it.kb0; kb < it.kb1; ++kb) {
            if (!mbar_wait(bars.empty(stage), phase ^ 1u, abort)) return;
            if (rank == 0) mbar_arrive_expect_tx(bars.full(stage), tx);
            const uint32_t fb = cluster_addr_of(bars.full(stage), 0);
            const uint32_t a = ring + stage * kDenseStageBytes, b = a + kDenseStageBytes / 2;
            const int k0 = kb * 64;
            if constexpr (kAN) {
                tma_load_2d_pair(a, mA, m, k0, fb);
                tma_load_2d_pair(a + 8192, mA, m + 64, k0, fb);
            } else {
                tma_load_2d_pair(a, mA, k0, m, fb);
            }
            if constexpr (kGated) {  // W1 viewed as [H][2][I]: the gate's or the up projection's columns
                tma_load_3d_pair(b, mB, n, rank, k0, fb);
                if (two) tma_load_3d_pair(b + 8192, mB, n + 64, rank, k0, fb);
            } else if constexpr (kBN) {
                tma_load_2d_pair(b, mB, n, k0, fb);
                if (two) tma_load_2d_pair(b + 8192, mB, n + 64, k0, fb);
            } else {
                tma_load_2d_pair(b, mB, k0, n, fb);
            }
            if (++stage == dense_stages<EPI>()) {
                stage = 0;
                phase ^= 1u;
            }
        }
    }
}

// -------------------------------------------------------------- MMA issuer
template <int MODE, int EPI>
__device__ void dense_mma(const DenseArgs& p, uint32_t ring, DenseBars bars, uint32_t tmem, volatile int* abort) {
    constexpr bool kAN = MODE == NN, kBN = MODE != KK;
    const uint32_t idesc = make_idesc_bf16(256, p.width, kAN, kBN);
    int stage = 0, it = 0;
    uint32_t phase = 0;
    for (DenseWalk<EPI> w(p); w.valid(); w.next(), ++it) {
        const DenseItem item = w.item();
        const int acc = it & 1;
        if (!warp_wait_uniform<true>(bars.tempty(acc), ((uint32_t)(it >> 1) & 1u) ^ 1u, abort)) return;
        tc_fence_after();
        const uint32_t d = tmem + (uint32_t)(acc * 256);
        for (int kb = item.kb0; kb < item.kb1; ++kb) {
            if (!warp_wait_uniform<true>(bars.full(stage), phase, abort)) return;
            tc_fence_after();
            const uint32_t a = ring + stage * kDenseStageBytes, b = a + kDenseStageBytes / 2;
            // the next 16 of K: 16 rows of 128 bytes (MN-major) or 32 bytes (K-major)
            const uint64_t ad = make_sdesc_sw128(a, kAN ? 8192 : 16, 1024), bd = make_sdesc_sw128(b, kBN ? 8192 : 16, 1024);
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    tc_mma_bf16_pair(d, ad + (kAN ? 128u : 2u) * kk, bd + (kBN ? 128u : 2u) * kk, idesc,
                                     kb > item.kb0 || kk ? 1u : 0u);
                tc_commit_pair(bars.empty(stage));
            }
            __syncwarp();
            if (++stage == dense_stages<EPI>()) {
                stage = 0;
                phase ^= 1u;
            }
        }
        if (elect_one()) tc_commit_pair(bars.tfull(acc));
        __syncwarp();
    }
}

// ---------------------------------------------------------------- epilogue
// Row r of a 32 x 32 f32 box in the 128-byte swizzle.
__device__ __forceinline__ void read_row_f32(uint32_t box, int r, float (&v)[32]) {
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        const int4 u = ld_shared_v4s(box + r * 128 + ((c ^ (r & 7)) << 4));
        v[4 * c] = __int_as_float(u.x);
        v[4 * c + 1] = __int_as_float(u.y);
        v[4 * c + 2] = __int_as_float(u.z);
        v[4 * c + 3] = __int_as_float(u.w);
    }
}

// 1 / (1 + e^-g), within a few units of 2^-23: the results are rounded to bf16.
__device__ __forceinline__ float sigmoid(float g) { return __fdividef(1.0f, 1.0f + __expf(-g)); }
// a = silu(clamp g) clamp u
__device__ __forceinline__ float gate_fwd(float g, float u, float c) {
    g = clamp_keep_nan(g, c);
    u = clamp_keep_nan(u, c);
    return g * sigmoid(g) * u;
}
// (dh_g, dh_u) of da
__device__ __forceinline__ float2 gate_bwd(float da, float g, float u, float c) {
    const float pg = clamp_passes(g, c), pu = clamp_passes(u, c);
    g = clamp_keep_nan(g, c);
    u = clamp_keep_nan(u, c);
    const float s = sigmoid(g), gs = g * s;
    return make_float2(pg * da * u * (s + gs * (1.0f - s)), pu * da * gs);
}
// 32 bf16 of a row: columns [0, n) of it (n >= 8, a multiple of 8).
__device__ __forceinline__ void store_row32(__nv_bfloat16* dst, const uint32_t (&p)[16], int n) {
#pragma unroll
    for (int c = 0; c < 4; ++c)
        if (8 * c < n) reinterpret_cast<uint4*>(dst)[c] = make_uint4(p[4 * c], p[4 * c + 1], p[4 * c + 2], p[4 * c + 3]);
}

template <int EPI>
__device__ void dense_epilogue(const CUtensorMap* m0, const CUtensorMap* m1, const DenseArgs& p, DenseBars bars,
                               uint32_t tmem, uint32_t stage, volatile int* abort, int warp, int lane, int rank) {
    const uint32_t tempty[2] = {cluster_addr_of(bars.tempty(0), 0), cluster_addr_of(bars.tempty(1), 0)};
    const int part = warp >> 2, quad = warp & 3;
    int it = 0;
    uint32_t hphase = 0;  // EPI_DGATE: h boxes waited for
    for (DenseWalk<EPI> w(p); w.valid(); w.next(), ++it) {
        const DenseItem item = w.item();
        const int acc = it & 1;
        const int row0 = item.m0 + 128 * rank + 32 * quad;
        const bool rows_live = row0 < p.M;
        // groups of 32 columns of this tile (gated forms: features), this warp's every other one
        const int cols = EPI == EPI_GATED || EPI == EPI_PART_GATED ? p.width / 2 : p.width;
        const int last = cols < p.N - item.n0 ? cols : p.N - item.n0;
        // EPI_DGATE: the first h boxes of the tile come while its products run
        auto fetch_h = [&](int c) {
            if (lane == 0) {
                mbar_arrive_expect_tx(bars.hin(warp), 8192u);
                tma_load_3d(stage, m1, item.n0 + 32 * c, 0, row0, bars.hin(warp));
                tma_load_3d(stage + 4096, m1, item.n0 + 32 * c, 1, row0, bars.hin(warp));
            }
        };
        if constexpr (EPI == EPI_DGATE) {
            if (rows_live && 32 * part < last) fetch_h(part);
        }
        if (!warp_wait(bars.tfull(acc), (uint32_t)(it >> 1) & 1u, abort)) break;
        tc_fence_after();
        const uint32_t t = tmem + (uint32_t)(acc * 256) + ((uint32_t)(quad * 32) << 16);
        const bool row_live = row0 + lane < p.M;
        bool ok = true;
        if (rows_live) {
            if constexpr (EPI == EPI_PART || EPI == EPI_PART_GATED) {
                constexpr int kHalves = EPI == EPI_PART_GATED ? 2 : 1;
#pragma unroll 1
                for (int c = part; c < kHalves * (cols / 32); c += 2) {
                    const int half = c / (cols / 32), f = 32 * (c - half * (cols / 32));
                    if (f >= last) continue;
                    uint32_t r0[32];
                    tmem_ld32_nowait(t + 32 * c, r0);
                    tmem_ld_wait();
                    if (lane == 0) bulk_wait_read<0>();
                    __syncwarp();
                    stage_row_sw128(stage, lane, r0);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        tma_store_4d(m0, item.n0 + f, half, row0, item.split, stage);
                        bulk_commit();
                    }
                }
            } else if constexpr (EPI == EPI_GATED) {
#pragma unroll 1
                for (int c = part; 32 * c < last; c += 2) {
                    uint32_t g[32], u[32], pk[16];
                    tmem_ld32_nowait(t + 32 * c, g);
                    tmem_ld32_nowait(t + cols + 32 * c, u);
                    tmem_ld_wait();
                    if (p.save_h) {
                        if (lane == 0) bulk_wait_read<0>();
                        __syncwarp();
                        stage_row_sw128(stage, lane, g);
                        stage_row_sw128(stage + 4096u, lane, u);
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) {
                            tma_store_3d(m1, item.n0 + 32 * c, 0, row0, stage);
                            tma_store_3d(m1, item.n0 + 32 * c, 1, row0, stage + 4096u);
                            bulk_commit();
                        }
                    }
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        pk[j] = pack_bf16x2(
                            gate_fwd(__uint_as_float(g[2 * j]), __uint_as_float(u[2 * j]), p.clamp),
                            gate_fwd(__uint_as_float(g[2 * j + 1]), __uint_as_float(u[2 * j + 1]), p.clamp));
                    if (row_live)
                        store_row32(p.out + (size_t)(row0 + lane) * p.N + item.n0 + 32 * c, pk, last - 32 * c);
                }
            } else {
#pragma unroll 1
                for (int c = part; 32 * c < last; c += 2) {
                    uint32_t da[32], pg[16], pu[16];
                    if (!warp_wait(bars.hin(warp), hphase, abort)) {
                        ok = false;
                        break;
                    }
                    hphase ^= 1u;
                    float g[32], u[32];
                    read_row_f32(stage, lane, g);
                    read_row_f32(stage + 4096u, lane, u);
                    __syncwarp();
                    if (32 * (c + 2) < last) fetch_h(c + 2);
                    // no code between: the registers hold nothing until the wait
                    tmem_ld32_nowait(t + 32 * c, da);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const float2 d0 = gate_bwd(__uint_as_float(da[2 * j]), g[2 * j], u[2 * j], p.clamp);
                        const float2 d1 = gate_bwd(__uint_as_float(da[2 * j + 1]), g[2 * j + 1], u[2 * j + 1], p.clamp);
                        pg[j] = pack_bf16x2(d0.x, d1.x);
                        pu[j] = pack_bf16x2(d0.y, d1.y);
                    }
                    if (row_live) {
                        __nv_bfloat16* out = p.out + (size_t)(row0 + lane) * 2 * p.N + item.n0 + 32 * c;
                        store_row32(out, pg, last - 32 * c);
                        store_row32(out + p.N, pu, last - 32 * c);
                    }
                }
            }
        }
        if (!ok) break;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(tempty[acc]);
    }
    if (lane == 0) bulk_wait_all();
    __syncwarp();
}

// Maps: a, b operands; c0 partial sums (EPI_PART); c1 h
// (EPI_GATED: store, EPI_DGATE: load).  a and dh leave by plain stores, 64
// contiguous bytes per row and thread.
struct DenseCta {
    uint32_t ring, boxes, tmem;
    DenseBars bars;
    volatile int* abort;
    int warp, lane, rank;
};
// Shared memory, barriers and TMEM of a CTA; returns when the pair is set up and
// the kernel before this one in the stream has ended.
template <int EPI>
__device__ __forceinline__ DenseCta dense_begin() {
    constexpr int kStages = dense_stages<EPI>();
    extern __shared__ uint8_t smem_raw[];
    DenseCta c;
    const uint32_t raw = smem_addr(smem_raw);
    c.ring = (raw + 1023u) & ~1023u;
    c.boxes = c.ring + kStages * kDenseStageBytes;
    const uint32_t bar0 = c.boxes + kDenseEpiWarps * dense_boxes<EPI>() * 4096;
    uint8_t* tail = smem_raw + (bar0 - raw);
    c.bars = DenseBars{bar0, kStages};
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tail + 8 * (2 * kStages + 5 + kDenseEpiWarps));
    c.abort = reinterpret_cast<volatile int*>(tmem_slot + 1);
    c.warp = threadIdx.x >> 5;
    c.lane = threadIdx.x & 31;
    c.rank = (int)cluster_ctarank();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(c.bars.full(s), 1);
            mbar_init(c.bars.empty(s), 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(c.bars.tfull(a), 1);
            mbar_init(c.bars.tempty(a), 2 * kDenseEpiWarps);
        }
        mbar_init(c.bars.drain(), 1);
        for (int w = 0; w < kDenseEpiWarps; ++w) mbar_init(c.bars.hin(w), 1);
        *c.abort = 0;
        fence_mbar_init();
    }
    if (c.warp == kDenseWarpMma) {
        tmem_alloc_pair(smem_addr(tmem_slot), 512);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    c.tmem = *tmem_slot;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    return c;
}
// The MMA warp's end: where a wait gave up, every MMA already issued (by this
// same elected lane) finishes before TMEM is released.
__device__ __forceinline__ void dense_drain(const DenseCta& c) {
    const bool aborted = __any_sync(0xffffffffu, *c.abort != 0);
    if (elect_one() && aborted) {
        tc_commit_pair_local(c.bars.drain());
        const uint64_t t0 = global_timer_ns();
        while (!mbar_try_wait(c.bars.drain(), 0) && global_timer_ns() - t0 < 100000000ull) {
        }
    }
    __syncwarp();
}
__device__ __forceinline__ void dense_end(const DenseCta& c, int32_t* status) {
    if (c.warp == kDenseWarpTma && c.lane == 0 && *c.abort) {
        // copies in flight land before the CTA's shared memory goes
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 2000000ull) {
        }
    }
    __syncwarp();
    tc_fence_before();
    cluster_sync();
    if (c.warp == kDenseWarpMma) {
        tc_fence_after();
        tmem_dealloc_pair(c.tmem, 512);
    }
    if (threadIdx.x == 0 && *c.abort) atomicOr(reinterpret_cast<int*>(status), 1);
}

template <int MODE, int EPI>
__global__ void __launch_bounds__(kDenseThreads, 1)
    dense_pair_kernel(const __grid_constant__ CUtensorMap mA, const __grid_constant__ CUtensorMap mB,
                      const __grid_constant__ CUtensorMap mC0, const __grid_constant__ CUtensorMap mC1,
                      const DenseArgs p) {
    if (threadIdx.x == 32 * kDenseWarpTma) {
        tma_prefetch_map(&mA);
        tma_prefetch_map(&mB);
        // EPI_GATED without save_h has no third map: none was encoded
        if (EPI != EPI_GATED || p.save_h) tma_prefetch_map(EPI == EPI_GATED || EPI == EPI_DGATE ? &mC1 : &mC0);
    }
    const DenseCta c = dense_begin<EPI>();
    if (c.warp == kDenseWarpTma) {
        if (c.lane == 0) dense_producer<MODE, EPI>(&mA, &mB, p, c.ring, c.bars, c.abort, c.rank);
    } else if (c.warp == kDenseWarpMma) {
        if (c.rank == 0) {
            dense_mma<MODE, EPI>(p, c.ring, c.bars, c.tmem, c.abort);
            dense_drain(c);
        }
    } else {
        dense_epilogue<EPI>(&mC0, &mC1, p, c.bars, c.tmem, c.boxes + c.warp * dense_boxes<EPI>() * 4096, c.abort, c.warp,
                            c.lane, c.rank);
    }
    dense_end(c, p.status);
}

// ------------------------------------------------- products with bf16 output
// Up to three products in one launch, each with its own operands' majorness.
constexpr int kPlainMost = 3;
struct PlainProblem {
    int M, N, tiles_m, tiles_n, kblocks, width;
    int a_mn, b_mn;  // MN-major operands
};
struct PlainArgs {
    int n;
    PlainProblem p[kPlainMost];
    int32_t* status;
};
struct PlainMaps {
    CUtensorMap m[3 * kPlainMost];  // A, B, D of each
};
struct PlainItem {
    int p, m0, n0;
};
// Round r of a cluster: item r n + c of the problems in order, or, every other
// round, from the far end, so that the costlier items of a round that straddles
// two problems go to the clusters that had the cheaper ones.
struct PlainWalk {
    const PlainArgs& a;
    int r, n, c, total;
    __device__ __forceinline__ PlainWalk(const PlainArgs& a_)
        : a(a_), r(0), n((int)gridDim.x >> 1), c((int)blockIdx.x >> 1), total(0) {
        for (int i = 0; i < a.n; ++i) total += a.p[i].tiles_m * a.p[i].tiles_n;
    }
    __device__ __forceinline__ int at() const { return r * n + ((r & 1) ? n - 1 - c : c); }
    // (a cluster past the end of one round may have an item in no later one)
    __device__ __forceinline__ bool valid() const { return at() < total; }
    __device__ __forceinline__ void next() { ++r; }
    __device__ __forceinline__ PlainItem item() const {
        int w = at(), i = 0;
        while (w >= a.p[i].tiles_m * a.p[i].tiles_n) w -= a.p[i].tiles_m * a.p[i].tiles_n, ++i;
        const PlainProblem& q = a.p[i];
        // eight row tiles by all column tiles at a time share their operands in L2
        const int per = 8 * q.tiles_n, group = w / per, l = w - group * per;
        const int rows = q.tiles_m - 8 * group < 8 ? q.tiles_m - 8 * group : 8;
        const int nt = l / rows, mt = 8 * group + l - nt * rows;
        return {i, mt * 256, nt * q.width};
    }
};

__global__ void __launch_bounds__(kDenseThreads, 1)
    plain_kernel(const __grid_constant__ PlainMaps maps, const __grid_constant__ PlainArgs a) {
    if (threadIdx.x == 32 * kDenseWarpTma)
        for (int i = 0; i < 3 * a.n; ++i) tma_prefetch_map(&maps.m[i]);
    const DenseCta c = dense_begin<EPI_PLAIN>();
    constexpr int kStages = dense_stages<EPI_PLAIN>();
    if (c.warp == kDenseWarpTma && c.lane == 0) {
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (PlainWalk w(a); w.valid() && ok; w.next()) {
            const PlainItem it = w.item();
            const PlainProblem& q = a.p[it.p];
            const CUtensorMap *mA = &maps.m[3 * it.p], *mB = mA + 1;
            const int half = q.width / 2, m = it.m0 + 128 * c.rank, n = it.n0 + half * c.rank;
            const bool two = half > 64;  // MN-major: boxes of 64 columns
            const uint32_t tx = 2u * (kDenseStageBytes / 2 + (q.b_mn ? (two ? 16384u : 8192u) : (uint32_t)half * 128u));
            for (int kb = 0; kb < q.kblocks; ++kb) {
                if (!mbar_wait(c.bars.empty(stage), phase ^ 1u, c.abort)) {
                    ok = false;
                    break;
                }
                if (c.rank == 0) mbar_arrive_expect_tx(c.bars.full(stage), tx);
                const uint32_t fb = cluster_addr_of(c.bars.full(stage), 0);
                const uint32_t sa = c.ring + stage * kDenseStageBytes, sb = sa + kDenseStageBytes / 2;
                const int k0 = kb * 64;
                if (q.a_mn) {
                    tma_load_2d_pair(sa, mA, m, k0, fb);
                    tma_load_2d_pair(sa + 8192, mA, m + 64, k0, fb);
                } else {
                    tma_load_2d_pair(sa, mA, k0, m, fb);
                }
                if (q.b_mn) {
                    tma_load_2d_pair(sb, mB, n, k0, fb);
                    if (two) tma_load_2d_pair(sb + 8192, mB, n + 64, k0, fb);
                } else {
                    tma_load_2d_pair(sb, mB, k0, n, fb);
                }
                if (++stage == kStages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
    } else if (c.warp == kDenseWarpMma && c.rank == 0) {
        int stage = 0, i = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (PlainWalk w(a); w.valid() && ok; w.next(), ++i) {
            const PlainProblem& q = a.p[w.item().p];
            const int acc = i & 1;
            if (!warp_wait_uniform<true>(c.bars.tempty(acc), ((uint32_t)(i >> 1) & 1u) ^ 1u, c.abort)) break;
            tc_fence_after();
            const uint32_t d = c.tmem + (uint32_t)(acc * 256);
            const uint32_t idesc = make_idesc_bf16(256, q.width, q.a_mn, q.b_mn);
            const uint32_t da = q.a_mn ? 128u : 2u, db = q.b_mn ? 128u : 2u;  // 16 of K, in 16 bytes
            for (int kb = 0; kb < q.kblocks; ++kb) {
                if (!warp_wait_uniform<true>(c.bars.full(stage), phase, c.abort)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t sa = c.ring + stage * kDenseStageBytes, sb = sa + kDenseStageBytes / 2;
                const uint64_t ad = make_sdesc_sw128(sa, q.a_mn ? 8192 : 16, 1024);
                const uint64_t bd = make_sdesc_sw128(sb, q.b_mn ? 8192 : 16, 1024);
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        tc_mma_bf16_pair(d, ad + da * kk, bd + db * kk, idesc, (kb | kk) != 0 ? 1u : 0u);
                    tc_commit_pair(c.bars.empty(stage));
                }
                __syncwarp();
                if (++stage == kStages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            if (!ok) break;
            if (elect_one()) tc_commit_pair(c.bars.tfull(acc));
            __syncwarp();
        }
        dense_drain(c);
    } else if (c.warp < kDenseEpiWarps) {
        const uint32_t tempty[2] = {cluster_addr_of(c.bars.tempty(0), 0), cluster_addr_of(c.bars.tempty(1), 0)};
        const uint32_t box = c.boxes + c.warp * 4096u;
        const int part = c.warp >> 2, quad = c.warp & 3;
        int i = 0;
        for (PlainWalk w(a); w.valid(); w.next(), ++i) {
            const PlainItem it = w.item();
            const PlainProblem& q = a.p[it.p];
            const int acc = i & 1, row0 = it.m0 + 128 * c.rank + 32 * quad;
            const int last = q.width < q.N - it.n0 ? q.width : q.N - it.n0;
            if (!warp_wait(c.bars.tfull(acc), (uint32_t)(i >> 1) & 1u, c.abort)) break;
            tc_fence_after();
            const uint32_t t = c.tmem + (uint32_t)(acc * 256) + ((uint32_t)(quad * 32) << 16);
            if (row0 < q.M) {
#pragma unroll 1
                for (int k = part; 64 * k < last; k += 2) {
                    uint32_t r0[32], r1[32], pk[32];
                    tmem_ld32_nowait(t + 64 * k, r0);
                    tmem_ld32_nowait(t + 64 * k + 32, r1);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        pk[j] = pack_bf16x2(__uint_as_float(r0[2 * j]), __uint_as_float(r0[2 * j + 1]));
                        pk[16 + j] = pack_bf16x2(__uint_as_float(r1[2 * j]), __uint_as_float(r1[2 * j + 1]));
                    }
                    if (c.lane == 0) bulk_wait_read<0>();
                    __syncwarp();
                    stage_row_sw128(box, c.lane, pk);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (c.lane == 0) {
                        tma_store_2d(&maps.m[3 * it.p + 2], it.n0 + 64 * k, row0, box);
                        bulk_commit();
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (c.lane == 0) mbar_arrive_cluster(tempty[acc]);
        }
        if (c.lane == 0) bulk_wait_all();
        __syncwarp();
    }
    __syncwarp();
    dense_end(c, a.status);
}

// ---------------------------------------------------------------- the join
// Sums of the K ranges' partial sums [splits][T][halves][n] in order, and the
// epilogue.  Eight columns per thread and half.
enum JoinEpi { JOIN_PLAIN, JOIN_GATED, JOIN_DGATE };
struct JoinArgs {
    const float* part;
    long long rows;
    int n, splits, halves;
    float clamp;
    void* out;   // JOIN_PLAIN: bf16 [rows][n]; JOIN_GATED: a; JOIN_DGATE: dh [rows][2][n]
    float* h;    // [rows][2][n]: JOIN_GATED written (may be null), JOIN_DGATE read
};
__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
    return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}
template <int EPI>
__global__ void __launch_bounds__(128) ffn_join_kernel(const JoinArgs p) {
    constexpr int kHalves = EPI == JOIN_GATED ? 2 : 1;
    asm volatile("griddepcontrol.launch_dependents;\n\tgriddepcontrol.wait;" ::: "memory");
    const int per = p.n / 8;
    const long long total = p.rows * per;
    const size_t stride = (size_t)p.rows * p.halves * p.n;
    for (long long i = (long long)blockIdx.x * 128 + threadIdx.x; i < total; i += (long long)gridDim.x * 128) {
        const long long row = i / per;
        const int c = (int)(i - row * per) * 8;
        float v[kHalves][8];
#pragma unroll
        for (int hf = 0; hf < kHalves; ++hf) {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[hf][j] = 0.0f;
            const float* src = p.part + ((size_t)row * p.halves + hf) * p.n + c;
#pragma unroll 4
            for (int s = 0; s < p.splits; ++s) {
                const float4 a = *reinterpret_cast<const float4*>(src + s * stride);
                const float4 b = *(reinterpret_cast<const float4*>(src + s * stride) + 1);
                v[hf][0] += a.x, v[hf][1] += a.y, v[hf][2] += a.z, v[hf][3] += a.w;
                v[hf][4] += b.x, v[hf][5] += b.y, v[hf][6] += b.z, v[hf][7] += b.w;
            }
        }
        auto* out = static_cast<__nv_bfloat16*>(p.out);
        float o[8];
        if constexpr (EPI == JOIN_PLAIN) {
            *reinterpret_cast<uint4*>(out + (size_t)row * p.n + c) = pack8(v[0]);
        } else if constexpr (EPI == JOIN_GATED) {
            if (p.h) {
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    float4* h = reinterpret_cast<float4*>(p.h + ((size_t)row * 2 + hf) * p.n + c);
                    h[0] = make_float4(v[hf][0], v[hf][1], v[hf][2], v[hf][3]);
                    h[1] = make_float4(v[hf][4], v[hf][5], v[hf][6], v[hf][7]);
                }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = gate_fwd(v[0][j], v[kHalves - 1][j], p.clamp);
            *reinterpret_cast<uint4*>(out + (size_t)row * p.n + c) = pack8(o);
        } else {
            const float* h = p.h + (size_t)row * 2 * p.n + c;
            float du[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float2 d = gate_bwd(v[0][j], h[j], h[p.n + j], p.clamp);
                o[j] = d.x;
                du[j] = d.y;
            }
            *reinterpret_cast<uint4*>(out + (size_t)row * 2 * p.n + c) = pack8(o);
            *reinterpret_cast<uint4*>(out + (size_t)row * 2 * p.n + p.n + c) = pack8(du);
        }
    }
}
template <int EPI>
int launch_join(const JoinArgs& a, cudaStream_t st) {
    const long long blocks = (a.rows * (a.n / 8) + 127) / 128;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)(blocks < 2432 ? blocks : 2432));
    cfg.blockDim = dim3(128);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    trace_pre(st);
    const cudaError_t e = cudaLaunchKernelEx(&cfg, ffn_join_kernel<EPI>, a);
    trace_post(st, "ffn_join");
    return (int)(e != cudaSuccess ? e : cudaGetLastError());
}

// ----------------------------------------------------------------- launches
int cdiv(long long a, int b) { return (int)((a + b - 1) / b); }

// Launches a kernel on pairs of SMs: one cluster per item up to those that fit
// at once.  first: the call's first kernel, which waits for all of the stream's
// earlier work.
template <typename K, typename... A>
int launch_pairs(K kernel, std::atomic<int> (&fits)[kMaxDevices], int smem, long long items, bool first,
                 const char* name, cudaStream_t st, const A&... args) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return (int)e;
    if (dev < 0 || dev >= kMaxDevices) return (int)cudaErrorInvalidDevice;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.blockDim = dim3(kDenseThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int fit = fits[dev].load(std::memory_order_relaxed);
    if (fit == 0) {
        // set once per device, outside any stream capture (on the first call)
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return (int)e;
        int sms = 0;
        e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return (int)e;
        cfg.gridDim = dim3((unsigned)(sms & ~1), 1, 1);
        e = cudaOccupancyMaxActiveClusters(&fit, kernel, &cfg);
        if (e != cudaSuccess) return (int)e;
        if (fit < 1) return (int)cudaErrorInvalidConfiguration;
        fits[dev].store(fit, std::memory_order_relaxed);
    }
    if (items <= 0) return 0;
    cfg.gridDim = dim3(2u * (unsigned)(items < fit ? items : fit), 1, 1);
    cfg.numAttrs = first ? 1 : 2;
    trace_pre(st);
    e = cudaLaunchKernelEx(&cfg, kernel, args...);
    trace_post(st, name);
    return (int)(e != cudaSuccess ? e : cudaGetLastError());
}
template <int MODE, int EPI>
int launch_dense(const DenseArgs& a, const DenseMaps& m, const char* name, cudaStream_t st, bool first = false) {
    static std::atomic<int> fits[kMaxDevices] = {};
    return launch_pairs(dense_pair_kernel<MODE, EPI>, fits, dense_smem<EPI>(),
                        (long long)a.tiles_m * a.tiles_n * a.splits, first, name, st, m.a, m.b, m.c0, m.c1, a);
}
int launch_plain(const PlainArgs& a, const PlainMaps& m, const char* name, cudaStream_t st) {
    static std::atomic<int> fits[kMaxDevices] = {};
    long long items = 0;
    for (int i = 0; i < a.n; ++i) items += (long long)a.p[i].tiles_m * a.p[i].tiles_n;
    return launch_pairs(plain_kernel, fits, dense_smem<EPI_PLAIN>(), items, false, name, st, m, a);
}

// Columns of a tile (gated: of both halves) and K ranges of a product: the
// cheapest in clocks of a pair, as measured.  A K block takes w + 256 (the
// bytes of its operands at 64 per clock and SM: 512 for the products of a 256
// wide tile too, but 384, not 256, at 128; 4096 x 2048 x 2816: three rounds at
// 256 54 us, five at 128 58 us).  K ranges cost the join's launch, 7000, and
// its reads and the partial sums' writes; without that term a block of 777
// tokens ran four joins for 16 us of its 66.
struct Shape {
    int width, splits;
};
Shape dense_shape(int M, int N, int kblocks, bool gated, bool may_split) {
    Shape best = {256, 1};
    long long cost = -1;
    for (int w = 256; w >= 128; w -= gated ? 128 : 64) {
        const long long tiles = (long long)cdiv(M, 256) * cdiv(N, gated ? w / 2 : w);
        const int most = w == 256 && may_split ? (int)(tiles < kDenseClusters ? kDenseClusters / tiles : 1) : 1;
        for (int s = 1; s <= most && s <= kblocks; ++s) {
            const long long rounds = (tiles * s + kDenseClusters - 1) / kDenseClusters;
            long long c = rounds * cdiv(kblocks, s) * (w + 256);
            if (s > 1) c += 7000 + (long long)M * N * (gated ? 2 : 1) * s * 8 / 2000;
            if (cost < 0 || c < cost) {
                cost = c;
                best = {w, s};
            }
        }
    }
    return best;
}

// One product of the block.
struct Product {
    int M, N, K;  // N: columns, or features of one half
    bool gated;   // B's columns are [2][N]
    bool may_split = true;
    Shape shape() const { return dense_shape(M, N, cdiv(K, 64), gated, may_split); }
    long long part_bytes() const {  // of the partial sums (0: one K range)
        const int s = shape().splits;
        return s > 1 ? (long long)s * M * (gated ? 2 : 1) * N * 4 : 0;
    }
    DenseArgs args(float clamp, int32_t* status) const {
        const Shape f = shape();
        DenseArgs a = {};
        a.M = M;
        a.N = N;
        a.tiles_m = cdiv(M, 256);
        a.tiles_n = cdiv(N, gated ? f.width / 2 : f.width);
        a.kblocks = cdiv(K, 64);
        a.splits = f.splits;
        a.width = f.width;
        a.clamp = clamp;
        a.status = status;
        return a;
    }
};

// Columns of a tile for several products in one launch: the cheapest of 256,
// 192 and 128 for all of them, in clocks of the busiest pair as PlainWalk deals
// the items out (256 once that is four rounds: the last one's waste is small).
int joint_width(const Product* q, int n) {
    int best = 256;
    long long cost = -1;
    for (int w = 256; w >= 128; w -= 64) {
        long long items = 0, most = 0, load[kDenseClusters] = {};
        for (int i = 0; i < n; ++i) {
            const long long tiles = (long long)cdiv(q[i].M, 256) * cdiv(q[i].N, w);
            if (items + tiles > 8 * kDenseClusters) return w == 256 ? 256 : best;
            for (long long t = 0; t < tiles; ++t, ++items) {
                const long long r = items / kDenseClusters, c = items % kDenseClusters;
                load[(r & 1) ? kDenseClusters - 1 - c : c] += (long long)cdiv(q[i].K, 64) * (w + 256) + 3000;
            }
        }
        for (long long l : load) most = l > most ? l : most;
        if (cost < 0 || most < cost) {
            cost = most;
            best = w;
        }
        if (items > 4 * kDenseClusters) return best;
    }
    return best;
}

// Tensor maps.  bf16 rows x cols, row-major: K-major operands take 64 columns x
// 128 rows, MN-major ones 64 x 64, stores 64 x 32.
int map_op(CUtensorMap* m, const void* p, long long rows, int cols, int box_rows, const char* what) {
    return abi_map_2d(m, p, 2, rows, cols, cols, 64, box_rows, what);
}

PlainProblem plain(const Product& q, int width, bool a_mn, bool b_mn) {
    return {q.M, q.N, cdiv(q.M, 256), cdiv(q.N, width), cdiv(q.K, 64), width, a_mn, b_mn};
}

Product fwd1(const moe_ffn_shape& s) { return {s.T, s.I, s.H, true}; }
Product fwd2(const moe_ffn_shape& s) { return {s.T, s.H, s.I, false}; }
Product dgate(const moe_ffn_shape& s) { return {s.T, s.I, s.H, false}; }

}  // namespace

long long ffn_part_bytes(const moe_ffn_shape& s) {
    long long most = 0;
    for (const Product& q : {fwd1(s), fwd2(s), dgate(s)})
        if (q.part_bytes() > most) most = q.part_bytes();
    return most;
}

int launch_ffn_forward(const moe_ffn_shape& s, const FfnPtrs& f, cudaStream_t st) {
    const float clamp = s.activation_clamp > 0.0f ? s.activation_clamp : INFINITY;
    int rc;
    {
        const Product q = fwd1(s);
        DenseArgs a = q.args(clamp, f.status);
        a.save_h = f.h != nullptr;
        DenseMaps m = {};
        if ((rc = map_op(&m.a, f.x, s.T, s.H, 128, "x"))) return rc;
        if ((rc = abi_map_nd(&m.b, f.W1, 2, {s.I, 2, s.H}, {64, 1, 64}, "W1 (gate/up halves)"))) return rc;
        int e;
        if (a.splits > 1) {
            if ((rc = abi_map_nd(&m.c0, f.part, 4, {s.I, 2, s.T, a.splits}, {32, 1, 32, 1}, "partial sums"))) return rc;
            e = launch_dense<KN, EPI_PART_GATED>(a, m, "ffn_gate_up", st, true);
            if (!e) e = launch_join<JOIN_GATED>({f.part, s.T, s.I, a.splits, 2, clamp, f.a, f.h}, st);
        } else {
            a.out = static_cast<__nv_bfloat16*>(f.a);
            if (f.h && (rc = abi_map_nd(&m.c1, f.h, 4, {s.I, 2, s.T}, {32, 1, 32}, "h (store)"))) return rc;
            e = launch_dense<KN, EPI_GATED>(a, m, "ffn_gate_up", st, true);
        }
        if (e) return abi_cuda_fail(e, "gate and up projection launch");
    }
    const Product q = fwd2(s);
    DenseArgs a = q.args(clamp, f.status);
    int e;
    if (a.splits > 1) {
        DenseMaps m = {};
        if ((rc = map_op(&m.a, f.a, s.T, s.I, 128, "a"))) return rc;
        if ((rc = map_op(&m.b, f.W2, s.I, s.H, 64, "W2"))) return rc;
        if ((rc = abi_map_nd(&m.c0, f.part, 4, {s.H, 1, s.T, a.splits}, {32, 1, 32, 1}, "partial sums"))) return rc;
        e = launch_dense<KN, EPI_PART>(a, m, "ffn_down", st);
        if (!e) e = launch_join<JOIN_PLAIN>({f.part, s.T, s.H, a.splits, 1, clamp, f.y, nullptr}, st);
    } else {
        PlainMaps m = {};
        PlainArgs pa = {1, {plain(q, a.width, false, true)}, f.status};
        if ((rc = map_op(&m.m[0], f.a, s.T, s.I, 128, "a"))) return rc;
        if ((rc = map_op(&m.m[1], f.W2, s.I, s.H, 64, "W2"))) return rc;
        if ((rc = map_op(&m.m[2], f.y, s.T, s.H, 32, "y (store)"))) return rc;
        e = launch_plain(pa, m, "ffn_down", st);
    }
    return e ? abi_cuda_fail(e, "down projection launch") : MOE_OK;
}

int launch_ffn_backward(const moe_ffn_shape& s, const FfnPtrs& f, cudaStream_t st) {
    const float clamp = s.activation_clamp > 0.0f ? s.activation_clamp : INFINITY;
    int rc, e;
    {  // da = dY W2^T, and dh from it
        const Product q = dgate(s);
        DenseArgs a = q.args(clamp, f.status);
        DenseMaps m = {};
        if ((rc = map_op(&m.a, f.dY, s.T, s.H, 128, "dY"))) return rc;
        if ((rc = map_op(&m.b, f.W2, s.I, s.H, a.width / 2, "W2 (K-major)"))) return rc;
        if (a.splits > 1) {
            if ((rc = abi_map_nd(&m.c0, f.part, 4, {s.I, 1, s.T, a.splits}, {32, 1, 32, 1}, "partial sums"))) return rc;
            e = launch_dense<KK, EPI_PART>(a, m, "ffn_dgate", st, true);
            if (!e) e = launch_join<JOIN_DGATE>({f.part, s.T, s.I, a.splits, 1, clamp, f.dh, f.h}, st);
        } else {
            a.out = static_cast<__nv_bfloat16*>(f.dh);
            if ((rc = abi_map_nd(&m.c1, f.h, 4, {s.I, 2, s.T}, {32, 1, 32}, "h"))) return rc;
            e = launch_dense<KK, EPI_DGATE>(a, m, "ffn_dgate", st, true);
        }
        if (e) return abi_cuda_fail(e, "dh launch");
    }
    // dW2 = a^T dY, dW1 = x^T dh, dx = dh W1^T: the deepest products first
    struct {
        Product q;
        bool a_mn, b_mn;
        const void *A, *B;
        void* D;
    } job[3] = {{{s.I, s.H, s.T, false, false}, true, true, f.a, f.dY, f.dW2},
                {{s.H, 2 * s.I, s.T, false, false}, true, true, f.x, f.dh, f.dW1},
                {{s.T, s.H, 2 * s.I, false, false}, false, false, f.dh, f.W1, f.dx}};
    if (2 * s.I > s.T) {
        const auto dx = job[2];
        job[2] = job[1];
        job[1] = job[0];
        job[0] = dx;
    }
    const Product qs[3] = {job[0].q, job[1].q, job[2].q};
    const int width = joint_width(qs, 3);
    PlainMaps m = {};
    PlainArgs a = {};
    a.n = 3;
    a.status = f.status;
    for (int i = 0; i < 3; ++i) {
        const auto& j = job[i];
        a.p[i] = plain(j.q, width, j.a_mn, j.b_mn);
        // rows and columns of the stored tensors: K x M or M x K, K x N or N x K
        if ((rc = j.a_mn ? map_op(&m.m[3 * i], j.A, j.q.K, j.q.M, 64, "A (MN-major)")
                         : map_op(&m.m[3 * i], j.A, j.q.M, j.q.K, 128, "A")))
            return rc;
        if ((rc = j.b_mn ? map_op(&m.m[3 * i + 1], j.B, j.q.K, j.q.N, 64, "B (MN-major)")
                         : map_op(&m.m[3 * i + 1], j.B, j.q.N, j.q.K, width / 2, "B")))
            return rc;
        if ((rc = map_op(&m.m[3 * i + 2], j.D, j.q.M, j.q.N, 32, "gradient (store)"))) return rc;
    }
    e = launch_plain(a, m, "ffn_grads", st);
    return e ? abi_cuda_fail(e, "gradient launch") : MOE_OK;
}

}  // namespace moe
