// Products with 4-bit weights and one scale per group, for a few rows of
// activations (decoding): a dense matrix, and the routed experts (both
// projections of every expert held that way).
//
//   y[r, n] = sum_k x[r, k] (code[n, k] - 8) sf[n, k / G]          G = 32, 64, 128
//
// Bound by DRAM: K / 2 + 2 K / G bytes per row of W.  At 6.8 TB/s that is 47
// weights per clock and SM, 2.7 instruction slots per weight and lane, so the
// products go to the tensor cores and the codes are unpacked two at a time:
// (w >> 4 m) & 0x000f000f | 0x43004300 is the bf16 pair 128 + code, exactly.
// The offset is taken out in FP32 through the accumulator's initial value,
//   sum x (code - 8) = [-136 sum_k x] + sum x (128 + code),
// one sum of x per row and group, made once per block.  A group's sum is then
// scaled and added in FP32; nothing is rounded before the output.
//
// mma m16n8k16: A = 16 rows of W, B = up to 8 rows of x (kNt column tiles of
// them: 8 or 16 rows to a job).  (tcgen05.mma would take the unpacked weights
// from shared memory or TMEM, one more trip from the registers that unpack them,
// for 8 of its columns.  That form has not been built or measured.)  The order of
// the codes in memory makes a lane's 16 bytes of a 128-code block the operands of
// its eight products: word 4 t + j holds codes 32 j + 8 t .. + 7, code 2 m in
// nibble m, code 2 m + 1 in nibble m + 4, so that lane t's pair m of group j meets
// x[32 j + 8 t + 2 m, + 1].
//
// A block takes a job (up to 8 or 16 rows that use the same matrix) and a range
// of tiles of 32 rows of W (W4_GATED: 16 gate rows and their 16 up rows); KS
// of its warps share a tile, every KS-th unit of 256 codes each, and join their
// FP32 sums in shared memory in a fixed order.  One lane copies its warp's next
// units ahead by TMA (a 32 x 128-byte box in the 128-byte swizzle, so that the
// fragments' 16-byte reads spread over the banks), across the tiles of the
// range: with a 16-byte copy per lane and fragment instead, the addresses alone
// took as many instructions as the products.  Scales come by plain loads, one
// row per lane and a unit ahead, and go to the fragments by shuffles.
//
// Measured (the bytes at the copy rate): one row of a 131072 x 7168 matrix, G =
// 128, 84.9 us, 5.7 TB/s (71); 16384 x 7168, G = 128: one row 17.2 us, 8 rows 20.3
// (8.9); 16380 x 7168, G = 32, 12 rows 30.2 (9.8).  In the steady state 51 % of
// the issue slots and 62 % of the ALU's are taken: what is left of the floor is
// latency of the unpacking, four warps to a scheduler.
#include <cmath>

#include "clamp.cuh"
#include "grouped_gemm_2sm.cuh"
#include "smem_limit.h"

namespace moe {

namespace {

constexpr int kSlots = 2;  // units of 256 codes held or in flight per warp
constexpr int kUnitBytes = 4096;  // 32 rows x 128 bytes
// 8-row fragments of a tile: two 16-row operands of the products.  (One operand,
// 64 registers and 32 warps per SM instead of 16 was slower: 16384 x 7168 at one
// row 20.6 us against 17.5, twice the bookkeeping and reads of x per weight.)
constexpr int kFrag = 4;
constexpr int kR = 8;  // rows of x that one product takes; a job has kNt times as many

enum W4Epi { W4_PLAIN, W4_GATED, W4_SLOT };

struct W4Args {
    const __nv_bfloat16* x;  // [rows, K]
    const __nv_bfloat16* sf;  // [E][N][K / G]
    int N;       // rows of one matrix (W4_GATED: 2 I)
    int F;       // output features: N, or I
    int K, E;
    int rows;    // rows of x (no ids)
    const int32_t* ids;  // expert of each slot, or null: one matrix, rows of x in order
    int slots;   // length of ids
    int busy;    // jobs to expect of them
    int xdiv;    // x row of a slot = slot / xdiv
    int tiles;   // of F
    int tpc;     // tiles per block
    int ks;      // warps per tile
    int R;       // rows of a job
    int kparts;  // blocks of a cluster that split K
    float clamp;    // W4_GATED: of gate and up, INFINITY: none
    uint32_t mask;  // 0x000f000f, unknown to the compiler (see pair128)
    const float* slot_w;  // W4_SLOT: weight of each slot
    void* out;   // W4_PLAIN, W4_GATED: bf16 [row or slot][F]; W4_SLOT: f32 [slot][F]
};

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The first product of a chain: c = (x, y, x, y) + a b.
__device__ __forceinline__ void mma_bf16_from(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1, float x, float y) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%10,%11};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(x), "f"(y));
}
// Codes 2 m and 2 m + 1 of a word as the bf16 pair 128 + code.  mask is
// 0x000f000f in a register: with both constants immediate this takes two
// logic instructions instead of one, and they bound these kernels.
template <int m>
__device__ __forceinline__ uint32_t pair128(uint32_t w, uint32_t mask) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, 0x43004300, 0xEA;" : "=r"(r) : "r"(w >> (4 * m)), "r"(mask));
    return r;
}
__device__ __forceinline__ uint32_t word_of(const uint4& v, int j) {
    return j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w;
}

// Byte offsets in a block's shared memory (from its first 1024-byte boundary).
// kparts: blocks of a cluster that share the tiles and split K; x and its sums
// are those of a block's own units, and the first block takes all partial sums.
struct W4Smem {
    int x, xs, red, bars, total;
};
__host__ __device__ __forceinline__ int w4_units(int K, int kparts) { return ((K + 255) / 256 + kparts - 1) / kparts; }
template <int G, int kNt>
__host__ __device__ __forceinline__ W4Smem w4_smem(int K, int nw, int rows, int kparts) {
    W4Smem s;
    const int kpad = w4_units(K, kparts) * 256;
    s.x = nw * kSlots * kUnitBytes;
    // a row of x and 64 bytes: the eight rows' 16-byte fragments in all banks
    s.xs = s.x + rows * (2 * kpad + 64);
    s.red = s.xs + (kpad / G) * kR * kNt * 4;
    s.bars = s.red + (kparts > 1 || kNt > 1 ? 1 : 2) * nw * 256 * kNt * 4;
    s.total = s.bars + nw * kSlots * 8 + 1024;
    return s;
}

// The scales of one 128-code block of a row.
template <int G>
struct W4Scales;
template <>
struct W4Scales<128> {
    typedef uint16_t T;
};
template <>
struct W4Scales<64> {
    typedef uint32_t T;
};
template <>
struct W4Scales<32> {
    typedef uint2 T;
};
// The scales of lane src's row, packed, and the i-th of them as a float.
__device__ __forceinline__ void scales_of(uint16_t v, int src, uint32_t (&u)[1]) {
    u[0] = __shfl_sync(0xffffffffu, (uint32_t)v, src);
}
__device__ __forceinline__ void scales_of(uint32_t v, int src, uint32_t (&u)[1]) { u[0] = __shfl_sync(0xffffffffu, v, src); }
__device__ __forceinline__ void scales_of(uint2 v, int src, uint32_t (&u)[2]) {
    u[0] = __shfl_sync(0xffffffffu, v.x, src);
    u[1] = __shfl_sync(0xffffffffu, v.y, src);
}
__device__ __forceinline__ float scale(uint32_t u, int i) { return __uint_as_float(i & 1 ? u & 0xffff0000u : u << 16); }

// mq: the codes as [E N] rows of K / 2 bytes.
template <int G, int EPI, int kNt>
__global__ void __launch_bounds__(512, 1) w4_kernel(const __grid_constant__ CUtensorMap mq, const W4Args p) {
    constexpr int kSw = G == 32 ? 2 : 1;              // words of a row's scales of a 128-code block
    constexpr int kTile = EPI == W4_GATED ? 16 : 32;  // output features of a tile
    constexpr int kSide = G == 32 || kNt > 1 ? 1 : 2;  // 128-code blocks worked on side by side: four chains of dependent products
    constexpr int kRows = kR * kNt;
    typedef typename W4Scales<G>::T Scales;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    __shared__ int row_of[kRows];  // row or slot of every row of the job
    __shared__ int job_n;
    __shared__ int abort_word;
    volatile int* abort = &abort_word;
    const int R = p.R;  // rows of a job, at most kRows
    const int nw = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    const int K = p.K, KB = K / 128, KS = p.ks, NG = nw / KS;
    const int ks = warp % KS, gi = warp / KS;
    // this block's units [U0, U) and elements [k0, k0 + kn) of K
    const int part = blockIdx.z, per = w4_units(K, p.kparts), U0 = part * per;
    const int U = U0 + per < (KB + 1) / 2 ? U0 + per : (KB + 1) / 2;
    const int k0 = U0 * 256, kn = (U * 256 < K ? U * 256 : K) - k0;  // w4_launch splits so that every part has units
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // ---- the job: its matrix and its rows
    int e = 0;
    if (p.ids) {
        const int s = blockIdx.y;
        e = __ldg(p.ids + s);
        if (e < 0 || e >= p.E) return;  // a dropped slot
        if (warp == 0) {
            // slots of expert e in order; every R-th of them leads a job
            int before = 0, n = 0;
            for (int base = 0; base < p.slots && n < R; base += 32) {
                const int i = base + lane;
                const bool same = i < p.slots && __ldg(p.ids + i) == e;
                before += __popc(__ballot_sync(0xffffffffu, same && i < s));
                const uint32_t from = __ballot_sync(0xffffffffu, same && i >= s);
                const int pos = n + __popc(from & ((1u << lane) - 1u));
                if (same && i >= s && pos < R) row_of[pos] = i;
                n += __popc(from);
            }
            if (lane == 0) job_n = before % R == 0 ? (n < R ? n : R) : 0;
        }
    } else {
        const int r0 = blockIdx.y * R;
        if (threadIdx.x < R) row_of[threadIdx.x] = r0 + threadIdx.x;
        if (threadIdx.x == 0) job_n = p.rows - r0 < R ? p.rows - r0 : R;
    }
    const uint32_t raw = smem_addr(smem_raw), base = (raw + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (base - raw);
    // (the offsets of the block's largest job: they do not wait for job_n)
    const W4Smem L = w4_smem<G, kNt>(K, nw, R, p.kparts);
    const uint32_t ring = base + warp * kSlots * kUnitBytes, bar = base + L.bars + warp * kSlots * 8;
    if (lane == 0) {
        for (int i = 0; i < kSlots; ++i) mbar_init(bar + 8 * i, 1);
        fence_mbar_init();
    }
    if (threadIdx.x == 0) *abort = 0;
    __syncthreads();
    const int n = job_n;
    if (n == 0) return;  // not the leading slot

    __nv_bfloat16* xsm = reinterpret_cast<__nv_bfloat16*>(smem + L.x);
    float* xs = reinterpret_cast<float*>(smem + L.xs);  // [K / G][kRows]: -136 sum of x
    float* red = reinterpret_cast<float*>(smem + L.red);

    // ---- the stream of this warp's weights: tiles gi, gi + NG, .. of the
    // block's range, units ks, ks + KS, .. of each.  Rows past the last of the
    // matrix are another's or zeros, and are not stored.
    const int tile0 = blockIdx.x * p.tpc;
    const int tile1 = tile0 + p.tpc < p.tiles ? tile0 + p.tpc : p.tiles;
    const long long row0 = (long long)e * p.N;
    int ft = tile0 + gi, fu = U0 + ks, fslot = 0;
    auto fetch = [&]() {
        if (ft < tile1 && fu < U) {
            if (lane == 0) {
                const uint32_t b = bar + 8 * fslot, dst = ring + fslot * kUnitBytes;
                const int y = (int)(row0 + ft * kTile);
                mbar_arrive_expect_tx(b, kUnitBytes);
                if constexpr (EPI == W4_GATED) {
                    tma_load_2d(dst, &mq, fu * 128, y, b);
                    tma_load_2d(dst + kUnitBytes / 2, &mq, fu * 128, y + p.F, b);
                } else {
                    tma_load_2d(dst, &mq, fu * 128, y, b);
                }
            }
            fu += KS;
            if (fu >= U) {
                fu = U0 + ks;
                ft += NG;
            }
        }
        fslot = fslot + 1 == kSlots ? 0 : fslot + 1;
    };
    for (int d = 0; d < kSlots - 1; ++d) fetch();
    // scales of row `lane` of the tile (clamped: a row past the last is not stored)
    const __nv_bfloat16* sf = p.sf + row0 * (K / G);
    int st = tile0 + gi, su = U0 + ks;
    const Scales* srow = nullptr;
    auto scale_row = [&]() {
        const int f = st * kTile + (EPI == W4_GATED ? lane & 15 : lane);
        const size_t row = (size_t)(f < p.F ? f : p.F - 1) + (EPI == W4_GATED && lane >= 16 ? p.F : 0);
        srow = reinterpret_cast<const Scales*>(sf + row * (K / G));
    };
    Scales snext[2] = {};
    auto fetch_scales = [&]() {
        if (st < tile1 && su < U) {
            snext[0] = __ldg(srow + 2 * su);
            snext[1] = 2 * su + 1 < KB ? __ldg(srow + 2 * su + 1) : Scales{};
            su += KS;
            if (su >= U) {
                su = U0 + ks;
                st += NG;
                scale_row();
            }
        }
    };
    scale_row();
    fetch_scales();

    // ---- x and its group sums
    asm volatile("griddepcontrol.wait;" ::: "memory");  // x may be the previous kernel's
    // A unit past an odd last block meets zeros: codes beyond the matrix's rows
    // (filled by the copy), x, its sums and the scales.
    const int xst = per * 256 + 32;  // elements between rows of x in shared memory
    if (kn & 255) {  // an odd last block
        for (int v = threadIdx.x; v < n * 16; v += blockDim.x)
            *reinterpret_cast<uint4*>(xsm + (v >> 4) * xst + kn + (v & 15) * 8) = make_uint4(0u, 0u, 0u, 0u);
        for (int v = threadIdx.x; v < (128 / G) * kRows; v += blockDim.x) xs[(kn / G) * kRows + v] = 0.0f;
    }
    for (int v = threadIdx.x; v < n * (kn / 8); v += blockDim.x) {  // kn / 8 is a multiple of 16: whole groups per row
        const int r = v / (kn / 8), c = v - r * (kn / 8);
        const uint4 u = *(reinterpret_cast<const uint4*>(p.x + (size_t)(row_of[r] / p.xdiv) * K + k0) + c);
        *reinterpret_cast<uint4*>(xsm + r * xst + c * 8) = u;
        float f[8], s = 0.0f;
        unpack_bf16x8(u, f);
#pragma unroll
        for (int i = 0; i < 8; ++i) s += f[i];
        // the last warp may be half full: groups of G / 8 <= 16 lanes stay whole
        const uint32_t act = v - lane + 32 <= n * (kn / 8) ? 0xffffffffu : 0x0000ffffu;
#pragma unroll
        for (int d = 1; d < G / 8; d <<= 1) s += __shfl_xor_sync(act, s, d);
        if ((c & (G / 8 - 1)) == 0) xs[(c / (G / 8)) * kRows + r] = -136.0f * s;
    }
    __syncthreads();

    // this lane's rows (a row past the job's repeats the last)
    const uint4* xrow[kNt];
#pragma unroll
    for (int nt = 0; nt < kNt; ++nt)
        xrow[nt] = reinterpret_cast<const uint4*>(xsm + (8 * nt + g < n ? 8 * nt + g : n - 1) * xst) + t;
    // y of feature f and row r of the job
    auto emit = [&](int f, int r, float v, float up) {
        if (f >= p.F || r >= n) return;
        const size_t o = (size_t)row_of[r] * p.F + f;
        if constexpr (EPI == W4_SLOT) {
            reinterpret_cast<float*>(p.out)[o] = __ldg(p.slot_w + row_of[r]) * v;
        } else {
            if constexpr (EPI == W4_GATED) {
                v = clamp_keep_nan(v, p.clamp);
                v = v / (1.0f + expf(-v)) * clamp_keep_nan(up, p.clamp);
            }
            reinterpret_cast<__nv_bfloat16*>(p.out)[o] = __float2bfloat16_rn(v);
        }
    };

    const uint32_t mask = p.mask;
    // 16-byte chunk 4 h + t of this lane's row of a fragment: swizzled by the row
    const uint32_t chunk[2] = {(uint32_t)(g * 128 + ((t ^ g) << 4)), (uint32_t)(g * 128 + (((4 + t) ^ g) << 4))};
    int slot = 0, buf = 0;
    uint32_t phase = 0;
    // every warp of a cluster takes part in its barriers: as many rounds for all
    const int rounds = (tile1 - tile0 + NG - 1) / NG;
    if (p.kparts > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    for (int round = 0; round < rounds; ++round) {
        const int tile = tile0 + gi + round * NG;
        const bool live = tile < tile1;
        if (kNt == 1 && p.kparts == 1 && !live) break;
        float acc[kNt][2][4];
        auto fill = [&](float v) {
#pragma unroll
            for (int i = 0; i < 8 * kNt; ++i) acc[i >> 3][(i >> 2) & 1][i & 3] = v;
        };
        fill(0.0f);
        for (int u = live ? U0 + ks : U; u < U; u += KS) {
            const Scales sc2[2] = {snext[0], snext[1]};
            fetch_scales();
            fetch();
            // a wait that gave up leaves NaN in the outputs and lets the others go
            if (!warp_wait(bar + 8 * slot, phase, abort)) fill(__uint_as_float(0x7fc00000u));
            const uint32_t unit = ring + slot * kUnitBytes;
#pragma unroll
            for (int h0 = 0; h0 < 2; h0 += kSide) {
                uint4 w[kSide][kFrag];
                uint32_t sc[kSide][kFrag][kSw];
#pragma unroll
                for (int h = 0; h < kSide; ++h)
#pragma unroll
                    for (int i = 0; i < kFrag; ++i) {
                        const int4 v = ld_shared_v4s(unit + i * 1024 + chunk[h0 + h]);
                        w[h][i] = make_uint4(v.x, v.y, v.z, v.w);
                        scales_of(sc2[h0 + h], g + 8 * i, sc[h][i]);
                    }
                float c[kSide][kNt][2][4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
#pragma unroll
                    for (int h = 0; h < kSide; ++h) {
                        const int kb = 2 * (u - U0) + h0 + h;  // of this block's part
                        uint4 b[kNt];
                        float2 start[kNt];
#pragma unroll
                        for (int nt = 0; nt < kNt; ++nt) {
                            b[nt] = xrow[nt][kb * 16 + j * 4];
                            if (j % (G / 32) == 0)
                                start[nt] = *reinterpret_cast<const float2*>(xs + ((kb * 128 + j * 32) / G) * kRows +
                                                                             8 * nt + 2 * t);
                        }
#pragma unroll
                        for (int rt = 0; rt < 2; ++rt) {
                            const uint32_t a0 = word_of(w[h][2 * rt], j), a1 = word_of(w[h][2 * rt + 1], j);
                            const uint32_t u0 = pair128<0>(a0, mask), u1 = pair128<1>(a0, mask),
                                           u2 = pair128<2>(a0, mask), u3 = pair128<3>(a0, mask);
                            const uint32_t v0 = pair128<0>(a1, mask), v1 = pair128<1>(a1, mask),
                                           v2 = pair128<2>(a1, mask), v3 = pair128<3>(a1, mask);
#pragma unroll
                            for (int nt = 0; nt < kNt; ++nt) {
                                float(&d)[4] = c[h][nt][rt];
                                if (j % (G / 32) == 0)
                                    mma_bf16_from(d, u0, v0, u1, v1, b[nt].x, b[nt].y, start[nt].x, start[nt].y);
                                else
                                    mma_bf16(d, u0, v0, u1, v1, b[nt].x, b[nt].y);
                            }
#pragma unroll
                            for (int nt = 0; nt < kNt; ++nt) mma_bf16(c[h][nt][rt], u2, v2, u3, v3, b[nt].z, b[nt].w);
                        }
                    }
                    if ((j + 1) % (G / 32) == 0) {
                        const int si = j / (G / 32);
#pragma unroll
                        for (int h = 0; h < kSide; ++h)
#pragma unroll
                            for (int rt = 0; rt < 2; ++rt) {
                                const float s0 = scale(sc[h][2 * rt][si / 2], si),
                                            s1 = scale(sc[h][2 * rt + 1][si / 2], si);
#pragma unroll
                                for (int nt = 0; nt < kNt; ++nt) {
                                    float(&o)[4] = acc[nt][rt];
                                    const float(&d)[4] = c[h][nt][rt];
                                    o[0] = fmaf(s0, d[0], o[0]);
                                    o[1] = fmaf(s0, d[1], o[1]);
                                    o[2] = fmaf(s1, d[2], o[2]);
                                    o[3] = fmaf(s1, d[3], o[3]);
                                }
                            }
                    }
                }
            }
            __syncwarp();  // every lane has read the slot before it is filled again
            if (++slot == kSlots) {
                slot = 0;
                phase ^= 1u;
            }
        }
        // register i of lane (g, t) of operand rt: row 16 rt + g + 8 (i / 2) of
        // the tile, row 2 t + i % 2 of the column tile nt: pair q = 4 nt + i of them
        auto put = [&](int q, float v0, float v1) {
            const int f = tile * kTile + g + 8 * ((q >> 1) & 1), r = 8 * (q >> 2) + 2 * t + (q & 1);
            if constexpr (EPI == W4_GATED) {
                emit(f, r, v0, v1);
            } else {
                emit(f, r, v0, 0.0f);
                emit(f + 16, r, v1, 0.0f);
            }
        };
        constexpr int kPairs = 4 * kNt;
        if (kNt == 1 && KS == 1 && p.kparts == 1) {
#pragma unroll
            for (int q = 0; q < kPairs; ++q) put(q, acc[q >> 2][0][q & 3], acc[q >> 2][1][q & 3]);
        } else {
            // The pairs of a tile: [warp][pair][operand][lane].  A cluster's blocks
            // finish a share of them each: [part][warp][pair of the share].. there
            constexpr int kPer = kPairs * 64;  // floats of a warp
            if (kNt > 1 || p.kparts > 1) {
                const int log_share = 31 - __clz(kPairs / p.kparts), share = 1 << log_share;  // kparts is 2 or 4
                const float* mine = red + ((part * nw + warp) << log_share) * 64 + lane;
                // every block has started, and has read the last round's sums
                asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
#pragma unroll
                for (int q = 0; q < kPairs; ++q) {
                    const uint32_t to = cluster_addr_of(smem_addr(mine + (q & (share - 1)) * 64), q >> log_share);
                    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to), "f"(acc[q >> 2][0][q & 3]) : "memory");
                    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to + 128), "f"(acc[q >> 2][1][q & 3]) : "memory");
                }
                asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
                if (live) {
                    for (int i = ks; i < share; i += KS) {
                        float v0 = 0.0f, v1 = 0.0f;
                        for (int c = 0; c < p.kparts; ++c)
                            for (int k = 0; k < KS; ++k) {
                                const float* o = red + (((c * nw + gi * KS + k) << log_share) + i) * 64 + lane;
                                v0 += o[0];
                                v1 += o[32];
                            }
                        put(part * share + i, v0, v1);
                    }
                }
                asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
            } else {
                float* mine = red + (size_t)(buf * nw + warp) * kPer + lane;
#pragma unroll
                for (int q = 0; q < kPairs; ++q) {
                    mine[q * 64] = acc[q >> 2][0][q & 3];
                    mine[q * 64 + 32] = acc[q >> 2][1][q & 3];
                }
                asm volatile("bar.sync %0, %1;" ::"r"(gi + 1), "r"(KS * 32) : "memory");
                const float* all = red + (size_t)(buf * nw + gi * KS) * kPer + lane;
                for (int q = ks; q < kPairs; q += KS) {
                    float v0 = 0.0f, v1 = 0.0f;
                    for (int k = 0; k < KS; ++k) {
                        v0 += all[k * kPer + q * 64];
                        v1 += all[k * kPer + q * 64 + 32];
                    }
                    put(q, v0, v1);
                }
                buf ^= 1;  // two halves in turn: two tiles on, this barrier has passed
            }
        }
    }
    if (p.kparts > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (*abort) {  // copies in flight land before the block's shared memory goes
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 2000000ull) {
        }
    }
}

// y[token] = sum over its slots in order of o[slot], skipping dropped ones.
__global__ void __launch_bounds__(256) w4_combine_kernel(const float* o, const int32_t* __restrict__ ids,
                                                         int T, int k, int E, int H, __nv_bfloat16* __restrict__ y) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const long long n4 = (long long)T * H / 4;
    for (long long v = (long long)blockIdx.x * 256 + threadIdx.x; v < n4; v += (long long)gridDim.x * 256) {
        const int tok = (int)(v * 4 / H), h = (int)(v * 4 - (long long)tok * H);
        float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
        for (int j = 0; j < k; ++j) {
            const int e = __ldg(ids + (size_t)tok * k + j);
            float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (e >= 0 && e < E) a = *reinterpret_cast<const float4*>(o + ((size_t)tok * k + j) * H + h);
            s.x += a.x;
            s.y += a.y;
            s.z += a.z;
            s.w += a.w;
        }
        uint2 u;
        u.x = pack_bf16x2(s.x, s.y);
        u.y = pack_bf16x2(s.z, s.w);
        *reinterpret_cast<uint2*>(y + (size_t)tok * H + h) = u;
    }
}

// W bf16 [E][K][N] -> codes [E][N][K / 2] and scales [E][N][K / G]: one thread
// per column and 128-code block.  Scale = max|w| / 7 rounded to bf16 (0 for a
// zero group), code = round(w / scale) + 8 in [0, 15].
template <int G>
__global__ void __launch_bounds__(128) w4_quantize_kernel(const __nv_bfloat16* __restrict__ W, int K, int N,
                                                          uint8_t* __restrict__ q, __nv_bfloat16* __restrict__ sf) {
    const int n = blockIdx.x * 128 + threadIdx.x;
    if (n >= N) return;
    const int kb = blockIdx.y;
    const size_t e = blockIdx.z;
    const __nv_bfloat16* w = W + (e * K + (size_t)kb * 128) * N + n;
    uint32_t words[16];
    float scale = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (j % (G / 32) == 0) {
            float amax = 0.0f;
            for (int i = 0; i < G; ++i) amax = fmaxf(amax, fabsf(__bfloat162float(__ldg(w + (size_t)(j * 32 + i) * N))));
            const __nv_bfloat16 s = __float2bfloat16_rn(amax / 7.0f);
            sf[(e * N + n) * (size_t)(K / G) + kb * (128 / G) + j / (G / 32)] = s;
            scale = __bfloat162float(s);
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            uint32_t u = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float v = __bfloat162float(__ldg(w + (size_t)(j * 32 + t * 8 + i) * N));
                const float r = scale > 0.0f ? rintf(v / scale) : 0.0f;
                const int code = (int)fminf(fmaxf(r, -8.0f), 7.0f) + 8;
                u |= (uint32_t)code << (4 * (i / 2 + 4 * (i & 1)));
            }
            words[t * 4 + j] = u;
        }
    }
    uint4* out = reinterpret_cast<uint4*>(q + (e * N + n) * (size_t)(K / 2) + (size_t)kb * 64);
#pragma unroll
    for (int t = 0; t < 4; ++t) out[t] = make_uint4(words[4 * t], words[4 * t + 1], words[4 * t + 2], words[4 * t + 3]);
}

constexpr int kW4Smem = 224 * 1024;  // dynamic shared memory of a block
constexpr int kSmSmem = 228 * 1024;  // of an SM, with 1 KB taken by every block

// Launch shape: warps per tile and tiles per block for blocks of nw warps,
// per_sm of them on an SM.  Two times bound a choice, and the larger one is
// made small: the busiest SM's units at the rate of its warps, and the longest
// chain of a warp over the blocks that follow one another.  In clocks, fitted
// to sweeps of both at 1 to 32 tokens: an SM takes 280 per unit with 16 warps,
// 437 with 8 (two column tiles: 340, 675); a warp alone 2200 (3200); a join of
// warps 600, and 100 of the SM's per warp of it, of a cluster 4000, in which all
// its blocks stand still; a block's start (job, x) 1200 and a third per element
// of x.  Clusters of four find room for 144 blocks on the 152 SMs (148 take
// twice as long); a few are left to another GPU's layout.
void w4_shape(W4Args* a, int jobs, int nw, int per_sm, int nt) {
    const long long U = w4_units(a->K, a->kparts), sms = a->kparts > 2 ? 136 : 152, slots = sms * per_sm;
    const long long start = 1200 + (long long)a->R * a->K / a->kparts / 3;
    long long best = -1;
    for (int ks = 1; ks <= nw; ks *= 2) {
        const int ng = nw / ks, join = a->kparts > 1 ? 4000 : ks > 1 ? 600 : 0, lone = nt > 1 ? 3200 : 2200;
        for (int rounds = 1; rounds <= 64; ++rounds) {
            const int tpc = ng * rounds;
            const long long tiles = tpc < a->tiles ? tpc : a->tiles;
            const long long blocks = (long long)jobs * a->kparts * ((a->tiles + tpc - 1) / tpc), on_sm = (blocks + sms - 1) / sms;
            const long long warps = (on_sm < per_sm ? on_sm : per_sm) * nw;
            const long long unit = nt > 1 ? 5400 / warps : 3500 / warps > 280 ? 3500 / warps : 280;
            const long long rate = on_sm * (tiles * (U * unit + (join ? 100 * ks : 0)) + (a->kparts > 1 ? rounds * join : 0) + start);
            const long long lat = (blocks + slots - 1) / slots * (3000 + rounds * (lone * ((U + ks - 1) / ks) + join));
            const long long cost = (lat > rate ? lat : rate) * 8 + (lat < rate ? lat : rate);
            if (best < 0 || cost < best) {
                best = cost;
                a->ks = ks;
                a->tpc = tpc;
            }
            if (tpc >= a->tiles) break;
        }
    }
}

// rows: rows that can share a job; groups of rows (no ids) or slots (ids) are
// the jobs.  after_own: the kernel before it in the stream is this file's and
// writes x only, so this one may start, find its job and fetch weights, while
// that one drains (it waits before it reads x).
template <int G, int EPI, int kNt>
int w4_launch(W4Args a, const uint8_t* q, int rows, bool after_own, const char* name, cudaStream_t st) {
    static SmemLimit limit;
    a.mask = 0x000f000fu;
    a.tiles = EPI == W4_GATED ? (a.F + 15) / 16 : (a.F + 31) / 32;
    constexpr int kRows = kR * kNt;
    a.R = (rows + (rows + kRows - 1) / kRows - 1) / ((rows + kRows - 1) / kRows);  // 20 rows: 10 and 10
    // K is split over a cluster where the rows of x leave an SM fewer than 16
    // warps (8 rows of a 7168 x 7168 matrix: 26.6 us with 8 warps, 17.2 us with
    // 16 and half of K each); where four parts are not enough, fewer rows per job.
    a.kparts = kNt;  // (two column tiles: the joins of a cluster alone)
    auto sixteen = [&](int parts) {  // one block of 16 warps or two of 8 fit an SM
        return w4_smem<G, kNt>(a.K, 16, a.R, parts).total <= kW4Smem ||
               2 * (w4_smem<G, kNt>(a.K, 8, a.R, parts).total + 1024) <= kSmSmem;
    };
    while (a.kparts < 4 && !sixteen(a.kparts) && w4_units(a.K, 2 * a.kparts) >= (kNt > 1 ? 4 : 8)) a.kparts *= 2;
    while (a.R > 1 && w4_smem<G, kNt>(a.K, 4, a.R, a.kparts).total > kW4Smem) --a.R;
    auto bytes = [&](int nw) { return w4_smem<G, kNt>(a.K, nw, a.R, a.kparts).total; };
    const int per_sm = 2 * (bytes(8) + 1024) <= kSmSmem ? 2 : 1;
    const int nw = per_sm == 2 ? 8 : bytes(16) <= kW4Smem ? 16 : bytes(8) <= kW4Smem ? 8 : 4;
    const int jobs = a.ids ? a.slots : (a.rows + a.R - 1) / a.R;
    w4_shape(&a, a.ids ? a.busy : jobs, nw, per_sm, kNt);
    if (const int e = limit.allow(w4_kernel<G, EPI, kNt>, kW4Smem)) return e;
    CUtensorMap m;
    if (abi_map_u8(&m, q, (long long)a.E * a.N, a.K / 2, 128, EPI == W4_GATED ? 16 : 32, "4-bit codes"))
        return (int)cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    int na = 0;
    if (after_own) {
        attr[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[na++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (a.kparts > 1) {
        attr[na].id = cudaLaunchAttributeClusterDimension;
        attr[na].val.clusterDim.x = attr[na].val.clusterDim.y = 1;
        attr[na++].val.clusterDim.z = a.kparts;
    }
    cfg.gridDim = dim3((a.tiles + a.tpc - 1) / a.tpc, jobs, a.kparts);
    cfg.blockDim = dim3(nw * 32);
    cfg.dynamicSmemBytes = bytes(nw);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = na;
    trace_pre(st);
    const cudaError_t e = cudaLaunchKernelEx(&cfg, w4_kernel<G, EPI, kNt>, m, a);
    trace_post(st, name);
    return (int)(e != cudaSuccess ? e : cudaGetLastError());
}
template <int G, int EPI>
int w4_launch_n(const W4Args& a, const uint8_t* q, int rows, bool after_own, const char* name, cudaStream_t st) {
    // More than eight rows of one matrix: two column tiles, the weights unpacked
    // once for 16 rows, where x leaves an SM 16 warps (16 rows, one or two tiles,
    // us: 16384 x 7168 G = 32 40.6 | 32.1, G = 128 34.6 | 25.6, 4096 x 4096 G =
    // 128 11.1 | 9.2) and the matrix has work for them (2048 x 2048 G = 32 6.3 |
    // 8.0, 1408 x 4096 at 12 rows 8.0 | 9.5).  An expert seldom has so many rows
    // that its second tile pays (32 tokens, top 2 of 8 experts of 2048 x 1408:
    // 35.4 | 51.5).
    if constexpr (EPI != W4_SLOT) {
        const bool two = rows > kR && !a.ids && (long long)a.N * a.K > (1 << 23) && a.K >= 1024 &&
                         w4_smem<G, 2>(a.K, 16, 2 * kR, 4).total <= kW4Smem;
        if (two) return w4_launch<G, EPI, 2>(a, q, rows, after_own, name, st);
    }
    return w4_launch<G, EPI, 1>(a, q, rows, after_own, name, st);
}
template <int EPI>
int w4_launch_g(int G, const W4Args& a, const uint8_t* q, int rows, bool after_own, const char* name,
                cudaStream_t st) {
    return G == 32   ? w4_launch_n<32, EPI>(a, q, rows, after_own, name, st)
           : G == 64 ? w4_launch_n<64, EPI>(a, q, rows, after_own, name, st)
                     : w4_launch_n<128, EPI>(a, q, rows, after_own, name, st);
}

}  // namespace

int launch_matvec_w4(int M, int N, int K, int G, const void* x, const uint8_t* q, const void* sf, void* y,
                     cudaStream_t st) {
    W4Args a = {};
    a.x = static_cast<const __nv_bfloat16*>(x);
    a.sf = static_cast<const __nv_bfloat16*>(sf);
    a.N = a.F = N;
    a.K = K;
    a.E = 1;
    a.rows = M;
    a.xdiv = 1;
    a.out = y;
    return w4_launch_g<W4_PLAIN>(G, a, q, M, false, "matvec_w4", st);
}

int launch_experts_w4(const W4Experts& w, cudaStream_t st) {
    W4Args a = {};
    a.x = static_cast<const __nv_bfloat16*>(w.x);
    a.sf = static_cast<const __nv_bfloat16*>(w.W1_sf);
    a.N = 2 * w.I;
    a.F = w.I;
    a.K = w.H;
    a.E = w.E;
    a.rows = w.T;
    a.ids = w.topk_idx;
    a.slots = w.T * w.k;
    // experts that uniform routing would touch, at most one per slot
    const double touched = w.E * (1.0 - pow(1.0 - (double)w.k / w.E, (double)w.T));
    a.busy = touched < 1.0 ? 1 : touched < a.slots ? (int)(touched + 0.5) : a.slots;
    a.xdiv = w.topk_idx ? w.k : 1;
    a.out = w.act;
    a.clamp = w.clamp;
    // Rows that a job is made for: twice an expert's mean share of the slots,
    // and one (an expert with more has several jobs).  More would cost shared
    // memory, so warps.
    const long long share = w.topk_idx ? (2ll * w.T * w.k + w.E - 1) / w.E + 1 : w.T;
    const int rows = (int)(share < w.T ? share : w.T);
    if (const int e = w4_launch_g<W4_GATED>(w.group, a, w.W1_q, rows, false, "experts_w4_gate_up", st)) return e;
    a.x = static_cast<const __nv_bfloat16*>(w.act);
    a.sf = static_cast<const __nv_bfloat16*>(w.W2_sf);
    a.N = a.F = w.H;
    a.K = w.I;
    a.xdiv = 1;
    if (!w.topk_idx) {
        a.out = w.y;
        return w4_launch_g<W4_PLAIN>(w.group, a, w.W2_q, rows, true, "experts_w4_down", st);
    }
    a.slot_w = w.topk_w;
    a.out = w.part;
    if (const int e = w4_launch_g<W4_SLOT>(w.group, a, w.W2_q, rows, true, "experts_w4_down", st)) return e;
    const long long blocks = ((long long)w.T * w.H / 4 + 255) / 256;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)(blocks < 1216 ? blocks : 1216));
    cfg.blockDim = dim3(256);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    trace_pre(st);
    const cudaError_t e = cudaLaunchKernelEx(&cfg, w4_combine_kernel, (const float*)w.part, w.topk_idx, w.T, w.k, w.E,
                                             w.H, static_cast<__nv_bfloat16*>(w.y));
    trace_post(st, "experts_w4_combine");
    return (int)(e != cudaSuccess ? e : cudaGetLastError());
}

int launch_quantize_w4(int E, int K, int N, int G, const void* W, uint8_t* q, void* sf, cudaStream_t st) {
    const dim3 grid((N + 127) / 128, K / 128, E);
    auto* w = static_cast<const __nv_bfloat16*>(W);
    auto* s = static_cast<__nv_bfloat16*>(sf);
    trace_pre(st);
    if (G == 32)
        w4_quantize_kernel<32><<<grid, 128, 0, st>>>(w, K, N, q, s);
    else if (G == 64)
        w4_quantize_kernel<64><<<grid, 128, 0, st>>>(w, K, N, q, s);
    else
        w4_quantize_kernel<128><<<grid, 128, 0, st>>>(w, K, N, q, s);
    trace_post(st, "quantize_w4");
    return (int)cudaGetLastError();
}

}  // namespace moe
