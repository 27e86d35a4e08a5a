// Forward of the dense gated feed-forward block for a few tokens (decoding):
//   h = x W1,  a = silu(h_g) h_u      and      y = a W2
// with W1 [H][2][I] and W2 [I][H] as they are (rows along the output).
//
// Bound by DRAM: every weight is read once and used for few products, so what
// counts is that every SM streams.  A tile of 64 output features (gated: 64 gate
// and the same 64 up features) goes to a cluster of up to four blocks that
// split K; the warps of a block split its part in units of 4 KB of weights with
// the x that they meet, fetched by TMA by each warp for itself, kFewSlots - 1
// ahead.  The FP32 sums of warps and blocks are joined in a fixed order through
// shared memory, every block of the cluster finishing a share of them.
//
// mma m16n8k16 with the weights as A (16 features x 16 of K, transposed out of
// the box by ldmatrix) and eight tokens as B; kNt such groups of tokens.
//
// Measured, 8 tokens (the 256-row tiles of the large form; the weights' bytes at
// the copy rate): 7168 x 2048 20.0 us (32.1; 13.0), 2048 x 1408 8.9 us (20.1;
// 2.6), 7168 x 18432 127 us (165; 117), and 16 tokens 21.7, 10.3 and 133 us
// (29.7, 20.5 and 137).
#include "clamp.cuh"
#include "grouped_gemm_2sm.cuh"
#include "smem_limit.h"

namespace moe {

namespace {

constexpr int kFewSlots = 3;
constexpr int kFewUnit = 4096;  // gated: 16 rows of K x (64 gate + 64 up); plain: 32 rows x 64
constexpr int kFewWarps = 8;
constexpr int kFewSmem = 113 * 1024;  // two blocks on an SM
constexpr int kFewLone = 115 * 1024;  // one block on an SM, beside one of the gated kernel's

struct FewArgs {
    int T, K, F;      // F: output features (gated: of one half)
    int kparts, per;  // blocks of a cluster, units of one
    float clamp;
    __nv_bfloat16* out;  // [T][F]
    float* h;            // gated: [T][2][F] or null
    int32_t* status;
};

__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t& a, uint32_t& b, uint32_t& c, uint32_t& d) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(a), "=r"(b), "=r"(c), "=r"(d)
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldmatrix_x4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldmatrix_x2(uint32_t addr, uint32_t& a, uint32_t& b) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x2.shared.b16 {%0,%1}, [%2];" : "=r"(a), "=r"(b) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma_few(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Bytes of a unit's x and of a block's shared memory.
__host__ __device__ constexpr int few_x_bytes(bool gated, int nt) { return nt * (gated ? 256 : 512); }
__host__ __device__ constexpr int few_smem(bool gated, int nt, int warps) {
    return 1024 + warps * kFewSlots * (kFewUnit + few_x_bytes(gated, nt) + 8);
}
__host__ __device__ constexpr int few_warps(bool gated, int nt) {
    int w = kFewWarps;
    while (few_smem(gated, nt, w) > kFewSmem) --w;
    return w;
}

static_assert(few_smem(true, 2, few_warps(true, 2)) + kFewLone + 2048 <= 228 * 1024, "one block of each kernel");

// Grid: (tiles of 64 features, jobs of 8 kNt tokens, kparts); clusters along z.
template <bool kGated, int kNt>
__global__ void __launch_bounds__(kFewWarps * 32, 2)
ffn_few_kernel(const __grid_constant__ CUtensorMap mW, const __grid_constant__ CUtensorMap mX, const FewArgs p) {
    constexpr int kDepth = kGated ? 16 : 32;    // of K in a unit
    constexpr int kMt = kGated ? 8 : 4;         // 16-feature tiles
    constexpr int kOut = 512 * kNt;             // outputs of a tile
    constexpr int kSums = kMt * 128 * kNt;      // its FP32 sums: gated, gate then up
    constexpr int kWarps = few_warps(kGated, kNt), kHalf = (kWarps + 1) / 2;
    constexpr uint32_t kX = few_x_bytes(kGated, kNt);
    static_assert((kHalf + 1) * kSums * 4 <= kWarps * kFewSlots * kFewUnit, "the joins take the ring's place");
    extern __shared__ uint8_t smem_raw[];
    __shared__ int abort_word;
    volatile int* abort = &abort_word;
    const uint32_t raw = smem_addr(smem_raw), base = (raw + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (base - raw);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int part = blockIdx.z;

    const int units = (p.K + kDepth - 1) / kDepth;
    const int u0 = part * p.per, u1 = u0 + p.per < units ? u0 + p.per : units;
    const int row0 = blockIdx.y * 8 * kNt, rows = p.T - row0 < 8 * kNt ? p.T - row0 : 8 * kNt;
    const int f0 = blockIdx.x * 64;
    const uint32_t ring = base + warp * kFewSlots * kFewUnit;
    const uint32_t xring = base + kWarps * kFewSlots * kFewUnit + warp * kFewSlots * kX;
    const uint32_t bar = base + kWarps * kFewSlots * (kFewUnit + kX) + warp * kFewSlots * 8;
    if (lane == 0) {
        for (int i = 0; i < kFewSlots; ++i) mbar_init(bar + 8 * i, 1);
        fence_mbar_init();
    }
    if (threadIdx.x == 0) *abort = 0;
    __syncthreads();

    // ---- this warp's units: u0 + warp, + kWarps, ..
    auto fetch_w = [&](int u, int slot) {
        const uint32_t b = bar + 8 * slot, dst = ring + slot * kFewUnit;
        mbar_arrive_expect_tx(b, kFewUnit + kX);
        if constexpr (kGated) {  // W1 viewed as [H][2][I]
            tma_load_3d(dst, &mW, f0, 0, u * kDepth, b);
            tma_load_3d(dst + kFewUnit / 2, &mW, f0, 1, u * kDepth, b);
        } else {
            tma_load_2d(dst, &mW, f0, u * kDepth, b);
        }
    };
    auto fetch_x = [&](int u, int slot) { tma_load_2d(xring + slot * kX, &mX, u * kDepth, row0, bar + 8 * slot); };
    int fu = u0 + warp;
    if (lane == 0)
        for (int i = 0; i < kFewSlots - 1; ++i)
            if (fu + i * kWarps < u1) fetch_w(fu + i * kWarps, i);
    asm volatile("griddepcontrol.wait;" ::: "memory");  // x may be the previous kernel's
    if (lane == 0)
        for (int i = 0; i < kFewSlots - 1; ++i)
            if (fu + i * kWarps < u1) fetch_x(fu + i * kWarps, i);
    fu += (kFewSlots - 1) * kWarps;

    float acc[kMt * kNt][4];
#pragma unroll
    for (int i = 0; i < kMt * kNt * 4; ++i) acc[i >> 2][i & 3] = 0.0f;
    // ldmatrix, weights: matrix l / 8 (features 0-7 and 8-15 of K rows 0-7, then
    // of rows 8-15), row l % 8; x: token l % 8, vector l / 8 of 8 of K
    const int lk = (lane & 7) + (lane >= 16 ? 8 : 0), lc = (lane >> 3) & 1, lr = lane & 7, lv = lane >> 3;
    int slot = 0;
    uint32_t phase = 0;
    for (int u = u0 + warp; u < u1; u += kWarps) {
        if (lane == 0 && fu < u1) {
            const int s = slot == 0 ? kFewSlots - 1 : slot - 1;
            fetch_w(fu, s);
            fetch_x(fu, s);
        }
        fu += kWarps;
        if (!warp_wait(bar + 8 * slot, phase, abort)) break;
        const uint32_t unit = ring + slot * kFewUnit, xu = xring + slot * kX;
        uint32_t b[kNt][4];
#pragma unroll
        for (int n = 0; n < kNt; ++n) {
            if constexpr (kGated)
                ldmatrix_x2(xu + (8 * n + lr) * 32 + (((lv & 1) ^ (lr >> 2)) << 4), b[n][0], b[n][1]);
            else
                ldmatrix_x4(xu + (8 * n + lr) * 64 + ((lv ^ (lr >> 1)) << 4), b[n]);
        }
#pragma unroll
        for (int s = 0; s < kDepth / 16; ++s) {
            const int k = 16 * s + lk;
#pragma unroll
            for (int m = 0; m < kMt; ++m) {
                // gated: tiles 0-3 of the gate's box, 4-7 of the up projection's
                const uint32_t box = unit + (kGated ? (m >> 2) * (kFewUnit / 2) : 0);
                const int c = 2 * (m & 3) + lc;
                uint32_t a0, a1, a2, a3;
                ldmatrix_x4_trans(box + k * 128 + ((c ^ (k & 7)) << 4), a0, a1, a2, a3);
#pragma unroll
                for (int n = 0; n < kNt; ++n)
                    mma_few(acc[m * kNt + n], a0, a1, a2, a3, b[n][2 * s], b[n][2 * s + 1]);
            }
        }
        __syncwarp();  // every lane has read the slot before it is filled again
        if (++slot == kFewSlots) {
            slot = 0;
            phase ^= 1u;
        }
    }
    // The next kernel's blocks take their places from here on: any sooner, and
    // they would crowd onto the SMs that are first to have room for a second one.
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // ---- the join: warps, then blocks.  The sums take the ring's place.
    __syncthreads();
    if (p.kparts > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    float4* red = reinterpret_cast<float4*>(smem);                     // [kHalf][kSums / 4]
    float* all = reinterpret_cast<float*>(smem + kHalf * kSums * 4);  // [kparts][gate, up][share], one share a block
    if (warp >= kHalf) {
#pragma unroll
        for (int i = 0; i < kMt * kNt; ++i)
            red[(warp - kHalf) * (kSums / 4) + i * 32 + lane] = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
    }
    __syncthreads();
    if (warp < kHalf) {
#pragma unroll
        for (int i = 0; i < kMt * kNt; ++i) {
            float4& r = red[warp * (kSums / 4) + i * 32 + lane];
            float4 v = warp + kHalf < kWarps ? r : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            r = make_float4(v.x + acc[i][0], v.y + acc[i][1], v.z + acc[i][2], v.w + acc[i][3]);
        }
    }
    __syncthreads();
    const int log_share = 31 - __clz(kOut / p.kparts), share = 1 << log_share;  // kparts is 1, 2 or 4
    constexpr int kHalves = kSums / kOut;
    if (p.kparts > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // all are past their rings
    for (int e = threadIdx.x; e < kSums / 4; e += kWarps * 32) {
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < kHalf; ++w) {
            const float4 r = red[w * (kSums / 4) + e];
            v = make_float4(v.x + r.x, v.y + r.y, v.z + r.z, v.w + r.w);
        }
        const int half = 4 * e / kOut, o = 4 * e % kOut, to = o >> log_share;
        const uint32_t dst = smem_addr(all + (part * kHalves + half) * share + o - to * share);
        asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(p.kparts > 1 ? cluster_addr_of(dst, to)
                                                                                       : dst),
                     "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
                     : "memory");
    }
    if (p.kparts > 1)
        cluster_sync();
    else
        __syncthreads();
    // sum (m kNt + n) 128 + 16 g + 4 t + i: feature 16 m + g + 8 (i / 2), token
    // 8 n + 2 t + i % 2; threads in the order of the features
    for (int q = threadIdx.x; q < share; q += kWarps * 32) {
        const int fl = q & 15, rl = (q >> 4) & 7, tile = (part * share + q) >> 7;
        const int j = (q & ~127) | (fl & 7) << 4 | rl >> 1 << 2 | fl >> 3 << 1 | (rl & 1);
        float v = 0.0f, up = 0.0f;
        for (int c = 0; c < p.kparts; ++c) {
            v += all[c * kHalves * share + j];
            if constexpr (kGated) up += all[(c * kHalves + 1) * share + j];
        }
        const int f = f0 + 16 * (tile / kNt) + fl, r = 8 * (tile % kNt) + rl;
        if (f >= p.F || r >= rows) continue;
        const size_t row = row0 + r;
        if constexpr (kGated) {
            if (p.h) {
                p.h[row * 2 * p.F + f] = v;
                p.h[row * 2 * p.F + p.F + f] = up;
            }
            const float gc = clamp_keep_nan(v, p.clamp), uc = clamp_keep_nan(up, p.clamp);
            v = gc / (1.0f + expf(-gc)) * uc;
        }
        p.out[row * p.F + f] = __float2bfloat16_rn(v);
    }
    if (*abort) {  // copies in flight land before the block's shared memory goes
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 2000000ull) {
        }
        if (threadIdx.x == 0) atomicOr(reinterpret_cast<int*>(p.status), 1);
    }
}

template <bool kGated, int kNt>
int launch_few(FewArgs a, const CUtensorMap& mw, const CUtensorMap& mx, bool after_own, const char* name,
               cudaStream_t st) {
    static SmemLimit limit;
    constexpr int kDepth = kGated ? 16 : 32, kBytes = few_smem(kGated, kNt, few_warps(kGated, kNt));
    const int tiles = (a.F + 63) / 64, jobs = (a.T + 8 * kNt - 1) / (8 * kNt);
    const int units = (a.K + kDepth - 1) / kDepth;
    // The split of K, us a forward of 8 tokens (H x I: this rule | without the
    // split | with twice the parts): a block for an SM, 7168 x 2048: 20.0 | 26.7
    // | 20.2, 8192 x 4096: 35.7 | 39.5 | 38.5, 2048 x 1408: 8.9 | 11.4 | 9.8, each
    // with two units a warp at least.
    a.kparts = 1;
    while (a.kparts < 4 && 2 * a.kparts * tiles * jobs <= 152 && units / (2 * a.kparts) >= 2 * kFewWarps) a.kparts *= 2;
    // A second block on half of the SMs or fewer leaves the rest idle at the end:
    // four times as many, where K is long enough to pay for the joins.  5120 x
    // 10240: 68.5 | 79.1 us, 5120 x 13824: 76.8 | 85.2; but 5120 x 15360: 93.9 |
    // 87.7, 2560 x 11520: 46.8 | 42.1.
    if (tiles * jobs > 152 && 2 * tiles * jobs <= 3 * 152 && units >= 256) a.kparts = 4;
    a.per = (units + a.kparts - 1) / a.kparts;
    // A down projection of no more blocks than SMs asks for so much that an SM
    // takes one of them beside a block of the first kernel, and no second one.
    const int bytes = !kGated && tiles * jobs * a.kparts <= 152 ? kFewLone : kBytes;
    if (const int e = limit.allow(ffn_few_kernel<kGated, kNt>, kFewLone)) return e;
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
    cfg.gridDim = dim3(tiles, jobs, a.kparts);
    cfg.blockDim = dim3(few_warps(kGated, kNt) * 32);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = na;
    trace_pre(st);
    const cudaError_t e = cudaLaunchKernelEx(&cfg, ffn_few_kernel<kGated, kNt>, mw, mx, a);
    trace_post(st, name);
    return (int)(e != cudaSuccess ? e : cudaGetLastError());
}

}  // namespace

// More than eight tokens: sixteen a job, each weight read once for them.  A
// small block's weights stay in the L2, and two jobs of eight have less to start
// (16 tokens, 512 x 256: 5.8 against 7.7 us; 1160 x 712: 7.8 against 9.0; but
// 2048 x 1408: 11.4 against 10.3, 7168 x 2048: 36.2 against 21.7).
static bool few_two(const moe_ffn_shape& s) { return s.T > 8 && (long long)s.H * s.I > (1 << 20); }

// Up to 16 tokens always; up to 128 while the jobs' tiles are not many more
// than the SMs (us, this form | the large one: 512 x 256, 128 tokens 6.2 | 11.3;
// 1160 x 712, 64: 9.7 | 14.4; 2048 x 1408, 32: 12.2 | 20.9, 96: 16.3 | 22.3, but
// 128, 256 tiles: 33.8 | 22.9; 4096 x 2048, 32: 18.3 | 25.8, but 64, 256 tiles:
// 29.1 | 27.6).
bool ffn_few_takes(const moe_ffn_shape& s) {
    const int per = few_two(s) ? 16 : 8, wide = s.H > s.I ? s.H : s.I;
    return s.T <= 16 || (s.T <= 128 && (long long)((s.T + per - 1) / per) * ((wide + 63) / 64) <= 200);
}

int launch_ffn_few(const moe_ffn_shape& s, const FfnPtrs& f, cudaStream_t st) {
    const bool two = few_two(s);
    int rc;
    CUtensorMap w1, w2, x, act;
    if ((rc = abi_map_nd(&w1, f.W1, 2, {s.I, 2, s.H}, {64, 1, 16}, "W1 (gate/up halves)"))) return rc;
    if ((rc = abi_map_2d(&w2, f.W2, 2, s.I, s.H, s.H, 64, 32, "W2"))) return rc;
    if ((rc = abi_map_2d(&x, f.x, 2, s.T, s.H, s.H, 16, two ? 16 : 8, "x"))) return rc;
    if ((rc = abi_map_2d(&act, f.a, 2, s.T, s.I, s.I, 32, two ? 16 : 8, "a"))) return rc;
    const float clamp = s.activation_clamp > 0.0f ? s.activation_clamp : INFINITY;
    const FewArgs up = {s.T, s.H, s.I, 0, 0, clamp, static_cast<__nv_bfloat16*>(f.a), f.h, f.status};
    int e = two ? launch_few<true, 2>(up, w1, x, false, "ffn_few_gate_up", st)
                : launch_few<true, 1>(up, w1, x, false, "ffn_few_gate_up", st);
    if (e) return abi_cuda_fail(e, "gate and up projection launch");
    const FewArgs down = {s.T, s.I, s.H, 0, 0, clamp, static_cast<__nv_bfloat16*>(f.y), nullptr, f.status};
    e = two ? launch_few<false, 2>(down, w2, act, true, "ffn_few_down", st)
            : launch_few<false, 1>(down, w2, act, true, "ffn_few_down", st);
    return e ? abi_cuda_fail(e, "down projection launch") : MOE_OK;
}

}  // namespace moe
