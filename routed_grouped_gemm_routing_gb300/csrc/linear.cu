// A projection with everything around its product, forward and backward:
//
//   z = x W + b     y = act(z) + r
//   dz = dy act'(z)     dx = dz W^T     dW = x^T dz     db = sum_rows dz     (dr = dy)
//
// 2 T K N operations forward, 4 T K N backward, bound by the tensor cores from a
// few hundred rows on.  The products are dense_pair.cuh's (256 x 256 tiles on
// pairs of SMs, tcgen05, operands by TMA as they lie).  The forward's epilogue
// takes the bias from L1, fetches the residual's boxes by TMA while the tile's
// products run, and leaves y (and for the backward z) by TMA: nothing of y is
// read or written twice.  Few tiles: the K range is split, FP32 partial sums
// are joined in a fixed order (linear_join).  Few rows: few_rows.cuh, every
// weight read once.
//
// z stays FP32 for the backward: a rounding of z would come on top of dz's and
// go into db without it.  dz is rounded once (an operand of dx and dW); db sums
// the unrounded FP32 dz in a fixed order.  Without an activation dz is dy itself,
// z is not kept and db takes one pass over dy, beside the products.
//
// Measured (operations at the burst rate, bytes at the copy rate): 8192 x 2048 x 7168
// with bias and residual 140 us forward (124), 271-285 us backward (248, under the power
// limit); 4096 x 2048 x 2816 with silu 42 + 67 us (24 + 49): 176 tiles are three rounds over 76
// pairs of SMs where 2.3 would do, and dz takes 16 us of its own; 8 x 2048 x 7168 9.7 us with
// the weights from DRAM (4.4), 5.8 with them in L2.
#include "dense_pair.cuh"
#include "few_rows.cuh"

namespace moe {

namespace {

// ---------------------------------------------------------------- forward
struct LinearArgs {
    DenseArgs d;
    LinearEpi e;
    __nv_bfloat16* y;
};

// 32 values of the bias, columns from n on; zero past N (a multiple of 8).
__device__ __forceinline__ void add_bias32(const LinearEpi& e, int n, int N, float (&v)[32]) {
    if (!e.bias) return;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        if (n + 8 * c >= N) return;
        if (e.bias_f32) {
            const float4* b = reinterpret_cast<const float4*>(static_cast<const float*>(e.bias) + n + 8 * c);
            const float4 lo = __ldg(b), hi = __ldg(b + 1);
            v[8 * c] += lo.x, v[8 * c + 1] += lo.y, v[8 * c + 2] += lo.z, v[8 * c + 3] += lo.w;
            v[8 * c + 4] += hi.x, v[8 * c + 5] += hi.y, v[8 * c + 6] += hi.z, v[8 * c + 7] += hi.w;
        } else {
            float f[8];
            unpack_bf16x8(__ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(e.bias) + n + 8 * c)), f);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[8 * c + j] += f[j];
        }
    }
}

template <int EPI>
__device__ void linear_epilogue(const CUtensorMap* mY, const CUtensorMap* mR, const CUtensorMap* mZ, const LinearArgs& a,
                                const DenseCta& c) {
    constexpr bool kR = EPI == EPI_LIN_R || EPI == EPI_LIN_RZ, kZ = EPI == EPI_LIN_Z || EPI == EPI_LIN_RZ;
    const DenseArgs& p = a.d;
    const uint32_t out = c.boxes + c.warp * dense_boxes<EPI>() * 4096, rin = out + 4096, zout = out + (kR ? 8192 : 4096);
    const uint32_t tempty[2] = {cluster_addr_of(c.bars.tempty(0), 0), cluster_addr_of(c.bars.tempty(1), 0)};
    const int part = c.warp >> 2, quad = c.warp & 3, lane = c.lane;
    int it = 0;
    uint32_t rphase = 0;
    for (DenseWalk<EPI> w(p); w.valid(); w.next(), ++it) {
        const DenseItem item = w.item();
        const int acc = it & 1, row0 = item.m0 + 128 * c.rank + 32 * quad;
        const bool live = row0 < p.M;
        const int last = p.width < p.N - item.n0 ? p.width : p.N - item.n0;
        auto fetch_r = [&](int k) {
            if (lane == 0) {
                mbar_arrive_expect_tx(c.bars.hin(c.warp), 4096u);
                tma_load_2d(rin, mR, item.n0 + 64 * k, row0, c.bars.hin(c.warp));
            }
        };
        if (kR && live && 64 * part < last) fetch_r(part);
        if (!warp_wait(c.bars.tfull(acc), (uint32_t)(it >> 1) & 1u, c.abort)) break;
        tc_fence_after();
        const uint32_t t = c.tmem + (uint32_t)(acc * 256) + ((uint32_t)(quad * 32) << 16);
        bool ok = true;
        if (live) {
#pragma unroll 1
            for (int k = part; 64 * k < last; k += 2) {
                uint32_t res[32], pk[32];
                if constexpr (kR) {
                    if (!warp_wait(c.bars.hin(c.warp), rphase, c.abort)) {
                        ok = false;
                        break;
                    }
                    rphase ^= 1u;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int4 u = ld_shared_v4s(rin + lane * 128 + ((j ^ (lane & 7)) << 4));
                        res[4 * j] = u.x, res[4 * j + 1] = u.y, res[4 * j + 2] = u.z, res[4 * j + 3] = u.w;
                    }
                    __syncwarp();
                    if (64 * (k + 2) < last) fetch_r(k + 2);
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float v[32];
                    tmem_ld32(t + 64 * k + 32 * h, v);
                    add_bias32(a.e, item.n0 + 64 * k + 32 * h, p.N, v);
                    if constexpr (kZ) {
                        if (lane == 0) bulk_wait_read<0>();
                        __syncwarp();
                        uint32_t zb[32];
#pragma unroll
                        for (int j = 0; j < 32; ++j) zb[j] = __float_as_uint(v[j]);
                        stage_row_sw128(zout, lane, zb);
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) {
                            tma_store_2d(mZ, item.n0 + 64 * k + 32 * h, row0, zout);
                            bulk_commit();
                        }
                    }
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        float lo = act_apply(a.e.act, v[2 * j]), hi = act_apply(a.e.act, v[2 * j + 1]);
                        if constexpr (kR) {
                            const uint32_t r2 = res[16 * h + j];
                            const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&r2));
                            lo += f.x, hi += f.y;
                        }
                        pk[16 * h + j] = pack_bf16x2(lo, hi);
                    }
                }
                if (lane == 0) bulk_wait_read<0>();
                __syncwarp();
                stage_row_sw128(out, lane, pk);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    tma_store_2d(mY, item.n0 + 64 * k, row0, out);
                    bulk_commit();
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

template <int EPI>
__global__ void __launch_bounds__(kDenseThreads, 1)
    linear_pair_kernel(const __grid_constant__ CUtensorMap mA, const __grid_constant__ CUtensorMap mB,
                       const __grid_constant__ CUtensorMap mY, const __grid_constant__ CUtensorMap mR,
                       const __grid_constant__ CUtensorMap mZ, const LinearArgs a) {
    if (threadIdx.x == 32 * kDenseWarpTma) {
        tma_prefetch_map(&mA);
        tma_prefetch_map(&mB);
        tma_prefetch_map(&mY);
        if (EPI == EPI_LIN_R || EPI == EPI_LIN_RZ) tma_prefetch_map(&mR);
        if (EPI == EPI_LIN_Z || EPI == EPI_LIN_RZ) tma_prefetch_map(&mZ);
    }
    const DenseCta c = dense_begin<EPI>(a.d.gave_up);
    if (c.warp == kDenseWarpTma) {
        if (c.lane == 0) dense_producer<KN, EPI>(&mA, &mB, a.d, c.ring, c.bars, c.abort, c.rank);
    } else if (c.warp == kDenseWarpMma) {
        if (c.rank == 0) {
            dense_mma<KN, EPI>(a.d, c.ring, c.bars, c.tmem, c.abort);
            dense_drain(c);
        }
    } else {
        linear_epilogue<EPI>(&mY, &mR, &mZ, a, c);
    }
    dense_end(c, a.d.status);
    if (*c.abort) {
        for (DenseWalk<EPI> w(a.d); w.valid(); w.next()) {
            const DenseItem it = w.item();
            const int2 r = dense_own_rows(c, it.m0, a.d.M);
            const int last = it.n0 + a.d.width < a.d.N ? it.n0 + a.d.width : a.d.N;
            dense_bad_tile(a.y, a.d.N, r.x, r.y, it.n0, last);
            dense_bad_tile(a.e.z, a.d.N, r.x, r.y, it.n0, last);
        }
    }
}

// The sum of the K ranges' partial sums [splits][T][N] in order and the layer's
// epilogue, eight columns per thread.
__global__ void __launch_bounds__(128)
    linear_join_kernel(const float* part, long long rows, int N, int splits, const LinearEpi e, __nv_bfloat16* y) {
    asm volatile("griddepcontrol.launch_dependents;\n\tgriddepcontrol.wait;" ::: "memory");
    const int per = N / 8;
    const long long total = rows * per;
    const size_t stride = (size_t)rows * N;
    for (long long i = (long long)blockIdx.x * 128 + threadIdx.x; i < total; i += (long long)gridDim.x * 128) {
        const long long row = i / per;
        const int c = (int)(i - row * per) * 8;
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = 0.0f;
        const float* src = part + (size_t)row * N + c;
#pragma unroll 4
        for (int s = 0; s < splits; ++s) {
            const float4 a = *reinterpret_cast<const float4*>(src + s * stride);
            const float4 b = *(reinterpret_cast<const float4*>(src + s * stride) + 1);
            v[0] += a.x, v[1] += a.y, v[2] += a.z, v[3] += a.w;
            v[4] += b.x, v[5] += b.y, v[6] += b.z, v[7] += b.w;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = e.finish(v[j], row, c + j, N);
        *reinterpret_cast<uint4*>(y + (size_t)row * N + c) = pack8(v);
    }
}

// ---------------------------------------------------------------- backward
// dz of dy and z, and each block's column sums of it (part [gridDim.y][N]), or
// db itself from a single row of blocks or (kDzCluster) blocks that are a cluster.  A lane takes eight columns, a warp
// every eighth row of the block's.
struct DzArgs {
    const __nv_bfloat16* dy;
    long long dy_stride, rows;
    int N, per;  // rows of a block
    const float* z;
    __nv_bfloat16* dz;  // null: not wanted (no activation)
    float* part;        // null: no db
    void* db;           // without part
    int db_f32;
};
constexpr int kDzWarps = 8;
// With an activation: four blocks on an SM with two rows ahead each keep as much in
// flight as two with four rows and hide more of the slopes' arithmetic (4096 x 2816
// silu 19 -> 16 us, gelu 25.5 -> 22).
constexpr int kDzBlocks = 4;

__device__ __forceinline__ void store_db(void* db, int f32, int n, float v) {
    if (f32)
        static_cast<float*>(db)[n] = v;
    else
        static_cast<__nv_bfloat16*>(db)[n] = __float2bfloat16_rn(v);
}

// kDzBeside: runs beside the products of the other gradients (see the launch), with no
// shared memory, which they leave none of: a warp's sums are a row of part.
enum DzForm { kDzPlain, kDzBeside, kDzCluster };
template <int kAct, int kForm>
__global__ void __launch_bounds__(32 * kDzWarps, kAct == MOE_ACT_NONE ? 1 : kDzBlocks) linear_dz_kernel(const DzArgs p) {
    constexpr bool kBeside = kForm == kDzBeside;
    __shared__ float red[kBeside ? 1 : kDzWarps][kBeside ? 1 : 256];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n = blockIdx.x * 256 + 8 * lane;
    const long long r0 = (long long)blockIdx.y * p.per, r1 = r0 + p.per < p.rows ? r0 + p.per : p.rows;
    float sum[8] = {};
    if (n < p.N) {
        constexpr int kAhead = kAct == MOE_ACT_NONE ? 8 : 2;  // rows whose loads are in flight together
        for (long long r = r0 + warp; r < r1; r += kDzWarps * kAhead) {
            uint4 dy[kAhead];
            float4 z[kAhead][2];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const long long at = r + u * kDzWarps;
                if (at >= r1) break;
                dy[u] = __ldg(reinterpret_cast<const uint4*>(p.dy + at * p.dy_stride + n));
                if constexpr (kAct != MOE_ACT_NONE) {
                    const float4* zp = reinterpret_cast<const float4*>(p.z + (size_t)at * p.N + n);
                    z[u][0] = __ldg(zp), z[u][1] = __ldg(zp + 1);
                }
            }
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const long long at = r + u * kDzWarps;
                if (at >= r1) break;
                float d[8];
                unpack_bf16x8(dy[u], d);
                if constexpr (kAct != MOE_ACT_NONE) {
                    const float v[8] = {z[u][0].x, z[u][0].y, z[u][0].z, z[u][0].w, z[u][1].x, z[u][1].y, z[u][1].z, z[u][1].w};
#pragma unroll
                    for (int j = 0; j < 8; ++j) d[j] *= act_slope<kAct>(v[j]);
                    *reinterpret_cast<uint4*>(p.dz + (size_t)at * p.N + n) = pack8(d);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) sum[j] += d[j];
            }
        }
    }
    if constexpr (kBeside) {
        if (n < p.N) {
            float4* d = reinterpret_cast<float4*>(p.part + ((size_t)blockIdx.y * kDzWarps + warp) * p.N + n);
            d[0] = make_float4(sum[0], sum[1], sum[2], sum[3]);
            d[1] = make_float4(sum[4], sum[5], sum[6], sum[7]);
        }
        asm volatile("griddepcontrol.wait;" ::: "memory");  // what comes after this kernel comes after the products too
        return;
    }
    if (!p.part && !p.db) return;
#pragma unroll
    for (int j = 0; j < 8; ++j) red[warp][8 * lane + j] = sum[j];
    __syncthreads();
    const int c = blockIdx.x * 256 + threadIdx.x;
    if constexpr (kForm == kDzCluster) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < kDzWarps; ++w) v += red[w][threadIdx.x];
        red[0][threadIdx.x] = v;  // (its one reader)
        __syncthreads();
        cluster_sync();
        if (threadIdx.x % gridDim.y == blockIdx.y && c < p.N) {
            v = 0.0f;
            for (uint32_t b = 0; b < gridDim.y; ++b) {
                float u;
                asm volatile("ld.shared::cluster.f32 %0, [%1];"
                             : "=f"(u)
                             : "r"(cluster_addr_of(smem_addr(&red[0][threadIdx.x]), b))
                             : "memory");
                v += u;
            }
            store_db(p.db, p.db_f32, c, v);
        }
        __syncthreads();
        cluster_sync();  // no block's memory goes while another reads it
        return;
    }
    if (c >= p.N) return;
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kDzWarps; ++w) v += red[w][threadIdx.x];
    if (gridDim.y == 1)
        store_db(p.db, p.db_f32, c, v);
    else
        p.part[(size_t)blockIdx.y * p.N + c] = v;
}

// db from the blocks' sums, in order.  32 columns a block, a warp every 32nd of them.
constexpr int kDbWarps = 32;
__global__ void __launch_bounds__(32 * kDbWarps) linear_db_kernel(const float* part, int parts, int N, void* db, int db_f32) {
    __shared__ float red[kDbWarps][33];
    asm volatile("griddepcontrol.launch_dependents;\n\tgriddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31, c = blockIdx.x * 32 + lane, w = threadIdx.x >> 5;
    float v = 0.0f;
    for (int i = w; i < parts; i += 4 * kDbWarps) {  // four loads in flight: their latency is what this takes
        float u[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) u[k] = i + k * kDbWarps < parts && c < N ? part[(size_t)(i + k * kDbWarps) * N + c] : 0.0f;
        v += (u[0] + u[1]) + (u[2] + u[3]);
    }
    red[w][lane] = v;
    __syncthreads();
    if (w || c >= N) return;
    float t[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < kDbWarps; ++i) t[i & 3] += red[i][lane];
    store_db(db, db_f32, c, (t[0] + t[1]) + (t[2] + t[3]));
}

// Rows of blocks of linear_dz_kernel, 32 rows each at least: as many as run at once.
int dz_parts(long long T, int N) {
    const long long cols = cdiv(N, 256), want = kDzBlocks * 152 / cols, most = (T + 31) / 32;
    const long long n = want < most ? want : most;
    return (int)(n < 1 ? 1 : n);
}
// Up to 256 rows a cluster adds up db: no second kernel, no sums in memory (100 x 2048 x
// 512 backward 8.0 -> 7.5 us, and some 3 us of the host's).  Blocks: a power of two, the last ones may have no row.
bool dz_cluster(long long T, int N) { return T <= 256 && dz_parts(T, N) > 1; }
int dz_cluster_blocks(int parts) { return parts <= 2 ? 2 : parts <= 4 ? 4 : 8; }
// Beside the products: one block for an SM at most (the next one would wait for
// their end), of 64 rows at least; 0: not in that form.  4096 x 2048 x 7168 145.1 us with the
// sums before the products, 133.7 beside them, 137.6 with 128 rows a block; small products
// lose up to 2.3 us (4096 x 512 x 512 23.3 and 25.6).
int beside_parts(long long T, int N) {
    const long long cols = cdiv(N, 256), most = T / 64;
    const long long n = 152 / cols < most ? 152 / cols : most;
    return (int)n;
}

// Launches a kernel that starts while the one before it (of the same call) ends.
template <typename K, typename... A>
int launch_after(K kernel, dim3 grid, int threads, const char* name, cudaStream_t st, A... args) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    trace_pre(st);
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    trace_post(st, name);
    return (int)(e != cudaSuccess ? e : cudaGetLastError());
}

int launch_linear_join(const float* part, long long rows, int N, int splits, const LinearEpi& epi, void* out,
                       cudaStream_t st) {
    const long long blocks = (rows * (N / 8) + 127) / 128;
    return launch_after(linear_join_kernel, dim3((unsigned)(blocks < 2432 ? blocks : 2432)), 128, "linear_join", st, part, rows, N,
                        splits, epi, static_cast<__nv_bfloat16*>(out));
}

template <int EPI>
int launch_linear_pair(const LinearArgs& a, const CUtensorMap (&m)[5], cudaStream_t st) {
    static std::atomic<int> fits[kMaxDevices] = {};
    return launch_pairs(linear_pair_kernel<EPI>, fits, dense_smem<EPI>(), (long long)a.d.tiles_m * a.d.tiles_n, true,
                        "linear", st, m[0], m[1], m[2], m[3], m[4], a);
}

// The form for few rows: jobs of eight rows, or of sixteen (from nine on, where the matrix is
// large).  us a forward with the weights from DRAM, eight a job | sixteen | tiles on SM
// pairs, K x N: 2048 x 7168, 12 rows 14.9 | 9.6 | 17.4, 32 rows 24.6 | 15.7 | 14.3; 7168 x 2048, 16 rows
// 9.0 | 8.8 | 14.9, 48 rows 45.2 | 15.9 | 16.9; 1024 x 1024, 64 rows 5.0 | 5.7 | 9.9; 4096 x 8192, 16 rows
// 26.7 | 15.2 | 18.3, 17 rows 49.4 | 26.2 | 18.4.  The bounds are the feed-forward block's and not the
// best everywhere: 2048 x 2816, 9 to 24 rows 6.3-6.7 | 6.9-8.5 (taken) | 12; 7168 x 2048, 96 rows 25.1
// (taken) | 16.4; 512 x 512, 160 rows 4.5 | 5.5 | 8.3 (taken).
bool linear_two(const moe_linear_shape& s) { return s.T > 8 && (long long)s.K * s.N > (1 << 20); }
bool linear_few(const moe_linear_shape& s) {
    const int per = linear_two(s) ? 16 : 8;
    return s.T <= 16 || (s.T <= 128 && (long long)((s.T + per - 1) / per) * ((s.N + 63) / 64) <= 200);
}
Product linear_product(const moe_linear_shape& s) { return {s.T, s.N, s.K, false}; }

// The gradients' products.  Together in one launch they have one range of K; one that is
// deep and has few tiles (dW of many rows and a narrow layer, dx of a wide one) leaves most
// pairs without work and is better by itself, its K split and joined (10000 x 64 x 72 silu
// backward 48.6 -> 27.9 us, 8192 x 2048 x 64 52.5 -> 27.9, 130 x 64 x 7168 32.4 -> 23.7).
Product dw_product(const moe_linear_shape& s) { return {s.K, s.N, s.T, false}; }
Product dx_product(const moe_linear_shape& s) { return {s.T, s.K, s.N, false}; }
// In clocks of a pair, with dense_shape's figures and 8000 for each launch of several.
// Together | alone, T x K x N: 130 x 64 x 4096 18.3 | 18.3 us, 8192 x 512 x 64 36.4 | 18.1, 2048 x 512 x 64
// 12.0 | 13.7 (together).  Near the border it errs to the side of together: 4096 x 2048 x 64 22.3 |
// 17.2, 8192 x 1024 x 1024 50.4 | 35.6.
long long alone_clocks(const Product& q) {
    const Shape f = q.shape();
    const long long tiles = (long long)cdiv(q.M, 256) * cdiv(q.N, f.width), kb = cdiv(q.K, 64);
    const long long rounds = (tiles * f.splits + kDenseClusters - 1) / kDenseClusters;
    return rounds * cdiv(kb, f.splits) * (f.width + 256) + 3000 +
           (f.splits > 1 ? 7000 + (long long)q.M * q.N * f.splits * 8 / 2000 : 0);
}
long long together_clocks(const Product* q, int n) {  // of the busiest pair, at least
    long long sum = 0, most = 0;
    for (int i = 0; i < n; ++i) {
        const long long item = (long long)cdiv(q[i].K, 64) * 512 + 3000;
        sum += item * cdiv(q[i].M, 256) * cdiv(q[i].N, 256);
        most = item > most ? item : most;
    }
    sum /= kDenseClusters;
    return sum > most ? sum : most;
}
// Which of n <= 2 products get a launch of their own (a bit each).
int split_alone(const Product* q, int n) {
    int best = 0;
    long long cost = n ? together_clocks(q, n) : 0;
    for (int alone = 1; alone < 1 << n; ++alone) {
        Product rest[2];
        int left = 0;
        long long c = 0;
        bool ok = true;
        for (int i = 0; i < n; ++i) {
            if (alone >> i & 1) {
                ok = ok && q[i].shape().splits > 1;
                c += alone_clocks(q[i]) + 8000;
            } else {
                rest[left++] = q[i];
            }
        }
        if (left) c += together_clocks(rest, left) + 8000;
        if (ok && c < cost) {
            cost = c;
            best = alone;
        }
    }
    return best;
}

}  // namespace

LinearSizes linear_sizes(const moe_linear_shape& s) {
    LinearSizes z = {0, 0, 0, 0};
    if (s.T == 0) return z;
    // of those that some set of wanted gradients splits
    const Product both[2] = {dw_product(s), dx_product(s)};
    const int mask = split_alone(both, 2) | split_alone(both, 1) | split_alone(both + 1, 1) << 1;
    for (int i = 0; i < 2; ++i)
        if (mask >> i & 1) z.grads = both[i].part_bytes() > z.grads ? both[i].part_bytes() : z.grads;
    z.part = linear_few(s) ? 0 : linear_product(s).part_bytes();
    z.dz = s.activation == MOE_ACT_NONE ? 0 : (long long)s.T * s.N * 2;
    const int parts = dz_parts(s.T, s.N);
    const int beside = s.activation == MOE_ACT_NONE ? beside_parts(s.T, s.N) * kDzWarps : 0;
    if (dz_cluster(s.T, s.N)) return z;
    z.sums = parts > 1 || beside ? (long long)(parts > beside ? parts : beside) * s.N * 4 : 0;
    return z;
}

int launch_linear_forward(const moe_linear_shape& s, const LinearPtrs& f, cudaStream_t st) {
    int rc, e;
    const LinearEpi epi = {s.activation, f.bias_f32, f.bias, static_cast<const __nv_bfloat16*>(f.residual), f.res_stride, f.z};
    if (linear_few(s)) {
        const bool two = linear_two(s);
        CUtensorMap w, x;
        if ((rc = abi_map_2d(&w, f.W, 2, s.K, s.N, s.N, 64, 32, "W"))) return rc;
        if ((rc = abi_map_2d(&x, f.x, 2, s.T, s.K, f.x_stride, 32, two ? 16 : 8, "x"))) return rc;
        const FewArgs a = {s.T, s.K, s.N, 0, 0, INFINITY, static_cast<__nv_bfloat16*>(f.y), nullptr, f.status, epi,
                           selftest_gave_up()};
        e = two ? launch_few<FEW_LINEAR, 2>(a, w, x, false, "linear_few", st)
                : launch_few<FEW_LINEAR, 1>(a, w, x, false, "linear_few", st);
        return e ? abi_cuda_fail(e, "linear launch") : MOE_OK;
    }
    const Product q = linear_product(s);
    LinearArgs a = {q.args(INFINITY, f.status), epi, static_cast<__nv_bfloat16*>(f.y)};
    a.d.part = f.part;
    a.d.gave_up = selftest_gave_up();
    CUtensorMap m[5] = {};  // x, W, y, residual, z
    if ((rc = abi_map_2d(&m[0], f.x, 2, s.T, s.K, f.x_stride, 64, 128, "x"))) return rc;
    if ((rc = map_op(&m[1], f.W, s.K, s.N, 64, "W"))) return rc;
    if (a.d.splits > 1) {
        DenseMaps d = {m[0], m[1], {}, {}};
        if ((rc = abi_map_nd(&d.c0, f.part, 4, {s.N, 1, s.T, a.d.splits}, {32, 1, 32, 1}, "partial sums"))) return rc;
        e = launch_dense<KN, EPI_PART>(a.d, d, "linear", st, true);
        if (!e) e = launch_linear_join(f.part, s.T, s.N, a.d.splits, epi, f.y, st);
        return e ? abi_cuda_fail(e, "linear launch") : MOE_OK;
    }
    if ((rc = map_op(&m[2], f.y, s.T, s.N, 32, "y (store)"))) return rc;
    if (f.residual && (rc = abi_map_2d(&m[3], f.residual, 2, s.T, s.N, f.res_stride, 64, 32, "residual"))) return rc;
    if (f.z && (rc = abi_map_2d(&m[4], f.z, 4, s.T, s.N, s.N, 32, 32, "z (store)"))) return rc;
    e = f.residual ? (f.z ? launch_linear_pair<EPI_LIN_RZ>(a, m, st) : launch_linear_pair<EPI_LIN_R>(a, m, st))
                   : (f.z ? launch_linear_pair<EPI_LIN_Z>(a, m, st) : launch_linear_pair<EPI_LIN>(a, m, st));
    return e ? abi_cuda_fail(e, "linear launch") : MOE_OK;
}

int launch_linear_backward(const moe_linear_shape& s, const LinearPtrs& f, cudaStream_t st) {
    int rc, e = 0;
    const void* dz = f.dy;
    long long dz_stride = f.dy_stride;
    const int parts = dz_parts(s.T, s.N);
    const bool grads = f.dx || f.dW, act = s.activation != MOE_ACT_NONE;
    const bool cluster = f.db && dz_cluster(s.T, s.N);
    // dW = x^T dz, dx = dz W^T
    Product wanted[2];
    int n_wanted = 0;
    if (f.dW) wanted[n_wanted++] = dw_product(s);
    if (f.dx) wanted[n_wanted++] = dx_product(s);
    const int alone = split_alone(wanted, n_wanted);
    const int beside = f.db && grads && !act && !cluster && !alone ? beside_parts(s.T, s.N) : 0;
    auto join_db = [&](int n) {
        return launch_after(linear_db_kernel, dim3(cdiv(s.N, 32)), 32 * kDbWarps, "linear_db", st,
                            static_cast<const float*>(f.sums), n, s.N, f.db, f.db_f32);
    };
    DzArgs da = {static_cast<const __nv_bfloat16*>(f.dy), f.dy_stride, s.T, s.N, (s.T + parts - 1) / parts, f.z,
                 static_cast<__nv_bfloat16*>(f.dz), f.db && parts > 1 && !cluster ? f.sums : nullptr,
                 parts > 1 && !cluster ? nullptr : f.db, f.db_f32};
    const dim3 dz_grid(cdiv(s.N, 256), cluster ? dz_cluster_blocks(parts) : parts);
    auto launch_dz = [&](auto plain_form, auto cluster_form) {
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = attr[0].val.clusterDim.z = 1;
        attr[0].val.clusterDim.y = dz_grid.y;
        cfg.gridDim = dz_grid;
        cfg.blockDim = dim3(32 * kDzWarps);
        cfg.stream = st;
        cfg.attrs = attr;
        cfg.numAttrs = cluster ? 1 : 0;
        trace_pre(st);
        const cudaError_t ce = cudaLaunchKernelEx(&cfg, cluster ? cluster_form : plain_form, da);
        trace_post(st, "linear_dz");
        return (int)(ce != cudaSuccess ? ce : cudaGetLastError());
    };
    if (act) {
        switch (s.activation) {
            case MOE_ACT_SILU:
                e = launch_dz(linear_dz_kernel<MOE_ACT_SILU, kDzPlain>, linear_dz_kernel<MOE_ACT_SILU, kDzCluster>);
                break;
            case MOE_ACT_GELU:
                e = launch_dz(linear_dz_kernel<MOE_ACT_GELU, kDzPlain>, linear_dz_kernel<MOE_ACT_GELU, kDzCluster>);
                break;
            default:
                e = launch_dz(linear_dz_kernel<MOE_ACT_GELU_TANH, kDzPlain>, linear_dz_kernel<MOE_ACT_GELU_TANH, kDzCluster>);
                break;
        }
        if (e) return abi_cuda_fail(e, "linear dz launch");
        dz = f.dz, dz_stride = s.N;
        if (da.part && (e = join_db(parts))) return abi_cuda_fail(e, "linear bias gradient launch");
    } else if (f.db && !beside) {
        e = launch_dz(linear_dz_kernel<MOE_ACT_NONE, kDzPlain>, linear_dz_kernel<MOE_ACT_NONE, kDzCluster>);
        if (e) return abi_cuda_fail(e, "linear column sums launch");
        if (da.part && (e = join_db(parts))) return abi_cuda_fail(e, "linear bias gradient launch");
    }
    if (!grads) return MOE_OK;
    // the deeper product first
    struct {
        Product q;
        bool mn;  // both operands lie along the output
        const void *A, *B;
        void* D;
        long long a_stride, b_stride;
    } job[2] = {{dw_product(s), true, f.x, dz, f.dW, f.x_stride, dz_stride},
                {dx_product(s), false, dz, f.W, f.dx, dz_stride, s.N}};
    bool first = !act && !f.db;  // of the call's kernels
    if (alone) {
        int bit = 1;
        for (auto& j : job) {
            if (!j.D) continue;
            const bool by_itself = alone & bit;
            bit <<= 1;
            if (!by_itself) continue;
            DenseArgs a = j.q.args(INFINITY, f.status);
            a.part = f.part;
            a.gave_up = selftest_gave_up();
            DenseMaps m = {};
            if ((rc = j.mn ? abi_map_2d(&m.a, j.A, 2, j.q.K, j.q.M, j.a_stride, 64, 64, "A (MN-major)")
                           : abi_map_2d(&m.a, j.A, 2, j.q.M, j.q.K, j.a_stride, 64, 128, "A")))
                return rc;
            if ((rc = j.mn ? abi_map_2d(&m.b, j.B, 2, j.q.K, j.q.N, j.b_stride, 64, 64, "B (MN-major)")
                           : abi_map_2d(&m.b, j.B, 2, j.q.N, j.q.K, j.b_stride, 64, a.width / 2, "B")))
                return rc;
            if ((rc = abi_map_nd(&m.c0, f.part, 4, {j.q.N, 1, j.q.M, a.splits}, {32, 1, 32, 1}, "partial sums"))) return rc;
            e = j.mn ? launch_dense<NN, EPI_PART>(a, m, "linear_dw", st, first)
                     : launch_dense<KK, EPI_PART>(a, m, "linear_dx", st, first);
            if (!e) e = launch_linear_join(f.part, j.q.M, j.q.N, a.splits, {}, j.D, st);
            if (e) return abi_cuda_fail(e, "linear gradient launch");
            first = false;
            j.D = nullptr;
        }
        if (!job[0].D && !job[1].D) return MOE_OK;
    }
    if (s.N > s.T) {
        const auto t = job[0];
        job[0] = job[1];
        job[1] = t;
    }
    Product qs[2];
    int n = 0;
    for (const auto& j : job)
        if (j.D) qs[n++] = j.q;
    const int width = joint_width(qs, n);
    PlainMaps m = {};
    PlainArgs a = {};
    a.n = n;
    a.status = f.status;
    a.gave_up = selftest_gave_up();
    int i = 0;
    for (const auto& j : job) {
        if (!j.D) continue;
        a.p[i] = plain(j.q, width, j.mn, j.mn, j.D);
        if ((rc = j.mn ? abi_map_2d(&m.m[3 * i], j.A, 2, j.q.K, j.q.M, j.a_stride, 64, 64, "A (MN-major)")
                       : abi_map_2d(&m.m[3 * i], j.A, 2, j.q.M, j.q.K, j.a_stride, 64, 128, "A")))
            return rc;
        if ((rc = j.mn ? abi_map_2d(&m.m[3 * i + 1], j.B, 2, j.q.K, j.q.N, j.b_stride, 64, 64, "B (MN-major)")
                       : abi_map_2d(&m.m[3 * i + 1], j.B, 2, j.q.N, j.q.K, j.b_stride, 64, width / 2, "B")))
            return rc;
        if ((rc = map_op(&m.m[3 * i + 2], j.D, j.q.M, j.q.N, 32, "gradient (store)"))) return rc;
        ++i;
    }
    // Without an activation the products start after all earlier work and the column
    // sums of dy run beside them, in what they leave of an SM (8192 x 2048 x 7168: 290
    // -> 268 us): dy is there before either starts.
    e = launch_plain(a, m, "linear_grads", st, first || beside > 0);
    if (!e && beside) {
        da.per = (s.T + beside - 1) / beside;
        da.part = f.sums;
        e = launch_after(linear_dz_kernel<MOE_ACT_NONE, kDzBeside>, dim3(dz_grid.x, beside), 32 * kDzWarps, "linear_dz", st, da);
        if (!e) e = join_db(beside * kDzWarps);
    }
    return e ? abi_cuda_fail(e, "linear gradient launch") : MOE_OK;
}

}  // namespace moe
