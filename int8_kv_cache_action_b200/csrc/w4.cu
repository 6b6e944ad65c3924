// Linear layer with 4-bit weights and group scales (definition in nomas.h).
//
// Kernels:
//   w4_quantize_kernel  one warp per (row, group)
//   w4_dequant_kernel   bf16(code * scale), bound by the weights it writes
//   w4_rows_kernel      y = x W^T for few rows of x, every code read once for 32 of them: bound by the codes'
//                       bytes and by widening them, about 20 instructions a word of 8.  The weights are widened in
//                       registers and go straight into the register form of the tensor-core product (m16n8k16,
//                       16 rows of W by 8 rows of x): one instruction per 8 weights of a lane, where fp32
//                       products would need one per weight and row of x.  tcgen05 would want the widened weights
//                       in shared memory first; for more rows of x others take over:
//   w4_tile_kernel      the same by tcgen05, the weights widened into TMEM
//   w4_dequant_kernel and nomas_linear_bf16, above 64 or 128 rows
#include <atomic>

#include "common.cuh"

namespace nomas {

// 8 codes (one word, code i in bits 4i .. 4i + 3) times a scale, as bf16 pairs (i, i + 4), i = 0 .. 3: with
// u = code + 8 in the low bits of the mantissa of 128 (0x4300, whose last place is 1) the bf16 is 128 + u, the
// code comes out of - 136 exactly, and the product with the scale is the one rounding.
__device__ __forceinline__ void w4_widen(uint32_t word, __nv_bfloat162 scale, uint32_t (&out)[4]) {
    const __nv_bfloat162 minus136 = __floats2bfloat162_rn(-136.0f, -136.0f);
    uint32_t mask = 0x000F000Fu, base = 0x43004300u;
    asm("" : "+r"(mask), "+r"(base));          // registers: an instruction holds one immediate
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t u;                            // (word >> 4 i & mask) | base in one instruction behind the shift
        asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(u) : "r"(word >> (4 * i)), "r"(mask), "r"(base));
        const __nv_bfloat162 w = __hmul2(__hadd2(*reinterpret_cast<const __nv_bfloat162 *>(&u), minus136), scale);
        out[i] = *reinterpret_cast<const uint32_t *>(&w);
    }
}

// D += A B: A 16 x 16 (rows of W), B 16 x 8 (rows of x), bf16 operands, fp32 sums.
__device__ __forceinline__ void mma_16x8x16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                            uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same with D = A B.
__device__ __forceinline__ void mma_16x8x16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                  uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

struct W4Params {
    const uint8_t *codes;
    const __nv_bfloat16 *scales;
    const __nv_bfloat16 *x;
    void *y;
    int64_t ldx, ldy;
    int64_t n;                                 // rows of W
    int32_t m, k, groups, group_log2, y_bf16;
};

__device__ __forceinline__ uint4 load_stream(const void *p) {
    uint4 v;
    asm("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

// A CTA: 16 RT rows of W, its warps chunks of 128 columns in turn.  In a chunk, lane 4 g + t holds columns 32 t ..
// 32 t + 31 of rows g and g + 8 of each 16 (16 bytes of codes a row; the 32 columns have one scale) and of row g of
// each 8 rows of x.  Which column of the chunk stands for which index of a product's inner dimension is free as long
// as both operands agree: a product takes 2 pairs of every lane's word.  The codes of the next chunk are on their way
// while a chunk is multiplied.
template <int RT>
struct W4Codes {
    uint4 w[RT][2];
    __nv_bfloat16 f[RT][2];
};

// CTAs of an SM, from the warps that the sums of RT * NT products leave registers for.  24 warps spill 52 to 116 bytes a
// thread with RT = 2, and pay on wide matrices (2 x 8192 -> 28001: 35.6 us, 43.9 with 20, 45.3 with 16).  The 16 warps of
// more rows of x spill too: 32 and 40 bytes with <2, 2>, 268 and 276 with <4, 2> (30 x 2048 -> 12288, 13.5 us where its
// bytes take 2.2), 8 to 32 with <4, 1>.
template <int NT, int RT, int WARPS>
constexpr int w4_ctas = (NT * RT <= 2 ? 24 : 16) / WARPS > 0 ? (NT * RT <= 2 ? 24 : 16) / WARPS : 1;

template <int NT, int RT, int WARPS>
__global__ void __launch_bounds__(32 * WARPS, w4_ctas<NT, RT, WARPS>) w4_rows_kernel(const W4Params p) {
    extern __shared__ float red[];             // [WARPS][8 NT][16 RT + 1]
    constexpr int LD = 16 * RT + 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int64_t n0 = (int64_t)blockIdx.x * (16 * RT);
    const int m0 = blockIdx.y * 8 * NT, m = min(p.m - m0, 8 * NT);      // rows of x
    const int chunks = p.k >> 7, tail = p.k & 127;
    // this CTA's rows: 32-bit offsets from the first; rows past the end repeat the last one, and their products go
    // nowhere
    const uint8_t *const codes = p.codes + n0 * (p.k / 2), *const scales = reinterpret_cast<const uint8_t *>(p.scales + n0 * p.groups);
    const uint32_t last = (uint32_t)min((int64_t)(16 * RT), p.n - n0) - 1;
    uint32_t code_at[RT][2], scale_at[RT][2];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t row = min((uint32_t)(16 * r + 8 * h + g), last);
            code_at[r][h] = row * (p.k / 2) + 16 * t;
            scale_at[r][h] = row * 2 * p.groups;
        }
    const __nv_bfloat16 *xr[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) xr[i] = p.x + (int64_t)(m0 + min(8 * i + g, m - 1)) * p.ldx + 32 * t;
    float acc[RT][NT][4];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[r][i][j] = 0.0f;

    auto load = [&](W4Codes<RT> &v, int c) {   // chunk c: columns 128 c ..
        const uint32_t group = (uint32_t)(c * 128 + 32 * t) >> p.group_log2;
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                v.w[r][h] = load_stream(codes + (code_at[r][h] + c * 64));
                v.f[r][h] = *reinterpret_cast<const __nv_bfloat16 *>(scales + (scale_at[r][h] + 2 * group));
            }
    };
    auto multiply = [&](const W4Codes<RT> &v, int c, bool in) {
        // the tensor cores truncate sums: short runs of columns are added up in rounded fp32, a whole chunk where its
        // sums fit the registers, else 32 columns
        constexpr bool WHOLE = RT * NT <= 2;
        float part[RT][NT][4];
        __nv_bfloat162 s[RT][2];
#pragma unroll
        for (int r = 0; r < RT; ++r) {
#pragma unroll
            for (int h = 0; h < 2; ++h) s[r][h] = __halves2bfloat162(v.f[r][h], v.f[r][h]);
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            uint32_t u[RT][2][4];
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint4 w = v.w[r][h];
                    w4_widen(q == 0 ? w.x : q == 1 ? w.y : q == 2 ? w.z : w.w, s[r][h], u[r][h]);
                }
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                uint4 xv = make_uint4(0, 0, 0, 0);
                if (in) xv = __ldg(reinterpret_cast<const uint4 *>(xr[i] + c * 128 + 8 * q));
                // pairs (0,4) (1,5) (2,6) (3,7) of 8 columns
                const uint32_t x0 = __byte_perm(xv.x, xv.z, 0x5410), x1 = __byte_perm(xv.x, xv.z, 0x7632);
                const uint32_t x2 = __byte_perm(xv.y, xv.w, 0x5410), x3 = __byte_perm(xv.y, xv.w, 0x7632);
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    if (q == 0 || !WHOLE)
                        mma_16x8x16_first(part[r][i], u[r][0][0], u[r][1][0], u[r][0][1], u[r][1][1], x0, x1);
                    else
                        mma_16x8x16(part[r][i], u[r][0][0], u[r][1][0], u[r][0][1], u[r][1][1], x0, x1);
                    mma_16x8x16(part[r][i], u[r][0][2], u[r][1][2], u[r][0][3], u[r][1][3], x2, x3);
                    if (q == 3 || !WHOLE) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) acc[r][i][j] += part[r][i][j];
                    }
                }
            }
        }
    };

    W4Codes<RT> now, next;
    if (warp < chunks) load(now, warp);
    for (int c = warp; c < chunks; c += 2 * WARPS) {
        if (c + WARPS < chunks) load(next, c + WARPS);
        multiply(now, c, true);
        if (c + WARPS >= chunks) break;
        if (c + 2 * WARPS < chunks) load(now, c + 2 * WARPS);
        multiply(next, c + WARPS, true);
    }
    // the last 32, 64 or 96 columns: lanes past them hold zeros
    if (tail && warp == chunks % WARPS) {
        const bool in = 32 * t < tail;
        if (in) {
            load(now, chunks);
        } else {
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int h = 0; h < 2; ++h) now.w[r][h] = make_uint4(0, 0, 0, 0), now.f[r][h] = __float2bfloat16_rn(0.0f);
        }
        multiply(now, chunks, in);
    }

    // acc: rows g and g + 8 of W, rows 8 i + 2 t and 8 i + 2 t + 1 of x
    float *mine = red + warp * 8 * NT * LD;
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) mine[(8 * i + 2 * t + (j & 1)) * LD + 16 * r + 8 * (j >> 1) + g] = acc[r][i][j];
    __syncthreads();
    for (int e = threadIdx.x; e < m * 16 * RT; e += 32 * WARPS) {
        const int row = e / (16 * RT), col = e % (16 * RT);
        if (n0 + col >= p.n) continue;
        float s = red[row * LD + col];
#pragma unroll
        for (int w = 1; w < WARPS; ++w) s += red[(w * 8 * NT + row) * LD + col];
        if (p.y_bf16)
            static_cast<__nv_bfloat16 *>(p.y)[(int64_t)(m0 + row) * p.ldy + n0 + col] = __float2bfloat16_rn(s);
        else
            static_cast<float *>(p.y)[(int64_t)(m0 + row) * p.ldy + n0 + col] = s;
    }
}

// ------------------------------------------------------------------------------------------------
// few rows of x by tcgen05
// ------------------------------------------------------------------------------------------------
// A CTA: 128 rows of W by a share of the columns, in slabs of 256 whose codes TMA brings some slabs ahead (rows are far
// apart: loaded by thread, one row each, a slab took 2 us); the CTAs of a cluster share the columns of the same rows.
// Eight warps widen: a thread takes 64 columns of its row per half slab and writes them straight to TMEM, where
// tcgen05.mma takes its A operand (a row a lane, two columns of W a 32-bit column), so the widened weights never pass
// through shared memory; x is the B operand, K-major with the 128-byte swizzle, its columns in the order in which words
// widen.  A ninth warp issues copies and products (issued by a widening warp, that warp held up the others: 1850 cycles
// a half slab instead of 700).  The tensor core truncates its sums, so the sums of every 512 columns leave TMEM for fp32
// additions in registers.  Two buffers of A and x, and two CTAs an SM, hide each other's waits.  At the end the CTAs of
// a cluster add their sums up through distributed shared memory, in rank order.
// A slab takes as long whatever the rows of x (8192 -> 28001: 2 rows 75 us, 16 rows 78, against 34 and 54 by
// w4_rows_kernel), so it pays from about 17 of them on.  64 x 8192 -> 8192: 33 us, where its bytes take 5.8.  No unit is
// near its limit there (tensor pipe 13 % busy, DRAM 12 %, half the issue slots): what is left is most likely the latency
// of a half slab's chain, from x to the product's commit, which two buffers and two CTAs an SM hide in part.
constexpr int kTileRows = 128, kSlab = 256, kTileThreads = 256;        // threads that widen; one more warp issues
constexpr uint32_t kTileTmem = 256, kTileD = 128;      // TMEM columns of a CTA: A at 0, D at kTileD
constexpr int kTileStage = kTileRows * kSlab / 2;
// Scales of kScaleSlabs slabs wait in shared memory, a row's at a pitch of an odd number of 4-byte banks.
constexpr int kScaleSlabs = 8, kScalePitch = kScaleSlabs * kSlab / 32 + 2;

struct W4Tile {
    W4Params p;
    int32_t slabs, share;                      // slabs of K, of a CTA
    int *err;
    uint64_t timeout_ns;
};

// 16 columns of this thread's lane.
__device__ __forceinline__ void tmem_ld16f_sync(uint32_t addr, float (&r)[16]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
                 "tcgen05.wait::ld.sync.aligned;"
                 : NOMAS_F8(0), NOMAS_F8(8)
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void w4_cluster_sync() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t w4_cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t w4_cluster_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ float w4_load_of(uint32_t shared_addr, uint32_t rank) {
    uint32_t at;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(shared_addr), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
    return v;
}

__device__ __forceinline__ void w4_store(const W4Params &p, int64_t row, int64_t col, float v) {
    if (p.y_bf16)
        static_cast<__nv_bfloat16 *>(p.y)[row * p.ldy + col] = __float2bfloat16_rn(v);
    else
        static_cast<float *>(p.y)[row * p.ldy + col] = v;
}

// NX: rows of x of a CTA, 32 or 64 (the product's N).
template <int NX>
struct TileSmem {
    static constexpr int kStages = NX == 64 ? 3 : 4;           // two CTAs fit an SM
    static constexpr int kX = NX * kSlab * 2;                  // a slab of x, later the CTA's sums
    static constexpr int kScales = kTileRows * kScalePitch * 2;
    static constexpr int kBytes = kStages * kTileStage + kX + kScales + 1024;      // slack for 1024-byte alignment
};

template <int NX>
__global__ void __launch_bounds__(kTileThreads + 32, 2) w4_tile_kernel(const __grid_constant__ CUtensorMap codes, const W4Tile a) {
    constexpr int XBLOCK = NX * 128, XHALF = 2 * XBLOCK;       // 64 columns of x, half a slab of it
    constexpr int XC = NX * 16 / kTileThreads;                 // 16-byte chunks of half a slab of x a thread
    constexpr int NC = NX / 2, STAGES = TileSmem<NX>::kStages; // columns of D a thread reads
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t done[2], ready[2], full[STAGES];
    __shared__ uint32_t tmem_at;
    __shared__ int abort_flag;
    const W4Params &p = a.p;
    uint8_t *const sw = smem_raw + ((0u - smem_u32(smem_raw)) & 1023u), *const sx = sw + STAGES * kTileStage;
    __nv_bfloat16 *const ss = reinterpret_cast<__nv_bfloat16 *>(sx + TileSmem<NX>::kX);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, part_of = warp >> 2 & 1;
    const uint32_t ranks = w4_cluster_size(), rank = w4_cluster_rank();
    const int64_t n0 = (int64_t)(blockIdx.x / ranks) * kTileRows;
    const int m0 = blockIdx.y * NX, m = min(p.m - m0, NX);
    const int first = rank * a.share, last = min(first + a.share, a.slabs);
    const int row_in = (warp & 3) * 32 + lane;                 // this thread's row of W, and lane of TMEM

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&done[i], 1);
            mbar_init(&ready[i], kTileThreads / 32);
        }
        for (int i = 0; i < STAGES; ++i) mbar_init(&full[i], 1);
        abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 0) {
        __syncwarp();
        tmem_alloc(&tmem_at, kTileTmem);
        tmem_relinquish();
    }
    auto fetch = [&](int slab) {               // one thread
        const int s = (slab - first) % STAGES;
        mbar_arrive_expect_tx(&full[s], kTileStage);
        tma_load_3d(sw + s * kTileStage, &codes, &full[s], slab * (kSlab / 2), (int)n0, 0);
    };
    // x: chunk e of half a slab is columns 8 (e & 15) .. of row e >> 4
    auto load_x = [&](uint4 (&v)[XC], int at) {
#pragma unroll
        for (int i = 0; i < XC; ++i) {
            const int e = tid + i * kTileThreads, xr = e >> 4, col = at + (e & 15) * 8;
            v[i] = make_uint4(0, 0, 0, 0);
            if (xr < m && at < last * kSlab && col < p.k)
                v[i] = __ldg(reinterpret_cast<const uint4 *>(p.x + (int64_t)(m0 + xr) * p.ldx + col));
        }
    };
    // scales of the slabs from `slab` on; zeros past the last group
    auto load_scales = [&](int slab) {
        constexpr int U = 8;                   // loads in flight
        const int left = last - slab, g0 = slab * kSlab >> p.group_log2;
        const int per_log2 = 8 + (left > 4 ? 3 : left > 2 ? 2 : left > 1 ? 1 : 0) - p.group_log2;
        for (int e0 = tid; e0 < kTileRows << per_log2; e0 += U * kTileThreads) {
            __nv_bfloat16 f[U];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int e = e0 + i * kTileThreads, r = e >> per_log2, g = g0 + (e & ((1 << per_log2) - 1));
                f[i] = __float2bfloat16_rn(0.0f);
                if (r < kTileRows && n0 + r < p.n && g < p.groups) f[i] = p.scales[(n0 + r) * p.groups + g];
            }
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int e = e0 + i * kTileThreads, r = e >> per_log2;
                if (r < kTileRows) ss[r * kScalePitch + (e & ((1 << per_log2) - 1))] = f[i];
            }
        }
    };
    uint4 xv[XC];
    float acc[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) acc[i] = 0.0f;
    if (warp < kTileThreads / 32) {
        load_x(xv, first * kSlab);
        if (first < last) load_scales(first);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_at, lanes = (uint32_t)((warp & 3) * 32) << 16;
    const Watchdog wd{a.err, &abort_flag, a.timeout_ns, 12};
    const int halves = first < last ? 2 * (last - first) : 0;
    // most waits find their phase complete: a test first (try_wait alone cost 240 cycles)
    auto wait = [&](uint64_t *bar, int phase, int site) { return mbar_test_wait(bar, phase & 1) || mbar_wait(bar, phase & 1, wd, site); };
    if (warp == kTileThreads / 32) {
        constexpr uint32_t idesc = idesc_bf16_f32(kTileRows, NX);
        const uint32_t d_tmem = __shfl_sync(0xffffffffu, tmem, 0);
        if (elect_one())
            for (int s = first; s < min(first + STAGES, last); ++s) fetch(s);
        int u = 0;
        for (; u < halves; ++u) {
            const int j = u & 1;
            if (!__all_sync(0xffffffffu, wait(&ready[j], u >> 1, 3))) break;
            tc_fence_after();
            if (elect_one()) {
                const uint64_t xd = sdesc_sw128(smem_u32(sx) + j * XHALF, 16, 1024);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    umma_ts(d_tmem + kTileD + ((u >> 2) & 1) * NX, d_tmem + j * 64 + 8 * k, xd + ((k / 4) * XBLOCK + (k % 4) * 32) / 16,
                            idesc, k > 0 || (u & 3) ? 1u : 0u);
                umma_commit(&done[j]);
                // both halves of the slab are widened: its stage is free
                const int to = first + (u >> 1) + STAGES;
                if (j == 1 && to < last) fetch(to);
            }
            __syncwarp();
        }
        if (u < halves && lane == 0) {
            // a wait ran out: products and copies in flight must end before TMEM and shared memory go
            for (int v = max(0, u - 2); v < u; ++v) mbar_drain(&done[v & 1], (v >> 1) & 1, 100000000ull);
            for (int s = u >> 1; s < min((u >> 1) + STAGES, last - first); ++s)
                mbar_drain(&full[s % STAGES], (s / STAGES) & 1, 100000000ull);
        }
        __syncwarp();
    } else {
        bool bad = false;
        // the sums of columns 512 e .. of this CTA's share: the products of four half slabs in one accumulator
        auto collect = [&](int e) {
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < NC; c += 16) {
                float d[16];
                tmem_ld16f_sync(tmem + lanes + kTileD + (e & 1) * NX + part_of * NC + c, d);
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[c + i] += d[i];
            }
        };
        // past the columns TMA fills with zeros, which are the code -8: its product with the scale of a group that K ends in
        // can overflow, and meets zeros of x, so the scale is 0 there (32 columns are in or past together)
        const int columns = p.k - first * kSlab - part_of * 64;
        int u = 0, collected = 0;
        for (; u < halves; ++u) {
            const int it = u >> 1, j = u & 1, s = it % STAGES;
            if (j == 0 && it > 0 && it % kScaleSlabs == 0) {
                named_bar_sync(1, kTileThreads);       // the last scales are read
                load_scales(first + it);
                named_bar_sync(1, kTileThreads);
            }
            bad = !wait(&full[s], it / STAGES, 1);
            if (u >= 2) bad |= !wait(&done[j], (u - 2) >> 1, 2);       // buffer j is free
            if (!__all_sync(0xffffffffu, !bad)) break;
            if (u > 4 && (u & 3) == 1) collect(collected++);
            const __nv_bfloat16 *const sr = ss + row_in * kScalePitch;
            const int col0 = (it % kScaleSlabs) * kSlab + j * 128 + part_of * 64;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const __nv_bfloat16 f = u * 128 + q * 32 < columns ? sr[(col0 + q * 32) >> p.group_log2] : __float2bfloat16_rn(0.0f);
                const uint4 w = *reinterpret_cast<const uint4 *>(sw + s * kTileStage + sw128_offset(row_in, j * 4 + part_of * 2 + q));
                const __nv_bfloat162 sc = __halves2bfloat162(f, f);
                uint32_t r[16];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t v[4];
                    w4_widen(i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w, sc, v);
#pragma unroll
                    for (int k = 0; k < 4; ++k) r[4 * i + k] = v[k];
                }
                tmem_st16(tmem + lanes + j * 64 + part_of * 32 + q * 16, r);
            }
#pragma unroll
            for (int i = 0; i < XC; ++i) {
                const int e = tid + i * kTileThreads, xr = e >> 4, c = e & 15;
                *reinterpret_cast<uint4 *>(sx + j * XHALF + (c >> 3) * XBLOCK + sw128_offset(xr, c & 7)) =
                    make_uint4(__byte_perm(xv[i].x, xv[i].z, 0x5410), __byte_perm(xv[i].x, xv[i].z, 0x7632),
                               __byte_perm(xv[i].y, xv[i].w, 0x5410), __byte_perm(xv[i].y, xv[i].w, 0x7632));
            }
            fence_proxy_async_smem();
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ready[j]);
            load_x(xv, first * kSlab + (u + 1) * 128);
        }
        // a warp whose wait ran out still meets the others at the barriers ahead: they may have waited in time
        if (u < halves)
            for (int it = (u >> 1) + 1; it < last - first; ++it)
                if (it % kScaleSlabs == 0) {
                    named_bar_sync(1, kTileThreads);
                    named_bar_sync(1, kTileThreads);
                }
        if (halves && u == halves) {
            // the last products, and with them all before
            if (__all_sync(0xffffffffu, wait(&done[(u - 1) & 1], (u - 1) >> 1, 4)))
                while (collected <= (u - 1) >> 2) collect(collected++);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, kTileTmem);
    }
    if (ranks == 1) {
        if (warp < kTileThreads / 32 && n0 + row_in < p.n) {
#pragma unroll
            for (int i = 0; i < NC; ++i)
                if (part_of * NC + i < m) w4_store(p, m0 + part_of * NC + i, n0 + row_in, acc[i]);
        }
        return;
    }
    // [NX][128] sums in the slab's place; every CTA of the cluster adds up its share of the rows of W
    float *const part = reinterpret_cast<float *>(sx);
    if (warp < kTileThreads / 32) {
#pragma unroll
        for (int i = 0; i < NC; ++i) part[(part_of * NC + i) * kTileRows + row_in] = acc[i];
    }
    w4_cluster_sync();
    const int rows = kTileRows / ranks;
    for (int e = tid; e < m * rows; e += kTileThreads + 32) {
        const int xr = e / rows, at = rank * rows + e % rows;
        if (n0 + at >= p.n) continue;
        float sum = 0.0f;
        for (uint32_t r = 0; r < ranks; ++r) sum += w4_load_of(smem_u32(part + xr * kTileRows + at), r);
        w4_store(p, m0 + xr, n0 + at, sum);
    }
    w4_cluster_sync();                         // the others may still read this CTA's sums
}

// A word of 8 codes a thread: 16 bytes out, whole lines a warp.
constexpr int kDequantUnroll = 4;

__global__ void __launch_bounds__(256) w4_dequant_kernel(const uint32_t *codes, const __nv_bfloat16 *scales, uint32_t words,
                                                         FastDiv row_words, int32_t groups, int32_t group_log2, uint4 *w) {
    const uint32_t first = blockIdx.x * (256 * kDequantUnroll) + threadIdx.x;
    uint32_t word[kDequantUnroll];
    __nv_bfloat16 f[kDequantUnroll];
#pragma unroll
    for (int u = 0; u < kDequantUnroll; ++u) {
        const uint32_t i = first + u * 256;
        if (i >= words) continue;
        const uint32_t row = fdiv(i, row_words), col = (i - row * row_words.d) * 8;
        word[u] = __ldg(codes + i);
        f[u] = scales[(int64_t)row * groups + (col >> group_log2)];
    }
#pragma unroll
    for (int u = 0; u < kDequantUnroll; ++u) {
        const uint32_t i = first + u * 256;
        if (i >= words) continue;
        uint32_t v[4];
        w4_widen(word[u], __halves2bfloat162(f[u], f[u]), v);
        w[i] = make_uint4(__byte_perm(v[0], v[1], 0x5410), __byte_perm(v[2], v[3], 0x5410), __byte_perm(v[0], v[1], 0x7632),
                          __byte_perm(v[2], v[3], 0x7632));
    }
}

__global__ void __launch_bounds__(256) w4_quantize_kernel(const __nv_bfloat16 *w, int64_t n, int32_t k, int64_t ldw,
                                                          int32_t groups, int32_t group, uint8_t *codes,
                                                          __nv_bfloat16 *scales) {
    const int64_t at = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    const int lane = threadIdx.x & 31;
    if (at >= n * groups) return;
    const int64_t row = at / groups;
    const int32_t gr = (int32_t)(at - row * groups), k0 = gr * group, k1 = min(k, k0 + group);
    const __nv_bfloat16 *src = w + row * ldw;
    float a = 0.0f;
    bool finite = true;
    for (int32_t c = k0 + lane; c < k1; c += 32) {
        const float v = fabsf(__bfloat162float(src[c]));
        finite &= v <= 3.402823466e38f;
        a = fmaxf(a, v);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, off));
    finite = __all_sync(0xffffffffu, finite);
    const __nv_bfloat16 sb = __float2bfloat16_rn(finite ? __fdiv_rn(a, 7.0f) : __int_as_float(0x7fffffff));
    const float s = __bfloat162float(sb);
    if (lane == 0) scales[at] = sb;
    for (int32_t c = k0 + 2 * lane; c < k1; c += 64) {
        uint32_t byte = 0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            int code = 0;
            if (s > 0.0f) code = (int)fminf(7.0f, fmaxf(-7.0f, rintf(__fdiv_rn(__bfloat162float(src[c + h]), s))));
            byte |= (uint32_t)(code + 8) << (4 * h);
        }
        codes[row * (k / 2) + c / 2] = (uint8_t)byte;
    }
}

// ------------------------------------------------------------------------------------------------
// fp32 results of many rows
// ------------------------------------------------------------------------------------------------
// The GEMM's sums stay in the tensor core, which truncates them: relative errors of 1.6e-6 at 2048 columns and 7.7e-6 at
// 8192, far below a bf16 result's rounding but not an fp32 one's.  There it runs on runs of kSumColumns columns, whose
// results are added up in rounded fp32 (7e-7).
constexpr int kSumColumns = 1024, kSumParts = 4;

__global__ void __launch_bounds__(256) w4_sum_kernel(const float4 *parts, int32_t n_parts, int64_t part4, int64_t rows, uint32_t row4,
                                                     float *y, int64_t ldy, uint32_t cols, int32_t add) {
    const int64_t total = rows * row4, stride = (int64_t)gridDim.x * blockDim.x;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += stride) {
        const int64_t row = i / row4;
        const uint32_t col = (uint32_t)(i - row * row4) * 4;
        float4 v[kSumParts];
#pragma unroll
        for (int k = 0; k < kSumParts; ++k)
            if (k < n_parts) v[k] = parts[k * part4 + i];
        float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        float *out = y + row * ldy + col;
        if (add)
            for (int j = 0; j < 4; ++j) s[j] = col + j < cols ? out[j] : 0.0f;
#pragma unroll
        for (int k = 0; k < kSumParts; ++k)
            if (k < n_parts) s[0] += v[k].x, s[1] += v[k].y, s[2] += v[k].z, s[3] += v[k].w;
        for (int j = 0; j < 4; ++j)
            if (col + j < cols) out[j] = s[j];
    }
}

// ------------------------------------------------------------------------------------------------
// host
// ------------------------------------------------------------------------------------------------

// Runs of columns that an fp32 result of the GEMM is summed in (1: the GEMM writes y itself), pitch of a part's rows.
static int64_t w4_runs(int64_t k_in, int y_dtype) {
    return y_dtype == NOMAS_DTYPE_F32 ? (k_in + kSumColumns - 1) / kSumColumns : 1;
}
static int64_t w4_part_pitch(int64_t n_out) { return (n_out + 3) / 4 * 4; }

// Bytes of the bf16 weights, at the front of the workspace.
static size_t w4_weight_bytes(int64_t n_out, int64_t k_in) { return ((size_t)n_out * (size_t)k_in * 2 + 255) / 256 * 256; }

static int enqueue_w4_sums(const void *x, int64_t m, int64_t k_in, int64_t ldx, const void *w, int64_t n_out, float *y, int64_t ldy,
                           float *parts, int32_t *status, nomas_stream stream) {
    const int64_t pitch = w4_part_pitch(n_out), runs = w4_runs(k_in, NOMAS_DTYPE_F32);
    const auto *xb = static_cast<const __nv_bfloat16 *>(x);
    const auto *wb = static_cast<const __nv_bfloat16 *>(w);
    for (int64_t r0 = 0; r0 < runs; r0 += kSumParts) {
        const int n = (int)(runs - r0 < kSumParts ? runs - r0 : kSumParts);
        for (int i = 0; i < n; ++i) {
            const int64_t k0 = (r0 + i) * kSumColumns, kc = k_in - k0 < kSumColumns ? k_in - k0 : kSumColumns;
            const int rc = nomas_linear_bf16(xb + k0, m, kc, ldx, wb + k0, n_out, k_in, parts + i * m * pitch, pitch, NOMAS_DTYPE_F32,
                                             status, stream);
            if (rc) return rc;
        }
        const int64_t total = m * (pitch / 4), most = (int64_t)sm_count() * 16, ctas = (total + 255) / 256;
        w4_sum_kernel<<<(unsigned)(ctas < most ? ctas : most), 256, 0, reinterpret_cast<cudaStream_t>(stream)>>>(
            reinterpret_cast<const float4 *>(parts), n, m * (pitch / 4), m, (uint32_t)(pitch / 4), y, ldy, (uint32_t)n_out, r0 > 0);
        const int rc = check_launch("w4_sum_kernel launch");
        if (rc) return rc;
    }
    return NOMAS_OK;
}

// Rows of x that need no GEMM: up to 128 of them the widened weights' way through memory costs more than it saves where
// rows are long, or W small (us, GEMM with its dequantise pass against this file's kernels: 128 x 2048 -> 2048 13 / 12,
// x 4096 -> 4096 23 / 24, where the two sides meet, x 8192 -> 2048 36 / 23, x 8192 -> 8192 65 / 57, x 2048 -> 12288 21 / 36).
static bool w4_few(int64_t m, int64_t n_out, int64_t k_in) {
    if (m <= NOMAS_W4_FEW_ROWS || (m <= 128 && (n_out <= 4096 || k_in >= 4096))) return true;
    // products that take less than the GEMM's launches (some 20 us)
    return m <= 4096 && m * n_out * k_in <= (int64_t)1 << 29;
}

static int group_log2_of(int group) { return group == 32 ? 5 : group == 64 ? 6 : group == 128 ? 7 : -1; }

static int check_w4_sizes(int64_t n_out, int64_t k_in) {
    if (n_out < 1 || k_in < 32 || k_in % 32 != 0) return NOMAS_EINVAL;
    // 32-bit offsets: of 32 rows in w4_rows_kernel, of words in w4_dequant_kernel
    if (n_out >= (int64_t)1 << 31 || k_in >= (int64_t)1 << 26 || n_out * (k_in / 8) >= (int64_t)1 << 31) return NOMAS_EUNSUPPORTED;
    return NOMAS_OK;
}

static int check_w4(const void *codes, const void *scales, int group, int64_t n_out, int64_t k_in) {
    if (!codes || !scales || !aligned16(codes) || !aligned16(scales) || group_log2_of(group) < 0) return NOMAS_EINVAL;
    return check_w4_sizes(n_out, k_in);
}

static int enqueue_w4_dequant(const uint8_t *codes, const void *scales, int group, int64_t n_out, int64_t k_in, void *w,
                              cudaStream_t st) {
    const int64_t words = n_out * (k_in / 8), per_cta = 256 * kDequantUnroll;
    w4_dequant_kernel<<<(unsigned)((words + per_cta - 1) / per_cta), 256, 0, st>>>(
        reinterpret_cast<const uint32_t *>(codes), static_cast<const __nv_bfloat16 *>(scales), (uint32_t)words,
        make_fastdiv((uint32_t)(k_in / 8)), (int32_t)((k_in + group - 1) / group), group_log2_of(group), static_cast<uint4 *>(w));
    return check_launch("w4_dequant_kernel launch");
}

template <int NT, int RT, int WARPS>
static int launch_w4_rows(const W4Params &p, cudaStream_t st) {
    constexpr int kBytes = WARPS * 8 * NT * (16 * RT + 1) * (int)sizeof(float);
    static_assert(kBytes <= 48 * 1024, "above 48 KB a kernel needs an attribute");
    // more rows of x than a CTA's registers sum: as many CTAs, which find the codes in L2
    const dim3 grid((unsigned)((p.n + 16 * RT - 1) / (16 * RT)), (unsigned)((p.m + 8 * NT - 1) / (8 * NT)));
    w4_rows_kernel<NT, RT, WARPS><<<grid, 32 * WARPS, kBytes, st>>>(p);
    return check_launch("w4_rows_kernel launch");
}

// Rows of W and warps of a CTA.  Long rows of wide matrices: 32 rows (x is read half as often) by 8 warps; else as
// many warps to a row as make some 2000 to 3000 in all, so that the codes on their way fill the machine, and 32 rows by 4
// warps where rows of x make x the larger part.  Measured in us, (rows / 16, warps):
//             (1,4)  (1,8) (1,16)  (2,4)  (2,8)                        (1,4)  (1,8) (1,16)  (2,4)  (2,8)
//    1 x 2048 -> 2048   3.6   2.9    2.8    4.8    3.8     30 x 2048 -> 2048   6.3   5.5    5.7   10.1    7.5
//    1 x 8192 -> 2048   9.8   6.3    5.3   13.5    9.6     30 x 8192 -> 2048  21.3  14.9   13.8   38.5   23.6
//    1 x 4096 -> 4096   6.0   5.0    6.1    7.9    6.0     30 x 4096 -> 4096  14.0  13.7   15.7   18.6   12.8
//    1 x 8192 -> 8192  17.7  19.3   20.9   22.5   14.7     30 x 8192 -> 8192  45.5  46.9   52.0   45.5   31.7
//    1 x 2048 -> 12288  6.2   7.0   10.6    6.7    6.8     30 x 2048 -> 12288 24.1  21.2   26.4   13.4   17.6
//    1 x 8192 -> 28001 39.3  40.9   61.8   35.5   35.7     30 x 8192 -> 28001  133   137    155    117     92
template <int NT>
static int pick_w4_rows(const W4Params &p, cudaStream_t st) {
    const int64_t tiles = (p.n + 15) / 16;
    if (p.k >= 4096 && tiles >= (NT == 1 ? 512 : 256)) return launch_w4_rows<NT, 2, 8>(p, st);
    if (tiles >= 640) return NT == 1 ? launch_w4_rows<NT, 1, 4>(p, st) : launch_w4_rows<NT, 2, 4>(p, st);
    if (p.k < 1024) return launch_w4_rows<NT, 1, 4>(p, st);
    if (tiles >= 256) return NT == 4 ? launch_w4_rows<NT, 2, 8>(p, st) : launch_w4_rows<NT, 1, 8>(p, st);
    return p.k >= (NT == 1 ? 2048 : 4096) ? launch_w4_rows<NT, 1, 16>(p, st) : launch_w4_rows<NT, 1, 8>(p, st);
}

// Whether few rows of x go to w4_tile_kernel rather than w4_rows_kernel, which takes 32 of them at a time and has less
// to set up (us, rows against tiles: 64 x 8192 -> 8192 64 / 33, x 2048 -> 12288 28 / 20, x 4096 -> 4096 19 / 15,
// x 2048 -> 2048 8 / 11; 30 x 8192 -> 8192 32 / 26, x 2048 -> 12288 14 / 16, x 4096 -> 4096 12 / 12; 16 x 8192 -> 8192
// 19 / 25; 128 x 2048 -> 2048 15 / 11).
static bool w4_tiles(int64_t m, int64_t n_out, int64_t k_in) {
    const int64_t weights = n_out * k_in;
    return m > 64 ? weights >= 1 << 22 : m > 32 ? weights >= 1 << 23 : m > 16 && weights >= 1 << 26;
}

template <int NX>
static int launch_w4_tile(const W4Params &p, int32_t *status, cudaStream_t st) {
    CUtensorMap map;
    const cuuint64_t dims[3] = {(cuuint64_t)p.k / 2, (cuuint64_t)p.n, 1};
    const cuuint64_t strides[2] = {(cuuint64_t)p.k / 2, (cuuint64_t)p.k / 2 * (cuuint64_t)p.n};
    const cuuint32_t box[3] = {kSlab / 2, kTileRows, 1};
    if (!make_tensor_map_3d(&map, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.codes, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B))
        return NOMAS_ECUDA;
    W4Tile a{};
    a.p = p;
    a.slabs = (p.k + kSlab - 1) / kSlab;
    a.err = reinterpret_cast<int *>(status);
    a.timeout_ns = wait_limit_ns();
    // CTAs of a cluster: the slabs that the busiest SM gets, two CTAs of it a fifth faster than one after the other, and
    // 1.7 slabs' time for each doubling of the cluster
    const int64_t blocks = (p.m + NX - 1) / NX, tiles = (p.n + kTileRows - 1) / kTileRows;
    int ranks = 1;
    int64_t least = INT64_MAX;
    for (int r = 1, step = 0; r <= 8 && r <= a.slabs; r *= 2, ++step) {
        const int64_t ctas = (tiles * blocks * r + sm_count() - 1) / sm_count(), share = (a.slabs + r - 1) / r;
        const int64_t cost = ctas * share * (ctas == 1 ? 10 : 8) + 17 * step;
        if (cost < least) least = cost, ranks = r;
    }
    a.share = (a.slabs + ranks - 1) / ranks;
    auto kernel = w4_tile_kernel<NX>;
    static std::atomic<uint64_t> allowed{0};   // devices on which the kernel may use its shared memory
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && (dev >= 64 || !(allowed.load() >> dev & 1))) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, TileSmem<NX>::kBytes);
        if (e == cudaSuccess && dev < 64) allowed.fetch_or((uint64_t)1 << dev);
    }
    if (e != cudaSuccess) return cuda_fail("cudaFuncSetAttribute(w4 smem)", (int)e, cudaGetErrorString(e));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles * ranks), (unsigned)blocks);
    cfg.blockDim = dim3(kTileThreads + 32);
    cfg.dynamicSmemBytes = TileSmem<NX>::kBytes;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)ranks;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kernel, map, a);
    return e == cudaSuccess ? NOMAS_OK : cuda_fail("w4_tile_kernel launch", (int)e, cudaGetErrorString(e));
}

}  // namespace nomas

using namespace nomas;

extern "C" int nomas_w4_quantize(const void *w, int64_t n_out, int64_t k_in, int64_t ldw, int group, uint8_t *codes,
                                 void *scales, nomas_stream stream) {
    int rc = check_w4(codes, scales, group, n_out, k_in);
    if (rc) return rc;
    if (!w || !aligned16(w) || ldw < k_in) return NOMAS_EINVAL;
    const int64_t groups = (k_in + group - 1) / group;
    if ((n_out * groups + 7) / 8 >= (int64_t)1 << 31) return NOMAS_EUNSUPPORTED;
    DeviceScope dev(codes);
    if (dev.rc) return dev.rc;
    w4_quantize_kernel<<<(unsigned)((n_out * groups + 7) / 8), 256, 0, reinterpret_cast<cudaStream_t>(stream)>>>(
        static_cast<const __nv_bfloat16 *>(w), n_out, (int32_t)k_in, ldw, (int32_t)groups, group, codes,
        static_cast<__nv_bfloat16 *>(scales));
    return check_launch("w4_quantize_kernel launch");
}

extern "C" int nomas_w4_dequant(const uint8_t *codes, const void *scales, int group, int64_t n_out, int64_t k_in, void *w,
                                nomas_stream stream) {
    int rc = check_w4(codes, scales, group, n_out, k_in);
    if (rc) return rc;
    if (!w || !aligned16(w)) return NOMAS_EINVAL;
    DeviceScope dev(codes);
    if (dev.rc) return dev.rc;
    return enqueue_w4_dequant(codes, scales, group, n_out, k_in, w, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" size_t nomas_w4a16_workspace_bytes(int64_t m, int64_t n_out, int64_t k_in, int y_dtype) {
    if (m < 1 || m >= (int64_t)1 << 31 || check_w4_sizes(n_out, k_in) || w4_few(m, n_out, k_in)) return 0;
    const int64_t runs = w4_runs(k_in, y_dtype);
    const int64_t parts = runs == 1 ? 0 : runs < kSumParts ? runs : kSumParts;
    return w4_weight_bytes(n_out, k_in) + (size_t)parts * (size_t)m * (size_t)w4_part_pitch(n_out) * sizeof(float);
}

extern "C" int nomas_w4a16_linear(const void *x, int64_t m, int64_t k_in, int64_t ldx, const uint8_t *codes,
                                  const void *scales, int group, int64_t n_out, void *y, int64_t ldy, int y_dtype,
                                  void *workspace, int32_t *status, nomas_stream stream) {
    int rc = check_w4(codes, scales, group, n_out, k_in);
    if (rc) return rc;
    if (m < 0 || !x || !y || !status || !aligned16(x) || !aligned16(y) || !aligned16(status)) return NOMAS_EINVAL;
    if (ldx < k_in || ldx % 8 != 0 || ldy < n_out) return NOMAS_EINVAL;
    if (y_dtype != NOMAS_DTYPE_F32 && y_dtype != NOMAS_DTYPE_BF16) return NOMAS_EINVAL;
    if (m >= (int64_t)1 << 31) return NOMAS_EUNSUPPORTED;
    if (!w4_few(m, n_out, k_in) && (!workspace || !aligned16(workspace))) return NOMAS_EINVAL;
    if (m == 0) return NOMAS_OK;
    DeviceScope dev(codes);
    if (dev.rc) return dev.rc;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (!w4_few(m, n_out, k_in)) {
        rc = enqueue_w4_dequant(codes, scales, group, n_out, k_in, workspace, st);
        if (rc) return rc;
        if (w4_runs(k_in, y_dtype) == 1)
            return nomas_linear_bf16(x, m, k_in, ldx, workspace, n_out, k_in, y, ldy, y_dtype, status, stream);
        return enqueue_w4_sums(x, m, k_in, ldx, workspace, n_out, static_cast<float *>(y), ldy,
                               reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + w4_weight_bytes(n_out, k_in)), status,
                               stream);
    }
    W4Params p{};
    p.codes = codes;
    p.scales = static_cast<const __nv_bfloat16 *>(scales);
    p.x = static_cast<const __nv_bfloat16 *>(x);
    p.y = y;
    p.ldx = ldx, p.ldy = ldy, p.n = n_out;
    p.m = (int32_t)m, p.k = (int32_t)k_in;
    p.groups = (int32_t)((k_in + group - 1) / group);
    p.group_log2 = group_log2_of(group);
    p.y_bf16 = y_dtype == NOMAS_DTYPE_BF16;
    if (w4_tiles(m, n_out, k_in))
        return m <= 32 ? launch_w4_tile<32>(p, status, st) : launch_w4_tile<64>(p, status, st);
    if (m <= 8) return pick_w4_rows<1>(p, st);
    if (m <= 16) return pick_w4_rows<2>(p, st);
    return pick_w4_rows<4>(p, st);
}
