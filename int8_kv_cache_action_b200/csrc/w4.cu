// Linear layer with 4-bit weights and group scales (definition in nomas.h).
//
// Kernels:
//   w4_quantize_kernel  one warp per (row, group)
//   w4_dequant_kernel   bf16(code * scale), 32 weights per thread (HBM-bound)
//   w4_rows_kernel      y = x W^T for up to NOMAS_W4_FEW_ROWS rows of x, every code read once: bound by the codes'
//                       bytes, so the weights are widened in registers and go straight into the register
//                       form of the tensor-core product (m16n8k16, 16 rows of W by 8 rows of x): one
//                       instruction per 8 weights of a lane, where fp32 products would need one per
//                       weight and row of x.  tcgen05 would want the widened weights in shared memory
//                       first; it takes over (w4_dequant_kernel, nomas_linear_bf16) for more rows.
#include <cstdlib>
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

template <int NT, int RT, int WARPS>
__global__ void __launch_bounds__(32 * WARPS) w4_rows_kernel(const W4Params p) {
    extern __shared__ float red[];             // [WARPS][8 NT][16 RT + 1]
    constexpr int LD = 16 * RT + 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int64_t n0 = (int64_t)blockIdx.x * (16 * RT);
    const int chunks = p.k >> 7, tail = p.k & 127;
    const uint8_t *codes[RT][2];
    const __nv_bfloat16 *scales[RT][2], *xr[NT];
    const int col0 = warp * 128 + 32 * t;
    // rows past the end repeat the last one: their products go nowhere
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t row = min(n0 + 16 * r + 8 * h + g, p.n - 1);
            codes[r][h] = p.codes + row * (p.k / 2) + col0 / 2;
            scales[r][h] = p.scales + row * p.groups;
        }
#pragma unroll
    for (int i = 0; i < NT; ++i) xr[i] = p.x + (int64_t)min(8 * i + g, p.m - 1) * p.ldx + col0;
    float acc[RT][NT][4];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[r][i][j] = 0.0f;

    auto load = [&](W4Codes<RT> &v, int c) {   // chunk c: columns 128 c ..
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                v.w[r][h] = load_stream(codes[r][h] + (c - warp) * 64);
                v.f[r][h] = scales[r][h][(c * 128 + 32 * t) >> p.group_log2];
            }
    };
    auto multiply = [&](const W4Codes<RT> &v, int c, bool in) {
        float part[RT][NT][4];
        __nv_bfloat162 s[RT][2];
#pragma unroll
        for (int r = 0; r < RT; ++r) {
#pragma unroll
            for (int h = 0; h < 2; ++h) s[r][h] = __halves2bfloat162(v.f[r][h], v.f[r][h]);
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) part[r][i][j] = 0.0f;
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
                if (in) xv = __ldg(reinterpret_cast<const uint4 *>(xr[i] + (c - warp) * 128 + 8 * q));
                // pairs (0,4) (1,5) (2,6) (3,7) of 8 columns
                const uint32_t x0 = __byte_perm(xv.x, xv.z, 0x5410), x1 = __byte_perm(xv.x, xv.z, 0x7632);
                const uint32_t x2 = __byte_perm(xv.y, xv.w, 0x5410), x3 = __byte_perm(xv.y, xv.w, 0x7632);
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    mma_16x8x16(part[r][i], u[r][0][0], u[r][1][0], u[r][0][1], u[r][1][1], x0, x1);
                    mma_16x8x16(part[r][i], u[r][0][2], u[r][1][2], u[r][0][3], u[r][1][3], x2, x3);
                }
            }
            // the tensor cores truncate sums: short runs of columns are added up in rounded fp32 (a whole chunk while
            // its sums fit the registers)
            if (q == 3 || RT * NT > 2) {
#pragma unroll
                for (int r = 0; r < RT; ++r)
#pragma unroll
                    for (int i = 0; i < NT; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            acc[r][i][j] += part[r][i][j];
                            part[r][i][j] = 0.0f;
                        }
            }
        }
    };

    W4Codes<RT> now, next;
    if (warp < chunks) load(now, warp);
    for (int c = warp; c < chunks; c += WARPS) {
        if (c + WARPS < chunks) load(next, c + WARPS);
        multiply(now, c, true);
        now = next;
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
    for (int e = threadIdx.x; e < NT * 8 * 16 * RT; e += 32 * WARPS) {
        const int row = e / (16 * RT), col = e % (16 * RT);
        if (row >= p.m || n0 + col >= p.n) continue;
        float s = red[row * LD + col];
#pragma unroll
        for (int w = 1; w < WARPS; ++w) s += red[(w * 8 * NT + row) * LD + col];
        if (p.y_bf16)
            static_cast<__nv_bfloat16 *>(p.y)[(int64_t)row * p.ldy + n0 + col] = __float2bfloat16_rn(s);
        else
            static_cast<float *>(p.y)[(int64_t)row * p.ldy + n0 + col] = s;
    }
}

// The same with x resident: the CTA holds all of x in shared memory, in the order in which lanes take it, and walks
// over tiles of rows of W; its warps are wk columns by WARPS / wk rows of 16 RT.  Every thread copies the codes it
// will widen itself, kW4Stages - 1 steps (chunks of its warp, over all tiles) ahead, through a ring of its own in shared
// memory; scales come one step ahead.
constexpr int kW4Stages = 4;

struct W4Resident {
    W4Params p;
    int32_t wk_log2, x_pitch;                  // x_pitch: bytes of a row of x in shared memory
    uint32_t tiles;
};

template <int NT, int RT>
constexpr int w4_buffers = NT * RT <= 4 ? 2 : 1;

template <int NT, int RT, int WARPS>
__global__ void __launch_bounds__(32 * WARPS, WARPS == 8 ? (RT * NT == 1 ? 3 : 2) : 1) w4_resident_kernel(const W4Resident a) {
    constexpr int S = kW4Stages, T = 32 * WARPS, LD = 16 * RT + 1, BUFFERS = w4_buffers<NT, RT>;
    extern __shared__ __align__(16) uint8_t smem[];
    const W4Params &p = a.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int wk = 1 << a.wk_log2, kw = warp & (wk - 1), rw = warp >> a.wk_log2;
    const int tile_rows = (16 * RT * WARPS) >> a.wk_log2, chunks = (p.k + 127) >> 7;
    const uint32_t ring_at = smem_u32(smem) + threadIdx.x * 16;
    uint8_t *const xs = smem + S * RT * 2 * T * 16;
    float *const red = reinterpret_cast<float *>(xs + p.m * a.x_pitch);     // [BUFFERS][WARPS][8 NT][LD]

    // the rows of W that this lane widens (g + 8 h of the warp's r-th 16; rows past the end repeat the last one), as
    // 32-bit byte offsets: codes for the tile being fetched, scales for the tile of the next step
    auto rows_of = [&](uint32_t tile, uint32_t pitch, uint32_t (&at)[RT][2]) {
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                at[r][h] = min(tile * tile_rows + rw * (16 * RT) + 16 * r + 8 * h + g, (uint32_t)p.n - 1) * pitch;
    };
    uint32_t fetch_tile = blockIdx.x, code_at[RT][2], scale_at[RT][2];
    int fetch_c = kw;
    rows_of(fetch_tile, p.k / 2, code_at);
    rows_of(fetch_tile, 2 * p.groups, scale_at);
    auto fetch = [&](int stage) {
        if (fetch_tile < a.tiles) {
            const int col = fetch_c * 128 + 32 * t, n = col < p.k ? 16 : 0;
            const uint32_t off = n ? col / 2 : 0;
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(ring_at + ((stage * RT + r) * 2 + h) * T * 16),
                                 "l"(p.codes + (code_at[r][h] + off)), "r"(n)
                                 : "memory");
            fetch_c += wk;
            if (fetch_c >= chunks) {
                fetch_c = kw;
                fetch_tile += gridDim.x;
                rows_of(fetch_tile, p.k / 2, code_at);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < S - 1; ++i) fetch(i);

    // x: 8 columns 128 c + 32 t + 8 q .. of a row as pairs (0,4) (1,5) (2,6) (3,7), 16 bytes at ((c * 4 + q) * 4 + t)
    for (int row = 0; row < p.m; ++row)
        for (int e = threadIdx.x; e < chunks * 16; e += T) {
            const int col = (e >> 4) * 128 + (e & 3) * 32 + ((e >> 2) & 3) * 8;
            uint4 v = make_uint4(0, 0, 0, 0);
            if (col < p.k) v = __ldg(reinterpret_cast<const uint4 *>(p.x + (int64_t)row * p.ldx + col));
            *reinterpret_cast<uint4 *>(xs + row * a.x_pitch + e * 16) =
                make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632), __byte_perm(v.y, v.w, 0x5410),
                           __byte_perm(v.y, v.w, 0x7632));
        }
    const uint8_t *xr[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) xr[i] = xs + min(8 * i + g, p.m - 1) * a.x_pitch + t * 16;

    __nv_bfloat16 next_f[RT][2];
    auto next_scales = [&](int c) {
        const int col = c * 128 + 32 * t;
        const uint32_t off = 2 * (col >> p.group_log2);
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                next_f[r][h] = col < p.k ? *reinterpret_cast<const __nv_bfloat16 *>(
                                               reinterpret_cast<const uint8_t *>(p.scales) + (scale_at[r][h] + off))
                                         : __float2bfloat16_rn(0.0f);
    };
    next_scales(kw);
    __syncthreads();

    int stage = 0, buffer = 0;
    for (uint32_t tile = blockIdx.x; tile < a.tiles; tile += gridDim.x) {
        float acc[RT][NT][4];
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[r][i][j] = 0.0f;
        for (int c = kw; c < chunks; c += wk) {
            fetch((stage + S - 1) % S);
            __nv_bfloat162 s[RT][2];
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int h = 0; h < 2; ++h) s[r][h] = __halves2bfloat162(next_f[r][h], next_f[r][h]);
            if (c + wk < chunks) {
                next_scales(c + wk);
            } else {
                rows_of(tile + gridDim.x, 2 * p.groups, scale_at);
                next_scales(kw);
            }
            asm volatile("cp.async.wait_group %0;" ::"n"(S - 1) : "memory");
            uint4 w[RT][2];
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    w[r][h] = *reinterpret_cast<const uint4 *>(smem + ((stage * RT + r) * 2 + h) * T * 16 + threadIdx.x * 16);
            stage = (stage + 1) % S;
            float part[RT][NT][4];
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int i = 0; i < NT; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) part[r][i][j] = 0.0f;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint32_t u[RT][2][4];
#pragma unroll
                for (int r = 0; r < RT; ++r)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        w4_widen(q == 0 ? w[r][h].x : q == 1 ? w[r][h].y : q == 2 ? w[r][h].z : w[r][h].w, s[r][h], u[r][h]);
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    const uint4 xv = *reinterpret_cast<const uint4 *>(xr[i] + (c * 4 + q) * 64);
#pragma unroll
                    for (int r = 0; r < RT; ++r) {
                        mma_16x8x16(part[r][i], u[r][0][0], u[r][1][0], u[r][0][1], u[r][1][1], xv.x, xv.y);
                        mma_16x8x16(part[r][i], u[r][0][2], u[r][1][2], u[r][0][3], u[r][1][3], xv.z, xv.w);
                    }
                }
                // the tensor cores truncate sums: short runs of columns are added up in rounded fp32 (a whole chunk
                // while its sums fit the registers)
                if (q == 3 || RT * NT > 2) {
#pragma unroll
                    for (int r = 0; r < RT; ++r)
#pragma unroll
                        for (int i = 0; i < NT; ++i)
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                acc[r][i][j] += part[r][i][j];
                                part[r][i][j] = 0.0f;
                            }
                }
            }
        }
        // acc: rows g and g + 8 of W, rows 8 i + 2 t and 8 i + 2 t + 1 of x; with two buffers one barrier of the warps
        // that share rows is enough
        float *all = red + (buffer * WARPS + (rw << a.wk_log2)) * 8 * NT * LD, *mine = all + kw * 8 * NT * LD;
        if (BUFFERS == 2) buffer ^= 1;
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) mine[(8 * i + 2 * t + (j & 1)) * LD + 16 * r + 8 * (j >> 1) + g] = acc[r][i][j];
        if (wk == 1)
            __syncwarp();
        else
            named_bar_sync(1 + rw, 32 * wk);
        const int64_t n0 = (int64_t)tile * tile_rows + rw * (16 * RT);
        for (int e = kw * 32 + lane; e < p.m * 16 * RT; e += 32 * wk) {
            const int row = e / (16 * RT), col = e % (16 * RT);
            if (n0 + col >= p.n) continue;
            float sum = all[row * LD + col];
            for (int w = 1; w < wk; ++w) sum += all[(w * 8 * NT + row) * LD + col];
            if (p.y_bf16)
                static_cast<__nv_bfloat16 *>(p.y)[(int64_t)row * p.ldy + n0 + col] = __float2bfloat16_rn(sum);
            else
                static_cast<float *>(p.y)[(int64_t)row * p.ldy + n0 + col] = sum;
        }
        if (BUFFERS == 1 && wk > 1) named_bar_sync(1 + rw, 32 * wk);
        if (BUFFERS == 1 && wk == 1) __syncwarp();
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

__global__ void __launch_bounds__(256) w4_dequant_kernel(const uint8_t *codes, const __nv_bfloat16 *scales, int64_t total32,
                                                         int32_t k32, int32_t groups, int32_t group_log2,
                                                         __nv_bfloat16 *w) {
    const int64_t stride = (int64_t)gridDim.x * blockDim.x;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total32; i += stride) {
        const int64_t row = i / k32;
        const int32_t col = (int32_t)(i - row * k32) * 32;
        const __nv_bfloat16 f = scales[row * groups + (col >> group_log2)];
        const __nv_bfloat162 s = __halves2bfloat162(f, f);
        const uint4 c = load_stream(codes + i * 16);
        const uint32_t word[4] = {c.x, c.y, c.z, c.w};
        uint4 *dst = reinterpret_cast<uint4 *>(w + i * 32);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            uint32_t u[4];
            w4_widen(word[q], s, u);
            dst[q] = make_uint4(__byte_perm(u[0], u[1], 0x5410), __byte_perm(u[2], u[3], 0x5410),
                                __byte_perm(u[0], u[1], 0x7632), __byte_perm(u[2], u[3], 0x7632));
        }
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
// host
// ------------------------------------------------------------------------------------------------

static int group_log2_of(int group) { return group == 32 ? 5 : group == 64 ? 6 : group == 128 ? 7 : -1; }

static int check_w4(const void *codes, const void *scales, int group, int64_t n_out, int64_t k_in) {
    if (!codes || !scales || !aligned16(codes) || !aligned16(scales) || group_log2_of(group) < 0) return NOMAS_EINVAL;
    if (n_out < 1 || k_in < 32 || k_in % 32 != 0) return NOMAS_EINVAL;
    if (n_out >= (int64_t)1 << 31 || k_in >= (int64_t)1 << 30) return NOMAS_EUNSUPPORTED;
    return NOMAS_OK;
}

static int enqueue_w4_dequant(const uint8_t *codes, const void *scales, int group, int64_t n_out, int64_t k_in, void *w,
                              cudaStream_t st) {
    const int64_t total = n_out * (k_in / 32), most = (int64_t)sm_count() * 8;
    const int64_t blocks = (total + 255) / 256;
    w4_dequant_kernel<<<(unsigned)(blocks < most ? blocks : most), 256, 0, st>>>(
        codes, static_cast<const __nv_bfloat16 *>(scales), total, (int32_t)(k_in / 32), (int32_t)((k_in + group - 1) / group),
        group_log2_of(group), static_cast<__nv_bfloat16 *>(w));
    return check_launch("w4_dequant_kernel launch");
}

template <int NT, int RT, int WARPS>
static int launch_w4_rows(const W4Params &p, cudaStream_t st) {
    constexpr int kBytes = WARPS * 8 * NT * (16 * RT + 1) * (int)sizeof(float);
    static_assert(kBytes <= 48 * 1024, "no opt-in");
    w4_rows_kernel<NT, RT, WARPS><<<(unsigned)((p.n + 16 * RT - 1) / (16 * RT)), 32 * WARPS, kBytes, st>>>(p);
    return check_launch("w4_rows_kernel launch");
}

template <int NT, int RT>
static int pick_w4_warps(const W4Params &p, int warps, cudaStream_t st) {
    if (warps == 4) return launch_w4_rows<NT, RT, 4>(p, st);
    if constexpr (NT * RT <= 4) {
        if (warps == 16) return launch_w4_rows<NT, RT, 16>(p, st);
    }
    if constexpr (NT * RT <= 8) return launch_w4_rows<NT, RT, 8>(p, st);
    return launch_w4_rows<NT, RT, 4>(p, st);
}

template <int NT, int RT, int WARPS>
static int launch_w4_resident(const W4Params &p, int wk_log2, cudaStream_t st) {
    W4Resident a{};
    a.p = p;
    a.wk_log2 = wk_log2;
    a.x_pitch = ((p.k + 127) / 128) * 256 + 64;         // neighbouring rows 64 bytes apart in the banks
    const int rows = (16 * RT * WARPS) >> wk_log2;
    a.tiles = (uint32_t)((p.n + rows - 1) / rows);
    const int64_t bytes = (int64_t)kW4Stages * RT * 2 * 32 * WARPS * 16 + (int64_t)p.m * a.x_pitch +
                          w4_buffers<NT, RT> * WARPS * 8 * NT * (16 * RT + 1) * (int64_t)sizeof(float);
    auto kernel = w4_resident_kernel<NT, RT, WARPS>;
    if (bytes > 224 * 1024 || (1 << wk_log2) > WARPS) return launch_w4_rows<NT, NT * RT <= 8 ? RT : 1, 8>(p, st);
    cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    int64_t ctas = (int64_t)sm_count() * (WARPS == 8 && bytes <= 112 * 1024 ? (RT * NT == 1 && bytes <= 74 * 1024 ? 3 : 2) : 1);
    if (ctas > a.tiles) ctas = a.tiles;
    kernel<<<(unsigned)ctas, 32 * WARPS, (size_t)bytes, st>>>(a);
    return check_launch("w4_resident_kernel launch");
}

template <int NT>
static int pick_w4_rows(const W4Params &p, cudaStream_t st) {
    static const int rt = getenv("W4RT") ? atoi(getenv("W4RT")) : 2, warps = getenv("W4W") ? atoi(getenv("W4W")) : 8;
    static const int wk = getenv("W4K") ? atoi(getenv("W4K")) : 3;
    if constexpr (NT <= 4) {
        if (wk >= 0) {
            if (warps == 16) return rt == 1 ? launch_w4_resident<NT, 1, 16>(p, wk, st) : launch_w4_resident<NT, 2, 16>(p, wk, st);
            return rt == 1 ? launch_w4_resident<NT, 1, 8>(p, wk, st) : launch_w4_resident<NT, 2, 8>(p, wk, st);
        }
    }
    return rt == 1 ? pick_w4_warps<NT, 1>(p, warps, st) : pick_w4_warps<NT, 2>(p, warps, st);
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

extern "C" size_t nomas_w4a16_workspace_bytes(int64_t m, int64_t n_out, int64_t k_in) {
    if (m <= NOMAS_W4_FEW_ROWS || n_out < 1 || k_in < 1) return 0;
    return (size_t)n_out * (size_t)k_in * 2;
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
    if (m > NOMAS_W4_FEW_ROWS && (!workspace || !aligned16(workspace))) return NOMAS_EINVAL;
    if (m == 0) return NOMAS_OK;
    DeviceScope dev(codes);
    if (dev.rc) return dev.rc;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (m > NOMAS_W4_FEW_ROWS) {
        rc = enqueue_w4_dequant(codes, scales, group, n_out, k_in, workspace, st);
        if (rc) return rc;
        return nomas_linear_bf16(x, m, k_in, ldx, workspace, n_out, k_in, y, ldy, y_dtype, status, stream);
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
    if (m <= 8) return pick_w4_rows<1>(p, st);
    if (m <= 16) return pick_w4_rows<2>(p, st);
    if (m <= 32) return pick_w4_rows<4>(p, st);
    return pick_w4_rows<8>(p, st);
}
