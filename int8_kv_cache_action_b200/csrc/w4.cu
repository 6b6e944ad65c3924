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
//                       in shared memory first; it takes over (w4_dequant_kernel, nomas_linear_bf16) for more rows.
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

// CTAs of an SM, from the warps that the sums of RT * NT products leave registers for.  24 warps spill a little with
// RT = 2, and pay on wide matrices (2 x 8192 -> 28001: 35.6 us, 43.9 with 20, 45.3 with 16).
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
// host
// ------------------------------------------------------------------------------------------------

// Rows of x that go to w4_rows_kernel: the GEMM's 128 x 256 tiles leave most SMs idle below 4096 rows of W (100 rows,
// 2048 x 2048: 19 us against 13; at 2048 -> 12288 the GEMM's 34 us are half of what four blocks of 32 rows take).
static bool w4_few(int64_t m, int64_t n_out) { return m <= NOMAS_W4_FEW_ROWS || (m <= 128 && n_out <= 4096); }

static int group_log2_of(int group) { return group == 32 ? 5 : group == 64 ? 6 : group == 128 ? 7 : -1; }

static int check_w4(const void *codes, const void *scales, int group, int64_t n_out, int64_t k_in) {
    if (!codes || !scales || !aligned16(codes) || !aligned16(scales) || group_log2_of(group) < 0) return NOMAS_EINVAL;
    if (n_out < 1 || k_in < 32 || k_in % 32 != 0) return NOMAS_EINVAL;
    // 32-bit offsets: of 32 rows in w4_rows_kernel, of words in w4_dequant_kernel
    if (n_out >= (int64_t)1 << 31 || k_in >= (int64_t)1 << 26 || n_out * (k_in / 8) >= (int64_t)1 << 31) return NOMAS_EUNSUPPORTED;
    return NOMAS_OK;
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
    if (n_out < 1 || k_in < 1 || w4_few(m, n_out)) return 0;
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
    if (!w4_few(m, n_out) && (!workspace || !aligned16(workspace))) return NOMAS_EINVAL;
    if (m == 0) return NOMAS_OK;
    DeviceScope dev(codes);
    if (dev.rc) return dev.rc;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (!w4_few(m, n_out)) {
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
    return pick_w4_rows<4>(p, st);
}
