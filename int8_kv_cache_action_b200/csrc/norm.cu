// Layer norm with a weight and bias row per group of rows, forward and backward (definition in nomas.h):
// the norm and modulation in front of the DiT's linear layers.
//
// Both directions are bound by HBM: the forward pass reads x and writes y, the backward pass reads dy and
// x and writes dx, about 8 and 14 flops a value.  A row stays in the registers of a team of threads (a
// power of two), so that the variance is a second sum over registers (exact differences, no sum of squares
// that cancels) and memory is read once.  26400 x 2048 in bf16, modulated by groups of 880 rows: forward 40 us,
// backward 60 us, both 5.4 TB/s, where a copy of this pattern reaches 5.5 to 5.8.
//   layernorm_row_kernel   forward, one row per team, loads straight into registers: few rows (latency), and
//                          groups of few rows
//   layernorm_fwd_kernel   forward, a CTA takes a contiguous share of the rows.  Every thread keeps its own
//                          ring of 16-byte chunks in shared memory, filled by asynchronous copies several rows
//                          ahead (nothing to synchronise: a thread reads what it copied); layouts that allow no
//                          copies of 8 bytes hold the next rows in registers.  A thread owns
//                          columns, whose weight and bias stay in its registers for a group, and takes R rows
//                          at a time, which share the two exchanges of sums between the warps.
//   layernorm_bwd_kernel   the same for dy and x; dw and db of a group add up in the registers in row order.  Groups
//                          inside a share are written at once; where a group goes on in the next share, its sums so
//                          far go to the workspace (two slots a CTA).
//   layernorm_grad_kernel  adds up the shares of such groups, in share order.
#include <atomic>

#include "common.cuh"

namespace nomas {

constexpr int kNormThreads = 256;

struct NormParams {
    const void *x, *w, *b;
    void *y;
    float *mean, *rstd;
    int64_t ldx, ldy, ldp;
    uint32_t rows, cols;
    FastDiv group;              // rows of a group
    int32_t team_log2;          // log2(threads of a team)
    int32_t p_bf16;
    float unit, eps;
    uint32_t share;             // rows of a CTA (layernorm_fwd_kernel)
};

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ uint32_t bf16x2_of(float lo, float hi) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&b);
}

// CH consecutive values at p + i as fp32, one wide access for CH = 4 or 8.
template <int CH>
__device__ __forceinline__ void load_chunk(const __nv_bfloat16 *p, float (&v)[CH]) {
    if constexpr (CH == 1) {
        v[0] = __bfloat162float(*p);
    } else if constexpr (CH == 4) {
        const uint2 c = *reinterpret_cast<const uint2 *>(p);
        v[0] = bf16_lo(c.x), v[1] = bf16_hi(c.x), v[2] = bf16_lo(c.y), v[3] = bf16_hi(c.y);
    } else {
        const uint4 c = *reinterpret_cast<const uint4 *>(p);
        v[0] = bf16_lo(c.x), v[1] = bf16_hi(c.x), v[2] = bf16_lo(c.y), v[3] = bf16_hi(c.y);
        v[4] = bf16_lo(c.z), v[5] = bf16_hi(c.z), v[6] = bf16_lo(c.w), v[7] = bf16_hi(c.w);
    }
}
template <int CH>
__device__ __forceinline__ void load_chunk(const float *p, float (&v)[CH]) {
    if constexpr (CH == 1) {
        v[0] = *p;
    } else {
#pragma unroll
        for (int i = 0; i < CH; i += 4) {
            const float4 c = *reinterpret_cast<const float4 *>(p + i);
            v[i] = c.x, v[i + 1] = c.y, v[i + 2] = c.z, v[i + 3] = c.w;
        }
    }
}
template <int CH>
__device__ __forceinline__ void store_chunk(__nv_bfloat16 *p, const float (&v)[CH]) {
    if constexpr (CH == 1)
        *p = __float2bfloat16_rn(v[0]);
    else if constexpr (CH == 4)
        *reinterpret_cast<uint2 *>(p) = make_uint2(bf16x2_of(v[0], v[1]), bf16x2_of(v[2], v[3]));
    else
        *reinterpret_cast<uint4 *>(p) =
            make_uint4(bf16x2_of(v[0], v[1]), bf16x2_of(v[2], v[3]), bf16x2_of(v[4], v[5]), bf16x2_of(v[6], v[7]));
}
template <int CH>
__device__ __forceinline__ void store_chunk(float *p, const float (&v)[CH]) {
    if constexpr (CH == 1) {
        *p = v[0];
    } else {
#pragma unroll
        for (int i = 0; i < CH; i += 4)
            *reinterpret_cast<float4 *>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
    }
}

// A row of w or b (bf16 or fp32).
template <int CH>
__device__ __forceinline__ void load_param(const void *base, int32_t bf16, int64_t at, float (&v)[CH]) {
    if (bf16)
        load_chunk<CH>(static_cast<const __nv_bfloat16 *>(base) + at, v);
    else
        load_chunk<CH>(static_cast<const float *>(base) + at, v);
}

// Two fp32 values in a register pair: the packed instructions of sm_100 do two roundings of fp32 each, at half the
// issue slots.  The wide kernels are close to bound by issue otherwise (forward, 26400 x 2048: 22 instructions a
// value and 56 us with scalar sums).
typedef unsigned long long Pair;
__device__ __forceinline__ Pair pair_of(float lo, float hi) {
    Pair r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void pair_split(Pair v, float &lo, float &hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }
__device__ __forceinline__ float pair_sum(Pair v) {
    float lo, hi;
    pair_split(v, lo, hi);
    return lo + hi;
}
__device__ __forceinline__ Pair add2(Pair a, Pair b) {
    Pair r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
    Pair r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
    Pair r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

template <int V>
constexpr int LOG2 = V <= 1 ? 0 : 1 + LOG2<V / 2>;
template <>
constexpr int LOG2<1> = 0;

// Sums of N values (N = 1, 2, 4, 8) over a team of 2^log2 threads; every thread gets them, in an order that
// depends on the team alone.  In a warp the N values are halved between the lanes as they are added up (N - 1
// + log2(32 / N) shuffles, not 5 N).  Teams of more than a warp meet in `red` (N floats per warp of the CTA and
// parity) at a barrier of their own; a team's threads call it equally often.
template <int N>
__device__ __forceinline__ void team_sum(float (&v)[N], int log2, float *red, int &parity) {
    const int lane = threadIdx.x & 31;
    if (log2 < 5) {
#pragma unroll
        for (int off = 1; off < 16; off <<= 1) {
            if (off >> log2) break;
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], off);
        }
        return;
    }
#pragma unroll
    for (int n = N / 2, off = 16; n >= 1; n >>= 1, off >>= 1) {
        const bool upper = lane & off;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const float give = upper ? v[i] : v[i + n], keep = upper ? v[i + n] : v[i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, give, off);
        }
    }
#pragma unroll
    for (int off = 16 / N; off >= 1; off >>= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], off);
    // value i is in the lanes 32 / N * i ..
    float s = v[0];
    int step = 32 / N;
    if (log2 > 5) {
        const int warp = threadIdx.x >> 5, warps = 1 << (log2 - 5), first = warp & ~(warps - 1);
        float *r = red + parity * (int)(blockDim.x >> 5) * N;
        parity ^= 1;            // the next sum's writes do not meet this one's reads
        if (lane % step == 0) r[warp * N + lane / step] = s;
        named_bar_sync(1 + (int)(threadIdx.x >> log2), 1 << log2);
        s = 0.0f;
        for (int e = lane; e < warps * N; e += 32) s += r[first * N + e];
#pragma unroll
        for (int off = 16; off >= N; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
        step = 1;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = __shfl_sync(0xffffffffu, s, i * step);
}

// Asynchronous copy of a chunk of BYTES (8 or 16) into shared memory, in the groups that ring_commit closes; zeros
// and no read where it is not live, so that the reader needs no branch.
template <int BYTES>
__device__ __forceinline__ void ring_load(uint32_t dst, const void *src, bool live) {
    const int n = live ? BYTES : 0;
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(BYTES), "r"(n) : "memory");
}
__device__ __forceinline__ void ring_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the newest N groups of this thread have landed.
template <int N>
__device__ __forceinline__ void ring_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Mean and 1 / sqrt(variance + eps) of the row in v; v becomes x - mean.
template <int CH, int NV>
__device__ __forceinline__ float centre_row(float (&v)[NV][CH], int lane, const NormParams &p, float *red, int &parity,
                                            float &mean) {
    const int team = 1 << p.team_log2;
    float s[1] = {0.0f};
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < CH; ++i) s[0] += v[j][i];
    team_sum<1>(s, p.team_log2, red, parity);
    mean = s[0] / (float)p.cols;
    s[0] = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const bool in = (uint32_t)(lane + j * team) * CH < p.cols;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            v[j][i] -= mean;
            if (in) s[0] = fmaf(v[j][i], v[j][i], s[0]);
        }
    }
    team_sum<1>(s, p.team_log2, red, parity);
    return rsqrtf(s[0] / (float)p.cols + p.eps);
}

template <typename TX, typename TY, int CH, int NV>
__global__ void __launch_bounds__(kNormThreads) layernorm_row_kernel(const NormParams p) {
    __shared__ float red[2 * kNormThreads / 32];
    const int team = 1 << p.team_log2, lane = threadIdx.x & (team - 1);
    const int64_t row = ((int64_t)blockIdx.x * kNormThreads + threadIdx.x) >> p.team_log2;
    const bool live = row < p.rows;
    const TX *x = static_cast<const TX *>(p.x) + row * p.ldx;
    const int64_t pg = live ? (int64_t)fdiv((uint32_t)row, p.group) * p.ldp : 0;
    float v[NV][CH], w[NV][CH], b[NV][CH];
    int parity = 0;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const uint32_t c = (uint32_t)(lane + j * team) * CH;
#pragma unroll
        for (int i = 0; i < CH; ++i) v[j][i] = b[j][i] = 0.0f, w[j][i] = 1.0f - p.unit;
        if (!live || c >= p.cols) continue;
        load_chunk<CH>(x + c, v[j]);
        if (p.w) load_param<CH>(p.w, p.p_bf16, pg + c, w[j]);
        if (p.b) load_param<CH>(p.b, p.p_bf16, pg + c, b[j]);
    }
    float mean;
    const float rstd = centre_row<CH, NV>(v, lane, p, red, parity, mean);
    if (!live) return;
    if (lane == 0) {
        if (p.mean) p.mean[row] = mean;
        if (p.rstd) p.rstd[row] = rstd;
    }
    TY *y = static_cast<TY *>(p.y) + row * p.ldy;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const uint32_t c = (uint32_t)(lane + j * team) * CH;
        if (c >= p.cols) continue;
#pragma unroll
        for (int i = 0; i < CH; ++i) v[j][i] = fmaf(v[j][i] * rstd, p.unit + w[j][i], b[j][i]);
        store_chunk<CH>(y + c, v[j]);
    }
}

// Forward ring: stages of R rows of x, two to four, so that three CTAs of 256 threads (one of 512) fit an SM; none in
// narrow layouts (no copies of 8 bytes and more), where the next rows wait in registers.
template <typename TX, int CH, int NV, int R, int T>
struct FwdRing {
    static constexpr int kStage = R * NV * CH * (int)sizeof(TX) * T;
    static constexpr int kFit = (T == 256 ? 72 : 200) * 1024 / kStage;
    static constexpr int kStages = CH == 1 ? 0 : kFit < 2 ? 2 : kFit > 4 ? 4 : kFit;
    static constexpr int kBytes = kStages * kStage;
};

// ALONE: one team a CTA (rows of more than half of what its threads hold at a chunk each).
template <typename TX, typename TY, int CH, int NV, int R, int T, bool ALONE>
__global__ void __launch_bounds__(T, T == 256 ? (CH == 1 ? 2 : 3) : 1) layernorm_fwd_kernel(const NormParams p) {
    constexpr bool RING = CH > 1;
    constexpr int S = RING ? FwdRing<TX, CH, NV, R, T>::kStages : 1, BYTES = CH * sizeof(TX);
    constexpr int E = NV * CH, P = E / 2;       // values of a row per thread, in pairs
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float red[2 * (T / 32) * R];
    const int team_log2 = ALONE ? LOG2<T> : p.team_log2, team = 1 << team_log2;
    const int lane = threadIdx.x & (team - 1), mine = ALONE ? 0 : threadIdx.x >> team_log2;
    const uint32_t teams = T >> team_log2;
    const uint32_t begin = blockIdx.x * p.share, end = min(p.rows, begin + p.share);
    const uint8_t *ring = smem + threadIdx.x * BYTES;
    const float inv = 1.0f / (float)p.cols;
    int parity = 0;
    // the batches of the share in order: R * teams rows from fetch_row, inside the group that ends at fetch_stop
    uint32_t fetch_row = begin, fetch_stop = begin;
    const uint32_t ring_at = smem_u32(ring);
    const TX *from = static_cast<const TX *>(p.x) + (int64_t)mine * p.ldx + lane * CH;
    const int64_t row_step = (int64_t)teams * p.ldx;
    TX next[RING ? 1 : R][RING ? 1 : E];
    auto fetch = [&](int stage) {
        if (fetch_row < end) {
            if (fetch_row >= fetch_stop)
                fetch_stop = (uint32_t)min((int64_t)end, ((int64_t)fdiv(fetch_row, p.group) + 1) * p.group.d);
            const TX *x = from + fetch_row * p.ldx;
            const uint32_t to = ring_at + stage * (R * NV * T * BYTES);
#pragma unroll
            for (int r = 0; r < R; ++r, x += row_step) {
                const bool live = fetch_row + r * teams + mine < fetch_stop;
#pragma unroll
                for (int j = 0; j < NV; ++j) {
                    const bool in = live && (uint32_t)(lane + j * team) * CH < p.cols;
                    if constexpr (RING)
                        ring_load<BYTES>(to + (r * NV + j) * T * BYTES, in ? x + j * team * CH : p.x, in);
                    else
                        next[r][j] = in ? x[j * team] : (TX)0.0f;
                }
            }
            fetch_row = min(fetch_row + R * teams, fetch_stop);
        }
        if constexpr (RING) ring_commit();
    };
    if constexpr (RING) {
#pragma unroll
        for (int k = 0; k < S - 1; ++k) fetch(k);
    } else {
        fetch(0);
    }
    int stage = 0, last = S - 1;
    for (uint32_t row = begin; row < end;) {
        const uint32_t g = fdiv(row, p.group), stop = (uint32_t)min((int64_t)end, ((int64_t)g + 1) * p.group.d);
        Pair f[P], b[P];                        // u + w and b of this thread's columns
        {
            float w[NV][CH], bias[NV][CH];
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const uint32_t c = (uint32_t)(lane + j * team) * CH;
#pragma unroll
                for (int i = 0; i < CH; ++i) w[j][i] = 1.0f - p.unit, bias[j][i] = 0.0f;
                if (p.w && c < p.cols) load_param<CH>(p.w, p.p_bf16, (int64_t)g * p.ldp + c, w[j]);
                if (p.b && c < p.cols) load_param<CH>(p.b, p.p_bf16, (int64_t)g * p.ldp + c, bias[j]);
            }
#pragma unroll
            for (int k = 0; k < P; ++k) {
                f[k] = pair_of(p.unit + w[2 * k / CH][2 * k % CH], p.unit + w[(2 * k + 1) / CH][(2 * k + 1) % CH]);
                b[k] = pair_of(bias[2 * k / CH][2 * k % CH], bias[(2 * k + 1) / CH][(2 * k + 1) % CH]);
            }
        }
        for (uint32_t r0 = row; r0 < stop; r0 += teams * R) {
            if constexpr (RING) {
                fetch(last);
                ring_wait<S - 1>();
            }
            Pair v[R][P];
            float s[R], mean[R];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                float fx[NV][CH];
#pragma unroll
                for (int j = 0; j < NV; ++j) {
                    if constexpr (RING)
                        load_chunk<CH>(reinterpret_cast<const TX *>(ring + ((stage * R + r) * NV + j) * T * BYTES), fx[j]);
                    else
                        fx[j][0] = (float)next[r][j];
                }
                Pair sum = 0;
#pragma unroll
                for (int k = 0; k < P; ++k) {
                    v[r][k] = pair_of(fx[2 * k / CH][2 * k % CH], fx[(2 * k + 1) / CH][(2 * k + 1) % CH]);
                    sum = add2(sum, v[r][k]);
                }
                s[r] = pair_sum(sum);
            }
            if constexpr (!RING) fetch(0);
            last = stage;
            stage = stage + 1 == S ? 0 : stage + 1;
            team_sum<R>(s, team_log2, red, parity);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                mean[r] = s[r] * inv;
                const Pair minus = pair_of(-mean[r], -mean[r]);
                Pair sum = 0;
#pragma unroll
                for (int j = 0; j < NV; ++j) {
                    const bool in = (uint32_t)(lane + j * team) * CH < p.cols;
                    if constexpr (CH == 1) {    // a pair is two chunks: where there is no column it holds the mean
                        float lo, hi;
                        pair_split(v[r][j / 2], lo, hi);
                        if (!in) (j & 1 ? hi : lo) = mean[r];
                        v[r][j / 2] = pair_of(lo, hi);
                        if ((j & 1) == 0) continue;
                        v[r][j / 2] = add2(v[r][j / 2], minus);
                        sum = fma2(v[r][j / 2], v[r][j / 2], sum);
                    } else {
                        const Pair before = sum;
#pragma unroll
                        for (int k = j * CH / 2; k < (j + 1) * CH / 2; ++k) {
                            v[r][k] = add2(v[r][k], minus);
                            sum = fma2(v[r][k], v[r][k], sum);
                        }
                        if (!in) sum = before;
                    }
                }
                s[r] = pair_sum(sum);
            }
            team_sum<R>(s, team_log2, red, parity);
            TY *y = static_cast<TY *>(p.y) + (int64_t)(r0 + mine) * p.ldy + lane * CH;
            const int64_t out_step = (int64_t)teams * p.ldy;
#pragma unroll
            for (int r = 0; r < R; ++r, y += out_step) {
                const uint32_t at = r0 + r * teams + mine;
                const float rstd = rsqrtf(s[r] * inv + p.eps);
                if (at >= stop) continue;
                if (lane == 0) {
                    if (p.mean) p.mean[at] = mean[r];
                    if (p.rstd) p.rstd[at] = rstd;
                }
                const Pair scale = pair_of(rstd, rstd);
                float out[NV][CH];
#pragma unroll
                for (int k = 0; k < P; ++k)
                    pair_split(fma2(mul2(v[r][k], scale), f[k], b[k]), out[2 * k / CH][2 * k % CH],
                               out[(2 * k + 1) / CH][(2 * k + 1) % CH]);
#pragma unroll
                for (int j = 0; j < NV; ++j)
                    if ((uint32_t)(lane + j * team) * CH < p.cols) store_chunk<CH>(y + j * team * CH, out[j]);
            }
        }
        row = stop;
    }
    if constexpr (RING) ring_wait<0>();
}

// Floats of a row of dw or db in the workspace: a multiple of 16 bytes.
__host__ __device__ constexpr int64_t part_pitch(int64_t cols) { return (cols + 3) / 4 * 4; }

struct NormBwdParams {
    const void *dy, *x, *w;
    const float *mean, *rstd;
    void *dx;
    float *dw, *db, *part;      // part: [CTAs][2][2][part_pitch] (share, head or tail of it, dw or db)
    int64_t lddy, ldx, lddx, ldp, ldg;
    uint32_t rows, cols, share; // share: rows of a CTA
    int32_t by_group;           // layernorm_grad_kernel: a grid row is a group
    FastDiv group;
    int32_t team_log2, p_bf16, grad_wide;       // grad_wide: rows of dw and db take 16-byte stores
    float unit;
};

// dw and db of a group (or of a part of one) from the CTA's threads: teams of the CTA hold the same columns.
template <int CH, int NV, int T, bool ALONE>
__device__ __forceinline__ void flush_grads(const NormBwdParams &p, Pair (&sum_w)[NV * CH / 2], Pair (&sum_b)[NV * CH / 2],
                                            float *dw, float *db, bool wide, float *meet, int team_log2) {
    float aw[NV][CH], ab[NV][CH];
#pragma unroll
    for (int k = 0; k < NV * CH / 2; ++k) {
        pair_split(sum_w[k], aw[2 * k / CH][2 * k % CH], aw[(2 * k + 1) / CH][(2 * k + 1) % CH]);
        pair_split(sum_b[k], ab[2 * k / CH][2 * k % CH], ab[(2 * k + 1) / CH][(2 * k + 1) % CH]);
        sum_w[k] = sum_b[k] = 0;
    }
    const int team = 1 << team_log2, lane = threadIdx.x & (team - 1), teams = T >> team_log2;
    if constexpr (!ALONE) {
        const int stride = team * CH * NV, mine = threadIdx.x >> team_log2;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < CH * NV; ++i)
                meet[mine * stride + i * team + lane] = g ? ab[i / CH][i % CH] : aw[i / CH][i % CH];
            __syncthreads();
            if (mine == 0) {
#pragma unroll
                for (int i = 0; i < CH * NV; ++i) {
                    float s = 0.0f;
                    for (int k = 0; k < teams; ++k) s += meet[k * stride + i * team + lane];
                    (g ? ab[i / CH][i % CH] : aw[i / CH][i % CH]) = s;
                }
            }
        }
    }
    if (threadIdx.x < team) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const uint32_t c = (uint32_t)(lane + j * team) * CH;
            if (c >= p.cols) continue;
            if (CH > 1 && wide) {
                if (dw) store_chunk<CH>(dw + c, aw[j]);
                if (db) store_chunk<CH>(db + c, ab[j]);
            } else {
#pragma unroll
                for (int i = 0; i < CH; ++i) {
                    if (dw) dw[c + i] = aw[j][i];
                    if (db) db[c + i] = ab[j][i];
                }
            }
        }
    }
}

// Backward ring: stages of R rows of x and dy, up to three (eight of single rows) in about 200 KB; without two (rows
// above 8192 columns in fp32), and in narrow layouts (no copies of 8 bytes and more), rows are loaded straight into
// registers.
template <typename TX, typename TY, int CH, int NV, int R, int T>
struct BwdRing {
    static constexpr int kStage = R * NV * CH * (int)(sizeof(TX) + sizeof(TY)) * T;
    static constexpr int kFit = 200 * 1024 / kStage;
    static constexpr int kMost = R == 1 && T == 256 ? 8 : 3;
    static constexpr int kStages = CH == 1 || kFit < 2 ? 0 : kFit < kMost ? kFit : kMost;
    static constexpr int kBytes = kStages * kStage;
};

template <typename TX, typename TY, int CH, int NV, int R, int T, bool ALONE>
__global__ void __launch_bounds__(T, T == 256 ? 2 : 1) layernorm_bwd_kernel(const NormBwdParams p) {
    constexpr bool RING = BwdRing<TX, TY, CH, NV, R, T>::kStages > 0;
    constexpr int S = RING ? BwdRing<TX, TY, CH, NV, R, T>::kStages : 1, XB = CH * sizeof(TX), YB = CH * sizeof(TY);
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float red[2 * (T / 32) * 2 * R];
    __shared__ float meet[ALONE ? 1 : T * CH * NV];
    const int team_log2 = ALONE ? LOG2<T> : p.team_log2, team = 1 << team_log2;
    const int lane = threadIdx.x & (team - 1), mine = ALONE ? 0 : threadIdx.x >> team_log2;
    const uint32_t teams = T >> team_log2;
    const uint32_t begin = blockIdx.x * p.share, end = min(p.rows, begin + p.share);
    constexpr int E = NV * CH, P = E / 2;       // values of a row per thread, in pairs
    Pair aw[P], ab[P];
    int parity = 0;
    const float inv = 1.0f / (float)p.cols;
#pragma unroll
    for (int k = 0; k < P; ++k) aw[k] = ab[k] = 0;

    // the batches of the share in order: R * teams rows from fetch_row, inside the group that ends at fetch_stop
    uint32_t fetch_row = begin, fetch_stop = begin;
    const uint8_t *ring_x = smem + threadIdx.x * XB, *ring_y = smem + S * R * NV * T * XB + threadIdx.x * YB;
    const uint32_t at_x = smem_u32(ring_x), at_y = smem_u32(ring_y);
    const TX *from_x = static_cast<const TX *>(p.x) + (int64_t)mine * p.ldx + lane * CH;
    const TY *from_y = static_cast<const TY *>(p.dy) + (int64_t)mine * p.lddy + lane * CH;
    const int64_t step_x = (int64_t)teams * p.ldx, step_y = (int64_t)teams * p.lddy;
    auto fetch = [&](int stage) {
        if (fetch_row < end) {
            if (fetch_row >= fetch_stop)
                fetch_stop = (uint32_t)min((int64_t)end, ((int64_t)fdiv(fetch_row, p.group) + 1) * p.group.d);
            const TX *x = from_x + fetch_row * p.ldx;
            const TY *dy = from_y + fetch_row * p.lddy;
            const uint32_t to_x = at_x + stage * (R * NV * T * XB), to_y = at_y + stage * (R * NV * T * YB);
#pragma unroll
            for (int r = 0; r < R; ++r, x += step_x, dy += step_y) {
                const bool live = fetch_row + r * teams + mine < fetch_stop;
#pragma unroll
                for (int j = 0; j < NV; ++j) {
                    const bool in = live && (uint32_t)(lane + j * team) * CH < p.cols;
                    ring_load<RING ? XB : 16>(to_x + (r * NV + j) * T * XB, in ? x + j * team * CH : p.x, in);
                    ring_load<RING ? YB : 16>(to_y + (r * NV + j) * T * YB, in ? dy + j * team * CH : p.dy, in);
                }
            }
            fetch_row = min(fetch_row + R * teams, fetch_stop);
        }
        ring_commit();
    };
    // without a ring the next batch waits in registers
    TX next_x[RING ? 1 : R][RING ? 1 : E];
    TY next_y[RING ? 1 : R][RING ? 1 : E];
    auto fetch_registers = [&]() {
        if (fetch_row >= end) return;
        if (fetch_row >= fetch_stop)
            fetch_stop = (uint32_t)min((int64_t)end, ((int64_t)fdiv(fetch_row, p.group) + 1) * p.group.d);
        const TX *x = from_x + fetch_row * p.ldx;
        const TY *dy = from_y + fetch_row * p.lddy;
#pragma unroll
        for (int r = 0; r < (RING ? 0 : R); ++r, x += step_x, dy += step_y) {
            const bool live = fetch_row + r * teams + mine < fetch_stop;
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const bool in = live && (uint32_t)(lane + j * team) * CH < p.cols;
#pragma unroll
                for (int i = 0; i < CH; ++i) {
                    next_x[r][j * CH + i] = in ? x[j * team * CH + i] : (TX)0.0f;
                    next_y[r][j * CH + i] = in ? dy[j * team * CH + i] : (TY)0.0f;
                }
            }
        }
        fetch_row = min(fetch_row + R * teams, fetch_stop);
    };
    int stage = 0, last = S - 1;
    if constexpr (RING) {
#pragma unroll
        for (int k = 0; k < S - 1; ++k) fetch(k);
    } else {
        fetch_registers();
    }
    for (uint32_t row = begin; row < end;) {
        const uint32_t g = fdiv(row, p.group);
        const int64_t g0 = (int64_t)g * p.group.d, g1 = min(g0 + (int64_t)p.group.d, (int64_t)p.rows);
        const uint32_t stop = (uint32_t)min((int64_t)end, g1);
        Pair f[P];                              // u + w
        {
            float w[NV][CH];
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const uint32_t c = (uint32_t)(lane + j * team) * CH;
#pragma unroll
                for (int i = 0; i < CH; ++i) w[j][i] = 1.0f - p.unit;
                if (p.w && c < p.cols) load_param<CH>(p.w, p.p_bf16, (int64_t)g * p.ldp + c, w[j]);
            }
#pragma unroll
            for (int k = 0; k < P; ++k)
                f[k] = pair_of(p.unit + w[2 * k / CH][2 * k % CH], p.unit + w[(2 * k + 1) / CH][(2 * k + 1) % CH]);
        }
        for (uint32_t r0 = row; r0 < stop; r0 += teams * R) {
            float mean[R], rstd[R], s[2 * R];
            Pair xh[R][P], gy[R][P];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const uint32_t at = r0 + r * teams + mine;
                mean[r] = at < stop ? __ldg(p.mean + at) : 0.0f;
                rstd[r] = at < stop ? __ldg(p.rstd + at) : 0.0f;
            }
            if constexpr (RING) {
                fetch(last);
                ring_wait<S - 1>();
            }
#pragma unroll
            for (int r = 0; r < R; ++r) {
                float fx[NV][CH], fy[NV][CH];
#pragma unroll
                for (int j = 0; j < NV; ++j) {
                    if constexpr (RING) {
                        const int slot = (stage * R + r) * NV + j;
                        load_chunk<CH>(reinterpret_cast<const TX *>(ring_x + slot * T * XB), fx[j]);
                        load_chunk<CH>(reinterpret_cast<const TY *>(ring_y + slot * T * YB), fy[j]);
                    } else {
#pragma unroll
                        for (int i = 0; i < CH; ++i) {
                            fx[j][i] = (float)next_x[r][j * CH + i];
                            fy[j][i] = (float)next_y[r][j * CH + i];
                        }
                    }
                }
#pragma unroll
                for (int k = 0; k < P; ++k) {
                    xh[r][k] = pair_of(fx[2 * k / CH][2 * k % CH], fx[(2 * k + 1) / CH][(2 * k + 1) % CH]);
                    gy[r][k] = pair_of(fy[2 * k / CH][2 * k % CH], fy[(2 * k + 1) / CH][(2 * k + 1) % CH]);
                }
            }
            if constexpr (!RING) fetch_registers();
            last = stage;
            stage = stage + 1 == S ? 0 : stage + 1;
            // rows past the group have dy = mean = rstd = 0 and add nothing.  Columns past the row have dy = 0, but x = 0 too,
            // whose xhat, -mean rstd, can overflow where every xhat of the row is small: it stays out of the second sum (odd
            // widths, whose pairs can end inside the row, take the mean for x)
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const Pair minus = pair_of(-mean[r], -mean[r]), scale = pair_of(rstd[r], rstd[r]);
                Pair s1 = 0, s2 = 0;
#pragma unroll
                for (int j = 0; j < NV; ++j) {
                    const bool in = (uint32_t)(lane + j * team) * CH < p.cols;
                    if constexpr (CH == 1) {    // a pair is two chunks
                        if (!in) {
                            float lo, hi;
                            pair_split(xh[r][j / 2], lo, hi);
                            (j & 1 ? hi : lo) = mean[r];
                            xh[r][j / 2] = pair_of(lo, hi);
                        }
                        if ((j & 1) == 0) continue;
                    }
                    const Pair before = s2;
#pragma unroll
                    for (int k = CH == 1 ? j / 2 : j * CH / 2; k < (j + 1) * CH / 2; ++k) {
                        const Pair xv = mul2(add2(xh[r][k], minus), scale), d = gy[r][k], gv = mul2(d, f[k]);
                        aw[k] = fma2(d, xv, aw[k]);
                        ab[k] = add2(ab[k], d);
                        s1 = add2(s1, gv);
                        s2 = fma2(gv, xv, s2);
                        xh[r][k] = xv;
                        gy[r][k] = gv;
                    }
                    if (CH > 1 && !in) s2 = before;
                }
                s[2 * r] = pair_sum(s1);
                s[2 * r + 1] = pair_sum(s2);
            }
            if (!p.dx) continue;
            team_sum<2 * R>(s, team_log2, red, parity);
            TX *dx = static_cast<TX *>(p.dx) + (int64_t)(r0 + mine) * p.lddx + lane * CH;
            const int64_t out_step = (int64_t)teams * p.lddx;
#pragma unroll
            for (int r = 0; r < R; ++r, dx += out_step) {
                if (r0 + r * teams + mine >= stop) continue;
                const float m1 = s[2 * r] * inv, m2 = s[2 * r + 1] * inv;
                const Pair minus1 = pair_of(-m1, -m1), minus2 = pair_of(-m2, -m2), scale = pair_of(rstd[r], rstd[r]);
                float out[NV][CH];
#pragma unroll
                for (int k = 0; k < P; ++k)
                    pair_split(mul2(scale, fma2(xh[r][k], minus2, add2(gy[r][k], minus1))), out[2 * k / CH][2 * k % CH],
                               out[(2 * k + 1) / CH][(2 * k + 1) % CH]);
#pragma unroll
                for (int j = 0; j < NV; ++j)
                    if ((uint32_t)(lane + j * team) * CH < p.cols) store_chunk<CH>(dx + j * team * CH, out[j]);
            }
        }
        if (p.dw || p.db) {
            float *dw, *db;
            bool wide = true;
            if (g0 >= begin && g1 <= end) {
                dw = p.dw ? p.dw + (int64_t)g * p.ldg : nullptr;
                db = p.db ? p.db + (int64_t)g * p.ldg : nullptr;
                wide = p.grad_wide;
            } else {            // slot 0: the group began in an earlier share, 1: it goes on in a later one
                dw = p.part + ((int64_t)blockIdx.x * 2 + (g0 < begin ? 0 : 1)) * 2 * part_pitch(p.cols);
                db = dw + part_pitch(p.cols);
            }
            flush_grads<CH, NV, T, ALONE>(p, aw, ab, dw, db, wide, meet, team_log2);
        }
        row = stop;
    }
    if constexpr (RING) ring_wait<0>();
}

// Groups that several shares hold.  Row y of the grid is group y, or with more groups than shares the group
// that begins in share y and goes on behind it, if there is one.  128 columns of dw or of db a CTA, ROWS shares
// at a time.
template <int ROWS>
__global__ void __launch_bounds__(32 * ROWS) layernorm_grad_kernel(const NormBwdParams p) {
    __shared__ float4 red[ROWS][32];
    griddep_wait();
    const int64_t g = p.by_group ? blockIdx.y : fdiv((uint32_t)min((int64_t)p.rows, ((int64_t)blockIdx.y + 1) * p.share) - 1, p.group);
    const int64_t g0 = g * p.group.d, g1 = min(g0 + (int64_t)p.group.d, (int64_t)p.rows);
    const int64_t first = g0 / p.share, final = (g1 - 1) / p.share, pitch = part_pitch(p.cols);
    if (first == final || (!p.by_group && first != blockIdx.y)) return;
    const int lane = threadIdx.x & 31, k = threadIdx.x >> 5;
    const int64_t at = (int64_t)blockIdx.x * 128 + lane * 4;            // 0 .. 2 pitch - 1: dw then db
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (at < 2 * pitch) {
        const float *part = p.part + at;
#pragma unroll 4
        for (int64_t b = first + k; b <= final; b += ROWS) {
            const float4 v = *reinterpret_cast<const float4 *>(part + (b * 2 + (b == first ? 1 : 0)) * 2 * pitch);
            s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
        }
    }
    red[k][lane] = s;
    __syncthreads();
    if (k != 0 || at >= 2 * pitch) return;
#pragma unroll
    for (int i = 1; i < ROWS; ++i) {
        const float4 v = red[i][lane];
        s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
    }
    const int64_t col = at < pitch ? at : at - pitch;
    float *out = at < pitch ? p.dw : p.db;
    if (!out) return;
    out += g * p.ldg + col;
    const float v[4] = {s.x, s.y, s.z, s.w};
    if (p.grad_wide && col + 4 <= p.cols)
        store_chunk<4>(out, v);
    else
        for (int i = 0; i < 4 && col + i < p.cols; ++i) out[i] = v[i];
}

// ------------------------------------------------------------------------------------------------
// host
// ------------------------------------------------------------------------------------------------

static bool dtype_ok(int t) { return t == NOMAS_DTYPE_F32 || t == NOMAS_DTYPE_BF16; }
static int dtype_size(int t) { return t == NOMAS_DTYPE_BF16 ? 2 : 4; }

// A matrix operand: element aligned, pitch at least the row.
static bool matrix_ok(const void *p, int64_t cols, int64_t ld, int dtype) {
    return p && reinterpret_cast<uintptr_t>(p) % dtype_size(dtype) == 0 && ld >= cols;
}
static bool wide_ok(const void *p, int64_t ld) { return !p || (aligned16(p) && ld % 8 == 0); }

static int check_norm(int64_t rows, int64_t cols, int64_t rows_per_group) {
    if (rows < 0 || cols < 1 || rows_per_group < 0) return NOMAS_EINVAL;
    if (cols > NOMAS_NORM_MAX_COLS || rows >= (int64_t)1 << 31) return NOMAS_EUNSUPPORTED;
    return NOMAS_OK;
}

// Rows of a group as a divisor below 2^31 (one group: any divisor above the last row).
static FastDiv group_div(int64_t rows, int64_t rows_per_group) {
    const int64_t most = ((int64_t)1 << 31) - 1;
    const int64_t d = rows_per_group == 0 ? rows : rows_per_group;
    return make_fastdiv((uint32_t)(d < 1 ? 1 : d > most ? most : d));
}

static int log2_at_least(int64_t v) {
    int l = 0;
    while (((int64_t)1 << l) < v) ++l;
    return l;
}

// Threads of a team (log2) for `chunks` chunks of a row, at most `per` of them a thread and 2^most threads:
// whole warps as soon as a row fills one.
static int team_of(int64_t chunks, int per, int most) {
    int l = log2_at_least((chunks + per - 1) / per);
    const int full = log2_at_least(chunks);
    if (l < 5) l = full < 5 ? full : 5;
    return l > most ? most : l;
}

// Dynamic shared memory above 48 KB has to be allowed per kernel and device: once for the largest size asked for.
struct SmemAllowed {
    std::atomic<int> bytes[64] = {};
    int operator()(const void *kernel, int want) {
        if (want <= 32 * 1024) return NOMAS_OK;       // with up to 16 KB of static shared memory
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e == cudaSuccess && dev >= 0 && dev < 64 && bytes[dev].load() >= want) return NOMAS_OK;
        if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, want);
        if (e != cudaSuccess) return cuda_fail("cudaFuncSetAttribute(layer norm smem)", (int)e, cudaGetErrorString(e));
        int had = dev < 64 ? bytes[dev].load() : want;
        while (had < want && !bytes[dev].compare_exchange_weak(had, want)) {
        }
        return NOMAS_OK;
    }
};

template <typename TX, typename TY, int CH, int NV>
static int launch_row(const NormParams &p, cudaStream_t st) {
    const int64_t threads = (int64_t)p.rows << p.team_log2;
    layernorm_row_kernel<TX, TY, CH, NV>
        <<<(unsigned)((threads + kNormThreads - 1) / kNormThreads), kNormThreads, 0, st>>>(p);
    return check_launch("layernorm_row_kernel launch");
}

// The row's loads spread over as many threads as a CTA has.  Narrow rows above 4096 columns spill about 320 bytes a thread.
template <typename TX, typename TY, int CH>
static int pick_row(NormParams &p, cudaStream_t st) {
    const int64_t chunks = (p.cols + CH - 1) / CH;
    p.team_log2 = team_of(chunks, 1, 8);
    const int64_t nv = (chunks + (1 << p.team_log2) - 1) >> p.team_log2;
    if (nv <= 1) return launch_row<TX, TY, CH, 1>(p, st);
    if (nv <= 4) return launch_row<TX, TY, CH, 4>(p, st);
    if (nv <= 8 || CH == 8) return launch_row<TX, TY, CH, 8>(p, st);
    if constexpr (CH < 8) {
        if (nv <= 16 || CH == 4) return launch_row<TX, TY, CH, 16>(p, st);
    }
    if constexpr (CH == 1) return launch_row<TX, TY, CH, 64>(p, st);
    return NOMAS_EUNSUPPORTED;                  // not reached: 16384 columns are 16 chunks of 4, 8 of 8
}

template <typename TX, typename TY, int CH, int NV, int R, int T, bool ALONE>
static int launch_fwd(NormParams &p, cudaStream_t st) {
    constexpr int kBytes = FwdRing<TX, CH, NV, R, T>::kBytes;
    auto kernel = layernorm_fwd_kernel<TX, TY, CH, NV, R, T, ALONE>;
    static SmemAllowed allowed;
    const int rc = allowed(reinterpret_cast<const void *>(kernel), kBytes);
    if (rc) return rc;
    const int64_t teams = T >> p.team_log2, ctas = (int64_t)sm_count() * (T == 512 ? 1 : CH == 1 || kBytes > 74 * 1024 ? 2 : 3);
    int64_t share = (p.rows + ctas - 1) / ctas;
    if (share < teams) share = teams;
    p.share = (uint32_t)share;
    kernel<<<(unsigned)((p.rows + share - 1) / share), T, kBytes, st>>>(p);
    return check_launch("layernorm_fwd_kernel launch");
}

// Values of a row per thread: 8 with 4 rows at a time, 16 with 2, then teams of 512 threads.  Narrow layouts hold the
// next rows in registers and take fewer rows at a time (26400 x 3581 in bf16: 125 us, its bytes 58); above 8192 columns
// these spill 64 to 140 bytes a thread.
template <typename TX, typename TY, int CH>
static int pick_fwd(NormParams &p, cudaStream_t st) {
    const int64_t chunks = (p.cols + CH - 1) / CH;
    constexpr int kLeast = CH == 1 ? 2 : 1;     // pairs of values
    p.team_log2 = team_of(chunks, kLeast, 8);
    if (chunks <= kLeast * 128) return launch_fwd<TX, TY, CH, kLeast, 4, 256, false>(p, st);
    if (chunks <= kLeast * 256) return launch_fwd<TX, TY, CH, kLeast, 4, 256, true>(p, st);
    if constexpr (CH == 1) {
        if (p.cols <= 2048) return launch_fwd<TX, TY, 1, 8, 2, 256, true>(p, st);
        p.team_log2 = 9;
        if (p.cols <= 4096) return launch_fwd<TX, TY, 1, 8, 2, 512, true>(p, st);
        if (p.cols <= 8192) return launch_fwd<TX, TY, 1, 16, 1, 512, true>(p, st);
        return launch_fwd<TX, TY, 1, 32, 1, 512, true>(p, st);
    } else {
        if (p.cols <= 2048) return launch_fwd<TX, TY, CH, 8 / CH, 4, 256, true>(p, st);
        if (p.cols <= 4096) return launch_fwd<TX, TY, CH, 16 / CH, 2, 256, true>(p, st);
        p.team_log2 = 9;
        if (p.cols <= 8192) return launch_fwd<TX, TY, CH, 16 / CH, 2, 512, true>(p, st);
        return launch_fwd<TX, TY, CH, 32 / CH, 1, 512, true>(p, st);
    }
}

template <typename TX, typename TY, int CH>
static int row_or_share(NormParams &p, cudaStream_t st) {
    // few rows: latency, not bandwidth.  Groups of few rows: a share would wait for each group's parameters and leave
    // most of its rows' places empty (26400 x 1024 in groups of one row: 188 us by shares)
    const int64_t chunks = (p.cols + CH - 1) / CH, teams = chunks >= kNormThreads ? 1 : kNormThreads / chunks;
    const bool few = p.rows <= (uint32_t)(2 * sm_count()) || p.group.d < 4 * teams;
    return few ? pick_row<TX, TY, CH>(p, st) : pick_fwd<TX, TY, CH>(p, st);
}

template <typename TX, typename TY>
static int any_fwd(NormParams &p, bool wide, cudaStream_t st) {
    constexpr int CH = sizeof(TX) == 2 && sizeof(TY) == 2 ? 8 : 4;     // 16 bytes of the wider type
    return wide ? row_or_share<TX, TY, CH>(p, st) : row_or_share<TX, TY, 1>(p, st);
}

// Shares of the backward pass: `per_sm` CTAs an SM, each with at least a round of rows.  The device holds as many at once,
// but for rows of more than 1024 columns with an fp32 side, whose ring leaves an SM one CTA of the two (13200 x 2048 in
// fp32: 61 us, 5.3 TB/s, as in bf16).
static void bwd_shares(int64_t rows, int64_t cols, int per_sm, int64_t *share, int64_t *ctas) {
    // small ones: a single share needs no second launch
    const int64_t most = per_sm * (int64_t)sm_count(), least = rows * cols <= 32768 ? rows : cols <= 512 ? 16 : 4;
    int64_t s = (rows + most - 1) / most;
    if (s < least) s = least;
    *share = s < 1 ? 1 : s;
    *ctas = (rows + *share - 1) / *share;
}

template <typename TX, typename TY, int CH, int NV, int R, int T, bool ALONE>
static int launch_bwd(NormBwdParams &p, int64_t ctas, cudaStream_t st) {
    constexpr int kBytes = BwdRing<TX, TY, CH, NV, R, T>::kBytes;
    auto kernel = layernorm_bwd_kernel<TX, TY, CH, NV, R, T, ALONE>;
    static SmemAllowed allowed;
    int rc = allowed(reinterpret_cast<const void *>(kernel), kBytes);
    if (rc) return rc;
    kernel<<<(unsigned)ctas, T, kBytes, st>>>(p);
    rc = check_launch("layernorm_bwd_kernel launch");
    if (rc || ctas == 1 || (!p.dw && !p.db)) return rc;
    const int64_t groups = ((int64_t)p.rows + p.group.d - 1) / p.group.d;
    p.by_group = groups < ctas;
    const dim3 grid((unsigned)((2 * part_pitch(p.cols) + 127) / 128), (unsigned)(p.by_group ? groups : ctas - 1));
    // a group's shares: as many rows of threads as give each a few to add
    const int64_t shares = p.group.d / p.share + 2 < ctas ? p.group.d / p.share + 2 : ctas;
    const bool many = shares > 64;
    const cudaError_t e = launch_pdl(many ? layernorm_grad_kernel<32> : layernorm_grad_kernel<8>, grid,
                                     dim3(many ? 1024 : 256), 0, st, p);
    return e == cudaSuccess ? NOMAS_OK : cuda_fail("layernorm_grad_kernel launch", (int)e, cudaGetErrorString(e));
}

// Values of a row per thread: 8 with 4 rows at a time, 16 with 2, then teams of 512 threads.  Narrow layouts hold the
// next rows in registers and take half as many values.  Above 8192 columns a thread's 32 values of u + w, x, dy, dw and db
// do not fit 128 registers and spill, 0.5 to 0.6 KB a thread with a ring and up to 2.7 without: 1000 x 16384 takes 51 us in
// bf16 (its bytes 15) and 161 in fp32 (30).
template <typename TX, typename TY, int CH>
static int pick_bwd(NormBwdParams &p, int64_t ctas, cudaStream_t st) {
    const int64_t chunks = (p.cols + CH - 1) / CH;
    constexpr int kLeast = CH == 1 ? 2 : 1;     // pairs of values
    p.team_log2 = team_of(chunks, kLeast, 8);
    // groups of few rows: batches stay inside a group, so one row of a team at a time
    const bool small = p.group.d <= 2 * (kNormThreads >> p.team_log2);
    if (chunks <= kLeast * 128)
        return small ? launch_bwd<TX, TY, CH, kLeast, 1, 256, false>(p, ctas, st) : launch_bwd<TX, TY, CH, kLeast, 4, 256, false>(p, ctas, st);
    if (chunks <= kLeast * 256)
        return small ? launch_bwd<TX, TY, CH, kLeast, 1, 256, true>(p, ctas, st) : launch_bwd<TX, TY, CH, kLeast, 4, 256, true>(p, ctas, st);
    if constexpr (CH == 1) {
        if (p.cols <= 2048) return launch_bwd<TX, TY, 1, 8, 1, 256, true>(p, ctas, st);
        p.team_log2 = 9;
        if (p.cols <= 4096) return launch_bwd<TX, TY, 1, 8, 2, 512, true>(p, ctas, st);
    } else {
        if (p.cols <= 2048) return launch_bwd<TX, TY, CH, 8 / CH, 4, 256, true>(p, ctas, st);
        if (p.cols <= 4096) return launch_bwd<TX, TY, CH, 16 / CH, 2, 256, true>(p, ctas, st);
        p.team_log2 = 9;
    }
    if (p.cols <= 8192) return launch_bwd<TX, TY, CH, 16 / CH, 1, 512, true>(p, ctas, st);
    return launch_bwd<TX, TY, CH, 32 / CH, 1, 512, true>(p, ctas, st);
}

template <typename TX, typename TY>
static int any_bwd(NormBwdParams &p, bool wide, int64_t ctas, cudaStream_t st) {
    constexpr int CH = sizeof(TX) == 2 && sizeof(TY) == 2 ? 8 : 4;
    return wide ? pick_bwd<TX, TY, CH>(p, ctas, st) : pick_bwd<TX, TY, 1>(p, ctas, st);
}

}  // namespace nomas

using namespace nomas;

extern "C" int nomas_layernorm_fwd(const void *x, int64_t rows, int64_t cols, int64_t ldx, int x_dtype, const void *w,
                                   const void *b, int64_t ldp, int p_dtype, int64_t rows_per_group, int unit_offset,
                                   float eps, void *y, int64_t ldy, int y_dtype, float *mean, float *rstd,
                                   nomas_stream stream) {
    if (!dtype_ok(x_dtype) || !dtype_ok(y_dtype) || !dtype_ok(p_dtype)) return NOMAS_EINVAL;
    int rc = check_norm(rows, cols, rows_per_group);
    if (rc) return rc;
    if (!matrix_ok(x, cols, ldx, x_dtype) || !matrix_ok(y, cols, ldy, y_dtype) || !(eps >= 0.0f)) return NOMAS_EINVAL;
    if ((w && !matrix_ok(w, cols, ldp, p_dtype)) || (b && !matrix_ok(b, cols, ldp, p_dtype))) return NOMAS_EINVAL;
    if (reinterpret_cast<uintptr_t>(mean) % 4 != 0 || reinterpret_cast<uintptr_t>(rstd) % 4 != 0) return NOMAS_EINVAL;
    if (x == y && (ldx != ldy || x_dtype != y_dtype)) return NOMAS_EINVAL;
    if (rows == 0) return NOMAS_OK;
    NormParams p{};
    p.x = x, p.w = w, p.b = b, p.y = y, p.mean = mean, p.rstd = rstd;
    p.ldx = ldx, p.ldy = ldy, p.ldp = ldp;
    p.rows = (uint32_t)rows, p.cols = (uint32_t)cols;
    p.group = group_div(rows, rows_per_group);
    p.p_bf16 = p_dtype == NOMAS_DTYPE_BF16;
    p.unit = unit_offset && w ? 1.0f : 0.0f;
    p.eps = eps;
    const bool wide = cols % 8 == 0 && wide_ok(x, ldx) && wide_ok(y, ldy) && wide_ok(w, ldp) && wide_ok(b, ldp);
    DeviceScope dev(x);
    if (dev.rc) return dev.rc;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (x_dtype == NOMAS_DTYPE_BF16)
        return y_dtype == NOMAS_DTYPE_BF16 ? any_fwd<__nv_bfloat16, __nv_bfloat16>(p, wide, st)
                                           : any_fwd<__nv_bfloat16, float>(p, wide, st);
    return y_dtype == NOMAS_DTYPE_BF16 ? any_fwd<float, __nv_bfloat16>(p, wide, st)
                                       : any_fwd<float, float>(p, wide, st);
}

extern "C" size_t nomas_layernorm_workspace_bytes(int64_t rows, int64_t cols, int64_t rows_per_group) {
    if (check_norm(rows, cols, rows_per_group)) return 0;
    int64_t share, ctas;
    bwd_shares(rows, cols, 2, &share, &ctas);
    const size_t n = ctas > 1 ? (size_t)ctas * 4 * (size_t)part_pitch(cols) * sizeof(float) : 0;
    return n < 16 ? 16 : n;
}

extern "C" int nomas_layernorm_bwd(const void *dy, int64_t lddy, int y_dtype, const void *x, int64_t ldx, int x_dtype,
                                   int64_t rows, int64_t cols, const void *w, int64_t ldp, int p_dtype,
                                   int64_t rows_per_group, int unit_offset, const float *mean, const float *rstd,
                                   void *dx, int64_t lddx, float *dw, float *db, int64_t ldg, void *workspace,
                                   nomas_stream stream) {
    if (!dtype_ok(x_dtype) || !dtype_ok(y_dtype) || !dtype_ok(p_dtype)) return NOMAS_EINVAL;
    int rc = check_norm(rows, cols, rows_per_group);
    if (rc) return rc;
    if (!matrix_ok(dy, cols, lddy, y_dtype) || !matrix_ok(x, cols, ldx, x_dtype) || !mean || !rstd) return NOMAS_EINVAL;
    if (reinterpret_cast<uintptr_t>(mean) % 4 != 0 || reinterpret_cast<uintptr_t>(rstd) % 4 != 0) return NOMAS_EINVAL;
    if (!dx && !dw && !db) return NOMAS_EINVAL;
    if ((w && !matrix_ok(w, cols, ldp, p_dtype)) || (dx && !matrix_ok(dx, cols, lddx, x_dtype))) return NOMAS_EINVAL;
    if ((dw && !matrix_ok(dw, cols, ldg, NOMAS_DTYPE_F32)) || (db && !matrix_ok(db, cols, ldg, NOMAS_DTYPE_F32)))
        return NOMAS_EINVAL;
    if (dx && ((dx == x && lddx != ldx) || (dx == dy && (lddx != lddy || x_dtype != y_dtype)))) return NOMAS_EINVAL;
    if ((dw || db) && (workspace ? !aligned16(workspace) : nomas_layernorm_workspace_bytes(rows, cols, rows_per_group) > 16))
        return NOMAS_EINVAL;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    DeviceScope dev(x);
    if (dev.rc) return dev.rc;
    if (rows == 0) {
        for (float *out : {dw, db}) {
            if (!out || rows_per_group != 0) continue;
            const cudaError_t e = cudaMemsetAsync(out, 0, (size_t)cols * sizeof(float), st);
            if (e != cudaSuccess) return cuda_fail("cudaMemsetAsync", (int)e, cudaGetErrorString(e));
        }
        return NOMAS_OK;
    }
    NormBwdParams p{};
    const bool wide = cols % 8 == 0 && wide_ok(dy, lddy) && wide_ok(x, ldx) && wide_ok(w, ldp) && wide_ok(dx, lddx);
    int64_t share, ctas;
    bwd_shares(rows, cols, cols > (wide ? 4096 : 2048) ? 1 : 2, &share, &ctas);    // 512 threads: one CTA an SM
    p.dy = dy, p.x = x, p.w = w, p.mean = mean, p.rstd = rstd, p.dx = dx, p.dw = dw, p.db = db;
    p.part = static_cast<float *>(workspace);
    p.lddy = lddy, p.ldx = ldx, p.lddx = lddx, p.ldp = ldp, p.ldg = ldg;
    p.rows = (uint32_t)rows, p.cols = (uint32_t)cols, p.share = (uint32_t)share;
    p.group = group_div(rows, rows_per_group);
    p.p_bf16 = p_dtype == NOMAS_DTYPE_BF16;
    p.unit = unit_offset && w ? 1.0f : 0.0f;
    p.grad_wide = wide_ok(dw, ldg) && wide_ok(db, ldg);
    if (x_dtype == NOMAS_DTYPE_BF16)
        return y_dtype == NOMAS_DTYPE_BF16 ? any_bwd<__nv_bfloat16, __nv_bfloat16>(p, wide, ctas, st)
                                           : any_bwd<__nv_bfloat16, float>(p, wide, ctas, st);
    return y_dtype == NOMAS_DTYPE_BF16 ? any_bwd<float, __nv_bfloat16>(p, wide, ctas, st)
                                       : any_bwd<float, float>(p, wide, ctas, st);
}
