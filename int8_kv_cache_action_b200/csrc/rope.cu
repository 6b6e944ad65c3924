// Rotary positions with several axes (definition in nomas.h): the elementwise step between the QKV
// projection and the append / attention.
//
// A call reads and writes every value once and is bound by HBM: 3 flops a value against 2 x 2 bytes.
// What a token's heads share is its D / 2 sines and cosines, so a CTA takes all heads (or 512 chunks of them) of some
// tokens, issues its first loads, computes the tokens' table while they are in flight and reads it from shared memory.
// No table in global memory, so nothing to keep between calls.  A thread keeps its chunk of its head from token to
// token, so that an item costs little more than its arithmetic (one head of 26400 tokens 14 us; 22 with the chunk, head
// and tensor worked out per item, about 100 instructions each).  26400 tokens of q and k of 16 x 128 in bf16: 81 us,
// 5.3 TB/s; a copy of this pattern reaches 5.5 to 5.8.
#include <cmath>
#include <cstring>

#include "common.cuh"

namespace nomas {

constexpr int kRopeThreads = 256;
constexpr int kRopeTable = 4096;               // (cos, sin) entries of a CTA's tokens: 32 KB
constexpr int kRopeMaxPairs = NOMAS_ROPE_MAX_HEAD_DIM / 2;

// How a pair's values are reached: in one 16-byte chunk (interleaved), in two chunks that the same thread holds (halves,
// where every axis' half is whole chunks of 16, or in bf16 of 8 bytes), or one by one (halves of other widths:
// rope_pairs_kernel).  26400 tokens of 2 x 16 x 128 in bf16, halves: chunks of 16 bytes (axes 32, 48, 48) 83 us, of 8
// (16, 56, 56) 76, one by one (44, 42, 42) 111, which is also what 16, 56, 56 took one by one.  The rule goes by alignment;
// the chunks of 16 bytes with two items a thread spill 28 to 32 bytes a thread, those of 8 none.
enum RopeForm { kRopeInside = 0, kRopeTwoChunks = 1, kRopePairs = 2 };

struct RopeTensor {
    const char *x;
    char *y;
    int64_t x_tok, x_head, y_tok, y_head;      // bytes
    uint32_t first_item, first_row;            // items and rows (heads) of a token in front of this tensor's
};

// What a pair's angle in turns is made of: for the grid the turns at index 0 and per index, in 2^-64, whose overflow
// drops whole turns exactly; for given positions `origin` holds the bits of the fp64 turns per unit.
struct __align__(16) RopePair {
    int64_t origin, step;
};

struct RopeParams {
    RopePair pair[kRopeMaxPairs];
    RopeTensor t[NOMAS_ROPE_MAX_TENSORS];
    const float *positions;                    // or null: the grid
    FastDiv plane, width;                      // grid_h * grid_w, grid_w
    FastDiv items;                             // items of a token, all tensors (rope_pairs_kernel: its warps a token)
    FastDiv per_head;                          // items of a head
    FastDiv per_token;                         // pairs of a head (all_pairs)
    uint32_t tokens, tokens_per_cta;
    uint32_t abreast;                          // tokens that the CTA's threads hold side by side
    uint32_t all_rows, rows_per_warp, warp_items;      // rope_pairs_kernel: rows of a token, of a warp; (token, rows) items
    int32_t n_tensors, inverse;
    int32_t axis_at[4];                        // first channel of each axis, end of the last
    int32_t pairs, all_pairs;                  // pairs that turn, head_dim / 2
};

// V values of T in one access.
template <int BYTES>
struct ChunkOf;
template <>
struct ChunkOf<16> {
    typedef uint4 type;
};
template <>
struct ChunkOf<8> {
    typedef uint2 type;
};
template <typename T, int V>
using Chunk = typename ChunkOf<V * (int)sizeof(T)>::type;

__device__ __forceinline__ void unpack(const uint4 &c, float (&v)[8]) {
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void unpack(const uint4 &c, float (&v)[4]) {
    v[0] = __uint_as_float(c.x), v[1] = __uint_as_float(c.y), v[2] = __uint_as_float(c.z), v[3] = __uint_as_float(c.w);
}
__device__ __forceinline__ void unpack(const uint2 &c, float (&v)[4]) {
    v[0] = __uint_as_float(c.x << 16), v[1] = __uint_as_float(c.x & 0xFFFF0000u);
    v[2] = __uint_as_float(c.y << 16), v[3] = __uint_as_float(c.y & 0xFFFF0000u);
}
__device__ __forceinline__ void pack(const float (&v)[8], uint4 &c) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&b);
    }
    c = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void pack(const float (&v)[4], uint4 &c) {
    c = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
}
__device__ __forceinline__ void pack(const float (&v)[4], uint2 &c) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
    c = make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
}

// The rotated chunk with the words behind its first `turned` channels as they were: channels that no axis
// holds keep every bit (a conversion would change a NaN's).
template <int V>
__device__ __forceinline__ uint4 keep_behind(uint4 out, const uint4 &in, int turned) {
    constexpr int per_word = V / 4;
    if (turned <= 0 * per_word) out.x = in.x;
    if (turned <= 1 * per_word) out.y = in.y;
    if (turned <= 2 * per_word) out.z = in.z;
    if (turned <= 3 * per_word) out.w = in.w;
    return out;
}

// First channel of item j in the two-chunk form, and how far its second chunk is: item j holds pairs
// j V .. j V + V - 1, whose axis starts at channel axis_at[a] = 2 x (pairs in front of it).  Behind the axes
// the item is two neighbouring chunks that pass through.
template <uint32_t V>
__device__ __forceinline__ void rope_two(const RopeParams &p, uint32_t j, uint32_t &c, uint32_t &apart) {
    const uint32_t ch = 2 * V * j;
    apart = V;
    c = ch;
#pragma unroll
    for (int a = 0; a < 3; ++a) {
        const uint32_t s = p.axis_at[a], e = p.axis_at[a + 1];
        if (ch >= s && ch < e) {
            apart = (e - s) / 2;
            c = s + (ch - s) / 2;
        }
    }
}

// Lanes hold different pairs, and reading the call's arguments by lane takes one access a lane: it is done once a CTA
// or warp, never once a token (26400 tokens of one head: 34 us when it was, 12 us).
__device__ __forceinline__ int rope_axis(const RopeParams &p, int i) {
    return 2 * i < p.axis_at[1] ? 0 : 2 * i < p.axis_at[2] ? 1 : 2;
}

// (cos, sin) of a pair at a token, sin negated for the inverse.  What is left of the angle after its whole turns are
// dropped keeps fp32's relative precision.
__device__ __forceinline__ float2 rope_angle(const RopeParams &p, const RopePair &r, int axis, uint32_t token) {
    float half_turns;
    if (p.positions) {
        const double turns = (double)__ldg(p.positions + 3 * (int64_t)token + axis) * __longlong_as_double(r.origin);
        half_turns = 2.0f * (float)(turns - rint(turns));
    } else {
        const uint32_t f = fdiv(token, p.plane), in = token - f * p.plane.d;
        const uint32_t row = fdiv(in, p.width), col = in - row * p.width.d;
        const uint64_t at = (uint64_t)r.origin + (uint64_t)r.step * (axis == 0 ? f : axis == 1 ? row : col);
        half_turns = (float)(int64_t)at * 0x1p-63f;
    }
    float s, c;
    sincospif(half_turns, &s, &c);
    return make_float2(c, p.inverse ? -s : s);
}

__device__ __forceinline__ void turn(float &a, float &b, const float2 &cs) {
    const float x = a, y = b;
    a = fmaf(x, cs.x, -(y * cs.y));
    b = fmaf(x, cs.y, y * cs.x);
}

// NS items of a token per thread: one while a token has no more items than the CTA threads (then `abreast` tokens side
// by side), else two, 256 apart, of the 512 that blockIdx.y names.
template <typename T, int V, int FORM, int NS>
__global__ void __launch_bounds__(kRopeThreads, 4) rope_kernel(const __grid_constant__ RopeParams p) {
    typedef Chunk<T, V> C;
    constexpr int U = 4 / NS;                  // tokens in flight
    __shared__ __align__(16) float2 table[kRopeTable];
    __shared__ RopePair pairs[kRopeMaxPairs];
    for (int i = threadIdx.x; i < p.pairs; i += blockDim.x) pairs[i] = p.pair[i];

    const uint32_t token0 = blockIdx.x * p.tokens_per_cta, n = min(p.tokens_per_cta, p.tokens - token0);
    const uint32_t side = NS == 1 ? fdiv(threadIdx.x, p.items) : 0;
    const char *x[NS];
    char *y[NS];
    int64_t x_step[NS], y_step[NS];
    uint32_t apart[NS];                        // bytes to an item's second chunk
    int pair0[NS];                             // its first pair
    bool live[NS];
#pragma unroll
    for (int s = 0; s < NS; ++s) {
        const uint32_t it = NS == 1 ? threadIdx.x - side * p.items.d : blockIdx.y * 512 + s * 256 + threadIdx.x;
        live[s] = NS == 1 ? side < p.abreast : it < p.items.d;
        int k = 0;
#pragma unroll
        for (int i = 1; i < NOMAS_ROPE_MAX_TENSORS; ++i)
            if (i < p.n_tensors && it >= p.t[i].first_item) k = i;
        const RopeTensor &t = p.t[k];
        const uint32_t in = it - t.first_item, head = fdiv(in, p.per_head), j = in - head * p.per_head.d;
        uint32_t c = j * V, gap = 0;
        if constexpr (FORM == kRopeTwoChunks) rope_two<V>(p, j, c, gap);
        apart[s] = gap * sizeof(T);
        pair0[s] = j * (FORM == kRopeTwoChunks ? V : V / 2);
        const int64_t tok = (int64_t)token0 + side;
        x[s] = t.x + tok * t.x_tok + (int64_t)head * t.x_head + c * sizeof(T);
        y[s] = t.y + tok * t.y_tok + (int64_t)head * t.y_head + c * sizeof(T);
        x_step[s] = t.x_tok * p.abreast;
        y_step[s] = t.y_tok * p.abreast;
    }
    for (uint32_t at = 0; at < n; at += U * p.abreast) {
        C v0[U][NS], v1[FORM == kRopeTwoChunks ? U : 1][NS];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int s = 0; s < NS; ++s) {
                if (live[s] && at + u * p.abreast + side < n) {
                    v0[u][s] = *reinterpret_cast<const C *>(x[s]);
                    if constexpr (FORM == kRopeTwoChunks) v1[u][s] = *reinterpret_cast<const C *>(x[s] + apart[s]);
                }
                x[s] += x_step[s];
            }
        if (at == 0) {
            __syncthreads();                   // the pairs
            for (uint32_t e = threadIdx.x; e < n * p.all_pairs; e += blockDim.x) {
                const uint32_t tok = fdiv(e, p.per_token), i = e - tok * p.all_pairs;
                if (i < (uint32_t)p.pairs) table[e] = rope_angle(p, pairs[i], rope_axis(p, i), token0 + tok);
            }
            __syncthreads();
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int s = 0; s < NS; ++s) {
                const uint32_t tok = at + u * p.abreast + side;
                if (live[s] && tok < n) {
                    const float2 *cs = table + tok * p.all_pairs + pair0[s];
                    float a[V];
                    unpack(v0[u][s], a);
                    if constexpr (FORM == kRopeInside) {
                        if (pair0[s] + V / 2 <= p.pairs) {
#pragma unroll
                            for (int i = 0; i < V / 2; ++i) turn(a[2 * i], a[2 * i + 1], cs[i]);
                            pack(a, v0[u][s]);
                        } else {               // the axes end in this chunk, or before it
#pragma unroll
                            for (int i = 0; i < V / 2; ++i)
                                if (pair0[s] + i < p.pairs) turn(a[2 * i], a[2 * i + 1], cs[i]);
                            const C in = v0[u][s];
                            pack(a, v0[u][s]);
                            v0[u][s] = keep_behind<V>(v0[u][s], in, 2 * (p.pairs - pair0[s]));
                        }
                        *reinterpret_cast<C *>(y[s]) = v0[u][s];
                    } else {
                        if (pair0[s] < p.pairs) {      // whole items turn or pass
                            float b[V];
                            unpack(v1[u][s], b);
#pragma unroll
                            for (int i = 0; i < V; ++i) turn(a[i], b[i], cs[i]);
                            pack(a, v0[u][s]);
                            pack(b, v1[u][s]);
                        }
                        *reinterpret_cast<C *>(y[s]) = v0[u][s];
                        *reinterpret_cast<C *>(y[s] + apart[s]) = v1[u][s];
                    }
                }
                y[s] += y_step[s];
            }
    }
}

// Pairs one by one: a lane holds pairs lane, lane + 32, .. of a head, whose channels and angle stay in registers for
// `rows` rows (heads) of a token; behind the axes it holds neighbouring channels, which pass through.  Element loads
// and stores, whole rows of a warp contiguous; a lane writes what it read, so in place is safe.
template <typename T>
__device__ __forceinline__ float value_of(T v) { return (float)v; }
template <typename T>
__device__ __forceinline__ T rounded(float v);
template <>
__device__ __forceinline__ float rounded<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 rounded<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

template <typename T, int NP>
__global__ void __launch_bounds__(kRopeThreads) rope_pairs_kernel(const __grid_constant__ RopeParams p) {
    constexpr int U = NP <= 2 ? 4 : 2;         // rows in flight
    const uint32_t lane = threadIdx.x & 31;
    uint32_t c1[NP], c2[NP];
    RopePair pair[NP];
#pragma unroll
    for (int k = 0; k < NP; ++k) {
        const int i = lane + 32 * k;
        c1[k] = 2 * i, c2[k] = 2 * i + 1;
        if (i >= p.pairs) continue;
        pair[k] = p.pair[i];
#pragma unroll
        for (int a = 0; a < 3; ++a) {
            const int s = p.axis_at[a], e = p.axis_at[a + 1];
            if (2 * i >= s && 2 * i < e) {
                c1[k] = s / 2 + i;
                c2[k] = c1[k] + (e - s) / 2;
            }
        }
    }
    for (uint32_t item = blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5); item < p.warp_items;
         item += gridDim.x * (kRopeThreads / 32)) {
        const uint32_t token = fdiv(item, p.items), part = item - token * p.items.d;
        float2 cs[NP];
#pragma unroll
        for (int k = 0; k < NP; ++k) {
            const int i = lane + 32 * k;
            if (i < p.pairs) cs[k] = rope_angle(p, pair[k], rope_axis(p, i), token);
        }
        const uint32_t first = part * p.rows_per_warp, last = min(first + p.rows_per_warp, p.all_rows);
        for (uint32_t r0 = first; r0 < last; r0 += U) {
            T a[U][NP], b[U][NP];
            T *to[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const uint32_t row = min(r0 + u, last - 1);
                int t = 0;
#pragma unroll
                for (int i = 1; i < NOMAS_ROPE_MAX_TENSORS; ++i)
                    if (i < p.n_tensors && row >= p.t[i].first_row) t = i;
                const uint32_t head = row - p.t[t].first_row;
                const T *x = reinterpret_cast<const T *>(p.t[t].x + token * p.t[t].x_tok + head * p.t[t].x_head);
                to[u] = reinterpret_cast<T *>(p.t[t].y + token * p.t[t].y_tok + head * p.t[t].y_head);
#pragma unroll
                for (int k = 0; k < NP; ++k)
                    if ((int)lane + 32 * k < p.all_pairs) a[u][k] = x[c1[k]], b[u][k] = x[c2[k]];
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (r0 + u >= last) break;
#pragma unroll
                for (int k = 0; k < NP; ++k) {
                    if ((int)lane + 32 * k >= p.all_pairs) continue;
                    if ((int)lane + 32 * k < p.pairs) {
                        float v = value_of(a[u][k]), w = value_of(b[u][k]);
                        turn(v, w, cs[k]);
                        a[u][k] = rounded<T>(v), b[u][k] = rounded<T>(w);
                    }
                    to[u][c1[k]] = a[u][k], to[u][c2[k]] = b[u][k];
                }
            }
        }
    }
}

template <typename T>
static int launch_rope_pairs(unsigned grid, const RopeParams &p, cudaStream_t st) {
    if (p.all_pairs <= 32)
        rope_pairs_kernel<T, 1><<<grid, kRopeThreads, 0, st>>>(p);
    else if (p.all_pairs <= 64)
        rope_pairs_kernel<T, 2><<<grid, kRopeThreads, 0, st>>>(p);
    else
        rope_pairs_kernel<T, 4><<<grid, kRopeThreads, 0, st>>>(p);
    return check_launch("rope_pairs_kernel launch");
}

template <typename T, int V, int FORM>
static int launch_rope(dim3 grid, unsigned threads, const RopeParams &p, cudaStream_t st) {
    if (p.items.d > kRopeThreads)
        rope_kernel<T, V, FORM, 2><<<grid, threads, 0, st>>>(p);
    else
        rope_kernel<T, V, FORM, 1><<<grid, threads, 0, st>>>(p);
    return check_launch("rope_kernel launch");
}

// The fraction of a number of turns, in 2^-64.  In long double: an index of the grid multiplies the rounding.
static int64_t rope_fraction(long double turns) {
    const long double part = turns - std::nearbyint(turns);            // exact, -1/2 .. 1/2
    return (int64_t)((uint64_t)std::llrint(part * 0x1p63L) << 1);
}

static bool rope_spec_ok(const nomas_rope_spec *s) {
    if (!s || s->head_dim < 8 || s->head_dim > NOMAS_ROPE_MAX_HEAD_DIM || s->head_dim % 8 != 0) return false;
    if (s->pairing != NOMAS_ROPE_INTERLEAVED && s->pairing != NOMAS_ROPE_HALVES) return false;
    if (!std::isfinite(s->theta) || s->theta <= 0.0) return false;
    int64_t sum = 0;
    for (int a = 0; a < 3; ++a) {
        if (s->axis_dim[a] < 0 || s->axis_dim[a] % 2 != 0) return false;
        sum += s->axis_dim[a];
    }
    return sum >= 2 && sum <= s->head_dim;
}

// Whether every value of y has a place of its own: heads inside a token's stride or tokens inside a head's.
static bool rope_places_apart(const nomas_rope_tensor &t, int64_t tokens, int64_t d) {
    auto apart = [d](int64_t outer, int64_t n_outer, int64_t inner, int64_t n_inner) {
        return (n_inner < 2 || inner >= d) &&
               (n_outer < 2 || (__int128)outer >= (__int128)(n_inner > 1 ? n_inner - 1 : 0) * inner + d);
    };
    return apart(t.y_tok_stride, tokens, t.y_head_stride, t.heads) || apart(t.y_head_stride, t.heads, t.y_tok_stride, tokens);
}

}  // namespace nomas

using namespace nomas;

extern "C" int nomas_rope(const nomas_rope_spec *spec, const nomas_rope_grid *grid, const float *positions,
                          int64_t tokens, const nomas_rope_tensor *tensors, int n_tensors, int dtype, int inverse,
                          nomas_stream stream) {
    if (!rope_spec_ok(spec) || !tensors || n_tensors < 1 || n_tensors > NOMAS_ROPE_MAX_TENSORS || tokens < 0)
        return NOMAS_EINVAL;
    if ((grid != nullptr) == (positions != nullptr)) return NOMAS_EINVAL;
    if (dtype != NOMAS_DTYPE_F32 && dtype != NOMAS_DTYPE_BF16) return NOMAS_EINVAL;
    RopeParams p{};
    if (grid) {
        if (grid->grid_h < 1 || grid->grid_w < 1 || (int64_t)grid->grid_h * grid->grid_w >= (int64_t)1 << 31)
            return NOMAS_EINVAL;
        for (int a = 0; a < 3; ++a)
            if (!std::isfinite(grid->origin[a]) || !std::isfinite(grid->step[a])) return NOMAS_EINVAL;
        p.plane = make_fastdiv((uint32_t)(grid->grid_h * grid->grid_w));
        p.width = make_fastdiv((uint32_t)grid->grid_w);
    } else if (reinterpret_cast<uintptr_t>(positions) % 4 != 0) {
        return NOMAS_EINVAL;
    }
    if (tokens >= (int64_t)1 << 31) return NOMAS_EUNSUPPORTED;

    const int esize = dtype == NOMAS_DTYPE_BF16 ? 2 : 4;
    int v = 16 / esize;                        // values of a chunk
    p.axis_at[0] = 0;
    for (int a = 0; a < 3; ++a) p.axis_at[a + 1] = p.axis_at[a] + spec->axis_dim[a];
    p.pairs = p.axis_at[3] / 2;
    p.all_pairs = spec->head_dim / 2;
    RopeForm form = kRopeInside;
    if (spec->pairing == NOMAS_ROPE_HALVES) {
        int all = spec->head_dim;
        for (int a = 0; a < 3; ++a) all |= spec->axis_dim[a];
        if (all % (2 * v) != 0) v = 4;         // chunks of 8 bytes in bf16
        form = all % (2 * v) == 0 ? kRopeTwoChunks : kRopePairs;
    }
    const int64_t per_head = spec->head_dim / (form == kRopeTwoChunks ? 2 * v : v);
    int64_t items = 0;
    for (int i = 0; i < n_tensors; ++i) {
        const nomas_rope_tensor &t = tensors[i];
        if (!t.x || !t.y || !aligned16(t.x) || !aligned16(t.y) || t.heads < 1) return NOMAS_EINVAL;
        for (int64_t s : {t.x_tok_stride, t.x_head_stride, t.y_tok_stride, t.y_head_stride})
            if (s % 8 != 0 || s < 0) return NOMAS_EINVAL;
        if (!rope_places_apart(t, tokens, spec->head_dim)) return NOMAS_EINVAL;
        for (int j = 0; j < n_tensors; ++j)
            if (j != i && (t.y == tensors[j].y || t.y == tensors[j].x)) return NOMAS_EINVAL;
        if (t.x == t.y && (t.x_tok_stride != t.y_tok_stride || t.x_head_stride != t.y_head_stride)) return NOMAS_EINVAL;
        p.t[i] = RopeTensor{static_cast<const char *>(t.x), static_cast<char *>(t.y), t.x_tok_stride * esize,
                            t.x_head_stride * esize, t.y_tok_stride * esize, t.y_head_stride * esize, (uint32_t)items, p.all_rows};
        p.all_rows += (uint32_t)t.heads;
        items += t.heads * per_head;
        if (items >= (int64_t)1 << 24) return NOMAS_EUNSUPPORTED;      // 512 a CTA along a grid's y
    }
    if (tokens == 0) return NOMAS_OK;
    // theta^(-2 i / d) as powers of one root: 127 products in the 64-bit mantissa of long double, each off by 2^-64 and by
    // the root's 2^-63, stay exact to 2^-55
    int pair = 0;
    for (int a = 0; a < 3; ++a) {
        if (spec->axis_dim[a] == 0) continue;
        const long double root = std::pow((long double)spec->theta, -2.0L / spec->axis_dim[a]);
        long double at = 1.0L / 6.283185307179586476925286766559L;
        for (int i = 0; i < spec->axis_dim[a] / 2; ++i, ++pair, at *= root) {
            const double turns = (double)at;
            if (!std::isfinite(turns) || (grid && (!std::isfinite(turns * grid->origin[a]) || !std::isfinite(turns * grid->step[a]))))
                return NOMAS_EINVAL;
            if (grid)
                p.pair[pair] = RopePair{rope_fraction(at * grid->origin[a]), rope_fraction(at * grid->step[a])};
            else
                std::memcpy(&p.pair[pair].origin, &turns, sizeof(turns));
        }
    }
    p.positions = positions;
    p.items = make_fastdiv((uint32_t)items);
    p.per_head = make_fastdiv((uint32_t)per_head);
    p.per_token = make_fastdiv((uint32_t)p.all_pairs);
    p.tokens = (uint32_t)tokens;
    p.n_tensors = n_tensors;
    p.inverse = inverse != 0;
    DeviceScope dev(tensors[0].x);
    if (dev.rc) return dev.rc;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const int64_t sms = sm_count();
    if (form == kRopePairs) {
        // rows that share a token's angles: 32, fewer while there would be fewer than 16 warps an SM
        p.rows_per_warp = 32;
        while (p.rows_per_warp > 4 && tokens * ((p.all_rows + p.rows_per_warp - 1) / p.rows_per_warp) < 16 * sms)
            p.rows_per_warp /= 2;
        const int64_t parts = (p.all_rows + p.rows_per_warp - 1) / p.rows_per_warp, warps = tokens * parts;
        if (warps >= (int64_t)1 << 31) return NOMAS_EUNSUPPORTED;
        p.items = make_fastdiv((uint32_t)parts);
        p.warp_items = (uint32_t)warps;
        int64_t grid = (warps + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
        if (grid > 4 * sms) grid = 4 * sms;    // as many as run at once: a warp sets its pairs up once
        return dtype == NOMAS_DTYPE_BF16 ? launch_rope_pairs<__nv_bfloat16>((unsigned)grid, p, st)
                                         : launch_rope_pairs<float>((unsigned)grid, p, st);
    }
    // threads for `abreast` tokens side by side; a CTA takes two rounds of loads of them, fewer while every SM
    // would not get four CTAs, at most a table
    p.abreast = items > kRopeThreads ? 1 : (uint32_t)(kRopeThreads / items);
    if (p.abreast > tokens) p.abreast = (uint32_t)tokens;
    const unsigned threads = items > kRopeThreads ? kRopeThreads : (unsigned)((p.abreast * items + 31) / 32 * 32);
    const int64_t parts = items > kRopeThreads ? (items + 511) / 512 : 1;
    int64_t per_cta = 2 * (items > kRopeThreads ? 2 : 4) * p.abreast;
    if (per_cta > tokens * parts / (4 * sms)) per_cta = tokens * parts / (4 * sms);
    if (per_cta > kRopeTable / p.all_pairs) per_cta = kRopeTable / p.all_pairs;
    if (per_cta < p.abreast) per_cta = p.abreast <= kRopeTable / p.all_pairs ? p.abreast : kRopeTable / p.all_pairs;
    p.tokens_per_cta = (uint32_t)per_cta;
    const dim3 grid_dim((unsigned)((tokens + per_cta - 1) / per_cta), (unsigned)parts);
    if (dtype == NOMAS_DTYPE_F32)
        return form == kRopeInside ? launch_rope<float, 4, kRopeInside>(grid_dim, threads, p, st)
                                   : launch_rope<float, 4, kRopeTwoChunks>(grid_dim, threads, p, st);
    if (form == kRopeInside) return launch_rope<__nv_bfloat16, 8, kRopeInside>(grid_dim, threads, p, st);
    return v == 8 ? launch_rope<__nv_bfloat16, 8, kRopeTwoChunks>(grid_dim, threads, p, st)
                  : launch_rope<__nv_bfloat16, 4, kRopeTwoChunks>(grid_dim, threads, p, st);
}
