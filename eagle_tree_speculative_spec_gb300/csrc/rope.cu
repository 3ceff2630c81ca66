// eagle3_rope_table, eagle3_rope: rotary positions of rows of heads, in whole or part of the head, with half or
// interleaved pairs and frequencies scaled for long contexts (include/eagle3_kv.h has the formulas).
//
// Sources: "EAGLE-3: Engineering Implementation of LLM Inference Acceleration", appendix C (rotate-half RoPE with
// inv_j = theta^(-2j/D)); the scaled frequencies are those of position interpolation (Chen et al., 2023), of the
// Llama 3.1 model card's configuration and of "YaRN: Efficient Context Window Extension" (Peng et al., 2023).
//
// A row's angles are shared by its heads: a CTA takes a few rows and first fills their cosines and sines into shared
// memory (series about the nearest quarter turn, turned() in rope.cuh; at most one angle a thread), then walks the heads.
// A thread's unit is the two runs of V elements that hold V pairs, so that it reads and writes both ends of each pair
// itself and the call can run in place; it stays with one row, whose cosines it holds in registers, and has four heads'
// loads in flight, the first four while the angles are made.
// Bound by memory and the latency of its waves: 3840 rows of 40 bf16 heads of 128 (78.6 MB) take 15.9 us, 5.0 TB/s (11.6 us
// at the copy's rate), in three waves of CTAs, each with its first loads and angles; with the cosines read from shared
// memory for every head (lanes 64 bytes apart: four-way conflicts) and one head at a time, 26.9 us.
#include "rope.cuh"

#include <algorithm>
#include <cmath>
#include <type_traits>

namespace e3 {
namespace {

constexpr int NT = 256;

struct Steps {
    uint64_t v[EAGLE3_ROPE_MAX_DIM / 2];
};

__global__ void rope_table_kernel(const __grid_constant__ Steps steps, int n, uint64_t *table) {
    const int j = threadIdx.x;
    if (j < n) table[j] = steps.v[j];
}

struct Params {
    int rows, heads, D, R, rows_per_cta, heads_per_cta;
    float amplitude;
    int inverse;
    int64_t x_rs, o_rs;
    const void *x;
    const int32_t *positions;
    const uint64_t *table;
    void *out;
};

// V consecutive elements as they lie in memory
template <typename T, int V>
struct Run {
    using Word = std::conditional_t<V == 1, T, uint4>;
    static constexpr int WORDS = V * sizeof(T) / sizeof(Word);
    Word w[WORDS];

    E3_DEV void load(const T *p) {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) w[i] = reinterpret_cast<const Word *>(p)[i];
    }
    E3_DEV void unpack(float (&v)[V]) const {
        if constexpr (V == 1) {
            v[0] = (float)w[0];
        } else {
            const T *e = reinterpret_cast<const T *>(w);
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = (float)e[i];
        }
    }
};

template <int V, typename T>
E3_DEV void store(T *p, const float (&v)[V]) {
    if constexpr (V == 1) {
        *p = (T)v[0];
    } else if constexpr (sizeof(T) == 2) {
        uint4 u;
        __nv_bfloat162 *h = reinterpret_cast<__nv_bfloat162 *>(&u);
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        *reinterpret_cast<uint4 *>(p) = u;
    } else {
        *reinterpret_cast<float4 *>(p) = *reinterpret_cast<const float4 *>(&v[0]);
        *reinterpret_cast<float4 *>(p + 4) = *reinterpret_cast<const float4 *>(&v[4]);
    }
}

// V = 8 pairs a unit where rotary_dim is a multiple of 16 (16- and 32-byte accesses), else one
template <typename T, int V, bool INTERLEAVED>
__global__ void __launch_bounds__(NT, 3) rope_kernel(const Params p) {
    constexpr int AHEAD = V * sizeof(T) > 16 ? 2 : 4;   // heads that a thread loads before it turns the first
    __shared__ float2 cs[NT];   // [row][pair]
    pdl_wait();
    pdl_trigger();
    const int half = p.R / 2;
    const int r0 = blockIdx.x * p.rows_per_cta, rn = min(p.rows_per_cta, p.rows - r0);
    const int h0 = blockIdx.y * p.heads_per_cta, h1 = min(p.heads, h0 + p.heads_per_cta);
    const int units = half / V + (p.D - p.R) / V;   // runs of pairs, then runs that are copied; at most NT
    const int slots = NT / units, slot = threadIdx.x / units, unit = threadIdx.x % units;
    const int at_once = min(p.rows_per_cta, slots), step = slots / at_once;   // rows at a time, heads of each
    const bool copy = unit >= half / V;
    const int first_r = slot < at_once * step && !(copy && p.x == p.out) ? slot / step : rn, first_h = h0 + slot % step;
    const int j = unit * V;
    const int da = copy ? p.R + (unit - half / V) * V : INTERLEAVED ? 2 * j : j;
    const int db = INTERLEAVED ? 2 * j + V : half + j;
    Run<T, V> ra[AHEAD], rb[AHEAD];
    auto load = [&](int r, int h) {
        const T *x = (const T *)p.x + (r0 + r) * p.x_rs;
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            if (h + k * step >= h1) break;
            ra[k].load(x + (size_t)(h + k * step) * p.D + da);
            if (!copy) rb[k].load(x + (size_t)(h + k * step) * p.D + db);
        }
    };
    if (first_r < rn) load(first_r, first_h);   // (these arrive while the angles are made)
    for (int i = threadIdx.x; i < rn * half; i += NT) {
        float2 w = turned(p.positions[r0 + i / half], p.table[i % half], p.amplitude);
        if (p.inverse) w.y = -w.y;
        cs[i] = w;
    }
    __syncthreads();
    for (int r = first_r; r < rn; r += at_once) {
        T *out = (T *)p.out + (r0 + r) * p.o_rs;
        float2 w[V];
#pragma unroll
        for (int i = 0; i < V; ++i) w[i] = copy ? make_float2(1.0f, 0.0f) : cs[r * half + j + i];
        for (int h = first_h; h < h1; h += AHEAD * step) {
            if (r != first_r || h != first_h) load(r, h);
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) {
                if (h + k * step >= h1) break;
                T *o = out + (size_t)(h + k * step) * p.D;
                float a[V], b[V];
                ra[k].unpack(a);
                if (!copy) {
                    rb[k].unpack(b);
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        // the pair's two elements: at the same place of both runs, or next to each other
                        float &u = INTERLEAVED && V > 1 ? (2 * i < V ? a[(2 * i) % V] : b[(2 * i) % V]) : a[i];
                        float &v = INTERLEAVED && V > 1 ? (2 * i < V ? a[(2 * i + 1) % V] : b[(2 * i + 1) % V]) : b[i];
                        const float c = u * w[i].x - v * w[i].y, s = v * w[i].x + u * w[i].y;
                        u = c;
                        v = s;
                    }
                    store<V>(o + db, b);
                }
                store<V>(o + da, a);
            }
        }
    }
}

template <typename T, int V>
cudaError_t launch(const Params &p, bool interleaved, dim3 grid, cudaStream_t stream) {
    return interleaved ? launch_pdl(rope_kernel<T, V, true>, grid, dim3(NT), 0, stream, p)
                       : launch_pdl(rope_kernel<T, V, false>, grid, dim3(NT), 0, stream, p);
}

}  // namespace
}  // namespace e3

using namespace e3;

extern "C" eagle3_status_t eagle3_rope_table(const eagle3_rope_table_args_t *a, eagle3_stream_t stream) {
    if (!a || !rope_dims_ok(a->rotary_dim, EAGLE3_ROPE_MAX_DIM)) return EAGLE3_ERR_INVALID_ARGUMENT;
    const int R = a->rotary_dim;
    const bool bands = a->scaling == EAGLE3_ROPE_BANDS, ramp = a->scaling == EAGLE3_ROPE_RAMP;
    if (a->scaling < EAGLE3_ROPE_NONE || a->scaling > EAGLE3_ROPE_RAMP || !(a->theta > 1.0) || !std::isfinite(a->theta))
        return EAGLE3_ERR_INVALID_ARGUMENT;
    if (a->scaling != EAGLE3_ROPE_NONE && !(a->factor >= 1.0 && std::isfinite(a->factor))) return EAGLE3_ERR_INVALID_ARGUMENT;
    if (a->scaling == EAGLE3_ROPE_BASE && R <= 2) return EAGLE3_ERR_INVALID_ARGUMENT;
    if ((bands || ramp) && !(a->original_positions >= 1 && a->low_turns > 0.0 && a->high_turns > a->low_turns &&
                             std::isfinite(a->high_turns)))
        return EAGLE3_ERR_INVALID_ARGUMENT;
    if (!a->table || ((uintptr_t)a->table & 7)) return EAGLE3_ERR_INVALID_ARGUMENT;
    const double two_pi = 6.283185307179586476925;
    double theta = a->theta, lo = 0.0, hi = 0.0;
    if (a->scaling == EAGLE3_ROPE_BASE) theta *= std::pow(a->factor, (double)R / (R - 2));
    if (ramp) {
        auto pair_of = [&](double turns) {
            return R * std::log(a->original_positions / (turns * two_pi)) / (2.0 * std::log(theta));
        };
        lo = std::fmax(std::floor(pair_of(a->high_turns)), 0.0);
        hi = std::fmin(std::ceil(pair_of(a->low_turns)), R - 1.0);
    }
    Steps steps;
    for (int j = 0; j < R / 2; ++j) {
        double f = std::pow(theta, -2.0 * j / R);
        if (a->scaling == EAGLE3_ROPE_LINEAR) f /= a->factor;
        if (bands) {
            const double t = a->original_positions * f / two_pi;
            const double k = std::fmin(std::fmax((t - a->low_turns) / (a->high_turns - a->low_turns), 0.0), 1.0);
            f = k * f + (1.0 - k) * f / a->factor;
        }
        if (ramp) {
            const double k = std::fmin(std::fmax((j - lo) / std::fmax(hi - lo, 0.001), 0.0), 1.0);
            f = (1.0 - k) * f + k * f / a->factor;
        }
        steps.v[j] = (uint64_t)std::floor(std::ldexp(f / two_pi, 64) + 0.5);   // f <= 1: below 2^62
    }
    rope_table_kernel<<<1, EAGLE3_ROPE_MAX_DIM / 2, 0, (cudaStream_t)stream>>>(steps, R / 2, a->table);
    return cudaGetLastError() == cudaSuccess ? EAGLE3_OK : EAGLE3_ERR_CUDA;
}

extern "C" eagle3_status_t eagle3_rope(const eagle3_rope_args_t *a, eagle3_stream_t stream) {
    if (!a || a->rows < 0 || a->n_heads < 1 || a->head_dim < 1 || !std::isfinite(a->amplitude) || a->x_row_stride < 0 ||
        a->out_row_stride < 0 || (a->inverse != 0 && a->inverse != 1) || a->layout < EAGLE3_ROPE_HALF ||
        a->layout > EAGLE3_ROPE_INTERLEAVED)
        return EAGLE3_ERR_INVALID_ARGUMENT;
    if (a->head_dim % 8 || a->head_dim > EAGLE3_ROPE_MAX_DIM || (a->elem_bytes != 2 && a->elem_bytes != 4) ||
        a->rows > MAX_DIM || a->n_heads > MAX_DIM / EAGLE3_ROPE_MAX_DIM)
        return EAGLE3_ERR_UNSUPPORTED;
    if (!rope_dims_ok(a->rotary_dim, a->head_dim)) return EAGLE3_ERR_INVALID_ARGUMENT;
    const int64_t dense = (int64_t)a->n_heads * a->head_dim;
    Params p;
    p.x_rs = a->x_row_stride ? a->x_row_stride : dense;
    p.o_rs = a->out_row_stride ? a->out_row_stride : dense;
    if (p.x_rs < dense || p.o_rs < dense || p.x_rs * a->elem_bytes % 16 || p.o_rs * a->elem_bytes % 16)
        return EAGLE3_ERR_INVALID_ARGUMENT;
    if (a->rows == 0) return EAGLE3_OK;
    if (!a->x || !a->out || !a->positions || !a->table || (((uintptr_t)a->x | (uintptr_t)a->out) & 15) ||
        ((uintptr_t)a->positions & 3) || ((uintptr_t)a->table & 7) || (a->x == a->out && p.x_rs != p.o_rs))
        return EAGLE3_ERR_INVALID_ARGUMENT;
    p.rows = a->rows;
    p.heads = a->n_heads;
    p.D = a->head_dim;
    p.R = a->rotary_dim;
    p.amplitude = a->amplitude;
    p.inverse = a->inverse;
    p.x = a->x;
    p.positions = a->positions;
    p.table = a->table;
    p.out = a->out;
    const int v = p.R % 16 == 0 ? 8 : 1;
    const int units = p.R / 2 / v + (p.D - p.R) / v;
    const int pass = NT / units;   // heads that a CTA takes at once
    // rows a CTA, as many at most as there are threads for angles: those with which the waves of CTAs, each of a thread's
    // heads and what a CTA costs besides, take the least time (3840 rows of 40 heads: 3 rows, 2.8 waves; 4 rows are 2.1,
    // and took 17.6 us).  Few rows: the heads are cut over CTAs too, so that every SM gets four
    const int sms = std::max(1, device_sm_count());   // (0: no device, which the launch will say)
    const int want = 4 * sms, resident = 3 * sms;
    int64_t least = 0;
    for (int n = 1; n <= NT / (p.R / 2) && (n == 1 || n <= pass); ++n) {
        const int64_t waves = ((p.rows + n - 1) / n + resident - 1) / resident, step = pass / n;
        const int64_t cost = waves * ((p.heads + step - 1) / step + 2);
        if (n == 1 || cost < least) least = cost, p.rows_per_cta = n;
    }
    const int rb = (p.rows + p.rows_per_cta - 1) / p.rows_per_cta;
    const int passes = (p.heads + pass - 1) / pass;
    int cuts = 1;
    while (cuts < passes && rb * (int64_t)cuts < want) ++cuts;
    p.heads_per_cta = (passes + cuts - 1) / cuts * pass;
    const dim3 grid((unsigned)rb, (unsigned)((p.heads + p.heads_per_cta - 1) / p.heads_per_cta));
    if (grid.y > 65535u) return EAGLE3_ERR_UNSUPPORTED;
    const bool il = a->layout == EAGLE3_ROPE_INTERLEAVED;
    const cudaStream_t st = (cudaStream_t)stream;
    cudaError_t e;
    if (a->elem_bytes == 2)
        e = v == 8 ? launch<__nv_bfloat16, 8>(p, il, grid, st) : launch<__nv_bfloat16, 1>(p, il, grid, st);
    else
        e = v == 8 ? launch<float, 8>(p, il, grid, st) : launch<float, 1>(p, il, grid, st);
    return e == cudaSuccess ? EAGLE3_OK : EAGLE3_ERR_CUDA;
}
