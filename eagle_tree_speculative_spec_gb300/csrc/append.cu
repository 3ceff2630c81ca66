// eagle3_append_kv: keys and values of new tokens into a paged cache, bf16 or e4m3 with a power-of-two scale for
// each 64 places of a page and head, the keys rotated on the way (include/eagle3_kv.h).
//
// Sources: "Speculative Decoding (EAGLE3) in the vLLM Neuron Framework", "EagleProposer: Draft Model Management"
// (slot = block_table[pos / block_size] * block_size + pos % block_size); "Advanced speculative decoding: tree drafts
// and EAGLE", "Implementation" (the accepted path's K/V are copied into the cache, not recomputed).
//
// A scale belongs to one group of 64 places of one head, keys and values apart: that is a job.  Its new rows are held
// in registers between the two passes over them (largest magnitude, codes), so that everything is read and written
// once.  Prompts: a CTA of 256 threads takes the jobs of a group, one after the other, with the group's cosines and
// sines in shared memory.  Few tokens a sequence (at most 8): a warp takes a job.
#include "e4m3.cuh"
#include "rope.cuh"

#include <cfloat>
#include <cmath>

namespace e3 {
namespace {

constexpr int GROUP = EAGLE3_KV_GROUP;
constexpr int NT = 256;
constexpr int FEW = 8;   // new tokens a sequence for which a warp takes a job

struct Params {
    int B, Hkv, D, n_rows, max_new, rows_per_seq, max_blocks, block_size, n_pages, R, half;
    int groups_per_seq;      // groups that max_new tokens can touch
    int jobs_per_cta;        // of the 2 * Hkv (head, K or V) jobs of a group
    int interleaved, wide;   // wide: the partner of 8 dims is 8 dims that start on 16 bytes
    float amplitude;
    int64_t rs;
    const __nv_bfloat16 *k, *v;
    const int32_t *cache_len, *n_new, *row_start, *row_ids, *block_table;
    const uint64_t *table;
    uint8_t *kc, *vc;
    uint8_t *ks, *vs;
    int32_t *dev_status;
};

// The new tokens of one group: places [lo, hi) of the group's 64 hold tokens j0 .. of the sequence
struct Span {
    int b, len, lo, hi, j0, page, place;   // place: the group's first place on its page
};

// false: nothing to do.  `first`: this thread reports what is wrong with the sequence.
E3_DEV bool find_span(const Params &p, int b, int g, bool first, Span &s) {
    s.b = b;
    const int len = s.len = __ldg(p.cache_len + b);
    int n = p.max_new;
    if (p.n_new) {
        n = __ldg(p.n_new + b);
    } else {
        const int32_t *ids = p.row_ids + (size_t)b * p.max_new;
        for (n = 0; n < p.max_new && __ldg(ids + n) >= 0; ++n) {
        }
    }
    if (n < 0 || n > p.max_new || len < 0 || (long long)len + n > (long long)p.max_blocks * p.block_size) {
        if (first && g == 0) flag(p.dev_status, EAGLE3_DEV_CAPACITY);
        return false;
    }
    // groups are counted in places: a page of fewer than 64 (bf16) holds part of one
    const long long base = ((long long)(len / GROUP) + g) * GROUP;
    const long long lo = max((long long)len, base), hi = min((long long)len + n, base + GROUP);
    if (lo >= hi) return false;
    s.lo = (int)(lo - base);
    s.hi = (int)(hi - base);
    s.j0 = (int)(lo - len);
    s.page = (int)(base / p.block_size);
    s.place = (int)(base % p.block_size);
    return true;
}

// source row of token j, or -1
E3_DEV int source_row(const Params &p, int b, int j) {
    long long r;
    if (p.row_ids) {
        const int id = __ldg(p.row_ids + (size_t)b * p.max_new + j);
        if (id < 0 || id >= p.rows_per_seq) return -1;
        r = (long long)b * p.rows_per_seq + id;
    } else if (p.row_start) {
        r = (long long)__ldg(p.row_start + b) + j;
    } else {
        r = (long long)b * p.max_new + j;
    }
    return r < 0 || r >= p.n_rows ? -1 : (int)r;
}

E3_DEV void unpack8(uint4 u, float (&v)[8]) {
    const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(&u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __bfloat1622float2(h[i]);
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}

// 8 dims of a key row from d0 on, turned; cs: the row's cosines and sines
E3_DEV void turn8(const Params &p, const __nv_bfloat16 *row, int d0, const float2 *cs, float (&v)[8]) {
    if (d0 >= p.R) return;
    if (p.interleaved) {
        if (d0 + 8 <= p.R) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 w = cs[d0 / 2 + i];
                const float a = v[2 * i], b = v[2 * i + 1];
                v[2 * i] = a * w.x - b * w.y;
                v[2 * i + 1] = b * w.x + a * w.y;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (d0 + 2 * i >= p.R) break;
                const float2 w = cs[d0 / 2 + i];
                const float a = v[2 * i], b = v[2 * i + 1];
                v[2 * i] = a * w.x - b * w.y;
                v[2 * i + 1] = b * w.x + a * w.y;
            }
        }
        return;
    }
    if (p.wide) {
        const bool upper = d0 >= p.half;
        const int j = upper ? d0 - p.half : d0;
        float o[8];
        unpack8(*reinterpret_cast<const uint4 *>(row + (upper ? j : d0 + p.half)), o);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 w = cs[j + i];
            v[i] = upper ? v[i] * w.x + o[i] * w.y : v[i] * w.x - o[i] * w.y;
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int d = d0 + i;
        if (d >= p.R) break;
        const bool upper = d >= p.half;
        const int j = upper ? d - p.half : d;
        const float2 w = cs[j];
        const float o = (float)row[upper ? j : d + p.half];
        v[i] = upper ? v[i] * w.x + o * w.y : v[i] * w.x - o * w.y;
    }
}

// 8 codes of another scale: by 2^-down, rounded again
E3_DEV uint2 scaled_down(uint2 c, float factor) {
    uint32_t w[2] = {c.x, c.y};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float2 a = from_e4m3x2(w[i] & 0xffffu), b = from_e4m3x2(w[i] >> 16);
        w[i] = to_e4m3x2(a.x * factor, a.y * factor) | to_e4m3x2(b.x * factor, b.y * factor) << 16;
    }
    return make_uint2(w[0], w[1]);
}

// One job (a head's keys or values of a group) by THREADS threads, ITEMS runs of 8 dims each.  cs: cosines and sines by
// [place - lo][pair], or null; scratch: a word a warp for the CTA's maximum.
template <int THREADS, int ITEMS, bool E4M3>
E3_DEV void append_job(const Params &p, const Span &s, int page, int job, int t, const float2 *cs, float *scratch) {
    const bool is_v = job >= p.Hkv;
    const int h = is_v ? job - p.Hkv : job;
    const int cpr = p.D / 8, n = (s.hi - s.lo) * cpr;
    const __nv_bfloat16 *src = (is_v ? p.v : p.k) + (size_t)h * p.D;
    uint8_t *dst = is_v ? p.vc : p.kc;
    float val[ITEMS][8];
    bool have[ITEMS];
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        const int it = t + i * THREADS;
        const int row = it / cpr, d0 = it % cpr * 8;
        have[i] = it < n;
        int r = -1;
        if (have[i]) {
            r = source_row(p, s.b, s.j0 + row);
            if (r < 0 && job == 0 && d0 == 0) flag(p.dev_status, EAGLE3_DEV_BAD_TOKEN);
            have[i] = r >= 0;
        }
        if (have[i]) unpack8(*reinterpret_cast<const uint4 *>(src + r * p.rs + d0), val[i]);
        if (have[i] && cs && !is_v) turn8(p, src + r * p.rs, d0, cs + row * p.half, val[i]);
        if (E4M3 && have[i]) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float a = fabsf(val[i][e]);
                if (a <= FLT_MAX)
                    top = fmaxf(top, a);
                else
                    val[i][e] = __int_as_float(0x7fc00000);
            }
        }
    }
    if constexpr (!E4M3) {
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            if (!have[i]) continue;
            const int it = t + i * THREADS;
            const int place = s.lo + it / cpr, d0 = it % cpr * 8;
            // a page may end inside the group
            const long long pos = (long long)s.page * p.block_size + s.place + place;
            const int id = __ldg(p.block_table + (size_t)s.b * p.max_blocks + (int)(pos / p.block_size));
            if (id < 0 || id >= p.n_pages) {
                if (job == 0 && d0 == 0) flag(p.dev_status, EAGLE3_DEV_CAPACITY);
                continue;
            }
            const long long slot = (long long)id * p.block_size + pos % p.block_size;
            uint4 u;
            __nv_bfloat162 *b2 = reinterpret_cast<__nv_bfloat162 *>(&u);
#pragma unroll
            for (int e = 0; e < 4; ++e) b2[e] = __floats2bfloat162_rn(val[i][2 * e], val[i][2 * e + 1]);
            *reinterpret_cast<uint4 *>(dst + ((size_t)slot * p.Hkv + h) * p.D * 2 + d0 * 2) = u;
        }
        return;
    } else {
#pragma unroll
        for (int x = 16; x; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
        uint8_t *scales = (is_v ? p.vs : p.ks) + ((size_t)page * p.Hkv + h) * (p.block_size / GROUP) + s.place / GROUP;
        int old = s.lo > 0 ? *scales : 0;
        if constexpr (THREADS > 32) {
            if ((t & 31) == 0) scratch[t >> 5] = top;
            __syncthreads();   // the scale has been read by everyone too
#pragma unroll
            for (int w = 0; w < THREADS / 32; ++w) top = fmaxf(top, scratch[w]);
            __syncthreads();
        } else {
            __syncwarp();
        }
        const int byte = max(old, scale_byte(top));
        if (t == 0) *scales = (uint8_t)byte;
        const float inv = inverse_scale(byte);
        uint8_t *codes = dst + (((size_t)page * p.Hkv + h) * p.block_size + s.place) * p.D;
        if (s.lo > 0 && byte > old) {
            // steps far below the new one leave nothing but the sign
            const float factor = byte - old > 40 ? 0.0f : __int_as_float((127 - (byte - old)) << 23);
            for (int it = t; it < s.lo * cpr; it += THREADS) {
                uint2 *c = reinterpret_cast<uint2 *>(codes + (size_t)it * 8);
                *c = scaled_down(*c, factor);
            }
        }
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            if (!have[i]) continue;
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = to_e4m3x2(val[i][2 * e] * inv, val[i][2 * e + 1] * inv);
            *reinterpret_cast<uint2 *>(codes + (size_t)s.lo * p.D + (size_t)(t + i * THREADS) * 8) =
                make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
        }
    }
}

// grid: (group of a sequence, share of its jobs, sequence)
template <int ITEMS, bool E4M3, bool BY_WARP>
__global__ void __launch_bounds__(NT) append_kernel(const Params p) {
    extern __shared__ float2 cs[];   // [new rows of the group][pair]
    __shared__ float scratch[NT / 32];
    pdl_wait();
    pdl_trigger();
    Span s;
    if (!find_span(p, blockIdx.z, blockIdx.x, threadIdx.x == 0 && blockIdx.y == 0, s)) return;
    int page = -1;
    if (E4M3) {
        page = __ldg(p.block_table + (size_t)s.b * p.max_blocks + s.page);
        if (page < 0 || page >= p.n_pages) {
            if (threadIdx.x == 0 && blockIdx.y == 0) flag(p.dev_status, EAGLE3_DEV_CAPACITY);
            return;
        }
    }
    const int j0 = blockIdx.y * p.jobs_per_cta, j1 = min(2 * p.Hkv, j0 + p.jobs_per_cta);
    if (p.table && j0 < p.Hkv) {   // some of the CTA's jobs are keys
        for (int i = threadIdx.x; i < (s.hi - s.lo) * p.half; i += NT)
            cs[i] = turned(s.len + s.j0 + i / p.half, __ldg(p.table + i % p.half), p.amplitude);
    }
    __syncthreads();
    const float2 *angles = p.table ? cs : nullptr;
    if constexpr (BY_WARP) {
        for (int job = j0 + (threadIdx.x >> 5); job < j1; job += NT / 32)
            append_job<32, ITEMS, E4M3>(p, s, page, job, threadIdx.x & 31, angles, nullptr);
    } else {
        for (int job = j0; job < j1; ++job) append_job<NT, ITEMS, E4M3>(p, s, page, job, threadIdx.x, angles, scratch);
    }
}

template <int ITEMS, bool E4M3, bool BY_WARP>
cudaError_t launch(const Params &p, dim3 grid, size_t smem, cudaStream_t stream) {
    static PerDevice<cudaError_t> attr;
    auto *kernel = append_kernel<ITEMS, E4M3, BY_WARP>;
    const cudaError_t e = attr.get([=] {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    GROUP * EAGLE3_ROPE_MAX_DIM / 2 * (int)sizeof(float2));
    });
    return e != cudaSuccess ? e : launch_pdl(kernel, grid, dim3(NT), smem, stream, p);
}

template <int ITEMS>
cudaError_t launch_by(const Params &p, bool e4m3, bool few, dim3 grid, size_t smem, cudaStream_t stream) {
    if (e4m3) return few ? launch<ITEMS, true, true>(p, grid, smem, stream) : launch<ITEMS, true, false>(p, grid, smem, stream);
    return few ? launch<ITEMS, false, true>(p, grid, smem, stream) : launch<ITEMS, false, false>(p, grid, smem, stream);
}

}  // namespace
}  // namespace e3

using namespace e3;

extern "C" eagle3_status_t eagle3_append_kv(const eagle3_append_kv_args_t *a, eagle3_stream_t stream) {
    if (!a || a->batch < 0 || a->n_kv_heads < 1 || a->head_dim < 1 || a->n_rows < 0 || a->max_new < 0 ||
        a->max_blocks < 1 || a->block_size < 1 || a->n_pages < 1 || a->row_stride < 0 ||
        (a->format != EAGLE3_KV_BF16 && a->format != EAGLE3_KV_E4M3))
        return EAGLE3_ERR_INVALID_ARGUMENT;
    const bool e4m3 = a->format == EAGLE3_KV_E4M3;
    if (e4m3 && a->block_size % GROUP) return EAGLE3_ERR_INVALID_ARGUMENT;
    if (a->rope_table && (!rope_dims_ok(a->rotary_dim, a->head_dim) || !std::isfinite(a->rope_amplitude) ||
                          a->rope_layout < EAGLE3_ROPE_HALF || a->rope_layout > EAGLE3_ROPE_INTERLEAVED))
        return EAGLE3_ERR_INVALID_ARGUMENT;
    if ((a->row_ids && (a->row_start || a->rows_per_seq < 1)) || (!a->n_new && !a->row_ids)) return EAGLE3_ERR_INVALID_ARGUMENT;
    if (a->head_dim % 8 || a->head_dim > EAGLE3_ROPE_MAX_DIM || a->n_kv_heads > 32767 || a->batch > 65535 ||
        (int64_t)a->max_blocks * a->block_size > MAX_DIM || a->max_new > MAX_DIM)
        return EAGLE3_ERR_UNSUPPORTED;
    const int64_t dense = (int64_t)a->n_kv_heads * a->head_dim;
    const int64_t rs = a->row_stride ? a->row_stride : dense;
    if (rs < dense || rs % 8) return EAGLE3_ERR_INVALID_ARGUMENT;
    if (a->batch == 0 || a->max_new == 0) return EAGLE3_OK;
    const void *wide[] = {a->k_new, a->v_new, a->k_cache, a->v_cache};
    for (const void *ptr : wide)
        if (!ptr || ((uintptr_t)ptr & 15)) return EAGLE3_ERR_INVALID_ARGUMENT;
    const void *words[] = {a->cache_len, a->block_table};
    for (const void *ptr : words)
        if (!ptr || ((uintptr_t)ptr & 3)) return EAGLE3_ERR_INVALID_ARGUMENT;
    if ((((uintptr_t)a->n_new | (uintptr_t)a->row_start | (uintptr_t)a->row_ids) & 3) || ((uintptr_t)a->rope_table & 7) ||
        (e4m3 && (!a->k_scale || !a->v_scale)))
        return EAGLE3_ERR_INVALID_ARGUMENT;
    Params p;
    p.B = a->batch;
    p.Hkv = a->n_kv_heads;
    p.D = a->head_dim;
    p.n_rows = a->n_rows;
    p.max_new = a->max_new;
    p.rows_per_seq = a->rows_per_seq;
    p.max_blocks = a->max_blocks;
    p.block_size = a->block_size;
    p.n_pages = a->n_pages;
    p.R = a->rope_table ? a->rotary_dim : 0;
    p.half = p.R / 2;
    p.interleaved = a->rope_layout == EAGLE3_ROPE_INTERLEAVED;
    p.wide = p.R % 16 == 0;
    p.amplitude = a->rope_amplitude;
    p.rs = rs;
    p.k = (const __nv_bfloat16 *)a->k_new;
    p.v = (const __nv_bfloat16 *)a->v_new;
    p.cache_len = a->cache_len;
    p.n_new = a->n_new;
    p.row_start = a->row_start;
    p.row_ids = a->row_ids;
    p.block_table = a->block_table;
    p.table = a->rope_table;
    p.kc = (uint8_t *)a->k_cache;
    p.vc = (uint8_t *)a->v_cache;
    p.ks = a->k_scale;
    p.vs = a->v_scale;
    p.dev_status = a->dev_status;
    const bool few = p.max_new <= FEW;
    // a sequence cannot get more than its pages hold
    const int reach = p.max_new < p.max_blocks * p.block_size ? p.max_new : p.max_blocks * p.block_size;
    p.groups_per_seq = (reach - 1 + GROUP - 1) / GROUP + 1;
    const int jobs = 2 * p.Hkv;
    // enough CTAs for every SM to have four; a share of jobs no smaller than its warps when a warp takes a job
    const int64_t ctas = (int64_t)p.groups_per_seq * p.B;
    int cuts = 1;
    while (cuts < jobs && ctas * cuts < 4 * device_sm_count()) cuts *= 2;
    p.jobs_per_cta = (jobs + cuts - 1) / cuts;
    if (few && p.jobs_per_cta < NT / 32) p.jobs_per_cta = jobs < NT / 32 ? jobs : NT / 32;
    const dim3 grid((unsigned)p.groups_per_seq, (unsigned)((jobs + p.jobs_per_cta - 1) / p.jobs_per_cta), (unsigned)p.B);
    const size_t smem = (size_t)(few ? FEW : GROUP) * p.half * sizeof(float2);
    const cudaStream_t st = (cudaStream_t)stream;
    const cudaError_t e = p.D <= 128 ? launch_by<4>(p, e4m3, few, grid, smem, st) : launch_by<8>(p, e4m3, few, grid, smem, st);
    return e == cudaSuccess ? EAGLE3_OK : EAGLE3_ERR_CUDA;
}
