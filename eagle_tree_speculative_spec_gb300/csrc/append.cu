// eagle3_append_kv: keys and values of new tokens into a paged cache, bf16 or e4m3 with a power-of-two scale for
// each 64 places of a page and head, the keys rotated on the way (include/eagle3_kv.h).
//
// Sources: "Speculative Decoding (EAGLE3) in the vLLM Neuron Framework", "EagleProposer: Draft Model Management"
// (slot = block_table[pos / block_size] * block_size + pos % block_size); "Advanced speculative decoding: tree drafts
// and EAGLE", "Implementation" (the accepted path's K/V are copied into the cache, not recomputed).
//
// A scale belongs to one group of 64 places of one head, keys and values apart: that is a job.  Its new rows are held
// in registers between the two passes over them (largest magnitude, codes), so that everything is read and written
// once.  A thread's unit is 16 dims of a row, both ends of their pairs among them.  Prompts: a CTA of 256 threads takes a run
// of jobs, one after the other, with their group's cosines and sines in shared memory, which the keys of all heads share.
// Few tokens a sequence (at most 8): a warp takes a job.
// Bound by latency: 16384 tokens of 8 heads of 128 (e4m3, 100.7 MB) take 25.7 us, 3.9 TB/s (14.8 us at the copy's rate).  17.7
// million warp instructions are 14 us of every scheduler; the rest is a job's chain from its loads over the maximum that a
// CTA's warps share to its codes, with three CTAs an SM to hide it (of 8 cycles an issue 1.5 wait for memory, 1.5 for
// another warp's turn, 0.7 at the barrier, 0.7 for a pipe).  Four CTAs an SM of 64 registers a thread and no load ahead took
// 29.3 us; addresses kept in registers, which spill, 27.0 us.
#include "e4m3.cuh"
#include "rope.cuh"

#include <algorithm>
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
    int jobs, jobs_per_cta;  // the (sequence, group, head, K or V) jobs of all groups
    int interleaved, paired;   // paired: dims lie in whole runs of 8 pairs
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

// Cosines and sines of a row are kept as pairs of pairs, in fours: within a four they are swapped about by the four's
// number, so that the lanes of eight consecutive fours meet all banks (a plain order: 4 of them at a time in 2 banks).
E3_DEV int two_at(int two) { return (two & ~3) | ((two ^ two >> 3) & 3); }
E3_DEV int pair_at(int j) { return two_at(j >> 1) * 2 + (j & 1); }
E3_DEV int cs_pitch(int half) { return (half + 7) & ~7; }

E3_DEV void unpack8(uint4 u, float *v) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

E3_DEV void turn(float &a, float &b, float cos, float sin) {
    const float x = a * cos - b * sin;
    b = b * cos + a * sin;
    a = x;
}

// A thread's unit, 16 dims of a row: the runs of 8 dims from da and from db on, which hold 8 whole pairs where
// p.paired; db < 0: the row ends after the first.
struct Unit {
    int da, db, pair;   // pair: the first of its pairs, -1 where it is not turned as a whole
};
E3_DEV Unit unit_of(const Params &p, int u) {
    if (p.paired && !p.interleaved && u < p.R / 16) return {8 * u, p.half + 8 * u, 8 * u};
    return {16 * u, 16 * u + 8 < p.D ? 16 * u + 8 : -1, p.paired && u < p.R / 16 ? 8 * u : -1};
}

// 8 dims from d0 on of a key row whose pairs do not lie in whole runs; cs: the row's cosines and sines
E3_DEV void turn_run(const Params &p, const __nv_bfloat16 *row, int d0, const float2 *cs, float *v) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int d = d0 + i;
        if (d >= p.R) break;
        if (p.interleaved) {
            if (i % 2 == 0) {
                const float2 w = cs[pair_at(d / 2)];
                turn(v[i], v[i + 1], w.x, w.y);
            }
        } else {
            const bool upper = d >= p.half;
            const int j = upper ? d - p.half : d;
            const float2 w = cs[pair_at(j)];
            const float o = (float)row[upper ? j : d + p.half];
            v[i] = upper ? v[i] * w.x + o * w.y : v[i] * w.x - o * w.y;
        }
    }
}

template <bool PAIRED>
E3_DEV void turn_unit(const Params &p, const Unit &un, const __nv_bfloat16 *row, const float2 *cs, float *v) {
    if constexpr (!PAIRED) {
        turn_run(p, row, un.da, cs, v);
        if (un.db >= 0) turn_run(p, row, un.db, cs, v + 8);
        return;
    }
    if (un.pair < 0) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 w = reinterpret_cast<const float4 *>(cs)[two_at(un.pair / 2 + i)];
        if (p.interleaved) {
            turn(v[4 * i], v[4 * i + 1], w.x, w.y);
            turn(v[4 * i + 2], v[4 * i + 3], w.z, w.w);
        } else {
            turn(v[2 * i], v[8 + 2 * i], w.x, w.y);
            turn(v[2 * i + 1], v[9 + 2 * i], w.z, w.w);
        }
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

E3_DEV float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

E3_DEV uint2 codes8(const float *v, float inv) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 x = __fmul2_rn(make_float2(v[2 * e], v[2 * e + 1]), make_float2(inv, inv));
        w[e] = to_e4m3x2(x.x, x.y);
    }
    return make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
}

E3_DEV uint4 bf16x8(const float *v) {
    uint4 u;
    __nv_bfloat162 *b2 = reinterpret_cast<__nv_bfloat162 *>(&u);
#pragma unroll
    for (int e = 0; e < 4; ++e) b2[e] = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
    return u;
}

// A job is a head's keys (even) or values (odd) of a group, by a warp or by the CTA; a CTA takes a run of the jobs of all
// groups.  A thread keeps its unit and its rows, ITEMS of them, for all jobs of a group, and loads the next job's before
// it converts this one's.
template <int ITEMS, bool E4M3, bool BY_WARP, bool PAIRED>
__global__ void __launch_bounds__(NT, ITEMS == 2 && PAIRED ? 3 : 1) append_kernel(const Params p) {
    constexpr int THREADS = BY_WARP ? 32 : NT;
    extern __shared__ float4 cs4[];   // [new rows of the group][pair]
    __shared__ float4 scratch[2][NT / 128];
    float2 *const cs = reinterpret_cast<float2 *>(cs4);
    pdl_wait();
    pdl_trigger();
    const int warp = threadIdx.x >> 5, t = BY_WARP ? threadIdx.x & 31 : threadIdx.x;
    const int units = (p.D + 15) / 16, step = THREADS / units;   // rows at a time
    const int row0 = t / units, u = t - row0 * units;
    const Unit un = unit_of(p, u);
    const int pitch = cs_pitch(p.half);
    const int at0 = blockIdx.x * p.jobs_per_cta, end = min(p.jobs - at0, p.jobs_per_cta) + at0;
    int parity = 0;
    for (int at = at0; at < end;) {
        const int group = at / (2 * p.Hkv), b = group / p.groups_per_seq;
        const int j0 = at - group * (2 * p.Hkv), j1 = min(2 * p.Hkv, j0 + (end - at));
        at += j1 - j0;
        Span s;
        if (!find_span(p, b, group - b * p.groups_per_seq, threadIdx.x == 0 && j0 == 0, s)) continue;
        const int32_t *bt = p.block_table + (size_t)s.b * p.max_blocks;
        int page = -1;
        if (E4M3) {
            page = __ldg(bt + s.page);
            if (page < 0 || page >= p.n_pages) {
                if (threadIdx.x == 0 && j0 == 0) flag(p.dev_status, EAGLE3_DEV_CAPACITY);
                continue;
            }
        }
        const bool reports = j0 == 0 && u == 0 && (!BY_WARP || warp == 0);
        int src[ITEMS];
        long long slot[ITEMS];   // the rows they come from and, bf16, the places they go to; src < 0: none
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const int row = row0 + i * step;
            src[i] = -1;
            if (row0 < step && row < s.hi - s.lo) {
                src[i] = source_row(p, s.b, s.j0 + row);
                if (src[i] < 0 && reports) flag(p.dev_status, EAGLE3_DEV_BAD_TOKEN);
            }
            if (!E4M3 && src[i] >= 0) {   // a page may end inside the group
                const int pos = s.len + s.j0 + row, block = pos / p.block_size;
                const int id = __ldg(bt + block);
                slot[i] = (long long)id * p.block_size + (pos - block * p.block_size);
                if (id < 0 || id >= p.n_pages) {
                    if (reports) flag(p.dev_status, EAGLE3_DEV_CAPACITY);
                    src[i] = -1;
                }
            }
        }
        uint4 next[ITEMS][2];
        auto fetch = [&](int job) {
            const __nv_bfloat16 *from = (job & 1 ? p.v : p.k) + (size_t)(job >> 1) * p.D;
#pragma unroll
            for (int i = 0; i < ITEMS; ++i) {
                next[i][0] = next[i][1] = make_uint4(0, 0, 0, 0);
                if (src[i] < 0) continue;
                next[i][0] = *reinterpret_cast<const uint4 *>(from + src[i] * p.rs + un.da);
                if (un.db >= 0) next[i][1] = *reinterpret_cast<const uint4 *>(from + src[i] * p.rs + un.db);
            }
        };
        const int first = BY_WARP ? j0 + warp : j0, jump = BY_WARP ? NT / 32 : 1;
        if (first < j1) fetch(first);
        __syncthreads();   // (the group before has been turned)
        if (p.table) {
            const int j = threadIdx.x % p.half;
            const uint64_t turns = __ldg(p.table + j);
            if (threadIdx.x < NT / p.half * p.half)
                for (int row = threadIdx.x / p.half; row < s.hi - s.lo; row += NT / p.half)
                    cs[row * pitch + pair_at(j)] = turned(s.len + s.j0 + row, turns, p.amplitude);
        }
        __syncthreads();
        for (int job = first; job < j1; job += jump) {
            const bool is_v = job & 1;
            const int h = job >> 1;
            const size_t head_page = (size_t)page * p.Hkv + h;
            uint8_t *scales = nullptr;
            int old = 0;
            if (E4M3) {
                scales = (is_v ? p.vs : p.ks) + head_page * (p.block_size / GROUP) + s.place / GROUP;
                if (s.lo > 0) old = *scales;
            }
            float val[ITEMS][16];
            float top = 0.0f;
#pragma unroll
            for (int i = 0; i < ITEMS; ++i) {
                unpack8(next[i][0], val[i]);
                unpack8(next[i][1], val[i] + 8);
            }
            if (job + jump < j1) fetch(job + jump);
            if (p.table && !is_v) {
#pragma unroll
                for (int i = 0; i < ITEMS; ++i)
                    if (src[i] >= 0)
                        turn_unit<PAIRED>(p, un, p.k + (size_t)h * p.D + src[i] * p.rs, cs + (row0 + i * step) * pitch, val[i]);
            }
            uint8_t *dst = is_v ? p.vc : p.kc;
            if constexpr (!E4M3) {
#pragma unroll
                for (int i = 0; i < ITEMS; ++i) {
                    if (src[i] < 0) continue;
                    uint8_t *to = dst + ((size_t)slot[i] * p.Hkv + h) * p.D * 2;
                    *reinterpret_cast<uint4 *>(to + un.da * 2) = bf16x8(val[i]);
                    if (un.db >= 0) *reinterpret_cast<uint4 *>(to + un.db * 2) = bf16x8(val[i] + 8);
                }
            } else {
#pragma unroll
                for (int i = 0; i < ITEMS; ++i)
#pragma unroll
                    for (int e = 0; e < 16; e += 2)   // (passes over NaN)
                        top = max3(top, fabsf(val[i][e]), fabsf(val[i][e + 1]));
                if (top > FLT_MAX) {   // infinities become NaN, and no scale follows them
                    top = 0.0f;
#pragma unroll
                    for (int i = 0; i < ITEMS; ++i)
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const float a = fabsf(val[i][e]);
                            if (a <= FLT_MAX)
                                top = fmaxf(top, a);
                            else
                                val[i][e] = __int_as_float(0x7fc00000);
                        }
                }
                // magnitudes are in the order of their bits
                top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
                if constexpr (!BY_WARP) {
                    if ((t & 31) == 0) reinterpret_cast<float *>(scratch[parity])[warp] = top;
                    __syncthreads();   // the scale has been read by everyone too
#pragma unroll
                    for (int w = 0; w < NT / 128; ++w) {
                        const float4 m = scratch[parity][w];
                        top = max3(max3(top, m.x, m.y), m.z, m.w);
                    }
                    parity ^= 1;
                } else {
                    __syncwarp();   // the scale has been read by all lanes
                }
                const int byte = max(old, scale_byte(top));
                if (t == 0) *scales = (uint8_t)byte;
                uint8_t *codes = dst + (head_page * p.block_size + s.place) * p.D;
                const float inv = inverse_scale(byte);
#pragma unroll
                for (int i = 0; i < ITEMS; ++i) {
                    if (src[i] < 0) continue;
                    uint8_t *to = codes + (size_t)(s.lo + row0 + i * step) * p.D;
                    *reinterpret_cast<uint2 *>(to + un.da) = codes8(val[i], inv);
                    if (un.db >= 0) *reinterpret_cast<uint2 *>(to + un.db) = codes8(val[i] + 8, inv);
                }
                if (s.lo > 0 && byte > old) {
                    // steps far below the new one leave nothing but the sign
                    const float factor = byte - old > 40 ? 0.0f : __int_as_float((127 - (byte - old)) << 23);
                    uint2 *c = reinterpret_cast<uint2 *>(codes);
                    const int n = s.lo * (p.D / 8);
                    constexpr int K = 8;   // loads in flight
                    for (int it = t; it < n; it += K * THREADS) {
                        uint2 w[K];
#pragma unroll
                        for (int k = 0; k < K; ++k) w[k] = it + k * THREADS < n ? c[it + k * THREADS] : make_uint2(0, 0);
#pragma unroll
                        for (int k = 0; k < K; ++k)
                            if (it + k * THREADS < n) c[it + k * THREADS] = scaled_down(w[k], factor);
                    }
                }
            }
        }
    }
}

template <int ITEMS, bool E4M3, bool BY_WARP, bool PAIRED>
cudaError_t launch(const Params &p, dim3 grid, size_t smem, cudaStream_t stream) {
    static PerDevice<cudaError_t> attr;
    auto *kernel = append_kernel<ITEMS, E4M3, BY_WARP, PAIRED>;
    const cudaError_t e = attr.get([=] {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    GROUP * EAGLE3_ROPE_MAX_DIM / 2 * (int)sizeof(float2));
    });
    return e != cudaSuccess ? e : launch_pdl(kernel, grid, dim3(NT), smem, stream, p);
}

template <int ITEMS, bool PAIRED>
cudaError_t launch_by(const Params &p, bool e4m3, bool few, dim3 grid, size_t smem, cudaStream_t stream) {
    if (e4m3) return few ? launch<ITEMS, true, true, PAIRED>(p, grid, smem, stream) : launch<ITEMS, true, false, PAIRED>(p, grid, smem, stream);
    return few ? launch<ITEMS, false, true, PAIRED>(p, grid, smem, stream) : launch<ITEMS, false, false, PAIRED>(p, grid, smem, stream);
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
    if (a->n_rows > 0 && (!a->k_new || !a->v_new)) return EAGLE3_ERR_INVALID_ARGUMENT;   // (no rows: nothing reads there)
    if (!a->k_cache || !a->v_cache) return EAGLE3_ERR_INVALID_ARGUMENT;
    const void *wide[] = {a->k_new, a->v_new, a->k_cache, a->v_cache};
    for (const void *ptr : wide)
        if ((uintptr_t)ptr & 15) return EAGLE3_ERR_INVALID_ARGUMENT;
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
    p.paired = p.R % 16 == 0 && p.D % 16 == 0;
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
    // one wave of CTAs, each with its run of jobs (16384 tokens of 8 heads: 9 jobs for each of 456; 8 for each of 512
    // took 31.8 us); no fewer than its warps when a warp takes a job.  bf16 jobs are short beside what a CTA begins with,
    // the table's angles: more CTAs, of fewer (7 x 999 tokens of 5 heads 7.4 us by two, 10.3 us by three jobs a CTA)
    const int64_t all = (int64_t)p.groups_per_seq * p.B * jobs;
    if (all > MAX_DIM) return EAGLE3_ERR_UNSUPPORTED;
    const int64_t most = (e4m3 ? 3 : 4) * (int64_t)std::max(1, device_sm_count());   // (0: no device, which the launch will say)
    // (of the groups that a sequence touches at most, one is there because tokens may begin inside a group: shares are of the others)
    const int64_t sure = (int64_t)((reach + GROUP - 1) / GROUP) * p.B * jobs;
    p.jobs = (int)all;
    p.jobs_per_cta = (int)((sure + most - 1) / most);
    const int least = few ? jobs < NT / 32 ? jobs : NT / 32 : 1;
    if (p.jobs_per_cta < least) p.jobs_per_cta = least;
    const dim3 grid((unsigned)((all + p.jobs_per_cta - 1) / p.jobs_per_cta));
    const size_t smem = (size_t)(few ? FEW : GROUP) * ((p.half + 7) / 8 * 8) * sizeof(float2);
    const cudaStream_t st = (cudaStream_t)stream;
    cudaError_t e;
    if (p.paired)
        e = p.D <= 128 ? launch_by<2, true>(p, e4m3, few, grid, smem, st) : launch_by<4, true>(p, e4m3, few, grid, smem, st);
    else
        e = p.D <= 128 ? launch_by<2, false>(p, e4m3, few, grid, smem, st) : launch_by<4, false>(p, e4m3, few, grid, smem, st);
    return e == cudaSuccess ? EAGLE3_OK : EAGLE3_ERR_CUDA;
}
