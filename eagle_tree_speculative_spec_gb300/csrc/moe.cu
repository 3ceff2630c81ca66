// eagle3_moe_route and eagle3_moe_combine: the row bookkeeping around the products by expert of a
// mixture-of-experts target's feed-forward layer (the layer's place: "EAGLE-3: Engineering
// Implementation of LLM Inference Acceleration", appendix C, where it is a dense SwiGLU).
//
// Routing.  One warp per row: a lane takes E / 32 logits as unsigned order keys, ranks them among
// themselves and lays them down in that order in shared memory, so that the largest top_k of the row are
// a merge of 32 sorted lists: a warp reduction of the heads' keys, one of the indices of those that have
// the maximum (the lowest, so ties are exact), and the winner's next key.  (Finding a lane's next key by
// a search among its registers took 850 instructions a row of 256 logits and 8 places, twice as many.)  32
// rows make a chunk; a row takes an expert at most once, so a chunk's choice of an expert is a 32-bit mask
// of rows, and a place's rank within the chunk is the population count of the mask below its row: a stable
// counting sort without any atomic whose order matters.  Up to 256 rows are one launch of a thread-block
// cluster, a chunk a block, whose places per expert the blocks read from one another's shared memory (64 rows
// of 256 experts: 7.5 us by two launches and 15 with their host time, 7.1 and 7.6 by one; with more chunks a
// block the rows are too few at a time: 512 rows 8.2 us by two launches, 12.6 by one).  More rows are two
// launches: the first also writes the places per (block, expert), the second adds the counts of the blocks
// before its own (at most 152 blocks, so at most 152 x 512 words read from L2 per block), scans the experts
// and places the rows.
//
// Combining.  A thread owns 8 columns of a row (or four vectors of 2 or 1, by alignment) and adds the row's
// top_k vectors in order in fp32; the loads of a row's places do not depend on one another.  Memory bound:
// every slot is read once (3840 x 8 rows of 4096 columns: 49 us, 93% of the copy bandwidth).
#include <algorithm>
#include <cmath>

#include "../../include/eagle3_chain.h"
#include "../../include/eagle3_moe.h"
#include "tc.cuh"

namespace e3 {
namespace {

constexpr int CHUNK = 32;             // rows of a mask
constexpr int ROUTE_THREADS = 1024;   // a warp per row of a chunk
constexpr int ROUTE_MAX_BLOCKS = 152;
constexpr int ROUTE_RANKS = 8;        // largest cluster (one launch)
constexpr int MAX_E = EAGLE3_MOE_MAX_EXPERTS;

struct RouteParams {
    int rows, E, k, sigmoid, renorm;
    float scale;
    int64_t ld;
    const float *logits;
    const int32_t *num_rows;
    int32_t *ids;
    float *weights;
    int32_t *offsets, *sorted, *slots, *dev_status;
    int32_t *counts;      // [blocks][E rounded up to 4] places per block (two launches)
    int chunks_per_block; // rows of block b: [b, b + 1) * chunks_per_block * CHUNK
    int ranks;            // one launch: blocks, a cluster; 0: two launches
};

E3_DEV int route_limit(const RouteParams &p) {
    if (!p.num_rows) return p.rows;
    const int n = *p.num_rows;
    if (n < 0 || n > p.rows) {
        if (blockIdx.x == 0 && threadIdx.x == 0) flag(p.dev_status, EAGLE3_DEV_CAPACITY);
        return n < 0 ? 0 : p.rows;
    }
    return n;
}

// The experts and weights of one row (all lanes of a warp); lane j < k returns place j's expert or -1.
// sorted: the warp's (PER + 1) x 32 words.
template <int PER>
E3_DEV int route_row(const RouteParams &p, int row, bool live, uint32_t *sorted) {
    const int lane = threadIdx.x & 31;
    uint32_t key[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = i * 32 + lane;
        key[i] = 0u;   // below the key of every finite number: not available
        if (live && e < p.E) {
            const float z = p.logits[(size_t)row * p.ld + e];
            // -0 + 0 = +0: equal numbers get equal keys
            if (isfinite(z)) key[i] = order_key(z + 0.0f);
        }
    }
    // ranks among the lane's own keys (equal ones by index), and the keys in that order, with a 0 behind
    int rank[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) rank[i] = 0;
#pragma unroll
    for (int i = 1; i < PER; ++i)
#pragma unroll
        for (int j = 0; j < i; ++j) {
            const bool first = key[j] >= key[i];
            rank[i] += first ? 1 : 0;
            rank[j] += first ? 0 : 1;
        }
    uint64_t order = 0;   // 4 bits an index, the first's lowest
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        sorted[rank[i] * 32 + lane] = key[i];
        order |= (uint64_t)i << (4 * rank[i]);
    }
    sorted[PER * 32 + lane] = 0u;
    uint32_t place_key = 0u, high = 0u, next = lane;   // next: this lane's head in `sorted`
    int place_id = -1;
    uint32_t head = sorted[next], head_id = (uint32_t)(order & 15u) * 32u + lane;
    for (int j = 0; j < p.k; ++j) {
        const uint32_t top = __reduce_max_sync(0xffffffffu, head);
        if (top == 0u) break;   // uniform: no finite logit is left
        const uint32_t at = __reduce_min_sync(0xffffffffu, head == top ? head_id : 0xffffffffu);
        if (head == top && head_id == at) {
            order >>= 4;
            next += 32;
            head = sorted[next];
            head_id = (uint32_t)(order & 15u) * 32u + lane;
        }
        if (j == 0) high = top;
        if (lane == j) {
            place_key = top;
            place_id = (int)at;
        }
    }
    // scores of the places; the largest logit is place 0's
    const float m = high ? key_to_float(high) : 0.0f;
    float score = 0.0f, total = 1.0f;
    if (place_id >= 0) {
        const float z = key_to_float(place_key);
        score = p.sigmoid ? 1.0f / (1.0f + expf(-z)) : expf(z - m);
    }
    if (p.renorm || !p.sigmoid) {
        float part = score;
        if (!p.renorm) {   // softmax over all finite logits
            part = 0.0f;
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (key[i]) part += expf(key_to_float(key[i]) - m);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
        total = part;
    }
    if (lane < p.k) {
        p.ids[(size_t)row * p.k + lane] = place_id;
        p.weights[(size_t)row * p.k + lane] = total > 0.0f ? score / total * p.scale : 0.0f;
    }
    return place_id;
}

// Exclusive scan over the experts of total[0 .. E) (shared memory, ROUTE_THREADS threads): returns
// this thread's (thread = expert) start, and the sum of all in *sum.
E3_DEV int scan_experts(int v, int *warp_sums, int *sum) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += up;
    }
    if (lane == 31) warp_sums[warp] = inc;
    __syncthreads();
    int w = warp_sums[lane];   // ROUTE_THREADS / 32 = 32 warps
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += up;
    }
    *sum = __shfl_sync(0xffffffffu, w, 31);
    const int before = __shfl_sync(0xffffffffu, w, warp > 0 ? warp - 1 : 0);
    return inc - v + (warp > 0 ? before : 0);
}

// Place (tid / k, tid % k) of the chunk at row0: its expert, or -1.  A chunk has at most 32 * 16 places.
E3_DEV int chunk_place(const RouteParams &p, int row0, int r) {
    const int row = row0 + r;
    return r < CHUNK && row < p.rows ? p.ids[(size_t)row0 * p.k + threadIdx.x] : -1;
}
// Its slot.  masks: the chunk's rows per expert; base: each expert's next slot.
E3_DEV void place(const RouteParams &p, int row0, int r, int id, const uint32_t *masks, const int *base) {
    const int row = row0 + r;
    if (r >= CHUNK || row >= p.rows) return;
    int slot = -1;
    if (id >= 0) {
        slot = base[id] + __popc(masks[id] & ((1u << r) - 1u));
        p.sorted[slot] = row;
    }
    p.slots[(size_t)row0 * p.k + threadIdx.x] = slot;
}

// Experts and weights of every row; and in one launch the offsets and slots, in two the places per expert of
// this block's rows.
template <int PER>
__global__ void __launch_bounds__(ROUTE_THREADS) moe_route_kernel(const RouteParams p) {
    extern __shared__ uint32_t lists[];
    __shared__ uint32_t masks[MAX_E];
    __shared__ int base[MAX_E], counts[MAX_E], warp_sums[32];
    pdl_wait();
    pdl_trigger();
    const int limit = route_limit(p);
    const int warp = threadIdx.x >> 5, first_row = blockIdx.x * p.chunks_per_block * CHUNK;
    int mine = 0;   // thread e: places of expert e in this block
    for (int c = 0; c < p.chunks_per_block; ++c) {
        const int row = first_row + c * CHUNK + warp;
        if (threadIdx.x < MAX_E) masks[threadIdx.x] = 0u;
        __syncthreads();
        if (row < p.rows) {
            const int id = route_row<PER>(p, row, row < limit, lists + warp * (PER + 1) * 32);
            if (id >= 0) atomicOr(&masks[id], 1u << warp);
        }
        __syncthreads();
        if (threadIdx.x < MAX_E) mine += __popc(masks[threadIdx.x]);
        if (!p.ranks) __syncthreads();
    }
    if (!p.ranks) {
        if (threadIdx.x < p.E) p.counts[(size_t)blockIdx.x * ((p.E + 3) & ~3) + threadIdx.x] = mine;
        return;
    }
    // one launch: every block holds a single chunk
    int all = mine, before = 0, total;   // of all ranks, of the ranks before this one
    if (p.ranks > 1) {
        if (threadIdx.x < MAX_E) counts[threadIdx.x] = mine;
        tc::cluster_sync();
        if (threadIdx.x < MAX_E) {
            all = 0;
            const uint32_t at = smem_u32(counts + threadIdx.x);
            for (int s = 0; s < p.ranks; ++s) {
                const int n = (int)__float_as_uint(tc::cluster_ld(tc::cluster_addr(at, s)));
                all += n;
                before += s < (int)blockIdx.x ? n : 0;
            }
        }
    }
    const int start = scan_experts(all, warp_sums, &total);
    if (threadIdx.x < MAX_E) base[threadIdx.x] = start + before;
    if (blockIdx.x == 0) {
        if (threadIdx.x < p.E) p.offsets[threadIdx.x] = start;
        if (threadIdx.x == 0) p.offsets[p.E] = total;
    }
    __syncthreads();
    const int r = threadIdx.x / p.k;
    place(p, first_row, r, chunk_place(p, first_row, r), masks, base);
    for (int s = total + blockIdx.x * ROUTE_THREADS + threadIdx.x; s < p.rows * p.k; s += p.ranks * ROUTE_THREADS)
        p.sorted[s] = -1;
    if (p.ranks > 1) tc::cluster_sync();   // no rank leaves while another reads its counts
}

__global__ void __launch_bounds__(ROUTE_THREADS) moe_place_kernel(const RouteParams p) {
    __shared__ uint32_t masks[MAX_E];
    __shared__ int base[MAX_E], warp_sums[32];
    __shared__ int4 before[ROUTE_THREADS], all[ROUTE_THREADS];   // [group][4 experts]
    pdl_wait();
    pdl_trigger();
    const int r = threadIdx.x / p.k, first_row = blockIdx.x * p.chunks_per_block * CHUNK;
    int id = chunk_place(p, first_row, r);   // in flight with the counts
    // thread (g, q): experts 4 q .. 4 q + 3 of blocks g, g + G, ..., 8 loads at a time
    const int quads = (p.E + 3) >> 2, bits = quads <= 32 ? 5 : quads <= 64 ? 6 : 7;
    const int q = threadIdx.x & ((1 << bits) - 1), g = threadIdx.x >> bits, G = ROUTE_THREADS >> bits;
    int4 sum = make_int4(0, 0, 0, 0), ahead = sum;
    if (q < quads) {
        const int4 *at = reinterpret_cast<const int4 *>(p.counts) + (size_t)g * quads + q;
        const int step = G * quads;
        int left = ((int)gridDim.x - g + G - 1) / G, left_ahead = ((int)blockIdx.x - g + G - 1) / G;
        for (; left > 0; left -= 8, left_ahead -= 8, at += 8 * step) {
            int4 v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = i < left ? __ldg(at + i * step) : make_int4(0, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                sum.x += v[i].x, sum.y += v[i].y, sum.z += v[i].z, sum.w += v[i].w;
                if (i < left_ahead) ahead.x += v[i].x, ahead.y += v[i].y, ahead.z += v[i].z, ahead.w += v[i].w;
            }
        }
    }
    all[threadIdx.x] = sum;
    before[threadIdx.x] = ahead;
    __syncthreads();
    int mine = 0, first = 0, total;
    if (threadIdx.x < p.E) {
        const int *sums = reinterpret_cast<const int *>(all) + threadIdx.x;
        const int *firsts = reinterpret_cast<const int *>(before) + threadIdx.x;
        for (int i = 0; i < G; ++i) {
            mine += sums[i << (bits + 2)];
            first += firsts[i << (bits + 2)];
        }
    }
    const int start = scan_experts(mine, warp_sums, &total);
    if (threadIdx.x < MAX_E) base[threadIdx.x] = start + first;
    if (blockIdx.x == 0) {
        if (threadIdx.x < p.E) p.offsets[threadIdx.x] = start;
        if (threadIdx.x == 0) p.offsets[p.E] = total;
    }
    for (int c = 0; c < p.chunks_per_block; ++c) {
        const int row0 = first_row + c * CHUNK;
        if (c > 0) id = chunk_place(p, row0, r);
        if (threadIdx.x < MAX_E) masks[threadIdx.x] = 0u;
        __syncthreads();
        if (id >= 0) atomicOr(&masks[id], 1u << r);
        __syncthreads();
        place(p, row0, r, id, masks, base);
        __syncthreads();
        if (threadIdx.x < MAX_E) base[threadIdx.x] += __popc(masks[threadIdx.x]);
    }
    const long long end = (long long)p.rows * p.k;
    for (long long s = total + (long long)blockIdx.x * ROUTE_THREADS + threadIdx.x; s < end;
         s += (long long)gridDim.x * ROUTE_THREADS)
        p.sorted[s] = -1;
}

// ---- combine ------------------------------------------------------------------------------------
constexpr int COMBINE_THREADS = 128;

struct CombineParams {
    int rows, n_slots, k, d;
    int64_t ld_y, ld_res, ld_out;
    const __nv_bfloat16 *y, *res;
    const int32_t *slots;
    const float *weights;
    __nv_bfloat16 *out;
    int32_t *dev_status;
};

template <int VEC>
struct Pack;
template <>
struct Pack<8> {
    using T = uint4;
};
template <>
struct Pack<2> {
    using T = uint32_t;
};
template <>
struct Pack<1> {
    using T = unsigned short;
};

template <int VEC>
E3_DEV void unpack(const typename Pack<VEC>::T &r, float (&v)[VEC]) {
    const __nv_bfloat16 *h = reinterpret_cast<const __nv_bfloat16 *>(&r);
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = __bfloat162float(h[i]);
}

// VEC columns a vector: 8 where every row starts on 16 bytes, 2 on 4, else 1.  A thread takes VECS vectors,
// COMBINE_THREADS apart, so that narrow ones keep as many bytes in flight (3840 x 8 rows of 4094 and 4095
// columns with one vector a thread: 79 and 126 us, 50 at 4096).
template <int VEC, int VECS>
__global__ void __launch_bounds__(COMBINE_THREADS) moe_combine_kernel(const CombineParams p) {
    using T = typename Pack<VEC>::T;
    pdl_wait();
    pdl_trigger();
    const int row = blockIdx.x;
    const int col = (blockIdx.y * VECS * COMBINE_THREADS + threadIdx.x) * VEC;
    constexpr int APART = COMBINE_THREADS * VEC;
    if (col >= p.d) return;   // VEC divides d
    float acc[VECS][VEC];
    T res[VECS];
#pragma unroll
    for (int u = 0; u < VECS; ++u) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) acc[u][i] = 0.0f;
        if (p.res && col + u * APART < p.d)
            // (past L1: out may be the same buffer, and a line's other columns another block's)
            res[u] = __ldcg(reinterpret_cast<const T *>(p.res + (size_t)row * p.ld_res + col + u * APART));
    }
    const int32_t *slots = p.slots + (size_t)row * p.k;
    const float *weights = p.weights + (size_t)row * p.k;
    for (int j0 = 0; j0 < p.k; j0 += 8) {   // the loads of 8 places together
        int at[8];
        float w[8];
        T raw[8][VECS];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            at[i] = j0 + i < p.k ? __ldg(slots + j0 + i) : -1;
            w[i] = j0 + i < p.k ? __ldg(weights + j0 + i) : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (at[i] >= p.n_slots) {
                flag(p.dev_status, EAGLE3_DEV_BAD_COUNTS);
                at[i] = -1;
            }
            if (at[i] < 0) continue;
            const __nv_bfloat16 *y = p.y + (size_t)at[i] * p.ld_y + col;
#pragma unroll
            for (int u = 0; u < VECS; ++u)
                if (VECS == 1 || col + u * APART < p.d) raw[i][u] = __ldg(reinterpret_cast<const T *>(y + u * APART));
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (at[i] < 0) continue;
#pragma unroll
            for (int u = 0; u < VECS; ++u) {
                float v[VEC];
                unpack<VEC>(raw[i][u], v);
#pragma unroll
                for (int c = 0; c < VEC; ++c) acc[u][c] = fmaf(w[i], v[c], acc[u][c]);
            }
        }
    }
#pragma unroll
    for (int u = 0; u < VECS; ++u) {
        if (col + u * APART >= p.d) break;
        if (p.res) {
            float v[VEC];
            unpack<VEC>(res[u], v);
#pragma unroll
            for (int i = 0; i < VEC; ++i) acc[u][i] += v[i];
        }
        T o;
        __nv_bfloat16 *h = reinterpret_cast<__nv_bfloat16 *>(&o);
#pragma unroll
        for (int i = 0; i < VEC; ++i) h[i] = __float2bfloat16_rn(acc[u][i]);
        *reinterpret_cast<T *>(p.out + (size_t)row * p.ld_out + col + u * APART) = o;
    }
}

// ---- host side ----------------------------------------------------------------------------------
struct RoutePlan {
    int blocks, chunks_per_block, ranks;
    size_t ws_bytes;
};

RoutePlan route_plan(const eagle3_moe_route_args_t *a) {
    const int chunks = (a->rows + CHUNK - 1) / CHUNK;
    RoutePlan pl;
    const bool one = chunks <= ROUTE_RANKS;
    pl.chunks_per_block = std::max(1, (chunks + ROUTE_MAX_BLOCKS - 1) / ROUTE_MAX_BLOCKS);
    pl.blocks = std::max(1, (chunks + pl.chunks_per_block - 1) / pl.chunks_per_block);
    pl.ranks = one ? pl.blocks : 0;
    pl.ws_bytes = !one ? (size_t)pl.blocks * ((a->n_experts + 3) & ~3) * sizeof(int32_t) : 0;
    return pl;
}

eagle3_status_t validate(const eagle3_moe_route_args_t *a) {
    if (!a) return EAGLE3_ERR_INVALID_ARGUMENT;
    if (a->rows < 0 || a->n_experts < 1 || a->top_k < 1 || a->top_k > a->n_experts) return EAGLE3_ERR_INVALID_ARGUMENT;
    if (a->scoring != EAGLE3_MOE_SOFTMAX && a->scoring != EAGLE3_MOE_SIGMOID) return EAGLE3_ERR_INVALID_ARGUMENT;
    if ((a->renormalize != 0 && a->renormalize != 1) || !std::isfinite(a->scale)) return EAGLE3_ERR_INVALID_ARGUMENT;
    if (a->ld_logits && a->ld_logits < a->n_experts) return EAGLE3_ERR_INVALID_ARGUMENT;
    if (a->n_experts > EAGLE3_MOE_MAX_EXPERTS || a->top_k > EAGLE3_MOE_MAX_TOP_K) return EAGLE3_ERR_UNSUPPORTED;
    // slots are 32-bit, and rows rounded up to whole blocks (at most a 152nd of them)
    if ((int64_t)a->rows * a->top_k > MAX_DIM - (1 << 24)) return EAGLE3_ERR_UNSUPPORTED;
    if (!a->expert_offsets) return EAGLE3_ERR_INVALID_ARGUMENT;
    if (a->rows && (!a->logits || !a->topk_ids || !a->topk_weights || !a->sorted_rows || !a->slots))
        return EAGLE3_ERR_INVALID_ARGUMENT;
    const uintptr_t all = (uintptr_t)a->logits | (uintptr_t)a->num_rows | (uintptr_t)a->topk_ids |
                          (uintptr_t)a->topk_weights | (uintptr_t)a->expert_offsets | (uintptr_t)a->sorted_rows |
                          (uintptr_t)a->slots | (uintptr_t)a->dev_status;
    return all & 3 ? EAGLE3_ERR_INVALID_ARGUMENT : EAGLE3_OK;
}

eagle3_status_t validate(const eagle3_moe_combine_args_t *a) {
    if (!a) return EAGLE3_ERR_INVALID_ARGUMENT;
    if (a->rows < 0 || a->n_slots < 0 || a->top_k < 1 || a->dim < 1) return EAGLE3_ERR_INVALID_ARGUMENT;
    if (a->top_k > EAGLE3_MOE_MAX_TOP_K || a->rows > MAX_DIM) return EAGLE3_ERR_UNSUPPORTED;
    if (a->dim > 65535 * COMBINE_THREADS) return EAGLE3_ERR_UNSUPPORTED;   // column blocks of the grid
    for (const int64_t ld : {a->ld_y, a->ld_res, a->ld_out})
        if (ld && ld < a->dim) return EAGLE3_ERR_INVALID_ARGUMENT;
    if (a->rows == 0) return EAGLE3_OK;
    if ((a->n_slots && !a->y) || !a->slots || !a->weights || !a->out) return EAGLE3_ERR_INVALID_ARGUMENT;
    if (((uintptr_t)a->y | (uintptr_t)a->residual | (uintptr_t)a->out) & 1) return EAGLE3_ERR_INVALID_ARGUMENT;
    if (((uintptr_t)a->slots | (uintptr_t)a->weights | (uintptr_t)a->dev_status) & 3)
        return EAGLE3_ERR_INVALID_ARGUMENT;
    return EAGLE3_OK;
}

template <int PER>
cudaError_t launch_route(int blocks, cudaStream_t st, const RouteParams &p) {
    constexpr int LISTS = CHUNK * (PER + 1) * 32 * 4;
    static PerDevice<cudaError_t> attr;
    const cudaError_t e = attr.get([] {
        return cudaFuncSetAttribute(moe_route_kernel<PER>, cudaFuncAttributeMaxDynamicSharedMemorySize, LISTS);
    });
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(ROUTE_THREADS);
    cfg.dynamicSmemBytes = LISTS;
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = std::max(1, p.ranks);
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = p.ranks > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, moe_route_kernel<PER>, p);
}

template <int VEC, int VECS>
cudaError_t launch_combine(cudaStream_t st, const CombineParams &p) {
    const int per_block = COMBINE_THREADS * VEC * VECS;
    return launch_pdl(moe_combine_kernel<VEC, VECS>, dim3(p.rows, (p.d + per_block - 1) / per_block),
                      dim3(COMBINE_THREADS), 0, st, p);
}

}  // namespace
}  // namespace e3

using namespace e3;

extern "C" size_t eagle3_moe_route_workspace_size(const eagle3_moe_route_args_t *a) {
    return validate(a) == EAGLE3_OK ? route_plan(a).ws_bytes : 0;
}

extern "C" eagle3_status_t eagle3_moe_route(const eagle3_moe_route_args_t *a, void *workspace, size_t ws_bytes,
                                            eagle3_stream_t stream) {
    const eagle3_status_t st = validate(a);
    if (st != EAGLE3_OK) return st;
    const RoutePlan pl = route_plan(a);
    if (pl.ws_bytes && (!workspace || ws_bytes < pl.ws_bytes || ((uintptr_t)workspace & 15)))
        return EAGLE3_ERR_WORKSPACE;
    RouteParams p;
    p.rows = a->rows;
    p.E = a->n_experts;
    p.k = a->top_k;
    p.sigmoid = a->scoring == EAGLE3_MOE_SIGMOID;
    p.renorm = a->renormalize;
    p.scale = a->scale;
    p.ld = a->ld_logits ? a->ld_logits : a->n_experts;
    p.logits = a->logits;
    p.num_rows = a->num_rows;
    p.ids = a->topk_ids;
    p.weights = a->topk_weights;
    p.offsets = a->expert_offsets;
    p.sorted = a->sorted_rows;
    p.slots = a->slots;
    p.dev_status = a->dev_status;
    p.counts = (int32_t *)workspace;
    p.chunks_per_block = pl.chunks_per_block;
    p.ranks = pl.ranks;
    const cudaStream_t s = (cudaStream_t)stream;
    const int per = (a->n_experts + 31) / 32;
    const cudaError_t e = per <= 2   ? launch_route<2>(pl.blocks, s, p)
                          : per <= 4 ? launch_route<4>(pl.blocks, s, p)
                          : per <= 8 ? launch_route<8>(pl.blocks, s, p)
                                     : launch_route<16>(pl.blocks, s, p);
    if (e != cudaSuccess) return EAGLE3_ERR_CUDA;
    if (!pl.ranks && launch_pdl(moe_place_kernel, dim3(pl.blocks), dim3(ROUTE_THREADS), 0, s, p) != cudaSuccess)
        return EAGLE3_ERR_CUDA;
    return EAGLE3_OK;
}

extern "C" eagle3_status_t eagle3_moe_combine(const eagle3_moe_combine_args_t *a, eagle3_stream_t stream) {
    const eagle3_status_t st = validate(a);
    if (st != EAGLE3_OK || a->rows == 0) return st;
    CombineParams p;
    p.rows = a->rows;
    p.n_slots = a->n_slots;
    p.k = a->top_k;
    p.d = a->dim;
    p.ld_y = a->ld_y ? a->ld_y : a->dim;
    p.ld_res = a->ld_res ? a->ld_res : a->dim;
    p.ld_out = a->ld_out ? a->ld_out : a->dim;
    p.y = (const __nv_bfloat16 *)a->y;
    p.res = (const __nv_bfloat16 *)a->residual;
    p.slots = a->slots;
    p.weights = a->weights;
    p.out = (__nv_bfloat16 *)a->out;
    p.dev_status = a->dev_status;
    // the widest vector that every row starts on
    int64_t step = p.d | p.ld_y | p.ld_out | (p.res ? p.ld_res : 0);
    const uintptr_t base = (uintptr_t)p.y | (uintptr_t)p.out | (uintptr_t)p.res;
    const cudaStream_t s = (cudaStream_t)stream;
    const cudaError_t e = step % 8 == 0 && base % 16 == 0  ? launch_combine<8, 1>(s, p)
                          : step % 2 == 0 && base % 4 == 0 ? launch_combine<2, 4>(s, p)
                                                           : launch_combine<1, 4>(s, p);
    return e == cudaSuccess ? EAGLE3_OK : EAGLE3_ERR_CUDA;
}
