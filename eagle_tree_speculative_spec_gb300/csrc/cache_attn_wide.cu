// eagle3_verify_attn_fp8 for many query rows (trees): the tcgen05 kernel, and the join of what its CTAs shared.
//
// A unit of work is a sequence, a KV head and up to 256 query rows (row = node * rep + head); its keys come in tiles of
// 128 places, the tree's nodes as one more.  The tiles of all units, one after the other, are cut into equal ranges, one
// for each CTA (one CTA an SM): ragged lengths, one long sequence and many short ones are all spread evenly, and a unit
// is cut only where a range ends.  Cut units leave unnormalised partial results, which a second kernel joins in order.
//
// S = Q K^T takes K's codes as they lie in memory: Q is held as two e4m3 parts (row scaled to at most 448; hi = e4m3(q),
// lo = e4m3(q - hi): 4 + 4 bits are bf16's 8), so that QK runs as two e4m3 products, in the time of one of bf16, and K is
// never converted.  P V runs in fp16: weights in 11 bits (8 bits of bf16, or two e4m3 parts whose floor is 2^-18 of the
// largest weight, would cost long sums), V's codes converted exactly, times the power of two by which their group's scale
// differs from the range's largest.
//
// Two streams of (S, P, O) in tensor memory keep the tensor cores busy while the other's softmax runs: with more than
// 128 rows a stream is a row tile and both take every key tile; with up to 128 the streams take alternate key tiles of
// the same rows and are added up at the end of the unit.
//   warp 0        TMA: K tiles into a ring of 3, V codes into a ring of 2
//   warp 1, 2     the MMAs of S, and of P V (one thread issues an MMA about every 110 cycles: two threads)
//   warp 3        looks a unit ahead: largest V scale of its range, the tree's scales and ancestor bits
//   warps 4..7    V codes to fp16; Q's parts and row scales of the next unit; the tree's K and V
//   warps 8..15   softmax of stream 0 and 1, a row a thread; at the end of a unit its results
// All waits are bounded; one that runs out sets EAGLE3_DEV_TIMEOUT and the CTA drains and exits.
#include "cache_attn.cuh"
#include "tc.cuh"
#include "tmap.cuh"

namespace e3 {
namespace {

constexpr int D = 128;
constexpr int BK = 128;                 // keys of a tile
constexpr int BT = 64;                  // nodes of the tree's tile
constexpr int KS = 3, VS = 2, VB = 2;   // stages: K codes, V codes, V in fp16
constexpr int INFO = 8;                 // tiles whose scales are on hand
constexpr int NT = 512;
constexpr int V_SHIFT = 6;              // V's fp16 values are 2^6 up: 448 -> 28672
constexpr uint32_t K_TILE = BK * D, V_TILE = 2 * K_TILE;
constexpr uint32_t Q_PART = 128 * D;    // a row tile of one part
constexpr uint32_t OFF_Q = 0;           // [row tile][hi, lo]
constexpr uint32_t OFF_K = OFF_Q + 4 * Q_PART;
constexpr uint32_t OFF_VR = OFF_K + KS * K_TILE;
constexpr uint32_t OFF_V = OFF_VR + VS * K_TILE;
constexpr uint32_t SMEM_DYN = OFF_V + VB * V_TILE + 1024;   // + alignment slack
constexpr uint32_t TM_O = 0, TM_S = 256;                    // each [stream] * 128 columns
constexpr int REGS_FEW = 64, REGS_SOFTMAX = 192;            // 2 * 128 * (64 + 192) = 65536 registers
constexpr int MERGE_WARPS = 8;

struct Smem {
    uint64_t k_full[KS], k_empty[KS], vr_full[VS], vr_empty[VS], v_full[VB], v_empty[VB];
    uint64_t s_full[2], p_full[2], pv_done[2], o_free[2];
    uint64_t q_full, q_empty;
    uint64_t info_full[INFO];
    uint64_t u_full[2], u_empty[2], r_full[2];   // by unit parity
    uint64_t x_full, x_empty;                    // stream 1's statistics, one row tile only
    uint64_t mma_done[2];
    uint64_t anc[2][64];
    float qf[2][256];
    float info_f[INFO][2];                       // score factors of the tile's two halves
    int info_keys[INFO];                         // keys of the tile that are there, -1: the tree
    int ev[2], tree_kb[2], odd_v[2];
    float x_m[128], x_l[128];
    long long warp_sum[NT / 32];
    long long start_off, total;
    int start_b, start_k;
    uint32_t tmem_base;
    int abort_flag;
};
static_assert(SMEM_DYN + sizeof(Smem) <= 232448, "shared memory budget");

struct Wide {
    CacheAttn a;
    int tiles2;                     // two row tiles (else one)
    int rows_per_group, row_groups, heads;   // heads = Hkv * row_groups: units of a sequence
    int least;                      // tiles of a range, at least, where there are fewer than CTAs want
    WaitRule wait;
    // workspace: tiles before each sequence [B + 1], then {total tiles of all units, CTAs that have any}; where each
    // CTA begins (tile of its first unit); partial results [2 * CTAs][rows_per_group]
    long long *cum;
    int4 *start;
    float *part_o, *part_ml;
};

E3_DEV int seq_len(const CacheAttn &a, int b) { return max(0, min(__ldg(a.prefix_len + b), a.max_prefix)); }
E3_DEV int seq_tiles(const CacheAttn &a, int L) { return max(1, (L + BK - 1) / BK + (a.tree_k ? 1 : 0)); }

// Tiles of a stream before the CTA's tile t
E3_DEV uint32_t stream_tiles(bool two, int m, uint32_t t) { return two ? t : (t + 1u - (uint32_t)m) >> 1; }

// A role's walk over its CTA's range
struct Walk {
    int b, k, i0, i1, nt, L, n;     // sequence, unit of the sequence, tiles [i0, i1) of nt, units so far
    long long left;
    E3_DEV bool begin(const Wide &p, const Smem &s, long long range) {
        b = s.start_b;
        k = s.start_k;
        left = range;
        n = 0;
        if (left <= 0) return false;
        L = seq_len(p.a, b);
        nt = seq_tiles(p.a, L);
        i0 = (int)s.start_off;
        i1 = (int)min((long long)nt, i0 + left);
        return true;
    }
    E3_DEV bool next(const Wide &p) {
        left -= i1 - i0;
        if (left <= 0) return false;
        ++n;
        if (++k == p.heads) {
            k = 0;
            ++b;
            L = seq_len(p.a, b);
            nt = seq_tiles(p.a, L);
        }
        i0 = 0;
        i1 = (int)min((long long)nt, left);
        return true;
    }
    E3_DEV bool is_tree(const Wide &p, int i) const { return p.a.tree_k && i == nt - 1; }
};

E3_DEV uint32_t hmul2(uint32_t a, uint32_t b) {
    const __half2 r = __hmul2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&r);
}

// 8 fp32 as the two e4m3 parts, 8 bytes each (what is not finite: NaN)
E3_DEV void two_parts(const float (&v)[8], uint2 &hi, uint2 &lo) {
    uint32_t h[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        h[i] = to_e4m3x2(v[2 * i], v[2 * i + 1]);
        const float2 back = from_e4m3x2(h[i]);
        l[i] = to_e4m3x2(v[2 * i] - back.x, v[2 * i + 1] - back.y);
    }
    hi = make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
    lo = make_uint2(l[0] | l[1] << 16, l[2] | l[3] << 16);
}

E3_DEV void bf16x8(uint4 u, float (&v)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

E3_DEV float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

E3_DEV float weight_of(float m, float l, float M) {
    return l == 0.0f ? 0.0f : m == -INFINITY ? 1.0f : fast_exp2(m - M);
}

__global__ void __launch_bounds__(NT, 1)
    cache_attn_wide_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                           const __grid_constant__ Wide p) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ Smem ss;
    const uint32_t sm = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t abort = smem_u32(&ss.abort_flag), limit = p.wait.limit;
    const CacheAttn &a = p.a;
    const bool two = p.tiles2 != 0;
    auto bar = [](uint64_t &b) { return smem_u32(&b); };

    if (tid == 0) {
        for (int s = 0; s < KS; ++s) {
            tc::mbar_init(&ss.k_full[s], 1 + missing_arrivals(p.wait, s, 0));
            tc::mbar_init(&ss.k_empty[s], 1);
        }
        for (int s = 0; s < VS; ++s) {
            tc::mbar_init(&ss.vr_full[s], 1);
            tc::mbar_init(&ss.vr_empty[s], 4);
        }
        for (int s = 0; s < VB; ++s) {
            tc::mbar_init(&ss.v_full[s], 4);
            tc::mbar_init(&ss.v_empty[s], 1);
        }
        for (int m = 0; m < 2; ++m) {
            tc::mbar_init(&ss.s_full[m], 1);
            tc::mbar_init(&ss.p_full[m], 4);
            tc::mbar_init(&ss.pv_done[m], 1);
            tc::mbar_init(&ss.o_free[m], 4);
            tc::mbar_init(&ss.u_full[m], 1);
            tc::mbar_init(&ss.u_empty[m], 12);
            tc::mbar_init(&ss.r_full[m], 4);
            tc::mbar_init(&ss.mma_done[m], 1);
        }
        for (int i = 0; i < INFO; ++i) tc::mbar_init(&ss.info_full[i], 1);
        tc::mbar_init(&ss.q_full, 4);
        tc::mbar_init(&ss.q_empty, 1);
        tc::mbar_init(&ss.x_full, 4);
        tc::mbar_init(&ss.x_empty, 4);
        ss.abort_flag = 0;
        ss.start_b = 0;
        tc::fence_barrier_init();
        tc::prefetch_tmap(&tm_k);
        tc::prefetch_tmap(&tm_v);
    }
    if (warp == 1) tc::tmem_alloc(&ss.tmem_base, 512);
    pdl_wait();
    pdl_trigger();

    // ---- this CTA's range: the tiles of all sequences summed up, then the sequence that holds its first
    long long total, range_lo, range_hi;
    {
        auto tiles_at = [&](int b) { return b < a.B ? (long long)seq_tiles(a, seq_len(a, b)) : 0ll; };
        // sum of the block's values before this thread's (inclusive of them in `all` for the whole block)
        auto scan = [&](long long v, long long &all) {
            long long x = v;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const long long y = __shfl_up_sync(0xffffffffu, x, d);
                if (lane >= d) x += y;
            }
            if (lane == 31) ss.warp_sum[warp] = x;
            __syncthreads();
            long long before = 0;
            all = 0;
            for (int w = 0; w < NT / 32; ++w) {
                if (w < warp) before += ss.warp_sum[w];
                all += ss.warp_sum[w];
            }
            __syncthreads();
            return before + x - v;
        };
        long long seqs = 0;
        for (int b0 = 0; b0 < a.B; b0 += NT) {
            long long all;
            const long long before = scan(tiles_at(b0 + tid), all);
            if (blockIdx.x == 0 && p.cum && b0 + tid < a.B) p.cum[b0 + tid] = seqs + before;
            seqs += all;
        }
        total = seqs * p.heads;
        // as many CTAs as leave each `least` tiles
        const long long ctas = max(1ll, min((long long)gridDim.x, total / p.least));
        if (blockIdx.x == 0 && tid == 0 && p.cum) {
            p.cum[a.B] = seqs;
            p.cum[a.B + 1] = total;
            p.cum[a.B + 2] = ctas;
        }
        const bool idle = blockIdx.x >= ctas;
        range_lo = idle ? total : blockIdx.x * total / ctas;
        range_hi = idle ? total : (blockIdx.x + 1) * total / ctas;
        if (!idle) {
            seqs = 0;
            for (int b0 = 0; b0 < a.B; b0 += NT) {
                long long all;
                const long long mine = tiles_at(b0 + tid), before = seqs + scan(mine, all);
                if (mine > 0 && before * p.heads <= range_lo && range_lo < (before + mine) * p.heads) {
                    const long long at = range_lo - before * p.heads;
                    ss.start_b = b0 + tid;
                    ss.start_k = (int)(at / mine);
                    ss.start_off = at % mine;
                    if (p.start) p.start[blockIdx.x] = make_int4(b0 + tid, (int)(at / mine), (int)(at % mine), 0);
                }
                seqs += all;
            }
        }
    }
    const long long range = range_hi - range_lo;
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = ss.tmem_base;

    // (each branch gives or takes by itself: the compiler allots registers by branch)
    Walk w;
    if (warp == 0) {
        // ------------------------------------------------------------------ TMA
        tc::registers_give<REGS_FEW>();
        if (tc::elect_one()) {
            uint32_t t = 0, tv = 0;
            bool ok = true;
            for (bool more = w.begin(p, ss, range); more && ok; more = ok && w.next(p)) {
                const int g = w.k / p.row_groups, sgroups = a.block_size / EAGLE3_KV_GROUP;
                const int32_t *bt = a.block_table + (size_t)w.b * a.max_blocks;
                for (int i = w.i0; i < w.i1; ++i, ++t) {
                    const int s = (int)(t % KS);
                    if (w.is_tree(p, i)) continue;   // (warps 4..7 fill that stage)
                    if (!tc::mbar_wait(bar(ss.k_empty[s]), ((t / KS) & 1u) ^ 1u, abort, limit)) {
                        ok = false;
                        break;
                    }
                    // two groups of 64 places; one that is not there starts above the pool and reads as zeros
                    int row[2];
                    float f[2];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int pos = i * BK + h * 64;
                        row[h] = -64;
                        f[h] = 1.0f;
                        if (pos >= w.L) continue;
                        const int page = __ldg(bt + pos / a.block_size), place = pos % a.block_size;
                        if (page < 0 || page >= a.n_pages) continue;
                        row[h] = (page * a.Hkv + g) * a.block_size + place;
                        f[h] = scale_of(__ldg(a.ks + ((size_t)page * a.Hkv + g) * sgroups + place / EAGLE3_KV_GROUP));
                    }
                    ss.info_f[t % INFO][0] = f[0];
                    ss.info_f[t % INFO][1] = f[1];
                    ss.info_keys[t % INFO] = min(BK, w.L - i * BK);
                    tc::mbar_arrive(bar(ss.info_full[t % INFO]));
                    tc::mbar_expect_tx(bar(ss.k_full[s]), K_TILE);
                    const uint32_t dst = sm + OFF_K + s * K_TILE;
                    tc::tma_load_2d(dst, &tm_k, 0, row[0], bar(ss.k_full[s]));
                    tc::tma_load_2d(dst + K_TILE / 2, &tm_k, 0, row[1], bar(ss.k_full[s]));
                    const int sv = (int)(tv % VS);
                    if (!tc::mbar_wait(bar(ss.vr_empty[sv]), ((tv / VS) & 1u) ^ 1u, abort, limit)) {
                        ok = false;
                        ++t;
                        break;
                    }
                    tc::mbar_expect_tx(bar(ss.vr_full[sv]), K_TILE);
                    const uint32_t dv = sm + OFF_VR + sv * K_TILE;
                    tc::tma_load_2d(dv, &tm_v, 0, row[0], bar(ss.vr_full[sv]));
                    tc::tma_load_2d(dv + K_TILE / 2, &tm_v, 0, row[1], bar(ss.vr_full[sv]));
                    ++tv;
                }
            }
            if (!ok) flag(a.dev_status, EAGLE3_DEV_TIMEOUT);
            // no TMA write may be in flight when the CTA exits: the last load of every stage
            const uint32_t t0 = tc::kiloclock();
            for (uint32_t u = t > KS ? t - KS : 0; u < t; ++u) tc::mbar_drain(bar(ss.k_full[u % KS]), (u / KS) & 1u, t0, limit);
            for (uint32_t u = tv > VS ? tv - VS : 0; u < tv; ++u)
                tc::mbar_drain(bar(ss.vr_full[u % VS]), (u / VS) & 1u, t0, limit);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------------ S = Q K^T
        tc::registers_give<REGS_FEW>();
        if (tc::elect_one()) {
            constexpr uint32_t IDESC = tc::idesc_e4m3(128, BK), IDESC_T = tc::idesc_e4m3(128, BT);
            uint32_t t = 0;
            bool ok = true;
            for (bool more = w.begin(p, ss, range); more && ok; more = ok && w.next(p)) {
                ok = tc::mbar_wait(bar(ss.q_full), w.n & 1u, abort, limit);
                for (int i = w.i0; i < w.i1 && ok; ++i, ++t) {
                    const int s = (int)(t % KS);
                    if (!tc::mbar_wait(bar(ss.k_full[s]), (t / KS) & 1u, abort, limit)) {
                        ok = false;
                        break;
                    }
                    const bool tree = w.is_tree(p, i);
                    const uint32_t kaddr = sm + OFF_K + s * K_TILE;
                    const int m0 = two ? 0 : (int)(t & 1u), m1 = two ? 2 : m0 + 1;
                    for (int m = m0; m < m1; ++m) {
                        // the buffer last held the weights of the stream's tile before
                        const uint32_t n = stream_tiles(two, m, t);
                        if (n > 0 && !tc::mbar_wait(bar(ss.pv_done[m]), (n - 1) & 1u, abort, limit)) {
                            ok = false;
                            break;
                        }
                        tc::fence_after();
                        const uint32_t d = tmem + TM_S + (uint32_t)(m * 128);
                        const uint32_t q = sm + OFF_Q + (two ? m : 0) * 2 * Q_PART;
                        if (!tree) {
#pragma unroll
                            for (int k = 0; k < 8; ++k)   // hi, then lo
                                tc::mma_e4m3_ss(d, tc::desc_sw128(q + (k >> 2) * Q_PART + (k & 3) * 32),
                                                tc::desc_sw128(kaddr + (k & 3) * 32), IDESC, k > 0 ? 1u : 0u);
                        } else {
#pragma unroll
                            for (int k = 0; k < 16; ++k)   // K in two parts too
                                tc::mma_e4m3_ss(d, tc::desc_sw128(q + ((k >> 2) & 1) * Q_PART + (k & 3) * 32),
                                                tc::desc_sw128(kaddr + (k >> 3) * (K_TILE / 2) + (k & 3) * 32), IDESC_T,
                                                k > 0 ? 1u : 0u);
                        }
                        tc::mma_commit(bar(ss.s_full[m]));
                    }
                    if (ok) tc::mma_commit(bar(ss.k_empty[s]));
                }
                if (ok) tc::mma_commit(bar(ss.q_empty));
            }
            if (!ok) flag(a.dev_status, EAGLE3_DEV_TIMEOUT);
            tc::mma_commit(bar(ss.mma_done[0]));
            tc::mbar_drain(bar(ss.mma_done[0]), 0, tc::kiloclock(), limit);
        }
        __syncwarp();
    } else if (warp == 2) {
        // ------------------------------------------------------------------ O += P V
        tc::registers_give<REGS_FEW>();
        if (tc::elect_one()) {
            constexpr uint32_t IDESC = tc::idesc_f16_bmn(128, D);
            uint32_t t = 0;
            bool ok = true;
            for (bool more = w.begin(p, ss, range); more && ok; more = ok && w.next(p)) {
                for (int i = w.i0; i < w.i1 && ok; ++i, ++t) {
                    const int s = (int)(t % VB);
                    if (!tc::mbar_wait(bar(ss.v_full[s]), (t / VB) & 1u, abort, limit)) {
                        ok = false;
                        break;
                    }
                    const int ksteps = (w.is_tree(p, i) ? BT : BK) / 16;
                    const uint32_t vaddr = sm + OFF_V + s * V_TILE;
                    const int m0 = two ? 0 : (int)(t & 1u), m1 = two ? 2 : m0 + 1;
                    const bool fresh = i - w.i0 < (two ? 1 : 2);   // the stream's first of the unit
                    for (int m = m0; m < m1; ++m) {
                        // (a unit's first overwrites O: the one before it must have been read)
                        if (!tc::mbar_wait(bar(ss.p_full[m]), stream_tiles(two, m, t) & 1u, abort, limit) ||
                            (fresh && w.n > 0 && !tc::mbar_wait(bar(ss.o_free[m]), (w.n - 1) & 1u, abort, limit))) {
                            ok = false;
                            break;
                        }
                        tc::fence_after();
                        const uint32_t t_p = tmem + TM_S + (uint32_t)(m * 128);
                        for (int kk = 0; kk < ksteps; ++kk)
                            tc::mma_bf16_ts(tmem + TM_O + (uint32_t)(m * 128), t_p + (uint32_t)(kk * 8),
                                            tc::desc_mn_sw128(vaddr + kk * 2048, V_TILE / 2, 1024), IDESC,
                                            !fresh || kk > 0 ? 1u : 0u);
                        tc::mma_commit(bar(ss.pv_done[m]));
                    }
                    if (ok) tc::mma_commit(bar(ss.v_empty[s]));
                }
            }
            if (!ok) flag(a.dev_status, EAGLE3_DEV_TIMEOUT);
            tc::mma_commit(bar(ss.mma_done[1]));
            tc::mbar_drain(bar(ss.mma_done[1]), 0, tc::kiloclock(), limit);
        }
        __syncwarp();
    } else if (warp == 3) {
        // ------------------------------------------------------------------ a unit ahead
        tc::registers_give<REGS_FEW>();
        bool ok = true;
        for (bool more = w.begin(p, ss, range); more && ok; more = ok && w.next(p)) {
            const int u = w.n & 1;
            if (w.n >= 2 && !tc::mbar_wait_warp(bar(ss.u_empty[u]), ((w.n - 2) >> 1) & 1u, abort, limit)) {
                ok = false;
                break;
            }
            const int g = w.k / p.row_groups, sgroups = a.block_size / EAGLE3_KV_GROUP;
            const int32_t *bt = a.block_table + (size_t)w.b * a.max_blocks;
            const bool tree = a.tree_k && w.i1 == w.nt;
            const int g0 = w.i0 * 2, g1 = (int)(((long long)min((long long)w.L, (long long)w.i1 * BK) + 63) / 64);
            int ev = 1;
            for (int x = g0 + lane; x < g1; x += 32) {
                const int pos = x * 64, page = __ldg(bt + pos / a.block_size), place = pos % a.block_size;
                if (page < 0 || page >= a.n_pages) continue;
                const int e = __ldg(a.vs + ((size_t)page * a.Hkv + g) * sgroups + place / EAGLE3_KV_GROUP);
                if (e != 255) ev = max(ev, e);
            }
            bool odd_k = false, odd_v = false;
            float km = 0.0f;
            if (tree) {
                const __nv_bfloat16 *tk = a.tree_k + (size_t)w.b * a.N * a.kv_ns + (size_t)g * D;
                const __nv_bfloat16 *tv = a.tree_v + (size_t)w.b * a.N * a.kv_ns + (size_t)g * D;
                float vm = 0.0f;
                for (int x = lane; x < a.N * (D / 8); x += 32) {
                    const int64_t at = (x >> 4) * a.kv_ns + (x & 15) * 8;
                    km = fmaxf(km, amax8(*reinterpret_cast<const uint4 *>(tk + at), odd_k));
                    vm = fmaxf(vm, amax8(*reinterpret_cast<const uint4 *>(tv + at), odd_v));
                }
                ev = max(ev, scale_byte(vm));
                for (int i = lane; i < a.N; i += 32) {
                    bool bad = false;
                    ss.anc[u][i] = path_bits(a.parents + (size_t)w.b * a.N, i, bad);
                    if (bad && w.k == 0) flag(a.dev_status, EAGLE3_DEV_BAD_TREE);
                }
            }
#pragma unroll
            for (int x = 16; x; x >>= 1) {
                ev = max(ev, __shfl_xor_sync(0xffffffffu, ev, x));
                km = fmaxf(km, __shfl_xor_sync(0xffffffffu, km, x));
            }
            odd_v = __any_sync(0xffffffffu, odd_v);
            if (lane == 0) {
                ss.ev[u] = ev;
                ss.tree_kb[u] = scale_byte(km);
                ss.odd_v[u] = tree && odd_v;
                const int L = __ldg(a.prefix_len + w.b);
                if ((L < 0 || L > a.max_prefix) && w.k == 0 && w.i0 == 0) flag(a.dev_status, EAGLE3_DEV_CAPACITY);
            }
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(bar(ss.u_full[u]));
        }
        if (!ok && lane == 0) flag(a.dev_status, EAGLE3_DEV_TIMEOUT);
    } else if (warp < 8) {
        // ------------------------------------------------------------------ conversions
        tc::registers_give<REGS_FEW>();
        const int cw = warp - 4;
        uint32_t t = 0, tv = 0;
        bool ok = true;
        for (bool more = w.begin(p, ss, range); more && ok; more = ok && w.next(p)) {
            const int u = w.n & 1, g = w.k / p.row_groups, row0 = w.k % p.row_groups * p.rows_per_group;
            if (!tc::mbar_wait_warp(bar(ss.u_full[u]), (w.n >> 1) & 1u, abort, limit) ||
                (w.n > 0 && !tc::mbar_wait_warp(bar(ss.q_empty), (w.n - 1) & 1u, abort, limit))) {
                ok = false;
                break;
            }
            // ---- Q's parts: 16 lanes a row, two rows at a time
            const int nrows = min(p.rows_per_group, a.N * a.rep - row0);
#pragma unroll 4
            for (int it = 0; it < p.rows_per_group / 8; ++it) {
                const int row = it * 8 + cw * 2 + (lane >> 4), c = lane & 15;
                uint4 x = make_uint4(0, 0, 0, 0);
                if (row < nrows) {
                    const int node = (row0 + row) / a.rep, head = g * a.rep + (row0 + row) % a.rep;
                    x = *reinterpret_cast<const uint4 *>(a.q + ((size_t)w.b * a.N + node) * a.q_ns + (size_t)head * D + c * 8);
                }
                bool odd = false;
                float top = amax8(x, odd);
#pragma unroll
                for (int d = 8; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                const int byte = scale_byte(top);
                const float up = inverse_scale(byte);
                float v[8];
                bf16x8(x, v);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = fabsf(v[e]) <= FLT_MAX ? v[e] * up : __int_as_float(0x7fc00000);
                uint2 hi, lo;
                two_parts(v, hi, lo);
                const uint32_t at = sm + OFF_Q + (row >> 7) * 2 * Q_PART + (row & 127) * 128 +
                                    ((((uint32_t)c >> 1) ^ ((uint32_t)row & 7u)) << 4) + (c & 1) * 8;
                asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(at), "r"(hi.x), "r"(hi.y) : "memory");
                asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(at + Q_PART), "r"(lo.x), "r"(lo.y) : "memory");
                if (c == 0) ss.qf[u][row] = a.scale_log2 * scale_of(byte);
            }
            const int evref = ss.ev[u];
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                tc::mbar_arrive(bar(ss.q_full));
                tc::mbar_arrive(bar(ss.r_full[u]));
            }
            const int sgroups = a.block_size / EAGLE3_KV_GROUP;
            const int32_t *bt = a.block_table + (size_t)w.b * a.max_blocks;
            for (int i = w.i0; i < w.i1; ++i, ++t) {
                const int s = (int)(t % VB);
                const uint32_t dst = sm + OFF_V + s * V_TILE;
                if (w.is_tree(p, i)) {
                    // ---- the tree: K in two parts into its stage, V in fp16
                    if (!tc::mbar_wait_warp(bar(ss.k_empty[t % KS]), ((t / KS) & 1u) ^ 1u, abort, limit) ||
                        !tc::mbar_wait_warp(bar(ss.v_empty[s]), ((t / VB) & 1u) ^ 1u, abort, limit)) {
                        ok = false;
                        break;
                    }
                    const uint32_t kd = sm + OFF_K + (t % KS) * K_TILE;
                    const int kb = ss.tree_kb[u];
                    const float kup = inverse_scale(kb), vup = inverse_scale(evref) * (float)(1 << V_SHIFT);
                    const size_t base = (size_t)w.b * a.N * a.kv_ns + (size_t)g * D;
#pragma unroll 2
                    for (int it = 0; it < BT / 8; ++it) {
                        const int row = it * 8 + cw * 2 + (lane >> 4), c = lane & 15;
                        uint4 xk = make_uint4(0, 0, 0, 0), xv = xk;
                        if (row < a.N) {
                            xk = *reinterpret_cast<const uint4 *>(a.tree_k + base + row * a.kv_ns + c * 8);
                            xv = *reinterpret_cast<const uint4 *>(a.tree_v + base + row * a.kv_ns + c * 8);
                        }
                        float v[8];
                        bf16x8(xk, v);
#pragma unroll
                        for (int e = 0; e < 8; ++e) v[e] = fabsf(v[e]) <= FLT_MAX ? v[e] * kup : __int_as_float(0x7fc00000);
                        uint2 hi, lo;
                        two_parts(v, hi, lo);
                        const uint32_t at = kd + row * 128 + ((((uint32_t)c >> 1) ^ ((uint32_t)row & 7u)) << 4) + (c & 1) * 8;
                        asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(at), "r"(hi.x), "r"(hi.y) : "memory");
                        asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(at + K_TILE / 2), "r"(lo.x), "r"(lo.y) : "memory");
                        bf16x8(xv, v);
                        uint32_t h[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float x0 = v[2 * e], x1 = v[2 * e + 1];
                            h[e] = pack_f16(fabsf(x0) <= FLT_MAX ? x0 * vup : 0.0f, fabsf(x1) <= FLT_MAX ? x1 * vup : 0.0f);
                        }
                        const uint32_t av = dst + (c >> 3) * (V_TILE / 2) + row * 128 +
                                            (((uint32_t)c & 7u) ^ ((uint32_t)row & 7u)) * 16;
                        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(av), "r"(h[0]), "r"(h[1]), "r"(h[2]),
                                     "r"(h[3])
                                     : "memory");
                    }
                    tc::fence_proxy_async_smem();
                    asm volatile("bar.sync 1, 128;" ::: "memory");   // all of K is there: one arrival
                    if (cw == 0 && lane == 0) {
                        ss.info_f[t % INFO][0] = ss.info_f[t % INFO][1] = scale_of(kb);
                        ss.info_keys[t % INFO] = -1;
                        tc::mbar_arrive(bar(ss.info_full[t % INFO]));
                        tc::mbar_arrive(bar(ss.k_full[t % KS]));
                    }
                    if (lane == 0) tc::mbar_arrive(bar(ss.v_full[s]));
                    continue;
                }
                // ---- V's codes of 32 keys a warp (all in one group): 8 lanes a key
                const int sv = (int)(tv % VS);
                const int pos = i * BK + cw * 32;
                int e = 1;
                if (pos < w.L) {
                    const int page = __ldg(bt + pos / a.block_size), place = pos % a.block_size;
                    if (page >= 0 && page < a.n_pages)
                        e = __ldg(a.vs + ((size_t)page * a.Hkv + g) * sgroups + place / EAGLE3_KV_GROUP);
                }
                // 2^(e - evref + V_SHIFT) in fp16: 0 where it is below its smallest
                const float vs = e == 255 ? __int_as_float(0x7fc00000) : exp2_int(e - evref + V_SHIFT);
                const uint32_t vs2 = pack_f16(vs, vs);
                if (!tc::mbar_wait_warp(bar(ss.vr_full[sv]), (tv / VS) & 1u, abort, limit) ||
                    !tc::mbar_wait_warp(bar(ss.v_empty[s]), ((t / VB) & 1u) ^ 1u, abort, limit)) {
                    ok = false;
                    break;
                }
                const uint32_t src = sm + OFF_VR + sv * K_TILE;
                const int c = lane & 7;
#pragma unroll
                for (int it = 0; it < 8; ++it) {
                    const int key = cw * 32 + it * 4 + (lane >> 3);
                    uint32_t x[4];
                    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                                 : "r"(src + key * 128 + (((uint32_t)c ^ ((uint32_t)key & 7u)) << 4)));
                    if (i * BK + key >= w.L) x[0] = x[1] = x[2] = x[3] = 0;   // whatever lies behind the last key
                    uint32_t y[8];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        y[2 * q] = hmul2(e4m3x2_f16(x[q]), vs2);
                        y[2 * q + 1] = hmul2(e4m3x2_f16(x[q] >> 16), vs2);
                    }
                    // 16 dims: two chunks of a block of 64; the upper block's lanes store theirs in the other order, so
                    // that 8 lanes fill all banks
                    const uint32_t blk = dst + (c >> 2) * (V_TILE / 2) + key * 128;
                    const bool swap = c >= 4;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t ch = (uint32_t)(2 * c + (swap ? 1 - h : h)) & 7u;
                        const uint32_t at = blk + ((ch ^ ((uint32_t)key & 7u)) << 4);
                        const bool second = swap ? h == 0 : h == 1;
                        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(second ? y[4] : y[0]),
                                     "r"(second ? y[5] : y[1]), "r"(second ? y[6] : y[2]), "r"(second ? y[7] : y[3])
                                     : "memory");
                    }
                }
                tc::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    tc::mbar_arrive(bar(ss.vr_empty[sv]));
                    tc::mbar_arrive(bar(ss.v_full[s]));
                }
                ++tv;
            }
            __syncwarp();
            if (ok && lane == 0) tc::mbar_arrive(bar(ss.u_empty[u]));
        }
        if (!ok && lane == 0) flag(a.dev_status, EAGLE3_DEV_TIMEOUT);
    } else {
        // ------------------------------------------------------------------ softmax and results
        tc::registers_take<REGS_SOFTMAX>();
        const int m = (warp - 8) >> 2, r = (warp & 3) * 32 + lane;   // stream, TMEM lane
        const uint32_t t_lane = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t t_s = t_lane + TM_S + (uint32_t)(m * 128), t_o = t_lane + TM_O + (uint32_t)(m * 128);
        uint32_t t = 0;
        bool ok = true;
        for (bool more = w.begin(p, ss, range); more && ok; more = ok && w.next(p)) {
            const int u = w.n & 1, g = w.k / p.row_groups, row0 = w.k % p.row_groups * p.rows_per_group;
            const int row = two ? m * 128 + r : r, nrows = min(p.rows_per_group, a.N * a.rep - row0);
            if (!tc::mbar_wait_warp(bar(ss.u_full[u]), (w.n >> 1) & 1u, abort, limit) ||
                !tc::mbar_wait_warp(bar(ss.r_full[u]), (w.n >> 1) & 1u, abort, limit)) {
                ok = false;
                break;
            }
            const float fr = ss.qf[u][row];
            uint64_t anc = 0;
            if (a.tree_k && w.i1 == w.nt && row < nrows) anc = ss.anc[u][(row0 + row) / a.rep];
            float m_run = -INFINITY, l_run = 0.0f;
            bool fresh = true;
            for (int i = w.i0; i < w.i1; ++i, ++t) {
                if (!two && (int)(t & 1u) != m) continue;
                if (!tc::mbar_wait_warp(bar(ss.info_full[t % INFO]), (t / INFO) & 1u, abort, limit) ||
                    !tc::mbar_wait_warp(bar(ss.s_full[m]), stream_tiles(two, m, t) & 1u, abort, limit)) {
                    ok = false;
                    break;
                }
                tc::fence_after();
                float sc[128];
#pragma unroll
                for (int q = 0; q < 4; ++q) tc::tmem_ld32_start(t_s + 32u * q, sc + 32 * q);
                // (a factor that underflows would make NaN of the masked scores; a NaN stays)
                float f0 = fr * ss.info_f[t % INFO][0], f1 = fr * ss.info_f[t % INFO][1];
                f0 = f0 < FLT_MIN ? FLT_MIN : f0;
                f1 = f1 < FLT_MIN ? FLT_MIN : f1;
                const int keys = ss.info_keys[t % INFO];
#pragma unroll
                for (int q = 0; q < 4; ++q) tc::tmem_ld32_wait(sc + 32 * q);
                if (keys < BK) {
                    uint32_t vis[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int n = keys - 32 * q;
                        vis[q] = keys < 0 ? (q < 2 ? (uint32_t)(anc >> (32 * q)) : 0u)
                                          : n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1u;
                    }
#pragma unroll
                    for (int e = 0; e < 128; ++e) sc[e] = (vis[e >> 5] >> (e & 31)) & 1u ? sc[e] : -INFINITY;
                }
                float mq[2][2] = {{-INFINITY, -INFINITY}, {-INFINITY, -INFINITY}};
#pragma unroll
                for (int e = 0; e < 128; e += 2) mq[e >> 6][(e >> 1) & 1] = max3(mq[e >> 6][(e >> 1) & 1], sc[e], sc[e + 1]);
                const float mx = fmaxf(fmaxf(mq[0][0], mq[0][1]) * f0, fmaxf(mq[1][0], mq[1][1]) * f1);
                const bool need = mx > m_run + RESCALE_LOG2;
                if (__any_sync(0xffffffffu, need)) {
                    const float m_new = need ? mx : m_run;
                    const float corr = need ? (m_run == -INFINITY ? 0.0f : fast_exp2(m_run - m_new)) : 1.0f;
                    l_run *= corr;
                    m_run = m_new;
                    // (the weights of the tile before have been multiplied: S waited for that)
                    if (!fresh) {
#pragma unroll 1
                        for (int q = 0; q < 4; ++q) {
                            float o[32];
                            tc::tmem_ld32(t_o + 32u * q, o);
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] *= corr;
                            tc::tmem_st32(t_o + 32u * q, o);
                        }
                    }
                }
                fresh = false;
                const float nm = m_run == -INFINITY ? 0.0f : WEIGHT_LOG2 - m_run;
                const float2 nm2 = make_float2(nm, nm);
                float2 sum[2] = {{0.0f, 0.0f}, {0.0f, 0.0f}};
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const float f = q ? f1 : f0;
                    const float2 f2 = make_float2(f, f);
                    uint32_t pk[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        const float2 x = __ffma2_rn(make_float2(sc[64 * q + 2 * e], sc[64 * q + 2 * e + 1]), f2, nm2);
                        const float2 y = make_float2(fast_exp2(x.x), fast_exp2(x.y));
                        sum[e & 1] = __fadd2_rn(sum[e & 1], y);
                        pk[e] = pack_f16(y.x, y.y);
                    }
                    tc::tmem_st32u(t_s + 32u * q, pk);
                }
                const float2 s2 = __fadd2_rn(sum[0], sum[1]);
                l_run += s2.x + s2.y;
                tc::fence_before();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(bar(ss.p_full[m]));
            }
            if (!ok) break;
            // ---- the unit's results
            float e0 = 1.0f, e1 = 0.0f, M = m_run, l = l_run;
            if (!two) {
                if (m == 1) {
                    if (w.n > 0 && !tc::mbar_wait_warp(bar(ss.x_empty), (w.n - 1) & 1u, abort, limit)) {
                        ok = false;
                        break;
                    }
                    ss.x_m[r] = m_run;
                    ss.x_l[r] = l_run;
                    __syncwarp();
                    if (lane == 0) {
                        tc::mbar_arrive(bar(ss.x_full));
                        tc::mbar_arrive(bar(ss.u_empty[u]));
                    }
                    continue;
                }
                if (!tc::mbar_wait_warp(bar(ss.x_full), w.n & 1u, abort, limit)) {
                    ok = false;
                    break;
                }
                const float m2 = ss.x_m[r], l2 = ss.x_l[r];
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(bar(ss.x_empty));
                M = fmaxf(m_run, m2);
                e0 = weight_of(m_run, l_run, M);
                e1 = weight_of(m2, l2, M);
                l = e0 * l_run + e1 * l2;
                const uint32_t n1 = stream_tiles(false, 1, t);
                if (n1 > 0 && !tc::mbar_wait_warp(bar(ss.pv_done[1]), (n1 - 1) & 1u, abort, limit)) {
                    ok = false;
                    break;
                }
            }
            const uint32_t done = stream_tiles(two, m, t);
            if (done > 0 && !tc::mbar_wait_warp(bar(ss.pv_done[m]), (done - 1) & 1u, abort, limit)) {
                ok = false;
                break;
            }
            tc::fence_after();
            const bool whole = w.i0 == 0 && w.i1 == w.nt;
            const bool mine = row < nrows;
            const int node = (row0 + row) / a.rep, head = g * a.rep + (row0 + row) % a.rep;
            const size_t at = ((size_t)w.b * a.N + (mine ? node : 0)) * a.Hq + (mine ? head : 0);
            const size_t part = (size_t)(2 * blockIdx.x + (w.n > 0 ? 1 : 0)) * p.rows_per_group + row;
            const int evref = ss.ev[u];
            const bool odd_v = ss.odd_v[u] != 0;
            // 2^(evref - 127 - V_SHIFT), in two steps where it is no normal number
            const float vs = scale_of(evref) * (1.0f / (1 << V_SHIFT));
            const float inv = whole ? (l == 0.0f ? 0.0f : 1.0f / l) : 1.0f;
#pragma unroll 1
            for (int q = 0; q < 4; ++q) {
                float o[32];
                tc::tmem_ld32(t_lane + TM_O + 32u * q + (two ? m * 128u : 0u), o);   // warp-collective
                if (!two) {
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = e0 != 0.0f ? o[e] * e0 : 0.0f;
                    float o2[32];
                    tc::tmem_ld32(t_lane + TM_O + 128u + 32u * q, o2);
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = e1 != 0.0f ? o[e] + o2[e] * e1 : o[e];
                } else if (l == 0.0f) {
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = 0.0f;
                }
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] *= vs;
                // infinities and NaN of the tree's values, to the rows that see them
                if (odd_v && mine) {
                    for (int j = 0; j < a.N; ++j) {
                        if (!(anc >> j & 1ull)) continue;
                        const __nv_bfloat16 *tv = a.tree_v + ((size_t)w.b * a.N + j) * a.kv_ns + (size_t)g * D + 32 * q;
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            const float x = (float)tv[e];
                            if (!(fabsf(x) <= FLT_MAX)) o[e] += x;
                        }
                    }
                }
                if (!mine) continue;
                if (whole) {
                    uint4 *dst = reinterpret_cast<uint4 *>(a.out + at * D + 32 * q);
#pragma unroll
                    for (int c8 = 0; c8 < 4; ++c8) {
                        uint32_t x[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const __nv_bfloat162 hv = __floats2bfloat162_rn(o[8 * c8 + 2 * e] * inv, o[8 * c8 + 2 * e + 1] * inv);
                            x[e] = *reinterpret_cast<const uint32_t *>(&hv);
                        }
                        dst[c8] = make_uint4(x[0], x[1], x[2], x[3]);
                    }
                } else {
                    float4 *dst = reinterpret_cast<float4 *>(p.part_o + part * D + 32 * q);
#pragma unroll
                    for (int c4 = 0; c4 < 8; ++c4) dst[c4] = make_float4(o[4 * c4], o[4 * c4 + 1], o[4 * c4 + 2], o[4 * c4 + 3]);
                }
            }
            tc::fence_before();
            __syncwarp();
            if (lane == 0) {
                tc::mbar_arrive(bar(ss.o_free[m]));
                if (!two) tc::mbar_arrive(bar(ss.o_free[1]));
                tc::mbar_arrive(bar(ss.u_empty[u]));
            }
            if (mine) {
                if (whole) {
                    if (a.lse) a.lse[at] = lse_of(M, l);
                } else {
                    *reinterpret_cast<float2 *>(p.part_ml + 2 * part) = make_float2(M, l);
                }
            }
        }
        if (!ok && lane == 0) flag(a.dev_status, EAGLE3_DEV_TIMEOUT);
    }

    tc::fence_before();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc::fence_after();
        tc::tmem_dealloc(tmem, 512);
    }
}

// Joins the units that were cut, in the order of their CTAs: grid (CTA whose range begins inside a unit, rows).
__global__ void __launch_bounds__(MERGE_WARPS * 32) cache_attn_join_kernel(const __grid_constant__ Wide p) {
    pdl_wait();
    pdl_trigger();
    const CacheAttn &a = p.a;
    const long long total = p.cum[a.B + 1], ctas = p.cum[a.B + 2];
    const long long c = blockIdx.x + 1;
    if (c >= ctas) return;
    const int4 st = p.start[c];
    if (st.z == 0) return;                              // begins with a unit
    const long long before = p.cum[st.x], nt = p.cum[st.x + 1] - before;
    const long long u0 = before * p.heads + st.y * nt;
    auto owner = [&](long long x) { return ((x + 1) * ctas - 1) / total; };
    const long long first = owner(u0), last = owner(u0 + nt - 1);
    if (first != c - 1) return;                         // not the unit's first cut
    // the first CTA's share: its second slot, unless its range begins with this unit
    const int4 s1 = p.start[first];
    const long long slot0 = 2 * first + (s1.x == st.x && s1.y == st.y ? 0 : 1);
    const int g = st.y / p.row_groups, row0 = st.y % p.row_groups * p.rows_per_group;
    const int nrows = min(p.rows_per_group, a.N * a.rep - row0), lane = threadIdx.x & 31;
    for (int row = blockIdx.y * MERGE_WARPS + (threadIdx.x >> 5); row < nrows; row += gridDim.y * MERGE_WARPS) {
        auto slot = [&](long long q) { return (size_t)(q == first ? slot0 : 2 * q) * p.rows_per_group + row; };
        float M = -INFINITY, l = 0.0f;
        for (long long q = first; q <= last; ++q) M = fmaxf(M, p.part_ml[2 * slot(q)]);
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (long long q = first; q <= last; ++q) {
            const float2 ml = *reinterpret_cast<const float2 *>(p.part_ml + 2 * slot(q));
            const float e = weight_of(ml.x, ml.y, M);
            const float4 x = *reinterpret_cast<const float4 *>(p.part_o + slot(q) * D + 4 * lane);
            l += e * ml.y;
            if (e != 0.0f) o = make_float4(o.x + e * x.x, o.y + e * x.y, o.z + e * x.z, o.w + e * x.w);
        }
        const int node = (row0 + row) / a.rep, head = g * a.rep + (row0 + row) % a.rep;
        store_row(a, ((size_t)st.x * a.N + node) * a.Hq + head, lane, M, l, o);
    }
}

struct Plan {
    Wide w;
    int ctas;
    size_t o_start, o_part, o_ml, bytes;
};

Plan plan(const CacheAttn &a, int requested) {
    Plan pl;
    Wide &w = pl.w;
    w = Wide();
    w.a = a;
    const int rows = a.N * a.rep;
    w.tiles2 = rows > 128;
    w.rows_per_group = w.tiles2 ? 256 : 128;
    w.row_groups = (rows + w.rows_per_group - 1) / w.rows_per_group;
    w.heads = a.Hkv * w.row_groups;
    const int64_t units = (int64_t)a.B * w.heads;
    const int64_t most = units * ((a.max_prefix + BK - 1) / BK + 1);
    const int64_t sms = device_sm_count() > 0 ? device_sm_count() : 1;
    int64_t ctas = requested > 0 ? units * requested : sms;
    if (ctas > most) ctas = most;
    if (ctas > 4 * 65535) ctas = 4 * 65535;
    w.least = requested > 0 ? 1 : 2;
    pl.ctas = (int)ctas;
    size_t at = 256;
    auto take = [&](size_t n) {
        const size_t o = at;
        at += (n + 255) / 256 * 256;
        return o;
    };
    take(((size_t)a.B + 3) * sizeof(long long));
    pl.o_start = take((size_t)ctas * sizeof(int4));
    pl.o_part = take((size_t)ctas * 2 * w.rows_per_group * D * sizeof(float));
    pl.o_ml = take((size_t)ctas * 2 * w.rows_per_group * 2 * sizeof(float));
    pl.bytes = at;
    return pl;
}

}  // namespace

size_t cache_attn_wide_workspace(const CacheAttn &a, int requested) { return plan(a, requested).bytes; }

eagle3_status_t cache_attn_wide(const CacheAttn &a, int requested, const WaitRule &wait, void *workspace, size_t bytes,
                                cudaStream_t stream) {
    Plan pl = plan(a, requested);
    if (!workspace || bytes < pl.bytes) return EAGLE3_ERR_WORKSPACE;
    uint8_t *ws = (uint8_t *)(((uintptr_t)workspace + 255) & ~(uintptr_t)255);
    pl.w.wait = wait;
    pl.w.cum = (long long *)ws;
    pl.w.start = (int4 *)(ws + pl.o_start - 256);
    pl.w.part_o = (float *)(ws + pl.o_part - 256);
    pl.w.part_ml = (float *)(ws + pl.o_ml - 256);
    const int64_t rows = (int64_t)a.n_pages * a.Hkv * a.block_size;
    CUtensorMap tk, tv;
    if (!tmap_rows(&tk, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, a.kc, (int)rows, D, D, 64) ||
        !tmap_rows(&tv, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, a.vc, (int)rows, D, D, 64))
        return EAGLE3_ERR_CUDA;
    static PerDevice<cudaError_t> attr;
    if (attr.get([] {
            return cudaFuncSetAttribute(cache_attn_wide_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM_DYN);
        }) != cudaSuccess)
        return EAGLE3_ERR_CUDA;
    if (launch_pdl(cache_attn_wide_kernel, dim3((unsigned)pl.ctas), dim3(NT), SMEM_DYN, stream, tk, tv, pl.w) != cudaSuccess)
        return EAGLE3_ERR_CUDA;
    if (pl.ctas > 1 && launch_pdl(cache_attn_join_kernel, dim3((unsigned)(pl.ctas - 1), 8), dim3(MERGE_WARPS * 32), 0, stream,
                                  pl.w) != cudaSuccess)
        return EAGLE3_ERR_CUDA;
    return EAGLE3_OK;
}

}  // namespace e3
