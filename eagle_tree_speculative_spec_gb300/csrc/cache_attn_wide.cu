// eagle3_verify_attn_fp8 for many query rows (trees): the tcgen05 kernel, and the join of what its CTAs shared.
//
// A unit of work is a sequence and a KV head; its query rows (row = node * rep + head) are cut into groups of 128, each with
// a CTA of its own, so that the CTAs of a unit read its keys at about the same time.  Keys come in tiles of 128 places, the
// tree's nodes as one more.  The tiles of all units, one after the other, are cut into equal ranges, one for each CTA (of a
// row group; one CTA an SM): ragged lengths, one long sequence and many short ones are all spread evenly, and a unit is
// cut only where a range ends.  Cut units leave unnormalised partial results, which a second kernel joins in order.
//
// S = Q K^T takes K's codes as they lie in memory: Q is held as two e4m3 parts (row scaled to at most 448; hi = e4m3(q),
// lo = e4m3(q - hi): 4 + 4 bits are bf16's 8), so that QK runs as two e4m3 products, in the time of one of bf16, and K is
// never converted.  The parts stay in tensor memory: read from shared memory for every tile, they would be half of its
// traffic.  P V runs in fp16: weights in 11 bits (8 bits of bf16, or two e4m3 parts whose floor is 2^-18 of the largest
// weight, would cost long sums) and V's codes, converted exactly; the scale of V's group is put on the weights, relative to
// the largest so far, by adding to the exponent.
//
//   warp 0        TMA: K tiles into a ring of 4, V codes into a ring of 2
//   warp 1, 2     the MMAs of S, and of P V (one thread issues an MMA about every 110 cycles: two threads)
//   warp 3        looks ahead: the places and scales of the next 32 tiles, a tile a lane (two dependent loads, which
//                 whoever needs them would wait for tile by tile)
//   warps 4..7    V codes to fp16; Q's parts, row scales and parents of the next unit; the tree's K and V
//   warps 8..15   softmax, two warps for each quarter of the rows, a row a thread: each takes one of the tile's two groups
//                 of 64 keys (so one scale), and they exchange the maxima; at the end of a unit its results
// Tensor memory: O 128 columns, two tiles of S, one of P (fp16 pairs), Q's parts.  S is free for the tile after next once the
// softmax has loaded it, so that QK runs two tiles ahead.
// Bound by its roles' own work: 64 trees of 60 nodes of 4 heads over 2048 positions take 207 us, 0.63 PFLOP/s, where tensor
// operations are 69; over 16384 positions 1049 us, 0.99 PFLOP/s.  A tile takes some 2060 cycles (its two groups of MMAs 1024
// each), a unit 11000 more: Q's parts, the tree and the results, in part beside the units before and after.  The kernel of the
// bf16 cache (verify_attn.cu), as many MMAs a tile, needs no conversions: 1800 cycles a tile, 134 and 882 us for the same
// two.  The loops are short because the roles' code together is more than the SM's instruction cache holds: what is rare is
// out of line, waits share one function, a unit's work runs in loops, not unrolled (307 to 225 us for the first).
// All waits are bounded; one that runs out sets EAGLE3_DEV_TIMEOUT and the CTA drains and exits.
#include "cache_attn.cuh"
#include "tc.cuh"
#include "tmap.cuh"

#include <algorithm>

namespace e3 {
namespace {

constexpr int D = 128;
constexpr int BK = 128;                 // keys of a tile
constexpr int BT = 64;                  // nodes of the tree's tile
constexpr int KS = 4, VS = 2, VB = 3;   // stages: K codes, V codes, V in fp16
constexpr int AHEAD = 32;               // tiles that warp 3 looks up at once, two such batches
constexpr int ROWS = 128;               // query rows of a CTA
constexpr int NT = 512;
constexpr int LEAST_SHIFT = -60;        // of V's scale on the weights: fp16 has nothing left of them long before
constexpr uint32_t K_TILE = BK * D, V_TILE = 2 * K_TILE;
constexpr uint32_t OFF_K = 0;
constexpr uint32_t OFF_VR = OFF_K + KS * K_TILE;
constexpr uint32_t OFF_V = OFF_VR + VS * K_TILE;
constexpr uint32_t OUT_WARP = 32 * 64;   // a softmax warp's 32 rows of 32 outputs in bf16
constexpr uint32_t OFF_OUT = OFF_V + VB * V_TILE;
constexpr uint32_t IN_WARP = 32 * 64;    // a converting warp's 32 rows of 32 query dims
constexpr uint32_t OFF_IN = OFF_OUT + 8 * OUT_WARP;
constexpr uint32_t SMEM_DYN = OFF_IN + 4 * IN_WARP + 1024;   // + alignment slack
// tensor memory, columns: O; S of two tiles; P; Q's parts, 32 columns each
constexpr uint32_t TM_O = 0, TM_S = 128, TM_P = 384, TM_Q = 448;
constexpr int JOIN_WARPS = 8;
constexpr int MOST_WAVES = 8;            // of CTAs: each has partial results of 131 KB in the workspace and an SM to itself

struct Smem {
    uint64_t k_full[KS], k_empty[KS], vr_full[VS], vr_empty[VS], v_full[VB], v_empty[VB];
    uint64_t s_full[2], s_empty[2], p_full, pv_done, o_free;
    uint64_t q_full, q_empty;
    uint64_t ahead_full[2], ahead_empty[2];
    uint64_t r_full[2], u_empty[2], tree_full[2];   // by unit parity
    uint64_t tree_rows;                          // the tree's K is in its stage
    uint64_t c_sync;                             // warps 4..7 among themselves (a wait that ends, unlike bar.sync)
    uint64_t mma_done[2];
    int par[2][64];                              // a node's parent, -1 where its path ends [unit parity]
    float qf[2][ROWS];
    float mx[2][2][ROWS];                        // [tile parity][half][row]
    float l[2][ROWS];                            // [half][row]
    int row[2 * AHEAD][2];                       // of the tile's two groups in the pool's map
    uchar4 scale[2 * AHEAD];                     // K, K, V, V
    int tree_k[2], tree_v[2], odd_v[2];          // the tree's scale bytes; whether a value is not finite
    uint2 tree_top[2][4];                        // by warp: the largest of K and V as bits, whether V has odd ones
    long long start_off, range;
    int start_b, start_k;
    uint32_t tmem_base;
    int abort_flag;
};
static_assert(SMEM_DYN + sizeof(Smem) <= 232448, "shared memory budget");
static_assert(KS >= LEAST_STAGES, "the timeout test stalls one of them");

struct Wide {
    CacheAttn a;
    int row_groups;
    uint32_t rep_magic;             // row / rep = umulhi(row, magic), 0: rep is 1
    int least;                      // tiles of a range, at least, where there are fewer than CTAs want
    WaitRule wait;
    // workspace: tiles before each sequence's first unit, as tiles of one head [B + 1], then {total tiles of all units,
    // ranges that have any}; where each range begins (tile of its first unit); partial results [2 * CTAs][ROWS]
    long long *cum;
    int4 *start;
    float *part_o, *part_ml;
};

// (exact: rows < 2^18, rep <= 2^12)
E3_DEV int row_node(const Wide &p, int row) { return p.rep_magic ? (int)__umulhi((uint32_t)row, p.rep_magic) : row; }
// element of query row `row` of the KV group g
E3_DEV size_t row_at(const Wide &p, int b, int g, int row) {
    const int node = row_node(p, row);
    return ((size_t)b * p.a.N + node) * p.a.q_ns + (size_t)(g * p.a.rep + row - node * p.a.rep) * D;
}

E3_DEV int seq_len(const CacheAttn &a, int b) { return max(0, min(__ldg(a.prefix_len + b), a.max_prefix)); }
E3_DEV int seq_tiles(const CacheAttn &a, int L) { return max(1, (L + BK - 1) / BK + (a.tree_k ? 1 : 0)); }

// A role's walk over its CTA's range
struct Walk {
    int b, k, i0, i1, nt, L, n;     // sequence, KV head, tiles [i0, i1) of nt, units so far
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
        if (++k == p.a.Hkv) {
            k = 0;
            ++b;
            L = seq_len(p.a, b);
            nt = seq_tiles(p.a, L);
        }
        i0 = 0;
        i1 = (int)min((long long)nt, left);
        return true;
    }
    // the tree comes before the last three tiles of the prefix, which hide its conversion
    E3_DEV int tree_at(const Wide &p) const { return p.a.tree_k ? max(0, nt - 4) : nt; }
    E3_DEV bool is_tree(const Wide &p, int i) const { return i == tree_at(p); }
    E3_DEV bool has_tree(const Wide &p) const { return i0 <= tree_at(p) && tree_at(p) < i1; }
    // the first place of a tile that is not the tree
    E3_DEV int place(const Wide &p, int i) const { return (i - (i > tree_at(p) ? 1 : 0)) * BK; }
};

// 8 fp32 as the two e4m3 parts, 8 bytes each
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

// 8 bf16 by a power of two, as chunk c of a row of two part tiles (128-byte rows, swizzled) `apart` bytes apart; what is
// not finite (odd: some may be) as NaN
E3_DEV void store_parts(uint4 x, float up, bool odd, uint8_t *tile, uint32_t apart, int row, int c) {
    float v[8];
    bf16x8(x, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= up;
    if (odd) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = fabsf(v[e]) <= FLT_MAX ? v[e] : __int_as_float(0x7fc00000);
    }
    uint2 hi, lo;
    two_parts(v, hi, lo);
    uint8_t *at = tile + row * 128 + ((((uint32_t)c >> 1) ^ ((uint32_t)row & 7u)) << 4) + (c & 1) * 8;
    *reinterpret_cast<uint2 *>(at) = hi;
    *reinterpret_cast<uint2 *>(at + apart) = lo;
}

// The nodes that a node sees: itself and its path
E3_DEV uint64_t path_of(const int *par, int i) {
    uint64_t bits = 0;
    for (; i >= 0; i = par[i]) bits |= 1ull << i;
    return bits;
}

E3_DEV float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Rare paths are marked as such, so that the code of the loops is short: all roles' loops together have to stay in the
// SM's instruction cache.
#define RARELY(x) __builtin_expect(!!(x), 0)

// A wait: one poll inline, the loop in one function for all roles (in line at every wait, the loops alone were some 6 KB of
// code that took turns in the instruction cache).
__device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity, uint32_t abort, uint32_t limit) {
    return tc::mbar_wait(bar, parity, abort, limit);
}
E3_DEV bool wait_one(uint32_t bar, uint32_t parity, uint32_t abort, uint32_t limit) {
    return tc::mbar_try(bar, parity) || wait_slow(bar, parity, abort, limit);
}
E3_DEV bool wait_warp(uint32_t bar, uint32_t parity, uint32_t abort, uint32_t limit) {
    const bool ok = wait_one(bar, parity, abort, limit);
    return __all_sync(0xffffffffu, ok);
}

__global__ void __launch_bounds__(NT, 1)
    cache_attn_wide_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                           const __grid_constant__ Wide p) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ Smem ss;
    uint8_t *smp = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t sm = smem_u32(smp);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t abort = smem_u32(&ss.abort_flag), limit = p.wait.limit;
    const CacheAttn &a = p.a;
    const int range_id = blockIdx.x / p.row_groups, row0 = blockIdx.x % p.row_groups * ROWS;   // this CTA's rows
    const int nrows = min(ROWS, a.N * a.rep - row0);
    auto bar = [](uint64_t &b) { return smem_u32(&b); };

    if (tid == 32) {
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
            tc::mbar_init(&ss.s_empty[m], 8);
            tc::mbar_init(&ss.ahead_full[m], 1);
            tc::mbar_init(&ss.ahead_empty[m], 9);   // the loads, eight softmax warps
            tc::mbar_init(&ss.r_full[m], 4);
            tc::mbar_init(&ss.u_empty[m], 8);
            tc::mbar_init(&ss.tree_full[m], 1);
            tc::mbar_init(&ss.mma_done[m], 1);
        }
        tc::mbar_init(&ss.p_full, 8);
        tc::mbar_init(&ss.pv_done, 1);
        tc::mbar_init(&ss.o_free, 8);
        tc::mbar_init(&ss.q_full, 4);
        tc::mbar_init(&ss.q_empty, 1);
        tc::mbar_init(&ss.c_sync, 4);
        tc::mbar_init(&ss.tree_rows, 4);
        ss.abort_flag = 0;
        tc::fence_barrier_init();
        tc::prefetch_tmap(&tm_k);
        tc::prefetch_tmap(&tm_v);
    }
    __syncwarp();
    if (warp == 1) tc::tmem_alloc(&ss.tmem_base, 512);
    pdl_wait();
    pdl_trigger();

    // ---- this CTA's range: the tiles of all sequences summed up, then the sequence that holds its first
    if (warp == 0) {
        auto tiles_at = [&](int b) { return b < a.B ? (long long)seq_tiles(a, seq_len(a, b)) : 0ll; };
        long long seqs = 0;
        for (int b = lane; b < a.B; b += 32) seqs += tiles_at(b);
#pragma unroll
        for (int d = 16; d; d >>= 1) seqs += __shfl_xor_sync(0xffffffffu, seqs, d);
        const long long total = seqs * a.Hkv;
        // as many ranges as leave each `least` tiles
        const long long ranges = max(1ll, min((long long)(gridDim.x / p.row_groups), total / p.least));
        const bool first = blockIdx.x == 0, idle = range_id >= ranges;
        const long long lo = idle ? total : range_id * total / ranges, hi = idle ? total : (range_id + 1) * total / ranges;
        if (lane == 0) {
            ss.range = hi - lo;
            if (first) {
                p.cum[a.B] = seqs;
                p.cum[a.B + 1] = total;
                p.cum[a.B + 2] = ranges;
            }
        }
        long long sum = 0;   // of the sequences before
        for (int b0 = 0; b0 < a.B && (first || (sum * a.Hkv <= lo && !idle)); b0 += 32) {
            const long long mine = tiles_at(b0 + lane);
            long long x = mine;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const long long y = __shfl_up_sync(0xffffffffu, x, d);
                if (lane >= d) x += y;
            }
            const long long before = sum + x - mine;
            if (first && b0 + lane < a.B) p.cum[b0 + lane] = before;
            if (mine > 0 && before * a.Hkv <= lo && lo < (before + mine) * a.Hkv) {
                const long long at = lo - before * a.Hkv;
                ss.start_b = b0 + lane;
                ss.start_k = (int)(at / mine);
                ss.start_off = at % mine;
                if (row0 == 0) p.start[range_id] = make_int4(b0 + lane, (int)(at / mine), (int)(at % mine), 0);
            }
            sum += __shfl_sync(0xffffffffu, x, 31);
        }
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const long long range = ss.range;
    const uint32_t tmem = ss.tmem_base;

    Walk w;
    if (warp == 0) {
        // ------------------------------------------------------------------ TMA
        if (tc::elect_one()) {
            uint32_t t = 0, tv = 0;
            bool ok = true;
            for (bool more = w.begin(p, ss, range); more && ok; more = ok && w.next(p)) {
                for (int i = w.i0; i < w.i1 && ok; ++i, ++t) {
                    if (t % AHEAD == 0 && !wait_one(bar(ss.ahead_full[t / AHEAD & 1]), t / (2 * AHEAD) & 1u, abort, limit)) {
                        ok = false;
                        break;
                    }
                    const int s = (int)(t % KS), sv = (int)(tv % VS);
                    const int r0 = ss.row[t % (2 * AHEAD)][0], r1 = ss.row[t % (2 * AHEAD)][1];
                    if (t % AHEAD == AHEAD - 1) tc::mbar_arrive(bar(ss.ahead_empty[t / AHEAD & 1]));
                    if (w.is_tree(p, i)) continue;   // (warps 4..7 fill that stage)
                    if (!wait_one(bar(ss.k_empty[s]), ((t / KS) & 1u) ^ 1u, abort, limit)) {
                        ok = false;
                        break;
                    }
                    tc::mbar_expect_tx(bar(ss.k_full[s]), K_TILE);
                    const uint32_t dst = sm + OFF_K + s * K_TILE, dv = sm + OFF_VR + sv * K_TILE;
                    tc::tma_load_2d(dst, &tm_k, 0, r0, bar(ss.k_full[s]));
                    tc::tma_load_2d(dst + K_TILE / 2, &tm_k, 0, r1, bar(ss.k_full[s]));
                    if (!wait_one(bar(ss.vr_empty[sv]), ((tv / VS) & 1u) ^ 1u, abort, limit)) {
                        ok = false;
                        ++t;
                        break;
                    }
                    tc::mbar_expect_tx(bar(ss.vr_full[sv]), K_TILE);
                    tc::tma_load_2d(dv, &tm_v, 0, r0, bar(ss.vr_full[sv]));
                    tc::tma_load_2d(dv + K_TILE / 2, &tm_v, 0, r1, bar(ss.vr_full[sv]));
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
        if (tc::elect_one()) {
            constexpr uint32_t IDESC = tc::idesc_e4m3(128, BK), IDESC_T = tc::idesc_e4m3(128, BT);
            uint32_t t = 0, trees = 0;
            bool ok = true;
            for (bool more = w.begin(p, ss, range); more && ok; more = ok && w.next(p)) {
                ok = wait_one(bar(ss.q_full), w.n & 1u, abort, limit);
                for (int i = w.i0; i < w.i1 && ok; ++i, ++t) {
                    const int s = (int)(t % KS);
                    if (!wait_one(bar(ss.k_full[s]), (t / KS) & 1u, abort, limit)) {
                        ok = false;
                        break;
                    }
                    const bool tree = w.is_tree(p, i);
                    const uint32_t kaddr = sm + OFF_K + s * K_TILE;
                    const int b = (int)(t & 1u);
                    if ((tree && !wait_one(bar(ss.tree_rows), trees++ & 1u, abort, limit)) ||
                        (t >= 2 && !wait_one(bar(ss.s_empty[b]), ((t - 2) >> 1) & 1u, abort, limit))) {
                        ok = false;
                        break;
                    }
                    tc::fence_after();
                    const uint32_t d = tmem + TM_S + (uint32_t)(b * BK), q = tmem + TM_Q;
                    if (!RARELY(tree)) {
#pragma unroll
                        for (int k = 0; k < 8; ++k)   // hi, then lo
                            tc::mma_e4m3_ts(d, q + (uint32_t)(k * 8), tc::desc_sw128(kaddr + (k & 3) * 32), IDESC, k > 0 ? 1u : 0u);
                    } else {
#pragma unroll
                        for (int k = 0; k < 16; ++k)   // K in two parts too
                            tc::mma_e4m3_ts(d, q + (uint32_t)((k & 7) * 8),
                                            tc::desc_sw128(kaddr + (k >> 3) * (K_TILE / 2) + (k & 3) * 32), IDESC_T,
                                            k > 0 ? 1u : 0u);
                    }
                    tc::mma_commit(bar(ss.s_full[b]));
                    tc::mma_commit(bar(ss.k_empty[s]));
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
        if (tc::elect_one()) {
            constexpr uint32_t IDESC = tc::idesc_f16_bmn(128, D);
            uint32_t t = 0;
            bool ok = true;
            for (bool more = w.begin(p, ss, range); more && ok; more = ok && w.next(p)) {
                for (int i = w.i0; i < w.i1 && ok; ++i, ++t) {
                    const int s = (int)(t % VB);
                    if (!wait_one(bar(ss.v_full[s]), (t / VB) & 1u, abort, limit)) {
                        ok = false;
                        break;
                    }
                    const bool tree = w.is_tree(p, i);
                    const uint32_t vaddr = sm + OFF_V + s * V_TILE;
                    const bool fresh = i == w.i0;
                    // (a unit's first overwrites O: the one before it must have been read)
                    if (!wait_one(bar(ss.p_full), t & 1u, abort, limit) ||
                        (fresh && w.n > 0 && !wait_one(bar(ss.o_free), (w.n - 1) & 1u, abort, limit))) {
                        ok = false;
                        break;
                    }
                    tc::fence_after();
#pragma unroll
                    for (int kk = 0; kk < BK / 16; ++kk)
                        if (kk < BT / 16 || !tree)
                            tc::mma_bf16_ts(tmem + TM_O, tmem + TM_P + (uint32_t)(kk * 8),
                                            tc::desc_mn_sw128(vaddr + kk * 2048, V_TILE / 2, 1024), IDESC,
                                            !fresh || kk > 0 ? 1u : 0u);
                    tc::mma_commit(bar(ss.pv_done));
                    tc::mma_commit(bar(ss.v_empty[s]));
                }
            }
            if (!ok) flag(a.dev_status, EAGLE3_DEV_TIMEOUT);
            tc::mma_commit(bar(ss.mma_done[1]));
            tc::mbar_drain(bar(ss.mma_done[1]), 0, tc::kiloclock(), limit);
        }
        __syncwarp();
    } else if (warp == 3) {
        // ------------------------------------------------------------------ places and scales ahead
        bool ok = true;
        uint32_t t = 0;
        for (bool more = w.begin(p, ss, range); more && ok; more = ok && w.next(p)) {
            const int g = w.k, sgroups = a.block_size / EAGLE3_KV_GROUP;
            const int32_t *bt = a.block_table + (size_t)w.b * a.max_blocks;
            for (int i = w.i0; i < w.i1;) {
                const uint32_t batch = t / AHEAD;
                if (t % AHEAD == 0 && batch >= 2 &&
                    !wait_warp(bar(ss.ahead_empty[batch & 1]), ((batch - 2) >> 1) & 1u, abort, limit)) {
                    ok = false;
                    break;
                }
                const int n = min(AHEAD - (int)(t % AHEAD), w.i1 - i);
                if (lane < n) {
                    // a group that is not there starts above the pool, where the load reads zeros
                    int row[2] = {-64, -64}, ks[2] = {127, 127}, vs[2] = {1, 1};
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int pos = w.place(p, i + lane) + h * 64;
                        if (pos >= w.L) continue;   // (the tree's own tile is not loaded whatever stands here)
                        const int page = __ldg(bt + pos / a.block_size), place = pos % a.block_size;
                        if (page < 0 || page >= a.n_pages) continue;
                        row[h] = (page * a.Hkv + g) * a.block_size + place;
                        const size_t at = ((size_t)page * a.Hkv + g) * sgroups + place / EAGLE3_KV_GROUP;
                        ks[h] = __ldg(a.ks + at);
                        vs[h] = __ldg(a.vs + at);
                    }
                    const int slot = (int)((t + lane) % (2 * AHEAD));
                    ss.row[slot][0] = row[0];
                    ss.row[slot][1] = row[1];
                    ss.scale[slot] = make_uchar4(ks[0], ks[1], vs[0], vs[1]);
                }
                t += n;
                i += n;
                __syncwarp();
                if (t % AHEAD == 0 && lane == 0) tc::mbar_arrive(bar(ss.ahead_full[batch & 1]));
            }
        }
        if (ok && t % AHEAD != 0 && lane == 0) tc::mbar_arrive(bar(ss.ahead_full[t / AHEAD & 1]));
        if (!ok && lane == 0) flag(a.dev_status, EAGLE3_DEV_TIMEOUT);
    } else if (warp < 8) {
        // ------------------------------------------------------------------ conversions
        const int cw = warp - 4;
        uint32_t t = 0, tv = 0, syncs = 0;
        bool ok = true;
        auto together = [&] {
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(bar(ss.c_sync));
            return wait_warp(bar(ss.c_sync), syncs++ & 1u, abort, limit);
        };
        for (bool more = w.begin(p, ss, range); more && ok; more = ok && w.next(p)) {
            const int u = w.n & 1, g = w.k;
            const bool tree = w.has_tree(p);
            // the tree's parents, which the rows' paths are followed through; the loads return while Q is loaded
            int par[2] = {-1, -1};
            if (cw == 0 && tree) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    if (lane + 32 * h < a.N) par[h] = __ldg(a.parents + (size_t)w.b * a.N + lane + 32 * h);
            }
            const int L_given = __ldg(a.prefix_len + w.b);
            // ---- Q's parts, a row a thread.  Loaded by 4 lanes a row, 32 dims at a time, twice (the second time from the
            // first-level cache): for the rows' maxima, then through shared memory to the rows' threads
            {
                const int r = cw * 32 + lane;
                uint8_t *buf = smp + OFF_IN + cw * IN_WARP;
                auto load = [&](int j, int c) {   // of row 8 j + lane / 4, dims [32 c + 8 (lane & 3), + 8)
                    const int row = min(cw * 32 + 8 * j + (lane >> 2), nrows - 1);
                    return __ldg(reinterpret_cast<const uint4 *>(a.q + row_at(p, w.b, g, row0 + row)) + 4 * c + (lane & 3));
                };
                uint32_t top[4] = {0, 0, 0, 0};
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int j = 0; j < 4; ++j) top[j] = max(top[j], amax_bits(load(j, c)));
                // something is not finite: the largest of the others, and NaN
                const bool odd = __any_sync(0xffffffffu, max(max(top[0], top[1]), max(top[2], top[3])) >= BF16_INF);
                if (RARELY(odd)) {
                    top[0] = top[1] = top[2] = top[3] = 0;
#pragma unroll 1
                    for (int c = 0; c < 4; ++c)
#pragma unroll
                        for (int j = 0; j < 4; ++j) top[j] = max(top[j], amax_bits_finite(load(j, c)));
                }
                uint32_t two[2] = {top[0] | top[1] << 16, top[2] | top[3] << 16};
#pragma unroll
                for (int d = 1; d < 4; d <<= 1)
#pragma unroll
                    for (int j = 0; j < 2; ++j) two[j] = max_u16x2(two[j], __shfl_xor_sync(0xffffffffu, two[j], d));
                // row 8 j + k's from lane 4 k
                const uint32_t t0 = __shfl_sync(0xffffffffu, two[0], (lane & 7) * 4), t1 = __shfl_sync(0xffffffffu, two[1], (lane & 7) * 4);
                const uint32_t tj = lane & 16 ? t1 : t0;
                const int byte = scale_byte_bits(lane & 8 ? tj >> 16 : tj & 0xffffu);
                const float up = r < nrows ? inverse_scale(byte) : 0.0f;   // (rows behind the last one: zeros)
                // (until here beside the unit before's last tiles)
                if ((w.n >= 2 && !wait_warp(bar(ss.u_empty[u]), ((w.n - 2) >> 1) & 1u, abort, limit)) ||
                    (w.n > 0 && !wait_warp(bar(ss.q_empty), (w.n - 1) & 1u, abort, limit))) {
                    ok = false;
                    break;
                }
                tc::fence_after();
                const uint32_t tq = tmem + ((uint32_t)(cw * 32) << 16) + TM_Q;
                uint4 x[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) x[j] = load(j, 0);
#pragma unroll 1
                for (int c = 0; c < 4; ++c) {   // 32 dims: 8 columns of each part; the next 32 on their way
                    uint32_t hi[8], lo[8];
                    __syncwarp();
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int rr = 8 * j + (lane >> 2);
                        *reinterpret_cast<uint4 *>(buf + rr * 64 + (((lane & 3) ^ (rr >> 1 & 3)) << 4)) = x[j];
                        x[j] = load(j, min(c + 1, 3));
                    }
                    __syncwarp();
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float v[8];
                        bf16x8(*reinterpret_cast<const uint4 *>(buf + lane * 64 + ((j ^ (lane >> 1 & 3)) << 4)), v);
#pragma unroll
                        for (int e = 0; e < 8; ++e) v[e] *= up;
                        if (RARELY(odd)) {
#pragma unroll
                            for (int e = 0; e < 8; ++e) v[e] = fabsf(v[e]) <= FLT_MAX ? v[e] : __int_as_float(0x7fc00000);
                        }
                        uint2 h2, l2;
                        two_parts(v, h2, l2);
                        hi[2 * j] = h2.x, hi[2 * j + 1] = h2.y, lo[2 * j] = l2.x, lo[2 * j + 1] = l2.y;
                    }
                    tc::tmem_st8u_start(tq + 8u * c, hi);
                    tc::tmem_st8u_start(tq + 32u + 8u * c, lo);
                }
                tc::tmem_st_wait();
                ss.qf[u][r] = a.scale_log2 * scale_of(byte);
                if (cw == 0) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int i = lane + 32 * h;
                        const bool none = i == 0 || par[h] < 0 || par[h] >= i;   // the root, or a parent that is none
                        ss.par[u][i] = none ? -1 : par[h];
                        if (RARELY(tree && i < a.N && none && !(i == 0 && par[h] == -1)) && w.k == 0)
                            flag(a.dev_status, EAGLE3_DEV_BAD_TREE);
                    }
                    if (RARELY(L_given < 0 || L_given > a.max_prefix) && lane == 0 && w.k == 0 && w.i0 == 0)
                        flag(a.dev_status, EAGLE3_DEV_CAPACITY);
                }
                tc::fence_before();
            }
            __syncwarp();
            if (lane == 0) {
                tc::mbar_arrive(bar(ss.q_full));
                tc::mbar_arrive(bar(ss.r_full[u]));
            }
            // the next unit's queries, and this unit's tree, into L2
            {
                Walk nx = w;
                if (nx.next(p)) {
                    const int row = cw * 32 + lane;
                    if (row < nrows) tc::prefetch_l2(a.q + row_at(p, nx.b, nx.k, row0 + row), 2 * D);
                }
                if (tree && cw < 2)
                    for (int i = lane; i < a.N; i += 32)
                        tc::prefetch_l2((cw ? a.tree_v : a.tree_k) + ((size_t)w.b * a.N + i) * a.kv_ns + (size_t)g * D, 2 * D);
            }
            for (int i = w.i0; i < w.i1; ++i, ++t) {
                const int s = (int)(t % VB);
                uint8_t *dst = smp + OFF_V + s * V_TILE;
                if (RARELY(w.is_tree(p, i))) {
                    // ---- the tree: V in fp16, K in two parts into its stage, each by the power of two of its largest
                    const int c = lane & 15, r0 = cw * 2 + (lane >> 4);
                    const size_t base = (size_t)w.b * a.N * a.kv_ns + (size_t)g * D + c * 8;
                    // (both passes are short loops: straight-line code that runs once a unit costs its fetch)
                    auto load = [&](const __nv_bfloat16 *src, int row) {
                        return __ldg(reinterpret_cast<const uint4 *>(src + base + (size_t)min(row, a.N - 1) * a.kv_ns));
                    };
                    // the largest of all rows, K's and V's in one word (a row behind the last is the last again)
                    uint32_t both = 0;
#pragma unroll
                    for (int row = r0; row < BT; row += 8)
                        both = max_u16x2(both, amax_bits(load(a.tree_k, row)) | amax_bits(load(a.tree_v, row)) << 16);
                    const bool odd_k = __any_sync(0xffffffffu, (both & 0xffffu) >= BF16_INF);
                    const bool odd_v = __any_sync(0xffffffffu, (both >> 16) >= BF16_INF);
                    if (RARELY(odd_k || odd_v)) {
                        both = 0;
#pragma unroll 1
                        for (int row = r0; row < BT; row += 8)
                            both = max_u16x2(both, amax_bits_finite(load(a.tree_k, row)) | amax_bits_finite(load(a.tree_v, row)) << 16);
                    }
#pragma unroll
                    for (int d = 16; d; d >>= 1) both = max_u16x2(both, __shfl_xor_sync(0xffffffffu, both, d));
                    if (lane == 0) ss.tree_top[u][cw] = make_uint2(both, odd_v ? 1u : 0u);
                    if (!together()) {
                        ok = false;
                        break;
                    }
                    uint2 all = ss.tree_top[u][0];
#pragma unroll
                    for (int j = 1; j < 4; ++j) {
                        all.x = max_u16x2(all.x, ss.tree_top[u][j].x);
                        all.y |= ss.tree_top[u][j].y;
                    }
                    const int kb = scale_byte_bits(all.x & 0xffffu), vb = scale_byte_bits(all.x >> 16);
                    if (!wait_warp(bar(ss.v_empty[s]), ((t / VB) & 1u) ^ 1u, abort, limit) ||
                        !wait_warp(bar(ss.k_empty[t % KS]), ((t / KS) & 1u) ^ 1u, abort, limit)) {
                        ok = false;
                        break;
                    }
                    const float kup = inverse_scale(kb), vup = inverse_scale(vb);
#pragma unroll 2
                    for (int row = r0; row < BT; row += 8) {
                        uint4 xk = load(a.tree_k, row), xv = load(a.tree_v, row);
                        if (row >= a.N) xk = xv = make_uint4(0, 0, 0, 0);
                        store_parts(xk, kup, odd_k, smp + OFF_K + (t % KS) * K_TILE, K_TILE / 2, row, c);
                        float v[8];
                        bf16x8(xv, v);
                        if (RARELY(odd_v)) {
#pragma unroll
                            for (int e = 0; e < 8; ++e) v[e] = fabsf(v[e]) <= FLT_MAX ? v[e] : 0.0f;
                        }
                        uint32_t h[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) h[e] = pack_f16(v[2 * e] * vup, v[2 * e + 1] * vup);
                        *reinterpret_cast<uint4 *>(dst + (c >> 3) * (V_TILE / 2) + row * 128 +
                                                   (((uint32_t)c & 7u) ^ ((uint32_t)row & 7u)) * 16) =
                            make_uint4(h[0], h[1], h[2], h[3]);
                    }
                    tc::fence_proxy_async_smem();
                    __syncwarp();
                    if (cw == 0 && lane == 0) {
                        ss.tree_k[u] = kb;
                        ss.tree_v[u] = vb;
                        ss.odd_v[u] = (int)all.y;
                        tc::mbar_arrive(bar(ss.tree_full[u]));
                        tc::mbar_arrive(bar(ss.k_full[t % KS]));   // (the stage's phase; its rows are announced by tree_rows)
                    }
                    if (lane == 0) {
                        tc::mbar_arrive(bar(ss.tree_rows));
                        tc::mbar_arrive(bar(ss.v_full[s]));
                    }
                    continue;
                }
                // ---- V's codes of 32 keys a warp: 8 lanes a key
                const int sv = (int)(tv % VS);
                if (!wait_warp(bar(ss.vr_full[sv]), (tv / VS) & 1u, abort, limit) ||
                    !wait_warp(bar(ss.v_empty[s]), ((t / VB) & 1u) ^ 1u, abort, limit)) {
                    ok = false;
                    break;
                }
                // (lanes: 4 chunks of 16 dims, 2 keys, 2 blocks of 64 dims, 2 keys: 8 lanes' stores fill all banks)
                const int c = (lane & 3) + (lane >> 3 & 1) * 4, k0 = cw * 32 + (lane >> 2 & 1) + (lane >> 4) * 2;
                const uint8_t *src = smp + OFF_VR + sv * K_TILE + k0 * 128;
                uint8_t *to = dst + (c >> 2) * (V_TILE / 2) + k0 * 128;
                const int first = w.place(p, i);
                const bool cut = first + BK > w.L;
#pragma unroll
                for (int it = 0; it < 8; it += 4) {
                    uint4 x[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j)   // key k0 + 4 (it + j): its low three bits are k0's, with bit 2 by j
                        x[j] = *reinterpret_cast<const uint4 *>(src + (it + j) * 512 + ((c ^ ((k0 + 4 * j) & 7)) << 4));
                    if (RARELY(cut)) {            // whatever lies behind the last key
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (first + k0 + 4 * (it + j) >= w.L) x[j] = make_uint4(0, 0, 0, 0);
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int key7 = (k0 + 4 * j) & 7, c0 = 2 * c & 7;
                        *reinterpret_cast<uint4 *>(to + (it + j) * 512 + ((c0 ^ key7) << 4)) =
                            make_uint4(e4m3x2_f16(x[j].x), e4m3x2_f16(x[j].x >> 16), e4m3x2_f16(x[j].y), e4m3x2_f16(x[j].y >> 16));
                        *reinterpret_cast<uint4 *>(to + (it + j) * 512 + (((c0 + 1) ^ key7) << 4)) =
                            make_uint4(e4m3x2_f16(x[j].z), e4m3x2_f16(x[j].z >> 16), e4m3x2_f16(x[j].w), e4m3x2_f16(x[j].w >> 16));
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
            if (ok && !tree && cw == 0 && lane == 0) tc::mbar_arrive(bar(ss.tree_full[u]));   // (a phase a unit)
        }
        if (!ok && lane == 0) flag(a.dev_status, EAGLE3_DEV_TIMEOUT);
    } else {
        // ------------------------------------------------------------------ softmax and results
        // (no way out of the loops: the two warps of a quarter meet at a barrier for every tile; after a wait that ran
        // out they go on without waiting, and follow no parents, which may not be there)
        const int quarter = warp & 3, half = (warp - 8) >> 2, r = quarter * 32 + lane;
        const uint32_t t_lane = tmem + ((uint32_t)(quarter * 32) << 16);
        auto pair_sync = [&] { asm volatile("bar.sync %0, 64;" ::"r"(1 + quarter) : "memory"); };
        uint32_t t = 0;
        bool ok = true;
        auto wait = [&](uint64_t &b, uint32_t parity) { ok = ok && wait_warp(bar(b), parity & 1u, abort, limit); };
        for (bool more = w.begin(p, ss, range); more; more = w.next(p)) {
            const int u = w.n & 1, g = w.k;
            wait(ss.r_full[u], w.n >> 1);
            const float fr = ss.qf[u][r];
            float m_run = -INFINITY, l_run = 0.0f;
            int evref = 0;                     // V's scale byte that O is relative to: the largest so far
            bool odd_v = false;
            for (int i = w.i0; i < w.i1; ++i, ++t) {
                const uint32_t batch = t / AHEAD;
                if (t % AHEAD == 0) wait(ss.ahead_full[batch & 1], batch >> 1);
                uchar4 sb = ss.scale[t % (2 * AHEAD)];
                if (t % AHEAD == AHEAD - 1) {
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(bar(ss.ahead_empty[batch & 1]));
                }
                const bool tree = w.is_tree(p, i);
                if (RARELY(tree)) {
                    wait(ss.tree_full[u], w.n >> 1);
                    sb = make_uchar4(ss.tree_k[u], ss.tree_k[u], ss.tree_v[u], ss.tree_v[u]);
                    odd_v = ss.odd_v[u] != 0;
                }
                wait(ss.s_full[t & 1], t >> 1);
                tc::fence_after();
                const uint32_t t_s = t_lane + TM_S + (t & 1) * BK + half * 64;
                float sc[64];
                tc::tmem_ld32_start(t_s, sc);
                tc::tmem_ld32_start(t_s + 32u, sc + 32);
                // (a factor that underflows would make NaN of the masked scores; a NaN stays)
                float f = fr * scale_of(half ? sb.y : sb.x);
                f = f < FLT_MIN ? FLT_MIN : f;
                const int keys = tree ? -1 : w.L - w.place(p, i) - 64 * half;   // of this half, 64 or more: all
                tc::tmem_ld32_wait(sc);
                tc::tmem_ld32_wait(sc + 32);
                tc::fence_before();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(bar(ss.s_empty[t & 1]));
                if (RARELY(tree || keys < 64)) {
                    uint64_t vis = keys > 0 ? (1ull << keys) - 1ull : 0ull;
                    if (tree) vis = ok && half == 0 && r < nrows ? path_of(ss.par[u], row_node(p, row0 + r)) : 0ull;
                    const uint32_t v0 = (uint32_t)vis, v1 = (uint32_t)(vis >> 32);
#pragma unroll
                    for (int e = 0; e < 64; ++e) sc[e] = ((e < 32 ? v0 : v1) >> (e & 31)) & 1u ? sc[e] : -INFINITY;
                }
                float mq[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) mq[e] = max3(sc[3 * e], sc[3 * e + 1], sc[3 * e + 2]);
#pragma unroll
                for (int e = 12; e < 64; e += 2) mq[(e >> 1) & 3] = max3(mq[(e >> 1) & 3], sc[e], sc[e + 1]);
                float mx = max3(fmaxf(mq[0], mq[1]), mq[2], mq[3]) * f;
                ss.mx[t & 1][half][r] = mx;
                pair_sync();
                mx = fmaxf(mx, ss.mx[t & 1][half ^ 1][r]);
                const bool need = mx > m_run + RESCALE_LOG2;
                const int ev = max(sb.z == 255 ? 0 : sb.z, sb.w == 255 ? 0 : sb.w);
                const bool moved = __any_sync(0xffffffffu, need || ev > evref);
                float corr = 1.0f;
                if (RARELY(moved)) {
                    const float m_new = need ? mx : m_run;
                    corr = need ? (m_run == -INFINITY ? 0.0f : fast_exp2(m_run - m_new)) : 1.0f;
                    l_run *= corr;
                    m_run = m_new;
                    if (ev > evref) {
                        corr *= exp2_int(evref - ev);
                        evref = ev;
                    }
                }
                // the weights by V's scale: 2^down of them; their sum without it
                const int vb = half ? sb.w : sb.z, down = vb == 255 ? 0 : max(LEAST_SHIFT, vb - evref);
                const float nm = (m_run == -INFINITY ? 0.0f : WEIGHT_LOG2 - m_run) + (float)down;
                const float2 f2 = make_float2(f, f), nm2 = make_float2(nm, nm);
                float2 sum[2] = {{0.0f, 0.0f}, {0.0f, 0.0f}};
                uint32_t pk[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    const float2 x = __ffma2_rn(make_float2(sc[2 * e], sc[2 * e + 1]), f2, nm2);
                    const float2 y = make_float2(fast_exp2(x.x), fast_exp2(x.y));
                    sum[e & 1] = __fadd2_rn(sum[e & 1], y);
                    pk[e] = pack_f16(y.x, y.y);
                }
                // (a NaN scale: the weight of the group's first key, which every query sees, so that all dims are NaN; the
                // sum of the weights has no values in it)
                if (RARELY(vb == 255)) pk[0] |= 0x7fffu;
                const float2 s2 = __fadd2_rn(sum[0], sum[1]);
                l_run += (s2.x + s2.y) * exp2_int(-down);
                // P, and O: once the tile before has been multiplied
                if (t > 0) {
                    wait(ss.pv_done, t - 1);
                    tc::fence_after();
                }
                if (!tree || half == 0) tc::tmem_st32u_start(t_lane + TM_P + half * 32u, pk);
                if (RARELY(moved && i > w.i0)) {
#pragma unroll 1
                    for (int q = 0; q < 2; ++q) {
                        float o[32];
                        const uint32_t t_o = t_lane + TM_O + half * 64u + 32u * q;
                        tc::tmem_ld32(t_o, o);
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] *= corr;
                        tc::tmem_st32(t_o, o);
                    }
                }
                tc::tmem_st_wait();
                tc::fence_before();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(bar(ss.p_full));
            }
            // ---- the unit's results: this half's columns
            ss.l[half][r] = l_run;
            pair_sync();
            const float l = ss.l[0][r] + ss.l[1][r];
            wait(ss.pv_done, t - 1);
            tc::fence_after();
            const bool whole = w.i0 == 0 && w.i1 == w.nt, mine = r < nrows;
            const int node = row_node(p, row0 + r), head = g * a.rep + row0 + r - node * a.rep;
            const size_t at = ((size_t)w.b * a.N + (mine ? node : 0)) * a.Hq + (mine ? head : 0);
            const size_t part = (size_t)(2 * blockIdx.x + (w.n > 0 ? 1 : 0)) * ROWS + r;
            const uint64_t anc = ok && odd_v && mine ? path_of(ss.par[u], node) : 0;
            // (a row without a key has summed up nothing)
            const float back = scale_of(evref), inv = whole ? (l == 0.0f ? 0.0f : 1.0f / l) : 1.0f;
#pragma unroll 1
            for (int q = 0; q < 2; ++q) {
                float o[32];
                const int c0 = half * 64 + 32 * q;
                tc::tmem_ld32(t_lane + TM_O + (uint32_t)c0, o);   // warp-collective
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = l != 0.0f ? o[e] * back : 0.0f;
                // infinities and NaN of the tree's values, to the rows that see them
                if (RARELY(odd_v && mine)) {
                    for (int j = 0; j < a.N; ++j) {
                        if (!(anc >> j & 1ull)) continue;
                        const __nv_bfloat16 *tv = a.tree_v + ((size_t)w.b * a.N + j) * a.kv_ns + (size_t)g * D + c0;
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            const float x = (float)tv[e];
                            if (!(fabsf(x) <= FLT_MAX)) o[e] += x;
                        }
                    }
                }
                if (whole) {
                    // through shared memory: a store of the warp writes 64 bytes of 8 rows, not 16 bytes of 32
                    uint8_t *buf = smp + OFF_OUT + (warp - 8) * OUT_WARP;
                    __syncwarp();
#pragma unroll
                    for (int c8 = 0; c8 < 4; ++c8) {
                        uint32_t x[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const __nv_bfloat162 hv = __floats2bfloat162_rn(o[8 * c8 + 2 * e] * inv, o[8 * c8 + 2 * e + 1] * inv);
                            x[e] = *reinterpret_cast<const uint32_t *>(&hv);
                        }
                        *reinterpret_cast<uint4 *>(buf + lane * 64 + ((c8 ^ (lane >> 1 & 3)) << 4)) =
                            make_uint4(x[0], x[1], x[2], x[3]);
                    }
                    __syncwarp();
#pragma unroll
                    for (int it = 0; it < 4; ++it) {
                        const int rr = it * 8 + (lane >> 2), row = quarter * 32 + rr;
                        const uint4 x = *reinterpret_cast<const uint4 *>(buf + rr * 64 + (((lane & 3) ^ (rr >> 1 & 3)) << 4));
                        if (row < nrows) {
                            const int nd = row_node(p, row0 + row);
                            const size_t to = ((size_t)w.b * a.N + nd) * a.Hq + g * a.rep + row0 + row - nd * a.rep;
                            *reinterpret_cast<uint4 *>(a.out + to * D + c0 + (lane & 3) * 8) = x;
                        }
                    }
                } else if (mine) {
                    float4 *dst = reinterpret_cast<float4 *>(p.part_o + part * D + c0);
#pragma unroll
                    for (int c4 = 0; c4 < 8; ++c4) dst[c4] = make_float4(o[4 * c4], o[4 * c4 + 1], o[4 * c4 + 2], o[4 * c4 + 3]);
                }
            }
            tc::fence_before();
            __syncwarp();
            if (lane == 0) {
                tc::mbar_arrive(bar(ss.o_free));
                tc::mbar_arrive(bar(ss.u_empty[u]));
            }
            if (mine && half == 0) {
                if (whole) {
                    if (a.lse) a.lse[at] = lse_of(m_run, l);
                } else {
                    *reinterpret_cast<float2 *>(p.part_ml + 2 * part) = make_float2(m_run, l);
                }
            }
            pair_sync();   // (the sums are read before the next unit's are written)
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

// Joins the units that were cut, in the order of their ranges: grid (range that begins inside a unit, row group, rows).
__global__ void __launch_bounds__(JOIN_WARPS * 32) cache_attn_join_kernel(const __grid_constant__ Wide p) {
    pdl_wait();
    pdl_trigger();
    const CacheAttn &a = p.a;
    const long long total = p.cum[a.B + 1], ranges = p.cum[a.B + 2];
    const long long c = blockIdx.x + 1;
    if (c >= ranges) return;
    const int4 st = p.start[c];
    if (st.z == 0) return;                              // begins with a unit
    const long long before = p.cum[st.x], nt = p.cum[st.x + 1] - before;
    const long long u0 = before * a.Hkv + st.y * nt;
    auto owner = [&](long long x) { return ((x + 1) * ranges - 1) / total; };
    const long long first = owner(u0), last = owner(u0 + nt - 1);
    if (first != c - 1) return;                         // not the unit's first cut
    // the first range's share: the second slot of its CTA, unless it begins with this unit
    const int4 s1 = p.start[first];
    const int second = s1.x == st.x && s1.y == st.y ? 0 : 1;
    const int g = st.y, row0 = blockIdx.y * ROWS, nrows = min(ROWS, a.N * a.rep - row0), lane = threadIdx.x & 31;
    for (int row = blockIdx.z * JOIN_WARPS + (threadIdx.x >> 5); row < nrows; row += gridDim.z * JOIN_WARPS) {
        auto slot = [&](long long q) {
            return (size_t)(2 * (q * p.row_groups + blockIdx.y) + (q == first ? second : 0)) * ROWS + row;
        };
        // 32 ranges at a time: their statistics by lanes, their results as many loads in flight as there are
        float M = -INFINITY, l = 0.0f;
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (long long q0 = first; q0 <= last; q0 += 32) {
            const int n = (int)min(32ll, last - q0 + 1);
            const float2 ml = lane < n ? *reinterpret_cast<const float2 *>(p.part_ml + 2 * slot(q0 + lane)) : make_float2(-INFINITY, 0.0f);
            float top = ml.x;
#pragma unroll
            for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            const float Mn = fmaxf(M, top), down = part_factor(M, l, Mn);
            l *= down;
            o = make_float4(o.x * down, o.y * down, o.z * down, o.w * down);
            M = Mn;
            const float e = part_factor(ml.x, ml.y, M);
            float sum = e * ml.y;
#pragma unroll
            for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
            l += sum;
#pragma unroll 4
            for (int q = 0; q < n; ++q) {
                const float eq = __shfl_sync(0xffffffffu, e, q);
                const float4 x = *reinterpret_cast<const float4 *>(p.part_o + slot(q0 + q) * D + 4 * lane);
                if (eq != 0.0f) o = make_float4(o.x + eq * x.x, o.y + eq * x.y, o.z + eq * x.z, o.w + eq * x.w);
            }
        }
        const int node = (row0 + row) / a.rep, head = g * a.rep + (row0 + row) % a.rep;
        store_row(a, ((size_t)st.x * a.N + node) * a.Hq + head, lane, M, l, o);
    }
}

struct Plan {
    Wide w;
    int ranges;
    size_t o_start, o_part, o_ml, bytes;
};

Plan plan(const CacheAttn &a) {
    Plan pl;
    Wide &w = pl.w;
    w = Wide();
    w.a = a;
    w.row_groups = (a.N * a.rep + ROWS - 1) / ROWS;
    w.rep_magic = a.rep == 1 ? 0u : (uint32_t)(((1ull << 32) + a.rep - 1) / a.rep);
    const int64_t units = (int64_t)a.B * a.Hkv, most = units * ((a.max_prefix + BK - 1) / BK + 1);
    const int sms = std::max(1, device_sm_count());
    int64_t ranges = a.requested > 0 ? std::min(units * a.requested, (int64_t)MOST_WAVES * sms / w.row_groups) : sms / w.row_groups;
    if (ranges > most) ranges = most;
    if (ranges < 1) ranges = 1;
    w.least = a.requested > 0 ? 1 : 2;
    pl.ranges = (int)ranges;
    const size_t ctas = (size_t)ranges * w.row_groups;
    size_t at = 256;
    auto take = [&](size_t n) {
        const size_t o = at;
        at += (n + 255) / 256 * 256;
        return o;
    };
    take(((size_t)a.B + 3) * sizeof(long long));
    pl.o_start = take((size_t)ranges * sizeof(int4));
    pl.o_part = take(ctas * 2 * ROWS * D * sizeof(float));
    pl.o_ml = take(ctas * 2 * ROWS * 2 * sizeof(float));
    pl.bytes = at;
    return pl;
}

}  // namespace

size_t cache_attn_wide_workspace(const CacheAttn &a) { return plan(a).bytes; }

eagle3_status_t cache_attn_wide(const CacheAttn &a, const WaitRule &wait, void *workspace, size_t bytes, cudaStream_t stream) {
    Plan pl = plan(a);
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
    if (launch_pdl(cache_attn_wide_kernel, dim3((unsigned)(pl.ranges * pl.w.row_groups)), dim3(NT), SMEM_DYN, stream, tk, tv, pl.w) != cudaSuccess)
        return EAGLE3_ERR_CUDA;
    if (pl.ranges > 1 && launch_pdl(cache_attn_join_kernel, dim3((unsigned)(pl.ranges - 1), (unsigned)pl.w.row_groups, 4),
                                    dim3(JOIN_WARPS * 32), 0, stream, pl.w) != cudaSuccess)
        return EAGLE3_ERR_CUDA;
    return EAGLE3_OK;
}

}  // namespace e3
