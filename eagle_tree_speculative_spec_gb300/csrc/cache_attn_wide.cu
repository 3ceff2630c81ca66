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
// largest weight, would cost long sums) and V's codes, converted exactly; the scale of V's group is put on the weights,
// relative to the largest so far, by adding to the exponent.
//
// Two streams of (S, P, O) in tensor memory keep the tensor cores busy while the other's softmax runs: with more than
// 128 rows a stream is a row tile and both take every key tile; with up to 128 the streams take alternate key tiles of
// the same rows and are added up at the end of the unit.
//   warp 0        TMA: K tiles into a ring of 3, V codes into a ring of 2
//   warp 1, 2     the MMAs of S, and of P V (one thread issues an MMA about every 110 cycles: two threads)
//   warp 3        looks ahead: the places and scales of the next 32 tiles, a tile a lane (two dependent loads, which
//                 whoever needs them would wait for tile by tile)
//   warps 4..7    V codes to fp16; Q's parts, row scales and ancestor bits of the next unit; the tree's K and V
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
constexpr int AHEAD = 32;               // tiles that warp 3 looks up at once, two such batches
constexpr int NT = 512;
constexpr int LEAST_SHIFT = -60;        // of V's scale on the weights: fp16 has nothing left of them long before
constexpr uint32_t K_TILE = BK * D, V_TILE = 2 * K_TILE;
constexpr uint32_t Q_PART = 128 * D;    // a row tile of one part
constexpr uint32_t OFF_Q = 0;           // [row tile][hi, lo]
constexpr uint32_t OFF_K = OFF_Q + 4 * Q_PART;
constexpr uint32_t OFF_VR = OFF_K + KS * K_TILE;
constexpr uint32_t OFF_V = OFF_VR + VS * K_TILE;
constexpr uint32_t SMEM_DYN = OFF_V + VB * V_TILE + 1024;   // + alignment slack
constexpr uint32_t TM_O = 0, TM_S = 256;                    // each [stream] * 128 columns
constexpr int REGS_FEW = 88, REGS_SOFTMAX = 168;            // 2 * 128 * (88 + 168) = 65536 registers
constexpr int MERGE_WARPS = 8;

struct Smem {
    uint64_t k_full[KS], k_empty[KS], vr_full[VS], vr_empty[VS], v_full[VB], v_empty[VB];
    uint64_t s_full[2], p_full[2], pv_done[2], o_free[2];
    uint64_t q_full, q_empty;
    uint64_t ahead_full[2], ahead_empty[2];
    uint64_t r_full[2], u_empty[2], tree_full[2];   // by unit parity
    uint64_t c_sync;                             // warps 4..7 among themselves (a wait that ends, unlike bar.sync)
    uint64_t x_full, x_empty;                    // stream 1's statistics, one row tile only
    uint64_t mma_done[2];
    uint64_t anc[2][64];
    float qf[2][256];
    int row[2 * AHEAD][2];                       // of the tile's two groups in the pool's map
    uchar4 scale[2 * AHEAD];                     // K, K, V, V
    int tree_k[2], tree_v[2], odd_v[2];          // the tree's scale bytes; whether a value is not finite
    uint32_t top_k[4], top_v[4];
    float x_m[128], x_l[128];
    int x_ev, x_odd;
    long long start_off, range;
    int start_b, start_k;
    uint32_t tmem_base;
    int abort_flag;
};
static_assert(SMEM_DYN + sizeof(Smem) <= 232448, "shared memory budget");

struct Wide {
    CacheAttn a;
    int tiles2;                     // two row tiles (else one)
    int rows_per_group, row_groups, heads;   // heads = Hkv * row_groups: units of a sequence
    uint32_t rep_magic;             // row / rep = umulhi(row, magic), 0: rep is 1
    int least;                      // tiles of a range, at least, where there are fewer than CTAs want
    WaitRule wait;
    // workspace: tiles before each sequence [B + 1], then {total tiles of all units, CTAs that have any}; where each
    // CTA begins (tile of its first unit); partial results [2 * CTAs][rows_per_group]
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

// The largest finite magnitudes of N rows, 16 lanes a row (the other 16 of a warp N more), as bits; whether the warp has
// anything that is not finite.  Two rows a word, and all words a step at a time: the exchanges overlap.
template <int N>
E3_DEV bool row_maxima(const uint4 (&x)[N], uint32_t (&top)[N]) {
    uint32_t all = 0;
#pragma unroll
    for (int j = 0; j < N; ++j) {
        top[j] = amax_bits(x[j]);
        all = max(all, top[j]);
    }
    const bool odd = __any_sync(0xffffffffu, all >= BF16_INF);
    if (odd) {
#pragma unroll
        for (int j = 0; j < N; ++j) top[j] = amax_bits_finite(x[j]);
    }
    uint32_t two[N / 2], other[N / 2];
#pragma unroll
    for (int j = 0; j < N / 2; ++j) two[j] = top[2 * j] | top[2 * j + 1] << 16;
#pragma unroll
    for (int d = 8; d; d >>= 1) {
#pragma unroll
        for (int j = 0; j < N / 2; ++j) other[j] = __shfl_xor_sync(0xffffffffu, two[j], d);
#pragma unroll
        for (int j = 0; j < N / 2; ++j) two[j] = max_u16x2(two[j], other[j]);
    }
#pragma unroll
    for (int j = 0; j < N / 2; ++j) {
        top[2 * j] = two[j] & 0xffffu;
        top[2 * j + 1] = two[j] >> 16;
    }
    return odd;
}

// The nodes that each node sees, by a warp: every node's set joined with that of the node it has got to, which moves
// twice as far each time
E3_DEV void tree_paths(const CacheAttn &a, int b, bool report, int lane, uint64_t *anc) {
    int to[2];
    uint64_t bits[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int i = lane + 32 * h;
        const int q = i < a.N ? __ldg(a.parents + (size_t)b * a.N + i) : -1;
        const bool bad = i < a.N && (i == 0 ? q != -1 : q < 0 || q >= i);
        if (bad && report) flag(a.dev_status, EAGLE3_DEV_BAD_TREE);
        to[h] = i == 0 || bad ? -1 : q;
        bits[h] = 1ull << i;
    }
    for (int step = 0; step < 6; ++step) {
        uint64_t more[2];
        int next[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int from = max(0, to[h]);
            const uint64_t b0 = __shfl_sync(0xffffffffu, bits[0], from & 31), b1 = __shfl_sync(0xffffffffu, bits[1], from & 31);
            const int n0 = __shfl_sync(0xffffffffu, to[0], from & 31), n1 = __shfl_sync(0xffffffffu, to[1], from & 31);
            more[h] = to[h] < 0 ? 0ull : from < 32 ? b0 : b1;
            next[h] = to[h] < 0 ? -1 : from < 32 ? n0 : n1;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            bits[h] |= more[h];
            to[h] = next[h];
        }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
        if (lane + 32 * h < a.N) anc[lane + 32 * h] = bits[h];
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
    uint8_t *smp = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t sm = smem_u32(smp);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t abort = smem_u32(&ss.abort_flag), limit = p.wait.limit;
    const CacheAttn &a = p.a;
    const bool two = p.tiles2 != 0;
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
            tc::mbar_init(&ss.p_full[m], 4);
            tc::mbar_init(&ss.pv_done[m], 1);
            tc::mbar_init(&ss.o_free[m], 4);
            tc::mbar_init(&ss.ahead_full[m], 1);
            tc::mbar_init(&ss.ahead_empty[m], 9);   // the loads, eight softmax warps
            tc::mbar_init(&ss.r_full[m], 4);
            tc::mbar_init(&ss.u_empty[m], 8);
            tc::mbar_init(&ss.tree_full[m], 1);
            tc::mbar_init(&ss.mma_done[m], 1);
        }
        tc::mbar_init(&ss.q_full, 4);
        tc::mbar_init(&ss.q_empty, 1);
        tc::mbar_init(&ss.c_sync, 4);
        tc::mbar_init(&ss.x_full, 4);
        tc::mbar_init(&ss.x_empty, 4);
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
        const long long total = seqs * p.heads;
        // as many CTAs as leave each `least` tiles
        const long long ctas = max(1ll, min((long long)gridDim.x, total / p.least));
        const bool first = blockIdx.x == 0, idle = blockIdx.x >= ctas;
        const long long lo = idle ? total : blockIdx.x * total / ctas, hi = idle ? total : (blockIdx.x + 1) * total / ctas;
        if (lane == 0) {
            ss.range = hi - lo;
            if (first) {
                p.cum[a.B] = seqs;
                p.cum[a.B + 1] = total;
                p.cum[a.B + 2] = ctas;
            }
        }
        long long sum = 0;   // of the sequences before
        for (int b0 = 0; b0 < a.B && (first || (sum * p.heads <= lo && !idle)); b0 += 32) {
            const long long mine = tiles_at(b0 + lane);
            long long x = mine;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const long long y = __shfl_up_sync(0xffffffffu, x, d);
                if (lane >= d) x += y;
            }
            const long long before = sum + x - mine;
            if (first && b0 + lane < a.B) p.cum[b0 + lane] = before;
            if (mine > 0 && before * p.heads <= lo && lo < (before + mine) * p.heads) {
                const long long at = lo - before * p.heads;
                ss.start_b = b0 + lane;
                ss.start_k = (int)(at / mine);
                ss.start_off = at % mine;
                p.start[blockIdx.x] = make_int4(b0 + lane, (int)(at / mine), (int)(at % mine), 0);
            }
            sum += __shfl_sync(0xffffffffu, x, 31);
        }
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const long long range = ss.range;
    const uint32_t tmem = ss.tmem_base;

    // (each branch gives or takes registers by itself: the compiler allots them by branch)
    Walk w;
    if (warp == 0) {
        // ------------------------------------------------------------------ TMA
        tc::registers_give<REGS_FEW>();
        if (tc::elect_one()) {
            uint32_t t = 0, tv = 0;
            bool ok = true;
            for (bool more = w.begin(p, ss, range); more && ok; more = ok && w.next(p)) {
                for (int i = w.i0; i < w.i1 && ok; ++i, ++t) {
                    if (t % AHEAD == 0 && !tc::mbar_wait(bar(ss.ahead_full[t / AHEAD & 1]), t / (2 * AHEAD) & 1u, abort, limit)) {
                        ok = false;
                        break;
                    }
                    const int s = (int)(t % KS), sv = (int)(tv % VS);
                    const int r0 = ss.row[t % (2 * AHEAD)][0], r1 = ss.row[t % (2 * AHEAD)][1];
                    if (t % AHEAD == AHEAD - 1) tc::mbar_arrive(bar(ss.ahead_empty[t / AHEAD & 1]));
                    if (w.is_tree(p, i)) continue;   // (warps 4..7 fill that stage)
                    if (!tc::mbar_wait(bar(ss.k_empty[s]), ((t / KS) & 1u) ^ 1u, abort, limit)) {
                        ok = false;
                        break;
                    }
                    tc::mbar_expect_tx(bar(ss.k_full[s]), K_TILE);
                    const uint32_t dst = sm + OFF_K + s * K_TILE, dv = sm + OFF_VR + sv * K_TILE;
                    tc::tma_load_2d(dst, &tm_k, 0, r0, bar(ss.k_full[s]));
                    tc::tma_load_2d(dst + K_TILE / 2, &tm_k, 0, r1, bar(ss.k_full[s]));
                    if (!tc::mbar_wait(bar(ss.vr_empty[sv]), ((tv / VS) & 1u) ^ 1u, abort, limit)) {
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
#pragma unroll
                        for (int kk = 0; kk < BK / 16; ++kk)
                            if (kk < ksteps)
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
        // ------------------------------------------------------------------ places and scales ahead
        tc::registers_give<REGS_FEW>();
        bool ok = true;
        uint32_t t = 0;
        for (bool more = w.begin(p, ss, range); more && ok; more = ok && w.next(p)) {
            const int g = w.k / p.row_groups, sgroups = a.block_size / EAGLE3_KV_GROUP;
            const int32_t *bt = a.block_table + (size_t)w.b * a.max_blocks;
            for (int i = w.i0; i < w.i1;) {
                const uint32_t batch = t / AHEAD;
                if (t % AHEAD == 0 && batch >= 2 &&
                    !tc::mbar_wait_warp(bar(ss.ahead_empty[batch & 1]), ((batch - 2) >> 1) & 1u, abort, limit)) {
                    ok = false;
                    break;
                }
                const int n = min(AHEAD - (int)(t % AHEAD), w.i1 - i);
                if (lane < n) {
                    // a group that is not there starts above the pool, where the load reads zeros
                    int row[2] = {-64, -64}, ks[2] = {127, 127}, vs[2] = {1, 1};
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const long long pos = (long long)(i + lane) * BK + h * 64;
                        if (pos >= w.L) continue;
                        const int page = __ldg(bt + (int)pos / a.block_size), place = (int)pos % a.block_size;
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
        tc::registers_give<REGS_FEW>();
        const int cw = warp - 4;
        uint32_t t = 0, tv = 0, syncs = 0;
        bool ok = true;
        auto together = [&] {
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(bar(ss.c_sync));
            return tc::mbar_wait_warp(bar(ss.c_sync), syncs++ & 1u, abort, limit);
        };
        for (bool more = w.begin(p, ss, range); more && ok; more = ok && w.next(p)) {
            const int u = w.n & 1, g = w.k / p.row_groups, row0 = w.k % p.row_groups * p.rows_per_group;
            if ((w.n >= 2 && !tc::mbar_wait_warp(bar(ss.u_empty[u]), ((w.n - 2) >> 1) & 1u, abort, limit)) ||
                (w.n > 0 && !tc::mbar_wait_warp(bar(ss.q_empty), (w.n - 1) & 1u, abort, limit))) {
                ok = false;
                break;
            }
            const bool tree = a.tree_k && w.i1 == w.nt;
            // ---- Q's parts: 16 lanes a row, two rows at a time, eight such pairs on their way
            const int nrows = min(p.rows_per_group, a.N * a.rep - row0);
            for (int it = 0; it < p.rows_per_group / 8; it += 8) {
                uint4 x[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int row = (it + j) * 8 + cw * 2 + (lane >> 4);
                    x[j] = make_uint4(0, 0, 0, 0);
                    if (row < nrows) x[j] = *reinterpret_cast<const uint4 *>(a.q + row_at(p, w.b, g, row0 + row) + (lane & 15) * 8);
                }
                uint32_t top[8];
                const bool odd = row_maxima<8>(x, top);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int row = (it + j) * 8 + cw * 2 + (lane >> 4), byte = scale_byte_bits(top[j]);
                    store_parts(x[j], inverse_scale(byte), odd, smp + OFF_Q + (row >> 7) * 2 * Q_PART, Q_PART, row & 127, lane & 15);
                    if ((lane & 15) == 0) ss.qf[u][row] = a.scale_log2 * scale_of(byte);
                }
            }
            tc::fence_proxy_async_smem();
            if (cw == 0) {
                if (tree) tree_paths(a, w.b, w.k == 0, lane, ss.anc[u]);
                const int L = __ldg(a.prefix_len + w.b);
                if (lane == 0 && (L < 0 || L > a.max_prefix) && w.k == 0 && w.i0 == 0) flag(a.dev_status, EAGLE3_DEV_CAPACITY);
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
                    const int ng = nx.k / p.row_groups, nrow0 = nx.k % p.row_groups * p.rows_per_group;
                    const int rows_next = min(p.rows_per_group, a.N * a.rep - nrow0);
                    for (int row = cw * 32 + lane; row < rows_next; row += 128)
                        tc::prefetch_l2(a.q + row_at(p, nx.b, ng, nrow0 + row), 2 * D);
                }
                if (tree && cw < 2)
                    for (int i = lane; i < a.N; i += 32)
                        tc::prefetch_l2((cw ? a.tree_v : a.tree_k) + ((size_t)w.b * a.N + i) * a.kv_ns + (size_t)g * D, 2 * D);
            }
            for (int i = w.i0; i < w.i1; ++i, ++t) {
                const int s = (int)(t % VB);
                uint8_t *dst = smp + OFF_V + s * V_TILE;
                if (w.is_tree(p, i)) {
                    // ---- the tree: V in fp16, K in two parts into its stage, each by the power of two of its largest
                    const int c = lane & 15, r0 = cw * 2 + (lane >> 4);
                    uint4 x[BT / 8];
                    bool odd = false;
                    // the rows of this warp in x, and the scale byte of them all
                    auto load = [&](const __nv_bfloat16 *src, uint32_t *tops, int &byte) {
                        src += (size_t)w.b * a.N * a.kv_ns + (size_t)g * D + c * 8;
#pragma unroll
                        for (int j = 0; j < BT / 8; ++j) {
                            x[j] = make_uint4(0, 0, 0, 0);
                            if (j * 8 + r0 < a.N) x[j] = *reinterpret_cast<const uint4 *>(src + (j * 8 + r0) * a.kv_ns);
                        }
                        uint32_t top[BT / 8], all = 0;
                        odd = row_maxima<BT / 8>(x, top);
#pragma unroll
                        for (int j = 0; j < BT / 8; ++j) all = max(all, top[j]);
                        all = max(all, __shfl_xor_sync(0xffffffffu, all, 16));
                        if (lane == 0) tops[cw] = all;
                        const bool got = together();
                        byte = scale_byte_bits(max(max(tops[0], tops[1]), max(tops[2], tops[3])));
                        return got;
                    };
                    int kb, vb;
                    if (cw == 0 && lane == 0) ss.odd_v[u] = 0;
                    if (!load(a.tree_v, ss.top_v, vb) ||
                        !tc::mbar_wait_warp(bar(ss.v_empty[s]), ((t / VB) & 1u) ^ 1u, abort, limit)) {
                        ok = false;
                        break;
                    }
                    if (lane == 0 && odd) ss.odd_v[u] = 1;
                    const float vup = inverse_scale(vb);
#pragma unroll
                    for (int j = 0; j < BT / 8; ++j) {
                        const int row = j * 8 + r0;
                        float v[8];
                        bf16x8(x[j], v);
                        if (odd) {
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
                    if (!load(a.tree_k, ss.top_k, kb) ||
                        !tc::mbar_wait_warp(bar(ss.k_empty[t % KS]), ((t / KS) & 1u) ^ 1u, abort, limit)) {
                        ok = false;
                        break;
                    }
#pragma unroll
                    for (int j = 0; j < BT / 8; ++j)
                        store_parts(x[j], inverse_scale(kb), odd, smp + OFF_K + (t % KS) * K_TILE, K_TILE / 2, j * 8 + r0, c);
                    tc::fence_proxy_async_smem();
                    if (!together()) {   // all of K is there: one arrival
                        ok = false;
                        break;
                    }
                    if (cw == 0 && lane == 0) {
                        ss.tree_k[u] = kb;
                        ss.tree_v[u] = vb;
                        tc::mbar_arrive(bar(ss.tree_full[u]));
                        tc::mbar_arrive(bar(ss.k_full[t % KS]));
                    }
                    if (lane == 0) tc::mbar_arrive(bar(ss.v_full[s]));
                    continue;
                }
                // ---- V's codes of 32 keys a warp: 8 lanes a key
                const int sv = (int)(tv % VS);
                if (!tc::mbar_wait_warp(bar(ss.vr_full[sv]), (tv / VS) & 1u, abort, limit) ||
                    !tc::mbar_wait_warp(bar(ss.v_empty[s]), ((t / VB) & 1u) ^ 1u, abort, limit)) {
                    ok = false;
                    break;
                }
                const uint8_t *src = smp + OFF_VR + sv * K_TILE;
                const int c = lane & 7;
#pragma unroll
                for (int it = 0; it < 8; it += 4) {
                    uint4 x[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int key = cw * 32 + (it + j) * 4 + (lane >> 3);
                        x[j] = *reinterpret_cast<const uint4 *>(src + key * 128 + (((uint32_t)c ^ ((uint32_t)key & 7u)) << 4));
                        if (i * BK + key >= w.L) x[j] = make_uint4(0, 0, 0, 0);   // whatever lies behind the last key
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int key = cw * 32 + (it + j) * 4 + (lane >> 3);
                        const uint4 lo = make_uint4(e4m3x2_f16(x[j].x), e4m3x2_f16(x[j].x >> 16), e4m3x2_f16(x[j].y),
                                                    e4m3x2_f16(x[j].y >> 16));
                        const uint4 hi = make_uint4(e4m3x2_f16(x[j].z), e4m3x2_f16(x[j].z >> 16), e4m3x2_f16(x[j].w),
                                                    e4m3x2_f16(x[j].w >> 16));
                        // 16 dims: two chunks of a block of 64; the upper block's lanes store theirs in the other order,
                        // so that 8 lanes fill all banks
                        uint8_t *blk = dst + (c >> 2) * (V_TILE / 2) + key * 128;
                        const bool swap = c >= 4;
                        const uint32_t c0 = (uint32_t)(2 * c) & 7u, key7 = (uint32_t)key & 7u;
                        *reinterpret_cast<uint4 *>(blk + (((c0 + (swap ? 1u : 0u)) ^ key7) << 4)) = swap ? hi : lo;
                        *reinterpret_cast<uint4 *>(blk + (((c0 + (swap ? 0u : 1u)) ^ key7) << 4)) = swap ? lo : hi;
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
        tc::registers_take<REGS_SOFTMAX>();
        const int m = (warp - 8) >> 2, r = (warp & 3) * 32 + lane;   // stream, TMEM lane
        const uint32_t t_lane = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t t_s = t_lane + TM_S + (uint32_t)(m * 128), t_o = t_lane + TM_O + (uint32_t)(m * 128);
        uint32_t t = 0;
        bool ok = true;
        for (bool more = w.begin(p, ss, range); more && ok; more = ok && w.next(p)) {
            const int u = w.n & 1, g = w.k / p.row_groups, row0 = w.k % p.row_groups * p.rows_per_group;
            const int row = two ? m * 128 + r : r, nrows = min(p.rows_per_group, a.N * a.rep - row0);
            if (!tc::mbar_wait_warp(bar(ss.r_full[u]), (w.n >> 1) & 1u, abort, limit)) {
                ok = false;
                break;
            }
            const float fr = ss.qf[u][row];
            float m_run = -INFINITY, l_run = 0.0f;
            int evref = 0;                     // V's scale byte that O is relative to: the largest so far
            bool fresh = true, odd_v = false;
            for (int i = w.i0; i < w.i1; ++i, ++t) {
                const uint32_t batch = t / AHEAD;
                if (t % AHEAD == 0 && !tc::mbar_wait_warp(bar(ss.ahead_full[batch & 1]), (batch >> 1) & 1u, abort, limit)) {
                    ok = false;
                    break;
                }
                uchar4 sb = ss.scale[t % (2 * AHEAD)];
                if (t % AHEAD == AHEAD - 1) {
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(bar(ss.ahead_empty[batch & 1]));
                }
                if (!two && (int)(t & 1u) != m) continue;
                const bool tree = w.is_tree(p, i);
                if (tree) {
                    if (!tc::mbar_wait_warp(bar(ss.tree_full[u]), (w.n >> 1) & 1u, abort, limit)) {
                        ok = false;
                        break;
                    }
                    sb = make_uchar4(ss.tree_k[u], ss.tree_k[u], ss.tree_v[u], ss.tree_v[u]);
                    odd_v = ss.odd_v[u] != 0;
                }
                if (!tc::mbar_wait_warp(bar(ss.s_full[m]), stream_tiles(two, m, t) & 1u, abort, limit)) {
                    ok = false;
                    break;
                }
                tc::fence_after();
                float sc[128];
#pragma unroll
                for (int q = 0; q < 4; ++q) tc::tmem_ld32_start(t_s + 32u * q, sc + 32 * q);
                // (a factor that underflows would make NaN of the masked scores; a NaN stays)
                float f0 = fr * scale_of(sb.x), f1 = fr * scale_of(sb.y);
                f0 = f0 < FLT_MIN ? FLT_MIN : f0;
                f1 = f1 < FLT_MIN ? FLT_MIN : f1;
                const int keys = tree ? -1 : min(BK, w.L - i * BK);
#pragma unroll
                for (int q = 0; q < 4; ++q) tc::tmem_ld32_wait(sc + 32 * q);
                if (keys < BK) {
                    uint64_t anc = 0;
                    if (tree && row < nrows) anc = ss.anc[u][row_node(p, row0 + row)];
                    uint32_t vis[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int n = keys - 32 * q;
                        vis[q] = keys < 0 ? (q < 2 ? (uint32_t)(anc >> (32 * (q & 1))) : 0u)
                                          : n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1u;
                    }
#pragma unroll
                    for (int e = 0; e < 128; ++e) sc[e] = (vis[e >> 5] >> (e & 31)) & 1u ? sc[e] : -INFINITY;
                }
                float mq[2][4];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) mq[h][e] = max3(sc[64 * h + 3 * e], sc[64 * h + 3 * e + 1], sc[64 * h + 3 * e + 2]);
#pragma unroll
                    for (int e = 12; e < 64; e += 2) mq[h][(e >> 1) & 3] = max3(mq[h][(e >> 1) & 3], sc[64 * h + e], sc[64 * h + e + 1]);
                }
                const float mx = fmaxf(max3(fmaxf(mq[0][0], mq[0][1]), mq[0][2], mq[0][3]) * f0,
                                       max3(fmaxf(mq[1][0], mq[1][1]), mq[1][2], mq[1][3]) * f1);
                const bool need = mx > m_run + RESCALE_LOG2;
                const int ev = max(sb.z == 255 ? 0 : sb.z, sb.w == 255 ? 0 : sb.w);
                const bool moved = __any_sync(0xffffffffu, need || ev > evref);
                float corr = 1.0f;
                if (moved) {
                    const float m_new = need ? mx : m_run;
                    corr = need ? (m_run == -INFINITY ? 0.0f : fast_exp2(m_run - m_new)) : 1.0f;
                    l_run *= corr;
                    m_run = m_new;
                    if (ev > evref) {
                        corr *= exp2_int(evref - ev);
                        evref = ev;
                    }
                }
                const float nm = m_run == -INFINITY ? 0.0f : WEIGHT_LOG2 - m_run;
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    // the weights by V's scale: 2^down of them; their sum without it
                    const int vb = q ? sb.w : sb.z, down = max(LEAST_SHIFT, vb - evref);
                    const float f = q ? f1 : f0, n = vb == 255 ? __int_as_float(0x7fc00000) : nm + (float)down;
                    const float2 f2 = make_float2(f, f), nm2 = make_float2(n, n);
                    float2 sum[2] = {{0.0f, 0.0f}, {0.0f, 0.0f}};
                    uint32_t pk[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        const float2 x = __ffma2_rn(make_float2(sc[64 * q + 2 * e], sc[64 * q + 2 * e + 1]), f2, nm2);
                        const float2 y = make_float2(fast_exp2(x.x), fast_exp2(x.y));
                        sum[e & 1] = __fadd2_rn(sum[e & 1], y);
                        pk[e] = pack_f16(y.x, y.y);
                    }
                    const float2 s2 = __fadd2_rn(sum[0], sum[1]);
                    l_run += (s2.x + s2.y) * exp2_int(-down);
                    tc::tmem_st32u_start(t_s + 32u * q, pk);
                }
                tc::tmem_st_wait();
                // O (now that the scores' registers are free; P V of the tile before is done, since S waited for it)
                if (moved && !fresh) {
#pragma unroll 1
                    for (int q = 0; q < 4; ++q) {
                        float o[32];
                        tc::tmem_ld32(t_o + 32u * q, o);
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] *= corr;
                        tc::tmem_st32(t_o + 32u * q, o);
                    }
                }
                fresh = false;
                tc::fence_before();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(bar(ss.p_full[m]));
            }
            if (!ok) break;
            // ---- the unit's results
            float e0 = scale_of(evref), e1 = 0.0f, M = m_run, l = l_run;   // factors of the streams' sums
            if (!two) {
                if (m == 1) {
                    if (w.n > 0 && !tc::mbar_wait_warp(bar(ss.x_empty), (w.n - 1) & 1u, abort, limit)) {
                        ok = false;
                        break;
                    }
                    ss.x_m[r] = m_run;
                    ss.x_l[r] = l_run;
                    if (r == 0) {
                        ss.x_ev = evref;
                        ss.x_odd = odd_v ? 1 : 0;
                    }
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
                const float m2 = ss.x_m[r], l2 = ss.x_l[r], v2 = scale_of(ss.x_ev);
                odd_v = odd_v || ss.x_odd != 0;
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(bar(ss.x_empty));
                M = fmaxf(m_run, m2);
                const float a0 = weight_of(m_run, l_run, M), a1 = weight_of(m2, l2, M);
                l = a0 * l_run + a1 * l2;
                e0 *= a0;
                e1 = v2 * a1;
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
            const int node = row_node(p, row0 + row), head = g * a.rep + row0 + row - node * a.rep;
            const size_t at = ((size_t)w.b * a.N + (mine ? node : 0)) * a.Hq + (mine ? head : 0);
            const size_t part = (size_t)(2 * blockIdx.x + (w.n > 0 ? 1 : 0)) * p.rows_per_group + row;
            const uint64_t anc = odd_v && mine ? ss.anc[u][node] : 0;
            const float inv = whole ? (l == 0.0f ? 0.0f : 1.0f / l) : 1.0f;
            const bool has0 = l_run != 0.0f && e0 != 0.0f, has1 = e1 != 0.0f;   // (a stream without a key has summed up nothing)
#pragma unroll 1
            for (int q = 0; q < 4; ++q) {
                float o[32];
                tc::tmem_ld32(t_lane + TM_O + 32u * q + (two ? m * 128u : 0u), o);   // warp-collective
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = has0 ? o[e] * e0 : 0.0f;
                if (!two) {
                    float o2[32];
                    tc::tmem_ld32(t_lane + TM_O + 128u + 32u * q, o2);
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = has1 ? o[e] + o2[e] * e1 : o[e];
                }
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
    w.rep_magic = a.rep == 1 ? 0u : (uint32_t)(((1ull << 32) + a.rep - 1) / a.rep);
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
