// eagle3_grouped_linear: matrix products grouped by expert with ragged row counts, on tcgen05 / TMEM
// (bf16 in, fp32 accumulate): the expert projections of a mixture-of-experts target's feed-forward
// layer, y_s = W_e x_s for the rows s that expert e received, with the SwiGLU of "EAGLE-3:
// Engineering Implementation of LLM Inference Acceleration", appendix C, as an epilogue.
//
// The operands are swapped: 128 weight rows (output columns) are the M side of the MMA and the rows
// of a group are the N side, because N may be any multiple of 16 up to 256 while M is fixed.  A group
// of any size then wastes at most 15 columns of its last tile, and a group of one row costs its
// weights' traffic and little else.
//
// Persistent, warp-specialised, one CTA per SM, two CTAs on one tile (PAIR, below) but for few weight rows;
// every CTA reads the offsets, and derives the tiles by a prefix sum over the groups:
//   warp 0      TMA producer: the weight tile (SwiGLU: 64 gate and 64 up rows), and the rows unless they
//               are gathered, by at most three boxes (a box costs about 70 cycles whatever its size:
//               boxes of 16 rows held a 3840 x 8192 x 4096 product to 835 TFLOP/s; it runs at 1860)
//   warp 1      TMEM owner; one lane issues tcgen05.mma (M = 128, or 256 for the pair, N = rows of the
//               tile, K = 16)
//   warps 2..5  epilogue: tcgen05.ld, SwiGLU, stores of two columns a lane.  TMEM lanes 0..63 hold gate
//               columns and 64..127 their up columns: two warps that share columns swap them through
//               shared memory, and each finishes half of the rows
//   warps 6..13 with row_ids only: gather the rows by 16-byte asynchronous copies into the swizzled
//               tile (TMA's four-row gathers cost as much as a box each: 2288 us for 3840 rows x 8 of
//               64 experts, k = 4096, 2 x 1024 columns)
// The accumulator is double-buffered in TMEM (2 x 256 columns).  The ring's stage holds a weight tile
// and as many rows as the largest tile of this call has, so the ring is deep (up to 12 stages) where
// groups are small and the call is bound by its weights' bytes.  Units run group by group, row tile
// fastest, so that the CTAs that share a weight tile run together.
//
// Where the units leave SMs idle, a cluster shares each one's k-blocks (SPLIT, below).
//
// Every mbarrier wait is bounded; on a timeout the kernel records EAGLE3_DEV_TIMEOUT, stops issuing
// work, drains its own TMA loads and frees its TMEM.
#include <algorithm>

#include "../../include/eagle3_chain.h"
#include "../../include/eagle3_moe.h"
#include "../../include/eagle3_testing.h"
#include "tc.cuh"
#include "tmap.cuh"

namespace e3 {
namespace {

constexpr int BM = 128, BK = 64;          // weight rows and k values of a tile
constexpr int MAX_ROWS = 256;             // rows of a tile (the MMA's N), a multiple of 16
constexpr int NTHREADS = 192, GATHER_WARPS = 8;
constexpr int GATHER_ROWS = 4 * GATHER_WARPS;   // rows of a pass: 8 threads a row
constexpr int W_BYTES = BM * BK * 2;
constexpr int ROW_BYTES = BK * 2;
constexpr int MAX_STAGES = 12;
constexpr int RING_BYTES = 205 * 1024;
constexpr int MAX_E = EAGLE3_MOE_MAX_EXPERTS;
constexpr int TMEM_COLS = 2 * MAX_ROWS;

struct Shared {
    float swap[2][2][32 * 32];   // SwiGLU: per pair of warps, what each hands to the other
    uint64_t full[MAX_STAGES], empty[MAX_STAGES], tfull[2], tempty[2], mma_done;
    uint32_t tmem_base;
    int abort, max_rows;
    int offsets[MAX_E + 1];
    int tiles[MAX_E + 1];   // exclusive prefix sums of the groups' row tiles
};
constexpr int SMEM = 1024 /* align */ + RING_BYTES + (int)sizeof(Shared);
static_assert(SMEM <= 232448, "shared memory budget");
static_assert(RING_BYTES / (W_BYTES + MAX_ROWS * ROW_BYTES) >= LEAST_STAGES, "stages of the largest tiles");

// Rows that a tile's boxes load: one box of 256, or up to three of 64 and one of 16 (at most the
// next multiple of 64; rows past the tile's are loaded and not used).
E3_DEV int box_rows(int n16) {
    const int rest = n16 & 63;
    return n16 > 192 ? 256 : (n16 & ~63) + (rest > 16 ? 64 : rest);
}
struct RowMaps {
    CUtensorMap b16, b64, b256;
};

struct GroupedParams {
    int E, m, n, k, n_src, kb_total, tiles_w;
    int64_t ld_out, ld_x;
    const __nv_bfloat16 *x;   // gathered rows
    __nv_bfloat16 *out;
    const int32_t *offsets, *row_ids;
    int32_t *dev_status;
    int paired;   // rows of out start on 4 bytes: two columns a store
    int ranks;    // SPLIT: CTAs of a cluster
    WaitRule wait;
};

// Row tiles of a group of cnt rows, and the rows of each but the last: even shares (in multiples of
// STEP: 16, or 32 for a pair of CTAs, which takes half each) of up to 8 tiles, whole tiles of 256 for
// larger groups.  (t <= 8 shares leave rows for the last: they pass cnt / t by less than 32 each,
// 31 (t - 1) in all, and cnt / t > 256 (t - 1) / t >= 32 (t - 1).)
E3_DEV int row_tiles(int cnt) { return (cnt + MAX_ROWS - 1) / MAX_ROWS; }
template <int STEP>
E3_DEV int round_rows(int rows) {
    return (rows + STEP - 1) / STEP * STEP;
}
template <int STEP>
E3_DEV int tile_rows(int cnt, int tiles) {
    return tiles > 8 ? MAX_ROWS : round_rows<STEP>((cnt + tiles - 1) / tiles);
}

// Weight tile mt (of both CTAs of a pair) of group e by rows [row0, row0 + rows), the MMA's N = n16.
struct Unit {
    int e, mt, row0, rows, n16;
};

template <int STEP>
E3_DEV Unit unit_at(const Shared &sh, const GroupedParams &p, int u) {
    const int q = u / p.tiles_w;
    int lo = 0, hi = p.E;   // tiles[lo] <= q < tiles[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (sh.tiles[mid] <= q)
            lo = mid;
        else
            hi = mid;
    }
    Unit w;
    w.e = lo;
    const int tiles = sh.tiles[lo + 1] - sh.tiles[lo], local = u - sh.tiles[lo] * p.tiles_w;
    const int cnt = sh.offsets[lo + 1] - sh.offsets[lo], per = tile_rows<STEP>(cnt, tiles);
    const int rt = local % tiles;
    w.mt = local / tiles;
    w.row0 = sh.offsets[lo] + rt * per;
    w.rows = min(per, cnt - rt * per);
    w.n16 = round_rows<STEP>(w.rows);
    return w;
}

// The division by the special function unit: straight-line code, so that a warp, which has its
// scheduler almost to itself here, works on many columns at once.  (An IEEE division is a branch per
// value; with it the SwiGLU epilogue took twice the main loop's time at k = 4096.)  The exponential is 2 +
// 1.2 |x| steps of fp32 off at the most and the division 2, against a bf16 result's 2^15; 0 where exp(-x)
// passes 2^126 (x below -87.3, where silu is above -2^-119).
E3_DEV float silu(float x) { return __fdividef(x, 1.0f + __expf(-x)); }

// 16 bytes to shared memory, or 16 zero bytes (src is not read then)
E3_DEV void copy16(uint32_t dst, const void *src, bool zero) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(zero ? 0 : 16) : "memory");
}
// arrive on bar once this thread's copies so far have landed
E3_DEV void copies_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];\n" ::"r"(bar) : "memory");
}
// Barrier `id` over two warps; the variant with a flag tells whether it was set for all threads.
E3_DEV void pair_sync(int id) { asm volatile("bar.sync %0, 64;\n" ::"r"(id) : "memory"); }
E3_DEV bool pair_all(int id, bool v) {
    uint32_t r;
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.u32 p, %2, 0;\n bar.red.and.pred q, %1, 64, p;\n selp.u32 %0, 1, 0, q;\n}\n"
        : "=r"(r)
        : "r"(id), "r"(v ? 1u : 0u)
        : "memory");
    return r != 0;
}

// Two neighbouring columns of a row, col even; the second may lie past n.
E3_DEV void store_pair(const GroupedParams &p, int row, int col, float a, float b) {
    __nv_bfloat16 *o = p.out + (size_t)row * p.ld_out + col;
    if (p.paired && col + 1 < p.n) {
        *reinterpret_cast<__nv_bfloat162 *>(o) = __floats2bfloat162_rn(a, b);
    } else {
        if (col < p.n) o[0] = __float2bfloat16_rn(a);
        if (col + 1 < p.n) o[1] = __float2bfloat16_rn(b);
    }
}

// PAIR: two CTAs of a cluster work on one unit, 256 weight rows (128 each) by up to 256 rows (half loaded by
// each), with MMAs that the even CTA issues for both.  Each SM's shared memory then takes 32 KB of loads and
// 32 KB of operand reads a k-block in place of 48 and 48, which at 128 bytes a cycle are 512 cycles, the MMAs'
// own time, in place of 750 (3840 rows x 8 of 64 experts, k = 4096, 2 x 1024 columns: 377 -> 325 us in a
// burst of a dozen calls; k = 1024, 4096 columns: 206 -> 179 us; in longer runs 339 to 374 by GPU and clock, 1520 to
// 1380 TFLOP/s, and 192 to 204).  The odd CTA's stages are announced to the even one by a thread that waits for them
// and arrives on its barrier, at cluster scope; commits go to the barriers of both.

// SPLIT: a cluster of p.ranks CTAs works on one unit, each on a range of the k-blocks, where the units leave SMs
// idle.  Chunks of 8 rows of the tile belong to the ranks in turn: each sends the others their chunks of its sums
// by remote stores over their rings, adds up its own in rank order and finishes them.
enum { SINGLE, PAIRED, SPLIT_K };
constexpr int SPLIT_ROWS = 8;   // rows of a chunk
__host__ __device__ constexpr int split_bytes(int ranks) {
    return ranks * ((MAX_ROWS / SPLIT_ROWS + ranks - 1) / ranks) * SPLIT_ROWS * BM * 4;
}
static_assert(split_bytes(2) <= RING_BYTES && split_bytes(3) <= RING_BYTES && split_bytes(4) <= RING_BYTES &&
                  split_bytes(5) <= RING_BYTES && split_bytes(6) <= RING_BYTES && split_bytes(7) <= RING_BYTES &&
                  split_bytes(8) <= RING_BYTES,
              "the ranks' sums fit the ring");

template <bool SWIGLU, bool GATHER, int MODE>
__global__ void __launch_bounds__(NTHREADS + (GATHER ? 32 * GATHER_WARPS : 0), 1)
    grouped_kernel(const __grid_constant__ RowMaps tm_x, const __grid_constant__ CUtensorMap tm_w,
                   const __grid_constant__ CUtensorMap tm_w2, const GroupedParams p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *ring = smem_raw + (-smem_u32(smem_raw) & 1023u);   // (the compiler knows it as shared memory)
    Shared &sh = *reinterpret_cast<Shared *>(ring + RING_BYTES);
    const uint32_t tid = tc::thread_index();
    const int warp = (int)(tid >> 5), lane = (int)(tid & 31u);
    constexpr bool PAIR = MODE == PAIRED, SPLIT = MODE == SPLIT_K;
    constexpr int STEP = PAIR ? 32 : 16;
    const int rank = PAIR ? (int)(blockIdx.x & 1u) : 0;   // in the pair (a cluster of two)
    const int unit0 = SPLIT ? (int)blockIdx.x / p.ranks : (int)blockIdx.x >> (PAIR ? 1 : 0);
    const int unit_step = SPLIT ? (int)gridDim.x : (int)gridDim.x >> (PAIR ? 1 : 0);   // (SPLIT: one unit)
    const int part = SPLIT ? (int)blockIdx.x % p.ranks : 0;                            // range of the k-blocks
    const int kb0 = SPLIT ? (int)((long long)p.kb_total * part / p.ranks) : 0;
    const int kb1 = SPLIT ? (int)((long long)p.kb_total * (part + 1) / p.ranks) : p.kb_total;

    if (threadIdx.x == 0) {
        for (int s = 0; s < MAX_STAGES; ++s) {
            // the load's arrival, the gathering threads', and in the even CTA of a pair the odd one's
            tc::mbar_init(&sh.full[s], 1 + (GATHER ? 32 * GATHER_WARPS : 0) + (PAIR && rank == 0 ? 1 : 0) +
                                           missing_arrivals(p.wait, s, SPLIT ? part : rank));
            tc::mbar_init(&sh.empty[s], 1);
        }
        for (int a = 0; a < 2; ++a) {
            tc::mbar_init(&sh.tfull[a], 1);
            tc::mbar_init(&sh.tempty[a], PAIR ? 8 : 4);
        }
        tc::mbar_init(&sh.mma_done, 1);
        sh.abort = 0;
        sh.max_rows = 16;
        tc::fence_barrier_init();
        if (!GATHER) {
            tc::prefetch_tmap(&tm_x.b16);
            tc::prefetch_tmap(&tm_x.b64);
            tc::prefetch_tmap(&tm_x.b256);
        }
        tc::prefetch_tmap(&tm_w);
        if (SWIGLU) tc::prefetch_tmap(&tm_w2);
    }
    if (warp == 1) {
        if (PAIR)
            tc::tmem2_alloc(&sh.tmem_base, TMEM_COLS);
        else
            tc::tmem_alloc(&sh.tmem_base, TMEM_COLS);
    }
    tc::fence_before();
    if (PAIR) {
        tc::cluster_sync();
    } else {
        __syncthreads();
    }
    tc::fence_after();
    const uint32_t tmem = sh.tmem_base;
    pdl_wait();   // the previous kernel's outputs: offsets, row ids, rows
    pdl_trigger();

    // the groups' row tiles
    bool bad = false;
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) {
        const int a = p.offsets[e], b = p.offsets[e + 1];
        const bool wrong = a < 0 || b < a || b > p.m || (e == 0 && a != 0);
        bad |= wrong;
        sh.offsets[e] = a;
        if (e == p.E - 1) sh.offsets[p.E] = b;
        if (!wrong && b > a) {   // (differences and tile counts of wild offsets would overflow)
            const int tiles = row_tiles(b - a);
            sh.tiles[e] = tiles;
            const int rows = tile_rows<STEP>(b - a, tiles) / (PAIR ? 2 : 1);   // of this CTA
            // (box_rows never decreases: a group's last tile needs no more)
            atomicMax(&sh.max_rows, GATHER ? rows : box_rows(rows));
        } else {
            sh.tiles[e] = 0;
        }
    }
    bad = __syncthreads_or(bad);
    if (warp == 0) {   // exclusive prefix sums, 32 groups at a time
        int run = 0;
        for (int e0 = 0; e0 < p.E; e0 += 32) {
            const int v = e0 + lane < p.E ? sh.tiles[e0 + lane] : 0;
            int inc = v;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int up = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += up;
            }
            if (e0 + lane < p.E) sh.tiles[e0 + lane] = run + inc - v;
            run += __shfl_sync(0xffffffffu, inc, 31);
        }
        if (lane == 0) sh.tiles[p.E] = run;
    }
    __syncthreads();
    const int units = bad ? 0 : sh.tiles[p.E] * p.tiles_w;
    if (bad && blockIdx.x == 0 && threadIdx.x == 0) flag(p.dev_status, EAGLE3_DEV_BAD_COUNTS);
    const int stage_bytes = W_BYTES + sh.max_rows * ROW_BYTES;   // a multiple of 2048
    // whole 1024-byte blocks keep the swizzle's phase; the deepest ring that fits
    const int stages = min(MAX_STAGES, RING_BYTES / stage_bytes);

    const uint32_t ring0 = smem_u32(ring), full0 = smem_u32(sh.full), empty0 = smem_u32(sh.empty);
    const uint32_t tfull0 = smem_u32(sh.tfull), tempty0 = smem_u32(sh.tempty), abort0 = smem_u32(&sh.abort);

    if (warp == 0) {
        // ------------------------------------------------------------------ TMA producer
        if (tc::elect_one()) {
            int stage = 0;
            uint32_t phase = 0, last_parity = 0, issued = 0;   // parity of the last load per stage
            bool ok = true;
            for (int u = unit0; ok && u < units; u += unit_step) {
                const Unit w = unit_at<STEP>(sh, p, u);
                const int mine = w.n16 / (PAIR ? 2 : 1), boxes = box_rows(mine);   // rows that this CTA loads
                const int row0 = w.row0 + rank * mine, mt = PAIR ? 2 * w.mt + rank : w.mt;
                for (int kb = kb0; kb < kb1; ++kb) {
                    const uint32_t full = full0 + stage * 8;
                    if (!tc::mbar_wait(empty0 + stage * 8, phase ^ 1u, abort0, p.wait.limit)) {
                        ok = false;
                        break;
                    }
                    tc::mbar_expect_tx(full, W_BYTES + (GATHER ? 0 : boxes * ROW_BYTES));
                    issued |= 1u << stage;
                    last_parity = (last_parity & ~(1u << stage)) | (phase << stage);
                    const uint32_t sw = ring0 + stage * stage_bytes, sx = sw + W_BYTES;
                    const int x = kb * BK;
                    if (SWIGLU) {
                        tc::tma_load_3d(sw, &tm_w, x, mt * (BM / 2), w.e, full);
                        tc::tma_load_3d(sw + W_BYTES / 2, &tm_w2, x, mt * (BM / 2), w.e, full);
                    } else {
                        tc::tma_load_3d(sw, &tm_w, x, mt * BM, w.e, full);
                    }
                    if (!GATHER) {
                        if (boxes == 256) {
                            tc::tma_load_2d(sx, &tm_x.b256, x, row0, full);
                        } else {
                            int r = 0;
                            for (; r + 64 <= boxes; r += 64)
                                tc::tma_load_2d(sx + r * ROW_BYTES, &tm_x.b64, x, row0 + r, full);
                            if (r < boxes) tc::tma_load_2d(sx + r * ROW_BYTES, &tm_x.b16, x, row0 + r, full);
                        }
                    }
                    if (++stage == stages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            if (!ok) flag(p.dev_status, EAGLE3_DEV_TIMEOUT);
            // no TMA write may still be in flight when the CTA exits: wait (bounded) for the last load
            // issued to every stage; these return at once when the loads were consumed
            const uint32_t t0 = tc::kiloclock();
            for (int st = 0; st < stages; ++st)
                if ((issued >> st) & 1u) tc::mbar_drain(full0 + st * 8, (last_parity >> st) & 1u, t0, p.wait.limit);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------------ MMA issuer
        if (PAIR && rank == 1) {
            // the odd CTA: its stages to the even one's barriers
            if (tc::elect_one()) {
                const uint32_t even = tc::cluster_addr(full0, 0);
                int stage = 0;
                uint32_t phase = 0;
                bool ok = true;
                for (int u = unit0; ok && u < units; u += unit_step)
                    for (int kb = kb0; kb < kb1; ++kb) {
                        if (!tc::mbar_wait(full0 + stage * 8, phase, abort0, p.wait.limit)) {
                            ok = false;
                            break;
                        }
                        if (GATHER) tc::fence_proxy_async_smem();   // the copies were made outside the async proxy
                        tc::mbar_arrive_cluster_smem(even + stage * 8);
                        if (++stage == stages) {
                            stage = 0;
                            phase ^= 1u;
                        }
                    }
                if (!ok) flag(p.dev_status, EAGLE3_DEV_TIMEOUT);
            }
        } else if (tc::elect_one()) {
            const uint64_t desc0 = tc::desc_sw128(ring0);
            int stage = 0, acc = 0;
            uint32_t phase = 0, acc_phase = 0;
            bool ok = true;
            for (int u = unit0; ok && u < units; u += unit_step) {
                const Unit w = unit_at<STEP>(sh, p, u);
                const uint32_t idesc = tc::idesc_bf16(PAIR ? 2 * BM : BM, w.n16);
                if (!tc::mbar_wait(tempty0 + acc * 8, acc_phase ^ 1u, abort0, p.wait.limit)) {
                    ok = false;
                    break;
                }
                tc::fence_after();
                const uint32_t d = tmem + (uint32_t)(acc * MAX_ROWS);
                for (int kb = kb0; kb < kb1; ++kb) {
                    const uint32_t full = full0 + stage * 8;
                    if (!(PAIR ? tc::mbar_wait_cluster_smem(full, phase, abort0, p.wait.limit)
                               : tc::mbar_wait(full, phase, abort0, p.wait.limit))) {
                        ok = false;
                        break;
                    }
                    if (GATHER) tc::fence_proxy_async_smem();   // the copies were made outside the async proxy
                    tc::fence_after();
                    // (descriptors count 16 bytes)
                    const uint64_t a = desc0 + (uint32_t)(stage * stage_bytes >> 4), b = a + (W_BYTES >> 4);
#pragma unroll
                    for (int k = 0; k < BK / 16; ++k) {
                        const uint32_t add = kb > kb0 || k > 0 ? 1u : 0u;
                        if (PAIR)
                            tc::mma2_bf16_ss(d, a + k * 2, b + k * 2, idesc, add);
                        else
                            tc::mma_bf16_ss(d, a + k * 2, b + k * 2, idesc, add);
                    }
                    if (PAIR)
                        tc::mma2_commit(empty0 + stage * 8, 3);
                    else
                        tc::mma_commit(empty0 + stage * 8);
                    if (++stage == stages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (!ok) break;
                if (PAIR)
                    tc::mma2_commit(tfull0 + acc * 8, 3);
                else
                    tc::mma_commit(tfull0 + acc * 8);
                acc_phase ^= (uint32_t)acc;
                acc ^= 1;
            }
            if (!ok) flag(p.dev_status, EAGLE3_DEV_TIMEOUT);
            // every MMA this thread issued must retire before TMEM is freed (bounded wait)
            if (PAIR)
                tc::mma2_commit(smem_u32(&sh.mma_done), 1);
            else
                tc::mma_commit(smem_u32(&sh.mma_done));
            tc::mbar_drain(smem_u32(&sh.mma_done), 0, tc::kiloclock(), p.wait.limit);
        }
        __syncwarp();
    } else if (GATHER && warp >= 6) {
        // ------------------------------------------------------------------ row gather (warps 6..13)
        // Thread t copies 16-byte piece t % 8 of rows t / 8 + 32 i; its arrival on the stage's barrier
        // follows its copies by itself.
        const int t = (int)tid - NTHREADS, piece = t & 7, first = t >> 3;
        const uint32_t dst0 = ring0 + W_BYTES + first * ROW_BYTES + ((piece ^ (first & 7)) << 4);
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int u = unit0; ok && u < units; u += unit_step) {
            const Unit w = unit_at<STEP>(sh, p, u);
            constexpr int PASSES = MAX_ROWS / (PAIR ? 2 : 1) / GATHER_ROWS;
            const int mine = w.n16 / (PAIR ? 2 : 1), from = rank * mine + first;   // rows that this CTA copies
            const __nv_bfloat16 *src[PASSES];
#pragma unroll
            for (int i = 0; i < PASSES; ++i) {
                if (GATHER_ROWS * i >= mine) continue;
                // rows past the tile's last repeat it
                int v = __ldg(p.row_ids + w.row0 + min(from + GATHER_ROWS * i, w.rows - 1));
                if (v < 0 || v >= p.n_src) {
                    flag(p.dev_status, EAGLE3_DEV_BAD_COUNTS);
                    v = 0;
                }
                src[i] = p.x + (size_t)v * p.ld_x + piece * 8;
            }
            for (int kb = kb0; kb < kb1; ++kb) {
                if (!tc::mbar_wait_warp(empty0 + stage * 8, phase ^ 1u, abort0, p.wait.limit)) {
                    ok = false;
                    break;
                }
                const uint32_t dst = dst0 + stage * stage_bytes;
                const bool past = kb * BK + piece * 8 >= p.k;   // k is a multiple of 8
                const int at = past ? 0 : kb * BK;
#pragma unroll
                for (int i = 0; i < PASSES; ++i)
                    if (first + GATHER_ROWS * i < mine) copy16(dst + i * GATHER_ROWS * ROW_BYTES, src[i] + at, past);
                copies_arrive(full0 + stage * 8);
                if (++stage == stages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
        asm volatile("cp.async.wait_all;\n" ::: "memory");
        if (!ok && lane == 0) flag(p.dev_status, EAGLE3_DEV_TIMEOUT);
    } else {
        // ------------------------------------------------------------------ epilogue (warps 2..5)
        const int quarter = warp & 3;   // TMEM lanes 32 * quarter .. + 31
        const uint32_t tempty_even = PAIR ? tc::cluster_addr(tempty0, 0) : tempty0;
        int acc = 0;
        uint32_t acc_phase = 0;
        Unit unit = {};   // SPLIT: the cluster's
        for (int u = unit0; u < units; u += unit_step) {
            const Unit w = unit_at<STEP>(sh, p, u);
            bool ok = tc::mbar_wait_warp(tfull0 + acc * 8, acc_phase, abort0, p.wait.limit);
            // (the two warps of a pair go on or leave together: they meet at barriers below)
            if (SWIGLU) ok = pair_all(1 + (quarter & 1), ok);
            if (!ok) {
                if (lane == 0) flag(p.dev_status, EAGLE3_DEV_TIMEOUT);
                break;
            }
            tc::fence_after();
            const uint32_t t_col = tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(acc * MAX_ROWS);
            if (SPLIT) {
                unit = w;
                tc::cluster_sync();   // all ranks' loads and MMAs have completed
                const int chunks = w.n16 / SPLIT_ROWS, each = (chunks + p.ranks - 1) / p.ranks;
                for (int c = 0; c < w.n16; c += 32) {
                    float v[32];
                    tc::tmem_ld32(t_col + c, v);
#pragma unroll
                    for (int i = 0; i < 32; i += SPLIT_ROWS) {
                        const int j = (c + i) / SPLIT_ROWS, to = j % p.ranks;
                        if (j >= chunks) continue;
                        const int word = (part * each + j / p.ranks) * SPLIT_ROWS * BM + quarter * 32 + lane;
                        const uint32_t at = tc::cluster_addr(ring0, to) + (uint32_t)(word * 4);
#pragma unroll
                        for (int r = 0; r < SPLIT_ROWS; ++r) tc::cluster_st(at + r * BM * 4, v[i + r]);
                    }
                }
                break;
            }
            const bool odd = lane & 1;
            const int mt = PAIR ? 2 * w.mt + rank : w.mt;
            // rows r, r + 1, ... of this lane's column: an even lane stores both columns of row r, its
            // odd neighbour those of row r + 1
            auto store32 = [&](float (&v)[32], int r0, int col) {
#pragma unroll
                for (int i = 0; i < 32; i += 2) {
                    const float other = __shfl_xor_sync(0xffffffffu, odd ? v[i] : v[i + 1], 1);
                    v[i] = odd ? other : v[i];
                    v[i + 1] = odd ? v[i + 1] : other;
                }
                const int first = r0 + (odd ? 1 : 0);
                if (p.paired && r0 + 32 <= w.rows && (col | 1) < p.n) {   // no row or column to leave out
                    uint8_t *o = (uint8_t *)(p.out + (size_t)(w.row0 + first) * p.ld_out + col);
                    const size_t step = (size_t)p.ld_out * 4;   // two rows
#pragma unroll
                    for (int i = 0; i < 32; i += 2, o += step)
                        *reinterpret_cast<__nv_bfloat162 *>(o) = __floats2bfloat162_rn(v[i], v[i + 1]);
                } else {
#pragma unroll
                    for (int i = 0; i < 32; i += 2)
                        if (first + i < w.rows) store_pair(p, w.row0 + first + i, col, v[i], v[i + 1]);
                }
                __syncwarp();   // (what follows, TMEM loads or a pair's barrier, wants the whole warp)
            };
            if (SWIGLU) {
                const int pair = quarter & 1, up = quarter >> 1;
                const int col = mt * (BM / 2) + pair * 32 + (lane & ~1);
                for (int c = 0; c < w.n16; c += 64) {   // the gate warp takes rows c.., the up warp c + 32..
                    const int mine = c + 32 * up, theirs = c + 32 * (up ^ 1);
                    float v[32];
                    if (theirs < w.n16) {
                        tc::tmem_ld32(t_col + theirs, v);
#pragma unroll
                        for (int i = 0; i < 32; ++i) sh.swap[pair][up][i * 32 + lane] = v[i];
                    }
                    pair_sync(1 + pair);
                    if (mine < w.n16) {
                        tc::tmem_ld32(t_col + mine, v);
                        const float *o = sh.swap[pair][up ^ 1] + lane;
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            const float other = o[i * 32];
                            v[i] = silu(up ? other : v[i]) * (up ? v[i] : other);
                        }
                        store32(v, mine, col);
                    }
                    pair_sync(1 + pair);   // both have read before the next rows overwrite
                }
            } else {
                const int col = mt * BM + quarter * 32 + (lane & ~1);
                for (int c = 0; c < w.n16; c += 32) {
                    float v[32];
                    tc::tmem_ld32(t_col + c, v);
                    store32(v, c, col);
                }
            }
            tc::fence_before();
            __syncwarp();
            if (PAIR)
                tc::mbar_arrive_cluster_if(tempty_even + acc * 8, lane == 0);
            else
                tc::mbar_arrive_if(tempty0 + acc * 8, lane == 0);
            acc_phase ^= (uint32_t)acc;
            acc ^= 1;
        }
        __syncwarp();
        if (SPLIT) {
            if (unit.rows == 0) tc::cluster_sync();   // (no unit, or a timeout: its sums are void)
            tc::cluster_sync();
            // this rank's chunks: 128 threads take a column each, or with SwiGLU a pair's column and half of the rows
            const int t = (int)tid - 64, chunks = unit.n16 / SPLIT_ROWS, each = (chunks + p.ranks - 1) / p.ranks;
            const int c = SWIGLU ? t & 63 : t, col = unit.mt * (SWIGLU ? BM / 2 : BM) + c;
            constexpr int ROWS = SWIGLU ? SPLIT_ROWS / 2 : SPLIT_ROWS;
            for (int j = part; j < chunks; j += p.ranks) {
                const int first = SWIGLU ? (t >> 6) * ROWS : 0;
                const float *from = reinterpret_cast<const float *>(ring) + (j / p.ranks * SPLIT_ROWS + first) * BM + c;
                float a[ROWS], b[ROWS];
#pragma unroll
                for (int r = 0; r < ROWS; ++r) a[r] = b[r] = 0.0f;
                for (int s = 0; s < p.ranks; ++s, from += each * SPLIT_ROWS * BM) {   // in rank order
#pragma unroll
                    for (int r = 0; r < ROWS; ++r) {
                        a[r] += from[r * BM];
                        if (SWIGLU) b[r] += from[r * BM + BM / 2];
                    }
                }
#pragma unroll
                for (int r = 0; r < ROWS; ++r) {
                    const int row = j * SPLIT_ROWS + first + r;
                    if (row < unit.rows && col < p.n)
                        p.out[(size_t)(unit.row0 + row) * p.ld_out + col] =
                            __float2bfloat16_rn(SWIGLU ? silu(a[r]) * b[r] : a[r]);
                }
            }
            __syncwarp();
        }
    }
    if (SPLIT && (warp < 2 || warp >= 6)) {   // (the epilogue's two)
        tc::cluster_sync();
        tc::cluster_sync();
    }

    tc::fence_before();
    if (PAIR) {   // no CTA leaves while the other may arrive on its barriers or multiply into its TMEM
        tc::cluster_sync();
    } else {
        __syncthreads();
    }
    if (warp == 1) {
        __syncwarp();
        tc::fence_after();
        if (PAIR)
            tc::tmem2_dealloc(tmem, TMEM_COLS);
        else
            tc::tmem_dealloc(tmem, TMEM_COLS);
    }
}

// ---- host side ----------------------------------------------------------------------------------
eagle3_status_t validate(const eagle3_grouped_linear_args_t *a) {
    if (!a) return EAGLE3_ERR_INVALID_ARGUMENT;
    if (a->n_groups < 1 || a->m < 0 || a->n < 1 || a->k < 1) return EAGLE3_ERR_INVALID_ARGUMENT;
    if (a->epilogue < EAGLE3_EPI_BF16 || a->epilogue > EAGLE3_EPI_BF16_ROPE) return EAGLE3_ERR_INVALID_ARGUMENT;
    if (a->epilogue != EAGLE3_EPI_BF16 && a->epilogue != EAGLE3_EPI_SWIGLU) return EAGLE3_ERR_UNSUPPORTED;
    if (a->n_groups > MAX_E || a->k % 8) return EAGLE3_ERR_UNSUPPORTED;
    if (a->m > MAX_DIM || a->n > MAX_DIM || a->k > MAX_DIM) return EAGLE3_ERR_UNSUPPORTED;
    const int64_t ld_x = a->ld_x ? a->ld_x : a->k, ld_w = a->ld_w ? a->ld_w : a->k, ld_o = a->ld_out ? a->ld_out : a->n;
    if (ld_x < a->k || ld_w < a->k || ld_o < a->n || ld_x % 8 || ld_w % 8) return EAGLE3_ERR_INVALID_ARGUMENT;
    if (a->m == 0) return EAGLE3_OK;
    if (!a->x || !a->w || !a->out || !a->offsets) return EAGLE3_ERR_INVALID_ARGUMENT;
    if (a->epilogue == EAGLE3_EPI_SWIGLU && !a->w2) return EAGLE3_ERR_INVALID_ARGUMENT;
    if (a->row_ids && a->n_src < 1) return EAGLE3_ERR_INVALID_ARGUMENT;
    if (((uintptr_t)a->x | (uintptr_t)a->w | (uintptr_t)a->w2) & 15) return EAGLE3_ERR_INVALID_ARGUMENT;
    if (((uintptr_t)a->offsets | (uintptr_t)a->row_ids | (uintptr_t)a->dev_status) & 3 || (uintptr_t)a->out & 1)
        return EAGLE3_ERR_INVALID_ARGUMENT;
    // units are counted in 32 bits
    if ((int64_t)((a->n + 63) / 64) * (a->m / MAX_ROWS + a->n_groups) > MAX_DIM) return EAGLE3_ERR_UNSUPPORTED;
    return EAGLE3_OK;
}

// CTAs, or clusters of `ranks`, that the device holds at once (a GPC with an odd number of SMs leaves one without
// a partner); -1 on an error.
template <bool SWIGLU, bool GATHER, int MODE>
int resident(int ranks) {
    const auto kernel = grouped_kernel<SWIGLU, GATHER, MODE>;
    return ranks == 1 ? resident_ctas(kernel, SMEM)
                      : resident_clusters(kernel, ranks, NTHREADS + (GATHER ? 32 * GATHER_WARPS : 0), SMEM);
}

template <bool SWIGLU, bool GATHER, int MODE>
cudaError_t launch_mode(int clusters, int ranks, cudaStream_t st, const RowMaps &tx, const CUtensorMap &tw,
                        const CUtensorMap &tw2, const GroupedParams &p) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)clusters * ranks);
    cfg.blockDim = dim3(NTHREADS + (GATHER ? 32 * GATHER_WARPS : 0));
    cfg.dynamicSmemBytes = SMEM;
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = ranks;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = ranks > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, grouped_kernel<SWIGLU, GATHER, MODE>, tx, tw, tw2, p);
}

// row_tiles: an upper bound on the call's row tiles
template <bool SWIGLU, bool GATHER>
cudaError_t launch_grouped(int64_t row_tiles, cudaStream_t st, const RowMaps &tx, const CUtensorMap &tw,
                           const CUtensorMap &tw2, GroupedParams &p) {
    static PerDevice<ClusterCounts> singles, pairs, splits;
    const ClusterCounts split = splits.get([] {
        ClusterCounts c = {};
        for (int r = 2; r <= MAX_CLUSTER; ++r) c.n[r] = resident<SWIGLU, GATHER, SPLIT_K>(r);
        return c;
    });
    if (!succeeded(split)) return cudaErrorUnknown;   // (not "none are resident": the cut decides the order of sums)
    // Few units: as many ranks as leave every unit a resident cluster, if that saves each CTA 6 k-blocks, and one
    // more for each 16 rows of a tile: a k-block takes 0.2 us, and sending, meeting and adding up 1 us for a few
    // rows, 5 us for 256.  (2 rows, 2 groups, 1024 columns: k = 14336 45 us by single CTAs, 15 by eight ranks, k =
    // 1024 7.3 and 6.0, k = 512 5.7 and 5.8; 500 rows, 2 groups, 512 columns: k = 4096 20 and 13, k = 1024 9.2 and 11.)
    // Every rank has a k-block: without one it would send what an earlier kernel left in tensor memory.
    p.ranks = 1;
    for (int r = 2; r <= std::min(MAX_CLUSTER, p.kb_total); ++r)
        if (row_tiles * p.tiles_w <= split.n[r] && p.kb_total - p.kb_total / r >= 6 + std::min(p.m, MAX_ROWS) / 16)
            p.ranks = r;
    if (p.ranks > 1)
        return launch_mode<SWIGLU, GATHER, SPLIT_K>((int)(row_tiles * p.tiles_w), p.ranks, st, tx, tw, tw2, p);
    // Pairs of CTAs, unless the last pair's odd CTA would be without weight rows and that is more than a
    // sixth of the work: one tile of weight rows (2048 rows x 8 of 64 experts, k = 4096, 128 columns) takes
    // 33 us by single CTAs and 53 us by pairs, three tiles 68 and 74 us, 16 tiles (3840 rows, 2 x 1024
    // columns) 377 and 325 us.  With few rows, where the weights' bytes bound the call, both are alike.
    if (p.tiles_w % 2 == 0 || p.tiles_w >= 5) {
        p.tiles_w = (p.tiles_w + 1) / 2;
        const ClusterCounts most = pairs.get([] { return ClusterCounts{{0, resident<SWIGLU, GATHER, PAIRED>(2)}}; });
        if (most.n[1] < 1) return cudaErrorUnknown;
        const int pairs_used = (int)std::min<int64_t>(most.n[1], row_tiles * p.tiles_w);
        return launch_mode<SWIGLU, GATHER, PAIRED>(pairs_used, 2, st, tx, tw, tw2, p);
    }
    const ClusterCounts most = singles.get([] { return ClusterCounts{{0, resident<SWIGLU, GATHER, SINGLE>(1)}}; });
    if (most.n[1] < 1) return cudaErrorUnknown;
    const int ctas = (int)std::min<int64_t>(most.n[1], row_tiles * p.tiles_w);
    return launch_mode<SWIGLU, GATHER, SINGLE>(ctas, 1, st, tx, tw, tw2, p);
}

}  // namespace
}  // namespace e3

using namespace e3;

static eagle3_status_t grouped_linear(const eagle3_grouped_linear_args_t *a, const WaitRule &wait,
                                      eagle3_stream_t stream) {
    const eagle3_status_t st = validate(a);
    if (st != EAGLE3_OK || a->m == 0) return st;
    const bool swiglu = a->epilogue == EAGLE3_EPI_SWIGLU;
    const int64_t ld_x = a->ld_x ? a->ld_x : a->k, ld_w = a->ld_w ? a->ld_w : a->k;
    const CUtensorMapDataType bf = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    CUtensorMap tw, tw2;
    RowMaps tx;
    if (!tmap_rows(&tw, bf, 2, a->w, a->n, a->k, ld_w, swiglu ? BM / 2 : BM, a->n_groups, a->n * ld_w))
        return EAGLE3_ERR_CUDA;
    tw2 = tx.b16 = tx.b64 = tx.b256 = tw;   // where unused
    if (swiglu && !tmap_rows(&tw2, bf, 2, a->w2, a->n, a->k, ld_w, BM / 2, a->n_groups, a->n * ld_w))
        return EAGLE3_ERR_CUDA;
    if (!a->row_ids && (!tmap_rows(&tx.b16, bf, 2, a->x, a->m, a->k, ld_x, 16) ||
                        !tmap_rows(&tx.b64, bf, 2, a->x, a->m, a->k, ld_x, 64) ||
                        !tmap_rows(&tx.b256, bf, 2, a->x, a->m, a->k, ld_x, 256)))
        return EAGLE3_ERR_CUDA;
    GroupedParams p;
    p.E = a->n_groups;
    p.m = a->m;
    p.n = a->n;
    p.k = a->k;
    p.n_src = a->n_src;
    p.kb_total = (a->k + BK - 1) / BK;
    p.tiles_w = (a->n + (swiglu ? 63 : BM - 1)) / (swiglu ? 64 : BM);
    p.ld_out = a->ld_out ? a->ld_out : a->n;
    p.ld_x = ld_x;
    p.x = (const __nv_bfloat16 *)a->x;
    p.out = (__nv_bfloat16 *)a->out;
    p.offsets = a->offsets;
    p.row_ids = a->row_ids;
    p.dev_status = a->dev_status;
    p.wait = wait;
    p.paired = p.ld_out % 2 == 0 && ((uintptr_t)a->out & 3) == 0;
    const int64_t row_tiles = a->m / MAX_ROWS + std::min(a->m, a->n_groups);
    const cudaStream_t s = (cudaStream_t)stream;
    const cudaError_t e = swiglu ? (a->row_ids ? launch_grouped<true, true>(row_tiles, s, tx, tw, tw2, p)
                                               : launch_grouped<true, false>(row_tiles, s, tx, tw, tw2, p))
                                 : (a->row_ids ? launch_grouped<false, true>(row_tiles, s, tx, tw, tw2, p)
                                               : launch_grouped<false, false>(row_tiles, s, tx, tw, tw2, p));
    return e == cudaSuccess ? EAGLE3_OK : EAGLE3_ERR_CUDA;
}

extern "C" eagle3_status_t eagle3_grouped_linear(const eagle3_grouped_linear_args_t *a, eagle3_stream_t stream) {
    return grouped_linear(a, WaitRule(), stream);
}

extern "C" eagle3_status_t eagle3_test_grouped_linear_timeout(const eagle3_grouped_linear_args_t *a, int32_t stall_block,
                                                              int32_t stall_rank, int64_t wait_limit_cycles,
                                                              eagle3_stream_t stream) {
    WaitRule wait;
    if (!stall_rule(&wait, stall_block, stall_rank, wait_limit_cycles)) return EAGLE3_ERR_INVALID_ARGUMENT;
    return grouped_linear(a, wait, stream);
}
