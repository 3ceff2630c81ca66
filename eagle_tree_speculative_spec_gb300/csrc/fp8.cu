// eagle3_quantize_fp8 and eagle3_linear_fp8: 8-bit projections, y = x W^T with e4m3 values, a scale
// for each row and 128 columns of x and one for each 128 x 128 block of W (the projections of
// "EAGLE-3: Engineering Implementation of LLM Inference Acceleration", section VIII and appendix C,
// for a target held in 8 bits).
//
// The scales change every 128 columns of k, so the tensor cores can only sum over one such block:
// each k-block's product goes to a TMEM buffer of its own, and the epilogue warps add it, times its
// two scales, to fp32 accumulators in registers while the next block's MMAs run.  (This also keeps
// the long sum out of the tensor cores' accumulation.)
//
// Two kernels (the rule between them stands at the launch), both warp-specialised: warp 0 loads by TMA into a
// ring, a lane of warp 1 issues tcgen05.mma (kind::f8f6f4, K = 32) and the other warps run the epilogue.
//   wide     128 rows x 256 weight rows a tile, persistent.  Rows are the M side, so a thread owns one
//            row and its scale is one number a k-block.
//   narrow   128 weight rows (M side) x up to 64 rows (N side, any multiple of 16): few rows, bound by
//            the weights' bytes.
// Where the tiles do not fill the GPU, the k-blocks of a tile are cut over the CTAs of a thread-block
// cluster; the ranks' sums meet in distributed shared memory and are added in rank order.
//
// Every mbarrier wait is bounded; on a timeout the kernel records EAGLE3_DEV_TIMEOUT, stops issuing
// work, drains its own TMA loads and frees its TMEM.
#include <algorithm>

#include <cuda_fp8.h>

#include "../../include/eagle3_fp8.h"
#include "../../include/eagle3_testing.h"
#include "tc.cuh"
#include "tmap.cuh"

namespace e3 {
namespace {

constexpr int BK = 128;                 // k values of a block and of a tile (128 bytes)
constexpr int BM = 128;
constexpr float E4M3_MAX = 448.0f;

// (By the special function unit: the exponential is 2 + 1.2 |x| steps of fp32 off at the most and the division
// 2, against a bf16 result's 2^15; 0 where exp(-x) passes 2^126, x below -87.3, where silu is above -2^-119.)
E3_DEV float silu(float x) { return __fdividef(x, 1.0f + __expf(-x)); }

struct Fp8Params {
    int m, n, k, epi, kb_total, n_blocks;   // n_blocks: row blocks of w_scale
    int64_t ld_out, ld_res;
    const float *x_scale, *w_scale, *w2_scale;
    const __nv_bfloat16 *residual;
    void *out;
    int32_t *dev_status;
    int tiles_m, tiles_n;   // wide: row tiles, column tiles
    int ranks;              // OUT_SPLIT: CTAs of a cluster, each a range of a tile's k-blocks (one tile a cluster)
    int tma_out;            // wide: outputs leave through shared memory and TMA stores
    int n16, stages;        // narrow: rows of a tile (multiple of 16), ring depth
    WaitRule wait;
};

// ---- quantisation -------------------------------------------------------------------------------
constexpr int QUANT_THREADS = 128;

struct QuantParams {
    int m, k;
    int64_t ld_x, ld_q;
    const __nv_bfloat16 *x;
    uint8_t *q;
    float *scale;
};

// The codes of a lane's 8 values by IEEE division.
__device__ __noinline__ uint2 codes_exact(uint4 raw, float s) {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    uint32_t q[2] = {0u, 0u};
#pragma unroll 1
    for (int i = 0; i < 4; ++i) {
        const float2 v = make_float2(__fdiv_rn(__uint_as_float(w[i] << 16), s),
                                     __fdiv_rn(__uint_as_float(w[i] & 0xffff0000u), s));
        const uint32_t c = (uint32_t)__nv_cvt_float2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3);
        if (i < 2)
            q[0] |= c << (16 * i);
        else
            q[1] |= c << (16 * (i - 2));
    }
    return make_uint2(q[0], q[1]);
}

// Quotients without a division (IEEE divisions made the kernel issue-bound: 42 us for 3840 x 14336 against
// 25 us of bytes).  With y the correctly rounded 1 / b and q0 = a y, q = q0 + (a - q0 b) y (each operation
// rounded once) is a / b correctly rounded: Markstein's correction step ("Computation of elementary
// functions on the IBM RISC System/6000 processor", 1990); y itself is one Newton step from an
// approximation.  His theorem wants q0 within a step of the quotient, which a y need not be; but a block's
// maximum and its values are bf16 numbers and the scale is such a number over 448, so that there are 128
// significands of scales and 128 x 128 of quotients: all were checked (for y0 up to 3 steps off), and
// powers of two change nothing as long as nothing under- or overflows (maxima from 2^-80 on).
constexpr uint32_t QUANT_LEAST = 0x1780u;   // bf16 bits of 2^-80
E3_DEV float scale_of(uint32_t top) {       // top: bf16 bits of the block's maximum, QUANT_LEAST or more
    constexpr float Y = 0x1.24924ap-9f;     // 1 / 448 rounded to nearest
    const float a = __uint_as_float(top << 16), q0 = a * Y;
    return fmaf(fmaf(-q0, E4M3_MAX, a), Y, q0);
}
E3_DEV float reciprocal_of(float s) {
    float y0;
    asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(y0) : "f"(s));
    return fmaf(y0, fmaf(-s, y0, 1.0f), y0);
}
// e4m3(x / s) for 8 values, y = 1 / s.  -0 keeps its sign.
E3_DEV uint2 codes(uint4 raw, float s, float y) {
    const float2 y2 = make_float2(y, y), s2 = make_float2(-s, -s);
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 x = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
        const float2 q0 = __fmul2_rn(x, y2);
        const float2 q = __ffma2_rn(__ffma2_rn(q0, s2, x), y2, q0);
        c[i] = (uint32_t)__nv_cvt_float2_to_fp8x2(q, __NV_SATFINITE, __NV_E4M3);
    }
    // (the signs of 4 values: the high bytes of two words)
    return make_uint2(c[0] | (c[1] << 16) | (__byte_perm(w[0], w[1], 0x7531) & 0x80808080u),
                      c[2] | (c[3] << 16) | (__byte_perm(w[2], w[3], 0x7531) & 0x80808080u));
}

// A half warp holds a block of 128 columns of one row, 8 values a lane; a warp takes two neighbouring
// blocks of R consecutive rows, all loads first, and writes the R scales of a block side by side.
template <int R, bool WHOLE>
E3_DEV void quantize_rows(const QuantParams &p, int row0, int col) {
    const int lane = threadIdx.x & 31;
    const bool in = col < p.k;   // k is a multiple of 16: 8 values are in or out together
    uint4 raw[R];
    const __nv_bfloat16 *x = p.x + (size_t)row0 * p.ld_x + col;
#pragma unroll
    for (int r = 0; r < R; ++r, x += p.ld_x) {
        raw[r] = make_uint4(0u, 0u, 0u, 0u);
        if (in && (WHOLE || row0 + r < p.m)) raw[r] = __ldcs(reinterpret_cast<const uint4 *>(x));
    }
    float scale = 0.0f;   // lane r of the half warp keeps row r's
    uint8_t *q = p.q + (size_t)row0 * p.ld_q + col;
#pragma unroll
    for (int r = 0; r < R; ++r, q += p.ld_q) {
        // |bf16| as integers: the largest of numbers, above them infinity, above that NaN
        uint32_t top = __vmaxu2(__vmaxu2(raw[r].x & 0x7fff7fffu, raw[r].y & 0x7fff7fffu),
                                __vmaxu2(raw[r].z & 0x7fff7fffu, raw[r].w & 0x7fff7fffu));
        top = max(top & 0xffffu, top >> 16);
#pragma unroll
        for (int o = 8; o; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));   // within 16 lanes
        float s;
        uint2 c;
        if (top >= QUANT_LEAST && top < 0x7f80u) {
            s = scale_of(top);
            c = codes(raw[r], s, reciprocal_of(s));
        } else {
            s = top >= 0x7f80u ? __int_as_float(0x7fffffff)
                : top == 0u    ? 1.0f
                               : __fdiv_rn(__uint_as_float(top << 16), E4M3_MAX);
            c = codes_exact(raw[r], s);
        }
        if (in && (WHOLE || row0 + r < p.m)) *reinterpret_cast<uint2 *>(q) = c;
        scale = (lane & 15) == r ? s : scale;
    }
    const int hl = lane & 15;
    if ((col & ~(BK - 1)) < p.k && hl < R && row0 + hl < p.m) p.scale[(size_t)(col / BK) * p.m + row0 + hl] = scale;
}

template <int R>
__global__ void __launch_bounds__(QUANT_THREADS) quantize_kernel(const QuantParams p) {
    pdl_wait();
    pdl_trigger();
    const int pairs = (p.k + 2 * BK - 1) / (2 * BK);
    const long long task = (long long)blockIdx.x * (QUANT_THREADS / 32) + (threadIdx.x >> 5);
    const int row0 = (int)(task / pairs) * R, col = (int)(task % pairs) * 2 * BK + (threadIdx.x & 31) * 8;
    if (row0 >= p.m) return;   // whole warps
    if (row0 + R <= p.m)
        quantize_rows<R, true>(p, row0, col);
    else
        quantize_rows<R, false>(p, row0, col);
}

// ---- output -------------------------------------------------------------------------------------
// Residuals are read past L1: out may be the same buffer, and a line's other columns another CTA's.
E3_DEV float res1(const __nv_bfloat16 *src) {
    return __uint_as_float((uint32_t)__ldcg(reinterpret_cast<const unsigned short *>(src)) << 16);
}
E3_DEV void add_quad(float *v, uint4 q) {   // 8 bf16
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] += __uint_as_float(w[i] << 16);
        v[2 * i + 1] += __uint_as_float(w[i] & 0xffff0000u);
    }
}
E3_DEV uint4 pack8(const float *v) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
// 4 consecutive outputs of a row from column col: residual, rounding, store (columns below n).
template <bool RES>
E3_DEV void store4(const Fp8Params &p, int row, int col, float4 v4) {
    float v[4] = {v4.x, v4.y, v4.z, v4.w};
    const bool whole = col + 4 <= p.n;
    if (!RES && p.epi == EAGLE3_EPI_F32) {
        float *o = (float *)p.out + (size_t)row * p.ld_out + col;
        if (whole && ((uintptr_t)o & 15) == 0) {
            *reinterpret_cast<float4 *>(o) = v4;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (col + i < p.n) o[i] = v[i];
        }
        return;
    }
    if (RES) {
        const __nv_bfloat16 *src = p.residual + (size_t)row * p.ld_res + col;
        if (whole && ((uintptr_t)src & 7) == 0) {
            const uint2 r = __ldcg(reinterpret_cast<const uint2 *>(src));
            v[0] += __uint_as_float(r.x << 16), v[1] += __uint_as_float(r.x & 0xffff0000u);
            v[2] += __uint_as_float(r.y << 16), v[3] += __uint_as_float(r.y & 0xffff0000u);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (col + i < p.n) v[i] += res1(src + i);
        }
    }
    __nv_bfloat16 *o = (__nv_bfloat16 *)p.out + (size_t)row * p.ld_out + col;
    if (whole && ((uintptr_t)o & 7) == 0) {
        const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
        *reinterpret_cast<uint2 *>(o) =
            make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (col + i < p.n) o[i] = __float2bfloat16_rn(v[i]);
    }
}

// A warp's staging box, 32 rows of 64 bytes in the 64-byte swizzle: 16-byte piece j, 4-byte word c and 2-byte half
// c of row r.
E3_DEV uint4 *box_quad(uint8_t *box, int r, int j) {
    return reinterpret_cast<uint4 *>(box + r * 64 + ((j ^ ((r >> 1) & 3)) << 4));
}
E3_DEV uint32_t *box_word(uint8_t *box, int r, int c) {
    return reinterpret_cast<uint32_t *>(box + r * 64 + (((c >> 2) ^ ((r >> 1) & 3)) << 4) + (c & 3) * 4);
}
E3_DEV unsigned short *box_half(uint8_t *box, int r, int c) {
    return reinterpret_cast<unsigned short *>(box + r * 64 + (((c >> 3) ^ ((r >> 1) & 3)) << 4) + (c & 7) * 2);
}
// Rows of any alignment leave a box by half warps, two rows a store.  These loops are short code without branches,
// 8 stores in flight: unrolled over a tile's rows and columns they were thousands of instructions, fetched anew
// for every tile.
E3_DEV void store_rows(uint8_t *box, float *o, int64_t ld, int rows, int most, int lane) {
    const int c = lane & 15, h = lane >> 4;
    o += h * ld + c;
#pragma unroll 1
    for (int r0 = h; r0 < rows + h; r0 += 16) {
        uint32_t w[8];
#pragma unroll
        for (int r = 0; r < 8; ++r) w[r] = *box_word(box, r0 + 2 * r, c);
#pragma unroll
        for (int r = 0; r < 8; ++r, o += 2 * ld)
            if (r0 + 2 * r < rows && c < most) *o = __uint_as_float(w[r]);
    }
}
// 32 bf16 columns, the first `most`.  Words leave on 4-byte boundaries: of a row that starts between two, lane c
// takes columns 2 c - 1 and 2 c (none, for c = 0).  The columns that are left, a row's first or last, follow, a
// row a lane.
E3_DEV void store_rows(uint8_t *box, __nv_bfloat16 *out, int64_t ld, int rows, int most, int lane) {
    unsigned short *base = reinterpret_cast<unsigned short *>(out);
    const int c = lane & 15, h = lane >> 4, odd0 = (int)((uintptr_t)out >> 1) & 1, turn = (int)ld & 1;
    const int odd = odd0 ^ (turn & h);   // rows h, h + 2, ... start between words
    const bool in = 2 * c + 1 - odd < most && (c > 0 || !odd);
    unsigned short *o = base + h * ld + 2 * c - odd;
#pragma unroll 1
    for (int r0 = h; r0 < rows + h; r0 += 16) {
        uint32_t w[8];
#pragma unroll
        for (int r = 0; r < 8; ++r) w[r] = *box_word(box, r0 + 2 * r, c);
#pragma unroll
        for (int r = 0; r < 8; ++r, o += 2 * ld) {
            const uint32_t before = __shfl_up_sync(0xffffffffu, w[r], 1);
            const uint32_t v = odd ? __byte_perm(before, w[r], 0x5432) : w[r];
            if (in && r0 + 2 * r < rows) *reinterpret_cast<uint32_t *>(o) = v;
        }
    }
    const int mine = odd0 ^ (turn & lane);
    unsigned short *row = base + (size_t)lane * ld;
    if (lane < rows && mine) row[0] = *box_half(box, lane, 0);
    if (lane < rows && ((most + mine) & 1)) row[most - 1] = *box_half(box, lane, most - 1);
}
// 32 columns, the first `most`, of `rows` rows from src to the box, 16 rows in flight
E3_DEV void load_rows(uint8_t *box, const __nv_bfloat16 *src, int64_t ld, int rows, int most, int lane) {
    const unsigned short *at = reinterpret_cast<const unsigned short *>(src) + lane;
#pragma unroll 1
    for (int r0 = 0; r0 < rows; r0 += 16) {
        unsigned short a[16];
#pragma unroll
        for (int r = 0; r < 16; ++r, at += ld) a[r] = r0 + r < rows && lane < most ? __ldcg(at) : (unsigned short)0;
#pragma unroll
        for (int r = 0; r < 16; ++r) *box_half(box, r0 + r, lane) = a[r];
    }
}

// ---- wide ---------------------------------------------------------------------------------------
// Three warpgroups: loads and MMAs (warps 0 and 1; 2 and 3 idle), and two of the epilogue.  The block is launched
// with 168 registers a thread (384 x 168 = 64512); the first group keeps 40 and the epilogue takes 232 (128 x 40 +
// 256 x 232 = 64512): 128 accumulators, two loads of 16, scales.  The instructions around the 128 additions of a
// k-block (waits that poll, addresses made anew) weigh as much as they do, so barriers go by precomputed
// shared-memory addresses, a poll is a handful of instructions, the thread index stays in a register, and the shared
// memory's base is an offset to its symbol, not an integer made a pointer, whose accesses would be generic (337 ->
// 309 us): 3840 x 2 * 14336 x 4096 412 -> 309 us in a burst of a dozen calls, 319 to 347 (2830 to 2600 TFLOP/s) by
// GPU and clock in longer runs; 3840 x 6144 x 4096 72 us.  (Four groups of 64 accumulators and 104 registers: 358
// us.) What bounds it: a tile moves 48 KB a k-block into shared memory and its MMAs read as much, 768 cycles at 128
// bytes a cycle for MMAs of 512 (707 k-blocks an SM: 262 us at 2070 MHz; without the additions the kernel takes
// 265); the rest are the waits for one TMEM load at a time and their additions.  Issue slots (50%) are not full.
constexpr int WIDE_BN = 256, WIDE_STAGES = 4, WIDE_EPI_WARPS = 8, WIDE_THREADS = 128 + 32 * WIDE_EPI_WARPS;
constexpr int WIDE_EPI0 = 4;   // first epilogue warp
constexpr int SPLIT_BN = 128, SPLIT_STAGES = 6;   // OUT_SPLIT's narrower tiles
constexpr int WIDE_A = BM * BK, WIDE_RING = WIDE_STAGES * (WIDE_A + WIDE_BN * BK);
static_assert(SPLIT_STAGES * (WIDE_A + SPLIT_BN * BK) <= WIDE_RING, "the ring of narrower tiles");
constexpr int WIDE_BOX = 32 * 64;   // output staging: 32 rows x 64 bytes a warp
// One barrier before and one after the MMAs of a k-block, both counted by its ring stage: full completes
// when the loads have landed and the epilogue warps have read the TMEM buffer (that of BUFS k-blocks
// before), done when the MMAs have run, which both frees the stage and fills the buffer.  (With barriers
// of their own for the buffers the issuing thread spent 640 cycles a k-block on waits and commits.)
struct WideShared {
    uint64_t full[SPLIT_STAGES], done[SPLIT_STAGES], mma_done, res[WIDE_EPI_WARPS];
    uint32_t tmem_base;
    int abort;
};
constexpr int WIDE_SMEM = 1024 + WIDE_RING + 2 * WIDE_EPI_WARPS * WIDE_BOX + (int)sizeof(WideShared);
static_assert(WIDE_SMEM <= 232448, "shared memory budget");
static_assert(WIDE_STAGES >= LEAST_STAGES && SPLIT_STAGES >= LEAST_STAGES, "stages");

// SPLIT: where rank src's sums of piece j (4 columns of each run, 128 rows) of an epilogue half lie in the ring of
// the rank that the piece belongs to, j / split_pieces: two quads of values, all rows of a quad side by side; byte
// offset of a row's first quad.
template <int BN>
__host__ __device__ constexpr int split_pieces(int ranks) {
    return (2 * BN / WIDE_EPI_WARPS / 4 + ranks - 1) / ranks;
}
template <int BN>
__host__ __device__ constexpr int split_bytes(int ranks) {
    return ranks * 2 * split_pieces<BN>(ranks) * 2 * BM * 16;
}
template <int BN>
E3_DEV uint32_t split_offset(int ranks, int src, int part, int j, int row) {
    const int each = split_pieces<BN>(ranks);
    return (uint32_t)((((src * 2 + part) * each + j % each) * 2 * BM + row) * 16);
}

template <int N>
E3_DEV void registers_give() {
    __syncwarp();
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(N));
}
template <int N>
E3_DEV void registers_take() {
    __syncwarp();
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(N));
}

// SPLIT: a cluster of p.ranks CTAs works on one tile (of 256 columns or 128), each on a range of the k-blocks.
// Pieces of 4 columns of both runs belong to the ranks in shares: each rank sends the others their pieces of its sums
// by remote stores (reading them took three times as long), and adds up and finishes its own.  The stores are bound
// by the bytes, some 20 a cycle (128 x 256 sums: 5 us; a lane's quads side by side, 64 bytes from the next lane's: 9 to
// 12), which narrower tiles halve.
// OUT: how outputs leave; RES: with residuals.  The variants are kernels of their own: what stands behind the main
// loop decides whether its 128 accumulators and scales stay in registers (stores by TMA and by the warps in one
// kernel: 3840 x 2 * 14336 x 4096 346 -> 444 us).
enum { OUT_TMA, OUT_STAGED, OUT_SPLIT };
template <bool SWIGLU, int OUT, bool RES, int BN = WIDE_BN>
__global__ void __launch_bounds__(WIDE_THREADS, 1)
    fp8_wide_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
                    const __grid_constant__ CUtensorMap tm_w2, const __grid_constant__ CUtensorMap tm_out,
                    const __grid_constant__ CUtensorMap tm_res, const Fp8Params p) {
    constexpr bool SPLIT = OUT == OUT_SPLIT, RES_TMA = OUT == OUT_TMA && RES;
    constexpr int RUN = 2 * BN / WIDE_EPI_WARPS;   // a thread's two runs of columns
    constexpr int STAGES = BN == WIDE_BN ? WIDE_STAGES : SPLIT_STAGES, STAGE = WIDE_A + BN * BK;
    constexpr int BUFS = 512 / BN;                 // TMEM buffers
    extern __shared__ uint8_t smem_raw[];
    uint8_t *ring = smem_raw + (-smem_u32(smem_raw) & 1023u);   // (the compiler knows it as shared memory)
    uint8_t *boxes = ring + WIDE_RING;
    WideShared &sh = *reinterpret_cast<WideShared *>(boxes + 2 * WIDE_EPI_WARPS * WIDE_BOX);
    const uint32_t tid = tc::thread_index();
    const int warp = (int)(tid >> 5), lane = (int)(tid & 31u);

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            tc::mbar_init(&sh.full[s],
                          1 + WIDE_EPI_WARPS + missing_arrivals(p.wait, s, SPLIT ? (int)blockIdx.x % p.ranks : 0));
            tc::mbar_init(&sh.done[s], 1);
        }
        tc::mbar_init(&sh.mma_done, 1);
        for (int w = 0; w < WIDE_EPI_WARPS; ++w) tc::mbar_init(&sh.res[w], 1);
        sh.abort = 0;
        tc::fence_barrier_init();
        tc::prefetch_tmap(&tm_x);
        tc::prefetch_tmap(&tm_w);
        if (SWIGLU) tc::prefetch_tmap(&tm_w2);
    }
    if (warp == 1) tc::tmem_alloc(&sh.tmem_base, BUFS * BN);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = sh.tmem_base;
    pdl_wait();
    pdl_trigger();
    const int units = p.tiles_m * p.tiles_n;
    const uint32_t ring0 = smem_u32(ring), full0 = smem_u32(sh.full), done0 = smem_u32(sh.done);
    const uint32_t abort0 = smem_u32(&sh.abort);
    const int ranks = SPLIT ? p.ranks : 1, rank = SPLIT ? (int)blockIdx.x % ranks : 0;
    const int unit0 = SPLIT ? (int)blockIdx.x / ranks : (int)blockIdx.x, unit_step = SPLIT ? units : (int)gridDim.x;
    const int kb0 = SPLIT ? (int)((long long)p.kb_total * rank / ranks) : 0;
    const int kb1 = SPLIT ? (int)((long long)p.kb_total * (rank + 1) / ranks) : p.kb_total;

    if (warp < WIDE_EPI0) {
        registers_give<40>();
        if (warp == 0) {
            // ------------------------------------------------------------------ TMA producer
            if (tc::elect_one()) {
                int stage = 0;
                uint32_t phase = 0, last_parity = 0, issued = 0;
                bool ok = true;
                for (int u = unit0; ok && u < units; u += unit_step) {
                    const int mb = u % p.tiles_m, nb = u / p.tiles_m;
                    for (int kb = kb0; kb < kb1; ++kb) {
                        if (!tc::mbar_wait(done0 + stage * 8, phase ^ 1u, abort0, p.wait.limit)) {
                            ok = false;
                            break;
                        }
                        const uint32_t full = full0 + stage * 8, sx = ring0 + stage * STAGE, sw = sx + WIDE_A;
                        tc::mbar_expect_tx(full, STAGE);
                        tc::tma_load_2d(sx, &tm_x, kb * BK, mb * BM, full);
                        if (SWIGLU) {
                            tc::tma_load_2d(sw, &tm_w, kb * BK, nb * (BN / 2), full);
                            tc::tma_load_2d(sw + BN * BK / 2, &tm_w2, kb * BK, nb * (BN / 2), full);
                        } else {
                            tc::tma_load_2d(sw, &tm_w, kb * BK, nb * BN, full);
                        }
                        issued |= 1u << stage;
                        last_parity = (last_parity & ~(1u << stage)) | (phase << stage);
                        if (++stage == STAGES) {
                            stage = 0;
                            phase ^= 1u;
                        }
                    }
                }
                if (!ok) flag(p.dev_status, EAGLE3_DEV_TIMEOUT);
                // no TMA write may still be in flight when the CTA exits (bounded waits)
                const uint32_t t0 = tc::kiloclock();
                for (int st = 0; st < STAGES; ++st)
                    if ((issued >> st) & 1u) tc::mbar_drain(full0 + st * 8, (last_parity >> st) & 1u, t0, p.wait.limit);
            }
            __syncwarp();
        } else if (warp == 1) {
            // ------------------------------------------------------------------ MMA issuer
            if (tc::elect_one()) {
                constexpr uint32_t IDESC = tc::idesc_e4m3(BM, BN);
                const uint64_t desc0 = tc::desc_sw128(ring0);
                int stage = 0, buf = 0;
                uint32_t phase = 0;
                bool ok = true;
                for (int u = unit0; ok && u < units; u += unit_step)
                    for (int kb = kb0; kb < kb1; ++kb) {
                        if (!tc::mbar_wait(full0 + stage * 8, phase, abort0, p.wait.limit)) {
                            ok = false;
                            break;
                        }
                        tc::fence_after();
                        // (descriptors count 16 bytes)
                        const uint64_t a = desc0 + (uint32_t)(stage * (STAGE >> 4)), b = a + (WIDE_A >> 4);
#pragma unroll
                        for (int k = 0; k < BK / 32; ++k)
                            tc::mma_e4m3_ss(tmem + buf * BN, a + k * 2, b + k * 2, IDESC, k > 0 ? 1u : 0u);
                        tc::mma_commit(done0 + stage * 8);
                        if (++stage == STAGES) {
                            stage = 0;
                            phase ^= 1u;
                        }
                        buf = (buf + 1) % BUFS;
                    }
                if (!ok) flag(p.dev_status, EAGLE3_DEV_TIMEOUT);
                // every MMA this thread issued must retire before TMEM is freed (bounded wait)
                tc::mma_commit(smem_u32(&sh.mma_done));
                tc::mbar_drain(smem_u32(&sh.mma_done), 0, tc::kiloclock(), p.wait.limit);
            }
            __syncwarp();
        }
        if (SPLIT) {   // (the epilogue's two)
            tc::cluster_sync();
            tc::cluster_sync();
        }
    } else {
        registers_take<232>();
        // ------------------------------------------------------------------ epilogue (warps 4..11)
        const int quarter = warp & 3, part = (warp - WIDE_EPI0) >> 2;
        uint8_t *box = boxes + (warp - WIDE_EPI0) * WIDE_BOX, *res_box = box + WIDE_EPI_WARPS * WIDE_BOX;
        const uint32_t res_bar = smem_u32(&sh.res[warp - WIDE_EPI0]);
        uint32_t res_phase = 0;
        // this thread's two runs of accumulator columns: neighbours, or gate and up of one run
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
        const uint32_t run_a = lanes + (SWIGLU ? RUN : 2 * RUN) * part;
        const uint32_t run_b = run_a + (SWIGLU ? BN / 2 : RUN);
        const int kb_total = kb1 - kb0;
        int stage = 0, buf = 0;
        uint32_t phase = 0;
        bool ok = true;
        if (lane == 0) {   // all buffers are free
#pragma unroll
            for (int i = 0; i < BUFS; ++i) tc::mbar_arrive(&sh.full[i]);
        }
        for (int u = unit0; ok && u < units; u += unit_step) {
            const int mb = u % p.tiles_m, nb = u / p.tiles_m;
            const int row = mb * BM + quarter * 32 + lane;
            const float *xs = p.x_scale + (size_t)kb0 * p.m + (row < p.m ? row : 0);
            const int block = min((SWIGLU ? nb * (BN / 2) + RUN * part : nb * BN + 2 * RUN * part) / BK, p.n_blocks - 1);
            const float *wa = p.w_scale + (size_t)block * p.kb_total + kb0;
            const float *wb = SWIGLU ? p.w2_scale + (size_t)block * p.kb_total + kb0 : wa;
            float acc[2 * RUN];
#pragma unroll
            for (int i = 0; i < 2 * RUN; ++i) acc[i] = 0.0f;
            // scales, far enough ahead of their use for a loaded L2: the row's two k-blocks ahead, the
            // weights' of 32 k-blocks, one a lane
            const float *at = xs;
            float sx = __ldg(at), sx1 = kb_total > 1 ? __ldg(at + p.m) : 0.0f, sa = 0.0f, sb = 0.0f;
            at += 2 * (size_t)p.m;
#pragma unroll 1
            for (int kb = 0; kb < kb_total; ++kb) {
                const float sx2 = kb + 2 < kb_total ? __ldg(at) : 0.0f;
                at += p.m;
                if ((kb & 31) == 0) {
                    const int i = min(kb + lane, kb_total - 1);
                    sa = __ldg(wa + i);
                    if (SWIGLU) sb = __ldg(wb + i);
                }
                const float fa = sx * __shfl_sync(0xffffffffu, sa, kb & 31);
                const float fb = SWIGLU ? sx * __shfl_sync(0xffffffffu, sb, kb & 31) : fa;
                if (!tc::mbar_wait_warp(done0 + stage * 8, phase, abort0, p.wait.limit)) {
                    ok = false;
                    break;
                }
                tc::fence_after();
                const uint32_t t = tmem + (uint32_t)(buf * BN);
                // 16 columns a load, the next one in flight while the last is added
                float v[2][16];
                tc::tmem_ld16_start(t + run_a, v[0]);
#pragma unroll
                for (int c = 0; c < RUN / 8; ++c) {
                    tc::tmem_ld_wait(v[c & 1]);
                    if (c + 1 < RUN / 8) {
                        tc::tmem_ld16_start(t + (c + 1 < RUN / 16 ? run_a + (c + 1) * 16
                                                                       : run_b + (c + 1 - RUN / 16) * 16),
                                            v[(c + 1) & 1]);
                    } else {   // the buffer is read: it may take the k-block after the next
                        // (the wait for the last load was the whole warp's)
                        tc::fence_before();
                        tc::mbar_arrive_if(full0 + ((stage + BUFS) % STAGES) * 8, lane == 0);
                    }
                    const float2 f = make_float2(c < RUN / 16 ? fa : fb, c < RUN / 16 ? fa : fb);
#pragma unroll
                    for (int i = 0; i < 16; i += 2) {
                        const float2 r = __ffma2_rn(make_float2(v[c & 1][i], v[c & 1][i + 1]), f,
                                                    make_float2(acc[c * 16 + i], acc[c * 16 + i + 1]));
                        acc[c * 16 + i] = r.x;
                        acc[c * 16 + i + 1] = r.y;
                    }
                }
                sx = sx1;
                sx1 = sx2;
                if (++stage == STAGES) {
                    stage = 0;
                    phase ^= 1u;
                }
                buf = (buf + 1) % BUFS;
            }
            if (!ok) {
                if (lane == 0) flag(p.dev_status, EAGLE3_DEV_TIMEOUT);
                break;
            }
            if (SPLIT) {
                // over the rings, when all ranks' loads and MMAs have completed
                tc::cluster_sync();
#pragma unroll
                for (int j = 0; j < RUN / 4; ++j) {
                    const uint32_t to = tc::cluster_addr(ring0, j / split_pieces<BN>(ranks)) +
                                        split_offset<BN>(ranks, rank, part, j, quarter * 32 + lane);
                    const float *v = acc + j * 4, *w = v + RUN;
                    tc::cluster_st4(to, v[0], v[1], v[2], v[3]);
                    tc::cluster_st4(to + BM * 16, w[0], w[1], w[2], w[3]);
                }
                break;   // one tile a cluster
            }
            const int cols = SWIGLU ? RUN : 2 * RUN, y = mb * BM + quarter * 32;
            const int col0 = nb * (SWIGLU ? BN / 2 : BN) + cols * part;
            const bool f32 = !SWIGLU && !RES && p.epi == EAGLE3_EPI_F32;
            const int rows = min(32, p.m - y);
            // Residuals by TMA too, 32 columns at a time to a box of their own, the next while these are added and
            // stored.  (Loads of a row a lane: 2000 x 6144 x 4096 66 us, 54 so; with the first box before the main
            // loop 52, but 3840 x 4096 x 14336 in place 246 us in place of 218.)
            if (RES_TMA && lane == 0 && col0 < p.n) {
                tc::mbar_expect_tx(res_bar, WIDE_BOX);
                tc::tma_load_2d(smem_u32(res_box), &tm_res, col0, y, res_bar);
            }
            // pieces of 64 bytes: 32 bf16 or 16 fp32 columns of the warp's 32 rows, in the 64-byte swizzle
#pragma unroll
            for (int c = 0; c < RUN / 8; ++c) {
                if (c * (f32 ? 16 : 32) >= cols) break;
                const int x = col0 + c * (f32 ? 16 : 32);
                if (OUT == OUT_TMA && lane == 0) tc::bulk_wait_read<0>();   // the box's last store has read it
                __syncwarp();
                if (SWIGLU) {
#pragma unroll
                    for (int i = 32 * c; i < 32 * c + 32; ++i) acc[i] = silu(acc[i]) * acc[RUN + i];
                }
                if (RES_TMA && ok && x < p.n) {
                    ok = tc::mbar_wait_warp(res_bar, res_phase, abort0, p.wait.limit);
                    res_phase ^= 1u;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        add_quad(acc + c % (RUN / 16) * 32 + 8 * j, *box_quad(res_box, lane, j));
                    __syncwarp();
                    if (ok && lane == 0 && c + 1 < 2 * RUN / 32 && x + 32 < p.n) {
                        tc::mbar_expect_tx(res_bar, WIDE_BOX);
                        tc::tma_load_2d(smem_u32(res_box), &tm_res, x + 32, y, res_bar);
                    }
                } else if (OUT == OUT_STAGED && RES && x < p.n) {
                    load_rows(box, p.residual + (size_t)y * p.ld_res + x, p.ld_res, rows, min(32, p.n - x), lane);
                    __syncwarp();
#pragma unroll
                    for (int j = 0; j < 4; ++j) add_quad(acc + c % (RUN / 16) * 32 + 8 * j, *box_quad(box, lane, j));
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint4 o;
                    if (f32) {
                        const float *v = acc + c * 16 + 4 * j;
                        o = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                                       __float_as_uint(v[3]));
                    } else {
                        o = pack8(acc + c % (RUN / 16) * 32 + 8 * j);
                    }
                    *box_quad(box, lane, j) = o;
                }
                if (OUT == OUT_TMA) {
                    tc::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0 && x < p.n && y < p.m) {
                        tc::tma_store_2d(&tm_out, x, y, box);
                        tc::bulk_commit();
                    }
                } else {
                    __syncwarp();
                    if (x >= p.n) continue;
                    const size_t at = (size_t)y * p.ld_out + x;
                    if (f32)
                        store_rows(box, (float *)p.out + at, p.ld_out, rows, p.n - x, lane);
                    else
                        store_rows(box, (__nv_bfloat16 *)p.out + at, p.ld_out, rows, min(32, p.n - x), lane);
                }
            }
            if (RES_TMA && !ok && lane == 0) {
                flag(p.dev_status, EAGLE3_DEV_TIMEOUT);
                tc::mbar_drain(res_bar, res_phase ^ 1u, tc::kiloclock(), p.wait.limit);
            }
        }
        if (lane == 0) tc::bulk_wait<0>();
        __syncwarp();
        if (SPLIT) {
            if (!ok) tc::cluster_sync();   // (after a timeout; its sums are void)
            tc::cluster_sync();
            const int mb = unit0 % p.tiles_m, nb = unit0 / p.tiles_m, row = mb * BM + quarter * 32 + lane;
            const int col0 = nb * (SWIGLU ? BN / 2 : BN) + (SWIGLU ? RUN : 2 * RUN) * part;
            const int each = split_pieces<BN>(ranks);
            for (int piece = rank * each; piece < min((rank + 1) * each, RUN / 4); ++piece) {
                const int j = piece * 4;
                float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f), b = a;
                for (int s = 0; s < ranks; ++s) {   // in rank order
                    const float4 *from = reinterpret_cast<const float4 *>(
                        ring + split_offset<BN>(ranks, s, part, piece, quarter * 32 + lane));
                    const float4 v = from[0], w = from[BM];
                    a.x += v.x, a.y += v.y, a.z += v.z, a.w += v.w;
                    b.x += w.x, b.y += w.y, b.z += w.z, b.w += w.w;
                }
                if (row >= p.m) continue;
                if (SWIGLU) {
                    a = make_float4(silu(a.x) * b.x, silu(a.y) * b.y, silu(a.z) * b.z, silu(a.w) * b.w);
                    store4<RES>(p, row, col0 + j, a);
                } else {
                    store4<RES>(p, row, col0 + j, a);
                    store4<RES>(p, row, col0 + RUN + j, b);
                }
            }
            __syncwarp();
        }
    }

    tc::fence_before();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc::fence_after();
        tc::tmem_dealloc(tmem, BUFS * BN);
    }
}

// ---- narrow -------------------------------------------------------------------------------------
constexpr int NARROW_EPI_WARPS = 8, NARROW_THREADS = 64 + 32 * NARROW_EPI_WARPS, NARROW_MAX = 64;
constexpr int NARROW_STAGES = 8, NARROW_TMEM = 256;
constexpr int NARROW_RING = 106 * 1024;   // two CTAs a SM
constexpr int NARROW_W = BM * BK;
struct NarrowShared {
    uint64_t full[NARROW_STAGES], empty[NARROW_STAGES], tfull[8], tempty[8], mma_done;
    uint32_t tmem_base;
    int abort;
    float scales[NARROW_EPI_WARPS][2][NARROW_MAX / 2];   // per epilogue warp: its rows' scales, double-buffered
};
constexpr int NARROW_SMEM = 1024 + NARROW_RING + (int)sizeof(NarrowShared);
static_assert(2 * (NARROW_SMEM + 1024) <= 228 * 1024, "two CTAs a SM");
static_assert(NARROW_RING >= NARROW_MAX * BM * 4, "the ranks' sums fit the ring");
static_assert(NARROW_RING / (NARROW_W + NARROW_MAX * BK) >= LEAST_STAGES, "stages of the largest tiles");

// NT: row capacity of a tile (TMEM buffers of NT columns, NT / 2 accumulators a thread).
// Grid: (cluster ranks = k ranges, weight tiles).
template <int NT, bool SWIGLU>
__global__ void __launch_bounds__(NARROW_THREADS, 2)
    fp8_narrow_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
                      const __grid_constant__ CUtensorMap tm_w2, const Fp8Params p) {
    constexpr int BUFS = NARROW_TMEM / NT;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *ring = smem_raw + (-smem_u32(smem_raw) & 1023u);
    NarrowShared &sh = *reinterpret_cast<NarrowShared *>(ring + NARROW_RING);
    volatile int *abort = &sh.abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int ranks = gridDim.x, rank = blockIdx.x, mt = blockIdx.y, rows = p.m;
    const int kb0 = (int)((long long)p.kb_total * rank / ranks);
    const int kb1 = (int)((long long)p.kb_total * (rank + 1) / ranks);
    const int stage_bytes = NARROW_W + p.n16 * BK, stages = p.stages;
    const long long wait_limit = (long long)p.wait.limit << 10;

    if (threadIdx.x == 0) {
        for (int s = 0; s < NARROW_STAGES; ++s) {
            tc::mbar_init(&sh.full[s], 1 + missing_arrivals(p.wait, s, rank));
            tc::mbar_init(&sh.empty[s], 1);
        }
        for (int b = 0; b < BUFS; ++b) {
            tc::mbar_init(&sh.tfull[b], 1);
            tc::mbar_init(&sh.tempty[b], NARROW_EPI_WARPS);
        }
        tc::mbar_init(&sh.mma_done, 1);
        sh.abort = 0;
        tc::fence_barrier_init();
        tc::prefetch_tmap(&tm_x);
        tc::prefetch_tmap(&tm_w);
        if (SWIGLU) tc::prefetch_tmap(&tm_w2);
    }
    if (warp == 1) tc::tmem_alloc(&sh.tmem_base, NARROW_TMEM);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = sh.tmem_base;
    // The weights' first k-blocks into L2 while the previous kernel ends (L2 is coherent: should that kernel
    // write them, the loads below still see what it wrote)
    if (warp == 0 && lane < 8 && kb0 + lane < kb1) {
        tc::tma_prefetch_2d(&tm_w, (kb0 + lane) * BK, SWIGLU ? mt * 64 : mt * BM);
        if (SWIGLU) tc::tma_prefetch_2d(&tm_w2, (kb0 + lane) * BK, mt * 64);
    }
    pdl_wait();
    pdl_trigger();

    if (warp == 0) {
        // ------------------------------------------------------------------ TMA producer
        int stage = 0;
        uint32_t phase = 0, last_parity = 0, issued = 0;   // lane 0
        bool ok = true;
        for (int kb = kb0; kb < kb1; ++kb) {
            int fine = 1;
            if (lane == 0) {
                fine = tc::mbar_wait(&sh.empty[stage], phase ^ 1u, abort, wait_limit) ? 1 : 0;
                if (fine) {
                    tc::mbar_expect_tx(&sh.full[stage], stage_bytes);
                    issued |= 1u << stage;
                    last_parity = (last_parity & ~(1u << stage)) | (phase << stage);
                }
            }
            fine = __shfl_sync(0xffffffffu, fine, 0);
            if (!fine) {
                ok = false;
                break;
            }
            uint8_t *sw = ring + stage * stage_bytes, *sx = sw + NARROW_W;
            if (SWIGLU) {
                if (lane < 8) {   // 16 gate and 16 up rows for the lanes of each quarter
                    const int q = lane >> 1, up = lane & 1;
                    tc::tma_load_2d(sw + lane * 16 * BK, up ? &tm_w2 : &tm_w, kb * BK, mt * 64 + q * 16,
                                    &sh.full[stage]);
                }
            } else if (lane == 0) {
                tc::tma_load_2d(sw, &tm_w, kb * BK, mt * BM, &sh.full[stage]);
            }
            if (16 * lane < p.n16)
                tc::tma_load_2d(sx + lane * 16 * BK, &tm_x, kb * BK, lane * 16, &sh.full[stage]);
            if (++stage == stages) {
                stage = 0;
                phase ^= 1u;
            }
        }
        if (lane == 0) {
            if (!ok) flag(p.dev_status, EAGLE3_DEV_TIMEOUT);
            const long long t0 = clock64();
            for (int st = 0; st < stages; ++st) {   // loads in flight (bounded waits)
                if (!((issued >> st) & 1u)) continue;
                const uint32_t par = (last_parity >> st) & 1u;
                while (!tc::mbar_try(&sh.full[st], par) && clock64() - t0 < wait_limit) {
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------------ MMA issuer
        if (tc::elect_one()) {
            const uint64_t desc0 = tc::desc_sw128(smem_u32(ring));
            const uint32_t idesc = tc::idesc_e4m3(BM, p.n16);
            int stage = 0, buf = 0;
            uint32_t phase = 0, buf_phase = 0;
            bool ok = true;
            for (int kb = kb0; kb < kb1; ++kb) {
                if (!tc::mbar_wait(&sh.tempty[buf], buf_phase ^ 1u, abort, wait_limit) ||
                    !tc::mbar_wait(&sh.full[stage], phase, abort, wait_limit)) {
                    ok = false;
                    break;
                }
                tc::fence_after();
                const uint64_t a = desc0 + (uint32_t)(stage * stage_bytes >> 4), b = a + (NARROW_W >> 4);
#pragma unroll
                for (int k = 0; k < BK / 32; ++k)
                    tc::mma_e4m3_ss(tmem + buf * NT, a + k * 2, b + k * 2, idesc, k > 0 ? 1u : 0u);
                tc::mma_commit(&sh.empty[stage]);
                tc::mma_commit(&sh.tfull[buf]);
                if (++stage == stages) {
                    stage = 0;
                    phase ^= 1u;
                }
                if (++buf == BUFS) {
                    buf = 0;
                    buf_phase ^= 1u;
                }
            }
            if (!ok) flag(p.dev_status, EAGLE3_DEV_TIMEOUT);
            tc::mma_commit(&sh.mma_done);
            const long long t0 = clock64();
            while (!tc::mbar_try(&sh.mma_done, 0) && clock64() - t0 < wait_limit) {
            }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------------ epilogue (warps 2..9)
        constexpr int HALF = NT / 2;   // rows of a warp: two warps share a quarter of the TMEM lanes
        const int quarter = warp & 3, r0 = (warp - 2) / 4 * HALF;
        const uint32_t t_col = tmem + ((uint32_t)(quarter * 32) << 16) + r0;
        const int block = SWIGLU ? mt / 2 : mt;
        const float *ws = (SWIGLU && lane >= 16 ? p.w2_scale : p.w_scale) + (size_t)block * p.kb_total;
        const uint32_t tfull0 = smem_u32(sh.tfull), tempty0 = smem_u32(sh.tempty), abort0 = smem_u32(&sh.abort);
        float acc[HALF];
#pragma unroll
        for (int i = 0; i < HALF; ++i) acc[i] = 0.0f;
        constexpr int PER = (HALF + 31) / 32;
        float sx[PER], sw = 0.0f;
        auto fetch = [&](int kb) {   // the k-block's scales: this lane's rows, and its weight row's
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int r = lane + 32 * i;
                sx[i] = r < HALF && r0 + r < rows ? __ldg(p.x_scale + (size_t)kb * p.m + r0 + r) : 0.0f;
            }
            sw = __ldg(ws + kb);
        };
        fetch(kb0);
        int buf = 0;
        uint32_t buf_phase = 0;
        for (int kb = kb0; kb < kb1; ++kb) {
            float *strip = sh.scales[warp - 2][kb & 1];
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (lane + 32 * i < HALF) strip[lane + 32 * i] = sx[i];
            const float fw = sw;
            if (kb + 1 < kb1) fetch(kb + 1);
            // (the vote also orders the strip's writes)
            if (!tc::mbar_wait_warp(tfull0 + buf * 8, buf_phase, abort0, p.wait.limit)) {
                if (lane == 0) flag(p.dev_status, EAGLE3_DEV_TIMEOUT);
                break;
            }
            __syncwarp();
            tc::fence_after();
#pragma unroll
            for (int c = 0; c < HALF; c += 16) {
                if (r0 + c < p.n16) {
                    float v[16];
                    tc::tmem_ld16_start(t_col + buf * NT + c, v);
                    tc::tmem_ld_wait(v);
#pragma unroll
                    for (int i = 0; i < 16; i += 4) {
                        const float4 f = *reinterpret_cast<const float4 *>(strip + c + i);
                        acc[c + i] = fmaf(v[i] * f.x, fw, acc[c + i]);
                        acc[c + i + 1] = fmaf(v[i + 1] * f.y, fw, acc[c + i + 1]);
                        acc[c + i + 2] = fmaf(v[i + 2] * f.z, fw, acc[c + i + 2]);
                        acc[c + i + 3] = fmaf(v[i + 3] * f.w, fw, acc[c + i + 3]);
                    }
                }
            }
            tc::fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(tempty0 + buf * 8);
            if (++buf == BUFS) {
                buf = 0;
                buf_phase ^= 1u;
            }
        }
        // this rank's sums, [row][weight row], over the ring: its last loads and MMAs have completed
        // (after a timeout another warp's may not have; the outputs are void then)
        float *sums = reinterpret_cast<float *>(ring) + r0 * BM + quarter * 32 + lane;
#pragma unroll
        for (int i = 0; i < HALF; ++i)
            if (r0 + i < rows) sums[i * BM] = acc[i];
    }

    tc::fence_before();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc::fence_after();
        tc::tmem_dealloc(tmem, NARROW_TMEM);
    }
    if (ranks > 1) {
        tc::cluster_sync();
    }
    // rows rank, rank + ranks, ...: the ranks' sums in rank order, the epilogue, the output
    const uint32_t base = smem_u32(ring);
    constexpr int OUT = SWIGLU ? 64 : BM;   // output columns of the tile
    const int mine = rows > rank ? (rows - rank + ranks - 1) / ranks : 0;
    for (int i = threadIdx.x; i < mine * OUT; i += NARROW_THREADS) {
        const int r = rank + (i / OUT) * ranks, j = i % OUT;
        const int at = SWIGLU ? (j >> 4) * 32 + (j & 15) : j;   // the column's (gate) lane
        const uint32_t addr = base + (uint32_t)(r * BM + at) * 4u;
        float y = 0.0f, y2 = 0.0f;
        for (int s = 0; s < ranks; ++s) {
            const uint32_t from = ranks > 1 ? tc::cluster_addr(addr, s) : addr;
            y += tc::cluster_ld(from);
            if (SWIGLU) y2 += tc::cluster_ld(from + 64u);
        }
        const int col = mt * OUT + j;
        if (col >= p.n) continue;
        if (SWIGLU) y = silu(y) * y2;
        const size_t row = r;
        if (p.epi == EAGLE3_EPI_F32) {
            ((float *)p.out)[row * p.ld_out + col] = y;
        } else {
            if (p.epi == EAGLE3_EPI_BF16_RESIDUAL) y += res1(p.residual + row * p.ld_res + col);
            ((__nv_bfloat16 *)p.out)[row * p.ld_out + col] = __float2bfloat16_rn(y);
        }
    }
    if (ranks > 1) {
        tc::cluster_sync();   // no rank leaves while another reads its sums
    }
}

// ---- host side ----------------------------------------------------------------------------------
eagle3_status_t validate(const eagle3_quantize_fp8_args_t *a) {
    if (!a) return EAGLE3_ERR_INVALID_ARGUMENT;
    if (a->rows < 0 || a->k < 1) return EAGLE3_ERR_INVALID_ARGUMENT;
    if (a->k % 16 || a->k > MAX_DIM || a->rows > MAX_DIM) return EAGLE3_ERR_UNSUPPORTED;
    const int64_t ld_x = a->ld_x ? a->ld_x : a->k, ld_q = a->ld_q ? a->ld_q : a->k;
    if (ld_x < a->k || ld_q < a->k || ld_x % 8 || ld_q % 16) return EAGLE3_ERR_INVALID_ARGUMENT;
    if (a->rows == 0) return EAGLE3_OK;
    if (!a->x || !a->q || !a->scale) return EAGLE3_ERR_INVALID_ARGUMENT;
    if (((uintptr_t)a->x | (uintptr_t)a->q) & 15 || (uintptr_t)a->scale & 3) return EAGLE3_ERR_INVALID_ARGUMENT;
    return EAGLE3_OK;
}

eagle3_status_t validate(const eagle3_linear_fp8_args_t *a) {
    if (!a) return EAGLE3_ERR_INVALID_ARGUMENT;
    if (a->m < 0 || a->n < 1 || a->k < 1) return EAGLE3_ERR_INVALID_ARGUMENT;
    if (a->epilogue < EAGLE3_EPI_BF16 || a->epilogue > EAGLE3_EPI_BF16_ROPE) return EAGLE3_ERR_INVALID_ARGUMENT;
    if (a->epilogue == EAGLE3_EPI_BF16_ROPE || a->k % 16) return EAGLE3_ERR_UNSUPPORTED;
    if (a->m > MAX_DIM || a->n > MAX_DIM || a->k > MAX_DIM) return EAGLE3_ERR_UNSUPPORTED;
    const int64_t ld_x = a->ld_x ? a->ld_x : a->k, ld_w = a->ld_w ? a->ld_w : a->k;
    if (ld_x < a->k || ld_w < a->k || ld_x % 16 || ld_w % 16) return EAGLE3_ERR_INVALID_ARGUMENT;
    for (const int64_t ld : {a->ld_out, a->ld_res})
        if (ld && ld < a->n) return EAGLE3_ERR_INVALID_ARGUMENT;
    if (a->m == 0) return EAGLE3_OK;
    if (!a->x || !a->x_scale || !a->w || !a->w_scale || !a->out) return EAGLE3_ERR_INVALID_ARGUMENT;
    if (a->epilogue == EAGLE3_EPI_SWIGLU && (!a->w2 || !a->w2_scale)) return EAGLE3_ERR_INVALID_ARGUMENT;
    if (a->epilogue == EAGLE3_EPI_BF16_RESIDUAL && !a->residual) return EAGLE3_ERR_INVALID_ARGUMENT;
    if (((uintptr_t)a->x | (uintptr_t)a->w | (uintptr_t)a->w2) & 15) return EAGLE3_ERR_INVALID_ARGUMENT;
    if (((uintptr_t)a->x_scale | (uintptr_t)a->w_scale | (uintptr_t)a->w2_scale | (uintptr_t)a->dev_status) & 3)
        return EAGLE3_ERR_INVALID_ARGUMENT;
    if (((uintptr_t)a->out & (a->epilogue == EAGLE3_EPI_F32 ? 3 : 1)) || ((uintptr_t)a->residual & 1))
        return EAGLE3_ERR_INVALID_ARGUMENT;
    return EAGLE3_OK;
}

// 32-row boxes of 64 bytes of an [m, n] matrix (the output, the residual), by TMA; false where its address or pitch
// rules that out
bool box_map(CUtensorMap *m, const eagle3_linear_fp8_args_t *a, const void *base, int64_t ld, bool f32) {
    const int es = f32 ? 4 : 2;
    if (((uintptr_t)base & 15) || (ld * es) % 16) return false;
    const CUtensorMapDataType type = f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    return tmap_rows(m, type, es, base, a->m, a->n, ld, 32, 0, 0, 64);
}

template <int NT, bool SWIGLU>
cudaError_t launch_narrow(int tiles, cudaStream_t st, const CUtensorMap &tx, const CUtensorMap &tw,
                          const CUtensorMap &tw2, const Fp8Params &p) {
    static PerDevice<ClusterCounts> cache;
    const ClusterCounts most = cache.get([] {
        ClusterCounts c = {};
        for (int r = 1; r <= MAX_CLUSTER; ++r)
            c.n[r] = resident_clusters(fp8_narrow_kernel<NT, SWIGLU>, r, NARROW_THREADS, NARROW_SMEM);
        return c;
    });
    if (!succeeded(most) || most.n[1] < 1) return cudaErrorUnknown;
    // As many ranks as leave every tile a resident cluster, two k-blocks each at least.  The query counts one CTA a
    // SM; shared memory, registers and TMEM hold two, and two keep more loads in flight (8 rows, 99 tiles of 2 *
    // 6306 x 11040: 45 us by single CTAs, 28 by clusters of two, 41 by three, of which 92 are resident; 48 tiles of
    // 6144 x 4096: 8.2 us by three ranks, 7.1 by four, 11.8 by six, of which 46 are).
    int ranks = 1;
    for (int r = 2; r <= MAX_CLUSTER; ++r)
        if (tiles <= 2 * most.n[r] && p.kb_total >= 2 * r) ranks = r;
    const dim3 grid(ranks, tiles);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(NARROW_THREADS);
    cfg.dynamicSmemBytes = NARROW_SMEM;
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = grid.x;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, fp8_narrow_kernel<NT, SWIGLU>, tx, tw, tw2, p);
}

template <bool SWIGLU, int OUT, bool RES, int BN = WIDE_BN>
int wide_clusters(int ranks) {
    const auto kernel = fp8_wide_kernel<SWIGLU, OUT, RES, BN>;
    return OUT == OUT_SPLIT ? resident_clusters(kernel, ranks, WIDE_THREADS, WIDE_SMEM) : resident_ctas(kernel, WIDE_SMEM);
}

// The weights' tensor maps with boxes of `rows` rows
bool weight_maps(CUtensorMap *tw, CUtensorMap *tw2, const eagle3_linear_fp8_args_t *a, int rows) {
    const CUtensorMapDataType u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
    const int64_t ld_w = a->ld_w ? a->ld_w : a->k;
    if (!tmap_rows(tw, u8, 1, a->w, a->n, a->k, ld_w, rows)) return false;
    *tw2 = *tw;   // where unused
    return a->epilogue != EAGLE3_EPI_SWIGLU || tmap_rows(tw2, u8, 1, a->w2, a->n, a->k, ld_w, rows);
}

template <bool SWIGLU, bool RES>
cudaError_t launch_wide(const eagle3_linear_fp8_args_t *a, cudaStream_t st, const CUtensorMap &tx, const CUtensorMap &to,
                        const CUtensorMap &tr, Fp8Params &p) {
    static PerDevice<ClusterCounts> cache;
    const ClusterCounts most = cache.get([] {
        ClusterCounts c = {};
        c.n[1] = std::min(wide_clusters<SWIGLU, OUT_TMA, RES>(1), wide_clusters<SWIGLU, OUT_STAGED, RES>(1));
        for (int r = 2; r <= MAX_CLUSTER; ++r)
            if (split_bytes<WIDE_BN>(r) <= WIDE_RING && split_bytes<SPLIT_BN>(r) <= WIDE_RING)
                c.n[r] = std::min(wide_clusters<SWIGLU, OUT_SPLIT, RES>(r),
                                  wide_clusters<SWIGLU, OUT_SPLIT, RES, SPLIT_BN>(r));
        return c;
    });
    if (!succeeded(most) || most.n[1] < 1) return cudaErrorUnknown;
    // Few tiles: their k-blocks over as many ranks as leave every tile a resident cluster, with tiles of 256 or 128
    // columns, by the k-blocks in a row: a CTA's own (0.35 us each, whatever the width: they wait for L2), and 17 or 7
    // for sending, meeting and adding up 128 x 256 or 128 x 128 sums.  (256 x 4096 x 14336: 44 us by single CTAs, 25 by
    // four ranks of 256 columns, 29 by two of 128; 128 x 4096 x 4096: 15, 13.6 by six, 9.2 by four of 128; 128 x 1024 x
    // 2048: 9.0 and 7.3 by eight of 128; x 1024: 6.3 either way.)
    const int cols = SWIGLU ? SPLIT_BN / 2 : SPLIT_BN, narrower_n = (p.n + cols - 1) / cols;
    const int64_t tiles = (int64_t)p.tiles_m * p.tiles_n, narrower = (int64_t)p.tiles_m * narrower_n;
    int64_t least = (tiles + most.n[1] - 1) / most.n[1] * p.kb_total;
    bool narrow = false;
    p.ranks = 1;
    for (int r = 2; r <= std::min(MAX_CLUSTER, p.kb_total); ++r) {
        const int own = (p.kb_total + r - 1) / r;
        if (tiles <= most.n[r] && own + 17 < least) least = own + 17, p.ranks = r, narrow = false;
        if (narrower <= most.n[r] && own + 7 < least) least = own + 7, p.ranks = r, narrow = true;
    }
    CUtensorMap tw, tw2;
    if (!weight_maps(&tw, &tw2, a, (narrow ? SPLIT_BN : WIDE_BN) / (SWIGLU ? 2 : 1))) return cudaErrorInvalidValue;
    if (narrow) p.tiles_n = narrower_n;
    cudaLaunchConfig_t cfg = {};
    const int64_t split = (narrow ? narrower : tiles) * p.ranks;
    cfg.gridDim = dim3((unsigned)(p.ranks > 1 ? split : std::min<int64_t>(most.n[1], tiles)));
    cfg.blockDim = dim3(WIDE_THREADS);
    cfg.dynamicSmemBytes = WIDE_SMEM;
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = p.ranks;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = p.ranks > 1 ? 2 : 1;
    if (narrow)
        return cudaLaunchKernelEx(&cfg, fp8_wide_kernel<SWIGLU, OUT_SPLIT, RES, SPLIT_BN>, tx, tw, tw2, to, tr, p);
    return p.ranks > 1 ? cudaLaunchKernelEx(&cfg, fp8_wide_kernel<SWIGLU, OUT_SPLIT, RES>, tx, tw, tw2, to, tr, p)
           : p.tma_out ? cudaLaunchKernelEx(&cfg, fp8_wide_kernel<SWIGLU, OUT_TMA, RES>, tx, tw, tw2, to, tr, p)
                       : cudaLaunchKernelEx(&cfg, fp8_wide_kernel<SWIGLU, OUT_STAGED, RES>, tx, tw, tw2, to, tr, p);
}

}  // namespace
}  // namespace e3

using namespace e3;

extern "C" eagle3_status_t eagle3_quantize_fp8(const eagle3_quantize_fp8_args_t *a, eagle3_stream_t stream) {
    const eagle3_status_t st = validate(a);
    if (st != EAGLE3_OK || a->rows == 0) return st;
    QuantParams p;
    p.m = a->rows;
    p.k = a->k;
    p.ld_x = a->ld_x ? a->ld_x : a->k;
    p.ld_q = a->ld_q ? a->ld_q : a->k;
    p.x = (const __nv_bfloat16 *)a->x;
    p.q = a->q;
    p.scale = a->scale;
    const int64_t pairs = (a->k + 2 * BK - 1) / (2 * BK);
    const int sms = device_sm_count(), per_block = QUANT_THREADS / 32;
    auto blocks = [&](int r) { return (pairs * ((a->rows + r - 1) / r) + per_block - 1) / per_block; };
    const cudaStream_t s = (cudaStream_t)stream;
    const int r = blocks(8) >= 4 * (int64_t)sms ? 8 : blocks(2) >= 2 * (int64_t)sms ? 2 : 1;
    const int64_t grid = blocks(r);
    if (grid > INT32_MAX) return EAGLE3_ERR_UNSUPPORTED;
    const cudaError_t e =
        r == 8   ? launch_pdl(quantize_kernel<8>, dim3((unsigned)grid), dim3(QUANT_THREADS), 0, s, p)
        : r == 2 ? launch_pdl(quantize_kernel<2>, dim3((unsigned)grid), dim3(QUANT_THREADS), 0, s, p)
                 : launch_pdl(quantize_kernel<1>, dim3((unsigned)grid), dim3(QUANT_THREADS), 0, s, p);
    return e == cudaSuccess ? EAGLE3_OK : EAGLE3_ERR_CUDA;
}

static eagle3_status_t linear_fp8(const eagle3_linear_fp8_args_t *a, const WaitRule &wait, eagle3_stream_t stream) {
    const eagle3_status_t st = validate(a);
    if (st != EAGLE3_OK || a->m == 0) return st;
    const bool swiglu = a->epilogue == EAGLE3_EPI_SWIGLU;
    const int64_t ld_x = a->ld_x ? a->ld_x : a->k;
    Fp8Params p;
    p.m = a->m;
    p.n = a->n;
    p.k = a->k;
    p.epi = a->epilogue;
    p.kb_total = (a->k + BK - 1) / BK;
    p.n_blocks = (a->n + BK - 1) / BK;
    p.ld_out = a->ld_out ? a->ld_out : a->n;
    p.ld_res = a->ld_res ? a->ld_res : a->n;
    p.x_scale = a->x_scale;
    p.w_scale = a->w_scale;
    p.w2_scale = a->w2_scale;
    p.residual = (const __nv_bfloat16 *)a->residual;
    p.out = a->out;
    p.dev_status = a->dev_status;
    p.wait = wait;
    const int sms = std::max(1, device_sm_count());
    const cudaStream_t s = (cudaStream_t)stream;
    const CUtensorMapDataType u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
    const int tiles_w = (a->n + (swiglu ? 63 : BM - 1)) / (swiglu ? 64 : BM);
    p.tiles_m = (a->m + BM - 1) / BM;
    p.tiles_n = (a->n + (swiglu ? WIDE_BN / 2 : WIDE_BN) - 1) / (swiglu ? WIDE_BN / 2 : WIDE_BN);
    // Few rows by the narrow kernel, from 25 rows on unless the wide one's tiles cover half of the SMs.
    // 8 x 6144 x 4096 (24 wide tiles): 7.0 us narrow, 14.5 wide; 64 rows 10.9 and 13.2.  24 x 24576 x 4096 (96): 22 and
    // 27; 32 rows 24.6 and 21.0, 64 rows 27 and 21.  96 x 4096 x 14336: 34 (with tiles of 128 rows) and 20.
    const bool narrow = tiles_w <= 65535 && (a->m <= 24 || (a->m <= NARROW_MAX && 2 * p.tiles_n < sms));
    CUtensorMap tx, tw, tw2, to, tr;
    if (!tmap_rows(&tx, u8, 1, a->x, a->m, a->k, ld_x, narrow ? 16 : BM)) return EAGLE3_ERR_CUDA;
    p.tma_out = p.n16 = p.stages = 0;
    p.ranks = 1;
    cudaError_t e;
    if (narrow) {
        if (!weight_maps(&tw, &tw2, a, swiglu ? 16 : BM)) return EAGLE3_ERR_CUDA;
        p.n16 = (a->m + 15) / 16 * 16;
        p.stages = std::min(NARROW_STAGES, NARROW_RING / (NARROW_W + p.n16 * BK));
        if (p.n16 <= 32)
            e = swiglu ? launch_narrow<32, true>(tiles_w, s, tx, tw, tw2, p)
                       : launch_narrow<32, false>(tiles_w, s, tx, tw, tw2, p);
        else
            e = swiglu ? launch_narrow<64, true>(tiles_w, s, tx, tw, tw2, p)
                       : launch_narrow<64, false>(tiles_w, s, tx, tw, tw2, p);
    } else {
        const int64_t tiles = (int64_t)p.tiles_m * p.tiles_n;
        if (tiles > MAX_DIM) return EAGLE3_ERR_UNSUPPORTED;   // tiles are counted in 32 bits
        const bool res = a->epilogue == EAGLE3_EPI_BF16_RESIDUAL;
        p.tma_out = box_map(&to, a, a->out, p.ld_out, a->epilogue == EAGLE3_EPI_F32) &&
                    (!res || box_map(&tr, a, a->residual, p.ld_res, false));
        if (!p.tma_out) to = tx;   // unused
        if (!p.tma_out || !res) tr = tx;
        e = swiglu                                      ? launch_wide<true, false>(a, s, tx, to, tr, p)
            : a->epilogue == EAGLE3_EPI_BF16_RESIDUAL ? launch_wide<false, true>(a, s, tx, to, tr, p)
                                                      : launch_wide<false, false>(a, s, tx, to, tr, p);
    }
    return e == cudaSuccess ? EAGLE3_OK : EAGLE3_ERR_CUDA;
}

extern "C" eagle3_status_t eagle3_linear_fp8(const eagle3_linear_fp8_args_t *a, eagle3_stream_t stream) {
    return linear_fp8(a, WaitRule(), stream);
}

extern "C" eagle3_status_t eagle3_test_linear_fp8_timeout(const eagle3_linear_fp8_args_t *a, int32_t stall_block,
                                                          int32_t stall_rank, int64_t wait_limit_cycles,
                                                          eagle3_stream_t stream) {
    WaitRule wait;
    if (!stall_rule(&wait, stall_block, stall_rank, wait_limit_cycles)) return EAGLE3_ERR_INVALID_ARGUMENT;
    return linear_fp8(a, wait, stream);
}
