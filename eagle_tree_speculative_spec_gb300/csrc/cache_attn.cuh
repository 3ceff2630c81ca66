// What the kernels of eagle3_verify_attn_fp8 share.
#pragma once

#include <cfloat>

#include "e4m3.cuh"
#include "eagle3_kv.h"

namespace e3 {

struct CacheAttn {
    int B, N, Hq, Hkv, rep, max_prefix, splits, split_chunks, row_groups, clustered;
    int requested;                  // parts of the prefix that the caller asks for, at most MAX_SPLITS; 0: the kernels' choice
    int max_blocks, block_size, n_pages;
    float scale_log2;               // sm_scale * log2(e)
    int64_t q_ns, kv_ns;
    const __nv_bfloat16 *q, *tree_k, *tree_v;
    const int32_t *parents;
    const uint8_t *kc, *vc, *ks, *vs;
    const int32_t *block_table, *prefix_len;
    __nv_bfloat16 *out;
    float *lse;
    int32_t *dev_status;
    // results of the splits: [split][B][N][Hq], o (unnormalised, times V's scale) where l is not 0
    float *part_o, *part_ml;
};

constexpr int MAX_SPLITS = 512;
constexpr float RESCALE_LOG2 = 8.0f;   // the running maximum moves once a score is this far above it
constexpr float WEIGHT_LOG2 = 7.0f;    // weights are held times 2^7: at most 2^15 in fp16

// 2^x on the special-function unit (flushes subnormal results to zero)
E3_DEV float fast_exp2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 2^n, 0 below 2^-126 (n at most 127)
E3_DEV float exp2_int(int n) { return n < -126 ? 0.0f : __int_as_float((n + 127) << 23); }

// the power of two that brings a row's largest magnitude to [2^to, 2^(to + 1)); 0 of a row that is all zero or not
// finite, and never so far that 2^-n or 2^n is not a normal number
E3_DEV int row_shift(float amax, int to) {
    const int e = (int)(__float_as_uint(amax) >> 23);
    return e == 0 || e == 255 ? 0 : max(-126, min(126, to + 127 - e));
}

E3_DEV uint32_t pack_f16(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

E3_DEV uint32_t max_u16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// the largest magnitude of 8 bf16 as its 15 bits, which are in order (BF16_INF and up: not finite), and of the finite ones
constexpr uint32_t BF16_INF = 0x7f80u;
E3_DEV uint32_t amax_bits(uint4 u) {
    const uint32_t m = max_u16x2(max_u16x2(u.x & 0x7fff7fffu, u.y & 0x7fff7fffu), max_u16x2(u.z & 0x7fff7fffu, u.w & 0x7fff7fffu));
    return max(m & 0xffffu, m >> 16);
}
E3_DEV uint32_t amax_bits_finite(uint4 u) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const uint32_t h = (e & 1 ? w[e >> 1] >> 16 : w[e >> 1]) & 0x7fffu;
        m = max(m, h < BF16_INF ? h : 0u);
    }
    return m;
}
// the largest finite magnitude of 8 bf16 (others: set in `odd`)
E3_DEV float amax8(uint4 u, bool &odd) {
    uint32_t m = amax_bits(u);
    if (m >= BF16_INF) {
        odd = true;
        m = amax_bits_finite(u);
    }
    return __uint_as_float(m << 16);
}
// scale_byte of a finite bf16 magnitude's bits
E3_DEV int scale_byte_bits(uint32_t m) { return max(1, (int)(m >> 7) - 8 + ((m & 0x7fu) > 0x60u ? 1 : 0)); }

// The nodes that node i sees: itself and its ancestors, up to the root or to a parent that is none
E3_DEV uint64_t path_bits(const int32_t *par, int i, bool &bad) {
    uint64_t bits = 1ull << i;
    for (;;) {
        const int q = __ldg(par + i);
        if (i == 0) {
            if (q != -1) bad = true;
            return bits;
        }
        if (q < 0 || q >= i) {
            bad = true;
            return bits;
        }
        i = q;
        bits |= 1ull << i;
    }
}

// What a part of a prefix counts by when parts are joined: 2^(m - M) of its row's maximum, 0 where it has summed up nothing (and
// may have left nothing).  No less than 2^-126 otherwise, so that what is not finite there (NaN codes and scales of V, a
// tree's values) reaches the row as it does inside a part; of finite values that is n 2^-118 of the largest at most, where
// the weights' floor inside a part is 2^-31 of it.
E3_DEV float part_factor(float m, float l, float M) {
    return m == -INFINITY ? (l == 0.0f ? 0.0f : 1.0f) : fmaxf(fast_exp2(m - M), FLT_MIN);   // (all scores NaN: a sum, no maximum)
}

E3_DEV float lse_of(float m, float l) {   // (the weights are 2^WEIGHT_LOG2 up)
    return l == 0.0f ? -INFINITY : m == -INFINITY ? l : ((m - WEIGHT_LOG2) + log2f(l)) * 0.6931471805599453f;
}

// A finished row: dims [4 lane, 4 lane + 4) of o by each lane of a warp
E3_DEV void store_row(const CacheAttn &p, size_t row, int lane, float m, float l, float4 o) {
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    __nv_bfloat162 w[2] = {__floats2bfloat162_rn(o.x * inv, o.y * inv), __floats2bfloat162_rn(o.z * inv, o.w * inv)};
    *reinterpret_cast<uint2 *>(p.out + row * 128 + 4 * lane) = *reinterpret_cast<const uint2 *>(w);
    if (p.lse && lane == 0) p.lse[row] = lse_of(m, l);
}

// many rows (cache_attn_wide.cu)
size_t cache_attn_wide_workspace(const CacheAttn &a);
eagle3_status_t cache_attn_wide(const CacheAttn &a, const WaitRule &wait, void *workspace, size_t bytes, cudaStream_t stream);

}  // namespace e3
