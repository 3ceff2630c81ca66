// eagle3_verify_attn_fp8: attention of single tokens and of tree nodes over an e4m3 paged cache with a power-of-two
// scale for each 64 places and KV head (include/eagle3_kv.h).
//
// Sources: "Advanced speculative decoding: tree drafts and EAGLE", sections "Why trees" and "Implementation" (each
// node sees the whole prefix plus itself and its ancestors); "EAGLE-3: Engineering Implementation of LLM Inference
// Acceleration", appendix C (GQA, 1/sqrt(D) scaling).
//
// Rows kernel: up to 8 or 16 query rows (row = node * rep + head of the KV group) by the warps of a CTA, each with 32
// keys of its own at a time and running maxima and sums of its own, merged at the end in warp order.  Nothing is
// staged: a lane reads 16 codes of a key row at once, and which dims of K (keys of V) a lane holds is laid out so that
// they are fragments of mma.m16n8k16 after conversion to fp16, which is exact.  The dims are permuted to match.
//   scores   S = Q K^T: lane (g, c) of a warp, g = lane / 4, c = lane % 4, reads key g of each 8, dims [16c, 16c + 16)
//            and [64 + 16c, 64 + 16c + 16): word w of the first run is the B fragment of k-step w, the k indices
//            {2c, 2c + 1, 2c + 8, 2c + 9} being the dims 16c + 4w + {0, 1, 2, 3}
//   values   O^T = V^T P^T, so that 8 rows of queries need 8 columns and not a tile of 16: S's registers are P^T's B
//            fragments as they are.  Keys {2c, 2c + 1, 2c + 8, 2c + 9} of each 16, dims [16g, 16g + 16): byte permutes
//            pair up two keys' codes of a dim; tile t of O^T holds the dims 16g + 2t (row g) and 16g + 2t + 1
//            (row g + 8), its columns 2c, 2c + 1 are rows of Q
// A warp's next K is loaded once the products with this one have been issued, its next V after the weights' products,
// and the pages two steps ahead: each load has about half a step to arrive, in no registers of its own.
// Rows beyond 16 are groups of CTAs of their own, which read the keys again.
// Bound by memory at the largest calls: 64 single tokens of 32 heads over up to 8192 positions (669 MB) take 115 us,
// 5.8 TB/s, one over 250000 (512 MB) 84 us, 6.1 TB/s; the copy's rate is 6.8.  With Q's rows as the tile's 16 (64 MMAs a
// step where 8 rows need 48, 64 more registers, loads only between steps) they took 174 and 216 us.  By waves and latency
// below that: 8 sequences of 4096 positions 17.5 us, 3.8 TB/s, 32 of them 54 to 56 us, 4.9 TB/s; 64 of 5 queries each, two
// groups of rows that each read the keys, 150 us, 3.6 TB/s.  One token over 4096 positions: 8.1 to 9.0 us, latency.
// Q is scaled by a power of two for each row so that fp16 holds it (bf16's 8 bits fit, elements 2^-36 below the row's
// largest vanish); the factor comes back with the scale of K's group in fp32.  Weights are held 2^7 up, so that fp16's
// 11 bits reach down to 2^-21 of the largest, and V's group scale is put on them relative to the largest so far.
#include "cache_attn.cuh"
#include "eagle3_testing.h"
#include "tc.cuh"

#include <cfloat>

namespace e3 {
namespace {

constexpr int D = 128;
constexpr int CHUNK = 32;           // keys of a warp's step: within one group of 64, so one scale and one page
constexpr int NW = 4;               // warps
constexpr int NT = NW * 32;
constexpr int MAX_ROWS = 16;
constexpr int O_PITCH = D + 4;

E3_DEV void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 16 codes that this grid reads once
E3_DEV uint4 ld_once(const uint8_t *p) {
    uint4 u;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "l"(p));
    return u;
}

// 16 bf16 as fp16 pairs, times a power of two
E3_DEV void bf16x16_f16(const uint4 (&in)[2], float factor, uint32_t (&out)[8]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t w[4] = {in[i].x, in[i].y, in[i].z, in[i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w[e]));
            out[4 * i + e] = pack_f16(f.x * factor, f.y * factor);
        }
    }
}

// The running state of a warp, rows g + 8 r
template <int NR>
struct RowState {
    float m[NR], l[NR];   // the maximum and this lane's share of the sum of row g + 8 r
    int ev;               // V's scale byte that o is relative to
    float o[8][NR][4];    // dims 16g + 2t + {0, 0, 1, 1} of rows 8r + 2c + {0, 1, 0, 1}
};

// The weights of a step of 32 keys, as B fragments, from its raw scores s (four tiles of 8 keys) by the rows' factors f;
// seen: bit 2 n + i of a row for this lane's key 2c + i of tile n; ev: V's scale byte.
template <int NR>
E3_DEV void softmax_step(RowState<NR> &st, float (&s)[4][4], const float (&f)[NR], const uint32_t (&seen)[NR], int ev,
                         uint32_t (&pf)[2][NR][2]) {
    float mx[NR];
    bool grown = ev > st.ev && ev != 255;
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        mx[r] = -INFINITY;
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float &x = s[n][2 * r + i];
                x = (seen[r] >> (2 * n + i)) & 1u ? x * f[r] : -INFINITY;
                mx[r] = fmaxf(mx[r], x);
            }
        grown = grown || mx[r] > st.m[r] + RESCALE_LOG2;
    }
    if (__any_sync(0xffffffffu, grown)) {
        const float down = ev > st.ev && ev != 255 ? exp2_int(st.ev - ev) : 1.0f;
        if (ev != 255) st.ev = max(st.ev, ev);
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
            mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
            const float m = fmaxf(st.m[r], mx[r]);
            const float e = st.m[r] == -INFINITY ? 0.0f : fast_exp2(st.m[r] - m);
            st.m[r] = m;
            st.l[r] *= e;
            const int c = threadIdx.x & 3;
            const float c0 = __shfl_sync(0xffffffffu, e, 8 * c) * down, c1 = __shfl_sync(0xffffffffu, e, 8 * c + 4) * down;
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                st.o[t][r][0] *= c0;
                st.o[t][r][1] *= c1;
                st.o[t][r][2] *= c0;
                st.o[t][r][3] *= c1;
            }
        }
    }
    const float vs = ev == 255 ? __int_as_float(0x7fc00000) : exp2_int(ev - st.ev);
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        const float nm = st.m[r] == -INFINITY ? 0.0f : WEIGHT_LOG2 - st.m[r];
        float sum = 0.0f;
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const float p0 = fast_exp2(s[n][2 * r] + nm), p1 = fast_exp2(s[n][2 * r + 1] + nm);
            sum += p0 + p1;
            pf[n >> 1][r][n & 1] = pack_f16(p0 * vs, p1 * vs);
        }
        st.l[r] += sum;
    }
}

// Where a step of 32 keys lies; ek, ev: its scale bytes
struct Place {
    size_t at;          // its first code
    int left, ek, ev;   // left: its keys that are there, 0 or less: none
};

E3_DEV float warp_max(float x) {
#pragma unroll
    for (int d = 16; d; d >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
    return x;
}
E3_DEV float warp_sum(float x) {
#pragma unroll
    for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    return x;
}

// grid: (split, KV head and group of rows, sequence); NR: 8 NR rows a group.  CLUSTERED: the splits are the CTAs of
// a cluster and read each other's results from shared memory; otherwise they leave theirs to the merge kernels.
template <int NR, bool CLUSTERED>
__global__ void __launch_bounds__(NT, NR == 1 ? 3 : 2) cache_attn_rows_kernel(const CacheAttn p) {
    constexpr int ROWS = 8 * NR;
    __shared__ float so[NW][ROWS][O_PITCH];
    __shared__ float sm[NW][ROWS], sl[NW][ROWS];
    __shared__ int sev[NW];
    pdl_wait();
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const int split = blockIdx.x, h = blockIdx.y / p.row_groups, b = blockIdx.z;
    const int row0 = blockIdx.y % p.row_groups * ROWS, nrows = min(ROWS, p.N * p.rep - row0);
    const bool reports = split == 0 && blockIdx.y == 0 && threadIdx.x == 0;
    const int32_t *bt = p.block_table + (size_t)b * p.max_blocks;
    int L = __ldg(p.prefix_len + b);
    if (L < 0 || L > p.max_prefix) {
        if (reports) flag(p.dev_status, EAGLE3_DEV_CAPACITY);
        L = max(0, min(L, p.max_prefix));
    }

    // ---- the prefix: chunks [c0, c1) of this split, one after the other by the warps
    const int chunks = (L + CHUNK - 1) / CHUNK;
    const int c0 = min(chunks, split * p.split_chunks), c1 = min(chunks, c0 + p.split_chunks);
    const int sgroups = p.block_size / EAGLE3_KV_GROUP;
    auto page_of = [&](int ch) { return ch < c1 ? __ldg(bt + ch * CHUNK / p.block_size) : -1; };
    auto place_of = [&](int ch, int page) {
        const int place = ch * CHUNK % p.block_size;
        const bool there = page >= 0 && page < p.n_pages;
        const size_t head_page = (size_t)(there ? page : 0) * p.Hkv + h;
        const size_t sg = head_page * sgroups + place / EAGLE3_KV_GROUP;
        Place w;
        w.at = (head_page * p.block_size + place) * D;
        w.left = there ? L - ch * CHUNK : 0;
        w.ek = there ? __ldg(p.ks + sg) : 1;   // (a page that is not there reads as zeros)
        w.ev = there ? __ldg(p.vs + sg) : 1;
        return w;
    };
    uint4 kw[4][2], vw[2][4];
    const uint4 zero = make_uint4(0, 0, 0, 0);
    auto load_k = [&](const Place &w) {
        const uint8_t *at = p.kc + w.at + (g * D + 16 * c);
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                kw[n][i] = 8 * n + g < w.left ? ld_once(at + 8 * n * D + 64 * i) : zero;
    };
    auto load_v = [&](const Place &w) {
        const uint8_t *at = p.vc + w.at + (2 * c * D + 16 * g);
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int key = 16 * k + (e & 1) + (e >> 1) * 8;
                vw[k][e] = key + 2 * c < w.left ? ld_once(at + key * D) : zero;
            }
    };
    int ch = c0 + warp;
    int page_next = page_of(ch + NW);
    Place at = place_of(ch, page_of(ch));
    load_k(at);
    load_v(at);

    // ---- Q: fragments of the rows of this lane, each row scaled to [2^12, 2^13)
    uint32_t qf[8][2 * NR];   // [k-step][row g + 8 r, then its second half]
    float f[NR];
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        const int row = g + 8 * r;
        float top = 0.0f;
        uint4 raw[2][2] = {{zero, zero}, {zero, zero}};
        if (row < nrows) {
            const int node = (row0 + row) / p.rep, head = h * p.rep + (row0 + row) % p.rep;
            const __nv_bfloat16 *src = p.q + ((size_t)b * p.N + node) * p.q_ns + (size_t)head * D + 16 * c;
            bool odd = false;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                raw[i >> 1][i & 1] = *reinterpret_cast<const uint4 *>(src + 64 * (i >> 1) + 8 * (i & 1));
                top = fmaxf(top, amax8(raw[i >> 1][i & 1], odd));
            }
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int up = row_shift(top, 12);
        f[r] = p.scale_log2 * exp2_int(-up);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint32_t w[8];
            bf16x16_f16(raw[i], exp2_int(up), w);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                qf[4 * i + k][r] = w[2 * k];
                qf[4 * i + k][NR + r] = w[2 * k + 1];
            }
        }
    }
    auto score = [&](float (&s)[4], int k, uint32_t b0, uint32_t b1) {   // (rows that there are not: zeros)
        mma_f16(s, qf[k][0], NR == 2 ? qf[k][NR - 1] : 0u, qf[k][NR], NR == 2 ? qf[k][2 * NR - 1] : 0u, b0, b1);
    };

    RowState<NR> st;
    st.ev = 0;
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        st.m[r] = -INFINITY;
        st.l[r] = 0.0f;
#pragma unroll
        for (int t = 0; t < 8; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) st.o[t][r][e] = 0.0f;
    }

    for (; ch < c1; ch += NW) {
        const Place next = place_of(ch + NW, page_next);
        page_next = page_of(ch + 2 * NW);
        float s[4][4];
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.0f;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const uint4 u = kw[n][k >> 2];
                const uint32_t w = (k & 3) == 0 ? u.x : (k & 3) == 1 ? u.y : (k & 3) == 2 ? u.z : u.w;
                score(s[n], k, e4m3x2_f16(w), e4m3x2_f16(w >> 16));
            }
        }
        load_k(next);
        const int left = L - ch * CHUNK;
        uint32_t seen[NR];
        seen[0] = 0xffu;
        if (left < CHUNK) {
            seen[0] = 0;
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i) seen[0] |= (8 * n + 2 * c + i < left ? 1u : 0u) << (2 * n + i);
        }
        float fs[NR];
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            seen[r] = seen[0];
            fs[r] = f[r] * scale_of(at.ek);
        }
        uint32_t pf[2][NR][2];
        softmax_step<NR>(st, s, fs, seen, at.ev, pf);
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                auto word = [&](const uint4 &u) { return w == 0 ? u.x : w == 1 ? u.y : w == 2 ? u.z : u.w; };
                const uint32_t r0 = word(vw[k][0]), r1 = word(vw[k][1]), r2 = word(vw[k][2]), r3 = word(vw[k][3]);
                const uint32_t lo0 = __byte_perm(r0, r1, 0x5140), hi0 = __byte_perm(r0, r1, 0x7362);
                const uint32_t lo1 = __byte_perm(r2, r3, 0x5140), hi1 = __byte_perm(r2, r3, 0x7362);
#pragma unroll
                for (int r = 0; r < NR; ++r) {
                    mma_f16(st.o[2 * w][r], e4m3x2_f16(lo0), e4m3x2_f16(lo0 >> 16), e4m3x2_f16(lo1),
                            e4m3x2_f16(lo1 >> 16), pf[k][r][0], pf[k][r][1]);
                    mma_f16(st.o[2 * w + 1][r], e4m3x2_f16(hi0), e4m3x2_f16(hi0 >> 16), e4m3x2_f16(hi1),
                            e4m3x2_f16(hi1 >> 16), pf[k][r][0], pf[k][r][1]);
                }
            }
        load_v(next);
        at = next;
    }

    // ---- the tree: its nodes as one or two more steps of the last split
    if (p.tree_k && split == p.splits - 1 && warp * CHUNK < p.N) {
        const int key0 = warp * CHUNK, keys = min(CHUNK, p.N - key0);
        const int32_t *par = p.parents + (size_t)b * p.N;
        // bf16 rows as fp16, K and V each by a power of two of their largest
        const __nv_bfloat16 *tk = p.tree_k + ((size_t)b * p.N + key0) * p.kv_ns + (size_t)h * D;
        const __nv_bfloat16 *tv = p.tree_v + ((size_t)b * p.N + key0) * p.kv_ns + (size_t)h * D;
        uint32_t anc[NR];   // which of these nodes a row sees
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            const int row = g + 8 * r;
            bool bad = false;
            anc[r] = row < nrows ? (uint32_t)(path_bits(par, (row0 + row) / p.rep, bad) >> key0) : 0u;
            if (bad && h == 0) flag(p.dev_status, EAGLE3_DEV_BAD_TREE);
        }
        float top = 0.0f;
        bool odd_k = false, odd_v = false;   // V is not finite somewhere: see below
        uint4 raw[8][2];                     // K's dims [64i + 16c, + 16) of key 8n + g, then V's
#pragma unroll
        for (int x = 0; x < 8; ++x)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const int key = 8 * (x >> 1) + g;
                raw[x][y] = key < keys ? *reinterpret_cast<const uint4 *>(tk + key * p.kv_ns + 64 * (x & 1) + 16 * c + 8 * y) : zero;
            }
#pragma unroll
        for (int x = 0; x < 8; ++x)
#pragma unroll
            for (int y = 0; y < 2; ++y) top = fmaxf(top, amax8(raw[x][y], odd_k));
        const int kup = row_shift(__uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top))), 8);   // to [2^8, 2^9), as the codes
        float s[4][4];
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.0f;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                uint32_t w[8];
                bf16x16_f16(raw[2 * n + i], exp2_int(kup), w);
#pragma unroll
                for (int k = 0; k < 4; ++k) score(s[n], 4 * i + k, w[2 * k], w[2 * k + 1]);
            }
        }
        // V's dims [16g, 16g + 16) of keys 16k + {2c, 2c + 1, 2c + 8, 2c + 9}
#pragma unroll
        for (int x = 0; x < 8; ++x)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const int key = 16 * (x >> 2) + 2 * c + (x & 1) + (x >> 1 & 1) * 8;
                raw[x][y] = key < keys ? *reinterpret_cast<const uint4 *>(tv + key * p.kv_ns + 16 * g + 8 * y) : zero;
            }
        top = 0.0f;
#pragma unroll
        for (int x = 0; x < 8; ++x)
#pragma unroll
            for (int y = 0; y < 2; ++y) top = fmaxf(top, amax8(raw[x][y], odd_v));
        const int vup = row_shift(__uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top))), 8);
        uint32_t seen[NR];
        float fs[NR];
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            seen[r] = 0;
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i) seen[r] |= (anc[r] >> (8 * n + 2 * c + i) & 1u) << (2 * n + i);
            fs[r] = f[r] * exp2_int(-kup);
        }
        uint32_t pf[2][NR][2];
        softmax_step<NR>(st, s, fs, seen, max(0, min(254, 127 - vup)), pf);
        const float vf = exp2_int(vup);
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                auto word = [&](int e, int d) {
                    const uint4 u = raw[4 * k + e][half];
                    return d == 0 ? u.x : d == 1 ? u.y : d == 2 ? u.z : u.w;
                };
#pragma unroll
                for (int d = 0; d < 4; ++d) {
                    auto at = [&](int e, bool upper) {
                        const float x = __uint_as_float(upper ? word(e, d) & 0xffff0000u : word(e, d) << 16);
                        return fabsf(x) <= FLT_MAX ? x * vf : 0.0f;
                    };
                    const uint32_t a0 = pack_f16(at(0, false), at(1, false)), a1 = pack_f16(at(0, true), at(1, true));
                    const uint32_t a2 = pack_f16(at(2, false), at(3, false)), a3 = pack_f16(at(2, true), at(3, true));
#pragma unroll
                    for (int r = 0; r < NR; ++r)
                        mma_f16(st.o[4 * half + d][r], a0, a1, a2, a3, pf[k][r][0], pf[k][r][1]);
                }
            }
        // infinities and NaN of V, which a weight of 0 would have spread over every row: to the rows that see them
        if (__any_sync(0xffffffffu, odd_v)) {
#pragma unroll
            for (int r = 0; r < NR; ++r)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t sees = __shfl_sync(0xffffffffu, anc[r], 8 * c + 4 * i);   // of row 8r + 2c + i
                    for (int key = 0; key < keys; ++key)
#pragma unroll
                        for (int t = 0; t < 8; ++t)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const float x = (float)tv[key * p.kv_ns + 16 * g + 2 * t + e];
                                if (!(fabsf(x) <= FLT_MAX) && (sees >> key & 1u)) st.o[t][r][2 * e + i] += x;
                            }
                }
        }
    }

    // ---- the warps' results, in warp order
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        float l = st.l[r];
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);
        if (c == 0) {
            sm[warp][g + 8 * r] = st.m[r];
            sl[warp][g + 8 * r] = l;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int t = 0; t < 8; t += 2)
                *reinterpret_cast<float4 *>(&so[warp][8 * r + 2 * c + i][16 * g + 2 * t]) =
                    make_float4(st.o[t][r][i], st.o[t][r][2 + i], st.o[t + 1][r][i], st.o[t + 1][r][2 + i]);
    }
    if (lane == 0) sev[warp] = st.ev;
    __syncthreads();
    for (int row = warp; row < nrows; row += NW) {
        float M = -INFINITY, l = 0.0f;
#pragma unroll
        for (int w = 0; w < NW; ++w) M = fmaxf(M, sm[w][row]);
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const float e = part_factor(sm[w][row], sl[w][row], M);
            l += e * sl[w][row];
            const float vs = e * scale_of(sev[w]);
            const float4 x = *reinterpret_cast<const float4 *>(&so[w][row][4 * lane]);
            if (e != 0.0f) o = make_float4(o.x + vs * x.x, o.y + vs * x.y, o.z + vs * x.z, o.w + vs * x.w);
        }
        const int node = (row0 + row) / p.rep, head = h * p.rep + (row0 + row) % p.rep;
        const size_t at_row = ((size_t)b * p.N + node) * p.Hq + head;
        if (p.splits == 1) {
            store_row(p, at_row, lane, M, l, o);
        } else if constexpr (CLUSTERED) {
            __syncwarp();   // (this row's statistics have been read)
            *reinterpret_cast<float4 *>(&so[0][row][4 * lane]) = o;
            if (lane == 0) sm[0][row] = M, sl[0][row] = l;
        } else {
            const size_t part = (size_t)split * p.B * p.N * p.Hq + at_row;
            if (l != 0.0f) *reinterpret_cast<float4 *>(p.part_o + part * D + 4 * lane) = o;   // (NaN too)
            if (lane == 0) *reinterpret_cast<float2 *>(p.part_ml + 2 * part) = make_float2(M, l);
        }
    }
    if constexpr (!CLUSTERED) return;
    // ---- the splits' results in their order, rows by turns of the cluster's warps
    tc::cluster_sync();
    for (int row = split * NW + warp; row < nrows; row += p.splits * NW) {
        float2 ml = make_float2(-INFINITY, 0.0f);
        if (lane < p.splits)
            ml = make_float2(tc::cluster_ld(tc::cluster_addr(smem_u32(&sm[0][row]), lane)),
                             tc::cluster_ld(tc::cluster_addr(smem_u32(&sl[0][row]), lane)));
        const float M = warp_max(ml.x), e = part_factor(ml.x, ml.y, M), l = warp_sum(e * ml.y);
        const uint32_t at = smem_u32(&so[0][row][4 * lane]);
        float4 x[MAX_CLUSTER], o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int s = 0; s < MAX_CLUSTER; ++s)
            if (s < p.splits) x[s] = tc::cluster_ld4(tc::cluster_addr(at, s));
#pragma unroll
        for (int s = 0; s < MAX_CLUSTER; ++s) {
            const float es = __shfl_sync(0xffffffffu, e, s);
            if (s < p.splits && es != 0.0f) o = make_float4(o.x + es * x[s].x, o.y + es * x[s].y, o.z + es * x[s].z, o.w + es * x[s].w);
        }
        const int node = (row0 + row) / p.rep, head = h * p.rep + (row0 + row) % p.rep;
        store_row(p, ((size_t)b * p.N + node) * p.Hq + head, lane, M, l, o);
    }
    tc::cluster_sync();   // no CTA leaves while another reads its results
}

// The splits' results where they are not a cluster.  Few splits: a warp a row.  Many: a CTA a row, a quarter of the splits to
// each of its warps.
constexpr int FEW_SPLITS = 16;   // 16384 rows of 2 splits and 128 threads a row took 14 us; 32 rows of 57 and a warp a row 9 us

// splits [s0, s1) of a row by their factors, with eight loads in flight; factor(s): of split s, the same in all lanes
template <typename F>
E3_DEV float4 weighted_sum(const CacheAttn &p, long long rows, long long row, int s0, int s1, int lane, F factor) {
    constexpr int K = 8;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int s = s0; s < s1; s += K) {
        float4 x[K];
        float e[K];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            e[k] = factor(min(s + k, s1 - 1));   // (a split with nothing to see has left nothing there)
            if (s + k >= s1) e[k] = 0.0f;
            if (e[k] != 0.0f) x[k] = *reinterpret_cast<const float4 *>(p.part_o + ((s + k) * rows + row) * D + 4 * lane);
        }
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (e[k] != 0.0f) o = make_float4(o.x + e[k] * x[k].x, o.y + e[k] * x[k].y, o.z + e[k] * x[k].z, o.w + e[k] * x[k].w);
    }
    return o;
}
E3_DEV float2 split_ml(const CacheAttn &p, long long rows, long long row, int s) {
    return s < p.splits ? *reinterpret_cast<const float2 *>(p.part_ml + 2 * (s * rows + row)) : make_float2(-INFINITY, 0.0f);
}

__global__ void __launch_bounds__(NT) cache_attn_merge_few_kernel(const CacheAttn p) {
    pdl_wait();
    pdl_trigger();
    const long long rows = (long long)p.B * p.N * p.Hq, row = (long long)blockIdx.x * NW + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (row >= rows) return;
    const float2 ml = split_ml(p, rows, row, lane);
    const float M = warp_max(ml.x), e = part_factor(ml.x, ml.y, M), l = warp_sum(e * ml.y);
    store_row(p, (size_t)row, lane, M, l, weighted_sum(p, rows, row, 0, p.splits, lane, [&](int s) { return __shfl_sync(0xffffffffu, e, s); }));
}

__global__ void __launch_bounds__(NT) cache_attn_merge_kernel(const CacheAttn p) {
    __shared__ float4 so[NW][32];
    __shared__ float sl[NW], sm[NW];
    __shared__ float sw[MAX_SPLITS];   // a split's factor
    pdl_wait();
    pdl_trigger();
    const long long rows = (long long)p.B * p.N * p.Hq, row = blockIdx.x;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float2 ml[MAX_SPLITS / NT];
    float M = -INFINITY, l = 0.0f;
#pragma unroll
    for (int i = 0; i < MAX_SPLITS / NT; ++i) {
        ml[i] = split_ml(p, rows, row, threadIdx.x + i * NT);
        M = fmaxf(M, ml[i].x);
    }
    M = warp_max(M);
    if (lane == 0) sm[warp] = M;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < NW; ++w) M = fmaxf(M, sm[w]);
#pragma unroll
    for (int i = 0; i < MAX_SPLITS / NT; ++i) {
        const float e = part_factor(ml[i].x, ml[i].y, M);
        sw[threadIdx.x + i * NT] = e;
        l += e * ml[i].y;
    }
    l = warp_sum(l);
    if (lane == 0) sl[warp] = l;
    __syncthreads();
    so[warp][lane] = weighted_sum(p, rows, row, p.splits * warp / NW, p.splits * (warp + 1) / NW, lane, [&](int s) { return sw[s]; });
    __syncthreads();
    if (warp != 0) return;
    l = 0.0f;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int w = 0; w < NW; ++w) {
        const float4 x = so[w][lane];
        l += sl[w];
        o = make_float4(o.x + x.x, o.y + x.y, o.z + x.z, o.w + x.w);
    }
    store_row(p, (size_t)row, lane, M, l, o);
}

// Parts of the prefix, of as many steps for a short sequence as for a long one, so that all CTAs take about the same
// time: the number that gives the least waves * (steps of a warp + what a CTA costs besides, in steps), about in us.
// Lengths are on the device, so half a wave more stands for the uneven end of all but a single wave, and the bound for the
// lengths: one far above them costs parts without keys (one sequence of 4096 positions by a bound of 4096, 16384 and
// 131072: 8.5, 12 and 26 us; 8: 18, 36 and 53; 32: 56, 66 and 82).
float plan_splits(CacheAttn &p) {
    const int chunks = (p.max_prefix + CHUNK - 1) / CHUNK;
    const bool one = p.N * p.rep <= 8;
    const float units = (float)p.B * p.Hkv * p.row_groups, resident = (float)device_sm_count() * (one ? 3 : 2);
    const float besides = one ? 3.0f : 8.0f;
    // One launch, joined within a cluster, where all clusters fit at once: a CTA then keeps its SM until the slowest of its
    // cluster is done, and clusters of many CTAs leave SMs out (64 sequences of up to 8192 positions, 4 parts: 154 us
    // as clusters, 116 us with a second kernel; 8 sequences of 4096, 7 parts: 25 and 17 us; one of 4096: 11 and 15 us a call).
    // More than 8 rows, up to 4 parts: also where an SM gets two CTAs, which such small clusters leave fewer SMs out for (7 x
    // 17 nodes of 12 heads over 3001 positions, 3 parts: 24.4 us as clusters, 25.1 with a second kernel; 4 nodes of 9
    // sequences over 4096, 4 parts: 26.5 and 27.9; 60 nodes of 2 sequences over 2048, 2 heads a KV head, 4 parts: 19.0 and
    // 20.5; with 2 parts 29.2 and 28.1, 22.5 and 22.6, but 3 or 4 are then the choice)
    auto as_cluster = [&](int s) {
        return s > 1 && s <= MAX_CLUSTER && units * s <= (s <= 4 && !one ? resident : (float)device_sm_count());
    };
    int best = 1;
    float least = 0.0f;
    for (int s = 1; s <= MAX_SPLITS && (s == 1 || s * NW <= chunks); ++s) {
        const float waves = units * s / resident;
        const float cost = (waves <= 1.0f ? 1.0f : waves + 0.5f) * ((chunks + s * NW - 1) / (s * NW) + besides) +
                           (s == 1 ? 0.0f : as_cluster(s) ? 0.5f : 4.0f + s / 24.0f);   // the join
        if (s == 1 || cost < least) least = cost, best = s;
        if (waves > 8.0f) break;
    }
    if (p.requested > 0) best = p.requested < chunks ? p.requested : chunks;
    if (best < 1) best = 1;
    p.split_chunks = (chunks + best - 1) / best;
    p.splits = chunks == 0 ? 1 : (chunks + p.split_chunks - 1) / p.split_chunks;
    p.clustered = as_cluster(p.splits);
    return least;
}

bool valid(const eagle3_verify_attn_fp8_args_t *a, eagle3_status_t *why) {
    *why = EAGLE3_ERR_INVALID_ARGUMENT;
    if (!a || a->batch < 0 || a->n_nodes < 1 || a->n_heads < 1 || a->n_kv_heads < 1 || a->head_dim < 1 ||
        a->max_prefix_len < 0 || a->num_splits < 0 || a->max_blocks < 1 || a->block_size < 1 ||
        a->block_size % EAGLE3_KV_GROUP || a->n_pages < 1 || a->q_node_stride < 0 || a->kv_node_stride < 0 ||
        !(a->sm_scale >= 0.0f && a->sm_scale <= FLT_MAX) || a->n_heads % a->n_kv_heads)
        return false;
    if (!a->tree_k != !a->tree_v || !a->tree_k != !a->parents) return false;
    if ((a->q_node_stride && (a->q_node_stride < (int64_t)a->n_heads * D || a->q_node_stride % 8)) ||
        (a->kv_node_stride && (a->kv_node_stride < (int64_t)a->n_kv_heads * D || a->kv_node_stride % 8)))
        return false;
    *why = EAGLE3_ERR_UNSUPPORTED;
    if (a->head_dim != D || a->n_nodes > 64 || a->batch > 65535 || a->n_heads > 4096 || a->max_prefix_len > MAX_DIM ||
        (int64_t)a->n_pages * a->n_kv_heads * a->block_size > MAX_DIM ||
        (int64_t)a->batch * a->n_nodes * a->n_heads > MAX_DIM)
        return false;
    *why = EAGLE3_ERR_CAPACITY;
    if ((int64_t)a->max_blocks * a->block_size < a->max_prefix_len) return false;
    *why = EAGLE3_OK;
    if (a->batch == 0) return true;
    *why = EAGLE3_ERR_INVALID_ARGUMENT;
    const void *wide[] = {a->q, a->k_cache, a->v_cache, a->out};
    for (const void *ptr : wide)
        if (!ptr || ((uintptr_t)ptr & 15)) return false;
    if (!a->k_scale || !a->v_scale || !a->block_table || !a->prefix_len ||
        (((uintptr_t)a->tree_k | (uintptr_t)a->tree_v) & 15) ||
        (((uintptr_t)a->block_table | (uintptr_t)a->prefix_len | (uintptr_t)a->parents | (uintptr_t)a->lse) & 3))
        return false;
    *why = EAGLE3_OK;
    return true;
}

CacheAttn plan(const eagle3_verify_attn_fp8_args_t *a, bool &wide) {
    CacheAttn p = {};
    p.B = a->batch;
    p.N = a->n_nodes;
    p.Hq = a->n_heads;
    p.Hkv = a->n_kv_heads;
    p.rep = a->n_heads / a->n_kv_heads;
    p.max_prefix = a->max_prefix_len;
    p.max_blocks = a->max_blocks;
    p.block_size = a->block_size;
    p.n_pages = a->n_pages;
    p.scale_log2 = (a->sm_scale > 0.0f ? a->sm_scale : 1.0f / sqrtf((float)D)) * 1.4426950408889634f;
    p.q_ns = a->q_node_stride ? a->q_node_stride : (int64_t)a->n_heads * D;
    p.kv_ns = a->kv_node_stride ? a->kv_node_stride : (int64_t)a->n_kv_heads * D;
    p.q = (const __nv_bfloat16 *)a->q;
    p.tree_k = (const __nv_bfloat16 *)a->tree_k;
    p.tree_v = (const __nv_bfloat16 *)a->tree_v;
    p.parents = a->parents;
    p.kc = a->k_cache;
    p.vc = a->v_cache;
    p.ks = a->k_scale;
    p.vs = a->v_scale;
    p.block_table = a->block_table;
    p.prefix_len = a->prefix_len;
    p.out = (__nv_bfloat16 *)a->out;
    p.lse = a->lse;
    p.dev_status = a->dev_status;
    p.row_groups = (p.N * p.rep + MAX_ROWS - 1) / MAX_ROWS;
    p.requested = a->num_splits < MAX_SPLITS ? a->num_splits : MAX_SPLITS;
    // 16 rows at a time by warps, or 128 by tensor memory: the latter reads a prefix once for up to 128 rows, but takes
    // 30 us to get going and to join.  Both are fits in us; measured, 4 heads a KV head over up to 2048 positions, 16 rows
    // at a time against 128: 16 nodes of 8 sequences 31 and 47 us, 8 nodes of 64 sequences 99 and 144, 60 nodes of one
    // sequence 22 and 33, of 16 sequences 157 and 74.
    const float tiles = (p.max_prefix + 127) / 128 + (p.tree_k ? 8.0f : 2.0f);
    const float wide_us = 30.0f + (float)p.B * p.Hkv * ((p.N * p.rep + 127) / 128) * tiles / 138.0f;
    wide = plan_splits(p) + 6.0f > wide_us && p.N * p.rep > MAX_ROWS;
    return p;
}

// launch_pdl by clusters of `ranks` CTAs along x
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl_clusters(void (*kernel)(KArgs...), dim3 grid, dim3 block, int ranks, cudaStream_t stream, Args &&...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.stream = stream;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)ranks;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = ranks > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<Args &&>(args)...);
}

// Whether a call wants its parts' workspace.  Parts that the caller asks for do, although a cluster, where the device's SMs
// allow one, has no use for it: such a call is taken or refused alike on every device, and on a machine without one.
bool wants_workspace(const CacheAttn &p) { return p.splits > 1 && (!p.clustered || p.requested > 0); }

size_t workspace_of(const CacheAttn &p) {
    return wants_workspace(p) ? (size_t)p.splits * p.B * p.N * p.Hq * (D + 2) * sizeof(float) + 256 : 0;
}

}  // namespace
}  // namespace e3

using namespace e3;

namespace {

// choice: KERNEL_AUTO, or a kernel by name (test hooks); false: that kernel does not take the call
enum { KERNEL_AUTO = 0, KERNEL_ROWS = 1, KERNEL_WIDE = 2 };
bool choose(const CacheAttn &p, int choice, bool &wide) {
    if (choice == KERNEL_AUTO) return true;
    wide = choice == KERNEL_WIDE;
    return !wide || p.N * p.rep > MAX_ROWS;
}

size_t workspace_size(const eagle3_verify_attn_fp8_args_t *a, int choice) {
    eagle3_status_t why;
    if (!valid(a, &why) || a->batch == 0) return 0;
    bool wide;
    const CacheAttn p = plan(a, wide);
    if (!choose(p, choice, wide)) return 0;
    return wide ? cache_attn_wide_workspace(p) : workspace_of(p);
}

eagle3_status_t verify_attn(const eagle3_verify_attn_fp8_args_t *a, int choice, const WaitRule &wait, void *workspace,
                            size_t workspace_bytes, cudaStream_t st) {
    eagle3_status_t why;
    if (!valid(a, &why) || a->batch == 0) return why;
    bool wide;
    CacheAttn p = plan(a, wide);
    if (!choose(p, choice, wide)) return EAGLE3_ERR_INVALID_ARGUMENT;
    if (wide) return cache_attn_wide(p, wait, workspace, workspace_bytes, st);
    if (wants_workspace(p)) {
        if (!workspace || workspace_bytes < workspace_of(p)) return EAGLE3_ERR_WORKSPACE;
        p.part_o = (float *)(((uintptr_t)workspace + 255) & ~(uintptr_t)255);
        p.part_ml = p.part_o + (size_t)p.splits * p.B * p.N * p.Hq * D;
    }
    const dim3 grid((unsigned)p.splits, (unsigned)(p.Hkv * p.row_groups), (unsigned)p.B);
    auto *kernel = p.N * p.rep <= 8 ? (p.clustered ? cache_attn_rows_kernel<1, true> : cache_attn_rows_kernel<1, false>)
                                    : (p.clustered ? cache_attn_rows_kernel<2, true> : cache_attn_rows_kernel<2, false>);
    if (launch_pdl_clusters(kernel, grid, dim3(NT), p.clustered ? p.splits : 1, st, p) != cudaSuccess)
        return EAGLE3_ERR_CUDA;
    if (p.splits > 1 && !p.clustered) {
        const long long rows = (long long)p.B * p.N * p.Hq;
        const cudaError_t e = p.splits <= FEW_SPLITS
                                  ? launch_pdl(cache_attn_merge_few_kernel, dim3((unsigned)((rows + NW - 1) / NW)), dim3(NT), 0, st, p)
                                  : launch_pdl(cache_attn_merge_kernel, dim3((unsigned)rows), dim3(NT), 0, st, p);
        if (e != cudaSuccess) return EAGLE3_ERR_CUDA;
    }
    return EAGLE3_OK;
}

}  // namespace

extern "C" size_t eagle3_verify_attn_fp8_workspace_size(const eagle3_verify_attn_fp8_args_t *a) {
    return workspace_size(a, KERNEL_AUTO);
}

extern "C" eagle3_status_t eagle3_verify_attn_fp8(const eagle3_verify_attn_fp8_args_t *a, void *workspace,
                                                  size_t workspace_bytes, eagle3_stream_t stream) {
    return verify_attn(a, KERNEL_AUTO, WaitRule(), workspace, workspace_bytes, (cudaStream_t)stream);
}

extern "C" size_t eagle3_test_verify_attn_fp8_workspace_size(const eagle3_verify_attn_fp8_args_t *a, int32_t kernel) {
    return kernel < KERNEL_ROWS || kernel > KERNEL_WIDE ? 0 : workspace_size(a, kernel);
}

extern "C" eagle3_status_t eagle3_test_verify_attn_fp8(const eagle3_verify_attn_fp8_args_t *a, void *workspace,
                                                       size_t workspace_bytes, int32_t kernel, int32_t stall_block,
                                                       int64_t wait_limit_cycles, eagle3_stream_t stream) {
    WaitRule wait;
    if (kernel < KERNEL_ROWS || kernel > KERNEL_WIDE || (stall_block >= 0 && kernel != KERNEL_WIDE) ||
        (stall_block != -1 && !stall_rule(&wait, stall_block, -1, wait_limit_cycles)))
        return EAGLE3_ERR_INVALID_ARGUMENT;
    return verify_attn(a, kernel, wait, workspace, workspace_bytes, (cudaStream_t)stream);
}
