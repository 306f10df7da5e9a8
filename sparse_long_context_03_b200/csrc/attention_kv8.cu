// attention_kv8.cu -- sparse GQA attention over the 8-bit paged cache.
//
// The formulas of attention.cu with K[s] = e4m3(k) * 2^ek and V[s] = e4m3(v)
// * 2^ev, one pair of exponents per block of tokens and KV group.  In the
// log2 domain, with c = sm_scale * log2(e), for a selected key i of a head:
//     u_i = c * 2^ek_i * (q . k_i) + ev_i,     w_i = 2^(u_i - ref),
//     O   = sum_i w_i v_i / sum_i w_i 2^-ev_i,
//     lse = ln2 * (ref + log2 sum_i w_i 2^-ev_i).
// Folding ev into the exponent bounds the weights that multiply V by the
// largest product of weight and scale; 2^-ev in the sum is exact.  ref moves
// only when a u exceeds it by more than 15 (weights stay below 2^15 in fp16),
// and is then put 7 below the largest u: nearly every block keeps it, and the
// check is one vote instead of a maximum over the warp.  A weight below fp16's
// normal range is off by at most 2^-25, against 2^7 of the key that set ref:
// 2^-32 of the softmax where V's scales are alike, 2^-28 where this key's is up
// to 2^4 below that one's.  Keys of scales farther below may be all that there
// is in a dim (the scale may be one outlier's, zeros around it), so in steps
// that have such keys the small weights are multiplied in further windows of
// 2^24 (take_small_weights): with a fifth of the pages 2^24 above the others
// 2048 rows take 828 us in place of 392.
//
// e4m3 converts to fp16 without loss, and the products run on fp16 matrix
// instructions with fp32 sums.  (The warp-level 8-bit matrix instructions are
// no way around the conversions: on this chip they are carried out as
// conversions and fp16 products, and with Q and the weights as sums of 8-bit
// parts a 2048-row prompt chunk took 786 us.)  Q is bf16: each head's row is
// multiplied by the power of two that puts its largest value into [2^14,
// 2^15), after which fp16 holds every bf16 value that is 2^-30 of the largest
// or more exactly; the weights are rounded to fp16 (2^-11, an eighth of what
// bf16 would lose; small ones as above), the sums are of the unrounded weights.
//
// Work unit: one warp owns 32 keys of a (query, KV group) pair at a time, all
// G <= 8 heads at once (keys on the matrix M dimension, heads on N = 8).  The
// selected rows go from global memory straight to registers, a quarter of a
// row to a lane.  For S = K Q^T any permutation of the head dims is allowed as
// long as Q has the same, so the lane's bytes are operands as they are; for
// O^T = V^T P^T a movmatrix per word takes them, two dims at a time, to the
// lanes that hold two keys each, and a byte permute pairs the keys.  There is
// no shared-memory stage and no swizzle: staging rows through shared memory
// passes every byte through it twice, and a gather alone then stops at 13 TB/s
// from L2 against 19 TB/s into registers.
//
// What bounds it: with three warps to a scheduler (the next step's K and V, in
// flight, take 64 of 168 registers) the loads and the instructions, 400 for a
// warp's 32 keys and a third of them conversions, overlap only in part: 2048
// query rows of a 32K sequence with k = 2048, 32 heads on 4 groups of 128 dims
// take 392 us, 11.0 TB/s of gathered rows; without the arithmetic 282, and 211
// if a scheduler issued on every cycle.  (The bf16 kernel's 2 times as many
// bytes take 555 us for as many rows.)  32 sequences decoding: 19.2 us, 3.5
// TB/s from HBM (bf16 with its combine: 33 us); the same rows' loads alone 15.
// Tried and slower: half the registers and 16 warps (457 us); V by cp.async
// through shared memory, read back transposed (446 us, with 16 warps 430); the
// next step's products with K among this step's with V (464 us: what is loaded
// then has less time to come); loads under a predicate in place of those that
// nobody needs (453 us); the rows of later steps asked into L2 beforehand
// (decode 26.7 us).
//
#include <cooperative_groups.h>

#include <type_traits>

#include "kernels.h"
#include "kv8.cuh"

namespace cg = cooperative_groups;

namespace dsa {

namespace {

constexpr int kMaxWarps = 8;     // warps of a CTA
constexpr int kMaxCluster = 8;   // CTAs of a cluster
constexpr float kRefNone = -3.402823466e38f;    // the least float: every finite u is above it
constexpr float kF16Normal = 6.103515625e-5f;   // 2^-14: fp16's least normal value
constexpr float kUp = 16777216.f;               // 2^24: from one window of weights to the next
constexpr int kNearLog2 = 4;                     // scales of V no more than 2^4 apart: one window is enough
constexpr float kNear = 1 << kNearLog2;

struct Kv8Args {
    const uint16_t *q;
    const uint8_t *kc, *vc;
    const uint16_t *exps;        // [pages, 64 / block, Hkv] pairs: K's byte low, V's high
    const int32_t *block_table, *seq_lens, *idx, *cu;
    int max_pages, num_pages, nseq, row_begin, n_rows, Hq, Hkv, k, block_shift;
    float scale_log2;
    uint16_t *out;
    float *lse;
};

// The K and V bytes of 16 keys: each lane holds dims tig * D/4 .. + D/4 - 1 of
// keys gid and gid + 8.
template <int D>
struct Tile {
    uint32_t k[2][D / 16], v[2][D / 16];
};

// A row's quarter in one load: 32 bytes (a 256-bit load) or 16.  The four
// lanes of a key then read its whole row, which costs the fewest passes
// through L1.
__device__ __forceinline__ void ldg_stream(uint32_t (&r)[8], const uint8_t *p) {
    asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "l"(p));
}
__device__ __forceinline__ void ldg_stream(uint32_t (&r)[4], const uint8_t *p) {
    asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "l"(p));
}

// Issues the loads of K or V (`to`, from `base`, the lane's quarter of a row)
// of keys half*16 .. +15 of the warp's 32: `row` holds, per lane, the cache
// row of its key.
template <int D>
__device__ __forceinline__ void load_half(uint32_t (&to)[2][D / 16], int row, int half, const uint8_t *base,
                                          uint32_t stride, int lane) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int r = __shfl_sync(0xFFFFFFFFu, row, half * 16 + (lane >> 2) + 8 * i);
        ldg_stream(to[i], base + (uint64_t)(uint32_t)r * stride);
    }
}

// Running state of one warp: lane (gid, tig) holds heads 2 tig and 2 tig + 1;
// o[w] are the products of one matrix instruction, for dims d = dim_of(gid, w)
// (o[w][0], o[w][1]: the two heads) and d + 1 (o[w][2], o[w][3]).
template <int D>
__device__ __forceinline__ int dim_of(int gid, int w) {
    return (gid >> 1) * (D / 4) + 4 * w + 2 * (gid & 1);
}

template <int D>
struct Kv8State {
    uint32_t q[D / 16][2];
    float c[2];                  // c / (the power of two on Q's row), of the two heads
    float o[D / 16][4];
    float ref[2], l[2];
    float far;                   // 2^4 / (the largest scale of V among the keys that moved ref)
};

template <int D>
__device__ __forceinline__ void clear_sums(Kv8State<D> &st) {
#pragma unroll
    for (int w = 0; w < D / 16; ++w)
#pragma unroll
        for (int i = 0; i < 4; ++i) st.o[w][i] = 0.f;
    st.ref[0] = st.ref[1] = kRefNone;
    st.l[0] = st.l[1] = 0.f;
    st.far = INFINITY;
}

template <int D>
__device__ __forceinline__ void load_q(Kv8State<D> &st, const uint16_t *qg, int G, float scale_log2, int lane) {
    const int gid = lane >> 2, tig = lane & 3;
    constexpr int N = D / 32;                       // 16-byte pieces of the lane's quarter of a row
    uint4 raw[N];
    uint32_t mx = 0;
#pragma unroll
    for (int j = 0; j < N; ++j) {
        raw[j] = make_uint4(0, 0, 0, 0);
        if (gid < G) raw[j] = reinterpret_cast<const uint4 *>(qg + (size_t)gid * D + tig * (D / 4))[j];
        const uint32_t w[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            mx = max(mx, (w[i] << 16) & 0x7FFF0000u);
            mx = max(mx, w[i] & 0x7FFF0000u);
        }
    }
    mx = max(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
    mx = max(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
    // largest |q| of the head's row is 2^(ef - 127) * 1.x; the factor is
    // 2^(141 - ef), its inverse 2^(ef - 141)
    const int ef = min(max((int)(mx >> 23), 15), 254);
    const float f = exp_byte_scale(268 - ef), inv = exp_byte_scale(ef - 14) * scale_log2;
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const uint32_t w[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            st.q[2 * j + i / 2][i & 1] =
                pack_f16x2(__uint_as_float(w[i] << 16) * f, __uint_as_float(w[i] & 0xFFFF0000u) * f);
    }
    st.c[0] = __shfl_sync(0xFFFFFFFFu, inv, tig * 8);       // head 2 tig is row gid = 2 tig
    st.c[1] = __shfl_sync(0xFFFFFFFFu, inv, tig * 8 + 4);
}

// What a key's scales come to, by the lane that looked the key up: `scales`
// is K's scale as the upper half of a float and the inverse of V's as the
// upper half in its lower half (powers of two: the halves are exact), `ev` is
// V's exponent.  A key that does not exist has ev = -inf, so its weight is 0.
struct KeyScales {
    uint32_t scales;
    float ev;
};
__device__ __forceinline__ KeyScales no_key() { return {0x3F800000u, -INFINITY}; }
// Of a pair of scale bytes, K's low.
__device__ __forceinline__ KeyScales key_scales(uint32_t e) {
    return {(e & 0xFFu) << 23 | (254u - (e >> 8)) << 7, (float)(int)(e >> 8) - 127.f};
}

// V's bytes of a tile's two words of eight keys each, as the matrix
// instruction's operand: the transpose takes them from a lane per key to a lane
// per two keys, two dims at a time; the byte permute makes pairs of keys of one
// dim.
__device__ __forceinline__ void mma_v(float (&d)[4], uint32_t v0, uint32_t v1, uint32_t b0, uint32_t b1,
                                      bool first = false) {
    const uint32_t x = __byte_perm(movmatrix_trans(v0), 0u, 0x3120), y = __byte_perm(movmatrix_trans(v1), 0u, 0x3120);
    mma_f16_16816(d, e4m3x2_to_f16x2((uint16_t)x), e4m3x2_to_f16x2((uint16_t)(x >> 16)),
                  e4m3x2_to_f16x2((uint16_t)y), e4m3x2_to_f16x2((uint16_t)(y >> 16)), b0, b1, first);
}

// Keys whose weights are below fp16's normal range: their weights are added to
// the sums, multiplied with V in windows of 2^24, each moved into that range,
// and their u is set to -inf, so that what follows passes them by.  After four
// windows the rest is below 2^-110 on a scale on which the reference's key has
// 2^7, and so below 2^-37 of the softmax whatever the scales.
template <int D>
__device__ __forceinline__ void take_small_weights(Kv8State<D> &st, const Tile<D> (&t)[2], float (&u)[2][4],
                                                   const float (&iv)[2][2]) {
    float up = kUp;
#pragma unroll 1
    for (int n = 0; n < 4; ++n, up *= kUp) {
        uint32_t b[2][2];
        bool some = false;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float x[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float p = fast_exp2(u[i][2 * h + j] - st.ref[j]);
                    x[j] = p < kF16Normal ? p * up : 0.f;
                    some = some || (x[j] > 0.f && x[j] < kF16Normal * kUp);
                    if (!(x[j] >= kF16Normal && x[j] < kF16Normal * kUp)) x[j] = 0.f;
                }
                b[i][h] = movmatrix_trans(pack_f16x2(x[0], x[1]));
            }
        if (!__any_sync(0xFFFFFFFFu, some)) break;  // none in this window or below it
        const float down = 1.f / up;
#pragma unroll
        for (int w = 0; w < D / 16; ++w) {
            float sum[4];
#pragma unroll
            for (int i = 0; i < 2; ++i) mma_v(sum, t[i].v[0][w], t[i].v[1][w], b[i][0], b[i][1], i == 0);
#pragma unroll
            for (int j = 0; j < 4; ++j) st.o[w][j] = fmaf(sum[j], down, st.o[w][j]);
        }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float p = fast_exp2(u[i][j] - st.ref[j & 1]);
            if (p < kF16Normal) {                   // not so for a NaN
                st.l[j & 1] = fmaf(p, iv[i][j >> 1], st.l[j & 1]);
                u[i][j] = -INFINITY;
            }
        }
}

// Attends to the 32 keys in t[0] and t[1]; kFar: V's scales may lie more than
// 2^4 below those seen before; scales(i, h) are those of the
// lane's key gid + 8 h of t[i], next_k(i) and next_v(i) issue the loads that
// take t[i]'s place, as soon as its registers are read (after both tiles: 22.1
// us against 21.5 for 32 sequences decoding).
template <int D, bool kFar, typename Scales, typename NextK, typename NextV>
__device__ __forceinline__ void attend_keys(Kv8State<D> &st, Tile<D> (&t)[2], Scales scales, NextK next_k,
                                            NextV next_v) {
    // two chains of products for each tile: half the latency
    float s[2][4], odd[2][4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int w = 0; w < D / 16; ++w) {
            const uint32_t x0 = t[i].k[0][w], x1 = t[i].k[1][w];
            mma_f16_16816(w & 1 ? odd[i] : s[i], e4m3x2_to_f16x2((uint16_t)x0), e4m3x2_to_f16x2((uint16_t)x1),
                                e4m3x2_to_f16x2((uint16_t)(x0 >> 16)), e4m3x2_to_f16x2((uint16_t)(x1 >> 16)),
                                st.q[w][0], st.q[w][1], w < 2);
        }
        next_k(i);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[i][j] += odd[i][j];
    float u[2][4], iv[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const KeyScales x = scales(i, h);
            const float ks = __uint_as_float(x.scales & 0xFFFF0000u);
            iv[i][h] = __uint_as_float(x.scales << 16);
            // K's scale first: the product is exact, and c with it could pass what a float holds
            u[i][2 * h] = fmaf(s[i][2 * h] * ks, st.c[0], x.ev);
            u[i][2 * h + 1] = fmaf(s[i][2 * h + 1] * ks, st.c[1], x.ev);
        }
    float mx[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) mx[i] = fmaxf(fmaxf(u[0][i], u[0][2 + i]), fmaxf(u[1][i], u[1][2 + i]));
    // 1 / (V's scale), the largest among the lane's keys (0 for a key that does not exist)
    const float farthest = fmaxf(fmaxf(iv[0][0], iv[0][1]), fmaxf(iv[1][0], iv[1][1]));
    const bool move = fmaxf(mx[0] - st.ref[0], mx[1] - st.ref[1]) > 15.f;
    if (__any_sync(0xFFFFFFFFu, move || (kFar && farthest > st.far))) {
        if (!kFar || __any_sync(0xFFFFFFFFu, move)) {
            float nearest = INFINITY;
            if (kFar) {
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int h = 0; h < 2; ++h) nearest = iv[i][h] > 0.f ? fminf(nearest, iv[i][h]) : nearest;
            }
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) {
                mx[0] = fmaxf(mx[0], __shfl_xor_sync(0xFFFFFFFFu, mx[0], o));
                mx[1] = fmaxf(mx[1], __shfl_xor_sync(0xFFFFFFFFu, mx[1], o));
                if (kFar) nearest = fminf(nearest, __shfl_xor_sync(0xFFFFFFFFu, nearest, o));
            }
            if (kFar) st.far = fminf(st.far, kNear * nearest);
            float alpha[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float ref = mx[i] - st.ref[i] > 15.f ? mx[i] - 7.f : st.ref[i];
                alpha[i] = fast_exp2(st.ref[i] - ref);
                st.ref[i] = ref;
                st.l[i] *= alpha[i];
            }
#pragma unroll
            for (int w = 0; w < D / 16; ++w) {
                st.o[w][0] *= alpha[0];
                st.o[w][1] *= alpha[1];
                st.o[w][2] *= alpha[0];
                st.o[w][3] *= alpha[1];
            }
        }
        if (kFar && __any_sync(0xFFFFFFFFu, farthest > st.far)) take_small_weights<D>(st, t, u, iv);
    }
    uint32_t b[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float p0 = fast_exp2(u[i][2 * h] - st.ref[0]), p1 = fast_exp2(u[i][2 * h + 1] - st.ref[1]);
            st.l[0] = fmaf(p0, iv[i][h], st.l[0]);
            st.l[1] = fmaf(p1, iv[i][h], st.l[1]);
            b[i][h] = movmatrix_trans(pack_f16x2(p0, p1));
        }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int w = 0; w < D / 16; ++w) mma_v(st.o[w], t[i].v[0][w], t[i].v[1][w], b[i][0], b[i][1]);
        next_v(i);
    }
}

// The sequence b and the position t of query row r; false for a row outside
// every sequence, which is left as it is.
__device__ __forceinline__ bool query_place(const Kv8Args &a, int r, int &b, int &t) {
    if (a.cu == nullptr) {
        b = r;
        t = a.seq_lens[b] - 1;
    } else {
        const int rr = a.row_begin + r;
        if (rr < *a.cu || rr >= a.cu[a.nseq]) return false;
        b = warp_find_seq(a.nseq, rr, [&](int i) { return a.cu[i]; });
        t = a.seq_lens[b] - a.cu[b + 1] + rr;
    }
    t = min(t, a.max_pages * kPage - 1);
    return true;
}

// Sums l over the lanes of a head.
template <int D>
__device__ __forceinline__ void sum_weights(Kv8State<D> &st) {
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
        st.l[0] += __shfl_xor_sync(0xFFFFFFFFu, st.l[0], o);
        st.l[1] += __shfl_xor_sync(0xFFFFFFFFu, st.l[1], o);
    }
}

// One warp's result for a pair: og and lg are its group's outputs.
template <int D>
__device__ __forceinline__ void write_pair(const Kv8State<D> &st, int G, uint16_t *og, float *lg, int lane) {
    const int gid = lane >> 2, tig = lane & 3;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int h = 2 * tig + i;
        if (h >= G) continue;
        const float inv = st.l[i] > 0.f ? 1.f / st.l[i] : 0.f;
#pragma unroll
        for (int w = 0; w < D / 16; ++w)
            *reinterpret_cast<uint32_t *>(og + (size_t)h * D + dim_of<D>(gid, w)) =
                pack_bf16x2(st.o[w][i] * inv, st.o[w][2 + i] * inv);
        if (lg != nullptr && gid == 0) lg[h] = st.l[i] > 0.f ? (st.ref[i] + __log2f(st.l[i])) * kLn2 : -INFINITY;
    }
}

// Shared memory of a joined pair: a part per warp (its sums), then what the
// joining of the warps and of the cluster's CTAs takes.  The sums' heads and
// quarters of a row lie so far apart that the lanes' stores meet no bank twice.
template <int D>
struct Join {
    static constexpr int kQuarter = D == 128 ? 36 : 16, kHead = D == 128 ? 148 : 66, kWarp = 8 * kHead;
    static __device__ __forceinline__ int at(int head, int dim) {
        return head * kHead + dim / (D / 4) * kQuarter + dim % (D / 4);
    }
    static size_t bytes(int warps, int ctas, int G) {
        const size_t slice = ((size_t)G * (D / 2) + ctas - 1) / ctas;
        if (warps * ctas == 1) return 0;
        size_t n = (size_t)warps * (kWarp * sizeof(float) + 8 * sizeof(float2));
        if (ctas > 1) n += ctas * (8 + slice) * sizeof(float2);
        return n;
    }
};

template <int D>
__global__ void __launch_bounds__(384, 1) sparse_kv8_kernel(const __grid_constant__ Kv8Args a) {
    extern __shared__ __align__(16) float smem[];
    using S = Join<D>;
    wait_for_last();
    const int lane = lane_id(), warp = threadIdx.x >> 5, W = blockDim.x >> 5;
    cg::cluster_group cluster = cg::this_cluster();
    const int C = (int)cluster.num_blocks(), crank = (int)cluster.block_rank();
    const int pair = blockIdx.x / C;
    const int r = pair / a.Hkv, g = pair % a.Hkv, G = a.Hq / a.Hkv;

    // 32 keys a step, the pair's warps taking steps in turn.  Nothing waits
    // for what it has just asked for: the indices are read three steps ahead,
    // the pages two, and the next step's K and V are asked for as soon as the
    // registers that this step's took are free.  The first indices are asked
    // for before the sequence's length is known.
    const int32_t *idx_row = a.idx + (size_t)r * a.k;
    const int step0 = crank * W + warp, nw = C * W;
    auto index_at = [&](int step) {
        const int e = step * 32 + lane;
        return e < a.k ? idx_row[e] : -1;
    };
    const int first = index_at(step0), second = index_at(step0 + nw);

    int b, t;
    if (!query_place(a, r, b, t)) return;           // the same answer in every CTA of a cluster
    const int n_vis = max(min(a.k, t + 1), 0);
    const int32_t *bt = a.block_table + (size_t)b * a.max_pages;
    const uint8_t *kg = a.kc + (size_t)g * D + (lane & 3) * (D / 4), *vg = a.vc + (size_t)g * D + (lane & 3) * (D / 4);
    const uint32_t stride = (uint32_t)a.Hkv * D;
    const int steps = (n_vis + 31) / 32;
    // of an index read, the selected position; -1 if it is none
    auto position = [&](int s, int step) { return step * 32 + lane < n_vis && s <= t ? s : -1; };
    auto page_of = [&](int s) { return s >= 0 ? bt[s / kPage] : -1; };
    // a key's scale bytes are looked at a step after they are asked for (at
    // once: 21.6 us against 20.3 for 32 sequences decoding)
    constexpr uint32_t kNoKey = 0x10000u;
    int row, some = -1;
    uint32_t raw;
    auto resolve = [&](int s, int page) {
        row = -1;
        raw = kNoKey;
        if (page >= 0 && page < a.num_pages) {
            row = page * kPage + s % kPage;
            raw = a.exps[(size_t)(row >> a.block_shift) * a.Hkv + g];
        }
        // an entry that selects nothing reads a row that another entry
        // selected, this step's or an earlier one's: with a weight of 0 its
        // values add nothing, and a NaN in them is the output's anyway
        const unsigned found = __ballot_sync(0xFFFFFFFFu, row >= 0);
        if (found != 0) some = __shfl_sync(0xFFFFFFFFu, row, __ffs(found) - 1);
        if (row < 0) row = some;
    };
    if (C > 1) cluster_arrive();                    // waited for before the first store to another CTA
    Kv8State<D> st;
    clear_sums<D>(st);
    // the first step that selects anything
    int step = step0, s0 = position(first, step0);
    resolve(s0, page_of(s0));
    while (some < 0 && (step += nw) < steps) {
        s0 = position(index_at(step), step);
        resolve(s0, page_of(s0));
    }
    if (some >= 0) {
        Tile<D> tile[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) load_half<D>(tile[h].k, row, h, kg, stride, lane);
#pragma unroll
        for (int h = 0; h < 2; ++h) load_half<D>(tile[h].v, row, h, vg, stride, lane);
        s0 = position(step == step0 ? second : index_at(step + nw), step + nw);
        int p0 = page_of(s0), s1 = index_at(step + 2 * nw);
        load_q<D>(st, a.q + ((size_t)r * a.Hq + (size_t)g * G) * D, G, a.scale_log2, lane);
        for (; step < steps; step += nw) {
            const KeyScales now = raw == kNoKey ? no_key() : key_scales(raw);
            // the next step's rows; behind the last step those of the last (a
            // branch around the loads would make them wait: 436 us became 752
            // on a 2048-row prompt chunk)
            resolve(s0, p0);
            s0 = position(s1, step + 2 * nw);
            p0 = page_of(s0);
            s1 = index_at(step + 3 * nw);
            attend_keys<D, true>(
                st, tile,
                [&](int i, int h) {
                    const int from = 16 * i + 8 * h + (lane >> 2);
                    return KeyScales{__shfl_sync(0xFFFFFFFFu, now.scales, from),
                                     __shfl_sync(0xFFFFFFFFu, now.ev, from)};
                },
                [&](int h) { load_half<D>(tile[h].k, row, h, kg, stride, lane); },
                [&](int h) { load_half<D>(tile[h].v, row, h, vg, stride, lane); });
        }
    }
    sum_weights<D>(st);
    const int gid = lane >> 2, tig = lane & 3;
    uint16_t *og = a.out + ((size_t)r * a.Hq + (size_t)g * G) * D;
    float *lg = a.lse != nullptr ? a.lse + (size_t)r * a.Hq + (size_t)g * G : nullptr;
    if (nw == 1) {
        write_pair<D>(st, G, og, lg, lane);
        return;
    }
    // join the warps' sums: within the CTA, then across the cluster
    float2 *ml = reinterpret_cast<float2 *>(smem + W * S::kWarp);   // [W][8] (ref, l)
    float2 *recv_ml = ml + W * 8;                                   // [C][8], from the cluster's CTAs
    float2 *recv = recv_ml + C * 8;                                 // [C][slice]
    float *own = smem + warp * S::kWarp;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int w = 0; w < D / 16; ++w)
            *reinterpret_cast<float2 *>(own + S::at(2 * tig + i, dim_of<D>(gid, w))) =
                make_float2(st.o[w][i], st.o[w][2 + i]);
        if (gid == 0) ml[warp * 8 + 2 * tig + i] = make_float2(st.ref[i], st.l[i]);
    }
    if (C > 1) cluster_wait();
    __syncthreads();
    const int n = G * (D / 2), slice = (n + C - 1) / C;
    for (int e = threadIdx.x; e < n; e += blockDim.x) {
        const int h = e / (D / 2), d = e % (D / 2) * 2;
        float M = kRefNone, L = 0.f, x = 0.f, y = 0.f;
#pragma unroll 4
        for (int w = 0; w < W; ++w) M = fmaxf(M, ml[w * 8 + h].x);
#pragma unroll 4
        for (int w = 0; w < W; ++w) {
            const float2 m = ml[w * 8 + h], v = *reinterpret_cast<const float2 *>(smem + w * S::kWarp + S::at(h, d));
            const float f = fast_exp2(m.x - M);
            L = fmaf(m.y, f, L);
            x = fmaf(v.x, f, x);
            y = fmaf(v.y, f, y);
        }
        if (C == 1) {
            const float inv = L > 0.f ? 1.f / L : 0.f;
            *reinterpret_cast<uint32_t *>(og + (size_t)h * D + d) = pack_bf16x2(x * inv, y * inv);
            if (lg != nullptr && d == 0) lg[h] = L > 0.f ? (M + __log2f(L)) * kLn2 : -INFINITY;
        } else {
            cluster.map_shared_rank(recv, e / slice)[crank * slice + e % slice] = make_float2(x, y);
            // the head's maximum and sum, to the CTA c by the c-th of the head's threads
            if (d / 2 < C) cluster.map_shared_rank(recv_ml, d / 2)[crank * 8 + h] = make_float2(M, L);
        }
    }
    if (C == 1) return;
    cluster.sync();
    for (int i = threadIdx.x; i < slice; i += blockDim.x) {
        const int e = crank * slice + i;
        if (e >= n) break;
        const int h = e / (D / 2), d = e % (D / 2) * 2;
        float top = kRefNone, sum = 0.f, x = 0.f, y = 0.f;
        for (int c = 0; c < C; ++c) top = fmaxf(top, recv_ml[c * 8 + h].x);
        for (int c = 0; c < C; ++c) {
            const float2 m = recv_ml[c * 8 + h], v = recv[c * slice + i];
            const float f = fast_exp2(m.x - top);
            sum = fmaf(m.y, f, sum);
            x = fmaf(v.x, f, x);
            y = fmaf(v.y, f, y);
        }
        const float inv = sum > 0.f ? 1.f / sum : 0.f;
        *reinterpret_cast<uint32_t *>(og + (size_t)h * D + d) = pack_bf16x2(x * inv, y * inv);
        if (lg != nullptr && d == 0) lg[h] = sum > 0.f ? (top + __log2f(sum)) * kLn2 : -INFINITY;
    }
}

// Where every pair has one warp: a CTA has the pairs of a query's neighbouring
// groups, one warp each, and looks the query's entries up once for all of
// them, a block of entries at a time, into shared memory: the rows, and the
// scales of each group.  Against a warp that looks up for itself this saved 45
// of 470 instructions per 32 keys, and pays with a block's start, where nothing
// is under way: 2048 rows (see the head of the file) took 391 us against 420,
// but 32 rows that are split 24.3 against 22.1, so those keep to
// sparse_kv8_kernel.  Blocks of 512 entries: 402 us, 1536: 399, 2048: 413; four
// entries to a thread looked up at once: 405.
// A block whose scales of V all lie within 2^4 of the largest so far takes the
// loop without the check for those below (checked at each step: 408 us).  Four
// CTAs to an SM with 64 dims (without that bound the compiler takes 153
// registers and three fit: 341 us against 306 for 2048 rows).
constexpr int kBlockKeys = 1024;
constexpr int kMaxGroups = 4;

template <int D>
__global__ void __launch_bounds__(kMaxGroups * 32, D == 64 ? 4 : 3) sparse_kv8_rows_kernel(const __grid_constant__ Kv8Args a, int block) {
    extern __shared__ __align__(16) int rows[];     // [block + 32], then the scales, [groups][block]
    __shared__ int some_row[kMaxGroups];
    wait_for_last();
    const int lane = lane_id(), warp = threadIdx.x >> 5, gid = lane >> 2, tig = lane & 3;
    const int groups = blockDim.x >> 5, per_row = a.Hkv / groups;
    const int r = blockIdx.x / per_row, g0 = blockIdx.x % per_row * groups, g = g0 + warp, G = a.Hq / a.Hkv;
    KeyScales *scales = reinterpret_cast<KeyScales *>(rows + block + 32);
    int b, t;
    if (!query_place(a, r, b, t)) return;
    const int n_vis = max(min(a.k, t + 1), 0);
    const int32_t *idx_row = a.idx + (size_t)r * a.k, *bt = a.block_table + (size_t)b * a.max_pages;
    const uint32_t stride = (uint32_t)a.Hkv * D;
    const uint8_t *kg = a.kc + (size_t)g * D + tig * (D / 4), *vg = a.vc + (size_t)g * D + tig * (D / 4);
    Kv8State<D> st;
    clear_sums<D>(st);
    load_q<D>(st, a.q + ((size_t)r * a.Hq + (size_t)g * G) * D, G, a.scale_log2, lane);

    int top = -1000;                                // the largest scale of V so far, its exponent
    for (int base = 0; base < n_vis; base += block) {
        const int n = (min(block, n_vis - base) + 31) / 32 * 32;
        if (base > 0) __syncthreads();              // the last block's keys are no longer read
        int some = -1;
        for (int i = threadIdx.x; i < n; i += blockDim.x) {
            const int s = base + i < n_vis ? idx_row[base + i] : -1;
            const int page = s >= 0 && s <= t ? bt[s / kPage] : -1;
            const bool there = page >= 0 && page < a.num_pages;
            const int row = there ? page * kPage + s % kPage : -1;
            rows[i] = row;
            some = max(some, row);
            for (int j = 0; j < groups; ++j)
                scales[j * block + i] =
                    there ? key_scales(a.exps[(size_t)(row >> a.block_shift) * a.Hkv + g0 + j]) : no_key();
        }
        some = __reduce_max_sync(0xFFFFFFFFu, some);
        if (lane == 0) some_row[warp] = some;
        __syncthreads();
        for (int w = 0; w < groups; ++w) some = max(some, some_row[w]);
        if (some < 0) continue;                     // nothing is selected here

        // an entry that selects nothing, and the step behind the last, read a row
        // that is selected, as in sparse_kv8_kernel
        for (int i = threadIdx.x; i < n + 32; i += blockDim.x)
            if (i >= n || rows[i] < 0) rows[i] = some;
        __syncthreads();
        auto load = [&](uint32_t(&to)[2][D / 16], const int(&from)[2], const uint8_t *base) {
#pragma unroll
            for (int h = 0; h < 2; ++h) ldg_stream(to[h], base + (uint64_t)(uint32_t)from[h] * stride);
        };
        const KeyScales *mine = scales + warp * block + gid;
        Tile<D> tile[2];
        int next[2][2];                             // the rows of a step, read before they are needed
        auto look = [&](int at) {
#pragma unroll
            for (int i = 0; i < 4; ++i) next[i / 2][i % 2] = rows[at + 8 * i + gid];
        };
        look(0);
#pragma unroll
        for (int i = 0; i < 2; ++i) load(tile[i].k, next[i], kg);
#pragma unroll
        for (int i = 0; i < 2; ++i) load(tile[i].v, next[i], vg);
        // the scales of V in this block, while the first rows are on their way
        float hi = -1000.f, lo = 1000.f;
#pragma unroll 4
        for (int i = lane; i < n; i += 32) {
            const float ev = scales[warp * block + i].ev;
            hi = fmaxf(hi, ev);
            lo = fminf(lo, ev > -INFINITY ? ev : lo);
        }
        top = max(top, __reduce_max_sync(0xFFFFFFFFu, (int)hi));
        const bool near = __all_sync(0xFFFFFFFFu, top - (int)lo <= kNearLog2);
        auto attend = [&](auto far) {
            for (int at = 0; at < n; at += 32) {
                look(at + 32);
                attend_keys<D, far>(
                    st, tile, [&](int i, int h) { return mine[at + 16 * i + 8 * h]; },
                    [&](int i) { load(tile[i].k, next[i], kg); }, [&](int i) { load(tile[i].v, next[i], vg); });
            }
        };
        if (near) {
            attend(std::false_type{});
        } else {
            st.far = exp2f((float)(kNearLog2 - top));
            attend(std::true_type{});
        }
    }
    sum_weights<D>(st);
    const size_t head = (size_t)r * a.Hq + (size_t)g * G;
    write_pair<D>(st, G, a.out + head * D, a.lse != nullptr ? a.lse + head : nullptr, lane);
}

// How many warps share a pair, and in how many CTAs.  Few pairs: as many CTAs
// as still run all at once, each on an SM that gathers for itself; warps in
// powers of two, which divide most budgets' steps.  Measured with k = 2048, 4
// groups of 128 dims, rows read from HBM: 4 rows (16 pairs) 8 CTAs of 4 warps
// 9.1 us, 8 of 8, of which 16 clusters do not fit, 14.3; 20 rows 4 CTAs of 4
// 18.6, of 6 23.8; 28 rows one CTA of 8 20.2, 2 of 6 22.4; 64 rows one of 4
// 39.6, one of 6 39.7, one of 8 40.4; 200 rows one of 4 100, one of 2 115.
// Many pairs: one warp each, and no join.  Its CTAs of four pairs then take the
// device by 1776 pairs at a time and about 3.3 times as long as 444 CTAs of one
// pair and four warps, so that what counts is which of the two ends evenly: 460
// rows in L2 106 us with four warps and 125 with one, 444 rows 99 and 84.
// Budgets below 1024 keep to one round of warps when they can: 148 rows with k =
// 512 in L2, 3 warps 14 us, 4 warps 17.
struct Split {
    int warps, ctas;
};
Split split_of(int64_t pairs, int k) {
    // 12 warps to an SM: what 168 registers allow with 128 dims (with 64 dims the
    // one-warp rows have 16; what is measured above is of 128)
    constexpr int kSms = 148, kSmWarps = 12;
    const int steps = (k + 31) / 32;
    auto rounds = [&](int64_t at_once) { return (pairs + at_once - 1) / at_once; };
    Split s{4, 1};
    if (pairs <= 12) s = {8, 8};
    else if (pairs <= 48) s = {4, 8};
    else if (pairs <= 96) s = {4, 4};
    else if (pairs <= kSms) s = {8, 1};
    else if (pairs > kSms * kSmWarps / 4 && steps < 32) s = {(int)(pairs < kSms * kSmWarps ? kSms * kSmWarps / pairs : 1), 1};
    else if (33 * rounds(kSms * kSmWarps) <= 10 * rounds(kSms * kSmWarps / 4)) s = {1, 1};
    while (s.ctas > 1 && s.warps * s.ctas > steps) s.ctas /= 2;
    if (s.warps > steps) s.warps = steps;
    return s;
}

template <int D>
cudaError_t launch(const Kv8Args &a, cudaStream_t stream) {
    const int64_t pairs = (int64_t)a.n_rows * a.Hkv;
    const Split sp = split_of(pairs, a.k);
    int groups = a.Hkv < kMaxGroups ? a.Hkv : kMaxGroups;
    while (a.Hkv % groups != 0) --groups;
    if (sp.warps * sp.ctas == 1 && groups > 1) {
        const int block = a.k < kBlockKeys ? (a.k + 31) / 32 * 32 : kBlockKeys;
        const size_t smem = (block + 32) * sizeof(int) + block * groups * sizeof(KeyScales);
        static_assert((kBlockKeys + 32) * sizeof(int) + kBlockKeys * kMaxGroups * sizeof(KeyScales) <= 48 << 10, "as below");
        return EarlyLaunch((unsigned)(pairs / groups), groups * 32, smem, stream)(sparse_kv8_rows_kernel<D>, a, block);
    }
    const size_t smem = Join<D>::bytes(sp.warps, sp.ctas, a.Hq / a.Hkv);
    static_assert(kMaxWarps * (Join<D>::kWarp + 16) * sizeof(float) + 8 * (D / 2 + 8 + kMaxCluster) * sizeof(float2) <= 48 << 10,
                  "within the default limit of dynamic shared memory");
    // a cluster only where it is needed: an SM holds 8 CTAs of a cluster launch,
    // even of clusters of one, but 12 one-warp CTAs of a plain one
    return EarlyLaunch((unsigned)(pairs * sp.ctas), sp.warps * 32, smem, stream,
                       sp.ctas > 1 ? sp.ctas : 0)(sparse_kv8_kernel<D>, a);
}

}  // namespace

cudaError_t launch_sparse_kv8(const uint16_t *q, const uint8_t *k_cache8, const uint8_t *v_cache8,
                              const uint8_t *kv_exp, int scale_block, const int32_t *block_table, int max_pages,
                              int num_pages, const int32_t *seq_lens, const int32_t *idx, const int32_t *cu, int nseq,
                              int row_begin, int n_rows, int Hq, int Hkv, int D, int k, float sm_scale, uint16_t *out,
                              float *lse, cudaStream_t stream) {
    if (n_rows == 0) return cudaSuccess;
    const int shift = scale_block == 16 ? 4 : (scale_block == 32 ? 5 : 6);
    const Kv8Args a{q, k_cache8, v_cache8, reinterpret_cast<const uint16_t *>(kv_exp), block_table, seq_lens, idx, cu,
                    max_pages, num_pages, nseq, row_begin, n_rows, Hq, Hkv, k, shift, sm_scale * kLog2e, out, lse};
    return D == 64 ? launch<64>(a, stream) : launch<128>(a, stream);
}

}  // namespace dsa
