// kv8_append.cu -- appending K and V tokens to the 8-bit paged cache.
//
// For a block of tokens and a head, with x the block's new tokens:
//     e   = the least exponent with max |x| <= 448 * 2^e, at least the
//           block's exponent when older tokens are in it;
//     new bytes  = e4m3(x * 2^-e)
//     old bytes  = e4m3(e4m3(byte) * 2^(e_old - e))   where e > e_old.
// The scale never falls, so a block's bytes are rewritten only when a token
// outgrows all before it, and the rewriting rounds only values that become
// subnormal in e4m3 (the scale is a power of two).
//
// Work unit: one CTA per (block of tokens, head), for K and V; the block's new
// values stay in registers between the maximum and the conversion, so K and V
// are read once.  One more CTA per block copies the indexer's keys.  Bound by
// HBM for prompts (2 bytes in, 1 byte out per value): a 32K prompt of 4 heads
// of 128 takes 20.4 us, 5.1 TB/s, against 16 us for a plain copy of as many
// bytes.  (K and V in CTAs of their own, with divisions in place of shifts,
// took 27.6 us: more instructions than the loads could hide.)  Single tokens
// are bound by the chain of loads length, page, scale: 1.8 us for 32 sequences.
#include "kernels.h"
#include "kv8.cuh"

namespace dsa {

namespace {

struct AppendArgs {
    const uint16_t *src[2];
    int64_t ld[2];
    const uint8_t *k8;
    const float *k_scale;
    const int32_t *cu, *seq_lens, *block_table;
    int nseq, n_tokens, max_pages, num_pages, Hkv, dI, shift;   // 2^shift tokens to a block
    uint8_t *dst[2];
    uint8_t *exps;
    uint8_t *k8_cache;
    float *k_scale_cache;
};

__device__ __forceinline__ uint32_t abs_max_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b & 0x7FFF7FFFu));
    return r;
}

// Eight bf16 values -> e4m3 of value * inv.
__device__ __forceinline__ uint2 to_e4m3x8(const uint4 &x, float inv) {
    const uint32_t in[4] = {x.x, x.y, x.z, x.w};
    uint16_t out[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        out[i] = f32x2_to_e4m3x2(__uint_as_float(in[i] << 16) * inv, __uint_as_float(in[i] & 0xFFFF0000u) * inv);
    return make_uint2((uint32_t)out[0] | (uint32_t)out[1] << 16, (uint32_t)out[2] | (uint32_t)out[3] << 16);
}

// Sixteen e4m3 bytes times f (a power of two), rounded again.
__device__ __forceinline__ uint4 rescale_e4m3x16(uint4 w, float f) {
    uint32_t *ws = reinterpret_cast<uint32_t *>(&w);
#pragma unroll
    for (int h = 0; h < 4; ++h) {
        const float2 lo = f16x2_to_float2(e4m3x2_to_f16x2((uint16_t)(ws[h] & 0xFFFFu)));
        const float2 hi = f16x2_to_float2(e4m3x2_to_f16x2((uint16_t)(ws[h] >> 16)));
        ws[h] = (uint32_t)f32x2_to_e4m3x2(lo.x * f, lo.y * f) | (uint32_t)f32x2_to_e4m3x2(hi.x * f, hi.y * f) << 16;
    }
    return w;
}

template <int D, int T, int kMaxNew>
__global__ void __launch_bounds__(T) kv8_append_kernel(const __grid_constant__ AppendArgs a) {
    constexpr int VPT = D / 8;                      // 16-byte pieces of a new token's row
    constexpr int kMaxVec = (kMaxNew * VPT + T - 1) / T;
    __shared__ uint32_t red[2][T / 32];
    wait_for_last();
    // The unit's sequence and its part of it: block j of those that the
    // sequence's new tokens touch.  Sequence b has the units from
    // cu[b] / block + 2 b on, at least as many as the blocks it touches.  The
    // unit's CTAs (heads, the indexer's keys) are neighbours: together they
    // read whole rows.
    const unsigned per = a.Hkv + (a.k8 != nullptr ? 1 : 0), u = blockIdx.x / per;
    const int g = blockIdx.x - u * per;
    int b, t0, n_new, j;
    if (a.cu == nullptr) {
        b = t0 = u;
        n_new = 1;
        j = 0;
    } else {
        b = warp_find_seq(a.nseq, u, [&](int i) { return (a.cu[i] >> a.shift) + 2 * i; });
        t0 = a.cu[b];
        n_new = a.cu[b + 1] - t0;
        j = u - ((t0 >> a.shift) + 2 * b);
        if (t0 < 0 || n_new <= 0 || n_new > a.n_tokens - t0 || (unsigned)j > (unsigned)(n_new >> a.shift) + 1) return;
    }
    const int len = a.seq_lens[b];
    if (len <= 0) return;
    const int pos0 = len - n_new;           // the first new token's position; tokens at negative ones have no place
    if (pos0 >= a.max_pages * kPage) return;
    const int start = ((pos0 >> a.shift) + j) * (1 << a.shift);     // the block's first position
    const int lo = max(start, max(pos0, 0)), hi = min(start + (1 << a.shift), len);
    if (lo >= hi || start >= a.max_pages * kPage) return;
    const int m = hi - lo, m_old = lo - start, tok = t0 + (lo - pos0);  // tok: the first among the new tokens
    const bool keys = g == a.Hkv;
    // the values are asked for before their page is known
    uint4 x[2][kMaxVec];
    uint32_t mx[2] = {0, 0};
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        const uint16_t *src = a.src[w] + tok * a.ld[w] + g * D + threadIdx.x % VPT * 8;
        const int64_t step = a.ld[w] * (T / VPT);
        src += threadIdx.x / VPT * a.ld[w];
#pragma unroll
        for (int i = 0; i < kMaxVec; ++i) {
            x[w][i] = make_uint4(0, 0, 0, 0);
            if (!keys && (int)threadIdx.x + i * T < m * VPT) x[w][i] = *reinterpret_cast<const uint4 *>(src);
            src += step;
        }
    }
    const int page = a.block_table[(size_t)b * a.max_pages + start / kPage];
    if (page < 0 || page >= a.num_pages) return;
    const int row = page * kPage + lo % kPage;

    if (keys) {                                     // the indexer's keys
        const int n16 = a.dI / 16;
        const uint4 *src = reinterpret_cast<const uint4 *>(a.k8 + (int64_t)tok * a.dI);
        uint4 *dst = reinterpret_cast<uint4 *>(a.k8_cache + (int64_t)row * a.dI);
        for (int i = threadIdx.x; i < m * n16; i += T) dst[i] = src[i];
        for (int i = threadIdx.x; i < m; i += T) a.k_scale_cache[row + i] = a.k_scale[tok + i];
        return;
    }
    uint8_t *exp_at = a.exps + (((size_t)page * (kPage >> a.shift) + (start % kPage >> a.shift)) * a.Hkv + g) * 2;
    const uint16_t e_both = m_old > 0 ? *reinterpret_cast<const uint16_t *>(exp_at) : kKv8ExpMin | kKv8ExpMin << 8;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
#pragma unroll
        for (int i = 0; i < kMaxVec; ++i) {
            mx[w] = abs_max_bf16x2(mx[w], x[w][i].x);
            mx[w] = abs_max_bf16x2(mx[w], x[w][i].y);
            mx[w] = abs_max_bf16x2(mx[w], x[w][i].z);
            mx[w] = abs_max_bf16x2(mx[w], x[w][i].w);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mx[w] = abs_max_bf16x2(mx[w], __shfl_xor_sync(0xFFFFFFFFu, mx[w], o));
        if (lane_id() == 0) red[w][threadIdx.x >> 5] = mx[w];
    }
    __syncthreads();
    int e_new = 0;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        const int e_old = e_both >> (8 * w) & 0xFF;
#pragma unroll
        for (int i = 0; i < T / 32; ++i) mx[w] = abs_max_bf16x2(mx[w], red[w][i]);
        const float amax = fmaxf(__uint_as_float(mx[w] << 16), __uint_as_float(mx[w] & 0xFFFF0000u));
        const int e = max(e_old, min(max(exp_byte_for(amax), kKv8ExpMin), kKv8ExpMax));
        e_new |= e << (8 * w);
        const float inv = exp_byte_scale(254 - e);
        const int stride = a.Hkv * D;
        uint8_t *dst = a.dst[w] + (int64_t)row * stride + g * D;
        uint8_t *to = dst + threadIdx.x / VPT * stride + threadIdx.x % VPT * 8;
#pragma unroll
        for (int i = 0; i < kMaxVec; ++i) {
            if ((int)threadIdx.x + i * T < m * VPT) *reinterpret_cast<uint2 *>(to) = to_e4m3x8(x[w][i], inv);
            to += T / VPT * stride;
        }
        if (m_old > 0 && e > e_old) {               // the older tokens' bytes to the new scale
            const int down = e_old - e;
            const float f = down > -127 ? exp_byte_scale(127 + down) : 0.f;
            for (int v = threadIdx.x; v < m_old * (D / 16); v += T) {
                uint4 *p = reinterpret_cast<uint4 *>(dst - (m_old - v / (D / 16)) * stride) + v % (D / 16);
                *p = rescale_e4m3x16(*p, f);
            }
        }
    }
    if (threadIdx.x == 0 && (m_old == 0 || e_new != e_both)) *reinterpret_cast<uint16_t *>(exp_at) = (uint16_t)e_new;
}

// kMaxNew: the most new tokens of one block
template <int D, int T, int kMaxNew>
cudaError_t launch(const AppendArgs &a, unsigned units, cudaStream_t stream) {
    return EarlyLaunch(units * (a.Hkv + (a.k8 != nullptr ? 1 : 0)), T, 0, stream)(kv8_append_kernel<D, T, kMaxNew>, a);
}

}  // namespace

cudaError_t launch_kv8_append(const uint16_t *K, int64_t ld_k, const uint16_t *V, int64_t ld_v, const uint8_t *k8,
                              const float *k_scale, const int32_t *cu, int nseq, int n_tokens,
                              const int32_t *seq_lens, const int32_t *block_table, int max_pages, int num_pages,
                              int Hkv, int D, int dI, int scale_block, uint8_t *k_cache8, uint8_t *v_cache8,
                              uint8_t *kv_exp, uint8_t *k8_cache, float *k_scale_cache, cudaStream_t stream) {
    if (nseq == 0 || n_tokens == 0) return cudaSuccess;
    const AppendArgs a{{K, V}, {ld_k, ld_v}, k8, k_scale, cu, seq_lens, block_table, nseq, n_tokens, max_pages,
                       num_pages, Hkv, dI, scale_block == 16 ? 4 : (scale_block == 32 ? 5 : 6), {k_cache8, v_cache8}, kv_exp, k8_cache, k_scale_cache};
    // a single token is 8 or 16 pieces of 16 bytes: two warps; a block of a
    // prompt is up to 1024 of them: eight warps with four pieces a thread
    if (cu == nullptr) return D == 64 ? launch<64, 64, 1>(a, nseq, stream) : launch<128, 64, 1>(a, nseq, stream);
    const unsigned units = (unsigned)(n_tokens / scale_block + 2 * nseq);
    return D == 64 ? launch<64, 256, kPage>(a, units, stream) : launch<128, 256, kPage>(a, units, stream);
}

}  // namespace dsa
