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
// Work unit: one CTA per (block of tokens, head, K or V); the block's new
// values stay in registers between the maximum and the conversion, so K and V
// are read once.  One more row of CTAs copies the indexer's keys.  Bound by
// HBM for prompts (2 bytes in, 1 byte out per value), by latency for single
// tokens.
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
    int nseq, n_tokens, max_pages, num_pages, Hkv, dI, block;
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

template <int D, int T, int kMaxNew>
__global__ void __launch_bounds__(T) kv8_append_kernel(const __grid_constant__ AppendArgs a) {
    constexpr int VPT = D / 8;                      // 16-byte pieces of a new token's row
    constexpr int kMaxVec = (kMaxNew * VPT + T - 1) / T;
    __shared__ uint32_t red[T / 32];
    // the unit's sequence and its part of it: block j of those that the
    // sequence's new tokens touch.  Sequence b has the units from
    // cu[b] / block + 2 b on, at least as many as the blocks it touches.
    // The unit's CTAs (heads, K and V, the indexer's keys) are neighbours:
    // together they read whole rows.
    const int per = 2 * a.Hkv + (a.k8 != nullptr ? 1 : 0), part = blockIdx.x % per;
    int b, t0, pos0, n_new, j;
    if (a.cu == nullptr) {
        b = blockIdx.x / per;
        t0 = b;
        n_new = 1;
        j = 0;
    } else {
        const int u = blockIdx.x / per;
        b = warp_find_seq(a.nseq, u, [&](int i) { return __ldg(a.cu + i) / a.block + 2 * i; });
        t0 = __ldg(a.cu + b);
        n_new = __ldg(a.cu + b + 1) - t0;
        j = u - (t0 / a.block + 2 * b);
        if (t0 < 0 || n_new <= 0 || (int64_t)t0 + n_new > a.n_tokens) return;
    }
    pos0 = __ldg(a.seq_lens + b) - n_new;           // the first new token's position
    if (pos0 < 0) return;
    const int blk = pos0 / a.block + j;             // the block within the sequence
    const int64_t start = (int64_t)blk * a.block;
    const int lo = (int)max(start, (int64_t)pos0);
    const int hi = (int)min(start + a.block, (int64_t)pos0 + n_new);
    if (lo >= hi || start / kPage >= a.max_pages) return;
    const int m = hi - lo, m_old = lo - (int)start;
    const int64_t tok = t0 + (lo - pos0);           // the first of them among the new tokens
    // the values are asked for before their page is known
    const int g = part >> 1, which = part & 1;
    const bool keys = part == 2 * a.Hkv;
    uint4 x[kMaxVec];
    uint32_t mx = 0;
#pragma unroll
    for (int i = 0; i < kMaxVec; ++i) {
        const int v = threadIdx.x + i * T;
        x[i] = make_uint4(0, 0, 0, 0);
        if (v < m * VPT && !keys)
            x[i] = __ldg(reinterpret_cast<const uint4 *>(a.src[which] + (tok + v / VPT) * a.ld[which] + (size_t)g * D) +
                         v % VPT);
    }
    const int page = __ldg(a.block_table + (size_t)b * a.max_pages + start / kPage);
    if (page < 0 || page >= a.num_pages) return;
    const int64_t row = (int64_t)page * kPage + lo % kPage;

    if (keys) {                                     // the indexer's keys
        const int n16 = a.dI / 16;
        const uint4 *src = reinterpret_cast<const uint4 *>(a.k8 + tok * a.dI);
        uint4 *dst = reinterpret_cast<uint4 *>(a.k8_cache + row * a.dI);
        for (int i = threadIdx.x; i < m * n16; i += T) dst[i] = __ldg(src + i);
        for (int i = threadIdx.x; i < m; i += T) a.k_scale_cache[row + i] = __ldg(a.k_scale + tok + i);
        return;
    }
    uint8_t *exp_at = a.exps + (((size_t)page * (kPage / a.block) + (start % kPage) / a.block) * a.Hkv + g) * 2 + which;
    const int e_old = m_old > 0 ? *exp_at : kKv8ExpMin;
#pragma unroll
    for (int i = 0; i < kMaxVec; ++i) {
        mx = abs_max_bf16x2(mx, x[i].x);
        mx = abs_max_bf16x2(mx, x[i].y);
        mx = abs_max_bf16x2(mx, x[i].z);
        mx = abs_max_bf16x2(mx, x[i].w);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = abs_max_bf16x2(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
    if (lane_id() == 0) red[threadIdx.x >> 5] = mx;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < T / 32; ++w) mx = abs_max_bf16x2(mx, red[w]);
    const float amax = fmaxf(__uint_as_float(mx << 16), __uint_as_float(mx & 0xFFFF0000u));
    const int e = max(e_old, min(max(exp_byte_for(amax), kKv8ExpMin), kKv8ExpMax));
    const float inv = exp_byte_scale(254 - e);
    uint8_t *dst = a.dst[which] + (row * a.Hkv + g) * D;
    const size_t stride = (size_t)a.Hkv * D;
#pragma unroll
    for (int i = 0; i < kMaxVec; ++i) {
        const int v = threadIdx.x + i * T;
        if (v < m * VPT) {
            uint32_t out[2];
            const uint32_t in[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint16_t p0 = f32x2_to_e4m3x2(__uint_as_float(in[2 * h] << 16) * inv,
                                                    __uint_as_float(in[2 * h] & 0xFFFF0000u) * inv);
                const uint16_t p1 = f32x2_to_e4m3x2(__uint_as_float(in[2 * h + 1] << 16) * inv,
                                                    __uint_as_float(in[2 * h + 1] & 0xFFFF0000u) * inv);
                out[h] = (uint32_t)p0 | (uint32_t)p1 << 16;
            }
            *reinterpret_cast<uint2 *>(dst + (v / VPT) * stride + (v % VPT) * 8) = make_uint2(out[0], out[1]);
        }
    }
    if (m_old > 0 && e > e_old) {                   // the older tokens' bytes to the new scale
        const int down = e_old - e;
        const float f = down > -127 ? exp_byte_scale(127 + down) : 0.f;
        uint8_t *old = dst - (size_t)m_old * stride;
        for (int v = threadIdx.x; v < m_old * (D / 16); v += T) {
            uint4 *p = reinterpret_cast<uint4 *>(old + (v / (D / 16)) * stride) + v % (D / 16);
            uint4 w = *p;
            uint32_t *ws = reinterpret_cast<uint32_t *>(&w);
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                const float2 lo2 = f16x2_to_float2(e4m3x2_to_f16x2((uint16_t)(ws[h] & 0xFFFFu)));
                const float2 hi2 = f16x2_to_float2(e4m3x2_to_f16x2((uint16_t)(ws[h] >> 16)));
                ws[h] = (uint32_t)f32x2_to_e4m3x2(lo2.x * f, lo2.y * f) |
                        (uint32_t)f32x2_to_e4m3x2(hi2.x * f, hi2.y * f) << 16;
            }
            *p = w;
        }
    }
    if (threadIdx.x == 0 && (m_old == 0 || e != e_old)) *exp_at = (uint8_t)e;
}

// kMaxNew: the most new tokens of one block
template <int D, int T, int kMaxNew>
cudaError_t launch(const AppendArgs &a, unsigned units, cudaStream_t stream) {
    kv8_append_kernel<D, T, kMaxNew><<<units * (2 * a.Hkv + (a.k8 != nullptr ? 1 : 0)), T, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv8_append(const uint16_t *K, int64_t ld_k, const uint16_t *V, int64_t ld_v, const uint8_t *k8,
                              const float *k_scale, const int32_t *cu, int nseq, int n_tokens,
                              const int32_t *seq_lens, const int32_t *block_table, int max_pages, int num_pages,
                              int Hkv, int D, int dI, int scale_block, uint8_t *k_cache8, uint8_t *v_cache8,
                              uint8_t *kv_exp, uint8_t *k8_cache, float *k_scale_cache, cudaStream_t stream) {
    if (nseq == 0 || n_tokens == 0) return cudaSuccess;
    const AppendArgs a{{K, V}, {ld_k, ld_v}, k8, k_scale, cu, seq_lens, block_table, nseq, n_tokens, max_pages,
                       num_pages, Hkv, dI, scale_block, {k_cache8, v_cache8}, kv_exp, k8_cache, k_scale_cache};
    // a single token is 8 or 16 pieces of 16 bytes: two warps; a block of a
    // prompt is up to 1024 of them: eight warps with four pieces a thread
    if (cu == nullptr) return D == 64 ? launch<64, 64, 1>(a, nseq, stream) : launch<128, 64, 1>(a, nseq, stream);
    const unsigned units = (unsigned)(n_tokens / scale_block + 2 * nseq);
    return D == 64 ? launch<64, 256, kPage>(a, units, stream) : launch<128, 256, kPage>(a, units, stream);
}

}  // namespace dsa
