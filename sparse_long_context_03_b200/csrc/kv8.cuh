// kv8.cuh -- device helpers of the 8-bit KV cache.
//
// A cached value is e4m3(byte) * 2^(e - 127): one scale byte e per block of
// tokens (16, 32 or 64 of a page), KV head and K or V.  Powers of two cost
// e4m3 nothing (a float format's relative step does not depend on the scale)
// and make a change of scale exact but for values that become subnormal.
#pragma once

#include "common.cuh"

namespace dsa {

// Scale bytes that the append writes: 2^-40 .. 2^40.  Within that range the
// attention's weights keep their fp32 exponent range (attention_kv8.cu).
constexpr int kKv8ExpMin = 127 - 40;
constexpr int kKv8ExpMax = 127 + 40;

// 2^(e - 127) for e in 1..254.
__device__ __forceinline__ float exp_byte_scale(int e) { return __uint_as_float((uint32_t)e << 23); }

// The least scale byte e with amax <= 448 * 2^(e - 127), unclamped.  448 =
// 1.75 * 2^8: the float's exponent field minus 8, one more where the mantissa
// exceeds 1.75.
__device__ __forceinline__ int exp_byte_for(float amax) {
    return (int)((__float_as_uint(amax) + 0x1FFFFFu) >> 23) - 8;
}

// Two e4m3 bytes -> two halves (exact).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t b) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;\n" : "=r"(r) : "h"(b));
    return r;
}

// Two floats -> two e4m3 bytes (lo in the low byte), nearest even, saturating.
__device__ __forceinline__ uint16_t f32x2_to_e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ float2 f16x2_to_float2(uint32_t h) {
    float lo, hi;
    asm("{\n .reg .f16 a, b;\n mov.b32 {a, b}, %2;\n cvt.f32.f16 %0, a;\n cvt.f32.f16 %1, b;\n}\n"
        : "=f"(lo), "=f"(hi)
        : "r"(h));
    return make_float2(lo, hi);
}

// D[16x8] += A[16x16] * B[16x8], fp16 inputs, fp32 accumulators; with `first`
// (known when compiling) D = A * B.
__device__ __forceinline__ void mma_f16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1, bool first = false) {
    if (first)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
            "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};\n"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
            "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A kernel may be launched to begin while its stream's last one ends (EarlyLaunch
// below), which hides most of a launch: 21.5 us against 24.5 for decoding
// 32 sequences one call after another.  Each of its threads then waits, before
// it touches memory, until the last kernel has ended and its writes are seen;
// and since that kernel may be the one that wrote what this one reads, nothing
// is read through the read-only path (ld.global.nc, __ldg), which is for data
// that no running kernel writes and which no wait holds back.
__device__ __forceinline__ void wait_for_last() { asm volatile("griddepcontrol.wait;\n" ::: "memory"); }
// A call's first kernel lets its second one, launched that way, begin.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory"); }

// A launch that begins early, in clusters of `ctas` if that is not 0.
struct EarlyLaunch {
    cudaLaunchAttribute attr[2] = {};
    cudaLaunchConfig_t cfg{};

    EarlyLaunch(unsigned grid, unsigned threads, size_t smem, cudaStream_t stream, unsigned ctas = 0) {
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = ctas;
        attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
        cfg.gridDim = dim3(grid);
        cfg.blockDim = dim3(threads);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = stream;
        cfg.attrs = attr;
        cfg.numAttrs = ctas > 0 ? 2 : 1;
    }
    EarlyLaunch(const EarlyLaunch &) = delete;
    EarlyLaunch &operator=(const EarlyLaunch &) = delete;

    template <typename... Params, typename... Args>
    cudaError_t operator()(void (*kernel)(Params...), Args... args) const {
        return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
    }
};

// Another CTA's shared memory may be written once that CTA has started: every
// thread arrives early and waits before its first store to it.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.aligned;\n" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.aligned;\n" ::: "memory"); }

// The largest b in [0, nseq) with first(b) <= key, by one warp: each round
// probes 32 places, so that up to 32 sequences take one load latency and
// 1024 two.  first must not decrease; first(0) <= key is taken for granted.
template <typename First>
__device__ __forceinline__ int warp_find_seq(int nseq, int key, First first) {
    const int lane = lane_id();
    int lo = 0, hi = nseq;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        const int at = lo + lane * step;
        const bool le = at < hi && first(at) <= key;
        const int n = __popc(__ballot_sync(0xFFFFFFFFu, le));
        lo += (n > 0 ? n - 1 : 0) * step;
        hi = min(lo + step, hi);
    }
    return lo;
}

}  // namespace dsa
