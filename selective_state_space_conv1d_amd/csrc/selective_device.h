// What the per-channel selective scan's kernels share (forward, gradient, single tokens).
#pragma once
#include <algorithm>
#include <cmath>

#include "ssd_device.h"
#include "ssd_kernels.h"

namespace ssd {

// Decay exponents are kept in base 2.
constexpr float kLog2e = 1.44269504088896340736f;

// A in base 2.  Minus infinity (a channel that forgets everything) becomes the lowest number: where a tile
// ends after the last token dt is 0, and 0 times infinity would not be 0.
__device__ __forceinline__ float base2_rate(float A) {
    const float r = A * kLog2e;
    return r == -__builtin_inff() ? -3.402823466e38f : r;
}

// dt of one (token, channel): + bias, softplus, clamp, as dt_prologue; softplus by the identity
// log1p(e) = e log(u) / (u - 1), u = 1 + e, whose rounding errors cancel (about 3e-7 relative).
struct SelDt {
    float bias, lo, hi;
    int softplus;
};
__device__ __forceinline__ float sel_softplus(float v) {
    const float e = __builtin_amdgcn_exp2f(v * kLog2e);
    const float u = 1.f + e;
    const float l = u == 1.f ? e : e * (__builtin_amdgcn_logf(u) * 0.69314718055994530942f) * __builtin_amdgcn_rcpf(u - 1.f);
    return v > 20.f ? v : l;
}
__device__ __forceinline__ float sel_sigmoid(float v) {
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-v * kLog2e));
}
template <int K>
__device__ __forceinline__ void sel_dts(float (&v)[K], const SelDt& p) {
#pragma unroll
    for (int i = 0; i < K; ++i) v[i] += p.bias;
    if (p.softplus)
#pragma unroll
        for (int i = 0; i < K; ++i) v[i] = sel_softplus(v[i]);
    if (p.lo < p.hi)
#pragma unroll
        for (int i = 0; i < K; ++i) v[i] = fminf(fmaxf(v[i], p.lo), p.hi);
}
__device__ __forceinline__ float sel_dt(float v, const SelDt& p) {
    float a[1] = {v};
    sel_dts(a, p);
    return a[0];
}

// B and C of n consecutive tokens, S consecutive states of each: rows that every lane of a wave reads
// alike.  They are held as loaded, in scalar registers (16 of them where S allows it), and widened by
// scalar shifts.  Rows are 16-byte aligned, `stride` bytes apart; none past row `last` is read (the
// last one repeats).
typedef const uint32_t __attribute__((address_space(4))) ScalarWord;
typedef const char __attribute__((address_space(4))) ScalarByte;
template <typename T, int S>
constexpr int kRowWords = S * static_cast<int>(sizeof(T)) / 4;
template <typename T, int S, int n_ = (kRowWords<T, S> >= 8 ? 1 : 8 / kRowWords<T, S>)>
struct SelRows {
    static constexpr int kWords = kRowWords<T, S>;
    static constexpr int n = n_;
    uint32_t bw[n][kWords], cw[n][kWords];
    template <bool WITH_C>
    __device__ __forceinline__ void load(const char* b, const char* c, uint32_t stride, int first, int last) {
#pragma unroll
        for (int t = 0; t < n; ++t) {
            const uint32_t o = static_cast<uint32_t>(first + t < last ? first + t : last) * stride;
            ScalarWord* p = (ScalarWord*)((ScalarByte*)(uintptr_t)b + o);
            ScalarWord* q = (ScalarWord*)((ScalarByte*)(uintptr_t)c + o);
#pragma unroll
            for (int i = 0; i < kWords; ++i) bw[t][i] = p[i];
            if constexpr (WITH_C)
#pragma unroll
                for (int i = 0; i < kWords; ++i) cw[t][i] = q[i];
        }
    }
    // keeps the values as loaded: widened ones from before are not held on to
    __device__ __forceinline__ void renew() {
#pragma unroll
        for (int t = 0; t < n; ++t)
#pragma unroll
            for (int i = 0; i < kWords; ++i) asm volatile("" : "+s"(bw[t][i]), "+s"(cw[t][i]));
    }
    static __device__ __forceinline__ float value(const uint32_t* w, int s) {
        if constexpr (sizeof(T) == 2) return __uint_as_float(s & 1 ? w[s / 2] & 0xffff0000u : w[s / 2] << 16);
        else return __uint_as_float(w[s]);
    }
    __device__ __forceinline__ float b(int t, int s) const { return value(bw[t], s); }
    __device__ __forceinline__ float c(int t, int s) const { return value(cw[t], s); }
};

// Which channels, and which batch entry, a workgroup has: 64-channel blocks never straddle groups.
struct SelBlock {
    int64_t b;
    int blk, g, c0, cend;
};
__host__ __device__ __forceinline__ int64_t sel_blocks(int D, int G) { return static_cast<int64_t>(G) * ((D / G + 63) / 64); }
__device__ __forceinline__ SelBlock sel_block(int64_t id, int D, int G) {
    const int cpg = D / G, per = (cpg + 63) / 64, nblk = per * G;
    SelBlock r;
    r.b = id / nblk;
    r.blk = static_cast<int>(id - r.b * nblk);
    r.g = r.blk / per;
    r.c0 = r.g * cpg + (r.blk - r.g * per) * 64;
    r.cend = (r.g + 1) * cpg;
    return r;
}

// Chunks that a sequence of L tokens is cut into at most: 32 tokens or more each, and no more than sqrt(L) of
// them, since a chunk's first state is joined from all before it.  One sequence, bf16, 16 states: 131072 x
// 64 channels 179 us (637 without the root), 16384 x 128 63 (129; with half as many 74); its gradient 598
// and 193 (587 and 391).
inline int64_t most_chunks(int64_t L) {
    return std::max<int64_t>(1, std::min<int64_t>(L / 32, static_cast<int64_t>(std::sqrt(static_cast<double>(L)))));
}

// v <- exp2(sum_k A2) v + end_k over `count` chunks k, `step` apart from `first` on (step may be negative):
// sums + k ss and ends + k es + s D hold a chunk's sum of dt and its S states.  Four chunks are loaded
// at a time: one after the other, their latencies would be most of a short chunk's time.
template <int S>
__device__ __forceinline__ void join_chunks(float (&v)[S], const float (&A2)[S], const float* sums, const float* ends, int first,
                                            int count, int step, int64_t ss, int64_t es, int64_t D) {
    for (int k = 0; k < count; k += 4) {
        float sum[4], end[4][S];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t c = first + step * (k + i < count ? k + i : count - 1);
            sum[i] = sums[c * ss];
#pragma unroll
            for (int s = 0; s < S; ++s) end[i][s] = ends[c * es + s * D];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (k + i < count)
#pragma unroll
                for (int s = 0; s < S; ++s) v[s] = fmaf(__builtin_amdgcn_exp2f(sum[i] * A2[s]), v[s], end[i][s]);
    }
}

}  // namespace ssd
