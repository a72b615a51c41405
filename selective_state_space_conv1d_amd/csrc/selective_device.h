// What the per-channel selective scan's kernels share (forward, gradient, single tokens).
#pragma once
#include "ssd_device.h"
#include "ssd_kernels.h"

namespace ssd {

// Decay exponents are kept in base 2.
constexpr float kLog2e = 1.44269504088896340736f;

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
__device__ __forceinline__ float sel_dt(float v, const SelDt& p) {
    v += p.bias;
    if (p.softplus) v = sel_softplus(v);
    if (p.lo < p.hi) v = fminf(fmaxf(v, p.lo), p.hi);
    return v;
}

// S consecutive values of a row that every lane of the wave reads: scalar loads (the row is 16-byte
// aligned and S >= 4), widened by scalar shifts.
typedef const uint32_t __attribute__((address_space(4))) ScalarWord;
template <typename T, int S>
__device__ __forceinline__ void load_uniform(const T* p, float (&o)[S]) {
    ScalarWord* q = (ScalarWord*)(uintptr_t)p;
    if constexpr (Vec16<T>::n == 8) {
#pragma unroll
        for (int i = 0; i < S / 2; ++i) {
            const uint32_t v = q[i];
            o[2 * i] = __uint_as_float(v << 16);
            o[2 * i + 1] = __uint_as_float(v & 0xffff0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < S; ++i) o[i] = __uint_as_float(q[i]);
    }
}

// Which channels, and which batch entry, a workgroup has: 64-channel blocks never straddle groups.
struct SelBlock {
    int64_t b;
    int blk, g, c0, cend;
};
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

}  // namespace ssd
