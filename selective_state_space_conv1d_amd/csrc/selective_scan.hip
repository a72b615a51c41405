// The per-channel selective scan: every channel d has its own decay row A[d, :] and its own step dt
// ("Mamba 与 Nemotron 系列模型深度调研", "Mamba 架构 / 1. Selective SSM 的直觉": the selective
// recurrence before heads share a decay).  Per batch entry and channel, with g(d) = d / (D/G):
//   h = exp(dt A[d,:]) * h + dt x B[g(d),:];   y = <h, C[g(d),:]> + Dskip[d] x;   out = y silu(z)
//
// Layout.  A workgroup owns 64 consecutive channels of one group (lane = channel) and all N states,
// its W waves S = N / W states each, in registers.  B and C of a token are then the same for a whole
// wave: they come in scalar registers and cost the vector pipe nothing, and the sum over a wave's
// states stays in the lane; only the W partial sums of y cross waves, through LDS.  The work of a
// token and channel that does not depend on the state (loads, softplus, gate) is done once, by the
// thread that owns (token, channel) in the tile of 16 tokens, before and after the scan of the tile.
//
// Bound: one exp and about four vector operations for each state of each token and channel; no
// product shares an operand across channels, so the matrix pipe does not apply.
#include "selective_device.h"

namespace ssd {

constexpr int kSelTile = 16;   // tokens staged at a time

template <typename T, typename TY, int S, int W>
__global__ __launch_bounds__(64 * W) void selective_scan_kernel(SelScanArgs a) {
    constexpr int N = S * W, TPT = kSelTile / W;   // tokens of a tile that one thread stages
    __shared__ float2 st[2][kSelTile][64];         // dt, dt * x
    __shared__ float part[2][W][kSelTile][64];
    const SelBlock k = sel_block(blockIdx.x, a.channels, a.ngroups);
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = k.c0 + lane;
    const bool ok = c < k.cend;
    const int cs = ok ? c : k.c0;                  // lanes past the group read its first channel, store nothing
    const int64_t L = a.seqlen, D = a.channels;
    const T* xp = static_cast<const T*>(a.x) + k.b * L * a.x_row_stride + cs;
    const T* zp = a.z ? static_cast<const T*>(a.z) + k.b * L * a.z_row_stride + cs : nullptr;
    const T* dp = static_cast<const T*>(a.dt) + k.b * L * D + cs;
    const T* Bp = static_cast<const T*>(a.B) + k.b * L * a.bc_row_stride + k.g * N + w * S;
    const T* Cp = static_cast<const T*>(a.C) + k.b * L * a.bc_row_stride + k.g * N + w * S;
    TY* yp = static_cast<TY*>(a.y) + k.b * L * D + cs;
    const SelDt dtp{a.dtp.bias ? a.dtp.bias[cs] : 0.f, a.dtp.lo, a.dtp.hi, a.dtp.softplus};
    const float Dv = a.D ? a.D[cs] : 0.f;
    float A2[S], h[S];
    const int64_t so = (k.b * D + cs) * N + w * S;
#pragma unroll
    for (int s = 0; s < S; ++s) {
        A2[s] = a.A[static_cast<int64_t>(cs) * N + w * S + s] * kLog2e;
        h[s] = a.init_state ? a.init_state[so + s] : 0.f;
    }
    float xr[TPT], zr[TPT], dr[TPT];
    auto load = [&](int64_t t0) {
#pragma unroll
        for (int i = 0; i < TPT; ++i) {
            const int64_t t = t0 + w + W * i;
            const bool in = t < L;
            const int64_t tt = in ? t : L - 1;
            xr[i] = static_cast<float>(xp[tt * a.x_row_stride]);
            dr[i] = static_cast<float>(dp[tt * D]);
            zr[i] = zp ? static_cast<float>(zp[tt * a.z_row_stride]) : 0.f;
        }
    };
    if (L > 0) load(0);
    int buf = 0;
    for (int64_t t0 = 0; t0 < L; t0 += kSelTile, buf ^= 1) {
        float xk[TPT], zk[TPT];
#pragma unroll
        for (int i = 0; i < TPT; ++i) {
            const int t = w + W * i;
            const float dt = t0 + t < L ? sel_dt(dr[i], dtp) : 0.f;   // past the end: the state stands still
            const float x = t0 + t < L ? xr[i] : 0.f;
            st[buf][t][lane] = make_float2(dt, dt * x);
            xk[i] = x;
            zk[i] = zr[i];
        }
        __syncthreads();
        if (t0 + kSelTile < L) load(t0 + kSelTile);
#pragma unroll 4
        for (int t = 0; t < kSelTile; ++t) {
            const int64_t row = t0 + t < L ? t0 + t : L - 1;
            float Bv[S], Cv[S];
            load_uniform<T, S>(Bp + row * a.bc_row_stride, Bv);
            load_uniform<T, S>(Cp + row * a.bc_row_stride, Cv);
            const float2 d = st[buf][t][lane];
            float y = 0.f;
#pragma unroll
            for (int s = 0; s < S; ++s) {
                const float e = __builtin_amdgcn_exp2f(d.x * A2[s]);
                h[s] = fmaf(e, h[s], d.y * Bv[s]);
                y = fmaf(h[s], Cv[s], y);
            }
            part[buf][w][t][lane] = y;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < TPT; ++i) {
            const int t = w + W * i;
            float y = Dv * xk[i];
#pragma unroll
            for (int v = 0; v < W; ++v) y += part[buf][v][t][lane];
            if (zp) y *= silu_f(zk[i]);
            if (ok && t0 + t < L) yp[(t0 + t) * D] = static_cast<TY>(y);
        }
    }
    if (a.final_state && ok) {
#pragma unroll
        for (int s = 0; s < S; ++s) a.final_state[so + s] = h[s];
    }
}

template <typename T, typename TY>
static hipError_t scan_t(const SelScanArgs& a, hipStream_t s) {
    const int64_t blocks = a.batch * a.ngroups * ((a.channels / a.ngroups + 63) / 64);
    const dim3 grid(static_cast<uint32_t>(blocks));
    switch (a.d_state) {
        case 16: hipLaunchKernelGGL((selective_scan_kernel<T, TY, 4, 4>), grid, dim3(256), 0, s, a); break;
        case 32: hipLaunchKernelGGL((selective_scan_kernel<T, TY, 8, 4>), grid, dim3(256), 0, s, a); break;
        case 64: hipLaunchKernelGGL((selective_scan_kernel<T, TY, 16, 4>), grid, dim3(256), 0, s, a); break;
        case 128: hipLaunchKernelGGL((selective_scan_kernel<T, TY, 16, 8>), grid, dim3(512), 0, s, a); break;
        default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

size_t selective_scan_workspace_bytes(int64_t, int64_t, int, int, int) { return 0; }

hipError_t launch_selective_scan(const SelScanArgs& a, Dt act, Dt ydt, void*, hipStream_t s) {
    if (a.batch == 0) return hipSuccess;
    if (act == Dt::BF16) return ydt == Dt::BF16 ? scan_t<bf16, bf16>(a, s) : scan_t<bf16, float>(a, s);
    return ydt == Dt::BF16 ? scan_t<float, bf16>(a, s) : scan_t<float, float>(a, s);
}

// One token per batch entry.  The state is read once and written once: an HBM stream.  A thread owns
// four states of a channel and walks batch entries with A, the skip weight and dt's bias in registers,
// kUpdInFlight entries' loads issued together; the N / 4 lanes of a channel add up y by lane moves.
constexpr int kSelUpdThreads = 256;
constexpr int kUpdInFlight = 4;

template <typename T, typename TY, int N>
__global__ __launch_bounds__(kSelUpdThreads) void selective_update_kernel(SelUpdateArgs a) {
    constexpr int Q = N / 4;
    const int64_t e = static_cast<int64_t>(blockIdx.x) * kSelUpdThreads + threadIdx.x;
    const int64_t D = a.channels;
    const bool ok = e < D * Q;
    const int64_t c = ok ? e / Q : 0;
    const int q = static_cast<int>(ok ? e % Q : 0);
    const int g = static_cast<int>(c / (D / a.ngroups));
    const int64_t bo = static_cast<int64_t>(g) * N + 4 * q;
    const SelDt dtp{a.dtp.bias ? a.dtp.bias[c] : 0.f, a.dtp.lo, a.dtp.hi, a.dtp.softplus};
    const float Dv = a.D ? a.D[c] : 0.f;
    const f32x4 A4 = *reinterpret_cast<const f32x4*>(a.A + c * N + 4 * q);
    const T* x = static_cast<const T*>(a.x);
    const T* z = static_cast<const T*>(a.z);
    const T* dt = static_cast<const T*>(a.dt);
    const T* B = static_cast<const T*>(a.B);
    const T* C = static_cast<const T*>(a.C);
    const int64_t b1 = (static_cast<int64_t>(blockIdx.y) + 1) * a.per_block;
    const int64_t bend = b1 < a.batch ? b1 : a.batch;
    for (int64_t b0 = static_cast<int64_t>(blockIdx.y) * a.per_block; b0 < bend; b0 += kUpdInFlight) {
        f32x4 h[kUpdInFlight];
        int64_t slot[kUpdInFlight];
#pragma unroll
        for (int i = 0; i < kUpdInFlight; ++i) {
            const int64_t b = b0 + i < bend ? b0 + i : bend - 1;
            slot[i] = seq_slot(a.slot_idx, b, a.nslots);
            h[i] = slot[i] >= 0 ? __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(
                                      a.state + (slot[i] * D + c) * N + 4 * q))
                                : f32x4{0.f, 0.f, 0.f, 0.f};
        }
#pragma unroll
        for (int i = 0; i < kUpdInFlight; ++i) {
            const bool in = ok && b0 + i < bend;
            const int64_t b = b0 + i < bend ? b0 + i : bend - 1;
            const float xv = static_cast<float>(x[b * a.x_row_stride + c]);
            const float dv = sel_dt(static_cast<float>(dt[b * D + c]), dtp);
            const float dx = dv * xv, d2 = dv * kLog2e;
            float y = 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float Bv = static_cast<float>(B[b * a.bc_row_stride + bo + k]);
                const float Cv = static_cast<float>(C[b * a.bc_row_stride + bo + k]);
                h[i][k] = fmaf(__builtin_amdgcn_exp2f(d2 * A4[k]), h[i][k], dx * Bv);
                y = fmaf(h[i][k], Cv, y);
            }
            y = group_sum_last<Q>(y);   // every lane takes part: those past the end hold channel 0's values
            if (in && q == Q - 1) {
                y = fmaf(Dv, xv, y);
                if (z) y *= silu_f(static_cast<float>(z[b * a.z_row_stride + c]));
                static_cast<TY*>(a.y)[b * D + c] = static_cast<TY>(y);
            }
            if (in && slot[i] >= 0)
                __builtin_nontemporal_store(h[i], reinterpret_cast<f32x4*>(a.state_out + (slot[i] * D + c) * N + 4 * q));
        }
    }
}

template <typename T, typename TY, int N>
static hipError_t update_n(SelUpdateArgs a, hipStream_t s) {
    const int64_t xb = (static_cast<int64_t>(a.channels) * (N / 4) + kSelUpdThreads - 1) / kSelUpdThreads;
    // batch entries per workgroup: enough workgroups to fill the chip a few times over, and no more
    // than 65535 rows of them
    int64_t per = kUpdInFlight;
    while (per < a.batch && (xb * ((a.batch + per - 1) / per) > 4096 || (a.batch + per - 1) / per > 65535)) per *= 2;
    a.per_block = per;
    hipLaunchKernelGGL((selective_update_kernel<T, TY, N>), dim3(static_cast<uint32_t>(xb), static_cast<uint32_t>((a.batch + per - 1) / per)),
                       dim3(kSelUpdThreads), 0, s, a);
    return hipGetLastError();
}

template <typename T, typename TY>
static hipError_t update_t(const SelUpdateArgs& a, hipStream_t s) {
    switch (a.d_state) {
        case 16: return update_n<T, TY, 16>(a, s);
        case 32: return update_n<T, TY, 32>(a, s);
        case 64: return update_n<T, TY, 64>(a, s);
        case 128: return update_n<T, TY, 128>(a, s);
        default: return hipErrorInvalidValue;
    }
}

hipError_t launch_selective_update(const SelUpdateArgs& a, Dt act, Dt ydt, hipStream_t s) {
    if (a.batch == 0) return hipSuccess;
    if (act == Dt::BF16) return ydt == Dt::BF16 ? update_t<bf16, bf16>(a, s) : update_t<bf16, float>(a, s);
    return ydt == Dt::BF16 ? update_t<float, bf16>(a, s) : update_t<float, float>(a, s);
}

}  // namespace ssd
