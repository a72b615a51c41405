// Gradient of the per-channel selective scan (selective_scan.hip has the forward and its layout).
// With dy = dout silu(z) and g_t the gradient of the state after token t:
//   g_t = C_t dy_t + a_{t+1} g_{t+1},   a_t = exp(dt_t A),  q_t = a_t h_{t-1},  h_t = q_t + dt_t x_t B_t
//   dC_t = sum_d dy h     dB_t = sum_d g dt x      dx = Dskip dy + dt <g, B>      dDskip = sum dy x
//   ddt = <g q, A> + x <g, B>                      dA = sum_t dt g q              dinit = a_1 g_1
//   dz = dout y silu'(z), and through the dt prologue: ddt_raw = ddt sigmoid(dt_raw + bias) (0 where clamped)
//
// Three launches.  (1) states: the forward recurrence alone, which leaves the state at the start of
// every tile of T tokens in the workspace.  (2) gradients: tiles from last to first; each tile's a and q
// are recomputed into registers (T x S = 64 of each) on the way forward and used on the way back.
// (3) sums: partial sums to dA, dDskip, ddt_bias, dB and dC, in a fixed order, so results do not
// depend on scheduling.
//
// The layout is the forward's: lane = channel, wave = S of the N states.  Sums over states stay in the
// lane; sums over channels (dB, dC: one value of each per token and state from 64 lanes) would cost
// more vector operations than everything else, so the matrix pipe takes them: with the values as the
// 16x4 operand and a one-hot 4x16 operand, v_mfma_f32_16x16x4_f32 adds lanes 16 apart into the column
// the one-hot names, in fp32; a tile's 64 (token, state) pairs fill four 16x16 accumulators, whose rows
// are then added by 3 additions and 2 lane exchanges.  (A product that is not finite makes the other
// tokens of its tile and column group non-finite too: 0 times infinity.)
#include "selective_device.h"

namespace ssd {

template <typename T, int S>
__device__ __forceinline__ void load_uniform(const T* p, float (&o)[S]) {
    ScalarWord* q = (ScalarWord*)(uintptr_t)p;
    if constexpr (sizeof(T) == 2) {
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

template <int S>
struct SelTile {
    static constexpr int T = 64 / S;   // tokens per tile: 64 (token, state) pairs a lane
};

// Offsets in floats of the workspace's parts.
struct SelBwdLayout {
    int64_t ckpt, dA, dD, dbias, dBC, total;
    int64_t tiles, blocks;
};
static SelBwdLayout bwd_layout(int64_t batch, int64_t L, int64_t D, int64_t G, int64_t N) {
    const int64_t S = N == 16 ? 4 : N == 32 ? 8 : N == 64 ? 8 : 16, T = 64 / S;
    SelBwdLayout l;
    l.tiles = (L + T - 1) / T;
    l.blocks = G * ((D / G + 63) / 64);
    int64_t at = 0;
    auto take = [&](int64_t n) {
        const int64_t o = at;
        at += (n + 3) & ~INT64_C(3);
        return o;
    };
    l.ckpt = take(batch * l.tiles * N * D);
    l.dA = take(batch * N * D);
    l.dD = take(batch * D);
    l.dbias = take(batch * D);
    l.dBC = take(l.blocks * batch * L * 2 * N);
    l.total = at;
    return l;
}

template <typename T_, int S, int W>
__global__ __launch_bounds__(64 * W) void selective_states_kernel(SelBwdArgs a, float* ckpt, int64_t tiles) {
    constexpr int N = S * W, T = SelTile<S>::T, TPT = (T + W - 1) / W;
    __shared__ float2 st[2][T][64];
    const SelBlock k = sel_block(blockIdx.x, a.channels, a.ngroups);
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = k.c0 + lane;
    const bool ok = c < k.cend;
    const int cs = ok ? c : k.c0;
    const int64_t L = a.seqlen, D = a.channels;
    const T_* xp = static_cast<const T_*>(a.x) + k.b * L * a.x_row_stride + cs;
    const T_* dp = static_cast<const T_*>(a.dt) + k.b * L * D + cs;
    const T_* Bp = static_cast<const T_*>(a.B) + k.b * L * a.bc_row_stride + k.g * N + w * S;
    const SelDt dtp{a.dtp.bias ? a.dtp.bias[cs] : 0.f, a.dtp.lo, a.dtp.hi, a.dtp.softplus};
    float A2[S], h[S];
#pragma unroll
    for (int s = 0; s < S; ++s) {
        A2[s] = a.A[static_cast<int64_t>(cs) * N + w * S + s] * kLog2e;
        h[s] = a.init_state && ok ? a.init_state[(k.b * D + cs) * N + w * S + s] : 0.f;
    }
    float xr[TPT], dr[TPT];
    auto load = [&](int64_t t0) {
#pragma unroll
        for (int i = 0; i < TPT; ++i) {
            const int64_t t = t0 + w + W * i < L ? t0 + w + W * i : L - 1;
            xr[i] = static_cast<float>(xp[t * a.x_row_stride]);
            dr[i] = static_cast<float>(dp[t * D]);
        }
    };
    if (L > 0) load(0);
    int buf = 0;
    for (int64_t tile = 0; tile < tiles; ++tile, buf ^= 1) {
        const int64_t t0 = tile * T;
#pragma unroll
        for (int s = 0; s < S; ++s)
            if (ok) ckpt[((k.b * tiles + tile) * N + w * S + s) * D + c] = h[s];
        if (tile + 1 == tiles) break;
#pragma unroll
        for (int i = 0; i < TPT; ++i) {
            const int t = w + W * i;
            if (t < T) {
                const float dt = sel_dt(dr[i], dtp);
                st[buf][t][lane] = ok ? make_float2(dt, dt * xr[i]) : make_float2(0.f, 0.f);
            }
        }
        __syncthreads();
        load(t0 + T);
#pragma unroll
        for (int t = 0; t < T; ++t) {
            float Bv[S];
            load_uniform<T_, S>(Bp + (t0 + t) * a.bc_row_stride, Bv);
            const float2 d = st[buf][t][lane];
#pragma unroll
            for (int s = 0; s < S; ++s) h[s] = fmaf(__builtin_amdgcn_exp2f(d.x * A2[s]), h[s], d.y * Bv[s]);
        }
    }
}

template <typename T_, typename TY, int S, int W, bool GATE>
__global__ __launch_bounds__(64 * W, 2) void selective_grad_kernel(SelBwdArgs a, float* ws, SelBwdLayout lay) {
    constexpr int N = S * W, T = SelTile<S>::T, TPT = (T + W - 1) / W;
    __shared__ float2 st[T][64];            // dt, dt * x
    __shared__ float sdy[T][64];            // dy
    __shared__ float2 part[W][T][64];       // <g, B>, <g q, A> over the wave's states
    __shared__ float ypart[GATE ? W : 1][GATE ? T : 1][64];
    const SelBlock k = sel_block(blockIdx.x, a.channels, a.ngroups);
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = k.c0 + lane;
    const bool ok = c < k.cend;
    const int cs = ok ? c : k.c0;
    const int64_t L = a.seqlen, D = a.channels;
    const T_* xp = static_cast<const T_*>(a.x) + k.b * L * a.x_row_stride + cs;
    const T_* zp = GATE ? static_cast<const T_*>(a.z) + k.b * L * a.z_row_stride + cs : nullptr;
    const T_* dp = static_cast<const T_*>(a.dt) + k.b * L * D + cs;
    const TY* gp = static_cast<const TY*>(a.dy) + k.b * L * D + cs;
    const T_* Bp = static_cast<const T_*>(a.B) + k.b * L * a.bc_row_stride + k.g * N + w * S;
    const T_* Cp = static_cast<const T_*>(a.C) + k.b * L * a.bc_row_stride + k.g * N + w * S;
    T_* dxp = static_cast<T_*>(a.dx) + k.b * L * D + cs;
    T_* ddp = static_cast<T_*>(a.ddt) + k.b * L * D + cs;
    T_* dzp = GATE ? static_cast<T_*>(a.dz) + k.b * L * D + cs : nullptr;
    float* bcp = ws + lay.dBC + (static_cast<int64_t>(k.blk) * a.batch + k.b) * L * 2 * N + w * S;
    const float* ckpt = ws + lay.ckpt + k.b * lay.tiles * N * D + cs;
    const SelDt dtp{a.dtp.bias ? a.dtp.bias[cs] : 0.f, a.dtp.lo, a.dtp.hi, a.dtp.softplus};
    const float Dv = a.D ? a.D[cs] : 0.f;
    float A2[S], dA[S], carry[S];
    const int64_t so = (k.b * D + cs) * N + w * S;
#pragma unroll
    for (int s = 0; s < S; ++s) {
        A2[s] = a.A[static_cast<int64_t>(cs) * N + w * S + s] * kLog2e;
        dA[s] = 0.f;
        carry[s] = a.dfinal_state && ok ? a.dfinal_state[so + s] : 0.f;
    }
    float dDv = 0.f, dbv = 0.f;
    for (int64_t tile = lay.tiles - 1; tile >= 0; --tile) {
        const int64_t t0 = tile * T;
        float xk[TPT], vk[TPT], yk[TPT], zk[TPT], dk[TPT];
#pragma unroll
        for (int i = 0; i < TPT; ++i) {
            const int t = w + W * i;
            const bool in = t < T && t0 + t < L && ok;
            const int64_t tt = t0 + t < L ? t0 + t : L - 1;
            xk[i] = in ? static_cast<float>(xp[tt * a.x_row_stride]) : 0.f;
            vk[i] = static_cast<float>(dp[tt * D]);
            yk[i] = in ? static_cast<float>(gp[tt * D]) : 0.f;
            zk[i] = GATE ? static_cast<float>(zp[tt * a.z_row_stride]) : 0.f;
            dk[i] = in ? sel_dt(vk[i], dtp) : 0.f;
            if (t < T) {
                st[t][lane] = make_float2(dk[i], dk[i] * xk[i]);
                sdy[t][lane] = GATE ? yk[i] * silu_f(zk[i]) : yk[i];
            }
        }
        float h[S], q[T][S], ea[T][S];
#pragma unroll
        for (int s = 0; s < S; ++s) h[s] = ok ? ckpt[(tile * N + w * S + s) * D] : 0.f;
        __syncthreads();
#pragma unroll
        for (int t = 0; t < T; ++t) {
            const int64_t row = t0 + t < L ? t0 + t : L - 1;
            float Bv[S], Cv[S];
            load_uniform<T_, S>(Bp + row * a.bc_row_stride, Bv);
            if constexpr (GATE) load_uniform<T_, S>(Cp + row * a.bc_row_stride, Cv);
            const float2 d = st[t][lane];
            float y = 0.f;
#pragma unroll
            for (int s = 0; s < S; ++s) {
                ea[t][s] = __builtin_amdgcn_exp2f(d.x * A2[s]);
                q[t][s] = ea[t][s] * h[s];
                h[s] = fmaf(d.y, Bv[s], q[t][s]);
                if constexpr (GATE) y = fmaf(h[s], Cv[s], y);
            }
            if constexpr (GATE) ypart[w][t][lane] = y;
        }
        f32x4 accB[4], accC[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) accB[m] = accC[m] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int t = T - 1; t >= 0; --t) {
            const int64_t row = t0 + t < L ? t0 + t : L - 1;
            float Bv[S], Cv[S];
            load_uniform<T_, S>(Bp + row * a.bc_row_stride, Bv);
            load_uniform<T_, S>(Cp + row * a.bc_row_stride, Cv);
            const float2 d = st[t][lane];
            const float dy = sdy[t][lane];
            float gB = 0.f, gA = 0.f;
#pragma unroll
            for (int s = 0; s < S; ++s) {
                const int f = s * T + t;   // the pair's place: accumulator f / 16, column f % 16
                const float hot = (lane & 15) == (f & 15) ? 1.f : 0.f;
                const float g = fmaf(Cv[s], dy, carry[s]);
                const float hv = fmaf(d.y, Bv[s], q[t][s]);
                accB[f >> 4] = __builtin_amdgcn_mfma_f32_16x16x4f32(g * d.y, hot, accB[f >> 4], 0, 0, 0);
                accC[f >> 4] = __builtin_amdgcn_mfma_f32_16x16x4f32(dy * hv, hot, accC[f >> 4], 0, 0, 0);
                gB = fmaf(g, Bv[s], gB);
                const float v = g * q[t][s];
                dA[s] = fmaf(d.x, v, dA[s]);
                gA = fmaf(A2[s], v, gA);
                carry[s] = ea[t][s] * g;
            }
            part[w][t][lane] = make_float2(gB, gA);
        }
        // rows of the accumulators: 4 in the lane, then lanes 16 and 32 apart; row r of lanes stores
        // accumulator r
        float vB = 0.f, vC = 0.f;
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            float b = (accB[m][0] + accB[m][1]) + (accB[m][2] + accB[m][3]);
            float e = (accC[m][0] + accC[m][1]) + (accC[m][2] + accC[m][3]);
            b += __shfl_xor(b, 16, 64);
            e += __shfl_xor(e, 16, 64);
            b += __shfl_xor(b, 32, 64);
            e += __shfl_xor(e, 32, 64);
            if ((lane >> 4) == m) {
                vB = b;
                vC = e;
            }
        }
        {
            const int t = lane % T, s = lane / T;   // lane = 16 m + column
            if (t0 + t < L) {
                bcp[(t0 + t) * 2 * N + s] = vB;
                bcp[(t0 + t) * 2 * N + N + s] = vC;
            }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < TPT; ++i) {
            const int t = w + W * i;
            if (t >= T || t0 + t >= L || !ok) continue;
            float gB = 0.f, gA = 0.f;
#pragma unroll
            for (int v = 0; v < W; ++v) {
                gB += part[v][t][lane].x;
                gA += part[v][t][lane].y;
            }
            const float dy = sdy[t][lane];
            dxp[(t0 + t) * D] = static_cast<T_>(fmaf(Dv, dy, dk[i] * gB));
            float dd = fmaf(gA, 1.f / kLog2e, xk[i] * gB);
            const float v = vk[i] + dtp.bias;
            if (dtp.lo < dtp.hi) {
                const float u = dtp.softplus ? sel_softplus(v) : v;
                if (!(u >= dtp.lo && u <= dtp.hi)) dd = 0.f;
            }
            if (dtp.softplus) dd *= __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-v * kLog2e));
            ddp[(t0 + t) * D] = static_cast<T_>(dd);
            dbv += dd;
            dDv = fmaf(dy, xk[i], dDv);
            if constexpr (GATE) {
                float y = Dv * xk[i];
#pragma unroll
                for (int u = 0; u < W; ++u) y += ypart[u][t][lane];
                const float sg = __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-zk[i] * kLog2e));
                dzp[(t0 + t) * D] = static_cast<T_>(yk[i] * y * sg * fmaf(zk[i], 1.f - sg, 1.f));
            }
        }
        __syncthreads();
    }
    if (ok) {
#pragma unroll
        for (int s = 0; s < S; ++s) {
            ws[lay.dA + (k.b * N + w * S + s) * D + c] = dA[s];
            if (a.dinit_state) a.dinit_state[so + s] = carry[s];
        }
    }
    part[w][0][lane] = make_float2(dDv, dbv);   // the last tile ended with a barrier
    __syncthreads();
    if (w == 0 && ok) {
        float u = 0.f, v = 0.f;
#pragma unroll
        for (int i = 0; i < W; ++i) {
            u += part[i][0][lane].x;
            v += part[i][0][lane].y;
        }
        ws[lay.dD + k.b * D + c] = u;
        ws[lay.dbias + k.b * D + c] = v;
    }
}

// Sums of the partial results: D N values of dA, D of dDskip and of ddt_bias over the batch, and
// B L G N values of dB and of dC over the group's channel blocks.
template <typename T>
__global__ __launch_bounds__(256) void selective_sums_kernel(SelBwdArgs a, const float* __restrict__ ws, SelBwdLayout lay) {
    const int64_t D = a.channels, N = a.d_state, G = a.ngroups, rows = a.batch * a.seqlen;
    int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i < (N + 2) * D) {
        const float* p = ws + (i < N * D ? lay.dA + i : i < (N + 1) * D ? lay.dD + i - N * D : lay.dbias + i - (N + 1) * D);
        const int64_t step = i < N * D ? N * D : D;
        float v = 0.f;
        for (int64_t b = 0; b < a.batch; ++b) v += p[b * step];
        if (i < N * D) a.dA[i % D * N + i / D] = v;
        else if (i < (N + 1) * D) { if (a.dD) a.dD[i - N * D] = v; }
        else if (a.ddt_bias) a.ddt_bias[i - (N + 1) * D] = v;
        return;
    }
    i -= (N + 2) * D;
    if (i >= rows * 2 * G * N) return;
    const int64_t n = i % N, which = i / N % 2, g = i / (2 * N) % G, row = i / (2 * N * G);
    const int64_t per = lay.blocks / G;
    const float* p = ws + lay.dBC + (g * per * rows + row) * 2 * N + which * N + n;
    float v = 0.f;
    for (int64_t k = 0; k < per; ++k) v += p[k * rows * 2 * N];
    (which ? static_cast<T*>(a.dC) : static_cast<T*>(a.dB))[(row * G + g) * N + n] = static_cast<T>(v);
}

template <typename T, typename TY, int S, int W>
static hipError_t bwd_launch(const SelBwdArgs& a, float* ws, const SelBwdLayout& lay, hipStream_t s) {
    const dim3 grid(static_cast<uint32_t>(a.batch * lay.blocks)), block(64 * W);
    if (a.batch > 0) {
        hipLaunchKernelGGL((selective_states_kernel<T, S, W>), grid, block, 0, s, a, ws + lay.ckpt, lay.tiles);
    }
    if (a.batch > 0 && a.z) hipLaunchKernelGGL((selective_grad_kernel<T, TY, S, W, true>), grid, block, 0, s, a, ws, lay);
    else if (a.batch > 0) hipLaunchKernelGGL((selective_grad_kernel<T, TY, S, W, false>), grid, block, 0, s, a, ws, lay);
    const int64_t n = (a.d_state + 2) * static_cast<int64_t>(a.channels) + a.batch * a.seqlen * 2 * a.ngroups * a.d_state;
    hipLaunchKernelGGL((selective_sums_kernel<T>), dim3(static_cast<uint32_t>((n + 255) / 256)), dim3(256), 0, s, a, ws, lay);
    return hipGetLastError();
}

template <typename T, typename TY>
static hipError_t bwd_t(const SelBwdArgs& a, float* ws, hipStream_t s) {
    const SelBwdLayout lay = bwd_layout(a.batch, a.seqlen, a.channels, a.ngroups, a.d_state);
    switch (a.d_state) {
        case 16: return bwd_launch<T, TY, 4, 4>(a, ws, lay, s);
        case 32: return bwd_launch<T, TY, 8, 4>(a, ws, lay, s);
        case 64: return bwd_launch<T, TY, 8, 8>(a, ws, lay, s);
        case 128: return bwd_launch<T, TY, 16, 8>(a, ws, lay, s);
        default: return hipErrorInvalidValue;
    }
}

size_t selective_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int channels, int ngroups, int d_state) {
    return static_cast<size_t>(bwd_layout(batch, seqlen, channels, ngroups, d_state).total) * sizeof(float);
}

hipError_t launch_selective_scan_bwd(const SelBwdArgs& a, Dt act, Dt ydt, void* workspace, hipStream_t s) {
    float* ws = static_cast<float*>(workspace);
    if (act == Dt::BF16) return ydt == Dt::BF16 ? bwd_t<bf16, bf16>(a, ws, s) : bwd_t<bf16, float>(a, ws, s);
    return ydt == Dt::BF16 ? bwd_t<float, bf16>(a, ws, s) : bwd_t<float, float>(a, ws, s);
}

}  // namespace ssd
