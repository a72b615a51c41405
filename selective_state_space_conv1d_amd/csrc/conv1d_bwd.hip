// Gradient of the causal depthwise conv + SiLU (conv1d.hip).  With u~ the input preceded by the conv
// state, p_t = bias + sum_k w[k] u~[t-3+k] and q_t = dout_t silu'(p_t):
//   du~[t] = sum_k w[k] q[t+3-k]     dw[k] = sum_{b,t} q[t] u~[t-3+k]     dbias = sum_{b,t} q
// The states' own gradients: conv_state_out[k] = u~[L-4+k] adds to du~, and conv_state_in's gradient is
// du~ at the four positions before the first token (the oldest feeds no output).
//
// A thread owns four channels (eight of bf16 would take more registers than two waves a SIMD have) and walks
// a tile of tokens with the last three inputs and q values in registers, so each input is read once (plus
// three rows on either side of a tile) and each output written once: bound by HBM.  Rows are taken four at a
// time, the next four loaded while four are computed.  dw and dbias are summed in registers over the tile,
// over the workgroup's tiles in LDS and over workgroups by a second launch, in a fixed order.
// 2 x 8192 x 18432, bf16: 378 us back to back, 4.8 TB/s of its 1.81 GB (a device copy: 5.2); 4 x 2048 x 8192:
// 97 us; 1 x 77 x 1792, fp32: 12 + 4 us, the chain of a tile's 16 rows.  Held to three waves a SIMD by its
// register count the first takes 481 us, with ordinary stores in place of non-temporal ones 420.
#include "ssd_device.h"
#include "ssd_kernels.h"

#include <type_traits>

namespace ssd {

constexpr int kCbV = 4;           // channels per thread
constexpr int kCbLanes = 64;      // threads across the channels of a workgroup
constexpr int kCbSub = 4;         // token tiles per workgroup, one for each wave

// Rows that a tile walks, its tokens and the three after them: 128, fewer where that gives less than two
// workgroups a CU (with an earlier form of the loop, 2 x 8192 x 18432, bf16: 408 us with 128, 440 with 64, 422
// with 256; 1 x 8192 x 18432: 204, 207, 241).
static int64_t tile_steps(int64_t batch, int64_t L, int64_t CD) {
    const int64_t cb = (CD + kCbLanes * kCbV - 1) / (kCbLanes * kCbV);
    int64_t steps = 128;
    while (steps > 16 && batch * cb * ((L + (steps - 3) * kCbSub - 1) / ((steps - 3) * kCbSub)) < 512) steps /= 2;
    return steps;
}

template <typename T>
__global__ __launch_bounds__(kCbLanes * kCbSub) void conv1d_bwd_kernel(ConvBwdArgs a, float* __restrict__ part,
                                                                       int64_t tblocks, int64_t cblocks, int64_t tokens) {
    constexpr int V = kCbV;
    typedef T Raw __attribute__((ext_vector_type(V)));
    __shared__ float red[kCbSub][5][V][kCbLanes];
    const int lane = threadIdx.x % kCbLanes, sub = __builtin_amdgcn_readfirstlane(threadIdx.x / kCbLanes);   // a wave's own tile
    const int64_t cb = blockIdx.x % cblocks, tb = blockIdx.x / cblocks % tblocks, b = blockIdx.x / (cblocks * tblocks);
    const int64_t CD = a.channels, L = a.seqlen;
    const bool ok = (cb * kCbLanes + lane) * V < CD;
    const int64_t c0 = ok ? (cb * kCbLanes + lane) * V : 0;
    const int64_t t0 = (tb * kCbSub + sub) * tokens;
    const int64_t t1 = t0 + tokens < L ? t0 + tokens : L;
    const T* xp = static_cast<const T*>(a.xbc) + b * L * a.xbc_row_stride + c0;
    const T* gp = static_cast<const T*>(a.dout) + b * L * CD + c0;
    T* dp = static_cast<T*>(a.dxbc) + b * L * CD + c0;
    const T* sin = a.state_in ? static_cast<const T*>(a.state_in) + (b * CD + c0) * 4 : nullptr;
    const T* dso = a.dstate_out ? static_cast<const T*>(a.dstate_out) + (b * CD + c0) * 4 : nullptr;
    T* dsi = a.dstate_in ? static_cast<T*>(a.dstate_in) + (b * CD + c0) * 4 : nullptr;
    float wt[4][V], bs[V], dw[4][V], db[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        bs[v] = a.bias ? static_cast<float>(static_cast<const T*>(a.bias)[c0 + v]) : 0.f;
        db[v] = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            wt[k][v] = static_cast<float>(static_cast<const T*>(a.w)[(c0 + v) * 4 + k]);
            dw[k][v] = 0.f;
        }
    }
    // du~[t] from outside the outputs: the stored windows
    auto stored = [&](int64_t t, int v) { return dso && t >= L - 4 ? static_cast<float>(dso[v * 4 + (t - L + 4)]) : 0.f; };
    if (ok && t0 < t1) {
        float u[7][V], q[7][V];     // u~ and q of tokens t-3 .. t+3
        Raw nu[4], ng[4];           // input and output gradient of the next four tokens, as loaded
        auto load = [&](int64_t t) {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int64_t row = t + r < L ? t + r : L - 1;
                nu[r] = __builtin_nontemporal_load(reinterpret_cast<const Raw*>(xp + row * a.xbc_row_stride));
                ng[r] = __builtin_nontemporal_load(reinterpret_cast<const Raw*>(gp + row * CD));
            }
        };
        load(t0);
#pragma unroll
        for (int r = 0; r < 3; ++r) {
            const int64_t t = t0 - 3 + r;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                u[r][v] = t >= 0 ? static_cast<float>(xp[t * a.xbc_row_stride + v]) : sin ? static_cast<float>(sin[v * 4 + 4 + t]) : 0.f;
                q[r][v] = 0.f;
            }
        }
        // rows t .. t+3: q there, then du~ of rows t-3 .. t, whose last q is now known.  EDGE: some of
        // them before the tile or its sequence, after the tile or in the last windows.
        auto rows = [&](int64_t t, auto edge) {
            constexpr bool EDGE = decltype(edge)::value;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const bool in = !EDGE || t + r < L, own = !EDGE || t + r < t1;
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const float p = fmaf(wt[3][v], u[r + 3][v], fmaf(wt[2][v], u[r + 2][v], fmaf(wt[1][v], u[r + 1][v], fmaf(wt[0][v], u[r][v], bs[v]))));
                    const float sg = __builtin_amdgcn_rcpf(1.f + __expf(-p));
                    // past the sequence's end there is no output
                    q[r + 3][v] = in ? q[r + 3][v] * sg * fmaf(p, 1.f - sg, 1.f) : 0.f;
                    if (own) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) dw[k][v] = fmaf(q[r + 3][v], u[r + k][v], dw[k][v]);
                        db[v] += q[r + 3][v];
                    }
                }
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int64_t at = t - 3 + r;
                float du[V];
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    du[v] = fmaf(wt[3][v], q[r][v], fmaf(wt[2][v], q[r + 1][v], fmaf(wt[1][v], q[r + 2][v], wt[0][v] * q[r + 3][v])));
                    if (EDGE && dso && at >= L - 4 && at < L) du[v] += stored(at, v);
                }
                if (!EDGE || (at >= t0 && at < t1)) {
                    Raw o;
#pragma unroll
                    for (int v = 0; v < V; ++v) o[v] = static_cast<T>(du[v]);
                    __builtin_nontemporal_store(o, reinterpret_cast<Raw*>(dp + at * CD));
                } else if (t0 == 0 && at < 0 && dsi) {
#pragma unroll
                    for (int v = 0; v < V; ++v) dsi[v * 4 + 4 + at] = static_cast<T>(du[v]);
                }
            }
        };
        for (int64_t t = t0; t < t1 + 3; t += 4) {
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    u[r + 3][v] = static_cast<float>(nu[r][v]);
                    q[r + 3][v] = static_cast<float>(ng[r][v]);
                }
            load(t + 4);
            if (t > t0 && t + 3 < t1 && t + 4 < L) rows(t, std::false_type{});
            else rows(t, std::true_type{});
#pragma unroll
            for (int r = 0; r < 3; ++r)
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    u[r][v] = u[r + 4][v];
                    q[r][v] = q[r + 4][v];
                }
        }
        if (t0 == 0 && dsi)
#pragma unroll
            for (int v = 0; v < V; ++v) dsi[v * 4] = static_cast<T>(stored(-4, v));
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int k = 0; k < 4; ++k) red[sub][k][v][lane] = dw[k][v];
        red[sub][4][v][lane] = db[v];
    }
    __syncthreads();
    // part[(b, tb)][5][CD]
    float* pp = part + (b * tblocks + tb) * 5 * CD;
    for (int i = threadIdx.x; i < 5 * V * kCbLanes; i += kCbLanes * kCbSub) {
        const int k = i / (V * kCbLanes), cc = i % (V * kCbLanes);
        const int64_t c = cb * kCbLanes * V + cc;
        if (c >= CD) continue;
        float v = 0.f;
#pragma unroll
        for (int j = 0; j < kCbSub; ++j) v += red[j][k][cc % V][cc / V];
        pp[k * CD + c] = v;
    }
}

// Sums of part over its n rows: dw[c][k] and dbias[c].
__global__ __launch_bounds__(256) void conv1d_bwd_sums_kernel(const float* __restrict__ part, int64_t n, int64_t CD,
                                                              float* __restrict__ dw, float* __restrict__ dbias) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= 5 * CD) return;
    float v = 0.f;
    for (int64_t r = 0; r < n; ++r) v += part[r * 5 * CD + i];
    const int64_t k = i / CD, c = i % CD;
    if (k < 4) dw[c * 4 + k] = v;
    else if (dbias) dbias[c] = v;
}

// L = 0: the conv state's gradient is the stored one's.
template <typename T>
__global__ __launch_bounds__(256) void conv1d_bwd_state_kernel(const T* __restrict__ dso, T* __restrict__ dsi, int64_t n) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i < n) dsi[i] = dso ? dso[i] : static_cast<T>(0.f);
}

static int64_t token_blocks(int64_t L, int64_t tokens) { return (L + tokens * kCbSub - 1) / (tokens * kCbSub); }

size_t conv1d_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t channels) {
    return static_cast<size_t>(batch * token_blocks(seqlen, tile_steps(batch, seqlen, channels) - 3) * 5 * channels) * sizeof(float);
}

template <typename T>
static hipError_t conv_bwd_t(const ConvBwdArgs& a, float* part, hipStream_t s) {
    constexpr int V = kCbV;
    const int64_t tokens = tile_steps(a.batch, a.seqlen, a.channels) - 3;
    const int64_t tb = token_blocks(a.seqlen, tokens), cb = (a.channels + kCbLanes * V - 1) / (kCbLanes * V);
    const int64_t blocks = a.batch * tb * cb;
    if (blocks > 0)
        hipLaunchKernelGGL((conv1d_bwd_kernel<T>), dim3(static_cast<uint32_t>(blocks)), dim3(kCbLanes * kCbSub), 0, s, a, part, tb, cb, tokens);
    else if (a.batch > 0 && a.dstate_in) {
        const int64_t n = a.batch * a.channels * 4;
        hipLaunchKernelGGL((conv1d_bwd_state_kernel<T>), dim3(static_cast<uint32_t>((n + 255) / 256)), dim3(256), 0, s,
                           static_cast<const T*>(a.dstate_out), static_cast<T*>(a.dstate_in), n);
    }
    hipLaunchKernelGGL(conv1d_bwd_sums_kernel, dim3(static_cast<uint32_t>((5 * a.channels + 255) / 256)), dim3(256), 0, s,
                       part, a.batch * tb, a.channels, a.dw, a.dbias);
    return hipGetLastError();
}

hipError_t launch_conv1d_bwd(const ConvBwdArgs& a, Dt act, void* workspace, hipStream_t s) {
    float* part = static_cast<float*>(workspace);
    return act == Dt::BF16 ? conv_bwd_t<bf16>(a, part, s) : conv_bwd_t<float>(a, part, s);
}

}  // namespace ssd
