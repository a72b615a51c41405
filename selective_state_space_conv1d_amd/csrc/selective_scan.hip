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
// Bound: the vector pipe.  A state of a token and channel takes six issue slots (a product, an exp2 of two
// slots, a product and two fmas) of four cycles for 64 lanes; no product shares an operand across channels, so
// the matrix pipe does not apply.  2 x 8192 tokens x 4096 channels, 16 states, bf16, z and states: 196 us
// (chunk states, five slots) + 273 us under the profiler, of which the states' slots take 128 and 164 and the
// tokens' own work (dt's softplus, gate, sums over waves) 40 and 85; 411 us back to back.
#include "selective_device.h"

namespace ssd {

constexpr int kSelTile = 16;   // tokens staged at a time

// Sequences are cut into chunks of `tokens` when there are too few workgroups otherwise (sel_chunks).
// Then a first launch (Y false) runs each chunk but the last, the first from the initial state and the
// others from zero, and leaves its final state [B][chunks][N][D] and its sum of dt [B][chunks][D]; a
// chunk's state at its first token follows from those of the chunks before it, since a chunk multiplies
// the state it starts from by exp(A sum dt).
struct SelChunks {
    int64_t tokens;
    int n;
    float* ends;
    float* sums;
};

template <typename T, typename TY, int S, int W, bool Y, bool GATE>
__global__ __launch_bounds__(64 * W) void selective_scan_kernel(SelScanArgs a, SelChunks ch) {
    constexpr int N = S * W, TPT = kSelTile / W;   // tokens of a tile that one thread stages
    constexpr int SUB = SelRows<T, S>::n;          // tokens whose B and C are in scalar registers
    constexpr int E = sizeof(T);
    // dt, dt * x; twice without y, which saves a barrier.  With y the waves that less LDS lets in are worth
    // more than the barrier (2 x 8192 x 4096, bf16: 484 us; both arrays twice, one barrier a tile: 514)
    __shared__ float2 st[Y ? 1 : 2][kSelTile][64];
    __shared__ float part[Y ? W : 1][kSelTile][64];   // y of the wave's states
    const int64_t per_chunk = a.batch * sel_blocks(a.channels, a.ngroups);
    const int chunk = static_cast<int>(blockIdx.x / per_chunk);
    const SelBlock k = sel_block(blockIdx.x % per_chunk, a.channels, a.ngroups);
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = k.c0 + lane;
    const bool ok = c < k.cend;
    const int cs = ok ? c : k.c0;                  // lanes past the group read its first channel, store nothing
    const int64_t D = a.channels;
    const int64_t r0 = k.b * a.seqlen + chunk * ch.tokens;   // first token row
    const int64_t left = a.seqlen - chunk * ch.tokens;
    const int L = static_cast<int>(left < ch.tokens ? left : ch.tokens);   // the chunk's tokens
    // per stream: the tile's first row (scalar, advanced tile by tile), and offsets in bytes from there
    // (16 rows and a bit, in 32 bits: row strides are at most 2^24 elements)
    const char* xp = static_cast<const char*>(a.x) + (r0 * a.x_row_stride + k.c0) * E;
    const char* zp = GATE ? static_cast<const char*>(a.z) + (r0 * a.z_row_stride + k.c0) * E : nullptr;
    const char* dp = static_cast<const char*>(a.dt) + (r0 * D + k.c0) * E;
    const char* Bp = static_cast<const char*>(a.B) + (r0 * a.bc_row_stride + k.g * N + w * S) * E;
    const char* Cp = static_cast<const char*>(a.C) + (r0 * a.bc_row_stride + k.g * N + w * S) * E;
    char* yp = static_cast<char*>(a.y) + (r0 * D + k.c0) * sizeof(TY);
    const uint32_t xs = static_cast<uint32_t>(a.x_row_stride) * E, zs = static_cast<uint32_t>(a.z_row_stride) * E;
    const uint32_t ds = static_cast<uint32_t>(D) * E, ys = static_cast<uint32_t>(D) * sizeof(TY), bs = static_cast<uint32_t>(a.bc_row_stride) * E;
    const uint32_t le = (cs - k.c0) * E;
    const SelDt dtp{a.dtp.bias ? a.dtp.bias[cs] : 0.f, a.dtp.lo, a.dtp.hi, a.dtp.softplus};
    const float Dv = a.D ? a.D[cs] : 0.f;
    float A2[S], h[S];
    const int64_t so = (k.b * D + cs) * N + w * S;
#pragma unroll
    for (int s = 0; s < S; ++s) {
        A2[s] = base2_rate(a.A[static_cast<int64_t>(cs) * N + w * S + s]);
        h[s] = (ch.n == 1 || (!Y && chunk == 0)) && a.init_state ? a.init_state[so + s] : 0.f;
    }
    // the first launch of a chunked scan keeps the initial state in the last chunk's place, which has no
    // other use: in the second the final state may be written over it before all have read it
    float* ends = ch.ends + (k.b * ch.n * N + w * S) * D + cs;
    if (!Y && chunk == 0 && ok)
#pragma unroll
        for (int s = 0; s < S; ++s) ends[((ch.n - 1) * N + s) * D] = h[s];
    if (Y && ch.n > 1) {
        if (chunk == 0)
#pragma unroll
            for (int s = 0; s < S; ++s) h[s] = ends[((ch.n - 1) * N + s) * D];
        join_chunks(h, A2, ch.sums + k.b * ch.n * D + cs, ends, 0, chunk, 1, D, N * D, D);
    }
    T xr[TPT], zr[TPT], dr[TPT];     // the next tile's values as loaded
    float xk[TPT], zk[TPT], sum = 0.f;
    uint32_t ahead = 0;
    // this thread's tokens first + w + W i of the tile, none past row `last`
    auto load = [&](int first, int last) {
#pragma unroll
        for (int i = 0; i < TPT; ++i) {
            const uint32_t t = static_cast<uint32_t>(first + w + W * i < last ? first + w + W * i : last);
            xr[i] = *reinterpret_cast<const T*>(xp + (le + t * xs));
            dr[i] = *reinterpret_cast<const T*>(dp + (le + t * ds));
            if constexpr (GATE) zr[i] = *reinterpret_cast<const T*>(zp + (le + t * zs));
        }
        // B and C of the tile, a token a lane: brings the rows, which each wave reads through the scalar
        // cache a few tokens before it needs them, near in time
        const uint32_t t = static_cast<uint32_t>(first + (lane & 15) < last ? first + (lane & 15) : last);
        ahead = *reinterpret_cast<const uint32_t*>((lane & 16 ? Cp : Bp) + static_cast<uint64_t>(t * bs));
    };
    // y of the tile before the one that starts at yp, whose partial sums lie in part; rows past `last` of
    // it do not exist
    auto finish = [&](int last) {
        if constexpr (Y) {
            float y[TPT];
#pragma unroll
            for (int i = 0; i < TPT; ++i) {
                y[i] = Dv * xk[i];
#pragma unroll
                for (int v = 0; v < W; ++v) y[i] += part[v][w + W * i][lane];
                if constexpr (GATE) y[i] *= silu_f(zk[i]);
            }
            char* base = yp - static_cast<int64_t>(kSelTile) * ys;
            auto store = [&](int i) {
                *reinterpret_cast<TY*>(base + (static_cast<uint32_t>(lane * sizeof(TY)) + static_cast<uint32_t>(w + W * i) * ys)) = static_cast<TY>(y[i]);
            };
            if (ok && last >= kSelTile - 1) {
#pragma unroll
                for (int i = 0; i < TPT; ++i) store(i);
            } else if (ok) {
#pragma unroll
                for (int i = 0; i < TPT; ++i)
                    if (w + W * i <= last) store(i);
            }
        }
    };
    SelRows<T, S> rows[2];
    float2 d[2][SUB];
    if (L > 0) {
        load(0, L - 1);
        rows[0].template load<Y>(Bp, Cp, bs, 0, L - 1);
    }
    int buf = 0;
    for (int t0 = 0; t0 < L; t0 += kSelTile, buf ^= Y ? 0 : 1) {
        const int last = L - 1 - t0;
        float xn[TPT], dn[TPT], zn[TPT];
#pragma unroll
        for (int i = 0; i < TPT; ++i) {
            xn[i] = static_cast<float>(xr[i]);
            dn[i] = static_cast<float>(dr[i]);
            if constexpr (GATE) zn[i] = static_cast<float>(zr[i]);
        }
        asm volatile("" ::"v"(ahead));
        sel_dts(dn, dtp);
        if (last < kSelTile - 1)                              // past the end the state stands still
#pragma unroll
            for (int i = 0; i < TPT; ++i)
                if (w + W * i > last) xn[i] = dn[i] = 0.f;
        if constexpr (Y) {
            __syncthreads();
            if (t0 > 0) finish(kSelTile);
        }
#pragma unroll
        for (int i = 0; i < TPT; ++i) {
            st[buf][w + W * i][lane] = make_float2(dn[i], dn[i] * xn[i]);
            if constexpr (!Y) sum += dn[i];
        }
        __syncthreads();
        load(kSelTile, last);
#pragma unroll
        for (int t = 0; t < SUB; ++t) d[0][t] = st[buf][t][lane];
#pragma unroll
        for (int i = 0; i < TPT; ++i) {
            xk[i] = xn[i];
            if constexpr (GATE) zk[i] = zn[i];
        }
#pragma unroll
        for (int u = 0; u < kSelTile; u += SUB) {
            const int at = (u / SUB) & 1;
            // the next tokens' B, C, dt and dt * x are fetched while these are used
            rows[at ^ 1].template load<Y>(Bp, Cp, bs, u + SUB, last);
            if (u + SUB < kSelTile)
#pragma unroll
                for (int t = 0; t < SUB; ++t) d[at ^ 1][t] = st[buf][u + SUB + t][lane];
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int t = 0; t < SUB; ++t) {
                float y = 0.f;
#pragma unroll
                for (int s = 0; s < S; ++s) {
                    const float e = __builtin_amdgcn_exp2f(d[at][t].x * A2[s]);
                    h[s] = fmaf(e, h[s], d[at][t].y * rows[at].b(t, s));
                    if constexpr (Y) y = fmaf(h[s], rows[at].c(t, s), y);
                }
                if constexpr (Y) part[w][u + t][lane] = y;
            }
        }
        xp += static_cast<int64_t>(kSelTile) * xs;
        dp += static_cast<int64_t>(kSelTile) * ds;
        if constexpr (GATE) zp += static_cast<int64_t>(kSelTile) * zs;
        Bp += static_cast<int64_t>(kSelTile) * bs;
        Cp += static_cast<int64_t>(kSelTile) * bs;
        yp += static_cast<int64_t>(kSelTile) * ys;
    }
    __syncthreads();
    if constexpr (Y) {
        if (L > 0) finish((L - 1) % kSelTile);
        if (a.final_state && ok && chunk == ch.n - 1) {
#pragma unroll
            for (int s = 0; s < S; ++s) a.final_state[so + s] = h[s];
        }
    } else {
        st[0][w][lane] = make_float2(sum, 0.f);
        __syncthreads();
        if (ok) {
#pragma unroll
            for (int s = 0; s < S; ++s) ends[(chunk * N + s) * D] = h[s];
            if (w == 0) {
                float v = 0.f;
#pragma unroll
                for (int i = 0; i < W; ++i) v += st[0][i][lane].x;
                ch.sums[(k.b * ch.n + chunk) * D + c] = v;
            }
        }
    }
}

constexpr int sel_waves(int d_state) { return d_state == 128 ? 8 : 4; }

// Chunks of a sequence.  The kernel wants three waves or more on each of the 1024 SIMDs; below 2048 waves
// in all, the second pass that chunks cost (5/6 of the first one's vector operations) is less than what
// stands idle.  Measured, 16 states, bf16: 2 x 8192 tokens x 4096 channels (512 waves) 1108 us in one
// chunk, 499 with 5120 waves, 490 with 6144, 484 with 8192, 490 with 12288; 6 x 2048 x 4096 (1536 waves) 338
// in one chunk, 303 in six; 8 x 2048 x 4096 (2048 waves) 341-366 in one, 450 in four.  Chunks of 32 tokens
// or more: 1 x 512 x 4096 29 us (38 with 16 tokens or more), 1 x 1024 x 1536 28 (37; 40 with 64).
static SelChunks sel_chunks(int64_t batch, int64_t L, int channels, int ngroups, int d_state) {
    const int64_t waves = batch * sel_blocks(channels, ngroups) * sel_waves(d_state);
    int64_t n = waves >= 2048 || waves == 0 ? 1 : (8192 + waves - 1) / waves;
    if (n > most_chunks(L)) n = most_chunks(L);
    int64_t tokens = (L + n - 1) / n;
    tokens = (tokens + kSelTile - 1) / kSelTile * kSelTile;
    if (n == 1) tokens = L > 0 ? L : 1;
    SelChunks c{tokens, static_cast<int>(L > 0 ? (L + tokens - 1) / tokens : 1), nullptr, nullptr};
    return c;
}

template <typename T, typename TY, int S, int W>
static hipError_t scan_launch(const SelScanArgs& a, const SelChunks& ch, hipStream_t s) {
    const int64_t per_chunk = a.batch * sel_blocks(a.channels, a.ngroups);
    if (ch.n > 1)
        hipLaunchKernelGGL((selective_scan_kernel<T, TY, S, W, false, false>), dim3(static_cast<uint32_t>(per_chunk * (ch.n - 1))),
                           dim3(64 * W), 0, s, a, ch);
    const dim3 grid(static_cast<uint32_t>(per_chunk * ch.n)), block(64 * W);
    if (a.z) hipLaunchKernelGGL((selective_scan_kernel<T, TY, S, W, true, true>), grid, block, 0, s, a, ch);
    else hipLaunchKernelGGL((selective_scan_kernel<T, TY, S, W, true, false>), grid, block, 0, s, a, ch);
    return hipGetLastError();
}

template <typename T, typename TY>
static hipError_t scan_t(const SelScanArgs& a, const SelChunks& ch, hipStream_t s) {
    switch (a.d_state) {
        case 16: return scan_launch<T, TY, 4, 4>(a, ch, s);
        case 32: return scan_launch<T, TY, 8, 4>(a, ch, s);
        case 64: return scan_launch<T, TY, 16, 4>(a, ch, s);
        case 128: return scan_launch<T, TY, 16, 8>(a, ch, s);
        default: return hipErrorInvalidValue;
    }
}

size_t selective_scan_workspace_bytes(int64_t batch, int64_t seqlen, int channels, int ngroups, int d_state) {
    const SelChunks c = sel_chunks(batch, seqlen, channels, ngroups, d_state);
    return c.n > 1 ? static_cast<size_t>(batch * c.n * (d_state + 1) * channels) * sizeof(float) : 0;
}

hipError_t launch_selective_scan(const SelScanArgs& a, Dt act, Dt ydt, void* workspace, hipStream_t s) {
    if (a.batch == 0) return hipSuccess;
    SelChunks c = sel_chunks(a.batch, a.seqlen, a.channels, a.ngroups, a.d_state);
    c.ends = static_cast<float*>(workspace);
    c.sums = c.ends + a.batch * c.n * a.d_state * static_cast<int64_t>(a.channels);
    if (act == Dt::BF16) return ydt == Dt::BF16 ? scan_t<bf16, bf16>(a, c, s) : scan_t<bf16, float>(a, c, s);
    return ydt == Dt::BF16 ? scan_t<float, bf16>(a, c, s) : scan_t<float, float>(a, c, s);
}

// One token per batch entry.  The state is read once and written once: an HBM stream.  A thread owns
// four states of a channel and walks batch entries with A, the skip weight and dt's bias in registers,
// kUpdInFlight entries' loads issued together; the N / 4 lanes of a channel add up y by lane moves.
// 256 entries x 8192 channels x 16 states in a pool of 320: 55-57 us back to back, 5.1 TB/s.  Four entries in
// flight 71 us with as many workgroups, eight 72; loads that bypass the caches: 4096 channels, fp32, 35 us
// where these take 28.5.  One entry x 4096 channels: 3.7 us, a launch and the chain of its loads.
constexpr int kSelUpdThreads = 256;
constexpr int kUpdInFlight = 2;

// Four consecutive values at any address that suits one of them.
template <typename T>
struct __attribute__((packed, aligned(sizeof(T)))) Four {
    T v[4];
};

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
        T xr[kUpdInFlight], dr[kUpdInFlight], zr[kUpdInFlight];
        Four<T> Bv[kUpdInFlight], Cv[kUpdInFlight];
#pragma unroll
        for (int i = 0; i < kUpdInFlight; ++i) {
            const int64_t b = b0 + i < bend ? b0 + i : bend - 1;
            slot[i] = seq_slot(a.slot_idx, b, a.nslots);
            h[i] = slot[i] >= 0 ? *reinterpret_cast<const f32x4*>(a.state + (slot[i] * D + c) * N + 4 * q)
                                : f32x4{0.f, 0.f, 0.f, 0.f};
            xr[i] = x[b * a.x_row_stride + c];
            dr[i] = dt[b * D + c];
            if (z) zr[i] = z[b * a.z_row_stride + c];
            Bv[i] = *reinterpret_cast<const Four<T>*>(B + b * a.bc_row_stride + bo);
            Cv[i] = *reinterpret_cast<const Four<T>*>(C + b * a.bc_row_stride + bo);
        }
#pragma unroll
        for (int i = 0; i < kUpdInFlight; ++i) {
            const bool in = ok && b0 + i < bend;
            const int64_t b = b0 + i < bend ? b0 + i : bend - 1;
            const float xv = static_cast<float>(xr[i]);
            const float dv = sel_dt(static_cast<float>(dr[i]), dtp);
            const float dx = dv * xv, d2 = dv * kLog2e;
            float y = 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                h[i][k] = fmaf(__builtin_amdgcn_exp2f(d2 * A4[k]), h[i][k], dx * static_cast<float>(Bv[i].v[k]));
                y = fmaf(h[i][k], static_cast<float>(Cv[i].v[k]), y);
            }
            y = group_sum_last<Q>(y);   // every lane takes part: those past the end hold channel 0's values
            if (in && q == Q - 1) {
                y = fmaf(Dv, xv, y);
                if (z) y *= silu_f(static_cast<float>(zr[i]));
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
    // batch entries per workgroup: about the 2048 workgroups that run at once (eight waves a SIMD) and no
    // more than 65535 rows of them.  256 entries x 8192 channels x 16 states, pool of 320: 56 us with 2048,
    // 76 with 1024, 67 with 4096 and four entries in flight; 64 entries: 17.3, 19.8 and 18.8 us.
    int64_t per = kUpdInFlight;
    while (per < a.batch && (xb * ((a.batch + per - 1) / per) > 2048 || (a.batch + per - 1) / per > 65535)) per *= 2;
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
