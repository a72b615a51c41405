// Gradient of the per-channel selective scan (selective_scan.hip has the forward and its layout).
// With dy = dout silu(z) and g_t the gradient of the state after token t:
//   g_t = C_t dy_t + a_{t+1} g_{t+1},   a_t = exp(dt_t A),  q_t = a_t h_{t-1},  h_t = q_t + dt_t x_t B_t
//   dC_t = sum_d dy h     dB_t = sum_d g dt x      dx = Dskip dy + dt <g, B>      dDskip = sum dy x
//   ddt = <g q, A> + x <g, B>                      dA = sum_t dt g q              dinit = a_1 g_1
//   dz = dout y silu'(z), and through the dt prologue: ddt_raw = ddt sigmoid(dt_raw + bias) (0 where clamped)
//
// Three launches.  (1) states: the forward recurrence alone, which leaves the state at the start of
// every tile of T tokens in the workspace.  (2) gradients: tiles from last to first; each tile's a and h
// are recomputed into registers (64 of each) on the way forward and used on the way back, where
// g_t q_t = (a_t g_t) h_{t-1} needs no q.  (3) sums:
// partial sums to dA, dDskip, ddt_bias, dB and dC, in a fixed order, so results do not depend on
// scheduling.  Long sequences are cut into chunks as in the forward: then (1) runs every chunk from a
// zero state and also leaves what a chunk's own outputs make of the gradient at its start, and (2)
// first derives the chunk's true state and gradient at its ends from those of the other chunks.
//
// The layout is the forward's: lane = channel (CPL of them, 64 apart), wave = S of the N states.  Sums
// over states stay in the lane.  Sums over channels (dB, dC: one value of each per token and state from
// 64 lanes) are made of two sums at a time: a level adds lanes a power of two apart in both and leaves
// one in the lanes whose bit is clear, the other in those where it is set, so that after six levels a
// register holds 64 finished sums, at 2.2 vector operations for each value summed.  (The fp32 matrix
// instruction against a one-hot operand takes fewer instructions, but holds the vector pipe for all of
// its 32 cycles, and was slower.)
//
// Bound: the vector pipe, about 21 issue slots of a state of a token and channel in (2), seven in (1), and
// the tokens' own work.  4 x 2048 tokens x 4096 channels, 16 states, bf16: 183 + 425 + 10 us under the
// profiler, 572 us back to back; the registers allow (2) two waves a SIMD, which leaves about a quarter of
// its time to waits.
#include "selective_device.h"

#include <algorithm>
#include <type_traits>

namespace ssd {

// States a lane, waves, channels a lane and tokens a tile (S T CPL = 64) for N states.
template <int N> struct SelGradShape;
template <> struct SelGradShape<16> { static constexpr int S = 4, W = 4, CPL = 2, T = 8; };
template <> struct SelGradShape<32> { static constexpr int S = 8, W = 4, CPL = 1, T = 8; };
template <> struct SelGradShape<64> { static constexpr int S = 8, W = 8, CPL = 1, T = 8; };
template <> struct SelGradShape<128> { static constexpr int S = 16, W = 8, CPL = 1, T = 4; };

// Waves of the gradients launch that run at once: two for each SIMD, which is what its registers allow.
constexpr int64_t kGradWaves = 2048;

constexpr int kStatesTile = 16;   // tokens staged at a time by the states launch

// Tokens of a chunk (all L: one chunk) for `waves` waves a chunk.  One chunk takes as many rounds of
// kGradWaves as it has, of which a last one that is not full takes 0.55 to 1; chunks take a tenth more work
// and some tokens' time each, and are made so many that they fill whole rounds, one to five.  Measured, 16
// states, bf16, 4096 channels (128 waves for each batch entry): 6 x 2048 tokens 855 us in 5 chunks (1122 in 3,
// which is 1.1 rounds), 10 x 2048 1392 in 8 (1844 in one), 17 x 1024 1227 in 4 (1512 in one), 24 x 1024 1576
// in one (1602 in 2).  Chunks have 32 tokens or more (3 x 333 x 768, 32 states, fp32: 69 us, with 64 or more
// 93, with 16 or more 73; 1 x 512 x 2048: 56, 69, 60).
static int64_t grad_chunk_tokens(int64_t waves, int64_t L) {
    int64_t best = L > 0 ? L : 1;
    const double last = static_cast<double>(waves % kGradWaves) / kGradWaves;
    const double one = waves <= kGradWaves ? 1. : waves / kGradWaves + (last > 0. ? std::max(0.55, 0.2 + 0.8 * last) : 0.);
    double least = one * (best + 16);
    for (int rounds = 1; waves > 0 && rounds <= 5; ++rounds) {
        int64_t n = rounds * kGradWaves / waves;
        if (n > most_chunks(L)) n = most_chunks(L);
        if (n < 2) continue;
        const int64_t tokens = ((L + n - 1) / n + kStatesTile - 1) / kStatesTile * kStatesTile;
        const double cost = 1.1 * rounds * (tokens + 16);
        if (cost < least) {
            least = cost;
            best = tokens;
        }
    }
    return best;
}

// Offsets in floats of the workspace's parts, and the chunks.
struct SelBwdLayout {
    int64_t ckpt, tsum, ends, grads, csum, dA, dD, dbias, dBC, total;
    int64_t tiles, blocks;   // tiles of a sequence; channel blocks of the gradients launch
    int64_t tokens;          // of a chunk
    int chunks;
};

template <int N>
static SelBwdLayout layout_n(int64_t batch, int64_t L, int64_t D, int64_t G) {
    typedef SelGradShape<N> Z;
    SelBwdLayout l;
    l.tiles = (L + Z::T - 1) / Z::T;
    l.blocks = G * ((D / G + 64 * Z::CPL - 1) / (64 * Z::CPL));
    l.tokens = grad_chunk_tokens(batch * l.blocks * Z::W, L);
    l.chunks = static_cast<int>(L > 0 ? (L + l.tokens - 1) / l.tokens : 1);
    int64_t at = 0;
    auto take = [&](int64_t n) {
        const int64_t o = at;
        at += (n + 3) & ~INT64_C(3);
        return o;
    };
    const bool split = l.chunks > 1;
    l.ckpt = take(batch * l.tiles * N * D);
    l.tsum = take(split ? batch * l.tiles * D : 0);
    l.ends = take(split ? batch * l.chunks * N * D : 0);
    l.grads = take(split ? batch * l.chunks * N * D : 0);
    l.csum = take(split ? batch * l.chunks * D : 0);
    l.dA = take(batch * l.chunks * N * D);
    l.dD = take(batch * l.chunks * D);
    l.dbias = take(batch * l.chunks * D);
    l.dBC = take(l.blocks * batch * L * 2 * N);
    l.total = at;
    return l;
}
static SelBwdLayout bwd_layout(int64_t batch, int64_t L, int64_t D, int64_t G, int64_t N) {
    switch (N) {
        case 16: return layout_n<16>(batch, L, D, G);
        case 32: return layout_n<32>(batch, L, D, G);
        case 64: return layout_n<64>(batch, L, D, G);
        default: return layout_n<128>(batch, L, D, G);
    }
}

// Level LEVEL of the lane sums: adds lanes 2^(5 - LEVEL) apart of a and of b; a's sums are left in the
// lanes whose bit 5 - LEVEL is clear, b's in the others.
template <int LEVEL>
__device__ __forceinline__ float merge_sums(float a, float b, int lane) {
    if constexpr (LEVEL == 0) {
        const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false);
        return __uint_as_float(r[0]) + __uint_as_float(r[1]);
    } else if constexpr (LEVEL == 1) {
        const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false, false);
        return __uint_as_float(r[0]) + __uint_as_float(r[1]);
    } else {
        // row_ror:8, row_half_mirror, quad_perm [2,3,0,1], quad_perm [1,0,3,2]: the mirror pairs other lanes
        // than 4 apart, but each of one half of the eight with one of the other, which is what the sum needs
        constexpr int ctrl = LEVEL == 2 ? 0x128 : LEVEL == 3 ? 0x141 : LEVEL == 4 ? 0x4E : 0xB1;
        const float x = a + dpp_f<ctrl, 0xF>(a), y = b + dpp_f<ctrl, 0xF>(b);
        return (lane >> (5 - LEVEL)) & 1 ? y : x;
    }
}
// Levels FROM, FROM + 1, ... over K registers, until one is left.
template <int FROM, int K>
__device__ __forceinline__ float merge_all(const float (&v)[K], int lane) {
    if constexpr (K == 1) {
        return v[0];
    } else {
        float r[K / 2];
#pragma unroll
        for (int i = 0; i < K / 2; ++i) r[i] = merge_sums<FROM>(v[2 * i], v[2 * i + 1], lane);
        return merge_all<FROM + 1>(r, lane);
    }
}
constexpr int ilog2(int n) { return n <= 1 ? 0 : 1 + ilog2(n / 2); }

// (1) SPLIT: chunks from a zero state, with the sums of dt and the gradients at their starts.
template <typename T_, typename TY, int S, int W, int T, bool SPLIT, bool GATE>
__global__ __launch_bounds__(64 * W) void selective_states_kernel(SelBwdArgs a, float* ws, SelBwdLayout lay) {
    constexpr int N = S * W, TPT = kStatesTile / W, E = sizeof(T_);
    constexpr int SUB = SelRows<T_, S>::n;
    __shared__ float2 st[2][kStatesTile][64];
    __shared__ float sdy[SPLIT ? 2 : 1][SPLIT ? kStatesTile : 1][64];
    const int64_t per_chunk = a.batch * sel_blocks(a.channels, a.ngroups);
    const int chunk = static_cast<int>(blockIdx.x / per_chunk);
    const SelBlock k = sel_block(blockIdx.x % per_chunk, a.channels, a.ngroups);
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = k.c0 + lane;
    const bool ok = c < k.cend;
    const int cs = ok ? c : k.c0;
    const int64_t D = a.channels;
    const int64_t r0 = k.b * a.seqlen + chunk * lay.tokens, left = a.seqlen - chunk * lay.tokens;
    const int L = static_cast<int>(left < lay.tokens ? left : lay.tokens);
    const char* xp = static_cast<const char*>(a.x) + (r0 * a.x_row_stride + k.c0) * E;
    const char* dp = static_cast<const char*>(a.dt) + (r0 * D + k.c0) * E;
    const char* zp = SPLIT && GATE ? static_cast<const char*>(a.z) + (r0 * a.z_row_stride + k.c0) * E : nullptr;
    const char* gp = SPLIT ? static_cast<const char*>(a.dy) + (r0 * D + k.c0) * sizeof(TY) : nullptr;
    const char* Bp = static_cast<const char*>(a.B) + (r0 * a.bc_row_stride + k.g * N + w * S) * E;
    const char* Cp = static_cast<const char*>(a.C) + (r0 * a.bc_row_stride + k.g * N + w * S) * E;
    const uint32_t xs = static_cast<uint32_t>(a.x_row_stride) * E, zs = static_cast<uint32_t>(a.z_row_stride) * E;
    const uint32_t ds = static_cast<uint32_t>(D) * E, gs = static_cast<uint32_t>(D) * sizeof(TY);
    const uint32_t bs = static_cast<uint32_t>(a.bc_row_stride) * E;
    const uint32_t le = (cs - k.c0) * E, ge = (cs - k.c0) * sizeof(TY);
    const SelDt dtp{a.dtp.bias ? a.dtp.bias[cs] : 0.f, a.dtp.lo, a.dtp.hi, a.dtp.softplus};
    float A2[S], h[S], p[S], gr[S], dsum = 0.f;
#pragma unroll
    for (int s = 0; s < S; ++s) {
        A2[s] = base2_rate(a.A[static_cast<int64_t>(cs) * N + w * S + s]);
        h[s] = !SPLIT && a.init_state ? a.init_state[(k.b * D + cs) * N + w * S + s] : 0.f;
        p[s] = 1.f;
        gr[s] = 0.f;
    }
    T_ xr[TPT], dr[TPT], zr[TPT];
    TY gv[TPT];
    uint32_t ahead = 0;
    auto load = [&](int first, int last) {
#pragma unroll
        for (int i = 0; i < TPT; ++i) {
            const uint32_t t = static_cast<uint32_t>(first + w + W * i < last ? first + w + W * i : last);
            xr[i] = *reinterpret_cast<const T_*>(xp + (le + t * xs));
            dr[i] = *reinterpret_cast<const T_*>(dp + (le + t * ds));
            if constexpr (SPLIT) gv[i] = *reinterpret_cast<const TY*>(gp + (ge + t * gs));
            if constexpr (SPLIT && GATE) zr[i] = *reinterpret_cast<const T_*>(zp + (le + t * zs));
        }
        const uint32_t t = static_cast<uint32_t>(first + (lane & 15) < last ? first + (lane & 15) : last);
        ahead = *reinterpret_cast<const uint32_t*>((SPLIT && (lane & 16) ? Cp : Bp) + static_cast<uint64_t>(t * bs));
    };
    SelRows<T_, S> rows[2];
    float2 d[2][SUB];
    float y[2][SUB];
    load(0, L - 1);
    rows[0].template load<SPLIT>(Bp, Cp, bs, 0, L - 1);
    float* cp = ws + lay.ckpt + ((k.b * lay.tiles + chunk * (lay.tokens / T)) * N + w * S) * D + cs;
    float* tp = ws + lay.tsum + (k.b * lay.tiles + chunk * (lay.tokens / T)) * D + cs;
    int buf = 0;
    for (int t0 = 0; t0 < L; t0 += kStatesTile, buf ^= 1) {
        const int last = L - 1 - t0;
        float xn[TPT], dn[TPT], yn[TPT];
#pragma unroll
        for (int i = 0; i < TPT; ++i) {
            xn[i] = static_cast<float>(xr[i]);
            dn[i] = static_cast<float>(dr[i]);
            yn[i] = 0.f;
            if constexpr (SPLIT) yn[i] = static_cast<float>(gv[i]);
            if constexpr (SPLIT && GATE) yn[i] *= silu_f(static_cast<float>(zr[i]));
        }
        asm volatile("" ::"v"(ahead));
        sel_dts(dn, dtp);
        if (last < kStatesTile - 1)
#pragma unroll
            for (int i = 0; i < TPT; ++i)
                if (w + W * i > last) xn[i] = dn[i] = yn[i] = 0.f;
#pragma unroll
        for (int i = 0; i < TPT; ++i) {
            st[buf][w + W * i][lane] = make_float2(dn[i], dn[i] * xn[i]);
            if constexpr (SPLIT) sdy[buf][w + W * i][lane] = yn[i];
        }
        __syncthreads();
        load(kStatesTile, last);
#pragma unroll
        for (int t = 0; t < SUB; ++t) {
            d[0][t] = st[buf][t][lane];
            if constexpr (SPLIT) y[0][t] = sdy[buf][t][lane];
        }
        // the first chunk's gradient at its start is nobody's
        auto tile = [&](auto with_g) {
            constexpr bool WITH_G = decltype(with_g)::value;
#pragma unroll
            for (int u = 0; u < kStatesTile; u += SUB) {
                const int at = (u / SUB) & 1;
                rows[at ^ 1].template load<SPLIT>(Bp, Cp, bs, u + SUB, last);
                if (u + SUB < kStatesTile)
#pragma unroll
                    for (int t = 0; t < SUB; ++t) {
                        d[at ^ 1][t] = st[buf][u + SUB + t][lane];
                        if constexpr (SPLIT) y[at ^ 1][t] = sdy[buf][u + SUB + t][lane];
                    }
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int t = 0; t < SUB; ++t) {
                    if ((u + t) % T == 0 && u + t <= last) {
                        // the state at the start of a tile, and the chunk's sum of dt before it
                        if (ok) {
                            int64_t row = D;
                            asm volatile("" : "+s"(row));   // rows' offsets are made here, not kept over the loop
#pragma unroll
                            for (int s = 0; s < S; ++s) cp[static_cast<int64_t>((u + t) / T * N + s) * row] = h[s];
                            if (SPLIT && w == 0) tp[static_cast<int64_t>((u + t) / T) * row] = dsum;
                        }
                    }
                    if constexpr (SPLIT) dsum += d[at][t].x;
#pragma unroll
                    for (int s = 0; s < S; ++s) {
                        const float e = __builtin_amdgcn_exp2f(d[at][t].x * A2[s]);
                        h[s] = fmaf(e, h[s], d[at][t].y * rows[at].b(t, s));
                        if constexpr (WITH_G) {
                            p[s] *= e;
                            gr[s] = fmaf(p[s], rows[at].c(t, s) * y[at][t], gr[s]);
                            // added here and not, as the compiler would have it, after the next tile's stores
                            asm volatile("" : "+v"(gr[s]));
                        }
                    }
                }
            }
        };
        if (SPLIT && chunk > 0) tile(std::integral_constant<bool, SPLIT>{});
        else tile(std::false_type{});
        xp += static_cast<int64_t>(kStatesTile) * xs;
        dp += static_cast<int64_t>(kStatesTile) * ds;
        if constexpr (SPLIT) gp += static_cast<int64_t>(kStatesTile) * gs;
        if constexpr (SPLIT && GATE) zp += static_cast<int64_t>(kStatesTile) * zs;
        Bp += static_cast<int64_t>(kStatesTile) * bs;
        Cp += static_cast<int64_t>(kStatesTile) * bs;
        cp += static_cast<int64_t>(kStatesTile / T) * N * D;
        tp += static_cast<int64_t>(kStatesTile / T) * D;
    }
    if (SPLIT && ok) {
        const int64_t bc = k.b * lay.chunks + chunk;
#pragma unroll
        for (int s = 0; s < S; ++s) {
            ws[lay.ends + (bc * N + w * S + s) * D + c] = h[s];
            ws[lay.grads + (bc * N + w * S + s) * D + c] = gr[s];
        }
        if (w == 0) ws[lay.csum + bc * D + c] = dsum;
    }
}

// What a thread keeps of its own (token, channel) from before the scan of the tile until after it: x, the
// derivative of the dt prologue, and dout silu'(z).
template <bool GATE> struct SelKeep { float x, ddt, dz; };
template <> struct SelKeep<false> { float x, ddt; };

// The kernel's arguments read from memory again wherever this is called: kept in scalar registers over
// the gradients kernel's loop, they would be moved to and from vector registers lane by lane.
typedef const SelBwdArgs __attribute__((address_space(4)))* SelBwdArgsPtr;
__device__ __forceinline__ SelBwdArgsPtr reread_args() {
    SelBwdArgsPtr p = (SelBwdArgsPtr)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(p));
    return p;
}

// (2)
template <typename T_, typename TY, int N, bool SPLIT, bool GATE>
__global__ __launch_bounds__(64 * SelGradShape<N>::W, 2) void selective_grad_kernel(SelBwdArgs a, float* ws, SelBwdLayout lay) {
    typedef SelGradShape<N> Z;
    constexpr int S = Z::S, W = Z::W, T = Z::T, P = Z::CPL, E = sizeof(T_);
    constexpr int TPT = (T + W - 1) / W;
    // levels of the lane sums over a token's 2 S values, tokens that share a register of finished sums
    constexpr int LV = ilog2(2 * S), TG = 64 / (2 * S);
    // sub-tiles whose B and C are in scalar registers: the whole tile where it takes 32 of them
    constexpr int SUB = 2 * T * kRowWords<T_, S> <= 32 ? T : SelRows<T_, S>::n;
    constexpr int K = T / SUB;
    __shared__ float2 st[T][P][64];         // dt, dt * x
    __shared__ float sdy[T][P][64];         // dy
    __shared__ float2 part[W][T][P][64];    // <g, B>, <g q, A2> over the wave's states
    __shared__ SelKeep<GATE> keep[T][P][64];
    __shared__ float ypart[GATE ? W : 1][GATE ? T : 1][P][64];
    const int64_t per_chunk = a.batch * lay.blocks;
    const int chunk = static_cast<int>(blockIdx.x / per_chunk);
    const int64_t bb = blockIdx.x % per_chunk, b = bb / lay.blocks;
    const int blk = static_cast<int>(bb - b * lay.blocks);
    const int cpg = a.channels / a.ngroups, bpg = (cpg + 64 * P - 1) / (64 * P);
    const int grp = blk / bpg, c0 = grp * cpg + (blk - grp * bpg) * 64 * P, cend = (grp + 1) * cpg;
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t D = a.channels;
    const int64_t r0 = b * a.seqlen + chunk * lay.tokens, left = a.seqlen - chunk * lay.tokens;
    const int L = static_cast<int>(left < lay.tokens ? left : lay.tokens);
    const int tiles = (L + T - 1) / T;
    int c[P];
    bool ok[P];
#pragma unroll
    for (int j = 0; j < P; ++j) {
        ok[j] = c0 + 64 * j + lane < cend;
        c[j] = ok[j] ? c0 + 64 * j + lane : c0;   // lanes past the group: that channel's data, zero inputs, no stores
    }
    const uint32_t bs = static_cast<uint32_t>(a.bc_row_stride) * E;
    const int64_t tile0 = b * lay.tiles + chunk * (lay.tokens / T);
    const bool ragged = c0 + 64 * P > cend;   // some lanes have no channel
    float bias[P], Dv[P], A2[P][S], dA[P][S], carry[P][S], hin[SPLIT ? P : 1][S], dDv[P], dbv[P];
#pragma unroll
    for (int j = 0; j < P; ++j) {
        bias[j] = a.dtp.bias ? a.dtp.bias[c[j]] : 0.f;
        Dv[j] = a.D ? a.D[c[j]] : 0.f;
        dDv[j] = dbv[j] = 0.f;
        const int64_t so = (b * D + c[j]) * N + w * S;
#pragma unroll
        for (int s = 0; s < S; ++s) {
            A2[j][s] = base2_rate(a.A[static_cast<int64_t>(c[j]) * N + w * S + s]);
            dA[j][s] = 0.f;
            carry[j][s] = a.dfinal_state && ok[j] ? a.dfinal_state[so + s] : 0.f;
            if constexpr (SPLIT) hin[j][s] = a.init_state ? a.init_state[so + s] : 0.f;
        }
        if constexpr (SPLIT) {
            const float *sums = ws + lay.csum + b * lay.chunks * D + c[j], *ends = ws + lay.ends + (b * lay.chunks * N + w * S) * D + c[j];
            const float* grads = ws + lay.grads + (b * lay.chunks * N + w * S) * D + c[j];
            join_chunks(hin[j], A2[j], sums, ends, 0, chunk, 1, D, N * D, D);
            join_chunks(carry[j], A2[j], sums, grads, lay.chunks - 1, lay.chunks - 1 - chunk, -1, D, N * D, D);
#pragma unroll
            for (int s = 0; s < S; ++s)
                if (!ok[j]) carry[j][s] = 0.f;
        }
    }
    T_ xr[TPT][P], dr[TPT][P], zr[TPT][P];   // the next tile's values as loaded
    TY gv[TPT][P];
    auto load = [&](int tile) {   // this thread's tokens w + W i of a tile, none past the chunk's last
        const SelBwdArgsPtr ka = reread_args();
        const int64_t row = r0 + tile * T;
        const int last = L - 1 - tile * T;
        const char* xp = static_cast<const char*>(ka->x) + row * ka->x_row_stride * E;
        const char* dp = static_cast<const char*>(ka->dt) + row * D * E;
        const char* gp = static_cast<const char*>(ka->dy) + row * D * sizeof(TY);
        const char* zp = GATE ? static_cast<const char*>(ka->z) + row * ka->z_row_stride * E : nullptr;
        const uint32_t xs = static_cast<uint32_t>(ka->x_row_stride) * E, zs = static_cast<uint32_t>(ka->z_row_stride) * E;
        const uint32_t ds = static_cast<uint32_t>(D) * E, gs = static_cast<uint32_t>(D) * sizeof(TY);
#pragma unroll
        for (int i = 0; i < TPT; ++i) {
            const uint32_t t = w + W * i < last ? w + W * i : last;
#pragma unroll
            for (int j = 0; j < P; ++j) {
                const uint32_t o = static_cast<uint32_t>(c[j]) * E;
                xr[i][j] = *reinterpret_cast<const T_*>(xp + (o + t * xs));
                dr[i][j] = *reinterpret_cast<const T_*>(dp + (o + t * ds));
                gv[i][j] = *reinterpret_cast<const TY*>(gp + (static_cast<uint32_t>(c[j]) * static_cast<uint32_t>(sizeof(TY)) + t * gs));
                if constexpr (GATE) zr[i][j] = *reinterpret_cast<const T_*>(zp + (o + t * zs));
            }
        }
    };
    float h[P][S], ts[P];
    auto load_state = [&](int tile) {
#pragma unroll
        for (int j = 0; j < P; ++j) {
            if constexpr (SPLIT) ts[j] = ws[lay.tsum + (tile0 + tile) * D + c[j]];
#pragma unroll
            for (int s = 0; s < S; ++s) h[j][s] = ws[lay.ckpt + ((tile0 + tile) * N + w * S + s) * D + c[j]];
        }
    };
    auto row_of = [&](const void* p, int tile) {   // this wave's states of the tile's first row of B or C
        return static_cast<const char*>(p) + ((r0 + tile * T) * a.bc_row_stride + grp * N + w * S) * E;
    };
    SelRows<T_, S, SUB> rows[2];
    if (tiles > 0) {
        load(tiles - 1);
        load_state(tiles - 1);
        rows[0].template load<true>(row_of(a.B, tiles - 1), row_of(a.C, tiles - 1), bs, 0, L - 1 - (tiles - 1) * T);
    }
    for (int tile = tiles - 1; tile >= 0; --tile) {
        const int last = L - 1 - tile * T;   // the tile's last row, if below T - 1
        const SelBwdArgsPtr kb = reread_args();
        const char *Bp = row_of(kb->B, tile), *Cp = row_of(kb->C, tile);
        float dt[TPT][P], slope[TPT][P], x[TPT][P], dy[TPT][P], dz[TPT][P];
#pragma unroll
        for (int i = 0; i < TPT; ++i)
#pragma unroll
            for (int j = 0; j < P; ++j) {
                x[i][j] = static_cast<float>(xr[i][j]);
                dt[i][j] = static_cast<float>(dr[i][j]) + bias[j];
                dy[i][j] = static_cast<float>(gv[i][j]);
                slope[i][j] = 1.f;
                dz[i][j] = 0.f;
                if constexpr (GATE) {
                    const float z = static_cast<float>(zr[i][j]), sg = sel_sigmoid(z);
                    dz[i][j] = dy[i][j] * sg * fmaf(z, 1.f - sg, 1.f);
                    dy[i][j] *= z * sg;
                }
            }
        if (a.dtp.softplus)
#pragma unroll
            for (int i = 0; i < TPT; ++i)
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    slope[i][j] = sel_sigmoid(dt[i][j]);
                    dt[i][j] = sel_softplus(dt[i][j]);
                }
        if (a.dtp.lo < a.dtp.hi)
#pragma unroll
            for (int i = 0; i < TPT; ++i)
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    if (!(dt[i][j] >= a.dtp.lo && dt[i][j] <= a.dtp.hi)) slope[i][j] = 0.f;
                    dt[i][j] = fminf(fmaxf(dt[i][j], a.dtp.lo), a.dtp.hi);
                }
        if (ragged || last < T - 1)   // no token or no channel there: nothing enters any sum
#pragma unroll
            for (int i = 0; i < TPT; ++i)
#pragma unroll
                for (int j = 0; j < P; ++j)
                    if (w + W * i > last || !ok[j]) x[i][j] = dt[i][j] = dy[i][j] = dz[i][j] = slope[i][j] = 0.f;
#pragma unroll
        for (int i = 0; i < TPT; ++i) {
            const int t = w + W * i;
            if (T % W != 0 && t >= T) continue;
#pragma unroll
            for (int j = 0; j < P; ++j) {
                keep[t][j][lane].x = x[i][j];
                keep[t][j][lane].ddt = slope[i][j];
                if constexpr (GATE) keep[t][j][lane].dz = dz[i][j];
                st[t][j][lane] = make_float2(dt[i][j], dt[i][j] * x[i][j]);
                sdy[t][j][lane] = dy[i][j];
            }
        }
        if constexpr (SPLIT)
#pragma unroll
            for (int j = 0; j < P; ++j)
#pragma unroll
                for (int s = 0; s < S; ++s) h[j][s] = fmaf(__builtin_amdgcn_exp2f(ts[j] * A2[j][s]), hin[j][s], h[j][s]);
        __syncthreads();
        // states before each token and after the last; decays, which 16 states a lane leave no registers
        // for: there the way back computes them again
        constexpr bool KEEP = S < 16;
        float hs[T + 1][P][S], ea[KEEP ? T : 1][P][S];
#pragma unroll
        for (int j = 0; j < P; ++j)
#pragma unroll
            for (int s = 0; s < S; ++s) hs[0][j][s] = h[j][s];
        float2 dn[2][P];
#pragma unroll
        for (int j = 0; j < P; ++j) dn[0][j] = st[0][j][lane];
#pragma unroll
        for (int u = 0; u < K; ++u) {
            const int at = u & 1;
            // the way back starts with the last rows of the way forward
            if (u + 1 < K) rows[at ^ 1].template load<true>(Bp, Cp, bs, (u + 1) * SUB, last);
#pragma unroll
            for (int v = 0; v < SUB; ++v) {
                const int t = u * SUB + v;
                // dt and dt x are read from LDS a token ahead
                if (t + 1 < T)
#pragma unroll
                    for (int j = 0; j < P; ++j) dn[(t + 1) & 1][j] = st[t + 1][j][lane];
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    const float2 d = dn[t & 1][j];
                    float y = 0.f;
#pragma unroll
                    for (int s = 0; s < S; ++s) {
                        const float e = __builtin_amdgcn_exp2f(d.x * A2[j][s]);
                        if constexpr (KEEP) ea[t][j][s] = e;
                        hs[t + 1][j][s] = fmaf(e, hs[t][j][s], d.y * rows[at].b(v, s));
                        if constexpr (GATE) y = fmaf(hs[t + 1][j][s], rows[at].c(v, s), y);
                    }
                    if constexpr (GATE) ypart[w][t][j][lane] = y;
                }
            }
        }
        float yn[2][P];
#pragma unroll
        for (int j = 0; j < P; ++j) yn[(T - 1) & 1][j] = sdy[T - 1][j][lane];
        rows[(K - 1) & 1].renew();
        float tok[T];
#pragma unroll
        for (int u = K - 1; u >= 0; --u) {
            const int at = u & 1;
            if (u > 0) rows[at ^ 1].template load<true>(Bp, Cp, bs, (u - 1) * SUB, last);
#pragma unroll
            for (int v = SUB - 1; v >= 0; --v) {
                const int t = u * SUB + v;
                if (t > 0)
#pragma unroll
                    for (int j = 0; j < P; ++j) {
                        dn[(t - 1) & 1][j] = st[t - 1][j][lane];
                        yn[(t - 1) & 1][j] = sdy[t - 1][j][lane];
                    }
                __builtin_amdgcn_sched_barrier(0);
                float pB[S], pC[S];
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    const float2 d = dn[t & 1][j];
                    const float dy = yn[t & 1][j];
                    float gB = 0.f, gA = 0.f;
#pragma unroll
                    for (int s = 0; s < S; ++s) {
                        const float g = fmaf(rows[at].c(v, s), dy, carry[j][s]);
                        pB[s] = j == 0 ? g * d.y : fmaf(g, d.y, pB[s]);
                        pC[s] = j == 0 ? dy * hs[t + 1][j][s] : fmaf(dy, hs[t + 1][j][s], pC[s]);
                        gB = fmaf(g, rows[at].b(v, s), gB);
                        carry[j][s] = (KEEP ? ea[KEEP ? t : 0][j][s] : __builtin_amdgcn_exp2f(d.x * A2[j][s])) * g;
                        const float x = carry[j][s] * hs[t][j][s];
                        dA[j][s] = fmaf(d.x, x, dA[j][s]);
                        gA = fmaf(A2[j][s], x, gA);
                    }
                    part[w][t][j][lane] = make_float2(gB, gA);
                }
                float vals[2 * S];
#pragma unroll
                for (int s = 0; s < S; ++s) {
                    vals[s] = pB[s];
                    vals[S + s] = pC[s];
                }
                tok[t] = merge_all<0>(vals, lane);
                if (t == T - 1) {   // the next tile's loads, once the last token's state and decay are free
                    load(tile > 0 ? tile - 1 : 0);
                    load_state(tile > 0 ? tile - 1 : 0);
                }
            }
        }
        // dA's products are added here and not, as the compiler would have it, after the next barrier
#pragma unroll
        for (int j = 0; j < P; ++j)
#pragma unroll
            for (int s = 0; s < S; ++s) asm volatile("" : "+v"(dA[j][s]));
        // lane bits 5, 4, ...: the value's bits 0, 1, ... (dB's S states, then dC's), then the token's
        float* bcp = ws + lay.dBC + (static_cast<int64_t>(blk) * a.batch * a.seqlen + r0 + tile * T) * 2 * N + w * S;
        const int rev = static_cast<int>(__brev(static_cast<uint32_t>(lane)) >> 26), val = rev & (2 * S - 1), tt = rev >> LV;
#pragma unroll
        for (int g = 0; g < T / TG; ++g) {
            float group[TG];
#pragma unroll
            for (int i = 0; i < TG; ++i) group[i] = tok[g * TG + i];
            const float v = merge_all<LV>(group, lane);
            const int t = g * TG + tt;
            if (t <= last) bcp[static_cast<uint32_t>(t * 2 * N + val / S * N + val % S)] = v;
        }
        __syncthreads();
        const SelBwdArgsPtr ka = reread_args();
        if (T % W == 0 || w < T) {
            float gB[TPT][P], gA[TPT][P], y[TPT][P], dx[TPT][P], dd[TPT][P];
#pragma unroll
            for (int i = 0; i < TPT; ++i)
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    const int t = w + W * i;
                    gB[i][j] = gA[i][j] = y[i][j] = 0.f;
#pragma unroll
                    for (int u = 0; u < W; ++u) {
                        const float2 pp = part[u][t][j][lane];
                        gB[i][j] += pp.x;
                        gA[i][j] += pp.y;
                        if constexpr (GATE) y[i][j] += ypart[u][t][j][lane];
                    }
                }
#pragma unroll
            for (int i = 0; i < TPT; ++i)
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    const int t = w + W * i;
                    const SelKeep<GATE> r = keep[t][j][lane];
                    const float dy = sdy[t][j][lane];
                    dx[i][j] = fmaf(Dv[j], dy, st[t][j][lane].x * gB[i][j]);
                    dd[i][j] = fmaf(gA[i][j], 1.f / kLog2e, r.x * gB[i][j]) * r.ddt;
                    dbv[j] += dd[i][j];
                    dDv[j] = fmaf(dy, r.x, dDv[j]);
                    if constexpr (GATE) y[i][j] = r.dz * fmaf(Dv[j], r.x, y[i][j]);
                }
            const int64_t out = (r0 + tile * T) * D * E;
            char *dxp = static_cast<char*>(ka->dx) + out, *ddp = static_cast<char*>(ka->ddt) + out;
            char* dzp = GATE ? static_cast<char*>(ka->dz) + out : nullptr;
            const uint32_t ds = static_cast<uint32_t>(D) * E;
#pragma unroll
            for (int j = 0; j < P; ++j) {
                const uint32_t o = static_cast<uint32_t>(c[j]) * E;
                auto store = [&](int i) {
                    const uint32_t at = o + static_cast<uint32_t>(w + W * i) * ds;
                    *reinterpret_cast<T_*>(dxp + at) = static_cast<T_>(dx[i][j]);
                    *reinterpret_cast<T_*>(ddp + at) = static_cast<T_>(dd[i][j]);
                    if constexpr (GATE) *reinterpret_cast<T_*>(dzp + at) = static_cast<T_>(y[i][j]);
                };
                if (!ragged && last >= T - 1) {
#pragma unroll
                    for (int i = 0; i < TPT; ++i) store(i);
                } else if (ok[j]) {
#pragma unroll
                    for (int i = 0; i < TPT; ++i)
                        if (w + W * i <= last) store(i);
                }
            }
        }
        if (tile > 0) rows[0].template load<true>(row_of(ka->B, tile - 1), row_of(ka->C, tile - 1), bs, 0, T - 1);
        __syncthreads();
    }
    const int64_t bc = b * lay.chunks + chunk;
#pragma unroll
    for (int j = 0; j < P; ++j) {
        part[w][0][j][lane] = make_float2(dDv[j], dbv[j]);   // the last tile ended with a barrier
        if (!ok[j]) continue;
#pragma unroll
        for (int s = 0; s < S; ++s) {
            ws[lay.dA + (bc * N + w * S + s) * D + c[j]] = dA[j][s];
            if (a.dinit_state && chunk == 0) a.dinit_state[(b * D + c[j]) * N + w * S + s] = carry[j][s];
        }
    }
    __syncthreads();
    if (w == 0)
#pragma unroll
        for (int j = 0; j < P; ++j) {
            if (!ok[j]) continue;
            float u = 0.f, v = 0.f;
#pragma unroll
            for (int i = 0; i < W; ++i) {
                u += part[i][0][j][lane].x;
                v += part[i][0][j][lane].y;
            }
            ws[lay.dD + bc * D + c[j]] = u;
            ws[lay.dbias + bc * D + c[j]] = v;
        }
}

// (3) D N values of dA, D of dDskip and of ddt_bias over batch and chunks, and B L G N values of dB and
// of dC over the group's channel blocks.
template <typename T>
__global__ __launch_bounds__(256) void selective_sums_kernel(SelBwdArgs a, const float* __restrict__ ws, SelBwdLayout lay) {
    const int64_t D = a.channels, N = a.d_state, G = a.ngroups, rows = a.batch * a.seqlen;
    int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i < (N + 2) * D) {
        const float* p = ws + (i < N * D ? lay.dA + i : i < (N + 1) * D ? lay.dD + i - N * D : lay.dbias + i - (N + 1) * D);
        const int64_t step = i < N * D ? N * D : D;
        float v = 0.f;
        for (int64_t b = 0; b < a.batch * lay.chunks; ++b) v += p[b * step];
        if (i < N * D) a.dA[i % D * N + i / D] = v;
        else if (i < (N + 1) * D) { if (a.dD) a.dD[i - N * D] = v; }
        else if (a.ddt_bias) a.ddt_bias[i - (N + 1) * D] = v;
        return;
    }
    i = 4 * (i - (N + 2) * D);   // four values a thread: N is a multiple of 4
    if (i >= rows * 2 * G * N) return;
    const int64_t n = i % N, which = i / N % 2, g = i / (2 * N) % G, row = i / (2 * N * G);
    const int64_t per = lay.blocks / G;
    const float* p = ws + lay.dBC + (g * per * rows + row) * 2 * N + which * N + n;
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
    for (int64_t k = 0; k < per; ++k) v += *reinterpret_cast<const f32x4*>(p + k * rows * 2 * N);
    T* o = (which ? static_cast<T*>(a.dC) : static_cast<T*>(a.dB)) + (row * G + g) * N + n;
#pragma unroll
    for (int k = 0; k < 4; ++k) o[k] = static_cast<T>(v[k]);
}

template <typename T, typename TY, int N, bool SPLIT, bool GATE>
static void bwd_main(const SelBwdArgs& a, float* ws, const SelBwdLayout& lay, hipStream_t s) {
    typedef SelGradShape<N> Z;
    constexpr int W = N == 128 ? 8 : 4, S = N / W;   // the states launch's waves and states a lane
    const dim3 g1(static_cast<uint32_t>(a.batch * sel_blocks(a.channels, a.ngroups) * lay.chunks));
    const dim3 g2(static_cast<uint32_t>(a.batch * lay.blocks * lay.chunks));
    if (a.seqlen > 0)
        hipLaunchKernelGGL((selective_states_kernel<T, TY, S, W, Z::T, SPLIT, GATE>), g1, dim3(64 * W), 0, s, a, ws, lay);
    hipLaunchKernelGGL((selective_grad_kernel<T, TY, N, SPLIT, GATE>), g2, dim3(64 * Z::W), 0, s, a, ws, lay);
}

template <typename T, typename TY, int N>
static hipError_t bwd_n(const SelBwdArgs& a, float* ws, hipStream_t s) {
    const SelBwdLayout lay = bwd_layout(a.batch, a.seqlen, a.channels, a.ngroups, a.d_state);
    if (a.batch > 0) {
        if (lay.chunks > 1) a.z ? bwd_main<T, TY, N, true, true>(a, ws, lay, s) : bwd_main<T, TY, N, true, false>(a, ws, lay, s);
        else a.z ? bwd_main<T, TY, N, false, true>(a, ws, lay, s) : bwd_main<T, TY, N, false, false>(a, ws, lay, s);
    }
    const int64_t n = (a.d_state + 2) * static_cast<int64_t>(a.channels) + a.batch * a.seqlen * a.ngroups * a.d_state / 2;
    hipLaunchKernelGGL((selective_sums_kernel<T>), dim3(static_cast<uint32_t>((n + 255) / 256)), dim3(256), 0, s, a, ws, lay);
    return hipGetLastError();
}

template <typename T, typename TY>
static hipError_t bwd_t(const SelBwdArgs& a, float* ws, hipStream_t s) {
    switch (a.d_state) {
        case 16: return bwd_n<T, TY, 16>(a, ws, s);
        case 32: return bwd_n<T, TY, 32>(a, ws, s);
        case 64: return bwd_n<T, TY, 64>(a, ws, s);
        case 128: return bwd_n<T, TY, 128>(a, ws, s);
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
