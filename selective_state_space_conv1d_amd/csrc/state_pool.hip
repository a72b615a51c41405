// Slots of state pools: copied (restored from a snapshot pool, forked), cleared, and the plan that
// compacts a pool ("MAX 平台 Nemotron-H 混合架构解析", 5.4: states live in pool slots that the kernels
// address directly; the modeling_nemotron_h.py walk-through, 部署时如何调这些缓存: snapshots for prefix
// caching).  Copying reads and writes each slot's bytes once: an HBM stream of 16-byte accesses.
#include "ssd_device.h"
#include "ssd_kernels.h"

namespace ssd {

constexpr int kPoolThreads = 256;
constexpr int kPoolFlight = 8;   // 16-byte loads in flight per thread
constexpr int64_t kPoolSpan = static_cast<int64_t>(kPoolThreads) * kPoolFlight * 16;   // bytes of a slot per workgroup

// Entries take effect in their order: an entry whose source is an earlier entry's destination copies
// what that entry left, and of two entries with one destination the later one stays.  Workgroups that
// each copy one entry keep to that when no destination occurs twice and none is another entry's
// source.  Every workgroup tests this on a bitmap of the destinations (slot mod 131072: slots that share a
// bit count as equal, which is on the safe side); when the test fails the workgroups of entry 0 copy
// all entries one after the other, each thread its own bytes, and the others leave.  The bitmap takes
// 16 KiB of LDS, which leaves room for the eight workgroups that a CU holds.
constexpr int kPoolBits = 131072;

__global__ __launch_bounds__(kPoolThreads) void pool_copy_kernel(PoolCopyArgs a, int64_t spans) {
    __shared__ uint32_t seen[kPoolBits / 32];
    __shared__ int ordered;
    const int64_t e0 = blockIdx.x / spans, span = blockIdx.x % spans;
    const bool same = a.src == a.dst && a.src_layer_bytes == a.dst_layer_bytes;
    auto dst_of = [&](int64_t e) -> int64_t {
        const int64_t d = a.dst_idx[e];
        return d >= 0 && d < a.dst_slots ? d : -1;
    };
    auto src_of = [&](int64_t e) -> int64_t {
        const int64_t s = a.src_idx[e];
        return s >= 0 && s < a.src_slots ? s : -1;
    };
    if (a.src && a.n > 1) {   // clearing a slot twice clears it
        const int words = static_cast<int>(((a.dst_slots < kPoolBits ? a.dst_slots : kPoolBits) + 31) / 32);
        for (int i = threadIdx.x; i < words; i += kPoolThreads) seen[i] = 0;
        if (threadIdx.x == 0) ordered = 0;
        __syncthreads();
        bool bad = false;
        for (int64_t e = threadIdx.x; e < a.n; e += kPoolThreads) {
            const int64_t d = dst_of(e), s = src_of(e);
            if (d < 0 || s < 0 || (same && d == s)) continue;
            const uint32_t bit = 1u << (d & 31);
            bad |= (atomicOr(&seen[(d % kPoolBits) / 32], bit) & bit) != 0;
        }
        __syncthreads();
        if (same)
            for (int64_t e = threadIdx.x; e < a.n; e += kPoolThreads) {
                const int64_t d = dst_of(e), s = src_of(e);
                if (d < 0 || s < 0 || d == s || s >= a.dst_slots) continue;   // past dst's slots: nobody's destination
                bad |= (seen[(s % kPoolBits) / 32] >> (s & 31) & 1u) != 0;
            }
        if (bad) ordered = 1;
        __syncthreads();
        if (ordered && e0 != 0) return;
    } else if (threadIdx.x == 0) {
        ordered = 0;
    }
    __syncthreads();
    const int64_t e1 = ordered ? a.n : e0 + 1;
    char* dp = static_cast<char*>(a.dst) + blockIdx.y * a.dst_layer_bytes;
    const char* sp = static_cast<const char*>(a.src) + blockIdx.y * a.src_layer_bytes;
    const int64_t at = span * kPoolSpan + threadIdx.x * 16;
    for (int64_t e = e0; e < e1; ++e) {
        const int64_t d = dst_of(e);
        const int64_t s = a.src ? src_of(e) : 0;
        if (d < 0 || s < 0 || (a.src && same && d == s)) continue;
        u32x4 v[kPoolFlight];
#pragma unroll
        for (int i = 0; i < kPoolFlight; ++i) {
            const int64_t o = at + static_cast<int64_t>(i) * kPoolThreads * 16;
            v[i] = u32x4{0, 0, 0, 0};
            if (a.src && o < a.slot_bytes) v[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(sp + s * a.slot_bytes + o));
        }
#pragma unroll
        for (int i = 0; i < kPoolFlight; ++i) {
            const int64_t o = at + static_cast<int64_t>(i) * kPoolThreads * 16;
            if (o < a.slot_bytes) __builtin_nontemporal_store(v[i], reinterpret_cast<u32x4*>(dp + d * a.slot_bytes + o));
        }
    }
}

hipError_t launch_pool_copy(const PoolCopyArgs& a, hipStream_t s) {
    if (a.n == 0 || a.layers == 0 || a.slot_bytes == 0) return hipSuccess;
    const int64_t spans = (a.slot_bytes + kPoolSpan - 1) / kPoolSpan;
    hipLaunchKernelGGL(pool_copy_kernel, dim3(static_cast<uint32_t>(a.n * spans), static_cast<uint32_t>(a.layers)),
                       dim3(kPoolThreads), 0, s, a, spans);
    return hipGetLastError();
}

// The compaction's plan, by one workgroup: a bitmap of the live slots and, word by word, how many are
// live below.  With `count` live slots, those below count stay; the k-th live slot from count on moves
// to the k-th free slot below count.
constexpr int kPlanThreads = 1024;

__global__ __launch_bounds__(kPlanThreads) void pool_compact_kernel(const int32_t* __restrict__ slot_idx, int64_t n, int nslots,
                                                                    int32_t* src, int32_t* dst, int32_t* __restrict__ out,
                                                                    int32_t* __restrict__ count_out) {
    __shared__ uint32_t live[kPoolMaxSlots / 32];
    __shared__ int below[kPoolMaxSlots / 32];   // live slots in the words before this one
    __shared__ int wsum[kPlanThreads / 64];
    const int words = (nslots + 31) / 32, tid = threadIdx.x;
    for (int i = tid; i < words; i += kPlanThreads) live[i] = 0;
    __syncthreads();
    for (int64_t i = tid; i < n; i += kPlanThreads) {
        const int s = slot_idx[i];
        if (s >= 0 && s < nslots) atomicOr(&live[s / 32], 1u << (s & 31));
        src[i] = dst[i] = -1;
    }
    __syncthreads();
    // each thread sums a run of words, then the runs are scanned over the workgroup
    const int per = (words + kPlanThreads - 1) / kPlanThreads;
    const int w0 = tid * per < words ? tid * per : words, w1 = w0 + per < words ? w0 + per : words;
    int mine = 0;
    for (int i = w0; i < w1; ++i) mine += __popc(live[i]);
    int incl = mine;
    for (int o = 1; o < 64; o <<= 1) {
        const int v = __shfl_up(incl, o, 64);
        if ((tid & 63) >= o) incl += v;
    }
    if ((tid & 63) == 63) wsum[tid / 64] = incl;
    __syncthreads();
    int before = incl - mine, count = 0;
    for (int i = 0; i < kPlanThreads / 64; ++i) {
        if (i < tid / 64) before += wsum[i];
        count += wsum[i];
    }
    for (int i = w0; i < w1; ++i) {
        below[i] = before;
        before += __popc(live[i]);
    }
    __syncthreads();
    auto rank = [&](int s) { return below[s / 32] + __popc(live[s / 32] & ((1u << (s & 31)) - 1u)); };
    auto is_live = [&](int s) { return (live[s / 32] >> (s & 31) & 1u) != 0; };
    const int stay = count < nslots ? rank(count) : count;   // live slots below count
    for (int s = tid; s < nslots; s += kPlanThreads) {
        if (s < count && !is_live(s)) dst[s - rank(s)] = s;
        if (s >= count && is_live(s)) src[rank(s) - stay] = s;
    }
    __syncthreads();
    for (int64_t i = tid; i < n; i += kPlanThreads) {
        const int s = slot_idx[i];
        out[i] = s >= count && s < nslots ? dst[rank(s) - stay] : s;   // padding stays as it is
    }
    if (tid == 0) *count_out = count;
}

hipError_t launch_pool_compact(const int32_t* slot_idx, int64_t n, int64_t nslots, int32_t* src_idx, int32_t* dst_idx,
                               int32_t* new_idx, int32_t* count, hipStream_t s) {
    hipLaunchKernelGGL(pool_compact_kernel, dim3(1), dim3(kPlanThreads), 0, s, slot_idx, n, static_cast<int>(nslots), src_idx,
                       dst_idx, new_idx, count);
    return hipGetLastError();
}

}  // namespace ssd
