// expert_map.hip -- the map between routed slots and expert-ordered rows: a stable
// counting sort of the slots (slot t k + j is choice j of token t) by expert.
//
// Row order is expert, then slot, so the result does not depend on how the work is split.
// The slots are cut into chunks, one per workgroup of 16 waves: a first launch counts each
// chunk's slots per expert, a second finds every chunk's first row per expert (from all
// chunks' counts, which it reads itself, spread over its threads: a third launch for the sums
// would cost more than these reads) and ranks its own slots.  Up to kOneChunk slots one
// workgroup does all of it in one launch.  Within a workgroup a wave owns a contiguous run of
// slots; the rank of a slot among the 64 of one step is the number of earlier lanes with the
// same expert, from one ballot per bit of the expert's number.  The traffic (12 bytes a slot)
// is nothing; two launches and the steps between their barriers are the time: 1024 slots of
// 256 experts take 4.0 us in one launch (5.8 in two), 2048 5.0 (6.1), 4096 7.0 (7.1), 8192
// 11.1 (7.4); 65536 slots 7.2, 262144 12.0 with at most 64 chunks (16 chunks: 9.4, 25.6; 128:
// 7.2, 11.8), ids in the caches; behind a kernel that streams 600 MB through those 65536 slots
// take 10.
#include "lanes.h"

namespace mxfp4 {

constexpr int kMapThreads = 1024;
constexpr int kMapWaves = kMapThreads / 64;
constexpr int kMapExperts = 1024;                 // G at most
constexpr int kOneChunk = 2048;                   // slots one workgroup sorts alone
constexpr int kMaxChunks = 64;

namespace {

// Expert of a slot, G if it has none here.
__device__ __forceinline__ int local_expert(const int32_t* __restrict__ ids, uint32_t slot, int slots, int first, int G)
{
    if (slot >= (uint32_t)slots)
        return G;
    const int64_t e = (int64_t)ids[slot] - first;
    return e >= 0 && e < G ? (int)e : G;
}

}  // namespace

__global__ __launch_bounds__(kMapThreads) void expert_count_kernel(const int32_t* __restrict__ ids,
                                                                   int32_t* __restrict__ counts, int slots,
                                                                   int chunk, int first, int G)
{
    __shared__ int32_t hist[kMapExperts];
    const int tid = threadIdx.x;
    if (tid < G)
        hist[tid] = 0;
    __syncthreads();
    const int64_t from = (int64_t)blockIdx.x * chunk;
    for (int64_t s = from + tid; s < from + chunk && s < slots; s += kMapThreads) {
        const int e = local_expert(ids, (uint32_t)s, slots, first, G);
        if (e < G)
            atomicAdd(&hist[e], 1);
    }
    __syncthreads();
    if (tid < G)
        counts[(int64_t)blockIdx.x * G + tid] = hist[tid];
}

template <bool kOne>
__global__ __launch_bounds__(kMapThreads) void expert_place_kernel(
    const int32_t* __restrict__ ids, const int32_t* __restrict__ counts, int32_t* __restrict__ offs,
    int32_t* __restrict__ pos, int32_t* __restrict__ src, int slots, int chunk, int first, int G, int g_log, int cap)
{
    // per wave and expert: first its number of slots, then the row of its next slot
    __shared__ int32_t next[kMapWaves][kMapExperts];
    __shared__ int32_t sums[2][kMapThreads];      // [before this chunk, in all chunks][part][expert]
    __shared__ int32_t part[kMapWaves];
    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    for (int i = tid; i < kMapWaves << g_log; i += kMapThreads)
        next[i >> g_log][i & ((1 << g_log) - 1)] = 0;
    // all chunks' counts: thread (q, g) takes every parts-th chunk's of expert g
    const int parts = kMapThreads >> g_log;
    if constexpr (!kOne) {
        const int g = tid & ((1 << g_log) - 1), q = tid >> g_log;
        int32_t before = 0, total = 0;
        if (g < G) {
            constexpr int kAhead = 8;
            for (int b0 = q; b0 < (int)gridDim.x; b0 += kAhead * parts) {
                int32_t c[kAhead];
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    const int b = b0 + u * parts;
                    c[u] = counts[(int64_t)min(b, (int)gridDim.x - 1) * G + g];
                }
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    const int b = b0 + u * parts;
                    before += b < (int)blockIdx.x ? c[u] : 0;
                    total += b < (int)gridDim.x ? c[u] : 0;
                }
            }
        }
        sums[0][tid] = before;
        sums[1][tid] = total;
    }
    __syncthreads();
    const int run = chunk / kMapWaves;            // slots of a wave (a multiple of 64)
    const int64_t from = (int64_t)blockIdx.x * chunk + wave * run;
    const int steps = from < slots ? (int)((min((int64_t)run, slots - from) + 63) / 64) : 0;
    for (int i = 0; i < steps; ++i) {
        const int e = local_expert(ids, (uint32_t)from + 64 * i + lane, slots, first, G);
        if (e < G)
            atomicAdd(&next[wave][e], 1);
    }
    __syncthreads();
    // expert tid: rows in all chunks, rows in those before this one, and its waves' counts
    int32_t mine[kMapWaves], before = 0, total = 0;
    if (tid < G) {
#pragma unroll
        for (int w = 0; w < kMapWaves; ++w)
            mine[w] = next[w][tid];
        if constexpr (kOne) {
#pragma unroll
            for (int w = 0; w < kMapWaves; ++w)
                total += mine[w];
        } else {
            const int filled = min(parts, (int)gridDim.x);
#pragma unroll 8
            for (int q = 0; q < filled; ++q) {
                before += sums[0][(q << g_log) + tid];
                total += sums[1][(q << g_log) + tid];
            }
        }
    }
    // first row of each expert: an exclusive sum over the experts, one per thread
    int32_t incl = total;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int32_t o = __shfl_up(incl, d, 64);
        incl += lane >= d ? o : 0;
    }
    if (lane == 63)
        part[wave] = incl;
    __syncthreads();
    int32_t start = incl - total;
#pragma unroll
    for (int w = 0; w < kMapWaves; ++w)
        start += w < wave ? part[w] : 0;
    if (tid < G) {
        if (blockIdx.x == 0) {
            offs[tid] = min(start, cap);
            if (tid == G - 1)
                offs[G] = min(start + total, cap);
        }
        int32_t at = start + before;
#pragma unroll
        for (int w = 0; w < kMapWaves; ++w) {
            next[w][tid] = at;
            at += mine[w];
        }
    }
    __syncthreads();
    const int bits = 32 - __builtin_clz(G);       // 0 .. G: G stands for "none"
    for (int i = 0; i < steps; ++i) {
        const uint32_t slot = (uint32_t)from + 64 * i + lane;
        const int e = local_expert(ids, slot, slots, first, G);
        uint64_t same = ~0ull;                    // the lanes with this lane's expert
        for (int b = 0; b < bits; ++b) {
            const bool bit = e >> b & 1;
            const uint64_t m = __ballot(bit);
            same &= bit ? m : ~m;
        }
        const int rank =
            __builtin_amdgcn_mbcnt_hi((uint32_t)(same >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)same, 0));
        int32_t row = -1;
        if (e < G)
            row = next[wave][e] + rank;
        wave_lds_order();                         // every lane has read its counter
        if (e < G && rank == 0)                   // one lane per expert moves it on
            next[wave][e] = row + (int)__popcll(same);
        wave_lds_order();
        if (slot < (uint32_t)slots) {
            const bool live = row >= 0 && row < cap;
            pos[slot] = live ? row : -1;
            if (src && live)
                src[row] = (int32_t)slot;
        }
    }
}

int64_t expert_map_chunks(int64_t slots)
{
    if (slots <= kOneChunk)
        return 0;
    const int64_t n = (slots + kMapThreads - 1) / kMapThreads;
    return n < kMaxChunks ? n : kMaxChunks;
}

hipError_t launch_expert_map(const int32_t* ids, int32_t* offs, int32_t* pos, int32_t* src, int32_t* counts,
                             int64_t slots, int32_t first, int32_t G, int64_t M_cap, hipStream_t stream)
{
    const int64_t chunks = expert_map_chunks(slots);
    int64_t size = chunks > 0 ? (slots + chunks - 1) / chunks : slots;
    size = (size + kMapThreads - 1) / kMapThreads * kMapThreads;      // whole steps of every wave
    int s = (int)slots, chunk = (int)size, f = first, g = G, g_log = 0, cap = (int)M_cap;
    while (1 << g_log < G)
        ++g_log;
    if (chunks > 0) {
        void* cargs[] = {(void*)&ids, (void*)&counts, (void*)&s, (void*)&chunk, (void*)&f, (void*)&g};
        hipError_t e = launch_kernel((const void*)expert_count_kernel, dim3((unsigned)chunks), dim3(kMapThreads),
                                     cargs, stream, false);
        if (e != hipSuccess)
            return e;
    }
    void* args[] = {(void*)&ids, (void*)&counts, (void*)&offs, (void*)&pos, (void*)&src, (void*)&s, (void*)&chunk,
                    (void*)&f, (void*)&g, (void*)&g_log, (void*)&cap};
    return launch_kernel(chunks > 0 ? (const void*)expert_place_kernel<false> : (const void*)expert_place_kernel<true>,
                         dim3((unsigned)(chunks > 0 ? chunks : 1)), dim3(kMapThreads), args, stream);
}

}  // namespace mxfp4
