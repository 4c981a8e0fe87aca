// expert_map.hip -- the map between routed slots and expert-ordered rows: a stable
// counting sort of the slots (slot t k + j is choice j of token t) by expert.
//
// Row order is expert, then slot, so the result does not depend on how the work is split.
// The slots are cut into chunks, one per workgroup of 16 waves: a first launch counts each
// chunk's slots per expert, a second finds every chunk's first row per expert (from all
// chunks' counts, which it reads itself: a third launch for the sums would cost more than
// these reads) and ranks its own slots.  Up to kOneChunk slots one workgroup does all of it
// in one launch.  Within a workgroup a wave owns a contiguous run of slots; the rank of a
// slot among the 64 of one step is the number of earlier lanes with the same expert, from
// one ballot per bit of the expert's number.
#include "strips.h"

namespace mxfp4 {

constexpr int kMapThreads = 1024;
constexpr int kMapWaves = kMapThreads / 64;
constexpr int kMapExperts = 1024;                 // G at most
constexpr int64_t kOneChunk = 4096;               // slots one workgroup sorts alone
constexpr int kMaxChunks = 64;

namespace {

// Expert of a slot, -1 if it has none here.
__device__ __forceinline__ int local_expert(const int32_t* __restrict__ ids, int64_t slot, int64_t slots, int first,
                                            int G)
{
    if (slot >= slots)
        return -1;
    const int64_t e = (int64_t)ids[slot] - first;
    return e >= 0 && e < G ? (int)e : -1;
}

}  // namespace

__global__ __launch_bounds__(kMapThreads) void expert_count_kernel(const int32_t* __restrict__ ids,
                                                                   int32_t* __restrict__ counts, int64_t slots,
                                                                   int64_t chunk, int first, int G)
{
    __shared__ int32_t hist[kMapExperts];
    const int tid = threadIdx.x;
    if (tid < G)
        hist[tid] = 0;
    __syncthreads();
    const int64_t from = (int64_t)blockIdx.x * chunk;
    const int64_t to = min(from + chunk, slots);
    for (int64_t s = from + tid; s < to; s += kMapThreads) {
        const int e = local_expert(ids, s, slots, first, G);
        if (e >= 0)
            atomicAdd(&hist[e], 1);
    }
    __syncthreads();
    if (tid < G)
        counts[(int64_t)blockIdx.x * G + tid] = hist[tid];
}

template <bool kOne>
__global__ __launch_bounds__(kMapThreads) void expert_place_kernel(
    const int32_t* __restrict__ ids, const int32_t* __restrict__ counts, int32_t* __restrict__ offs,
    int32_t* __restrict__ pos, int32_t* __restrict__ src, int64_t slots, int64_t chunk, int first, int G, int cap)
{
    // per wave and expert: first its number of slots, then the row of its next slot
    __shared__ int32_t next[kMapWaves][kMapExperts];
    __shared__ int32_t part[kMapWaves];
    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    if (tid < G)
        for (int w = 0; w < kMapWaves; ++w)
            next[w][tid] = 0;
    // all chunks' counts of expert tid: those before this chunk, and the total
    int32_t before = 0, total = 0;
    if (!kOne && tid < G) {
        for (int b = 0; b < (int)gridDim.x; ++b) {
            const int32_t c = counts[(int64_t)b * G + tid];
            before += b < (int)blockIdx.x ? c : 0;
            total += c;
        }
    }
    __syncthreads();
    const int64_t run = chunk / kMapWaves;        // slots of a wave (a multiple of 64)
    const int64_t from = (int64_t)blockIdx.x * chunk + wave * run;
    for (int64_t s = from; s < from + run && s < slots; s += 64) {
        const int e = local_expert(ids, s + lane, slots, first, G);
        if (e >= 0)
            atomicAdd(&next[wave][e], 1);
    }
    __syncthreads();
    if (kOne && tid < G)
        for (int w = 0; w < kMapWaves; ++w)
            total += next[w][tid];
    // first row of each expert: an exclusive sum over the experts, one per thread
    int32_t incl = tid < G ? total : 0;
    for (int d = 1; d < 64; d <<= 1) {
        const int32_t o = __shfl_up(incl, d, 64);
        incl += lane >= d ? o : 0;
    }
    if (lane == 63)
        part[wave] = incl;
    __syncthreads();
    int32_t start = incl - (tid < G ? total : 0);
    for (int w = 0; w < kMapWaves; ++w)
        start += w < wave ? part[w] : 0;
    if (blockIdx.x == 0 && tid < G) {
        offs[tid] = min(start, cap);
        if (tid == G - 1)
            offs[G] = min(start + total, cap);
    }
    if (tid < G) {
        int32_t at = start + before;
        for (int w = 0; w < kMapWaves; ++w) {
            const int32_t c = next[w][tid];
            next[w][tid] = at;
            at += c;
        }
    }
    __syncthreads();
    const int bits = 32 - __builtin_clz(G);       // 0 .. G: G stands for "none"
    for (int64_t s = from; s < from + run && s < slots; s += 64) {
        const int64_t slot = s + lane;
        const int e = local_expert(ids, slot, slots, first, G);
        const int key = e < 0 ? G : e;
        uint64_t same = ~0ull;                    // the lanes with this lane's expert
        for (int b = 0; b < bits; ++b) {
            const bool bit = key >> b & 1;
            const uint64_t m = __ballot(bit);
            same &= bit ? m : ~m;
        }
        const int rank = __popcll(same & ((1ull << lane) - 1));
        int32_t row = -1;
        if (e >= 0) {
            row = next[wave][e] + rank;
            if (rank == 0)                        // one lane per expert moves its counter on
                next[wave][e] = row + (int)__popcll(same);
        }
        if (slot < slots) {
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
    const int64_t n = (slots + kOneChunk - 1) / kOneChunk;
    return n < kMaxChunks ? n : kMaxChunks;
}

hipError_t launch_expert_map(const int32_t* ids, int32_t* offs, int32_t* pos, int32_t* src, int32_t* counts,
                             int64_t slots, int32_t first, int32_t G, int64_t M_cap, hipStream_t stream)
{
    const int64_t chunks = expert_map_chunks(slots);
    int64_t s = slots, chunk = slots;
    if (chunks > 0)
        chunk = (slots + chunks - 1) / chunks;
    chunk = (chunk + kMapThreads - 1) / kMapThreads * kMapThreads;   // whole steps of every wave
    int f = first, g = G, cap = (int)M_cap;
    if (chunks > 0) {
        void* cargs[] = {(void*)&ids, (void*)&counts, (void*)&s, (void*)&chunk, (void*)&f, (void*)&g};
        hipError_t e = launch_kernel((const void*)expert_count_kernel, dim3((unsigned)chunks), dim3(kMapThreads),
                                     cargs, stream, false);
        if (e != hipSuccess)
            return e;
    }
    void* args[] = {(void*)&ids, (void*)&counts, (void*)&offs, (void*)&pos, (void*)&src, (void*)&s, (void*)&chunk,
                    (void*)&f, (void*)&g, (void*)&cap};
    return launch_kernel(chunks > 0 ? (const void*)expert_place_kernel<false> : (const void*)expert_place_kernel<true>,
                         dim3((unsigned)(chunks > 0 ? chunks : 1)), dim3(kMapThreads), args, stream);
}

}  // namespace mxfp4
