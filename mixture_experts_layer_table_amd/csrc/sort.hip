// Token slots sorted by expert: ids [T,k] -> the first row of each expert, the
// row of each slot, the slot of each row. Stable: rows go by (expert, f), f = t*k + j.
//
// The rank of a slot among its expert's is the number of earlier slots with the
// same id. A wave takes 64 consecutive slots a step: lanes with equal ids find
// each other by one ballot per bit of the id, and a counter per expert carries
// the count over the wave's steps. The counters of all waves are then summed in
// order, rounded up to `align` and scanned over the experts. Integers only, and no
// rank comes from an atomic (the one-launch form adds up whole counts with them, in
// any order), so the table is a pure function of the ids.
//
// Below kSortFew slots and up to kSortFewE experts it is one launch: workgroups of 1,024
// slots, each of which counts all slots for itself, those ahead of its own apart.
// Up to 64 of them read the same 256 KiB from L2, which is cheaper than a second
// launch; what bounds it is the chain of barriers and dependent accesses. From
// there on, three launches: a count per wave, a scan over the waves, and the placing.
// One launch against three, us in a graph of calls, ids spread over the experts: 8
// slots 4.8 / 9.7, 16,384 slots 8.0 / 32, 65,535 slots 17 / 33 (256 experts) and 19 / 22
// (8 experts); at 131,072 slots they meet (29 / 34 and about 34 / 26). Equal keys of a
// wave add to one LDS counter in turn, those of slots without an expert here too, so
// one launch takes longer for ids that are not spread, where three take the same. Of
// 256 experts, half of the slots on one: 13 / 32 at 16,384 slots, 35 / 32 at 65,535; all
// on one, or 98% without an expert here: 19 / 32 and 60 / 32.
#include <algorithm>

#include "common.h"
#include "kernels.h"
#include "timing.h"

namespace mok {
namespace {

constexpr int kSortWaves = 16;
constexpr int64_t kSortChunk = kSortWaves * 64;   // slots of a workgroup
constexpr int64_t kSortFew = 64 * kSortChunk;
constexpr int kSortFewE = 512;                    // counters of 16 waves: 32 KiB of LDS
constexpr int64_t kSortGroups = 1024;             // most waves of the three-launch form

struct SortArgs {
    const int32_t *ids;
    int32_t *offsets, *slots, *row_slots;
    int32_t *counts, *totals;   // workspace: [groups][E], [E]
    int64_t n, cap, chunk;      // slots, entries of row_slots, slots per wave (a multiple of 64)
    int E, align, bits, groups;
};

// Key of slot f: its expert, or E for none (also past the last slot).
__device__ __forceinline__ int sort_key(const SortArgs &a, int64_t f) {
    const int id = f < a.n ? a.ids[f] : -1;
    return (uint32_t)id < (uint32_t)a.E ? id : a.E;
}

// The lanes of the wave that hold the same key as this one.
__device__ __forceinline__ uint64_t same_key(int key, int bits) {
    uint64_t m = ~0ull;
    for (int b = 0; b < bits; ++b) {
        const uint64_t v = __ballot((key >> b) & 1);
        m &= (key >> b) & 1 ? v : ~v;
    }
    return m;
}

// Rank of this lane's slot among the wave's slots of its key so far; `count`
// (one entry per key, this wave's own) moves on by the step's slots. Volatile:
// what a lane reads here another lane wrote in the step before.
__device__ __forceinline__ int take_rank(volatile int32_t *count, int key, int bits) {
    const uint64_t m = same_key(key, bits);
    const int lane = (int)(threadIdx.x & 63);
    const uint64_t below = m & ((1ull << lane) - 1);
    const int before = count[key];   // a wave's LDS accesses complete in order: every lane reads before one adds
    if (below == 0) count[key] = before + __popcll(m);
    return before + __popcll(below);
}

__device__ __forceinline__ int wave_scan(int v) {   // inclusive
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(v, d);
        if ((int)(threadIdx.x & 63) >= d) v += o;
    }
    return v;
}

// Unsigned: a sort near the limits has v + align - 1 past 2^31, the rounded value below it.
__device__ __forceinline__ constexpr int round_up(int v, int align) {
    return (int)(((uint32_t)v + (uint32_t)align - 1u) / (uint32_t)align * (uint32_t)align);
}
static_assert(round_up(2147483000, 1000) == 2147483000 && round_up(2147482001, 1000) == 2147483000, "no wrap");

__global__ __launch_bounds__(64 * kSortWaves) void sort_few(SortArgs a) {
    __shared__ int32_t count[kSortWaves][kSortFewE + 1];
    __shared__ int32_t ahead[kSortFewE + 1], total[kSortFewE + 1];   // slots before this workgroup's, and all others
    __shared__ int32_t first[kSortFewE + 1];
    __shared__ int32_t wave_sum[kSortWaves];
    const int tid = (int)threadIdx.x, wave = tid >> 6, lane = tid & 63;
    const int64_t f = blockIdx.x * kSortChunk + tid;
    const int key = sort_key(a, f);
    for (int e = lane; e <= a.E; e += 64) count[wave][e] = 0;
    if (tid <= a.E) total[tid] = ahead[tid] = 0;
    __syncthreads();
    const int rank = take_rank(count[wave], key, a.bits);
    constexpr int B = 8;   // slots in flight per thread
    for (int64_t g0 = 0; g0 < a.n; g0 += B * kSortChunk) {
        int k[B];
#pragma unroll
        for (int i = 0; i < B; ++i) k[i] = sort_key(a, g0 + i * kSortChunk + tid);
#pragma unroll
        for (int i = 0; i < B; ++i) {
            const int64_t chunk = g0 / kSortChunk + i;
            if (chunk < (int64_t)blockIdx.x) atomicAdd(&ahead[k[i]], 1);
            else if (chunk * kSortChunk < a.n) atomicAdd(&total[k[i]], 1);
        }
    }
    __syncthreads();
    int sum = 0, mine = 0;
    if (tid < a.E) {
        int before = ahead[tid];
        sum = before + total[tid];
#pragma unroll
        for (int w = 0; w < kSortWaves; ++w) {
            const int c = count[w][tid];
            count[w][tid] = before;
            before += c;
        }
        mine = round_up(sum, a.align);
    }
    int incl = wave_scan(mine);
    if (lane == 63) wave_sum[wave] = incl;
    __syncthreads();
    for (int w = 0; w < wave; ++w) incl += wave_sum[w];
    if (tid < a.E) {
        first[tid] = incl - mine;
        if (blockIdx.x == 0) a.offsets[tid] = incl - mine;
        if (tid % a.groups == (int)blockIdx.x)
            for (int r = incl - mine + sum; r < incl; ++r) a.row_slots[r] = -1;
    }
    if (tid == a.E - 1) {
        first[a.E] = incl;
        if (blockIdx.x == 0) a.offsets[a.E] = incl;
    }
    __syncthreads();
    if (f < a.n) {
        const int row = key < a.E ? first[key] + count[wave][key] + rank : -1;
        a.slots[f] = row;
        if (row >= 0) a.row_slots[row] = (int32_t)f;
    }
    for (int64_t r = first[a.E] + f; r < a.cap; r += a.groups * kSortChunk) a.row_slots[r] = -1;
}

// Slots per expert of this wave's chunk.
__global__ __launch_bounds__(64) void sort_count(SortArgs a) {
    extern __shared__ int32_t lds[];   // [E + 1]
    for (int e = threadIdx.x; e <= a.E; e += 64) lds[e] = 0;
    const int64_t f0 = blockIdx.x * a.chunk;
    for (int64_t f = f0; f < min(f0 + a.chunk, a.n); f += 64)
        take_rank(lds, sort_key(a, f + threadIdx.x), a.bits);
    for (int e = threadIdx.x; e < a.E; e += 64) a.counts[(int64_t)blockIdx.x * a.E + e] = lds[e];
}

// counts -> exclusive sums over the waves, totals: 64 experts x 16 runs of waves a workgroup.
__global__ __launch_bounds__(1024) void sort_scan(SortArgs a) {
    __shared__ int32_t sum[16][64];
    const int c = (int)threadIdx.x & 63, run = (int)threadIdx.x >> 6, e = (int)blockIdx.x * 64 + c;
    const int per = (a.groups + 15) / 16, g0 = run * per, g1 = min(g0 + per, a.groups);
    int s = 0;
    if (e < a.E)
        for (int g = g0; g < g1; ++g) s += a.counts[(int64_t)g * a.E + e];
    sum[run][c] = s;
    __syncthreads();
    if (e >= a.E) return;
    int before = 0;
    for (int r = 0; r < run; ++r) before += sum[r][c];
    for (int g = g0; g < g1; ++g) {
        const int n = a.counts[(int64_t)g * a.E + e];
        a.counts[(int64_t)g * a.E + e] = before;
        before += n;
    }
    if (run == 15) a.totals[e] = before;   // the last run ends with the sum over all, also where it holds no wave
}

__global__ __launch_bounds__(64) void sort_place(SortArgs a) {
    extern __shared__ int32_t next[];   // [E + 1]: the next row of each expert for this wave's slots
    const int lane = (int)threadIdx.x;
    int end = 0;
    for (int e0 = 0; e0 < a.E; e0 += 64) {
        const int e = e0 + lane;
        const int total = e < a.E ? a.totals[e] : 0;
        const int mine = round_up(total, a.align), incl = end + wave_scan(mine);
        if (e < a.E) {
            next[e] = incl - mine + a.counts[(int64_t)blockIdx.x * a.E + e];
            if (blockIdx.x == 0) a.offsets[e] = incl - mine;
            if (e % a.groups == (int)blockIdx.x)
                for (int r = incl - mine + total; r < incl; ++r) a.row_slots[r] = -1;
        }
        end = __shfl(incl, 63);
    }
    if (blockIdx.x == 0 && lane == 0) a.offsets[a.E] = end;
    if (lane == 0) next[a.E] = 0;
    for (int64_t r = end + (int64_t)blockIdx.x * 64 + lane; r < a.cap; r += (int64_t)a.groups * 64) a.row_slots[r] = -1;
    const int64_t f0 = blockIdx.x * a.chunk;
    for (int64_t f1 = f0; f1 < min(f0 + a.chunk, a.n); f1 += 64) {
        const int64_t f = f1 + lane;
        const int key = sort_key(a, f), row = take_rank(next, key, a.bits);
        if (f < a.n) a.slots[f] = key < a.E ? row : -1;
        if (f < a.n && key < a.E) a.row_slots[row] = (int32_t)f;
    }
}

}  // namespace

bool sort_plan(int64_t T, int k, int E, int align, SortPlan *p) {
    if (T < 0 || T >= (int64_t(1) << 31) || k < 1 || E < 1 || E > 4096 || align < 1 || align > 1024) return false;
    const int64_t n = T * k;
    const int64_t rows = (n + std::min<int64_t>(E, n) * (align - 1)) / align * align;
    if (n >= (int64_t(1) << 31) || rows >= (int64_t(1) << 31)) return false;
    p->n = n;
    p->rows = rows;
    p->few = n < kSortFew && E <= kSortFewE;
    const int64_t waves = std::max<int64_t>(1, std::min(kSortGroups, (n + 1023) / 1024));
    p->chunk = p->few ? kSortChunk : std::max<int64_t>(64, (n + waves * 64 - 1) / (waves * 64) * 64);
    p->groups = (int)std::max<int64_t>(1, (n + p->chunk - 1) / p->chunk);
    p->bytes = p->few ? 0 : ((size_t)p->groups + 1) * E * 4;
    return true;
}

mok_status launch_sort_tokens(const SortPlan &p, int E, int align, const int32_t *ids, void *workspace,
                              int32_t *offsets, int32_t *slots, int32_t *row_slots, hipStream_t st) {
    SortArgs a{};
    a.ids = ids;
    a.offsets = offsets;
    a.slots = slots;
    a.row_slots = row_slots;
    a.counts = static_cast<int32_t *>(workspace);
    a.totals = a.counts + (int64_t)p.groups * E;
    a.n = p.n;
    a.cap = p.rows;
    a.chunk = p.chunk;
    a.E = E;
    a.align = align;
    a.groups = p.groups;
    while ((1 << a.bits) <= E) ++a.bits;   // keys 0 .. E
    KernelTimer tm("sort_tokens", st);
    if (p.few) {
        sort_few<<<(unsigned)p.groups, 64 * kSortWaves, 0, st>>>(a);
    } else {
        const size_t lds = ((size_t)E + 1) * 4;
        sort_count<<<(unsigned)p.groups, 64, lds, st>>>(a);
        sort_scan<<<(unsigned)((E + 63) / 64), 1024, 0, st>>>(a);
        sort_place<<<(unsigned)p.groups, 64, lds, st>>>(a);
    }
    return check_hip(hipGetLastError(), "mok_sort_tokens");
}

}  // namespace mok
