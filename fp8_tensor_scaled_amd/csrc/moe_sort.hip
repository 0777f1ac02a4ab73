// Places of (token, choice) pairs sorted by expert: a counting sort that
// keeps the pairs' order within an expert.
//
// A workgroup takes 1024 pairs at a time, one a lane.  The lanes of a wave that
// have a bin (an expert, or none) in common find each other with ten ballots;
// a wave writes its count for each bin it meets to LDS, a lane per bin adds the
// waves' counts up, and a pair's place is
//     the bin's first row + pairs of the bin before this workgroup
//     + those in the waves before + those on lower lanes.
// Up to kSingle pairs one workgroup does it all: its own counts are the bins'.
// Up to kCountAll each workgroup reads all pairs and counts those before its
// share and those from there on.  Past that a first launch counts the bins of
// each workgroup's share, and each workgroup of the second adds those counts
// up for itself.  No atomics hand out places, so the order is the same each
// time.
//
// The data are few (4 bytes in and out per pair): bound by the launches and by
// the chain of loads, counts and barriers of one workgroup (1024 pairs of 64
// experts 3.9 us, 131072 7.8, 2097152 30).

#include "expert_block.hpp"
#include "rows.hpp"

namespace fp8lin {

namespace {

constexpr int kT = 1024, kWaves = kT / kWave;
constexpr int kBins = 512 + 1;    // experts, and the pairs of none
constexpr int kSingle = kT;       // pairs that one workgroup sorts in one launch
constexpr int kMostShares = 128;  // workgroups of a longer sort

// Pairs up to which each workgroup counts all of them.  One launch so / two, us in
// a graph: 64 experts 4096 pairs 5.0 / 6.7, 16384 6.1 / 7.1, 32768 7.8 / 7.1; 7
// experts 4.8 / 6.6, 6.0 / 6.8, 7.6 / 6.8; 256 experts 5.5 / 7.5, 6.7 / 7.7, 8.3 / 8.4.
constexpr int kCountAll = 16384;

enum Mode { kOne, kCounting, kCounted };

__device__ __forceinline__ int bin_of(int id, int experts) {
    return id >= 0 && id < experts ? id : experts;
}

// Lanes of the wave whose bin is this lane's, among those that take part.
__device__ __forceinline__ uint64_t lanes_like(int bin, bool part) {
    uint64_t like = __ballot(part);
#pragma unroll
    for (int b = 0; b < 10; ++b) {
        const bool bit = (bin >> b) & 1;
        const uint64_t set = __ballot(bit);
        like &= bit ? set : ~set;
    }
    return like;
}

// v's sum over the lanes before this one in the workgroup.
__device__ __forceinline__ int sum_before(int v, int* of_wave) {
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    int up = v;
#pragma unroll
    for (int d = 1; d < kWave; d *= 2) {
        const int o = __shfl_up(up, d, kWave);
        up += lane >= d ? o : 0;
    }
    if (lane == kWave - 1) of_wave[wave] = up;
    __syncthreads();
    int before = up - v;
    for (int w = 0; w < wave; ++w) before += of_wave[w];
    return before;
}

struct Share {
    int first, last;  // pairs
};
__device__ __forceinline__ Share share_of(int pairs) {
    const int64_t each = ((int64_t)pairs + gridDim.x - 1) / gridDim.x;
    const int64_t whole = (each + kT - 1) / kT * kT;
    const int64_t first = whole * blockIdx.x;
    Share s;
    s.first = first < pairs ? (int)first : pairs;
    s.last = first + whole < pairs ? (int)(first + whole) : pairs;
    return s;
}

// counts [share][experts + 1]
__global__ __launch_bounds__(kT) void sort_count_kernel(MoeSortLaunch p) {
    __shared__ int count[kBins];
    int* counts = static_cast<int*>(p.ws);
    const int bins = p.experts + 1;
    const Share s = share_of(p.pairs);
    for (int b = threadIdx.x; b < bins; b += kT) count[b] = 0;
    __syncthreads();
    for (int i = s.first + threadIdx.x; i < s.last; i += kT)
        atomicAdd(&count[bin_of(p.ids[i], p.experts)], 1);
    __syncthreads();
    for (int b = threadIdx.x; b < bins; b += kT) counts[blockIdx.x * bins + b] = count[b];
}

template <Mode MODE>
__global__ __launch_bounds__(kT) void sort_place_kernel(MoeSortLaunch p) {
    __shared__ int next[kBins];             // a bin's next row
    __shared__ int of_wave[kWaves][kBins];  // a bin's pairs in the waves (before one)
    __shared__ int before[kBins], total[kBins];  // a bin's pairs before this share, and the rest
    __shared__ int scan[kWaves];
    const int tid = threadIdx.x, wave = tid / kWave, lane = tid % kWave;
    const int bins = p.experts + 1;
    const Share s = share_of(p.pairs);

    if constexpr (MODE == kCounting) {
        // neighbouring lanes count in copies of their own, so that few of them meet,
        // which they do where experts are few; the copies' adding up costs the others
        // as much.  16384 pairs, 16 copies / 8 / 1, us in a graph: 7 experts 6.0 / 5.9 /
        // 7.6, 16 6.0 / 5.8 / 6.6, 32 6.0 / 5.8 / 5.8, 64 6.2 / 6.0 / 5.9, 255 6.8 / 6.5 /
        // 6.2; 256 experts 6.7 with 8, 6.3 with 1.
        int* count = &of_wave[0][0];  // [2][copies][bins]
        const int copies = 2 * 16 * bins <= kWaves * kBins ? 16 : 8;
        for (int b = tid; b < 2 * copies * bins; b += kT) count[b] = 0;
        __syncthreads();
        int* mine = count + lane % copies * bins;
        // (eight loads under way at a time)
        for (int i = tid; i < p.pairs; i += 8 * kT) {
            int id[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) id[k] = i + k * kT < p.pairs ? p.ids[i + k * kT] : 0;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int at = i + k * kT;
                if (at < p.pairs)
                    atomicAdd(mine + (at < s.first ? 0 : copies * bins) + bin_of(id[k], p.experts),
                              1);
            }
        }
        __syncthreads();
        if (tid < bins) {
            int a = 0, b = 0;
            for (int c = 0; c < copies; ++c) {
                a += count[c * bins + tid];
                b += count[(copies + c) * bins + tid];
            }
            before[tid] = a;
            total[tid] = b;
        }
    }
    if constexpr (MODE == kCounted) {
        // the bins' counts, all shares' and those before this one: `parts` lanes
        // share a bin
        const int* counts = static_cast<const int*>(p.ws);
        for (int b = tid; b < bins; b += kT) total[b] = before[b] = 0;
        __syncthreads();
        const int parts = kT / bins > 0 ? kT / bins : 1;
        const int bin = tid % bins, part = tid / bins;
        if (part < parts) {
            int all = 0, mine = 0;
            for (int k = part; k < (int)gridDim.x; k += 8 * parts) {
                int v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int share = k + i * parts;
                    v[i] = share < (int)gridDim.x ? counts[share * bins + bin] : 0;
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    all += v[i];
                    mine += k + i * parts < (int)blockIdx.x ? v[i] : 0;
                }
            }
            atomicAdd(&total[bin], all - mine);
            atomicAdd(&before[bin], mine);
        }
    }
    if constexpr (MODE != kOne) {
        __syncthreads();
        const int n = tid < bins ? before[tid] + total[tid] : 0;
        const int at = sum_before(n, scan);
        if (tid < bins) {
            next[tid] = at + before[tid];
            if (blockIdx.x == 0) p.offsets[tid] = at;
        }
    }

    for (int first = s.first; first < s.last || (MODE == kOne && first == 0); first += kT) {
        for (int b = tid; b < kWaves * bins; b += kT) of_wave[b / bins][b % bins] = 0;
        const int i = first + tid;
        const bool part = i < s.last;
        const int bin = part ? bin_of(p.ids[i], p.experts) : 0;
        const uint64_t like = lanes_like(bin, part);
        const int below = __popcll(like & ((1ull << lane) - 1));
        __syncthreads();
        if (part && below == 0) of_wave[wave][bin] = __popcll(like);
        __syncthreads();
        int run = 0;
        if (tid < bins) {
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                const int n = of_wave[w][tid];
                of_wave[w][tid] = run;
                run += n;
            }
        }
        if constexpr (MODE == kOne) {
            const int at = sum_before(run, scan);
            if (tid < bins) next[tid] = p.offsets[tid] = at;
        }
        __syncthreads();
        if (part) {
            const int at = next[bin] + of_wave[wave][bin] + below;
            p.slots[i] = at;
            if (p.order) p.order[at] = i;
        }
        __syncthreads();
        if constexpr (MODE != kOne) {
            if (tid < bins) next[tid] += run;
        }
    }
}

int shares_of(int64_t pairs) {
    if (pairs <= kSingle) return 1;
    const int64_t need = (pairs + kT - 1) / kT;
    return (int)(need < kMostShares ? need : kMostShares);
}

}  // namespace

size_t moe_sort_workspace(int64_t pairs, int64_t experts) {
    const int shares = shares_of(pairs);
    return pairs > kCountAll ? sizeof(int) * (size_t)shares * (size_t)(experts + 1) : 0;
}

hipError_t launch_moe_sort(const MoeSortLaunch& q, hipStream_t stream) {
    const int shares = shares_of(q.pairs);
    if (shares == 1) {
        hipLaunchKernelGGL(sort_place_kernel<kOne>, dim3(1), dim3(kT), 0, stream, q);
        return hipGetLastError();
    }
    if (q.pairs <= kCountAll) {
        hipLaunchKernelGGL(sort_place_kernel<kCounting>, dim3(shares), dim3(kT), 0, stream, q);
        return hipGetLastError();
    }
    hipLaunchKernelGGL(sort_count_kernel, dim3(shares), dim3(kT), 0, stream, q);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(sort_place_kernel<kCounted>, dim3(shares), dim3(kT), 0, stream, q);
    return hipGetLastError();
}

}  // namespace fp8lin
