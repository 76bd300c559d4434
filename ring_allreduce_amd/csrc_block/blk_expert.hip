// blk_expert.hip -- tokens sorted by expert, moved to their experts' rows and summed
// back, with the gradients (expert_sort, expert_dispatch, expert_combine and its
// backward call).
#include "blk_common.hpp"

namespace blk {

// ------------------------------------------------------------------- sort --
//
// A counting sort.  The pairs are cut into pieces of N x 64 consecutive ones, one wave each,
// and kSortWaves pieces make a workgroup's share:  hist[g][e] = pairs of expert e in share
// g;  its exclusive sum over g, plus the counts of the share's earlier waves, plus the rank
// within the piece is the pair's rank.  Within 64 pairs a lane finds the lanes of its own key
// with one ballot per key bit, so ranks need no atomics between waves and the order is
// stable.
//
// Bound by latency: one workgroup does everything for up to 4096 pairs, two launches (count,
// place) sum the counts of up to 32 shares in the second one, and three (count, sum over
// shares, place) sort the rest.  A lane takes as few of 1, 2, 4 or 8 pairs as that allows,
// since its pairs go one after another: 64 pairs 4.9 us (3.0 on the GPU), 4096 7.9, 16384
// 10.0, 65536 11.1; 524288 of 256 experts 16.8, of which the 12 MB that are read and written
// are 3.

constexpr int kItems = 8;              // pairs per lane, at most
constexpr int kSortWaves = 4;          // waves per workgroup of the forms of several launches
constexpr int kOneWaves = 16;          // waves of the one-workgroup form, at most
constexpr int kOneItems = 4;           // its pairs per lane, at most: with 8 the others are faster
constexpr int kFewShares = 32;         // shares whose sums every workgroup finds by itself

struct SortArgs {
    const void* ids;
    uint64_t id_ld;
    int32_t pairs, k, experts, bits;
    int32_t capacity;
    int32_t rows, shares;
    int32_t* slots;
    int32_t* sources;
    int32_t* counts;
    int32_t* offsets;
    int32_t* hist;      // [shares][experts]
};

// The keys of the wave's pairs, first + i * 64 + lane; `experts` where there is none.  The
// loads go out together, those past the end to the last pair.
template <typename I, int N>
__device__ __forceinline__ void load_keys(const SortArgs& a, int first, int (&key)[N]) {
    const int lane = threadIdx.x & 63;
    I id[N] = {};
    if (a.pairs > 0) {
        uint64_t at[N];
#pragma unroll
        for (int i = 0; i < N; ++i) at[i] = (uint64_t)min(first + i * 64 + lane, a.pairs - 1);
        if (a.id_ld != (uint64_t)a.k) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const uint32_t t = (uint32_t)at[i] / (uint32_t)a.k;
                at[i] += (uint64_t)t * (a.id_ld - (uint64_t)a.k);
            }
        }
#pragma unroll
        for (int i = 0; i < N; ++i) id[i] = ((const I*)a.ids)[at[i]];
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
        key[i] = first + i * 64 + lane < a.pairs && id[i] >= 0 && id[i] < (I)a.experts ? (int)id[i] : a.experts;
}

// Places the wave's N x 64 pairs; base[e] is the rank of expert e's next pair.  Each
// step is done for all items before the next, so that a wave, which may have its SIMD to
// itself, does not wait for one item's chain of ballots, atomic, shuffle and store after
// another; LDS keeps the atomics of a wave in their order.
template <int N>
__device__ __forceinline__ void place_piece(const SortArgs& a, const int (&key)[N], int first,
                                            int* base, const int* start) {
    const int lane = threadIdx.x & 63;
    uint64_t same[N];     // the lanes whose key equals this lane's
#pragma unroll
    for (int i = 0; i < N; ++i) same[i] = ~0ull;
    for (int b = 0; b < a.bits; ++b) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const bool one = (key[i] >> b) & 1;
            const uint64_t ones = __ballot(one);
            same[i] &= one ? ones : ~ones;
        }
    }
    int rank[N], slot[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        rank[i] = 0;
        if (lane == __ffsll((unsigned long long)same[i]) - 1 && key[i] < a.experts)
            rank[i] = atomicAdd(&base[key[i]], __popcll(same[i]));
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        rank[i] = __shfl(rank[i], __ffsll((unsigned long long)same[i]) - 1) + __popcll(same[i] & ((1ull << lane) - 1));
        slot[i] = -1;
        if (key[i] < a.experts) {
            if (a.capacity == 0)
                slot[i] = start[key[i]] + rank[i];
            else if (rank[i] < a.capacity)
                slot[i] = key[i] * a.capacity + rank[i];
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int p = first + i * 64 + lane;
        if (p < a.pairs) {
            a.slots[p] = slot[i];
            if (slot[i] >= 0) a.sources[slot[i]] = p;
        }
    }
}

__device__ __forceinline__ int lanes_upto(int n) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int up = __shfl_up(n, d);
        if (lane >= d) n += up;
    }
    return n;
}

// start[e] = counts[0] + .. + counts[e - 1] in LDS, by the whole workgroup.
__device__ __forceinline__ void prefix_counts(const int* counts, int* start, int experts) {
    if (threadIdx.x < 64) {
        const int lane = threadIdx.x;
        int n[RR_MAX_EXPERTS / 64];
#pragma unroll
        for (int q = 0; q < RR_MAX_EXPERTS / 64; ++q) n[q] = q * 64 + lane < experts ? counts[q * 64 + lane] : 0;
        int before = 0;
#pragma unroll
        for (int q = 0; q < RR_MAX_EXPERTS / 64; ++q) {
            if (q * 64 >= experts) break;
            const int upto = lanes_upto(n[q]);
            if (q * 64 + lane < experts) start[q * 64 + lane] = before + upto - n[q];
            before += __shfl(upto, 63);
        }
        if (lane == 0) start[experts] = before;
    }
    __syncthreads();
}

// offsets, and -1 in the rows no pair has.
__device__ __forceinline__ void fill_unused(const SortArgs& a, const int* counts, const int* start) {
    const int threads = (int)blockDim.x, thread = (int)threadIdx.x;
    if (blockIdx.x == 0)
        for (int e = thread; e <= a.experts; e += threads) a.offsets[e] = a.capacity ? e * a.capacity : start[e];
    if (a.capacity == 0) {
        for (int64_t r = (int64_t)start[a.experts] + (int64_t)blockIdx.x * threads + thread; r < a.rows;
             r += (int64_t)gridDim.x * threads)
            a.sources[r] = -1;
        return;
    }
    for (int e = (int)blockIdx.x; e < a.experts; e += (int)gridDim.x)
        for (int64_t r = (int64_t)min(counts[e], a.capacity) + thread; r < a.capacity; r += threads)
            a.sources[(int64_t)e * a.capacity + r] = -1;
}

// The waves' counts of their keys: mine[e] of each, all zero before.
template <int N>
__device__ __forceinline__ void count_keys(const SortArgs& a, const int (&key)[N], int* mine) {
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (key[i] < a.experts) atomicAdd(&mine[key[i]], 1);
}

// Workgroups go to the 8 XCDs in turn; each XCD gets shares that follow one another, so that
// an expert's neighbouring rows are written through one L2.
__device__ __forceinline__ int share_of_block(const SortArgs& a) {
    const int x = (int)blockIdx.x & 7, each = a.shares >> 3, more = a.shares & 7;
    return x * each + min(x, more) + ((int)blockIdx.x >> 3);
}

template <typename I, int N>
__global__ void __launch_bounds__(64 * kSortWaves) sort_count_kernel(const SortArgs a) {
    extern __shared__ int lds[];
    const int share = share_of_block(a);
    int key[N];
    load_keys<I>(a, (share * kSortWaves + (int)(threadIdx.x >> 6)) * N * 64, key);
    for (int e = threadIdx.x; e < a.experts; e += blockDim.x) lds[e] = 0;
    __syncthreads();
    count_keys(a, key, lds);
    __syncthreads();
    for (int e = threadIdx.x; e < a.experts; e += blockDim.x)
        a.hist[(uint64_t)share * a.experts + e] = lds[e];
}

// Exclusive sum of hist over the shares: a wave an expert, a lane four shares at a time.
__global__ void __launch_bounds__(256) sort_sum_kernel(const SortArgs a) {
    const int e = blockIdx.x * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
    if (e >= a.experts) return;
    int before = 0;
    for (int64_t c0 = 0; c0 < a.shares; c0 += 256) {
        int n[4], sum = 0;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int64_t c = c0 + lane * 4 + u;
            n[u] = c < a.shares ? a.hist[(uint64_t)c * a.experts + e] : 0;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) sum += n[u];
        const int upto = lanes_upto(sum);
        int at = before + upto - sum;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int64_t c = c0 + lane * 4 + u;
            if (c < a.shares) a.hist[(uint64_t)c * a.experts + e] = at;
            at += n[u];
        }
        before += __shfl(upto, 63);
    }
    if (lane == 0) a.counts[e] = before;
}

// base[w][e]: counts of the waves -> rank of wave w's first pair of expert e, from `at`;
// returns the rank of the first pair behind them.
__device__ __forceinline__ int ranks_of_waves(int* base, int waves, int experts, int e, int at) {
    for (int w = 0; w < waves; ++w) {
        const int n = base[w * experts + e];
        base[w * experts + e] = at;
        at += n;
    }
    return at;
}

// FEW: hist holds the shares' counts, which are summed here; otherwise sort_sum_kernel has.
template <typename I, int N, bool FEW>
__global__ void __launch_bounds__(64 * kSortWaves) sort_place_kernel(const SortArgs a) {
    extern __shared__ int lds[];
    constexpr int THREADS = 64 * kSortWaves, EACH = (RR_MAX_EXPERTS + THREADS - 1) / THREADS;
    const int wave = threadIdx.x >> 6, share = share_of_block(a);
    int* start = lds;                                  // experts + 1
    int* base = lds + a.experts + 1;                   // [kSortWaves][experts]
    int* sums = base + kSortWaves * a.experts;         // experts, if FEW
    const int first = (share * kSortWaves + wave) * N * 64;
    int key[N], before[EACH];
    load_keys<I>(a, first, key);
#pragma unroll
    for (int u = 0; u < EACH; ++u) {
        if (u * THREADS >= a.experts) break;
        const int e = u * THREADS + (int)threadIdx.x;
        const int* const from = a.hist + min(e, a.experts - 1);
        if constexpr (!FEW) {
            before[u] = from[(uint64_t)share * a.experts];
        } else {
            int all = 0;
            before[u] = 0;
            for (int c0 = 0; c0 < a.shares; c0 += 16) {
                int n[16];
#pragma unroll
                for (int c = 0; c < 16; ++c) n[c] = from[min(c0 + c, a.shares - 1) * a.experts];
#pragma unroll
                for (int c = 0; c < 16; ++c) {
                    all += c0 + c < a.shares ? n[c] : 0;
                    before[u] += c0 + c < share ? n[c] : 0;
                }
            }
            if (e < a.experts) {
                sums[e] = all;
                if (blockIdx.x == 0) a.counts[e] = all;
            }
        }
    }
    for (int i = threadIdx.x; i < kSortWaves * a.experts; i += THREADS) base[i] = 0;
    __syncthreads();
    count_keys(a, key, base + wave * a.experts);
    const int* const counts = FEW ? sums : a.counts;
    if (FEW) __syncthreads();
    if (a.capacity == 0) prefix_counts(counts, start, a.experts);
    else __syncthreads();
    fill_unused(a, counts, start);
#pragma unroll
    for (int u = 0; u < EACH; ++u) {
        const int e = u * THREADS + (int)threadIdx.x;
        if (e < a.experts) ranks_of_waves(base, kSortWaves, a.experts, e, before[u]);
    }
    __syncthreads();
    place_piece(a, key, first, base + wave * a.experts, start);
}

// Everything in one workgroup: wave w takes N x 64 pairs.
template <typename I, int N>
__global__ void __launch_bounds__(64 * kOneWaves) sort_one_kernel(const SortArgs a) {
    extern __shared__ int lds[];
    const int wave = threadIdx.x >> 6, waves = (int)blockDim.x >> 6;
    int* counts = lds;                                 // experts
    int* start = lds + a.experts;                      // experts + 1
    int* base = lds + 2 * a.experts + 1;               // [waves][experts]
    int key[N];
    load_keys<I>(a, wave * N * 64, key);
    for (int i = threadIdx.x; i < waves * a.experts; i += blockDim.x) base[i] = 0;
    __syncthreads();
    count_keys(a, key, base + wave * a.experts);
    __syncthreads();
    for (int e = threadIdx.x; e < a.experts; e += blockDim.x)
        a.counts[e] = counts[e] = ranks_of_waves(base, waves, a.experts, e, 0);
    __syncthreads();
    if (a.capacity == 0) prefix_counts(counts, start, a.experts);
    place_piece(a, key, wave * N * 64, base + wave * a.experts, start);
    fill_unused(a, counts, start);
}

// --------------------------------------------------------------- row moves --
//
// All bound by HBM: a row is a few KiB, so the copies are made of 16-byte accesses
// by a group of threads per token (a wave for short rows, a workgroup for long
// ones), which reads a token's row once and writes all its copies, or reads all its
// copies and writes the sum once.  16384 tokens of 4 rows of 4096 bf16, one kernel again and
// again: copies 131 us (671 MB: 5.1 TB/s), sums 131 (5.1), both gradients 231 with dropped rows
// (1136 MB: 4.9).  Between others the caches move time from one to the next: copies take 109
// behind a kernel that wrote little, and leave what the caches hold of their 537 MB to be
// written under the next one; sums take 165 right behind them, 126 with a read of 1 GiB between.
// Loads behind branches made them 134, 176 and 402.

struct MoveArgs {
    const void* in;      // x, rows or dout
    const void* in2;     // combine backward: rows
    void* out;
    uint64_t in_ld, in2_ld, out_ld;
    const int32_t* slots;
    const int32_t* sources;
    const float* weights;
    float* dweights;
    int32_t tokens, k, rows, hidden;
    int32_t token_blocks;  // workgroups that take tokens; later ones fill unused rows
    float unused;          // with this
};

constexpr int kMoveBlock = 256;
constexpr int kClearRows = 32;   // rows whose source a clearing workgroup looks at

__device__ __forceinline__ int slot_of(const MoveArgs& a, int t, int j) {
    const int s = a.slots[(uint64_t)t * a.k + j];
    return s >= 0 && s < a.rows ? s : -1;
}

// a.unused in the rows without a pair, of kClearRows rows from `first`, a wave its share of them.
template <typename T>
__device__ __forceinline__ void clear_rows(const MoveArgs& a, int64_t first) {
    constexpr int EACH = kClearRows / (kMoveBlock / 64);
    const int lane = threadIdx.x & 63;
    first += (int64_t)(threadIdx.x >> 6) * EACH;
    bool clear = false;
    if (lane < EACH && first + lane < a.rows) {
        const int p = a.sources[first + lane];
        clear = p < 0 || (int64_t)p >= (int64_t)a.tokens * a.k;
    }
    uint64_t left = __ballot(clear);
    Vec<T> fill;
#pragma unroll
    for (int i = 0; i < Vec<T>::N; ++i) fill.e[i] = (T)a.unused;
    while (left) {
        const int b = __ffsll((unsigned long long)left) - 1;
        left &= left - 1;
        T* row = (T*)a.out + (uint64_t)(first + b) * a.out_ld;
        for (int c = lane * Vec<T>::N; c < a.hidden; c += 64 * Vec<T>::N) store_vec(row, c, a.hidden, fill);
    }
}

// A loop over the row's whole vectors, whose loads have no branches, and one over the
// elements left behind them.  Rows that are not there are read as row 0 and not counted.

// G threads per token (a power of two, 8 .. 256).
template <typename T, int G>
__global__ void __launch_bounds__(kMoveBlock) dispatch_kernel(const MoveArgs a) {
    constexpr int N = Vec<T>::N;
    if ((int)blockIdx.x >= a.token_blocks) {
        clear_rows<T>(a, (int64_t)((int)blockIdx.x - a.token_blocks) * kClearRows);
        return;
    }
    const int t = (int)blockIdx.x * (kMoveBlock / G) + (int)threadIdx.x / G;
    if (t >= a.tokens) return;
    const int g = threadIdx.x % G, whole = a.hidden / N * N;
    const T* x = (const T*)a.in + (uint64_t)t * a.in_ld;
    for (int c = g * N; c < whole; c += G * N) {
        const u32x4 v = load_raw(x + c);
        for (int j = 0; j < a.k; ++j) {
            const int s = slot_of(a, t, j);
            if (s >= 0) reinterpret_cast<Loose<T>*>((T*)a.out + (uint64_t)s * a.out_ld + c)->v = v;
        }
    }
    for (int c = whole + g; c < a.hidden; c += G) {
        const T v = x[c];
        for (int j = 0; j < a.k; ++j) {
            const int s = slot_of(a, t, j);
            if (s >= 0) ((T*)a.out)[(uint64_t)s * a.out_ld + c] = v;
        }
    }
}

// J rows of a token at a time (the smallest of 1, 2, 4, 8 that takes all k, if one does).
template <typename T, int G, int J>
__global__ void __launch_bounds__(kMoveBlock) combine_kernel(const MoveArgs a) {
    constexpr int N = Vec<T>::N;
    const int t = (int)blockIdx.x * (kMoveBlock / G) + (int)threadIdx.x / G;
    if (t >= a.tokens) return;
    const int g = threadIdx.x % G, whole = a.hidden / N * N;
    T* out = (T*)a.out + (uint64_t)t * a.out_ld;
    int s[J];
    float w[J];
    const auto slots = [&](int j0) {
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int at = min(j0 + j, a.k - 1);
            s[j] = j0 + j < a.k ? slot_of(a, t, at) : -1;
            w[j] = a.weights ? a.weights[(uint64_t)t * a.k + at] : 1.0f;
        }
    };
    slots(0);
    for (int c = g * N; c < whole; c += G * N) {
        float sum[N];
#pragma unroll
        for (int i = 0; i < N; ++i) sum[i] = 0.0f;
        for (int j0 = 0; j0 < a.k; j0 += J) {
            if (a.k > J) slots(j0);
            u32x4 v[J];
#pragma unroll
            for (int j = 0; j < J; ++j) v[j] = load_raw((const T*)a.in + (uint64_t)max(s[j], 0) * a.in_ld + c);
#pragma unroll
            for (int j = 0; j < J; ++j)
                if (s[j] >= 0)
#pragma unroll
                    for (int i = 0; i < N; ++i) sum[i] = fmaf(w[j], (float)vec_of<T>(v[j]).e[i], sum[i]);
        }
        Vec<T> r;
#pragma unroll
        for (int i = 0; i < N; ++i) r.e[i] = (T)sum[i];
        reinterpret_cast<Loose<T>*>(out + c)->v = __builtin_bit_cast(u32x4, r);
    }
    for (int c = whole + g; c < a.hidden; c += G) {
        float sum = 0.0f;
        for (int j = 0; j < a.k; ++j) {
            const int at = slot_of(a, t, j);
            if (at >= 0)
                sum = fmaf(a.weights ? a.weights[(uint64_t)t * a.k + j] : 1.0f,
                           (float)((const T*)a.in)[(uint64_t)at * a.in_ld + c], sum);
        }
        out[c] = (T)sum;
    }
}

// G = 64 or 256 threads per token.  The dot products are summed per thread in column
// order, then over the lanes of a wave, then over the waves.
template <typename T, int G, int J>
__global__ void __launch_bounds__(kMoveBlock) combine_backward_kernel(const MoveArgs a) {
    constexpr int N = Vec<T>::N;
    constexpr int W = G / 64;
    __shared__ float part[W][J];
    if ((int)blockIdx.x >= a.token_blocks) {
        clear_rows<T>(a, (int64_t)((int)blockIdx.x - a.token_blocks) * kClearRows);
        return;
    }
    const int t = (int)blockIdx.x * (kMoveBlock / G) + (int)threadIdx.x / G;
    if (t >= a.tokens) return;        // whole waves, and with G = 256 the whole workgroup
    const int g = threadIdx.x % G, whole = a.hidden / N * N;
    const T* d = (const T*)a.in + (uint64_t)t * a.in_ld;
    const T* rows = a.dweights ? (const T*)a.in2 : d;    // d: read, and not counted
    const uint64_t rows_ld = a.dweights ? a.in2_ld : 0;
    for (int j0 = 0; j0 < a.k; j0 += J) {
        int s[J];
        float w[J], dot[J];
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int at = min(j0 + j, a.k - 1);
            s[j] = j0 + j < a.k ? slot_of(a, t, at) : -1;
            w[j] = a.weights ? a.weights[(uint64_t)t * a.k + at] : 1.0f;
            dot[j] = 0.0f;
        }
        for (int c = g * N; c < whole; c += G * N) {
            const u32x4 dv = load_raw(d + c);
            u32x4 v[J];
#pragma unroll
            for (int j = 0; j < J; ++j) v[j] = load_raw(rows + (uint64_t)max(s[j], 0) * rows_ld + c);
#pragma unroll
            for (int j = 0; j < J; ++j) {
                if (s[j] < 0) continue;
                if (a.out) {
                    Vec<T> r;
#pragma unroll
                    for (int i = 0; i < N; ++i) r.e[i] = (T)(w[j] * (float)vec_of<T>(dv).e[i]);
                    reinterpret_cast<Loose<T>*>((T*)a.out + (uint64_t)s[j] * a.out_ld + c)->v =
                        __builtin_bit_cast(u32x4, r);
                }
#pragma unroll
                for (int i = 0; i < N; ++i)
                    dot[j] = fmaf((float)vec_of<T>(dv).e[i], (float)vec_of<T>(v[j]).e[i], dot[j]);
            }
        }
        for (int c = whole + g; c < a.hidden; c += G) {
            const float dv = (float)d[c];
#pragma unroll
            for (int j = 0; j < J; ++j) {
                if (s[j] < 0) continue;
                if (a.out) ((T*)a.out)[(uint64_t)s[j] * a.out_ld + c] = (T)(w[j] * dv);
                if (a.dweights) dot[j] = fmaf(dv, (float)rows[(uint64_t)s[j] * rows_ld + c], dot[j]);
            }
        }
        if (!a.dweights) continue;
#pragma unroll
        for (int j = 0; j < J; ++j) dot[j] = lane_sum<64>(dot[j]);
        if constexpr (W > 1) {
            __syncthreads();          // the previous round's sums have been read
            if ((threadIdx.x & 63) == 0)
#pragma unroll
                for (int j = 0; j < J; ++j) part[threadIdx.x >> 6][j] = dot[j];
            __syncthreads();
#pragma unroll
            for (int j = 0; j < J; ++j) {
                dot[j] = 0.0f;
#pragma unroll
                for (int q = 0; q < W; ++q) dot[j] += part[q][j];
            }
        }
        if (g == 0)
#pragma unroll
            for (int j = 0; j < J; ++j)
                if (j0 + j < a.k) a.dweights[(uint64_t)t * a.k + j0 + j] = s[j] >= 0 ? dot[j] : 0.0f;
    }
}

// ------------------------------------------------------------------ host side --

constexpr uint64_t kMaxInt = 0x7FFFFFFFull;

static rr_status_t check_sort(size_t tokens, int k, int experts, size_t capacity) {
    if (k < 1 || experts < 1) return RR_ERR_INVALID;
    if (experts > RR_MAX_EXPERTS || tokens > kMaxInt / (uint64_t)k) return RR_ERR_UNSUPPORTED;
    // the last workgroup's pieces may reach past the pairs, and must still count in 32 bits
    if ((uint64_t)tokens * k > kMaxInt - 64 * kItems * kSortWaves) return RR_ERR_UNSUPPORTED;
    if (capacity > kMaxInt / (uint64_t)experts) return RR_ERR_UNSUPPORTED;
    return RR_OK;
}

// The fewest pairs a lane of 1, 2, 4 .. at_most with which `waves` waves take all.
static int items_for(uint64_t pairs, int waves, int at_most) {
    int n = 1;
    while (n < at_most && pairs > (uint64_t)64 * n * waves) n *= 2;
    return n;
}
// Few shares while four pairs a lane or fewer allow that (65536 pairs in 64 shares of four:
// 10.5 us, in 32 of eight 12.1); four too while a compute unit has no second share (131072
// pairs 12.2 instead of 14.7; 524288 of 256 experts 17.5 instead of 16.9).
static int sort_items(uint64_t pairs) {
    const int n = items_for(pairs, kSortWaves * kFewShares, 4);
    return n == 4 && pairs > (uint64_t)64 * 4 * kSortWaves * 256 ? kItems : n;
}
// One share at least: no pairs have counts and unused rows too.
static uint64_t sort_shares(uint64_t pairs) {
    return pairs ? ceil_div(pairs, 64 * sort_items(pairs) * kSortWaves) : 1;
}
// base, counts and start of every expert in the LDS of one workgroup
static bool one_workgroup(uint64_t pairs, int experts) {
    return pairs <= (uint64_t)64 * kOneItems * kOneWaves && experts <= 512;
}

template <typename I, int N> static void run_one(const SortArgs& a, hipStream_t s) {
    const unsigned pieces = (unsigned)ceil_div(a.pairs, 64 * N), waves = pieces < 4 ? 4 : pieces;
    const size_t lds = ((waves + 2) * (size_t)a.experts + 1) * sizeof(int32_t);
    sort_one_kernel<I, N><<<1, 64 * waves, lds, s>>>(a);
}

template <typename I, int N> static void run_shares(const SortArgs& a, hipStream_t s) {
    const unsigned grid = (unsigned)a.shares;
    const size_t word = sizeof(int32_t), lds = ((kSortWaves + 2) * (size_t)a.experts + 1) * word;
    sort_count_kernel<I, N><<<grid, 64 * kSortWaves, a.experts * word, s>>>(a);
    // a thread of the place kernel sums the counts of one expert in 256 after another: 32
    // shares of 1024 experts 18.2 us, with the kernel that sums them 16.0
    if (N <= 4 && a.shares * ceil_div(a.experts, 64 * kSortWaves) <= kFewShares) {
        if constexpr (N <= 4) sort_place_kernel<I, N, true><<<grid, 64 * kSortWaves, lds, s>>>(a);
    } else {
        sort_sum_kernel<<<(unsigned)ceil_div(a.experts, 4), 256, 0, s>>>(a);
        sort_place_kernel<I, N, false><<<grid, 64 * kSortWaves, lds, s>>>(a);
    }
}

template <typename I> static rr_status_t run_sort(const SortArgs& a, hipStream_t s) {
    if (one_workgroup((uint64_t)a.pairs, a.experts)) {
        const int n = items_for((uint64_t)a.pairs, kOneWaves, kOneItems);
        if (n == 1) run_one<I, 1>(a, s);
        else if (n == 2) run_one<I, 2>(a, s);
        else run_one<I, 4>(a, s);
    } else {
        const int n = sort_items((uint64_t)a.pairs);
        if (n == 1) run_shares<I, 1>(a, s);
        else if (n == 2) run_shares<I, 2>(a, s);
        else if (n == 4) run_shares<I, 4>(a, s);
        else run_shares<I, 8>(a, s);
    }
    return launched();
}

// Shared by the row moves: sizes, index tensors and the matrices that are present.
static rr_status_t check_move(size_t tokens, size_t hidden, int k, size_t rows, int dt) {
    if (!is_float_type(dt) || k < 1 || hidden < 1) return RR_ERR_INVALID;
    if (hidden > kMaxInt - 4096 || rows > kMaxInt || tokens > (kMaxInt - kMoveBlock) / (uint64_t)k)
        return RR_ERR_UNSUPPORTED;
    return RR_OK;
}
static bool good_rows(const rr_rows_t& r, size_t count, size_t hidden, int dt) {
    if (count == 0) return true;
    return r.data && aligned_to(r.data, type_bytes(dt)) && r.ld >= hidden && r.ld <= (1ull << 40);
}
static uint64_t reach(const rr_rows_t& r, size_t count, size_t hidden, int dt) {
    return extent(count, r.ld, hidden, type_bytes(dt));
}

// Threads per token: enough for one 16-byte vector each, so that short rows do not
// leave most of a workgroup idle.
static int group_for(size_t hidden, int dt) {
    const uint64_t vecs = ceil_div(hidden * type_bytes(dt), 16);
    int g = 8;
    while (g < kMoveBlock && (uint64_t)g < vecs) g *= 2;
    return g;
}

// A launch holds fewer than 2^32 threads.
static bool grid_fits(uint64_t blocks) { return blocks < (1ull << 32) / kMoveBlock; }

// Rows of a token at a time.
static int together(int k) { return k <= 1 ? 1 : k <= 2 ? 2 : k <= 4 ? 4 : 8; }

template <typename T, int J> static void launch_combine(const MoveArgs& a, int g, unsigned grid, hipStream_t s) {
    switch (g) {
        case 8: combine_kernel<T, 8, J><<<grid, kMoveBlock, 0, s>>>(a); break;
        case 16: combine_kernel<T, 16, J><<<grid, kMoveBlock, 0, s>>>(a); break;
        case 32: combine_kernel<T, 32, J><<<grid, kMoveBlock, 0, s>>>(a); break;
        case 64: combine_kernel<T, 64, J><<<grid, kMoveBlock, 0, s>>>(a); break;
        case 128: combine_kernel<T, 128, J><<<grid, kMoveBlock, 0, s>>>(a); break;
        default: combine_kernel<T, 256, J><<<grid, kMoveBlock, 0, s>>>(a); break;
    }
}
template <typename T> static void launch_combine(const MoveArgs& a, int g, unsigned grid, hipStream_t s) {
    switch (together(a.k)) {
        case 1: launch_combine<T, 1>(a, g, grid, s); break;
        case 2: launch_combine<T, 2>(a, g, grid, s); break;
        case 4: launch_combine<T, 4>(a, g, grid, s); break;
        default: launch_combine<T, 8>(a, g, grid, s); break;
    }
}
template <typename T, int G> static void launch_backward(const MoveArgs& a, unsigned grid, hipStream_t s) {
    switch (together(a.k)) {
        case 1: combine_backward_kernel<T, G, 1><<<grid, kMoveBlock, 0, s>>>(a); break;
        case 2: combine_backward_kernel<T, G, 2><<<grid, kMoveBlock, 0, s>>>(a); break;
        case 4: combine_backward_kernel<T, G, 4><<<grid, kMoveBlock, 0, s>>>(a); break;
        default: combine_backward_kernel<T, G, 8><<<grid, kMoveBlock, 0, s>>>(a); break;
    }
}

#define BLK_BY_TYPE(dt, CALL)                 \
    switch (dt) {                             \
        case RR_FP32: { CALL(float); break; } \
        case RR_BF16: { CALL(bf16); break; }  \
        default: { CALL(f16); break; }        \
    }

#define BLK_BY_GROUP(g, T, KERNEL, grid, s, a)                            \
    switch (g) {                                                         \
        case 8: KERNEL<T, 8><<<grid, kMoveBlock, 0, s>>>(a); break;      \
        case 16: KERNEL<T, 16><<<grid, kMoveBlock, 0, s>>>(a); break;    \
        case 32: KERNEL<T, 32><<<grid, kMoveBlock, 0, s>>>(a); break;    \
        case 64: KERNEL<T, 64><<<grid, kMoveBlock, 0, s>>>(a); break;    \
        case 128: KERNEL<T, 128><<<grid, kMoveBlock, 0, s>>>(a); break;  \
        default: KERNEL<T, 256><<<grid, kMoveBlock, 0, s>>>(a); break;   \
    }

}  // namespace blk

using namespace blk;

static rr_status_t dispatch(rr_rows_t x, size_t tokens, size_t hidden, int k, rr_dtype_t dt,
                            const int32_t* slots, const int32_t* sources, size_t rows, float unused,
                            rr_rows_t out, rr_stream_t stream) {
    const rr_status_t st = check_move(tokens, hidden, k, rows, dt);
    if (st != RR_OK) return st;
    if (!good_rows(x, tokens, hidden, dt) || !good_rows(out, rows, hidden, dt))
        return RR_ERR_INVALID;
    const uint64_t pairs = (uint64_t)tokens * k;
    if ((tokens && (!slots || !aligned_to(slots, 4))) || (rows && (!sources || !aligned_to(sources, 4))))
        return RR_ERR_INVALID;
    const uint64_t n_out = reach(out, rows, hidden, dt);
    if (overlap(x.data, reach(x, tokens, hidden, dt), out.data, n_out) ||
        overlap(slots, pairs * 4, out.data, n_out) || overlap(sources, rows * 4, out.data, n_out))
        return RR_ERR_INVALID;
    if (rows == 0) return RR_OK;
    MoveArgs a = {};
    a.in = x.data;
    a.in_ld = x.ld;
    a.out = out.data;
    a.out_ld = out.ld;
    a.slots = slots;
    a.sources = sources;
    a.tokens = (int32_t)tokens;
    a.k = k;
    a.rows = (int32_t)rows;
    a.hidden = (int32_t)hidden;
    const int g = group_for(hidden, dt);
    if (!grid_fits(ceil_div(tokens, kMoveBlock / g) + ceil_div(rows, kClearRows)))
        return RR_ERR_UNSUPPORTED;
    a.token_blocks = (int32_t)ceil_div(tokens, kMoveBlock / g);
    a.unused = unused;
    const unsigned grid = (unsigned)(a.token_blocks + ceil_div(rows, kClearRows));
    hipStream_t s = (hipStream_t)stream;
#define CALL(T) BLK_BY_GROUP(g, T, dispatch_kernel, grid, s, a)
    BLK_BY_TYPE(dt, CALL)
#undef CALL
    return launched();
}

extern "C" {

rr_status_t expert_sort_workspace(size_t tokens, int k, int experts, size_t* bytes) {
    if (!bytes) return RR_ERR_INVALID;
    const rr_status_t st = check_sort(tokens, k, experts, 0);
    if (st != RR_OK) return st;
    const uint64_t pairs = (uint64_t)tokens * k;
    *bytes = one_workgroup(pairs, experts) ? 0 : sort_shares(pairs) * experts * sizeof(int32_t);
    return RR_OK;
}

rr_status_t expert_sort(const void* ids, int id_bytes, size_t id_ld, size_t tokens, int k,
                        int experts, size_t capacity, int32_t* slots, int32_t* sources,
                        int32_t* counts, int32_t* offsets, void* workspace,
                        size_t workspace_bytes, rr_stream_t stream) {
    rr_status_t st = check_sort(tokens, k, experts, capacity);
    if (st != RR_OK) return st;
    const uint64_t pairs = (uint64_t)tokens * k;
    const uint64_t rows = capacity ? (uint64_t)experts * capacity : pairs;
    if (id_bytes != 4 && id_bytes != 8) return RR_ERR_INVALID;
    if (!counts || !offsets || !aligned_to(counts, 4) || !aligned_to(offsets, 4))
        return RR_ERR_INVALID;
    if (pairs && (!ids || !slots || !aligned_to(ids, (uint64_t)id_bytes) ||
                  !aligned_to(slots, 4) || id_ld < (size_t)k || id_ld > (1ull << 40)))
        return RR_ERR_INVALID;
    if (rows && (!sources || !aligned_to(sources, 4))) return RR_ERR_INVALID;
    size_t need = 0;
    if ((st = expert_sort_workspace(tokens, k, experts, &need)) != RR_OK) return st;
    if (need && (!workspace || !aligned_to(workspace, 4) || workspace_bytes < need))
        return RR_ERR_INVALID;
    const struct { const void* p; uint64_t n; } b[] = {
        {ids, extent(tokens, id_ld, k, id_bytes)}, {slots, pairs * 4}, {sources, rows * 4},
        {counts, (uint64_t)experts * 4}, {offsets, (uint64_t)experts * 4 + 4}, {workspace, need}};
    for (int i = 0; i < 6; ++i)
        for (int j = i + 1; j < 6; ++j)
            if (overlap(b[i].p, b[i].n, b[j].p, b[j].n)) return RR_ERR_INVALID;
    SortArgs a = {};
    a.ids = ids;
    a.id_ld = id_ld;
    a.pairs = (int32_t)pairs;
    a.k = k;
    a.experts = experts;
    while ((1 << a.bits) <= experts) ++a.bits;      // keys 0 .. experts
    a.capacity = (int32_t)capacity;
    a.rows = (int32_t)rows;
    a.shares = (int32_t)sort_shares(pairs);
    a.slots = slots;
    a.sources = sources;
    a.counts = counts;
    a.offsets = offsets;
    a.hist = (int32_t*)workspace;
    return id_bytes == 4 ? run_sort<int32_t>(a, (hipStream_t)stream)
                         : run_sort<int64_t>(a, (hipStream_t)stream);
}

rr_status_t expert_dispatch(rr_rows_t x, size_t tokens, size_t hidden, int k, rr_dtype_t dt,
                            const int32_t* slots, const int32_t* sources, size_t rows,
                            rr_rows_t out, rr_stream_t stream) {
    return dispatch(x, tokens, hidden, k, dt, slots, sources, rows, 0.0f, out, stream);
}

rr_status_t expert_dispatch_scales(rr_rows_t scales, size_t tokens, size_t blocks, int k,
                                   const int32_t* slots, const int32_t* sources, size_t rows,
                                   rr_rows_t out, rr_stream_t stream) {
    return dispatch(scales, tokens, blocks, k, RR_FP32, slots, sources, rows, 1.0f, out, stream);
}

rr_status_t expert_combine(rr_rows_t in, size_t rows, size_t hidden, rr_dtype_t dt,
                           const int32_t* slots, const float* weights, size_t tokens, int k,
                           rr_rows_t out, rr_stream_t stream) {
    const rr_status_t st = check_move(tokens, hidden, k, rows, dt);
    if (st != RR_OK) return st;
    if (!good_rows(in, rows, hidden, dt) || !good_rows(out, tokens, hidden, dt))
        return RR_ERR_INVALID;
    const uint64_t pairs = (uint64_t)tokens * k;
    if (tokens && (!slots || !aligned_to(slots, 4) || !aligned_to(weights, 4)))
        return RR_ERR_INVALID;
    const uint64_t n_out = reach(out, tokens, hidden, dt);
    if (overlap(in.data, reach(in, rows, hidden, dt), out.data, n_out) ||
        overlap(slots, pairs * 4, out.data, n_out) || overlap(weights, pairs * 4, out.data, n_out))
        return RR_ERR_INVALID;
    if (tokens == 0) return RR_OK;
    MoveArgs a = {};
    a.in = in.data;
    a.in_ld = in.ld;
    a.out = out.data;
    a.out_ld = out.ld;
    a.slots = slots;
    a.weights = weights;
    a.tokens = (int32_t)tokens;
    a.k = k;
    a.rows = (int32_t)rows;
    a.hidden = (int32_t)hidden;
    if (rows == 0) {               // no slot has a row: something to read and not count
        a.in = out.data;
        a.in_ld = 0;
    }
    const int g = group_for(hidden, dt);
    if (!grid_fits(ceil_div(tokens, kMoveBlock / g))) return RR_ERR_UNSUPPORTED;
    const unsigned grid = (unsigned)ceil_div(tokens, kMoveBlock / g);
    hipStream_t s = (hipStream_t)stream;
#define CALL(T) launch_combine<T>(a, g, grid, s)
    BLK_BY_TYPE(dt, CALL)
#undef CALL
    return launched();
}

rr_status_t expert_combine_backward(rr_rows_t dout, rr_rows_t in, size_t rows, size_t hidden,
                                    rr_dtype_t dt, const int32_t* slots, const int32_t* sources,
                                    const float* weights, size_t tokens, int k, rr_rows_t drows,
                                    float* dweights, rr_stream_t stream) {
    const rr_status_t st = check_move(tokens, hidden, k, rows, dt);
    if (st != RR_OK) return st;
    if (!good_rows(dout, tokens, hidden, dt)) return RR_ERR_INVALID;
    if (dweights && !good_rows(in, rows, hidden, dt)) return RR_ERR_INVALID;
    if (drows.data && !good_rows(drows, rows, hidden, dt)) return RR_ERR_INVALID;
    const uint64_t pairs = (uint64_t)tokens * k;
    if (tokens && (!slots || !aligned_to(slots, 4) || !aligned_to(weights, 4) ||
                   !aligned_to(dweights, 4)))
        return RR_ERR_INVALID;
    if (drows.data && rows && (!sources || !aligned_to(sources, 4))) return RR_ERR_INVALID;
    const struct { const void* p; uint64_t n; } read[] = {
        {dout.data, reach(dout, tokens, hidden, dt)},
        {dweights ? in.data : nullptr, reach(in, rows, hidden, dt)},
        {slots, pairs * 4}, {sources, rows * 4}, {weights, pairs * 4}};
    const uint64_t n_rows = drows.data ? reach(drows, rows, hidden, dt) : 0;
    for (const auto& r : read)
        if (overlap(r.p, r.n, drows.data, n_rows) || overlap(r.p, r.n, dweights, pairs * 4))
            return RR_ERR_INVALID;
    if (overlap(drows.data, n_rows, dweights, pairs * 4)) return RR_ERR_INVALID;
    MoveArgs a = {};
    a.in = dout.data;
    a.in_ld = dout.ld;
    a.in2 = rows ? in.data : dout.data;   // without rows: something to read and not count
    a.in2_ld = rows ? in.ld : 0;
    a.out = rows ? drows.data : nullptr;
    a.out_ld = drows.ld;
    a.slots = slots;
    a.sources = sources;
    a.weights = weights;
    a.dweights = dweights;
    a.tokens = (int32_t)tokens;
    a.k = k;
    a.rows = (int32_t)rows;
    a.hidden = (int32_t)hidden;
    if (!a.out && !a.dweights) return RR_OK;
    const bool wide = group_for(hidden, dt) > 64;
    const uint64_t token_blocks = wide ? tokens : ceil_div(tokens, kMoveBlock / 64);
    const uint64_t blocks = token_blocks + (a.out ? ceil_div(rows, kClearRows) : 0);
    if (!grid_fits(blocks)) return RR_ERR_UNSUPPORTED;
    a.token_blocks = (int32_t)token_blocks;
    const unsigned grid = (unsigned)blocks;
    if (grid == 0) return RR_OK;
    hipStream_t s = (hipStream_t)stream;
#define CALL(T)                                  \
    if (wide)                                    \
        launch_backward<T, 256>(a, grid, s);     \
    else                                         \
        launch_backward<T, 64>(a, grid, s);
    BLK_BY_TYPE(dt, CALL)
#undef CALL
    return launched();
}

}  // extern "C"
