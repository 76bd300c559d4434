// blk_gemm.hpp -- the matrix products behind block_linear and its gradients.
//
// Three forms, all out[i][j] = sum over c of P(i, c) Q(j, c):
//   forward  i = row, j = n, c = k:    P = x,  Q = w_e         both contiguous along c
//   dx       i = row, j = k, c = n:    P = dz, Q = w_e         Q contiguous along j
//   dw       i = n,   j = k, c = row:  P = dz, Q = x           both contiguous along i, j
#pragma once

#include <type_traits>

#include "blk_common.hpp"

namespace blk {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
#define BLK_LDS __attribute__((address_space(3)))

enum GemmForm { kForward = 0, kByX = 1, kByW = 2 };
enum GemmTile { kTile256 = 0, kTile128 = 1, kTile64 = 2, kInner64 = 3, kStream16 = 4, kStream32 = 5,
                kStream64 = 6, kDot = 7 };
constexpr int tile_rows(int tile) {
    return tile == kTile256 ? 256 : tile == kTile128 ? 128 : tile == kTile64 || tile == kInner64 || tile == kStream64 ? 64
           : tile == kStream32 ? 32 : tile == kDot ? 4 : 16;
}

struct GemmArgs {
    const void *p, *q;
    uint64_t p_ld, q_ld, q_group;    // q_group: elements from one group's Q to the next
    int32_t rows;                    // rows of all groups (P and out, or the contraction)
    int32_t i, j, c;                 // sizes; the grouped one of i and c is not read
    int32_t groups;
    const int32_t* offsets;          // or null: rows / groups rows each
    // epilogue
    const void *bias, *residual;
    void *z, *out;
    uint64_t residual_ld, z_ld, out_ld, out_group;
    int32_t act;
    int32_t wide_out;                // out in fp32
    int32_t tiles_i, tiles_j;        // tiles_i: an upper bound over all groups
    int32_t splits;                  // parts of the contraction
    float* part;                     // [splits][rows of out][j], if splits > 1, or whole tiles of
                                     // the last round
    uint64_t part_stride;            // elements of one part
    int32_t slots, steps;            // of the last round (slots 0: as it is), see last_round_parts
    // of a gated product: j is the columns of out, z and the parts have 2 j
    uint64_t q_half;                 // elements from the gate's Q to the other projection's
    // of 8-bit operands: a scale for each 128 of a row of P, and for 128 x 128 of Q
    const float *p_scale, *q_scale;
    int32_t blocks;                  // along the contraction
    int32_t q_rows;                  // blocks of 128 rows in Q, each half of a gated one
    // of a gated product whose z is kept in 8 bits (z is null then), by 256 x 256 tiles only
    uint8_t* z8;
    float* z8_scale;                 // [rows][2][q_rows]
    uint64_t z8_ld;
};

// What the host chose for one product; see blk_linear.hip.
struct GemmPlan {
    int32_t form, tile;
    int32_t direct;                  // kStream*: rows of both operands at 16-byte boundaries
    int32_t deep;                    // kTile128, kTile64: four stages in LDS, else two
    int32_t narrow;                  // kStream*: 16 columns a workgroup, else 32
    int cols() const { return tile < kInner64 ? tile_rows(tile) : tile >= kStream16 && narrow ? 16 : 32; }
};

rr_status_t launch_gemm_bf16(const GemmArgs& a, const GemmPlan& p, hipStream_t s);
rr_status_t launch_gemm_f16(const GemmArgs& a, const GemmPlan& p, hipStream_t s);
rr_status_t launch_gated_bf16(const GemmArgs& a, const GemmPlan& p, hipStream_t s);
rr_status_t launch_gated_f16(const GemmArgs& a, const GemmPlan& p, hipStream_t s);
rr_status_t launch_gemm8_bf16(const GemmArgs& a, const GemmPlan& p, hipStream_t s);
rr_status_t launch_gemm8_f16(const GemmArgs& a, const GemmPlan& p, hipStream_t s);
rr_status_t launch_gated8_bf16(const GemmArgs& a, const GemmPlan& p, hipStream_t s);
rr_status_t launch_gated8_f16(const GemmArgs& a, const GemmPlan& p, hipStream_t s);

// ------------------------------------------------------------------- groups --

struct Range {
    int32_t group;   // -1: rows of no group
    int32_t lo, hi;
};

// Range r of rows: 0 is what lies before the first group, groups + 1 what lies after
// the last one.  Whatever the offsets hold, 0 <= lo <= hi <= rows.
__device__ __forceinline__ Range range_of(const GemmArgs& a, int r) {
    Range g = {-1, 0, 0};
    if (r > a.groups + 1) return g;
    if (!a.offsets) {
        if (r < 1 || r > a.groups) return g;
        const int32_t each = a.rows / a.groups;
        return {r - 1, (r - 1) * each, r * each};
    }
    const auto edge = [&](int k) { return min(max(a.offsets[k], 0), a.rows); };
    g.lo = r == 0 ? 0 : edge(r - 1);
    g.hi = r > a.groups ? a.rows : edge(r);
    if (g.hi < g.lo) g.hi = g.lo;
    if (r >= 1 && r <= a.groups) g.group = r - 1;
    return g;
}

// Row tiles of `height` rows, counted through the ranges one after another.  A wave looks at
// 64 ranges at a time, a lane each; of the first 64 it keeps what it found.
struct RowTiles {
    Range first;      // of this lane
    int n, upto;      // its tiles, and those up to and with it
    int total;        // of all ranges
};

__device__ __forceinline__ int lanes_upto(int n) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int up = __shfl_up(n, d);
        if (lane >= d) n += up;
    }
    return n;
}

// Called by whole waves.  Offsets that descend make ranges that overlap, and of them more tiles
// than the host counted, up to 2^34: those beyond its count are left out.
__device__ __forceinline__ RowTiles count_tiles(const GemmArgs& a, int height) {
    RowTiles t = {};
    if (a.groups == 1 && !a.offsets) {
        t.total = (a.rows + height - 1) / height;
        return t;
    }
    for (int r0 = 0; r0 < a.groups + 2; r0 += 64) {
        const Range r = range_of(a, r0 + (int)(threadIdx.x & 63));
        const int n = (r.hi - r.lo + height - 1) / height, upto = lanes_upto(n);
        if (r0 == 0) t.first = r, t.n = n, t.upto = upto;
        t.total = min(t.total + __shfl(upto, 63), a.tiles_i);
    }
    t.total = __builtin_amdgcn_readfirstlane(t.total);
    return t;
}

// The range and the first row of row tile `tile`.  Called by whole waves; false past the end.
__device__ __forceinline__ bool find_tile(const GemmArgs& a, const RowTiles& t, int tile, int height, Range& g) {
    if (tile >= t.total) return false;
    if (a.groups == 1 && !a.offsets) {
        g = {0, tile * height, a.rows};
        return true;
    }
    int before = 0;
    for (int r0 = 0; r0 < a.groups + 2; r0 += 64) {
        Range r = t.first;
        int n = t.n, upto = t.upto;
        if (r0 > 0) {
            r = range_of(a, r0 + (int)(threadIdx.x & 63));
            n = (r.hi - r.lo + height - 1) / height;
            upto = lanes_upto(n);
        }
        const uint64_t past = __ballot(tile < before + upto);
        if (past) {
            const int at = __ffsll((unsigned long long)past) - 1;
            g.group = __shfl(r.group, at);
            g.lo = __shfl(r.lo, at) + (tile - before - (__shfl(upto, at) - __shfl(n, at))) * height;
            g.hi = __shfl(r.hi, at);
            return true;
        }
        before += __shfl(upto, 63);
    }
    return false;
}

// The last, partly filled round of workgroups: `rest` tiles on a device that takes `slots` at
// once.  Into how many parts of the contraction each of these tiles is cut, so that they fill
// the device too; 1 where the time saved (1.75 us a step of a 256 x 256 tile) does not pay for
// the parts' way through memory (0.12 us each) and the launch that adds them (4 us).
__host__ __device__ inline int last_round_parts(unsigned rest, unsigned slots, int steps) {
    if (rest == 0) return 1;
    int s = (int)(slots / rest);
    s = s > 8 ? 8 : s;
    s = s > steps / 4 ? steps / 4 : s;
    if (s < 2 || 14 * steps * (s - 1) <= s * (32 + (int)rest * s)) return 1;
    return s;
}

// ----------------------------------------------------------------- the tiles --
//
// A tile of an operand in LDS is 64 deep along c, in one of two layouts:
//   contiguous along c:  [row][64], the eight 16-byte pieces of a row permuted by the
//     row number, so that the 16 rows a fragment read touches lie in different banks;
//   contiguous along the rows:  [64][rows], the 32-byte pieces (16 rows) of a line
//     permuted by the line number, for the transposing read, in which 16 lanes
//     read four lines of 16 rows and each gets four values of one row.
constexpr int kDepth = 64;

template <bool ACROSS, int ROWS> struct Tile {
    static constexpr int kBytes = ROWS * kDepth * 2;
    __device__ __forceinline__ static int mix(int line) {
        return ((line & 3) | ((line >> 1) & 4)) & (ROWS / 16 - 1);
    }
    // (row, c) of the first of the 8 elements in 16-byte piece `id` of the tile
    __device__ __forceinline__ static void place(int id, int& row, int& c) {
        if constexpr (!ACROSS) {
            row = id >> 3;
            c = ((id & 7) ^ (row & 7)) << 3;
        } else {
            c = id / (ROWS / 8);
            const int at = id % (ROWS / 8);
            row = (((at >> 1) ^ mix(c)) << 4) + ((at & 1) << 3);
        }
    }
};

// Reads fragments of 16 rows, 32 deep, of the tiles in LDS: a lane gets row lane % 16 of
// block x, c + (lane / 16) * 8 .. + 7.  Of a block's address only the lane's part takes
// registers: the block row, the half and the operand's place are constants of the
// instruction, and going to another place is one addition.
template <bool ACROSS, int ROWS> struct Reader {
    uint32_t at[2];
    __device__ __forceinline__ void start(uint32_t tile, int row) {    // row: a wave's first, of the tile
        const int lane = threadIdx.x & 63;
        if constexpr (!ACROSS) {
            const int r = row + (lane & 15);
#pragma unroll
            for (int h = 0; h < 2; ++h)
                at[h] = tile + r * (kDepth * 2) + ((((lane >> 4) + h * 4) ^ (lane & 7)) << 4);
        } else {
            const int line = (lane >> 4) * 8 + ((lane & 15) >> 2);
            at[0] = tile + line * (ROWS * 2) + (((row >> 4) ^ Tile<ACROSS, ROWS>::mix(line)) << 5) + (lane & 3) * 8;
        }
    }
    __device__ __forceinline__ void move(uint32_t by) {
        at[0] += by;
        if constexpr (!ACROSS) at[1] += by;
    }
    template <typename V> __device__ __forceinline__ V fragment(int x, int half) const {
        if constexpr (!ACROSS) {
            return __builtin_bit_cast(V, *(const BLK_LDS u32x4*)(uintptr_t)(at[half] + x * 16 * kDepth * 2));
        } else {
            s16x4 v[2];
            const uint32_t from = at[0] ^ (x << 5);
#pragma unroll
            for (int h = 0; h < 2; ++h)
                v[h] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    (BLK_LDS s16x4*)(uintptr_t)(from + (half * 32 + h * 4) * (ROWS * 2)));
            return __builtin_bit_cast(V, v);
        }
    }
};

template <typename T> struct Mma;
template <> struct Mma<bf16> {
    typedef bf16x8 V;
    __device__ __forceinline__ static f32x4 run(V a, V b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
};
template <> struct Mma<f16> {
    typedef f16x8 V;
    __device__ __forceinline__ static f32x4 run(V a, V b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    }
};

// The thread's number, as a value of this place in the program: what is made from it is
// made here again instead of being held in registers through the products before.
__device__ __forceinline__ int here() {
    int t = (int)threadIdx.x;
    asm volatile("" : "+v"(t));
    return t;
}

__device__ __forceinline__ const char* uniform(const char* p) {
    const uint64_t v = (uint64_t)p;
    const uint32_t lo = __builtin_amdgcn_readfirstlane((int)(uint32_t)v);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((int)(uint32_t)(v >> 32));
    return (const char*)((uint64_t)hi << 32 | lo);
}

// Loads straight from memory into LDS, 16 bytes a lane, a wave 1 KiB of the tile at a
// time; the permutation is on the side of the addresses read.  A piece outside the
// operand gets an offset outside the buffer descriptor's range, for which the hardware
// gives zeros.  The instruction has no register result; the caller waits for it
// (arrived()) before the barrier behind which the tile is read.
constexpr uint32_t kReach = 0x80000000u;   // rows of a tile span at most 256 * 2^22 * 2 bytes

// THREADS: that load a tile together; PART: of a larger workgroup.
template <typename T, bool ACROSS, int ROWS, int THREADS, bool PART> struct Direct {
    static constexpr int kPieces = ROWS * kDepth / 8 / THREADS;
    const char* base;
    uint64_t step;
    uint32_t at[kPieces];
    int left;
    uint32_t mine;                   // of this wave in the tile
    u32x4 rsrc;
    uint32_t to;
    __device__ __forceinline__ void start(const T* b, uint64_t ld, int r0, int r_end, int c0, int end) {
        base = (const char*)(b + (ACROSS ? (uint64_t)c0 * ld + r0 : (uint64_t)r0 * ld + c0));
        step = (ACROSS ? ld : 1) * kDepth * sizeof(T);
        left = end - c0;
        mine = (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6) * 1024);
        if constexpr (PART) mine %= THREADS * 16;
        const int thread = PART ? here() % THREADS : here();
#pragma unroll
        for (int k = 0; k < kPieces; ++k) {
            int y, x;
            Tile<ACROSS, ROWS>::place(k * THREADS + thread, y, x);
            const uint64_t off = (ACROSS ? (uint64_t)x * ld + y : (uint64_t)y * ld + x) * sizeof(T);
            at[k] = r0 + y < r_end ? (uint32_t)off : kReach;
        }
    }
    // The next 64 deep tile into LDS at `tile`: aim(), then every piece once.  Tiles past the
    // end come as zeros.
    __device__ __forceinline__ void aim(uint32_t tile) {
        const uint64_t p = (uint64_t)uniform(base);
        rsrc = u32x4{(uint32_t)p, (uint32_t)(p >> 32) & 0xFFFF, kReach, 0x00027000};
        to = tile + mine;
        if (left < kDepth) {
            const int thread = PART ? here() % THREADS : here();
#pragma unroll
            for (int k = 0; k < kPieces; ++k) {
                int y, x;
                Tile<ACROSS, ROWS>::place(k * THREADS + thread, y, x);
                if (x >= left) at[k] = kReach;
            }
        }
        left -= kDepth;
        base += step;
    }
    __device__ __forceinline__ void piece(int k) const { issue(rsrc, at[k], to + k * THREADS * 16); }
    // m0 is one of the registers that the compiler allocates for itself only (which it warns of),
    // but it does merge its own writes of m0 across instructions that are not known to write it.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
    __device__ __forceinline__ static void issue(u32x4 rsrc, uint32_t offset, uint32_t to) {
        asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %0, 0 offen lds"
                     :
                     : "s"(rsrc), "v"(offset), "s"(to)
                     : "m0", "memory");
    }
#pragma clang diagnostic pop
};

// The rows of both halves of a gated product's Q, one behind the other in a tile.
template <typename T, bool ACROSS, int ROWS, int THREADS, bool PART> struct Twin {
    typedef Direct<T, ACROSS, ROWS / 2, THREADS, PART> D;
    static constexpr int kPieces = 2 * D::kPieces;
    D one, two;
    __device__ __forceinline__ void start(const T* b, uint64_t half, uint64_t ld, int r0, int r_end, int c0, int end) {
        one.start(b, ld, r0, r_end, c0, end);
        two.start(b + half, ld, r0, r_end, c0, end);
    }
    __device__ __forceinline__ void aim(uint32_t tile) {
        one.aim(tile);
        two.aim(tile + Tile<ACROSS, ROWS / 2>::kBytes);
    }
    __device__ __forceinline__ void piece(int k) const {
        if (k < D::kPieces) one.piece(k);
        else two.piece(k - D::kPieces);
    }
};

// This wave's loads into LDS but the last LATER are there and its reads of LDS are done,
// then every wave's.
template <int LATER> __device__ __forceinline__ void arrived() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" : : "n"(LATER) : "memory");
}

// ---------------------------------------------------------------- the epilogue --

// N (4 or 8) neighbouring columns of one output row, in one access a matrix; any
// alignment, and element by element past the last column (load_some, store_some).
template <typename T, int N> struct Some {
    T e[N];
};
template <int BYTES> struct Words;
template <> struct Words<8> { typedef uint32_t V __attribute__((ext_vector_type(2))); };
template <> struct Words<16> { typedef u32x4 V; };
template <typename T, int BYTES> struct __attribute__((packed, aligned(sizeof(T)))) LooseWords {
    typename Words<BYTES>::V v;
};

template <typename T, int N> __device__ __forceinline__ Some<T, N> load_some(const T* p, int n) {
    Some<T, N> r;
    if constexpr (N == 1) {
        r.e[0] = *p;
    } else if (n >= N) {
        r = __builtin_bit_cast(Some<T, N>, ((const LooseWords<T, N * sizeof(T)>*)p)->v);
    } else {
#pragma unroll
        for (int e = 0; e < N; ++e) r.e[e] = e < n ? p[e] : (T)0.0f;
    }
    return r;
}
template <typename T, int N> __device__ __forceinline__ void store_some(T* p, int n, const float (&v)[N]) {
    Some<T, N> r;
#pragma unroll
    for (int e = 0; e < N; ++e) r.e[e] = (T)v[e];
    if constexpr (N == 1) {
        *p = r.e[0];
    } else if (n >= N) {
        ((LooseWords<T, N * sizeof(T)>*)p)->v = __builtin_bit_cast(typename Words<N * sizeof(T)>::V, r);
    } else {
#pragma unroll
        for (int e = 0; e < N; ++e)
            if (e < n) p[e] = r.e[e];
    }
}
template <int N> __device__ __forceinline__ void store_wide(float* p, int n, const float (&v)[N]) {
    if constexpr (N == 1) {
        *p = v[0];
    } else {
#pragma unroll
        for (int h = 0; h < N; h += 4) {
            const float w[4] = {v[h], v[h + 1], v[h + 2], v[h + 3]};
            if (n > h) store_some<float, 4>(p + h, n - h, w);
        }
    }
}

// z = sum + bias, out = act(z) + residual; zeros for a row of no group.
template <typename T, int N>
__device__ __forceinline__ Some<T, N> bias_of(const GemmArgs& a, int group, int j) {
    if (!a.bias || group < 0 || j >= a.j) return Some<T, N>{};
    return load_some<T, N>((const T*)a.bias + (uint64_t)group * a.j + j, a.j - j);
}
// z, residual and out: of the first of the N columns; n: how many there are.
template <typename T, int N>
__device__ __forceinline__ void finish(const GemmArgs& a, int group, int n, float (&v)[N],
                                       const Some<T, N>& bias, const Some<T, N>& residual, T* z, void* out) {
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] = group < 0 ? 0.0f : v[e] + (float)bias.e[e];
    if (a.z) store_some<T, N>(z, n, v);
    if (group >= 0) {
        if (a.act != RR_ACT_NONE) act_values(a.act, v);
        if (a.residual)
#pragma unroll
            for (int e = 0; e < N; ++e) v[e] += (float)residual.e[e];
    }
    if (a.wide_out)
        store_wide<N>((float*)out, n, v);
    else
        store_some<T, N>((T*)out, n, v);
}
template <typename T, int N>
__device__ __forceinline__ void finish(const GemmArgs& a, int group, int i, int j, float (&v)[N]) {
    if (j >= a.j) return;
    Some<T, N> r = {};
    if (a.residual && group >= 0)
        r = load_some<T, N>((const T*)a.residual + (uint64_t)i * a.residual_ld + j, a.j - j);
    const uint64_t at = (a.out_group ? (uint64_t)group * a.out_group : 0) + (uint64_t)i * a.out_ld + j;
    finish<T, N>(a, group, a.j - j, v, bias_of<T, N>(a, group, j), r,
                 (T*)a.z + (uint64_t)i * a.z_ld + j, (char*)a.out + at * (a.wide_out ? 4 : sizeof(T)));
}

// g u, rounded to 32 bits: where a rounding to fp16 follows in the same block of code, the compiler
// makes both one instruction with one rounding, and out would depend on whether z is kept in 8 bits.
template <int N> __device__ __forceinline__ void times(float (&g)[N], const float (&u)[N]) {
#pragma unroll
    for (int e = 0; e < N; ++e) {
        g[e] *= u[e];
        asm("" : "+v"(g[e]));
    }
}

// Both halves' sums of N neighbouring columns: z = sums + bias, out = act(z gate) times z of the
// other; zeros for a row of no group.  z and out: of the first of the columns.
template <typename T, int N>
__device__ __forceinline__ void finish_gated(const GemmArgs& a, int group, int n, float (&g)[N], float (&u)[N],
                                             const Some<T, N>& g_bias, const Some<T, N>& u_bias, T* z, T* out) {
#pragma unroll
    for (int e = 0; e < N; ++e) {
        g[e] = group < 0 ? 0.0f : g[e] + (float)g_bias.e[e];
        u[e] = group < 0 ? 0.0f : u[e] + (float)u_bias.e[e];
    }
    if (a.z) {
        store_some<T, N>(z, n, g);
        store_some<T, N>(z + a.j, n, u);
    }
    act_values(a.act, g);
    times(g, u);
    store_some<T, N>(out, n, g);
}
template <typename T, int N>
__device__ __forceinline__ Some<T, N> gated_bias_of(const GemmArgs& a, int group, int half, int j) {
    if (!a.bias || group < 0 || j >= a.j) return Some<T, N>{};
    return load_some<T, N>((const T*)a.bias + ((uint64_t)group * 2 + half) * a.j + j, a.j - j);
}
template <typename T, int N>
__device__ __forceinline__ void finish_gated(const GemmArgs& a, int group, int i, int j, float (&g)[N], float (&u)[N]) {
    if (j >= a.j) return;
    finish_gated<T, N>(a, group, a.j - j, g, u, gated_bias_of<T, N>(a, group, 0, j), gated_bias_of<T, N>(a, group, 1, j),
                       (T*)a.z + (uint64_t)i * a.z_ld + j, (T*)a.out + (uint64_t)i * a.out_ld + j);
}

// ------------------------------------------------------------------ 8-bit values --

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// The least power of two p with a / p <= 448 = 1.75 * 2^8, at least 2^-126; 1 for 0.  Its
// exponent is a's less 8, or less 7 where a's mantissa is over 1.75.
__device__ __forceinline__ float scale_of(float a) {
    const uint32_t bits = __builtin_bit_cast(uint32_t, a);
    const int e = (int)(bits >> 23) - 8 + ((bits & 0x7FFFFF) > 0x600000);
    return a == 0.0f ? 1.0f : __builtin_bit_cast(float, (uint32_t)max(e, 1) << 23);
}
// 1 / p: exponents 254 - e of e = 1 .. 247
__device__ __forceinline__ float inverse_of(float scale) {
    return __builtin_bit_cast(float, 0x7F000000u - __builtin_bit_cast(uint32_t, scale));
}
// The largest finite magnitude.
__device__ __forceinline__ float largest_of(const float (&v)[8]) {
    float a = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) a = fmaxf(a, fabsf(v[e]) < INFINITY ? fabsf(v[e]) : 0.0f);
    return a;
}
// In e4m3, times 1 / p: exact but for the rounding to e4m3.
__device__ __forceinline__ u32x2 narrow(const float (&v)[8], float inverse) {
    u32x2 w;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float f[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = fabsf(v[h * 4 + e]) < INFINITY ? v[h * 4 + e] * inverse : NAN;
        int word = __builtin_amdgcn_cvt_pk_fp8_f32(f[0], f[1], 0, false);
        word = __builtin_amdgcn_cvt_pk_fp8_f32(f[2], f[3], word, true);
        w[h] = (uint32_t)word;
    }
    return w;
}
__device__ __forceinline__ void store_eight(uint8_t* p, int n, u32x2 v) {
    if (n >= 8) {
        ((LooseWords<uint8_t, 8>*)p)->v = v;
    } else {
        for (int e = 0; e < n; ++e) p[e] = (uint8_t)(v[e >> 2] >> (e & 3) * 8);
    }
}

// ------------------------------------------------------------- where a tile is --

struct Spot {
    Range g;
    int i0, i_end, c0, c_end, j0, split;
    int parts;        // of the contraction, in the last round: 1, or this is part `split` of
    unsigned tile;    // its tile `tile`
};

// Workgroup -> tile.  Workgroups go to the 8 XCDs in turn, each with an L2 of its own:
// every XCD takes one stretch of the tiles, and a stretch goes through kHigh rows of tiles
// column by column, so that the 32 tiles in flight on an XCD share operands.  6 rows: with 8,
// the tiles that finish together lie a power of two apart, and their residuals and results
// on the same channels of memory (8192 x 8192 x 4096 with all of the epilogue: 469 us with 8,
// 476 with 4, 439 with 6; without the stretches 526).
constexpr unsigned kHigh = 6;

template <bool BY_ROWS, int TI, int TJ>
__device__ __forceinline__ bool find_spot(const GemmArgs& a, const RowTiles& rows, unsigned number, Spot& s) {
    const unsigned tiles_i = BY_ROWS ? (unsigned)rows.total : (unsigned)a.tiles_i;
    const unsigned tiles = tiles_i * (unsigned)a.tiles_j;
    if (tiles == 0) return false;
    s.parts = 1;
    s.tile = 0;
    if (a.slots) {
        const unsigned whole = tiles / (unsigned)a.slots * (unsigned)a.slots, rest = tiles - whole;
        const int parts = last_round_parts(rest, (unsigned)a.slots, a.steps);
        if (number >= whole && parts > 1) {
            const unsigned i = number - whole;
            if (i >= rest * (unsigned)parts) return false;
            s.parts = parts;
            s.tile = i % rest;
            s.split = (int)(i / rest);
            number = whole + s.tile;
        }
    }
    const unsigned outer = number / tiles, id = number % tiles;
    if (outer >= (unsigned)a.splits * (BY_ROWS ? 1u : (unsigned)a.groups)) return false;
    const unsigned xcd = id & 7, each = tiles >> 3, more = tiles & 7;
    const unsigned at = xcd * each + min(xcd, more) + (id >> 3);
    const unsigned tall = kHigh * (unsigned)a.tiles_j, first = at / tall * kHigh;
    const unsigned high = min(kHigh, tiles_i - first), in = at % tall;
    const int ti = (int)(first + in % high);
    s.j0 = (int)(in / high) * TJ;
    int c_lo, c_hi;
    if constexpr (BY_ROWS) {
        if (s.parts == 1) s.split = (int)outer;
        if (!find_tile(a, rows, ti, TI, s.g)) return false;
        s.i0 = s.g.lo;
        s.i_end = s.g.hi;
        c_lo = 0;
        c_hi = s.g.group < 0 ? 0 : a.c;
    } else {
        if (s.parts == 1) s.split = (int)(outer / (unsigned)a.groups);
        s.g = range_of(a, (int)(outer % (unsigned)a.groups) + 1);
        s.i0 = ti * TI;
        s.i_end = a.i;
        c_lo = s.g.lo;
        c_hi = s.g.hi;
    }
    s.g.group = __builtin_amdgcn_readfirstlane(s.g.group);
    s.i0 = __builtin_amdgcn_readfirstlane(s.i0);
    s.i_end = __builtin_amdgcn_readfirstlane(s.i_end);
    c_lo = __builtin_amdgcn_readfirstlane(c_lo);
    c_hi = __builtin_amdgcn_readfirstlane(c_hi);
    s.c0 = c_lo;
    s.c_end = c_hi;
    const int parts = a.splits * s.parts;    // one of them is 1
    if (parts > 1) {
        const int each_c = ((c_hi - c_lo + kDepth - 1) / kDepth + parts - 1) / parts;
        const int64_t lo = c_lo + (int64_t)s.split * each_c * kDepth;
        s.c0 = (int)min(lo, (int64_t)c_hi);
        s.c_end = (int)min(lo + (int64_t)each_c * kDepth, (int64_t)c_hi);
    }
    return true;
}

// The results of the workgroup: FI x FJ blocks of 16 x 16 a wave.  The matrix instruction
// takes Q as its first operand, so that a lane's four results are neighbours in a row.
// Written from there, an access would touch 16 rows at 32 bytes each, all on one channel
// of the L2 where the rows are a power of two apart (8192 x 8192 outputs of a contraction one
// row deep: 171 us); instead 16 rows of every wave at a time go through LDS in 32 bits
// and leave as whole rows of the tile, 8 columns a thread (58 us).
template <typename T, bool BY_ROWS, int TI, int TJ, int WI, int WJ, int FI, int FJ>
__device__ __forceinline__ void write_out(const GemmArgs& a, const Spot& s, BLK_LDS char* room,
                                          const f32x4 (&acc)[FI][FJ]) {
    constexpr int THREADS = 64 * WI * WJ, LINE = TJ + 4, ROWS = 16 * WI, GROUPS = TJ / 8;
    constexpr int BUFFER = ROWS * LINE, EACH = ROWS * GROUPS / THREADS;
    static_assert(THREADS % GROUPS == 0, "a thread keeps its columns");
    BLK_LDS float* const store = (BLK_LDS float*)room;
    const int thread = here(), lane = thread & 63, wave = thread >> 6;
    const bool whole = a.splits == 1 && s.parts == 1, add = whole && a.residual && s.g.group >= 0;
    if (!whole && s.g.group < 0) return;        // join_kernel knows
    if (thread >= THREADS) {                    // of another part: there for the barriers
        for (int x = 0; x < FI; ++x) __syncthreads();
        return;
    }
    const int col = thread % GROUPS * 8, n = a.j - s.j0 - col;
    // A tile of whole columns knows that of all its threads.  With the last columns, the tile
    // takes one way for all threads too: two in one wave, for its whole and its cut pieces of
    // 8 columns, would be two epilogues (3000 x 3001 x 3001 with GELU 102 us instead of 87).
    const bool inside = s.j0 + TJ <= a.j;
    // A matrix's rows: those of block row 0 by 32-bit offsets from the tile's corner, and 16
    // rows on for each block row (rows are at most 2^22 elements apart).
    const uint64_t corner_out = (a.out_group && whole ? (uint64_t)s.g.group * a.out_group : 0);
    const uint32_t wide = whole && !a.wide_out ? sizeof(T) : 4;
    const uint64_t out_ld = whole ? a.out_ld : s.parts > 1 ? (uint64_t)TJ : (uint64_t)a.j;
    const uint64_t part_row = BY_ROWS ? (uint64_t)s.i0 : (uint64_t)s.g.group * a.i + s.i0;
    const char* out = whole ? (const char*)a.out + (corner_out + (uint64_t)s.i0 * out_ld + s.j0) * wide
                      : s.parts > 1
                          ? (const char*)(a.part + ((uint64_t)s.tile * s.parts + s.split) * (TI * TJ))
                          : (const char*)(a.part + (uint64_t)s.split * a.part_stride + part_row * out_ld + s.j0);
    const char* z = (const char*)a.z + ((uint64_t)s.i0 * a.z_ld + s.j0) * sizeof(T);
    const char* res = (const char*)a.residual + ((uint64_t)s.i0 * a.residual_ld + s.j0) * sizeof(T);
    out = uniform(out);
    z = uniform(z);
    res = uniform(res);
    uint32_t at_out[EACH], at_z[EACH], at_res[EACH];
    int left[EACH];                                   // rows from this one to the tile's end
#pragma unroll
    for (int t = 0; t < EACH; ++t) {
        const int r = t * (THREADS / GROUPS) + thread / GROUPS;
        const uint32_t row = r / 16 * (TI / WI) + r % 16;
        at_out[t] = (row * (uint32_t)out_ld + col) * wide;
        at_z[t] = (row * (uint32_t)a.z_ld + col) * (uint32_t)sizeof(T);
        at_res[t] = (row * (uint32_t)a.residual_ld + col) * (uint32_t)sizeof(T);
        left[t] = n > 0 ? s.i_end - s.i0 - (int)row : 0;
    }
    const Some<T, 8> bias = whole ? bias_of<T, 8>(a, s.g.group, s.j0 + col) : Some<T, 8>{};
    Some<T, 8> residual[EACH] = {}, later[EACH] = {};
    const auto fetch = [&](Some<T, 8> (&to)[EACH], int x) {
        const char* from = res + (uint64_t)(x * 16) * a.residual_ld * sizeof(T);
#pragma unroll
        for (int t = 0; t < EACH; ++t)
            if (x * 16 < left[t]) to[t] = load_some<T, 8>((const T*)(from + at_res[t]), 8);
    };
    if (add && inside) fetch(residual, 0);
    for (int x = 0; x < FI; ++x) {
        BLK_LDS float* const buf = store + (x & 1) * BUFFER;
        BLK_LDS float* const mine = buf + (wave / WJ * 16 + (lane & 15)) * LINE + wave % WJ * (TJ / WJ) + (lane >> 4) * 4;
        if (add && inside && x + 1 < FI) fetch(later, x + 1);
#pragma unroll
        for (int u = 0; u < FI; ++u)
            if (u == x)
#pragma unroll
                for (int y = 0; y < FJ; ++y) *(BLK_LDS f32x4*)(mine + y * 16) = acc[u][y];
        __syncthreads();
        char* const to = (char*)out + (uint64_t)(x * 16) * out_ld * wide;
        const char* const to_z = z + (uint64_t)(x * 16) * a.z_ld * sizeof(T);
#pragma unroll
        for (int t = 0; t < EACH; ++t) {
            const BLK_LDS float* const from = buf + (t * (THREADS / GROUPS) + thread / GROUPS) * LINE + col;
            if (x * 16 >= left[t]) continue;
            const f32x4 lo = *(const BLK_LDS f32x4*)from, hi = *(const BLK_LDS f32x4*)(from + 4);
            float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
            if (!whole) {
                store_wide<8>((float*)(to + at_out[t]), n, v);
            } else if (inside) {
                finish<T, 8>(a, s.g.group, 8, v, bias, residual[t], (T*)(to_z + at_z[t]), to + at_out[t]);
            } else {
                Some<T, 8> r = {};
                if (add) r = load_some<T, 8>((const T*)(res + (uint64_t)(x * 16) * a.residual_ld * sizeof(T) + at_res[t]), n);
                finish<T, 8>(a, s.g.group, n, v, bias, r, (T*)(to_z + at_z[t]), to + at_out[t]);
            }
        }
#pragma unroll
        for (int t = 0; t < EACH; ++t) residual[t] = later[t];
    }
}

// The same of a gated product: the tile's columns are TJ / 2 of the gate and the other
// projection's behind them, so a thread finds both sums of its 8 columns in LDS.  (Of tiles whose
// contraction is in no parts but those of the workgroup.)
template <typename T, int TI, int TJ, int WI, int WJ, int FI, int FJ>
__device__ __forceinline__ void write_gated(const GemmArgs& a, const Spot& s, BLK_LDS char* room,
                                            const f32x4 (&acc)[FI][FJ]) {
    constexpr int THREADS = 64 * WI * WJ, LINE = TJ + 4, ROWS = 16 * WI, HALF = TJ / 2, GROUPS = HALF / 8;
    constexpr int BUFFER = ROWS * LINE;
    static_assert(ROWS * GROUPS <= THREADS, "a thread has one piece of 16 rows a wave");
    BLK_LDS float* const store = (BLK_LDS float*)room;
    const int thread = here(), lane = thread & 63, wave = thread >> 6;
    if (thread >= THREADS) {                    // of another part: there for the barriers
        for (int x = 0; x < FI; ++x) __syncthreads();
        return;
    }
    const int col = thread % GROUPS * 8, r = thread / GROUPS, j = s.j0 + col, n = a.j - j;
    const int row = r / 16 * (TI / WI) + r % 16, i = s.i0 + row;
    const int left = r < ROWS && n > 0 ? s.i_end - i : 0;
    const Some<T, 8> g_bias = gated_bias_of<T, 8>(a, s.g.group, 0, j), u_bias = gated_bias_of<T, 8>(a, s.g.group, 1, j);
    T* const z = (T*)a.z + (uint64_t)i * a.z_ld + j;
    T* const out = (T*)a.out + (uint64_t)i * a.out_ld + j;
    for (int x = 0; x < FI; ++x) {
        BLK_LDS float* const buf = store + (x & 1) * BUFFER;
        BLK_LDS float* const mine = buf + (wave / WJ * 16 + (lane & 15)) * LINE + wave % WJ * (TJ / WJ) + (lane >> 4) * 4;
#pragma unroll
        for (int u = 0; u < FI; ++u)
            if (u == x)
#pragma unroll
                for (int y = 0; y < FJ; ++y) *(BLK_LDS f32x4*)(mine + y * 16) = acc[u][y];
        __syncthreads();
        if (x * 16 >= left) continue;
        const BLK_LDS float* const from = buf + r * LINE + col;
        float g[8], u[8];
#pragma unroll
        for (int h = 0; h < 8; h += 4) {
            const f32x4 gv = *(const BLK_LDS f32x4*)(from + h), uv = *(const BLK_LDS f32x4*)(from + HALF + h);
#pragma unroll
            for (int e = 0; e < 4; ++e) g[h + e] = gv[e], u[h + e] = uv[e];
        }
        const uint64_t down = (uint64_t)(x * 16);
        finish_gated<T, 8>(a, s.g.group, n, g, u, g_bias, u_bias, z + down * a.z_ld, out + down * a.out_ld);
    }
}

template <int N> struct Int {
    static constexpr int value = N;
};

// ------------------------------------------------------------------ the product --

// Bound, at 256 x 256, by power and the way from the L2s into LDS: with all loads but the
// first taken out 8192 x 8192 x 8192 takes 646 us (1700 TFLOP/s), with loads that all hit the
// L2 742, as it is 770 (1430).  A tile of 256 x 256 moves 64 KiB into LDS for 8.4 MFLOP; 128 x
// 128 ones move twice that for their work and reach 12 TB/s between L2s and LDS at 700
// TFLOP/s.  Eight waves of 128 x 64 keep a step's reads of LDS at 192 KiB; four of 128 x 128
// read 128 KiB but leave a SIMD one wave (the loop 7% faster, start and end 60 us slower).
//
// STAGES tiles of the operands are in LDS or on their way there, and of Q half a step longer
// one more: its loads and P's then go out in different halves of a step, where both at once
// wait for each other (8192 x 8192 x 8192 810 us instead of 772, 1600 x 4096 x 4096 69 instead
// of 59, small products 2%).  At 256 x 256 these are all 160 KB.  Where a compute unit has one
// or two workgroups, the time of a step is the loads' way through memory, and four stages
// take as many steps to hide it.
//
// PARTS parts of the contraction are multiplied by as many sets of waves, whose sums meet in
// LDS, so that few rows fill the device without a second launch that adds them up.
//
// GATED: Q's tile is TJ / 2 rows of each of two matrices, for TJ / 2 columns of out; of few rows
// only, kInner64 (blk_tile.hpp has the others).
template <typename T, bool PA, bool QA, bool BY_ROWS, int TI, int TJ, int WI, int WJ, int STAGES, int PARTS = 1,
          bool GATED = false>
__global__ void __launch_bounds__(64 * WI * WJ * PARTS, STAGES * (TI + TJ) * kDepth * 2 > 81920 && WI * WJ == 4 ? 1 : 2)
gemm_kernel(const GemmArgs a) {
    typedef typename Mma<T>::V V;
    constexpr int THREADS = 64 * WI * WJ, FI = TI / WI / 16, FJ = TJ / WJ / 16;
    constexpr int PB = Tile<PA, TI>::kBytes, QB = Tile<QA, TJ>::kBytes;
    constexpr uint32_t PLACES = STAGES * PB + (STAGES + 1) * QB;    // P's, then Q's
    constexpr uint32_t OUT = 2 * 16 * WI * (TJ + 4) * 4;   // write_out's place
    __shared__ __align__(PB) char lds[OUT > PARTS * PLACES ? OUT : PARTS * PLACES];
    BLK_LDS char* const room = (BLK_LDS char*)lds;
    RowTiles rows = {};
    if constexpr (BY_ROWS) rows = count_tiles(a, TI);
    Spot s;
    if (!find_spot<BY_ROWS, TI, GATED ? TJ / 2 : TJ>(a, rows, blockIdx.x, s)) return;
    const T* const p = (const T*)a.p;
    const T* const q = (const T*)a.q + (BY_ROWS && s.g.group > 0 ? (uint64_t)s.g.group * a.q_group : 0);
    int wave = threadIdx.x >> 6, part = 0, tiles = (s.c_end - s.c0 + kDepth - 1) / kDepth;
    if constexpr (PARTS > 1) {
        part = __builtin_amdgcn_readfirstlane(wave / (WI * WJ));
        wave %= WI * WJ;
        tiles = (tiles + PARTS - 1) / PARTS;       // of each; the last ones may be past the end
        const int64_t lo = s.c0 + (int64_t)part * tiles * kDepth;
        s.c0 = (int)min(lo, (int64_t)s.c_end);
        s.c_end = (int)min(lo + (int64_t)tiles * kDepth, (int64_t)s.c_end);
    }
    const int wi = wave / WJ * (TI / WI), wj = wave % WJ * (TJ / WJ);
    Reader<PA, TI> rp;
    Reader<QA, TJ> rq;
    const uint32_t p_at = (uint32_t)(uintptr_t)room + part * PLACES, q_at = p_at + STAGES * PB;
    rp.start(p_at, wi);
    rq.start(q_at, wj);
    f32x4 acc[FI][FJ];
#pragma unroll
    for (int x = 0; x < FI; ++x)
#pragma unroll
        for (int y = 0; y < FJ; ++y) acc[x][y] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    // Half a tile (32 deep) is multiplied from registers while the next half is read into
    // others.  Behind the barrier in the middle of a tile the next tile has arrived; the loads
    // of P that are STAGES tiles ahead follow into the place just read, those of Q, which has
    // one place more, in the next tile's first half.
    typedef Direct<T, PA, TI, THREADS, (PARTS > 1)> DP;
    typedef std::conditional_t<GATED, Twin<T, QA, TJ, THREADS, (PARTS > 1)>, Direct<T, QA, TJ, THREADS, (PARTS > 1)>> DQ;
    constexpr int PIECES = DP::kPieces + DQ::kPieces;
    DP lp;
    DQ lq;
    lp.start(p, a.p_ld, s.i0, s.i_end, s.c0, s.c_end);
    if constexpr (GATED) lq.start(q, a.q_half, a.q_ld, s.j0, a.j, s.c0, s.c_end);
    else lq.start(q, a.q_ld, s.j0, a.j, s.c0, s.c_end);
    V fp[2][FI], fq[2][FJ];
    // reads of the other half in the first part of the block rows, so that they are done
    // when the last ones are
    constexpr int READS = FI / 2;
    const auto read = [&](int half, int x) {
#pragma unroll
        for (int y = x * FJ / READS; y < (x + 1) * FJ / READS; ++y) fq[half][y] = rq.template fragment<V>(y, half);
#pragma unroll
        for (int r = x * FI / READS; r < (x + 1) * FI / READS; ++r) fp[half][r] = rp.template fragment<V>(r, half);
    };
    const auto multiply = [&](auto now_) {
        constexpr int now = decltype(now_)::value;
        __builtin_amdgcn_s_setprio(now);     // loads and first reads behind the barrier go first
#pragma unroll
        for (int x = 0; x < FI; ++x) {
            if constexpr (now == 0) {
#pragma unroll
                for (int k = x * DQ::kPieces / FI; k < (x + 1) * DQ::kPieces / FI; ++k) lq.piece(k);
            } else {
#pragma unroll
                for (int k = x * DP::kPieces / FI; k < (x + 1) * DP::kPieces / FI; ++k) lp.piece(k);
            }
            if (x < READS) read(now ^ 1, x);
            if (now == 1 && x == FI / 2) __builtin_amdgcn_s_setprio(0);
#pragma unroll
            for (int y = 0; y < FJ; ++y) acc[x][y] = Mma<T>::run(fq[now][y], fp[now][x], acc[x][y]);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    if (tiles > 0) {
#pragma unroll
        for (int t = 0; t < STAGES; ++t) {
            lp.aim(p_at + t * PB);
            lq.aim(q_at + t * QB);
#pragma unroll
            for (int k = 0; k < DP::kPieces; ++k) lp.piece(k);
#pragma unroll
            for (int k = 0; k < DQ::kPieces; ++k) lq.piece(k);
        }
        arrived<PIECES * (STAGES - 1)>();
#pragma unroll
        for (int x = 0; x < READS; ++x) read(0, x);
    }
    // the places of the tile that is read, and where Q's loads go
    uint32_t p_now = 0, q_now = 0, q_new = STAGES * QB;
    for (int t = 0; t < tiles; ++t) {
        __builtin_amdgcn_s_waitcnt(0xC07F);  // the reads of half 0, before new ones
        lq.aim(q_at + q_new);
        q_new = q_now;
        multiply(Int<0>());
        // all but the loads behind the next tile's: of Q one tile's more than of P
        arrived<PIECES * (STAGES - 2) + DQ::kPieces>();
        lp.aim(p_at + p_now);
        const uint32_t by_p = p_now == (STAGES - 1) * PB ? -p_now : PB;
        const uint32_t by_q = q_now == STAGES * QB ? -q_now : QB;
        p_now += by_p;
        q_now += by_q;
        rp.move(by_p);
        rq.move(by_q);
        multiply(Int<1>());
    }
    arrived<0>();                            // the zeros past the end as well
    if constexpr (PARTS > 1) {
        BLK_LDS f32x4* const sums = (BLK_LDS f32x4*)room + (wave * FI * FJ * 64 + (threadIdx.x & 63));
        constexpr int EACH = WI * WJ * FI * FJ * 64;
        if (part > 0)
#pragma unroll
            for (int f = 0; f < FI * FJ; ++f) sums[(part - 1) * EACH + f * 64] = acc[f / FJ][f % FJ];
        __syncthreads();
        if (part == 0)
#pragma unroll
            for (int f = 0; f < FI * FJ; ++f)
#pragma unroll
                for (int m = 0; m < PARTS - 1; ++m) acc[f / FJ][f % FJ] += sums[m * EACH + f * 64];
        __syncthreads();
    }
    if constexpr (GATED) write_gated<T, TI, TJ, WI, WJ, FI, FJ>(a, s, room, acc);
    else write_out<T, BY_ROWS, TI, TJ, WI, WJ, FI, FJ>(a, s, room, acc);
}

// ------------------------------------------------------------ few rows: one pass --
//
// The forward product of a few rows is the read of the weights (4 x 4096 x 4096 bf16: 9.9 us,
// 4 x 8192 x 4096 15.7; 4 x 8192 x 8192 27, 4.9 TB/s, where the tiles above need 24).  A
// workgroup takes 16 FI rows x 16 FJ columns, its waves
// parts of the contraction, 128 deep each in turn;
// operands go from memory to registers in the fragments' own layout (a lane's 16 bytes
// are 8 values of one row, four lanes make 64 neighbouring bytes), and the waves' sums
// meet in LDS, added in the order of the waves.
constexpr int kStreamWaves = 8, kStreamDepth = 128;

template <typename T, int R, bool DIRECT> struct Strip {
    const T* base;
    uint64_t ld;
    int row, row_end, c_end;
    uint32_t at[R];
    __device__ __forceinline__ void start(const T* b, uint64_t stride, int r0, int r_end, int end) {
        const int lane = threadIdx.x & 63;
        row = r0;
        row_end = r_end;
        c_end = end;
        ld = stride;
        base = DIRECT ? (const T*)uniform((const char*)(b + (uint64_t)r0 * stride)) : b;
        if constexpr (DIRECT)
#pragma unroll
            for (int f = 0; f < R; ++f) {
                const int y = f * 16 + (lane & 15);
                at[f] = r0 + y < r_end ? (uint32_t)((uint64_t)y * stride * sizeof(T)) : kReach;
            }
    }
    __device__ __forceinline__ void load(u32x4 (&v)[4][R], int c0) const {
        const int lane = threadIdx.x & 63;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            constexpr int N = Vec<T>::N;
            const int c = c0 + s * 4 * N + (lane >> 4) * N;
#pragma unroll
            for (int f = 0; f < R; ++f) {
                if constexpr (DIRECT) {
                    const auto rsrc = __builtin_amdgcn_make_buffer_rsrc((void*)base, 0, kReach, 0x00027000);
                    v[s][f] = __builtin_amdgcn_raw_buffer_load_b128(
                        rsrc, c < c_end ? at[f] + (uint32_t)c * (uint32_t)sizeof(T) : kReach, 0, 0);
                } else if constexpr (sizeof(T) == 1) {
                    // rows of at least 16 bytes: whole pieces, the last one's without its first
                    const int y = row + f * 16 + (lane & 15), from = min(c, c_end - 16);
                    const u32x4 t = load_raw(base + (uint64_t)min(y, row_end - 1) * ld + from);
                    v[s][f] = zero_unless(y < row_end, drop_first(t, min(c - from, 16)));
                } else {
                    Vec<T> t;
#pragma unroll
                    for (int e = 0; e < N; ++e) t.e[e] = (T)0.0f;
                    const int y = row + f * 16 + (lane & 15);
                    if (y < row_end && c < c_end) t = load_vec(base + (uint64_t)y * ld, c, c_end);
                    v[s][f] = __builtin_bit_cast(u32x4, t);
                }
            }
        }
    }
};

// The waves' sums, added in the order of the waves.
template <typename T, int FI, int FJ>
__device__ __forceinline__ void finish_stream_plain(const GemmArgs& a, int group, int i0, int i_end, int j0, int wave,
                                                    const f32x4 (&sums)[kStreamWaves][FI * FJ][64]) {
    const int lane = threadIdx.x & 63;
    for (int f = wave; f < FI * FJ; f += kStreamWaves) {
        f32x4 v = sums[0][f][lane];
#pragma unroll
        for (int w = 1; w < kStreamWaves; ++w) v += sums[w][f][lane];
        const int i = i0 + f / FJ * 16 + (lane & 15);
        const int j = j0 + f % FJ * 16 + (lane >> 4) * 4;
        float o[4] = {v[0], v[1], v[2], v[3]};
        if (i >= i_end || j >= a.j) continue;
        if (a.splits == 1)
            finish<T, 4>(a, group, i, j, o);
        else if (group >= 0)
            store_wide<4>(a.part + (uint64_t)blockIdx.z * a.part_stride + (uint64_t)i * a.j + j, a.j - j, o);
    }
}

// The same of a gated product: 16 columns of each projection.
template <typename T, int FI>
__device__ __forceinline__ void finish_stream(const GemmArgs& a, int group, int i0, int i_end, int j0, int wave,
                                              const f32x4 (&sums)[kStreamWaves][FI * 2][64]) {
    const int lane = threadIdx.x & 63;
    for (int f = wave; f < FI; f += kStreamWaves) {
        f32x4 g = sums[0][f * 2][lane], u = sums[0][f * 2 + 1][lane];
#pragma unroll
        for (int w = 1; w < kStreamWaves; ++w) {
            g += sums[w][f * 2][lane];
            u += sums[w][f * 2 + 1][lane];
        }
        const int i = i0 + f * 16 + (lane & 15), j = j0 + (lane >> 4) * 4;
        if (i >= i_end || j >= a.j) continue;
        float gv[4] = {g[0], g[1], g[2], g[3]}, uv[4] = {u[0], u[1], u[2], u[3]};
        if (a.splits == 1) {
            finish_gated<T, 4>(a, group, i, j, gv, uv);
        } else if (group >= 0) {
            float* const to = a.part + (uint64_t)blockIdx.z * a.part_stride + (uint64_t)i * 2 * a.j + j;
            store_wide<4>(to, a.j - j, gv);
            store_wide<4>(to + a.j, a.j - j, uv);
        }
    }
}

// GATED (FJ 2): 16 columns of the gate and the same 16 of the other projection.
template <typename T, int FI, int FJ, bool DIRECT, bool GATED = false>
__global__ void __launch_bounds__(64 * kStreamWaves) stream_kernel(const GemmArgs a) {
    typedef typename Mma<T>::V V;
    __shared__ f32x4 sums[kStreamWaves][FI * FJ][64];
    Range g;
    if (!find_tile(a, count_tiles(a, 16 * FI), (int)blockIdx.y, 16 * FI, g)) return;
    g.group = __builtin_amdgcn_readfirstlane(g.group);
    const int i0 = __builtin_amdgcn_readfirstlane(g.lo), i_end = __builtin_amdgcn_readfirstlane(g.hi);
    constexpr int HALVES = GATED ? 2 : 1, EACH = FJ / HALVES;
    const int j0 = (int)blockIdx.x * (16 * EACH), lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    int c_lo = 0, c_end = g.group < 0 ? 0 : a.c;
    if (a.splits > 1) {
        const int each = ((a.c + kStreamDepth - 1) / kStreamDepth + a.splits - 1) / a.splits * kStreamDepth;
        c_lo = (int)min((int64_t)blockIdx.z * each, (int64_t)c_end);
        c_end = (int)min((int64_t)c_lo + each, (int64_t)c_end);
    }
    Strip<T, FI, DIRECT> sp;
    Strip<T, EACH, DIRECT> sq[HALVES];
    sp.start((const T*)a.p, a.p_ld, i0, i_end, c_end);
#pragma unroll
    for (int h = 0; h < HALVES; ++h)
        sq[h].start((const T*)a.q + (g.group > 0 ? (uint64_t)g.group * a.q_group : 0) + h * a.q_half, a.q_ld, j0, a.j, c_end);
    f32x4 acc[FI][FJ];
#pragma unroll
    for (int x = 0; x < FI; ++x)
#pragma unroll
        for (int y = 0; y < FJ; ++y) acc[x][y] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    u32x4 vp[4][FI], vq[HALVES][4][EACH];
    const auto load = [&](u32x4 (&to_p)[4][FI], u32x4 (&to_q)[HALVES][4][EACH], int at) {
#pragma unroll
        for (int h = 0; h < HALVES; ++h) sq[h].load(to_q[h], at);
        sp.load(to_p, at);
    };
    int c = c_lo + wave * kStreamDepth;
    if (c < c_end) load(vp, vq, c);
    while (c < c_end) {
        c += kStreamWaves * kStreamDepth;
        u32x4 np[4][FI], nq[HALVES][4][EACH];
        if (c < c_end) load(np, nq, c);
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int x = 0; x < FI; ++x)
#pragma unroll
                for (int y = 0; y < FJ; ++y)
                    acc[x][y] = Mma<T>::run(__builtin_bit_cast(V, vq[y / EACH][s][y % EACH]),
                                            __builtin_bit_cast(V, vp[s][x]), acc[x][y]);
#pragma unroll
        for (int s = 0; s < 4; ++s) {
#pragma unroll
            for (int x = 0; x < FI; ++x) vp[s][x] = np[s][x];
#pragma unroll
            for (int y = 0; y < FJ; ++y) vq[y / EACH][s][y % EACH] = nq[y / EACH][s][y % EACH];
        }
    }
#pragma unroll
    for (int x = 0; x < FI; ++x)
#pragma unroll
        for (int y = 0; y < FJ; ++y) sums[wave][x * FJ + y][lane] = acc[x][y];
    __syncthreads();
    if constexpr (GATED) finish_stream<T, FI>(a, g.group, i0, i_end, j0, wave, sums);
    else finish_stream_plain<T, FI, FJ>(a, g.group, i0, i_end, j0, wave, sums);
}

// -------------------------------------------------------- one to four rows: dots --
//
// Up to four rows of one group: a wave goes along one row of the weights, or two, 1 KiB of
// each at a time, and adds products in 32 bits on the vector units.  The weights are read in
// memory's own order and at any alignment: 1 x 8192 x 8192 takes 23 us (5.8 TB/s) against 27 of
// the one-pass form above, 1 x 4096 x 4096 7.3 against 9.9, 3 x 572 x 2366 (rows without whole
// 16-byte pieces) 6.2 against 16.  Every row of x costs as many loads from the caches as the
// weights do from memory, so with aligned rows it ends at two (2 x 8192 x 8192: 23 against 27;
// 4: 46 against 27).
constexpr int kDotWaves = 4;

// GATED (R 2): the wave's rows are one of each projection.
template <typename T, int M, int R, bool GATED = false>
__global__ void __launch_bounds__(64 * kDotWaves) dot_kernel(const GemmArgs a) {
    const int lane = threadIdx.x & 63;
    const int j0 = ((int)blockIdx.x * kDotWaves + (int)(threadIdx.x >> 6)) * (GATED ? 1 : R);
    if (j0 >= a.j) return;
    const T *w[R], *x[M];
#pragma unroll
    for (int r = 0; r < R; ++r)
        w[r] = (const T*)a.q + (GATED ? r * a.q_half + (uint64_t)j0 * a.q_ld : (uint64_t)min(j0 + r, a.j - 1) * a.q_ld);
#pragma unroll
    for (int m = 0; m < M; ++m) x[m] = (const T*)a.p + (uint64_t)m * a.p_ld;
    float sum[M][R];
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
        for (int r = 0; r < R; ++r) sum[m][r] = 0.0f;
    const auto add = [&](const u32x4 (&wv)[R], const u32x4 (&xv)[M]) {
        float f[M][8];
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
            for (int e = 0; e < 8; ++e) f[m][e] = (float)vec_of<T>(xv[m]).e[e];
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float v = (float)vec_of<T>(wv[r]).e[e];
#pragma unroll
                for (int m = 0; m < M; ++m) sum[m][r] = fmaf(f[m][e], v, sum[m][r]);
            }
    };
    constexpr int STEP = 64 * 8, AHEAD = 4;
    int c = 0;
    for (; c + AHEAD * STEP <= a.c; c += AHEAD * STEP) {
        u32x4 wv[AHEAD][R], xv[AHEAD][M];
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
#pragma unroll
            for (int r = 0; r < R; ++r) wv[u][r] = load_raw(w[r] + c + u * STEP + lane * 8);
#pragma unroll
            for (int m = 0; m < M; ++m) xv[u][m] = load_raw(x[m] + c + u * STEP + lane * 8);
        }
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) add(wv[u], xv[u]);
    }
    const int whole = a.c / 8 * 8;
    for (c += lane * 8; c < whole; c += STEP) {
        u32x4 wv[R], xv[M];
#pragma unroll
        for (int r = 0; r < R; ++r) wv[r] = load_raw(w[r] + c);
#pragma unroll
        for (int m = 0; m < M; ++m) xv[m] = load_raw(x[m] + c);
        add(wv, xv);
    }
    if (whole + lane < a.c)
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
            for (int r = 0; r < R; ++r)
                sum[m][r] = fmaf((float)x[m][whole + lane], (float)w[r][whole + lane], sum[m][r]);
    if constexpr (GATED) {
        float g[1] = {0.0f}, u[1] = {0.0f};
#pragma unroll
        for (int m = 0; m < M; ++m) {
            const float gate = lane_sum<64>(sum[m][0]), other = lane_sum<64>(sum[m][1]);
            g[0] = lane == m ? gate : g[0];
            u[0] = lane == m ? other : u[0];
        }
        if (lane < M) finish_gated<T, 1>(a, 0, lane, j0, g, u);
        return;
    }
    float mine = 0.0f;
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float all = lane_sum<64>(sum[m][r]);
            mine = lane == m * R + r ? all : mine;
        }
    const int m = lane / R, j = j0 + lane % R;
    float v[1] = {mine};
    if (m < M && j < a.j) finish<T, 1>(a, 0, m, j, v);
}

template <typename T, int M, int R, bool GATED = false> static void launch_dot(const GemmArgs& a, hipStream_t s) {
    const unsigned grid = (unsigned)ceil_div(a.j, (uint64_t)(GATED ? 1 : R) * kDotWaves);
    dot_kernel<T, M, R, GATED><<<grid, 64 * kDotWaves, 0, s>>>(a);
}

// ----------------------------------------------------- parts of the contraction --

// The group of a row of the products by rows; -1: none.
__device__ __forceinline__ int group_of(const GemmArgs& a, int row) {
    if (!a.offsets) return a.groups > 1 ? row / (a.rows / a.groups) : 0;
    int lo = 0, hi = a.groups + 1;           // the first of the offsets beyond the row
    while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (a.offsets[mid] <= row) lo = mid + 1;
        else hi = mid;
    }
    return lo > a.groups ? -1 : lo - 1;
}

// Adds the parts in their order and finishes the rows: four columns a thread.
template <typename T> __global__ void __launch_bounds__(256) join_kernel(const GemmArgs a, int by_rows) {
    const unsigned wide = (unsigned)(a.j + 3) / 4;
    const uint64_t id = (uint64_t)blockIdx.x * 256 + threadIdx.x;
    const uint64_t row = id / wide;
    const int j = (int)(id % wide) * 4;
    const uint64_t rows = by_rows ? (uint64_t)a.rows : (uint64_t)a.groups * a.i;
    if (row >= rows) return;
    const int group = by_rows ? group_of(a, (int)row) : (int)(row / a.i);
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (group >= 0)
#pragma unroll 8
        for (int s = 0; s < a.splits; ++s) {
            const float* from = a.part + (uint64_t)s * a.part_stride + row * a.j + j;
            const Some<float, 4> p = load_some<float, 4>(from, a.j - j);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] += p.e[e];
        }
    finish<T, 4>(a, group, by_rows ? (int)row : (int)(row % a.i), j, v);
}

// The same of a gated product: four columns of out a thread.
template <typename T> __global__ void __launch_bounds__(256) join_gated_kernel(const GemmArgs a) {
    const unsigned wide = (unsigned)(a.j + 3) / 4;
    const uint64_t id = (uint64_t)blockIdx.x * 256 + threadIdx.x;
    const uint64_t row = id / wide;
    const int j = (int)(id % wide) * 4;
    if (row >= (uint64_t)a.rows) return;
    const int group = group_of(a, (int)row);
    float g[4] = {}, u[4] = {};
    if (group >= 0)
#pragma unroll 4
        for (int s = 0; s < a.splits; ++s) {
            const float* from = a.part + (uint64_t)s * a.part_stride + row * 2 * a.j + j;
            const Some<float, 4> gp = load_some<float, 4>(from, a.j - j), up = load_some<float, 4>(from + a.j, a.j - j);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                g[e] += gp.e[e];
                u[e] += up.e[e];
            }
        }
    finish_gated<T, 4>(a, group, (int)row, j, g, u);
}

// Adds the parts of the last round's tiles: 32 rows a workgroup.
template <typename T, bool BY_ROWS, int TI, int TJ>
__global__ void __launch_bounds__(256) join_last_kernel(const GemmArgs a) {
    RowTiles rows = {};
    if constexpr (BY_ROWS) rows = count_tiles(a, TI);
    const unsigned tiles = (BY_ROWS ? (unsigned)rows.total : (unsigned)a.tiles_i) * (unsigned)a.tiles_j;
    const unsigned whole = tiles / (unsigned)a.slots * (unsigned)a.slots, rest = tiles - whole;
    if (blockIdx.x >= rest || last_round_parts(rest, (unsigned)a.slots, a.steps) < 2) return;
    Spot s;
    if (!find_spot<BY_ROWS, TI, TJ>(a, rows, whole + blockIdx.x, s)) return;
    constexpr int GROUPS = TJ / 8;
    const int col = (int)threadIdx.x % GROUPS * 8, j = s.j0 + col;
    if (j >= a.j) return;
    const int n = a.j - j;
    const Some<T, 8> bias = bias_of<T, 8>(a, s.g.group, j);
    for (int row = (int)(blockIdx.y * 32 + threadIdx.x / GROUPS), k = 0; k < 32; k += 256 / GROUPS, row += 256 / GROUPS) {
        const int i = s.i0 + row;
        if (i >= s.i_end) return;
        float v[8] = {};
        if (s.g.group >= 0)
            for (int p = 0; p < s.parts; ++p) {
                const float* from = a.part + ((uint64_t)s.tile * s.parts + p) * (TI * TJ) + row * TJ + col;
                const f32x4 lo = *(const f32x4*)from, hi = *(const f32x4*)(from + 4);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    v[e] += lo[e];
                    v[4 + e] += hi[e];
                }
            }
        Some<T, 8> r = {};
        if (a.residual && s.g.group >= 0) r = load_some<T, 8>((const T*)a.residual + (uint64_t)i * a.residual_ld + j, n);
        const uint64_t at = (a.out_group ? (uint64_t)s.g.group * a.out_group : 0) + (uint64_t)i * a.out_ld + j;
        finish<T, 8>(a, s.g.group, n, v, bias, r, (T*)a.z + (uint64_t)i * a.z_ld + j,
                     (char*)a.out + at * (a.wide_out ? 4 : sizeof(T)));
    }
}

// -------------------------------------------------------------------- launching --

template <typename T, bool PA, bool QA, bool BY_ROWS>
static void launch_form(const GemmArgs& a, const GemmPlan& p, hipStream_t s) {
    const unsigned grid = (unsigned)a.tiles_i * a.tiles_j * a.splits * (BY_ROWS ? 1u : (unsigned)a.groups);
    if constexpr (BY_ROWS && !PA && !QA)
        if (p.tile == kInner64) {
            gemm_kernel<T, PA, QA, BY_ROWS, 64, 32, 2, 1, 3, 4><<<grid, 512, 0, s>>>(a);
            return;
        }
    if (p.tile == kTile256) {
        gemm_kernel<T, PA, QA, BY_ROWS, 256, 256, 2, 4, 2><<<grid + (unsigned)a.slots, 512, 0, s>>>(a);
        if (a.slots) join_last_kernel<T, BY_ROWS, 256, 256><<<dim3((unsigned)a.slots / 2, 8), 256, 0, s>>>(a);
    }
    else if (p.tile == kTile128 && p.deep) gemm_kernel<T, PA, QA, BY_ROWS, 128, 128, 2, 2, 4><<<grid, 256, 0, s>>>(a);
    else if (p.tile == kTile128) gemm_kernel<T, PA, QA, BY_ROWS, 128, 128, 2, 2, 2><<<grid, 256, 0, s>>>(a);
    else if (p.deep) gemm_kernel<T, PA, QA, BY_ROWS, 64, 64, 2, 2, 4><<<grid, 256, 0, s>>>(a);
    else gemm_kernel<T, PA, QA, BY_ROWS, 64, 64, 2, 2, 2><<<grid, 256, 0, s>>>(a);
}

template <typename T, int FI> static void launch_stream(const GemmArgs& a, const GemmPlan& p, hipStream_t s) {
    const dim3 grid((unsigned)a.tiles_j, (unsigned)a.tiles_i, (unsigned)a.splits);
    const int threads = 64 * kStreamWaves;
    if (p.direct && p.narrow) stream_kernel<T, FI, 1, true><<<grid, threads, 0, s>>>(a);
    else if (p.direct) stream_kernel<T, FI, 2, true><<<grid, threads, 0, s>>>(a);
    else if (p.narrow) stream_kernel<T, FI, 1, false><<<grid, threads, 0, s>>>(a);
    else stream_kernel<T, FI, 2, false><<<grid, threads, 0, s>>>(a);
}

template <typename T> static rr_status_t launch_gemm(const GemmArgs& a, const GemmPlan& p, hipStream_t s) {
    if (p.tile == kDot) {
        // two rows of the weights a wave where that leaves no compute unit empty
        if (a.rows == 1 && a.j >= 2048) launch_dot<T, 1, 2>(a, s);
        else if (a.rows == 1) launch_dot<T, 1, 1>(a, s);
        else if (a.rows == 2) launch_dot<T, 2, 1>(a, s);
        else if (a.rows == 3) launch_dot<T, 3, 1>(a, s);
        else launch_dot<T, 4, 1>(a, s);
    } else if (p.tile >= kStream16) {
        if (p.tile == kStream16) launch_stream<T, 1>(a, p, s);
        else if (p.tile == kStream32) launch_stream<T, 2>(a, p, s);
        else launch_stream<T, 4>(a, p, s);
    } else if (p.form == kForward) {
        launch_form<T, false, false, true>(a, p, s);
    } else if (p.form == kByX) {
        launch_form<T, false, true, true>(a, p, s);
    } else {
        launch_form<T, true, true, false>(a, p, s);
    }
    const rr_status_t st = launched();
    if (st != RR_OK || a.splits == 1) return st;
    const bool by_rows = p.form != kByW;
    const uint64_t rows = by_rows ? (uint64_t)a.rows : (uint64_t)a.groups * a.i;
    const uint64_t blocks = ceil_div(rows * ceil_div(a.j, 4), 256);
    join_kernel<T><<<(unsigned)blocks, 256, 0, s>>>(a, by_rows);
    return launched();
}

}  // namespace blk
