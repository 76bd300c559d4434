// blk_product.hpp -- the host side that the entry points of a block's products share: the
// operands, the choice of kernel and the scratch memory of one product (blk_linear.hip), and
// the conversions of 8-bit operands (blk_quant.hip).
#pragma once

#include "blk_gemm.hpp"

namespace blk {

constexpr uint64_t kMaxSize = 0x7FFFFFFFull - 1024;
constexpr uint64_t kMaxLd = 1ull << 22;
constexpr unsigned kSlots = 256;             // 256 x 256 tiles that a device takes at once: one a compute unit
constexpr uint64_t kBlock = 128;             // elements of a row, or rows and elements, with one scale

inline bool rows_ok(const rr_rows_t& r, uint64_t rows, uint64_t width, uint64_t bytes) {
    return rows == 0 || (r.data && aligned_to(r.data, bytes) && r.ld >= width);
}
inline bool rows_ok_if(const rr_rows_t& r, uint64_t rows, uint64_t width, uint64_t bytes) {
    return !r.data || rows_ok(r, rows, width, bytes);
}

// An operand of 16-byte pieces: its rows start at them and, where the pieces lie along the
// contraction, end at them too (past a row's end there may be anything).
inline bool good_rows(const rr_rows_t& r, uint64_t group, uint64_t width, uint64_t piece = 8) {
    return aligned_to(r.data, 16) && r.ld % piece == 0 && group % piece == 0 && width % piece == 0;
}

// Rows that the tiles of blk_tile.hpp take as they are: whole words of 4 bytes, as the loads into
// LDS need, and no less than a piece.
inline bool word_rows(const rr_rows_t& r, uint64_t group, uint64_t width, uint64_t bytes) {
    return aligned_to(r.data, 4) && r.ld * bytes % 4 == 0 && group * bytes % 4 == 0 && width * bytes % 4 == 0 &&
           width * bytes >= 16;
}

struct Operand {
    rr_rows_t rows;
    uint64_t count, width, groups, group;  // rows of a group, row length, groups and their distance
    const float* scales = nullptr;         // of 8-bit values, to be copied in 16 bits
    uint64_t high = 1, part = 0;           // rows with one scale; those after which its blocks begin anew
    bool good() const { return !scales && good_rows(rows, groups > 1 ? group : 0, width); }
    uint64_t copy_bytes() const {
        return ceil_div(groups * count * ceil_div(width, 8) * 16, 256) * 256;
    }
};

// One product: `k` has the sizes and the epilogue.
struct Product {
    int form;
    Operand p, q;
    GemmArgs k;
};

rr_status_t check_linear_sizes(const rr_linear_t* a, uint64_t x_bytes, uint64_t w_bytes);
GemmArgs groups_of(const rr_linear_t* a);
uint64_t row_tiles(const rr_linear_t* a, uint64_t height);
GemmPlan choose(const rr_linear_t* a, int form, int* splits, int* slots);
uint64_t product_bytes(const rr_linear_t* a, int form, const Operand& p, const Operand& q);
rr_status_t run_product(const rr_linear_t* a, Product r, void* workspace, hipStream_t s);
Operand rows_of(const rr_linear_t* a, const rr_rows_t& r, uint64_t width);
Operand weights_of(const rr_linear_t* a);

// Column sums of the rows of each group, in the gradients of the activation and of the gate:
// threads of a workgroup across the columns (8 each); parts of a group's rows, enough workgroups to
// fill the device and four rows a thread; and the sum of the parts, [groups][splits][n].
uint64_t sum_threads(const rr_linear_t* a);
uint64_t sum_splits(const rr_linear_t* a);
rr_status_t launch_sums(const float* part, int splits, uint64_t n, int groups, float* db, hipStream_t s);

// Bytes that the weights reach over.
inline uint64_t weights_extent(const rr_linear_t* a, uint64_t bytes) {
    return extent(a->groups, a->w_stride, extent(a->n, a->w_ld, a->k, 1), bytes);
}

// ------------------------------------------------------------- 8-bit operands --

// Rows of `groups` matrices in 8 bits and in dt, and their scales: one for `high` rows (1 or
// 128) x 128 columns, the blocks of rows beginning anew after every `part` of a group's rows.
struct BlockArgs {
    void* wide;              // dt
    uint8_t* narrow;
    float* scales;
    uint64_t wide_ld, wide_group, narrow_ld, narrow_group;
    uint64_t rows, groups;   // rows of a group
    uint64_t part;
    int32_t width, blocks;   // columns, and blocks of them
    int32_t filled;          // columns of the wide rows to write: zeros behind `width`
    int32_t high;
};
rr_status_t launch_back(const BlockArgs& a, int dt, hipStream_t s);   // narrow -> wide
// Byte rows of one or two operands to rows of `filled` bytes, whole 16-byte pieces, at `wide`, with
// zeros behind.
struct Pack8Args {
    BlockArgs part[2];
};
rr_status_t launch_pack8(const Pack8Args& a, int parts, hipStream_t s);

}  // namespace blk
