// Linear layers with one weight per group of a packed batch, on gfx950:
//     y_r = W_n x_r + b_n   for the rows r of group n,
// and the backward pass grad_x_r = W_n^T g_r, grad_W_n = sum_r g_r x_r^T,
// grad_b_n = sum_r g_r.
//
// The group sizes are device data, so a launch covers the largest number of
// row tiles that any split of R rows into N groups can have, and every
// workgroup finds its own group from the offsets (64 groups at a time, one
// lane each); workgroups beyond the last tile leave.
#include "dmr_internal.h"
#include "grouped_linear.h"

namespace dmr {

// The tile side, the rows of a piece of the weight gradient, and the slots
// that the pieces of groups longer than one piece can take: a group of
// r > rows has at most 2 floor(r / rows) of them.
GroupedPieces grouped_pieces(int64_t R, int64_t N, int32_t cin, int32_t cout, bool half) {
    // 256 only where the groups' tiles are many before any piece is cut (2
    // groups of 256 to 512, 16384 rows in bfloat16: 59 us with, 50 without)
    const int64_t weights256 = N * ((cin + 255) / 256) * ((cout + 255) / 256);
    const bool large = half && cin > 128 && cout > 128 && R >= 512 * N && weights256 >= 64;
    const int64_t side = cin <= 64 && cout <= 64 ? 64 : large ? 256 : 128;
    const int64_t tiles = ((cin + side - 1) / side) * ((cout + side - 1) / side);
    // a piece is at most one of the places' shares of the work: 256 compute
    // units with one workgroup of the largest tiles, two or four of the others
    const int64_t want = (side == 256 ? 256 : side == 128 ? 512 : 1024) / tiles;
    int64_t rows = want > 0 ? (R + want - 1) / want : R;
    rows = (rows + 127) / 128 * 128;
    rows = rows < 512 ? 512 : rows > 8192 ? 8192 : rows;
    if (R <= 1024) rows = 1024;   // short enough to need no second launch
    return {(int)rows, (int)side, R > rows ? 2 * (R / rows) : 0};
}

// The largest tiles have no form for arrays that are not aligned.
int grouped_weight_side(const GroupedPieces& p, bool vec) { return p.side == 256 && !vec ? 128 : p.side; }

// The tile by the widths and by how many there are: the larger, the fewer
// bytes for a product, but they have to fill 256 compute units. (bfloat16,
// forward: 2048 rows of 512 to 512, 19.3 us with 256 x 256 tiles, 11.0 with
// 128 x 128, 9.4 with 64 x 128; 8192 of 1024 to 1024, 128 tiles of 256 x 256,
// 35.3 and 31.5 with 128 x 128, but the backward's transposed weight 103 and
// 117. 2^20 rows of 64 to 64: 60 us with 64 x 256, 63 with 64 x 128. 217632 rows
// of 64 to 3 in float32: 17.7 us with 16 x 256, 14.3 with 16 x 128.)
RowsTile grouped_rows_tile(int64_t R, int64_t N, int32_t n_out, bool half, bool backward, bool vec) {
    const auto tiles = [&](int bn, int bm) { return (R / bm + 1) * ceil_div(n_out, bn); };
    if (R <= 16 * N) return {64, 16};
    if (n_out <= 16) return {16, 128};
    if (n_out <= 64 || tiles(128, 128) < 256) return half && tiles(64, 256) >= 256 ? RowsTile{64, 256} : RowsTile{64, 128};
    if (half && vec && n_out > 128 && R >= 512 * N && tiles(256, 256) >= (backward ? 112 : 224)) return {256, 256};
    return {128, 128};
}

// Both gradients in one launch where small tiles serve both: narrow layers,
// and calls of so few tiles that one gradient's leave the device unfilled.
// What one waits for, the other fills, and the upstream gradients are read
// while they are near. (One launch against two, us.
// Float32: 217632 rows of 64 to 64, 53 and 64, of 16 to 256, 100 and 172;
// 8192 of 256 to 256, 37 and 70; 2048 of 1024 to 1024, 1552 tiles, 115 and
// 94. 16 bits: 1003 rows of 37 to 19, 15.9 and 20.7; 2^20 of 64 to 64, 120
// and 129; 8192 of 256 to 256, 18.4 and 30.8; 16384 of 256 to 512, 2112
// tiles, 41 and 49; 64 groups of one row, 1024 to 1024, 16384 tiles, 187 and
// 118; 166428 rows of 240 to 64, 61 and 66, but 400000 of 512 to 64, 276 and
// 261.)
bool grouped_together(int64_t R, int64_t N, int32_t cin, int32_t cout, bool half) {
    if (R == 0) return false;
    const int64_t few = half ? 2304 : 1536;
    const bool narrow = cin <= 64 || (cin <= 256 && cout <= 64);
    const int64_t row_tiles = most_row_tiles(R, N, R <= 16 * N ? 16 : 128) * ceil_div(cin, 64);
    const int64_t items = (R / grouped_pieces(R, N, cin, cout, half).rows + N) * ceil_div(cin, 64) * ceil_div(cout, 64);
    return (row_tiles + items <= few || narrow) && row_tiles + items <= 1 << 23;
}

bool grouped_add_fits(int64_t N, int32_t cin, int32_t cout) {
    return add_blocks((int64_t)cin * cout + cout) * N <= kMaxWorkItems / 256;
}

bool grouped_sums_fit(int64_t R, int64_t N, int32_t cin, int32_t cout, bool half) {
    const GroupedPieces p = grouped_pieces(R, N, cin, cout, half);
    const int side = grouped_weight_side(p, false);   // of the tiles that are more
    const int64_t items = (R / p.rows + N) * ceil_div(cin, side) * ceil_div(cout, side), round = 8 * kPieceRun;
    if ((items + round - 1) / round * round > kMaxWorkItems / 256) return false;
    return p.slots == 0 || grouped_add_fits(N, cin, cout);
}

hipError_t launch_grouped_add_pieces(const GroupedLinearArgs& a, const GroupedPieces& p) {
    switch (a.dtype) {
        case DMR_FLOAT32: return add_pieces<float>(a, p);
        case DMR_FLOAT16: return add_pieces<_Float16>(a, p);
        case DMR_BFLOAT16: return add_pieces<__bf16>(a, p);
    }
    return hipErrorInvalidValue;
}
hipError_t launch_grouped_linear_forward(const GroupedLinearArgs& a) {
    switch (a.dtype) {
        case DMR_FLOAT32: return launch_forward<float>(a);
        case DMR_FLOAT16: return launch_forward<_Float16>(a);
        case DMR_BFLOAT16: return launch_forward<__bf16>(a);
    }
    return hipErrorInvalidValue;
}
hipError_t launch_grouped_linear_backward(const GroupedLinearArgs& a) {
    switch (a.dtype) {
        case DMR_FLOAT32: return launch_backward<float, float, float, 1>(a);
        case DMR_FLOAT16: return launch_backward<_Float16, _Float16, _Float16, 1>(a);
        case DMR_BFLOAT16: return launch_backward<__bf16, __bf16, __bf16, 1>(a);
    }
    return hipErrorInvalidValue;
}

}  // namespace dmr
