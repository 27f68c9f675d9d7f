// m3_kv_attend_tile.hip -- attention over the paged 8-bit cache for many rows a
// sequence (prompts, pieces of prompts).
//
// The products of m3_kv_attend.hip, S^T = K Q^T and O^T = V^T P^T with the scores
// kept in registers, but bound by the matrix rate instead of by memory: a
// workgroup of NW waves takes 16 QT NW rows, and its waves share each tile of 64
// keys, which the workgroup turns from codes into bf16 (K; V of fp32 rows) or fp16 (V) once
// and holds in LDS.
// The LDS image is the operands themselves: a 1 KiB piece is the 64 lanes' 16
// bytes of one MFMA operand, so every read is one linear ds_read_b128 that QT
// products use. Two images alternate: the next tile's codes are on their way to
// registers while this tile is computed, and are written to the other image
// before the one barrier of a tile.
//
// A tile's probabilities are formed with the reference as it stands, beside the next
// tile's scores; only where one leaves fp16's range is the maximum taken, the sums
// scaled and the tile's probabilities formed again. No maximum is needed otherwise: 16
// probabilities, none negative, whose fp32 sum stays below 2^15 are below it themselves.
//
// 2048 rows after 30720 tokens (16 heads over 4 of 128, e4m3): 562 us with the join, 947
// TFLOP/s; 4 prompts of 2048 (32 heads over 8 of 64, int8): 106 us, 650 TFLOP/s of the pairs
// that the mask leaves. There the vector unit is the busiest (69%, the products 25%): 10.2
// vector instructions are executed for each such score (7.9 in the other case), where the
// softmax itself takes four: exponential, its argument, sum, rounding. The rest are the
// conversions of codes, masks, and pairs that the mask drops; at 64 there are half the
// products to hide them behind. fp32 rows take three products where bf16 rows take one: one
// prompt of 2048, 16 heads over 4 of 64, 128, 256: 57, 103, 164 us (bf16, 256: 103).
#include "m3_attend_tile.h"

namespace m3 {

hipError_t launch_attend_tile(const AttendDev& of, m3_dtype io, hipStream_t s) {
    AttendDev d = of;
    // Columns side by side: as many as leave their keys in an XCD's 4 MiB of L2. Whole
    // columns where all XCDs get as many of them, or nearly so.
    const int64_t columns = d.blocks / d.row_tiles, each = (columns + 7) / 8;
    d.columns = 0;
    d.grid = d.blocks;
    if (!d.packed && (columns % 8 == 0 || columns >= 64) && 8 * each * d.row_tiles <= INT32_MAX) {
        const int64_t fit = (int64_t(4) << 20) / (d.split_tiles * kTile * 2 * d.D);
        d.columns = int(std::min(each, std::max<int64_t>(1, fit)));
        d.grid = 8 * each * d.row_tiles;
    }
    return of.form == kPlain ? launch_tile_form<kPlain>(d, io, s) : launch_attend_tile_view(d, io, s);
}

}  // namespace m3
