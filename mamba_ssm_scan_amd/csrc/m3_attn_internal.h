// m3_attn_internal.h -- what the attention layer's entry points (m3_attn_host.cpp)
// hand to its kernel launchers. Not part of the public ABI.
#pragma once
#include "../../include/m3_attn.h"
#include "m3_internal.h"

namespace m3 {

struct RopeArgs {
    const void* x;
    void* y;
    int64_t x_tok, x_head, y_tok, y_head;  // strides, elements
    int64_t tokens;
    int32_t heads, D;
    m3_dtype io;
    const int32_t* positions;
    m3_rotary rot;
    int32_t backward;
    bool wide;  // pointers and strides take 16-byte accesses
    hipStream_t stream;
};
hipError_t launch_rope(const RopeArgs& a);

struct AppendArgs {
    m3_kv_cache c;
    m3_kv_batch b;
    m3_rows k, v, q, q_out;  // q.p NULL: no queries
    int32_t q_heads;
    m3_dtype io;
    m3_rotary rot;  // inv_freq NULL: no rotation
    bool wide;
    hipStream_t stream;
};
hipError_t launch_kv_append(const AppendArgs& a);

// Blocks of 16 tokens that an append launches workgroups for: every sequence's as many as
// max_q rows may touch, or, where that is more than twice as many, one sequence's after
// the other's (unit_of).
struct AppendPlan {
    int64_t each;    // blocks of a sequence; 0: one after the other
    int64_t blocks;
};
inline AppendPlan append_plan(const m3_kv_batch& b) {
    const int64_t each = (b.max_q + 14) / 16 + 1, packed = b.tokens / 16 + 2 * b.batch;
    if (b.cu_q && 2 * packed <= b.batch * each) return AppendPlan{0, packed};
    return AppendPlan{each, b.batch * each};
}

struct ReadArgs {
    m3_kv_cache c;
    int64_t batch, max_pages, max_count;
    const int32_t* first;
    const int32_t* count;
    const int32_t* pages;
    void* k_out;
    void* v_out;
    m3_dtype io;
    hipStream_t stream;
};
hipError_t launch_kv_read(const ReadArgs& a);

// How the rows and keys of an attend call are cut: a tile of `rows` (row, head of
// a group) pairs of one sequence and key head, its keys in tiles of 64. The kernel
// for many rows: `splits` workgroups along a row tile's keys, at most `split_tiles`
// tiles each (cut_of). The kernel for few: `items` > 0 gives every workgroup an even share of all
// tiles, 0 a row tile each.
struct PrefixPlan {       // of the prefix, where it is a part of its own
    bool tile;            // its own launch of the kernel for many rows; else items of the other's launch
    int32_t rows;
    int64_t row_tiles;    // of a group
    bool packed;
    int32_t items;        // (group, row tile) pairs
    int32_t splits;
    int64_t split_tiles, blocks;
    size_t slots, solo, solo_own;  // where parts lie, in rows: of even shares, of a run that one workgroup holds
};
struct AttendPlan {
    bool tile;            // the kernel for many rows a sequence
    int32_t rows;         // rows of a tile
    int64_t row_tiles;    // per sequence
    int32_t splits;
    int64_t split_tiles;
    int32_t items;        // (sequence, row tile) pairs
    bool packed;          // they follow one another (unit_of), as max_q is loose
    int64_t blocks;       // workgroups
    size_t o_off, ml_off, total;  // workspace: the shares (even ones), sums of parts, (unit, sum) pairs
    bool parts;           // the prefix and the sequences' own keys as parts
    PrefixPlan prefix;
};
constexpr int32_t kPrefixPiece = 4;     // least tiles of a piece of a prefix (many rows)
constexpr int32_t kPieceTiles = 8;      // least tiles of a piece, where a row tile's keys are cut (many rows)
constexpr int32_t kAttendItems = 2048;  // most items whose first tiles a workgroup holds
// Rows of a workgroup of the kernel for many rows, by headdim (<= 64, <= 128, <= 256);
// bf16 rows up to headdim 128 also half of them.
constexpr int32_t kTileRowsBf16[3] = {128, 256, 128}, kTileRowsF32[3] = {64, 128, 128};
struct AttendArgs {
    m3_kv_cache c;
    m3_kv_batch b;
    m3_rows q;
    void* out;
    float* lse;
    int32_t q_heads;
    m3_dtype io;
    float scale;
    m3_kv_view view;      // sinks 0 without a window
    AttendPlan plan;
    void* workspace;
    bool wide;
    hipStream_t stream;
};
// Whether a (bounded) view takes the kernels' VIEW form.
inline bool has_view(const m3_kv_view& v) { return v.sinks > 0 || v.groups > 0; }
AttendPlan attend_plan(const m3_kv_cache& c, const m3_kv_batch& b, const m3_kv_view& view, int32_t q_heads,
                       m3_dtype io);
hipError_t launch_kv_attend(const AttendArgs& a);

}  // namespace m3
