// m3_attn_host.cpp -- the C entry points of the attention layer (m3_attn.h):
// argument checks, planning and dispatch. Host code only; every check runs
// before the first HIP call.
#include <cmath>

#include "m3_attn_internal.h"
#include "m3_host_checks.h"

namespace {

using m3::aligned;
using m3::check_dtype;
using m3::covered;
using m3::dense;
using m3::io_size;
using m3::overlaps;
using m3::Range;
using m3::rows_overlap;
using m3::set_error;

// the thread's error detail is cleared at entry, as by every call of the library
void clear_error() { set_error(M3_OK, "%s", ""); }

constexpr int64_t kMaxStride = int64_t(1) << 31;  // times 2^30 tokens and 4 bytes: still within 64 bits

m3_status check_rows(const char* name, const m3_rows* r, int64_t tokens, size_t es) {
    if (!r || (!r->p && tokens > 0)) return set_error(M3_EINVAL, "%s is NULL", name);
    if (!aligned(r->p, es)) return set_error(M3_EALIGN, "%s is not aligned to its entries", name);
    if (r->token_stride < 0 || r->head_stride < 0 || r->token_stride > kMaxStride || r->head_stride > kMaxStride)
        return set_error(M3_EINVAL, "%s: a stride is negative or above 2^31", name);
    return M3_OK;
}
// an output's rows must not share entries
m3_status check_out_rows(const char* name, const m3_rows& r, int64_t tokens, int64_t heads, int64_t D) {
    const bool head_inner = (heads == 1 || r.head_stride >= D) &&
                            (tokens <= 1 || r.token_stride >= (heads - 1) * r.head_stride + D);
    const bool token_inner = (tokens <= 1 || r.token_stride >= D) &&
                             (heads == 1 || r.head_stride >= (tokens - 1) * r.token_stride + D);
    if (!head_inner && !token_inner) return set_error(M3_EINVAL, "%s: rows overlap (strides)", name);
    return M3_OK;
}
bool wide_rows(const m3_rows& r, size_t es) {
    return aligned(r.p, 16) && r.token_stride * es % 16 == 0 && r.head_stride * es % 16 == 0;
}

m3_status check_rotary(const m3_rotary* r, int32_t D) {
    if (!r->inv_freq) return set_error(M3_EINVAL, "inv_freq is NULL");
    if (!aligned(r->inv_freq, 4)) return set_error(M3_EALIGN, "inv_freq is not 4-byte aligned");
    if (r->rot < 2 || r->rot % 2 != 0 || r->rot > D)
        return set_error(M3_EINVAL, "rot %d must be even, 2 .. headdim %d", r->rot, D);
    if (!std::isfinite(r->mscale)) return set_error(M3_EINVAL, "mscale is not finite");
    return M3_OK;
}

m3_status check_cache(const m3_kv_cache* c) {
    if (!c) return set_error(M3_EINVAL, "cache is NULL");
    if (c->format != M3_KV_INT8 && c->format != M3_KV_FP8)
        return set_error(M3_EDTYPE, "unknown cache format %d", c->format);
    if (c->num_pages < 0 || c->num_pages > (int64_t(1) << 31))
        return set_error(M3_EINVAL, "num_pages %lld out of range", (long long)c->num_pages);
    if (c->page_size < M3_KV_BLOCK || (c->page_size & (c->page_size - 1)) || c->page_size > (1 << 20))
        return set_error(M3_EINVAL, "page_size %d must be a power of two, 16 .. 2^20", c->page_size);
    if (c->heads < 1 || c->heads > 65536) return set_error(M3_EINVAL, "cache heads %d out of range", c->heads);
    if (c->headdim < 16 || c->headdim % 16 != 0 || c->headdim > 256)
        return set_error(M3_EUNSUPPORTED, "cache headdim %d must be a multiple of 16 up to 256", c->headdim);
    if (c->num_pages * (double)c->heads * c->page_size * c->headdim > 1e15 ||
        c->num_pages * (double)c->heads * (c->page_size / M3_KV_BLOCK) >= 2147483648.0)
        return set_error(M3_EINVAL, "the cache's sizes are out of range");  // (2^31 blocks: 512 GiB of K at headdim 16)
    const void* p[] = {c->k, c->v, c->k_scale, c->v_scale};
    const char* name[] = {"cache k", "cache v", "cache k_scale", "cache v_scale"};
    for (int j = 0; j < 4; ++j) {
        if (!p[j] && c->num_pages > 0) return set_error(M3_EINVAL, "%s is NULL", name[j]);
        if (!aligned(p[j], 16)) return set_error(M3_EALIGN, "%s is not 16-byte aligned", name[j]);
    }
    return M3_OK;
}
size_t cache_codes(const m3_kv_cache& c) {
    return size_t(c.num_pages) * size_t(c.heads) * size_t(c.page_size) * size_t(c.headdim);
}
size_t cache_scales(const m3_kv_cache& c) {
    return size_t(c.num_pages) * size_t(c.heads) * size_t(c.page_size / M3_KV_BLOCK) * 4;
}

m3_status check_pages(int64_t batch, const int32_t* pages, int64_t max_pages) {
    if (max_pages < 0 || max_pages > (int64_t(1) << 31))
        return set_error(M3_EINVAL, "max_pages %lld out of range", (long long)max_pages);
    if (!pages && batch > 0 && max_pages > 0) return set_error(M3_EINVAL, "pages is NULL");
    if (!aligned(pages, 4)) return set_error(M3_EALIGN, "pages is not 4-byte aligned");
    return M3_OK;
}
m3_status check_batch(const m3_kv_batch* b) {
    if (!b) return set_error(M3_EINVAL, "batch is NULL");
    if (b->batch < 0 || b->batch > (int64_t(1) << 30) || b->tokens < 0 || b->tokens > (int64_t(1) << 30))
        return set_error(M3_EINVAL, "batch %lld or tokens %lld out of range", (long long)b->batch,
                         (long long)b->tokens);
    if (b->max_q < 0 || b->max_kv < 0) return set_error(M3_EINVAL, "max_q or max_kv is negative");
    if (!b->cu_q && b->tokens != b->batch)
        return set_error(M3_ESHAPE, "cu_q is NULL, but tokens %lld is not batch %lld", (long long)b->tokens,
                         (long long)b->batch);
    if (!b->kv_len && b->batch > 0) return set_error(M3_EINVAL, "kv_len is NULL");
    if (!aligned(b->kv_len, 4) || !aligned(b->cu_q, 4))
        return set_error(M3_EALIGN, "kv_len or cu_q is not 4-byte aligned");
    return check_pages(b->batch, b->pages, b->max_pages);
}
// the bounds that size a launch, no larger than they can be
m3_kv_batch bounded(const m3_kv_batch& b, const m3_kv_cache& c) {
    m3_kv_batch r = b;
    r.max_q = b.cu_q ? std::min(b.max_q, b.tokens) : std::min<int64_t>(b.max_q, 1);
    const int64_t room = b.max_pages > (int64_t(1) << 31) / c.page_size ? int64_t(1) << 31 : b.max_pages * c.page_size;
    r.max_kv = std::min(std::min(b.max_kv, room), (int64_t(1) << 31) - 256);  // (tile ends stay within 32 bits)
    return r;
}

// the plain view of m3_kv_attend
m3_kv_view plain(int32_t causal, int64_t window) { return m3_kv_view{causal ? 1 : 0, window, 0, 0, 0, nullptr, nullptr, nullptr}; }
// A view whose window's end no position reaches, so that sums with it stay in range; as for
// sinks. (max_prefix is a stride too: its bound is the launch's, most_prefix.)
m3_kv_view bounded(const m3_kv_view& v) {
    m3_kv_view r = v;
    r.causal = v.causal ? 1 : 0;
    r.window = std::min(v.window, int64_t(1) << 31);
    r.sinks = v.window > 0 ? std::min(v.sinks, (int64_t(1) << 31) - 256) : 0;  // (as max_kv)
    if (v.max_prefix == 0) r.groups = 0;
    return r;
}

m3_status check_attend(const m3_kv_cache* c, const m3_kv_batch* b, const m3_kv_view* v, int32_t q_heads, m3_dtype io) {
    m3_status s;
    if ((s = check_cache(c)) != M3_OK || (s = check_batch(b)) != M3_OK || (s = check_dtype(io)) != M3_OK) return s;
    if (!v) return set_error(M3_EINVAL, "view is NULL");
    if (q_heads < 1 || q_heads > 65536 || q_heads % c->heads != 0)
        return set_error(M3_EINVAL, "q_heads %d must be a multiple of the cache's heads %d", q_heads, c->heads);
    if (v->window < 0) return set_error(M3_EINVAL, "window %lld < 0", (long long)v->window);
    if (v->window > 0 && !v->causal) return set_error(M3_EUNSUPPORTED, "a window needs causal attention");
    if (b->tokens * q_heads > INT32_MAX) return set_error(M3_EUNSUPPORTED, "tokens * q_heads is above 2^31");
    if (v->sinks < 0) return set_error(M3_EINVAL, "sinks %lld < 0", (long long)v->sinks);
    if (v->groups < 0 || v->groups > (int64_t(1) << 30) || v->max_prefix < 0 || v->max_prefix > (int64_t(1) << 31))
        return set_error(M3_EINVAL, "groups %lld or max_prefix %lld out of range", (long long)v->groups,
                         (long long)v->max_prefix);
    if (v->groups == 0) return M3_OK;
    if (!v->group_start && v->groups != 1) return set_error(M3_EINVAL, "group_start is NULL, but there are %lld groups", (long long)v->groups);
    if (!v->prefix_count) return set_error(M3_EINVAL, "prefix_count is NULL");
    if (!v->prefix_pages && v->max_prefix > 0) return set_error(M3_EINVAL, "prefix_pages is NULL");
    if (!aligned(v->group_start, 4) || !aligned(v->prefix_count, 4) || !aligned(v->prefix_pages, 4))
        return set_error(M3_EALIGN, "group_start, prefix_count or prefix_pages is not 4-byte aligned");
    return M3_OK;
}

}  // namespace

namespace m3 {

// Above 64 (row, head of a group) pairs a sequence (32 for fp32 rows and above headdim
// 128, where the other kernel holds fewer rows a wave), the kernel that shares each tile
// of keys among 64 to 256 rows (m3_kv_attend_tile.hip). 64 sequences of 4096 tokens, 8
// heads, that kernel and the one for few: headdim 128, 64 pairs 249 and 182 us, 96 252 and
// 241, 128 255 and 328; headdim 256, 32 pairs 332 and 348, 48 335 and 487; 16 of them in
// fp32, headdim 128, 32 pairs 77 and 65, 64 80 and 98.
//   A causal prompt whose workgroups would all run at once (two a CU up to headdim 64,
// one above) ends with its last row tiles, so it takes half the rows a workgroup: one
// prompt of 2048, 32 heads over 8, headdim 64 40 us and 49 with all rows, 128 68 and 83;
// two of them 66 and 60, 127 and 98. A piece (fewer rows than half the keys) has row
// tiles of nearly one length and keeps them whole (2048 of 32768: 562 us, 783 halved).
//   Keys are split, at least 8 tiles of 64 a workgroup, while there are fewer workgroups
// than CUs (one prompt of 2048, 16 heads over 2 of 128: 64 us, 76 up to two a CU). The
// splits come from the bound max_kv, their lengths from the keys that each row tile sees
// (cut_of): 512 rows that end at 8192 under a bound of 131072 59.7 us, under their own 59.3
// (294 with lengths from the bound). The halved rows need a tight bound: one prompt of 2048
// under 4096 49 us at headdim 64 and 83 at 128, four of them under 131072 118 us and 108.
// Else rows of a tile: 16 while a sequence has no more pairs, otherwise 32 (each key read once for
// twice the rows; at headdim above 128 the registers hold 16). A row tile and key head
// is a workgroup's where that fills the chip (two workgroups a CU, one above headdim
// 128: 128 sequences of 2112 tokens, 4 heads, 54 us and 66 by even shares with their
// join; of 127 .. 4095 tokens 71 and 77) or every sequence is short (16 tiles: 64
// sequences of 701 tokens 15 and 26 us); else all tiles are dealt out in even shares
// (64 sequences of 200 .. 8000 tokens: 68 us, 109 without), which a loose max_kv does
// not hurt.
//   max_q may be far above most sequences' rows. The kernel is chosen by four times the
// mean where that is less, and the pairs are numbered one sequence's after the other's
// (unit_of) instead of max_q's for each where that leaves out the half of them, or seven of
// eight in the kernel for many rows, which then loses its order (longest tiles of all
// sequences first, a column's in one XCD). Under a bound of all rows instead of the
// longest's: 128 single tokens over 2100 57 us and 49 (187 by the bound alone), 64 prompts
// of 300 113 and 100 (402), 4 prompts of 2048 108 and 107 (142 with the pairs packed).
static AttendPlan one_pass_plan(const m3_kv_cache& c, const m3_kv_batch& b, const m3_kv_view& view, int32_t q_heads,
                                m3_dtype io) {
    AttendPlan p{};
    const int32_t causal = view.causal;
    const int64_t window = view.window;
    const int64_t group = q_heads / c.heads;
    // what a sequence's rows are taken to be: the bound, or four times the mean below it
    const int64_t mean = b.cu_q && b.batch > 0 ? (b.tokens + b.batch - 1) / b.batch : 1;
    const int64_t most = std::min(b.max_q, 4 * mean), pairs = most * group;
    auto each = [&](int64_t rows) { return std::max<int64_t>(1, (b.max_q * group + rows - 1) / rows); };
    auto packed = [&](int64_t rows) { return b.tokens * group / rows + b.batch; };
    const int width = c.headdim <= 64 ? 0 : c.headdim <= 128 ? 1 : 2;
    p.tile = pairs > (io == M3_BF16 && width < 2 ? 64 : 32);
    p.rows = p.tile ? (io == M3_BF16 ? kTileRowsBf16 : kTileRowsF32)[width] : pairs <= 16 || width == 2 ? 16 : 32;
    if (p.tile && io == M3_BF16 && width < 2 && causal && 2 * most > b.max_kv &&
        c.heads * std::min(b.batch * each(p.rows), packed(p.rows)) <= (width == 0 ? 512 : 256))
        p.rows /= 2;
    p.row_tiles = each(p.rows);
    p.packed = b.cu_q && (p.tile ? 8 : 2) * packed(p.rows) <= b.batch * p.row_tiles;
    int64_t tiles = (b.max_kv + 63) / 64;
    if (window > 0) tiles = std::min(tiles, (window + (p.rows - 1) / group + 1 + 62) / 64 + 1 + (view.sinks + 63) / 64);
    tiles = std::max<int64_t>(1, tiles);
    const int64_t items = p.packed ? packed(p.rows) : b.batch * p.row_tiles, base = std::max<int64_t>(1, items * c.heads);
    const int64_t busy = std::max<int64_t>(1, std::min(items, b.cu_q ? packed(p.rows) : items) * c.heads);
    p.splits = 1;
    p.split_tiles = tiles;
    p.blocks = base;
    size_t parts = 0;  // rows of parts
    if (p.tile) {
        const int64_t want = std::max<int64_t>(1, std::min<int64_t>(256 / busy, tiles / m3::kPieceTiles));
        p.split_tiles = (tiles + want - 1) / want;
        p.splits = int32_t((tiles + p.split_tiles - 1) / p.split_tiles);
        p.blocks = base * p.splits;
        if (p.splits > 1) parts = size_t(p.splits) * size_t(b.tokens) * size_t(q_heads);
    } else if (const int64_t full = width == 2 ? 256 : 512;
               tiles > 16 && base < full && items <= kAttendItems && items * (has_view(view) ? 2 * tiles + 16 : tiles) <= INT32_MAX) {
        p.items = int32_t(items);
        // (a share of 4 tiles each; under sinks or prefixes items are multiples of 4)
        p.blocks = std::min<int64_t>(full, has_view(view) ? base * ((tiles + 3) / 4) : (base * tiles + 3) / 4);
        parts = size_t(2 * p.blocks) * size_t(p.rows);
        p.o_off = (size_t(items + 2) * 4 + 255) / 256 * 256;
    }
    p.ml_off = p.o_off + parts * size_t(c.headdim) * 4;
    p.total = parts ? p.ml_off + parts * 8 : 0;
    return p;
}

// The prefix and the sequences' own keys as parts; `p` is the plan of one pass, for few rows a
// sequence. 16 rows a tile in either case (32 leave registers for one wave a SIMD: 16 steps
// behind 8192 tokens 27 us and 33).
//   The groups' row tiles are items of the launch for few rows, whose waves each convert the
// keys anew, up to 8192 (row tile, key head, tile of 64 keys) triples, and while the sequences' own
// row tiles do not fill the chip by themselves; beyond, the kernel for many rows
// converts them once for 128 rows (256 where these alone fill a quarter of the chip, and parts
// are few) in a launch of its own. Steps with 16 heads over 4 of 128: behind 8192 tokens 16 / 32 / 64
// sequences 27 / 34 / 49 us and 32 / 38 / 46, behind 65536 4 / 8 / 16 of them 36 / 47 / 72 and 48 / 49 / 51;
// 128 of them behind 4096 54 and 40.
static AttendPlan parts_plan(AttendPlan p, const m3_kv_cache& c, const m3_kv_batch& b, const m3_kv_view& view,
                             int32_t q_heads, m3_dtype io) {
    PrefixPlan f{};
    const int64_t group = q_heads / c.heads, groups = view.groups, every = b.tokens * q_heads;
    const int width = c.headdim <= 64 ? 0 : c.headdim <= 128 ? 1 : 2;
    const int64_t tiles = (b.max_kv + 63) / 64, pre = (std::min(b.max_kv, view.max_prefix * c.page_size) + 63) / 64;
    // (group, row tile) pairs, each group's as many as all rows fill, or one group's after the other's
    auto busy = [&](int64_t rows) { return b.tokens * group / rows + groups; };
    auto count = [&](int64_t rows) {
        f.rows = int32_t(rows);
        f.row_tiles = std::max<int64_t>(1, (b.tokens * group + rows - 1) / rows);
        f.packed = view.group_start && 2 * busy(rows) <= groups * f.row_tiles;
        return f.packed ? busy(rows) : groups * f.row_tiles;
    };
    p.rows = 16;
    p.row_tiles = std::max<int64_t>(1, (b.max_q * group + 15) / 16);
    const int64_t packed = b.tokens * group / 16 + b.batch;
    p.packed = b.cu_q && 2 * packed <= b.batch * p.row_tiles;
    const int64_t own = p.packed ? packed : b.batch * p.row_tiles;
    const int64_t full = width == 2 ? 256 : 512, shared = count(16);  // workgroups at once
    f.tile = std::min(shared, busy(16)) * c.heads * pre > 8192 || own * c.heads >= full || shared + own > kAttendItems ||
             (shared + own) * (2 * tiles + 16) > INT32_MAX;  // (runs count a multiple of a share)
    size_t rows = 0;  // of parts
    if (!f.tile) {
        f.items = int32_t(shared);
        p.items = int32_t(shared + own);
        const int64_t four = c.heads * (std::min(shared, busy(16)) * ((pre + 3) / 4) + own * ((tiles + 3) / 4));
        p.blocks = std::max<int64_t>(1, std::min(full, four));
    } else {
        const int64_t most = (io == M3_BF16 ? kTileRowsBf16 : kTileRowsF32)[width];
        const bool half = io == M3_BF16 && width < 2 && std::min(count(most), busy(most)) * c.heads <= 64;
        const int64_t items = count(half ? most / 2 : most);
        const int64_t work = std::max<int64_t>(1, std::min(items, busy(f.rows)) * c.heads);
        const int64_t want = std::max<int64_t>(1, std::min<int64_t>(256 / work, pre / kPrefixPiece));
        f.split_tiles = std::max<int64_t>(1, (pre + want - 1) / want);
        f.splits = int32_t(std::max<int64_t>(1, (pre + f.split_tiles - 1) / f.split_tiles));
        f.blocks = items * c.heads * f.splits;
        rows = size_t(f.splits) * size_t(every);
        p.items = tiles > 16 && own * c.heads < full && own <= kAttendItems && own * (2 * tiles + 16) <= INT32_MAX ? int32_t(own) : 0;
        p.blocks = p.items ? std::min<int64_t>(full, own * c.heads * ((tiles + 3) / 4)) : std::max<int64_t>(1, own * c.heads);
    }
    f.slots = rows;
    if (p.items) rows += size_t(2 * p.blocks) * size_t(p.rows);
    f.solo = rows;
    if (!f.tile) rows += size_t(every);
    f.solo_own = rows;
    if (p.items) rows += size_t(every);
    p.parts = true;
    p.prefix = f;
    p.o_off = p.items ? (size_t(p.items + 2) * 4 + 255) / 256 * 256 : 0;
    p.ml_off = p.o_off + rows * size_t(c.headdim) * 4;
    p.total = p.ml_off + rows * 8;
    return p;
}

// Parts where they save enough, by what the prefix takes either way (us; from measurements). A wave's pass of up to 16 rows
// over a tile of 64 keys at headdim 128 takes 1 / 358 of the chip (32 rows: 1.4 times that), a pass of 128 rows in the
// kernel for many rows 1 / 136 (256 rows: 1.6 times); passes of fp32 rows half as much again (that and the factors
// of other headdims are set by the size of the products, not fitted). Parts of
// their own cost 3 more where the one pass deals out shares and joins anyway, else 10, the launch for many rows 10 to
// 12 on top. 16 heads over 4 of 128, parts and one pass, behind 512 tokens 16 / 64 sequences 17 / 24 us and 15 / 17;
// behind 2048 8 / 16 / 64 / 128 of them 17 / 18 / 29 / 35 and 16 / 23 / 37 / 44; behind 8192 2 / 4 / 16 / 128 of them 18
// / 18 / 24 / 47 and 17 / 23 / 37 / 129.
AttendPlan attend_plan(const m3_kv_cache& c, const m3_kv_batch& b, const m3_kv_view& view, int32_t q_heads,
                       m3_dtype io) {
    const AttendPlan one = one_pass_plan(c, b, view, q_heads, io);
    if (view.groups == 0 || view.window > 0 || one.tile || b.batch <= view.groups) return one;
    const AttendPlan two = parts_plan(one, c, b, view, q_heads, io);
    const int64_t group = q_heads / c.heads, pre = (std::min(b.max_kv, view.max_prefix * c.page_size) + 63) / 64;
    const double scale = double(c.heads * pre) * (c.headdim <= 64 ? 0.5 : c.headdim <= 128 ? 1. : 2.) * (io == M3_F32 ? 1.5 : 1.);
    auto tiles_of = [&](const int64_t all, int64_t each, int64_t n) { return double(std::min(n * each, b.tokens * group / all + n)); };
    const double apart = tiles_of(one.rows, one.row_tiles, b.batch) * (one.rows == 32 ? 1.4 : 1.) * scale / 358;
    const PrefixPlan& f = two.prefix;
    const double rows = tiles_of(f.rows, f.row_tiles, view.groups) * scale;
    const double together = f.tile ? rows * f.rows / 128. * (f.rows > 128 ? 0.8 : 1.) / 136 + (one.items ? 15 : 20)
                                   : rows / 358 + (one.items ? 3 : 10);
    return together < apart ? two : one;
}

}  // namespace m3

extern "C" {

m3_status m3_rope(const m3_rows* x, const m3_rows* y, int64_t tokens, int32_t heads, int32_t headdim,
                  m3_dtype io_dtype, const int32_t* positions, const m3_rotary* rotary, int32_t backward,
                  void* stream) {
    clear_error();
    m3_status s;
    if ((s = check_dtype(io_dtype)) != M3_OK) return s;
    if (tokens < 0 || tokens > (int64_t(1) << 30))
        return set_error(M3_EINVAL, "tokens %lld out of range", (long long)tokens);
    if (heads < 1 || heads > 65536) return set_error(M3_EINVAL, "heads %d out of range", heads);
    if (headdim < 2 || headdim > 65536) return set_error(M3_EINVAL, "headdim %d out of range", headdim);
    const size_t es = io_size(io_dtype);
    if ((s = check_rows("x", x, tokens, es)) != M3_OK) return s;
    if ((s = check_rows("y", y, tokens, es)) != M3_OK) return s;
    if ((s = check_out_rows("y", *y, tokens, heads, headdim)) != M3_OK) return s;
    if (!rotary) return set_error(M3_EINVAL, "rotary is NULL");
    if ((s = check_rotary(rotary, headdim)) != M3_OK) return s;
    if (!positions && tokens > 0) return set_error(M3_EINVAL, "positions is NULL");
    if (!aligned(positions, 4)) return set_error(M3_EALIGN, "positions is not 4-byte aligned");
    const Range ry = covered("y", *y, tokens, heads, headdim, es);
    const bool in_place = x->p == y->p && x->token_stride == y->token_stride && x->head_stride == y->head_stride;
    if (!in_place && rows_overlap(*y, heads, *x, heads, tokens, headdim, es))
        return set_error(M3_EINVAL, "y overlaps x");
    const Range in[] = {dense("positions", positions, size_t(tokens) * 4),
                        dense("inv_freq", rotary->inv_freq, size_t(rotary->rot) * 2)};
    for (const Range& r : in)
        if (overlaps(ry, r)) return set_error(M3_EINVAL, "y overlaps %s", r.name);
    if (tokens == 0) return M3_OK;
    m3::RopeArgs a{x->p, y->p, x->token_stride, x->head_stride, y->token_stride, y->head_stride, tokens, heads,
                   headdim, io_dtype, positions, *rotary, backward, wide_rows(*x, es) && wide_rows(*y, es),
                   reinterpret_cast<hipStream_t>(stream)};
    const hipError_t e = m3::launch_rope(a);
    if (e != hipSuccess) return set_error(M3_EHIP, "rope launch failed: %s", hipGetErrorString(e));
    return M3_OK;
}

m3_status m3_kv_append(const m3_kv_cache* cache, const m3_kv_batch* batch, const m3_rows* k, const m3_rows* v,
                       const m3_rows* q, const m3_rows* q_out, int32_t q_heads, m3_dtype io_dtype,
                       const m3_rotary* rotary, void* stream) {
    clear_error();
    m3_status s;
    if ((s = check_cache(cache)) != M3_OK || (s = check_batch(batch)) != M3_OK || (s = check_dtype(io_dtype)) != M3_OK)
        return s;
    const size_t es = io_size(io_dtype);
    const int64_t T = batch->tokens, D = cache->headdim;
    if ((s = check_rows("k", k, T, es)) != M3_OK) return s;
    if ((s = check_rows("v", v, T, es)) != M3_OK) return s;
    if ((q == nullptr) != (q_out == nullptr)) return set_error(M3_EINVAL, "q and q_out must be given together");
    if (rotary && (s = check_rotary(rotary, cache->headdim)) != M3_OK) return s;
    const Range pool[] = {dense("cache k", cache->k, cache_codes(*cache)), dense("cache v", cache->v, cache_codes(*cache)),
                          dense("cache k_scale", cache->k_scale, cache_scales(*cache)),
                          dense("cache v_scale", cache->v_scale, cache_scales(*cache))};
    Range in[8] = {covered("k", *k, T, cache->heads, D, es), covered("v", *v, T, cache->heads, D, es),
                   dense("kv_len", batch->kv_len, size_t(batch->batch) * 4),
                   dense("cu_q", batch->cu_q, size_t(batch->batch + 1) * 4),
                   dense("pages", batch->pages, size_t(batch->batch) * size_t(batch->max_pages) * 4),
                   dense("inv_freq", rotary ? rotary->inv_freq : nullptr, rotary ? size_t(rotary->rot) * 2 : 0),
                   {"q", 0, 0}, {"q_out", 0, 0}};
    bool wide = wide_rows(*k, es) && wide_rows(*v, es);
    if (q) {
        if (q_heads < 1 || q_heads > 65536) return set_error(M3_EINVAL, "q_heads %d out of range", q_heads);
        if ((s = check_rows("q", q, T, es)) != M3_OK) return s;
        if ((s = check_rows("q_out", q_out, T, es)) != M3_OK) return s;
        if ((s = check_out_rows("q_out", *q_out, T, q_heads, D)) != M3_OK) return s;
        in[6] = covered("q", *q, T, q_heads, D, es);
        in[7] = covered("q_out", *q_out, T, q_heads, D, es);
        wide = wide && wide_rows(*q, es) && wide_rows(*q_out, es);
        const bool in_place = q->p == q_out->p && q->token_stride == q_out->token_stride &&
                              q->head_stride == q_out->head_stride;
        if (rows_overlap(*q_out, q_heads, *k, cache->heads, T, D, es)) return set_error(M3_EINVAL, "q_out overlaps k");
        if (rows_overlap(*q_out, q_heads, *v, cache->heads, T, D, es)) return set_error(M3_EINVAL, "q_out overlaps v");
        if (!in_place && rows_overlap(*q_out, q_heads, *q, q_heads, T, D, es))
            return set_error(M3_EINVAL, "q_out overlaps q");
        for (int j = 2; j < 6; ++j)
            if (overlaps(in[7], in[j])) return set_error(M3_EINVAL, "q_out overlaps %s", in[j].name);
    }
    for (int p = 0; p < 4; ++p) {
        for (const Range& r : in)
            if (overlaps(pool[p], r)) return set_error(M3_EINVAL, "%s overlaps %s", pool[p].name, r.name);
        for (int o = p + 1; o < 4; ++o)
            if (overlaps(pool[p], pool[o])) return set_error(M3_EINVAL, "%s overlaps %s", pool[p].name, pool[o].name);
    }
    m3::AppendArgs a{*cache, bounded(*batch, *cache), *k, *v, q ? *q : m3_rows{nullptr, 0, 0},
                     q ? *q_out : m3_rows{nullptr, 0, 0}, q_heads, io_dtype,
                     rotary ? *rotary : m3_rotary{nullptr, 0, 0, 1.f}, wide, reinterpret_cast<hipStream_t>(stream)};
    if (T == 0 || batch->batch == 0 || a.b.max_q == 0) return M3_OK;
    if (m3::append_plan(a.b).blocks > INT32_MAX)
        return set_error(M3_EUNSUPPORTED, "batch times max_q / 16 is above 2^31");
    const hipError_t e = m3::launch_kv_append(a);
    if (e != hipSuccess) return set_error(M3_EHIP, "append launch failed: %s", hipGetErrorString(e));
    return M3_OK;
}

m3_status m3_kv_read(const m3_kv_cache* cache, int64_t batch, const int32_t* first, const int32_t* count,
                     const int32_t* pages, int64_t max_pages, int64_t max_count, void* k_out, void* v_out,
                     m3_dtype io_dtype, void* stream) {
    clear_error();
    m3_status s;
    if ((s = check_cache(cache)) != M3_OK || (s = check_dtype(io_dtype)) != M3_OK) return s;
    if (batch < 0 || batch > (int64_t(1) << 30) || max_count < 0 || max_count > INT32_MAX)
        return set_error(M3_EINVAL, "batch %lld or max_count %lld out of range", (long long)batch, (long long)max_count);
    if ((s = check_pages(batch, pages, max_pages)) != M3_OK) return s;
    if (batch == 0 || max_count == 0) return M3_OK;
    if (!first || !count) return set_error(M3_EINVAL, "first or count is NULL");
    if (!aligned(first, 4) || !aligned(count, 4)) return set_error(M3_EALIGN, "first or count is not 4-byte aligned");
    if (!k_out || !v_out) return set_error(M3_EINVAL, "k_out or v_out is NULL");
    if (!aligned(k_out, 16) || !aligned(v_out, 16)) return set_error(M3_EALIGN, "k_out or v_out is not 16-byte aligned");
    const int64_t blocks = (max_count + 14) / 16 + 1;
    if (batch > INT32_MAX / blocks) return set_error(M3_EUNSUPPORTED, "batch times max_count / 16 is above 2^31");
    const size_t bytes = size_t(batch) * size_t(max_count) * size_t(cache->heads) * size_t(cache->headdim) * io_size(io_dtype);
    const Range out[] = {dense("k_out", k_out, bytes), dense("v_out", v_out, bytes)};
    const Range in[] = {dense("cache k", cache->k, cache_codes(*cache)), dense("cache v", cache->v, cache_codes(*cache)),
                        dense("cache k_scale", cache->k_scale, cache_scales(*cache)),
                        dense("cache v_scale", cache->v_scale, cache_scales(*cache)),
                        dense("first", first, size_t(batch) * 4), dense("count", count, size_t(batch) * 4),
                        dense("pages", pages, size_t(batch) * size_t(max_pages) * 4)};
    for (const Range& o : out)
        for (const Range& r : in)
            if (overlaps(o, r)) return set_error(M3_EINVAL, "%s overlaps %s", o.name, r.name);
    if (overlaps(out[0], out[1])) return set_error(M3_EINVAL, "k_out overlaps v_out");
    m3::ReadArgs a{*cache, batch, max_pages, max_count, first, count, pages, k_out, v_out, io_dtype,
                   reinterpret_cast<hipStream_t>(stream)};
    const hipError_t e = m3::launch_kv_read(a);
    if (e != hipSuccess) return set_error(M3_EHIP, "read launch failed: %s", hipGetErrorString(e));
    return M3_OK;
}

size_t m3_kv_attend_workspace_size(const m3_kv_cache* cache, const m3_kv_batch* batch, int32_t q_heads,
                                   m3_dtype io_dtype, int32_t causal, int64_t window) {
    const m3_kv_view view = plain(causal, window);
    return m3_kv_attend_view_workspace_size(cache, batch, &view, q_heads, io_dtype);
}

size_t m3_kv_attend_view_workspace_size(const m3_kv_cache* cache, const m3_kv_batch* batch, const m3_kv_view* view,
                                        int32_t q_heads, m3_dtype io_dtype) {
    clear_error();
    if (check_attend(cache, batch, view, q_heads, io_dtype) != M3_OK) return 0;
    return m3::attend_plan(*cache, bounded(*batch, *cache), bounded(*view), q_heads, io_dtype).total;
}

m3_status m3_kv_attend(const m3_kv_cache* cache, const m3_kv_batch* batch, const m3_rows* q, void* out, float* lse,
                       int32_t q_heads, m3_dtype io_dtype, float scale, int32_t causal, int64_t window,
                       void* workspace, size_t workspace_bytes, void* stream) {
    const m3_kv_view view = plain(causal, window);
    return m3_kv_attend_view(cache, batch, &view, q, out, lse, q_heads, io_dtype, scale, workspace, workspace_bytes, stream);
}

m3_status m3_kv_attend_view(const m3_kv_cache* cache, const m3_kv_batch* batch, const m3_kv_view* view,
                            const m3_rows* q, void* out, float* lse, int32_t q_heads, m3_dtype io_dtype, float scale,
                            void* workspace, size_t workspace_bytes, void* stream) {
    clear_error();
    m3_status s = check_attend(cache, batch, view, q_heads, io_dtype);
    if (s != M3_OK) return s;
    const size_t es = io_size(io_dtype);
    const int64_t T = batch->tokens, D = cache->headdim;
    if ((s = check_rows("q", q, T, es)) != M3_OK) return s;
    if (!out && T > 0) return set_error(M3_EINVAL, "out is NULL");
    if (!aligned(out, 16)) return set_error(M3_EALIGN, "out is not 16-byte aligned");
    if (!aligned(lse, 4)) return set_error(M3_EALIGN, "lse is not 4-byte aligned");
    if (!std::isfinite(scale)) return set_error(M3_EINVAL, "scale is not finite");
    m3::AttendArgs a{*cache, bounded(*batch, *cache), *q, out, lse, q_heads, io_dtype, scale, bounded(*view),
                     {}, workspace, wide_rows(*q, es), reinterpret_cast<hipStream_t>(stream)};
    a.plan = m3::attend_plan(*cache, a.b, a.view, q_heads, io_dtype);
    const size_t rows = size_t(T) * size_t(q_heads);
    const Range outs[] = {dense("out", out, rows * size_t(D) * es), dense("lse", lse, rows * 4),
                          dense("workspace", workspace, workspace_bytes)};
    const Range in[] = {covered("q", *q, T, q_heads, D, es), dense("kv_len", batch->kv_len, size_t(batch->batch) * 4),
                        dense("cu_q", batch->cu_q, size_t(batch->batch + 1) * 4),
                        dense("pages", batch->pages, size_t(batch->batch) * size_t(batch->max_pages) * 4),
                        dense("cache k", cache->k, cache_codes(*cache)), dense("cache v", cache->v, cache_codes(*cache)),
                        dense("cache k_scale", cache->k_scale, cache_scales(*cache)),
                        dense("cache v_scale", cache->v_scale, cache_scales(*cache)),
                        dense("group_start", view->group_start, size_t(view->groups + 1) * 4),
                        dense("prefix_count", view->prefix_count, size_t(view->groups) * 4),
                        dense("prefix_pages", view->prefix_pages, size_t(view->groups) * size_t(view->max_prefix) * 4)};
    for (int o = 0; o < 3; ++o) {
        for (const Range& r : in)
            if (overlaps(outs[o], r)) return set_error(M3_EINVAL, "%s overlaps %s", outs[o].name, r.name);
        for (int p = o + 1; p < 3; ++p)
            if (overlaps(outs[o], outs[p])) return set_error(M3_EINVAL, "%s overlaps %s", outs[o].name, outs[p].name);
    }
    if (T == 0 || batch->batch == 0 || a.b.max_q == 0) return M3_OK;
    if (a.plan.total > 0) {
        if (!workspace || workspace_bytes < a.plan.total)
            return set_error(M3_EWORKSPACE, "workspace of %zu bytes, %zu needed", workspace_bytes, a.plan.total);
        if (!aligned(workspace, 16)) return set_error(M3_EALIGN, "workspace is not 16-byte aligned");
    }
    if (a.plan.blocks > INT32_MAX - 7 || a.plan.prefix.blocks > INT32_MAX - 7) return set_error(M3_EUNSUPPORTED, "too many workgroups");
    const hipError_t e = m3::launch_kv_attend(a);
    if (e != hipSuccess) return set_error(M3_EHIP, "attend launch failed: %s", hipGetErrorString(e));
    return M3_OK;
}

}  // extern "C"
