// How paged_query_attention's tensor-core kernel cuts its work: row tiles, work items, and parts of an item's keys with
// the space of their partial sums.  No CUDA header, so that a host compiler takes it too.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define KVP_HOST_DEVICE __host__ __device__
#else
#define KVP_HOST_DEVICE
#endif

namespace kvp {

// Pairs of 128-row tiles of a sequence's K/V head in the tensor-core kernel.
KVP_HOST_DEVICE inline int prompt_tiles(int queries, int group) {
    return static_cast<int>((static_cast<int64_t>(queries) * group + 255) / 256);
}
// Bound of a call's (pair, K/V head): each sequence has at most max_queries rows, all of them num_tokens, and one pair
// of each sequence is not full.
inline int64_t prompt_items(int batch, int heads, int group, int num_tokens, int max_queries) {
    const int64_t each = static_cast<int64_t>(batch) * prompt_tiles(max_queries, group);
    const int64_t all = static_cast<int64_t>(num_tokens) * group / 256 + batch;
    return (each < all ? each : all) * heads;
}

// Few items over long contexts leave most SMs idle: then an item's keys are cut into parts of at least 512, as many as the
// SMs take, and joined by a second launch.  (83 rows of 16 / 2 heads of 64 after 8k tokens, FP8, two sequences: 178 us
// whole, 32 in parts; 200 rows of 5 heads after 4.4k, float16: 69 and 21.  The join and the parts' own beginnings are about
// 10 us, so that shorter contexts stay whole.)
//
// Partial sums are laid out [part][row][query head].  Rows are the call's tokens, or, where q has more rows than the
// sequences may use (a padded buffer), max_queries places per sequence: min(num_tokens, batch max_queries) of them.  A call
// has at least that many times G H / 256 items and num_sms / items parts of each, so that parts times rows times query heads
// are at most 256 per SM.
struct QueryParts {
    int splits;                        // parts of each item's keys; 1: whole
    bool by_sequence;                  // rows are places of the sequences
    int64_t rows;                      // rows of a part
    int64_t space;                     // (part, row, query head) for this call and any of no more sequences, rows and positions
};
inline QueryParts query_parts(int num_sms, int batch, int heads, int group, int num_tokens, int max_queries, int max_context,
                              int window) {
    const int64_t items = prompt_items(batch, heads, group, num_tokens, max_queries);
    const int64_t reach = static_cast<int64_t>(window) + max_queries;
    const int64_t keys = window > 0 && reach < max_context ? reach : max_context;
    const int64_t most = keys / 512 < 32 ? keys / 512 : 32, parts = items > 0 ? num_sms / items : 0;
    const int64_t places = static_cast<int64_t>(batch) * max_queries;
    QueryParts p{1, places < num_tokens, places < num_tokens ? places : num_tokens, 0};
    if (most < 2) return p;
    if (parts >= 2) p.splits = static_cast<int>(parts < most ? parts : most);
    const int64_t all = static_cast<int64_t>(num_sms) * 256, need = most * p.rows * heads * group;
    p.space = need < all ? need : all;
    return p;
}
// The row of a part that holds row i of sequence s, whose first row of q is `first`.
KVP_HOST_DEVICE inline int64_t part_row(bool by_sequence, int max_queries, int s, int first, int i) {
    return (by_sequence ? static_cast<int64_t>(s) * max_queries : first) + i;
}

}  // namespace kvp
