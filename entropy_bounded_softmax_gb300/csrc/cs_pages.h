// Whole-number arithmetic of the operators around a paged key-value cache that
// decides where they read and write, in range for every input.  Free of CUDA, so
// that it runs on the host too.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define CS_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define CS_HOST_DEVICE inline
#endif

namespace cs {

CS_HOST_DEVICE uint32_t pages_of(uint32_t tokens, uint32_t page) {
    return tokens / page + (tokens % page != 0);
}

// What a sequence asks of paged_extend: `fresh` tokens behind its `len`, `need`
// pages behind its `held`; fresh and need 0 where `bad`.
struct Claim {
    int32_t len, fresh, held, need;
    bool bad;
};

// held: the pages it has, where `given`, or those of its tokens.  A row of the
// table holds at most 2^30 tokens and max_new is at most 2^30, so that the tokens
// after the call, up to 2^31, and their pages are counted without a sign.
CS_HOST_DEVICE Claim claim_of(int32_t len, int32_t fresh, bool given, int32_t held,
                              int32_t max_new, int32_t max_pages, int32_t page_size) {
    Claim c;
    c.len = len;
    c.fresh = fresh;
    c.bad = len < 0 || fresh < 0 || fresh > max_new;
    c.held = given ? held : len < 0 ? 0 : static_cast<int32_t>(pages_of(len, page_size));
    // Tokens without pages, or more pages than the row has entries.
    c.bad = c.bad || c.held < 0 || c.held > max_pages ||
            static_cast<int64_t>(c.held) * page_size < len;
    if (c.bad) c.fresh = 0;
    c.need = 0;
    if (!c.bad) {
        const uint32_t want =
            pages_of(static_cast<uint32_t>(len) + static_cast<uint32_t>(fresh), page_size);
        c.bad = want > static_cast<uint32_t>(max_pages);   // taken as far as the row goes
        const int32_t most = c.bad ? max_pages : static_cast<int32_t>(want);
        c.need = most > c.held ? most - c.held : 0;
    }
    return c;
}

// A sequence's tokens, and how many of them are new.
struct TreeLens {
    int32_t len, fresh;
};

// The nearest in range of any two numbers; most: the tokens of a table's row.
CS_HOST_DEVICE TreeLens tree_lens_of(int32_t len, int32_t fresh, int32_t most,
                                     int32_t new_tokens) {
    TreeLens x;
    x.len = len < 0 ? 0 : len < most ? len : most;
    const int32_t top = new_tokens < x.len ? new_tokens : x.len;
    x.fresh = fresh < 0 ? 0 : fresh < top ? fresh : top;
    return x;
}

// Where a group's share of a batch's list begins: place g0 lies in sequence b,
// whose first place is base.
struct TreeStart {
    int32_t b, base;
    TreeLens n;
};

// From what the walk that looks for it left in memory, which is anything where
// the lengths were changed under the call and it found none.
CS_HOST_DEVICE TreeStart tree_start_of(const int32_t* found, int32_t g0, int32_t batch,
                                       int32_t most, int32_t new_tokens) {
    TreeStart x;
    x.b = found[0] < 0 ? 0 : found[0] < batch ? found[0] : batch - 1;
    x.base = found[1] < 0 ? 0 : found[1] < g0 ? found[1] : g0;
    x.n = tree_lens_of(found[2], found[3], most, new_tokens);
    return x;
}

}  // namespace cs
