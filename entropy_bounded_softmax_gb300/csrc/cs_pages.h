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

}  // namespace cs
