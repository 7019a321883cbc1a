// pa_prompt_walk.cuh — tiles of packed prompts by their index. Of CUDA it uses the warp
// intrinsics alone, so that a host program which provides them (tests/prompt_walk_host.cpp)
// runs this very code.
#pragma once

#include "pa_internal.h"

namespace pa {

// One tile of one prompt.
struct PromptTile {
    int seq;    // -1: the index lies behind the last tile
    int start;  // the prompt's first packed row
    int len;    // its tokens
    int tile;   // which of the prompt's tiles
};

// Finds tiles of the packed prompts by their index, a whole warp at a time. The prompts
// come 32 at a time (one per lane), each with tiles(its length) tiles; among the tiles
// of the 32 those with the most work come first: rank r of a prompt's `count` tiles is
// tile r when `reversed` (a query tile attends to the tiles before it), else tile
// count - 1 - r (a key tile is attended to by those behind it), and the ranks descend. A
// prompt with bad bounds (outside [0, total_tokens], negative length, longer than max_seq_len,
// or with a first row before the end of an earlier prompt) has no tile; `bad` reports that the
// lane met one. So the prompts that have tiles are disjoint, and all their tiles of B tokens are
// at most total_tokens / B + num_seqs. Indices that ascend read each prompt once.
struct PromptWalk {
    int base = 0;      // prompts of the lanes: base ..
    int seen = 0;      // tiles before them
    int start = 0, len = 0, count = 0;   // the lane's prompt
    int total = 0;     // tiles of the 32
    int reach = 0, next_reach = 0;       // the furthest end of the prompts before the 32, and with them
    int rank = 0, above = 0, upto = 0;   // the last rank, tiles of higher ranks, and with this one's
    bool loaded = false, bad = false;

    template <typename Tiles>
    __device__ __forceinline__ void load(const PrefillParams& p, Tiles tiles) {
        const int lane = threadIdx.x & 31, s = base + lane;
        start = len = 0;
        int end = 0;
        bool descends = false;
        if (s < p.num_seqs) {
            start = __ldg(p.cu_seqlens + s);
            end = __ldg(p.cu_seqlens + s + 1);
            len = end - start;
            descends = end < start;
            if (start < 0 || end < start || end > p.total_tokens || len > p.max_seq_len) {
                bad = true;
                len = end = 0;
            }
        }
        // Bounds that never descend hold no overlap.
        if (__any_sync(0xffffffffu, descends || (len > 0 && start < reach))) {
            int far = end;   // the furthest end up to each prompt, then before it
#pragma unroll 1
            for (int off = 1; off < 32; off <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, far, off);
                if (lane >= off) far = max(far, y);
            }
            far = __shfl_up_sync(0xffffffffu, far, 1);
            if (len > 0 && start < (lane > 0 ? max(far, reach) : reach)) {
                bad = true;
                len = 0;
            }
        }
        next_reach = max(reach, __reduce_max_sync(0xffffffffu, end));
        count = tiles(len);
        total = __reduce_add_sync(0xffffffffu, count);
        rank = above = upto = 0;   // (the rank of the 32 before means nothing here: the next search starts anew)
        loaded = true;
    }

    // Tiles of the 32 prompts with rank r or above.
    __device__ __forceinline__ int from_rank(int r) const {
        return __reduce_add_sync(0xffffffffu, max(0, count - r));
    }

    template <typename Tiles>
    __device__ __forceinline__ PromptTile find(const PrefillParams& p, Tiles tiles, int u, bool reversed) {
        PromptTile t;
        t.seq = -1;
        t.start = t.len = t.tile = 0;
        if (u < seen) {  // behind an index that came before: from the start again
            base = seen = reach = 0;
            loaded = false;
        }
        if (!loaded) load(p, tiles);
        while (u >= seen + total) {
            if (base + 32 >= p.num_seqs) return t;
            base += 32;
            seen += total;
            reach = next_reach;
            load(p, tiles);
        }
        // the rank: from_rank(rank) > v >= from_rank(rank + 1); mostly the last one still
        const int v = u - seen;
        for (int i = 0; i < 4 && v >= upto && rank > 0; ++i) {  // the next ones below
            --rank;
            above = upto;
            upto = from_rank(rank);
        }
        if (v < above || v >= upto) {
            rank = 0;
            int high = __reduce_max_sync(0xffffffffu, count);
            while (high - rank > 1) {
                const int mid = (rank + high) >> 1;
                if (from_rank(mid) > v)
                    rank = mid;
                else
                    high = mid;
            }
            above = from_rank(rank + 1);
            upto = from_rank(rank);
        }
        const uint32_t have = __ballot_sync(0xffffffffu, count > rank);
        const bool mine = count > rank && __popc(have & ((1u << (threadIdx.x & 31)) - 1u)) == v - above;
        const int l = __ffs(__ballot_sync(0xffffffffu, mine)) - 1;
        t.seq = base + l;
        t.start = __shfl_sync(0xffffffffu, start, l);
        t.len = __shfl_sync(0xffffffffu, len, l);
        const int n = __shfl_sync(0xffffffffu, count, l);
        t.tile = reversed ? rank : n - 1 - rank;
        return t;
    }
};

}  // namespace pa
