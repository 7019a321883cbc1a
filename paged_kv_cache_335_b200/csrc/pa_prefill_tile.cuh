// pa_prefill_tile.cuh — tiles of packed prompts, shared by the kernels of
// pa_prefill.cu and pa_prefill_simt.cu.
#pragma once

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {

// One tile of one prompt.
struct PromptTile {
    int seq;    // -1: the index lies behind the last tile
    int start;  // the prompt's first packed row
    int len;    // its tokens
    int tile;   // which of the prompt's tiles
};

// Tile `u` of the packed prompts, found by a whole warp from the sequence starts (32
// prompts per step): prompts in order, each with tiles(its length) tiles, counted from
// the last to the first when `reversed`. A prompt with bad bounds (outside
// [0, total_tokens], negative length, or longer than max_seq_len) has no tile; *bad
// reports it.
template <typename Tiles>
__device__ __forceinline__ PromptTile prompt_tile(const PrefillParams& p, Tiles tiles, int u,
                                                  bool reversed, bool* bad) {
    const int lane = threadIdx.x & 31;
    PromptTile r;
    r.seq = -1;
    int seen = 0;
    for (int base = 0; base < p.num_seqs; base += 32) {
        const int s = base + lane;
        int a = 0, len = 0;
        if (s < p.num_seqs) {
            a = __ldg(p.cu_seqlens + s);
            const int b = __ldg(p.cu_seqlens + s + 1);
            len = b - a;
            if (a < 0 || b < a || b > p.total_tokens || len > p.max_seq_len) {
                *bad = true;
                len = 0;
            }
        }
        const int nt = tiles(len);
        int x = nt;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, off);
            if (lane >= off) x += y;
        }
        const int mine = seen + x - nt;  // tiles before this lane's prompt
        const bool hit = u >= mine && u < mine + nt;
        const uint32_t hits = __ballot_sync(0xffffffffu, hit);
        if (hits) {
            const int l = __ffs(hits) - 1;
            const int t = u - __shfl_sync(0xffffffffu, mine, l);
            const int n = __shfl_sync(0xffffffffu, nt, l);
            r.seq = base + l;
            r.start = __shfl_sync(0xffffffffu, a, l);
            r.len = __shfl_sync(0xffffffffu, len, l);
            r.tile = reversed ? n - 1 - t : t;
            return r;
        }
        seen += __shfl_sync(0xffffffffu, x, 31);
    }
    return r;
}

}  // namespace pa
