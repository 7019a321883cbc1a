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

// Finds tiles of the packed prompts by their index, a whole warp at a time: prompts in
// order, each with tiles(its length) tiles, counted from the last to the first when
// `reversed`. A prompt with bad bounds (outside [0, total_tokens], negative
// length, or longer than max_seq_len) has no tile; `bad` reports that the lane met one.
// The warp holds 32 prompts (one per lane) and the number of tiles before them; an index at
// or behind those goes on from there, so indices that ascend read each prompt once.
struct PromptWalk {
    int base = 0;      // prompts of the lanes: base ..
    int seen = 0;      // tiles before them
    int start = 0, len = 0, count = 0, before = 0;   // the lane's prompt, its tiles, tiles before it
    int total = 0;     // tiles of the 32
    bool loaded = false, bad = false;

    template <typename Tiles>
    __device__ __forceinline__ void load(const PrefillParams& p, Tiles tiles) {
        const int lane = threadIdx.x & 31;
        const int s = base + lane;
        start = len = 0;
        if (s < p.num_seqs) {
            start = __ldg(p.cu_seqlens + s);
            const int b = __ldg(p.cu_seqlens + s + 1);
            len = b - start;
            if (start < 0 || b < start || b > p.total_tokens || len > p.max_seq_len) {
                bad = true;
                len = 0;
            }
        }
        count = tiles(len);
        int x = count;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, off);
            if (lane >= off) x += y;
        }
        before = seen + x - count;
        total = __shfl_sync(0xffffffffu, x, 31);
        loaded = true;
    }

    template <typename Tiles>
    __device__ __forceinline__ PromptTile find(const PrefillParams& p, Tiles tiles, int u, bool reversed) {
        PromptTile r;
        r.seq = -1;
        r.start = r.len = r.tile = 0;
        if (u < seen) {  // behind an index that came before: from the start again
            base = seen = 0;
            loaded = false;
        }
        if (!loaded) load(p, tiles);
        while (u >= seen + total) {
            if (base + 32 >= p.num_seqs) return r;
            base += 32;
            seen += total;
            load(p, tiles);
        }
        const uint32_t hits = __ballot_sync(0xffffffffu, u >= before && u < before + count);
        const int l = __ffs(hits) - 1;
        const int t = u - __shfl_sync(0xffffffffu, before, l);
        const int n = __shfl_sync(0xffffffffu, count, l);
        r.seq = base + l;
        r.start = __shfl_sync(0xffffffffu, start, l);
        r.len = __shfl_sync(0xffffffffu, len, l);
        r.tile = reversed ? n - 1 - t : t;
        return r;
    }
};

}  // namespace pa
