// pa_evict.cu — eviction from the paged cache by accumulated attention weight,
// and the accumulation of a decode step's weights.
//
// A few tokens receive most of the attention a cache is given; the others can
// go with little loss (the "heavy hitter" observation of Zhang et al., "H2O:
// Heavy-Hitter Oracle for Efficient Generative Inference of Large Language
// Models"). weights[s][kh][t] accumulates the softmax weight token t received
// from every query so far; eviction keeps, per sequence and kv head, the
// `recent` last tokens and the heaviest of the others, `budget` in all.
//
// Layout after an eviction. Attention does not care in which slot a token
// lies, so as few rows as possible are moved: with edge = budget - recent, the
// heavy tokens that already lie below `edge` stay, the others fill the slots
// below `edge` whose tokens go (i-th such slot, i-th such token), and the recent
// tokens follow in order at edge .. budget - 1. (Compacting in order instead
// would move every row behind the first hole.)
//
// Three kernels: select (one CTA per sequence and kv head: radix selection of
// the threshold weight, then ranks by population counts), fill (rows into
// holes: reads at or above edge, writes below it, so in any order), shift (the
// recent rows, in ascending chunks since source and target may overlap).
#include <math.h>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {

static __device__ unsigned int s_status_evict;

namespace {

__device__ __forceinline__ int clamp_len(int n, int max_n, bool report) {
    if (n < 0 || n > max_n) {
        if (report) atomicOr(&s_status_evict, kStatusBadIndex);
        n = n < 0 ? 0 : max_n;
    }
    return n;
}

// Order-preserving key of a weight: NaN counts as -infinity, -0 as +0.
__device__ __forceinline__ uint32_t weight_key(float w) {
    if (w != w) w = -INFINITY;
    const uint32_t u = __float_as_uint(w + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// ---------------------------------------------------------------------------
// fill and shift
// ---------------------------------------------------------------------------
// Row (token position t of sequence s, kv head kh) of the pools in 16-byte
// vectors; -1 for a block id outside the pool.
__device__ __forceinline__ int64_t row_of(const EvictParams& p, int s, int kh, int t) {
    const int32_t b = __ldg(p.block_tables + (int64_t)s * p.table_stride + (t >> p.log2_block_size));
    if ((unsigned)b >= (unsigned)p.num_blocks) {
        atomicOr(&s_status_evict, kStatusBadIndex);
        return -1;
    }
    return (((int64_t)b * p.num_kv_heads + kh) * p.block_size + (t & (p.block_size - 1))) * p.row_vecs;
}

// Rows into the holes below edge. A warp takes 32 slots, and moves the rows of
// those that change, 32 / row_vecs rows (of K and of V) per step.
constexpr int kFillWarps = 8;
__device__ __forceinline__ void fill_rows(const EvictParams& p, int s, int kh, int j, int edge) {
    const int lane = threadIdx.x & 31;
    const int64_t row = (int64_t)s * p.num_kv_heads + kh;
    int64_t src = -1, dst = -1;
    if (j < edge) {
        const int from = p.kept[row * p.budget + j];
        if (from != j) {
            src = row_of(p, s, kh, from);
            dst = row_of(p, s, kh, j);
            if (src < 0 || dst < 0) src = dst = -1;
        }
    }
    uint32_t todo = __ballot_sync(0xffffffffu, dst >= 0);
    const int rows = 32 / p.row_vecs, sub = lane / p.row_vecs, c = lane % p.row_vecs;
    constexpr int kU = 4;
    while (todo) {
        uint4 kv[kU], vv[kU];
        int64_t d[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            int mine = -1;
            for (int r = 0; r < rows && todo; ++r) {
                const int b = __ffs(todo) - 1;
                todo &= todo - 1;
                if (r == sub) mine = b;
            }
            const int64_t a = __shfl_sync(0xffffffffu, src, mine < 0 ? 0 : mine);
            d[u] = __shfl_sync(0xffffffffu, dst, mine < 0 ? 0 : mine);
            if (mine < 0) d[u] = -1;
            if (d[u] >= 0) {
                kv[u] = ld_v4(p.k_cache + a + c);
                vv[u] = ld_v4(p.v_cache + a + c);
            }
        }
#pragma unroll
        for (int u = 0; u < kU; ++u)
            if (d[u] >= 0) {
                p.k_cache[d[u] + c] = kv[u];
                p.v_cache[d[u] + c] = vv[u];
            }
    }
}

__global__ void __launch_bounds__(kFillWarps * 32)
evict_fill_kernel(const EvictParams p) {
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int kh = blockIdx.y, s = blockIdx.z;
    const int n = clamp_len(__ldg(p.context_lens + s), p.max_context_len, false);
    if (n > p.budget)
        fill_rows(p, s, kh, blockIdx.x * kFillWarps * 32 + threadIdx.x, p.budget - p.recent);
}

// The recent rows: slot edge + i gets position n - recent + i. One CTA per
// (K or V, kv head, sequence) goes through them in ascending chunks that are read whole
// before any is written: a slot written by a chunk is the source of no later one.
constexpr int kShiftThreads = 512;
constexpr int kShiftU = 8;
template <int kThreads>
__device__ __forceinline__ void shift_rows(const EvictParams& p, uint4* cache, int s, int kh, int n, int edge) {
    const int c = threadIdx.x % p.row_vecs, r0 = threadIdx.x / p.row_vecs;
    const int rows = kThreads / p.row_vecs;  // per pass
    for (int base = 0; base < p.recent; base += rows * kShiftU) {
        uint4 v[kShiftU];
        int64_t d[kShiftU];
#pragma unroll
        for (int u = 0; u < kShiftU; ++u) {
            const int i = base + u * rows + r0;
            d[u] = -1;
            if (i < p.recent) {
                const int64_t a = row_of(p, s, kh, n - p.recent + i);
                d[u] = row_of(p, s, kh, edge + i);
                if (a < 0) d[u] = -1;
                if (d[u] >= 0) v[u] = ld_v4(cache + a + c);
            }
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < kShiftU; ++u)
            if (d[u] >= 0) cache[d[u] + c] = v[u];
        __syncthreads();
    }
}

__global__ void __launch_bounds__(kShiftThreads)
evict_shift_kernel(const EvictParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int kh = blockIdx.y, s = blockIdx.z;
    const int n = clamp_len(__ldg(p.context_lens + s), p.max_context_len, false);
    if (n > p.budget)
        shift_rows<kShiftThreads>(p, blockIdx.x ? p.v_cache : p.k_cache, s, kh, n, p.budget - p.recent);
}

// ---------------------------------------------------------------------------
// select
// ---------------------------------------------------------------------------
// The threshold key is found digit by digit (11, 11 and 10 bits; four of 8 in short contexts,
// where counting 2048 bins would cost more than a pass over the keys) from histograms in shared
// memory; the keys lie there too, so that the weights are read once (contexts above what it
// holds read them again in every pass). A warp owns a run of 32-token words, a lane a
// token of each, and takes kBatch words at a time: with one load per step a row of 32K
// took 53 us, each step a memory latency. The first digit is sign, exponent and two
// bits of a heavy-tailed distribution, a few dozen bins: each bin has kCopies places,
// so that a warp's lanes collide less.
constexpr int kCopies = 4;
constexpr int kBatch = 8;
constexpr int kMaxWarps = 32;

template <int kThreads_>
struct Select {
    static constexpr int kThreads = kThreads_, kWarps = kThreads / 32;
    static constexpr int kDigit = kThreads == 256 ? 8 : 11, kBins = 1 << kDigit;
    static constexpr int kListCap = kThreads == 256 ? 4096 : 8192;  // movers listed per round, where
                                                                    // the histograms were
    static_assert(kListCap >= kBins * kCopies && kBins >= kThreads, "histograms");
};

// Shared memory: [chosen bits: words][holes or movers before a word: words]
// [histograms, then the mover list: kListCap][scan: kMaxWarps + misc][keys].
template <int kThreads>
__device__ __forceinline__ int block_scan_exclusive(int v, int* sm, int& total) {
    constexpr int kWarps = kThreads / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off) x += y;
    }
    if (lane == 31) sm[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int w = lane < kWarps ? sm[lane] : 0;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, w, off);
            if (lane >= off) w += y;
        }
        if (lane < kWarps) sm[lane] = w;
    }
    __syncthreads();
    total = sm[kWarps - 1];
    const int r = x - v + (warp ? sm[warp - 1] : 0);
    __syncthreads();
    return r;
}

// f(word, key, token exists) for each word of the warp's run w0 .. w1, in order; keys of the
// first `cand` tokens, from shared memory or made of the weights. (The weights are read by
// plain loads: the read-only path is not for what this kernel may overwrite in place.)
template <bool kShared, typename F>
__device__ __forceinline__ void each_word(const float* w, const uint32_t* keys, int w0, int w1, int cand, F f) {
    const int lane = threadIdx.x & 31;
    for (int i = w0; i < w1; i += kBatch) {
        uint32_t k[kBatch];
#pragma unroll
        for (int e = 0; e < kBatch; ++e) {
            const int t = 32 * (i + e) + lane;
            k[e] = 0u;
            if (i + e < w1 && t < cand) k[e] = kShared ? keys[t] : weight_key(w[t]);
        }
#pragma unroll
        for (int e = 0; e < kBatch; ++e)
            if (i + e < w1) f(i + e, k[e], 32 * (i + e) + lane < cand);
    }
}

// Marks the kept candidates of a row in `bits`, with the holes below edge or the movers behind
// it before each word; returns the number of holes.
template <int kThreads, bool kShared>
__device__ __forceinline__ int select_row(const float* w, int cand, int edge, uint32_t* bits, int* before,
                                          int* hist, int* scan, uint32_t* keys) {
    using C = Select<kThreads>;
    constexpr int kWarps = C::kWarps, kBins = C::kBins;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    volatile int* misc = scan + kMaxWarps;  // bin, remaining rank
    const int words = (cand + 31) / 32;
    const int wpw = (words + kWarps - 1) / kWarps;
    const int w0 = min(words, warp * wpw), w1 = min(words, w0 + wpw);
    if constexpr (kShared) {
        // four tokens per load where the row is aligned, eight loads of a thread in flight
        const int quads = (reinterpret_cast<uintptr_t>(w) & 15u) == 0 ? cand / 4 : 0;
        for (int i0 = tid; i0 < quads; i0 += kBatch * kThreads) {
            float4 x[kBatch];
#pragma unroll
            for (int e = 0; e < kBatch; ++e)
                if (i0 + e * kThreads < quads) x[e] = reinterpret_cast<const float4*>(w)[i0 + e * kThreads];
#pragma unroll
            for (int e = 0; e < kBatch; ++e)
                if (i0 + e * kThreads < quads)
                    reinterpret_cast<uint4*>(keys)[i0 + e * kThreads] =
                        make_uint4(weight_key(x[e].x), weight_key(x[e].y), weight_key(x[e].z), weight_key(x[e].w));
        }
        for (int t = 4 * quads + tid; t < cand; t += kThreads) keys[t] = weight_key(w[t]);
        __syncthreads();
    }
    // The edge-th largest key among the candidates, and how many of the tokens
    // that hold exactly that key are taken (the lowest indices).
    uint32_t prefix = 0, known = 0;   // digits found so far and their bits
    int want = edge;                  // rank of the threshold within the tokens matching `prefix`
    if (edge > 0) {
        for (int shift = 32 - C::kDigit; known != 0xffffffffu; shift = max(0, shift - C::kDigit)) {
            const uint32_t mask = ~known >> shift;   // the digit: the last one may be shorter
            for (int b = tid; b < kBins; b += kThreads) reinterpret_cast<int4*>(hist)[b] = make_int4(0, 0, 0, 0);
            __syncthreads();
            each_word<kShared>(w, keys, w0, w1, cand, [&](int, uint32_t key, bool in) {
                if (in && (key & known) == prefix)
                    atomicAdd(&hist[((key >> shift) & mask) * kCopies + (lane & (kCopies - 1))], 1);
            });
            __syncthreads();
            // bins from the top, kBins / kThreads to a thread: the one that holds rank `want`
            constexpr int kMine = kBins / kThreads;
            int c[kMine], sum = 0;
#pragma unroll
            for (int i = 0; i < kMine; ++i) {
                const int4 h = reinterpret_cast<const int4*>(hist)[kBins - 1 - (tid * kMine + i)];
                c[i] = h.x + h.y + h.z + h.w;
                sum += c[i];
            }
            int total;
            int above = block_scan_exclusive<kThreads>(sum, scan, total);
#pragma unroll
            for (int i = 0; i < kMine; ++i) {
                if (above < want && want <= above + c[i]) {
                    misc[0] = kBins - 1 - (tid * kMine + i);
                    misc[1] = want - above;
                }
                above += c[i];
            }
            __syncthreads();
            prefix |= (uint32_t)misc[0] << shift;
            want = misc[1];
            known |= mask << shift;
            __syncthreads();
        }
    }
    const uint32_t thr = prefix;
    // Each word's tokens above the threshold and on it, one word per lane in turn (a word costs two
    // comparisons and two votes; the counting below is a lane's work for a word).
    int eq_count = 0;
    for (int i = w0; i < w1; i += 32) {
        uint32_t mine_gt = 0, mine_eq = 0;
        each_word<kShared>(w, keys, i, min(i + 32, w1), cand, [&](int j, uint32_t key, bool in) {
            const uint32_t gt = __ballot_sync(0xffffffffu, in && key > thr);
            const uint32_t eq = __ballot_sync(0xffffffffu, in && key == thr);
            if (lane == j - i) {
                mine_gt = gt;
                mine_eq = eq;
            }
        });
        if (edge == 0) mine_gt = mine_eq = 0;
        if (i + lane < w1) {
            bits[i + lane] = mine_gt;
            before[i + lane] = (int)mine_eq;
        }
        eq_count += __popc(mine_eq);
    }
    int total;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) eq_count += __shfl_xor_sync(0xffffffffu, eq_count, off);
    // lane 0 carries the warp's count: exclusive prefix over the warps
    int eq_before = block_scan_exclusive<kThreads>(lane == 0 ? eq_count : 0, scan, total);
    eq_before = __shfl_sync(0xffffffffu, eq_before, 0);
    // inclusive sum over the lanes
    auto lanes_sum = [&](int x) {
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, off);
            if (lane >= off) x += y;
        }
        return x;
    };
    auto below_mask = [&](int i) {  // tokens of word i below edge: holes count there, movers above it
        const int below = max(0, min(32, edge - 32 * i));
        return below == 32 ? 0xffffffffu : (1u << below) - 1u;
    };
    int holes = 0, movers = 0;
    for (int i = w0; i < w1; i += 32) {
        const bool have = i + lane < w1;
        uint32_t eq = have ? (uint32_t)before[i + lane] : 0u;
        const int sum = lanes_sum(__popc(eq));
        // of the equal ones the lowest `want` are taken; one word at most is cut
        int take = want - (eq_before + sum - __popc(eq));
        if (take <= 0) eq = 0;
        for (; __popc(eq) > take && eq != 0; eq &= ~(0x80000000u >> __clz(eq))) {
        }
        eq_before += __shfl_sync(0xffffffffu, sum, 31);
        if (have) {
            const uint32_t cm = bits[i + lane] | eq, bm = below_mask(i + lane);
            bits[i + lane] = cm;
            holes += __popc(~cm & bm);
            movers += __popc(cm & ~bm);
        }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        holes += __shfl_xor_sync(0xffffffffu, holes, off);
        movers += __shfl_xor_sync(0xffffffffu, movers, off);
    }
    // holes before each word below edge, movers before each word above it (the
    // word that holds edge itself counts movers; its holes come last)
    int hb = block_scan_exclusive<kThreads>(lane == 0 ? holes : 0, scan, total);
    const int num_holes = total;
    int mb = block_scan_exclusive<kThreads>(lane == 0 ? movers : 0, scan, total);
    hb = __shfl_sync(0xffffffffu, hb, 0);
    mb = __shfl_sync(0xffffffffu, mb, 0);
    for (int i = w0; i < w1; i += 32) {
        const bool have = i + lane < w1;
        const uint32_t bm = below_mask(i + lane), cm = have ? bits[i + lane] : bm;
        const int h = __popc(~cm & bm), m = have ? __popc(cm & ~bm) : 0;
        const int hs = lanes_sum(h), ms = lanes_sum(m);
        if (have) before[i + lane] = bm == 0xffffffffu ? hb + hs - h : mb + ms - m;
        hb += __shfl_sync(0xffffffffu, hs, 31);
        mb += __shfl_sync(0xffffffffu, ms, 31);
    }
    __syncthreads();
    return num_holes;
}

// kMove: also the rows (else evict_fill_kernel and evict_shift_kernel follow).
template <int kThreads, bool kShared, bool kMove>
__global__ void __launch_bounds__(kThreads, kThreads != 256 ? 1 : kMove ? 4 : 5)
evict_select_kernel(const EvictParams p) {
    constexpr int kWarps = kThreads / 32, kListCap = Select<kThreads>::kListCap;
    extern __shared__ __align__(16) uint32_t sm_u[];
    const int kh = blockIdx.x, s = blockIdx.y;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int words_cap = (p.max_context_len + 127) / 128 * 4;   // (the list stays 16-byte aligned)
    uint32_t* bits = sm_u;                                    // chosen tokens
    int* before = reinterpret_cast<int*>(bits + words_cap);
    int* list = before + words_cap;
    int* scan = list + kListCap;
    asm volatile("griddepcontrol.launch_dependents;");
    const int n = clamp_len(__ldg(p.context_lens + s), p.max_context_len, tid == 0 && kh == 0);
    const int64_t row = (int64_t)s * p.num_kv_heads + kh;
    const float* w = p.weights + row * p.weights_stride;
    float* wo = p.weights_out + row * p.weights_stride;
    int32_t* kept = p.kept + row * p.budget;
    const int new_n = min(n, p.budget);
    if (kh == 0 && tid == 0) p.new_context_lens[s] = new_n;
    if (n <= p.budget) {  // nothing to evict
        for (int j = tid; j < p.budget; j += kThreads) kept[j] = j < n ? j : -1;
        if (wo != w)
            for (int j = tid; j < n; j += kThreads) wo[j] = w[j];
        for (int64_t j = n + tid; j < p.weights_stride; j += kThreads) wo[j] = 0.f;
        return;
    }
    const int edge = p.budget - p.recent, cand = n - p.recent;  // cand > edge
    const int words = (cand + 31) / 32;
    const int num_holes = select_row<kThreads, kShared>(
        w, cand, edge, bits, before, list, scan, reinterpret_cast<uint32_t*>(scan + kMaxWarps + 4));
    const int edge_word = edge / 32;
    // The i-th mover goes to the i-th hole, kListCap of them per round.
    for (int r0 = 0; r0 < num_holes; r0 += kListCap) {
        for (int i = edge_word + warp; i < words; i += kWarps) {
            const int below = max(0, min(32, edge - 32 * i));
            const uint32_t bm = below == 32 ? 0xffffffffu : (1u << below) - 1u;
            const uint32_t m = bits[i] & ~bm;
            const int rank = before[i] + __popc(m & ((1u << lane) - 1u)) - r0;
            if ((m >> lane & 1u) && rank >= 0 && rank < kListCap) list[rank] = 32 * i + lane;
        }
        __syncthreads();
        // (kPlaced words at a time, their weights in flight together)
        constexpr int kPlaced = 8;
        for (int i0 = warp; 32 * i0 < edge; i0 += kPlaced * kWarps) {
            int src[kPlaced];
            float v[kPlaced];
#pragma unroll
            for (int e = 0; e < kPlaced; ++e) {
                const int i = i0 + e * kWarps, j = 32 * i + lane;
                src[e] = -1;
                if (32 * i >= edge) continue;
                const int below = min(32, edge - 32 * i);
                const uint32_t bm = below == 32 ? 0xffffffffu : (1u << below) - 1u;
                const uint32_t h = ~bits[i] & bm;
                // the word that holds edge: its holes are the last ones
                const int base = below == 32 ? before[i] : num_holes - __popc(h);
                const int rank = base + __popc(h & ((1u << lane) - 1u)) - r0;
                if (h >> lane & 1u) {
                    if (rank >= 0 && rank < kListCap) src[e] = list[rank];
                } else if (r0 == 0 && j < edge) {
                    src[e] = j;
                }
                // (a mover's place is >= edge: not yet overwritten when the weights are in place)
                if (src[e] >= 0) v[e] = w[src[e]];
            }
#pragma unroll
            for (int e = 0; e < kPlaced; ++e) {
                const int j = 32 * (i0 + e * kWarps) + lane;
                if (src[e] < 0) continue;
                kept[j] = src[e];
                wo[j] = v[e];
            }
        }
        __syncthreads();
    }
    if (num_holes == 0)
        for (int j = tid; j < edge; j += kThreads) {
            kept[j] = j;
            if (wo != w) wo[j] = w[j];
        }
    __syncthreads();
    // recent tokens, ascending (in place, a chunk is read before it is written)
    for (int j0 = 0; j0 < p.recent; j0 += kThreads) {
        const int j = j0 + tid;
        float v = 0.f;
        if (j < p.recent) {
            kept[edge + j] = cand + j;
            v = w[cand + j];
        }
        __syncthreads();
        if (j < p.recent) wo[edge + j] = v;
        __syncthreads();
    }
    for (int64_t j = p.budget + tid; j < p.weights_stride; j += kThreads) wo[j] = 0.f;
    if constexpr (kMove) {
        __syncthreads();   // `kept` is written
        for (int j = tid - lane; j < edge; j += kThreads) fill_rows(p, s, kh, j + lane, edge);
        __syncthreads();   // the fill reads rows behind edge before the shift writes them
        shift_rows<kThreads>(p, p.k_cache, s, kh, n, edge);
        shift_rows<kThreads>(p, p.v_cache, s, kh, n, edge);
    }
}

// ---------------------------------------------------------------------------
// the weights of a decode step
// ---------------------------------------------------------------------------
// weights[s][kh][t] += sum over the heads of the group of 2^(score - lse), with
// lse the log-sum-exp (log2 units) of the head's partitions: the decode kernel left
// every score (log2 units) and each partition's running max and sum.
constexpr int kAddThreads = 256;
constexpr int kAddTokens = 4;  // per thread, consecutive: one 16-byte load per head
constexpr int kMaxHeads = 8;   // of a group, per round: their scores are on the way while the warps
                               // (one per head) form the log-sum-exps

__global__ void __launch_bounds__(kAddThreads)
add_weights_kernel(const AddWeightsParams p) {
    __shared__ float lse[kMaxHeads];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int kh = blockIdx.y, s = blockIdx.z;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int n = clamp_len(__ldg(p.context_lens + s), p.max_context_len, false);
    if ((int)(blockIdx.x * kAddThreads * kAddTokens) >= n) return;
    const int t = (blockIdx.x * kAddThreads + threadIdx.x) * kAddTokens;
    const int group = p.num_heads / p.num_kv_heads;
    const int parts = (n + p.partition_size - 1) / p.partition_size;
    float* w = p.weights + ((int64_t)s * p.num_kv_heads + kh) * p.weights_stride + t;
    float acc[kAddTokens] = {0.f, 0.f, 0.f, 0.f};
    for (int h0 = 0; h0 < group; h0 += kMaxHeads) {
        const int heads = min(kMaxHeads, group - h0);
        const float* sc = p.scores + ((int64_t)s * p.num_heads + kh * group + h0) * p.score_stride + t;
        float4 x[kMaxHeads];
#pragma unroll
        for (int h = 0; h < kMaxHeads; ++h)
            if (h < heads && t < n) x[h] = __ldcs(reinterpret_cast<const float4*>(sc + (int64_t)h * p.score_stride));
        for (int h = warp; h < heads; h += kAddThreads / 32) {
            const float2* ml = reinterpret_cast<const float2*>(p.ml) +
                               ((int64_t)s * p.num_heads + kh * group + h0 + h) * p.num_partitions;
            float M = -INFINITY, L = 0.f;
            for (int j = lane; j < parts; j += 32) M = fmaxf(M, ml[j].x);
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
            for (int j = lane; j < parts; j += 32)
                if (ml[j].x != -INFINITY) L = fmaf(ml[j].y, exp2f(ml[j].x - M), L);
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) L += __shfl_xor_sync(0xffffffffu, L, off);
            // no partition had a score (every block id was bad): no weights
            if (lane == 0) lse[h] = L == 0.f ? INFINITY : M + log2f(L);
        }
        __syncthreads();
#pragma unroll
        for (int h = 0; h < kMaxHeads; ++h) {
            if (h >= heads || t >= n) break;
            const float e = lse[h];
            acc[0] += exp2f(x[h].x - e);
            acc[1] += exp2f(x[h].y - e);
            acc[2] += exp2f(x[h].z - e);
            acc[3] += exp2f(x[h].w - e);
        }
        __syncthreads();
    }
    if (t + kAddTokens <= n && (reinterpret_cast<uintptr_t>(w) & 15u) == 0) {
        float4 x = *reinterpret_cast<const float4*>(w);
        x.x += acc[0];
        x.y += acc[1];
        x.z += acc[2];
        x.w += acc[3];
        *reinterpret_cast<float4*>(w) = x;
    } else {
#pragma unroll
        for (int u = 0; u < kAddTokens; ++u)
            if (t + u < n) w[u] += acc[u];
    }
}

}  // namespace

template <int kThreads>
static constexpr size_t evict_smem_bytes(int max_context_len, bool keys) {
    const size_t words = ((size_t)max_context_len + 127) / 128 * 4;
    return 4 * (2 * words + Select<kThreads>::kListCap + kMaxWarps + 4 + (keys ? 32 * words : 0));
}

constexpr size_t kMaxSmem = 227 * 1024;
constexpr int kShortContext = 4096;   // contexts up to this take the 256-thread form

int evict_max_context() { return (int)((kMaxSmem - evict_smem_bytes<1024>(0, false)) / 32 * 128); }

// A kernel that starts while the one before it ends (it waits for it itself).
template <typename K>
static cudaError_t launch_dependent(K kernel, dim3 grid, int threads, size_t smem, cudaStream_t stream,
                                    const EvictParams& p) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <int kThreads, bool kShared, bool kMove>
static cudaError_t launch_select(const EvictParams& p, cudaStream_t stream) {
    // The limit is the kernel's, for every host thread at once: the same in every call, whatever
    // this one takes.
    const size_t smem = evict_smem_bytes<kThreads>(p.max_context_len, kShared);
    const size_t limit = kThreads == 256 ? evict_smem_bytes<kThreads>(kShortContext, kShared) : kMaxSmem;
    cudaError_t e = cudaFuncSetAttribute(evict_select_kernel<kThreads, kShared, kMove>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, (int)limit);
    if (e != cudaSuccess) return e;
    evict_select_kernel<kThreads, kShared, kMove>
        <<<dim3((unsigned)p.num_kv_heads, (unsigned)p.num_seqs), kThreads, smem, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_evict(const EvictParams& p, cudaStream_t stream) {
    const dim3 rows((unsigned)p.num_kv_heads, (unsigned)p.num_seqs);
    // A row of a short context is bound by its barriers: fewer threads, more rows per SM. Where such
    // rows fill the SMs, each also moves its own keys and values: 16 x 40 rows of 2064
    // tokens take 19.7 us on the device, with the two further launches 20.5 and 4 us more of host time.
    if (p.max_context_len <= kShortContext && (int64_t)rows.x * rows.y >= 148)
        return launch_select<256, true, true>(p, stream);
    cudaError_t e = p.max_context_len <= kShortContext ? launch_select<256, true, false>(p, stream)
                    : evict_smem_bytes<1024>(p.max_context_len, true) <= kMaxSmem
                        ? launch_select<1024, true, false>(p, stream)
                        : launch_select<1024, false, false>(p, stream);
    if (e != cudaSuccess) return e;
    if (p.max_context_len <= p.budget) return cudaSuccess;  // no sequence is over its budget
    const int edge = p.budget - p.recent;
    if (edge > 0) {
        const unsigned chunks = (unsigned)((edge + kFillWarps * 32 - 1) / (kFillWarps * 32));
        e = launch_dependent(evict_fill_kernel, dim3(chunks, rows.x, rows.y), kFillWarps * 32, 0, stream, p);
        if (e != cudaSuccess) return e;
    }
    if (p.recent > 0)
        e = launch_dependent(evict_shift_kernel, dim3(2, rows.x, rows.y), kShiftThreads, 0, stream, p);
    return e;
}

cudaError_t launch_add_weights(const AddWeightsParams& p, cudaStream_t stream) {
    if (p.max_context_len == 0) return cudaSuccess;
    const int per = kAddThreads * kAddTokens;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((p.max_context_len + per - 1) / per), (unsigned)p.num_kv_heads,
                       (unsigned)p.num_seqs);
    cfg.blockDim = dim3(kAddThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, add_weights_kernel, p);
}

cudaError_t read_status_evict(unsigned* bits, bool clear) {
    cudaError_t e = cudaMemcpyFromSymbol(bits, s_status_evict, sizeof(unsigned));
    if (e != cudaSuccess || !clear || *bits == 0) return e;
    const unsigned zero = 0;
    return cudaMemcpyToSymbol(s_status_evict, &zero, sizeof(unsigned));
}

}  // namespace pa
