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
// select
// ---------------------------------------------------------------------------
constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 256;
constexpr int kListCap = 8192;  // movers listed per round

// Shared memory: [chosen bits: words][holes or movers before a word: words]
// [mover list: kListCap][histogram: kBins][misc].
__device__ __forceinline__ int block_scan_exclusive(int v, int* sm, int& total) {
    // sm: kSelWarps + 1 ints
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
        int w = sm[lane];
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, w, off);
            if (lane >= off) w += y;
        }
        sm[lane] = w;
    }
    __syncthreads();
    total = sm[kSelWarps - 1];
    const int r = x - v + (warp ? sm[warp - 1] : 0);
    __syncthreads();
    return r;
}

__global__ void __launch_bounds__(kSelThreads, 1)
evict_select_kernel(const EvictParams p) {
    extern __shared__ __align__(16) uint32_t sm_u[];
    const int kh = blockIdx.x, s = blockIdx.y;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int words_cap = (p.max_context_len + 31) / 32;
    uint32_t* bits = sm_u;                                    // chosen tokens
    int* before = reinterpret_cast<int*>(bits + words_cap);   // per word: see below
    int* list = before + words_cap;
    int* hist = list + kListCap;
    int* scan = hist + kBins;                                 // kSelWarps
    volatile int* misc = scan + kSelWarps;                    // bin, remaining
    const int n = clamp_len(__ldg(p.context_lens + s), p.max_context_len, tid == 0 && kh == 0);
    const int64_t row = (int64_t)s * p.num_kv_heads + kh;
    const float* w = p.weights + row * p.weights_stride;
    float* wo = p.weights_out + row * p.weights_stride;
    int32_t* kept = p.kept + row * p.budget;
    const int new_n = min(n, p.budget);
    if (kh == 0 && tid == 0) p.new_context_lens[s] = new_n;
    if (n <= p.budget) {  // nothing to evict
        for (int j = tid; j < p.budget; j += kSelThreads) kept[j] = j < n ? j : -1;
        if (wo != w)
            for (int j = tid; j < n; j += kSelThreads) wo[j] = w[j];
        for (int j = n + tid; j < p.weights_stride; j += kSelThreads) wo[j] = 0.f;
        return;
    }
    const int edge = p.budget - p.recent, cand = n - p.recent;  // cand > edge
    const int words = (cand + 31) / 32;

    // The edge-th largest key among the candidates, and how many of the tokens
    // that hold exactly that key are taken (the lowest indices).
    uint32_t prefix = 0;
    int want = edge;  // rank of the threshold within the tokens matching `prefix`
    if (edge > 0) {
        for (int shift = 24; shift >= 0; shift -= 8) {
            for (int b = tid; b < kBins; b += kSelThreads) hist[b] = 0;
            __syncthreads();
            const uint32_t high = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
            for (int t = tid; t < cand; t += kSelThreads) {
                const uint32_t key = weight_key(w[t]);
                if ((key & high) == prefix) atomicAdd(&hist[(key >> shift) & 255u], 1);
            }
            __syncthreads();
            if (warp == 0) {  // bins from the top: the one that holds rank `want`
                int c[8], sum = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    c[i] = hist[255 - (lane * 8 + i)];
                    sum += c[i];
                }
                int x = sum;
#pragma unroll
                for (int off = 1; off < 32; off <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, x, off);
                    if (lane >= off) x += y;
                }
                int above = x - sum;
                if (above < want && want <= x) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        if (above < want && want <= above + c[i]) {
                            misc[0] = 255 - (lane * 8 + i);
                            misc[1] = want - above;
                        }
                        above += c[i];
                    }
                }
            }
            __syncthreads();
            prefix |= (uint32_t)misc[0] << shift;
            want = misc[1];
            __syncthreads();
        }
    }
    const uint32_t thr = prefix;
    // Equal keys before each word (a warp owns a run of words; lane = token).
    const int wpw = (words + kSelWarps - 1) / kSelWarps;
    const int w0 = min(words, warp * wpw), w1 = min(words, w0 + wpw);
    int eq_count = 0;
    for (int i = w0; i < w1; ++i) {
        const int t = 32 * i + lane;
        const bool eq = edge > 0 && t < cand && weight_key(w[t]) == thr;
        eq_count += __popc(__ballot_sync(0xffffffffu, eq));
    }
    int total;
    // lane 0 carries the warp's count: exclusive prefix over the warps
    int eq_before = block_scan_exclusive(lane == 0 ? eq_count : 0, scan, total);
    eq_before = __shfl_sync(0xffffffffu, eq_before, 0);
    int holes = 0, movers = 0;
    for (int i = w0; i < w1; ++i) {
        const int t = 32 * i + lane;
        const uint32_t key = t < cand ? weight_key(w[t]) : 0u;
        const bool eq = edge > 0 && t < cand && key == thr;
        const uint32_t em = __ballot_sync(0xffffffffu, eq);
        const int rank = eq_before + __popc(em & ((1u << lane) - 1u));
        const bool take = edge > 0 && t < cand && (key > thr || (eq && rank < want));
        const uint32_t cm = __ballot_sync(0xffffffffu, take);
        eq_before += __popc(em);
        // tokens of this word below edge: holes count there, movers above it
        const int below = max(0, min(32, edge - 32 * i));
        const uint32_t bm = below == 32 ? 0xffffffffu : (1u << below) - 1u;
        if (lane == 0) {
            bits[i] = cm;
            before[i] = 0;
        }
        holes += __popc(~cm & bm);
        movers += __popc(cm & ~bm);
    }
    // holes before each word below edge, movers before each word above it (the
    // word that holds edge itself counts movers; its holes come last)
    int hb = block_scan_exclusive(lane == 0 ? holes : 0, scan, total);
    const int num_holes = total;
    int mb = block_scan_exclusive(lane == 0 ? movers : 0, scan, total);
    hb = __shfl_sync(0xffffffffu, hb, 0);
    mb = __shfl_sync(0xffffffffu, mb, 0);
    for (int i = w0; i < w1; ++i) {
        const uint32_t cm = bits[i];
        const int below = max(0, min(32, edge - 32 * i));
        const uint32_t bm = below == 32 ? 0xffffffffu : (1u << below) - 1u;
        if (lane == 0) before[i] = below == 32 ? hb : mb;
        hb += __popc(~cm & bm);
        mb += __popc(cm & ~bm);
    }
    __syncthreads();
    const int edge_word = edge / 32;
    // The i-th mover goes to the i-th hole, kListCap of them per round.
    for (int r0 = 0; r0 < num_holes; r0 += kListCap) {
        for (int i = edge_word + warp; i < words; i += kSelWarps) {
            const int below = max(0, min(32, edge - 32 * i));
            const uint32_t bm = below == 32 ? 0xffffffffu : (1u << below) - 1u;
            const uint32_t m = bits[i] & ~bm;
            const int rank = before[i] + __popc(m & ((1u << lane) - 1u)) - r0;
            if ((m >> lane & 1u) && rank >= 0 && rank < kListCap) list[rank] = 32 * i + lane;
        }
        __syncthreads();
        for (int i = warp; 32 * i < edge; i += kSelWarps) {
            const int below = min(32, edge - 32 * i);
            const uint32_t bm = below == 32 ? 0xffffffffu : (1u << below) - 1u;
            const uint32_t h = ~bits[i] & bm;
            // the word that holds edge: its holes are the last ones
            const int base = below == 32 ? before[i] : num_holes - __popc(h);
            const int rank = base + __popc(h & ((1u << lane) - 1u)) - r0;
            const int j = 32 * i + lane;
            if (h >> lane & 1u) {
                if (rank >= 0 && rank < kListCap) {
                    const int src = list[rank];
                    kept[j] = src;
                    wo[j] = w[src];  // src >= edge > j: not yet overwritten
                }
            } else if (r0 == 0 && j < edge) {
                kept[j] = j;
                if (wo != w) wo[j] = w[j];
            }
        }
        __syncthreads();
    }
    if (num_holes == 0)
        for (int j = tid; j < edge; j += kSelThreads) {
            kept[j] = j;
            if (wo != w) wo[j] = w[j];
        }
    __syncthreads();
    // recent tokens, ascending (in place, a chunk is read before it is written)
    for (int j0 = 0; j0 < p.recent; j0 += kSelThreads) {
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
    for (int j = p.budget + tid; j < p.weights_stride; j += kSelThreads) wo[j] = 0.f;
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
__global__ void __launch_bounds__(kFillWarps * 32)
evict_fill_kernel(const EvictParams p) {
    const int kh = blockIdx.y, s = blockIdx.z;
    const int lane = threadIdx.x & 31;
    const int edge = p.budget - p.recent;
    const int n = clamp_len(__ldg(p.context_lens + s), p.max_context_len, false);
    if (n <= p.budget) return;
    const int j = (blockIdx.x * kFillWarps + (threadIdx.x >> 5)) * 32 + lane;
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

// The recent rows: slot edge + i gets position n - recent + i. One CTA per
// (K or V, kv head, sequence) goes through them in ascending chunks that are read whole
// before any is written: a slot written by a chunk is the source of no later one.
constexpr int kShiftThreads = 512;
constexpr int kShiftU = 8;
__global__ void __launch_bounds__(kShiftThreads)
evict_shift_kernel(const EvictParams p) {
    const int kh = blockIdx.y, s = blockIdx.z;
    const int n = clamp_len(__ldg(p.context_lens + s), p.max_context_len, false);
    if (n <= p.budget) return;
    const int edge = p.budget - p.recent;
    uint4* cache = blockIdx.x ? p.v_cache : p.k_cache;
    const int c = threadIdx.x % p.row_vecs, r0 = threadIdx.x / p.row_vecs;
    const int rows = kShiftThreads / p.row_vecs;  // per pass
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

// ---------------------------------------------------------------------------
// the weights of a decode step
// ---------------------------------------------------------------------------
// weights[s][kh][t] += sum over the heads of the group of 2^(score - lse), with
// lse the log-sum-exp (log2 units) of the head's partitions: the decode kernel left
// every score (log2 units) and each partition's running max and sum.
constexpr int kAddThreads = 256;
constexpr int kAddTokens = 4;  // per thread
constexpr int kMaxHeads = 32;  // of a group, per round

__global__ void __launch_bounds__(kAddThreads)
add_weights_kernel(const AddWeightsParams p) {
    __shared__ float lse[kMaxHeads];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int kh = blockIdx.y, s = blockIdx.z;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int n = clamp_len(__ldg(p.context_lens + s), p.max_context_len, false);
    const int t0 = blockIdx.x * kAddThreads * kAddTokens;
    if (t0 >= n) return;
    const int group = p.num_heads / p.num_kv_heads;
    const int parts = (n + p.partition_size - 1) / p.partition_size;
    float* w = p.weights + ((int64_t)s * p.num_kv_heads + kh) * p.weights_stride;
    float acc[kAddTokens];
#pragma unroll
    for (int u = 0; u < kAddTokens; ++u) acc[u] = 0.f;
    for (int h0 = 0; h0 < group; h0 += kMaxHeads) {
        const int heads = min(kMaxHeads, group - h0);
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
        const float* sc = p.scores + ((int64_t)s * p.num_heads + kh * group + h0) * p.score_stride;
        for (int h = 0; h < heads; ++h) {
            const float e = lse[h];
#pragma unroll
            for (int u = 0; u < kAddTokens; ++u) {
                const int t = t0 + u * kAddThreads + threadIdx.x;
                if (t < n) acc[u] += exp2f(__ldg(sc + (int64_t)h * p.score_stride + t) - e);
            }
        }
        __syncthreads();
    }
#pragma unroll
    for (int u = 0; u < kAddTokens; ++u) {
        const int t = t0 + u * kAddThreads + threadIdx.x;
        if (t < n) w[t] += acc[u];
    }
}

}  // namespace

static size_t evict_smem_bytes(int max_context_len) {
    const size_t words = ((size_t)max_context_len + 31) / 32;
    return 4 * (2 * words + kListCap + kBins + kSelWarps + 4);
}

int evict_max_context() { return (int)((227 * 1024 - evict_smem_bytes(0)) / 8 * 32); }

cudaError_t launch_evict(const EvictParams& p, cudaStream_t stream) {
    const size_t smem = evict_smem_bytes(p.max_context_len);
    cudaError_t e = cudaFuncSetAttribute(evict_select_kernel,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    const dim3 rows((unsigned)p.num_kv_heads, (unsigned)p.num_seqs);
    evict_select_kernel<<<rows, kSelThreads, smem, stream>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    if (p.max_context_len <= p.budget) return cudaSuccess;  // no sequence is over its budget
    const int edge = p.budget - p.recent;
    if (edge > 0) {
        const unsigned chunks = (unsigned)((edge + kFillWarps * 32 - 1) / (kFillWarps * 32));
        evict_fill_kernel<<<dim3(chunks, rows.x, rows.y), kFillWarps * 32, 0, stream>>>(p);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    if (p.recent > 0) {
        evict_shift_kernel<<<dim3(2, rows.x, rows.y), kShiftThreads, 0, stream>>>(p);
        e = cudaGetLastError();
    }
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
