// pa_prefill.cu — prompt attention and prompt weights on the 5th-generation tensor
// cores (bf16).
//
// out[i] = softmax over t <= i of (scale q_i . k_t) applied to v, per prompt and head
// ("PagedAttention原理详解…", § 显存消耗的三大来源, for every query of the prompt at
// once), in one pass over the keys with the running maximum and sum of the
// softmax (Milakov and Gimelshein, "Online normalizer calculation for softmax").
//
// Attention. A row block is 128 consecutive tokens of one prompt under one head. The
// row blocks of a kv head are counted tile by tile, the heads of its group inside
// a tile; an item is two consecutive ones, so that both read the same K and V
// tiles (two heads of one tile, or two tiles of one head) and one's products run while the
// other's softmax does. Roles of a CTA:
//   warp 16: issues S_b = Q_b K^T (128 x 128, K = head_dim, A and B in shared memory)
//     and O_b += P_b V (A = P from TMEM, B = V read MN-major), completions by commit;
//   warp 17: loads Q and the ring of K and V tiles by TMA, and finds the next item;
//   warps 0..7 and 8..15: the softmax of row blocks 0 and 1, two threads per row (of warps
//     that share TMEM lanes), which exchange the row's maximum in every tile and its sum at
//     the end. The scores are read twice (for the maximum, then for the weights): kept in
//     registers, they left the rest of the loop to local memory, and with shared
//     memory taking all of the L1 cache each of those loads is an L2 access. P (bf16)
//     overwrites the first half of each thread's scores in TMEM, or has its own columns;
//   warps 18 and 19: on the tiles that the diagonal crosses, zero the elements of V that are
//     not finite, and the rows behind the prompt, before the tensor core reads
//     them: a masked weight is 0, and 0 x infinity would not be. The epilogue adds the
//     elements so taken out to the rows that attend to them.
// The weights are 2^(score - m) with m a reference that moves (a published idea) only when a row's
// maximum exceeds it by more than 2^kRescaleLog2 (numerator and denominator share it, so
// the result is the exact softmax); O is then rescaled in TMEM by its row's own
// threads. What a row does depends on its own scores alone. P is rounded to bf16 for
// the product (an operand of the tensor core); its sum takes the fp32 weights.
//
// Weights. weights[t] = sum over heads of the group and queries i >= t of
// 2^(score - lse_i): S^T = K Q^T with the keys as rows, so that a key's sum stays in one
// thread (two: one per half of the queries' columns, four per SM sub-partition, which hide
// more of each other's waits than two: 873 -> 665 us at 8K under 64/8 heads); query tiles
// stream past two key tiles, so that each is read from L2 half as often.
//
// Both kernels stay on their SM and take item after item: the grid is one CTA per item, and a
// running CTA cancels the launch of one that has not started and does its work
// (cluster launch control), so that the next item's tiles load while this one's
// epilogue runs, and long and short prompts balance without a counter in memory.
//
// Bounds of the attention: the tensor cores (64 cycles per 128 x 128 x 16 product: 1024 per
// key tile and row block at head_dim 128), the exponential unit (16 per cycle and SM:
// 1024 cycles per 128 x 128 weights) and, in between, the chain S -> softmax -> P V ->
// next S of a row block (about 1500 + 512 + 512 + 380 cycles), which the other row
// block only partly covers. 16K tokens of 64/8 heads, tensor pipe 55% active at 4K: 3.56 ms =
// 1235 TFLOP/s in a short row of launches, 4.0 ms = 1100 in a long one, whose clock
// the power cap holds lower. A product of 64 keys costs the cycles of one of 128, so smaller
// steps with two score buffers were slower (4.4 ms against 4.0 at the time).
// Bound of the weights: the exponential unit (71% active at 4K); 8K tokens of 64/8 heads 0.69 to
// 0.74 ms.
#include <math.h>

#include <algorithm>

#include "pa_device.cuh"
#include "pa_internal.h"
#include "pa_prefill_tile.cuh"
#include "pa_tma.cuh"
#include "pa_umma.cuh"

namespace pa {

static __device__ unsigned int s_status_prefill;

namespace {

constexpr int kBlk = 128;                 // tokens of a tile
constexpr int kHalfBytes = kBlk * 128;    // 64 of a tile's head_dim elements: 128 rows x 128 bytes
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kRescaleLog2 = 8.f;

// Bounded wait; gives up at once when another role already gave up.
__device__ __forceinline__ bool wait_or_dead(volatile int* dead, uint32_t bar, uint32_t parity,
                                             uint64_t limit_ns = kWaitLimitNs) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = global_timer_ns();
    for (;;) {
#pragma unroll 1
        for (int i = 0; i < 64; ++i)
            if (mbar_try_wait(bar, parity)) return true;
        if (*dead != 0) return false;
        if (global_timer_ns() - t0 > limit_ns) {
            atomicOr(&s_status_prefill, kStatusTimeout);
            *dead = 1;
            return false;
        }
    }
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

// 2^x of two values, x <= 128, on the fp32 units instead of the exponential unit: with n =
// round(x) (by adding 1.5 x 2^23) and f = x - n in [-1/2, 1/2], 2^f by its degree-5
// polynomial of least relative error (Remez exchange; below 2.4e-7 in fp32 arithmetic),
// times 2^n made of its exponent bits. x <= -127 gives 0, NaN stays NaN.
__device__ __forceinline__ float2 exp2_poly(float2 x) {
    const float2 big = make_float2(12582912.f, 12582912.f);
    asm("max.NaN.f32 %0, %0, 0fC2FE0000;" : "+f"(x.x));  // -127
    asm("max.NaN.f32 %0, %0, 0fC2FE0000;" : "+f"(x.y));
    const float2 t = add2(x, big);
    const float2 f = add2(x, sub2(big, t));
    auto both = [](float c) { return make_float2(c, c); };
    float2 y = fma2(f, both(0.0013276472454890609f), both(0.009675540961325169f));
    y = fma2(f, y, both(0.05550713092088699f));
    y = fma2(f, y, both(0.24022120237350464f));
    y = fma2(f, y, both(0.6931469440460205f));
    y = fma2(f, y, both(1.0000001192092896f));
    return mul2(y, make_float2(__int_as_float((__float_as_int(t.x) << 23) + 0x3f800000),
                               __int_as_float((__float_as_int(t.y) << 23) + 0x3f800000)));
}

// 2^x of the pair with index c of a row: one of every eight pairs by polynomial, the others
// by the exponential unit (none, 1, 2 and 3 of eight measured: 8K weights 703, 661, 664
// and 688 us, ragged prompts of head_dim 64 122, 117, 117 and 118 us).
__device__ __forceinline__ float2 exp2_pair(float2 x, int c) {
    if (c % 8 == 7) return exp2_poly(x);  // (compile time)
    return make_float2(ex2(x.x), ex2(x.y));
}

__device__ __forceinline__ void sts128(uint32_t addr, uint4 x) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};"
                 :: "r"(addr), "r"(x.x), "r"(x.y), "r"(x.z), "r"(x.w) : "memory");
}
// Bits 15 and 31: whether the lower and upper bf16 of a word are infinite or NaN (an exponent
// of all ones, to which one more unit carries into the sign's place).
__device__ __forceinline__ uint32_t odd_bf16(uint32_t w) {
    return ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
}

// One tile of a packed tensor into shared memory, half by half.
template <int D>
__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap* map, int head, int token,
                                          uint32_t bar) {
    mbar_arrive_expect_tx(bar, D / 64 * kHalfBytes);
#pragma unroll
    for (int h = 0; h < D / 64; ++h) tma_load_3d(dst + h * kHalfBytes, map, 64 * h, head, token, bar);
}

// Descriptor words of a tile: K-major (head_dim contiguous, as A or B of a product over
// head_dim), and as V, whose product runs over the rows.
__device__ __forceinline__ uint32_t rows_lo(uint32_t tile) { return umma_desc_lo(tile, 16); }
__device__ __forceinline__ uint32_t v_lo(uint32_t tile) { return umma_desc_lo(tile, kHalfBytes); }
constexpr uint32_t kDescHi = umma_desc_hi(1024);

// S = A B^T over head_dim, A and B tiles in shared memory (their rows_lo).
template <int D>
__device__ __forceinline__ void issue_qk(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc) {
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
        const uint32_t at = ((k >> 2) * kHalfBytes + (k & 3) * 32) >> 4;
        umma_ss_words(d, a + at, b + at, kDescHi, idesc, k > 0);
    }
}

// ---------------------------------------------------------------------------
// items
// ---------------------------------------------------------------------------
// What a CTA works on next: one (prompt, kv head, tile), decoded by one of its warps.
struct Item {
    int seq;    // kNothing: the index lies behind the last one; kEnd: no more
    int start, len, tile, kh;
};
constexpr int kNothing = -1, kEnd = -2;

// Shared-memory places of the hand-over of items: four slots in turn.
constexpr int kSlots = 4;
// The walker runs ahead of the others and may wait for a slot as long as an item takes (weights
// of 866 heads and 113K queries: over a second). A role that cannot go on gives up after
// kWaitLimitNs and ends this wait with it.
constexpr uint64_t kItemLimitNs = 100 * kWaitLimitNs;
struct ItemBars {
    uint32_t full, empty, answer;  // [kSlots], [kSlots], and of the launch control's answer
    volatile int* slots;           // [kSlots][8]
    uint32_t response;             // 16 bytes
};
constexpr int kItemBars = 2 * kSlots + 1, kItemBytes = 32 * kSlots + 16;

// Ask for the launch of a pending CTA to be cancelled; the answer (16 bytes) completes on bar.
__device__ __forceinline__ void ask_next(uint32_t response, uint32_t bar) {
    mbar_arrive_expect_tx(bar, 16);
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];"
                 :: "r"(response), "r"(bar) : "memory");
}
// The cancelled CTA's index, or -1: none was left.
__device__ __forceinline__ int answer_index(uint32_t response) {
    uint32_t yes, x;
    asm volatile("{\n\t.reg .b128 h;\n\t.reg .pred p;\n\t.reg .b32 y, z, w;\n\tld.shared.b128 h, [%2];\n\t"
                 "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\tmov.u32 %1, 0;\n\t"
                 "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%1, y, z, w}, h;\n\t}"
                 : "=r"(yes), "=r"(x) : "r"(response) : "memory");
    return yes ? (int)x : -1;
}

// One warp: hands over the CTA's first item (index = tile * heads + kv head), calls load(item) (false: gave up), and goes on
// with the next.
template <typename Tiles, typename Load>
__device__ __forceinline__ void walk_items(const PrefillParams& p, int heads, const ItemBars& ib, volatile int* dead,
                                           bool reversed, Tiles tiles, Load load) {
    const int lane = threadIdx.x & 31;
    int id = blockIdx.x;
    PromptWalk walk;
    for (int n = 0;; ++n) {
        Item it;
        it.seq = kEnd;
        if (id >= 0) {
            it.kh = id % heads;
            const PromptTile u = walk.find(p, tiles, id / heads, reversed);
            it.seq = u.seq;
            it.start = u.start;
            it.len = u.len;
            it.tile = u.tile;
            if (walk.bad) {
                atomicOr(&s_status_prefill, kStatusBadIndex);
                walk.bad = false;
            }
        }
        const int slot = n % kSlots;
        if (n >= kSlots &&
            !__all_sync(0xffffffffu, wait_or_dead(dead, ib.empty + 8 * slot, ((n / kSlots) & 1) ^ 1,
                                                      kItemLimitNs)))
            return;
        if (lane == 0) {
            volatile int* d = ib.slots + 8 * slot;
            d[0] = it.seq;
            if (it.seq >= 0) {
                d[1] = it.start;
                d[2] = it.len;
                d[3] = it.tile;
                d[4] = it.kh;
            }
            mbar_arrive(ib.full + 8 * slot);
            if (id >= 0) ask_next(ib.response, ib.answer);
        }
        __syncwarp();
        if (id < 0) return;
        const bool ok = it.seq < 0 || __all_sync(0xffffffffu, load(it));
        // (also after a give-up: the answer is on its way into shared memory)
        if (!__all_sync(0xffffffffu, mbar_wait_bounded(ib.answer, n & 1))) {
            if (lane == 0) atomicOr(&s_status_prefill, kStatusTimeout);
            *dead = 1;
            return;
        }
        if (!ok) return;
        id = answer_index(ib.response);
        __syncwarp();
        fence_async_smem();  // the answer is read before the next one is written
    }
}

// The other warps: the n-th item; seq = kEnd after the last or a give-up. Its slot holds
// until leave_item.
__device__ __forceinline__ Item peek_item(const ItemBars& ib, int n) {
    const volatile int* d = ib.slots + 8 * (n % kSlots);
    Item it;
    it.seq = d[0];
    it.start = d[1];
    it.len = d[2];
    it.tile = d[3];
    it.kh = d[4];
    return it;
}
__device__ __forceinline__ bool wait_item(const ItemBars& ib, volatile int* dead, int n) {
    return __all_sync(0xffffffffu, wait_or_dead(dead, ib.full + 8 * (n % kSlots), (n / kSlots) & 1));
}
__device__ __forceinline__ void leave_item(const ItemBars& ib, int n) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(ib.empty + 8 * (n % kSlots));
}
__device__ __forceinline__ Item take_item(const ItemBars& ib, volatile int* dead, int n) {
    Item it;
    it.seq = kEnd;
    if (!wait_item(ib, dead, n)) return it;
    it = peek_item(ib, n);
    leave_item(ib, n);
    return it;
}

__device__ __forceinline__ ItemBars item_bars(uint32_t bars, uint8_t* bytes, int takers) {
    ItemBars ib;
    ib.full = bars;
    ib.empty = bars + 8 * kSlots;
    ib.answer = bars + 16 * kSlots;
    ib.response = smem_u32(bytes);
    ib.slots = reinterpret_cast<volatile int*>(bytes + 16);
    if (threadIdx.x == 0) {
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(ib.full + 8 * i, 1);
            mbar_init(ib.empty + 8 * i, takers);
        }
        mbar_init(ib.answer, 1);
    }
    return ib;
}

// A place in a ring of S stages: stage and the parity of its present use.
template <int S>
struct Place {
    int st = 0;
    uint32_t par = 0;
    __device__ __forceinline__ Place next() const {
        Place r = *this;
        if (++r.st == S) r.st = 0, r.par ^= 1;
        return r;
    }
};

// ---------------------------------------------------------------------------
// attention
// ---------------------------------------------------------------------------
constexpr int kCleaners = 2;              // warps
constexpr int kSoftWarps = 16;            // eight per row block, then products, loads, cleaners
constexpr int kAttnThreads = 32 * (kSoftWarps + 2 + kCleaners);
constexpr int kSoftRegs = 104, kOtherRegs = 64;   // of a thread, of the 640 x 96 launched
constexpr uint32_t kAttnTmemCols = 512;   // S_0, S_1 (128 columns each), O_0, O_1

template <int D>
struct AttnCfg {
    static constexpr int kTile = D / 64 * kHalfBytes;
    static constexpr int kStages = D == 128 ? 5 : 8;          // K and V tiles, alternating
    static constexpr int kRing = 2 * kTile;                   // after the two Q tiles
    // a row's maxima, at the end its sums, [2 row blocks][2 halves][128]
    static constexpr int kXch = kRing + kStages * kTile;
    static constexpr int kItems = kXch + 4 * kBlk * 4;
    static constexpr int kBars = kItems + kItemBytes;
    // q 2, its release 2, full S, empty S, s 2, p 2, pv 2, o 2, note 2, edge 2, clean 2, fin
    static constexpr int kNumBars = 2 * kStages + 19 + kItemBars;
    static constexpr int kSmem = kBars + 8 * kNumBars + 32;   // + TMEM slot, dead, taken 4, noted 2
    static constexpr uint32_t kColO = 256;
    // At head_dim 64 TMEM has room for P beside S (at 128 P overwrites its thread's scores), and
    // the next scores need not wait for P V: their product goes first.
    static constexpr bool kOwnP = D == 64;
    __host__ __device__ static constexpr uint32_t col_p(int b, int half) {
        return kOwnP ? 384 + 64 * b + 32 * half : kBlk * b + 64 * half;
    }
    static constexpr uint32_t kIdescQK = umma_idesc(kBlk, kBlk, false);
    static constexpr uint32_t kIdescPV = umma_idesc(kBlk, D, true);
    static_assert(kSmem <= 227 * 1024, "shared memory of a CTA");
};
constexpr uint32_t kNegateA = 1u << 13;   // of the instruction descriptor

// Row blocks 2 tile and 2 tile + 1 of a kv head (the last one of an odd count is alone): how
// many, and the token tiles of both, which are also their last key tiles.
struct Blocks {
    int nb, tile0, tile1;
    __device__ __forceinline__ Blocks(const Item& it, int group) {
        nb = min(2, (it.len + kBlk - 1) / kBlk * group - 2 * it.tile);
        tile0 = 2 * it.tile / group;
        tile1 = (2 * it.tile + nb - 1) / group;
    }
    __device__ __forceinline__ int last(int b) const { return b ? tile1 : tile0; }
};

// Whether `pred` holds for any thread of the two warps that share rows (barrier `id`).
__device__ __forceinline__ bool pair_any(int id, bool pred) {
    uint32_t r;
    asm volatile("{\n .reg .pred p, q;\n setp.ne.u32 q, %2, 0;\n"
                 " bar.red.or.pred p, %1, 64, q;\n selp.u32 %0, 1, 0, p;\n}"
                 : "=r"(r) : "r"(id), "r"((uint32_t)pred) : "memory");
    return r != 0;
}

// A thread's half of a row's scores (64, at ts), 32 at a time. kDiagonal: of the tile that the
// diagonal crosses, 32 x 32 of a warp's scores lie before the diagonal (side + g < 0), on it or
// (> 0) behind it, all masked. (The other tiles' loops are free of the tests: with
// them in the loops 16K tokens took 3% longer.)
template <bool kDiagonal>
__device__ __forceinline__ float row_maximum(uint32_t ts, int side) {
    const int lane = threadIdx.x & 31;
    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
    for (int g = 0; g < 2; ++g) {
        if (kDiagonal && side + g > 0) continue;
        uint32_t s[32];
        tmem_ld32(ts + 32 * g, s);
        if (kDiagonal && side + g == 0) {
#pragma unroll
            for (int c = 0; c < 32; ++c)
                if (c > lane) s[c] = 0xff800000u;
        }
#pragma unroll
        for (int c = 0; c < 32; c += 8)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                mx[i] = fmaxf(fmaxf(mx[i], __uint_as_float(s[c + i])), __uint_as_float(s[c + 4 + i]));
    }
    return fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
}

// Their weights 2^(s sl - ms), bf16, to TMEM at tp (after `ready`), and their fp32 sum.
template <bool kDiagonal, typename Ready>
__device__ __forceinline__ float put_weights(uint32_t ts, uint32_t tp, int side, float sl, float ms, Ready ready) {
    const int lane = threadIdx.x & 31;
    const float2 sl2 = make_float2(sl, sl), ms2 = make_float2(-ms, -ms);
    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
    for (int g = 0; g < 2; ++g) {
        uint32_t w[16];
        if (kDiagonal && side + g > 0) {
#pragma unroll
            for (int c = 0; c < 16; ++c) w[c] = 0u;
        } else {
            uint32_t s[32];
            tmem_ld32(ts + 32 * g, s);
            if (kDiagonal && side + g == 0) {
#pragma unroll
                for (int c = 0; c < 32; ++c)
                    if (c > lane) s[c] = 0xff800000u;
            }
#pragma unroll
            for (int c = 0; c < 16; ++c) {
                float2 x = fma2(make_float2(__uint_as_float(s[2 * c]), __uint_as_float(s[2 * c + 1])), sl2, ms2);
                x = exp2_pair(x, c);
                w[c] = bf16x2(x.x, x.y);
                sum[c & 1] = add2(sum[c & 1], x);
            }
        }
        if (g == 0) ready();
        tmem_st16_issue(tp + 16 * g, w);
    }
    tmem_wait_st();
    return (sum[0].x + sum[1].x) + (sum[0].y + sum[1].y);
}

template <int D>
__global__ void __launch_bounds__(kAttnThreads, 1)
prefill_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
               const __grid_constant__ CUtensorMap vmap, const PrefillParams p) {
    using C = AttnCfg<D>;
    constexpr int S_ = C::kStages;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int group = p.num_heads / p.num_kv_heads;
    const uint32_t raw = smem_u32(smem);
    if (raw & 1023u) {
        if (threadIdx.x == 0) atomicOr(&s_status_prefill, kStatusSmemAlign);
        return;
    }
    const uint32_t bars = smem_u32(smem + C::kBars);
    const uint32_t b_q = bars, b_qfree = b_q + 16, b_full = b_qfree + 16, b_empty = b_full + 8 * S_,
                   b_s = b_empty + 8 * S_, b_p = b_s + 16, b_pv = b_p + 16, b_o = b_pv + 16, b_note = b_o + 16,
                   b_edge = b_note + 16, b_clean = b_edge + 16, b_fin = b_clean + 16;
    const ItemBars ib = item_bars(b_fin + 8, smem + C::kItems, kSoftWarps + 1 + kCleaners);
    uint32_t* tslot = reinterpret_cast<uint32_t*>(smem + C::kBars + 8 * C::kNumBars);
    volatile int* dead = reinterpret_cast<volatile int*>(tslot + 1);
    volatile int* taken = dead + 1;   // [2 edge slots][cleaners]: elements were zeroed
    volatile int* noted = taken + 2 * kCleaners;   // [2] of a row block: in one of its item's edge tiles
    const uint32_t qbuf = raw, ring = raw + C::kRing;
    if (threadIdx.x == 0) {
        for (int i = 0; i < S_; ++i) {
            mbar_init(b_full + 8 * i, 1);
            mbar_init(b_empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(b_q + 8 * i, 1);
            mbar_init(b_qfree + 8 * i, 1);
            mbar_init(b_s + 8 * i, 1);
            mbar_init(b_p + 8 * i, kSoftWarps / 2);
            mbar_init(b_pv + 8 * i, 1);
            mbar_init(b_o + 8 * i, 1);
            mbar_init(b_note + 8 * i, 1);
            mbar_init(b_edge + 8 * i, 1);
            mbar_init(b_clean + 8 * i, kCleaners);
        }
        mbar_init(b_fin, 1);
        *dead = 0;
        fence_barrier_init();
    }
    if (warp == kSoftWarps) tmem_alloc(smem_u32(tslot), kAttnTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = *tslot;
    auto wait = [&](uint32_t bar, uint32_t parity) {
        return __all_sync(0xffffffffu, wait_or_dead(dead, bar, parity));
    };

    // The 640 threads' 96 registers, divided anew (the launch checks that there are as many).
    if (warp < kSoftWarps)
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    else
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp < kSoftWarps) {  // softmax of row block b: half a row per thread
        const int b = warp >> 3, half = (warp >> 2) & 1, row = threadIdx.x & 127;
        const int pair_id = 1 + 4 * b + (warp & 3);
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t tp = tm + lanes + C::col_p(b, half);
        const uint32_t ts = tm + lanes + kBlk * b + 64 * half, to = tm + lanes + C::kColO + D * b + D / 2 * half;
        float* xch = reinterpret_cast<float*>(smem + C::kXch) + 2 * kBlk * b + row;
        // (its sign is in the product; not 0, so that a masked -infinity stays one)
        const float sl = fmaxf(fabsf(p.scale_log2), 1e-30f);
        uint32_t par_s = 0, par_o = 0;
        bool ok = true;
        for (int n = 0; ok; ++n, leave_item(ib, n - 1)) {
            // (the two warps agree on every give-up: one would wait for the other at the barrier)
            if (pair_any(pair_id, !wait_item(ib, dead, n))) break;
            const int seq = ib.slots[8 * (n % kSlots)];
            if (seq == kEnd) break;
            if (seq < 0) continue;
            int last;      // the row block's last key tile: the one on the diagonal
            {
                const Blocks k(peek_item(ib, n), group);
                if (b >= k.nb) continue;
                last = k.last(b);
            }
            float m = -INFINITY, ms = 0.f;
            float l = 0.f;   // this thread's half of the sum
            for (int j = 0; j <= last; ++j, par_s ^= 1) {
                ok = wait(b_s + 8 * b, par_s);
                const int side = 2 * half - (warp & 3);
                float mt = -INFINITY;
                if (ok) {
                    tc_fence_after();
                    mt = j < last ? row_maximum<false>(ts, side) : row_maximum<true>(ts, side);
                    // (the other thread has read the last one: it did so before its weights,
                    // which S_b's product waited for)
                    xch[half * kBlk] = mt;
                }
                // both halves' maxima are known
                if (pair_any(pair_id, !ok)) {
                    ok = false;
                    break;
                }
                mt = fmaxf(mt, xch[(half ^ 1) * kBlk]);
                if (j == 0) {
                    m = mt;
                    ms = m == -INFINITY ? 0.f : m * sl;   // (no score above -infinity yet: weights 0)
                } else {
                    const bool move = (mt - m) * sl > kRescaleLog2;
                    if (__any_sync(0xffffffffu, move)) {
                        // O is at rest: S_b's commit came after the last PV of this row block, or
                        // that is waited for
                        if (C::kOwnP) wait(b_pv + 8 * b, par_s ^ 1);
                        tc_fence_after();
                        const float al = move ? ex2((m - mt) * sl) : 1.f;
                        if (move) {
                            m = mt;
                            ms = m * sl;
                        }
                        l *= al;
#pragma unroll 1
                        for (int c = 0; c < D / 2; c += 16) {
                            uint32_t o[16];
                            tmem_ld16(to + c, o);
#pragma unroll
                            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * al);
                            tmem_st16(to + c, o);
                        }
                    }
                }
                auto ready = [&] {
                    if (C::kOwnP) {  // the last P is no longer read (at the first: parity of no use)
                        wait(b_pv + 8 * b, par_s ^ 1);
                        tc_fence_after();
                    }
                };
                l += j < last ? put_weights<false>(ts, tp, side, sl, ms, ready)
                              : put_weights<true>(ts, tp, side, sl, ms, ready);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(b_p + 8 * b);
            }
            if (ok) ok = wait(b_o + 8 * b, par_o) && wait(b_note + 8 * b, par_o);
            par_o ^= 1;
            if (ok) xch[half * kBlk] = l;
            if (pair_any(pair_id, !ok)) break;
            tc_fence_after();
            l = xch[0] + xch[kBlk];
            const float inv = 1.f / l;
            const Item it = peek_item(ib, n);
            const Blocks k(it, group);
            const int qi = last * kBlk + row;
            const bool live = qi < it.len;
            const int head = it.kh * group + (2 * it.tile + b) % group;
            uint16_t* out = static_cast<uint16_t*>(p.out) +
                            ((int64_t)it.start * p.num_heads + head) * D + D / 2 * half;
            const int64_t out_stride = (int64_t)p.num_heads * D;
            const int row0 = qi - (lane & 3);   // the first row of this thread's four lanes
#pragma unroll 1
            for (int c = 0; c < D / 2; c += 32) {
                uint32_t o[32];
                __syncwarp();
                tmem_ld32(to + c, o);
                uint32_t w[16];
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    w[i] = bf16x2(__uint_as_float(o[2 * i]) * inv, __uint_as_float(o[2 * i + 1]) * inv);
                // a row per thread would touch a line per thread in each store: four lanes exchange
                // their 16-byte chunks, so that a store writes 64 bytes of each of eight rows
#pragma unroll
                for (int mask = 1; mask < 4; mask <<= 1) {
                    const bool up = lane & mask;
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        if ((i >> 2) & mask) continue;
                        uint32_t &lo = w[i], &hi = w[i + 4 * mask];
                        const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? lo : hi, mask);
                        if (up)
                            lo = got;
                        else
                            hi = got;
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (row0 + i < it.len)
                        st_v4(out + (row0 + i) * out_stride + c + 8 * (lane & 3),
                              make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]));
            }
            if (noted[b] != 0) {
                // elements of V taken out of the edge tiles: infinite or NaN, they add to
                // whatever the row holds
                __syncwarp();
                for (int t = k.tile0 * kBlk; live && t <= qi; ++t) {
                    const uint16_t* v = static_cast<const uint16_t*>(p.v) + (int64_t)(it.start + t) * p.v_stride +
                                        (int64_t)it.kh * D + D / 2 * half;
#pragma unroll 1
                    for (int c = 0; c < D / 2; ++c) {
                        const float x = bf16_lo(v[c]);
                        uint16_t* at = out + qi * out_stride + c;
                        if (!(fabsf(x) < INFINITY)) *at = float_to_bf16_bits(bf16_lo(*at) + x);
                    }
                }
            }
            if (live && half == 0 && p.lse != nullptr)
                p.lse[(int64_t)head * p.total_tokens + it.start + qi] = (ms + log2f(l)) * kLn2;
            __syncwarp();
            tc_fence_before();               // O is read before the next item's first PV
            named_barrier(pair_id, 64);      // and the sums before its first maxima
        }
    } else if (warp == kSoftWarps) {  // products
        // The whole warp walks the tiles (what the descriptors are made of stays warp-uniform);
        // one thread issues.
        const uint32_t idqk = C::kIdescQK | (p.scale_log2 < 0.f ? kNegateA : 0u);
        const bool one = elect_one();
        Place<S_> cur;                      // of the next K tile
        uint32_t par_q[2] = {0, 0}, par_p[2] = {0, 0};
        int edges = 0;
        bool ok = true;
        // S_b from the K tile in stage st
        auto qk = [&](int b, int st, bool last) {
            const uint32_t q_lo = rows_lo(qbuf + b * C::kTile), k_lo = rows_lo(ring + st * C::kTile);
            if (one) {
                issue_qk<D>(tm + kBlk * b, q_lo, k_lo, idqk);
                umma_commit(b_s + 8 * b);
                if (last) umma_commit(b_qfree + 8 * b);
            }
            __syncwarp();
        };
        for (int n = 0; ok; ++n) {
            const Item it = take_item(ib, dead, n);
            if (it.seq == kEnd) break;
            if (it.seq < 0) continue;
            const Blocks k(it, group);
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                if (b >= k.nb || !ok) continue;
                ok = wait(b_q + 8 * b, par_q[b]) && (b > 0 || wait(b_full + 8 * cur.st, cur.par));
                par_q[b] ^= 1;
                if (ok) qk(b, cur.st, k.last(b) == 0);
            }
            if (!ok) break;
            if (one) umma_commit(b_empty + 8 * cur.st);
            __syncwarp();
            int note = 0;
            for (int j = 0; j <= k.tile1 && ok; ++j) {
                const Place<S_> pv = cur.next(), pk = pv.next();
                bool have_v = false, have_k = false;
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    if (b >= k.nb || j > k.last(b) || !ok) continue;
                    if (!have_v) {
                        have_v = true;
                        if (j >= k.tile0) {
                            ok = wait(b_clean + 8 * (edges & 1), (edges >> 1) & 1);
                            if (ok)
                                for (int c = 0; c < kCleaners; ++c) note |= taken[(edges & 1) * kCleaners + c];
                            ++edges;
                        } else {
                            ok = wait(b_full + 8 * pv.st, pv.par);
                        }
                    }
                    if (!ok || !(ok = wait(b_p + 8 * b, par_p[b]))) continue;
                    par_p[b] ^= 1;
                    tc_fence_after();
                    const uint32_t lo = v_lo(ring + pv.st * C::kTile);
                    const bool last = j == k.last(b);
                    auto next_scores = [&] {
                        if (last) return;
                        if (!have_k && !(ok = wait(b_full + 8 * pk.st, pk.par))) return;
                        have_k = true;
                        qk(b, pk.st, j + 1 == k.last(b));
                    };
                    if (C::kOwnP) next_scores();
                    if (one) {
#pragma unroll
                        for (int i = 0; i < kBlk / 16; ++i)
                            umma_ts_words(tm + C::kColO + D * b, tm + C::col_p(b, i >> 2) + 8 * (i & 3), lo + 128 * i,
                                          kDescHi, C::kIdescPV, i > 0 || j > 0);
                        if (C::kOwnP) umma_commit(b_pv + 8 * b);
                        if (last) {
                            umma_commit(b_o + 8 * b);
                            noted[b] = note;
                            mbar_arrive(b_note + 8 * b);
                        }
                    }
                    __syncwarp();
                    if (!C::kOwnP) next_scores();
                }
                if (ok && one) {
                    umma_commit(b_empty + 8 * pv.st);
                    if (have_k) umma_commit(b_empty + 8 * pk.st);
                }
                __syncwarp();
                cur = pk;
            }
        }
        // every product issued here is complete before TMEM is freed
        if (one) umma_commit(b_fin);
        __syncwarp();
        if (!mbar_wait_bounded(b_fin, 0)) atomicOr(&s_status_prefill, kStatusTimeout);
    } else if (warp == kSoftWarps + 1) {  // loads
        if (lane == 0) {
            prefetch_tensormap(&qmap);
            prefetch_tensormap(&kmap);
            prefetch_tensormap(&vmap);
        }
        Place<S_> at;
        int loaded = 0;                    // tiles of the ring
        int used_q[2] = {0, 0}, edges = 0, edge1 = 0, edge2 = 0;   // the last two edge tiles' places
        walk_items(
            p, p.num_kv_heads, ib, dead, true, [group](int len) { return ((len + kBlk - 1) / kBlk * group + 1) / 2; },
            [&](const Item& it) {
                bool ok = true;
                if (lane == 0) {
                    const Blocks k(it, group);
                    auto load_q = [&](int b) {
                        if (used_q[b] > 0 && !wait_or_dead(dead, b_qfree + 8 * b, (used_q[b] - 1) & 1)) return false;
                        ++used_q[b];
                        load_tile<D>(qbuf + b * C::kTile, &qmap, it.kh * group + (2 * it.tile + b) % group,
                                     it.start + k.last(b) * kBlk, b_q + 8 * b);
                        return true;
                    };
                    // K (even) or V (odd) of key tile i / 2
                    for (int i = 0; i < 2 * (k.tile1 + 1) && ok; ++i, ++loaded, at = at.next()) {
                        if (loaded >= S_ && !(ok = wait_or_dead(dead, b_empty + 8 * at.st, at.par ^ 1))) break;
                        if (i == 0 && !(ok = load_q(0))) break;
                        const int j = i >> 1;
                        const bool edge = (i & 1) && j >= k.tile0;
                        if (edge) {
                            // the tile that used this edge slot before has been released, so
                            // nobody still waits for that use's phases
                            if (edges >= 2 && edge2 + S_ > loaded &&
                                !(ok = wait_or_dead(dead, b_empty + 8 * (edge2 % S_), (edge2 / S_) & 1)))
                                break;
                        }
                        if (loaded != p.test_skip_position)
                            load_tile<D>(ring + at.st * C::kTile, i & 1 ? &vmap : &kmap, it.kh,
                                         it.start + j * kBlk, b_full + 8 * at.st);
                        if (edge) {
                            mbar_arrive(b_edge + 8 * (edges & 1));
                            edge2 = edge1;
                            edge1 = loaded;
                            ++edges;
                        }
                        if (i == 0 && k.nb == 2) ok = load_q(1);
                    }
                }
                __syncwarp();
                return ok;
            });
        if (lane == 0 && *dead != 0) {  // given up: the loads in flight land before the CTA ends
            bool landed = true;
            for (int b = 0; b < 2; ++b)
                if (used_q[b] > 0) landed &= mbar_wait_bounded(b_q + 8 * b, (used_q[b] - 1) & 1);
            for (int i = max(0, loaded - S_); i < loaded; ++i)
                landed &= mbar_wait_bounded(b_full + 8 * (i % S_), (i / S_) & 1);
            if (!landed) atomicOr(&s_status_prefill, kStatusTimeout);
        }
    } else {  // cleaners
        const int t = threadIdx.x - 32 * (kSoftWarps + 2);
        Place<S_> at;
        int edges = 0;
        bool ok = true;
        for (int n = 0; ok; ++n) {
            const Item it = take_item(ib, dead, n);
            if (it.seq == kEnd) break;
            if (it.seq < 0) continue;
            const Blocks k(it, group);
            for (int j = 0; j <= k.tile1 && ok; ++j) {
                at = at.next();  // V of key tile j
                if (j >= k.tile0) {
                    const int slot = edges & 1;
                    // the load is under way (so `full` is in its phase), then landed
                    ok = wait(b_edge + 8 * slot, (edges >> 1) & 1) && wait(b_full + 8 * at.st, at.par);
                    ++edges;
                    if (!ok) break;
                    const uint32_t buf = ring + at.st * C::kTile;
                    const int rows = it.len - j * kBlk;  // of the prompt
                    constexpr int kChunks = D / 64 * kBlk * 8 / (32 * kCleaners);   // per thread
                    uint32_t found = 0;
#pragma unroll 8
                    for (int i = 0; i < kChunks; ++i) {
                        const int c = t + 32 * kCleaners * i;  // (a row's eight chunks, in whatever order)
                        const int r = (c >> 3) & (kBlk - 1);
                        const uint4 x = lds128(buf + 16 * c);
                        if (r >= rows)
                            sts128(buf + 16 * c, make_uint4(0u, 0u, 0u, 0u));
                        else
                            found |= odd_bf16(x.x) | odd_bf16(x.y) | odd_bf16(x.z) | odd_bf16(x.w);
                    }
                    if (found) {  // take the elements out of this thread's chunks
                        for (int i = 0; i < kChunks; ++i) {
                            const int c = t + 32 * kCleaners * i;
                            uint4 x = lds128(buf + 16 * c);
                            uint32_t* w = &x.x;
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const uint32_t odd = odd_bf16(w[e]);
                                if (odd & 0x8000u) w[e] &= 0xffff0000u;
                                if (odd & 0x80000000u) w[e] &= 0x0000ffffu;
                            }
                            sts128(buf + 16 * c, x);
                        }
                    }
                    const bool any = __any_sync(0xffffffffu, found != 0);
                    if (lane == 0) taken[slot * kCleaners + (t >> 5)] = any;
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(b_clean + 8 * slot);
                }
                at = at.next();
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kSoftWarps) tmem_dealloc(tm, kAttnTmemCols);
}

// ---------------------------------------------------------------------------
// weights
// ---------------------------------------------------------------------------
constexpr int kSumWarps = 16;             // eight per key tile, then products, loads, items
constexpr int kWThreads = 32 * (kSumWarps + 3);
constexpr uint32_t kWTmemCols = 512;      // S^T of two key tiles, two buffers each

template <int D>
struct WeightsCfg {
    static constexpr int kTile = D / 64 * kHalfBytes;
    static constexpr int kStages = 3;                         // query tiles with their log-sum-exps
    static constexpr int kRing = 4 * kTile;                   // after two pairs of key tiles
    static constexpr int kLse = kRing + kStages * kTile;      // [stage][128] floats
    static constexpr int kXch = kLse + kStages * kBlk * 4;    // [2 key tiles][128] sums of a half
    static constexpr int kItems = kXch + 2 * kBlk * 4;
    static constexpr int kBars = kItems + kItemBytes;
    // k 2, its release 2, full S, empty S, s 2 x 2, its release 2 x 2, fin
    static constexpr int kNumBars = 4 + 2 * kStages + 8 + 1 + kItemBars;
    static constexpr int kSmem = kBars + 8 * kNumBars + 8;    // + TMEM slot, dead
    static_assert(kSmem <= 227 * 1024, "shared memory of a CTA");
};

// An item's queries: tiles of 128 from the first that counts for its first key tile.
struct Queries {
    int len, key0, first, tiles;
    __device__ __forceinline__ Queries(const Item& it, int last_queries) {
        len = it.len;
        key0 = 2 * it.tile * kBlk;
        first = max(key0, last_queries > 0 ? len - last_queries : 0);
        tiles = (len - first + kBlk - 1) / kBlk;
    }
    __device__ __forceinline__ int q0(int qt) const { return first + qt * kBlk; }
    __device__ __forceinline__ bool exists(int w) const { return key0 + w * kBlk < len; }
    // whether any query of tile qt sees a key of key tile w
    __device__ __forceinline__ bool meets(int w, int qt) const {
        return exists(w) && q0(qt) + kBlk > key0 + w * kBlk;
    }
};

// The heads of the group that an item takes: all, or (item kv heads 2 kh and 2 kh + 1) a half.
struct Heads {
    int first, last;
    bool split;
    __device__ __forceinline__ Heads(Item& it, const PrefillParams& p) {
        const int group = p.num_heads / p.num_kv_heads;
        split = p.split_heads != 0;
        first = split && (it.kh & 1) ? group / 2 : 0;
        last = split && !(it.kh & 1) ? group / 2 : group;
        if (split) it.kh >>= 1;
    }
};

template <int D>
__global__ void __launch_bounds__(kWThreads, 1)
prefill_weights_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                       const PrefillParams p) {
    using C = WeightsCfg<D>;
    constexpr int S_ = C::kStages;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t raw = smem_u32(smem);
    if (raw & 1023u) {
        if (threadIdx.x == 0) atomicOr(&s_status_prefill, kStatusSmemAlign);
        return;
    }
    const uint32_t bars = smem_u32(smem + C::kBars);
    const uint32_t b_k = bars, b_kfree = b_k + 16, b_full = b_kfree + 16, b_empty = b_full + 8 * S_,
                   b_s = b_empty + 8 * S_, b_sfree = b_s + 32, b_fin = b_sfree + 32;
    const ItemBars ib = item_bars(b_fin + 8, smem + C::kItems, kSumWarps + 2);
    uint32_t* tslot = reinterpret_cast<uint32_t*>(smem + C::kBars + 8 * C::kNumBars);
    volatile int* dead = reinterpret_cast<volatile int*>(tslot + 1);
    float* lse = reinterpret_cast<float*>(smem + C::kLse);   // negated, in log2 units
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(b_k + 8 * i, 2);
            mbar_init(b_kfree + 8 * i, 1);
        }
        for (int i = 0; i < S_; ++i) {
            mbar_init(b_full + 8 * i, 1);
            mbar_init(b_empty + 8 * i, 1 + kSumWarps);   // the product's end, and the readers of lse
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(b_s + 8 * i, 1);
            mbar_init(b_sfree + 8 * i, kSumWarps / 2);
        }
        mbar_init(b_fin, 1);
        *dead = 0;
        fence_barrier_init();
    }
    if (warp == kSumWarps) tmem_alloc(smem_u32(tslot), kWTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = *tslot;
    auto wait = [&](uint32_t bar, uint32_t parity) {
        return __all_sync(0xffffffffu, wait_or_dead(dead, bar, parity));
    };

    if (warp < kSumWarps) {  // two threads per key of key tile w, one per half of the queries' columns
        const int w = warp >> 3, half = (warp >> 2) & 1, row = threadIdx.x & 127;
        const int pair_id = 1 + 4 * w + (warp & 3);
        const uint32_t ts = tm + ((uint32_t)(32 * (warp & 3)) << 16) + 2 * kBlk * w + 64 * half;
        float* xch = reinterpret_cast<float*>(smem + C::kXch) + kBlk * w + row;
        const float sl = fabsf(p.scale_log2);
        const float2 sl2 = make_float2(sl, sl);
        Place<S_> at;
        Place<2> buf;
        bool ok = true;
        for (int n = 0; ok; ++n) {
            Item it = take_item(ib, dead, n);
            if (pair_any(pair_id, it.seq == kEnd)) break;   // (the two warps agree, as on a give-up below)
            if (it.seq < 0) continue;
            const Queries qs(it, p.last_queries);
            const Heads hs(it, p);
            const int key = qs.key0 + w * kBlk + row;
            float sum = 0.f;
            for (int h = hs.first; h < hs.last && ok; ++h)
                for (int qt = 0; qt < qs.tiles; ++qt, at = at.next()) {
                    if (!(ok = wait(b_full + 8 * at.st, at.par))) break;
                    if (qs.meets(w, qt)) {
                        if (!(ok = wait(b_s + 16 * w + 8 * buf.st, buf.par))) break;
                        tc_fence_after();
                        const int q0 = qs.q0(qt);
                        float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                        for (int g = 0; g < 2; ++g) {
                            // of these 32 queries' columns those from the key on, within the prompt, count
                            const int col0 = 64 * half + 32 * g;
                            const int first = qs.key0 + w * kBlk + 32 * (warp & 3) - q0 - col0;   // of the warp's first key
                            const int end = qs.len - q0 - col0;
                            const float* lq = lse + at.st * kBlk + col0;
                            uint32_t s[32];
                            tmem_ld32(ts + kBlk * buf.st + 32 * g, s);
                            if (g == 1) {
                                tc_fence_before();
                                __syncwarp();
                                if (lane == 0) mbar_arrive(b_sfree + 16 * w + 8 * buf.st);
                            }
                            if (first > 31 || end <= 0) continue;   // none (of any of the warp's keys)
                            if (first + 31 <= 0 && end >= 32) {     // all
#pragma unroll
                                for (int c = 0; c < 32; c += 4) {
                                    const float4 e = *reinterpret_cast<const float4*>(lq + c);
                                    const float2 x = fma2(make_float2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])),
                                                          sl2, make_float2(e.x, e.y));
                                    const float2 y = fma2(make_float2(__uint_as_float(s[c + 2]), __uint_as_float(s[c + 3])),
                                                          sl2, make_float2(e.z, e.w));
                                    acc[0] = add2(acc[0], exp2_pair(x, c / 2));
                                    acc[1] = add2(acc[1], exp2_pair(y, c / 2 + 1));
                                }
                            } else {  // the diagonal, or the prompt's end
                                const int lo = first + lane;
#pragma unroll
                                for (int c = 0; c < 32; ++c) {
                                    const float x = ex2(fmaf(__uint_as_float(s[c]), sl, lq[c]));
                                    if (c >= lo && c < end) acc[c & 1].x += x;
                                }
                            }
                        }
                        sum += (acc[0].x + acc[0].y) + (acc[1].x + acc[1].y);
                        buf = buf.next();
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(b_empty + 8 * at.st);
                }
            if (half == 1) *xch = sum;
            if (pair_any(pair_id, !ok)) break;
            if (half == 0 && key < qs.len) {
                float* to = p.weights + ((int64_t)it.seq * p.num_kv_heads + it.kh) * p.weights_stride + key;
                sum += *xch;
                // two items add to what was zeroed: 0 + a + b is 0 + b + a, bit for bit
                if (hs.split)
                    atomicAdd(to, sum);
                else
                    *to = sum;
            }
            __syncwarp();
            named_barrier(pair_id, 64);   // the sums are read before the next ones
        }
    } else if (warp == kSumWarps) {  // products
        const uint32_t idesc = umma_idesc(kBlk, kBlk, false) | (p.scale_log2 < 0.f ? kNegateA : 0u);
        const bool one = elect_one();
        Place<2> kt, buf[2];
        Place<S_> at;
        bool ok = true;
        for (int n = 0; ok; ++n) {
            Item it = take_item(ib, dead, n);
            if (it.seq == kEnd) break;
            if (it.seq < 0) continue;
            const Queries qs(it, p.last_queries);
            const Heads hs(it, p);
            ok = wait(b_k + 8 * kt.st, kt.par);
            for (int h = hs.first; h < hs.last && ok; ++h)
                for (int qt = 0; qt < qs.tiles && ok; ++qt, at = at.next()) {
                    ok = wait(b_full + 8 * at.st, at.par);
                    const uint32_t q_lo = rows_lo(raw + C::kRing + at.st * C::kTile);
#pragma unroll
                    for (int w = 0; w < 2; ++w) {
                        if (!ok || !qs.meets(w, qt)) continue;
                        // (the first wait of a buffer is for no use yet)
                        if (!(ok = wait(b_sfree + 16 * w + 8 * buf[w].st, buf[w].par ^ 1))) continue;
                        tc_fence_after();
                        const uint32_t d = tm + 2 * kBlk * w + kBlk * buf[w].st;
                        const uint32_t k_lo = rows_lo(raw + (2 * kt.st + w) * C::kTile);
                        if (one) {
                            issue_qk<D>(d, k_lo, q_lo, idesc);
                            umma_commit(b_s + 16 * w + 8 * buf[w].st);
                        }
                        __syncwarp();
                        buf[w] = buf[w].next();
                    }
                    if (ok && one) umma_commit(b_empty + 8 * at.st);
                    __syncwarp();
                }
            if (ok && one) umma_commit(b_kfree + 8 * kt.st);
            __syncwarp();
            kt = kt.next();
        }
        if (one) umma_commit(b_fin);
        __syncwarp();
        if (!mbar_wait_bounded(b_fin, 0)) atomicOr(&s_status_prefill, kStatusTimeout);
    } else if (warp == kSumWarps + 1) {  // loads
        if (lane == 0) {
            prefetch_tensormap(&qmap);
            prefetch_tensormap(&kmap);
        }
        Place<2> kt;
        Place<S_> at;
        int keys = 0, loaded = 0;
        bool ok = true;
        for (int n = 0; ok; ++n) {
            Item it = take_item(ib, dead, n);
            if (it.seq == kEnd) break;
            if (it.seq < 0) continue;
            const Queries qs(it, p.last_queries);
            const Heads hs(it, p);
            const int head0 = it.kh * (p.num_heads / p.num_kv_heads);
            float mine[4];
            auto fetch = [&](int h, int qt) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int i = qs.q0(qt) + 32 * e + lane;
                    mine[e] = h < hs.last && i < qs.len
                                  ? -kLog2e * __ldg(p.lse + (int64_t)(head0 + h) * p.total_tokens + it.start + i)
                                  : 0.f;
                }
            };
            fetch(hs.first, 0);
            if (!(ok = wait(b_kfree + 8 * kt.st, kt.par ^ 1))) break;   // (the first two are for no use yet)
            if (lane == 0) {
                for (int w = 0; w < 2; ++w) {
                    if (qs.exists(w))
                        load_tile<D>(raw + (2 * kt.st + w) * C::kTile, &kmap, it.kh, it.start + qs.key0 + w * kBlk,
                                     b_k + 8 * kt.st);
                    else
                        mbar_arrive(b_k + 8 * kt.st);
                }
            }
            __syncwarp();
            ++keys;
            kt = kt.next();
            for (int h = hs.first; h < hs.last && ok; ++h)
                for (int qt = 0; qt < qs.tiles; ++qt, ++loaded, at = at.next()) {
                    if (!(ok = wait(b_empty + 8 * at.st, at.par ^ 1))) break;
#pragma unroll
                    for (int e = 0; e < 4; ++e) lse[at.st * kBlk + 32 * e + lane] = mine[e];
                    __syncwarp();
                    if (lane == 0 && loaded != p.test_skip_position)
                        load_tile<D>(raw + C::kRing + at.st * C::kTile, &qmap, head0 + h, it.start + qs.q0(qt),
                                     b_full + 8 * at.st);
                    __syncwarp();
                    if (qt + 1 < qs.tiles)
                        fetch(h, qt + 1);
                    else
                        fetch(h + 1, 0);
                }
        }
        if (lane == 0 && *dead != 0) {  // given up: the loads in flight land before the CTA ends
            bool landed = true;
            for (int i = max(0, keys - 2); i < keys; ++i)
                landed &= mbar_wait_bounded(b_k + 8 * (i & 1), (i >> 1) & 1);
            for (int i = max(0, loaded - S_); i < loaded; ++i)
                landed &= mbar_wait_bounded(b_full + 8 * (i % S_), (i / S_) & 1);
            if (!landed) atomicOr(&s_status_prefill, kStatusTimeout);
        }
    } else {  // items: pairs of key tiles
        walk_items(p, p.split_heads ? 2 * p.num_kv_heads : p.num_kv_heads, ib, dead, false, [](int len) { return (len + 2 * kBlk - 1) / (2 * kBlk); },
                   [](const Item&) { return true; });
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kSumWarps) tmem_dealloc(tm, kWTmemCols);
}

template <int D>
cudaError_t launch_prefill_t(const PrefillParams& p, const CUtensorMap& qmap, const CUtensorMap& kmap,
                             const CUtensorMap& vmap, cudaStream_t stream) {
    using C = AttnCfg<D>;
    cudaError_t e = cudaFuncSetAttribute(prefill_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         C::kSmem);
    if (e != cudaSuccess) return e;
    // what setmaxnreg hands out must have been launched, or its warps would wait for ever
    cudaFuncAttributes attr;
    e = cudaFuncGetAttributes(&attr, prefill_kernel<D>);
    if (e != cudaSuccess) return e;
    if (attr.numRegs * kAttnThreads < 32 * (kSoftWarps * kSoftRegs + (kAttnThreads / 32 - kSoftWarps) * kOtherRegs))
        return cudaErrorLaunchOutOfResources;
    const int64_t group = p.num_heads / p.num_kv_heads;
    // at least one more than there are pairs: its CTAs look every prompt over
    const int64_t pairs = ((int64_t)(p.total_tokens / kBlk + p.num_seqs) * group + p.num_seqs) / 2 + 1;
    if (pairs * p.num_kv_heads > INT32_MAX) return cudaErrorInvalidConfiguration;
    prefill_kernel<D><<<(unsigned)(pairs * p.num_kv_heads), kAttnThreads, C::kSmem, stream>>>(qmap, kmap, vmap, p);
    return cudaGetLastError();
}

template <int D>
cudaError_t launch_weights_t(const PrefillParams& p, const CUtensorMap& qmap, const CUtensorMap& kmap,
                             cudaStream_t stream) {
    using C = WeightsCfg<D>;
    cudaError_t e = cudaFuncSetAttribute(prefill_weights_kernel<D>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    PrefillParams q = p;
    // Half the heads per item where an item is long: with whole groups the longest of 8K under 64/8
    // heads (512 steps) outlasted the average SM's share (450). Short items (a window)
    // would only read their keys twice.
    const int64_t queries = p.last_queries > 0 ? std::min(p.last_queries, p.max_seq_len) : p.max_seq_len;
    q.split_heads = p.num_heads / p.num_kv_heads >= 2 && queries >= 2048;
    const int64_t tiles = (int64_t)(p.total_tokens / (2 * kBlk) + p.num_seqs) + 1;   // pairs
    const int64_t items = tiles * p.num_kv_heads * (q.split_heads ? 2 : 1);
    if (items > INT32_MAX) return cudaErrorInvalidConfiguration;
    prefill_weights_kernel<D><<<(unsigned)items, kWThreads, C::kSmem, stream>>>(qmap, kmap, q);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prefill(const PrefillParams& p, const CUtensorMap& qmap, const CUtensorMap& kmap,
                           const CUtensorMap& vmap, cudaStream_t stream) {
    return p.head_dim == 64 ? launch_prefill_t<64>(p, qmap, kmap, vmap, stream)
                            : launch_prefill_t<128>(p, qmap, kmap, vmap, stream);
}

cudaError_t launch_prefill_weights(const PrefillParams& p, const CUtensorMap& qmap,
                                   const CUtensorMap& kmap, cudaStream_t stream) {
    return p.head_dim == 64 ? launch_weights_t<64>(p, qmap, kmap, stream)
                            : launch_weights_t<128>(p, qmap, kmap, stream);
}

cudaError_t read_status_prefill(unsigned* bits, bool clear) {
    cudaError_t e = cudaMemcpyFromSymbol(bits, s_status_prefill, sizeof(unsigned));
    if (e != cudaSuccess || !clear || *bits == 0) return e;
    const unsigned zero = 0;
    return cudaMemcpyToSymbol(s_status_prefill, &zero, sizeof(unsigned));
}

}  // namespace pa
