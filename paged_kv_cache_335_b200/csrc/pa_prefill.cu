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
// a tile; a CTA takes two consecutive ones, so that both read the same K and V
// tiles (two heads of one tile, or two tiles of one head) and one's products run while the
// other's softmax does. Roles:
//   warp 16: issues S_b = Q_b K^T (128 x 128, K = head_dim, A and B in shared memory)
//     and O_b += P_b V (A = P from TMEM, B = V read MN-major), completions by commit;
//   warp 17: loads Q and the ring of K and V tiles by TMA;
//   warps 0..7 and 8..15: the softmax of row blocks 0 and 1, two threads per row (of warps
//     that share TMEM lanes), which exchange the row's maximum in every tile and its sum at
//     the end. P (bf16) overwrites the first half of its S in TMEM;
//   warps 18 and 19: on the tiles that the diagonal crosses, zero the elements of V that are
//     not finite, and the rows behind the prompt, before the tensor core reads
//     them: a masked weight is 0, and 0 x infinity would not be. The epilogue adds the
//     elements so taken out to the rows that attend to them.
// The weights are 2^(score - m) with m a reference that moves only when a row's
// maximum exceeds it by more than 2^kRescaleLog2 (numerator and denominator share it, so
// the result is the exact softmax); O is then rescaled in TMEM by its row's own
// thread. What a row does depends on its own scores alone. P is rounded to bf16 for
// the product (an operand of the tensor core); its sum takes the fp32 weights.
//
// Weights. weights[t] = sum over heads of the group and queries i >= t of
// 2^(score - lse_i): S^T = K Q^T with the keys as rows, so that a key's sum stays in one
// thread; query tiles stream past one key tile. Two CTAs per SM.
//
// Bound by the tensor cores (2 x 1024 cycles per tile pair and row block at head_dim 128)
// and the exponential unit (16 per cycle and SM: 1024 cycles per 128 x 128 weights) alike.
#include <math.h>

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
#ifndef PA_ATTN_POLY
#define PA_ATTN_POLY 0
#endif
#ifndef PA_WEIGHTS_POLY
#define PA_WEIGHTS_POLY 2
#endif

// Bounded wait; gives up at once when another role already gave up.
__device__ __forceinline__ bool wait_or_dead(volatile int* dead, uint32_t bar, uint32_t parity) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = global_timer_ns();
    for (;;) {
#pragma unroll 1
        for (int i = 0; i < 64; ++i)
            if (mbar_try_wait(bar, parity)) return true;
        if (*dead != 0) return false;
        if (global_timer_ns() - t0 > kWaitLimitNs) {
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

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "mov.b64 c, {%6, %7};\n\tfma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 sub2(float2 a, float2 b) {
    return fma2(b, make_float2(-1.f, -1.f), a);
}
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

// 2^x of two values, x <= 128, on the fp32 units instead of the exponential unit: with n =
// round(x) (by adding 1.5 x 2^23) and f = x - n in [-1/2, 1/2], 2^f by its degree-5
// polynomial of least relative error (Remez exchange; below 2.4e-7 in fp32 arithmetic),
// and n added to the exponent bits. x <= -127 gives 0.
__device__ __forceinline__ float2 exp2_poly(float2 x) {
    const float2 big = make_float2(12582912.f, 12582912.f);
    x.x = fmaxf(x.x, -127.f);
    x.y = fmaxf(x.y, -127.f);
    const float2 t = add2(x, big);
    const float2 f = add2(x, sub2(big, t));
    auto both = [](float c) { return make_float2(c, c); };
    float2 y = fma2(f, both(0.0013276472454890609f), both(0.009675540961325169f));
    y = fma2(f, y, both(0.05550713092088699f));
    y = fma2(f, y, both(0.24022120237350464f));
    y = fma2(f, y, both(0.6931469440460205f));
    y = fma2(f, y, both(1.0000001192092896f));
    return make_float2(__int_as_float(__float_as_int(y.x) + (__float_as_int(t.x) << 23)),
                       __int_as_float(__float_as_int(y.y) + (__float_as_int(t.y) << 23)));
}

// 2^x of the pair with index c of a row: kPoly of every eight pairs by polynomial, the
// others by the exponential unit, which alone would bound the kernel.
template <int kPoly>
__device__ __forceinline__ float2 exp2_pair(float2 x, int c) {
    if ((c & 7) * kPoly % 8 + kPoly > 7) return exp2_poly(x);  // spread evenly (compile time)
    return make_float2(ex2(x.x), ex2(x.y));
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
// attention
// ---------------------------------------------------------------------------
constexpr int kCleaners = 2;              // warps
constexpr int kSoftWarps = 16;             // eight per row block, then products, loads, cleaners
constexpr int kAttnThreads = 32 * (kSoftWarps + 2 + kCleaners);
constexpr uint32_t kAttnTmemCols = 512;   // S_0, S_1 (128 columns each), O_0, O_1

template <int D>
struct AttnCfg {
    static constexpr int kTile = D / 64 * kHalfBytes;
    static constexpr int kStages = D == 128 ? 5 : 8;          // K and V tiles, alternating
    static constexpr int kRing = 2 * kTile;                   // after the two Q tiles
    static constexpr int kExt = kRing + kStages * kTile;
    // q 2, full S, empty S, s 2, p 2, o 2, edge 2, clean 2, fin
    static constexpr int kNumBars = 2 * kStages + 13;
    static constexpr int kXch = kExt + (8 * kNumBars + 12 + 15) / 16 * 16;  // + TMEM slot, dead, taken out
    // a row's maxima, at the end its sums, [2 row blocks][2 halves][128]
    static constexpr int kSmem = kXch + 4 * kBlk * 4;
    static constexpr uint32_t kColO = 256;
    static constexpr uint32_t kIdescQK = umma_idesc(kBlk, kBlk, false);
    static constexpr uint32_t kIdescPV = umma_idesc(kBlk, D, true);
    static_assert(kSmem <= 227 * 1024, "shared memory of a CTA");
};
constexpr uint32_t kNegateA = 1u << 13;   // of the instruction descriptor

// Whether `pred` holds for any thread of the two warps that share rows (barrier `id`).
__device__ __forceinline__ bool pair_any(int id, bool pred) {
    uint32_t r;
    asm volatile("{\n .reg .pred p, q;\n setp.ne.u32 q, %2, 0;\n"
                 " bar.red.or.pred p, %1, 64, q;\n selp.u32 %0, 1, 0, p;\n}"
                 : "=r"(r) : "r"(id), "r"((uint32_t)pred) : "memory");
    return r != 0;
}

// The weights 2^(s sl - ms) of half a row: bf16 into TMEM at ts; returns their fp32 sum in
// two parts.
template <int kPoly>
__device__ __forceinline__ float2 put_weights(const uint32_t (&s)[64], float sl, float ms, uint32_t ts) {
    const float2 sl2 = make_float2(sl, sl), ms2 = make_float2(-ms, -ms);
    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
    for (int g = 0; g < 64; g += 32) {
        uint32_t w[16];
#pragma unroll
        for (int c = 0; c < 16; ++c) {
            const int at = g + 2 * c;
            const float2 x = exp2_pair<kPoly>(
                fma2(make_float2(__uint_as_float(s[at]), __uint_as_float(s[at + 1])), sl2, ms2), c);
            w[c] = bf16x2(x.x, x.y);
            sum[c & 1] = add2(sum[c & 1], x);
        }
        tmem_st16_issue(ts + g / 2, w);
    }
    tmem_wait_st();
    return add2(sum[0], sum[1]);
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
    const int kh = blockIdx.x % p.num_kv_heads;
    bool bad = false;
    const PromptTile u = prompt_tile(
        p, [group](int len) { return ((len + kBlk - 1) / kBlk * group + 1) / 2; },
        blockIdx.x / p.num_kv_heads, true, &bad);
    if (bad && kh == 0) atomicOr(&s_status_prefill, kStatusBadIndex);
    if (u.seq < 0) return;
    const uint32_t raw = smem_u32(smem);
    if (raw & 1023u) {
        if (threadIdx.x == 0) atomicOr(&s_status_prefill, kStatusSmemAlign);
        return;
    }
    // row blocks 2 u.tile and 2 u.tile + 1 (the last one of an odd count is alone)
    const int blocks = (u.len + kBlk - 1) / kBlk * group;
    const int nb = min(2, blocks - 2 * u.tile);
    const int tile0 = 2 * u.tile / group, tile1 = (2 * u.tile + nb - 1) / group;
    const int nkmax = tile1 + 1;

    uint8_t* ext = smem + C::kExt;
    const uint32_t bars = smem_u32(ext);
    const uint32_t b_q = bars, b_full = b_q + 16, b_empty = b_full + 8 * S_, b_s = b_empty + 8 * S_,
                   b_p = b_s + 16, b_o = b_p + 16, b_edge = b_o + 16, b_clean = b_edge + 16,
                   b_fin = b_clean + 16;
    uint32_t* tslot = reinterpret_cast<uint32_t*>(ext + 8 * C::kNumBars);
    volatile int* dead = reinterpret_cast<volatile int*>(tslot + 1);
    volatile int* taken = reinterpret_cast<volatile int*>(tslot + 2);
    const uint32_t qbuf = raw, ring = raw + C::kRing;
    if (threadIdx.x == 0) {
        for (int i = 0; i < S_; ++i) {
            mbar_init(b_full + 8 * i, 1);
            mbar_init(b_empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(b_q + 8 * i, 1);
            mbar_init(b_s + 8 * i, 1);
            mbar_init(b_p + 8 * i, kSoftWarps / 2);
            mbar_init(b_o + 8 * i, 1);
            mbar_init(b_edge + 8 * i, 1);
            mbar_init(b_clean + 8 * i, kCleaners);
        }
        mbar_init(b_fin, 1);
        *dead = 0;
        *taken = 0;
        fence_barrier_init();
    }
    if (warp == kSoftWarps) tmem_alloc(smem_u32(tslot), kAttnTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = *tslot;

    // 640 threads get 96 registers each: the 512 of the softmax take 104, the others 64
    if (warp < kSoftWarps)
        asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
    else
        asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    if (warp < kSoftWarps) {  // softmax of row block b: half a row per thread
        const int b = warp >> 3, half = (warp >> 2) & 1, row = threadIdx.x & 127;
        if (b < nb) {
            const int last = b ? tile1 : tile0;   // key tile on the diagonal
            const int head = kh * group + (2 * u.tile + b) % group;
            const int qi = last * kBlk + row;
            const int pair_id = 1 + 4 * b + (warp & 3);
            const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
            const uint32_t ts = tm + lanes + 128 * b, to = tm + lanes + C::kColO + D * b + D / 2 * half;
            float* xch = reinterpret_cast<float*>(smem + C::kXch) + 2 * kBlk * b + row;
            // (its sign is in the product; not 0, so that a masked -infinity stays one)
            const float sl = fmaxf(fabsf(p.scale_log2), 1e-30f);
            float m = -INFINITY, ms = 0.f;
            float2 l2 = make_float2(0.f, 0.f);
            bool ok = true;
            for (int j = 0; j <= last; ++j) {
                ok = __all_sync(0xffffffffu, wait_or_dead(dead, b_s + 8 * b, j & 1));
                uint32_t s[64];
                float mt = -INFINITY;
                if (ok) {
                    tc_fence_after();
                    tmem_ld64_issue(ts + 64 * half, s);
                    tmem_wait_ld(s);
                    if (j == last) {  // the tile the diagonal crosses
                        const int lim = qi - j * kBlk - 64 * half;
#pragma unroll
                        for (int c = 0; c < 64; ++c)
                            if (c > lim) s[c] = 0xff800000u;
                    }
                    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int c = 0; c < 64; c += 8)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            mx[i] = fmaxf(fmaxf(mx[i], __uint_as_float(s[c + i])), __uint_as_float(s[c + 4 + i]));
                    mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                    // (the other thread has read the last one: it did so before its weights,
                    // which S_b's product waited for)
                    xch[half * kBlk] = mt;
                }
                // both halves are in registers (P may overwrite S) and their maxima known
                if (pair_any(pair_id, !ok)) {
                    ok = false;
                    break;
                }
                mt = fmaxf(mt, xch[(half ^ 1) * kBlk]);
                if (j == 0) {
                    m = mt;
                    ms = m * sl;
                } else {
                    const bool move = (mt - m) * sl > kRescaleLog2;
                    if (__any_sync(0xffffffffu, move)) {
                        // S_b's commit came after the last PV of this row block: O is at rest
                        const float al = move ? ex2((m - mt) * sl) : 1.f;
                        if (move) {
                            m = mt;
                            ms = m * sl;
                        }
                        l2.x *= al;
                        l2.y *= al;
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
                if (j == last)
                    l2 = add2(l2, put_weights<0>(s, sl, ms, ts + 32 * half));
                else
                    l2 = add2(l2, put_weights<PA_ATTN_POLY>(s, sl, ms, ts + 32 * half));
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(b_p + 8 * b);
            }
            if (ok) ok = wait_or_dead(dead, b_o + 8 * b, 0);
            // (and the cleaners' note, for the fix below)
            for (int c = 0; ok && c <= tile1 - tile0; ++c) ok = wait_or_dead(dead, b_clean + 8 * c, 0);
            if (ok) xch[half * kBlk] = l2.x + l2.y;
            if (!pair_any(pair_id, !ok)) {
                tc_fence_after();
                const float l = xch[0] + xch[kBlk], inv = 1.f / l;
                const bool live = qi < u.len;
                const bool fix = *taken != 0;
                uint16_t* dst = static_cast<uint16_t*>(p.out) +
                                ((int64_t)(u.start + qi) * p.num_heads + head) * D + D / 2 * half;
#pragma unroll 1
                for (int c = 0; c < D / 2; c += 32) {
                    uint32_t o[32];
                    __syncwarp();
                    tmem_ld32(to + c, o);
                    if (!live) continue;
                    float f[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) f[i] = __uint_as_float(o[i]) * inv;
                    if (fix) {
                        for (int t = tile0 * kBlk; t <= qi; ++t) {
                            const uint4* src = reinterpret_cast<const uint4*>(
                                static_cast<const uint16_t*>(p.v) + (int64_t)(u.start + t) * p.v_stride +
                                (int64_t)kh * D + D / 2 * half + c);
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                float x[8];
                                Elem<__nv_bfloat16>::widen(ld_v4(src + i), x);
#pragma unroll
                                for (int e = 0; e < 8; ++e)
                                    if (!(fabsf(x[e]) < INFINITY)) f[8 * i + e] += x[e];
                            }
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        st_v4(dst + c + 8 * i,
                              make_uint4(bf16x2(f[8 * i], f[8 * i + 1]), bf16x2(f[8 * i + 2], f[8 * i + 3]),
                                         bf16x2(f[8 * i + 4], f[8 * i + 5]), bf16x2(f[8 * i + 6], f[8 * i + 7])));
                }
                if (live && half == 0 && p.lse != nullptr)
                    p.lse[(int64_t)head * p.total_tokens + u.start + qi] = (ms + log2f(l)) * kLn2;
            }
        }
    } else if (warp == kSoftWarps) {  // products
        // The whole warp walks the tiles (what the descriptors are made of stays warp-uniform);
        // one thread issues.
        const uint32_t idqk = C::kIdescQK | (p.scale_log2 < 0.f ? kNegateA : 0u);
        const bool one = elect_one();
        auto wait = [&](uint32_t bar, uint32_t parity) {
            return __all_sync(0xffffffffu, wait_or_dead(dead, bar, parity));
        };
        // S_b from the K tile in stage st
        auto qk = [&](int b, int st) {
            const uint32_t q_lo = rows_lo(qbuf + b * C::kTile), k_lo = rows_lo(ring + st * C::kTile);
            if (one) {
                issue_qk<D>(tm + kBlk * b, q_lo, k_lo, idqk);
                umma_commit(b_s + 8 * b);
            }
            __syncwarp();
        };
        bool ok = true;
        for (int b = 0; b < nb && ok; ++b) {
            ok = wait(b_q + 8 * b, 0) && (b > 0 || wait(b_full, 0));
            if (ok) qk(b, 0);
        }
        if (ok && one) umma_commit(b_empty);
        __syncwarp();
        // ring place (stage, parity) of V tile j, and of K tile j + 1 behind it
        int sv = 1, sk = 2;
        uint32_t pv = 0, pk = 0;
        for (int j = 0; j < nkmax && ok; ++j) {
            bool have_v = false, have_k = false;
            for (int b = 0; b < nb && ok; ++b) {
                const int last = (b ? tile1 : tile0);   // key tile on the diagonal
                if (j > last) continue;
                if (!have_v) {
                    ok = j >= tile0 ? wait(b_clean + 8 * (j - tile0), 0) : wait(b_full + 8 * sv, pv);
                    have_v = true;
                }
                if (!ok || !(ok = wait(b_p + 8 * b, j & 1))) break;
                tc_fence_after();
                const uint32_t lo = v_lo(ring + sv * C::kTile);
                if (one) {
#pragma unroll
                    for (int k = 0; k < kBlk / 16; ++k)
                        umma_ts_words(tm + C::kColO + D * b, tm + kBlk * b + 8 * k, lo + 128 * k, kDescHi,
                                      C::kIdescPV, k > 0 || j > 0);
                    if (j == last) umma_commit(b_o + 8 * b);
                }
                __syncwarp();
                if (j < last) {
                    if (!have_k) {
                        if (!(ok = wait(b_full + 8 * sk, pk))) break;
                        have_k = true;
                    }
                    qk(b, sk);
                }
            }
            if (ok) {
                if (one) {
                    umma_commit(b_empty + 8 * sv);
                    if (have_k) umma_commit(b_empty + 8 * sk);
                }
                __syncwarp();
                for (int n = 0; n < 2; ++n) {
                    if (++sv == S_) sv = 0, pv ^= 1;
                    if (++sk == S_) sk = 0, pk ^= 1;
                }
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
            auto load_q = [&](int b) {
                load_tile<D>(qbuf + b * C::kTile, &qmap, kh * group + (2 * u.tile + b) % group,
                             u.start + (b ? tile1 : tile0) * kBlk, b_q + 8 * b);
            };
            // Tile i of the ring: K (even) or V (odd) of key tile i / 2. The V tiles that
            // the diagonal crosses complete on barriers of their own; nothing is
            // loaded into their stages after them.
            bool ok = true;
            int issued = 0;
            for (int i = 0; i < 2 * nkmax; ++i) {
                const int st = i % S_, j = i >> 1;
                if (i >= S_ && !(ok = wait_or_dead(dead, b_empty + 8 * st, ((i / S_) & 1) ^ 1))) break;
                if (i == 0) load_q(0);
                const bool v = i & 1;
                load_tile<D>(ring + st * C::kTile, v ? &vmap : &kmap, kh, u.start + j * kBlk,
                             v && j >= tile0 ? b_edge + 8 * (j - tile0) : b_full + 8 * st);
                if (i == 0 && nb == 2) load_q(1);
                issued = i + 1;
            }
            if (!ok) {  // given up: the loads in flight land before the CTA ends
                bool landed = mbar_wait_bounded(b_q, 0) && (nb < 2 || mbar_wait_bounded(b_q + 8, 0));
                for (int i = max(0, issued - S_); i < issued; ++i) {
                    const int j = i >> 1;
                    landed &= (i & 1) && j >= tile0 ? mbar_wait_bounded(b_edge + 8 * (j - tile0), 0)
                                                    : mbar_wait_bounded(b_full + 8 * (i % S_), (i / S_) & 1);
                }
                if (!landed) atomicOr(&s_status_prefill, kStatusTimeout);
            }
        }
    } else {  // cleaners
        const int t = threadIdx.x - 32 * (kSoftWarps + 2);
        for (int c = 0; c <= tile1 - tile0; ++c) {
            const int j = tile0 + c;
            if (!__all_sync(0xffffffffu, wait_or_dead(dead, b_edge + 8 * c, 0))) break;
            const uint32_t buf = ring + ((2 * j + 1) % S_) * C::kTile;
            const int rows = u.len - j * kBlk;  // of the prompt
            bool found = false;
#pragma unroll 4
            for (int i = t; i < D / 64 * kBlk * 8; i += 32 * kCleaners) {
                const int r = (i >> 3) & (kBlk - 1);
                const uint32_t at = buf + 16 * i;  // (a row's eight chunks, in whatever order)
                uint4 x = lds128(at);
                uint32_t* xw = &x.x;
                bool odd = r >= rows;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    // an exponent of all ones: infinite or NaN
                    const bool lo = (xw[e] & 0x7f80u) == 0x7f80u, hi = (xw[e] & 0x7f800000u) == 0x7f800000u;
                    if (lo) xw[e] &= 0xffff0000u;
                    if (hi) xw[e] &= 0x0000ffffu;
                    odd |= lo | hi;
                    found |= (lo | hi) && r < rows;
                }
                if (r >= rows) x = make_uint4(0u, 0u, 0u, 0u);
                if (odd)
                    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};"
                                 :: "r"(at), "r"(x.x), "r"(x.y), "r"(x.z), "r"(x.w) : "memory");
            }
            if (found) *taken = 1;
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(b_clean + 8 * c);
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
constexpr int kWThreads = 192;            // four warps that sum, products, loads
constexpr uint32_t kWTmemCols = 256;      // S^T twice

template <int D>
struct WeightsCfg {
    static constexpr int kTile = D / 64 * kHalfBytes;
    static constexpr int kStages = 2;
    static constexpr int kRing = kTile;                       // after the key tile
    static constexpr int kLse = kRing + kStages * kTile;      // [4 warps][128] floats
    static constexpr int kExt = kLse + 4 * kBlk * 4;
    static constexpr int kNumBars = 1 + 2 * kStages + 2 + 2 + 1;  // k, full, empty, s, free, fin
    static constexpr int kSmem = kExt + 8 * kNumBars + 16;
    static_assert(2 * (kSmem + 1024) <= 228 * 1024, "two CTAs per SM");
};

template <int D>
__global__ void __launch_bounds__(kWThreads, 2)
prefill_weights_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                       const PrefillParams p) {
    using C = WeightsCfg<D>;
    constexpr int S_ = C::kStages;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int group = p.num_heads / p.num_kv_heads;
    const int kh = blockIdx.x % p.num_kv_heads;
    bool bad = false;
    const PromptTile u = prompt_tile(p, [](int len) { return (len + kBlk - 1) / kBlk; },
                                     blockIdx.x / p.num_kv_heads, false, &bad);
    if (bad && kh == 0) atomicOr(&s_status_prefill, kStatusBadIndex);
    if (u.seq < 0) return;
    const uint32_t raw = smem_u32(smem);
    if (raw & 1023u) {
        if (threadIdx.x == 0) atomicOr(&s_status_prefill, kStatusSmemAlign);
        return;
    }
    const int key0 = u.tile * kBlk;
    const int first = p.last_queries > 0 ? max(0, u.len - p.last_queries) : 0;  // first query that counts
    const int q_tile0 = max(key0, first) / kBlk;
    const int q_tiles = (u.len + kBlk - 1) / kBlk - q_tile0;
    const int steps = q_tiles * group;      // (head, query tile), heads outermost

    uint8_t* ext = smem + C::kExt;
    const uint32_t bars = smem_u32(ext);
    const uint32_t b_k = bars, b_full = b_k + 8, b_empty = b_full + 8 * S_, b_s = b_empty + 8 * S_,
                   b_free = b_s + 16, b_fin = b_free + 16;
    uint32_t* tslot = reinterpret_cast<uint32_t*>(ext + 8 * C::kNumBars);
    volatile int* dead = reinterpret_cast<volatile int*>(tslot + 1);
    if (threadIdx.x == 0) {
        mbar_init(b_k, 1);
        for (int i = 0; i < S_; ++i) {
            mbar_init(b_full + 8 * i, 1);
            mbar_init(b_empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(b_s + 8 * i, 1);
            mbar_init(b_free + 8 * i, 4);
        }
        mbar_init(b_fin, 1);
        *dead = 0;
        fence_barrier_init();
    }
    if (warp == 4) tmem_alloc(smem_u32(tslot), kWTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = *tslot;

    if (warp < 4) {  // a thread per key
        float* lq = reinterpret_cast<float*>(smem + C::kLse) + warp * kBlk;  // this warp's own
        const int key = key0 + threadIdx.x;
        const uint32_t ts = tm + ((uint32_t)(32 * warp) << 16);
        const float sl = fabsf(p.scale_log2);
        const float2 sl2 = make_float2(sl, sl);
        float sum = 0.f;
        bool ok = true;
        int h = 0, qt = 0;
        // the log-sum-exps of a step's queries, four to a lane, negated, in log2 units
        float mine[4];
        auto fetch = [&](int hh, int tt) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = (q_tile0 + tt) * kBlk + 32 * e + lane;
                mine[e] = hh < group && i < u.len
                              ? -kLog2e * __ldg(p.lse + (int64_t)(kh * group + hh) * p.total_tokens + u.start + i)
                              : 0.f;
            }
        };
        fetch(0, 0);
        for (int n = 0; n < steps; ++n) {
            __syncwarp();  // the previous step's are read
#pragma unroll
            for (int e = 0; e < 4; ++e) lq[32 * e + lane] = mine[e];
            const int q0 = (q_tile0 + qt) * kBlk;
            if (++qt == q_tiles) {
                qt = 0;
                ++h;
            }
            fetch(h, qt);
            __syncwarp();
            if (!(ok = __all_sync(0xffffffffu, wait_or_dead(dead, b_s + 8 * (n & 1), (n >> 1) & 1)))) break;
            tc_fence_after();
            const uint32_t at = ts + 128 * (n & 1);
            const bool whole = q0 >= key0 + kBlk && q0 >= first && q0 + kBlk <= u.len;
            const int lo = max(key, first) - q0, hi = u.len - q0;   // columns that count
            float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                uint32_t s[64];
                tmem_ld64_issue(at + 64 * half, s);
                tmem_wait_ld(s);
                if (half == 1) {  // S^T is in registers
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(b_free + 8 * (n & 1));
                }
                if (whole) {
#pragma unroll
                    for (int c = 0; c < 64; c += 4) {
                        const float4 e = *reinterpret_cast<const float4*>(lq + 64 * half + c);
                        float2 x = fma2(make_float2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), sl2,
                                        make_float2(e.x, e.y));
                        float2 y = fma2(make_float2(__uint_as_float(s[c + 2]), __uint_as_float(s[c + 3])), sl2,
                                        make_float2(e.z, e.w));
                        acc[0] = add2(acc[0], exp2_pair<PA_WEIGHTS_POLY>(x, c / 2));
                        acc[1] = add2(acc[1], exp2_pair<PA_WEIGHTS_POLY>(y, c / 2 + 1));
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < 64; ++c) {
                        const int col = 64 * half + c;
                        if (col >= lo && col < hi) acc[0].x += ex2(fmaf(__uint_as_float(s[c]), sl, lq[col]));
                    }
                }
            }
            sum += (acc[0].x + acc[0].y) + (acc[1].x + acc[1].y);
        }
        if (ok && key < u.len)
            p.weights[((int64_t)u.seq * p.num_kv_heads + kh) * p.weights_stride + key] = sum;
    } else if (warp == 4) {  // products
        const uint32_t idesc = umma_idesc(kBlk, kBlk, false) | (p.scale_log2 < 0.f ? kNegateA : 0u);
        const bool one = elect_one();
        const uint32_t k_lo = rows_lo(raw);
        auto wait = [&](uint32_t bar, uint32_t parity) {
            return __all_sync(0xffffffffu, wait_or_dead(dead, bar, parity));
        };
        bool ok = wait(b_k, 0);
        int st = 0;
        uint32_t ph = 0;
        for (int n = 0; n < steps && ok; ++n) {
            if (n >= 2 && !(ok = wait(b_free + 8 * (n & 1), ((n >> 1) & 1) ^ 1))) break;
            if (!(ok = wait(b_full + 8 * st, ph))) break;
            tc_fence_after();
            const uint32_t d = tm + kBlk * (n & 1), q_lo = rows_lo(raw + C::kRing + st * C::kTile);
            if (one) {
                issue_qk<D>(d, k_lo, q_lo, idesc);
                umma_commit(b_s + 8 * (n & 1));
                umma_commit(b_empty + 8 * st);
            }
            __syncwarp();
            if (++st == S_) st = 0, ph ^= 1;
        }
        if (one) umma_commit(b_fin);
        __syncwarp();
        if (!mbar_wait_bounded(b_fin, 0)) atomicOr(&s_status_prefill, kStatusTimeout);
    } else if (lane == 0) {  // loads
        load_tile<D>(raw, &kmap, kh, u.start + key0, b_k);
        bool ok = true;
        int n = 0;
        for (int h = 0; h < group && ok; ++h) {
            for (int qt = 0; qt < q_tiles; ++qt, ++n) {
                if (n >= S_ && !(ok = wait_or_dead(dead, b_empty + 8 * (n % S_), ((n / S_) & 1) ^ 1))) break;
                load_tile<D>(raw + C::kRing + (n % S_) * C::kTile, &qmap, kh * group + h,
                             u.start + (q_tile0 + qt) * kBlk, b_full + 8 * (n % S_));
            }
        }
        if (!ok) {  // given up: the loads in flight land before the CTA ends
            bool landed = mbar_wait_bounded(b_k, 0);
            for (int i = max(0, n - S_); i < n; ++i)
                landed &= mbar_wait_bounded(b_full + 8 * (i % S_), (i / S_) & 1);
            if (!landed) atomicOr(&s_status_prefill, kStatusTimeout);
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 4) tmem_dealloc(tm, kWTmemCols);
}

template <int D>
cudaError_t launch_prefill_t(const PrefillParams& p, const CUtensorMap& qmap, const CUtensorMap& kmap,
                             const CUtensorMap& vmap, cudaStream_t stream) {
    using C = AttnCfg<D>;
    cudaError_t e = cudaFuncSetAttribute(prefill_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         C::kSmem);
    if (e != cudaSuccess) return e;
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
    const int64_t tiles = (int64_t)(p.total_tokens / kBlk + p.num_seqs) + 1;
    if (tiles * p.num_kv_heads > INT32_MAX) return cudaErrorInvalidConfiguration;
    prefill_weights_kernel<D><<<(unsigned)(tiles * p.num_kv_heads), kWThreads, C::kSmem, stream>>>(qmap, kmap, p);
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
