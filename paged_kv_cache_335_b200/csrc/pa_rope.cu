// pa_rope.cu — rotary positions with several axes, fused with the paged append.
//
// Frequency i turns the pair (x_a, x_b) of a q or k row by the angle
//   theta_i = position[axis(i)] * inv_freq[i]
// (rotary position embedding: Su et al., "RoFormer: Enhanced Transformer with
// Rotary Position Embedding", eq. 34; images and video give each token a
// position per axis, and axis(i) says which one frequency i follows), and k
// and v then go to their cache slots as in kv_append_kernel. One pass: q, k
// and v are read once, q_out and the slots written once; k is never written
// back in between.
//
// The angle is formed as a fraction of a turn in 64-bit fixed point: turns[i] =
// inv_freq[i] / (2 pi) modulo 1, in units of 2^-64, times the integer position,
// modulo 2^64. Only the rounding of turns[i] grows with the position (the angle is off by
// at most |position| (1 + |inv_freq|) 2^-65 turns), where a 32-bit float product of a
// position near 10^5 would be off by 10^-2 radians. All 64 bits are then rounded once to
// fp32 half-turns in [-1, 1] for sincospif, so that a small angle, whose leading bits are
// zeros or ones, keeps 24 bits of its own.
//
// Bound by HBM for prompts and by launch latency for a decode step, so: every
// thread moves units of 16 elements (32 bytes of bf16), kept as loaded until the table of
// cosines is there, and the table (one entry per token and frequency) is computed once per
// CTA for all heads.
#include <math.h>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {

static __device__ unsigned int s_status_rope;

namespace {

constexpr int kThreads = 256;
// CTAs per SM. Loads in flight come from many threads with one unit each: 16K tokens of
// 64/8 heads (671 MB) take 129 us = 5.2 TB/s at 5 CTAs, 134 at 4, 185 at 6 (spilled); two
// units per thread at 4 CTAs 136, three at 3 CTAs 152 us.
constexpr int kCtas = 5;
constexpr int kMaxTokens = 4;   // tokens per CTA
constexpr int kMaxHalf = 64;    // frequencies

// Eight consecutive elements as loaded.
template <typename T>
struct Eight {
    uint4 v[sizeof(T) / 2];
    __device__ __forceinline__ void load(const T* p) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) v[i] = ld_stream(p + 16 / sizeof(T) * i);
    }
    __device__ __forceinline__ void widen(float (&f)[8]) const {
        if constexpr (sizeof(T) == 4) {
            float a[4], b[4];
            Elem<float>::widen(v[0], a);
            Elem<float>::widen(v[1], b);
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = a[i], f[4 + i] = b[i];
        } else {
            Elem<__nv_bfloat16>::widen(v[0], f);
        }
    }
};

template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&f)[8]) {
    if constexpr (sizeof(T) == 4) {
        reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = (uint32_t)float_to_bf16_bits(f[2 * i]) |
                   ((uint32_t)float_to_bf16_bits(f[2 * i + 1]) << 16);
        st_v4(p, make_uint4(w[0], w[1], w[2], w[3]));
    }
}

// Eight codes of x / scale (binary32 division), as the quantising append forms
// them: FP8 E4M3 rounded to nearest even and saturated, or int8 clamped to
// +-127 then rounded to nearest even.
template <int FMT>
__device__ __forceinline__ void store8_codes(uint8_t* p, const float (&f)[8], float sc) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float y[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = __fdiv_rn(f[4 * i + j], sc);
        if (FMT == 2)
            w[i] = e4m3x2_code(y[0], y[1]) | (e4m3x2_code(y[2], y[3]) << 16);
        else
            w[i] = int8_code(y[0]) | (int8_code(y[1]) << 8) | (int8_code(y[2]) << 16) |
                   (int8_code(y[3]) << 24);
    }
    *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
}

// grid = (token groups, parts of a token's rows). T: type of q, k, v and q_out;
// FMT: 0 / 1 = the caches hold T, 2 / 3 = E4M3 / int8 codes. A unit is two pieces of 8
// elements of a row: both members of eight pairs, or (pairs of neighbours, or no
// rotation) 16 consecutive elements.
template <typename T, int FMT>
__global__ void __launch_bounds__(kThreads, kCtas)
rope_append_kernel(const __grid_constant__ RopeParams p) {
    __shared__ float2 table[kMaxTokens][kMaxHalf];
    const int token0 = blockIdx.x * p.tokens_per_cta;
    const int ntok = min(p.tokens_per_cta, p.num_tokens - token0);
    const int lg = p.head_dim == 128 ? 3 : 2;              // units per row: 1 << lg
    const int rows = p.num_heads + 2 * p.num_kv_heads;
    const int rot_units = p.half / 8;
    const int part = ((rows << lg) + gridDim.y - 1) / gridDim.y;
    const int u0 = blockIdx.y * part, per_token = min(part, (rows << lg) - u0);

    // this thread's unit: token tk, unit u0 + u
    int tk = per_token > 0 ? 0 : ntok, u = threadIdx.x;
    Eight<T> a, b;
    // a unit's row and piece of it, its first element and the other piece's distance
    struct Place {
        int row, c, at, second;
    };
    auto place = [&] {
        Place r;
        r.row = (u0 + u) >> lg;
        r.c = (u0 + u) & ((1 << lg) - 1);
        const bool split = r.row < p.num_heads + p.num_kv_heads && r.c < rot_units && !p.adjacent;
        r.at = split ? 8 * r.c : 16 * r.c;
        r.second = split ? p.half : 8;
        return r;
    };
    auto load = [&] {  // the first unit at or behind (tk, u)
        while (tk < ntok && u >= per_token) {
            u -= per_token;
            ++tk;
        }
        if (tk >= ntok) return;
        const Place r = place();
        const int64_t t = token0 + tk;
        const T* src;
        if (r.row < p.num_heads)
            src = static_cast<const T*>(p.q) + t * p.q_stride + (int64_t)r.row * p.head_dim;
        else if (r.row < p.num_heads + p.num_kv_heads)
            src = static_cast<const T*>(p.k) + t * p.k_stride +
                  (int64_t)(r.row - p.num_heads) * p.head_dim;
        else
            src = static_cast<const T*>(p.v) + t * p.v_stride +
                  (int64_t)(r.row - p.num_heads - p.num_kv_heads) * p.head_dim;
        a.load(src + r.at);
        b.load(src + r.at + r.second);
    };
    load();
    for (int i = threadIdx.x; i < ntok * p.half; i += kThreads) {
        const int t = i / p.half, f = i - t * p.half;
        const int32_t pos = __ldg(p.positions + (int64_t)p.axis[f] * p.num_tokens + token0 + t);
        const uint64_t turn = (uint64_t)(int64_t)pos * p.turns[f];
        float s, c;
        sincospif((float)(int64_t)turn * 0x1p-63f, &s, &c);
        table[t][f] = make_float2(c * p.mscale, s * p.mscale);
    }
    __syncthreads();
    for (; tk < ntok; u += kThreads, load()) {
        const Place r = place();
        int row = r.row;
        const int c = r.c, at = r.at, second = r.second;
        float x[8], y[8];
        a.widen(x);
        b.widen(y);
        if (row < p.num_heads + p.num_kv_heads && c < rot_units) {
            const float4* cs = reinterpret_cast<const float4*>(&table[tk][8 * c]);  // two at a time
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float4 w = cs[j];
                if (p.adjacent) {  // frequencies 2j, 2j + 1: pairs (4j, 4j + 1), (4j + 2, 4j + 3) of x then y
                    float* z = j < 2 ? x + 4 * j : y + 4 * (j - 2);
                    const float z0 = z[0], z1 = z[1], z2 = z[2], z3 = z[3];
                    z[0] = z0 * w.x - z1 * w.y;
                    z[1] = z1 * w.x + z0 * w.y;
                    z[2] = z2 * w.z - z3 * w.w;
                    z[3] = z3 * w.z + z2 * w.w;
                } else {
                    const float x0 = x[2 * j], x1 = x[2 * j + 1], y0 = y[2 * j], y1 = y[2 * j + 1];
                    x[2 * j] = x0 * w.x - y0 * w.y;
                    y[2 * j] = y0 * w.x + x0 * w.y;
                    x[2 * j + 1] = x1 * w.z - y1 * w.w;
                    y[2 * j + 1] = y1 * w.z + x1 * w.w;
                }
            }
        }
        const int64_t t = token0 + tk;
        if (row < p.num_heads) {
            T* dst = static_cast<T*>(p.q_out) + (t * p.num_heads + row) * p.head_dim + at;
            store8<T>(dst, x);
            store8<T>(dst + second, y);
            continue;
        }
        row -= p.num_heads;
        const bool is_v = row >= p.num_kv_heads;
        if (is_v) row -= p.num_kv_heads;
        const int64_t slot = __ldg(p.slot_mapping + t);
        if (slot < 0) continue;  // padding token
        if (slot >= p.num_slots) {
            atomicOr(&s_status_rope, kStatusBadIndex);
            continue;
        }
        const int64_t blk = slot >> p.log2_block_size;
        const int64_t off = slot & (p.block_size - 1);
        const int64_t to = ((blk * p.num_kv_heads + row) * p.block_size + off) * p.head_dim + at;
        if constexpr (FMT >= 2) {
            uint8_t* dst = static_cast<uint8_t*>(is_v ? p.v_cache : p.k_cache) + to;
            const float sc = __ldg((is_v ? p.v_scale : p.k_scale) + row);
            store8_codes<FMT>(dst, x, sc);
            store8_codes<FMT>(dst + second, y, sc);
        } else {
            T* dst = static_cast<T*>(is_v ? p.v_cache : p.k_cache) + to;
            store8<T>(dst, x);
            store8<T>(dst + second, y);
        }
    }
}

}  // namespace

cudaError_t launch_rope_append(RopeParams p, int dtype, cudaStream_t stream) {
    const int units = (p.num_heads + 2 * p.num_kv_heads) * (p.head_dim / 16);
    // Many tokens: several per CTA, so the table is one entry per thread. A
    // decode step: a token's rows over several CTAs, one unit per thread.
    p.tokens_per_cta = p.num_tokens >= 2 * 148 * kMaxTokens ? kMaxTokens : 1;
    const unsigned parts = p.tokens_per_cta > 1 ? 1u : (unsigned)((units + kThreads - 1) / kThreads);
    const dim3 grid((unsigned)((p.num_tokens + p.tokens_per_cta - 1) / p.tokens_per_cta), parts);
    switch (dtype) {
        case 0: rope_append_kernel<float, 0><<<grid, kThreads, 0, stream>>>(p); break;
        case 1: rope_append_kernel<__nv_bfloat16, 1><<<grid, kThreads, 0, stream>>>(p); break;
        case 2: rope_append_kernel<__nv_bfloat16, 2><<<grid, kThreads, 0, stream>>>(p); break;
        default: rope_append_kernel<__nv_bfloat16, 3><<<grid, kThreads, 0, stream>>>(p); break;
    }
    return cudaGetLastError();
}

cudaError_t read_status_rope(unsigned* bits, bool clear) {
    cudaError_t e = cudaMemcpyFromSymbol(bits, s_status_rope, sizeof(unsigned));
    if (e != cudaSuccess || !clear || *bits == 0) return e;
    const unsigned zero = 0;
    return cudaMemcpyToSymbol(s_status_rope, &zero, sizeof(unsigned));
}

}  // namespace pa
