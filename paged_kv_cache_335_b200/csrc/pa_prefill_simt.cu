// pa_prefill_simt.cu — prompt attention and prompt weights on the CUDA cores, in
// fp32: what pa_prefill and pa_prefill_weights run for fp32 inputs.
//
// out[i] = softmax over t <= i of (scale q_i . k_t) applied to v, per prompt and head
// ("PagedAttention原理详解…", § 显存消耗的三大来源, for every query of the prompt at
// once), in one pass over the keys with the running maximum and sum of the
// softmax (Milakov and Gimelshein, "Online normalizer calculation for softmax").
//
// CTA = 64 queries of one head against tiles of 64 keys; thread (ty, tx) of
// 16 x 16 holds the scores of queries 4 ty .. and keys tx, tx + 16, .. and a 4 x D/16 block
// of the output. Rows lie as in memory, 4 floats longer in shared memory, so that
// 16-byte reads along a row are free of bank conflicts, and the next tile's K and V
// arrive by cp.async meanwhile. The weights of a query pass through shared
// memory within its warp. Bound by the fp32 fma rate (64 x 64 x D x 2 per tile: 2.2 us of an
// SM at D = 64) and by the longest prompt's row of tiles.
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "pa_device.cuh"
#include "pa_internal.h"
#include "pa_prefill_tile.cuh"

namespace pa {

static __device__ unsigned int s_status_prefill_simt;

namespace {

constexpr int kB = 64;            // queries and keys of a tile
constexpr int kThreads = 256;
constexpr int kPad = kB + 4;      // row of a transposed tile (floats)

// Rows [row0, row0 + 64) x D of a packed tensor, transposed to dst[d][row];
// rows at or past `end` become zeros.
template <int D>
__device__ __forceinline__ void load_t(float* dst, const float* src, int64_t stride, int row0, int end) {
    for (int i = threadIdx.x; i < kB * (D / 4); i += kThreads) {
        const int r = i % kB, c = i / kB;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (row0 + r < end) v = *reinterpret_cast<const float4*>(src + (int64_t)(row0 + r) * stride + 4 * c);
        dst[(4 * c + 0) * kPad + r] = v.x;
        dst[(4 * c + 1) * kPad + r] = v.y;
        dst[(4 * c + 2) * kPad + r] = v.z;
        dst[(4 * c + 3) * kPad + r] = v.w;
    }
}

// s[4][4] = a . b for rows 4 ty .. of `at` and 4 tx .. of `bt` (both transposed).
template <int D>
__device__ __forceinline__ void dot_tile(const float* at, const float* bt, int ty, int tx, float (&s)[4][4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll 8
    for (int d = 0; d < D; ++d) {
        const float4 a = *reinterpret_cast<const float4*>(at + d * kPad + 4 * ty);
        const float4 b = *reinterpret_cast<const float4*>(bt + d * kPad + 4 * tx);
        const float av[4] = {a.x, a.y, a.z, a.w}, bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) s[i][j] = fmaf(av[i], bv[j], s[i][j]);
    }
}

// Rows [row0, row0 + 64) x D of a packed tensor by cp.async, `pitch` floats apart in shared
// memory; rows at or past `end` become zeros.
template <int D>
__device__ __forceinline__ void load_async(float* dst, int pitch, const float* src, int64_t stride, int row0,
                                           int end) {
    for (int i = threadIdx.x; i < kB * (D / 4); i += kThreads) {
        const int r = i / (D / 4), c = i % (D / 4);
        const bool in = row0 + r < end;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                     :: "r"((uint32_t)__cvta_generic_to_shared(dst + r * pitch + 4 * c)),
                        "l"(src + (int64_t)(in ? row0 + r : 0) * stride + 4 * c), "r"(in ? 16 : 0)
                     : "memory");
    }
}

template <int D>
constexpr size_t smem_prefill() {
    return sizeof(float) * kB * (3 * (size_t)(D + 4) + 2 * (size_t)D + kPad);
}

template <int D>
__global__ void __launch_bounds__(kThreads)
prefill_simt_kernel(const PrefillParams p) {
    extern __shared__ __align__(16) float sm[];
    constexpr int kPitch = D + 4;
    float* qs = sm;                        // [kB][kPitch]
    float* ks = qs + kB * kPitch;          // [2][kB][kPitch]
    float* vs = ks + 2 * kB * kPitch;      // [2][kB][D]
    float* ps = vs + 2 * kB * D;           // [kB][kPad] weights
    const auto tiles = [](int len) { return (len + kB - 1) / kB; };
    PromptWalk walk;
    const PromptTile t = walk.find(p, tiles, blockIdx.x / p.num_heads, true);
    const int h = blockIdx.x % p.num_heads;
    if (walk.bad && h == 0) atomicOr(&s_status_prefill_simt, kStatusBadIndex);
    if (t.seq < 0) return;
    const int kh = h / (p.num_heads / p.num_kv_heads);
    const float* q = static_cast<const float*>(p.q) + (int64_t)h * D;
    const float* k = static_cast<const float*>(p.k) + (int64_t)kh * D;
    const float* v = static_cast<const float*>(p.v) + (int64_t)kh * D;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int end = t.start + t.len, q0 = t.tile * kB;
    auto load_kv = [&](int buf, int j0) {
        load_async<D>(ks + buf * kB * kPitch, kPitch, k, p.k_stride, t.start + j0, end);
        load_async<D>(vs + buf * kB * D, D, v, p.v_stride, t.start + j0, end);
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    load_async<D>(qs, kPitch, q, p.q_stride, t.start + q0, end);
    load_kv(0, 0);
    float2 o[4][D / 32];
    float m[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int j = 0; j < D / 32; ++j) o[i][j] = make_float2(0.f, 0.f);
    }
    for (int j0 = 0, buf = 0; j0 <= q0; j0 += kB, buf ^= 1) {
        if (j0 + kB <= q0) {
            load_kv(buf ^ 1, j0 + kB);
            asm volatile("cp.async.wait_group 1;" ::: "memory");
        } else {
            asm volatile("cp.async.wait_group 0;" ::: "memory");
        }
        __syncthreads();
        const float* kb = ks + buf * kB * kPitch + tx * kPitch;
        const float* vb = vs + buf * kB * D + 4 * tx;
        const float* qb = qs + 4 * ty * kPitch;
        // sums over even and odd dimensions side by side: two products per instruction
        float2 s2[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) s2[i][j] = make_float2(0.f, 0.f);
#pragma unroll 4
        for (int d = 0; d < D; d += 4) {
            float4 a[4], b[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                a[i] = *reinterpret_cast<const float4*>(qb + i * kPitch + d);
                b[i] = *reinterpret_cast<const float4*>(kb + 16 * i * kPitch + d);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s2[i][j] = fma2(make_float2(a[i].x, a[i].y), make_float2(b[j].x, b[j].y), s2[i][j]);
                    s2[i][j] = fma2(make_float2(a[i].z, a[i].w), make_float2(b[j].z, b[j].w), s2[i][j]);
                }
        }
        const bool diag = j0 == q0;
        float s[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float mx = -INFINITY;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[i][j] = s2[i][j].x + s2[i][j].y;
                s[i][j] = diag && tx + 16 * j > 4 * ty + i ? -INFINITY : s[i][j] * p.scale_log2;
                mx = fmaxf(mx, s[i][j]);
            }
#pragma unroll
            for (int off = 1; off < 16; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
            const float old = m[i];
            m[i] = fmaxf(old, mx);
            const float mn = m[i] == -INFINITY ? 0.f : m[i];  // (no score above -infinity yet: weights 0)
            const float al = exp2f(old - mn);
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[i][j] = exp2f(s[i][j] - mn);
                sum += s[i][j];
                ps[(4 * ty + i) * kPad + tx + 16 * j] = s[i][j];
            }
            l[i] = fmaf(l[i], al, sum);
#pragma unroll
            for (int j = 0; j < D / 32; ++j) o[i][j] = mul2(o[i][j], make_float2(al, al));
        }
        __syncwarp();  // a query's weights come from the 16 lanes of its ty
        // on the diagonal a key past the query is left out, not multiplied by a
        // weight of 0: its value may be infinite or NaN
        auto add_values = [&](auto on_diagonal) {
#pragma unroll 2
            for (int c = 0; c < kB; c += 4) {
                float4 w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const float4*>(ps + (4 * ty + i) * kPad + c);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
#pragma unroll
                    for (int g = 0; g < D / 64; ++g) {
                        const float4 x = *reinterpret_cast<const float4*>(vb + (c + e) * D + 64 * g);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            if (decltype(on_diagonal)::value && c + e > 4 * ty + i) continue;
                            const float wi = e == 0 ? w[i].x : e == 1 ? w[i].y : e == 2 ? w[i].z : w[i].w;
                            const float2 w2 = make_float2(wi, wi);
                            o[i][2 * g] = fma2(w2, make_float2(x.x, x.y), o[i][2 * g]);
                            o[i][2 * g + 1] = fma2(w2, make_float2(x.z, x.w), o[i][2 * g + 1]);
                        }
                    }
                }
            }
        };
        if (diag)
            add_values(std::true_type());
        else
            add_values(std::false_type());
        __syncthreads();  // the buffers are read before the next tile but one
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int off = 1; off < 16; off <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], off);
        const int row = q0 + 4 * ty + i;
        if (row >= t.len) continue;
        const float inv = 1.f / l[i];
        float* dst = static_cast<float*>(p.out) + ((int64_t)(t.start + row) * p.num_heads + h) * D;
#pragma unroll
        for (int g = 0; g < D / 64; ++g)
            *reinterpret_cast<float4*>(dst + 64 * g + 4 * tx) =
                make_float4(o[i][2 * g].x * inv, o[i][2 * g].y * inv, o[i][2 * g + 1].x * inv,
                            o[i][2 * g + 1].y * inv);
        if (p.lse != nullptr && tx == 0)
            p.lse[(int64_t)h * p.total_tokens + t.start + row] = (m[i] + log2f(l[i])) * 0.6931471805599453f;
    }
}

// weights[s][kh][t] = sum over the heads of the group and the queries i >= t of
// exp(scale q_i . k_t - lse_i): CTA = 64 keys of one kv head against tiles of 64
// queries. Every sum is formed in a fixed order.
template <int D>
__global__ void __launch_bounds__(kThreads)
prefill_weights_simt_kernel(const PrefillParams p) {
    extern __shared__ __align__(16) float sm[];
    float* kt = sm;                  // [D][kPad]
    float* qt = kt + D * kPad;
    float* lq = qt + D * kPad;       // [kB] log-sum-exp of the queries, log2 units
    const auto tiles = [](int len) { return (len + kB - 1) / kB; };
    PromptWalk walk;
    const PromptTile t = walk.find(p, tiles, blockIdx.x / p.num_kv_heads, false);
    const int kh = blockIdx.x % p.num_kv_heads;
    if (walk.bad && kh == 0) atomicOr(&s_status_prefill_simt, kStatusBadIndex);
    if (t.seq < 0) return;
    const int group = p.num_heads / p.num_kv_heads;
    const float* k = static_cast<const float*>(p.k) + (int64_t)kh * D;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int end = t.start + t.len, k0 = t.tile * kB;
    const int first = p.last_queries > 0 ? max(0, t.len - p.last_queries) : 0;
    load_t<D>(kt, k, p.k_stride, t.start + k0, end);
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    for (int g = 0; g < group; ++g) {
        const int h = kh * group + g;
        const float* q = static_cast<const float*>(p.q) + (int64_t)h * D;
        for (int i0 = max(k0, first / kB * kB); i0 < t.len; i0 += kB) {
            __syncthreads();
            load_t<D>(qt, q, p.q_stride, t.start + i0, end);
            if (threadIdx.x < kB) {
                const int i = i0 + threadIdx.x;
                lq[threadIdx.x] = i < t.len ? __ldg(p.lse + (int64_t)h * p.total_tokens + t.start + i) *
                                                  1.4426950408889634f
                                            : 0.f;
            }
            __syncthreads();
            float s[4][4];
            dot_tile<D>(kt, qt, ty, tx, s);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float sum = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int qi = i0 + 4 * tx + j;
                    if (qi >= first && qi < t.len && k0 + 4 * ty + i <= qi)
                        sum += exp2f(fmaf(s[i][j], p.scale_log2, -lq[4 * tx + j]));
                }
                acc[i] += sum;
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int off = 1; off < 16; off <<= 1) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], off);
        const int tok = k0 + 4 * ty + i;
        if (tx == 0 && tok < t.len)
            p.weights[((int64_t)t.seq * p.num_kv_heads + kh) * p.weights_stride + tok] = acc[i];
    }
}

template <int D>
cudaError_t launch_prefill_t(const PrefillParams& p, cudaStream_t stream) {
    // one more than there can be tiles: its CTAs look every prompt over
    const int64_t ctas = ((int64_t)(p.total_tokens / kB) + p.num_seqs + 1) * p.num_heads;
    if (ctas > INT32_MAX) return cudaErrorInvalidConfiguration;
    // Two CTAs share an SM at D = 64 (more work in flight: 536 CTAs take 148 us, one at a time
    // 156). With no more than two per SM in all, the longest tile's time is the kernel's, and it
    // is shorter alone, the others queueing for the SMs that finish (280 CTAs: 77 us
    // against 92): more shared memory than half an SM's keeps a second one away.
    constexpr size_t alone = std::max(smem_prefill<D>(), (size_t)120 * 1024);
    const size_t smem = ctas <= 2 * 148 ? alone : smem_prefill<D>();
    // (the limit is the kernel's, for every host thread at once: the same in every call)
    cudaError_t e = cudaFuncSetAttribute(prefill_simt_kernel<D>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, (int)alone);
    if (e != cudaSuccess) return e;
    prefill_simt_kernel<D><<<(unsigned)ctas, kThreads, smem, stream>>>(p);
    return cudaGetLastError();
}

template <int D>
cudaError_t launch_weights_t(const PrefillParams& p, cudaStream_t stream) {
    constexpr size_t smem = sizeof(float) * (2 * (size_t)D * kPad + kB);
    cudaError_t e = cudaFuncSetAttribute(prefill_weights_simt_kernel<D>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    // one more than there can be tiles: its CTAs look every prompt over
    const int64_t ctas = ((int64_t)(p.total_tokens / kB) + p.num_seqs + 1) * p.num_kv_heads;
    if (ctas > INT32_MAX) return cudaErrorInvalidConfiguration;
    prefill_weights_simt_kernel<D><<<(unsigned)ctas, kThreads, smem, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prefill_simt(const PrefillParams& p, cudaStream_t stream) {
    return p.head_dim == 64 ? launch_prefill_t<64>(p, stream) : launch_prefill_t<128>(p, stream);
}

cudaError_t launch_prefill_weights_simt(const PrefillParams& p, cudaStream_t stream) {
    return p.head_dim == 64 ? launch_weights_t<64>(p, stream) : launch_weights_t<128>(p, stream);
}

cudaError_t read_status_prefill_simt(unsigned* bits, bool clear) {
    cudaError_t e = cudaMemcpyFromSymbol(bits, s_status_prefill_simt, sizeof(unsigned));
    if (e != cudaSuccess || !clear || *bits == 0) return e;
    const unsigned zero = 0;
    return cudaMemcpyToSymbol(s_status_prefill_simt, &zero, sizeof(unsigned));
}

}  // namespace pa
