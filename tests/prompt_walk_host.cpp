// Runs csrc/pa_prompt_walk.cuh on the host: 32 lanes as coroutines that meet at every warp
// intrinsic, so that the code the kernels compile is what is tested.
#include <cuda_runtime.h>
#include <stdint.h>
#include <ucontext.h>

#include <algorithm>
#include <functional>
#include <memory>
#include <vector>

namespace {

constexpr int kLanes = 32;

struct Warp {
    ucontext_t main, lane[kLanes];
    std::unique_ptr<char[]> stack[kLanes];
    int32_t value[2][kLanes];
    int calls[kLanes] = {};
    bool done[kLanes] = {};
    int cur = 0;
    std::function<void()> body;
};
Warp* g_warp;

void lane_main() {
    Warp& w = *g_warp;
    w.body();
    w.done[w.cur] = true;
    swapcontext(&w.lane[w.cur], &w.main);
}

// Every lane's value, once all have come here.
const int32_t* meet(int32_t v) {
    Warp& w = *g_warp;
    const int l = w.cur, buf = w.calls[l]++ & 1;
    w.value[buf][l] = v;
    swapcontext(&w.lane[l], &w.main);
    return w.value[buf];
}

// False if the lanes did not make the same number of calls.
bool run_warp(std::function<void()> body) {
    Warp w;
    w.body = body;
    g_warp = &w;
    for (int l = 0; l < kLanes; ++l) {
        w.stack[l].reset(new char[64 * 1024]);
        getcontext(&w.lane[l]);
        w.lane[l].uc_stack.ss_sp = w.stack[l].get();
        w.lane[l].uc_stack.ss_size = 64 * 1024;
        w.lane[l].uc_link = nullptr;
        makecontext(&w.lane[l], lane_main, 0);
    }
    for (;;) {
        for (int l = 0; l < kLanes; ++l) {
            w.cur = l;
            swapcontext(&w.main, &w.lane[l]);
        }
        const int n = std::count(w.done, w.done + kLanes, true);
        for (int l = 1; l < kLanes; ++l)
            if (w.calls[l] != w.calls[0]) return false;
        if (n == kLanes) return true;
        if (n != 0) return false;
    }
}

struct ThreadIdx {
    struct X {
        operator int() const { return g_warp->cur; }
    } x;
} threadIdx;

template <typename T> T __ldg(const T* p) { return *p; }
int __reduce_add_sync(unsigned, int v) {
    const int32_t* a = meet(v);
    int s = 0;
    for (int l = 0; l < kLanes; ++l) s += a[l];
    return s;
}
int __reduce_max_sync(unsigned, int v) {
    const int32_t* a = meet(v);
    return *std::max_element(a, a + kLanes);
}
unsigned __ballot_sync(unsigned, bool v) {
    const int32_t* a = meet(v);
    unsigned b = 0;
    for (int l = 0; l < kLanes; ++l) b |= (a[l] ? 1u : 0u) << l;
    return b;
}
bool __any_sync(unsigned m, bool v) { return __ballot_sync(m, v) != 0; }
int __shfl_sync(unsigned, int v, int src) { return meet(v)[src & 31]; }
int __shfl_up_sync(unsigned, int v, int d) {
    const int l = g_warp->cur;
    return meet(v)[l >= d ? l - d : l];
}
int __popc(unsigned x) { return __builtin_popcount(x); }
int __ffs(int x) { return __builtin_ffs(x); }
using std::max;
using std::min;

}  // namespace

#undef __forceinline__
#define __forceinline__ inline
#include "pa_prompt_walk.cuh"

// The tiles that one walk finds for `n` indices in turn: out[i] = (seq, start, len, tile). A
// prompt of `len` tokens has ceil(ceil(len / block) * group / per) tiles. Returns -1 if the
// lanes parted or saw different tiles, else whether a lane met a bad prompt.
extern "C" int prompt_walk(const int32_t* cu_seqlens, int num_seqs, int total_tokens, int max_seq_len, int block,
                           int group, int per, int reversed, const int32_t* index, int n, int32_t* out) {
    pa::PrefillParams p = {};
    p.cu_seqlens = cu_seqlens;
    p.num_seqs = num_seqs;
    p.total_tokens = total_tokens;
    p.max_seq_len = max_seq_len;
    bool same = true, bad = false;
    const bool ok = run_warp([&] {
        pa::PromptWalk walk;
        for (int i = 0; i < n; ++i) {
            const pa::PromptTile t = walk.find(
                p, [&](int len) { return ((len + block - 1) / block * group + per - 1) / per; }, index[i],
                reversed != 0);
            const int32_t got[4] = {t.seq, t.start, t.len, t.tile};
            if (g_warp->cur == 0)
                std::copy(got, got + 4, out + 4 * i);
            else
                same = same && std::equal(got, got + 4, out + 4 * i);
            bad = bad || walk.bad;
        }
    });
    return ok && same ? bad : -1;
}
