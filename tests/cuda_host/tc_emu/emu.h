// emu.h — runs a tensor-core kernel's source on the host, one fiber per CUDA thread.
//
// What is asynchronous on the GPU is asynchronous here: copies into shared memory land one by
// one in any order, products are done in their order of issue, and both only when the
// scheduler takes them. Warps go on in an order drawn from a seed, one of them as far as it
// can before another does: so a warp may be arbitrarily late after any arrival. An mbarrier
// tells the parity of its phase only, as the real one. When nothing can go on, all waits run
// out, as their poll limit does on the GPU.
#pragma once
#include <ucontext.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <functional>
#include <map>
#include <random>
#include <vector>

namespace emu {

struct Bar { int count = 0, pending = 0, tx = 0, phase = 0; };

struct Index { unsigned x = 0, y = 0, z = 0; };

struct Cta {
    ucontext_t sched;
    std::vector<ucontext_t> ctx;
    std::vector<std::vector<char>> stacks;
    std::vector<int> state;            // 0 can go on, 1 waits for a change, 2 finished
    std::map<const void *, Bar> bars;
    std::vector<std::function<void()>> products;
    size_t products_done = 0;
    std::vector<std::function<void()>> copies;
    std::vector<float> tmem;           // 128 lanes x 512 columns, 32 bits each
    std::mt19937 rng;
    std::vector<int> rank;             // of the warps, then products, then copies
    int cur = 0, threads = 0, steps = 0;
    bool out_of_polls = false;
    // meetings of a warp's lanes and of the block's threads
    struct Meeting { int in = 0; unsigned long long round = 0; };
    std::vector<Meeting> warps;
    Meeting block, parts[16];
    std::vector<std::vector<std::function<void()>>> own_copies;  // of a thread, until it asks for their arrival
    std::vector<uint32_t> slot;
    std::function<void()> body;
};

inline Cta *&cta() { static Cta *c = nullptr; return c; }
inline uint8_t *shared_memory = nullptr;  // the kernel's own array, 1024-byte aligned

inline void changed()
{
    for (int &s : cta()->state) if (s == 1) s = 0;
}
inline void pause(int state)  // let another fiber go on; state 1: until something has changed
{
    Cta &c = *cta();
    const int me = c.cur;
    c.state[me] = state;
    swapcontext(&c.ctx[me], &c.sched);
}
inline void trampoline()
{
    Cta &c = *cta();
    const int me = c.cur;
    c.body();
    c.state[me] = 2;
    changed();
}

}  // namespace emu
inline emu::Index blockIdx, gridDim;
namespace emu {

inline void run(int threads, unsigned x, unsigned blocks, uint32_t seed, std::function<void()> body)
{
    Cta c;
    cta() = &c;
    c.body = body;
    c.threads = threads;
    blockIdx.x = x;
    gridDim.x = blocks;
    c.rng.seed(seed);
    c.tmem.assign(128 * 512, std::nanf(""));
    const int warps = threads / 32;
    c.ctx.resize(threads);
    c.stacks.assign(threads, std::vector<char>(1 << 16));
    c.state.assign(threads, 0);
    c.warps.resize(warps);
    c.slot.assign(threads, 0);
    c.own_copies.resize(threads);
    c.rank.resize(warps + 2);
    for (int i = 0; i < warps + 2; ++i) c.rank[i] = i;
    for (int t = 0; t < threads; ++t) {
        getcontext(&c.ctx[t]);
        c.ctx[t].uc_stack.ss_sp = c.stacks[t].data();
        c.ctx[t].uc_stack.ss_size = c.stacks[t].size();
        c.ctx[t].uc_link = &c.sched;
        makecontext(&c.ctx[t], trampoline, 0);
    }
    for (;;) {
        if (c.steps++ % 997 == 0) std::shuffle(c.rank.begin(), c.rank.end(), c.rng);
        bool moved = false;
        for (int who : c.rank) {
            if (who < warps) {
                for (int t = who * 32; t < who * 32 + 32; ++t)
                    if (c.state[t] == 0) {
                        c.cur = t;
                        swapcontext(&c.sched, &c.ctx[t]);
                        moved = true;
                    }
            } else if (who == warps) {
                if (c.products_done < c.products.size()) {
                    c.products[c.products_done++]();
                    moved = true;
                }
            } else if (!c.copies.empty()) {
                const size_t i = c.rng() % c.copies.size();
                auto f = c.copies[i];
                c.copies.erase(c.copies.begin() + i);
                f();
                moved = true;
            }
            if (moved) break;
        }
        if (moved) continue;
        if (std::all_of(c.state.begin(), c.state.end(), [](int s) { return s == 2; })) return;
        if (c.out_of_polls) { std::fprintf(stderr, "threads wait for one another\n"); std::abort(); }
        c.out_of_polls = true;
        changed();
    }
}

// All lanes of this thread's warp (or all threads) have come here.
inline void meet(Cta::Meeting &m, int of)
{
    const auto round = m.round;
    if (++m.in == of) {
        m.in = 0;
        ++m.round;
        changed();
        return;
    }
    while (m.round == round) pause(1);
}
inline int lane() { return cta()->cur & 31; }
inline Cta::Meeting &warp() { return cta()->warps[cta()->cur >> 5]; }

// bar.sync id, n: the first n threads here.
inline void part_sync(int id, int n) { meet(cta()->parts[id], n); }
inline void absent() { std::fprintf(stderr, "this instruction is not emulated\n"); std::abort(); }

// What every lane brings, as all of them see it.
inline std::vector<uint32_t> exchange(uint32_t mine)
{
    Cta &c = *cta();
    c.slot[c.cur] = mine;
    meet(warp(), 32);
    const uint32_t *at = c.slot.data() + (c.cur & ~31);
    std::vector<uint32_t> all(at, at + 32);
    meet(warp(), 32);
    return all;
}

}  // namespace emu

// ---------------------------------------------------------------- CUDA's names
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#define threadIdx (emu::Index{(unsigned)emu::cta()->cur})
#define __noinline__
#define __launch_bounds__(...)

inline bool __all_sync(unsigned, bool x)
{
    for (uint32_t y : emu::exchange(x)) if (!y) return false;
    return true;
}
inline bool __any_sync(unsigned, bool x)
{
    for (uint32_t y : emu::exchange(x)) if (y) return true;
    return false;
}
inline float __shfl_xor_sync(unsigned, float x, int mask)
{
    uint32_t u;
    std::memcpy(&u, &x, 4);
    u = emu::exchange(u)[emu::lane() ^ mask];
    std::memcpy(&x, &u, 4);
    return x;
}
inline float __shfl_sync(unsigned, float x, int from)
{
    uint32_t u;
    std::memcpy(&u, &x, 4);
    u = emu::exchange(u)[from & 31];
    std::memcpy(&x, &u, 4);
    return x;
}
inline int __shfl_sync(unsigned, int x, int from) { return (int)emu::exchange((uint32_t)x)[from & 31]; }
inline unsigned __ballot_sync(unsigned, bool x)
{
    unsigned bits = 0, i = 0;
    for (uint32_t y : emu::exchange(x)) bits |= (y != 0) << i++;
    return bits;
}
inline int __ffs(unsigned x) { return __builtin_ffs((int)x); }
inline float __fdividef(float a, float b) { return a / b; }
template <typename T> inline T atomicOr(T *p, T x) { const T old = *p; *p = old | x; return old; }
inline void __syncwarp() { emu::meet(emu::warp(), 32); }
inline void __syncthreads() { emu::meet(emu::cta()->block, emu::cta()->threads); }
template <typename T> inline T __ldg(const T *p) { return *p; }
inline uint32_t __float_as_uint(float x) { uint32_t u; std::memcpy(&u, &x, 4); return u; }
using std::max;
using std::min;

// A launch: its CTAs one after another, each with the next seed; of persistent kernels
// emu::ctas of them (0: as many as were asked for).
namespace emu {
inline unsigned ctas = 1;
inline uint32_t seed = 0;
}
inline cudaError_t cudaGetLastError() { return cudaSuccess; }
// kernel<<<...>>>(args): every block of the grid.
namespace emu {
template <typename... A, typename... B>
inline void launch(void (*kernel)(A...), unsigned blocks, int threads, int, cudaStream_t, B... args)
{
    for (unsigned x = 0; x < blocks; ++x) run(threads, x, blocks, seed++, [&] { kernel(A(args)...); });
}
}
template <typename F> inline cudaError_t cudaFuncSetAttribute(F *, cudaFuncAttribute, int) { return cudaSuccess; }
template <typename P>
inline cudaError_t cudaLaunchKernelEx(const cudaLaunchConfig_t *cfg, void (*kernel)(P), const P &params)
{
    const unsigned ctas = emu::ctas ? emu::ctas : cfg->gridDim.x;
    for (unsigned x = 0; x < ctas; ++x)
        emu::run((int)cfg->blockDim.x, x, ctas, emu::seed++, [&] { kernel(params); });
    return cudaSuccess;
}
