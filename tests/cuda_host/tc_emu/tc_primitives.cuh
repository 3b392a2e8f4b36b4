// tc_primitives.cuh — the host's form of the kernels' primitives (see emu.h), under the names
// of the file of the same name and of the device part of kda_attn_tc.cuh. A tile is kept as
// blocks of 64 channels with 128 rows of 128 bytes, without the swizzle.
#pragma once
#include "emu.h"

struct CUtensorMap_st;

namespace kda {
namespace tc {

constexpr uint32_t kSpinLimit = 1u << 20;
typedef uint64_t f32x2;

inline uint32_t smem_u32(const void *p) { return (uint32_t)(static_cast<const uint8_t *>(p) - emu::shared_memory); }
inline uint8_t *shared_at(uint32_t a) { return emu::shared_memory + a; }

// ---------------------------------------------------------------- mbarriers
inline void settle(emu::Bar &b)
{
    if (b.pending == 0 && b.tx == 0) {
        b.phase ^= 1;
        b.pending = b.count;
        emu::changed();
    }
}
inline emu::Bar &bar_at(const void *p) { return emu::cta()->bars.at(p); }
inline void mbar_init(uint64_t *p, uint32_t count) { emu::cta()->bars[p] = emu::Bar{(int)count, (int)count, 0, 0}; }
inline void fence_mbar_init() {}
inline void arrived(uint64_t *p, int tx = 0)
{
    emu::Bar &b = bar_at(p);
    if (b.pending <= 0) { std::fprintf(stderr, "an arrival too many\n"); std::abort(); }
    b.tx += tx;
    --b.pending;
    settle(b);
}
inline void landed(uint64_t *p, int bytes)
{
    emu::Bar &b = bar_at(p);
    b.tx -= bytes;
    settle(b);
}
inline void mbar_arrive(uint64_t *p) { arrived(p); emu::pause(0); }
inline void mbar_arrive_expect_tx(uint64_t *p, uint32_t bytes) { arrived(p, (int)bytes); }
inline bool passed(uint64_t *p, uint32_t parity) { return (uint32_t)bar_at(p).phase != parity; }
inline bool mbar_wait(uint64_t *p, uint32_t parity, volatile int *abort, int *err, int code, uint32_t = 0)
{
    for (;;) {
        if (passed(p, parity)) return true;
        if (*abort) return false;
        if (emu::cta()->out_of_polls) break;
        emu::pause(1);
    }
    *abort = 1;
    if (*err == 0) *err = code;
    emu::changed();
    return false;
}
inline bool mbar_drain(uint64_t *p, uint32_t parity, int *err, int code)
{
    while (!passed(p, parity)) {
        if (emu::cta()->out_of_polls) { if (*err == 0) *err = code; return false; }
        emu::pause(1);
    }
    return true;
}
inline bool wait_both(uint64_t *a, int na, uint64_t *b, int nb, volatile int *abort, int *err, int code, uint32_t)
{
    const bool odd = emu::lane() & 1;
    return __all_sync(~0u, mbar_wait(odd ? b : a, (odd ? nb : na) & 1, abort, err, code));
}

inline bool wait_three(uint64_t *a, int na, uint64_t *b, int nb, uint64_t *c, int nc, volatile int *abort, int *err,
                       int code, uint32_t)
{
    const int which = emu::lane() % 3;
    return __all_sync(~0u, mbar_wait(which == 0 ? a : which == 1 ? b : c, (which == 0 ? na : which == 1 ? nb : nc) & 1,
                                     abort, err, code));
}

// ---------------------------------------------------------------- copies
// A tensor map holds its base, its dimensions and its box here.
struct Map { const uint16_t *base; uint64_t d, heads, tokens, last; uint32_t box[4]; };
inline void load_box(uint8_t *dst, const void *map, int x, int head, int token, uint64_t *bar)
{
    Map m;
    std::memcpy(&m, map, sizeof m);
    emu::cta()->copies.push_back([=] {
        for (int r = 0; r < 128; ++r)
            for (int c = 0; c < 64; ++c) {
                const bool in = x + c < (int)m.d && token + r >= 0 && token + r < (int)m.tokens;
                const uint16_t v = in ? m.base[((uint64_t)(token + r) * m.heads + head) * m.d + x + c] : 0;
                std::memcpy(dst + r * 128 + c * 2, &v, 2);
            }
        landed(bar, 128 * 128);
    });
}
template <int D> inline void load_tile(uint8_t *dst, const void *map, int head, int token, uint64_t *bar)
{
    for (int b = 0; b < (D + 63) / 64; ++b) load_box(dst + b * 16384, map, b * 64, head, token, bar);
}
// A map of rows of a head's channels, and one of queries {channel, head of a group, kv head, token}.
inline void tma_load_2d(void *dst, const void *map, int x, int row, uint64_t *bar)
{
    Map m;
    std::memcpy(&m, map, sizeof m);
    emu::cta()->copies.push_back([=] {
        for (uint64_t r = 0; r < m.box[1]; ++r)
            for (int c = 0; c < 64; ++c) {
                const bool in = x + c < (int)m.d && row + r < m.heads;
                const uint16_t v = in ? m.base[(row + r) * m.d + x + c] : 0;
                std::memcpy(static_cast<uint8_t *>(dst) + r * 128 + c * 2, &v, 2);
            }
        landed(bar, (int)m.box[1] * 128);
    });
}
inline void tma_load_4d(void *dst, const void *map, int x, int y, int z, int w, uint64_t *bar)
{
    Map m;
    std::memcpy(&m, map, sizeof m);
    emu::cta()->copies.push_back([=] {
        for (uint64_t t = 0; t < m.box[3]; ++t)
            for (uint64_t g = 0; g < m.box[1]; ++g)
                for (int c = 0; c < 64; ++c) {
                    const bool in = x + c < (int)m.d && w + t < m.last;
                    const uint16_t v =
                        in ? m.base[(((w + t) * m.tokens + z) * m.heads + y + g) * m.d + x + c] : 0;
                    std::memcpy(static_cast<uint8_t *>(dst) + (t * m.box[1] + g) * 128 + c * 2, &v, 2);
                }
        landed(bar, (int)(m.box[1] * m.box[3]) * 128);
    });
}
inline uint32_t sw128(int row, int byte) { return row * 128 + byte; }
inline void fence_proxy_async_smem() {}
inline void cp_async4(void *dst, const void *src, bool real)
{
    emu::cta()->own_copies[emu::cta()->cur].push_back([=] {
        if (real) std::memcpy(dst, src, 4);
        else std::memset(dst, 0, 4);
    });
}
inline void copy16(uint32_t dst, const void *src, int bytes)
{
    emu::cta()->own_copies[emu::cta()->cur].push_back([=] {
        std::memset(shared_at(dst), 0, 16);
        std::memcpy(shared_at(dst), src, bytes);
    });
}
inline void cp_async_wait_all()
{
    auto own = std::move(emu::cta()->own_copies[emu::cta()->cur]);
    emu::cta()->own_copies[emu::cta()->cur].clear();
    emu::pause(0);
    for (auto &f : own) f();
}
inline void cp_async_arrive(uint64_t *bar)
{
    auto &own = emu::cta()->own_copies[emu::cta()->cur];
    emu::cta()->copies.push_back([bar, all = std::move(own)] {
        for (auto &f : all) f();
        arrived(bar);
    });
    own.clear();
}

// ---------------------------------------------------------------- tensor memory
inline void tmem_alloc(uint32_t *slot, uint32_t) { *slot = 0; }
inline void tmem_relinquish() {}
inline void tmem_dealloc(uint32_t, uint32_t) {}
inline void tc_fence_before_sync() {}
inline void tc_fence_after_sync() {}
template <int N> inline void more_registers() {}
template <int N> inline void fewer_registers() {}
inline float &cell(int lane, int col) { return emu::cta()->tmem[lane * 512 + col]; }
inline int own_lane(uint32_t taddr) { return (int)(taddr >> 16) + emu::lane(); }
inline void tmem_start(uint32_t taddr, float *v)
{
    for (int i = 0; i < 32; ++i) v[i] = cell(own_lane(taddr), (taddr & 0xffff) + i);
}
inline void tmem_ready(float *) {}
inline void tmem_ld16_sync(uint32_t taddr, float *v)
{
    for (int i = 0; i < 16; ++i) v[i] = cell(own_lane(taddr), (taddr & 0xffff) + i);
}
inline void tmem_st16(uint32_t taddr, const uint32_t *v)
{
    for (int i = 0; i < 16; ++i) std::memcpy(&cell(own_lane(taddr), (taddr & 0xffff) + i), &v[i], 4);
}
inline void tmem_st_wait() {}

// ---------------------------------------------------------------- products
inline float bf(uint16_t x) { uint32_t u = (uint32_t)x << 16; float f; std::memcpy(&f, &u, 4); return f; }
inline float in_tile(uint32_t tile, int r, int c)
{
    uint16_t v;
    std::memcpy(&v, shared_at(tile + (c >> 6) * 16384 + r * 128 + (c & 63) * 2), 2);
    return bf(v);
}
template <int D> inline void mma_rows_rows(uint32_t acc, uint32_t x, uint32_t y, uint32_t lead)
{
    if (!lead) return;
    emu::cta()->products.push_back([=] {
        for (int r = 0; r < 128; ++r)
            for (int j = 0; j < 128; ++j) {
                float s = 0;
                for (int c = 0; c < D; ++c) s += in_tile(x, r, c) * in_tile(y, j, c);
                cell(r, acc + j) = s;
            }
    });
}
template <int D, int kHalf>
inline void mma_weights_rows(uint32_t acc, uint32_t w, uint32_t y, bool accumulate, uint32_t lead)
{
    if (!lead) return;
    emu::cta()->products.push_back([=] {
        for (int r = 0; r < 128; ++r)
            for (int c = 0; c < D; ++c) {
                float s = accumulate ? cell(r, acc + c) : 0.f;
                for (int j = 0; j < 128; ++j) {
                    uint32_t two;
                    std::memcpy(&two, &cell(r, w + (j >> 6) * kHalf + (j & 63) / 2), 4);
                    s += bf(j & 1 ? two >> 16 : two & 0xffff) * in_tile(y, j, c);
                }
                cell(r, acc + c) = s;
            }
    });
}
template <int D> inline void mma_rows_half(uint32_t acc, uint32_t x, uint32_t y, int h, uint32_t lead)
{
    if (!lead) return;
    emu::cta()->products.push_back([=] {
        for (int r = 0; r < 128; ++r)
            for (int j = 0; j < 64; ++j) {
                float s = 0;
                for (int c = 0; c < D; ++c) s += in_tile(x, r, c) * in_tile(y, h * 64 + j, c);
                cell(r, acc + j) = s;
            }
    });
}
template <int D>
inline void mma_weights_half(uint32_t acc, uint32_t w, uint32_t y, int h, int groups, bool accumulate, uint32_t lead)
{
    if (!lead) return;
    emu::cta()->products.push_back([=] {
        for (int r = 0; r < 128; ++r)
            for (int c = 0; c < D; ++c) {
                float s = accumulate ? cell(r, acc + c) : 0.f;
                for (int j = 0; j < 16 * std::min(groups, 4); ++j) {
                    uint32_t two;
                    std::memcpy(&two, &cell(r, w + j / 2), 4);
                    s += bf(j & 1 ? two >> 16 : two & 0xffff) * in_tile(y, h * 64 + j, c);
                }
                cell(r, acc + c) = s;
            }
    });
}
inline void commit(uint64_t *bar, uint32_t lead)
{
    if (!lead) return;
    emu::cta()->products.push_back([=] { arrived(bar); });
    emu::pause(0);
}

// ---------------------------------------------------------------- arithmetic
inline f32x2 pack2(float a, float b) { float v[2] = {a, b}; f32x2 r; std::memcpy(&r, v, 8); return r; }
inline void unpack2(f32x2 x, float &a, float &b) { float v[2]; std::memcpy(v, &x, 8); a = v[0]; b = v[1]; }
template <typename F> inline f32x2 both(F f, f32x2 x, f32x2 y, f32x2 z = 0)
{
    float a, b, c, d, e, g;
    unpack2(x, a, b); unpack2(y, c, d); unpack2(z, e, g);
    return pack2(f(a, c, e), f(b, d, g));
}
inline f32x2 fma2(f32x2 x, f32x2 y, f32x2 z) { return both([](float a, float b, float c) { return std::fma(a, b, c); }, x, y, z); }
inline f32x2 add2(f32x2 x, f32x2 y) { return both([](float a, float b, float) { return a + b; }, x, y); }
inline f32x2 mul2(f32x2 x, f32x2 y) { return both([](float a, float b, float) { return a * b; }, x, y); }
inline float exp2_fast(float x) { return std::exp2(x); }
inline float max3(float a, float b, float c) { return std::fmax(std::fmax(a, b), c); }
inline uint32_t bf16x2(float lo, float hi)
{
    auto bits = [](float f) { __nv_bfloat16 b = __float2bfloat16_rn(f); uint16_t u; std::memcpy(&u, &b, 2); return (uint32_t)u; };
    return bits(hi) << 16 | bits(lo);
}

}  // namespace tc
}  // namespace kda
