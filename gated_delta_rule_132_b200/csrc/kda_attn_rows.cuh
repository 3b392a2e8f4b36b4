// kda_attn_rows.cuh — softmax attention and its gradients one row at a time, one
// warp per row, fp32 throughout. Only visible keys are read, so what masked places
// hold cannot reach a result.
#pragma once

#include <math.h>

#include "kda_attn.cuh"

namespace kda {

// Lane l of a warp holds the elements [l * V, (l + 1) * V) of a head's row, V = D / 32.
template <typename T, int D>
__device__ __forceinline__ void load_row(const T *row, float (&x)[D / 32])
{
    constexpr int V = D / 32;
    const T *p = row + (threadIdx.x & 31) * V;
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = to_f32(p[i]);
}

template <typename T, int D>
__device__ __forceinline__ void store_row(T *row, const float (&x)[D / 32])
{
    constexpr int V = D / 32;
    T *p = row + (threadIdx.x & 31) * V;
#pragma unroll
    for (int i = 0; i < V; ++i) p[i] = from_f32<T>(x[i]);
}

__device__ __forceinline__ float warp_sum(float x)
{
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
    return x;
}

template <int V>
__device__ __forceinline__ float row_dot(const float (&a)[V], const float (&b)[V])
{
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) s = fmaf(a[i], b[i], s);
    return warp_sum(s);
}

// Whether a row holds nothing but finite numbers, by the whole warp.
template <typename T, int D> __device__ __forceinline__ bool row_finite(const T *row)
{
    float x[D / 32], odd = 0.f;
    load_row<T, D>(row, x);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) odd = fmaf(x[i], 0.f, odd);  // NaN if x is not
    return __all_sync(0xffffffffu, odd == 0.f);
}

// Running softmax of one query row: m the maximum of the scaled scores so far, l
// the sum of e^(s - m), acc the same sum over the values.
template <int V>
struct RowSoftmax {
    float m = -INFINITY, l = 0.f, acc[V];
    __device__ RowSoftmax()
    {
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = 0.f;
    }
    __device__ __forceinline__ void add(float s, const float (&v)[V])
    {
        const float m_new = fmaxf(m, s);
        // nothing but -inf so far: every term is 0 (and -inf - -inf would be NaN)
        const float ref = m_new == -INFINITY ? 0.f : m_new;
        const float keep = expf(m - ref), p = expf(s - ref);
        l = l * keep + p;
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = fmaf(acc[i], keep, p * v[i]);
        m = m_new;
    }
};

// Causal attention of the token `row` of a sequence that starts at `start`, for
// query head h: writes o and lse.
template <typename T, int D>
__device__ void attn_row_fwd(const AttnProblem &p, int row, int start, int h, T *o, float *lse)
{
    constexpr int V = D / 32;
    const int hk = h / (p.Hq / p.Hkv);
    const size_t at = ((size_t)row * p.Hq + h) * D;
    const size_t kv = (size_t)p.Hkv * D;
    const T *k = static_cast<const T *>(p.k) + (size_t)hk * D;
    const T *v = static_cast<const T *>(p.v) + (size_t)hk * D;
    float q[V], x[V], y[V];
    load_row<T, D>(static_cast<const T *>(p.q) + at, q);
    RowSoftmax<V> sm;
    for (int c = start; c <= row; ++c) {
        load_row<T, D>(k + c * kv, x);
        load_row<T, D>(v + c * kv, y);
        sm.add(row_dot(q, x) * p.scale, y);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) y[i] = sm.acc[i] / sm.l;
    store_row<T, D>(o + at, y);
    if (lse && (threadIdx.x & 31) == 0) lse[(size_t)row * p.Hq + h] = sm.m + logf(sm.l);
}

// Query gradient of one row. delta [Hq, tokens]: D_r = <dO_r, o_r>.
template <typename T, int D>
__device__ void attn_row_dq(const AttnProblem &p, int row, int start, int h, const float *lse,
                            const float *delta, const T *dO, T *gq)
{
    constexpr int V = D / 32;
    const int hk = h / (p.Hq / p.Hkv);
    const size_t at = ((size_t)row * p.Hq + h) * D;
    const size_t kv = (size_t)p.Hkv * D;
    const T *k = static_cast<const T *>(p.k) + (size_t)hk * D;
    const T *v = static_cast<const T *>(p.v) + (size_t)hk * D;
    float q[V], g[V], x[V], y[V], acc[V] = {};
    load_row<T, D>(static_cast<const T *>(p.q) + at, q);
    load_row<T, D>(dO + at, g);
    const float z = lse[(size_t)row * p.Hq + h], del = delta[(size_t)h * p.tokens + row];
    for (int c = start; c <= row; ++c) {
        load_row<T, D>(k + c * kv, x);
        load_row<T, D>(v + c * kv, y);
        const float pr = expf(row_dot(q, x) * p.scale - z);
        const float ds = pr * (row_dot(g, y) - del) * p.scale;
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = fmaf(ds, x[i], acc[i]);
    }
    store_row<T, D>(gq + at, acc);
}

// Key and value gradients of one token, summed over the query heads of its group.
template <typename T, int D>
__device__ void attn_row_dkv(const AttnProblem &p, int col, int seq_end, int hk,
                             const float *lse, const float *delta, const T *dO, T *gk, T *gv)
{
    constexpr int V = D / 32;
    const int G = p.Hq / p.Hkv;
    const size_t at = ((size_t)col * p.Hkv + hk) * D;
    const T *q = static_cast<const T *>(p.q);
    float k[V], v[V], x[V], g[V], ak[V] = {}, av[V] = {};
    load_row<T, D>(static_cast<const T *>(p.k) + at, k);
    load_row<T, D>(static_cast<const T *>(p.v) + at, v);
    for (int h = hk * G; h < (hk + 1) * G; ++h)
        for (int r = col; r < seq_end; ++r) {
            const size_t i0 = (size_t)r * p.Hq + h;
            load_row<T, D>(q + i0 * D, x);
            load_row<T, D>(dO + i0 * D, g);
            const float pr = expf(row_dot(x, k) * p.scale - lse[i0]);
            const float ds = pr * (row_dot(g, v) - delta[(size_t)h * p.tokens + r]) * p.scale;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                ak[i] = fmaf(ds, x[i], ak[i]);
                av[i] = fmaf(pr, g[i], av[i]);
            }
        }
    store_row<T, D>(gk + at, ak);
    store_row<T, D>(gv + at, av);
}

}  // namespace kda
