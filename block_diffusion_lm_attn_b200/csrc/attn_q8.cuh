// Block decode over a KV cache in 8 bits (sm_100a), plain form: a warp per
// query row, lane l holding dims l, l + 32, ...
#pragma once

#include "cache_q8.cuh"

namespace bd {

struct Q8Attn {
    const bf16 *q;
    const uint8_t *k, *v;
    const float *ks, *vs;
    const int32_t *cache_len;
    bf16 *out;
    float *lse;
    int B, Hq, Hkv, b, d, S_cap, T, groups, mode;
    float scale_log2;
};

__device__ __forceinline__ float e4m3_value(uint8_t c)
{
    return float2_of_e4m3x2(c).x;
}

template <int DH>
__global__ void __launch_bounds__(128) bd_decode_q8_simt_kernel(const Q8Attn p)
{
    constexpr int E = DH / 32;
    const int lane = threadIdx.x & 31;
    const long long row = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (row >= (long long)p.B * p.Hq * p.b)
        return;
    const int j = (int)(row % p.b);
    const int hq = (int)(row / p.b % p.Hq), i = (int)(row / p.b / p.Hq);
    const int len = p.cache_len[i];
    const int own = p.mode == 2 ? 0 : p.b;
    const bool bad = len < 0 || (long long)len + own > p.S_cap;
    const int n = bad ? 0 : len + (p.mode == 0 ? p.b : p.mode == 1 ? j + 1 : 0);
    const size_t head = (size_t)i * p.Hkv + hq / (p.Hq / p.Hkv);
    const uint8_t *k = p.k + head * p.S_cap * DH, *v = p.v + head * p.S_cap * DH;
    float q[E], o[E];
    for (int e = 0; e < E; ++e) {
        q[e] = __bfloat162float(p.q[row * DH + e * 32 + lane]);
        o[e] = 0.f;
    }
    float m = -INFINITY, l = 0.f;
    for (int c = 0; c < n; ++c) {
        float x = 0.f;
        for (int e = 0; e < E; ++e)
            x += q[e] * e4m3_value(k[(size_t)c * DH + e * 32 + lane]);
        for (int s = 16; s; s >>= 1)
            x += __shfl_xor_sync(0xffffffffu, x, s);
        x *= p.ks[head * p.groups + c / p.T] * p.scale_log2;
        const float mn = fmaxf(m, x);
        const float a = m == -INFINITY ? 0.f : exp2f(m - mn), w = exp2f(x - mn);
        l = l * a + w;
        const float sv = w * p.vs[head * p.groups + c / p.T];
        for (int e = 0; e < E; ++e)
            o[e] = o[e] * a + sv * e4m3_value(v[(size_t)c * DH + e * 32 + lane]);
        m = mn;
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    for (int e = 0; e < E; ++e)
        p.out[row * DH + e * 32 + lane] = __float2bfloat16_rn(bad ? NAN : o[e] * inv);
    if (lane == 0)
        p.lse[row] = bad ? NAN : l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
    if (bad && lane == 0 && j == 0 && hq == 0)
        raise_device_code(DEV_BAD_CACHE_LEN);
}

} // namespace bd
