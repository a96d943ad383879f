// KV cache in 8 bits (sm_100a): quantising rows as they are written, and
// reading them back.
//
// A cache holds e4m3 codes c [B, Hkv, S_cap, d] and, for every group of T
// consecutive positions of a kv-head, one fp32 scale s: the value is c s.
// The writer gives a group the smallest power of two s = 2^k >= 2^-64 with
// amax <= 448 s over the rows that it then holds (448: the largest e4m3), and
// codes rne(x / s).  With a power of two, x / s is exact, c s is exact in
// bf16, and rows that stay in a partly filled group are requantised without a
// second rounding unless they fall below the smallest code: c' = c s / s'.
// Nothing of an older, larger scale remains: rows of a rejected draft stop
// costing precision with the next write.
//
// Bound by HBM: 2 bytes read and 1 written per value on the way in, the
// reverse on the way back; the rows that share the first written group are
// read once more.
#pragma once

#include <cuda_fp8.h>

#include "bd_common.cuh"
#include "bd_mask.cuh"

namespace bd {

constexpr int kQ8Threads = 256;
constexpr int kQ8MinExp = -64;

struct Q8Params {
    uint8_t *k_cache, *v_cache; // e4m3 [B, Hkv, S_cap, d]
    float *k_scale, *v_scale;   // [B, Hkv, ceil(S_cap / T)]
    int32_t *cache_len;
    const int32_t *n_new;       // [B], or NULL: b rows of every sequence
    const bf16 *k_new, *v_new;  // [B, Hkv, b, d]
    bf16 *k_out, *v_out;        // read back: [B, Hkv, S_cap, d]
    int B, Hkv, b, d, S_cap, T, groups;
};

// two floats to two e4m3 codes, lo in the low byte: round to nearest even,
// +-448 beyond the range, NaN kept
__device__ __forceinline__ uint16_t e4m3x2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
// two e4m3 codes to two halves (exact)
__device__ __forceinline__ uint32_t half2_of_e4m3x2(uint16_t c)
{
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(c));
    return r;
}
__device__ __forceinline__ float2 float2_of_e4m3x2(uint16_t c)
{
    const uint32_t h = half2_of_e4m3x2(c);
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

// k of the smallest power of two with amax <= 448 * 2^k, -64 or more.  448 =
// 1.75 * 2^8: a mantissa above 1.75 takes the next exponent.  amax is finite.
__device__ __forceinline__ int q8_scale_exp(float amax)
{
    const uint32_t u = __float_as_uint(amax);
    const int e = (int)(u >> 23) - 127;
    const int k = e - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    return max(k, kQ8MinExp);
}
__device__ __forceinline__ float exp2_int(int k) // -126 <= k <= 127
{
    return __uint_as_float((uint32_t)(k + 127) << 23);
}

__device__ __forceinline__ uint32_t umax_u16x2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// One CTA per (touched group, kv-head and K or V, sequence).  NV: vectors of
// 8 values a thread, held in registers between the maximum and the codes as
// they were read (bf16, or codes of rows that stay): 4 registers a vector
// where floats took 8, and so four CTAs to an SM where there were two.
// Non-negative bf16 order as their bits do, so the maximum is taken on pairs
// of 16 bits.
template <int NV>
__global__ void __launch_bounds__(kQ8Threads, 4)
    bd_cache_append_q8_kernel(const Q8Params p)
{
    __shared__ float red[kQ8Threads / 32];
    const int i = blockIdx.z, h = blockIdx.y >> 1, is_v = blockIdx.y & 1;
    const int len = p.cache_len[i];
    const int n = p.n_new ? p.n_new[i] : p.b;
    if (n < 0 || n > p.b || len < 0 || (long long)len + n > p.S_cap) {
        if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0)
            raise_device_code(DEV_BAD_CACHE_LEN);
        return;
    }
    const int g = len / p.T + blockIdx.x; // this CTA's group
    if (n == 0 || (long long)g * p.T >= (long long)len + n)
        return;
    const size_t head = (size_t)i * p.Hkv + h;
    uint8_t *codes = (is_v ? p.v_cache : p.k_cache) + head * p.S_cap * p.d;
    float *scale = (is_v ? p.v_scale : p.k_scale) + head * p.groups + g;
    const bf16 *src = (is_v ? p.v_new : p.k_new) + head * p.b * p.d;
    const int vpr = p.d / 8; // vectors per row: a power of two
    const int shift = 31 - __clz(vpr);
    const int total = p.T * vpr;
    const float old = *scale;
    const int row0 = g * p.T;

    uint4 w[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int e = v * blockDim.x + threadIdx.x;
        const int row = row0 + (e >> shift), col = (e & (vpr - 1)) * 8;
        w[v] = make_uint4(0, 0, 0, 0);
        if (e < total && row >= len && row < len + n) {
            w[v] = *reinterpret_cast<const uint4 *>(src + (size_t)(row - len) * p.d + col);
        } else if (e < total && row < len) {
            const uint2 c = *reinterpret_cast<const uint2 *>(codes + (size_t)row * p.d + col);
            w[v].x = c.x;
            w[v].y = c.y;
        }
    }
    // the 8 values of vector v
    auto values = [&](int v, bool kept, float *x) {
        const uint32_t ws[4] = {w[v].x, w[v].y, w[v].z, w[v].w};
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            if (kept) {
                const float2 f = float2_of_e4m3x2((uint16_t)(ws[t >> 1] >> (16 * (t & 1))));
                x[2 * t] = f.x * old;
                x[2 * t + 1] = f.y * old;
            } else {
                x[2 * t] = __uint_as_float(ws[t] << 16);
                x[2 * t + 1] = __uint_as_float(ws[t] & 0xffff0000u);
            }
        }
    };
    float amax = 0.f; // of the finite values
    uint32_t top = 0;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        if (row0 + ((v * (int)blockDim.x + (int)threadIdx.x) >> shift) < len) {
            float x[8];
            values(v, true, x);
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                const float m = fabsf(x[t]);
                amax = m < INFINITY ? fmaxf(amax, m) : amax;
            }
        } else {
            top = umax_u16x2(top, w[v].x & 0x7fff7fffu);
            top = umax_u16x2(top, w[v].y & 0x7fff7fffu);
            top = umax_u16x2(top, w[v].z & 0x7fff7fffu);
            top = umax_u16x2(top, w[v].w & 0x7fff7fffu);
        }
    }
    if ((top & 0xffffu) >= 0x7f80u || (top >> 16) >= 0x7f80u) {
        top = 0; // an infinity or a NaN: once more, without them
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            if (row0 + ((v * (int)blockDim.x + (int)threadIdx.x) >> shift) < len)
                continue;
            float x[8];
            values(v, false, x);
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                const float m = fabsf(x[t]);
                amax = m < INFINITY ? fmaxf(amax, m) : amax;
            }
        }
    }
    amax = fmaxf(amax, fmaxf(__uint_as_float(top << 16), __uint_as_float(top & 0xffff0000u)));
    // non-negative floats order as their bits do
    amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));
    if ((threadIdx.x & 31) == 0)
        red[threadIdx.x >> 5] = amax;
    __syncthreads(); // also: every thread has read the old scale
    amax = red[0];
    for (int x = 1; x < (int)blockDim.x / 32; ++x)
        amax = fmaxf(amax, red[x]);
    const int k = q8_scale_exp(amax);
    const float s = exp2_int(k), inv = exp2_int(-k);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int e = v * blockDim.x + threadIdx.x;
        const int row = row0 + (e >> shift), col = (e & (vpr - 1)) * 8;
        // rows that stay keep their codes under the same scale
        if (e >= total || row >= len + n || (row < len && s == old))
            continue;
        float x[8];
        if (row < len)
            values(v, true, x);
        else
            values(v, false, x);
        uint2 c;
        c.x = (uint32_t)e4m3x2(x[0] * inv, x[1] * inv) |
              (uint32_t)e4m3x2(x[2] * inv, x[3] * inv) << 16;
        c.y = (uint32_t)e4m3x2(x[4] * inv, x[5] * inv) |
              (uint32_t)e4m3x2(x[6] * inv, x[7] * inv) << 16;
        *reinterpret_cast<uint2 *>(codes + (size_t)row * p.d + col) = c;
    }
    if (threadIdx.x == 0)
        *scale = s;
}

// cache_len[i] += n_new[i] where both are in range; after the rows' kernel,
// which reads the old lengths.
__global__ void __launch_bounds__(256)
    bd_cache_advance_kernel(const Q8Params p, int report)
{
    const int i = blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= p.B)
        return;
    const int len = p.cache_len[i];
    const int n = p.n_new ? p.n_new[i] : p.b;
    if (n < 0 || n > p.b || len < 0 || (long long)len + n > p.S_cap) {
        if (report)
            raise_device_code(DEV_BAD_CACHE_LEN);
        return;
    }
    p.cache_len[i] = len + n;
}

// Rows 0 .. cache_len[i]-1 back to bf16 (exact for a power-of-two scale, else
// rounded to nearest even).  A thread takes 16 codes; grid: x = runs of
// 16-code vectors of one head, y = kv-head and K or V, z = sequence.
__global__ void __launch_bounds__(kQ8Threads)
    bd_cache_read_q8_kernel(const Q8Params p)
{
    const int i = blockIdx.z, h = blockIdx.y >> 1, is_v = blockIdx.y & 1;
    const int len = p.cache_len[i];
    if (len < 0 || len > p.S_cap) {
        if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0)
            raise_device_code(DEV_BAD_CACHE_LEN);
        return;
    }
    const size_t head = (size_t)i * p.Hkv + h;
    const long long e = ((long long)blockIdx.x * blockDim.x + threadIdx.x) * 16;
    const int row = (int)(e / p.d);
    if (row >= len)
        return;
    const uint8_t *codes = (is_v ? p.v_cache : p.k_cache) + head * p.S_cap * p.d;
    const float s = (is_v ? p.v_scale : p.k_scale)[head * p.groups + row / p.T];
    bf16 *out = (is_v ? p.v_out : p.k_out) + head * p.S_cap * p.d;
    const uint4 w = *reinterpret_cast<const uint4 *>(codes + e);
    const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
    uint32_t o[8];
#pragma unroll
    for (int t = 0; t < 8; ++t) {
        const float2 f = float2_of_e4m3x2((uint16_t)(ws[t >> 1] >> (16 * (t & 1))));
        o[t] = pack_bf16x2(f.x * s, f.y * s);
    }
    uint4 *dst = reinterpret_cast<uint4 *>(out + e);
    dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
    dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
}

} // namespace bd
