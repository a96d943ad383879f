// KV cache in 8 bits (sm_100a): quantising rows as they are written, and
// reading them back.
//
// A cache holds e4m3 codes c [B, Hkv, S_cap, d] and, for every group of T
// consecutive positions of a kv-head, one fp32 scale s: the value is c s.
// The writer gives a group the smallest power of two s = 2^k >= 2^-64 with
// amax <= 448 s over the rows that it then holds (448: the largest e4m3), and
// codes rne(x / s).  With a power of two, x / s is exact, c s is exact in
// bf16, and rows that stay in a partly filled group are requantised, c' = rne(c s /
// s'), without a second rounding from 2^-6 s' on, where codes have their three
// bits; below, to a multiple of 2^-9 s'.  The scale falls again with the next write
// behind a rejected draft's large rows, the bits that they cost the prefix do not
// come back.
//
// Bound by HBM: 2 bytes read and 1 written per value on the way in, the
// reverse on the way back; the rows that share the first written group are
// read once more.  Measured: a prompt of 8192 rows (4 sequences, 8 kv-heads, d =
// 128) into an empty cache 31.7 us, 6.4 TB/s (with half the values a thread and
// accesses of 16 and 8 bytes 37.7, with floats in registers 99); up to 28 rows
// behind 64 prefixes 7.6 us; 16 sequences of 4001 to 8192 rows back 94 us, 6.5 TB/s.
#pragma once

#include <cuda_fp8.h>

#include "bd_common.cuh"
#include "bd_mask.cuh"

namespace bd {

constexpr int kQ8Threads = 256;
constexpr int kQ8MinExp = -64;
constexpr int kQ8MaxExp = 120; // of the largest bf16, 255 2^120

struct Q8Params {
    uint8_t *k_cache, *v_cache; // e4m3 [B, Hkv, S_cap, d]
    float *k_scale, *v_scale;   // [B, Hkv, ceil(S_cap / T)]
    int32_t *cache_len;
    const int32_t *n_new;       // [B], or NULL: b rows of every sequence
    const bf16 *k_new, *v_new;  // [B, Hkv, b, d]
    bf16 *k_out, *v_out;        // read back: [B, Hkv, S_cap, d]
    int B, Hkv, b, d, S_cap, T, groups;
};

// 32 bytes at a 16-byte aligned address, in one access where it is a multiple of
// 32 (a warp's lanes then cover whole lines at once: reading a cache back took 103
// us with two stores of 16 bytes a lane and takes 94 us)
__device__ __forceinline__ void st32(void *p, const uint32_t *r)
{
    if ((reinterpret_cast<uintptr_t>(p) & 31) == 0) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(r[0]),
                     "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                     : "memory");
    } else {
        uint4 *q = static_cast<uint4 *>(p);
        q[0] = make_uint4(r[0], r[1], r[2], r[3]);
        q[1] = make_uint4(r[4], r[5], r[6], r[7]);
    }
}
__device__ __forceinline__ void ld32(const void *p, uint32_t *r)
{
    if ((reinterpret_cast<uintptr_t>(p) & 31) == 0) {
        asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                       "=r"(r[6]), "=r"(r[7])
                     : "l"(p));
    } else {
        const uint4 a = static_cast<const uint4 *>(p)[0], b = static_cast<const uint4 *>(p)[1];
        r[0] = a.x; r[1] = a.y; r[2] = a.z; r[3] = a.w;
        r[4] = b.x; r[5] = b.y; r[6] = b.z; r[7] = b.w;
    }
}

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

// k of the smallest power of two with amax <= 448 * 2^k, `least` or more.  448 =
// 1.75 * 2^8: a mantissa above 1.75 takes the next exponent.  amax is finite.
__device__ __forceinline__ int q8_scale_exp(float amax, int least)
{
    const uint32_t u = __float_as_uint(amax);
    const int e = (int)(u >> 23) - 127;
    const int k = e - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    return max(k, least);
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

// Four codes with those above 240 in size, but no NaN, as 240: at the scale 2^120
// the next code, 256, would stand for 2^128, which neither fp32 nor bf16 holds.
__device__ __forceinline__ uint32_t q8_limit_codes(uint32_t c)
{
    uint32_t r = 0;
#pragma unroll
    for (int t = 0; t < 32; t += 8) {
        const uint32_t x = (c >> t) & 255u, a = x & 127u;
        r |= (a > 0x77u && a < 0x7fu ? (x & 128u) | 0x77u : x) << t;
    }
    return r;
}

// One CTA per (touched group, kv-head and K or V, sequence).  NV: vectors of
// 16 values a thread, held in registers between the maximum and the codes as
// they were read (bf16, or codes of rows that stay): 8 registers a vector
// where floats took 16, and so four CTAs to an SM where there were two.
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
    const int vpr = p.d / 16; // vectors per row: a power of two
    const int shift = 31 - __clz(vpr);
    const int total = p.T * vpr;
    const float old = *scale;
    const int row0 = g * p.T;

    uint32_t w[NV][8];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int e = v * blockDim.x + threadIdx.x;
        const int row = row0 + (e >> shift), col = (e & (vpr - 1)) * 16;
#pragma unroll
        for (int k = 0; k < 8; ++k)
            w[v][k] = 0;
        if (e < total && row >= len && row < len + n) {
            ld32(src + (size_t)(row - len) * p.d + col, w[v]);
        } else if (e < total && row < len) {
            const uint4 c = *reinterpret_cast<const uint4 *>(codes + (size_t)row * p.d + col);
            w[v][0] = c.x; w[v][1] = c.y; w[v][2] = c.z; w[v][3] = c.w;
        }
    }
    // values 8 k .. 8 k + 7 of vector v
    auto values = [&](int v, int k, bool kept, float *x) {
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            if (kept) {
                const float2 f = float2_of_e4m3x2((uint16_t)(w[v][2 * k + (t >> 1)] >> (16 * (t & 1))));
                x[2 * t] = f.x * old;
                x[2 * t + 1] = f.y * old;
            } else {
                x[2 * t] = __uint_as_float(w[v][4 * k + t] << 16);
                x[2 * t + 1] = __uint_as_float(w[v][4 * k + t] & 0xffff0000u);
            }
        }
    };
    float amax = 0.f; // of the finite values
    auto finite_max = [&](int v, bool kept) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            float x[8];
            values(v, k, kept, x);
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                const float m = fabsf(x[t]);
                amax = m < INFINITY ? fmaxf(amax, m) : amax;
            }
        }
    };
    uint32_t top = 0;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        if (row0 + ((v * (int)blockDim.x + (int)threadIdx.x) >> shift) < len) {
            finite_max(v, true);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                top = umax_u16x2(top, w[v][k] & 0x7fff7fffu);
        }
    }
    if ((top & 0xffffu) >= 0x7f80u || (top >> 16) >= 0x7f80u) {
        top = 0; // an infinity or a NaN: once more, without them
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            if (row0 + ((v * (int)blockDim.x + (int)threadIdx.x) >> shift) < len)
                continue;
            finite_max(v, false);
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
    const int k = q8_scale_exp(amax, kQ8MinExp);
    const float s = exp2_int(k), inv = exp2_int(-k);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int e = v * blockDim.x + threadIdx.x;
        const int row = row0 + (e >> shift), col = (e & (vpr - 1)) * 16;
        // rows that stay keep their codes under the same scale
        if (e >= total || row >= len + n || (row < len && s == old))
            continue;
        uint32_t c[4];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            float x[8];
            if (row < len)
                values(v, k, true, x);
            else
                values(v, k, false, x);
            c[2 * k] = (uint32_t)e4m3x2(x[0] * inv, x[1] * inv) |
                       (uint32_t)e4m3x2(x[2] * inv, x[3] * inv) << 16;
            c[2 * k + 1] = (uint32_t)e4m3x2(x[4] * inv, x[5] * inv) |
                           (uint32_t)e4m3x2(x[6] * inv, x[7] * inv) << 16;
        }
        *reinterpret_cast<uint4 *>(codes + (size_t)row * p.d + col) = make_uint4(c[0], c[1], c[2], c[3]);
    }
    if (k == kQ8MaxExp) { // (apart from the loop above, which it would slow by 1.5 %)
        for (int e = threadIdx.x; e < total; e += blockDim.x) {
            const int row = row0 + (e >> shift), col = (e & (vpr - 1)) * 16;
            if (row >= len + n)
                break;
            uint4 *at = reinterpret_cast<uint4 *>(codes + (size_t)row * p.d + col); // this thread's
            const uint4 c = *at;
            *at = make_uint4(q8_limit_codes(c.x), q8_limit_codes(c.y), q8_limit_codes(c.z), q8_limit_codes(c.w));
        }
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
// rounded to nearest even).  A thread takes 16 codes and writes 32 bytes at
// once; grid: x = runs of 16-code vectors of one head, y = kv-head and K or V, z =
// sequence.  (Two and four vectors a thread, all loads first: 1 and 8 % slower.)
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
    if (e >= (long long)len * p.d)
        return;
    const uint8_t *codes = (is_v ? p.v_cache : p.k_cache) + head * p.S_cap * p.d;
    const int shift = 31 - __clz(p.d * p.T); // codes of a group: a power of two
    const float s = (is_v ? p.v_scale : p.k_scale)[head * p.groups + (e >> shift)];
    bf16 *out = (is_v ? p.v_out : p.k_out) + head * p.S_cap * p.d;
    const uint4 w = *reinterpret_cast<const uint4 *>(codes + e);
    const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
    uint32_t o[8];
#pragma unroll
    for (int t = 0; t < 8; ++t) {
        const float2 f = float2_of_e4m3x2((uint16_t)(ws[t >> 1] >> (16 * (t & 1))));
        o[t] = pack_bf16x2(f.x * s, f.y * s);
    }
    st32(out + e, o);
}

} // namespace bd
