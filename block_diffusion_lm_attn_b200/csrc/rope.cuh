// Rotary positions of queries and keys (sm_100a).
//
// Pair i of a row at position p, (x_a, x_b) with a, b = i, i + rot/2 (half
// layout) or 2i, 2i + 1 (interleaved), turns by the angle t = p f_i:
//     y_a = m (x_a cos t - x_b sin t),   y_b = m (x_b cos t + x_a sin t),
// m the attention factor of a scaled table (1 without one).  The adjoint,
// which takes the gradient of y to that of x, turns by -t.  Dims from rot on
// are copied.
//
// The angle is taken in turns, p f_i / 2 pi, in double precision, and only its
// fraction goes on in float: at position 10^6 a float angle is already off by
// 2^-4, the fraction of the double one by 2^-32 of a turn.
//
// Bound by HBM: each value is read and written once.  A thread keeps one
// row's cosines and sines of 8 pairs in registers and walks over heads, which
// share them, so the trigonometry (8 double products and 8 sincospi a thread)
// is paid once per `heads` heads; the first heads' values are on their way
// meanwhile.  Measured: 40 heads of 4 x 4096 rows, d = 128, 55 us, 6.1 TB/s; one
// decoded block of 16 sequences 6.3 us.
#pragma once

#include "bd_common.cuh"
#include "bd_mask.cuh"

namespace bd {

constexpr int kRopeThreads = 256;

struct RopeParams {
    const bf16 *q, *k;
    bf16 *q_out, *k_out;
    const double *inv_freq;
    const int32_t *start;     // [B] or NULL
    const int32_t *positions; // [B, N] or NULL
    int B, Hq, Hkv, N, d, rot, period;
    int heads;                // heads per CTA
    int copy;                 // the dims from rot on have to be copied
    float mscale;
    float sign;               // -1: adjoint
};

__device__ __forceinline__ void unpack8(const uint4 &v, float *x)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ uint4 pack8(const float *x)
{
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                      pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}

// Thread = (row, unit of 16 dims): pairs 8u .. 8u + 7 for u < rot / 16, dims
// to copy for the units behind.  Grid: x = tiles of rows of all sequences,
// y = groups of p.heads heads (queries first, then keys).
template <bool INTERLEAVED>
__global__ void __launch_bounds__(kRopeThreads)
    bd_rope_kernel(const RopeParams p)
{
    const int units = p.d / 16;
    const int rows_cta = kRopeThreads / units;
    const int tiles = (p.N + rows_cta - 1) / rows_cta;
    const int i = blockIdx.x / tiles;
    const int n = (blockIdx.x % tiles) * rows_cta + threadIdx.x / units;
    const int u = threadIdx.x % units;
    if (n >= p.N)
        return;
    const bool turn = u * 16 < p.rot;
    if (!turn && !p.copy)
        return;
    // the two 16-byte chunks of the unit
    const int a = INTERLEAVED || !turn ? u * 16 : u * 8;
    const int b = INTERLEAVED || !turn ? u * 16 + 8 : p.rot / 2 + u * 8;
    const int h0 = blockIdx.y * p.heads, h1 = min(h0 + p.heads, p.Hq + p.Hkv);
    auto at = [&](int h) -> size_t {
        const size_t hh = h < p.Hq ? (size_t)i * p.Hq + h : (size_t)i * p.Hkv + (h - p.Hq);
        return (hh * p.N + n) * p.d;
    };
    constexpr int U = 4; // heads whose loads are in flight together
    uint4 va[U], vb[U];
    auto load = [&](int h) {
#pragma unroll
        for (int w = 0; w < U; ++w)
            if (h + w < h1) {
                const bf16 *src = (h + w < p.Hq ? p.q : p.k) + at(h + w);
                va[w] = *reinterpret_cast<const uint4 *>(src + a);
                vb[w] = *reinterpret_cast<const uint4 *>(src + b);
            }
    };
    load(h0); // on their way while the angles are taken
    float c[8], s[8];
    if (turn) {
        const long long pos = p.positions ? (long long)p.positions[(size_t)i * p.N + n]
                                          : (long long)(p.start ? p.start[i] : 0) + n % p.period;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            double t = (double)pos * (p.inv_freq[u * 8 + e] * 0.15915494309189533577);
            t -= rint(t);
            sincospif(2.f * (float)t, &s[e], &c[e]);
            c[e] *= p.mscale;
            s[e] *= p.mscale * p.sign;
        }
    }
    for (int h = h0; h < h1; h += U) {
        if (h != h0)
            load(h);
#pragma unroll
        for (int w = 0; w < U; ++w)
            if (h + w < h1) {
                bf16 *dst = (h + w < p.Hq ? p.q_out : p.k_out) + at(h + w);
                if (turn) {
                    float x[8], y[8];
                    unpack8(va[w], x);
                    unpack8(vb[w], y);
                    if (INTERLEAVED) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float x0 = x[2 * e], x1 = x[2 * e + 1];
                            const float y0 = y[2 * e], y1 = y[2 * e + 1];
                            x[2 * e] = x0 * c[e] - x1 * s[e];
                            x[2 * e + 1] = x1 * c[e] + x0 * s[e];
                            y[2 * e] = y0 * c[e + 4] - y1 * s[e + 4];
                            y[2 * e + 1] = y1 * c[e + 4] + y0 * s[e + 4];
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const float x0 = x[e];
                            x[e] = x0 * c[e] - y[e] * s[e];
                            y[e] = y[e] * c[e] + x0 * s[e];
                        }
                    }
                    va[w] = pack8(x);
                    vb[w] = pack8(y);
                }
                *reinterpret_cast<uint4 *>(dst + a) = va[w];
                *reinterpret_cast<uint4 *>(dst + b) = vb[w];
            }
    }
}

} // namespace bd
