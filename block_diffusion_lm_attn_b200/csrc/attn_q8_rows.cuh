// Block decode over a KV cache in 8 bits for few query rows (sm_100a).
//
// The mathematics of attn_q8_tc.cuh, for units (a sequence and a kv-head) of
// at most 16 query rows (32 below d = 128), single tokens above all.  There the
// 128-row tile of tcgen05 would be almost empty while its softmax still walks 128
// columns a tile; here a warp takes 8, 16 or 32 rows with mma.sync.m16n8k16, and
// what a key costs is fetching and converting its 2 d codes.
//
// Bound by HBM, then by the instructions of a key (about 15 a warp, two thirds
// of them the conversion of codes to f16).  So: one persistent CTA per SM, 8
// warps, each on its own: its own ring of two 8 KB stages of K and V filled by
// TMA, its own running maximum, sum and O in registers, no barrier between
// warps until the segment's end, where the 8 results meet in shared memory.
// Segments are QtSource's; cut units are merged by bd_decode_stream_combine_kernel.
// Measured: single tokens of 24 prefixes of 4096 to 32768 keys, 32 query heads on
// 8, d = 128: 129 us, 6.4 TB/s (141 us, 5.9 TB/s, where calls in a row hold the
// card at its power limit); the same rows as 16 (below) 145 us (164 us), on the
// 128-row tiles 268 us at the time.  A third stage: 144 us (141 us).
//
// Operands straight from the codes as they lie: the order of d within a
// product, and of the columns of O, is free as long as both sides share it.
// Thread (g, t) = (lane / 4, lane % 4) reads d / 4 neighbouring codes of key g
// for K (d = d/4 t + ..) and d / 8 of keys 2t, 2t + 1, 2t + 8, 2t + 9 for V (d
// = d/8 g + ..), 16 bytes at once and without bank conflicts at d = 128.
//
// R = 16 or 32 rows: the queries, and P, are the left operand (16 rows each),
// keys and columns of V the right one (8); a thread ends up with d / 4
// neighbouring columns of O of rows g and g + 8.  R = 8 (every head group of 8 or
// fewer with one token): the other way round, S^T = K Q^T and O^T = V^T P^T, keys
// and columns of V as the 16 rows of the left operand, which halves the products,
// the exponentials and the registers of Q and O; P^T passes from one product to
// the other through movmatrix.
#pragma once

#include "attn_q8_tc.cuh"

namespace bd {

constexpr int kQrWarps = 8;
constexpr int kQrThreads = 32 * kQrWarps;
constexpr int kQrStages = 2;
constexpr int kQrTile = 4096; // bytes of K (and of V) in a stage
constexpr int kQrPitch = kTcD + 4; // floats between rows of a warp's result

// The shared-memory layout (offsets from a 1024-byte aligned base) for R query rows.
template <int R> struct Qr {
    static constexpr int kMerge = R == 8 ? 8 : 16; // rows merged at a time
    static constexpr int kRing = 0;                // [warp][stage][K, V]
    static constexpr int kO = kRing + kQrWarps * kQrStages * 2 * kQrTile; // [warp][kMerge][pitch] f32
    static constexpr int kMl = kO + kQrWarps * kMerge * kQrPitch * 4;   // [warp][kMerge] (l, its exponent)
    static constexpr int kBar = kMl + kQrWarps * kMerge * 8;
    static constexpr int kBytes = kBar + 8 * kQrWarps * kQrStages + 16 + 1024;
    static_assert(kBytes <= 227 * 1024, "more shared memory than a CTA may have");
};

__device__ __forceinline__ void mma_f16(float *c, const uint32_t *a, uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The transpose of an 8 x 8 matrix of halves, two a thread.
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x)
{
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

// W words (4 W codes) from shared memory
template <int W>
__device__ __forceinline__ void qr_lds(uint32_t addr, uint32_t *x)
{
    if constexpr (W == 8) {
        qr_lds<4>(addr, x);
        qr_lds<4>(addr ^ 16, x + 4);
    } else if constexpr (W == 4) {
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "r"(addr));
    } else if constexpr (W == 2) {
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(x[0]), "=r"(x[1]) : "r"(addr));
    } else {
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(x[0]) : "r"(addr));
    }
}

// The place of 16-byte chunk c of row r in a stage of DH-byte rows, under the
// swizzle of DH bytes: bits 4.. of the address are xored with bits 7..
template <int DH>
__device__ __forceinline__ uint32_t qr_place(int r, int c)
{
    const int s = DH == 128 ? r & 7 : DH == 64 ? (r >> 1) & 3 : (r >> 2) & 1;
    return (uint32_t)(r * DH + ((c ^ s) << 4));
}

template <int DH, int R>
__global__ void __launch_bounds__(kQrThreads, 1)
    bd_decode_q8_rows_kernel(const __grid_constant__ CUtensorMap tm_k,
                             const __grid_constant__ CUtensorMap tm_v, const QtParams p)
{
    constexpr int KS = kQrTile / DH; // keys of a step
    constexpr int KW = DH / 16;      // words of a key's codes a thread takes for K
    constexpr int VW = DH / 32;      // and for V
    constexpr int NT = DH / 8;       // 8-column tiles of O
    constexpr bool kSwap = R == 8;
    constexpr int MT = kSwap ? 1 : R / 16; // tiles of rows
    typedef Qr<R> S;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = smem_u32(smem_raw);
    const uint32_t base = (raw_addr + 1023u) & ~1023u;
    uint8_t *sbase = smem_raw + (base - raw_addr);
    float *s_o = reinterpret_cast<float *>(sbase + S::kO);
    float2 *s_ml = reinterpret_cast<float2 *>(sbase + S::kMl);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(sbase + S::kBar + 8 * kQrWarps * kQrStages);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    const uint32_t ring = base + S::kRing + warp * (kQrStages * 2 * kQrTile);
    auto bar = [&](int s) { return base + S::kBar + 8 * (warp * kQrStages + s); };

    if (threadIdx.x == 0) {
        for (int s = 0; s < kQrWarps * kQrStages; ++s)
            mbar_init(base + S::kBar + 8 * s, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        p.pp.cut_desc[blockIdx.x] = make_int4(0, 0, 0, 0);
    }
    __syncthreads();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    QtSource<5> src;
    src.init(p.pp);
    Seg sg, nx;
    bool more = src.next(p.pp, nx);
    int issued = 0, used = 0; // stages of this warp, filled and emptied

    // this warp's step i of segment s, into the next stage
    auto fill = [&](const Seg &s, int i) {
        const int ks = s.lo0 + (i * kQrWarps + warp) * KS;
        if (ks >= s.hi0)
            return;
        const int st = issued % kQrStages;
        if (lane == 0) {
            const uint32_t dst = ring + st * (2 * kQrTile);
            mbar_expect_tx(bar(st), 2 * kQrTile);
            tma_load_3d(dst, &tm_k, 0, ks, s.kvhead, bar(st));
            tma_load_3d(dst + kQrTile, &tm_v, 0, ks, s.kvhead, bar(st));
        }
        ++issued;
    };
    for (int i = 0; more && i < kQrStages; ++i)
        fill(nx, i);
    // The queries of a segment as they lie, rows g and g + 8 of each 16 (g of 8),
    // and the scales of this warp's first 32 keys: loaded before the segment's
    // start, so that they are on their way while the one before is merged.
    uint2 qw[MT][2][DH / 16];
    auto load_queries = [&](const Seg &s) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int h = 0; h < (kSwap ? 1 : 2); ++h) {
                const int r = mt * 16 + h * 8 + g;
                const bool valid = r < s.nrows;
                const uint2 *row = reinterpret_cast<const uint2 *>(
                    p.q + ((size_t)s.out_row0 + (valid ? r : 0)) * DH + t * (DH / 4));
#pragma unroll
                for (int i = 0; i < DH / 16; ++i)
                    qw[mt][h][i] = valid ? row[i] : make_uint2(0, 0);
            }
    };
    // scales of a 32-key part, two runs of 16 keys; keys that are none take
    // neutral ones (kQtMidScale: see vmin)
    auto scales = [&](const Seg &s, int k0, float2 *e) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int key = k0 + 16 * c;
            e[c] = make_float2(1.f, kQtMidScale);
            if (key < s.hi0) {
                const size_t at = (size_t)s.kvhead * p.groups + (key >> p.tshift);
                e[c] = make_float2(p.ks[at], p.vs[at]);
            }
        }
    };
    float2 es[2];
    if (more) {
        load_queries(nx);
        scales(nx, nx.lo0 + warp * KS, es);
    }

    while (more) {
        sg = nx;
        // queries: f16 of 2^-k q (exact but far below the row's largest) in
        // the layout of their operand, and 2^k
        uint32_t qf[MT][DH / 16][kSwap ? 2 : 4];
        float qs[MT][2];
        int seen[MT][2];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int h = 0; h < (kSwap ? 1 : 2); ++h) {
                float amax = 0.f;
                bool finite = true;
#pragma unroll
                for (int i = 0; i < DH / 16; ++i) {
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const uint32_t v = x ? qw[mt][h][i].y : qw[mt][h][i].x;
                        const float a = fabsf(__uint_as_float(v << 16));
                        const float b = fabsf(__uint_as_float(v & 0xffff0000u));
                        finite = finite && a < INFINITY && b < INFINITY;
                        amax = fmax3(amax, a, b);
                    }
                }
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
                const unsigned all = __ballot_sync(0xffffffffu, finite);
                finite = ((all >> (lane & ~3)) & 15u) == 15u;
                const int k = q8_scale_exp(finite ? amax : 0.f, kQtMinQExp);
                const float inv = finite ? exp2_int(-k) : NAN;
                qs[mt][h] = exp2_int(k);
#pragma unroll
                for (int i = 0; i < DH / 16; ++i) {
                    qf[mt][i][kSwap ? 0 : h] = pack_f16x2(__uint_as_float(qw[mt][h][i].x << 16) * inv,
                                              __uint_as_float(qw[mt][h][i].x & 0xffff0000u) * inv);
                    qf[mt][i][kSwap ? 1 : 2 + h] = pack_f16x2(__uint_as_float(qw[mt][h][i].y << 16) * inv,
                                                  __uint_as_float(qw[mt][h][i].y & 0xffff0000u) * inv);
                }
            }
        // of the rows whose scores this thread gets: g and g + 8, or 2t and 2t + 1
        if constexpr (kSwap) {
            qs[0][1] = __shfl_sync(0xffffffffu, qs[0][0], 8 * t + 4);
            qs[0][0] = __shfl_sync(0xffffffffu, qs[0][0], 8 * t);
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = kSwap ? 2 * t + h : mt * 16 + h * 8 + g;
                const int jr = min(r, sg.nrows - 1) % p.pp.b; // (one tile of rows a unit)
                seen[mt][h] = min(sg.hi0, sg.len + (p.pp.mode == 0 ? p.pp.b : p.pp.mode == 1 ? jr + 1 : 0));
            }
        const int full_end = min(sg.fhi0, sg.hi0); // keys that every row sees

        constexpr int NO = kSwap ? NT / 2 : NT;
        float o[MT][NO][4];
        float m[MT][2], l[MT][2];
        float vmin = kQtMidScale, vmax = kQtMidScale; // V's scales so far
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
            for (int n = 0; n < NO; ++n)
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    o[mt][n][x] = 0.f;
            m[mt][0] = m[mt][1] = -INFINITY;
            l[mt][0] = l[mt][1] = 0.f;
        }
        // V codes of 16 keys, those of none as zeros: no code of them may be used
        auto load_v = [&](int c, int ks, int part, uint32_t vb, bool ragged, uint32_t (*v)[VW]) {
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int r = c * 16 + 2 * t + (x & 1) + 8 * (x >> 1);
                const int byte = g * (DH / 8);
                qr_lds<VW>(vb + qr_place<DH>(part * 32 + r, byte >> 4) + (byte & 15), v[x]);
                if (ragged && ks + r >= sg.hi0) {
#pragma unroll
                    for (int w = 0; w < VW; ++w)
                        v[x][w] = 0;
                }
            }
        };
        for (int i = 0;; ++i) {
            const int k0 = sg.lo0 + (i * kQrWarps + warp) * KS;
            if (k0 >= sg.hi0)
                break;
            const int st = used % kQrStages;
            const uint32_t kb = ring + st * (2 * kQrTile), vb = kb + kQrTile;
            mbar_wait_warp(bar(st), (uint32_t)((used / kQrStages) & 1), abort_flag);
#pragma unroll 1
            for (int part = 0; part < KS / 32; ++part) {
                const int ks = k0 + part * 32;
                if (ks >= sg.hi0)
                    break;
                const float2 ec[2] = {es[0], es[1]};
                vmin = fminf(vmin, fminf(ec[0].y, ec[1].y));
                vmax = fmaxf(vmax, fmaxf(ec[0].y, ec[1].y));
                // the next part's scales are on their way meanwhile
                scales(sg, part + 1 < KS / 32 ? ks + 32 : k0 + kQrWarps * KS, es);
                if constexpr (kSwap) {
                    // S^T = K Q^T, 16 keys at a time: keys g and g + 8, rows 2t, 2t + 1
                    float s[2][4];
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        uint32_t x0[KW], x1[KW];
                        const int r = part * 32 + c * 16 + g;
                        const int byte = t * (DH / 4);
                        qr_lds<KW>(kb + qr_place<DH>(r, byte >> 4) + (byte & 15), x0);
                        qr_lds<KW>(kb + qr_place<DH>(r + 8, byte >> 4) + (byte & 15), x1);
#pragma unroll
                        for (int y = 0; y < 4; ++y)
                            s[c][y] = 0.f;
#pragma unroll
                        for (int w = 0; w < KW; ++w) {
                            const uint32_t a[4] = {half2_of_e4m3x2((uint16_t)x0[w]),
                                                   half2_of_e4m3x2((uint16_t)x1[w]),
                                                   half2_of_e4m3x2((uint16_t)(x0[w] >> 16)),
                                                   half2_of_e4m3x2((uint16_t)(x1[w] >> 16))};
                            mma_f16(s[c], a, qf[0][w][0], qf[0][w][1]);
                        }
                    }
                    if (ks + 32 > full_end) {
#pragma unroll
                        for (int c = 0; c < 2; ++c)
#pragma unroll
                            for (int y = 0; y < 4; ++y)
                                if (ks + c * 16 + g + 8 * (y >> 1) >= seen[0][y & 1])
                                    s[c][y] = -INFINITY;
                    }
                    const float lv[2] = {lg2(ec[0].y), lg2(ec[1].y)};
                    const float iv[2] = {1.f / ec[0].y, 1.f / ec[1].y};
                    float a[2][2], mx[2]; // of the rows 2t + h
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        // (no less than 2^-126: a masked score stays -inf)
                        a[h][0] = fmaxf(ec[0].x * p.pp.scale_log2 * qs[0][h], 1.2e-38f);
                        a[h][1] = fmaxf(ec[1].x * p.pp.scale_log2 * qs[0][h], 1.2e-38f);
                        mx[h] = fmaxf(fmaf(fmaxf(s[0][h], s[0][2 + h]), a[h][0], lv[0]),
                                      fmaf(fmaxf(s[1][h], s[1][2 + h]), a[h][1], lv[1]));
#pragma unroll
                        for (int w = 4; w < 32; w <<= 1)
                            mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], w));
                    }
                    const bool n0 = mx[0] > m[0][0] + (kQtTop + kQtLazy), n1 = mx[1] > m[0][1] + (kQtTop + kQtLazy);
                    if (__any_sync(0xffffffffu, n0 || n1)) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            float c = 1.f;
                            if (h ? n1 : n0) {
                                c = m[0][h] == -INFINITY ? 0.f : ex2(m[0][h] - (mx[h] - kQtTop));
                                l[0][h] = m[0][h] == -INFINITY ? l[0][h] : l[0][h] * c;
                                m[0][h] = mx[h] - kQtTop;
                            }
#pragma unroll
                            for (int n = 0; n < NO; ++n) {
                                o[0][n][h] *= c;
                                o[0][n][2 + h] *= c;
                            }
                        }
                    }
                    const float nm[2] = {m[0][0] == -INFINITY ? 0.f : -m[0][0], m[0][1] == -INFINITY ? 0.f : -m[0][1]};
                    uint32_t pf[2][2];
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float y[4];
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            y[x] = ex2(fmaf(s[c][x], a[x & 1][c], lv[c] + nm[x & 1]));
                        l[0][0] = fmaf(y[0] + y[2], iv[c], l[0][0]);
                        l[0][1] = fmaf(y[1] + y[3], iv[c], l[0][1]);
                        pf[c][0] = movmatrix_trans(pack_f16x2(y[0], y[1]));
                        pf[c][1] = movmatrix_trans(pack_f16x2(y[2], y[3]));
                    }
                    // O^T += V^T P^T, 16 keys at a time
                    const bool ragged = ks + 32 > sg.hi0;
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        uint32_t v[4][VW]; // keys 2t, 2t + 1, 2t + 8, 2t + 9
                        load_v(c, ks, part, vb, ragged, v);
#pragma unroll
                        for (int w = 0; w < VW; ++w)
#pragma unroll
                            for (int half = 0; half < 2; ++half) {
                                // codes of two keys side by side, two columns
                                const uint32_t lo = __byte_perm(v[0][w], v[1][w], half ? 0x7362 : 0x5140);
                                const uint32_t hi = __byte_perm(v[2][w], v[3][w], half ? 0x7362 : 0x5140);
                                const uint32_t a4[4] = {half2_of_e4m3x2((uint16_t)lo),
                                                        half2_of_e4m3x2((uint16_t)(lo >> 16)),
                                                        half2_of_e4m3x2((uint16_t)hi),
                                                        half2_of_e4m3x2((uint16_t)(hi >> 16))};
                                mma_f16(o[0][2 * w + half], a4, pf[c][0], pf[c][1]);
                            }
                    }
                } else {
                    // S = Q K^T, 8 keys at a time
                    float s[MT][4][4];
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
                        uint32_t x[KW];
                        const int r = part * 32 + n * 8 + g;
                        const int byte = t * (DH / 4);
                        qr_lds<KW>(kb + qr_place<DH>(r, byte >> 4) + (byte & 15), x);
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                            for (int y = 0; y < 4; ++y)
                                s[mt][n][y] = 0.f;
#pragma unroll
                        for (int w = 0; w < KW; ++w) {
                            const uint32_t b0 = half2_of_e4m3x2((uint16_t)x[w]);
                            const uint32_t b1 = half2_of_e4m3x2((uint16_t)(x[w] >> 16));
#pragma unroll
                            for (int mt = 0; mt < MT; ++mt)
                                mma_f16(s[mt][n], qf[mt][w], b0, b1);
                        }
                    }
                    const float lv[2] = {lg2(ec[0].y), lg2(ec[1].y)};
                    const float iv[2] = {1.f / ec[0].y, 1.f / ec[1].y};
                    uint32_t pf[MT][2][4];
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                        for (int h = 0; h < 2; ++h) { // rows g, g + 8
                            if (ks + 32 > full_end) {
#pragma unroll
                                for (int n = 0; n < 4; ++n)
#pragma unroll
                                    for (int y = 0; y < 2; ++y)
                                        if (ks + n * 8 + 2 * t + y >= seen[mt][h])
                                            s[mt][n][2 * h + y] = -INFINITY;
                            }
                            // (no less than 2^-126: a masked score stays -inf)
                            const float a0 = fmaxf(ec[0].x * p.pp.scale_log2 * qs[mt][h], 1.2e-38f);
                            const float a1 = fmaxf(ec[1].x * p.pp.scale_log2 * qs[mt][h], 1.2e-38f);
                            const float x0 = fmaxf(fmax3(s[mt][0][2 * h], s[mt][0][2 * h + 1], s[mt][1][2 * h]), s[mt][1][2 * h + 1]);
                            const float x1 = fmaxf(fmax3(s[mt][2][2 * h], s[mt][2][2 * h + 1], s[mt][3][2 * h]), s[mt][3][2 * h + 1]);
                            float mx = fmaxf(fmaf(x0, a0, lv[0]), fmaf(x1, a1, lv[1]));
                            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                            const bool need = mx > m[mt][h] + (kQtTop + kQtLazy);
                            if (__any_sync(0xffffffffu, need)) {
                                float c = 1.f;
                                if (need) {
                                    c = m[mt][h] == -INFINITY ? 0.f : ex2(m[mt][h] - (mx - kQtTop));
                                    l[mt][h] = m[mt][h] == -INFINITY ? l[mt][h] : l[mt][h] * c;
                                    m[mt][h] = mx - kQtTop;
                                }
#pragma unroll
                                for (int n = 0; n < NT; ++n) {
                                    o[mt][n][2 * h] *= c;
                                    o[mt][n][2 * h + 1] *= c;
                                }
                            }
                            const float nm = m[mt][h] == -INFINITY ? 0.f : -m[mt][h];
#pragma unroll
                            for (int c = 0; c < 2; ++c) {
                                float y[4];
#pragma unroll
                                for (int x = 0; x < 4; ++x)
                                    y[x] = ex2(fmaf(s[mt][2 * c + (x >> 1)][2 * h + (x & 1)], c ? a1 : a0, lv[c] + nm));
                                l[mt][h] = fmaf((y[0] + y[1]) + (y[2] + y[3]), iv[c], l[mt][h]);
                                pf[mt][c][h] = pack_f16x2(y[0], y[1]);
                                pf[mt][c][2 + h] = pack_f16x2(y[2], y[3]);
                            }
                        }
                    // O += P V, 16 keys at a time
                    const bool ragged = ks + 32 > sg.hi0;
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        uint32_t v[4][VW]; // keys 2t, 2t + 1, 2t + 8, 2t + 9
                        load_v(c, ks, part, vb, ragged, v);
#pragma unroll
                        for (int w = 0; w < VW; ++w)
#pragma unroll
                            for (int half = 0; half < 2; ++half) {
                                // codes of two keys side by side, two columns
                                const uint32_t lo = __byte_perm(v[0][w], v[1][w], half ? 0x7362 : 0x5140);
                                const uint32_t hi = __byte_perm(v[2][w], v[3][w], half ? 0x7362 : 0x5140);
#pragma unroll
                                for (int x = 0; x < 2; ++x) {
                                    const uint32_t b0 = half2_of_e4m3x2((uint16_t)(x ? lo >> 16 : lo));
                                    const uint32_t b1 = half2_of_e4m3x2((uint16_t)(x ? hi >> 16 : hi));
#pragma unroll
                                    for (int mt = 0; mt < MT; ++mt)
                                        mma_f16(o[mt][4 * w + 2 * half + x], pf[mt][c], b0, b1);
                                }
                            }
                    }
                }
            }
            __syncwarp(); // every lane has read the stage
            ++used;
            fill(sg, i + kQrStages);
        }
        // V's scales too far apart (kQtSpread): the sums once more, from scores
        // taken once more, in units of 2^u, u raised to a row's maximum where that
        // lies kQtLazy above.  (Found out, and summed, as the keys go by, it cost
        // every call 2 to 10 %.)
        float u[MT][2];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            u[mt][0] = m[mt][0];
            u[mt][1] = m[mt][1];
        }
        if (__builtin_expect(vmax > vmin * kQtSpread, 0)) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                l[mt][0] = l[mt][1] = 0.f;
                u[mt][0] = u[mt][1] = -INFINITY;
            }
            for (int i = 0; i < kQrStages; ++i)
                fill(sg, i);
            for (int i = 0;; ++i) {
                const int k0 = sg.lo0 + (i * kQrWarps + warp) * KS;
                if (k0 >= sg.hi0)
                    break;
                const int st = used % kQrStages;
                const uint32_t kb = ring + st * (2 * kQrTile);
                mbar_wait_warp(bar(st), (uint32_t)((used / kQrStages) & 1), abort_flag);
                // 8 keys at a time: rows g and g + 8 at keys 2t and 2t + 1, or key g at
                // rows 2t and 2t + 1 (with 8 keys of zeros behind them)
#pragma unroll 1
                for (int ks = k0; ks < min(k0 + KS, sg.hi0); ks += 8) {
                    uint32_t x[KW];
                    const int byte = t * (DH / 4);
                    qr_lds<KW>(kb + qr_place<DH>(ks - k0 + g, byte >> 4) + (byte & 15), x);
                    const float e = p.ks[(size_t)sg.kvhead * p.groups + (ks >> p.tshift)] * p.pp.scale_log2;
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        float s[4] = {};
#pragma unroll
                        for (int w = 0; w < KW; ++w) {
                            const uint32_t lo = half2_of_e4m3x2((uint16_t)x[w]);
                            const uint32_t hi = half2_of_e4m3x2((uint16_t)(x[w] >> 16));
                            if constexpr (kSwap) {
                                const uint32_t a[4] = {lo, 0, hi, 0};
                                mma_f16(s, a, qf[0][w][0], qf[0][w][1]);
                            } else {
                                mma_f16(s, qf[mt][w], lo, hi);
                            }
                        }
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            constexpr int N = kSwap ? 1 : 2; // keys of the row
                            const float a = fmaxf(e * qs[mt][h], 1.2e-38f);
                            float y[N], xm = -INFINITY;
#pragma unroll
                            for (int n = 0; n < N; ++n) {
                                y[n] = (ks + (kSwap ? g : 2 * t + n) < seen[mt][h] ? s[N * h + n] : -INFINITY) * a;
                                xm = fmaxf(xm, y[n]);
                            }
#pragma unroll
                            for (int w = kSwap ? 4 : 1; w < (kSwap ? 32 : 4); w <<= 1)
                                xm = fmaxf(xm, __shfl_xor_sync(0xffffffffu, xm, w));
                            if (xm > u[mt][h] + kQtLazy) {
                                l[mt][h] = u[mt][h] == -INFINITY ? l[mt][h] : l[mt][h] * ex2(u[mt][h] - xm);
                                u[mt][h] = xm;
                            }
#pragma unroll
                            for (int n = 0; n < N; ++n)
                                l[mt][h] += ex2(y[n] - (u[mt][h] == -INFINITY ? 0.f : u[mt][h]));
                        }
                    }
                }
                __syncwarp();
                ++used;
                fill(sg, i + kQrStages);
            }
        }
        // the next segment's first steps are on their way during the merge
        more = src.next(p.pp, nx);
        for (int i = 0; more && i < kQrStages; ++i)
            fill(nx, i);
        if (more) {
            load_queries(nx);
            scales(nx, nx.lo0 + warp * KS, es);
        }

#pragma unroll
        for (int mt = 0; mt < MT; ++mt) { // 16 (8) rows at a time
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float x = l[mt][h];
#pragma unroll
                for (int w = kSwap ? 4 : 1; w < (kSwap ? 32 : 4); w <<= 1)
                    x += __shfl_xor_sync(0xffffffffu, x, w);
                const int r = warp * S::kMerge + (kSwap ? 2 * t + h : h * 8 + g);
                float unit = u[mt][h];
                const float to_unit = qt_normalise(x, unit, m[mt][h]);
                if (kSwap ? g == 0 : t == 0)
                    s_ml[r] = make_float2(x, unit);
#pragma unroll
                for (int n = 0; n < NO; ++n) {
                    o[mt][n][kSwap ? h : 2 * h] *= to_unit;
                    o[mt][n][kSwap ? 2 + h : 2 * h + 1] *= to_unit;
                }
                float *dst = s_o + (size_t)r * kQrPitch + (kSwap ? g * (DH / 8) : t * (DH / 4));
                if constexpr (kSwap) {
#pragma unroll
                    for (int n = 0; n < NO; n += 2) // tile n: columns 2 n and 2 n + 1 of the thread's
                        *reinterpret_cast<float4 *>(dst + 2 * n) = make_float4(
                            o[mt][n][h], o[mt][n][2 + h], o[mt][n + 1][h], o[mt][n + 1][2 + h]);
                } else {
#pragma unroll
                    for (int n = 0; n < NT; n += 4) {
                        // column tile n holds columns NT 2t + n and NT (2t + 1) + n
                        *reinterpret_cast<float4 *>(dst + n) = make_float4(
                            o[mt][n][2 * h], o[mt][n + 1][2 * h], o[mt][n + 2][2 * h], o[mt][n + 3][2 * h]);
                        *reinterpret_cast<float4 *>(dst + NT + n) =
                            make_float4(o[mt][n][2 * h + 1], o[mt][n + 1][2 * h + 1], o[mt][n + 2][2 * h + 1],
                                        o[mt][n + 3][2 * h + 1]);
                    }
                }
            }
            __syncthreads();
            // 8 columns of a row at a time
            for (int e = threadIdx.x; e < min(S::kMerge, sg.nrows - mt * 16) * (DH / 8); e += kQrThreads) {
                const int r = e / (DH / 8), col = (e % (DH / 8)) * 8;
                float mx = -INFINITY;
#pragma unroll
                for (int w = 0; w < kQrWarps; ++w)
                    mx = fmaxf(mx, s_ml[w * S::kMerge + r].y);
                float ls = 0.f, acc[8] = {};
#pragma unroll
                for (int w = 0; w < kQrWarps; ++w) {
                    const float2 ml = s_ml[w * S::kMerge + r];
                    const float f = ml.y == -INFINITY ? 1.f : ex2(ml.y - mx);
                    ls = fmaf(ml.x, f, ls); // a NaN shows in l whatever its unit is
                    const float4 *x = reinterpret_cast<const float4 *>(s_o + (size_t)(w * S::kMerge + r) * kQrPitch + col);
                    const float4 y0 = x[0], y1 = x[1];
                    acc[0] = fmaf(y0.x, f, acc[0]); acc[1] = fmaf(y0.y, f, acc[1]);
                    acc[2] = fmaf(y0.z, f, acc[2]); acc[3] = fmaf(y0.w, f, acc[3]);
                    acc[4] = fmaf(y1.x, f, acc[4]); acc[5] = fmaf(y1.y, f, acc[5]);
                    acc[6] = fmaf(y1.z, f, acc[6]); acc[7] = fmaf(y1.w, f, acc[7]);
                }
                const float inv = ls == 0.f ? 0.f : 1.f / ls;
                const float lse = ls == 0.f ? -INFINITY : ((mx == -INFINITY ? 0.f : mx) + __log2f(ls)) * kLn2;
                const size_t grow = (size_t)sg.out_row0 + mt * 16 + r;
                const size_t prow = ((size_t)blockIdx.x * 2 + sg.slot) * kTcM + mt * 16 + r;
#pragma unroll
                for (int x = 0; x < 8; ++x)
                    acc[x] *= inv;
                if (sg.complete) {
                    *reinterpret_cast<uint4 *>(p.pp.out + grow * DH + col) =
                        make_uint4(pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3]),
                                   pack_bf16x2(acc[4], acc[5]), pack_bf16x2(acc[6], acc[7]));
                    if (col == 0)
                        p.pp.lse[grow] = lse;
                } else {
                    float4 *dst = reinterpret_cast<float4 *>(p.pp.part_o + prow * kTcD + col);
                    dst[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
                    dst[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
                    if (col == 0)
                        p.pp.part_lse[prow] = lse;
                }
            }
            __syncthreads();
        }
        if (!sg.complete && sg.last_cta >= 0 && threadIdx.x == 0)
            p.pp.cut_desc[blockIdx.x] = make_int4(sg.nrows, sg.last_cta, sg.out_row0, 0);
    }
    if (p.whole)
        q8_fill_empty_unit<DH>(p.pp);
    // wait (bounded) for copies that an aborted wait has left in flight
    const long long c0 = clock64();
    for (int x = max(issued - kQrStages, 0); x < issued; ++x)
        while (!mbar_try_wait(bar(x % kQrStages), (uint32_t)((x / kQrStages) & 1)) &&
               clock64() - c0 < kWaitCycles) {}
}

} // namespace bd
