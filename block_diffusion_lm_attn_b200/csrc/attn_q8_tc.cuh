// Block decode over a KV cache in 8 bits on the tensor cores (sm_100a).
//
// A value is a code times its group's scale, K = s_K c_K and V = s_V c_V, and
// the codes go through the tensor cores as they are; the scales, constant over
// 16 keys at least, are applied to the scores:
//     x_j   = log2(e) / sqrt(d) * s_K(j) 2^e (hi + lo) . c_K(j)
//     P_j   = 2^(x_j + log2 s_V(j) - M),  O = sum_j P_j c_V(j),
//     l     = sum_j P_j / s_V(j),         out = O / l,  lse = ln 2 (M + log2 l)
// for any M; M follows max_j (x_j + log2 s_V(j)), so that P fits 11 bits.  Where
// V's scales lie so far apart that a P beside M could be 0 in fp32 although its
// key has weight (kQtSpread), l is summed from 2^(x_j - U) instead, U following
// max_j x_j: a second exponential a score, in tiles that hardly a model has.
// (Looking for them costs 0.7 us of the 79 below, calls in a row.)
// A query row q = 2^e (hi + lo) is split into two e4m3 halves: hi rounds 2^-e q
// to 4 significant bits, lo rounds the rest to 4 more, together the 8 of a bf16
// for values from 2^-10 of the row's largest on; smaller ones are off by at most
// 2^-17 of the largest, where codes end.  (The kernel for few rows takes queries
// in f16, which holds these too.)  S = Q K^T is then two kind::f8f6f4 products straight on the codes in shared
// memory, at the price of one bf16 product.  V's codes become f16 (exact) on
// their way to the second product, since P needs more than e4m3's 4 bits.
//
// Persistent, one CTA per SM, over units of a sequence, a kv-head and 128
// query rows: whole ones, or equal ranges of 128-key tiles whose pieces
// bd_decode_q8_combine_kernel merges (QtSource).  Roles:
//   warps 0-3, 4-7  softmax, thread = query row = TMEM lane; the warpgroups
//                   take alternate key tiles, and the one without a segment's
//                   last tile splits the next segment's queries meanwhile
//   warp 8          the work list, TMA of K and V, cp.async of the scales
//   warps 9, 10     issue of QK, of PV
//   warps 12-15     V codes to f16
// TMEM: S (128 columns), a P in f16 (64) and an O (128) for each warpgroup.
// Shared memory: Q (hi and lo, 16 KB each), four stages of K and three of V (16
// KB), two buffers of V in f16 (32 KB).
//
// S goes to registers at once, 128 a thread, and with it read the next QK may run:
// one S serves both warpgroups.  Each has an O, a running maximum and a sum of
// its own, joined in the epilogue, so that no tile waits for another's softmax.
//
// Bound: a tile takes 1900 cycles.  Its exponentials alone are 1024 (the two
// warpgroups' overlap and take 1980 together), its products 1150, its shared-memory
// traffic of 176 KB 1400, its bytes at the measured HBM rate 1385; without the
// exponentials, without the conversion, with half of either product it would
// still be 1750 to 1800 each: what is left are hand-overs, 100 to 250 cycles each.
// Calls in a row are bound by the card's power: 1600 MHz.  Also built: S and P in
// the same columns with two S, one warp for both products, two for the
// conversion (2 us more, of 81); one O, the maximum handed from warpgroup to
// warpgroup (every raise of it stops both); every tile shared by the warpgroups,
// 64 keys each (twice the waits and arrivals a key); a quarter of the
// exponentials on the FMA pipe, or integer operations for the conversion (no
// gain, and 2 us more).
// Measured: 16 sequences over 8192 keys, 32 query heads on 8, blocks of 32, d =
// 128: 78 us, 3.5 TB/s and 880 TFLOP/s (bf16 counting: QK runs as two products
// of half the price); 94 us where calls in a row hold the card at its power
// limit.
#pragma once

#include "attn_tc_persist.cuh"
#include "cache_q8.cuh"

namespace bd {

constexpr int kQtThreads = 512;
constexpr int kQtTile = kTcN * kTcD; // bytes of a key tile's codes
constexpr int kQtKStages = 4, kQtVStages = 3;

// shared-memory layout (offsets from a 1024-byte aligned base)
constexpr int kQtSmemQ = 0; // hi, lo
constexpr int kQtSmemK = kQtSmemQ + 2 * kQtTile;
constexpr int kQtSmemV = kQtSmemK + kQtKStages * kQtTile;
constexpr int kQtSmemW = kQtSmemV + kQtVStages * kQtTile; // V in f16: 2 buffers
constexpr int kQtSmemSc = kQtSmemW + 2 * kTileBytes; // 8 tiles: 8 scales of K, 8 of V
constexpr int kQtSmemL = kQtSmemSc + 8 * 64;         // (l, u, 2^(M - u)) [2][2][128]
constexpr int kQtSmemQs = kQtSmemL + 4 * kTcM * 16;       // row scales of Q [2][128]
constexpr int kQtSmemSeg = kQtSmemQs + 2 * kTcM * 4;      // 4 segments, 128 B each
constexpr int kQtSmemBar = kQtSmemSeg + 4 * 128;
constexpr int kQtSmemBytes = kQtSmemBar + 512 + 1024; // + alignment slack
static_assert(kQtSmemBytes <= 227 * 1024, "more shared memory than a CTA may have");

// The work list, walked by one converged warp.  It is DecSource's (units x
// tiles, cut into equal ranges, or whole units) but for four things.  The warp
// reads 32 lengths at a time (one after another they took 3 us for 16
// sequences and 8 us for 64, at the head of every launch).  No more CTAs take
// part than there are tiles, so that the merge of a short launch walks over no
// empty pieces.  Units stay whole where the longest is at most 12 tiles above
// the mean of the CTAs, about what a second segment and the merge cost (blocks of
// 32 over 8192 keys, d = 128, 15 and 16 sequences of 8 kv-heads, 12.3 and 8.8
// tiles above: whole 77.1 and 78.0 us, cut 76.1 and 80.5; one sequence of 2
// kv-heads, 777 keys, d = 64, 6 above: 8.5 and 10.5).  And a range is not so
// many tiles, but so much work: behind each unit's tiles lie TAIL positions for
// what a segment costs besides its tiles (verification over 64 ragged prefixes,
// CTAs with 2 to 10 segments: 206 us without, 178 us with 4 to 6).
constexpr int kQtWhole = 12;

template <int TAIL>
struct QtSource {
    long long t, t1, t0, T; // positions: next, end and start of this CTA's, all
    long long seq_base;
    int seq, seq_tiles, len, G;

    // a * b / c, and a / b with the rest; 64-bit divisions, some 100 cycles
    // each, only where the numbers ask for them
    __device__ static long long muldiv(long long a, int b, long long c)
    {
        const long long x = a * b;
        return (x | c) >> 31 ? x / c : (long long)((unsigned)x / (unsigned)c);
    }
    __device__ static int divmod(long long a, int b, int &rest)
    {
        if (a >> 31) {
            rest = (int)(a % b);
            return (int)(a / b);
        }
        rest = (int)((unsigned)a % (unsigned)b);
        return (int)((unsigned)a / (unsigned)b);
    }
    __device__ static int tiles_of(const PParams &p, int i, int &len)
    {
        len = i < p.B ? p.cache_len[i] : 0;
        return i < p.B ? max(0, decode_unit_tiles(len, p.b, p.nkeys, p.mode)) : 0;
    }
    // positions of a unit of so many tiles
    __device__ static int span(int tiles) { return tiles ? tiles + TAIL : 0; }
    __device__ void init(const PParams &p)
    {
        const int lane = threadIdx.x & 31;
        const int ups = p.Hkv * p.row_tiles; // units per sequence
        long long sum = 0, sum_pos = 0;
        int maxt = 0, n, first = 0; // tiles of sequence `lane`
        for (int i = lane; i < p.B; i += 32) {
            const int ti = tiles_of(p, i, n);
            first = i == lane ? ti : first;
            sum += ti;
            sum_pos += span(ti);
            maxt = max(maxt, ti);
        }
        if (p.B <= 32) { // tiles of a sequence are below 2^23
            sum = __reduce_add_sync(0xffffffffu, (unsigned)sum);
            sum_pos = __reduce_add_sync(0xffffffffu, (unsigned)sum_pos);
        } else {
#pragma unroll
            for (int o = 16; o; o >>= 1) {
                sum += __shfl_xor_sync(0xffffffffu, sum, o);
                sum_pos += __shfl_xor_sync(0xffffffffu, sum_pos, o);
            }
        }
        maxt = __reduce_max_sync(0xffffffffu, maxt);
        const long long tiles = sum * ups, units = (long long)p.B * ups;
        T = sum_pos * ups;
        G = (int)min((long long)gridDim.x, max(tiles, 1LL));
        t = t0 = t1 = seq_base = 0;
        seq = seq_tiles = len = 0;
        if (units <= gridDim.x && (long long)(maxt - kQtWhole) * G <= tiles) {
            // CTA c takes unit c
            if (blockIdx.x < units) {
                seq = blockIdx.x / ups;
                seq_tiles = tiles_of(p, seq, len);
                t = t0 = (long long)(blockIdx.x % ups) * span(seq_tiles);
                t1 = t0 + span(seq_tiles);
            }
            return;
        }
        if ((int)blockIdx.x >= G)
            return;
        t = t0 = muldiv(T, blockIdx.x, G);
        t1 = muldiv(T, blockIdx.x + 1, G);
        // the sequence that holds position t0 < T
        for (int i0 = 0; i0 < p.B; i0 += 32) {
            const long long mine = (long long)span(i0 ? tiles_of(p, i0 + lane, n) : first) * ups;
            long long incl = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long up = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o)
                    incl += up;
            }
            const int before = __popc(__ballot_sync(0xffffffffu, seq_base + incl <= t0));
            if (before < 32) {
                seq_base += __shfl_sync(0xffffffffu, incl - mine, before);
                seq = i0 + before;
                break;
            }
            seq_base += __shfl_sync(0xffffffffu, incl, 31);
        }
        seq_tiles = tiles_of(p, seq, len);
    }
    __device__ bool next(const PParams &p, Seg &sg)
    {
        const int ups = p.Hkv * p.row_tiles;
        for (;;) {
            if (t >= t1)
                return false;
            while (t >= seq_base + (long long)ups * span(seq_tiles)) {
                seq_base += (long long)ups * span(seq_tiles);
                seq_tiles = tiles_of(p, ++seq, len);
            }
            int kt0; // first tile in the unit `uis` of the sequence
            const int uis = divmod(t - seq_base, span(seq_tiles), kt0);
            const long long u0 = t - kt0; // the unit's first position
            if (kt0 >= seq_tiles) { // behind its tiles
                t = u0 + span(seq_tiles);
                continue;
            }
            const int n = (int)min((long long)(seq_tiles - kt0), t1 - t);
            t += n;
            const int g = uis / p.row_tiles, rt = uis % p.row_tiles;
            sg.kvhead = seq * p.Hkv + g;
            sg.qrow0 = rt * kTcM;
            sg.nrows = min(kTcM, p.rows_unit - rt * kTcM);
            sg.lo0 = kt0 * kTcN;
            sg.hi0 = min((kt0 + n) * kTcN, len + decode_own_keys(p.b, p.mode));
            sg.fhi0 = len + (p.mode == 0 ? p.b : 0);
            sg.nt = n;
            sg.len = len;
            sg.out_row0 = (seq * p.Hq + g * (p.Hq / p.Hkv)) * p.b + rt * kTcM;
            sg.complete = n == seq_tiles;
            sg.slot = u0 < t0 ? 0 : 1;
            // range x starts at floor(T x / G), so the last x starting at or
            // before position e is floor(((e + 1) G - 1) / T)
            sg.last_cta = -1;
            if (!sg.complete && sg.slot == 1) {
                const long long e = (u0 + seq_tiles) * G - 1;
                sg.last_cta = (e | T) >> 31 ? (int)(e / T) : (int)((unsigned)e / (unsigned)T);
            }
            return true;
        }
    }
};

struct QtParams {
    PParams pp; // sizes, outputs and scratch, as the bf16 decode's
    const bf16 *q;
    const float *ks, *vs; // [B * Hkv, groups]
    int groups, tshift;   // log2 of the positions per group
    int whole;            // no unit can be cut: CTA c takes unit c, nothing is merged
};

// A unit without a key tile, by the CTA that has it, where no second kernel
// fills such rows: an invalid length gives NaN rows, an empty prefix in mode 2
// rows with no visible key (out 0, lse -inf).
template <int DH> __device__ __forceinline__ void q8_fill_empty_unit(const PParams &p)
{
    const int ups = p.Hkv * p.row_tiles, seq = blockIdx.x / ups;
    const int tiles = decode_unit_tiles(p.cache_len[seq], p.b, p.nkeys, p.mode);
    if (tiles > 0)
        return;
    const int uis = blockIdx.x % ups, g = uis / p.row_tiles, rt = uis % p.row_tiles;
    const size_t row0 = ((size_t)seq * p.Hq + g * (p.Hq / p.Hkv)) * p.b + rt * kTcM;
    const int nrows = min(kTcM, p.rows_unit - rt * kTcM);
    for (int e = threadIdx.x; e < nrows * DH; e += blockDim.x)
        p.out[row0 * DH + e] = __float2bfloat16_rn(tiles < 0 ? NAN : 0.f);
    for (int r = threadIdx.x; r < nrows; r += blockDim.x)
        p.lse[row0 + r] = tiles < 0 ? NAN : -INFINITY;
    if (threadIdx.x == 0 && tiles < 0)
        raise_device_code(DEV_BAD_CACHE_LEN);
}

// D[tmem] (+)= A[smem desc] * B[smem desc] of e4m3 codes
__device__ __forceinline__ void tc_mma8_ss_p(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                             uint32_t idesc, uint32_t accumulate, uint32_t leader)
{
    asm volatile("{\n\t.reg .pred p, q;\n\t"
                 "setp.ne.b32 p, %4, 0;\n\t"
                 "setp.ne.b32 q, %5, 0;\n\t"
                 "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
                 "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(leader)
                 : "memory");
}

// Instruction descriptor with fp32 accumulators and format 0 operands: e4m3
// in kind::f8f6f4, f16 in kind::f16.
__host__ __device__ constexpr uint32_t idesc_fmt0(int M, int N, int b_mn)
{
    return (1u << 4) | ((uint32_t)b_mn << 16) | ((uint32_t)(N >> 3) << 17) |
           ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ float lg2(float x)
{
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// P is an operand of the tensor cores beside V, so 16 bits: f16, since its 11
// bits show in out and bf16's 8 would show eight times as much.  P reaches
// 2^kQtTop where the maximum was last raised, and 2^(kQtTop + kQtLazy) before it
// is raised again.  2^15 is the largest power of two in f16; below 2^-17 of the
// largest P, at worst, the smaller ones are rounded to multiples of 2^-27 of it.
// What n keys lose so is at most n 2^-28 of the largest: with 2^17 keys 2^-11, no
// more than P's other rounding, with 2^20 keys 2^-8, as out's own (and only if
// the errors all point one way).  A raise stops the warpgroup for some 1000
// cycles: with 6 and 8, heads of large scores took 1.3 us a tile where others took
// 1.1.  l is the sum of P before its rounding, in fp32: lse loses nothing.
constexpr float kQtTop = 3.f, kQtLazy = 12.f;

// l may be summed from P as long as no weight of consequence is 0 in P.  With
// V's scales 2^w apart at most, x the score (in log2) of a key and X the row's
// largest, its P is 2^(x - X - w + kQtTop) or more: above fp32's 2^-126, at w =
// 72, for weights from 2^-57 of the largest on.  A raise of M by more than 126,
// which takes the sum before it to 0, asks for scores 126 - w - kQtLazy = 42
// apart.  Both bounds hold what 2^30 keys can lose below 2^-12.  Counting from
// 2^-8 keeps 1 / s_V, and with it l over 2^30 keys, in range too: V's scales
// from 2^-80 to 2^64 take the sum from P if they lie no further apart.
constexpr float kQtSpread = 4722366482869645213696.f; // 2^72
constexpr float kQtMidScale = 1.f / 256;

// A finished run's sum of weights, l 2^u, as l in [1, 2) (0 without a visible
// key, NaN stays) and an exponent u that a float holds; returns what O, in units
// of 2^m, is multiplied by to be in units of 2^u.
__device__ __forceinline__ float qt_normalise(float &l, float &u, float m)
{
    const bool some = l > 0.f && l < INFINITY;
    const int k = some ? min((int)(__float_as_uint(l) >> 23) - 127, 126) : 0;
    const float f = some ? ex2(m - u - (float)k) : 1.f;
    l *= exp2_int(-k);
    u += (float)k;
    return f;
}

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t *r)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

// 16 columns of tensor memory, with their wait
__device__ __forceinline__ void tmem_ld16_wait(uint32_t a0, uint32_t *r)
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {"
                 "%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
                 "tcgen05.wait::ld.sync.aligned;"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
                   "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
                   "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(a0)
                 : "memory");
}

// two halves to two e4m3 codes, as e4m3x2
__device__ __forceinline__ uint16_t e4m3x2_of_half2(uint32_t x)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(x));
    return r;
}
__device__ __forceinline__ uint32_t half2_sub(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// The smallest exponent of a query row's scale: 2^k and 2^-k stay normal.  A row of
// the smallest normal values, 2^-126, is then still split from 1 on, and with K's
// largest scale has scores that count.
constexpr int kQtMinQExp = -126;

// A query row (thread = row) as two halves of e4m3 codes, hi and lo, in the
// 128-byte swizzle of 128-byte rows at `dst` and `dst` + kQtTile; returns the
// row's scale.
template <int DH>
__device__ __forceinline__ float qt_split_row(const bf16 *src, bool valid, uint32_t dst, int row)
{
    uint4 w[DH / 8];
#pragma unroll
    for (int i = 0; i < DH / 8; ++i)
        w[i] = valid ? reinterpret_cast<const uint4 *>(src)[i] : make_uint4(0, 0, 0, 0);
    uint32_t top = 0; // non-negative bf16 order as their bits do
#pragma unroll
    for (int i = 0; i < DH / 8; ++i) {
        top = umax_u16x2(top, umax_u16x2(w[i].x & 0x7fff7fffu, w[i].y & 0x7fff7fffu));
        top = umax_u16x2(top, umax_u16x2(w[i].z & 0x7fff7fffu, w[i].w & 0x7fff7fffu));
    }
    const float amax = fmaxf(__uint_as_float(top << 16), __uint_as_float(top & 0xffff0000u));
    const bool finite = (top & 0xffffu) < 0x7f80u && (top >> 16) < 0x7f80u;
    // 2^-k q reaches 448 at most
    const int k = q8_scale_exp(finite ? amax : 0.f, kQtMinQExp);
    const float inv = finite ? exp2_int(-k) : NAN;
#pragma unroll
    for (int c = 0; c < DH / 16; ++c) { // 16 codes of each half
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint4 v = w[2 * c + i];
            const uint32_t ws[4] = {v.x, v.y, v.z, v.w};
            uint32_t h[4], r[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                // f16 holds 8 bits of everything that a code can show of it
                const uint32_t x = pack_f16x2(__uint_as_float(ws[t] << 16) * inv,
                                              __uint_as_float(ws[t] & 0xffff0000u) * inv);
                h[t] = e4m3x2_of_half2(x);
                r[t] = e4m3x2_of_half2(half2_sub(x, half2_of_e4m3x2((uint16_t)h[t])));
            }
            hi[2 * i] = h[0] | h[1] << 16;
            hi[2 * i + 1] = h[2] | h[3] << 16;
            lo[2 * i] = r[0] | r[1] << 16;
            lo[2 * i + 1] = r[2] | r[3] << 16;
        }
        const uint32_t at = dst + row * 128 + ((c ^ (row & 7)) << 4);
        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(hi[0]), "r"(hi[1]),
                     "r"(hi[2]), "r"(hi[3]) : "memory");
        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at + kQtTile), "r"(lo[0]),
                     "r"(lo[1]), "r"(lo[2]), "r"(lo[3]) : "memory");
    }
    return finite ? exp2_int(k) : NAN;
}

// Bounded wait by a converged warp, as mbar_wait_warp, with one vote a poll and
// no divergent path in between: the kernel waits about 20 times a tile.
__device__ __forceinline__ bool qt_wait(uint32_t bar, uint32_t parity, volatile int *abort_flag)
{
    if (__builtin_expect(__all_sync(0xffffffffu, mbar_try_wait(bar, parity)), 1))
        return true;
    const long long t0 = clock64();
    for (;;) {
        if (__all_sync(0xffffffffu, mbar_try_wait_sleep(bar, parity, BD_WAIT_SLEEP_NS)))
            return true;
        if (__any_sync(0xffffffffu, *abort_flag))
            return false;
        if (__any_sync(0xffffffffu, clock64() - t0 > kWaitCycles)) {
            *abort_flag = 1;
            raise_device_code(DEV_WAIT_TIMEOUT);
            return false;
        }
    }
}

// NG: scales a tile has of K and of V each, 128 / (positions per group).
template <int DH, int NG>
__global__ void __launch_bounds__(kQtThreads, 1)
    bd_decode_q8_tc_kernel(const __grid_constant__ CUtensorMap tm_k,
                           const __grid_constant__ CUtensorMap tm_v, const QtParams p)
{
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = smem_u32(smem_raw);
    const uint32_t base = (raw_addr + 1023u) & ~1023u;
    uint8_t *sbase = smem_raw + (base - raw_addr);

    const uint32_t bar0 = base + kQtSmemBar;
    auto bar_kfull = [&](int s) { return bar0 + 8 * s; };
    auto bar_kempty = [&](int s) { return bar0 + 32 + 8 * s; };
    auto bar_vfull = [&](int s) { return bar0 + 64 + 8 * s; };
    auto bar_vempty = [&](int s) { return bar0 + 88 + 8 * s; };
    auto bar_ifull = [&](int s) { return bar0 + 112 + 8 * s; };  // segment si & 3
    auto bar_iempty = [&](int s) { return bar0 + 144 + 8 * s; };
    auto bar_sfull = [&](int w) { return bar0 + 176 + 8 * w; };  // S, of a tile j with j & 1 = w
    auto bar_pv = [&](int w) { return bar0 + 192 + 8 * w; };     // its P, its V in f16
    auto bar_odone = [&](int w) { return bar0 + 208 + 8 * w; };  // its PV done
    auto bar_qfull = [&](int s) { return bar0 + 224 + 8 * s; };  // queries of segment si & 1
    const uint32_t bar_l = bar0 + 240;     // both sums of a segment written
    const uint32_t bar_ofree = bar0 + 248; // both O read out
    const uint32_t bar_final = bar0 + 256;
    const uint32_t bar_sfree = bar0 + 264; // S read by its warpgroup
    static_assert(kQtKStages == 4 && kQtVStages == 3, "barrier layout");
    volatile int *abort_flag = reinterpret_cast<volatile int *>(sbase + kQtSmemBar + 272);
    volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(sbase + kQtSmemBar + 280);
    Seg *seg_ring = reinterpret_cast<Seg *>(sbase + kQtSmemSeg); // nt = 0: no more
    float4 *s_l = reinterpret_cast<float4 *>(sbase + kQtSmemL);
    float *s_qs = reinterpret_cast<float *>(sbase + kQtSmemQs);
    const float *s_sc = reinterpret_cast<const float *>(sbase + kQtSmemSc);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < 4; ++s) {
            mbar_init(bar_kfull(s), 1 + 2 * NG); // + a copy of each scale
            mbar_init(bar_kempty(s), 1);
            mbar_init(bar_ifull(s), 1);
            mbar_init(bar_iempty(s), 14); // 8 softmax warps, QK, PV, 4 converters
        }
        for (int s = 0; s < 3; ++s) {
            mbar_init(bar_vfull(s), 1);
            mbar_init(bar_vempty(s), 4);
        }
        for (int w = 0; w < 2; ++w) {
            mbar_init(bar_sfull(w), 1);
            mbar_init(bar_pv(w), 4 + 4); // softmax warps, converters
            mbar_init(bar_odone(w), 1);
            mbar_init(bar_qfull(w), 4);
        }
        mbar_init(bar_l, 256);
        mbar_init(bar_ofree, 8);
        mbar_init(bar_final, 2);
        mbar_init(bar_sfree, 4);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == 8 && lane < 2) // the first copy would wait for its map
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(lane ? &tm_v : &tm_k)) : "memory");
    if (warp == 9) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32((const void *)tmem_slot)), "r"(512));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const uint32_t t_p = tmem + 128, t_o = tmem + 256; // 64 and 128 columns a warpgroup
    // the combine kernel may be scheduled now; it reads nothing of this
    // launch before the whole grid has finished
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // a barrier wait by a converged warp
    auto wait = [&](uint32_t bar, uint32_t parity) { return qt_wait(bar, parity, abort_flag); };

    // the end of a warp that issued products: wait (bounded) for all of both
    auto drain = [&](uint32_t ld) {
        tc_commit_p(bar_final, ld);
        const long long c0 = clock64();
        while (!mbar_try_wait(bar_final, 0) && clock64() - c0 < kWaitCycles) {}
        __syncwarp();
    };

    // Registers: a softmax thread holds a row of S, 128.  2 x 128 x (184 + 72) is
    // what the launch has, 512 x 128.
    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        if (warp == 8) {
            // -------------------------- work list; loads of K, V and the scales
            QtSource<5> src;
            src.init(p.pp);
            if (lane == 0)
                p.pp.cut_desc[blockIdx.x] = make_int4(0, 0, 0, 0);
            Seg sg;
            bool ok = true;
            int g = 0, vs = 0;           // running tile counter, its V stage
            uint32_t vpar = 1;           // parity of the wait for that stage
            int kiss = 0, viss = 0;      // tiles issued
            for (int si = 0; ok; ++si) {
                const int slot = si & 3;
                if (si >= 4 && !(ok = wait(bar_iempty(slot), (uint32_t)(((si - 4) >> 2) & 1))))
                    break;
                const bool got = src.next(p.pp, sg);
                if (lane == 0) {
                    if (got)
                        seg_ring[slot] = sg;
                    else
                        seg_ring[slot].nt = 0;
                    mbar_arrive(bar_ifull(slot));
                }
                __syncwarp();
                if (!got)
                    break;
                // its queries, which a warpgroup reads when the segment before is
                // all but done
                if (si > 0)
                    for (int e = lane * 128; e < sg.nrows * DH * 2; e += 32 * 128)
                        asm volatile("prefetch.global.L2 [%0];" ::"l"(
                            reinterpret_cast<const char *>(p.q + (size_t)sg.out_row0 * DH) + e));
                for (int it = 0; it < sg.nt; ++it, ++g) {
                    const int ks = sg.lo0 + it * kTcN, s = g & 3;
                    if (g >= 4 && !(ok = wait(bar_kempty(s), (uint32_t)((g >> 2) & 1) ^ 1u)))
                        break;
                    // injected fault: this tile never arrives
                    const bool skip = g == 0 && blockIdx.x == 0 && lane == 0 &&
                                      atomicExch(&g_fault_skip_k, 0) != 0;
                    if (lane == 0 && !skip) {
                        mbar_expect_tx(bar_kfull(s), kQtTile);
                        tma_load_3d(base + kQtSmemK + s * kQtTile, &tm_k, 0, ks, sg.kvhead, bar_kfull(s));
                        kiss = g + 1;
                    }
                    // Scales: one lane each, K's first.  Groups with no visible key
                    // give 0, which no visible score is multiplied by.  A slot is
                    // taken again 8 tiles on, behind QK_{g-4}, so behind the load
                    // of S_{g-6} and the softmax of tile g - 8 before it.
                    if (lane < 2 * NG) {
                        const int key = ks + (kTcN / NG) * (lane % NG);
                        const bool in = key < sg.hi0;
                        const float *from = (lane < NG ? p.ks : p.vs) + (size_t)sg.kvhead * p.groups +
                                            (in ? key / (kTcN / NG) : 0);
                        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(
                                         base + kQtSmemSc + (g & 7) * 64 + (lane / NG) * 32 + (lane % NG) * 4),
                                     "l"(from), "r"(in ? 4 : 0)
                                     : "memory");
                        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(
                                         bar_kfull(s))
                                     : "memory");
                    }
                    if (g >= kQtVStages && !(ok = wait(bar_vempty(vs), vpar)))
                        break;
                    if (lane == 0) {
                        mbar_expect_tx(bar_vfull(vs), kQtTile);
                        tma_load_3d(base + kQtSmemV + vs * kQtTile, &tm_v, 0, ks, sg.kvhead, bar_vfull(vs));
                        viss = g + 1;
                    }
                    __syncwarp();
                    if (++vs == kQtVStages) {
                        vs = 0;
                        vpar ^= 1;
                    }
                }
            }
            // wait (bounded) for every copy this role issued
            asm volatile("cp.async.wait_all;" ::: "memory");
            if (lane == 0) {
                const long long c0 = clock64();
                for (int x = max(kiss - kQtKStages, 0); x < kiss; ++x)
                    while (!mbar_try_wait(bar_kfull(x & 3), (uint32_t)((x >> 2) & 1)) &&
                           clock64() - c0 < kWaitCycles) {}
                for (int x = max(viss - kQtVStages, 0); x < viss; ++x)
                    while (!mbar_try_wait(bar_vfull(x % kQtVStages), (uint32_t)((x / kQtVStages) & 1)) &&
                           clock64() - c0 < kWaitCycles) {}
            }
        } else if (warp == 9) {
            // ---------------------------------------------------- issue of QK
            const uint32_t ld = elect_one();
            constexpr uint32_t idesc_qk = idesc_fmt0(kTcM, kTcN, 0);
            bool ok = true;
            int j = 0;
            for (int si = 0; ok; ++si) {
                if (!(ok = wait(bar_ifull(si & 3), (uint32_t)((si >> 2) & 1))))
                    break;
                const int n = seg_ring[si & 3].nt;
                if (n == 0 || !(ok = wait(bar_qfull(si & 1), (uint32_t)((si >> 1) & 1))))
                    break;
                for (int i = 0; i < n; ++i, ++j) {
                    // K is there, and S of tile j - 1 has been read
                    if (!(ok = wait(bar_kfull(j & 3), (uint32_t)((j >> 2) & 1))) ||
                        (j > 0 && !(ok = wait(bar_sfree, (uint32_t)((j - 1) & 1)))))
                        break;
                    tc_fence_after();
                    const uint32_t qb = base + kQtSmemQ, kb = base + kQtSmemK + (uint32_t)(j & 3) * kQtTile;
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int kk = 0; kk < DH / 32; ++kk)
                            tc_mma8_ss_p(tmem, smem_desc_sw128(qb + h * kQtTile + kk * 32, 16, 1024),
                                         smem_desc_sw128(kb + kk * 32, 16, 1024), idesc_qk,
                                         h || kk ? 1u : 0u, ld);
                    tc_commit_p(bar_sfull(j & 1), ld);
                    tc_commit_p(bar_kempty(j & 3), ld);
                }
                __syncwarp();
                if (ok && lane == 0)
                    mbar_arrive(bar_iempty(si & 3));
            }
            drain(ld);
        } else if (warp == 10) {
            // ---------------------------------------------------- issue of PV
            const uint32_t ld = elect_one();
            // O has DH columns; a 64-column half of V at least
            constexpr uint32_t idesc_pv = idesc_fmt0(kTcM, DH > 64 ? 128 : 64, 1);
            bool ok = true;
            int j = 0;
            for (int si = 0; ok; ++si) {
                if (!(ok = wait(bar_ifull(si & 3), (uint32_t)((si >> 2) & 1))))
                    break;
                const int n = seg_ring[si & 3].nt;
                // O was last read out by the epilogue of segment si - 1
                if (n == 0 || (si >= 1 && !(ok = wait(bar_ofree, (uint32_t)((si - 1) & 1)))))
                    break;
                for (int i = 0; i < n; ++i, ++j) {
                    const int w = j & 1;
                    if (!(ok = wait(bar_pv(w), (uint32_t)((j >> 1) & 1))))
                        break;
                    tc_fence_after();
                    const uint32_t vb = base + kQtSmemW + (uint32_t)w * kTileBytes;
#pragma unroll
                    for (int kk = 0; kk < kTcN / 16; ++kk)
                        tc_mma_ts_p(t_o + w * 128, t_p + w * 64 + kk * 8,
                                    smem_desc_sw128(vb + kk * 2048, kHalfTileBytes, 1024), idesc_pv,
                                    (i > 1 || kk > 0) ? 1u : 0u, ld);
                    tc_commit_p(bar_odone(w), ld);
                }
                __syncwarp();
                if (ok && lane == 0)
                    mbar_arrive(bar_iempty(si & 3));
            }
            drain(ld);
        } else if (warp >= 12) {
            // ------------------------------------------------ V codes to f16
            const int cw = warp - 12;
            bool ok = true;
            int j = 0, vs = 0;
            uint32_t vpar = 0;
            for (int si = 0; ok; ++si) {
                if (!(ok = wait(bar_ifull(si & 3), (uint32_t)((si >> 2) & 1))))
                    break;
                const Seg &sg = seg_ring[si & 3];
                const int nt = sg.nt, lo = sg.lo0, hi = sg.hi0;
                __syncwarp();
                if (nt == 0)
                    break;
                if (lane == 0)
                    mbar_arrive(bar_iempty(si & 3));
                for (int it = 0; it < nt; ++it, ++j) {
                    const int b = j & 1, ks = lo + it * kTcN;
                    // the f16 buffer was last read by the PV of tile j - 2
                    if (!(ok = wait(bar_vfull(vs), vpar)) ||
                        (j >= 2 && !(ok = wait(bar_odone(b), (uint32_t)(((j - 2) >> 1) & 1)))))
                        break;
                    // 8 lanes take half a row each of rows r and r ^ 5 (64 codes
                    // = 4 vectors of 16): their reads of the swizzled codes and
                    // their writes of the swizzled halves each cover all banks.
                    const uint32_t src = base + kQtSmemV + (uint32_t)vs * kQtTile;
                    const uint32_t dst = base + kQtSmemW + (uint32_t)b * kTileBytes;
                    // rows of 8: pairs (0, 5), (2, 7), (4, 1), (6, 3)
                    const int hrow = (lane >> 3) * 2;
                    const int r8 = (lane & 4) ? (hrow ^ 5) : hrow;
                    const int u4 = lane & 3;
                    constexpr int H = DH <= 64 ? 1 : 2; // halves of 64 columns
                    const int rr = 32 * cw; // this warp's rows
                    uint32_t x[4 * H][4]; // all loads go out first
#pragma unroll
                    for (int i = 0; i < 4 * H; ++i) {
                        const int r = rr + 8 * (i / H) + r8;
                        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                     : "=r"(x[i][0]), "=r"(x[i][1]), "=r"(x[i][2]), "=r"(x[i][3])
                                     : "r"(src + r * 128 + ((((i % H) * 4 + u4) ^ r8) << 4))
                                     : "memory");
                    }
                    if (ks + rr + 32 > hi) { // not keys: no code of theirs may be used
#pragma unroll
                        for (int i = 0; i < 4 * H; ++i)
                            if (ks + rr + 8 * (i / H) + r8 >= hi)
                                x[i][0] = x[i][1] = x[i][2] = x[i][3] = 0;
                    }
#pragma unroll
                    for (int i = 0; i < 4 * H; ++i) {
                        uint32_t y[8];
#pragma unroll
                        for (int t = 0; t < 8; ++t)
                            y[t] = half2_of_e4m3x2((uint16_t)(x[i][t >> 1] >> (16 * (t & 1))));
                        const uint32_t row = dst + (i % H) * kHalfTileBytes + (rr + 8 * (i / H) + r8) * 128;
                        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(
                                         row + (((2 * u4) ^ r8) << 4)),
                                     "r"(y[0]), "r"(y[1]), "r"(y[2]), "r"(y[3])
                                     : "memory");
                        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(
                                         row + (((2 * u4 + 1) ^ r8) << 4)),
                                     "r"(y[4]), "r"(y[5]), "r"(y[6]), "r"(y[7])
                                     : "memory");
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(bar_pv(b));
                        mbar_arrive(bar_vempty(vs));
                    }
                    if (++vs == kQtVStages) {
                        vs = 0;
                        vpar ^= 1;
                    }
                }
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
        // ------------------------------------------- softmax and epilogue
        const int wg = warp >> 2;
        const int row = threadIdx.x & (kTcM - 1);
        const int wrow = row & ~31; // first row of this warp
        const uint32_t lane_off = (uint32_t)wrow << 16;
        const uint32_t ts = tmem + lane_off;
        const uint32_t tp = t_p + wg * 64 + lane_off;    // this warpgroup's P
        const uint32_t t_ow = t_o + wg * 128 + lane_off;   // and O
        // The queries of segment si, by one warpgroup, into the buffer that
        // no QK reads any more.
        auto split = [&](int si) -> bool {
            if (!wait(bar_ifull(si & 3), (uint32_t)((si >> 2) & 1)))
                return false;
            const Seg &sg = seg_ring[si & 3];
            if (sg.nt == 0)
                return true;
            s_qs[(si & 1) * kTcM + row] = qt_split_row<DH>(
                p.q + ((size_t)sg.out_row0 + row) * DH, row < sg.nrows, base + kQtSmemQ, row);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0)
                mbar_arrive(bar_qfull(si & 1));
            return true;
        };
        bool ok = wg == 0 || split(0);
        int j0 = 0; // tile of the CTA at the segment's start
        for (int si = 0; ok; ++si) {
            if (!(ok = wait(bar_ifull(si & 3), (uint32_t)((si >> 2) & 1))))
                break;
            const Seg &sg = seg_ring[si & 3];
            const int n = sg.nt;
            if (n == 0)
                break;
            if (!(ok = wait(bar_qfull(si & 1), (uint32_t)((si >> 1) & 1))))
                break;
            const float qs = s_qs[(si & 1) * kTcM + row] * p.pp.scale_log2;
            const int nrows = sg.nrows, lo = sg.lo0, hi = sg.hi0;
            const int full_end = min(sg.fhi0, hi); // keys that every row sees
            const int jr = (sg.qrow0 + min(row, nrows - 1)) % p.pp.b;
            // keys that this row sees
            const int seen = min(hi, sg.len + (p.pp.mode == 0 ? p.pp.b : p.pp.mode == 1 ? jr + 1 : 0));
            const bool live = wrow < nrows; // a warp without rows only arrives
            float m = -INFINITY, l = 0.f; // running maximum (raised lazily), sum
            float vmin = kQtMidScale, vmax = kQtMidScale; // V's scales so far
            float u = INFINITY; // finite once they lie far apart: l is in units of 2^u, not 2^m
            for (int i = (j0 ^ wg) & 1; i < n; i += 2) {
                const int j = j0 + i; // tile
                if (!(ok = wait(bar_sfull(wg), (uint32_t)((j >> 1) & 1))))
                    break;
                // PV_{j-2}, which reads P and writes O.  (It is waited for here by
                // every warp and for every tile: no phase can be mistaken.)
                auto prev_done = [&] { return ok = i < 2 || wait(bar_odone(wg), (uint32_t)(((j - 2) >> 1) & 1)); };
                if (live) {
                    tc_fence_after();
                    uint32_t sr[kTcN];
                    tmem_ld32x4_wait(ts, ts + 32, ts + 64, ts + 96, sr, sr + 32, sr + 64, sr + 96);
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(bar_sfree);
                    float s[kTcN];
#pragma unroll
                    for (int c = 0; c < kTcN; ++c)
                        s[c] = __uint_as_float(sr[c]);
                    const int ks = lo + i * kTcN;
                    if (ks + kTcN > full_end) {
#pragma unroll
                        for (int w = 0; w < kTcN / 32; ++w) {
                            const uint32_t mk = range_bits(0, seen - ks - 32 * w);
#pragma unroll
                            for (int c = 0; c < 32; ++c)
                                s[32 * w + c] = ((mk >> c) & 1u) ? s[32 * w + c] : -INFINITY;
                        }
                    }
                    // the scales, as the multiplier of the scores and as the
                    // term that P has from V; a masked score has to stay -inf,
                    // so the product is no less than 2^-126 (where x is 0
                    // anyway)
                    float ea[NG], ev[NG];
                    const float *sc = s_sc + (j & 7) * 16;
                    float mt = -INFINITY;
#pragma unroll
                    for (int c = 0; c < NG; ++c) {
                        const bool in = ks + c * (kTcN / NG) < hi;
                        ea[c] = fmaxf(sc[c] * qs, 1.2e-38f);
                        ev[c] = in ? sc[8 + c] : kQtMidScale;
                        vmin = fminf(vmin, ev[c]);
                        vmax = fmaxf(vmax, ev[c]);
                        const float *x = s + c * (kTcN / NG);
                        float mc[2] = {fmaxf(x[0], x[1]), fmaxf(x[2], x[3])};
#pragma unroll
                        for (int y = 4; y < kTcN / NG; y += 4) {
                            mc[0] = fmax3(mc[0], x[y], x[y + 1]);
                            mc[1] = fmax3(mc[1], x[y + 2], x[y + 3]);
                        }
                        mt = fmaxf(mt, fmaf(fmaxf(mc[0], mc[1]), ea[c], lg2(ev[c])));
                    }
                    if (!prev_done())
                        break;
                    tc_fence_after();
                    const bool need = mt > m + (kQtTop + kQtLazy);
                    const bool wide = vmax > vmin * kQtSpread; // and so from here on
                    if (__any_sync(0xffffffffu, need || wide)) {
                        if (__builtin_expect(wide, 0)) { // the sum apart
                            float xm = -INFINITY;
#pragma unroll
                            for (int c = 0; c < kTcN; ++c)
                                xm = fmaxf(xm, s[c] * ea[c / (kTcN / NG)]);
                            u = u < INFINITY ? u : m;
                            if (xm > u + kQtLazy) {
                                l = u == -INFINITY ? l : l * ex2(u - xm);
                                u = xm;
                            }
                            const float nu = u == -INFINITY ? 0.f : -u;
#pragma unroll
                            for (int c = 0; c < kTcN; ++c)
                                l += ex2(fmaf(s[c], ea[c / (kTcN / NG)], nu));
                        }
                        float c = 1.f;
                        if (need) {
                            c = m == -INFINITY ? 0.f : ex2(m - (mt - kQtTop));
                            l = m == -INFINITY || wide ? l : l * c; // 0, or NaN for good
                            m = mt - kQtTop;
                        }
                        // the TMEM read-modify-write of O is warp-collective
                        if (i > 1) {
#pragma unroll 1
                            for (int q4 = 0; q4 < DH / 16; ++q4) {
                                uint32_t o[16];
                                tmem_ld16_wait(t_ow + q4 * 16, o);
#pragma unroll
                                for (int x = 0; x < 16; ++x)
                                    o[x] = __float_as_uint(__uint_as_float(o[x]) * c);
                                tmem_st16(t_ow + q4 * 16, o);
                            }
                        }
                    }
                    const float nm = m == -INFINITY ? 0.f : -m;
#pragma unroll
                    for (int c = 0; c < NG; ++c) {
                        constexpr int W = kTcN / NG;
                        const float o = lg2(ev[c]) + nm;
                        float r0 = 0.f, r1 = 0.f, r2 = 0.f, r3 = 0.f;
                        uint32_t pk[W / 2];
#pragma unroll
                        for (int x = 0; x < W; x += 4) {
                            float y0, y1, y2, y3;
                            ffma2(y0, y1, s[c * W + x], s[c * W + x + 1], ea[c], ea[c], o, o);
                            ffma2(y2, y3, s[c * W + x + 2], s[c * W + x + 3], ea[c], ea[c], o, o);
                            y0 = ex2(y0);
                            y1 = ex2(y1);
                            y2 = ex2(y2);
                            y3 = ex2(y3);
                            fadd2(r0, r1, r0, r1, y0, y1);
                            fadd2(r2, r3, r2, r3, y2, y3);
                            pk[x / 2] = pack_f16x2(y0, y1);
                            pk[x / 2 + 1] = pack_f16x2(y2, y3);
                            // stored 32 keys at a time (16: a group of them)
                            if (W >= 32 && (x & 31) == 28)
                                tmem_st16(tp + c * (W / 2) + (x & ~31) / 2, pk + (x & ~31) / 2);
                        }
                        if (W == 16)
                            tmem_st8(tp + c * 8, pk);
                        l = fmaf((r0 + r1) + (r2 + r3), wide ? 0.f : 1.f / ev[c], l);
                    }
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                } else {
                    if (lane == 0)
                        mbar_arrive(bar_sfree);
                    if (!prev_done())
                        break;
                }
                if (lane == 0)
                    mbar_arrive(bar_pv(wg));
            }
            if (!ok)
                break;
            const int jl = j0 + n - 1; // last tile of the segment
            // The warpgroup without it readies the next queries, once the last
            // QK has finished (QK_{jl-1}, which it has seen, is behind QK_{jl-2}:
            // the wait cannot mistake that phase).
            if ((jl & 1) != wg &&
                (!(ok = wait(bar_sfull(jl & 1), (uint32_t)((jl >> 1) & 1))) || !(ok = split(si + 1))))
                break;
            u = u < INFINITY ? u : m;
            const float to_u = qt_normalise(l, u, m);
            s_l[((si & 1) * 2 + wg) * kTcM + row] = make_float4(l, u, to_u, 0.f);
            mbar_arrive(bar_l);
            // The last PV.  (The phase before on that barrier, PV_{jl-2}, was
            // waited for by the warpgroup of tile jl before it arrived here.)
            if (!(ok = wait(bar_l, (uint32_t)(si & 1))) ||
                !(ok = wait(bar_odone(jl & 1), (uint32_t)((jl >> 1) & 1))))
                break;
            tc_fence_after();
            // factors of the two O to the common exponent; with one tile, one O
            // is unwritten
            const float4 l0 = s_l[(si & 1) * 2 * kTcM + row], l1 = s_l[((si & 1) * 2 + 1) * kTcM + row];
            const bool use0 = n > 1 || (j0 & 1) == 0, use1 = n > 1 || (j0 & 1) == 1;
            const float mx = fmaxf(l0.y, l1.y);
            const float f0 = l0.y == -INFINITY ? 1.f : ex2(l0.y - mx);
            const float f1 = l1.y == -INFINITY ? 1.f : ex2(l1.y - mx);
            const float ls = l0.x * f0 + l1.x * f1; // a NaN shows in l whatever u is
            const float inv = ls == 0.f ? 0.f : 1.f / ls;
            const float w0 = l0.z * (f0 * inv), w1 = l1.z * (f1 * inv);
            const bool valid = row < nrows;
            const size_t grow = (size_t)sg.out_row0 + row;
            const size_t prow = ((size_t)blockIdx.x * 2 + sg.slot) * kTcM + row;
            constexpr int kCols = DH >= 64 ? DH / 2 : DH; // columns of O a warpgroup takes
            if (live && (DH >= 64 || wg == 0)) {
#pragma unroll 1
                for (int q4 = 0; q4 < kCols / 32; ++q4) {
                    const int col = wg * kCols + q4 * 32;
                    uint32_t o[32], o1[32];
                    tmem_ld32x2_wait(t_o + lane_off + col, t_o + 128 + lane_off + col, o, o1);
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const float x = use0 ? __uint_as_float(o[i]) * w0 : 0.f;
                        o[i] = __float_as_uint(use1 ? fmaf(__uint_as_float(o1[i]), w1, x) : x);
                    }
                    if (sg.complete) {
                        if (valid) {
                            bf16 *dst = p.pp.out + grow * DH + col;
#pragma unroll
                            for (int i = 0; i < 32; i += 16) {
                                uint32_t y[8];
#pragma unroll
                                for (int x = 0; x < 8; ++x)
                                    y[x] = pack_bf16x2(__uint_as_float(o[i + 2 * x]), __uint_as_float(o[i + 2 * x + 1]));
                                st32(dst + i, y);
                            }
                        }
                    } else {
                        // column by column: 128 contiguous bytes a warp, where
                        // 16 bytes of each of 32 rows would be as many
                        // transactions as rows
                        float *dst = p.pp.part_o + ((size_t)blockIdx.x * 2 + sg.slot) * (kTcM * kTcD) +
                                     (size_t)col * kTcM + row;
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            dst[i * kTcM] = __uint_as_float(o[i]);
                    }
                }
            }
            if (valid && wg == 0)
                (sg.complete ? p.pp.lse + grow : p.pp.part_lse + prow)[0] =
                    ls == 0.f ? -INFINITY : ((mx == -INFINITY ? 0.f : mx) + __log2f(ls)) * kLn2;
            if (!sg.complete && sg.last_cta >= 0 && threadIdx.x == 0)
                p.pp.cut_desc[blockIdx.x] = make_int4(nrows, sg.last_cta, sg.out_row0, 0);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(bar_ofree);
                mbar_arrive(bar_iempty(si & 3));
            }
            j0 += n;
        }
    }

    if (p.whole)
        q8_fill_empty_unit<DH>(p.pp);
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
    }
}

// Merges the pieces of the units that range boundaries cut, and fills the rows
// of sequences without a tile, as bd_decode_stream_combine_kernel does, from
// pieces that lie column by column ([128 columns][128 rows]): lane = row, a
// warp takes 16 columns, so every load is one line of 128 bytes.  Grid (G, 4):
// CTA (c, rg) takes rows 32 rg .. 32 rg + 31 of the unit of descriptor c.
// Launched as a programmatic dependent of the attention kernel.
template <int DH>
__global__ void __launch_bounds__(16 * DH / 8) bd_decode_q8_combine_kernel(const PParams p)
{
    const int c = blockIdx.x, rg = blockIdx.y;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (rg == 0) { // an invalid length: NaN rows; mode 2 over nothing: out 0, lse -inf
        for (int i = c; i < p.B; i += gridDim.x) {
            const int tiles = decode_unit_tiles(p.cache_len[i], p.b, p.nkeys, p.mode);
            if (tiles > 0)
                continue;
            const size_t row0 = (size_t)i * p.Hq * p.b;
            for (long long e = threadIdx.x; e < (long long)p.Hq * p.b * DH; e += blockDim.x)
                p.out[row0 * DH + e] = __float2bfloat16_rn(tiles < 0 ? NAN : 0.f);
            for (int r = threadIdx.x; r < p.Hq * p.b; r += blockDim.x)
                p.lse[row0 + r] = tiles < 0 ? NAN : -INFINITY;
            if (threadIdx.x == 0 && tiles < 0)
                raise_device_code(DEV_BAD_CACHE_LEN);
        }
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int4 desc = p.cut_desc[c];
    const int last = desc.y, row = rg * 32 + lane;
    if (rg * 32 >= desc.x)
        return;
    float m = -INFINITY, z = 0.f, acc[16];
#pragma unroll
    for (int i = 0; i < 16; ++i)
        acc[i] = 0.f;
    for (int x = c; x <= last; ++x) {
        const size_t piece = (size_t)x * 2 + (x == c ? 1 : 0);
        const float ls = p.part_lse[piece * kTcM + row];
        const float *src = p.part_o + piece * (kTcM * kTcD) + (size_t)warp * 16 * kTcM + row;
        float v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i)
            v[i] = src[i * kTcM];
        if (ls == -INFINITY)
            continue; // no visible key in this piece
        const float mn = fmaxf(m, ls);
        const float a = ex2((m - mn) * kLog2e); // 0 while m is -inf
        const float w = ex2((ls - mn) * kLog2e);
        z = z * a + w;
#pragma unroll
        for (int i = 0; i < 16; ++i)
            acc[i] = acc[i] * a + w * v[i];
        m = mn;
    }
    if (row >= desc.x)
        return;
    const float inv = z == 0.f ? 0.f : 1.f / z;
    uint32_t y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        y[i] = pack_bf16x2(acc[2 * i] * inv, acc[2 * i + 1] * inv);
    st32(p.out + ((size_t)desc.z + row) * DH + warp * 16, y);
    if (warp == 0)
        p.lse[(size_t)desc.z + row] = z == 0.f ? -INFINITY : m + __logf(z);
}

} // namespace bd
