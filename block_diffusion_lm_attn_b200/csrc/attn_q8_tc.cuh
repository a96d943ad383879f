// Block decode over a KV cache in 8 bits on the tensor cores (sm_100a).
//
// A value is a code times its group's scale, K = s_K c_K and V = s_V c_V, and
// the codes go through the tensor cores as they are; the scales, constant over
// 16 keys at least, are applied to the scores:
//     x_j   = log2(e) / sqrt(d) * s_K(j) 2^e (hi + lo) . c_K(j)
//     P_j   = 2^(x_j + log2 s_V(j) - M),  O = sum_j P_j c_V(j),
//     l     = sum_j P_j / s_V(j),         out = O / l,  lse = ln 2 (M + log2 l)
// for any M; M follows max_j (x_j + log2 s_V(j)), so that P fits 11 bits.
// A query row q = 2^e (hi + lo) is split into two e4m3 halves: hi rounds 2^-e q
// to 4 significant bits, lo rounds the rest to 4 more, which a bf16 has.  S =
// Q K^T is then two kind::f8f6f4 products straight on the codes in shared
// memory, at the price of one bf16 product.  V's codes become f16 (exact) on
// their way to the second product, since P needs more than e4m3's 4 bits.
//
// Persistent, one CTA per SM, over units of a sequence, a kv-head and 128
// query rows: whole ones, or equal ranges of 128-key tiles whose pieces
// bd_decode_stream_combine_kernel merges (QtSource).  Roles:
//   warps 0-3, 4-7  softmax, thread = query row = TMEM lane; one warpgroup
//                   takes the first 64 keys of every tile, one the last
//   warp 8          the work list, TMA of K
//   warp 9          MMA issue: the QK of a tile, then the PVs of the tile
//                   before, over segment boundaries
//   warp 10         TMA of V, cp.async of the scales
//   warps 12-15     V codes to f16; the table of scales; at the end of a
//                   segment the next one's queries
// TMEM: S of one tile (128 columns), P of the two halves (f16, 32 each), an O
// for each warpgroup (128 each), Q (hi and lo, 32 each).
//
// A warpgroup reads its half of S into registers at once, so the next tile's
// QK runs under its exponentials, and keeps an O, a running maximum and a sum
// of its own: the two meet only in the epilogue, which joins them.  (With one
// O and the maximum handed from step to step a step took 2500 cycles, a third
// of them for the hand-over and the wait for S.)
#pragma once

#include "attn_tc_persist.cuh"
#include "cache_q8.cuh"

namespace bd {

constexpr int kQtThreads = 512;

constexpr int kQtTile = kTcN * kTcD; // bytes of a key tile's codes
constexpr int kQtKStages = 4, kQtVStages = 4;
constexpr int kQtChunks = kTcN / 16; // runs of 16 keys: one scale each
constexpr int kQtStep = 64;          // keys per softmax step: two steps a tile

// shared-memory layout (offsets from a 1024-byte aligned base)
constexpr int kQtSmemK = 0;
constexpr int kQtSmemV = kQtSmemK + kQtKStages * kQtTile;
constexpr int kQtSmemW = kQtSmemV + kQtVStages * kQtTile; // V in f16: 2 buffers
constexpr int kQtSmemRaw = kQtSmemW + 2 * kTileBytes;     // scales, 16 a stage
constexpr int kQtSmemTab = kQtSmemRaw + kQtVStages * 64;  // 4 tables of 8 float4
constexpr int kQtSmemL = kQtSmemTab + 4 * kQtChunks * 16; // (l, M) [2][2][128]
constexpr int kQtSmemQs = kQtSmemL + 4 * kTcM * 8;        // row scales of Q [2][128]
constexpr int kQtSmemSeg = kQtSmemQs + 2 * kTcM * 4;      // 4 segments, 128 B each
constexpr int kQtSmemBar = kQtSmemSeg + 4 * 128;
constexpr int kQtSmemBytes = kQtSmemBar + 512 + 1024; // + alignment slack
static_assert(kQtSmemBytes <= 227 * 1024, "more shared memory than a CTA may have");

// The work list, walked by one converged warp.  It is DecSource's (units x
// tiles, cut into equal ranges, or whole units) but for three things: the
// warp reads 32 lengths at a time (one after another they took 3 us for 16
// sequences and 8 us for 64, at the head of every launch); no more CTAs take
// part than there are tiles, so that the merge of a short launch walks over no
// empty pieces; and units stay whole only where the longest is at most 3 tiles
// above the mean of the CTAs, about what merging costs.
struct QtSource {
    long long t, t1, t0, T;
    long long seq_base;
    int seq, seq_tiles, len, G;

    __device__ static int tiles_of(const PParams &p, int i, int &len)
    {
        len = i < p.B ? p.cache_len[i] : 0;
        return i < p.B ? max(0, decode_unit_tiles(len, p.b, p.nkeys, p.mode)) : 0;
    }
    __device__ void init(const PParams &p)
    {
        const int lane = threadIdx.x & 31;
        const int ups = p.Hkv * p.row_tiles; // units per sequence
        long long sum = 0;
        int maxt = 0, n;
        for (int i = lane; i < p.B; i += 32) {
            const int ti = tiles_of(p, i, n);
            sum += ti;
            maxt = max(maxt, ti);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1)
            sum += __shfl_xor_sync(0xffffffffu, sum, o);
        maxt = __reduce_max_sync(0xffffffffu, maxt);
        T = sum * ups;
        G = (int)min((long long)gridDim.x, max(T, 1LL));
        const long long units = (long long)p.B * ups;
        t = t0 = t1 = seq_base = 0;
        seq = seq_tiles = len = 0;
        if (units <= gridDim.x && (long long)(maxt - 3) * G <= T) {
            // CTA c takes unit c
            if (blockIdx.x < units) {
                seq = blockIdx.x / ups;
                seq_tiles = tiles_of(p, seq, len);
                t = t0 = (long long)(blockIdx.x % ups) * seq_tiles;
                t1 = t0 + seq_tiles;
            }
            return;
        }
        if ((int)blockIdx.x >= G)
            return;
        t = t0 = range_start(T, G, blockIdx.x);
        t1 = range_start(T, G, blockIdx.x + 1);
        // the sequence that holds tile t0 < T
        for (int i0 = 0; i0 < p.B; i0 += 32) {
            const long long mine = (long long)tiles_of(p, i0 + lane, n) * ups;
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
        if (t >= t1)
            return false;
        const int ups = p.Hkv * p.row_tiles;
        while (t >= seq_base + (long long)ups * seq_tiles) {
            seq_base += (long long)ups * seq_tiles;
            seq_tiles = tiles_of(p, ++seq, len);
        }
        const long long local = t - seq_base;
        const int uis = (int)(local / seq_tiles); // unit inside the sequence
        const int kt0 = (int)(local % seq_tiles);
        const int n = (int)min((long long)(seq_tiles - kt0), t1 - t);
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
        const long long u0 = seq_base + (long long)uis * seq_tiles;
        sg.slot = u0 < t0 ? 0 : 1;
        // range x starts at floor(T x / G), so the last x starting at or
        // before tile e is floor(((e + 1) G - 1) / T)
        sg.last_cta = !sg.complete && sg.slot == 1 ? (int)(((u0 + seq_tiles) * G - 1) / T) : -1;
        t += n;
        return true;
    }
};

struct QtParams {
    PParams pp; // sizes, outputs and scratch, as the bf16 decode's
    const bf16 *q;
    const float *ks, *vs; // [B * Hkv, groups]
    int groups, tshift;   // log2 of the positions per group
};

// D[tmem] (+)= A[tmem] * B[smem desc] of e4m3 codes
__device__ __forceinline__ void tc_mma8_ts_p(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                             uint32_t idesc, uint32_t accumulate, uint32_t leader)
{
    asm volatile("{\n\t.reg .pred p, q;\n\t"
                 "setp.ne.b32 p, %4, 0;\n\t"
                 "setp.ne.b32 q, %5, 0;\n\t"
                 "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
                 "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(leader)
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

// P reaches 2^kQtTop where the maximum was last raised, and 2^(kQtTop +
// kQtLazy) before it is raised again: the largest f16 is above 2^15, and the
// smallest normal one then 2^-20 of the row's largest P.
constexpr float kQtTop = 6.f, kQtLazy = 8.f;

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t *r)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

// A query row as two halves of e4m3 codes, and its scale.
template <int DH>
__device__ __forceinline__ float qt_split_row(const bf16 *src, bool valid, uint32_t *hi, uint32_t *lo)
{
    const uint4 *row = reinterpret_cast<const uint4 *>(src);
    uint4 w[DH / 8];
#pragma unroll
    for (int i = 0; i < DH / 8; ++i)
        w[i] = valid ? row[i] : make_uint4(0, 0, 0, 0);
    float amax = 0.f;
    bool finite = true;
#pragma unroll
    for (int i = 0; i < DH / 8; ++i) {
        const uint32_t ws[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const float a = fabsf(__uint_as_float(ws[t] << 16));
            const float b = fabsf(__uint_as_float(ws[t] & 0xffff0000u));
            finite = finite && a < INFINITY && b < INFINITY;
            amax = fmax3(amax, a, b);
        }
    }
    // 2^-k q reaches 448 at most; k stays where 2^k and 2^-k are normal
    const int k = max(q8_scale_exp(finite ? amax : 0.f), -100);
    const float inv = finite ? exp2_int(-k) : NAN;
#pragma unroll
    for (int i = 0; i < DH / 8; ++i) {
        const uint32_t ws[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
        uint32_t h[4], r[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const float a = __uint_as_float(ws[t] << 16) * inv;
            const float b = __uint_as_float(ws[t] & 0xffff0000u) * inv;
            h[t] = e4m3x2(a, b);
            const float2 f = float2_of_e4m3x2((uint16_t)h[t]);
            r[t] = e4m3x2(a - f.x, b - f.y);
        }
        hi[2 * i] = h[0] | h[1] << 16;
        hi[2 * i + 1] = h[2] | h[3] << 16;
        lo[2 * i] = r[0] | r[1] << 16;
        lo[2 * i + 1] = r[2] | r[3] << 16;
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

template <int DH>
__global__ void __launch_bounds__(kQtThreads, 1)
    bd_decode_q8_tc_kernel(const __grid_constant__ CUtensorMap tm_k,
                           const __grid_constant__ CUtensorMap tm_v, const QtParams p)
{
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = smem_u32(smem_raw);
    const uint32_t base = (raw_addr + 1023u) & ~1023u;
    uint8_t *sbase = smem_raw + (base - raw_addr);

    const uint32_t bar0 = base + kQtSmemBar;
    // What the MMAs of a tile wait for arrives on one barrier each: for the QK
    // of tile j, K and the reads of S of tile j - 1; for its PVs, P of both
    // warpgroups and V in f16.
    auto bar_qk = [&](int s) { return bar0 + 8 * s; };          // tile j & 3
    auto bar_kempty = [&](int s) { return bar0 + 32 + 8 * s; };
    auto bar_vfull = [&](int s) { return bar0 + 64 + 8 * s; };
    auto bar_vempty = [&](int s) { return bar0 + 96 + 8 * s; };
    auto bar_ifull = [&](int s) { return bar0 + 128 + 8 * s; }; // segment si & 3
    auto bar_iempty = [&](int s) { return bar0 + 160 + 8 * s; };
    auto bar_pv = [&](int s) { return bar0 + 192 + 8 * s; };    // tile j & 1
    auto bar_odone = [&](int s) { return bar0 + 208 + 8 * s; }; // PVs of tile j & 1 done
    // S of tile j & 1, its scales and those of the queries: one buffer of S,
    // but the converters arrive up to a tile ahead
    auto bar_sfull = [&](int s) { return bar0 + 224 + 8 * s; };
    const uint32_t bar_qfull = bar0 + 240;
    const uint32_t bar_qfree = bar0 + 248; // last QK of a segment done
    const uint32_t bar_l = bar0 + 256;     // both sums of a segment written
    const uint32_t bar_ofree = bar0 + 264; // both O read out
    const uint32_t bar_final = bar0 + 272;
    static_assert(kQtKStages == 4 && kQtVStages == 4, "barrier layout");
    volatile int *abort_flag = reinterpret_cast<volatile int *>(sbase + kQtSmemBar + 288);
    volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(sbase + kQtSmemBar + 296);
    Seg *seg_ring = reinterpret_cast<Seg *>(sbase + kQtSmemSeg); // nt = 0: no more
    float2 *s_l = reinterpret_cast<float2 *>(sbase + kQtSmemL);
    float *s_qs = reinterpret_cast<float *>(sbase + kQtSmemQs);
    float4 *s_tab = reinterpret_cast<float4 *>(sbase + kQtSmemTab);
    const float *s_raw = reinterpret_cast<const float *>(sbase + kQtSmemRaw);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < 4; ++s) {
            mbar_init(bar_qk(s), 1 + 8); // TMA, softmax warps
            mbar_init(bar_kempty(s), 1);
            mbar_init(bar_vfull(s), 1 + 2 * kQtChunks); // + a copy of each scale
            mbar_init(bar_vempty(s), 3);
            mbar_init(bar_ifull(s), 1);
            mbar_init(bar_iempty(s), 14); // 8 softmax warps, MMA, V, 4 converters
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(bar_pv(s), 8 + 3); // softmax warps, converters
            mbar_init(bar_odone(s), 1);
            mbar_init(bar_sfull(s), 5); // the MMA, 4 converters
        }
        mbar_init(bar_qfull, 4);
        mbar_init(bar_qfree, 1);
        mbar_init(bar_l, 256);
        mbar_init(bar_ofree, 8);
        mbar_init(bar_final, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == 9) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32((const void *)tmem_slot)), "r"(512));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const uint32_t t_p = tmem + 128, t_o = tmem + 192, t_q = tmem + 448;
    // the combine kernel may be scheduled now; it reads nothing of this
    // launch before the whole grid has finished
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // a barrier wait by a converged warp
    auto wait = [&](uint32_t bar, uint32_t parity) { return qt_wait(bar, parity, abort_flag); };

    if (warp == 8) {
        // ------------------------------------------ work list, loads of K
        QtSource src;
        src.init(p.pp);
        if (lane == 0)
            p.pp.cut_desc[blockIdx.x] = make_int4(0, 0, 0, 0);
        // an empty range (more CTAs than tiles) contributes an empty piece
        // to any cut unit that spans it
        if (src.t0 == src.t1)
            for (int r = lane; r < kTcM; r += 32)
                p.pp.part_lse[(size_t)blockIdx.x * 2 * kTcM + r] = -INFINITY;
        Seg sg;
        bool ok = true;
        int g = 0; // running tile counter
        int kiss = 0;
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
            for (int it = 0; it < sg.nt; ++it, ++g) {
                const int s = g & 3;
                if (g >= 4 && !(ok = wait(bar_kempty(s), (uint32_t)((g >> 2) & 1) ^ 1u)))
                    break;
                // injected fault: this tile never arrives
                const bool skip = g == 0 && blockIdx.x == 0 && lane == 0 &&
                                  atomicExch(&g_fault_skip_k, 0) != 0;
                if (lane == 0 && !skip) {
                    mbar_expect_tx(bar_qk(s), kQtTile);
                    tma_load_3d(base + kQtSmemK + s * kQtTile, &tm_k, 0, sg.lo0 + it * kTcN, sg.kvhead,
                                bar_qk(s));
                    kiss = g + 1;
                }
                __syncwarp();
            }
        }
        // wait (bounded) for every copy this role issued
        if (lane == 0) {
            const long long c0 = clock64();
            for (int x = kiss > 4 ? kiss - 4 : 0; x < kiss; ++x)
                while (!mbar_try_wait(bar_qk(x & 3), (uint32_t)((x >> 2) & 1)) &&
                       clock64() - c0 < kWaitCycles) {}
        }
    } else if (warp == 10) {
        // ------------------------------------- loads of V and the scales
        bool ok = true;
        int g = 0, viss = 0;
        for (int si = 0; ok; ++si) {
            if (!(ok = wait(bar_ifull(si & 3), (uint32_t)((si >> 2) & 1))))
                break;
            const Seg &sg = seg_ring[si & 3];
            const int nt = sg.nt, lo = sg.lo0, hi = sg.hi0, head = sg.kvhead;
            __syncwarp();
            if (nt == 0)
                break;
            if (lane == 0)
                mbar_arrive(bar_iempty(si & 3));
            for (int it = 0; it < nt; ++it, ++g) {
                const int ks = lo + it * kTcN;
                const int s = g & 3;
                if (g >= 4 && !(ok = wait(bar_vempty(s), (uint32_t)((g >> 2) & 1) ^ 1u)))
                    break;
                if (lane == 0) {
                    mbar_expect_tx(bar_vfull(s), kQtTile);
                    tma_load_3d(base + kQtSmemV + s * kQtTile, &tm_v, 0, ks, head, bar_vfull(s));
                    viss = g + 1;
                }
                // lanes 0-7: scales of K, 8-15: of V; chunks with no visible
                // key read nothing
                if (lane < 2 * kQtChunks) {
                    const int key = ks + 16 * (lane & 7);
                    const bool in = key < hi;
                    const float *src = (lane < 8 ? p.ks : p.vs) + (size_t)head * p.groups +
                                       (in ? key >> p.tshift : 0);
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(
                                     base + kQtSmemRaw + s * 64 + lane * 4),
                                 "l"(src), "r"(in ? 4 : 0)
                                 : "memory");
                    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(
                                     bar_vfull(s))
                                 : "memory");
                }
                __syncwarp();
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        if (lane == 0) {
            const long long c0 = clock64();
            for (int x = viss > 4 ? viss - 4 : 0; x < viss; ++x)
                while (!mbar_try_wait(bar_vfull(x & 3), (uint32_t)((x >> 2) & 1)) &&
                       clock64() - c0 < kWaitCycles) {}
        }
    } else if (warp == 9) {
        // ---------------------------------------------------- MMA issue
        const uint32_t ld = elect_one();
        constexpr uint32_t idesc_qk = idesc_fmt0(kTcM, kTcN, 0);
        // O has DH columns; a 64-column half of V at least
        constexpr uint32_t idesc_pv = idesc_fmt0(kTcM, DH > 64 ? 128 : 64, 1);
        bool ok = true;
        // cursor of the QKs: tile qj of the CTA, tile qi of the qn of its segment qs
        int qj = 0, qi = 0, qn = 0, qs = 0;
        auto next_qk = [&]() { // the next tile's QK, if there is one
            if (qi == qn) {
                if (!(ok = wait(bar_ifull(qs & 3), (uint32_t)((qs >> 2) & 1))))
                    return;
                qn = seg_ring[qs & 3].nt;
                qi = 0;
                if (qn == 0 || !(ok = wait(bar_qfull, (uint32_t)(qs & 1))))
                    return;
                ++qs;
            }
            const int s = qj & 3;
            if (!(ok = wait(bar_qk(s), (uint32_t)((qj >> 2) & 1))))
                return;
            tc_fence_after();
            const uint32_t kb = base + kQtSmemK + (uint32_t)s * kQtTile;
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int kk = 0; kk < DH / 32; ++kk)
                    tc_mma8_ts_p(tmem, t_q + h * 32 + kk * 8, smem_desc_sw128(kb + kk * 32, 16, 1024),
                                 idesc_qk, h || kk ? 1u : 0u, ld);
            tc_commit_p(bar_sfull(qj & 1), ld);
            tc_commit_p(bar_kempty(s), ld);
            ++qj;
            if (++qi == qn)
                tc_commit_p(bar_qfree, ld);
        };
        next_qk();
        int j = 0; // tile of the PVs
        for (int si = 0; ok && j < qj; ++si) {
            // known, as its first QK was issued
            const int n = seg_ring[si & 3].nt, hi = seg_ring[si & 3].hi0 - seg_ring[si & 3].lo0;
            for (int i = 0; i < n; ++i, ++j) {
                next_qk();
                const int b = j & 1;
                // O was last read out by the epilogue of segment si - 1
                if (!ok || (i == 0 && si >= 1 && !(ok = wait(bar_ofree, (uint32_t)((si - 1) & 1)))) ||
                    !(ok = wait(bar_pv(b), (uint32_t)((j >> 1) & 1))))
                    break;
                tc_fence_after();
                const uint32_t vb = base + kQtSmemW + (uint32_t)b * kTileBytes;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    // (the last tile may have no key in its second half)
                    if (half == 1 && i * kTcN + kQtStep >= hi)
                        break;
#pragma unroll
                    for (int kk = 0; kk < kQtStep / 16; ++kk)
                        tc_mma_ts_p(t_o + half * 128, t_p + half * 32 + kk * 8,
                                    smem_desc_sw128(vb + half * (kQtStep * 128) + kk * 2048,
                                                    kHalfTileBytes, 1024),
                                    idesc_pv, (i > 0 || kk > 0) ? 1u : 0u, ld);
                }
                tc_commit_p(bar_odone(b), ld);
            }
            __syncwarp();
            if (ok && lane == 0)
                mbar_arrive(bar_iempty(si & 3));
        }
        tc_commit_p(bar_final, ld);
        const long long c0 = clock64();
        while (!mbar_try_wait(bar_final, 0) && clock64() - c0 < kWaitCycles) {}
        __syncwarp();
    } else if (warp >= 12) {
        // ------- V codes to f16, the table of scales, the split of queries
        const int cw = warp - 12;
        const int row = 32 * cw + lane;
        // The queries of segment si; the buffer was last read by the QKs of
        // the segment before.
        auto split = [&](int si) -> bool {
            if (!wait(bar_ifull(si & 3), (uint32_t)((si >> 2) & 1)))
                return false;
            const Seg &sg = seg_ring[si & 3];
            if (sg.nt == 0)
                return true;
            uint32_t hi[DH / 4], lo[DH / 4];
            const float qs =
                qt_split_row<DH>(p.q + ((size_t)sg.out_row0 + row) * DH, row < sg.nrows, hi, lo);
            // behind the last QK of segment si - 1, which was issued behind
            // the reads of every earlier segment's S and row scales
            if (si >= 1 && !wait(bar_qfree, (uint32_t)((si - 1) & 1)))
                return false;
            s_qs[(si & 1) * kTcM + row] = qs;
            tc_fence_after();
            const uint32_t tq = t_q + ((uint32_t)(32 * cw) << 16);
#pragma unroll
            for (int c = 0; c < DH / 32; ++c) {
                tmem_st8(tq + 8 * c, hi + 8 * c);
                tmem_st8(tq + 32 + 8 * c, lo + 8 * c);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(bar_qfull);
            return true;
        };
        bool ok = split(0);
        int j = 0;
        for (int si = 0; ok; ++si) {
            if (!(ok = wait(bar_ifull(si & 3), (uint32_t)((si >> 2) & 1))))
                break;
            const Seg &sg = seg_ring[si & 3];
            const int nt = sg.nt, lo = sg.lo0, hi = sg.hi0;
            if (nt == 0)
                break;
            for (int it = 0; it < nt; ++it, ++j) {
                const int s = j & 3, ks = lo + it * kTcN;
                if (cw != 1 && !(ok = wait(bar_vfull(s), (uint32_t)((j >> 2) & 1))))
                    break;
                // the f16 buffer was last read by the PVs of tile j - 2;
                // the softmax of that tile lies behind them
                const int b = j & 1;
                if (j >= 2 && !(ok = wait(bar_odone(b), (uint32_t)(((j - 2) >> 1) & 1))))
                    break;
                if (cw == 0) {
                    if (lane < kQtChunks) {
                        float4 e = make_float4(1.f, 0.f, 0.f, 0.f);
                        if (ks + 16 * lane < hi) {
                            const float sv = s_raw[s * 16 + 8 + lane];
                            e.x = s_raw[s * 16 + lane] * p.pp.scale_log2;
                            e.y = lg2(sv);
                            e.z = 1.f / sv;
                        }
                        s_tab[(j & 3) * kQtChunks + lane] = e;
                    }
                }
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(bar_sfull(b));
                // 8 lanes take half a row each of rows r and r ^ 5 (64 codes
                // = 4 vectors of 16): their reads of the swizzled codes and
                // their writes of the swizzled halves each cover all banks.
                const uint32_t src = base + kQtSmemV + (uint32_t)s * kQtTile;
                const uint32_t dst = base + kQtSmemW + (uint32_t)b * kTileBytes;
                // rows of 8: pairs (0, 5), (2, 7), (4, 1), (6, 3)
                const int hrow = (lane >> 3) * 2;
                const int r8 = (lane & 4) ? (hrow ^ 5) : hrow;
                const int u4 = lane & 3;
                constexpr int H = DH <= 64 ? 1 : 2; // halves of 64 columns
                // 16 rows at a time: warps 12, 14, 15 take 6, 4 and 6 such
                // pairs of 8; warp 13 shares its scheduler with the MMA warp
                // and takes none
                if (cw == 1)
                    continue;
                const int row0 = cw == 0 ? 0 : cw == 2 ? 48 : 80;
                const int row1 = cw == 0 ? 48 : cw == 2 ? 80 : 128;
#pragma unroll 1
                for (int rr = row0; rr < row1; rr += 16) {
                    uint32_t x[2 * H][4];
#pragma unroll
                    for (int i = 0; i < 2 * H; ++i) {
                        const int r = rr + 8 * (i / H) + r8;
                        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                     : "=r"(x[i][0]), "=r"(x[i][1]), "=r"(x[i][2]), "=r"(x[i][3])
                                     : "r"(src + r * 128 + ((((i % H) * 4 + u4) ^ r8) << 4))
                                     : "memory");
                    }
                    if (ks + rr + 16 > hi) { // not keys: no code of theirs may be used
#pragma unroll
                        for (int i = 0; i < 2 * H; ++i)
                            if (ks + rr + 8 * (i / H) + r8 >= hi)
                                x[i][0] = x[i][1] = x[i][2] = x[i][3] = 0;
                    }
#pragma unroll
                    for (int i = 0; i < 2 * H; ++i) {
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
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(bar_pv(b));
                    mbar_arrive(bar_vempty(s));
                }
            }
            __syncwarp();
            if (ok && lane == 0)
                mbar_arrive(bar_iempty(si & 3));
            ok = ok && split(si + 1);
        }
    } else if (warp < 8) {
        // ------------------------------------------- softmax and epilogue
        const int wg = warp >> 2;
        const int row = threadIdx.x & (kTcM - 1);
        const int wrow = row & ~31; // first row of this warp
        const uint32_t lane_off = (uint32_t)wrow << 16;
        const uint32_t ts = tmem + wg * kQtStep + lane_off; // its half of S
        const uint32_t t_ow = t_o + wg * 128 + lane_off; // this warpgroup's O
        if (lane == 0)
            mbar_arrive(bar_qk(0)); // no S before tile 0
        bool ok = true;
        int j0 = 0; // tile of the CTA at the segment's start
        for (int si = 0; ok; ++si) {
            if (!(ok = wait(bar_ifull(si & 3), (uint32_t)((si >> 2) & 1))))
                break;
            const Seg &sg = seg_ring[si & 3];
            if (sg.nt == 0)
                break;
            const int n = sg.nt, nrows = sg.nrows, lo = sg.lo0, hi = sg.hi0;
            const int full_end = min(sg.fhi0, hi); // keys that every row sees
            const int jr = (sg.qrow0 + min(row, nrows - 1)) % p.pp.b;
            // keys that this row sees
            const int seen = min(hi, sg.len + (p.pp.mode == 0 ? p.pp.b : p.pp.mode == 1 ? jr + 1 : 0));
            const bool live = wrow < nrows; // a warp without rows only arrives
            // tiles in which this warp has rows and keys: all of them, or all but
            // the last, or none
            const int n_own = live ? (hi - lo + kTcN - 1 - wg * kQtStep) / kTcN : 0;
            float m = -INFINITY, l = 0.f; // running maximum (raised lazily), sum
            for (int i = 0; i < n_own; ++i) {
                const int j = j0 + i; // tile
                const int ks = lo + i * kTcN + wg * kQtStep;
                if (!(ok = wait(bar_sfull(j & 1), (uint32_t)((j >> 1) & 1))))
                    break;
                tc_fence_after();
                uint32_t sr[kQtStep];
                tmem_ld32x2_wait(ts, ts + 32, sr, sr + 32);
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(bar_qk((j + 1) & 3));
                float s[kQtStep];
#pragma unroll
                for (int c = 0; c < kQtStep; ++c)
                    s[c] = __uint_as_float(sr[c]);
                if (ks + kQtStep > full_end) {
#pragma unroll
                    for (int w = 0; w < kQtStep / 32; ++w) {
                        const uint32_t mk = range_bits(0, seen - ks - 32 * w);
#pragma unroll
                        for (int c = 0; c < 32; ++c)
                            s[32 * w + c] = ((mk >> c) & 1u) ? s[32 * w + c] : -INFINITY;
                    }
                }
                constexpr int C = kQtStep / 16;
                const float4 *tab = s_tab + (j & 3) * kQtChunks + wg * C;
                const float qs = s_qs[(si & 1) * kTcM + row];
                float4 e[C];
                float mt = -INFINITY;
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    const float *x = s + 16 * c;
                    const float m0 = fmax3(fmax3(x[0], x[1], x[2]), fmax3(x[3], x[4], x[5]), fmax3(x[6], x[7], x[8]));
                    const float m1 = fmax3(fmax3(x[9], x[10], x[11]), fmax3(x[12], x[13], x[14]), x[15]);
                    e[c] = tab[c];
                    // the product is no less than 2^-126: a masked score has
                    // to stay -inf (and below that x is 0 anyway)
                    e[c].x = fmaxf(e[c].x * qs, 1.2e-38f);
                    mt = fmaxf(mt, fmaf(fmaxf(m0, m1), e[c].x, e[c].y));
                }
                const bool need = mt > m + (kQtTop + kQtLazy);
                if (__any_sync(0xffffffffu, need)) {
                    float c = 1.f;
                    if (need) {
                        c = m == -INFINITY ? 0.f : ex2(m - (mt - kQtTop));
                        l = m == -INFINITY ? l : l * c; // 0, or NaN for good
                        m = mt - kQtTop;
                    }
                    if (i > 0) { // the TMEM read-modify-write of O is warp-collective
                        if (!(ok = wait(bar_odone((j - 1) & 1), (uint32_t)(((j - 1) >> 1) & 1))))
                            break;
                        tc_fence_after();
#pragma unroll 1
                        for (int q4 = 0; q4 < DH / 32; ++q4) {
                            uint32_t o[32];
                            tmem_ld32_wait(t_ow + q4 * 32, o);
#pragma unroll
                            for (int x = 0; x < 32; ++x)
                                o[x] = __float_as_uint(__uint_as_float(o[x]) * c);
                            tmem_st32(t_ow + q4 * 32, o);
                        }
                    }
                }
                const float nm = m == -INFINITY ? 0.f : -m;
                uint32_t pk[kQtStep / 2];
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    const float o = e[c].y + nm;
                    float r0 = 0.f, r1 = 0.f;
#pragma unroll
                    for (int x = 16 * c; x < 16 * c + 16; x += 2) {
                        float y0, y1;
                        ffma2(y0, y1, s[x], s[x + 1], e[c].x, e[c].x, o, o);
                        y0 = ex2(y0);
                        y1 = ex2(y1);
                        fadd2(r0, r1, r0, r1, y0, y1);
                        pk[x / 2] = pack_f16x2(y0, y1);
                    }
                    l = fmaf(r0 + r1, e[c].z, l);
                }
                // P of the tile before has been used
                if (j >= 1 && !(ok = wait(bar_odone((j - 1) & 1), (uint32_t)(((j - 1) >> 1) & 1))))
                    break;
                tc_fence_after();
                tmem_st32(t_p + wg * 32 + lane_off, pk);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(bar_pv(j & 1));
            }
            for (int i = n_own; ok && i < n; ++i) { // only the arrivals
                const int j = j0 + i;
                if (!(ok = wait(bar_sfull(j & 1), (uint32_t)((j >> 1) & 1))))
                    break;
                if (lane == 0) {
                    mbar_arrive(bar_qk((j + 1) & 3));
                    mbar_arrive(bar_pv(j & 1));
                }
            }
            if (!ok)
                break;
            const int jl = j0 + n - 1; // last tile of the segment
            s_l[((si & 1) * 2 + wg) * kTcM + row] = make_float2(l, m);
            mbar_arrive(bar_l);
            // The last PVs.  (The phase before on that barrier is behind QK_jl,
            // which this warp has seen.)
            if (!(ok = wait(bar_l, (uint32_t)(si & 1))) ||
                !(ok = wait(bar_odone(jl & 1), (uint32_t)((jl >> 1) & 1))))
                break;
            tc_fence_after();
            // factors of the two O to the common maximum; O_1 is unwritten
            // where the segment has no key in a second half
            const float2 l0 = s_l[(si & 1) * 2 * kTcM + row], l1 = s_l[((si & 1) * 2 + 1) * kTcM + row];
            const bool two = hi - lo > kQtStep;
            const float mx = fmaxf(l0.y, l1.y);
            const float f0 = l0.y == -INFINITY ? 1.f : ex2(l0.y - mx);
            const float f1 = l1.y == -INFINITY ? 1.f : ex2(l1.y - mx);
            const float ls = l0.x * f0 + l1.x * f1; // a NaN shows in l whatever m is
            const float inv = ls == 0.f ? 0.f : 1.f / ls;
            const float w0 = f0 * inv, w1 = f1 * inv;
            const bool valid = row < nrows;
            const size_t grow = (size_t)sg.out_row0 + row;
            const size_t prow = ((size_t)blockIdx.x * 2 + sg.slot) * kTcM + row;
            constexpr int kCols = DH >= 64 ? DH / 2 : DH; // columns of O a warpgroup takes
            if (live && (DH >= 64 || wg == 0)) {
#pragma unroll
                for (int q4 = 0; q4 < kCols / 32; ++q4) {
                    const int col = wg * kCols + q4 * 32;
                    uint32_t o[32], o1[32];
                    tmem_ld32x2_wait(t_o + lane_off + col, t_o + 128 + lane_off + col, o, o1);
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const float x = __uint_as_float(o[i]) * w0;
                        o[i] = __float_as_uint(two ? fmaf(__uint_as_float(o1[i]), w1, x) : x);
                    }
                    if (valid && sg.complete) {
                        uint4 *dst = reinterpret_cast<uint4 *>(p.pp.out + grow * DH + col);
#pragma unroll
                        for (int i = 0; i < 32; i += 8) {
                            uint4 v4;
                            v4.x = pack_bf16x2(__uint_as_float(o[i]), __uint_as_float(o[i + 1]));
                            v4.y = pack_bf16x2(__uint_as_float(o[i + 2]), __uint_as_float(o[i + 3]));
                            v4.z = pack_bf16x2(__uint_as_float(o[i + 4]), __uint_as_float(o[i + 5]));
                            v4.w = pack_bf16x2(__uint_as_float(o[i + 6]), __uint_as_float(o[i + 7]));
                            dst[i / 8] = v4;
                        }
                    } else if (valid) {
                        uint4 *dst = reinterpret_cast<uint4 *>(p.pp.part_o + prow * kTcD + col);
#pragma unroll
                        for (int i = 0; i < 32; i += 4)
                            dst[i / 4] = make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]);
                    }
                }
            }
            if (valid && wg == 0)
                (sg.complete ? p.pp.lse + grow : p.pp.part_lse + prow)[0] =
                    ls == 0.f ? -INFINITY : ((l0.y == -INFINITY && l1.y == -INFINITY ? 0.f : mx) + __log2f(ls)) * kLn2;
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

    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
    }
}

} // namespace bd
