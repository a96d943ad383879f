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
// Persistent, one CTA per SM, over the work list of the bf16 decode
// (DecSource: whole units, or equal ranges of 128-key tiles merged by
// bd_decode_stream_combine_kernel).  Roles:
//   warps 0-3, 4-7  softmax, thread = query row = TMEM lane; one warpgroup
//                   takes the first 64 keys of every tile, one the last
//   warp 8          the work list, TMA of K
//   warp 9          MMA issue: the QK of a tile, then the PVs of the tile
//                   before, step by step, over segment boundaries
//   warp 10         TMA of V, cp.async of the scales
//   warps 12-15     per tile: the table of scales, V codes to f16
// TMEM: S/P of two tiles (64 columns a step; P, f16, over its own S), O (128),
// two buffers of Q (hi and lo, 32 columns each).
//
// O has one running maximum.  It is handed from step to step, warpgroup to
// warpgroup, in shared memory, before the exponentials: a step waits for the
// one before it only with its maximum in hand.  Each warpgroup has its own sum
// l, relative to the maximum at its last step; the epilogue joins the two.
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
constexpr int kQtSmemM = kQtSmemTab + 4 * kQtChunks * 16; // running maxima [2][128]
constexpr int kQtSmemL = kQtSmemM + 2 * kTcM * 4;         // (l, M) [2][2][128]
constexpr int kQtSmemQs = kQtSmemL + 4 * kTcM * 8;        // row scales of Q [2][128]
constexpr int kQtSmemSeg = kQtSmemQs + 2 * kTcM * 4;      // 4 segments, 128 B each
constexpr int kQtSmemBar = kQtSmemSeg + 4 * 128;
constexpr int kQtSmemBytes = kQtSmemBar + 512 + 1024; // + alignment slack
static_assert(kQtSmemBytes <= 227 * 1024, "more shared memory than a CTA may have");

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

// A query row as two halves of e4m3 codes in tensor memory, hi in columns
// [tq, tq + 32), lo behind it, and its scale; thread = row.  The row is read
// twice (the second time from L1), which saves 64 registers.
template <int DH>
__device__ __forceinline__ float qt_split_row(const bf16 *src, bool valid, uint32_t tq)
{
    const uint4 *row = reinterpret_cast<const uint4 *>(src);
    float amax = 0.f;
    bool finite = true;
#pragma unroll
    for (int i = 0; i < DH / 8; ++i) {
        const uint4 w = valid ? row[i] : make_uint4(0, 0, 0, 0);
        const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
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
    for (int c = 0; c < DH / 32; ++c) { // 32 dims
        uint32_t hi[8], lo[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint4 w = valid ? row[4 * c + i] : make_uint4(0, 0, 0, 0);
            const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
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
        tmem_st8(tq + 8 * c, hi);
        tmem_st8(tq + 32 + 8 * c, lo);
    }
    return finite ? exp2_int(k) : NAN;
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
    auto bar_kfull = [&](int s) { return bar0 + 8 * s; };
    auto bar_kempty = [&](int s) { return bar0 + 32 + 8 * s; };
    auto bar_vfull = [&](int s) { return bar0 + 64 + 8 * s; };
    auto bar_vempty = [&](int s) { return bar0 + 96 + 8 * s; };
    auto bar_ifull = [&](int s) { return bar0 + 128 + 8 * s; }; // segment si & 3
    auto bar_iempty = [&](int s) { return bar0 + 160 + 8 * s; };
    auto bar_sfull = [&](int s) { return bar0 + 192 + 8 * s; }; // S of tile j & 1, and its scales
    auto bar_pfull = [&](int s) { return bar0 + 224 + 8 * s; }; // P of step t & 3
    auto bar_w = [&](int s) { return bar0 + 256 + 8 * s; };     // V of tile j & 1 in f16
    auto bar_wfree = [&](int s) { return bar0 + 272 + 8 * s; }; // both its PVs done
    auto bar_qfull = [&](int s) { return bar0 + 304 + 8 * s; };
    // maximum of step t & 1 handed on, 32 rows each
    auto bar_mtok = [&](int s, int w) { return bar0 + 320 + 32 * s + 8 * w; };
    const uint32_t bar_l = bar0 + 384;     // both sums of a segment written
    const uint32_t bar_ofree = bar0 + 392; // O read out
    const uint32_t bar_final = bar0 + 400;
    auto bar_odone = [&](int s) { return bar0 + 408 + 8 * s; }; // PV of step t & 3
    static_assert(kQtKStages == 4 && kQtVStages == 4, "barrier layout");
    volatile int *abort_flag = reinterpret_cast<volatile int *>(sbase + kQtSmemBar + 448);
    volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(sbase + kQtSmemBar + 456);
    Seg *seg_ring = reinterpret_cast<Seg *>(sbase + kQtSmemSeg); // nt = 0: no more
    float *s_m = reinterpret_cast<float *>(sbase + kQtSmemM);
    float2 *s_l = reinterpret_cast<float2 *>(sbase + kQtSmemL);
    float *s_qs = reinterpret_cast<float *>(sbase + kQtSmemQs);
    float4 *s_tab = reinterpret_cast<float4 *>(sbase + kQtSmemTab);
    const float *s_raw = reinterpret_cast<const float *>(sbase + kQtSmemRaw);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < 4; ++s) {
            mbar_init(bar_kfull(s), 1);
            mbar_init(bar_kempty(s), 1);
            mbar_init(bar_vfull(s), 1 + 2 * kQtChunks); // + a copy of each scale
            mbar_init(bar_vempty(s), 4);
            mbar_init(bar_ifull(s), 1);
            mbar_init(bar_iempty(s), 14); // 8 softmax warps, MMA, V, 4 converters
            mbar_init(bar_pfull(s), 4);
            mbar_init(bar_odone(s), 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(bar_sfull(s), 2); // the MMA, the table
            mbar_init(bar_w(s), 4);
            mbar_init(bar_wfree(s), 1);
            mbar_init(bar_qfull(s), 128);
            for (int w = 0; w < 4; ++w)
                mbar_init(bar_mtok(s, w), 1);
        }
        mbar_init(bar_l, 256);
        mbar_init(bar_ofree, 256);
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
    const uint32_t t_o = tmem + 256, t_q = tmem + 384;
    // the combine kernel may be scheduled now; it reads nothing of this
    // launch before the whole grid has finished
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // a barrier wait by a converged warp
    auto wait = [&](uint32_t bar, uint32_t parity) { return mbar_wait_warp(bar, parity, abort_flag); };

    if (warp == 8) {
        // ------------------------------------------ work list, loads of K
        DecSource src;
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
                    mbar_expect_tx(bar_kfull(s), kQtTile);
                    tma_load_3d(base + kQtSmemK + s * kQtTile, &tm_k, 0, sg.lo0 + it * kTcN, sg.kvhead,
                                bar_kfull(s));
                    kiss = g + 1;
                }
                __syncwarp();
            }
        }
        // wait (bounded) for every copy this role issued
        if (lane == 0) {
            const long long c0 = clock64();
            for (int x = kiss > 4 ? kiss - 4 : 0; x < kiss; ++x)
                while (!mbar_try_wait(bar_kfull(x & 3), (uint32_t)((x >> 2) & 1)) &&
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
        // cursor of the PVs: tile j of the CTA, tile i of the n of its segment si
        int j = 0, i = 0, n = 0, si = 0;
        int hi = 0; // keys of the segment from its first tile on
        auto next_qk = [&]() { // the next tile's QK, if there is one to issue
            if (qi == qn) {
                // One segment ahead of the PVs at most: the queries behind
                // that are split only after PVs that wait in this loop.
                if (qn && qs > si)
                    return;
                if (qn) { // segment qs is through
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(bar_iempty(qs & 3));
                    ++qs;
                    qn = qi = 0;
                }
                if (!(ok = wait(bar_ifull(qs & 3), (uint32_t)((qs >> 2) & 1))))
                    return;
                qn = seg_ring[qs & 3].nt;
                if (qn == 0 || !(ok = wait(bar_qfull(qs & 1), (uint32_t)((qs >> 1) & 1))))
                    return;
            }
            const int s = qj & 3;
            if (!(ok = wait(bar_kfull(s), (uint32_t)((qj >> 2) & 1))))
                return;
            tc_fence_after();
            // the S buffer held P of tile qj - 2, whose PVs were issued before
            const uint32_t ts = tmem + (uint32_t)(qj & 1) * kTcN;
            const uint32_t tq = t_q + (uint32_t)(qs & 1) * 64;
            const uint32_t kb = base + kQtSmemK + (uint32_t)s * kQtTile;
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int kk = 0; kk < DH / 32; ++kk)
                    tc_mma8_ts_p(ts, tq + h * 32 + kk * 8, smem_desc_sw128(kb + kk * 32, 16, 1024),
                                 idesc_qk, h || kk ? 1u : 0u, ld);
            tc_commit_p(bar_sfull(qj & 1), ld);
            tc_commit_p(bar_kempty(s), ld);
            ++qj;
            ++qi;
        };
        next_qk();
        while (ok && j < qj) {
            if (i == n) {
                // known: QK_j was issued, and a slot of the ring is not
                // rewritten before this segment's epilogue
                n = seg_ring[si & 3].nt;
                hi = seg_ring[si & 3].hi0 - seg_ring[si & 3].lo0;
                i = 0;
            }
            if (qj == j + 1) { // QK_{j+1} goes out before the PVs of tile j
                next_qk();
                if (!ok)
                    break;
            }
            // O was last read out by the epilogue of segment si - 1
            if (i == 0 && si >= 1 && !(ok = wait(bar_ofree, (uint32_t)((si - 1) & 1))))
                break;
            const int b = j & 1;
            if (!(ok = wait(bar_w(b), (uint32_t)((j >> 1) & 1))))
                break;
#pragma unroll 1
            for (int half = 0; half < 2; ++half) {
                const int pb = 2 * b + half;
                if (!(ok = wait(bar_pfull(pb), (uint32_t)((j >> 1) & 1))))
                    break;
                tc_fence_after();
                const uint32_t vb = base + kQtSmemW + (uint32_t)b * kTileBytes + half * (kQtStep * 128);
                const uint32_t tp = tmem + (uint32_t)pb * kQtStep;
                if (half == 0 || i * kTcN + kQtStep < hi) {
#pragma unroll
                    for (int kk = 0; kk < kQtStep / 16; ++kk)
                        tc_mma_ts_p(t_o, tp + kk * 8,
                                    smem_desc_sw128(vb + kk * 2048, kHalfTileBytes, 1024), idesc_pv,
                                    (i > 0 || half > 0 || kk > 0) ? 1u : 0u, ld);
                }
                tc_commit_p(bar_odone(pb), ld);
            }
            if (!ok)
                break;
            tc_commit_p(bar_wfree(b), ld);
            ++j;
            if (++i == n)
                ++si;
            if (qj == j)
                next_qk();
        }
        tc_commit_p(bar_final, ld);
        const long long c0 = clock64();
        while (!mbar_try_wait(bar_final, 0) && clock64() - c0 < kWaitCycles) {}
        __syncwarp();
    } else if (warp >= 12) {
        // ------------------------- the table of scales, V codes to f16
        const int cw = warp - 12;
        bool ok = true;
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
                if (!(ok = wait(bar_vfull(s), (uint32_t)((j >> 2) & 1))))
                    break;
                // the f16 buffer was last read by the PVs of tile j - 2;
                // the softmax of that tile lies behind them
                const int b = j & 1;
                if (j >= 2 && !(ok = wait(bar_wfree(b), (uint32_t)(((j - 2) >> 1) & 1))))
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
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(bar_sfull(b));
                }
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
                // warp cw: rows 32 cw .. 32 cw + 31; all loads go out first
                uint32_t x[4 * H][4];
#pragma unroll
                for (int i = 0; i < 4 * H; ++i) {
                    const int r = 32 * cw + 8 * (i / H) + r8;
                    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(x[i][0]), "=r"(x[i][1]), "=r"(x[i][2]), "=r"(x[i][3])
                                 : "r"(src + r * 128 + ((((i % H) * 4 + u4) ^ r8) << 4))
                                 : "memory");
                }
                if (ks + 32 * cw + 32 > hi) { // not keys: no code of theirs may be used
#pragma unroll
                    for (int i = 0; i < 4 * H; ++i)
                        if (ks + 32 * cw + 8 * (i / H) + r8 >= hi)
                            x[i][0] = x[i][1] = x[i][2] = x[i][3] = 0;
                }
#pragma unroll
                for (int i = 0; i < 4 * H; ++i) {
                    uint32_t y[8];
#pragma unroll
                    for (int t = 0; t < 8; ++t)
                        y[t] = half2_of_e4m3x2((uint16_t)(x[i][t >> 1] >> (16 * (t & 1))));
                    const uint32_t row = dst + (i % H) * kHalfTileBytes + (32 * cw + 8 * (i / H) + r8) * 128;
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
                    mbar_arrive(bar_w(b));
                    mbar_arrive(bar_vempty(s));
                }
            }
            __syncwarp();
            if (ok && lane == 0)
                mbar_arrive(bar_iempty(si & 3));
        }
    } else if (warp < 8) {
        // ------------------------------------------- softmax and epilogue
        const int wg = warp >> 2;
        const int row = threadIdx.x & (kTcM - 1);
        const int wrow = row & ~31; // first row of this warp
        const uint32_t lane_off = (uint32_t)wrow << 16;
        // Splits the query rows of segment si, by one warpgroup.  Its buffer
        // was last read by the QKs of segment si - 2, finished before that
        // segment's epilogue was.
        auto split = [&](int si) -> bool {
            if (!wait(bar_ifull(si & 3), (uint32_t)((si >> 2) & 1)))
                return false;
            const Seg &sg = seg_ring[si & 3];
            if (sg.nt == 0)
                return true;
            const float qs = qt_split_row<DH>(p.q + ((size_t)sg.out_row0 + row) * DH, row < sg.nrows,
                                              t_q + (uint32_t)(si & 1) * 64 + lane_off);
            s_qs[(si & 1) * kTcM + row] = qs;
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(bar_qfull(si & 1));
            return true;
        };
        bool ok = wg == 1 || split(0);
        int j0 = 0; // tile of the CTA at the segment's start
        for (int si = 0; ok; ++si) {
            if (!(ok = wait(bar_ifull(si & 3), (uint32_t)((si >> 2) & 1))))
                break;
            const Seg &sg = seg_ring[si & 3];
            if (sg.nt == 0)
                break;
            if (!(ok = wait(bar_qfull(si & 1), (uint32_t)((si >> 1) & 1))))
                break;
            const float qs = s_qs[(si & 1) * kTcM + row];
            const int n = sg.nt, nrows = sg.nrows, lo = sg.lo0;
            const int full_end = min(sg.fhi0, sg.hi0); // keys that every row sees
            const int jr = (sg.qrow0 + min(row, nrows - 1)) % p.pp.b;
            // keys that this row sees
            const int seen = min(sg.hi0, sg.len + (p.pp.mode == 0 ? p.pp.b : p.pp.mode == 1 ? jr + 1 : 0));
            const bool live = wrow < nrows; // a warp without rows only arrives
            float m_own = -INFINITY, l = 0.f;
            for (int i = 0; i < n; ++i) {
                const int j = j0 + i, t = 2 * j + wg; // tile, step
                const uint32_t ts = tmem + (uint32_t)(t & 3) * kQtStep + lane_off;
                const int ks = lo + i * kTcN + wg * kQtStep;
                if (!(ok = wait(bar_sfull(j & 1), (uint32_t)((j >> 1) & 1))))
                    break;
                if (!live || ks >= sg.hi0) { // no rows, or (in the last step) no keys
                    if (t >= 1 && !(ok = wait(bar_mtok(wg ^ 1, warp & 3), (uint32_t)(((t - 1) >> 1) & 1))))
                        break;
                    s_m[wg * kTcM + row] = s_m[(wg ^ 1) * kTcM + row];
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(bar_mtok(wg, warp & 3));
                        mbar_arrive(bar_pfull(t & 3));
                    }
                    continue;
                }
                tc_fence_after();
                uint32_t sr[kQtStep];
                tmem_ld32x2_wait(ts, ts + 32, sr, sr + 32);
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
                // the maximum up to the step before
                if (t >= 1 && !(ok = wait(bar_mtok(wg ^ 1, warp & 3), (uint32_t)(((t - 1) >> 1) & 1))))
                    break;
                const bool first = i == 0 && wg == 0; // of the segment
                const float m_prev = first ? -INFINITY : s_m[(wg ^ 1) * kTcM + row];
                const bool need = mt > m_prev + (kQtTop + kQtLazy);
                const float m = need ? mt - kQtTop : m_prev;
                // the TMEM read-modify-write of O is warp-collective
                if (!first && __any_sync(0xffffffffu, need)) {
                    // PV_{t-1}.  Its barrier's phase before, PV_{t-5}, is of
                    // tile j - 2 or older, whose PVs QK_j was issued behind.
                    if (!(ok = wait(bar_odone((t - 1) & 3), (uint32_t)(((t - 1) >> 2) & 1))))
                        break;
                    tc_fence_after();
                    const float c = !need ? 1.f : m_prev == -INFINITY ? 0.f : ex2(m_prev - m);
#pragma unroll 1
                    for (int q4 = 0; q4 < DH / 32; ++q4) {
                        uint32_t o[32];
                        tmem_ld32_wait(t_o + lane_off + q4 * 32, o);
#pragma unroll
                        for (int x = 0; x < 32; ++x)
                            o[x] = __float_as_uint(__uint_as_float(o[x]) * c);
                        tmem_st32(t_o + lane_off + q4 * 32, o);
                    }
                    tmem_wait_st();
                    tc_fence_before();
                }
                s_m[wg * kTcM + row] = m;
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(bar_mtok(wg, warp & 3));
                if (m > m_own) {
                    l = m_own == -INFINITY ? l : l * ex2(m_own - m); // 0, or NaN for good
                    m_own = m;
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
                tmem_st32(ts, pk);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(bar_pfull(t & 3));
            }
            if (!ok)
                break;
            const int jl = j0 + n - 1; // last tile of the segment
            // the warpgroup without the last step readies the next queries
            if (wg == 0 && !(ok = split(si + 1)))
                break;
            s_l[((si & 1) * 2 + wg) * kTcM + row] = make_float2(l, m_own);
            mbar_arrive(bar_l);
            if (!(ok = wait(bar_l, (uint32_t)(si & 1))))
                break;
            const float2 other = s_l[((si & 1) * 2 + (wg ^ 1)) * kTcM + row];
            const float m = fmaxf(m_own, other.y);
            const float l0 = m_own == -INFINITY ? l : l * ex2(m_own - m);
            const float l1 = other.y == -INFINITY ? other.x : other.x * ex2(other.y - m);
            l = l0 + l1; // a NaN shows in l whatever m is
            // the last PV; the PVs of tile jl - 2 lie behind QK_jl, which both
            // warpgroups have seen
            if (!(ok = wait(bar_odone(2 * (jl & 1) + 1), (uint32_t)((jl >> 1) & 1))))
                break;
            tc_fence_after();
            const bool valid = row < nrows;
            const float inv = l == 0.f ? 0.f : 1.f / l;
            const size_t grow = (size_t)sg.out_row0 + row;
            const size_t prow = ((size_t)blockIdx.x * 2 + sg.slot) * kTcM + row;
            constexpr int kCols = DH >= 64 ? DH / 2 : DH; // columns of O a warpgroup takes
            if (live && (DH >= 64 || wg == 0)) {
#pragma unroll
                for (int q4 = 0; q4 < kCols / 32; ++q4) {
                    const int col = wg * kCols + q4 * 32;
                    uint32_t o[32];
                    tmem_ld32_wait(t_o + lane_off + col, o);
                    if (valid && sg.complete) {
                        uint4 *dst = reinterpret_cast<uint4 *>(p.pp.out + grow * DH + col);
#pragma unroll
                        for (int i = 0; i < 32; i += 8) {
                            uint4 v4;
                            v4.x = pack_bf16x2(__uint_as_float(o[i]) * inv, __uint_as_float(o[i + 1]) * inv);
                            v4.y = pack_bf16x2(__uint_as_float(o[i + 2]) * inv, __uint_as_float(o[i + 3]) * inv);
                            v4.z = pack_bf16x2(__uint_as_float(o[i + 4]) * inv, __uint_as_float(o[i + 5]) * inv);
                            v4.w = pack_bf16x2(__uint_as_float(o[i + 6]) * inv, __uint_as_float(o[i + 7]) * inv);
                            dst[i / 8] = v4;
                        }
                    } else if (valid) {
                        float4 *dst = reinterpret_cast<float4 *>(p.pp.part_o + prow * kTcD + col);
#pragma unroll
                        for (int i = 0; i < 32; i += 4)
                            dst[i / 4] = make_float4(
                                __uint_as_float(o[i]) * inv, __uint_as_float(o[i + 1]) * inv,
                                __uint_as_float(o[i + 2]) * inv, __uint_as_float(o[i + 3]) * inv);
                    }
                }
            }
            if (valid && wg == 0)
                (sg.complete ? p.pp.lse + grow : p.pp.part_lse + prow)[0] =
                    l == 0.f ? -INFINITY : (m + __log2f(l)) * kLn2;
            if (!sg.complete && sg.last_cta >= 0 && threadIdx.x == 0)
                p.pp.cut_desc[blockIdx.x] = make_int4(nrows, sg.last_cta, sg.out_row0, 0);
            tc_fence_before();
            mbar_arrive(bar_ofree);
            __syncwarp();
            if (lane == 0)
                mbar_arrive(bar_iempty(si & 3));
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
