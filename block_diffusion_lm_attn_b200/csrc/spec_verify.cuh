// Verifying drafted tokens against the target's probabilities (sm_100a).
//
// Position j of a draft x with draft probabilities q_j and target
// probabilities p_j is accepted while u_j q_j(x_j) < p_j(x_j); at the first
// refusal n the next token is drawn from the residual max(p_n - q_n, 0), or
// from p_n where nothing is left of it; with every position accepted, from
// the row behind, p_n with n = n_draft.  Drawing: the lowest t whose running
// sum C_t of weights exceeds r C_V.  The accepted tokens and the drawn one are
// then distributed as the target's own.
//
// Products of two floats are exact in double, so each acceptance is decided
// exactly; the running sums are double too, added in a fixed order.
//
// Bound by reading one row of p and one of q per sequence (8 V bytes), and for
// few sequences by latency: the gathers of the acceptance, the rows, the entry
// in its segment, each waits for the one before.  A cluster of 8 CTAs takes a
// sequence, an eighth of the vocabulary each, and exchanges the eight sums
// through shared memory; a lane has 32 numbers on their way.  Measured: 7.5 us
// for one sequence of 50001 entries (one CTA a sequence: 36), 19.3 us for 64 of
// 131072, 3.5 TB/s (137; half as many numbers on their way: 29; rows that are not
// on 32-byte boundaries: 20.8).
#pragma once

#include <limits.h>

#include "bd_common.cuh"
#include "cache_q8.cuh"

namespace bd {

constexpr int kVerifyCluster = 8;
constexpr int kVerifySeg = 512; // vocabulary entries per segment: 16 a lane
constexpr int kVerifyMaxVocab = 1 << 22;

struct VerifyParams {
    const int32_t *draft;     // [B, b]
    const float *draft_prob;  // [B, b, V], or NULL: all mass on the drafted token
    const float *target_prob; // [B, b + 1, V]
    const float *u_accept;    // [B, b]
    const float *u_sample;    // [B]
    const int32_t *n_draft;   // [B] or NULL: b
    int32_t *n_accept, *next_token;
    int B, b, V;
};

__device__ __forceinline__ double warp_sum(double v)
{
#pragma unroll
    for (int o = 16; o; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Accepted positions of the nd drafted ones of sequence i, by one converged
// warp; -1 for a draft length or a drafted token out of range.
__device__ __forceinline__ int verify_accept(const VerifyParams &p, int i, int nd, int lane)
{
    if (nd < 0 || nd > p.b)
        return -1;
    int n = nd;
    bool bad = false;
    for (int j0 = 0; j0 < nd; j0 += 32) {
        const int j = j0 + lane;
        bool refuse = false;
        if (j < nd) {
            const int x = p.draft[(size_t)i * p.b + j];
            if (x < 0 || x >= p.V) {
                bad = true;
            } else {
                const double pj = p.target_prob[((size_t)i * (p.b + 1) + j) * p.V + x];
                const double qj = p.draft_prob ? p.draft_prob[((size_t)i * p.b + j) * p.V + x] : 1.f;
                refuse = !((double)p.u_accept[(size_t)i * p.b + j] * qj < pj);
            }
        }
        const unsigned m = __ballot_sync(0xffffffffu, refuse);
        if (m && n == nd)
            n = j0 + __ffs(m) - 1;
    }
    return __any_sync(0xffffffffu, bad) ? -1 : n;
}

__device__ __forceinline__ void cluster_arrive()
{
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait()
{
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// the double at `addr` of this CTA's shared memory, in CTA `rank` of the cluster
__device__ __forceinline__ double cluster_ld(uint32_t addr, uint32_t rank)
{
    double v;
    asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\t"
                 "ld.shared::cluster.f64 %0, [a];\n\t}"
                 : "=d"(v)
                 : "r"(addr), "r"(rank)
                 : "memory");
    return v;
}
// sum over lanes 0 .. lane
__device__ __forceinline__ double warp_scan(double v, int lane)
{
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const double up = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o)
            v += up;
    }
    return v;
}

// Cluster = sequence, CTA = a run of `segs` segments of the vocabulary.
template <int THREADS>
__global__ void __cluster_dims__(kVerifyCluster, 1, 1) __launch_bounds__(THREADS, 1024 / THREADS)
    bd_spec_verify_kernel(const VerifyParams p, int segs)
{
    extern __shared__ double seg[]; // sum of each segment's weights
    __shared__ double s_total[2];   // this CTA's, of each pass
    __shared__ int s_n, s_nd;
    const int i = blockIdx.x / kVerifyCluster, rank = blockIdx.x % kVerifyCluster;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // Either output may lie in n_draft's buffer: every CTA reads its counts here,
    // once, and nothing is written before a barrier of the cluster is behind.
    if (warp == 0) {
        const int nd = p.n_draft ? p.n_draft[i] : p.b;
        const int n = verify_accept(p, i, nd, lane);
        if (lane == 0) {
            s_n = n;
            s_nd = nd;
        }
    }
    __syncthreads();
    const int n = max(s_n, 0), nd = s_nd;
    const float *pr = p.target_prob + ((size_t)i * (p.b + 1) + n) * p.V;
    const float *qr = n < nd && p.draft_prob ? p.draft_prob + ((size_t)i * p.b + n) * p.V : nullptr;
    const int point = n < nd && !p.draft_prob ? p.draft[(size_t)i * p.b + n] : -1;
    const int v0 = rank * segs * kVerifySeg; // this CTA's entries
    const int v1 = min(p.V, v0 + segs * kVerifySeg);
    // (a bad sequence, for every CTA of its cluster, has no entries)
    const int mine = v1 > v0 && s_n >= 0 ? (v1 - v0 + kVerifySeg - 1) / kVerifySeg : 0;
    bool residual = n < nd;

    constexpr int E = kVerifySeg / 32;
    // weights of entries t + step * e below v1, all of them if `full`
    auto weights = [&](int t, int step, bool full, auto use) {
        float a[E], b[E];
        const float *pt = pr + t, *qt = (residual && qr ? qr : pr) + t;
        if (full) {
#pragma unroll
            for (int e = 0; e < E; ++e)
                a[e] = pt[step * e];
#pragma unroll
            for (int e = 0; e < E; ++e)
                b[e] = residual && qr ? qt[step * e] : 0.f;
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const bool in = t + step * e < v1;
                a[e] = in ? pt[step * e] : 0.f;
                b[e] = in && residual && qr ? qt[step * e] : 0.f;
            }
        }
#pragma unroll
        for (int e = 0; e < E; ++e) {
            if (residual && t + step * e == point)
                b[e] = 1.f;
            // NaN counts as 0; a > b decides, so the conversions of the
            // others are of no consequence
            use(e, a[e] > b[e] ? (double)a[e] - (double)b[e] : 0.0);
        }
    };
    // rows on 32-byte boundaries: weights of entries t .. t + 7 and 256 on, 8 at
    // a load
    const bool wide = ((reinterpret_cast<uintptr_t>(pr) | reinterpret_cast<uintptr_t>(qr)) & 31) == 0;
    auto wide_weights = [&](int t, auto use) {
        static_assert(E == 16, "two runs of 8");
        uint32_t a[16], b[16];
        ld32(pr + t, a);
        ld32(pr + t + 256, a + 8);
#pragma unroll
        for (int e = 0; e < 16; ++e)
            b[e] = 0;
        if (residual && qr) {
            ld32(qr + t, b);
            ld32(qr + t + 256, b + 8);
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            const float x = __uint_as_float(a[e]);
            const float y = residual && t + (e & 7) + 32 * (e & 8) == point ? 1.f : __uint_as_float(b[e]);
            use(e, x > y ? (double)x - (double)y : 0.0);
        }
    };
    double total = 0.0, before = 0.0; // of the cluster; of the CTAs before this one
    int owner_last = -1;              // last CTA with mass
    int pass = 0;
    for (;; ++pass) {
        for (int g = warp; g < mine; g += THREADS / 32) {
            double part = 0.0;
            const int t0 = v0 + g * kVerifySeg;
            auto add = [&](int, double w) { part += w; };
            if (wide && t0 + kVerifySeg <= v1)
                wide_weights(t0 + 8 * lane, add);
            else
                weights(t0 + lane, 32, t0 + kVerifySeg <= v1, add);
            part = warp_sum(part);
            if (lane == 0)
                seg[g] = part;
        }
        __syncthreads();
        if (warp == 0) {
            double sum = 0.0;
            for (int g = lane; g < mine; g += 32)
                sum += seg[g];
            sum = warp_sum(sum);
            if (lane == 0)
                s_total[pass] = sum;
        }
        __syncthreads();
        cluster_arrive();
        cluster_wait();
        const uint32_t addr = smem_u32(&s_total[pass]);
        total = before = 0.0;
#pragma unroll
        for (int r = 0; r < kVerifyCluster; ++r) {
            const double x = cluster_ld(addr, r);
            if (r < rank)
                before += x;
            total += x;
            if (x > 0.0)
                owner_last = r;
        }
        if (total > 0.0 || !residual)
            break;
        residual = false; // nothing left of p - q: draw from p
    }
    cluster_arrive(); // the sums have been read; waited for before the exit
    // the CTA whose entries hold the drawn one: the first whose running sum
    // passes `want`, or the last with mass
    const double u = p.u_sample[i];
    const double want = u > 0.0 ? u * total : 0.0; // (a NaN draws the first)
    const double own = s_total[pass];
    const bool here = own > 0.0 && before <= want && (before + own > want || rank == owner_last);
    if (rank == 0 && threadIdx.x == 0) {
        if (s_n < 0)
            raise_device_code(DEV_BAD_CACHE_LEN);
        p.n_accept[i] = max(s_n, 0);
        if (total <= 0.0)
            p.next_token[i] = -1;
    }
    if (warp == 0 && here) {
        // the segment, 32 at a time
        double run = before;
        int g = -1, last = -1;
        double at = 0.0, last_at = 0.0; // sum before segments g, last
        for (int g0 = 0; g0 < mine && g < 0; g0 += 32) {
            const double x = g0 + lane < mine ? seg[g0 + lane] : 0.0;
            const double incl = run + warp_scan(x, lane);
            const unsigned hit = __ballot_sync(0xffffffffu, x > 0.0 && incl > want);
            const unsigned mass = __ballot_sync(0xffffffffu, x > 0.0);
            if (hit) {
                g = g0 + __ffs(hit) - 1;
                at = __shfl_sync(0xffffffffu, incl - x, __ffs(hit) - 1);
            }
            if (mass) {
                last = g0 + 31 - __clz(mass);
                last_at = __shfl_sync(0xffffffffu, incl - x, 31 - __clz(mass));
            }
            run = __shfl_sync(0xffffffffu, incl, 31);
        }
        if (g < 0) {
            g = last;
            at = last_at;
        }
        // lane l takes entries E l .. E l + E - 1 of segment g
        const int t0 = v0 + g * kVerifySeg + lane * E;
        double sum = 0.0;
        int last_pos = -1;
        weights(t0, 1, false, [&](int e, double w) {
            sum += w;
            if (w > 0.0)
                last_pos = t0 + e;
        });
        double c = at + (warp_scan(sum, lane) - sum);
        int found = INT_MAX;
        weights(t0, 1, false, [&](int e, double w) {
            c += w;
            if (w > 0.0 && c > want && found == INT_MAX)
                found = t0 + e;
        });
        found = __reduce_min_sync(0xffffffffu, found);
        last_pos = __reduce_max_sync(0xffffffffu, last_pos);
        if (lane == 0)
            p.next_token[i] = found == INT_MAX ? last_pos : found;
    }
    cluster_wait();
}

} // namespace bd
