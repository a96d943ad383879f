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
// Bound by reading one row of p and one of q per sequence (8 V bytes).
#pragma once

#include "bd_common.cuh"

namespace bd {

constexpr int kVerifyThreads = 1024;
constexpr int kVerifySeg = 1024;            // vocabulary entries per segment
constexpr int kVerifyMaxVocab = 4096 * kVerifySeg;

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

// Accepted positions of sequence i, by one converged warp; -1 for a draft
// length or a drafted token out of range.
__device__ __forceinline__ int verify_accept(const VerifyParams &p, int i, int lane)
{
    const int nd = p.n_draft ? p.n_draft[i] : p.b;
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

// One CTA per sequence.
__global__ void __launch_bounds__(kVerifyThreads)
    bd_spec_verify_kernel(const VerifyParams p)
{
    extern __shared__ double seg[]; // sum of each segment's weights
    __shared__ int s_n;
    __shared__ int s_alive;
    const int i = blockIdx.x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp == 0) {
        const int n = verify_accept(p, i, lane);
        if (lane == 0) {
            s_n = n;
            s_alive = 0;
            if (n < 0)
                raise_device_code(DEV_BAD_CACHE_LEN);
            p.n_accept[i] = max(n, 0);
            p.next_token[i] = -1;
        }
    }
    __syncthreads();
    const int n = s_n;
    if (n < 0)
        return;
    const int nd = p.n_draft ? p.n_draft[i] : p.b;
    const float *pr = p.target_prob + ((size_t)i * (p.b + 1) + n) * p.V;
    const float *qr = n < nd && p.draft_prob ? p.draft_prob + ((size_t)i * p.b + n) * p.V : nullptr;
    const int point = n < nd && !p.draft_prob ? p.draft[(size_t)i * p.b + n] : -1;
    const int segs = (p.V + kVerifySeg - 1) / kVerifySeg;
    bool residual = n < nd;

    auto weight = [&](int t) -> double {
        double w = pr[t];
        if (residual)
            w -= qr ? (double)qr[t] : (t == point ? 1.0 : 0.0);
        return w > 0.0 ? w : 0.0;
    };
    for (;;) {
        for (int g = warp; g < segs; g += kVerifyThreads / 32) {
            double part = 0.0;
#pragma unroll 8
            for (int t = g * kVerifySeg + lane; t < min(p.V, (g + 1) * kVerifySeg); t += 32)
                part += weight(t);
            part = warp_sum(part);
            if (lane == 0) {
                seg[g] = part;
                if (part > 0.0)
                    s_alive = 1;
            }
        }
        __syncthreads();
        if (s_alive || !residual)
            break;
        residual = false; // nothing left of p - q: draw from p
        __syncthreads();
    }
    if (warp != 0 || !s_alive)
        return;
    double total = 0.0;
    int last = 0; // last segment with mass
    for (int g = 0; g < segs; ++g) {
        total += seg[g];
        if (seg[g] > 0.0)
            last = g;
    }
    const double want = (double)p.u_sample[i] * total;
    double before = 0.0;
    int g = 0;
    for (; g < last; ++g) {
        if (before + seg[g] > want)
            break;
        before += seg[g];
    }
    // lane l takes entries 32 l .. 32 l + 31 of segment g
    const int t0 = g * kVerifySeg + lane * 32, t1 = min(p.V, t0 + 32);
    double mine = 0.0;
    int last_pos = -1;
    for (int t = t0; t < t1; ++t) {
        const double w = weight(t);
        mine += w;
        if (w > 0.0)
            last_pos = t;
    }
    double incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const double up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o)
            incl += up;
    }
    double run = before + (incl - mine);
    int found = INT_MAX;
    for (int t = t0; t < t1; ++t) {
        const double w = weight(t);
        run += w;
        if (w > 0.0 && run > want) {
            found = t;
            break;
        }
    }
    found = __reduce_min_sync(0xffffffffu, found);
    last_pos = __reduce_max_sync(0xffffffffu, last_pos);
    if (lane == 0)
        p.next_token[i] = found == INT_MAX ? last_pos : found;
}

} // namespace bd
