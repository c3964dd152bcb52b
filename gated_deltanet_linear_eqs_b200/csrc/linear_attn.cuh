// linear_attn.cuh -- what the kernels of the decayed linear attention share.
//
// Per document and head, with a decay e^g (g <= 0, one per head) and a state S in R^{d x d}:
//     S_t = e^g S_{t-1} + k_t v_t^T,      y_t = scale S_t^T q_t.
// Over a run of n tokens (local indices i, j; S the state before it):
//     y_i = scale ( sum_{j <= i} e^{g (i - j)} (q_i . k_j) v_j + e^{g (i + 1)} S^T q_i )
//     S'  = e^{g n} S + sum_j e^{g (n - 1 - j)} k_j v_j^T
// The gradients are the same two formulas with the tensors in other places:
//     dq: q <- dy, k <- v, v <- k, state S^T                           (forward in time)
//     dv: q <- k,  k <- q, v <- dy, state R, with the time reversed    (R = dL/dS)
//     dk: q <- v,  k <- dy, v <- q, state R^T, with the time reversed
// Reversed, the run sums over i >= j, the carried R (gradient of the state after the run) weighs
// e^{g (n - 1 - j)} in token j, and R' = e^{g n} R + scale sum_i e^{g (i + 1)} q_i dy_i^T, which is
// dL/dS before the run.  So one kernel, told the places ("roles") and the direction, runs all of
// them.
//
// Documents are cut into segments of L tokens that run side by side.  A first pass sums every
// segment's own k v^T ("local" states); the second starts each segment from
// sum over the segments behind it of e^{g (tokens between)} local + e^{g (..)} s_in.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace gdn {

constexpr int kLaChunk = 64;

struct LaParams {
    const void *q, *k, *v;  // roles: [T, heads, d] each
    void* out;              // [T, H, d]
    const float* log_decay;
    const float* s_in;      // state the first (reversed: last) segment starts from; NULL = 0
    float* s_out;           // state behind the last (reversed: first) segment; NULL = not written
    float* local;           // [segments, H, d, d] local states (NULL: one segment per document)
    const int32_t* cu;      // packed documents, or NULL: dense sequences of T tokens
    int num_seqs, T;        // T: tokens per sequence (dense) or of the packed stream
    int H;                  // states (and output heads)
    int qdiv, kdiv, vdiv;   // states per head of the role's tensor
    int L;                  // segment length, a multiple of kLaChunk
    float p_scale, inter_scale, state_scale;
    int reverse;
    int state_t;            // states in memory are [v role][k role] rather than [k role][v role]
    int state_only;         // first pass: write local states, no outputs
    int out_f32;            // outputs in fp32 (partial sums of shared heads)
    int* status;
};

struct LaSegment {
    int doc, idx, count;   // document, segment within it, segments of the document
    int t0, len;           // first token (of the whole stream) and tokens of the segment
    int doc_len;
    int first_id;          // id of the document's segment 0
};

// The segment with index `id` of the grid, found by the whole block (at least 256 threads; every
// thread calls it and gets the answer).  Returns false past the last segment.  Bounds taken from
// cu_seqlens are clamped to the stream, so that a bad value cannot lead outside the tensors.
__device__ __forceinline__ bool la_find_segment(const LaParams& p, int id, LaSegment* out) {
    if (p.cu == nullptr) {
        const int per = (p.T + p.L - 1) / p.L;
        const int doc = id / per;
        if (doc >= p.num_seqs) return false;
        out->doc = doc;
        out->idx = id - doc * per;
        out->count = per;
        out->t0 = doc * p.T + out->idx * p.L;
        out->len = min(p.L, p.T - out->idx * p.L);
        out->doc_len = p.T;
        out->first_id = doc * per;
        return true;
    }
    __shared__ int s_sum[8];
    __shared__ LaSegment s_seg;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int base = 0;
    for (int n0 = 0; n0 < p.num_seqs; n0 += 256) {
        const int n = n0 + tid;
        int t0 = 0, len = 0, cnt = 0;
        if (tid < 256 && n < p.num_seqs) {
            t0 = min(max(p.cu[n], 0), p.T);
            len = min(max(p.cu[n + 1], t0), p.T) - t0;
            cnt = max(1, (len + p.L - 1) / p.L);
        }
        int incl = cnt;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        if (tid < 256 && lane == 31) s_sum[warp] = incl;
        __syncthreads();
        int total = 0, before = 0;
#pragma unroll
        for (int w = 0; w < 8; ++w) {
            if (w < warp) before += s_sum[w];
            total += s_sum[w];
        }
        incl += before;
        if (tid < 256 && cnt > 0 && id - base >= incl - cnt && id - base < incl) {
            const int idx = id - base - (incl - cnt);
            s_seg = {n, idx, cnt, t0 + idx * p.L, min(p.L, len - idx * p.L), len, id - idx};
        }
        __syncthreads();
        if (id - base < total) {
            *out = s_seg;
            return true;
        }
        base += total;
    }
    return false;
}

// e^{g n} as a sum of two floats (a relative error of 2^-48 or so): it multiplies the state once a
// chunk, where one float's error would be the same each time and add up.
__device__ __forceinline__ float2 la_power2(float g, int n) {
    const double e = exp((double)g * n);
    const float hi = (float)e;
    return make_float2(hi, (float)(e - (double)hi));
}

template <int D>
__device__ __forceinline__ size_t la_state_index(int kk, int vv, int state_t) {
    return state_t ? (size_t)vv * D + kk : (size_t)kk * D + vv;
}

// The bf16 passes on the tensor cores (linear_attn_tc.cu).
cudaError_t launch_la_tc(const LaParams& p, int nseg, int d, cudaStream_t st);

struct LaPlan {
    int L;       // segment length
    int nseg;    // segments (packed: an upper bound)
    bool split;  // some document may have more than one segment
};

}  // namespace gdn
