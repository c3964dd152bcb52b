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
// Where the documents and heads are too few for the SMs, a chain (document, head) is cut along time.  A first
// pass sums every piece's own k v^T ("local" states), and a piece starts from
// sum over the pieces behind it of e^{g (tokens between)} local + e^{g (..)} s_in.
// fp32: segments of L tokens, one CTA each (LaSegment).  bf16: the chains' chunks are laid end to end and cut
// into equal shares, one CTA each, so that a CTA walks the end of one chain and the start of the next (LaPiece).
#pragma once

#include "common.cuh"
#include "internal.h"

namespace gdn {

constexpr int kLaChunk = 64;

// How the bf16 kernel's CTAs share the chains: in turn; cut into equal shares; or, packed documents of unlike
// lengths, longest first, in turn, back and forth (24 documents of 0 to 1200 tokens with 16 heads of 64: 43 us where
// plain turns took 60 us).
enum { LA_WALK_TURN = 0, LA_WALK_CUT = 1, LA_WALK_SORTED = 2 };

struct LaParams {
    const void *q, *k, *v;  // roles: [T, heads, d] each
    void* out;              // [T, H, d]
    const float* log_decay;
    const float* s_in;      // state the first (reversed: last) segment starts from; NULL = 0
    float* s_out;           // state behind the last (reversed: first) segment; NULL = not written
    float* local;           // fp32: [segments, H, d, d], bf16: [CTAs, d, d] local states (NULL: no chain is cut)
    const int32_t* cu;      // packed documents, or NULL: dense sequences of T tokens
    int num_seqs, T;        // T: tokens per sequence (dense) or of the packed stream
    int H;                  // states (and output heads)
    int qdiv, kdiv, vdiv;   // states per head of the role's tensor
    int L;                  // fp32: segment length, a multiple of kLaChunk
    int walk;               // bf16: LA_WALK_*
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
        const int per = (p.T - 1) / p.L + 1;
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
            cnt = (max(len, 1) - 1) / p.L + 1;
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

// ---- bf16: the shares of the CTAs -------------------------------------------------------------
// A chain of c chunks counts kLaStart + c units, kLaStart for what its start and end cost; all chains' units are
// laid end to end (document by document, its heads in turn) and cut into equal shares of at least kLaShare
// units.  A CTA whose share ends inside a chain leaves that chain's local state in slot [CTA].
constexpr int kLaStart = 3, kLaShare = 8;
constexpr int kLaCtas = 148;   // one a SM
constexpr int kLaDocs = 147;   // documents that are cut (which needs fewer chains than SMs) or sorted at most

// A cut pays where the longest chain takes longer than the two passes over the shares: uncut, a chain takes
// 6 + 1.4 us a chunk; cut, 31 + 2.4 us a chunk of a share (three launches; the two passes 0.9 and 1.5).  Measured
// uncut and cut, d = 128: one document of 2048 tokens 50 and 38 us with 16 heads, 54 and 62 us with 64, 58 and 97 us
// with 120; of 8192 tokens with 64 heads 187 and 160 us; of 1024 tokens with 16 heads 28 and 37 us.  d = 64: 2048
// tokens 47 and 34 us with 32 heads, 1024 tokens 26 and 33 us.  The gradients lie close by.
__host__ __device__ inline bool la_cut_pays(long long longest, long long all) {
    return longest > 16 + 2 * all / kLaCtas;
}

struct LaDocs {
    int cut;                  // LA_WALK_CUT, and the lengths are such that it pays
    int count;                // pieces of this CTA (cut)
    int units[kLaDocs + 1];   // cut: units of one head before each document; sorted: the documents by length
    int t0[kLaDocs], len[kLaDocs];
};
struct alignas(16) LaPiece {  // (whole words of 16 bytes: read from shared memory at once)
    int doc, h;
    int t0;            // the document's first token
    int nch, last;     // its chunks, and the tokens of the last
    int w0, w1;        // the chunks of this piece, counted in walking order
    __device__ bool starts() const { return w0 == 0; }
    __device__ bool ends() const { return w1 == nch; }
};

__device__ __forceinline__ void la_document(const LaParams& p, int doc, int* t0, int* len) {
    if (p.cu == nullptr) {
        *t0 = doc * p.T;
        *len = p.T;
    } else {  // clamped to the stream: a bad value cannot lead outside the tensors
        *t0 = min(max(p.cu[doc], 0), p.T);
        *len = min(max(p.cu[doc + 1], *t0), p.T) - *t0;
    }
}

// The documents' table, by the whole block (blockDim.x >= 160; ends with a __syncthreads).
__device__ __forceinline__ void la_make_docs(const LaParams& p, LaDocs* d) {
    const int tid = threadIdx.x;
    if (tid < p.num_seqs) {
        int t0, len;
        la_document(p, tid, &t0, &len);
        d->t0[tid] = t0;
        d->len[tid] = len;
    }
    if (tid == 0) d->cut = 0;
    __syncthreads();
    if (p.walk == LA_WALK_SORTED) {
        if (tid < p.num_seqs) {
            int rank = 0;
            const int len = d->len[tid];
            for (int n = 0; n < p.num_seqs; ++n) rank += d->len[n] > len || (d->len[n] == len && n < tid);
            d->units[rank] = tid;
        }
    } else if (tid < 32) {
        int base = 0, longest = 0;
        for (int n0 = 0; n0 < p.num_seqs; n0 += 32) {
            const int n = n0 + tid;
            const int u = n < p.num_seqs ? kLaStart + (d->len[n] + kLaChunk - 1) / kLaChunk : 0;
            longest = max(longest, __reduce_max_sync(0xffffffffu, u) - kLaStart);
            int incl = u;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, incl, o);
                if (tid >= o) incl += y;
            }
            if (n < p.num_seqs) d->units[n] = base + incl - u;
            base += __shfl_sync(0xffffffffu, incl, 31);
        }
        if (tid == 0) {
            d->units[p.num_seqs] = base;
            d->cut = la_cut_pays(longest, (long long)p.H * (base - kLaStart * p.num_seqs));
        }
    }
    __syncthreads();
}

__device__ __forceinline__ int la_shares(int all, int ctas) { return min(ctas, max(1, all / kLaShare)); }
__device__ __forceinline__ int la_share(int all, int i, int shares) { return (int)((long long)all * i / shares); }

// The pieces of share `share` where chains are cut, in order; returns their number (at most the chains').  One
// thread.  With `open_only` those that the next share goes on from.
__device__ __forceinline__ int la_cut_pieces(const LaParams& p, const LaDocs* d, int share, bool open_only,
                                             LaPiece* out) {
    const int all = p.H * d->units[p.num_seqs], shares = la_shares(all, kLaCtas);
    if (share >= shares) return 0;
    int pos = la_share(all, share, shares), doc = 0, count = 0;
    const int hi = la_share(all, share + 1, shares);
    while (p.H * d->units[doc + 1] <= pos) ++doc;
    int h = (pos - p.H * d->units[doc]) / (d->units[doc + 1] - d->units[doc]);
    while (pos < hi) {
        const int u = d->units[doc + 1] - d->units[doc], first = p.H * d->units[doc] + h * u + kLaStart;
        const int nch = u - kLaStart, w0 = max(pos - first, 0), w1 = min(hi - first, nch);
        // (an empty chain goes to the share that holds the last of its start's units)
        if ((nch > 0 ? w1 > w0 : pos < first && first <= hi) && !(open_only && w1 == nch))
            out[count++] = {doc, h, d->t0[doc], nch, d->len[doc] - (nch - 1) * kLaChunk, w0, w1};
        pos = first + nch;
        if (++h == p.H) {
            h = 0;
            ++doc;
        }
    }
    return count;
}

// The chain in place `pos` where none is cut.
__device__ __forceinline__ void la_chain(const LaParams& p, const LaDocs* d, int pos, LaPiece* out) {
    const int at = pos / p.H;
    out->doc = p.walk == LA_WALK_SORTED ? d->units[at] : at;
    out->h = pos - at * p.H;
    int len;
    la_document(p, out->doc, &out->t0, &len);
    out->nch = out->w1 = (len + kLaChunk - 1) / kLaChunk;
    out->last = len - (out->nch - 1) * kLaChunk;
    out->w0 = 0;
}

// The bf16 passes on the tensor cores (linear_attn_tc.cu).
cudaError_t launch_la_tc(const LaParams& p, int d, cudaStream_t st);
// Between the two passes: every slot's local state becomes the state at the end of its piece.
cudaError_t launch_la_scan(const LaParams& p, int d, cudaStream_t st);

struct LaPlan {
    int L;       // fp32: segment length
    int nseg;    // fp32: segments (packed: an upper bound)
    bool split;  // some chain may be cut
};

}  // namespace gdn
