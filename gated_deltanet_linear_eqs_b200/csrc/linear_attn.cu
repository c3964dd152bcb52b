// linear_attn.cu -- the decayed linear attention: segment plan, the passes of the prompt and of its
// gradients, the fp32 kernel, the sum over shared heads and the one-token step.
// The formulas and the roles that the kernels play are in linear_attn.cuh.
#include "linear_attn.cuh"
#include "sm100.cuh"

namespace gdn {

namespace {

// ============================================================================ fp32 kernel
// One CTA per (segment, head, VS columns of v), 256 threads, 64-token chunks on the CUDA cores: the columns
// of the state and of the outputs do not depend on each other, so they are cut over CTAs at the price of
// computing the scores in each.  Q^T and K^T (token fastest), V and the state's columns live in shared
// memory; the products are register tiles: 4 x 4 for the scores, 2 tokens x VS/8 columns for the outputs,
// TK x TV for the state.
template <int D, int VS>
struct LaSimt {
    static constexpr int C = kLaChunk;
    static constexpr int LT = C + 4;                 // row stride of the transposed tiles
    static constexpr int QT = 0;                     // [D][LT]
    static constexpr int KT = QT + D * LT;           // [D][LT]
    static constexpr int V = KT + D * LT;            // [C][VS]
    static constexpr int S = V + C * VS;             // [D][VS]
    static constexpr int PT = S + D * VS;            // [C][LT]: row j, column i
    static constexpr int PW = PT + C * LT;           // e^{g n}, n = 0 .. C
    static constexpr int DEC = PW + C + 4;           // e^{g n} as two floats: of a full chunk, of the last one
    static constexpr int BYTES = (DEC + 4) * 4;
    static constexpr int TK = D == 128 && VS == 64 ? 8 : 4;  // the state's tile of a thread
    static constexpr int TV = D * VS / 256 / TK;
    static constexpr int GV = VS / TV;                       // threads across the columns
};

template <int D, int VS>
__global__ void __launch_bounds__(256)
la_simt_kernel(const LaParams p) {
    using M = LaSimt<D, VS>;
    constexpr int C = M::C, LT = M::LT;
    extern __shared__ float sm[];
    float *qt = sm + M::QT, *kt = sm + M::KT, *vs = sm + M::V, *S = sm + M::S, *pt = sm + M::PT,
          *pw = sm + M::PW;
    const int h = blockIdx.x % p.H, tid = threadIdx.x, c0 = blockIdx.y * VS;
    LaSegment sg;
    if (!la_find_segment(p, blockIdx.x / p.H, &sg)) return;
    if (p.state_only && sg.idx == (p.reverse ? 0 : sg.count - 1)) return;  // nobody starts behind it
    const float g = p.log_decay[h];
    const int nch = (sg.len + C - 1) / C;
    float2* dec2 = reinterpret_cast<float2*>(sm + M::DEC);
    if (tid >= 192) {  // (one warp's worth of threads takes the 64-bit exponentials)
        if (tid < 194) dec2[tid - 192] = la_power2(g, tid == 192 ? C : sg.len - (nch - 1) * C);
    }
    for (int n = tid; n <= C; n += 256) pw[n] = expf(g * (float)n);

    // ---- the state this segment starts from: element e is (k, v column) in memory order
    const size_t DD = (size_t)D * D;
    auto memory = [&](int e) { return p.state_t ? (c0 + e / D) * D + e % D : e / VS * D + c0 + e % VS; };
    auto local_at = [&](int e) { return p.state_t ? e % D * VS + e / D : e; };
    if (p.state_only) {
        for (int e = tid; e < D * VS; e += 256) S[e] = 0.f;
    } else {
        const int behind = p.reverse ? sg.count - 1 - sg.idx : sg.idx;
        const float* s_in = p.s_in ? p.s_in + ((size_t)sg.doc * p.H + h) * DD : nullptr;
        float2 full = make_float2(0.f, 0.f), last = full;
        if (behind > 0) {
            full = la_power2(g, p.L);
            last = la_power2(g, sg.doc_len - (sg.count - 1) * p.L);
        }
#pragma unroll 4
        for (int e = tid; e < D * VS; e += 256) {
            const int at = memory(e);
            float x = s_in ? s_in[at] : 0.f;
            for (int b = 0; b < behind; ++b) {
                const int r = p.reverse ? sg.count - 1 - b : b;
                const float2 w = r == sg.count - 1 ? last : full;
                x = fmaf(x, w.x, fmaf(x, w.y, p.local[((size_t)(sg.first_id + r) * p.H + h) * DD + at]));
            }
            S[local_at(e)] = x;
        }
    }

    const float* q = static_cast<const float*>(p.q);
    const float* k = static_cast<const float*>(p.k);
    const float* v = static_cast<const float*>(p.v);
    const int Hq = p.H / p.qdiv, Hk = p.H / p.kdiv, Hv = p.H / p.vdiv;
    const int warp = tid >> 5, lane = tid & 31;
    for (int cc = 0; cc < nch; ++cc) {
        const int c = p.reverse ? nch - 1 - cc : cc;
        const int n = min(C, sg.len - c * C);
        const size_t tok = (size_t)sg.t0 + (size_t)c * C;
        const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
        __syncthreads();  // the last chunk's tiles are read
        // rows past the end of the document are zero; a warp takes 8 tokens x 16 columns, so that the
        // transposed stores fall into different banks
        {
            const int i = (warp & 7) * 8 + (lane & 7);
#pragma unroll
            for (int x0 = 0; x0 < D; x0 += 16) {
                const int x = x0 + (lane >> 3) * 4;
                const float4 a = i < n ? load4(k + ((tok + i) * Hk + h / p.kdiv) * D + x) : zero;
                kt[(x + 0) * LT + i] = a.x; kt[(x + 1) * LT + i] = a.y;
                kt[(x + 2) * LT + i] = a.z; kt[(x + 3) * LT + i] = a.w;
                if (!p.state_only) {
                    const float4 w = i < n ? load4(q + ((tok + i) * Hq + h / p.qdiv) * D + x) : zero;
                    qt[(x + 0) * LT + i] = w.x; qt[(x + 1) * LT + i] = w.y;
                    qt[(x + 2) * LT + i] = w.z; qt[(x + 3) * LT + i] = w.w;
                }
            }
        }
        for (int e = tid; e < C * (VS / 4); e += 256) {
            const int i = e / (VS / 4), x = (e % (VS / 4)) * 4;
            store4(vs + i * VS + x, i < n ? load4(v + ((tok + i) * Hv + h / p.vdiv) * D + c0 + x) : zero);
        }
        __syncthreads();
        if (!p.state_only) {
            // ---- scores, their decay and mask: pt[j][i]
            {
                const int j0 = (tid / 16) * 4, i0 = (tid % 16) * 4;
                float acc[4][4] = {};
#pragma unroll 16
                for (int x = 0; x < D; ++x) {
                    const float4 a = load4(kt + x * LT + j0), b = load4(qt + x * LT + i0);
                    const float av[4] = {a.x, a.y, a.z, a.w}, bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
                    for (int r = 0; r < 4; ++r)
#pragma unroll
                        for (int s = 0; s < 4; ++s) acc[r][s] = fmaf(av[r], bv[s], acc[r][s]);
                }
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    float o[4];
#pragma unroll
                    for (int s = 0; s < 4; ++s) {
                        const int d = p.reverse ? j0 + r - (i0 + s) : i0 + s - (j0 + r);
                        o[s] = d >= 0 ? acc[r][s] * pw[d] * p.p_scale : 0.f;
                    }
                    store4(pt + (j0 + r) * LT + i0, make_float4(o[0], o[1], o[2], o[3]));
                }
            }
            __syncthreads();
            // ---- outputs: a warp's 8 rows, 2 a thread; VS / 8 columns
            constexpr int CPL = VS / 8;
            float acc[2][CPL] = {};
            const int i0 = warp * 8 + (lane >> 3) * 2, s0 = (lane & 7) * CPL;
            auto product = [&](const float* a, const float* b, int len) {
#pragma unroll 16
                for (int x = 0; x < len; ++x) {
                    const float2 u = *reinterpret_cast<const float2*>(a + x * LT + i0);
                    float bv[CPL];
#pragma unroll
                    for (int s = 0; s < CPL; s += 4) {
                        const float4 w = load4(b + x * VS + s0 + s);
                        bv[s] = w.x; bv[s + 1] = w.y; bv[s + 2] = w.z; bv[s + 3] = w.w;
                    }
#pragma unroll
                    for (int s = 0; s < CPL; ++s) {
                        acc[0][s] = fmaf(u.x, bv[s], acc[0][s]);
                        acc[1][s] = fmaf(u.y, bv[s], acc[1][s]);
                    }
                }
            };
            product(qt, S, D);
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int i = i0 + r;
                const float f = i < n ? pw[p.reverse ? n - 1 - i : i + 1] * p.inter_scale : 0.f;
#pragma unroll
                for (int s = 0; s < CPL; ++s) acc[r][s] *= f;
            }
            product(pt, vs, C);
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                if (i0 + r >= n) continue;
                float* o = static_cast<float*>(p.out) + ((tok + i0 + r) * p.H + h) * D + c0 + s0;
#pragma unroll
                for (int s = 0; s < CPL; s += 4)
                    store4(o + s, make_float4(acc[r][s], acc[r][s + 1], acc[r][s + 2], acc[r][s + 3]));
            }
            __syncthreads();  // S is read above
        }
        // ---- state
        {
            constexpr int TK = M::TK, TV = M::TV;
            const int k0 = (tid / M::GV) * TK, v0 = (tid % M::GV) * TV;
            const float2 dec = dec2[n < C];
            float acc[TK][TV] = {};
#pragma unroll 2
            for (int j = 0; j < n; j += 4) {  // (rows from n on are zero)
                float kw[TK][4], f[4];
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    f[u] = j + u < n ? pw[p.reverse ? j + u + 1 : n - 1 - j - u] * p.state_scale : 0.f;
#pragma unroll
                for (int r = 0; r < TK; ++r) {
                    const float4 a = load4(kt + (k0 + r) * LT + j);
                    kw[r][0] = a.x * f[0]; kw[r][1] = a.y * f[1]; kw[r][2] = a.z * f[2]; kw[r][3] = a.w * f[3];
                }
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    float bv[TV];
#pragma unroll
                    for (int s = 0; s < TV; ++s) bv[s] = vs[(j + u) * VS + v0 + s];
#pragma unroll
                    for (int r = 0; r < TK; ++r)
#pragma unroll
                        for (int s = 0; s < TV; ++s) acc[r][s] = fmaf(kw[r][u], bv[s], acc[r][s]);
                }
            }
#pragma unroll
            for (int r = 0; r < TK; ++r)
#pragma unroll
                for (int s = 0; s < TV; ++s) {
                    float* x = S + (k0 + r) * VS + v0 + s;
                    *x = fmaf(*x, dec.x, fmaf(*x, dec.y, acc[r][s]));
                }
        }
    }
    __syncthreads();
    // ---- what is behind the segment: its local state, or the document's last state
    float* dst = nullptr;
    if (p.state_only)
        dst = p.local + ((size_t)(sg.first_id + sg.idx) * p.H + h) * DD;
    else if (p.s_out && sg.idx == (p.reverse ? 0 : sg.count - 1))
        dst = p.s_out + ((size_t)sg.doc * p.H + h) * DD;
    if (dst)
        for (int e = tid; e < D * VS; e += 256) dst[memory(e)] = S[local_at(e)];
}

template <int D, int VS>
cudaError_t launch_simt(const LaParams& p, int nseg, cudaStream_t st) {
    cudaError_t e = cudaFuncSetAttribute(la_simt_kernel<D, VS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         LaSimt<D, VS>::BYTES);
    if (e != cudaSuccess) return e;
    la_simt_kernel<D, VS><<<dim3((unsigned)((size_t)nseg * p.H), D / VS), 256, LaSimt<D, VS>::BYTES, st>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_pass(const LaParams& p, int nseg, int d, int dtype, cudaStream_t st) {
    if (dtype == GDN_BF16) return launch_la_tc(p, nseg, d, st);
    // 32 columns a CTA while 64 would leave SMs idle: the scores are then computed once more
    const bool wide = (long long)nseg * p.H * (d / 64) >= 148;
    if (d == 128) return wide ? launch_simt<128, 64>(p, nseg, st) : launch_simt<128, 32>(p, nseg, st);
    return wide ? launch_simt<64, 64>(p, nseg, st) : launch_simt<64, 32>(p, nseg, st);
}

// ============================================================================ shared heads
// dk and dv of a k / v head shared by `group` heads: the sum of the heads' parts, in fp32 and in
// head order.  part [T, H, d] fp32 -> out [T, H / group, d].
template <typename T>
__global__ void __launch_bounds__(256)
la_group_sum_kernel(const float* __restrict__ part, T* __restrict__ out, size_t n4, int d4, int group) {
    for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < n4; i += (size_t)gridDim.x * 256) {
        const size_t head = i / d4;
        const int x = (int)(i % d4);
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int m = 0; m < group; ++m) {
            const float4 a = __ldcs(reinterpret_cast<const float4*>(part) + (head * group + m) * d4 + x);
            s.x += a.x; s.y += a.y; s.z += a.z; s.w += a.w;
        }
        store4(out + i * 4, s);
    }
}

cudaError_t launch_group_sum(const float* part, void* out, size_t tokens, int Hk, int d, int group, int dtype,
                             cudaStream_t st) {
    const size_t n4 = tokens * Hk * (d / 4);
    const unsigned grid = (unsigned)min((n4 + 255) / 256, (size_t)148 * 16);
    if (dtype == GDN_BF16)
        la_group_sum_kernel<<<grid, 256, 0, st>>>(part, static_cast<__nv_bfloat16*>(out), n4, d / 4, group);
    else
        la_group_sum_kernel<<<grid, 256, 0, st>>>(part, static_cast<float*>(out), n4, d / 4, group);
    return cudaGetLastError();
}

// ============================================================================ one token
// S <- e^g S + k v^T, y = scale S^T q = scale (e^g S^T q + (k . q) v): one read and one write of the
// fp32 state.  One CTA per (sequence, head, 64 columns), 128 threads; 16 lanes read 256
// consecutive bytes of a row, every thread keeps its D/8 rows' values between the read and the
// write.
constexpr int kStepThreads = 128;
constexpr int kStepCols = 64;

template <int D, typename T>
__global__ void __launch_bounds__(kStepThreads)
la_step_kernel(const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v,
               const float* __restrict__ log_decay, float* __restrict__ state, T* __restrict__ y, int H,
               int group, float scale) {
    constexpr int LPR = kStepCols / 4, RPW = 32 / LPR, NW = kStepThreads / 32, ROWS = D / (RPW * NW);
    __shared__ float s_k[D], s_q[D], s_kq;
    __shared__ float4 s_red[NW][LPR];
    const int nh = blockIdx.x, h = nh % H;
    const size_t kv = (size_t)(nh / H) * (H / group) + h / group;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int cg = lane % LPR, rsub = lane / LPR;
    const int col = blockIdx.y * kStepCols + cg * 4;
    float* S = state + (size_t)nh * D * D;
    float4 s[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i)
        s[i] = __ldcs(reinterpret_cast<const float4*>(S + (size_t)((i * NW + warp) * RPW + rsub) * D + col));
    const float a = expf(log_decay[h]);
    const float4 vv = load4(v + kv * D + col);
    if (warp == 0) {
        float kq = 0.f;
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
            const float x = to_f32(k[kv * D + lane + 32 * j]), z = to_f32(q[(size_t)nh * D + lane + 32 * j]);
            s_k[lane + 32 * j] = x;
            s_q[lane + 32 * j] = z;
            kq = fmaf(x, z, kq);
        }
        kq = warp_sum(kq);
        if (lane == 0) s_kq = kq;
    }
    __syncthreads();
    float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int row = (i * NW + warp) * RPW + rsub;
        const float z = s_q[row], x = s_k[row];
        r.x = fmaf(s[i].x, z, r.x); r.y = fmaf(s[i].y, z, r.y);
        r.z = fmaf(s[i].z, z, r.z); r.w = fmaf(s[i].w, z, r.w);
        s[i].x = fmaf(a, s[i].x, x * vv.x); s[i].y = fmaf(a, s[i].y, x * vv.y);
        s[i].z = fmaf(a, s[i].z, x * vv.z); s[i].w = fmaf(a, s[i].w, x * vv.w);
        __stcs(reinterpret_cast<float4*>(S + (size_t)row * D + col), s[i]);
    }
#pragma unroll
    for (int o = LPR; o < 32; o <<= 1) {
        r.x += __shfl_xor_sync(0xffffffffu, r.x, o); r.y += __shfl_xor_sync(0xffffffffu, r.y, o);
        r.z += __shfl_xor_sync(0xffffffffu, r.z, o); r.w += __shfl_xor_sync(0xffffffffu, r.w, o);
    }
    if (rsub == 0) s_red[warp][cg] = r;
    __syncthreads();
    if (warp == 0 && rsub == 0) {
#pragma unroll
        for (int w = 1; w < NW; ++w) {
            const float4 b = s_red[w][cg];
            r.x += b.x; r.y += b.y; r.z += b.z; r.w += b.w;
        }
        const float kq = s_kq;
        store4(y + (size_t)nh * D + col,
               make_float4(scale * fmaf(a, r.x, kq * vv.x), scale * fmaf(a, r.y, kq * vv.y),
                           scale * fmaf(a, r.z, kq * vv.z), scale * fmaf(a, r.w, kq * vv.w)));
    }
}

template <int D, typename T>
cudaError_t launch_step(const LaStepArgs& a, cudaStream_t st) {
    la_step_kernel<D, T><<<dim3((unsigned)(a.N * a.H), D / kStepCols), kStepThreads, 0, st>>>(
        static_cast<const T*>(a.q), static_cast<const T*>(a.k), static_cast<const T*>(a.v), a.log_decay, a.state,
        static_cast<T*>(a.y), a.H, a.H / a.Hk, a.scale);
    return cudaGetLastError();
}

// ============================================================================ plan
// One segment per document where the documents alone give every SM work; otherwise segments long
// enough for their start states (d x d fp32 each) to stay a small part of their tokens.
constexpr int kMinSegment[2] = {512, 64};  // bf16, fp32 (whose chunks take about ten times as long)

LaPlan make_plan(int num_seqs, int T, int H, bool packed, int dtype) {
    const long long tokens = packed ? T : (long long)num_seqs * T;
    LaPlan pl;
    pl.L = (T + kLaChunk - 1) / kLaChunk * kLaChunk;
    if ((long long)num_seqs * H < 148) {
        const long long want = (tokens * H + 147) / 148;
        long long L = (want + kLaChunk - 1) / kLaChunk * kLaChunk;
        if (L < kMinSegment[dtype]) L = kMinSegment[dtype];
        if (L < pl.L) pl.L = (int)L;
    }
    pl.split = pl.L < T;
    pl.nseg = packed ? T / pl.L + num_seqs : num_seqs * ((T + pl.L - 1) / pl.L);
    return pl;
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

LaLayout la_layout(bool backward, int num_seqs, int T, int H, int Hk, int d, bool packed) {
    const size_t tokens = packed ? (size_t)T : (size_t)num_seqs * T;
    LaLayout l;
    l.off_local = 0;
    l.off_dk = 0;
    for (int dtype : {GDN_BF16, GDN_FP32}) {  // the size serves both types
        const LaPlan pl = make_plan(num_seqs, T, H, packed, dtype);
        const size_t n = pl.split ? up256((size_t)pl.nseg * H * d * d * 4) : 0;
        l.off_dk = n > l.off_dk ? n : l.off_dk;
    }
    l.off_dv = l.off_dk;
    l.total = l.off_dk;
    if (backward && Hk < H) {
        l.off_dv = l.off_dk + up256(tokens * H * d * 4);
        l.total = l.off_dv + up256(tokens * H * d * 4);
    }
    return l;
}

cudaError_t launch_linear_attn(const LaArgs& a, cudaStream_t st) {
    const bool packed = a.cu_seqlens != nullptr;
    const LaPlan pl = make_plan(a.num_seqs, a.T, a.H, packed, a.dtype);
    const LaLayout lay = la_layout(a.dy != nullptr, a.num_seqs, a.T, a.H, a.Hk, a.d, packed);
    char* ws = static_cast<char*>(a.ws);
    const int group = a.H / a.Hk;
    LaParams p{};
    p.log_decay = a.log_decay;
    p.local = pl.split ? reinterpret_cast<float*>(ws + lay.off_local) : nullptr;
    p.cu = a.cu_seqlens;
    p.num_seqs = a.num_seqs;
    p.T = a.T;
    p.H = a.H;
    p.L = pl.L;
    p.status = a.status;
    cudaError_t e;
    const auto roles = [&](const void* q, int qdiv, const void* k, int kdiv, const void* v, int vdiv) {
        p.q = q; p.qdiv = qdiv; p.k = k; p.kdiv = kdiv; p.v = v; p.vdiv = vdiv;
    };
    const auto run = [&](bool state_only) {
        p.state_only = state_only;
        return launch_pass(p, pl.nseg, a.d, a.dtype, st);
    };
    // forward in time: the local states of k, v, then y from s0 (or dq from s0 and dy)
    p.p_scale = p.inter_scale = a.scale;
    p.state_scale = 1.f;
    roles(a.q, 1, a.k, group, a.v, group);
    if (pl.split && (e = run(true)) != cudaSuccess) return e;
    p.s_in = a.s0;
    if (a.dy == nullptr) {
        p.out = a.y;
        p.s_out = a.s_final;
        return run(false);
    }
    roles(a.dy, 1, a.v, group, a.k, group);
    p.out = a.dq;
    p.state_t = 1;
    if ((e = run(false)) != cudaSuccess) return e;
    // reversed: the local states of q, dy, then dv and ds0, then dk
    p.reverse = 1;
    p.inter_scale = 1.f;
    p.state_scale = a.scale;
    p.state_t = 0;
    roles(a.k, group, a.q, 1, a.dy, 1);
    if (pl.split && (e = run(true)) != cudaSuccess) return e;
    float* part_k = reinterpret_cast<float*>(ws + lay.off_dk);
    float* part_v = reinterpret_cast<float*>(ws + lay.off_dv);
    p.out_f32 = group > 1;
    p.s_in = a.ds_final;
    p.s_out = a.ds0;
    p.out = group > 1 ? part_v : a.dv_out;
    if ((e = run(false)) != cudaSuccess) return e;
    roles(a.v, group, a.dy, 1, a.q, 1);
    p.out = group > 1 ? part_k : a.dk_out;
    p.s_out = nullptr;
    p.state_t = 1;
    if ((e = run(false)) != cudaSuccess) return e;
    if (group > 1) {
        const size_t tokens = packed ? (size_t)a.T : (size_t)a.num_seqs * a.T;
        if ((e = launch_group_sum(part_k, a.dk_out, tokens, a.Hk, a.d, group, a.dtype, st)) != cudaSuccess) return e;
        return launch_group_sum(part_v, a.dv_out, tokens, a.Hk, a.d, group, a.dtype, st);
    }
    return cudaSuccess;
}

cudaError_t launch_linear_attn_step(const LaStepArgs& a, cudaStream_t st) {
    if (a.dtype == GDN_BF16)
        return a.d == 128 ? launch_step<128, __nv_bfloat16>(a, st) : launch_step<64, __nv_bfloat16>(a, st);
    return a.d == 128 ? launch_step<128, float>(a, st) : launch_step<64, float>(a, st);
}

}  // namespace gdn
