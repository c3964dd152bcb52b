// linear_attn.cu -- the decayed linear attention: segment plan, the passes of the prompt and of its
// gradients, the fp32 kernel, the sum over shared heads and the one-token step.
// The formulas and the roles that the kernels play are in linear_attn.cuh.
#include "linear_attn.cuh"
#include "sm100.cuh"

namespace gdn {

namespace {

// ============================================================================ fp32 kernel
// One CTA per (segment, head, VS columns of v), 8 warps, 64-token chunks on warp-level tf32 products.  The
// columns of the state and of the outputs do not depend on each other, so they are cut over CTAs at the price
// of computing the scores in each.
//
// A product of fp32 values x y is taken as xh yh + xh yl + xl yh, x = xh + xl with xh = x rounded to tf32's 11
// bits (Markidis et al. 2018, Ootomo and Yokota 2022): what is left out is 2^-22 of |x y|, against 2^-24 for a fused
// multiply-add, and the sums stay fp32.
// Tiles of a chunk (Q, K, V rows with padded strides, so that fragments are read without bank conflicts) come
// by asynchronous copies into two buffers, the next chunk's while this one is computed; the state is kept in
// fragments (registers) and copied to shared memory as the operand of Q S.
template <int D, int VS>
struct LaTf {
    static constexpr int C = kLaChunk;
    static constexpr int LD = D + 4, LV = VS + 8, LP = C + 4;  // row strides in floats
    static constexpr int Q = 0, K = Q + C * LD, V = K + C * LD, BUF = V + C * LV;
    static constexpr int S = 2 * BUF;                // [D][LV]
    static constexpr int P = S + D * LV;             // [i][j]
    static constexpr int PW = P + C * LP;            // e^{g n}, n = 0 .. C
    static constexpr int DEC = PW + C + 4;           // e^{g n} as two floats: of a full chunk, of the last one
    static constexpr int BYTES = (DEC + 4) * 4;
    static constexpr int SG = D / 16;                // 16-row tiles of the state
    static constexpr int SN = VS / 8 / (8 / SG);     // its 8-column tiles of a warp (D = 64: two warps a row tile)
    static constexpr int YN = VS / 16;               // 8-column tiles of the outputs of a warp (4 x 2 warps)
};

__device__ __forceinline__ void tf_split(float x, uint32_t& hi, uint32_t& lo) {
    // to nearest, ties away (a NaN stays one in lo; within 2^-12 of the largest float hi is infinite)
    hi = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;
    lo = __float_as_uint(x - __uint_as_float(hi));
}
__device__ __forceinline__ void tf_mma(float* c, const uint32_t* a, const uint32_t* b) {
    asm volatile(
        "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
// acc[n] += A (16 x k) B (k x 8 N): lane 4 r + c reads a(r, c), a(r + 8, c), a(r, c + 4), a(r + 8, c + 4) of each
// 8-wide step of A and b(c, r), b(c + 4, r) of each 8-column tile of B.  The tensor cores' sums are truncated,
// not rounded, so they are kept short: the small products in sums of their own, the large ones 8 steps long,
// added to acc by the CUDA cores (an error of 3e-7 of y, 1.1e-6 with one long sum).
template <int N, typename FA, typename FB>
__device__ __forceinline__ void tf_product(float (*acc)[4], int k, FA a, FB b) {
#pragma unroll 1
    for (int k0 = 0; k0 < k; k0 += 64) {
        float big[N][4] = {}, small[N][4] = {};
#pragma unroll 2
        for (int x = k0; x < k0 + 64; x += 8) {
            uint32_t ah[4], al[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) tf_split(a(8 * (e & 1), x + 4 * (e >> 1)), ah[e], al[e]);
#pragma unroll
            for (int n = 0; n < N; ++n) {
                uint32_t bh[2], bl[2];
                tf_split(b(x, 8 * n), bh[0], bl[0]);
                tf_split(b(x + 4, 8 * n), bh[1], bl[1]);
                tf_mma(small[n], al, bh);
                tf_mma(big[n], ah, bh);
                tf_mma(small[n], ah, bl);
            }
        }
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[n][e] += big[n][e] + small[n][e];
    }
}
__device__ __forceinline__ void copy16(float* dst, const float* src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(sm100::smem_u32(dst)), "l"(src),
                 "r"(there ? 16 : 0)
                 : "memory");
}

template <int D, int VS>
__global__ void __launch_bounds__(256)
la_tf_kernel(const LaParams p) {
    using M = LaTf<D, VS>;
    constexpr int C = M::C;
    extern __shared__ float4 sm4[];
    float* sm = reinterpret_cast<float*>(sm4);
    float *S = sm + M::S, *P = sm + M::P, *pw = sm + M::PW;
    const int h = blockIdx.x % p.H, tid = threadIdx.x, c0 = blockIdx.y * VS;
    const int warp = tid >> 5, lane = tid & 31, lr = lane >> 2, lc = lane & 3;
    LaSegment sg;
    if (!la_find_segment(p, blockIdx.x / p.H, &sg)) return;
    if (p.state_only && sg.idx == (p.reverse ? 0 : sg.count - 1)) return;  // nobody starts behind it
    const int nch = (sg.len + C - 1) / C;
    const float* q = static_cast<const float*>(p.q);
    const float* k = static_cast<const float*>(p.k);
    const float* v = static_cast<const float*>(p.v);
    const int Hq = p.H / p.qdiv, Hk = p.H / p.kdiv, Hv = p.H / p.vdiv;
    auto place = [&](int cc) { return p.reverse ? nch - 1 - cc : cc; };
    // rows past the end of the document are zero (and not read)
    auto fetch = [&](int cc) {
        float* to = sm + (cc & 1) * M::BUF;
        const int c = place(cc), n = min(C, sg.len - c * C);
        const size_t tok = (size_t)sg.t0 + (size_t)c * C;
        for (int e = tid; e < C * (D / 4); e += 256) {
            const int i = e / (D / 4), x = (e % (D / 4)) * 4;
            const size_t at = i < n ? tok + i : tok;
            copy16(to + M::K + i * M::LD + x, k + (at * Hk + h / p.kdiv) * D + x, i < n);
            if (!p.state_only) copy16(to + M::Q + i * M::LD + x, q + (at * Hq + h / p.qdiv) * D + x, i < n);
        }
        for (int e = tid; e < C * (VS / 4); e += 256) {
            const int i = e / (VS / 4), x = (e % (VS / 4)) * 4;
            const size_t at = i < n ? tok + i : tok;
            copy16(to + M::V + i * M::LV + x, v + (at * Hv + h / p.vdiv) * D + c0 + x, i < n);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    if (nch > 0) fetch(0);

    const float g = p.log_decay[h];
    float2* dec2 = reinterpret_cast<float2*>(sm + M::DEC);
    if (tid >= 192 && tid < 194) dec2[tid - 192] = la_power2(g, tid == 192 ? C : sg.len - (nch - 1) * C);
    for (int n = tid; n <= C; n += 256) pw[n] = expf(g * (float)n);

    // ---- the state: this warp's 16 rows k, SN tiles of 8 columns v, in fragments
    const int sk = warp % M::SG * 16 + lr, sv = warp / M::SG * M::SN * 8;
    const size_t DD = (size_t)D * D;
    auto memory = [&](int n, int e) {  // element e of tile n
        const int kk = sk + 8 * (e >> 1), vv = c0 + sv + 8 * n + 2 * lc + (e & 1);
        return p.state_t ? vv * D + kk : kk * D + vv;
    };
    float st[M::SN][4];
    const float* s_in = !p.state_only && p.s_in ? p.s_in + ((size_t)sg.doc * p.H + h) * DD : nullptr;
#pragma unroll
    for (int n = 0; n < M::SN; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) st[n][e] = s_in ? s_in[memory(n, e)] : 0.f;
    const int behind = p.state_only ? 0 : p.reverse ? sg.count - 1 - sg.idx : sg.idx;
    if (behind > 0) {
        const float2 full = la_power2(g, p.L), last = la_power2(g, sg.doc_len - (sg.count - 1) * p.L);
        for (int b = 0; b < behind; ++b) {
            const int r = p.reverse ? sg.count - 1 - b : b;
            // (offsets that fall and rise again make more segments than the grid: those have no local state)
            if (sg.first_id + r >= (int)(gridDim.x / p.H)) continue;
            const float2 w = r == sg.count - 1 ? last : full;
            const float* loc = p.local + ((size_t)(sg.first_id + r) * p.H + h) * DD;
#pragma unroll
            for (int n = 0; n < M::SN; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) st[n][e] = fmaf(st[n][e], w.x, fmaf(st[n][e], w.y, loc[memory(n, e)]));
        }
    }
    auto publish = [&]() {
#pragma unroll
        for (int n = 0; n < M::SN; ++n)
#pragma unroll
            for (int r = 0; r < 2; ++r)
                *reinterpret_cast<float2*>(S + (sk + 8 * r) * M::LV + sv + 8 * n + 2 * lc) =
                    make_float2(st[n][2 * r], st[n][2 * r + 1]);
    };
    if (!p.state_only) publish();

    const int i0 = warp % 4 * 16, half = warp / 4;  // this warp's tokens and half of the columns
    for (int cc = 0; cc < nch; ++cc) {
        const int c = place(cc), n = min(C, sg.len - c * C);
        const float *qs = sm + (cc & 1) * M::BUF + M::Q, *ks = sm + (cc & 1) * M::BUF + M::K,
                    *vs = sm + (cc & 1) * M::BUF + M::V;
        if (cc + 1 < nch) {
            fetch(cc + 1);
            asm volatile("cp.async.wait_group 1;" ::: "memory");
        } else {
            asm volatile("cp.async.wait_group 0;" ::: "memory");
        }
        __syncthreads();
        if (!p.state_only) {
            // ---- scores of tokens i0 .. +15, keys 32 half .. +31, decayed and masked
            float acc[4][4] = {};
            tf_product<4>(acc, D, [&](int r, int x) { return qs[(i0 + lr + r) * M::LD + x + lc]; },
                          [&](int x, int m) { return ks[(32 * half + m + lr) * M::LD + x + lc]; });
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    float o[2];
                    const int i = i0 + lr + 8 * r, j = 32 * half + 8 * m + 2 * lc;
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int d = p.reverse ? j + e - i : i - j - e;
                        o[e] = d >= 0 ? acc[m][2 * r + e] * pw[d] * p.p_scale : 0.f;
                    }
                    *reinterpret_cast<float2*>(P + i * M::LP + j) = make_float2(o[0], o[1]);
                }
            __syncthreads();
            // ---- outputs of tokens i0 .. +15, columns VS / 2 half ..
            float y[M::YN][4] = {};
            const int v0 = VS / 2 * half;
            tf_product<M::YN>(y, D, [&](int r, int x) { return qs[(i0 + lr + r) * M::LD + x + lc]; },
                              [&](int x, int m) { return S[(x + lc) * M::LV + v0 + m + lr]; });
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int i = i0 + lr + 8 * r;
                const float f = i < n ? pw[p.reverse ? n - 1 - i : i + 1] * p.inter_scale : 0.f;
#pragma unroll
                for (int m = 0; m < M::YN; ++m) {
                    y[m][2 * r] *= f;
                    y[m][2 * r + 1] *= f;
                }
            }
            tf_product<M::YN>(y, C, [&](int r, int x) { return P[(i0 + lr + r) * M::LP + x + lc]; },
                              [&](int x, int m) { return vs[(x + lc) * M::LV + v0 + m + lr]; });
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int i = i0 + lr + 8 * r;
                if (i >= n) continue;
                float* o = static_cast<float*>(p.out) + (((size_t)sg.t0 + (size_t)c * C + i) * p.H + h) * D + c0 + v0;
#pragma unroll
                for (int m = 0; m < M::YN; ++m)
                    *reinterpret_cast<float2*>(o + 8 * m + 2 * lc) = make_float2(y[m][2 * r], y[m][2 * r + 1]);
            }
        }
        // ---- state: the chunk's own sum, weighted in token j, then added to the decayed state
        {
            float acc[M::SN][4] = {};
            tf_product<M::SN>(acc, C,
                              [&](int r, int x) {
                                  const int j = x + lc;
                                  const float f = p.reverse ? pw[j + 1] : j < n ? pw[n - 1 - j] : 0.f;
                                  return ks[j * M::LD + sk + r] * (f * p.state_scale);
                              },
                              [&](int x, int m) { return vs[(x + lc) * M::LV + sv + m + lr]; });
            const float2 dec = dec2[n < C];
#pragma unroll
            for (int m = 0; m < M::SN; ++m)
#pragma unroll
                for (int e = 0; e < 4; ++e) st[m][e] = fmaf(st[m][e], dec.x, fmaf(st[m][e], dec.y, acc[m][e]));
        }
        __syncthreads();  // S, P and this chunk's tiles are read
        if (!p.state_only && cc + 1 < nch) publish();
    }
    // ---- what is behind the segment: its local state, or the document's last state
    float* dst = nullptr;
    if (p.state_only)
        dst = p.local + ((size_t)(sg.first_id + sg.idx) * p.H + h) * DD;
    else if (p.s_out && sg.idx == (p.reverse ? 0 : sg.count - 1))
        dst = p.s_out + ((size_t)sg.doc * p.H + h) * DD;
    if (dst)
#pragma unroll
        for (int n = 0; n < M::SN; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) dst[memory(n, e)] = st[n][e];
}

template <int D, int VS>
cudaError_t launch_tf(const LaParams& p, int nseg, cudaStream_t st) {
    cudaError_t e = cudaFuncSetAttribute(la_tf_kernel<D, VS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         LaTf<D, VS>::BYTES);
    if (e != cudaSuccess) return e;
    la_tf_kernel<D, VS><<<dim3((unsigned)((size_t)nseg * p.H), D / VS), 256, LaTf<D, VS>::BYTES, st>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_f32(const LaParams& p, int nseg, int d, cudaStream_t st) {
    // 32 columns a CTA where all those CTAs run at once (the scores are then computed more often): 64 tokens of
    // 74 heads of 64 take 8.9 us so and 11.1 us with 64 columns, of 100 heads 15.8 and 11.2 us
    const bool wide = (long long)nseg * p.H * (d / 32) > 148;
    if (d == 128) return wide ? launch_tf<128, 64>(p, nseg, st) : launch_tf<128, 32>(p, nseg, st);
    return wide ? launch_tf<64, 64>(p, nseg, st) : launch_tf<64, 32>(p, nseg, st);
}

// ============================================================================ shared heads
// dk and dv of a k / v head shared by `group` heads: the sum of the heads' parts, in fp32 and in
// head order.  part [T, H, d] fp32 -> out [T, H / group, d]; rows outside the documents have no parts and are left.
template <typename T>
__global__ void __launch_bounds__(256)
la_group_sum_kernel(const float* __restrict__ part, T* __restrict__ out, int tokens, int Hk, int d4, int group,
                    const int32_t* __restrict__ cu, int num_seqs) {
    int first = 0, last = tokens;
    if (cu != nullptr) {
        first = min(max(cu[0], 0), tokens);
        last = min(max(cu[num_seqs], first), tokens);
    }
    const size_t n4 = (size_t)last * Hk * d4;
    for (size_t i = (size_t)first * Hk * d4 + (size_t)blockIdx.x * 256 + threadIdx.x; i < n4; i += (size_t)gridDim.x * 256) {
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

cudaError_t launch_group_sum(const float* part, void* out, const LaArgs& a, cudaStream_t st) {
    const int tokens = a.cu_seqlens ? a.T : a.num_seqs * a.T, group = a.H / a.Hk, d4 = a.d / 4;
    const size_t n4 = (size_t)tokens * a.Hk * d4;
    const unsigned grid = (unsigned)min((n4 + 255) / 256, (size_t)148 * 16);
    if (a.dtype == GDN_BF16)
        la_group_sum_kernel<<<grid, 256, 0, st>>>(part, static_cast<__nv_bfloat16*>(out), tokens, a.Hk, d4, group,
                                                  a.cu_seqlens, a.num_seqs);
    else
        la_group_sum_kernel<<<grid, 256, 0, st>>>(part, static_cast<float*>(out), tokens, a.Hk, d4, group, a.cu_seqlens,
                                                  a.num_seqs);
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
// Chains are cut where there are fewer of them than SMs and a cut pays.  bf16: equal shares of the CTAs, la_cut_pays
// (of packed documents only the sum of the lengths is known here: the kernels decide once more).  fp32: segments
// of at least one chunk, where a CTA for each 32 columns of each chain would leave SMs idle, the more so the
// longer the chains (of packed documents twice the mean is taken).  Measured in fp32, d = 128, cut and uncut: 128
// tokens with 2 heads 18 and 21 us, with 24 heads 27 and 22 us; 512 tokens with 24 heads 72 and 76 us, with 32 heads
// 84 and 75 us; 2048 tokens with 40 heads 333 and 399 us, with 64 heads 517 and 397 us; d = 64: 512 tokens with 48
// heads 37 and 47 us, with 100 heads 72 and 62 us.
LaPlan make_plan(int num_seqs, int T, int H, int d, bool packed, int dtype) {
    const long long tokens = packed ? T : (long long)num_seqs * T, chains = (long long)num_seqs * H;
    const long long chunks = (T + kLaChunk - 1) / kLaChunk;
    LaPlan pl;
    pl.L = (int)chunks * kLaChunk;
    pl.split = chains < kLaCtas && T > kLaChunk;
    if (dtype == GDN_BF16) {
        pl.split = pl.split && la_cut_pays(chunks, (packed ? 1 : num_seqs) * chunks * H);
    } else if (pl.split) {
        const long long mean = 2 * ((chunks + num_seqs - 1) / num_seqs), n = packed && mean < chunks ? mean : chunks;
        const long long want = (tokens * H + kLaCtas - 1) / kLaCtas;
        const long long L = (want + kLaChunk - 1) / kLaChunk * kLaChunk;
        if (L < pl.L && chains * (d / 32) * (n + 6) <= 200 * n) pl.L = (int)L;
        pl.split = pl.L < T;
    }
    pl.nseg = packed ? T / pl.L + num_seqs : num_seqs * ((T - 1) / pl.L + 1);
    return pl;
}

size_t local_bytes(const LaPlan& pl, int H, int d, int dtype) {
    return !pl.split ? 0 : (dtype == GDN_BF16 ? (size_t)kLaCtas : (size_t)pl.nseg * H) * d * d * sizeof(float);
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

LaLayout la_layout(bool backward, int num_seqs, int T, int H, int Hk, int d, bool packed) {
    const size_t tokens = packed ? (size_t)T : (size_t)num_seqs * T;
    LaLayout l;
    l.off_local = 0;
    l.off_dk = 0;
    for (int dtype : {GDN_BF16, GDN_FP32}) {  // the size serves both types
        const size_t n = up256(local_bytes(make_plan(num_seqs, T, H, d, packed, dtype), H, d, dtype));
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
    const LaPlan pl = make_plan(a.num_seqs, a.T, a.H, a.d, packed, a.dtype);
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
    p.walk = pl.split ? LA_WALK_CUT : packed && a.num_seqs <= kLaDocs ? LA_WALK_SORTED : LA_WALK_TURN;
    p.status = a.status;
    cudaError_t e;
    const auto roles = [&](const void* q, int qdiv, const void* k, int kdiv, const void* v, int vdiv) {
        p.q = q; p.qdiv = qdiv; p.k = k; p.kdiv = kdiv; p.v = v; p.vdiv = vdiv;
    };
    const auto run = [&](bool state_only) {
        p.state_only = state_only;
        return a.dtype == GDN_BF16 ? launch_la_tc(p, a.d, st) : launch_f32(p, pl.nseg, a.d, st);
    };
    // the local states, and (bf16) from them the states between the pieces: p's roles are set, s_in not yet used
    const auto locals = [&](const float* s_in) {
        p.s_in = nullptr;
        p.s_out = nullptr;
        if (cudaError_t f = run(true)) return f;
        p.s_in = s_in;
        return a.dtype == GDN_BF16 ? launch_la_scan(p, a.d, st) : cudaSuccess;
    };
    // forward in time: the local states of k, v, then y from s0 (or dq from s0 and dy)
    p.p_scale = p.inter_scale = a.scale;
    p.state_scale = 1.f;
    roles(a.q, 1, a.k, group, a.v, group);
    if (pl.split && (e = locals(a.s0)) != cudaSuccess) return e;
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
    if (pl.split && (e = locals(a.ds_final)) != cudaSuccess) return e;
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
        if ((e = launch_group_sum(part_k, a.dk_out, a, st)) != cudaSuccess) return e;
        return launch_group_sum(part_v, a.dv_out, a, st);
    }
    return cudaSuccess;
}

cudaError_t launch_linear_attn_step(const LaStepArgs& a, cudaStream_t st) {
    if (a.dtype == GDN_BF16)
        return a.d == 128 ? launch_step<128, __nv_bfloat16>(a, st) : launch_step<64, __nv_bfloat16>(a, st);
    return a.d == 128 ? launch_step<128, float>(a, st) : launch_step<64, float>(a, st);
}

}  // namespace gdn
