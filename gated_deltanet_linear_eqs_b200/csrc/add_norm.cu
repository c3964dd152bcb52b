// add_norm.cu -- the root-mean-square norm with the residual's addition, and its reverse mode.
//
//     h = x + residual,   n = h / sqrt(mean(h^2) + eps),   o = (1 + w) n          per row of C values
//
// (the zero-centred gain of the gated RMSNorm).  The norm is taken of the 32-bit sum; h is its
// rounding.  8-bit outputs: for every `group` columns scale = max|o| / 448 and o8 = e4m3(o / scale),
// quantised from the 32-bit o.  Reverse mode, from the stored h:
//     dn = d_o (1 + w),   dx = (dn - n mean(dn n)) / sqrt(mean(h^2) + eps) + d_h,   dw = sum_rows d_o n.
//
// Streaming passes bound by HBM.  A row is held in registers by one block (8 consecutive values a
// thread and vector, at most kVec vectors a thread), so everything is read once; several rows' blocks
// share an SM, and their loads hide each other's row sums.  Products and sums are packed, two 32-bit values an
// instruction: with single ones the SMs issue for half the time and more, and the passes take a fifth longer.
// Measured, 16 bits: 32768 rows of 2048 with a residual 83 us (6.5 TB/s); 8191 rows of 5120 to 8 bits 53 us
// (5.5 TB/s); 16384 rows of 4096 in the reverse mode 102 us (5.3 TB/s); 50 and 97 us in short runs.
#include <cuda_fp8.h>
#include <float.h>

#include "common.cuh"
#include "internal.h"
#include "sm100.cuh"

namespace gdn {

namespace {

using sm100::add2;
using sm100::fma2;
using sm100::mul2;
using sm100::pair;
using sm100::unpair;

constexpr int kVec = 4;             // vectors of 8 values a thread, at most
constexpr int kNormBwdBlocks = 592; // blocks of the reverse mode (four an SM): rows of the dw partials

// 8 values as four pairs of floats
__device__ __forceinline__ void st8(__nv_bfloat16* p, const uint64_t* x) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float a, b;
        unpair(x[j], a, b);
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        w[j] = *reinterpret_cast<const uint32_t*>(&h);
    }
    __stcs(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
}
__device__ __forceinline__ void st8(float* p, const uint64_t* x) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float4 f;
        unpair(x[2 * i], f.x, f.y);
        unpair(x[2 * i + 1], f.z, f.w);
        __stcs(reinterpret_cast<float4*>(p) + i, f);
    }
}
// 8 values as loaded, unpacked when they are needed (16-bit values take half the registers until then)
template <typename T>
struct Raw8 {
    uint4 u[sizeof(T) / 2];
    __device__ __forceinline__ void load(const T* p) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) u[i] = __ldcs(reinterpret_cast<const uint4*>(p) + i);
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) u[i] = make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void get(uint64_t* x) const {
        if constexpr (sizeof(T) == 2) {
            const uint32_t w[4] = {u[0].x, u[0].y, u[0].z, u[0].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = pair(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xffff0000u));
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                x[2 * i] = pair(__uint_as_float(u[i].x), __uint_as_float(u[i].y));
                x[2 * i + 1] = pair(__uint_as_float(u[i].z), __uint_as_float(u[i].w));
            }
        }
    }
};
// 8 of the weights (read by every row: cached)
__device__ __forceinline__ void ld_w(const float* p, uint64_t* x) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float4 a = __ldg(reinterpret_cast<const float4*>(p) + i);
        x[2 * i] = pair(a.x, a.y);
        x[2 * i + 1] = pair(a.z, a.w);
    }
}
__device__ __forceinline__ float sum_pair(uint64_t x) {
    float a, b;
    unpair(x, a, b);
    return a + b;
}
// the larger, NaN if either is
__device__ __forceinline__ float max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}
__device__ __forceinline__ float max_abs8(const uint64_t* v) {
    float top = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float a, b;
        unpair(v[j], a, b);
        asm("max.NaN.abs.f32 %0, %0, %1, %2;" : "+f"(top) : "f"(a), "f"(b));
    }
    return top;
}
__device__ __forceinline__ float warp_max_nan(float x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x = max_nan(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}

// Sums over the block's threads (in warp order, so the same on every run); `s` is used once a call.
template <int N>
__device__ __forceinline__ void block_sum(float (&x)[N], float (*s)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = warp_sum(x[i]);
    const int nw = blockDim.x >> 5;
    if (nw == 1) return;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) s[threadIdx.x >> 5][i] = x[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = 0.f;
    for (int w = 0; w < nw; ++w)
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] += s[w][i];
}

// OUT: 0 = o in T, 1 = e4m3 with a scale a row, 2 = e4m3 with a scale for every 128 columns
template <typename T, int NV, int OUT>
__global__ void __launch_bounds__(512)
add_norm_kernel(const T* x, const T* res, const float* __restrict__ w, void* o,
                T* h, float* scales, int C, float eps) {  // h and o may be x or res
    __shared__ float s_sum[16][1], s_max[16];
    const long long row = blockIdx.x;
    const int nvec = C / 8, tid = threadIdx.x;
    // the whole row is asked for before anything waits on it
    Raw8<T> xv[NV], rv[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = tid + i * blockDim.x;
        xv[i].zero();
        rv[i].zero();
        if (c < nvec) {
            xv[i].load(x + row * C + c * 8);
            if (res) rv[i].load(res + row * C + c * 8);
        }
    }
    uint64_t v[NV][4], ss2 = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = tid + i * blockDim.x;
        xv[i].get(v[i]);
        if (res) {
            uint64_t r[4];
            rv[i].get(r);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[i][j] = add2(v[i][j], r[j]);
        }
        if (h && c < nvec) st8(h + row * C + c * 8, v[i]);
#pragma unroll
        for (int j = 0; j < 4; ++j) ss2 = fma2(v[i][j], v[i][j], ss2);
    }
    float ss[1] = {sum_pair(ss2)};
    block_sum(ss, s_sum);
    const float r = 1.f / sqrtf(ss[0] / (float)C + eps);
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = tid + i * blockDim.x;
        if (c >= nvec) continue;
        uint64_t g[4];
        ld_w(w + c * 8, g);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[i][j] = mul2(v[i][j], pair(r, r));
            v[i][j] = fma2(v[i][j], g[j], v[i][j]);
        }
        if constexpr (OUT == 0) st8(static_cast<T*>(o) + row * C + c * 8, v[i]);
        if constexpr (OUT == 1) top = max_nan(top, max_abs8(v[i]));
    }
    if constexpr (OUT != 0) {
        if constexpr (OUT == 1) {
            top = warp_max_nan(top);
            if ((tid & 31) == 0) s_max[tid >> 5] = top;
            __syncthreads();
            for (int k = 0; k < (int)(blockDim.x >> 5); ++k) top = max_nan(top, s_max[k]);
            if (tid == 0) scales[row] = __fdiv_rn(top, 448.f);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = tid + i * blockDim.x;
            if constexpr (OUT == 2) {  // 16 neighbouring threads hold a group
                top = max_abs8(v[i]);
#pragma unroll
                for (int q = 8; q > 0; q >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, q));
            }
            float scale = __fdiv_rn(top, 448.f);
            if (OUT == 2 && c < nvec && (tid & 15) == 0) scales[row * (C / 128) + c / 16] = scale;
            if (c >= nvec) continue;
            if (scale > 0.f && scale < FLT_MIN) {  // its reciprocal would not be finite
                scale *= 18446744073709551616.f;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    v[i][j] = mul2(v[i][j], pair(18446744073709551616.f, 18446744073709551616.f));
            }
            // o / scale: the product with the reciprocal, corrected by its remainder, so that no more values than
            // with a division fall on the other side of a tie (7 of 10 million, and the same time).  A group of
            // zeros keeps the scale 0 and gives zeros; one with an infinity has no remainders.
            const float inv = scale == 0.f ? 0.f : __frcp_rn(scale), neg = scale <= FLT_MAX ? -scale : 0.f;
            uint32_t u[2];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float2 f;
                const uint64_t t = mul2(v[i][j], pair(inv, inv));
                unpair(fma2(fma2(t, pair(neg, neg), v[i][j]), pair(inv, inv), t), f.x, f.y);
                const uint32_t q = __nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3);
                u[j / 2] = j % 2 ? u[j / 2] | (q << 16) : q;
            }
            __stcs(reinterpret_cast<uint2*>(static_cast<uint8_t*>(o) + row * C + c * 8), make_uint2(u[0], u[1]));
        }
    }
}

// Rows blockIdx.x, + gridDim.x, ..: dx, and the block's part of dw in part[blockIdx.x][C].
template <typename T, int NV>
__global__ void __launch_bounds__(512)
add_norm_bwd_kernel(const T* __restrict__ h, const float* __restrict__ w, const T* d_o,
                    const T* d_h, T* dx, float* __restrict__ part, long long rows, int C,  // dx may be d_o or d_h
                    float eps) {
    __shared__ float s_sum[2][16][2];
    const int nvec = C / 8, tid = threadIdx.x;
    uint64_t acc[NV][4];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0;
    int turn = 0;
    for (long long row = blockIdx.x; row < rows; row += gridDim.x, turn ^= 1) {
        // the whole row is asked for before anything waits on it
        Raw8<T> hv[NV], gv[NV], ev[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = tid + i * blockDim.x;
            hv[i].zero();
            gv[i].zero();
            ev[i].zero();
            if (c < nvec) {
                hv[i].load(h + row * C + c * 8);
                gv[i].load(d_o + row * C + c * 8);
                if (d_h) ev[i].load(d_h + row * C + c * 8);
            }
        }
        uint64_t s0 = 0, s1 = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = tid + i * blockDim.x;
            if (c >= nvec) continue;
            uint64_t wv[4], v[4], g[4];
            ld_w(w + c * 8, wv);
            hv[i].get(v);
            gv[i].get(g);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s0 = fma2(v[j], v[j], s0);
                s1 = fma2(v[j], fma2(g[j], wv[j], g[j]), s1);
            }
        }
        float s[2] = {sum_pair(s0), sum_pair(s1)};
        block_sum(s, s_sum[turn]);  // two buffers: the next row's writes need not wait for this one's reads
        const float r = 1.f / sqrtf(s[0] / (float)C + eps);
        const float m = -s[1] * r / (float)C;  // - mean(dn n)
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = tid + i * blockDim.x;
            if (c >= nvec) continue;
            uint64_t wv[4], v[4], g[4], e[4];
            ld_w(w + c * 8, wv);
            hv[i].get(v);
            gv[i].get(g);
            ev[i].get(e);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint64_t n = mul2(v[j], pair(r, r));
                acc[i][j] = fma2(g[j], n, acc[i][j]);
                e[j] = fma2(pair(r, r), fma2(n, pair(m, m), fma2(g[j], wv[j], g[j])), e[j]);
            }
            st8(dx + row * C + c * 8, e);
        }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = tid + i * blockDim.x;
        if (c < nvec) st8(part + (size_t)blockIdx.x * C + c * 8, acc[i]);
    }
}

// dw[c] = sum of the partials, in the same order on every run: 32 warps share the blocks of 32 columns.
__global__ void __launch_bounds__(1024)
add_norm_dw_kernel(const float* __restrict__ part, float* __restrict__ dw, int blocks, int C) {
    __shared__ float s[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    float t = 0.f;
    if (c < C) {
#pragma unroll 8
        for (int b = warp; b < blocks; b += 32) t += __ldcs(part + (size_t)b * C + c);
    }
    s[warp][lane] = t;
    __syncthreads();
    t = warp_sum(s[lane][warp]);  // column `warp` of the 32
    if (lane == 0 && blockIdx.x * 32 + warp < C) dw[blockIdx.x * 32 + warp] = t;
}

// threads of a block for C columns with NV vectors a thread
int threads_for(int C, int nv) {
    const int per = (C / 8 + nv - 1) / nv;
    return (per + 31) / 32 * 32;
}
// Vectors a thread: one where a row fits a warp, two while the block has at most 512 threads, else four.  16 bits,
// with one, two and four: 32768 rows of 2048 forward 83, 83 and 84 us, 8191 rows of 5120 to 8 bits 50, 50 and 51 us;
// 16384 rows of 4096 in the reverse mode 140 us with one (its registers: fewer rows at once) and 100 us with two.
int vectors_for(int C) { return C <= 256 ? 1 : C <= 8192 ? 2 : kVec; }

template <typename T, int NV>
cudaError_t launch_fwd(const AddNormArgs& a, cudaStream_t st) {
    const unsigned grid = (unsigned)a.rows;
    const int threads = threads_for(a.C, NV);
    const T *x = static_cast<const T*>(a.x), *res = static_cast<const T*>(a.residual);
    T* h = static_cast<T*>(a.h);
    if (a.scales == nullptr)
        add_norm_kernel<T, NV, 0><<<grid, threads, 0, st>>>(x, res, a.w, a.o, h, nullptr, a.C, a.eps);
    else if (a.group == a.C && a.C != 128)
        add_norm_kernel<T, NV, 1><<<grid, threads, 0, st>>>(x, res, a.w, a.o, h, a.scales, a.C, a.eps);
    else
        add_norm_kernel<T, NV, 2><<<grid, threads, 0, st>>>(x, res, a.w, a.o, h, a.scales, a.C, a.eps);
    return cudaGetLastError();
}
template <typename T>
cudaError_t launch_fwd_type(const AddNormArgs& a, cudaStream_t st) {
    switch (vectors_for(a.C)) {
        case 1: return launch_fwd<T, 1>(a, st);
        case 2: return launch_fwd<T, 2>(a, st);
        default: return launch_fwd<T, kVec>(a, st);
    }
}

unsigned bwd_blocks(long long rows) { return (unsigned)(rows < kNormBwdBlocks ? rows : kNormBwdBlocks); }

template <typename T, int NV>
cudaError_t launch_bwd(const AddNormArgs& a, cudaStream_t st) {
    const unsigned grid = bwd_blocks(a.rows);
    float* part = static_cast<float*>(a.ws);
    add_norm_bwd_kernel<T, NV><<<grid, threads_for(a.C, NV), 0, st>>>(
        static_cast<const T*>(a.h), a.w, static_cast<const T*>(a.d_o), static_cast<const T*>(a.d_h),
        static_cast<T*>(a.dx), part, a.rows, a.C, a.eps);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    add_norm_dw_kernel<<<(unsigned)((a.C + 31) / 32), 1024, 0, st>>>(part, a.dw, (int)grid, a.C);
    return cudaGetLastError();
}
template <typename T>
cudaError_t launch_bwd_type(const AddNormArgs& a, cudaStream_t st) {
    switch (vectors_for(a.C)) {
        case 1: return launch_bwd<T, 1>(a, st);
        case 2: return launch_bwd<T, 2>(a, st);
        default: return launch_bwd<T, kVec>(a, st);
    }
}

}  // namespace

size_t add_norm_workspace_bytes(long long rows, int C) {
    return rows < 1 ? 0 : (size_t)bwd_blocks(rows) * C * sizeof(float);
}

cudaError_t launch_add_norm(const AddNormArgs& a, cudaStream_t st) {
    if (a.rows == 0) return cudaSuccess;
    return a.dtype == GDN_BF16 ? launch_fwd_type<__nv_bfloat16>(a, st) : launch_fwd_type<float>(a, st);
}

cudaError_t launch_add_norm_backward(const AddNormArgs& a, cudaStream_t st) {
    if (a.rows == 0) return cudaMemsetAsync(a.dw, 0, sizeof(float) * a.C, st);
    return a.dtype == GDN_BF16 ? launch_bwd_type<__nv_bfloat16>(a, st) : launch_bwd_type<float>(a, st);
}

}  // namespace gdn
