// rotary.cu -- rotary positions of q and k.
//
// The first r of a head's d values form r / 2 pairs (a, b): elements (i, i + r/2) in the half layout,
// (2 i, 2 i + 1) in the interleaved one.  At position p, pair i turns by the angle p f_i:
//     (a, b) -> scale (a cos - b sin, b cos + a sin),
// and by -p f_i in the inverse form, which is also the gradient.  The other d - r values are kept.
//
// The angle is taken in 64 bits (a position of a million times a frequency of one is known to
// 1e-10 of a turn), reduced to a fraction of a turn there, and its sine and cosine in 32 bits.
// A block serves a few tokens: it computes their r / 2 (cos, sin) once into shared memory and then
// turns all heads of q and k with them, so that the trigonometry is shared by the heads and the
// pass is bound by HBM (x read once, y written once).
#include "common.cuh"
#include "internal.h"

namespace gdn {

namespace {

constexpr int kRotThreads = 256;
constexpr int kRotTokens = 8;  // tokens of a block, at most

template <typename T, int VEC>
__device__ __forceinline__ void rot_load(const T* p, float* x) {
    if constexpr (VEC == 1) {
        x[0] = to_f32(*p);
    } else {
        const uint4 u = __ldcs(reinterpret_cast<const uint4*>(p));
        const T* t = reinterpret_cast<const T*>(&u);
#pragma unroll
        for (int i = 0; i < VEC; ++i) x[i] = to_f32(t[i]);
    }
}
template <typename T, int VEC>
__device__ __forceinline__ void rot_store(T* p, const float* x) {
    if constexpr (VEC == 1) {
        *p = from_f32<T>(x[0]);
    } else {
        uint4 u;
        T* t = reinterpret_cast<T*>(&u);
#pragma unroll
        for (int i = 0; i < VEC; ++i) t[i] = from_f32<T>(x[i]);
        __stcs(reinterpret_cast<uint4*>(p), u);
    }
}

// VEC elements a thread and access: 16 bytes where every piece of the layout is a multiple of them,
// else single elements.  A unit is what a thread turns at once: VEC elements of both halves of the pairs
// (half layout), VEC / 2 whole pairs (interleaved, VEC > 1), one pair (VEC = 1), or VEC kept elements.
template <typename T, int VEC, bool INTER>
__global__ void __launch_bounds__(kRotThreads)
rotary_kernel(const RotaryArgs p, int tokens, int units) {
    extern __shared__ float2 cs[];  // [tokens][r / 2]
    const int half = p.r / 2, tid = threadIdx.x;
    const int t0 = blockIdx.x * tokens;
    const int nt = min(tokens, p.T - t0);
    for (int e = tid; e < nt * half; e += kRotThreads) {
        const int t = e / half;
        const double turns = (double)p.positions[t0 + t] * ((double)p.inv_freq[e - t * half] * 0.15915494309189535);
        float s, c;
        sincospif(2.f * (float)(turns - rint(turns)), &s, &c);
        cs[e] = make_float2(c * p.scale, (p.inverse ? -s : s) * p.scale);
    }
    __syncthreads();
    const int heads = p.a[0].heads + p.a[1].heads;
    const int turned = INTER && VEC > 1 ? p.r / VEC : half / VEC;  // units that turn; the others are kept
    // a block's threads cover whole heads; a head with more units than threads takes several steps
    const int hpb = units < kRotThreads ? kRotThreads / units : 1;
    const int hh = units < kRotThreads ? tid / units : 0;
    if (hh >= hpb) return;
    const int u0 = units < kRotThreads ? tid - hh * units : tid;
    // Two heads a step: both heads' loads are on their way before either is stored.
    const int rows = nt * heads, step = hpb * (int)gridDim.y;
    for (int row = hh + hpb * (int)blockIdx.y; row < rows; row += 2 * step) {
        const T* x[2];
        T* y[2];
        const float2* w[2];
        const bool both = row + step < rows;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const int at = b && both ? row + step : row;
            const int t = at / heads;
            int h = at - t * heads;
            const bool second = h >= p.a[0].heads;
            if (second) h -= p.a[0].heads;
            x[b] = static_cast<const T*>(second ? p.a[1].x : p.a[0].x) +
                   (long long)(t0 + t) * (second ? p.a[1].ldx : p.a[0].ldx) + (long long)h * p.d;
            y[b] = static_cast<T*>(second ? p.a[1].y : p.a[0].y) +
                   (long long)(t0 + t) * (second ? p.a[1].ldy : p.a[0].ldy) + (long long)h * p.d;
            w[b] = cs + t * half;
        }
        for (int u = u0; u < units; u += kRotThreads) {
            const bool turn = u < turned;
            const int ia = !turn ? p.r + (u - turned) * VEC : INTER ? (VEC > 1 ? u * VEC : 2 * u) : u * VEC;
            const int ib = INTER ? 2 * u + 1 : half + u * VEC;  // (not of whole interleaved pairs)
            constexpr bool PAIRS = INTER && VEC > 1;
            float v[2][VEC], z[2][VEC];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                if (b && !both) break;
                rot_load<T, VEC>(x[b] + ia, v[b]);
                if (!PAIRS && turn) rot_load<T, VEC>(x[b] + ib, z[b]);
            }
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                if (b && !both) break;
                if (turn) {
                    float o[VEC], n[VEC];
                    if constexpr (PAIRS) {
#pragma unroll
                        for (int i = 0; i < VEC / 2; ++i) {
                            const float2 f = w[b][u * (VEC / 2) + i];
                            o[2 * i] = v[b][2 * i] * f.x - v[b][2 * i + 1] * f.y;
                            o[2 * i + 1] = v[b][2 * i + 1] * f.x + v[b][2 * i] * f.y;
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < VEC; ++i) {
                            const float2 f = w[b][u * VEC + i];
                            o[i] = v[b][i] * f.x - z[b][i] * f.y;
                            n[i] = z[b][i] * f.x + v[b][i] * f.y;
                        }
                        rot_store<T, VEC>(y[b] + ib, n);
                    }
                    rot_store<T, VEC>(y[b] + ia, o);
                } else {
                    rot_store<T, VEC>(y[b] + ia, v[b]);
                }
            }
        }
    }
}

template <typename T, int VEC, bool INTER>
cudaError_t launch(const RotaryArgs& a, bool keep, cudaStream_t st) {
    const int turned = INTER && VEC > 1 ? a.r / VEC : a.r / 2 / VEC;
    const int units = turned + (keep ? (a.d - a.r) / VEC : 0);
    // many tokens: kRotTokens a block; few: one, and its heads over several blocks, so that the SMs
    // share them and a thread has few dependent steps (the angles are computed again in each)
    int tokens = a.T / (148 * 4);
    tokens = tokens < 1 ? 1 : tokens > kRotTokens ? kRotTokens : tokens;
    const unsigned grid = (unsigned)((a.T + tokens - 1) / tokens);
    const int hpb = units < kRotThreads ? kRotThreads / units : 1;
    const int steps = (tokens * (a.a[0].heads + a.a[1].heads) + 2 * hpb - 1) / (2 * hpb);
    int split = 148 * 4 / (int)(grid < 148 * 4 ? grid : 148 * 4);
    split = split > steps ? steps : split;
    rotary_kernel<T, VEC, INTER><<<dim3(grid, (unsigned)split), kRotThreads,
                                   (size_t)tokens * (a.r / 2) * sizeof(float2), st>>>(a, tokens, units);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_type(const RotaryArgs& a, cudaStream_t st) {
    constexpr int VEC = 16 / (int)sizeof(T);
    // kept elements need no copy where both tensors are turned in place
    bool keep = false;
    for (const RotaryTensor& t : a.a) keep |= t.heads > 0 && t.x != t.y;
    keep = keep && a.r < a.d;
    const bool wide = (a.interleaved ? a.r : a.r / 2) % VEC == 0;
    if (a.interleaved) return wide ? launch<T, VEC, true>(a, keep, st) : launch<T, 1, true>(a, keep, st);
    return wide ? launch<T, VEC, false>(a, keep, st) : launch<T, 1, false>(a, keep, st);
}

}  // namespace

cudaError_t launch_rotary(const RotaryArgs& a, cudaStream_t st) {
    if (a.T == 0) return cudaSuccess;
    return a.dtype == GDN_BF16 ? launch_type<__nv_bfloat16>(a, st) : launch_type<float>(a, st);
}

}  // namespace gdn
