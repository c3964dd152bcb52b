// rotary.cu -- rotary positions of q and k.
//
// The first r of a head's d values form r / 2 pairs (a, b): elements (i, i + r/2) in the half layout,
// (2 i, 2 i + 1) in the interleaved one.  At position p, pair i turns by the angle p f_i:
//     (a, b) -> scale (a cos - b sin, b cos + a sin),
// and by -p f_i in the inverse form, which is also the gradient.  The other d - r values are kept.
//
// Angles: f_i / (2 pi) is taken to 64 bits after the point of a turn, so that p f_i / (2 pi) modulo one
// turn is the low word of an integer product: no error grows with the position beyond the 2^-53 of the
// frequency itself, and up to r = 128 no 64-bit float is touched per token (a lane keeps two frequencies; those
// of wider heads are converted at every token).
//
// A warp serves a token at a time.  Its lanes compute the r / 2 (cos, sin) into shared memory (each lane
// keeps its frequencies), then turn all heads of q and k with them, 16 bytes of both halves of the pairs a
// lane.  The trigonometry is shared by the heads, warps wait for no other warp, and the pass is bound by
// HBM (x read once, y written once).
#include "common.cuh"
#include "internal.h"
#include "sm100.cuh"

namespace gdn {

namespace {

using sm100::fma2;
using sm100::mul2;
using sm100::pair;
using sm100::unpair;

constexpr int kRotWarps = 4;    // of a block
constexpr int kRotBlocks = 10;  // on an SM at once
constexpr int kRotFreqs = 2;    // frequencies a lane keeps in registers

template <typename T, int VEC>
__device__ __forceinline__ void rot_load(const T* p, float* x) {
    if constexpr (VEC == 1) {
        x[0] = to_f32(*p);
    } else {
        const uint4 u = __ldcs(reinterpret_cast<const uint4*>(p));
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (VEC == 8) {
                x[2 * i] = __uint_as_float(w[i] << 16);
                x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            } else {
                x[i] = __uint_as_float(w[i]);
            }
        }
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

// f / (2 pi) in units of 2^-64 turns (whole turns drop out)
__device__ __forceinline__ uint64_t turns_of(float f) {
    const double t = (double)f * 0.15915494309189535;
    return (uint64_t)((t - floor(t)) * 18446744073709551616.0);  // below 2^64: t - floor(t) is at most 1 - 2^-53
}

// VEC elements a lane and access: 16 bytes where every piece of the layout is a multiple of them, else single
// elements.  A unit is what a lane turns in a head: VEC elements of both halves of the pairs (half
// layout), VEC / 2 whole pairs (interleaved, VEC > 1), one pair (VEC = 1), or VEC kept elements.
template <typename T, int VEC, bool INTER>
__global__ void __launch_bounds__(kRotWarps * 32, kRotBlocks)
rotary_kernel(const RotaryArgs p, int units, int turned, int per_block) {
    constexpr bool PAIRS = INTER && VEC > 1;
    extern __shared__ float4 s_cs[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, half = p.r / 2;
    const int pad = (half + 3) & ~3;
    float* cw = reinterpret_cast<float*>(s_cs) + warp * 2 * pad;  // cos; sin behind it
    float* sw = cw + pad;
    uint64_t f[kRotFreqs];
#pragma unroll
    for (int i = 0; i < kRotFreqs; ++i) f[i] = lane + 32 * i < half ? turns_of(p.inv_freq[lane + 32 * i]) : 0;
    const int hpw = units < 32 ? 32 / units : 1;  // heads the lanes cover at once
    const int hh = units < 32 ? lane / units : 0, u0 = units < 32 ? lane - hh * units : lane;
    const int first = blockIdx.y * per_block, last = min(first + per_block, p.a[0].heads + p.a[1].heads);
    // (counted down: a step past the last token may not fit 31 bits)
    for (int left = p.T - (int)(blockIdx.x * kRotWarps + warp); left > 0; left -= gridDim.x * kRotWarps) {
        const int t = p.T - left;
        const long long pos = p.positions[t];
        __syncwarp();  // the last token's factors are read
        for (int i = lane, k = 0; i < half; i += 32, ++k) {
            const uint64_t fr = k < kRotFreqs ? (k == 0 ? f[0] : f[kRotFreqs - 1]) : turns_of(p.inv_freq[i]);
            const int turn = (int)(uint32_t)(((uint64_t)pos * fr + 0x80000000ull) >> 32);  // in 2^-32 turns
            float s, c;
            sincospif((float)turn * (1.f / 2147483648.f), &s, &c);
            cw[i] = c * p.scale;
            sw[i] = (p.inverse ? -s : s) * p.scale;
        }
        __syncwarp();
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            const RotaryTensor& a = p.a[w];
            const int off = w ? p.a[0].heads : 0;
            const int h1 = min(last - off, a.heads);
            if (hh >= hpw) continue;
            const T* xt = static_cast<const T*>(a.x) + (long long)t * a.ldx;
            T* yt = static_cast<T*>(a.y) + (long long)t * a.ldy;
#pragma unroll 2
            for (int h = max(first - off, 0) + hh; h < h1; h += hpw) {
                const T* x = xt + h * p.d;
                T* y = yt + h * p.d;
                for (int u = u0; u < units; u += 32) {
                    if (u >= turned) {
                        const int at = p.r + (u - turned) * VEC;
                        float v[VEC];
                        rot_load<T, VEC>(x + at, v);
                        rot_store<T, VEC>(y + at, v);
                    } else if constexpr (PAIRS) {
                        float v[VEC];
                        rot_load<T, VEC>(x + u * VEC, v);
#pragma unroll
                        for (int i = 0; i < VEC / 2; ++i) {
                            const float c = cw[u * (VEC / 2) + i], s = sw[u * (VEC / 2) + i];
                            const uint64_t o = fma2(pair(v[2 * i + 1], v[2 * i]), pair(-s, s),
                                                    mul2(pair(v[2 * i], v[2 * i + 1]), pair(c, c)));
                            unpair(o, v[2 * i], v[2 * i + 1]);
                        }
                        rot_store<T, VEC>(y + u * VEC, v);
                    } else if constexpr (VEC > 1) {
                        float v[VEC], z[VEC];
                        rot_load<T, VEC>(x + u * VEC, v);
                        rot_load<T, VEC>(x + half + u * VEC, z);
#pragma unroll
                        for (int i = 0; i < VEC; i += 4) {
                            const float4 c = load4(cw + u * VEC + i), s = load4(sw + u * VEC + i);
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const uint64_t c2 = e ? pair(c.z, c.w) : pair(c.x, c.y);
                                const uint64_t s2 = e ? pair(s.z, s.w) : pair(s.x, s.y);
                                const uint64_t m2 = e ? pair(-s.z, -s.w) : pair(-s.x, -s.y);
                                const uint64_t a2 = pair(v[i + 2 * e], v[i + 2 * e + 1]);
                                const uint64_t b2 = pair(z[i + 2 * e], z[i + 2 * e + 1]);
                                unpair(fma2(b2, m2, mul2(a2, c2)), v[i + 2 * e], v[i + 2 * e + 1]);
                                unpair(fma2(a2, s2, mul2(b2, c2)), z[i + 2 * e], z[i + 2 * e + 1]);
                            }
                        }
                        rot_store<T, VEC>(y + u * VEC, v);
                        rot_store<T, VEC>(y + half + u * VEC, z);
                    } else {
                        const int ia = INTER ? 2 * u : u, ib = INTER ? 2 * u + 1 : half + u;
                        const float v = to_f32(x[ia]), z = to_f32(x[ib]), c = cw[u], s = sw[u];
                        y[ia] = from_f32<T>(v * c - z * s);
                        y[ib] = from_f32<T>(z * c + v * s);
                    }
                }
            }
        }
    }
}

template <typename T, int VEC, bool INTER>
cudaError_t launch(const RotaryArgs& a, bool keep, cudaStream_t st) {
    const int turned = INTER && VEC > 1 ? a.r / VEC : a.r / 2 / VEC;
    const int units = turned + (keep ? (a.d - a.r) / VEC : 0);
    const int heads = a.a[0].heads + a.a[1].heads;
    // three times the blocks that fit the SMs at once walk over the tokens (32768 tokens of 18 heads of 128: 54 to 55 us;
    // once 2% more, six times as much, a warp a token 4%); few tokens: the heads go over several blocks, each of
    // which computes the angles again
    const int blocks = a.T / kRotWarps + (a.T % kRotWarps != 0), fit = 148 * kRotBlocks;
    const int hpw = units < 32 ? 32 / units : 1;
    int split = fit / blocks;
    const int most = (heads + hpw - 1) / hpw;
    split = split < 1 ? 1 : split > most ? most : split;
    const int per = (heads + split - 1) / split;
    const size_t smem = (size_t)kRotWarps * 2 * ((a.r / 2 + 3) & ~3) * sizeof(float);
    const dim3 grid((unsigned)(blocks < 3 * fit ? blocks : 3 * fit), (unsigned)((heads + per - 1) / per));
    rotary_kernel<T, VEC, INTER><<<grid, kRotWarps * 32, smem, st>>>(a, units, turned, per);
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
