// linear_attn_tc.cu -- the bf16 passes of the decayed linear attention on tcgen05.
//
// Formulas, roles and the shares of the CTAs: linear_attn.cuh.  A CTA walks the 64-token chunks of its chains (or
// pieces of them) one after the other; all its warps count the chunks on, so that the loads and the front of
// the next chain run beside the back of the last.
// With the state kept transposed (row v, column k), a chunk is four products:
//     SC  = K Q^T              (scores, row j, column i)
//     LOC = V~ K               V~ = V^T diag(weights), an A operand in TMEM
//     Ys  = S^T Q^T            S^T in bf16, an A operand in TMEM
//     Yi  = V^T P              P = SC decayed and masked, bf16, in shared memory
// and y_i = Yi + e^{g (i + 1)} Ys, S <- e^{g n} S + LOC.
//  - The state lives in fp32 registers of the compute warps and is only rounded to bf16 as Ys's
//    operand.  LOC is a fresh fp32 accumulator each chunk: added into the state by the CUDA cores, its
//    sums do not suffer from the tensor cores' truncating accumulation over a long sequence.
//  - The decay weights would cost the products' exactness if they were rounded to bf16 with V.  So a weight
//    is cut into three bf16 pieces w1 + w2 + w3, and v w into three: p1 = bf16(v w1); s = bf16(p2 + e1), where
//    p2 = bf16(v w2) and e1 = v w1 - p1 (exact: the product of two 8-bit significands has 16 bits); and the rest,
//    the exact rounding errors of p2 and of the sum (which is exact as s - p2 - e1 since w1 is taken so far below
//    the weight that |p2| > |e1|) plus v w3, rounded: off by 2^-24 of v w in the root mean square and 2^-21 at most,
//    about as an fp32 product is.  Nine packed bf16 instructions for two values; LOC is three products and
//    s_final has fp32 accuracy.  (Four pieces take five instructions, but the tensor cores, which the kernel keeps
//    busy 70% of its cycles, a sixth longer.)  P is rounded to bf16 once (y is bf16).
//  - A operands in TMEM rather than shared memory: the products are bound by shared-memory bandwidth
//    (an A of 128 x 16 costs as much of it as a B of 128 columns), which V~ and S^T do not touch.
// Warps 0-7 prepare a chunk (V~, transposed on the way from shared memory to TMEM by ldmatrix, and P; two
// warps a TMEM lane quadrant), warps 8-15 finish it (the state, the outputs), so that one chunk's front
// runs beside its predecessor's back; warp 16 loads by TMA through a ring of stages, warps 17 to 19 issue the
// products.  Full chunks' outputs leave by TMA.  Every wait is bounded; one that gives up records
// GDN_ERR_TIMEOUT.
// Measured, d = 128: 148 chains of 64 chunks 124 us, 1.9 us a chunk and SM, 5.0 TB/s of the 6.45 that a copy
// reaches.  No one unit bounds it: leaving out the outputs, V~'s arithmetic, P's decay, two of LOC's three
// products or the trips to HBM shortens it by 11, 9, 5, 9 and 14%.  (The SMs' clock falls from 1.9 to 1.5 GHz
// under a second of it.)  8 sequences of 4096 tokens, 32 heads: 227 us (256 chains on 148 SMs), their gradients
// 700 us in three passes; 32768 tokens in 4 documents, 16 heads, cut: 177 us, of it 60 the first pass, 8 the
// states between and 107 the second.  (Short runs; a second and more of load: 205 us for the last, 830 us the gradients.)
#include <mutex>
#include <type_traits>

#include "linear_attn.cuh"
#include "sm100.cuh"

namespace gdn {

namespace {

using namespace sm100;

constexpr int kTcThreads = 640;  // five warpgroups
// Registers a thread: 96 at launch (640 threads), of which the front, loading and issuing warps
// give some to the back warps, which hold the state.  The shares must not exceed what the block was launched with:
// 128 (2 x 80 + 2 x 136 + 48) <= 640 x 96.  (88, 128 and 48: 32768 tokens in 4 documents take 1% longer.)
constexpr int kLaunchRegs = 96, kFrontRegs = 80, kBackRegs = 136, kIoRegs = 48;
static_assert(128 * (2 * kFrontRegs + 2 * kBackRegs + kIoRegs) <= kTcThreads * kLaunchRegs, "register shares");

template <int D, bool STATE>
struct TcLayout {
    static constexpr int KB = D / 64;             // 64-column panels of a tile
    static constexpr int TILE = KB * 8192;        // 64 tokens x D, 128-byte rows
    static constexpr int NT = STATE ? 2 : 3;      // K, V (, Q)
    static constexpr int STAGES = 3;
    static constexpr int STAGE = NT * TILE;
    static constexpr int P = STAGES * STAGE;      // [j][i] bf16, one for each stage
    static constexpr int Y = P + (STATE ? 0 : STAGES * 8192);  // outputs on their way out: 32 x 32 a back warp
    static constexpr int TAB = Y + (STATE ? 0 : 8 * 2048);     // decay of the scores by 64 + i - j, two copies
    static constexpr int SW = TAB + 1024;         // weights of V~, by pairs of tokens: [32][4] (three pieces)
    static constexpr int FI = SW + 2 * 512;       // factors of Ys: [64]; both for full chunks and for the last one
    static constexpr int DEC = FI + 2 * 256;      // e^{g n} (decay_steps), for the same
    static constexpr int BAR = DEC + 32;
    static constexpr int MISC = BAR + 22 * 8;     // TMEM base, abort flag, zero word
    static constexpr int WALK = MISC + 16;        // every warp's place between its pieces
    static constexpr int PIECES = WALK + 20 * 16;
    static constexpr int DOCS = PIECES + (int)sizeof(LaPiece) * kLaDocs;
    static constexpr int BYTES = DOCS + ((int)sizeof(LaDocs) + 15) / 16 * 16;
    // TMEM columns; the first pass, which has room, keeps two V~ and two LOC and so has one product in
    // progress while the next is prepared and the last is read
    static constexpr int NB = STATE ? 2 : 1;
    static constexpr uint32_t T_SC = 0, T_V = STATE ? 0 : 64, T_LOC = STATE ? 256 : 192, T_YI = 320, T_YS = 384,
                              T_S = 448;
};
// B_*: arrivals of copies and products; C_*: of the compute warps (8 each).  A wait knows a phase by its
// parity, so no barrier may complete a phase before every waiter has seen the one before:
//   LOC(c + 1) follows C_V(c + 1) and C_L(c), and each of those its warps' wait for LOC(c) (with two buffers:
//   the same of the buffer's own turns, each with its own barriers); SC(c + 1) follows C_P(c), behind B_SC(c);
//   Ys and Yi(c + 1) follow C_S(c + 1), behind B_Y(c).  The front may be up to the ring ahead of the warp
//   that issues Yi, so C_P is a barrier a stage, like B_FULL: its next phase needs the stage loaded again,
//   which needs SC and Yi to be done with it.
enum { B_FULL = 0, B_EMPTY = 3, B_SC = 6, B_LOC, B_Y = B_LOC + 2, B_FIN,
       C_FIX = B_FIN + 3, C_V, C_P = C_V + 2, C_L = C_P + 3, C_S = C_L + 2, B_COUNT };

__device__ __forceinline__ uint32_t pack_rn(float a, float b) {
    const __nv_bfloat162 x = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&x);
}
// The weights of V~ in pieces, by pairs of tokens; the factor of Ys in token i.  The first piece is the rounding of
// a value 2.25 / 256 below the weight: 1.25 to 3.25 parts of 256 are left to the second, more than the rounding
// errors of products with the first (1 part) and than the first's own.
__device__ __forceinline__ void front_table(uint32_t* sw, int pair_, float g, int n, float scale, bool rev) {
    float w[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int j = 2 * pair_ + e;
        w[e] = rev || j < n ? expf(g * (float)(rev ? j + 1 : n - 1 - j)) * scale : 0.f;
    }
#pragma unroll
    for (int t = 0; t < 3; ++t) {
        const float below = t == 0 ? 1.f - 2.25f / 256.f : 1.f;
        const uint32_t x = pack_rn(w[0] * below, w[1] * below);
        w[0] -= __uint_as_float(x << 16);
        w[1] -= __uint_as_float(x & 0xffff0000u);
        sw[4 * pair_ + t] = x;
    }
}
__device__ __forceinline__ float back_factor(float g, int i, int n, float scale, bool rev) {
    return !rev || i < n ? expf(g * (float)(rev ? n - 1 - i : i + 1)) * scale : 0.f;
}

// The state's factor e^{g n} of a full chunk.  One float of it would be off the same way every time.  So its two
// neighbouring floats take turns: with rho of a step from the nearest one to the next lost a chunk, the steps taken in
// the chunks that have c and more to go are rint(c rho).  Over any run of chunks the product is off by one step
// (2^-23) at most, however long the run, and a document's factors do not depend on what its CTA walked before.
// (8 sequences of 4096 tokens, 32 heads: 222 us with one float, 224 us so, 226 us with a second packed multiply-add an
// element for e^{g n}'s low part.)
__device__ __forceinline__ float2 decay_steps(float g, int n) {
    const float2 w = la_power2(g, n);
    const int to = w.y < 0.f ? -1 : 1;
    const float step = __int_as_float(__float_as_int(w.x) + to) - w.x;
    return make_float2(w.x, w.y / step * (float)to);
}
__device__ __forceinline__ float decay_of(float2 d, int left) {
    return __int_as_float(__float_as_int(d.x) + __float2int_rn((float)left * d.y) -
                          __float2int_rn((float)(left - 1) * d.y));
}

// MODE: what a pass writes
enum { M_OUT = 0, M_STATE = 1, M_OUT_F32 = 2 };

template <int D, bool REV, int MODE>
__global__ void __launch_bounds__(kTcThreads, 1)
la_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
             const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_y, const LaParams p) {
    constexpr bool STATE = MODE == M_STATE;
    using L = TcLayout<D, STATE>;
    constexpr int KB = L::KB, C = kLaChunk;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::BAR);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + L::MISC);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + L::MISC + 4);
    volatile int* never = reinterpret_cast<volatile int*>(sm + L::MISC + 8);
    LaDocs* docs = reinterpret_cast<LaDocs*>(sm + L::DOCS);
    if (tid == 0) {
        // a stage is free when all issuing warps' products have read it
        for (int b = 0; b < B_COUNT; ++b)
            mbar_init(&bars[b], b >= C_FIX ? 8 : !STATE && b >= B_EMPTY && b < B_SC ? 3 : 1);
        *abort_flag = 0;
        *never = 0;
        fence_mbar_init();
    }
    if (warp == 17) tmem_alloc(tmem_slot, 512);
    if (p.walk != LA_WALK_TURN) la_make_docs(p, docs);
    LaPiece* pieces = reinterpret_cast<LaPiece*>(sm + L::PIECES);
    if (p.walk == LA_WALK_CUT && docs->cut && tid == 0)
        docs->count = la_cut_pieces(p, docs, blockIdx.x, STATE, pieces);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // The next piece of this CTA.  Every warp keeps its place (and its piece's document and head) in shared memory:
    // registers are short, and they are needed once a piece.
    volatile int* my_walk = reinterpret_cast<volatile int*>(sm + L::WALK) + warp * 4;
    const bool cut = p.walk == LA_WALK_CUT && docs->cut;
    my_walk[0] = cut ? 0 : blockIdx.x;
    auto next_piece = [&](LaPiece* pc, uint32_t lanes = 0xffffffffu) {
        const int at = my_walk[0];
        __syncwarp(lanes);
        if (cut) {
            if (at >= docs->count) return false;
            *pc = pieces[at];
            my_walk[0] = at + 1;
        } else {
            // the first pass has nothing to do; sorted, every second round runs the other way
            if (STATE || at >= p.num_seqs * p.H) return false;
            la_chain(p, docs, at, pc);
            my_walk[0] = p.walk == LA_WALK_SORTED ? (2 * (at / gridDim.x) + 2) * gridDim.x - 1 - at
                                                  : at + gridDim.x;
        }
        my_walk[1] = pc->doc;
        my_walk[2] = pc->h;
        my_walk[3] = pc->ends();
        return true;
    };

    auto wait = [&](int bar, uint32_t parity) { return wait_all(&bars[bar], parity, abort_flag, bar); };
    // A piece's chunks are counted down: `left` of them, this one included.  The document's last, the only one
    // that can be short, is the last of a piece that ends, or (reversed) the first of one that starts.
    auto odd = [&](const LaPiece& pc) { return pc.nch > 0 && (REV ? pc.starts() : pc.ends()) ? pc.last : C; };
    auto tokens = [&](const LaPiece& pc, int left, int odd_n) {
        return left == (REV ? pc.w1 - pc.w0 : 1) ? odd_n : C;
    };

    constexpr bool MOVE = D == 128;  // D = 64 needs no more than 96 registers
    if (warp >= 16) {
        if constexpr (MOVE) regs_down<kIoRegs>();
    }
    if (warp == 16) {
        // ---------------------------------------------------------------- loads
        if (lane == 0) {
            int it = 0;  // chunks so far
            bool ok = true;
            LaPiece pc;
            while (ok && next_piece(&pc, 1u)) {
                int z = pc.t0 + (REV ? pc.nch - 1 - pc.w0 : pc.w0) * C;
                for (int left = pc.w1 - pc.w0; left > 0; --left, ++it, z += REV ? -C : C) {
                    const int s = it % L::STAGES;
                    if (it >= L::STAGES && !mbar_wait(&bars[B_EMPTY + s], ((it / L::STAGES) - 1) & 1, abort_flag)) {
                        if (!*abort_flag) *abort_flag = B_EMPTY + s + 1;
                        ok = false;
                        break;
                    }
                    uint64_t* full = &bars[B_FULL + s];
                    mbar_arrive_expect_tx(full, L::STAGE);
                    uint8_t* dst = sm + s * L::STAGE;
#pragma unroll
                    for (int b = 0; b < KB; ++b) {
                        tma_load_3d(dst + b * 8192, &tm_k, 64 * b, pc.h / p.kdiv, z, full);
                        tma_load_3d(dst + L::TILE + b * 8192, &tm_v, 64 * b, pc.h / p.vdiv, z, full);
                        if (!STATE) tma_load_3d(dst + 2 * L::TILE + b * 8192, &tm_q, 64 * b, pc.h / p.qdiv, z, full);
                    }
                }
            }
            // copies still in flight land, and the products that read them end, before the CTA may (bounded)
            for (int k = it > L::STAGES ? it - L::STAGES : 0; k < it; ++k) {
                mbar_wait(&bars[B_FULL + k % L::STAGES], (k / L::STAGES) & 1, never, 100000000ull);
                if (ok) mbar_wait(&bars[B_EMPTY + k % L::STAGES], (k / L::STAGES) & 1, abort_flag, 100000000ull);
            }
        }
        __syncwarp();
    } else if (warp == 17 || (!STATE && warp > 17)) {
        // ---------------------------------------------------------------- products
        // Three warps issue, LOC the first, Ys and Yi the second, SC the third: an issuing warp is held while its
        // products run, and the waits of one chain then run beside the products of the others.  A whole warp walks and
        // one lane issues.  (With a single lane walking, every product's descriptors go through vector
        // registers: 110 cycles a product.)
        const bool leader = elect_one();
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        constexpr uint32_t ID_SC = idesc_bf16(64, 64, false, false);
        constexpr uint32_t ID_YS = idesc_bf16(128, 64, false, false);
        constexpr uint32_t ID_LOC = idesc_bf16(128, D, false, true);
        constexpr uint32_t ID_YI = idesc_bf16(128, 64, true, true);
        // V^T as an MN-major A of 128 rows; for D = 64 rows 64..127 repeat rows 0..63 (LBO 0)
        constexpr uint32_t VLBO = D == 128 ? 8192 : 0;
        const uint32_t s0 = smem_u32(sm);
        bool ok = true;
        // products over the K steps of 16: A and B advance by constants
        auto steps = [&](auto f) {
            f(std::integral_constant<int, 0>());
            f(std::integral_constant<int, 1>());
            f(std::integral_constant<int, 2>());
            f(std::integral_constant<int, 3>());
        };
        int s = 0;             // the chunk's stage
        uint32_t st = s0;      // and its address
        uint32_t full_ph = 0;  // the parity of its arrival
        int last_s = 0;        // the chunk before
        uint32_t last_ph = 0;
        auto next_stage = [&]() {
            last_s = s;
            last_ph = full_ph;
            st += L::STAGE;
            if (++s == L::STAGES) {
                s = 0;
                st = s0;
                full_ph ^= 1;
            }
        };
        int it = 0;
        LaPiece pc;
        if (warp == 17) {
            while (ok && next_piece(&pc))
                for (int left = pc.w1 - pc.w0; left > 0; --left, ++it, next_stage()) {
                    const int b = it % L::NB, use = it / L::NB;
                    // the chunk is in shared memory, V~ is stored (K's zeroed rows before it), the last LOC is read
                    ok = wait(B_FULL + s, full_ph) && wait(C_V + b, use & 1) &&
                         (use == 0 || wait(C_L + b, (use - 1) & 1));
                    if (!ok) break;
                    tc_fence_after();
                    if (leader) {
                        const uint32_t k = desc_lo(st, 8192), d = tm + L::T_LOC + 128 * b, v = tm + L::T_V + 128 * b;
                        steps([&](auto kk) { mma_ts<ID_LOC, kk != 0>(d, v + 8 * kk, k + 128 * kk); });
                        steps([&](auto kk) { mma_ts<ID_LOC, true>(d, v + 32 + 8 * kk, k + 128 * kk); });
                        steps([&](auto kk) { mma_ts<ID_LOC, true>(d, v + 64 + 8 * kk, k + 128 * kk); });
                        mma_commit(&bars[B_LOC + b]);
                        mma_commit(&bars[B_EMPTY + s]);
                    }
                    __syncwarp();
                }
        } else if (warp == 19) {
            uint32_t fix_ph = 0;
            while (ok && next_piece(&pc)) {
                const int odd_n = odd(pc);
                for (int left = pc.w1 - pc.w0; left > 0; --left, ++it, next_stage()) {
                    const bool tail = tokens(pc, left, odd_n) < C;
                    // the chunk is in shared memory; its scores' region is free (the last P is stored)
                    ok = wait(B_FULL + s, full_ph) && (!tail || wait(C_FIX, fix_ph)) &&
                         (it == 0 || wait(C_P + last_s, last_ph));
                    if (!ok) break;
                    if (tail) fix_ph ^= 1;
                    tc_fence_after();
                    if (leader) {
                        const uint32_t k = desc_lo(st, 16), q = k + (2 * L::TILE >> 4);
                        steps([&](auto kk) { mma_ss<ID_SC, kk != 0>(tm + L::T_SC, k + 2 * kk, q + 2 * kk); });
                        if constexpr (KB == 2)
                            steps([&](auto kk) {
                                mma_ss<ID_SC, true>(tm + L::T_SC, k + 512 + 2 * kk, q + 512 + 2 * kk);
                            });
                        mma_commit(&bars[B_SC]);
                        mma_commit(&bars[B_EMPTY + s]);
                    }
                    __syncwarp();
                }
            }
        } else {
            while (ok && next_piece(&pc))
                for (int left = pc.w1 - pc.w0; left > 0; --left, ++it, next_stage()) {
                    // the chunk is in shared memory, the state before it stored, the last outputs read
                    ok = wait(B_FULL + s, full_ph) && wait(C_S, it & 1);
                    if (!ok) break;
                    tc_fence_after();
                    if (leader) {
                        const uint32_t q = desc_lo(st + 2 * L::TILE, 16);
                        steps([&](auto kk) { mma_ts<ID_YS, kk != 0>(tm + L::T_YS, tm + L::T_S + 8 * kk, q + 2 * kk); });
                        if constexpr (KB == 2)
                            steps([&](auto kk) {
                                mma_ts<ID_YS, true>(tm + L::T_YS, tm + L::T_S + 32 + 8 * kk, q + 512 + 2 * kk);
                            });
                    }
                    __syncwarp();
                    ok = wait(C_P + s, full_ph);  // (V's zeroed rows too: the warps that zero them store P afterwards)
                    if (!ok) break;
                    tc_fence_after();
                    if (leader) {
                        const uint32_t v = desc_lo(st + L::TILE, VLBO), pp = desc_lo(s0 + L::P + s * 8192, 8192);
                        steps([&](auto kk) { mma_ss<ID_YI, kk != 0>(tm + L::T_YI, v + 128 * kk, pp + 128 * kk); });
                        mma_commit(&bars[B_Y]);
                        mma_commit(&bars[B_EMPTY + s]);
                    }
                    __syncwarp();
                }
        }
        // no product may still be running when the CTA ends
        if (leader) {
            mma_commit(&bars[B_FIN + warp - 17]);
            mbar_wait(&bars[B_FIN + warp - 17], 0, never, 100000000ull);
        }
        __syncwarp();
    } else if (warp < 8) {
        if constexpr (MOVE) regs_down<kFrontRegs>();
        // ---------------------------------------------------------------- front: V~ and P
        // After a wait that gave up the warps walk on (the waits then return at once), so that all of them
        // still meet at the named barriers.
        const int quad = warp & 3, half = warp >> 2;
        const uint32_t tl = tmem + (static_cast<uint32_t>(quad * 32) << 16);
        uint32_t w1[4], w2[4], w3[4];  // of the tokens 32 half + 8 u + 2 (lane % 4) + 0..1
        auto weights = [&](bool last) {
            const uint32_t* sw = reinterpret_cast<const uint32_t*>(sm + L::SW) + last * 128;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const uint4 x = *reinterpret_cast<const uint4*>(sw + 4 * (16 * half + 4 * u + (lane & 3)));
                w1[u] = x.x; w2[u] = x.y; w3[u] = x.z;
            }
        };
        float* tab = reinterpret_cast<float*>(sm + L::TAB);
        const int j0 = 16 * quad + (lane >> 2), i0 = 32 * half + 2 * (lane & 3);
        const int k0 = 64 + i0 - j0;  // this lane's first entry of the scores' decay
        const float2* t0 = reinterpret_cast<const float2*>(tab + (k0 & 1) * 128 + (k0 & ~1));
        const uint32_t p0 = smem_u32(sm + L::P) + j0 * 128 + 4 * (lane & 3);
        uint32_t v0[2][2];  // ldmatrix rows of V: 16-row block r, tokens 16 x ..
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int m = lane >> 3, j = 32 * half + 16 * x + 8 * (m >> 1) + (lane & 7);
                const int v8 = (4 * quad + 2 * r + (m & 1)) & (D / 8 - 1);
                v0[r][x] = smem_u32(sm + L::TILE + (v8 >> 3) * 8192) + swz(j, v8 & 7);
            }
        int s = 0, it = 0;
        uint32_t full_ph = 0;
        LaPiece pc;
        while (next_piece(&pc)) {
            // the piece's tables, once the last piece's are read
            const float g = p.log_decay[pc.h];
            named_sync(1, 256);
            if (tid < 64) front_table(reinterpret_cast<uint32_t*>(sm + L::SW) + (tid >> 5) * 128, tid & 31, g,
                                      tid < 32 ? C : pc.last, p.state_scale, REV);
            if (!STATE) {  // tab[e] for 64 + i - j = e; the second copy is one entry ahead (pairs then are aligned)
                const int e = (tid & 127) + (tid >> 7), d = REV ? 64 - e : e - 64;
                tab[tid] = d >= 0 && d < 64 ? expf(g * (float)d) * p.p_scale : 0.f;
            }
            named_sync(1, 256);
            weights(false);
            const int odd_n = odd(pc);
            for (int left = pc.w1 - pc.w0; left > 0; --left, ++it) {
                const int n = tokens(pc, left, odd_n);
                const int buf = it % L::NB, use = it / L::NB;
                wait(B_FULL + s, full_ph);
                if (n < C) {
                    // rows past the document's end hold other documents' tokens (or nothing): K and V are zeroed
                    weights(true);
#pragma unroll 1
                    for (int e = tid; e < (C - n) * 8 * 2 * KB; e += 256) {
                        const int r = n + (e >> 3) / (2 * KB), panel = (e >> 3) % (2 * KB);
                        *reinterpret_cast<uint4*>(sm + s * L::STAGE + panel * 8192 + r * 128 + (e & 7) * 16) =
                            make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                    named_sync(1, 256);
                    if (lane == 0) mbar_arrive(&bars[C_FIX]);
                }
                // ---- V~: rows v = 32 quad .. +31 (D = 64: twice), tokens 32 half .. +31, in three pieces
                {
                    uint32_t w[3][16];
                    __syncwarp();
#pragma unroll
                    for (int r = 0; r < 2; ++r)  // 16 rows each
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            uint32_t v[4];
                            ldsm_x4_t(v0[r][x] + s * L::STAGE, v[0], v[1], v[2], v[3]);
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int u = 2 * x + (e >> 1), at = 8 * r + 4 * x + e;
                                const uint32_t p1 = mul_bf16x2(v[e], w1[u]), p2 = mul_bf16x2(v[e], w2[u]);
                                const uint32_t e1 = fma_bf16x2(v[e], w1[u], p1 ^ 0x80008000u);
                                const uint32_t e2 = fma_bf16x2(v[e], w2[u], p2 ^ 0x80008000u);
                                const uint32_t sum = add_bf16x2(p2, e1), es = sub_bf16x2(e1, sub_bf16x2(sum, p2));
                                w[0][at] = p1;
                                w[1][at] = sum;
                                w[2][at] = fma_bf16x2(v[e], w3[u], add_bf16x2(es, e2));
                            }
                        }
                    if (use > 0) wait(B_LOC + buf, (use - 1) & 1);  // the last V~ is read
                    tc_fence_after();
                    tmem_st_frag_x3(tl + L::T_V + 128 * buf + 16 * half, w);
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars[C_V + buf]);
                }
                // ---- P: rows j = 16 quad .. +15, columns i = 32 half .. +31.  Its buffer is the stage's own: with
                // the stage loaded again, the Yi that read the buffer is done.
                if (!STATE) {
                    wait(B_SC, it & 1);
                    tc_fence_after();
                    float x[16];
                    tmem_ld_frag<4>(tl + L::T_SC + 32 * half, x);
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const uint32_t at = p0 + s * 8192 + (((4 * half + u) ^ (j0 & 7)) << 4);
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            const float2 f = t0[4 * u - 4 * r];
                            float y0, y1;
                            unpair(mul2(pair(x[4 * u + 2 * r], x[4 * u + 2 * r + 1]), pair(f.x, f.y)), y0, y1);
                            asm volatile("st.shared.b32 [%0], %1;" ::"r"(at + 1024 * r), "r"(pack_rn(y0, y1))
                                         : "memory");
                        }
                    }
                    tc_fence_before();
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars[C_P + s]);
                }
                if (REV && n < C) weights(false);
                if (++s == L::STAGES) {
                    s = 0;
                    full_ph ^= 1;
                }
            }
        }
    } else if (warp < 16) {
        // ---------------------------------------------------------------- back: the state and the outputs
        if constexpr (MOVE) regs_up<kBackRegs>();
        const int wb = warp - 8, quad = wb & 3, half = wb >> 2;
        const int vv = (quad * 32 + lane) & (D - 1);      // the state's row; D = 64: lanes 64.. repeat it
        const bool mine = quad * 32 < D;                  // this warp writes results
        const uint32_t tl = tmem + (static_cast<uint32_t>(quad * 32) << 16);
        constexpr int NS = D / 2;                         // state columns of this thread: half NS ..
        const size_t DD = (size_t)D * D;
        uint64_t S[NS / 2];
        // element (v, k) in memory
        const int at0 = p.state_t ? vv * D + half * NS : half * NS * D + vv, at1 = p.state_t ? 1 : D;
        // the state in bf16 as the A operand of Ys
        auto store_state = [&]() {
#pragma unroll
            for (int x0 = 0; x0 < NS / 2; x0 += 16) {
                uint32_t w[16];
#pragma unroll
                for (int x = 0; x < 16; ++x) {
                    float a, b;
                    unpair(S[x0 + x], a, b);
                    w[x] = pack_rn(a, b);
                }
                tmem_st16(tl + L::T_S + half * (NS / 2) + x0, w);
            }
            tc_fence_before();
        };
        uint8_t* ybuf = sm + L::Y + wb * 2048;  // this warp's 32 tokens x 32 columns, 64-byte rows, swizzled
        bool ok = true;
        int it = 0;
        LaPiece pc;
        while (next_piece(&pc)) {
            // the state that the piece starts from: the chain's, or what the CTA before leaves behind
            const size_t chain = ((size_t)pc.doc * p.H + pc.h) * DD;
            const float* from = STATE ? nullptr
                                : !pc.starts() ? p.local + (blockIdx.x - 1) * DD
                                : p.s_in ? p.s_in + chain : nullptr;
#pragma unroll
            for (int x = 0; x < NS / 2; ++x)
                S[x] = from ? pair(from[at0 + 2 * x * at1], from[at0 + (2 * x + 1) * at1]) : 0;
            // the piece's tables, once the last piece's are read
            const float g = p.log_decay[pc.h];
            named_sync(2, 256);
            if (tid >= 256 + 192) {
                if (tid < 256 + 194)  // (the last chunk's once a document: the nearest float)
                    reinterpret_cast<float2*>(sm + L::DEC)[tid - 448] =
                        tid == 448 ? decay_steps(g, C) : make_float2(la_power2(g, pc.last).x, 0.f);
            } else if (!STATE && tid < 256 + 128) {
                reinterpret_cast<float*>(sm + L::FI)[tid - 256] =
                    back_factor(g, tid & 63, tid < 256 + 64 ? C : pc.last, p.inter_scale, REV);
            }
            named_sync(2, 256);
            if (!STATE && pc.w1 > pc.w0) {
                store_state();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[C_S]);
            }
            int row = pc.t0 + (REV ? pc.nch - 1 - pc.w0 : pc.w0) * C;
            const int odd_n = odd(pc);
            for (int left = pc.w1 - pc.w0; left > 0; --left, ++it, row += REV ? -C : C) {
                const int n = tokens(pc, left, odd_n);
                const int buf = it % L::NB, use = it / L::NB;
                const bool tail = n < C;
                const float* fi = reinterpret_cast<const float*>(sm + L::FI) + tail * 64;
                const float w = decay_of(reinterpret_cast<const float2*>(sm + L::DEC)[tail], left);
                // ---- state behind the chunk
                ok = wait(B_LOC + buf, use & 1) && ok;
                tc_fence_after();
                {
                    const uint64_t wx = pair(w, w);
#pragma unroll
                    for (int b = 0; b < NS / 2; b += 16) {
                        float x[32];
                        tmem_ld32(tl + L::T_LOC + 128 * buf + half * NS + 2 * b, x);
#pragma unroll
                        for (int e = 0; e < 16; ++e) S[b + e] = fma2(S[b + e], wx, pair(x[2 * e], x[2 * e + 1]));
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[C_L + buf]);
                // ---- outputs: columns v = 32 quad .. +31, tokens 32 half .. +31
                if (!STATE) {
                    ok = wait(B_Y, it & 1) && ok;  // Ys has read the state, too
                    tc_fence_after();
                    if (left > 1) store_state();
                    if (lane == 0) bulk_wait_read();  // the last chunk's outputs have left the staging tile
                    __syncwarp();
                    const size_t step = (size_t)p.H * D;
#pragma unroll
                    for (int r = 0; r < 2; ++r) {   // 16 lanes each
                        float y[16], z[16];
                        const uint32_t at = tl + (16u * r << 16) + 32 * half;
                        tmem_ld_frag4x2(at + L::T_YI, at + L::T_YS, y, z);
                        if (r == 1) {  // the state is stored and the outputs are read
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0 && left > 1) mbar_arrive(&bars[C_S]);
                        }
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            const float2 f = *reinterpret_cast<const float2*>(fi + 32 * half + 8 * u + 2 * (lane & 3));
                            const uint64_t f2 = pair(f.x, f.y);
#pragma unroll
                            for (int e = 4 * u; e < 4 * u + 4; e += 2)
                                unpair(fma2(f2, pair(z[e], z[e + 1]), pair(y[e], y[e + 1])), y[e], y[e + 1]);
                        }
                        if (!mine) continue;
                        if constexpr (MODE == M_OUT_F32) {
                            float* o = static_cast<float*>(p.out) + (size_t)row * step + my_walk[2] * D;
                            if (ok)
#pragma unroll
                                for (int e = 0; e < 16; ++e) {
                                    const int i = 32 * half + 8 * (e >> 2) + 2 * (lane & 3) + (e & 1);
                                    const int v = 32 * quad + 16 * r + 8 * ((e >> 1) & 1) + (lane >> 2);
                                    if (i < n) o[(size_t)i * step + v] = y[e];
                                }
                        } else {
                            __syncwarp();
                            // transposed into the staging tile, 8 x 8 blocks of (token, v)
#pragma unroll
                            for (int u = 0; u < 4; u += 2) {
                                const int m = lane >> 3;
                                const int i = 8 * (u + (m >> 1)) + (lane & 7), v8 = 2 * r + (m & 1);
                                stsm_x4_t(smem_u32(ybuf) + i * 64 + ((v8 ^ ((i >> 1) & 3)) << 4),
                                          pack_rn(y[4 * u], y[4 * u + 1]), pack_rn(y[4 * u + 2], y[4 * u + 3]),
                                          pack_rn(y[4 * u + 4], y[4 * u + 5]), pack_rn(y[4 * u + 6], y[4 * u + 7]));
                            }
                        }
                    }
                    if (MODE == M_OUT && mine) {
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (32 * half + 32 <= n) {
                            if (lane == 0 && ok) {
                                tma_store_3d(&tm_y, ybuf, 32 * quad, my_walk[2], row + 32 * half);
                                bulk_commit();
                            }
                        } else if (ok) {  // the document's last rows
                            __nv_bfloat16* o =
                                static_cast<__nv_bfloat16*>(p.out) + (size_t)row * step + my_walk[2] * D + 32 * quad;
#pragma unroll 1
                            for (int e = lane; e < (n - 32 * half) * 4; e += 32) {
                                const int i = e >> 2, v8 = e & 3;
                                *reinterpret_cast<uint4*>(o + (size_t)(32 * half + i) * step + 8 * v8) =
                                    *reinterpret_cast<const uint4*>(ybuf + i * 64 + ((v8 ^ ((i >> 1) & 3)) << 4));
                            }
                            __syncwarp();
                        }
                    }
                }
            }
            // ---- what is behind the piece
            float* dst = nullptr;
            if (STATE)
                dst = p.local + blockIdx.x * DD;
            else if (p.s_out && my_walk[3])
                dst = p.s_out + ((size_t)my_walk[1] * p.H + my_walk[2]) * DD;
            if (ok && dst && mine)
#pragma unroll
                for (int x = 0; x < NS / 2; ++x) {
                    float a, b;
                    unpair(S[x], a, b);
                    dst[at0 + 2 * x * at1] = a;
                    dst[at0 + (2 * x + 1) * at1] = b;
                }
        }
        if (!STATE && lane == 0) bulk_wait_read();
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 17) tmem_dealloc(tmem, 512);
    if (tid == 0 && *abort_flag) {
        (void)GDN_GUARD(false, p.status, DBG_WAIT, (long)(*abort_flag - 1) * 65536 + D + MODE * 2 + REV);
        record_status(p.status, GDN_ERR_TIMEOUT);
    }
}

// ============================================================================ between the passes
// Slot i holds the local state of the piece that share i leaves unfinished; it becomes the state at that piece's
// end.  One block per 1024 elements of a chain, which walks the chain's slots, eight loads ahead.
__global__ void __launch_bounds__(256)
la_scan_kernel(const LaParams p, int DD) {
    __shared__ LaDocs docs;
    la_make_docs(p, &docs);
    if (!docs.cut) return;
    const int doc = blockIdx.y / p.H, h = blockIdx.y - doc * p.H;
    const int all = p.H * docs.units[p.num_seqs], shares = la_shares(all, kLaCtas);
    const int nch = docs.units[doc + 1] - docs.units[doc] - kLaStart;
    const int first = p.H * docs.units[doc] + h * (nch + kLaStart) + kLaStart;  // where the chain's chunks begin
    int i0 = (int)((long long)first * shares / all);  // the share that holds the first chunk
    if (la_share(all, i0 + 1, shares) <= first) ++i0;
    if (la_share(all, i0 + 1, shares) >= first + nch) return;  // the chain is not cut
    const int len = docs.len[doc];
    const int e = (blockIdx.x * 256 + threadIdx.x) * 4;
    const float g = p.log_decay[h];
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (p.s_in) x = load4(p.s_in + (size_t)blockIdx.y * DD + e);
    // full pieces between have one of two lengths: their powers are kept
    int known = -1;
    float2 w = make_float2(0.f, 0.f);
    int w0 = 0;
    for (int i = i0;;) {
        float4 loc[8];
        int end[8], m = 0;
        for (; m < 8 && i + m < shares; ++m) {  // (a chain's last share leaves no slot)
            end[m] = la_share(all, i + m + 1, shares) - first;
            if (end[m] >= nch) break;
            loc[m] = load4(p.local + (size_t)(i + m) * DD + e);
        }
#pragma unroll
        for (int b = 0; b < 8; ++b) {
            if (b >= m) break;
            int n = (end[b] - w0) * kLaChunk;
            if (p.reverse && w0 == 0) n += len - nch * kLaChunk;  // the document's last chunk comes first
            if (n != known) {
                known = n;
                w = la_power2(g, n);
            }
            x.x = fmaf(x.x, w.x, fmaf(x.x, w.y, loc[b].x));
            x.y = fmaf(x.y, w.x, fmaf(x.y, w.y, loc[b].y));
            x.z = fmaf(x.z, w.x, fmaf(x.z, w.y, loc[b].z));
            x.w = fmaf(x.w, w.x, fmaf(x.w, w.y, loc[b].w));
            store4(p.local + (size_t)(i + b) * DD + e, x);
            w0 = end[b];
        }
        if (m < 8) break;
        i += 8;
    }
}

// ============================================================================ host side
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        cudaDriverEntryPointQueryResult q;
        void* f = nullptr;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(f);
    });
    return fn;
}

// [tokens, heads, d] bf16, boxes of `side` tokens x 1 head x `side` columns (64: tiles, 32: a back warp's
// outputs); tokens past the end read as zero
bool make_map(CUtensorMap* m, const void* base, long long tokens, int heads, int d, unsigned side = 64) {
    EncodeTiledFn enc = encode_fn();
    if (!enc) return false;
    cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)tokens};
    cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)heads * d * 2};
    cuuint32_t box[3] = {side, 1, side}, es[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE,
               side == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool REV, int MODE>
cudaError_t launch(const LaParams& p, cudaStream_t st) {
    const long long tokens = p.cu ? p.T : (long long)p.num_seqs * p.T;
    CUtensorMap mq, mk, mv, my;
    if (!make_map(&mk, p.k, tokens, p.H / p.kdiv, D) || !make_map(&mv, p.v, tokens, p.H / p.vdiv, D) ||
        !make_map(&mq, p.q, tokens, p.H / p.qdiv, D))
        return cudaErrorInvalidValue;
    my = mq;
    if (MODE == M_OUT && !make_map(&my, p.out, tokens, p.H, D, 32)) return cudaErrorInvalidValue;
    constexpr int bytes = TcLayout<D, MODE == M_STATE>::BYTES + 1024;
    const cudaError_t e = cudaFuncSetAttribute(la_tc_kernel<D, REV, MODE>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    if (D == 128) {  // the register shares rest on what the kernel is launched with
        cudaFuncAttributes at;
        const cudaError_t f = cudaFuncGetAttributes(&at, la_tc_kernel<D, REV, MODE>);
        if (f != cudaSuccess) return f;
        if (at.numRegs < kLaunchRegs) return cudaErrorInvalidConfiguration;
    }
    const long long chains = (long long)p.num_seqs * p.H;
    // chains of unlike lengths that are not sorted are left to the hardware's turns
    const bool each = p.walk == LA_WALK_TURN && p.cu;
    const unsigned ctas = p.walk == LA_WALK_CUT || (!each && chains > kLaCtas) ? kLaCtas : (unsigned)chains;
    la_tc_kernel<D, REV, MODE><<<ctas, kTcThreads, bytes, st>>>(mq, mk, mv, my, p);
    return cudaGetLastError();
}

template <int D>
cudaError_t launch_d(const LaParams& p, cudaStream_t st) {
    if (p.state_only) return p.reverse ? launch<D, true, M_STATE>(p, st) : launch<D, false, M_STATE>(p, st);
    if (!p.reverse) return launch<D, false, M_OUT>(p, st);  // (dq has a head for each state: never in parts)
    return p.out_f32 ? launch<D, true, M_OUT_F32>(p, st) : launch<D, true, M_OUT>(p, st);
}

}  // namespace

cudaError_t launch_la_tc(const LaParams& p, int d, cudaStream_t st) {
    return d == 128 ? launch_d<128>(p, st) : launch_d<64>(p, st);
}

cudaError_t launch_la_scan(const LaParams& p, int d, cudaStream_t st) {
    la_scan_kernel<<<dim3((unsigned)(d * d / 1024), (unsigned)(p.num_seqs * p.H)), 256, 0, st>>>(p, d * d);
    return cudaGetLastError();
}

}  // namespace gdn
