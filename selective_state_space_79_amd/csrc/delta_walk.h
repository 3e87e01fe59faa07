// delta_walk.h -- the walks of the gated delta rule over the chunks of a piece, with time and against it.
#ifndef SSM_DELTA_WALK_H
#define SSM_DELTA_WALK_H

#include "delta.h"

namespace {
namespace dl {

using namespace ssm_detail;

constexpr int pass_waves(int KD, int PARTS, int MODE) {   // per SIMD
    return KD == 256 ? (PARTS == 1 ? 2 : 1) : PARTS == 1 && MODE == kDeltaFull ? 3 : 2;
}

// LDS of the walks.  Two sets of tiles, so that the next chunk's rows and A are asked for a chunk
// ahead; queries have one, refilled as soon as they are read.  (float32 rows pass through registers.)
template <int PARTS, int KD, int MODE> struct PassRoom {
    static constexpr int SETS = PARTS == 1 ? 2 : 1, ASETS = MODE == kDeltaFull && PARTS > 1 ? 1 : 2, PB = 2 * 512;
    alignas(16) uint16_t K[SETS * PARTS * kChunk * KD], V[SETS * PARTS * kChunk * kCols], A[ASETS * 3 * PB];
    alignas(16) uint16_t Q[MODE == kDeltaFull ? PARTS * kChunk * KD : 8], P[MODE == kDeltaFull ? 3 * PB : 8];
    Steps<kChunk> steps[2];
};
template <int PARTS, int KD> struct RevRoom {
    static constexpr int SETS = PARTS == 1 ? 2 : 1, PB = 2 * 512;
    alignas(16) uint16_t K[SETS * PARTS * kChunk * KD], Q[SETS * PARTS * kChunk * KD], V[SETS * PARTS * kChunk * kCols], A[2 * 3 * PB], P[3 * PB];
    Steps<kChunk> steps[2];
};

// ---------------------------------------------------------------- the walk
// One workgroup walks one piece of one head's sequence for 64 columns of the state, 16 a wave, in
// chunks of 32 tokens: 64 would halve the splits of the state into parts, but take the LDS of
// four workgroups on a CU and twice the time from chunk to chunk.
//
// 131072 tokens of 16 heads of 128 in 16 pieces: outputs 1090 us, the pieces' own states and
// transitions (twice the columns) 1280.  Bound by issue: matrix products run in 37% and 35% of the
// cycles, other vector instructions in 52% and 58%, both at once in 11% and 13%, one or the other in
// 78% and 80%; of the vector instructions 264 of 408 a chunk split float32 values into parts.  A wave
// alone on its SIMD takes 2.3 us a chunk, two to three 2.0, so a CU gains little from more than one
// workgroup: whole sequences wait for themselves (8 ragged prompts of 1 to 3001 tokens, 287 us).  Not
// kept: products interleaved with the splits by hand (slower), the splits' rests by two-term dot
// products (3 to 6%, and not right in one form), a fourth wave a SIMD for the pieces' states (0%), the
// next chunk's loads one by one between the products (the ragged prompts 297 -> 326 us: 950 of a
// chunk's 7000 cycles go into their issue wherever it is), their windows from increments (1%).
template <int PARTS, int KD, int MODE>
__device__ __forceinline__ void pass_walk(const DeltaPass& p, uint32_t unit, PassRoom<PARTS, KD, MODE>& room) {
    constexpr bool FULL = MODE == kDeltaFull, KEEP = MODE == kDeltaKeep, DMA = PARTS == 1;
    constexpr int C = kChunk, IT = C / 16, KB = KD / 32, NTILE = 3, PB = 2 * 512, WP = 3;   // parts of what is no bf16 input
    constexpr int SETS = DMA ? 2 : 1, ASETS = PassRoom<PARTS, KD, MODE>::ASETS, KE = PARTS * C * KD, VE = PARTS * C * kCols;
    uint16_t *const Ks = room.K, *const Vs = room.V, *const As = room.A, *const Q = room.Q, *const Ps = room.P;
    Steps<C>* const steps = room.steps;
    const int tid = threadIdx.x, lane = tid & 63, g4 = lane >> 4, l16 = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const Where w = find_piece(p, unit, MODE == kDeltaStates ? p.vslices + p.kslices : p.vslices, !KEEP);
    // columns of the transition: the same walk from the unit matrix, without values
    const bool trans = MODE == kDeltaStates && w.slice >= p.vslices;
    // no piece starts from a last one's state, but its transition leads back in the gradients
    if (!w.on || (MODE == kDeltaStates && w.last && !(trans && p.trans_t && !w.first))) return;
    const int width = trans ? p.dk : p.dv, h = w.h;
    const int c_slice = (trans ? w.slice - p.vslices : w.slice) * kCols, c_wave = c_slice + 16 * wave, col = c_wave + l16;
    const bool active = c_wave < width;                      // this wave has columns
    const int64_t lo = w.lo, hi = w.hi, ssz = int64_t(p.dk) * p.dv;

    f32x4 S[2 * KB];
    const float* src = nullptr;
    if constexpr (MODE != kDeltaStates) {
        if (p.pieced && w.sq.end - w.sq.start > p.piece)
            src = p.carry + (w.pi * p.H + h) * ssz;
        else if (p.s_in)
            src = p.s_in + (int64_t(w.slot) * p.H + h) * ssz;
    }
    load_state<KB>(S, src, p.dk, p.dv, c_wave, lane);
    if (trans) {
#pragma unroll
        for (int m = 0; m < 2 * KB; ++m)
#pragma unroll
            for (int r = 0; r < 4; ++r) S[m][r] = 32 * (m >> 1) + 8 * g4 + 4 * (m & 1) + r == col ? 1.0f : 0.0f;
    }
    if constexpr (FULL) {   // the tile above the diagonal that shares a block with one on it stays zero
        for (int i = tid; i < WP * PB / 2; i += kThreads) reinterpret_cast<uint32_t*>(Ps)[i] = 0;
    }

    const int64_t nch = (hi - lo + C - 1) / C;
    const Blocked at(p, w, lo);
    Rows<PARTS, C, KD, kThreads> rk, rq;
    Rows<PARTS, C, kCols, kThreads> rv;
    rk.prepare(p.k, int64_t(h / p.rep) * p.dk, p.sk, p.dk, tid);
    rq.prepare(p.q, int64_t(h / p.rep) * p.dk, p.sq, p.dk, tid);
    rv.prepare(p.v, int64_t(h) * p.dv + c_slice, p.sv, p.dv - c_slice, tid);
    const bool ahead = DMA && p.wide;
    auto load_k = [&](int64_t n) { rk.load(Ks + (SETS == 2 && n & 1 ? KE : 0), wave, lo + n * C, hi); };
    auto load_v = [&](int64_t n) {
        if (!trans) rv.load(Vs + (SETS == 2 && n & 1 ? VE : 0), wave, lo + n * C, hi);
    };
    auto load_q = [&](int64_t n) {
        if constexpr (FULL) rq.load(Q, wave, lo + n * C, hi);
    };
    auto load_a = [&](int64_t n, int lane) { at.load(As + (ASETS == 2 && n & 1 ? WP * PB : 0), &steps[n & 1], p, n, h, wave, lane); };
    if (nch > 0) {
        if (p.wide) {
            load_k(0);
            load_v(0);
            load_q(0);
        }
        load_a(0, lane);
    }
    wait_memory<0>();

    for (int64_t n = 0; n < nch; ++n) {
        const int64_t c0 = lo + n * C;
        const Steps<C>& st = steps[n & 1];
        uint16_t* const K = Ks + (SETS == 2 && n & 1 ? KE : 0);
        uint16_t* const V = Vs + (SETS == 2 && n & 1 ? VE : 0);
        const uint16_t* const A = As + (ASETS == 2 && n & 1 ? WP * PB : 0);
        // the lane as the loop's own value: operand addresses are cheap to form anew
        int lane = __builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0u));
        asm volatile("" : "+v"(lane));
        const int tid = 64 * wave + lane, g4 = lane >> 4, l16 = lane & 15;
        // this chunk's rows and A; what a wave stored since they were asked for may still be under way
        constexpr int OUT = C / 4;
        if (!active || MODE == kDeltaStates)
            wait_memory<0>();
        else if (FULL && DMA && p.pairs)
            wait_memory<OUT / 2>();
        else if (KEEP && at.starts(n - 1))
            wait_memory<2 * KB + OUT>();
        else
            wait_memory<OUT>();
        lds_barrier();
        if (!ahead) {
            if (!DMA && p.wide) {
                rk.store(K, tid);
                if (!trans) rv.store(V, tid);
                if constexpr (FULL) rq.store(Q, tid);
                if (n + 1 < nch) {
                    load_k(n + 1);
                    load_v(n + 1);
                    load_q(n + 1);
                }
            } else {
                rk.copy(K, tid, c0, hi);
                if (!trans) rv.copy(V, tid, c0, hi);
                if constexpr (FULL) rq.copy(Q, tid, c0, hi);
            }
            lds_barrier();
        }
        if (ASETS == 2 && n + 1 < nch) {
            if (ahead) {
                load_k(n + 1);
                load_v(n + 1);
            }
            load_a(n + 1, lane);
        }
        if constexpr (KEEP) {
            if (active && at.starts(n))
                store_state<KB>(S, p.keep + (at.block(n) * p.H + h) * ssz, p.dk, p.dv, c_wave, p.dv % 4 == 0, lane);
        }
        const uint32_t base = row_base<KD>(lane), bpair = pair_base<KD>(lane), b32 = row_base<32>(lane);
        // ---- what the state is read for: K S (paired rows) and Q S
        f32x4 acc[IT], o[IT], pt = {0.0f, 0.0f, 0.0f, 0.0f};
        u32x4 xp[WP], ab[IT][WP];
        // a tile of P on or below the diagonal each but the last wave
        const int pi = wave < 1 ? 0 : 1, pj = wave < 2 ? 0 : 1;
        if (active) {
#pragma unroll
            for (int i = 0; i < IT; ++i) acc[i] = o[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            u32x4 ka[2][IT][PARTS], qa[2][IT][PARTS], px[2][PARTS], py[2][PARTS];   // operands one step ahead
            auto read = [&](int kb) {
#pragma unroll
                for (int x = 0; x < PARTS; ++x) {
#pragma unroll
                    for (int i = 0; i < IT; ++i) {
                        ka[kb & 1][i][x] = pair_op<KD>(K + x * C * KD, 0, i, kb, bpair);
                        if constexpr (FULL) qa[kb & 1][i][x] = row_op<KD>(Q + x * C * KD, 16 * i, kb, base);
                    }
                    if constexpr (FULL) {
                        px[kb & 1][x] = row_op<KD>(K + x * C * KD, 16 * pj, kb, base);
                        py[kb & 1][x] = row_op<KD>(Q + x * C * KD, 16 * pi, kb, base);
                    }
                }
            };
            read(0);
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) {
                if (kb + 1 < KB) read(kb + 1);
                u32x4 sp[WP];
                pair_parts<WP>(S[2 * kb], S[2 * kb + 1], sp);
                mma_tiles<IT, PARTS, WP>(ka[kb & 1], sp, acc);
                if constexpr (FULL) {
                    mma_tiles<IT, PARTS, WP>(qa[kb & 1], sp, o);
                    pt = mma_parts<PARTS, PARTS>(px[kb & 1], py[kb & 1], pt);
                }
                if constexpr (!DMA) __builtin_amdgcn_sched_barrier(0);   // three parts of operands fill the registers
            }
#pragma unroll
            for (int i = 0; i < IT; ++i)
#pragma unroll
                for (int k = 0; k < WP; ++k) ab[i][k] = row_op<32>(A + k * PB + 512 * i, 0, 0, b32);
            // beta X = beta V - beta e^G K S
            f32x4 x[2];
            u32x4 v[PARTS];
            if (!trans) {
                const uint32_t bv = col_base<kCols, 0>(16 * wave, lane);
#pragma unroll
                for (int i = 0; i < PARTS; ++i) v[i] = col_op<kCols>(V + i * C * kCols, 0, 0, 0, bv);
            }
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int t0 = 8 * g4 + 4 * half;
                const f32x4 f = *reinterpret_cast<const f32x4*>(&st.bin[t0]), b = *reinterpret_cast<const f32x4*>(&st.beta[t0]);
#pragma unroll
                for (int r = 0; r < 4; r += 2) {
                    float y = 0.0f, z = 0.0f;
                    if (!trans) unpack<PARTS>(v, 2 * half + r / 2, y, z);
                    x[half][r] = fmaf(-f[r], acc[half][r], b[r] * y);
                    x[half][r + 1] = fmaf(-f[r + 1], acc[half][r + 1], b[r + 1] * z);
                }
            }
            pair_parts<WP>(x[0], x[1], xp);
            if constexpr (FULL) {
#pragma unroll
                for (int i = 0; i < IT; ++i) {
                    const f32x4 e = *reinterpret_cast<const f32x4*>(&st.in[16 * i + 4 * g4]);
#pragma unroll
                    for (int r = 0; r < 4; ++r) o[i][r] *= e[r] * p.scale;
                }
            }
        }
        if constexpr (FULL) {
            if (!active) {      // the others have it from their walk over the state's rows
#pragma unroll
                for (int kb = 0; kb < KB; ++kb) {
                    u32x4 x[PARTS], y[PARTS];
#pragma unroll
                    for (int i = 0; i < PARTS; ++i) {
                        x[i] = row_op<KD>(K + i * C * KD, 16 * pj, kb, base);
                        y[i] = row_op<KD>(Q + i * C * KD, 16 * pi, kb, base);
                    }
                    pt = mma_parts<PARTS, PARTS>(x, y, pt);
                }
            }
            if (wave < NTILE) {
                const int i = 16 * pi + l16, j0 = 16 * pj + 4 * g4;
                const int to = 512 * pi + at_piece<32>(l16, 2 * pj + (g4 >> 1)) + 4 * (g4 & 1);
                const float gi = st.hi[i], ei = st.lo[i];
                const f32x4 gj = *reinterpret_cast<const f32x4*>(&st.hi[j0]), ej = *reinterpret_cast<const f32x4*>(&st.lo[j0]);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float e = __builtin_amdgcn_exp2f((gi - gj[r]) + (ei - ej[r]));
                    pt[r] = j0 + r <= i ? pt[r] * (e * p.scale) : 0.0f;
                }
                uint32_t x[WP], y[WP];
                split<WP>(pt[0], pt[1], x);
                split<WP>(pt[2], pt[3], y);
#pragma unroll
                for (int k = 0; k < WP; ++k) *reinterpret_cast<uint2*>(Ps + k * PB + to) = uint2{x[k], y[k]};
            }
            lds_barrier();      // P is there; q has been read
            if (ahead && n + 1 < nch) load_q(n + 1);
        }
        if (active) {
            // ---- U = A beta X
#pragma unroll
            for (int i = 0; i < IT; ++i) acc[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            mma_tiles<IT, WP, WP>(ab, xp, acc);
            if constexpr (KEEP) {
                const int64_t pitch = int64_t(p.H) * p.dv * 4;
                store_tiles<C, true>(acc, reinterpret_cast<char*>(p.rows) + c0 * pitch + int64_t(h) * p.dv * 4, pitch, hi - c0,
                                     c_wave, p.dv, true, false, lane);
            }
            // ---- the outgoing state
            const uint32_t bk = col_base<KD, 1>(0, lane);
            constexpr int G = FULL || KB < 4 ? 4 : 8;       // tiles of the state at a time
            u32x4 ka[G][PARTS];
            auto read = [&](int m0) {
#pragma unroll
                for (int m = 0; m < G; ++m)
#pragma unroll
                    for (int i = 0; i < PARTS; ++i) ka[m][i] = col_op<KD>(K + i * C * KD, 0, (m0 + m) >> 1, m & 1, bk);
            };
            read(0);
            f32x4 x[2];
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const f32x4 f = *reinterpret_cast<const f32x4*>(&st.out[8 * g4 + 4 * half]);
#pragma unroll
                for (int r = 0; r < 4; ++r) x[half][r] = acc[half][r] * f[r];
            }
            u32x4 up[WP];
            pair_parts<WP>(x[0], x[1], up);
            const float tail = st.tail[0];
#pragma unroll
            for (int m0 = 0; m0 < 2 * KB; m0 += G) {
                if (m0 > 0) read(m0);
#pragma unroll
                for (int m = m0; m < m0 + G; ++m)
#pragma unroll
                    for (int r = 0; r < 4; ++r) S[m][r] *= tail;
                mma_tiles<G, PARTS, WP>(ka, up, &S[m0]);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        if constexpr (FULL) {
            if constexpr (ASETS == 1) {
                lds_barrier();      // A has been read
                if (n + 1 < nch) load_a(n + 1, lane);
            }
            if (active) {
                // ---- the chunk's own share, P U
#pragma unroll
                for (int i = 0; i < IT; ++i)
#pragma unroll
                    for (int k = 0; k < WP; ++k) ab[i][k] = row_op<32>(Ps + k * PB + 512 * i, 0, 0, b32);
                u32x4 up[WP];
                pair_parts<WP>(acc[0], acc[1], up);
                mma_tiles<IT, WP, WP>(ab, up, o);
                constexpr int OE = PARTS == 1 ? 2 : 4;
                const int64_t pitch = p.so * OE;
                store_tiles<C, false>(o, static_cast<char*>(p.out) + c0 * pitch + int64_t(h) * p.dv * OE, pitch, hi - c0, c_wave,
                                      p.dv, PARTS > 1, p.pairs, lane);
            }
        }
    }

    // ---------------------------------------------- the state that leaves
    if (!active) return;
    if constexpr (MODE == kDeltaStates) {
        if (trans) {
            const int64_t to = (w.pi * p.H + h) * int64_t(p.dk) * p.dk;
            store_state<KB>(S, p.trans + to, p.dk, p.dk, c_wave, p.dk % 4 == 0, lane);
            if (p.trans_t) {
#pragma unroll
                for (int m = 0; m < 2 * KB; ++m)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int row = 32 * (m >> 1) + 8 * g4 + 4 * (m & 1) + r;
                        if (row < p.dk && col < p.dk) p.trans_t[to + int64_t(col) * p.dk + row] = S[m][r];
                    }
            }
        } else {
            store_state<KB>(S, p.carry + (w.pi * p.H + h) * ssz, p.dk, p.dv, c_wave, p.dv % 4 == 0, lane);
        }
    } else if (FULL && w.last && p.s_out) {
        store_state<KB>(S, p.s_out + (int64_t(w.slot) * p.H + h) * ssz, p.dk, p.dv, c_wave, false, lane);
    }
}

// ---------------------------------------------------------------- the walk against time
// As pass_walk without outputs, with the gradient of the state in the registers; p.v is
// the gradient of o.
template <int PARTS, int KD, int MODE>
__device__ __forceinline__ void rev_walk(const DeltaPass& p, uint32_t unit, RevRoom<PARTS, KD>& room) {
    constexpr bool KEEP = MODE == kDeltaKeep, DMA = PARTS == 1;
    constexpr int C = kChunk, IT = C / 16, KB = KD / 32, PB = 2 * 512, WP = 3;
    constexpr int SETS = DMA ? 2 : 1, KE = PARTS * C * KD, VE = PARTS * C * kCols;
    uint16_t *const Ks = room.K, *const Qs = room.Q, *const Vs = room.V, *const As = room.A, *const PT = room.P;
    Steps<C>* const steps = room.steps;
    const int tid = threadIdx.x, lane = tid & 63, g4 = lane >> 4, l16 = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const Where w = find_piece(p, unit, p.vslices, false);
    if (!w.on || (MODE == kDeltaStates && w.first)) return;   // no piece starts from a first one's gradient
    const int h = w.h, c_slice = w.slice * kCols, c_wave = c_slice + 16 * wave;
    const bool active = c_wave < p.dv;
    const int64_t lo = w.lo, hi = w.hi, ssz = int64_t(p.dk) * p.dv;

    f32x4 S[2 * KB];
    const float* src = nullptr;
    if constexpr (KEEP) {
        if (p.pieced && w.sq.end - w.sq.start > p.piece)
            src = p.carry + (w.pi * p.H + h) * ssz;
        else if (p.s_in)
            src = p.s_in + (int64_t(w.slot) * p.H + h) * ssz;
    }
    load_state<KB>(S, src, p.dk, p.dv, c_wave, lane);

    const int64_t nch = (hi - lo + C - 1) / C;
    const Blocked at(p, w, lo);
    Rows<PARTS, C, KD, kThreads> rk, rq;
    Rows<PARTS, C, kCols, kThreads> rv;
    rk.prepare(p.k, int64_t(h / p.rep) * p.dk, p.sk, p.dk, tid);
    rq.prepare(p.q, int64_t(h / p.rep) * p.dk, p.sq, p.dk, tid);
    rv.prepare(p.v, int64_t(h) * p.dv + c_slice, p.sv, p.dv - c_slice, tid);
    const bool ahead = DMA && p.wide;
    auto load = [&](int64_t n) {
        const bool odd = SETS == 2 && (n & 1);
        rk.load(Ks + (odd ? KE : 0), wave, lo + n * C, hi);
        rq.load(Qs + (odd ? KE : 0), wave, lo + n * C, hi);
        rv.load(Vs + (odd ? VE : 0), wave, lo + n * C, hi);
    };
    auto load_a = [&](int64_t n, int lane) { at.load(As + (n & 1 ? WP * PB : 0), &steps[n & 1], p, n, h, wave, lane); };
    // a block's last chunk is the first one here
    auto starts = [&](int64_t n) { return !at.two || (n & 1) || n == nch - 1; };
    if (nch > 0) {
        if (p.wide) load(nch - 1);
        load_a(nch - 1, lane);
    }
    wait_memory<0>();

    for (int64_t n = nch - 1; n >= 0; --n) {
        const int64_t c0 = lo + n * C;
        const Steps<C>& st = steps[n & 1];
        const bool odd = SETS == 2 && (n & 1);
        uint16_t* const K = Ks + (odd ? KE : 0);
        uint16_t* const Q = Qs + (odd ? KE : 0);
        uint16_t* const V = Vs + (odd ? VE : 0);
        const uint16_t* const A = As + (n & 1 ? WP * PB : 0);
        int lane = __builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0u));
        asm volatile("" : "+v"(lane));
        const int tid = 64 * wave + lane, g4 = lane >> 4, l16 = lane & 15;
        // what a wave stored since this chunk's rows were asked for may still be under way
        constexpr int OUT = C / 4 + C / 8;   // Z, and the gradient of v in pairs or more
        if (!active || !KEEP)
            wait_memory<0>();
        else if (starts(n + 1))
            wait_memory<2 * KB + OUT>();
        else
            wait_memory<OUT>();
        lds_barrier();
        if (!ahead) {
            if (!DMA && p.wide) {
                rk.store(K, tid);
                rq.store(Q, tid);
                rv.store(V, tid);
                if (n > 0) load(n - 1);
            } else {
                rk.copy(K, tid, c0, hi);
                rq.copy(Q, tid, c0, hi);
                rv.copy(V, tid, c0, hi);
            }
            lds_barrier();
        }
        if (n > 0) {
            if (ahead) load(n - 1);
            load_a(n - 1, lane);
        }
        if constexpr (KEEP) {
            if (active && starts(n))
                store_state<KB>(S, p.keep + (at.block(n) * p.H + h) * ssz, p.dk, p.dv, c_wave, p.dv % 4 == 0, lane);
        }
        put_pt<PARTS, KD>(Q, K, PT, st, p.scale, wave, lane);
        // ---- what reaches U from behind: e^{G_C - G} K dS
        f32x4 acc[IT];
        u32x4 v[PARTS], ab[IT][WP];
        if (active) {
            const uint32_t bpair = pair_base<KD>(lane);
#pragma unroll
            for (int i = 0; i < IT; ++i) acc[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            u32x4 ka[2][IT][PARTS];   // operands one step ahead
            auto read = [&](int kb) {
#pragma unroll
                for (int i = 0; i < IT; ++i)
#pragma unroll
                    for (int x = 0; x < PARTS; ++x) ka[kb & 1][i][x] = pair_op<KD>(K + x * C * KD, 0, i, kb, bpair);
            };
            read(0);
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) {
                if (kb + 1 < KB) read(kb + 1);
                u32x4 sp[WP];
                pair_parts<WP>(S[2 * kb], S[2 * kb + 1], sp);
                mma_tiles<IT, PARTS, WP>(ka[kb & 1], sp, acc);
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int i = 0; i < IT; ++i) {
                const f32x4 e = *reinterpret_cast<const f32x4*>(&st.out[8 * g4 + 4 * i]);
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[i][r] *= e[r];
            }
            const uint32_t bv = col_base<kCols, 0>(16 * wave, lane), bt = tri_t_base(lane);
#pragma unroll
            for (int i = 0; i < PARTS; ++i) v[i] = col_op<kCols>(V + i * C * kCols, 0, 0, 0, bv);
#pragma unroll
            for (int i = 0; i < IT; ++i)
#pragma unroll
                for (int k = 0; k < WP; ++k) ab[i][k] = tri_t_op(A + k * PB, i, bt);
        }
        lds_barrier();      // P^T is there
        if (active) {
            const uint32_t b32 = row_base<32>(lane), bk = col_base<KD, 1>(0, lane);
            {
                u32x4 pt[IT][WP];
#pragma unroll
                for (int i = 0; i < IT; ++i)
#pragma unroll
                    for (int k = 0; k < WP; ++k) pt[i][k] = row_op<32>(PT + k * PB + 512 * i, 0, 0, b32);
                mma_tiles<IT, WP, PARTS>(pt, v, acc);
            }
            u32x4 up[WP];
            pair_parts<WP>(acc[0], acc[1], up);
#pragma unroll
            for (int i = 0; i < IT; ++i) acc[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            mma_tiles<IT, WP, WP>(ab, up, acc);
            // ---- the gradient of the incoming state
            constexpr int G = 4;       // tiles of the state at a time
            u32x4 qa[G][PARTS], ka[G][PARTS];
            auto read = [&](int m0) {
#pragma unroll
                for (int m = 0; m < G; ++m)
#pragma unroll
                    for (int i = 0; i < PARTS; ++i) {
                        qa[m][i] = col_op<KD>(Q + i * C * KD, 0, (m0 + m) >> 1, m & 1, bk);
                        ka[m][i] = col_op<KD>(K + i * C * KD, 0, (m0 + m) >> 1, m & 1, bk);
                    }
            };
            read(0);
            f32x4 x[2], y[2];
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int t0 = 8 * g4 + 4 * half;
                const f32x4 e = *reinterpret_cast<const f32x4*>(&st.in[t0]), b = *reinterpret_cast<const f32x4*>(&st.bin[t0]);
#pragma unroll
                for (int r = 0; r < 4; r += 2) {
                    float a, z;
                    unpack<PARTS>(v, 2 * half + r / 2, a, z);
                    x[half][r] = a * (e[r] * p.scale);
                    x[half][r + 1] = z * (e[r + 1] * p.scale);
                }
#pragma unroll
                for (int r = 0; r < 4; ++r) y[half][r] = -b[r] * acc[half][r];
            }
            u32x4 dp[WP], rp[WP];
            pair_parts<WP>(x[0], x[1], dp);
            pair_parts<WP>(y[0], y[1], rp);
            const float tail = st.tail[0];
#pragma unroll
            for (int m0 = 0; m0 < 2 * KB; m0 += G) {
                if (m0 > 0) read(m0);
#pragma unroll
                for (int m = m0; m < m0 + G; ++m)
#pragma unroll
                    for (int r = 0; r < 4; ++r) S[m][r] *= tail;
                mma_tiles<G, PARTS, WP>(qa, dp, &S[m0]);
                mma_tiles<G, PARTS, WP>(ka, rp, &S[m0]);
                __builtin_amdgcn_sched_barrier(0);
            }
            if constexpr (KEEP) {
                const int64_t pitch = int64_t(p.H) * p.dv * 4;
                store_tiles<C, true>(acc, reinterpret_cast<char*>(p.rows) + c0 * pitch + int64_t(h) * p.dv * 4, pitch, hi - c0,
                                     c_wave, p.dv, true, false, lane);
#pragma unroll
                for (int i = 0; i < IT; ++i) {
                    const f32x4 b = *reinterpret_cast<const f32x4*>(&st.given[8 * g4 + 4 * i]);
#pragma unroll
                    for (int r = 0; r < 4; ++r) acc[i][r] *= b[r];
                }
                constexpr int E = PARTS == 1 ? 2 : 4;
                const int64_t vp = int64_t(p.H) * p.dv * E;
                store_tiles<C, true>(acc, static_cast<char*>(p.dv_out) + c0 * vp + int64_t(h) * p.dv * E, vp, hi - c0, c_wave, p.dv,
                                     PARTS > 1, p.pairs, lane);
            }
        }
    }
    if (!active) return;
    float* dst = nullptr;
    if constexpr (MODE == kDeltaStates) dst = p.carry + (w.pi * p.H + h) * ssz;
    else if (w.first && p.s_out) dst = p.s_out + (int64_t(w.slot) * p.H + h) * ssz;
    if (dst) store_state<KB>(S, dst, p.dk, p.dv, c_wave, false, lane);
}

}  // namespace dl
}  // namespace

#endif
