// delta_bwd.hip -- gradients of the gated delta rule.
//
// With dS_out the gradient of the state behind a chunk (and the names of delta.h),
//
//   dU = P^T dO + (e^{G_C-G} K) dS_out       Z = A^T dU       dR = beta Z = dV
//   dS_in = e^{G_C} dS_out + scale (e^G Q)^T dO - (e^G K)^T dR
//   dQ = scale e^G dO S_in^T + D K           D_ij = scale e^{G_i-G_j} dO_i . U_j, j <= i
//   dK = e^{G_C-G} U dS_out^T - e^G dR S_in^T + D^T Q + (N + N^T) K
//                                            N_ij = -beta_i e^{G_i-G_j} Z_i . U_j, j < i
//   dbeta_i = Z_i . r_i = Z_i . X_i - sum_{j<i} (Z_i . U_j) M_ij
//
// (r = U / beta, but beta may be zero.)  The decay of token t scales all that the state holds
// then, so dg_t = <dS'_t, S'_t>; between tokens it changes by what is read and what is written:
//
//   dg_t = dg_{t+1} + o_t . do_t - v_t . dv_t        behind a chunk <dS_out, S_out>
//
// and o_t . do_t = q_t . dq_t.  Two walks over the chunks, the forward's and one against time,
// leave S_in and dS_out of every chunk in memory; all gradients of a chunk are then formed by a
// workgroup of its own.
#include "delta.h"

namespace {
namespace dl {

using namespace ssm_detail;

// ---------------------------------------------------------------- the walk against time
// As delta_pass_kernel, with the gradient of the state in the registers; p.v is the gradient of o.
template <int PARTS, int KD, int C, int MODE>
__global__ void __launch_bounds__(kThreads, KD == 256 ? 1 : 2) delta_rev_kernel(DeltaPass p) {
    constexpr bool DMA = PARTS == 1;
    constexpr int IT = C / 16, JB = C / 32, KB = KD / 32, NB = tri_blocks<C>(), PB = NB * 512, WP = 3;
    __shared__ __align__(16) uint16_t K[PARTS * C * KD], Q[PARTS * C * KD], V[PARTS * C * kCols], A[WP * PB], PT[WP * PB];
    __shared__ Steps<C> steps[2];
    const int tid = threadIdx.x, lane = tid & 63, g4 = lane >> 4, l16 = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const Where w = find_piece(p, p.vslices, false);
    if (!w.on || (MODE == kDeltaStates && w.first)) return;   // no piece starts from a first one's gradient
    const int h = w.h, c_slice = w.slice * kCols, c_wave = c_slice + 16 * wave, col = c_wave + l16;
    const bool active = c_wave < p.dv;
    const int64_t lo = w.lo, hi = w.hi, ssz = int64_t(p.dk) * p.dv;

    f32x4 S[2 * KB];
    const float* src = nullptr;
    if constexpr (MODE != kDeltaStates) {
        if (p.pieced && w.sq.end - w.sq.start > p.piece)
            src = p.carry + (w.pi * p.H + h) * ssz;
        else if (p.s_in)
            src = p.s_in + (int64_t(w.slot) * p.H + h) * ssz;
    }
#pragma unroll
    for (int m = 0; m < 2 * KB; ++m)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int row = 32 * (m >> 1) + 8 * g4 + 4 * (m & 1) + r;
            S[m][r] = src && row < p.dk && col < p.dv ? src[int64_t(row) * p.dv + col] : 0.0f;
        }

    const int64_t nch = (hi - lo + C - 1) / C;
    const Chunks ch(p, C);
    const int64_t first = uniform(piece_base(ch, w.seq)) + (lo - w.sq.start) / C;
    const uint16_t* const tri = p.tri + (first * p.H + h) * tri_elems<C>();
    auto load_a = [&](int64_t n, int lane) { load_tri<C, 4>(tri + n * p.H * tri_elems<C>(), A, wave, lane); };
    const bool step_wave = wave == 3;
    float gn = 0.0f, bn = 0.0f;
    auto fetch = [&](int64_t n, int lane) {
        const int64_t t = lo + n * C + lane;
        const bool on = n >= 0 && lane < C && t < hi;
        gn = on ? p.g[t * p.sg + h] : 0.0f;
        bn = on ? p.beta[t * p.H + h] : 0.0f;
    };
    if (step_wave) {
        fetch(nch - 1, lane);
        put_steps<C>(steps[(nch - 1) & 1], gn, bn, lane);
        fetch(nch - 2, lane);
    }
    Rows<PARTS, C, KD, kThreads> rk, rq;
    Rows<PARTS, C, kCols, kThreads> rv;
    rk.prepare(p.k, int64_t(h / p.rep) * p.dk, p.sk, p.dk, tid);
    rq.prepare(p.q, int64_t(h / p.rep) * p.dk, p.sq, p.dk, tid);
    rv.prepare(p.v, int64_t(h) * p.dv + c_slice, p.sv, p.dv - c_slice, tid);
    const bool ahead = DMA && p.wide;
    if (nch > 0) {
        const int64_t c0 = lo + (nch - 1) * C;
        if (p.wide) {
            rk.load(K, wave, c0, hi);
            rq.load(Q, wave, c0, hi);
            rv.load(V, wave, c0, hi);
        }
        load_a(nch - 1, lane);
    }
    wait_memory<0>();

    for (int64_t n = nch - 1; n >= 0; --n) {
        const int64_t c0 = lo + n * C;
        const Steps<C>& st = steps[n & 1];
        int lane = __builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0u));
        asm volatile("" : "+v"(lane));
        const int tid = 64 * wave + lane, g4 = lane >> 4, l16 = lane & 15;
        wait_memory<0>();
        lds_barrier();
        if (!ahead) {
            if (!DMA && p.wide) {
                rk.store(K, tid);
                rq.store(Q, tid);
                rv.store(V, tid);
                if (n > 0) {
                    rk.load(K, wave, c0 - C, hi);
                    rq.load(Q, wave, c0 - C, hi);
                    rv.load(V, wave, c0 - C, hi);
                }
            } else {
                rk.copy(K, tid, c0, hi);
                rq.copy(Q, tid, c0, hi);
                rv.copy(V, tid, c0, hi);
            }
            lds_barrier();
        }
        if (MODE == kDeltaKeep && active) {
            float* const at = p.keep + ((first + n) * p.H + h) * ssz;
#pragma unroll
            for (int m = 0; m < 2 * KB; ++m)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int row = 32 * (m >> 1) + 8 * g4 + 4 * (m & 1) + r;
                    if (row < p.dk && col < p.dv) at[int64_t(row) * p.dv + col] = S[m][r];
                }
        }
        put_pt<PARTS, KD, C, 4>(Q, K, PT, st, p.scale, wave, lane);
        if (step_wave && n > 0) {
            put_steps<C>(steps[(n - 1) & 1], gn, bn, lane);
            fetch(n - 2, lane);
        }
        // ---- what reaches U from behind: e^{G_C - G} K dS
        f32x4 acc[IT];
        u32x4 v[JB][PARTS];
        if (active) {
            const uint32_t bpair = pair_base<KD>(lane);
#pragma unroll
            for (int i = 0; i < IT; ++i) acc[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) {
                u32x4 sp[WP];
                pair_parts<WP>(S[2 * kb], S[2 * kb + 1], sp);
#pragma unroll
                for (int i = 0; i < IT; ++i) {
                    u32x4 a[PARTS];
#pragma unroll
                    for (int x = 0; x < PARTS; ++x) a[x] = pair_op<KD>(K + x * C * KD, 32 * (i >> 1), i & 1, kb, bpair);
                    acc[i] = mma_parts<PARTS, WP>(a, sp, acc[i]);
                }
            }
#pragma unroll
            for (int i = 0; i < IT; ++i) {
                const f32x4 e = *reinterpret_cast<const f32x4*>(&st.out[32 * (i >> 1) + 8 * g4 + 4 * (i & 1)]);
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[i][r] *= e[r];
            }
            const uint32_t bv = col_base<kCols, 0>(16 * wave, lane);
#pragma unroll
            for (int jb = 0; jb < JB; ++jb)
#pragma unroll
                for (int i = 0; i < PARTS; ++i) v[jb][i] = col_op<kCols>(V + i * C * kCols, 32 * jb, 0, 0, bv);
        }
        lds_barrier();      // P^T is there; the gradient of o has been read
        if (ahead && n > 0) rv.load(V, wave, c0 - C, hi);
        if (active) {
            const uint32_t b32 = row_base<32>(lane), bt = tri_t_base(lane), bk = col_base<KD, 1>(0, lane);
#pragma unroll
            for (int i = 0; i < IT; ++i)
#pragma unroll
                for (int ip = i / 2; ip < JB; ++ip) {
                    u32x4 a[WP];
#pragma unroll
                    for (int k = 0; k < WP; ++k) a[k] = row_op<32>(PT + k * PB + pt_block<C>(i, ip) * 512, 0, 0, b32);
                    acc[i] = mma_parts<WP, PARTS>(a, v[ip], acc[i]);
                }
            u32x4 up[JB][WP];
#pragma unroll
            for (int ip = 0; ip < JB; ++ip) pair_parts<WP>(acc[2 * ip], acc[2 * ip + 1], up[ip]);
#pragma unroll
            for (int i = 0; i < IT; ++i) {
                acc[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int ip = i / 2; ip < JB; ++ip) {
                    u32x4 a[WP];
#pragma unroll
                    for (int k = 0; k < WP; ++k) a[k] = tri_t_op(A + k * PB, ip, i >> 1, i & 1, bt);
                    acc[i] = mma_parts<WP, WP>(a, up[ip], acc[i]);
                }
            }
            // ---- the gradient of the incoming state
            const float tail = st.tail;
#pragma unroll
            for (int m = 0; m < 2 * KB; ++m)
#pragma unroll
                for (int r = 0; r < 4; ++r) S[m][r] *= tail;
#pragma unroll
            for (int jb = 0; jb < JB; ++jb) {
                f32x4 x[2], y[2];
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const int t0 = 32 * jb + 8 * g4 + 4 * half;
                    const f32x4 e = *reinterpret_cast<const f32x4*>(&st.in[t0]), b = *reinterpret_cast<const f32x4*>(&st.bin[t0]);
#pragma unroll
                    for (int r = 0; r < 4; r += 2) {
                        float u, z;
                        unpack<PARTS>(v[jb], 2 * half + r / 2, u, z);
                        x[half][r] = u * (e[r] * p.scale);
                        x[half][r + 1] = z * (e[r + 1] * p.scale);
                    }
#pragma unroll
                    for (int r = 0; r < 4; ++r) y[half][r] = -b[r] * acc[2 * jb + half][r];
                }
                u32x4 dp[WP], rp[WP];
                pair_parts<WP>(x[0], x[1], dp);
                pair_parts<WP>(y[0], y[1], rp);
#pragma unroll
                for (int m = 0; m < 2 * KB; ++m) {
                    u32x4 a[PARTS], b[PARTS];
#pragma unroll
                    for (int i = 0; i < PARTS; ++i) {
                        a[i] = col_op<KD>(Q + i * C * KD, 32 * jb, m >> 1, m & 1, bk);
                        b[i] = col_op<KD>(K + i * C * KD, 32 * jb, m >> 1, m & 1, bk);
                    }
                    S[m] = mma_parts<PARTS, WP>(a, dp, S[m]);
                    S[m] = mma_parts<PARTS, WP>(b, rp, S[m]);
                }
            }
        }
        lds_barrier();      // q, k and A have been read
        if (n > 0) {
            if (ahead) {
                rk.load(K, wave, c0 - C, hi);
                rq.load(Q, wave, c0 - C, hi);
            }
            load_a(n - 1, lane);
        }
    }
    if (!active) return;
    float* dst = nullptr;
    if constexpr (MODE == kDeltaStates) dst = p.carry + (w.pi * p.H + h) * ssz;
    else if (w.first && p.s_out) dst = p.s_out + (int64_t(w.slot) * p.H + h) * ssz;
    if (!dst) return;
#pragma unroll
    for (int m = 0; m < 2 * KB; ++m)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int row = 32 * (m >> 1) + 8 * g4 + 4 * (m & 1) + r;
            if (row < p.dk && col < p.dv) dst[int64_t(row) * p.dv + col] = S[m][r];
        }
}

// ---------------------------------------------------------------- a chunk's gradients
struct GradArgs {
    DeltaPass p;
    const void* dout;
    const float* keep_d;    // [chunks][H][dk][dv]: dS_out
    void* dq;               // I/O type, or float32 per head (wide_out)
    void* dk;
    void* dv;
    float* dbeta;
    float* dg;
    double* part;           // [chunks][H] sums of dg (a decay per head), else null
    int64_t so, sdq;        // elements between tokens of dout, of dq and dk
    int32_t wide_out, pairs_k, pairs_v;
};

template <int CTRL> __device__ inline float plus_lane(float v) {
    return v + __uint_as_float(__builtin_amdgcn_update_dpp(0u, __float_as_uint(v), CTRL, 0xf, 0xf, true));
}
// The sum over the 16 lanes of a row, in each of them.
__device__ inline float sum16(float v) {
    v = plus_lane<0xB1>(v);
    v = plus_lane<0x4E>(v);
    v = plus_lane<0x141>(v);
    return plus_lane<0x140>(v);
}

// 8 values from column c on of a row of w float32 values; zero behind its end.
__device__ inline void load_row8(const float* row, bool on, int c, int w, bool vec, f32x4& x, f32x4& y) {
    x = y = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    if (!on) return;
    if (vec) {
        if (c < w) x = *reinterpret_cast<const f32x4*>(row + c);
        if (c + 4 < w) y = *reinterpret_cast<const f32x4*>(row + c + 4);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (c + e < w) x[e] = row[c + e];
            if (c + 4 + e < w) y[e] = row[c + 4 + e];
        }
    }
}

// Transposed left operand from 16 x 32 blocks in order of the rows: tile jt of the columns, the
// contraction over the 32 rows of pair ib.
template <int C> __device__ inline u32x4 block_t_op(const uint16_t* t, int ib, int jt, int lane) {
    const int g = lane >> 4, m = 8 * (g & 1) + ((lane >> 2) & 3), jb = jt >> 1, piece = 2 * (jt & 1) + ((lane & 3) >> 1);
    const char* const at = reinterpret_cast<const char*>(t) +
                           1024 * (g < 2 ? p_block(2 * ib, jb) : p_block(2 * ib + 1, jb)) + 8 * (lane & 1);
    const int tw = 2 * (g & 1);
    const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(at + 64 * m + 16 * (piece ^ tw)));
    const s16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(at + 64 * (m + 4) + 16 * (piece ^ (tw + 1))));
    const uint2 u = __builtin_bit_cast(uint2, x), v = __builtin_bit_cast(uint2, y);
    return u32x4{u.x, u.y, v.x, v.y};
}

constexpr int kGradThreads = 512, kGradWaves = 8;

// One workgroup per chunk and head.  First each wave forms U and Z of 16 columns of v (VS at a
// time) from the states of both sides, as the walks do; they go to LDS, and each wave
// then takes 16 columns of dq and dk, for which the states are read along their rows; the two
// matrices over the chunk's tokens, D and N, are shared out in tiles.
template <int PARTS, int KD, int C, int VS>
__global__ void __launch_bounds__(kGradThreads, 2) delta_grad_kernel(GradArgs ga) {
    const DeltaPass& p = ga.p;
    constexpr int IT = C / 16, JB = C / 32, KB = KD / 32, NB = tri_blocks<C>(), PB = NB * 512, WP = 3, TRI = WP * PB;
    constexpr int NTILE = IT * (IT + 1) / 2, MT = (NTILE + kGradWaves - 1) / kGradWaves;
    constexpr int NC = KD > 128 ? KD / 128 : 1;      // tiles of 16 columns of dq and dk a wave
    constexpr int VB = VS / 32;
    // at 64 tokens the first step's matrices lie where U and Z go after it
    constexpr bool ALIAS = C == 64;
    constexpr int UZE = 2 * WP * C * VS;
    static_assert(PARTS * C * VS + (ALIAS ? 2 * TRI : 0) <= UZE && 2 * TRI <= UZE, "what shares the place of U and Z fits");
    __shared__ __align__(16) uint16_t K[PARTS * C * KD], Q[PARTS * C * KD], O[PARTS * C * VS], UZ[UZE];
    __shared__ __align__(16) uint16_t own[ALIAS ? 8 : 2 * TRI];
    __shared__ Steps<C> st;
    __shared__ float pz[kGradWaves][C], pg[kGradWaves][C], pm[IT][C];
    __shared__ double ps[kGradWaves];
    uint16_t* const V = UZ;
    uint16_t* const A = ALIAS ? UZ + PARTS * C * VS : own;
    uint16_t* const PT = A + TRI;
    uint16_t* const Us = UZ;
    uint16_t* const Zs = UZ + WP * C * VS;

    const int tid = threadIdx.x, lane = tid & 63, g4 = lane >> 4, l16 = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const Chunks ch(p, C);
    const int64_t ci = blockIdx.x;
    const int h = blockIdx.y;
    const int seq = find_seq(ch, ci);
    const Seq sq = seq < 0 ? Seq{0, 0} : seq_range(ch, seq);
    const int64_t c0 = seq < 0 ? 0 : sq.start + (ci - piece_base(ch, seq)) * C, hi = sq.end;
    if (seq < 0 || c0 < sq.start || c0 >= hi) {
        if (ga.part && tid == 0) ga.part[ci * p.H + h] = 0.0;
        return;
    }
    const int64_t ssz = int64_t(p.dk) * p.dv;
    const float* const Sin = p.keep + (ci * p.H + h) * ssz;
    const float* const Sout = ga.keep_d + (ci * p.H + h) * ssz;

    for (int i = tid; i < kGradWaves * C; i += kGradThreads) (&pz[0][0])[i] = (&pg[0][0])[i] = 0.0f;
    for (int i = tid; i < IT * C; i += kGradThreads) (&pm[0][0])[i] = 0.0f;
    if (lane == 0) ps[wave] = 0.0;
    if (wave == 7) {
        const int64_t t = c0 + lane;
        const bool on = lane < C && t < hi;
        put_steps<C>(st, on ? p.g[t * p.sg + h] : 0.0f, on ? p.beta[t * p.H + h] : 0.0f, lane);
    }
    f32x4 aq[NC][IT], az[NC][IT], au[NC][IT], ap[MT], an[MT];
    const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int i = 0; i < IT; ++i) aq[c][i] = az[c][i] = au[c][i] = zero;
#pragma unroll
    for (int m = 0; m < MT; ++m) ap[m] = an[m] = zero;
    const auto tile = [](int m, int& it, int& jt) {
        it = m < 1 ? 0 : m < 3 ? 1 : m < 6 ? 2 : 3;
        jt = m - it * (it + 1) / 2;
    };
    {
        Rows<PARTS, C, KD, kGradThreads> rk, rq;
        rk.prepare(p.k, int64_t(h / p.rep) * p.dk, p.sk, p.dk, tid);
        rq.prepare(p.q, int64_t(h / p.rep) * p.dk, p.sq, p.dk, tid);
        if (p.wide) {
            rk.load(K, wave, c0, hi);
            rq.load(Q, wave, c0, hi);
            if constexpr (PARTS > 1) {
                rk.store(K, tid);
                rq.store(Q, tid);
            }
        } else {
            rk.copy(K, tid, c0, hi);
            rq.copy(Q, tid, c0, hi);
        }
        load_tri<C, kGradWaves>(p.tri + (ci * p.H + h) * tri_elems<C>(), A, wave, lane);
    }
    const bool vec = p.dv % 4 == 0;
    const int slices = (p.dv + VS - 1) / VS;
    for (int sl = 0; sl < slices; ++sl) {
        const int c_slice = sl * VS;
        {
            Rows<PARTS, C, VS, kGradThreads> ro, rv;
            ro.prepare(ga.dout, int64_t(h) * p.dv + c_slice, ga.so, p.dv - c_slice, tid);
            rv.prepare(p.v, int64_t(h) * p.dv + c_slice, p.sv, p.dv - c_slice, tid);
            if (p.wide) {
                ro.load(O, wave, c0, hi);
                rv.load(V, wave, c0, hi);
                if constexpr (PARTS > 1) {
                    ro.store(O, tid);
                    rv.store(V, tid);
                }
            } else {
                ro.copy(O, tid, c0, hi);
                rv.copy(V, tid, c0, hi);
            }
        }
        wait_memory<0>();
        __syncthreads();
        if (sl == 0) {
            put_pt<PARTS, KD, C, kGradWaves>(Q, K, PT, st, p.scale, wave, lane);
            __syncthreads();
        }
        // ---------------------------------------- U and Z of this wave's columns
        f32x4 U[IT], Z[IT];
        if (wave < VS / 16) {
            const int c_wave = c_slice + 16 * wave, col = c_wave + l16;
            const uint32_t bpair = pair_base<KD>(lane);
            f32x4 W[IT];
            double cross = 0.0;
#pragma unroll
            for (int i = 0; i < IT; ++i) U[i] = W[i] = zero;
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) {
                f32x4 s[2], d[2];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int row = 32 * kb + 8 * g4 + e;
                    const bool on = row < p.dk && col < p.dv;
                    s[e >> 2][e & 3] = on ? Sin[int64_t(row) * p.dv + col] : 0.0f;
                    d[e >> 2][e & 3] = on ? Sout[int64_t(row) * p.dv + col] : 0.0f;
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) cross = fma(double(s[e >> 2][e & 3]), double(d[e >> 2][e & 3]), cross);
                u32x4 sp[WP], dp[WP];
                pair_parts<WP>(s[0], s[1], sp);
                pair_parts<WP>(d[0], d[1], dp);
#pragma unroll
                for (int i = 0; i < IT; ++i) {
                    u32x4 a[PARTS];
#pragma unroll
                    for (int x = 0; x < PARTS; ++x) a[x] = pair_op<KD>(K + x * C * KD, 32 * (i >> 1), i & 1, kb, bpair);
                    U[i] = mma_parts<PARTS, WP>(a, sp, U[i]);
                    W[i] = mma_parts<PARTS, WP>(a, dp, W[i]);
                }
            }
            cross *= double(st.tail);
            const uint32_t bv = col_base<VS, 0>(16 * wave, lane), b32 = row_base<32>(lane), bt = tri_t_base(lane);
            f32x4 X[IT];
            u32x4 xp[JB][WP], op[JB][PARTS], v[JB][PARTS];
#pragma unroll
            for (int jb = 0; jb < JB; ++jb) {
                f32x4 x[2];
#pragma unroll
                for (int i = 0; i < PARTS; ++i) {
                    v[jb][i] = col_op<VS>(V + i * C * VS, 32 * jb, 0, 0, bv);
                    op[jb][i] = col_op<VS>(O + i * C * VS, 32 * jb, 0, 0, bv);
                }
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const int t0 = 32 * jb + 8 * g4 + 4 * half;
                    const f32x4 f = *reinterpret_cast<const f32x4*>(&st.in[t0]), b = *reinterpret_cast<const f32x4*>(&st.beta[t0]);
                    f32x4& X1 = X[2 * jb + half];
#pragma unroll
                    for (int r = 0; r < 4; r += 2) {
                        float y, z;
                        unpack<PARTS>(v[jb], 2 * half + r / 2, y, z);
                        X1[r] = fmaf(-f[r], U[2 * jb + half][r], y);
                        X1[r + 1] = fmaf(-f[r + 1], U[2 * jb + half][r + 1], z);
                    }
#pragma unroll
                    for (int r = 0; r < 4; ++r) x[half][r] = b[r] * X1[r];
                }
                pair_parts<WP>(x[0], x[1], xp[jb]);
            }
#pragma unroll
            for (int i = 0; i < IT; ++i) {
                U[i] = zero;
#pragma unroll
                for (int jb = 0; jb <= i / 2; ++jb) {
                    u32x4 a[WP];
#pragma unroll
                    for (int k = 0; k < WP; ++k) a[k] = row_op<32>(A + k * PB + p_block(i, jb) * 512, 0, 0, b32);
                    U[i] = mma_parts<WP, WP>(a, xp[jb], U[i]);
                }
                const f32x4 e = *reinterpret_cast<const f32x4*>(&st.out[32 * (i >> 1) + 8 * g4 + 4 * (i & 1)]);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    W[i][r] *= e[r];
                    cross = fma(double(U[i][r]), double(W[i][r]), cross);
                }
#pragma unroll
                for (int ip = i / 2; ip < JB; ++ip) {
                    u32x4 a[WP];
#pragma unroll
                    for (int k = 0; k < WP; ++k) a[k] = row_op<32>(PT + k * PB + pt_block<C>(i, ip) * 512, 0, 0, b32);
                    W[i] = mma_parts<WP, PARTS>(a, op[ip], W[i]);
                }
            }
            u32x4 wp[JB][WP];
#pragma unroll
            for (int ip = 0; ip < JB; ++ip) pair_parts<WP>(W[2 * ip], W[2 * ip + 1], wp[ip]);
#pragma unroll
            for (int i = 0; i < IT; ++i) {
                Z[i] = zero;
#pragma unroll
                for (int ip = i / 2; ip < JB; ++ip) {
                    u32x4 a[WP];
#pragma unroll
                    for (int k = 0; k < WP; ++k) a[k] = tri_t_op(A + k * PB, ip, i >> 1, i & 1, bt);
                    Z[i] = mma_parts<WP, WP>(a, wp[ip], Z[i]);
                }
                const int t0 = 32 * (i >> 1) + 8 * g4 + 4 * (i & 1);
                const f32x4 b = *reinterpret_cast<const f32x4*>(&st.beta[t0]);
                float vv[4];
#pragma unroll
                for (int r = 0; r < 4; r += 2) unpack<PARTS>(v[i >> 1], 2 * (i & 1) + r / 2, vv[r], vv[r + 1]);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    W[i][r] = b[r] * Z[i][r];
                    const float zx = sum16(Z[i][r] * X[i][r]), vr = sum16(vv[r] * W[i][r]);
                    if (l16 == 0) {
                        pz[wave][t0 + r] += zx;
                        pg[wave][t0 + r] -= vr;
                    }
                }
            }
            constexpr int E = PARTS == 1 ? 2 : 4;
            const int64_t pitch = int64_t(p.H) * p.dv * E;
            store_tiles<C, true>(W, static_cast<char*>(ga.dv) + c0 * pitch + int64_t(h) * p.dv * E, pitch, hi - c0, c_wave, p.dv,
                                 PARTS > 1, ga.pairs_v, lane);
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) cross += __shfl_xor(cross, d);
            if (lane == 0) ps[wave] += cross;
        }
        __syncthreads();        // v and, at 64 tokens, A and P^T have been read
        if (wave < VS / 16) {
#pragma unroll
            for (int i = 0; i < IT; ++i)
#pragma unroll
                for (int r = 0; r < 4; r += 2) {
                    const int t = 32 * (i >> 1) + 8 * g4 + 4 * (i & 1) + r, c = 16 * wave + l16;
                    uint32_t u[WP], z[WP];
                    split<WP>(U[i][r], U[i][r + 1], u);
                    split<WP>(Z[i][r], Z[i][r + 1], z);
#pragma unroll
                    for (int k = 0; k < WP; ++k) {
                        const int o0 = k * C * VS + at_piece<VS>(t, c >> 3) + (c & 7), o1 = k * C * VS + at_piece<VS>(t + 1, c >> 3) + (c & 7);
                        Us[o0] = static_cast<uint16_t>(u[k]);
                        Us[o1] = static_cast<uint16_t>(u[k] >> 16);
                        Zs[o0] = static_cast<uint16_t>(z[k]);
                        Zs[o1] = static_cast<uint16_t>(z[k] >> 16);
                    }
                }
        }
        __syncthreads();
        // ---------------------------------------- products over the columns of v
        const uint32_t bvs = row_base<VS>(lane);
#pragma unroll
        for (int vb = 0; vb < VB; ++vb) {
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                const int i0 = 16 * (wave + kGradWaves * c), row = i0 + l16;
                if (i0 >= p.dk) continue;
                f32x4 x, y;
                u32x4 sp[WP], dp[WP];
                load_row8(Sin + int64_t(row) * p.dv, row < p.dk, c_slice + 32 * vb + 8 * g4, p.dv, vec, x, y);
                pair_parts<WP>(x, y, sp);
                load_row8(Sout + int64_t(row) * p.dv, row < p.dk, c_slice + 32 * vb + 8 * g4, p.dv, vec, x, y);
                pair_parts<WP>(x, y, dp);
#pragma unroll
                for (int i = 0; i < IT; ++i) {
                    u32x4 o[PARTS], u[WP], z[WP];
#pragma unroll
                    for (int k = 0; k < PARTS; ++k) o[k] = row_op<VS>(O + k * C * VS, 16 * i, vb, bvs);
#pragma unroll
                    for (int k = 0; k < WP; ++k) {
                        u[k] = row_op<VS>(Us + k * C * VS, 16 * i, vb, bvs);
                        z[k] = row_op<VS>(Zs + k * C * VS, 16 * i, vb, bvs);
                    }
                    aq[c][i] = mma_parts<PARTS, WP>(o, sp, aq[c][i]);
                    az[c][i] = mma_parts<WP, WP>(z, sp, az[c][i]);
                    au[c][i] = mma_parts<WP, WP>(u, dp, au[c][i]);
                }
            }
#pragma unroll
            for (int mm = 0; mm < MT; ++mm) {
                const int m = wave + kGradWaves * mm;
                if (m >= NTILE) break;
                int it, jt;
                tile(m, it, jt);
                u32x4 o[PARTS], u[WP], z[WP];
#pragma unroll
                for (int k = 0; k < PARTS; ++k) o[k] = row_op<VS>(O + k * C * VS, 16 * it, vb, bvs);
#pragma unroll
                for (int k = 0; k < WP; ++k) {
                    u[k] = row_op<VS>(Us + k * C * VS, 16 * jt, vb, bvs);
                    z[k] = row_op<VS>(Zs + k * C * VS, 16 * it, vb, bvs);
                }
                ap[mm] = mma_parts<WP, PARTS>(u, o, ap[mm]);
                an[mm] = mma_parts<WP, WP>(u, z, an[mm]);
            }
        }
        __syncthreads();        // U, Z and the gradient of o have been read
    }
    // ---------------------------------------- D and N, tiles on and below the diagonal
    uint16_t* const Ds = UZ;
    uint16_t* const Ns = UZ + TRI;
    const uint32_t base = row_base<KD>(lane);
#pragma unroll
    for (int mm = 0; mm < MT; ++mm) {
        const int m = wave + kGradWaves * mm;
        if (m >= NTILE) break;
        int it, jt;
        tile(m, it, jt);
        f32x4 kk = zero;
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
            u32x4 x[PARTS], y[PARTS];
#pragma unroll
            for (int i = 0; i < PARTS; ++i) {
                x[i] = row_op<KD>(K + i * C * KD, 16 * jt, kb, base);
                y[i] = row_op<KD>(K + i * C * KD, 16 * it, kb, base);
            }
            kk = mma_parts<PARTS, PARTS>(x, y, kk);
        }
        const int i = 16 * it + l16, j0 = 16 * jt + 4 * g4;
        const float gi = st.hi[i], ei = st.lo[i], b = st.beta[i];
        float miss = 0.0f;
        f32x4 d, n;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const float e = __builtin_amdgcn_exp2f((gi - st.hi[j0 + r]) + (ei - st.lo[j0 + r]));
            d[r] = j0 + r <= i ? ap[mm][r] * (e * p.scale) : 0.0f;
            const float z = j0 + r < i ? an[mm][r] * e : 0.0f;
            n[r] = -b * z;
            miss = fmaf(z, j0 + r < i ? kk[r] : 0.0f, miss);
        }
        miss += __shfl_xor(miss, 16);
        miss += __shfl_xor(miss, 32);
        if (g4 == 0) pm[jt][i] = miss;
        const int o = p_block(it, jt >> 1) * 512 + 4 * (g4 & 1);
        const int at = o + at_piece<32>(l16, 2 * (jt & 1) + (g4 >> 1)), above = o + at_piece<32>(l16, 2 + (g4 >> 1));
        uint32_t x[WP], y[WP], u[WP], v[WP];
        split<WP>(d[0], d[1], x);
        split<WP>(d[2], d[3], y);
        split<WP>(n[0], n[1], u);
        split<WP>(n[2], n[3], v);
#pragma unroll
        for (int k = 0; k < WP; ++k) {
            *reinterpret_cast<uint2*>(Ds + k * PB + at) = uint2{x[k], y[k]};
            *reinterpret_cast<uint2*>(Ns + k * PB + at) = uint2{u[k], v[k]};
            if (it == jt && (it & 1) == 0) {   // the tile above the diagonal that shares this block
                *reinterpret_cast<uint2*>(Ds + k * PB + above) = uint2{0, 0};
                *reinterpret_cast<uint2*>(Ns + k * PB + above) = uint2{0, 0};
            }
        }
    }
    __syncthreads();
    // ---------------------------------------- dq and dk of this wave's columns
    {
        const uint32_t b32 = row_base<32>(lane);
        const int oe = PARTS > 1 || ga.wide_out ? 4 : 2;
        const int64_t pitch = ga.sdq * oe, at = c0 * pitch + int64_t(ga.wide_out ? h : h / p.rep) * p.dk * oe;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int i0 = 16 * (wave + kGradWaves * c);
            if (i0 >= p.dk) continue;
#pragma unroll
            for (int i = 0; i < IT; ++i) {
                const int t0 = 16 * i + 4 * g4;
                const f32x4 e = *reinterpret_cast<const f32x4*>(&st.in[t0]), f = *reinterpret_cast<const f32x4*>(&st.bin[t0]);
                const f32x4 l = *reinterpret_cast<const f32x4*>(&st.out[t0]);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    aq[c][i][r] *= e[r] * p.scale;
                    au[c][i][r] = fmaf(l[r], au[c][i][r], -f[r] * az[c][i][r]);
                }
            }
            const uint32_t bc = col_base<KD, 0>(i0, lane);
            u32x4 k[JB][PARTS], q[JB][PARTS];
#pragma unroll
            for (int jb = 0; jb < JB; ++jb)
#pragma unroll
                for (int i = 0; i < PARTS; ++i) {
                    k[jb][i] = col_op<KD>(K + i * C * KD, 32 * jb, 0, 0, bc);
                    q[jb][i] = col_op<KD>(Q + i * C * KD, 32 * jb, 0, 0, bc);
                }
#pragma unroll
            for (int i = 0; i < IT; ++i)
#pragma unroll
                for (int jb = 0; jb < JB; ++jb) {
                    u32x4 a[WP];
                    if (jb <= i / 2) {
#pragma unroll
                        for (int w = 0; w < WP; ++w) a[w] = row_op<32>(Ds + w * PB + p_block(i, jb) * 512, 0, 0, b32);
                        aq[c][i] = mma_parts<WP, PARTS>(a, k[jb], aq[c][i]);
#pragma unroll
                        for (int w = 0; w < WP; ++w) a[w] = row_op<32>(Ns + w * PB + p_block(i, jb) * 512, 0, 0, b32);
                        au[c][i] = mma_parts<WP, PARTS>(a, k[jb], au[c][i]);
                    }
                    if (jb >= i / 2) {
#pragma unroll
                        for (int w = 0; w < WP; ++w) a[w] = block_t_op<C>(Ds + w * PB, jb, i, lane);
                        au[c][i] = mma_parts<WP, PARTS>(a, q[jb], au[c][i]);
#pragma unroll
                        for (int w = 0; w < WP; ++w) a[w] = block_t_op<C>(Ns + w * PB, jb, i, lane);
                        au[c][i] = mma_parts<WP, PARTS>(a, k[jb], au[c][i]);
                    }
                }
            store_tiles<C, false>(aq[c], static_cast<char*>(ga.dq) + at, pitch, hi - c0, i0, p.dk, oe == 4, ga.pairs_k, lane);
            store_tiles<C, false>(au[c], static_cast<char*>(ga.dk) + at, pitch, hi - c0, i0, p.dk, oe == 4, ga.pairs_k, lane);
            // o . do = q . dq of each token
#pragma unroll
            for (int i = 0; i < IT; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int t = 16 * i + 4 * g4 + r, col = i0 + l16, o = at_piece<KD>(t, col >> 3) + (col & 7);
                    float x = 0.0f;
#pragma unroll
                    for (int w = PARTS - 1; w >= 0; --w) x += __uint_as_float(uint32_t(Q[w * C * KD + o]) << 16);
                    const float s = sum16(x * aq[c][i][r]);
                    if (l16 == 0) pg[wave][t] += s;
                }
        }
    }
    __syncthreads();
    if (wave == 0) {
        double x = 0.0, end = 0.0;
        float z = 0.0f;
        const int64_t t = c0 + lane;
        const bool on = lane < C && t < hi;
        if (lane < C) {
#pragma unroll
            for (int k = 0; k < kGradWaves; ++k) {
                x += double(pg[k][lane]);
                z += pz[k][lane];
            }
#pragma unroll
            for (int k = 0; k < IT; ++k) z -= pm[k][lane];
        }
#pragma unroll
        for (int k = 0; k < kGradWaves; ++k) end += ps[k];
        const double s = scan_f64(x);                       // of the tokens up to this one
        const double dg = end + (lane_f64(s, 63) - s) + x;
        if (on) {
            ga.dbeta[t * p.H + h] = z;
            if (!ga.part) ga.dg[t * p.H + h] = float(dg);
        }
        if (ga.part) {
            const double all = lane_f64(scan_f64(on ? dg : 0.0), 63);
            if (lane == 0) ga.part[ci * p.H + h] = all;
        }
    }
}

// dg per head: the chunks' sums, in a fixed order.
__global__ void __launch_bounds__(kThreads) delta_dg_sum_kernel(const double* part, float* dg, int64_t n, int H) {
    __shared__ double sums[kThreads];
    const int h = blockIdx.x;
    double s = 0.0;
    for (int64_t i = threadIdx.x; i < n; i += kThreads) s += part[i * H + h];
    sums[threadIdx.x] = s;
    __syncthreads();
    for (int d = kThreads / 2; d > 0; d >>= 1) {
        if (int(threadIdx.x) < d) sums[threadIdx.x] += sums[threadIdx.x + d];
        __syncthreads();
    }
    if (threadIdx.x == 0) dg[h] = float(sums[0]);
}

// Sums of dq and dk over the heads that share a row, in order, rounded once.
struct FoldArgs {
    const float* from[2];
    void* to[2];
    int64_t rows;          // tokens x kheads
    int32_t rep, width;
};
template <typename IO, int VW> __global__ void __launch_bounds__(kThreads) delta_fold_kernel(FoldArgs a) {
    typedef float vf __attribute__((ext_vector_type(VW)));
    const int64_t per = a.width / VW, n = a.rows * per, step = int64_t(gridDim.x) * kThreads;
    const float* const from = a.from[blockIdx.y];
    IO* const to = static_cast<IO*>(a.to[blockIdx.y]);
    for (int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x; i < n; i += step) {
        const int64_t row = i / per, c = (i - row * per) * VW;
        vf s = {};
#pragma unroll 4
        for (int r = 0; r < a.rep; ++r) s += *reinterpret_cast<const vf*>(from + (row * a.rep + r) * a.width + c);
        IO x[VW];
#pragma unroll
        for (int e = 0; e < VW; ++e) x[e] = IOT<IO>::from_f32(s[e]);
        __builtin_memcpy(to + row * a.width + c, x, sizeof(x));
    }
}

// Rows of no sequence (before the first and behind the last): zero gradients.  The widths are in
// bytes, multiples of 2.
struct ZeroRows {
    char* rows[5];
    int64_t width[5];
};
__global__ void __launch_bounds__(kThreads) delta_zero_kernel(DeltaPass p, ZeroRows z) {
    const int64_t lo = seq_range(p, 0).start, hi = seq_range(p, p.nseq - 1).end;
    const int64_t free = p.T - (hi > lo ? hi - lo : 0);
    for (int64_t i = blockIdx.x; i < free; i += gridDim.x) {
        const int64_t t = i < lo ? i : p.T - free + i;
#pragma unroll
        for (int k = 0; k < 5; ++k)
            for (int64_t e = threadIdx.x; z.rows[k] && e < z.width[k] / 2; e += kThreads)
                reinterpret_cast<uint16_t*>(z.rows[k] + t * z.width[k])[e] = 0;
    }
}

// ---------------------------------------------------------------- host
struct GradPlan {
    int chunk;
    int64_t nchunks, piece, npieces;
    bool pieced;
    size_t tri, keep, carry, trans, part, wide;   // bytes of one buffer each
    size_t bytes;
};

inline int make_grad_plan(const ssm_linattn_dims* d, bool packed, GradPlan* pl) {
    pl->chunk = d->io_dtype == SSM_BF16 && d->dk <= 128 && d->dv <= 128 ? 64 : 32;
    const int64_t each = packed ? d->tokens : d->tokens / d->nseq;
    const int64_t piece = d->piece_len;
    pl->pieced = piece > 0 && piece < each;
    pl->piece = pl->pieced ? piece : (int64_t(1) << 31);
    pl->npieces = !pl->pieced ? d->nseq : packed ? d->tokens / piece + d->nseq : d->nseq * cdiv(each, piece);
    pl->nchunks = count_chunks(d, packed, pl->chunk);
    if (pl->npieces > kMostGroups / (d->nheads * (cdiv(d->dv, kCols) + cdiv(d->dk, kCols))) || pl->nchunks > kMostGroups)
        return SSM_ERR_DIMS;
    const size_t nk = static_cast<size_t>(pl->nchunks * d->nheads), np = static_cast<size_t>(pl->npieces * d->nheads);
    const size_t state = static_cast<size_t>(d->dk * d->dv) * 4;
    pl->tri = up256(nk * (pl->chunk == 64 ? tri_elems<64>() : tri_elems<32>()) * 2);
    pl->keep = up256(nk * state);
    pl->carry = pl->pieced ? up256(np * state) : 0;
    pl->trans = pl->pieced ? up256(np * static_cast<size_t>(d->dk * d->dk) * 4) : 0;
    pl->part = d->head_decay ? up256(nk * 8) : 0;
    pl->wide = d->nheads > d->kheads ? up256(static_cast<size_t>(d->tokens * d->nheads * d->dk) * 4) : 0;
    pl->bytes = pl->tri + 2 * (pl->keep + pl->carry + pl->trans + pl->wide) + pl->part;
    return SSM_OK;
}

template <int C, int MODE> void run_rev(const DeltaPass& p, bool f32, hipStream_t s) {
    const dim3 grid(static_cast<uint32_t>(int64_t(p.npieces) * p.H * p.vslices)), block(kThreads);
#define SSM_REV(K)                                                                                  \
    do {                                                                                            \
        if constexpr (C == 32) {                                                                    \
            if (f32) launch_kernel(delta_rev_kernel<3, K, C, MODE>, grid, block, 0, s, p);          \
            else launch_kernel(delta_rev_kernel<1, K, C, MODE>, grid, block, 0, s, p);              \
        } else if constexpr (K <= 128) {                                                            \
            launch_kernel(delta_rev_kernel<1, K, C, MODE>, grid, block, 0, s, p);                   \
        }                                                                                           \
    } while (0)
    if (p.dk <= 64) SSM_REV(64);
    else if (p.dk <= 128) SSM_REV(128);
    else SSM_REV(256);
#undef SSM_REV
}

inline void run_rev(const DeltaPass& p, bool f32, int chunk, bool keep, hipStream_t s) {
    if (chunk == 64) {
        if (keep) run_rev<64, kDeltaKeep>(p, f32, s);
        else run_rev<64, kDeltaStates>(p, f32, s);
    } else {
        if (keep) run_rev<32, kDeltaKeep>(p, f32, s);
        else run_rev<32, kDeltaStates>(p, f32, s);
    }
}

inline void run_grad(const GradArgs& a, bool f32, int chunk, int64_t nchunks, hipStream_t s) {
    const dim3 grid(static_cast<uint32_t>(nchunks), a.p.H), block(kGradThreads);
    const auto start = [&](auto* kernel) { launch_kernel(kernel, grid, block, 0, s, a); };
    const int dk = a.p.dk;
    if (chunk == 64) {
        if (dk <= 64) start(delta_grad_kernel<1, 64, 64, 128>);
        else start(delta_grad_kernel<1, 128, 64, 128>);
    } else if (!f32) {
        if (dk <= 128) start(delta_grad_kernel<1, 128, 32, 128>);
        else start(delta_grad_kernel<1, 256, 32, 128>);
    } else {
        if (dk <= 64) start(delta_grad_kernel<3, 64, 32, 128>);
        else if (dk <= 128) start(delta_grad_kernel<3, 128, 32, 128>);
        else start(delta_grad_kernel<3, 256, 32, 64>);   // 128 columns of v would not fit the LDS
    }
}

template <typename IO> void run_fold(const FoldArgs& a, bool v4, hipStream_t s) {
    const int64_t n = a.rows * a.width / (v4 ? 4 : 1), blocks = cdiv(n, kThreads);
    const dim3 grid(static_cast<uint32_t>(blocks < 16384 ? blocks : 16384), 2), block(kThreads);
    if (v4) launch_kernel(delta_fold_kernel<IO, 4>, grid, block, 0, s, a);
    else launch_kernel(delta_fold_kernel<IO, 1>, grid, block, 0, s, a);
}

}  // namespace dl
}  // namespace

extern "C" {

size_t ssm_delta_bwd_workspace_bytes(const ssm_linattn_dims* dims) {
    la::Sizes z;
    dl::GradPlan pl;
    if (la::check_dims(dims, &z) != SSM_OK) return 0;
    size_t n = 0;
    if (dl::make_grad_plan(dims, true, &pl) == SSM_OK) n = pl.bytes;
    if (dims->tokens % dims->nseq == 0 && dl::make_grad_plan(dims, false, &pl) == SSM_OK && pl.bytes > n) n = pl.bytes;
    return n;
}

int ssm_delta_bwd(const void* q, const void* k, const void* v, const float* g, const float* beta,
                  const int32_t* cu_seqlens, const float* s0, const void* dout, const float* ds_last,
                  const ssm_delta_grads* grads, const ssm_linattn_dims* dims, void* stream) {
    using namespace dl;
    if (!dims || !q || !k || !v || !g || !beta || !dout || !grads || !grads->dq || !grads->dk || !grads->dv || !grads->dg ||
        !grads->dbeta)
        return SSM_ERR_NULL;
    if (s0 && !grads->ds0) return SSM_ERR_NULL;
    Sizes z;
    int st = check_dims(dims, &z);
    if (st != SSM_OK) return st;
    const ssm_linattn_dims& d = *dims;
    if (!cu_seqlens && d.tokens % d.nseq != 0) return SSM_ERR_DIMS;
    const int64_t lim = int64_t(1) << 40;
    if (d.nseq > lim / (d.nheads * d.dk * d.dv)) return SSM_ERR_DIMS;
    const ssm_delta_grads& gr = *grads;
    if (misaligned(q, z.e) || misaligned(k, z.e) || misaligned(v, z.e) || misaligned(dout, z.e) || misaligned(g, 4) ||
        misaligned(beta, 4) || misaligned(cu_seqlens, 4) || misaligned(s0, 4) || misaligned(ds_last, 4) ||
        misaligned(gr.dq, z.e) || misaligned(gr.dk, z.e) || misaligned(gr.dv, z.e) || misaligned(gr.dg, 4) ||
        misaligned(gr.dbeta, 4) || misaligned(gr.ds0, 4))
        return SSM_ERR_ALIGN;
    GradPlan pl;
    st = make_grad_plan(dims, cu_seqlens != nullptr, &pl);
    if (st != SSM_OK) return st;
    if (!d.workspace || d.workspace_bytes < pl.bytes || misaligned(d.workspace, 256)) return SSM_ERR_WORKSPACE;
    const int64_t wk = d.kheads * d.dk, wv = d.nheads * d.dv;
    const size_t nstate = static_cast<size_t>(d.nseq * d.nheads * d.dk * d.dv) * 4;
    const size_t ng = static_cast<size_t>(d.nheads * (d.head_decay ? 1 : d.tokens)) * 4;
    const size_t nb = static_cast<size_t>(d.nheads * d.tokens) * 4;
    const Area in[] = {rows_of(q, d.tokens, z.q, wk, z.e), rows_of(k, d.tokens, z.k, wk, z.e),
                       rows_of(v, d.tokens, z.v, wv, z.e), rows_of(dout, d.tokens, z.o, wv, z.e), flat(g, ng), flat(beta, nb),
                       flat(cu_seqlens, static_cast<size_t>(d.nseq + 1) * 4), flat(s0, nstate), flat(ds_last, nstate)};
    const Area out[] = {flat(gr.dq, static_cast<size_t>(d.tokens * wk * z.e)), flat(gr.dk, static_cast<size_t>(d.tokens * wk * z.e)),
                        flat(gr.dv, static_cast<size_t>(d.tokens * wv * z.e)), flat(gr.dg, ng), flat(gr.dbeta, nb),
                        flat(gr.ds0, nstate), flat(d.workspace, pl.bytes)};
    if (clash(in, out)) return SSM_ERR_ALIAS;

    char* ws = static_cast<char*>(d.workspace);
    auto take = [&](size_t n) {
        char* r = ws;
        ws += n;
        return reinterpret_cast<float*>(r);
    };
    uint16_t* const tri = reinterpret_cast<uint16_t*>(take(pl.tri));
    float* const keep_s = take(pl.keep);
    float* const keep_d = take(pl.keep);
    float* const carry_s = take(pl.carry);
    float* const carry_d = take(pl.carry);
    float* const trans = take(pl.trans);
    float* const trans_t = take(pl.trans);
    float* const wq = take(pl.wide);
    float* const wkk = take(pl.wide);
    double* const part = reinterpret_cast<double*>(take(pl.part));

    const bool f32 = d.io_dtype == SSM_F32, shared = d.nheads > d.kheads;
    DeltaPass f = {};
    f.q = q; f.k = k; f.v = v; f.g = g; f.beta = beta; f.cu = cu_seqlens; f.s_in = s0;
    f.tri = tri; f.keep = keep_s; f.carry = carry_s; f.trans = trans; f.trans_t = trans_t;
    f.sq = z.q; f.sk = z.k; f.sv = z.v; f.sg = d.head_decay ? 0 : d.nheads;
    f.T = d.tokens; f.L = cu_seqlens ? 0 : d.tokens / d.nseq;
    f.piece = pl.piece;
    f.rep = static_cast<int32_t>(d.nheads / d.kheads); f.H = static_cast<int32_t>(d.nheads);
    f.dk = static_cast<int32_t>(d.dk); f.dv = static_cast<int32_t>(d.dv);
    f.vslices = static_cast<int32_t>(cdiv(d.dv, kCols)); f.kslices = static_cast<int32_t>(cdiv(d.dk, kCols));
    f.nseq = f.nslots = static_cast<int32_t>(d.nseq);
    f.npieces = static_cast<int32_t>(pl.npieces); f.pieced = pl.pieced;
    f.wide = wide_rows(q, z.q, d.dk, z.e) && wide_rows(k, z.k, d.dk, z.e) && wide_rows(v, z.v, d.dv, z.e) &&
             wide_rows(dout, z.o, d.dv, z.e);
    f.scale = d.scale;
    DeltaPass r = f;     // against time
    r.v = dout; r.sv = z.o; r.s_in = ds_last; r.s_out = gr.ds0; r.keep = keep_d; r.carry = carry_d;
    GradArgs a = {};
    a.p = f; a.dout = dout; a.keep_d = keep_d; a.so = z.o;
    a.dq = shared ? static_cast<void*>(wq) : gr.dq; a.dk = shared ? static_cast<void*>(wkk) : gr.dk; a.dv = gr.dv;
    a.dbeta = gr.dbeta; a.dg = gr.dg; a.part = d.head_decay ? part : nullptr;
    a.sdq = d.nheads * d.dk; a.wide_out = shared;
    a.pairs_k = !shared && pair_rows(gr.dq, a.sdq, d.dk) && pair_rows(gr.dk, a.sdq, d.dk);
    a.pairs_v = pair_rows(gr.dv, wv, d.dv);

    hipStream_t s = static_cast<hipStream_t>(stream);
    launch_error = hipSuccess;
    launch_delta_tri(f, f32, pl.chunk, pl.nchunks, s);
    if (pl.pieced) {
        launch_delta_pass(f, f32, pl.chunk, kDeltaStates, s);
        launch_delta_carry(f, false, s);
        run_rev(r, f32, pl.chunk, false, s);
        launch_delta_carry(r, true, s);
    }
    launch_delta_pass(f, f32, pl.chunk, kDeltaKeep, s);
    run_rev(r, f32, pl.chunk, true, s);
    run_grad(a, f32, pl.chunk, pl.nchunks, s);
    if (shared) {
        const FoldArgs fa = {{wq, wkk}, {gr.dq, gr.dk}, d.tokens * d.kheads, f.rep, f.dk};
        const bool v4 = d.dk % 4 == 0 && !misaligned(gr.dq, 4 * z.e) && !misaligned(gr.dk, 4 * z.e);
        if (f32) run_fold<float>(fa, v4, s);
        else run_fold<uint16_t>(fa, v4, s);
    }
    if (d.head_decay)
        launch_kernel(delta_dg_sum_kernel, dim3(static_cast<uint32_t>(d.nheads)), dim3(kThreads), 0, s,
                      static_cast<const double*>(part), gr.dg, pl.nchunks, f.H);
    if (cu_seqlens) {
        const ZeroRows zero = {{static_cast<char*>(gr.dq), static_cast<char*>(gr.dk), static_cast<char*>(gr.dv),
                                d.head_decay ? nullptr : reinterpret_cast<char*>(gr.dg), reinterpret_cast<char*>(gr.dbeta)},
                               {wk * z.e, wk * z.e, wv * z.e, d.nheads * 4, d.nheads * 4}};
        launch_kernel(delta_zero_kernel, dim3(256), dim3(kThreads), 0, s, f, zero);
    }
    return launch_error == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

}  // extern "C"
