// delta_bwd.hip -- gradients of the gated delta rule.
//
// With dS_out the gradient of the state behind a chunk (and the names of delta.h),
//
//   dU = P^T dO + (e^{G_C-G} K) dS_out       Z = A^T dU       dR = beta Z = dV
//   dS_in = e^{G_C} dS_out + scale (e^G Q)^T dO - (e^G K)^T dR
//   dQ = scale e^G dO S_in^T + D K           D_ij = scale e^{G_i-G_j} dO_i . U_j, j <= i
//   dK = e^{G_C-G} U dS_out^T - e^G dR S_in^T + D^T Q + (N + N^T) K
//                                            N_ij = -beta_i e^{G_i-G_j} Z_i . U_j, j < i
//   dbeta_i = Z_i . r_i = Z_i . U_i / beta_i
//
// The decay of token t scales all that is written before it and read at it or later, so with what
// token i reads of S_in, what of token j's row is left in dS_out, and what i reads of j,
//
//   in_i = scale e^{G_i} dO_i . S_in^T q_i - beta_i e^{G_i} Z_i . S_in^T k_i
//   out_j = e^{G_C-G_j} U_j . dS_out^T k_j           W_ij = D_ij q_i . k_j + N_ij k_i . k_j, j < i
//   dg_t = e^{G_C} <S_in, dS_out> + sum_{i>=t} in_i + sum_{j<t} out_j + sum_{i>=t>j} W_ij
//
// Each term has the decays between as a factor.  (dg_t = dg_{t+1} + q_t . dq_t - v_t . dv_t, which
// needs no W, holds what a token reads of itself twice, without any decay: a dg of e^-10 would be what
// two such numbers leave of each other.)  Two walks over the chunks, the forward's and one against
// time, leave S_in and U, dS_out and Z of every chunk in memory; all gradients of a chunk are then
// formed by a workgroup of its own.
#include "delta_walk.h"

namespace {
namespace dl {

using namespace ssm_detail;

// Steps below this count as this in the gradients, so that r = U / beta is there for a step of
// zero too.  What they then add to a state is 2^-64 of what a step of one would, far below its
// rounding; the gradient of v is formed with the step as it came.
constexpr float kLeastStep = 5.42101086e-20f;   // 2^-64

// ---------------------------------------------------------------- the walks, with time and against it
// Neither waits for the other, and one alone leaves a SIMD without work between a chunk's
// products: one launch has the workgroups of both, two of which fit a CU.  4 x 4096 tokens of 32
// heads of 128: 335 and 510 us one after the other, 670 together, in which 1.7 GB of states, U and
// Z are written; a wave a SIMD issues vector instructions in 38% of its cycles alone, and both walks
// in 50%.  Three float32 documents of 8 heads: 85 and 124 us, and 127.
template <int PARTS, int KD, int MODE>
__global__ void __launch_bounds__(kThreads, KD == 256 ? 1 : 2) delta_walks_kernel(DeltaPass f, DeltaPass r, uint32_t nf) {
    union Room {
        PassRoom<PARTS, KD, MODE> f;
        RevRoom<PARTS, KD> r;
    };
    __shared__ Room room;
    if (blockIdx.x < nf) pass_walk<PARTS, KD, MODE>(f, blockIdx.x, room.f);
    else rev_walk<PARTS, KD, MODE>(r, blockIdx.x - nf, room.r);
}


// ---------------------------------------------------------------- a chunk's gradients
struct GradArgs {
    DeltaPass p;
    const void* dout;
    const float* keep_d;    // [chunks][H][dk][dv]: dS_out
    const float* z;         // [T][H][dv]: Z
    void* dq;               // I/O type, [T][kheads][dk]
    void* dk;
    float* sum_q;           // float32: sums over the heads so far, or each head's (wide_out)
    float* sum_k;
    float* dbeta;
    float* dg;
    double* part;           // [chunks][H] sums of dg (a decay per head), else null
    int64_t so, sdq;        // elements between tokens of dout, of dq and dk
    int32_t heads;          // of a workgroup
    int32_t wide_out, pairs_k;
};

template <int CTRL> __device__ inline float plus_lane(float v) {
    return v + __uint_as_float(__builtin_amdgcn_update_dpp(0u, __float_as_uint(v), CTRL, 0xf, 0xf, true));
}
// The sum over 4, 8 or 16 neighbouring lanes, in each of them.
__device__ inline float sum4(float v) { return plus_lane<0x4E>(plus_lane<0xB1>(v)); }
__device__ inline float sum8(float v) { return plus_lane<0x141>(sum4(v)); }
__device__ inline float sum16(float v) { return plus_lane<0x140>(sum8(v)); }

// Four values from column c on of a row of w, as they lie in memory; zero behind its end.  With
// `vec` a row's values come in whole fours.
template <typename IO> struct Raw4 {
    uint32_t u[sizeof(IO)];
    __device__ inline void load(const IO* row, bool on, int c, int w, bool vec) {
#pragma unroll
        for (int k = 0; k < int(sizeof(IO)); ++k) u[k] = 0;
        if (!on || c >= w) return;
        if (vec) {
            __builtin_memcpy(u, __builtin_assume_aligned(row + c, 4 * sizeof(IO)), sizeof(u));
        } else {
            IO raw[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) raw[e] = c + e < w ? row[c + e] : IO(0);
            __builtin_memcpy(u, raw, sizeof(u));
        }
    }
    __device__ inline f32x4 values() const {
        IO raw[4];
        __builtin_memcpy(raw, u, sizeof(raw));
        f32x4 x;
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = IOT<IO>::to_f32(raw[e]);
        return x;
    }
};

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

// Adds the tiles that store_tiles left as float32 in order of the tokens.
template <int C>
__device__ inline void add_tiles(f32x4 (&o)[C / 16], const float* row0, int64_t pitch, int64_t rows, int c_wave, int width, int lane) {
    const Rsrc ro = rows_rsrc(reinterpret_cast<char*>(const_cast<float*>(row0)), pitch, rows, C);
    const StoreRows to(pitch, false, C, lane >> 4);
    const int col = c_wave + (lane & 15);
    const uint32_t o0 = to.first(col < width, 4 * col);
    uint32_t x[C / 4];
#pragma unroll
    for (int i = 0; i < C / 4; ++i) x[i] = __builtin_amdgcn_raw_buffer_load_b32(ro, o0 + to.row(16 * (i >> 2) + (i & 3)), 0, 0);
#pragma unroll
    for (int i = 0; i < C / 4; ++i) o[i >> 2][i & 3] += __uint_as_float(x[i]);
}

// One workgroup per chunk and head, or the heads that share its q and k one after the other: what is
// contracted over the columns of v goes in steps of 32 of them, U, Z and the gradient of o through
// LDS, the states along their rows straight into registers, 16 or 32 columns of dq and dk a wave; the
// matrices over the chunk's tokens, D, N and W, are shared out in tiles.
//
// The states take 128 of the 224 KB that a chunk of 64 tokens and a head of 128 x 128 reads, so the
// bytes and their latency bound it: 4 x 4096 tokens of 32 heads, two on each q and k, in 762 us, 2.4 GB
// read and 0.5 written by the counters (2.1 and 0.5 are needed), 3.9 TB/s; waves wait in 53% of their
// cycles, vector instructions and matrix products take 30 and 23% of a SIMD's.  W, its sums and those of
// what comes in and goes out take 30 us more than the rows of v and the one sum without them did.  Loads
// are asked for a step ahead, as far as 256 registers allow: all at the step's start, 28 registers a lane
// lay in scratch memory, and those bytes took 50 us.
template <int PARTS, int KD, int C, int W>   // W waves
__global__ void __launch_bounds__(64 * W, 2) delta_grad_kernel(GradArgs ga) {
    typedef typename std::conditional<PARTS == 1, uint16_t, float>::type IO;
    const DeltaPass& p = ga.p;
    constexpr int IT = C / 16, JB = C / 32, KB = KD / 32, NB = tri_blocks<C>(), PB = NB * 512, WP = 3, TRI = WP * PB;
    constexpr int NTILE = IT * (IT + 1) / 2, MT = (NTILE + W - 1) / W;
    constexpr int NC = KD / (16 * W);                // tiles of 16 columns of dq and dk a wave
    constexpr int CPT = 32 * C / (64 * W) > 4 ? 8 : 4, N4 = CPT / 4;   // columns a thread brings of a step's rows
    constexpr int STEP = (2 * WP + PARTS) * C * 32;  // U, Z and the gradient of o, 32 columns
    __shared__ __align__(16) uint16_t K[PARTS * C * KD], Q[PARTS * C * KD], buf[STEP > 2 * TRI ? STEP : 2 * TRI];
    __shared__ Steps<C> st;
    __shared__ __align__(16) float pin[W][C], pout[W][C], wrow[IT][C], wcol[IT][C], zu[C];
    __shared__ double ps[W];
    uint16_t* const Us = buf;
    uint16_t* const Zs = buf + WP * C * 32;
    uint16_t* const Os = buf + 2 * WP * C * 32;

    const int tid = threadIdx.x;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const Chunks ch(p, C);
    const int64_t ci = blockIdx.x;
    const int h0 = blockIdx.y * ga.heads, hk = h0 / p.rep;
    const int seq = find_seq(ch, ci);
    const Seq sq = seq < 0 ? Seq{0, 0} : seq_range(ch, seq);
    const int64_t c0 = seq < 0 ? 0 : sq.start + (ci - piece_base(ch, seq)) * C, hi = sq.end;
    if (seq < 0 || c0 < sq.start || c0 >= hi) {
        for (int h = h0 + tid; ga.part && h < h0 + ga.heads; h += 64 * W) ga.part[ci * p.H + h] = 0.0;
        return;
    }
    const int64_t ssz = int64_t(p.dk) * p.dv;
    Rows<PARTS, C, KD, 64 * W> rk, rq;
    rk.prepare(p.k, int64_t(hk) * p.dk, p.sk, p.dk, tid);
    rq.prepare(p.q, int64_t(hk) * p.dk, p.sq, p.dk, tid);
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
    for (int h = h0; h < h0 + ga.heads; ++h) {
        if (h > h0) __syncthreads();    // the last head's sums have been read
        // the lane as the loop's own value: operand addresses are cheap to form anew
        int lane = __builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0u));
        asm volatile("" : "+v"(lane));
        const int tid = 64 * wave + lane, g4 = lane >> 4, l16 = lane & 15;
        const float* const Sin = p.keep + (ci * p.H + h) * ssz;
        const float* const Sout = ga.keep_d + (ci * p.H + h) * ssz;
        for (int i = tid; i < W * C; i += 64 * W) (&pin[0][0])[i] = (&pout[0][0])[i] = 0.0f;
        if (wave == W - 1) {
            const int64_t t = c0 + lane;
            const bool on = lane < C && t < hi;
            const double s = sum_decays(on ? p.g[t * p.sg + h] : 0.0f, lane < C), end = lane_f64(s, C - 1);
            if (lane < C) put_steps<C>(st, s, end, on ? p.beta[t * p.H + h] : 0.0f, p.least, lane);
        }
        const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
        f32x4 aq[NC][IT], az[NC][IT], au[NC][IT], ap[MT], an[MT];
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
        // rows of a step: 4 or 8 threads a token
        const int ts = tid / (32 / CPT), cs = CPT * (tid % (32 / CPT));
        const bool mine = ts < C, here = mine && c0 + ts < hi;
        const bool vec = p.dv % 4 == 0;
        const IO* const orow = static_cast<const IO*>(ga.dout) + (c0 + ts) * ga.so + int64_t(h) * p.dv;
        u32x4 nu[N4], nz[N4], ns[NC][2], nd[NC][2];
        Raw4<IO> no[N4];
        const Rsrc wu = rows_rsrc(reinterpret_cast<char*>(p.rows + (c0 * p.H + h) * p.dv), int64_t(p.H) * p.dv * 4, hi - c0, C);
        const Rsrc wz = rows_rsrc(const_cast<char*>(reinterpret_cast<const char*>(ga.z + (c0 * p.H + h) * p.dv)), int64_t(p.H) * p.dv * 4, hi - c0, C);
        const Rsrc ws = rows_rsrc(const_cast<char*>(reinterpret_cast<const char*>(Sin)), ssz * 4, 1, 1);
        const Rsrc wd = rows_rsrc(const_cast<char*>(reinterpret_cast<const char*>(Sout)), ssz * 4, 1, 1);
        // four values at column c of a row of v that begins at byte `row` of a window
        const auto four = [&](const Rsrc& w, uint32_t row, int c) {
            if (vec) return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(w, c < p.dv ? row + 4 * c : kPast, 0, 0));
            u32x4 x;
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = __builtin_amdgcn_raw_buffer_load_b32(w, c + e < p.dv ? row + 4 * (c + e) : kPast, 0, 0);
            return x;
        };
        const uint32_t trow = mine ? uint32_t(ts) * uint32_t(p.H * p.dv * 4) : kPast;
        const auto ask = [&](int c) {
#pragma unroll
            for (int x = 0; x < N4; ++x) {
                nu[x] = four(wu, trow, c + cs + 4 * x);
                nz[x] = four(wz, trow, c + cs + 4 * x);
                no[x].load(orow, here, c + cs + 4 * x, p.dv, p.wide);
            }
        };
        const auto ask_state = [&](const Rsrc& w, u32x4 (&n)[NC][2], int c) {
#pragma unroll
            for (int k = 0; k < NC; ++k)
#pragma unroll
                for (int x = 0; x < 2; ++x)   // rows it does not have lie behind the window
                    n[k][x] = four(w, uint32_t(16 * (wave + W * k) + l16) * uint32_t(p.dv * 4), c + 8 * g4 + 4 * x);
        };
        const auto f4 = [](const u32x4& x) { return __builtin_bit_cast(f32x4, x); };
        float s_zu = 0.0f;
        double cross = 0.0;
        ask(0);
        ask_state(ws, ns, 0);
        ask_state(wd, nd, 0);
        const uint32_t b32 = row_base<32>(lane);
        for (int c = 0; c < p.dv; c += 32) {
            if (mine) {
#pragma unroll
                for (int x = 0; x < N4; ++x) {
                    const f32x4 u = f4(nu[x]), z = f4(nz[x]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) s_zu = fmaf(z[e], u[e], s_zu);
                    // rows lie in tiles of 16 x 32, part by part
                    const int cc = cs + 4 * x, to = (ts >> 4) * 512 + at_piece<32>(ts & 15, cc >> 3) + (cc & 4);
                    const auto put = [&](uint16_t* at, const f32x4& x, auto parts) {
                        constexpr int N = decltype(parts)::value;
                        uint32_t a[N], b[N];
                        split<N>(x[0], x[1], a);
                        split<N>(x[2], x[3], b);
#pragma unroll
                        for (int k = 0; k < N; ++k) *reinterpret_cast<uint2*>(at + k * C * 32 + to) = uint2{a[k], b[k]};
                    };
                    put(Us, u, std::integral_constant<int, WP>{});
                    put(Zs, z, std::integral_constant<int, WP>{});
                    put(Os, no[x].values(), std::integral_constant<int, PARTS>{});
                }
            }
            u32x4 sp[NC][WP];
#pragma unroll
            for (int n = 0; n < NC; ++n) {
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int e = 0; e < 4; ++e) cross = fma(double(f4(ns[n][x])[e]), double(f4(nd[n][x])[e]), cross);
                pair_parts<WP>(f4(ns[n][0]), f4(ns[n][1]), sp[n]);
            }
            lds_barrier();
            const bool more = c + 32 < p.dv;
            if (more) ask(c + 32);
            // one state after the other: both in parts would not fit the registers
#pragma unroll
            for (int i = 0; i < IT; ++i) {
                u32x4 o[PARTS], z[WP];
#pragma unroll
                for (int k = 0; k < PARTS; ++k) o[k] = row_op<32>(Os + k * C * 32 + 512 * i, 0, 0, b32);
#pragma unroll
                for (int k = 0; k < WP; ++k) z[k] = row_op<32>(Zs + k * C * 32 + 512 * i, 0, 0, b32);
#pragma unroll
                for (int n = 0; n < NC; ++n) {
                    aq[n][i] = mma_parts<PARTS, WP>(o, sp[n], aq[n][i]);
                    az[n][i] = mma_parts<WP, WP>(z, sp[n], az[n][i]);
                }
                __builtin_amdgcn_sched_barrier(0);   // operands read further ahead would not fit either
            }
#pragma unroll
            for (int n = 0; n < NC; ++n) pair_parts<WP>(f4(nd[n][0]), f4(nd[n][1]), sp[n]);
            if (more) ask_state(ws, ns, c + 32);
#pragma unroll
            for (int i = 0; i < IT; ++i) {
                u32x4 u[WP];
#pragma unroll
                for (int k = 0; k < WP; ++k) u[k] = row_op<32>(Us + k * C * 32 + 512 * i, 0, 0, b32);
#pragma unroll
                for (int n = 0; n < NC; ++n) au[n][i] = mma_parts<WP, WP>(u, sp[n], au[n][i]);
                __builtin_amdgcn_sched_barrier(0);
            }
            if (more) ask_state(wd, nd, c + 32);
#pragma unroll
            for (int mm = 0; mm < MT; ++mm) {
                const int m = wave + W * mm;
                if (m >= NTILE) break;
                int it, jt;
                tile(m, it, jt);
                u32x4 o[PARTS], u[WP], z[WP];
#pragma unroll
                for (int k = 0; k < PARTS; ++k) o[k] = row_op<32>(Os + k * C * 32 + 512 * it, 0, 0, b32);
#pragma unroll
                for (int k = 0; k < WP; ++k) {
                    u[k] = row_op<32>(Us + k * C * 32 + 512 * jt, 0, 0, b32);
                    z[k] = row_op<32>(Zs + k * C * 32 + 512 * it, 0, 0, b32);
                }
                ap[mm] = mma_parts<WP, PARTS>(u, o, ap[mm]);
                an[mm] = mma_parts<WP, WP>(u, z, an[mm]);
                __builtin_amdgcn_sched_barrier(0);
            }
            lds_barrier();
        }
        s_zu = CPT == 8 ? sum4(s_zu) : sum8(s_zu);
        if (mine && cs == 0) zu[ts] = s_zu;
        cross *= double(st.tail[0]);
        wait_memory<0>();
        __syncthreads();        // q and k are there
        // ---------------------------------------- D, N and W, tiles on and below the diagonal
        uint16_t* const Ds = buf;
        uint16_t* const Ns = buf + TRI;
        const uint32_t base = row_base<KD>(lane);
#pragma unroll
        for (int mm = 0; mm < MT; ++mm) {
            const int m = wave + W * mm;
            if (m >= NTILE) break;
            int it, jt;
            tile(m, it, jt);
            const int i = 16 * it + l16, j0 = 16 * jt + 4 * g4;
            const float gi = st.hi[i], ei = st.lo[i], b = st.beta[i];
            f32x4 qk = zero, kk = zero;
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) {
                u32x4 x[PARTS], y[PARTS], z[PARTS];
#pragma unroll
                for (int k = 0; k < PARTS; ++k) {
                    x[k] = row_op<KD>(K + k * C * KD, 16 * jt, kb, base);
                    y[k] = row_op<KD>(Q + k * C * KD, 16 * it, kb, base);
                    z[k] = row_op<KD>(K + k * C * KD, 16 * it, kb, base);
                }
                qk = mma_parts<PARTS, PARTS>(x, y, qk);
                kk = mma_parts<PARTS, PARTS>(x, z, kk);
                __builtin_amdgcn_sched_barrier(0);
            }
            f32x4 d, n, w;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float e = __builtin_amdgcn_exp2f((gi - st.hi[j0 + r]) + (ei - st.lo[j0 + r]));
                d[r] = j0 + r <= i ? ap[mm][r] * (e * p.scale) : 0.0f;
                n[r] = j0 + r < i ? -b * (an[mm][r] * e) : 0.0f;
                w[r] = j0 + r < i ? fmaf(d[r], qk[r], n[r] * kk[r]) : 0.0f;
            }
            {
                float s = (w[0] + w[1]) + (w[2] + w[3]);
                s += __shfl_xor(s, 16);
                s += __shfl_xor(s, 32);
                if (g4 == 0) wrow[jt][i] = s;
#pragma unroll
                for (int r = 0; r < 4; ++r) w[r] = sum16(w[r]);
                if (l16 == 0) *reinterpret_cast<f32x4*>(&wcol[it][j0]) = w;
            }
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
        const auto element = [&](const uint16_t* t, int r, int col) {
            const int o = at_piece<KD>(r, col >> 3) + (col & 7);
            float x = 0.0f;
#pragma unroll
            for (int w = PARTS - 1; w >= 0; --w) x += __uint_as_float(uint32_t(t[w * C * KD + o]) << 16);
            return x;
        };
        {
            // a head of those that share q and k adds to the sum of the ones before it, or stands alone
            const bool sum = h > h0, wide = PARTS > 1 || ga.wide_out || h + 1 < h0 + ga.heads;
            const int64_t row0 = c0 * ga.sdq + int64_t(ga.wide_out ? h : hk) * p.dk, pitch4 = ga.sdq * 4;
            float *const tq = ga.sum_q + row0, *const tk = ga.sum_k + row0;
            const int oe = wide ? 4 : 2;
            const int64_t pitch = ga.sdq * oe;
            char* const to_q = wide ? reinterpret_cast<char*>(tq) : static_cast<char*>(ga.dq) + row0 * oe;
            char* const to_k = wide ? reinterpret_cast<char*>(tk) : static_cast<char*>(ga.dk) + row0 * oe;
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                const int i0 = 16 * (wave + W * c);
                if (i0 >= p.dk) continue;
#pragma unroll
                for (int i = 0; i < IT; ++i) {
                    const int t0 = 16 * i + 4 * g4;
                    const f32x4 e = *reinterpret_cast<const f32x4*>(&st.in[t0]), f = *reinterpret_cast<const f32x4*>(&st.bin[t0]);
                    const f32x4 l = *reinterpret_cast<const f32x4*>(&st.out[t0]);
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float q = element(Q, t0 + r, i0 + l16), k = element(K, t0 + r, i0 + l16), z = f[r] * az[c][i][r];
                        aq[c][i][r] *= e[r] * p.scale;
                        au[c][i][r] *= l[r];
                        const float in = sum16(fmaf(q, aq[c][i][r], -(z * k))), out = sum16(au[c][i][r] * k);
                        if (l16 == 0) {
                            pin[wave][t0 + r] += in;
                            pout[wave][t0 + r] += out;
                        }
                        au[c][i][r] -= z;
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
                if (sum) {
                    add_tiles<C>(aq[c], tq, pitch4, hi - c0, i0, p.dk, lane);
                    add_tiles<C>(au[c], tk, pitch4, hi - c0, i0, p.dk, lane);
                }
                store_tiles<C, false>(aq[c], to_q, pitch, hi - c0, i0, p.dk, wide, ga.pairs_k, lane);
                store_tiles<C, false>(au[c], to_k, pitch, hi - c0, i0, p.dk, wide, ga.pairs_k, lane);
            }
        }
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) cross += __shfl_xor(cross, d);
        if (lane == 0) ps[wave] = cross;
        __syncthreads();
        if (wave == 0) {
            double x = 0.0, y = 0.0, dg = 0.0;
            const int64_t t = c0 + lane;
            const bool on = lane < C && t < hi;
            if (lane < C) {
                // the sum of W over i >= t > j by rows less columns from t on
#pragma unroll
                for (int k = 0; k < IT; ++k) {
                    if (k <= lane / 16) x += double(wrow[k][lane]);
                    if (k >= lane / 16) x -= double(wcol[k][lane]);
                }
#pragma unroll
                for (int k = 0; k < W; ++k) {
                    x += double(pin[k][lane]);
                    y += double(pout[k][lane]);
                }
            }
#pragma unroll
            for (int k = 0; k < W; ++k) dg += ps[k];
            // from this token on, and up to the one before: no differences of longer sums, which would
            // leave 2^-53 of what no decay has made small
            const double after = __shfl(scan_f64(__shfl(x, 63 - lane)), 63 - lane), before = __shfl_up(scan_f64(y), 1);
            dg += after + (lane > 0 ? before : 0.0);
            if (on) {
                ga.dbeta[t * p.H + h] = zu[lane] / st.beta[lane];     // Z . r = Z . U / beta
                if (!ga.part) ga.dg[t * p.H + h] = float(dg);
            }
            if (ga.part) {
                const double all = lane_f64(scan_f64(on ? dg : 0.0), 63);
                if (lane == 0) ga.part[ci * p.H + h] = all;
            }
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
struct GradPlan : Cut {
    int chunk, heads;   // heads of a workgroup over a chunk's gradients
    int64_t nchunks;
    size_t tri, steps, keep, rows, carry, trans, part, wide;   // bytes of one buffer each
    size_t bytes;
};

inline int make_grad_plan(const ssm_linattn_dims* d, bool packed, GradPlan* pl) {
    const int64_t vs = cdiv(d->dv, kCols), ks = cdiv(d->dk, kCols);
    pl->chunk = d->io_dtype == SSM_BF16 ? 64 : 32;
    pl->nchunks = count_chunks(d, packed, pl->chunk);
    if (!cut_sequences(d, packed, choose_piece(d, packed, 1, 2), 2 * vs, 2 * vs + ks, pl) || pl->nchunks > kMostGroups) return SSM_ERR_DIMS;
    const size_t nk = static_cast<size_t>(pl->nchunks * d->nheads), np = static_cast<size_t>(pl->npieces * d->nheads);
    const size_t state = static_cast<size_t>(d->dk * d->dv) * 4;
    pl->tri = up256(nk * (pl->chunk == 64 ? tri_elems<64>() : tri_elems<32>()) * 2);
    pl->steps = nk * static_cast<size_t>(pl->chunk / kChunk) * sizeof(Steps<kChunk>);
    pl->keep = up256(nk * state);
    pl->rows = up256(static_cast<size_t>(d->tokens * d->nheads * d->dv) * 4);
    pl->carry = pl->pieced ? up256(np * state) : 0;
    pl->trans = pl->pieced ? up256(np * static_cast<size_t>(d->dk * d->dk) * 4) : 0;
    pl->part = d->head_decay ? up256(nk * 8) : 0;
    // Heads that share q and k go one after the other where the chunks fill the card without them,
    // and else leave their gradients in float32 to be summed.  Measured, us in turn and summed, heads
    // of 128 in bf16: 128 workgroups (2048 tokens, 32 heads on 4) 484 and 355, 256 (on 8) 393 and
    // 346, 512 (2048 on 16; 4096 on 8) 333 and 348, 603 and 632, 4096 (4 x 4096 on 16) 1441 and 1560.
    const bool shared = d->nheads > d->kheads, in_turn = shared && pl->nchunks * d->kheads >= 2 * kCus;
    pl->heads = in_turn ? static_cast<int>(d->nheads / d->kheads) : 1;
    const size_t wide = shared && !in_turn ? d->nheads : in_turn && d->io_dtype == SSM_BF16 ? d->kheads : 0;
    pl->wide = up256(static_cast<size_t>(d->tokens * d->dk) * wide * 4);
    pl->bytes = pl->tri + pl->steps + 2 * (pl->keep + pl->rows + pl->carry + pl->trans + pl->wide) + pl->part;
    return SSM_OK;
}

template <int MODE> void run_walks(const DeltaPass& f, const DeltaPass& r, bool f32, hipStream_t s) {
    const int64_t units = int64_t(f.npieces) * f.H;
    const uint32_t nf = static_cast<uint32_t>(units * (MODE == kDeltaStates ? f.vslices + f.kslices : f.vslices));
    const dim3 grid(nf + static_cast<uint32_t>(units * f.vslices)), block(kThreads);
#define SSM_WALKS(K)                                                                                \
    do {                                                                                            \
        if (f32) launch_kernel(delta_walks_kernel<3, K, MODE>, grid, block, 0, s, f, r, nf);        \
        else launch_kernel(delta_walks_kernel<1, K, MODE>, grid, block, 0, s, f, r, nf);            \
    } while (0)
    if (f.dk <= 64) SSM_WALKS(64);
    else if (f.dk <= 128) SSM_WALKS(128);
    else SSM_WALKS(256);
#undef SSM_WALKS
}

inline void run_grad(const GradArgs& a, bool f32, int64_t nchunks, hipStream_t s) {
    const dim3 grid(static_cast<uint32_t>(nchunks), a.p.H / a.heads);
#define SSM_GRAD(K, W)                                                                              \
    do {                                                                                            \
        if (f32) launch_kernel(delta_grad_kernel<3, K, 32, W>, grid, dim3(64 * W), 0, s, a);        \
        else launch_kernel(delta_grad_kernel<1, K, 64, W>, grid, dim3(64 * W), 0, s, a);            \
    } while (0)
    if (a.p.dk <= 64) SSM_GRAD(64, 4);
    else if (a.p.dk <= 128) SSM_GRAD(128, 4);
    else SSM_GRAD(256, 8);
#undef SSM_GRAD
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
    float* const steps = take(pl.steps);
    float* const keep_s = take(pl.keep);
    float* const keep_d = take(pl.keep);
    float* const rows_u = take(pl.rows);
    float* const rows_z = take(pl.rows);
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
    f.tri = tri; f.steps = steps; f.keep = keep_s; f.carry = carry_s; f.trans = trans; f.trans_t = trans_t;
    f.sq = z.q; f.sk = z.k; f.sv = z.v; f.sg = d.head_decay ? 0 : d.nheads;
    f.T = d.tokens; f.L = cu_seqlens ? 0 : d.tokens / d.nseq;
    f.piece = pl.piece; f.block = pl.chunk;
    f.rep = static_cast<int32_t>(d.nheads / d.kheads); f.H = static_cast<int32_t>(d.nheads);
    f.dk = static_cast<int32_t>(d.dk); f.dv = static_cast<int32_t>(d.dv);
    f.vslices = static_cast<int32_t>(cdiv(d.dv, kCols)); f.kslices = static_cast<int32_t>(cdiv(d.dk, kCols));
    f.nseq = f.nslots = static_cast<int32_t>(d.nseq);
    f.npieces = static_cast<int32_t>(pl.npieces); f.pieced = pl.pieced;
    f.wide = wide_rows(q, z.q, d.dk, z.e) && wide_rows(k, z.k, d.dk, z.e) && wide_rows(v, z.v, d.dv, z.e) &&
             wide_rows(dout, z.o, d.dv, z.e);
    f.scale = d.scale; f.least = kLeastStep; f.rows = rows_u;
    DeltaPass r = f;     // against time
    r.v = dout; r.sv = z.o; r.s_in = ds_last; r.s_out = gr.ds0; r.keep = keep_d; r.carry = carry_d;
    r.rows = rows_z; r.dv_out = gr.dv; r.pairs = pair_rows(gr.dv, wv, d.dv);
    GradArgs a = {};
    a.p = f; a.dout = dout; a.keep_d = keep_d; a.z = rows_z; a.so = z.o;
    a.heads = pl.heads; a.wide_out = shared && pl.heads == 1;
    a.dq = gr.dq; a.dk = gr.dk;
    // float32 sums stand where they belong; those of bf16 gradients, and each head's, in the workspace
    a.sum_q = f32 && !a.wide_out ? static_cast<float*>(gr.dq) : wq;
    a.sum_k = f32 && !a.wide_out ? static_cast<float*>(gr.dk) : wkk;
    a.dbeta = gr.dbeta; a.dg = gr.dg; a.part = d.head_decay ? part : nullptr;
    a.sdq = (a.wide_out ? d.nheads : d.kheads) * d.dk;
    a.pairs_k = pair_rows(gr.dq, a.sdq, d.dk) && pair_rows(gr.dk, a.sdq, d.dk);

    hipStream_t s = static_cast<hipStream_t>(stream);
    launch_error = hipSuccess;
    launch_delta_tri(f, f32, pl.nchunks, s);
    if (pl.pieced) {
        run_walks<kDeltaStates>(f, r, f32, s);
        launch_delta_carry(f, &r, s);
    }
    run_walks<kDeltaKeep>(f, r, f32, s);
    run_grad(a, f32, pl.nchunks, s);
    if (a.wide_out) {
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
