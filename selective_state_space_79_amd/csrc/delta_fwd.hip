// delta_fwd.hip -- the gated delta rule: the triangular systems of all chunks, the walk over
// them (packed sequences, cut into pieces along the tokens when there are few heads and
// sequences) and the single-token step.
#include "delta_walk.h"

namespace {
namespace dl {

using namespace ssm_detail;

// ---------------------------------------------------------------- the triangular systems
// A = (I + beta M)^-1 of one chunk and head, unit lower triangular.  The diagonal blocks of 16
// by forward substitution, a column a lane; then the blocks below, -A_22 M_21 A_11, first of 16
// in 32 and then of 32 in 64, in float32 products (with bf16 parts the splits would cost more
// than these few products).  Forward substitution and not powers of M: for equal keys these
// grow like binomials and cancel.  131072 tokens of 16 heads of 128: 226 us, 268 MB of keys read and
// 470 MB written (3.3 TB/s); most of a wave's time it waits, for its rows or at a barrier (77%).
template <int PARTS, int KD, int C>
__global__ void __launch_bounds__(kThreads) delta_tri_kernel(DeltaPass p) {
    constexpr int IT = C / 16, KB = KD / 32, NTILE = IT * (IT + 1) / 2, P = C + 4, NB = tri_blocks<C>();
    __shared__ __align__(16) uint16_t K[PARTS * C * KD];
    __shared__ __align__(16) float M[C * P], A[C * P];
    __shared__ Steps<C> st;
    const int tid = threadIdx.x, lane = tid & 63, g4 = lane >> 4, l16 = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const Chunks ch(p, C);
    const int64_t ci = blockIdx.x;
    const int h = blockIdx.y;
    const int seq = find_seq(ch, ci);
    if (seq < 0) return;
    const Seq sq = seq_range(ch, seq);
    const int64_t c0 = sq.start + (ci - piece_base(ch, seq)) * C;
    if (c0 < sq.start || c0 >= sq.end) return;
    Rows<PARTS, C, KD, kThreads> rk;
    rk.prepare(p.k, int64_t(h / p.rep) * p.dk, p.sk, p.dk, tid);
    if (p.wide) {
        rk.load(K, wave, c0, sq.end);
        if constexpr (PARTS > 1) rk.store(K, tid);
    } else {
        rk.copy(K, tid, c0, sq.end);
    }
    if (wave == 3) {
        const int64_t t = c0 + lane;
        const bool on = lane < C && t < sq.end;
        const float beta = on ? p.beta[t * p.H + h] : 0.0f;
        const double s = sum_decays(on ? p.g[t * p.sg + h] : 0.0f, lane < C), end = lane_f64(s, C - 1);
        if (lane < C) put_steps<C>(st, s, end, beta, p.least, lane);
        // for the walks' chunks, sums of their own
        constexpr int per = C / kChunk;
        const double middle = per == 2 ? lane_f64(s, kChunk - 1) : 0.0;
        const bool second = lane >= kChunk;
        auto* const to = reinterpret_cast<Steps<kChunk>*>(p.steps + ((ci * per + (second ? 1 : 0)) * p.H + h) * 256);
        if (lane < C)
            put_steps<kChunk>(*to, second ? s - middle : s, second || per == 1 ? end - (second ? middle : 0.0) : middle, beta, p.least,
                              lane % kChunk);
    }
    wait_memory<0>();
    __syncthreads();
    const uint32_t base = row_base<KD>(lane);
    for (int m = wave; m < NTILE; m += 4) {
        const int it = m < 1 ? 0 : m < 3 ? 1 : m < 6 ? 2 : 3, jt = m - it * (it + 1) / 2;
        f32x4 a = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
            u32x4 x[PARTS], y[PARTS];
#pragma unroll
            for (int i = 0; i < PARTS; ++i) {
                x[i] = row_op<KD>(K + i * C * KD, 16 * jt, kb, base);
                y[i] = row_op<KD>(K + i * C * KD, 16 * it, kb, base);
            }
            a = mma_parts<PARTS, PARTS>(x, y, a);
        }
        const int i = 16 * it + l16, j0 = 16 * jt + 4 * g4;
        const float gi = st.hi[i], ei = st.lo[i], b = st.beta[i];
        f32x4 w;
#pragma unroll
        for (int r = 0; r < 4; ++r)
            w[r] = j0 + r < i ? a[r] * (b * __builtin_amdgcn_exp2f((gi - st.hi[j0 + r]) + (ei - st.lo[j0 + r]))) : 0.0f;
        *reinterpret_cast<f32x4*>(&M[i * P + j0]) = w;
    }
    __syncthreads();
    if (wave == 0 && g4 < IT) {
        float x[16];
        const float* m = M + (16 * g4) * P + 16 * g4;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float v = i == l16 ? 1.0f : 0.0f;
#pragma unroll
            for (int j4 = 0; j4 < i; j4 += 4) {
                const f32x4 w = *reinterpret_cast<const f32x4*>(m + i * P + j4);
#pragma unroll
                for (int j = j4; j < j4 + 4 && j < i; ++j) v = fmaf(-w[j - j4], x[j], v);
            }
            x[i] = v;
            A[(16 * g4 + i) * P + 16 * g4 + l16] = v;
        }
    }
    __syncthreads();
    const auto f32 = [](float a, float b, const f32x4& c) { return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0); };
    // 16 in 32: of the contraction, lane group g takes 4g + r in step r, so that a float4 is the
    // left operand of four steps and a product the right one of the next
    if (wave < IT / 2) {
        const int a0 = 32 * wave, b0 = a0 + 16;
        const f32x4 m = *reinterpret_cast<const f32x4*>(&M[(b0 + l16) * P + a0 + 4 * g4]);
        f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f}, y = x;
#pragma unroll
        for (int r = 0; r < 4; ++r) x = f32(m[r], A[(a0 + 4 * g4 + r) * P + a0 + l16], x);
        const f32x4 a = *reinterpret_cast<const f32x4*>(&A[(b0 + l16) * P + b0 + 4 * g4]);
#pragma unroll
        for (int r = 0; r < 4; ++r) y = f32(a[r], x[r], y);
#pragma unroll
        for (int r = 0; r < 4; ++r) A[(b0 + 4 * g4 + r) * P + a0 + l16] = -y[r];
    }
    __syncthreads();
    if constexpr (C == 64) {   // 32 in 64, 16 columns a wave
        if (wave < 2) {
            f32x4 x[2];
#pragma unroll
            for (int rt = 0; rt < 2; ++rt) {
                x[rt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
                for (int kt = wave; kt < 2; ++kt) {   // A's first block row has no second block
                    const f32x4 m = *reinterpret_cast<const f32x4*>(&M[(32 + 16 * rt + l16) * P + 16 * kt + 4 * g4]);
#pragma unroll
                    for (int r = 0; r < 4; ++r) x[rt] = f32(m[r], A[(16 * kt + 4 * g4 + r) * P + 16 * wave + l16], x[rt]);
                }
            }
#pragma unroll
            for (int rt = 0; rt < 2; ++rt) {
                f32x4 y = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int kt = 0; kt <= rt; ++kt) {
                    const f32x4 a = *reinterpret_cast<const f32x4*>(&A[(32 + 16 * rt + l16) * P + 32 + 16 * kt + 4 * g4]);
#pragma unroll
                    for (int r = 0; r < 4; ++r) y = f32(a[r], x[kt][r], y);
                }
#pragma unroll
                for (int r = 0; r < 4; ++r) A[(32 + 16 * rt + 4 * g4 + r) * P + 16 * wave + l16] = -y[r];
            }
        }
        __syncthreads();
    }
    // out: tiles in paired rows, the pieces of a row as the walk's reads want them
    uint16_t* const out = p.tri + (ci * p.H + h) * tri_elems<C>();
    const int m = lane >> 2, piece = (lane & 3) ^ twist<32>(m);
    for (int b = wave; b < NB; b += 4) {
        const int it = C == 32 ? b : b < 2 ? b : 2 + (b - 2) / 2, jb = C == 32 ? 0 : b < 2 ? 0 : (b - 2) & 1;
        const int i = 32 * (it >> 1) + 8 * (m >> 2) + 4 * (it & 1) + (m & 3), j0 = 32 * jb + 8 * piece;
        u32x4 v[3];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int j = j0 + 2 * e;
            uint32_t w[3];
            split<3>(j <= i ? A[i * P + j] : 0.0f, j + 1 <= i ? A[i * P + j + 1] : 0.0f, w);
#pragma unroll
            for (int k = 0; k < 3; ++k) v[k][e] = w[k];
        }
#pragma unroll
        for (int k = 0; k < 3; ++k) *reinterpret_cast<u32x4*>(out + (k * NB + b) * 512 + 8 * lane) = v[k];
    }
}

// ---------------------------------------------------------------- the walk
template <int PARTS, int KD, int MODE>
__global__ void __launch_bounds__(kThreads, pass_waves(KD, PARTS, MODE)) delta_pass_kernel(DeltaPass p) {
    __shared__ PassRoom<PARTS, KD, MODE> room;
    pass_walk<PARTS, KD, MODE>(p, blockIdx.x, room);
}

// ---------------------------------------------------------------- pieces' starting states
// Walks the pieces of one sequence and head for 64 columns of the state (128 with keys over 128, where
// 512 threads share the rows of W; their 256 registers do not hold S, N, the parts and the rows ahead,
// and 564 bytes of a lane lie in scratch memory), 16 a wave: each piece's own end state N is replaced by the state S it starts from, and
// the next one starts from W S + N with the piece's transition W (against time its transpose).  W
// does not depend on what came before, so its rows are asked for four tiles of 16 ahead, and all
// waves share their split.  A piece after the other is latency: 16 pieces of 16 heads of 128 in
// 100 us; with 128 columns, two waves a SIMD, a piece took 8.8 us instead of 6.3.
constexpr int carry_threads(int KD) { return KD == 256 ? 512 : 256; }

template <int KD, bool REV>
__device__ __forceinline__ void carry_walk(const DeltaPass& p, int h, uint16_t (&Ws)[2][3 * 16 * KD]) {
    constexpr int KB = KD / 32, WP = 3, TPR = carry_threads(KD) / 16, VPT = KD / TPR, AHEAD = 4;   // threads of a tile's row, values of each
    const int tid = threadIdx.x, lane = tid & 63, g4 = lane >> 4, l16 = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int seq = blockIdx.z;
    const int slot = REV ? seq : find_slot(p.slots, p.nslots, seq);
    if (slot < 0) return;
    const Seq sq = seq_range(p, seq);
    const int64_t base = uniform(piece_base(p, seq));
    int64_t n = (sq.end - sq.start + p.piece - 1) / p.piece;
    if (n < 2) return;   // a single piece starts from the user's state
    if (base + n > p.npieces) n = p.npieces - base;
    const int c_wave = blockIdx.x * (carry_threads(KD) / 4) + 16 * wave;
    const int64_t ssz = int64_t(p.dk) * p.dv, tsz = int64_t(p.dk) * p.dk;
    const auto number = [&](int64_t k) { return (base + (REV ? n - 1 - k : k)) * p.H + h; };
    f32x4 S[2 * KB];
    load_state<KB>(S, p.s_in ? p.s_in + (int64_t(slot) * p.H + h) * ssz : nullptr, p.dk, p.dv, c_wave, lane);
    // tile m of the rows of piece k's transition: row ti in the order of the state's tiles
    const int ti = tid / TPR, tc = tid % TPR * VPT, to = at_piece<KD>(ti, tc >> 3) + (tc & 7);
    float ahead[AHEAD][VPT];
    const auto ask = [&](int64_t k, int m, float (&x)[VPT]) {
        const int out = 32 * (m >> 1) + 8 * (ti >> 2) + 4 * (m & 1) + (ti & 3);
        const float* const q = (REV ? p.trans_t : p.trans) + number(k) * tsz + int64_t(out) * p.dk + tc;
        if (k + 1 >= n) return;
        if (p.dk % VPT == 0 && VPT > 1) {
#pragma unroll
            for (int e = 0; e < VPT; ++e) x[e] = 0.0f;
            if (out < p.dk && tc < p.dk) __builtin_memcpy(x, q, sizeof(x));
        } else {
#pragma unroll
            for (int e = 0; e < VPT; ++e) x[e] = out < p.dk && tc + e < p.dk ? q[e] : 0.0f;
        }
    };
#pragma unroll
    for (int m = 0; m < AHEAD; ++m) ask(0, m, ahead[m]);
    const uint32_t b = row_base<KD>(lane);
    for (int64_t k = 0; k < n; ++k) {
        float* const own = p.carry + number(k) * ssz;
        f32x4 N[2 * KB];
        load_state<KB>(N, k + 1 < n ? own : nullptr, p.dk, p.dv, c_wave, lane);
        store_state<KB>(S, own, p.dk, p.dv, c_wave, p.dv % 4 == 0, lane);
        if (k + 1 == n) return;
        u32x4 sp[KB][WP];
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) pair_parts<WP>(S[2 * kb], S[2 * kb + 1], sp[kb]);
#pragma unroll
        for (int m = 0; m < 2 * KB; ++m) {
            uint16_t* const W = Ws[m & 1];
            float (&x)[VPT] = ahead[m % AHEAD];
#pragma unroll
            for (int e = 0; e < VPT; e += 2) {
                uint32_t w[WP];
                split<WP>(x[e], x[e + 1], w);
#pragma unroll
                for (int c = 0; c < WP; ++c) *reinterpret_cast<uint32_t*>(W + c * 16 * KD + to + e) = w[c];
            }
            ask(k + (m + AHEAD) / (2 * KB), (m + AHEAD) % (2 * KB), x);
            lds_barrier();      // the tile is there, and the one before has been read
            f32x4 c[2] = {N[m], {0.0f, 0.0f, 0.0f, 0.0f}};
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) {
                u32x4 a[WP];
#pragma unroll
                for (int i = 0; i < WP; ++i) a[i] = row_op<KD>(W + i * 16 * KD, 0, kb, b);
                c[kb & 1] = mma_parts<WP, WP>(a, sp[kb], c[kb & 1]);
            }
            S[m] = c[0] + c[1];
        }
    }
}

// The heads of p and, of the gradients, those of r behind them.
template <int KD, bool GRADS>
__global__ void __launch_bounds__(carry_threads(KD)) delta_carry_kernel(DeltaPass p, DeltaPass r) {
    __shared__ __align__(16) uint16_t Ws[2][3 * 16 * KD];
    const int h = blockIdx.y;
    if (!GRADS || h < p.H) carry_walk<KD, false>(p, h, Ws);
    else carry_walk<KD, true>(r, h - p.H, Ws);
}

// ---------------------------------------------------------------- single tokens
struct StepArgs {
    const void* q;
    const void* k;
    const void* v;
    const float* g;
    const float* beta;
    const int32_t* slots;
    float* states;
    void* o;
    int64_t sq, sk, sv, so, sg;
    int32_t H, rep, dk, dv, nslots, nslices, tpr_log2;
    float scale;
};

// One workgroup per sequence, head and slice of up to 64 of the state's columns, which it holds
// in registers: R rows of 4 columns a thread, all asked for at once.  What the old state holds
// under k and under q is summed over the rows in one pass and one exchange, and the output is
// (S'^T q + (k . q) u) scale, so the state is read once and written once.  Bound by those bytes:
// 256 sequences of 32 heads of 128 x 128 in 198 us on the card, 5.4 TB/s; one sequence of 32 heads
// of 128 x 128 in 6.0, the latency of one round of loads and, with slices of 16 columns, of sixteen
// threads that add up 64 rows.
template <typename IO, int R>
__global__ void __launch_bounds__(kThreads) delta_step_kernel(StepArgs p) {
    constexpr int VW = 4;
    __shared__ float sq[SSM_LINATTN_MAX_DIM], sk[SSM_LINATTN_MAX_DIM];
    __shared__ __align__(16) float red[2][kThreads * VW];
    __shared__ __align__(16) float us[kCols];
    __shared__ float kq[kWaves];
    __shared__ int dups[kWaves];
    const int tid = threadIdx.x;
    const int per = p.H * p.nslices;
    const int b = blockIdx.x / per, at = blockIdx.x % per, h = at / p.nslices, slice = at % p.nslices;
    int slot = b;
    bool dup = false;
    if (p.slots) {
        slot = p.slots[b];
        if (slot < 0 || slot >= p.nslots) return;
        for (int i = tid; i < b; i += kThreads) dup = dup || p.slots[i] == slot;
    }
    const int tpr = 1 << p.tpr_log2, rows = kThreads >> p.tpr_log2;
    const int r0 = tid >> p.tpr_log2, c0 = VW * (tid & (tpr - 1)), w = VW * tpr, col = slice * w + c0;
    const bool on = col < p.dv, whole = col + VW <= p.dv;
    float* S = p.states + (int64_t(slot) * p.H + h) * p.dk * p.dv + col;
    f32x4 s[R];
#pragma unroll
    for (int n = 0; n < R; ++n) {
        const int r = r0 + n * rows;
        s[n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        if (on && r < p.dk) {
            if (whole) {
                __builtin_memcpy(&s[n], S + int64_t(r) * p.dv, sizeof(s[n]));
            } else {
#pragma unroll
                for (int e = 0; e < VW; ++e)
                    if (col + e < p.dv) s[n][e] = S[int64_t(r) * p.dv + e];
            }
        }
    }
    const IO* q = static_cast<const IO*>(p.q) + b * p.sq + int64_t(h / p.rep) * p.dk;
    const IO* k = static_cast<const IO*>(p.k) + b * p.sk + int64_t(h / p.rep) * p.dk;
    float both = 0.0f;
    {
        const float x = tid < p.dk ? IOT<IO>::to_f32(q[tid]) : 0.0f, y = tid < p.dk ? IOT<IO>::to_f32(k[tid]) : 0.0f;
        sq[tid] = x;
        sk[tid] = y;
        both = x * y;
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) both += __shfl_xor(both, d);
    if ((tid & 63) == 0) kq[tid >> 6] = both;
    if (p.slots) {
        const bool any = __ballot(dup) != 0;
        if ((tid & 63) == 0) dups[tid >> 6] = any;
    }
    float g = p.g[b * p.sg + h];
    g = g < kMinDecay ? kMinDecay : g;
    const float a = __builtin_amdgcn_exp2f(g * kLog2e), beta = p.beta[int64_t(b) * p.H + h];
    float v = 0.0f;
    if (tid < w && slice * w + tid < p.dv) v = IOT<IO>::to_f32(static_cast<const IO*>(p.v)[b * p.sv + int64_t(h) * p.dv + slice * w + tid]);
    __syncthreads();
    if (p.slots && (dups[0] | dups[1] | dups[2] | dups[3])) return;
    f32x4 xk = {0.0f, 0.0f, 0.0f, 0.0f}, xq = xk;
#pragma unroll
    for (int n = 0; n < R; ++n) {
        const int r = r0 + n * rows;
        if (r < p.dk) {
            xk += sk[r] * s[n];
            xq += sq[r] * s[n];
        }
    }
    *reinterpret_cast<f32x4*>(&red[0][tid * VW]) = xk;
    *reinterpret_cast<f32x4*>(&red[1][tid * VW]) = xq;
    __syncthreads();
    if (tid < w) {
        float y = 0.0f, z = 0.0f;
        for (int r = 0; r < rows; ++r) {
            y += red[0][r * w + tid];
            z += red[1][r * w + tid];
        }
        const float u = beta * fmaf(-a, y, v);
        us[tid] = u;
        const int cc = slice * w + tid;
        if (cc < p.dv)
            static_cast<IO*>(p.o)[b * p.so + int64_t(h) * p.dv + cc] =
                IOT<IO>::from_f32(p.scale * fmaf((kq[0] + kq[1]) + (kq[2] + kq[3]), u, a * z));
    }
    __syncthreads();
    const f32x4 u = *reinterpret_cast<const f32x4*>(&us[c0]);
#pragma unroll
    for (int n = 0; n < R; ++n) {
        const int r = r0 + n * rows;
        if (!(on && r < p.dk)) continue;
        const f32x4 x = a * s[n] + sk[r] * u;
        if (whole) {
            __builtin_memcpy(S + int64_t(r) * p.dv, &x, sizeof(x));
        } else {
#pragma unroll
            for (int e = 0; e < VW; ++e)
                if (col + e < p.dv) S[int64_t(r) * p.dv + e] = x[e];
        }
    }
}

// ---------------------------------------------------------------- host: plans
struct Plan : Cut {
    int64_t nchunks;
    size_t tri, steps, carry, trans;   // bytes
    size_t bytes() const { return tri + steps + carry + trans; }
};

inline int make_plan(const ssm_linattn_dims* d, bool packed, Plan* pl) {
    const int64_t vs = cdiv(d->dv, kCols), ks = cdiv(d->dk, kCols);
    pl->nchunks = count_chunks(d, packed, kChunk);
    if (!cut_sequences(d, packed, choose_piece(d, packed, 2, 1), vs, vs + ks, pl) || pl->nchunks > 2 * kMostGroups) return SSM_ERR_DIMS;
    pl->tri = up256(static_cast<size_t>(pl->nchunks * d->nheads * tri_elems<kChunk>()) * 2);
    pl->steps = static_cast<size_t>(pl->nchunks * d->nheads) * sizeof(Steps<kChunk>);
    pl->carry = pl->pieced ? up256(static_cast<size_t>(pl->npieces * d->nheads * d->dk * d->dv) * 4) : 0;
    pl->trans = pl->pieced ? up256(static_cast<size_t>(pl->npieces * d->nheads * d->dk * d->dk) * 4) : 0;
    return SSM_OK;
}

template <int C> void run_tri(const DeltaPass& p, bool f32, int64_t nchunks, hipStream_t s) {
    const dim3 grid(static_cast<uint32_t>(nchunks), p.H), block(kThreads);
#define SSM_TRI(K)                                                                                                \
    do {                                                                                                          \
        if constexpr (C == 32) {                                                                                  \
            if (f32) launch_kernel(delta_tri_kernel<3, K, C>, grid, block, 0, s, p);                              \
            else launch_kernel(delta_tri_kernel<1, K, C>, grid, block, 0, s, p);                                  \
        } else {                                                                                                  \
            launch_kernel(delta_tri_kernel<1, K, C>, grid, block, 0, s, p);                                       \
        }                                                                                                         \
    } while (0)
    if (p.dk <= 64) SSM_TRI(64);
    else if (p.dk <= 128) SSM_TRI(128);
    else SSM_TRI(256);
#undef SSM_TRI
}

template <int MODE> void run_pass(const DeltaPass& p, bool f32, hipStream_t s) {
    const int64_t slices = MODE == kDeltaStates ? p.vslices + p.kslices : p.vslices;
    const dim3 grid(static_cast<uint32_t>(int64_t(p.npieces) * p.H * slices)), block(kThreads);
#define SSM_PASS(K)                                                                                 \
    do {                                                                                            \
        if (f32) launch_kernel(delta_pass_kernel<3, K, MODE>, grid, block, 0, s, p);                \
        else launch_kernel(delta_pass_kernel<1, K, MODE>, grid, block, 0, s, p);                    \
    } while (0)
    if (p.dk <= 64) SSM_PASS(64);
    else if (p.dk <= 128) SSM_PASS(128);
    else SSM_PASS(256);
#undef SSM_PASS
}

}  // namespace dl
}  // namespace

void ssm_detail::launch_delta_tri(const DeltaPass& p, bool f32, int64_t nchunks, hipStream_t s) {
    if (p.block == 64) dl::run_tri<64>(p, f32, nchunks, s);
    else dl::run_tri<32>(p, f32, nchunks, s);
}

void ssm_detail::launch_delta_carry(const DeltaPass& p, const DeltaPass* r, hipStream_t s) {
#define SSM_CARRY(K)                                                                        \
    do {                                                                                    \
        const dim3 block(dl::carry_threads(K)),                                             \
            grid(static_cast<uint32_t>(cdiv(p.dv, block.x / 4)), r ? 2 * p.H : p.H, p.nseq); \
        if (r) launch_kernel(dl::delta_carry_kernel<K, true>, grid, block, 0, s, p, *r);    \
        else launch_kernel(dl::delta_carry_kernel<K, false>, grid, block, 0, s, p, p);      \
    } while (0)
    if (p.dk <= 64) SSM_CARRY(64);
    else if (p.dk <= 128) SSM_CARRY(128);
    else SSM_CARRY(256);
#undef SSM_CARRY
}

extern "C" {

size_t ssm_delta_fwd_workspace_bytes(const ssm_linattn_dims* dims) {
    la::Sizes z;
    dl::Plan pl;
    if (la::check_dims(dims, &z) != SSM_OK) return 0;
    // with and without cu_seqlens: the larger of the two
    size_t n = 0;
    if (dl::make_plan(dims, true, &pl) == SSM_OK) n = pl.bytes();
    if (dims->tokens % dims->nseq == 0 && dl::make_plan(dims, false, &pl) == SSM_OK && pl.bytes() > n) n = pl.bytes();
    return n;
}

int ssm_delta_fwd(const void* q, const void* k, const void* v, const float* g, const float* beta,
                  const int32_t* cu_seqlens, const int32_t* slots, const float* s0, void* o, float* s_last,
                  const ssm_linattn_dims* dims, void* stream) {
    using namespace dl;
    if (!dims || !q || !k || !v || !g || !beta || !o) return SSM_ERR_NULL;
    if (slots && !s0 && !s_last) return SSM_ERR_NULL;
    Sizes z;
    int st = check_dims(dims, &z);
    if (st != SSM_OK) return st;
    const ssm_linattn_dims& d = *dims;
    if (!cu_seqlens && d.tokens % d.nseq != 0) return SSM_ERR_DIMS;
    const bool states = s0 || s_last;
    const int64_t lim = int64_t(1) << 40;
    if (states && (d.nslots < 1 || d.nslots > (int64_t(1) << 31) - 1 || (!slots && d.nslots < d.nseq) ||
                   d.nslots > lim / (d.nheads * d.dk * d.dv)))
        return SSM_ERR_DIMS;
    if (misaligned(q, z.e) || misaligned(k, z.e) || misaligned(v, z.e) || misaligned(o, z.e) || misaligned(g, 4) ||
        misaligned(beta, 4) || misaligned(cu_seqlens, 4) || misaligned(slots, 4) || misaligned(s0, 4) || misaligned(s_last, 4))
        return SSM_ERR_ALIGN;
    Plan pl;
    st = make_plan(dims, cu_seqlens != nullptr, &pl);
    if (st != SSM_OK) return st;
    const size_t need = pl.bytes();
    if (!d.workspace || d.workspace_bytes < need || misaligned(d.workspace, 256)) return SSM_ERR_WORKSPACE;
    const size_t nstate = states ? static_cast<size_t>(d.nslots * d.nheads * d.dk * d.dv) * 4 : 0;
    const int64_t wk = d.kheads * d.dk, wv = d.nheads * d.dv;
    const Area in[] = {rows_of(q, d.tokens, z.q, wk, z.e), rows_of(k, d.tokens, z.k, wk, z.e),
                       rows_of(v, d.tokens, z.v, wv, z.e),
                       flat(g, static_cast<size_t>(d.nheads * (d.head_decay ? 1 : d.tokens)) * 4),
                       flat(beta, static_cast<size_t>(d.nheads * d.tokens) * 4),
                       flat(cu_seqlens, static_cast<size_t>(d.nseq + 1) * 4), flat(slots, static_cast<size_t>(d.nseq) * 4),
                       flat(s0 == s_last ? nullptr : s0, nstate)};
    const Area out[] = {rows_of(o, d.tokens, z.o, wv, z.e), flat(s_last, nstate), flat(d.workspace, need)};
    if (clash(in, out)) return SSM_ERR_ALIAS;

    DeltaPass p = {};
    p.q = q; p.k = k; p.v = v; p.out = o; p.g = g; p.beta = beta; p.cu = cu_seqlens; p.slots = slots;
    p.s_in = s0; p.s_out = s_last;
    p.sq = z.q; p.sk = z.k; p.sv = z.v; p.so = z.o; p.sg = d.head_decay ? 0 : d.nheads;
    p.T = d.tokens; p.L = cu_seqlens ? 0 : d.tokens / d.nseq;
    p.piece = pl.piece; p.block = kChunk;
    p.rep = static_cast<int32_t>(d.nheads / d.kheads); p.H = static_cast<int32_t>(d.nheads);
    p.dk = static_cast<int32_t>(d.dk); p.dv = static_cast<int32_t>(d.dv);
    p.vslices = static_cast<int32_t>(cdiv(d.dv, kCols)); p.kslices = static_cast<int32_t>(cdiv(d.dk, kCols));
    p.nseq = static_cast<int32_t>(d.nseq); p.nslots = static_cast<int32_t>(states ? d.nslots : d.nseq);
    p.npieces = static_cast<int32_t>(pl.npieces); p.pieced = pl.pieced;
    p.wide = wide_rows(q, z.q, d.dk, z.e) && wide_rows(k, z.k, d.dk, z.e) && wide_rows(v, z.v, d.dv, z.e);
    p.pairs = pair_rows(o, z.o, d.dv);
    p.scale = d.scale;
    char* ws = static_cast<char*>(d.workspace);
    p.tri = reinterpret_cast<uint16_t*>(ws);
    p.steps = reinterpret_cast<float*>(ws + pl.tri);
    p.carry = reinterpret_cast<float*>(ws + pl.tri + pl.steps);
    p.trans = reinterpret_cast<float*>(ws + pl.tri + pl.steps + pl.carry);
    const bool f32 = d.io_dtype == SSM_F32;
    hipStream_t s = static_cast<hipStream_t>(stream);
    launch_error = hipSuccess;
    launch_delta_tri(p, f32, pl.nchunks, s);
    if (pl.pieced) {
        run_pass<kDeltaStates>(p, f32, s);
        launch_delta_carry(p, nullptr, s);
    }
    run_pass<kDeltaFull>(p, f32, s);
    return launch_error == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

int ssm_delta_step(const void* q, const void* k, const void* v, const float* g, const float* beta, const int32_t* slots,
                   float* states, void* o, const ssm_linattn_dims* dims, void* stream) {
    using namespace dl;
    if (!dims || !q || !k || !v || !g || !beta || !states || !o) return SSM_ERR_NULL;
    Sizes z;
    const int st = check_dims(dims, &z);
    if (st != SSM_OK) return st;
    const ssm_linattn_dims& d = *dims;
    if (d.tokens != d.nseq) return SSM_ERR_DIMS;
    if (d.nslots < 1 || d.nslots > (int64_t(1) << 31) - 1 || (!slots && d.nslots < d.nseq) ||
        d.nslots > (int64_t(1) << 40) / (d.nheads * d.dk * d.dv))
        return SSM_ERR_DIMS;
    if (misaligned(q, z.e) || misaligned(k, z.e) || misaligned(v, z.e) || misaligned(o, z.e) || misaligned(g, 4) ||
        misaligned(beta, 4) || misaligned(slots, 4) || misaligned(states, 4))
        return SSM_ERR_ALIGN;
    const size_t nstate = static_cast<size_t>(d.nslots * d.nheads * d.dk * d.dv) * 4;
    const int64_t wk = d.kheads * d.dk, wv = d.nheads * d.dv;
    const Area in[] = {rows_of(q, d.tokens, z.q, wk, z.e), rows_of(k, d.tokens, z.k, wk, z.e),
                       rows_of(v, d.tokens, z.v, wv, z.e),
                       flat(g, static_cast<size_t>(d.nheads * (d.head_decay ? 1 : d.tokens)) * 4),
                       flat(beta, static_cast<size_t>(d.nheads * d.tokens) * 4), flat(slots, static_cast<size_t>(d.nseq) * 4)};
    const Area out[] = {rows_of(o, d.tokens, z.o, wv, z.e), flat(states, nstate)};
    if (clash(in, out)) return SSM_ERR_ALIAS;

    StepArgs a = {};
    a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta; a.slots = slots; a.states = states; a.o = o;
    a.sq = z.q; a.sk = z.k; a.sv = z.v; a.so = z.o; a.sg = d.head_decay ? 0 : d.nheads;
    a.H = static_cast<int32_t>(d.nheads); a.rep = static_cast<int32_t>(d.nheads / d.kheads);
    a.dk = static_cast<int32_t>(d.dk); a.dv = static_cast<int32_t>(d.dv); a.nslots = static_cast<int32_t>(d.nslots);
    a.scale = d.scale;
    // up to 64 columns a workgroup, halved while the card has room for more workgroups and a row
    // of the slice is still 64 bytes
    int lg = 0;
    while ((4 << lg) < d.dv && lg < 4) ++lg;
    while ((4 << lg) > 16 && cdiv(d.dv, 4 << lg) * d.nheads * d.nseq < 512) --lg;
    a.tpr_log2 = lg;
    a.nslices = static_cast<int32_t>(cdiv(d.dv, 4 << lg));
    const int64_t blocks = d.nseq * d.nheads * a.nslices;
    if (blocks > 2 * kMostGroups) return SSM_ERR_DIMS;
    const dim3 grid(static_cast<uint32_t>(blocks)), block(kThreads);
    const int rows = static_cast<int>(cdiv(d.dk, kThreads >> lg));   // of a thread: 16 at most
    hipStream_t s = static_cast<hipStream_t>(stream);
    launch_error = hipSuccess;
#define SSM_STEP(R)                                                                                  \
    do {                                                                                             \
        if (d.io_dtype == SSM_BF16) launch_kernel(delta_step_kernel<uint16_t, R>, grid, block, 0, s, a); \
        else launch_kernel(delta_step_kernel<float, R>, grid, block, 0, s, a);                       \
    } while (0)
    if (rows <= 4) SSM_STEP(4);
    else if (rows <= 8) SSM_STEP(8);
    else SSM_STEP(16);
#undef SSM_STEP
    return launch_error == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

}  // extern "C"
