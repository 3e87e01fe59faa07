// linattn.h -- the chunked pass of linear attention with a decay for each head, shared by
// the forward (linattn_fwd.hip) and the gradients (linattn_bwd.hip) of libssm.
//
// One pass computes, for rows x1 (query role), x2 (key role) and x3 (value role) of one
// head, with a state R of kd x vd values,
//
//   R_t   = e^{g_t} R_{t-1} + w x2_t x3_t^T          out_t = o R_t^T x1_t
//
// in order of time or against it.  With tokens in chunks of C and G the inclusive sums of
// g inside the chunk,
//
//   out_i = o [ e^{G_i} R_in^T x1_i + sum_{j<=i} w e^{G_i-G_j} (x1_i . x2_j) x3_j ]
//   R_out = e^{G_C} R_in + sum_j w e^{G_C-G_j} x2_j x3_j^T
//
// The forward is (x1, x2, x3) = (q, k, v).  The gradients are three more of the same:
// dq = (do, v, k) in order of time, dk = (v, do, q) and dv = (k, q, do) against it, since
// with dS_t = scale q_t do_t^T + e^{g_{t+1}} dS_{t+1} the gradient of the state,
// dq_t = scale S_t do_t, dk_t = dS_t v_t and dv_t = dS_t^T k_t.
#pragma once

#include "rows.h"

namespace ssm_detail {

struct LinattnPass {
    const void* x1;
    const void* x2;
    const void* x3;
    const void* x4;           // rows dotted with the state's share of the output (row dots)
    void* out;                // I/O type, or float32 when out_f32
    const float* g;           // log decays
    const int32_t* cu;        // starts of the packed sequences; null: equal lengths
    const int32_t* slots;     // state index of each sequence; null: its own number
    const float* s_in;        // user's starting states, nullable
    float* s_out;             // user's final states, nullable
    float* carry;             // [pieces][H][kd][vd] (or transposed): the pieces' states
    float* tot;               // [pieces][H]: the pieces' decays
    float* dots;              // row dots: [slices][T][H] of x4 . (state's share)
    float* cross;             // row dots with CROSS: [slices][T][H], see linattn_bwd.hip
    int64_t s1, s2, s3, s4, so, sg;   // elements between tokens
    int64_t T, L;             // tokens; tokens of each sequence when cu is null
    int64_t piece;            // tokens of a piece (a multiple of the chunk)
    int32_t r1, r2, r3, r4;   // heads that share one head of x1, x2, x3, x4
    int32_t H, kd, vd, nslices;
    int32_t nseq, nslots, npieces, pieced;
    int32_t st_t;             // states lie (vd, kd) instead of (kd, vd)
    int32_t reverse, out_f32;
    int32_t vec;              // bit n: rows of x1.. x4 (bits 0..3) and out (bit 4) allow 16-byte access
    float wscale, oscale;
};

// The launches return false for sizes that no kernel covers (nothing launched).
enum LinattnMode { kLinStates = 0, kLinFull = 1, kLinDots = 2, kLinCross = 3 };
bool launch_linattn_pass(const LinattnPass& p, bool f32, LinattnMode mode, hipStream_t s);       // modes 0, 1
bool launch_linattn_grad_pass(const LinattnPass& p, bool f32, LinattnMode mode, hipStream_t s);  // modes 2, 3
void launch_linattn_carry(const LinattnPass& p, hipStream_t s);
// columns of the output that one workgroup computes
int linattn_slice(int64_t kd, int64_t vd);

}  // namespace ssm_detail

namespace {
namespace la {

using ssm_detail::LinattnPass;

constexpr int kThreads = 256;
constexpr int kWaves = 4;
constexpr float kMinDecay = -128.0f;   // e^-128 is zero in float32; keeps sums of -inf apart

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

__device__ inline uint32_t pack2(float a, float b) {
    const f32x2 x = {a, b};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(x, bf16x2));
}
__device__ inline float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ inline float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// x = hi + lo in two bf16 parts (hi = bf16(x), lo = bf16(x - hi)): what is left out is
// under 2^-17 of x, so products of split operands keep float32 sums to about 2^-17.
__device__ inline void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
    hi = pack2(a, b);
    lo = pack2(a - bf_lo(hi), b - bf_hi(hi));
}

__device__ inline f32x4 mma(const u32x4& a, const u32x4& b, const f32x4& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c,
                                                   0, 0, 0);
}

// ---------------------------------------------------------------- where the sequences lie
struct Seq {
    int64_t start, end;   // tokens
};

__device__ inline Seq seq_range(const LinattnPass& p, int s) {
    if (!p.cu) return {int64_t(s) * p.L, int64_t(s + 1) * p.L};
    int64_t a = p.cu[s], b = p.cu[s + 1];
    a = a < 0 ? 0 : (a > p.T ? p.T : a);
    b = b < a ? a : (b > p.T ? p.T : b);
    return {a, b};
}

// Pieces are numbered floor(start / piece) + s upwards for sequence s: the next sequence's
// first number is never below the end of this one's, because floor((start + n) / piece) + 1
// >= floor(start / piece) + ceil(n / piece).  Numbers that no piece has are skipped.
__device__ inline int64_t piece_base(const LinattnPass& p, int s) {
    if (!p.cu) return int64_t(s) * ((p.L + p.piece - 1) / p.piece);
    int64_t a = p.cu[s];
    a = a < 0 ? 0 : (a > p.T ? p.T : a);
    return a / p.piece + s;
}

// The sequence of piece number `pi`, or -1: each round of 64 lanes narrows the range 64-fold.
__device__ inline int find_seq(const LinattnPass& p, int64_t pi) {
    if (!p.cu) {
        const int s = int(pi / ((p.L + p.piece - 1) / p.piece));
        return s < p.nseq ? s : -1;
    }
    const int lane = threadIdx.x & 63;
    int lo = 0, n = p.nseq;
    for (;;) {
        const int step = (n + 63) / 64;
        const int at = lane * step;
        const bool le = at < n && piece_base(p, lo + at) <= pi;
        const int cnt = __popcll(__ballot(le));
        if (cnt == 0) return -1;
        if (step == 1) return lo + cnt - 1;
        lo += (cnt - 1) * step;
        n = n - (cnt - 1) * step < step ? n - (cnt - 1) * step : step;
    }
}

// The state index of sequence s, or -1 when its slot is out of range or an earlier
// sequence names it already (every wave of a workgroup finds the same answer).
__device__ inline int find_slot(const int32_t* slots, int nslots, int s) {
    if (!slots) return s;
    const int slot = slots[s];
    if (slot < 0 || slot >= nslots) return -1;
    const int lane = threadIdx.x & 63;
    bool dup = false;
    for (int b = lane; b < s; b += 64) dup = dup || slots[b] == slot;
    return __ballot(dup) ? -1 : slot;
}

// Element offset of piece p of 8 bf16 in row r of a tile with W columns.  The pieces of a
// row are permuted by the row so that both reads of a tile touch distinct banks: 8 rows at
// one piece (operands along a row), and 4 rows at 4 neighbouring pieces (transposed).
template <int W> __device__ inline int at_piece(int r, int p) {
    if constexpr (W >= 128)
        return r * W + 8 * (p ^ (4 * (r & 3) + ((r >> 2) & 3)));
    else if constexpr (W == 64)
        return r * W + 8 * (p ^ (4 * ((r >> 1) & 1) + ((r >> 2) & 3)));
    else
        return r * W + 8 * (p ^ ((r >> 2) & 3));
}

// Operand along the rows of a tile: lane 16g + i gets columns 32 kb + 8g .. + 7 of row r0 + i.
template <int W> __device__ inline u32x4 row_op(const uint16_t* t, int r0, int kb, int lane) {
    return *reinterpret_cast<const u32x4*>(t + at_piece<W>(r0 + (lane & 15), 4 * kb + (lane >> 4)));
}

// Transposed operand (ds_read_b64_tr_b16: of the four bf16 that lanes 4j + a of a group of
// 16 address, lane 4a + e gets element e of lane 4j + a as its element j).  Contraction
// slots 0..7 of lane 16g + i are rows r0 + 8g .. + 7; its column is
//   spread = 0: c0 + i;   spread = 1: c0 + 8 (i / 4) + i % 4.
template <int W, int SPREAD> __device__ inline u32x4 col_op(const uint16_t* t, int r0, int c0, int lane) {
    const int j = (lane >> 2) & 3, a = lane & 3;
    const int r = r0 + 8 * (lane >> 4) + j;
    const int c = c0 + (SPREAD ? 8 : 4) * a;
    const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(t + at_piece<W>(r, c >> 3) + (c & 7)));
    const s16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(t + at_piece<W>(r + 4, c >> 3) + (c & 7)));
    const uint2 u = __builtin_bit_cast(uint2, x), v = __builtin_bit_cast(uint2, y);
    return u32x4{u.x, u.y, v.x, v.y};
}

// ---------------------------------------------------------------- rows into tiles
// A tile of C rows of W columns on its way from memory to LDS in this thread's registers.
template <int PARTS, int C, int W> struct Stage {
    static constexpr int N = C * W / 8 / kThreads;   // pieces of 8 values per thread
    static_assert(C * W / 8 % kThreads == 0, "whole pieces per thread");
    u32x4 r[N][PARTS];   // 8 bf16, or 8 float32

    // rows of tokens first .. (or downwards), those in [lo, hi) only; `row` points at the
    // head's first column, w columns are real
    __device__ inline void load(const char* row, int64_t stride, int64_t c0, bool rev, int64_t lo, int64_t hi, int w,
                                bool vec) {
        constexpr int E = PARTS == 1 ? 2 : 4;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int idx = int(threadIdx.x) + kThreads * n;
            const int rr = idx / (W / 8), col = 8 * (idx % (W / 8));
            const int64_t t = c0 + (rev ? C - 1 - rr : rr);
            const bool ok = t >= lo && t < hi && col < w;
            const char* q = row + (t * stride + col) * E;
#pragma unroll
            for (int h = 0; h < PARTS; ++h) r[n][h] = u32x4{0, 0, 0, 0};
            if (ok) {
                if (vec) {
#pragma unroll
                    for (int h = 0; h < PARTS; ++h) r[n][h] = *reinterpret_cast<const u32x4*>(q + 16 * h);
                } else if constexpr (PARTS == 1) {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (col + e < w)
                            r[n][0][e / 2] |= uint32_t(reinterpret_cast<const uint16_t*>(q)[e]) << (16 * (e & 1));
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (col + e < w) r[n][e / 4][e % 4] = reinterpret_cast<const uint32_t*>(q)[e];
                }
            }
        }
    }
    __device__ inline void store(uint16_t* tile) const {
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int idx = int(threadIdx.x) + kThreads * n;
            const int o = at_piece<W>(idx / (W / 8), idx % (W / 8));
            if constexpr (PARTS == 1) {
                *reinterpret_cast<u32x4*>(tile + o) = r[n][0];
            } else {
                u32x4 hi, lo;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    uint32_t a, b;
                    const u32x4& v = r[n][e / 2];
                    split2(__uint_as_float(v[2 * (e & 1)]), __uint_as_float(v[2 * (e & 1) + 1]), a, b);
                    hi[e] = a;
                    lo[e] = b;
                }
                *reinterpret_cast<u32x4*>(tile + o) = hi;
                *reinterpret_cast<u32x4*>(tile + C * W + o) = lo;
            }
        }
    }
};

// Decays of one chunk.  The sums run in float64 and are kept in two floats, so that a
// difference of two of them is right to float32 of the difference, however far they fell.
template <int C> struct Decays {
    float hi[C], lo[C];   // G in log2 units
    float in[C];          // e^{G_i}: the incoming state's share at row i
    float out[C];         // w e^{G_C - G_j}: row j's share in the outgoing state
    float all;            // e^{G_C}
};

__device__ inline double shfl_up_f64(double v, int d) {
    return __hiloint2double(__shfl_up(__double2hiint(v), d), __shfl_up(__double2loint(v), d));
}

// One wave: lane r brings row r's log decay.  Returns the chunk's total in log2 units.
template <int C> __device__ inline double scan_decays(Decays<C>& d, float g, float wscale, int lane) {
    g = g < kMinDecay ? kMinDecay : g;
    double s = lane < C ? double(g) * 1.4426950408889634 : 0.0;
#pragma unroll
    for (int k = 1; k < C; k <<= 1) {
        const double o = shfl_up_f64(s, k);
        if (lane >= k) s += o;
    }
    const double end = __hiloint2double(__shfl(__double2hiint(s), C - 1), __shfl(__double2loint(s), C - 1));
    if (lane < C) {
        const float hi = float(s);
        d.hi[lane] = hi;
        d.lo[lane] = float(s - double(hi));
        d.in[lane] = __builtin_amdgcn_exp2f(hi);
        d.out[lane] = wscale * __builtin_amdgcn_exp2f(float(end - s));
        if (lane == C - 1) d.all = __builtin_amdgcn_exp2f(hi);
    }
    return end;
}

// ---------------------------------------------------------------- the pass
// One workgroup of four waves walks one piece of one head's sequence for 64 * NT columns
// of the output.  Each wave keeps the state's 16 * NT columns of its own in registers, in
// the layout in which the matrix unit leaves a product; the rows of a tile of 16 are
// numbered (8a + 4t + b for row 4a + b of tile t of a pair) so that a pair of tiles is the
// right operand of the read-out as it stands, with no exchange between lanes.
template <int PARTS, int KD, int NT, int C, int MODE>
__global__ void __launch_bounds__(kThreads, 2) linattn_pass_kernel(ssm_detail::LinattnPass p) {
    using namespace ssm_detail;
    constexpr bool FULL = MODE >= kLinFull, DOTS = MODE >= kLinDots, CROSS = MODE == kLinCross;
    constexpr int BV = 64 * NT, IT = C / 16, JB = C / 32, KB = KD / 32;
    __shared__ __align__(16) uint16_t X2[PARTS * C * KD];
    __shared__ __align__(16) uint16_t X3[PARTS * C * BV];
    __shared__ __align__(16) uint16_t X1[FULL ? PARTS * C * KD : 8];
    __shared__ __align__(16) uint16_t PT[FULL ? 2 * C * C : 8];   // decayed x1 . x2, two parts
    __shared__ __align__(16) uint16_t X4[DOTS ? PARTS * C * BV : 8];
    __shared__ float part[DOTS ? kWaves * C : 1];
    __shared__ float rowsum[CROSS ? kWaves * C : 1];
    __shared__ float colsum[CROSS ? kWaves * C : 1];
    __shared__ Decays<C> dec;

    const int tid = threadIdx.x, lane = tid & 63, g4 = lane >> 4, l16 = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    // neighbouring workgroups run on different XCDs: give each XCD neighbouring heads, so
    // that slices of one head and heads that share rows meet in one L2
    const int per = p.H * p.nslices;
    int at = int(blockIdx.x % per);
    if (per % 8 == 0) at = (at % 8) * (per / 8) + at / 8;
    const int64_t pi = blockIdx.x / per;
    const int h = at / p.nslices, slice = at % p.nslices;
    const int seq = find_seq(p, pi);
    if (seq < 0) return;
    const Seq sq = seq_range(p, seq);
    const int64_t local = pi - piece_base(p, seq), len = sq.end - sq.start;
    if (local < 0 || (local > 0 && local * p.piece >= len)) return;
    const int slot = find_slot(p.slots, p.nslots, seq);
    if (slot < 0) return;
    const int64_t lo = sq.start + local * p.piece;                     // this piece's tokens
    const int64_t hi = sq.end - lo > p.piece ? lo + p.piece : sq.end;
    const bool last = p.reverse ? local == 0 : hi == sq.end;
    if (!FULL && last) return;                                         // no piece starts from its state

    constexpr int E = PARTS == 1 ? 2 : 4;
    const int c_wave = slice * BV + wave * 16 * NT;                    // this wave's first column
    const char* b1 = FULL ? static_cast<const char*>(p.x1) + int64_t(h / p.r1) * p.kd * E : nullptr;
    const char* b2 = static_cast<const char*>(p.x2) + int64_t(h / p.r2) * p.kd * E;
    const char* b3 = static_cast<const char*>(p.x3) + (int64_t(h / p.r3) * p.vd + slice * BV) * E;
    const char* b4 = DOTS ? static_cast<const char*>(p.x4) + (int64_t(h / p.r4) * p.vd + slice * BV) * E : nullptr;
    const int w3 = p.vd - slice * BV;

    f32x4 S[2 * KB][NT];
    // ------------------------------------------------ starting state
    const int64_t rs = p.st_t ? 1 : p.vd, cs = p.st_t ? p.kd : 1;
    const int64_t ssz = int64_t(p.kd) * p.vd;
    const float* src = nullptr;
    if (FULL) {
        if (p.pieced)
            src = p.carry + (pi * p.H + h) * ssz;
        else if (p.s_in)
            src = p.s_in + (int64_t(slot) * p.H + h) * ssz;
    }
#pragma unroll
    for (int m = 0; m < 2 * KB; ++m)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = 32 * (m >> 1) + 8 * g4 + 4 * (m & 1) + r, col = c_wave + 16 * nt + l16;
                S[m][nt][r] = src && row < p.kd && col < p.vd ? src[row * rs + col * cs] : 0.0f;
            }

    // tiles above the diagonal that share a block of 32 with one on it stay zero
    if constexpr (FULL) {
        for (int i = tid; i < 2 * C * C / 2; i += kThreads) reinterpret_cast<uint32_t*>(PT)[i] = 0;
    }

    Stage<PARTS, C, KD> t1, t2;
    Stage<PARTS, C, BV> t3, t4;
    float gnext = 0.0f;
    double total = 0.0;
    const int64_t nch = (hi - lo + C - 1) / C;
    auto fetch = [&](int64_t n) {
        const int64_t c0 = lo + (p.reverse ? nch - 1 - n : n) * C;
        if constexpr (FULL) t1.load(b1, p.s1, c0, p.reverse, lo, hi, p.kd, p.vec & 1);
        t2.load(b2, p.s2, c0, p.reverse, lo, hi, p.kd, p.vec & 2);
        t3.load(b3, p.s3, c0, p.reverse, lo, hi, w3, p.vec & 4);
        if constexpr (DOTS) t4.load(b4, p.s4, c0, p.reverse, lo, hi, w3, p.vec & 8);
        if (wave == 0) {
            // against time the decay of a step belongs to the later of its two tokens
            const int64_t t = c0 + (p.reverse ? C - 1 - lane : lane);
            const int64_t tg = p.reverse ? t + 1 : t;
            const bool ok = lane < C && t >= lo && t < hi && tg < sq.end;
            gnext = ok ? p.g[tg * p.sg + h] : 0.0f;
        }
    };
    if (nch > 0) fetch(0);

    for (int64_t n = 0; n < nch; ++n) {
        const int64_t c0 = lo + (p.reverse ? nch - 1 - n : n) * C;
        __syncthreads();                        // the last chunk's readers are done
        if constexpr (FULL) t1.store(X1);
        t2.store(X2);
        t3.store(X3);
        if constexpr (DOTS) t4.store(X4);
        if (wave == 0) total += scan_decays<C>(dec, gnext, p.wscale, lane);
        if (n + 1 < nch) fetch(n + 1);
        __syncthreads();

        f32x4 acc[IT][NT];
        if constexpr (FULL) {
            // ---- P = x1 . x2 under the decays, tiles of 16 x 16 on and below the diagonal
            for (int m = wave; m < IT * (IT + 1) / 2; m += kWaves) {
                const int it = m < 1 ? 0 : m < 3 ? 1 : m < 6 ? 2 : 3;
                const int jt = m - it * (it + 1) / 2;
                f32x4 a = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int kb = 0; kb < KB; ++kb) {
                    const u32x4 k0 = row_op<KD>(X2, 16 * jt, kb, lane), q0 = row_op<KD>(X1, 16 * it, kb, lane);
                    a = mma(k0, q0, a);
                    if constexpr (PARTS == 2) {
                        const u32x4 k1 = row_op<KD>(X2 + C * KD, 16 * jt, kb, lane);
                        const u32x4 q1 = row_op<KD>(X1 + C * KD, 16 * it, kb, lane);
                        a = mma(k1, q0, a);
                        a = mma(k0, q1, a);
                    }
                }
                const int i = 16 * it + l16, j0 = 16 * jt + 4 * g4;
                const float gi = dec.hi[i], ei = dec.lo[i];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float w = __builtin_amdgcn_exp2f((gi - dec.hi[j0 + r]) + (ei - dec.lo[j0 + r]));
                    a[r] = j0 + r <= i ? a[r] * (w * p.wscale) : 0.0f;
                }
                uint2 hiw, low;
                split2(a[0], a[1], hiw.x, low.x);
                split2(a[2], a[3], hiw.y, low.y);
                const int o = at_piece<C>(i, j0 >> 3) + (j0 & 7);
                *reinterpret_cast<uint2*>(PT + o) = hiw;
                *reinterpret_cast<uint2*>(PT + C * C + o) = low;
                if constexpr (CROSS) {
                    // the other product of the same rows: x3 . x4, over this slice's columns
                    f32x4 b = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int kb = 0; kb < BV / 32; ++kb) {
                        const u32x4 k0 = row_op<BV>(X3, 16 * jt, kb, lane), q0 = row_op<BV>(X4, 16 * it, kb, lane);
                        b = mma(k0, q0, b);
                        if constexpr (PARTS == 2) {
                            const u32x4 k1 = row_op<BV>(X3 + C * BV, 16 * jt, kb, lane);
                            const u32x4 q1 = row_op<BV>(X4 + C * BV, 16 * it, kb, lane);
                            b = mma(k1, q0, b);
                            b = mma(k0, q1, b);
                        }
                    }
                    // sums below the diagonal, by rows and by columns of the same products
                    float row = 0.0f, csum[4];
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float x = j0 + r < i ? a[r] * b[r] : 0.0f;
                        row += x;
                        float col = x;
#pragma unroll
                        for (int d = 1; d < 16; d <<= 1) col += __shfl_xor(col, d);
                        csum[r] = col;
                    }
                    row += __shfl_xor(row, 16);
                    row += __shfl_xor(row, 32);
                    // each (tile row, tile column) is one slot: fixed order, no atomics
                    if (g4 == 0) rowsum[jt * C + i] = row;
                    if (l16 == 0) {
#pragma unroll
                        for (int r = 0; r < 4; ++r) colsum[it * C + j0 + r] = csum[r];
                    }
                }
            }
            // ---- the incoming state's share, e^{G_i} R^T x1_i
#pragma unroll
            for (int it = 0; it < IT; ++it)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) acc[it][nt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) {
                u32x4 sh[NT], sl[NT];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const f32x4& s = S[2 * kb + (e >> 1)][nt];
                        uint32_t a, b;
                        split2(s[2 * (e & 1)], s[2 * (e & 1) + 1], a, b);
                        sh[nt][e] = a;
                        sl[nt][e] = b;
                    }
#pragma unroll
                for (int it = 0; it < IT; ++it) {
                    const u32x4 q0 = row_op<KD>(X1, 16 * it, kb, lane);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        acc[it][nt] = mma(q0, sh[nt], acc[it][nt]);
                        acc[it][nt] = mma(q0, sl[nt], acc[it][nt]);
                    }
                    if constexpr (PARTS == 2) {
                        const u32x4 q1 = row_op<KD>(X1 + C * KD, 16 * it, kb, lane);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) acc[it][nt] = mma(q1, sh[nt], acc[it][nt]);
                    }
                }
            }
#pragma unroll
            for (int it = 0; it < IT; ++it) {
                const f32x4 e = *reinterpret_cast<const f32x4*>(&dec.in[16 * it + 4 * g4]);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int r = 0; r < 4; ++r) acc[it][nt][r] *= e[r];
                if constexpr (DOTS) {
                    f32x4 d = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const int col = wave * 16 * NT + 16 * nt + l16;
                            const int o = at_piece<BV>(16 * it + 4 * g4 + r, col >> 3) + (col & 7);
                            float x = __uint_as_float(uint32_t(X4[o]) << 16);
                            if constexpr (PARTS == 2) x += __uint_as_float(uint32_t(X4[C * BV + o]) << 16);
                            d[r] = fmaf(x, acc[it][nt][r], d[r]);
                        }
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        float v = d[r];
#pragma unroll
                        for (int k = 1; k < 16; k <<= 1) v += __shfl_xor(v, k);
                        if (l16 == 0) part[wave * C + 16 * it + 4 * g4 + r] = v;
                    }
                }
            }
            __syncthreads();                    // P (and the dots) are there
            if constexpr (DOTS) {
                if (tid < C) {
                    const int64_t t = c0 + (p.reverse ? C - 1 - tid : tid);
                    if (t >= lo && t < hi) {
                        float v = 0.0f;
#pragma unroll
                        for (int w = 0; w < kWaves; ++w) v += part[w * C + tid];
                        const int64_t o = (int64_t(slice) * p.T + t) * p.H + h;
                        p.dots[o] = v * p.oscale;
                        if constexpr (CROSS) {
                            const int it = tid >> 4;
                            float rsv = 0.0f, csv = 0.0f;
                            for (int m = 0; m <= it; ++m) rsv += rowsum[m * C + tid];
                            for (int m = it; m < IT; ++m) csv += colsum[m * C + tid];
                            p.cross[o] = (rsv - csv) * p.oscale;
                        }
                    }
                }
            }
        }

        // ---- the chunk's own share, P x3, and the outgoing state
        u32x4 v0[JB][NT], v1[PARTS == 2 ? JB : 1][NT];
#pragma unroll
        for (int jb = 0; jb < JB; ++jb)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                v0[jb][nt] = col_op<BV, 0>(X3, 32 * jb, wave * 16 * NT + 16 * nt, lane);
                if constexpr (PARTS == 2)
                    v1[jb][nt] = col_op<BV, 0>(X3 + C * BV, 32 * jb, wave * 16 * NT + 16 * nt, lane);
            }
        if constexpr (FULL) {
#pragma unroll
            for (int it = 0; it < IT; ++it)
#pragma unroll
                for (int jb = 0; jb <= it / 2; ++jb) {
                    const u32x4 p0 = row_op<C>(PT, 16 * it, jb, lane), p1 = row_op<C>(PT + C * C, 16 * it, jb, lane);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        acc[it][nt] = mma(p0, v0[jb][nt], acc[it][nt]);
                        acc[it][nt] = mma(p1, v0[jb][nt], acc[it][nt]);
                        if constexpr (PARTS == 2) acc[it][nt] = mma(p0, v1[jb][nt], acc[it][nt]);
                    }
                }
        }
        const float all = dec.all;
#pragma unroll
        for (int m = 0; m < 2 * KB; ++m)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int r = 0; r < 4; ++r) S[m][nt][r] *= all;
#pragma unroll
        for (int jb = 0; jb < JB; ++jb) {
            u32x4 vh[NT], vl[NT];
            const f32x4 f0 = *reinterpret_cast<const f32x4*>(&dec.out[32 * jb + 8 * g4]);
            const f32x4 f1 = *reinterpret_cast<const f32x4*>(&dec.out[32 * jb + 8 * g4 + 4]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float x = bf_lo(v0[jb][nt][e]), y = bf_hi(v0[jb][nt][e]);
                    if constexpr (PARTS == 2) {
                        x += bf_lo(v1[jb][nt][e]);
                        y += bf_hi(v1[jb][nt][e]);
                    }
                    const f32x4& f = e < 2 ? f0 : f1;
                    uint32_t a, b;
                    split2(x * f[2 * (e & 1)], y * f[2 * (e & 1) + 1], a, b);
                    vh[nt][e] = a;
                    vl[nt][e] = b;
                }
#pragma unroll
            for (int m = 0; m < 2 * KB; ++m) {
                const u32x4 k0 = col_op<KD, 1>(X2, 32 * jb, 32 * (m >> 1) + 4 * (m & 1), lane);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    S[m][nt] = mma(k0, vh[nt], S[m][nt]);
                    S[m][nt] = mma(k0, vl[nt], S[m][nt]);
                }
                if constexpr (PARTS == 2) {
                    const u32x4 k1 = col_op<KD, 1>(X2 + C * KD, 32 * jb, 32 * (m >> 1) + 4 * (m & 1), lane);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) S[m][nt] = mma(k1, vh[nt], S[m][nt]);
                }
            }
        }

        if constexpr (FULL) {
#pragma unroll
            for (int it = 0; it < IT; ++it)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int row = 16 * it + 4 * g4 + r;
                    const int64_t t = c0 + (p.reverse ? C - 1 - row : row);
                    if (t < lo || t >= hi) continue;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const int col = c_wave + 16 * nt + l16;
                        if (col >= p.vd) continue;
                        const int64_t o = t * p.so + int64_t(h) * p.vd + col;
                        const float x = acc[it][nt][r] * p.oscale;
                        if (PARTS == 2 || p.out_f32)
                            static_cast<float*>(p.out)[o] = x;
                        else
                            static_cast<uint16_t*>(p.out)[o] = IOT<uint16_t>::from_f32(x);
                    }
                }
        }
    }

    // ------------------------------------------------ the state that leaves
    float* dst = nullptr;
    float mul = 1.0f;
    if (FULL) {
        if (last && p.s_out) {
            dst = p.s_out + (int64_t(slot) * p.H + h) * ssz;
            // against time the state before the first token has that token's decay too
            if (p.reverse && sq.end > sq.start) {
                const float g = p.g[sq.start * p.sg + h];
                mul = __builtin_amdgcn_exp2f((g < kMinDecay ? kMinDecay : g) * kLog2e);
            }
        }
    } else {
        dst = p.carry + (pi * p.H + h) * ssz;
        if (wave == 0 && lane == 0 && slice == 0) p.tot[pi * p.H + h] = __builtin_amdgcn_exp2f(float(total));
    }
    if (dst) {
#pragma unroll
        for (int m = 0; m < 2 * KB; ++m)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int row = 32 * (m >> 1) + 8 * g4 + 4 * (m & 1) + r, col = c_wave + 16 * nt + l16;
                    if (row < p.kd && col < p.vd) dst[row * rs + col * cs] = mul * S[m][nt][r];
                }
    }
}

// Chooses the kernel of a pass's sizes and starts it.
template <int MODE> inline bool launch_pass(const ssm_detail::LinattnPass& p, bool f32, hipStream_t s) {
    const int64_t blocks = int64_t(p.npieces) * p.H * p.nslices;
    const dim3 grid(static_cast<uint32_t>(blocks)), block(kThreads);
    const bool two = ssm_detail::linattn_slice(p.kd, p.vd) == 128;
#define SSM_LIN_CASE(K, NTV, CF)                                                                    \
    do {                                                                                            \
        if (f32)                                                                                    \
            launch_kernel(linattn_pass_kernel<2, K, NTV, CF, MODE>, grid, block, 0, s, p);           \
        else                                                                                        \
            launch_kernel(linattn_pass_kernel<1, K, NTV, 64, MODE>, grid, block, 0, s, p);           \
    } while (0)
    if (p.kd <= 64) {
        if (two) SSM_LIN_CASE(64, 2, 64); else SSM_LIN_CASE(64, 1, 64);
    } else if (p.kd <= 128) {
        if (two) SSM_LIN_CASE(128, 2, 32); else SSM_LIN_CASE(128, 1, 32);
    } else if (p.kd <= 256) {
        SSM_LIN_CASE(256, 1, 32);
    } else {
        return false;
    }
#undef SSM_LIN_CASE
    return true;
}

// ---------------------------------------------------------------- host: checks
struct Sizes {
    int64_t q, k, v, o;   // strides
    int64_t e;            // bytes of an element
};

inline int check_dims(const ssm_linattn_dims* d, Sizes* z) {
    if (!d) return SSM_ERR_NULL;
    if (d->tokens < 1 || d->nseq < 1 || d->nheads < 1 || d->kheads < 1 || d->dk < 1 || d->dv < 1) return SSM_ERR_EMPTY;
    if (d->io_dtype != SSM_F32 && d->io_dtype != SSM_BF16) return SSM_ERR_DTYPE;
    if (d->nheads % d->kheads != 0 || d->dk > SSM_LINATTN_MAX_DIM || d->dv > SSM_LINATTN_MAX_DIM) return SSM_ERR_DIMS;
    if (d->nseq > 65535 || d->nheads > 65535 || d->tokens > (int64_t(1) << 31) - 1) return SSM_ERR_DIMS;
    if (d->head_decay != 0 && d->head_decay != 1) return SSM_ERR_DIMS;
    if (d->reserved != 0) return SSM_ERR_DIMS;
    if (d->piece_len < 0 || d->piece_len % 64 != 0 || d->piece_len > (int64_t(1) << 31)) return SSM_ERR_DIMS;
    z->q = d->q_stride ? d->q_stride : d->kheads * d->dk;
    z->k = d->k_stride ? d->k_stride : d->kheads * d->dk;
    z->v = d->v_stride ? d->v_stride : d->nheads * d->dv;
    z->o = d->o_stride ? d->o_stride : d->nheads * d->dv;
    const int64_t lim = int64_t(1) << 40;
    if (z->q < d->kheads * d->dk || z->k < d->kheads * d->dk || z->v < d->nheads * d->dv || z->o < d->nheads * d->dv)
        return SSM_ERR_DIMS;
    for (const int64_t s : {z->q, z->k, z->v, z->o})
        if (s > lim / d->tokens) return SSM_ERR_DIMS;
    z->e = d->io_dtype == SSM_BF16 ? 2 : 4;
    return SSM_OK;
}

inline size_t up256(size_t n) { return (n + 255) / 256 * 256; }

inline bool rows16(const void* q, int64_t stride, int64_t width, int64_t e) {
    return !misaligned(q, 16) && stride * e % 16 == 0 && width * e % 16 == 0 && width % 8 == 0;
}


}  // namespace la
}  // namespace
