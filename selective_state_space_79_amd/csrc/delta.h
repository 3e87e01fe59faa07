// delta.h -- the gated delta rule, shared by the forward (delta_fwd.hip) and the gradients
// (delta_bwd.hip) of libssm.  Per head, with a state S of dk x dv values,
//
//   S'_t = e^{g_t} S_{t-1}     r_t = v_t - S'_t^T k_t     S_t = S'_t + k_t u_t^T,  u_t = beta_t r_t
//   o_t = scale S_t^T q_t
//
// With tokens in chunks of C, G the inclusive sums of g inside the chunk and
// M_ij = e^{G_i - G_j} k_i . k_j below the diagonal, the rows u of a chunk solve a triangular
// system whose matrix does not depend on the state:
//
//   (I + beta M) U = beta (V - e^G K S_in)         U = A beta X,  A = (I + beta M)^-1
//   O = scale (e^G Q S_in) + P U                    P_ij = scale e^{G_i - G_j} q_i . k_j, j <= i
//   S_out = e^{G_C} S_in + (e^{G_C - G} K)^T U
//
// A is formed for all chunks at once before the walk over them (delta_tri_kernel) and lies in
// memory as the walk's left operand, three bf16 parts of each value, which hold a float32
// whole.  Everything else of a chunk is the state's columns' own affair: a wave keeps 16
// columns of S in registers and needs nothing of the other columns.
//
// Rows of tiles.  A product leaves rows 4a + b of a tile of 16 in lane group a, register b; the
// right operand of the next one wants rows 8a + 0..7 of 32 there.  So the tiles (half 0 and 1)
// of a pair of 32 tokens hold tokens 8a + 4 half + b in row 4a + b, and a product's result is
// the next one's operand as it stands ("paired rows" below).
#pragma once

#include "linattn.h"

namespace ssm_detail {

struct DeltaPass {
    const void* q;
    const void* k;
    const void* v;            // or the gradient of o (reverse)
    void* out;
    const float* g;
    const float* beta;
    const int32_t* cu;
    const int32_t* slots;
    const float* s_in;        // user's starting states, nullable
    float* s_out;             // user's final states, nullable
    uint16_t* tri;            // [chunks][H][3 parts][blocks of 16 x 32]: A
    float* keep;              // [chunks][H][dk][dv]: the state each chunk starts from (reverse: its gradient behind)
    float* carry;             // [pieces][H][dk][dv]: the pieces' own end states, then their starting states
    float* trans;             // [pieces][H][dk][dk]: what a piece makes of the state it starts from
    float* trans_t;           // the same transposed, nullable
    int64_t sq, sk, sv, so, sg;   // elements between tokens
    int64_t T, L;
    int64_t piece;            // tokens of a piece (a multiple of the chunk)
    int32_t rep, H, dk, dv;
    int32_t vslices, kslices; // of 64 columns of v, and of the transition
    int32_t nseq, nslots, npieces, pieced;
    int32_t wide, pairs;
    float scale;
};

// kDeltaStates: the pieces' own end states and transitions; kDeltaFull: the outputs (reverse:
// the final gradients alone); kDeltaKeep: the state at each chunk's start (reverse: its gradient
// at the chunk's end).
enum DeltaMode { kDeltaStates = 0, kDeltaFull = 1, kDeltaKeep = 2 };
void launch_delta_tri(const DeltaPass& p, bool f32, int chunk, int64_t nchunks, hipStream_t s);
void launch_delta_pass(const DeltaPass& p, bool f32, int chunk, DeltaMode mode, hipStream_t s);
void launch_delta_carry(const DeltaPass& p, bool reverse, hipStream_t s);

}  // namespace ssm_detail

namespace {
namespace dl {

using namespace la;
using ssm_detail::DeltaPass;

constexpr int kCols = 64;   // columns of the state a workgroup: four waves of 16

// blocks of 16 x 32 on and below the diagonal of a chunk (p_block numbers them)
template <int C> constexpr int tri_blocks() { return C == 64 ? 6 : 2; }
template <int C> constexpr int tri_elems() { return 3 * tri_blocks<C>() * 512; }

// Chunks of the packed sequences, numbered as pieces are.
struct Chunks {
    const int32_t* cu;
    int64_t T, L, piece;
    int32_t nseq;
    template <typename P> __device__ Chunks(const P& p, int c) : cu(p.cu), T(p.T), L(p.L), piece(c), nseq(p.nseq) {}
};
inline int64_t count_chunks(const ssm_linattn_dims* d, bool packed, int c) {
    return packed ? d->tokens / c + d->nseq : d->nseq * cdiv(d->tokens / d->nseq, c);
}

// A chunk's decays and step sizes, one value a token.
template <int C> struct __align__(16) Steps {
    float hi[C], lo[C];    // G in log2 units, as two floats
    float in[C];           // e^{G_i}
    float out[C];          // e^{G_C - G_i}
    float beta[C];
    float bin[C];          // beta_i e^{G_i}
    float tail;            // e^{G_C}
};
// One wave: lane r brings row r's log decay and beta.  The sums run in float64, so that a
// difference of two of them is right to float32 of the difference, however far they fell.
template <int C> __device__ inline void put_steps(Steps<C>& d, float g, float beta, int lane) {
    g = g < kMinDecay ? kMinDecay : g;
    const double s = scan_f64(lane < C ? double(g) * 1.4426950408889634 : 0.0);
    const double end = lane_f64(s, C - 1);
    if (lane < C) {
        const float hi = float(s), e = exp2_of(s);
        d.hi[lane] = hi;
        d.lo[lane] = float(s - double(hi));
        d.in[lane] = e;
        d.out[lane] = exp2_of(end - s);
        d.beta[lane] = beta;
        d.bin[lane] = beta * e;
        if (lane == 0) d.tail = exp2_of(end);
    }
}

// Operand along the rows of a tile in paired order: lane 16g + i takes columns 32 kb + 8g ..
// + 7 of row r0 + 8 (i / 4) + 4 half + i % 4 (rows 4 further on differ in the twist's lowest bit).
template <int W> __device__ inline uint32_t pair_base(int lane) {
    return 2 * at_piece<W>(8 * ((lane >> 2) & 3) + (lane & 3), lane >> 4);
}
template <int W> __device__ inline u32x4 pair_op(const uint16_t* t, int r0, int half, int kb, uint32_t base) {
    return *reinterpret_cast<const u32x4*>(reinterpret_cast<const char*>(t) + (base ^ (64 * kb + 16 * half)) +
                                           2 * W * (r0 + 4 * half));
}

// A transposed as a left operand: its tiles hold paired rows, so the contraction's tokens 8g ..
// + 7 of a pair are rows 4g .. + 3 of the pair's two tiles.  Output rows in paired order.
__device__ inline uint32_t tri_t_base(int lane) {
    const int g = lane >> 4;
    return 2 * ((4 * g + ((lane >> 2) & 3)) * 32 + 8 * ((lane & 3) ^ g));
}
__device__ inline u32x4 tri_t_op(const uint16_t* t, int ip, int jp, int half, uint32_t base) {
    const char* const at = reinterpret_cast<const char*>(t) + base + 8 * half;
    const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(at + 1024 * p_block(2 * ip, jp)));
    const s16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(at + 1024 * p_block(2 * ip + 1, jp)));
    const uint2 u = __builtin_bit_cast(uint2, x), v = __builtin_bit_cast(uint2, y);
    return u32x4{u.x, u.y, v.x, v.y};
}

// Two tiles of a pair (tokens 8g + 4 half + r) as the right operand of a product over the
// tokens, in N bf16 parts.
template <int N> __device__ inline void pair_parts(const f32x4& a, const f32x4& b, u32x4 (&p)[N]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const f32x4& x = e < 2 ? a : b;
        uint32_t w[N];
        split<N>(x[2 * (e & 1)], x[2 * (e & 1) + 1], w);
#pragma unroll
        for (int k = 0; k < N; ++k) p[k][e] = w[k];
    }
}

// Values 2e, 2e + 1 of an operand in PARTS parts, as float32.
template <int PARTS> __device__ inline void unpack(const u32x4 (&v)[PARTS], int e, float& x, float& y) {
    x = bf_lo(v[PARTS - 1][e]);
    y = bf_hi(v[PARTS - 1][e]);
#pragma unroll
    for (int i = PARTS - 2; i >= 0; --i) {
        x += bf_lo(v[i][e]);
        y += bf_hi(v[i][e]);
    }
}

// A matrix of A's kind from memory straight into LDS, a kilobyte a wave at a time.
template <int C, int NW> __device__ inline void load_tri(const uint16_t* from, uint16_t* to, int wave, int lane) {
    constexpr int KB = tri_elems<C>() / 512;
    const u32x4 w = rows_window(reinterpret_cast<const char*>(from), 2 * tri_elems<C>(), 1, 1);
#pragma unroll
    for (int i = 0; i < (KB + NW - 1) / NW; ++i) {
        const int b = wave + NW * i;
        if (b < KB) load_lds16(w, lds_address(to) + 1024 * b, uint32_t(1024 * b + 16 * lane));
    }
}

// Rows of a chunk that a workgroup of T threads brings into a tile of W columns: straight into
// LDS (bf16), through registers (float32) or value by value (any rows).
template <int PARTS, int C, int W, int T> struct Rows {
    Tile<PARTS, C, W, T> t;
    const char* base;
    int64_t pitch;
    int w;
    __device__ inline void prepare(const void* p, int64_t first, int64_t stride, int width, int tid) {
        constexpr int E = PARTS == 1 ? 2 : 4;
        base = static_cast<const char*>(p) + first * E;
        pitch = stride * E;
        w = width;
        t.prepare(tid, pitch, false, width);
    }
    __device__ inline void load(uint16_t* to, int wave, int64_t c0, int64_t hi) { t.load(to, wave, base + c0 * pitch, pitch, hi - c0); }
    __device__ inline void store(uint16_t* to, int tid) const { t.store(to, tid); }
    __device__ inline void copy(uint16_t* to, int tid, int64_t c0, int64_t hi) const {
        Tile<PARTS, C, W, T>::copy_any(to, tid, base + c0 * pitch, pitch, hi - c0, false, w);
    }
};

// Where a workgroup's piece lies, or that it has none.
struct Where {
    int64_t pi, lo, hi;
    Seq sq;
    int slice, h, seq, slot;
    bool first, last, on;
};
template <typename P> __device__ inline Where find_piece(const P& p, int nslices, bool need_slot) {
    Where w;
    w.on = false;
    const int per = p.H * nslices;
    int at = int(blockIdx.x % per);
    if (per % 8 == 0) at = (at % 8) * (per / 8) + at / 8;   // neighbouring heads to one XCD
    w.pi = blockIdx.x / per;
    w.slice = uniform(at % nslices);
    w.h = uniform(at / nslices);
    const int seq = w.seq = find_seq(p, w.pi);
    if (seq < 0) return w;
    w.sq = seq_range(p, seq);
    const int64_t local = w.pi - piece_base(p, seq), len = w.sq.end - w.sq.start;
    if (local < 0 || (local > 0 && local * p.piece >= len)) return w;
    w.slot = need_slot ? find_slot(p.slots, p.nslots, seq) : seq;
    if (w.slot < 0) return w;
    w.lo = w.sq.start + local * p.piece;
    w.hi = w.sq.end - w.lo > p.piece ? w.lo + p.piece : w.sq.end;
    w.first = local == 0;
    w.last = w.hi == w.sq.end;
    w.on = true;
    return w;
}

// Stores a wave's tiles of a chunk, 16 columns from c_wave on of rows of `width`: in order of the
// tokens, or as paired rows.  Rows behind the window and columns behind the row's are not written.
template <int C, bool PAIRED>
__device__ inline void store_tiles(const f32x4 (&o)[C / 16], char* row0, int64_t pitch, int64_t rows, int c_wave, int width,
                                   bool f32, bool pairs, int lane) {
    const int g4 = lane >> 4, l16 = lane & 15;
    const Rsrc ro = rows_rsrc(row0, pitch, rows, C);
    const StoreRows to(pitch, false, C, PAIRED ? 2 * g4 : g4);
    const auto row = [&](int i, int r) { return to.row((PAIRED ? 32 * (i >> 1) + 4 * (i & 1) : 16 * i) + r); };
    if (f32) {
        const int col = c_wave + l16;
        const uint32_t o0 = to.first(col < width, 4 * col);
#pragma unroll
        for (int x = 0; x < C / 4; ++x)
            __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(o[x >> 2][x & 3]), ro, o0 + row(x >> 2, x & 3), 0, 0);
    } else if (pairs) {
        // neighbouring lanes swap one row for another: two columns of one row each
        const bool odd = lane & 1;
        const uint32_t pick = odd ? 0x03020706u : 0x05040100u;
        const int even = c_wave + (l16 & ~1);
        const uint32_t o0 = to.first(even < width, 2 * even) + (odd ? to.row(1) : 0u);
#pragma unroll
        for (int i = 0; i < C / 16; ++i)
#pragma unroll
            for (int r = 0; r < 4; r += 2) {
                const uint32_t own = pack2(o[i][r], o[i][r + 1]);
                __builtin_amdgcn_raw_buffer_store_b32(__builtin_amdgcn_perm(swap1(own), own, pick), ro, o0 + row(i, r), 0, 0);
            }
    } else {
        const int col = c_wave + l16;
        const uint32_t o0 = to.first(col < width, 2 * col);
#pragma unroll
        for (int x = 0; x < C / 4; ++x)
            __builtin_amdgcn_raw_buffer_store_b16(IOT<uint16_t>::from_f32(o[x >> 2][x & 3]), ro, o0 + row(x >> 2, x & 3), 0, 0);
    }
}

// P transposed, the left operand of P^T dO: tiles of 16 tokens j in paired rows, the
// contraction over the tokens i of the same or a later pair.
template <int C> __device__ constexpr int pt_block(int jt, int ip) { return C == 32 ? jt : jt < 2 ? 2 * jt + ip : 2 + jt; }
template <int PARTS, int KD, int C, int NW>
__device__ inline void put_pt(const uint16_t* Q, const uint16_t* K, uint16_t* PT, const Steps<C>& st, float scale, int wave,
                              int lane) {
    constexpr int N = C == 64 ? 12 : 4, KB = KD / 32, PB = tri_blocks<C>() * 512;
    const int g4 = lane >> 4, l16 = lane & 15;
    const uint32_t base = row_base<KD>(lane), bpair = pair_base<KD>(lane);
    for (int m = wave; m < N; m += NW) {
        const int jt = C == 32 ? m >> 1 : m < 8 ? m >> 2 : 2 + ((m - 8) >> 1), it = C == 32 ? m & 1 : m < 8 ? m & 3 : 2 + (m & 1);
        f32x4 a = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
            u32x4 x[PARTS], y[PARTS];
#pragma unroll
            for (int i = 0; i < PARTS; ++i) {
                x[i] = row_op<KD>(Q + i * C * KD, 16 * it, kb, base);
                y[i] = pair_op<KD>(K + i * C * KD, 32 * (jt >> 1), jt & 1, kb, bpair);
            }
            a = mma_parts<PARTS, PARTS>(x, y, a);
        }
        const int j = 32 * (jt >> 1) + 8 * (l16 >> 2) + 4 * (jt & 1) + (l16 & 3), i0 = 16 * it + 4 * g4;
        const float gj = st.hi[j], ej = st.lo[j];
        const f32x4 gi = *reinterpret_cast<const f32x4*>(&st.hi[i0]), ei = *reinterpret_cast<const f32x4*>(&st.lo[i0]);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const float e = __builtin_amdgcn_exp2f((gi[r] - gj) + (ei[r] - ej));
            a[r] = j <= i0 + r ? a[r] * (e * scale) : 0.0f;
        }
        uint32_t x[3], y[3];
        split<3>(a[0], a[1], x);
        split<3>(a[2], a[3], y);
        uint16_t* const o = PT + pt_block<C>(jt, it >> 1) * 512 + at_piece<32>(l16, 2 * (it & 1) + (g4 >> 1)) + 4 * (g4 & 1);
#pragma unroll
        for (int k = 0; k < 3; ++k) *reinterpret_cast<uint2*>(o + k * PB) = uint2{x[k], y[k]};
    }
}

}  // namespace dl
}  // namespace
