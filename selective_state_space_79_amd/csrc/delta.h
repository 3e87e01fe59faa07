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

#include <cmath>
#include <type_traits>

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
    uint16_t* tri;            // [blocks][H][3 parts][tiles' pairs of 16 x 32]: A
    float* steps;             // [chunks][H]: decays and steps of a walk's chunk (Steps<32>)
    float* keep;              // [blocks][H][dk][dv]: the state each block starts from (reverse: its gradient behind)
    float* rows;              // [T][H][dv]: U (reverse: Z), with keep
    void* dv_out;             // the gradient of v (with keep, against time)
    float* carry;             // [pieces][H][dk][dv]: the pieces' own end states, then their starting states
    float* trans;             // [pieces][H][dk][dk]: what a piece makes of the state it starts from
    float* trans_t;           // the same transposed, nullable
    int64_t sq, sk, sv, so, sg;   // elements between tokens
    int64_t T, L;
    int64_t piece;            // tokens of a piece (a multiple of the chunk)
    int32_t rep, H, dk, dv;
    int32_t block;            // tokens of A, keep: a chunk (32), or two of them
    int32_t vslices, kslices; // of 64 columns of v, and of the transition
    int32_t nseq, nslots, npieces, pieced;
    int32_t wide, pairs;
    float scale;
    float least;              // the least size of a step that the gradients count with
};

// kDeltaStates: the pieces' own end states and transitions; kDeltaFull: the outputs;
// kDeltaKeep: the state at each block's start and U (reverse: its gradient at the block's end, and Z).
enum DeltaMode { kDeltaStates = 0, kDeltaFull = 1, kDeltaKeep = 2 };
void launch_delta_tri(const DeltaPass& p, bool f32, int64_t nchunks, hipStream_t s);
void launch_delta_carry(const DeltaPass& p, const DeltaPass* r, hipStream_t s);   // r: the walk against time

}  // namespace ssm_detail

namespace {
namespace dl {

using namespace la;
using ssm_detail::DeltaPass;

constexpr int kCols = 64;   // columns of the state a workgroup: four waves of 16
constexpr int kChunk = 32;  // tokens of a walk's chunk

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
    float given[C];        // beta as it came
    float tail[C];         // e^{G_C}
};
// One wave: lane r brings row r's log decay and beta.  The sums run in float64, so that a
// difference of two of them is right to float32 of the difference, however far they fell.
// Returns the sums up to each row, in log2 units.
__device__ inline double sum_decays(float g, bool on) {
    g = g < kMinDecay ? kMinDecay : g;
    return scan_f64(on ? double(g) * 1.4426950408889634 : 0.0);
}
// Row r's values from the sums up to it and up to the chunk's end; zero steps count as `least`.
template <int C> __device__ inline void put_steps(Steps<C>& d, double s, double end, float beta, float least, int r) {
    const float hi = float(s), e = exp2_of(s);
    const float b = fabsf(beta) < least ? copysignf(least, beta) : beta;
    d.hi[r] = hi;
    d.lo[r] = float(s - double(hi));
    d.in[r] = e;
    d.out[r] = exp2_of(end - s);
    d.beta[r] = b;
    d.bin[r] = b * e;
    d.given[r] = beta;
    d.tail[r] = exp2_of(end);
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
// + 7 are rows 4g .. + 3 of the two tiles.  Output rows in paired order.
__device__ inline uint32_t tri_t_base(int lane) {
    const int g = lane >> 4;
    return 2 * ((4 * g + ((lane >> 2) & 3)) * 32 + 8 * ((lane & 3) ^ g));
}
__device__ inline u32x4 tri_t_op(const uint16_t* t, int half, uint32_t base) {
    const char* const at = reinterpret_cast<const char*>(t) + base + 8 * half;
    const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)at);
    const s16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(at + 1024));
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

// c[t] += a[t] b for N tiles, part by part over all of them: products that wait for one another
// lie N apart.
template <int N, int NA, int NB>
__device__ inline void mma_tiles(const u32x4 (&a)[N][NA], const u32x4 (&b)[NB], f32x4* c) {
    constexpr int most = (NA > NB ? NA : NB) - 1;
#pragma unroll
    for (int i = 0; i < NA; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j)
            if (i + j <= most) {
#pragma unroll
                for (int t = 0; t < N; ++t) c[t] = mma(a[t][i], b[j], c[t]);
            }
}

// Four values each of the four lanes of a quad, transposed: lane b gets value b of each.
__device__ inline f32x4 quad_transpose(const f32x4& x, int lane) {
    const auto swap = [](float v, auto ctrl) {
        return __uint_as_float(__builtin_amdgcn_update_dpp(0u, __float_as_uint(v), decltype(ctrl)::value, 0xf, 0xf, true));
    };
    using One = std::integral_constant<int, 0xB1>;   // lane ^ 1
    using Two = std::integral_constant<int, 0x4E>;   // lane ^ 2
    const bool o1 = lane & 1, o2 = lane & 2;
    f32x4 y, z;
#pragma unroll
    for (int h = 0; h < 4; h += 2) {
        const float give = swap(o1 ? x[h] : x[h + 1], One{});
        y[h] = o1 ? give : x[h];
        y[h + 1] = o1 ? x[h + 1] : give;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const float give = swap(o2 ? y[h] : y[h + 2], Two{});
        z[h] = o2 ? give : y[h];
        z[h + 2] = o2 ? y[h + 2] : give;
    }
    return z;
}

// A wave's 16 columns from c_wave on of a state (null: zeros), in the layout of a product's tiles.
template <int KB> __device__ inline void load_state(f32x4 (&S)[2 * KB], const float* at, int dk, int dv, int c_wave, int lane) {
    const int g4 = lane >> 4, col = c_wave + (lane & 15);
    const Rsrc ro = __builtin_amdgcn_make_buffer_rsrc(const_cast<float*>(at), 0, at ? dk * dv * 4 : 0, 0x00020000);
    const uint32_t o0 = (col < dv ? uint32_t(4 * col) : kPast) + uint32_t(32 * g4 * dv);
#pragma unroll
    for (int m = 0; m < 2 * KB; ++m)
#pragma unroll
        for (int r = 0; r < 4; ++r)
            S[m][r] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(
                ro, o0 + uint32_t(4 * (32 * (m >> 1) + 4 * (m & 1) + r) * dv), 0, 0));
}

// Writes a wave's 16 columns from c_wave on of a state.  Through a window on the whole state, so
// that rows and columns it does not have are dropped and every wave has as many stores under way.
// With `vec` (dv in whole fours) four lanes swap rows for columns: a quarter of the stores.
template <int KB>
__device__ inline void store_state(const f32x4 (&S)[2 * KB], float* at, int dk, int dv, int c_wave, bool vec, int lane) {
    const int g4 = lane >> 4, l16 = lane & 15;
    const Rsrc ro = __builtin_amdgcn_make_buffer_rsrc(at, 0, dk * dv * 4, 0x00020000);
    if (vec) {
        const int col = c_wave + (l16 & ~3);
        const uint32_t o0 = (col < dv ? uint32_t(4 * col) : kPast) + uint32_t(4 * (8 * g4 + (l16 & 3)) * dv);
#pragma unroll
        for (int m = 0; m < 2 * KB; ++m)
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, quad_transpose(S[m], lane)), ro,
                                                   o0 + uint32_t(4 * (32 * (m >> 1) + 4 * (m & 1)) * dv), 0, 0);
    } else {
        const int col = c_wave + l16;
        const uint32_t o0 = (col < dv ? uint32_t(4 * col) : kPast) + uint32_t(32 * g4 * dv);
#pragma unroll
        for (int m = 0; m < 2 * KB; ++m)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(S[m][r]), ro,
                                                      o0 + uint32_t(4 * (32 * (m >> 1) + 4 * (m & 1) + r) * dv), 0, 0);
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

// Where a workgroup's piece lies (its number: `unit`), or that it has none.
struct Where {
    int64_t pi, lo, hi;
    Seq sq;
    int slice, h, seq, slot;
    bool first, last, on;
};
template <typename P> __device__ inline Where find_piece(const P& p, uint32_t unit, int nslices, bool need_slot) {
    Where w;
    w.on = false;
    const int per = p.H * nslices;
    int at = int(unit % per);
    if (per % 8 == 0) at = (at % 8) * (per / 8) + at / 8;   // neighbouring heads to one XCD
    w.pi = uniform(int(unit / per));
    w.slice = uniform(at % nslices);
    w.h = uniform(at / nslices);
    const int seq = w.seq = uniform(find_seq(p, w.pi));
    if (seq < 0) return w;
    w.sq = seq_range(p, seq);
    const int64_t local = uniform(w.pi - piece_base(p, seq)), len = w.sq.end - w.sq.start;
    if (local < 0 || (local > 0 && local * p.piece >= len)) return w;
    w.slot = need_slot ? uniform(find_slot(p.slots, p.nslots, seq)) : seq;
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

// P transposed, the left operand of P^T dO: tiles of 16 tokens j in paired rows, the contraction
// over all tokens i of the chunk; a tile a wave.
template <int PARTS, int KD>
__device__ inline void put_pt(const uint16_t* Q, const uint16_t* K, uint16_t* PT, const Steps<kChunk>& st, float scale, int wave,
                              int lane) {
    constexpr int KB = KD / 32, TE = kChunk * KD;
    const int g4 = lane >> 4, l16 = lane & 15, jt = wave >> 1, it = wave & 1;
    const uint32_t base = row_base<KD>(lane), bpair = pair_base<KD>(lane);
    f32x4 a = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
        u32x4 x[PARTS], y[PARTS];
#pragma unroll
        for (int i = 0; i < PARTS; ++i) {
            x[i] = row_op<KD>(Q + i * TE, 16 * it, kb, base);
            y[i] = pair_op<KD>(K + i * TE, 0, jt, kb, bpair);
        }
        a = mma_parts<PARTS, PARTS>(x, y, a);
    }
    const int j = 8 * (l16 >> 2) + 4 * jt + (l16 & 3), i0 = 16 * it + 4 * g4;
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
    uint16_t* const o = PT + jt * 512 + at_piece<32>(l16, 2 * it + (g4 >> 1)) + 4 * (g4 & 1);
#pragma unroll
    for (int k = 0; k < 3; ++k) *reinterpret_cast<uint2*>(o + k * 1024) = uint2{x[k], y[k]};
}

// Where the blocks of A and of kept states lie that a piece's chunks belong to.
struct Blocked {
    int64_t first;     // number of the piece's first block
    int two;           // 1: two chunks to a block
    template <typename P> __device__ inline Blocked(const P& p, const Where& w, int64_t lo) {
        const Chunks ch(p, p.block);
        two = p.block > kChunk;
        first = uniform(piece_base(ch, w.seq) + ((lo - w.sq.start) >> (two ? 6 : 5)));
    }
    __device__ inline int64_t block(int64_t n) const { return first + (n >> two); }
    __device__ inline bool starts(int64_t n) const { return !two || (n & 1) == 0; }
    // A of a chunk into LDS: the blocks on the diagonal of a larger matrix's inverse are the
    // inverses of its own
    __device__ inline void load(uint16_t* to, Steps<kChunk>* st, const DeltaPass& p, int64_t n, int h, int wave, int lane) const {
        constexpr int NB = tri_blocks<kChunk>();
        const int64_t all = two ? tri_elems<64>() : tri_elems<32>();
        const u32x4 w = rows_window(reinterpret_cast<const char*>(p.tri + (block(n) * p.H + h) * all), 2 * all, 1, 1);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int b = wave + 4 * i, part = b >> 1, half = b & 1;   // 3 parts of 2 blocks
            if (b >= 3 * NB) break;
            const int from = !two ? b : 6 * part + ((n & 1) ? 3 + 2 * half : half);
            load_lds16(w, lds_address(to) + 1024 * b, uint32_t(1024 * from + 16 * lane));
        }
        static_assert(sizeof(Steps<kChunk>) == 1024, "what a wave loads at once");
        if (wave == 3)
            load_lds16(rows_window(reinterpret_cast<const char*>(p.steps + (((first << two) + n) * p.H + h) * 256),
                                   1024, 1, 1), lds_address(st), 16 * lane);
    }
};

// Pieces along the tokens, the library's choice: 0 for none.  A sequence's chunks go one after the
// other, so its length is what a call takes while the card has room; in pieces it takes `turns`
// times a piece's and what a full card adds (its own states and transitions first, twice the work
// of a walk), and the joints, each the time of dk / 2 tokens (more with keys over 128, whose carry
// keeps part of its values in scratch memory).  All in tokens of a walk; `share` workgroups of a walk fill a CU.  The lengths of
// packed sequences are not known here; the longest is taken for one and a half times the mean, so one
// long sequence among many short ones stays whole unless the caller names a piece (16384 + 15 x 64 tokens
// of 8 heads of 128: 1357 us whole, 284 in pieces of 1024; gradients 2374 and 723).
//
// Measured, us in pieces and whole, heads of 128 in bf16: forward 8192 tokens of 16 heads 231 and
// 683, of 64 heads 616 and 743, of 128 heads 923 and 789 (whole is chosen), 2 x 4096 of 32 299 and
// 365, 4 x 4096 of 32 529 and 395 (whole); 1000 + 333 + 47 float32 tokens of 8 heads of 64 and 96
// 63 and 121.  Gradients: 8192 of 16 heads 641 and 1068, of 4096 and
// 32 heads 609 and 664, of 4096 and 16 heads of 256 1018 and 938 (whole).
inline int64_t choose_piece(const ssm_linattn_dims* d, bool packed, int share, int turns) {
    const double mean = double(d->tokens) / d->nseq;
    const double longest = packed && d->nseq > 1 ? 1.5 * mean : mean;
    const double load = double(d->tokens) * d->nheads * cdiv(d->dv, kCols) / kCus;   // a workgroup on each CU
    const double joint = d->dk > 128 ? d->dk * d->dk / 256.0 : 0.5 * d->dk;
    const double least = std::sqrt(0.5 * joint * longest);
    const int64_t piece = static_cast<int64_t>(std::ceil((load / share > least ? load / share : least) / 64)) * 64;
    // 128: what two more launches take
    return turns * double(piece) + 1.2 * load + joint * longest / piece + 128 < longest ? piece : 0;
}

// Workgroups of a walk's launch: 2^31 threads, where a grid has fewer than 2^32.
constexpr int64_t kMostWalks = 2 * kMostGroups;

// How the sequences are cut, and the numbers that their pieces have.
struct Cut {
    int64_t piece, npieces;
    bool pieced;
};
// Cuts as the caller asks, or into pieces of `choice` tokens (0: none).  A piece and head is `whole`
// workgroups of the largest launch where nothing is cut and `cut` where something is.  False where a
// launch would pass its limit, which the library's own pieces never do: it cuts only where sequences x
// heads x slices of v are under 320, and then makes no more than 512 pieces of a slice.
inline bool cut_sequences(const ssm_linattn_dims* d, bool packed, int64_t choice, int64_t whole, int64_t cut, Cut* c) {
    const int64_t each = packed ? d->tokens : d->tokens / d->nseq, piece = d->piece_len ? d->piece_len : choice;
    c->pieced = piece > 0 && piece < each;
    c->piece = c->pieced ? piece : (int64_t(1) << 31);
    c->npieces = !c->pieced ? d->nseq : packed ? d->tokens / piece + d->nseq : d->nseq * cdiv(each, piece);
    return c->npieces <= kMostWalks / (d->nheads * (c->pieced ? cut : whole));
}

}  // namespace dl
}  // namespace
