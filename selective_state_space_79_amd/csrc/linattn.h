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
    void* out;                // I/O type, or float32 when out_f32
    const float* g;           // log decays
    const int32_t* cu;        // starts of the packed sequences; null: equal lengths
    const int32_t* slots;     // state index of each sequence; null: its own number
    const float* s_in;        // user's starting states, nullable
    float* s_out;             // user's final states, nullable
    float* carry;             // [pieces][H][kd][vd] (or transposed): the pieces' states
    float* tot;               // [pieces][H]: the pieces' decays
    int64_t s1, s2, s3, so, sg;   // elements between tokens
    int64_t T, L;             // tokens; tokens of each sequence when cu is null
    int64_t piece;            // tokens of a piece (a multiple of the chunk)
    int32_t r1, r2, r3;       // heads that share one head of x1, x2, x3
    int32_t H, kd, vd, nslices;
    int32_t nseq, nslots, npieces, pieced;
    int32_t st_t;             // states lie (vd, kd) instead of (kd, vd)
    int32_t reverse, out_f32;
    int32_t wide;             // rows of x1 .. x3 allow 16-byte loads at 32-bit offsets
    int32_t pairs;            // out allows stores of two bf16
    float wscale, oscale;
};

// Passes of one launch, over the grid's y: they differ in rows, direction and states only.
struct LinattnPasses {
    LinattnPass p[2];
};

// kLinStates: the pieces' own end states; kLinFull: the outputs.
enum LinattnMode { kLinStates = 0, kLinFull = 1 };
void launch_linattn_pass(const LinattnPasses& p, int count, bool f32, LinattnMode mode, hipStream_t s);
void launch_linattn_carry(const LinattnPasses& p, int count, hipStream_t s);
// How a pass over vd columns is cut: 128 columns of a head to a workgroup, 64, or two heads
// of up to 64 that share x1 and x2
enum LinattnShape { kWide, kNarrow, kTwoHeads };
inline LinattnShape linattn_shape(int64_t vd, bool pairs) { return vd > 64 ? kWide : pairs ? kTwoHeads : kNarrow; }
inline int linattn_slice(int64_t vd) { return vd > 64 ? 128 : 64; }

}  // namespace ssm_detail

namespace {
namespace la {

using ssm_detail::LinattnPass;

constexpr int kThreads = 256;
constexpr int kWaves = 4;
constexpr int64_t kCus = 256;
constexpr float kMinDecay = -128.0f;   // e^-128 is zero in float32; keeps sums of -inf apart
constexpr float kLn2 = 0.69314718f;

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

// Two values in N bf16 parts each (part 0 is bf16(x), the next the rounded rest, ...), packed
// in pairs.  One rounding leaves at most 2^-9 of the power of two above x, so three parts, which
// hold 24 bits, leave nothing of a float32 (two would leave up to 2^-17 of x).
template <int N> __device__ inline void split(float a, float b, uint32_t (&w)[N]) {
#pragma unroll
    for (int n = 0; n < N; ++n) {
        w[n] = pack2(a, b);
        a -= bf_lo(w[n]);
        b -= bf_hi(w[n]);
    }
}

__device__ inline f32x4 mma(const u32x4& a, const u32x4& b, const f32x4& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c,
                                                   0, 0, 0);
}

// ---------------------------------------------------------------- where the sequences lie
struct Seq {
    int64_t start, end;   // tokens
};

// A value that all lanes have, for the scalar unit: what was read through a pointer that
// stores may reach stays in vector registers else, and all that is worked out from it.
__device__ inline int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ inline int64_t uniform(int64_t v) {
    return int64_t(uint64_t(uint32_t(uniform(int(v)))) | (uint64_t(uint32_t(uniform(int(v >> 32)))) << 32));
}

template <typename P> __device__ inline Seq seq_range(const P& p, int s) {
    if (!p.cu) return {int64_t(s) * p.L, int64_t(s + 1) * p.L};
    int64_t a = uniform(p.cu[s]), b = uniform(p.cu[s + 1]);
    a = a < 0 ? 0 : (a > p.T ? p.T : a);
    b = b < a ? a : (b > p.T ? p.T : b);
    return {a, b};
}

// Pieces are numbered floor(start / piece) + s upwards for sequence s: the next sequence's
// first number is never below the end of this one's, because floor((start + n) / piece) + 1
// >= floor(start / piece) + ceil(n / piece).  Numbers that no piece has are skipped.
template <typename P> __device__ inline int64_t piece_base(const P& p, int s) {
    if (!p.cu) return int64_t(s) * ((p.L + p.piece - 1) / p.piece);
    int64_t a = p.cu[s];
    a = a < 0 ? 0 : (a > p.T ? p.T : a);
    return a / p.piece + s;
}

// The sequence of piece number `pi`, or -1: each round of 64 lanes narrows the range 64-fold.
template <typename P> __device__ inline int find_seq(const P& p, int64_t pi) {
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
template <int W> __device__ constexpr int twist(int r) {
    return W >= 128 ? 4 * (r & 3) + ((r >> 2) & 3) : W == 64 ? 4 * ((r >> 1) & 1) + ((r >> 2) & 3) : (r >> 2) & 3;
}
template <int W> __device__ constexpr int at_piece(int r, int p) { return r * W + 8 * (p ^ twist<W>(r)); }

// Byte offset of a lane's operand along the rows of a tile: lane 16g + i takes columns 8g ..
// + 7 of row i.  Rows 16 n further on are twisted alike, and columns 32 kb further on differ
// in bits of their own: (offset ^ 64 kb) + 2 W r0.  Offsets are formed by such steps from one
// value a chunk, since each would else cost a handful of vector instructions, which is what
// the passes spend most of their time on (left to the compiler: 529 a wave and chunk beside
// 97 matrix products).
template <int W> __device__ inline uint32_t row_base(int lane) { return 2 * at_piece<W>(lane & 15, lane >> 4); }
template <int W> __device__ inline u32x4 row_op(const uint16_t* t, int r0, int kb, uint32_t base) {
    return *reinterpret_cast<const u32x4*>(reinterpret_cast<const char*>(t) + (base ^ (64 * kb)) + 2 * W * r0);
}

// Transposed operand (ds_read_b64_tr_b16: of the four bf16 that lanes 4j + a of a group of
// 16 address, lane 4a + e gets element e of lane 4j + a as its element j).  Contraction
// slots 0..7 of lane 16g + i are rows r0 + 8g .. + 7; its column is
//   SPREAD = 0: c0 + i;   SPREAD = 1: 32 kb + 4 half + 8 (i / 4) + i % 4.
// Rows 4 further on differ in the twist's lowest bit.
template <int W, int SPREAD> __device__ inline uint32_t col_base(int c0, int lane) {
    const int r = 8 * (lane >> 4) + ((lane >> 2) & 3), c = c0 + (SPREAD ? 8 : 4) * (lane & 3);
    return 2 * (at_piece<W>(r, c >> 3) + (c & 7));
}
template <int W> __device__ inline u32x4 col_op(const uint16_t* t, int r0, int kb, int half, uint32_t base) {
    const char* const at = reinterpret_cast<const char*>(t) + 2 * W * r0 + 8 * half;
    const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(at + (base ^ (64 * kb))));
    const s16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(at + 8 * W + (base ^ (64 * kb + 16))));
    const uint2 u = __builtin_bit_cast(uint2, x), v = __builtin_bit_cast(uint2, y);
    return u32x4{u.x, u.y, v.x, v.y};
}

// Products of operands in NA and NB parts: those whose part numbers add up to at most `most`
// (the rest is below what the parts themselves leave out).
template <int NA, int NB>
__device__ inline f32x4 mma_parts(const u32x4 (&a)[NA], const u32x4 (&b)[NB], f32x4 c) {
    constexpr int most = (NA > NB ? NA : NB) - 1;
#pragma unroll
    for (int i = 0; i < NA; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j)
            if (i + j <= most) c = mma(a[i], b[j], c);
    return c;
}

// The value of the lane's neighbour (lanes 2n and 2n + 1 swap).
__device__ inline uint32_t swap1(uint32_t v) { return __builtin_amdgcn_update_dpp(0u, v, 0xB1, 0xf, 0xf, true); }

// Waits until at most N vector-memory operations are under way (the instruction's own
// encoding, so that the compiler counts from it too).
template <int N> __device__ inline void wait_memory() {
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
    asm volatile("" ::: "memory");
}

// Barrier for LDS traffic only: outstanding loads of the next chunk are not waited for.
__device__ inline void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// ---------------------------------------------------------------- memory
// Rows of a chunk through a buffer descriptor on its first token: rows at or behind `hi`
// and columns past the row's end read as zero and are not written.
typedef __amdgpu_buffer_rsrc_t Rsrc;
constexpr uint32_t kPast = 0x80000000u;   // an offset past every window (windows are < 2^31)
constexpr int64_t kMostHeads = 32767;
static_assert(64 * kMostHeads * SSM_LINATTN_MAX_DIM * 4 < int64_t(kPast), "a chunk's widest window: float32 rows of all heads");

// Byte offsets of a lane's outputs in a chunk's window: value (4 g4 + r) of the chunk's c tokens,
// in order of time or against it, at byte `at` of its row.  Columns that the head does not have
// (`on` false) lie kPast behind their own row, wherever the row steps lead: kPast + [0, window),
// which neither falls back into the window nor passes 2^32.
struct StoreRows {
    int pitch, lane0;
    __host__ __device__ inline StoreRows(int64_t row_bytes, bool rev, int c, int g4) {
        pitch = rev ? -int(row_bytes) : int(row_bytes);
        lane0 = int(row_bytes) * (rev ? c - 1 : 0) + 4 * g4 * pitch;
    }
    __host__ __device__ inline uint32_t first(bool on, int at) const { return uint32_t(lane0) + (on ? uint32_t(at) : kPast); }
    __host__ __device__ inline uint32_t row(int r) const { return uint32_t(r * pitch); }
};

__device__ inline Rsrc rows_rsrc(const char* row0, int64_t pitch, int64_t rows, int c) {
    const int64_t n = rows < c ? rows : c;
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(row0), 0, int(n * pitch), 0x00020000);
}

// 16 bytes per lane from a window straight into LDS: lane l's bytes land at lds + 16 l (lds
// wave-uniform); one more vector-memory operation under way, which the caller waits for
// (wait_memory) before a barrier.  Written out, because the compiler waits for all such loads
// before every LDS access it cannot tell apart from theirs, which would undo loading ahead.
// There is no register output.  The wait states cover m0 and descriptors that vector
// instructions left behind.
__device__ inline void load_lds16(const u32x4& window, uint32_t lds, uint32_t voff) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 :
                 : "s"(lds), "v"(voff), "s"(window)
                 : "memory", "m0");
}
__device__ inline uint32_t lds_address(const void* q) {
    return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const void*)q));
}
__device__ inline u32x4 rows_window(const char* row0, int64_t pitch, int64_t rows, int c) {
    const int64_t n = (rows < c ? rows : c) * pitch;
    const uint64_t a = reinterpret_cast<uint64_t>(row0);
    return u32x4{uint32_t(__builtin_amdgcn_readfirstlane(int(a))),
                 uint32_t(__builtin_amdgcn_readfirstlane(int(a >> 32))) & 0xffffu,
                 uint32_t(__builtin_amdgcn_readfirstlane(int(n))), 0x00020000u};
}

// A tile of C rows of W columns from memory to LDS.  bf16 rows (PARTS 1) go straight there,
// each lane fetching the piece that its slot of the permuted row holds; float32 rows
// (PARTS 3) pass through registers, where they are split.
template <int PARTS, int C, int W, int T, int HW = W> struct Tile {   // T threads
    static constexpr bool HALF = C * W / 8 < T;                 // fewer pieces of 8 values than threads
    static constexpr int N = HALF ? 1 : C * W / 8 / T;          // pieces per thread
    static_assert(HALF ? PARTS > 1 : C * W / 8 % T == 0, "whole pieces per thread");
    static constexpr int E = PARTS == 1 ? 2 : 4;
    static constexpr int RS = T / (W / 8);    // rows between a thread's pieces
    static constexpr int Q = PARTS == 1 ? 1 : 2;     // 16-byte loads per piece

    // HW columns of the tile belong to one head, w of them real: column c of the tile is
    // column c % HW of the (c / HW)-th head, w behind the one before
    __device__ static inline int column(int c, int w) { return HW == W ? c : (c / HW) * w + c % HW; }
    // Byte offsets of a thread's pieces from the chunk's first token: the first of even and of
    // odd pieces (rows RS apart are twisted alike, or every second of them), past the window
    // where there is no such column; further ones step by rows and stay past it.
    static constexpr int ODD = PARTS == 1 && twist<W>(RS) != 0 ? 2 : 1;
    uint32_t off[ODD];
    int step;
    __device__ inline void prepare(int tid, int64_t pitch, bool rev, int w) {
        step = int(rev ? -ODD * RS * pitch : ODD * RS * pitch);
#pragma unroll
        for (int n = 0; n < ODD; ++n) {
            const int rr = tid / (W / 8) + RS * n, slot = tid % (W / 8);
            const int col = 8 * (PARTS == 1 ? slot ^ twist<W>(rr) : slot);
            off[n] = col % HW < w && (!HALF || rr < C) ? uint32_t((rev ? C - 1 - rr : rr) * int(pitch) + column(col, w) * E)
                                                       : kPast;
        }
    }
    u32x4 r[PARTS == 1 ? 1 : N][Q];

    __device__ inline void load(uint16_t* tile, int wave, const char* row0, int64_t pitch, int64_t rows) {
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const uint32_t o = off[n % ODD] + uint32_t(n / ODD * step);
            if constexpr (PARTS == 1) {
                load_lds16(rows_window(row0, pitch, rows, C), lds_address(tile) + 16 * (T * n + 64 * wave), o);
            } else {
                const Rsrc b = rows_rsrc(row0, pitch, rows, C);
#pragma unroll
                for (int h = 0; h < Q; ++h)
                    r[n][h] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(b, o + 16 * h, 0, 0));
            }
        }
    }
    // float32 rows: what load() brought, in parts
    __device__ inline void store(uint16_t* tile, int tid) const {
        if constexpr (PARTS > 1) {
#pragma unroll
            for (int n = 0; n < N; ++n)
                if (!HALF || tid < C * W / 8) put(tile, tid + T * n, r[n]);
        }
    }
    __device__ static inline void put(uint16_t* tile, int idx, const u32x4 (&x)[Q]) {
        const int o = at_piece<W>(idx / (W / 8), idx % (W / 8));
        if constexpr (PARTS == 1) {
            *reinterpret_cast<u32x4*>(tile + o) = x[0];
        } else {
            u32x4 v[PARTS];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                uint32_t w[PARTS];
                split<PARTS>(__uint_as_float(x[e / 2][2 * (e & 1)]), __uint_as_float(x[e / 2][2 * (e & 1) + 1]), w);
#pragma unroll
                for (int k = 0; k < PARTS; ++k) v[k][e] = w[k];
            }
#pragma unroll
            for (int k = 0; k < PARTS; ++k) *reinterpret_cast<u32x4*>(tile + k * C * W + o) = v[k];
        }
    }
    // any alignment, any row length w: value by value
    __device__ static inline void copy_any(uint16_t* tile, int tid, const char* row0, int64_t pitch, int64_t rows, bool rev,
                                           int w) {
#pragma unroll 1
        for (int n = 0; n < N; ++n) {
            const int idx = tid + T * n;
            if (HALF && idx >= C * W / 8) break;
            const int col = 8 * (idx % (W / 8)), rr = rev ? C - 1 - idx / (W / 8) : idx / (W / 8);
            const char* q = row0 + rr * pitch + column(col, w) * E;
            u32x4 x[Q];
#pragma unroll
            for (int h = 0; h < Q; ++h) x[h] = u32x4{0, 0, 0, 0};
            // values past the row's end are read from its last column and dropped, so that the
            // eight loads go out together
            const int left = rr < rows ? w - col % HW : 0;
            if (left > 0) {
                uint32_t y[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int c = e < left ? e : left - 1;
                    if constexpr (PARTS == 1) y[e] = reinterpret_cast<const uint16_t*>(q)[c];
                    else y[e] = reinterpret_cast<const uint32_t*>(q)[c];
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const uint32_t z = e < left ? y[e] : 0u;
                    if constexpr (PARTS == 1) x[0][e / 2] |= z << (16 * (e & 1));
                    else x[e / 4][e % 4] = z;
                }
            }
            put(tile, idx, x);
        }
    }
};

// Decays of one chunk.  The sums run in float64 and are kept in two floats, so that a
// difference of two of them is right to float32 of the difference, however far they fell.
// The state in registers is R / s with a scale s that takes the chunks' decays in its place, in
// float64: slow decays are rounded once a half-life instead of once a chunk.  It is folded in
// where it would fall to 1/2, so that R / s reaches no further than R does (further down costs
// range, not time: the same within 1% at 2^-60).
template <int C> struct __align__(16) Decays {
    float hi[C], lo[C];   // G in log2 units
    float in[C];          // o s e^{G_i}: the incoming state's share at row i
    float out[C];         // w e^{G_C - G_j} / s': row j's share in the outgoing state
    float fold;           // what the state is multiplied with: 1, or s e^{G_C} where s' is 1 again
};

// v of the lane that a DPP control names, 0 where there is none (or the row is masked out).
template <int CTRL, int ROWS> __device__ inline double dpp_f64(double v) {
    const int lo = __builtin_amdgcn_update_dpp(0, __double2loint(v), CTRL, ROWS, 0xf, false);
    const int hi = __builtin_amdgcn_update_dpp(0, __double2hiint(v), CTRL, ROWS, 0xf, false);
    return __hiloint2double(hi, lo);
}
// Inclusive sum over the lanes of a wave: within rows of 16, then over the rows.
__device__ inline double scan_f64(double v) {
    v += dpp_f64<0x111, 0xf>(v);   // from 1, 2, 4, 8 lanes below
    v += dpp_f64<0x112, 0xf>(v);
    v += dpp_f64<0x114, 0xf>(v);
    v += dpp_f64<0x118, 0xf>(v);
    v += dpp_f64<0x142, 0xa>(v);   // lane 15 of rows 0 and 2 to rows 1 and 3
    v += dpp_f64<0x143, 0xc>(v);   // lane 31 to rows 2 and 3
    return v;
}
__device__ inline double lane_f64(double v, int lane) {
    return __hiloint2double(__builtin_amdgcn_readlane(__double2hiint(v), lane),
                            __builtin_amdgcn_readlane(__double2loint(v), lane));
}

// 2^x with the part of x that float32 drops brought back: a decay of 2^-50 would else be off
// by 2^-19 of itself, and the decays' gradient sums such errors over a piece.
__device__ inline float exp2_of(double x) {
    const float hi = float(x), e = __builtin_amdgcn_exp2f(hi);
    return fmaf(e * kLn2, float(x - double(hi)), e);
}

// One wave: lane r brings row r's log decay and works out the chunk's values.
template <int C> struct DecayLane {
    double scale = 0.0;   // log2 of s, the same in every lane
    // Without a read-out the chunks come last one first (see the pass), and `scale` is the
    // decay of those behind: the state is a plain sum.
    __device__ inline void ahead(Decays<C>& d, float g, float wscale, int lane) {
        g = g < kMinDecay ? kMinDecay : g;
        const double s = scan_f64(lane < C ? double(g) * 1.4426950408889634 : 0.0);
        const double end = lane_f64(s, C - 1);
        if (lane < C) d.out[lane] = wscale * exp2_of(scale + (end - s));
        if (lane == 0) d.fold = 1.0f;
        scale += end;
    }
    __device__ inline void next(Decays<C>& d, float g, float wscale, float oscale, int lane) {
        g = g < kMinDecay ? kMinDecay : g;
        const double s = scan_f64(lane < C ? double(g) * 1.4426950408889634 : 0.0);
        const double end = lane_f64(s, C - 1);
        const bool fold = !(fabs(scale + end) < 1.0);
        if (lane < C) {
            const float hi = float(s);
            d.hi[lane] = hi;
            d.lo[lane] = float(s - double(hi));
            d.in[lane] = oscale * exp2_of(scale + s);
            d.out[lane] = wscale * exp2_of(fold ? end - s : -scale - s);
            if (lane == 0) d.fold = fold ? exp2_of(scale + end) : 1.0f;
        }
        scale = fold ? 0.0 : scale + end;
    }
};

// Blocks of 16 x 32 of P that hold a tile on or below the diagonal: rows 16 it, columns 32 jb.
__device__ constexpr int p_block(int it, int jb) { return it < 2 ? it : 2 * it - 2 + jb; }

// ---------------------------------------------------------------- the pass
// One workgroup walks one piece of one head's sequence for 16 columns of the output per
// wave.  Each wave keeps the state's columns of its own in registers, in the layout in which
// the matrix unit leaves a product; the rows of a tile of 16 are numbered (8a + 4t + b for
// row 4a + b of tile t of a pair) so that a pair of tiles is the right operand of the
// read-out as it stands, with no exchange between lanes.  The decays of keys go to the value
// rows, so that the state's left operand is the key rows as read.
//
// Eight waves (128 columns) share the tiles and the products x1 . x2, and two such
// workgroups fit a CU up to 128 state rows.  Heads of up to 64 columns that share x1 and x2
// go two to a workgroup (NH), each with its own decays on the same products; other narrow
// heads take four waves.
//
// What bounds it: the issue of vector and matrix instructions.  A wave and chunk of 64 tokens of
// a 128 x 128 head takes 119 matrix products (16 cycles each) and 600 vector instructions (4
// cycles each), half of them the split of the state and of the decayed values into bf16 parts;
// counted on 131072 tokens of 16 heads matrix products run in 46% of the SIMD cycles and vector
// instructions in 58%, both at once in 16%: one or the other in 88%.  LDS is busy in 55% of the
// cycles, 45% of those in bank conflicts.  The output pass takes 571 us there (3.8 TB/s of rows;
// a plain copy 5.15) and the states pass before it 221 us (4.9 TB/s; one or the other in 75%); dq
// and dk in float32 of 4 x 4096 tokens of 32 heads 308 us.  Tried without gain: 32 columns a wave
// from registers, keys two products ahead, the parts' rests by two-term products, the heads of
// the second round of P's tiles on waves of their own.
//
// Parts: what is not a bf16 input (the state, the decayed products and values, float32 rows)
// goes into the products in three bf16 parts, which hold a float32 whole.  Two parts would take
// a fifth less of either unit (131072 tokens of 16 heads 776 us against 860) and leave out up to
// 2^-17 of each operand: outputs where terms cancel show that.
constexpr int pass_waves(int KD, int NW) { return KD == 256 ? NW / 4 : NW / 2; }   // per SIMD

template <int PARTS, int KD, int NW, int C, int MODE, int NH>
__global__ void __launch_bounds__(64 * NW, pass_waves(KD, NW)) linattn_pass_kernel(ssm_detail::LinattnPasses passes) {
    using namespace ssm_detail;
    const LinattnPass& p = passes.p[blockIdx.y];
    constexpr bool FULL = MODE == kLinFull;
    constexpr int T = 64 * NW, BV = 16 * NW, IT = C / 16, JB = C / 32, KB = KD / 32;
    constexpr int TW = NH == 1 ? NW - 1 : NW;         // waves with tiles of P: the one with the decays has none
    constexpr int NTILE = IT * (IT + 1) / 2, MT = (NTILE + TW - 1) / TW;   // tiles of P, and the most of one wave
    constexpr int WP = 3;                             // parts of the state, of P and of the decayed values
    constexpr int NBLK = C == 64 ? 6 : 2, PB = NBLK * 512;
    constexpr int HW = BV / NH, WH = NW / NH;         // columns and waves of one head
    static_assert(C == 64 || C == 32, "chunk");
    static_assert(NH == 1 || NH == 2, "heads");
    static_assert(NH * PB <= C * BV || NH == 1, "two heads' third part of P fits where x3 was");
    // bf16 rows come straight into LDS, each tile as soon as the last chunk's readers are
    // done with it: x2 (read to the end) and without a read-out x3 have a second tile, where
    // that still leaves room for two workgroups on a CU.  P takes that room at 128 state rows,
    // and two heads' P at 64: there the state goes on before P x3, and x2 is free after it
    // (EARLY).  At 128 rows two heads' P takes more than that: its third part goes where x3 was,
    // and x3 is asked for behind everything else (OVER; 250 us against 263 with one workgroup
    // on a CU, 2 x 8192 tokens of 64 heads).  float32 rows are held in registers from one chunk to
    // the next.
    constexpr bool DMA = PARTS == 1, EARLY = DMA && FULL && (KD == 128 || (KD == 64 && NH == 2)),
                   OVER = EARLY && KD == 128 && NH == 2, TWO2 = DMA && !EARLY, TWO3 = DMA && !FULL;
    constexpr int PL = OVER ? WP - 1 : WP;            // parts of P in its own place
    __shared__ __align__(16) uint16_t X2a[PARTS * C * KD], X2b[TWO2 ? C * KD : 8];
    __shared__ __align__(16) uint16_t X3a[PARTS * C * BV], X3b[TWO3 ? C * BV : 8];
    __shared__ __align__(16) uint16_t X1[FULL ? PARTS * C * KD : 8];
    __shared__ __align__(16) uint16_t PTs[FULL ? NH * PL * PB : 8];   // decayed x1 . x2, per head
    __shared__ Decays<C> decs[2][NH];
    const int tid = threadIdx.x, lane = tid & 63, g4 = lane >> 4, l16 = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    // neighbouring workgroups run on different XCDs: give each XCD neighbouring heads, so
    // that slices of one head and heads that share rows meet in one L2
    const int per = p.H / NH * p.nslices;
    int at = int(blockIdx.x % per);
    if (per % 8 == 0) at = (at % 8) * (per / 8) + at / 8;
    const int64_t pi = blockIdx.x / per;
    const int slice = uniform(at % p.nslices), h0 = uniform(at / p.nslices) * NH, hw = wave / WH, h = h0 + hw;   // h: this wave's head
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
    const bool rev = p.reverse;

    constexpr int E = PARTS == 1 ? 2 : 4;
    const int c_wave = slice * BV + (wave % WH) * 16;             // this wave's first column of its head
    const char* b1 = FULL ? static_cast<const char*>(p.x1) + int64_t(uniform(h0 / p.r1)) * p.kd * E : nullptr;
    const char* b2 = static_cast<const char*>(p.x2) + int64_t(uniform(h0 / p.r2)) * p.kd * E;
    const char* b3 = static_cast<const char*>(p.x3) + (int64_t(uniform(h0 / p.r3)) * p.vd + slice * BV) * E;
    const int w3 = p.vd - slice * BV;
    const int64_t pitch1 = p.s1 * E, pitch2 = p.s2 * E, pitch3 = p.s3 * E;

    // ------------------------------------------------ starting state
    f32x4 S[2 * KB];
    const int64_t rs = p.st_t ? 1 : p.vd, cs = p.st_t ? p.kd : 1;
    const int64_t ssz = int64_t(p.kd) * p.vd;
    const float* src = nullptr;
    if (FULL) {
        if (p.pieced && len > p.piece)
            src = p.carry + (pi * p.H + h) * ssz;
        else if (p.s_in)
            src = p.s_in + (int64_t(slot) * p.H + h) * ssz;
    }
#pragma unroll
    for (int m = 0; m < 2 * KB; ++m)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int row = 32 * (m >> 1) + 8 * g4 + 4 * (m & 1) + r, col = c_wave + l16;
            S[m][r] = src && row < p.kd && col < p.vd ? src[row * rs + col * cs] : 0.0f;
        }
    // tiles above the diagonal that share a block with one on it stay zero
    if constexpr (FULL) {
        for (int i = tid; i < NH * PL * PB / 2; i += T) reinterpret_cast<uint32_t*>(PTs)[i] = 0;
    }

    const int64_t nch = (hi - lo + C - 1) / C;
    // The pieces' own states are summed from each piece's last chunk to its first: what is read
    // last is what the pass with the read-out asks for first, and is still in the memory-side
    // cache as far as that goes (131072 tokens of 16 heads 812 -> 798 us, 2 x 8192 tokens of 64
    // shared heads 197 -> 190).
    const bool back = rev == FULL;
    auto first_of = [&](int64_t n) { return lo + (back ? nch - 1 - n : n) * C; };
    // the last wave of a head brings its decays, a chunk ahead; against time the decay of a
    // step belongs to the later of its two tokens
    const bool dec_wave = wave % WH == WH - 1;
    DecayLane<C> dl;
    const float p_scale = p.wscale * p.oscale;
    float gn = 0.0f;
    auto decay = [&](int64_t n, int lane) {
        const int64_t t = first_of(n) + (rev ? C - 1 - lane : lane), tg = rev ? t + 1 : t;
        return n < nch && lane < C && t < hi && tg < sq.end ? p.g[tg * p.sg + h] : 0.0f;
    };
    if (dec_wave && nch > 0) {
        if constexpr (FULL) dl.next(decs[0][hw], decay(0, lane), p.wscale, p.oscale, lane);
        else dl.ahead(decs[0][hw], decay(0, lane), p.wscale, lane);
        gn = decay(1, lane);
    }
    Tile<PARTS, C, KD, T> t1, t2;
    Tile<PARTS, C, BV, T, HW> t3;
    t2.prepare(tid, pitch2, rev, p.kd);
    t3.prepare(tid, pitch3, rev, w3);
    if constexpr (FULL) t1.prepare(tid, pitch1, rev, p.kd);
    // the tile of chunk n, at once (bf16) or into registers; `any` rows are copied at the
    // chunk's own turn
    auto load1 = [&](int64_t n) {
        const int64_t c0 = first_of(n);
        t1.load(X1, wave, b1 + c0 * pitch1, pitch1, hi - c0);
    };
    auto load2 = [&](int64_t n, uint16_t* to) {
        const int64_t c0 = first_of(n);
        t2.load(to, wave, b2 + c0 * pitch2, pitch2, hi - c0);
    };
    auto load3 = [&](int64_t n, uint16_t* to) {
        const int64_t c0 = first_of(n);
        t3.load(to, wave, b3 + c0 * pitch3, pitch3, hi - c0);
    };
    const bool ahead = DMA && p.wide;          // tiles are loaded ahead of their chunk
    if (p.wide && nch > 0) {
        load2(0, X2a);
        load3(0, X3a);
        if constexpr (FULL) load1(0);
    }
    if constexpr (DMA) wait_memory<0>();

    // one chunk; ODD picks the tiles of odd chunks where there are two
    auto chunk = [&](const int64_t n, auto odd_c) {
        constexpr bool ODD = decltype(odd_c)::value;
        uint16_t* const X2 = TWO2 && ODD ? X2b : X2a;
        uint16_t* const X3 = TWO3 && ODD ? X3b : X3a;
        Decays<C>& dec = decs[ODD][hw];
        uint16_t* const PT = PTs + hw * PL * PB;
        const int64_t c0 = first_of(n);
        // the lane as the loop's own value: operand addresses are cheap to form anew, and held
        // across the loop they would take the registers that the state needs
        int lane = __builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0u));
        asm volatile("" : "+v"(lane));
        const int tid = 64 * wave + lane, g4 = lane >> 4, l16 = lane & 15;
        if (ahead) {
            // this chunk's rows; what was stored since they were asked for may still be under way
            if constexpr (!FULL || OVER)
                wait_memory<0>();
            else if (p.pairs)
                wait_memory<2 * IT>();
            else
                wait_memory<4 * IT>();
            lds_barrier();
        } else {
            lds_barrier();                      // the last chunk's readers are done
            const int64_t rows = hi - c0;
            if (!DMA && p.wide) {
                t2.store(X2, tid);
                if constexpr (FULL) t1.store(X1, tid);
                t3.store(X3, tid);
                if (n + 1 < nch) {
                    load2(n + 1, X2);
                    load3(n + 1, X3);
                    if constexpr (FULL) load1(n + 1);
                }
            } else {
                t2.copy_any(X2, tid, b2 + c0 * pitch2, pitch2, rows, rev, p.kd);
                if constexpr (FULL) t1.copy_any(X1, tid, b1 + c0 * pitch1, pitch1, rows, rev, p.kd);
                t3.copy_any(X3, tid, b3 + c0 * pitch3, pitch3, rows, rev, w3);
            }
            lds_barrier();
        }
        if (ahead && n + 1 < nch) {
            if constexpr (TWO2) load2(n + 1, ODD ? X2a : X2b);
            if constexpr (TWO3) load3(n + 1, ODD ? X3a : X3b);
        }
        auto next = [&] {                        // the next chunk's decays
            if (dec_wave && n + 1 < nch) {
                if constexpr (FULL) dl.next(decs[!ODD][hw], gn, p.wscale, p.oscale, lane);
                else dl.ahead(decs[!ODD][hw], gn, p.wscale, lane);
                gn = decay(n + 2, lane);
            }
        };
        // the value rows of this wave's columns
        const int w0 = wave * 16;                // this wave's first column of the tile
        const uint32_t base3 = col_base<BV, 0>(w0, lane), base2 = col_base<KD, 1>(0, lane), base = row_base<KD>(lane);
        u32x4 v[JB][PARTS];
        auto values = [&] {
#pragma unroll
            for (int jb = 0; jb < JB; ++jb)
#pragma unroll
                for (int i = 0; i < PARTS; ++i) v[jb][i] = col_op<BV>(X3 + i * C * BV, 32 * jb, 0, 0, base3);
        };

        f32x4 acc[IT];
        uint2 third[OVER ? MT : 1][NH];
        if constexpr (FULL) {
            // ---- P = x1 . x2 under the decays, tiles of 16 x 16 on and below the diagonal
#pragma unroll
            for (int mm = 0; mm < MT; ++mm) {
                const int m = wave + TW * mm;
                if (m >= NTILE || wave >= TW) break;
                const int it = m < 1 ? 0 : m < 3 ? 1 : m < 6 ? 2 : 3;
                const int jt = m - it * (it + 1) / 2;
                f32x4 a = {0.0f, 0.0f, 0.0f, 0.0f};
                constexpr int AHEAD = PARTS == 1 ? (KB < 4 ? KB : 4) : 1;   // operands in flight
#pragma unroll
                for (int k0 = 0; k0 < KB; k0 += AHEAD) {
                    u32x4 k[AHEAD][PARTS], q[AHEAD][PARTS];
#pragma unroll
                    for (int x = 0; x < AHEAD * PARTS; ++x) {
                        const int kb = x / PARTS, i = x % PARTS;
                        k[kb][i] = row_op<KD>(X2 + i * C * KD, 16 * jt, k0 + kb, base);
                        q[kb][i] = row_op<KD>(X1 + i * C * KD, 16 * it, k0 + kb, base);
                    }
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int kb = 0; kb < AHEAD; ++kb) a = mma_parts<PARTS, PARTS>(k[kb], q[kb], a);
                }
                const int i = 16 * it + l16, j0 = 16 * jt + 4 * g4;
                const int o = p_block(it, jt >> 1) * 512 + at_piece<32>(l16, 2 * (jt & 1) + (g4 >> 1)) + 4 * (g4 & 1);
                f32x4 raw = a;
#pragma unroll
                for (int hh = 0; hh < NH; ++hh) {
                    const Decays<C>& dd = decs[ODD][hh];
                    const float gi = dd.hi[i], ei = dd.lo[i];
                    const f32x4 gj = *reinterpret_cast<const f32x4*>(&dd.hi[j0]), ej = *reinterpret_cast<const f32x4*>(&dd.lo[j0]);
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float w = __builtin_amdgcn_exp2f((gi - gj[r]) + (ei - ej[r]));
                        a[r] = j0 + r <= i ? raw[r] * (w * p_scale) : 0.0f;
                    }
                    uint32_t u[WP], v[WP];
                    split<WP>(a[0], a[1], u);
                    split<WP>(a[2], a[3], v);
#pragma unroll
                    for (int k = 0; k < PL; ++k) *reinterpret_cast<uint2*>(PTs + (hh * PL + k) * PB + o) = uint2{u[k], v[k]};
                    if constexpr (OVER) third[mm][hh] = uint2{u[WP - 1], v[WP - 1]};
                }
            }
            next();
            __builtin_amdgcn_s_setprio(1);   // a workgroup in its products goes before one that stores or waits (1.5%)
            // ---- the incoming state's share, e^{G_i} R^T x1_i
#pragma unroll
            for (int it = 0; it < IT; ++it) acc[it] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) {
                u32x4 q[IT][PARTS];
#pragma unroll
                for (int x = 0; x < IT * PARTS; ++x)
                    q[x / PARTS][x % PARTS] = row_op<KD>(X1 + (x % PARTS) * C * KD, 16 * (x / PARTS), kb, base);
                if (PARTS == 1) __builtin_amdgcn_sched_barrier(0);
                u32x4 sp[WP];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const f32x4& s = S[2 * kb + (e >> 1)];
                    uint32_t w[WP];
                    split<WP>(s[2 * (e & 1)], s[2 * (e & 1) + 1], w);
#pragma unroll
                    for (int k = 0; k < WP; ++k) sp[k][e] = w[k];
                }
#pragma unroll
                for (int it = 0; it < IT; ++it) acc[it] = mma_parts<PARTS, WP>(q[it], sp, acc[it]);
            }
#pragma unroll
            for (int it = 0; it < IT; ++it) {
                const f32x4 e = *reinterpret_cast<const f32x4*>(&dec.in[16 * it + 4 * g4]);
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[it][r] *= e[r];
            }
        } else {
            next();
        }
        values();

        // ---- the outgoing state
        auto onward = [&] {
            const float fold = __builtin_bit_cast(float, __builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, dec.fold)));
            if (fold != 1.0f) {
#pragma unroll
                for (int m = 0; m < 2 * KB; ++m)
#pragma unroll
                    for (int r = 0; r < 4; ++r) S[m][r] *= fold;
            }
#pragma unroll
            for (int jb = 0; jb < JB; ++jb) {
                u32x4 vp[WP];
                const f32x4 f0 = *reinterpret_cast<const f32x4*>(&dec.out[32 * jb + 8 * g4]);
                const f32x4 f1 = *reinterpret_cast<const f32x4*>(&dec.out[32 * jb + 8 * g4 + 4]);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float x = bf_lo(v[jb][PARTS - 1][e]), y = bf_hi(v[jb][PARTS - 1][e]);
#pragma unroll
                    for (int i = PARTS - 2; i >= 0; --i) {
                        x += bf_lo(v[jb][i][e]);
                        y += bf_hi(v[jb][i][e]);
                    }
                    const f32x4& f = e < 2 ? f0 : f1;
                    uint32_t w[WP];
                    split<WP>(x * f[2 * (e & 1)], y * f[2 * (e & 1) + 1], w);
#pragma unroll
                    for (int k = 0; k < WP; ++k) vp[k][e] = w[k];
                }
                constexpr int AHEAD = PARTS == 1 ? (EARLY ? 2 : 4) : 1;   // operands in flight
#pragma unroll
                for (int m0 = 0; m0 < 2 * KB; m0 += AHEAD) {
                    u32x4 k[AHEAD][PARTS];
#pragma unroll
                    for (int x = 0; x < AHEAD * PARTS; ++x) {
                        const int m = m0 + x / PARTS, i = x % PARTS;
                        k[x / PARTS][i] = col_op<KD>(X2 + i * C * KD, 32 * jb, m >> 1, m & 1, base2);
                    }
                    if (AHEAD > 1) __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int x = 0; x < AHEAD; ++x) S[m0 + x] = mma_parts<PARTS, WP>(k[x], vp, S[m0 + x]);
                }
            }
        };
        if constexpr (FULL) {
            lds_barrier();                      // P is there; x1 and x3 have been read
            // no registers are left to hold the loads' offsets there (EARLY): kept in scratch memory
            // they would be waited for behind every load and store under way
            if (ahead && n + 1 < nch) {
                if constexpr (!OVER) {
                    if constexpr (EARLY) t3.prepare(tid, pitch3, rev, w3);
                    load3(n + 1, X3);
                }
                if constexpr (EARLY) t1.prepare(tid, pitch1, rev, p.kd);
                load1(n + 1);
            }
            if constexpr (OVER) {               // P's third part; what lies above the diagonal is x3's still
#pragma unroll
                for (int mm = 0; mm < MT; ++mm) {
                    const int m = wave + TW * mm;
                    if (m >= NTILE + IT) break;
                    const int z = m - NTILE;    // of 4: the tiles beside (0, 0) and (2, 2) of either head
                    const int it = z >= 0 ? z & 2 : m < 1 ? 0 : m < 3 ? 1 : m < 6 ? 2 : 3;
                    const int jt = z >= 0 ? it + 1 : m - it * (it + 1) / 2;
                    const int o = p_block(it, jt >> 1) * 512 + at_piece<32>(l16, 2 * (jt & 1) + (g4 >> 1)) + 4 * (g4 & 1);
#pragma unroll
                    for (int hh = 0; hh < NH; ++hh)
                        if (z < 0 || (z & 1) == hh)
                            *reinterpret_cast<uint2*>(X3 + hh * PB + o) = z < 0 ? third[mm][hh] : uint2{0, 0};
                }
            }
            if constexpr (EARLY) {
                onward();
                if (OVER || (ahead && n + 1 < nch)) lds_barrier();   // x2 has been read; P is there whole
                if (ahead && n + 1 < nch) {
                    t2.prepare(tid, pitch2, rev, p.kd);
                    load2(n + 1, X2);
                }
            }
            // ---- the chunk's own share, P x3
            const uint32_t base_p = row_base<32>(lane);
#pragma unroll
            for (int jb = 0; jb < JB; ++jb)
#pragma unroll
                for (int it = 2 * jb; it < IT; ++it) {
                    u32x4 q[WP];
#pragma unroll
                    for (int k = 0; k < WP; ++k)
                        q[k] = row_op<32>((k < PL ? PT + k * PB : X3 + hw * PB) + p_block(it, jb) * 512, 0, 0, base_p);
                    acc[it] = mma_parts<WP, PARTS>(q, v[jb], acc[it]);
                }
            if constexpr (!EARLY) onward();
        } else {
            onward();
        }

        __builtin_amdgcn_s_setprio(0);
        if constexpr (FULL) {
            // rows behind the piece's end fall outside the window, as do columns past the head's
            const int oe = PARTS == 3 || p.out_f32 ? 4 : 2;
            const int64_t pitch64 = p.so * oe;
            const Rsrc ro = rows_rsrc(static_cast<char*>(p.out) + c0 * pitch64 + int64_t(h) * p.vd * oe, pitch64, hi - c0, C);
            const StoreRows to(pitch64, rev, C, g4);
            if (oe == 4) {
                const int col = c_wave + l16;
                const uint32_t o0 = to.first(col < p.vd, 4 * col);
#pragma unroll
                for (int x = 0; x < 4 * IT; ++x)
                    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(acc[x >> 2][x & 3]), ro,
                                                          o0 + to.row(16 * (x >> 2) + (x & 3)), 0, 0);
            } else if (p.pairs) {
                // neighbouring lanes swap one row for another: two columns of one row each
                const bool odd = lane & 1;
                const uint32_t pick = odd ? 0x03020706u : 0x05040100u;   // own and the neighbour's halves
                const int col = c_wave + (l16 & ~1);
                const uint32_t o0 = to.first(col < p.vd, 2 * col) + (odd ? to.row(1) : 0u);
#pragma unroll
                for (int it = 0; it < IT; ++it)
#pragma unroll
                    for (int r = 0; r < 4; r += 2) {
                        const uint32_t own = pack2(acc[it][r], acc[it][r + 1]);
                        __builtin_amdgcn_raw_buffer_store_b32(__builtin_amdgcn_perm(swap1(own), own, pick), ro,
                                                              o0 + to.row(16 * it + r), 0, 0);
                    }
            } else {
                const int col = c_wave + l16;
                const uint32_t o0 = to.first(col < p.vd, 2 * col);
#pragma unroll
                for (int x = 0; x < 4 * IT; ++x)
                    __builtin_amdgcn_raw_buffer_store_b16(IOT<uint16_t>::from_f32(acc[x >> 2][x & 3]), ro,
                                                          o0 + to.row(16 * (x >> 2) + (x & 3)), 0, 0);
            }
        }
        if constexpr (OVER) {
            if (ahead && n + 1 < nch) {
                lds_barrier();                  // P has been read
                t3.prepare(tid, pitch3, rev, w3);
                load3(n + 1, X3);
            }
        }
    };
    for (int64_t n = 0; n < nch; n += 2) {
        chunk(n, std::false_type{});
        if (n + 1 < nch) chunk(n + 1, std::true_type{});
    }

    // ------------------------------------------------ the state that leaves
    float* dst = nullptr;
    // the scale that the registers' state still has, from its head's wave
    float mul = 1.0f;
    if (FULL) {
        __syncthreads();
        if (dec_wave && lane == 0) decs[0][hw].fold = exp2_of(dl.scale);
        __syncthreads();
        mul = decs[0][hw].fold;
        if (last && p.s_out) {
            dst = p.s_out + (int64_t(slot) * p.H + h) * ssz;
            // against time the state before the first token has that token's decay too
            if (rev && sq.end > sq.start) {
                const float g = p.g[sq.start * p.sg + h];
                mul *= __builtin_amdgcn_exp2f((g < kMinDecay ? kMinDecay : g) * kLog2e);
            }
        }
    } else {
        dst = p.carry + (pi * p.H + h) * ssz;
        if (dec_wave && lane == 0 && slice == 0) p.tot[pi * p.H + h] = exp2_of(dl.scale);
    }
    if (dst) {
#pragma unroll
        for (int m = 0; m < 2 * KB; ++m)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = 32 * (m >> 1) + 8 * g4 + 4 * (m & 1) + r, col = c_wave + l16;
                if (row < p.kd && col < p.vd) dst[row * rs + col * cs] = mul * S[m][r];
            }
    }
}

// Chooses the kernel of a pass's sizes and starts it.
template <int MODE> inline void launch_pass(const ssm_detail::LinattnPasses& q, int count, bool f32, hipStream_t s) {
    const LinattnPass& p = q.p[0];
    // two heads in a workgroup share loads and products, but while each head finds a CU of its
    // own four waves of one SIMD each are sooner done than eight (three float32 prompts of up to
    // 130 tokens and 6 heads 26.5 us against 30.7 with two; 2 x 8192 tokens of 64 heads 286 us
    // against 254 with two)
    const bool two = p.r1 % 2 == 0 && p.r2 % 2 == 0 && int64_t(p.npieces) * p.H > kCus;
    const int shape = ssm_detail::linattn_shape(p.vd, two);
    const int64_t blocks = int64_t(p.npieces) * (shape == ssm_detail::kTwoHeads ? p.H / 2 : p.H) * p.nslices;
    const dim3 grid(static_cast<uint32_t>(blocks), count), block(shape == ssm_detail::kNarrow ? 256 : 512);
    // float32 rows take three times the LDS: chunks of 32 keep two workgroups on a CU
    const auto start = [&](auto* kernel) { launch_kernel(kernel, grid, block, 0, s, q); };
#define SSM_LIN_CASE(K, NW, NH)                                                                     \
    do {                                                                                            \
        if (f32) start(linattn_pass_kernel<3, K, NW, 32, MODE, NH>);                                \
        else start(linattn_pass_kernel<1, K, NW, 64, MODE, NH>);                                    \
    } while (0)
#define SSM_LIN_WAVES(K)                                                                            \
    do {                                                                                            \
        if (shape == ssm_detail::kWide) SSM_LIN_CASE(K, 8, 1);                                      \
        else if (shape == ssm_detail::kNarrow) SSM_LIN_CASE(K, 4, 1);                               \
        else SSM_LIN_CASE(K, 8, 2);                                                                 \
    } while (0)
    if (p.kd <= 64)
        SSM_LIN_WAVES(64);
    else if (p.kd <= 128)
        SSM_LIN_WAVES(128);
    else
        SSM_LIN_WAVES(256);
#undef SSM_LIN_WAVES
#undef SSM_LIN_CASE
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
    if (d->nseq > 65535 || d->nheads > kMostHeads || d->tokens > (int64_t(1) << 31) - 1) return SSM_ERR_DIMS;
    if (d->head_decay != 0 && d->head_decay != 1) return SSM_ERR_DIMS;
    if (d->reserved != 0) return SSM_ERR_DIMS;
    if (d->piece_len < 0 || d->piece_len % 64 != 0 || d->piece_len > (int64_t(1) << 31)) return SSM_ERR_DIMS;
    z->q = d->q_stride ? d->q_stride : d->kheads * d->dk;
    z->k = d->k_stride ? d->k_stride : d->kheads * d->dk;
    z->v = d->v_stride ? d->v_stride : d->nheads * d->dv;
    z->o = d->o_stride ? d->o_stride : d->nheads * d->dv;
    const int64_t lim = int64_t(1) << 40;
    // output windows of a chunk stay below 2^31 bytes
    if (z->o * (d->io_dtype == SSM_BF16 ? 2 : 4) >= (int64_t(1) << 24)) return SSM_ERR_DIMS;
    if (z->q < d->kheads * d->dk || z->k < d->kheads * d->dk || z->v < d->nheads * d->dv || z->o < d->nheads * d->dv)
        return SSM_ERR_DIMS;
    for (const int64_t s : {z->q, z->k, z->v, z->o})
        if (s > lim / d->tokens) return SSM_ERR_DIMS;
    z->e = d->io_dtype == SSM_BF16 ? 2 : 4;
    return SSM_OK;
}

// Workgroups of one launch: a grid has fewer than 2^32 threads.
constexpr int64_t kMostGroups = int64_t(1) << 22;

inline size_t up256(size_t n) { return (n + 255) / 256 * 256; }

// Rows that the 16-byte loads at 32-bit offsets of a chunk can take.
inline bool wide_rows(const void* q, int64_t stride, int64_t width, int64_t e) {
    return !misaligned(q, 16) && stride * e % 16 == 0 && width % 8 == 0 && stride * e < (int64_t(1) << 24);
}
inline bool pair_rows(const void* q, int64_t stride, int64_t width) {
    return !misaligned(q, 4) && stride % 2 == 0 && width % 2 == 0;
}

}  // namespace la
}  // namespace
