// mxs_tree_attention.hip -- attention of the drafted tokens of a batch of
// sequences over the paged 4-bit K/V cache.
//
// Sequence b has len cached tokens, found through its row of the page table;
// its n = cu[b + 1] - cu[b] query tokens are the last n of them (the drafted
// tokens, written to the cache before the call). Query token i sees every
// token of the context (the first len - n) and those drafted tokens whose bit
// is set in row i of the mask (without a mask: drafted tokens j <= i):
//   s_t = scale q[i, h] . K[t, g],   p = softmax over the seen t,
//   out[i, h] = sum_t p_t V[t, g],   g = h / G,  G = Hq / Hkv,
// and 0 where nothing is seen. One query token and no mask is plain decode;
// n in the hundreds is a chunk of a prompt.
//
// Rows. The n G query rows that share a KV head (row i G + h % G) are cut
// into tiles of 16 columns of the bf16 matrix instruction
// v_mfma_f32_16x16x32_bf16, in transposed form:
//   scores  S^T[t, r] = sum_d K[t, d] q[r, d]: A = K, lane (i, c) = token i of
//           a 16-token tile, words c NDP .. c NDP + NDP - 1 of its row (a word
//           is 8 dims, one 32-bit load), one word a step; B = the queries;
//   output  O^T[d, r] += sum_t V[t, d] p[t, r]: A = V, lane (i, c) = dims i DL ..
//           i DL + DL - 1 of tokens 4 c + r of two tiles; B = p, which the
//           score step leaves in exactly this lane layout.
// D is padded to 32 NDP = 64, 128 or 256 dims with zero query dims.
//
// Values. A 4-bit code in sign-magnitude form is the bit pattern of the
// subnormal e4m3 number code 2^-9, so v_cvt_scalef32_pk_bf16_fp8 turns two
// codes and the block's E8M0 scale into two exact bf16 values code 2^(s - 9)
// (scale bytes 0 to 2, values below 2^-122, round to multiples of 2^-124);
// the factors 2^9 go into the score scale and the final normalisation.
// A block with byte 0xFF is NaN. bf16 queries enter as they are; fp32 queries
// as the exact sum of three bf16 parts, and so do their softmax weights p. For
// bf16 queries p is rounded to one bf16: the error is independent from token to
// token, and of the size of the output's own rounding (together 0.0016 to 0.0022
// root mean square of the output, by shape and inputs, where two parts give 0.0015
// to 0.0018). Two parts cost 3 % in decode (100.4 against 97.7
// us at 32 ragged sequences), 14 % at 8 x 26 drafted tokens (103 against 90.5) and
// 18 % at 16 x 64 (556 against 470). A caller who wants whole weights passes the
// same queries as fp32 (8 sequences of 8192 tokens: 36 against 28 us). The sum
// that normalises is that of the rounded values, so one dominant token gives its V
// exactly. Maxima, sums and outputs are fp32.
//
// Kernels, by the rows n G of a KV head (tree_plan; bf16 / fp32 queries):
//   k_tree_rows  up to 16 (D <= 128, large batches: 32) / 16: every wave its own
//                tokens
//   k_tree_tile  up to 128 / 64, D > 128: four waves share stages in LDS
//   k_tree_pair  more: eight waves share stages and take turns
// One kernel serves a call, chosen by max_q: a prompt chunk among decoding
// sequences puts those into its tiles too (31 single tokens on 4096 and a chunk of
// 512: 315 us together, 45 + 135 in two calls).
// A device-side schedule (below) cuts the work into equal shares.
// Measured (MI355X, 8 KV heads, D = 128, pages of 64 tokens; bf16, fp32 queries):
//   32 sequences, one token, 4 query heads a KV head, 4915 to 16384 cached
//   tokens: 96 us, 3.9 TB/s of codes and scales (loads alone: 88 us)
//   one sequence of 2048, 8192, 32768 tokens, 8 query heads: 13.4, 14.7, 27.0 us
//   (15.4, 16.9, 31.6): the schedule and the join are most of the short ones
//   8 x 26 drafted tokens, 8 query heads, up to 8192 tokens: 90 us, 368 TFLOP/s
//   (all of 8192: 100, 203 us)
//   16 x 64, up to 16384 tokens: 470 us, 655 TFLOP/s (see k_tree_pair)
//   chunk of 512 behind 8192: 209 us (415); 4096 from nothing: 1405 us (2398)
// Registers: k_tree_rows of fp32 queries at D = 128 spills 28 bytes a lane (at
// D = 96, 60), k_tree_tile of bf16 at D > 128 48; the others no vector registers,
// all three kernels 76 to 157 scalar ones. 64 rows a wave (k_tree_tile with CT = 4)
// would halve the LDS reads of the many-row kernels; in the present order of work
// it spills 110 registers and is slower.
#include <cmath>
#include <type_traits>

#include "mxs_device.h"
#include "mxs_internal.h"

namespace mxs {

namespace {

typedef float f4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));
typedef uint32_t u2 __attribute__((ext_vector_type(2)));

constexpr int kRowTiles = 2;         // 16-token tiles of a wave's step in k_tree_rows
constexpr int kRowSets = 3;          // steps whose codes a wave holds or has in flight (bf16: one or two within 2 %)
constexpr int kNTL = 4;              // 16-token tiles of a stage in k_tree_tile
constexpr int kStep = 16 * kNTL;     // tokens of a stage

struct TreeArgs {
    const void *q;
    int64_t ldq;                     // elements between query tokens (heads D apart)
    bool qvec;                       // query rows 16-byte aligned
    const uint8_t *kc, *ks, *vc, *vs;
    int64_t pages;
    const int32_t *table;
    int64_t ldt;
    const int32_t *lens, *cu;
    const uint64_t *mask;
    int words;
    int B, Hq, Hkv, G, D;
    int total_q, max_q, max_len, ps;
    uint32_t pmul, pshift;           // t / ps
    float scale2;                    // |scale| log2(e) 2^9
    bool negate;                     // scale < 0: queries enter negated
    int R, U, P;                     // rows of a tile, tokens of a unit, workgroups: powers of two
    int Rs, Us, Ps;                  // their logarithms
    int ms, cap;                     // a share has at least 2^ms units, and a tile's 2^-cap
    int HG, groups;                  // KV heads of a tile, Hkv / HG
    int nrt;                         // row tiles of a head at most
    int join;                        // a k_tree_join follows
    int JR;                          // its rows of a workgroup
    void *out;
    int64_t ldo;
    float *po, *pml;                 // [2 share + k, HG, R, D], [2 share + k, HG, R, (m, l)]
    int *todo;                       // [8 entry + .]: see JoinOf
    int NT;                          // tiles at most, where they are no more than P: a todo entry each, else 0
};

// t / ps for 0 <= t < 2^31: pmul = ceil(2^(31 + l) / ps), l = ceil(log2 ps)
__device__ __forceinline__ int page_of(const TreeArgs &a, int t) {
    return a.ps == 1 ? t : (int)(__umulhi((uint32_t)t, a.pmul) >> a.pshift);
}

// four codes, one in the low nibble of each byte -> their e4m3 bytes
__device__ __forceinline__ uint32_t e4m3_codes(uint32_t x) {
    const uint32_t s = x & 0x08080808u, m = s >> 3;
    return (((x & 0x07070707u) ^ (s - m)) + m) | (s << 4);
}

typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
template <bool HI>
__device__ __forceinline__ uint32_t cvt2(uint32_t bytes, float scale) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(bytes, scale, HI));
}

// e4m3 bytes of a word's even and odd dims: the codes, or (OFF) code + 8, whose
// pattern is the number itself
template <bool OFF>
__device__ __forceinline__ void word_bytes(uint32_t w, uint32_t &even, uint32_t &odd) {
    if constexpr (OFF) {
        w ^= 0x88888888u;
        even = w & 0x0F0F0F0Fu;
        odd = (w >> 4) & 0x0F0F0F0Fu;
    } else {
        even = e4m3_codes(w);
        odd = e4m3_codes(w >> 4);
    }
}
// A word's 8 values, in the dim order 0 2 4 6 1 3 5 7
template <bool OFF>
__device__ __forceinline__ bf8 word_values(uint32_t w, float scale) {
    uint32_t e, o;
    word_bytes<OFF>(w, e, o);
    const u4 r = {cvt2<false>(e, scale), cvt2<true>(e, scale), cvt2<false>(o, scale), cvt2<true>(o, scale)};
    return __builtin_bit_cast(bf8, r);
}
__device__ __forceinline__ constexpr int word_dim(int s) { return s < 4 ? 2 * s : 2 * (s - 4) + 1; }

__device__ __forceinline__ float scale_of(uint32_t byte) { return __uint_as_float(byte << 23); }

// x as the sum of N bf16 parts, each the nearest to what the earlier ones leave
template <int N>
__device__ __forceinline__ void split_bf16(float x, __bf16 p[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        p[i] = (__bf16)x;
        x -= (float)p[i];
    }
}

// max over the four lanes c = 0..3 of a column
__device__ __forceinline__ float col_max(float x) {
    const uint32_t u = __float_as_uint(x);
    const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    const float y = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
    const uint32_t v = __float_as_uint(y);
    const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
// ------------------------------------------------------------------ shares
// The work of a call is a line of units: sequence by sequence, tile (HG KV
// heads, R of the n G rows of each) by tile, U tokens by U tokens (a sequence of
// no tokens has one empty unit a tile, which writes its zeros). It is cut into
// P' equal shares, one a workgroup, from the lengths that the call finds on the
// device: ragged batches are balanced, and a captured graph stays so when its
// lengths change. Every row tile of a sequence has the units of its whole length:
// where there is no mask, tokens past a tile's last row are computed and hidden,
// so a prompt from nothing does twice the work that its rows see (196 TFLOP/s of
// the seen pairs at 4096 tokens, 679 for a chunk of 512 behind 8192).
// A tile that lies in one share is written to `out`; the
// pieces of the others go to the workspace (a share has at most two: the end of
// a tile, k = 0, and the start of one, k = 1) and k_tree_join adds them.
struct Seq {
    int len, n, q0;                  // cached tokens, query tokens, first query token
    uint32_t nrt, T;                 // row tiles of a head, units of a tile
};
__device__ __forceinline__ Seq seq_of(const TreeArgs &a, int b) {
    Seq s;
    const int len = a.lens[b];
    s.len = len < 0 ? 0 : (len > a.max_len ? a.max_len : len);
    int q0 = a.cu[b], q1 = a.cu[b + 1];
    q0 = q0 < 0 ? 0 : (q0 > a.total_q ? a.total_q : q0);
    q1 = q1 < q0 ? q0 : (q1 > a.total_q ? a.total_q : q1);
    s.q0 = q0;
    s.n = q1 - q0 > a.max_q ? a.max_q : q1 - q0;
    s.nrt = ((uint32_t)(s.n * a.G) + a.R - 1) >> a.Rs;
    s.T = s.len > 0 ? ((uint32_t)s.len + a.U - 1) >> a.Us : 1u;
    return s;
}
__device__ __forceinline__ uint32_t units_of(const TreeArgs &a, const Seq &s) {
    return (uint32_t)a.groups * s.nrt * s.T;
}

// inclusive sum over the wave's lanes
__device__ __forceinline__ uint32_t wave_scan(uint32_t x) {
    x += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x111, 0xF, 0xF, true);    // lanes 1, 2, 4, 8 to the left
    x += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x112, 0xF, 0xF, true);    // in rows of 16
    x += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x114, 0xF, 0xF, true);
    x += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x118, 0xF, 0xF, true);
    x += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x142, 0xA, 0xF, false);   // the last lane of the row before
    x += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x143, 0xC, 0xF, false);   // lane 31
    return x;
}

struct Shares {
    uint32_t W, P;                   // units, shares
    int shift;                       // little work: shares of 2^shift units; else -1 and P = 2^Ps
    int Ps;
    __device__ __forceinline__ uint32_t start(uint32_t p) const {
        return shift >= 0 ? (p < P ? p << shift : W) : (uint32_t)(((uint64_t)p * W) >> Ps);    // floor(p W / P)
    }
    // the share of unit x (else the last p with p W < (x + 1) P)
    __device__ __forceinline__ uint32_t owner(uint32_t x) const {
        return shift >= 0 ? x >> shift : (uint32_t)(((double)(x + 1) * (double)P - 1.0) / (double)W);
    }
};

// 64 sequences, one a lane, and the line of units up to them
struct Window {
    int b0;                          // first sequence, a multiple of 64
    Seq s;                           // of sequence b0 + lane
    uint32_t units, end;             // of it; the units of the sequences up to it
    __device__ __forceinline__ void load(const TreeArgs &a, int b, uint32_t before, int lane) {
        b0 = b;
        units = 0;
        if (b + lane < a.B) {
            s = seq_of(a, b + lane);
            units = units_of(a, s);
        }
        end = before + wave_scan(units);
    }
    __device__ __forceinline__ uint32_t last() const { return (uint32_t)__builtin_amdgcn_readlane((int)end, 63); }
    __device__ __forceinline__ uint32_t first(int l) const {          // first unit of lane l's sequence
        return (uint32_t)__builtin_amdgcn_readlane((int)(end - units), l);
    }
    __device__ __forceinline__ Seq seq(int l) const {
        Seq r;
        r.len = __builtin_amdgcn_readlane(s.len, l);
        r.n = __builtin_amdgcn_readlane(s.n, l);
        r.q0 = __builtin_amdgcn_readlane(s.q0, l);
        r.nrt = (uint32_t)__builtin_amdgcn_readlane((int)s.nrt, l);
        r.T = (uint32_t)__builtin_amdgcn_readlane((int)s.T, l);
        return r;
    }
    // the lane of the sequence of unit x, which lies in a window from this one on
    __device__ __forceinline__ int find(const TreeArgs &a, uint32_t x, int lane) {
        for (;;) {
            const uint64_t past = __ballot(end > x);
            if (past) return __builtin_ctzll(past);
            if (b0 + 64 >= a.B) return -1;
            load(a, b0 + 64, last(), lane);
        }
    }
};
// The shares, and the window of the first 64 sequences
__device__ __forceinline__ Shares shares_of(const TreeArgs &a, Window &w, int lane) {
    Shares h;
    w.load(a, 0, 0, lane);
    h.W = w.last();
    uint32_t T = w.units ? w.s.T : 0u;
    for (int b = 64; b < a.B; b += 64) {
        Window v;
        v.load(a, b, h.W, lane);
        h.W = v.last();
        T = v.units && v.s.T > T ? v.s.T : T;
    }
    // the longest tile in at most 2^cap shares: a join of many small pieces
    // costs more than it gains
    int sh = a.ms;
    while (__ballot(T > (1u << (sh + a.cap)))) ++sh;
    const uint32_t most = (h.W + (1u << sh) - 1) >> sh;
    h.shift = most <= (uint32_t)a.P ? sh : -1;
    h.P = h.shift >= 0 ? most : (uint32_t)a.P;
    h.Ps = a.Ps;
    return h;
}

// A piece of a share: tokens t0 .. t1 - 1 of one tile
struct Place {
    int b, g, row;                   // sequence, first KV head and first row of the tile
    int len, ctx, n, q0;             // cached tokens, context, query tokens, first query token
    int t0, t1;
    int64_t slot;                    // workspace slot, -1: the whole tile
};

// What k_tree_join finds in a todo entry. Entries are those of the tiles ((b,
// head group, row tile), NT > 0) or of the shares that hold a tile's first piece
// but not its last; an entry with last <= first needs no join. The entry of a
// share is written by the share ((0, -1) where no tile starts that it does not
// end), that of a tile by the share of its first unit; entries of no tile are
// left, and told by the sequence's n. What no one wrote is not read.
struct JoinOf {
    int first, last;                 // shares of its first and last piece
    int q0, n, g, row;               // Place's
};

// f(place) for every piece of this workgroup's share. Consecutive shares (row
// tiles of one KV head, then its neighbours in the same 128-byte lines of the
// cache) go to one XCD: workgroups are dealt to the 8 XCDs in turn.
template <typename F>
__device__ __forceinline__ void for_each_piece(const TreeArgs &a, int lane, F f) {
    Window win;
    const Shares h = shares_of(a, win, lane);
    const uint32_t per = (h.P + 7) / 8, p = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
    if (a.join && a.NT == 0 && threadIdx.x == 0) {       // nothing to join yet; the number of shares
        if ((blockIdx.x >> 3) < per && p < h.P) {
            a.todo[8 * p] = 0;                           // both: the workspace holds anything, and the join
            a.todo[8 * p + 1] = -1;                      // compares them
        }
        if (blockIdx.x == 0) a.todo[8 * a.P] = (int)h.P;
    }
    if ((blockIdx.x >> 3) >= per || p >= h.P) return;
    uint32_t x = h.start(p);
    const uint32_t end = h.start(p + 1);
    while (x < end) {
        const int l = win.find(a, x, lane);
        if (l < 0) return;
        const Seq s = win.seq(l);
        const int b = win.b0 + l;
        const uint32_t first = win.first(l);
        const uint32_t tile = s.T == 1 ? x - first : (x - first) / s.T, u0 = (x - first) - tile * s.T;
        const uint32_t gt = s.nrt == 1 ? tile : tile / s.nrt;
        const uint32_t u1 = s.T - u0 < end - x ? s.T : u0 + (end - x);
        auto uni = [](int v) { return __builtin_amdgcn_readfirstlane(v); };
        Place pl;
        pl.b = uni(b);
        pl.g = uni((int)gt * a.HG);
        pl.row = uni((int)(tile - gt * s.nrt) * a.R);
        pl.len = uni(s.len);
        pl.n = uni(s.n);
        pl.q0 = uni(s.q0);
        pl.ctx = uni(s.len > s.n ? s.len - s.n : 0);
        pl.t0 = uni((int)u0 * a.U);
        pl.t1 = uni(u1 == s.T ? s.len : (int)u1 * a.U);
        pl.slot = u0 == 0 && u1 == s.T ? -1 : 2 * (int64_t)p + (u0 > 0 ? 0 : 1);
        if (a.join && u0 == 0 && (u1 < s.T || a.NT) && threadIdx.x == 0) {
            const int64_t entry = a.NT ? ((int64_t)b * a.groups + gt) * a.nrt + (tile - gt * s.nrt) : p;
            int *t = a.todo + 8 * entry;
            t[0] = (int)p;
            t[1] = u1 < s.T ? (int)h.owner(x + s.T - 1) : -1;
            t[2] = pl.q0;
            t[3] = pl.n;
            t[4] = pl.g;
            t[5] = pl.row;
        }
        f(pl);
        x += u1 - u0;
    }
}

// Bits of drafted tokens 64 k .. 64 k + 63 that query token i sees
__device__ __forceinline__ uint64_t mask_word(const TreeArgs &a, const Place &p, int i, int k) {
    if (a.mask) return k < a.words ? a.mask[(int64_t)(p.q0 + i) * a.words + k] : 0ull;
    const int d = i - 64 * k;
    return d >= 63 ? ~0ull : (d < 0 ? 0ull : (2ull << d) - 1);
}

// Bits of tokens lt .. lt + 63 that query token i sees
__device__ __forceinline__ uint64_t mask_window(const TreeArgs &a, const Place &p, int i, int lt) {
    const int j = lt - p.ctx;
    if (j <= -64) return ~0ull;
    if (j < 0) return (mask_word(a, p, i, 0) << -j) | ((1ull << -j) - 1);
    const int k = j >> 6, s = j & 63;
    uint64_t w = mask_word(a, p, i, k) >> s;
    if (s) w |= mask_word(a, p, i, k + 1) << (64 - s);
    return w;
}

// Query rows of a wave, as the loads leave them: 16 bytes each where the rows
// are aligned (qvec). Lane (r, c), step b: the dims of word c NDP + b of row r.
template <int NDP, int CT, int PARTS>
struct RawQueries {
    typedef std::conditional_t<PARTS == 1, uint16_t, float> T;
    static constexpr int N = PARTS == 1 ? 1 : 2;                // 16-byte loads of 8 elements
    u4 raw[CT][NDP][N];
    int i[CT];                                                   // query token of the column, -1: no row
    __device__ __forceinline__ void load(const TreeArgs &a, const Place &p, int g, int row0, int lane) {
        const int r = lane & 15, c = lane >> 4;
#pragma unroll
        for (int t = 0; t < CT; ++t) {
            const int row = row0 + 16 * t + r;
            const bool on = row < p.n * a.G;
            const int tok = on ? row / a.G : 0, h = on ? g * a.G + row - tok * a.G : 0;
            i[t] = on ? tok : -1;
            const T *q = static_cast<const T *>(a.q) + (int64_t)(p.q0 + tok) * a.ldq + (int64_t)h * a.D;
#pragma unroll
            for (int b = 0; b < NDP; ++b) {
                const int d0 = 8 * (c * NDP + b);
                const T *e = q + (d0 < a.D ? d0 : 0);
                if (a.qvec) {
#pragma unroll
                    for (int k = 0; k < N; ++k) raw[t][b][k] = reinterpret_cast<const u4 *>(e)[k];
                } else if constexpr (PARTS == 1) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) raw[t][b][0][k] = e[2 * k] | (uint32_t)e[2 * k + 1] << 16;
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k) raw[t][b][k >> 2][k & 3] = __float_as_uint(e[k]);
                }
            }
        }
    }
    // as B operands, zero past the rows and past D
    __device__ __forceinline__ void operands(const TreeArgs &a, int lane, bf8 qf[CT][NDP][PARTS]) const {
        const int c = lane >> 4;
#pragma unroll
        for (int t = 0; t < CT; ++t)
#pragma unroll
            for (int b = 0; b < NDP; ++b) {
                const bool in = i[t] >= 0 && 8 * (c * NDP + b) < a.D;
#pragma unroll
                for (int s = 0; s < 8; ++s) {
                    const int d = word_dim(s);
                    float x;
                    if constexpr (PARTS == 1)
                        x = __uint_as_float(d & 1 ? raw[t][b][0][d >> 1] & 0xFFFF0000u : raw[t][b][0][d >> 1] << 16);
                    else
                        x = __uint_as_float(raw[t][b][d >> 2][d & 3]);
                    x = in ? (a.negate ? -x : x) : 0.f;
                    __bf16 part[PARTS];
                    split_bf16<PARTS>(x, part);
#pragma unroll
                    for (int k = 0; k < PARTS; ++k) qf[t][b][k][s] = part[k];
                }
            }
    }
};

// Operands that take the offset of 8 codes out of the scores: A = the scales of
// a lane's K blocks as bf16, three times each (a 0xFF byte gives Inf, and NaN in
// the sum); B = -8 2^-9 times the sum of the lane's query dims of each block,
// as three bf16 parts
template <int NDP>
__device__ __forceinline__ bf8 query_sums(const bf8 qf[NDP][1]) {
    constexpr int KB = NDP == 8 ? 2 : 1;
    bf8 r;
#pragma unroll
    for (int s = 0; s < 8; ++s) r[s] = (__bf16)0.f;
#pragma unroll
    for (int k = 0; k < KB; ++k) {
        float x = 0.f;
#pragma unroll
        for (int b = k * (NDP / KB); b < (k + 1) * (NDP / KB); ++b)
#pragma unroll
            for (int s = 0; s < 8; ++s) x += (float)qf[b][0][s];
        __bf16 part[3];
        split_bf16<3>(x * -0.015625f, part);
#pragma unroll
        for (int s = 0; s < 3; ++s) r[3 * k + s] = part[s];
    }
    return r;
}
template <int NDP>
__device__ __forceinline__ bf8 scale_operand(const uint32_t e[NDP == 8 ? 2 : 1]) {
    const uint32_t s = e[0] * 0x00800080u;
    if constexpr (NDP == 8) {
        const uint32_t x = e[1] << 7;
        return __builtin_bit_cast(bf8, u4{s, (e[0] << 7) | (x << 16), x | (x << 16), 0u});
    }
    return __builtin_bit_cast(bf8, u4{s, e[0] << 7, 0u, 0u});
}

template <int NDP>
struct Raw {
    static constexpr int KB = NDP == 8 ? 2 : 1;      // blocks a lane's K words touch
    static constexpr int VW = NDP == 8 ? 2 : 1;      // words a lane's V dims touch
};

// Byte offsets of a lane inside a cache row; dims past D fall back to the
// row's first block (their query dims are zero, their outputs not stored)
template <int NDP>
struct LaneAt {
    uint32_t k[Raw<NDP>::KB], kb[Raw<NDP>::KB], v, vb;
    __device__ __forceinline__ LaneAt(int lane, int D) {
        const int i = lane & 15, c = lane >> 4;
#pragma unroll
        for (int b = 0; b < Raw<NDP>::KB; ++b) {
            const int w = c * NDP + 4 * b;                           // first word
            k[b] = 8 * w < D ? 4 * w : 0;
            kb[b] = 8 * w < D ? w >> 2 : 0;
        }
        const int d = i * 2 * NDP;                                   // first V dim
        v = d < D ? d / 2 : 0;
        vb = d < D ? d >> 5 : 0;
    }
};

// A lane's K words of the cache row at p, V word(s) of the row at p
template <int NDP>
__device__ __forceinline__ void load_k(uint32_t k[NDP], const uint8_t *p, const LaneAt<NDP> &at) {
    if constexpr (NDP == 2) {
        const u2 w = *reinterpret_cast<const u2 *>(p + at.k[0]);
        k[0] = w[0];
        k[1] = w[1];
    } else {
#pragma unroll
        for (int b = 0; b < Raw<NDP>::KB; ++b) {
            const u4 w = *reinterpret_cast<const u4 *>(p + at.k[b]);
#pragma unroll
            for (int j = 0; j < 4; ++j) k[4 * b + j] = w[j];
        }
    }
}
template <int NDP>
__device__ __forceinline__ void load_v(uint32_t v[Raw<NDP>::VW], const uint8_t *p, const LaneAt<NDP> &at) {
    if constexpr (NDP == 2) {
        v[0] = *reinterpret_cast<const uint16_t *>(p + at.v);
    } else if constexpr (NDP == 4) {
        v[0] = *reinterpret_cast<const uint32_t *>(p + at.v);
    } else {
        const u2 w = *reinterpret_cast<const u2 *>(p + at.v);
        v[0] = w[0];
        v[1] = w[1];
    }
}
// The D / 32 scale bytes of one row, in one or two words: one load where D is
// not padded (FULL), else a byte load each, those past the row repeating its
// last byte. No load sits behind a branch: at the join of the two paths the
// compiler would wait for every load in flight.
template <int NDP, bool FULL>
__device__ __forceinline__ void load_scales(uint32_t x[Raw<NDP>::KB], const uint8_t *p, int nd) {
    if constexpr (FULL && NDP == 8) {
        const u2 w = *reinterpret_cast<const u2 *>(p);
        x[0] = w[0];
        x[1] = w[1];
    } else if constexpr (FULL && NDP == 4) {
        x[0] = *reinterpret_cast<const uint32_t *>(p);
    } else if constexpr (FULL) {
        x[0] = *reinterpret_cast<const uint16_t *>(p);
    } else {
        uint32_t b[NDP];
#pragma unroll
        for (int i = 0; i < NDP; ++i) b[i] = p[i < nd ? i : nd - 1];
#pragma unroll
        for (int i = 0; i < Raw<NDP>::KB; ++i) {
            x[i] = 0;
#pragma unroll
            for (int j = 0; j < (NDP < 4 ? NDP : 4); ++j) x[i] |= b[4 * i + j] << (8 * j);
        }
    }
}

// Running state of a wave: columns r of its CT tiles. m is the reference the
// exponents are taken from (raw score units), l the sum of the weights, formed
// by the matrix product of p with ones (the same in all four registers): it
// sums the very values that multiply V, and costs the vector ALU nothing.
template <int NDP, int CT>
struct State {
    f4 acc[CT][2 * NDP];
    float m[CT];
    f4 l[CT];
    f4 w[CT];                        // sum of p times the offset's value 8 2^(s - 9) of the lane's V block
    uint32_t nan[CT];                // bit rr: the output's dims of register rr are NaN (see give_nan)
};

// Scores of tokens that a column's row does not see (bit 16 u + 4 c + s clear)
template <int CT, int NTL>
__device__ __forceinline__ void hide(f4 sc[CT][NTL], const uint64_t seen[CT], int c) {
#pragma unroll
    for (int t = 0; t < CT; ++t) {
        const uint64_t w = seen[t] >> (4 * c);
#pragma unroll
        for (int u = 0; u < NTL; ++u)
#pragma unroll
            for (int s = 0; s < 4; ++s) sc[t][u][s] = (w >> (16 * u + s)) & 1 ? sc[t][u][s] : -INFINITY;
    }
}

// Scores to weights p = 2^((s - m) scale2) (0 for hidden ones; scale2 > 0).
// The reference m moves only when a score exceeds it by more than 2^6 (in the
// exponent), so most steps leave the accumulators alone; p stays below 2^6.
// EXACT (fp32): the difference first, so that the product's rounding scales
// with the exponent and not with the score; bf16: one operation instead of two.
template <int NDP, int CT, int NTL, bool EXACT>
__device__ __forceinline__ void soften(State<NDP, CT> &st, f4 sc[CT][NTL], float scale2) {
    float top[CT];
    bool grow = false;
#pragma unroll
    for (int t = 0; t < CT; ++t) {
        float x = -INFINITY;
#pragma unroll
        for (int u = 0; u < NTL; ++u)
#pragma unroll
            for (int s = 0; s < 4; ++s) x = fmaxf(x, sc[t][u][s]);
        top[t] = col_max(x);
        grow |= (top[t] - st.m[t]) * scale2 > 6.f || (st.m[t] == -INFINITY && top[t] > -INFINITY);
    }
    if (__ballot(grow)) {
#pragma unroll
        for (int t = 0; t < CT; ++t) {
            const float m = fmaxf(st.m[t], top[t]);
            const float f = st.m[t] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f((st.m[t] - m) * scale2);
            st.m[t] = m;
            st.l[t] *= f;
            st.w[t] *= f;
#pragma unroll
            for (int n = 0; n < 2 * NDP; ++n) st.acc[t][n] *= f;
        }
    }
#pragma unroll
    for (int t = 0; t < CT; ++t) {
        const float mr = st.m[t] == -INFINITY ? 0.f : st.m[t], ms = mr * scale2;
#pragma unroll
        for (int u = 0; u < NTL; ++u)
#pragma unroll
            for (int s = 0; s < 4; ++s)
                sc[t][u][s] = __builtin_amdgcn_exp2f(EXACT ? (sc[t][u][s] - mr) * scale2
                                                             : __builtin_fmaf(sc[t][u][s], scale2, -ms));
    }
}

// V of tokens 4 c + s of one tile, in token pairs: o[n] = dim i DL + n of
// tokens (0, 1) and (2, 3)
template <int NDP, bool OFF>
__device__ __forceinline__ void v_pairs(const uint32_t v[4][Raw<NDP>::VW], const float sc[4],
                                        uint32_t o[2 * NDP][2]) {
#pragma unroll
    for (int j = 0; j < 4; j += 2) {
#pragma unroll
        for (int w = 0; w < Raw<NDP>::VW; ++w) {
            uint32_t x[2][4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float s = sc[j + h];
                uint32_t e, d;
                word_bytes<OFF>(v[j + h][w], e, d);
                x[h][0] = cvt2<false>(e, s);                          // dims 0, 2
                x[h][1] = cvt2<false>(d, s);                          // dims 1, 3
                if constexpr (NDP != 2) {
                    x[h][2] = cvt2<true>(e, s);                       // dims 4, 6
                    x[h][3] = cvt2<true>(d, s);                       // dims 5, 7
                }
            }
#pragma unroll
            for (int k = 0; k < (NDP == 2 ? 2 : 4); ++k) {
                const int dim = 8 * w + (k >> 1) * 4 + (k & 1);
                o[dim][j >> 1] = __builtin_amdgcn_perm(x[1][k], x[0][k], 0x05040100u);
                o[dim + 2][j >> 1] = __builtin_amdgcn_perm(x[1][k], x[0][k], 0x07060302u);
            }
        }
    }
}
// The 2 NDP V operands of two tiles (tile n = dim i DL + n of lane (i, c)); OFF:
// `off` is the operand of a code of 0 in the lane's blocks, converted as the
// codes are. It has their range and rounding: no sum of it overflows where theirs
// does not, and zeros cancel to the last bit at any scale.
template <int NDP, bool OFF>
__device__ __forceinline__ void v_operands(const uint32_t v[2][4][Raw<NDP>::VW], const uint32_t vb[2][4],
                                           bf8 out[2 * NDP], bf8 &off) {
    constexpr uint32_t kZero = 0x0808u;                               // two codes of 0, 8 added
    uint32_t o[2][2 * NDP][2], w[2][2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        float sc[4];
#pragma unroll
        for (int s = 0; s < 4; ++s) sc[s] = scale_of(vb[u][s]);
        v_pairs<NDP, OFF>(v[u], sc, o[u]);
#pragma unroll
        for (int s = 0; s < 2; ++s)
            w[u][s] = OFF ? __builtin_amdgcn_perm(cvt2<false>(kZero, sc[2 * s + 1]), cvt2<false>(kZero, sc[2 * s]),
                                                  0x05040100u)
                          : 0u;
    }
#pragma unroll
    for (int n = 0; n < 2 * NDP; ++n) out[n] = __builtin_bit_cast(bf8, u4{o[0][n][0], o[0][n][1], o[1][n][0], o[1][n][1]});
    off = __builtin_bit_cast(bf8, u4{w[0][0], w[0][1], w[1][0], w[1][1]});
}

// B operands of p for tiles u0, u0 + 1, in PP bf16 parts
template <int PP>
__device__ __forceinline__ void p_operands(f4 p0, f4 p1, bf8 out[PP]) {
    float x[8] = {p0[0], p0[1], p0[2], p0[3], p1[0], p1[1], p1[2], p1[3]};
#pragma unroll
    for (int k = 0; k < PP; ++k) {
        u4 w;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const bf2 h = {(__bf16)x[2 * j], (__bf16)x[2 * j + 1]};
            w[j] = __builtin_bit_cast(uint32_t, h);
            if (k + 1 < PP) {
                x[2 * j] -= __uint_as_float(w[j] << 16);
                x[2 * j + 1] -= __uint_as_float(w[j] & 0xFFFF0000u);
            }
        }
        out[k] = __builtin_bit_cast(bf8, w);
    }
}
// A operand of ones: its product with p is sum_t p_t in every register
__device__ __forceinline__ bf8 ones() {
    const u4 w = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
    return __builtin_bit_cast(bf8, w);
}

// V blocks that are NaN (byte 0xFF) would reach rows that do not see their
// token, as 0 times NaN, where a step holds tokens that some rows do not see.
// There such blocks leave the matrix product (their byte becomes 0; the result
// has a bit for every lane whose byte it was), and the rows that see the token
// note which of their dims are NaN: lanes = the 16 dim groups of token tk.
__device__ __forceinline__ uint64_t take_nan(uint32_t &byte) {
    const uint64_t bad = __ballot(byte == 0xFFu);
    if (byte == 0xFFu) byte = 0;
    return bad;
}
template <int NDP, int CT>
__device__ __forceinline__ void note_nan(State<NDP, CT> &st, uint32_t lanes, int tk, const uint64_t seen[CT], int c) {
#pragma unroll
    for (int t = 0; t < CT; ++t)
        if ((seen[t] >> tk) & 1) st.nan[t] |= (lanes >> (4 * c)) & 15u;
}
template <int NDP, int CT>
__device__ __forceinline__ void give_nan(State<NDP, CT> &st) {
#pragma unroll
    for (int t = 0; t < CT; ++t) {
        if (!__ballot(st.nan[t] != 0)) continue;
#pragma unroll
        for (int rr = 0; rr < 4; ++rr)
#pragma unroll
            for (int n = 0; n < 2 * NDP; ++n) st.acc[t][n][rr] = (st.nan[t] >> rr) & 1 ? NAN : st.acc[t][n][rr];
    }
}

// Outputs of one column: lane (r, c) holds dims (4 c + rr) DL + n of row r.
// A whole tile: normalised, rounded once, to `out` (0 where nothing was seen);
// a piece: (m, l) and the unnormalised sums for k_tree_join.
template <int NDP, int CT, int PARTS>
__device__ __forceinline__ void store_rows(const TreeArgs &a, const Place &p, const State<NDP, CT> &st, int g,
                                           int row0, int lane) {
    constexpr int DL = 2 * NDP;
    const int r = lane & 15, c = lane >> 4;
#pragma unroll
    for (int t = 0; t < CT; ++t) {
        const int row = row0 + 16 * t + r;
        if (row >= p.n * a.G) continue;
        const int i = row / a.G, h = g * a.G + row - i * a.G;
        if (p.slot < 0) {
            const float f = st.m[t] == -INFINITY ? 0.f : 512.f / st.l[t][0];
#pragma unroll
            for (int rr = 0; rr < 4; ++rr) {
                const int d0 = (4 * c + rr) * DL;
                if (d0 >= a.D) continue;
                const int64_t e = (int64_t)(p.q0 + i) * a.ldo + (int64_t)h * a.D + d0;
#pragma unroll
                for (int n = 0; n < DL; ++n) {
                    const float x = st.acc[t][n][rr] * f;
                    if constexpr (PARTS == 1) static_cast<__bf16 *>(a.out)[e + n] = (__bf16)x;
                    else static_cast<float *>(a.out)[e + n] = x;
                }
            }
        } else {
            const int64_t at = (p.slot * a.HG + (g - p.g)) * a.R + (row - p.row);
            if (c == 0) {
                a.pml[2 * at] = st.m[t] == -INFINITY ? -INFINITY : st.m[t] * a.scale2;
                a.pml[2 * at + 1] = st.l[t][0];
            }
#pragma unroll
            for (int rr = 0; rr < 4; ++rr) {
                const int d0 = (4 * c + rr) * DL;
                if (d0 >= a.D) continue;
                float *o = a.po + at * a.D + d0;
#pragma unroll
                for (int n = 0; n < DL; ++n) o[n] = st.acc[t][n][rr];
            }
        }
    }
}

// The offset of 8 codes leaves the outputs
template <int NDP, int CT>
__device__ __forceinline__ void take_offset(State<NDP, CT> &st) {
#pragma unroll
    for (int t = 0; t < CT; ++t)
#pragma unroll
        for (int n = 0; n < 2 * NDP; ++n) st.acc[t][n] -= st.w[t];
}

// States of two waves over the same rows, through LDS in lane order (CT (2 NDP
// + 1) KiB): M = max m, sums and outputs scaled by 2^((m - M) scale2)
template <int NDP, int CT>
__device__ __forceinline__ void give_state(const State<NDP, CT> &st, float *ex, int lane) {
    f4 *e = reinterpret_cast<f4 *>(ex) + lane;
#pragma unroll
    for (int t = 0; t < CT; ++t) {
#pragma unroll
        for (int n = 0; n < 2 * NDP; ++n) e[64 * (t * (2 * NDP + 1) + n)] = st.acc[t][n];
        e[64 * (t * (2 * NDP + 1) + 2 * NDP)] = f4{st.m[t], st.l[t][0], 0.f, 0.f};
    }
}
template <int NDP, int CT>
__device__ __forceinline__ void take_state(State<NDP, CT> &st, const float *ex, int lane, float scale2) {
    const f4 *e = reinterpret_cast<const f4 *>(ex) + lane;
#pragma unroll
    for (int t = 0; t < CT; ++t) {
        const f4 ml = e[64 * (t * (2 * NDP + 1) + 2 * NDP)];
        const float m = ml[0], M = fmaxf(st.m[t], m);
        const float f0 = st.m[t] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f((st.m[t] - M) * scale2);
        const float f1 = m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f((m - M) * scale2);
        st.m[t] = M;
        st.l[t] = st.l[t] * f0 + ml[1] * f1;
#pragma unroll
        for (int n = 0; n < 2 * NDP; ++n) st.acc[t][n] = st.acc[t][n] * f0 + e[64 * (t * (2 * NDP + 1) + n)] * f1;
    }
}

// Few rows: wave (head w % HG, part w / HG) takes the 16 CT rows of one of the
// tile's HG heads and turns of 16 NTL tokens, which it dequantises in registers.
// The heads of a token lie side by side in its cache row: read together they
// use whole 128-byte lines (a head alone has 64 bytes of codes and 4 of scales in
// a row at D = 128, and its neighbours would fetch the lines again: 135 against
// 102 us for 32 sequences of up to 16384 tokens). The
// parts of a head are merged in LDS, the upper half into the lower, by halves.
// Lane = token finds the pool rows and loads both scale rows, one load each,
// and passes them to the lanes that need them through LDS.
// Here the vector ALU counts, and codes cost it least with 8 added, where the
// e4m3 pattern is the number itself: K enters as (code + 8) 2^(s - 9) and a
// product of the lane's block scales with -8 times the sum of its query dims
// (in three bf16 parts) takes the excess out of the scores; V enters likewise,
// and a product of p with the offsets (State::w) takes it out at the end.
// fp32 queries keep the exact codes.
__host__ __device__ constexpr int rows_waves(int NDP, int CT) { return NDP * CT <= 4 ? 8 : 4; }
// f(0), f(1), ... f(N - 1) with constant arguments
template <int N, int I = 0, typename F>
__device__ __forceinline__ void unroll_sets(F f) {
    if constexpr (I < N) {
        f(std::integral_constant<int, I>{});
        unroll_sets<N, I + 1>(f);
    }
}
template <int NDP, int CT, int NTL, int SETS, int PARTS, bool FULL>
__global__ __launch_bounds__(64 * rows_waves(NDP, CT)) void k_tree_rows(TreeArgs a) {
    constexpr int PP = PARTS, NT = 2 * NDP, KB = Raw<NDP>::KB, VW = Raw<NDP>::VW, STEP = 16 * NTL;
    constexpr bool OFF = PARTS == 1;
    constexpr uint64_t ALL = ~0ull >> (64 - STEP);
    constexpr int NW = rows_waves(NDP, CT);
    __shared__ __attribute__((aligned(16))) float ex[NW / 2][CT * (NT + 1) * 256];
    __shared__ __attribute__((aligned(16))) int rowbuf[NW][SETS][STEP];
    __shared__ __attribute__((aligned(16))) uint32_t scbuf[NW][2][STEP][KB];           // scale rows of K, of V
    const int lane = threadIdx.x & 63, i = lane & 15, c = lane >> 4;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int nd = a.D / 32, parts = NW / a.HG, part = w / a.HG, turn = parts * STEP;
    for_each_piece(a, lane, [&](const Place &p) {
        State<NDP, CT> st;
#pragma unroll
        for (int t = 0; t < CT; ++t) {
            st.m[t] = -INFINITY;
            st.l[t] = f4{0.f, 0.f, 0.f, 0.f};
            st.w[t] = f4{0.f, 0.f, 0.f, 0.f};
            st.nan[t] = 0;
#pragma unroll
            for (int n = 0; n < NT; ++n) st.acc[t][n] = f4{0.f, 0.f, 0.f, 0.f};
        }
        const LaneAt<NDP> at(lane, a.D);
        const int g = p.g + (w - part * a.HG);
        const uint8_t *kc = a.kc + g * (a.D / 2), *vc = a.vc + g * (a.D / 2);
        const uint8_t *ks = a.ks + g * nd, *vs = a.vs + g * nd;
        const uint32_t cs = (uint32_t)a.Hkv * (a.D / 2), ss = (uint32_t)a.Hkv * nd;
        const int32_t *table = a.table + (int64_t)p.b * a.ldt;

        // pool row of token lt + lane (-1: past the range, or no valid page)
        auto page_at = [&](int lt) { return table[page_of(a, min(lt + lane, p.t1 - 1))]; };
        auto row_at = [&](int lt, int page) {
            const int t = lt + lane;
            return lane < STEP && t < p.t1 && (uint32_t)page < (uint64_t)a.pages ? page * a.ps + (t - page_of(a, t) * a.ps) : -1;
        };
        uint32_t k[SETS][NTL][NDP], v[SETS][NTL][4][VW], ksc[SETS][KB], vsc[SETS][KB];
        uint64_t valid[SETS];
        auto load_ks = [&](auto J, int row) {
            const uint64_t r = (uint32_t)max(row, 0);
            load_scales<NDP, FULL>(ksc[J], ks + r * ss, nd);
            load_scales<NDP, FULL>(vsc[J], vs + r * ss, nd);
#pragma unroll
            for (int u = 0; u < NTL; ++u)
                load_k<NDP>(k[J][u], kc + (uint64_t)(uint32_t)max(rowbuf[w][J][16 * u + i], 0) * cs, at);
        };
        auto load_vs = [&](auto J) {
#pragma unroll
            for (int u = 0; u < NTL; ++u)
#pragma unroll
                for (int s = 0; s < 4; ++s)
                    load_v<NDP>(v[J][u][s], vc + (uint64_t)(uint32_t)max(rowbuf[w][J][16 * u + 4 * c + s], 0) * cs, at);
        };
        auto rows_of = [&](auto J, int lt, int page) {
            const int row = row_at(lt, page);
            if (lane < STEP) rowbuf[w][J][lane] = row;
            return row;
        };

        bf8 qf[CT][NDP][PARTS], qoff[CT];
        int iq[CT], page = -1;
        // One step: the tokens at lt, whose codes are set J; the codes of the step
        // SETS turns on are loaded into J as it is used up
        auto step = [&](auto J, int lt) {
            const int next = lt + SETS * turn;
            if (lane < STEP) {
#pragma unroll
                for (int b = 0; b < KB; ++b) {
                    scbuf[w][0][lane][b] = ksc[J][b];
                    scbuf[w][1][lane][b] = vsc[J][b];
                }
            }
            const int row = rows_of(J, next, page);
            page = page_at(next + turn);
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            const uint8_t *kb = reinterpret_cast<const uint8_t *>(scbuf[w][0]);
            const uint8_t *vbp = reinterpret_cast<const uint8_t *>(scbuf[w][1]);

            f4 sc[CT][NTL];
#pragma unroll
            for (int u = 0; u < NTL; ++u) {
                uint32_t e[KB];
#pragma unroll
                for (int b = 0; b < KB; ++b) e[b] = kb[4 * KB * (16 * u + i) + at.kb[b]];
#pragma unroll
                for (int t = 0; t < CT; ++t) sc[t][u] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int b = 0; b < NDP; ++b) {
                    const bf8 kv = word_values<OFF>(k[J][u][b], scale_of(e[KB == 2 ? b >> 2 : 0]));
#pragma unroll
                    for (int t = 0; t < CT; ++t)
#pragma unroll
                        for (int j = 0; j < PARTS; ++j)
                            sc[t][u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kv, qf[t][b][j], sc[t][u], 0, 0, 0);
                }
                if constexpr (OFF) {
                    const bf8 es = scale_operand<NDP>(e);
#pragma unroll
                    for (int t = 0; t < CT; ++t)
                        sc[t][u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(es, qoff[t], sc[t][u], 0, 0, 0);
                }
            }
            uint32_t vb[NTL][4];
#pragma unroll
            for (int u = 0; u < NTL; ++u)
#pragma unroll
                for (int s = 0; s < 4; ++s) vb[u][s] = vbp[4 * KB * (16 * u + 4 * c + s) + at.vb];
            load_ks(J, row);
            __builtin_amdgcn_sched_barrier(0);

            if (valid[J] != ALL || lt + STEP > p.ctx) {
                uint64_t seen[CT];
#pragma unroll
                for (int t = 0; t < CT; ++t) seen[t] = valid[J] & mask_window(a, p, iq[t], lt);
                hide<CT, NTL>(sc, seen, c);
#pragma unroll
                for (int u = 0; u < NTL; ++u)
#pragma unroll
                    for (int s = 0; s < 4; ++s) {
                        if (!((valid[J] >> (16 * u + 4 * c + s)) & 1)) vb[u][s] = 0;
                        const uint64_t bad = take_nan(vb[u][s]);
                        if (bad)
                            for (int j = 0; j < 4; ++j)
                                note_nan<NDP, CT>(st, (uint32_t)(bad >> (16 * j)) & 0xFFFFu, 16 * u + 4 * j + s, seen, c);
                    }
            }
            soften<NDP, CT, NTL, PARTS == 3>(st, sc, a.scale2);
#pragma unroll
            for (int u = 0; u < NTL; u += 2) {
                bf8 vf[NT], off;
                v_operands<NDP, OFF>(&v[J][u], &vb[u], vf, off);
#pragma unroll
                for (int t = 0; t < CT; ++t) {
                    bf8 pf[PP];
                    p_operands<PP>(sc[t][u], sc[t][u + 1], pf);
#pragma unroll
                    for (int j = 0; j < PP; ++j)
                        st.l[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ones(), pf[j], st.l[t], 0, 0, 0);
                    if constexpr (OFF)
                        st.w[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(off, pf[0], st.w[t], 0, 0, 0);
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int j = 0; j < PP; ++j)
                            st.acc[t][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf[n], pf[j], st.acc[t][n], 0, 0, 0);
                }
            }
            load_vs(J);
            valid[J] = __ballot(row >= 0);
            __builtin_amdgcn_sched_barrier(0);
        };

        int lt = p.t0 + part * STEP;
        if (lt < p.t1) {
            int pages[SETS];
#pragma unroll
            for (int j = 0; j < SETS; ++j) pages[j] = page_at(lt + j * turn);
            RawQueries<NDP, CT, PARTS> rq;
            rq.load(a, p, g, p.row, lane);
            unroll_sets<SETS>([&](auto J) {
                const int row = rows_of(J, lt + J * turn, pages[J]);
                valid[J] = __ballot(row >= 0);
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                load_ks(J, row);
                load_vs(J);
            });
            page = page_at(lt + SETS * turn);
            rq.operands(a, lane, qf);
#pragma unroll
            for (int t = 0; t < CT; ++t) {
                iq[t] = max(rq.i[t], 0);
                if constexpr (OFF) qoff[t] = query_sums<NDP>(qf[t]);
            }
            for (; lt < p.t1; lt += SETS * turn)
                unroll_sets<SETS>([&](auto J) {
                    if (J == 0 || lt + J * turn < p.t1) step(J, lt + J * turn);
                });
        }
        if constexpr (OFF) take_offset<NDP, CT>(st);
        give_nan<NDP, CT>(st);

        for (int half = parts / 2; half; half /= 2) {
            if (part >= half && part < 2 * half) give_state<NDP, CT>(st, ex[w - half * a.HG], lane);
            __syncthreads();
            if (part < half) take_state<NDP, CT>(st, ex[w], lane, a.scale2);
            __syncthreads();
        }
        if (part == 0) store_rows<NDP, CT, PARTS>(a, p, st, g, p.row, lane);
    });
}

// Order of a block of N LDS reads that feed M matrix instructions each: six
// reads ahead. Left alone, the compiler reads each operand right before its use
// and waits out the LDS latency every time.
template <int N, int M>
__device__ __forceinline__ void pipeline() {
    constexpr int AHEAD = N < 6 ? N : 6;
    __builtin_amdgcn_sched_group_barrier(0x100, AHEAD, 0);
    unroll_sets<N - AHEAD>([](auto) {
        __builtin_amdgcn_sched_group_barrier(0x008, M, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
    });
    __builtin_amdgcn_sched_group_barrier(0x008, M * AHEAD, 0);
}

// Many rows: the four waves of a workgroup share every 64-token stage. Each
// dequantises one 16-token tile of K and of V into LDS, in the operands' own
// lane order (64 lanes x 16 bytes an operand: reads without bank conflicts),
// then multiplies all of the stage (or half of it, WT = 2) with its own 16 CT
// rows. Two LDS buffers: one barrier a stage, the next stage's codes in flight
// meanwhile. With WT = 2 the two waves of a row tile are merged at the end.
template <int NDP>
struct TileLds {
    static constexpr int NT = 2 * NDP, TILES = kStep / 16;
    uint32_t k[2][TILES * NDP][64][4];
    uint32_t v[2][TILES / 2 * NT][64][4];
    uint64_t nan[2][TILES][4];
    uint32_t valid[2][TILES];
};

template <int NDP, int CT, int WT, int PARTS>
__global__ __launch_bounds__(256, NDP == 8 ? 1 : 2) void k_tree_tile(TreeArgs a) {
    constexpr int PP = PARTS, NT = 2 * NDP, WR = 4 / WT, NTW = kNTL / WT;
    constexpr int KB = Raw<NDP>::KB, VW = Raw<NDP>::VW;
    extern __shared__ __attribute__((aligned(16))) unsigned char lds_raw[];
    auto &lds = *reinterpret_cast<TileLds<NDP> *>(lds_raw);
    const int lane = threadIdx.x & 63, i = lane & 15, c = lane >> 4;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wr = w % WR, wt = w / WR;
    for_each_piece(a, lane, [&](const Place &p) {
    const int row0 = p.row + wr * 16 * CT;
    const bool busy = row0 < p.n * a.G;

    State<NDP, CT> st;
#pragma unroll
    for (int t = 0; t < CT; ++t) {
        st.m[t] = -INFINITY;
        st.l[t] = f4{0.f, 0.f, 0.f, 0.f};
        st.w[t] = f4{0.f, 0.f, 0.f, 0.f};
        st.nan[t] = 0;
#pragma unroll
        for (int n = 0; n < NT; ++n) st.acc[t][n] = f4{0.f, 0.f, 0.f, 0.f};
    }
    if (p.t0 < p.t1) {
        const LaneAt<NDP> at(lane, a.D);
        const uint8_t *kc = a.kc + p.g * (a.D / 2), *vc = a.vc + p.g * (a.D / 2);
        const uint8_t *ks = a.ks + p.g * (a.D / 32), *vs = a.vs + p.g * (a.D / 32);
        const int32_t *table = a.table + (int64_t)p.b * a.ldt;
        const uint32_t cs = (uint32_t)a.Hkv * (a.D / 2), ss = (uint32_t)a.Hkv * (a.D / 32);

        // token 16 w + i of the stage at lt: its page, its pool row
        auto page_at = [&](int lt) { return table[page_of(a, min(lt + 16 * w + i, p.t1 - 1))]; };
        auto row_at = [&](int lt, int page) {
            const int t = lt + 16 * w + i;
            return t < p.t1 && (uint32_t)page < (uint64_t)a.pages ? page * a.ps + (t - page_of(a, t) * a.ps) : -1;
        };
        uint32_t k[NDP], kb[KB], v[4][VW], vb[4];
        auto load = [&](int row) {
            const uint64_t r = (uint32_t)max(row, 0);
            load_k<NDP>(k, kc + r * cs, at);
#pragma unroll
            for (int b = 0; b < KB; ++b) kb[b] = ks[r * ss + at.kb[b]];
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const uint64_t rv = (uint32_t)max(__shfl(row, 4 * c + s), 0);
                load_v<NDP>(v[s], vc + rv * cs, at);
                vb[s] = vs[rv * ss + at.vb];
            }
        };

        int page = page_at(p.t0);
        RawQueries<NDP, CT, PARTS> rq;
        rq.load(a, p, p.g, row0, lane);
        int row = row_at(p.t0, page);
        load(row);
        page = page_at(p.t0 + kStep);
        bf8 qf[CT][NDP][PARTS];
        rq.operands(a, lane, qf);
        int iq[CT];
#pragma unroll
        for (int t = 0; t < CT; ++t) iq[t] = max(rq.i[t], 0);
        int buf = 0;
        for (int lt = p.t0; lt < p.t1; lt += kStep, buf ^= 1) {
            // this wave's tiles into LDS
            const uint32_t ok = (uint32_t)__ballot(row >= 0) & 0xFFFFu;
            const bool edge = lt + kStep > p.ctx || lt + kStep > p.t1;
            if (lane == 0) lds.valid[buf][w] = ok;
#pragma unroll
            for (int b = 0; b < NDP; ++b)
                *reinterpret_cast<bf8 *>(lds.k[buf][w * NDP + b][lane]) =
                    word_values<false>(k[b], scale_of(kb[KB == 2 ? b >> 2 : 0]));
            __builtin_amdgcn_sched_barrier(0);
            if (edge || ok != 0xFFFFu) {
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    if (!((ok >> (4 * c + s)) & 1)) vb[s] = 0;
                    if (edge) {
                        const uint64_t bad = take_nan(vb[s]);
                        if (lane == 0) lds.nan[buf][w][s] = bad;
                    }
                }
            }
            {
                uint32_t o[NT][2];
                float vsc[4];
#pragma unroll
                for (int s = 0; s < 4; ++s) vsc[s] = scale_of(vb[s]);
                v_pairs<NDP, false>(v, vsc, o);
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    *reinterpret_cast<u2 *>(&lds.v[buf][(w >> 1) * NT + n][lane][2 * (w & 1)]) = u2{o[n][0], o[n][1]};
            }
            __builtin_amdgcn_sched_barrier(0);
            row = row_at(lt + kStep, page);
            page = page_at(lt + 2 * kStep);
            load(row);
            lds_barrier();
            if (!busy) continue;

            f4 sc[CT][NTW];
#pragma unroll
            for (int u = 0; u < NTW; ++u) {
#pragma unroll
                for (int t = 0; t < CT; ++t) sc[t][u] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int b = 0; b < NDP; ++b) {
                    const bf8 kv = *reinterpret_cast<const bf8 *>(lds.k[buf][(wt * NTW + u) * NDP + b][lane]);
#pragma unroll
                    for (int t = 0; t < CT; ++t)
#pragma unroll
                        for (int j = 0; j < PARTS; ++j)
                            sc[t][u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kv, qf[t][b][j], sc[t][u], 0, 0, 0);
                }
            }
            pipeline<NTW * NDP, CT * PARTS>();
            // V operand j = (tiles, n) of the wave's tokens, VP of them read ahead
            constexpr int VP = 4;
            auto v_at = [&](int j) {
                return *reinterpret_cast<const bf8 *>(lds.v[buf][(wt * NTW / 2 + j / NT) * NT + j % NT][lane]);
            };
            bf8 vf[VP];
#pragma unroll
            for (int j = 0; j < VP; ++j) vf[j] = v_at(j);
            __builtin_amdgcn_sched_barrier(0);
            const uint64_t valid = (uint64_t)(lds.valid[buf][0] | lds.valid[buf][1] << 16) |
                                   (uint64_t)(lds.valid[buf][2] | lds.valid[buf][3] << 16) << 32;
            if (valid != ~0ull || edge) {
                uint64_t seen[CT];
#pragma unroll
                for (int t = 0; t < CT; ++t) seen[t] = (valid & mask_window(a, p, iq[t], lt)) >> (16 * NTW * wt);
                hide<CT, NTW>(sc, seen, c);
                if (edge)
                    for (int u = 0; u < NTW; ++u)
                        for (int s = 0; s < 4; ++s) {
                            const uint64_t bad = lds.nan[buf][wt * NTW + u][s];
                            if (bad)
                                for (int j = 0; j < 4; ++j)
                                    note_nan<NDP, CT>(st, (uint32_t)(bad >> (16 * j)) & 0xFFFFu, 16 * u + 4 * j + s, seen,
                                                      c);
                        }
            }
            soften<NDP, CT, NTW, PARTS == 3>(st, sc, a.scale2);
#pragma unroll
            for (int u = 0; u < NTW; u += 2) {
                bf8 pf[CT][PP];
#pragma unroll
                for (int t = 0; t < CT; ++t) {
                    p_operands<PP>(sc[t][u], sc[t][u + 1], pf[t]);
#pragma unroll
                    for (int j = 0; j < PP; ++j)
                        st.l[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ones(), pf[t][j], st.l[t], 0, 0, 0);
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const int j = u / 2 * NT + n;
                    const bf8 vv = vf[j % VP];
                    if (j + VP < NTW / 2 * NT) vf[j % VP] = v_at(j + VP);
#pragma unroll
                    for (int t = 0; t < CT; ++t)
#pragma unroll
                        for (int k = 0; k < PP; ++k)
                            st.acc[t][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vv, pf[t][k], st.acc[t][n], 0, 0, 0);
                }
            }
        }
    }
    give_nan<NDP, CT>(st);
    if constexpr (WT == 2) {
        __syncthreads();
        float *ex = reinterpret_cast<float *>(lds_raw) + wr * CT * (NT + 1) * 256;
        if (wt == 1) give_state<NDP, CT>(st, ex, lane);
        __syncthreads();
        if (wt == 0) take_state<NDP, CT>(st, ex, lane, a.scale2);
    }
    if (busy && wt == 0) store_rows<NDP, CT, PARTS>(a, p, st, p.g, row0, lane);
    __syncthreads();                 // the next piece writes the same LDS
    });
}

// Most rows: eight waves, 256 (CT 1: 128) rows. Two halves of the workgroup take
// turns: in every phase one half feeds the matrix cores (p V of the stage before
// and the scores of this one, all from LDS) while the other half uses the vector
// ALU (softmax, dequantising the next stage, addresses), and a barrier swaps
// them. Left to themselves the waves run through the same kind of work
// together, and each unit idles in turn. Half 0 dequantises K, half 1 V:
//   phase  2 k      half 0: PV(k - 1), QK(k)          half 1: V(k), softmax(k - 1)
//   phase  2 k + 1  half 0: K(k + 1), softmax(k)      half 1: PV(k - 1), QK(k)
// so two LDS buffers serve: K(k) is read in phases 2 k and 2 k + 1 and written
// again in 2 k + 3; V(k) is read in 2 k + 2 and 2 k + 3, written again in 2 k + 4.
// 16 x 64 drafted tokens over up to 16384 (8 query heads): four waves without
// turns 500 us; eight waves without turns, one barrier a stage, 488; turns 516,
// with the matrix half's waves first in issue 470; on a slower card 500, with the
// next stage's tiles written before the softmax 474. No unit is near its limit:
// of the call's 1.03 million cycles the matrix cores are busy in 37 %, the vector
// ALU issues in at most 53 %, LDS serves the operands (256 KiB a stage) in 27 %.
// The phases overlap too little. Waves whose rows lie past the tile's end go
// through the same work (8 x 26 drafted tokens: 208 rows at most in tiles of 256,
// 31 % of the cycles matrix, 50 % vector, 22 % LDS).
template <int NDP, int CT, int PARTS>
__global__ __launch_bounds__(512) void k_tree_pair(TreeArgs a) {
    constexpr int PP = PARTS, NT = 2 * NDP, NTW = kNTL;
    constexpr int KB = Raw<NDP>::KB, VW = Raw<NDP>::VW, VP = 4;
    extern __shared__ __attribute__((aligned(16))) unsigned char lds_raw[];
    auto &lds = *reinterpret_cast<TileLds<NDP> *>(lds_raw);
    const int lane = threadIdx.x & 63, i = lane & 15, c = lane >> 4;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int half = w >> 2, tw = w & 3;                 // the tile of K or V that this wave dequantises
    for_each_piece(a, lane, [&](const Place &p) {
        const int row0 = p.row + w * 16 * CT;
        const bool busy = row0 < p.n * a.G;
        State<NDP, CT> st;
#pragma unroll
        for (int t = 0; t < CT; ++t) {
            st.m[t] = -INFINITY;
            st.l[t] = f4{0.f, 0.f, 0.f, 0.f};
            st.w[t] = f4{0.f, 0.f, 0.f, 0.f};
            st.nan[t] = 0;
#pragma unroll
            for (int n = 0; n < NT; ++n) st.acc[t][n] = f4{0.f, 0.f, 0.f, 0.f};
        }
        if (p.t0 < p.t1) {
            const LaneAt<NDP> at(lane, a.D);
            const uint8_t *codes = (half ? a.vc : a.kc) + p.g * (a.D / 2);
            const uint8_t *scales = (half ? a.vs : a.ks) + p.g * (a.D / 32);
            const int32_t *table = a.table + (int64_t)p.b * a.ldt;
            const uint32_t cs = (uint32_t)a.Hkv * (a.D / 2), ss = (uint32_t)a.Hkv * (a.D / 32);
            const int N = (p.t1 - p.t0 + kStep - 1) / kStep;             // stages
            auto page_at = [&](int lt) { return table[page_of(a, min(lt + 16 * tw + i, p.t1 - 1))]; };
            auto row_at = [&](int lt, int page) {
                const int t = lt + 16 * tw + i;
                return t < p.t1 && (uint32_t)page < (uint64_t)a.pages ? page * a.ps + (t - page_of(a, t) * a.ps) : -1;
            };
            // codes and scales of this wave's tile: K as the lane's words of one
            // token, V as the lane's words of four
            constexpr int RW = NDP > 4 * VW ? NDP : 4 * VW;
            uint32_t raw[RW], rb[4];
            auto load = [&](int row) {
                if (half == 0) {
                    const uint64_t r = (uint32_t)max(row, 0);
                    load_k<NDP>(raw, codes + r * cs, at);
#pragma unroll
                    for (int b = 0; b < KB; ++b) rb[b] = scales[r * ss + at.kb[b]];
                } else {
#pragma unroll
                    for (int s = 0; s < 4; ++s) {
                        const uint64_t r = (uint32_t)max(__shfl(row, 4 * c + s), 0);
                        load_v<NDP>(raw + s * VW, codes + r * cs, at);
                        rb[s] = scales[r * ss + at.vb];
                    }
                }
            };
            int page = page_at(p.t0);
            RawQueries<NDP, CT, PARTS> rq;
            rq.load(a, p, p.g, row0, lane);
            int row = row_at(p.t0, page);
            load(row);
            page = page_at(p.t0 + kStep);
            bf8 qf[CT][NDP][PARTS];
            rq.operands(a, lane, qf);
            int iq[CT];
#pragma unroll
            for (int t = 0; t < CT; ++t) iq[t] = max(rq.i[t], 0);

            // stage k's tile of this wave into LDS, stage k + 1's loads under way
            auto stage = [&](int k) {
                const int lt = p.t0 + k * kStep, buf = k & 1;
                const uint32_t ok = (uint32_t)__ballot(row >= 0) & 0xFFFFu;
                if (half == 0) {
                    if (lane == 0) lds.valid[buf][tw] = ok;
#pragma unroll
                    for (int b = 0; b < NDP; ++b)
                        *reinterpret_cast<bf8 *>(lds.k[buf][tw * NDP + b][lane]) =
                            word_values<false>(raw[b], scale_of(rb[KB == 2 ? b >> 2 : 0]));
                } else {
                    if (lt + kStep > p.ctx || lt + kStep > p.t1 || ok != 0xFFFFu) {
#pragma unroll
                        for (int s = 0; s < 4; ++s) {
                            if (!((ok >> (4 * c + s)) & 1)) rb[s] = 0;
                            if (lt + kStep > p.ctx || lt + kStep > p.t1) {
                                const uint64_t bad = take_nan(rb[s]);
                                if (lane == 0) lds.nan[buf][tw][s] = bad;
                            }
                        }
                    }
                    uint32_t v[4][VW], o[NT][2];
                    float vsc[4];
#pragma unroll
                    for (int s = 0; s < 4; ++s) {
                        vsc[s] = scale_of(rb[s]);
#pragma unroll
                        for (int b = 0; b < VW; ++b) v[s][b] = raw[s * VW + b];
                    }
                    v_pairs<NDP, false>(v, vsc, o);
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        *reinterpret_cast<u2 *>(&lds.v[buf][(tw >> 1) * NT + n][lane][2 * (tw & 1)]) = u2{o[n][0], o[n][1]};
                }
                __builtin_amdgcn_sched_barrier(0);
                row = row_at(lt + kStep, page);
                page = page_at(lt + 2 * kStep);
                load(row);
            };

            f4 sc[CT][NTW];
            bf8 pf[NTW / 2][CT][PP];
            // p V of a stage
            auto values = [&](int vbuf) {
                auto v_at = [&](int j) { return *reinterpret_cast<const bf8 *>(lds.v[vbuf][j][lane]); };
                bf8 vf[VP];
#pragma unroll
                for (int j = 0; j < VP; ++j) vf[j] = v_at(j);
#pragma unroll
                for (int u = 0; u < NTW / 2; ++u) {
#pragma unroll
                    for (int t = 0; t < CT; ++t)
#pragma unroll
                        for (int j = 0; j < PP; ++j)
                            st.l[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ones(), pf[u][t][j], st.l[t], 0, 0, 0);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const int j = u * NT + n;
                        const bf8 vv = vf[j % VP];
                        if (j + VP < NTW / 2 * NT) vf[j % VP] = v_at(j + VP);
#pragma unroll
                        for (int t = 0; t < CT; ++t)
#pragma unroll
                            for (int q = 0; q < PP; ++q)
                                st.acc[t][n] =
                                    __builtin_amdgcn_mfma_f32_16x16x32_bf16(vv, pf[u][t][q], st.acc[t][n], 0, 0, 0);
                    }
                }
            };
            // scores of a stage
            auto scores = [&](int kb) {
                auto k_at = [&](int j) { return *reinterpret_cast<const bf8 *>(lds.k[kb][j][lane]); };
                bf8 kf[VP];
#pragma unroll
                for (int j = 0; j < VP; ++j) kf[j] = k_at(j);
#pragma unroll
                for (int u = 0; u < NTW; ++u) {
#pragma unroll
                    for (int t = 0; t < CT; ++t) sc[t][u] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int b = 0; b < NDP; ++b) {
                        const int j = u * NDP + b;
                        const bf8 kv = kf[j % VP];
                        if (j + VP < NTW * NDP) kf[j % VP] = k_at(j + VP);
#pragma unroll
                        for (int t = 0; t < CT; ++t)
#pragma unroll
                            for (int q = 0; q < PARTS; ++q)
                                sc[t][u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kv, qf[t][b][q], sc[t][u], 0, 0, 0);
                    }
                }
            };
            // vector half of stage k: its softmax
            auto weigh = [&](int k) {
                const int lt = p.t0 + k * kStep, buf = k & 1;
                const bool edge = lt + kStep > p.ctx || lt + kStep > p.t1;
                const uint64_t valid = (uint64_t)(lds.valid[buf][0] | lds.valid[buf][1] << 16) |
                                       (uint64_t)(lds.valid[buf][2] | lds.valid[buf][3] << 16) << 32;
                if (valid != ~0ull || edge) {
                    uint64_t seen[CT];
#pragma unroll
                    for (int t = 0; t < CT; ++t) seen[t] = valid & mask_window(a, p, iq[t], lt);
                    hide<CT, NTW>(sc, seen, c);
                    if (edge)
                        for (int u = 0; u < NTW; ++u)
                            for (int s = 0; s < 4; ++s) {
                                const uint64_t bad = lds.nan[buf][u][s];
                                if (bad)
                                    for (int j = 0; j < 4; ++j)
                                        note_nan<NDP, CT>(st, (uint32_t)(bad >> (16 * j)) & 0xFFFFu, 16 * u + 4 * j + s,
                                                          seen, c);
                            }
                }
                soften<NDP, CT, NTW, PARTS == 3>(st, sc, a.scale2);
#pragma unroll
                for (int u = 0; u < NTW; u += 2)
#pragma unroll
                    for (int t = 0; t < CT; ++t) p_operands<PP>(sc[t][u], sc[t][u + 1], pf[u / 2][t]);
            };

            stage(0);
            // every wave meets the same 2 N + 2 barriers; half 1 is a phase behind
            if (half) lds_barrier();
            lds_barrier();
            scores(0);
            lds_barrier();
            stage(1);
            weigh(0);
            for (int k = 1; k < N; ++k) {
                lds_barrier();
                __builtin_amdgcn_s_setprio(1);       // the matrix half issues first
                values((k & 1) ^ 1);
                scores(k & 1);
                __builtin_amdgcn_s_setprio(0);
                lds_barrier();
                stage(k + 1);        // past the last stage: its rows are clamped, its tiles not read
                weigh(k);
            }
            lds_barrier();
            values((N & 1) ^ 1);
            if (!half) lds_barrier();
        }
        give_nan<NDP, CT>(st);
        if (busy) store_rows<NDP, CT, PARTS>(a, p, st, p.g, row0, lane);
        __syncthreads();                 // the next piece writes the same LDS
    });
}

// Rows of tiles that lie in several shares: out = sum_s O_s 2^(m_s - M) 2^9 /
// sum_s l_s 2^(m_s - M). Workgroup (x, y): the tile of todo entry x, JR of its
// rows from y JR on. A group of LR >= D / 4 lanes holds
// a row (four dims a lane) and every SL-th piece; the SL groups of a row are
// added in LDS in order. Few pieces: many rows at a time; many: many groups a row.
template <typename T>
__global__ __launch_bounds__(256) void k_tree_join(TreeArgs a) {
    __shared__ __attribute__((aligned(16))) f4 so[256];
    __shared__ float2 sml[32];
    const int tid = threadIdx.x;
    const int *e = a.todo + 8 * (int64_t)blockIdx.x;
    const JoinOf t = {e[0], e[1], e[2], e[3], e[4], e[5]};
    if (a.NT) {                                          // is there such a tile?
        const int per = a.groups * a.nrt, b = blockIdx.x / per, rt = blockIdx.x % a.nrt;
        if ((uint32_t)rt >= seq_of(a, b).nrt) return;
    } else if ((int)blockIdx.x >= a.todo[8 * a.P]) {
        return;
    }
    const int p0 = t.first;
    if (t.last <= p0) return;
    const int SR = a.HG * a.R, ns = t.last - p0 + 1;
    const int LR = a.D <= 32 ? 8 : (a.D <= 64 ? 16 : (a.D <= 128 ? 32 : 64)), groups = 256 / LR;
    int SL = 1;
    while (4 * SL < ns && 2 * SL <= groups) SL *= 2;
    const int grp = tid / LR, sl = grp % SL, d = 4 * (tid % LR) < a.D ? 4 * (tid % LR) : 0;
    const bool mine = 4 * (tid % LR) < a.D;
    // every thread makes the same number of turns: the barriers are inside
    for (int k0 = 0; k0 < a.JR; k0 += groups / SL) {
        const int k = k0 + grp / SL, in = blockIdx.y * a.JR + k;
        const int gi = in / a.R, row = t.row + in - gi * a.R;
        const bool on = k < a.JR && in < SR && row < t.n * a.G;
        float M = -INFINITY, L = 0.f;
        f4 o = {0.f, 0.f, 0.f, 0.f};
        if (on)
            for (int s0 = sl; s0 < ns; s0 += 4 * SL) {
                float m[4], l[4];
                f4 v[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int s = s0 + j * SL < ns ? s0 + j * SL : ns - 1;
                    // slot 1 of the tile's first share, slot 0 of the others
                    const int64_t at = (2 * (int64_t)(p0 + s) + (s == 0 ? 1 : 0)) * SR + in;
                    const float2 ml = reinterpret_cast<const float2 *>(a.pml)[at];
                    m[j] = s0 + j * SL < ns ? ml.x : -INFINITY;
                    l[j] = ml.y;
                    v[j] = *reinterpret_cast<const f4 *>(a.po + at * a.D + d);
                }
                const float Mn = fmaxf(fmaxf(fmaxf(M, m[0]), fmaxf(m[1], m[2])), m[3]);
                const float f0 = M == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(M - Mn);
                L *= f0;
                o *= f0;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (s0 + j * SL >= ns) continue;
                    const float f = m[j] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m[j] - Mn);
                    L += l[j] * f;
                    o += v[j] * f;
                }
                M = Mn;
            }
        if (SL > 1) {
            so[tid] = o;
            if (tid % LR == 0) sml[grp] = make_float2(M, L);
            __syncthreads();
            if (sl == 0) {
                for (int j = 1; j < SL; ++j) M = fmaxf(M, sml[grp + j].x);
                const float own = sml[grp].x, f0 = own == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(own - M);
                L *= f0;
                o *= f0;
                for (int j = 1; j < SL; ++j) {
                    const float2 ml = sml[grp + j];
                    const float f = ml.x == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(ml.x - M);
                    L += ml.y * f;
                    o += so[tid + j * LR] * f;
                }
            }
            __syncthreads();
        }
        if (on && mine && sl == 0) {
            const int i = row / a.G, h = (t.g + gi) * a.G + row - i * a.G;
            const float norm = M == -INFINITY ? 0.f : 512.f / L;
            T *out = static_cast<T *>(a.out) + ((int64_t)t.q0 + i) * a.ldo + (int64_t)h * a.D + d;
#pragma unroll
            for (int j = 0; j < 4; ++j) out[j] = (T)(o[j] * norm);
        }
    }
}

struct TreePlan {
    int NDP, CT, NW, WT;             // WT 0: k_tree_rows; NW 8: k_tree_pair
    int R, U, P, HG;
    int ms, cap;
    int64_t nrt;
    int64_t bound;                   // units at most (kMostUnits + 1: more than the device counts)
    int join;                        // some tile may lie in several shares
};

// The device counts rows and units in 32 bits. Sizes that are each allowed have
// products past 64 bits, so the host stops counting at kMostUnits + 1.
constexpr int64_t kMostUnits = 1 << 30;
int64_t count(int64_t a, int64_t b) {
    int64_t r;
    return __builtin_mul_overflow(a, b, &r) || r > kMostUnits ? kMostUnits + 1 : r;
}

// Kernel, tile and number of workgroups from what the host knows: eight waves
// (four where one needs more than 256 registers) fit on each of the 256 CUs.
TreePlan tree_plan(mxs_dtype dt, int64_t B, int64_t max_q, int64_t max_len, int64_t Hq, int64_t Hkv, int64_t D) {
    TreePlan p;
    p.NDP = D <= 64 ? 2 : (D <= 128 ? 4 : 8);
    const int64_t rows = count(max_q, Hq / Hkv);
    const bool bf = dt == MXS_BF16;
    int64_t slots;
    // Up to 16 rows every wave takes its own tokens (against stages in LDS at 8
    // sequences of 8192 tokens, 8 heads of 128 bf16: 8 rows 27.3, 41.4 us, 16 rows
    // 29.5, 42.2; fp32 38.4, 42.6). From 17 to 32 the batch decides: 24 rows of 32
    // sequences of 500 and 16384 tokens take 17.5 against 23.6 and 217 against 246
    // us (heads of 64: 130, 187), but 8 sequences of 500 and 2048 17.4 against
    // 16.2 and 28.3 against 23.5, for a stage feeds four waves from few tokens.
    if (rows <= 16 || (rows <= 32 && bf && p.NDP <= 4 && B * Hkv >= 256)) {
        p.WT = 0;
        p.CT = rows > 16 ? 2 : 1;
        p.R = 16 * p.CT;
        const int nw = rows_waves(p.NDP, p.CT);
        // heads that fill two 128-byte lines of codes; fewer where that would
        // leave less than 256 workgroups at 32 pieces a tile
        p.ms = 0;
        p.cap = 6;
        p.HG = D <= 64 ? 8 : (D <= 128 ? 4 : 2);
        while (p.HG > 1 && (p.HG > nw || Hkv % p.HG || B * (Hkv / p.HG) * 32 < 256)) p.HG /= 2;
        p.U = nw / p.HG * 16 * kRowTiles;
        if (max_len <= 512) {        // one workgroup a head, no join: 11.9 against 13.1 us at 500 tokens
            p.HG = 1;
            for (p.U = 64; p.U < max_len; p.U *= 2) {}
        }
        slots = 256;
    } else {
        // Graph replays at 8 sequences of 8192 tokens, heads of 128: 64 bf16 rows in
        // two row groups of two waves each 51.4 us, in four of one 60.0 (fp32, 32
        // rows: 49.8, 63.1); 256 rows by pairs of waves 103.0, by four waves 113.0
        // (fp32, 128 rows: 110, 118), 128 rows alike.
        p.CT = bf ? 2 : 1;
        p.NW = rows > 64 * p.CT && p.NDP <= 4 ? 8 : 4;
        p.WT = rows <= 32 * p.CT ? 2 : 1;
        p.R = 16 * p.CT * (p.NW / p.WT);
        p.HG = 1;
        p.U = kStep;
        p.ms = 1;
        p.cap = 5;
        slots = p.NDP == 8 || p.NW == 8 ? 256 : 512;
    }
    const int64_t T = max_len > 0 ? ceil_div(max_len, (int64_t)p.U) : 1;
    p.nrt = ceil_div(rows, (int64_t)p.R);
    p.bound = count(count(count(B, Hkv / p.HG), p.nrt), T);
    for (p.P = 8; p.P < slots && ((int64_t)p.P << p.ms) < p.bound;) p.P *= 2;
    p.join = T > 1;
    return p;
}

template <int NDP, int CT, int PARTS>
hipError_t rows_go(const TreeArgs &a, unsigned grid, hipStream_t st) {
    if (a.D == 32 * NDP)
        hipLaunchKernelGGL((k_tree_rows<NDP, CT, kRowTiles, kRowSets, PARTS, true>), dim3(grid),
                           dim3(64 * rows_waves(NDP, CT)), 0, st, a);
    else
        hipLaunchKernelGGL((k_tree_rows<NDP, CT, kRowTiles, kRowSets, PARTS, false>), dim3(grid),
                           dim3(64 * rows_waves(NDP, CT)), 0, st, a);
    return hipGetLastError();
}
template <int NDP, int CT, int WT, int PARTS>
hipError_t tile_go(const TreeArgs &a, unsigned grid, hipStream_t st) {
    constexpr size_t lds = sizeof(TileLds<NDP>);
    static_assert(WT == 1 || lds >= (size_t)2 * CT * (2 * NDP + 1) * 1024, "merge space");
    hipLaunchKernelGGL((k_tree_tile<NDP, CT, WT, PARTS>), dim3(grid), dim3(256), lds, st, a);
    return hipGetLastError();
}
template <int NDP, int CT, int PARTS>
hipError_t tile_go(const TreePlan &p, const TreeArgs &a, unsigned grid, hipStream_t st) {
    if constexpr (NDP <= 4)
        if (p.NW == 8) {
            hipLaunchKernelGGL((k_tree_pair<NDP, CT, PARTS>), dim3(grid), dim3(512),
                               sizeof(TileLds<NDP>), st, a);
            return hipGetLastError();
        }
    return p.WT == 1 ? tile_go<NDP, CT, 1, PARTS>(a, grid, st) : tile_go<NDP, CT, 2, PARTS>(a, grid, st);
}
template <int NDP>
hipError_t tree_go(const TreePlan &p, const TreeArgs &a, unsigned grid, bool f32, hipStream_t st) {
    if (f32) return p.WT == 0 ? rows_go<NDP, 1, 3>(a, grid, st) : tile_go<NDP, 1, 3>(p, a, grid, st);
    if (p.WT) return tile_go<NDP, 2, 1>(p, a, grid, st);
    if constexpr (NDP <= 4)
        if (p.CT == 2) return rows_go<NDP, 2, 1>(a, grid, st);
    return rows_go<NDP, 1, 1>(a, grid, st);
}

}  // namespace

size_t attend_kv4_tree_workspace(mxs_dtype dt, int64_t B, int64_t max_q, int64_t max_len, int64_t Hq, int64_t Hkv,
                                 int64_t D) {
    const TreePlan p = tree_plan(dt, B, max_q, max_len, Hq, Hkv, D);
    // pieces (outputs, then maxima and sums), then todo
    return p.join ? (size_t)(2 * p.P) * p.HG * p.R * (D + 2) * sizeof(float) + (size_t)(p.P + 1) * 32 : 0;
}

bool attend_kv4_tree_supported(mxs_dtype dt, int64_t B, int64_t max_q, int64_t max_len, int64_t Hq, int64_t Hkv,
                               int64_t D) {
    return count(max_q, Hq / Hkv) <= kMostUnits && tree_plan(dt, B, max_q, max_len, Hq, Hkv, D).bound <= kMostUnits;
}

hipError_t launch_attend_kv4_tree(const void *q, mxs_dtype dt, int64_t ldq, const mxs_kv4_cache &c,
                                  const int32_t *table, int64_t ldt, const int32_t *lens, const int32_t *cu,
                                  const uint64_t *mask, int64_t words, int64_t B, int64_t total_q, int64_t max_q,
                                  int64_t max_len, int64_t Hq, float scale, void *out, int64_t ldo, void *ws,
                                  hipStream_t st) {
    const TreePlan p = tree_plan(dt, B, max_q, max_len, Hq, c.H, c.D);
    TreeArgs a{};
    const int es = dt == MXS_BF16 ? 2 : 4;
    a.q = q; a.ldq = ldq;
    a.qvec = reinterpret_cast<uintptr_t>(q) % 16 == 0 && (ldq * es % 16 == 0 || total_q == 1); a.kc = c.kc; a.ks = c.ks; a.vc = c.vc; a.vs = c.vs; a.pages = c.pages;
    a.table = table; a.ldt = ldt; a.lens = lens; a.cu = cu; a.mask = mask; a.words = (int)words;
    a.B = (int)B; a.Hq = (int)Hq; a.Hkv = c.H; a.G = (int)(Hq / c.H); a.D = c.D;
    a.total_q = (int)total_q; a.max_q = (int)max_q; a.max_len = (int)max_len; a.ps = c.page_size;
    int l = 0;
    while (((int64_t)1 << l) < c.page_size) ++l;
    if (l > 0) {
        a.pmul = (uint32_t)((((uint64_t)1 << (31 + l)) + c.page_size - 1) / (uint64_t)c.page_size);
        a.pshift = l - 1;
    }
    // at least 2^-126, so that a hidden score stays -inf at scale 0
    a.scale2 = fmaxf((float)(fabs((double)scale) * 1.4426950408889634074 * 512.0), 1.17549435e-38f);
    a.negate = std::signbit(scale);
    a.R = p.R; a.U = p.U; a.P = p.P; a.ms = p.ms; a.HG = p.HG; a.groups = c.H / p.HG;
    a.Rs = __builtin_ctz(p.R); a.Us = __builtin_ctz(p.U); a.Ps = __builtin_ctz(p.P);
    a.out = out; a.ldo = ldo;
    a.po = static_cast<float *>(ws);
    a.pml = a.po + (int64_t)(2 * p.P) * p.HG * p.R * c.D;
    a.todo = reinterpret_cast<int *>(a.pml + (int64_t)(2 * p.P) * p.HG * p.R * 2);
    a.join = p.join;
    a.nrt = (int)p.nrt;
    a.cap = p.cap;
    const int64_t tiles = B * (c.H / p.HG) * p.nrt;
    a.NT = tiles <= p.P ? (int)tiles : 0;
    const int64_t entries = a.NT ? a.NT : p.P;
    a.JR = (int)ceil_div(entries * p.HG * p.R, 2048);            // about 2048 workgroups, at most 16 rows each
    a.JR = a.JR > 16 ? 16 : a.JR;
    const unsigned grid = (unsigned)p.P;
    hipError_t e;
    const bool f32 = dt == MXS_F32;
    if (p.NDP == 2) e = tree_go<2>(p, a, grid, f32, st);
    else if (p.NDP == 4) e = tree_go<4>(p, a, grid, f32, st);
    else e = tree_go<8>(p, a, grid, f32, st);
    if (e != hipSuccess || !p.join) return e;
    const dim3 jg((unsigned)entries, (unsigned)ceil_div(p.HG * p.R, a.JR));
    if (f32) hipLaunchKernelGGL((k_tree_join<float>), jg, dim3(256), 0, st, a);
    else hipLaunchKernelGGL((k_tree_join<__bf16>), jg, dim3(256), 0, st, a);
    return hipGetLastError();
}

}  // namespace mxs
