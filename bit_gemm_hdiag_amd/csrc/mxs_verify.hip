// mxs_verify.hip -- verification of drafted tokens against the target's logits.
//
// A row of logits l with maximum m stands for the weights e(v) = exp((l(v) - m)
// / T) and their sum Z. What the target still has to give after children of a
// node were rejected is, up to its sum, max(e(v) - S q(v), 0) with one number S:
// with r = max(e - S q, 0) and R = sum r, the next remainder max(r / R - q', 0),
// q' = q / left without the rejected tokens, is max(e - (S + R / left) q, 0) / R
// (the rejected tokens' own weights are 0 by then: u < 1). So a rejection costs
// one pass over e and q, nothing is stored, and the last remainder can be
// sampled from the logits again.
//
// A token is chosen by where a sum of up to a million weights crosses a random
// number, so the exponentials and sums that decide are in 64 bits.
#include <cmath>

#include "mxs_device.h"
#include "mxs_internal.h"

namespace mxs {

namespace {

constexpr int kPiece = 1024;            // logits of a wave: 16 of each lane
constexpr int kMaxNodes = 1024;
constexpr int kMaxChunks = 64;          // of a row: one of each lane

// A row is cut into at most 64 chunks of 4096 (up to 2^18 tokens) or 16384 logits.
// The large ones are a tenth quicker to sum (57 against 64 us for 794 rows of 128000
// bf16, half of them greedy) and twice as slow to draw from (22 against 13 us).
inline int chunk_size(int64_t V) { return V <= 4096 * kMaxChunks ? 4096 : 16384; }

// Element k of a lane's 16 within a piece: whole 16-byte vectors
template <typename T>
__device__ __forceinline__ int piece_index(int lane, int k) {
    constexpr int E = 16 / sizeof(T);
    return 64 * E * (k / E) + E * lane + k % E;
}

// A lane's 16 logits of a whole piece as they lie in memory, and as numbers
template <typename T>
struct Piece {
    static constexpr int E = 16 / sizeof(T), N = 16 / E;
    u32x4 w[N];
    __device__ __forceinline__ void load(const T *p, int lane) {
#pragma unroll
        for (int k = 0; k < N; ++k) __builtin_memcpy(&w[k], p + 64 * E * k + E * lane, 16);
    }
    __device__ __forceinline__ void get(float v[16]) const {
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            if constexpr (sizeof(T) == 2) {
                const uint32_t u = w[k / 8][k % 8 / 2];
                v[k] = __uint_as_float(k & 1 ? u & 0xFFFF0000u : u << 16);
            } else {
                v[k] = __uint_as_float(w[k / 4][k % 4]);
            }
        }
    }
};

// A row's weights are 2^(l c - k), c = log2(e) / T and k the whole number next to m c:
// exp((l - m) / T) but for a factor that the row has in common. With N + f = l c, |f| <=
// 1/2, that is 2^(N - k) p(f), p the polynomial of degree 10 that interpolates 2^f at
// the Chebyshev points, 0 among them: with the roundings 3.4 2^-53 off. That of f adds 0.4
// 2^-53, and c's own, as another T would, 1.2 2^-53 (m - l) / T. Sums against the maxima
// of waves, chunks and rows differ by powers of two, which are exact. N - k is taken
// from the low bits of l c + 1.5 2^52 - k. (Degree 8 would be 9600 2^-53 off.)
struct Scale {
    double c, lo;                       // log2(e) / T; (l - m) below which a weight counts as 0 (2^-1000)
    __device__ __forceinline__ explicit Scale(float t) {
        const bool greedy = !(t > 0.f);
        c = greedy ? 1.0 : 1.4426950408889634074 / (double)t;
        lo = -693.14718055994530942 * (greedy ? 1.0 : (double)t);
    }
};
// p <- p f + c for four numbers, c a constant in scalar registers (the compiler
// would copy it into the result's registers first, an instruction more each time). Each
// result is written before the last f is read, so it shares no register with one.
__device__ __forceinline__ void horner4(double p[4], const double f[4], double c) {
    asm("v_fma_f64 %0, %0, %4, %8\n\tv_fma_f64 %1, %1, %5, %8\n\tv_fma_f64 %2, %2, %6, %8\n\tv_fma_f64 %3, %3, %7, %8"
        : "+&v"(p[0]), "+&v"(p[1]), "+&v"(p[2]), "+&v"(p[3])
        : "v"(f[0]), "v"(f[1]), "v"(f[2]), "v"(f[3]), "s"(c));
}
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
// p 2^n for the n in the low bits of kn
__device__ __forceinline__ double scaled(double p, double kn) {
    u32x2 u = __builtin_bit_cast(u32x2, p);
    u.y += __builtin_bit_cast(u32x2, kn).x << 20;
    return __builtin_bit_cast(double, u);
}
constexpr double kMagic = 6755399441055744.0;
constexpr double kP10 = 7.072585949269223e-09, kP9 = 1.0208690299958306e-07, kP8 = 1.321544258792169e-06,
                 kP7 = 1.5252657260200837e-05, kP6 = 0.0001540353044173605, kP5 = 0.0013333558230164974,
                 kP4 = 0.009618129107606888, kP3 = 0.05550410866444772, kP2 = 0.24022650695910097,
                 kP1 = 0.69314718055995;
struct Weight {
    double m, c, lo, magic;             // magic: 1.5 2^52 - k
    float low;
    bool apart;                         // the weight is 1 at m and 0 elsewhere: m is infinite, or |m| c above 2^36,
                                        // and any other fp32 number more than 2^-24 |m| away from m
    __device__ __forceinline__ Weight(float mx, Scale t) : m((double)mx), c(t.c), lo(t.lo), low((float)((double)mx + t.lo)) {
        const double k = exponent(mx);
        apart = !(fabs(k) < 0x1p36);
        magic = kMagic - k;
    }
    __device__ __forceinline__ double exponent(float mx) const { return rint((double)mx * c); }
    // What a weight against the maximum mx counts against this one
    __device__ __forceinline__ double of(float mx) const {
        const double k = exponent(mx), n = k - (kMagic - magic);
        if (apart || !(fabs(k) < 0x1p36)) return (double)mx == m ? 1.0 : 0.0;
        return n < -1000.0 ? 0.0 : __longlong_as_double((int64_t)(1023 + (int)n) << 52);
    }
    // Where sums need none of the exceptions below: a finite maximum, T < inf, and
    // an fp32 number near m + lo. Weights below that one's, about 2^-1000, those of
    // NaN and -inf among them, count as that (the median of three is the smallest
    // where one is NaN): nothing beside the maximum's in the sum of a row, and below
    // what a remainder counts (left_of).
    __device__ __forceinline__ bool plain() const {
        const double d = (double)low - m;
        return !apart && c > 0.0 && d <= 0.9 * lo && d >= 1.02 * lo;
    }
    __device__ __forceinline__ void raw4(const float l[4], double w[4]) const {
        double kn[4], f[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const double x = (double)__builtin_amdgcn_fmed3f(l[k], low, INFINITY);
            kn[k] = fma(x, c, magic);
            f[k] = fma(x, c, magic - kn[k]);
            w[k] = fma(kP10, f[k], kP9);
        }
        horner4(w, f, kP8);
        horner4(w, f, kP7);
        horner4(w, f, kP6);
        horner4(w, f, kP5);
        horner4(w, f, kP4);
        horner4(w, f, kP3);
        horner4(w, f, kP2);
        horner4(w, f, kP1);
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = scaled(fma(w[k], f[k], 1.0), kn[k]);
    }
    __device__ __forceinline__ double power(double l) const {
        const double kn = fma(l, c, magic), f = fma(l, c, magic - kn);
        double p = fma(kP10, f, kP9);
        p = fma(p, f, kP8);
        p = fma(p, f, kP7);
        p = fma(p, f, kP6);
        p = fma(p, f, kP5);
        p = fma(p, f, kP4);
        p = fma(p, f, kP3);
        p = fma(p, f, kP2);
        p = fma(p, f, kP1);
        return scaled(fma(p, f, 1.0), kn);
    }
    // Weights below 2^-1000 are 0, and those of NaN and of -inf at any T (at T = inf all
    // others are 1)
    __device__ __forceinline__ double operator()(float l) const {
        if (!(l > -INFINITY)) return 0.0;
        if (apart) return (double)l == m ? 1.0 : 0.0;
        return (double)l - m < lo ? 0.0 : power((double)l);
    }
};

// Sums, maxima and running sums over the lanes of a wave by moves within the
// vector unit: the last lane of each 16 passes its total on
template <int CTRL, int ROWS>
__device__ __forceinline__ double moved(double v) {
    const uint64_t u = (uint64_t)__double_as_longlong(v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, ROWS, 0xF, false);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, ROWS, 0xF, false);
    return __longlong_as_double((int64_t)(((uint64_t)hi << 32) | lo));
}
__device__ __forceinline__ double wave_scan(double v) {
    v += moved<0x111, 0xF>(v);          // the lane 1, 2, 4, 8 before this one within 16
    v += moved<0x112, 0xF>(v);
    v += moved<0x114, 0xF>(v);
    v += moved<0x118, 0xF>(v);
    v += moved<0x142, 0xA>(v);          // lane 15 and 47 to the 16 behind them
    v += moved<0x143, 0xC>(v);          // lane 31 to the 32 behind it
    return v;
}
__device__ __forceinline__ double lane_of(double v, int lane) {
    const uint64_t u = (uint64_t)__double_as_longlong(v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, lane);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), lane);
    return __longlong_as_double((int64_t)(((uint64_t)hi << 32) | lo));
}
__device__ __forceinline__ double wave_sum(double v) { return lane_of(wave_scan(v), 63); }
template <int CTRL, int ROWS>
__device__ __forceinline__ float larger(float v) {
    const int u = __float_as_int(v);
    return fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(u, u, CTRL, ROWS, 0xF, false)));
}
__device__ __forceinline__ float wave_max(float v) {
    v = larger<0x111, 0xF>(v);
    v = larger<0x112, 0xF>(v);
    v = larger<0x114, 0xF>(v);
    v = larger<0x118, 0xF>(v);
    v = larger<0x142, 0xA>(v);
    v = larger<0x143, 0xC>(v);
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}
template <int CTRL, int ROWS>
__device__ __forceinline__ int smaller(int v) {
    const int u = __builtin_amdgcn_update_dpp(v, v, CTRL, ROWS, 0xF, false);
    return u < v ? u : v;
}
__device__ __forceinline__ int wave_min(int v) {
    v = smaller<0x111, 0xF>(v);
    v = smaller<0x112, 0xF>(v);
    v = smaller<0x114, 0xF>(v);
    v = smaller<0x118, 0xF>(v);
    v = smaller<0x142, 0xA>(v);
    v = smaller<0x143, 0xC>(v);
    return __builtin_amdgcn_readlane(v, 63);
}

__device__ __forceinline__ int64_t ceil_div_dev(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Where a walk ended: the row of the last kept node, whether its chunks are summed,
// and what was taken out of it: S q, or `gone` tokens
struct State {
    double S;
    int32_t cur, gone;
    int32_t sums;           // 0: nothing to draw (no node); else what is left to sum
};
enum { kNone = 0, kSummed = 1, kLeaf = 2, kRemainder = 3 };

struct Args {
    const void *logits;
    int64_t ldl, V, B, total, ldd;
    const int64_t *tokens;
    const int32_t *parents, *cu;
    const float *draft, *temperature;
    const double *uniform;
    int32_t *path, *count;
    int64_t *next;
    float *mx;              // [total, C] maximum of each chunk
    double *sum;            // [total, C] its weights' sum; greedy rows: index of the maximum
    double *rest;           // [B, C] sums of a remainder's chunks
    struct State *state;    // [B] where the walk ended
    int32_t *gone;          // [total] tokens taken out of that node's row
    int C, chunk, max_n, replacement;
    bool direct;            // grid of k_row_stats: (chunk, node, sequence) instead of (chunk, row)
};

// The sequence of a row (the number of sequences that end at or before it), B if none
__device__ __forceinline__ int64_t sequence_of(const Args &a, int64_t row, int lane) {
    int64_t b = 0;
    for (int64_t i = 0; i < a.B; i += 64) {
        const bool in = i + lane < a.B;
        const int c = __popcll(__ballot(in && a.cu[i + lane + 1] <= row));
        b += c;
        if (c < 64) break;
    }
    return b;
}

// What is left of a weight: masked tokens, which sums may have as 2^-1000, have nothing
__device__ __forceinline__ double left_of(double x) { return x > 0x1p-990 ? x : 0.0; }
__device__ __forceinline__ double clean(float q) { return q > 0.f && q < INFINITY ? (double)q : 0.0; }

// A chunk of a row, by a workgroup of 256 or (WAVE) by one wave: its maximum, and the
// sum of the weights against it (greedy rows: the lowest index of the maximum). A wave
// takes G pieces, all loaded before the first is used. The piece that passes the end of the row is
// loaded from 1024 logits before the end, less those that the piece before it has.
template <typename T, int G, bool WAVE>
__device__ __forceinline__ void chunk_stats(const Args &a, int64_t row, int c, float t) {
    constexpr int WAVES = WAVE ? 1 : 4;
    const int lane = threadIdx.x & 63, wave = WAVE ? 0 : threadIdx.x >> 6;
    const T *p = static_cast<const T *>(a.logits) + row * a.ldl;
    const int V = (int)a.V, from = (c * WAVES * G + wave) * kPiece;  // pieces from, from + WAVES, ..
    Piece<T> w[G];
    if (V >= kPiece) {
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const int at = from + WAVES * g * kPiece;
            if (at < V) w[g].load(p + (at + kPiece <= V ? at : V - kPiece), lane);
        }
    }
    const bool greedy = !(t > 0.f);
    const Scale sc(t);
    float m = -INFINITY;
    double s = 0.0;
    int best = 0x7FFFFFFF;
    if (V >= kPiece) {
        float v[G][16];
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const int at = from + WAVES * g * kPiece;
            if (at >= V) break;
            w[g].get(v[g]);
            if (at + kPiece > V) {
#pragma unroll
                for (int k = 0; k < 16; ++k) v[g][k] = V - kPiece + piece_index<T>(lane, k) < at ? -INFINITY : v[g][k];
            }
#pragma unroll
            for (int k = 0; k < 16; ++k) m = fmaxf(m, v[g][k]);      // ignores NaN
        }
        m = wave_max(m);
        const Weight e(m, sc);
        if (greedy) {
#pragma unroll
            for (int g = G - 1; g >= 0; --g) {
                const int at = from + WAVES * g * kPiece, first = at + kPiece <= V ? at : V - kPiece;
                if (at >= V) continue;
#pragma unroll
                for (int k = 15; k >= 0; --k) best = v[g][k] == m ? first + piece_index<T>(lane, k) : best;
            }
        } else if (e.plain()) {
#pragma unroll
            for (int g = 0; g < G; ++g) {
                if (from + WAVES * g * kPiece >= V) break;
#pragma unroll
                for (int k = 0; k < 16; k += 4) {
                    double r[4];
                    e.raw4(v[g] + k, r);
                    s += (r[0] + r[1]) + (r[2] + r[3]);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        }
    } else if (wave == 0) {
        for (int i = lane; i < V; i += 64) m = fmaxf(m, load1<T>(p + i));
        m = wave_max(m);
        for (int i = V - 1 - lane; i >= 0 && greedy; i -= 64) best = load1<T>(p + i) == m ? i : best;
    }
    const Weight e(m, sc);
    if (!greedy && !(V >= kPiece && e.plain())) {         // few tokens, or what the quick sum cannot take
#pragma unroll 1
        for (int g = 0; g < G; ++g) {
            const int at = from + WAVES * g * kPiece;
#pragma unroll 1
            for (int i = at + lane; i < at + kPiece && i < V; i += 64) s += e(load1<T>(p + i));
        }
    }
    s = greedy ? (double)wave_min(best) : wave_sum(s);
    if constexpr (WAVE) {
        if (lane == 0) {
            a.mx[row * a.C + c] = m;
            a.sum[row * a.C + c] = s;
        }
        return;
    }
    __shared__ float ms[4];
    __shared__ double ss[4];
    if (lane == 0) {
        ms[wave] = m;
        ss[wave] = s;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        const float mm = fmaxf(fmaxf(ms[0], ms[1]), fmaxf(ms[2], ms[3]));
        double r = greedy ? 2147483647.0 : 0.0;
        const Weight all(mm, sc);
#pragma unroll 1
        for (int i = 0; i < 4; ++i) {
            if (greedy) r = ms[i] == mm && ss[i] < r ? ss[i] : r;
            else r += ss[i] * all.of(ms[i]);
        }
        a.mx[row * a.C + c] = mm;
        a.sum[row * a.C + c] = r;
    }
}

// The chunks of every node that has children (16 trees of 64 nodes over 128000 bf16:
// 64 us with the leaves, 51 without, by workgroups). 163 rows of 128000 bf16 take 24.6 us
// (8 us of bytes at the copy rate; from the caches no less). 23 vector instructions a
// logit, most of them in 64 bits, are 12 us of issue at four cycles; CUs are busy for 17
// us, in 73 % of which they issue, and the rest is the way to the first logits of 5216
// short waves on 4096 places. Three multiply-adds more a logit cost 3 us.
template <typename T, int G, bool WAVE>
__global__ __launch_bounds__(256) void k_row_stats(Args a) {
    int64_t row, b;
    if (a.direct) {
        b = blockIdx.z;
        row = (int64_t)a.cu[b] + blockIdx.y;
    } else {
        row = blockIdx.y + (int64_t)blockIdx.z * 65535;
        if (row >= a.total) return;
        b = sequence_of(a, row, threadIdx.x & 63);
        if (b >= a.B) return;
    }
    const int c0 = a.cu[b], c1 = a.cu[b + 1] < a.total ? a.cu[b + 1] : (int)a.total;
    const int n = c1 - c0 < a.max_n ? c1 - c0 : a.max_n, i = (int)(row - c0);
    if (c0 < 0 || i >= n) return;
    bool parent = false;
    if (a.parents) {
        for (int j = i + 1 + threadIdx.x; j < n; j += 256) parent |= a.parents[c0 + j] == i;
        parent = __syncthreads_or(parent);
    } else {
        parent = i + 1 < n;
    }
    if (!parent) return;
    const int c = WAVE ? blockIdx.x * 4 + (threadIdx.x >> 6) : blockIdx.x;
    if (c < a.C) chunk_stats<T, G, WAVE>(a, row, c, a.temperature ? a.temperature[b] : 1.f);
}

// What the walks left to be summed, before the next tokens are drawn: the chunks of
// a last node without children, or those of max(e - S q, 0)
template <typename T, int G>
__global__ __launch_bounds__(256) void k_rest(Args a) {
    __shared__ double ss[4];
    const int64_t b = blockIdx.y;
    const State w = a.state[b];
    if (w.sums < kLeaf) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = blockIdx.x;
    const int64_t row = w.cur;
    const float t = a.temperature ? a.temperature[b] : 1.f;
    if (w.sums == kLeaf) {
        chunk_stats<T, G, false>(a, row, c, t);
        return;
    }
    const T *p = static_cast<const T *>(a.logits) + row * a.ldl;
    const float *q = a.draft + row * a.ldd;
    const Weight e(wave_max(lane < a.C ? a.mx[row * a.C + lane] : -INFINITY), Scale(t));
    const int V = (int)a.V;
    double s = 0.0;
    if (V >= kPiece && e.plain()) {
#pragma unroll 1
        for (int g = 0; g < G; ++g) {
            const int at = (c * 4 * G + wave + 4 * g) * kPiece, base = at + kPiece <= V ? at : V - kPiece;
            if (at >= V) break;
            Piece<T> w16;
            w16.load(p + base, lane);
            f32x4 q4[4];
#pragma unroll
            for (int k = 0; k < 16; k += 4) __builtin_memcpy(&q4[k / 4], q + base + piece_index<T>(lane, k), 16);
            float v[16];
            w16.get(v);
            if (at != base) {
#pragma unroll
                for (int k = 0; k < 16; ++k) v[k] = base + piece_index<T>(lane, k) < at ? -INFINITY : v[k];
            }
#pragma unroll
            for (int k = 0; k < 16; k += 4) {
                double r[4];
                e.raw4(v + k, r);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const double x = r[j] - w.S * clean(q4[k / 4][j]);
                    s += left_of(x);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    } else {
#pragma unroll 1
        for (int i = c * a.chunk + (int)threadIdx.x; i < (c + 1) * a.chunk && i < V; i += 256)
            s += left_of(e(load1<T>(p + i)) - w.S * clean(q[i]));
    }
    s = wave_sum(s);
    if (lane == 0) ss[wave] = s;
    __syncthreads();
    if (threadIdx.x == 0) a.rest[b * a.C + c] = ((ss[0] + ss[1]) + ss[2]) + ss[3];
}

// Four consecutive logits (or draft probabilities) at p, of which `left` exist
template <typename T>
__device__ __forceinline__ f32x4 load4(const T *p, int64_t left, float missing) {
    f32x4 v;
    if (left >= 4) {
        if constexpr (sizeof(T) == 2) {
            uint32_t u[2];
            __builtin_memcpy(u, p, 8);
            v = f32x4{__uint_as_float(u[0] << 16), __uint_as_float(u[0] & 0xFFFF0000u), __uint_as_float(u[1] << 16),
                      __uint_as_float(u[1] & 0xFFFF0000u)};
        } else {
            __builtin_memcpy(&v, p, 16);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = i < left ? load1<T>(p + i) : missing;
    }
    return v;
}

// One workgroup a sequence walks its tree. The first wave tries the children; the
// workgroup prepares what that reads (maximum and sum of every node's row, weight
// and draft probability of every token), and sums a remainder where there is
// another child to try. The code runs once or twice a call, so its loops stay rolled:
// fetching instructions costs more than running them (27 against 13 us, with the draw,
// for 16 trees of 64 nodes). A remainder is summed at about 100 GB/s, what one workgroup
// reads: 4 us for 50021 fp32 tokens; 16 trees of 16 nodes drawn from a distribution over
// 128000 bf16 tokens spend 80 us here.
template <typename T>
__global__ __launch_bounds__(1024) void k_walk(Args a) {
    __shared__ float node_m[kMaxNodes], node_q[kMaxNodes];
    __shared__ double node_z[kMaxNodes], node_e[kMaxNodes], node_u[kMaxNodes];
    __shared__ int node_p[kMaxNodes];             // parent of a node that can be accepted, else -1
    __shared__ int node_best[kMaxNodes], node_x[kMaxNodes];
    __shared__ int gone[kMaxNodes];               // children of the current node that were taken out (no draft)
    __shared__ int has_child[kMaxNodes];
    __shared__ double sums[16];
    __shared__ struct {
        double S;
        int cur, gone, sum;
    } w;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t b = blockIdx.x;
    int c0 = a.cu[b], c1 = a.cu[b + 1];
    const float t = a.temperature ? a.temperature[b] : 1.f;
    c0 = c0 < 0 ? 0 : c0;
    c1 = c1 > a.total ? (int)a.total : c1;
    const int rows = c1 > c0 ? c1 - c0 : 0;
    const int n = rows < a.max_n ? rows : a.max_n;
    for (int i = tid; i < rows; i += 1024) a.path[c0 + i] = i == 0 && n > 0 ? 0 : -1;
    if (n == 0) {
        if (tid == 0) {
            a.count[b] = 0;
            a.next[b] = -1;
            a.state[b].sums = kNone;
        }
        return;
    }
    const bool greedy = !(t > 0.f);
    const Scale sc(t);
    const T *logits = static_cast<const T *>(a.logits) + (int64_t)c0 * a.ldl;
    const float *draft = a.draft && !greedy ? a.draft + (int64_t)c0 * a.ldd : nullptr;
    for (int i = tid; i < n; i += 1024) has_child[i] = 0;
    __syncthreads();
    // the tokens' own logits
    for (int i = tid; i < n; i += 1024) {
        const int p = a.parents ? a.parents[c0 + i] : i - 1;
        const int64_t x = a.tokens[c0 + i];
        const bool below = i > 0 && p >= 0 && p < i, ok = below && x >= 0 && x < a.V;
        if (below) has_child[p] = 1;
        node_u[i] = a.uniform[c0 + i];
        node_p[i] = ok ? p : -1;
        node_x[i] = ok ? (int)x : -1;
        node_e[i] = ok && !greedy ? (double)load1<T>(logits + p * a.ldl + x) : 0.0;
        node_q[i] = ok && draft ? (float)clean(draft[p * a.ldd + x]) : 1.f;
    }
    // maximum and sum of every row from its chunks, by the other waves first (rows
    // without children have none; what is read there is not used)
    for (int i = 15 - wave; i < n; i += 16) {
        const int64_t at = (int64_t)(c0 + i) * a.C + lane;
        const float mc = lane < a.C ? a.mx[at] : -INFINITY;
        const double zc = lane < a.C ? a.sum[at] : 0.0;
        const float m = wave_max(mc);
        double z;
        int best = 0x7FFFFFFF;
        if (greedy) {
            best = wave_min(mc == m ? (int)zc : best);
            z = m == -INFINITY ? 0.0 : 1.0;
        } else {
            z = wave_sum(zc * Weight(m, sc).of(mc));
        }
        if (lane == 0) {
            node_m[i] = m;
            node_z[i] = z;
            node_best[i] = m == -INFINITY ? -1 : best;
        }
    }
    if (tid == 0) w.gone = 0;
    __syncthreads();
    for (int i = tid; i < n; i += 1024) {
        const int p = node_p[i];
        if (p >= 0) node_e[i] = greedy ? (node_x[i] == node_best[p] ? 1.0 : 0.0) : Weight(node_m[p], sc)((float)node_e[i]);
    }
    __syncthreads();

    // the walk: all lanes of the first wave go the same way
    int cur = 0, next_child = 1, kept = 1;
    double S = 0.0, R = node_z[0], left = 1.0;
    const int pieces = (int)ceil_div_dev(a.V, kPiece);
    for (;;) {
        if (wave == 0) {
            bool sum = false;
            int ngone = w.gone;
            for (;;) {
                // the next child of cur
                int i = -1;
                for (int i0 = next_child & ~63; i0 < n && i < 0; i0 += 64) {
                    const int j = i0 + lane;
                    const uint64_t kids = __ballot(j < n && j >= next_child && node_p[j] == cur);
                    if (kids) i = i0 + __ffsll((long long)kids) - 1;
                }
                if (i < 0) {
                    sum = false;                      // no other child: the draw sums what is left
                    break;
                }
                if (sum) break;
                next_child = i + 1;
                const double e = node_e[i], q = (double)node_q[i], u = node_u[i];
                bool ok;
                if (greedy) {
                    ok = e > 0.0;
                } else if (draft) {
                    ok = left > 0.0 && u * q * R < fmax(e - S * q, 0.0) * left;
                    if (!ok && left > 0.0) {
                        S += R / left;
                        if (!a.replacement) left -= q;
                        sum = true;
                    }
                } else {
                    double r = e;
                    for (int k = 0; k < ngone; ++k)               // the same token among its elder siblings
                        if (node_x[gone[k]] == node_x[i]) r = 0.0;
                    ok = u * R < r;
                    if (!ok && r > 0.0) {
                        if (lane == 0) gone[ngone] = i;
                        // all lanes read it for the next child
                        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                        __builtin_amdgcn_wave_barrier();
                        ++ngone;
                        R = R > r ? R - r : 0.0;
                    }
                }
                if (ok) {
                    if (lane == 0) a.path[c0 + kept] = i;
                    ++kept;
                    cur = i;
                    S = 0.0;
                    left = 1.0;
                    R = node_z[i];
                    ngone = 0;
                }
            }
            if (lane == 0) {
                w.S = S;
                w.cur = cur;
                w.gone = ngone;
                w.sum = sum;
            }
        }
        __syncthreads();
        if (!w.sum) break;
        // the remainder's sum, a wave a piece, four values of a lane at a time; the next
        // four are loaded before these are used
        const T *row = logits + (int64_t)w.cur * a.ldl;
        const float *qrow = draft + (int64_t)w.cur * a.ldd;
        const Weight e(node_m[w.cur], sc);
        const double s0 = w.S;
        const int turns = 4 * ((pieces - wave + 15) / 16);
        auto place = [&](int j) { return (int64_t)(wave + 16 * (j >> 2)) * kPiece + 256 * (j & 3) + 4 * lane; };
        f32x4 v = load4<T>(row + place(0), a.V - place(0), -INFINITY), q = load4<float>(qrow + place(0), a.V - place(0), 0.f);
        f32x4 v1 = load4<T>(row + place(1), a.V - place(1), -INFINITY), q1 = load4<float>(qrow + place(1), a.V - place(1), 0.f);
        double s = 0.0;
        const bool plain = e.plain();
#pragma unroll 1
        for (int j = 0; j < turns; ++j) {
            const f32x4 v0 = v, q0 = q;
            const int64_t at = place(j + 2 < turns ? j + 2 : j);
            v = v1;
            q = q1;
            v1 = load4<T>(row + at, a.V - at, -INFINITY);
            q1 = load4<float>(qrow + at, a.V - at, 0.f);
            double r[4];
            if (plain) {
                const float x[4] = {v0[0], v0[1], v0[2], v0[3]};
                e.raw4(x, r);
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k) r[k] = e(v0[k]);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const double x = r[k] - s0 * clean(q0[k]);
                s += left_of(x);
            }
        }
        s = wave_sum(s);
        if (lane == 0) sums[wave] = s;
        __syncthreads();
        R = wave_sum(lane < 16 ? sums[lane] : 0.0);
    }
    const int end = w.cur, ngone = w.gone;
    for (int k = tid; k < ngone; k += 1024) a.gone[c0 + k] = node_x[gone[k]];
    if (tid == 0) {
        a.count[b] = kept;
        a.state[b] = State{w.S, c0 + end, ngone, !has_child[end] ? kLeaf : (draft && w.S > 0.0 ? kRemainder : kSummed)};
    }
}

// The next token of every sequence: the chunk where the cumulated sum of what is
// left crosses the random number, then the token in it. What a chunk has left without
// the tokens taken out of it is a difference, which rounding can leave above 0 where
// they were all it had: a chunk in which nothing is found counts as 0 from then on.
template <typename T>
__global__ __launch_bounds__(1024) void k_draw(Args a) {
    __shared__ double sums[kMaxChunks], wsum[16];
    __shared__ int firsts[16], lasts[16];
    __shared__ struct {
        double target, before;
        int at, past;
    } w;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t b = blockIdx.x;
    const State st = a.state[b];
    if (st.sums == kNone) return;
    const float t = a.temperature ? a.temperature[b] : 1.f;
    const bool greedy = !(t > 0.f);
    const int c0 = a.cu[b] < 0 ? 0 : a.cu[b];
    const float mc = lane < a.C ? a.mx[(int64_t)st.cur * a.C + lane] : -INFINITY;
    const double zc = lane < a.C ? a.sum[(int64_t)st.cur * a.C + lane] : 0.0;
    const double u = a.uniform[c0];
    const float m = wave_max(mc);
    if (greedy || m == -INFINITY) {
        const int best = wave_min(mc == m ? (int)zc : 0x7FFFFFFF);
        if (tid == 0) a.next[b] = m == -INFINITY ? -1 : best;
        return;
    }
    const Weight e(m, Scale(t));
    const T *row = static_cast<const T *>(a.logits) + (int64_t)st.cur * a.ldl;
    // the sums of the remainder's chunks, or those of the row's less the tokens taken
    // out; the row's own where nothing is left of it
    bool rem = st.sums == kRemainder, whole = false;
    uint64_t empty = 0;
#pragma unroll 1
    for (;;) {
        if (wave == 0) {
            double s = 0.0;
            if (lane < a.C) {
                if (rem) {
                    s = a.rest[b * a.C + lane];
                } else {
                    s = zc * e.of(mc);
                    for (int k = 0; k < st.gone && !whole; ++k) {
                        const int x = a.gone[c0 + k];
                        if (x / a.chunk == lane) s = fmax(s - e(load1<T>(row + x)), 0.0);
                    }
                }
            }
            if (empty >> lane & 1) s = 0.0;
            const double upto = wave_scan(s), target = u * lane_of(upto, 63);
            // first one whose inclusive sum is past the target, else the last that holds anything
            const uint64_t found = __ballot(s > 0.0 && upto > target), any = __ballot(s > 0.0);
            int at = -1;
            if (found) at = __ffsll((long long)found) - 1;
            else if (any) at = 63 - __clzll((long long)any);
            const double before = lane_of(upto - s, at < 0 ? 0 : at);
            if (lane == 0) {
                w.at = at;
                w.before = before;
                w.target = target;
                w.past = !found;
            }
        }
        __syncthreads();
        // 4096 tokens at a time, four of a thread
        int first = 0x7FFFFFFF, last = -1;
        double base = w.before;
        const double target = w.target;
        if (w.at >= 0) {
#pragma unroll 1
            for (int i = 0; i < a.chunk; i += 4096) {
                const int64_t at = (int64_t)w.at * a.chunk + i + 4 * tid;
                const f32x4 v = load4<T>(row + at, a.V - at, -INFINITY);
                f32x4 q = {0, 0, 0, 0};
                if (rem) q = load4<float>(a.draft + (int64_t)st.cur * a.ldd + at, a.V - at, 0.f);
                double r[4], part = 0.0;
#pragma unroll
                for (int k = 0; k < 4; ++k) r[k] = rem ? left_of(e(v[k]) - st.S * clean(q[k])) : e(v[k]);
                for (int j = 0; j < st.gone && !whole; ++j) {
                    const int64_t k = a.gone[c0 + j] - at;
#pragma unroll
                    for (int l = 0; l < 4; ++l) r[l] = k == l ? 0.0 : r[l];
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) part += r[k];
                const double inc = wave_scan(part);
                if (lane == 63) wsum[wave] = inc;
                __syncthreads();
                const double waves = wave_scan(lane < 16 ? wsum[lane] : 0.0);
                double s = base + (wave ? lane_of(waves, wave - 1) : 0.0) + (inc - part);
                base += lane_of(waves, 15);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    s += r[k];
                    if (r[k] > 0.0) {
                        last = (int)at + k;
                        if (s > target && first == 0x7FFFFFFF) first = last;
                    }
                }
                __syncthreads();
            }
        }
        first = wave_min(first);
        last = ~wave_min(~last);                      // ~ turns the order round
        if (lane == 0) {
            firsts[wave] = first;
            lasts[wave] = last;
        }
        __syncthreads();
        first = wave_min(firsts[lane & 15]);
        last = ~wave_min(~lasts[lane & 15]);
        const int x = w.past || first == 0x7FFFFFFF ? last : first;
        if (x >= 0 || whole) {
            if (tid == 0) a.next[b] = x;
            return;
        }
        if (w.at >= 0) {
            empty |= 1ull << w.at;
        } else {                                      // nothing but rounding was left of any chunk
            rem = false;
            whole = true;
            empty = 0;
        }
        __syncthreads();
    }
}

struct Layout {
    size_t mx, sum, rest, state, gone, bytes;
    int C;
};

Layout layout(int64_t B, int64_t total, int64_t V) {
    Layout l{};
    l.C = (int)ceil_div(V, (int64_t)chunk_size(V));
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t o = at;
        at += (bytes + 15) / 16 * 16;
        return o;
    };
    l.mx = take((size_t)total * l.C * 4);
    l.sum = take((size_t)total * l.C * 8);
    l.rest = take((size_t)B * l.C * 8);
    l.state = take((size_t)B * sizeof(State));
    l.gone = take((size_t)total * 4);
    l.bytes = at;
    return l;
}

}  // namespace

size_t verify_tree_workspace(int64_t B, int64_t total, int64_t V) { return layout(B, total, V).bytes; }

hipError_t launch_verify_tree(const void *logits, mxs_dtype dt, int64_t ldl, int64_t V, const int64_t *tokens,
                              const int32_t *parents, const int32_t *cu, int64_t B, int64_t total, int64_t max_n,
                              const float *draft, int64_t ldd, int32_t replacement, const float *temperature,
                              const double *uniform, int32_t *path, int32_t *count, int64_t *next, void *ws,
                              hipStream_t st) {
    Args a{};
    a.logits = logits; a.ldl = ldl; a.V = V; a.B = B; a.total = total; a.ldd = ldd;
    a.tokens = tokens; a.parents = parents; a.cu = cu; a.draft = draft; a.temperature = temperature;
    a.uniform = uniform; a.path = path; a.count = count; a.next = next;
    a.max_n = (int)max_n; a.replacement = replacement;
    const Layout l = layout(B, total, V);
    a.C = l.C;
    a.chunk = chunk_size(V);
    uint8_t *w = static_cast<uint8_t *>(ws);
    a.mx = reinterpret_cast<float *>(w + l.mx);
    a.sum = reinterpret_cast<double *>(w + l.sum);
    a.rest = reinterpret_cast<double *>(w + l.rest);
    a.state = reinterpret_cast<State *>(w + l.state);
    a.gone = reinterpret_cast<int32_t *>(w + l.gone);
    hipError_t e;
    if (total > 0 && max_n > 0) {
        // a wave a chunk where those alone fill the chip, else a workgroup: 25 us either way
        // for 32 chains of 8 nodes over 128000 bf16, 40 against 51 for 16 trees of 64
        const bool by_wave = a.chunk == 4096 && total * a.C >= 4096;
        const unsigned gx = (unsigned)(by_wave ? ceil_div(a.C, 4) : a.C);
        // a node and chunk, unless a loose max_n would leave most workgroups without a node:
        // then a row and chunk, and its sequence is looked for
        a.direct = B * max_n <= 2 * total + 64;
        const dim3 grid = a.direct ? dim3(gx, (unsigned)max_n, (unsigned)B)
                                   : dim3(gx, (unsigned)(total < 65535 ? total : 65535),
                                          (unsigned)ceil_div(total, (int64_t)65535));
        if (by_wave) {
            if (dt == MXS_BF16) hipLaunchKernelGGL((k_row_stats<uint16_t, 4, true>), grid, dim3(256), 0, st, a);
            else hipLaunchKernelGGL((k_row_stats<float, 4, true>), grid, dim3(256), 0, st, a);
        } else if (a.chunk == 4096) {
            if (dt == MXS_BF16) hipLaunchKernelGGL((k_row_stats<uint16_t, 1, false>), grid, dim3(256), 0, st, a);
            else hipLaunchKernelGGL((k_row_stats<float, 1, false>), grid, dim3(256), 0, st, a);
        } else {
            if (dt == MXS_BF16) hipLaunchKernelGGL((k_row_stats<uint16_t, 4, false>), grid, dim3(256), 0, st, a);
            else hipLaunchKernelGGL((k_row_stats<float, 4, false>), grid, dim3(256), 0, st, a);
        }
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    if (dt == MXS_BF16) hipLaunchKernelGGL(k_walk<uint16_t>, dim3((unsigned)B), dim3(1024), 0, st, a);
    else hipLaunchKernelGGL(k_walk<float>, dim3((unsigned)B), dim3(1024), 0, st, a);
    if ((e = hipGetLastError()) != hipSuccess || total == 0 || max_n == 0) return e;
    const dim3 grid((unsigned)a.C, (unsigned)B);
    if (a.chunk == 4096) {
        if (dt == MXS_BF16) hipLaunchKernelGGL((k_rest<uint16_t, 1>), grid, dim3(256), 0, st, a);
        else hipLaunchKernelGGL((k_rest<float, 1>), grid, dim3(256), 0, st, a);
    } else {
        if (dt == MXS_BF16) hipLaunchKernelGGL((k_rest<uint16_t, 4>), grid, dim3(256), 0, st, a);
        else hipLaunchKernelGGL((k_rest<float, 4>), grid, dim3(256), 0, st, a);
    }
    if ((e = hipGetLastError()) != hipSuccess) return e;
    if (dt == MXS_BF16) hipLaunchKernelGGL(k_draw<uint16_t>, dim3((unsigned)B), dim3(1024), 0, st, a);
    else hipLaunchKernelGGL(k_draw<float>, dim3((unsigned)B), dim3(1024), 0, st, a);
    return hipGetLastError();
}

}  // namespace mxs
