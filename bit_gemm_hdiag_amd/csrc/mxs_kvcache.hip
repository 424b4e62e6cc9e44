// mxs_kvcache.hip -- rotary positions, and the paged 4-bit K/V cache written
// and read in place.
//
// The cache holds keys and values as 4-bit MXINT (gist.science/nl
// "Technische Samenvatting" §4, W4A4KV4) in the layout of mxs_quantize_kv:
// slot s of the pool is one token, codes [slot, H, D/2], E8M0 bytes
// [slot, H, D/32].
//
// Rotary positions turn the pair (a, b) of dims number i at position t by the
// angle t f_i:  a' = a cos - b sin,  b' = b cos + a sin.  The angle is formed
// in turns, t (f_i / 2 pi), in fp64, and reduced by its nearest whole number
// before anything is rounded to fp32, so positions of a million cost no
// accuracy. The cosines and sines of a workgroup's tokens are computed once
// into LDS and shared by all its heads.
#include <cmath>
#include <type_traits>

#include "mxs_device.h"
#include "mxs_internal.h"

namespace mxs {

namespace {

constexpr double kInv2Pi = 0.15915494309189533577;

// n / d for n < 65536, d <= 65536: m = ceil(2^32 / d), 0 for d = 1
// (n (m d - 2^32) < n d <= 2^32, so the product's high word is exact)
struct Div16 {
    uint32_t m, d;
};
Div16 div16(uint32_t d) { return Div16{d <= 1 ? 0u : (uint32_t)((0x100000000ull + d - 1) / d), d ? d : 1u}; }
__device__ __forceinline__ uint32_t quot(uint32_t n, Div16 v) { return v.m ? __umulhi(n, v.m) : n; }

__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
    typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
    const bf2 r = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, r);
}

// ---------------------------------------------------------------------- rope
// V elements at p (16 bytes where V > 1), widened to fp32 / rounded once
template <typename T, int V>
__device__ __forceinline__ void get(const T *p, float v[V]) {
    if constexpr (V == 1) {
        v[0] = load1<T>(p);
    } else if constexpr (sizeof(T) == 2) {
        const u32x4 u = *reinterpret_cast<const u32x4 *>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(u[i] << 16);
            v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
        }
    } else {
        const f32x4 u = *reinterpret_cast<const f32x4 *>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = u[i];
    }
}
template <typename T, int V>
__device__ __forceinline__ void put(T *p, const float v[V]) {
    if constexpr (V == 1) {
        if constexpr (sizeof(T) == 2) *p = (uint16_t)bf16_pair(v[0], 0.f);
        else *p = v[0];
    } else if constexpr (sizeof(T) == 2) {
        const u32x4 u = {bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]), bf16_pair(v[6], v[7])};
        *reinterpret_cast<u32x4 *>(p) = u;
    } else {
        *reinterpret_cast<f32x4 *>(p) = f32x4{v[0], v[1], v[2], v[3]};
    }
}

struct RopeArgs {
    const void *x;
    void *y;
    int64_t T, xt, xh, yt, yh;      // element strides of tokens and heads
    const int64_t *pos;
    const double *freq;
    int H, D, half;
    int TB, HB;                     // tokens and heads of a workgroup
    Div16 units, heads;             // units of a head, heads of a workgroup
    float mscale;
};

// Bound by HBM: x read and y written once, the angles are one fp64 product and
// one sincospi a token and pair, shared by the heads. 2048 tokens of 64 heads of
// 128 bf16 take 11.5 us (5.8 TB/s, against 5.0 of a 2 GiB copy: the caches hold
// part of it), 64 tokens 2.7 us, of which the launch is most. Rows that no 16-byte
// access fits (V = 1) take 29.9 us there, and 54.7 where 20 of the 128 dims turn
// and the rest is copied element by element.
// One unit is V elements of the first and V of the second half of a head's
// rotated part (PAIRS: 2 V consecutive elements of V pairs; V = 1: one pair),
// or V elements that pass through.
template <typename T, int V, bool PAIRS>
__global__ __launch_bounds__(256) void k_rope(RopeArgs a) {
    extern __shared__ __attribute__((aligned(16))) float cs[];      // [TB][half] cosines, then sines
    const int half = a.half, tid = threadIdx.x;
    const int64_t t0 = (int64_t)blockIdx.x * a.TB;
    const int nt = a.T - t0 < a.TB ? (int)(a.T - t0) : a.TB;
    const int h0 = blockIdx.y * a.HB, nh = a.H - h0 < a.HB ? a.H - h0 : a.HB;
    float *sn = cs + a.TB * half;
    for (int e = tid; e < nt * half; e += 256) {
        const int tl = e / half, i = e - tl * half;
        const double turns = (double)a.pos[t0 + tl] * (a.freq[i] * kInv2Pi);
        float s, c;
        sincospif(2.f * (float)(turns - rint(turns)), &s, &c);
        cs[e] = c * a.mscale;
        sn[e] = s * a.mscale;
    }
    __syncthreads();
    const T *x = static_cast<const T *>(a.x);
    T *y = static_cast<T *>(a.y);
    const int rotu = half / V;                          // rotating units of a head
    const uint32_t total = (uint32_t)nt * a.HB * a.units.d;
#pragma unroll 2
    for (uint32_t e = tid; e < total; e += 256) {
        const uint32_t th = quot(e, a.units);
        const int u = (int)(e - th * a.units.d);
        const uint32_t tl = quot(th, a.heads);
        const int h = (int)(th - tl * a.heads.d);
        if (h >= nh) continue;
        const T *xr = x + (t0 + tl) * a.xt + (int64_t)(h0 + h) * a.xh;
        T *yr = y + (t0 + tl) * a.yt + (int64_t)(h0 + h) * a.yh;
        if (u < rotu) {
            const int i = u * V, o0 = PAIRS ? 2 * i : i, o1 = PAIRS ? 2 * i + V : i + half;
            float p[V], q[V], c[V], s[V];
            get<T, V>(xr + o0, p);
            get<T, V>(xr + o1, q);
#pragma unroll
            for (int k = 0; k < V; ++k) {
                c[k] = cs[tl * half + i + k];
                s[k] = sn[tl * half + i + k];
            }
            if constexpr (PAIRS && V > 1) {
#pragma unroll
                for (int k = 0; k < V; k += 2) {
                    const float a0 = p[k], b0 = p[k + 1], a1 = q[k], b1 = q[k + 1];
                    p[k] = a0 * c[k / 2] - b0 * s[k / 2];
                    p[k + 1] = b0 * c[k / 2] + a0 * s[k / 2];
                    q[k] = a1 * c[(k + V) / 2] - b1 * s[(k + V) / 2];
                    q[k + 1] = b1 * c[(k + V) / 2] + a1 * s[(k + V) / 2];
                }
            } else {
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    const float a0 = p[k], b0 = q[k];
                    p[k] = a0 * c[k] - b0 * s[k];
                    q[k] = b0 * c[k] + a0 * s[k];
                }
            }
            put<T, V>(yr + o0, p);
            put<T, V>(yr + o1, q);
        } else {
            const int o = 2 * half + (u - rotu) * V;
            float p[V];
            get<T, V>(xr + o, p);
            put<T, V>(yr + o, p);
        }
    }
}

template <typename T, int V, bool PAIRS>
hipError_t rope_go(RopeArgs a, hipStream_t st) {
    const int units = a.half / V + (a.D - 2 * a.half) / V;
    // 256 units in a workgroup, one a thread, whole heads first, then tokens.
    // Four a thread (and a quarter of the sines and cosines) are slower at any
    // number of tokens: 3.7 against 2.6 us at 8 tokens of 64 heads of 128 bf16,
    // 22.0 against 20.9 at 4096.
    const int64_t want = 256;
    a.HB = a.H;
    while (a.HB > 1 && (int64_t)a.HB * units > want) a.HB = (a.HB + 1) / 2;
    int64_t tb = a.HB == a.H ? want / ((int64_t)a.HB * units) : 1;
    const int64_t cap = a.half ? 4096 / a.half : 64;   // LDS: 8 bytes a token and pair
    tb = tb > cap ? cap : tb;
    a.TB = (int)(tb < 1 ? 1 : tb);
    a.units = div16(units);
    a.heads = div16(a.HB);
    const int64_t gx = ceil_div(a.T, (int64_t)a.TB);
    hipLaunchKernelGGL((k_rope<T, V, PAIRS>), dim3((unsigned)gx, (unsigned)ceil_div(a.H, a.HB)), dim3(256),
                       (size_t)a.TB * a.half * 8 + 16, st, a);
    return hipGetLastError();
}

template <typename T>
hipError_t rope_type(const RopeArgs &a, bool vec, bool pairs, hipStream_t st) {
    constexpr int V = 16 / sizeof(T);
    if (vec) return pairs ? rope_go<T, V, true>(a, st) : rope_go<T, V, false>(a, st);
    return pairs ? rope_go<T, 1, true>(a, st) : rope_go<T, 1, false>(a, st);
}

// -------------------------------------------------------------------- append
struct AppendArgs {
    const void *k, *v;
    int64_t T, kt, kh, vt, vh;
    const int64_t *slots, *pos;
    const double *freq;
    uint8_t *kc, *ks, *vc, *vs;
    int64_t nslots;
    int H, D, half;
    int TB;
    Div16 words, hwords;            // 8-element words of a token row, of a head
    Div16 chunk;                    // words of a token row that a workgroup takes
    float mscale;
};

// The 8 elements of a word and, for a rotation of halves, the 8 that they pair
// with, as the loads left them (widening waits for them)
template <typename T, bool VEC>
struct Eight {
    static constexpr int N = VEC ? (int)sizeof(T) / 2 : 8;
    typedef std::conditional_t<VEC, u32x4, T> E;
    E e[N];
    __device__ __forceinline__ void load(const T *p) {
#pragma unroll
        for (int i = 0; i < N; ++i) e[i] = reinterpret_cast<const E *>(p)[i];
    }
    __device__ __forceinline__ float get(int i) const {
        if constexpr (!VEC) {
            return load1<T>(&e[i]);
        } else if constexpr (sizeof(T) == 2) {
            const uint32_t w = e[0][i >> 1];
            return __uint_as_float(i & 1 ? w & 0xFFFF0000u : w << 16);
        } else {
            return __uint_as_float(e[i >> 2][i & 3]);
        }
    }
};

// MXINT4 of one quad's 32 fp64 values, 8 a lane: the rule of quantize_pack8
// without its rounding to fp32, so that a rotated key's code depends on no
// intermediate precision (values on a rounding border would)
__device__ __forceinline__ uint32_t pack8_f64(const double v[8], uint32_t &byte) {
    double m = 0.0;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const double x = fabs(v[i]);
        bad |= !(x <= 1.7976931348623157e308);
        m = x > m ? x : m;
    }
    uint32_t e = bad ? 0x7FFu : (uint32_t)(__double_as_longlong(m) >> 52);
    e = quad_max_u32(e);
    bad = e == 0x7FFu;
    int s = (int)e - 1023 - 2;                    // m - 2 = 2 at 4 bits; e = 0 (all zero) clamps
    s = s < -127 ? -127 : (s > 127 ? 127 : s);
    byte = bad ? 0xFFu : (uint32_t)(s + 127);
    const double inv = __longlong_as_double((int64_t)(1023 - s) << 52);
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const double t = rint(v[i] * inv);
        const int c = (int)fmin(fmax(t, -7.0), 7.0);
        w |= ((uint32_t)c & 15u) << (4 * i);
    }
    return bad ? 0u : w;
}

// K and V are read once and 17/64 (bf16) of their bytes written. Without rotation
// bound by HBM: 32768 tokens of 8 heads of 128 bf16 29.0 us (5.9 TB/s; cold, 42 to 46).
// With it the fp64 sincospi of every token and pair (computed once for the heads)
// and the fp64 products, behind a barrier between loads and stores in the K
// workgroups, add 1.5 us at 2048 tokens (5.7 us) and 24 us at 32768 (52.7); fp32
// would put keys near a rounding border on either side of it. fp32 inputs: 48.1 us
// at 32768 tokens, rotated 67.6.
// ROT 0: none; 1: halves, whole words pair with whole words (half % 8 == 0); 2:
// pairs; 3: halves of any size (the partners are loaded one by one). A thread
// takes WPT words, all loaded before the first is quantised; the cosines and
// sines of the workgroup's tokens are formed while the loads are in flight.
template <typename T, bool VEC, int ROT, int WPT>
__global__ __launch_bounds__(256) void k_kv4_append(AppendArgs a) {
    extern __shared__ __attribute__((aligned(16))) double cs64[];
    const int tid = threadIdx.x, half = a.half;
    const int64_t t0 = (int64_t)blockIdx.x * a.TB;
    const int nt = a.T - t0 < a.TB ? (int)(a.T - t0) : a.TB;
    const bool isv = blockIdx.y != 0;
    const bool rot = ROT != 0 && !isv;
    const T *x = static_cast<const T *>(isv ? a.v : a.k);
    const int64_t xt = isv ? a.vt : a.kt, xh = isv ? a.vh : a.kh;
    uint8_t *codes = isv ? a.vc : a.kc, *scales = isv ? a.vs : a.ks;
    // a quad's four lanes hold one 32-block of one token: the words of a head
    // are a multiple of four, so every branch below is taken by whole quads
    const uint32_t w0 = blockIdx.z * a.chunk.d;
    Eight<T, VEC> own[WPT], other[WPT];
    int64_t slot[WPT];
    uint32_t tl[WPT], w[WPT], wd[WPT];
#pragma unroll
    for (int k = 0; k < WPT; ++k) {
        const uint32_t e = tid + 256u * k;
        tl[k] = quot(e, a.chunk);
        w[k] = w0 + e - tl[k] * a.chunk.d;
        const bool on = tl[k] < (uint32_t)nt && w[k] < a.words.d;
        if (!on) {
            tl[k] = 0;
            w[k] = w0;
        }
        slot[k] = on ? a.slots[t0 + tl[k]] : -1;
        const uint32_t h = quot(w[k], a.hwords);
        wd[k] = w[k] - h * a.hwords.d;
        const T *r = x + (t0 + tl[k]) * xt + (int64_t)h * xh;
        own[k].load(r + 8 * wd[k]);
        if (ROT == 1 && !isv) {
            const int d = 8 * (int)wd[k];
            other[k].load(r + (d < half ? d + half : (d < 2 * half ? d - half : d)));
        }
    }
    double *sn64 = cs64 + a.TB * half;
    if (rot) {
        for (int e = tid; e < nt * half; e += 256) {
            const int l = e / half, i = e - l * half;
            const double turns = (double)a.pos[t0 + l] * (a.freq[i] * kInv2Pi);
            double s, c;
            sincospi(2.0 * (turns - rint(turns)), &s, &c);
            cs64[e] = c * (double)a.mscale;
            sn64[e] = s * (double)a.mscale;
        }
        __syncthreads();
    }
#pragma unroll
    for (int k = 0; k < WPT; ++k) {
        if ((uint64_t)slot[k] >= (uint64_t)a.nslots) continue;
        const int d0 = 8 * (int)wd[k];
        uint32_t word, byte;
        if (rot) {
            double v[8];
            const double *c = cs64 + tl[k] * half, *s = sn64 + tl[k] * half;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int d = d0 + i;
                const double p = (double)own[k].get(i);
                v[i] = p;
                if (d >= 2 * half) continue;
                if constexpr (ROT == 2) {
                    const double q = (double)own[k].get(i ^ 1);
                    v[i] = i & 1 ? p * c[d >> 1] + q * s[d >> 1] : p * c[d >> 1] - q * s[d >> 1];
                } else {
                    const bool first = d < half;
                    const int j = first ? d : d - half;
                    double q;
                    if constexpr (ROT == 1) {
                        q = (double)other[k].get(i);
                    } else {
                        const uint32_t h = quot(w[k], a.hwords);
                        q = (double)load1<T>(x + (t0 + tl[k]) * xt + (int64_t)h * xh + (first ? d + half : d - half));
                    }
                    v[i] = first ? p * c[j] - q * s[j] : p * c[j] + q * s[j];
                }
            }
            word = pack8_f64(v, byte);
        } else {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = own[k].get(i);
            word = (uint32_t)quantize_pack8(v, 4, byte);
        }
        const int64_t cw = slot[k] * a.words.d + w[k];    // word of the pool
        reinterpret_cast<uint32_t *>(codes)[cw] = word;
        if ((w[k] & 3) == 0) scales[cw >> 2] = (uint8_t)byte;
    }
}

template <typename T, bool VEC, int ROT>
hipError_t append_go(AppendArgs a, hipStream_t st) {
    // One word a thread until the chip is full four times over, then four. Graph
    // replays at 8 heads of 128 bf16, one against four words: 8 tokens 2.3 against
    // 3.1 us (rotated 3.2, 6.9), 4096 tokens 5.3, 5.5 (8.6, 9.6), 8192 9.6, 8.7
    // (15.3, 16.0), 16384 (27.6, 28.0), 32768 31.4, 29.0 (52.4, 51.5). The border is
    // the unrotated call's; a rotated one would gain up to 4 % between 8192 and
    // 16384 tokens by a later one. Whole tokens to a workgroup (and
    // their cosines and sines in LDS, 16 bytes a token and pair), or a chunk of one.
    const int64_t words = a.words.d;
    const int wpt = 2 * a.T * words < 4 * 256 * 2048 ? 1 : 4;
    int64_t tb = 256 * wpt / words;
    const int64_t cap = ROT ? 2048 / a.half : tb;
    tb = tb > cap ? cap : tb;
    a.TB = (int)(tb < 1 ? 1 : tb);
    a.chunk = div16((uint32_t)(words < 256 * wpt ? words : 256 * wpt));
    const dim3 grid((unsigned)ceil_div(a.T, (int64_t)a.TB), 2, (unsigned)ceil_div(words, (int64_t)a.chunk.d));
    const size_t lds = ROT ? (size_t)a.TB * a.half * 16 : 0;
    if (wpt == 1) hipLaunchKernelGGL((k_kv4_append<T, VEC, ROT, 1>), grid, dim3(256), lds, st, a);
    else hipLaunchKernelGGL((k_kv4_append<T, VEC, ROT, 4>), grid, dim3(256), lds, st, a);
    return hipGetLastError();
}

template <typename T>
hipError_t append_type(const AppendArgs &a, bool vec, int rot, hipStream_t st) {
    switch (rot) {
        case 0: return vec ? append_go<T, true, 0>(a, st) : append_go<T, false, 0>(a, st);
        case 1: return vec ? append_go<T, true, 1>(a, st) : append_go<T, false, 1>(a, st);
        case 2: return vec ? append_go<T, true, 2>(a, st) : append_go<T, false, 2>(a, st);
        default: return vec ? append_go<T, true, 3>(a, st) : append_go<T, false, 3>(a, st);
    }
}

// ---------------------------------------------------------------------- read
struct ReadArgs {
    const uint8_t *kc, *ks, *vc, *vs;
    const int64_t *slots;
    void *k, *v;
    int64_t T, kt, kh, vt, vh, nslots;
    int TB;
    Div16 words, hwords, chunk;
};

// Bound by the writes: 65536 rows of 8 heads of 128 bf16 take 60 us cold (5.6
// TB/s), 32768 rows 28 us when the caches hold part of them; 32768 rows of fp32 78.
// A thread takes WPT words (8 values each); all its codes and scales are loaded
// before the first is widened
template <typename T, bool VEC, int WPT>
__global__ __launch_bounds__(256) void k_kv4_read(ReadArgs a) {
    const bool isv = a.k == nullptr || blockIdx.y != 0;
    const uint32_t *codes = reinterpret_cast<const uint32_t *>(isv ? a.vc : a.kc);
    const uint8_t *scales = isv ? a.vs : a.ks;
    T *y = static_cast<T *>(isv ? a.v : a.k);
    const int64_t yt = isv ? a.vt : a.kt, yh = isv ? a.vh : a.kh;
    const int64_t t0 = (int64_t)blockIdx.x * a.TB;
    const int nt = a.T - t0 < a.TB ? (int)(a.T - t0) : a.TB;
    const uint32_t w0 = blockIdx.z * a.chunk.d;
    int64_t slot[WPT];
    uint32_t tl[WPT], w[WPT], c[WPT], b[WPT];
#pragma unroll
    for (int k = 0; k < WPT; ++k) {
        const uint32_t e = threadIdx.x + 256u * k;
        tl[k] = quot(e, a.chunk);
        w[k] = w0 + e - tl[k] * a.chunk.d;
        const bool on = tl[k] < (uint32_t)nt && w[k] < a.words.d;
        if (!on) {
            tl[k] = 0;
            w[k] = w0;
        }
        slot[k] = on ? a.slots[t0 + tl[k]] : -1;
    }
#pragma unroll
    for (int k = 0; k < WPT; ++k) {
        const int64_t cw = ((uint64_t)slot[k] < (uint64_t)a.nslots ? slot[k] : 0) * a.words.d + w[k];
        c[k] = codes[cw];
        b[k] = scales[cw >> 2];
    }
#pragma unroll
    for (int k = 0; k < WPT; ++k) {
        if ((uint64_t)slot[k] >= (uint64_t)a.nslots) continue;
        const uint32_t h = quot(w[k], a.hwords), wd = w[k] - h * a.hwords.d;
        // a marked block is NaN whatever its codes (Inf would do for zeros only)
        const float s = b[k] == 0xFFu ? NAN : e8m0_to_f32(b[k]);
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = (float)((int32_t)(c[k] << (28 - 4 * i)) >> 28) * s;
        T *r = y + (t0 + tl[k]) * yt + (int64_t)h * yh + 8 * wd;
        if constexpr (VEC) {
            put<T, 16 / sizeof(T)>(r, f);
            if constexpr (sizeof(T) == 4) put<T, 4>(r + 4, f + 4);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) put<T, 1>(r + i, f + i);
        }
    }
}

template <typename T>
hipError_t read_type(ReadArgs a, bool vec, hipStream_t st) {
    const int64_t words = a.words.d;
    // as in append_go; one against four words: 8 tokens 2.3 against 2.9 us, 4096
    // 5.8, 6.0, 8192 9.2, 9.0, 16384 16.2, 15.3
    const int wpt = 2 * a.T * words < 4 * 256 * 2048 ? 1 : 4;
    const int64_t tb = 256 * wpt / words;
    a.TB = (int)(tb < 1 ? 1 : tb);
    a.chunk = div16((uint32_t)(words < 256 * wpt ? words : 256 * wpt));
    const dim3 grid((unsigned)ceil_div(a.T, (int64_t)a.TB), a.k && a.v ? 2 : 1,
                    (unsigned)ceil_div(words, (int64_t)a.chunk.d));
    if (wpt == 1) {
        if (vec) hipLaunchKernelGGL((k_kv4_read<T, true, 1>), grid, dim3(256), 0, st, a);
        else hipLaunchKernelGGL((k_kv4_read<T, false, 1>), grid, dim3(256), 0, st, a);
    } else {
        if (vec) hipLaunchKernelGGL((k_kv4_read<T, true, 4>), grid, dim3(256), 0, st, a);
        else hipLaunchKernelGGL((k_kv4_read<T, false, 4>), grid, dim3(256), 0, st, a);
    }
    return hipGetLastError();
}

bool rows16(const void *p, int64_t a, int64_t b, int es) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && a * es % 16 == 0 && b * es % 16 == 0;
}

}  // namespace

void rope_frequencies(int32_t rot, double base, int32_t scaling, double factor, double low, double high,
                      double original_length, double *freq) {
    if (scaling == MXS_ROPE_NTK) base *= pow(factor, (double)rot / (rot - 2));
    for (int32_t i = 0; i < rot / 2; ++i) {
        double f = pow(base, -2.0 * i / rot);
        if (scaling == MXS_ROPE_LINEAR) f /= factor;
        if (scaling == MXS_ROPE_PARTS) {
            double k = (original_length * f * kInv2Pi - low) / (high - low);
            k = k < 0 ? 0 : (k > 1 ? 1 : k);
            f *= k + (1 - k) / factor;
        }
        freq[i] = f;
    }
}

hipError_t launch_rope(const void *x, mxs_dtype dt, int64_t T, int64_t H, int64_t D, int64_t ldt, int64_t ldh,
                       const int64_t *positions, const double *freq, int32_t rot, int32_t layout, float mscale,
                       void *y, int64_t ldyt, int64_t ldyh, hipStream_t st) {
    RopeArgs a{};
    a.x = x; a.y = y; a.T = T; a.xt = ldt; a.xh = ldh; a.yt = ldyt; a.yh = ldyh;
    a.pos = positions; a.freq = freq; a.H = (int)H; a.D = (int)D; a.half = rot / 2; a.mscale = mscale;
    const int es = dt == MXS_BF16 ? 2 : 4, V = 16 / es;
    const bool pairs = layout == MXS_ROPE_PAIRS;
    // 16-byte accesses: aligned rows, and whole vectors in both halves and in the rest of the head
    const bool vec = rows16(x, ldt, ldh, es) && rows16(y, ldyt, ldyh, es) && (rot / 2) % V == 0 && (D - rot) % V == 0;
    return dt == MXS_BF16 ? rope_type<uint16_t>(a, vec, pairs, st) : rope_type<float>(a, vec, pairs, st);
}

hipError_t launch_kv4_append(const mxs_kv4_cache &c, const void *k, const void *v, mxs_dtype dt, int64_t T,
                             int64_t ldkt, int64_t ldkh, int64_t ldvt, int64_t ldvh, const int64_t *slots,
                             const int64_t *positions, const double *freq, int32_t rot, int32_t layout,
                             float mscale, hipStream_t st) {
    AppendArgs a{};
    a.k = k; a.v = v; a.T = T; a.kt = ldkt; a.kh = ldkh; a.vt = ldvt; a.vh = ldvh;
    a.slots = slots; a.pos = positions; a.freq = freq;
    a.kc = c.kc; a.ks = c.ks; a.vc = c.vc; a.vs = c.vs;
    a.nslots = c.pages * c.page_size;
    a.H = c.H; a.D = c.D; a.half = positions ? rot / 2 : 0; a.mscale = mscale;
    a.words = div16(c.H * (c.D / 8));
    a.hwords = div16(c.D / 8);
    const int es = dt == MXS_BF16 ? 2 : 4;
    const bool vec = rows16(k, ldkt, ldkh, es) && rows16(v, ldvt, ldvh, es);
    const int r = a.half == 0 ? 0 : (layout == MXS_ROPE_PAIRS ? 2 : (a.half % 8 == 0 ? 1 : 3));
    return dt == MXS_BF16 ? append_type<uint16_t>(a, vec, r, st) : append_type<float>(a, vec, r, st);
}

hipError_t launch_kv4_read(const mxs_kv4_cache &c, const int64_t *slots, int64_t T, mxs_dtype dt, void *k,
                           int64_t ldkt, int64_t ldkh, void *v, int64_t ldvt, int64_t ldvh, hipStream_t st) {
    ReadArgs a{};
    a.kc = c.kc; a.ks = c.ks; a.vc = c.vc; a.vs = c.vs; a.slots = slots; a.k = k; a.v = v; a.T = T;
    a.kt = ldkt; a.kh = ldkh; a.vt = ldvt; a.vh = ldvh; a.nslots = c.pages * c.page_size;
    a.words = div16(c.H * (c.D / 8));
    a.hwords = div16(c.D / 8);
    const int es = dt == MXS_BF16 ? 2 : 4;
    const bool vec = (!k || rows16(k, ldkt, ldkh, es)) && (!v || rows16(v, ldvt, ldvh, es));
    return dt == MXS_BF16 ? read_type<uint16_t>(a, vec, st) : read_type<float>(a, vec, st);
}

}  // namespace mxs
