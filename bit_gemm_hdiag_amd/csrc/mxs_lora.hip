// mxs_lora.hip -- low-rank adapters of many requests beside a shared projection.
//
//     Y[t] += scale[a] B[a] (A[a] X[t]),  a = ids[t].
//
// Rows of one adapter are taken together, up to 64 a tile. The first kernel forms
// V = A X for a tile and a slice of K (partial sums, a slice each), the second adds
// the slices in order and Y += scale B V. Both are products of 16 x 16 tiles on the
// matrix cores: the rows of the adapter are the rows of a tile, tokens its columns,
// so that a lane ends with four consecutive elements of one token. A column of a
// tile depends on its own token alone: columns past a group's end repeat one of
// its tokens and are not stored, and where a token sits does not change its value.
//
// Bound by memory: the adapters' bytes for few rows (64 rows on 32 adapters of rank
// 64, 28672 x 8192: 16 + 48 us for 33 + 132 MB, half of the copy rate: each workgroup
// waits for its rows, then V, then B; B alone takes 34 us), X and Y for prompts (4096 rows
// of 8192 x 8192 at rank 16: 24 us for 67 MB of X, 68 for 268 MB of Y, 3.9 TB/s). 8 rows
// on 4 adapters take 3.6 + 5.6 us, mostly latency.
#include "mxs_device.h"
#include "mxs_internal.h"

namespace mxs {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kTile = 64;               // tokens of a tile
constexpr int kSmall = 64;              // up to so many rows every workgroup finds its group by itself

struct Tile {
    int32_t adapter, start, count;
};

struct LoraArgs {
    const void *X, *A, *B;
    const int32_t *ids, *rank;
    const float *scale;
    float *Y, *V;                       // V: [splits, M, Rp] partial sums
    int64_t M, K, N, ldx, ldy;
    int n, R, Rp;                       // adapters, stored rank, rank rounded up to 16
    int splits;
    int64_t kper;                       // K of a slice
    int64_t nper;                       // columns of Y a workgroup takes (a multiple of 64)
    int32_t *order;                     // rows by adapter
    Tile *tiles;
    int32_t *ntiles;
};

// ----------------------------------------------------------------- the groups
// cnt[id] before this row is added. The rows of a prompt have one id: lanes that
// all have the same are added by one of them (64 additions to one place take turns).
__device__ __forceinline__ int count_rows(int32_t *cnt, int32_t id) {
    const uint64_t on = __ballot(1), same = __ballot(__builtin_amdgcn_readfirstlane(id) == id);
    if (same == on) {
        const int lane = threadIdx.x & 63, before = __popcll(on & ((1ull << lane) - 1));
        int at = 0;
        if (before == 0) at = atomicAdd(&cnt[id], __popcll(on));
        return __builtin_amdgcn_readfirstlane(at) + before;
    }
    return atomicAdd(&cnt[id], 1);
}

// One workgroup: rows counted by adapter, adapters cut into tiles, rows put in
// place. The order of the rows of one adapter is left to the atomics: no value
// depends on it.
__global__ __launch_bounds__(1024) void k_lora_group(LoraArgs a) {
    extern __shared__ int32_t cnt[];    // [n] counts, then the next place of each adapter
    __shared__ int rows_of[16], tiles_of[16];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    for (int i = tid; i < a.n; i += 1024) cnt[i] = 0;
    __syncthreads();
    // 4096 rows at a time: one wait for their ids
    for (int64_t t0 = tid; t0 < a.M; t0 += 4096) {
        int32_t id[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) id[k] = t0 + 1024 * k < a.M ? a.ids[t0 + 1024 * k] : -1;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if ((uint32_t)id[k] < (uint32_t)a.n) count_rows(cnt, id[k]);
    }
    __syncthreads();
    const int per = (a.n + 1023) / 1024;
    int rows = 0, tiles = 0;
    for (int i = tid * per; i < (tid + 1) * per && i < a.n; ++i) {
        rows += cnt[i];
        tiles += (cnt[i] + kTile - 1) / kTile;
    }
    int r = rows, s = tiles;            // inclusive sums over the lanes
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int y = __shfl_up(r, o), z = __shfl_up(s, o);
        if (lane >= o) {
            r += y;
            s += z;
        }
    }
    if (lane == 63) {
        rows_of[wave] = r;
        tiles_of[wave] = s;
    }
    __syncthreads();
    r -= rows;
    s -= tiles;
    for (int w = 0; w < wave; ++w) {
        r += rows_of[w];
        s += tiles_of[w];
    }
    for (int i = tid * per; i < (tid + 1) * per && i < a.n; ++i) {
        const int c = cnt[i];
        cnt[i] = r;
        for (int k = 0; k < c; k += kTile) a.tiles[s++] = Tile{i, r + k, c - k < kTile ? c - k : kTile};
        r += c;
    }
    if (tid == 1023) *a.ntiles = s;
    __syncthreads();
    for (int64_t t0 = tid; t0 < a.M; t0 += 4096) {
        int32_t id[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) id[k] = t0 + 1024 * k < a.M ? a.ids[t0 + 1024 * k] : -1;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if ((uint32_t)id[k] < (uint32_t)a.n) a.order[count_rows(cnt, id[k])] = (int32_t)(t0 + 1024 * k);
    }
}

// The group of this workgroup: its adapter, the number of its rows, and the rows
// themselves in LDS (places past the count repeat the first). Few rows: workgroup
// i takes the rows of row i's adapter if no earlier row has it.
__device__ __forceinline__ bool find_group(const LoraArgs &a, bool small, int32_t *rows, int &adapter, int &count) {
    const int lane = threadIdx.x & 63, i = blockIdx.x;
    if (small) {
        const int32_t id = lane < a.M ? a.ids[lane] : -1;
        adapter = __shfl(id, i);
        if ((uint32_t)adapter >= (uint32_t)a.n) return false;
        const uint64_t same = __ballot(id == adapter);
        if (__ffsll((long long)same) - 1 != i) return false;
        count = __popcll(same);
        if (threadIdx.x < 64) {
            rows[lane] = i;
            __builtin_amdgcn_wave_barrier();
            if (id == adapter) rows[__popcll(same & ((1ull << lane) - 1))] = lane;
        }
    } else {
        if (i >= *a.ntiles) return false;
        const Tile t = a.tiles[i];
        adapter = t.adapter;
        count = t.count;
        if (threadIdx.x < 64) rows[lane] = a.order[t.start + (lane < count ? lane : 0)];
    }
    __syncthreads();
    return true;
}

__device__ __forceinline__ int rank_of(const LoraArgs &a, int adapter) {
    if (!a.rank) return a.R;
    const int r = a.rank[adapter];
    return r < 0 ? 0 : (r > a.R ? a.R : r);
}

// 16 bytes of a row: K 8 of a 32-deep bf16 step, 4 of a 16-deep fp32 step
template <typename T>
__device__ __forceinline__ u32x4 load16(const T *p) {
    u32x4 v;
    __builtin_memcpy(&v, p, 16);
    return v;
}

template <typename T>
__device__ __forceinline__ f32x4 mma(u32x4 a, u32x4 b, f32x4 c) {
    if constexpr (sizeof(T) == 2) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c,
                                                       0, 0, 0);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a[j]), __uint_as_float(b[j]), c, 0, 0, 0);
        return c;
    }
}

// ---------------------------------------------------------------- V = A X
// NT tiles of 16 ranks by TT tiles of 16 tokens a wave; the four waves of a
// workgroup share the slice of K and add their sums in LDS in their order. X and A
// go from memory to the matrix cores' operands directly (both have K adjacent), the
// loads of 128 K (64 in fp32) of a wave before the first is used.
template <typename T, int NT, int TT>
__device__ __forceinline__ void shrink(const LoraArgs &a, const int32_t *rows, int adapter, int count, int rank,
                                       int r0, int t0, float *lds) {
    constexpr int E = 16 / sizeof(T), STEP = 4 * E;         // elements of a lane and of a step
    constexpr int U = 4;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = lane & 15, g = lane >> 4;
    const T *x[TT], *w[NT];
#pragma unroll
    for (int t = 0; t < TT; ++t)
        x[t] = static_cast<const T *>(a.X) + (int64_t)rows[t0 + 16 * t + col] * a.ldx + E * g;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        int r = r0 + 16 * t + col;
        r = r < rank ? r : rank - 1;
        w[t] = static_cast<const T *>(a.A) + ((int64_t)adapter * a.R + r) * a.K + E * g;
    }
    f32x4 acc[NT][TT];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int t = 0; t < TT; ++t) acc[i][t] = f32x4{0, 0, 0, 0};
    const int64_t k0 = (int64_t)blockIdx.y * a.kper, k1 = k0 + a.kper < a.K ? k0 + a.kper : a.K;
    int64_t k = k0 + (int64_t)wave * (U * STEP);
    for (; k + U * STEP <= k1; k += 4 * U * STEP) {
        u32x4 xv[U][TT], wv[U][NT];
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int t = 0; t < TT; ++t) xv[u][t] = load16(x[t] + k + u * STEP);
#pragma unroll
            for (int t = 0; t < NT; ++t) wv[u][t] = load16(w[t] + k + u * STEP);
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int t = 0; t < TT; ++t) acc[i][t] = mma<T>(wv[u][i], xv[u][t], acc[i][t]);
    }
    for (; k < k1; k += STEP) {                             // the end of K, less than a wave's share
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const u32x4 wv = load16(w[i] + k);
#pragma unroll
            for (int t = 0; t < TT; ++t) acc[i][t] = mma<T>(wv, load16(x[t] + k), acc[i][t]);
        }
    }
    // [wave][token][rank of this workgroup], added in the order of the waves
    constexpr int W = 16 * NT + 4, S = 16 * TT * W;
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int t = 0; t < TT; ++t)
            *reinterpret_cast<f32x4 *>(lds + wave * S + (16 * t + col) * W + 16 * i + 4 * g) = acc[i][t];
    __syncthreads();
    float *out = a.V + (int64_t)blockIdx.y * a.M * a.Rp;
    const int there = count - t0 < 16 * TT ? count - t0 : 16 * TT;
    for (int e = threadIdx.x; e < there * 4 * NT; e += 256) {
        const int t = e / (4 * NT), q = e - t * (4 * NT), r = r0 + 4 * q;
        if (r >= a.Rp) continue;
        f32x4 v = *reinterpret_cast<const f32x4 *>(lds + t * W + 4 * q);
#pragma unroll
        for (int k = 1; k < 4; ++k) v += *reinterpret_cast<const f32x4 *>(lds + k * S + t * W + 4 * q);
        *reinterpret_cast<f32x4 *>(out + (int64_t)rows[t0 + t] * a.Rp + r) = v;
    }
}

// A workgroup takes 32 tokens of a tile (blockIdx.z: which, and which ranks): with 64
// registers leave two waves a SIMD at ranks above 32, and 301 fp32 rows of 4096 take 8.8
// instead of 7.2 us, prompts of 4096 rows 25.5 instead of 24.0
template <typename T, int NT>
__global__ __launch_bounds__(256) void k_lora_shrink(LoraArgs a, bool small) {
    __shared__ __attribute__((aligned(16))) float lds[4 * 32 * (16 * NT + 4)];
    __shared__ int32_t rows[kTile];
    int adapter, count;
    if (!find_group(a, small, rows, adapter, count)) return;
    const int rank = rank_of(a, adapter), r0 = (blockIdx.z >> 1) * 16 * NT, t0 = 32 * (blockIdx.z & 1);
    if (r0 >= rank || t0 >= count) return;
    if (count - t0 <= 16) shrink<T, NT, 1>(a, rows, adapter, count, rank, r0, t0, lds);
    else shrink<T, NT, 2>(a, rows, adapter, count, rank, r0, t0, lds);
}

// ------------------------------------------------------------ Y += scale B V
// Parts of V in LDS: [part][token][place]. bf16: the three bf16 numbers that
// add up to an fp32 one, places of ranks rounded up to 32; fp32: itself, to 16.
template <typename T>
struct Parts {
    static constexpr int P = sizeof(T) == 2 ? 3 : 1;
    static constexpr int D = sizeof(T) == 2 ? 32 : 16;      // ranks of a step
    static constexpr int E = 16 / sizeof(T);
};

// Elements r0 .. r0 + E - 1 of a row of B; zeros from the rank on
template <typename T>
__device__ __forceinline__ u32x4 load_b(const T *row, int r0, int rank) {
    constexpr int E = 16 / sizeof(T);
    u32x4 v = {0, 0, 0, 0};
    if (r0 + E <= rank) return load16(row + r0);
    if (r0 < rank) {
        T e[E];
#pragma unroll
        for (int j = 0; j < E; ++j) e[j] = r0 + j < rank ? row[r0 + j] : T(0);
        __builtin_memcpy(&v, e, 16);
    }
    return v;
}

// Eight bf16 numbers, the infinities among them 0
__device__ __forceinline__ u32x4 without_infinities(u32x4 b) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t u = b[j];
        b[j] = ((u & 0x7FFFu) == 0x7F80u ? 0u : u & 0xFFFFu) | ((u & 0x7FFF0000u) == 0x7F800000u ? 0u : u & 0xFFFF0000u);
    }
    return b;
}

// A wave takes CT tiles of 16 columns at a time: their rows of B are loaded before
// anything waits, then V's parts are read from LDS once for all of them, while
// the next 16 tokens' part of Y is on its way.
template <typename T, int STEPS, int CT>
struct Columns {
    u32x4 b[CT][STEPS];
    __device__ __forceinline__ void load(const LoraArgs &a, int64_t c, int adapter, int rank) {
        const int lane = threadIdx.x & 63, col = lane & 15, g = lane >> 4;
#pragma unroll
        for (int i = 0; i < CT; ++i) {
            const int64_t n = c + 16 * i + col < a.N ? c + 16 * i + col : a.N - 1;
            const T *row = static_cast<const T *>(a.B) + ((int64_t)adapter * a.N + n) * a.R;
#pragma unroll
            for (int s = 0; s < STEPS; ++s) b[i][s] = load_b<T>(row, s * Parts<T>::D + Parts<T>::E * g, rank);
        }
    }
};

template <int CT>
__device__ __forceinline__ void load_y(const float *y, int64_t left, f32x4 v[CT]) {
#pragma unroll
    for (int i = 0; i < CT; ++i) {
        if (left >= 16 * i + 4) {
            __builtin_memcpy(&v[i], y + 16 * i, 16);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) v[i][j] = 16 * i + j < left ? y[16 * i + j] : 0.f;
        }
    }
}
template <int CT>
__device__ __forceinline__ void store_y(float *y, int64_t left, const f32x4 v[CT]) {
#pragma unroll
    for (int i = 0; i < CT; ++i) {
        if (left >= 16 * i + 4) {
            __builtin_memcpy(y + 16 * i, &v[i], 16);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (16 * i + j < left) y[16 * i + j] = v[i][j];
        }
    }
}

// One column tile of 16 tokens: B's infinities meet every part of V, or the first alone
template <typename T, int STEPS, bool FIRST>
__device__ __forceinline__ f32x4 tile_sum(Columns<T, STEPS, 1> b, const T *v0) {
    constexpr int P = Parts<T>::P, D = Parts<T>::D, W = STEPS * D + Parts<T>::E;
    f32x4 acc = {0, 0, 0, 0};
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
#pragma unroll
        for (int q = 0; q < P; ++q)
            acc = mma<T>(FIRST && q ? without_infinities(b.b[0][s]) : b.b[0][s],
                         *reinterpret_cast<const u32x4 *>(v0 + q * kTile * W + s * D), acc);
    return acc;
}

template <typename T, int STEPS, int CT>
struct Expand {
    Columns<T, STEPS, CT> w;
    f32x4 y[CT], later[CT];
    // the rows of B and the first 16 tokens' part of Y at columns c
    __device__ __forceinline__ void load(const LoraArgs &a, const int32_t *rows, int adapter, int count, int rank, int64_t c) {
        const int lane = threadIdx.x & 63, col = lane & 15, g = lane >> 4;
        w.load(a, c, adapter, rank);
        if (col < count) load_y<CT>(a.Y + (int64_t)rows[col] * a.ldy + c + 4 * g, a.N - c - 4 * g, later);
    }
    __device__ __forceinline__ void run(const LoraArgs &a, const T *parts, const int32_t *rows, int adapter, int count,
                                        int rank, float scale, int64_t c, int64_t c1) {
        constexpr int P = Parts<T>::P, D = Parts<T>::D, E = Parts<T>::E, W = STEPS * D + E;
        const int lane = threadIdx.x & 63, col = lane & 15, g = lane >> 4;
        const int64_t first = c;
        bool left_out = false;
        for (; c < c1; c += 64 * CT) {
            const int64_t at = c + 4 * g, left = a.N - at;
            auto row = [&](int t) { return a.Y + (int64_t)rows[t + col] * a.ldy + at; };
#pragma unroll 1
            for (int t = 0; t < count; t += 16) {
#pragma unroll
                for (int i = 0; i < CT; ++i) y[i] = later[i];
                if (t + 16 + col < count) load_y<CT>(row(t + 16), left, later);
                f32x4 acc[CT];
#pragma unroll
                for (int i = 0; i < CT; ++i) acc[i] = f32x4{0, 0, 0, 0};
#pragma unroll
                for (int s = 0; s < STEPS; ++s)
#pragma unroll
                    for (int q = 0; q < P; ++q) {
                        const u32x4 v = *reinterpret_cast<const u32x4 *>(parts + (q * kTile + t + col) * W + s * D + E * g);
#pragma unroll
                        for (int i = 0; i < CT; ++i) acc[i] = mma<T>(w.b[i][s], v, acc[i]);
                    }
                if (t + 16 >= count && c + 64 * CT < c1) load(a, rows, adapter, count, rank, c + 64 * CT);
                const bool nan = P > 1 && is_nan(acc);
                left_out |= nan;
                if (t + col < count && !nan) {
#pragma unroll
                    for (int i = 0; i < CT; ++i) y[i] += scale * acc[i];
                    store_y<CT>(row(t), left, y);
                }
            }
        }
        if (P > 1 && __ballot(left_out)) rest(a, parts, rows, adapter, count, rank, scale, first, c1);
    }
    __device__ static __forceinline__ bool is_nan(const f32x4 acc[CT]) {
        bool nan = false;
#pragma unroll
        for (int i = 0; i < CT; ++i)
            nan |= __builtin_isunordered(acc[i][0], acc[i][1]) || __builtin_isunordered(acc[i][2], acc[i][3]);
        return nan;
    }
    // What run() left out: lanes whose sums came out as NaN. An infinity of B meets a number
    // as its first part only here: the others may be 0, and their product with it NaN.
    __device__ static __forceinline__ void rest(const LoraArgs &a, const T *parts, const int32_t *rows, int adapter,
                                                int count, int rank, float scale, int64_t c, int64_t c1) {
        constexpr int W = STEPS * Parts<T>::D + Parts<T>::E;
        const int lane = threadIdx.x & 63, col = lane & 15, g = lane >> 4;
        Columns<T, STEPS, 1> b;
#pragma unroll 1
        for (; c < c1; c += 64 * CT) {
#pragma unroll 1
            for (int t = 0; t < count; t += 16) {
                const T *v0 = parts + (t + col) * W + Parts<T>::E * g;
                bool nan = false;
#pragma unroll 1
                for (int i = 0; i < CT; ++i) {
                    b.load(a, c + 16 * i, adapter, rank);
                    const f32x4 v = tile_sum<T, STEPS, false>(b, v0);
                    nan |= __builtin_isunordered(v[0], v[1]) || __builtin_isunordered(v[2], v[3]);
                }
                nan &= t + col < count;
                if (!__ballot(nan)) continue;
#pragma unroll 1
                for (int i = 0; i < CT; ++i) {
                    b.load(a, c + 16 * i, adapter, rank);
                    const f32x4 v = tile_sum<T, STEPS, true>(b, v0);
                    if (nan) {
                        const int64_t at = c + 16 * i + 4 * g;
                        float *row = a.Y + (int64_t)rows[t + col] * a.ldy + at;
                        f32x4 u[1];
                        load_y<1>(row, a.N - at, u);
                        u[0] += scale * v;
                        store_y<1>(row, a.N - at, u);
                    }
                }
            }
        }
    }
};

// Registers are kept to four waves a SIMD (three where LDS allows no more): unbounded, the
// sums go to accumulation registers and the code for infinities costs a wave (64 rows on
// 32 adapters 52 instead of 48 us, prompts of 4096 rows 76 instead of 68)
template <typename T, int STEPS, int CT>
__global__ __launch_bounds__(256, STEPS <= 2 ? 4 : 3) void k_lora_expand(LoraArgs a, bool small) {
    constexpr int P = Parts<T>::P, D = Parts<T>::D, E = Parts<T>::E, Rd = STEPS * D, W = Rd + E;
    __shared__ __attribute__((aligned(16))) T parts[P * kTile * W];      // a row's place: 16 bytes of padding
    __shared__ int32_t rows[kTile];
    int adapter, count;
    if (!find_group(a, small, rows, adapter, count)) return;
    const int rank = rank_of(a, adapter);
    if (rank == 0) return;
    const int64_t c0 = (int64_t)blockIdx.y * a.nper, c1 = c0 + a.nper < a.N ? c0 + a.nper : a.N;
    const int64_t c = c0 + 16 * CT * (threadIdx.x >> 6);
    const float scale = a.scale ? a.scale[adapter] : 1.f;
    // V, four ranks of a token at a time: the slices' sums are loaded eight together
    const int places = (count + 15) / 16 * 16;
    for (int e = threadIdx.x; e < places * (Rd / 4); e += 256) {
        const int t = e / (Rd / 4), r = 4 * (e - t * (Rd / 4));
        f32x4 v = {0, 0, 0, 0};
        if (r < rank && t < count) {
            const float *p = a.V + (int64_t)rows[t] * a.Rp + r;
            for (int s = 0; s < a.splits; s += 8) {
                f32x4 part[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    part[j] = f32x4{0, 0, 0, 0};
                    if (s + j < a.splits) part[j] = *reinterpret_cast<const f32x4 *>(p + (int64_t)(s + j) * a.M * a.Rp);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) v += part[j];
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = r + j < rank ? v[j] : 0.f;
        if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int q = 0; q < 3; ++q) {
                // cut, not rounded: no part overflows, and three of 8 bits hold all 24 (those
                // above 2^-133, the smallest bf16 number)
                uint32_t h[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    h[j] = v[j] == v[j] ? __float_as_uint(v[j]) & 0xFFFF0000u : 0x7FC00000u;
                    v[j] = __builtin_isinf(v[j]) ? 0.f : v[j] - __uint_as_float(h[j]);
                }
                *reinterpret_cast<uint2 *>(parts + (q * kTile + t) * W + r) = make_uint2(h[0] >> 16 | h[1], h[2] >> 16 | h[3]);
            }
        } else {
            *reinterpret_cast<f32x4 *>(parts + t * W + r) = v;
        }
    }
    Expand<T, STEPS, CT> x;
    if (c < c1) x.load(a, rows, adapter, count, rank, c);
    __syncthreads();
    x.run(a, parts, rows, adapter, count, rank, scale, c, c1);
}

// Column tiles of a wave (two instead of four at 33 to 64 ranks: 52 against 60 us, more waves fit)
constexpr int wide_tiles(int steps) { return steps <= 1 ? 4 : (steps <= 4 ? 2 : 1); }

struct Plan {
    bool small, wide;                   // wide: wide_tiles(steps) tiles of columns a wave, else one
    int64_t tiles;                      // at most
    int splits, nt, steps;
    int64_t kper, nper;
    size_t order, list, ntiles, V, bytes;
    int Rp;
};

Plan plan_of(int64_t M, const mxs_lora &s) {
    Plan p{};
    const int es = s.dtype == MXS_BF16 ? 2 : 4;
    p.small = M <= kSmall;
    const int64_t full = ceil_div(M, (int64_t)kTile), own = s.n < M ? s.n : M;
    p.tiles = p.small ? M : full + own;
    const int64_t busy = own > full ? own : full;           // tiles to expect
    p.Rp = (s.R + 15) / 16 * 16;
    p.nt = p.Rp <= 16 ? 1 : (p.Rp <= 32 ? 2 : 4);
    p.steps = (int)ceil_div(s.R, es == 2 ? 32 : 16);
    p.steps = p.steps <= 2 ? p.steps : (p.steps <= 4 ? 4 : 8);
    const int64_t ranks = ceil_div(p.Rp, 16 * p.nt);
    // slices of K until the chip is filled, as many as let V's partial sums stay below an
    // eighth of X (or 2 MiB) wanted at most, each whole turns of the four waves: rounded
    // down, so that there may be up to twice as many slices
    const int64_t turn = 1024 / es, turns = ceil_div(s.K, turn);
    const int64_t eighth = s.K * es / (32 * p.Rp), room = ((int64_t)1 << 19) / (M * p.Rp);
    const int64_t most = p.small ? 16 : (eighth > room ? eighth : room);
    int64_t want = ceil_div(1024, busy * ranks);
    want = want < most ? want : most;
    want = want < 1 ? 1 : (want > 64 ? 64 : want);
    p.kper = turn * (turns > want ? turns / want : 1);
    while (ceil_div(s.K, p.kper) > 128) p.kper += turn;
    p.splits = (int)ceil_div(s.K, p.kper);
    // Rows of V that a workspace has room for: M times the slices, and no fewer than any
    // smaller M takes, so that one for the largest batch serves all. The slices number less
    // than 2 want; each of these bounds does not fall as M grows: a turn a slice (at most
    // 128); twice what fills the chip (busy >= M / 64); twice `most`.
    int64_t rows = M * (turns < 128 ? turns : 128);
    auto bound = [&](int64_t r) { rows = rows < r ? rows : r; };
    if (p.small) {
        bound(32 * M);
    } else {
        const int64_t share = M * (eighth < 1 ? 1 : eighth), least = ((int64_t)1 << 19) / p.Rp;
        bound(M + 2 * 1024 * kTile / ranks);
        bound(2 * (share > least ? share : least));
    }
    // columns of Y a workgroup takes: 64 where 256 would leave the chip unfilled, else 512
    // (prompts of 4096 rows: 79 us at 256, 74 at 512, 90 at 1024; 64 rows on 32 adapters: 67,
    // 57, 55), and more from 4096 workgroups on
    p.wide = busy * ceil_div(s.N, (int64_t)256) >= 512;
    p.nper = p.wide ? 512 : 64;
    while (p.wide && p.nper < 2048 && busy * ceil_div(s.N, 2 * p.nper) >= 4096) p.nper *= 2;
    while (ceil_div(s.N, p.nper) > 65535) p.nper *= 2;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t o = at;
        at += (bytes + 255) / 256 * 256;
        return o;
    };
    p.V = take((size_t)rows * p.Rp * 4);
    if (!p.small) {
        p.order = take((size_t)M * 4);
        p.list = take((size_t)p.tiles * sizeof(Tile));
        p.ntiles = take(4);
    }
    p.bytes = at;
    return p;
}

template <typename T, int STEPS>
void go_expand(const LoraArgs &a, const Plan &p, hipStream_t st) {
    const dim3 grid((unsigned)p.tiles, (unsigned)ceil_div(a.N, p.nper));
    if (p.wide) hipLaunchKernelGGL((k_lora_expand<T, STEPS, wide_tiles(STEPS)>), grid, dim3(256), 0, st, a, p.small);
    else hipLaunchKernelGGL((k_lora_expand<T, STEPS, 1>), grid, dim3(256), 0, st, a, p.small);
}

template <typename T>
hipError_t go(LoraArgs a, const Plan &p, hipStream_t st) {
    hipError_t e;
    if (!p.small) {
        hipLaunchKernelGGL(k_lora_group, dim3(1), dim3(1024), (size_t)a.n * 4, st, a);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    // tiles of at most 32 rows have no second half
    const int halves = a.M > 32 ? 2 : 1;
    const dim3 gs((unsigned)p.tiles, (unsigned)p.splits, (unsigned)(2 * ceil_div(p.Rp, 16 * p.nt) - 2 + halves));
    if (p.nt == 1) hipLaunchKernelGGL((k_lora_shrink<T, 1>), gs, dim3(256), 0, st, a, p.small);
    else if (p.nt == 2) hipLaunchKernelGGL((k_lora_shrink<T, 2>), gs, dim3(256), 0, st, a, p.small);
    else hipLaunchKernelGGL((k_lora_shrink<T, 4>), gs, dim3(256), 0, st, a, p.small);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    switch (p.steps) {
        case 1: go_expand<T, 1>(a, p, st); break;
        case 2: go_expand<T, 2>(a, p, st); break;
        case 4: go_expand<T, 4>(a, p, st); break;
        default:                            // fp32 ranks above 64
            if constexpr (sizeof(T) == 4) go_expand<T, 8>(a, p, st);
    }
    return hipGetLastError();
}

}  // namespace

size_t lora_add_workspace(int64_t M, const mxs_lora &set) { return plan_of(M, set).bytes; }

hipError_t launch_lora_add(const void *X, int64_t M, int64_t ldx, const int32_t *ids, const mxs_lora &set, float *Y,
                           int64_t ldy, void *ws, hipStream_t st) {
    const Plan p = plan_of(M, set);
    uint8_t *w = static_cast<uint8_t *>(ws);
    LoraArgs a{};
    a.X = X; a.A = set.A; a.B = set.B; a.ids = ids; a.rank = set.rank; a.scale = set.scale;
    a.Y = Y; a.V = reinterpret_cast<float *>(w + p.V);
    a.M = M; a.K = set.K; a.N = set.N; a.ldx = ldx; a.ldy = ldy;
    a.n = set.n; a.R = set.R; a.Rp = p.Rp; a.splits = p.splits; a.kper = p.kper; a.nper = p.nper;
    a.order = reinterpret_cast<int32_t *>(w + p.order);
    a.tiles = reinterpret_cast<Tile *>(w + p.list);
    a.ntiles = reinterpret_cast<int32_t *>(w + p.ntiles);
    return set.dtype == MXS_BF16 ? go<uint16_t>(a, p, st) : go<float>(a, p, st);
}

}  // namespace mxs
