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
    int64_t kper;                       // K of a slice (a multiple of 128)
    int64_t nper;                       // columns of Y a workgroup takes (a multiple of 64)
    int32_t *order;                     // rows by adapter
    Tile *tiles;
    int32_t *ntiles;
};

// ----------------------------------------------------------------- the groups
// One workgroup: rows counted by adapter, adapters cut into tiles, rows put in
// place. The order of the rows of one adapter is left to the atomics: no value
// depends on it.
__global__ __launch_bounds__(1024) void k_lora_group(LoraArgs a) {
    extern __shared__ int32_t cnt[];    // [n] counts, then the next place of each adapter
    __shared__ int rows_of[16], tiles_of[16];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    for (int i = tid; i < a.n; i += 1024) cnt[i] = 0;
    __syncthreads();
    for (int64_t t = tid; t < a.M; t += 1024) {
        const int32_t id = a.ids[t];
        if ((uint32_t)id < (uint32_t)a.n) atomicAdd(&cnt[id], 1);
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
    for (int64_t t = tid; t < a.M; t += 1024) {
        const int32_t id = a.ids[t];
        if ((uint32_t)id < (uint32_t)a.n) a.order[atomicAdd(&cnt[id], 1)] = (int32_t)t;
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
// workgroup share the slice of K and add their sums in LDS in their order.
template <typename T, int NT, int TT>
__device__ __forceinline__ void shrink(const LoraArgs &a, const int32_t *rows, int adapter, int count, int rank,
                                       int r0, float *lds) {
    constexpr int E = 16 / sizeof(T), STEP = 4 * E;         // elements of a lane and of a step
    constexpr int U = 4;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = lane & 15, g = lane >> 4;
    const T *x[TT], *w[NT];
#pragma unroll
    for (int t = 0; t < TT; ++t)
        x[t] = static_cast<const T *>(a.X) + (int64_t)rows[16 * t + col] * a.ldx + E * g;
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
    // [token][rank of this workgroup]: one wave's sums after the other
    constexpr int W = 16 * NT + 4;
    for (int v = 0; v < 4; ++v) {
        if (wave == v) {
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int t = 0; t < TT; ++t) {
                    f32x4 *p = reinterpret_cast<f32x4 *>(lds + (16 * t + col) * W + 16 * i + 4 * g);
                    *p = v == 0 ? acc[i][t] : *p + acc[i][t];
                }
        }
        __syncthreads();
    }
    float *out = a.V + (int64_t)blockIdx.y * a.M * a.Rp;
    for (int e = threadIdx.x; e < count * 4 * NT; e += 256) {
        const int t = e / (4 * NT), q = e - t * (4 * NT), r = r0 + 4 * q;
        if (r < a.Rp)
            *reinterpret_cast<f32x4 *>(out + (int64_t)rows[t] * a.Rp + r) = *reinterpret_cast<const f32x4 *>(lds + t * W + 4 * q);
    }
}

template <typename T, int NT>
__global__ __launch_bounds__(256) void k_lora_shrink(LoraArgs a, bool small) {
    extern __shared__ __attribute__((aligned(16))) float lds[];
    __shared__ int32_t rows[kTile];
    int adapter, count;
    if (!find_group(a, small, rows, adapter, count)) return;
    const int rank = rank_of(a, adapter), r0 = blockIdx.z * 16 * NT;
    if (r0 >= rank) return;
    if (count <= 16) shrink<T, NT, 1>(a, rows, adapter, count, rank, r0, lds);
    else if (count <= 32) shrink<T, NT, 2>(a, rows, adapter, count, rank, r0, lds);
    else shrink<T, NT, 4>(a, rows, adapter, count, rank, r0, lds);
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

// Elements r0 .. r0 + E - 1 of row n of B; zeros from the rank on
template <typename T, bool VEC>
__device__ __forceinline__ u32x4 load_b(const T *row, int r0, int rank) {
    constexpr int E = 16 / sizeof(T);
    u32x4 v = {0, 0, 0, 0};
    if (r0 >= rank) return v;
    if (VEC && r0 + E <= rank) return load16(row + r0);
    T e[E];
#pragma unroll
    for (int j = 0; j < E; ++j) e[j] = r0 + j < rank ? row[r0 + j] : T(0);
    __builtin_memcpy(&v, e, 16);
    return v;
}

template <typename T, bool VECB, bool VECY>
__global__ __launch_bounds__(256) void k_lora_expand(LoraArgs a, bool small) {
    extern __shared__ __attribute__((aligned(16))) uint8_t raw[];
    __shared__ int32_t rows[kTile];
    constexpr int P = Parts<T>::P, D = Parts<T>::D, E = Parts<T>::E;
    int adapter, count;
    if (!find_group(a, small, rows, adapter, count)) return;
    const int rank = rank_of(a, adapter);
    if (rank == 0) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = lane & 15, g = lane >> 4;
    const int steps = (rank + D - 1) / D, Rd = steps * D;
    const int W = Rd + E;                                   // a row's place in LDS: 16 bytes of padding
    T *parts = reinterpret_cast<T *>(raw);
    const int subs = (count + 15) / 16;
    const float scale = a.scale ? a.scale[adapter] : 1.f;
    for (int e = threadIdx.x; e < subs * 16 * Rd; e += 256) {
        const int t = e / Rd, r = e - t * Rd;
        float v = 0.f;
        if (r < rank && t < count) {
            const float *p = a.V + (int64_t)rows[t] * a.Rp + r;
            for (int s = 0; s < a.splits; ++s) v += p[(int64_t)s * a.M * a.Rp];
        }
        if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int q = 0; q < 3; ++q) {
                // cut, not rounded: no part overflows, and three of 8 bits hold all 24
                const uint32_t h = v == v ? __float_as_uint(v) & 0xFFFF0000u : 0x7FC00000u;
                parts[(q * kTile + t) * W + r] = (uint16_t)(h >> 16);
                v = __builtin_isinf(v) ? 0.f : v - __uint_as_float(h);
            }
        } else {
            parts[t * W + r] = v;
        }
    }
    __syncthreads();
    const int64_t c0 = (int64_t)blockIdx.y * a.nper, c1 = c0 + a.nper < a.N ? c0 + a.nper : a.N;
    for (int64_t c = c0 + 16 * wave; c < c1; c += 64) {
        const int64_t n = c + col < a.N ? c + col : a.N - 1;
        const T *brow = static_cast<const T *>(a.B) + ((int64_t)adapter * a.N + n) * a.R;
        f32x4 acc[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) acc[t] = f32x4{0, 0, 0, 0};
        for (int s = 0; s < steps; ++s) {
            const u32x4 b = load_b<T, VECB>(brow, s * D + E * g, rank);
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                if (t >= subs) break;
#pragma unroll
                for (int q = 0; q < P; ++q) {
                    const u32x4 v = *reinterpret_cast<const u32x4 *>(parts + (q * kTile + 16 * t + col) * W + s * D + E * g);
                    acc[t] = mma<T>(b, v, acc[t]);
                }
            }
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const int i = 16 * t + col;
            if (i >= count) continue;
            const int64_t at = c + 4 * g;
            float *y = a.Y + (int64_t)rows[i] * a.ldy + at;
            if (VECY && at + 4 <= a.N) {
                f32x4 v = *reinterpret_cast<f32x4 *>(y);
                v += scale * acc[t];
                *reinterpret_cast<f32x4 *>(y) = v;
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (at + j < a.N) y[j] += scale * acc[t][j];
            }
        }
    }
}

struct Plan {
    bool small;
    int64_t tiles;                      // at most
    int splits, nt;
    int64_t kper, nper;
    size_t order, list, ntiles, V, bytes;
    int Rp;
};

Plan plan_of(int64_t M, const mxs_lora &s) {
    Plan p{};
    p.small = M <= kSmall;
    p.tiles = p.small ? M : ceil_div(M, (int64_t)kTile) + (s.n < M ? s.n : M);
    p.Rp = (s.R + 15) / 16 * 16;
    p.nt = p.Rp <= 16 ? 1 : (p.Rp <= 32 ? 2 : 4);
    const int64_t ranks = ceil_div(p.Rp, 16 * p.nt);
    // slices of K until the chip is busy: at least 512 of K each, few where they are read by many
    const int64_t busy = p.small ? M : ceil_div(M, (int64_t)kTile);
    int64_t want = ceil_div(512, busy * ranks), most = p.small ? 16 : 4;
    want = want < most ? want : most;
    const int64_t fit = ceil_div(s.K, 512);
    want = want < fit ? want : fit;
    want = want < 1 ? 1 : want;
    p.kper = ceil_div(ceil_div(s.K, want), 128) * 128;
    p.splits = (int)ceil_div(s.K, p.kper);
    // columns of Y: 64 and more until there are 1024 workgroups
    p.nper = 64;
    while (p.nper < 1024 && busy * ceil_div(s.N, 2 * p.nper) >= 1024) p.nper *= 2;
    while (ceil_div(s.N, p.nper) > 65535) p.nper *= 2;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t o = at;
        at += (bytes + 255) / 256 * 256;
        return o;
    };
    p.V = take((size_t)p.splits * M * p.Rp * 4);
    if (!p.small) {
        p.order = take((size_t)M * 4);
        p.list = take((size_t)p.tiles * sizeof(Tile));
        p.ntiles = take(4);
    }
    p.bytes = at;
    return p;
}

template <typename T>
hipError_t go(LoraArgs a, const Plan &p, hipStream_t st) {
    hipError_t e;
    if (!p.small) {
        hipLaunchKernelGGL(k_lora_group, dim3(1), dim3(1024), (size_t)a.n * 4, st, a);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    const dim3 gs((unsigned)p.tiles, (unsigned)p.splits, (unsigned)ceil_div(p.Rp, 16 * p.nt));
    const size_t ls = (size_t)kTile * (16 * p.nt + 4) * 4;
    if (p.nt == 1) hipLaunchKernelGGL((k_lora_shrink<T, 1>), gs, dim3(256), ls, st, a, p.small);
    else if (p.nt == 2) hipLaunchKernelGGL((k_lora_shrink<T, 2>), gs, dim3(256), ls, st, a, p.small);
    else hipLaunchKernelGGL((k_lora_shrink<T, 4>), gs, dim3(256), ls, st, a, p.small);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    constexpr int D = Parts<T>::D, E = Parts<T>::E;
    const size_t le = (size_t)Parts<T>::P * kTile * (ceil_div(a.R, D) * D + E) * sizeof(T);
    const dim3 ge((unsigned)p.tiles, (unsigned)ceil_div(a.N, p.nper));
    const bool vecb = a.R % E == 0, vecy = reinterpret_cast<uintptr_t>(a.Y) % 16 == 0 && a.ldy % 4 == 0;
    if (vecb && vecy) hipLaunchKernelGGL((k_lora_expand<T, true, true>), ge, dim3(256), le, st, a, p.small);
    else if (vecb) hipLaunchKernelGGL((k_lora_expand<T, true, false>), ge, dim3(256), le, st, a, p.small);
    else if (vecy) hipLaunchKernelGGL((k_lora_expand<T, false, true>), ge, dim3(256), le, st, a, p.small);
    else hipLaunchKernelGGL((k_lora_expand<T, false, false>), ge, dim3(256), le, st, a, p.small);
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
